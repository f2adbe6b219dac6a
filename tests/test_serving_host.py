"""Host-side checks (no GPU) of the calls around the paged cache in a serving step: invalid arguments are refused
with the documented status before anything is enqueued, and the bindings refuse tensors of other element types."""
import os
import shutil
import subprocess

import pytest

import bit_quantized_moe_q4k_gb300 as q4k

from test_attention_host import PAGED_REFUSALS

torch = pytest.importorskip("torch")

A16 = 1 << 20          # a fake 16-byte-aligned address; never dereferenced by these calls


class FakeCuda:
    """What a binding reads of a device tensor before it calls the library."""
    is_cuda = True

    def __init__(self, dtype):
        self.dtype = dtype

    def data_ptr(self):
        return A16


def tables(**kw):
    a = dict(kept=A16, new=A16, fixed=A16, batch=3, m=7, mp=4, page=16, np=8, held=A16, free=A16, count=A16, table=A16, ho=A16, co=A16,
             qs=A16, lens=A16, pos=A16, slots=A16)
    a.update(kw)
    return q4k.load().q4k_page_tables(a["kept"], a["new"], a["fixed"], a["batch"], a["m"], a["mp"], a["page"], a["np"], a["held"],
                                      a["free"], a["count"], a["table"], a["ho"], a["co"], a["qs"], a["lens"], a["pos"], a["slots"],
                                      None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 2), (dict(m=-1), 2), (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(np=0), 2), (dict(mp=0), 2),
    (dict(mp=1 << 27), 9), (dict(m=(1 << 24) + 1), 9), (dict(batch=8193), 9),
    (dict(kept=None), 1), (dict(new=None), 1), (dict(held=None), 1), (dict(free=None), 1), (dict(count=None), 1), (dict(table=None), 1),
    (dict(ho=None), 1), (dict(co=None), 1), (dict(qs=None), 1), (dict(lens=None), 1), (dict(batch=0, qs=None), 1),
    (dict(kept=A16 + 2), 7), (dict(fixed=A16 + 1), 7), (dict(table=A16 + 2), 7), (dict(pos=A16 + 2), 7), (dict(slots=A16 + 4), 7),
])
def test_tables_rejects(kw, status):
    assert tables(**kw) == status
    assert q4k.load().q4k_last_error_string()


def test_tables_binding_refuses_other_element_types():
    i32, i64, f32 = (FakeCuda(t) for t in (torch.int32, torch.int64, torch.float32))
    good = [i32, i32, i32, 3, 7, 4, 16, 8, i32, i32, i32, i32, i32, i32, i32, i32, i32, i64, i32]
    for at, x in enumerate(good):
        if isinstance(x, int):
            continue
        for other in (i32, i64, f32):
            if other.dtype == x.dtype:
                continue
            args = list(good)
            args[at] = other
            with pytest.raises(ValueError):
                q4k.q4k_page_tables(*args, stream=0)


def verify(**kw):
    a = dict(x=A16, dtype=0, m=7, v=100, xs=100, q=A16, qs=100, tok=A16, st=A16, batch=3, t=A16, ua=A16, us=A16, lens=A16, acc=A16,
             nxt=A16, kept=A16, ws=A16, wsb=None)
    a.update(kw)
    lib = q4k.load()
    if a["wsb"] is None:
        a["wsb"] = lib.q4k_verify_drafts_workspace_size(3, 7, 100)
    return lib.q4k_verify_drafts(a["x"], a["dtype"], a["m"], a["v"], a["xs"], a["q"], a["qs"], a["tok"], a["st"], a["batch"], a["t"],
                                 a["ua"], a["us"], a["lens"], a["acc"], a["nxt"], a["kept"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 13), (dict(m=-1), 2), (dict(batch=-1), 2), (dict(v=0), 2), (dict(xs=99), 2), (dict(qs=99), 2),
    (dict(m=(1 << 24) + 1), 9), (dict(batch=(1 << 24) + 1), 9), (dict(v=(1 << 20) + 1, xs=1 << 21, qs=1 << 21), 9),
    (dict(x=None), 1), (dict(tok=None), 1), (dict(st=None), 1), (dict(ua=None), 1), (dict(us=None), 1), (dict(acc=None), 1),
    (dict(nxt=None), 1), (dict(lens=None), 1), (dict(x=A16 + 2), 7), (dict(dtype=1, x=A16 + 1), 7), (dict(q=A16 + 2), 7),
    (dict(tok=A16 + 1), 7), (dict(kept=A16 + 2), 7), (dict(ws=None), 4), (dict(wsb=16), 4), (dict(ws=A16 + 16), 4),
])
def test_verify_rejects(kw, status):
    assert verify(**kw) == status
    assert q4k.load().q4k_last_error_string()


def test_verify_empty_and_workspace():
    assert verify(batch=0) == 0
    lib = q4k.load()
    assert lib.q4k_verify_drafts_workspace_size(3, 7, 50001) % 256 == 0
    for bad in ((-1, 1, 100), (1, -1, 100), (1, 1, 0), (1, 1, (1 << 20) + 1), (1, (1 << 24) + 1, 100)):
        assert lib.q4k_verify_drafts_workspace_size(*bad) == 0


def test_verify_workspace_of_the_largest_call_serves_all():
    size = q4k.load().q4k_verify_drafts_workspace_size
    for vocab in (1, 4096, 4097, 32000, 50001, 131072, 151936, 1 << 20):
        sizes = [size(1, m, vocab) for m in range(4000)] + [size(1, m, vocab) for m in (1 << 13, 1 << 20, 1 << 24)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[-1] > 0
    for m in (1, 3, 108, 109, 380, 1000):
        sizes = [size(1, m, v) for v in range(1, 1 << 18, 997)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert len({size(b, 300, 50001) for b in (0, 1, 7, 300, 1 << 24)}) == 1


def test_verify_binding_refuses_other_element_types():
    i32, i64, f32, f16, u8 = (FakeCuda(t) for t in (torch.int32, torch.int64, torch.float32, torch.float16, torch.uint8))
    good = [f32, 7, 100, 100, f32, 100, i32, i32, 3, f32, f32, f32, i32, i32, i32, i32, u8, 1 << 20, i32]
    for at, x in enumerate(good):
        if isinstance(x, int):
            continue
        for other in (i32, i64, f32, f16, u8):
            if other.dtype == x.dtype:
                continue
            args = list(good)
            args[at] = other
            with pytest.raises(ValueError):
                q4k.q4k_verify_drafts(*args, stream=0)


def prefix(**kw):
    a = dict(q=A16, dtype=0, m=3, hq=8, hk=2, d=128, qs=1024, kc=A16, vc=A16, ksc=A16, vsc=A16, qst=A16, lens=A16, table=A16, batch=2,
             mp=4, page=16, np=8, gs=A16, pl=A16, groups=1, maxq=2, maxl=64, maxp=32, scale=0.1, window=0, out=A16, os=1024, ws=A16,
             wsb=None)
    a.update(kw)
    lib = q4k.load()
    if a["wsb"] is None:
        a["wsb"] = lib.q4k_shared_prefix_attention_workspace_size(2, 1, 3, 8, 2, 128)
    return lib.q4k_shared_prefix_attention(
        a["q"], a["dtype"], a["m"], a["hq"], a["hk"], a["d"], a["qs"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["qst"], a["lens"],
        a["table"], a["batch"], a["mp"], a["page"], a["np"], a["gs"], a["pl"], a["groups"], a["maxq"], a["maxl"], a["maxp"], a["scale"],
        a["window"], a["out"], a["os"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,status", PAGED_REFUSALS + [
    (dict(hq=7), 2), (dict(hq=1), 2), (dict(maxq=-1), 2), (dict(maxl=-1), 2), (dict(window=-1), 2), (dict(qs=1022), 2),
    (dict(qs=1026), 7), (dict(os=1020), 2), (dict(q=None), 1), (dict(out=None), 1), (dict(q=A16 + 4), 7), (dict(out=A16 + 8), 7),
    (dict(ws=None), 4), (dict(wsb=1024), 4), (dict(ws=A16 + 16), 4), (dict(hq=65538, qs=1 << 24, os=1 << 24), 9),
    (dict(groups=-1), 2), (dict(maxp=-1), 2), (dict(groups=(1 << 24) + 1), 9), (dict(gs=None), 1), (dict(pl=None), 1),
    (dict(gs=A16 + 2), 7), (dict(pl=A16 + 1), 7),
])
def test_prefix_rejects(kw, status):
    assert prefix(**kw) == status
    assert q4k.load().q4k_last_error_string()


def test_prefix_empty_and_workspace():
    assert prefix(m=0) == 0
    assert prefix(batch=0) == 0
    lib = q4k.load()
    own = lib.q4k_paged_attention_workspace_size(64, 64, 32, 8, 128)
    assert lib.q4k_shared_prefix_attention_workspace_size(64, 0, 64, 32, 8, 128) == own
    some = lib.q4k_shared_prefix_attention_workspace_size(64, 1, 64, 32, 8, 128)
    assert some > own and some % 256 == 0
    # beyond 2^20 query rows nothing is shared, and no place for it is asked for
    assert lib.q4k_shared_prefix_attention_workspace_size(64, 1, (1 << 20) // 32 + 1, 32, 8, 128) == own
    for bad in ((1, 1, 1, 32, 4, 96), (1, 1, 1, 30, 4, 128), (-1, 1, 1, 32, 4, 128), (1, -1, 1, 32, 4, 128)):
        assert lib.q4k_shared_prefix_attention_workspace_size(*bad) == 0


def test_prefix_workspace_rises_with_the_call():
    size = q4k.load().q4k_shared_prefix_attention_workspace_size
    for hq, hk, d in ((32, 8, 128), (14, 2, 64), (8, 1, 128), (5, 5, 64)):
        most = (1 << 20) // hq
        for sizes in ([size(64, 3, m, hq, hk, d) for m in [*range(1, 700), 4096, most - 1, most]], [size(b, 3, 600, hq, hk, d) for b in range(1, 700)],
                      [size(300, g, 600, hq, hk, d) for g in range(1, 400)]):
            assert all(x <= y for x, y in zip(sizes, sizes[1:]))


def test_prefix_binding_refuses_other_element_types():
    f32, f8, i32, u8, f16 = (FakeCuda(t) for t in (torch.float32, torch.float8_e4m3fn, torch.int32, torch.uint8, torch.float16))
    good = [f32, 3, 8, 2, 128, 1024, f8, f8, f32, f32, i32, i32, i32, 2, 4, 16, 8, i32, i32, 1, 2, 64, 32, 0.1, 0, f32, 1024, u8, 1 << 30,
            i32]
    for at, x in enumerate(good):
        if isinstance(x, (int, float)):
            continue
        for other in (f16, f32 if x is not f32 else i32):
            args = list(good)
            args[at] = other
            with pytest.raises(ValueError):
                q4k.q4k_shared_prefix_attention(*args, stream=0)


PIECES = r"""
#include <cstdio>
#include <cstdlib>
#include "q4k_pieces.cuh"
using namespace q4k;
static long long worst = -(1LL << 60);
static void check(const int* tile, long long tiles, int kv_heads) {
    int64_t tokens = 0, pieces = 0;
    for (long long i = 0; i < tiles; ++i) tokens += tile[i];
    const int length = own_length(tokens, kv_heads);
    for (long long i = 0; i < tiles; ++i) pieces += pieces_of_tile(tile[i], length);
    const long long over = pieces - most_own_pieces(tiles, kv_heads);
    if (over > worst) worst = over;
    if (over > 0 || length < kOwnLeast || length % 32) {
        printf("kv_heads %d, %lld tiles, %lld tokens, length %d: %lld pieces too many\n", kv_heads, tiles, (long long)tokens, length, over);
        exit(1);
    }
}
int main() {
    static int tile[4096];
    const int kv[] = {1, 2, 3, 4, 5, 7, 8, 16, 24, 32, 64, 1000, 2736, 2737, 65535};
    srand(1);
    for (int h : kv)
        for (int tiles = 1; tiles <= 40; ++tiles)
            for (int k = 3; k < 40; ++k)          // equal lengths whose total is next to 32 k for each of the pieces
                for (int off = -2; off <= 40; ++off) {
                    const int64_t each = 32LL * k * kOwnPieces / h / tiles + off;
                    for (int i = 0; i < tiles; ++i) tile[i] = each < 0 ? 0 : (int)each;
                    check(tile, tiles, h);
                }
    for (int n = 0; n < 20000; ++n) {             // totals there, cut anywhere, and row tiles that see nothing
        const int h = kv[rand() % 15], tiles = 2 + rand() % 300;
        const int64_t total = 32LL * (3 + rand() % 30) * kOwnPieces / h + rand() % 600;
        int64_t left = total;
        for (int i = 0; i < tiles; ++i) {
            tile[i] = i == tiles - 1 ? (int)left : (int)(left * (rand() % 1000) / 1000 / (rand() % 8 + 1));
            left -= tile[i];
        }
        check(tile, tiles, h);
    }
    for (int h : kv) {                            // the longest rows of tables
        for (int i = 0; i < 4096; ++i) tile[i] = (1 << 30) - i % 3;
        check(tile, 4096, h);
    }
    printf("%lld\n", worst);
    return 0;
}
"""


def test_pieces_of_own_parts_have_room(tmp_path):
    """Behind shared prefixes: as many pieces as the workspace has room for, whatever the lengths."""
    compiler = shutil.which("g++")
    if not compiler:
        pytest.skip("no host compiler")
    (tmp_path / "pieces.cpp").write_text(PIECES)
    csrc = os.path.join(os.path.dirname(q4k.__file__), "csrc")
    subprocess.run([compiler, "-std=c++17", "-O2", "-I", csrc, str(tmp_path / "pieces.cpp"), "-o", str(tmp_path / "pieces")], check=True)
    r = subprocess.run([str(tmp_path / "pieces")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) >= -1   # (the cases come next to the bound)
