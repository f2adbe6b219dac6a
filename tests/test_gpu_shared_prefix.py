"""GPU tests of q4k_shared_prefix_attention against the plain fp64 attention of the same tokens, sequence by sequence.

Tolerance, per row: that of q4k_paged_attention (test_gpu_attention.py), and joining the two parts of a row, k pieces of the shared one
at a time: a weight 2^(reference - top) is off by ex2's 2^-22 and by half a step of a difference of up to 24 (2^-21 ln 2; the weight of
what is further off is below 2^-24); products, sums and the quotient of numerator and denominator by (2 k + 8) u. Each counts
twice at most, times sum_j p_j |v_j|."""
import math

import numpy as np
import pytest

import bit_quantized_moe_q4k_gb300 as q4k

from helpers import dev, err_flag, host
from test_gpu_attention import DT, U, Cache, attention_ref, f64, q_starts, rows

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TIMEOUT, PAGE_FLAG, SEQ_FLAG = 10, 11, 12


@pytest.fixture(autouse=True)
def share_whatever_can_be(monkeypatch):
    monkeypatch.setenv("Q4K_SHARE_PREFIX", "1")


class Shared:
    """groups: (shared tokens, [(new tokens, cached tokens behind the shared ones and before the new)]); before and behind: sequences
    outside the groups, the same with no shared tokens."""

    def __init__(self, seed, groups, hk, d, page, pow2=True, before=(), behind=()):
        self.groups, self.page, self.hk, self.d = groups, page, hk, d
        lone = [(0, [s]) for s in before], [(0, [s]) for s in behind]
        alls = lone[0] + list(groups) + lone[1]
        self.new = [n for _, seqs in alls for n, _ in seqs]
        self.lens = [max(p + o + n, 0) for p, seqs in alls for n, o in seqs]
        own = [[max(-(-max(p + o + n, 0) // page) - p // page, 0) for n, o in seqs] for p, seqs in alls]
        pages = sum(p // page + sum(o) for (p, _), o in zip(alls, own)) + 2
        self.cache = Cache(seed, pages, hk, page, d, pow2)
        width = max([1] + [-(-x // page) for x in self.lens] + [p // page for p, _ in alls]) + 1
        self.table = np.full((len(self.new), width), 0x7FFFFFF0, np.int32)
        at = i = 0
        for (p, _), o in zip(alls, own):
            first = self.cache.order[at:at + p // page]
            at += p // page
            for n in o:
                self.table[i, :p // page] = first
                self.table[i, p // page:p // page + n] = self.cache.order[at:at + n]
                at += n
                i += 1
        self.start = np.cumsum([len(before)] + [len(s) for _, s in groups]).astype(np.int32)
        self.prefix = np.array([p for p, _ in groups], np.int32)
        self.seed = seed

    def run(self, hq, dtype, window=0, gain=1.0, pad=0, check=True, flagged=0, hints=None, table=None, start=None, prefix=None,
            times=2, max_prefix=None, ws=None, raw_lens=None, raw_starts=None):
        g = np.random.default_rng(self.seed + 1)
        hk, d, m, b = self.hk, self.d, sum(self.new), len(self.new)
        c = self.cache
        c.upload()
        table = self.table if table is None else table
        start, prefix = self.start if start is None else start, self.prefix if prefix is None else prefix
        q = rows(g.standard_normal((m, hq * d)) * gain, dtype, hq * d + pad)
        out = torch.full((max(m, 1), hq * d + pad), 7.0, dtype=DT[dtype], device="cuda")
        nbytes = q4k.q4k_shared_prefix_attention_workspace_size(b, len(prefix), m, hq, hk, d)
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
        flag, scale = err_flag(), 1 / math.sqrt(d)
        maxq, maxl = hints or (max(self.new), max(self.lens))
        got = []
        for _ in range(times):
            q4k.q4k_shared_prefix_attention(
                q, m, hq, hk, d, hq * d + pad, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"], dev(np.asarray(raw_starts or q_starts(self.new), np.int32)),
                dev(np.array(raw_lens or self.lens, np.int32)), dev(table), b, table.shape[1], self.page, c.pages, dev(np.asarray(start, np.int32)),
                dev(np.asarray(prefix, np.int32)), len(prefix), maxq, maxl,
                int(max([0, *prefix])) if max_prefix is None else max_prefix, scale, window, out, hq * d + pad, ws, nbytes, flag)
            got.append(f64(out))
        assert int(host(flag)[0]) == flagged
        assert all(np.array_equal(x, got[0], equal_nan=True) for x in got)
        if pad:
            assert (got[0][:, hq * d:] == 7.0).all()
        got = got[0][:m, :hq * d].reshape(m, hq, d)
        if check:
            qs = f64(q)[:m, :hq * d].reshape(m, hq, d)
            ref, tol = attention_ref(qs, c, self.table, self.new, self.lens, hq // hk, scale, window, dtype)
            none, rel = attention_ref(qs, self._magnitudes(), self.table, self.new, self.lens, hq // hk, scale, window, "f32")
            pieces = 152
            tol += 2 * (2.0 ** -22 + 2.0 ** -21 * math.log(2) + (2 * pieces + 8) * U) * none
            worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-300))
            assert np.isfinite(got).all() and worst <= 1, f"{worst} of the bound"
        return got

    def _magnitudes(self):
        """The same cache with |v|: its attention is sum_j p_j |v_j|."""
        c = Cache.__new__(Cache)
        c.__dict__.update(self.cache.__dict__)
        c.codes = {"k": self.cache.codes["k"], "v": self.cache.codes["v"] & 0x7F}
        return c


def samples(n, new=1, own=7):
    return [(new, own + 3 * i) for i in range(n)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_types_and_pages(page, d, dtype):
    Shared(page + d, [(400, samples(5))], 2, d, page).run(8, dtype, pad=16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shared", [1, 15, 16, 17, 31, 32, 127, 128, 129, 144, 255, 256, 257, 1000, 3001])
def test_lengths_of_the_prefix(shared, dtype):
    Shared(shared, [(shared, samples(3, own=0))], 2, 64, 16).run(4, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 2), (3, 1), (14, 2), (16, 2), (32, 4), (16, 1), (20, 1), (8, 8)])
def test_head_groups(hq, hk, dtype):
    Shared(hq, [(300, [(1, 5), (2, 0), (3, 40)])], hk, 128, 32).run(hq, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs,new,hq,hk", [
    (2, 1, 1, 1), (31, 1, 4, 1), (32, 1, 4, 1), (33, 1, 4, 1), (64, 1, 4, 1), (65, 2, 4, 1), (100, 1, 16, 2), (40, 5, 7, 1), (130, 1, 32, 4)])
def test_rows_of_one_and_several_row_tiles(seqs, new, hq, hk, dtype):
    Shared(seqs, [(500, [(new, i % 9) for i in range(seqs)])], hk, 64, 32).run(hq, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("groups", [
    [(300, samples(3)), (0, samples(2)), (77, samples(9)), (2000, samples(2))],
    [(64, samples(1)), (64, samples(1)), (640, samples(4, 2))],
    [(200, []), (200, samples(2)), (200, [])],
    [(100 * k, samples(2 + k % 3, 1 + k % 2)) for k in range(1, 41)],
    [(900, [(0, 5), (1, 6), (0, 2), (2, 3)]), (700, [(0, 1), (0, 2)]), (800, [(0, 5), (1, 1)])],
    [(16, samples(30)), (4000, samples(2)), (17, samples(30))],
])
def test_several_groups(groups, dtype):
    Shared(len(groups), groups, 2, 64, 16).run(6, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_outside_the_groups(dtype):
    Shared(3, [(250, samples(4)), (130, samples(3))], 2, 128, 16, before=[(1, 40), (2, 0)], behind=[(1, 300), (0, 9), (3, 20)]).run(8, dtype)
    Shared(4, [], 2, 128, 16, before=[(1, 40), (2, 0)]).run(8, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 16, 33, 100, 260, 1000])
def test_windows(window, dtype):
    """Rows that see all, some and nothing of what is shared."""
    Shared(window, [(300, [(1, 0), (3, 17), (2, 120), (1, 400)]), (150, samples(3, 4))], 2, 64, 16).run(4, dtype, window)
    Shared(window, [(1300, [(1 + i % 3, 9 * i) for i in range(40)])], 1, 128, 32).run(7, dtype, window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_new_tokens_inside_the_prefix(dtype):
    """Sequences whose new tokens begin before the prefix ends: what lies before all of them is shared."""
    Shared(5, [(300, [(1, -100), (1, 20), (5, -44)])], 2, 64, 16).run(4, dtype)
    Shared(6, [(300, [(1, -300 + 0), (1, 20)])], 2, 64, 16).run(4, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_prefixes(dtype):
    Shared(7, [(20011, samples(6))], 1, 64, 64).run(4, dtype)
    Shared(8, [(9000, samples(40))], 2, 128, 128).run(8, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beside_prompts(dtype):
    """Calls that go to the prompt kernels in part: a group with a prompt reads its prefix itself, another shares it."""
    Shared(9, [(200, [(1, 0), (150, 10), (1, 5)]), (400, samples(6))], 2, 128, 32).run(64, dtype, pad=16)
    Shared(10, [(200, [(130, 0), (150, 10)])], 2, 64, 32).run(64, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scales_and_magnitudes(dtype):
    Shared(11, [(400, samples(5))], 2, 128, 16, pow2=False).run(8, dtype)
    s = Shared(12, [(400, samples(5)), (90, samples(3))], 2, 128, 16)
    s.cache.scale["v"][:] = (2.0 ** np.resize([-40.0, 0.0, 30.0, -64.0, -3.0], s.cache.scale["v"].size)).reshape(s.cache.scale["v"].shape)
    s.run(8, dtype)
    for gain in (0.0, 1e-30, 30.0):
        Shared(13, [(300, samples(40))], 2, 64, 16).run(8, dtype, gain=gain)
    assert np.isfinite(Shared(14, [(300, samples(40))], 2, 64, 16).run(8, dtype, gain=1e20, check=False)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq", [4, 32])
@pytest.mark.parametrize("window", [0, 100])
def test_nan_reaches_only_the_rows_that_see_it(window, hq, dtype):
    """NaN in one value dim, or in a key, of one token, in the shared part and behind it."""
    groups, page, hk, d, dim = [(208, [(2, 30 + 5 * i) for i in range(6)]), (100, samples(3))], 16, 2, 64, 5
    clean = Shared(15, groups, hk, d, page).run(hq, dtype, window)
    first = [sum(len(s) for _, s in groups[:k]) for k in range(2)]
    for side in "vk":
        for group, tok in ((0, 207), (0, 170), (0, 3), (1, 95), (0, 215)):
            s = Shared(15, groups, hk, d, page)
            entry = s.table[first[group], tok // page]
            s.cache.codes[side][entry, 1, tok % page, dim] = 0xFF
            got = s.run(hq, dtype, window, check=False)
            holds = [entry in s.table[i, :-(-s.lens[i] // page)] for i in range(len(s.new))]
            pos = np.concatenate([np.arange(length - n, length) for n, length in zip(s.new, s.lens)])
            holds = np.repeat(holds, s.new)
            sees = holds & (tok <= pos) & ((tok > pos - window) if window else True)
            want = np.zeros_like(clean, bool)
            want[sees, hq // hk:, dim if side == "v" else slice(None)] = True
            assert np.array_equal(np.isnan(got), want), (side, group, tok)
            assert np.array_equal(got[~sees], clean[~sees]) and np.array_equal(got[:, :hq // hk], clean[:, :hq // hk])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_in_a_query_and_in_slots_past_the_end(dtype):
    s = Shared(16, [(208, samples(5))], 2, 64, 16)
    for i, n in enumerate(s.lens):
        for side in "kv":
            s.cache.codes[side][s.table[i, (n - 1) // 16], :, (n - 1) % 16 + 1:] = 0x7F
    s.run(8, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [-1, 0x7FFFFFFF])
def test_bad_page_ids(bad, dtype):
    """In the shared part: flagged, its tokens are seen by no row of the group; the other group is right."""
    s = Shared(17, [(300, samples(4)), (300, samples(3))], 2, 64, 16)
    good = s.run(8, dtype)
    table = s.table.copy()
    table[:4, 3] = bad
    got = s.run(8, dtype, table=table, check=False, flagged=PAGE_FLAG)
    assert np.isfinite(got).all() and np.array_equal(got[4:], good[4:]) and not np.array_equal(got[:4], good[:4])
    # the tokens of page 3 carry no weight: as if the sequences had never held them
    t = Shared(17, [(300, samples(4)), (300, samples(3))], 2, 64, 16)
    t.cache.codes["v"][s.table[0, 3]] = 0x70
    t.cache.scale["v"][s.table[0, 3]] = 1e30
    assert np.array_equal(t.run(8, dtype, table=table, check=False, flagged=PAGE_FLAG), got)


@pytest.mark.parametrize("start,prefix", [([0, 3, 2, 7], [100, 100, 100]), ([-1, 3, 5, 7], [100, 100, 100]), ([0, 3, 5, 8], [100, 100, 100])])
def test_malformed_groups_share_nothing(start, prefix):
    s = Shared(18, [(100, samples(3)), (100, samples(2)), (100, samples(2))], 2, 64, 16)
    s.run(8, "f32", start=start, prefix=prefix, flagged=SEQ_FLAG)


def test_prefix_lengths_out_of_range():
    """Longer than the table's row: cut to what lies before the new tokens. Negative: nothing."""
    s = Shared(19, [(96, samples(3, own=0))], 2, 64, 16)
    s.table[1:, :6] = s.table[0, :6]
    s.run(8, "f32", prefix=[-5], max_prefix=96, flagged=SEQ_FLAG)


def test_hints_do_not_change_results_much():
    for hints in ((1, 1), (300, 100000), (0, 0)):
        Shared(20, [(400, samples(5, 2)), (90, samples(3))], 2, 64, 16).run(8, "f32", hints=hints)
        Shared(20, [(400, samples(5, 2)), (90, samples(3))], 2, 64, 16).run(8, "bf16", hints=hints)
    for most in (0, 15, 16, 1 << 29):
        Shared(21, [(400, samples(5, 2))], 2, 64, 16).run(8, "f32", max_prefix=most)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_other_streams_and_graphs(dtype):
    """The same bits on another stream; a captured call replayed as sequences grow; two graphs with workspaces of their own at once."""
    a = Shared(22, [(700, samples(9))], 2, 128, 32)
    want = a.run(8, dtype)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = a.run(8, dtype)
    torch.cuda.current_stream().wait_stream(st)
    assert np.array_equal(want, got)
    made, kept = [], []
    for k in range(2):
        s = Shared(23 + k, [(300 + 50 * k, [(1, 40)] * 6), (128, [(1, 40)] * 3)], 2, 64, 16)
        s.cache.upload()
        q = rows(np.random.default_rng(k).standard_normal((9, 8 * 64)), dtype)
        out, lens = torch.empty_like(q), dev(np.array(s.lens, np.int32) - 20)
        nbytes = q4k.q4k_shared_prefix_attention_workspace_size(9, 2, 9, 8, 2, 64)
        ws, flag = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda"), err_flag()
        fixed = [dev(q_starts(s.new)), lens, dev(s.table), dev(s.start), dev(s.prefix)]

        def call(s=s, q=q, out=out, ws=ws, nbytes=nbytes, flag=flag, f=fixed):
            c = s.cache
            q4k.q4k_shared_prefix_attention(q, 9, 8, 2, 64, 512, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"], f[0], f[1],
                                            f[2], 9, s.table.shape[1], 16, c.pages, f[3], f[4], 2, 1, 4096, 400, 0.125, 0, out, 512,
                                            ws, nbytes, flag)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        made.append((s, q, out, lens, graph, flag))
        kept.append((ws, fixed))   # a graph holds addresses only
    streams = [torch.cuda.Stream() for _ in made]
    for step in range(1, 4):
        for s, q, out, lens, graph, flag in made:
            lens.add_(1)
        torch.cuda.synchronize()
        for (s, q, out, lens, graph, flag), st in zip(made, streams):
            with torch.cuda.stream(st):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for s, q, out, lens, graph, flag in made:
            ls = host(lens).tolist()
            ref, tol = attention_ref(f64(q).reshape(9, 8, 64), s.cache, s.table, s.new, ls, 4, 0.125, 0, dtype)
            assert int(flag) == 0 and (np.abs(f64(out).reshape(9, 8, 64) - ref) <= 2 * tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("length,hk", [(3000, 2), (30000, 8)])
def test_waits_that_run_out(length, hk, dtype, monkeypatch):
    """A wait limit of nothing: the flag is raised or the call gets through (where a CTA has so few tiles that its pages are looked
    up without a wait), and the next call is right."""
    s = Shared(25, [(length, samples(40))], hk, 128, 64)
    want = s.run(8, dtype, check=False)
    for limit in (1, 100, 3000, 20000):
        monkeypatch.setenv("Q4K_WAIT_NS", str(limit))
        c, m, b = s.cache, sum(s.new), len(s.new)
        q, out = rows(np.random.default_rng(0).standard_normal((m, 8 * 128)), dtype), torch.empty((m, 8 * 128), dtype=DT[dtype], device="cuda")
        nbytes = q4k.q4k_shared_prefix_attention_workspace_size(b, 1, m, 8, hk, 128)
        ws, flag = torch.zeros(nbytes, dtype=torch.uint8, device="cuda"), err_flag()
        q4k.q4k_shared_prefix_attention(q, m, 8, hk, 128, 1024, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"],
                                        dev(q_starts(s.new)), dev(np.array(s.lens, np.int32)), dev(s.table), b, s.table.shape[1], 64, c.pages,
                                        dev(s.start), dev(s.prefix), 1, 1, max(s.lens), length, 0.1, 0, out, 1024, ws, nbytes, flag)
        torch.cuda.synchronize()
        assert int(flag) in (0, TIMEOUT) and (limit > 1 or length < 30000 or int(flag) == TIMEOUT)
        monkeypatch.delenv("Q4K_WAIT_NS")
        assert np.array_equal(want, s.run(8, dtype, check=False))


def test_offsets_past_32_bits():
    """A cache whose shared and own pages lie beyond 2^32 bytes."""
    hk, page, d, hq = 8, 128, 128, 16
    pages = (1 << 32) // (hk * page * d) + 64
    k = torch.zeros((pages, hk, page, d), dtype=torch.uint8, device="cuda")
    v, ks, vs = torch.zeros_like(k), torch.ones((pages, hk), device="cuda"), torch.ones((pages, hk), device="cuda")
    small = Cache(9, 4, hk, page, d)
    place = [pages - 1, 3, pages - 40, pages - 7]
    for i, p in enumerate(place):
        for full, s in ((k, "k"), (v, "v")):
            full[p] = dev(small.codes[s][i])
        ks[p], vs[p] = dev(small.scale["k"][i]), dev(small.scale["v"][i])
    order = np.array([[0, 1, 2], [0, 1, 3]])
    table = dev(np.array(place, np.int32)[order])
    for dtype in ("f32", "bf16"):
        q = rows(np.random.default_rng(3).standard_normal((3, hq * d)), dtype)
        out = torch.empty_like(q)
        nbytes = q4k.q4k_shared_prefix_attention_workspace_size(2, 1, 3, hq, hk, d)
        ws, flag = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), err_flag()
        q4k.q4k_shared_prefix_attention(q, 3, hq, hk, d, hq * d, k, v, ks, vs, dev(np.array([0, 1, 3], np.int32)),
                                        dev(np.array([300, 310], np.int32)), table, 2, 3, page, pages, dev(np.array([0, 2], np.int32)),
                                        dev(np.array([270], np.int32)), 1, 2, 310, 270, 0.09, 0, out, hq * d, ws, nbytes, flag)
        ref, tol = attention_ref(f64(q).reshape(3, hq, d), small, order, [1, 2], [300, 310], hq // hk, 0.09, 0, dtype)
        assert int(flag) == 0 and (np.abs(f64(out).reshape(3, hq, d) - ref) <= 2 * tol).all()


@pytest.mark.parametrize("setting", [None, "0"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_shared_goes_by_size(dtype, setting, monkeypatch):
    """Calls and groups on both sides of the rules: the same tokens, shared or not."""
    monkeypatch.delenv("Q4K_SHARE_PREFIX") if setting is None else monkeypatch.setenv("Q4K_SHARE_PREFIX", setting)
    Shared(30, [(400, samples(5))], 2, 64, 16).run(8, dtype)                                 # a small call
    Shared(31, [(2000, samples(40, own=0))], 8, 64, 64).run(32, dtype)
    Shared(32, [(1000, samples(2)), (1500, samples(70)), (900, samples(3, 2)), (30, samples(9))], 8, 64, 32).run(32, dtype)  # some groups of a large one
    Shared(33, [(700, samples(2)) for _ in range(30)], 8, 64, 32).run(32, dtype, max_prefix=1 << 30)  # no group
    Shared(34, [(1500, samples(70))], 8, 64, 32).run(32, dtype, window=300)
    for most in (2500, 1 << 29):   # long own parts by the hint, and a hint that says nothing
        Shared(35, [(1000, samples(70))], 8, 64, 32).run(32, dtype, hints=(1, most))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_malformed_lengths(dtype):
    """Lengths below the new tokens, below zero: flagged, clamped; the group shares what lies before all its new tokens, here nothing."""
    s = Shared(40, [(200, [(1, 9), (4, -202), (1, 5), (2, -202)]), (300, samples(6))], 2, 64, 16)
    assert s.lens[1] == 2 and s.lens[3] == 0
    raw = list(s.lens)
    raw[3] = -7
    s.run(8, dtype, raw_lens=raw, flagged=SEQ_FLAG)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_malformed_starts(dtype):
    """Starts that fall or leave the rows: flagged, nothing is shared, no access leaves its buffer."""
    s = Shared(41, [(200, samples(6, 2)), (300, samples(6))], 2, 64, 16)
    good = q_starts(s.new).tolist()
    for raw in ([0, 2, 4, 3, 8, 10, 12, 13, 14, 15, 16, 17, 18], [-5, *good[1:]], [*good[:-1], 1000], [18] * 13, good[::-1]):
        flagged = 0 if raw == [18] * 13 else SEQ_FLAG   # (no sequence has rows: within the rules)
        s.run(8, dtype, raw_starts=raw, flagged=flagged, check=False, times=1)   # (rows of two sequences are either's)
    s.run(8, dtype)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_sequences_than_the_plan_holds_at_hand(dtype, window):
    """Lengths and places of sequences, and groups, that are looked up in device memory."""
    Shared(42, [(200, [(1 + i % 2, i % 20) for i in range(2100)])], 1, 64, 16, before=[(1, 30)] * 9).run(2, dtype, window)
    Shared(43, [(64 + 16 * (k % 3), samples(2 + k % 3)) for k in range(200)], 1, 64, 16).run(2, dtype, window)
    Shared(44, [(160, samples(12)) for k in range(180)], 1, 64, 16).run(1, dtype, window)   # both


def test_more_rows_than_are_shared():
    """q4k_paged_attention's own result, bit for bit."""
    hq, hk, d, page, batch, n = 32, 4, 64, 16, 8200, 4
    m, c = batch * n, Cache(45, 12, hk, page, d)
    c.upload()
    table, starts, lens = dev(np.resize(c.order[:12], (batch, 3)).astype(np.int32)), dev(np.arange(0, m + 1, n, dtype=np.int32)), dev(np.full(batch, 40, np.int32))
    q = rows(np.random.default_rng(45).standard_normal((m, hq * d)), "bf16")
    flag, outs = err_flag(), [torch.empty_like(q), torch.empty_like(q)]
    for shared, out in enumerate(outs):
        args = (q, m, hq, hk, d, hq * d, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"], starts, lens, table, batch, 3, page, 12)
        if shared:
            nbytes = q4k.q4k_shared_prefix_attention_workspace_size(batch, 1, m, hq, hk, d)
            ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
            q4k.q4k_shared_prefix_attention(*args, dev(np.array([0, batch], np.int32)), dev(np.array([32], np.int32)), 1, n, 40, 32, 0.125, 0, out,
                                            hq * d, ws, nbytes, flag)
        else:
            nbytes = q4k.q4k_paged_attention_workspace_size(batch, m, hq, hk, d)
            ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
            q4k.q4k_paged_attention(*args, n, 40, 0.125, 0, out, hq * d, ws, nbytes, flag)
    assert int(flag) == 0 and torch.equal(*outs)


def test_one_workspace_for_calls_in_turn():
    """Calls of other sizes and types on the same bytes, one after another."""
    made = [(Shared(50, [(700, samples(9))], 2, 128, 32), 8, "f32"), (Shared(51, [(300, samples(70)), (900, samples(12, 3))], 4, 64, 16), 16, "bf16"),
            (Shared(52, [(2000, samples(7, 2))], 1, 64, 64), 4, "bf16")]
    need = max(q4k.q4k_shared_prefix_attention_workspace_size(len(s.new), len(s.prefix), sum(s.new), hq, s.hk, s.d) for s, hq, _ in made)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    want = [s.run(hq, dtype) for s, hq, dtype in made]
    for _ in range(2):
        for (s, hq, dtype), w in zip(made, want):
            assert np.array_equal(s.run(hq, dtype, check=False, times=1, ws=ws), w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,own", [
    (8, 8, [11009] * 4), (8, 2, [19585] * 9), (8, 1, [32001] * 11), (4, 2, [6529] * 27),
    (8, 1, [103252, 56271, 42002, 21075, 89009, 13510, 10247, 17084])])
def test_own_parts_of_more_tokens_than_whole_pieces(hq, hk, own, dtype):
    """Own tokens that are a little more than 32 k for each of the pieces that a call is cut into."""
    Shared(60, [(128, [(1, n - 1) for n in own])], hk, 64, 64).run(hq, dtype, times=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_without_new_tokens_do_not_lead_their_group(dtype):
    """Ended ones at a group's start, whose rows of the page table hold anything."""
    s = Shared(61, [(320, [(0, -320), (0, 5), (1, 7), (2, 0)]), (300, [(0, -300), (1, 1), (1, 4)]), (96, [(0, 0), (0, 0)])], 2, 64, 16)
    assert s.lens[0] == 0 and s.lens[4] == 0
    s.table[[0, 4]], s.table[1] = 0x7FFFFFF0, -1
    s.run(8, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_workspace_without_room_for_what_is_shared(dtype, monkeypatch):
    """One that was sized for q4k_paged_attention, for a call of more rows than are shared, or short by 256 bytes: every sequence reads its prefix
    itself, with q4k_paged_attention's own result."""
    s = Shared(62, [(300, samples(5))], 2, 64, 16)
    size = q4k.q4k_shared_prefix_attention_workspace_size
    monkeypatch.setenv("Q4K_SHARE_PREFIX", "0")
    want = s.run(8, dtype)
    monkeypatch.setenv("Q4K_SHARE_PREFIX", "1")
    assert not np.array_equal(s.run(8, dtype), want)
    for nbytes in (q4k.q4k_paged_attention_workspace_size(5, 5, 8, 2, 64), size(5, 1, 1 << 20, 8, 2, 64), size(5, 1, 5, 8, 2, 64) - 256):
        ws = torch.full((nbytes + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        monkeypatch.setattr(q4k, "q4k_shared_prefix_attention_workspace_size", lambda *a: nbytes)
        assert np.array_equal(s.run(8, dtype, ws=ws[:nbytes]), want)
        assert (ws[nbytes:] == 0xA5).all()
    monkeypatch.setattr(q4k, "q4k_shared_prefix_attention_workspace_size", lambda *a: q4k.q4k_paged_attention_workspace_size(5, 5, 8, 2, 64) - 1)
    with pytest.raises(q4k.Q4KError):
        s.run(8, dtype, ws=ws)
