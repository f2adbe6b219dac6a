"""Host-side checks (no GPU) of the attention-side calls: q4k_qk_norm_rope, q4k_kv_append and
q4k_paged_attention reject invalid arguments with the documented status before anything is
enqueued, accept empty batches, and their bindings refuse tensors of other element types."""
import pytest

import bit_quantized_moe_q4k_gb300 as q4k

torch = pytest.importorskip("torch")

A16 = 1 << 20          # a fake 16-byte-aligned address; never dereferenced by these calls
OFF4, OFF8 = A16 + 4, A16 + 8


def norm_rope(**kw):
    a = dict(q=A16, k=A16, dtype=0, m=3, hq=8, hk=2, d=128, qs=1024, ks=256, wq=A16, wk=A16, eps=1e-6, pos=A16, f=A16,
             rot=128, mode=0, qo=A16, ko=A16, odt=0, qos=1024, kos=256)
    a.update(kw)
    return q4k.load().q4k_qk_norm_rope(a["q"], a["k"], a["dtype"], a["m"], a["hq"], a["hk"], a["d"], a["qs"], a["ks"],
                                       a["wq"], a["wk"], a["eps"], a["pos"], a["f"], a["rot"], a["mode"], a["qo"],
                                       a["ko"], a["odt"], a["qos"], a["kos"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 13), (dict(odt=-1), 13), (dict(m=-1), 2), (dict(d=96), 2), (dict(d=512), 2),
    (dict(hq=-1), 2), (dict(hq=0, hk=0), 2), (dict(hq=65536), 9), (dict(rot=8), 2), (dict(rot=144), 2), (dict(rot=-16), 2),
    (dict(mode=2), 8), (dict(qs=1023), 2), (dict(kos=255), 2), (dict(qs=1026), 7), (dict(dtype=1, qs=1028), 7),
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(f=None), 1),
    (dict(q=OFF8), 7), (dict(ko=OFF8), 7), (dict(wq=OFF4), 7), (dict(wk=OFF4), 7), (dict(f=OFF4), 7),
])
def test_norm_rope_rejects(kw, status):
    assert norm_rope(**kw) == status
    assert q4k.load().q4k_last_error_string()


def test_norm_rope_empty_batch():
    assert norm_rope(m=0) == 0


def append(**kw):
    a = dict(k=A16, v=A16, dtype=0, m=3, hk=2, d=128, ks=256, vs=256, wk=A16, eps=1e-6, f=A16, rot=128, mode=0, qst=A16,
             lens=A16, table=A16, batch=2, mp=4, page=16, np=8, kc=A16, vc=A16, ksc=A16, vsc=A16)
    a.update(kw)
    return q4k.load().q4k_kv_append(a["k"], a["v"], a["dtype"], a["m"], a["hk"], a["d"], a["ks"], a["vs"], a["wk"],
                                    a["eps"], a["f"], a["rot"], a["mode"], a["qst"], a["lens"], a["table"], a["batch"],
                                    a["mp"], a["page"], a["np"], a["kc"], a["vc"], a["ksc"], a["vsc"], None, None)


PAGED_REFUSALS = [
    (dict(dtype=7), 13), (dict(m=-1), 2), (dict(batch=-1), 2), (dict(d=256), 2), (dict(d=80), 2), (dict(hk=0), 2),
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(np=0), 2), (dict(mp=0), 2),
    (dict(mp=1 << 27), 9), (dict(m=(1 << 24) + 1), 9), (dict(batch=(1 << 24) + 1), 9),
    (dict(qst=None), 1), (dict(lens=None), 1), (dict(table=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(ksc=None), 1), (dict(vsc=None), 1), (dict(kc=OFF8), 7), (dict(vc=OFF4), 7), (dict(qst=A16 + 2), 7),
    (dict(vsc=A16 + 1), 7),
]


@pytest.mark.parametrize("kw,status", PAGED_REFUSALS + [
    (dict(rot=24), 2), (dict(mode=5), 8), (dict(f=None), 1), (dict(wk=OFF4), 7), (dict(ks=255), 2), (dict(vs=258), 7),
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=OFF4), 7), (dict(hk=65536, ks=1 << 23, vs=1 << 23), 9),
])
def test_append_rejects(kw, status):
    assert append(**kw) == status
    assert q4k.load().q4k_last_error_string()


def test_append_empty():
    assert append(m=0) == 0
    assert append(batch=0) == 0


def attention(**kw):
    a = dict(q=A16, dtype=0, m=3, hq=8, hk=2, d=128, qs=1024, kc=A16, vc=A16, ksc=A16, vsc=A16, qst=A16, lens=A16,
             table=A16, batch=2, mp=4, page=16, np=8, maxq=2, maxl=64, scale=0.1, window=0, out=A16, os=1024, ws=A16,
             wsb=None)
    a.update(kw)
    lib = q4k.load()
    if a["wsb"] is None:
        a["wsb"] = lib.q4k_paged_attention_workspace_size(2, 3, 8, 2, 128)
    return lib.q4k_paged_attention(a["q"], a["dtype"], a["m"], a["hq"], a["hk"], a["d"], a["qs"], a["kc"], a["vc"],
                                   a["ksc"], a["vsc"], a["qst"], a["lens"], a["table"], a["batch"], a["mp"], a["page"],
                                   a["np"], a["maxq"], a["maxl"], a["scale"], a["window"], a["out"], a["os"], a["ws"],
                                   a["wsb"], None, None)


@pytest.mark.parametrize("kw,status", PAGED_REFUSALS + [
    (dict(hq=7), 2), (dict(hq=1), 2), (dict(maxq=-1), 2), (dict(maxl=-1), 2), (dict(window=-1), 2), (dict(qs=1022), 2),
    (dict(qs=1026), 7), (dict(os=1020), 2), (dict(q=None), 1), (dict(out=None), 1), (dict(q=OFF4), 7), (dict(out=OFF8), 7),
    (dict(ws=None), 4), (dict(wsb=1024), 4), (dict(ws=A16 + 16), 4), (dict(hq=65538, qs=1 << 24, os=1 << 24), 9),
])
def test_attention_rejects(kw, status):
    assert attention(**kw) == status
    assert q4k.load().q4k_last_error_string()


def test_attention_empty_and_workspace():
    assert attention(m=0) == 0
    assert attention(batch=0) == 0
    lib = q4k.load()
    assert lib.q4k_paged_attention_workspace_size(1, 1, 32, 4, 128) % 256 == 0
    assert lib.q4k_paged_attention_workspace_size(1, 1, 32, 4, 96) == 0
    assert lib.q4k_paged_attention_workspace_size(1, 1, 30, 4, 128) == 0
    assert lib.q4k_paged_attention_workspace_size(-1, 1, 32, 4, 128) == 0


class FakeCuda:
    """What a binding reads of a device tensor before it calls the library."""
    is_cuda = True

    def __init__(self, dtype):
        self.dtype = dtype

    def data_ptr(self):
        return A16


def test_bindings_refuse_other_element_types():
    f32, f16, bf, i32, i64 = (FakeCuda(t) for t in (torch.float32, torch.float16, torch.bfloat16, torch.int32,
                                                    torch.int64))
    f64, u8 = FakeCuda(torch.float64), FakeCuda(torch.uint8)

    def nr(q=f32, k=f32, w=bf, pos=i32, f=f64, out=f32):
        q4k.q4k_qk_norm_rope(q, k, 0, 8, 2, 128, 1024, 256, w, w, 1e-6, pos, f, 128, 0, out, out, 1024, 256, stream=0)

    nr()
    for bad in (dict(q=f16), dict(q=bf), dict(w=f32), dict(pos=i64), dict(f=f32), dict(out=f16)):
        with pytest.raises(ValueError):
            nr(**bad)

    def at(q=f32, kc=u8, ks=f32, qs=i32, out=f32):
        q4k.q4k_paged_attention(q, 0, 8, 2, 128, 1024, kc, u8, ks, f32, qs, i32, i32, 1, 4, 16, 8, 1, 64, 0.1, 0, out,
                                1024, u8, 0, stream=0)

    at()
    for bad in (dict(q=f16), dict(out=bf), dict(kc=bf), dict(ks=bf), dict(qs=i64)):
        with pytest.raises(ValueError):
            at(**bad)

    def ap(k=f32, v=f32, w=bf, table=i32):
        q4k.q4k_kv_append(k, v, 0, 2, 128, 256, 256, w, 1e-6, f64, 128, 0, i32, i32, table, 1, 4, 16, 8, u8, u8, f32,
                          f32, stream=0)

    ap()
    for bad in (dict(k=bf), dict(v=f16), dict(w=f32), dict(table=i64)):
        with pytest.raises(ValueError):
            ap(**bad)


def test_host_tensors_are_refused():
    x = torch.zeros(8)
    with pytest.raises(ValueError):
        q4k.q4k_qk_norm_rope(x, None, 1, 1, 0, 64, 64, 64, None, None, 1e-6, None, None, 0, 0, x, None, 64, 64, stream=0)


def test_bindings_take_raw_addresses_for_rows():
    """Addresses pass where tensors do; the rows' element type is the other tensor's, and one tensor is asked for."""
    f32, bf, i32, f64, u8 = (FakeCuda(t) for t in (torch.float32, torch.bfloat16, torch.int32, torch.float64, torch.uint8))

    def nr(q, k, qo, ko):
        q4k.q4k_qk_norm_rope(q, k, 0, 8, 2, 128, 1024, 256, bf, bf, 1e-6, i32, f64, 128, 0, qo, ko, 1024, 256, stream=0)

    def ap(k, v):
        q4k.q4k_kv_append(k, v, 0, 2, 128, 256, 256, bf, 1e-6, f64, 128, 0, i32, i32, i32, 1, 4, 16, 8, u8, u8, f32, f32, stream=0)

    def at(q, out):
        q4k.q4k_paged_attention(q, 0, 8, 2, 128, 1024, A16, u8, f32, f32, i32, i32, A16, 1, 4, 16, 8, 1, 64, 0.1, 0, out, 1024,
                                A16, 0, stream=0)

    nr(A16, f32, f32, A16)
    nr(bf, A16, A16, f32)
    nr(f32, None, None, f32)
    ap(A16, bf)
    ap(f32, A16)
    at(A16, bf)
    at(f32, A16)
    for call in (lambda: nr(A16, A16, f32, f32), lambda: nr(f32, f32, A16, None), lambda: ap(A16, A16), lambda: at(A16, A16),
                 lambda: at(None, A16)):
        with pytest.raises(ValueError, match="element type"):
            call()
    for call in (lambda: at(f32, bf), lambda: ap(bf, f32), lambda: ap(A16, i32)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("raw", [True, False])
def test_the_current_stream_with_and_without_torchs_raw_getter(raw, monkeypatch):
    """The raw getter is not part of torch's public interface: without it the public one is asked."""
    from types import SimpleNamespace

    from bit_quantized_moe_q4k_gb300 import _lib
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=77))
    if raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 78 + device, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert _lib._stream(None) == (78 if raw else 77)
    assert _lib._stream(5) == 5 and _lib._stream(SimpleNamespace(cuda_stream=6)) == 6
