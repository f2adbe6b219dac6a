"""GPU parity of the attention side (q4k_qk_norm_rope, q4k_kv_append, q4k_paged_attention) with
plain fp64 implementations written here, through the C ABI.

Tolerances are counted from the kernels' roundings, u = 2^-24 (half a step of fp32):
  * norm and rotation: the sum of squares has at most 13 additions, all terms positive (13 u,
    halved by the root), mean, eps, root and reciprocal 3.5 u, two products 2 u: 12 u of the normed
    value; sine and cosine are within 5.4 u (3 u pi/4 from the reduced angle in fp32, 2 u of the polynomials,
    0.3 u of the 32-bit turn); two products and a sum: 2 u. Together below 24 u (|a| + |b|).
  * the append adds half a step of e4m3: 2^-4 |x|, or 2^-10 of the scale where that is larger.
  * attention, per row: |ds| <= S (2^-22 + (d/16 + 8) 2^-23) with S the largest sum_c |q_c k_c| *
    scale (the split of q, the chain of tensor-core sums, truncating), x's own rounding
    2^-23 (|x| + |e|), ex2 2^-22; a weight error dp / p moves the result by at most twice that times
    sum_j p_j |v_j|; summing n tokens adds (n/64 + 40) u of the same. fp16 weights (bf16 rows)
    add 2^-11 of it, and the store half a step of the output type.
"""
import math
from pathlib import Path

import numpy as np
import pytest

import bit_quantized_moe_q4k_gb300 as q4k
from bit_quantized_moe_q4k_gb300 import inputs

from helpers import dev, err_flag, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(x, dtype, stride=None):
    """Device rows of x [m, n] in `dtype`, `stride` elements apart (the gap holds NaN)."""
    m, n = x.shape
    t = torch.full((max(m, 1), stride or n), float("nan"), dtype=DT[dtype], device="cuda")
    t[:m, :n] = dev(x.astype(np.float32)).to(DT[dtype])
    return t


# ---- e4m3 --------------------------------------------------------------------------------------

def e4m3_values():
    c = np.arange(256)
    s, e, f = np.where(c & 128, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = s * np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))
    v[[0x7F, 0xFF]] = np.nan
    return v


E4M3 = e4m3_values()


def e4m3_round(x):
    """Codes of x: nearest, ties to even, saturating (finite x)."""
    pos = E4M3[:0x7F]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 0x7E)
    lo = hi - 1
    d0, d1 = a - pos[lo], pos[hi] - a
    code = np.where(d0 < d1, lo, np.where(d1 < d0, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(amax):
    if amax == 0:
        return -64
    return max(-64, math.ceil(math.log2(amax / 448.0) - 1e-13))


# ---- norm and rotation -------------------------------------------------------------------------

def norm_rope_ref(x, w, pos, inv_freq, mode):
    """x [m, heads, d] in fp64 -> (result, |a| + |b| of each element's pair)."""
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
    out, mag = y.copy(), np.abs(y)
    half = len(inv_freq)
    if half:
        ang = pos.astype(np.float64)[:, None] * inv_freq
        turn = np.exp(1j * ang)[:, None, :]
        a, b = (slice(0, half), slice(half, 2 * half)) if mode == "halves" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
        z = (y[..., a] + 1j * y[..., b]) * turn
        out[..., a], out[..., b] = z.real, z.imag
        mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, mag


def freqs(rot, theta=1e6):
    return theta ** (-np.arange(rot // 2, dtype=np.float64) / max(1, rot // 2))


MODES = {"halves": q4k.ROPE_HALVES, "pairs": q4k.ROPE_PAIRS}


def run_norm_rope(seed, m, hq, hk, d, rot, mode, dtype, odtype, norm=True, pos=None, pad=0, theta=1e6):
    g = np.random.default_rng(seed)
    row = (hq + hk) * d + pad
    x = rows(g.standard_normal((m, row)) * np.exp(g.standard_normal((1, row))), dtype)
    pos = g.integers(0, 1 << 20, m).astype(np.int32) if pos is None else np.asarray(pos, np.int32)
    wq, wk = (inputs.to_bf16_bits((1 + 0.2 * g.standard_normal(d)).astype(np.float32)) for _ in range(2))
    f = freqs(rot, theta)
    qo = torch.full((m, hq * d + 16), float("nan"), dtype=DT[odtype], device="cuda")
    ko = torch.full((m, hk * d + 16), float("nan"), dtype=DT[odtype], device="cuda")
    q4k.q4k_qk_norm_rope(x if hq else None, x[:, hq * d:] if hk else None, m, hq, hk, d, row, row,
                         dev(wq.view(np.int16)) if norm else None, dev(wk.view(np.int16)) if norm else None, EPS,
                         dev(pos), dev(f) if rot else None, rot, MODES[mode], qo if hq else None, ko if hk else None,
                         hq * d + 16, hk * d + 16)
    xs = f64(x)
    for out, heads, w, at in ((qo, hq, wq, 0), (ko, hk, wk, hq * d)):
        if not heads:
            continue
        wf = (w.astype(np.uint32) << 16).view(np.float32).astype(np.float64) if norm else None
        ref, mag = norm_rope_ref(xs[:, at:at + heads * d].reshape(m, heads, d), wf, pos, f, mode)
        got = f64(out)
        assert np.isnan(got[:, heads * d:]).all(), "wrote past the heads"
        got = got[:, :heads * d].reshape(m, heads, d)
        tol = 24 * U * mag + (STEP[odtype] * np.abs(ref) * (1 + 2.0 ** -10) if odtype == "bf16" else 0)
        worst = np.max(np.abs(got - ref) - tol)
        assert worst <= 0, f"off by {worst} beyond the bound"


@pytest.mark.parametrize("dtype,odtype", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mode", ["halves", "pairs"])
def test_norm_rope_types(d, mode, dtype, odtype):
    run_norm_rope(d, 5, 3, 2, d, d, mode, dtype, odtype)


@pytest.mark.parametrize("m,hq,hk,rot,mode,norm,pad", [
    (1, 32, 4, 128, "halves", True, 0), (1, 1, 0, 128, "pairs", True, 8), (7, 0, 5, 64, "halves", True, 0),
    (33, 5, 1, 16, "pairs", True, 24), (2, 7, 7, 48, "halves", False, 8), (3, 2, 2, 0, "halves", True, 0),
    (3, 2, 2, 112, "pairs", False, 0), (300, 9, 3, 128, "halves", True, 64),
])
def test_norm_rope_shapes(m, hq, hk, rot, mode, norm, pad):
    run_norm_rope(m + rot, m, hq, hk, 128, rot, mode, "f32", "f32", norm, pad=pad)


def test_norm_rope_far_and_negative_positions():
    """Positions to the ends of int32: the angle loses nothing to its size (fp64's own product is
    off by 2^-53 of up to 2^31 radians here, 2^-22: the reference is formed from exact integers)."""
    pos = np.array([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789], np.int64)
    d, theta = 64, 10000.0
    x = np.random.default_rng(3).standard_normal((len(pos), d))
    f = freqs(d, theta)
    xt = rows(x, "f32")
    out = torch.empty_like(xt)
    q4k.q4k_qk_norm_rope(xt, None, len(pos), 1, 0, d, d, d, None, None, EPS, dev(pos.astype(np.int32)), dev(f), d,
                         q4k.ROPE_HALVES, out, None, d, d)
    from fractions import Fraction
    tau = Fraction(62831853071795864769252867665590057683943387987502116419498891846156328125724, 10 ** 76)
    ang = np.empty((len(pos), d // 2))
    for i, p in enumerate(pos):
        for j, v in enumerate(f):
            turns = Fraction(float(v)) * int(p) / tau
            ang[i, j] = float((turns - math.floor(turns)) * tau)
    xs = f64(xt)
    z = (xs[:, :d // 2] + 1j * xs[:, d // 2:]) * np.exp(1j * ang)
    ref = np.concatenate([z.real, z.imag], 1)
    mag = np.tile(np.abs(xs[:, :d // 2]) + np.abs(xs[:, d // 2:]), (1, 2))
    # F is cut to 2^-64 of a turn and its 53-bit source: |pos| * 2^-63 turns at most
    assert (np.abs(f64(out) - ref) <= (24 * U + 2 * math.pi * 2.0 ** -31) * mag).all()


def test_norm_rope_in_place_and_nonfinite():
    """A result may replace its input; an infinity or NaN in one head leaves the other heads alone."""
    m, d = 4, 128
    g = np.random.default_rng(5)
    x = rows(g.standard_normal((m, 3 * d)), "f32")
    x[1, d + 5] = float("nan")
    x[2, 2 * d] = float("inf")
    pos, f = dev(np.arange(m, dtype=np.int32)), dev(freqs(64))
    out = torch.empty_like(x)
    q4k.q4k_qk_norm_rope(x, None, m, 3, 0, d, 3 * d, 3 * d, None, None, EPS, pos, f, 64, 0, out, None, 3 * d, 3 * d)
    y = x.clone()
    q4k.q4k_qk_norm_rope(y, None, m, 3, 0, d, 3 * d, 3 * d, None, None, EPS, pos, f, 64, 0, y, None, 3 * d, 3 * d)
    assert torch.equal(out.view(torch.int32), y.view(torch.int32))
    bad = ~np.isfinite(host(out))
    assert set(zip(*np.where(bad))) <= {(1, d + 5), (1, d + 37), (2, 2 * d), (2, 2 * d + 32)} and bad.sum() >= 2


# ---- the paged cache ---------------------------------------------------------------------------

class Cache:
    """Random codes and power-of-two scales; every slot filled (recycled pages), NaN codes in none."""

    def __init__(self, seed, pages, heads, page, d, pow2=True):
        g = np.random.default_rng(seed)
        self.heads, self.page, self.d, self.pages = heads, page, d, pages
        shape = (pages, heads, page, d)
        self.codes = {s: e4m3_round(g.standard_normal(shape) * 60) for s in "kv"}
        self.scale = {"k": 2.0 ** g.integers(-9, -5, shape[:2]), "v": 2.0 ** g.integers(-12, -4, shape[:2])}
        if not pow2:
            self.scale = {s: v * g.uniform(1, 2, shape[:2]) for s, v in self.scale.items()}
        self.scale = {s: v.astype(np.float32) for s, v in self.scale.items()}
        self.order = g.permutation(pages).astype(np.int32)

    def upload(self):
        self.dev = {s: dev(self.codes[s]) for s in "kv"}
        self.dev_scale = {s: dev(self.scale[s]) for s in "kv"}

    def values(self, side, ids, length):
        """[heads, length, d] fp64 values of the pages `ids`."""
        v = E4M3[self.codes[side][ids]] * self.scale[side][ids].astype(np.float64)[..., None, None]
        return v.transpose(1, 0, 2, 3).reshape(self.heads, -1, self.d)[:, :length]


def tables(cache, lens, extra=1):
    """Page table rows taken from the cache's permutation; entries past the last page are junk."""
    need = [-(-n // cache.page) for n in lens]
    t = np.full((len(lens), max(need + [1]) + extra), 0x7FFFFFF0, np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = cache.order[at:at + n]
        at += n
    assert at <= cache.pages
    return t


def q_starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


# ---- append ------------------------------------------------------------------------------------

def run_append(seed, new, ctx, heads, d, page, dtype, rot=None, mode="halves", norm=True, gain=1.0, times=1):
    g = np.random.default_rng(seed)
    lens = [n + c for n, c in zip(new, ctx)]
    pages = sum(-(-n // page) for n in lens) + 2
    c = Cache(seed, pages, heads, page, d)
    c.upload()
    table = tables(c, lens)
    m = sum(new)
    rot = d if rot is None else rot
    kv = rows(g.standard_normal((m, 2 * heads * d)) * gain, dtype, 2 * heads * d + 8)
    w = inputs.to_bf16_bits((1 + 0.2 * g.standard_normal(d)).astype(np.float32))
    f = freqs(rot)
    flag = err_flag()
    for _ in range(times):
        q4k.q4k_kv_append(kv, kv[:, heads * d:], m, heads, d, 2 * heads * d + 8, 2 * heads * d + 8,
                          dev(w.view(np.int16)) if norm else None, EPS, dev(f) if rot else None, rot, MODES[mode],
                          dev(q_starts(new)), dev(np.array(lens, np.int32)), dev(table), len(new), table.shape[1], page,
                          pages, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"], flag)
    assert int(host(flag)[0]) == 0
    codes = {s: host(c.dev[s]) for s in "kv"}
    scale = {s: host(c.dev_scale[s]) for s in "kv"}
    x = f64(kv)[:m, :2 * heads * d].reshape(m, 2, heads, d)
    wf = (w.astype(np.uint32) << 16).view(np.float32).astype(np.float64) if norm else None
    seen = {s: np.zeros(c.codes[s].shape[:3], bool) for s in "kv"}
    row = 0
    for i, (n, length) in enumerate(zip(new, lens)):
        pos = np.arange(length - n, length)
        k, mag = norm_rope_ref(x[row:row + n, 0], wf, pos, f, mode)
        err = {"k": 24 * U * mag, "v": np.zeros_like(mag)}
        val = {"k": k, "v": x[row:row + n, 1]}
        for p in range((length - n) // page, -(-length // page)) if n else ():
            lo, hi = max(length - n, p * page), min(length, (p + 1) * page)
            pid, held = table[i, p], max(length - n, p * page) - p * page
            for s in "kv":
                for h in range(heads):
                    part = val[s][lo - (length - n):hi - (length - n), h]
                    slack = err[s][lo - (length - n):hi - (length - n), h]
                    amax = np.abs(part).max()
                    ok = {exponent(amax), exponent(max(0, amax - slack.max())), exponent(amax + slack.max())}
                    old = c.scale[s][pid, h]
                    want = {max(2.0 ** e, old) if held else 2.0 ** e for e in ok}
                    sc = float(scale[s][pid, h])
                    assert sc in want, (s, pid, h, sc, want)
                    got = E4M3[codes[s][pid, h, held:hi - p * page]] * sc
                    tol = np.maximum(2.0 ** -4 * np.abs(part), 2.0 ** -10 * sc) * (1 + 2.0 ** -20) + slack
                    assert (np.abs(got - part) <= tol).all()
                    again = e4m3_round(E4M3[c.codes[s][pid, h, :held]] * (old / sc)) if held else None
                    if held:
                        assert np.array_equal(E4M3[codes[s][pid, h, :held]], E4M3[again])
                    seen[s][pid, h, :hi - p * page] = True
        row += n
    for s in "kv":  # every other slot as it was
        assert np.array_equal(codes[s][~seen[s]], c.codes[s][~seen[s]])
        touched = seen[s].any(-1)
        assert np.array_equal(scale[s][~touched], c.scale[s][~touched])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_pages_and_types(page, d, dtype):
    run_append(page + d, [1, 5, page, 2 * page + 3], [0, page - 2, 7, 1], 2, d, page, dtype)


@pytest.mark.parametrize("new,ctx,kw", [
    ([1], [0], {}), ([1], [15], {}), ([1], [16], {}), ([1, 0, 1], [3, 9, 0], {}),
    ([300], [0], dict(mode="pairs")), ([2, 40, 1], [31, 0, 200], dict(rot=32, norm=False)),
    ([3, 3], [5, 20], dict(rot=0)), ([4], [6], dict(gain=1e-6, norm=False, rot=0)),
    ([4], [6], dict(gain=1e5, norm=False, rot=0)), ([4, 1], [6, 9], dict(gain=0.0, norm=False)),
    ([1] * 70, list(range(70)), {}),
])
def test_append_lengths(new, ctx, kw):
    run_append(len(new) + new[0], new, ctx, 3, 128, 16, "f32", **kw)


def test_append_twice_changes_nothing():
    run_append(9, [5, 1], [3, 18], 2, 128, 16, "f32", gain=1e3, norm=False, times=3)


def test_append_token_by_token_equals_at_once():
    """Power-of-two scales: a page filled one token at a time holds the values of one call, but
    where a code passed through e4m3's subnormals under a larger scale."""
    heads, d, page, n = 2, 64, 32, 32
    g = np.random.default_rng(12)
    kv = rows(g.standard_normal((n, 2 * heads * d)) * np.exp(0.3 * g.standard_normal((n, 1))), "f32")
    table = dev(np.array([[1]], np.int32))
    got = []
    for steps in ([n], [1] * n):
        c = Cache(1, 2, heads, page, d)
        c.upload()
        at = 0
        for s in steps:
            q4k.q4k_kv_append(kv[at:], kv[at:, heads * d:], s, heads, d, 2 * heads * d, 2 * heads * d, None, EPS, None, 0,
                              0, dev(np.array([0, s], np.int32)), dev(np.array([at + s], np.int32)), table, 1, 1, page,
                              2, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"])
            at += s
        got.append([E4M3[host(c.dev[s])[1]] * host(c.dev_scale[s])[1].astype(np.float64)[:, None, None] for s in "kv"]
                   + [host(c.dev_scale[s])[1] for s in "kv"])
    a, b = got
    for i in (2, 3):
        assert np.array_equal(a[i], b[i])
    for i in (0, 1):
        unit = a[i + 2].astype(np.float64)[:, None, None]
        assert (np.abs(a[i] - b[i]) <= np.where(np.abs(a[i]) >= unit * 2.0 ** -6, 0.0, unit * 2.0 ** -9)).all()


def test_append_nonfinite():
    """Infinities saturate at the scale of the finite values, NaN stays NaN, the rest is as ever."""
    heads, d, page = 1, 64, 16
    x = np.ones((3, 2 * d))
    x[0, 3], x[1, 4], x[2, d + 1], x[1, d + 2] = np.inf, np.nan, -np.inf, np.nan
    kv = rows(x, "f32")
    c = Cache(2, 1, heads, page, d)
    c.upload()
    q4k.q4k_kv_append(kv, kv[:, d:], 3, heads, d, 2 * d, 2 * d, None, EPS, None, 0, 0, dev(np.array([0, 3], np.int32)),
                      dev(np.array([3], np.int32)), dev(np.zeros((1, 1), np.int32)), 1, 1, page, 1, c.dev["k"],
                      c.dev["v"], c.dev_scale["k"], c.dev_scale["v"])
    for s, at in (("k", 0), ("v", d)):
        sc = float(host(c.dev_scale[s])[0, 0])
        assert sc == 2.0 ** exponent(1.0)
        got = E4M3[host(c.dev[s])[0, 0, :3]] * sc
        want = x[:, at:at + d].copy()
        want[np.isinf(want)] = np.sign(want[np.isinf(want)]) * 448 * sc
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("what", ["page_high", "page_negative", "len_short", "len_long", "start_falls", "start_past"])
def test_append_bad_indexes_raise_the_flag(what):
    """Indexes that do not fit: the flag is raised, nothing outside the right pages is written."""
    heads, d, page, pages = 2, 64, 16, 6
    c = Cache(4, pages, heads, page, d)
    c.upload()
    start, lens = np.array([0, 3, 6], np.int32), np.array([3, 20], np.int32)
    table = np.array([[0, 1], [2, 3]], np.int32)
    status = 12
    if what == "page_high":
        table[0, 0], status = pages, 11
    elif what == "page_negative":
        table[0, 0], status = -1, 11
    elif what == "len_short":
        lens[0] = 2
    elif what == "len_long":
        lens[1] = 33
    elif what == "start_falls":
        start[:] = [0, 7, 6]
    else:
        start[2] = 9
    kv = rows(np.random.default_rng(1).standard_normal((6, 2 * heads * d)), "f32")
    flag = err_flag()
    q4k.q4k_kv_append(kv, kv[:, heads * d:], 6, heads, d, 2 * heads * d, 2 * heads * d, None, EPS, None, 0, 0, dev(start),
                      dev(lens), dev(table), 2, 2, page, pages, c.dev["k"], c.dev["v"], c.dev_scale["k"],
                      c.dev_scale["v"], flag)
    assert int(host(flag)[0]) == status
    for s in "kv":
        assert np.array_equal(host(c.dev[s])[4:], c.codes[s][4:])
        if what.startswith("page"):
            assert np.array_equal(host(c.dev[s])[:2], c.codes[s][:2])  # dropped, not written elsewhere


# ---- attention ---------------------------------------------------------------------------------

def attention_ref(q, cache, table, new, lens, group, scale, window, dtype):
    """fp64 result and bound, [m, q_heads, d]."""
    m, hq, d = q.shape
    out, tol = np.zeros((m, hq, d)), np.zeros((m, hq, d))
    row = 0
    for i, (n, length) in enumerate(zip(new, lens)):
        ids = table[i, :-(-length // cache.page)]
        k, v = (cache.values(s, ids, length) for s in "kv")
        for r in range(n):
            pos = length - n + r
            lo = max(0, pos - window + 1) if window else 0
            if pos < 0:
                continue
            for h in range(hq):
                kk, vv, qq = k[h // group, lo:pos + 1], v[h // group, lo:pos + 1], q[row + r, h]
                s = kk @ qq * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                big = scale * (np.abs(kk) @ np.abs(qq)).max()
                ds = big * (2.0 ** -22 + (d / 16 + 8) * 2.0 ** -23)
                x = (np.abs(s).max() * 1.45 + 64 + 14) * 2.0 ** -23 + 2.0 ** -22
                mean_abs = p @ np.abs(vv)
                rel = 2 * (ds + x) + ((pos + 1 - lo) / 64 + 40) * U
                if dtype == "bf16":
                    rel += 2.0 ** -11 * 1.01
                out[row + r, h] = p @ vv
                tol[row + r, h] = rel * mean_abs + STEP[dtype] * np.abs(out[row + r, h]) * 1.01
        row += n
    return out, tol


def run_attention(seed, new, lens, hq, hk, d, page, dtype, window=0, q_gain=1.0, pow2=True, pad=0, hints=None,
                  cache=None, table=None, check=True, flagged=0, codes_after=None):
    g = np.random.default_rng(seed)
    c = cache or Cache(seed, sum(-(-n // page) for n in lens) + 2, hk, page, d, pow2)
    if codes_after:
        codes_after(c)
    c.upload()
    table = tables(c, lens) if table is None else table
    m = sum(new)
    q = rows(g.standard_normal((m, hq * d)) * q_gain, dtype, hq * d + pad)
    out = torch.full((max(m, 1), hq * d + pad), 7.0, dtype=DT[dtype], device="cuda")
    nbytes = q4k.q4k_paged_attention_workspace_size(len(new), m, hq, hk, d)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    flag = err_flag()
    scale = 1 / math.sqrt(d)
    maxq, maxl = hints or (max(new), max(lens))
    for _ in range(2):
        q4k.q4k_paged_attention(q, m, hq, hk, d, hq * d + pad, c.dev["k"], c.dev["v"], c.dev_scale["k"],
                                c.dev_scale["v"], dev(q_starts(new)), dev(np.array(lens, np.int32)), dev(table),
                                len(new), table.shape[1], page, c.pages, maxq, maxl, scale, window, out, hq * d + pad,
                                ws, nbytes, flag)
    got = f64(out)
    assert int(host(flag)[0]) == flagged
    if pad:
        assert (got[:, hq * d:] == 7.0).all()
    got = got[:m, :hq * d].reshape(m, hq, d)
    if check:
        ref, tol = attention_ref(f64(q)[:m, :hq * d].reshape(m, hq, d), c, table, new, lens, hq // hk, scale, window, dtype)
        worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-300))
        assert np.isfinite(got).all() and worst <= 1, f"{worst} of the bound"
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 129, 700])
def test_attention_single_token_lengths(length, d, dtype):
    run_attention(length, [1], [length], 8, 2, d, 16, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 2), (3, 1), (14, 2), (16, 2), (32, 4), (16, 1), (20, 1), (40, 1)])
def test_attention_head_groups(hq, hk, dtype):
    run_attention(hq, [1, 1, 2], [40, 3, 90], hq, hk, 128, 32, dtype)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_pages_ragged_batch(page, dtype):
    run_attention(page, [1] * 7, [1, 16, 127, 128, 129, 500, 33], 6, 2, 128, page, dtype, pad=16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,window", [
    ([3], [3], 0), ([5, 1, 4], [50, 1, 4], 0), ([9], [300], 0), ([1, 2], [200, 100], 1), ([4], [200], 16),
    ([4, 1], [200, 129], 17), ([6], [100], 100), ([6], [100], 1000), ([0, 1, 0], [5, 9, 0], 0),
    ([33], [33], 0), ([70, 1, 40], [70, 300, 111], 0), ([130], [200], 0), ([130], [200], 33), ([257, 129], [257, 700], 0),
    ([300], [421], 150),
])
def test_attention_several_tokens_and_windows(new, lens, window, dtype):
    run_attention(sum(lens), new, lens, 8, 2, 128, 32, dtype, window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,hq,hk,page,window", [
    ([100], [100], 4, 4, 16, 0), ([90, 300], [90, 300], 7, 1, 64, 0), ([150], [1000], 3, 3, 128, 64),
    ([65, 66, 1, 200], [65, 400, 50, 201], 10, 2, 16, 0),
])
def test_attention_prompts_short_heads(new, lens, hq, hk, page, window, dtype):
    run_attention(sum(lens), new, lens, hq, hk, 64, page, dtype, window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens,hq,hk,page,window", [
    ([130], [200], 64, 8, 32, 0), ([130], [200], 64, 8, 32, 33), ([257, 129], [257, 700], 32, 8, 16, 0), ([300], [421], 32, 2, 64, 150),
    ([70, 1, 40], [70, 300, 111], 64, 4, 32, 0), ([65, 66, 1, 200], [65, 400, 50, 201], 28, 2, 16, 0), ([500], [500], 8, 8, 128, 0),
    ([0, 300, 2], [7, 1300, 2], 14, 1, 128, 1), ([128, 128], [128, 256], 16, 1, 64, 100),
])
def test_attention_prompts_of_many_rows(new, lens, hq, hk, page, window, d, dtype):
    """Batches with enough rows that prompts go to the prompt kernels, alone or next to sequences that decode."""
    run_attention(sum(lens) + 1, new, lens, hq, hk, d, page, dtype, window, pad=16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,hq", [([1, 2], [70, 300], 8), ([150, 1], [150, 300], 64)])
def test_attention_largest_window(new, lens, hq, dtype):
    wide = run_attention(54, new, lens, hq, 2, 128, 16, dtype, window=0x7FFFFFFF)
    assert np.array_equal(wide, run_attention(54, new, lens, hq, 2, 128, 16, dtype, window=0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_prompts_of_many_rows_scales_and_magnitudes(dtype):
    def spread(c):
        c.scale["v"][:] = (2.0 ** np.resize([-40.0, 0.0, 30.0, -64.0, -3.0], c.scale["v"].size)).reshape(c.scale["v"].shape)
    run_attention(51, [1, 3, 100], [130, 90, 120], 64, 8, 128, 16, dtype, pow2=False)
    run_attention(52, [1, 2, 90], [130, 90, 200], 64, 8, 128, 16, dtype, codes_after=spread)
    for gain in (0.0, 1e-30, 30.0):
        run_attention(53, [140], [180], 32, 4, 128, 16, dtype, q_gain=gain)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_long_axis_is_split(dtype):
    run_attention(5, [1], [20011], 8, 1, 128, 64, dtype)
    run_attention(6, [1, 1, 1], [9000, 2, 4097], 4, 2, 64, 16, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("long", [9000, 24000, 33333, 60001])
def test_attention_one_long_sequence_among_short_ones(long, dtype):
    """The long one's axis is cut into many pieces, joined in two levels; the short ones share its last piece."""
    run_attention(31, [1] * 40, [1 + i % 3 for i in range(20)] + [long] + [2] * 19, 8, 2, 64, 128, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,longest", [(20, 200), (40, 511), (70, 200), (70, 700), (200, 60)])
def test_attention_many_short_sequences(batch, longest, dtype):
    """A CTA per tile, more tiles than CTAs, and tiles that are cut although they are many."""
    run_attention(55, [1] * batch, [1 + 37 * i % longest for i in range(batch - 1)] + [longest], 8, 8, 64, 32, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,window", [
    ([1, 1, 1], [300, 5000, 0], 0), ([1, 0, 3], [2100, 0, 2047], 0), ([2], [20000], 0), ([1, 4], [7000, 9001], 3000)])
def test_attention_few_long_sequences(new, lens, window, dtype):
    """Few tiles: each is shared by clusters of CTAs, in proportion to its length. (A length below its new rows is flagged.)"""
    run_attention(32, new, lens, 8, 2, 128, 64, dtype, window=window, flagged=12 if any(l < n for n, l in zip(new, lens)) else 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gain", [0.0, 1e-30, 30.0, 1e20])
def test_attention_query_magnitudes(gain, dtype):
    """Queries of any size; at 1e20 the softmax is a choice of one token."""
    if gain < 1e10:
        run_attention(8, [1, 2], [70, 90], 8, 2, 128, 16, dtype, q_gain=gain)
        run_attention(9, [140], [180], 8, 2, 128, 16, dtype, q_gain=gain)
    else:
        assert np.isfinite(run_attention(8, [1, 2], [70, 90], 8, 2, 128, 16, dtype, q_gain=gain, check=False)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_any_positive_scale(dtype):
    run_attention(21, [1, 3, 100], [130, 90, 120], 8, 2, 128, 16, dtype, pow2=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_value_scales_far_apart(dtype):
    """Pages of tiny values next to pages of large ones: each keeps its weight in the sum."""
    def spread(c):
        c.scale["v"][:] = (2.0 ** np.resize([-40.0, 0.0, 30.0, -64.0, -3.0], c.scale["v"].size)).reshape(c.scale["v"].shape)
    run_attention(22, [1, 2, 90], [130, 90, 200], 8, 2, 128, 16, dtype, codes_after=spread)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,hq", [([1, 1], [5, 33], 8), ([3], [40], 8), ([80], [100], 8), ([200, 2], [200, 18], 8),
                                         ([80], [100], 64), ([200, 2], [200, 18], 64)])
def test_attention_nan_in_slots_past_the_end(new, lens, hq, dtype):
    page = 16

    def spoil(c):
        at = 0
        for n in lens:
            k = -(-n // page)
            last = c.order[at + k - 1]
            at += k
            for s in "kv":
                c.codes[s][last, :, n - (k - 1) * page:] = 0x7F
    run_attention(sum(lens), new, lens, hq, 2, 128, page, dtype, codes_after=spoil)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,length,window,hq", [(4, 40, 0, 4), (6, 200, 20, 4), (150, 200, 0, 4), (150, 300, 40, 4),
                                                (150, 200, 0, 32), (150, 300, 40, 32)])
def test_attention_nan_reaches_only_the_rows_that_see_it(n, length, window, hq, d, dtype):
    """NaN in one value dim of one token: that dim of the rows that see the token, nothing else;
    NaN in a key: every dim of those rows."""
    page, hk, dim = 16, 2, 5
    lens = [length]
    clean = run_attention(n, [n], lens, hq, hk, d, page, dtype, window)
    for side in "vk":
        for tok in (length - n // 2, length - 1, length - n - 3 if window else length - n + 1):
            def spoil(c):
                c.codes[side][c.order[tok // page], 1, tok % page, dim] = 0xFF
            got = run_attention(n, [n], lens, hq, hk, d, page, dtype, window, codes_after=spoil, check=False)
            pos = np.arange(length - n, length)
            sees = (tok <= pos) & (tok > pos - window if window else True)
            want = np.zeros_like(clean, bool)
            want[sees, hq // hk:, dim if side == "v" else slice(None)] = True
            assert np.array_equal(np.isnan(got), want), (side, tok)
            if side == "v":
                assert np.array_equal(got[~want], clean[~want])
            else:
                assert np.array_equal(got[~sees], clean[~sees]) and np.array_equal(got[:, :hq // hk], clean[:, :hq // hk])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,length,hq", [(1, 40, 4), (1, 9000, 4), (3, 40, 4), (90, 120, 4), (90, 120, 64)])
def test_attention_nan_query(n, length, hq, dtype):
    """A NaN in a query makes its row NaN (not the zero of a row that sees nothing), and no other row."""
    hk, d, page = 2, 64, 16
    c = Cache(1, -(-length // page), hk, page, d)
    c.upload()
    q = rows(np.random.default_rng(1).standard_normal((n, hq * d)), dtype)
    q[n // 2, d + 3] = float("nan")
    out = torch.empty_like(q)
    nbytes = q4k.q4k_paged_attention_workspace_size(1, n, hq, hk, d)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    q4k.q4k_paged_attention(q, n, hq, hk, d, hq * d, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"],
                            dev(np.array([0, n], np.int32)), dev(np.array([length], np.int32)),
                            dev(tables(c, [length])), 1, -(-length // page) + 1, page, c.pages, n, length, 0.125, 0, out,
                            hq * d, ws, nbytes)
    bad = np.isnan(f64(out).reshape(n, hq, d))
    want = np.zeros_like(bad)
    want[n // 2, 1] = True
    assert np.array_equal(bad, want)


def test_attention_results_do_not_depend_on_hints_or_neighbours():
    """Hints choose kernels and grids: a sequence's result stays within the bound whatever they say."""
    for hints in ((1, 1), (300, 100000), (0, 0)):
        run_attention(31, [1, 40, 2], [400, 90, 17], 8, 2, 128, 16, "f32", hints=hints)
        run_attention(32, [1, 140, 2], [400, 190, 17], 8, 2, 128, 16, "bf16", hints=hints)
        run_attention(33, [1, 140, 2], [400, 190, 17], 64, 8, 128, 16, "f32", hints=hints)
        run_attention(34, [1, 140, 2], [400, 190, 17], 64, 8, 128, 16, "bf16", hints=hints)


def test_attention_rows_before_the_sequence_are_zero():
    got = run_attention(3, [4, 2], [2, 0], 8, 2, 128, 16, "f32", flagged=12, table=np.array([[1], [0]], np.int32),
                        cache=Cache(3, 2, 2, 16, 128))
    assert (got[:2] == 0).all() and (got[4:] == 0).all() and (got[2:4] != 0).any()


@pytest.mark.parametrize("new,hq", [([1, 1], 8), ([90, 1], 8), ([90, 1], 64)])
def test_attention_bad_page_ids(new, hq):
    """A page id outside the cache: flagged, its tokens are not seen; the other sequence is right."""
    page, lens = 16, [100, 40]
    c = Cache(6, 12, 2, page, 128)
    table = tables(c, lens)
    good = run_attention(6, new, lens, hq, 2, 128, page, "f32", cache=c, table=table)
    for bad in (-1, 12, 0x7FFFFFFF):
        t = table.copy()
        t[0, 2] = bad
        got = run_attention(6, new, lens, hq, 2, 128, page, "f32", cache=c, table=t, check=False, flagged=11)
        assert np.isfinite(got).all() and np.array_equal(got[new[0]:], good[new[0]:])
        assert not np.array_equal(got[:new[0]], good[:new[0]])


def test_attention_bad_lengths():
    """Lengths past the page table's row are cut to it and flagged."""
    page = 16
    c = Cache(7, 6, 2, page, 128)
    table = np.array([[0, 1]], np.int32)
    run_attention(7, [1], [32], 8, 2, 128, page, "f32", cache=c, table=table)
    got = run_attention(7, [1], [1 << 30], 8, 2, 128, page, "f32", cache=c, table=table, check=False, flagged=12)
    assert np.array_equal(got, run_attention(7, [1], [32], 8, 2, 128, page, "f32", cache=c, table=table))


def test_attention_same_bits_every_call_and_on_another_stream():
    a = run_attention(40, [1, 1, 60], [5000, 70, 64], 8, 2, 128, 32, "f32", check=False)
    b = run_attention(40, [1, 1, 60], [5000, 70, 64], 8, 2, 128, 32, "f32", check=False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c = run_attention(40, [1, 1, 60], [5000, 70, 64], 8, 2, 128, 32, "f32", check=False)
    torch.cuda.current_stream().wait_stream(s)
    assert np.array_equal(a, b) and np.array_equal(a, c)


def test_attention_offsets_past_32_bits():
    """A cache whose last pages lie beyond 2^32 bytes."""
    hk, page, d = 8, 128, 128
    pages = (1 << 32) // (hk * page * d) + 64
    k = torch.zeros((pages, hk, page, d), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.ones((pages, hk), device="cuda")
    vs = torch.ones((pages, hk), device="cuda")
    g = np.random.default_rng(2)
    ids = np.array([[pages - 1, 3, pages - 40]], np.int32)
    small = Cache(9, 3, hk, page, d)
    for i in range(3):
        for full, s in ((k, "k"), (v, "v")):
            full[int(ids[0, i])] = dev(small.codes[s][i])
        ks[int(ids[0, i])] = dev(small.scale["k"][i])
        vs[int(ids[0, i])] = dev(small.scale["v"][i])
    for n, hq, dtype in ((1, hk, "f32"), (160, hk, "f32"), (240, 2 * hk, "f32"), (240, 2 * hk, "bf16")):
        q = rows(g.standard_normal((n, hq * d)), dtype)
        out = torch.empty_like(q)
        nbytes = q4k.q4k_paged_attention_workspace_size(1, n, hq, hk, d)
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        q4k.q4k_paged_attention(q, n, hq, hk, d, hq * d, k, v, ks, vs, dev(np.array([0, n], np.int32)),
                                dev(np.array([300], np.int32)), dev(ids), 1, 3, page, pages, n, 300, 0.09, 0, out,
                                hq * d, ws, nbytes)
        ref, tol = attention_ref(f64(q).reshape(n, hq, d), small, np.array([[0, 1, 2]]), [n], [300], hq // hk, 0.09, 0, dtype)
        assert (np.abs(f64(out).reshape(n, hq, d) - ref) <= tol).all()
    # an append into the last page
    kv = rows(g.standard_normal((1, 2 * hk * d)), "f32")
    q4k.q4k_kv_append(kv, kv[:, hk * d:], 1, hk, d, 2 * hk * d, 2 * hk * d, None, EPS, None, 0, 0,
                      dev(np.array([0, 1], np.int32)), dev(np.array([1], np.int32)),
                      dev(np.array([[pages - 1]], np.int32)), 1, 1, page, pages, k, v, ks, vs)
    got = E4M3[host(v[pages - 1, :, 0])] * host(vs[pages - 1]).astype(np.float64)[:, None]
    x = f64(kv)[0, hk * d:].reshape(hk, d)
    assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * host(vs[pages - 1])[:, None])).all()


def test_decoder_layer_example():
    """Prompts and then single tokens give what the same tokens give in one call, up to the cache's rounding: a page whose
    scale grows under later tokens has its codes rounded twice, by e4m3's 2^-4 at most each, in a sum of many."""
    import sys
    sys.path.insert(0, str(Path(__file__).resolve().parent.parent / "examples"))
    import decoder_layer as ex
    prompts, steps = (5, 33, 130), 4
    xs, out, layer, _ = ex.run(prompts, steps, seed=3, hidden=512, inter=256, experts=4, top_k=4)
    lens = [n + steps for n in prompts]
    cache = ex.Cache(len(lens), max(lens), layer.hk, layer.d)
    cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens])
    y = layer.forward(torch.cat(xs), pos, ex.starts(lens), cache, max(lens), max(lens), layer.buffers(sum(lens), len(lens)))
    layer.check()
    for a, b in zip(y.split(lens), out):
        a, b = f64(a), f64(b)
        assert np.isfinite(a).all()
        assert (np.linalg.norm(a - b, axis=1) <= 2.0 ** -4 * np.linalg.norm(a, axis=1)).all()


def test_the_three_calls_in_a_graph():
    """Append and attend captured once and replayed with new inputs in the same buffers."""
    hq, hk, d, page = 8, 2, 128, 16
    c = Cache(50, 8, hk, page, d)
    c.upload()
    qkv = torch.empty((2, (hq + 2 * hk) * d), device="cuda")
    row = (hq + 2 * hk) * d
    q = torch.empty((2, hq * d), device="cuda")
    out = torch.empty_like(q)
    f, pos = dev(freqs(d)), dev(np.array([20, 40], np.int32))
    w = dev(inputs.to_bf16_bits(np.ones(d, np.float32)).view(np.int16))
    lens, start, table = dev(np.array([21, 41], np.int32)), dev(np.array([0, 1, 2], np.int32)), dev(np.arange(6, dtype=np.int32).reshape(2, 3))
    nbytes = q4k.q4k_paged_attention_workspace_size(2, 2, hq, hk, d)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def step():
        q4k.q4k_qk_norm_rope(qkv, None, 2, hq, 0, d, row, row, w, None, EPS, pos, f, d, 0, q, None, hq * d, hq * d)
        q4k.q4k_kv_append(qkv[:, hq * d:], qkv[:, (hq + hk) * d:], 2, hk, d, row, row, w, EPS, f, d, 0, start, lens,
                          table, 2, 3, page, 8, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"])
        q4k.q4k_paged_attention(q, 2, hq, hk, d, hq * d, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"],
                                start, lens, table, 2, 3, page, 8, 1, 48, 0.09, 0, out, hq * d, ws, nbytes)

    qkv.normal_()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        qkv.normal_()
        keep = [t.clone() for t in (*c.dev.values(), *c.dev_scale.values())]
        graph.replay()
        got = out.clone()
        for t, k in zip((*c.dev.values(), *c.dev_scale.values()), keep):
            t.copy_(k)
        step()
        assert torch.equal(got, out)


# ---- one sequence over a long cache --------------------------------------------------------------

class LongCache:
    """One sequence's pages in a cache made on the device: random codes (no NaN) and power-of-two scales."""

    def __init__(self, seed, length, heads, page, d):
        g = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.page, self.d, self.length = heads, page, d, length
        self.pages = -(-length // page) + 1
        shape = (self.pages, heads, page, d)
        self.codes = {s: (torch.randn(shape, generator=g, device="cuda") * 60).clamp(-440, 440).to(torch.float8_e4m3fn)
                      for s in "kv"}
        self.scale = {s: torch.ldexp(torch.ones((), device="cuda"), torch.randint(lo, lo + 4, shape[:2], generator=g, device="cuda"))
                      for s, lo in (("k", -9), ("v", -10))}
        self.table = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32)[None, :-1].contiguous()

    def values(self, side):
        """[heads, length, d] in fp64, on the device."""
        ids = self.table[0].long()
        v = self.codes[side].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * self.scale[side][ids].double()[..., None, None]
        return v.transpose(0, 1).reshape(self.heads, -1, self.d)[:, :self.length]


def long_attention_ref(q, cache, n, group, scale, dtype):
    """attention_ref for one sequence's last n tokens, on the device: (result, bound), [n, q_heads, d]."""
    d, length = cache.d, cache.length
    q = q.double().view(n, -1, d)
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    k, v = cache.values("k"), cache.values("v")
    for r in range(n):
        seen = length - n + r + 1
        for h in range(q.shape[1]):
            kk, vv = k[h // group, :seen], v[h // group, :seen]
            s = kk @ q[r, h] * scale
            p = torch.softmax(s, 0)
            ds = scale * (kk.abs() @ q[r, h].abs()).max() * (2.0 ** -22 + (d / 16 + 8) * 2.0 ** -23)
            x = (s.abs().max() * 1.45 + 64 + 14) * 2.0 ** -23 + 2.0 ** -22
            rel = 2 * (ds + x) + (seen / 64 + 40) * U + (2.0 ** -11 * 1.01 if dtype == "bf16" else 0.0)
            out[r, h] = p @ vv
            tol[r, h] = rel * (p @ vv.abs()) + STEP[dtype] * out[r, h].abs() * 1.01
    return out, tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hk", [1, 2, 3])
@pytest.mark.parametrize("n,length", [(1, 34816), (1, 40000), (2, 131071)])
def test_attention_one_sequence_over_a_long_cache(n, length, hk, d, dtype):
    """Few tiles and a long axis: more than sixteen clusters share a tile and join it in two levels. The same bits each time."""
    group, page = 4, 64
    c = LongCache(length + hk, length, hk, page, d)
    q = rows(np.random.default_rng(length + d).standard_normal((n, group * hk * d)), dtype)
    scale, nbytes = 1 / math.sqrt(d), q4k.q4k_paged_attention_workspace_size(1, n, group * hk, hk, d)
    start, lens = dev(np.array([0, n], np.int32)), dev(np.array([length], np.int32))
    flag, got = err_flag(), []
    for fill in (0xFF, 0, 0x55):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(20):
            out = torch.full_like(q, 7.0)
            q4k.q4k_paged_attention(q, n, group * hk, hk, d, group * hk * d, c.codes["k"], c.codes["v"], c.scale["k"], c.scale["v"],
                                    start, lens, c.table, 1, c.table.shape[1], page, c.pages, n, length, scale, 0, out,
                                    group * hk * d, ws, nbytes, flag)
            got.append(out)
    assert int(host(flag)[0]) == 0
    assert all(torch.equal(got[0], x) for x in got[1:])
    ref, tol = long_attention_ref(q, c, n, group, scale, dtype)
    worst = float(((got[0].double().view_as(ref) - ref).abs() / tol).max())
    assert worst <= 1, f"{worst} of the bound"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,page,n,length", [(64, 16, 60, 4003), (128, 16, 61, 4003), (128, 128, 63, 9001)])
def test_attention_prompt_over_many_tiles(d, page, n, length, dtype):
    """The prompt kernels' rings of pages and slots turn over many times. The same bits each time."""
    group, hk = 8, 8
    c = LongCache(length + d, length, hk, page, d)
    q = rows(np.random.default_rng(length + d).standard_normal((n, group * hk * d)), dtype)
    scale, nbytes = 1 / math.sqrt(d), q4k.q4k_paged_attention_workspace_size(1, n, group * hk, hk, d)
    ws, flag, got = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), err_flag(), []
    start, lens = dev(np.array([0, n], np.int32)), dev(np.array([length], np.int32))
    for _ in range(10):
        out = torch.full_like(q, 7.0)
        q4k.q4k_paged_attention(q, n, group * hk, hk, d, group * hk * d, c.codes["k"], c.codes["v"], c.scale["k"], c.scale["v"],
                                start, lens, c.table, 1, c.table.shape[1], page, c.pages, n, length, scale, 0, out,
                                group * hk * d, ws, nbytes, flag)
        got.append(out)
    assert int(host(flag)[0]) == 0
    assert all(torch.equal(got[0], x) for x in got[1:])
    ref, tol = long_attention_ref(q, c, n, group, scale, dtype)
    worst = float(((got[0].double().view_as(ref) - ref).abs() / tol).max())
    assert worst <= 1, f"{worst} of the bound"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_prompt_wait_limit_runs_out(d, dtype, monkeypatch):
    """Short wait limits (Q4K_WAIT_NS) make the prompt kernels' roles give up at different places: they leave together, the
    products under way finish before tensor memory is freed, Q4K_ERR_TIMEOUT is in the device flag, and the next call
    with the default limit is right. A call that no wait of ran out is right too."""
    n, length, hq, hk, page = 300, 1500, 32, 4, 32
    c = LongCache(d, length, hk, page, d)
    q = rows(np.random.default_rng(d).standard_normal((n, hq * d)), dtype)
    nbytes = q4k.q4k_paged_attention_workspace_size(1, n, hq, hk, d)
    ws, start, lens = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), dev(np.array([0, n], np.int32)), dev(np.array([length], np.int32))

    def call():
        out, flag = torch.full_like(q, 7.0), err_flag()
        q4k.q4k_paged_attention(q, n, hq, hk, d, hq * d, c.codes["k"], c.codes["v"], c.scale["k"], c.scale["v"], start, lens,
                                c.table, 1, c.table.shape[1], page, c.pages, n, length, 0.1, 0, out, hq * d, ws, nbytes, flag)
        return out, int(host(flag)[0])

    good, status = call()
    assert status == 0
    for limit in (1, 200, 500, 1000, 2000, 4000, 8000, 20000, 100000):
        monkeypatch.setenv("Q4K_WAIT_NS", str(limit))
        for _ in range(3):
            out, status = call()
            assert status == 10 or (status == 0 and limit > 1 and torch.equal(out, good)), limit
        monkeypatch.delenv("Q4K_WAIT_NS")
        out, status = call()
        assert status == 0 and torch.equal(out, good)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gain", [1e5, 1e7, 1e9, 1e20])
def test_attention_prompt_query_magnitudes(gain, d, dtype):
    """Scores so large that the softmax is a choice of one token: its values, no NaN."""
    new, lens, hq, hk, page = [60], [200], 64, 8, 16
    c = Cache(77, 14, hk, page, d)
    table = tables(c, lens)
    got = run_attention(77, new, lens, hq, hk, d, page, dtype, q_gain=gain, check=False, cache=c, table=table)
    q = f64(rows(np.random.default_rng(77).standard_normal((60, hq * d)) * gain, dtype)).reshape(60, hq, d)
    k, v = (c.values(s, table[0, :13], 200) for s in "kv")
    apart = 0
    for r in range(60):
        for h in range(hq):
            s = np.sort(np.stack([k[h // 8, :141 + r] @ q[r, h], np.arange(141 + r)], 1).view("f8,f8"), axis=0, order="f0")
            top, second = s["f0"][-1, 0], s["f0"][-2, 0]
            off = (d / 16 + 8) * 2.0 ** -22 * (np.abs(k[h // 8, :141 + r]) @ np.abs(q[r, h])).max()
            if (top - second - 2 * off) / math.sqrt(d) < 40:  # e^-40 of the others' values is below a rounding
                continue
            apart += 1
            want = v[h // 8, int(s["f1"][-1, 0])]
            assert (np.abs(got[r, h] - want) <= (STEP[dtype] + 2.0 ** -11) * np.abs(want) + 2.0 ** -40).all()
    assert apart > 1000 and np.isfinite(got).all()


# ---- a dominant token whose value is zero ---------------------------------------------------------
# The weights p_j enter the product with V as P_j = 2^B p_j s_j / W, s_j the V scale of j's page, W the largest p_j s_j. An
# fp16 term is off by 2^-11 P_j, or 2^-25 below fp16's normal numbers; the second term of fp32 rows is held times 2^11, so
# both together are off by 2^-22 P_j or 2^-36. B is 15; 9 in the prompt kernel for bf16. So sum_j |dp_j| |v_j| is at most
# 2^-22 or 2^-11 of sum_j p_j |v_j|, plus 2^-36 or 2^-25 times 2^-B W sum_j |code_j|.

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,length,hq,hk,d", [(1, 300, 8, 2, 128), (2, 9000, 4, 1, 64), (60, 400, 64, 8, 128), (65, 333, 64, 8, 64)])
@pytest.mark.parametrize("nats", [12.0, 16.0, 20.0])
@pytest.mark.parametrize("up", [0, 6])
def test_attention_dominant_token_without_value(up, nats, n, length, hq, hk, d, dtype):
    """A sink: the first token's score is `nats` above the others' and its values are zero, so the result is made of weights
    of e^-nats; its page's V scale is 2^up times the others'."""
    g = np.random.default_rng(int(nats) + length)
    page, scale = 16, 1 / math.sqrt(d)
    c = Cache(length + d, -(-length // page), hk, page, d)
    c.scale["k"][:], c.scale["v"][:] = 2.0 ** -7, 2.0 ** -6
    table = c.order[None, :].copy()
    u = g.choice([-1.0, 1.0], (hk, d))
    c.codes["k"][table[0, 0], :, 0] = e4m3_round(u * 128)  # K of the first token: u
    c.codes["v"][table[0, 0], :, 0] = 0
    c.scale["v"][table[0, 0]] *= 2.0 ** up
    c.upload()
    q = np.repeat(u, hq // hk, 0) * nats / math.sqrt(d) + 0.5 * g.standard_normal((n, hq, d))
    q = rows(q.reshape(n, hq * d), dtype)
    out, flag = torch.empty_like(q), err_flag()
    nbytes = q4k.q4k_paged_attention_workspace_size(1, n, hq, hk, d)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    q4k.q4k_paged_attention(q, n, hq, hk, d, hq * d, c.dev["k"], c.dev["v"], c.dev_scale["k"], c.dev_scale["v"],
                            dev(np.array([0, n], np.int32)), dev(np.array([length], np.int32)), dev(table), 1, table.shape[1],
                            page, c.pages, n, length, scale, 0, out, hq * d, ws, nbytes, flag)
    assert int(host(flag)[0]) == 0
    qs = f64(q).reshape(n, hq, d)
    ref, tol = attention_ref(qs, c, table, [n], [length], hq // hk, scale, 0, dtype)
    k, codes = c.values("k", table[0], length), np.abs(E4M3[c.codes["v"][table[0]]]).transpose(1, 0, 2, 3).reshape(hk, -1, d)
    s_v = np.repeat(c.scale["v"][table[0]].T.astype(np.float64), page, 1)  # [hk, tokens]
    bits = 36 + 15 if dtype == "f32" else 25 + (9 if n > 8 else 15)
    least = 1.0
    for r in range(n):
        seen = length - n + r + 1
        for h in range(hq):
            x = k[h // (hq // hk), :seen] @ qs[r, h] * scale
            p = np.exp(x - x.max())
            p /= p.sum()
            least = min(least, p[0])
            floor = 2.0 ** -bits * (p * s_v[h // (hq // hk), :seen]).max() * codes[h // (hq // hk), :seen].sum(0)
            weight = 2.0 ** -22 * (p @ (codes[h // (hq // hk), :seen] * s_v[h // (hq // hk), :seen, None])) if dtype == "f32" else 0.0
            tol[r, h] += floor + weight
    assert least > 0.5  # the sink dominates every row
    worst = np.max(np.abs(f64(out).reshape(n, hq, d) - ref) / np.maximum(tol, 1e-300))
    assert worst <= 1, f"{worst} of the bound"


# ---- append: several heads a CTA -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,ctx,heads,d,page,kw", [
    ([4003], [37], 8, 128, 16, {}), ([1800, 3], [5, 0], 5, 64, 16, dict(mode="pairs")), ([2500, 0, 1400], [9, 3, 31], 8, 64, 32, {}),
    ([8191], [37], 8, 128, 64, {}), ([8000], [63], 5, 128, 64, dict(rot=64)), ([14001], [100], 3, 128, 128, dict(gain=30.0, norm=False)),
    ([2600], [11], 8, 64, 16, dict(rot=0, norm=False)),
])
def test_append_prompts_of_several_heads(new, ctx, heads, d, page, kw, dtype):
    """Prompts of so many pages that a CTA takes a page's heads one after the other, all of them or a share that may be the
    smaller one, behind a prefix that ends inside a page, whose codes are rounded again for every head."""
    run_append(sum(new) + heads, new, ctx, heads, d, page, dtype, **kw)


# ---- V scales at the ends of their range ----------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,hq,hk,d", [([1, 2], [130, 90], 8, 2, 128), ([1], [5000], 8, 1, 64), ([60], [200], 64, 8, 128), ([60], [200], 64, 8, 64)])
@pytest.mark.parametrize("exps", [[-80], [-80, 16], [16, -80, -30]])
def test_attention_value_scales_at_the_ends(exps, new, lens, hq, hk, d, dtype):
    """(attention_ref's bound for x allows two roundings of values below 128 in log2 units.)"""
    def ends(c):
        c.scale["v"][:] = (2.0 ** np.resize(np.array(exps, float), c.scale["v"].size)).reshape(c.scale["v"].shape)
    run_attention(60 + len(exps), new, lens, hq, hk, d, 16, dtype, codes_after=ends)
