"""Cases that measure the attention half of a decoder layer: the per-head norm with the position
rotation, the append to a paged 8-bit cache, and attention over that cache.

`own` selects what `run` does: False computes each operator in a plain form from elementary torch
operations, True calls the library. Everything else is shared: the cases (`listed`, `draw`), the
inputs (`prepare`), the work each cannot do without (`work`) and the results in 64 bits (`exact`).

The cache: codes in float8_e4m3fn, [num_pages, kv_heads, page_size, head_dim], one power-of-two
scale per (page, kv head) in fp32; value = code * scale. A sequence's tokens lie in the pages of
its page table row, in order. New tokens of sequence i are rows q_start[i] .. q_start[i+1] of the
inputs and the last tokens of its seq_lens[i] cached ones.
"""
import math
import random

import numpy as np
import torch

own = False

THETA = 1.0e6
EPS = 1.0e-6
E4M3_MAX = 448.0
MIN_EXP = -64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


# ---- cases -------------------------------------------------------------------------------------

def _norm(name, tokens, q_heads, kv_heads, dim, dtype, rot, mode, pos_max):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "rot": rot, "mode": mode, "pos_max": pos_max}


def _append(name, batch, q_lo, q_hi, ctx_lo, ctx_hi, kv_heads, dim, page, dtype, rot, mode, lens):
    return {"name": name, "op": "append", "batch": batch, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "rot": rot, "mode": mode, "lens": lens}


def _attn(name, batch, q_lo, q_hi, ctx_lo, ctx_hi, q_heads, kv_heads, dim, page, dtype, window, lens):
    return {"name": name, "op": "attention", "batch": batch, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "window": window, "lens": lens}


def listed():
    return [
        # one sequence's decode step: latency
        _norm("norm_rope_token", 1, 32, 4, 128, "f32", 128, "halves", 40000),
        # an odd decode batch, short heads, rotation of half of each head in neighbouring pairs
        _norm("norm_rope_batch_partial", 61, 12, 2, 64, "bf16", 32, "pairs", 130000),
        # a whole prompt, read out of the fused projection's rows
        _norm("norm_rope_prompt", 8192, 32, 8, 128, "bf16", 128, "halves", 8192),
        # one sequence's decode step: latency, a partly filled page
        _append("append_token", 1, 1, 1, 776, 776, 4, 128, 16, "f32", 128, "halves", 1),
        # a large decode batch of ragged sequences: every page partly filled or new
        _append("append_batch", 256, 1, 1, 1, 2000, 8, 128, 32, "f32", 128, "halves", 2),
        # a prompt behind a cached prefix that ends inside a page
        _append("append_prompt", 1, 8191, 8191, 37, 37, 8, 128, 64, "bf16", 128, "halves", 3),
        # one sequence's decode step with a short context: latency
        _attn("attn_token_short", 1, 1, 1, 508, 508, 32, 4, 128, 16, "f32", 0, 4),
        # one sequence's decode step with a long context: the axis has to be split
        _attn("attn_token_long", 1, 1, 1, 131070, 131070, 32, 4, 128, 64, "f32", 0, 5),
        # a ragged decode batch
        _attn("attn_batch", 64, 1, 1, 1, 8191, 32, 8, 128, 32, "bf16", 0, 6),
        # a few tokens a sequence to verify, an odd group of heads, a sliding window
        _attn("attn_few_window", 9, 1, 6, 200, 6000, 14, 2, 64, 16, "f32", 1024, 7),
        # a prompt from nothing
        _attn("attn_prompt", 1, 8192, 8192, 0, 0, 32, 8, 128, 64, "bf16", 0, 8),
        # prompts in chunks of odd sizes behind cached ones, together with sequences that decode
        _attn("attn_chunks", 6, 1, 700, 0, 6000, 16, 2, 128, 128, "f32", 0, 9),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attention", "attention"])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["f32", "bf16"])
    kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    rot = rng.choice([dim, dim, dim // 2])
    mode = rng.choice(["halves", "halves", "pairs"])
    lens = rng.randrange(1 << 30)
    if op == "norm_rope":
        group = rng.choice([1, 4, 7, 8])
        c = _norm("", _log_int(rng, 1, 8191), min(32, kv * group), kv, dim, dtype, rot, mode, rng.choice([4000, 40000, 130000]))
        del c["name"]
        return c
    if op == "append":
        if rng.random() < 0.5:  # decode
            batch, q_lo, q_hi, ctx = _log_int(rng, 1, 256), 1, 1, _log_int(rng, 1, 2000)
        else:                   # prompts
            batch, q_lo, q_hi, ctx = _log_int(rng, 1, 6), 1, _log_int(rng, 20, 1300), _log_int(rng, 1, 500)
        c = _append("", batch, q_lo, q_hi, 0, ctx, kv, dim, page, dtype, rot, mode, lens)
        del c["name"]
        return c
    q_heads = min(32, kv * rng.choice([1, 2, 3, 4, 7, 8, 16]) if kv < 8 else kv * rng.choice([1, 2, 4]))
    window = rng.choice([0, 0, 0, 128, 1000])
    kind = rng.choice(["decode", "decode", "few", "prompt"])
    if kind == "decode":
        batch = _log_int(rng, 1, 64)
        c = _attn("", batch, 1, 1, 0, min(131070, _log_int(rng, 16, 400000 // batch)), q_heads, kv, dim, page, dtype, window, lens)
    elif kind == "few":
        c = _attn("", _log_int(rng, 1, 24), 1, rng.randint(2, 9), 0, _log_int(rng, 16, 7000), q_heads, kv, dim, page, dtype, window, lens)
    else:
        q_hi = _log_int(rng, 20, 2500)
        batch = rng.randint(1, 4) if q_hi < 900 else 1
        c = _attn("", batch, max(1, q_hi // 3), q_hi, 0, _log_int(rng, 1, 4000), q_heads, kv, dim, page, dtype, window, lens)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, cached tokens after them) of each sequence: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    new, total = [], []
    for _ in range(case["batch"]):
        q = r.randint(case["q_lo"], case["q_hi"])
        new.append(q)
        total.append(q + r.randint(case["ctx_lo"], case["ctx_hi"]))
    return new, total


def _visible(case):
    """(query, key) pairs a head computes, and the cached tokens that some query sees."""
    new, total = _lengths(case)
    w, pairs, seen = case["window"], 0, 0
    for n, length in zip(new, total):
        first = length - n
        pos = np.arange(first, length)
        pairs += int(np.minimum(pos + 1, w if w else length).sum())
        seen += length - (max(0, first - w + 1) if w else 0)
    return pairs, seen


def work(case):
    d, size = case["dim"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm_rope":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * d
        return {"bytes": 2 * n * size + case["tokens"] * 4, "flops": 7 * n}
    new, total = _lengths(case)
    if case["op"] == "append":
        n = sum(new) * case["kv_heads"] * d
        pages = sum((t + case["page"] - 1) // case["page"] - (t - n_) // case["page"] for n_, t in zip(new, total))
        return {"bytes": 2 * n * size + 2 * n + pages * case["kv_heads"] * 2 * 4, "flops": 12 * n}
    pairs, seen = _visible(case)
    rows = sum(new) * case["q_heads"] * d
    pages = (seen + case["page"] - 1) // case["page"]
    return {"bytes": 2 * rows * size + 2 * seen * case["kv_heads"] * d + pages * case["kv_heads"] * 8,
            "flops": 4 * d * case["q_heads"] * pairs}


# ---- inputs ------------------------------------------------------------------------------------

def _exponent(amax):
    """The least e >= MIN_EXP with amax <= 448 * 2^e (64 bits)."""
    f, a = torch.frexp(amax.double())   # amax = f * 2^a, f in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(f <= 0.875, a - 9, a - 8)
    return torch.where(amax > 0, e.clamp_min(MIN_EXP), torch.full_like(e, MIN_EXP))


def _filled_cache(values):
    """Codes and scales of pages [num_pages, kv_heads, page, dim] of values."""
    e = _exponent(values.abs().amax(dim=(2, 3)))
    scale = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e).float()
    return (values / scale[:, :, None, None]).to(F8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    dt, d, hkv = DTYPES[case["dtype"]], case["dim"], case["kv_heads"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    s = {"case": dict(case), "flag": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] != "attention":
        half = case["rot"] // 2
        s["inv_freq"] = THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s["w_q"] = (1 + 0.1 * randn(d)).to(torch.bfloat16)
        s["w_k"] = (1 + 0.1 * randn(d)).to(torch.bfloat16)
        m = case["tokens"] if case["op"] == "norm_rope" else sum(_lengths(case)[0])
        # the rows of a fused projection, heads side by side (queries then keys, or keys then values), some dims larger
        heads = hkv + (case["q_heads"] if case["op"] == "norm_rope" else hkv)
        s["x"] = (randn(m, heads, d) * torch.exp(0.5 * randn(1, heads, d))).to(dt).reshape(m, -1)
        if case["op"] == "norm_rope":
            first = torch.randint(0, max(1, case["pos_max"] - m + 1), (1,), generator=g, device="cuda")
            if m <= 256:   # a decode batch: each token has a position of its own
                s["pos"] = torch.randint(0, case["pos_max"], (m,), generator=g, device="cuda").to(torch.int32)
            else:          # a prompt
                s["pos"] = (first + torch.arange(m, device="cuda")).to(torch.int32)
            return s
    new, total = _lengths(case)
    page = case["page"]
    counts = [(t + page - 1) // page for t in total]
    pool = sum(counts) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["batch"], max(counts)), -1, dtype=torch.int32)
    ids, at = order.cpu(), 0
    for i, n in enumerate(counts):
        table[i, :n] = ids[at:at + n]
        at += n
    s["table"] = table.cuda()
    s["seq_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    s["pages"], s["m"], s["max_q"], s["max_len"] = pool, sum(new), max(new), max(total)
    # cached keys: some dims much larger than others; cached values: tokens of different size
    s["k_cache"], s["k_scale"] = _filled_cache(randn(pool, hkv, page, d) * torch.exp(0.4 * randn(1, hkv, 1, d)))
    s["v_cache"], s["v_scale"] = _filled_cache(randn(pool, hkv, page, d) * torch.exp(0.7 * randn(pool, hkv, page, 1)))
    if case["op"] == "attention":
        s["q"] = (1.3 * randn(s["m"], case["q_heads"] * d)).to(dt)
        s["scale"] = 1.0 / math.sqrt(d)
    return s


# ---- the plain form ----------------------------------------------------------------------------

def _norm_rope_plain(x, w, pos, inv_freq, mode):
    """x [m, heads, d] in fp32 or 64 bits, in that type."""
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)
    half = inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq
    c, s = torch.cos(angle).to(x.dtype)[:, None], torch.sin(angle).to(x.dtype)[:, None]
    r = y[..., :2 * half]
    if mode == "halves":
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([r, y[..., 2 * half:]], -1)


def _plain_norm_rope(s):
    c = s["case"]
    m, hq, hkv, d = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    x = s["x"].view(m, hq + hkv, d).float()
    q = _norm_rope_plain(x[:, :hq], s["w_q"], s["pos"], s["inv_freq"], c["mode"])
    k = _norm_rope_plain(x[:, hq:], s["w_k"], s["pos"], s["inv_freq"], c["mode"])
    dt = s["x"].dtype
    return {"q": q.to(dt).reshape(m, -1), "k": k.to(dt).reshape(m, -1)}


def _rows(s):
    """Sequence and position of each new token."""
    t = torch.arange(s["m"], device="cuda")
    seq = torch.searchsorted(s["q_start"].long(), t, right=True) - 1
    start = s["q_start"].long()
    pos = s["seq_lens"].long()[seq] - start[seq + 1] + t
    return seq, pos


def _append_plain(cache, scale, x, page_of, slot):
    """Cache and scales after x [m, kv_heads, d] (64 bits) went to (page_of, slot)."""
    pages, heads = scale.shape
    page_size = cache.shape[2]
    index = page_of[:, None].expand(-1, heads)
    amax = torch.zeros(pages, heads, dtype=torch.float64, device="cuda")
    amax.scatter_reduce_(0, index, x.abs().amax(-1), "amax")
    held = torch.full((pages,), page_size, device="cuda").scatter_reduce_(0, page_of, slot, "amin")
    touched = torch.zeros(pages, dtype=torch.bool, device="cuda").index_fill_(0, page_of, True)
    fresh = torch.ldexp(torch.ones_like(amax), _exponent(amax)).float()
    grown = torch.where((held == 0)[:, None], fresh, torch.maximum(scale, fresh))
    new_scale = torch.where(touched[:, None], grown, scale)
    # tokens that a touched page held already, at the new scale
    old = touched[:, None] & (torch.arange(page_size, device="cuda") < held[:, None])
    again = (cache.float() * (scale / new_scale)[:, :, None, None]).to(F8)
    codes = torch.where(old[:, None, :, None], again.view(torch.uint8), cache.view(torch.uint8))
    unit = new_scale.double()[page_of][:, :, None]
    codes[page_of, :, slot] = (x / unit).clamp(-E4M3_MAX, E4M3_MAX).float().to(F8).view(torch.uint8)
    return codes.view(F8), new_scale


def _plain_append(s):
    c = s["case"]
    hkv, d, page = c["kv_heads"], c["dim"], c["page"]
    seq, pos = _rows(s)
    page_of = s["table"].long()[seq, pos // page]
    slot = pos % page
    x = s["x"].view(s["m"], 2 * hkv, d).double()
    k = _norm_rope_plain(x[:, :hkv], s["w_k"], pos, s["inv_freq"], c["mode"])
    kc, ks = _append_plain(s["k_cache"], s["k_scale"], k, page_of, slot)
    vc, vs = _append_plain(s["v_cache"], s["v_scale"], x[:, hkv:], page_of, slot)
    return {"k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs}


def _plain_attention(s):
    c = s["case"]
    hq, hkv, d, page, b = c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["batch"]
    group, width, length = hq // hkv, s["max_q"], s["table"].shape[1] * page
    table = s["table"].long().clamp_min(0)
    col = torch.arange(length, device="cuda")
    held = (col < s["seq_lens"][:, None])[:, None, :, None]

    def tokens(cache, scale):  # [b, kv_heads, length, d] in fp32, zero past each sequence's end
        x = cache.view(torch.uint8)[table].view(F8).float() * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(b, hkv, length, d).masked_fill_(~held, 0.0)

    seq, pos = _rows(s)
    row = torch.arange(s["m"], device="cuda") - s["q_start"].long()[seq]
    q = torch.zeros(b, width, hq, d, device="cuda")
    q[seq, row] = s["q"].view(s["m"], hq, d).float()
    at = torch.full((b, width), -1, dtype=torch.long, device="cuda")
    at[seq, row] = pos
    q = q.view(b, width, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * width, d)
    x = torch.matmul(q, tokens(s["k_cache"], s["k_scale"]).transpose(2, 3)).view(b, hkv, group, width, length)
    keep = col <= at[..., None]
    if c["window"]:
        keep &= col > at[..., None] - c["window"]
    x.mul_(s["scale"]).masked_fill_(~keep[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hkv, group * width, length), tokens(s["v_cache"], s["v_scale"]))
    o = o.view(b, hkv, group, width, d) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, width, hq * d)
    return o[seq, row].to(s["q"].dtype)


# ---- the library's form ------------------------------------------------------------------------

def _own_norm_rope(s):
    import bit_quantized_moe_q4k_gb300 as q4k
    c = s["case"]
    m, hq, hkv, d = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    row = (hq + hkv) * d
    q_out = torch.empty(m, hq * d, dtype=s["x"].dtype, device="cuda")
    k_out = torch.empty(m, hkv * d, dtype=s["x"].dtype, device="cuda")
    q4k.q4k_qk_norm_rope(s["x"], s["x"][:, hq * d:], m, hq, hkv, d, row, row, s["w_q"], s["w_k"], EPS,
                         s["pos"], s["inv_freq"], c["rot"], q4k.ROPE_HALVES if c["mode"] == "halves" else
                         q4k.ROPE_PAIRS, q_out, k_out, hq * d, hkv * d)
    return {"q": q_out, "k": k_out}


def _own_append(s):
    import bit_quantized_moe_q4k_gb300 as q4k
    c = s["case"]
    hkv, d = c["kv_heads"], c["dim"]
    q4k.q4k_kv_append(s["x"], s["x"][:, hkv * d:], s["m"], hkv, d, 2 * hkv * d, 2 * hkv * d,
                      s["w_k"], EPS, s["inv_freq"], c["rot"], q4k.ROPE_HALVES if c["mode"] == "halves" else
                      q4k.ROPE_PAIRS, s["q_start"], s["seq_lens"], s["table"], c["batch"], s["table"].shape[1],
                      c["page"], s["pages"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["flag"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _own_attention(s):
    import bit_quantized_moe_q4k_gb300 as q4k
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["dim"]
    if "workspace" not in s:  # kept by the program between its calls
        n = q4k.q4k_paged_attention_workspace_size(c["batch"], s["m"], hq, hkv, d)
        s["workspace"], s["workspace_bytes"] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
    out = torch.empty_like(s["q"])
    q4k.q4k_paged_attention(s["q"], s["m"], hq, hkv, d, hq * d, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                            s["q_start"], s["seq_lens"], s["table"], c["batch"], s["table"].shape[1], c["page"],
                            s["pages"], s["max_q"], s["max_len"], s["scale"], c["window"], out, hq * d, s["workspace"],
                            s["workspace_bytes"], s["flag"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "append": _own_append, "attention": _own_attention}[op](state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append, "attention": _plain_attention}[op](state)


# ---- in 64 bits --------------------------------------------------------------------------------

def _rotated(x, w, pos, inv_freq, mode):
    """One head's rows in 64 bits: the norm, then each pair of dims as a complex number turned by its angle."""
    x = x.double()
    x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    n = inv_freq.numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * inv_freq[None])
    out = x.clone()
    first, second = (slice(0, n), slice(n, 2 * n)) if mode == "halves" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    z = torch.complex(x[:, first].contiguous(), x[:, second].contiguous()) * turn
    out[:, first], out[:, second] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    hkv, d = case["kv_heads"], case["dim"]
    hq = case.get("q_heads", 0)
    if case["op"] == "norm_rope":
        m = case["tokens"]
        heads = [_rotated(s["x"][:, h * d:(h + 1) * d], s["w_q"] if h < hq else s["w_k"], s["pos"], s["inv_freq"],
                          case["mode"]) for h in range(hq + hkv)]
        return {"q": torch.cat(heads[:hq], 1).reshape(m, -1), "k": torch.cat(heads[hq:], 1).reshape(m, -1)}
    new, total = _lengths(case)
    table = s["table"].cpu().numpy()
    page = case["page"]
    if case["op"] == "append":
        out = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double(), "k_scale": s["k_scale"].double(),
               "v_scale": s["v_scale"].double()}
        row = 0
        for i, (n, length) in enumerate(zip(new, total)):
            x = s["x"][row:row + n].double().view(n, -1, d)
            pos = torch.arange(length - n, length, device="cuda")
            kv = {"k": torch.stack([_rotated(x[:, h], s["w_k"], pos, s["inv_freq"], case["mode"])
                                    for h in range(hkv)]), "v": x[:, hkv:].transpose(0, 1)}
            for p in range((length - n) // page, (length + page - 1) // page):
                lo, hi = max(length - n, p * page), min(length, (p + 1) * page)
                pid = int(table[i, p])
                for side in "kv":
                    part = kv[side][:, lo - (length - n):hi - (length - n)]
                    codes, scale = out[side + "_cache"][pid], out[side + "_scale"][pid]
                    unit = torch.ldexp(torch.ones_like(scale), _exponent(part.abs().amax(dim=(1, 2))))
                    held = lo - p * page
                    if held:
                        unit = torch.maximum(unit, scale)
                        codes[:, :held] *= (scale / unit)[:, None, None]
                    codes[:, held:hi - p * page] = part / unit[:, None, None]
                    out[side + "_scale"][pid] = unit
            row += n
        return out
    out = torch.zeros(s["m"], hq, d, dtype=torch.float64, device="cuda")
    row = 0
    for i, (n, length) in enumerate(zip(new, total)):
        ids = torch.from_numpy(table[i, :(length + page - 1) // page]).long().cuda()
        k = (s["k_cache"].view(torch.uint8)[ids].view(F8).double() * s["k_scale"][ids].double()[..., None, None])
        v = (s["v_cache"].view(torch.uint8)[ids].view(F8).double() * s["v_scale"][ids].double()[..., None, None])
        pos = torch.arange(length - n, length, device="cuda")[:, None]
        col = torch.arange(length, device="cuda")[None]
        bias = torch.zeros(n, length, dtype=torch.float64, device="cuda")
        bias[(col > pos) | ((col <= pos - case["window"]) if case["window"] else (col < 0))] = -math.inf
        for h in range(hq):
            kh, vh = (t[:, h * hkv // hq].reshape(-1, d)[:length] for t in (k, v))
            a = torch.softmax(s["q"][row:row + n].view(n, hq, d)[:, h].double() @ kh.T * s["scale"] + bias, -1)
            out[row:row + n, h] = a @ vh
        row += n
    return out.view(s["m"], -1)

