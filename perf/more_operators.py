"""Cases that measure a serving step's operators around the paged cache: page tables built on the device
from the sequences' lengths, attention for sequences that share a prefix, and the verification of drafted
tokens against the target's distribution.

`own` selects what `run` does: False computes each operator in a plain form from elementary torch
operations, True calls the library. Everything else is shared: the cases (`listed`, `draw`), the
inputs (`prepare`), the work each cannot do without (`work`) and the results in 64 bits (`exact`).

A batch: sequence i's new tokens are rows q_start[i] .. q_start[i+1] - 1 and the last of its seq_lens[i]
cached ones; token j lies in page page_table[i][j // page], slot j % page.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
F32_MAX = 3.4028234663852886e38
GREEDY = 2.0 ** -64   # temperatures not above this choose the largest logit


# ---- cases -------------------------------------------------------------------------------------

def _tables(name, batch, new_lo, new_hi, kept_hi, back, fixed_hi, ended, page, pad, short, lens):
    return {"name": name, "op": "tables", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "kept_hi": kept_hi,
            "back": back, "fixed_hi": fixed_hi, "ended": ended, "page": page, "pad": pad, "short": short, "lens": lens}


def _prefix(name, groups, seqs_lo, seqs_hi, prefix_lo, prefix_hi, q_lo, q_hi, own_lo, own_hi, q_heads, kv_heads, dim, page,
            dtype, window, lens):
    return {"name": name, "op": "prefix", "groups": groups, "seqs_lo": seqs_lo, "seqs_hi": seqs_hi, "prefix_lo": prefix_lo,
            "prefix_hi": prefix_hi, "q_lo": q_lo, "q_hi": q_hi, "own_lo": own_lo, "own_hi": own_hi, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "window": window, "lens": lens}


def _verify(name, batch, k_lo, k_hi, vocab, dtype, drafts, greedy, lens):
    return {"name": name, "op": "verify", "batch": batch, "k_lo": k_lo, "k_hi": k_hi, "vocab": vocab, "dtype": dtype,
            "drafts": drafts, "greedy": greedy, "lens": lens}


def listed():
    return [
        # a few sequences' decode step, some of which need a page: latency
        _tables("tables_few", 7, 1, 1, 900, 0, 0, 0.0, 16, 1, False, 1),
        # a large batch with drafts: tokens rejected in the last step, ended sequences, shared first pages, a padded graph
        _tables("tables_batch", 1000, 1, 6, 4000, 5, 24, 0.1, 32, 500, False, 2),
        # prompts in one step, more than there are pages for
        _tables("tables_prompts", 40, 500, 6000, 700, 0, 0, 0.2, 16, 0, True, 3),
        # four samples of a short prompt: latency
        _prefix("prefix_few", 1, 4, 4, 508, 508, 1, 1, 0, 40, 32, 4, 128, 16, "f32", 0, 4),
        # samples of one long prompt, one token each
        _prefix("prefix_samples", 1, 64, 64, 8192, 8192, 1, 1, 0, 600, 32, 8, 128, 64, "bf16", 0, 5),
        # drafted tokens of a tree of samples in fp32, an odd group of heads, a prefix that ends inside a page
        _prefix("prefix_drafts", 1, 24, 24, 3001, 3001, 1, 5, 0, 300, 14, 2, 64, 16, "f32", 0, 6),
        # several prompts with samples of each, of all lengths, some alone
        _prefix("prefix_groups", 7, 1, 20, 100, 9000, 1, 3, 0, 1500, 16, 4, 128, 32, "bf16", 0, 7),
        # a large batch behind one long document
        _prefix("prefix_document", 1, 256, 256, 32768, 32768, 1, 1, 0, 1000, 32, 8, 128, 128, "bf16", 0, 8),
        # one sequence's drafts: latency
        _verify("verify_one", 1, 4, 4, 32000, "f32", True, 0.0, 9),
        # drafts without probabilities (looked up in the text), an odd vocabulary, half of the sequences greedy
        _verify("verify_lookup", 33, 0, 7, 50001, "bf16", False, 0.5, 10),
        # an ordinary batch with a draft model
        _verify("verify_batch", 64, 1, 5, 131072, "bf16", True, 0.0, 11),
        # a large batch in fp32
        _verify("verify_large", 256, 3, 3, 131072, "f32", True, 0.1, 12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["tables", "prefix", "prefix", "verify"])
    lens = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        if rng.random() < 0.6:   # decoding
            c = _tables("", _log_int(rng, 1, 1000), rng.choice([0, 1]), rng.randint(1, 6), _log_int(rng, 16, 4000),
                        rng.choice([0, 5]), rng.choice([0, 0, 24]), rng.choice([0.0, 0.1]), page, rng.choice([0, 1, 300]),
                        rng.random() < 0.2, lens)
        else:                    # prompts
            hi = _log_int(rng, 20, 6000)
            c = _tables("", _log_int(rng, 1, 40), max(1, hi // 3), hi, _log_int(rng, 16, 700), 0, rng.choice([0, 8]),
                        rng.choice([0.0, 0.2]), page, rng.choice([0, 100]), rng.random() < 0.3, lens)
    elif op == "prefix":
        dim, kv, dtype = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8]), rng.choice(["f32", "bf16"])
        q_heads = min(32, kv * rng.choice([1, 2, 3, 4, 7, 8]) if kv < 8 else kv * rng.choice([1, 2, 4]))
        groups = rng.choice([1, 1, 1, rng.randint(2, 8)])
        seqs = _log_int(rng, 2, 200 // groups)
        q_hi = rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 8, 120) if seqs * groups < 30 else 4])
        prefix = _log_int(rng, 30, max(100, min(60000, 4000000 // (seqs * groups * q_hi))))
        c = _prefix("", groups, 1 if groups > 1 else seqs, seqs, prefix if groups == 1 else max(1, prefix // 4), prefix,
                    1, q_hi, 0, _log_int(rng, 1, 1200), q_heads, kv, dim, page, dtype,
                    rng.choice([0, 0, 0, 128, 1000]), lens)
    else:
        vocab = _log_int(rng, 1000, 200000)
        batch = _log_int(rng, 1, 200)
        k_hi = rng.randint(1, 8)
        while batch * (k_hi + 1) * vocab > 100_000_000:
            batch = (batch + 1) // 2
        c = _verify("", batch, rng.choice([0, 1, k_hi]), k_hi, vocab, rng.choice(["f32", "bf16"]), rng.random() < 0.7,
                    rng.choice([0.0, 0.0, 0.3, 1.0]), lens)
    del c["name"]
    return c


def _table_lengths(case):
    """Per sequence: tokens kept, new ones wanted, pages held, first entries that are another's."""
    r = random.Random(case["lens"])
    page, out = case["page"], []
    for _ in range(case["batch"]):
        fixed = r.randint(0, case["fixed_hi"]) if r.random() < 0.5 else 0
        kept = fixed * page + r.randint(0, case["kept_hi"])
        held = max(-(-(kept + r.randint(0, case["back"])) // page) - fixed, 0)
        new = r.randint(case["new_lo"], case["new_hi"])
        if r.random() < case["ended"]:
            kept, new = 0, 0
        out.append((kept, new, held, fixed))
    return out


def _table_sizes(case):
    """Rows of the outputs, entries of a table row, pages taken if there are enough, and given back."""
    seqs, page = _table_lengths(case), case["page"]
    need = [max(-(-(k + n) // page) - f, 0) for k, n, h, f in seqs]
    take = sum(max(w - s[2], 0) for w, s in zip(need, seqs))
    give = sum(max(s[2] - w, 0) for w, s in zip(need, seqs))
    width = max(max(w, s[2]) + s[3] for w, s in zip(need, seqs)) + 2
    return max(1, sum(s[1] for s in seqs) + case["pad"]), width, take, give


def _prefix_lengths(case):
    """Per group: shared tokens and, per sequence, (new tokens, cached tokens with them)."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["groups"]):
        shared = r.randint(case["prefix_lo"], case["prefix_hi"])
        seqs = []
        for _ in range(r.randint(case["seqs_lo"], case["seqs_hi"])):
            n = r.randint(case["q_lo"], case["q_hi"])
            seqs.append((n, shared + r.randint(case["own_lo"], case["own_hi"]) + n))
        out.append((shared, seqs))
    return out


def _verify_lengths(case):
    """Rows of each sequence: its last token and its drafts."""
    r = random.Random(case["lens"])
    return [1 + r.randint(case["k_lo"], case["k_hi"]) for _ in range(case["batch"])]


def work(case):
    if case["op"] == "tables":
        m, _, take, give = _table_sizes(case)
        # kept, new, held, fixed in; held, length, start out; a page id read and written for each taken and given; pos and slot
        return {"bytes": 4 * 7 * case["batch"] + 8 * (take + give) + 12 * m, "flops": 0}
    if case["op"] == "verify":
        rows = _verify_lengths(case)
        size = 4 if case["dtype"] == "f32" else 2
        drafts = case["batch"] * case["vocab"] * 4 if case["drafts"] and case["k_hi"] else 0
        return {"bytes": sum(rows) * case["vocab"] * size + drafts, "flops": 4 * sum(rows) * case["vocab"]}
    d, size, page, w = case["dim"], 4 if case["dtype"] == "f32" else 2, case["page"], case["window"]
    rows = tokens = pairs = 0
    for shared, seqs in _prefix_lengths(case):
        whole, first = shared // page * page, None
        for n, length in seqs:
            at = length - n - w + 1 if w else 0
            first = max(at, 0) if first is None else min(first, max(at, 0))
            tokens += length - max(whole, at)
            pairs += sum(min(p + 1, w) if w else p + 1 for p in range(length - n, length))
            rows += n
        tokens += max(whole - first, 0)
    return {"bytes": 2 * rows * case["q_heads"] * d * size + 2 * tokens * case["kv_heads"] * d
            + (tokens + page - 1) // page * case["kv_heads"] * 8, "flops": 4 * d * case["q_heads"] * pairs}


# ---- inputs ------------------------------------------------------------------------------------

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_tables(case, g, s):
    seqs, page = _table_lengths(case), case["page"]
    m, width, take, give = _table_sizes(case)
    held = sum(x[2] for x in seqs)
    spare = max(0, take - give - 1 - take // 4) if case["short"] else max(0, take - give) + 40
    shared = sum(x[3] for x in seqs)
    pool = held + shared + spare
    order = torch.randperm(max(pool, 1), generator=g, device="cuda").to(torch.int32)
    ids, at = order.cpu(), 0
    table = torch.full((case["batch"], width), -1, dtype=torch.int32)
    for i, (_, _, h, f) in enumerate(seqs):
        table[i, :f + h] = ids[at:at + f + h]
        at += f + h
    free = torch.full((max(pool, 1),), -1, dtype=torch.int32)
    free[:spare] = ids[at:at + spare]
    kept, new, held, fixed = (list(x) for x in zip(*seqs))
    s.update(kept=_i32(kept), new=_i32(new), held=_i32(held), fixed=_i32(fixed), table=table.cuda(), free=free.cuda(),
             count=_i32([spare]), m=m, width=width, pages=max(pool, 1))


def _filled_cache(values):
    """Codes in e4m3 and a power-of-two scale for each (page, head) of pages [num_pages, kv_heads, page, dim] of values."""
    f, a = torch.frexp(values.abs().amax(dim=(2, 3)).double())   # 448 = 0.875 * 2^9
    scale = torch.ldexp(torch.ones_like(f), torch.where(f <= 0.875, a - 9, a - 8)).float()
    return (values / scale[:, :, None, None]).to(F8), scale


def _prepare_prefix(case, g, s):
    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    page, d, hkv = case["page"], case["dim"], case["kv_heads"]
    groups = _prefix_lengths(case)
    flat = [x for _, seqs in groups for x in seqs]
    counts, starts, at = [], [0], 0
    for shared, seqs in groups:
        whole = shared // page
        counts.append((whole, [-(-length // page) - whole for _, length in seqs]))
        starts.append(starts[-1] + len(seqs))
    pool = sum(w + sum(o) for w, o in counts) + 3
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(flat), -(-max(x[1] for x in flat) // page)), -1, dtype=torch.int32)
    i = 0
    for whole, owned in counts:
        first = ids[at:at + whole]
        at += whole
        for n in owned:
            table[i, :whole] = first
            table[i, whole:whole + n] = ids[at:at + n]
            at += n
            i += 1
    new = [x[0] for x in flat]
    s.update(table=table.cuda(), seq_lens=_i32([x[1] for x in flat]), q_start=_i32(np.concatenate([[0], np.cumsum(new)]).tolist()),
             group_start=_i32(starts), prefix_lens=_i32([x[0] for x in groups]), m=sum(new), max_q=max(new),
             max_len=max(x[1] for x in flat), max_prefix=max(x[0] for x in groups), pages=pool, batch=len(flat))
    # cached keys: some dims much larger than others; cached values: tokens of different size
    s["k_cache"], s["k_scale"] = _filled_cache(randn(pool, hkv, page, d) * torch.exp(0.4 * randn(1, hkv, 1, d)))
    s["v_cache"], s["v_scale"] = _filled_cache(randn(pool, hkv, page, d) * torch.exp(0.7 * randn(pool, hkv, page, 1)))
    s["q"] = (1.3 * randn(s["m"], case["q_heads"] * d)).to(DTYPES[case["dtype"]])
    s["scale"] = 1.0 / math.sqrt(d)


def _prepare_verify(case, g, s):
    rows, v = _verify_lengths(case), case["vocab"]
    m, b = sum(rows), case["batch"]
    starts = np.concatenate([[0], np.cumsum(rows)])
    # a few likely tokens, a long tail; some tokens masked out by the grammar
    logits = 2.0 * torch.randn(m, v, generator=g, device="cuda")
    logits += 9.0 * (torch.rand(m, v, generator=g, device="cuda") < 12.0 / v)
    draft = logits + 0.7 * torch.randn(m, v, generator=g, device="cuda")
    logits[:, torch.randint(0, v, (v // 50,), generator=g, device="cuda")] = -math.inf
    temperature = 0.5 + torch.rand(b, generator=g, device="cuda")
    temperature[torch.rand(b, generator=g, device="cuda") < case["greedy"]] = 0.0
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), torch.tensor(rows, device="cuda"), output_size=m)
    q = torch.softmax(draft / temperature[seq].clamp_min(0.3)[:, None], -1)
    # each draft is drawn from the row before it
    cum = torch.cumsum(q, -1, dtype=torch.float64)
    u = torch.rand(m, 1, generator=g, device="cuda", dtype=torch.float64) * cum[:, -1:]
    drawn = torch.searchsorted(cum, u, right=True).clamp_max(v - 1).view(-1).to(torch.int32)
    tokens = torch.randint(0, v, (m,), generator=g, device="cuda").to(torch.int32)
    tokens[1:] = drawn[:-1]
    s.update(logits=logits.to(DTYPES[case["dtype"]]), probs=q if case["drafts"] else None, tokens=tokens,
             q_start=_i32(starts.tolist()), temperature=temperature, m=m, max_rows=max(rows),
             u_accept=torch.rand(m, generator=g, device="cuda"), u_sample=torch.rand(b, generator=g, device="cuda"),
             seq_lens=_i32([700 + n for n in rows]))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    s = {"case": dict(case), "flag": torch.zeros(1, dtype=torch.int32, device="cuda")}
    {"tables": _prepare_tables, "prefix": _prepare_prefix, "verify": _prepare_verify}[case["op"]](case, g, s)
    return s


# ---- the plain form ----------------------------------------------------------------------------

def _exclusive(x):
    return torch.cumsum(x, 0) - x


def _plain_tables(s):
    page, m, width, pages = s["case"]["page"], s["m"], s["width"], s["pages"]
    kept, new, held, fixed = (s[k].long() for k in ("kept", "new", "held", "fixed"))
    need = (torch.div(kept + new + page - 1, page, rounding_mode="floor") - fixed).clamp_min(0)
    take, give = (need - held).clamp_min(0), (held - need).clamp_min(0)
    count, gives = s["count"].long(), give.sum()
    served = (take == 0) | (torch.cumsum(take, 0) <= count + gives)
    new, need = torch.where(served, new, 0), torch.where(served, need, held)
    take = torch.where(served, take, 0)
    taken = take.sum()
    # the stack: free pages, then those given back in order
    e = torch.arange(width, device="cuda")[None] - fixed[:, None]
    table = s["table"].long()
    back = (e >= need[:, None]) & (e < held[:, None])
    place = torch.where(back, count + _exclusive(give)[:, None] + e - need[:, None], pages)
    stack = torch.cat([s["free"].long(), torch.zeros(1, dtype=torch.long, device="cuda")])
    stack = stack.scatter(0, place.view(-1), table.view(-1))
    # pages taken from its top
    want = (e >= held[:, None]) & (e < need[:, None])
    top = count + gives - 1 - (_exclusive(take)[:, None] + e - held[:, None])
    table = torch.where(want, stack[torch.where(want, top, 0)], table)
    left = count + gives - taken
    at = torch.arange(pages, device="cuda")
    free = torch.where((at >= count) & (at < left), stack[:-1], s["free"].long())
    start = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(new, 0)])
    r = torch.arange(m, device="cuda")
    seq = torch.searchsorted(start, r, right=True) - 1
    inside = seq < kept.numel()
    seq = seq.clamp_max(kept.numel() - 1)
    pos = torch.where(inside, kept[seq] + r - start[seq], 0)
    slot = torch.where(inside, table[seq, pos // page] * page + pos % page, -1)
    i32 = torch.int32
    return {"table": table.to(i32), "held": need.to(i32), "free": free.to(i32), "count": left.to(i32), "q_start": start.to(i32),
            "seq_lens": (kept + new).to(i32), "pos": pos.to(i32), "slots": slot}


def _plain_prefix(s):
    c = s["case"]
    hq, hkv, d, page, w = c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["window"]
    rep = hq // hkv
    q = s["q"].view(s["m"], hq, d).float()
    out = torch.empty(s["m"], hq, d, device="cuda")

    def tokens(cache, scale, ids):   # [.., kv_heads, length, d] in fp32 of pages [.., n]
        x = cache.view(torch.uint8)[ids].view(F8).float() * scale[ids][..., None, None]
        return x.transpose(-4, -3).flatten(-3, -2)

    row = seq = 0
    for shared, seqs in _prefix_lengths(c):
        b, n, whole = len(seqs), sum(x[0] for x in seqs), shared // page
        width = max(x[0] for x in seqs)
        table = s["table"][seq:seq + b].long()
        of = torch.repeat_interleave(torch.arange(b, device="cuda"), torch.tensor([x[0] for x in seqs], device="cuda"), output_size=n)
        start, lens = s["q_start"][seq:seq + b + 1].long(), s["seq_lens"][seq:seq + b].long()
        at = torch.arange(n, device="cuda") + row - start[of]
        pos = lens[of] - (start[1:] - start[:-1])[of] + at
        owned = max(-(-x[1] // page) for x in seqs) - whole
        mine = table[:, whole:whole + owned].clamp_min(0)
        held = whole * page + torch.arange(owned * page, device="cuda") < lens[:, None]
        qp = torch.zeros(b, width, hq, d, device="cuda")
        qp[of, at] = q[row:row + n]
        pp = torch.full((b, width), -1, dtype=torch.long, device="cuda")
        pp[of, at] = pos
        qp = qp.view(b, width, hkv, rep, d).permute(2, 0, 3, 1, 4)            # [hkv, b, rep, width, d]
        flat = qp.reshape(hkv, -1, d)
        kp, vp = (tokens(s[k + "_cache"], s[k + "_scale"], table[0, :whole]) for k in "kv")   # [hkv, whole * page, d]
        ko, vo = (tokens(s[k + "_cache"], s[k + "_scale"], mine).masked_fill_(~held[:, None, :, None], 0.0)
                  .transpose(0, 1) for k in "kv")                               # [hkv, b, owned * page, d]
        x = torch.cat([torch.matmul(flat, kp.transpose(1, 2)).view(hkv, b, rep, width, whole * page),
                       torch.matmul(qp.reshape(hkv, b, rep * width, d), ko.transpose(2, 3))
                       .view(hkv, b, rep, width, owned * page)], -1)
        col = torch.arange((whole + owned) * page, device="cuda")
        keep = col <= pp[..., None]
        if w:
            keep &= col > pp[..., None] - w
        x.mul_(s["scale"]).masked_fill_(~keep[None, :, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x[..., :whole * page].reshape(hkv, b * rep * width, whole * page), vp).view(hkv, b, rep, width, d)
        o += torch.matmul(x[..., whole * page:].reshape(hkv, b, rep * width, owned * page), vo).view(hkv, b, rep, width, d)
        o /= torch.where(total > 0, total, 1.0)
        out[row:row + n] = o.permute(1, 3, 0, 2, 4).reshape(b, width, hq, d)[of, at]
        row, seq = row + n, seq + b
    return out.view(s["m"], hq * d).to(s["q"].dtype)


def _plain_verify(s):
    c = s["case"]
    v, m, b, most = c["vocab"], s["m"], c["batch"], s["max_rows"]
    start = s["q_start"].long()
    n = start[1:] - start[:-1]
    r = torch.arange(m, device="cuda")
    seq = torch.searchsorted(start, r, right=True) - 1
    temp = s["temperature"].double()[seq][:, None]
    x = torch.nan_to_num(s["logits"].float(), nan=-math.inf, posinf=F32_MAX, neginf=-math.inf).double()
    top = x.amax(-1, keepdim=True)
    best = torch.where(x == top, torch.arange(v, device="cuda"), v).amin(-1, keepdim=True)
    # in place: the rows are as large as the vocabulary
    p = x.sub_(top).div_(torch.where(temp > GREEDY, temp, 1.0)).exp_()
    p /= p.sum(-1, keepdim=True)
    p = torch.where(temp > GREEDY, p, (torch.arange(v, device="cuda") == best).double())
    nxt = s["tokens"].long().roll(-1)[:, None]
    pd = p.gather(1, nxt)[:, 0]
    qd = s["probs"].double().gather(1, nxt)[:, 0] if s["probs"] is not None else torch.ones_like(pd)
    ok = torch.zeros(b, most, dtype=torch.bool, device="cuda")
    drafted = r + 1 < start[seq + 1]
    ok[seq, r - start[seq]] = drafted & (s["u_accept"].double() * qd < pd)
    accepted = ok.long().cumprod(1).sum(1)
    row = start[:-1] + accepted
    rest = p[row]
    rejected = (accepted < n - 1)[:, None]
    if s["probs"] is not None:
        left = (rest - s["probs"][row].double()).clamp_min(0.0)
    else:
        left = rest.scatter(1, nxt[row], 0.0)
    left = torch.where(rejected, left, rest)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, rest)
    cum = torch.cumsum(left, -1)
    at = (cum <= s["u_sample"].double()[:, None] * cum[:, -1:]).sum(-1)
    last = torch.where(left > 0, torch.arange(v, device="cuda"), -1).amax(-1)
    i32 = torch.int32
    return {"accepted": accepted.to(i32), "next": torch.minimum(at, last).to(i32),
            "kept": (s["seq_lens"].long() - n + 1 + accepted).to(i32)}


# ---- the library's form ------------------------------------------------------------------------

def _own_tables(s):
    import bit_quantized_moe_q4k_gb300 as q4k
    c = s["case"]
    if "out" not in s:   # the step's buffers, kept by the program
        e = lambda n, t=torch.int32: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
        b = c["batch"]
        s["out"] = {"table": s["table"], "held": e(b), "free": s["free"], "count": e(1), "q_start": e(b + 1), "seq_lens": e(b),
                    "pos": e(s["m"]), "slots": e(s["m"], torch.int64)}
    o = s["out"]
    q4k.q4k_page_tables(s["kept"], s["new"], s["fixed"], c["batch"], s["m"], s["width"], c["page"], s["pages"], s["held"],
                        s["free"], s["count"], s["table"], o["held"], o["count"], o["q_start"], o["seq_lens"], o["pos"],
                        o["slots"], s["flag"])
    return o


def _own_prefix(s):
    import bit_quantized_moe_q4k_gb300 as q4k
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["dim"]
    if "workspace" not in s:
        n = q4k.q4k_shared_prefix_attention_workspace_size(s["batch"], c["groups"], s["m"], hq, hkv, d)
        s["workspace"], s["workspace_bytes"] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
    out = torch.empty_like(s["q"])
    q4k.q4k_shared_prefix_attention(
        s["q"], s["m"], hq, hkv, d, hq * d, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q_start"], s["seq_lens"],
        s["table"], s["batch"], s["table"].shape[1], c["page"], s["pages"], s["group_start"], s["prefix_lens"], c["groups"],
        s["max_q"], s["max_len"], s["max_prefix"], s["scale"], c["window"], out, hq * d, s["workspace"], s["workspace_bytes"],
        s["flag"])
    return out


def _own_verify(s):
    import bit_quantized_moe_q4k_gb300 as q4k
    c = s["case"]
    v, b = c["vocab"], c["batch"]
    if "workspace" not in s:
        n = q4k.q4k_verify_drafts_workspace_size(b, s["m"], v)
        s["workspace"], s["workspace_bytes"] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
    accepted, nxt, kept = (torch.empty(b, dtype=torch.int32, device="cuda") for _ in range(3))
    q4k.q4k_verify_drafts(s["logits"], s["m"], v, v, s["probs"], v, s["tokens"], s["q_start"], b, s["temperature"],
                          s["u_accept"], s["u_sample"], s["seq_lens"], accepted, nxt, kept, s["workspace"],
                          s["workspace_bytes"], s["flag"])
    return {"accepted": accepted, "next": nxt, "kept": kept}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "prefix": _own_prefix, "verify": _own_verify}[op](state)
    return {"tables": _plain_tables, "prefix": _plain_prefix, "verify": _plain_verify}[op](state)


# ---- in 64 bits --------------------------------------------------------------------------------

def _exact_tables(case, s):
    page, m = case["page"], s["m"]
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    count = int(s["count"].cpu()[0])
    stack = free[:count].tolist()
    seqs, want = _table_lengths(case), []
    for i, (k, n, h, f) in enumerate(seqs):
        need = max(-(-(k + n) // page) - f, 0)
        want.append(need)
        stack += table[i, f + need:f + h].tolist()
    held, lens, starts, pos, slots = [], [], [0], [], []
    short = False
    for i, ((k, n, h, f), need) in enumerate(zip(seqs, want)):
        short = short or need - h > len(stack)   # one that lacks a page leaves none to those after it
        if need > h and short:
            n, need = 0, h
        for e in range(h, need):
            table[i, f + e] = stack.pop()
        held.append(need)
        lens.append(k + n)
        starts.append(starts[-1] + n)
        for t in range(k, k + n):
            pos.append(t)
            slots.append(int(table[i, t // page]) * page + t % page)
    if len(stack) > count:
        free[count:len(stack)] = stack[count:]
    pos += [0] * (m - len(pos))
    slots += [-1] * (m - len(slots))
    i64 = lambda x: torch.tensor(np.asarray(x, dtype=np.int64), device="cuda")  # noqa: E731
    return {"table": i64(table), "held": i64(held), "free": i64(free), "count": i64([len(stack)]), "q_start": i64(starts),
            "seq_lens": i64(lens), "pos": i64(pos), "slots": i64(slots)}


def _exact_prefix(case, s):
    hq, hkv, d, page, w = case["q_heads"], case["kv_heads"], case["dim"], case["page"], case["window"]
    out = torch.empty(s["m"], hq, d, dtype=torch.float64, device="cuda")

    def tokens(k, ids):   # [n * page, kv_heads, d]
        x = s[k + "_cache"].view(torch.uint8)[ids].view(F8).double() * s[k + "_scale"][ids].double()[..., None, None]
        return x.permute(1, 0, 2, 3).reshape(hkv, -1, d)

    row = i = 0
    for shared, seqs in _prefix_lengths(case):
        whole = shared // page
        first = {k: tokens(k, s["table"][i, :whole].long()) for k in "kv"}
        for n, length in seqs:
            ids = s["table"][i, whole:-(-length // page)].long()
            k, v = (torch.cat([first[x], tokens(x, ids)], 1)[:, :length] for x in "kv")
            pos = torch.arange(length - n, length, device="cuda")[:, None]
            col = torch.arange(length, device="cuda")[None]
            bias = torch.zeros(n, length, dtype=torch.float64, device="cuda")
            bias[(col > pos) | ((col <= pos - w) if w else (col < 0))] = -math.inf
            q = s["q"][row:row + n].double().view(n, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            a = torch.softmax(torch.matmul(q, k[:, None].transpose(2, 3)) * s["scale"] + bias, -1)
            out[row:row + n] = torch.matmul(a, v[:, None]).permute(2, 0, 1, 3).reshape(n, hq, d)
            row, i = row + n, i + 1
    return out.view(s["m"], -1)


def _exact_verify(case, s):
    start = s["q_start"].cpu().tolist()
    tokens, u_accept = s["tokens"].cpu().tolist(), s["u_accept"].cpu().tolist()
    u_sample, temperature = s["u_sample"].cpu().tolist(), s["temperature"].cpu().tolist()
    accepted, nxt, kept = [], [], []

    def target(r, t):
        x = s["logits"][r].cpu().double().numpy()
        x[np.isnan(x)] = -np.inf
        x = np.minimum(x, F32_MAX)
        if not t > GREEDY:
            p = np.zeros(len(x))
            p[int(np.argmax(x))] = 1.0
            return p
        p = np.exp((x - x.max()) / t)
        return p / p.sum()

    for i in range(case["batch"]):
        a, last = start[i], start[i + 1] - 1
        p = target(a, temperature[i])
        rest = None
        while a < last:
            d = tokens[a + 1]
            q = s["probs"][a].cpu().double().numpy() if s["probs"] is not None else np.eye(1, len(p), d)[0]
            if not u_accept[a] * q[d] < p[d]:
                rest = np.maximum(p - q, 0.0) if s["probs"] is not None else np.where(np.arange(len(p)) == d, 0.0, p)
                break
            a += 1
            p = target(a, temperature[i])
        if rest is None or not rest.sum() > 0:
            rest = p
        cum = np.cumsum(rest)
        at = min(int(np.searchsorted(cum, u_sample[i] * cum[-1], side="right")), int(np.nonzero(rest)[0][-1]))
        accepted.append(a - start[i])
        nxt.append(at)
        kept.append(int(s["seq_lens"][i]) - (last - a))
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
    return {"accepted": i64(accepted), "next": i64(nxt), "kept": i64(kept)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "prefix": _exact_prefix, "verify": _exact_verify}[case["op"]](case, s)
