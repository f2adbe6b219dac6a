"""GPU tests of q4k_page_tables against a plain walk over the sequences with a Python list as the stack of free
pages. Every result is a whole number: equal or wrong."""
import numpy as np
import pytest

import bit_quantized_moe_q4k_gb300 as q4k

from helpers import dev, err_flag, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PAGE_FLAG, SEQ_FLAG = 11, 12


def plain(kept, new, fixed, held, table, free, count, m, page):
    """The call's results for valid lengths, and the flags it may raise."""
    b, width = table.shape
    table, free, stack, flags = table.copy(), free.copy(), free[:count].tolist(), set()
    new, rows = list(new), 0
    for i in range(b):   # tokens without a row, or without a table entry
        if kept[i] + new[i] > width * page:
            new[i] = 0
            flags.add(SEQ_FLAG)
    for i in range(b):
        rows += new[i]
        if rows > m and new[i]:
            new[i] = 0
            flags.add(SEQ_FLAG)
    need = [max(-(-(kept[i] + new[i]) // page) - fixed[i], 0) for i in range(b)]
    for i in range(b):
        stack += table[i, fixed[i] + need[i]:fixed[i] + held[i]].tolist()
    short = False
    pos, slots, start = [], [], [0]
    for i in range(b):
        short = short or need[i] - held[i] > len(stack)
        if need[i] > held[i] and short:
            new[i], need[i] = 0, held[i]
            flags.add(PAGE_FLAG)
        for e in range(held[i], need[i]):
            table[i, fixed[i] + e] = stack.pop()
        for t in range(kept[i], kept[i] + new[i]):
            pos.append(t)
            slots.append(int(table[i, t // page]) * page + t % page)
        start.append(start[-1] + new[i])
    if len(stack) > count:
        free[count:len(stack)] = stack[count:]
    pos += [0] * (m - len(pos))
    slots += [-1] * (m - len(slots))
    return dict(table=table, free=free, held=need, count=[len(stack)], start=start, lens=[k + n for k, n in zip(kept, new)],
                pos=pos, slots=slots), flags


class Step:
    """Random lengths of one step and the pages behind them."""

    def __init__(self, seed, batch, page, new_hi, kept_hi, spare, fixed_hi=0, back=0, ended=0.0, pad=0, width=None):
        g = np.random.default_rng(seed)
        self.page = page
        self.fixed = g.integers(0, fixed_hi + 1, batch) * (g.random(batch) < 0.5)
        self.kept = self.fixed * page + g.integers(0, kept_hi + 1, batch)
        self.held = np.maximum(-(-(self.kept + g.integers(0, back + 1, batch)) // page) - self.fixed, 0)
        self.new = g.integers(0, new_hi + 1, batch)
        over = g.random(batch) < ended
        self.kept[over] = 0
        self.new[over] = 0
        most = int(max([1, *(self.fixed + self.held), *(-(-(self.kept + self.new) // page))]))
        self.width = width or most + 1
        used = int((self.fixed + self.held).sum())
        ids = g.permutation(used + spare + 1)
        self.pages = len(ids)
        self.table = np.full((batch, self.width), -7, np.int64)
        at = 0
        for i in range(batch):
            n = int(self.fixed[i] + self.held[i])
            self.table[i, :n] = ids[at:at + n]
            at += n
        self.free = np.full(self.pages, -9, np.int64)
        self.free[:spare] = ids[at:at + spare]
        self.count = spare
        self.m = int(self.new.sum()) + pad
        self.batch = batch

    def want(self, m=None):
        ints = lambda a: [int(x) for x in a]  # noqa: E731
        return plain(ints(self.kept), ints(self.new), ints(self.fixed), ints(self.held), self.table, self.free, self.count,
                     self.m if m is None else m, self.page)

    def device(self):
        i32 = lambda a: dev(np.asarray(a, np.int32).reshape(-1) if np.ndim(a) < 2 else np.asarray(a, np.int32))  # noqa: E731
        return {k: i32(v) for k, v in (("kept", self.kept), ("new", self.new), ("fixed", self.fixed), ("held", self.held),
                                       ("table", self.table), ("free", self.free), ("count", [self.count]))}


def call(s, t, m=None, in_place=False, fixed=True, rows=True):
    b, m = s.batch, s.m if m is None else m
    e = lambda n, d=torch.int32: torch.full((max(n, 1),), -77, dtype=d, device="cuda")  # noqa: E731
    out = dict(table=t["table"], free=t["free"], held=t["held"] if in_place else e(b), count=t["count"] if in_place else e(1),
               start=e(b + 1), lens=t["kept"] if in_place else e(b), pos=e(m + 3), slots=e(m + 3, torch.int64))
    flag = err_flag()
    q4k.q4k_page_tables(t["kept"], t["new"], t["fixed"] if fixed else None, b, m, s.width, s.page, s.pages, t["held"], t["free"],
                        t["count"], t["table"], out["held"], out["count"], out["start"], out["lens"], out["pos"] if rows else None,
                        out["slots"] if rows else None, flag)
    return out, flag


def check(out, want, m):
    for k, v in want.items():
        got = host(out[k])
        if k in ("pos", "slots"):
            assert (got[m:] == -77).all(), f"{k}: wrote past the rows"
            got = got[:m]
        got = got[:np.size(v)] if np.ndim(v) == 1 else got
        assert np.array_equal(got, np.asarray(v)), k


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("batch,new_hi,kept_hi,fixed_hi,back,ended,pad", [
    (1, 1, 0, 0, 0, 0.0, 0), (1, 5, 900, 0, 0, 0.0, 0), (7, 1, 300, 0, 0, 0.0, 2), (31, 6, 700, 3, 200, 0.2, 9),
    (256, 4, 900, 5, 5, 0.1, 0), (257, 4, 900, 5, 5, 0.1, 70), (1500, 3, 500, 2, 300, 0.3, 11), (5, 4000, 50, 1, 0, 0.0, 3),
    (64, 0, 800, 0, 700, 0.5, 4), (33, 300, 200, 0, 900, 0.3, 0),
])
def test_tables(page, batch, new_hi, kept_hi, fixed_hi, back, ended, pad):
    s = Step(batch + page, batch, page, new_hi, kept_hi, 4000 // page + batch * (1 + new_hi // page), fixed_hi, back, ended, pad)
    want, flags = s.want()
    assert not flags
    t = s.device()
    out, flag = call(s, t)
    check(out, want, s.m)
    assert int(flag) == 0
    again, flag = call(s, t)   # the lengths as they were: the same result
    check(again, want, s.m)
    t = s.device()
    out, flag = call(s, t, in_place=True)
    check(out, want, s.m)


@pytest.mark.parametrize("batch,new_hi,kept_hi,spare,back,ended", [
    (9, 40, 100, 3, 0, 0.0), (9, 40, 100, 0, 0, 0.0), (300, 5, 100, 20, 0, 0.1), (1100, 30, 100, 400, 60, 0.1), (3, 2000, 0, 200, 0, 0.0),
])
def test_short_of_pages(batch, new_hi, kept_hi, spare, back, ended):
    """From the first sequence that lacks a page on, those that need one wait; the others go on."""
    s = Step(batch, batch, 16, new_hi, kept_hi, spare, 0, back, ended, 5)
    want, flags = s.want()
    assert flags <= {PAGE_FLAG}
    out, flag = call(s, s.device())
    check(out, want, s.m)
    assert int(flag) == (PAGE_FLAG if flags else 0)


@pytest.mark.parametrize("batch,new_hi,cut", [(6, 9, 7), (40, 5, 50), (700, 4, 300), (2, 1, 1), (3, 4, 100)])
def test_more_tokens_than_rows(batch, new_hi, cut):
    s = Step(batch, batch, 32, new_hi, 90, 4 * batch)
    s.new[0] = max(s.new[0], 1)
    s.m = int(s.new.sum())
    s.width += 1
    m = max(0, s.m - cut)
    s.table = np.concatenate([s.table, np.full((batch, 1), -7)], 1)
    want, flags = s.want(m)
    assert flags == {SEQ_FLAG}
    out, flag = call(s, s.device(), m=m)
    check(out, want, m)
    assert int(flag) == SEQ_FLAG


def test_more_tokens_than_the_table_holds():
    s = Step(4, 12, 16, 3, 40, 50)
    s.new[5] = 16 * s.width - s.kept[5] + 1
    s.new[7] = 2 ** 31 - 1
    want, flags = s.want()
    assert flags == {SEQ_FLAG}
    out, flag = call(s, s.device())
    check(out, want, s.m)
    assert int(flag) == SEQ_FLAG


def test_full_rows_and_all_pages():
    """Every entry of every row, the last page of the pool; then everything given back at once."""
    b, w, page = 37, 5, 64
    s = Step(0, b, page, 0, 0, b * w)
    s.width, s.pages = w, b * w
    s.table = np.full((b, w), -7)
    s.free = np.random.default_rng(1).permutation(b * w)
    s.new = np.full(b, w * page)
    s.m = b * w * page
    want, flags = s.want()
    assert not flags and want["count"] == [0]
    t = s.device()
    out, flag = call(s, t, in_place=True)
    check(out, want, s.m)
    t["kept"].zero_()
    t["new"].zero_()
    out, flag = call(s, t, in_place=True)
    assert int(flag) == 0 and int(out["count"][0]) == b * w and (host(out["held"]) == 0).all()
    assert np.array_equal(host(out["free"]), want["table"].reshape(-1))
    assert (host(out["pos"])[:s.m] == 0).all() and (host(out["slots"])[:s.m] == -1).all()


def test_no_rows_no_sequences():
    s = Step(2, 5, 16, 0, 60, 4, back=60)
    want, _ = s.want()
    out, flag = call(s, s.device(), rows=False)
    for k in ("pos", "slots"):
        want.pop(k)
    check(out, want, 0)
    s = Step(2, 0, 16, 0, 0, 4, pad=6)
    out, flag = call(s, s.device())
    assert int(flag) == 0 and int(out["start"][0]) == 0 and int(out["count"][0]) == 4
    assert (host(out["pos"])[:6] == 0).all() and (host(out["slots"])[:6] == -1).all()


@pytest.mark.parametrize("new_hi", [9, 700])
def test_without_fixed_entries_and_large_ids(new_hi):
    """No fixed entries; with many new tokens slots beyond 32 bits."""
    s = Step(11, 20, 128, new_hi, 900, 60 + 20 * (new_hi // 128))
    s.pages = 1 << 30   # ids in the stack up to the pool's end; only the entries that are read exist
    s.free = s.free.copy()
    s.free[:s.count] = (1 << 30) - 1 - np.arange(s.count)
    want, _ = s.want()
    out, flag = call(s, s.device(), fixed=False)
    check(out, want, s.m)
    assert int(flag) == 0 and (new_hi < 100 or max(want["slots"]) > 1 << 32)


@pytest.mark.parametrize("kw", ["count", "count_negative", "kept", "kept_far", "new", "held", "fixed", "twice"])
def test_malformed_lengths(kw):
    """Values that leave their ranges: flagged, and nothing outside the buffers is touched (guards behind each)."""
    s = Step(3, 300, 16, 5, 200, 700, fixed_hi=2, back=100)
    g = np.random.default_rng(5)
    some = g.permutation(300)[:40]
    if kw == "count":
        s.count = s.pages + 100
    elif kw == "count_negative":
        s.count = -5
    elif kw == "kept":
        s.kept[some] = -3
    elif kw == "kept_far":
        s.kept[some] = 2 ** 31 - 1
    elif kw == "new":
        s.new[some] = -1
    elif kw == "held":
        s.held[some] = 2 ** 31 - 1
    elif kw == "fixed":
        s.fixed[some] = s.width + 5
    else:   # the stack full already: what is given back finds no place
        s.count = s.pages
        s.free = np.arange(s.pages)
        s.kept[:] = 0
        s.new[:] = 0
    t = s.device()
    sizes = {"table": s.batch * s.width, "free": s.pages, "held": s.batch, "count": 1, "start": s.batch + 1, "lens": s.batch,
             "pos": s.m, "slots": s.m}
    big = {k: torch.full((n + 64,), -77, dtype=torch.int64 if k == "slots" else torch.int32, device="cuda") for k, n in sizes.items()}
    big["table"][:sizes["table"]] = t["table"].view(-1)
    big["free"][:sizes["free"]] = t["free"]
    flag = err_flag()
    q4k.q4k_page_tables(t["kept"], t["new"], t["fixed"], s.batch, s.m, s.width, s.page, s.pages, t["held"], big["free"], t["count"],
                        big["table"], big["held"], big["count"], big["start"], big["lens"], big["pos"], big["slots"], flag)
    assert int(flag) in (PAGE_FLAG, SEQ_FLAG)
    for k, n in sizes.items():
        assert (host(big[k])[n:] == -77).all(), k
    start = host(big["start"])[:s.batch + 1]
    assert start[0] == 0 and (np.diff(start) >= 0).all() and start[-1] <= s.m
    assert 0 <= int(big["count"][0]) <= s.pages


def test_captured_steps():
    """A captured step that goes on from its own results: lengths grow, drafts are rejected, sequences end and begin."""
    b, page, pages, width, m = 24, 16, 400, 20, 150
    g = np.random.default_rng(8)
    t = {k: torch.zeros(b, dtype=torch.int32, device="cuda") for k in ("kept", "new", "held")}
    table = torch.full((b, width), -7, dtype=torch.int32, device="cuda")
    free0 = g.permutation(pages)
    free, count = dev(free0.astype(np.int32)), dev(np.array([pages], np.int32))
    start = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
    pos, slots = torch.zeros(m, dtype=torch.int32, device="cuda"), torch.zeros(m, dtype=torch.int64, device="cuda")
    flag = err_flag()

    def step():
        q4k.q4k_page_tables(t["kept"], t["new"], None, b, m, width, page, pages, t["held"], free, count, table, t["held"], count, start,
                            t["kept"], pos, slots, flag)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ref_table, ref_free, ref_held, ref_count = np.full((b, width), -7), free0.copy(), [0] * b, pages
    lens = [0] * b
    for k in range(40):
        kept = [0 if n and g.random() < 0.08 else max(n - int(g.integers(0, 4)), 0) for n in lens]
        new = [0 if x == 0 and n else int(g.integers(0, 40 if n == 0 else 6)) for x, n in zip(kept, lens)]
        while sum(new) > m:
            new[new.index(max(new))] = 0
        new = [min(n, width * page - x) for x, n in zip(kept, new)]
        want, flags = plain(kept, new, [0] * b, ref_held, ref_table, ref_free, ref_count, m, page)
        assert not flags
        t["kept"].copy_(dev(np.array(kept, np.int32)))
        t["new"].copy_(dev(np.array(new, np.int32)))
        graph.replay()
        check(dict(table=table, free=free, held=t["held"], count=count, start=start, lens=t["kept"],
                   pos=torch.cat([pos, pos.new_full((1,), -77)]), slots=torch.cat([slots, slots.new_full((1,), -77)])), want, m)
        ref_table, ref_free, ref_held, ref_count, lens = want["table"], want["free"], want["held"], want["count"][0], want["lens"]
        owned = [int(p) for i in range(b) for p in ref_table[i, :ref_held[i]]] + [int(p) for p in ref_free[:ref_count]]
        assert sorted(owned) == list(range(pages))
    assert int(flag) == 0


def test_other_stream_and_two_at_once():
    """Two calls on different streams with buffers of their own."""
    steps = [Step(k, 400, 16, 5, 300, 900, back=40) for k in (1, 2)]
    want = [s.want()[0] for s in steps]
    on = [torch.cuda.Stream() for _ in steps]
    ts = [s.device() for s in steps]
    torch.cuda.synchronize()
    outs = []
    for s, t, st in zip(steps, ts, on):
        with torch.cuda.stream(st):
            outs.append(call(s, t)[0])
    torch.cuda.synchronize()
    for s, o, w in zip(steps, outs, want):
        check(o, w, s.m)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("batch,new_hi,kept_hi,spare,pad", [
    (1, 17000, 50, 1100, 2), (3, 30001, 900, 9000, 7), (300, 70, 400, 9000, 9001), (5000, 9, 300, 9000, 0), (20, 3000, 200, 700, 1), (2, 0, 90, 5, 16391)])
def test_many_rows(batch, new_hi, kept_hi, spare, pad, page, shift):
    """More rows than one cluster writes; outputs that begin at and beside a 16-byte boundary; positions or slots alone."""
    s = Step(batch + page, batch, page, new_hi, kept_hi, spare, 2, 30, 0.1, pad, width=(kept_hi + new_hi) // page + 4)
    if batch == 1:
        s.new[:], s.m = new_hi, new_hi + pad
    want, flags = s.want()
    assert s.m > 16384 and flags <= {PAGE_FLAG}
    for rows in ("both", "pos", "slots"):
        t = s.device()
        e = lambda n, d=torch.int32: torch.full((n,), -77, dtype=d, device="cuda")  # noqa: E731
        pos, slots = e(s.m + 8)[shift:], e(s.m + 8, torch.int64)[shift:]
        out = dict(table=t["table"], free=t["free"], held=e(batch), count=e(1), start=e(batch + 1), lens=e(batch), pos=pos, slots=slots)
        flag = err_flag()
        q4k.q4k_page_tables(t["kept"], t["new"], t["fixed"], batch, s.m, s.width, page, s.pages, t["held"], t["free"], t["count"],
                            t["table"], out["held"], out["count"], out["start"], out["lens"], pos if rows != "slots" else None,
                            slots if rows != "pos" else None, flag)
        for k in ("pos", "slots"):
            if rows not in ("both", k):
                assert (host(out.pop(k)) == -77).all()
        check(out, {k: v for k, v in want.items() if k in out}, s.m)
        assert int(flag) == (PAGE_FLAG if flags else 0)


def test_most_sequences():
    for new_hi in (1, 5):   # in the cluster, and with a second kernel
        s = Step(50 + new_hi, 8192, 16, new_hi, 200, 9000, 2, 60, 0.2, 3)
        want, flags = s.want()
        assert not flags and (s.m > 16384) == (new_hi == 5)
        out, flag = call(s, s.device())
        check(out, want, s.m)
        assert int(flag) == 0


def test_captured_prompts_in_chunks():
    """Rows by the second kernel, captured, lengths and held pages in place: each replay goes on where the last one ended."""
    batch, chunk, page, steps = 20, 900, 32, 3
    s = Step(70, batch, page, 0, 0, 20 * (steps * chunk // page + 1), width=steps * chunk // page + 2)
    s.new[:], s.m = chunk, batch * chunk
    t = s.device()
    out, flag = call(s, t, in_place=True)   # outside a graph first: the state it leaves is put back
    t2 = s.device()
    for k in t:
        t[k].copy_(t2[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4k.q4k_page_tables(t["kept"], t["new"], t["fixed"], batch, s.m, s.width, page, s.pages, t["held"], t["free"], t["count"], t["table"],
                            t["held"], t["count"], out["start"], t["kept"], out["pos"], out["slots"], flag)
    assert s.m > 16384
    for _ in range(steps):
        want, flags = s.want()
        assert not flags
        graph.replay()
        torch.cuda.synchronize()
        check(dict(table=t["table"], free=t["free"], held=t["held"], count=t["count"], start=out["start"], lens=t["kept"], pos=out["pos"],
                   slots=out["slots"]), want, s.m)
        s.kept, s.held, s.count = np.array(want["lens"]), np.array(want["held"]), want["count"][0]
        s.table, s.free = want["table"], want["free"]
    assert int(flag) == 0
