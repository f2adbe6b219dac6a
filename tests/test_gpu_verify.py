"""GPU tests of q4k_verify_drafts against a walk over the sequences in extended precision (numpy's long double). The
results are whole numbers: equal or wrong, but for a draw next to a border between tokens. A weight is off by 2^-31 of itself
(half a unit of 2^-31 in a table of powers and half in the product with the rest of the exponent), and, cut to the sums' unit of 2^-b
of the largest weight, b = 62 - ceil(log2 n), by that. So a cumulative sum of n weights is off by at
most E = 2^-31 + n 2^-b of the whole, which is not less than the largest weight; what is taken away for a draft,
another sum's share, brings it to 2 E, and the goal, a share of the whole, to 4 E. (Acceptances are decided to 2^-41.) In acceptances a random number within 2^-36 of the
border is not expected from the seeds here; the reference says so if one comes."""
import math

import numpy as np
import pytest

import bit_quantized_moe_q4k_gb300 as q4k

from helpers import dev, err_flag, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32_MAX = np.longdouble(np.finfo(np.float32).max)
SEQ_FLAG, TOKEN_FLAG = 12, 14
NEAR = 2.0 ** -36


def target(x, t):
    """p of a row of logits (float32 values), or None where no token has any."""
    x = x.astype(np.longdouble)
    x[np.isnan(x)] = -np.inf
    x = np.minimum(x, F32_MAX)
    if x.max() == -np.inf:
        return None
    if not t > 2.0 ** -64:
        p = np.zeros(len(x), np.longdouble)
        p[int(np.argmax(x))] = 1
        return p
    p = np.exp((x - x.max()) / np.longdouble(t))
    return p / p.sum()


def plain(x, probs, tokens, start, temperature, u_accept, u_sample, lens, strict=True, drawn=None):
    acc, nxt, kept, flags = [], [], [], set()
    for i in range(len(start) - 1):
        a, last = start[i], start[i + 1] - 1
        if last < a:
            acc.append(0), nxt.append(-1), kept.append(lens[i])
            continue
        t = 1.0 if temperature is None else temperature[i]
        p, rejected = target(x[a], t), False
        while a < last:
            d = tokens[a + 1]
            if not 0 <= d < x.shape[1]:
                flags.add(TOKEN_FLAG)
                rejected = True
                break
            u = max(0, np.longdouble(u_accept[a]))   # in this order NaN counts as 0
            q = np.longdouble(1) if probs is None else max(0, np.longdouble(probs[a][d]))
            if p is None:
                rejected = True
                break
            if strict and u * q > 0 and p[d] > 0:
                assert abs(u * q / p[d] - 1) > NEAR, "a random number next to the border: take another seed"
            if not (u * q < p[d]):
                rejected = True
                break
            a += 1
            p = target(x[a], t)
        acc.append(a - start[i])
        kept.append(lens[i] - (last - a))
        if p is None:
            flags.add(TOKEN_FLAG)
            nxt.append(-1)
            continue
        rest = p
        if rejected:
            d = tokens[a + 1]
            if probs is None:
                rest = p.copy()
                if 0 <= d < len(p):
                    rest[d] = 0
            else:
                rest = np.maximum(p - np.maximum(np.nan_to_num(probs[a].astype(np.longdouble), nan=0.0), 0), 0)
            if not rest.sum() > 0:
                rest = p
        cum = np.cumsum(rest)
        goal = min(max(0, np.longdouble(u_sample[i])), 1) * cum[-1]
        at = min(int(np.searchsorted(cum, goal, side="right")), int(np.nonzero(rest)[0][-1]))
        if drawn is not None and drawn[i] != at:   # next to a border?
            j, n = drawn[i], len(p)
            e = 4 * (2.0 ** -31 + n * 2.0 ** -(62 - math.ceil(math.log2(n))))   # p sums to 1
            if 0 <= j < n and rest[j] > 0 and cum[j] - rest[j] - e <= goal <= cum[j] + e:
                at = j
        nxt.append(at)
    return acc, nxt, kept, flags


class Batch:
    def __init__(self, seed, rows, vocab, dtype="f32", probs=True, temperature="mixed", spread=2.0, like=0.7, pad=0, shift=0):
        g = np.random.default_rng(seed)
        self.rows, self.v, self.m, self.b = rows, vocab, sum(rows), len(rows)
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(int).tolist()
        m = max(self.m, 1)
        x = spread * g.standard_normal((m, vocab)) + 8.0 * (g.random((m, vocab)) < 8.0 / vocab)
        draft = x + like * g.standard_normal((m, vocab))
        q = np.exp(draft - draft.max(1, keepdims=True))
        q /= q.sum(1, keepdims=True)
        self.tokens = g.integers(0, vocab, m).tolist()
        for r in range(m - 1):
            self.tokens[r + 1] = int(np.searchsorted(np.cumsum(q[r]), g.random() * (1 - 1e-9)))
        self.x = torch.from_numpy(x.astype(np.float32))
        if dtype == "bf16":
            self.x = self.x.bfloat16()
        self.probs = q.astype(np.float32) if probs else None
        self.t = {"mixed": (0.4 + g.random(self.b)) * (g.random(self.b) < 0.75), "one": None, "greedy": np.zeros(self.b),
                  "warm": 0.3 + 1.5 * g.random(self.b)}[temperature]
        self.t = None if self.t is None else self.t.astype(np.float32)
        self.ua, self.us = g.random(m).astype(np.float32), g.random(self.b).astype(np.float32)
        self.lens = (100 + np.arange(self.b) + np.array(rows)).tolist()
        self.pad, self.shift = pad, shift

    def rows_on_device(self, x):
        """[m, vocab] rows `vocab + pad` apart, `shift` elements behind an aligned address; NaN between them."""
        m, v = x.shape
        flat = torch.full((m * (v + self.pad) + self.shift,), float("nan"), dtype=x.dtype, device="cuda")
        t = flat[self.shift:].view(m, v + self.pad)
        t[:, :v] = x.cuda()
        return t

    def call(self, workspace=None, fill=0x5A):
        i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
        need = q4k.q4k_verify_drafts_workspace_size(self.b, self.m, self.v)
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda") if workspace is None else workspace
        out = [torch.full((self.b + 8,), -77, dtype=torch.int32, device="cuda") for _ in range(3)]
        flag = err_flag()
        probs = None if self.probs is None else self.rows_on_device(torch.from_numpy(self.probs))
        q4k.q4k_verify_drafts(self.rows_on_device(self.x), self.m, self.v, self.v + self.pad, probs, self.v + self.pad,
                              i32(self.tokens), i32(self.start), self.b, None if self.t is None else dev(self.t), dev(self.ua), dev(self.us),
                              i32(self.lens), *out, ws, ws.numel(), flag)
        got = [host(o) for o in out]
        assert all((g[self.b:] == -77).all() for g in got)
        return [g[:self.b].tolist() for g in got], int(flag)

    def check(self, strict=True):
        got, flag = self.call()
        acc, nxt, kept, flags = plain(self.x.float().numpy(), self.probs, self.tokens, self.start, self.t, self.ua, self.us, self.lens, strict,
                                      got[1])
        assert got[0] == acc
        assert got[1] == nxt
        assert got[2] == kept
        assert flag in flags if flags else flag == 0
        return acc, nxt


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("rows,vocab", [
    ([1], 1), ([5], 2), ([3, 1, 4], 7), ([5], 1000), ([2, 0, 9, 1, 0, 3], 4096), ([1] * 40, 5003), ([20, 33], 8192), ([4] * 9, 50001),
    ([6], 131072), ([2, 3], 200003),
])
def test_verify(rows, vocab, probs, dtype):
    Batch(vocab + len(rows), rows, vocab, dtype, probs).check()


@pytest.mark.parametrize("temperature", ["one", "greedy", "warm"])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 3), (8, 0), (3, 4), (7, 1)])
def test_temperatures_and_strides(temperature, probs, pad, shift):
    for dtype in ("f32", "bf16"):
        Batch(pad + 31 * shift, [4, 1, 6, 2], 3001, dtype, probs, temperature, pad=pad, shift=shift).check()


@pytest.mark.parametrize("seed", range(6))
def test_many_sequences(seed):
    """A few hundred decisions and draws each: tokens of all ranks are drawn."""
    g = np.random.default_rng(seed)
    b = Batch(seed, g.integers(0, 6, 300).tolist(), 2000, ["f32", "bf16"][seed % 2], seed % 3 > 0, "warm", spread=0.5 + seed, like=0.3)
    acc, nxt = b.check()
    assert len(set(nxt)) > 20 and len(set(acc)) > (1 if b.probs is None else 3)


def test_flat_distribution():
    """Every token as likely as any other: the draw is the random number's place in the vocabulary."""
    b = Batch(1, [1] * 64, 131072, probs=False, temperature="one")
    b.x.zero_()
    acc, nxt = b.check(strict=False)   # sums and goals are exact here
    assert nxt == [min(int(np.float64(u) * 131072), 131071) for u in b.us]


def test_equal_logits_take_the_lowest_index():
    b = Batch(2, [3] * 12, 9000, temperature="greedy", probs=False)
    g = np.random.default_rng(0)
    for r in range(b.m):
        at = np.sort(g.permutation(9000)[:4])
        b.x[r, at] = 50.0
        if r % 3 < 2:
            b.tokens[r + 1] = int(at[0] if r % 2 else at[1])
    acc, _ = b.check()
    assert set(acc) >= {0, 1}


def test_masked_infinite_and_nan_logits():
    b = Batch(3, [4] * 30, 3000)
    g = np.random.default_rng(4)
    for r in range(b.m):
        kind = r % 6
        at = g.permutation(3000)
        if kind == 1:
            b.x[r, at[:2990]] = -math.inf
        elif kind == 2:
            b.x[r, at[:7]] = math.nan
        elif kind == 3:
            b.x[r, at[:3]] = math.inf
        elif kind == 4:
            b.x[r, at[:2999]] = torch.finfo(torch.float32).min
        elif kind == 5:
            b.x[r, at[:2000]] = -math.inf
            b.x[r, at[2000:2500]] = math.nan
    b.check()


def test_rows_without_any_token():
    b = Batch(5, [3, 2, 1, 4], 700, temperature="warm")
    b.x[4] = -math.inf           # the second sequence's bonus row
    b.x[5] = math.nan            # the third one's only row
    b.x[6] = -math.inf           # the last one's first
    b.ua[3] = 0.0
    b.check()


def test_drafts_outside_the_vocabulary():
    for probs in (True, False):
        b = Batch(6, [3, 3, 3], 600, probs=probs)
        b.tokens[1], b.tokens[4], b.tokens[8] = 600, -1, 2 ** 31 - 1
        b.check()


def test_probabilities_at_their_ends():
    """Zero, one, NaN, negative and unnormalised draft probabilities; random numbers 0, 1 and beyond."""
    b = Batch(7, [3] * 40, 500)
    g = np.random.default_rng(1)
    for i in range(40):
        r = b.start[i]
        d = b.tokens[r + 1]
        b.probs[r, d] = [0.0, 1.0, np.nan, -0.5, 2.0, 1e-30, np.finfo(np.float32).tiny / 4, 0.25][i % 8]
        if i % 5 == 0:
            b.probs[r, g.permutation(500)[:100]] = np.nan
        if i % 5 == 1:
            b.probs[r] = 1.0     # nothing is left of any token
            b.ua[r] = 0.999
        b.ua[r + 1] = [0.0, 1.0, -1.0, np.nan, 5.0][i % 5]
        b.us[i] = [0.0, 1.0, -1.0, np.nan, 7.0, np.float32(1 - 2.0 ** -24), 1e-45, 0.5][i % 8]
    b.check()


@pytest.mark.parametrize("vocab", [300, 50001])
def test_acceptance_next_to_the_border(vocab):
    """u next to p(d): the fp32 numbers on both sides of it, 2^-24 apart and less; half of them are accepted."""
    b = Batch(8 + vocab, [2] * 128, vocab, probs=False, temperature="warm")
    x = b.x.numpy()
    want = []
    for i in range(b.b):
        r = b.start[i]
        order = np.argsort(-x[r])
        d = int(order[i % 5])
        p = target(x[r], b.t[i])[d]
        u = np.float32(p)
        if (i % 2 == 0) == bool(np.longdouble(u) < p):   # even: on or above it
            u = np.nextafter(u, np.float32(2.0 if i % 2 == 0 else -1.0))
        b.tokens[r + 1], b.ua[r] = d, u
        want.append(int(np.longdouble(u) < p))
    acc, _ = b.check(strict=False)
    assert acc == want and 40 < sum(want) < 90


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_draws_next_to_the_border(dtype):
    """u next to a cumulative sum of 131072 tokens: the fp32 numbers on both sides of it."""
    b = Batch(9, [1] * 48, 131072, dtype, probs=False, temperature="warm", spread=1.0)
    x = b.x.float().numpy()
    for i in range(b.b):
        cum = np.cumsum(target(x[i], b.t[i]))
        j = int(np.searchsorted(cum, (i + 0.5) / b.b))
        u = np.float32(cum[j])
        b.us[i] = u if i % 2 else np.nextafter(u, np.float32(0 if np.longdouble(u) >= cum[j] else 1))
    b.check(strict=False)


def test_optional_arguments_and_aliases():
    b = Batch(10, [2, 3], 400)
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    want, flag = b.call()
    ws = torch.empty(q4k.q4k_verify_drafts_workspace_size(2, 5, 400), dtype=torch.uint8, device="cuda")
    acc, nxt, lens = i32([0, 0]), i32([0, 0]), i32(b.lens)
    args = [b.x.cuda(), 5, 400, 400, dev(b.probs), 400, i32(b.tokens), i32(b.start), 2, dev(b.t), dev(b.ua), dev(b.us)]
    q4k.q4k_verify_drafts(*args, None, acc, nxt, None, ws, ws.numel())
    assert [host(acc).tolist(), host(nxt).tolist()] == want[:2]
    q4k.q4k_verify_drafts(*args, lens, acc, nxt, lens, ws, ws.numel())
    assert host(lens).tolist() == want[2]


def test_no_rows_at_all():
    b = Batch(11, [0, 0, 0], 100)
    got, flag = b.call()
    assert got == [[0, 0, 0], [-1, -1, -1], b.lens] and flag == 0


@pytest.mark.parametrize("start", [[0, 5, 2, 6], [-3, 2, 4, 6], [0, 2, 4, 60], [6, 4, 2, 0], [9, 9, 9, 9]])
def test_malformed_starts(start):
    b = Batch(12, [2, 2, 2], 500)
    b.start = start
    got, flag = b.call(fill=0)
    assert flag in (SEQ_FLAG, TOKEN_FLAG)
    assert all(0 <= a <= 6 for a in got[0])


def test_captured_and_on_two_streams():
    """Replays with new inputs in the same buffers; two graphs with workspaces of their own at once."""
    batches = [Batch(20 + k, [1 + (i + k) % 5 for i in range(30)], 8000, ["f32", "bf16"][k], True) for k in range(2)]
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    made = []
    for b in batches:
        s = dict(x=b.x.cuda(), q=dev(b.probs), tok=i32(b.tokens), st=i32(b.start), t=dev(b.t), ua=dev(b.ua), us=dev(b.us), lens=i32(b.lens),
                 out=[i32([0] * b.b) for _ in range(3)], flag=err_flag(),
                 ws=torch.empty(q4k.q4k_verify_drafts_workspace_size(b.b, b.m, b.v), dtype=torch.uint8, device="cuda"))

        def run(s=s, b=b):
            q4k.q4k_verify_drafts(s["x"], b.m, b.v, b.v, s["q"], b.v, s["tok"], s["st"], b.b, s["t"], s["ua"], s["us"], s["lens"],
                                  *s["out"], s["ws"], s["ws"].numel(), s["flag"])
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        made.append((s, g))
    streams = [torch.cuda.Stream() for _ in made]
    for k in range(5):
        rng = np.random.default_rng(k)
        for b, (s, g) in zip(batches, made):
            b.ua, b.us = rng.random(b.m).astype(np.float32), rng.random(b.b).astype(np.float32)
            s["ua"].copy_(dev(b.ua))
            s["us"].copy_(dev(b.us))
        torch.cuda.synchronize()
        for (s, g), st in zip(made, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for b, (s, g) in zip(batches, made):
            acc, nxt, kept, _ = plain(b.x.float().numpy(), b.probs, b.tokens, b.start, b.t, b.ua, b.us, b.lens)
            assert [host(o).tolist() for o in s["out"]] == [acc, nxt, kept]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_vocabulary(dtype):
    Batch(60, [3, 1, 2], 1 << 20, dtype, temperature="warm").check()
    Batch(61, [2, 2], (1 << 20) - 1, dtype, probs=False, temperature="warm").check()


@pytest.mark.parametrize("t", [1e38, 3e38, 1e-37, 2.0 ** -63])
def test_nan_and_infinite_logits_at_extreme_temperatures(t):
    b = Batch(62, [2] * 20, 900, probs=False, temperature="one")
    b.t = np.full(b.b, t, np.float32)
    b.x[::2, 5:450] = math.nan
    b.x[1::3, 100:600] = -math.inf
    b.check()


def test_kept_in_place_of_the_lengths():
    b = Batch(63, [3, 0, 2, 5], 800)
    want = plain(b.x.numpy(), b.probs, b.tokens, b.start, b.t, b.ua, b.us, b.lens)
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    lens, acc, nxt, flag = i32(b.lens), i32([0] * 4), i32([0] * 4), err_flag()
    ws = torch.empty(q4k.q4k_verify_drafts_workspace_size(b.b, b.m, b.v), dtype=torch.uint8, device="cuda")
    q4k.q4k_verify_drafts(b.x.cuda(), b.m, b.v, b.v, dev(b.probs), b.v, i32(b.tokens), i32(b.start), b.b, dev(b.t), dev(b.ua), dev(b.us), lens,
                          acc, nxt, lens, ws, ws.numel(), flag)
    assert [host(o).tolist() for o in (acc, nxt, lens)] == list(want[:3]) and int(flag) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("probs", [True, False])
def test_infinite_temperature(probs, dtype):
    """Every token whose logit is above -inf is as likely as any other."""
    b = Batch(64, [3] * 60, 2000, dtype, probs, "one")
    b.x[::3, 100:900] = -math.inf
    b.x[1::7, 300:305] = math.nan
    b.x[2::5, 1000:1003] = math.inf
    b.t = np.full(b.b, np.inf, np.float32)
    got, flag = b.call()
    flat = torch.where(b.x.float() > -math.inf, 0.0, -math.inf).numpy()   # NaN: no probability
    acc, nxt, kept, flags = plain(flat, b.probs, b.tokens, b.start, None, b.ua, b.us, b.lens, drawn=got[1])
    assert got == [acc, nxt, kept] and not flags and flag == 0


def test_infinite_temperature_and_logits_far_apart():
    """A logit further below the largest than the largest finite number has no probability, at any temperature."""
    b = Batch(65, [1] * 32, 700, probs=False, temperature="one")
    b.x[:] = -3e38
    b.x[:, 200:203] = 3e38
    b.x[::2, 5] = 1e38
    b.t = np.full(b.b, np.inf, np.float32)
    got, flag = b.call()
    assert flag == 0
    for i in range(b.b):
        left = [5, 200, 201, 202] if i % 2 == 0 else [200, 201, 202]
        assert got[1][i] == left[int(np.float64(b.us[i]) * len(left))]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
@pytest.mark.parametrize("vocab,pad,shift", [(3001, 0, 0), (3001, 5, 3), (3000, 7, 1), (2999, 3, 2), (50001, 2, 1)])
def test_one_infinite_or_nan_logit_anywhere(vocab, pad, shift, value, dtype):
    """Rows that begin off a 16-byte boundary and end off one; next to the row's largest logit, at its ends and between."""
    b = Batch(66 + vocab, [2] * 48, vocab, dtype, probs=False, temperature="warm", pad=pad, shift=shift)
    g = np.random.default_rng(vocab + pad)
    for r in range(b.m):
        top = int(b.x[r].float().argmax())
        at = [0, vocab - 1, max(top - 1, 0), min(top + 1, vocab - 1), 1, vocab - 2, int(g.integers(vocab)), int(g.integers(vocab))][r // 2 % 8]
        b.x[r, at] = value
    b.check()


@pytest.mark.parametrize("temperature", ["greedy", "warm"])
@pytest.mark.parametrize("start", [[0, 5, 2], [0, 5, 2, 6], [-3, 2, 4, 6], [0, 2, 4, 60], [6, 4, 2, 0], [9, 9, 9, 9], [0, 6, 3, 6], [2, 4, 4, 5]])
def test_malformed_starts_on_any_workspace(start, temperature):
    """Results are of the inputs alone, and are tokens or -1."""
    b = Batch(12, [2, 2, 2], 500, temperature=temperature)
    b.start, b.b = start, len(start) - 1
    got = [b.call(fill=fill) for fill in (0x00, 0x5A, 0x7F, 0xFF)]
    assert all(x == got[0] for x in got)
    (acc, nxt, kept), flag = got[0]
    assert flag == (0 if start == [2, 4, 4, 5] else SEQ_FLAG) or flag == TOKEN_FLAG
    assert all(0 <= a < 6 for a in acc) and all(-1 <= x < 500 for x in nxt)


@pytest.mark.parametrize("vocab", [1 << 20, (1 << 19) + 1])
def test_acceptance_next_to_the_border_behind_many_small_weights(vocab):
    """One large weight, and as many as there are tokens a little above the unit of the sums."""
    b = Batch(67, [2] * 8, vocab, probs=False, temperature="one")
    want = []
    for i in range(b.b):
        r, d = b.start[i], 1000 * i + 3
        b.x[r] = float(np.log((1.1, 1.5, 1.9, 2.6)[i // 2]) - 42 * np.log(2.0))
        b.x[r, d] = 0.0
        p = target(b.x[r].numpy(), 1.0)[d]
        u = np.float32(p)
        if (i % 2 == 0) == bool(np.longdouble(u) < p):   # even: on or above it
            u = np.nextafter(u, np.float32(2.0 if i % 2 == 0 else -1.0))
        b.tokens[r + 1], b.ua[r] = d, u
        want.append(int(np.longdouble(u) < p))
    acc, _ = b.check(strict=False)
    assert acc == want and sum(want) == 4


@pytest.mark.parametrize("probs_off", [0.0, 1e-7, 1e-6, 1e-5, 1e-3])
@pytest.mark.parametrize("vocab", [3000, 50001])
def test_draws_where_draft_and_target_nearly_agree(vocab, probs_off):
    """A rejected draft whose probabilities are the target's but for some 2^-24 of them, so that what is left is as small: drawn in exact
    arithmetic all the same, but for the weights' errors: 4 E of the whole sum in a cumulative one (as above); what is left of a token by
    2^-31 of its weight and, q times the sum, by E of it."""
    b = Batch(68 + vocab, [2] * 64, vocab, temperature="one", spread=1.0)
    g = np.random.default_rng(vocab)
    p = [target(x, 1.0) for x in b.x.numpy()]
    b.probs[:] = [(q * (1 + probs_off * g.standard_normal(vocab))).astype(np.float32) for q in p]
    b.ua[:] = 2.0   # every draft is rejected
    got, flag = b.call()
    assert flag == 0 and got[0] == [0] * b.b
    e = 2.0 ** -31 + vocab * 2.0 ** -(62 - math.ceil(math.log2(vocab)))
    for i in range(b.b):
        r, j = b.start[i], got[1][i]
        left = p[r] - b.probs[r].astype(np.longdouble)
        rest = np.maximum(left, 0)
        cum = np.cumsum(rest)
        goal = np.longdouble(b.us[i]) * cum[-1]
        assert 0 <= j < vocab and left[j] > -(2.0 ** -31 + e) * p[r][j]
        assert cum[j] - rest[j] - 4 * e <= goal <= cum[j] + 4 * e


def test_one_workspace_for_calls_of_all_sizes():
    """Sized for the most rows, with bytes behind it that no call touches."""
    made = [Batch(70 + n, [3] * n, 32000, temperature="warm") for n in (1, 5, 36, 127)]
    need = max(q4k.q4k_verify_drafts_workspace_size(b.b, b.m, b.v) for b in made)
    assert need == q4k.q4k_verify_drafts_workspace_size(made[-1].b, made[-1].m, made[-1].v)
    for b in made:
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        got, flag = b.call(workspace=ws[:need])
        assert got == list(plain(b.x.numpy(), b.probs, b.tokens, b.start, b.t, b.ua, b.us, b.lens, drawn=got[1])[:3]) and flag == 0
        assert (ws[need:] == 0xA5).all()
