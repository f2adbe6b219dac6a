"""A serving step of the four calls together, captured once and replayed: page tables on the device, the new tokens' keys and values
appended, attention behind the shared prefix, drafts verified, whose kept lengths begin the next step.

Each step is checked on its own inputs: tables against the plain walk (equal), what the cache holds against the tokens' keys and values
(half a step of e4m3: 2^-4 |x|, or 2^-10 of the page's scale), attention in fp64 over the cache's own codes (the tolerance of
test_gpu_shared_prefix.py), the verdicts against the walk in extended precision."""
import numpy as np
import pytest

import bit_quantized_moe_q4k_gb300 as q4k

from helpers import dev, err_flag, host
from test_gpu_attention import E4M3, U, attention_ref, f64, q_starts
from test_gpu_tables import plain as plain_tables
from test_gpu_verify import plain as plain_verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PAGE, HK, HQ, D, VOCAB, DRAFTS = 16, 2, 8, 64, 640, 3


class Codes:
    """The device's cache as attention_ref reads it."""

    def __init__(self, k, v, ks, vs, absolute=False):
        self.codes = {"k": host(k), "v": host(v) & (0x7F if absolute else 0xFF)}
        self.scale = {"k": host(ks), "v": host(vs)}
        self.page, self.heads = PAGE, HK

    def values(self, side, ids, length):
        x = E4M3[self.codes[side][ids]] * self.scale[side][ids].astype(np.float64)[:, :, None, None]
        return x.transpose(1, 0, 2, 3).reshape(HK, -1, D)[:, :length]


@pytest.mark.parametrize("setting", [None, "1"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,shared", [(9, 70), (40, 200)])
def test_drafts_behind_a_shared_prefix(batch, shared, dtype, setting, monkeypatch):
    if setting:
        monkeypatch.setenv("Q4K_SHARE_PREFIX", setting)
    else:
        monkeypatch.delenv("Q4K_SHARE_PREFIX", raising=False)
    g = np.random.default_rng(batch)
    tt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    # a token's query, key and value; each key and value has an element of 1, so that pages' scales never grow
    table_of = lambda w: dev(np.clip(0.4 * g.standard_normal((VOCAB, w)), -1, 1).astype(np.float32)).to(tt)  # noqa: E731
    eq, ek, ev = table_of(HQ * D), table_of(HK * D), table_of(HK * D)
    ek[:, ::D] = 1.0
    ev[:, ::D] = 1.0
    mix = dev((g.standard_normal((HQ * D, VOCAB)) / 3).astype(np.float32))
    fixed, width, rows = shared // PAGE, (shared + 200) // PAGE + 2, DRAFTS + 1
    new_first = shared % PAGE + 1                                         # the rest of the prompt comes with the first step
    m = batch * max(rows, new_first) + 5                                  # a padded batch
    pages = fixed + batch * 8 + 3
    ids = g.permutation(pages)
    table = np.full((batch, width), -3, np.int32)
    table[:, :fixed] = ids[:fixed]
    free = np.concatenate([ids[fixed:], np.full(fixed, -9)]).astype(np.int32)
    k, v = (torch.zeros((pages, HK, PAGE, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((pages, HK), device="cuda") for _ in range(2))
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    # the prefix's whole pages, written once
    prompt = g.integers(0, VOCAB, shared)
    whole = fixed * PAGE
    first = dev(prompt[:whole])
    flag = err_flag()
    q4k.q4k_kv_append(ek[first], ev[first], whole, HK, D, HK * D, HK * D, None, 1e-6, None, 0, 0, i32([0, whole]), i32([whole]),
                      i32(table[:1]), 1, width, PAGE, pages, k, v, ks, vs, flag)
    # state on the device
    t = dict(kept=i32([whole] * batch), new=i32([rows] * batch), fixed=i32([fixed] * batch), held=i32([0] * batch), free=dev(free),
             count=i32([pages - fixed]), table=dev(table), lens=i32([0] * batch), start=i32([0] * (batch + 1)), pos=i32([0] * m),
             slots=torch.zeros(m, dtype=torch.int64, device="cuda"), tokens=i32([0] * m), accepted=i32([0] * batch), next=i32([0] * batch),
             ua=torch.zeros(m, device="cuda"), us=torch.zeros(batch, device="cuda"), temperature=torch.ones(batch, device="cuda"),
             group=i32([0, batch]), prefix=i32([shared]), logits=torch.zeros((m, VOCAB), device="cuda"),
             probs=torch.zeros((m, VOCAB), device="cuda"), out=torch.zeros((m, HQ * D), dtype=tt, device="cuda"),
             q=torch.zeros((m, HQ * D), dtype=tt, device="cuda"))
    ws_a = torch.full((q4k.q4k_shared_prefix_attention_workspace_size(batch, 1, m, HQ, HK, D),), 0xFF, dtype=torch.uint8, device="cuda")
    ws_v = torch.full((q4k.q4k_verify_drafts_workspace_size(batch, m, VOCAB),), 0xFF, dtype=torch.uint8, device="cuda")

    def step(max_q):
        q4k.q4k_page_tables(t["kept"], t["new"], t["fixed"], batch, m, width, PAGE, pages, t["held"], t["free"], t["count"], t["table"],
                            t["held"], t["count"], t["start"], t["lens"], t["pos"], t["slots"], flag)
        tokens = t["tokens"].long()
        t["q"].copy_(eq[tokens])
        q4k.q4k_kv_append(ek[tokens], ev[tokens], m, HK, D, HK * D, HK * D, None, 1e-6, None, 0, 0, t["start"], t["lens"], t["table"],
                          batch, width, PAGE, pages, k, v, ks, vs, flag)
        q4k.q4k_shared_prefix_attention(t["q"], m, HQ, HK, D, HQ * D, k, v, ks, vs, t["start"], t["lens"], t["table"], batch, width, PAGE,
                                        pages, t["group"], t["prefix"], 1, max_q, shared + 200, shared, 0.125, 0, t["out"], HQ * D, ws_a,
                                        len(ws_a), flag)
        torch.matmul(t["out"].float(), mix, out=t["logits"])
        q4k.q4k_verify_drafts(t["logits"], m, VOCAB, VOCAB, t["probs"], VOCAB, t["tokens"], t["start"], batch, t["temperature"], t["ua"],
                              t["us"], t["lens"], t["accepted"], t["next"], t["kept"], ws_v, len(ws_v), flag)

    text = [list(prompt[:whole]) for _ in range(batch)]                   # what each sequence's cache holds
    todo = [list(prompt[whole:]) + [int(g.integers(VOCAB))] for _ in range(batch)]   # its rows of the coming step that are no drafts
    graph = None
    for at in range(6):
        drafts = 0 if at == 0 else DRAFTS
        new = [len(x) + drafts for x in todo]
        if at == 3:
            new[2] = 0                                                    # a sequence that pauses
        if at >= 4:
            new[5] = 0
            t["kept"][5:6] = 0                                            # one that has ended
        probs = np.abs(g.standard_normal((m, VOCAB))).astype(np.float32) ** 4
        probs /= probs.sum(1, keepdims=True)
        tokens, r = g.integers(0, VOCAB, m), 0
        for i in range(batch):
            if new[i] == 0:
                continue
            tokens[r:r + len(todo[i])] = todo[i]
            r += new[i]
        ua, us = g.random(m).astype(np.float32) * 0.2, g.random(batch).astype(np.float32)
        if drafts == 0:
            ua[:] = 0.0                                                   # the prompt's rows pass as drafts that are always accepted
        else:
            t["temperature"].copy_(dev(np.resize([0.7, 0.0, 1.3], batch).astype(np.float32)))
        for name, x in (("tokens", tokens), ("new", new)):
            t[name].copy_(i32(x))
        for name, x in (("probs", probs), ("ua", ua), ("us", us)):
            t[name].copy_(dev(x))
        ints = lambda name: [int(x) for x in host(t[name])]  # noqa: E731
        want, flags = plain_tables(ints("kept"), new, ints("fixed"), ints("held"), host(t["table"]), host(t["free"]), ints("count")[0], m, PAGE)
        assert not flags
        kept = ints("kept")
        t["out"].fill_(0)
        if graph is None and at >= 1:
            saved = {name: x.clone() for name, x in t.items()}
            step(rows)                                                    # once outside, as a warm-up of the library's product; then undone
            torch.cuda.synchronize()
            for name, x in saved.items():
                t[name].copy_(x)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(rows)
        if graph is None:
            step(new_first)
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert int(flag) == 0
        for name, x in want.items():
            got = host(t[name])
            assert np.array_equal(got, np.asarray(x).reshape(got.shape)), (at, name)
        # the cache: every sequence's tokens at their places
        start, lens, tab = want["start"], want["lens"], host(t["table"])
        cache, c = Codes(k, v, ks, vs), {}
        for i in range(batch):
            text[i] = text[i][:kept[i]] + [int(x) for x in tokens[start[i]:start[i + 1]]]
            assert len(text[i]) == lens[i]
            if not lens[i]:
                continue
            for side, e in (("k", ek), ("v", ev)):
                x = f64(e[dev(np.asarray(text[i]))]).reshape(lens[i], HK, D)
                page_ids = tab[i, :-(-lens[i] // PAGE)]
                x = x.transpose(1, 0, 2)
                scale = np.repeat(cache.scale[side][page_ids].astype(np.float64), PAGE, 0)[:lens[i]].T[:, :, None]
                assert (np.abs(cache.values(side, page_ids, lens[i]) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale)).all(), (at, i, side)
        # attention over what the cache holds
        n = start[-1]
        new_rows = np.diff(start).tolist()
        q = f64(t["q"])[:n].reshape(n, HQ, D)
        ref, tol = attention_ref(q, cache, tab, new_rows, lens, HQ // HK, 0.125, 0, dtype)
        none, _ = attention_ref(q, Codes(k, v, ks, vs, True), tab, new_rows, lens, HQ // HK, 0.125, 0, "f32")
        tol = tol + 2 * (2.0 ** -22 + 2.0 ** -21 + (2 * 152 + 8) * U) * none
        assert (np.abs(f64(t["out"])[:n].reshape(n, HQ, D) - ref) <= tol).all(), at
        assert (f64(t["out"])[n:] == 0).all()                             # rows behind the last sequence
        # the verdicts, from the logits that the call read
        got = ints("next")
        acc, nxt, stay, flags = plain_verify(host(t["logits"]), probs, tokens.tolist(), start, host(t["temperature"]), ua, us, lens, drawn=got)
        assert ints("accepted") == acc and got == nxt and ints("kept") == stay
        for i in range(batch):
            if new_rows[i]:
                todo[i] = [got[i]]
    assert max(ints("accepted")) > 0 and min(ints("accepted")) < DRAFTS   # drafts of both kinds came
