"""pa_tree_decode where the largest tree is far above the batch's, and the calls of a verification step back to back on
the device, each reading what the one before has just written."""
import random

import pytest
import torch

import paged_kv_cache_232_gb300 as pa
from test_gpu_tree import Batch
from tree_testutil import gen, randn, tree_sees, words_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (8, 2, 128), (16, 1, 128), (4, 1, 64), (3, 1, 96), (4, 2, 256), (16, 1, 256)])
@pytest.mark.parametrize("ns,most", [([1, 3], 300), ([1, 300, 2], 300), ([130, 0, 1, 7], 513), ([5], 2000)])
def test_largest_tree_far_above_the_batch(hq, hkv, d, ns, most):
    """max_q_len is a bound (a captured call keeps it): blocks of tokens in which a sequence has no rows are passed over."""
    b = Batch("bf16", hq, hkv, d, 16, ns, [(211 * i + 40) % 700 for i in range(len(ns))], seed=most + d,
              extra_words=-(-most // 64) - max(1, -(-max(ns) // 64)))
    b.max_n = most
    pa.pa_device_errors(clear=True)
    out = b.run()
    assert pa.pa_device_errors(clear=True) == 0
    b.check(out)


@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 2, 128, 16), (8, 8, 64, 32), (16, 4, 128, 8)])
def test_each_call_reads_what_the_one_before_wrote(hq, hkv, d, bs):
    """Room for the drafted tokens, attention, the accepted path, the rest given back, a fork, decode and a causal chunk, without
    another kernel between them: the same as with a wait after each call."""
    dt, S, mb = torch.bfloat16, 40, 64 * 16 // bs
    nb = S * mb + 5
    g, rng = gen(bs + d), random.Random(bs)
    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)
    kc, vc = (randn(g, (nb, bs, hkv, d), dt) for _ in range(2))
    free0 = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    ws = torch.empty(pa.pa_resize_workspace_size(S, nb), device="cuda", dtype=torch.uint8)
    most, parents = 12, [-1] * S
    for s in range(1, S, 4):          # every fourth sequence is ended and becomes a fork of the one before
        parents[s] = s - 1

    def make(turn):
        """A step's inputs: lengths, trees, paths."""
        ns = [rng.randint(1, most) for _ in range(S)]
        ctx = [rng.randint(1, 900) for _ in range(S)]
        sees = [tree_sees(rng, n) for n in ns]
        paths = [sorted(rng.sample(range(n), rng.randint(1, n))) for n in ns]
        loc = i32([sum(ns[:s]) for s in range(S + 1)])
        return dict(ctx=i32(ctx), grown=i32([c + n for c, n in zip(ctx, ns)]), loc=loc,
                    mask=torch.tensor([w for x in sees for w in words_of(x, 1)], device="cuda"),
                    path=i32([p + [-1] * (most - len(p)) for p in paths]), acc=i32([len(p) for p in paths]),
                    ended=i32([0 if p >= 0 else -1 for p in parents]), parents=i32(parents),
                    q=randn(g, (sum(ns), hq, d), dt), dq=randn(g, (S, hq, d), dt),
                    none=torch.zeros(S, device="cuda", dtype=torch.int32))

    tws = torch.empty(pa.pa_tree_workspace_size(hq, hkv, d, most), device="cuda", dtype=torch.uint8)
    dws = torch.empty(max(16, pa.pa_decode_workspace_size(S, hq, d, mb * bs, 0)), device="cuda", dtype=torch.uint8)

    def step(x, wait):
        st = dict(k=kc.clone(), v=vc.clone(), bt=torch.full((S, mb), -1, device="cuda", dtype=torch.int32),
                  lens=torch.zeros(S, device="cuda", dtype=torch.int32), ref=torch.zeros(nb, device="cuda", dtype=torch.int32),
                  free=free0.clone(), count=i32([nb]), new=torch.zeros(S, device="cuda", dtype=torch.int32),
                  out=torch.zeros_like(x["q"]), dec=torch.zeros_like(x["dq"]), chunk=torch.zeros_like(x["dq"]))
        one = torch.arange(S + 1, device="cuda", dtype=torch.int32)

        def resize(new):
            pa.pa_resize_pages(st["k"], st["v"], st["bt"], st["lens"], new, st["ref"], st["free"], st["count"], ws)

        calls = [lambda: resize(x["ctx"]), lambda: resize(x["grown"]),
                 lambda: pa.pa_tree_decode(st["out"], x["q"], st["k"], st["v"], st["bt"], x["loc"], st["lens"], x["mask"], most,
                                           0.1, tws),
                 lambda: pa.pa_tree_commit(st["k"], st["v"], st["bt"], x["loc"], st["lens"], x["path"], x["acc"], st["new"]),
                 lambda: resize(st["new"]), lambda: resize(x["ended"]),
                 lambda: pa.pa_fork_pages(st["bt"], st["lens"], x["parents"], st["ref"], bs),
                 lambda: pa.pa_decode(st["dec"], x["dq"], st["k"], st["v"], st["bt"], st["lens"], mb * bs, 0.1, workspace=dws),
                 lambda: pa.pa_prefill_chunk(st["chunk"], x["dq"], st["k"], st["v"], st["bt"], one, st["lens"], 1, 0.1),
                 lambda: resize(x["none"])]
        torch.cuda.synchronize()
        for call in calls:
            call()
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return st

    pa.pa_device_errors(clear=True)
    for turn in range(6):
        x = make(turn)
        want, got = step(x, True), step(x, False)
        for name in want:
            assert torch.equal(want[name], got[name]), (turn, name)
        assert got["count"].item() == nb and not got["ref"].any()
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("hq,S,longest", [(8, 6, 5000), (4, 200, 900), (4, 3, 100)])
def test_copy_of_pages_that_a_decode_step_has_just_written(hq, S, longest):
    """The step's rows (one call writes and decodes; with a bound on the lengths that asks for a merge, though no row has
    anything to merge) are in the copies that follow at once."""
    dt, bs, hkv, d = torch.bfloat16, 16, 4, 128
    g, nb, mb = gen(S), 4 * S + 1, -(-longest // 16)
    kc, vc = (randn(g, (nb, bs, hkv, d), dt) for _ in range(2))
    lens = [1 + (7 * i) % 30 for i in range(S)]
    bt = torch.full((S, mb), -1, device="cuda", dtype=torch.int32)
    bt[:, :2] = torch.randperm(nb, generator=g, device="cuda")[:2 * S].view(S, 2).to(torch.int32)
    cl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    last = torch.gather(bt.long(), 1, ((cl.long() - 1) // bs)[:, None])[:, 0]
    used = torch.zeros(nb, device="cuda", dtype=torch.bool)
    used[bt[:, :2].long()] = True
    to = torch.nonzero(~used)[:S, 0]
    pairs = torch.stack([last, to], 1).to(torch.int32).contiguous()
    ws = torch.empty(max(16, pa.pa_decode_workspace_size(S, hq, d, longest, 0)), device="cuda", dtype=torch.uint8)
    q, out = randn(g, (S, hq, d), dt), torch.empty((S, hq, d), device="cuda", dtype=dt)
    at = (cl.long() - 1) % bs
    for _ in range(10):
        k, v = randn(g, (S, hkv, d), dt), randn(g, (S, hkv, d), dt)
        torch.cuda.synchronize()
        pa.pa_decode_write(out, q, kc, vc, bt, cl, longest, 0.1, k, v, last * bs + at, workspace=ws)
        pa.pa_copy_pages(kc, vc, pairs)
        assert torch.equal(kc[to, at], k) and torch.equal(vc[to, at], v)
        assert torch.equal(kc[to], kc[last]) and torch.equal(vc[to], vc[last])
