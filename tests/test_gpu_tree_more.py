"""pa_tree_decode where the largest tree is far above the batch's, and the calls of a verification step back to back on
the device, each reading what the one before has just written."""
import random

import pytest
import torch

import paged_kv_cache_232_gb300 as pa
from test_gpu_tree import Batch
from tree_testutil import attend64, gen, half_step, randn, tiny, tree_sees, words_of

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


def _check_weights(out, q, k, v, sees, scale, what):
    """The bound of tree_testutil with weights of twice the type's bits: a weight enters the product as its rounded value and
    the rounded remainder, so it is off by u^2 of itself (u: half a step of the type) instead of u, and in fp16, where a
    remainder below 2^-20 of the largest weight is subnormal, by at most 2^-31 of the sum; twice as many additions."""
    dt, T = out.dtype, k.shape[0]
    want, spread, mag, ds = attend64(q, k, v, sees, scale)
    e = ds + 2.0 ** -20 + half_step(dt) ** 2
    d = e / (1 - e) * spread + (2 * T / 16 + 40) * 2.0 ** -23 * mag
    if dt == torch.float16:
        d = d + T * 2.0 ** -31 * v.double().abs().amax() * sees.any(-1)[:, None, None, None]
    err = (out.double().reshape(want.shape) - want).abs()
    bad = ~(err <= half_step(dt) * (want.abs() + d) + d + tiny(dt))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off; largest error {float(err.max()):.3e}"


@pytest.mark.parametrize("ty", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,d,n", [(2, 1, 128, 9), (4, 1, 128, 12), (8, 2, 128, 30), (4, 1, 128, 70), (2, 2, 64, 16), (3, 1, 64, 20),
                                          (8, 1, 64, 16), (6, 2, 96, 40), (2, 1, 256, 16), (4, 1, 256, 16), (4, 2, 256, 33)])
def test_weights_keep_their_remainders(ty, hq, hkv, d, n):
    """A value is off by its own rounding and hardly more: as pa_prefill_chunk's, whose causal chunk a chain of drafted tokens
    is.  Contexts within a tile, over several and split over CTAs; references raised on the way; every kernel."""
    for ctxs, growth in (([0, 40, 300], 0), ([9000, 5, 700], 0), ([1500, 700, 30], 30)):
        b = Batch(ty, hq, hkv, d, 16, [n] * 3, ctxs, seed=d + n + growth)
        if growth:                        # keys that grow along the context
            for s in range(3):
                t = torch.arange(b.lens[s], device="cuda")
                b.k[s] = (b.k[s].float() * (t.float()[:, None, None] / b.lens[s] * growth)).to(b.dt)
                b.kc[b.bt[s, t // 16].long(), t % 16] = b.k[s]
        out = b.run()
        for s in range(3):
            at = slice(b.loc[s], b.loc[s + 1])
            _check_weights(out[at], b.q[at], b.k[s], b.v[s], b.all_seen(s), b.scale, f"{ctxs[s]} tokens, growth {growth}")


@pytest.mark.parametrize("ty,value", [("fp16", "inf"), ("bf16", "-inf"), ("bf16", "nan"), ("fp16", "nan")])
@pytest.mark.parametrize("hq,hkv,d,n", [(4, 2, 128, 9), (8, 2, 128, 16), (16, 2, 128, 16), (8, 2, 128, 70), (4, 2, 64, 16), (16, 2, 64, 16),
                                          (4, 2, 256, 16), (16, 2, 256, 16)])
def test_cached_value_that_is_not_finite_spoils_its_column_alone(ty, value, hq, hkv, d, n):
    """A V row of the context, which every drafted token sees: that column of its KV head's rows is not finite, whatever the
    number of rows (32, 64, 128 and more of them), and nothing else changes.  In a tile of context alone and in the
    last one, beside the drafted tokens."""
    b = Batch(ty, hq, hkv, d, 16, [n, n], [270, 100], seed=n + d)
    want, kept, g = b.run(), b.vc.clone(), hq // hkv
    assert want.isfinite().all()
    for t, col in ((30, 5), (269, d - 1)):
        b.vc[b.bt[0, t // 16].long(), t % 16, 1, col] = float(value)
        out = b.run()
        assert not out[:n, g:, col].isfinite().any()
        out[:n, g:, col] = want[:n, g:, col]
        assert torch.equal(out, want)
        b.vc.copy_(kept)


@pytest.mark.parametrize("hq,hkv,d,n", [(4, 2, 128, 9), (8, 2, 128, 16), (16, 2, 128, 16), (8, 2, 64, 70), (16, 2, 256, 16)])
def test_scores_that_are_all_minus_infinity(hq, hkv, d, n):
    """Such rows are zero, as those that see nothing; the other KV head's rows are not touched by it."""
    b = Batch("bf16", hq, hkv, d, 16, [n, n], [270, 3], seed=n)
    want, g = b.run(), hq // hkv
    b.q[:, g:, 0] = 1.0
    b.kc[:, :, 1, 0] = float("-inf")
    out = b.run()
    assert not out[:, g:].any() and torch.equal(out[:, :g], want[:, :g])
