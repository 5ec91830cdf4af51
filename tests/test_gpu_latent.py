"""pa_latent_decode and pa_latent_prefill_chunk against attention in 64 bits (bounds:
latent_testutil).  Rows of the cache that no sequence owns hold NaN and unused table entries point
past the pool, so that a read out of place shows."""
import math

import pytest
import torch

import paged_kv_cache_232_gb300 as pa
from latent_testutil import ROPE, TYPES, check_attend, check_write, gen, half_step, norm64, paged, randn, table, turn64

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(192)


def _ws(h, dl, max_q=1):
    return torch.full((pa.pa_latent_workspace_size(h, dl, max_q),), 0xFF, device="cuda", dtype=torch.uint8)


def _decode(q, cache, bt, lens, scale=SCALE, ws=None):
    dl = cache.shape[2] - ROPE
    out = torch.full((*q.shape[:2], dl), float("nan"), device="cuda", dtype=q.dtype)
    cl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    pa.pa_latent_decode(out, q, cache, bt, cl, scale, _ws(q.shape[1], dl) if ws is None else ws)
    return out


def _check_decode(ty, h, dl, bs, lens, seed, q_scale=1.0):
    g = gen(seed)
    cache, bt, rows = paged(g, lens, bs, dl, TYPES[ty])
    q = randn(g, (len(lens), h, dl + ROPE), TYPES[ty], q_scale)
    pa.pa_device_errors(clear=True)
    out = _decode(q, cache, bt, lens)
    assert pa.pa_device_errors(clear=True) == 0
    for s, r in enumerate(rows):
        check_attend(out[s:s + 1], q[s:s + 1], r, SCALE, dl, 1, f"sequence {s} of {lens[s]}")


@pytest.mark.parametrize("ty,h,dl,bs,lens", [
    ("fp16", 16, 512, 16, [1]),
    ("fp16", 16, 512, 16, [130]),
    ("bf16", 16, 512, 16, [64, 1, 0, 63, 65, 128, 7]),
    ("fp16", 1, 512, 16, [5, 300]),
    ("bf16", 17, 512, 8, [200, 9, 64]),
    ("fp16", 32, 512, 32, [77, 250, 31]),
    ("bf16", 33, 512, 64, [100, 64, 1]),
    ("fp16", 64, 512, 128, [129, 500]),
    ("fp16", 65, 512, 64, [70, 0, 3]),
    ("bf16", 128, 512, 16, [333, 64]),
    ("fp16", 113, 512, 8, [90]),
    ("fp16", 16, 256, 16, [1, 64, 200]),
    ("bf16", 24, 256, 8, [500, 13]),
    ("fp16", 64, 256, 32, [129, 66]),
    ("bf16", 128, 256, 128, [300, 257]),
])
def test_decode_matches_formula(ty, h, dl, bs, lens):
    _check_decode(ty, h, dl, bs, lens, seed=h + sum(lens))


@pytest.mark.parametrize("ty,h,bs", [("fp16", 16, 16), ("bf16", 64, 64), ("fp16", 128, 64)])
def test_decode_splits_long_contexts(ty, h, bs):
    """One and few sequences: every CTA gets a part of a context, its partials are joined."""
    _check_decode(ty, h, 512, bs, [20011], seed=1)
    _check_decode(ty, h, 512, bs, [9000, 12345, 17], seed=2)


@pytest.mark.parametrize("h", [16, 70])
def test_decode_many_sequences(h):
    """More sequences than threads of a CTA and than CTAs, empty ones among them."""
    lens = [(37 * i) % 150 for i in range(701)]
    _check_decode("fp16", h, 512, 16, lens, seed=3)


@pytest.mark.parametrize("h,dl", [(16, 512), (64, 512), (128, 512), (32, 256)])
def test_decode_finds_each_token(h, dl):
    """A query that matches one token's row alone returns that token's latent part to half a step: every
    position of the context in turn (a sequence each), so a token dropped, doubled or misplaced shows."""
    dt, bs, L = torch.float16, 16, 150
    g = gen(h)
    cache, bt, rows = paged(g, [L], bs, dl, dt)
    r = rows[0]
    q = (r * (200.0 / (r.double() ** 2).sum(1, keepdim=True) / SCALE)).to(dt)[:, None].expand(L, h, dl + ROPE).contiguous()
    out = _decode(q, cache, bt.expand(L, -1).contiguous(), [L] * L)
    s = torch.einsum("ak,tk->at", q[:, 0].double(), r.double()) * SCALE
    w = torch.softmax(s, -1)
    other = (1 - w.diagonal()).max()
    assert other < 2.0 ** -14      # (of the inputs: the match dominates)
    want = r[:, None, :dl].double()
    err = (out.double() - want).abs()
    assert (err <= half_step(dt) * want.abs() + 2.0 ** -12 * 8 + 2.0 ** -25).all()


@pytest.mark.parametrize("h", [16, 40, 128])
def test_decode_rising_scores_rescale(h):
    """Scores that grow along the context by far more than the lazy rescale's 2^8, others that fall: heads of
    both kinds, in both halves of a pair."""
    dt, dl, L = torch.float16, 512, 1000
    g = gen(9)
    cache, bt, rows = paged(g, [L], 16, dl, dt)
    r = rows[0].clone()
    q = randn(g, (1, h, dl + ROPE), dt, 0.05)
    r[:, dl] = torch.linspace(-8, 8, L, device="cuda").to(dt)
    q[0, :, dl] = torch.linspace(-60, 60, h, device="cuda").to(dt)
    blocks = bt[0, :-(-L // 16)].long()
    t = torch.arange(L, device="cuda")
    cache[blocks[t // 16], t % 16] = r
    out = _decode(q, cache, bt, [L], scale=1.0)
    check_attend(out, q, r, 1.0, dl, 1, "rising scores")


def _rising(g, q, rows, cache, bt, dl, bs, seqs):
    """Scores that grow along each sequence for the query rows [n, H] with a positive column dl of q, and fall for the
    others: by sequence the rows that rise are all, the first 64 of a unit, those behind them, or a mixed set, so that the
    two CTAs of a pair rescale in the same tiles, in different ones, or not at all."""
    for s in seqs:
        r, at = rows[s], q[s]
        if not len(r):
            continue
        r[:, dl] = torch.linspace(-8, 8, len(r), device="cuda").to(r.dtype)
        t = torch.arange(len(r), device="cuda")
        cache[bt[s, t // bs].long(), t % bs] = r
        n = at.shape[0] * at.shape[1]
        up = torch.arange(n, device="cuda")
        up = (up >= 0, up % 128 < 64, up % 128 >= 64, up % 3 == 0, up < 0)[s % 5].view(at.shape[:2])
        size = torch.linspace(20, 60, n, device="cuda").view(at.shape[:2])
        at[..., dl] = torch.where(up, size, -size).to(q[s].dtype)


@pytest.mark.parametrize("ty", ["fp16", "bf16"])
@pytest.mark.parametrize("h,dl", [(65, 512), (100, 256), (100, 512), (128, 256), (128, 512)])
def test_decode_rescales_in_many_tiles_of_several_units(h, dl, ty):
    """Three units a pair and more, of one to six tiles, whose rows outgrow their reference in most tiles: the factors
    of every tile reach both CTAs of the pair in time (both parities, across the units' ends)."""
    g = gen(61 + h)
    lens = [1 + (97 * i) % 700 for i in range(240)]
    bs = 16
    cache, bt, rows = paged(g, lens, bs, dl, TYPES[ty])
    q = randn(g, (len(lens), 1, h, dl + ROPE), TYPES[ty], 0.05)
    _rising(g, q, rows, cache, bt, dl, bs, range(len(lens)))
    q = q[:, 0]
    pa.pa_device_errors(clear=True)
    out = _decode(q, cache, bt, lens, scale=1.0)
    for _ in range(10):
        assert torch.equal(_decode(q, cache, bt, lens, scale=1.0), out)
    assert pa.pa_device_errors(clear=True) == 0
    for s, r in enumerate(rows):
        check_attend(out[s:s + 1], q[s:s + 1], r, 1.0, dl, 1, f"sequence {s} of {lens[s]}")


@pytest.mark.parametrize("ty", ["fp16", "bf16"])
@pytest.mark.parametrize("h,dl,n", [(16, 512, 8), (48, 256, 5), (128, 512, 3)])
def test_chunk_rescales_in_many_tiles_of_several_units(h, dl, n, ty):
    """The same over chunks of a few tokens, in units of 128, 96 and 128 rows (one to three units a chunk)."""
    g = gen(71 + h)
    lens = [n + (89 * i) % 600 for i in range(110)]
    bs, C = 32, 110
    cache, bt, rows = paged(g, lens, bs, dl, TYPES[ty])
    q = randn(g, (C, n, h, dl + ROPE), TYPES[ty], 0.05)
    _rising(g, q, rows, cache, bt, dl, bs, range(C))
    q = q.flatten(0, 1)

    def call():
        out = torch.full((C * n, h, dl), float("nan"), device="cuda", dtype=TYPES[ty])
        pa.pa_latent_prefill_chunk(out, q, cache, bt, torch.arange(0, C * n + 1, n, device="cuda", dtype=torch.int32),
                                   torch.tensor(lens, device="cuda", dtype=torch.int32), n, 1.0, _ws(h, dl, n))
        return out

    pa.pa_device_errors(clear=True)
    out = call()
    for _ in range(10):
        assert torch.equal(call(), out)
    assert pa.pa_device_errors(clear=True) == 0
    for c, r in enumerate(rows):
        check_attend(out[c * n:(c + 1) * n], q[c * n:(c + 1) * n], r, 1.0, dl, n, f"chunk {c} of {lens[c]}")


@pytest.mark.parametrize("ty", ["fp16", "bf16"])
@pytest.mark.parametrize("h", [16, 128])
def test_decode_many_small_equal_weights(h, ty):
    """One token far above 40,000 equal ones of 2^-22 its weight each (1 % together): their common rounding must not
    show, so the weights may not be fp16 subnormals."""
    dt, dl, L = TYPES[ty], 512, 40001
    g = gen(15)
    cache, bt, rows = paged(g, [L], 64, dl, dt)
    r = rows[0]
    r[:] = 0
    r[1:, :dl] = 1.0
    r[:, dl] = 0.75
    r[7, dl], r[7, :dl], r[0, :dl] = 16.0, 0.0, 1.0
    blocks = bt[0, :-(-L // 64)].long()
    t = torch.arange(L, device="cuda")
    cache[blocks[t // 64], t % 64] = r
    q = torch.zeros((1, h, dl + ROPE), device="cuda", dtype=dt)
    q[..., dl] = 1.0
    out = _decode(q, cache, bt, [L], scale=1.0)
    check_attend(out, q, r, 1.0, dl, 1, "small weights")


def test_decode_negative_and_zero_scale():
    g = gen(4)
    cache, bt, rows = paged(g, [333], 16, 512, torch.float16)
    q = randn(g, (1, 16, 576), torch.float16)
    for sc in (-SCALE, 0.0):
        out = _decode(q, cache, bt, [333], scale=sc)
        ref = attend_sign(q, rows[0], sc)
        check_attend(out, ref[0], rows[0], ref[1], 512, 1, f"scale {sc}")


def attend_sign(q, rows, sc):
    """(q with the scale's sign, |scale|): the same scores."""
    return (-q, -sc) if sc < 0 else (q, sc)


@pytest.mark.parametrize("h", [16, 128])
def test_decode_nonfinite_rows_stay_in_their_sequence(h):
    g = gen(5)
    lens = [100, 90, 80]
    cache, bt, rows = paged(g, lens, 16, 512, torch.bfloat16)
    q = randn(g, (3, h, 576), torch.bfloat16)
    q[1, 3, 0] = float("nan")
    out = _decode(q, cache, bt, lens)
    assert torch.isnan(out[1, 3]).all()
    keep = torch.ones(h, dtype=torch.bool, device="cuda")
    keep[3] = False
    assert torch.isfinite(out[1, keep]).all()
    for s in (0, 2):
        check_attend(out[s:s + 1], q[s:s + 1], rows[s], SCALE, 512, 1, f"sequence {s}")
    cache[bt[0, 2].long(), 5] = float("inf")     # token 37 of sequence 0: inf - inf in its output
    out2 = _decode(q, cache, bt, lens)
    assert torch.isnan(out2[0]).any() and torch.equal(out2[2], out[2])


@pytest.mark.parametrize("h", [8, 100])
def test_decode_bad_lengths_and_blocks_are_flagged(h):
    g = gen(6)
    lens = [100, 90, 80]
    cache, bt, rows = paged(g, lens, 16, 512, torch.bfloat16)
    q = randn(g, (3, h, 576), torch.bfloat16)
    pa.pa_device_errors(clear=True)
    out = _decode(q, cache, bt, [100, -5, bt.shape[1] * 16 + 1])
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_LENGTH
    assert not out[1].any() and not out[2].any()
    check_attend(out[:1], q[:1], rows[0], SCALE, 512, 1, "the good one")
    bt[1, 1] = cache.shape[0]
    bt[1, 2] = -3
    out = _decode(q, cache, bt, lens)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BLOCK
    r = rows[1].clone()
    r[16:48] = 0                                  # bad blocks read as zeros
    check_attend(out[1:2], q[1:2], r, SCALE, 512, 1, "zeros for the bad blocks")
    check_attend(out[2:], q[2:], rows[2], SCALE, 512, 1, "the good one")


@pytest.mark.parametrize("h", [16, 128])
def test_decode_repeats_bit_for_bit(h):
    g = gen(7)
    lens = [3000, 17, 5000]
    cache, bt, rows = paged(g, lens, 16, 512, torch.bfloat16)
    q = randn(g, (3, h, 576), torch.bfloat16)
    ws = _ws(h, 512)
    first = _decode(q, cache, bt, lens, ws=ws)
    for _ in range(5):
        assert torch.equal(_decode(q, cache, bt, lens, ws=ws), first)


@pytest.mark.parametrize("ty,h,dl,bs,ql,ctx", [
    ("fp16", 16, 512, 16, [1, 4, 5], [0, 100, 64]),
    ("bf16", 16, 512, 16, [70, 3], [130, 0]),
    ("fp16", 24, 256, 8, [1, 129, 0, 40], [700, 0, 50, 33]),
    ("fp16", 128, 512, 64, [65, 2], [10, 200]),
    ("bf16", 64, 512, 32, [33], [0]),
    ("fp16", 3, 512, 128, [150, 21], [1, 300]),
    ("fp16", 5, 256, 16, [2, 3, 1], [500, 2, 64]),
    ("bf16", 100, 256, 8, [20], [45]),
])
def test_chunk_matches_formula(ty, h, dl, bs, ql, ctx):
    g = gen(h + sum(ql))
    kl = [a + b for a, b in zip(ql, ctx)]
    cache, bt, rows = paged(g, kl, bs, dl, TYPES[ty])
    T = sum(ql)
    q = randn(g, (T + 2, h, dl + ROPE), TYPES[ty])
    out = torch.full((T + 2, h, dl), 7.0, device="cuda", dtype=TYPES[ty])
    loc = [sum(ql[:i]) for i in range(len(ql) + 1)]
    pa.pa_device_errors(clear=True)
    pa.pa_latent_prefill_chunk(out, q, cache, bt, torch.tensor(loc, device="cuda", dtype=torch.int32),
                               torch.tensor(kl, device="cuda", dtype=torch.int32), max(ql), SCALE, _ws(h, dl, max(ql)))
    assert pa.pa_device_errors(clear=True) == 0
    for c, n in enumerate(ql):
        if n:
            check_attend(out[loc[c]:loc[c + 1]], q[loc[c]:loc[c + 1]], rows[c], SCALE, dl, n, f"chunk {c}")
    assert (out[T:] == 7).all(), "rows behind the last chunk"


@pytest.mark.parametrize("ty,h,dl,ql,ctx", [("fp16", 128, 256, 1500, 3), ("bf16", 3, 256, 2100, 40), ("fp16", 30, 512, 1000, 0)])
def test_chunk_long(ty, h, dl, ql, ctx):
    """More units in a chunk than threads look for a range's start, units of one token, of 42 and of 4."""
    g = gen(ql)
    cache, bt, rows = paged(g, [ql + ctx, 5], 64, dl, TYPES[ty])
    q = randn(g, (ql + 2, h, dl + ROPE), TYPES[ty])
    out = torch.full((ql + 2, h, dl), float("nan"), device="cuda", dtype=TYPES[ty])
    pa.pa_device_errors(clear=True)
    pa.pa_latent_prefill_chunk(out, q, cache, bt, torch.tensor([0, ql, ql + 2], device="cuda", dtype=torch.int32),
                               torch.tensor([ql + ctx, 5], device="cuda", dtype=torch.int32), ql, SCALE, _ws(h, dl, ql))
    assert pa.pa_device_errors(clear=True) == 0
    for j0 in list(range(0, ql, 97)) + [ql - 1]:      # rows spread over the chunk, each over its own prefix
        check_attend(out[j0:j0 + 1], q[j0:j0 + 1], rows[0][:ctx + j0 + 1], SCALE, dl, 1, f"token {j0}")
    check_attend(out[ql:], q[ql:], rows[1], SCALE, dl, 2, "the short chunk")
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("h", [4, 20])
def test_chunk_many_chunks(h):
    """More chunks than threads of a CTA, empty ones among them."""
    n, dl = 900, 256
    ql = [(5 * i) % 4 for i in range(n)]
    kl = [a + (13 * i) % 200 for i, a in enumerate(ql)]
    g = gen(31)
    cache, bt, rows = paged(g, kl, 16, dl, torch.float16)
    loc = [sum(ql[:i]) for i in range(n + 1)]
    q = randn(g, (loc[-1], h, dl + ROPE), torch.float16)
    out = torch.full((loc[-1], h, dl), float("nan"), device="cuda", dtype=torch.float16)
    pa.pa_latent_prefill_chunk(out, q, cache, bt, torch.tensor(loc, device="cuda", dtype=torch.int32),
                               torch.tensor(kl, device="cuda", dtype=torch.int32), 3, SCALE, _ws(h, dl, 3))
    assert pa.pa_device_errors(clear=True) == 0
    for c in range(n):
        if ql[c]:
            check_attend(out[loc[c]:loc[c + 1]], q[loc[c]:loc[c + 1]], rows[c], SCALE, dl, ql[c], f"chunk {c}")


@pytest.mark.parametrize("h", [16, 128])
def test_cache_past_32_bit_offsets(h):
    """Blocks whose rows lie past 2^31 elements (and 2^32 bytes) of the cache: written, then attended."""
    dt, dl, bs = torch.bfloat16, 512, 64
    nb = (2 ** 31 // ((dl + ROPE) * bs)) + 40
    cache = torch.empty((nb, bs, dl + ROPE), device="cuda", dtype=dt)
    L = 300
    blocks = torch.arange(nb - 1, nb - 7, -1, device="cuda", dtype=torch.int32)
    bt = blocks[None].contiguous()
    cache[blocks.long()] = float("nan")
    g = gen(41)
    kv = randn(g, (L, dl + ROPE), dt)
    pos = torch.arange(L, device="cuda")
    slots = bt[0, pos // bs].long() * bs + pos % bs
    assert int(slots.min()) * (dl + ROPE) > 2 ** 31
    pa.pa_device_errors(clear=True)
    pa.pa_latent_rope_and_cache(kv, cache, slots, torch.zeros_like(pos), table(1, ROPE))     # position 0: unturned
    rows = cache[bt[0, pos // bs].long(), pos % bs]
    assert torch.equal(rows, kv)
    q = randn(g, (1, h, dl + ROPE), dt)
    out = _decode(q, cache, bt, [L])
    assert pa.pa_device_errors(clear=True) == 0
    check_attend(out, q, rows, SCALE, dl, 1, "far blocks")


def test_chunk_of_single_tokens_equals_decode():
    """q_len 1 everywhere: the decode call's result bit for bit when the units are the same size."""
    g = gen(8)
    lens = [100, 1, 640, 333]
    cache, bt, rows = paged(g, lens, 16, 512, torch.bfloat16)
    q = randn(g, (4, 64, 576), torch.bfloat16)
    out = torch.empty((4, 64, 512), device="cuda", dtype=torch.bfloat16)
    pa.pa_latent_prefill_chunk(out, q, cache, bt, torch.arange(5, device="cuda", dtype=torch.int32),
                               torch.tensor(lens, device="cuda", dtype=torch.int32), 1, SCALE, _ws(64, 512))
    assert torch.equal(out, _decode(q, cache, bt, lens))


def test_chunk_bad_lengths_are_flagged_and_skipped():
    g = gen(10)
    ql, kl = [4, 5, 6, 3], [40, 50, 60, 30]
    cache, bt, rows = paged(g, kl, 16, 512, torch.float16)
    q = randn(g, (18, 16, 576), torch.float16)
    loc = [0, 4, 9, 15, 18]

    def call(loc_, kl_, max_q):
        out = torch.full((18, 16, 512), 7.0, device="cuda", dtype=torch.float16)
        pa.pa_latent_prefill_chunk(out, q, cache, bt, torch.tensor(loc_, device="cuda", dtype=torch.int32),
                                   torch.tensor(kl_, device="cuda", dtype=torch.int32), max_q, SCALE, _ws(16, 512, 6))
        return out, pa.pa_device_errors(clear=True)

    pa.pa_device_errors(clear=True)
    out, err = call(loc, [40, 4, 60, 30], 6)              # chunk 1 longer than its kv length
    assert err == pa.PA_DEVERR_LENGTH and (out[4:9] == 7).all()
    check_attend(out[9:15], q[9:15], rows[2], SCALE, 512, 6, "chunk 2")
    out, err = call(loc, kl, 5)                           # chunk 2 longer than max_q_len
    assert err == pa.PA_DEVERR_LENGTH and (out[9:15] == 7).all()
    check_attend(out[15:], q[15:], rows[3], SCALE, 512, 3, "chunk 3")
    out, err = call([0, 4, 9, 15, 19], kl, 6)             # chunk 3 past the rows of q
    assert err == pa.PA_DEVERR_LENGTH and (out[15:] == 7).all()
    out, err = call(loc, [40, 50, bt.shape[1] * 16 + 1, 30], 6)
    assert err == pa.PA_DEVERR_LENGTH and (out[9:15] == 7).all()
    out, err = call([0, 0, 0, 0, 0], kl, 6)               # nothing to do
    assert err == 0 and (out == 7).all()


@pytest.mark.parametrize("heads", [(16, 16), (128, 16), (128, 100)])
def test_two_streams_with_their_own_workspaces(heads):
    g = gen(12)
    lens = [4000, 2500]
    cache, bt, rows = paged(g, lens, 16, 512, torch.bfloat16)
    qs = [randn(g, (2, h, 576), torch.bfloat16) for h in heads]
    want = [_decode(q, cache, bt, lens) for q in qs]
    cl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    outs, wss = [torch.empty_like(w) for w in want], [_ws(h, 512) for h in heads]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(8):
        for q, o, ws, st in zip(qs, outs, wss, streams):
            pa.pa_latent_decode(o, q, cache, bt, cl, SCALE, ws, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_two_captured_graphs_share_a_workspace():
    """Replayed one after the other on one stream: the second's call does not see what the first's left."""
    g = gen(14)
    cases = []
    ws = _ws(128, 512)
    for h, lens in ((128, [3000, 40]), (100, [900, 2222])):
        cache, bt, _ = paged(g, lens, 16, 512, torch.bfloat16)
        q, cl = randn(g, (2, h, 576), torch.bfloat16), torch.tensor(lens, device="cuda", dtype=torch.int32)
        out = torch.zeros((2, h, 512), device="cuda", dtype=torch.bfloat16)
        want = _decode(q, cache, bt, lens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.pa_latent_decode(out, q, cache, bt, cl, SCALE, ws)
        cases.append((graph, out, want, (cache, bt, q, cl)))
    for _ in range(3):
        for graph, out, _, _ in cases:
            out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _ in cases:
        assert torch.equal(out, want)


@pytest.mark.parametrize("h", [16, 128])
def test_step_graph_replay(h):
    """A captured write + decode step, replayed on new inputs, equals the eager step bit for bit."""
    g = gen(13)
    lens = [200, 1, 77, 640]
    dt, dl, bs = torch.bfloat16, 512, 16
    cache, bt, _ = paged(g, lens, bs, dl, dt, fill=0.0)
    cl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    pos = cl.long() - 1
    slots = bt[torch.arange(4, device="cuda"), pos // bs].long() * bs + pos % bs
    cs, w, ws = table(1000, ROPE), randn(g, (dl,), dt).abs() + 0.5, _ws(h, dl)
    kv, q = randn(g, (4, dl + ROPE), dt), randn(g, (4, h, dl + ROPE), dt)
    out = torch.empty((4, h, dl), device="cuda", dtype=dt)

    def step():
        pa.pa_latent_rope_and_cache(kv, cache, slots, pos, cs, weight=w, q_pe=q[..., dl:], q=q)
        pa.pa_latent_decode(out, q, cache, bt, cl, SCALE, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        gg = gen(seed)
        kv0, q0 = randn(gg, kv.shape, dt), randn(gg, q.shape, dt)
        kv.copy_(kv0)
        q.copy_(q0)
        step()
        torch.cuda.synchronize()
        want, want_cache = out.clone(), cache.clone()
        q.copy_(q0)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(cache, want_cache)


@pytest.mark.parametrize("inter", [False, True])
def test_layer_prefill_then_decode_against_expanded_attention(inter):
    """The operators as a layer uses them: write + chunk for a prompt in two chunks, then write + decode
    steps, from the raw projections; against expanded attention (per-head keys and values made from the
    latents) in 64 bits over the same 16-bit cache rows and absorbed queries."""
    dt, dl, h, bs, nope, vd = torch.float16, 512, 16, 16, 128, 128
    g = gen(21)
    total, first, second = 90, 50, 36            # then single tokens
    bt = torch.randperm(8, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    cache = torch.full((8, bs, dl + ROPE), float("nan"), device="cuda", dtype=dt)
    cs, w = table(200, ROPE), randn(g, (dl,), torch.float32, 0.1).add_(1).to(dt)
    w_uk, w_uv = randn(g, (h, nope, dl), torch.float64, 0.05), randn(g, (h, vd, dl), torch.float64, 0.05)
    kv = randn(g, (total, dl + ROPE), dt, 1.5)
    qn, pe = randn(g, (total, h, nope), torch.float64), randn(g, (total, h, ROPE), dt)
    q = torch.zeros((total, h, dl + ROPE), device="cuda", dtype=dt)
    q[..., :dl] = torch.einsum("thn,hnd->thd", qn, w_uk).to(dt)
    out = torch.zeros((total, h, dl), device="cuda", dtype=dt)
    pos = torch.arange(total, device="cuda")
    slots = bt[0, pos // bs].long() * bs + pos % bs
    ws = _ws(h, dl, first)
    pa.pa_device_errors(clear=True)
    at = 0
    for n in (first, second, 1, 1, 1, 1):
        s = slice(at, at + n)
        pa.pa_latent_rope_and_cache(kv[s], cache, slots[s], pos[s], cs, weight=w, q_pe=pe[s], q=q[s], interleaved=inter)
        kl = torch.tensor([at + n], device="cuda", dtype=torch.int32)
        if n > 1:
            loc = torch.tensor([0, n], device="cuda", dtype=torch.int32)
            pa.pa_latent_prefill_chunk(out[s], q[s], cache, bt, loc, kl, n, SCALE, ws)
        else:
            pa.pa_latent_decode(out[s], q[s], cache, bt, kl, SCALE, ws)
        at += n
    assert pa.pa_device_errors(clear=True) == 0
    # the cache: norms and rotations of the raw projections
    rows = cache[bt[0, pos // bs].long(), pos % bs]
    c = norm64(kv[:, :dl], w, 1e-6)
    check_write(rows[:, :dl], c, c.abs(), "latents")
    kr, km = turn64(kv[:, None, dl:].double(), cs[:total], inter)
    check_write(rows[:, dl:], kr[:, 0], km[:, 0], "keys")
    # every token over its own prefix (a chunk row by itself)
    for t in range(total):
        check_attend(out[t:t + 1], q[t:t + 1], rows[:t + 1], SCALE, dl, 1, f"token {t}")
    # the layer's output (values through the up-projection) against expanded attention from the unrounded queries:
    # the queries' rounding moves a score by at most u sum |q k|, everything else is bounded above
    r64 = rows.double()
    k_nope, v = torch.einsum("td,hnd->htn", r64[:, :dl], w_uk), torch.einsum("td,hvd->htv", r64[:, :dl], w_uv)
    qpe = turn64(pe.double(), cs[:total], inter)[0]
    s = (torch.einsum("qhn,htn->hqt", qn, k_nope) + torch.einsum("qhr,tr->hqt", qpe, r64[:, dl:])) * SCALE
    p = torch.softmax(s.masked_fill(torch.ones(total, total, device="cuda").triu(1).bool(), -math.inf), -1)
    want = torch.einsum("hqt,htv->qhv", p, v)
    got = torch.einsum("qhd,hvd->qhv", out.double(), w_uv)
    u = half_step(dt)
    # a score moves by ds (the roundings of q, and the kernel's fp32 sums), a weight by a factor of at most
    # exp(2 ds) and its own rounding; then the roundings of the output enter through |w_uv|
    qa = torch.cat([torch.einsum("thn,hnd->thd", qn, w_uk), qpe], -1).abs()
    ds = (u + 2.0 ** -16) * SCALE * torch.einsum("qhd,td->qht", qa, r64.abs()).amax(-1)
    e = torch.expm1(2 * ds) + u + 2.0 ** -14
    spread = torch.einsum("hqt,htv->qhv", p, v.abs()) + want.abs()
    allow = (e / (1 - e))[..., None] * spread + 2 * u * torch.einsum("qhd,hvd->qhv", out.double().abs(), w_uv.abs())
    assert ((got - want).abs() <= allow).all()
