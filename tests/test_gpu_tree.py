"""pa_tree_decode against attention in 64 bits (bounds: tree_testutil).  Rows of the caches that no sequence owns hold
NaN and unused table entries point past the pool, so that a read out of place shows."""
import math
import random

import pytest
import torch

import paged_kv_cache_232_gb300 as pa
from tree_testutil import TYPES, check_tree, gen, paged_kv, randn, tree_sees, words_of

pytestmark = pytest.mark.gpu


class Batch:
    """Trees of ns[s] drafted tokens behind ctxs[s] cached ones; sees[s]: which drafted token sees which."""

    def __init__(self, ty, hq, hkv, d, bs, ns, ctxs, seed, sees=None, extra_words=0, q_scale=1.0, total=None):
        g, rng = gen(seed), random.Random(seed)
        self.dt, self.ns, self.ctxs = TYPES[ty], ns, ctxs
        self.lens = [n + c if n else c for n, c in zip(ns, ctxs)]
        self.kc, self.vc, self.bt, self.k, self.v = paged_kv(g, self.lens, bs, hkv, d, self.dt, total=total)
        self.sees = sees or [tree_sees(rng, n) for n in ns]
        self.words = max(1, -(-max(ns) // 64)) + extra_words
        rows = [r for s in self.sees for r in words_of(s, self.words)]
        self.loc = [0]
        for n in ns:
            self.loc.append(self.loc[-1] + n)
        self.mask = torch.tensor(rows, device="cuda", dtype=torch.int64).reshape(self.loc[-1], self.words)
        self.q = randn(g, (self.loc[-1], hq, d), self.dt, q_scale)
        self.q_loc = torch.tensor(self.loc, device="cuda", dtype=torch.int32)
        self.sl = torch.tensor(self.lens, device="cuda", dtype=torch.int32)
        self.scale = 1.0 / math.sqrt(d)
        self.max_n, self.heads, self.d = max(ns), (hq, hkv), d

    def ws(self):
        return torch.full((pa.pa_tree_workspace_size(*self.heads, self.d, self.max_n),), 0xFF, device="cuda", dtype=torch.uint8)

    def run(self, out=None, ws=None, stream=None):
        out = torch.full_like(self.q, float("nan")) if out is None else out
        pa.pa_tree_decode(out, self.q, self.kc, self.vc, self.bt, self.q_loc, self.sl, self.mask, self.max_n, self.scale,
                          self.ws() if ws is None else ws, stream=stream)
        return out

    def all_seen(self, s):
        n = self.ns[s]
        tree = torch.tensor(self.sees[s], device="cuda", dtype=torch.bool).reshape(n, n)
        return torch.cat([torch.ones((n, self.ctxs[s]), device="cuda", dtype=torch.bool), tree], 1)

    def check(self, out, which=None):
        for s in range(len(self.ns)) if which is None else which:
            a, b = self.loc[s], self.loc[s + 1]
            if a < b:
                check_tree(out[a:b], self.q[a:b], self.k[s], self.v[s], self.all_seen(s), self.scale,
                           f"sequence {s}: {self.ns[s]} drafted behind {self.ctxs[s]}")


def _check(*args, **kw):
    b = Batch(*args, **kw)
    pa.pa_device_errors(clear=True)
    out = b.run()
    assert pa.pa_device_errors(clear=True) == 0
    b.check(out)


@pytest.mark.parametrize("ty,hq,hkv,d,bs,ns,ctxs", [
    ("fp16", 2, 2, 128, 16, [1], [0]),
    ("fp16", 2, 1, 128, 16, [1], [127]),
    ("bf16", 4, 2, 128, 16, [3, 1, 0, 7], [128, 0, 50, 125]),
    ("fp16", 8, 2, 128, 8, [8, 8], [300, 9]),
    ("bf16", 8, 1, 128, 32, [4, 2], [100, 260]),
    ("fp16", 8, 1, 128, 16, [5, 8], [77, 128]),          # 64 rows
    ("bf16", 16, 2, 128, 64, [16, 9], [500, 1]),         # 128 rows
    ("fp16", 3, 1, 128, 16, [11], [200]),                # odd group
    ("bf16", 5, 1, 128, 16, [25, 24], [64, 3]),
    ("fp16", 14, 2, 64, 16, [6, 18], [129, 10]),
    ("bf16", 16, 1, 64, 128, [3], [1000]),
    ("fp16", 4, 4, 64, 8, [1, 33], [0, 127]),
    ("bf16", 2, 2, 64, 16, [128], [50]),
    ("fp16", 4, 2, 96, 16, [7, 30], [100, 0]),
    ("bf16", 6, 2, 96, 32, [40], [333]),
    ("fp16", 4, 4, 256, 16, [5, 32], [63, 64]),
    ("bf16", 8, 2, 256, 8, [16], [200]),
    ("fp16", 16, 1, 256, 64, [8, 3], [65, 400]),
    ("bf16", 4, 2, 128, 16, [65, 64], [40, 300]),        # two blocks of tokens, the second not in every sequence
    ("fp16", 8, 1, 128, 16, [70, 3, 33], [200, 5, 0]),   # five blocks
    ("bf16", 16, 1, 64, 16, [100], [77]),                # thirteen blocks in two passes
    ("fp16", 16, 2, 256, 16, [20, 9], [100, 31]),
    ("fp16", 2, 1, 128, 16, [300], [10]),                # more drafted tokens than keys of a tile
])
def test_matches_formula(ty, hq, hkv, d, bs, ns, ctxs):
    _check(ty, hq, hkv, d, bs, ns, ctxs, seed=hq * d + sum(ns))


@pytest.mark.parametrize("hq,hkv,d,n", [(2, 2, 128, 5), (8, 2, 128, 16), (4, 1, 128, 33), (4, 4, 64, 9), (2, 1, 256, 20)])
def test_long_contexts_are_split(hq, hkv, d, n):
    """One and few sequences: every CTA gets a part of a context, its partials are joined."""
    _check("fp16", hq, hkv, d, 16, [n], [20011], seed=1)
    _check("bf16", hq, hkv, d, 32, [n, 1, n], [9000, 12345, 17], seed=2)


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (16, 2, 64)])
def test_many_sequences(hq, hkv, d):
    """More sequences than threads of a CTA and than CTAs, some without a tree."""
    _check("fp16", hq, hkv, d, 16, [i % 6 for i in range(701)], [(37 * i) % 150 for i in range(701)], seed=3)


@pytest.mark.parametrize("hq,hkv,d,n", [(16, 8, 128, 5), (32, 8, 128, 16), (64, 8, 128, 16), (32, 4, 128, 40), (64, 4, 128, 130),
                                        (8, 8, 64, 6), (16, 4, 64, 64), (8, 8, 256, 4), (32, 8, 256, 40)])
def test_many_units_a_cta(hq, hkv, d, n):
    """A CTA has more units than are told ahead of their work, most of a single tile."""
    _check("bf16", hq, hkv, d, 16, [1 + (7 * i) % n for i in range(300)], [(53 * i) % 290 for i in range(300)], seed=n)


@pytest.mark.parametrize("ty", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,d,n", [(1, 1, 128, 21), (4, 1, 128, 16), (8, 1, 128, 16), (2, 2, 64, 20), (2, 1, 256, 16)])
def test_any_mask(ty, hq, hkv, d, n):
    """Masks that are no trees: rows that do not see themselves, that see later tokens, and none; words behind the
    last token and bits from n on are not looked at."""
    rng = random.Random(n)
    sees = [[[rng.random() < 0.4 for _ in range(n)] for _ in range(n)] for _ in range(3)]
    sees[0][3], sees[2][0] = [False] * n, [False] * n
    b = Batch(ty, hq, hkv, d, 16, [n, n, n], [0, 100, 127], seed=5, sees=sees, extra_words=1)
    want = b.run()
    b.check(want)
    assert not want[3].any()                       # no context and an empty mask: zero
    b.mask[:, -1] = -1
    b.mask[:, 0] |= -1 << n
    out = b.run()
    assert torch.equal(out, want)


@pytest.mark.parametrize("hq,hkv,d,n,pad", [(2, 1, 128, 16, 5), (8, 1, 128, 16, 16), (2, 2, 64, 40, 7), (2, 1, 256, 30, 3),
                                              (2, 1, 128, 200, 150), (8, 1, 64, 70, 30)])
def test_padded_tokens_rows_may_hold_anything(hq, hkv, d, n, pad):
    """Rows of drafted tokens that nobody sees were never written: NaN and infinities there change nothing."""
    rng = random.Random(7)
    sees = [tree_sees(rng, n) for _ in range(2)]
    for s in sees:
        for j in range(n - pad, n):
            s[j] = [False] * n
    b = Batch("bf16", hq, hkv, d, 16, [n, n], [0, 123], seed=8, sees=sees)
    want = b.run()
    b.check(want)
    for s in range(2):
        for j in range(n - pad, n):
            t = b.ctxs[s] + j
            at = (b.bt[s, t // 16].long(), t % 16)
            b.kc[at] = float("nan") if j % 2 else float("-inf")
            b.vc[at] = float("inf") if j % 2 else float("nan")
    assert torch.equal(b.run(), want)


def test_value_that_is_not_finite_reaches_the_rows_that_see_it_alone():
    """One such row in the last tile, in an earlier one (trees over several tiles), in blocks of tokens that other CTAs
    work, in each half of a row's columns, and several at once."""
    for n, hq, hkv, d in ((12, 2, 1, 128), (12, 8, 1, 128), (12, 16, 1, 128), (12, 1, 1, 64), (12, 2, 1, 256), (300, 1, 1, 128),
                          (300, 2, 1, 64), (150, 2, 1, 256), (40, 8, 2, 128)):
        sees = [[[k <= j for k in range(n)] for j in range(n)]]
        b = Batch("fp16", hq, hkv, d, 16, [n], [250], seed=9, sees=sees)
        want = b.run()
        for rows, col, value in (([5], d - 3, "inf"), ([n - 1], 2, "nan"), ([n // 2, n // 2 + 3], d // 2 - 1, "-inf")):
            kept = b.vc.clone()
            for j in rows:
                t = 250 + j
                b.vc[b.bt[0, t // 16].long(), t % 16, 0, col] = float(value)
            out = b.run()
            g = hq // hkv
            assert torch.equal(out[:rows[0], :g], want[:rows[0], :g]) and out[rows[0]:, :g].isnan().all(), (n, hq, d, rows)
            assert torch.equal(out[:, g:], want[:, g:])          # the other KV heads' rows
            b.vc = kept


@pytest.mark.parametrize("d,n", [(128, 40), (64, 9), (256, 16)])
def test_finds_each_token(d, n):
    """A query that matches one token's key alone returns that token's value to half a step: every position of the
    context and every drafted token in turn (a sequence each), so a token dropped, doubled or misplaced shows."""
    dt, bs, ctx = torch.float16, 16, 150
    g = gen(d)
    sees = [[[True] * n] * n for _ in range(8)]
    b = Batch("fp16", 1, 1, d, bs, [n] * 8, [ctx + s for s in range(8)], seed=d, sees=sees)
    b.scale = 4.0                                          # a match scores 4 D, every other key at least 8 less
    for s in range(8):
        keys = torch.sign(torch.randn((b.lens[s], d), generator=g, device="cuda")).to(dt)
        t = torch.arange(b.lens[s], device="cuda")
        b.k[s] = keys[:, None]
        b.kc[b.bt[s, t // bs].long(), t % bs] = b.k[s]
        for first in range(0, b.lens[s], n):
            at = torch.arange(first, first + n, device="cuda") % b.lens[s]
            b.q[b.loc[s]:b.loc[s + 1], 0] = keys[at]
            out = b.run()
            b.check(out, [s])
            assert ((out[b.loc[s]:b.loc[s + 1], 0] - b.v[s][at, 0]).abs() <= 2.0 ** -6).all()


@pytest.mark.parametrize("ty", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,d,n", [(2, 1, 128, 8), (16, 1, 128, 8), (4, 1, 128, 12), (1, 1, 64, 30), (8, 2, 256, 9)])
def test_rising_scores_are_rescaled(ty, hq, hkv, d, n):
    """Keys that grow along the context (the running maximum rises by far more than 2^8 a tile), and fall."""
    for rising in (True, False):
        b = Batch(ty, hq, hkv, d, 16, [n, n], [1500, 700], seed=11)
        for s in range(2):
            t = torch.arange(b.lens[s], device="cuda")
            f = (t if rising else t.flip(0)).float()[:, None, None] / b.lens[s] * 30
            b.k[s] = (b.k[s].float() * f).to(b.dt)
            b.kc[b.bt[s, t // 16].long(), t % 16] = b.k[s]
        out = b.run()
        b.check(out)


def test_scales_below_and_at_zero():
    b = Batch("bf16", 4, 2, 128, 16, [9, 4], [130, 70], seed=12)
    for scale in (-0.09, 0.0, 1e-30, 0.7):
        b.scale = scale
        b.check(b.run())


def test_chain_equals_causal_chunk():
    """A tree without branches is a causal chunk: both calls within their bounds of the same formula."""
    n = 20
    sees = [[[k <= j for k in range(n)] for j in range(n)] for _ in range(3)]
    b = Batch("fp16", 8, 4, 128, 16, [n] * 3, [100, 0, 333], seed=13, sees=sees)
    out = b.run()
    b.check(out)
    ref = torch.empty_like(out)
    pa.pa_prefill_chunk(ref, b.q, b.kc, b.vc, b.bt, b.q_loc, b.sl, n, b.scale)
    b.check(ref)


def test_rows_of_no_sequence_and_bad_lengths():
    """Rows before the first and behind the last sequence stay; a sequence with bad lengths is skipped and flagged, the
    others are right."""
    b = Batch("bf16", 4, 2, 128, 16, [5, 6, 7, 4], [40, 50, 60, 70], seed=14)
    want = b.run()
    q, mask = b.q, b.mask
    b.q = torch.cat([torch.full_like(q[:3], float("nan")), q, torch.full_like(q[:2], float("nan"))])
    b.mask = torch.cat([mask[:3], mask, mask[:2]])
    b.q_loc += 3
    pa.pa_device_errors(clear=True)
    out = b.run(out=torch.full_like(b.q, 7.0))
    assert pa.pa_device_errors(clear=True) == 0
    assert torch.equal(out[3:-2], want) and (out[:3] == 7).all() and (out[-2:] == 7).all()
    cap = b.bt.shape[1] * 16
    for s, bad in ((1, 3), (2, cap + 1), (3, -1)):
        b.sl = torch.tensor(b.lens, device="cuda", dtype=torch.int32)
        b.sl[s] = bad
        out = b.run(out=torch.full_like(b.q, 7.0))
        assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_LENGTH
        for i in range(4):
            part, ref = out[3 + b.loc[i]:3 + b.loc[i + 1]], want[b.loc[i]:b.loc[i + 1]]
            assert (part == 7).all() if i == s else torch.equal(part, ref), (s, i)
    # a tree larger than max_q_len, rows outside the tensors
    b.sl = torch.tensor(b.lens, device="cuda", dtype=torch.int32)
    b.max_n = 6
    out = b.run(out=torch.full_like(b.q, 7.0))
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_LENGTH and (out[3 + b.loc[2]:3 + b.loc[3]] == 7).all()
    b.max_n = 7
    b.q_loc[4] = b.q.shape[0] + 1
    b.run(out=torch.full_like(b.q, 7.0))
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_LENGTH


def test_bad_pages_are_flagged():
    """A table entry outside the pool reads as zeros and sets its bit."""
    b = Batch("fp16", 4, 2, 128, 16, [5, 6], [140, 150], seed=15)
    b.run()
    b.bt[0, 2] = -5
    b.bt[1, 0] = b.kc.shape[0]
    pa.pa_device_errors(clear=True)
    out = b.run()
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BLOCK
    b.k[0][32:48], b.v[0][32:48], b.k[1][:16], b.v[1][:16] = 0, 0, 0, 0
    b.check(out)


def test_repeated_calls_are_bitwise_equal():
    b = Batch("bf16", 16, 8, 128, 16, [16] * 20, [(97 * i) % 900 for i in range(20)], seed=16)
    want = b.run()
    ws = b.ws()
    for _ in range(10):
        assert torch.equal(b.run(ws=ws), want)


def test_cache_past_32_bit_offsets():
    """Pages whose bytes and elements lie past 2^32 and 2^31."""
    hkv, d, bs = 8, 128, 16
    nb = 2 ** 31 // (hkv * d * bs) + 40
    b = Batch("bf16", 16, hkv, d, bs, [9, 8], [200, 300], seed=17, total=None)
    big = [torch.zeros((nb, bs, hkv, d), device="cuda", dtype=b.dt) for _ in range(2)]
    ids = b.bt[b.bt < b.kc.shape[0]]
    for c, small in zip(big, (b.kc, b.vc)):
        c[nb - 1 - ids.long()] = small[ids.long()]
    want = b.run()
    b.bt = torch.where(b.bt < b.kc.shape[0], nb - 1 - b.bt, b.bt)
    b.kc, b.vc = big
    assert torch.equal(b.run(), want)


def test_two_streams_with_a_workspace_each():
    bs = [Batch("bf16", 8, 4, 128, 16, [12] * 8, [500 + 40 * i for i in range(8)], seed=18),
          Batch("bf16", 8, 1, 128, 16, [33] * 3, [900, 10, 4000], seed=19)]
    want = [b.run() for b in bs]
    outs, wss = [torch.empty_like(w) for w in want], [b.ws() for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(8):
        for b, o, ws, st in zip(bs, outs, wss, streams):
            b.run(out=o, ws=ws, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_graphs_share_a_workspace_and_take_new_inputs():
    """Two captured calls replayed in turn over one workspace; lengths, masks and queries change between replays."""
    bs = [Batch("fp16", 8, 4, 128, 16, [12] * 4, [500, 30, 1000, 64], seed=20),
          Batch("fp16", 8, 4, 64, 16, [9, 2, 7], [2000, 10, 300], seed=21),
          Batch("bf16", 8, 1, 128, 16, [40, 12], [700, 90], seed=23)]
    ws = torch.full((max(b.ws().numel() for b in bs),), 0xFF, device="cuda", dtype=torch.uint8)
    graphs, outs = [], []
    for b in bs:
        b.run(ws=ws)
        outs.append(torch.zeros_like(b.q))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.run(out=outs[-1], ws=ws)
        graphs.append(graph)
    for step in range(3):
        for b, o, graph in zip(bs, outs, graphs):
            o.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for b, o in zip(bs, outs):
            assert torch.equal(o, b.run())
            b.check(o)
        for b in bs:      # a shorter context (the drafted rows are then others), other queries
            s = step % len(b.ns)
            b.sl[s] -= 5
            b.ctxs = [c - 5 if i == s else c for i, c in enumerate(b.ctxs)]
            b.k[s], b.v[s] = b.k[s][:-5], b.v[s][:-5]
            b.q.copy_(randn(gen(step), b.q.shape, b.dt))


def test_other_device_and_wrong_tensors_are_refused():
    b = Batch("bf16", 4, 2, 128, 16, [5], [40], seed=22)
    ok = dict(out=torch.empty_like(b.q), q=b.q, k_cache=b.kc, v_cache=b.vc, block_tables=b.bt, query_start_loc=b.q_loc,
              seq_lens=b.sl, tree_mask=b.mask, max_q_len=5, scale=0.1, workspace=b.ws())
    for name, bad, err in (("out", b.q[:4], ValueError), ("q", b.q.float(), TypeError), ("v_cache", b.vc[:, :8], ValueError),
                           ("v_cache", b.vc.cpu(), ValueError), ("k_cache", b.kc.transpose(1, 2), ValueError),
                           ("block_tables", b.bt.long(), TypeError), ("query_start_loc", b.q_loc[:1], ValueError),
                           ("tree_mask", b.mask.int(), TypeError), ("tree_mask", b.mask[:3], ValueError),
                           ("seq_lens", b.sl.cpu(), ValueError), ("workspace", None, pa.PagedAttnError),
                           ("max_q_len", 65, pa.PagedAttnError), ("scale", float("nan"), pa.PagedAttnError)):
        with pytest.raises(err):
            pa.pa_tree_decode(**{**ok, name: bad})
    pa.pa_tree_decode(**ok)
