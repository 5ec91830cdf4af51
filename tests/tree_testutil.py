"""Inputs, 64-bit references and error bounds for the attention of drafted trees.  Everything here is torch in
float64 on the tensors' own device; nothing uses the package.

Bound (u: half a step of the 16-bit type relative to the value, 2^-8 bf16, 2^-11 fp16; `tiny`: half the smallest
step, 2^-25 for fp16, nothing for bf16's range):

scores: products of 16-bit values are exact in fp32, their sums (the tensor core adds 16 at a time, at most one step
2^-23 lost an addition: D / 16 + 16 additions) and the scale: ds = (D / 16 + 20) 2^-23 |scale| sum |q_i k_i|.  A weight
then is off by e = ds + 2^-20 (the exponent's argument, one rounding of a value up to 2^4 in size, and ex2, 2 ulp) + u
(rounded for the product), relative; in fp16 weights below 2^-20 of the largest are subnormal and off by at most 2^-31 of
the sum instead.  l sums the rounded weights.  So the output is off by at most e / (1 - e) sum w |v - o| + T 2^-31
max |v| (fp16) plus the fp32 sums, (T / 16 + 40) 2^-23 sum w |v| (T keys; 40 for rescales, the join of the copies and
that of the split), then rounded to the type.
"""
import math

import torch

from latent_testutil import TYPES, gen, half_step, randn, table, tiny  # noqa: F401


def paged_kv(g, lens, bs, hkv, d, dt, spare=3, fill=float("nan"), total=None):
    """Shuffled K/V caches for sequences of these lengths (rows past them hold `fill`), the block table (unused
    entries point past the pool) and each sequence's K and V rows."""
    nb = [-(-x // bs) for x in lens]
    total = total or sum(nb) + spare
    kc, vc = (torch.full((total, bs, hkv, d), fill, device=g.device, dtype=dt) for _ in range(2))
    perm = torch.randperm(total, generator=g, device=g.device)
    bt = torch.full((len(lens), max(1, max(nb)) + 1), 2 ** 30, device=g.device, dtype=torch.int32)
    at, ks, vs = 0, [], []
    for s, (n, x) in enumerate(zip(nb, lens)):
        blocks = perm[at:at + n]
        at += n
        bt[s, :n] = blocks.to(torch.int32)
        k, v = randn(g, (x, hkv, d), dt), randn(g, (x, hkv, d), dt)
        if x:
            t = torch.arange(x, device=g.device)
            kc[blocks[t // bs], t % bs] = k
            vc[blocks[t // bs], t % bs] = v
        ks.append(k)
        vs.append(v)
    return kc, vc, bt, ks, vs


def words_of(sees, words):
    """Mask rows (list of lists of truth values) as int64 words."""
    rows = []
    for r in sees:
        m = sum(1 << k for k, x in enumerate(r) if x)
        rows.append([((m >> 64 * w & (1 << 64) - 1) ^ 1 << 63) - (1 << 63) for w in range(words)])
    return rows


def tree_sees(rng, n):
    """A random tree's mask: each token sees itself and its ancestors."""
    sees = []
    for j in range(n):
        p = rng.randint(-1, j - 1)
        row = list(sees[p]) if p >= 0 else [False] * n
        row[j] = True
        sees.append(row)
    return sees


def attend64(q, k, v, sees, scale):
    """q [n, Hq, D] over k, v [T, Hkv, D] where sees [n, T]: (out, sum w |v - o|, sum w |v|, largest ds) in float64."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    gq = hq // hkv
    q, k, v = q.double().reshape(n, hkv, gq, d), k.double(), v.double()
    s = torch.einsum("jhgd,thd->jhgt", q, k) * scale
    s = s.masked_fill(~sees[:, None, None], -math.inf)
    w = torch.softmax(s, -1)
    w = torch.where(sees.any(-1)[:, None, None, None], w, torch.zeros_like(w))
    out = torch.einsum("jhgt,thd->jhgd", w, v)
    mag = torch.einsum("jhgt,thd->jhgd", w, v.abs())
    ds = (d / 16 + 20) * 2.0 ** -23 * abs(scale) * torch.einsum("jhgd,thd->jhgt", q.abs(), k.abs()).amax(-1, keepdim=True)
    spread = mag + out.abs()
    if s.numel() * d < 1 << 26:
        spread = torch.einsum("jhgt,jhgtd->jhgd", w, (v.permute(1, 0, 2)[None, :, None] - out[:, :, :, None]).abs())
    return out, spread, mag, ds


def check_tree(got, q, k, v, sees, scale, what):
    dt, T = got.dtype, k.shape[0]
    out, spread, mag, ds = attend64(q, k, v, sees, scale)
    e = ds + 2.0 ** -20 + half_step(dt)
    d = e / (1 - e) * spread + (T / 16 + 40) * 2.0 ** -23 * mag
    if dt == torch.float16:
        d = d + T * 2.0 ** -31 * v.double().abs().amax() * sees.any(-1)[:, None, None, None]
    err = (got.double().reshape(out.shape) - out).abs()
    bad = ~(err <= half_step(dt) * (out.abs() + d) + d + tiny(dt))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off; largest error "
                           f"{float(err.max()):.3e}, allowed there {float(d.flatten()[err.argmax()]):.3e}")
