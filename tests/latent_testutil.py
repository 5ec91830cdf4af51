"""Inputs, 64-bit references and error bounds for the norm + rotary writes and the latent-cache
attention.  Everything here is torch in float64 on the tensors' own device; nothing uses the package.

Bounds (u: half a step of the 16-bit type relative to the value, 2^-8 bf16, 2^-11 fp16; `tiny`: half
the smallest step, 2^-25 for fp16, nothing for bf16's range):

writes      a result is c a - s b with a, b normalised in fp32: the sum of D <= 512 squares (16 terms a
            lane, five shuffles: 21 roundings), the division by D and + eps (2), rsqrtf (2 ulp = 4
            roundings), two products, two roundings of the turn: under 32 half steps of fp32, 2^-19,
            of |c a| + |s b|; then one rounding to the type.
attention   scores: products of 16-bit values are exact in fp32, their sums (the tensor core adds 16
            at a time, at most one step 2^-23 lost an addition: (DL + 64) / 16 + 16 additions) and the
            scale: ds = (K / 16 + 20) 2^-23 scale sum |q_i k_i|.  A weight then is off by e = ds + 2^-20
            (the exponent's argument, up to 2^4 in size and rounded twice, and ex2, 2 ulp) + u (rounded for the
            product), relative; l sums the rounded weights.  So the output is off by at most
            e / (1 - e) sum w |v - o| plus the fp32 sums, (T / 16 + 32) 2^-23 sum w |v| (T keys; the 32
            for rescales and the join of the split), then rounded to the type.
"""
import math

import torch

ROPE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return 2.0 ** -25 if dt == torch.float16 else 0.0


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def randn(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device=g.device, dtype=torch.float32) * scale).to(dt)


def table(max_pos, dim, device="cuda", theta=1.0e6):
    f = theta ** (-2.0 * torch.arange(dim // 2, device=device, dtype=torch.float64) / dim)
    a = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32)


def norm64(x, w, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def turn64(y, cs, interleaved=False):
    """(value, |c a| + |s b|) of rows y [n, h, d] turned by cs [n, d]."""
    half = y.shape[-1] // 2
    c, s = cs[:, None, :half].double(), cs[:, None, half:].double()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :half], y[..., half:])
    v = (a * c - b * s, b * c + a * s)
    m = ((a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs())
    if interleaved:
        return torch.stack(v, -1).flatten(-2), torch.stack(m, -1).flatten(-2)
    return torch.cat(v, -1), torch.cat(m, -1)


def check_write(got, want, mag, what):
    dt = got.dtype
    d = 2.0 ** -19 * mag
    bad = (got.double() - want).abs() > half_step(dt) * (want.abs() + d) + d + tiny(dt)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off"


def paged(g, lens, bs, dl, dt, spare=3, fill=float("nan")):
    """A shuffled latent cache for sequences of these lengths (rows past them hold `fill`), and the
    table: unused entries point past the pool."""
    nb = [-(-x // bs) for x in lens]
    total = sum(nb) + spare
    cache = torch.full((total, bs, dl + ROPE), fill, device=g.device, dtype=dt)
    perm = torch.randperm(total, generator=g, device=g.device)
    mb = max(1, max(nb)) + 1
    table_ = torch.full((len(lens), mb), 2 ** 30, device=g.device, dtype=torch.int32)
    at = 0
    rows = []
    for s, (n, x) in enumerate(zip(nb, lens)):
        blocks = perm[at:at + n]
        at += n
        table_[s, :n] = blocks.to(torch.int32)
        r = randn(g, (x, dl + ROPE), dt)
        if x:
            t = torch.arange(x, device=g.device)
            cache[blocks[t // bs], t % bs] = r
        rows.append(r)
    return cache, table_, rows


def attend64(q, rows, scale, dl, n):
    """q [n, H, K] over the rows [T, K] of one sequence (the n query tokens are its last ones):
    (out, sum w |v - o|, sum w |v|, largest ds) in float64."""
    T, K = rows.shape
    q, r = q.double(), rows.double()
    s = torch.einsum("jhk,tk->jht", q, r) * scale
    sees = torch.arange(T, device=q.device) <= (T - n + torch.arange(n, device=q.device))[:, None]
    s = s.masked_fill(~sees[:, None], -math.inf)
    w = torch.softmax(s, -1)
    v = r[:, :dl]
    out = torch.einsum("jht,td->jhd", w, v)
    mag = torch.einsum("jht,td->jhd", w, v.abs())
    ds = (K / 16 + 20) * 2.0 ** -23 * scale * torch.einsum("jhk,tk->jht", q.abs(), r.abs()).amax(-1, keepdim=True)
    spread = mag + out.abs()
    if T * n * q.shape[1] * dl < 1 << 26:   # the tighter sum w |v - o| where it is small enough to form
        spread = torch.einsum("jht,jhtd->jhd", w, (v[None, None] - out[:, :, None]).abs())
    return out, spread, mag, ds


def check_attend(got, q, rows, scale, dl, n, what):
    dt = got.dtype
    if rows.shape[0] == 0:
        assert not got.any(), f"{what}: an empty context gives zeros"
        return
    out, spread, mag, ds = attend64(q, rows, scale, dl, n)
    e = ds + 2.0 ** -20 + half_step(dt)
    d = e / (1 - e) * spread + (rows.shape[0] / 16 + 32) * 2.0 ** -23 * mag
    err = (got.double() - out).abs()
    bad = ~(err <= half_step(dt) * (out.abs() + d) + d + tiny(dt))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off; largest error "
                           f"{float(err.max()):.3e}, allowed there {float(d.flatten()[err.argmax()]):.3e}")
