"""Cases, plain forms and exact values of four operators around the paged caches.

norm_rope      pa_norm_rope_reshape_and_cache: RMS norm of every query and key head, rotary embedding
               and the paged KV write in one pass over the rows of a qkv projection.
latent_write   pa_latent_rope_and_cache: the row a latent-attention layer caches for a token -- its
               normalised latent vector and the rotated key part all heads share -- written to its
               slot of a paged latent cache, and the queries' rotary parts rotated.
latent_decode  pa_latent_decode: one query token a sequence over the paged latent cache (absorbed
               form: every head's keys are the cached row, its values the row's latent part).
latent_chunk   pa_latent_prefill_chunk: ragged chunks of new tokens over the same cache,
               bottom-right causal.

A case is a dict of plain values; `prepare` makes its inputs on the GPU, `run` makes one pass
(elementary torch operations in 32 bits, or the package's kernels where `own` is true) and `exact`
is the definition in 64 bits.
"""
import math
import random

import torch

own = False

ROPE = 64          # columns of the rotary part of a latent cache row
THETA = 1.0e6      # base of the rotary embedding
EPS = 1.0e-6       # of the norms


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


# ------------------------------------------------------------------------------ the cases


def listed():
    return [
        # one request's decode step in one layer: a single token, latency only
        dict(name="norm_rope_single", op="norm_rope", dtype="bf16", tokens=1, hq=16, hkv=8, dim=128, block=16,
             max_pos=32768, pad=0, fused=True),
        # the new tokens of a decode batch of 257 with padded rows, separate q / k / v tensors
        dict(name="norm_rope_batch", op="norm_rope", dtype="fp16", tokens=257, hq=32, hkv=8, dim=96, block=32,
             max_pos=8192, pad=26, fused=False),
        # the prefill of a long batch: 64K rows cut out of the fused qkv projection, bandwidth scale
        dict(name="norm_rope_prefill", op="norm_rope", dtype="bf16", tokens=65536, hq=16, hkv=8, dim=128, block=16,
             max_pos=32768, pad=0, fused=True),
        # the new tokens of a decode batch of 64, all heads on one GPU
        dict(name="latent_write_step", op="latent_write", dtype="bf16", tokens=64, heads=128, latent=512, block=64,
             max_pos=32768, pad=6, norm=True, interleaved=True),
        # the prefill of a long batch with 16 heads, bandwidth scale
        dict(name="latent_write_prefill", op="latent_write", dtype="bf16", tokens=32771, heads=16, latent=512, block=16,
             max_pos=32768, pad=0, norm=True, interleaved=False),
        # one request at a short context: latency only
        dict(name="latent_decode_single", op="latent_decode", dtype="fp16", seqs=1, heads=16, latent=512, block=16,
             lo=1000, hi=1000, empty=0),
        # a decode batch of ragged short contexts, 16 heads
        dict(name="latent_decode_batch", op="latent_decode", dtype="bf16", seqs=64, heads=16, latent=512, block=16,
             lo=100, hi=2048, empty=0),
        # few long contexts: the long axis has to be split
        dict(name="latent_decode_long", op="latent_decode", dtype="fp16", seqs=4, heads=64, latent=512, block=64,
             lo=32000, hi=32768, empty=0),
        # a large batch with 128 heads: as much tensor work as memory traffic
        dict(name="latent_decode_wide", op="latent_decode", dtype="bf16", seqs=128, heads=128, latent=512, block=64,
             lo=1024, hi=8192, empty=2),
        # verification of a few drafted tokens a sequence: short chunks over long contexts
        dict(name="latent_chunk_verify", op="latent_chunk", dtype="bf16", chunks=32, heads=16, latent=512, block=16,
             qlo=3, qhi=5, clo=512, chi=4096),
        # chunked prefill of four requests, all heads: dense tensor work
        dict(name="latent_chunk_prefill", op="latent_chunk", dtype="bf16", chunks=4, heads=128, latent=512, block=64,
             qlo=512, qhi=512, clo=0, chi=4096),
        # ragged chunks from one token on, odd head count, the narrow latent, blocks of 8 tokens
        dict(name="latent_chunk_odd", op="latent_chunk", dtype="fp16", chunks=9, heads=24, latent=256, block=8,
             qlo=1, qhi=129, clo=0, chi=700),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ones' ranges: sizes spread over their logarithm, at most the cost of the
    largest listed case of its operator."""
    op = rng.choice(["norm_rope", "latent_write", "latent_decode", "latent_chunk"])
    dtype = rng.choice(["bf16", "fp16"])
    limit = {}
    for c in listed():
        if c["op"] == op:
            w = work(c)
            limit = {k: max(limit.get(k, 0), v) for k, v in w.items()}
    while True:
        if op == "norm_rope":
            hkv = rng.choice([1, 2, 3, 4, 8])
            case = dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 65536), hkv=hkv, hq=hkv * rng.choice([1, 2, 4, 7, 8]),
                        dim=rng.choice([64, 96, 128, 256]), block=rng.choice([8, 16, 32, 64, 128]),
                        max_pos=_log_int(rng, 64, 65536), fused=rng.random() < 0.5)
            case["pad"] = rng.randint(0, case["tokens"] // 4)
        elif op == "latent_write":
            case = dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 65536), heads=_log_int(rng, 1, 128),
                        latent=rng.choice([256, 512]), block=rng.choice([8, 16, 32, 64, 128]),
                        max_pos=_log_int(rng, 64, 65536), norm=rng.random() < 0.75, interleaved=rng.random() < 0.5)
            case["pad"] = rng.randint(0, case["tokens"] // 4)
        elif op == "latent_decode":
            hi = _log_int(rng, 1, 65536)
            seqs = _log_int(rng, 1, 256)
            case = dict(op=op, dtype=dtype, seqs=seqs, heads=_log_int(rng, 1, 128), latent=rng.choice([256, 512]),
                        block=rng.choice([8, 16, 32, 64, 128]), lo=rng.randint(1, hi), hi=hi,
                        empty=rng.randint(0, seqs // 8))
        else:
            qhi, chi = _log_int(rng, 1, 1024), _log_int(rng, 1, 16384)
            case = dict(op=op, dtype=dtype, chunks=_log_int(rng, 1, 64), heads=_log_int(rng, 1, 128),
                        latent=rng.choice([256, 512]), block=rng.choice([8, 16, 32, 64, 128]),
                        qlo=rng.randint(1, qhi), qhi=qhi, clo=rng.randint(0, chi), chi=chi)
        w = work(case)
        if all(w[k] <= limit[k] for k in limit):
            return case


def _spread(lo, hi, n, salt):
    """n whole numbers evenly spread over [lo, hi] in a fixed shuffled order."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]
    random.Random(1000 * n + salt).shuffle(v)
    return v


def _decode_lens(case):
    lens = _spread(case["lo"], case["hi"], case["seqs"], 1)
    for i in range(case["empty"]):       # batch slots not in use
        lens[(7 * i + 3) % len(lens)] = 0
    return lens


def _chunk_lens(case):
    """(query lengths, kv lengths) of the chunks; a kv length is the cached context plus the chunk."""
    ql = _spread(case["qlo"], case["qhi"], case["chunks"], 2)
    cl = _spread(case["clo"], case["chi"], case["chunks"], 3)
    return ql, [q + c for q, c in zip(ql, cl)]


def work(case):
    """Bytes and operations one pass cannot do without: every input read once, every output written
    once; a product's multiply and add are two operations."""
    op = case["op"]
    if op == "norm_rope":
        n, live, d = case["tokens"], case["tokens"] - case["pad"], case["dim"]
        b = 2 * n * case["hq"] * d * 2                           # q in and out
        b += live * case["hkv"] * d * 2 * 2 * 2                  # k and v in and out
        b += min(n, case["max_pos"]) * d * 4 + n * 16            # table rows, slots and positions
        return {"bytes": b, "flops": 8 * d * (n * case["hq"] + live * case["hkv"])}
    if op == "latent_write":
        n, live, row = case["tokens"], case["tokens"] - case["pad"], case["latent"] + ROPE
        b = 2 * live * row * 2 + 2 * n * case["heads"] * ROPE * 2
        b += min(n, case["max_pos"]) * ROPE * 4 + n * 16 + case["latent"] * 2
        return {"bytes": b, "flops": 6 * (live * row + n * case["heads"] * ROPE)}
    row, lat, h = case["latent"] + ROPE, case["latent"], case["heads"]
    if op == "latent_decode":
        lens = _decode_lens(case)
        keys, pairs, rows, tables = sum(lens), sum(lens), len(lens), sum(-(-x // case["block"]) for x in lens)
    else:
        ql, kl = _chunk_lens(case)
        keys, rows, tables = sum(kl), sum(ql), sum(-(-x // case["block"]) for x in kl)
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(ql, kl))
    b = keys * row * 2 + rows * h * (row + lat) * 2 + 4 * tables
    return {"bytes": b, "flops": 2 * pairs * h * (row + lat)}


# ------------------------------------------------------------------------------ the inputs


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _table(max_pos, dim):
    """cos / sin of every position and pair, [max_pos, dim] float32 (angles and functions in 64 bits)."""
    f = THETA ** (-2.0 * torch.arange(dim // 2, device="cuda", dtype=torch.float64) / dim)
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).to(torch.float32)


def _slots(g, case, n_slots):
    """Distinct slots, `pad` of them -1, and the rows that have one."""
    n = case["tokens"]
    slots = torch.randperm(n_slots, generator=g, device="cuda")[:n]
    if case["pad"]:
        slots[torch.randperm(n, generator=g, device="cuda")[:case["pad"]]] = -1
    return slots, torch.nonzero(slots >= 0)[:, 0]


def _paged(g, case, lens, dtype):
    """A latent cache in a shuffled pool that fits all sequences, and their block table (-1 past the end)."""
    bs, row = case["block"], case["latent"] + ROPE
    nb = [-(-x // bs) for x in lens]
    total = sum(nb) + 3
    cache = torch.empty((total, bs, row), device="cuda", dtype=dtype)
    step = max(1, (1 << 26) // (bs * row))
    for i in range(0, total, step):
        j = min(total, i + step)
        cache[i:j] = _randn(g, (j - i, bs, row), dtype)
    mb = max(1, max(nb))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor([sum(nb[:i]) for i in range(len(nb))], device="cuda")
    count = torch.tensor(nb, device="cuda")
    col = torch.arange(mb, device="cuda")
    idx = (start[:, None] + col[None, :]).clamp(max=total - 1)
    table = torch.where(col[None, :] < count[:, None], perm[idx], torch.full_like(perm[idx], -1))
    return cache, table.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, op = _dtype(case), case["op"]
    s = {"case": case}
    if op in ("norm_rope", "latent_write"):
        n, bs = case["tokens"], case["block"]
        blocks = -(-n // bs) + 2
        s["slots"], s["rows"] = _slots(g, case, blocks * bs)
        s["pos"] = torch.randint(0, case["max_pos"], (n,), generator=g, device="cuda")
    if op == "norm_rope":
        hq, hkv, d = case["hq"], case["hkv"], case["dim"]
        if case["fused"]:      # rows of one projection's output
            qkv = _randn(g, (n, (hq + 2 * hkv) * d), dt, 1.5)
            s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
            s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
            s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        else:
            s["q"], s["k"], s["v"] = (_randn(g, (n, h, d), dt, 1.5) for h in (hq, hkv, hkv))
        s["qw"], s["kw"] = (_randn(g, (d,), torch.float32, 0.2).add_(1.0).to(dt) for _ in range(2))
        s["kc"], s["vc"] = (_randn(g, (blocks, bs, hkv, d), dt) for _ in range(2))
        s["cs"] = _table(case["max_pos"], d)
        s["q_out"] = torch.zeros((n, hq, d), device="cuda", dtype=dt)
    elif op == "latent_write":
        h, lat = case["heads"], case["latent"]
        s["kv"] = _randn(g, (n, lat + ROPE), dt, 1.5)
        s["w"] = _randn(g, (lat,), torch.float32, 0.2).add_(1.0).to(dt) if case["norm"] else None
        # the rotary parts are the last columns of the per-head query projection (128 columns before them)
        s["q_pe"] = _randn(g, (n, h, 128 + ROPE), dt)[:, :, 128:]
        s["q"] = torch.zeros((n, h, lat + ROPE), device="cuda", dtype=dt)
        s["cache"] = _randn(g, (blocks, bs, lat + ROPE), dt)
        s["cs"] = _table(case["max_pos"], ROPE)
    else:
        if op == "latent_decode":
            lens = _decode_lens(case)
            rows = len(lens)
        else:
            ql, lens = _chunk_lens(case)
            rows = sum(ql)
            loc = [sum(ql[:i]) for i in range(len(ql) + 1)]
            s["ql"], s["loc"] = ql, loc
            s["q_loc"] = torch.tensor(loc, device="cuda", dtype=torch.int32)
        s["lens"] = lens
        s["cl"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        s["cache"], s["bt"] = _paged(g, case, lens, dt)
        h, lat = case["heads"], case["latent"]
        s["q"] = _randn(g, (rows, h, lat + ROPE), dt)
        s["out"] = torch.zeros((rows, h, lat), device="cuda", dtype=dt)
        s["scale"] = 1.0 / math.sqrt(128 + ROPE)     # heads of 128 columns and their rotary part
        if own:
            import paged_kv_cache_232_gb300 as pa
            s["ws"] = torch.empty(pa.pa_latent_workspace_size(h, lat, 1 if op == "latent_decode" else max(ql)),
                                  device="cuda", dtype=torch.uint8)
    return s


# ------------------------------------------------------------------------------ the plain forms


def _norm(x, w):
    y = x * torch.rsqrt(torch.sum(x * x, -1, keepdim=True) / x.shape[-1] + EPS)
    return y if w is None else y * w.to(x.dtype)


def _rotate(x, cs, interleaved=False):
    """Rows x [n, heads, d] turned by the table rows cs [n, d]."""
    half = x.shape[-1] // 2
    c, s = cs[:, None, :half].to(x.dtype), cs[:, None, half:].to(x.dtype)
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _attend(q, kv, mask, scale, lat):
    """Softmax attention of q [b, r, row] over kv [b, t, row] (values: its first lat columns), where mask
    [b, r or 1, t] is true; a row that sees nothing is zero.  In the type of q."""
    s = torch.matmul(q, kv.transpose(1, 2)) * scale
    s = torch.where(mask, s, torch.full_like(s, -math.inf))
    m = torch.amax(s, -1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    l = torch.sum(p, -1, keepdim=True)
    return torch.matmul(p, kv[..., :lat]) / torch.where(l > 0, l, torch.ones_like(l))


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = _dtype(case)
    if op == "norm_rope":
        cs = s["cs"][s["pos"]]
        s["q_out"].copy_(_rotate(_norm(s["q"].float(), s["qw"]), cs))
        k = _rotate(_norm(s["k"].float(), s["kw"]), cs).to(dt)
        at, live = s["rows"], s["slots"][s["rows"]]
        s["kc"].flatten(0, 1)[live] = k[at]
        s["vc"].flatten(0, 1)[live] = s["v"][at]
        return s["q_out"], s["kc"], s["vc"]
    if op == "latent_write":
        lat, inter = case["latent"], case["interleaved"]
        cs = s["cs"][s["pos"]]
        s["q"][..., lat:] = _rotate(s["q_pe"].float(), cs, inter).to(dt)
        kv = s["kv"].float()
        c = kv[:, :lat] if s["w"] is None else _norm(kv[:, :lat], s["w"])
        row = torch.cat([c, _rotate(kv[:, None, lat:], cs, inter)[:, 0]], -1).to(dt)
        at, live = s["rows"], s["slots"][s["rows"]]
        s["cache"].flatten(0, 1)[live] = row[at]
        return s["q"][..., lat:], s["cache"]
    lat, bs = case["latent"], case["block"]
    if op == "latent_decode":
        t = torch.arange(s["bt"].shape[1] * bs, device="cuda")
        kv = s["cache"][s["bt"].clamp(min=0).long()].flatten(1, 2).float()
        s["out"].copy_(_attend(s["q"].float(), kv, t[None, None, :] < s["cl"][:, None, None], s["scale"], lat))
        return s["out"]
    h = case["heads"]
    for c, (n, kl) in enumerate(zip(s["ql"], s["lens"])):
        r0 = s["loc"][c]
        kv = s["cache"][s["bt"][c, :-(-kl // bs)].long()].flatten(0, 1)[None, :kl].float()
        q = s["q"][r0:r0 + n].float().flatten(0, 1)[None]
        last = torch.arange(n, device="cuda").repeat_interleave(h) + (kl - n)
        mask = torch.arange(kl, device="cuda")[None, None, :] <= last[None, :, None]
        s["out"][r0:r0 + n] = _attend(q, kv, mask, s["scale"], lat)[0].unflatten(0, (n, h)).to(dt)
    return s["out"]


def _run_own(s):
    import paged_kv_cache_232_gb300 as pa

    case, op = s["case"], s["case"]["op"]
    if op == "norm_rope":
        pa.pa_norm_rope_reshape_and_cache(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["kc"], s["vc"], s["slots"],
                                          s["pos"], s["cs"], eps=EPS, q_out=s["q_out"])
        return s["q_out"], s["kc"], s["vc"]
    if op == "latent_write":
        pa.pa_latent_rope_and_cache(s["kv"], s["cache"], s["slots"], s["pos"], s["cs"], weight=s["w"], eps=EPS,
                                    q_pe=s["q_pe"], q=s["q"], interleaved=case["interleaved"])
        return s["q"][..., case["latent"]:], s["cache"]
    if op == "latent_decode":
        pa.pa_latent_decode(s["out"], s["q"], s["cache"], s["bt"], s["cl"], s["scale"], s["ws"])
    else:
        pa.pa_latent_prefill_chunk(s["out"], s["q"], s["cache"], s["bt"], s["q_loc"], s["cl"], max(s["ql"]),
                                   s["scale"], s["ws"])
    return s["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------ the definitions in 64 bits


def _turn(x, table, pos, pairs):
    """x [n, h, d] in 64 bits with column pairs (i, j) of `pairs` turned by the table's angles."""
    y = x.clone()
    half = len(pairs)
    for p, (i, j) in enumerate(pairs):
        c = table[pos, p].double()[:, None]
        s = table[pos, half + p].double()[:, None]
        y[..., i] = c * x[..., i] - s * x[..., j]
        y[..., j] = s * x[..., i] + c * x[..., j]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        d = case["dim"]
        pairs = [(i, i + d // 2) for i in range(d // 2)]

        def rows(x, w):
            x = x.double()
            rms = (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
            return _turn(x / rms * w.double(), s["cs"], s["pos"], pairs)

        kc, vc = s["kc"].double(), s["vc"].double()
        k, v = rows(s["k"], s["kw"]), s["v"].double()
        bs = case["block"]
        for a, b in ((kc, k), (vc, v)):
            a[s["slots"][s["rows"]] // bs, s["slots"][s["rows"]] % bs] = b[s["rows"]]
        return rows(s["q"], s["qw"]), kc, vc
    if op == "latent_write":
        lat = case["latent"]
        pairs = [(2 * i, 2 * i + 1) if case["interleaved"] else (i, i + ROPE // 2) for i in range(ROPE // 2)]
        kv = s["kv"].double()
        c = kv[:, :lat]
        if s["w"] is not None:
            c = c / (c.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["w"].double()
        kr = _turn(kv[:, None, lat:], s["cs"], s["pos"], pairs)[:, 0]
        cache, bs = s["cache"].double(), case["block"]
        at = s["slots"][s["rows"]]
        cache[at // bs, at % bs] = torch.cat([c, kr], 1)[s["rows"]]
        return _turn(s["q_pe"].double(), s["cs"], s["pos"], pairs), cache
    # attention, one sequence at a time: weights exp(s - max) over the keys a row sees
    lat, bs, h = case["latent"], case["block"], case["heads"]
    out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
    ql = [1] * len(s["lens"]) if op == "latent_decode" else s["ql"]
    r0 = 0
    for c, (n, kl) in enumerate(zip(ql, s["lens"])):
        if kl > 0:
            pages = s["bt"][c, :(kl + bs - 1) // bs].long()
            kv = s["cache"].index_select(0, pages).reshape(-1, lat + ROPE)[:kl].double()
            for j0 in range(0, n, 64):
                j1 = min(n, j0 + 64)
                sc = torch.einsum("jhd,td->jht", s["q"][r0 + j0:r0 + j1].double(), kv) * s["scale"]
                sees = torch.arange(kl, device="cuda") <= (kl - n + torch.arange(j0, j1, device="cuda"))[:, None]
                w = torch.softmax(sc.masked_fill(~sees[:, None, :], -math.inf), -1)
                out[r0 + j0:r0 + j1] = torch.einsum("jht,td->jhd", w, kv[:, :lat])
        r0 += n
    return out
