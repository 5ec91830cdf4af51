"""Cases, plain forms and exact values of five operators around speculative decoding and shared pages.

tree_decode   pa_tree_decode: attention of a tree of drafted tokens for each sequence over the paged K/V
              cache -- every token sees the cached context and the drafted tokens that its mask names.
tree_commit   pa_tree_commit: the rows of the accepted path moved to the front of the drafted ones, in all
              layers, and the sequences' new lengths.
copy_pages    pa_copy_pages: pages copied to other pages in all layers (copy on write, relocation).
fork_pages    pa_fork_pages: empty sequences become forks of others by sharing their pages; every second
              pass frees them again (pa_resize_pages).
resize_pages  pa_resize_pages: sequences to new lengths, with pages from and back to the free list and
              a shared last page copied before it is written; every second pass takes the lengths back.

A case is a dict of plain values; `prepare` makes its inputs on the GPU, `run` makes one pass
(elementary torch operations, or the package's kernels where `own` is true) and `exact` is the
definition in 64 bits.
"""
import math
import random

import torch

own = False

LATENT_ROW = 576   # columns of a latent cache row (512 and the rotary part)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


# ------------------------------------------------------------------------------ the cases


def listed():
    return [
        # one request verifying eight drafted tokens at a short context: latency only
        dict(name="tree_single", op="tree_decode", dtype="bf16", seqs=1, hq=16, hkv=8, dim=128, block=16, nlo=8, nhi=8,
             clo=1000, chi=1000, pad=0),
        # a decode batch with trees of up to sixteen tokens over ragged contexts, some of them padded: memory bound
        dict(name="tree_batch", op="tree_decode", dtype="bf16", seqs=64, hq=16, hkv=8, dim=128, block=16, nlo=12, nhi=16,
             clo=100, chi=4096, pad=1),
        # few long contexts, an odd number of drafted tokens: the long axis has to be split
        dict(name="tree_long", op="tree_decode", dtype="fp16", seqs=4, hq=32, hkv=8, dim=128, block=32, nlo=25, nhi=25,
             clo=30000, chi=32768, pad=0),
        # large trees in a large batch: as much tensor work as memory traffic
        dict(name="tree_wide", op="tree_decode", dtype="bf16", seqs=64, hq=32, hkv=8, dim=128, block=16, nlo=64, nhi=64,
             clo=1024, chi=8192, pad=0),
        # the accepted tokens of a batch of 33 in one layer: latency only
        dict(name="commit_layer", op="tree_commit", dtype="fp16", seqs=33, layers=1, row=1024, latent=False, block=16, nlo=9,
             nhi=16, clo=100, chi=2048),
        # the accepted tokens of a batch of 64 in all layers at once
        dict(name="commit_model", op="tree_commit", dtype="bf16", seqs=64, layers=28, row=1024, latent=False, block=16, nlo=64,
             nhi=64, clo=100, chi=512),
        # copy on write of the last page of seven sequences, latent cache: latency only
        dict(name="copy_few", op="copy_pages", dtype="bf16", pairs=7, layers=1, row=LATENT_ROW, latent=True, block=64,
             pages=256),
        # a preempted batch's pages relocated in all layers: bandwidth scale
        dict(name="copy_many", op="copy_pages", dtype="bf16", pairs=777, layers=16, row=1024, latent=False, block=16,
             pages=2048),
        # parallel sampling: eight prompts, eight samples each
        dict(name="fork_samples", op="fork_pages", parents=8, children=7, block=16, clo=100, chi=4096),
        # many samples of long prompts
        dict(name="fork_long", op="fork_pages", parents=16, children=31, block=16, clo=8000, chi=32768),
        # a verification step of 64 sequences, half of them forks that share their last page
        dict(name="resize_step", op="resize_pages", dtype="bf16", seqs=64, layers=1, row=1024, latent=False, block=16, clo=100,
             chi=4096, more=16, forks=32, drop=0),
        # a batch in which every second sequence ends, the others take a chunk of 512 tokens more
        dict(name="resize_churn", op="resize_pages", dtype="fp16", seqs=509, layers=2, row=64, latent=False, block=16, clo=100,
             chi=16384, more=512, forks=64, drop=2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ones' ranges: sizes spread over their logarithm, at most the cost of the
    largest listed case of its operator."""
    op = rng.choice(["tree_decode", "tree_decode", "tree_commit", "copy_pages", "fork_pages", "resize_pages"])
    limit = {}
    for c in listed():
        if c["op"] == op:
            w = work(c)
            limit = {k: max(limit.get(k, 0), v) for k, v in w.items()}
    while True:
        case = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), block=rng.choice([8, 16, 32, 64, 128]))
        if op == "tree_decode":
            hkv, nhi, chi = rng.choice([1, 2, 3, 4, 8]), _log_int(rng, 1, 200), _log_int(rng, 1, 32768)
            case.update(seqs=_log_int(rng, 1, 128), hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]),
                        dim=rng.choice([64, 96, 128, 256]), nlo=rng.randint(1, nhi), nhi=nhi, clo=rng.randint(0, chi), chi=chi,
                        pad=rng.randint(0, 2))
        elif op == "fork_pages":
            del case["dtype"]
            chi = _log_int(rng, 1, 32768)
            case.update(parents=_log_int(rng, 1, 32), children=_log_int(rng, 1, 31), clo=rng.randint(1, chi), chi=chi)
        else:
            case.update(layers=_log_int(rng, 1, 32), latent=rng.random() < 0.25)
            case["row"] = LATENT_ROW if case["latent"] else rng.choice([64, 128, 192, 256, 512, 1024])
            chi = _log_int(rng, 1, 4096)
            if op == "tree_commit":
                nhi = _log_int(rng, 1, 200)
                case.update(seqs=_log_int(rng, 1, 128), nlo=rng.randint(1, nhi), nhi=nhi, clo=rng.randint(0, chi), chi=chi)
            elif op == "copy_pages":
                case["pairs"] = _log_int(rng, 1, 2000)
                case["pages"] = 2 * case["pairs"] + rng.randint(0, 100)
            else:
                case.update(seqs=_log_int(rng, 1, 300), clo=rng.randint(1, chi), chi=chi, more=_log_int(rng, 1, 600),
                            drop=rng.choice([0, 0, 2, 3]))
                case["forks"] = rng.randint(0, case["seqs"] // 2)
        w = work(case)
        if all(w[k] <= limit[k] for k in limit) and _cache_bytes(case) <= 2 << 30:
            return case


def _spread(lo, hi, n, salt):
    """n whole numbers evenly spread over [lo, hi] in a fixed shuffled order."""
    v = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]
    random.Random(1000 * n + salt).shuffle(v)
    return v


def _tree_lens(case):
    """(drafted tokens, kv lengths) of the sequences; a kv length is the cached context plus the drafted tokens."""
    n = _spread(case["nlo"], case["nhi"], case["seqs"], 2)
    c = _spread(case["clo"], case["chi"], case["seqs"], 3)
    return n, [a + b for a, b in zip(n, c)]


def _accepted(case):
    """Accepted tokens of each sequence: one to eight, at most a tree's."""
    return [min(n, 1 + (5 * i + n) % 8) for i, n in enumerate(_tree_lens(case)[0])]


def _pages(length, block):
    return -(-length // block)


def _resize_lens(case):
    """(lengths, new lengths, which sequence each is a fork of or -1): sequence 2 i + 1 is a fork of 2 i."""
    lens = _spread(case["clo"], case["chi"], case["seqs"], 4)
    forks = [i - 1 if i % 2 and i < 2 * case["forks"] else -1 for i in range(len(lens))]
    lens = [x if f < 0 else lens[f] for x, f in zip(lens, forks)]
    new = [x + case["more"] for x in lens]
    if case["drop"]:
        new = [0 if i % case["drop"] == 0 else x for i, x in enumerate(new)]
    return lens, new, forks


def _cache_bytes(case):
    """Bytes of the case's caches."""
    op, bs = case["op"], case["block"]
    if op == "fork_pages":
        return 0
    if op == "copy_pages":
        pages = case["pages"]
    elif op == "resize_pages":
        lens, new, _ = _resize_lens(case)
        pages = sum(_pages(max(a, b), bs) for a, b in zip(lens, new))
    else:
        pages = sum(_pages(x, bs) for x in _tree_lens(case)[1])
    if op == "tree_decode":
        return pages * bs * case["hkv"] * case["dim"] * 4
    return pages * bs * case["layers"] * _row_bytes(case)


def _row_bytes(case):
    """Bytes of a token's row in a layer, K and V together."""
    return case["row"] * 2 * (1 if case["latent"] else 2)


def work(case):
    """Bytes and operations one pass cannot do without: every input read once, every output written
    once; a product's multiply and add are two operations."""
    op, bs = case["op"], case["block"]
    if op == "tree_decode":
        n, kl = _tree_lens(case)
        hq, hkv, d = case["hq"], case["hkv"], case["dim"]
        b = sum(kl) * hkv * d * 4 + 2 * sum(n) * hq * d * 2 + sum(n) * 8 * -(-max(n) // 64)
        b += 4 * sum(_pages(x, bs) for x in kl)
        return {"bytes": b, "flops": 4 * d * hq * sum(x * (y - x) + x * (x + 1) // 2 for x, y in zip(n, kl))}
    if op == "tree_commit":
        acc = _accepted(case)
        return {"bytes": sum(acc) * (2 * case["layers"] * _row_bytes(case) + 4) + 16 * case["seqs"], "flops": 0}
    if op == "copy_pages":
        return {"bytes": case["pairs"] * (2 * case["layers"] * bs * _row_bytes(case) + 8), "flops": 0}
    if op == "fork_pages":   # a table entry read and written, a count read and written, for each page that a child gets
        pages = sum(_pages(x, bs) for x in _spread(case["clo"], case["chi"], case["parents"], 5))
        return {"bytes": pages * case["children"] * 4 + pages * 12 + 8 * case["parents"] * (1 + case["children"]), "flops": 0}
    lens, new, _ = _resize_lens(case)
    moved = sum(abs(_pages(a, bs) - _pages(b, bs)) for a, b in zip(lens, new))
    return {"bytes": 16 * moved + 12 * case["seqs"], "flops": 0}


# ------------------------------------------------------------------------------ the inputs


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _table(g, counts, spare):
    """Pages of sequences with so many each, out of a shuffled pool with some to spare: the block table (-1 past a
    sequence's end), the pool's size, and the ids not in use."""
    total, mb = sum(counts) + spare, max(1, max(counts))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor(counts, device="cuda")
    start = torch.cumsum(count, 0) - count
    col = torch.arange(mb, device="cuda")
    got = perm[(start[:, None] + col).clamp(max=total - 1)]
    return torch.where(col < count[:, None], got, torch.full_like(got, -1)).contiguous(), total, perm[sum(counts):].clone()


def _trees(case, seed):
    """A tree for each sequence: the drafted tokens' parents (-1: the last token of the context), each before its children."""
    rng = random.Random(seed)
    return [[rng.randint(max(-1, j - 1 - n // 2), j - 1) for j in range(n)] for n in _tree_lens(case)[0]]


def _int32(v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


def _caches(g, case, pages):
    """The caches of all layers, [layers, pages, block, heads, dim], or of latent rows [layers, pages, block, row]."""
    if case["latent"]:
        return _randn(g, (case["layers"], pages, case["block"], case["row"]), _dtype(case)), None
    shape = (case["layers"], pages, case["block"], max(1, case["row"] // 128), min(128, case["row"]))
    if shape[3] * shape[4] != case["row"]:
        shape = shape[:3] + (case["row"] // 64, 64)
    return _randn(g, shape, _dtype(case)), _randn(g, shape, _dtype(case))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, bs = case["op"], case["block"]
    s = {"case": case, "turn": 0}
    if op in ("tree_decode", "tree_commit"):
        n, kl = _tree_lens(case)
        loc = [0]
        for x in n:
            loc.append(loc[-1] + x)
        s["loc"], s["lens"] = _int32(loc), _int32(kl)
        s["bt"], pages, _ = _table(g, [_pages(x, bs) for x in kl], 3)
        trees = _trees(case, seed)
    if op == "tree_decode":
        dt, rows, words = _dtype(case), loc[-1], -(-max(n) // 64)
        shape = (pages, bs, case["hkv"], case["dim"])
        s["kc"], s["vc"] = _randn(g, shape, dt), _randn(g, shape, dt)
        s["q"] = _randn(g, (rows, case["hq"], case["dim"]), dt)
        s["out"] = torch.zeros_like(s["q"])
        bits, at = [], []
        for i, parents in enumerate(trees):
            own_bits = []
            for j, p in enumerate(parents):   # a padded token (the last ones of a tree) sees no drafted token
                m = 0 if j >= len(parents) - case["pad"] else (own_bits[p] if p >= 0 else 0) | 1 << j
                own_bits.append(m)
                bits.append([((m >> 64 * w & (1 << 64) - 1) ^ 1 << 63) - (1 << 63) for w in range(words)])
                at.append(i * max(n) + j)
        s["mask"] = torch.tensor(bits, device="cuda", dtype=torch.int64)
        s["at"] = torch.tensor(at, device="cuda")
        s["max_n"], s["scale"] = max(n), 1.0 / math.sqrt(case["dim"])
    elif op == "tree_commit":
        rng = random.Random(seed + 1)
        acc, path = _accepted(case), []
        for x, k in zip(n, acc):
            path.append(sorted(rng.sample(range(x), k)) + [-1] * (max(acc) - k))
        s["path"], s["acc"], s["host_path"] = _int32(path), _int32(acc), path
        s["kc"], s["vc"] = _caches(g, case, pages)
        s["new"] = torch.zeros_like(s["lens"])
    elif op == "copy_pages":
        s["kc"], s["vc"] = _caches(g, case, case["pages"])
        s["pairs"] = torch.randperm(case["pages"], generator=g, device="cuda").to(torch.int32)[:2 * case["pairs"]].view(-1, 2)
    elif op == "fork_pages":
        pn, cn = case["parents"], case["children"]
        lens = _spread(case["clo"], case["chi"], pn, 5)
        counts = [0] * (pn * (cn + 1))
        for i, x in enumerate(lens):
            counts[i * (cn + 1)] = _pages(x, bs)
        s["bt"], pages, _ = _table(g, counts, 5)
        s["lens"] = torch.zeros(len(counts), device="cuda", dtype=torch.int32)
        s["lens"][::cn + 1] = _int32(lens)
        s["parents"] = _int32([-1 if i % (cn + 1) == 0 else i - i % (cn + 1) for i in range(len(counts))])
        s["ended"] = torch.where(s["parents"] < 0, torch.full_like(s["parents"], -1), torch.zeros_like(s["parents"]))
        s["ref"] = torch.zeros(pages, device="cuda", dtype=torch.int32)
        s["ref"][s["bt"][s["bt"] >= 0].long()] = 1
        s["free"] = torch.arange(pages, device="cuda", dtype=torch.int32)   # (no page of a parent ever gets free)
        s["count"] = _int32([0])
        s["kc"] = s["vc"] = torch.zeros((1, pages, bs, 1, 8), device="cuda", dtype=torch.float16)
    else:
        lens, new, forks = _resize_lens(case)
        held = [_pages(x, bs) if f < 0 else 0 for x, f in zip(lens, forks)]
        spare = sum(_pages(max(a, b), bs) for a, b in zip(lens, new)) - sum(held) + case["seqs"]
        counts = held + [_pages(max(new), bs)]       # (the last row only makes the table wide enough for the new lengths)
        s["bt"], pages, free = _table(g, counts, max(0, spare - counts[-1]))
        free = torch.cat([s["bt"][-1][:counts[-1]], free])
        s["bt"] = s["bt"][:-1].contiguous()
        src = torch.tensor([i if f < 0 else f for i, f in enumerate(forks)], device="cuda")
        s["bt"] = s["bt"][src].contiguous()
        live = s["bt"] >= 0
        s["ref"] = torch.bincount(s["bt"][live].long(), minlength=pages).to(torch.int32)
        s["count"] = _int32([free.numel()])
        s["free"] = torch.cat([free, torch.full((pages - free.numel(),), -1, device="cuda", dtype=torch.int32)])
        s["lens"], s["old"], s["new"] = _int32(lens), _int32(lens), _int32(new)
        s["kc"], s["vc"] = _caches(g, case, pages)
    return s


# ------------------------------------------------------------------------------ the plain forms


def _plain_tree_decode(s):
    case = s["case"]
    hkv, d, bs, nm = case["hkv"], case["dim"], case["block"], s["max_n"]
    g = case["hq"] // hkv
    n = (s["loc"][1:] - s["loc"][:-1]).long()
    ctx = s["lens"].long() - n
    rows = (s["loc"][:-1, None].long() + torch.arange(nm, device="cuda")).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)        # [S, Hkv, n G, D]
    pages = s["bt"].clamp(min=0).long()
    k = s["kc"][pages].flatten(1, 2).float().transpose(1, 2)                                      # [S, Hkv, T, D]
    rel = torch.arange(k.shape[2], device="cuda") - ctx[:, None]                                  # [S, T]: < 0 in the context
    words = s["mask"][rows]                                                                       # [S, n, W]
    word = torch.gather(words, 2, (rel.clamp(min=0) // 64).clamp(max=words.shape[2] - 1)[:, None].expand(-1, nm, -1))
    bit = (word >> (rel.clamp(min=0) % 64)[:, None]) & 1
    sees = (rel < 0)[:, None] | ((rel >= 0) & (rel < n[:, None]))[:, None] & (bit == 1)           # [S, n, T]
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    x = torch.where(sees.repeat_interleave(g, 1)[:, None], x, torch.full_like(x, -math.inf))
    m = torch.amax(x, -1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    l = torch.sum(p, -1, keepdim=True)
    o = torch.matmul(p, s["vc"][pages].flatten(1, 2).float().transpose(1, 2)) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.unflatten(2, (nm, g)).permute(0, 2, 1, 3, 4).flatten(2, 3).flatten(0, 1)                # [S n, Hq, D]
    s["out"].copy_(o[s["at"]])
    return s["out"]


def _slots(bt, pos, bs):
    """Slots of positions pos [S, n] of the sequences."""
    return torch.gather(bt, 1, pos // bs).long() * bs + pos % bs


def _kv(s):
    return (s["kc"],) if s["vc"] is None else (s["kc"], s["vc"])


def _move_rows(cache, dst, src):
    flat = cache.flatten(1, 2)
    flat[:, dst] = flat[:, src]
    return cache


def _plain_tree_commit(s):
    bs = s["case"]["block"]
    ctx = s["lens"] - (s["loc"][1:] - s["loc"][:-1])
    i = torch.minimum(torch.arange(s["path"].shape[1], device="cuda"), s["acc"][:, None].long() - 1)   # (the last one again)
    src = _slots(s["bt"], ctx[:, None].long() + torch.gather(s["path"], 1, i), bs).flatten()
    dst = _slots(s["bt"], ctx[:, None].long() + i, bs).flatten()
    s["new"].copy_(ctx + s["acc"])
    return tuple(map(lambda c: _move_rows(c, dst, src), _kv(s))) + (s["new"],)


def _plain_copy_pages(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()

    def copy(c):
        c[:, dst] = c[:, src]
        return c

    return tuple(map(copy, _kv(s)))


def _plain_fork(s):
    bs = s["case"]["block"]
    par, lens = s["parents"].long(), s["lens"]
    p = par.clamp(min=0)
    ok = (par >= 0) & (lens == 0) & (par[p] < 0)
    col = torch.arange(s["bt"].shape[1], device="cuda")
    new = ok[:, None] & (col < ((lens[p] + bs - 1) // bs)[:, None])
    rows = s["bt"][p]
    s["bt"].copy_(torch.where(new, rows, s["bt"]))
    s["ref"].index_add_(0, torch.where(new, rows, torch.zeros_like(rows)).flatten().long(), new.flatten().to(torch.int32))
    lens.copy_(torch.where(ok, lens[p], lens))


def _plain_resize(s, new):
    bs = s["case"]["block"]
    bt, lens, ref, free, count = s["bt"], s["lens"], s["ref"], s["free"], s["count"]
    mb, nb = bt.shape[1], ref.shape[0]
    col = torch.arange(mb, device="cuda")
    valid = (new >= 0) & (new <= mb * bs)
    have, want = (lens + bs - 1) // bs, (new + bs - 1) // bs
    grows = valid & (new > lens)
    last = torch.gather(bt, 1, (have - 1).clamp(min=0)[:, None].long())[:, 0]        # the page that holds the last token
    cow = (grows & (lens % bs != 0) & (ref[last.clamp(min=0).long()] > 1)).to(torch.int32)
    demand = torch.where(grows, want - have + cow, torch.zeros_like(want))
    end = torch.cumsum(demand, 0)
    ok = valid & ((demand == 0) | (end <= count))
    taken = torch.amax(torch.where(ok & (demand > 0), end, torch.zeros_like(end)))
    first = have - cow
    gets = (ok & grows)[:, None] & (col >= first[:, None]) & (col < want[:, None])
    at = count - 1 - ((end - demand)[:, None] + col - first[:, None])
    page = torch.where(gets, free[at.clamp(0, nb - 1).long()], torch.full_like(bt, -1))
    drops = ok[:, None] & (col >= want[:, None]) & (col < have[:, None])
    copies = ok & (cow == 1)
    # the rows of a shared last page; a sequence that needs none repeats the first one's copy (where there is none at
    # all: a page onto itself)
    pick = torch.where(copies, torch.arange(len(copies), device="cuda"), torch.argmax(copies.to(torch.int32)))
    src = last[pick].clamp(min=0).long()
    dst = torch.gather(page[pick], 1, (have[pick] - 1).clamp(min=0)[:, None].long())[:, 0].long()
    dst = torch.where(copies[pick], dst, src)
    held = torch.arange(bs, device="cuda") < (lens[pick] % bs)[:, None]

    def copy(c):
        keep = held.view((1,) + held.shape + (1,) * (c.dim() - 3))
        c[:, dst] = torch.where(keep, c[:, src], c[:, dst])
        return c

    caches = tuple(map(copy, _kv(s)))
    less = torch.zeros(nb + 1, device="cuda", dtype=torch.int32)
    less.index_add_(0, torch.where(drops, bt, torch.full_like(bt, nb)).flatten().long(), torch.ones_like(bt).flatten())
    less.index_add_(0, torch.where(copies, last, torch.full_like(last, nb)).long(), torch.ones_like(last))
    less = less[:nb]
    ref.sub_(less)
    freed = (less > 0) & (ref == 0)
    more = torch.zeros(nb + 1, device="cuda", dtype=torch.int32)
    more.index_fill_(0, torch.where(gets, page, torch.full_like(page, nb)).flatten().long(), 1)
    ref.copy_(torch.where(more[:nb] > 0, more[:nb], ref))
    bt.copy_(torch.where(gets, page, torch.where(drops, torch.full_like(bt, -1), bt)))
    rank = torch.cumsum(freed, 0) - 1
    to = torch.where(freed, (count - taken) + rank, torch.full_like(rank, nb))
    longer = torch.cat([free, free[:1]])
    longer[to] = torch.arange(nb, device="cuda", dtype=torch.int32)
    free.copy_(longer[:nb])
    count.copy_(count - taken + torch.sum(freed))
    lens.copy_(torch.where(ok, new, lens))
    return caches


def _run_plain(s):
    op = s["case"]["op"]
    if op == "tree_decode":
        return _plain_tree_decode(s)
    if op == "tree_commit":
        return _plain_tree_commit(s)
    if op == "copy_pages":
        return _plain_copy_pages(s)
    s["turn"] ^= 1
    if op == "fork_pages":
        if s["turn"]:
            _plain_fork(s)
        else:
            _plain_resize(s, s["ended"])
        return s["bt"], s["lens"], s["ref"]
    return (s["bt"], s["lens"], s["ref"], s["free"], s["count"]) + _plain_resize(s, s["new"] if s["turn"] else s["old"])


def _run_own(s):
    import paged_kv_cache_232_gb300 as pa

    case, op = s["case"], s["case"]["op"]
    if "ws" not in s:    # a program allocates its workspace once
        size = 16
        if op == "tree_decode":
            size = pa.pa_tree_workspace_size(case["hq"], case["hkv"], case["dim"], s["max_n"])
        elif op in ("fork_pages", "resize_pages"):
            size = pa.pa_resize_workspace_size(s["bt"].shape[0], s["ref"].shape[0])
        s["ws"] = torch.empty(size, device="cuda", dtype=torch.uint8)
    if op == "tree_decode":
        pa.pa_tree_decode(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["loc"], s["lens"], s["mask"], s["max_n"], s["scale"],
                          s["ws"])
        return s["out"]
    if op == "tree_commit":
        pa.pa_tree_commit(s["kc"], s["vc"], s["bt"], s["loc"], s["lens"], s["path"], s["acc"], s["new"])
        return _kv(s) + (s["new"],)
    if op == "copy_pages":
        pa.pa_copy_pages(s["kc"], s["vc"], s["pairs"])
        return _kv(s)
    s["turn"] ^= 1
    if op == "fork_pages":
        if s["turn"]:
            pa.pa_fork_pages(s["bt"], s["lens"], s["parents"], s["ref"], case["block"])
        else:
            pa.pa_resize_pages(s["kc"], s["vc"], s["bt"], s["lens"], s["ended"], s["ref"], s["free"], s["count"], s["ws"])
        return s["bt"], s["lens"], s["ref"]
    pa.pa_resize_pages(s["kc"], s["vc"], s["bt"], s["lens"], s["new"] if s["turn"] else s["old"], s["ref"], s["free"],
                       s["count"], s["ws"])
    return (s["bt"], s["lens"], s["ref"], s["free"], s["count"]) + _kv(s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op, bs = case["op"], case["block"]
    if op == "fork_pages":
        return None
    if op == "tree_decode":   # a sequence and a KV head at a time, from the drafted tokens' ancestors
        d, hkv = case["dim"], case["hkv"]
        g = case["hq"] // hkv
        out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
        r0 = 0
        for i, (parents, kl) in enumerate(zip(_trees(case, seed), _tree_lens(case)[1])):
            n = len(parents)
            pages = s["bt"][i, :_pages(kl, bs)].long()
            k, v = (c.index_select(0, pages).reshape(-1, hkv, d)[:kl].double() for c in (s["kc"], s["vc"]))
            sees = [[False] * n for _ in parents]
            for j in range(n - case["pad"]):
                a = j
                while a >= 0:
                    sees[j][a] = True
                    a = parents[a]
            sees = torch.cat([torch.ones((n, kl - n), device="cuda", dtype=torch.bool), torch.tensor(sees, device="cuda")], 1)
            q = s["q"][r0:r0 + n].double().reshape(n, hkv, g, d)
            for h in range(hkv):
                x = torch.einsum("jgd,td->jgt", q[:, h], k[:, h]) * s["scale"]
                w = torch.softmax(x.masked_fill(~sees[:, None], -math.inf), -1)
                w = torch.where(sees.any(1)[:, None, None], w, torch.zeros_like(w))
                out[r0:r0 + n, h * g:(h + 1) * g] = torch.einsum("jgt,td->jgd", w, v[:, h])
            r0 += n
        return out
    caches = [c.double() for c in _kv(s)]
    if op == "tree_commit":
        table, n, kl = s["bt"].tolist(), *_tree_lens(case)
        frm, to = [], []
        for i, k in enumerate(_accepted(case)):
            c = kl[i] - n[i]
            for j in range(k):
                a, b = c + s["host_path"][i][j], c + j
                frm.append((table[i][a // bs], a % bs))
                to.append((table[i][b // bs], b % bs))
        a, b = torch.tensor(frm, device="cuda").T, torch.tensor(to, device="cuda").T
        for c in caches:
            c[:, b[0], b[1]] = c[:, a[0], a[1]].clone()
        return tuple(caches) + (None,)
    if op == "copy_pages":
        for a, b in s["pairs"].tolist():
            for c in caches:
                c[:, b] = c[:, a]
        return tuple(caches)
    # the pages that sequences sharing a partly filled last page get for their own, in the sequences' order
    lens, new, _ = _resize_lens(case)
    table, ref, free, n = s["bt"].tolist(), s["ref"].tolist(), s["free"].tolist(), s["count"].item()
    for i, (x, y) in enumerate(zip(lens, new)):
        if y > x:
            page = table[i][_pages(x, bs) - 1]
            if x % bs and ref[page] > 1:
                n -= 1
                for c in caches:
                    c[:, free[n], :x % bs] = c[:, page, :x % bs]
            n -= _pages(y, bs) - _pages(x, bs)
    return (None,) * 5 + tuple(caches)
