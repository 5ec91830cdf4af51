"""pa_copy_pages, pa_tree_commit, pa_fork_pages and pa_resize_pages against a model of the tables, counts and free list in
Python lists.  Data are moved, not computed: every comparison is exact."""
import random

import pytest
import torch

import paged_kv_cache_232_gb300 as pa
from tree_testutil import check_tree, gen, randn, table, tree_sees, words_of

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, device="cuda", dtype=torch.int32)


def caches(g, layers, pages, bs, hkv, d, latent=False, dt=torch.bfloat16):
    """Caches of random bits (NaN payloads among them), all layers in one tensor."""
    shape = (layers, pages, bs) + ((d,) if latent else (hkv, d))
    def one():
        return torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda", dtype=torch.int16).view(dt)
    return one(), None if latent else one()


def bits(c):
    return None if c is None else c.view(torch.int16).clone()


def same(a, b):
    return a is None and b is None or torch.equal(a.view(torch.int16), b.view(torch.int16))


SHAPES = [  # layers, block, heads, dim, latent
    (1, 16, 8, 128, False), (3, 8, 1, 64, False), (2, 32, 3, 96, False), (1, 64, 1, 576, True), (5, 128, 2, 256, False),
    (2, 16, 1, 8, False), (33, 16, 2, 64, False)]


@pytest.mark.parametrize("layers,bs,hkv,d,latent", SHAPES)
@pytest.mark.parametrize("pairs", [1, 7, 300])
def test_copy_pages(layers, bs, hkv, d, latent, pairs):
    g, nb = gen(pairs + d), 2 * pairs + 5
    kc, vc = caches(g, layers, nb, bs, hkv, d, latent)
    pick = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)[:2 * pairs].view(-1, 2).contiguous()
    pick[pairs // 2:, 0] = pick[pairs // 2, 0].clone()          # one page copied many times
    if pairs > 1:
        pick[0, 0], pick[1, 1] = -1, -1                  # skipped
    want = [bits(kc), bits(vc)]
    live = pick[(pick >= 0).all(1)].long()
    for w in want:
        if w is not None:
            w[:, live[:, 1]] = w[:, live[:, 0]]
    pa.pa_device_errors(clear=True)
    pa.pa_copy_pages(kc, vc, pick)
    assert pa.pa_device_errors(clear=True) == 0
    assert same(kc, want[0]) and same(vc, want[1])
    if layers == 1:                                      # a layer's cache without the layer dimension
        kc, vc = caches(g, 1, nb, bs, hkv, d, latent)
        want = [bits(kc[0]), None if latent else bits(vc[0])]
        for w in want:
            if w is not None:
                w[live[:, 1]] = w[live[:, 0]]
        pa.pa_copy_pages(kc[0], None if latent else vc[0], pick)
        assert same(kc[0], want[0]) and (latent or same(vc[0], want[1]))


def test_copy_pages_out_of_the_pool():
    g = gen(2)
    kc, vc = caches(g, 2, 9, 16, 2, 64)
    want = [bits(kc), bits(vc)]
    for w in want:
        w[:, 3] = w[:, 1]
    pa.pa_device_errors(clear=True)
    pa.pa_copy_pages(kc, vc, i32([[1, 3], [9, 4], [2, 9], [-2, 5], [6, 2 ** 31 - 1]]))
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BLOCK
    assert same(kc, want[0]) and same(vc, want[1])
    pa.pa_copy_pages(kc, vc, i32([]).view(0, 2))
    assert same(kc, want[0])


def test_pages_past_32_bit_offsets():
    """A cache of more than 2^32 bytes in one layer and of more than 2^31 elements over the layers."""
    bs, hkv, d = 16, 8, 128
    nb = 2 ** 32 // (bs * hkv * d * 2) + 7
    kc = torch.zeros((1, nb, bs, hkv, d), device="cuda", dtype=torch.bfloat16)
    row = randn(gen(3), (bs, hkv, d), torch.bfloat16)
    kc[0, 5] = row
    pa.pa_copy_pages(kc, kc[:0].new_zeros(kc.shape), i32([[5, nb - 1]]))
    assert torch.equal(kc[0, nb - 1], row)
    bt, new = i32([[nb - 1, nb - 2]]), i32([0])
    pa.pa_tree_commit(kc[0], torch.zeros_like(kc[0]), bt, i32([0, 16]), i32([20]), i32([[11]]), i32([1]), new)
    assert torch.equal(kc[0, nb - 1, 4], row[15]) and new.item() == 5


@pytest.mark.parametrize("layers,bs,hkv,d,latent", SHAPES)
def test_commit(layers, bs, hkv, d, latent):
    rng, g = random.Random(bs + d), gen(d)
    ns = [1, 5, 16, 0, 40, 300, 7, 64]
    ctxs = [0, 30, 8, 12, 127, 5, 1, 64]
    lens = [a + b for a, b in zip(ns, ctxs)]
    pages = [-(-x // bs) for x in lens]
    nb = sum(pages) + 3
    perm = list(range(nb))
    rng.shuffle(perm)
    bt, at = [], 0
    for n in pages:
        bt.append(perm[at:at + n] + [2 ** 30] * (max(pages) - n))
        at += n
    # the whole tree, none, one, a chain that starts late, every second token
    paths = [[0], [], list(range(16)), [], list(range(3, 40)), list(range(0, 300, 2))[:140], [6], sorted(rng.sample(range(64), 9))]
    most = max(map(len, paths))
    kc, vc = caches(g, layers, nb, bs, hkv, d, latent)
    want = [bits(kc), bits(vc)]
    for w in want:
        if w is None:
            continue
        for s, p in enumerate(paths):
            src = [(bt[s][(ctxs[s] + t) // bs], (ctxs[s] + t) % bs) for t in p]
            dst = [(bt[s][(ctxs[s] + i) // bs], (ctxs[s] + i) % bs) for i in range(len(p))]
            if p:
                a, b = torch.tensor(src, device="cuda").T, torch.tensor(dst, device="cuda").T
                w[:, b[0], b[1]] = w[:, a[0], a[1]].clone()
    loc = [0]
    for n in ns:
        loc.append(loc[-1] + n)
    new = i32([-7] * len(ns))
    pa.pa_device_errors(clear=True)
    pa.pa_tree_commit(kc, vc, i32(bt), i32(loc), i32(lens), i32([p + [-9] * (most - len(p)) for p in paths]),
                      i32([len(p) for p in paths]), new)
    assert pa.pa_device_errors(clear=True) == 0
    assert same(kc, want[0]) and same(vc, want[1])
    assert new.tolist() == [c + len(p) for c, p in zip(ctxs, paths)]


def test_commit_refuses_paths_and_lengths():
    """A path that does not rise in its tree, too many entries, bad lengths: no row of that sequence moves, the others'
    do; a page outside the pool keeps its row."""
    g = gen(4)
    kc, vc = caches(g, 2, 20, 16, 2, 64)
    bt = torch.arange(20, device="cuda", dtype=torch.int32).view(5, 4)
    loc, lens = i32([0, 5, 10, 15, 20, 25]), [20, 30, 40, 50, 60]
    good = [[2, 4, 0]] * 5

    def run(paths, acc, lens_, want_bits, moved, new_want, table=bt):
        before = [bits(kc), bits(vc)]
        new = i32([-7] * 5)
        pa.pa_device_errors(clear=True)
        pa.pa_tree_commit(kc, vc, table, loc, i32(lens_), i32(paths), i32(acc), new)
        assert pa.pa_device_errors(clear=True) == want_bits
        assert new.tolist() == new_want
        for c, b in ((kc, before[0]), (vc, before[1])):
            for s in range(5):
                if s not in moved:
                    assert torch.equal(c.view(torch.int16)[:, 4 * s:4 * s + 4], b[:, 4 * s:4 * s + 4]), s
                else:
                    for i, t in enumerate((2, 4)):
                        f, to = lens[s] - 5 + t, lens[s] - 5 + i
                        assert torch.equal(c.view(torch.int16)[:, 4 * s + to // 16, to % 16], b[:, 4 * s + f // 16, f % 16])

    new = [x - 3 for x in lens]
    run(good, [2] * 5, lens, 0, range(5), new)
    for bad in ([4, 2, 0], [2, 2, 0], [-1, 2, 0], [2, 5, 0]):
        run([good[0], bad] + good[2:], [2] * 5, lens, pa.PA_DEVERR_PATH, (0, 2, 3, 4), [new[0], 25] + new[2:])
    for acc in (4, -1, 6):
        run(good, [2, 2, acc, 2, 2], lens, pa.PA_DEVERR_PATH, (0, 1, 3, 4), new[:2] + [35] + new[3:])
    for bad in (4, -3, 65):
        run(good, [2] * 5, lens[:3] + [bad] + lens[4:], pa.PA_DEVERR_LENGTH, (0, 1, 2, 4), new[:3] + [bad] + new[4:])
    table = bt.clone()
    table[4, 3] = 20
    run(good, [2] * 5, lens, pa.PA_DEVERR_BLOCK, (0, 1, 2, 3), new, table)


# ------------------------------------------------------------------------------ forks and lengths


class Ledger:
    """The tables, counts and free list as Python lists, and what the calls do to them."""

    def __init__(self, rng, seqs, mb, bs, nb):
        self.bs, self.mb, self.nb = bs, mb, nb
        self.bt, self.lens, self.ref = [[-1] * mb for _ in range(seqs)], [0] * seqs, [0] * nb
        self.free = list(range(nb))
        rng.shuffle(self.free)
        self.count = nb
        self.cells = {}                       # (page, row) -> what is stored there

    def pages(self, n):
        return -(-n // self.bs)

    def fork(self, parents):
        for s, p in enumerate(parents):
            if p >= 0:
                n = self.pages(self.lens[p])
                self.bt[s][:n] = self.bt[p][:n]
                for i in self.bt[p][:n]:
                    self.ref[i] += 1
                self.lens[s] = self.lens[p]

    def resize(self, new):
        """Returns the (from, to, rows) copies and whether some sequence got too few pages."""
        count, ref0, drops, copies, short = self.count, list(self.ref), [], [], False
        demands = []
        for s, n in enumerate(new):
            have, cow = self.lens[s], False
            if n > have and have % self.bs:
                cow = ref0[self.bt[s][self.pages(have) - 1]] > 1
            demands.append((max(0, self.pages(n) - self.pages(have)) + cow if n > have else 0, cow))
        end = 0
        for s, (n, (demand, cow)) in enumerate(zip(new, demands)):
            if n < 0 or n == self.lens[s]:
                continue
            end += demand
            if demand and end > count:
                short = True
                continue
            old, have, want = self.lens[s], self.pages(self.lens[s]), self.pages(n)
            got = [self.free[count - 1 - (end - demand + i)] for i in range(demand)]
            for i in got:
                self.ref[i] = 1
            if cow:
                copies.append((self.bt[s][have - 1], got[0], old % self.bs))
                drops.append(self.bt[s][have - 1])
                self.bt[s][have - 1] = got.pop(0)
            self.bt[s][have:have + len(got)] = got
            if n < old:
                drops += self.bt[s][want:have]
                self.bt[s][want:have] = [-1] * (have - want)
            self.lens[s] = n
            if demand:                        # (a refused sequence takes none, nor do those behind it)
                self.count = count - end
        freed = []
        for i in drops:
            self.ref[i] -= 1
            if self.ref[i] == 0:
                freed.append(i)
        self.free[self.count:self.count + len(freed)] = sorted(freed)
        self.count += len(freed)
        return copies, short


class Device:
    """The same on the GPU, with caches whose rows tell them apart."""

    def __init__(self, m, layers=1, hkv=1, d=8, latent=False, seed=1):
        self.m, g = m, gen(seed)
        self.bt, self.lens, self.ref = i32(m.bt), i32(m.lens), i32(m.ref)
        self.free, self.count = i32(m.free), i32([m.count])
        self.kc, self.vc = caches(g, layers, m.nb, m.bs, hkv, d, latent)
        self.ws = torch.full((pa.pa_resize_workspace_size(len(m.bt), m.nb),), 0xFF, device="cuda", dtype=torch.uint8)

    def fork(self, parents):
        pa.pa_fork_pages(self.bt, self.lens, i32(parents), self.ref, self.m.bs)

    def resize(self, new, stream=None):
        pa.pa_resize_pages(self.kc, self.vc, self.bt, self.lens, i32(new), self.ref, self.free, self.count, self.ws)

    def check(self, what):
        m = self.m
        assert self.lens.tolist() == m.lens, what
        assert self.ref.tolist() == m.ref, what
        assert self.count.tolist() == [m.count], what
        assert self.free.tolist() == m.free, what
        assert self.bt.tolist() == m.bt, what


def step(m, dev, new, what, errors=0):
    want = [bits(dev.kc), bits(dev.vc)]
    copies, short = m.resize(new)
    for w in want:
        if w is not None:
            src = w.clone()
            for a, b, rows in copies:
                w[:, b, :rows] = src[:, a, :rows]
    pa.pa_device_errors(clear=True)
    dev.resize(new)
    assert pa.pa_device_errors(clear=True) == errors | (pa.PA_DEVERR_PAGES if short else 0), what
    dev.check(what)
    assert same(dev.kc, want[0]) and same(dev.vc, want[1]), what
    return copies


@pytest.mark.parametrize("seqs,mb,bs,nb,layers,hkv,d,latent", [
    (1, 3, 16, 5, 1, 1, 8, False), (5, 9, 8, 40, 2, 3, 64, False), (40, 20, 16, 500, 1, 1, 576, True),
    (300, 6, 32, 1400, 1, 1, 8, False), (1100, 4, 16, 3000, 1, 1, 8, False), (7, 300, 128, 1500, 1, 1, 8, False)])
def test_forks_and_lengths_follow_the_model(seqs, mb, bs, nb, layers, hkv, d, latent):
    """A random history: growth, shrinking, freeing, forks, with the list running out at times."""
    rng = random.Random(seqs)
    m = Ledger(rng, seqs, mb, bs, nb)
    dev = Device(m, layers, hkv, d, latent)
    cow = 0
    for turn in range(12):
        new = []
        for n in m.lens:
            kind = rng.random()
            most = mb * bs if turn % 4 == 3 else min(mb * bs, n + 3 * bs)
            new.append(-1 if kind < 0.2 else 0 if kind < 0.3 else n if kind < 0.35 else rng.randint(0, n) if kind < 0.5 else
                       rng.randint(n, max(n, most)))
        cow += len(step(m, dev, new, f"turn {turn}"))
        live = [s for s, n in enumerate(m.lens) if n]
        parents = [rng.choice(live) if n == 0 and live and rng.random() < 0.7 else -1 for n in m.lens]
        m.fork(parents)
        dev.fork(parents)
        assert pa.pa_device_errors(clear=True) == 0
        dev.check(f"forks of turn {turn}")
        used = [i for r, n in zip(m.bt, m.lens) for i in r[:m.pages(n)]]
        assert all(m.ref[i] == used.count(i) for i in set(used)) and m.count + len(set(used)) == nb
    assert cow > 0 or seqs == 1
    step(m, dev, [0] * seqs, "all freed")
    assert m.count == nb


@pytest.mark.parametrize("seqs,mb,bs,nb", [(12, 2500, 8, 16384), (12, 2500, 8, 16385), (30, 2500, 8, 50021), (700, 150, 16, 70000)])
def test_large_pools(seqs, mb, bs, nb):
    """Pools whose freed pages are put back by many blocks, and the largest that one block takes."""
    rng = random.Random(nb)
    m = Ledger(rng, seqs, mb, bs, nb)
    dev = Device(m)
    for turn in range(6):
        most = mb * bs
        step(m, dev, [-1 if rng.random() < 0.2 else rng.choice([0, rng.randint(0, most), rng.randint(0, most)]) for _ in range(seqs)],
             f"turn {turn}")
    step(m, dev, [0] * seqs, "all freed")
    assert m.count == nb


def test_sharers_that_grow_together_get_their_own_page():
    """All forks of a sequence grow in one call: everybody's last page is its own, the shared one is free again."""
    m = Ledger(random.Random(5), 6, 8, 16, 60)
    dev = Device(m, layers=3, hkv=2, d=64)
    step(m, dev, [37, 0, 0, 0, 32, 0], "prompt")
    forks = [-1, 0, 0, 0, -1, 4]
    m.fork(forks)
    dev.fork(forks)
    dev.check("forks")
    assert len(step(m, dev, [40, 38, 55, 37, 33, 48], "grow")) == 3       # the fourth keeps its length
    # its page is its own now (count 1): the next token needs no copy, and full pages are never copied
    assert len(step(m, dev, [41, 39, 56, 38, 34, 49], "grow again")) == 0
    # shrunk into a full page that is still shared: a copy before it grows
    assert len(step(m, dev, [20, -1, -1, -1, 10, 10], "shrink")) == 0
    assert len(step(m, dev, [21, -1, -1, -1, 11, 12], "grow into a shared page")) == 3


def test_list_that_runs_out_serves_the_first():
    m = Ledger(random.Random(6), 5, 8, 16, 6)
    dev = Device(m)
    step(m, dev, [16, 40, 64, 16, 0], "the third and fourth keep their length")
    assert m.lens == [16, 40, 0, 0, 0] and m.count == 2
    step(m, dev, [0, -1, 32, 0, 0], "pages that get free in a call serve the next one")
    assert m.count == 1


def test_fork_refusals():
    m = Ledger(random.Random(7), 6, 4, 16, 30)
    dev = Device(m)
    step(m, dev, [20, 40, 0, 0, 0, 0], "prompts")
    for parents in ([-1, 0, -1, -1, -1, -1],       # the child has tokens
                    [-1, -1, 6, -1, -1, -1], [-1, -1, -2, -1, -1, -1],   # no such parent
                    [-1, -1, 2, -1, -1, -1]):      # itself
        dev.fork(parents)
        assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_FORK
        dev.check(parents)
    # a parent that is forked in the same call: refused for its child only
    dev.fork([-1, -1, 0, 2, 1, -1])
    m.fork([-1, -1, 0, -1, 1, -1])
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_FORK
    dev.check("chain")
    # a fork of an empty sequence is empty
    dev.fork([-1, -1, -1, 5, -1, -1])
    assert pa.pa_device_errors(clear=True) == 0
    dev.check("empty")
    dev.lens[0] = 65
    dev.fork([-1, -1, -1, 0, -1, -1])
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_LENGTH
    dev.lens[0] = 20
    dev.check("length")


def test_resize_refusals():
    m = Ledger(random.Random(8), 4, 4, 16, 20)
    dev = Device(m)
    step(m, dev, [20, 40, 17, 0], "prompts")
    for new in ([-1, 65, -1, -1], [-1, -2, -1, -1]):
        dev.resize(new)
        assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_LENGTH
        dev.check(new)
    # a list whose length cannot be: nothing is done
    dev.count.fill_(21)
    dev.resize([64, 0, 64, 64])
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_COUNT and dev.count.item() == 21
    dev.count.fill_(m.count)
    dev.check("count")
    # a page that nobody holds any more is not dropped twice
    page = m.bt[1][2]
    dev.ref[page] = 0
    dev.resize([-1, 10, -1, -1])
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_COUNT
    assert dev.ref[page].item() == 0 and dev.count.item() == m.count + 1
    # a list that holds a page in use, and no page at all
    dev.free[dev.count.item() - 1], dev.free[dev.count.item() - 2] = m.bt[0][0], 99
    dev.resize([-1, -1, -1, 32])
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_COUNT
    assert dev.bt[3].tolist()[:2] == [m.bt[0][0], -1]
    # tables that name pages outside the pool
    dev.bt[0, 1] = 20
    dev.resize([0, -1, -1, -1])
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BLOCK and dev.lens[0].item() == 0


def test_graph_replays_a_loop_of_lengths():
    """Growth, fork and freeing captured once and replayed with other lengths."""
    rng = random.Random(9)
    m = Ledger(rng, 9, 8, 16, 200)
    dev = Device(m, layers=2)
    new, parents = i32([0] * 9), i32([-1] * 9)
    dev.resize([0] * 9)
    dev.fork([-1] * 9)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_resize_pages(dev.kc, dev.vc, dev.bt, dev.lens, new, dev.ref, dev.free, dev.count, dev.ws)
        pa.pa_fork_pages(dev.bt, dev.lens, parents, dev.ref, 16)
    for _ in range(6):
        lens = [rng.choice([-1, 0, rng.randint(0, 128)]) for _ in range(9)]
        m.resize(lens)
        live, empty = [s for s in range(9) if m.lens[s]], [s for s in range(9) if not m.lens[s]]
        forks = [live[0] if s in empty[:2] and live else -1 for s in range(9)]
        m.fork(forks)
        new.copy_(i32(lens))
        parents.copy_(i32(forks))
        graph.replay()
        dev.check(lens)


def test_two_streams_with_a_ledger_each():
    devs = []
    for seed in (1, 2):
        m = Ledger(random.Random(seed), 50, 20, 16, 900)
        devs.append((m, Device(m, seed=seed), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for turn in range(8):
        for m, dev, st in devs:
            new = [min(320, n + 17) if (s + turn) % 5 else 0 for s, n in enumerate(m.lens)]
            m.resize(new)
            with torch.cuda.stream(st):
                dev.resize(new)
    torch.cuda.synchronize()
    for m, dev, _ in devs:
        dev.check("after 8 turns")


def test_speculative_loop():
    """The calls of a verification step in a row, without a look at the device: room for the drafted tokens, their
    rows written (norm and rotation), attention over the tree, the accepted path moved to the front, the rest given
    back; every second sequence starts as a fork.  The tokens that stay are the accepted ones' rows, and the last
    step's attention is that of the formula over them."""
    dt, bs, hq, hkv, d, S, nb, mb = torch.float16, 16, 4, 2, 64, 6, 200, 12
    g, rng = gen(31), random.Random(31)
    cs, one = table(400, d), torch.ones(d, device="cuda", dtype=dt)
    kc, vc = (torch.full((nb, bs, hkv, d), float("nan"), device="cuda", dtype=dt) for _ in range(2))
    bt, lens = torch.full((S, mb), -1, device="cuda", dtype=torch.int32), i32([0] * S)
    ref, free, count = i32([0] * nb), torch.randperm(nb, generator=g, device="cuda").to(torch.int32), i32([nb])
    ws = torch.empty(pa.pa_resize_workspace_size(S, nb), device="cuda", dtype=torch.uint8)
    new_lens = i32([0] * S)

    def resize(target):
        pa.pa_resize_pages(kc, vc, bt, lens, target, ref, free, count, ws)

    def write(seq, pos, slot_pos):
        """Rows of tokens of sequences seq at positions pos into the slots of slot_pos; their K/V as written."""
        n = len(seq)
        q, k, v = randn(g, (n, hq, d), dt), randn(g, (n, hkv, d), dt), randn(g, (n, hkv, d), dt)
        slots = bt[seq, slot_pos // bs].long() * bs + slot_pos % bs
        out = torch.empty_like(q)
        pa.pa_norm_rope_reshape_and_cache(q, k, v, one, one, kc, vc, slots, pos, cs, q_out=out)
        return out, kc.flatten(0, 1)[slots].clone(), vc.flatten(0, 1)[slots].clone()

    pa.pa_device_errors(clear=True)
    prompt = [21, 0, 40, 0, 16, 0]
    resize(i32(prompt))
    seq = torch.tensor([s for s, n in enumerate(prompt) for _ in range(n)], device="cuda")
    pos = torch.tensor([t for n in prompt for t in range(n)], device="cuda")
    _, k, v = write(seq, pos, pos)
    rows = [[(k[i], v[i]) for i in torch.nonzero(seq == s)[:, 0].tolist()] for s in range(S)]
    pa.pa_fork_pages(bt, lens, i32([-1, 0, -1, 2, -1, 4]), ref, bs)
    for s in (1, 3, 5):
        rows[s] = list(rows[s - 1])
    for turn in range(5):
        ns = [rng.randint(1, 11) for _ in range(S)]
        ctx = [len(r) for r in rows]
        sees, parents = [], []
        for n in ns:
            up = [rng.randint(-1, j - 1) for j in range(n)]
            m, depth = pa.tree_mask(up)
            parents.append((up, depth))
            sees.append([[bool(int(m[j, 0]) >> k & 1) for k in range(n)] for j in range(n)])
        mask = torch.tensor([w for s in sees for w in words_of(s, 1)], device="cuda")
        loc = [sum(ns[:s]) for s in range(S + 1)]
        resize(i32([c + n for c, n in zip(ctx, ns)]))
        seq = torch.tensor([s for s, n in enumerate(ns) for _ in range(n)], device="cuda")
        at = torch.tensor([c + j for c, n in zip(ctx, ns) for j in range(n)], device="cuda")
        pos = torch.tensor([c + int(x) for c, (_, dep) in zip(ctx, parents) for x in dep], device="cuda")
        q, k, v = write(seq, pos, at)
        out = torch.empty_like(q)
        tws = torch.empty(pa.pa_tree_workspace_size(hq, hkv, d, max(ns)), device="cuda", dtype=torch.uint8)
        pa.pa_tree_decode(out, q, kc, vc, bt, i32(loc), lens, mask, max(ns), 0.125, tws)
        paths = []
        for s, n in enumerate(ns):
            a, path = rng.randrange(n), []
            while a >= 0:
                path.insert(0, a)
                a = parents[s][0][a]
            paths.append(path)
        most = max(map(len, paths))
        pa.pa_tree_commit(kc, vc, bt, i32(loc), lens, i32([p + [-1] * (most - len(p)) for p in paths]),
                          i32([len(p) for p in paths]), new_lens)
        resize(new_lens)
        for s, n in enumerate(ns):
            a, b = loc[s], loc[s + 1]
            ks, vs = (torch.stack([r[i] for r in rows[s]] + list(x[a:b])) for i, x in ((0, k), (1, v)))
            vis = torch.cat([torch.ones((n, ctx[s]), device="cuda", dtype=torch.bool), torch.tensor(sees[s], device="cuda")], 1)
            check_tree(out[a:b], q[a:b], ks, vs, vis, 0.125, f"turn {turn}, sequence {s}")
            rows[s] += [(k[a + j], v[a + j]) for j in paths[s]]
    assert pa.pa_device_errors(clear=True) == 0
    assert lens.tolist() == [len(r) for r in rows]
    for s in range(S):
        t = torch.arange(len(rows[s]), device="cuda")
        where = (bt[s, t // bs].long(), t % bs)
        assert torch.equal(kc[where], torch.stack([r[0] for r in rows[s]]))
        assert torch.equal(vc[where], torch.stack([r[1] for r in rows[s]]))
    resize(i32([0] * S))
    assert count.item() == nb and not ref.any() and sorted(free.tolist()) == list(range(nb))
    assert (bt == -1).all()
