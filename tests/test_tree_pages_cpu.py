"""Host-side refusals, sizes and the tree mask of the drafted-tree and page entry points (no GPU: every refusal comes
before any device call)."""
import ctypes
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_232_gb300 as pa


@pytest.fixture(scope="module")
def lib():
    return pa.load()


VP, ODD, NEW = ctypes.c_void_p(16), ctypes.c_void_p(8), ctypes.c_void_p(48)     # never dereferenced


def test_tree_mask_is_the_ancestors():
    rng = random.Random(1)
    for n in (1, 2, 63, 64, 65, 200):
        parents = [rng.randint(-1, j - 1) for j in range(n)]
        mask, depth = pa.tree_mask(parents)
        assert mask.shape == (n, -(-n // 64)) and mask.dtype == np.int64
        for j in range(n):
            seen, a = set(), j
            while a >= 0:
                seen.add(a)
                a = parents[a]
            bits = {k for k in range(64 * mask.shape[1]) if int(mask[j, k // 64]) >> (k % 64) & 1}
            assert bits == seen and depth[j] == len(seen) - 1
    assert pa.tree_mask([-1, 0], mask_words=3)[0].shape == (2, 3)
    assert pa.tree_mask([])[0].shape == (0, 0)


def test_tree_mask_refusals(lib):
    for bad in ([0], [-1, 1], [-1, -2], [-1, 0, 5]):
        with pytest.raises(pa.PagedAttnError):
            pa.tree_mask(bad)
    with pytest.raises(ValueError):
        pa.tree_mask([[-1]])
    up = (ctypes.c_int * 3)(-1, 0, 0)
    out = (ctypes.c_int64 * 6)(*[7] * 6)
    assert lib.pa_tree_mask(out, None, up, -1, 1) == -2 and lib.pa_tree_mask(out, None, up, 3, 0) == -2
    assert lib.pa_tree_mask(None, None, up, 3, 1) == -1 and lib.pa_tree_mask(out, None, None, 3, 1) == -1
    up[2] = 2
    assert lib.pa_tree_mask(out, None, up, 3, 2) == -5 and list(out) == [7] * 6       # nothing written
    up[2] = 0
    assert lib.pa_tree_mask(out, None, up, 3, 2) == 0 and list(out) == [1, 0, 3, 0, 5, 0]
    assert lib.pa_tree_mask(None, None, None, 0, 0) == 0


def test_tree_decode_refusals(lib):
    size = lib.pa_tree_workspace_size(16, 8, 128, 20)

    def call(out=VP, q=VP, kc=VP, vc=VP, bt=VP, mb=8, loc=VP, sl=VP, mask=VP, words=1, S=2, mq=20, tq=40, hq=16, hkv=8, d=128,
             bs=16, nb=10, sc=0.1, dt=1, ws=VP, wb=size):
        return lib.pa_tree_decode(out, q, kc, vc, bt, mb, loc, sl, mask, words, S, mq, tq, hq, hkv, d, bs, nb, sc, dt, ws, wb,
                                  None)
    for name in ("out", "q", "kc", "vc", "bt", "loc", "sl", "mask"):
        assert call(**{name: None}) == -1, name
    for name in ("out", "q", "kc", "vc", "ws"):
        assert call(**{name: ODD}) == -6, name
    for bad in (dict(S=-1), dict(mq=-1), dict(tq=-1), dict(mb=0), dict(nb=0), dict(hq=0), dict(hkv=0), dict(hq=15),
                dict(words=-1), dict(words=0), dict(mq=65), dict(sc=float("inf")), dict(bs=0), dict(d=0)):
        assert call(**bad) == -2, bad
    for bad in (dict(hkv=1, hq=17), dict(d=80), dict(d=512), dict(bs=24), dict(dt=2), dict(mb=2 ** 28), dict(nb=2 ** 31),
                dict(tq=2 ** 28), dict(tq=2 ** 31, hq=1, hkv=1), dict(mq=2 ** 25, words=2 ** 20)):
        assert call(**bad) == -3, bad
    assert call(ws=None) == -7 and call(wb=size - 1) == -7
    assert call(S=0, out=None, ws=None) == 0 and call(mq=0, q=None) == 0 and call(tq=0, q=None) == 0


def test_tree_workspace_size():
    """Descriptors, the exp-sum pairs and the partials of two units a CTA; 96 columns run in the 128-column kernel."""
    def want(rows, d):
        return 2 * 160 * 16 + 2 * 160 * rows * 8 + 2 * 160 * rows * d * 4
    size = pa.pa_tree_workspace_size
    assert size(8, 8, 128, 1) == size(16, 8, 128, 16) == size(16, 1, 128, 2) == want(32, 128)
    assert size(16, 8, 128, 17) == size(3, 1, 96, 21) == want(64, 128)
    assert size(16, 8, 64, 33) == size(8, 8, 64, 128) == size(8, 8, 64, 1000) == want(128, 64)
    assert size(16, 8, 128, 0) == size(17, 1, 128, 4) == size(8, 8, 80, 4) == size(9, 8, 128, 4) == 0


def test_pages_refusals(lib):
    def copy(kc=VP, vc=VP, L=2, pairs=VP, n=3, row=256, bs=16, nb=10):
        return lib.pa_copy_pages(kc, vc, L, pairs, n, row, bs, nb, None)

    def commit(kc=VP, vc=VP, L=2, bt=VP, mb=8, loc=VP, sl=VP, path=VP, mp=4, acc=VP, new=NEW, S=2, row=256, bs=16, nb=10):
        return lib.pa_tree_commit(kc, vc, L, bt, mb, loc, sl, path, mp, acc, new, S, row, bs, nb, None)

    def fork(bt=VP, mb=8, sl=VP, par=VP, S=2, ref=VP, bs=16, nb=10):
        return lib.pa_fork_pages(bt, mb, sl, par, S, ref, bs, nb, None)

    size = lib.pa_resize_workspace_size(2, 10)

    def resize(kc=VP, vc=VP, L=2, bt=VP, mb=8, sl=VP, new=NEW, S=2, ref=VP, fl=VP, fc=VP, row=256, bs=16, nb=10, ws=VP, wb=size):
        return lib.pa_resize_pages(kc, vc, L, bt, mb, sl, new, S, ref, fl, fc, row, bs, nb, ws, wb, None)

    for fn, names in ((copy, ("kc", "pairs")), (commit, ("kc", "bt", "loc", "sl", "path", "acc", "new")),
                      (fork, ("bt", "sl", "par", "ref")), (resize, ("kc", "bt", "sl", "new", "ref", "fl", "fc"))):
        for name in names:
            assert fn(**{name: None}) == -1, (fn, name)
    for fn in (copy, commit, resize):
        assert fn(kc=ODD) == -6 and fn(vc=ODD) == -6
        for bad in (dict(L=0), dict(row=0), dict(row=-16), dict(nb=0), dict(bs=0)):
            assert fn(**bad) == -2, (fn, bad)
        for bad in (dict(row=24), dict(bs=20), dict(nb=2 ** 31), dict(row=2 ** 40), dict(L=2 ** 20)):
            assert fn(**bad) == -3, (fn, bad)
    for fn in (commit, fork, resize):
        assert fn(S=-1) == -2 and fn(mb=0) == -2 and fn(mb=2 ** 28) == -3 and fn(bs=12) == -3 and fn(nb=0) == -2
    assert copy(n=-1) == -2 and copy(n=2 ** 40) == -3 and copy(n=0, pairs=None) == 0
    assert commit(mp=-1) == -2 and commit(S=0, bt=None) == 0
    assert commit(sl=NEW) == -2 and commit(acc=NEW) == -2 and resize(sl=NEW) == -2     # read and written by one call
    assert fork(S=0, bt=None) == 0 and fork(nb=2 ** 31) == -3
    assert resize(ws=None) == -7 and resize(wb=size - 1) == -7 and resize(ws=ODD) == -6 and resize(S=0, bt=None) == 0


def test_resize_workspace_size():
    size = pa.pa_resize_workspace_size
    assert size(1, 1) == 256 + 256 + 256 and size(64, 40000) == 256 + 64 * 16 + 5120
    assert size(0, 10) == size(4, 0) == size(4, 2 ** 31) == 0


def test_bindings_check_shapes_first():
    """The Python calls refuse mismatched tensors by name (CPU tensors are refused last)."""
    i32 = torch.int32
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    bt, sl, new = torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i32)
    q, mask = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(6, 1, dtype=torch.int64)

    def tree(**kw):
        a = dict(out=q, q=q, k_cache=kc, v_cache=kc, block_tables=bt, query_start_loc=sl, seq_lens=sl, tree_mask=mask,
                 max_q_len=4, scale=0.1, workspace=None)
        pa.pa_tree_decode(**{**a, **kw})
    for name, bad in (("q", q[0]), ("k_cache", kc[0]), ("block_tables", bt[0]), ("tree_mask", mask[:, 0])):
        with pytest.raises(ValueError, match=f"{name} must be"):
            tree(**{name: bad})
    with pytest.raises(TypeError):
        tree(q=q.float())
    with pytest.raises(ValueError, match="CUDA"):
        tree()
    for bad in (kc[0], kc[None, None], kc[0, 0]):
        with pytest.raises(ValueError, match="k_cache must be"):
            pa.pa_copy_pages(bad, bad, bt[:, :2])
    with pytest.raises(ValueError, match="k_cache must be"):
        pa.pa_copy_pages(kc[0, 0], None, bt[:, :2])
    with pytest.raises(TypeError):
        pa.pa_copy_pages(kc.float(), kc.float(), bt[:, :2])
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_copy_pages(kc, kc, bt[:, :2])
    with pytest.raises(ValueError, match="ref_counts must be"):
        pa.pa_fork_pages(bt, sl, new, bt, 16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_fork_pages(bt, sl, new, sl, 16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_resize_pages(kc, kc, bt, sl, new, sl, sl, sl, None)
