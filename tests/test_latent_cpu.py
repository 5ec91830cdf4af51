"""Host-side refusals and sizes of the norm + rotary write and the latent-cache entry points (no GPU:
every refusal comes before any device call)."""
import ctypes
import os
import re

import pytest
import torch

import paged_kv_cache_232_gb300 as pa
from paged_kv_cache_232_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    return pa.load()


VP, ODD = ctypes.c_void_p(16), ctypes.c_void_p(8)     # never dereferenced


def test_norm_rope_refusals(lib):
    def call(q_out=VP, qos=2048, q=VP, qs=2048, k=VP, ks=1024, v=VP, vs=1024, qw=VP, kw=VP, eps=1e-6, kc=VP, vc=VP, sm=VP,
             pos=VP, cs=VP, n=4, hq=16, hkv=8, d=128, bs=16, nb=10, mp=100, dt=1):
        return lib.pa_norm_rope_reshape_and_cache(q_out, qos, q, qs, k, ks, v, vs, qw, kw, eps, kc, vc, sm, pos, cs, n, hq,
                                                  hkv, d, bs, nb, mp, dt, None)
    for name in ("q_out", "q", "k", "v", "qw", "kw", "kc", "vc", "sm", "pos", "cs"):
        assert call(**{name: None}) == -1, name
    for name in ("q_out", "q", "k", "v", "qw", "kw", "kc", "vc", "cs"):
        assert call(**{name: ODD}) == -6, name
    for bad in (dict(n=-1), dict(hq=0), dict(hkv=0), dict(nb=0), dict(mp=0), dict(bs=0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(qs=2040), dict(qos=2047), dict(ks=1000), dict(vs=1016)):
        assert call(**bad) == -2, bad
    for bad in (dict(d=80), dict(dt=2)):
        assert call(**bad) == -3, bad
    for bad in (dict(qs=2052), dict(ks=1028), dict(vs=1025), dict(qos=2049)):
        assert call(**bad) == -6, bad
    assert call(n=0, q=None) == 0


def test_latent_write_refusals(lib):
    def call(q=VP, pe=VP, pts=2048, phs=128, kv=VP, kvs=576, w=VP, eps=1e-6, c=VP, sm=VP, pos=VP, cs=VP, n=4, h=16, dl=512,
             rd=64, bs=16, nb=10, mp=100, inter=0, dt=1):
        return lib.pa_latent_rope_and_cache(q, pe, pts, phs, kv, kvs, w, eps, c, sm, pos, cs, n, h, dl, rd, bs, nb, mp,
                                            inter, dt, None)
    for name in ("q", "kv", "c", "sm", "pos", "cs"):
        assert call(**{name: None}) == -1, name
    for name in ("q", "pe", "kv", "w", "c", "cs"):
        assert call(**{name: ODD}) == -6, name
    for bad in (dict(n=-1), dict(h=0), dict(nb=0), dict(mp=0), dict(kvs=568), dict(phs=56), dict(pts=1976), dict(eps=-1.0)):
        assert call(**bad) == -2, bad
    for bad in (dict(dl=384), dict(rd=32), dict(bs=24), dict(dt=5), dict(h=129)):
        assert call(**bad) == -3, bad
    for bad in (dict(kvs=580), dict(phs=132), dict(pts=2050)):
        assert call(**bad) == -6, bad
    assert call(n=0, kv=None) == 0


def test_latent_attention_refusals(lib):
    size = lib.pa_latent_workspace_size(16, 512, 1)

    def decode(out=VP, q=VP, c=VP, bt=VP, mb=8, cl=VP, S=2, h=16, dl=512, rd=64, bs=16, nb=10, sc=0.1, dt=1, ws=VP, wb=size):
        return lib.pa_latent_decode(out, q, c, bt, mb, cl, S, h, dl, rd, bs, nb, sc, dt, ws, wb, None)

    def chunk(loc=VP, C=2, mq=1, tq=8, h=16, ws=VP, wb=size, kl=VP):
        return lib.pa_latent_prefill_chunk(VP, VP, VP, VP, 8, loc, kl, C, mq, tq, h, 512, 64, 16, 10, 0.1, 1, ws, wb, None)
    for name in ("out", "q", "c", "bt", "cl"):
        assert decode(**{name: None}) == -1, name
    for name in ("out", "q", "c", "ws"):
        assert decode(**{name: ODD}) == -6, name
    for bad in (dict(S=-1), dict(mb=0), dict(nb=0), dict(h=0), dict(sc=float("inf"))):
        assert decode(**bad) == -2, bad
    for bad in (dict(h=129), dict(dl=128), dict(rd=128), dict(bs=48), dict(dt=3), dict(mb=2 ** 28), dict(nb=2 ** 31),
                dict(S=2 ** 28)):
        assert decode(**bad) == -3, bad
    assert decode(ws=None) == -7 and decode(wb=size - 1) == -7
    assert decode(S=0, out=None, ws=None) == 0
    assert chunk(loc=None) == -1 and chunk(kl=None) == -1
    assert chunk(C=-1) == -2 and chunk(mq=-1) == -2 and chunk(tq=-1) == -2
    assert chunk(mq=5) == -7          # larger units than a decode's
    assert chunk(C=0, loc=None) == 0 and chunk(mq=0) == 0 and chunk(tq=0) == 0


def test_latent_workspace_size():
    """Descriptors, the exp-sum pairs and the partials of two units a CTA."""
    def want(rows, dl):
        return 2 * 160 * 16 + 2 * 160 * rows * 8 + 2 * 160 * rows * dl * 4
    size = pa.pa_latent_workspace_size
    assert size(16, 512) == size(1, 512, 5) == want(16, 512)
    assert size(17, 512) == size(16, 512, 2) == want(32, 512)
    assert size(33, 512) == size(128, 512) == size(16, 512, 100) == want(64, 512)
    assert size(24, 256, 129) == want(64, 256)
    assert size(129, 512) == size(16, 300) == size(0, 512) == size(16, 512, -1) == 0


def test_bindings_check_shapes_first():
    """The Python calls refuse mismatched tensors (CPU tensors are refused last, so shapes are tried here)."""
    c = torch.zeros(4, 16, 576, dtype=torch.bfloat16)
    q = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    bt, cl = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    out = torch.zeros(2, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa.pa_latent_decode(out, q[:, :, :500], c, bt, cl, 0.1, None)
    with pytest.raises(ValueError):
        pa.pa_latent_decode(out[:, :, :256], q, c, bt, cl, 0.1, None)
    with pytest.raises(ValueError):
        pa.pa_latent_decode(out, q, c, bt[:1], cl, 0.1, None)
    with pytest.raises(ValueError):
        pa.pa_latent_decode(out, q, c, bt, cl, 0.1, None)          # CPU tensors
    with pytest.raises(TypeError):
        pa.pa_latent_decode(out.float(), q.float(), c.float(), bt, cl, 0.1, None)
    k = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    kc = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    w, sl, cs = torch.zeros(128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64), torch.zeros(9, 128)
    qq = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa.pa_norm_rope_reshape_and_cache(qq, k, k, w[:64], w, kc, kc, sl, sl, cs)
    with pytest.raises(ValueError):
        pa.pa_norm_rope_reshape_and_cache(qq, k, k, w, w, kc, kc, sl[:1], sl, cs)
    with pytest.raises(ValueError):
        pa.pa_norm_rope_reshape_and_cache(qq, k, k, w, w, kc, kc, sl, sl, cs)
    with pytest.raises(ValueError):
        pa.pa_latent_rope_and_cache(c[:, 0], c, torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int64),
                                    torch.zeros(9, 64), q_pe=q[..., 512:])


def test_bindings_refuse_other_numbers_of_dimensions():
    """By name and with the shape that was meant, not by an unpacking error."""
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    c, q, kv = torch.zeros(4, 16, 576, dtype=bf), torch.zeros(2, 16, 576, dtype=bf), torch.zeros(2, 576, dtype=bf)
    bt, cl, sl, cs = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i64), torch.zeros(9, 64)
    out = torch.zeros(2, 16, 512, dtype=bf)

    def write(**kw):
        a = dict(kv=kv, latent_cache=c, slot_mapping=sl, positions=sl, cos_sin=cs)
        pa.pa_latent_rope_and_cache(**{**a, **kw})
    for name, bad in (("q_pe", torch.zeros(2, 16 * 64, dtype=bf)), ("q_pe", torch.zeros(64, dtype=bf)),
                      ("q_pe", torch.zeros(2, 4, 4, 64, dtype=bf)), ("kv", kv[0]), ("kv", kv[None]), ("kv", kv[0, 0]),
                      ("cos_sin", cs[0]), ("cos_sin", cs[0, 0]), ("latent_cache", c[0])):
        with pytest.raises(ValueError, match=f"{name} must be"):
            write(**({"q_pe": bad, "q": q} if name == "q_pe" else {name: bad}))
    with pytest.raises(ValueError, match="come together"):
        write(q_pe=q[..., 512:])
    for name, args in (("q", (out, q[0], c, bt, cl)), ("q", (out, q[None], c, bt, cl)), ("block_tables", (out, q, c, bt[0], cl)),
                       ("block_tables", (out, q, c, bt[None], cl)), ("latent_cache", (out, q, c[0], bt, cl))):
        with pytest.raises(ValueError, match=f"{name} must be"):
            pa.pa_latent_decode(*args, 0.1, None)
        with pytest.raises(ValueError, match=f"{name} must be"):
            pa.pa_latent_prefill_chunk(*args[:4], cl, args[4], 1, 0.1, None)
    k, kc, w = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(4, 16, 8, 64, dtype=bf), torch.zeros(64, dtype=bf)
    for name, kw in (("q", dict(q=k[0])), ("q", dict(q=k[None])), ("k_cache", dict(k_cache=kc[0])),
                     ("k_cache", dict(k_cache=kc[None])), ("cos_sin", dict(cos_sin=cs[0])), ("cos_sin", dict(cos_sin=cs[0, 0]))):
        a = dict(q=k, key=k, value=k, q_weight=w, k_weight=w, k_cache=kc, v_cache=kc, slot_mapping=sl, positions=sl, cos_sin=cs)
        with pytest.raises(ValueError, match=f"{name} must be"):
            pa.pa_norm_rope_reshape_and_cache(**{**a, **kw})


def test_device_error_bits_match_the_header():
    """Every cause has a bit of its own, under the same name in the header and the package."""
    with open(os.path.join(_build.INCLUDE, "pagedattn.h")) as f:
        bits = {m[1]: int(m[2]) for m in re.finditer(r"#define (PA_DEVERR_[A-Z]+) (\d+)u", f.read())}
    assert bits == {k: v for k, v in vars(pa).items() if k.startswith("PA_DEVERR_")}
    assert sorted(bits.values()) == [1 << i for i in range(len(bits))] and "PA_DEVERR_SMEM" in bits
