"""pa_norm_rope_reshape_and_cache and pa_latent_rope_and_cache against their formulas in 64 bits
(bounds: latent_testutil)."""
import pytest
import torch

import paged_kv_cache_232_gb300 as pa
from latent_testutil import ROPE, TYPES, check_write, gen, half_step, norm64, randn, table, turn64

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _slots(g, n, n_slots, pad):
    s = torch.randperm(n_slots, generator=g, device="cuda")[:n]
    s[torch.randperm(n, generator=g, device="cuda")[:pad]] = -1
    return s


def _norm_rope(dt, n, hq, hkv, d, bs, fused, pad, in_place=False, max_pos=5000, seed=1, scale=1.5, eps=EPS):
    g = gen(seed)
    if fused:
        qkv = randn(g, (n, (hq + 2 * hkv) * d + 8), dt, scale)
        q, k, v = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in
                   ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    else:
        q, k, v = (randn(g, (n, h, d), dt, scale) for h in (hq, hkv, hkv))
    qw, kw = (randn(g, (d,), torch.float32, 0.2).add_(1).to(dt) for _ in range(2))
    blocks = -(-n // bs) + 2
    slots = _slots(g, n, blocks * bs, pad)
    pos = torch.randint(0, max_pos, (n,), generator=g, device="cuda")
    pos[:2] = torch.tensor([0, max_pos - 1], device="cuda")[:n]
    kc, vc = (randn(g, (blocks, bs, hkv, d), dt) for _ in range(2))
    cs = table(max_pos, d)
    return dict(q=q, k=k, v=v, qw=qw, kw=kw, kc=kc, vc=vc, slots=slots, pos=pos, cs=cs, eps=eps)


def _run_norm_rope(a, q_out):
    pa.pa_norm_rope_reshape_and_cache(a["q"], a["k"], a["v"], a["qw"], a["kw"], a["kc"], a["vc"], a["slots"], a["pos"],
                                      a["cs"], eps=a["eps"], q_out=q_out)


def _check_norm_rope(a, q0, kc0, vc0, q_out):
    cs = a["cs"][a["pos"]]
    check_write(q_out, *turn64(norm64(q0, a["qw"], a["eps"]), cs), "q")
    k, km = turn64(norm64(a["k"], a["kw"], a["eps"]), cs)
    live = a["slots"] >= 0
    at = a["slots"][live]
    kc, vc = a["kc"].flatten(0, 1), a["vc"].flatten(0, 1)
    check_write(kc[at], k[live], km[live], "k_cache")
    want_v, rest = vc0.flatten(0, 1).clone(), torch.ones(kc.shape[0], dtype=torch.bool, device="cuda")
    want_v[at] = a["v"][live]
    rest[at] = False
    assert torch.equal(vc, want_v), "v_cache"
    assert torch.equal(kc[rest], kc0.flatten(0, 1)[rest]), "untouched slots of k_cache"


@pytest.mark.parametrize("ty", ["bf16", "fp16"])
@pytest.mark.parametrize("n,hq,hkv,d,bs,fused,pad", [
    (1, 16, 8, 128, 16, True, 0), (3, 1, 1, 64, 8, False, 1), (77, 21, 3, 96, 32, True, 9), (130, 7, 1, 256, 128, False, 0),
    (5000, 16, 8, 128, 16, True, 500), (33, 64, 8, 64, 16, True, 33)])
def test_norm_rope_matches_formula(ty, n, hq, hkv, d, bs, fused, pad):
    dt = TYPES[ty]
    a = _norm_rope(dt, n, hq, hkv, d, bs, fused, pad, seed=n + d)
    q0, kc0, vc0 = a["q"].clone(), a["kc"].clone(), a["vc"].clone()
    pa.pa_device_errors(clear=True)
    out = torch.full((n, hq, d), float("nan"), device="cuda", dtype=dt)
    _run_norm_rope(a, out)
    _check_norm_rope(a, q0, kc0, vc0, out)
    assert torch.equal(a["q"], q0), "q is only read"
    _run_norm_rope(a, None)          # in place, over the (strided) q
    assert torch.equal(a["q"], out)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("ty", ["bf16", "fp16"])
@pytest.mark.parametrize("n,hq,hkv,d", [(3, 64, 8, 256), (700, 25, 4, 256), (9, 64, 16, 128), (2, 61, 2, 96), (5, 128, 3, 64)])
def test_norm_rope_more_head_rows_than_a_block_holds(ty, n, hq, hkv, d):
    """A block of 512 threads holds 32 head rows of 256 columns, 64 of 96 or 128, 128 of 64: the others in further
    passes over the tokens (the last one partly filled), q rewritten in place too."""
    a = _norm_rope(TYPES[ty], n, hq, hkv, d, 16, True, n // 3, seed=n + hq)
    q0, kc0, vc0 = a["q"].clone(), a["kc"].clone(), a["vc"].clone()
    pa.pa_device_errors(clear=True)
    out = torch.full((n, hq, d), float("nan"), device="cuda", dtype=TYPES[ty])
    _run_norm_rope(a, out)
    _check_norm_rope(a, q0, kc0, vc0, out)
    _run_norm_rope(a, None)
    assert torch.equal(a["q"], out)
    assert pa.pa_device_errors(clear=True) == 0


def test_norm_rope_extremes():
    """Rows of zeros (eps alone under the root), of the largest values and of tiny ones."""
    a = _norm_rope(torch.bfloat16, 4, 4, 2, 128, 16, False, 0, seed=5)
    a["q"][0] = 0
    a["q"][1] = 3.0e18          # its square is within fp32
    a["q"][2] = 1.0e-20
    a["k"][3] = 0
    out = torch.empty_like(a["q"])
    q0, kc0, vc0 = a["q"].clone(), a["kc"].clone(), a["vc"].clone()
    _run_norm_rope(a, out)
    _check_norm_rope(a, q0, kc0, vc0, out)
    assert not out[0].any()


def test_norm_rope_without_eps_and_a_nan_row():
    a = _norm_rope(torch.float16, 6, 4, 2, 64, 16, False, 0, seed=6, eps=0.0)
    a["q"][2, 1, 5] = float("nan")
    out = torch.empty_like(a["q"])
    q0 = a["q"].clone()
    _run_norm_rope(a, out)
    keep = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.isnan(out[2, 1]).all() and torch.isfinite(out[keep]).all()      # a head's row stays its own
    want, mag = turn64(norm64(q0, a["qw"], 0.0), a["cs"][a["pos"]])
    check_write(out[keep], want[keep], mag[keep], "the other rows")


# bf16 rows at the ends of the format: all values alike, one value alone, and a mixed row
_ENDS = [lambda r: r.fill_(1e-20), lambda r: r.fill_(1e-36), lambda r: r.fill_(-2.0 ** -133), lambda r: r.fill_(3.0e38),
         lambda r: r.zero_()[..., 5].fill_(2.0 ** -126), lambda r: r.zero_()[..., 9].fill_(2.0 ** -133),
         lambda r: r.zero_()[..., 3].fill_(3.0e38), lambda r: r.mul_(1e-25), lambda r: r.mul_(1e-37), lambda r: r.mul_(1e37)]


def _check_ends(got, want, mag, what):
    """check_write's bound, and half the smallest step of bf16 (2^-133): these rows' results reach down there."""
    d = 2.0 ** -19 * mag
    bad = (got.double() - want).abs() > half_step(got.dtype) * (want.abs() + d) + d + 2.0 ** -134
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values off"


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 1e-31, 1e-29, 1e-6])
def test_norm_rope_rows_at_the_ends_of_the_format(d, eps):
    """eps of any size next to rows whose squares leave fp32, each beside ordinary rows of the same warp; values are
    copied whatever their size."""
    eps = torch.tensor(eps, dtype=torch.float32).item()
    n = len(_ENDS)
    a = _norm_rope(torch.bfloat16, n, 4, 3, d, 16, False, 0, seed=12, eps=eps)
    for i, make in enumerate(_ENDS):
        make(a["q"][i, i % 4])
        make(a["k"][i, i % 3])
        make(a["v"][i, (i + 1) % 3])
    out = torch.empty_like(a["q"])
    q0 = a["q"].clone()
    _run_norm_rope(a, out)
    cs = a["cs"][a["pos"]]
    _check_ends(out, *turn64(norm64(q0, a["qw"], eps), cs), "q")
    _check_ends(a["kc"].flatten(0, 1)[a["slots"]], *turn64(norm64(a["k"], a["kw"], eps), cs), "k_cache")
    assert torch.equal(a["vc"].flatten(0, 1)[a["slots"]], a["v"]), "v_cache"


@pytest.mark.parametrize("dl", [256, 512])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 1e-31, 1e-29, 1e-6])
def test_latent_write_rows_at_the_ends_of_the_format(dl, eps):
    eps = torch.tensor(eps, dtype=torch.float32).item()
    a = _latent(torch.bfloat16, len(_ENDS) + 2, 0, dl, 16, 0, True, seed=13)
    for i, make in enumerate(_ENDS):
        make(a["kv"][i, :dl])
    pa.pa_latent_rope_and_cache(a["kv"], a["cache"], a["slots"], a["pos"], a["cs"], weight=a["w"], eps=eps)
    want = norm64(a["kv"][:, :dl], a["w"], eps)
    _check_ends(a["cache"].flatten(0, 1)[a["slots"]][:, :dl], want, want.abs(), "latent part")


def test_norm_rope_bad_rows_are_flagged_and_left():
    a = _norm_rope(torch.bfloat16, 8, 4, 2, 128, 16, False, 0, seed=7)
    a["pos"][2], a["pos"][5] = -1, 5000
    a["slots"][3] = a["kc"].shape[0] * 16
    out = torch.full((8, 4, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    kc0, vc0 = a["kc"].clone(), a["vc"].clone()
    pa.pa_device_errors(clear=True)
    _run_norm_rope(a, out)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_POSITION | pa.PA_DEVERR_SLOT
    assert (out[2] == 7).all() and (out[5] == 7).all()
    good = torch.tensor([0, 1, 4, 6, 7], device="cuda")
    changed = (a["kc"].flatten(0, 1) != kc0.flatten(0, 1)).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert sorted(changed) == sorted(a["slots"][good].tolist())
    changed = (a["vc"].flatten(0, 1) != vc0.flatten(0, 1)).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert sorted(changed) == sorted(a["slots"][good].tolist())


def _latent(dt, n, h, dl, bs, pad, norm, seed, max_pos=3000, kv_extra=0):
    g = gen(seed)
    blocks = -(-n // bs) + 2
    kv = randn(g, (n, dl + ROPE + kv_extra), dt, 1.5)[:, :dl + ROPE]
    pe = randn(g, (n, h, 40 + ROPE), dt)[:, :, 40:] if h else None
    return dict(kv=kv, pe=pe, q=randn(g, (n, h, dl + ROPE), dt) if h else None,
                w=randn(g, (dl,), torch.float32, 0.2).add_(1).to(dt) if norm else None,
                slots=_slots(g, n, blocks * bs, pad), pos=torch.randint(0, max_pos, (n,), generator=g, device="cuda"),
                cs=table(max_pos, ROPE), cache=randn(g, (blocks, bs, dl + ROPE), dt))


@pytest.mark.parametrize("ty", ["bf16", "fp16"])
@pytest.mark.parametrize("n,h,dl,bs,pad,norm,inter,extra", [
    (1, 16, 512, 16, 0, True, False, 0), (64, 128, 512, 64, 6, True, True, 64), (333, 7, 256, 8, 30, True, False, 8),
    (50, 1, 256, 128, 0, False, True, 0), (9, 0, 512, 32, 2, True, True, 0), (4001, 8, 512, 16, 11, False, False, 0)])
def test_latent_write_matches_formula(ty, n, h, dl, bs, pad, norm, inter, extra):
    a = _latent(TYPES[ty], n, h, dl, bs, pad, norm, seed=n + h, kv_extra=extra)
    cache0, q0 = a["cache"].clone(), None if h == 0 else a["q"].clone()
    pa.pa_device_errors(clear=True)
    pa.pa_latent_rope_and_cache(a["kv"], a["cache"], a["slots"], a["pos"], a["cs"], weight=a["w"], eps=EPS,
                                q_pe=a["pe"], q=a["q"], interleaved=inter)
    cs = a["cs"][a["pos"]]
    live = a["slots"] >= 0
    at = a["slots"][live]
    rows = a["cache"].flatten(0, 1)
    kr, km = turn64(a["kv"][:, None, dl:].double(), cs, inter)
    check_write(rows[at][:, dl:], kr[live, 0], km[live, 0], "key part")
    if norm:
        c = norm64(a["kv"][:, :dl], a["w"], EPS)[live]
        check_write(rows[at][:, :dl], c, c.abs(), "latent part")
    else:
        assert torch.equal(rows[at][:, :dl], a["kv"][live, :dl]), "without a weight the latent part is copied"
    rest = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(rows[rest], cache0.flatten(0, 1)[rest]), "untouched slots"
    if h:
        check_write(a["q"][..., dl:], *turn64(a["pe"].double(), cs, inter), "q")
        assert torch.equal(a["q"][..., :dl], q0[..., :dl]), "the other columns of q"
        # in place: q_pe is q's own last columns
        q2 = q0.clone()
        q2[..., dl:] = a["pe"]
        pa.pa_latent_rope_and_cache(a["kv"], a["cache"], a["slots"], a["pos"], a["cs"], weight=a["w"], eps=EPS,
                                    q_pe=q2[..., dl:], q=q2, interleaved=inter)
        assert torch.equal(q2, a["q"])
    assert pa.pa_device_errors(clear=True) == 0


def test_latent_write_bad_rows_are_flagged_and_left():
    a = _latent(torch.float16, 6, 4, 256, 16, 0, True, seed=3)
    a["pos"][1], a["slots"][4] = 3000, -2
    q0, c0 = a["q"].clone(), a["cache"].clone()
    pa.pa_device_errors(clear=True)
    pa.pa_latent_rope_and_cache(a["kv"], a["cache"], a["slots"], a["pos"], a["cs"], weight=a["w"], q_pe=a["pe"], q=a["q"])
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_POSITION | pa.PA_DEVERR_SLOT
    assert torch.equal(a["q"][1], q0[1]) and not torch.equal(a["q"][4], q0[4])
    changed = (a["cache"].flatten(0, 1) != c0.flatten(0, 1)).any(1).nonzero()[:, 0].tolist()
    assert sorted(changed) == sorted(a["slots"][[0, 2, 3, 5]].tolist())


def test_writes_on_a_side_stream():
    a = _norm_rope(torch.bfloat16, 300, 16, 8, 128, 16, True, 10, seed=11)
    q0, kc0, vc0 = a["q"].clone(), a["kc"].clone(), a["vc"].clone()
    out = torch.empty((300, 16, 128), device="cuda", dtype=torch.bfloat16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pa.pa_norm_rope_reshape_and_cache(a["q"], a["k"], a["v"], a["qw"], a["kw"], a["kc"], a["vc"], a["slots"], a["pos"],
                                      a["cs"], eps=EPS, q_out=out, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    _check_norm_rope(a, q0, kc0, vc0, out)


def test_norm_rope_feeds_decode():
    """A decode step as a user runs it: norm + rotation + write, then pa_decode over contexts that include the new
    rows; against attention in 64 bits over the written cache and queries."""
    g = gen(17)
    dt, S, hq, hkv, d, bs = torch.bfloat16, 5, 16, 8, 128, 16
    lens = [40, 1, 129, 16, 300]
    mb = 20
    bt = torch.randperm(S * mb, generator=g, device="cuda").to(torch.int32).view(S, mb).contiguous()
    kc, vc = (randn(g, (S * mb, bs, hkv, d), dt) for _ in range(2))
    qkv = randn(g, (S, (hq + 2 * hkv) * d), dt)
    q, k, v = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    qw, kw = (randn(g, (d,), torch.float32, 0.2).add_(1).to(dt) for _ in range(2))
    cl = torch.tensor(lens, device="cuda", dtype=torch.int32)
    pos = cl.long() - 1
    slots = bt[torch.arange(S, device="cuda"), pos // bs].long() * bs + pos % bs
    cs = table(400, d)
    qr, out = torch.empty((S, hq, d), device="cuda", dtype=dt), torch.empty((S, hq, d), device="cuda", dtype=dt)
    pa.pa_device_errors(clear=True)
    pa.pa_norm_rope_reshape_and_cache(q, k, v, qw, kw, kc, vc, slots, pos, cs, q_out=qr)
    ws = torch.empty(max(16, pa.pa_decode_workspace_size(S, hq, d, max(lens))), device="cuda", dtype=torch.uint8)
    pa.pa_decode(out, qr, kc, vc, bt, cl, max(lens), d ** -0.5, ws)
    assert pa.pa_device_errors(clear=True) == 0
    check_write(qr, *turn64(norm64(q, qw, EPS), cs[pos]), "q")
    kn = kc.flatten(0, 1)[slots]
    check_write(kn, *turn64(norm64(k, kw, EPS), cs[pos]), "k")
    for s, L in enumerate(lens):
        t = torch.arange(L, device="cuda")
        at = bt[s, t // bs].long() * bs + t % bs
        kk = kc.flatten(0, 1)[at].double().repeat_interleave(hq // hkv, 1)
        vv = vc.flatten(0, 1)[at].double().repeat_interleave(hq // hkv, 1)
        w = torch.softmax(torch.einsum("hd,thd->ht", qr[s].double(), kk) * d ** -0.5, -1)
        want, mag = torch.einsum("ht,thd->hd", w, vv), torch.einsum("ht,thd->hd", w, vv.abs())
        # fp32 sums: the allowance pa_decode's own tests use, and one rounding to the type
        assert ((out[s].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4 * mag + 1e-6).all(), f"sequence {s}"
