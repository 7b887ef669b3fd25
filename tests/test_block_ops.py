"""Norm, join, dropout and the gated feed-forward block against 64-bit
references.

Tolerances are counted, element by element, before any run: half a step of the
output's type relative to the value, plus a number of fp32 half steps (u = 2^-24)
times the magnitude that the formula reaches with every term taken positive.
A sum of C terms in any order is off by at most C u of its magnitude; the
activations' hardware exponential and reciprocal and the square roots take at
most 64 u between them at the arguments used here (|v| below 8: the rounding of
the exponent's argument costs |v| u).  Intermediate roundings of the
feed-forward block to bf16 are carried through the following products the same
way.
"""
import math

import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu
U = R.U
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def H():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import dimensional_fft_long_amd as H

    H.get_lib()
    return H


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def check(name, got, ref, tol):
    assert got.shape == ref.shape, name
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol)[bad].max()):.3g} of the bound"


def rng_words(seed=0x0123456789ABCDEF, offset=(1 << 33) + 5):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def sum_ch(t):
    return t.sum([0] + list(range(2, t.dim())))


# ------------------------------------------------------------- norm and join

def join_case(dtype, B, C, dims, gate=True, scale=True, post=True, pre=True, act="sigmoid", p=0.0, seed=0):
    g = gen(seed + C + sum(dims))
    s = (B, C) + tuple(dims)
    d = {"x": rand(g, s, dtype), "m": rand(g, s, dtype, 1.5), "gate": rand(g, s, dtype) if gate else None,
         "scale": 0.5 + torch.rand(C, generator=g, device="cuda") if scale else None,
         "w_post": 1.0 + rand(g, (C,), scale=0.2) if post else None,
         "w_pre": 1.0 + rand(g, (C,), scale=0.2) if pre else None}
    return d, rand(g, s, dtype), rand(g, s, dtype) if pre else None, dict(gate_act=act, eps=1e-5, p=p)


def check_join(H, d, dout, dh, kw, rng=None, fwd=None, bwd=None):
    p, eps, act = kw["p"], kw["eps"], kw["gate_act"]
    x, m = d["x"].double(), d["m"].double()
    dt, C = d["x"].dtype, x.shape[1]
    keep = R.keep_mask(int(rng[0]), int(rng[1]), p, x.shape).cuda() if p else None
    leaves = {k: v.double().requires_grad_() for k, v in d.items() if v is not None}
    out, h = R.join(**{k: leaves.get(k) for k in d}, gate_act=act, eps=eps, keep=keep, p=p)
    pairs = [(out, dout.double())] if dout is not None else []
    if dh is not None:
        pairs.append((h, dh.double()))
    ref = dict(zip(leaves, torch.autograd.grad([a for a, _ in pairs], list(leaves.values()), [b for _, b in pairs],
                                               allow_unused=True)))
    out, h = out.detach(), h.detach() if h is not None else None
    half = R.HALF[dt]
    k = (C + 64) * U
    one = torch.ones((), dtype=torch.float64, device="cuda")
    sc = R.ch(d["scale"].double(), x).abs() if d["scale"] is not None else one
    wp = R.ch(d["w_post"].double(), x).abs() if d["w_post"] is not None else one
    rm = R.rms(m, eps) if d["w_post"] is not None else one
    if d["gate"] is not None:
        gv = d["gate"].double()
        A = R.act(act, gv).abs()
        s = torch.sigmoid(gv)
        dA = {"none": torch.ones_like(gv), "sigmoid": s * (1 - s), "silu": s * (1 + gv.abs() * (1 - s))}[act]
    else:
        A = dA = one
    n = m.abs() * rm * wp
    kp = keep.double() / (1 - p) if p else one
    omag = x.abs() + n * A * sc * kp
    got_out, got_h = fwd if fwd else H.block_join_fwd(**d, **kw, rng=rng)
    check("out", got_out, out, half * out.abs() + k * omag)
    g = bwd if bwd else H.block_join_bwd(d["x"], d["m"], dout, dh, *[d[q] for q in ("gate", "scale", "w_post", "w_pre")],
                                         **kw, rng=rng)
    k2 = k + (x.numel() // C // 64) * U
    S = dout.double().abs() if dout is not None else torch.zeros_like(x)
    if h is not None:
        wq = R.ch(d["w_pre"].double(), x).abs()
        ro = R.rms(out, eps)
        rho = 1 + (out.abs() * omag).mean(1, keepdim=True) * ro ** 2
        check("h", got_h, h, half * h.abs() + k * (omag * ro * wq + h.abs() * rho))
        if dh is not None:
            q = dh.double().abs()
            dn = q * wq
            S = S + ro * dn * (1 + rho) + ro ** 3 * (omag * (dn * out.abs()).mean(1, keepdim=True)
                                                     + out.abs() * (dn * omag).mean(1, keepdim=True)
                                                     + 3 * rho * out.abs() * (dn * out.abs()).mean(1, keepdim=True))
            check("dw_pre", g["dw_pre"], ref["w_pre"], U * ref["w_pre"].abs() + k2 * sum_ch(q * ro * (omag + out.abs() * rho)))
        else:
            assert not g["dw_pre"].any()
    else:
        assert got_h is None and g["dw_pre"] is None
    check("dx", g["dx"], ref["x"], half * ref["x"].abs() + k * S)
    S = S * kp
    if d["gate"] is not None:
        check("dgate", g["dgate"], ref["gate"], half * ref["gate"].abs() + 2 * k * S * sc * n * dA)
    if d["scale"] is not None:
        check("dscale", g["dscale"], ref["scale"], U * ref["scale"].abs() + 2 * k2 * sum_ch(S * A * n))
    if d["w_post"] is not None:
        check("dw_post", g["dw_post"], ref["w_post"], U * ref["w_post"].abs() + 2 * k2 * sum_ch(S * A * sc * m.abs() * rm))
    e = S * sc * A * wp
    if d["w_post"] is not None:
        e = rm * e + m.abs() * rm ** 3 * (e * m.abs()).mean(1, keepdim=True)
    check("dm", g["dm"], ref["m"], half * ref["m"].abs() + 3 * k * e)


SHAPES = [  # B, C, dims
    (1, 1, (1,)), (3, 5, (1,)), (4, 1024, (1,)), (2, 1021, (1, 1)), (1, 8192, (1,)), (2, 4100, (1, 1, 1)),
    (2, 3, (2,)), (1, 7, (3, 1)), (5, 16, (7,)), (2, 64, (8,)), (3, 100, (37, 3)), (1, 9, (5, 5, 5)),
    (2, 64, (16, 32)), (1, 33, (1001,)), (2, 128, (8, 129)), (1, 300, (257,)), (1, 700, (40,)), (1, 2050, (9,)),
    (1, 4096, (16,)), (1, 5000, (11,)), (1, 8192, (8,)), (1, 8191, (3,)), (1, 4, (70000,)),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,C,dims", SHAPES, ids=lambda v: str(v))
def test_join_shapes(H, B, C, dims, dtype):
    print(f"[join] B={B} C={C} dims={dims} {dtype}", flush=True)
    p = 0.3 if (C + dims[0]) % 2 else 0.0
    d, dout, dh, kw = join_case(dtype, B, C, dims, act=("sigmoid", "silu", "none")[(C + B) % 3], p=p)
    check_join(H, d, dout, dh, kw, rng=rng_words() if p else None)


@pytest.mark.parametrize("gate,scale,post,pre", [(0, 0, 0, 0), (1, 0, 0, 0), (0, 1, 0, 1), (0, 0, 1, 0), (1, 1, 0, 1),
                                                 (1, 0, 1, 1), (0, 1, 1, 0), (0, 0, 0, 1)])
@pytest.mark.parametrize("dims", [(1,), (45,)], ids=["token", "grid"])
def test_join_parts(H, gate, scale, post, pre, dims):
    d, dout, dh, kw = join_case(F32, 2, 40, dims, gate, scale, post, pre, act="silu", p=0.2)
    check_join(H, d, dout, dh, kw, rng=rng_words(-7, 3))
    if pre:   # one gradient alone
        check_join(H, d, dout, None, kw, rng=rng_words(-7, 3))
        check_join(H, d, None, dh, kw, rng=rng_words(-7, 3))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,C,dims", SHAPES, ids=lambda v: str(v))
def test_norm_shapes(H, B, C, dims, dtype):
    print(f"[norm] B={B} C={C} dims={dims} {dtype}", flush=True)
    g = gen(C + sum(dims))
    x, dh = rand(g, (B, C) + dims, dtype), rand(g, (B, C) + dims, dtype)
    w = 1.0 + rand(g, (C,), scale=0.2)
    eps, half, k = 1e-5, R.HALF[dtype], (C + 64) * U
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    r = R.rms(xd, eps)
    h = xd * r * R.ch(wd, xd)
    dx, dw = torch.autograd.grad(h, [xd, wd], dh.double())
    xd, r, h = xd.detach(), r.detach(), h.detach()
    check("h", H.block_norm_fwd(x, w, eps), h, (half + 2 * k) * h.abs())
    gx, gw = H.block_norm_bwd(x, w, dh, eps)
    dn = dh.double().abs() * R.ch(w.double(), xd).abs()
    check("dx", gx, dx, half * dx.abs() + 6 * k * (r * dn + xd.abs() * r ** 3 * (dn * xd.abs()).mean(1, keepdim=True)))
    k2 = 3 * k + (x.numel() // C // 64) * U
    check("dw", gw, dw, U * dw.abs() + k2 * sum_ch(dh.double().abs() * xd.abs() * r))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,C,dims", [(2, 1, (300001,)), (1, 2, (530000,)), (2, 3, (270001,)), (3, 4, (200002,)),
                                      (1, 5, (601, 1000)), (2, 8, (262147,)), (1, 9, (530001,))], ids=lambda v: str(v))
def test_few_channels_many_positions(H, B, C, dims, dtype):
    """Workgroups of one to four waves."""
    test_norm_shapes(H, B, C, dims, dtype)
    p = 0.3 if C in (3, 8) else 0.0
    d, dout, dh, kw = join_case(dtype, B, C, dims, act="silu", p=p)
    check_join(H, d, dout, dh, kw, rng=rng_words() if p else None)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,C,dims", [(1, 283, (2, 10037)), (2, 264, (8200,)), (2, 717, (684,)), (1, 1000, (4099,)),
                                      (2, 520, (9000,)), (1, 2048, (520,)), (1, 2048, (1037,)), (1, 1536, (8192,)),
                                      (3, 1030, (23,)), (1, 700, (4, 8))], ids=lambda v: str(v))
def test_join_many_channels(H, B, C, dims, dtype):
    """The join's backward with its tensors in LDS: rows of whole 16-byte pieces
    and others, several tiles a workgroup and less than one."""
    p = 0.3 if B * C * math.prod(dims) < 2 ** 21 else 0.0
    d, dout, dh, kw = join_case(dtype, B, C, dims, act=("sigmoid", "silu", "none")[C % 3], p=p)
    rng = rng_words() if p else None
    check_join(H, d, dout, dh, kw, rng=rng)
    g = H.block_join_bwd(d["x"], d["m"], dout, dh, *[d[q] for q in ("gate", "scale", "w_post", "w_pre")], **kw, rng=rng)
    buf = {}
    for k, t in (("x", d["x"]), ("m", d["m"]), ("gate", d["gate"]), ("dh", dh)):   # one tensor at a time off its 16 bytes
        buf[k] = torch.empty(t.numel() + 1, dtype=dtype, device="cuda")[1:].view(t.shape).copy_(t)
    for k in buf:
        a = {q: buf[q] if q == k else (dh if q == "dh" else d[q]) for q in buf}
        r = H.block_join_bwd(a["x"], a["m"], dout, a["dh"], a["gate"], d["scale"], d["w_post"], d["w_pre"], **kw, rng=rng)
        assert all(torch.equal(r[q], g[q]) for q in g), k


@pytest.mark.parametrize("L", [2000, 2001])
@pytest.mark.parametrize("gate,scale,post,pre", [(0, 0, 0, 0), (1, 0, 0, 0), (0, 1, 0, 1), (0, 0, 1, 0), (1, 0, 1, 1)])
def test_join_parts_of_many_channels(H, gate, scale, post, pre, L):
    for dtype in (F32, BF16):
        d, dout, dh, kw = join_case(dtype, 1, 400, (L,), gate, scale, post, pre, act="silu", p=0.2)
        check_join(H, d, dout, dh, kw, rng=rng_words(-7, 3))
        if pre:
            check_join(H, d, dout, None, kw, rng=rng_words(-7, 3))
            check_join(H, d, None, dh, kw, rng=rng_words(-7, 3))


def test_join_rows_of_zeros_and_large_values(H):
    """A position whose channels are all zero has the finite factor eps^(-1/2);
    a dropped element passes x through whatever the branch holds there."""
    d, dout, dh, kw = join_case(F32, 2, 24, (19,), p=0.4)
    d["m"][:, :, 3] = 0.0
    d["x"][:, :, 3] = 0.0
    check_join(H, d, dout, dh, kw, rng=rng_words())
    rng = rng_words(9, 0)
    keep = R.keep_mask(9, 0, 0.4, d["x"].shape).cuda()
    dd = dict(d, w_post=None, w_pre=None)
    dd["m"] = torch.where(keep, d["m"], torch.full_like(d["m"], float("nan")))
    out, _ = H.block_join_fwd(**dd, **kw, rng=rng)
    assert torch.equal(out[~keep], d["x"][~keep]) and bool(torch.isfinite(out).all())
    # non-finite values stay in their own position
    d["m"][0, 5, 7] = float("inf")
    out, h = H.block_join_fwd(**d, **dict(kw, p=0.0))
    ok = torch.ones_like(out, dtype=torch.bool)
    ok[0, :, 7] = False
    assert bool(torch.isfinite(out[ok]).all()) and bool(torch.isfinite(h[ok]).all())
    assert not bool(torch.isfinite(out[0, 5, 7]))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_join_at_odd_addresses(H, dtype):
    """Tensors that start at any element of a buffer."""
    for off in (1, 3):
        d, dout, dh, kw = join_case(dtype, 2, 20, (6, 11), p=0.1)

        def moved(t):
            buf = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
            v = buf[off:].view(t.shape)
            v.copy_(t)
            return v

        d = {k: moved(v) for k, v in d.items()}
        out, h = moved(d["x"]), moved(d["x"])
        H.block_join_fwd(**d, **kw, rng=rng_words(), out=out, h=h)
        check_join(H, d, moved(dout), moved(dh), kw, rng=rng_words(), fwd=(out, h))


def test_join_gradients_against_differences(H):
    """Directional differences of the forward kernel against the backward's
    gradients: the rounding of the outputs over the step, plus the difference
    quotient's own error, taken from the 64-bit formula at the same step."""
    d, dout, dh, kw = join_case(F32, 2, 12, (5, 3), act="silu", p=0.25)
    rng = rng_words(77, 1)
    keep = R.keep_mask(77, 1, 0.25, d["x"].shape).cuda()
    grads = H.block_join_bwd(d["x"], d["m"], dout, dh, d["gate"], d["scale"], d["w_post"], d["w_pre"], **kw, rng=rng)
    g, step = gen(5), 2.0 ** -6

    def ref(v):
        o, h = R.join(**{k: t.double() for k, t in v.items()}, gate_act="silu", eps=kw["eps"], keep=keep, p=0.25)
        return float((o * dout.double()).sum() + (h * dh.double()).sum())

    def own(v):
        o, h = H.block_join_fwd(**v, **kw, rng=rng)
        return float((o.double() * dout.double()).sum() + (h.double() * dh.double()).sum())

    o, h = H.block_join_fwd(**d, **kw, rng=rng)
    mag = float((dout.abs() * (d["x"].abs() + (o - d["x"]).abs())).sum() + 4 * (dh.abs() * (h.abs() + 1)).sum())
    for name in d:
        v = rand(g, d[name].shape).sign()
        up, dn = dict(d), dict(d)
        up[name], dn[name] = d[name] + step * v, d[name] - step * v
        real = (up[name].double() - dn[name].double())           # the step as rounded
        slope = float((grads["d" + name].double() * real).sum())
        xs = {k: t.double().requires_grad_() for k, t in d.items()}
        ro, rh = R.join(**xs, gate_act="silu", eps=kw["eps"], keep=keep, p=0.25)
        (rg,) = torch.autograd.grad((ro * dout.double()).sum() + (rh * dh.double()).sum(), [xs[name]])
        curve = abs(ref(up) - ref(dn) - float((rg * real).sum()))
        k = (12 + 64) * U
        assert abs(own(up) - own(dn) - slope) <= curve + 4 * k * mag, name


# ------------------------------------------------------------------- dropout

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 63, 1023, 4096, 100003])
def test_dropout_masks(H, n, dtype):
    for p, seed, offset in ((0.5, 0, 0), (0.1, -1, 2 ** 32 - 2), (0.999, 12345, -3), (2.0 ** -33, 1, 1), (0.0, 5, 5)):
        print(f"[dropout] n={n} p={p} {dtype}", flush=True)
        x = rand(gen(n), (n,), dtype)
        y = H.dropout_fwd(x, p, rng_words(seed, offset))
        keep = R.keep_mask(seed, offset, p, (n,)).cuda()
        f = torch.tensor(1.0 / (1.0 - p), dtype=F32, device="cuda")
        want = torch.where(keep, (x.float() * f).to(dtype), torch.zeros_like(x))  # one product, one rounding: exact
        assert torch.equal(y, want)
        assert torch.equal(H.dropout_bwd(x, p, rng_words(seed, offset)), want)


def test_dropout_odd_addresses_nan_and_empty(H):
    rng = rng_words(3, 3)
    for dtype in (F32, BF16):
        x = rand(gen(1), (1000,), dtype)
        y = torch.full_like(x, 7.0)
        H.dropout_fwd(x[1:990], 0.5, rng, y=y[5:994])
        keep = R.keep_mask(3, 3, 0.5, (989,)).cuda()
        assert torch.equal(y[5:994], torch.where(keep, x[1:990] * 2, torch.zeros_like(x[1:990])))
        assert bool((y[:5] == 7).all()) and bool((y[994:] == 7).all())
        z = torch.full((64,), float("nan"), dtype=dtype, device="cuda")
        out = H.dropout_fwd(z, 0.5, rng)
        k = R.keep_mask(3, 3, 0.5, (64,)).cuda()
        assert bool(torch.isnan(out[k]).all()) and not bool(out[~k].any())
        assert H.dropout_fwd(z[:0], 0.5, rng).numel() == 0


def test_join_draws_dropouts_mask(H):
    """The join's mask is dropout's of the same words on the branch."""
    g = gen(3)
    x, m, rng = rand(g, (2, 6, 13)), rand(g, (2, 6, 13)), rng_words(4, 4)
    out, _ = H.block_join_fwd(x, m, p=0.5, rng=rng)
    assert torch.equal(out, x + H.dropout_fwd(m, 0.5, rng))


# -------------------------------------------------------------- feed-forward

def ffn_case(dtype, B, C, F, dims, seed=0):
    g = gen(seed + C + F + sum(dims))
    return (rand(g, (B, C) + tuple(dims), dtype), rand(g, (F, C), dtype, C ** -0.5), rand(g, (F, C), dtype, C ** -0.5),
            rand(g, (C, F), dtype, F ** -0.5), rand(g, (B, C) + tuple(dims), dtype))


def check_ffn(H, x, Wg, Wu, Wd, dy, act, fwd=None, bwd=None):
    dt, C, F = x.dtype, x.shape[1], Wg.shape[0]
    half = R.HALF[dt]
    L = math.prod(x.shape[2:])
    X = x.double().transpose(0, 1).reshape(C, -1)       # [C, T]
    DY = dy.double().transpose(0, 1).reshape(C, -1)
    T = X.shape[1]
    wg, wu, wd = Wg.double(), Wu.double(), Wd.double()
    leaves = [t.clone().requires_grad_() for t in (X, wg, wu, wd)]
    Y = leaves[3] @ (R.act(act, leaves[1] @ leaves[0]) * (leaves[2] @ leaves[0]))
    dX, dwg, dwu, dwd = torch.autograd.grad(Y, leaves, DY)
    Y = Y.detach()
    g, u = wg @ X, wu @ X
    gl = g.clone().requires_grad_()
    a = R.act(act, gl)
    (da,) = torch.autograd.grad(a.sum(), gl)
    a = a.detach()
    h = a * u
    kC, kF, kT = (C + 64) * U, (F + 64) * U, (T + 64) * U
    eg0, eu0 = kC * (wg.abs() @ X.abs()), kC * (wu.abs() @ X.abs())
    eh = half * h.abs() + 1.13 * eg0 * u.abs() + a.abs() * eu0 + 16 * U * (g.abs() + 1) * u.abs()

    def grid(t):   # [C, T] -> x's shape
        return t.reshape(C, x.shape[0], L).transpose(0, 1).reshape(x.shape)

    y = fwd if fwd is not None else H.gated_ffn_fwd(x, Wg, Wu, Wd, act)
    check("y", y, grid(Y), grid(half * Y.abs() + wd.abs() @ eh + kF * (wd.abs() @ h.abs()) + 1e-30))
    gx, gg, gu, gd = bwd if bwd else H.gated_ffn_bwd(x, Wg, Wu, Wd, dy, act)
    dh = wd.t() @ DY
    edh = kC * (wd.t().abs() @ DY.abs())
    eg, eu = eg0 + half * g.abs(), eu0 + half * u.abs()
    dg, du = dh * u * da, dh * a
    edg = half * dg.abs() + edh * (u * da).abs() + dh.abs() * (eu * da.abs() + u.abs() * eg + 16 * U * u.abs())
    edu = half * du.abs() + edh * a.abs() + dh.abs() * (1.13 * eg + 16 * U * (g.abs() + 1))
    check("dx", gx, grid(dX), grid(half * dX.abs() + wg.t().abs() @ edg + wu.t().abs() @ edu
                                   + 2 * kF * (wg.t().abs() @ dg.abs() + wu.t().abs() @ du.abs()) + 1e-30))
    check("dWg", gg, dwg, half * dwg.abs() + edg @ X.abs().t() + kT * (dg.abs() @ X.abs().t()) + 1e-30)
    check("dWu", gu, dwu, half * dwu.abs() + edu @ X.abs().t() + kT * (du.abs() @ X.abs().t()) + 1e-30)
    check("dWd", gd, dwd, half * dwd.abs() + DY.abs() @ eh.t() + kT * (DY.abs() @ h.abs().t()) + 1e-30)


FFN = [  # B, C, F, dims
    (1, 1, 1, (1,)), (1, 8, 8, (8,)), (2, 3, 5, (7,)), (4, 64, 256, (1,)), (17, 72, 136, (1,)), (40, 256, 512, (1,)),
    (3, 1024, 520, (1,)), (1, 64, 256, (16, 16)), (2, 128, 512, (40, 16)), (1, 100, 333, (37, 53)),
    (2, 32, 128, (8, 8, 8)), (5, 40, 96, (24,)), (3, 264, 200, (72,)), (1, 520, 1032, (264,)), (2, 129, 257, (513,)),
    (9, 16, 48, (3, 5)), (1, 8, 16, (4096,)), (1, 256, 264, (520,)), (70, 24, 40, (1,)), (300, 136, 72, (1,)),
    (2, 320, 640, (1000,)), (2, 136, 520, (5120,)), (2, 136, 520, (5119,)), (1, 1032, 264, (10240,)),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,C,F,dims", FFN, ids=lambda v: str(v))
def test_ffn_shapes(H, B, C, F, dims, dtype):
    act = ("silu", "gelu", "sigmoid")[(B + C) % 3]
    print(f"[ffn] B={B} C={C} F={F} dims={dims} {dtype} {act}", flush=True)
    check_ffn(H, *ffn_case(dtype, B, C, F, dims), act)


def test_ffn_non_finite_values_stay_in_their_position(H):
    for dtype in (F32, BF16):
        x, Wg, Wu, Wd, dy = ffn_case(dtype, 2, 40, 72, (33,))
        want = H.gated_ffn_fwd(x, Wg, Wu, Wd)
        x2 = x.clone()
        x2[0, 3, 5], x2[1, 7, 32], x2[1, 0, 0] = float("nan"), float("inf"), -float("inf")
        y = H.gated_ffn_fwd(x2, Wg, Wu, Wd)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[0, :, 5] = hit[1, :, 32] = hit[1, :, 0] = True
        assert torch.equal(y[~hit], want[~hit]) and not bool(torch.isfinite(y[hit]).any())


def test_ffn_large_and_tiny_fp32_values(H):
    """fp32 keeps its range: products near the type's largest value, weights far below one."""
    x, Wg, Wu, Wd, dy = ffn_case(F32, 1, 24, 40, (17,))
    y1 = H.gated_ffn_fwd(x, Wg * 0 + 1e-3, Wu * 1e19, Wd * 1e17, act="sigmoid")
    y0 = H.gated_ffn_fwd(x, Wg * 0 + 1e-3, Wu * 1e-15, Wd * 1e-15, act="sigmoid")
    ref = R.ffn(x.double(), Wg.double() * 0 + float(torch.tensor(1e-3)), Wu.double(), Wd.double(), "sigmoid")
    mag = float(ref.abs().max())
    # scaled weights round once each (2 half steps); the sums as in check_ffn, taken against the largest result
    for y, f in ((y1, 1e36), (y0, 1e-30)):
        assert float((y.double() / f - ref).abs().max()) <= (24 + 40 + 128) * U * 24 * mag


# ------------------------------------------------ streams, graphs, determinism

def _all_ops(H, t, p=0.2):
    x, m, gate, dout, dh, sc, w1, w2, Wg, Wu, Wd, rng = t
    h = H.block_norm_fwd(x, w1)
    out, h2 = H.block_join_fwd(x, m, gate, sc, w1, w2, p=p, rng=rng)
    r = [h, out, h2, H.dropout_fwd(x, 0.5, rng), H.gated_ffn_fwd(x, Wg, Wu, Wd), *H.block_norm_bwd(x, w1, dh)]
    g = H.block_join_bwd(x, m, dout, dh, gate, sc, w1, w2, p=p, rng=rng)
    return r + [g[k] for k in sorted(g)] + list(H.gated_ffn_bwd(x, Wg, Wu, Wd, dout))


def _tensors(dtype=BF16, B=2, C=48, dims=(9, 16), F=80, seed=1):
    g = gen(seed)
    s = (B, C) + dims
    return [rand(g, s, dtype) for _ in range(5)] + [1 + rand(g, (C,), scale=0.1) for _ in range(3)] + \
        [rand(g, (F, C), dtype, 0.1), rand(g, (F, C), dtype, 0.1), rand(g, (C, F), dtype, 0.1), rng_words(8, 8)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_same_bits_every_time(H, dtype):
    t = _tensors(dtype, 3, 96, (40, 33), 200)
    first = _all_ops(H, t)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, _all_ops(H, t)))


def test_calls_on_other_streams(H):
    """Two streams at once, each with its own inputs: the workspaces are apart."""
    sets = [_tensors(seed=s) for s in (1, 2)]
    want = [_all_ops(H, t) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _all_ops(H, sets[i])
    torch.cuda.synchronize()
    for w, q in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, q))
    s = streams[0]
    x, w = sets[0][0], sets[0][6]
    s.wait_stream(torch.cuda.current_stream())
    h = H.block_norm_fwd(x, w, stream=s)
    y = H.gated_ffn_fwd(x, *sets[0][8:11], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(h, want[0][0]) and torch.equal(y, want[0][4])


def test_two_graphs_replay_like_eager_calls(H):
    """Two captured graphs, replayed in turn and together with eager work
    between the replays: each holds its own workspaces; new inputs and advanced
    dropout words are seen by the replays."""
    sets = [_tensors(seed=s) for s in (3, 4)]
    for t in sets:
        _all_ops(H, t)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in sets:
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            outs.append(_all_ops(H, t))
        graphs.append(g)
    for rep in range(3):
        for t in sets:
            t[0].copy_(rand(gen(50 + rep), t[0].shape, BF16))
            t[-1][1] += 1000
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        got = [[v.clone() for v in o] for o in outs]
        _ = (sets[0][0].float() * 2).sum()
        want = [_all_ops(H, t) for t in sets]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b)), rep


def test_empty_calls(H):
    w, wf = torch.ones(6, device="cuda"), torch.ones(5, 6, device="cuda")
    for shape in ((0, 6, 4), (2, 6, 0), (2, 6, 3, 0)):
        x = torch.zeros(shape, device="cuda")
        assert H.block_norm_fwd(x, w).shape == x.shape
        dx, dw = H.block_norm_bwd(x, w, x)
        assert dx.shape == x.shape and not dw.any()
        o, h = H.block_join_fwd(x, x, x, w, w, w)
        g = H.block_join_bwd(x, x, x, x, x, w, w, w)
        assert not g["dscale"].any() and not g["dw_post"].any() and not g["dw_pre"].any() and o.shape == h.shape
        for dt in (F32, BF16):
            xb, wb = x.to(dt), wf.to(dt)
            assert H.gated_ffn_fwd(xb, wb, wb, wb.t().contiguous()).shape == x.shape
            r = H.gated_ffn_bwd(xb, wb, wb, wb.t().contiguous(), xb)
            assert r[0].shape == x.shape and not any(v.any() for v in r[1:])


def test_refusals_on_the_device(H):
    x, w = torch.zeros(2, 6, 8, device="cuda"), torch.ones(6, device="cuda")
    with pytest.raises(ValueError):
        H.block_norm_fwd(x, w, h=x)
    with pytest.raises(ValueError):
        H.block_join_fwd(x, x, h=x.clone())
    with pytest.raises(ValueError):
        H.block_join_bwd(x, x, x, x)                       # dh without w_pre
    out = torch.empty_like(x)
    with pytest.raises(ValueError):
        H.block_join_fwd(x, x.clone(), w_pre=w, out=out, h=out)
    with pytest.raises(TypeError):
        H.block_join_fwd(x, x, p=0.1)                      # no rng
    with pytest.raises(TypeError):
        H.block_norm_fwd(x.transpose(1, 2), w)
    with pytest.raises(TypeError):
        H.block_norm_fwd(x.half(), w)
    W = torch.zeros(4 * 6 + 1, device="cuda")
    with pytest.raises(H.HyenandError) as e:               # weights off a 16-byte address
        H.gated_ffn_fwd(x, W[1:].view(4, 6), W[:24].view(4, 6), W[:24].view(6, 4))
    assert e.value.code == H.ERR_INVALID_ARG
    with pytest.raises(H.HyenandError) as e:
        H.gated_ffn_fwd(x, *[torch.zeros(s, device="cuda") for s in ((4, 6), (4, 6), (6, 4))],
                        workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == H.ERR_WORKSPACE


def test_inputs_and_their_neighbours_stay_as_they_were(H):
    """Nothing outside the outputs is written."""
    t = _tensors(F32, 1, 20, (7, 5), 33)
    kept = [v.clone() for v in t]
    _all_ops(H, t)
    assert all(torch.equal(a, b) for a, b in zip(t, kept))
    x = t[0]
    buf = torch.full((3, *x.shape), 9.0, device="cuda")
    H.block_norm_fwd(x, t[6], h=buf[1])
    assert bool((buf[0] == 9).all()) and bool((buf[2] == 9).all())
    xb = torch.zeros(1, 24, 7, 8, device="cuda", dtype=BF16)
    ob = torch.full((3, *xb.shape), 9.0, device="cuda", dtype=BF16)
    W = torch.ones(40, 24, device="cuda", dtype=BF16)
    H.gated_ffn_fwd(xb, W, W, W.t().contiguous(), y=ob[1])
    assert bool((ob[0] == 9).all()) and bool((ob[2] == 9).all()) and not ob[1].any()


# ------------------------------------------------------- the layer, together

def test_layer_with_the_convolution(H):
    """norm -> gated convolution -> join (with the next norm) -> feed-forward ->
    join, forward and backward through autograd, against the same layer in 64
    bits.  The bar is the convolution's own: max |d| / max |ref| <= 1e-4."""
    dims, B, C, F = (8, 16), 2, 12, 20
    g = gen(11)
    s = (B, C) + dims
    v = {"x": rand(g, s), "al": rand(g, (C,)), "be": rand(g, (C,)), "K": rand(g, (C, 15, 31), scale=0.1),
         "gate": rand(g, s), "s1": 0.5 + rand(g, (C,), scale=0.1), "s2": 0.5 + rand(g, (C,), scale=0.1),
         "Wg": rand(g, (F, C), scale=0.3), "Wu": rand(g, (F, C), scale=0.3), "Wd": rand(g, (C, F), scale=0.3)}
    v.update({f"w{i}": 1 + rand(g, (C,), scale=0.1) for i in range(4)})
    dy, dh = rand(g, s), rand(g, s)
    rng = rng_words(21, 0)

    def own(t):
        m = H.gated_fftconv(H.block_norm(t["x"], t["w0"]), t["al"], t["be"], t["K"])
        x, h = H.block_join(t["x"], m, t["gate"], t["s1"], t["w1"], t["w2"], p=0.2, rng=rng)
        h = H.dropout(h, 0.1, rng + torch.tensor([0, 1000], device="cuda"))
        return H.block_join(x, H.gated_ffn(h, t["Wg"], t["Wu"], t["Wd"]), scale=t["s2"], w_pre=t["w3"])

    def conv(u, K):
        n = [2 * k for k in dims]
        at = torch.zeros((C, *n), dtype=u.dtype)
        at = torch.roll(torch.nn.functional.pad(K, (0, 1, 0, 1)), shifts=(-(dims[0] - 1), -(dims[1] - 1)), dims=(1, 2))
        y = torch.fft.irfftn(torch.fft.rfftn(u, s=n, dim=(2, 3)) * torch.fft.rfftn(at, dim=(1, 2)), s=n, dim=(2, 3))
        return y[:, :, :dims[0], :dims[1]]

    def ref(t):
        eps = 1e-6
        h = t["x"] * R.rms(t["x"], eps) * R.ch(t["w0"], t["x"])
        m = conv(torch.sigmoid(R.ch(t["al"], h) * h + R.ch(t["be"], h)) * h, t["K"])
        x, h = R.join(t["x"], m, t["gate"], t["s1"], t["w1"], t["w2"], keep=R.keep_mask(21, 0, 0.2, s), p=0.2, eps=eps)
        h = torch.where(R.keep_mask(21, 1000, 0.1, s), h / 0.9, torch.zeros_like(h))
        return R.join(x, R.ffn(h, t["Wg"], t["Wu"], t["Wd"], "silu"), scale=t["s2"], w_pre=t["w3"], eps=eps)

    a = {k: t.clone().requires_grad_() for k, t in v.items()}
    b = {k: t.double().cpu().requires_grad_() for k, t in v.items()}
    oa, ob = own(a), ref(b)
    ga = torch.autograd.grad(oa, list(a.values()), [dy, dh])
    gb = torch.autograd.grad(ob, list(b.values()), [dy.double().cpu(), dh.double().cpu()])
    for name, p, q in zip(["out", "h"] + list(v), list(oa) + list(ga), list(ob) + list(gb)):
        p, q = p.detach().double().cpu(), q.detach()
        assert float((p - q).abs().max() / q.abs().max()) <= 1e-4, name


@pytest.mark.parametrize("pre", [True, False], ids=["with-next-norm", "alone"])
def test_autograd_is_the_backward_call(H, pre):
    """Every differentiable call gives its backward's gradients, with inputs
    missing, gradients expanded or absent, and outputs unused."""
    t = _tensors(F32, 2, 24, (5, 7), 40, seed=9)
    x, m, gate, dout, dh, s, w1, w2, Wg, Wu, Wd, rng = t
    w2 = w2 if pre else None
    leaf = [v.clone().requires_grad_() if v is not None else None for v in (x, m, gate, s, w1, w2)]
    kw = dict(gate_act="silu", p=0.3, rng=rng)
    out, h = H.block_join(leaf[0], leaf[1], leaf[2], leaf[3], leaf[4], leaf[5], **kw)
    assert (h is None) == (not pre)
    (out * dout).sum().backward()                          # h unused
    want = H.block_join_bwd(x, m, dout, None, gate, s, w1, w2, **kw)
    for v, k in zip(leaf, ("dx", "dm", "dgate", "dscale", "dw_post", "dw_pre")):
        if v is not None and (k != "dw_pre" or pre):
            assert torch.equal(v.grad, want[k]), k
    a = x.clone().requires_grad_()
    H.block_join(a, m)[0].sum().backward()                 # an expanded gradient, every option absent
    assert torch.equal(a.grad, torch.ones_like(a))
    a, b = x.clone().requires_grad_(), w1.clone().requires_grad_()
    H.block_norm(a, b).sum().backward()
    da, db = H.block_norm_bwd(x, w1, torch.ones_like(x))
    assert torch.equal(a.grad, da) and torch.equal(b.grad, db)
    a = x.clone().requires_grad_()
    H.dropout(a, 0.3, rng).sum().backward()
    assert torch.equal(a.grad, H.dropout_bwd(torch.ones_like(x), 0.3, rng))
    a = x.clone().requires_grad_()
    H.dropout(a, 0.0, None).sum().backward()
    assert torch.equal(a.grad, torch.ones_like(a))
    ws = [v.clone().requires_grad_() for v in (x, Wg, Wu, Wd)]
    H.gated_ffn(*ws, act="gelu").backward(dout)
    for v, q in zip(ws, H.gated_ffn_bwd(x, Wg, Wu, Wd, dout, act="gelu")):
        assert torch.equal(v.grad, q)


@pytest.mark.parametrize("C,F,T", [(24, 520, 100), (128, 1032, 200), (100, 513, 77), (64, 512, 200), (40, 520, 16384),
                                   (128, 520, 16376)], ids=lambda v: str(v))
def test_ffn_both_forms_for_few_channels(H, C, F, T):
    """bf16 with at most 128 channels, on both sides of 512 hidden rows and 16384 positions."""
    check_ffn(H, *ffn_case(BF16, 1, C, F, (T,)), "silu")


def test_part_of_a_larger_gradient(H):
    """A gradient that arrives as an odd slice of another, off a 16-byte address."""
    x, Wg, Wu, Wd, _ = ffn_case(F32, 1, 3, 5, (7,))
    d = rand(gen(5), (2, 3, 7))
    ws = [t.clone().requires_grad_() for t in (x, Wg, Wu, Wd)]
    both = torch.cat([torch.zeros_like(x), H.gated_ffn(*ws)])
    both.backward(d)
    assert d[1:].data_ptr() % 16
    for v, q in zip(ws, H.gated_ffn_bwd(x, Wg, Wu, Wd, d[1:].clone())):
        assert torch.equal(v.grad, q)


def test_two_host_threads_on_one_stream(H):
    """Calls of two threads interleave on a stream: each thread has its own workspaces."""
    import threading
    sets = [_tensors(seed=s, dtype=F32) for s in (5, 6)]
    want = [_all_ops(H, t) for t in sets]
    got, gate = [None, None], threading.Barrier(2)

    def run(i):
        gate.wait()
        got[i] = [_all_ops(H, sets[i]) for _ in range(20)]

    ts = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for w, reps in zip(want, got):
        assert all(torch.equal(a, b) for r in reps for a, b in zip(w, r))


def test_workspaces_grow_and_are_kept(H):
    """Calls of growing and shrinking sizes share one workspace of the largest."""
    H.release_workspaces()
    for T in (70, 700, 90, 5000, 71):
        case = ffn_case(F32, 1, 24, 40, (T,))
        check_ffn(H, *case, "silu")
    held = [b.numel() for k, b in H._ws_cache.items() if k[0] == "gated_ffn_bwd"]
    assert held == [H.gated_ffn_bwd_workspace_bytes(1, 24, 40, (5000,), F32)]
    H.release_workspaces()


def test_weights_beyond_32_bits(H):
    """Weights of more than 2^31 elements: all hidden rows zero but the last 64,
    which alone then make the results; a sum over no positions clears as many."""
    C, F, k = 65536, 32840, 64
    x, Wg, Wu, Wd, dy = ffn_case(BF16, 1, C, k, (72,))
    big = [torch.zeros(s, dtype=BF16, device="cuda") for s in ((F, C), (F, C), (C, F))]
    big[0][-k:], big[1][-k:], big[2][:, -k:] = Wg, Wu, Wd
    y = H.gated_ffn_fwd(x, *big)
    dx, gg, gu, gd = H.gated_ffn_bwd(x, *big, dy)
    check_ffn(H, x, Wg, Wu, Wd, dy, "silu", fwd=y, bwd=(dx, gg[-k:], gu[-k:], gd[:, -k:]))
    few = x[:, :, :3].contiguous()
    check_ffn(H, few, Wg, Wu, Wd, few, "silu", fwd=H.gated_ffn_fwd(few, *big))
    for g in (gg, gu):
        assert not bool(g[:-k].any())
    del dx, gg, gu, gd, g
    H.release_workspaces()
    for g in H.gated_ffn_bwd(x[:0], *big, x[:0])[1:]:
        assert not bool(g[-1].any()) and not bool(g[0].any())


def test_offsets_beyond_32_bits(H):
    """Tensors of more than 2^31 elements (and bytes past 2^32): the last
    positions of each result against the 64-bit reference of those positions
    alone (they depend on no others; the parameter gradients, which do, are taken
    from the call on the part)."""
    n = (1 << 31) + 8 * 1001
    x = torch.empty(n, dtype=BF16, device="cuda")
    x.normal_(generator=gen(1))
    rng = rng_words(5, 7)
    y = H.dropout_fwd(x, 0.5, rng)
    part = rng.clone()
    part[1] += (n - 4096) // 4
    assert torch.equal(y[-4096:], H.dropout_fwd(x[-4096:].clone(), 0.5, part))
    del y
    C, L = 136, 1 << 23
    x = torch.empty(2, C, L, dtype=BF16, device="cuda")
    x.normal_(generator=gen(2))
    w = 1 + rand(gen(3), (C,), scale=0.1)

    def end(t, k=64):
        return t[1:, :, -k:].contiguous()

    h = H.block_norm_fwd(x, w)
    xt = end(x).double()
    ref = xt * R.rms(xt, 1e-6) * R.ch(w.double(), xt)
    check("h", end(h), ref, (R.HALF[BF16] + 2 * (C + 64) * U) * ref.abs())
    out, _ = H.block_join_fwd(x, h, x, w, w)
    g = H.block_join_bwd(x, h, x, None, x, w, w)
    d = {"x": end(x), "m": end(h), "gate": end(x), "scale": w, "w_post": w, "w_pre": None}
    gt = H.block_join_bwd(d["x"], d["m"], end(x), None, d["gate"], w, w)
    gt.update({k: end(g[k]) for k in ("dx", "dm", "dgate")})
    check_join(H, d, end(x), None, dict(gate_act="sigmoid", eps=1e-6, p=0.0), fwd=(end(out), None), bwd=gt)
    del g, gt, out
    for F, Cf in ((16, C), (40, 128)):                     # the tiles; one launch
        xf = x[:, :Cf].contiguous() if Cf != C else x
        Wg, Wu, Wd = (rand(gen(i), s, BF16, 0.1) for i, s in ((4, (F, Cf)), (5, (F, Cf)), (6, (Cf, F))))
        y = H.gated_ffn_fwd(xf, Wg, Wu, Wd)
        cut, dy = end(xf, 4096), end(xf, 4096)
        bwd = list(H.gated_ffn_bwd(cut, Wg, Wu, Wd, dy))
        if Cf == C:
            bwd[0] = end(H.gated_ffn_bwd(xf, Wg, Wu, Wd, xf)[0], 4096)
        check_ffn(H, cut, Wg, Wu, Wd, dy, "silu", fwd=end(y, 4096), bwd=bwd)
    H.release_workspaces()


def test_second_derivatives_are_refused(H):
    x = torch.ones(1, 3, 4, device="cuda", requires_grad=True)
    w = torch.ones(3, device="cuda", requires_grad=True)
    (gx,) = torch.autograd.grad(H.block_norm(x, w).sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(gx.sum(), [x])


def test_changed_dropout_words_are_noticed(H):
    """Words advanced in place between forward and backward would draw another
    mask: autograd refuses them."""
    x = torch.ones(1, 3, 8, device="cuda", requires_grad=True)
    rng = rng_words(1, 1)
    y = H.dropout(x, 0.5, rng)
    rng[1] += 2
    with pytest.raises(RuntimeError):
        y.sum().backward()
