"""The residual block's entry points on the host: every refusal returns before
anything is launched (no GPU needed), sizes of the workspaces, and the
generator's published test vectors against the tests' own reference."""
import ctypes
import math
import os

import pytest
import torch

from block_ref import philox_words


@pytest.fixture(scope="module")
def H():
    import dimensional_fft_long_amd as H

    if not os.path.exists(H.LIB_PATH):
        from dimensional_fft_long_amd import build

        build.build()
    H.get_lib()
    return H


FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10001)
AT4 = ctypes.c_void_p(0x10004)


def _dims(*v):
    return (ctypes.c_int64 * len(v))(*v)


SHAPES = [  # d, dims, code
    (0, (4,), 2), (4, (1, 1, 1, 1), 2), (2, (4, -1), 1), (1, (1 << 61,), 2), (3, (1 << 31, 1 << 31, 1 << 31), 2),
]


def test_norm_refusals(H):
    lib = H.get_lib()
    f = lambda x=FAKE, w=FAKE, h=FAKE, B=1, C=4, d=1, dims=_dims(5), dt=0, eps=1e-6: \
        lib.hyenand_block_norm_fwd(x, w, h, B, C, d, dims, dt, eps, None)
    b = lambda x=FAKE, w=FAKE, dh=FAKE, dx=FAKE, dw=FAKE, B=1, C=4, d=1, dims=_dims(5), dt=0, eps=1e-6, ws=FAKE, \
        nb=1 << 30: lib.hyenand_block_norm_bwd(x, w, dh, dx, dw, B, C, d, dims, dt, eps, ws, nb, None)
    for k in ("x", "w", "h"):
        assert f(**{k: None}) == 1 and f(**{k: ODD}) == 1, k
    for k in ("x", "w", "dh", "dx", "dw"):
        assert b(**{k: None}) == 1 and b(**{k: ODD}) == 1, k
    for g in (f, b):
        assert g(B=-1) == 1 and g(C=-1) == 1 and g(dt=2) == 1 and g(dims=None) == 1 and g(C=8193) == 2
        for eps in (0.0, -1e-6, 1e-40, math.inf, math.nan):
            assert g(eps=eps) == 1
        for d, dims, code in SHAPES:
            assert g(d=d, dims=_dims(*dims)) == code, dims
    assert f(dt=1, x=ctypes.c_void_p(0x10001)) == 1
    need = lib.hyenand_block_norm_bwd_workspace_bytes(1, 4, 1, _dims(5), 0)
    assert need > 0
    assert b(ws=None) == 3 and b(nb=need - 1) == 3 and b(ws=ODD) == 1
    # empty calls: nothing to write forward; backward without channels neither
    assert f(x=None, h=None, w=None, B=0) == 0 and f(x=None, C=0) == 0 and f(x=None, dims=_dims(0)) == 0
    assert b(x=None, dw=None, C=0) == 0
    assert lib.hyenand_block_norm_bwd_workspace_bytes(0, 4, 1, _dims(5), 0) == 0
    assert lib.hyenand_block_norm_bwd_workspace_bytes(1, 8193, 1, _dims(5), 0) == 0


def _join(H, **kw):
    v = dict(gate=0x10000, scale=0x10000, w_post=0x10000, w_pre=0x10000, rng=0x10000, p=0.1, eps=1e-6, gate_act=1)
    v.update(kw)
    return H.block._Join(*[v[k] for k, _ in H.block._Join._fields_])


def _grads(H, **kw):
    v = {k: kw.get(k, 0x10000) for k, _ in H.block._JoinGrads._fields_}
    return H.block._JoinGrads(*[v[k] for k, _ in H.block._JoinGrads._fields_])


def test_join_refusals(H):
    lib = H.get_lib()

    def f(x=FAKE, m=FAKE, out=FAKE, h=FAKE, B=1, C=4, d=1, dims=_dims(5), dt=0, j=None, null=False, **kw):
        j = _join(H, **kw)
        return lib.hyenand_block_join_fwd(x, m, None if null else ctypes.byref(j), out, h, B, C, d, dims, dt, None)

    def b(x=FAKE, m=FAKE, dout=FAKE, dh=FAKE, B=1, C=4, d=1, dims=_dims(5), dt=0, ws=FAKE, nb=1 << 30, g=None,
          nog=False, null=False, **kw):
        j, g = _join(H, **kw), g or _grads(H)
        return lib.hyenand_block_join_bwd(x, m, None if null else ctypes.byref(j), dout, dh,
                                          None if nog else ctypes.byref(g), B, C, d, dims, dt, ws, nb, None)

    for k in ("x", "m", "out"):
        assert f(**{k: None}) == 1 and f(**{k: ODD}) == 1, k
    for k in ("x", "m"):
        assert b(**{k: None}) == 1 and b(**{k: ODD}) == 1, k
    assert f(h=None) == 1 and f(w_pre=None) == 1          # h goes with w_pre
    assert b(dout=ODD) == 1 and b(dh=ODD) == 1
    for q in (f, b):
        assert q(null=True) == 1 and q(B=-1) == 1 and q(C=-2) == 1 and q(dt=9) == 1 and q(C=8193) == 2
        assert q(dims=None) == 1
        for k in ("gate", "scale", "w_post", "w_pre"):
            assert q(**{k: 0x10001}) == 1, k
        for act in (-1, 3, 7):
            assert q(gate_act=act) == 1
        for eps in (0.0, 1e-40, math.nan, math.inf):
            assert q(eps=eps) == 1
        for p in (-0.1, 1.0, 2.0, math.nan):
            assert q(p=p) == 1
        assert q(rng=None) == 1 and q(rng=0x10004) == 1
        for d, dims, code in SHAPES:
            assert q(d=d, dims=_dims(*dims)) == code, dims
    # a gradient exactly where the input is
    assert b(nog=True) == 1
    for k in ("dx", "dm", "dgate", "dscale", "dw_post", "dw_pre"):
        assert b(g=_grads(H, **{k: None})) == 1 and b(g=_grads(H, **{k: 0x10001})) == 1, k
    assert b(gate=None) == 1 and b(scale=None) == 1 and b(w_post=None) == 1
    assert b(w_pre=None, g=_grads(H, dw_pre=None)) == 1   # dh without w_pre
    need = lib.hyenand_block_join_bwd_workspace_bytes(1, 4, 1, _dims(5), 0)
    assert b(ws=None) == 3 and b(nb=need - 1) == 3 and b(ws=ODD) == 1
    assert f(x=None, m=None, out=None, h=None, B=0) == 0 and f(x=None, C=0) == 0 and b(x=None, C=0) == 0


def test_dropout_refusals(H):
    lib = H.get_lib()
    f = lambda x=FAKE, y=FAKE, n=8, dt=0, p=0.5, r=FAKE: lib.hyenand_dropout(x, y, n, dt, p, r, None)
    assert f(x=None) == 1 and f(y=None) == 1 and f(x=ODD) == 1 and f(y=ODD) == 1 and f(n=-1) == 1 and f(dt=2) == 1
    for p in (-0.5, 1.0, 1.5, math.nan):
        assert f(p=p) == 1
    assert f(r=None) == 1 and f(r=AT4) == 1
    assert f(n=(1 << 38) + 1) == 2
    assert f(x=None, y=None, n=0) == 0


def test_ffn_refusals(H):
    lib = H.get_lib()
    names = ("x", "Wg", "Wu", "Wd", "y")
    bnames = ("x", "Wg", "Wu", "Wd", "dy", "dx", "dWg", "dWu", "dWd")

    def f(B=1, C=8, F=16, d=1, dims=_dims(5), dt=0, act=2, ws=FAKE, nb=1 << 40, **kw):
        return lib.hyenand_gated_ffn_fwd(*[kw.get(k, FAKE) for k in names], B, C, F, d, dims, dt, act, ws, nb, None)

    def b(B=1, C=8, F=16, d=1, dims=_dims(5), dt=0, act=2, ws=FAKE, nb=1 << 40, **kw):
        return lib.hyenand_gated_ffn_bwd(*[kw.get(k, FAKE) for k in bnames], B, C, F, d, dims, dt, act, ws, nb, None)

    for q, ks in ((f, names), (b, bnames)):
        for k in ks:
            assert q(**{k: None}) == 1 and q(**{k: ODD}) == 1 and q(**{k: AT4}) == 1, k
        assert q(B=-1) == 1 and q(C=-1) == 1 and q(F=0) == 1 and q(F=-4) == 1 and q(dt=4) == 1 and q(dims=None) == 1
        for act in (0, 4, -1):
            assert q(act=act) == 1
        assert q(C=65537) == 2 and q(F=65537) == 2
        assert q(dims=_dims((1 << 30) + 1)) == 2 and q(B=2, dims=_dims((1 << 29) + 1)) == 2
        for d, dims, code in SHAPES:
            assert q(d=d, dims=_dims(*dims)) == code, dims
    for q, size in ((f, lib.hyenand_gated_ffn_workspace_bytes), (b, lib.hyenand_gated_ffn_bwd_workspace_bytes)):
        need = size(2, 24, 48, 2, _dims(5, 7), 0)
        assert need > 0
        kw = dict(B=2, C=24, F=48, d=2, dims=_dims(5, 7))
        assert q(ws=None, **kw) == 3 and q(nb=need - 1, **kw) == 3 and q(ws=ctypes.c_void_p(0x10010), **kw) == 1
        assert size(2, 24, 0, 2, _dims(5, 7), 0) == 0 and size(0, 24, 48, 2, _dims(5, 7), 0) == 0
    assert f(x=None, y=None, B=0) == 0 and f(x=None, C=0) == 0 and f(x=None, dims=_dims(0)) == 0
    assert b(x=None, dWg=None, C=0) == 0


def test_python_checks(H):
    """The binding's own checks, before any call (host and meta tensors)."""
    x = torch.zeros(2, 3, 4)
    with pytest.raises(TypeError):
        H.block_norm_fwd(x, torch.zeros(3))
    with pytest.raises(TypeError):
        H.block_join_fwd(x, x)
    with pytest.raises(TypeError):
        H.dropout_fwd(x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        H.gated_ffn_fwd(x, x, x, x)
    blk = H.block
    with pytest.raises(ValueError):
        blk._rng(None, 1.0, x.device)
    with pytest.raises(TypeError):
        blk._rng(torch.zeros(2), 0.1, x.device)
    with pytest.raises(TypeError):
        blk._rng(torch.zeros(3, dtype=torch.int64), 0.1, x.device)
    assert blk._rng(None, 0.0, x.device) == 0.0
    with pytest.raises(TypeError):
        blk._channel(torch.zeros(4), "w", x)
    with pytest.raises(TypeError):
        blk._channel(torch.zeros(3, dtype=torch.float64), "w", x)
    with pytest.raises(TypeError):
        blk._like(x.double(), "m", x)
    with pytest.raises(TypeError):
        blk._like(torch.zeros(2, 3, 8)[..., ::2], "m", x)
    with pytest.raises(ValueError):
        blk._like(torch.zeros(2, 3, 5), "m", x)
    with pytest.raises(ValueError):
        blk._act("relu", ("silu",))


def test_generator_reference_against_published_vectors():
    """Philox 4x32-10 of the counter words 0 and all ones (the generator's
    published known answers; the second has counter words 2 and 3 set, which the
    reference takes as an option)."""
    assert philox_words(0, 0, 4).tolist() == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    got = philox_words(0xFFFFFFFFFFFFFFFF, 0xFFFFFFFFFFFFFFFF, 4, high=(0xFFFFFFFF, 0xFFFFFFFF)).tolist()
    assert got == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
