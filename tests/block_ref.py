"""Plain 64-bit references of the residual block's operators for the tests, with
the magnitudes that their error bounds are counted in.  Not the library's code:
gradients come from torch's differentiation of the forward formulas."""
import math

import numpy as np
import torch

U = 2.0 ** -24          # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def philox_words(seed, offset, n, high=(0, 0)):
    """n words of Philox 4x32-10 at counters offset, offset + 1, ..: uint32."""
    nb = (n + 3) // 4
    ctr = (np.arange(nb, dtype=np.uint64) + np.uint64(offset & 0xFFFFFFFFFFFFFFFF))
    m32 = np.uint64(0xFFFFFFFF)
    c = [ctr & m32, ctr >> np.uint64(32), np.full(nb, high[0], np.uint64), np.full(nb, high[1], np.uint64)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & m32, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & m32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).reshape(-1)[:n]


def keep_mask(seed, offset, p, shape):
    n = math.prod(shape)
    return torch.from_numpy(philox_words(seed, offset, n) >= int(p * 2 ** 32)).reshape(tuple(shape))


def ch(v, like):
    return v.reshape((1, -1) + (1,) * (like.dim() - 2))


def act(name, v):
    if name == "none":
        return v
    if name == "gelu":
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
    return torch.sigmoid(v) * (v if name == "silu" else 1.0)


def rms(t, eps):
    return torch.rsqrt(t.square().mean(1, keepdim=True) + eps)


def join(x, m, gate=None, scale=None, w_post=None, w_pre=None, gate_act="sigmoid", eps=1e-6, keep=None, p=0.0):
    """(out, h) in the inputs' own precision (64-bit inputs here)."""
    n = m * rms(m, eps) * ch(w_post, m) if w_post is not None else m
    b = n * (act(gate_act, gate) if gate is not None else 1.0) * (ch(scale, m) if scale is not None else 1.0)
    if keep is not None:
        b = torch.where(keep, b / (1.0 - p), torch.zeros_like(b))
    out = x + b
    return out, (out * rms(out, eps) * ch(w_pre, out) if w_pre is not None else None)


def ffn(x, Wg, Wu, Wd, name):
    xf = x.flatten(2)
    return torch.stack([Wd @ (act(name, Wg @ v) * (Wu @ v)) for v in xf]).reshape(x.shape)
