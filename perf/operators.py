"""The operators of the residual block around the gated convolution, as cases
to measure: the norm ahead of a block (``norm``), the join behind it (``join``:
norm of the block's output, gate, residual scale, dropout, residual sum and the
next block's norm), dropout from a counter-based generator (``dropout``) and
the gated feed-forward block (``ffn``).

Tensors have the convolution's layout [B, C, n_0, .., n_{d-1}]; sums over
channels run per batch entry and grid position.  ``run`` computes an operator
in its plain form with elementary torch operations, or, with ``own`` set, with
the package's entry points.
"""
import math

import torch

own = False

SEED_WORDS = (0x243F6A8885A308D3, 12345)  # the generator's (seed, offset) the masks of a pass start from


# --------------------------------------------------------------------- cases

def _case(name, op, mode, dtype, B, C, dims, F=0, act="", p=0.0, post=True, pre=True):
    dims = tuple(dims) + (0,) * (3 - len(dims))
    c = {"op": op, "mode": mode, "dtype": dtype, "B": B, "C": C, "n0": dims[0], "n1": dims[1], "n2": dims[2],
         "F": F, "act": act, "p": p, "post": post, "pre": pre}
    return dict(c, name=name) if name else c


def listed():
    return [
        # One token of four streams through the end of a block: only latency counts.
        _case("join_token_bf16", "join", "fwd", "bf16", 4, 1024, (1,), act="silu"),
        # Inference on the 256x256 image workload of the benchmark.
        _case("join_fwd_256sq_f32", "join", "fwd", "f32", 8, 64, (256, 256), act="sigmoid"),
        # A training step of the 1024x1024 bf16 workload, with dropout: the largest tensors.
        _case("join_train_1024sq_bf16", "join", "train", "bf16", 2, 128, (1024, 1024), act="sigmoid", p=0.1),
        # A grid whose rows are neither even nor aligned, channels no multiple of eight.
        _case("join_train_odd_bf16", "join", "train", "bf16", 3, 100, (37, 53), act="silu", p=0.25),
        # The norm ahead of a wide block on long 1-D signals, in training.
        _case("norm_train_16k_bf16", "norm", "train", "bf16", 2, 1024, (16384,)),
        # The norm ahead of the 128^3 volume workload, at inference.
        _case("norm_fwd_128cube_f32", "norm", "fwd", "f32", 1, 32, (128, 128, 128)),
        # Dropout and its gradient on the 256x256 workload's activations.
        _case("dropout_train_256sq_f32", "dropout", "train", "f32", 8, 64, (256, 256), p=0.1),
        # Dropout of a small odd tensor.
        _case("dropout_fwd_odd_bf16", "dropout", "fwd", "bf16", 1, 7, (1001,), p=0.5),
        # One token of four streams through the feed-forward block: the weights are the traffic.
        _case("ffn_token_bf16", "ffn", "fwd", "bf16", 4, 1024, (1,), F=4096, act="silu"),
        # Inference on the 1024x1024 bf16 workload: few channels, two million positions.
        _case("ffn_fwd_1024sq_bf16", "ffn", "fwd", "bf16", 2, 128, (1024, 1024), F=512, act="silu"),
        # A training step of a wide block on long 1-D signals: the matrix cores are the bound.
        _case("ffn_train_16k_bf16", "ffn", "train", "bf16", 2, 1024, (16384,), F=4096, act="silu"),
        # A training step in fp32 at sizes that fit no tile.
        _case("ffn_train_odd_f32", "ffn", "train", "f32", 3, 100, (37, 53), F=333, act="gelu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["join", "join", "norm", "dropout", "ffn", "ffn"])
    mode = rng.choice(["fwd", "train"])
    dtype = rng.choice(["f32", "bf16"])
    d = rng.choice([1, 1, 2, 3])
    B = _log(rng, 1, 16)
    even = rng.random() < 0.5  # half of the cases on sizes that divide well

    def size(lo, hi):
        v = _log(rng, lo, hi)
        return max(8, v // 8 * 8) if even and hi >= 8 and v > 4 else v

    if op == "ffn":
        C, F = size(8, 1024), size(16, 4096)
        # positions: at most the largest listed case's products, and 2^29 hidden values
        most = min(2 ** 21, 1024 * 4096 * 32768 // (C * F), 2 ** 29 // F)
    else:
        C, F = size(1, 1536), 0
        most = 2 ** 27 // C
    L = _log(rng, 1, max(1, most // B))
    dims = []
    for k in range(d - 1):
        dims.append(_log(rng, 1, max(1, min(512, L))))
        L = max(1, L // dims[-1])
    dims.append(max(8, L // 8 * 8) if even and L > 8 else L)
    p = rng.choice([0.0, 0.1, 0.3]) if op == "join" else (rng.choice([0.1, 0.5, 0.85]) if op == "dropout" else 0.0)
    act = rng.choice(["silu", "gelu"]) if op == "ffn" else (rng.choice(["none", "sigmoid", "silu"]) if op == "join" else "")
    post = rng.random() < 0.8 if op == "join" else True
    pre = rng.random() < 0.8 if op == "join" else True
    return _case("", op, mode, dtype, B, C, dims, F=F, act=act, p=p, post=post, pre=pre)


def _dims(case):
    return tuple(n for n in (case["n0"], case["n1"], case["n2"]) if n)


def work(case):
    B, C, F, L = case["B"], case["C"], case["F"], math.prod(_dims(case))
    es = 4 if case["dtype"] == "f32" else 2
    n, train, op = B * C * L, case["mode"] == "train", case["op"]
    if op == "norm":     # x -> h; then dh -> dx, dw
        return {"bytes": es * n * (4 if train else 2) + 4 * C * (2 if train else 1), "flops": n * (12 if train else 4)}
    if op == "join":     # x, m, gate -> out[, h]; then dout[, dh] -> dx, dm, dgate
        t = 4 + case["pre"] + ((4 + case["pre"]) if train else 0)
        return {"bytes": es * n * t + 4 * C * (6 if train else 3), "flops": n * (50 if train else 15)}
    if op == "dropout":  # x -> y; then dy -> dx
        return {"bytes": es * n * (4 if train else 2), "flops": n * (2 if train else 1)}
    if train:            # x, weights, dy -> y, dx and the weights' gradients
        return {"bytes": es * (4 * n + 6 * C * F), "flops": 18 * C * F * B * L}
    return {"bytes": es * (2 * n + 3 * C * F), "flops": 6 * C * F * B * L}


# -------------------------------------------------------------------- inputs

def _inputs(case, seed):
    """Activations and gradients of unit size, gains near one, residual scales
    and weights as at the start of training."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    B, C, F, dims = case["B"], case["C"], case["F"], _dims(case)

    def act():
        return torch.randn((B, C) + dims, generator=g, device="cuda", dtype=dt)

    def gain():
        return 1.0 + 0.1 * torch.randn(C, generator=g, device="cuda")

    train, op = case["mode"] == "train", case["op"]
    s = {"x": act()}
    if op == "norm":
        s["w"] = gain()
        if train:
            s["dh"] = act()
    elif op == "join":
        s.update(m=act(), gate=act(), scale=0.05 + torch.rand(C, generator=g, device="cuda"))
        s["w_post"] = gain() if case["post"] else None
        s["w_pre"] = gain() if case["pre"] else None
        if train:
            s["dout"] = act()
            s["dh"] = act() if case["pre"] else None
    elif op == "ffn":
        s["Wg"] = torch.randn((F, C), generator=g, device="cuda", dtype=dt) * C ** -0.5
        s["Wu"] = torch.randn((F, C), generator=g, device="cuda", dtype=dt) * C ** -0.5
        s["Wd"] = torch.randn((C, F), generator=g, device="cuda", dtype=dt) * F ** -0.5
        if train:
            s["dy"] = act()
    elif train:
        s["dy"] = act()
    s["rng"] = torch.tensor([(SEED_WORDS[0] + seed) % 2 ** 63, SEED_WORDS[1]], dtype=torch.int64, device="cuda")
    s["case"] = case
    return s


def prepare(case, seed):
    return _inputs(case, seed)


EPS = 1e-6


# --------------------------------------------------------------- plain forms

def _mul32(a, b):
    """(high, low) 32-bit words of the product of 32-bit words held in int64;
    b is a Python integer.  Two partial products, each below 2^48."""
    p0, p1 = a * (b & 0xFFFF), a * (b >> 16)
    mid = p1 + (p0 >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (p0 & 0xFFFF)


def _random_words(rng, n):
    """n words of the counter-based generator (Philox 4x32 with 10 rounds; Salmon
    et al., "Parallel random numbers: as easy as 1, 2, 3", 2011): element e
    takes word e % 4 of the block at counter offset + e // 4."""
    k0, k1 = rng[0] & 0xFFFFFFFF, (rng[0] >> 32) & 0xFFFFFFFF
    q = torch.arange((n + 3) // 4, device=rng.device, dtype=torch.int64) + rng[1]
    c0, c1 = q & 0xFFFFFFFF, (q >> 32) & 0xFFFFFFFF
    c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0)
    for _ in range(10):
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack((c0, c1, c2, c3), dim=1).reshape(-1)[:n]


def _keep(rng, p, shape):
    """The factor of every element: 0 where dropped, 1 / (1 - p) where kept."""
    n = math.prod(shape)
    return (_random_words(rng, n) >= int(p * 2 ** 32)).to(torch.float32).mul_(1.0 / (1.0 - p)).reshape(shape)


def _ch(v, like):
    return v.reshape((1, -1) + (1,) * (like.dim() - 2))


def _sum_ch(t):
    """Sum over batch and positions, per channel."""
    return t.sum(dim=[0] + list(range(2, t.dim())))


def _rinv(t):
    return torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS)


def _norm_grad(t, r, w, dh):
    """Gradients of t r w to t and w (r = 1 / rms over the channels)."""
    dw = _sum_ch(dh * t * r)
    dn = dh * _ch(w, t)
    return r * dn - t * (r * r * r) * (dn * t).mean(dim=1, keepdim=True), dw


def _act(name, v):
    """Activation and its derivative."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
        return v * cdf, cdf + v * torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))
    s = torch.sigmoid(v)
    if name == "sigmoid":
        return s, s * (1.0 - s)
    return v * s, s * (1.0 + v * (1.0 - s))


def _plain_norm(s):
    dt, x = s["x"].dtype, s["x"].float()
    r = _rinv(x)
    out = {"h": (x * r * _ch(s["w"], x)).to(dt)}
    if "dh" in s:
        dx, dw = _norm_grad(x, r, s["w"], s["dh"].float())
        out.update(dx=dx.to(dt), dw=dw)
    return out


def _plain_join(s):
    c, dt = s["case"], s["x"].dtype
    x, m = s["x"].float(), s["m"].float()
    a, da = _act(c["act"], s["gate"].float())
    r = _rinv(m) if c["post"] else None
    n = m * r * _ch(s["w_post"], m) if c["post"] else m
    sc = _ch(s["scale"], m)
    keep = _keep(s["rng"], c["p"], m.shape) if c["p"] else None
    b = sc * a * n
    o = x + (b * keep if c["p"] else b)
    res = {"out": o.to(dt)}
    if c["pre"]:
        ro = _rinv(o)
        res["h"] = (o * ro * _ch(s["w_pre"], o)).to(dt)
    if "dout" in s:
        do = s["dout"].float()
        if c["pre"]:
            dn, res["dw_pre"] = _norm_grad(o, ro, s["w_pre"], s["dh"].float())
            do = do + dn
        res["dx"] = do.to(dt)
        db = do * keep if c["p"] else do
        res["dscale"] = _sum_ch(db * a * n)
        res["dgate"] = (db * sc * n * da).to(dt)
        dn = db * sc * a
        if c["post"]:
            dn, res["dw_post"] = _norm_grad(m, r, s["w_post"], dn)
        res["dm"] = dn.to(dt)
    return res


def _plain_dropout(s):
    c, dt = s["case"], s["x"].dtype
    keep = _keep(s["rng"], c["p"], s["x"].shape)
    out = {"y": (s["x"].float() * keep).to(dt)}
    if "dy" in s:
        out["dx"] = (s["dy"].float() * keep).to(dt)
    return out


def _plain_ffn(s):
    c, dt = s["case"], s["x"].dtype
    x = s["x"].float().flatten(2)
    Wg, Wu, Wd = s["Wg"].float(), s["Wu"].float(), s["Wd"].float()
    train = "dy" in s
    y, dx = torch.empty_like(x), torch.empty_like(x) if train else None
    dWg, dWu, dWd = (torch.zeros_like(w) for w in (Wg, Wu, Wd)) if train else (None, None, None)
    for b in range(c["B"]):
        g, u = Wg @ x[b], Wu @ x[b]
        a, da = _act(c["act"], g)
        h = a * u
        y[b] = Wd @ h
        if train:
            dy = s["dy"][b].float().flatten(1)
            dh = Wd.t() @ dy
            du, dg = dh * a, dh * u * da
            dx[b] = Wg.t() @ dg + Wu.t() @ du
            xt = x[b].t()
            dWg += dg @ xt
            dWu += du @ xt
            dWd += dy @ h.t()
    out = {"y": y.view(s["x"].shape).to(dt)}
    if train:
        out.update(dx=dx.view(s["x"].shape).to(dt), dWg=dWg.to(dt), dWu=dWu.to(dt), dWd=dWd.to(dt))
    return out


# ------------------------------------------------------ the package's operators

def _own(s):
    import dimensional_fft_long_amd as H

    c = s["case"]
    if c["op"] == "norm":
        out = {"h": H.block_norm_fwd(s["x"], s["w"], eps=EPS)}
        if "dh" in s:
            out["dx"], out["dw"] = H.block_norm_bwd(s["x"], s["w"], s["dh"], eps=EPS)
        return out
    if c["op"] == "join":
        kw = dict(gate=s["gate"], scale=s["scale"], w_post=s["w_post"], w_pre=s["w_pre"], gate_act=c["act"], eps=EPS,
                  p=c["p"], rng=s["rng"] if c["p"] else None)
        o, h = H.block_join_fwd(s["x"], s["m"], **kw)
        out = {"out": o}
        if c["pre"]:
            out["h"] = h
        if "dout" in s:
            g = H.block_join_bwd(s["x"], s["m"], s["dout"], s["dh"], **kw)
            out.update({k: v for k, v in g.items() if v is not None})
        return out
    if c["op"] == "dropout":
        out = {"y": H.dropout_fwd(s["x"], c["p"], s["rng"])}
        if "dy" in s:
            out["dx"] = H.dropout_bwd(s["dy"], c["p"], s["rng"])
        return out
    out = {"y": H.gated_ffn_fwd(s["x"], s["Wg"], s["Wu"], s["Wd"], act=c["act"])}
    if "dy" in s:
        out["dx"], out["dWg"], out["dWu"], out["dWd"] = H.gated_ffn_bwd(s["x"], s["Wg"], s["Wu"], s["Wd"], s["dy"],
                                                                       act=c["act"])
    return out


ORDER = ("y", "h", "out", "dx", "dm", "dgate", "dscale", "dw", "dw_post", "dw_pre", "dWg", "dWu", "dWd")


def run(state):
    res = _own(state) if own else {"norm": _plain_norm, "join": _plain_join, "dropout": _plain_dropout,
                                   "ffn": _plain_ffn}[state["case"]["op"]](state)
    return {k: res[k] for k in ORDER if k in res}


# -------------------------------------------------- the definition in 64 bits

def _philox64(rng, n):
    """The same generator from its definition, on full 64-bit products."""
    key, off = int(rng[0]), int(rng[1])
    k = [key & 0xFFFFFFFF, key >> 32 & 0xFFFFFFFF]
    i = torch.arange(n, device=rng.device, dtype=torch.int64)
    ctr = (i >> 2) + off
    w = [ctr & 0xFFFFFFFF, ctr >> 32 & 0xFFFFFFFF, torch.zeros_like(ctr), torch.zeros_like(ctr)]

    def words(mult, v):
        high = (((v >> 16) * mult) + (((v & 0xFFFF) * mult) >> 16)) >> 16
        return high & 0xFFFFFFFF, (v * mult) & 0xFFFFFFFF  # the product modulo 2^64 keeps its low word

    for _ in range(10):
        ha, la = words(0xD2511F53, w[0])
        hb, lb = words(0xCD9E8D57, w[2])
        w = [hb ^ w[1] ^ k[0], lb, ha ^ w[3] ^ k[1], la]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    lane = i & 3
    return torch.where(lane < 2, torch.where(lane == 0, w[0], w[1]), torch.where(lane == 2, w[2], w[3]))


def _dropped64(t, rng, p):
    keep = torch.cat([_philox64(torch.stack((rng[0], rng[1] + a // 4)), min(2 ** 24, t.numel() - a)) >= math.floor(p * 2 ** 32)
                      for a in range(0, t.numel(), 2 ** 24)]).reshape(t.shape)
    return torch.where(keep, t / (1.0 - p), torch.zeros((), dtype=t.dtype, device=t.device))


def exact(case, seed):
    s = _inputs(case, seed)
    d = {k: v.double().detach() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    train, op = case["mode"] == "train", case["op"]

    def leaf(*names):
        for k in names:
            if k in d:
                d[k].requires_grad_(train)

    def rms_normed(t, w):
        ms = t.square().sum(1, keepdim=True) / t.shape[1]
        return t / torch.sqrt(ms + EPS) * w.view((-1,) + (1,) * (t.dim() - 2))

    def activation(v):
        if case["act"] == "none":
            return v
        if case["act"] == "gelu":
            return v * torch.special.ndtr(v)
        return 1 / (1 + torch.exp(-v)) * (v if case["act"] == "silu" else 1)

    def grads(pairs, names):
        names = [k for k in names if k in d]
        for k, v in zip(names, torch.autograd.grad([a for a, _ in pairs], [d[k] for k in names], [b for _, b in pairs])):
            res["d" + k] = v

    res = {}
    if op == "norm":
        leaf("x", "w")
        res["h"] = rms_normed(d["x"], d["w"])
        if train:
            grads([(res["h"], d["dh"])], ["x", "w"])
    elif op == "join":
        leaf("x", "m", "gate", "scale", "w_post", "w_pre")
        n = rms_normed(d["m"], d["w_post"]) if case["post"] else d["m"]
        b = d["scale"].view((-1,) + (1,) * (n.dim() - 2)) * activation(d["gate"]) * n
        res["out"] = d["x"] + (_dropped64(b, s["rng"], case["p"]) if case["p"] else b)
        if case["pre"]:
            res["h"] = rms_normed(res["out"], d["w_pre"])
        if train:
            grads([(res["out"], d["dout"])] + ([(res["h"], d["dh"])] if case["pre"] else []),
                  ["x", "m", "gate", "scale", "w_post", "w_pre"])
    elif op == "dropout":
        res["y"] = _dropped64(d["x"], s["rng"], case["p"])
        if train:
            res["dx"] = _dropped64(d["dy"], s["rng"], case["p"])
    else:
        leaf("x", "Wg", "Wu", "Wd")
        parts = []
        tot = {}
        for b in range(case["B"]):  # one batch entry at a time bounds the memory
            xb = d["x"].detach()[b].flatten(1).requires_grad_(train)
            yb = d["Wd"] @ (activation(d["Wg"] @ xb) * (d["Wu"] @ xb))
            parts.append(yb.detach())
            if train:
                for k, v in zip(("x", "Wg", "Wu", "Wd"),
                                torch.autograd.grad(yb, [xb, d["Wg"], d["Wu"], d["Wd"]], d["dy"][b].flatten(1))):
                    tot[k] = tot.get(k, []) + [v] if k == "x" else (tot[k] + v if k in tot else v)
        res["y"] = torch.stack(parts).view(d["x"].shape)
        if train:
            res["dx"] = torch.stack(tot["x"]).view(d["x"].shape)
            res.update({"d" + k: tot[k] for k in ("Wg", "Wu", "Wd")})
    return {k: res[k].detach() for k in ORDER if k in res}
