"""The training and serving operators around the fused linear layer, as they are measured.

Six operators of one transformer feed-forward sublayer, forward and backward:

* ``dropout``       y = residual + keep * x / (1 - p), the keep decisions from Philox4x32-10 on the element's
                    place, so that no mask is stored
* ``norm``          s = residual + dropout(x), z = layer norm of s, with the row statistics kept
* ``norm_back``     the gradients of ``norm``: of s (the residual's), of x, of gamma and of beta
* ``glu``           h = act(x Wg^T) * (x Wu^T) from the stacked weight [Wg; Wu]; when ``aux`` the two
                    projections are kept for the backward pass
* ``glu_back``      dh = dy Wd, then the gradients of the two projections
* ``weight_grad``   dW = dy^T x, added to an earlier gradient when ``accumulate``

``own`` says whose code ``run`` calls: elementary torch operations, or this repository's kernels.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}
_EPS = 1e-5


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the activations of a short prompt in a small model's embedding dropout: latency counts
        dict(name="dropout_small", op="dropout", M=64, N=768, x="f16", s="f16", residual=False, p=0.1),
        # the end of a sublayer of a large training batch: dropout and the residual add in one pass
        dict(name="dropout_residual", op="dropout", M=8192, N=4096, x="bf16", s="bf16", residual=True, p=0.1),
        # a few rows of an odd width, fp32 residual stream: fine tuning on short texts
        dict(name="norm_few_odd_rows", op="norm", M=33, N=1001, x="f16", s="f32", z="f16", param="f32", residual=True, p=0.1),
        # post-norm sublayer end of a large training batch
        dict(name="norm_batch", op="norm", M=8192, N=4096, x="bf16", s="bf16", z="bf16", param="bf16", residual=True, p=0.1),
        # its backward pass in a small model whose residual stream is fp32
        dict(name="norm_back_narrow", op="norm_back", M=2048, N=768, x="bf16", s="f32", z="bf16", param="f32", stream=False, p=0.1),
        # the same at the large batch, pre-norm: a gradient also arrives on the residual stream
        dict(name="norm_back_batch", op="norm_back", M=8192, N=4096, x="bf16", s="bf16", z="bf16", param="bf16", stream=True, p=0.1),
        # one new token of one sequence being answered: the weights are read once
        dict(name="swiglu_one_token", op="glu", act="swiglu", M=1, N=8192, K=4096, t="bf16", aux=False),
        # training forward of the GeGLU block of the repository's MLP width
        dict(name="geglu_train", op="glu", act="geglu", M=8192, N=2048, K=768, t="bf16", aux=True),
        # backward through the block on a ragged batch of packed texts
        dict(name="geglu_back_ragged", op="glu_back", act="geglu", M=2047, N=1000, K=768, t="f16"),
        # backward through the block of a large layer
        dict(name="swiglu_back_large", op="glu_back", act="swiglu", M=4096, N=8192, K=4096, t="bf16"),
        # the gradient of a small weight over many tokens, added to the fp32 gradient of earlier micro-batches
        dict(name="weight_grad_small", op="weight_grad", tokens=8191, out=768, into=768, t="bf16", g="f32", accumulate=True),
        # the gradient of a large layer's stacked gate and up weight
        dict(name="weight_grad_large", op="weight_grad", tokens=4096, out=8192, into=4096, t="bf16", g="bf16", accumulate=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["dropout", "norm", "norm_back", "glu", "glu_back", "weight_grad"])
    if op in ("dropout", "norm", "norm_back"):
        N = _log(rng, 64, 16384)
        M = _log(rng, 1, max(1, min(8192, (8192 * 4096) // N)))
        if rng.random() < 0.6:
            N = max(8, N // 8 * 8)  # most models have aligned widths, and every fifth drawn one is any number
        x = rng.choice(["f16", "bf16", "f32"])
        s = rng.choice([x, "f32"])
        p = rng.choice([0.0, 0.05, 0.1, 0.5])
        if op == "dropout":
            return dict(op=op, M=M, N=N, x=x, s=s, residual=rng.random() < 0.5, p=p)
        z, param = rng.choice([x, s]), rng.choice([x, "f32"])
        if op == "norm":
            return dict(op=op, M=M, N=N, x=x, s=s, z=z, param=param, residual=rng.random() < 0.8, p=p)
        return dict(op=op, M=M, N=N, x=x, s=s, z=z, param=param, stream=rng.random() < 0.5, p=p)
    t = rng.choice(["f16", "bf16"])
    if op == "weight_grad":
        out, into = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 512)
        tokens = _log(rng, 1, max(1, min(16384, (4096 * 8192 * 4096) // (out * into))))
        return dict(op=op, tokens=tokens, out=out, into=into, t=t, g=rng.choice([t, "f32"]), accumulate=rng.random() < 0.5)
    N, K = 8 * _log(rng, 16, 1024), 8 * _log(rng, 16, 512)
    M = _log(rng, 1, 8192)
    M = max(1, min(M, (4096 * 8192 * 4096) // (2 * N * K)))
    act = rng.choice(["swiglu", "geglu"])
    if op == "glu_back":
        return dict(op=op, act=act, M=M, N=N, K=K, t=t)
    aux = rng.random() < 0.5 or act == "geglu"
    return dict(op=op, act=act, M=M, N=N, K=K, t=t, aux=aux)


def work(case):
    op = case["op"]
    if op == "weight_grad":
        r, o, i, e, g = case["tokens"], case["out"], case["into"], _BYTES[case["t"]], _BYTES[case["g"]]
        return {"bytes": r * (o + i) * e + o * i * g * (2 if case["accumulate"] else 1), "flops": 2 * r * o * i}
    M, N = case["M"], case["N"]
    if op == "glu":
        K, e = case["K"], _BYTES[case["t"]]
        return {"bytes": e * (M * K + 2 * N * K + M * N * (3 if case["aux"] else 1)), "flops": 4 * M * N * K}
    if op == "glu_back":
        K, e = case["K"], _BYTES[case["t"]]
        return {"bytes": e * (M * K + N * K + 4 * M * N), "flops": 2 * M * N * K}
    x, s = _BYTES[case["x"]], _BYTES[case["s"]]
    if op == "dropout":
        return {"bytes": M * N * (x + s * (2 if case["residual"] else 1)), "flops": 2 * M * N}
    z, w = _BYTES[case["z"]], _BYTES[case["param"]]
    if op == "norm":
        return {"bytes": M * N * (x + s * (2 if case["residual"] else 1) + z) + 2 * N * w + 8 * M, "flops": 10 * M * N}
    return {"bytes": M * N * (z + s * (3 if case["stream"] else 2) + x) + N * w + 8 * M + 8 * N, "flops": 15 * M * N}


# ------------------------------------------------------------------------------------------------ inputs
def _normal(gen, shape, kind, scale=1.0, shift=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(scale).add_(shift).to(_TYPES[kind])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "weight_grad":
        r, o, i, t, g = case["tokens"], case["out"], case["into"], case["t"], case["g"]
        st["dy"] = _normal(gen, (r, o), t, 0.05)
        st["x"] = _normal(gen, (r, i), t)
        st["before"] = _normal(gen, (o, i), g, 0.5) if case["accumulate"] else None
        st["dw"] = torch.empty((o, i), dtype=_TYPES[g], device="cuda")
        if own:
            st["plan"] = _plan(o, i, r, dtype=t, kind="WGRAD", out_dtype=g, residual_dtype=g, has_residual=case["accumulate"], b_major=1)
        return st
    M, N = case["M"], case["N"]
    if op == "glu":
        K, t = case["K"], case["t"]
        st["x"] = _normal(gen, (M, K), t)
        st["w"] = _normal(gen, (2 * N, K), t, 1.0 / math.sqrt(K))
        st["h"] = torch.empty((M, N), dtype=_TYPES[t], device="cuda")
        st["gu"] = torch.empty((M, 2 * N), dtype=_TYPES[t], device="cuda") if case["aux"] else None
        if own:
            kind = {"swiglu": "SWIGLU", "geglu": "GEGLU_TANH"}[case["act"]] + ("_AUX" if case["aux"] else "")
            st["plan"] = _plan(M, N, K, dtype=t, kind=kind, out_dtype=t)
        return st
    if op == "glu_back":
        K, t = case["K"], case["t"]
        st["dy"] = _normal(gen, (M, K), t, 0.05)
        st["wd"] = _normal(gen, (K, N), t, 1.0 / math.sqrt(N))
        st["gu"] = _normal(gen, (M, 2 * N), t)
        st["dgu"] = torch.empty((M, 2 * N), dtype=_TYPES[t], device="cuda")
        if own:
            kind = {"swiglu": "DSWIGLU", "geglu": "DGEGLU_TANH"}[case["act"]]
            st["plan"] = _plan(M, N, K, dtype=t, kind=kind, out_dtype=t, b_major=1)
        return st
    # the counter of the random numbers: a seed of the run and an offset of the step, each a 64-bit number
    st["rng"] = ((seed * 0x9E3779B97F4A7C15 + 0x1234567) % 2**64, (seed * 0xD1B54A32D192ED03 + 7) % 2**64)
    empty = lambda kind: torch.empty((M, N), dtype=_TYPES[kind], device="cuda")  # noqa: E731
    if op == "dropout":
        st["x"] = _normal(gen, (M, N), case["x"])
        st["residual"] = _normal(gen, (M, N), case["s"], 2.0) if case["residual"] else None
        st["y"] = empty(case["s"])
        return st
    st["gamma"] = _normal(gen, (N,), case["param"], 0.1, 1.0)
    if op == "norm":
        st["x"] = _normal(gen, (M, N), case["x"])
        st["residual"] = _normal(gen, (M, N), case["s"], 2.0, 0.25) if case["residual"] else None
        st["beta"] = _normal(gen, (N,), case["param"], 0.1)
        st["sum"], st["z"] = empty(case["s"]), empty(case["z"])
        st["mean"], st["rstd"] = (torch.empty(M, dtype=torch.float32, device="cuda") for _ in range(2))
        return st
    # norm_back: what the forward pass kept, and the gradients that arrive
    st["sum"] = _normal(gen, (M, N), case["s"], 2.0, 0.25)
    wide = st["sum"].double()
    mean = wide.mean(dim=1)
    st["mean"] = mean.float()
    st["rstd"] = (1.0 / torch.sqrt((wide - mean[:, None]).square().mean(dim=1) + _EPS)).float()
    del wide
    st["dz"] = _normal(gen, (M, N), case["z"], 0.05)
    st["dsum"] = _normal(gen, (M, N), case["s"], 0.05) if case["stream"] else None
    st["dres"], st["dx"] = empty(case["s"]), empty(case["x"])
    st["dgamma"], st["dbeta"] = (torch.empty(N, dtype=torch.float32, device="cuda") for _ in range(2))
    if own:
        import gemm_bias_activation_tcgen05_b200 as fl
        st["ws_bytes"] = fl.fl_layernorm_grad_workspace_size(M, N)
        st["ws"] = torch.empty(max(st["ws_bytes"], 16), dtype=torch.uint8, device="cuda")
    return st


def _plan(M, N, K, **epi):
    """A plan, which a user's program makes once for a layer's shape and keeps."""
    import gemm_bias_activation_tcgen05_b200 as fl
    return fl.Plan(M, N, K, **epi)


# ------------------------------------------------------------------------------------------------ the operators
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import gemm_bias_activation_tcgen05_b200 as fl
    case = st["case"]
    op = case["op"]
    if op == "weight_grad":
        st["plan"].execute(st["dy"], st["x"], residual=st["before"], out=st["dw"])
        return st["dw"]
    if op == "glu":
        st["plan"].execute(st["x"], st["w"], aux=st["gu"], out=st["h"])
        return (st["h"], st["gu"]) if case["aux"] else st["h"]
    if op == "glu_back":
        st["plan"].execute(st["dy"], st["wd"], aux=st["gu"], out=st["dgu"])
        return st["dgu"]
    M, N, p = case["M"], case["N"], case["p"]
    seed, offset = st["rng"]
    if op == "dropout":
        fl.fl_dropout(st["x"], st["residual"], st["y"], M, N, case["x"], case["s"], p=p, seed=seed, offset=offset)
        return st["y"]
    types = (case["x"], case["s"], case["z"], case["param"])
    if op == "norm":
        fl.fl_dropout_layernorm(st["x"], st["residual"], st["gamma"], st["beta"], st["sum"], st["z"], st["mean"], st["rstd"],
                                M, N, *types, eps=_EPS, p=p, seed=seed, offset=offset)
        return st["sum"], st["z"], st["mean"], st["rstd"]
    fl.fl_dropout_layernorm_backward(st["dz"], st["dsum"], st["sum"], st["mean"], st["rstd"], st["gamma"], st["dres"], st["dx"],
                                     st["dgamma"], st["dbeta"], M, N, *types, workspace=st["ws"], workspace_bytes=st["ws_bytes"],
                                     p=p, seed=seed, offset=offset)
    return st["dres"], st["dx"], st["dgamma"], st["dbeta"]


def _philox(M, N, seed, offset):
    """The 32-bit random number of each element, as int64 [M, N]: word n % 4 of Philox4x32-10 (Salmon et al., 2011)
    with the seed as key and the counter (m * ceil(N / 4) + n / 4, offset), both 64 bits, low half first."""
    low = 0xFFFFFFFF
    groups = (N + 3) // 4
    block = torch.arange(M * groups, dtype=torch.int64, device="cuda")
    c0, c1 = block & low, block >> 32
    c2 = torch.full_like(block, offset & low)
    c3 = torch.full_like(block, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):  # the ten rounds of the generator
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products: their high halves are masked after the shift
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), dim=1).reshape(M, groups * 4)[:, :N]


def _dropped(x, case, rng):
    """keep * x / (1 - p) in 32 bits; an element is dropped where its random number is below p * 2^32."""
    p = float(np.float32(case["p"]))
    x = x.float()
    if p == 0.0:
        return x
    kept = _philox(case["M"], case["N"], *rng) >= int(p * 2.0**32)
    return torch.where(kept, x * float(np.float32(1.0 / (1.0 - p))), torch.zeros_like(x))


def _gate(act, g):
    """act(g) and its derivative, in 32 bits."""
    if act == "swiglu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "weight_grad":
        dw = st["dy"].float().t() @ st["x"].float()
        if case["accumulate"]:
            dw = dw + st["before"].float()
        return dw.to(_TYPES[case["g"]])
    if op == "glu":
        t, N = _TYPES[case["t"]], case["N"]
        gu = st["x"].float() @ st["w"].float().t()
        h = (_gate(case["act"], gu[:, :N])[0] * gu[:, N:]).to(t)
        return (h, gu.to(t)) if case["aux"] else h
    if op == "glu_back":
        t, N = _TYPES[case["t"]], case["N"]
        dh = st["dy"].float() @ st["wd"].float()
        g, u = st["gu"][:, :N].float(), st["gu"][:, N:].float()
        a, da = _gate(case["act"], g)
        return torch.cat((dh * u * da, dh * a), dim=1).to(t)
    if op == "dropout":
        y = _dropped(st["x"], case, st["rng"])
        if case["residual"]:
            y = y + st["residual"].float()
        return y.to(_TYPES[case["s"]])
    gamma = st["gamma"].float()
    if op == "norm":
        s = _dropped(st["x"], case, st["rng"])
        if case["residual"]:
            s = s + st["residual"].float()
        mean = s.mean(dim=1)
        d = s - mean[:, None]
        rstd = 1.0 / torch.sqrt((d * d).mean(dim=1) + _EPS)
        z = d * rstd[:, None] * gamma + st["beta"].float()
        return s.to(_TYPES[case["s"]]), z.to(_TYPES[case["z"]]), mean, rstd
    dz = st["dz"].float()
    unit = (st["sum"].float() - st["mean"][:, None]) * st["rstd"][:, None]
    g = dz * gamma
    ds = (g - g.mean(dim=1, keepdim=True) - unit * (g * unit).mean(dim=1, keepdim=True)) * st["rstd"][:, None]
    if case["stream"]:
        ds = ds + st["dsum"].float()
    dx = _dropped(ds, case, st["rng"])
    return ds.to(_TYPES[case["s"]]), dx.to(_TYPES[case["x"]]), (dz * unit).sum(dim=0), dz.sum(dim=0)


# ------------------------------------------------------------------------------------------------ 64 bits
def _keep64(case, rng):
    """Factor of each element, in 64 bits: 0 where dropped, else 1 / (1 - p)."""
    M, N, p = case["M"], case["N"], float(np.float32(case["p"]))
    if p == 0.0:
        return 1.0
    seed, offset = rng
    groups = -(-N // 4)
    mask, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    n = np.arange(M * groups, dtype=np.uint64)
    ctr = [n & mask, n >> sh, np.full_like(n, offset & 0xFFFFFFFF), np.full_like(n, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        p0 = ctr[0] * np.uint64(0xD2511F53)
        p1 = ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(p1 >> sh) ^ ctr[1] ^ np.uint64((key[0] + r * 0x9E3779B9) % 2**32), p1 & mask,
               (p0 >> sh) ^ ctr[3] ^ np.uint64((key[1] + r * 0xBB67AE85) % 2**32), p0 & mask]
    words = np.stack([c.astype(np.uint32) for c in ctr], axis=-1).reshape(M, 4 * groups)[:, :N]
    kept = torch.from_numpy(np.ascontiguousarray(words >= np.uint32(int(p * 4294967296.0)))).cuda()
    return kept.double() / (1.0 - p)


def _act64(act, v):
    """act(v) and its derivative through the logistic function, in 64 bits."""
    if act == "swiglu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    k = 2.0 * math.sqrt(2.0 / math.pi)  # (1 + tanh(y)) / 2 is the logistic function of 2 y
    s = torch.sigmoid(k * (v + 0.044715 * v**3))
    return v * s, s + v * s * (1 - s) * k * (1 + 0.134145 * v**2)


def exact(case, seed):
    st = prepare(case, seed)
    wide = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op == "weight_grad":
        out = torch.einsum("ro,ri->oi", wide["dy"], wide["x"])
        return out + wide["before"] if case["accumulate"] else out
    if op == "glu":
        wg, wu = wide["w"][: case["N"]], wide["w"][case["N"]:]
        g, u = torch.einsum("mk,nk->mn", wide["x"], wg), torch.einsum("mk,nk->mn", wide["x"], wu)
        h = _act64(case["act"], g)[0] * u
        return (h, torch.cat((g, u), dim=1)) if case["aux"] else h
    if op == "glu_back":
        dh = torch.einsum("mk,kn->mn", wide["dy"], wide["wd"])
        g, u = wide["gu"].split(case["N"], dim=1)
        a, slope = _act64(case["act"], g)
        return torch.cat((dh * slope * u, dh * a), dim=1)
    keep = _keep64(case, st["rng"])
    if op == "dropout":
        y = wide["x"] * keep
        return y + wide["residual"] if case["residual"] else y
    if op == "norm":
        s = wide["x"] * keep
        if case["residual"]:
            s = s + wide["residual"]
        var, mean = torch.var_mean(s, dim=1, correction=0)
        rstd = (var + _EPS).rsqrt()
        return s, (s - mean[:, None]) * rstd[:, None] * wide["gamma"] + wide["beta"], mean, rstd
    N = case["N"]
    unit = (wide["sum"] - wide["mean"][:, None]) * wide["rstd"][:, None]
    g = wide["dz"] * wide["gamma"]
    a = torch.einsum("mn->m", g)[:, None] / N
    b = torch.einsum("mn,mn->m", g, unit)[:, None] / N
    ds = wide["rstd"][:, None] * (g - a - unit * b)
    if case["stream"]:
        ds = ds + wide["dsum"]
    return ds, ds * keep, torch.einsum("mn,mn->n", wide["dz"], unit), wide["dz"].sum(dim=0)
