"""GPU parity of the gated linear units, their backward and the weight gradient.

Against the float64 oracle, element by element.  Bounds, with e = 2^-24:
  * an accumulator of K products: the tensor core adds 16 products a step into fp32 and may cut
    instead of rounding, so at most K/16 + 16 steps of 2e each: (K/16 + 16)·2e·Σ|a||w|;
  * σ(y) from the special-function unit: relative (2^-20 + |y|·2^-22) (two results near 2^-22 each, and
    the rounding of y, which moves e^(-y) by |y|·e); values below 2^-126 may be flushed to zero;
  * one rounding to the output type: half a step.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import training as T
from tests import parity as P

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF_MIN = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}
KIND = {"SWIGLU": ("SWIGLU", "SWIGLU_AUX", "DSWIGLU"), "GEGLU_TANH": (None, "GEGLU_TANH_AUX", "DGEGLU_TANH")}


@pytest.fixture(scope="module")
def fl():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import gemm_bias_activation_tcgen05_b200 as m
    return m


def within(got, want, tol, dtype, what):
    assert got.shape == want.shape
    bound = tol + P.ULP_REL[dtype] / 2 * (np.abs(want) + tol) + HALF_MIN[dtype] + 2.0 ** -120
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / bound):.2f} of the "
                           f"bound at {np.unravel_index(np.nanargmax(np.abs(got - want) / bound), got.shape)}")


def acc_err(a, w):
    """Bound on the error of a·w (float64 a [m,k], w [k,n])."""
    return (a.shape[1] / 16 + 16) * 2 * E * (np.abs(a) @ np.abs(w))


def sigma(x, kind):
    """(y, σ(y), y') of the gate x·σ(y)."""
    k = 2 * math.sqrt(2 / math.pi)
    y, dy = (x, np.ones_like(x)) if kind == "SWIGLU" else (k * (x + 0.044715 * x**3), k * (1 + 0.134145 * x * x))
    return y, T._logistic(kind, x)[0], dy


def gate_err(x, kind):
    """Bounds on the errors of act(x) and act'(x) for an exact x."""
    y, s, dy = sigma(x, kind)
    rel = 2.0 ** -20 + np.abs(y) * 2.0 ** -22
    t = np.abs(x) * dy
    return rel * np.abs(x) * s, rel * s * (1 + 2 * t) + s * t * 2.0 ** -22


def mat(rows, cols, dtype, seed, scale=1.0, ld=0):
    """CPU matrix and its device copy with pitch ld (NaN between the rows)."""
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(rows, cols, generator=g) * scale).to(P.TD[dtype])
    d = torch.full((rows, ld or cols), float("nan"), dtype=P.TD[dtype], device="cuda")
    d[:, :cols] = t.cuda()
    return P.to64(t), d


def up8(n):
    return -(-n // 8) * 8


def run(fl, plan, *args, **kw):
    try:
        plan.execute(*args, **kw)
        assert plan.check() == fl.FL_OK, fl.fl_last_error()
        return plan.info()
    finally:
        plan.free()


def check_glu(h, gu, x, W, kind, dtype, what):
    want, exact = T.glu(x, W, kind)
    N = want.shape[1]
    d = acc_err(x, W.T)
    g, u, dg, du = exact[:, :N], exact[:, N:], d[:, :N], d[:, N:]
    act = np.abs(T.gate(g, kind))
    da = 1.13 * dg + gate_err(g, kind)[0] + gate_err(g + dg, kind)[0]  # |act'| < 1.13
    within(h, want, da * (np.abs(u) + du) + act * du + 2 * E * np.abs(want), dtype, what + " h")
    if gu is not None:
        within(gu, exact, d, dtype, what + " gu")


def _glu(fl, M, N, K, kind="SWIGLU", dtype="bf16", out_dtype=None, aux=False, pad=0, scale=None, noalloc=False):
    out_dtype = out_dtype or dtype
    lda, ldo = up8(K) + pad, up8(N) + pad
    x, dx = mat(M, K, dtype, M + N, 1.0, lda)
    W, dW = mat(2 * N, K, dtype, N + K, scale or 1 / math.sqrt(max(K, 1)), lda)
    h = torch.full((M, ldo), float("nan"), dtype=P.TD[out_dtype], device="cuda")
    gu = torch.full((M, 2 * N), float("nan"), dtype=P.TD[out_dtype], device="cuda") if aux else None
    epi = dict(kind=KIND[kind][1 if aux else 0], out_dtype=out_dtype, lda=lda, ldb=lda, ldo=ldo)
    if noalloc:
        fl.fl_execute_noalloc(M, N, K, dtype, "32F", fl.make_epilogue(**epi), dx, dW, aux=gu, out=h)
        torch.cuda.synchronize()
        info = None
    else:
        info = run(fl, fl.Plan(M, N, K, dtype=dtype, **epi), dx, dW, aux=gu, out=h)
    check_glu(P.to64(h[:, :N]), None if gu is None else P.to64(gu), x, W, kind, out_dtype, f"{kind} {M}x{N}x{K} {dtype} {info}")
    assert torch.isnan(h[:, N:].float()).all(), "written into the row padding"


GLU_SHAPES = [(1, 128, 64), (1, 8, 8), (5, 200, 72), (1, 2056, 1032), (8, 520, 4096), (9, 264, 136), (16, 1000, 520), (17, 136, 64),
              (33, 512, 200), (64, 1032, 1000), (128, 640, 264), (129, 264, 72), (300, 520, 768), (777, 1000, 520), (2100, 1288, 328)]


@pytest.mark.parametrize("M,N,K", GLU_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_swiglu(fl, M, N, K, dtype):
    _glu(fl, M, N, K, dtype=dtype)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 77, 100), (40, 33, 57), (300, 333, 123), (2, 5, 700), (260, 1, 9)])
def test_swiglu_ragged(fl, M, N, K):
    _glu(fl, M, N, K)
    _glu(fl, M, N, K, dtype="f16", out_dtype="bf16", pad=16)


@pytest.mark.parametrize("M", [1, 2, 7, 300])
def test_swiglu_without_depth_and_large_gates(fl, M):
    _glu(fl, M, 64, 0)
    _glu(fl, M, 128, 256, scale=8.0)  # gates of a hundred: σ saturates at both ends


@pytest.mark.parametrize("M,N,K", [(1, 128, 64), (5, 200, 72), (64, 1032, 1000), (129, 264, 72), (777, 1000, 520), (2100, 1288, 328),
                                   (300, 8, 1)])
@pytest.mark.parametrize("kind,dtype", [("SWIGLU", "bf16"), ("GEGLU_TANH", "bf16"), ("GEGLU_TANH", "f16")])
def test_glu_aux(fl, M, N, K, kind, dtype):
    _glu(fl, M, N, K, kind, dtype, aux=True)


SPLIT = [(40, 264, 4096), (64, 1000, 4000), (300, 520, 3000), (257, 64, 8192), (600, 136, 2049)]


@pytest.mark.parametrize("M,N,K", SPLIT)
def test_few_tiles_in_k_splits(fl, M, N, K):
    """Shapes whose tiles leave most of the GPU idle: K is cut, and a second kernel does the epilogue."""
    for kind, b_major in (("SWIGLU", 0), ("GEGLU_TANH_AUX", 0), ("DSWIGLU", 1)):
        i = fl.fl_plan_preview(M, N, K, "bf16", kind=kind, b_major=b_major, lda=up8(K), ldb=up8(N if b_major else K))
        assert i["split_k"] > 1 and i["launches_per_execute"] == 2, (kind, i)
    _glu(fl, M, N, K)
    _glu(fl, M, N - 3, K, dtype="f16")
    _glu(fl, M, N, K, "GEGLU_TANH", aux=True)
    _glu(fl, M, N, K, "SWIGLU", "f16", aux=True, pad=8)
    _glu(fl, M, N, K, noalloc=True)
    _dglu(fl, M, N, K)
    _dglu(fl, M, N, K, "GEGLU_TANH", "f16", pad=8)
    _dglu(fl, M, N, K, in_place=True)


def test_glu_noalloc(fl):
    _glu(fl, 3, 264, 520, noalloc=True)
    _glu(fl, 300, 264, 520, aux=True, kind="GEGLU_TANH", noalloc=True)


def check_dglu(dgu, dy, Wd, gu, kind, dtype, what):
    want, dh = T.glu_backward(dy, Wd, gu, kind)
    N = dh.shape[1]
    d = acc_err(dy, Wd)
    g, u = gu[:, :N], gu[:, N:]
    act, slope = T.gate(g, kind), T.gate_grad(g, kind)
    ea, es = gate_err(g, kind)
    tol = np.concatenate([(np.abs(dh) + d) * np.abs(u) * es + d * np.abs(u * slope), (np.abs(dh) + d) * ea + d * np.abs(act)], axis=1)
    within(dgu, want, tol + 3 * E * np.abs(want), dtype, what)


def _dglu(fl, M, N, K, kind="SWIGLU", dtype="bf16", out_dtype=None, pad=0, in_place=False):
    out_dtype = out_dtype or dtype
    dy, d_dy = mat(M, K, dtype, M + 1, 0.5, up8(K) + pad)
    Wd, dW = mat(K, N, dtype, N + 1, 1 / math.sqrt(N), up8(N) + pad)
    gu, dgu_in = mat(M, 2 * N, out_dtype, K + 1, 2.0)
    out = dgu_in if in_place else torch.full((M, 2 * N + pad), float("nan"), dtype=P.TD[out_dtype], device="cuda")
    info = run(fl, fl.Plan(M, N, K, dtype=dtype, kind=KIND[kind][2], out_dtype=out_dtype, b_major=1, lda=up8(K) + pad,
                           ldb=up8(N) + pad, ldo=2 * N + (0 if in_place else pad)), d_dy, dW, aux=dgu_in, out=out)
    check_dglu(P.to64(out[:, :2 * N]), dy, Wd, gu, kind, out_dtype, f"D{kind} {M}x{N}x{K} {dtype} {info}")
    assert torch.isnan(out[:, 2 * N:].float()).all()
    if not in_place:
        assert np.array_equal(P.to64(dgu_in), gu), "aux was written"


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (5, 136, 72), (130, 264, 1), (257, 1000, 520), (2047, 1000, 768), (700, 2056, 264),
                                   (4100, 520, 72), (64, 4096, 64)])
@pytest.mark.parametrize("kind,dtype", [("SWIGLU", "bf16"), ("GEGLU_TANH", "f16"), ("GEGLU_TANH", "bf16")])
def test_dglu(fl, M, N, K, kind, dtype):
    _dglu(fl, M, N, K, kind, dtype)


def test_dglu_options(fl):
    _dglu(fl, 300, 264, 200, pad=8)
    _dglu(fl, 300, 264, 200, dtype="f16", out_dtype="bf16", pad=24)
    _dglu(fl, 3000, 1032, 200, in_place=True)
    _dglu(fl, 70, 64, 0)  # dh = 0


@pytest.mark.parametrize("kind", ["SWIGLU", "GEGLU_TANH"])
def test_gates_at_the_ends_of_the_range(fl, kind):
    """Gates as large as the type holds: the derivative is 1 or 0 there, never 0·∞."""
    M, N, K = 64, 64, 64
    dy, d_dy = mat(M, K, "bf16", 1, 0.5)
    Wd, dW = mat(K, N, "bf16", 2)
    gu = torch.randn(M, 2 * N, generator=torch.Generator().manual_seed(3)).bfloat16()
    big = torch.tensor([250.0, -250.0, 1e19, -1e19, 3e38, -3e38, float("inf"), 0.0]).bfloat16()
    gu[:, :N] = big.repeat(M, N // 8)
    out = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    run(fl, fl.Plan(M, N, K, kind=KIND[kind][2], out_dtype="bf16", b_major=1), d_dy, dW, aux=gu.cuda(), out=out)
    g, u = P.to64(gu[:, :N]), P.to64(gu[:, N:])
    dh, d = dy @ Wd, acc_err(dy, Wd)
    slope = np.where(g == 0, 0.5, (g > 0).astype(float))
    within(P.to64(out[:, :N]), dh * u * slope, d * np.abs(u) + 3 * E * np.abs(dh * u), "bf16", "dg")
    fin = np.abs(g) < 1e18  # the others overflow in the product with dh
    within(np.where(fin, P.to64(out[:, N:]), 0), np.where(fin, dh * np.maximum(g, 0), 0), np.where(fin, d * np.abs(g), 0) + 1e-30,
           "bf16", "du")


def _wgrad(fl, M, N, tokens, dtype="bf16", out_dtype="f32", accumulate=False, scale=1.0, pad=0, in_place=False, res_dtype=None,
           noalloc=False):
    res_dtype = res_dtype or out_dtype
    dy, d_dy = mat(tokens, M, dtype, M + 5, 0.25, up8(M) + pad)
    x, d_x = mat(tokens, N, dtype, N + 5, 1.0, up8(N) + pad)
    ldo = up8(N) + pad
    before, d_before = mat(M, N, res_dtype, 9, 2.0, ldo) if accumulate else (None, None)
    out = d_before if in_place else torch.full((M, ldo), float("nan"), dtype=P.TD[out_dtype], device="cuda")
    epi = dict(kind="WGRAD", out_dtype=out_dtype, residual_dtype=res_dtype, has_residual=accumulate, scale=scale, b_major=1,
               lda=up8(M) + pad, ldb=up8(N) + pad, ldo=ldo, ldr=ldo)
    if noalloc:
        fl.fl_execute_noalloc(M, N, tokens, dtype, "32F", fl.make_epilogue(**epi), d_dy, d_x, residual=d_before, out=out)
        torch.cuda.synchronize()
        info = None
    else:
        info = run(fl, fl.Plan(M, N, tokens, dtype=dtype, **epi), d_dy, d_x, residual=d_before, out=out)
    want = T.weight_grad(dy, x, before, scale)
    tol = acc_err(dy.T, x) * abs(scale) + 3 * E * np.abs(want)
    tol += 32 * 2 * E * abs(scale) * (np.abs(dy.T) @ np.abs(x))  # the sum of at most 32 partial results
    if accumulate:
        tol += 2 * E * abs(scale) * np.abs(before)
    within(P.to64(out[:, :N]), want, tol, out_dtype, f"WGRAD {M}x{N} of {tokens} {dtype}->{out_dtype} {info}")
    assert torch.isnan(out[:, N:].float()).all()
    return info


@pytest.mark.parametrize("M,N,tokens", [(8, 8, 1), (768, 768, 2047), (128, 256, 4096), (264, 520, 63), (1000, 328, 777), (1, 1, 300),
                                        (77, 33, 129), (300, 515, 1000), (2056, 1032, 65), (64, 64, 20000), (4100, 4100, 200)])
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "f32"), ("f16", "f16")])
def test_weight_grad(fl, M, N, tokens, dtype, out_dtype):
    _wgrad(fl, M, N, tokens, dtype, out_dtype)


def test_weight_grad_options(fl):
    for shape in [(768, 520, 4000), (2600, 2600, 300), (75, 77, 1000)]:  # with and without K splits, ragged ends
        _wgrad(fl, *shape, accumulate=True)
        _wgrad(fl, *shape, accumulate=True, in_place=True, scale=0.5)
        _wgrad(fl, *shape, out_dtype="bf16", accumulate=True, in_place=True)
        _wgrad(fl, *shape, out_dtype="bf16", res_dtype="f32", accumulate=True, pad=8)
        _wgrad(fl, *shape, out_dtype="f32", res_dtype="f16", accumulate=True, pad=8)
        _wgrad(fl, *shape, noalloc=True, accumulate=True)
        _wgrad(fl, *shape, dtype="f16", scale=-3.0, pad=16)
    _wgrad(fl, 264, 136, 0, accumulate=True)  # no tokens: the earlier gradient
    _wgrad(fl, 264, 136, 0)
    assert _wgrad(fl, 256, 256, 16384)["split_k"] > 1


@pytest.mark.parametrize("out_dtype,tokens,deep", [("f32", 130, 1), ("f32", 3100, 2), ("bf16", 300, 1), ("bf16", 700, 2), ("f16", 64, 1)])
def test_weight_grad_of_many_tiles_accumulates(fl, out_dtype, tokens, deep):
    """Several tiles a pair: the residual of a tile's first block is sent for during the tile before; both stage depths."""
    for M, N, in_place in [(2600, 2600, False), (5001, 1339, True)]:
        info = _wgrad(fl, M, N, tokens, dtype="f16" if out_dtype == "f16" else "bf16", out_dtype=out_dtype, accumulate=True,
                      in_place=in_place)
        assert info["split_k"] == 1 and info["stages"] == (5 if deep == 1 else 3) and info["grid"] == 148


@pytest.mark.parametrize("M,N,tokens,split", [(2304, 2304, 16384, False), (2304, 2304, 4099, False), (512, 512, 16384, True)])
@pytest.mark.parametrize("res_dtype", [None, "f32", "bf16"])
def test_long_sums_are_as_exact_as_fp32(fl, M, N, tokens, split, res_dtype):
    """Runs of 896 tokens: 56 steps of 16, each of which loses at most 2^-23 of the sum so far (rounded towards zero), so that
    the runs' errors together are below 56 * 2^-23 = 6.7e-6 of the result's norm, and at most 21 additions to nearest add
    21 * 2^-24 = 1.3e-6.  One sum of 16384 tokens measured 1.9e-5."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    dy, x = (torch.randn(tokens, c, generator=gen, device="cuda").bfloat16() for c in (M, N))
    before = torch.randn(M, N, generator=gen, device="cuda").to(P.TD[res_dtype]) if res_dtype else None
    out = torch.empty(M, N, device="cuda")
    info = run(fl, fl.Plan(M, N, tokens, kind="WGRAD", b_major=1, out_dtype="f32", has_residual=before is not None,
                           residual_dtype=res_dtype or "f32"), dy, x, residual=before, out=out)
    assert (info["split_k"] > 1) == split
    rows = slice(M - 300, M)
    want = dy[:, rows].double().T @ x.double()
    if before is not None:
        want += before[rows].double()
    assert (out[rows].double() - want).norm() / want.norm() < 8e-6


def test_plans_repeat_bit_for_bit_and_in_graphs(fl):
    """Each kind twice on new data through one plan, eagerly and in a replayed graph: the same bits."""
    M, N, K = 520, 776, 264
    cases = [("SWIGLU", 0, (M, K), (2 * N, K), None, (M, N)), ("GEGLU_TANH_AUX", 0, (M, K), (2 * N, K), "out", (M, N)),
             ("DSWIGLU", 1, (M, K), (K, N), "in", (M, 2 * N)), ("WGRAD", 1, (K, M), (K, N), None, (M, N))]
    for kind, b_major, sa, sw, aux, so in cases:
        mk = lambda s, seed: torch.randn(*s, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()  # noqa: E731
        plan = fl.Plan(M, N, K, kind=kind, out_dtype="bf16", b_major=b_major)
        A, W, gu, out = mk(sa, 1), mk(sw, 2), (mk((M, 2 * N), 3) if aux else None), torch.empty(so, dtype=torch.bfloat16, device="cuda")
        plan.execute(A, W, aux=gu, out=out)
        torch.cuda.synchronize()
        first = (out.clone(), gu.clone() if aux else None)
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            plan.execute(A, W, aux=gu, out=out)
        out.zero_()
        if aux == "out":
            gu.zero_()
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and (not aux or torch.equal(gu, first[1])), kind
        A.copy_(mk(sa, 7))
        g.replay()
        plan2 = torch.empty_like(out)
        torch.cuda.synchronize()
        plan.execute(A, W, aux=gu, out=plan2)
        assert plan.check() == fl.FL_OK
        assert torch.equal(out, plan2) and not torch.equal(out, first[0]), kind
        plan.free()


@pytest.mark.parametrize("kind", ["SWIGLU", "GEGLU_TANH"])
def test_a_training_step_of_the_block(fl, kind):
    """x -> gated block -> down projection -> dropout + residual + LayerNorm, and all the way back: every step against the
    oracle on the step's own inputs, and the gradients against float64 autograd through the whole block."""
    M, N, D, p, seed, off, eps, t = 300, 520, 264, 0.1, 17, 4, 1e-5, "bf16"
    x, dx = mat(M, D, t, 1)
    W, dW = mat(2 * N, D, t, 2, 1 / math.sqrt(D))
    Wd, dWd = mat(D, N, t, 3, 1 / math.sqrt(N))
    dz, ddz = mat(M, D, t, 4, 0.5)
    new = lambda *s, dt=torch.bfloat16: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    h, gu, y, s, z, dres, ddy, dgu, dxb = (new(M, N), new(M, 2 * N), new(M, D), new(M, D), new(M, D), new(M, D), new(M, D),
                                           new(M, 2 * N), new(M, D))
    mean, rstd, dgam, dbet = (new(n, dt=torch.float32) for n in (M, M, D, D))
    gW, gWd = new(2 * N, D, dt=torch.float32), new(D, N, dt=torch.float32)
    gamma, beta = torch.linspace(0.5, 1.5, D).cuda(), torch.linspace(-1, 1, D).cuda()
    run(fl, fl.Plan(M, N, D, kind=KIND[kind][1], out_dtype=t), dx, dW, aux=gu, out=h)
    run(fl, fl.Plan(M, D, N, kind="NONE", out_dtype=t), h, dWd, out=y)
    fl.fl_dropout_layernorm(y, dx, gamma, beta, s, z, mean, rstd, M, D, t, t, t, "f32", eps=eps, p=p, seed=seed, offset=off)
    ws_n = fl.fl_layernorm_grad_workspace_size(M, D)
    ws = torch.empty(ws_n, dtype=torch.uint8, device="cuda")
    fl.fl_dropout_layernorm_backward(ddz, None, s, mean, rstd, gamma, dres, ddy, dgam, dbet, M, D, t, t, t, "f32", workspace=ws,
                                     workspace_bytes=ws_n, p=p, seed=seed, offset=off)
    run(fl, fl.Plan(M, N, D, kind=KIND[kind][2], out_dtype=t, b_major=1), ddy, dWd, aux=gu, out=dgu)
    run(fl, fl.Plan(2 * N, D, M, kind="WGRAD", out_dtype="f32", b_major=1), dgu, dx, out=gW)
    run(fl, fl.Plan(D, N, M, kind="WGRAD", out_dtype="f32", b_major=1), ddy, h, out=gWd)
    # the block's input gets the block's gradient and the residual's
    run(fl, fl.Plan(M, D, 2 * N, kind="NONE", out_dtype=t, residual_dtype=t, has_residual=True, b_major=1), dgu, dW, residual=dres, out=dxb)
    check_glu(P.to64(h), P.to64(gu), x, W, kind, t, "step")
    check_dglu(P.to64(dgu), P.to64(ddy), Wd, P.to64(gu), kind, t, "step")
    # float64 autograd of the whole block
    leaf = [torch.from_numpy(a).requires_grad_() for a in (x, W, Wd)] + [v.double().cpu().requires_grad_() for v in (gamma, beta)]
    tx, tW, tWd, tg, tb = leaf
    v = tx @ tW.T
    act = torch.nn.functional.silu(v[:, :N]) if kind == "SWIGLU" else torch.nn.functional.gelu(v[:, :N], approximate="tanh")
    keep = torch.from_numpy(T.keep_mask(M, D, p, seed, off)).double() / (1 - float(np.float32(p)))
    zz = torch.nn.functional.layer_norm(tx + ((act * v[:, N:]) @ tWd.T) * keep, (D,), tg, tb, eps)
    (zz * torch.from_numpy(dz)).sum().backward()
    # bf16 tensors on the way: z has h, y, s, z rounded, a gradient up to six more; each rounding moves its tensor by at
    # most 2^-8 of every element, and the maps between them have gains near one here, so a few times 2^-8 in the 2-norm
    for got, want, n, what in [(z, zz.detach(), 4, "z"), (dxb, tx.grad, 10, "dx"), (gW, tW.grad, 9, "dW"), (gWd, tWd.grad, 8, "dWd"),
                               (dgam, tg.grad, 4, "dgamma"), (dbet, tb.grad, 1, "dbeta")]:
        rel = float((got.double().cpu() - want).norm() / want.norm())
        assert rel <= n * 2.0 ** -8, (what, rel)


@pytest.mark.parametrize("kind", ["SWIGLU", "GEGLU_TANH"])
@pytest.mark.parametrize("M,N,K,split", [(64, 64, 64, False), (300, 264, 200, False), (64, 1000, 4000, True)])
def test_nan_gates_give_nan_gradients(fl, kind, M, N, K, split):
    """act(NaN) and act'(NaN) are NaN: both gradients of such a place are, and no other place's is."""
    dy, d_dy = mat(M, K, "bf16", 1, 0.5)
    Wd, dW = mat(K, N, "bf16", 2, 1 / math.sqrt(N))
    gu = torch.randn(M, 2 * N, generator=torch.Generator().manual_seed(3)).bfloat16()
    nan = np.zeros((M, N), bool)
    nan[::7, ::5] = nan[M - 1, N - 1] = nan[0, 1] = True
    gu[:, :N][torch.from_numpy(nan)] = float("nan")
    out = torch.zeros(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    info = run(fl, fl.Plan(M, N, K, kind=KIND[kind][2], out_dtype="bf16", b_major=1), d_dy, dW, aux=gu.cuda(), out=out)
    assert (info["split_k"] > 1) == split
    got = P.to64(out)
    for name, half in (("dg", got[:, :N]), ("du", got[:, N:])):
        assert np.array_equal(np.isnan(half), nan), name
    clean = np.where(np.tile(nan, (1, 2)), 0.0, P.to64(gu))
    both = np.concatenate([nan, nan], axis=1)
    want, dh = T.glu_backward(dy, Wd, clean, kind)
    assert (dh != 0).all()
    assert np.abs(np.where(both, 0, got - want)).max() <= 2.0 ** -7 * np.abs(want).max()


def _long_sum(fl, M, N, tokens, dtype, out_dtype, res_dtype=None, rows=300):
    """(result, its value in 64 bits) of the last rows of a weight gradient of many tokens, and the plan's info."""
    gen = torch.Generator(device="cuda").manual_seed(tokens + M)
    dy, x = (torch.randn(tokens, c, generator=gen, device="cuda").to(P.TD[dtype]) for c in (M, N))
    before = torch.randn(M, N, generator=gen, device="cuda").to(P.TD[res_dtype]) if res_dtype else None
    out = torch.empty(M, N, device="cuda", dtype=P.TD[out_dtype])
    info = run(fl, fl.Plan(M, N, tokens, dtype=dtype, kind="WGRAD", b_major=1, out_dtype=out_dtype, has_residual=before is not None,
                           residual_dtype=res_dtype or "f32"), dy, x, residual=before, out=out)
    want = torch.zeros(rows, N, dtype=torch.float64, device="cuda") if before is None else before[M - rows:].double()
    for t in range(0, tokens, 16384):
        want += dy[t:t + 16384, M - rows:].double().T @ x[t:t + 16384].double()
    return out[M - rows:].double(), want, info


@pytest.mark.parametrize("M,N,tokens,split_tokens", [(2304, 2304, 4099, 0), (2304, 2304, 16384, 0), (512, 512, 131072, 7282)])
@pytest.mark.parametrize("res_dtype", [None, "f32", "bf16"])
def test_long_fp32_sums_hold_the_error_of_a_run(fl, M, N, tokens, split_tokens, res_dtype):
    """The documented error of a run, 9e-7 of the norm, and the additions of up to 147 runs to nearest, each off by at most
    2^-25 (rms) of the sum: √147·2^-25 = 3.6e-7, together below 1.3e-6.  One sum is off by 1.1e-9 a token: 4.4e-6 at 4099, 8e-6
    in a K split of 7282 tokens."""
    got, want, info = _long_sum(fl, M, N, tokens, "bf16", "f32", res_dtype)
    assert -(-tokens // info["split_k"]) == (split_tokens or tokens)
    rel = float((got - want).norm() / want.norm())
    assert rel < 1.3e-6, rel


@pytest.mark.parametrize("M,N,tokens,split_tokens,dtype,out_dtype", [
    (2304, 2304, 131072, 0, "f16", "f16"), (2304, 2304, 262144, 0, "bf16", "bf16"), (512, 512, 262144, 14564, "f16", "f16")])
@pytest.mark.parametrize("res_dtype", [None, "out", "f32"])
def test_long_16_bit_sums_are_not_biased(fl, M, N, tokens, split_tokens, dtype, out_dtype, res_dtype):
    """Accumulators that round towards zero shrink a sum by up to 1.1e-9 a token.  Sums are taken in runs of at most 8192
    (f16) or 65536 (bf16) tokens, so the result is shrunk by at most 9e-6 or 7.2e-5; the rounding of 300 x N results to their own
    type (2.1e-4 or 1.7e-3 rms) moves the mean by four deviations, 1e-6 or 8e-6, at most.  One sum would shrink by 1.4e-4 of
    131072 tokens, 2.9e-4 of 262144."""
    got, want, info = _long_sum(fl, M, N, tokens, dtype, out_dtype, out_dtype if res_dtype == "out" else res_dtype)
    assert -(-tokens // info["split_k"]) == (split_tokens or tokens)
    shrink = float(((got - want) * want).sum() / (want * want).sum())
    assert abs(shrink) < (1e-5 if out_dtype == "f16" else 8e-5), shrink


@pytest.mark.parametrize("tokens,dtype", [(8300, "f16"), (65700, "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_long_16_bit_sums_of_ragged_weights(fl, tokens, dtype, accumulate):
    """Just past one run, odd sizes and pitches, the earlier gradient in place: every element, and nothing between the rows.
    The bound of an accumulator of K products (above), two roundings to nearest and the result's own."""
    M, N, ld = 2101, 2099, 2104
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    dy, x = (torch.full((tokens, ld), float("nan"), dtype=P.TD[dtype], device="cuda") for _ in range(2))
    for t, c in ((dy, M), (x, N)):
        t[:, :c] = torch.randn(tokens, c, generator=gen, device="cuda").to(P.TD[dtype])
    out = torch.full((M, ld), float("nan"), dtype=P.TD[dtype], device="cuda")
    a, b = dy[:, :M].double(), x[:, :N].double()
    want, size = a.T @ b, a.abs().T @ b.abs()
    if accumulate:
        out[:, :N] = (50 * torch.randn(M, N, generator=gen, device="cuda")).to(P.TD[dtype])
        want += out[:, :N].double()
        size += out[:, :N].double().abs()
    info = run(fl, fl.Plan(M, N, tokens, dtype=dtype, kind="WGRAD", b_major=1, out_dtype=dtype, has_residual=accumulate,
                           residual_dtype=dtype, lda=ld, ldb=ld, ldo=ld, ldr=ld), dy, x, residual=out if accumulate else None, out=out)
    assert info["split_k"] == 1 and info["stages"] == 3
    within(P.to64(out[:, :N]), want.cpu().numpy(), ((tokens / 16 + 16) * 2 * E * size).cpu().numpy() + 2 * E * np.abs(want.cpu().numpy()),
           dtype, f"{tokens} tokens")
    assert torch.isnan(out[:, N:].float()).all()


@pytest.mark.parametrize("M,N,tokens", [(536, 4016, 1770), (2304, 2304, 16384), (512, 512, 131072)])
def test_long_fp32_sums_of_f16_hold_the_error_of_a_run(fl, M, N, tokens):
    """f16 products have 22 bits where bf16's have 16, of which the accumulator keeps fewer: the documented 1.1e-6 of a run, with
    the additions' 3.6e-7 (as above) 1.16e-6, so below 1.3e-6."""
    got, want, _ = _long_sum(fl, M, N, tokens, "f16", "f32")
    rel = float((got - want).norm() / want.norm())
    assert rel < 1.3e-6, rel
