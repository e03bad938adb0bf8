"""GPU parity of dropout, dropout + residual + LayerNorm and its backward pass.

Every output is compared with the float64 oracle element by element.  The bounds are those of
fp32 arithmetic in the kernels' order, with e = 2^-24 (half a step of fp32):
  * y = residual + x·k, k = 1/(1 − p) rounded: three roundings, 3e·(|x·k| + |y|);
  * a sum over a row: every term passes at most c = 16·⌈N/8192⌉ + 64 additions (a thread's own,
    the butterfly's five, the 32 warps'), so its error is at most c·e·Σ|terms|;
  * a column sum over M rows: at most M + 64 additions a term;
  * one rounding to the output type: half a step of it (plus half its smallest step).
Kept and dropped places have to be the oracle's exactly.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import training as T
from tests import parity as P

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF_MIN = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}
FP32_TINY = 2.0 ** -126  # products below the normal range lose bits


@pytest.fixture(scope="module")
def fl():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import gemm_bias_activation_tcgen05_b200 as m
    return m


def half(v, dtype):
    return P.ULP_REL[dtype] / 2 * np.abs(v) + HALF_MIN[dtype]


def within(got, want, tol, dtype, what):
    """|got − want| ≤ tol (before the output's own rounding) + half a step of the type."""
    assert got.shape == want.shape
    bound = tol + half(np.abs(want) + tol, dtype)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / bound):.2f} of the "
                           f"bound at {np.unravel_index(np.nanargmax(np.abs(got - want) / bound), got.shape)}")


def draw(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(P.TD[dtype])


def dev(t, ld=0, off=0):
    """A device copy of a CPU matrix whose rows have pitch ld and start `off` elements into the buffer;
    what lies between is NaN.  Returns (view, pitch)."""
    M, N = t.shape
    ld = ld or N
    buf = torch.full((M * ld + off,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[off:off + M * ld].view(M, ld)[:, :N]
    v.copy_(t.cuda())
    return v, ld


def untouched(v):
    """What lies between a view's rows is still NaN."""
    M, N = v.shape
    ld = v.stride(0)
    whole = torch.as_strided(v, (M, ld), (ld, 1), v.storage_offset())
    return bool(torch.isnan(whole[:, N:].float()).all())


def out(M, N, dtype, ld=0, off=0):
    return dev(torch.full((M, N), float("nan"), dtype=P.TD[dtype]), ld, off)


# ---------------------------------------------------------------- dropout
SHAPES = [(1, 1), (3, 7), (64, 768), (33, 1001), (1, 4096), (700, 520), (5, 16392), (2500, 24)]


def _dropout(fl, M, N, xt, yt, p, residual=True, seed=2**63 + 11, offset=2**35 + 3, lds=(0, 0, 0), offs=(0, 0, 0)):
    x = draw((M, N), xt, M + N)
    r = draw((M, N), yt, M * 3 + N, 2.0) if residual else None
    dx, ldx = dev(x, lds[0], offs[0])
    dr, ldr = dev(r, lds[1], offs[1]) if residual else (None, 0)
    y, ldy = out(M, N, yt, lds[2], offs[2])
    fl.fl_dropout(dx, dr, y, M, N, xt, yt, p=p, seed=seed, offset=offset, ld_x=ldx, ld_r=ldr, ld_y=ldy)
    torch.cuda.synchronize()
    xk = T.dropout(P.to64(x), p, seed, offset)
    want = xk + P.to64(r) if residual else xk
    within(P.to64(y), want, 3 * E * (np.abs(xk) + np.abs(want)), yt, f"dropout {M}x{N} {xt}->{yt}")
    if not residual and p > 0:
        assert np.array_equal(P.to64(y) == 0, (xk == 0)), "kept places differ"
    assert untouched(y)


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
def test_dropout(fl, M, N, xt, yt):
    _dropout(fl, M, N, xt, yt, 0.25)
    _dropout(fl, M, N, xt, yt, 0.1, residual=False)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -32, 0.5, 0.999])
def test_dropout_probabilities(fl, p):
    _dropout(fl, 100, 200, "f32", "f32", p)


@pytest.mark.parametrize("lds,offs", [((773, 770, 769), (0, 0, 0)), ((776, 784, 792), (0, 0, 0)), ((776, 776, 776), (1, 0, 0)),
                                      ((776, 776, 776), (0, 0, 3))])
def test_dropout_pitches(fl, lds, offs):
    _dropout(fl, 40, 768, "bf16", "bf16", 0.3, lds=lds, offs=offs)


def test_dropout_backward_is_itself_in_place_and_dropped_values_do_not_count(fl):
    M, N, p, seed, off = 50, 96, 0.4, 5, 6
    keep = T.keep_mask(M, N, p, seed, off)
    g = draw((M, N), "f32", 1)
    bad = torch.from_numpy(np.where(keep, P.to64(g), np.where(np.arange(N) % 2, np.inf, np.nan))).float().cuda()
    fl.fl_dropout(bad, None, bad, M, N, "f32", "f32", p=p, seed=seed, offset=off)
    torch.cuda.synchronize()
    want = T.dropout(P.to64(g), p, seed, off)
    within(P.to64(bad), want, 3 * E * np.abs(want), "f32", "in place")
    # infinities and NaN in kept places stay where they are
    x = torch.full((M, N), float("inf"), device="cuda")
    y = torch.empty_like(x)
    fl.fl_dropout(x, None, y, M, N, "f32", "f32", p=p, seed=seed, offset=off)
    assert np.array_equal(np.isinf(P.to64(y)), keep) and not torch.isnan(y).any()


def test_dropout_offset_on_the_device_in_a_replayed_graph(fl):
    M, N, p, seed = 65, 130, 0.5, 77
    x = draw((M, N), "f16", 2)
    dx, y = x.cuda(), torch.empty(M, N, dtype=torch.float16, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fl.fl_dropout(dx, None, y, M, N, "f16", "f16", p=p, seed=seed, offset=10, offset_dev=step)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.fl_dropout(dx, None, y, M, N, "f16", "f16", p=p, seed=seed, offset=10, offset_dev=step)
        step += 1
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        want = T.dropout(P.to64(x), p, seed, 10 + i)
        within(P.to64(y), want, 3 * E * np.abs(want), "f16", f"replay {i}")


# ---------------------------------------------------------------- forward
def sums(N):
    return (16 * -(-N // 8192) + 64) * E


def check_forward(got, x, r, gamma, beta, eps, p, seed, off, types, what):
    xt, st, zt = types
    s, z, mean, rstd = T.dropout_layernorm(x, r, gamma, beta, eps, p, seed, off)
    N = x.shape[1]
    xk = T.dropout(x, p, seed, off)
    ds = 3 * E * (np.abs(xk) + np.abs(s))
    c = sums(N)
    dmean = c * np.abs(s).mean(axis=1) + ds.mean(axis=1) + E * np.abs(mean) * 2
    d = s - mean[:, None]
    # the error of a difference, and of 1/√(mean d² + eps) through Σ d²
    dd = ds + dmean[:, None] + E * np.abs(d)
    dvar = c * (d * d).mean(axis=1) + (2 * np.abs(d) * dd + dd * dd).mean(axis=1)
    var = 1.0 / rstd ** 2
    rel = np.where(dvar < 0.5 * var, 1.0 / np.sqrt(1.0 - np.minimum(dvar / var, 0.5)) - 1.0, np.inf) + 4 * E
    g = 1.0 if gamma is None else np.abs(gamma)[None, :]
    b = 0.0 if beta is None else np.abs(beta)[None, :]
    dz = g * rstd[:, None] * (dd + (np.abs(d) + dd) * rel[:, None]) + 3 * E * (np.abs(z) + b)
    if got["sum"] is not None:
        within(got["sum"], s, ds, st, what + " sum")
    within(got["z"], z, dz, zt, what + " z")
    if got["mean"] is not None:
        within(got["mean"], mean, dmean, "f32", what + " mean")
        within(got["rstd"], rstd, rstd * rel, "f32", what + " rstd")


def _forward(fl, M, N, types=("bf16", "bf16", "bf16", "bf16"), p=0.1, eps=1e-5, residual=True, affine=True, keep_sum=True,
             stats=True, pad=0, off=0, shift=0.3, seed=123, offset=456):
    xt, st, zt, pt = types
    x, r = draw((M, N), xt, M + N, 1.0, shift), draw((M, N), st, M + 2 * N, 2.0, shift) if residual else None
    gamma, beta = (draw((1, N), pt, N, 0.2, 1.0), draw((1, N), pt, N + 1, 0.2)) if affine else (None, None)
    ld = N + pad if pad else 0
    dx, ldx = dev(x, ld, off)
    dr, ldr = dev(r, ld, off) if residual else (None, 0)
    dg, db = (dev(gamma, 0, off)[0], dev(beta, 0, off)[0]) if affine else (None, None)
    s, lds = out(M, N, st, ld, off) if keep_sum else (None, 0)
    z, ldz = out(M, N, zt, ld, off)
    mean, rstd = (torch.full((M,), float("nan"), device="cuda") for _ in range(2)) if stats else (None, None)
    fl.fl_dropout_layernorm(dx, dr, dg, db, s, z, mean, rstd, M, N, *types, eps=eps, p=p, seed=seed, offset=offset,
                            ld_x=ldx, ld_r=ldr, ld_sum=lds, ld_z=ldz)
    torch.cuda.synchronize()
    f = lambda t: None if t is None else P.to64(t)  # noqa: E731
    got = dict(sum=f(s), z=f(z), mean=f(mean), rstd=f(rstd))
    flat = lambda t: None if t is None else P.to64(t)[0]  # noqa: E731
    check_forward(got, P.to64(x), f(r), flat(gamma), flat(beta), eps, p, seed, offset, types[:3], f"{M}x{N} {types}")
    assert untouched(z) and (s is None or untouched(s))


ROWS = [(1, 1), (4, 3), (33, 100), (700, 512), (33, 513), (2048, 768), (33, 1001), (40, 1032), (9, 2040), (600, 4096), (5, 4104),
        (3, 8192), (3, 8200), (2, 16384), (2, 16400), (3, 20001), (1300, 40)]


@pytest.mark.parametrize("M,N", ROWS)
def test_dropout_layernorm(fl, M, N):
    _forward(fl, M, N)
    _forward(fl, M, N, ("f16", "f32", "f16", "f32"))


@pytest.mark.parametrize("types", [("f32", "f32", "f32", "f32"), ("bf16", "f32", "f32", "bf16"), ("f32", "f16", "bf16", "f16"),
                                   ("f16", "f16", "f32", "f32")])
def test_dropout_layernorm_types(fl, types):
    for M, N in [(70, 264), (300, 1000), (4, 16384)]:
        _forward(fl, M, N, types)


@pytest.mark.parametrize("kw", [dict(residual=False), dict(affine=False), dict(keep_sum=False, stats=False), dict(p=0.0),
                                dict(p=0.9), dict(pad=3), dict(pad=8), dict(off=1), dict(off=8, pad=8), dict(shift=50.0),
                                dict(seed=2**64 - 1, offset=2**64 - 1)])
def test_dropout_layernorm_options(fl, kw):
    _forward(fl, 100, 768, **kw)
    _forward(fl, 3, 16640, **kw)


@pytest.mark.parametrize("N", [9, 65, 513, 1031, 2049, 4095, 5121, 8191, 8193, 16383])
def test_rows_that_start_anywhere(fl, N):
    """Odd widths, pitches and bases in every type: each row starts at another place of a 16-byte word."""
    M = 37 if N < 4000 else 11
    for types in (("bf16", "bf16", "bf16", "bf16"), ("f16", "f32", "f32", "f16"), ("f32", "bf16", "f16", "f32")):
        for kw in (dict(), dict(off=1), dict(pad=3, off=5)):
            _forward(fl, M, N, types, **kw)
            _backward(fl, M, N, types, **kw)
    _forward(fl, 400, N, pad=1)
    _backward(fl, 400, N, pad=1)
    _dropout(fl, M, N, "bf16", "bf16", 0.3, lds=(N + 3, N + 1, N), offs=(1, 0, 3))
    _dropout(fl, M, N, "f32", "f16", 0.3, lds=(N + 3, N + 1, N + 2), offs=(1, 3, 5))


def test_dropout_layernorm_in_place(fl):
    """z over x and sum over the residual: every element is read before it is written."""
    for M, N in [(500, 4096), (3, 20000)]:
        x, r = draw((M, N), "bf16", 1), draw((M, N), "bf16", 2)
        dx, dr = x.cuda(), r.cuda()
        mean, rstd = (torch.empty(M, device="cuda") for _ in range(2))
        fl.fl_dropout_layernorm(dx, dr, None, None, dr, dx, mean, rstd, M, N, "bf16", "bf16", "bf16", eps=1e-5, p=0.2, seed=3)
        torch.cuda.synchronize()
        got = dict(sum=P.to64(dr), z=P.to64(dx), mean=P.to64(mean), rstd=P.to64(rstd))
        check_forward(got, P.to64(x), P.to64(r), None, None, 1e-5, 0.2, 3, 0, ("bf16",) * 3, f"in place {M}x{N}")


def test_constant_rows(fl):
    # σ² = 0: rstd = 1/√eps exactly as the formula says, z = beta
    M, N = 3, 1000
    x = torch.full((M, N), 1.5, dtype=torch.float16, device="cuda")
    beta = torch.randn(N, device="cuda")
    z = torch.empty(M, N, device="cuda")
    mean, rstd = (torch.empty(M, device="cuda") for _ in range(2))
    fl.fl_dropout_layernorm(x, None, None, beta, None, z, mean, rstd, M, N, "f16", "f16", "f32", eps=1e-5)
    assert torch.equal(z, beta.expand(M, N)) and torch.equal(mean, torch.full((M,), 1.5, device="cuda"))
    assert np.abs(P.to64(rstd) * np.sqrt(float(np.float32(1e-5))) - 1).max() < 4 * E


# ---------------------------------------------------------------- backward
def check_backward(got, dz, dsum, s, mean, rstd, gamma, p, seed, off, types, what):
    xt, st, zt = types
    dres, dx, dgamma, dbeta = T.dropout_layernorm_backward(dz, dsum, s, mean, rstd, gamma, p, seed, off)
    M, N = dz.shape
    u = (s - mean[:, None]) * rstd[:, None]
    du = 2 * E * rstd[:, None] * np.abs(s - mean[:, None]) + E * np.abs(u)
    g = dz if gamma is None else dz * gamma
    c = sums(N)
    gu = np.abs(g * u)
    da = (c + E) * np.abs(g).mean(axis=1, keepdims=True) + 2 * E * np.abs(g.mean(axis=1, keepdims=True))
    db = (c + 2 * E) * gu.mean(axis=1, keepdims=True) + (np.abs(g) * du).mean(axis=1, keepdims=True)
    b = np.abs((g * u).mean(axis=1, keepdims=True))
    a = np.abs(g.mean(axis=1, keepdims=True))
    tol = rstd[:, None] * (E * np.abs(g) + da + np.abs(u) * db + du * b + 4 * E * (np.abs(g) + a + np.abs(u) * b))
    if dsum is not None:
        tol = tol + E * np.abs(dres)
    if got.get("dres") is not None:
        within(got["dres"], dres, tol, st, what + " dres")
    if got.get("dx") is not None:
        # a kept place has ds's error times k = 1/(1 - p) (rounded) and the product's rounding; a dropped one is exactly 0
        # (whether a place is kept is the mask's to say: where a row has one element ds itself is 0 up to its error)
        k = 1.0 / (1.0 - p)
        kept = T.keep_mask(M, N, p, seed, off) if p > 0 else np.ones((M, N), bool)
        within(got["dx"], dx, np.where(kept, k * (1 + 2 * E) * tol + 2 * E * np.abs(dx), 0.0), xt, what + " dx")
        assert not got["dx"][~kept].any(), what + ": a dropped place has a gradient"
    if got.get("dgamma") is not None:
        within(got["dgamma"], dgamma, (M + 64) * E * np.abs(dz * u).sum(axis=0) + (np.abs(dz) * du).sum(axis=0), "f32", what + " dgamma")
    if got.get("dbeta") is not None:
        within(got["dbeta"], dbeta, (M + 64) * E * np.abs(dz).sum(axis=0), "f32", what + " dbeta")


def _backward(fl, M, N, types=("bf16", "bf16", "bf16", "bf16"), p=0.1, stream_grad=True, affine=True, want="dres dx dgamma dbeta",
              pad=0, off=0, seed=123, offset=456, torch_stream=None):
    xt, st, zt, pt = types
    s = draw((M, N), st, M + N, 2.0, 0.3)
    dz = draw((M, N), zt, M + 2 * N)
    dsum = draw((M, N), st, M + 3 * N) if stream_grad else None
    gamma = draw((1, N), pt, N, 0.2, 1.0) if affine else None
    s64 = P.to64(s)
    mean = s64.mean(axis=1).astype(np.float32)
    rstd = (1.0 / np.sqrt(s64.var(axis=1) + 1e-5)).astype(np.float32)
    ld = N + pad if pad else 0
    d_dz, ld_dz = dev(dz, ld, off)
    d_s, ld_s = dev(s, ld, off)
    d_dsum, ld_dsum = dev(dsum, ld, off) if stream_grad else (None, 0)
    dg = dev(gamma, 0, off)[0] if affine else None
    dres, ld_dres = out(M, N, st, ld, off) if "dres" in want else (None, 0)
    dx, ld_dx = out(M, N, xt, ld, off) if "dx" in want else (None, 0)
    dgamma = torch.full((N,), float("nan"), device="cuda") if "dgamma" in want else None
    dbeta = torch.full((N,), float("nan"), device="cuda") if "dbeta" in want else None
    n = fl.fl_layernorm_grad_workspace_size(M, N)
    ws = torch.full((max(n, 16) // 4 + 4,), float("nan"), device="cuda")  # no initial contents needed; a guard behind it
    fl.fl_dropout_layernorm_backward(d_dz, d_dsum, d_s, torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda(), dg, dres, dx,
                                     dgamma, dbeta, M, N, *types, workspace=ws, workspace_bytes=n, p=p, seed=seed, offset=offset,
                                     ld_dz=ld_dz, ld_dsum=ld_dsum, ld_sum=ld_s, ld_dres=ld_dres, ld_dx=ld_dx)
    torch.cuda.synchronize()
    assert torch.isnan(ws[n // 4:]).all(), "written behind the workspace"
    f = lambda t: None if t is None else P.to64(t)  # noqa: E731
    check_backward(dict(dres=f(dres), dx=f(dx), dgamma=f(dgamma), dbeta=f(dbeta)), P.to64(dz), f(dsum), s64,
                   mean.astype(np.float64), rstd.astype(np.float64), None if gamma is None else P.to64(gamma)[0], p, seed, offset,
                   types[:3], f"{M}x{N} {types} {want}")
    assert (dres is None or untouched(dres)) and (dx is None or untouched(dx))


@pytest.mark.parametrize("M,N", ROWS + [(3000, 96), (20000, 8)])
def test_dropout_layernorm_backward(fl, M, N):
    _backward(fl, M, N)
    _backward(fl, M, N, ("f16", "f32", "f16", "f32"), stream_grad=False)


@pytest.mark.parametrize("types", [("f32", "f32", "f32", "f32"), ("bf16", "f32", "f32", "bf16"), ("f32", "f16", "bf16", "f16"),
                                   ("f16", "f16", "f32", "f32")])
def test_dropout_layernorm_backward_types(fl, types):
    for M, N in [(70, 264), (300, 1000), (310, 8192), (160, 16384)]:
        _backward(fl, M, N, types)


@pytest.mark.parametrize("M,N", [(3600, 520), (3601, 768), (3600, 767), (3600, 1032), (3600, 1535), (3600, 2056), (3600, 2305)])
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16", "bf16"), ("f16", "f32", "f16", "f32"), ("f32", "f32", "f32", "bf16")])
def test_many_rows_of_three_vectors_a_thread(fl, M, N, types):
    """Enough rows for the kernels that hold three vectors a thread; widths that leave threads idle, odd ones too."""
    _forward(fl, M, N, types)
    _backward(fl, M, N, types)


@pytest.mark.parametrize("M,N", [(40, 4104), (300, 6144), (21, 5003), (9, 8200), (160, 12288), (5, 10001)])
def test_wide_rows_of_three_vectors_a_thread_backward(fl, M, N):
    _backward(fl, M, N)
    _backward(fl, M, N, ("f32", "f32", "f32", "f32"), stream_grad=False)


@pytest.mark.parametrize("kw", [dict(affine=False), dict(p=0.0), dict(p=0.75), dict(want="dx"), dict(want="dres"),
                                dict(want="dgamma"), dict(want="dbeta"), dict(want="dres dgamma dbeta"), dict(pad=3),
                                dict(pad=8), dict(off=1), dict(seed=2**64 - 1, offset=2**64 - 1)])
def test_dropout_layernorm_backward_options(fl, kw):
    _backward(fl, 500, 768, **kw)
    _backward(fl, 150, 16640, **kw)


def test_backward_in_place(fl):
    """dres over dsum, dx over dz: every element is read before it is written."""
    for M, N in [(700, 1024), (200, 20000)]:
        s, dz, dsum = (draw((M, N), "bf16", i, 1.5) for i in (1, 2, 3))
        s64 = P.to64(s)
        mean, rstd = s64.mean(axis=1).astype(np.float32), (1 / np.sqrt(s64.var(axis=1) + 1e-5)).astype(np.float32)
        a, b = dz.cuda(), dsum.cuda()
        fl.fl_dropout_layernorm_backward(a, b, s.cuda(), torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda(), None, b, a,
                                         None, None, M, N, "bf16", "bf16", "bf16", p=0.3, seed=9)
        torch.cuda.synchronize()
        check_backward(dict(dres=P.to64(b), dx=P.to64(a)), P.to64(dz), P.to64(dsum), s64, mean.astype(np.float64),
                       rstd.astype(np.float64), None, 0.3, 9, 0, ("bf16",) * 3, f"in place {M}x{N}")


def test_a_workspace_for_many_rows_serves_fewer(fl):
    for N in (768, 1000, 1536, 2560, 4096, 8200, 20000):
        sizes = [fl.fl_layernorm_grad_workspace_size(M, N) for M in (0, 1, 7, 100, 147, 148, 149, 591, 592, 593, 3552, 3553, 100000)]
        assert sizes == sorted(sizes) and all(n % 16 == 0 for n in sizes)


def test_backward_of_no_rows_and_repeatable(fl):
    N = 100
    g = torch.full((N,), float("nan"), device="cuda")
    b = g.clone()
    n = fl.fl_layernorm_grad_workspace_size(0, N)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    some = torch.empty(16, device="cuda")
    fl.fl_dropout_layernorm_backward(some, None, some, some, some, None, None, None, g, b, 0, N, "f32", "f32", "f32", workspace=ws,
                                     workspace_bytes=n)
    torch.cuda.synchronize()
    assert not g.any() and not b.any()
    # the same call twice gives the same bits
    M, N = 3001, 776
    s, dz = draw((M, N), "bf16", 1).cuda(), draw((M, N), "bf16", 2).cuda()
    mean, rstd = s.float().mean(1), 1 / (s.float().var(1, correction=0) + 1e-5).sqrt()
    n = fl.fl_layernorm_grad_workspace_size(M, N)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):
        o = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), *(torch.empty(N, device="cuda") for _ in range(2))]
        fl.fl_dropout_layernorm_backward(dz, None, s, mean, rstd, None, o[0], None, o[1], o[2], M, N, "bf16", "bf16", "bf16",
                                         workspace=ws, workspace_bytes=n)
        outs.append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_forward_and_backward_in_one_graph_on_another_stream(fl):
    M, N, p, seed = 130, 1032, 0.2, 31
    x, r, dz = (draw((M, N), "bf16", i) for i in (1, 2, 3))
    dx, dr, ddz = x.cuda(), r.cuda(), dz.cuda()
    s, z, dres, dxo = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    mean, rstd = (torch.empty(M, device="cuda") for _ in range(2))
    dg, db = (torch.empty(N, device="cuda") for _ in range(2))
    n = fl.fl_layernorm_grad_workspace_size(M, N)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step():
        fl.fl_dropout_layernorm(dx, dr, None, None, s, z, mean, rstd, M, N, "bf16", "bf16", "bf16", eps=1e-5, p=p, seed=seed)
        fl.fl_dropout_layernorm_backward(ddz, None, s, mean, rstd, None, dres, dxo, dg, db, M, N, "bf16", "bf16", "bf16",
                                         workspace=ws, workspace_bytes=n, p=p, seed=seed)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (s, z, dres, dxo, mean, rstd, dg, db):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    check_forward(dict(sum=P.to64(s), z=P.to64(z), mean=P.to64(mean), rstd=P.to64(rstd)), P.to64(x), P.to64(r), None, None, 1e-5, p,
                  seed, 0, ("bf16",) * 3, "graph")
    check_backward(dict(dres=P.to64(dres), dx=P.to64(dxo), dgamma=P.to64(dg), dbeta=P.to64(db)), P.to64(dz), None, P.to64(s),
                   P.to64(mean), P.to64(rstd), None, p, seed, 0, ("bf16",) * 3, "graph")


# ---------------------------------------------------------------- rows that hold infinities
@pytest.mark.parametrize("N", [96, 101, 768, 4096, 4099, 16384, 16400])
@pytest.mark.parametrize("types", [("f32", "f32", "f32", "f32"), ("bf16", "f32", "f16", "f32")])
def test_a_row_with_an_infinity_has_its_mean(fl, N, types):
    """Row 1 holds +inf, row 2 -inf, row 3 both, row 4 a NaN: mean, rstd and z as the definition gives them, other rows as ever."""
    M, xt, zt = 6, types[0], types[2]
    x = draw((M, N), xt, N)
    x[1, 3], x[2, N - 1], x[3, 0], x[3, N - 1], x[4, 5] = float("inf"), -float("inf"), float("inf"), -float("inf"), float("nan")
    z = torch.zeros(M, N, dtype=P.TD[zt], device="cuda")
    mean, rstd = (torch.zeros(M, device="cuda") for _ in range(2))
    fl.fl_dropout_layernorm(x.cuda(), None, None, None, None, z, mean, rstd, M, N, *types, eps=1e-5)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        _, z64, mean64, rstd64 = T.dropout_layernorm(P.to64(x), None, None, None, 1e-5)
    assert np.isinf(mean64[1]) and np.isinf(mean64[2]) and np.isnan(mean64[3]) and np.isnan(mean64[4])
    for got, want, what in ((mean, mean64, "mean"), (rstd, rstd64, "rstd"), (z, z64, "z")):
        got = P.to64(got)
        assert np.array_equal(np.isnan(got), np.isnan(want)), what
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf]) and np.isfinite(got[~inf & ~np.isnan(want)]).all(), what


@pytest.mark.parametrize("N", [96, 101, 4096, 16400])
def test_a_gradient_with_an_infinity_as_the_definition_gives_it(fl, N):
    """dz of row 1 holds an infinity: infinite and NaN places of dres are the definition's, the other rows are as ever."""
    M = 3
    s, dz = draw((M, N), "f32", 1), draw((M, N), "f32", 2)
    dz[1, 4] = float("inf")
    s64 = P.to64(s)
    mean, rstd = s64.mean(axis=1).astype(np.float32), (1 / np.sqrt(s64.var(axis=1) + 1e-5)).astype(np.float32)
    dres = torch.zeros(M, N, device="cuda")
    fl.fl_dropout_layernorm_backward(dz.cuda(), None, s.cuda(), torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda(), None,
                                     dres, None, None, None, M, N, "f32", "f32", "f32")
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        want = T.dropout_layernorm_backward(P.to64(dz), None, s64, mean.astype(np.float64), rstd.astype(np.float64), None)[0]
    got = P.to64(dres)
    assert np.isinf(want[1]).any() and np.isnan(want[1]).any()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert np.isfinite(got[[0, 2]]).all()


def test_a_step_of_an_empty_batch(fl):
    """No rows: every call succeeds on torch's empty tensors, whose address is null, and the parameters' gradients are 0."""
    N, e = 264, torch.empty(0, 264, device="cuda")
    v = torch.empty(0, device="cuda")
    dgamma, dbeta = (torch.full((N,), float("nan"), device="cuda") for _ in range(2))
    fl.fl_dropout(e, e, e, 0, N, "f32", "f32", p=0.1, seed=1)
    fl.fl_dropout_layernorm(e, e, None, None, e, e, v, v, 0, N, "f32", "f32", "f32", p=0.1, seed=1)
    fl.fl_dropout_layernorm_backward(e, e, e, v, v, None, e, e, dgamma, dbeta, 0, N, "f32", "f32", "f32", p=0.1, seed=1)
    torch.cuda.synchronize()
    assert not dgamma.any() and not dbeta.any()
