"""CPU tests of the training entry points' refusals: each documented status before any CUDA call."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def fl():
    from gemm_bias_activation_tcgen05_b200 import build
    build.build()
    import gemm_bias_activation_tcgen05_b200 as m
    return m


def test_dropout_descriptor_matches_the_header(fl, tmp_path):
    c = tmp_path / "t.c"
    c.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fused_linear.h"\nint main(void) {\n'
                 '  printf("%zu %zu %zu %zu %zu\\n", sizeof(fl_dropout_desc), offsetof(fl_dropout_desc, p),\n'
                 '         offsetof(fl_dropout_desc, seed), offsetof(fl_dropout_desc, offset), offsetof(fl_dropout_desc, offset_dev));\n'
                 '  return 0;\n}\n')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    vals = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    D = fl.fl_dropout_desc
    assert vals == [ctypes.sizeof(D), D.p.offset, D.seed.offset, D.offset.offset, D.offset_dev.offset]


def _drop(fl, p=0.1, reserved=0, dev=None):
    return ctypes.byref(fl.fl_dropout_desc(p, reserved, 1, 2, dev))


def _dropout(fl, x=16, r=None, y=16, M=4, N=4, ldx=0, ldr=0, ldy=0, xt=1, yt=1, drop=None):
    return fl.LIB.fl_dropout(x, r, y, M, N, ldx, ldr, ldy, xt, yt, drop, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), "FL_ERR_INVALID_ARG"), (dict(y=None), "FL_ERR_INVALID_ARG"), (dict(M=-1), "FL_ERR_INVALID_ARG"),
    (dict(N=-1), "FL_ERR_INVALID_ARG"), (dict(N=2**31), "FL_ERR_INVALID_ARG"), (dict(M=2**31), "FL_ERR_INVALID_ARG"),
    (dict(xt=3), "FL_ERR_INVALID_ARG"), (dict(yt=-1), "FL_ERR_INVALID_ARG"), (dict(ldx=3), "FL_ERR_INVALID_ARG"),
    (dict(r=16, ldr=2), "FL_ERR_INVALID_ARG"), (dict(ldy=-4), "FL_ERR_INVALID_ARG"), (dict(x=17), "FL_ERR_ALIGNMENT"),
    (dict(y=18, yt=2), "FL_ERR_ALIGNMENT"), (dict(p=1.0), "FL_ERR_INVALID_ARG"), (dict(p=-0.1), "FL_ERR_INVALID_ARG"),
    (dict(p=float("nan")), "FL_ERR_INVALID_ARG"), (dict(reserved=1), "FL_ERR_INVALID_ARG"), (dict(dev=20), "FL_ERR_ALIGNMENT"),
    (dict(M=0), "FL_OK"), (dict(N=0), "FL_OK"),
])
def test_dropout_refusals(fl, kw, status):
    d = {k: kw.pop(k) for k in ("p", "reserved", "dev") if k in kw}
    st = _dropout(fl, drop=_drop(fl, **d), **kw)
    assert fl.STATUS_NAMES[st] == status, fl.fl_last_error()
    assert (st == fl.FL_OK) == (fl.fl_last_error() == "")


def _forward(fl, x=16, r=None, g=None, b=None, s=None, z=16, mean=None, rstd=None, M=4, N=4, lds=(0, 0, 0, 0),
             types=(1, 1, 1, 1), eps=1e-5, drop=None):
    return fl.LIB.fl_dropout_layernorm(x, r, g, b, s, z, mean, rstd, M, N, *lds, *types, eps, drop, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), "FL_ERR_INVALID_ARG"), (dict(z=None), "FL_ERR_INVALID_ARG"), (dict(mean=16), "FL_ERR_INVALID_ARG"),
    (dict(rstd=16), "FL_ERR_INVALID_ARG"), (dict(M=-1), "FL_ERR_INVALID_ARG"), (dict(eps=-1.0), "FL_ERR_INVALID_ARG"),
    (dict(eps=float("nan")), "FL_ERR_INVALID_ARG"), (dict(types=(1, 1, 1, 9)), "FL_ERR_INVALID_ARG"),
    (dict(types=(1, 9, 1, 1)), "FL_ERR_INVALID_ARG"), (dict(lds=(3, 0, 0, 0)), "FL_ERR_INVALID_ARG"),
    (dict(r=16, lds=(0, 3, 0, 0)), "FL_ERR_INVALID_ARG"), (dict(s=16, lds=(0, 0, 3, 0)), "FL_ERR_INVALID_ARG"),
    (dict(lds=(0, 0, 0, 3)), "FL_ERR_INVALID_ARG"), (dict(g=17), "FL_ERR_ALIGNMENT"), (dict(b=17), "FL_ERR_ALIGNMENT"),
    (dict(mean=18, rstd=16), "FL_ERR_ALIGNMENT"), (dict(s=17), "FL_ERR_ALIGNMENT"), (dict(M=0), "FL_OK"), (dict(N=0), "FL_OK"),
])
def test_forward_refusals(fl, kw, status):
    st = _forward(fl, **kw)
    assert fl.STATUS_NAMES[st] == status, fl.fl_last_error()


def _backward(fl, dz=16, dsum=None, s=16, mean=16, rstd=16, g=None, dres=16, dx=None, dg=None, db=None, M=4, N=4,
              lds=(0, 0, 0, 0, 0), types=(1, 1, 1, 1), drop=None, ws=None, n=0):
    return fl.LIB.fl_dropout_layernorm_backward(dz, dsum, s, mean, rstd, g, dres, dx, dg, db, M, N, *lds, *types, drop, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dz=None), "FL_ERR_INVALID_ARG"), (dict(s=None), "FL_ERR_INVALID_ARG"), (dict(mean=None), "FL_ERR_INVALID_ARG"),
    (dict(rstd=None), "FL_ERR_INVALID_ARG"), (dict(dres=None), "FL_ERR_INVALID_ARG"), (dict(N=-2), "FL_ERR_INVALID_ARG"),
    (dict(types=(7, 1, 1, 1)), "FL_ERR_INVALID_ARG"), (dict(lds=(3, 0, 0, 0, 0)), "FL_ERR_INVALID_ARG"),
    (dict(dsum=16, lds=(0, 3, 0, 0, 0)), "FL_ERR_INVALID_ARG"), (dict(lds=(0, 0, 3, 0, 0)), "FL_ERR_INVALID_ARG"),
    (dict(lds=(0, 0, 0, 3, 0)), "FL_ERR_INVALID_ARG"), (dict(dx=16, lds=(0, 0, 0, 0, 3)), "FL_ERR_INVALID_ARG"),
    (dict(dz=17), "FL_ERR_ALIGNMENT"), (dict(dg=18), "FL_ERR_ALIGNMENT"), (dict(mean=18), "FL_ERR_ALIGNMENT"),
    (dict(g=17), "FL_ERR_ALIGNMENT"),
])
def test_backward_refusals(fl, kw, status):
    st = _backward(fl, **kw)
    assert fl.STATUS_NAMES[st] == status, fl.fl_last_error()


def test_workspace_refusals(fl):
    n = ctypes.c_size_t()
    assert fl.LIB.fl_layernorm_grad_workspace_size(4, 4, None) == fl.FL_ERR_INVALID_ARG
    assert fl.LIB.fl_layernorm_grad_workspace_size(-1, 4, ctypes.byref(n)) == fl.FL_ERR_INVALID_ARG
    assert fl.LIB.fl_layernorm_grad_workspace_size(4, 2**31, ctypes.byref(n)) == fl.FL_ERR_INVALID_ARG


# ---------------------------------------------------------------- the gated linear units and the weight gradient
def _plan(fl, kind, M=256, N=256, K=64, dtype="bf16", **epi):
    e = fl.make_epilogue(kind=kind, **epi)
    info = fl.fl_plan_info()
    st = fl.LIB.fl_plan_preview(M, N, K, fl.DTYPES[dtype], fl.COMPUTES["32F_3XTF32" if dtype == "f32" else "32F"], ctypes.byref(e), 148,
                                232448, ctypes.byref(info))
    return st, info


@pytest.mark.parametrize("kind,kw,status", [
    ("SWIGLU", dict(b_major=1), "FL_ERR_UNSUPPORTED"), ("SWIGLU", dict(out_dtype="f32"), "FL_ERR_UNSUPPORTED"),
    ("SWIGLU", dict(dtype="f32"), "FL_ERR_UNSUPPORTED"), ("SWIGLU", dict(unfused=True), "FL_ERR_UNSUPPORTED"),
    ("SWIGLU", dict(has_residual=True), "FL_ERR_UNSUPPORTED"), ("SWIGLU", dict(scale=0.5), "FL_ERR_UNSUPPORTED"),
    ("SWIGLU", dict(schedule="stream_k"), "FL_ERR_UNSUPPORTED"), ("SWIGLU", dict(K=60), "FL_ERR_ALIGNMENT"),
    ("SWIGLU", dict(N=100, ldo=100), "FL_ERR_ALIGNMENT"), ("SWIGLU", dict(N=100, ldo=104), "FL_OK"),
    ("SWIGLU_AUX", dict(N=100, ldo=104), "FL_ERR_ALIGNMENT"), ("GEGLU_TANH_AUX", dict(N=104), "FL_OK"),
    ("DSWIGLU", dict(), "FL_ERR_UNSUPPORTED"), ("DSWIGLU", dict(b_major=1), "FL_OK"),
    ("DSWIGLU", dict(b_major=1, ldo=504), "FL_ERR_INVALID_ARG"), ("DSWIGLU", dict(b_major=1, N=100, ldb=104, ldo=208), "FL_ERR_ALIGNMENT"),
    ("DGEGLU_TANH", dict(b_major=1, out_dtype="f32"), "FL_ERR_UNSUPPORTED"), ("DGEGLU_TANH", dict(b_major=1, scale=2.0), "FL_ERR_UNSUPPORTED"),
    ("WGRAD", dict(), "FL_ERR_UNSUPPORTED"), ("WGRAD", dict(b_major=1, out_dtype="f32", K=77), "FL_OK"),
    ("WGRAD", dict(b_major=1, lda=248), "FL_ERR_INVALID_ARG"), ("WGRAD", dict(b_major=1, M=250), "FL_ERR_ALIGNMENT"),
    ("WGRAD", dict(b_major=1, M=250, lda=256, has_residual=True, scale=0.5), "FL_OK"),
    ("WGRAD", dict(b_major=1, dtype="f32"), "FL_ERR_UNSUPPORTED"), ("WGRAD", dict(b_major=1, K=-1), "FL_ERR_INVALID_ARG"),
])
def test_pair_kind_refusals(fl, kind, kw, status):
    st, _ = _plan(fl, kind, **kw)
    assert fl.STATUS_NAMES[st] == status, fl.fl_last_error()
    # fl_execute_noalloc refuses the same, before any device call
    if st != fl.FL_OK:
        shape = {k: kw.get(k, d) for k, d in (("M", 256), ("N", 256), ("K", 64))}
        dtype = kw.get("dtype", "bf16")
        e = fl.make_epilogue(kind=kind, **{k: v for k, v in kw.items() if k not in ("M", "N", "K", "dtype")})
        assert fl.LIB.fl_execute_noalloc(shape["M"], shape["N"], shape["K"], fl.DTYPES[dtype],
                                         fl.COMPUTES["32F_3XTF32" if dtype == "f32" else "32F"], ctypes.byref(e), 16, 16, None, None,
                                         None, 16, None) == st


@pytest.mark.parametrize("kind", ["SWIGLU", "SWIGLU_AUX", "DSWIGLU", "WGRAD"])
def test_pair_configurations(fl, kind):
    """Every choice fits the GPU: shared memory, stages, whole pairs, splits no more than K blocks."""
    import random
    rng = random.Random(kind)
    for _ in range(300):
        M, N, K = (8 * rng.randint(1, 1500) for _ in range(3))
        st, i = _plan(fl, kind, M, N, K, b_major=int(kind in ("DSWIGLU", "WGRAD")), out_dtype=rng.choice(["bf16", "f16"]))
        assert st == fl.FL_OK, fl.fl_last_error()
        if i.cta_pair:
            assert i.smem_bytes <= 232448 and i.stages >= 3 and i.grid % 2 == 0 and 0 < i.grid <= 148
            assert 1 <= i.split_k <= max(1, -(-K // 64)) and (i.split_k == 1 or i.split_k * -(-M // 256) * -(-N // i.tile_n) <= 148)
        assert i.launches_per_execute == (2 if i.split_k > 1 else 1)


@pytest.mark.parametrize("M,N", [(0, 8), (8, 0), (0, 0)])
def test_empty_matrices_have_no_addresses(fl, M, N):
    """The pointer of an empty tensor is null: an empty batch is no error."""
    none = dict(M=M, N=N)
    assert _dropout(fl, x=None, y=None, **none) == fl.FL_OK, fl.fl_last_error()
    assert _forward(fl, x=None, z=None, **none) == fl.FL_OK, fl.fl_last_error()
    assert _backward(fl, dz=None, s=None, mean=None, rstd=None, dres=None, **none) == fl.FL_OK, fl.fl_last_error()
    # what is wrong stays wrong
    assert _dropout(fl, x=None, y=None, M=M, N=N, xt=9) == fl.FL_ERR_INVALID_ARG
    assert _forward(fl, x=None, z=None, M=M, N=N, eps=-1.0) == fl.FL_ERR_INVALID_ARG
    assert _dropout(fl, x=None, y=None, M=-1, N=N) == fl.FL_ERR_INVALID_ARG
