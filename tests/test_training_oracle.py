"""CPU pins of oracle/training.py: published vectors, finite differences, torch in float64."""
from __future__ import annotations

import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import training as T


def test_philox_published_vectors():
    # the known-answer vectors that its authors publish with the generator (philox4x32, 10 rounds)
    for ctr, key, want in [
        ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
        ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
        ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
         (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
    ]:
        assert tuple(int(v) for v in T.philox4x32(ctr, key)) == want


def test_keep_mask_is_a_place_s_own_number():
    # a row's numbers depend on (m, n) and N alone; element by element from the definition
    M, N, p, seed, off = 5, 11, 0.3, 2**63 + 12345, 2**40 + 9
    mask = T.keep_mask(M, N, p, seed, off)
    thr = int(np.float32(p) * 2.0**32)
    for m in range(M):
        for n in range(N):
            b = m * 3 + n // 4
            w = T.philox4x32((b, 0, off & 0xFFFFFFFF, off >> 32), (seed & 0xFFFFFFFF, seed >> 32))[n % 4]
            assert mask[m, n] == (int(w) >= thr)
    big = T.keep_mask(400, 1000, 0.1, 3, 4)
    # 400000 draws: the share dropped is within five standard deviations of p
    assert abs((~big).mean() - 0.1) < 5 * np.sqrt(0.09 / big.size)


def _diff(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("kind", ["SWIGLU", "GEGLU_TANH"])
def test_gate_against_torch_and_differences(kind):
    v = np.linspace(-8, 8, 401)
    t = torch.from_numpy(v)
    ref = torch.nn.functional.silu(t) if kind == "SWIGLU" else torch.nn.functional.gelu(t, approximate="tanh")
    assert np.abs(T.gate(v, kind) - ref.numpy()).max() < 1e-14
    assert np.abs(T.gate_grad(v, kind) - _diff(lambda x: T.gate(x, kind), v, 1.0)).max() < 1e-8


def test_layernorm_backward_against_differences():
    r = np.random.default_rng(0)
    M, N, p, seed, off, eps = 3, 10, 0.4, 7, 11, 1e-5
    x, res, dz, dsum = (r.standard_normal((M, N)) for _ in range(4))
    gamma, beta = r.standard_normal(N), r.standard_normal(N)

    def loss(x, res, gamma, beta):
        s, z, _, _ = T.dropout_layernorm(x, res, gamma, beta, eps, p, seed, off)
        return (z * dz).sum() + (s * dsum).sum()

    s, _, mean, rstd = T.dropout_layernorm(x, res, gamma, beta, eps, p, seed, off)
    grads = T.dropout_layernorm_backward(dz, dsum, s, mean, rstd, gamma, p, seed, off)
    args = [x, res, gamma, beta]
    for i, g in ((1, grads[0]), (0, grads[1]), (2, grads[2]), (3, grads[3])):
        d = r.standard_normal(args[i].shape)
        f = lambda a, i=i: loss(*[a if j == i else args[j] for j in range(4)])  # noqa: E731
        assert abs(_diff(f, args[i], d) - (g * d).sum()) < 1e-7
    z = torch.nn.functional.layer_norm(torch.from_numpy(s), (N,), torch.from_numpy(gamma), torch.from_numpy(beta), eps)
    assert np.abs(z.numpy() - T.dropout_layernorm(x, res, gamma, beta, eps, p, seed, off)[1]).max() < 1e-13


@pytest.mark.parametrize("kind", ["SWIGLU", "GEGLU_TANH"])
def test_gated_block_gradients_against_differences(kind):
    r = np.random.default_rng(1)
    M, N, K, D = 4, 6, 5, 3
    x, W, Wd = r.standard_normal((M, K)), r.standard_normal((2 * N, K)), r.standard_normal((D, N))
    dy = r.standard_normal((M, D))
    h, gu = T.glu(x, W, kind)
    assert np.allclose(h, [[T.gate(x[m] @ W[n], kind) * (x[m] @ W[N + n]) for n in range(N)] for m in range(M)])
    dgu, dh = T.glu_backward(dy, Wd, gu, kind)
    assert np.allclose(dh, dy @ Wd)

    def loss(x, W, Wd):
        return ((T.glu(x, W, kind)[0] @ Wd.T) * dy).sum()

    for i, g in ((0, dgu @ W), (1, T.weight_grad(dgu, x)), (2, T.weight_grad(dy, h))):
        args = [x, W, Wd]
        d = r.standard_normal(args[i].shape)
        f = lambda a, i=i, args=args: loss(*[a if j == i else args[j] for j in range(3)])  # noqa: E731
        assert abs(_diff(f, args[i], d) - (g * d).sum()) < 1e-6
    assert np.allclose(T.weight_grad(dy, h, Wd, 0.5), 0.5 * (dy.T @ h + Wd))


def test_the_kernels_generator_on_the_host(tmp_path):
    """The row kernels' own generator, whose first two rounds are folded, compiled for the host by nvcc: the published vectors,
    and random counters and keys; blocks from 2^32 on (matrices of 2^34 elements) in the form that holds their high half."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("needs nvcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / "philox_check"
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a",
                        os.path.join(root, "tests", "c", "philox_check.cu"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    rng = np.random.default_rng(5)
    words = [int(v) for v in rng.integers(0, 2**64, 300, dtype=np.uint64)]
    cases = [(big, block >> (0 if big else 32), seed, off) for big in (0, 1)
             for block, seed, off in zip(words[::3], words[1::3], words[2::3])]
    cases += [(0, 0, 0, 0), (1, 0, 0, 0), (1, 2**64 - 1, 2**64 - 1, 2**64 - 1), (1, 2**32, 7, 9), (1, 2**32 - 1, 7, 9), (0, 2**32 - 1, 7, 9),
              (1, 0x85A308D3243F6A88, 0x299F31D0A4093822, 0x0370734413198A2E)]
    r = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True, timeout=120)
    got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert r.returncode == 0 and len(got) == len(cases)
    half = 0xFFFFFFFF
    for (big, block, seed, off), words4 in zip(cases, got):
        want = T.philox4x32((block & half, block >> 32, off & half, off >> 32), (seed & half, seed >> 32))
        assert words4 == tuple(int(v) for v in want), (big, hex(block), hex(seed), hex(off))
