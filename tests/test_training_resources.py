"""Registers and spills of the training kernels, from the assembler's report that build.py keeps."""
from __future__ import annotations

import re

import pytest

from tests.test_resources import _entries, _select


@pytest.mark.parametrize("prefix,threads,ctas", [
    ("_ZN2fl15fl_pair_tcgen05", 320, 1),        # one CTA of ten warps per SM, no spills
    ("_ZN2fl19fl_glu_small_kernelILi0ELi0ELi1E", 256, 2),  # few rows: two CTAs of eight warps
    ("_ZN2fl19fl_glu_small_kernelILi0ELi1ELi1E", 256, 2),
    ("_ZN2fl17fl_dropout_kernelILi0E", 256, 8),  # the typed dropout: every warp an SM holds
    ("_ZN2fl17fl_dropout_kernelILi1E", 256, 8),
    ("_ZN2fl20fl_dropout_ln_kernelILi256ELi2ELi1E", 256, 2),
    ("_ZN2fl24fl_dropout_ln_bwd_kernelILi256ELi2ELi1E", 256, 1),
])
def test_kernels_keep_their_ctas_and_do_not_spill(prefix, threads, ctas):
    for name, v in _select(_entries(), prefix).items():
        assert v["regs"] * threads * ctas <= 65536, (name, v)
        # (the long sums hold 128 of the 168 registers that ten warps leave a thread; a few of the others wait in memory)
        long_sums = name.startswith(("_ZN2fl15fl_pair_tcgen05ILi7E", "_ZN2fl15fl_pair_tcgen05ILi8E"))
        assert v["spill"] <= (192 if long_sums else 0), (name, v)


def _row_kernels(prefix):
    """(T, V, untyped, regs, spill) of every instantiation <T, V, XT, ST, ZT>."""
    for name, v in _select(_entries(), prefix).items():
        args = re.match(r"_ZN2fl\d+fl_dropout_ln(?:_bwd)?_kernelILi(\d+)ELi(\d+)ELi(n?\d)E", name).groups()
        yield int(args[0]), int(args[1]), args[2] == "n1", v["regs"], v["spill"], name


@pytest.mark.parametrize("prefix,kernels,block", [("_ZN2fl20fl_dropout_ln_kernel", 12, 128),
                                                  ("_ZN2fl24fl_dropout_ln_bwd_kernel", 11, 256)])
def test_every_row_kernel_fits_its_threads_and_does_not_spill(prefix, kernels, block):
    """Every length of row in every type.  The 1024-thread forms, which have 64 registers a thread, may store and load 16 bytes
    together (typed) or 64 (untyped)."""
    seen = set()
    for T, V, untyped, regs, spill, name in _row_kernels(prefix):
        seen.add((T, V))
        assert regs * max(T, block) <= 65536, name
        assert spill <= (0 if T < 1024 else 64 if untyped else 16), (name, spill)
    assert len(seen) == kernels, sorted(seen)
