"""Registers and spills of the training kernels, from the assembler's report that build.py keeps."""
from __future__ import annotations

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
