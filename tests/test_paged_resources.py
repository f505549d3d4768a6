"""Compiler resources of the paged-cache kernels (CPU, needs nvcc).

The chunk kernel re-splits the 168 registers per thread that it is launched with, like the other
forward kernels; the decode kernel keeps Q, the output and a tile's scores in registers.  Neither
may spill.
"""

import re

import pytest

from tests.test_build_resources import NVCC, _fwd2_launch_regs, report  # noqa: F401
from tests.test_build_resources import pytestmark as needs_nvcc

pytestmark = needs_nvcc


def _kernels(report, name):  # noqa: F811
    return {n: r for n, r in report.items() if re.search(rf"\d{name}", n)}


def test_chunk_kernel_registers(report):  # noqa: F811
    found = _kernels(report, "paged_fwd_kernelI")
    assert len(found) == 2  # d = 64 and 128
    for name, r in found.items():
        assert r["regs"] == _fwd2_launch_regs(), (name, r)


@pytest.mark.parametrize("name,count", [
    ("paged_fwd_kernelI", 2), ("paged_fwd_merge_kernelI", 2), ("paged_decode_kernelI", 2),
    ("paged_decode_merge_kernelI", 2), ("paged_append_kernelI", 8),
])
def test_no_spills(report, name, count):  # noqa: F811
    found = _kernels(report, name)
    assert len(found) == count, sorted(found)
    for n, r in found.items():
        assert r.get("spill", 0) == 0, (n, r)
