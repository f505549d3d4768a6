"""Calls of the paged-cache operators at the edges of what they allow: arguments on the device that
are out of range, sequences that are skipped, and values that are not finite.
"""

import numpy as np
import pytest
import torch

from tests._paged import Batch
from tests._util import to_f64
from tests.test_gpu_paged import check, fused, swa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start", [(1 << 63) - 1, (1 << 63) - 5, (1 << 63) - 900, -1 << 63])
@pytest.mark.parametrize("n", [20, 900])  # a CTA and a warp per token
def test_append_refuses_starts_at_the_ends_of_64_bits(swa, start, n):
    """start + t passes 2^63: no slot is written, the queries are zeros, other sequences are right."""
    rng = np.random.default_rng(6)
    k, q = fused(rng, 4 + n, 2, 64, 0), fused(rng, 4 + n, 4, 64, 0)
    kd = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vd = torch.zeros_like(kd)
    table = torch.tensor([[3], [0]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4, 4 + n], device="cuda")
    first = torch.tensor([5, start], dtype=torch.int64, device="cuda")
    out = swa.swa_paged_append(k, k, kd, vd, table, cu, first, q=q)
    assert swa.swa_get_device_status() == 6
    for c in (kd, vd):
        assert torch.equal(c[3, :, 5:9].transpose(0, 1), k[:4])
        c[3, :, 5:9] = 0
        assert not bool(c.any())
    assert torch.equal(out[:4], q[:4]) and not bool(out[4:].any())


@pytest.mark.parametrize("start", [(1 << 63) - 1, (1 << 63) - 25, (1 << 63) - 30, -1 << 63])
@pytest.mark.parametrize("which", [0, 2])
def test_chunk_refuses_starts_at_the_ends_of_64_bits(swa, start, which):
    """start + 30 passes 2^63 (or stays below it by nothing): flagged, no row written, others right."""
    b = Batch([30, 12, 30], [5, 100, 0], 4, 2, 64, 16, 64, 2)
    first = b.t_first.clone()
    first[which] = start
    out = torch.full((72, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 72), 7.0, device="cuda")
    swa.swa_attn_chunk_paged(b.q.cuda(), b.k_cache, b.v_cache, b.t_table, b.t_cu, first, b.W,
                             b.scale, n_sink=2, out=out, lse=lse)
    assert swa.swa_get_device_status() == 6
    want, want_lse, tol, tol_lse = b.expect()
    for i in range(3):
        rows = slice(int(b.cu[i]), int(b.cu[i + 1]))
        if i == which:
            assert bool((out[rows] == 7).all()) and bool((lse[:, rows] == 7).all())
        else:
            check(to_f64(out[rows]), want[rows], tol[rows], "out")
            check(to_f64(lse[:, rows].T), want_lse[rows], tol_lse[rows], "lse")
