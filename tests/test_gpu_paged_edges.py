"""Calls of the paged-cache operators at the edges of what they allow: arguments on the device that
are out of range, sequences that are skipped, and values that are not finite.
"""

import numpy as np
import pytest
import torch

from tests._paged import Batch
from tests._util import to_f64
from tests.test_gpu_paged import (FULL, check, check_batch, fused, run_chunk, run_decode,  # noqa: F401
                                  swa)

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


def nan_memory(*shapes):
    """Leaves NaN in the blocks that the next tensors of these shapes get."""
    held = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for shape, dtype in shapes]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("cu,first,skipped", [
    ([0, 20, 50, 60], [5, -1, 0], [(20, 50)]),                    # a negative start
    ([0, 20, 50, 60], [1 << 62, 100, 0], [(0, 20)]),              # an end past the table
    ([0, 20, 50, 61], [5, 100, 0], [(50, 60)]),                   # offsets past the tokens
    ([-4, 20, 50, 60], [5, 100, 0], [(0, 20)]),                   # offsets before them
    ([3, 20, 50, 56], [5, -7, 0], [(0, 3), (20, 50), (56, 60)]),  # and padding on either side
    ([0, 20, 50, 60], [-1, -1, -1], [(0, 60)]),
    ([0, 60, 60, 60], [-1, 100, 0], [(0, 60)]),
])
def test_chunk_rows_of_skipped_sequences_are_zero(swa, cu, first, skipped):
    """In tensors that the call allocates every row that no sequence writes is zero."""
    b = Batch([20, 30, 10], [5, 100, 0], 4, 2, 64, 16, 64, 0)
    t_cu = torch.tensor(cu, dtype=torch.int64, device="cuda")
    t_first = torch.tensor(first, dtype=torch.int64, device="cuda")
    q = b.q.cuda()
    nan_memory(((60, 4, 64), torch.bfloat16), ((4, 60), torch.float32))
    out, lse = swa.swa_attn_chunk_paged(q, b.k_cache, b.v_cache, b.t_table, t_cu, t_first, b.W,
                                        b.scale, return_lse=True)
    assert swa.swa_get_device_status() == 6
    zero = torch.zeros(60, dtype=torch.bool)
    for lo, hi in skipped:
        zero[lo:hi] = True
    zero = zero.cuda()
    assert bool((out[zero] == 0).all()) and bool((lse[:, zero] == 0).all())
    written = out[~zero].float().abs().amax(-1)  # a row of d values is not all zero by chance
    assert bool((written > 0).all()) and bool(torch.isfinite(lse[:, ~zero]).all())


@pytest.mark.parametrize("cu", [[0, 20, 10, 60], [50, 0, 60, 60], [10, 40, 20, 30], [60, 0, 0, 60],
                                [0, 60, 59, 60], [0, 5, (1 << 63) - 1, -1]])
def test_chunk_skips_all_under_disordered_offsets(swa, cu):
    """Offsets out of order: flagged, rows of new tensors are zero, the caller's are left."""
    b = Batch([20, 30, 10], [5, 100, 0], 4, 2, 64, 16, 64, 0)
    t_cu = torch.tensor(cu, device="cuda")
    args = (b.q.cuda(), b.k_cache, b.v_cache, b.t_table, t_cu, b.t_first, b.W, b.scale)
    nan_memory(((60, 4, 64), torch.bfloat16), ((4, 60), torch.float32))
    out, lse = swa.swa_attn_chunk_paged(*args, return_lse=True)
    assert swa.swa_get_device_status() == 6
    assert bool((out == 0).all()) and bool((lse == 0).all())
    out.fill_(7)
    lse.fill_(7)
    swa.swa_attn_chunk_paged(*args, out=out, lse=lse)
    assert swa.swa_get_device_status() == 6
    assert bool((out == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("start", [-1, 1 << 20, (1 << 63) - 1])
def test_empty_sequences_may_have_any_start(swa, start):
    """A batch of fixed size padded with empty sequences: no flag, by append or by attention."""
    b = Batch([3, 0, 40, 0], [7, 0, 130, 0], 4, 2, 64, 16, 50, 2)
    first = b.t_first.clone()
    first[1] = first[3] = start
    out, lse = swa.swa_attn_chunk_paged(b.q.cuda(), b.k_cache, b.v_cache, b.t_table, b.t_cu, first,
                                        b.W, b.scale, n_sink=2, return_lse=True)
    assert swa.swa_get_device_status() == 0
    check_batch(b, out, lse.T)
    k = torch.randn((43, 2, 64), device="cuda").bfloat16()
    swa.swa_paged_append(k, k, b.k_cache, b.v_cache, b.t_table, b.t_cu, first)
    assert swa.swa_get_device_status() == 0
    none = torch.zeros_like(b.t_cu)
    out = swa.swa_attn_chunk_paged(b.q.cuda(), b.k_cache, b.v_cache, b.t_table, none,
                                   torch.full_like(first, start), b.W, b.scale)
    assert swa.swa_get_device_status() == 0
    assert bool((out == 0).all())


def not_finite(b, q, k):
    """[tokens, H] rows whose softmax has a NaN or +infinity among its seen scores; q [tokens, H, d]
    and the one sequence's keys k [positions, Hkv, d] in 64 bits."""
    n, H, d = q.shape
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.einsum("thgd,khd->thgk", q.reshape(n, b.Hkv, H // b.Hkv, d), k)
    qp = b.starts[0] + np.arange(n)
    seen = (b.pos_of[0] <= qp[:, None]) & (b.pos_of[0] > qp[:, None] - b.W)
    return ((np.isnan(x) | np.isposinf(x)) & seen[:, None, None]).any(-1).reshape(n, H)


@pytest.mark.parametrize("what", ["key", "query"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [10, 700, 15000, 30010])
def test_a_nan_is_not_lost_between_parts(swa, what, value, at):
    """Few rows over many keys, so the work of a row is cut into parts: a NaN or infinite score in
    any of them makes the row and its log-sum-exp NaN, and no other row."""
    b = Batch([17], [30000], 8, 2, 128, 16, FULL, 0)
    q = b.q.cuda()
    page, slot = int(b.table[0, at // 16]), at % 16
    if what == "key":
        b.k_cache[page, 1, slot, 5] = value
        b.keys[0][at, 1, 5] = value
    else:
        q[at % 17, at % 8, 5] = value
    bad = not_finite(b, to_f64(q), b.keys[0].double().numpy())
    assert bad.any() and not bad.all()
    out, lse = swa.swa_attn_chunk_paged(q, b.k_cache, b.v_cache, b.t_table, b.t_cu, b.t_first, b.W,
                                        b.scale, return_lse=True)
    assert np.array_equal(np.isnan(to_f64(lse.T)), bad)
    assert np.array_equal(np.isnan(to_f64(out)).any(-1), bad)
    assert np.array_equal(np.isnan(to_f64(out)).all(-1), bad)
    # the last token alone
    out, lse = swa.swa_attn_decode_paged(q[-1:], b.k_cache, b.v_cache, b.t_table, b.t_first + 16,
                                         b.W, b.scale, return_lse=True)
    bad = bad[-1:]
    assert np.array_equal(np.isnan(to_f64(lse)), bad)
    assert np.array_equal(np.isnan(to_f64(out)).any(-1), bad)
    assert np.array_equal(np.isnan(to_f64(out)).all(-1), bad)


def test_a_nan_query_in_one_part(swa):
    """A row whose work is one part, or one warp's keys: output and log-sum-exp are NaN."""
    b = Batch([1] * 4, [0, 3, 200, 17], 8, 2, 64, 16, FULL, 0)
    q = b.q.cuda()
    q[1, 2, 0] = q[2, 7, 63] = q[0, 0, 9] = float("nan")
    for out, lse in (swa.swa_attn_decode_paged(q, b.k_cache, b.v_cache, b.t_table, b.t_first, b.W,
                                               b.scale, return_lse=True),
                     swa.swa_attn_chunk_paged(q, b.k_cache, b.v_cache, b.t_table, b.t_cu,
                                              b.t_first, b.W, b.scale, return_lse=True)):
        if lse.shape != (4, 8):
            lse = lse.T
        bad = torch.isnan(q).any(-1)
        assert torch.equal(torch.isnan(lse), bad)
        assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(
            torch.isnan(out).any(-1), bad)


@pytest.mark.parametrize("first_seen", [130, 1300, 20000])
def test_keys_of_the_lowest_value(swa, first_seen):
    """The keys before first_seen hold the type's lowest value in one dimension, so that their scores
    are -infinity in 32 bits and their weights zero: the rows are those of the keys behind them."""
    n = first_seen + 300
    b = Batch([1], [n - 1], 8, 2, 64, 16, FULL, 0)
    b.q[:, :, 0] = 4.0
    lowest = torch.finfo(torch.bfloat16).min
    at = torch.from_numpy(b.table[0, np.arange(first_seen) // 16].astype(np.int64)).cuda()
    slot = torch.from_numpy(np.arange(first_seen) % 16).cuda()
    b.k_cache[at, :, slot, 0] = lowest
    # the definition on the keys behind: a window of the 300 last positions
    near = Batch([1], [n - 1], 8, 2, 64, 16, 300, 0)
    near.q, near.pos_of = b.q, [np.arange(first_seen, n)]
    near.keys, near.vals = [b.keys[0][first_seen:]], [b.vals[0][first_seen:]]
    for run in (run_decode, run_chunk):
        out, lse = run(swa, b)
        check_batch(near, out, lse.T if run is run_chunk else lse)
    assert swa.swa_get_device_status() == 0


@pytest.mark.parametrize("pos,H,Hkv,d,page", [
    ([1, 2, 4, 7, 12, 15, 30, 61], 32, 8, 64, 16),
    ([3, 9, 33, 100], 40, 2, 128, 32),
])
def test_decode_weights_keep_32_bits(swa, pos, H, Hkv, d, page):
    """The weights reach the second product with an error of 2^-16, as two terms of 16 bits: each
    term is rounded by at most 2^-8 of what it stands for, the second stands for the first one's
    rounding.  (With one term the weights are off by up to 2^-8.)"""
    b = Batch([1] * len(pos), pos, H, Hkv, d, page, FULL, 0, seed=11)
    out, lse = run_decode(swa, b)
    want, want_lse, tol, tol_lse = b.expect()
    b.vals = [v.abs() for v in b.vals]
    mean_abs = b.expect()[0]  # the weighted mean of |v|
    tol -= (2.0 ** -8 - 2.0 ** -16) * mean_abs * (1 + 2.0 ** -8)
    check(to_f64(out), want, tol, "out")
    check(to_f64(lse), want_lse, tol_lse, "lse")


def test_workspaces_that_share_memory_are_refused(swa):
    """A workspace of enough elements that lie on one another, or not side by side."""
    b = Batch([1] * 2, [5, 100], 4, 2, 64, 16, 64, 0)
    need = max(swa.swa_chunk_paged_workspace_bytes(2, 2, 4, 2, 64),
               swa.swa_decode_paged_workspace_bytes(2, 4, 2, 64))
    one = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for bad in (one[:1].expand(need), one.expand(need // 256 + 1, 256),
                torch.zeros((need, 2), dtype=torch.uint8, device="cuda")[:, 0]):
        for run in (run_chunk, run_decode):
            with pytest.raises(ValueError):
                run(swa, b, workspace=bad)
    for run in (run_chunk, run_decode):
        with pytest.raises(TypeError):
            run(swa, b, workspace=need)
    good = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for run in (run_chunk, run_decode):
        out, lse = run(swa, b, workspace=good)
        check_batch(b, out, lse.T if run is run_chunk else lse)
