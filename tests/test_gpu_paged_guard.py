"""Guard bands around every buffer the paged-cache operators write.

As in test_gpu_guard_bands: each output, workspace and cache lies inside a larger buffer whose
margins must be bit-identical after the call, and the guarded results equal, bit for bit, those on
plainly allocated buffers.
"""

import pytest
import torch

from tests._paged import Batch
from tests.test_gpu_guard_bands import OFFSETS, Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def swa(cuda_ok):
    import sliding_window_sparse_b200 as m

    return m


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (7, 1, 64), (4, 4, 64)])
def test_chunk(swa, offset, H, Hkv, d):
    b = Batch([130, 0, 33, 1], [70, 5, 900, 4000], H, Hkv, d, 16, 300, 3, "nhd", trail=9)
    args = (b.q.cuda(), b.k_cache, b.v_cache, b.t_table, b.t_cu, b.t_first, 300, b.scale)
    want = swa.swa_attn_chunk_paged(*args, n_sink=3, return_lse=True)
    out = Guarded((b.total, H, d), torch.bfloat16, offset, fill=torch.zeros(()))
    lse = Guarded((H, b.total), torch.float32, offset, fill=torch.zeros(()))
    ws = Guarded((swa.swa_chunk_paged_workspace_bytes(4, b.total, H, Hkv, d),), torch.uint8, 0)
    swa.swa_attn_chunk_paged(*args, n_sink=3, out=out.t, lse=lse.t, workspace=ws.t)
    assert all(g.margins_intact() for g in (out, lse, ws))
    assert torch.equal(out.t, want[0]) and torch.equal(lse.t, want[1])
    assert swa.swa_get_device_status() == 0


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 128), (7, 1, 64), (40, 2, 64)])
def test_decode(swa, offset, H, Hkv, d):
    pos = [700, 0, 129, 4000, 15]
    b = Batch([1] * 5, pos, H, Hkv, d, 16, 300, 3, "hnd")
    b.t_first[2] = -1
    args = (b.q.cuda(), b.k_cache, b.v_cache, b.t_table, b.t_first, 300, b.scale)
    want = swa.swa_attn_decode_paged(*args, n_sink=3, return_lse=True)
    out = Guarded((5, H, d), torch.bfloat16, offset)
    lse = Guarded((5, H), torch.float32, offset)
    ws = Guarded((swa.swa_decode_paged_workspace_bytes(5, H, Hkv, d),), torch.uint8, 0)
    swa.swa_attn_decode_paged(*args, n_sink=3, out=out.t, lse=lse.t, workspace=ws.t)
    assert all(g.margins_intact() for g in (out, lse, ws))
    assert torch.equal(out.t, want[0]) and torch.equal(lse.t, want[1])
    assert swa.swa_get_device_status() == 0


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("n", [5, 900])  # a CTA and a warp per token
def test_append(swa, offset, n):
    H, Hkv, d, page = 6, 2, 64, 24
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn((n, Hkv, d), generator=g, device="cuda").bfloat16()
    q = torch.randn((n, H, d), generator=g, device="cuda").bfloat16()
    pages = n // page + 2
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    cu = torch.tensor([0, n], device="cuda")
    start = torch.tensor([13], device="cuda")
    inv = torch.rand(16, generator=g, device="cuda")
    zero = torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    kc, vc = zero.clone(), zero.clone()
    want = swa.swa_paged_append(k, -k, kc, vc, table, cu, start, q=q, inv_freq=inv)
    gk, gv = (Guarded(zero.shape, torch.bfloat16, offset, fill=zero) for _ in range(2))
    gq = Guarded((n, H, d), torch.bfloat16, offset)
    swa.swa_paged_append(k, -k, gk.t, gv.t, table, cu, start, q=q, q_out=gq.t, inv_freq=inv)
    assert all(x.margins_intact() for x in (gk, gv, gq))
    assert torch.equal(gk.t, kc) and torch.equal(gv.t, vc) and torch.equal(gq.t, want)
    assert swa.swa_get_device_status() == 0
