"""Workspace sizes of the paged attention calls: zero exactly where the call refuses the sizes."""

import pytest

from tests.test_paged_abi import cache, chunk, decode, native  # noqa: F401


@pytest.mark.parametrize("n_seq,total,H,Hkv,d", [
    (1, 8, 258, 2, 64),              # 129 heads a group
    (1, (1 << 31) - 300, 1024, 8, 64),  # a unit list of more than 2^30 entries
    (2, 8, 4, 3, 64), (1, 8, 4, 2, 96), ((1 << 20) + 1, 8, 1, 1, 64), (0, 8, 4, 2, 64),
])
def test_chunk_sizes_that_are_refused(native, n_seq, total, H, Hkv, d):  # noqa: F811
    assert native.lib().swa_chunk_paged_workspace_bytes(n_seq, total, H, Hkv, d) == 0
    assert chunk(native, cache(native, slot_stride=d), n_seq=n_seq, total=total, H=H, Hkv=Hkv,
                 d=d) in (1, 2)


@pytest.mark.parametrize("B,H,Hkv,d", [
    (1 << 22, 8, 8, 64), ((1 << 24) - 1, 2, 1, 128), (1 << 24, 1, 1, 64), (2, 4, 3, 64),
])
def test_decode_sizes_that_are_refused(native, B, H, Hkv, d):  # noqa: F811
    assert native.lib().swa_decode_paged_workspace_bytes(B, H, Hkv, d) == 0
    assert decode(native, cache(native, slot_stride=d), B=B, H=H, Hkv=Hkv, d=d) in (1, 2)


def test_largest_sizes(native):  # noqa: F811
    lib = native.lib()
    assert lib.swa_chunk_paged_workspace_bytes(1, 8, 256, 2, 64) > 0
    assert lib.swa_chunk_paged_workspace_bytes(1 << 20, 1 << 20, 1, 1, 128) > 0
    assert lib.swa_decode_paged_workspace_bytes(1 << 21, 8, 8, 64) > 0
