"""What the paged-cache entry points refuse, before they touch the GPU (no compute call is made)."""

import ctypes

import pytest

FAKE = 0x100000  # aligned non-null address: never dereferenced


@pytest.fixture(scope="module")
def native():
    from sliding_window_sparse_b200 import build

    build.build()
    from sliding_window_sparse_b200 import _native

    return _native


def cache(native, **kw):
    c = dict(k=FAKE, v=FAKE, table=FAKE, page_stride=16 * 2 * 64, head_stride=16 * 64,
             slot_stride=64, n_pages=10, max_pages=4, table_stride=4, page_size=16)
    c.update(kw)
    return native.PagedCache(**c)


BAD_CACHES = [
    dict(k=None), dict(v=None), dict(table=None), dict(k=FAKE + 8), dict(table=FAKE + 2),
    dict(page_stride=0), dict(page_stride=-2048), dict(head_stride=1028), dict(slot_stride=56),
    dict(page_stride=1 << 39), dict(n_pages=0), dict(n_pages=(1 << 31) - 1), dict(max_pages=0),
    dict(table_stride=3), dict(page_size=0), dict(page_size=12), dict(page_size=4),
    dict(page_size=65544), dict(max_pages=1 << 27, table_stride=1 << 27),
]


def append(native, c, rotation=None, **kw):
    a = dict(k=FAKE, ks=128, v=FAKE, vs=128, q=FAKE, qs=256, qo=FAKE, qos=256, cu=FAKE, qst=FAKE,
             n_seq=1, total=8, H=4, Hkv=2, d=64)
    a.update(kw)
    return native.lib().swa_paged_append(
        a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["qo"], a["qos"], c and ctypes.byref(c),
        rotation and ctypes.byref(rotation), a["cu"], a["qst"], a["n_seq"], a["total"], a["H"],
        a["Hkv"], a["d"], 0, None)


def chunk(native, c, **kw):
    a = dict(q=FAKE, cu=FAKE, qst=FAKE, out=FAKE, n_seq=1, total=8, H=4, Hkv=2, d=64, W=16, sink=0,
             scale=0.1, ws=FAKE, more=0)
    a.update(kw)
    need = native.lib().swa_chunk_paged_workspace_bytes(1, 8, 4, 2, 64)
    return native.lib().swa_attn_chunk_paged(
        a["q"], c and ctypes.byref(c), a["cu"], a["qst"], a["out"], None, a["n_seq"], a["total"],
        a["H"], a["Hkv"], a["d"], a["W"], a["sink"], a["scale"], 0, a["ws"], need + a["more"], None)


def decode(native, c, **kw):
    a = dict(q=FAKE, pos=FAKE, out=FAKE, B=2, H=4, Hkv=2, d=64, W=16, sink=0, scale=0.1, ws=FAKE,
             more=0)
    a.update(kw)
    need = native.lib().swa_decode_paged_workspace_bytes(2, 4, 2, 64)
    return native.lib().swa_attn_decode_paged(
        a["q"], c and ctypes.byref(c), a["pos"], a["out"], None, a["B"], a["H"], a["Hkv"], a["d"],
        a["W"], a["sink"], a["scale"], a["ws"], need + a["more"], None)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(native, bad):
    for call in (append, chunk, decode):
        assert call(native, cache(native, **bad)) == 1


def test_no_cache(native):
    for call in (append, chunk, decode):
        assert call(native, None) == 1


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(cu=None), 1), (dict(qst=None), 1),
    (dict(q=None), 1), (dict(qo=None), 1),           # queries in without out, and the reverse
    (dict(k=FAKE + 8), 1), (dict(qo=FAKE + 8), 1), (dict(ks=120), 1), (dict(ks=132), 1),
    (dict(vs=64), 1), (dict(qs=255), 1), (dict(qos=200), 1),
    (dict(qs=264), 1),                               # in place with other strides
    (dict(n_seq=0), 1), (dict(total=0), 1), (dict(total=1 << 31), 1), (dict(Hkv=0), 1),
    (dict(H=0), 1), (dict(d=96), 2), (dict(n_seq=1 << 24), 2),
], ids=str)
def test_append_refuses(native, bad, code):
    assert append(native, cache(native), **bad) == code


@pytest.mark.parametrize("bad", [
    dict(inv_freq=None), dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=80),
    dict(positions=FAKE, n_axes=0), dict(positions=FAKE, n_axes=3, positions_stride=7),
    dict(pair_axis=FAKE),
], ids=str)
def test_rotation_refuses(native, bad):
    r = dict(inv_freq=FAKE, positions=None, pair_axis=None, positions_stride=8, rot_dim=64,
             interleaved=0, n_axes=0)
    r.update(bad)
    assert append(native, cache(native), native.Rotation(**r)) == 1


COMMON = [
    (dict(q=None), 1), (dict(out=None), 1), (dict(q=FAKE + 8), 1), (dict(out=FAKE + 8), 1),
    (dict(H=5), 1), (dict(Hkv=0), 1), (dict(W=0), 1), (dict(scale=0.0), 1),
    (dict(scale=float("inf")), 1), (dict(sink=-1), 1), (dict(sink=129), 1), (dict(d=32), 2),
    (dict(ws=None), 4), (dict(ws=FAKE + 16), 4),
]


@pytest.mark.parametrize("bad,code", COMMON + [
    (dict(cu=None), 1), (dict(qst=None), 1), (dict(n_seq=0), 1), (dict(total=0), 1),
    (dict(total=(1 << 31) - 256), 1), (dict(H=258), 2), (dict(n_seq=1 << 24), 2), (dict(more=-1), 4),
], ids=str)
def test_chunk_refuses(native, bad, code):
    assert chunk(native, cache(native), **bad) == code


@pytest.mark.parametrize("bad,code", COMMON + [
    (dict(pos=None), 1), (dict(B=0), 1), (dict(B=1 << 24), 2), (dict(B=1 << 22, H=8), 2),
    (dict(more=-1), 4),
], ids=str)
def test_decode_refuses(native, bad, code):
    assert decode(native, cache(native), **bad) == code


def test_workspace_sizes(native):
    lib = native.lib()
    for n in (lib.swa_chunk_paged_workspace_bytes(3, 700, 32, 8, 128),
              lib.swa_decode_paged_workspace_bytes(3, 32, 8, 128)):
        assert n > 0 and n % 256 == 0
    assert lib.swa_chunk_paged_workspace_bytes(0, 700, 32, 8, 128) == 0
    assert lib.swa_chunk_paged_workspace_bytes(3, 0, 32, 8, 128) == 0
    assert lib.swa_chunk_paged_workspace_bytes(3, 700, 32, 7, 128) == 0
    assert lib.swa_decode_paged_workspace_bytes(0, 32, 8, 128) == 0
    assert lib.swa_decode_paged_workspace_bytes(3, 32, 8, 96) == 0


@pytest.mark.parametrize("n_seq,H,Hkv", [((1 << 20) + 1, 1, 1), ((1 << 17) + 1, 8, 8)])
def test_chunk_refuses_too_many_sequences(native, n_seq, H, Hkv):
    assert chunk(native, cache(native), n_seq=n_seq, H=H, Hkv=Hkv) == 2
    assert native.lib().swa_chunk_paged_workspace_bytes(n_seq, 700, H, Hkv, 128) == 0
    assert native.lib().swa_chunk_paged_workspace_bytes(n_seq - 1, 700, H, Hkv, 128) > 0


def test_packed_cache_is_the_structure(native):
    fields = (FAKE, FAKE + 256, FAKE + 512, 8192, 1024, 128, 7, 5, 9, 64)
    packed = native.pack_paged_cache(*fields)
    assert len(packed) == ctypes.sizeof(native.PagedCache)
    c = native.PagedCache.from_buffer_copy(packed)
    assert tuple(getattr(c, name) for name, _ in c._fields_) == fields
