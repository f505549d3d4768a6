"""The paged-cache operators against their definition in 64 bits.

Every slot that no query may see holds NaN, every table entry that no call may look up an id out
of range, so a stray read shows in the output or in the device status.
"""

import numpy as np
import pytest
import torch

from tests._paged import ANY_ENTRY, Batch, rotate, rotation_tolerance
from tests._util import to_f64

pytestmark = pytest.mark.gpu

FULL = 1 << 40  # a window past every sequence


@pytest.fixture(scope="module")
def swa(cuda_ok):
    import sliding_window_sparse_b200 as m

    return m


def check(got, want, tol, what):
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, first at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]:.6g} for "
                           f"{want[bad][0]:.6g} +- {tol[bad][0]:.2g}")


def run_chunk(swa, b, **kw):
    out, lse = swa.swa_attn_chunk_paged(b.q.cuda(), b.k_cache, b.v_cache, b.t_table, b.t_cu,
                                        b.t_first, b.W, b.scale, n_sink=b.sinks, return_lse=True,
                                        **kw)
    return out, lse


def run_decode(swa, b, pos=None, q=None, **kw):
    pos = b.t_first if pos is None else pos
    return swa.swa_attn_decode_paged(b.q.cuda() if q is None else q, b.k_cache, b.v_cache,
                                     b.t_table, pos, b.W, b.scale, n_sink=b.sinks,
                                     return_lse=True, **kw)


def check_batch(b, out, lse, drop=None, what=""):
    """out [total, H, d] and lse [total, H] on the rows of sequences."""
    want, want_lse, tol, tol_lse = b.expect(drop)
    rows = slice(int(b.cu[0]), int(b.cu[-1]))
    check(to_f64(out)[rows], want[rows], tol[rows], what + " out")
    check(to_f64(lse)[rows], want_lse[rows], tol_lse[rows], what + " lse")


CHUNKS = [
    # lens, starts, H, Hkv, d, page, W, sinks, layout
    ([1], [0], 1, 1, 64, 8, 1, 0, "hnd"),                               # one token, one key
    ([5], [1000], 8, 2, 64, 16, 512, 0, "hnd"),
    ([1, 0, 3], [0, 7, 130], 4, 2, 128, 16, FULL, 0, "nhd"),            # an empty sequence
    ([0, 2, 0, 0], [0, 5, 0, 9], 4, 4, 64, 32, 7, 0, "hnd"),
    ([300], [0], 4, 2, 128, 64, FULL, 0, "hnd"),
    ([127, 128, 129], [1, 0, 255], 8, 8, 64, 48, 100, 0, "nhd"),        # pages straddle tiles
    ([33, 64, 65], [500, 17, 4], 12, 4, 128, 24, 129, 3, "hnd"),        # G = 3, page 24
    ([70, 1], [200, 999], 7, 1, 64, 256, 64, 128, "nhd"),               # G = 7, a tile of sinks
    ([41], [4000], 40, 2, 128, 128, 1000, 4, "hnd"),                    # G = 20
    ([9, 2], [100, 0], 96, 1, 64, 40, 50, 1, "hnd"),                    # G = 96
    ([3, 4], [64, 300], 256, 2, 64, 16, 90, 2, "nhd"),                  # G = 128
    ([260], [3], 4, 4, 64, 64, 1, 0, "hnd"),                            # W = 1
    ([130], [300], 4, 1, 128, 8, 1, 1, "hnd"),                          # W = 1 and a sink
    ([200, 10], [50, 2000], 16, 2, 128, 16, 15, 128, "hnd"),            # more sinks than window
    ([513], [20000], 32, 8, 128, 16, 4096, 0, "hnd"),
    ([2] * 40, list(range(0, 4000, 100)), 8, 2, 128, 16, 333, 2, "nhd"),
    ([1] * 200, [37 * i % 1500 for i in range(200)], 4, 2, 64, 16, 256, 4, "hnd"),
    ([17], [30000], 8, 2, 128, 16, FULL, 0, "hnd"),                     # few rows, many keys
    ([1], [9999], 8, 1, 128, 65536, FULL, 0, "hnd"),                    # one page holds it all
]


@pytest.mark.parametrize("case", CHUNKS, ids=lambda c: str(c)[:60])
def test_chunk(swa, case):
    lens, starts, H, Hkv, d, page, W, sinks, layout = case
    b = Batch(lens, starts, H, Hkv, d, page, W, sinks, layout, seed=sum(lens) + H)
    out, lse = run_chunk(swa, b)
    assert swa.swa_get_device_status() == 0
    check_batch(b, out, lse.T, what=str(case)[:40])


DECODES = [
    # positions, H, Hkv, d, page, W, sinks, layout
    ([0], 1, 1, 64, 8, 1, 0, "hnd"),
    ([999], 32, 8, 128, 16, 4096, 0, "hnd"),
    ([0, 1, 7, 8, 63, 64, 65, 127, 128], 8, 2, 64, 16, FULL, 0, "nhd"),
    ([300, 5000, 17], 4, 4, 128, 48, 100, 4, "hnd"),
    ([77, 10000], 7, 1, 128, 24, 1000, 128, "nhd"),                     # G = 7
    ([500, 3, 129], 16, 1, 64, 64, 64, 1, "hnd"),                       # G = 16
    ([400, 90], 40, 2, 128, 32, 257, 2, "hnd"),                         # G = 20: two head blocks
    ([130, 64], 96, 1, 64, 8, FULL, 0, "hnd"),                          # G = 96
    ([20, 500], 600, 2, 64, 128, FULL, 0, "nhd"),                       # G = 300
    ([12345, 0, 4096], 12, 4, 128, 128, 1, 0, "hnd"),                   # W = 1
    ([70000], 8, 1, 128, 256, FULL, 0, "hnd"),
    ([(91 * i) % 3000 for i in range(300)], 8, 2, 64, 16, 512, 4, "hnd"),
    ([200, 150, 129, 128, 127], 8, 8, 128, 16, 1, 128, "nhd"),          # sinks, W = 1
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: str(c)[:60])
def test_decode(swa, case):
    pos, H, Hkv, d, page, W, sinks, layout = case
    b = Batch([1] * len(pos), pos, H, Hkv, d, page, W, sinks, layout, seed=sum(pos) + H)
    out, lse = run_decode(swa, b)
    assert swa.swa_get_device_status() == 0
    check_batch(b, out, lse, what=str(case)[:40])


def test_decode_padded_rows(swa):
    """pos = -1: zero and -infinity, whatever the table row holds; others are not touched by it."""
    b = Batch([1] * 5, [50, 700, 3, 64, 128], 8, 2, 64, 16, 100, 2)
    pos = b.t_first.clone()
    pos[1] = pos[4] = -1
    b.t_table[1] = ANY_ENTRY
    out = torch.full((5, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 8), 7.0, device="cuda")
    run_decode(swa, b, pos, out=out, lse=lse)
    assert swa.swa_get_device_status() == 0
    want, want_lse, tol, tol_lse = b.expect()
    for i in (0, 2, 3):
        check(to_f64(out[i]), want[i], tol[i], "out")
        check(to_f64(lse[i]), want_lse[i], tol_lse[i], "lse")
    for i in (1, 4):
        assert bool((out[i] == 0).all()) and bool(torch.isneginf(lse[i]).all())
    every = torch.full((5,), -1, dtype=torch.int64, device="cuda")
    run_decode(swa, b, every, out=out, lse=lse)
    assert swa.swa_get_device_status() == 0
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_decode_bad_positions_are_flagged(swa):
    b = Batch([1] * 3, [50, 70, 3], 8, 2, 64, 16, 100, 0)
    pos = b.t_first.clone()
    pos[0], pos[2] = -2, b.max_pages * 16
    out, lse = run_decode(swa, b, pos)
    assert swa.swa_get_device_status() == 6
    want, want_lse, tol, tol_lse = b.expect()
    check(to_f64(out[1]), want[1], tol[1], "out")
    for i in (0, 2):
        assert bool((out[i] == 0).all()) and bool(torch.isneginf(lse[i]).all())


@pytest.mark.parametrize("lead,trail", [(0, 0), (3, 0), (0, 200), (130, 7)])
def test_chunk_leaves_other_rows(swa, lead, trail):
    """Rows of tokens outside every sequence keep their contents; in new tensors they are zero."""
    b = Batch([20, 0, 45], [100, 9, 0], 4, 2, 64, 16, 64, 2, lead=lead, trail=trail)
    out = torch.full((b.total, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, b.total), 7.0, device="cuda")
    run_chunk(swa, b, out=out, lse=lse)
    check_batch(b, out, lse.T)
    rest = torch.ones(b.total, dtype=torch.bool)
    rest[lead:lead + 65] = False
    rest = rest.cuda()
    assert bool((out[rest] == 7).all()) and bool((lse[:, rest] == 7).all())
    trash = torch.full((1 << 22,), float("nan"), device="cuda")  # what a new tensor may hold
    del trash
    out, lse = run_chunk(swa, b)
    check_batch(b, out, lse.T)
    assert bool((out[rest] == 0).all()) and bool((lse[:, rest] == 0).all())
    mine = torch.full((4, b.total), 7.0, device="cuda")
    out, lse = run_chunk(swa, b, lse=mine)  # a new out beside the caller's lse
    assert bool((out[rest] == 0).all()) and bool((mine[:, rest] == 7).all())
    assert swa.swa_get_device_status() == 0


def test_chunk_bad_sequences_are_flagged_and_skipped(swa):
    """A negative start and an end past the table: flagged, rows not written, others right."""
    for which, start in ((0, -1), (2, None)):
        b = Batch([20, 30, 10], [5, 100, 0], 4, 2, 64, 16, 64, 0)
        first = b.t_first.clone()
        first[which] = start if start is not None else b.max_pages * 16 - 9
        out = torch.full((60, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, 60), 7.0, device="cuda")
        swa.swa_attn_chunk_paged(b.q.cuda(), b.k_cache, b.v_cache, b.t_table, b.t_cu, first, b.W,
                                 b.scale, out=out, lse=lse)
        assert swa.swa_get_device_status() == 6
        want, want_lse, tol, tol_lse = b.expect()
        for i in range(3):
            rows = slice(int(b.cu[i]), int(b.cu[i + 1]))
            if i == which:
                assert bool((out[rows] == 7).all()) and bool((lse[:, rows] == 7).all())
            else:
                check(to_f64(out[rows]), want[rows], tol[rows], "out")


@pytest.mark.parametrize("cu", [[0, 20, 10, 60], [0, 20, 50, 61], [-4, 20, 50, 60]])
def test_chunk_bad_offsets_are_flagged(swa, cu):
    b = Batch([20, 30, 10], [5, 100, 0], 4, 2, 64, 16, 64, 0)
    t_cu = torch.tensor(cu, dtype=torch.int64, device="cuda")
    swa.swa_attn_chunk_paged(b.q.cuda(), b.k_cache, b.v_cache, b.t_table, t_cu, b.t_first, b.W)
    assert swa.swa_get_device_status() == 6
    kv = torch.zeros((60, 2, 64), dtype=torch.bfloat16, device="cuda")
    swa.swa_paged_append(kv, kv, b.k_cache, b.v_cache, b.t_table, t_cu, b.t_first)
    assert swa.swa_get_device_status() == 6


@pytest.mark.parametrize("entry", [-1, "n_pages", 0x7FFFFFFF, -0x80000000])
def test_visible_pages_out_of_range_count_as_zeros(swa, entry):
    b = Batch([20, 30], [5, 100], 4, 2, 64, 16, 64, 2)
    entry = b.n_pages if entry == "n_pages" else entry
    b.t_table[1, 5] = entry
    out, lse = run_chunk(swa, b)
    assert swa.swa_get_device_status() == 6
    check_batch(b, out, lse.T, drop={(1, 5)})
    b = Batch([1, 1], [5, 100], 4, 2, 64, 16, 64, 2)
    b.t_table[1, 5] = entry
    out, lse = run_decode(swa, b)
    assert swa.swa_get_device_status() == 6
    check_batch(b, out, lse, drop={(1, 5)})


def test_scores_of_lowest_values(swa):
    """Keys that drive every visible score to about -10^4 of the others' keep the softmax finite;
    a row that sees one key returns its value."""
    b = Batch([40], [60], 4, 2, 64, 16, 30, 0)
    b.keys[0][:] = b.keys[0] * 200
    b.q[:] = b.q * 8
    at = torch.from_numpy(b.table[0, b.pos_of[0] // 16].astype(np.int64)).cuda()
    slot = torch.from_numpy(b.pos_of[0] % 16).cuda()
    b.k_cache[at, :, slot] = b.keys[0].cuda()
    out, lse = run_chunk(swa, b)
    check_batch(b, out, lse.T)
    one = Batch([1], [60], 4, 2, 64, 16, 1, 0)
    out, _ = run_decode(swa, one)
    want = one.vals[0][0].repeat_interleave(2, 0)
    assert torch.equal(out[0].cpu(), want)


def test_decode_equals_chunk_of_one(swa):
    pos = [0, 5, 64, 129, 2000]
    b = Batch([1] * 5, pos, 16, 2, 128, 16, 500, 3, "nhd")
    out, lse = run_decode(swa, b)
    out2, lse2 = run_chunk(swa, b)
    want, want_lse, tol, tol_lse = b.expect()
    check(to_f64(out), to_f64(out2), 2 * tol, "out")
    check(to_f64(lse), to_f64(lse2.T), 2 * tol_lse, "lse")


def test_repeated_calls_are_bit_identical(swa):
    """No atomics in the sums: the same call gives the same bits, with any workspace contents."""
    b = Batch([100, 300, 7], [1000, 0, 5000], 8, 2, 128, 16, 700, 4)
    need = swa.swa_chunk_paged_workspace_bytes(3, b.total, 8, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    first = run_chunk(swa, b, workspace=ws)
    for _ in range(3):
        again = run_chunk(swa, b)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
    b = Batch([1] * 7, [1000, 0, 5000, 3, 8, 9, 4000], 8, 2, 128, 16, 3000, 4)
    need = swa.swa_decode_paged_workspace_bytes(7, 8, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    first = run_decode(swa, b, workspace=ws)
    for _ in range(3):
        again = run_decode(swa, b)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_far_pages(swa):
    """Slots whose element offset passes 2^32: a cache of 4.6 GB of which a few pages are used."""
    n_pages, page, Hkv, d = 140000, 64, 4, 64
    b = Batch([70], [300], 8, Hkv, d, page, 200, 2)
    k = torch.empty((n_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    assert (n_pages - 100) * Hkv * page * d > 1 << 31
    table = b.t_table.clone()
    live = table != ANY_ENTRY
    table[live] += n_pages - b.n_pages
    k[-b.n_pages:], v[-b.n_pages:] = b.k_cache, b.v_cache
    out, lse = swa.swa_attn_chunk_paged(b.q.cuda(), k, v, table, b.t_cu, b.t_first, b.W, b.scale,
                                        n_sink=2, return_lse=True)
    check_batch(b, out, lse.T)
    one = Batch([1], [369], 8, Hkv, d, page, 200, 2)
    table = one.t_table.clone()
    live = table != ANY_ENTRY
    table[live] += n_pages - one.n_pages
    k[-one.n_pages:], v[-one.n_pages:] = one.k_cache, one.v_cache
    out, lse = swa.swa_attn_decode_paged(one.q.cuda(), k, v, table, one.t_first, one.W, one.scale,
                                         n_sink=2, return_lse=True)
    check_batch(one, out, lse)
    new = torch.randn((1, Hkv, d), device="cuda").bfloat16()
    table[0, 5] = n_pages - 1
    swa.swa_paged_append(new, -new, k, v, table, torch.tensor([0, 1], device="cuda"), one.t_first)
    assert torch.equal(k[-1, :, 369 % page], new[0]) and torch.equal(v[-1, :, 369 % page], -new[0])
    assert swa.swa_get_device_status() == 0


def test_streams_and_graphs(swa):
    """Two calls at once on streams of their own, and both operators captured and replayed with
    other inputs in the same buffers."""
    b = Batch([200, 30], [500, 0], 8, 2, 128, 16, 300, 2)
    e = Batch([1] * 9, [10, 200, 3000, 0, 64, 65, 1, 2, 900], 8, 2, 128, 16, 300, 2)
    want = run_chunk(swa, b) + run_decode(swa, e)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        got1 = [run_chunk(swa, b) for _ in range(5)]
    with torch.cuda.stream(s2):
        got2 = [run_decode(swa, e) for _ in range(5)]
    torch.cuda.synchronize()
    for x, y in zip(got1, got2):
        assert all(torch.equal(g, w) for g, w in zip(x + y, want))

    q, qd, first, pos = b.q.cuda(), e.q.cuda(), b.t_first.clone(), e.t_first.clone()
    out, lse = torch.empty_like(q), torch.empty((8, b.total), device="cuda")
    outd, lsed = torch.empty_like(qd), torch.empty((9, 8), device="cuda")
    ws = torch.empty(swa.swa_chunk_paged_workspace_bytes(2, b.total, 8, 2, 128),
                     dtype=torch.uint8, device="cuda")
    wsd = torch.empty(swa.swa_decode_paged_workspace_bytes(9, 8, 2, 128), dtype=torch.uint8,
                      device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa.swa_attn_chunk_paged(q, b.k_cache, b.v_cache, b.t_table, b.t_cu, first, b.W, b.scale,
                                 n_sink=2, out=out, lse=lse, workspace=ws)
        swa.swa_attn_decode_paged(qd, e.k_cache, e.v_cache, e.t_table, pos, e.W, e.scale,
                                  n_sink=2, out=outd, lse=lsed, workspace=wsd)
    for shift in (0, 1):
        if shift:  # other queries, a row that became padding
            q.neg_()
            qd.neg_()
            pos[4] = -1
        ws.fill_(255)
        wsd.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        ref = swa.swa_attn_chunk_paged(q, b.k_cache, b.v_cache, b.t_table, b.t_cu, first, b.W,
                                       b.scale, n_sink=2, return_lse=True)
        refd = swa.swa_attn_decode_paged(qd, e.k_cache, e.v_cache, e.t_table, pos, e.W, e.scale,
                                         n_sink=2, return_lse=True)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
        assert torch.equal(outd, refd[0]) and torch.equal(lsed, refd[1])
    assert swa.swa_get_device_status() == 0


def test_wrapper_refusals(swa):
    b = Batch([4], [10], 4, 2, 64, 16, 8, 0)
    q = b.q.cuda()

    def chunk(**kw):
        a = dict(q=q, k=b.k_cache, v=b.v_cache, t=b.t_table, cu=b.t_cu, first=b.t_first)
        a.update(kw)
        extra = {n: a[n] for n in ("out", "lse") if n in a}
        return swa.swa_attn_chunk_paged(a["q"], a["k"], a["v"], a["t"], a["cu"], a["first"], 8,
                                        **extra)

    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(t=b.t_table.long()),
                dict(t=b.t_table.cpu()), dict(t=b.t_table.T), dict(cu=b.t_cu.int()),
                dict(first=b.t_first[:0]), dict(k=b.k_cache[..., :32]),
                dict(v=b.v_cache.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(out=torch.empty_like(q)[:2]), dict(lse=torch.empty((4, 3), device="cuda"))):
        with pytest.raises(ValueError):
            chunk(**bad)
    kv = q[:, :2]
    assert not kv.is_contiguous()
    with pytest.raises(ValueError):
        swa.swa_paged_append(kv.transpose(0, 1), kv, b.k_cache, b.v_cache, b.t_table, b.t_cu,
                             b.t_first)
    with pytest.raises(ValueError):
        swa.swa_paged_append(kv, kv, b.k_cache, b.v_cache, b.t_table, b.t_cu, b.t_first,
                             positions=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(swa.SwaError):
        swa.swa_attn_chunk_paged(q, b.k_cache, b.v_cache, b.t_table, b.t_cu, b.t_first, 8,
                                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------------------- append

APPENDS = [
    # lens, starts, H, Hkv, d, page, layout, rot, interleaved, axes, q
    ([1], [0], 4, 2, 64, 8, "hnd", 64, False, 0, True),
    ([1] * 70, [53 * i for i in range(70)], 32, 8, 128, 16, "hnd", 128, False, 0, True),
    ([5, 0, 130, 1], [3, 9, 60, 100000], 8, 2, 128, 48, "nhd", 64, True, 3, True),
    ([33], [7], 12, 4, 64, 24, "nhd", 16, True, 0, True),
    ([40, 2], [0, 1000000], 7, 1, 128, 64, "hnd", 128, False, 3, True),
    ([9], [4], 4, 2, 64, 16, "hnd", 0, False, 0, True),                 # no rotation
    ([300, 0, 0], [0, 0, 0], 4, 4, 128, 256, "nhd", 96, False, 1, False),
    ([2] * 300, [17 * i for i in range(300)], 4, 2, 64, 16, "hnd", 32, True, 0, False),
    ([77], [20], 64, 32, 128, 16, "hnd", 128, True, 0, True),           # several items a thread
]


def fused(rng, total, heads, d, apart):
    """bf16 [total, heads, d] whose rows lie `apart` heads apart, on the device."""
    x = torch.from_numpy(rng.standard_normal((total, heads + apart, d))).to(torch.bfloat16)
    return x.cuda()[:, :heads]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: str(c)[:60])
@pytest.mark.parametrize("inplace", [False, True])
def test_append(swa, case, inplace):
    lens, starts, H, Hkv, d, page, layout, rot, inter, axes, with_q = case
    rng = np.random.default_rng(len(lens) + H)
    cu = np.concatenate([[0], np.cumsum(lens)]) + 2
    total = int(cu[-1]) + 3
    k, v = fused(rng, total, Hkv, d, 1), fused(rng, total, Hkv, d, 3)
    q = fused(rng, total, H, d, 2) if with_q else None
    pages = [sorted({p // page for p in range(s, s + n)}) for n, s in zip(lens, starts)]
    n_pages = sum(map(len, pages)) + 1
    ids = rng.permutation(n_pages)
    table = np.full((len(lens), max(max(p, default=0) for p in pages) + 1), ANY_ENTRY, np.int32)
    flat = 0
    for b, ps in enumerate(pages):
        for p in ps:
            table[b, p] = ids[flat]
            flat += 1
    kc = torch.from_numpy(rng.standard_normal((n_pages, Hkv, page, d))).to(torch.bfloat16)
    kd, vd = Batch._device(kc, layout), Batch._device(-kc, layout)
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    tok_pos = np.zeros(total, np.int64)
    for b, (n, s) in enumerate(zip(lens, starts)):
        tok_pos[cu[b]:cu[b + 1]] = np.arange(s, s + n)
    pos = np.repeat(tok_pos[:, None], rot // 2, 1)
    kw = {}
    if axes:
        ax = rng.integers(0, 1 << 20, (axes, total))
        which = rng.integers(0, axes, rot // 2).astype(np.int32)
        pos = ax[which].T
        kw = dict(positions=torch.from_numpy(ax).cuda(), pair_axis=torch.from_numpy(which).cuda())
    if rot:
        kw |= dict(inv_freq=torch.from_numpy(inv).cuda(), interleaved=inter)
    q_host, k_host = (None if x is None else to_f64(x) for x in (q, k))
    q_out = None
    if with_q and inplace:
        q_out = q
    got = swa.swa_paged_append(k, v, kd, vd, torch.from_numpy(table).cuda(),
                               torch.from_numpy(cu).cuda(),
                               torch.tensor(starts, dtype=torch.int64).cuda(), q=q, q_out=q_out,
                               **kw)
    assert swa.swa_get_device_status() == 0
    rows = slice(int(cu[0]), int(cu[-1]))
    if with_q:
        check(to_f64(got)[rows], rotate(q_host, pos, inv, inter)[rows],
              rotation_tolerance(q_host, pos, inv, inter)[rows], "q")
        rest = np.ones(total, bool)
        rest[rows] = False
        want = q_host[rest] if inplace else 0 * q_host[rest]
        assert np.array_equal(to_f64(got)[rest], want)
    else:
        assert got is None
    want_k, tol_k = to_f64(kc), np.zeros(kc.shape)
    want_v = -want_k
    want_k = want_k.copy()
    rk, tk = rotate(k_host, pos, inv, inter), rotation_tolerance(k_host, pos, inv, inter)
    for b, n in enumerate(lens):
        for t in range(int(cu[b]), int(cu[b + 1])):
            page_id, slot = table[b, tok_pos[t] // page], tok_pos[t] % page
            want_k[page_id, :, slot], tol_k[page_id, :, slot] = rk[t], tk[t]
            want_v[page_id, :, slot] = to_f64(v[t])
    check(to_f64(kd), want_k, tol_k, "k cache")  # slots not written: bit for bit
    assert np.array_equal(to_f64(vd), want_v)


def test_append_bad_entries_write_nothing(swa):
    rng = np.random.default_rng(5)
    k, q = fused(rng, 40, 2, 64, 0), fused(rng, 40, 4, 64, 0)
    kd = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vd = torch.zeros_like(kd)
    table = torch.tensor([[0, 4], [-1, 2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20, 40], device="cuda")
    out = swa.swa_paged_append(k, k, kd, vd, table, cu, torch.tensor([0, 0], device="cuda"), q=q)
    assert swa.swa_get_device_status() == 6
    for c in (kd, vd):
        assert torch.equal(c[0].transpose(0, 1), k[:16])
        assert torch.equal(c[2, :, :4].transpose(0, 1), k[36:])
        assert int((c != 0).sum()) == int((k[:16] != 0).sum()) + int((k[36:] != 0).sum())
    assert torch.equal(out[:16], q[:16]) and torch.equal(out[36:], q[36:])
    assert int((out[16:36] != 0).sum()) == 0
    for start in (-1, 32):  # a negative start, a position past the table
        swa.swa_paged_append(k, k, kd, vd, table, cu, torch.tensor([start, 16], device="cuda"))
        assert swa.swa_get_device_status() == 6
    inv = torch.ones(16, device="cuda")
    pos = torch.arange(40, device="cuda").repeat(2, 1)
    good = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    good[:] = torch.tensor([[0, 1], [2, 3]])
    swa.swa_paged_append(k, k, kd, vd, good, cu, torch.tensor([0, 0], device="cuda"),
                         inv_freq=inv, positions=pos,
                         pair_axis=torch.full((16,), 2, dtype=torch.int32, device="cuda"))
    assert swa.swa_get_device_status() == 6


# ---------------------------------------------------------------------------- together

@pytest.mark.parametrize("W,sinks", [(FULL, 0), (100, 0), (64, 3)])
def test_serving_run(swa, W, sinks):
    """Prefill in two chunks and then single tokens, from a paged cache whose pages behind the
    window are given back, equals one packed prefill of the rotated rows (swa_attn_varlen)."""
    H, Hkv, d, page, n_seq = 8, 2, 128, 16, 3
    full = [210, 75, 131]  # whole lengths; the last 4 tokens one at a time
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = [torch.randn((n, H + 2 * Hkv, d), generator=g, device="cuda").bfloat16() for n in full]
    inv = (10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2))).float()
    max_pages = max(full) // page + 1
    n_pages = n_seq * max_pages
    table = torch.randperm(n_pages, generator=g, device="cuda").int().view(n_seq, max_pages)
    kc = torch.full((n_pages, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kc, vc = kc.transpose(1, 2), kc.clone().transpose(1, 2)
    outs, rotated = [[] for _ in full], [[] for _ in full]

    def feed(cut):  # cut: (begin, end) per sequence
        rows = torch.cat([x[a:e] for x, (a, e) in zip(qkv, cut)])
        cu = torch.tensor([0] + list(np.cumsum([e - a for a, e in cut])), device="cuda")
        start = torch.tensor([a for a, _ in cut], device="cuda")
        q = swa.swa_paged_append(rows[:, H:H + Hkv], rows[:, H + Hkv:], kc, vc, table, cu, start,
                                 q=rows[:, :H], inv_freq=inv)
        if all(e - a == 1 for a, e in cut):
            out = swa.swa_attn_decode_paged(q, kc, vc, table, start, W, n_sink=sinks)
        else:
            out = swa.swa_attn_chunk_paged(q, kc, vc, table, cu, start, W, n_sink=sinks)
        for b in range(n_seq):
            outs[b].append(out[cu[b]:cu[b + 1]])
            rotated[b].append(q[cu[b]:cu[b + 1]])
            # give back the pages that no later query can see
            low = max(0, cut[b][1] - W + 1)
            for p in range(max_pages):
                if (p + 1) * page <= low and p * page >= sinks and table[b, p] >= 0:
                    kc[table[b, p]] = float("nan")
                    vc[table[b, p]] = float("nan")
                    table[b, p] = -1

    feed([(0, 60), (0, 0), (0, 100)])
    feed([(60, 206), (0, 71), (100, 127)])
    for i in range(4):
        feed([(206 + i, 207 + i), (71 + i, 72 + i), (127 + i, 128 + i)])
    assert swa.swa_get_device_status() == 0

    q = torch.cat([torch.cat(r) for r in rotated])
    cu = torch.tensor([0] + list(np.cumsum(full)), device="cuda")
    flat = torch.cat(qkv)
    # the rotated keys, from a cache of one page per sequence of 256 slots
    kk = torch.zeros((n_seq, Hkv, 256, d), dtype=torch.bfloat16, device="cuda")
    vv = torch.zeros_like(kk)
    swa.swa_paged_append(flat[:, H:H + Hkv], flat[:, H + Hkv:], kk, vv,
                         torch.arange(n_seq, device="cuda").int()[:, None], cu,
                         torch.zeros(n_seq, dtype=torch.int64, device="cuda"), inv_freq=inv)
    k = torch.cat([kk[b, :, :n].transpose(0, 1) for b, n in enumerate(full)]).contiguous()
    v = torch.cat([vv[b, :, :n].transpose(0, 1) for b, n in enumerate(full)]).contiguous()
    want = swa.swa_attn_varlen(q, k, v, cu, max(full), min(W, 1 << 20), n_sink=sinks)
    got = torch.cat([torch.cat(o) for o in outs])
    # either side rounds its weights (a weighted mean of |v| is at most the largest) and its output
    err = np.abs(to_f64(got) - to_f64(want))
    assert (err <= 2 * 2.0 ** -8 * (np.abs(to_f64(want)) + 1.01 * np.abs(to_f64(v)).max())).all()
    # the first rows see one key: their output is its value, bit for bit
    for b in range(n_seq):
        assert torch.equal(got[cu[b]], v[cu[b]].repeat_interleave(H // Hkv, 0))


# ---------------------------------------------------------------------------- at large

def test_many_sequences(swa):
    """Thousands of sequences, most of them empty or short: a unit list that does not fit the
    schedule's shared memory, runs that skip long stretches of empty entries."""
    rng = np.random.default_rng(1)
    n = 6000
    lens = rng.choice([0, 1, 2, 40], n, p=[0.5, 0.4, 0.09, 0.01]).tolist()
    starts = rng.integers(0, 40, n).tolist()
    b = Batch(lens, starts, 8, 8, 64, 8, 20, 1, seed=2)
    out, lse = run_chunk(swa, b)
    assert swa.swa_get_device_status() == 0
    check_batch(b, out, lse.T)
    pos = rng.integers(0, 300, 3000).tolist()
    e = Batch([1] * 3000, pos, 4, 4, 64, 8, 100, 1, seed=3)
    padded = torch.from_numpy(rng.random(3000) < 0.3).cuda()
    out, lse = run_decode(swa, e, torch.where(padded, -1, e.t_first))
    assert swa.swa_get_device_status() == 0
    want, want_lse, tol, tol_lse = e.expect()
    keep = (~padded).cpu().numpy()
    check(to_f64(out)[keep], want[keep], tol[keep], "out")
    check(to_f64(lse)[keep], want_lse[keep], tol_lse[keep], "lse")
    assert bool((out[padded] == 0).all()) and bool(torch.isneginf(lse[padded]).all())


@pytest.mark.parametrize("seed", range(40))
def test_sweep(swa, seed):
    """Random batches: group sizes, pages, layouts, windows, sinks, lengths and starts."""
    rng = np.random.default_rng(1000 + seed)

    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    Hkv = int(rng.choice([1, 2, 3, 4]))
    G = int(rng.choice([1, 2, 3, 4, 5, 8, 16, 17, 32]))
    d = int(rng.choice([64, 128]))
    page = int(rng.choice([8, 16, 24, 32, 40, 64, 96, 128, 256]))
    W = log_int(1, 3000) if rng.random() < 0.8 else FULL
    sinks = int(rng.choice([0, 0, 1, 4, 127, 128]))
    n = log_int(1, 12)
    layout = str(rng.choice(["hnd", "nhd"]))
    if seed % 2:
        pos = [log_int(1, 9000) - 1 for _ in range(n)]
        b = Batch([1] * n, pos, G * Hkv, Hkv, d, page, W, sinks, layout, seed=seed)
        out, lse = run_decode(swa, b)
    else:
        lens = [int(rng.choice([0, 1, log_int(1, 300)])) for _ in range(n)]
        lens[0] = max(1, lens[0])
        starts = [log_int(1, 4000) - 1 for _ in range(n)]
        b = Batch(lens, starts, G * Hkv, Hkv, d, page, W, sinks, layout, seed=seed,
                  lead=int(rng.integers(0, 3)), trail=int(rng.integers(0, 3)))
        out, lse = run_chunk(swa, b)
        lse = lse.T
    assert swa.swa_get_device_status() == 0
    check_batch(b, out, lse)


SHORT_UNITS = [
    # lens, starts, H, Hkv, d, page, W, sinks, lead, trail: units of a few key tiles, which the
    # schedule hands out whole (fewer units than SMs, one and several rounds of them)
    ([600], [0], 48, 48, 64, 16, 100, 0, 0, 0),
    ([700], [5], 40, 40, 128, 64, 300, 2, 0, 3),
    ([300, 1, 0, 260, 130], [0, 7, 9, 4000, 255], 24, 24, 64, 32, 129, 0, 2, 40),
    ([400], [100], 128, 16, 128, 8, 128, 128, 0, 0),
    ([500, 500], [0, 64], 36, 36, 64, 128, 1, 1, 1, 0),
]


@pytest.mark.parametrize("case", SHORT_UNITS, ids=lambda c: str(c)[:60])
def test_short_units(swa, case):
    lens, starts, H, Hkv, d, page, W, sinks, lead, trail = case
    b = Batch(lens, starts, H, Hkv, d, page, W, sinks, "hnd", seed=H, lead=lead, trail=trail)
    out, lse = run_chunk(swa, b)
    assert swa.swa_get_device_status() == 0
    check_batch(b, out, lse.T, what=str(case)[:40])
    rest = torch.ones(b.total, dtype=torch.bool)
    rest[lead:int(b.cu[-1])] = False
    assert bool((out[rest.cuda()] == 0).all()) and bool((lse.T[rest.cuda()] == 0).all())


def test_no_tokens(swa):
    """A step in which every sequence is empty: padding alone, zeros in what the call allocates."""
    b = Batch([0, 0], [5, 0], 8, 2, 128, 16, 100, 0, trail=70)
    out, lse = run_chunk(swa, b)
    assert bool((out == 0).all()) and bool((lse == 0).all())
    kept, kept_lse = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    run_chunk(swa, b, out=kept, lse=kept_lse)
    assert bool((kept == 7).all()) and bool((kept_lse == 7).all())
    before = b.k_cache.clone()
    k = torch.ones((b.total, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = swa.swa_paged_append(k, k, b.k_cache, b.v_cache, b.t_table, b.t_cu, b.t_first,
                             q=b.q.cuda())
    assert bool((q == 0).all())
    assert torch.equal(b.k_cache.view(torch.int16), before.view(torch.int16))
    pos = torch.tensor([-1, -1], device="cuda")
    out, lse = run_decode(swa, b, pos, q=b.q[:2].cuda())
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    assert swa.swa_get_device_status() == 0
