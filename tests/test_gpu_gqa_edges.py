"""Grouped-query attention where a cache ends: shares and pages that the buffer
cuts short, and pages that were given back."""
import numpy as np
import pytest
import torch

import oracle as O
from kv_cache_decode_csa2_b200 import csa2 as B
from tests.gqa_cases import DEV, PAGE, Cache, bf16, bounds, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def attend(cache, q, seq, pos, window, n_sink, group):
    """(out, lse, status word) of one call."""
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    call = B.GqaAttn(cache.c, q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), out, window=window,
                     n_sink=n_sink, seq_of_query=torch.tensor(seq, dtype=torch.int32, device=DEV), lse=lse,
                     group_queries=group)
    call.run()
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), int(call.status.item())


def check(cache, q64, seq, pos, out, lse, window, n_sink, there):
    """Every query against the oracle over the rows it sees of the first
    there[sequence] positions."""
    for i in range(len(pos)):
        rows = O.visible_rows(int(pos[i]), window, n_sink)
        rows = rows[rows < there[seq[i]]]
        if len(rows) == 0:
            assert (out[i] == 0).all() and (lse[i] == -np.inf).all(), f"query {i} sees nothing"
            continue
        o, l, spread, reach, total = O.gqa_attention(q64[i], cache.values("k", seq[i], rows),
                                                     cache.values("v", seq[i], rows))
        bo, bl = bounds(o, l, spread, reach, total, len(rows), cache.D)
        assert (np.abs(out[i] - o) <= bo).all() and (np.abs(lse[i] - l) <= bl).all(), f"query {i} at {pos[i]}"


WINDOWS = [(0, 0), (20, 3), (90, 2), (5, 0)]


@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [False, True])
def test_a_last_share_cut_short(group, D, window, n_sink):
    """Sequence 1's share of a contiguous plane ends after 100 of 128 rows:
    a query past them is reported and sees those before, the others of its
    run see theirs, and nothing is read behind the buffer."""
    rng = np.random.default_rng(31)
    cache = Cache(rng, 2, 128, 2, D, paged=False)
    cache.c = B.KVCache(2, D, *(B.Rows(x[:228], seq_rows=128) for x in cache.dev.values()))
    seq, pos = [1] * 6 + [0, 0], [99, 110, 64, 98, 127, 3, 127, 50]
    q, q64 = bf16(1.5 * rng.standard_normal((8, 6, D)))
    out, lse, status = attend(cache, q, seq, pos, window, n_sink, group)
    assert status == 6
    check(cache, q64, seq, pos, out, lse, window, n_sink, [128, 100])
    good = [0, 2, 3, 5, 6, 7]
    out, lse, status = attend(cache, q[good], [seq[i] for i in good], [pos[i] for i in good], window, n_sink, group)
    assert status == 0
    check(cache, q64[good], [seq[i] for i in good], [pos[i] for i in good], out, lse, window, n_sink, [128, 100])


@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (40, 2)])
@pytest.mark.parametrize("group", [False, True])
def test_a_last_page_cut_short(group, Hq, Hkv, window, n_sink):
    """The plane ends 20 rows into the page that holds positions 64 to 127 of
    sequence 0, in one plane after another; the pages behind it are whole."""
    rng = np.random.default_rng(32)
    D, last = 128, 5
    for cut in range(4):
        cache = Cache(rng, 2, 192, Hkv, D, paged=False)
        table = np.array([[0, last, 2], [3, 1, 4]], np.int32)
        rows = []
        for i, x in enumerate(cache.planes.values()):
            y = np.empty_like(x)
            for s in range(2):
                for p in range(3):
                    y[table[s, p] * PAGE:(table[s, p] + 1) * PAGE] = x[s * 192 + p * PAGE:s * 192 + (p + 1) * PAGE]
            d = torch.from_numpy(y).to(DEV)
            rows.append(B.Rows(d[:last * PAGE + 20] if i == cut else d, page_table=torch.from_numpy(table).to(DEV)))
        cache.c = B.KVCache(Hkv, D, *rows)
        seq, pos = [0, 0, 0, 1, 1], [83, 70, 100, 191, 80]
        q, q64 = bf16(1.5 * rng.standard_normal((5, Hq, D)))
        out, lse, status = attend(cache, q, seq, pos, window, n_sink, group)
        assert status == 6
        check(cache, q64, seq, pos, out, lse, window, n_sink, [84, 192])
        keep = [0, 1, 3, 4]
        out, lse, status = attend(cache, q[keep], [seq[i] for i in keep], [pos[i] for i in keep], window, n_sink, group)
        assert status == 0
        check(cache, q64[keep], [seq[i] for i in keep], [pos[i] for i in keep], out, lse, window, n_sink, [84, 192])


@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_given_back_between_far_windows(D, group):
    """Queries of one run far apart: pages that no window or sink reaches are
    gone from the table, in three ways; one that a window reaches is an error."""
    rng = np.random.default_rng(33)
    cache = Cache(rng, 1, 1024, 2, D, paged=True)
    seq, pos = [0] * 5, [1000, 130, 131, 40, 1001]
    q, q64 = bf16(1.5 * rng.standard_normal((5, 6, D)))
    for window, n_sink, gone in ((20, 3, range(3, 15)), (2, 0, [1, *range(3, 15)]), (64, 70, range(4, 14))):
        for value in (-1, -7, 10 ** 6):
            table = cache.dev_table.clone()
            table[0, list(gone)] = value
            rows = [B.Rows(x, page_table=table) for x in cache.dev.values()]
            call = B.KVCache(2, D, *rows)
            was, cache.c = cache.c, call
            out, lse, status = attend(cache, q, seq, pos, window, n_sink, group)
            cache.c = was
            assert status == 0
            check(cache, q64, seq, pos, out, lse, window, n_sink, [1024])
    table = cache.dev_table.clone()
    table[0, 2] = -1
    cache.c = B.KVCache(2, D, *(B.Rows(x, page_table=table) for x in cache.dev.values()))
    out, lse, status = attend(cache, q, seq, pos, 20, 3, group)
    assert status == 6
    check(cache, q64[[0, 3, 4]], [0] * 3, [1000, 40, 1001], out[[0, 3, 4]], lse[[0, 3, 4]], 20, 3, [1024])


@pytest.mark.parametrize("group", [False, True])
def test_logits_that_vanish(group):
    """Zero and tiny queries under a tiny softmax scale: every row that is seen
    weighs the same, none that is not."""
    rng = np.random.default_rng(34)
    cache = Cache(rng, 1, 200, 1, 128, paged=True)
    q = rng.standard_normal((6, 4, 128))
    q[0], q[2], q[3, 1], q[4] = 0, 0, 0, q[4] * 1e-30
    q, q64 = bf16(q)
    pos = [150, 151, 199, 30, 77, 0]
    for window, n_sink in ((0, 0), (40, 3)):
        out = torch.empty((6, 4, 128), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((6, 4), device=DEV)
        call = B.GqaAttn(cache.c, q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), out, window=window,
                         n_sink=n_sink, seq_of_query=torch.zeros(6, dtype=torch.int32, device=DEV), lse=lse,
                         softmax_scale=1e-20, group_queries=group)
        call.run()
        B.check_status(call.status)
        check_attention(cache, q64, [0] * 6, pos, out, lse, window, n_sink, scale=float(np.float32(1e-20)))


@pytest.mark.parametrize("D,G,nq", [(64, 40, 16384), (128, 40, 16384), (64, 300, 1400), (128, 1, 16384)])
def test_more_blocks_than_threads(D, G, nq):
    """The most queries of a call, in blocks of as few as one: the threads
    that look for where a CTA starts have several blocks each."""
    rng = np.random.default_rng(35)
    lens = [900, 64, 333, 5, 128, 700, 1, 512]
    cache = Cache(rng, 8, 900, 1, D, paged=True, lens=lens)
    seq = np.repeat(np.arange(8), nq // 8)
    pos = np.array([rng.integers(-1, lens[s]) for s in seq])
    q, q64 = bf16(rng.standard_normal((nq, G, D)).astype(np.float32))
    for window, n_sink in ((0, 0), (100, 3)):
        out, lse, status = attend(cache, q, seq, pos, window, n_sink, True)
        assert status == 0
        check_attention(cache, q64, seq, pos, torch.from_numpy(out), torch.from_numpy(lse), window, n_sink,
                        only=range(0, nq, nq // 60))


@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (7, 3), (64, 64), (128, 130), (129, 0), (300, 65), (2 ** 31 - 1, 5)])
def test_windows_of_wide_heads(window, n_sink, group):
    rng = np.random.default_rng(window % 1000 + n_sink)
    cache = Cache(rng, 2, 700, 2, 128, paged=True)
    pos = [0, 1, 2, 62, 63, 64, 65, 127, 128, 129, 191, 192, 300, 301, 302, 699]
    seq = [0] * 8 + [1] * 8
    q, q64 = bf16(1.5 * rng.standard_normal((16, 16, 128)))
    out, lse, status = attend(cache, q, seq, pos, window, n_sink, group)
    assert status == 0
    check(cache, q64, seq, pos, out, lse, window, n_sink, [700, 700])
