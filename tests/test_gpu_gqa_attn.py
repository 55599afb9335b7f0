"""Grouped-query attention over the FP4 cache (csa2_gqa_attn_fp4,
csa2_gqa_window_attn_fp4) against the float64 oracle: head layouts, lengths
from one row on, windows and sinks, pages, padding, unwritten rows, refused
rows, streams and graphs."""
import numpy as np
import pytest
import torch

import oracle as O
from kv_cache_decode_csa2_b200 import csa2 as B
from tests.gqa_cases import DEV, PAGE, Cache, bf16, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def attend(cache, q, seq, pos, window=0, n_sink=0, **kw):
    """(out, lse) of one call; the status word must be clean."""
    nq, Hq, D = q.shape
    out = torch.full((nq, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((nq, Hq), 7.0, dtype=torch.float32, device=DEV)
    t = dict(seq_of_query=torch.tensor(seq, dtype=torch.int32, device=DEV), lse=lse, **kw)
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)
    if window:
        B.check_status(B.csa2_gqa_window_attn_fp4(cache.c, q.to(DEV), p, out, window, n_sink, **t))
    else:
        B.check_status(B.csa2_gqa_attn_fp4(cache.c, q.to(DEV), p, out, **t))
    return out, lse


def queries(rng, nq, Hq, D, scale=1.5):
    return bf16(scale * rng.standard_normal((nq, Hq, D)))


# (Hq, Hkv): one head per KV head, groups of 3, 8, 12, 16 and 40, one KV head for all
HEADS = [(4, 4), (6, 2), (8, 1), (64, 8), (24, 2), (32, 2), (40, 1), (9, 9), (64, 1), (60, 20)]


@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_heads(Hq, Hkv, D, group):
    rng = np.random.default_rng(Hq * 100 + Hkv + D)
    lens = [1, 200, 77]
    cache = Cache(rng, 3, 200, Hkv, D, paged=True, lens=lens)
    seq, pos = [0, 1, 1, 1, 2, 2], [0, 197, 198, 199, 76, -1]
    q, q64 = queries(rng, len(pos), Hq, D)
    out, lse = attend(cache, q, seq, pos, group_queries=group)
    check_attention(cache, q64, seq, pos, out, lse)


@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 4097])
def test_lengths(n, paged, group):
    rng = np.random.default_rng(n)
    cache = Cache(rng, 2, n, 2, 128, paged, lens=[n, max(1, n // 3)])
    seq = [0] * min(n, 3) + [1]
    pos = list(range(n - min(n, 3), n)) + [max(1, n // 3) - 1]
    q, q64 = queries(rng, len(pos), 8, 128)
    out, lse = attend(cache, q, seq, pos, group_queries=group)
    check_attention(cache, q64, seq, pos, out, lse)


@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (7, 3), (64, 64), (100, 4), (129, 0), (128, 130), (300, 65),
                                           (1000, 4), (2 ** 31 - 1, 5)])
def test_windows_and_sinks(window, n_sink, group):
    rng = np.random.default_rng(window % 1000 + n_sink)
    cache = Cache(rng, 2, 700, 2, 64, paged=True)
    pos = [0, 1, 2, 62, 63, 64, 65, 127, 128, 129, 191, 192, 300, 301, 302, 699]
    seq = [0] * 8 + [1] * 8
    q, q64 = queries(rng, len(pos), 6, 64)
    out, lse = attend(cache, q, seq, pos, window, n_sink, group_queries=group)
    check_attention(cache, q64, seq, pos, out, lse, window, n_sink)


@pytest.mark.parametrize("group", [False, True])
def test_every_position_of_a_chunk(group):
    """A prefill chunk at odd offsets, several sequences in one tile, padding between them."""
    rng = np.random.default_rng(3)
    cache = Cache(rng, 4, 400, 2, 128, paged=True)
    pos = list(range(211, 300)) + [-1] * 3 + list(range(0, 5)) + [-1] + list(range(350, 400)) + [17]
    seq = [2] * 92 + [0] * 6 + [3] * 50 + [1]
    for window, n_sink in ((0, 0), (50, 2)):
        q, q64 = queries(rng, len(pos), 10, 128)
        out, lse = attend(cache, q, seq, pos, window, n_sink, group_queries=group)
        check_attention(cache, q64, seq, pos, out, lse, window, n_sink)


@pytest.mark.parametrize("group", [False, True])
def test_positions_in_any_order(group):
    """Queries of a sequence need not be consecutive or ascending, nor the sequences."""
    rng = np.random.default_rng(4)
    cache = Cache(rng, 3, 333, 1, 128, paged=False)
    seq = rng.integers(0, 3, 70).tolist()
    pos = rng.integers(-1, 333, 70).tolist()
    q, q64 = queries(rng, 70, 5, 128)
    for window, n_sink in ((0, 0), (40, 9)):
        out, lse = attend(cache, q, seq, pos, window, n_sink, group_queries=group)
        check_attention(cache, q64, seq, pos, out, lse, window, n_sink)


@pytest.mark.parametrize("group", [False, True])
def test_values_no_query_sees_do_not_matter(group):
    """NaN scales in rows past a query's position, outside its window and in
    later queries' rows: the outputs are those of zero rows there."""
    rng = np.random.default_rng(5)
    cache = Cache(rng, 1, 260, 2, 128, paged=False, garbage=0xFF, lens=[260])
    seq, pos = [0] * 5, [99, 100, 130, 131, 258]
    q, q64 = queries(rng, 5, 16, 128)
    for kind in "kv":
        cache.planes[kind + "_scales"][[60, 131, 259]] = 0x7F       # 60 is the first query's, 131 the fourth's
        cache.planes[kind + "_codes"][[60, 131, 259]] = 0xFF
    cache.push()
    out, lse = attend(cache, q, seq, pos, 40, 10, group_queries=group)
    check_attention(cache, q64, seq, pos, out, lse, 40, 10, only=[1, 2, 4])
    assert torch.isnan(out[[0, 3]]).all() and torch.isnan(lse[[0, 3]]).all()


@pytest.mark.parametrize("group", [False, True])
def test_extreme_values(group):
    """The largest and smallest stored values and query magnitudes; one logit
    far above the others, late in the rows."""
    rng = np.random.default_rng(6)
    cache = Cache(rng, 1, 300, 1, 128, paged=False)
    for kind in "kv":
        cache.planes[kind + "_scales"][5] = 0x7E                    # 448
        cache.planes[kind + "_codes"][5] = 0x77                     # 6
        cache.planes[kind + "_scales"][6] = 0x01                    # 2^-9
        cache.planes[kind + "_scales"][7] = 0
    cache.push()
    q = rng.standard_normal((6, 4, 128))
    q[0] *= 1e-30
    q[1] *= 1e-6
    q[2] *= 20.0
    q[3] = 0.0
    q[4, :, 0] = 2.0 ** 20                                          # beside values near 1
    q[5] *= np.exp(4 * rng.standard_normal((4, 128)))
    q, q64 = bf16(q)
    out, lse = attend(cache, q, [0] * 6, [299] * 6, group_queries=group)
    check_attention(cache, q64, [0] * 6, [299] * 6, out, lse)


def test_flat_rows_beside_one_sink_still_count():
    """One row 20 (log2) above 60,000 equal ones: the many hold 6% of the mass."""
    n, D = 60000, 64
    rng = np.random.default_rng(7)
    cache = Cache(rng, 1, n, 1, D, paged=False, lens=[1])
    cache.planes["k_codes"][1:n], cache.planes["k_scales"][1:n] = 0, 0x38
    cache.planes["k_codes"][0], cache.planes["k_scales"][0] = 0x22, 0x38    # ones
    cache.planes["v_codes"][1:n], cache.planes["v_scales"][1:n] = 0x22, 0x38
    cache.planes["v_codes"][0], cache.planes["v_scales"][0] = 0, 0x38
    cache.push()
    q, q64 = bf16(np.full((1, 2, D), 20 * np.log(2) / 8))                   # logit 64 q / 8 = 20 ln 2
    for group in (False, True):
        out, lse = attend(cache, q, [0], [n - 1], group_queries=group)
        check_attention(cache, q64, [0], [n - 1], out, lse)
        assert (out > 0.05).all()


def test_padded_planes_and_keys_as_values():
    rng = np.random.default_rng(8)
    for kw in (dict(pad_bytes=2), dict(same=True)):
        cache = Cache(rng, 2, 150, 2, 128, paged=True, **kw)
        q, q64 = queries(rng, 2, 8, 128)
        for group in (False, True):
            out, lse = attend(cache, q, [1, 0], [149, 80], group_queries=group)
            check_attention(cache, q64, [1, 0], [149, 80], out, lse)


def test_planes_with_tables_of_their_own():
    """Each plane with its own page order (and one of them contiguous)."""
    rng = np.random.default_rng(9)
    cache = Cache(rng, 2, 200, 2, 64, paged=False)
    rows = {}
    for i, (name, x) in enumerate(cache.planes.items()):
        if i == 2:
            rows[name] = B.Rows(torch.from_numpy(x).to(DEV), seq_rows=cache.R)
            continue
        order = rng.permutation(x.shape[0] // PAGE)
        y = np.empty_like(x)
        for page, to in enumerate(order):
            y[to * PAGE:(to + 1) * PAGE] = x[page * PAGE:(page + 1) * PAGE]
        rows[name] = B.Rows(torch.from_numpy(y).to(DEV), page_rows=PAGE,
                            page_table=torch.tensor(order.reshape(2, -1), dtype=torch.int32, device=DEV))
    cache.c = B.KVCache(2, 64, *rows.values())
    q, q64 = queries(rng, 4, 8, 64)
    for group in (False, True):
        out, lse = attend(cache, q, [1, 1, 0, 0], [198, 199, 70, 71], group_queries=group)
        check_attention(cache, q64, [1, 1, 0, 0], [198, 199, 70, 71], out, lse)


def test_larger_pages_and_softmax_scale():
    rng = np.random.default_rng(10)
    cache = Cache(rng, 1, 500, 2, 128, paged=False)
    table = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device=DEV)
    r = [B.Rows(cache.dev[k], page_table=table, page_rows=128) for k in cache.planes]
    cache.c = B.KVCache(2, 128, *r)
    q, q64 = queries(rng, 3, 4, 128)
    for group in (False, True):
        out, lse = attend(cache, q, [0] * 3, [497, 498, 499], group_queries=group, softmax_scale=0.21)
        check_attention(cache, q64, [0] * 3, [497, 498, 499], out, lse, scale=float(np.float32(0.21)))


def test_bad_rows_are_reported_and_skipped():
    """A position past the plane, a page out of range, a negative sequence:
    INDEX_RANGE, the other queries of the call unharmed."""
    rng = np.random.default_rng(11)
    for group in (False, True):
        cache = Cache(rng, 2, 128, 1, 64, paged=True)
        cache.dev_table[0, 1] = 10 ** 6
        q, q64 = queries(rng, 3, 4, 64)
        for seq, pos, good in (([0, 1, 1], [100, 127, 5], [1, 2]), ([1, 1, 1], [127, 128, 10 ** 6], [0]),
                               ([-1, 1, 1], [4, 90, 91], [1, 2])):
            out = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device=DEV)
            lse = torch.zeros((3, 4), device=DEV)
            st = B.csa2_gqa_attn_fp4(cache.c, q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), out, lse=lse,
                                     seq_of_query=torch.tensor(seq, dtype=torch.int32, device=DEV), group_queries=group)
            assert int(st.item()) == 6
            check_attention(cache, q64, seq, pos, out, lse, only=good)
    cache = Cache(rng, 2, 128, 1, 64, paged=False)
    out = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device=DEV)
    st = B.csa2_gqa_attn_fp4(cache.c, q[:1].to(DEV), torch.tensor([128], dtype=torch.int32, device=DEV), out)
    assert int(st.item()) == 6                  # inside the buffer, but the next sequence's first row


def test_rows_past_four_gigabytes():
    """Pages at the far end of a plane of more than 2^32 bytes."""
    rng = np.random.default_rng(12)
    Hkv, D, n = 8, 128, 100
    rows = (5 << 30) // (Hkv * D // 2) // PAGE * PAGE
    cache = Cache(rng, 1, n, Hkv, D, paged=False)
    last = rows // PAGE - 1
    table = torch.tensor([[last, 3]], dtype=torch.int32, device=DEV)
    r = []
    for name, x in cache.planes.items():
        big = torch.empty((rows, x.shape[1]), dtype=torch.uint8, device=DEV)
        big[last * PAGE:], big[3 * PAGE:4 * PAGE] = torch.from_numpy(x[:64]).to(DEV), torch.from_numpy(x[64:128]).to(DEV)
        r.append(B.Rows(big, page_table=table))
    cache.c = B.KVCache(Hkv, D, *r)
    q, q64 = queries(rng, 2, 16, D)
    for group in (False, True):
        out, lse = attend(cache, q, [0, 0], [98, 99], group_queries=group)
        check_attention(cache, q64, [0, 0], [98, 99], out, lse)


def test_many_queries_and_no_seq():
    """More queries than CTAs, each its own sequence (seq_of_query NULL)."""
    rng = np.random.default_rng(13)
    lens = rng.integers(1, 130, 700).tolist()
    cache = Cache(rng, 700, 130, 1, 64, paged=True, lens=lens)
    pos = [n - 1 for n in lens]
    q, q64 = queries(rng, 700, 3, 64)
    for group in (False, True):
        out = torch.zeros((700, 3, 64), dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros((700, 3), device=DEV)
        B.check_status(B.csa2_gqa_attn_fp4(cache.c, q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), out,
                                           lse=lse, group_queries=group))
        check_attention(cache, q64, list(range(700)), pos, out, lse, only=range(0, 700, 7))


def test_repeats_are_bit_equal_and_unwritten_outputs_stay():
    rng = np.random.default_rng(14)
    cache = Cache(rng, 2, 3000, 2, 128, paged=True)
    q, _ = queries(rng, 9, 16, 128)
    seq, pos = [0] * 5 + [1] * 4, [2990, 2991, 2992, 2993, 2994, 7, 8, 9, 10]
    for group in (False, True):
        a, la = attend(cache, q, seq, pos, group_queries=group)
        for _ in range(3):
            b, lb = attend(cache, q, seq, pos, group_queries=group)
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_graphs_streams_and_a_shared_workspace():
    """Two captured calls that share one workspace, replayed with other
    contents and positions; an eager call on another stream beside them."""
    rng = np.random.default_rng(15)
    cache = Cache(rng, 2, 900, 2, 128, paged=True)
    need = B.lib().csa2_gqa_attn_workspace(4, 16, 2, 128)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    seq, calls = [0, 0, 1, 1], []
    for window in (0, 100):
        q, q64 = queries(rng, 4, 16, 128)
        qd = q.to(DEV)
        p = torch.tensor([10, 11, 20, 21], dtype=torch.int32, device=DEV)
        out, lse = torch.empty_like(qd), torch.empty((4, 16), device=DEV)
        call = B.GqaAttn(cache.c, qd, p, out, seq_of_query=torch.tensor(seq, dtype=torch.int32, device=DEV), lse=lse,
                         window=window, n_sink=3 if window else 0, group_queries=bool(window), ws=ws)
        call.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call.run()
        calls.append((graph, call, qd, p, out, lse, window))
    side = torch.cuda.Stream()
    for rep in range(3):
        pos = [100 * rep + 300, 100 * rep + 301, 899, -1]
        fresh = []
        for graph, call, qd, p, out, lse, window in calls:
            q, q64 = queries(rng, 4, 16, 128)
            qd.copy_(q)
            p.copy_(torch.tensor(pos, dtype=torch.int32))
            fresh.append(q64)
        torch.cuda.synchronize()
        other, _ = queries(rng, 1, 16, 128)
        out2 = torch.empty((1, 16, 128), dtype=torch.bfloat16, device=DEV)
        od, op = other.to(DEV), torch.tensor([512], dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        st = B.csa2_gqa_attn_fp4(cache.c, od, op, out2, stream=side)
        for graph, *_ in calls:
            graph.replay()
        torch.cuda.synchronize()
        B.check_status(st)
        for (graph, call, qd, p, out, lse, window), q64 in zip(calls, fresh):
            B.check_status(call.status)
            check_attention(cache, q64, seq, pos, out, lse, window, 3 if window else 0)


def test_shards_of_a_context_combine():
    """Attention over two halves of the rows, joined by csa2_attn_combine, is
    attention over all of them."""
    rng = np.random.default_rng(16)
    cache = Cache(rng, 1, 640, 2, 128, paged=False)
    q, q64 = queries(rng, 1, 8, 128)
    whole, whole_lse = attend(cache, q, [0], [600])
    first, first_lse = attend(cache, q, [0], [319])
    r = [B.Rows(cache.dev[k][320:], seq_rows=320) for k in cache.planes]
    cache.c = B.KVCache(2, 128, *r)
    rest, rest_lse = attend(cache, q, [0], [280])
    out, lse = torch.empty_like(whole), torch.empty_like(whole_lse)
    B.check_status(B.csa2_attn_combine(torch.stack((first, rest)), torch.stack((first_lse, rest_lse)), out, lse_out=lse))
    # each part's bf16 output and the joined one round by 2^-8; spread bounds |o|
    spread = np.abs(cache.values("v", 0, np.arange(600))).max()
    assert (out.double() - whole.double()).abs().max().item() <= 4 * 2.0 ** -8 * spread
    assert torch.allclose(lse, whole_lse, rtol=2.0 ** -20, atol=2.0 ** -18)


@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(300, 1), (514, 2)])
def test_groups_of_more_heads_than_a_block_holds(Hq, Hkv, group):
    rng = np.random.default_rng(17)
    cache = Cache(rng, 2, 150, Hkv, 64, paged=True)
    seq, pos = [0, 0, 1, 1], [148, 149, 3, -1]
    q, q64 = queries(rng, 4, Hq, 64)
    for window, n_sink in ((0, 0), (30, 2)):
        out, lse = attend(cache, q, seq, pos, window, n_sink, group_queries=group)
        check_attention(cache, q64, seq, pos, out, lse, window, n_sink)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (700, 5)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [3, 8])
def test_runs_of_many_sizes_in_one_call(G, D, window, n_sink):
    """Runs of 1 to 33 queries in one call, over few rows and over many that
    several CTAs share: every fill of a block, from one row to all of it, next
    to every other."""
    rng = np.random.default_rng(G + D)
    sizes = [1, 5, 8, 9, 16, 17, 32, 33, 2, 21, 7, 22]
    lens = [2900, 6000, 40, 1200, 5, 17, 700, 33, 4000, 21, 7, 22]
    rng.shuffle(lens)
    lens = [max(n, r) for n, r in zip(lens, sizes)]
    cache = Cache(rng, len(sizes), max(lens), 2, D, paged=True, lens=lens)
    seq = [s for s, r in enumerate(sizes) for _ in range(r)]
    pos = [lens[s] - r + i for s, r in enumerate(sizes) for i in range(r)]
    q, q64 = queries(rng, len(pos), 2 * G, D)
    out, lse = attend(cache, q, seq, pos, window, n_sink, group_queries=True)
    check_attention(cache, q64, seq, pos, out, lse, window, n_sink, only=range(0, len(pos), 3))
    again, lse2 = attend(cache, q, seq, pos, window, n_sink, group_queries=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("group", [False, True])
def test_two_handles_on_two_streams(group):
    """Calls in flight together, each with the workspace of its own handle."""
    rng = np.random.default_rng(18)
    cache = Cache(rng, 2, 2500, 2, 128, paged=True)
    seq, pos = [0, 0, 1, 1], [2498, 2499, 1000, 1001]
    calls = []
    for _ in range(2):
        q, q64 = queries(rng, 4, 16, 128)
        out = torch.empty((4, 16, 128), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((4, 16), device=DEV)
        h = B.GqaAttn(cache.c, q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), out, lse=lse,
                      seq_of_query=torch.tensor(seq, dtype=torch.int32, device=DEV), group_queries=group)
        calls.append((h, q64, out, lse, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for h, _, _, _, st in calls:
            h.run(stream=st)
    torch.cuda.synchronize()
    for h, q64, out, lse, _ in calls:
        B.check_status(h.status)
        check_attention(cache, q64, seq, pos, out, lse)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (20, 3)])
@pytest.mark.parametrize("group", [False, True])
def test_positions_past_every_row_harm_no_neighbour(group, window, n_sink):
    """Positions far past the rows (what an uninitialised tensor may hold) in
    the same run as good ones, at a number of rows that is no multiple of a
    page: reported, the others exact, and no longer a call than any."""
    rng = np.random.default_rng(19)
    cache = Cache(rng, 2, 192, 1, 64, paged=False, lens=[100, 100])
    for x in cache.planes.values():
        x[100:200] = x[192:292].copy()                # sequence 1 from row 100 on
    cache.R = 100
    cache.push()
    seq, pos = [0] * 4 + [1] * 4, [98, 99, 100, 2 ** 31 - 1, 0x7F7F7F7F, 64, 10 ** 9, 99]
    q, q64 = queries(rng, 8, 4, 64)
    out = torch.zeros((8, 4, 64), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((8, 4), device=DEV)
    call = B.GqaAttn(cache.c, q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV), out, lse=lse, window=window,
                     n_sink=n_sink, seq_of_query=torch.tensor(seq, dtype=torch.int32, device=DEV), group_queries=group)
    call.run()
    assert int(call.status.item()) == 6
    check_attention(cache, q64, seq, pos, out, lse, window, n_sink, only=[0, 1, 5, 7])


@pytest.mark.parametrize("group", [False, True])
def test_a_block_of_positions_past_every_row(group):
    """A whole block of such positions, each its own sequence, one head per KV head."""
    rng = np.random.default_rng(20)
    cache = Cache(rng, 1, 64, 1, 64, paged=False)
    q, _ = queries(rng, 300, 1, 64)
    pos = torch.full((300,), 0x7F7F7F7F, dtype=torch.int32, device=DEV)
    out = torch.zeros((300, 1, 64), dtype=torch.bfloat16, device=DEV)
    st = B.csa2_gqa_attn_fp4(cache.c, q.to(DEV), pos, out, group_queries=group)
    assert int(st.item()) == 6


@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("nq,Hq", [(6, 4), (40, 8)])
def test_logits_of_any_size(nq, Hq, group):
    """Queries of neighbouring rows whose logits lie between 2^0 and 2^100 (a
    diverged layer, a buffer nobody wrote), in every other head all of them
    negative.  Where one row's logit is ahead of every other by more than twice
    their error and 40 more, its weight is 1 to 300 e^-40 < 2^-49: the output
    is its values, rounded as a weight of f16 and to bf16, and the lse its
    logit.  Everywhere the output is an average."""
    rng = np.random.default_rng(21)
    cache = Cache(rng, 1, 300, 1, 128, paged=False)
    u = np.sign(rng.standard_normal(128))
    c, sc = O.fp4_quantize(u + 0.5 * rng.standard_normal((300, 128)))
    cache.planes["k_codes"][:300], cache.planes["k_scales"][:300] = c, sc
    cache.push()
    sizes = [4, 18, 27, 0, 22, 100, 3, 28, 20, 2, 33, 26, 60]
    e = np.array([sizes[i % len(sizes)] for i in range(nq)])
    q = rng.standard_normal((nq, Hq, 128))
    q[:, 1::2] = -u * np.abs(q[:, 1::2])
    q, q64 = bf16(q * 2.0 ** e[:, None, None])
    seq, pos = [0] * nq, list(range(300 - nq, 300))
    out, lse = attend(cache, q, seq, pos, group_queries=group)
    check_attention(cache, q64, seq, pos, out, lse, only=np.flatnonzero(e < 8))
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    certain = 0
    for i in np.flatnonzero(e > 8):
        k, v = (cache.values(x, 0, np.arange(pos[i] + 1))[:, 0] for x in "kv")
        assert (np.abs(out[i]) <= np.abs(v).max(0) * (1 + 2.0 ** -7)).all()
        logit = q64[i] @ k.T / np.sqrt(128)
        assert (logit[1::2] < 0).all()
        d = (128 + 4) * 2.0 ** -24 * (np.abs(q64[i]) @ np.abs(k).T / np.sqrt(128)).max(1)
        order = np.argsort(logit, 1)
        for h in range(Hq):
            first, second = order[h, -1], order[h, -2]
            if logit[h, first] - logit[h, second] > 2 * d[h] + 40:
                certain += 1
                assert (np.abs(out[i, h] - v[first]) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(v[first]) + 2.0 ** -40).all()
            assert abs(lse[i, h] - logit[h, first]) <= d[h] + np.log(300) + 2.0 ** -22 * abs(logit[h, first])
    assert certain > 0.9 * (e > 8).sum() * Hq


@pytest.mark.parametrize("group", [False, True])
def test_a_handle_dropped_while_its_stream_works(group):
    """Made on one stream, run with another as the current one, dropped: its
    workspace is not handed out before the other stream is through."""
    rng = np.random.default_rng(22)
    cache = Cache(rng, 1, 3000, 2, 128, paged=True)
    pos = [2996, 2997, 2998, 2999]
    q, q64 = queries(rng, 4, 16, 128)
    out, lse = torch.empty((4, 16, 128), dtype=torch.bfloat16, device=DEV), torch.empty((4, 16), device=DEV)
    status = B.new_status(DEV)
    qd, p = q.to(DEV), torch.tensor(pos, dtype=torch.int32, device=DEV)
    seq = torch.zeros(4, dtype=torch.int32, device=DEV)
    call = B.GqaAttn(cache.c, qd, p, out, seq_of_query=seq, lse=lse, group_queries=group, status=status)
    at, n = call.keep["ws"].data_ptr(), call.keep["ws"].numel()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)             # about 10 ms
        call.run()
    del call
    again = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert again.data_ptr() != at
    again.fill_(0xFF)
    torch.cuda.synchronize()
    B.check_status(status)
    check_attention(cache, q64, [0] * 4, pos, out, lse)
