"""csa2_kv_append_fp4 (float32 and bfloat16 rows) against the oracle: codes,
scales and stored values bit for bit, rotated queries within their rounding,
and the cache followed by attention as a layer uses it."""
import numpy as np
import pytest
import torch

import oracle as O
from kv_cache_decode_csa2_b200 import csa2 as B
from tests.gqa_cases import DEV, PAGE, Cache, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def table(n_pos, rot):
    ang = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)


def to_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16)


class Batch:
    """n tokens of S sequences with padding rows, their q, k, v side by side
    (or apart) on the device, and the host's rotated values."""

    def __init__(self, rng, cache, Hq, seq, pos, rot, pairs, dt, packed=True, n_pos=None, change=None):
        Hkv, D, n = cache.Hkv, cache.D, len(pos)
        H = Hq + 2 * Hkv
        x = rng.standard_normal((n, H, D)).astype(np.float32)
        x *= np.where(rng.random((n, H, 1)) < 0.1, 30.0, 1.0).astype(np.float32)
        if change is not None:
            change(x)
        xd = torch.from_numpy(x).to(DEV).to(dt)
        self.x = xd.float().cpu().numpy()
        self.seq, self.pos, self.n, self.Hq = np.array(seq), np.array(pos), n, Hq
        parts = xd.split((Hq, Hkv, Hkv), 1) if packed else [t.contiguous() for t in xd.split((Hq, Hkv, Hkv), 1)]
        self.q, self.k, self.v = parts
        n_pos = int(max(pos)) + 1 if n_pos is None else n_pos
        cs = table(n_pos, rot)
        self.cos_sin = torch.from_numpy(cs).to(DEV) if rot else None
        turned = self.x.copy()
        if rot:
            at = np.maximum(self.pos, 0)
            a = cs[np.minimum(at, n_pos - 1)]
            turned[:, :Hq + Hkv] = O.rotate_heads(self.x[:, :Hq + Hkv], a[:, :rot // 2], a[:, rot // 2:], pairs)
        self.turned = turned
        self.kw = dict(seq_of_row=torch.tensor(seq, dtype=torch.int32, device=DEV), cos_sin=self.cos_sin,
                       interleaved=pairs)
        self.q_out = torch.full((n, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
        self.k_out = torch.full((n, Hkv, D), 9.0, dtype=torch.bfloat16, device=DEV)
        self.v_out = torch.full((n, Hkv, D), 9.0, dtype=torch.bfloat16, device=DEV)
        if Hq:
            self.kw.update(q=self.q, q_out=self.q_out)
        self.kw.update(k_out=self.k_out, v_out=self.v_out)

    def run(self, cache, **kw):
        p = torch.tensor(self.pos, dtype=torch.int32, device=DEV)
        return B.csa2_kv_append_fp4(cache.c, self.k, self.v, p, **{**self.kw, **kw})

    def check(self, cache, live=None):
        """Planes and outputs after the call: written rows hold the oracle's
        bytes, every other byte is what it was."""
        live = self.pos >= 0 if live is None else live
        Hq, Hkv, D = self.Hq, cache.Hkv, cache.D
        w = Hkv * D
        want = {k: p.copy() for k, p in cache.planes.items()}
        for kind, first, out in (("k", Hq, self.k_out), ("v", Hq + Hkv, self.v_out)):
            c, sc = O.fp4_quantize(self.turned[:, first:first + Hkv].reshape(self.n, w))
            for i in np.flatnonzero(live):
                at = cache.rows_of(self.seq[i], self.pos[i])
                want[kind + "_codes"][at, :w // 2], want[kind + "_scales"][at, :w // 32] = c[i], sc[i]
            stored = O.fp4_dequant(c, sc, w).reshape(self.n, Hkv, D)
            got = out.double().cpu().numpy()
            assert np.array_equal(got[live], stored[live])
            assert (got[~live] == 9).all()
        for k, p in want.items():
            assert np.array_equal(cache.dev[k].cpu().numpy(), p), k
            cache.planes[k] = p
        if Hq:
            q = self.q_out.double().cpu().numpy()
            assert np.array_equal(q[live], to_bf16(self.turned[:, :Hq]).double().numpy()[live])
            assert (q[~live] == 9).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 16), (64, 32), (64, 48), (64, 64), (128, 0), (128, 48), (128, 64),
                                   (128, 96), (128, 128)])
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
def test_append_matches_oracle(D, rot, pairs, dt):
    rng = np.random.default_rng(D + rot)
    cache = Cache(rng, 3, 150, 2, D, paged=True)
    seq = [0, 2, 2, 2, 1, 1, 0, 0]
    pos = [149, 0, 1, 2, 63, 64, -1, -5]
    b = Batch(rng, cache, 6, seq, pos, rot, pairs, dt)
    B.check_status(b.run(cache))
    b.check(cache)


@pytest.mark.parametrize("Hq,Hkv,n", [(0, 1, 1), (1, 1, 1), (3, 3, 5), (7, 1, 33), (64, 8, 32), (5, 5, 900), (64, 8, 2000)])
def test_append_heads_and_lengths(Hq, Hkv, n):
    """One token to a chunk that fills the device, odd head counts, no queries."""
    rng = np.random.default_rng(n + Hq)
    cache = Cache(rng, 1, 1, Hkv, 128, paged=False, garbage=3) if n == 1 else Cache(rng, 1, n + 7, Hkv, 128, paged=True,
                                                                                  lens=[7], garbage=3)
    pos = np.arange(n) + cache.R - PAGE * ((n + 63) // PAGE) if n == 1 else np.arange(7, n + 7)
    b = Batch(rng, cache, Hq, [0] * n, pos.tolist(), 128, False, torch.bfloat16, packed=n % 2 == 0)
    B.check_status(b.run(cache))
    b.check(cache)


def test_append_without_extra_outputs_and_in_place():
    rng = np.random.default_rng(21)
    cache = Cache(rng, 1, 70, 1, 64, paged=False)
    b = Batch(rng, cache, 4, [0, 0], [3, 68], 64, False, torch.bfloat16, packed=False)
    q = b.q.clone()
    B.check_status(b.run(cache, k_out=None, v_out=None, q=q, q_out=q))     # the queries turn in place
    b.q_out = q
    B.check_status(b.run(cache))
    b.q_out = q
    b.check(cache)


def test_append_special_values():
    """Zero blocks, scales at both ends, exact midpoints, infinities and NaN."""
    rng = np.random.default_rng(22)
    cache = Cache(rng, 1, 64, 1, 64, paged=False)
    mid = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0, -0.0, 6, -6, 7, 1,
                    2, 3, 4, .5, 1.5, -1, -2, -3, -4, -.5, -1.5], np.float32)

    def change(x):
        x[0] = 0
        x[1] *= 1e-6
        x[2] *= 1e-3
        x[3] *= 1e5
        x[4, :, :32], x[4, :, 32:] = mid, mid * 2.0 ** -9

    for dt in (torch.bfloat16, torch.float32):
        b = Batch(rng, cache, 1, [0] * 6, [0, 1, 2, 3, 4, 63], 0, False, dt, change=change)
        B.check_status(b.run(cache))
        b.check(cache)

        def odd(x):
            x[0, :, 3], x[0, :, 40] = np.inf, -np.inf
            x[1, :, 33] = np.nan

        b = Batch(rng, cache, 0, [0, 0], [7, 8], 0, False, dt, change=odd)
        B.check_status(b.run(cache))
        for kind, out in (("k", b.k_out), ("v", b.v_out)):
            sc = cache.dev[kind + "_scales"].cpu().numpy()
            cd = cache.dev[kind + "_codes"].cpu().numpy()
            assert sc[7].tolist() == [0x7E, 0x7E] and sc[8, 1] == 0x7F and sc[8, 0] != 0x7F
            assert (cd[8, 16:] == 0).all() and cd[7, 1] >> 4 == 7 and cd[7, 20] & 15 == 15
            v = out.double().cpu().numpy()
            assert v[0, 0, 3] == 2688 and v[0, 0, 40] == -2688
            assert np.isnan(v[1, 0, 32:]).all() and np.isfinite(v[1, 0, :32]).all()
        cache.planes = {k: t.cpu().numpy() for k, t in cache.dev.items()}


def test_append_refuses_tokens_out_of_range():
    """Past the rotation table, the pages, or a contiguous share: reported,
    nothing of that token written, the others stored."""
    rng = np.random.default_rng(23)
    cache = Cache(rng, 2, 128, 1, 64, paged=True)
    cache.dev_table[1, 1] = 10 ** 6
    b = Batch(rng, cache, 2, [0, 0, 1, 1, 0, -1], [100, 127, 63, 64, 128, 1], 64, True, torch.float32, n_pos=127)
    assert int(b.run(cache).item()) == 6
    b.check(cache, live=np.array([True, False, True, False, False, False]))
    cache = Cache(rng, 2, 128, 1, 64, paged=False)
    b = Batch(rng, cache, 2, [0, 0, 1, 1], [127, 128, 5, 128], 0, False, torch.bfloat16)
    assert int(b.run(cache).item()) == 6        # position 128 of sequence 0 is sequence 1's first row
    b.check(cache, live=np.array([True, False, True, False]))


def test_append_of_nothing():
    rng = np.random.default_rng(24)
    cache = Cache(rng, 1, 64, 1, 64, paged=False)
    e = torch.empty((0, 1, 64), device=DEV)
    B.check_status(B.csa2_kv_append_fp4(cache.c, e, e, torch.empty(0, dtype=torch.int32, device=DEV)))


def test_append_past_four_gigabytes_and_in_a_graph():
    rng = np.random.default_rng(25)
    Hkv, D = 8, 128
    rows = (5 << 30) // (Hkv * D // 2) // PAGE * PAGE
    tab = torch.tensor([[rows // PAGE - 1]], dtype=torch.int32, device=DEV)
    planes = [torch.zeros((rows, w), dtype=torch.uint8, device=DEV) for w in (512, 32, 512, 32)]
    c = B.KVCache(Hkv, D, *(B.Rows(x, page_table=tab) for x in planes))
    x = torch.randn(2, 3, Hkv, D, device=DEV)
    pos = torch.tensor([0, 63, 62], dtype=torch.int32, device=DEV)
    call = B.KVAppend(c, x[0], x[1], pos, seq_of_row=torch.zeros(3, dtype=torch.int32, device=DEV))
    call.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    for rep in range(2):
        x.normal_()
        graph.replay()
        B.check_status(call.status)
        for i in range(2):
            cd, sc = O.fp4_quantize(x[i].cpu().numpy().reshape(3, -1))
            at = [rows - 64, rows - 1, rows - 2]
            assert np.array_equal(planes[2 * i][at].cpu().numpy(), cd)
            assert np.array_equal(planes[2 * i + 1][at].cpu().numpy(), sc)


def test_append_on_another_stream():
    rng = np.random.default_rng(26)
    cache = Cache(rng, 1, 64, 2, 64, paged=True)
    b = Batch(rng, cache, 2, [0, 0], [5, 6], 64, False, torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    st = b.run(cache, stream=s)
    s.synchronize()
    B.check_status(st)
    b.check(cache)


def test_a_layer_over_prefill_and_decode():
    """A prompt in two chunks, then tokens one by one, of three ragged
    sequences: each step appends and attends, dense and windowed, on one
    cache; every output is the oracle's over the values stored so far."""
    rng = np.random.default_rng(27)
    S, Hq, Hkv, D = 3, 16, 2, 128
    cache = Cache(rng, S, 400, Hkv, D, paged=True, lens=[1] * S)
    have = [0, 0, 0]
    for lens in ([130, 37, 5], [64, 100, 1], [1, 1, 1], [1, 1, 1], [3, 5, 2]):
        T = max(lens)
        seq = np.repeat(np.arange(S), T)
        pos = np.concatenate([[have[s] + t if t < lens[s] else -1 for t in range(T)] for s in range(S)])
        b = Batch(rng, cache, Hq, seq.tolist(), pos.tolist(), 128, False, torch.bfloat16, n_pos=512)
        B.check_status(b.run(cache))
        b.check(cache)
        q64 = b.q_out.double().cpu().numpy()
        p = torch.tensor(pos, dtype=torch.int32, device=DEV)
        sq = torch.tensor(seq, dtype=torch.int32, device=DEV)
        some = rng.permutation(len(pos))[:24]
        for window, n_sink in ((0, 0), (50, 4)):
            out, lse = torch.empty_like(b.q_out), torch.empty((len(pos), Hq), device=DEV)
            call = B.GqaAttn(cache.c, b.q_out, p, out, seq_of_query=sq, lse=lse, window=window, n_sink=n_sink,
                             group_queries=T > 1)
            call.run()
            B.check_status(call.status)
            check_attention(cache, q64, seq, pos, out, lse, window, n_sink, only=some)
        have = [h + n for h, n in zip(have, lens)]
