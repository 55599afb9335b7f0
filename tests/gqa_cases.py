"""Random grouped-query caches and batches for the tests of csa2_kv_append_fp4
and csa2_gqa_attn_fp4, and the error bounds their results are held to."""
import numpy as np
import torch

import oracle as O
from kv_cache_decode_csa2_b200 import csa2 as B

DEV = "cuda"
PAGE = 64


class Cache:
    """Planes of S sequences of up to `rows` positions, filled with FP4 rows
    of normal values; host copies of the bytes.  Rows nobody wrote hold
    `garbage` bytes (0xFF is a NaN scale)."""

    def __init__(self, rng, S, rows, Hkv, D, paged, garbage=0xFF, pad_bytes=0, same=False, lens=None):
        self.S, self.Hkv, self.D, self.paged = S, Hkv, D, paged
        self.R = -(-rows // PAGE) * PAGE
        n = S * self.R + (2 * PAGE if paged else 0)
        self.table = None
        if paged:
            self.table = rng.permutation(n // PAGE)[:S * self.R // PAGE].astype(np.int32).reshape(S, -1)
        self.planes = {}
        for name, w in (("k_codes", Hkv * D // 2), ("k_scales", Hkv * D // 32), ("v_codes", Hkv * D // 2),
                        ("v_scales", Hkv * D // 32)):
            step = 16 if "codes" in name else D // 32
            self.planes[name] = np.full((n, w + pad_bytes * step), garbage, np.uint8)
        lens = [rows] * S if lens is None else lens
        for s in range(S):
            for kind in "kv":
                x = rng.standard_normal((lens[s], Hkv * D)) * np.exp(rng.standard_normal((lens[s], 1)))
                c, sc = O.fp4_quantize(x)
                at = self.rows_of(s, np.arange(lens[s]))
                self.planes[kind + "_codes"][at, :c.shape[1]] = c
                self.planes[kind + "_scales"][at, :sc.shape[1]] = sc
        self.same = same
        self.push()

    def rows_of(self, s, pos):
        if self.table is None:
            return s * self.R + pos
        return self.table[s, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE

    def push(self):
        """Device copies of the planes."""
        self.dev = {k: torch.from_numpy(v).to(DEV) for k, v in self.planes.items()}
        self.dev_table = None if self.table is None else torch.from_numpy(self.table).to(DEV)
        v = [B.Rows(self.dev[k], page_table=self.dev_table, page_rows=PAGE, seq_rows=self.R) for k in self.planes]
        self.c = B.KVCache(self.Hkv, self.D, v[0], v[1], *(v[:2] if self.same else v[2:]))

    def values(self, kind, s, pos):
        """float64 [len(pos)][Hkv][D] of the host bytes."""
        kind = "k" if self.same else kind
        at = self.rows_of(s, np.asarray(pos))
        w = self.Hkv * self.D
        x = O.fp4_dequant(self.planes[kind + "_codes"][at, :w // 2], self.planes[kind + "_scales"][at, :w // 32], w)
        return x.reshape(len(at), self.Hkv, self.D)


def bf16(x):
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


def bounds(o, lse, spread, reach, total, n, D):
    """(|out - o|, |lse - lse64|) at most.  Counted: the bf16 output, half a
    step of eps 2^-7; a weight rounded to f16, 2^-11 of it; logits summed in
    fp32 over D products and scaled, (D + 4) 2^-24 of the products' sum,
    which moves numerator and denominator alike at worst in opposite
    directions; n weights and n products summed in fp32 (one step each,
    2^-23); exponentials and rescalings, 2^-20.  A weight is held as
    2^(s - m + 10) with m at most the largest logit so far, so that a row's
    largest is at least 2^10; f16's smallest step is 2^-24, so each weight is
    off by up to 2^-25 absolutely, 2^-35 of the sum of weights."""
    d_logit = ((D + 4) * 2.0 ** -24 * reach)[:, None]
    w = 2.0 ** -11 + 2 * d_logit + 2 * n * 2.0 ** -23 + 2.0 ** -20
    return 2.0 ** -8 * np.abs(o) + w * spread + 2.0 ** -35 * total + 1e-30, d_logit[:, 0] + n * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)


def check_attention(cache, q64, seq, pos, out, lse, window=0, n_sink=0, scale=None, only=None):
    """Every query's output and lse against the oracle."""
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in range(len(pos)) if only is None else only:
        rows = O.visible_rows(int(pos[i]), window, n_sink) if pos[i] >= 0 else np.zeros(0, np.int64)
        o, l, spread, reach, total = O.gqa_attention(q64[i], cache.values("k", seq[i], rows),
                                                     cache.values("v", seq[i], rows), scale)
        if len(rows) == 0:
            assert (out[i] == 0).all() and (lse[i] == -np.inf).all(), f"query {i} sees nothing"
            continue
        bo, bl = bounds(o, l, spread, reach, total, len(rows), cache.D)
        err = np.abs(out[i] - o)
        assert (err <= bo).all(), f"query {i} at {pos[i]}: {np.nanmax(err / bo):.3g} of the bound, worst {np.nanmax(err):.3g}"
        el = np.abs(lse[i] - l)
        assert (el <= bl).all(), f"query {i} at {pos[i]}: lse off by {np.nanmax(el):.3g}, bound {bl.min():.3g}"
