"""The grouped-query entry points without a GPU: refusals of the C ABI and of
the binding, workspace sizes, struct layout, the failed launch; and pins of
the oracle's grouped-query functions on something other than themselves."""
import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest
import torch

import kv_cache_decode_csa2_b200 as K
import oracle as O
from kv_cache_decode_csa2_b200 import csa2 as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, BIG = 1 << 20, 1 << 40
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: only without a GPU")


def _rows(row_bytes, base=A, n_rows=4096, seq_rows=4096, page_rows=0, max_pages=0, table=None):
    r = B.csa2_rows()
    r.base, r.row_bytes, r.n_rows = base, row_bytes, n_rows
    r.page_table, r.page_rows, r.max_pages, r.seq_rows = table, page_rows, max_pages, seq_rows
    return r


def _cache(Hkv=8, D=128, **change):
    c = B.csa2_kv_cache()
    c.Hkv, c.D = Hkv, D
    for name, w in (("k_codes", D // 2), ("k_scales", D // 32), ("v_codes", D // 2), ("v_scales", D // 32)):
        setattr(c, name, change.get(name, _rows(Hkv * w, base=A + (1 << 20) * (name[0] == "v"))))
    return c


def _append(c, bf16=False, q=A, k=A, v=A, n=4, Hq=64, ld_q=8192, ld_k=1024, ld_v=1024, seq=None, pos=A, cos=A, n_pos=9,
            rot=128, q_out=A + 64, k_out=None, v_out=None, status=A):
    fn = K.lib().csa2_kv_append_fp4_bf16 if bf16 else K.lib().csa2_kv_append_fp4
    return fn(q, k, v, n, Hq, ld_q, ld_k, ld_v, seq, pos, cos, n_pos, rot, 0, ctypes.byref(c) if c else None, q_out,
              k_out, v_out, status, None)


def _attn(c, q=A, pos=A, nq=3, Hq=64, out=A, lse=None, ws=A, ws_bytes=BIG, status=A, window=None, n_sink=0):
    L = K.lib()
    head = (q, ctypes.byref(c) if c else None, None, pos, nq, Hq)
    tail = (0.0, 1, out, lse, ws, ws_bytes, status, None)
    if window is None:
        return L.csa2_gqa_attn_fp4(*head, *tail)
    return L.csa2_gqa_window_attn_fp4(*head, window, n_sink, *tail)


def test_append_refuses_bad_arguments():
    c = _cache()
    for kw, code in ((dict(k=None), 1), (dict(v=None), 1), (dict(pos=None), 1), (dict(status=None), 1), (dict(n=-1), 1),
                     (dict(q=None), 1), (dict(q_out=None), 1), (dict(Hq=0), 1), (dict(q=A + 8), 1), (dict(k=A + 4), 1),
                     (dict(q_out=A + 8), 1), (dict(k_out=A + 8), 1), (dict(v_out=A + 8), 1), (dict(ld_k=1020), 1),
                     (dict(ld_k=1022), 1), (dict(ld_v=512), 1), (dict(ld_q=8188), 1), (dict(cos=None), 1),
                     (dict(cos=A + 4), 1), (dict(n_pos=0), 1), (dict(rot=8), 2), (dict(rot=-16), 2), (dict(rot=144), 2),
                     (dict(Hq=1025, ld_q=1 << 20), 2), (dict(Hq=-1), 2)):
        assert _append(c, **kw) == code, kw
    assert _append(c, bf16=True, ld_k=1028) == 1                 # bf16 rows start on 16 bytes: multiples of 8 values
    assert _append(None) == 1
    for bad in (_cache(D=96), _cache(D=512), _cache(Hkv=0), _cache(Hkv=257)):
        assert _append(bad) == 2
    for bad in (_cache(k_codes=_rows(496)), _cache(v_codes=_rows(520)), _cache(k_scales=_rows(28)),
                _cache(v_scales=_rows(34)), _cache(k_codes=_rows(512, base=None)), _cache(v_codes=_rows(512, base=A + 8)),
                _cache(k_scales=_rows(32, n_rows=0)), _cache(k_codes=_rows(512, table=A, page_rows=32, max_pages=2)),
                _cache(v_scales=_rows(32, table=A, page_rows=64, max_pages=0)), _cache(k_codes=_rows(512, seq_rows=-1))):
        assert _append(bad) == 1
    for name, w in (("v_codes", 512), ("v_scales", 32)):         # keys and values in one plane
        assert _append(_cache(**{name: _rows(w)})) == 1
    # an output over an input of another layout
    assert _append(c, ld_q=8200, q_out=A, bf16=True) == 1 and _append(c, q_out=A) == 1
    assert _append(c, k_out=A) == 1 and _append(c, v_out=A, ld_v=1032, bf16=True) == 1
    assert _append(c, n=0, k=None, v=None, pos=None, q=None, Hq=0, q_out=None) == 0     # nothing to do


def test_attention_refuses_bad_arguments():
    c = _cache()
    for kw, code in ((dict(q=None), 1), (dict(pos=None), 1), (dict(out=None), 1), (dict(status=None), 1), (dict(nq=0), 1),
                     (dict(q=A + 8), 1), (dict(out=A + 2), 1), (dict(nq=16385), 2), (dict(Hq=60), 2), (dict(Hq=0), 2),
                     (dict(Hq=1032), 2), (dict(ws=None), 3), (dict(ws=A + 16), 3), (dict(ws_bytes=1000), 3),
                     (dict(window=0), 1), (dict(window=-3), 1), (dict(window=4, n_sink=-1), 1),
                     (dict(window=4, n_sink=2, ws=None), 3)):
        assert _attn(c, **kw) == code, kw
    assert _attn(None) == 1
    for bad in (_cache(D=512), _cache(Hkv=0)):
        assert _attn(bad) == 2
    for bad in (_cache(k_codes=_rows(496)), _cache(v_scales=_rows(28)), _cache(v_codes=_rows(512, base=None))):
        assert _attn(bad) == 1


def test_workspace_sizes():
    w = K.lib().csa2_gqa_attn_workspace
    assert w(1, 64, 8, 128) >= 64 * 128 * 4
    assert w(1, 64, 8, 128) <= w(4096, 64, 8, 128) < 1 << 28
    for bad in ((0, 64, 8, 128), (16385, 64, 8, 128), (1, 64, 7, 128), (1, 64, 8, 96), (1, 0, 8, 128), (1, 64, 0, 128),
                (1, 2048, 8, 128), (1, 512, 257, 64)):
        assert w(*bad) == 0, bad


@no_gpu
def test_failed_launches_are_reported():
    for D in (64, 128):
        c = _cache(D=D)
        assert _append(c, rot=64) == 4
        assert _append(c, bf16=True, rot=0, cos=None) == 4
        assert _attn(c) == 4
        assert _attn(c, window=100, n_sink=4) == 4
    assert _attn(_cache(Hkv=1), nq=1) == 4


@no_gpu
def test_random_arguments_return_documented_codes():
    rng = random.Random(5)

    def p():
        return rng.choice([None, A, A, A + 4, A + 8])

    def i():
        return rng.choice([-1, 0, 1, 2, 8, 16, 64, 128, 1024, 1025, 8192, 16384, 16385, 1 << 30])

    def rows():
        return _rows(rng.choice([0, 4, 16, 32, 34, 64, 256, 512, 1024]), base=p(), n_rows=rng.choice([0, 1, 4096, 1 << 31]),
                     seq_rows=rng.choice([-1, 0, 64]), table=p(), page_rows=rng.choice([0, 32, 64, 128]),
                     max_pages=rng.choice([0, 1, 8]))

    for _ in range(600):
        c = _cache(rng.choice([-1, 0, 1, 8, 256, 300]), rng.choice([0, 64, 128, 512]),
                   **{k: rows() for k in ("k_codes", "k_scales", "v_codes", "v_scales") if rng.random() < 0.3})
        n = i()
        assert _append(c, bf16=rng.random() < 0.5, q=p(), k=p(), v=p(), n=n, Hq=i(), ld_q=i(), ld_k=i(), ld_v=i(),
                       seq=p(), pos=p(), cos=p(), n_pos=i(), rot=i(), q_out=p(), k_out=p(), v_out=p(),
                       status=p()) in ({0, 1, 2, 4} if n == 0 else {1, 2, 4})
        assert _attn(c, q=p(), pos=p(), nq=i(), Hq=i(), out=p(), lse=p(), ws=p(), ws_bytes=max(0, i()) * 1024, status=p(),
                     window=rng.choice([None, -1, 0, 1, 64, 2 ** 31 - 1]), n_sink=i()) in {1, 2, 3, 4}


def test_the_binding_refuses_before_the_library():
    n = torch.zeros(2, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):                              # planes on the CPU
        B.KVCache(1, 128, *(B.Rows(n) for _ in range(4)))
    with pytest.raises(ValueError):
        B._heads(torch.zeros(4, 2, 64), 2, 64, torch.bfloat16, 4, "k")
    with pytest.raises(ValueError):
        B._heads(torch.zeros(4, 3, 64), 2, 64, torch.float32, 4, "k")
    with pytest.raises(ValueError):                              # heads apart
        B._heads(torch.zeros(4, 2, 128)[:, :, :64], 2, 64, torch.float32, 4, "k")
    assert B._heads(torch.zeros(4, 5, 64)[:, 1:3], 2, 64, torch.float32, 4, "k") == 320
    assert B._heads(torch.zeros(1, 2, 64), 2, 64, torch.float32, 1, "k") == 128


class _Stream:
    def __init__(self, raw):
        self.cuda_stream, self.waited = raw, []

    def wait_event(self, event):
        self.waited.append(event)


class _Tensor:
    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream.cuda_stream)


@pytest.mark.parametrize("given", [False, True])
def test_scratch_is_held_for_every_stream_that_works_with_it(monkeypatch, given):
    """A handle made on stream 7 and run on 8 and 9, as the current stream or
    by name: its scratch is recorded on both before each first launch, which
    waits for it to be made; a capturing stream cannot wait."""
    current, capturing = [_Stream(7)], []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: current[-1].cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: current[-1])

    class using:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            current.append(self.s)

        def __exit__(self, *a):
            current.pop()

    monkeypatch.setattr(torch.cuda, "stream", using)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[-1].cuda_stream in capturing)
    launched = []
    t = _Tensor()
    call = object.__new__(B.GqaAttn)
    call.name, call.device, call.args, call.scratch = "fake", torch.device("cuda:0"), (), (t,)
    call.streams, call.made = {7}, "made"
    call.fn = lambda raw: launched.append((raw, list(t.streams))) or 0
    eight, nine = _Stream(8), _Stream(9)
    for s in (None, eight, eight, nine):
        if s is None:
            call.run()
        elif given:
            call.run(stream=s)
        else:
            with using(s):
                call.run()
    assert launched == [(7, []), (8, [8]), (8, [8]), (9, [8, 9])]
    assert eight.waited == nine.waited == ["made"]
    capturing.append(10)
    ten = _Stream(10)
    call.run(stream=ten)
    assert t.streams[-1] == 10 and ten.waited == [] and launched[-1][0] == 10


def test_ctypes_struct_matches_the_header(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in B.csa2_kv_cache._fields_]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "csa2.h"', "int main(void) {",
             '  printf("%zu", sizeof(csa2_kv_cache));']
    lines += [f'  printf(" %zu", offsetof(csa2_kv_cache, {f}));' for f in names] + ["  return 0;", "}"]
    (tmp_path / "probe.c").write_text("\n".join(lines))
    subprocess.run([gcc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "probe.c"), "-o",
                    str(tmp_path / "probe")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "probe")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(B.csa2_kv_cache)] + [getattr(B.csa2_kv_cache, f).offset for f in names]


# ----------------------------------------------------------------- the oracle's pins
@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_is_a_complex_product(pairs):
    rng = np.random.default_rng(1)
    x, ang = rng.standard_normal((5, 3, 64)), rng.uniform(0, 7, (5, 24))
    y = O.rotate_heads(x, np.cos(ang), np.sin(ang), pairs)
    assert np.array_equal(y[:, :, 48:], x[:, :, 48:])
    a, b = (slice(0, 48, 2), slice(1, 48, 2)) if pairs else (slice(0, 24), slice(24, 48))
    z = (x[:, :, a] + 1j * x[:, :, b]) * np.exp(1j * ang)[:, None]
    assert np.allclose(y[:, :, a] + 1j * y[:, :, b], z, rtol=0, atol=1e-13)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (1, 0), (5, 2), (3, 9), (100, 4)])
def test_visible_rows_position_by_position(window, n_sink):
    for pos in range(12):
        want = [p for p in range(pos + 1) if window == 0 or pos - p < window or p < n_sink]
        assert O.visible_rows(pos, window, n_sink).tolist() == want


def test_gqa_attention_is_sdpa_and_sparse_attention():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((6, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    o, lse, spread, reach, total = O.gqa_attention(q, k, v)
    t = [torch.from_numpy(np.ascontiguousarray(x)) for x in (q[:, None], k.transpose(1, 0, 2), v.transpose(1, 0, 2))]
    want = torch.nn.functional.scaled_dot_product_attention(t[0][None], t[1][None].repeat_interleave(3, 1),
                                                            t[2][None].repeat_interleave(3, 1))[0, :, 0].numpy()
    assert np.allclose(o, want, rtol=0, atol=1e-13)
    assert (np.abs(o) <= spread + 1e-15).all() and (spread <= total + 1e-15).all() and (reach > 0).all()
    same = O.gqa_attention(q, k[:, :1], k[:, :1])
    ref = O.sparse_attention(q, k[:, 0])
    assert np.allclose(same[0], ref[0], rtol=0, atol=1e-13) and np.allclose(same[1], ref[1], rtol=0, atol=1e-13)
    empty = O.gqa_attention(q, k[:0], v[:0])
    assert (empty[0] == 0).all() and (empty[1] == -np.inf).all()
