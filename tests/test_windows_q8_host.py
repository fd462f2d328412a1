"""Window attention and the 8-bit cache, as far as they go without a GPU (CPU).

* The plain forms in oracle/windows.py against closed forms and brute force.
* Every refusal of the C entry points: a call that passes all checks ends with PA_ERR_CUDA here.
"""

import numpy as np
import pytest
import torch

from oracle.windows import Cache8, attend_seen, seen
from test_operators_host import ALIGN, BF16, CUDA, DTYPE, F16, F32, I32, INVALID, SHAPE, STRIDE, U8, UNSUPPORTED, Call, desc


# ---- plain forms ---------------------------------------------------------------------------------------
def test_seen_positions():
    assert seen(9, 3, 0).tolist() == [7, 8, 9]
    assert seen(9, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert seen(9, 3, 7).tolist() == list(range(10))      # sinks that reach the window
    assert seen(9, 3, 100).tolist() == list(range(10))    # and beyond
    assert seen(1, 3, 2).tolist() == [0, 1]
    assert seen(0, 1, 0).tolist() == [0]
    assert seen(4, 0, 0).tolist() == list(range(5))


def test_window_attention_against_torch():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 64)), rng.standard_normal((40, 2, 64)), rng.standard_normal((40, 2, 64))
    j = torch.arange(40)
    mask = ((j > 29 - 11) & (j <= 29)) | (j < 3)
    t = [torch.from_numpy(x) for x in (q, k, v)]
    ref = torch.nn.functional.scaled_dot_product_attention(
        t[0][:, None], t[1].transpose(0, 1).repeat_interleave(2, 0), t[2].transpose(0, 1).repeat_interleave(2, 0),
        attn_mask=mask[None, None], scale=0.3)
    assert np.allclose(attend_seen(q, k, v, 29, 11, 3, 0.3), ref[:, 0].numpy(), atol=1e-12)
    assert not attend_seen(q, k[:0], v[:0], -1, 11, 3, 0.3).any()


def fresh(nb, H, B, D):
    return Cache8(np.full((nb, H, B, D), 7, np.uint8), np.full((nb, H), np.nan, np.float32))


def test_a_filled_frame_is_within_half_a_step():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((64, 3, 64)) * 10.0 ** rng.uniform(-3, 3, (1, 3, 1))).astype(np.float16)
    c = fresh(8, 3, 8, 64)
    table = rng.permutation(8)
    c.append(table, 64, x)
    y = c.values(table, 64)
    steps = c.steps[table].repeat(8, 0)[..., None].astype(np.float64)
    # code x r is rounded by half at most; step is 1 / r within 2^-24
    assert (np.abs(y - x.astype(np.float64)) <= steps * (0.5 + 127 * 2.0 ** -24)).all()
    top = np.abs(x.astype(np.float64)).reshape(8, 8, 3, 64).max((1, 3))
    assert (c.steps[table] <= top / 127 * (1 + 2.0 ** -7) * (1 + 2.0 ** -22)).all()   # 8 bits of r: no more than 2^-7 lost


def test_growing_a_frame_token_by_token():
    """However a frame grows, each token is off by less than a final step: halves of it, a quarter, an eighth ..."""
    rng = np.random.default_rng(3)
    for seed in range(20):
        x = (rng.standard_normal((32, 2, 64)) * 2.0 ** rng.uniform(-8, 8, (32, 1, 1))).astype(np.float16)
        c = fresh(2, 2, 32, 64)
        for n in range(1, 33):
            c.append([1, 0], n, x[n - 1:n])
        assert c.codes.min() >= 1 or seed  # the other frame is untouched
        y = c.values([1], 32)
        assert (np.abs(y - x.astype(np.float64)) < c.steps[1][:, None] * (1 + 127 * 2.0 ** -24)).all()
        grown = c.steps[1].astype(np.float64)
        first = fresh(1, 2, 32, 64)
        first.append([0], 1, x[:1])
        k = np.log2(grown / first.steps[0])
        assert np.array_equal(k, np.rint(k)) and (k >= 0).all()      # powers of two apart


def test_corner_frames():
    c = fresh(1, 1, 8, 64)
    c.append([0], 1, np.zeros((1, 1, 64)))
    assert (c.codes[0, 0, 0] == 128).all() and np.isclose(c.steps[0, 0], 2.0 ** -60 / 127, rtol=1e-6)
    c.append([0], 2, np.full((1, 1, 64), 2.0 ** 60 * 8, np.float32))    # beyond what counts: clamped
    v = c.values([0], 2)
    assert not v[0].any() and 2.0 ** 59 < v[1].min() <= 2.0 ** 60
    c.append([0], 3, np.full((1, 1, 64), np.nan))
    assert np.isnan(c.values([0], 3)).all() and (c.codes[0, 0, 2] == 128).all()
    c.append([0], 4, np.ones((1, 1, 64)))                               # stays NaN until it is begun anew
    assert np.isnan(c.steps[0, 0])
    c.append([0], 1, np.ones((1, 1, 64)))
    assert np.allclose(c.values([0], 1), 1)


# ---- refusals --------------------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("descriptors point at no memory: only where a call cannot launch")


def test_decode_window_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_decode_window", q=D(F16, 2, 8, 64), kc=D(F16, 4, 16, 2, 64), vc=D(F16, 4, 16, 2, 64), bt=D(I32, 2, 3), cl=D(I32, 2),
             window=5, sinks=0, scale=0.1, out=D(F16, 2, 8, 64), stream=None)
    assert f() == CUDA and f(window=2 ** 31 - 1, sinks=2 ** 31 - 1) == CUDA
    for name in ("q", "kc", "vc", "bt", "cl", "out"):
        assert f(**{name: None}) == INVALID, name
    for window, sinks in ((0, 0), (-1, 0), (0, 4), (5, -1)):
        assert f(window=window, sinks=sinks) == INVALID
    assert f(q=D(BF16, 2, 8, 64)) == DTYPE and f(out=D(BF16, 2, 8, 64)) == DTYPE and f(bt=D(F32, 2, 3)) == DTYPE
    assert f(kc=D(U8, 4, 16, 2, 64)) == DTYPE
    assert f(q=D(F16, 2, 7, 64)) == SHAPE and f(q=D(F16, 2, 8, 128)) == SHAPE and f(cl=D(I32, 3)) == SHAPE
    assert f(vc=D(F16, 5, 16, 2, 64)) == SHAPE
    assert f(q=D(F16, 2, 34, 64), out=D(F16, 2, 34, 64)) == UNSUPPORTED
    assert f(bt=D(I32, 2, 3, stride=(2, 1))) == STRIDE
    assert f(q=D(F16, 2, 8, 64, data=0x10008)) == ALIGN
    for shape in ((4, 12, 2, 64), (4, 16, 2, 32), (4, 512, 2, 64)):
        c = D(F16, *shape)
        assert f(kc=c, vc=c, q=D(F16, 2, 8, shape[3]), out=D(F16, 2, 8, shape[3])) == UNSUPPORTED
    c = D(F32, 4, 16, 2, 64)
    assert f(kc=c, vc=c) == UNSUPPORTED
    # 2^20 sequences of 2^27 parts of 16 keys, but no more than 30 of them in a window
    wide = dict(q=D(F16, 2 ** 20, 8, 64), out=D(F16, 2 ** 20, 8, 64), bt=D(I32, 2 ** 20, 2 ** 27 - 1), cl=D(I32, 2 ** 20))
    assert f(**wide, window=2 ** 31 - 1) == UNSUPPORTED and f(**wide, window=464) == CUDA
    assert f(q=D(F16, 0, 8, 64), out=D(F16, 0, 8, 64), bt=D(I32, 0, 3), cl=D(I32, 0)) == 0


def test_prefill_window_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_prefill_window", q=D(F16, 7, 8, 128), kc=D(F16, 4, 16, 2, 128), vc=D(F16, 4, 16, 2, 128), bt=D(I32, 2, 3), cl=D(I32, 2),
             qs=D(I32, 3), window=5, sinks=1, scale=0.1, out=D(F16, 7, 8, 128), stream=None)
    assert f() == CUDA
    for name in ("q", "kc", "vc", "bt", "cl", "qs", "out"):
        assert f(**{name: None}) == INVALID, name
    for window, sinks, scale in ((0, 0, 0.1), (-3, 0, 0.1), (5, -1, 0.1), (5, 0, 0.0), (5, 0, -0.1), (5, 0, float("nan")), (5, 0, float("inf"))):
        assert f(window=window, sinks=sinks, scale=scale) == INVALID
    assert f(q=D(BF16, 7, 8, 128)) == DTYPE and f(out=D(BF16, 7, 8, 128)) == DTYPE and f(qs=D(F32, 3)) == DTYPE
    assert f(q=D(F16, 7, 5, 128)) == SHAPE and f(out=D(F16, 7, 4, 128)) == SHAPE and f(out=D(F16, 6, 8, 128)) == SHAPE
    assert f(qs=D(I32, 2)) == SHAPE and f(vc=D(F16, 4, 8, 2, 128)) == SHAPE
    assert f(q=D(F16, 7, 34, 128), out=D(F16, 7, 34, 128)) == UNSUPPORTED
    for shape in ((4, 16, 2, 64), (4, 256, 2, 128), (4, 24, 2, 128)):
        c = D(F16, *shape)
        assert f(kc=c, vc=c, q=D(F16, 7, 8, shape[3]), out=D(F16, 7, 8, shape[3])) == UNSUPPORTED
    assert f(vc=D(F16, 4, 16, 2, 128, stride=(4096, 256, 128, 2))) == STRIDE
    assert f(q=D(F16, 0, 8, 128), out=D(F16, 0, 8, 128)) == 0


def q8(pa, **more):
    D = lambda *a, **k: desc(pa, *a, **k)
    return {"kc": D(U8, 4, 2, 16, 64), "vc": D(U8, 4, 2, 16, 64), "ks": D(F32, 4, 2), "vs": D(F32, 4, 2), **more}


def check_q8_caches(pa, f):
    D = lambda *a, **k: desc(pa, *a, **k)
    for name in ("kc", "vc", "ks", "vs"):
        assert f(**{name: None}) == INVALID, name
    assert f(kc=D(F16, 4, 2, 16, 64)) == DTYPE and f(vc=D(F16, 4, 2, 16, 64)) == DTYPE
    assert f(ks=D(F16, 4, 2)) == DTYPE and f(vs=D(I32, 4, 2)) == DTYPE
    assert f(vc=D(U8, 4, 2, 8, 64)) == SHAPE and f(ks=D(F32, 5, 2)) == SHAPE and f(vs=D(F32, 4, 3)) == SHAPE and f(vs=D(F32, 8)) == SHAPE
    assert f(kc=D(U8, 4, 2, 16, 64, stride=(2064, 1024, 64, 1))) == STRIDE
    assert f(ks=D(F32, 4, 2, stride=(1, 1))) == STRIDE and f(vs=D(F32, 4, 2, stride=(4, 2))) == STRIDE
    assert f(ks=D(F32, 4, 2, stride=(7, 1))) == f()                   # steps in wider rows
    assert f(kc=D(U8, 4, 2, 16, 64, data=0x10008)) == ALIGN and f(ks=D(F32, 4, 2, data=0x10002)) == ALIGN
    for shape in ((4, 2, 16, 96), (4, 2, 4, 64), (4, 2, 24, 64), (4, 2, 512, 64)):
        c = D(U8, *shape)
        assert f(kc=c, vc=c) == UNSUPPORTED, shape


def test_append_q8_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_cache_append_q8", k=D(F16, 7, 2, 64), v=D(F16, 7, 2, 64), bt=D(I32, 2, 3), cl=D(I32, 2), qs=D(I32, 3), **q8(pa), stream=None)
    assert f() == CUDA
    check_q8_caches(pa, f)
    for name in ("k", "v", "bt", "cl"):
        assert f(**{name: None}) == INVALID, name
    assert f(qs=None) == SHAPE                                        # 7 rows for 2 sequences
    assert f(qs=None, k=D(F16, 2, 2, 64), v=D(F16, 2, 2, 64)) == CUDA
    assert f(k=D(F32, 7, 2, 64)) == DTYPE and f(v=D(BF16, 7, 2, 64)) == DTYPE and f(qs=D(F32, 3)) == DTYPE
    assert f(k=D(F16, 7, 3, 64)) == SHAPE and f(v=D(F16, 6, 2, 64)) == SHAPE and f(qs=D(I32, 2)) == SHAPE and f(bt=D(I32, 3, 3)) == SHAPE
    assert f(k=D(F16, 7, 2, 64, stride=(132, 64, 1))) == ALIGN and f(k=D(F16, 7, 2, 64, stride=(256, 128, 1))) == STRIDE
    many = 2 ** 26                                                    # one token each: as many frames
    assert f(qs=None, k=D(F16, many, 2, 64), v=D(F16, many, 2, 64), bt=D(I32, many, 3), cl=D(I32, many)) == UNSUPPORTED
    assert f(k=D(F16, 0, 2, 64), v=D(F16, 0, 2, 64)) == 0
    assert f(qs=None, k=D(F16, 0, 2, 64), v=D(F16, 0, 2, 64), bt=D(I32, 0, 3), cl=D(I32, 0)) == 0


def test_read_q8_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_cache_read_q8", **q8(pa), slots=D(I32, 3), ko=D(BF16, 3, 2, 64), vo=D(BF16, 3, 2, 64), stream=None)
    assert f() == CUDA
    check_q8_caches(pa, f)
    for name in ("slots", "ko", "vo"):
        assert f(**{name: None}) == INVALID, name
    assert f(ko=D(F32, 3, 2, 64)) == DTYPE and f(vo=D(F16, 3, 2, 64)) == DTYPE
    assert f(ko=D(BF16, 4, 2, 64)) == SHAPE and f(slots=D(I32, 4)) == SHAPE and f(vo=D(BF16, 3, 2, 128)) == SHAPE
    assert f(slots=D(I32, 0), ko=D(BF16, 0, 2, 64), vo=D(BF16, 0, 2, 64)) == 0


def test_decode_q8_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_decode_q8", q=D(F16, 2, 8, 64), **q8(pa), bt=D(I32, 2, 3), cl=D(I32, 2), window=0, sinks=0, scale=0.1,
             out=D(F16, 2, 8, 64), stream=None)
    assert f() == CUDA and f(window=3, sinks=9) == CUDA
    check_q8_caches(pa, f)
    for name in ("q", "bt", "cl", "out"):
        assert f(**{name: None}) == INVALID, name
    for window, sinks in ((0, 1), (-1, 0), (3, -1)):
        assert f(window=window, sinks=sinks) == INVALID
    assert f(q=D(F32, 2, 8, 64)) == DTYPE and f(out=D(BF16, 2, 8, 64)) == DTYPE
    assert f(q=D(F16, 2, 7, 64)) == SHAPE and f(q=D(F16, 2, 8, 128)) == SHAPE and f(out=D(F16, 3, 8, 64)) == SHAPE
    assert f(q=D(F16, 2, 34, 64), out=D(F16, 2, 34, 64)) == UNSUPPORTED
    assert f(bt=D(I32, 2, 2 ** 28)) == UNSUPPORTED
    assert f(q=D(F16, 0, 8, 64), out=D(F16, 0, 8, 64), bt=D(I32, 0, 3), cl=D(I32, 0)) == 0


def test_copy_blocks_takes_8_bit_frames_and_their_steps(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_copy_blocks", kc=D(U8, 4, 2, 16, 64), vc=D(U8, 4, 2, 16, 64), pairs=D(I32, 1, 2), stream=None)
    assert f() == CUDA
    assert f(kc=D(F32, 4, 1, 1, 8), vc=D(F32, 4, 1, 1, 8)) == CUDA


def test_append_q8_refuses_what_a_launch_does_not_number(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_cache_append_q8", k=D(F16, 64, 2, 64), v=D(F16, 64, 2, 64), bt=D(I32, 2, 3), cl=D(I32, 2), qs=D(I32, 3), **q8(pa), stream=None)
    for seqs, code in ((2 ** 24 - 2, CUDA), (2 ** 24 - 1, UNSUPPORTED), (2 ** 31 - 2, UNSUPPORTED)):   # 64 / 16 + 2 S against 2^25
        assert f(bt=D(I32, seqs, 3), cl=D(I32, seqs), qs=D(I32, seqs + 1)) == code, seqs
