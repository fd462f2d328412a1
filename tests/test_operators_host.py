"""The rotating append, the 4-bit cache and the block-sparse decode, as far as they go without a GPU (CPU).

* The plain forms in oracle/operators.py against closed forms and brute force.
* Every refusal of the C entry points: the arguments are checked before anything touches a device, so a
  call that passes all checks ends with PA_ERR_CUDA here, and one that does not with its own code.
"""

import ctypes as C
import math

import numpy as np
import pytest
import torch

from oracle.operators import (attend, block_bounds, block_scores, cos_sin_table, quantise_q4, rotate, select_blocks,
                              values_q4)

INVALID, DTYPE, SHAPE, STRIDE, ALIGN, CUDA, UNSUPPORTED = -1, -2, -3, -4, -5, -9, -10


# ---- plain forms ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 64])
def test_rotation_keeps_lengths_and_relative_angles(rot, interleaved):
    rng = np.random.default_rng(1)
    table = cos_sin_table(64, rot)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    at = lambda x, p: rotate(x, table, [p], interleaved)[0, 0]
    assert np.linalg.norm(at(q, 17)) == pytest.approx(np.linalg.norm(q), rel=1e-6)
    # q . k depends on the distance of the positions alone
    assert at(q, 9) @ at(k, 4) == pytest.approx(at(q, 41) @ at(k, 36), rel=1e-5)
    assert np.array_equal(at(q, 0), q[0, 0])
    assert np.array_equal(at(q, 5)[rot:], q[0, 0, rot:])


def test_quantised_rows_are_within_half_a_step():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((200, 64)) * 10.0 ** rng.uniform(-3, 3, (200, 1)) + rng.standard_normal((200, 1))).astype(np.float32)
    rows = quantise_q4(x)
    assert rows.shape == (200, 40)
    y = values_q4(rows)
    g = x.reshape(200, 2, 32).astype(np.float64)
    step = (g.max(-1) - g.min(-1)) / 15
    # half a step, widened by what fp16 rounds of the step (2^-11, 15 times) and of offset and value (2^-11 of the largest)
    tol = step * (0.5 + 16 * 2.0 ** -11) + 2 * 2.0 ** -11 * np.abs(g).max(-1) + 2.0 ** -24
    assert (np.abs(y.reshape(g.shape) - g) <= tol[..., None]).all()


def test_quantised_corner_groups():
    x = np.zeros((6, 32), np.float32)
    x[1] = 3.5                                        # one value: no step
    x[2, :2] = [-1e6, 1e6]                            # beyond fp16: clamped
    x[3, 5] = np.nan
    x[4, 6] = -np.inf
    x[5] = np.linspace(0, 15, 32)
    y = values_q4(quantise_q4(x))
    assert np.array_equal(y[0], np.zeros(32)) and np.array_equal(y[1], np.full(32, 3.5))
    # clamped to +-65024; the step 130048 / 15 = 8669.9 is 8672 in fp16, and -65024 + 15 * 8672 = 65056
    assert y[2, 0] == -65024 and y[2, 1] == 65056
    assert np.isnan(y[3]).all() and np.isnan(y[4]).all()
    assert np.array_equal(y[5], np.rint(np.linspace(0, 15, 32)))


def test_codes_stand_for_what_the_bytes_say():
    row = np.zeros(40, np.uint8)
    row[0] = 0xA3                                     # element 0: 3, element 1: 10
    row[16] = 0x0F                                    # element 32: 15
    row[32:40] = np.array([0.5, -1.0, 2.0, 0.25], np.float16).view(np.uint8)
    v = values_q4(row)
    assert v[0] == 0.5 and v[1] == 4.0 and v[2] == -1.0 and v[32] == 30.25 and v[33] == 0.25


def test_scores_bound_every_product():
    rng = np.random.default_rng(3)
    k = rng.standard_normal((5, 8, 2, 64)).astype(np.float32)
    q = rng.standard_normal((6, 64)).astype(np.float32)
    b = np.stack([block_bounds(f, 8) for f in k])
    s = block_scores(q, b)
    for h in range(2):
        best = np.einsum("nbd,gd->nbg", k[:, :, h].astype(np.float64), q[3 * h:3 * h + 3].astype(np.float64)).max((1, 2))
        assert (s[:, h] >= best - 1e-3).all()
    one = block_scores(q[:2], np.stack([k[:, 0], k[:, 0]], axis=2))  # bounds of a single key: the product itself
    assert np.allclose(one, np.stack([k[:, 0, 0] @ q[0], k[:, 0, 1] @ q[1]], 1), atol=1e-4)


def test_selection_order():
    scores = np.array([[1.0], [5.0], [5.0], [4.0], [5.0], [0.0]], np.float32)
    assert select_blocks(scores, 2, 0, 0).tolist() == [[1, 2]]
    assert select_blocks(scores, 3, 0, 1).tolist() == [[1, 2, 5]]
    assert select_blocks(scores, 3, 1, 1).tolist() == [[0, 1, 5]]
    assert select_blocks(scores, 2, 4, 4).tolist() == [[0, 1]]       # more kept than taken: the lower ones
    assert select_blocks(scores, 8, 0, 0).tolist() == [[0, 1, 2, 3, 4, 5, -1, -1]]


def test_plain_attention_against_torch():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((4, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    t = [torch.from_numpy(x) for x in (q, k, v)]
    ref = torch.nn.functional.scaled_dot_product_attention(t[0][:, None], t[1].transpose(0, 1).repeat_interleave(2, 0),
                                                           t[2].transpose(0, 1).repeat_interleave(2, 0), scale=0.3)
    assert np.allclose(attend(q, k, v, 0.3), ref[:, 0].numpy(), atol=1e-12)
    assert not attend(q, k[:0], v[:0], 0.3).any()


# ---- refusals --------------------------------------------------------------------------------------------
F32, F16, BF16, I32, U8 = 0, 1, 2, 3, 4


def desc(pa, dtype, *shape, stride=None, data=0x10000):
    """A tensor descriptor of memory that is never touched."""
    d = pa.PaTensor()
    d.data, d.dtype, d.ndim = data, dtype, len(shape)
    step = 1
    strides = []
    for n in reversed(shape):
        strides.insert(0, step)
        step *= n
    for i, n in enumerate(shape):
        d.shape[i] = n
        d.stride[i] = (stride or strides)[i]
    return d


class Call:
    """A call's arguments by name; variants replace some of them."""

    def __init__(self, pa, fn, **args):
        self.pa, self.fn, self.args = pa, fn, args

    def __call__(self, **other):
        args = {**self.args, **other}
        return getattr(self.pa.LIB, self.fn)(*[C.byref(x) if isinstance(x, C.Structure) else x for x in args.values()])


@pytest.fixture(scope="module")
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("descriptors point at no memory: only where a call cannot launch")


@pytest.fixture()
def rope(pa, no_gpu):
    return Call(pa, "pa_cache_append_rope", k=desc(pa, F16, 3, 2, 64), v=desc(pa, F16, 3, 2, 64), slots=desc(pa, I32, 3),
                kc=desc(pa, F16, 4, 16, 2, 64), vc=desc(pa, F16, 4, 16, 2, 64), pos=desc(pa, I32, 3), cs=desc(pa, F32, 100, 64),
                inter=0, q=desc(pa, F16, 3, 8, 64), qo=desc(pa, F16, 3, 8, 64), stream=None)


def test_rope_refusals(pa, rope):
    D = lambda *a, **k: desc(pa, *a, **k)
    assert rope() == CUDA
    assert rope(q=None, qo=None) == CUDA
    assert rope(k=D(F16, 0, 2, 64), v=D(F16, 0, 2, 64), slots=D(I32, 0), pos=D(I32, 0), q=None, qo=None) == 0
    for name in ("k", "v", "slots", "kc", "vc", "pos", "cs", "q", "qo"):
        assert rope(**{name: None}) == INVALID, name
    assert rope(pos=None, cs=None, q=None, qo=None) == INVALID        # pa_cache_append does that
    assert rope(inter=2) == INVALID
    assert rope(k=D(BF16, 3, 2, 64)) == DTYPE
    assert rope(q=D(BF16, 3, 8, 64)) == DTYPE
    assert rope(cs=D(F16, 100, 64)) == DTYPE
    assert rope(pos=D(F32, 3)) == DTYPE
    assert rope(kc=D(U8, 4, 2, 16, 40)) == DTYPE
    assert rope(vc=D(F16, 5, 16, 2, 64)) == SHAPE
    assert rope(pos=D(I32, 4)) == SHAPE
    assert rope(slots=D(I32, 2)) == SHAPE
    assert rope(q=D(F16, 4, 8, 64)) == SHAPE
    assert rope(qo=D(F16, 3, 4, 64)) == SHAPE
    for r in (0, 8, 24, 80):                                          # not a multiple of 16, or more than D
        assert rope(cs=D(F32, 100, r)) == SHAPE, r
    assert rope(cs=D(F32, 100, 64, stride=(32, 1))) == STRIDE
    assert rope(cs=D(F32, 100, 64, stride=(66, 1))) == ALIGN
    assert rope(cs=D(F32, 100, 64, data=0x10004)) == ALIGN
    assert rope(q=D(F16, 3, 8, 64, stride=(516, 64, 1))) == ALIGN
    assert rope(q=D(F16, 3, 8, 64, stride=(1024, 128, 1))) == STRIDE
    assert rope(k=D(F32, 3, 2, 256), v=D(F32, 3, 2, 256), kc=D(F32, 4, 16, 2, 256), vc=D(F32, 4, 16, 2, 256)) == UNSUPPORTED


@pytest.fixture()
def append4(pa, no_gpu):
    return Call(pa, "pa_cache_append_q4", k=desc(pa, F16, 3, 2, 64), v=desc(pa, F16, 3, 2, 64), slots=desc(pa, I32, 3),
                kc=desc(pa, U8, 4, 2, 16, 40), vc=desc(pa, U8, 4, 2, 16, 40), pos=desc(pa, I32, 3), cs=desc(pa, F32, 100, 64),
                inter=0, q=desc(pa, F16, 3, 8, 64), qo=desc(pa, F16, 3, 8, 64), stream=None)


def test_append_q4_refusals(pa, append4):
    D = lambda *a, **k: desc(pa, *a, **k)
    assert append4() == CUDA
    assert append4(pos=None, cs=None, q=None, qo=None) == CUDA
    for name in ("k", "v", "slots", "kc", "vc", "pos", "cs", "q", "qo"):
        assert append4(**{name: None}) == INVALID, name
    assert append4(pos=None, cs=None) == INVALID                      # queries without a rotation
    assert append4(k=D(F32, 3, 2, 64)) == DTYPE
    assert append4(kc=D(F16, 4, 2, 16, 40)) == DTYPE
    assert append4(vc=D(F16, 4, 2, 16, 40)) == DTYPE
    assert append4(vc=D(U8, 4, 2, 8, 40)) == SHAPE
    assert append4(k=D(F16, 3, 2, 128)) == SHAPE
    assert append4(kc=D(U8, 4, 2, 16, 40, stride=(1300, 640, 40, 1))) == STRIDE
    assert append4(vc=D(U8, 4, 2, 16, 40, stride=(1296, 640, 40, 1))) == STRIDE
    assert append4(kc=D(U8, 4, 2, 16, 40, data=0x10008)) == ALIGN
    for w in (32, 48, 160):
        c = D(U8, 4, 2, 16, w)
        assert append4(kc=c, vc=c) == UNSUPPORTED, w
    for b in (4, 24, 512):
        c = D(U8, 4, 2, b, 40)
        assert append4(kc=c, vc=c) == UNSUPPORTED, b
    big = D(U8, 2 ** 27, 2, 16, 40)
    assert append4(kc=big, vc=big) == UNSUPPORTED                     # slots pass int32


def test_read_q4_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_cache_read_q4", kc=D(U8, 4, 2, 16, 80), vc=D(U8, 4, 2, 16, 80), slots=D(I32, 3), ko=D(BF16, 3, 2, 128),
             vo=D(BF16, 3, 2, 128), stream=None)
    assert f() == CUDA
    for name in ("kc", "vc", "slots", "ko", "vo"):
        assert f(**{name: None}) == INVALID, name
    assert f(ko=D(F32, 3, 2, 128)) == DTYPE and f(vo=D(F16, 3, 2, 128)) == DTYPE
    assert f(ko=D(BF16, 4, 2, 128)) == SHAPE and f(slots=D(I32, 4)) == SHAPE
    assert f(slots=D(I32, 0), ko=D(BF16, 0, 2, 128), vo=D(BF16, 0, 2, 128)) == 0


def test_decode_q4_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_decode_q4", q=D(F16, 2, 8, 64), kc=D(U8, 4, 2, 16, 40), vc=D(U8, 4, 2, 16, 40), bt=D(I32, 2, 3), cl=D(I32, 2),
             scale=0.1, out=D(F16, 2, 8, 64), stream=None)
    assert f() == CUDA
    for name in ("q", "kc", "vc", "bt", "cl", "out"):
        assert f(**{name: None}) == INVALID, name
    assert f(q=D(F32, 2, 8, 64)) == DTYPE and f(out=D(BF16, 2, 8, 64)) == DTYPE
    assert f(q=D(F16, 2, 7, 64)) == SHAPE                             # 7 heads over 2
    assert f(q=D(F16, 2, 1, 64)) == SHAPE
    assert f(q=D(F16, 2, 8, 128)) == SHAPE
    assert f(out=D(F16, 2, 4, 64)) == SHAPE and f(bt=D(I32, 3, 3)) == SHAPE and f(cl=D(I32, 3)) == SHAPE
    assert f(q=D(F16, 2, 34, 64), out=D(F16, 2, 34, 64)) == UNSUPPORTED   # 17 query heads a key head
    assert f(bt=D(I32, 2, 2 ** 28)) == UNSUPPORTED
    assert f(bt=D(I32, 2, 3, stride=(2, 1))) == STRIDE
    assert f(q=D(F16, 0, 8, 64), out=D(F16, 0, 8, 64), bt=D(I32, 0, 3), cl=D(I32, 0)) == 0


def test_bounds_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_block_bounds", kc=D(F16, 4, 16, 2, 64), bt=D(I32, 2, 3), cl=D(I32, 2), first=D(I32, 2), b=D(F16, 4, 2, 2, 64),
             stream=None)
    assert f() == CUDA and f(first=None) == CUDA
    for name in ("kc", "bt", "cl", "b"):
        assert f(**{name: None}) == INVALID, name
    assert f(b=D(BF16, 4, 2, 2, 64)) == DTYPE and f(first=D(F32, 2)) == DTYPE
    assert f(b=D(F16, 5, 2, 2, 64)) == SHAPE and f(b=D(F16, 4, 2, 1, 64)) == SHAPE and f(first=D(I32, 3)) == SHAPE
    assert f(kc=D(F32, 4, 16, 2, 64)) == UNSUPPORTED and f(kc=D(F16, 4, 12, 2, 64)) == UNSUPPORTED


def test_select_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_select_blocks", q=D(F16, 2, 8, 64), b=D(F16, 4, 2, 2, 64), bt=D(I32, 2, 3), cl=D(I32, 2), B=16, first=1, last=1,
             sel=D(I32, 2, 2, 5), stream=None)
    assert f() == CUDA
    for name in ("q", "b", "bt", "cl", "sel"):
        assert f(**{name: None}) == INVALID, name
    assert f(first=-1) == INVALID and f(last=-1) == INVALID
    assert f(q=D(BF16, 2, 8, 64)) == DTYPE and f(sel=D(F32, 2, 2, 5)) == DTYPE
    assert f(b=D(F16, 4, 2, 3, 64)) == SHAPE and f(sel=D(I32, 2, 3, 5)) == SHAPE and f(sel=D(I32, 2, 2, 0)) == SHAPE
    assert f(sel=D(I32, 2, 2, 5, stride=(5, 5, 1))) == STRIDE and f(sel=D(I32, 2, 2, 5, stride=(20, 10, 2))) == STRIDE
    for b in (0, 4, 12, 512):
        assert f(B=b) == UNSUPPORTED, b


def test_decode_selected_refusals(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_decode_selected", q=D(F16, 2, 8, 64), kc=D(F16, 4, 16, 2, 64), vc=D(F16, 4, 16, 2, 64), bt=D(I32, 2, 3), cl=D(I32, 2),
             sel=D(I32, 2, 2, 5), scale=0.1, out=D(F16, 2, 8, 64), stream=None)
    assert f() == CUDA
    for name in ("q", "kc", "vc", "bt", "cl", "sel", "out"):
        assert f(**{name: None}) == INVALID, name
    assert f(q=D(BF16, 2, 8, 64)) == DTYPE and f(out=D(BF16, 2, 8, 64)) == DTYPE
    assert f(sel=D(I32, 3, 2, 5)) == SHAPE and f(q=D(F16, 2, 3, 64)) == SHAPE
    c = D(F32, 4, 16, 2, 64)
    assert f(kc=c, vc=c) == UNSUPPORTED
    c = D(F16, 4, 10, 2, 64)
    assert f(kc=c, vc=c) == UNSUPPORTED


def test_copy_blocks_takes_4_bit_frames(pa, no_gpu):
    D = lambda *a, **k: desc(pa, *a, **k)
    f = Call(pa, "pa_copy_blocks", kc=D(U8, 4, 2, 16, 40), vc=D(U8, 4, 2, 16, 40), pairs=D(I32, 1, 2), stream=None)
    assert f() == CUDA
    assert f(kc=D(U8, 4, 1, 1, 40), vc=D(U8, 4, 1, 1, 40)) == ALIGN   # frames of 40 bytes
    assert f(vc=D(F16, 4, 2, 16, 40)) == DTYPE
