"""Clipping by the global norm (ttt_clip_gradients through the C ABI) against float64.

Tolerances: the norm is summed in fp64 from fp32 sums of eight squares (each sum within 8 * 2^-24 of its
value): 5e-7.  A scaled value is one fp32 product and one rounding: 2^-8 (bf16) or 2^-23 (fp32, factor and product) of
the value, plus the factor's own error, the norm's."""
import math

import pytest
import torch

from vision_test_token_b200 import clip_gradients

pytestmark = pytest.mark.gpu

NORM = 5e-7
VALUE = {torch.bfloat16: 2 ** -8 + 1e-6, torch.float32: 2 ** -23 + 2 ** -24 + NORM}


def _norm(xs):
    return math.sqrt(sum(float(x.double().square().sum()) for x in xs))


def _check(xs, max_norm, out):
    before = [x.clone() for x in xs]
    norm = clip_gradients(xs, max_norm, out=out)
    torch.cuda.synchronize()
    want = _norm(before)
    assert norm.shape == (1,) and norm.dtype == torch.float32
    assert abs(float(norm) - want) <= NORM * want
    f = min(1.0, max_norm / want) if want > 0 else 1.0
    for x, o, b in zip(xs, out or xs, before):
        if out is not None:
            assert torch.equal(x, b)
        err = (o.double() - b.double() * f).abs()
        assert (err <= VALUE[o.dtype] * (b.double() * f).abs() + 1e-40).all()
    return norm


def _tensors(sizes, dev, seed=0, offset=False):
    g = torch.Generator(device=dev).manual_seed(seed)
    xs = []
    for i, n in enumerate(sizes):
        dt = (torch.bfloat16, torch.float32)[i % 2]
        k = i % 9 if offset else 0
        xs.append((torch.randn(n + k, generator=g, device=dev) * 10 ** (i % 3 - 1)).to(dt)[k:])
    return xs


SIZES = [
    [1], [7, 8], [0, 5, 0], [16384, 16385, 65536, 65537, 3], [1000003, 17, 2, 31, 32, 33, 4099, 300007],
    list(range(0, 700)),                        # more tensors than one launch's table holds
]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("offset", [False, True])
@pytest.mark.parametrize("apart", [False, True])
def test_clip(cuda_dev, sizes, offset, apart):
    for max_norm in (1.0, 1e6, 0.0):
        xs = _tensors(sizes, cuda_dev, len(sizes), offset)
        out = None
        if apart:                               # outputs whose alignment differs from the inputs'
            out = [torch.empty(x.numel() + 3, dtype=x.dtype, device=cuda_dev)[3:] if i % 2 else torch.empty_like(x)
                   for i, x in enumerate(xs)]
        _check(xs, max_norm, out)


def test_nothing_else_is_written(cuda_dev):
    buf = torch.full((5, 1001), 2.0, device=cuda_dev)
    xs = [buf[i, 1:1000] for i in (0, 2, 4)]
    _check(xs, 1.0, None)
    assert (buf[1] == 2).all() and (buf[3] == 2).all() and (buf[:, 0] == 2).all() and (buf[:, 1000] == 2).all()


def test_large_tensor(cuda_dev):
    """More than 2^31 elements, and the tail past them."""
    n = 2 ** 31 + 77
    x = torch.zeros(n, dtype=torch.bfloat16, device=cuda_dev)
    x[-40:] = 3.0
    x[5] = 4.0
    norm = clip_gradients([x], 1.0)
    want = math.sqrt(40 * 9 + 16)
    assert abs(float(norm) - want) <= NORM * want
    assert abs(float(x[-1]) * want - 3) <= 3 * 2 ** -8 and abs(float(x[5]) * want - 4) <= 4 * 2 ** -8
    assert int(torch.count_nonzero(x[: 2 ** 30])) == 1
    del x
    torch.cuda.empty_cache()


def test_extreme_values(cuda_dev):
    """Squares beyond fp32's range on either side; infinities and NaN."""
    one = lambda v, dt=torch.float32: torch.full((100,), v, dtype=dt, device=cuda_dev)  # noqa: E731
    for v in (1e30, 1e-25, 1e-30):
        for dt in (torch.float32, torch.bfloat16):
            xs = [one(v, dt), one(0.0)]
            norm = clip_gradients(xs, 1.0)
            want = 10 * float(one(v, dt)[0].double())
            assert abs(float(norm) - want) <= 1e-6 * want
            assert abs(float(xs[0][0].double()) / (v if want < 1 else 0.1) - 1) <= 2 ** -7
    xs = [one(2.0), one(float("inf"))]
    assert float(clip_gradients(xs, 1.0)) == math.inf
    assert not xs[0].any() and torch.isnan(xs[1]).all()
    xs = [one(2.0), one(float("nan"))]
    assert math.isnan(float(clip_gradients(xs, 1.0)))
    assert torch.isnan(xs[0]).all()
    xs = [one(0.0)]
    assert float(clip_gradients(xs, 0.0)) == 0 and not xs[0].any()
    xs = [one(2.0)]
    assert abs(float(clip_gradients(xs, math.inf)) - 20) <= 1e-5 and (xs[0] == 2).all()


def test_same_bits_twice_and_captured(cuda_dev):
    xs = _tensors([100003, 77, 500000], cuda_dev, 5)
    out = [torch.empty_like(x) for x in xs]
    n1 = clip_gradients(xs, 1.0, out=out)
    first = [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        n2 = clip_gradients(xs, 1.0, out=out)
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n1, n2) and all(torch.equal(a, b) for a, b in zip(first, out))


def test_refusals(cuda_dev):
    x = torch.ones(64, device=cuda_dev)
    for bad in ([], [x.cpu()], [x.half()], [x.view(8, 8).t()], [x, x.cpu()]):
        with pytest.raises(ValueError):
            clip_gradients(bad, 1.0)
    for kw in (dict(out=[]), dict(out=[x[:5]]), dict(out=[x.bfloat16()])):
        with pytest.raises(ValueError):
            clip_gradients([x], 1.0, **kw)
    for grads, max_norm, out in (([x, x], 1.0, None),                        # the same tensor twice
                                 ([x[:40], x[30:]], 1.0, None),              # overlapping
                                 ([x[:40]], 1.0, [x[8:48]]),                 # an output over part of its input
                                 ([x[:8], x[8:16]], 1.0, [x[8:16], x[:8]]),  # an output over another's input
                                 ([x], -1.0, None), ([x], float("nan"), None)):
        with pytest.raises(RuntimeError, match="INVALID"):
            clip_gradients(grads, max_norm, out=out)
    assert (x == 1).all()
