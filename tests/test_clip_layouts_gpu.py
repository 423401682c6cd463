"""Clipping of gradients that are laid out by token ([B][heads][N][d] views of [B][N][heads][d] tensors), as the backward pass of the
gated delta rule gives them for such inputs.

Tolerances as in test_clip_gpu: the norm 5e-7; a scaled value one fp32 product and one rounding, and the norm's error."""
import pytest
import torch

from tests.test_clip_gpu import NORM, VALUE, _check
from tests.test_gated_delta_gpu import INPUTS, _make, _on
from vision_test_token_b200 import backward_gated_delta, clip_gradients

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,hk,h,N", [(2, 1, 2, 90), (1, 2, 2, 1), (3, 1, 1, 33)])
def test_token_major_gradients(cuda_dev, dtype, B, hk, h, N):
    y = _on(_make(B, hk, h, N, 64, 128, dtype, "tokens", "shared", seed=60), cuda_dev)
    grads = list(backward_gated_delta(*(y[n] for n in INPUTS), y["dZ"], W0=y["W0"]))
    if h > 1 and N > 1:
        assert not grads[2].is_contiguous() and grads[2].transpose(1, 2).is_contiguous()
    whole = [g.clone(memory_format=torch.contiguous_format) for g in grads]
    norm = clip_gradients(grads, 0.5)
    torch.cuda.synchronize()
    want = torch.stack([g.double().square().sum() for g in whole]).sum().sqrt()
    assert abs(float(norm) / float(want) - 1) <= NORM and float(want) > 0.5
    for g, w in zip(grads, whole):
        exact = w.double() * (0.5 / want)
        assert ((g.double() - exact).abs() <= VALUE[g.dtype] * exact.abs() + 1e-40).all()


def test_into_outputs(cuda_dev):
    xs = [torch.randn((2, 40, 3, 64), device=cuda_dev).to(dt).transpose(1, 2) for dt in (torch.bfloat16, torch.float32)]
    xs.append(torch.randn((2, 40, 3), device=cuda_dev).transpose(1, 2))
    out = [torch.empty_like(x) for x in xs]
    assert all(o.stride() == x.stride() for o, x in zip(out, xs))
    _check(xs, 1.0, out)


def test_refusals(cuda_dev):
    x = torch.ones((2, 40, 3, 64), device=cuda_dev).transpose(1, 2)
    for bad in (x[:, :, ::2], x[..., :32], x.transpose(0, 1), x.transpose(2, 3), x[:, :2]):
        with pytest.raises(ValueError):
            clip_gradients([bad], 1.0)
    with pytest.raises(ValueError):                               # an output in another order
        clip_gradients([x], 1.0, out=[torch.empty((2, 3, 40, 64), device=cuda_dev)])
    with pytest.raises(ValueError):
        clip_gradients([x.contiguous()], 1.0, out=[torch.empty_like(x)])
    assert (x == 1).all()
