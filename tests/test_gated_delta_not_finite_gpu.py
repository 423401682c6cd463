"""A NaN or an infinity of one token reaches that token and later ones only, as in the recurrence, although the tokens of a
chunk are computed together: what comes before has the bits of a call without it."""
import pytest
import torch

from tests.test_gated_delta_gpu import INPUTS, _make, _on
from vision_test_token_b200 import forward_gated_delta

pytestmark = pytest.mark.gpu

N = 70


def _run(y):
    W1 = torch.empty((y["V"].shape[0], y["V"].shape[1], y["V"].shape[3], y["Q"].shape[3]), device=y["Q"].device)
    Z = forward_gated_delta(*(y[n] for n in INPUTS), W0=y["W0"], W1_out=W1)
    torch.cuda.synchronize()
    return Z, W1


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name,value", [("K", "nan"), ("V", "nan"), ("G", "nan"), ("Beta", "nan"), ("Q", "nan"), ("K", "inf"),
                                        ("V", "-inf"), ("Beta", "inf"), ("Q", "inf")])
def test_one_token(cuda_dev, dtype, d, name, value):
    y = _on(_make(2, 1, 2, N, d, d, dtype, w0="each", seed=40), cuda_dev)
    clean_Z, clean_W1 = _run(y)
    for t in (0, 1, 7, 15, 16, 17, 30, 31, 32, 50, 63, 64, 69):
        bad = dict(y)
        bad[name] = y[name].clone()
        at = (1, 0, t) + ((5,) if bad[name].dim() == 4 else ())
        bad[name][at] = float(value)
        Z, W1 = _run(bad)
        heads = slice(None) if name in ("Q", "K") else slice(0, 1)          # one key head, two value heads
        features = slice(5, 6) if name == "V" else slice(None)
        assert torch.equal(Z[0], clean_Z[0]) and torch.equal(W1[0], clean_W1[0])
        assert torch.equal(Z[1, :, :t], clean_Z[1, :, :t])
        hit = Z[1, heads, t:, features]
        if name == "Q":
            assert not torch.isfinite(hit[:, 0]).any() and torch.equal(Z[1, :, t + 1:], clean_Z[1, :, t + 1:])
            assert torch.equal(W1, clean_W1)
            continue
        assert not torch.isfinite(hit).any() and not torch.isfinite(W1[1, heads, features]).any()
        if heads != slice(None):
            assert torch.equal(Z[1, 1], clean_Z[1, 1]) and torch.equal(W1[1, 1], clean_W1[1, 1])
        if name == "V":
            rest = [i for i in range(d) if i != 5]
            assert torch.equal(Z[1, 0][:, rest], clean_Z[1, 0][:, rest]) and torch.equal(W1[1, 0, rest], clean_W1[1, 0, rest])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padding_without_lengths(cuda_dev, dtype):
    """A padded batch given without its lengths, NaN in the padding: the real rows are those of the call with them."""
    lengths = [70, 1, 33, 64, 0, 47]
    y = _on(_make(6, 2, 2, N, 64, 128, dtype, w0="each", seed=41), cuda_dev)
    for n in INPUTS:
        for b, m in enumerate(lengths):
            y[n][b, :, m:] = float("nan")
    Z, _ = _run(y)
    want = forward_gated_delta(*(y[n] for n in INPUTS), W0=y["W0"], lengths=torch.tensor(lengths, dtype=torch.int32, device=cuda_dev))
    for b, m in enumerate(lengths):
        assert torch.isfinite(want[b, :, :m]).all()
        assert torch.equal(Z[b, :, :m], want[b, :, :m])
        assert torch.isnan(Z[b, :, m:]).all()
