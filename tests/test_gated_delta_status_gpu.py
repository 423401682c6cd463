"""A device-side wait that ran out in a gated delta call is seen through the workspace that the caller passed."""
import pytest
import torch

from tests.test_gated_delta_gpu import INPUTS, _make, _on
from vision_test_token_b200 import (backward_gated_delta, capi, forward_gated_delta, gated_delta_workspace,
                                    workspace_status)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("backward", [False, True])
def test_status_of_a_passed_workspace(cuda_dev, backward):
    y = _on(_make(2, 1, 2, 100, 64, 128, w0="shared", seed=50), cuda_dev)
    args = [y[n] for n in INPUTS]
    ws = gated_delta_workspace(y["Q"], y["V"], backward=backward)
    shape = capi.make_delta_shape(2, 1, 2, 100, 64, 128, capi.TTT_BF16)
    assert ws.numel() == capi.ttt_gated_delta_workspace_bytes(int(backward), shape)

    def call(**kw):
        if backward:
            return backward_gated_delta(*args, y["dZ"], W0=y["W0"], **kw)
        return [forward_gated_delta(*args, W0=y["W0"], **kw)]

    word = ws[:4].view(torch.int32)
    word.fill_(1)                                                 # as a call that gave up leaves it
    assert workspace_status(ws) == capi.TTT_ERR_TIMEOUT
    assert workspace_status(ws) == capi.TTT_OK                    # told once
    word.fill_(1)
    got = call(ws=ws)                                             # the status is the last call's
    assert workspace_status(ws) == capi.TTT_OK
    for a, b in zip(got, call()):
        assert torch.equal(a, b)


def test_workspace_refusals(cuda_dev):
    y = _on(_make(1, 1, 1, 10, 64, 64, seed=51), cuda_dev)
    with pytest.raises(ValueError):
        gated_delta_workspace(y["Q"][..., :32], y["V"])
    with pytest.raises(ValueError):
        gated_delta_workspace(y["Q"].cpu(), y["V"].cpu())
    ws = gated_delta_workspace(y["Q"], y["V"])
    with pytest.raises(RuntimeError, match="WORKSPACE"):          # a forward call's is too small for the backward pass
        backward_gated_delta(*(y[n] for n in INPUTS), y["dZ"], ws=ws)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("backward", [False, True])
def test_empty_sequences_leave_the_workspace_alone(cuda_dev, dtype, backward):
    """Nothing behind a sequence's end is read: a batch of empty sequences makes nothing of its tokens in the workspace."""
    y = _on(_make(2, 1, 2, 100, 64, 64, dtype, w0="none", seed=52), cuda_dev)
    args = [y[n] for n in INPUTS]
    ws = gated_delta_workspace(y["Q"], y["V"], backward=backward)
    ws.fill_(0xA5)
    lengths = torch.tensor([0, -3], dtype=torch.int32, device=cuda_dev)
    if backward:
        backward_gated_delta(*args, y["dZ"], lengths=lengths, ws=ws)
    else:
        forward_gated_delta(*args, lengths=lengths, ws=ws)
    torch.cuda.synchronize()
    assert (ws[256:] == 0xA5).all()                               # the header holds the status
