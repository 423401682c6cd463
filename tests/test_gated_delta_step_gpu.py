"""The one-step recurrence on batches large enough for four state rows per thread (from 512 state rows per SM on): slots in any order,
unused and shared ones, both tokens' types.  Tolerances as for small batches (fp32 arithmetic, one rounding of bf16 outputs)."""
import pytest
import torch

import oracle
from tests.parity import rel_max_err
from tests.test_gated_delta_gpu import INPUTS, STEP_STATES, STEP_TOKENS, _make, _on
from vision_test_token_b200 import step_gated_delta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv,n", [(128, 128, 1), (64, 128, 3), (128, 64, 2)])
@pytest.mark.parametrize("shared", [False, True])
def test_large_batches(cuda_dev, dtype, dk, dv, n, shared):
    hk, h = 4, 8
    sms = torch.cuda.get_device_properties(cuda_dev).multi_processor_count
    B = 512 * sms // (h * dv) + 5
    x = _make(B, hk, h, n, dk, dv, dtype, "tokens", "none", seed=70)
    y = _on(x, cuda_dev)
    g = torch.Generator().manual_seed(71)
    slots = torch.randperm(B + 7, generator=g)[:B].to(torch.int32)
    slots[3] = slots[B - 2] = -1
    if shared:                                                    # rows 10 and 40 before and after one another's CTAs
        slots[40] = slots[10]
        slots[B - 1] = slots[10]
        slots[20] = slots[0]
    W = torch.randn((B + 7, h, dv, dk), generator=g) / dk ** 0.5
    got = W.to(cuda_dev)
    Z = torch.full_like(y["V"], 9.0)
    step_gated_delta(*(y[k] for k in INPUTS), got, slots=slots.to(cuda_dev), scale=0.5, Z=Z)
    torch.cuda.synchronize()
    want, wantZ = W.double(), torch.full(x["V"].shape, 9.0, dtype=torch.float64)
    rows = {}
    for b, s in enumerate(slots.tolist()):
        if s >= 0:
            rows.setdefault(s, []).append(b)
    for length in sorted({len(r) for r in rows.values()}):        # states that as many rows name, as one batch of longer sequences
        some = [(s, r) for s, r in rows.items() if len(r) == length]
        pick = torch.tensor([r for _, r in some])
        seq = [x[k][pick.flatten()].unflatten(0, pick.shape).transpose(1, 2).flatten(2, 3) for k in INPUTS]
        at = torch.tensor([s for s, _ in some])
        Zr, W1r = oracle.gated_delta(*seq, W[at], scale=0.5)
        want[at] = torch.from_numpy(W1r)
        wantZ[pick.flatten()] = torch.from_numpy(Zr).unflatten(2, (length, n)).transpose(1, 2).flatten(0, 1)
    assert rel_max_err(got, want.numpy()) <= STEP_STATES
    used = slots >= 0
    assert rel_max_err(Z[used.to(cuda_dev)], wantZ[used].numpy()) <= STEP_TOKENS[dtype]
    assert (Z[(~used).to(cuda_dev)] == 9.0).all()
    idle = torch.tensor([s for s in range(B + 7) if s not in rows])
    assert torch.equal(got[idle.to(cuda_dev)].cpu(), W[idle])
