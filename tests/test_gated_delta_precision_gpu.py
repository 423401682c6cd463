"""Results of the gated delta rule are as good as fp32 computations: W1, dG, dBeta and dW0 of either tokens' type, and
all outputs of fp32 tokens, against the fp64 oracle; bf16 outputs are the fp64 values rounded once, but for few near a tie.

Tolerance, as a 2-norm of the error over that of the result: operands are three bf16 parts, 2^-24 of the value each (6e-8).
A matrix instruction cuts each of its 16 products at a quarter of the last place of the largest addend, an eighth on average,
and the sum towards zero: (16 / 8 + 1 / 2) 2^-24 = 1.5e-7 of the sum at the worst sign pattern.  The longest sum is d / 16 = 8 instructions,
whose partial sums are half of the result on average: sqrt(8) 1.5e-7 / 2 = 2.1e-7 for products of random signs.  Results pass through at
most six such products (A or K W^T, R, E, the state, two of the gradients'): sqrt(6) 2.1e-7 = 5.2e-7, and up to twice that
where a gradient is the difference of larger terms: 1e-6.
bf16 outputs: an error of e times the root mean square moves a value x over a tie with the probability 2 e rms / step, the step
being 2^-8 |x| at least; for a normal distribution down to 1e-3 of it, the mean of rms / |x| is about 6: with e = 2e-7 (all but the
worst of the above) 2 * 2e-7 * 2^8 * 6 = 6e-4 of the values: 1e-3.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gated_delta_gpu import INPUTS, _lengths, _make, _on
from vision_test_token_b200 import backward_gated_delta, forward_gated_delta

pytestmark = pytest.mark.gpu

TOL = 1e-6
MOVED = 1e-3


def _rel(got, ref):
    g, r = got.double().cpu().numpy(), np.asarray(ref, np.float64)
    assert g.shape == r.shape
    return float(np.linalg.norm(g - r) / np.linalg.norm(r))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hk,h,N,dk,dv,gate,w0", [
    (1, 2, 300, 64, 64, 0.1, "shared"),
    (2, 2, 517, 128, 128, 0.1, "each"),
    (1, 2, 300, 128, 64, 0.0, "each"),          # no gate: a state that remembers all tokens
    (1, 2, 300, 64, 128, 3.0, "shared"),        # strong gates: a state of a few tokens
    (20, 20, 200, 128, 128, 0.02, "shared"),    # two tiles of state rows per CTA
])
def test_fp32_results(cuda_dev, dtype, hk, h, N, dk, dv, gate, w0):
    x = _make(2, hk, h, N, dk, dv, dtype, "tokens", w0, seed=N, gate=gate)
    lengths = [N, N - 41]
    y, lens, scale = _on(x, cuda_dev), _lengths(lengths, cuda_dev), dk ** -0.5
    args = [y[n] for n in INPUTS]
    W1 = torch.empty((2, h, dv, dk), device=cuda_dev)
    Z = forward_gated_delta(*args, W0=y["W0"], lengths=lens, scale=scale, W1_out=W1)
    grads = backward_gated_delta(*args, y["dZ"], W0=y["W0"], dW1=y["dW1"], lengths=lens, scale=scale)
    cpu = [x[n] for n in INPUTS]
    want = oracle.gated_delta(*cpu, x["W0"], lengths, scale)
    want += oracle.gated_delta_backward(*cpu, x["dZ"], x["W0"], x["dW1"], lengths, scale)
    for name, a, b in zip(("Z", "W1", "dQ", "dK", "dV", "dG", "dBeta", "dW0"), (Z, W1) + tuple(grads), want):
        if a.dtype == torch.float32:
            assert _rel(a, b) <= TOL, name
        else:
            once = torch.from_numpy(np.asarray(b)).to(torch.bfloat16)
            assert float((a.cpu() != once).double().mean()) <= MOVED, name
