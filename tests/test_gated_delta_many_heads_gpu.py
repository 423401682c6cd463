"""The gated delta rule where a call has many heads of d_v = 128 in bf16 (the state in tensor memory, chunks of 64 tokens),
against the fp64 oracle; and token tensors whose tokens are one row broadcast, which no tensor map describes.

Tolerances as for few heads: the same operands are carried as two bf16 parts, the chunks are twice as long and half
as many, and the inverse of a chunk's triangular system is joined from blocks with the same parts.
"""
import pytest
import torch

import oracle
from tests.parity import rel_max_err
from tests.test_gated_delta_gpu import INPUTS, STATES, TOKENS, _check_backward, _check_forward, _lengths, _make, _on
from vision_test_token_b200 import backward_gated_delta, forward_gated_delta, step_gated_delta

pytestmark = pytest.mark.gpu

HEADS = {128: (20, 1, 2), 64: (40, 1, 2)}      # (B, key heads, heads): more than 32 x 128 values of state per SM


@pytest.mark.parametrize("N", [1, 63, 64, 65, 128, 200, 321])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_lengths_of_chunks(cuda_dev, N, dk, layout):
    B, hk, h = HEADS[dk]
    x = _make(B, hk, h, N, dk, 128, "bf16", layout, ("none", "shared", "each")[N % 3], seed=N + dk)
    _check_forward(x, cuda_dev, "bf16", scale=dk ** -0.5)
    _check_backward(x, cuda_dev, "bf16", scale=dk ** -0.5, last=N % 2 == 0)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_padded_batch(cuda_dev, dk, layout):
    """NaN behind each sequence's end: not read, and the rows there are left as they were."""
    B, hk, h = HEADS[dk]
    N = 150
    lengths = [(150, 0, 1, 63, 64, 65, 97, 128, 129, 149)[b % 10] for b in range(B)]
    x = _make(B, hk, h, N, dk, 128, "bf16", layout, "each", seed=3)
    for n in INPUTS + ("dZ",):
        for b, m in enumerate(lengths):
            x[n][b, :, m:] = float("nan")
    _check_forward(x, cuda_dev, "bf16", lengths)
    _check_backward(x, cuda_dev, "bf16", lengths)
    y, lens = _on(x, cuda_dev), _lengths(lengths, cuda_dev)
    Z = torch.full_like(y["V"], 7.0)
    forward_gated_delta(*(y[n] for n in INPUTS), W0=y["W0"], lengths=lens, Z=Z)
    out = [torch.full_like(y[n], 7.0) for n in INPUTS] + [torch.full_like(y["W0"], 7.0)]
    backward_gated_delta(*(y[n] for n in INPUTS), y["dZ"], W0=y["W0"], lengths=lens, out=out)
    torch.cuda.synchronize()
    for t in [Z] + out[:5]:
        for b, m in enumerate(lengths):
            assert (t[b, :, m:] == 7.0).all()
            assert torch.isfinite(t[b, :, :m]).all()
    assert not torch.isnan(out[5]).any() and not out[5][1].any()


def test_no_tokens_at_all(cuda_dev):
    x = _make(20, 1, 2, 70, 128, 128, w0="each", seed=4)
    y = _on(x, cuda_dev)
    W1 = torch.empty_like(y["W0"])
    Z = torch.full_like(y["V"], 7.0)
    forward_gated_delta(*(y[n] for n in INPUTS), W0=y["W0"], lengths=_lengths([0] * 20, cuda_dev), Z=Z, W1_out=W1)
    got = backward_gated_delta(*(y[n] for n in INPUTS), y["dZ"], W0=y["W0"], dW1=y["dW1"], lengths=_lengths([-3] * 20, cuda_dev))
    torch.cuda.synchronize()
    assert (Z == 7.0).all() and torch.equal(W1, y["W0"]) and torch.equal(got[5], y["dW1"])
    assert not any(t.any() for t in got[:5])


def test_hard_gates_and_repeated_keys(cuda_dev):
    x = _make(40, 1, 1, 200, 128, 128, w0="shared", seed=5)
    g = x["G"]
    g[:, :, :40] = 0.0
    g[:, :, 40:80] = -20.0
    g[::2, :, 80] = g[::2, :, 81] = g[::2, :, 127] = g[1::2, :, 128] = -float("inf")
    g[:, :, 129:150] = -1e4
    g[:, :, 150:] = -1e-6
    _check_forward(x, cuda_dev, "bf16")
    _check_backward(x, cuda_dev, "bf16")
    x = _make(40, 1, 1, 130, 128, 128, w0="shared", seed=6, gate=1e-3)
    x["K"][:] = x["K"][:, :, :1]
    x["Beta"][:] = 1.0
    x["Beta"][:, :, ::3] = 0.0
    _check_forward(x, cuda_dev, "bf16")
    _check_backward(x, cuda_dev, "bf16")


def test_strided_outputs_and_a_shared_batch(cuda_dev):
    """Keys and queries that all images share, outputs cut from wider buffers: nothing outside them is written."""
    B, N, h, d = 20, 100, 2, 128
    x = _make(B, h, h, N, d, d, layout="tokens", w0="none", seed=8)
    y = _on(x, cuda_dev)
    for n in ("Q", "K"):
        x[n] = x[n][:1].expand(B, h, N, d)
        y[n] = y[n][:1].expand(B, h, N, d)
    cut = lambda t: t[:, 1:1 + N, 1:1 + h].transpose(1, 2)  # noqa: E731
    wide = lambda: torch.full((B, N + 2, h + 2, d), 3.0, dtype=torch.bfloat16, device=cuda_dev)  # noqa: E731
    Z, out = wide(), [wide() for _ in range(3)]
    forward_gated_delta(*(y[n] for n in INPUTS), Z=cut(Z))
    dG, dBeta = torch.empty((2, B, h, N), device=cuda_dev)
    backward_gated_delta(*(y[n] for n in INPUTS), y["dZ"], out=[cut(t) for t in out] + [dG, dBeta, None])
    torch.cuda.synchronize()
    want = [oracle.gated_delta(*(x[n] for n in INPUTS))[0]] + list(oracle.gated_delta_backward(*(x[n] for n in INPUTS), x["dZ"]))
    for t, ref in zip([Z] + out, want):
        assert rel_max_err(cut(t), ref) <= TOKENS["bf16"]
        cut(t).fill_(3.0)
        assert (t == 3.0).all()
    assert rel_max_err(dG, want[4]) <= STATES["bf16"] and rel_max_err(dBeta, want[5]) <= STATES["bf16"]


@pytest.mark.parametrize("B", [1, 40])
@pytest.mark.parametrize("names", [("K",), ("Q", "V"), ("Q", "K", "V", "dZ")])
def test_one_row_for_all_tokens(cuda_dev, B, names):
    """A token stride of zero."""
    N = 100
    x = _make(B, 1, 1, N, 128, 128, w0="shared", seed=9)
    y = _on(x, cuda_dev)
    for n in names:
        x[n] = x[n][:, :, :1].expand(-1, -1, N, -1)
        y[n] = y[n][:, :, :1].expand(-1, -1, N, -1)
    Z = torch.empty((B, 1, N, 128), dtype=torch.bfloat16, device=cuda_dev)
    forward_gated_delta(*(y[n] for n in INPUTS), W0=y["W0"], Z=Z)
    out = [torch.empty(x[n].shape, dtype=x[n].dtype, device=cuda_dev) for n in INPUTS] + [torch.empty_like(y["W0"])]
    backward_gated_delta(*(y[n] for n in INPUTS), y["dZ"], W0=y["W0"], dW1=y["dW1"], out=out)
    torch.cuda.synchronize()
    assert rel_max_err(Z, oracle.gated_delta(*(x[n] for n in INPUTS), x["W0"])[0]) <= TOKENS["bf16"]
    want = oracle.gated_delta_backward(*(x[n] for n in INPUTS), x["dZ"], x["W0"], x["dW1"])
    for name, a, b in zip(("dQ", "dK", "dV", "dG", "dBeta", "dW0"), out, want):
        assert rel_max_err(a, b) <= (TOKENS if name in ("dQ", "dK", "dV") else STATES)["bf16"], name


def test_same_bits_in_graphs_and_on_streams(cuda_dev):
    xs = [_make(20, 1, 2, 130 + 60 * i, 128, 128, layout="tokens", seed=20 + i) for i in range(2)]
    ys = [_on(x, cuda_dev) for x in xs]
    call = lambda y: [forward_gated_delta(*(y[k] for k in INPUTS), W0=y["W0"])] + list(  # noqa: E731
        backward_gated_delta(*(y[k] for k in INPUTS), y["dZ"], W0=y["W0"]))
    want = [[t.clone() for t in call(y)] for y in ys]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call(ys[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            eager = call(ys[1])
        torch.cuda.synchronize()
        for got, ref in zip((captured, eager), want):
            for a, b in zip(got, ref):
                assert torch.equal(a, b)


def test_lengths_inside_an_output_are_refused(cuda_dev):
    y = _on(_make(2, 1, 1, 40, 64, 64, seed=30), cuda_dev)
    Z = torch.empty((2, 1, 40, 64), dtype=torch.bfloat16, device=cuda_dev)
    lengths = Z.view(torch.int32).flatten()[:2]
    lengths.fill_(40)
    args = [y[n] for n in INPUTS]
    with pytest.raises(RuntimeError, match="INVALID"):
        forward_gated_delta(*args, lengths=lengths, Z=Z)
    W = torch.zeros((2, 1, 64, 64), device=cuda_dev)
    with pytest.raises(RuntimeError, match="INVALID"):
        step_gated_delta(*args, W=W, slots=W.view(torch.int32).flatten()[:2])


@pytest.mark.parametrize("h", [2, 20])
def test_images_far_apart(cuda_dev, h):
    """Images more than 2^31 elements apart in one buffer: the same bits as side by side."""
    B, N, d = 2, 70, 128
    y = _on(_make(B, h, h, N, d, d, layout="tokens", w0="shared", seed=11), cuda_dev)
    far = 2 ** 31 + 2 ** 10
    buf = torch.zeros(far + 8 * N * h * d, dtype=torch.bfloat16, device=cuda_dev)
    cut = lambda i: torch.as_strided(buf, (B, h, N, d), (far, d, 8 * h * d, 1), i * h * d)  # noqa: E731
    z = dict(y)
    for i, n in enumerate(("Q", "K", "V", "dZ")):
        z[n] = cut(i)
        z[n].copy_(y[n])
    Z = forward_gated_delta(*(y[n] for n in INPUTS), W0=y["W0"])
    forward_gated_delta(*(z[n] for n in INPUTS), W0=y["W0"], Z=cut(4))
    assert torch.equal(cut(4), Z)
    want = backward_gated_delta(*(y[n] for n in INPUTS), y["dZ"], W0=y["W0"], dW1=y["dW1"])
    got = [cut(5), cut(6), cut(7)] + [torch.empty_like(t) for t in want[3:]]
    backward_gated_delta(*(z[n] for n in INPUTS), z["dZ"], W0=y["W0"], dW1=y["dW1"], out=got)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
