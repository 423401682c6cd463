"""Parity of the gated delta rule (forward, backward and the one-step recurrence, through the C ABI) against the
fp64 oracle.

Tolerances (max|error| / max|reference| of each output).  An output in bf16 is rounded once: half a step, 2^-8 of
the value.  Inside, bf16 tokens are exact operands and everything else is carried as two bf16 parts, 2^-16 of
the value per operand: up to four products in sequence per chunk, three dropped or rounded terms each,
a factor of about two between the sum of a product's terms and its result, and a state that remembers a handful of
chunks, all with random signs: sqrt(4 * 3) * 2 * sqrt(5) * 2^-17 is about 1e-4 at the worst element.
fp32 tokens: three parts (2^-24) and fp32 accumulation, whose error is the framework's fp32 bound, 1e-5.
The recurrence (step) computes in fp32 throughout.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.parity import rel_max_err
from vision_test_token_b200 import backward_gated_delta, clip_gradients, forward_gated_delta, step_gated_delta

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOKENS = {"bf16": 2 ** -8 + 1e-4, "fp32": 1e-5}      # outputs in the tokens' type
STATES = {"bf16": 1e-4, "fp32": 1e-5}                # fp32 outputs
STEP_TOKENS = {"bf16": 2 ** -8 + 1e-6, "fp32": 2e-6}
STEP_STATES = 2e-6


def _make(B, hk, h, N, dk, dv, dtype="bf16", layout="heads", w0="shared", seed=0, gate=0.1):
    """CPU tensors; token tensors are [B][heads][N][d] views of buffers laid out by head or by token."""
    g = torch.Generator().manual_seed(seed)

    def tokens(heads, d, unit):
        shape = (B, N, heads, d) if layout == "tokens" else (B, heads, N, d)
        x = torch.randn(shape, generator=g)
        if unit:
            x = x / x.norm(dim=-1, keepdim=True)
        x = x.to(DT[dtype])
        return x.transpose(1, 2) if layout == "tokens" else x

    x = dict(Q=tokens(hk, dk, True), K=tokens(hk, dk, True), V=tokens(h, dv, False))
    shape = (B, N, h) if layout == "tokens" else (B, h, N)
    x["G"], x["Beta"] = -gate * torch.rand(shape, generator=g).log().neg(), torch.rand(shape, generator=g)
    if layout == "tokens":
        x["G"], x["Beta"] = x["G"].transpose(1, 2), x["Beta"].transpose(1, 2)
    wshape = {"none": None, "shared": (h, dv, dk), "each": (B, h, dv, dk)}[w0]
    x["W0"] = None if wshape is None else torch.randn(wshape, generator=g) / dk ** 0.5
    x["dZ"] = tokens(h, dv, False)
    x["dW1"] = torch.randn((B, h, dv, dk), generator=g)
    return x


def _on(x, dev):
    """The tensors on the device with the strides they have here."""
    return {k: None if v is None else torch.empty_strided(v.shape, v.stride(), dtype=v.dtype, device=dev).copy_(v)
            for k, v in x.items()}


INPUTS = ("Q", "K", "V", "G", "Beta")


def _lengths(lengths, dev):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev)


def _check_forward(x, dev, dtype, lengths=None, scale=1.0):
    y = _on(x, dev)
    B, h, N, dv = x["V"].shape
    W1 = torch.full((B, h, dv, x["Q"].shape[3]), float("nan"), device=dev)
    Z = forward_gated_delta(*(y[n] for n in INPUTS), W0=y["W0"], lengths=_lengths(lengths, dev), scale=scale, W1_out=W1)
    torch.cuda.synchronize()
    Zr, W1r = oracle.gated_delta(*(x[n] for n in INPUTS), x["W0"], lengths, scale)
    assert Z.dtype == x["V"].dtype and Z.shape == x["V"].shape
    assert rel_max_err(Z, Zr) <= TOKENS[dtype]
    assert rel_max_err(W1, W1r) <= STATES[dtype]
    return Z, W1


def _check_backward(x, dev, dtype, lengths=None, scale=1.0, last=True):
    y = _on(x, dev)
    got = backward_gated_delta(*(y[n] for n in INPUTS), y["dZ"], W0=y["W0"], dW1=y["dW1"] if last else None,
                               lengths=_lengths(lengths, dev), scale=scale)
    torch.cuda.synchronize()
    want = oracle.gated_delta_backward(*(x[n] for n in INPUTS), x["dZ"], x["W0"], x["dW1"] if last else None, lengths, scale)
    assert (got[5] is None) == (x["W0"] is None)
    for name, a, b in zip(("dQ", "dK", "dV", "dG", "dBeta", "dW0"), got, want):
        if a is not None:
            tol = TOKENS[dtype] if name in ("dQ", "dK", "dV") else STATES[dtype]
            assert rel_max_err(a, b) <= tol, name
    return got


SHAPES = [
    (1, 1, 1, 1, 64, 64),          # one token
    (2, 1, 1, 2, 128, 128),
    (1, 2, 2, 31, 64, 64),         # one short of a chunk
    (2, 1, 2, 32, 64, 128),        # one chunk, shared keys, d_k != d_v
    (1, 1, 3, 33, 128, 64),        # one past a chunk
    (2, 2, 2, 64, 64, 64),         # one group of the backward pass
    (1, 1, 1, 65, 128, 128),
    (1, 2, 4, 196, 64, 64),
    (2, 3, 3, 257, 128, 128),
    (1, 1, 2, 1000, 128, 128),
    (40, 2, 2, 5, 64, 64),         # many short sequences
    (160, 1, 2, 70, 64, 64),       # more tiles of state rows than warps that run at a time
    (80, 1, 2, 70, 128, 128),
]


@pytest.mark.parametrize("B,hk,h,N,dk,dv", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_forward(cuda_dev, B, hk, h, N, dk, dv, dtype, layout):
    x = _make(B, hk, h, N, dk, dv, dtype, layout, ("none", "shared", "each")[N % 3], seed=N)
    _check_forward(x, cuda_dev, dtype, scale=1.0 if dk == 64 else dk ** -0.5)


@pytest.mark.parametrize("B,hk,h,N,dk,dv", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_backward(cuda_dev, B, hk, h, N, dk, dv, dtype, layout):
    x = _make(B, hk, h, N, dk, dv, dtype, layout, ("none", "shared", "each")[N % 3], seed=N + 1)
    _check_backward(x, cuda_dev, dtype, scale=1.0 if dk == 64 else dk ** -0.5, last=N % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_lengths(cuda_dev, dtype, layout):
    """A padded batch: whole, empty, one-token, chunk-aligned and ragged sequences; what lies behind a sequence's
    end is NaN and is not read, and the rows there are left as they were."""
    B, hk, h, N = 6, 1, 2, 100
    lengths = [100, 0, 1, 64, 97, 33]
    x = _make(B, hk, h, N, 64, 128, dtype, layout, "each", seed=3)
    for n in INPUTS + ("dZ",):
        for b, m in enumerate(lengths):
            x[n][b, :, m:] = float("nan")
    _check_forward(x, cuda_dev, dtype, lengths)
    _check_backward(x, cuda_dev, dtype, lengths)
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
    assert not torch.isnan(out[5]).any() and not (out[5][1]).any()     # no token: no gradient of a readout


def test_lengths_out_of_range_are_clamped(cuda_dev):
    x = _make(2, 1, 1, 40, 64, 64, w0="each", seed=4)
    y = _on(x, cuda_dev)
    W1 = torch.empty((2, 1, 64, 64), device=cuda_dev)
    Z = forward_gated_delta(*(y[n] for n in INPUTS), W0=y["W0"], lengths=_lengths([1000, -5], cuda_dev), W1_out=W1)
    Zr, W1r = oracle.gated_delta(*(x[n] for n in INPUTS), x["W0"], [40, 0])
    assert rel_max_err(Z, Zr) <= TOKENS["bf16"] and rel_max_err(W1, W1r) <= STATES["bf16"]
    assert torch.equal(W1[1].cpu(), x["W0"][1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_hard_gates(cuda_dev, dtype):
    """Gates that drop the state (-inf), that are strong enough to underflow, and none at all."""
    x = _make(1, 1, 1, 200, 64, 64, dtype, w0="shared", seed=5)
    g = x["G"][0, 0]
    g[:40] = 0.0
    g[40:80] = -20.0
    g[80] = g[81] = g[127] = g[128] = -float("inf")
    g[129:150] = -1e4
    g[150:] = -1e-6
    _check_forward(x, cuda_dev, dtype)
    _check_backward(x, cuda_dev, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeated_keys(cuda_dev, dtype):
    """Neighbouring tokens with the same key and step sizes up to one: the chunk's triangular system is far from
    the identity (its inverse is not a short power series)."""
    x = _make(1, 1, 1, 130, 64, 64, dtype, w0="shared", seed=6, gate=1e-3)
    x["K"][:] = x["K"][:, :, :1]
    x["Beta"][:] = 1.0
    _check_forward(x, cuda_dev, dtype)
    x["Beta"][0, 0, ::3] = 0.0
    _check_forward(x, cuda_dev, dtype)
    _check_backward(x, cuda_dev, dtype)


def test_overshooting_steps(cuda_dev):
    """Step sizes between one and two (beta k k^T reflects): still contracting for unit keys."""
    x = _make(1, 2, 2, 150, 64, 64, w0="shared", seed=7)
    x["Beta"].add_(0.9)
    _check_forward(x, cuda_dev, "bf16")
    _check_backward(x, cuda_dev, "bf16")


def test_views_of_one_projection(cuda_dev):
    """Q, K, V cut from the rows of one projection, gradients cut from the rows of another buffer, a broadcast
    gate: no copies, and nothing outside the views is written."""
    B, N, h, d = 2, 70, 2, 64
    x = _make(B, h, h, N, d, d, layout="tokens", w0="none", seed=8)
    buf = torch.zeros((B, N, 3 * h + 1, d), dtype=torch.bfloat16, device=cuda_dev)
    cut = lambda t, i: t[:, :, i * h:(i + 1) * h].transpose(1, 2)  # noqa: E731
    for i, n in enumerate(("Q", "K", "V")):
        cut(buf, i).copy_(x[n])
    x["G"] = x["G"][:, :1, :].expand(B, h, N)
    x["Beta"] = x["Beta"][:1].expand(B, h, N)
    G = x["G"][:, :1].to(cuda_dev).expand(B, h, N)
    Beta = x["Beta"][:1].to(cuda_dev).expand(B, h, N)
    Z = torch.full((B, N, h + 2, d), 3.0, dtype=torch.bfloat16, device=cuda_dev)
    forward_gated_delta(cut(buf, 0), cut(buf, 1), cut(buf, 2), G, Beta, Z=Z[:, :, 1:1 + h].transpose(1, 2))
    Zr, _ = oracle.gated_delta(*(x[n] for n in INPUTS))
    assert rel_max_err(Z[:, :, 1:1 + h].transpose(1, 2), Zr) <= TOKENS["bf16"]
    assert (Z[:, :, 0] == 3.0).all() and (Z[:, :, -1] == 3.0).all()
    dbuf = torch.full_like(buf, 3.0)
    dG, dBeta = torch.empty((2, B, N, h), device=cuda_dev).transpose(2, 3)
    backward_gated_delta(cut(buf, 0), cut(buf, 1), cut(buf, 2), G, Beta, x["dZ"].to(cuda_dev),
                         out=(cut(dbuf, 0), cut(dbuf, 1), cut(dbuf, 2), dG, dBeta, None))
    want = oracle.gated_delta_backward(*(x[n] for n in INPUTS), x["dZ"])
    for a, b in zip((cut(dbuf, 0), cut(dbuf, 1), cut(dbuf, 2)), want):
        assert rel_max_err(a, b) <= TOKENS["bf16"]
    assert rel_max_err(dG, want[3]) <= STATES["bf16"] and rel_max_err(dBeta, want[4]) <= STATES["bf16"]
    assert (dbuf[:, :, -1] == 3.0).all()


def test_gradients_agree_with_differences(cuda_dev):
    """The fp32 gradients against central differences of the fp64 oracle along random directions."""
    x = _make(2, 1, 2, 70, 64, 64, "fp32", w0="shared", seed=9)
    got = dict(zip(INPUTS + ("W0",), _check_backward(x, cuda_dev, "fp32", [70, 41])))
    g = torch.Generator().manual_seed(10)

    def total(y):
        Z, W1 = oracle.gated_delta(*(y[n] for n in INPUTS), y["W0"], [70, 41])
        return float((Z * x["dZ"].double().numpy()).sum() + (W1 * x["dW1"].double().numpy()).sum())

    y = {k: v.double() for k, v in x.items()}
    for name, grad in got.items():
        d = torch.randn(x[name].shape, generator=g, dtype=torch.float64)
        diff = (total({**y, name: y[name] + 1e-6 * d}) - total({**y, name: y[name] - 1e-6 * d})) / 2e-6
        along = grad.double().cpu() * d
        # 1e-5 of the largest element, summed with random signs over all of them
        tol = 1e-5 * float(grad.abs().max()) * along.numel() ** 0.5 * 4 + 1e-5
        assert abs(diff - float(along.sum())) <= tol, name


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,hk,h,n,dk,dv", [(1, 1, 1, 1, 64, 64), (3, 2, 4, 1, 128, 64), (5, 1, 2, 4, 64, 128),
                                            (64, 4, 8, 1, 128, 128), (17, 3, 3, 2, 128, 128)])
def test_step(cuda_dev, B, hk, h, n, dk, dv, dtype):
    x = _make(B, hk, h, n, dk, dv, dtype, "tokens", "each", seed=B)
    y = _on(x, cuda_dev)
    g = torch.Generator().manual_seed(B)
    slots = torch.randperm(B + 3, generator=g)[:B].to(torch.int32)
    W = torch.randn((B + 3, h, dv, dk), generator=g)
    for b in range(B):
        W[slots[b]] = x["W0"][b]
    got = W.to(cuda_dev)
    Z = step_gated_delta(*(y[k] for k in INPUTS), got, slots=slots.to(cuda_dev), scale=0.5)
    Zr, W1r = oracle.gated_delta(*(x[k] for k in INPUTS), x["W0"], scale=0.5)
    want = W.double().numpy()
    want[slots.numpy()] = W1r
    assert rel_max_err(Z, Zr) <= STEP_TOKENS[dtype]
    assert rel_max_err(got, want) <= STEP_STATES
    others = [s for s in range(B + 3) if s not in slots.tolist()]
    assert torch.equal(got[others].cpu(), W[others])
    plain = x["W0"].to(cuda_dev)
    Z2 = step_gated_delta(*(y[k] for k in INPUTS), plain, scale=0.5)      # row b uses state b
    assert torch.equal(Z, Z2) and torch.equal(plain, got[slots.long().to(cuda_dev)])


def test_step_unused_rows(cuda_dev):
    """Rows without a state (slots outside the cache) leave their Z and every state as they were."""
    x = _make(6, 1, 2, 1, 64, 64, w0="each", seed=11)
    y = _on(x, cuda_dev)
    slots = torch.tensor([2, -1, 4, 5, 0, -7], dtype=torch.int32, device=cuda_dev)      # the cache has 4 states
    W = y["W0"][:4].clone()
    Z = torch.full_like(y["V"], 9.0)
    step_gated_delta(*(y[k] for k in INPUTS), W, slots=slots, Z=Z)
    Zr, W1r = oracle.gated_delta(*(x[k][[0, 4]] for k in INPUTS), x["W0"][[2, 0]])
    assert rel_max_err(Z[[0, 4]], Zr) <= STEP_TOKENS["bf16"]
    assert rel_max_err(W[[2, 0]], W1r) <= STEP_STATES
    assert (Z[[1, 2, 3, 5]] == 9.0).all() and torch.equal(W[[1, 3]], y["W0"][[1, 3]])


@pytest.mark.parametrize("B", [5, 300])
def test_step_rows_that_share_a_state(cuda_dev, B):
    """Rows that name the same state take their steps in batch order, as one longer sequence."""
    n = 2
    x = _make(B, 1, 2, n, 64, 64, w0="none", seed=12)
    y = _on(x, cuda_dev)
    slots = [1, 0, 1, -1, 1] + [0] * (B - 5)
    W0 = torch.randn((2, 2, 64, 64), generator=torch.Generator().manual_seed(1)) / 8
    W = W0.to(cuda_dev)
    Z = step_gated_delta(*(y[k] for k in INPUTS), W, slots=torch.tensor(slots, dtype=torch.int32, device=cuda_dev))
    for s in (0, 1):
        rows = [b for b in range(B) if slots[b] == s]
        seq = [x[k][rows].transpose(0, 1).flatten(1, 2)[None] for k in INPUTS]
        Zr, W1r = oracle.gated_delta(*seq, W0[s])
        assert rel_max_err(Z[rows].transpose(0, 1).flatten(1, 2)[None], Zr) <= STEP_TOKENS["bf16"]
        assert rel_max_err(W[s:s + 1], W1r) <= STEP_STATES
    assert not Z[3].any()


def test_step_far_into_a_large_cache(cuda_dev):
    """A state whose elements lie past 2^31 in the cache."""
    x = _make(1, 4, 4, 1, 128, 128, w0="each", seed=13)
    y = _on(x, cuda_dev)
    n = 2 ** 31 // (4 * 128 * 128) + 2
    W = torch.empty((n, 4, 128, 128), device=cuda_dev)
    W[n - 1] = y["W0"][0]
    Z = step_gated_delta(*(y[k] for k in INPUTS), W, slots=torch.tensor([n - 1], dtype=torch.int32, device=cuda_dev))
    Zr, W1r = oracle.gated_delta(*(x[k] for k in INPUTS), x["W0"])
    assert rel_max_err(Z, Zr) <= STEP_TOKENS["bf16"] and rel_max_err(W[n - 1:], W1r) <= STEP_STATES
    del W
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_then_decode(cuda_dev, dtype):
    """Serving: the states of whole prompts go into a cache, then single tokens follow; the readouts are those of
    the whole sequences."""
    B, hk, h, N, tail = 3, 1, 2, 80, 5
    x = _make(B, hk, h, N + tail, 128, 64, dtype, "tokens", "shared", seed=14)
    y = _on(x, cuda_dev)
    cut = lambda a, b: [y[k][:, :, a:b] for k in INPUTS]  # noqa: E731
    cache = torch.zeros((7, h, 64, 128), device=cuda_dev)
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device=cuda_dev)
    W1 = torch.empty((B, h, 64, 128), device=cuda_dev)
    Z = [forward_gated_delta(*cut(0, N), W0=y["W0"], W1_out=W1)]
    cache[slots.long()] = W1
    for t in range(N, N + tail):
        Z.append(step_gated_delta(*cut(t, t + 1), cache, slots=slots))
    Zr, W1r = oracle.gated_delta(*(x[k] for k in INPUTS), x["W0"])
    assert rel_max_err(torch.cat(Z, 2), Zr) <= TOKENS[dtype]
    assert rel_max_err(cache[slots.long()], W1r) <= STATES[dtype]


def test_chunks_of_a_long_prompt(cuda_dev):
    """A prompt given in pieces, each starting from the weights the last one left."""
    x = _make(2, 2, 2, 150, 64, 64, w0="each", seed=15)
    y = _on(x, cuda_dev)
    W, Z = y["W0"], []
    for a, b in ((0, 50), (50, 51), (51, 150)):
        W1 = torch.empty_like(W)
        Z.append(forward_gated_delta(*(y[k][:, :, a:b].contiguous() for k in INPUTS), W0=W, W1_out=W1))
        W = W1
    Zr, W1r = oracle.gated_delta(*(x[k] for k in INPUTS), x["W0"])
    assert rel_max_err(torch.cat(Z, 2), Zr) <= TOKENS["bf16"] and rel_max_err(W, W1r) <= STATES["bf16"]


def test_training_step(cuda_dev):
    """Training: forward, a loss, backward, clipping by the global norm; a small step along the clipped gradients
    lowers the loss by what they say."""
    x = _make(2, 1, 2, 90, 64, 64, "fp32", w0="shared", seed=16)
    y = _on(x, cuda_dev)
    target = torch.randn(x["V"].shape, generator=torch.Generator().manual_seed(17)).to(cuda_dev)
    Z = forward_gated_delta(*(y[k] for k in INPUTS), W0=y["W0"])
    grads = list(backward_gated_delta(*(y[k] for k in INPUTS), (Z - target) / Z.numel(), W0=y["W0"]))
    whole = [g.clone() for g in grads]
    norm = clip_gradients(grads, 1e-3)
    want = torch.stack([g.double().square().sum() for g in whole]).sum().sqrt()
    assert abs(float(norm) / float(want) - 1) <= 1e-6
    assert float(want) > 1e-3
    for g, w in zip(grads, whole):
        assert rel_max_err(g, (w.double() * 1e-3 / want).cpu().numpy()) <= 1e-6
    loss = lambda Zr: 0.5 * float(((Zr - target.double().cpu().numpy()) ** 2).mean())  # noqa: E731
    names = INPUTS + ("W0",)
    before = loss(oracle.gated_delta(*(x[k] for k in names))[0])
    lr = 1e-2
    moved = [x[k].double() - lr * g.double().cpu() for k, g in zip(names, grads)]
    after = loss(oracle.gated_delta(*moved)[0])
    said = lr * sum(float((g.double() * w.double()).sum()) for g, w in zip(grads, whole))
    assert abs((before - after) / said - 1) <= 1e-2        # curvature over a step of length 1e-5


def test_same_bits_twice(cuda_dev):
    x = _make(3, 2, 4, 300, 128, 128, layout="tokens", seed=18)
    y = _on(x, cuda_dev)
    run = lambda: [forward_gated_delta(*(y[k] for k in INPUTS), W0=y["W0"])] + list(  # noqa: E731
        backward_gated_delta(*(y[k] for k in INPUTS), y["dZ"], W0=y["W0"], dW1=y["dW1"]))
    for a, b in zip(run(), run()):
        assert torch.equal(a, b)


def test_graphs_and_streams(cuda_dev):
    """Two captured graphs and an eager call on a third stream, replayed against one another: no shared scratch."""
    xs = [_make(2, 1, 2, 120 + 40 * i, 64, 64, layout="tokens", seed=20 + i) for i in range(3)]
    ys = [_on(x, cuda_dev) for x in xs]
    outs, graphs = [], []
    call = lambda y, Z, W1: [forward_gated_delta(*(y[k] for k in INPUTS), W0=y["W0"], Z=Z, W1_out=W1)] + list(  # noqa: E731
        backward_gated_delta(*(y[k] for k in INPUTS), y["dZ"], W0=y["W0"]))
    buf = [(torch.zeros_like(y["V"]), torch.zeros((2, 2, 64, 64), device=cuda_dev)) for y in ys]
    want = [[t.clone() for t in call(y, *b)] for y, b in zip(ys, buf)]
    torch.cuda.synchronize()
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(ys[i], *buf[i]))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            eager = call(ys[2], *buf[2])
        torch.cuda.synchronize()
        for got, ref in zip(outs + [eager], want):
            for a, b in zip(got, ref):
                assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Z = forward_gated_delta(*(ys[0][k] for k in INPUTS), W0=ys[0]["W0"], stream=side)
    side.synchronize()
    assert torch.equal(Z, want[0][0])


def test_refusals(cuda_dev):
    x = _on(_make(2, 1, 2, 40, 64, 64, seed=30), cuda_dev)
    args = [x[k] for k in INPUTS]
    swap = lambda i, t: args[:i] + [t] + args[i + 1:]  # noqa: E731
    for bad in (swap(0, x["Q"][:, :, :39]), swap(1, x["K"].float()), swap(2, x["V"][:, :1].expand(2, 3, 40, 64)[:, :, :, :32]),
                swap(3, x["G"].bfloat16()), swap(4, x["Beta"][:, :1]), swap(0, x["Q"].cpu()), swap(0, x["Q"][0]),
                swap(2, x["V"].transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            forward_gated_delta(*bad)
    for kw in (dict(W0=x["W0"].bfloat16()), dict(W0=x["W0"][:1]), dict(lengths=torch.ones(2, device=cuda_dev)),
               dict(lengths=torch.ones(3, dtype=torch.int32, device=cuda_dev)), dict(Z=x["V"].float()),
               dict(W1_out=x["W0"])):
        with pytest.raises(ValueError):
            forward_gated_delta(*args, **kw)
    three = [x["Q"][:, :1].expand(2, 3, 40, 64)] + args[1:]
    with pytest.raises(ValueError):
        forward_gated_delta(*three)                                 # 2 value heads, 3 key heads
    wide = [torch.zeros((1, 1, 4, 96), dtype=torch.bfloat16, device=cuda_dev)] * 2 + [args[2][:1, :1, :4], args[3][:1, :1, :4],
                                                                                       args[4][:1, :1, :4]]
    for fn, what in ((lambda: forward_gated_delta(*wide), "UNSUPPORTED"),
                     (lambda: forward_gated_delta(*args, scale=float("nan")), "INVALID"),
                     (lambda: forward_gated_delta(*args, Z=x["V"]), "INVALID"),              # over an input
                     (lambda: forward_gated_delta(*args, Z=x["V"][:1].expand(2, 2, 40, 64)), "INVALID"),
                     (lambda: forward_gated_delta(*args, ws=torch.empty(256, dtype=torch.uint8, device=cuda_dev)), "WORKSPACE"),
                     (lambda: step_gated_delta(*args, W=x["W0"][None]), "INVALID")):         # fewer states than rows
        with pytest.raises(RuntimeError, match=what):
            fn()
    odd = torch.zeros((2, 1, 40, 72), dtype=torch.bfloat16, device=cuda_dev)
    with pytest.raises(RuntimeError, match="ALIGNMENT"):
        forward_gated_delta(odd[..., 4:68], *args[1:])
    with pytest.raises(ValueError):
        backward_gated_delta(*args, x["dZ"][:, :1])
    with pytest.raises(ValueError):
        backward_gated_delta(*args, x["dZ"], out=(None,) * 5 + (x["W0"],))
    with pytest.raises(ValueError):
        step_gated_delta(*args, W=x["W0"])
    torch.cuda.synchronize()
