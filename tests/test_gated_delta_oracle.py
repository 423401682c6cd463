"""Pins of the fp64 oracle of the gated delta rule (CPU): special cases that another pinned function gives,
torch double-precision autograd, central differences, and invariants."""
import numpy as np
import pytest
import torch

import oracle


def _inputs(B, hk, h, N, dk, dv, seed, shared=True):
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    return dict(Q=unit(r.standard_normal((B, hk, N, dk))), K=unit(r.standard_normal((B, hk, N, dk))),
                V=r.standard_normal((B, h, N, dv)), G=-r.exponential(0.2, (B, h, N)),
                Beta=r.uniform(0.0, 1.0, (B, h, N)),
                W0=r.standard_normal((h, dv, dk) if shared else (B, h, dv, dk)) / np.sqrt(dk))


def test_without_a_gate_it_is_minibatch_training_with_one_token():
    """g = 0 and beta = 2 eta: the pinned mini-batch oracle with batches of one token."""
    x = _inputs(2, 3, 3, 17, 8, 8, 0)
    eta = 0.3
    Z, W1 = oracle.gated_delta(x["Q"], x["K"], x["V"], np.zeros((2, 3, 17)), np.full((2, 3, 17), 2 * eta), x["W0"])
    Zr, W1r = oracle.linear_minibatch(x["Q"], x["K"], x["V"], x["W0"], eta, 1, "prefix")
    np.testing.assert_allclose(Z, Zr, rtol=0, atol=1e-12)
    np.testing.assert_allclose(W1, W1r, rtol=0, atol=1e-12)


def test_beta_zero_only_fades_and_scale_scales():
    x = _inputs(1, 1, 2, 6, 4, 5, 1)
    Z, W1 = oracle.gated_delta(x["Q"], x["K"], x["V"], x["G"], 0 * x["Beta"], x["W0"], scale=0.25)
    fade = np.exp(np.cumsum(x["G"], axis=-1))
    np.testing.assert_allclose(W1, fade[..., -1, None, None] * x["W0"], atol=1e-14)
    np.testing.assert_allclose(Z, 0.25 * fade[..., None] * np.einsum("hvk,bhnk->bhnv", x["W0"], np.repeat(x["Q"], 2, 1)),
                               atol=1e-14)


def test_a_gate_of_minus_infinity_starts_afresh():
    x = _inputs(1, 2, 2, 9, 4, 4, 2)
    x["G"][:, :, 4] = -np.inf
    Z, W1 = oracle.gated_delta(**x)
    y = {k: (v[:, :, 4:] if k != "W0" else None) for k, v in x.items()}
    y["G"] = y["G"].copy()
    y["G"][:, :, 0] = 0.0
    Zr, W1r = oracle.gated_delta(**y)
    np.testing.assert_allclose(Z[:, :, 4:], Zr, atol=1e-14)
    np.testing.assert_allclose(W1, W1r, atol=1e-14)


def test_a_key_stored_with_beta_one_is_read_back():
    """beta = 1 and a unit key: the weights map the last key to its value exactly."""
    x = _inputs(2, 1, 1, 7, 6, 3, 3)
    x["Beta"][:] = 1.0
    x["Q"][:, :, -1] = x["K"][:, :, -1]
    Z, _ = oracle.gated_delta(**x)
    np.testing.assert_allclose(Z[:, :, -1], x["V"][:, :, -1], atol=1e-12)


def test_lengths_cut_the_sequence():
    x = _inputs(3, 1, 2, 8, 4, 4, 4, shared=False)
    for k in ("Q", "K", "V", "G", "Beta"):
        x[k][1, :, 5:] = np.nan
        x[k][2] = np.nan
    Z, W1 = oracle.gated_delta(lengths=[8, 5, 0], **x)
    Zr, W1r = oracle.gated_delta(**{k: (v[1:2] if k == "W0" else v[1:2, :, :5]) for k, v in x.items()})
    np.testing.assert_array_equal(Z[1:2, :, :5], Zr)
    np.testing.assert_array_equal(W1[1:2], W1r)
    np.testing.assert_array_equal(W1[2], x["W0"][2])
    assert not Z[1, :, 5:].any() and not Z[2].any()


def _torch_forward(Q, K, V, G, Beta, W0, scale):
    r = V.shape[1] // Q.shape[1]
    Q, K = Q.repeat_interleave(r, 1), K.repeat_interleave(r, 1)
    W, Z = W0.expand(V.shape[0], *W0.shape[-3:]), []
    for t in range(V.shape[2]):
        W = W * G[:, :, t].exp()[..., None, None]
        e = V[:, :, t] - (W @ K[:, :, t, :, None])[..., 0]
        W = W + (Beta[:, :, t, None] * e)[..., None] * K[:, :, t, None, :]
        Z.append(scale * (W @ Q[:, :, t, :, None])[..., 0])
    return torch.stack(Z, 2), W


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("last", [True, False])
def test_gradients_agree_with_autograd(shared, last):
    B, hk, h, N, dk, dv = 2, 2, 4, 6, 3, 5
    x = _inputs(B, hk, h, N, dk, dv, 5, shared)
    r = np.random.default_rng(6)
    dZ, dW1 = r.standard_normal((B, h, N, dv)), r.standard_normal((B, h, dv, dk)) if last else None
    names = ["Q", "K", "V", "G", "Beta", "W0"]
    leaf = {n: torch.tensor(x[n]).requires_grad_() for n in names}
    Z, W = _torch_forward(*(leaf[n] for n in names), 0.7)
    total = (Z * torch.tensor(dZ)).sum() + ((W * torch.tensor(dW1)).sum() if last else 0)
    want = torch.autograd.grad(total, [leaf[n] for n in names])
    got = oracle.gated_delta_backward(x["Q"], x["K"], x["V"], x["G"], x["Beta"], dZ, x["W0"], dW1, scale=0.7)
    for n, a, b in zip(names, got, want):
        np.testing.assert_allclose(a, b.numpy(), atol=1e-12, err_msg=n)


def test_gradients_agree_with_central_differences():
    B, hk, h, N, dk, dv = 2, 1, 2, 5, 3, 2
    x = _inputs(B, hk, h, N, dk, dv, 7)
    lengths = [5, 3]
    r = np.random.default_rng(8)
    dZ, dW1 = r.standard_normal((B, h, N, dv)), r.standard_normal((B, h, dv, dk))

    def total(y):
        Z, W1 = oracle.gated_delta(lengths=lengths, scale=0.5, **y)
        return float((Z * dZ).sum() + (W1 * dW1).sum())

    got = oracle.gated_delta_backward(x["Q"], x["K"], x["V"], x["G"], x["Beta"], dZ, x["W0"], dW1, lengths, 0.5)
    for name, grad in zip(["Q", "K", "V", "G", "Beta", "W0"], got):
        for _ in range(12):
            at = tuple(r.integers(0, n) for n in x[name].shape)
            step = np.zeros_like(x[name])
            step[at] = 1e-5
            diff = (total({**x, name: x[name] + step}) - total({**x, name: x[name] - step})) / 2e-5
            # truncation about 1e-10, rounding of the totals (about 10) about 1e-10
            assert abs(diff - grad[at]) <= 2e-9, (name, at)
