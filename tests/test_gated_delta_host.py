"""Host-side checks of the gated delta and clipping entry points (no GPU needed): workspace sizes, and
requests that are refused before anything touches the GPU."""
import ctypes

import pytest

from vision_test_token_b200 import build, capi

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (capi.TTT_ERR_INVALID_ARG, capi.TTT_ERR_UNSUPPORTED, capi.TTT_ERR_ALIGNMENT,
                                              capi.TTT_ERR_WORKSPACE)
BASE = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return capi.lib()


def _shape(**kw):
    base = dict(batch=2, qk_heads=2, heads=4, tokens=50, d_k=64, d_v=128, dtype=capi.TTT_BF16)
    base.update(kw)
    return capi.make_delta_shape(**base)


class Call:
    """A forward call on made-up addresses, 1 GiB apart: every check up to the pointers' own passes."""

    def __init__(self, **shape):
        self.shape = s = _shape(**shape)
        self.views = {}
        for i, (name, heads, width) in enumerate((("Q", s.qk_heads, s.d_k), ("K", s.qk_heads, s.d_k), ("V", s.heads, s.d_v),
                                                  ("G", s.heads, 1), ("Beta", s.heads, 1), ("Z", s.heads, s.d_v))):
            self.views[name] = capi.TttView(BASE + (i << 30), heads * s.tokens * width, s.tokens * width, width)
        self.W0, self.shared, self.lengths, self.scale = None, 0, None, 1.0
        self.W1 = None
        self.ws, self.ws_bytes = BASE + (10 << 30), 1 << 30

    def run(self):
        v = self.views
        return capi.ttt_forward_gated_delta(v["Q"], v["K"], v["V"], v["G"], v["Beta"], self.W0, self.shared, self.lengths,
                                            self.scale, v["Z"], self.W1, self.shape, self.ws, self.ws_bytes, None)


def test_workspace_sizes():
    # forward, bf16: at least the gates and two 32 x 32 matrices of two bf16 parts per image, head and 32 tokens
    assert capi.ttt_gated_delta_workspace_bytes(0, _shape()) > 2 * 4 * 2 * (384 + 2 * 2 * 32 * 32 * 2)
    # it follows the batch, and not the strides
    assert capi.ttt_gated_delta_workspace_bytes(0, _shape(batch=200)) > 90 * capi.ttt_gated_delta_workspace_bytes(0, _shape())
    for bad in (dict(d_k=96), dict(heads=3), dict(tokens=0), dict(dtype=2)):
        for backward in (0, 1):
            assert capi.ttt_gated_delta_workspace_bytes(backward, _shape(**bad)) == 0
    assert capi.ttt_gated_delta_workspace_bytes(1, _shape()) > capi.ttt_gated_delta_workspace_bytes(0, _shape())
    assert capi.ttt_clip_workspace_bytes(0) == 0 < capi.ttt_clip_workspace_bytes(1) < capi.ttt_clip_workspace_bytes(1000)


@pytest.mark.parametrize("kw,expected", [
    (dict(batch=0), INVALID), (dict(tokens=0), INVALID), (dict(heads=3), INVALID), (dict(qk_heads=0), INVALID),
    (dict(dtype=7), INVALID), (dict(d_k=32), UNSUPPORTED), (dict(d_v=256), UNSUPPORTED),
    (dict(batch=1 << 16, tokens=1 << 25), UNSUPPORTED),
])
def test_shapes_are_refused(kw, expected):
    c = Call()
    c.shape = _shape(**kw)
    assert c.run() == expected


def test_good_arguments_reach_the_pointer_checks():
    # made-up addresses are no device memory
    assert Call().run() == INVALID
    c = Call()
    c.ws_bytes = capi.ttt_gated_delta_workspace_bytes(0, c.shape) - 1
    assert c.run() == WORKSPACE
    c.ws = None
    assert c.run() == WORKSPACE


def test_alignment_is_checked():
    for name in ("Q", "K", "V", "Z"):
        c = Call()
        c.views[name].data = c.views[name].data + 8
        assert c.run() == ALIGNMENT
        c = Call()
        c.views[name].token_stride += 4
        assert c.run() == ALIGNMENT
    for name in ("G", "Beta"):
        c = Call()
        c.views[name].data = c.views[name].data + 2
        assert c.run() == ALIGNMENT
    c = Call()
    c.W0 = BASE + (12 << 30) + 8
    assert c.run() == ALIGNMENT
    c = Call()
    c.ws += 16
    assert c.run() == ALIGNMENT


def test_bad_values_are_refused():
    for change in (dict(scale=float("nan")), dict(scale=float("inf"))):
        c = Call()
        c.__dict__.update(change)
        assert c.run() == INVALID
    for name in ("Q", "G", "Z"):
        c = Call()
        c.views[name].data = None
        assert c.run() == INVALID
        c = Call()
        c.views[name].head_stride = -64
        assert c.run() == INVALID
    assert capi.ttt_forward_gated_delta(None, None, None, None, None, None, 0, None, 1.0, None, None, _shape(), BASE, 1 << 30,
                                        None) == INVALID


def test_backward_and_step_are_checked():
    c = Call()
    v = c.views
    d = [capi.TttView(BASE + ((20 + i) << 30), x.batch_stride, x.head_stride, x.token_stride)
         for i, x in enumerate((v["Q"], v["K"], v["V"], v["G"], v["Beta"]))]

    def backward(dW0=None, W0=None, ws_bytes=1 << 30, dQ=d[0]):
        return capi.ttt_backward_gated_delta(v["Q"], v["K"], v["V"], v["G"], v["Beta"], W0, 0, None, 1.0, v["Z"], None, c.shape,
                                             BASE + (10 << 30), ws_bytes, dQ, *d[1:], dW0, None)

    assert backward(dW0=BASE + (30 << 30)) == INVALID            # a gradient of weights that are not there
    assert backward(ws_bytes=256) == WORKSPACE
    assert backward(dQ=None) == INVALID
    assert backward() == INVALID                                 # made-up addresses

    def step(W=BASE + (12 << 30), n_slots=2, shape=c.shape):
        return capi.ttt_step_gated_delta(v["Q"], v["K"], v["V"], v["G"], v["Beta"], W, n_slots, None, 1.0, v["Z"], shape, None)

    assert step(W=None) == INVALID and step(n_slots=0) == INVALID and step(n_slots=1) == INVALID
    assert step(W=BASE + (12 << 30) + 4) == ALIGNMENT and step(shape=_shape(d_k=16)) == UNSUPPORTED


def _clip(grads, out, counts, dtypes=None, max_norm=1.0, ws_bytes=1 << 20):
    n = len(grads)
    vp, ll, ci = ctypes.c_void_p * n, ctypes.c_longlong * n, ctypes.c_int * n
    return capi.ttt_clip_gradients(vp(*grads), vp(*out), ll(*counts), ci(*(dtypes or [capi.TTT_FP32] * n)), n, max_norm, BASE,
                                   BASE + (1 << 30), ws_bytes, None)


def test_clip_is_checked():
    a, b = BASE + (2 << 30), BASE + (3 << 30)
    assert _clip([a], [a], [4], max_norm=-1.0) == INVALID
    assert _clip([a], [a], [4], max_norm=float("nan")) == INVALID
    assert _clip([a], [a], [4], dtypes=[5]) == INVALID
    assert _clip([a], [a], [-1]) == INVALID
    assert _clip([a], [None], [4]) == INVALID
    assert _clip([a + 2], [a + 2], [4]) == ALIGNMENT
    assert _clip([a], [a], [4], ws_bytes=8) == WORKSPACE
    assert _clip([a, a], [a, a], [4, 4]) == INVALID              # twice
    assert _clip([a, b], [b, a], [4, 4]) == INVALID              # over another's input
    assert _clip([a], [BASE], [4]) == INVALID                    # over the norm
    assert _clip([a], [a], [4]) == INVALID                       # made-up addresses
