"""The gated delta rule (forward over whole sequences, backward, one-step recurrence on a cache of states)
and clipping by the global gradient norm: their cases, their plain forms in elementary torch operations,
their definition in 64 bits, and the calls a user makes of the library.

The gated delta rule is test-time training of the linear inner model, one token at a time, with a
forget gate: with W [dv][dk] the inner model, g_t <= 0 the log of the gate and beta_t the step size,

    W_t = exp(g_t) W_{t-1} + beta_t (v_t - exp(g_t) W_{t-1} k_t) k_t^T,      z_t = scale W_t q_t.

With g = 0 and beta = 2 eta it is the linear head trained in mini-batches of one token.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------
def _delta(name, op, B, hk, h, N, dk, dv, dtype="bf16", layout="heads", ragged=False, w0="none", dW1=False):
    return {"name": name, "op": op, "B": B, "hk": hk, "h": h, "N": N, "dk": dk, "dv": dv, "dtype": dtype,
            "layout": layout, "ragged": ragged, "w0": w0, "dW1": dW1}


def _step(name, B, hk, h, n, dk, dv, slots, dtype="bf16", unused=0):
    return {"name": name, "op": "step", "B": B, "hk": hk, "h": h, "N": n, "dk": dk, "dv": dv, "dtype": dtype,
            "slots": slots, "unused": unused}


def _clip(name, count, total, dtype, max_norm, sizes):
    return {"name": name, "op": "clip", "count": count, "total": total, "dtype": dtype, "max_norm": max_norm,
            "sizes": sizes}


def listed():
    return [
        # one 224 x 224 image's 14 x 14 tokens through the three heads of a small layer: a latency case
        _delta("fwd_196", "forward", 1, 3, 3, 196, 64, 64, w0="shared"),
        # a batch of 1248 x 1248 images of different sizes, padded to 78 x 78 tokens, per-head starting weights
        _delta("fwd_6084_ragged", "forward", 8, 6, 6, 6084, 64, 64, ragged=True, w0="shared"),
        # prefill of one long prompt: 16 key heads shared by 32 value heads, projections laid out by token
        _delta("fwd_8192_shared_keys", "forward", 1, 16, 32, 8192, 128, 128, layout="tokens", w0="each"),
        # a check run in fp32
        _delta("fwd_1000_fp32", "forward", 2, 4, 4, 1000, 64, 64, dtype="fp32", w0="each"),
        # training step of a small layer on 14 x 14 tokens
        _delta("bwd_196", "backward", 4, 3, 3, 196, 64, 64, w0="shared"),
        # training step on long sequences
        _delta("bwd_4096", "backward", 2, 16, 16, 4096, 128, 128, layout="tokens", w0="shared"),
        # training step on a padded batch, shared key heads, with a gradient of the last state
        _delta("bwd_1531_ragged", "backward", 3, 4, 8, 1531, 128, 128, layout="tokens", ragged=True, w0="each",
               dW1=True),
        # one request's next token: a latency case
        _step("step_1", 1, 16, 32, 1, 128, 128, 4),
        # a full serving batch, its states at arbitrary places of the cache, some rows of the batch empty
        _step("step_256", 256, 16, 32, 1, 128, 128, 320, unused=9),
        # a few drafted tokens a sequence in one call
        _step("step_33x3", 33, 12, 12, 3, 64, 64, 40),
        # the gradients of a small model's layers: many small tensors
        _clip("clip_60_small", 60, 400_000, "mixed", 1.0, 11),
        # the gradients of a model of a quarter of a billion weights
        _clip("clip_60_large", 60, 250_000_000, "mixed", 1.0, 12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "step", "clip"])
    if op == "clip":
        c = _clip("", rng.randint(2, 60), _log_int(rng, 1_000, 200_000_000), rng.choice(["bf16", "fp32", "mixed"]),
                  rng.choice([0.5, 1.0, 1e6]), rng.randrange(1 << 20))
    elif op == "step":
        d = rng.choice([64, 128])
        hk = _log_int(rng, 1, 16)
        B = _log_int(rng, 1, 200)
        c = _step("", B, hk, hk * rng.choice([1, 1, 2]), rng.choice([1, 1, 1, 2, 4]), d, rng.choice([64, 128]),
                  B + rng.randint(0, 40), rng.choice(["bf16", "bf16", "fp32"]), unused=rng.randint(0, B // 4))
    else:
        N = _log_int(rng, 1, 6000)
        most = 100_000 // N                      # (image, head) pairs: bounds the work of a case
        hk = _log_int(rng, 1, max(1, min(16, most)))
        r = rng.choice([1, 1, 2, 4]) if hk * 4 <= most else 1
        B = _log_int(rng, 1, max(1, min(32, most // (hk * r))))
        c = _delta("", op, B, hk, hk * r, N, rng.choice([64, 128]), rng.choice([64, 128]),
                   rng.choice(["bf16", "bf16", "bf16", "fp32"]), rng.choice(["heads", "tokens"]), rng.random() < 0.4,
                   rng.choice(["none", "shared", "each"]), op == "backward" and rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------
def _clip_sizes(case):
    """Sizes that spread over their logarithm and add up to about the total; one of a single element."""
    r = random.Random(case["sizes"])
    w = [math.exp(r.uniform(0.0, 5.0)) for _ in range(case["count"])]
    s = sum(w)
    n = [max(1, int(case["total"] * x / s)) for x in w]
    n[0] = 1
    return n


def _clip_dtypes(case):
    one = {"bf16": ["bf16"], "fp32": ["fp32"], "mixed": ["bf16", "bf16", "fp32"]}[case["dtype"]]
    return [_DT[one[i % len(one)]] for i in range(case["count"])]


def _tokens(case, heads, width, gen, dtype, unit=False):
    """[B][heads][N][width], laid out by head or (a transposed view) by token."""
    B, N = case["B"], case["N"]
    shape = (B, N, heads, width) if case.get("layout") == "tokens" else (B, heads, N, width)
    x = torch.randn(shape, generator=gen, device="cuda")
    if unit:
        x = x / x.norm(dim=-1, keepdim=True)
    x = x.to(dtype)
    return x.transpose(1, 2) if case.get("layout") == "tokens" else x


def _gates(case, heads, gen):
    shape = (case["B"], case["N"], heads) if case.get("layout") == "tokens" else (case["B"], heads, case["N"])
    g = torch.nn.functional.logsigmoid(torch.randn(shape, generator=gen, device="cuda") * 1.5 + 4.0)
    beta = torch.sigmoid(torch.randn(shape, generator=gen, device="cuda"))
    return (g.transpose(1, 2), beta.transpose(1, 2)) if case.get("layout") == "tokens" else (g, beta)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "clip":
        std = 0.02
        grads = []
        for i, (n, dt) in enumerate(zip(_clip_sizes(case), _clip_dtypes(case))):
            x = (torch.randn(n + 1, generator=gen, device="cuda") * std).to(dt)
            grads.append(x[1:] if i % 5 == 4 else x[:n])       # views into larger buffers, as a flat bucket gives
        s["grads"], s["max_norm"] = grads, case["max_norm"]
        s["out"] = [torch.empty_like(x) for x in grads]
        return s
    B, hk, h, N, dk, dv = (case[x] for x in ("B", "hk", "h", "N", "dk", "dv"))
    dt = _DT[case["dtype"]]
    s["Q"] = _tokens(case, hk, dk, gen, dt, unit=True)
    s["K"] = _tokens(case, hk, dk, gen, dt, unit=True)
    s["V"] = _tokens(case, h, dv, gen, dt)
    s["G"], s["Beta"] = _gates(case, h, gen)
    s["scale"] = 1.0 if dk == 64 else dk ** -0.5
    if case["op"] == "step":
        s["W"] = torch.randn((case["slots"], h, dv, dk), generator=gen, device="cuda") / math.sqrt(dk)
        slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        if case["unused"]:
            slots[torch.randperm(B, generator=gen, device="cuda")[:case["unused"]]] = -1
        s["slots"] = slots
        s["Z"] = torch.zeros_like(s["V"])
        return s
    s["lengths"] = None
    if case["ragged"]:
        lengths = torch.randint(0, N + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        lengths[0] = N
        s["lengths"] = lengths
    shape = {"none": None, "shared": (h, dv, dk), "each": (B, h, dv, dk)}[case["w0"]]
    s["W0"] = None if shape is None else torch.randn(shape, generator=gen, device="cuda") / math.sqrt(dk)
    if case["op"] == "forward":
        s["W1"] = torch.empty((B, h, dv, dk), device="cuda")
    else:
        s["dZ"] = _tokens(case, h, dv, gen, dt)
        s["dW1"] = torch.randn((B, h, dv, dk), generator=gen, device="cuda") if case["dW1"] else None
    return s


# ---------------------------------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------------------------------
_C = 64        # tokens a chunk


def _chunks(x, n):
    """[B][h][N][...] padded with zeros to n chunks of _C tokens: [B][h][n][_C][...]."""
    B, h, N = x.shape[:3]
    if n * _C != N:
        x = torch.cat([x, x.new_zeros((B, h, n * _C - N) + x.shape[3:])], dim=2)
    return x.reshape((B, h, n, _C) + x.shape[3:])


def _delta_chunked(Q, K, V, G, Beta, W0, lengths, scale):
    """Z and the last state, both in 32 bits.  Inside a chunk of C tokens with the running log gates b,
    the token updates u solve (I + L) u = beta (v - exp(b) W k), L_ij = beta_i exp(b_i - b_j) k_i.k_j (j < i),
    so that only the state goes from chunk to chunk."""
    B, h, N, dv = V.shape
    r = h // Q.shape[1]
    q, k = (x.float().repeat_interleave(r, dim=1) for x in (Q, K))
    v, g, beta = V.float(), G.double(), Beta.float()
    if lengths is not None:
        live = (torch.arange(N, device=V.device)[None, :] < lengths[:, None])[:, None, :]
        g, beta = torch.where(live, g, 0.0), torch.where(live, beta, 0.0)
    n = -(-N // _C)
    q, k, v, g, beta = (_chunks(x, n) for x in (q, k, v, g, beta))
    b = torch.cumsum(g, dim=-1)
    diff = b[..., :, None] - b[..., None, :]
    i = torch.arange(_C, device=V.device)
    lower, strict = i[:, None] >= i[None, :], i[:, None] > i[None, :]
    decay = torch.exp(torch.where(lower, diff, -math.inf)).float()
    gam, suf = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None]
    L = torch.where(strict, decay * (k @ k.transpose(-1, -2)) * beta[..., None], 0.0)
    T = torch.eye(_C, device=V.device).expand_as(L)
    s = 1
    while s < _C:                # the inverse of I + L, by blocks of twice the size
        blk = (i[:, None] // s % 2 == 1) & (i[:, None] // s - 1 == i[None, :] // s)
        T = T - T @ torch.where(blk, L, 0.0) @ T
        s *= 2
    Uv = T @ (beta[..., None] * v)
    Wk = T @ (beta[..., None] * gam * k)
    A = scale * decay * (q @ k.transpose(-1, -2))
    qg, ku = scale * gam * q, suf * k
    S = v.new_zeros((B, h, dv, Q.shape[3])) if W0 is None else W0.float().expand(B, h, dv, Q.shape[3])
    Z = []
    for c in range(n):
        U = Uv[:, :, c] - Wk[:, :, c] @ S.transpose(-1, -2)
        Z.append(qg[:, :, c] @ S.transpose(-1, -2) + A[:, :, c] @ U)
        S = gam[:, :, c, -1, :, None] * S + U.transpose(-1, -2) @ ku[:, :, c]
    Z = torch.cat(Z, dim=2)[:, :, :N]
    return (Z if lengths is None else torch.where(live[..., None], Z, 0.0)), S


def _plain_backward(s):
    names = ["Q", "K", "V", "G", "Beta"] + (["W0"] if s["W0"] is not None else [])
    x = {n: s[n].detach().float().requires_grad_() for n in names}
    with torch.enable_grad():
        Z, S = _delta_chunked(x["Q"], x["K"], x["V"], x["G"], x["Beta"], x.get("W0"), s["lengths"], s["scale"])
        total = (Z * s["dZ"].float()).sum()
        if s["dW1"] is not None:
            total = total + (S * s["dW1"]).sum()
        grads = torch.autograd.grad(total, [x[n] for n in names])
    return {"d" + n: d.to(s[n].dtype) for n, d in zip(names, grads)}


def _plain_step(s):
    Q, K, V, G, Beta, W, slots = (s[x] for x in ("Q", "K", "V", "G", "Beta", "W", "slots"))
    r = V.shape[1] // Q.shape[1]
    q, k = (x.float().repeat_interleave(r, dim=1) for x in (Q, K))
    used = (slots >= 0)[:, None, None, None]
    at = slots.clamp(min=0).long()
    S = W[at]
    for t in range(V.shape[2]):
        S = torch.exp(G[:, :, t].float())[..., None, None] * S
        u = Beta[:, :, t].float()[..., None] * (V[:, :, t].float() - (S * k[:, :, t, None, :]).sum(-1))
        S = S + u[..., None] * k[:, :, t, None, :]
        z = s["scale"] * (S * q[:, :, t, None, :]).sum(-1)
        s["Z"][:, :, t] = torch.where(used[..., 0], z, s["Z"][:, :, t].float()).to(V.dtype)
    place = torch.where(slots >= 0, at, W.shape[0])
    W.copy_(torch.cat([W, W.new_zeros((1,) + W.shape[1:])]).index_copy(0, place, S)[:-1])
    return {"Z": s["Z"], "W": W}


def _plain_clip(s):
    sq = torch.stack([x.double().square().sum() for x in s["grads"]]).sum()
    norm = sq.sqrt()
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
    return [norm.float()] + [(x.float() * coef).to(x.dtype) for x in s["grads"]]


# ---------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import vision_test_token_b200 as ttt
        if op == "forward":
            Z = ttt.forward_gated_delta(s["Q"], s["K"], s["V"], s["G"], s["Beta"], W0=s["W0"], lengths=s["lengths"],
                                        scale=s["scale"], W1_out=s["W1"])
            return {"Z": Z, "W1": s["W1"]}
        if op == "backward":
            d = ttt.backward_gated_delta(s["Q"], s["K"], s["V"], s["G"], s["Beta"], s["dZ"], W0=s["W0"], dW1=s["dW1"],
                                         lengths=s["lengths"], scale=s["scale"])
            return {n: x for n, x in zip(("dQ", "dK", "dV", "dG", "dBeta", "dW0"), d) if x is not None}
        if op == "step":
            ttt.step_gated_delta(s["Q"], s["K"], s["V"], s["G"], s["Beta"], s["W"], slots=s["slots"],
                                 scale=s["scale"], Z=s["Z"])
            return {"Z": s["Z"], "W": s["W"]}
        norm = ttt.clip_gradients(s["grads"], s["max_norm"], out=s["out"])
        return [norm.reshape(())] + s["out"]
    if op == "forward":
        Z, S = _delta_chunked(s["Q"], s["K"], s["V"], s["G"], s["Beta"], s["W0"], s["lengths"], s["scale"])
        return {"Z": Z.to(s["V"].dtype), "W1": S}
    if op == "backward":
        return _plain_backward(s)
    return _plain_step(s) if op == "step" else _plain_clip(s)


def work(case):
    if case["op"] == "clip":
        size = sum(n * (2 if dt == torch.bfloat16 else 4) for n, dt in zip(_clip_sizes(case), _clip_dtypes(case)))
        return {"bytes": 2 * size, "flops": 3 * sum(_clip_sizes(case))}
    B, hk, h, N, dk, dv = (case[x] for x in ("B", "hk", "h", "N", "dk", "dv"))
    e = 2 if case["dtype"] == "bf16" else 4
    state = h * dv * dk * 4
    qk, v, gates = 2 * B * hk * N * dk * e, B * h * N * dv * e, 2 * B * h * N * 4
    if case["op"] == "step":
        live = (B - case["unused"]) / B
        return {"bytes": live * (qk + 2 * v + gates + 2 * B * state), "flops": live * 8 * B * h * N * dk * dv}
    live = 0.5 + 0.5 / B if case["ragged"] else 1.0        # lengths are uniform, the first row's is whole
    w0 = {"none": 0, "shared": 1, "each": B}[case["w0"]] * state
    if case["op"] == "forward":
        return {"bytes": live * (qk + 2 * v + gates) + w0 + B * state, "flops": live * 8 * B * h * N * dk * dv}
    return {"bytes": live * (2 * qk + 3 * v + 2 * gates) + 2 * w0 + (B * state if case["dW1"] else 0),
            "flops": live * 22 * B * h * N * dk * dv}


# ---------------------------------------------------------------------------------------------------
# The definition, token by token, in 64 bits
# ---------------------------------------------------------------------------------------------------
def _sequence(s):
    """Inputs in 64 bits, by token: q, k [N][B][h][dk], v [N][B][h][dv], the gate a, beta [N][B][h]."""
    r = s["V"].shape[1] // s["Q"].shape[1]
    by_token = lambda x: x.double().permute(2, 0, 1, *range(3, x.dim())).contiguous()  # noqa: E731
    q, k = (by_token(s[n]).repeat_interleave(r, dim=2) for n in ("Q", "K"))
    return q, k, by_token(s["V"]), by_token(s["G"]).exp(), by_token(s["Beta"])


def _exact_forward(s, keep):
    q, k, v, a, beta = _sequence(s)
    N, B, h, dk = q.shape
    dv = v.shape[3]
    W0 = s["W0"]
    S = torch.zeros((B, h, dv, dk), dtype=torch.float64, device=q.device)
    if W0 is not None:
        S = S + W0.double()
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(N, device=q.device)[:, None] < s["lengths"][None, :]).double()
        a = torch.where(live[..., None] > 0, a, 1.0)
        beta = beta * live[..., None]
    states, resid, Z = [S], [], []
    for t in range(N):
        D = S * a[t, :, :, None, None]
        e = v[t] - torch.einsum("bhvk,bhk->bhv", D, k[t])
        S = torch.baddbmm(D.flatten(0, 1), (beta[t, :, :, None] * e).flatten(0, 1)[:, :, None],
                          k[t].flatten(0, 1)[:, None, :]).view_as(S)
        Z.append(torch.einsum("bhvk,bhk->bhv", S, q[t]))
        if keep:
            states.append(S)
            resid.append(e)
    Z = torch.stack(Z) * s["scale"]
    if live is not None:
        Z = Z * live[..., None, None]
    return q, k, a, beta, live, states, resid, Z.permute(1, 2, 0, 3), S


def _exact_backward(s):
    q, k, a, beta, live, states, resid, _, _ = _exact_forward(s, True)
    N, B, h, dk = q.shape
    dz = s["dZ"].double().permute(2, 0, 1, 3) * s["scale"]
    if live is not None:
        dz = dz * live[..., None, None]
    D = torch.zeros_like(states[0]) if s["dW1"] is None else s["dW1"].double()
    dq, dkk, dv, dg, db = [], [], [], [], []
    for t in reversed(range(N)):
        before, after, e = states[t], states[t + 1], resid[t]
        dq.append(torch.einsum("bhvk,bhv->bhk", after, dz[t]))
        D = D + dz[t][..., None] * q[t][..., None, :]
        du = torch.einsum("bhvk,bhk->bhv", D, k[t])
        de = beta[t][..., None] * du
        faded = before * a[t][..., None, None]
        db.append((du * e).sum(-1))
        dv.append(de)
        dkk.append(torch.einsum("bhvk,bhv->bhk", D, beta[t][..., None] * e) - torch.einsum("bhvk,bhv->bhk", faded, de))
        D = D - de[..., None] * k[t][..., None, :]
        dg.append((D * faded).sum((-1, -2)))
        D = D * a[t][..., None, None]
    order = lambda x: torch.stack(x[::-1]).permute(1, 2, 0, *range(3, x[0].dim() + 1))  # noqa: E731
    dq, dkk, dv, dg, db = (order(x) for x in (dq, dkk, dv, dg, db))
    if live is not None:
        mask = live.t()[:, None, :]
        dg, db = dg * mask, db * mask
    shared = lambda x: x.reshape(B, s["Q"].shape[1], -1, N, dk).sum(2)  # noqa: E731
    out = {"dQ": shared(dq), "dK": shared(dkk), "dV": dv, "dG": dg, "dBeta": db}
    if s["W0"] is not None:
        out["dW0"] = D if s["W0"].dim() == 4 else D.sum(0)
    return out


def _exact_step(s):
    slots = s["slots"].tolist()
    W, Z = s["W"].double(), s["Z"].double()
    rows = [b for b, p in enumerate(slots) if p >= 0]
    if not rows:
        return {"Z": Z, "W": W}
    pick = torch.tensor(rows, device=W.device)
    part = {n: s[n][pick] for n in ("Q", "K", "V", "G", "Beta")}
    where = s["slots"][pick].long()
    part.update(W0=W[where], lengths=None, scale=s["scale"])
    got = _exact_forward(part, False)
    Z[pick] = got[-2]
    W[where] = got[-1]
    return {"Z": Z, "W": W}


def _exact_clip(s):
    grads = [x.double() for x in s["grads"]]
    norm = math.sqrt(sum(float((x * x).sum()) for x in grads))
    coef = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
    return [torch.tensor(norm, dtype=torch.float64)] + [x * coef for x in grads]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        return _exact_clip(s)
    if case["op"] == "step":
        return _exact_step(s)
    if case["op"] == "forward":
        got = _exact_forward(s, False)
        return {"Z": got[-2], "W1": got[-1]}
    if case["B"] * case["h"] * case["N"] * case["dk"] * case["dv"] * 8 > 40e9:
        return None                              # the states of every token would not fit comfortably
    return _exact_backward(s)
