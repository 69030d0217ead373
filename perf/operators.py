"""Cases of the recurrent policy's operators and their plain forms.

The operators are those of a sequence model whose core is a selective state
space recurrence, over rows of T steps as everywhere in this package:

* `conv`   the short causal convolution in front of the scan (rows, rows with
           gradients, one step per sequence);
* `scan`   the selective scan h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t,
           y_t = C_t . h_t (rows, rows with gradients, one step per sequence);
* `clip`   the global norm of a model's gradients, and the gradients scaled to
           at most `max_norm`.

`run` computes a case with elementary torch operations in float32, or, where
`own` is true, through linear_recurrence_scan_row_amd.  `exact` computes it in
float64 step by step from the recurrences, with the gradients from automatic
differentiation, so it shares no formula with either.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEVICE = "cuda"


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one prompt of odd length through one layer's convolution
        dict(name="conv_prompt", op="conv", train=False, N=1, D=4096, T=8191, W=4, dtype="bf16",
             flags=False, lengths=False, state=False),
        # the PPO rollout window of 4096 environments: episodes begin inside the rows
        dict(name="conv_rollouts_train", op="conv", train=True, N=4096, D=64, T=128, W=4,
             dtype="f32", flags=True, lengths=False, state=True),
        # one new token for one sequence: latency
        dict(name="conv_step_one", op="conv_step", N=1, D=2048, W=4, dtype="f32", slots=False,
             flags=False),
        # one token for each of a large batch, states in a pool
        dict(name="conv_step_many", op="conv_step", N=512, D=8192, W=4, dtype="bf16", slots=True,
             flags=True),
        # one prompt, the state kept for generation
        dict(name="scan_prompt_one", op="scan", train=False, N=1, D=4096, S=16, T=4096, G=1,
             dtype="bf16", z=True, flags=False, lengths=False, state=False),
        # prompts of different lengths padded to one odd length, grouped B and C
        dict(name="scan_prompt_ragged", op="scan", train=False, N=6, D=1536, S=16, T=2049, G=2,
             dtype="f16", z=True, flags=False, lengths=True, state=True),
        # a training step's layer over token rows
        dict(name="scan_train_tokens", op="scan", train=True, N=8, D=2048, S=16, T=2048, G=1,
             dtype="bf16", z=True, flags=False, lengths=False, state=False),
        # a training step's layer over the PPO rollout window, with episode starts
        dict(name="scan_train_rollouts", op="scan", train=True, N=4096, D=64, S=16, T=128, G=1,
             dtype="f32", z=False, flags=True, lengths=False, state=True),
        # one new token for one sequence: latency
        dict(name="scan_step_one", op="scan_step", N=1, D=2048, S=16, G=1, dtype="f32", z=True,
             slots=False, flags=False),
        # one token (or one action) for each of a large batch, states in a pool
        dict(name="scan_step_many", op="scan_step", N=512, D=4096, S=16, G=1, dtype="bf16",
             z=True, slots=True, flags=True),
        # the gradients of a small policy network
        dict(name="clip_policy", op="clip", tensors=26, total=400_003, dtype="f32"),
        # the gradients of a large model, as a few large tensors and many small ones
        dict(name="clip_model", op="clip", tensors=60, total=400_000_000, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("conv", "conv", "conv_step", "scan", "scan", "scan", "scan_step", "clip"))
    dtype = rng.choice(("f32", "bf16", "f16"))
    if op == "clip":
        return dict(op=op, tensors=rng.randint(1, 60), total=_log_int(rng, 2_000, 300_000_000),
                    dtype=dtype)
    if op in ("conv_step", "scan_step"):
        N, D = _log_int(rng, 1, 512), _log_int(rng, 32, 4096)
        c = dict(op=op, N=N, D=D, dtype=dtype, slots=rng.random() < 0.5,
                 flags=rng.random() < 0.5)
        if op == "conv_step":
            return dict(c, W=rng.choice((2, 3, 4)))
        G = rng.choice((1, 1, 2))
        return dict(c, D=D + D % G, S=rng.choice((4, 8, 16, 16, 24, 32, 64)), G=G,
                    z=rng.random() < 0.7)
    flags = rng.random() < 0.4
    c = dict(op=op, train=rng.random() < 0.5, dtype=dtype, flags=flags,
             lengths=not flags and rng.random() < 0.4, state=rng.random() < 0.5)
    S = rng.choice((4, 8, 16, 16, 24, 32, 64)) if op == "scan" else 16
    most = min(400_000_000 // S, 33_000_000)  # steps of a row, over all rows
    T = _log_int(rng, 1, 16384)
    N = _log_int(rng, 1, max(1, min(4096, most // (64 * T))))
    D = _log_int(rng, 16, max(17, min(8192, most // (N * T))))
    if op == "conv":
        return dict(c, N=N, D=D, T=T, W=rng.choice((2, 3, 4)))
    G = rng.choice((1, 1, 2))
    return dict(c, N=N, D=D + D % G, S=S, T=T, G=G, z=rng.random() < 0.6)


# ------------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, device=DEVICE, generator=g) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, device=DEVICE, generator=g)

    s = {"case": dict(case)}
    op = case["op"]
    if op == "clip":
        # a few tensors hold most of the elements; none is empty, and sizes are odd
        k, total = case["tensors"], case["total"]
        r = np.random.RandomState((k * 1_000_003 + total) % (1 << 31))
        share = r.pareto(0.7, k) + 0.01
        sizes = np.maximum(1, (share / share.sum() * total).astype(np.int64))
        s["grads"] = [normal(int(n), scale=1e-3) for n in sizes]
        s["out"] = [torch.empty_like(x) for x in s["grads"]]
        s["max_norm"] = 0.37 * 1e-3 * math.sqrt(total)
        return s
    N, D = case["N"], case["D"]
    if op in ("conv", "conv_step"):
        W = case["W"]
        s["weight"] = normal(D, W, scale=1 / math.sqrt(W), dtype=torch.float32)
        s["bias"] = normal(D, scale=0.1, dtype=torch.float32)
    else:
        S, G = case["S"], case["G"]
        s["A"] = -(torch.arange(1, S + 1, device=DEVICE, dtype=torch.float32)
                   * torch.exp(0.1 * normal(D, S, dtype=torch.float32)))
        s["D"] = 1 + normal(D, scale=0.1, dtype=torch.float32)
        # softplus(delta_bias) is log-uniform over 0.001 .. 0.1
        step = torch.exp(uniform(D) * math.log(100.0) + math.log(1e-3))
        s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    if op in ("conv_step", "scan_step"):
        P = N + N // 4 + 1 if case["slots"] else N  # places of the pool
        if case["slots"]:
            s["slots"] = torch.randperm(P, device=DEVICE, generator=g)[:N].to(torch.int32)
        if case["flags"]:
            s["flags"] = (uniform(N) < 0.05).to(torch.uint8)
        if op == "conv_step":
            s["x"] = normal(N, D)
            s["state"] = normal(P, D, W - 1)
            return s
        xz = normal(N, 2 * D)  # one projection's output: u and the gate
        s["u"] = xz[:, :D]
        if case["z"]:
            s["z"] = xz[:, D:]
        s["delta"] = normal(N, D, scale=0.3)
        bc = normal(N, 2 * G * S)
        s["B"] = bc[:, :G * S].view(N, G, S)
        s["C"] = bc[:, G * S:].view(N, G, S)
        s["state"] = normal(P, D, S, scale=0.1, dtype=torch.float32)
        return s
    T = case["T"]
    if case["flags"]:
        s["flags"] = (uniform(N, T) < 0.01).to(torch.uint8)
    if case["lengths"]:
        lengths = (uniform(N) * (T + 1)).to(torch.int32).clamp_(max=T)
        lengths[0] = T
        s["lengths"] = lengths
    xz = normal(N, 2 * D, T)  # one projection's output: the input rows and the gate's
    if op == "conv":
        s["x"] = xz[:, :D]
        if case["state"]:
            s["state"] = normal(N, D, W - 1)
        if case["train"]:
            s["grad_out"] = normal(N, D, T)
        return s
    s["u"] = xz[:, :D]
    if case["z"]:
        s["z"] = xz[:, D:]
    s["delta"] = normal(N, D, T, scale=0.3)
    bc = normal(N, 2 * G * S, T)
    s["B"] = bc[:, :G * S].view(N, G, S, T)
    s["C"] = bc[:, G * S:].view(N, G, S, T)
    if case["state"]:
        s["state"] = normal(N, D, S, scale=0.1, dtype=torch.float32)
    if case["train"]:
        s["grad_y"] = normal(N, D, T)
        if case["state"]:
            s["grad_state"] = normal(N, D, S, scale=0.1, dtype=torch.float32)
    return s


def work(case):
    """Inputs read once, outputs written once; one operation for each product,
    sum and exponential of the recurrences."""
    op = case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "clip":
        return {"bytes": 2 * e * case["total"] + 8, "flops": 3 * case["total"]}
    N, D = case["N"], case["D"]
    if op == "conv_step":
        W = case["W"]
        return {"bytes": N * D * e * (2 + 2 * (W - 1)) + 4 * D * (W + 1),
                "flops": N * D * (2 * W + 4)}
    if op == "scan_step":
        S, G = case["S"], case["G"]
        return {"bytes": N * D * (8 * S + e * (4 if case["z"] else 3)) + e * 2 * N * G * S
                + 4 * D * (S + 2), "flops": N * D * (7 * S + 12)}
    T = case["T"]
    rows = N * D * T
    flags = N * T if case["flags"] else 0
    if op == "conv":
        W = case["W"]
        state = N * D * (W - 1) * e
        small = 4 * D * (W + 1)
        if not case["train"]:
            return {"bytes": rows * e * 2 + flags + small + state * (2 if case["state"] else 1),
                    "flops": rows * (2 * W + 4)}
        return {"bytes": rows * e * 4 + flags + 2 * small + state * (2 if case["state"] else 0),
                "flops": rows * (8 * W + 12)}
    S, G = case["S"], case["G"]
    state = N * D * S * 4
    bc = N * 2 * G * S * T * e
    small = 4 * D * (S + 2)
    z = 1 if case["z"] else 0
    if not case["train"]:
        return {"bytes": rows * e * (3 + z) + bc + flags + small
                + state * (2 if case["state"] else 1), "flops": rows * (7 * S + 8)}
    return {"bytes": rows * e * (6 + 2 * z) + 2 * bc + flags + 2 * small
            + state * (3 if case["state"] else 0), "flops": rows * (23 * S + 24)}


# --------------------------------------------------------------- plain operators
def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20))))


def _starts(flags):
    return None if flags is None else flags != 0


def _valid(lengths, T):
    """[N, 1, T]: the steps before each sequence's end."""
    t = torch.arange(T, device=DEVICE)
    return (t[None] < lengths[:, None])[:, None]


def _taps(x, state, W, starts):
    """W arrays: the input j steps back, 0 across an episode's start (or before
    the first step, unless a state holds those inputs)."""
    N, D, T = x.shape
    before = x.new_zeros(N, D, W - 1) if state is None else state.float()
    padded = torch.cat([before, x], dim=2)
    keep = [None]
    if starts is not None:
        # `keep[j]`: no episode starts in the last j steps, step t included
        open_ = torch.cat([torch.ones(N, W - 1, dtype=torch.bool, device=DEVICE), ~starts], 1)
        keep += [torch.stack([open_[:, W - 1 - i:W - 1 - i + T] for i in range(j)]).all(0)
                 for j in range(1, W)]
    taps = [padded[:, :, W - 1 - j:W - 1 - j + T] for j in range(W)]
    return [t if j == 0 or starts is None else t * keep[j][:, None] for j, t in enumerate(taps)], \
        keep, padded


def _conv_plain(s):
    c = s["case"]
    x = s["x"].float()
    N, D, T = x.shape
    W = c["W"]
    w, bias = s["weight"], s["bias"]
    starts, lengths = _starts(s.get("flags")), s.get("lengths")
    taps, keep, padded = _taps(x, s.get("state"), W, starts)
    pre = bias[:, None] + sum(w[:, W - 1 - j, None] * taps[j] for j in range(W))
    sig = 1 / (1 + torch.exp(-pre))
    out = pre * sig
    valid = None if lengths is None else _valid(lengths, T)
    if valid is not None:
        out = torch.where(valid, out, 0)
    dt = s["x"].dtype
    if not c["train"]:
        # the last W-1 inputs of each sequence, 0 before its last episode's start
        end = (torch.full((N,), T, device=DEVICE) if lengths is None else lengths).long()
        at = end[:, None] + torch.arange(W - 1, device=DEVICE)
        final = padded.gather(2, at[:, None].expand(N, D, W - 1))
        if starts is not None:
            last = torch.where(starts, torch.arange(T, device=DEVICE), -W).amax(1)
            final = final * ((at - (W - 1)) >= last[:, None])[:, None]
        return out.to(dt), final.to(dt)
    go = s["grad_out"].float()
    dpre = go * sig * (1 + pre * (1 - sig))
    if valid is not None:
        dpre = torch.where(valid, dpre, 0)
    back = [dpre * w[:, W - 1 - j, None] if j == 0 or starts is None
            else dpre * w[:, W - 1 - j, None] * keep[j][:, None] for j in range(W)]
    dpad = x.new_zeros(N, D, T + W - 1)
    for j in range(W):
        dpad[:, :, W - 1 - j:W - 1 - j + T] += back[j]
    grads = {"x": dpad[:, :, W - 1:].to(dt),
             "weight": torch.stack([(dpre * taps[W - 1 - k]).sum((0, 2)) for k in range(W)], 1),
             "bias": dpre.sum((0, 2))}
    if c["state"]:
        grads["state"] = dpad[:, :, :W - 1].to(dt)
    return out.to(dt), grads


def _conv_step_plain(s):
    state, at = s["state"], s.get("slots")
    at = slice(None) if at is None else at.long()
    before = state[at].float()
    if "flags" in s:
        before = before * (s["flags"] == 0)[:, None, None]
    full = torch.cat([before, s["x"].float()[:, :, None]], 2)
    pre = (full * s["weight"]).sum(2) + s["bias"]
    state[at] = full[:, :, 1:].to(state.dtype)
    return (pre / (1 + torch.exp(-pre))).to(s["x"].dtype), state


def _rows_scan(a, b, h):
    """h_t = a_t h_{t-1} + b_t along the last axis, h_{-1} = h, by doubling."""
    if h is not None:
        b = torch.cat([b[..., :1] + a[..., :1] * h[..., None], b[..., 1:]], -1)
    k = 1
    while k < a.shape[-1]:
        b = torch.cat([b[..., :k], torch.addcmul(b[..., k:], a[..., k:], b[..., :-k])], -1)
        a = torch.cat([a[..., :k], a[..., k:] * a[..., :-k]], -1)
        k *= 2
    return b


def _spread(x, D):
    """[N, G, S, ...] for each of D channels (a view where there is one group)."""
    G = x.shape[1]
    x = x.float()
    return x if G == 1 else x.repeat_interleave(D // G, 1)


def _scan_plain(s):
    c = s["case"]
    u, raw = s["u"].float(), s["delta"].float() + s["delta_bias"][:, None]
    N, D, T = u.shape
    A, skip = s["A"], s["D"]
    B, C = _spread(s["B"], D), _spread(s["C"], D)
    starts, lengths = _starts(s.get("flags")), s.get("lengths")
    delta = _softplus(raw)
    valid = None if lengths is None else _valid(lengths, T)
    live = delta if valid is None else torch.where(valid, delta, 0)
    a = torch.exp(live[:, :, None] * A[:, :, None])
    if starts is not None:
        a = torch.where(starts[:, None, None], 0, a)
    h0 = s.get("state")
    h = _rows_scan(a, (live * u)[:, :, None] * B, h0)
    y0 = (h * C).sum(2) + skip[:, None] * u
    dt = s["u"].dtype
    gate = None
    if c["z"]:
        z = s["z"].float()
        sig = 1 / (1 + torch.exp(-z))
        gate = z * sig
    y = y0 if gate is None else y0 * gate
    if valid is not None:
        y = torch.where(valid, y, 0)
    if not c["train"]:
        return y.to(dt), h[..., -1].contiguous()
    gy = s["grad_y"].float()
    if valid is not None:
        gy = torch.where(valid, gy, 0)
    grads = {}
    if c["z"]:
        grads["z"] = (gy * y0 * sig * (1 + z * (1 - sig))).to(dt)
        gy = gy * gate
    # dL/dh_t = C_t gy_t + a_{t+1} dL/dh_{t+1}, from the last step back
    gin = C * gy[:, :, None]
    if "grad_state" in s:
        gin[..., -1] += s["grad_state"]
    anext = torch.cat([a[..., 1:], torch.ones_like(a[..., :1])], -1)
    gh = _rows_scan(anext.flip(-1), gin.flip(-1), None).flip(-1)
    first = torch.zeros_like(h[..., 0]) if h0 is None else h0
    ah = a * torch.cat([first[..., None], h[..., :-1]], -1)
    gb = (gh * B).sum(2)
    gdelta = (gh * ah * A[:, :, None]).sum(2) + u * gb
    if valid is not None:
        gdelta = torch.where(valid, gdelta, 0)
        gb = torch.where(valid, gb, 0)
    graw = gdelta / (1 + torch.exp(-raw))
    G = c["G"]
    grads["u"] = (live * gb + skip[:, None] * gy).to(dt)
    grads["delta"] = graw.to(dt)
    grads["A"] = (gh * ah * live[:, :, None]).sum((0, 3))
    grads["B"] = (gh * (live * u)[:, :, None]).view(N, G, D // G, c["S"], T).sum(2).to(dt)
    grads["C"] = (h * gy[:, :, None]).view(N, G, D // G, c["S"], T).sum(2).to(dt)
    grads["D"] = (gy * u).sum((0, 2))
    grads["delta_bias"] = graw.sum((0, 2))
    if c["state"]:
        grads["state"] = a[..., 0] * gh[..., 0]
    return y.to(dt), grads


def _scan_step_plain(s):
    state, at = s["state"], s.get("slots")
    at = slice(None) if at is None else at.long()
    u = s["u"].float()
    D = u.shape[1]
    delta = _softplus(s["delta"].float() + s["delta_bias"])
    h = state[at]
    if "flags" in s:
        h = h * (s["flags"] == 0)[:, None, None]
    h = torch.exp(delta[:, :, None] * s["A"]) * h + (delta * u)[:, :, None] * _spread(s["B"], D)
    state[at] = h
    y = (h * _spread(s["C"], D)).sum(2) + s["D"] * u
    if "z" in s:
        z = s["z"].float()
        y = y * z / (1 + torch.exp(-z))
    return y.to(s["u"].dtype), state


def _clip_plain(s):
    sums = torch.stack([x.float().square().sum(dtype=torch.float64) for x in s["grads"]])
    norm = sums.sum().sqrt()
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
    return norm.reshape(1), [(x.float() * scale).to(x.dtype) for x in s["grads"]]


# ------------------------------------------------------- the package's operators
def _conv_own(s):
    import linear_recurrence_scan_row_amd as rl
    c = s["case"]
    kw = dict(state=s.get("state"), flags=s.get("flags"), lengths=s.get("lengths"))
    out, final = rl.causal_conv(s["x"], s["weight"], s["bias"], with_state=not c["train"], **kw)
    if not c["train"]:
        return out, final
    g = rl.causal_conv_backward(s["grad_out"], s["x"], s["weight"], s["bias"], **kw)
    grads = {"x": g.x, "weight": g.weight, "bias": g.bias}
    if c["state"]:
        grads["state"] = g.state
    return out, grads


def _conv_step_own(s):
    import linear_recurrence_scan_row_amd as rl
    out = rl.causal_conv_step(s["x"], s["weight"], s["bias"], s["state"], slots=s.get("slots"),
                              flags=s.get("flags"))
    return out, s["state"]


def _scan_own(s):
    import linear_recurrence_scan_row_amd as rl
    c = s["case"]
    kw = dict(D=s["D"], z=s.get("z"), delta_bias=s["delta_bias"], state=s.get("state"),
              flags=s.get("flags"), lengths=s.get("lengths"))
    args = (s["u"], s["delta"], s["A"], s["B"], s["C"])
    if not c["train"]:
        y, final, _ = rl.selective_scan(*args, with_state=True, **kw)
        return y, final
    y, _, checkpoints = rl.selective_scan(*args, with_checkpoints=True, **kw)
    g = rl.selective_scan_backward(s["grad_y"], *args, checkpoints,
                                   grad_state=s.get("grad_state"), **kw)
    grads = {"u": g.u, "delta": g.delta, "A": g.A, "B": g.B, "C": g.C, "D": g.D,
             "delta_bias": g.delta_bias}
    if c["z"]:
        grads["z"] = g.z
    if c["state"]:
        grads["state"] = g.state
    return y, grads


def _scan_step_own(s):
    import linear_recurrence_scan_row_amd as rl
    y = rl.selective_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], D=s["D"],
                          z=s.get("z"), delta_bias=s["delta_bias"], slots=s.get("slots"),
                          flags=s.get("flags"))
    return y, s["state"]


def _clip_own(s):
    import linear_recurrence_scan_row_amd as rl
    norm = rl.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
    return norm, s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _conv_own, "conv_step": _conv_step_own, "scan": _scan_own,
                "scan_step": _scan_step_own, "clip": _clip_own}[op](state)
    return {"conv": _conv_plain, "conv_step": _conv_step_plain, "scan": _scan_plain,
            "scan_step": _scan_step_plain, "clip": _clip_plain}[op](state)


# ------------------------------------------------------------- the definitions
def _double(s, names):
    return {k: s[k].double().requires_grad_() for k in names if k in s}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        grads = [x.double() for x in s["grads"]]
        norm = torch.sqrt(sum((x * x).sum() for x in grads))
        scale = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        return norm.reshape(1), [x * scale for x in grads]
    if op in ("conv_step", "scan_step"):
        return _exact_step(s)
    train = case["train"]
    with torch.set_grad_enabled(train):
        d = _double(s, ("x", "u", "weight", "bias", "delta", "A", "B", "C", "D", "z",
                        "delta_bias", "state"))
        out, final = (_exact_conv if op == "conv" else _exact_scan)(s, d)
        if not train:
            return out.detach(), final.detach()
        total = (out * s["grad_out" if op == "conv" else "grad_y"].double()).sum()
        if "grad_state" in s:
            total = total + (final * s["grad_state"].double()).sum()
        total.backward()
    return out.detach(), {k: v.grad for k, v in d.items()}


def _exact_conv(s, d):
    """Step by step over the window of the last W inputs."""
    case = s["case"]
    N, D, T, W = case["N"], case["D"], case["T"], case["W"]
    x = d["x"]
    begin = d["state"] if "state" in d else x.new_zeros(N, D, W - 1)
    rows = torch.cat([begin, x], 2)
    # the episode that each input belongs to; a tap counts within its own episode
    episode = torch.zeros(N, T + W - 1, dtype=torch.long, device=DEVICE)
    if "flags" in s:
        episode[:, W - 1:] = (s["flags"] != 0).long().cumsum(1)
    pre = d["bias"][:, None].expand(D, T)[None]
    for k in range(W):
        same = episode[:, k:k + T] == episode[:, W - 1:]
        pre = pre + torch.where(same[:, None], rows[:, :, k:k + T], 0.0) * d["weight"][:, k, None]
    out = pre * torch.sigmoid(pre)
    ends = s["lengths"].tolist() if "lengths" in s else [T] * N
    if "lengths" in s:
        out = out * (torch.arange(T, device=DEVICE) < s["lengths"][:, None])[:, None]
    if case["train"]:
        return out, None
    final = torch.stack([rows[n, :, e:e + W - 1]
                         * (episode[n, e:e + W - 1] == episode[n, e + W - 2]) for n, e in
                         enumerate(ends)])
    return out, final


def _exact_scan(s, d):
    case = s["case"]
    N, D, S, T, G = (case[k] for k in ("N", "D", "S", "T", "G"))
    h = d["state"] if "state" in d else torch.zeros(N, D, S, device=DEVICE, dtype=torch.float64)
    delta = torch.logaddexp(d["delta"] + d["delta_bias"][:, None],
                            torch.zeros((), device=DEVICE, dtype=torch.float64))
    # one row of the coefficients for all the channels of a group
    shape = (N, G, D // G)
    rows = [v.reshape(*shape, T).unbind(3) for v in (delta, d["u"])]
    Bs, Cs = d["B"].unbind(3), d["C"].unbind(3)
    A, skip = d["A"].view(G, D // G, S), d["D"].view(G, D // G)
    h = h.reshape(*shape, S)
    ys = []
    for t in range(T):
        if "flags" in s:
            h = h * (s["flags"][:, t] == 0).double().view(N, 1, 1, 1)
        dt, u = rows[0][t], rows[1][t]
        new = torch.exp(dt[..., None] * A) * h + (dt * u)[..., None] * Bs[t][:, :, None]
        if "lengths" in s:
            new = torch.where((t < s["lengths"]).view(N, 1, 1, 1), new, h)
        h = new
        ys.append(torch.matmul(h, Cs[t][..., None])[..., 0] + skip * u)
    y = torch.stack(ys, 3).reshape(N, D, T)
    if "z" in d:
        y = y * d["z"] * torch.sigmoid(d["z"])
    if "lengths" in s:
        y = y * (torch.arange(T, device=DEVICE) < s["lengths"][:, None])[:, None]
    return y, h.reshape(N, D, S)


def _exact_step(s):
    case = s["case"]
    N = case["N"]
    places = s["slots"].tolist() if "slots" in s else list(range(N))
    at = torch.tensor(places, device=DEVICE)
    state = s["state"].double()
    old = state[at]
    if "flags" in s:
        old[s["flags"] != 0] = 0.0
    if case["op"] == "conv_step":
        window = torch.cat([old, s["x"].double().unsqueeze(2)], 2)
        pre = torch.einsum("ndw,dw->nd", window, s["weight"].double()) + s["bias"].double()
        state[at] = window[:, :, 1:]
        return pre * torch.sigmoid(pre), state
    D, S, G = case["D"], case["S"], case["G"]
    u = s["u"].double()
    raw = s["delta"].double() + s["delta_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    group = torch.arange(D, device=DEVICE) // (D // G)
    new = old * torch.exp(torch.einsum("nd,ds->nds", dt, s["A"].double())) \
        + torch.einsum("nd,nds->nds", dt * u, s["B"].double()[:, group])
    state[at] = new
    y = torch.einsum("nds,nds->nd", new, s["C"].double()[:, group]) + s["D"].double() * u
    if "z" in s:
        z = s["z"].double()
        y = y * z * torch.sigmoid(z)
    return y, state
