"""The block operators in 64 bits, step by step from their definitions, with a
bound on the error of each output for an evaluation in float32.

As in sequence_reference.py, every function returns {output: (value, bound)},
and the bounds are running error analyses: beside each quantity its magnitude
and the error that float32 roundings of u = 2^-24 relative can have built up.
The counts for the gated recurrence, relative unless said otherwise:
  * a sigmoid: the argument's error, (|raw| + 3 (|gate| + |bias|) + 4) u (the constant
    and products that its two parts meet in one sum, that sum, the exponential's own
    two) times 1 - sigmoid, and 4 for sum and reciprocal;
  * the rate scale softplus(decay): 8; L = rate times r: r's, the rate's and 2;
  * a = exp(-L): L times L's error and 2, and 6; and 2^-126 absolute, since the
    exponential of less than float32's smallest normal number is 0;
  * 1 - a: L exp(-L) / (1 - a), at most 1, times L's error, and 6; the root of
    (1 - a)(1 + a): half its factors' errors, and 4;
  * a step of a recurrence adds 4 (product, sum, and the regrouping of the scan);
  * each further product or sum adds 1; a sum of n terms adds n, in any order.
"""
import torch

from .sequence_reference import U, d64, ends_of, over_of, sigmoid, starts_of


def softplus(x):
    return torch.logaddexp(x, torch.zeros_like(x))


def gated(x, input_gate, decay_gate, decay, input_bias=None, decay_bias=None, scale=8.0,
          state=None, flags=None, convention=0, lengths=None, grad_out=None, grad_final=None):
    x, ig, dg, decay = d64(x), d64(input_gate), d64(decay_gate), d64(decay)
    N, D, T = x.shape
    ib = torch.zeros(D, dtype=torch.float64) if input_bias is None else d64(input_bias)
    db = torch.zeros(D, dtype=torch.float64) if decay_bias is None else d64(decay_bias)
    starts, ends = starts_of(flags, convention, N, T), ends_of(lengths, N, T)
    over = over_of(flags, convention, ends, N)
    inside = (torch.arange(T)[None] < ends[:, None])[:, None].expand(N, D, T)  # [N, D, T]
    raw_i, raw_r = ig + ib[:, None], dg + db[:, None]
    # of what is masked nothing is used
    raw_i, raw_r = torch.where(inside, raw_i, 0.0), torch.where(inside, raw_r, 0.0)
    ig, dg = torch.where(inside, ig, 0.0), torch.where(inside, dg, 0.0)
    x = torch.where(inside, x, 0.0)
    i, r = sigmoid(raw_i), sigmoid(raw_r)

    def sig_err(s, raw, v, b):
        return U * ((1 - s) * (raw.abs() + 3 * (v.abs() + b.abs()[:, None]) + 4) + 4)

    ei, er = sig_err(i, raw_i, ig, ib), sig_err(r, raw_r, dg, db)
    rate = scale * softplus(decay)[:, None]
    L = rate * r
    eL = er + 10 * U
    a, d = torch.exp(-L), -torch.expm1(-L)
    slope = torch.where(d > 0, L * a / torch.where(d > 0, d, 1.0), 1.0)
    ed = eL * slope + 6 * U
    ea = L * (eL + 2 * U) + 6 * U
    low = torch.where(L > 80, 2.0 ** -126, 0.0)
    beta = torch.sqrt(d * (1 + a))
    eb = (ed + ea) / 2 + 4 * U
    ix = i * x
    b = beta * ix
    err_b = b.abs() * (eb + ei + 3 * U)
    a = torch.where(inside, a, 1.0)
    ea = torch.where(inside, ea, 0.0)
    da = a * ea + torch.where(inside, low, 0.0)  # a's absolute error
    b, err_b = torch.where(inside, b, 0.0), torch.where(inside, err_b, 0.0)

    zeros = torch.zeros(N, D, dtype=torch.float64)
    h = zeros if state is None else d64(state)
    m, e = h.abs(), zeros
    hs, es, before, mbefore, ebefore = [], [], [], [], []
    for t in range(T):
        cut = starts[:, t][:, None] & inside[:, :, t]
        h, m, e = (torch.where(cut, 0.0, v) for v in (h, m, e))
        before.append(h), mbefore.append(m), ebefore.append(e)
        at, live = a[:, :, t], inside[:, :, t]
        new = at * h + b[:, :, t]
        new_m = at * m + b[:, :, t].abs()
        new_e = at * e + da[:, :, t] * (m + e) + err_b[:, :, t] + 4 * U * new_m
        h, m, e = (torch.where(live, p, q) for p, q in ((new, h), (new_m, m), (new_e, e)))
        hs.append(torch.where(live, h, 0.0)), es.append(torch.where(live, e, 0.0))

    def stack(rows):
        return torch.stack(rows, 2) if T > 0 else torch.zeros(N, D, 0, dtype=torch.float64)

    keep = ~over[:, None]
    res = {"out": (stack(hs), stack(es)), "final": (h * keep, e * keep)}
    if grad_out is None:
        return res
    g = torch.where(inside, d64(grad_out), 0.0)
    right = zeros if grad_final is None else d64(grad_final) * keep
    rm, re = right.abs(), zeros
    lam, lam_m, lam_e = [None] * T, [None] * T, [None] * T
    for t in reversed(range(T)):
        live = inside[:, :, t]
        lam[t] = torch.where(live, g[:, :, t] + right, 0.0)
        lam_m[t] = torch.where(live, g[:, :, t].abs() + rm, 0.0)
        lam_e[t] = torch.where(live, re + 4 * U * lam_m[t], 0.0)
        at = a[:, :, t]
        cut = starts[:, t][:, None] & live
        new = (at * lam[t], at * lam_m[t],
               at * lam_e[t] + da[:, :, t] * (lam_m[t] + lam_e[t]) + at * U * lam_m[t])
        right, rm, re = (torch.where(cut, 0.0, torch.where(live, p, q))
                         for p, q in zip(new, (right, rm, re)))
    res["state"] = (right, re)
    lam, lam_m, lam_e = stack(lam), stack(lam_m), stack(lam_e)
    before, mbefore, ebefore = stack(before), stack(mbefore), stack(ebefore)
    gx, gx_m = lam * beta * i, lam_m * beta * i
    gx_e = lam_e * beta * i + gx_m * (eb + ei + 3 * U)
    gi, gi_m = gx * x * (1 - i), gx_m * x.abs() * (1 - i)
    gi_e = gx_e * x.abs() * (1 - i) + gx_m * x.abs() * (i * ei + 2 * U) + 3 * U * gi_m
    inv = torch.where(beta > 0, 1 / torch.where(beta > 0, beta, 1.0), 0.0)
    gain = a * inv * ix
    term, term_m = L * a * (gain - before), L * a * (gain.abs() + mbefore)
    term_e = term_m * (eL + ea + 6 * U) + L * low * (gain.abs() + mbefore + ix.abs()) \
        + L * a * (gain.abs() * (ea + eb + ei + 6 * U) + ebefore)
    rate_g, rate_m = lam * term, lam_m * term_m
    rate_e = lam_e * term_m + lam_m * term_e + 2 * U * rate_m
    gr, gr_m = rate_g * (1 - r), rate_m * (1 - r)
    gr_e = rate_e * (1 - r) + rate_m * (r * er + 2 * U) + U * gr_m
    res["x"], res["input_gate"], res["decay_gate"] = (gx, gx_e), (gi, gi_e), (gr, gr_e)

    def total(v, v_m, v_e):
        return v.sum((0, 2)), v_e.sum((0, 2)) + N * T * U * v_m.sum((0, 2))

    res["input_bias"], res["decay_bias"] = total(gi, gi_m, gi_e), total(gr, gr_m, gr_e)
    sp = softplus(decay)
    ratio = torch.where(decay < -30, 1.0, sigmoid(decay) / torch.where(decay < -30, 1.0, sp))
    s, s_e = total(rate_g, rate_m, rate_e)
    res["decay"] = (s * ratio, s_e * ratio + 24 * U * (s * ratio).abs())
    return res


EPS = 1e-6


def rms_norm(x, weight=None, residual=None, eps=EPS, lengths=None, grad_out=None, grad_sum=None):
    """Over dimension 1 of [N, D, T] or [N, D].  The counts: a sum over D channels D / 32
    + 16 (a thread's serial part, and the lanes and waves that meet), its root's
    reciprocal half of that and 4; each further product or sum 1; a sum over
    sequences and steps one for each."""
    dims = x.dim()
    dtype = x.dtype
    total = x if residual is None else x + residual  # one rounding, as it is stored
    s = d64(total)
    if dims == 2:
        s = s.unsqueeze(2)
    N, D, T = s.shape
    inside = (torch.arange(T)[None] < ends_of(lengths, N, T)[:, None])[:, None].expand(N, D, T)
    s = torch.where(inside, s, 0.0)
    w = torch.ones(D, dtype=torch.float64) if weight is None else d64(weight)
    w = w[:, None]
    n = D / 32 + 16
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    er = n / 2 * U + 4 * U
    xh = s * r
    y = torch.where(inside, xh * w, 0.0)
    y_e = y.abs() * (er + 3 * U)

    def back(v, e):
        return (v, e) if dims == 3 else (v.squeeze(2), e.squeeze(2))

    most = y.abs().amax(1) if D > 0 else torch.zeros(N, T, dtype=torch.float64)
    scale = torch.where(inside[:, 0] if D > 0 else torch.zeros(N, T, dtype=torch.bool),
                        torch.clamp(most / 448, min=2.0 ** -120), 0.0)
    scale_e = scale * (er + 5 * U)
    # one rounding to e4m3: half of its step, 2^-4 of the value or 2^-10 below the
    # smallest normal one
    q_e = y_e + (y.abs() + y_e) * 2.0 ** -4 + 2.0 ** -10 * (scale + scale_e)[:, None]
    res = {"out": back(y, y_e), "sum": back(s, torch.zeros_like(s)),
           "dequantized": back(y, q_e),
           "scale": (scale, scale_e) if dims == 3 else (scale[:, 0], scale_e[:, 0])}
    if grad_out is None:
        return res
    g = d64(grad_out).reshape(N, D, T)
    g = torch.where(inside, g, 0.0)
    gw = g * w
    c, c_m = (gw * xh).mean(1, keepdim=True), (gw * xh).abs().mean(1, keepdim=True)
    c_e = c_m * (er + (n + 4) * U)
    gx = r * (gw - xh * c)
    gx_e = r * (gw.abs() * (er + 3 * U) + xh.abs() * (c.abs() * (2 * er + 4 * U) + c_e))
    if grad_sum is not None:
        gs = torch.where(inside, d64(grad_sum).reshape(N, D, T), 0.0)
        gx = gx + gs
        gx_e = gx_e + U * gs.abs()
    gx, gx_e = torch.where(inside, gx, 0.0), torch.where(inside, gx_e, 0.0)
    res["x"] = back(gx, gx_e)
    terms = (g * xh).abs().sum((0, 2))
    res["weight"] = ((g * xh).sum((0, 2)), terms * (er + 2 * U + N * T * U))
    return res
