"""The sequence operators in 64 bits, step by step from their definitions, with
a bound on the error of each output for an evaluation in float32.

Every function returns {output: (value, bound)}.  The bounds are running error
analyses: beside each quantity its magnitude (the same sums over absolute
values) and the error that float32 roundings of u = 2^-24 relative can have
built up, carried through the recurrences.  The counts of roundings:
  * dt = softplus(delta + bias) is good to 12 roundings, and the sum's own
    rounding, |raw| u absolute, reaches dt relative to at most |raw| u more;
  * a = exp(dt A): the exponent's error (dt's, A's constant, the product)
    times |dt A|, and 4 for the exponential;
  * a step of a recurrence adds 4 (product, sum, and the regrouping of the
    scan, which adds a few sums per 8 steps);
  * a sum of n terms adds n, whatever its order.
`tolerance` adds the one rounding to the storage type.
"""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11,
             torch.float64: 0.0}
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25,
        torch.float64: 0.0}

ON_START, AFTER_DONE = 0, 1


def d64(t):
    return None if t is None else t.detach().cpu().double()


def tolerance(value, bound, dtype):
    return bound + HALF_STEP[dtype] * (value.abs() + bound) + TINY[dtype]


def starts_of(flags, convention, N, T):
    """[N, T + 1] bool: an episode starts at step t (column T: after the row)."""
    s = torch.zeros(N, T + 1, dtype=torch.bool)
    if flags is not None:
        f = flags.cpu() != 0
        if convention == ON_START:
            s[:, :T] = f
        else:
            s[:, 1:] = f
    return s


def ends_of(lengths, N, T):
    if lengths is None:
        return torch.full((N,), T)
    return lengths.cpu().long().clamp(0, T)


def over_of(flags, convention, ends, N):
    """Whether the step after each row's last one starts an episode."""
    over = torch.zeros(N, dtype=torch.bool)
    if flags is not None and convention == AFTER_DONE:
        for n in range(N):
            if ends[n] > 0:
                over[n] = bool(flags[n, ends[n] - 1] != 0)
    return over


def sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def silu_parts(x):
    """silu(x), its slope, and the slope's magnitude sig (1 + |x| (1 - sig))."""
    s = sigmoid(x)
    return x * s, s * (1 + x * (1 - s)), s * (1 + x.abs() * (1 - s))


# ------------------------------------------------------------- the convolution
def conv(x, weight, bias=None, state=None, flags=None, convention=ON_START, lengths=None,
         silu=True, grad_out=None, grad_final=None):
    x, w, bias, state = d64(x), d64(weight), d64(bias), d64(state)
    N, D, T = x.shape
    W = w.shape[1]
    starts, ends = starts_of(flags, convention, N, T), ends_of(lengths, N, T)
    over = over_of(flags, convention, ends, N)
    rows = torch.cat([x.new_zeros(N, D, W - 1) if state is None else state, x], 2)
    # keep[n, t, j]: input t - j is in step t's episode
    keep = torch.ones(N, T, W, dtype=torch.bool)
    for j in range(1, W):
        for t in range(T):
            keep[:, t, j] = keep[:, t, j - 1] & ~starts[:, t - j + 1] if t - j + 1 >= 0 \
                else keep[:, t, j - 1]
    live = torch.arange(T) < ends[:, None]
    zero = rows.new_zeros(())
    taps = [torch.where((keep[:, :, j] & live)[:, None], rows[:, :, W - 1 - j:W - 1 - j + T], zero)
            for j in range(W)]
    b = x.new_zeros(D) if bias is None else bias
    pre = b[:, None] + sum(w[:, W - 1 - j, None] * taps[j] for j in range(W))
    mag = b.abs()[:, None] + sum((w[:, W - 1 - j, None] * taps[j]).abs() for j in range(W))
    e_pre = (W + 2) * U * mag
    act, slope, slope_mag = silu_parts(pre) if silu else (pre, torch.ones_like(pre),
                                                          torch.ones_like(pre))
    # sigmoid: the exponent's rounding |pre| u, and 6 for exp, sum, reciprocal
    e_act = 1.1 * e_pre + (8 + 2 * pre.abs()) * U * act.abs()
    mask = live[:, None]
    r = {"out": (torch.where(mask, act, zero), torch.where(mask, e_act, zero))}
    final = x.new_zeros(N, D, W - 1)
    seen = torch.zeros(N, W - 1, dtype=torch.bool)
    for n in range(N):
        for i in range(W - 1):
            at = int(ends[n]) - (W - 1) + i
            seen[n, i] = not over[n] and not any(bool(starts[n, t]) for t in
                                                 range(max(at + 1, 0), int(ends[n])))
            if seen[n, i]:
                final[n, :, i] = rows[n, :, at + W - 1]
    r["final"] = (final, torch.zeros_like(final))
    if grad_out is None:
        return r
    go = torch.where(mask, d64(grad_out), zero)
    dpre, m_dpre = go * slope, go.abs() * slope_mag
    # the slope's own slope is below 0.5
    e_dpre = go.abs() * (0.5 * e_pre if silu else 0) + (14 + 4 * pre.abs()) * U * m_dpre
    grow = torch.zeros(3, N, D, T + W - 1, dtype=torch.float64)
    for j in range(W):
        for q, v in enumerate((dpre, m_dpre, e_dpre)):
            ww = w[:, W - 1 - j, None] if q == 0 else w[:, W - 1 - j, None].abs()
            grow[q, :, :, W - 1 - j:W - 1 - j + T] += torch.where(
                keep[:, None, :, j], ww * v, zero)
    e_grow = grow[2] + (W + 2) * U * grow[1]
    if grad_final is not None:
        gf = d64(grad_final)
        for n in range(N):
            for i in range(W - 1):
                if seen[n, i]:
                    grow[0, n, :, int(ends[n]) + i] += gf[n, :, i]
                    e_grow[n, :, int(ends[n]) + i] += 2 * U * gf[n, :, i].abs()
    r["x"] = (grow[0][:, :, W - 1:], e_grow[:, :, W - 1:])
    r["state"] = (grow[0][:, :, :W - 1], e_grow[:, :, :W - 1])
    terms = N + T + 8

    def total(v, m, e):
        return v.sum((0, 2)), e.sum((0, 2)) + terms * U * m.sum((0, 2))

    per = [total(dpre * taps[W - 1 - k], m_dpre * taps[W - 1 - k].abs(),
                 e_dpre * taps[W - 1 - k].abs()) for k in range(W)]
    r["weight"] = (torch.stack([p[0] for p in per], 1), torch.stack([p[1] for p in per], 1))
    r["bias"] = total(dpre, m_dpre, e_dpre)
    return r


# -------------------------------------------------------------------- the scan
def scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, state=None, flags=None,
         convention=ON_START, lengths=None, softplus=True, grad_y=None, grad_final=None):
    u, delta, A, B, C, z, h0 = (d64(t) for t in (u, delta, A, B, C, z, state))
    N, ch, T = u.shape
    S = A.shape[1]
    if B.dim() == 3:
        B, C = B[:, None], C[:, None]
    G = B.shape[1]
    Bs, Cs = (v.repeat_interleave(ch // G, 1) for v in (B, C))  # [N, ch, S, T]
    skip = u.new_zeros(ch) if D is None else d64(D)
    raw = delta + (0 if delta_bias is None else d64(delta_bias)[:, None])
    zero = u.new_zeros(())
    starts, ends = starts_of(flags, convention, N, T), ends_of(lengths, N, T)
    over = over_of(flags, convention, ends, N)
    live = (torch.arange(T) < ends[:, None])[:, None]  # [N, 1, T]
    dt = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    dt, um = torch.where(live, dt, zero), torch.where(live, u, zero)
    r_dt = (12 if softplus else 0) + raw.abs() + 1  # dt's relative error / u
    Bs, Cs = torch.where(live[:, :, None], Bs, zero), torch.where(live[:, :, None], Cs, zero)
    x = dt[:, :, None] * A[:, :, None]
    a = torch.exp(x)
    a = torch.where(starts[:, None, None, :T] & live[:, :, None], zero, a)
    r_a = 4 + x.abs() * (r_dt[:, :, None] + 4)
    b = (dt * um)[:, :, None] * Bs
    h = u.new_zeros(N, ch, S, T + 1)  # h[..., t + 1] after step t
    m, e = torch.zeros_like(h), torch.zeros_like(h)
    if h0 is not None:
        h[..., 0], m[..., 0] = h0, h0.abs()
    for t in range(T):
        at = a[..., t]
        h[..., t + 1] = torch.where(at == 0, zero, at * h[..., t]) + b[..., t]
        m[..., t + 1] = at * m[..., t] + b[..., t].abs()
        e[..., t + 1] = at * e[..., t] + at * m[..., t] * r_a[..., t] * U \
            + (r_dt[:, :, None, t] + 4) * U * b[..., t].abs() + 4 * U * m[..., t + 1]
    hp, mp, ep = h[..., :T], m[..., :T], e[..., :T]
    h, m, e = h[..., 1:], m[..., 1:], e[..., 1:]
    y0 = (Cs * h).sum(2) + skip[:, None] * um
    m_y0 = (Cs.abs() * m).sum(2) + (skip[:, None] * um).abs()
    e_y0 = (Cs.abs() * e).sum(2) + (S + 4) * U * m_y0
    if z is None:
        gate, gate_slope, m_slope, r_gate = (torch.ones_like(u), None, None, zero)
    else:
        gate, gate_slope, m_slope = silu_parts(z)
        r_gate = 10 + 2 * z.abs()
    r = {"y": (torch.where(live, y0 * gate, zero),
               torch.where(live, (e_y0 + r_gate * U * m_y0) * gate.abs(), zero))}
    last, last_e = (h[..., -1], e[..., -1]) if T else (
        torch.zeros(N, ch, S, dtype=torch.float64) if h0 is None else h0,
        torch.zeros(N, ch, S, dtype=torch.float64))
    stop = over[:, None, None]
    r["final"] = (torch.where(stop, zero, last), torch.where(stop, zero, last_e))
    if grad_y is None:
        return r
    go = torch.where(live, d64(grad_y), zero)
    gy = go * gate
    e_gy = r_gate * U * gy.abs()
    g = u.new_zeros(N, ch, S, T)
    mg, eg = torch.zeros_like(g), torch.zeros_like(g)
    right = [u.new_zeros(N, ch, S) for _ in range(3)]  # a g, its magnitude and error
    if grad_final is not None:
        gf = torch.where(stop, zero, d64(grad_final))
        right[0], right[1] = gf, gf.abs()
    for t in reversed(range(T)):
        own = Cs[..., t] * gy[:, :, None, t]
        g[..., t] = own + right[0]
        mg[..., t] = own.abs() + right[1]
        eg[..., t] = Cs[..., t].abs() * e_gy[:, :, None, t] + U * own.abs() + right[2] \
            + 4 * U * mg[..., t]
        at = a[..., t]
        right = [torch.where(at == 0, zero, at * g[..., t]), at * mg[..., t],
                 at * eg[..., t] + r_a[..., t] * U * at * mg[..., t]]
    r["state"] = (right[0], right[2] + 2 * U * right[1])
    w = torch.where(a == 0, zero, a * hp)
    mw, ew = a * mp, a * ep + (r_a + 1) * U * a * mp
    q, mq = g * w, mg * mw
    eq = eg * mw + mg * ew + 2 * U * mq
    gB = (g * Bs).sum(2)
    m_gB = (mg * Bs.abs()).sum(2)
    e_gB = (eg * Bs.abs()).sum(2) + (S + 2) * U * m_gB
    Ad = A[None, :, :, None]
    gdt = (q * Ad).sum(2) + um * gB
    m_gdt = (mq * Ad.abs()).sum(2) + um.abs() * m_gB
    e_gdt = (eq * Ad.abs()).sum(2) + um.abs() * e_gB + (S + 6) * U * m_gdt
    if softplus:
        s = sigmoid(raw)
        gdt, m_gdt = gdt * s, m_gdt * s
        e_gdt = e_gdt * s + (10 + 2 * raw.abs()) * U * m_gdt
    gdt, m_gdt, e_gdt = (torch.where(live, v, zero) for v in (gdt, m_gdt, e_gdt))
    r["delta"] = (gdt, e_gdt)
    m_gu = dt.abs() * m_gB + (skip[:, None] * gy).abs()
    r["u"] = (torch.where(live, dt * gB + skip[:, None] * gy, zero), torch.where(
        live, dt.abs() * (e_gB + r_dt * U * m_gB) + skip.abs()[:, None] * e_gy + 4 * U * m_gu,
        zero))
    terms = N + T + 8

    def total(v, mm, ee, dims):
        return v.sum(dims), ee.sum(dims) + terms * U * mm.sum(dims)

    dts = dt[:, :, None]
    r["A"] = total(q * dts, mq * dts.abs(),
                   eq * dts.abs() + r_dt[:, :, None] * U * mq * dts.abs(), (0, 3))
    r["D"] = total(gy * um, (gy * um).abs(), e_gy * um.abs(), (0, 2))
    r["delta_bias"] = total(gdt, m_gdt, e_gdt, (0, 2))
    du = (dt * um)[:, :, None]

    def groups(v, mm, ee):
        v, mm, ee = (k.view(N, G, ch // G, S, T).sum(2) for k in (v, mm, ee))
        return v, ee + (ch // G + 8) * U * mm

    r["B"] = groups(g * du, mg * du.abs(), eg * du.abs() + (r_dt[:, :, None] + 4) * U * mg
                    * du.abs())
    gys = gy[:, :, None]
    r["C"] = groups(h * gys, m * gys.abs(), e * gys.abs() + m * e_gy[:, :, None])
    if z is not None:
        r["z"] = (go * y0 * gate_slope, go.abs() * (e_y0 * m_slope + (16 + 4 * z.abs()) * U * m_y0
                                                    * m_slope))
    return r


# ---------------------------------------------------------------- the clipping
def clip(grads, max_norm, eps):
    """norm, and each tensor scaled; the scale rounds once to float32 and the
    product once."""
    norm = sum(float((d64(g) ** 2).sum()) for g in grads) ** 0.5
    scale = 1.0 if norm == 0 else min(1.0, max_norm / (norm + eps))
    return norm, [(d64(g) * scale, 3 * U * (d64(g) * scale).abs()) for g in grads]
