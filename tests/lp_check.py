"""Plain fp64 forms of the log-probability operators and the tolerances their
kernels are held to.

Error budget of the kernels (fp32 arithmetic, u = 2^-24 the half step of one
rounding, relative):

* an exponential 2^a of the statistics: the hardware's error (2 units in the
  last place, taken as 2^-21) and the rounding of a (a difference, a product
  with a rounded constant: 3 u |a| absolute, times ln 2);
* a sum of V such terms: every thread adds its share one after the other and
  the partial sums are merged, V / 256 + 64 additions at most: that many u.
  ``delta`` is the relative error of the sum d that follows;
* log p = -(log d + (M - x) / T): delta, and 6 u of its value and of 1;
* H = log d - u / d: 4 delta (1 + H), since both parts are at most 1 + H + the
  sum of the terms' own |a| errors, which delta's second part covers;
* p_c: delta and the exponent's rounding, 4 u (|log2 p_c| + |log2 d|).
A result is rounded once to its type: half a step, finfo.eps / 2 of the value,
and for fp16 half its subnormal spacing, 2^-25. Results below 2^-126 are
flushed to 0."""
from __future__ import annotations

import torch

U = 2.0 ** -24


def rows_ref(x, target, temperature=1.0, ignore_index=-100):
    """fp64 (valid, logq [n, V], logp [n], entropy [n])."""
    z = x.double() / temperature
    m = z.amax(1, keepdim=True)
    logq = z - m - (z - m).exp().sum(1, keepdim=True).log()
    t = target.long()
    valid = (t != ignore_index) & (t >= 0) & (t < x.shape[1])
    logp = logq.gather(1, torch.where(valid, t, 0)[:, None])[:, 0]
    p = logq.exp()
    h = -torch.where(p > 0, p * logq, torch.where(logq.isnan(), logq, 0.0)).sum(1)
    return valid, logq, torch.where(valid, logp, 0.0), torch.where(valid, h, 0.0)


def others(p, rows, cols):
    """1 - p_t as the sum of the other columns: the subtraction from 1 would lose it in fp64 too where p_t is near 1."""
    p = p[rows]
    p[torch.arange(len(rows), device=p.device), cols] = 0.0
    return p.sum(1)


def grad_ref(logq, valid, target, g, h, temperature=1.0):
    """(1/T) [g (onehot - p) - h p (log p + H)] of every row, fp64; 0 on rows that are not valid."""
    p = logq.exp()
    plogp = torch.where(p > 0, p * logq, 0.0)
    ent = -plogp.sum(1, keepdim=True)
    g = torch.where(valid, g.double(), 0.0)[:, None]
    h = torch.where(valid, h.double(), 0.0)[:, None]
    q = -p
    rows = valid.nonzero().flatten()
    cols = target.long()[rows]
    q[rows, cols] = others(p, rows, cols)
    out = g * q - torch.where(h != 0, h * (plogp + p * ent), 0.0)
    out[~valid] = 0.0
    return out / temperature


def delta(x, temperature=1.0):
    """Relative error of a row's exp-sum [n]: sum over p_c of the exponential's error, and the additions."""
    z = x.double() / temperature
    a = (z - z.amax(1, keepdim=True)).clamp_min(-1e4)
    q = torch.softmax(a, 1)
    return (q * (2.0 ** -21 + 3 * U * a.abs())).sum(1) + (x.shape[1] / 256 + 64) * U


def tol_logp(d, logp):
    return d + 6 * U * (1 + logp.abs())


def tol_entropy(d, h):
    return 4 * d * (1 + h)


def tol_grad(x, ref, logq, valid, target, g, h, dg, dh, dtype, temperature=1.0):
    """Elementwise tolerance of the gradient. dg: the error of g [n] itself (dh of h)."""
    d = delta(x, temperature)[:, None]
    p = logq.exp()
    lp = logq.clamp_min(-1e4).abs()
    plogp = torch.where(p > 0, p * lp, 0.0)
    ent = plogp.sum(1, keepdim=True)
    g, h = g.double().abs()[:, None], h.double().abs()[:, None]
    dg, dh = dg.double().abs()[:, None], dh.double().abs()[:, None]
    q = p.clone()
    rows = valid.nonzero().flatten()
    cols = target.long()[rows]
    q[rows, cols] = others(p, rows, cols)
    size = g * q + h * (plogp + p * ent)
    rel = 2 * d + 8 * U * (1 + lp / 0.69 + logq.amax(1, keepdim=True).abs() / 0.69)
    own = dg * q + dh * (plogp + p * ent)
    own = own + h * p * (4 * d * (1 + ent) + 8 * U * (lp + ent))  # H and log p inside the entropy's part
    tol = (size * rel + own) / temperature * 1.01 + torch.finfo(dtype).eps / 2 * ref.abs()
    # flushed exponentials, and fp16's subnormals
    tol = tol + (g + h * 200) / temperature * 2.0 ** -125 + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -149)
    tol[~valid] = 0.0
    return tol


def policy_ref(x, target, adv, old, ref, weight, lo, hi, kl_coef, ent_coef, temperature, reduction, up,
               ignore_index=-100):
    """fp64 policy loss: dict with loss, grad, stats and their tolerances."""
    valid, logq, logp, ent = rows_ref(x, target, temperature, ignore_index)
    n = x.shape[0]
    one = torch.ones(n, dtype=torch.float64, device=x.device)
    w = one if weight is None else torch.where(valid, weight.double(), 0.0)
    live = valid & (w != 0)
    w = torch.where(live, w, 0.0)
    a = torch.where(live, adv.double(), 0.0)
    o = logp if old is None else torch.where(live, old.double(), 0.0)
    lp = torch.where(live, logp, 0.0)
    r = torch.where(live, (lp - o).exp(), 1.0)
    u1, u2 = -a * r, -a * r.clamp(1 - lo, 1 + hi)
    loss = torch.maximum(u1, u2)
    slope = torch.where(u1 >= u2, u1, 0.0)
    kl = torch.zeros_like(loss)
    d = delta(x, temperature)
    tl = torch.where(live, tol_logp(d, lp), 0.0)
    te = torch.where(live, tol_entropy(d, ent), 0.0)
    tr = r * (1.01 * tl + 2.0 ** -21)
    dslope = a.abs() * tr
    dloss = a.abs() * tr + 4 * U * loss.abs()
    dkl = torch.zeros_like(kl)
    if ref is not None:
        gap = torch.where(live, ref.double() - lp, 0.0)
        kl = gap.exp() - gap - 1
        eg = gap.exp()
        dkl = (1 - eg).abs() * 1.01 * tl + 2 * eg * tl ** 2 + 2.0 ** -20 * (eg + gap.abs())
        dkl = torch.where(gap.abs() < 0.24, (1 - eg).abs() * 1.01 * tl + tl ** 2 + 2.0 ** -20 * kl + 4 * U * gap.abs() * tl, dkl)
        loss = loss + kl_coef * kl
        slope = slope + kl_coef * (1 - eg)
        dslope = dslope + kl_coef * (1.01 * eg * tl + 2.0 ** -21 * (1 - eg).abs()) + 4 * U * slope.abs()
        dloss = dloss + kl_coef * dkl
    loss = loss - ent_coef * ent
    dloss = dloss + abs(ent_coef) * te + 8 * U * (loss.abs() + abs(ent_coef) * ent)
    total = w.sum() if reduction == "mean" else torch.ones((), dtype=torch.float64, device=x.device)
    inv = 1 / total if float(total) != 0 else total * 0
    upv = torch.ones(1, dtype=torch.float64, device=x.device) if up is None else up.double()
    row = torch.where(live, w * loss, 0.0)
    drow = torch.where(live, w.abs() * dloss + 2 * U * row.abs(), 0.0)
    if reduction == "none":
        out, dout = row, drow
    else:
        out, dout = (row.sum() * inv).reshape(1), (drow.sum() * inv.abs()).reshape(1)
        dout = dout + 4 * U * out.abs()
    scale = w * inv * upv
    g, h = slope * scale, -ent_coef * scale
    dg = dslope * scale.abs() + 6 * U * g.abs()
    grad = grad_ref(logq, live, target, g, h, temperature)
    tg = tol_grad(x, grad, logq, live, target, g, h, dg, 4 * U * h.abs(), x.dtype, temperature)
    stats = torch.stack([torch.where(live, logp, 0.0), torch.where(live, ent, 0.0), torch.where(live, r, 0.0),
                         torch.where(live, kl, 0.0)], 1)
    tstats = torch.stack([tl, te, torch.where(live, tr, 0.0), torch.where(live, dkl, 0.0)], 1)
    tstats = tstats + 2 * U * stats.abs()
    return dict(loss=out, tol_loss=dout, grad=grad, tol_grad=tg, stats=stats, tol_stats=tstats, live=live)


def pair_losses(h, kind, beta, eps):
    """Loss and slope of h [P], fp64."""
    z = beta * h
    if kind == "sigmoid":
        sp = torch.nn.functional.softplus
        return ((1 - eps) * sp(-z) + eps * sp(z),
                beta * (eps * torch.sigmoid(z) - (1 - eps) * torch.sigmoid(-z)))
    if kind == "hinge":
        return (1 - z).clamp_min(0.0), torch.where(z < 1, torch.full_like(z, -beta), 0.0)
    m = h - 0.5 / beta
    return m * m, 2 * m


def preference_ref(x, target, offsets, ref, kind, beta, eps, normalize, reduction, up, ignore_index=-100):
    """fp64 preference loss: dict with loss, seq, grad and their tolerances."""
    valid, logq, logp, _ = rows_ref(x, target, 1.0, ignore_index)
    off = offsets.long().tolist()
    pairs, dev = len(off) // 2, x.device
    d = delta(x, 1.0)
    tl = torch.where(valid, tol_logp(d, logp), 0.0)
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    s, n, ds = [], [], []
    for b, e in zip(off[:-1], off[1:]):
        s.append(logp[b:e].sum() if e > b else zero)
        n.append(valid[b:e].sum().double() if e > b else zero)
        ds.append((tl[b:e] + U * logp[b:e].abs()).sum() if e > b else zero)
    stack = lambda v: torch.stack(v) if v else torch.zeros(0, dtype=torch.float64, device=dev)  # noqa: E731
    s, n, ds = stack(s), stack(n), stack(ds)
    if normalize:
        s, ds = s / n.clamp_min(1), ds / n.clamp_min(1)
    h = s[:pairs] - s[pairs:]
    dh = ds[:pairs] + ds[pairs:]
    if ref is not None:
        h = h - (ref[:pairs].double() - ref[pairs:].double())
    live = (n[:pairs] > 0) & (n[pairs:] > 0)
    loss, slope = pair_losses(h, kind, beta, eps)
    loss, slope = torch.where(live, loss, 0.0), torch.where(live, slope, 0.0)
    curve = {"sigmoid": beta * beta / 4, "hinge": 0.0, "squared": 2.0}[kind]
    dslope = curve * dh
    dloss = slope.abs() * dh + curve * dh ** 2
    upv = torch.ones(1, dtype=torch.float64, device=dev) if up is None else up.double()
    count = live.sum().double()
    inv = 1.0
    if reduction == "mean":
        inv = float(1 / count) if float(count) else 0.0
    out = loss if reduction == "none" else (loss.sum() * inv).reshape(1)
    dout = dloss if reduction == "none" else (dloss.sum() * inv).reshape(1)
    slope, dslope = slope * inv * upv, dslope * inv * upv.abs()
    g, dg = torch.zeros(x.shape[0], dtype=torch.float64, device=dev), torch.zeros(x.shape[0], dtype=torch.float64, device=dev)
    used = torch.zeros(x.shape[0], dtype=torch.bool, device=dev)
    for j, (b, e) in enumerate(zip(off[:-1], off[1:])):
        c = slope[j % pairs] * (1 if j < pairs else -1)
        dc = dslope[j % pairs]
        if normalize and float(n[j]) > 0:
            c, dc = c / n[j], dc / n[j]
        if live[j % pairs]:
            g[b:e], dg[b:e] = c, dc + 4 * U * c.abs()
            used[b:e] = True
    use = valid & used
    g, dg = torch.where(use, g, 0.0), torch.where(use, dg, 0.0)
    z = torch.zeros_like(g)
    grad = grad_ref(logq, use, target, g, z)
    tg = tol_grad(x, grad, logq, use, target, g, z, dg, z, x.dtype)
    return dict(loss=out, tol_loss=dout + 4 * U * out.abs(), seq=s, tol_seq=ds + 2 * U * s.abs(), grad=grad,
                tol_grad=tg)


def check(got, want, tol, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} for {tuple(want.shape)}"
    same = (got == want) | (got.isnan() & want.isnan())
    over = ~same & ~((got - want).abs() <= tol)
    if over.any():
        i = int(((got - want).abs() / tol.clamp_min(1e-300)).masked_fill(~over, -1.0).flatten().nan_to_num(1e300).argmax())
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} off; worst at {i}: "
                             f"{float(got.flatten()[i])!r} for {float(want.flatten()[i])!r}, "
                             f"tolerance {float(tol.expand_as(want).flatten()[i]):.3e}")
