"""Plain fp64 forms of the 8-bit serving head's operators and the tolerances
their kernels are held to (u = 2^-24, half a step of fp32).

* Norm and quantising. h = x + r is rounded once (u), the sum of H squares adds
  up at most 32 values a thread one after the other and then 10 levels of lanes
  and warps (42 u, half of it on the root), and the mean, the root, two
  divisions, and four products round once each: a value v = y / scale is
  (1 + 21 + 8) u off before it is rounded to e4m3, taken as 2^-19 of it. The
  rounding is to the nearest e4m3: the byte lies between those of v (1 - 2^-19)
  and v (1 + 2^-19). A scale is off by 2^-19 too. residual_out: the sum's u and
  half a step of its type.
* Product. With S = sum |a b| over the row and column (scales in), the tensor core
  adds 128 products in 4 instructions, which cut off what lies under their
  largest term's last place: 16 u of the block's S are granted it. The scales'
  product, the addition to the running sum of up to ceil(K / 128) blocks and the
  bias round to nearest: (ceil(K / 128) + 3) u. Then half a step of the output's type.
* Verification. A probability: an exponential (2^-21) of an exponent that is a
  difference, times a rounded constant (3 u |a| ln 2, a = log2 of it), over a sum of
  such terms, V / 256 + 64 additions in a row at most: rel(V). The decision
  (in logarithms) and the place of the drawn token are checked against the fp64
  probabilities with that room on both sides; a log-probability is off by rel(V), and 6 u of its
  parts |x - M| / T and log s."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
BLOCK, TOP, MIN_SCALE = 128, 448.0, 2.0 ** -126
SLACK = 2.0 ** -19
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


# ---------------------------------------------------------------------- 8-bit blocks
def block_scales(y, tall=1):
    """fp64 scales of blocks of `tall` rows and 128 columns, by a loop over the blocks."""
    rows, cols = y.shape
    out = torch.empty(-(-rows // tall), -(-cols // BLOCK), dtype=torch.float64, device=y.device)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            t = y[i * tall:(i + 1) * tall, j * BLOCK:(j + 1) * BLOCK].abs()
            out[i, j] = t.max() / TOP if not t.isnan().any() else float("nan")
    return out.clamp_min(MIN_SCALE)


def spread(scale, rows, cols, tall=1):
    return scale.double().repeat_interleave(tall, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def e4m3(x):
    """fp64 values of the nearest e4m3 (ties to even), saturated."""
    return x.clamp(-TOP, TOP).float().to(torch.float8_e4m3fn).double()


def check_blocks(q, scale, y, tall=1, slack=SLACK):
    """q and scale are the 8-bit form of fp64 y."""
    want = block_scales(y, tall)
    assert scale.shape == want.shape and scale.dtype == torch.float32
    assert ((scale.double() - want).abs() <= slack * want).all()
    v = y / spread(want, *y.shape, tall)
    lo, hi = e4m3(v - slack * v.abs()), e4m3(v + slack * v.abs())
    got = q.double()
    assert ((got >= lo) & (got <= hi)).all()
    # zeros stay zeros, and a block of them has the least scale
    assert (got[y == 0] == 0).all()


def rows8(q):
    """Strides of an 8-bit matrix."""
    assert q.dtype == torch.float8_e4m3fn and q.stride(1) == 1 and q.data_ptr() % 16 == 0
    assert q.shape[0] < 2 or q.stride(0) % 16 == 0


def norm_ref(x, weight, residual, eps):
    """fp64 (h, y)."""
    h = x.double() if residual is None else x.double() + residual.double()
    return h, h / ((h * h).mean(1, keepdim=True) + eps).sqrt() * weight.double()


# ---------------------------------------------------------------------- product
def gemm_ref(a, sa, b, sb, bias=None):
    """fp64 (D, S)."""
    x = a.double() * spread(sa, *a.shape)
    w = b.double() * spread(sb, *b.shape, BLOCK)
    d = x @ w.t()
    return (d if bias is None else d + bias.double()), x.abs() @ w.abs().t()


def check_gemm(out, a, sa, b, sb, bias=None):
    d, s = gemm_ref(a, sa, b, sb, bias)
    blocks = sa.shape[1]
    tol = s * (16 + blocks + 3) * U + d.abs() * HALF[out.dtype] * (1 + 2.0 ** -10) + (d.abs() + s) * U
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert ((out.double() - d).abs() <= tol).all(), float(((out.double() - d).abs() / tol).max())


# ---------------------------------------------------------------------- verification
def rel(vocab, amax=64.0):
    return 2.0 ** -21 + 3 * U * amax * 0.6931 + (vocab / 256 + 64) * U


def softmax(z, t):
    return torch.softmax(z.double() / (float(t) if t else 1.0), -1)


def logs(z, y, d, u, t):
    """fp64 (log p, log q, log u) of draft d."""
    lp = float(torch.log_softmax(z.double() / (t or 1.0), 0)[d])
    lq = 0.0 if y is None else float(torch.log_softmax(y.double() / (t or 1.0), 0)[d])
    return lp, lq, math.log(u) if u > 0 else -math.inf


def stays_by(z, y, d, u, t):
    """By how much log u + log q lies below log p (above 0: the draft stays)."""
    lp, lq, lu = logs(z, y, d, u, t)
    return -math.inf if lp == -math.inf else lp - lq - lu


def room_by(z, y, d, u, t):
    """What rounding may make of it: rel(V) in either sum, and 8 u of the logarithms' own parts."""
    size = sum(abs(v) for v in logs(z, y, d, u, t) if math.isfinite(v))
    return 4 * rel(z.shape[0]) + 8 * U * (size + 64)


def check_sequence(z, y, draft, u, r, t, accepted, tokens, logp):
    """One sequence's answer (lists) against fp64: z [K + 1, V], y [K, V] or None, draft [K]."""
    K, V = z.shape[0] - 1, z.shape[1]
    assert 0 <= accepted <= K and len(tokens) == len(logp) == K + 1
    e = rel(V)
    for i in range(K + 1):
        if i > accepted:
            assert tokens[i] == -1 and logp[i] == 0
            continue
        has = i < K and 0 <= draft[i] < V
        p = softmax(z[i], t)
        q = None
        if has:
            if y is None:
                q = torch.zeros_like(p)
                q[draft[i]] = 1.0
            else:
                q = softmax(y[i], t)
        best = int((z[i] == z[i].max()).nonzero()[0])
        if i < accepted:
            assert has and tokens[i] == draft[i]
            if t == 0:
                assert draft[i] == best
            else:
                assert stays_by(z[i], None if y is None else y[i], draft[i], u[i], t) > -room_by(z[i], None if y is None else y[i], draft[i], u[i], t)
        else:
            if has:
                if t == 0:
                    assert draft[i] != best
                else:
                    assert stays_by(z[i], None if y is None else y[i], draft[i], u[i], t) < room_by(z[i], None if y is None else y[i], draft[i], u[i], t)
            tok = tokens[i]
            assert 0 <= tok < V
            if t == 0:
                assert tok == best
            else:
                w = (p - q).clamp_min(0) if has else p
                room = 4 * e * (2.0 if has else 1.0)

                def drawn(w):
                    total, upto = float(w.sum()), w.cumsum(0)
                    below = float(upto[tok - 1]) if tok else 0.0
                    return (below <= r * total + room and float(upto[tok]) >= r * total - room
                            and (float(w[tok]) > 0 or room >= float(p[tok]) * 1e-3))
                if has and float(w.sum()) <= room:
                    # max(p - q, 0) adds up to less than what the roundings of p and q may be, e (p + q) in a term:
                    # where fp32 finds nothing left the draw is p's, else one of the terms that are above 0 within
                    # those roundings (a sum of true terms may well be as small as this)
                    assert drawn(p) or float(p[tok] - q[tok]) > -e * float(p[tok] + q[tok])
                else:
                    assert drawn(w)
        x = z[i].double()
        s = float((x[x > -float("inf")].max() - x[tokens[i]]) / (t or 1.0)) if tokens[i] >= 0 else 0.0
        want = float(torch.log_softmax(x / (float(t) if t else 1.0), 0)[tokens[i]])
        tol = rel(V, 0.0) + 6 * U * (abs(want) + 2 * s + 13)
        assert abs(logp[i] - want) <= tol, (logp[i], want, tol)


def check_verify(z, y, draft, u, r, temps, got):
    accepted, tokens, logp = (v.cpu() for v in got)
    assert accepted.dtype == torch.int32 and tokens.dtype == draft.dtype and logp.dtype == torch.float32
    for b in range(z.shape[0]):
        t = float(temps[b]) if torch.is_tensor(temps) else float(torch.tensor(temps, dtype=torch.float32))
        check_sequence(z[b], None if y is None else y[b], draft[b].tolist(), u[b].tolist(), float(r[b]), t,
                       int(accepted[b]), tokens[b].tolist(), logp[b].tolist())
