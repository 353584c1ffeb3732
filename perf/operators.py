"""Cases that measure the log-probability operators: token log-probabilities
with their gradient, the clipped policy loss, the paired preference loss and
the log-probabilities of a linear head, each beside its plain form.

The plain forms are elementary torch operations in fp32 (row-level scalars in
fp64); ``exact`` holds the definitions in fp64, with the gradients taken by
differentiation instead of from a formula.
"""
from __future__ import annotations

import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # scoring one step of eight sequences while they are sampled: the smallest call
        dict(name="logprob_step", op="logprob", rows=8, vocab=128256, pad=0, masked=0, dtype="bf16", temperature=0.7,
             entropy=True, backward=False, ignored=0.0, int32=False),
        # scoring a batch of rollouts under the old or the reference policy
        dict(name="logprob_score", op="logprob", rows=8192, vocab=128256, pad=0, masked=0, dtype="bf16",
             temperature=1.0, entropy=True, backward=False, ignored=0.05, int32=False),
        # a loss of the user's own over the log-probabilities: forward and backward, odd rows
        dict(name="logprob_train", op="logprob", rows=2049, vocab=50257, pad=0, masked=0, dtype="f32",
             temperature=1.0, entropy=True, backward=True, ignored=0.25, int32=True),
        # a micro-step of a small policy
        dict(name="policy_small", op="policy", rows=64, vocab=32000, pad=0, masked=0, dtype="f16", temperature=1.0,
             clip_low=0.2, clip_high=0.2, kl=0.04, entropy=0.0, ref=True, weighted=False, reduction="mean",
             scale=4096.0, ignored=0.1, int32=False),
        # the step of a large-vocabulary policy over a batch of rollouts, prompts masked
        dict(name="policy_step", op="policy", rows=8192, vocab=128256, pad=0, masked=0, dtype="bf16", temperature=1.0,
             clip_low=0.2, clip_high=0.28, kl=0.04, entropy=0.001, ref=True, weighted=True, reduction="mean",
             scale=1.0, ignored=0.3, int32=False),
        # ragged rows in a wider buffer, vocabulary padding masked, summed for accumulation over micro-batches
        dict(name="policy_ragged", op="policy", rows=2500, vocab=50257, pad=3, masked=0, dtype="bf16",
             temperature=0.9, clip_low=0.1, clip_high=0.3, kl=0.1, entropy=0.01, ref=True, weighted=False,
             reduction="sum", scale=0.01, ignored=0.2, int32=True),
        # a few short pairs
        dict(name="preference_small", op="preference", pairs=4, length=48, vocab=32000, pad=0, masked=0, dtype="bf16",
             kind="sigmoid", beta=0.1, smoothing=0.0, normalize=False, ref=True, scale=1.0, ignored=0.2, int32=False),
        # a batch of long pairs at a large vocabulary
        dict(name="preference_step", op="preference", pairs=8, length=512, vocab=128256, pad=0, masked=0,
             dtype="bf16", kind="sigmoid", beta=0.1, smoothing=0.1, normalize=False, ref=True, scale=1.0,
             ignored=0.3, int32=False),
        # length-normalised, without a reference, odd vocabulary with masked padding columns
        dict(name="preference_norm", op="preference", pairs=6, length=150, vocab=50257, pad=7, masked=20, dtype="f16",
             kind="hinge", beta=2.0, smoothing=0.0, normalize=True, ref=False, scale=512.0, ignored=0.25, int32=True),
        # log-probabilities of four tokens straight from the hidden states
        dict(name="linear_step", op="linear", rows=4, hidden=4096, vocab=128256, bias=False, temperature=1.0,
             entropy=True, backward=False, ignored=0.0),
        # scoring rollouts from the hidden states, no logits in memory
        dict(name="linear_score", op="linear", rows=4096, hidden=4096, vocab=128256, bias=False, temperature=0.8,
             entropy=True, backward=False, ignored=0.3),
        # training through the linear head, biased, rows not a multiple of a tile
        dict(name="linear_train", op="linear", rows=2000, hidden=2048, vocab=64000, bias=True, temperature=1.0,
             entropy=True, backward=True, ignored=0.25),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprob", "policy", "preference", "linear"])
    if op == "linear":
        hidden, vocab = 8 * _log_int(rng, 32, 640), 8 * _log_int(rng, 125, 16032)
        rows = _log_int(rng, 1, max(1, min(4096, 2 * 10 ** 12 // (hidden * vocab))))
        return dict(op=op, rows=rows, hidden=hidden, vocab=vocab, bias=rng.random() < 0.5,
                    temperature=rng.choice([1.0, 0.7, 1.3]), entropy=rng.random() < 0.7,
                    backward=rng.random() < 0.5 and rows * hidden * vocab < 3 * 10 ** 11, ignored=rng.choice([0.0, 0.2, 0.5]))
    vocab = _log_int(rng, 1000, 256000)
    case = dict(op=op, vocab=vocab, pad=rng.choice([0, 0, 1, 5, 8]), masked=rng.choice([0, 0, 17]),
                dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), ignored=rng.choice([0.0, 0.1, 0.4]),
                int32=rng.random() < 0.5)
    most = 8192 * 128256 // 2 // (vocab * SIZES[case["dtype"]])
    scale = 1024.0 if case["dtype"] == "f16" else rng.choice([1.0, 0.37])
    if op == "preference":
        length = _log_int(rng, 4, 700)
        pairs = _log_int(rng, 1, max(1, min(64, most // (2 * length))))
        return case | dict(pairs=pairs, length=length, kind=rng.choice(["sigmoid", "hinge", "squared"]),
                           beta=rng.choice([0.05, 0.1, 0.5]), smoothing=rng.choice([0.0, 0.1]),
                           normalize=rng.random() < 0.4, ref=rng.random() < 0.7, scale=scale)
    case["rows"] = _log_int(rng, 1, max(1, min(8192, most)))
    case["temperature"] = rng.choice([1.0, 1.0, 0.6, 1.4])
    if op == "logprob":
        return case | dict(entropy=rng.random() < 0.6, backward=rng.random() < 0.6)
    return case | dict(clip_low=rng.choice([0.1, 0.2]), clip_high=rng.choice([0.2, 0.28]), kl=rng.choice([0.0, 0.05]),
                       entropy=rng.choice([0.0, 0.01]), ref=True, weighted=rng.random() < 0.5,
                       reduction=rng.choice(["mean", "sum", "none"]), scale=scale)


def _valid_rows(case):
    n = _rows(case)
    return n - int(case["ignored"] * n)


def _rows(case):
    return 2 * case["pairs"] * case["length"] if case["op"] == "preference" else case["rows"]


# ---------------------------------------------------------------------- inputs
def _targets(n, vocab, ignored, gen, int32):
    t = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    drop = int(ignored * n)
    if drop:
        t[torch.randperm(n, generator=gen, device="cuda")[:drop]] = IGNORE
    return t.to(torch.int32) if int32 else t


def _logits(n, case, target, gen):
    """Rows like a language model's: a wide base, a few raised columns, and on most rows a raised target."""
    vocab, live = case["vocab"], case["vocab"] - case["masked"]
    x = torch.empty(n, vocab + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda").normal_(0.0, 2.0, generator=gen)
    x = x[:, :vocab]
    rows = torch.arange(n, device="cuda")
    columns = torch.randint(0, live, (n, 4), generator=gen, device="cuda")
    x.scatter_(1, columns, (7.0 + 6.0 * torch.rand(n, 4, generator=gen, device="cuda")).to(x.dtype))
    lift = 14.0 * torch.rand(n, generator=gen, device="cuda") - 1.0
    x[rows, target.long().clamp(0, live - 1)] = lift.to(x.dtype)
    if case["masked"]:
        x[:, live:] = -math.inf
    return x


def _logp_of(x, target, temperature, bias=None):
    """fp32 log-probabilities for making inputs, block by block."""
    out = torch.zeros(x.shape[0], device="cuda")
    for r in range(0, x.shape[0], 1024):
        z = x[r:r + 1024].float() / temperature
        out[r:r + 1024] = z.gather(1, target[r:r + 1024].long().clamp_min(0)[:, None])[:, 0] - torch.logsumexp(z, 1)
    return torch.where(target >= 0, out, torch.zeros_like(out))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, vocab = _rows(case), case["vocab"]
    state = dict(case=case)
    if case["op"] == "linear":
        hidden = case["hidden"]
        state["target"] = _targets(n, vocab, case["ignored"], gen, False)
        state["weight"] = torch.empty(vocab, hidden, dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.02, generator=gen)
        # hidden states lean towards their target's weight row, so log-probabilities are spread
        lean = state["weight"][state["target"].clamp_min(0)].float()
        lean *= (28.0 * torch.rand(n, 1, generator=gen, device="cuda") - 2.0) / lean.norm(dim=1, keepdim=True) ** 2
        base = torch.empty(n, hidden, device="cuda").normal_(0.0, 100.0 / math.sqrt(hidden), generator=gen)
        state["hidden"] = (base + lean * 0.5).to(torch.bfloat16)
        state["bias"] = None
        if case["bias"]:
            state["bias"] = torch.empty(vocab, dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.5, generator=gen)
    else:
        live = dict(case, vocab=vocab - case["masked"])
        state["target"] = _targets(n, live["vocab"], case["ignored"], gen, case["int32"])
        state["logits"] = _logits(n, case, state["target"], gen)
    if case.get("backward"):
        state["grad_logp"] = torch.randn(n, generator=gen, device="cuda") / n
        state["grad_entropy"] = torch.randn(n, generator=gen, device="cuda") * 0.1 / n if case["entropy"] else None
    if case["op"] == "policy":
        logp = _logp_of(state["logits"], state["target"], case["temperature"])
        # the ratio to the old policy keeps off the clip borders, where either branch is right
        shift = torch.randn(n, generator=gen, device="cuda") * 0.2
        for border in (math.log1p(-case["clip_low"]), math.log1p(case["clip_high"])):
            near = (shift - border).abs() < 0.004
            shift = torch.where(near, torch.full_like(shift, border + 0.006), shift)
        state["old_logp"] = logp - shift
        state["ref_logp"] = logp + torch.randn(n, generator=gen, device="cuda") * 0.3 if case["ref"] else None
        state["advantage"] = torch.randn(n, generator=gen, device="cuda") + 0.25
        state["row_weight"] = torch.rand(n, generator=gen, device="cuda") + 0.1 if case["weighted"] else None
        shape = n if case["reduction"] == "none" else 1
        state["grad_output"] = torch.full((shape,), case["scale"], device="cuda")
    if case["op"] == "preference":
        # ragged lengths that add up to the batch; every sequence keeps at least one token
        length, seqs = case["length"], 2 * case["pairs"]
        cut = (torch.rand(seqs, generator=gen, device="cuda") - 0.5) * length
        ends = torch.arange(1, seqs + 1, device="cuda") * length + cut.long()
        ends[-1] = n
        state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), ends])
        state["offsets"] = state["offsets"].to(torch.int32 if case["int32"] else torch.int64)
        state["target"][state["offsets"][:-1].long()] = 1
        state["logits"][state["offsets"][:-1].long(), 1] = 3.0
        logp = _logp_of(state["logits"], state["target"], 1.0).double()
        sums = _segment_sums(logp, state["offsets"])
        state["ref_logp"] = (sums + torch.randn(seqs, generator=gen, device="cuda") * 6.0).float() if case["ref"] else None
        if case["kind"] == "hinge" and case["ref"]:
            # the margin keeps off the hinge's corner, where either slope is right
            state["ref_logp"] = _off_the_corner(case, state, sums)
        state["grad_output"] = torch.full((1,), case["scale"], device="cuda")
    return state


def _segment_sums(values, offsets):
    total = torch.cat([torch.zeros(1, dtype=torch.float64, device="cuda"), values.cumsum(0)])
    return total[offsets.long()[1:]] - total[offsets.long()[:-1]]


def _off_the_corner(case, state, sums):
    ref, pairs = state["ref_logp"].double(), case["pairs"]
    value = sums
    if case["normalize"]:
        count = _segment_sums((state["target"] >= 0).double(), state["offsets"])
        value, ref = sums / count, ref / count
    h = (value[:pairs] - value[pairs:]) - (ref[:pairs] - ref[pairs:])
    near = (case["beta"] * h - 1.0).abs() < 0.01
    ref[:pairs] = torch.where(near, ref[:pairs] + 0.05 / case["beta"], ref[:pairs])
    return ref.float()


# ---------------------------------------------------------------------- plain forms
def _log_softmax(x, temperature):
    z = x.float() / temperature
    z = z - z.amax(1, keepdim=True)
    return z - z.exp().sum(1, keepdim=True).log()


def _picked(logq, target):
    keep = target >= 0
    index = torch.where(keep, target, torch.zeros_like(target)).long()
    logp = logq.gather(1, index[:, None])[:, 0]
    return keep, index, torch.where(keep, logp, torch.zeros_like(logp))


def _entropy(logq, keep):
    p = logq.exp()
    h = -torch.where(p > 0, p * logq, torch.zeros_like(p)).sum(1)
    return torch.where(keep, h, torch.zeros_like(h))


def _gradient(logq, keep, index, h, g_logp, g_entropy, temperature):
    """d/dx of sum(g_logp logp + g_entropy H): (g (onehot - p) - g_H p (log p + H)) / T, fp32."""
    zero = torch.zeros((), device="cuda")
    g = torch.where(keep, g_logp.float(), zero)[:, None]
    p = logq.exp()
    out = -g * p
    if g_entropy is not None:
        ge = torch.where(keep, g_entropy.float(), zero)[:, None]
        out = out - torch.where(p > 0, ge * p * (logq + h[:, None]), zero)
    out.scatter_add_(1, index[:, None], g)
    return out / temperature


def _plain_logprob(s, c):
    logq = _log_softmax(s["logits"], c["temperature"])
    keep, index, logp = _picked(logq, s["target"])
    out = {"logp": logp}
    h = _entropy(logq, keep) if c["entropy"] else None
    if c["entropy"]:
        out["entropy"] = h
    if c["backward"]:
        grad = _gradient(logq, keep, index, h, s["grad_logp"], s["grad_entropy"], c["temperature"])
        out["grad"] = grad.to(s["logits"].dtype)
    return out


def _plain_policy(s, c):
    logq = _log_softmax(s["logits"], c["temperature"])
    keep, index, logp = _picked(logq, s["target"])
    h = _entropy(logq, keep)
    zero, one = torch.zeros((), dtype=torch.float64, device="cuda"), torch.ones((), dtype=torch.float64, device="cuda")
    lp, adv = logp.double(), s["advantage"].double()
    ratio = (lp - s["old_logp"].double()).exp()
    clipped = ratio.clamp(1.0 - c["clip_low"], 1.0 + c["clip_high"])
    loss = torch.maximum(-adv * ratio, -adv * clipped)
    slope = torch.where(-adv * ratio >= -adv * clipped, -adv * ratio, zero)
    kl = zero.expand_as(lp)
    if c["ref"]:
        gap = s["ref_logp"].double() - lp
        kl = gap.exp() - gap - 1.0
        loss = loss + c["kl"] * kl
        slope = slope + c["kl"] * (1.0 - gap.exp())
    loss = loss - c["entropy"] * h.double()
    weight = torch.where(keep, s["row_weight"].double() if c["weighted"] else one, zero)
    total = weight.sum() if c["reduction"] == "mean" else one
    loss = torch.where(keep, weight * loss, zero) / total
    scale = weight / total * s["grad_output"].double()
    grad = _gradient(logq, keep, index, h, slope * scale, -c["entropy"] * scale, c["temperature"])
    stats = torch.stack([logp.double(), h.double(), torch.where(keep, ratio, zero), torch.where(keep, kl, zero)], 1)
    loss = loss if c["reduction"] == "none" else loss.sum().reshape(1)
    return {"loss": loss.float(), "grad": grad.to(s["logits"].dtype), "stats": stats.float()}


def _plain_preference(s, c):
    logq = _log_softmax(s["logits"], 1.0)
    keep, index, logp = _picked(logq, s["target"])
    pairs, offsets = c["pairs"], s["offsets"].long()
    sums = _segment_sums(logp.double(), offsets)
    count = _segment_sums(keep.double(), offsets)
    value = sums / count if c["normalize"] else sums
    h = value[:pairs] - value[pairs:]
    if s["ref_logp"] is not None:
        ref = s["ref_logp"].double()
        h = h - (ref[:pairs] - ref[pairs:])
    b, e = c["beta"], c["smoothing"]
    if c["kind"] == "sigmoid":
        loss = (1.0 - e) * (1.0 + (-b * h).exp()).log() + e * (1.0 + (b * h).exp()).log()
        slope = b * (1.0 / (1.0 + (-b * h).exp()) - (1.0 - e))
    elif c["kind"] == "hinge":
        loss = (1.0 - b * h).clamp_min(0.0)
        slope = -b * (b * h < 1.0).double()
    else:
        loss = (h - 0.5 / b) ** 2
        slope = 2.0 * (h - 0.5 / b)
    slope = slope / pairs * s["grad_output"].double()
    per_seq = torch.cat([slope, -slope])
    if c["normalize"]:
        per_seq = per_seq / count
    per_row = per_seq.repeat_interleave(offsets[1:] - offsets[:-1], output_size=index.numel())
    grad = _gradient(logq, keep, index, None, per_row, None, 1.0)
    return {"loss": loss.mean().reshape(1).float(), "seq_logp": value.float(), "grad": grad.to(s["logits"].dtype)}


def _plain_linear(s, c):
    hidden, weight = s["hidden"].float(), s["weight"].float()
    z = hidden @ weight.t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    logq = _log_softmax(z, c["temperature"])
    keep, index, logp = _picked(logq, s["target"])
    out = {"logp": logp}
    h = _entropy(logq, keep) if c["entropy"] else None
    if c["entropy"]:
        out["entropy"] = h
    if c["backward"]:
        dz = _gradient(logq, keep, index, h, s["grad_logp"], s["grad_entropy"], c["temperature"])
        out["grad_hidden"] = (dz @ weight).to(torch.bfloat16)
        out["grad_weight"] = (dz.t() @ hidden).to(torch.bfloat16)
        if s["bias"] is not None:
            out["grad_bias"] = dz.sum(0).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------- the framework's calls
def _own_logprob(s, c):
    import softmax_cross_entropy_pass_gb300 as ce
    logp, entropy, stats = ce.ce_token_logprob(s["logits"], s["target"], temperature=c["temperature"],
                                               with_entropy=c["entropy"])
    out = {"logp": logp}
    if c["entropy"]:
        out["entropy"] = entropy
    if c["backward"]:
        grad = torch.empty(s["logits"].shape, dtype=s["logits"].dtype, device="cuda")
        out["grad"] = ce.ce_token_logprob_backward(s["logits"], s["target"], stats, s["grad_logp"],
                                                   grad_entropy=s["grad_entropy"], temperature=c["temperature"],
                                                   grad=grad)
    return out


def _own_policy(s, c):
    import softmax_cross_entropy_pass_gb300 as ce
    grad = torch.empty(s["logits"].shape, dtype=s["logits"].dtype, device="cuda")
    stats = torch.empty(c["rows"], 4, device="cuda")
    loss, grad = ce.ce_policy_fwd_bwd(s["logits"], s["target"], s["advantage"], old_logp=s["old_logp"],
                                      ref_logp=s["ref_logp"], row_weight=s["row_weight"], clip_low=c["clip_low"],
                                      clip_high=c["clip_high"], kl_coef=c["kl"], entropy_coef=c["entropy"],
                                      temperature=c["temperature"], reduction=c["reduction"],
                                      grad_output=s["grad_output"], grad=grad, row_stats=stats)
    return {"loss": loss, "grad": grad, "stats": stats}


def _own_preference(s, c):
    import softmax_cross_entropy_pass_gb300 as ce
    grad = torch.empty(s["logits"].shape, dtype=s["logits"].dtype, device="cuda")
    loss, seq_logp, grad = ce.ce_preference_fwd_bwd(s["logits"], s["target"], s["offsets"], ref_logp=s["ref_logp"],
                                                    loss_kind=c["kind"], beta=c["beta"],
                                                    label_smoothing=c["smoothing"] if c["kind"] == "sigmoid" else 0.0,
                                                    length_normalize=c["normalize"],
                                                    grad_output=s["grad_output"], grad=grad)
    return {"loss": loss, "seq_logp": seq_logp, "grad": grad}


def _own_linear(s, c):
    import softmax_cross_entropy_pass_gb300 as ce
    if not c["backward"]:
        bias = None if s["bias"] is None else s["bias"].float()
        logp, entropy, _ = ce.flce_token_logprob(s["hidden"], s["weight"], s["target"], bias=bias,
                                                 temperature=c["temperature"], with_entropy=c["entropy"])
        return {"logp": logp, "entropy": entropy} if c["entropy"] else {"logp": logp}
    hidden, weight = s["hidden"].detach().requires_grad_(), s["weight"].detach().requires_grad_()
    leaves, bias = [hidden, weight], None
    if s["bias"] is not None:
        leaves.append(s["bias"].detach().requires_grad_())
        bias = leaves[2].float()
    outs = ce.linear_token_logprob(hidden, weight, s["target"], bias=bias, temperature=c["temperature"],
                                   with_entropy=c["entropy"])
    outs = list(outs) if c["entropy"] else [outs]
    given = [s["grad_logp"], s["grad_entropy"]] if c["entropy"] else [s["grad_logp"]]
    grads = torch.autograd.grad(outs, leaves, given)
    out = {"logp": outs[0].detach()}
    if c["entropy"]:
        out["entropy"] = outs[1].detach()
    out["grad_hidden"], out["grad_weight"] = grads[0], grads[1]
    if bias is not None:
        out["grad_bias"] = grads[2]
    return out


def run(state):
    c = state["case"]
    if own:
        call = {"logprob": _own_logprob, "policy": _own_policy, "preference": _own_preference, "linear": _own_linear}
    else:
        call = {"logprob": _plain_logprob, "policy": _plain_policy, "preference": _plain_preference,
                "linear": _plain_linear}
    return call[c["op"]](state, c)


# ---------------------------------------------------------------------- work
def work(case):
    n, live, vocab = _rows(case), _valid_rows(case), case["vocab"]
    if case["op"] == "linear":
        hidden = case["hidden"]
        product = 2 * live * hidden * vocab
        heads = vocab * hidden * 2 + live * hidden * 2 + n * 16
        if not case["backward"]:
            return {"bytes": heads, "flops": product}
        # the logits once, and the two gradient products; the weights and hidden states once, both gradients written
        return {"bytes": heads + n * hidden * 2 + vocab * hidden * 2, "flops": 3 * product}
    size = SIZES[case["dtype"]]
    read, wrote = live * vocab * size, n * vocab * size
    flops = 4 * live * vocab
    rows = n * (8 + 16)
    if case["op"] == "logprob" and not case["backward"]:
        return {"bytes": read + rows, "flops": flops}
    return {"bytes": read + wrote + rows, "flops": 2 * flops}


# ---------------------------------------------------------------------- the definitions in 64 bits
def _blocks(n, vocab):
    step = max(1, (1 << 27) // vocab)
    return [(r, min(n, r + step)) for r in range(0, n, step)]


def _exact_rows(z, target):
    """log-probability and entropy of rows of z (fp64, differentiable); 0 where the target is ignored."""
    logq = torch.log_softmax(z, 1)
    keep = target >= 0
    logp = logq.gather(1, target.clamp_min(0).long()[:, None])[:, 0]
    entropy = torch.special.entr(logq.exp()).sum(1)
    return logp * keep, entropy * keep


def _exact_logits(x, target, temperature, cotangents):
    """(logp, entropy, gradient) of logits given a function block -> (g_logp, g_entropy)."""
    n, vocab = x.shape
    logp = torch.zeros(n, dtype=torch.float64, device="cuda")
    entropy, grad = torch.zeros_like(logp), None
    if cotangents is not None:
        grad = torch.zeros(n, vocab, dtype=torch.float64, device="cuda")
    for lo, hi in _blocks(n, vocab):
        z = x[lo:hi].double() / temperature
        lp = torch.log_softmax(z, 1)
        t = target[lo:hi]
        keep = t >= 0
        logp[lo:hi] = lp.gather(1, t.clamp_min(0).long()[:, None])[:, 0] * keep
        q = lp.exp()
        ent = torch.special.entr(q).sum(1) * keep
        entropy[lo:hi] = ent
        if cotangents is None:
            continue
        # the vector-Jacobian product of log-softmax, applied to d(logp) and, through q, to d(entropy)
        g, ge = cotangents(lo, hi, logp[lo:hi], ent)
        up = torch.zeros_like(lp)
        up.scatter_(1, t.clamp_min(0).long()[:, None], (g * keep)[:, None])
        if ge is not None:
            # d entr(e^l) / dl = -e^l (l + 1), which tends to 0 as l falls
            up -= (ge * keep)[:, None] * torch.where(q > 0, q * (lp + 1.0), torch.zeros_like(q))
        grad[lo:hi] = (up - q * up.sum(1, keepdim=True)) / temperature
    return logp, entropy, grad


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    target = s["target"]
    if op == "linear":
        if 2.0 * c["rows"] * c["hidden"] * c["vocab"] * (3 if c["backward"] else 1) > 1.2e13:
            return None
        h, w = s["hidden"].double(), s["weight"].double()
        logp = torch.zeros(c["rows"], dtype=torch.float64, device="cuda")
        entropy, dh, dw = torch.zeros_like(logp), torch.zeros_like(h), None
        db = torch.zeros(c["vocab"], dtype=torch.float64, device="cuda")
        if c["backward"]:
            dw = torch.zeros_like(w)
        for lo, hi in _blocks(c["rows"], c["vocab"]):
            z = h[lo:hi] @ w.t()
            if s["bias"] is not None:
                z += s["bias"].double()
            z = (z / c["temperature"]).requires_grad_(c["backward"])
            lp, ent = _exact_rows(z, target[lo:hi])
            logp[lo:hi], entropy[lo:hi] = lp.detach(), ent.detach()
            if c["backward"]:
                total = (lp * s["grad_logp"][lo:hi].double()).sum()
                if c["entropy"]:
                    total = total + (ent * s["grad_entropy"][lo:hi].double()).sum()
                dz = torch.autograd.grad(total, z)[0] / c["temperature"]
                dh[lo:hi] = dz @ w
                dw += dz.t() @ h[lo:hi]
                db += dz.sum(0)
        out = {"logp": logp}
        if c["entropy"]:
            out["entropy"] = entropy
        if c["backward"]:
            out["grad_hidden"], out["grad_weight"] = dh, dw
            if s["bias"] is not None:
                out["grad_bias"] = db
        return out
    x = s["logits"]
    if op == "logprob":
        def given(lo, hi, logp, ent):
            ge = s["grad_entropy"]
            return s["grad_logp"][lo:hi].double(), None if ge is None else ge[lo:hi].double()
        logp, entropy, grad = _exact_logits(x, target, c["temperature"], given if c["backward"] else None)
        out = {"logp": logp}
        if c["entropy"]:
            out["entropy"] = entropy
        if c["backward"]:
            out["grad"] = grad
        return out
    if op == "policy":
        keep = (target >= 0).double()
        weight = keep * s["row_weight"].double() if c["weighted"] else keep
        total = weight.sum() if c["reduction"] == "mean" else torch.ones((), dtype=torch.float64, device="cuda")
        weight = weight / total
        loss = torch.zeros_like(keep)
        ratio, kl = torch.zeros_like(keep), torch.zeros_like(keep)

        def row_loss(lo, hi, logp, ent):
            lp, en = logp.detach().requires_grad_(), ent.detach().requires_grad_()
            r = torch.exp(lp - s["old_logp"][lo:hi].double())
            a = s["advantage"][lo:hi].double()
            value = -torch.minimum(a * r, a * r.clamp(1.0 - c["clip_low"], 1.0 + c["clip_high"]))
            ratio[lo:hi] = r.detach() * keep[lo:hi]
            if c["ref"]:
                gap = s["ref_logp"][lo:hi].double() - lp
                k = torch.expm1(gap) - gap
                kl[lo:hi] = k.detach() * keep[lo:hi]
                value = value + c["kl"] * k
            value = (value - c["entropy"] * en) * weight[lo:hi]
            loss[lo:hi] = value.detach()
            up = s["grad_output"].double()
            g, ge = torch.autograd.grad((value * (up[lo:hi] if c["reduction"] == "none" else up)).sum(), [lp, en],
                                        allow_unused=True)
            return g, ge
        logp, entropy, grad = _exact_logits(x, target, c["temperature"], row_loss)
        return {"loss": loss if c["reduction"] == "none" else loss.sum().reshape(1), "grad": grad,
                "stats": torch.stack([logp, entropy, ratio, kl], 1)}
    # preference: the sequence values first, the loss differentiated at that level, then the rows
    logp, _, _ = _exact_logits(x, target, 1.0, None)
    off, pairs = s["offsets"].long().tolist(), c["pairs"]
    sums = torch.stack([logp[a:b].sum() for a, b in zip(off[:-1], off[1:])])
    count = torch.stack([(target[a:b] >= 0).sum().double() for a, b in zip(off[:-1], off[1:])])
    sums.requires_grad_()
    value = sums / count if c["normalize"] else sums
    h = value[:pairs] - value[pairs:]
    if s["ref_logp"] is not None:
        h = h - (s["ref_logp"][:pairs].double() - s["ref_logp"][pairs:].double())
    z = c["beta"] * h
    if c["kind"] == "sigmoid":
        loss = -(1.0 - c["smoothing"]) * torch.nn.functional.logsigmoid(z) - c["smoothing"] * torch.nn.functional.logsigmoid(-z)
    elif c["kind"] == "hinge":
        loss = torch.relu(1.0 - z)
    else:
        loss = torch.square(h - 1.0 / (2.0 * c["beta"]))
    per_seq = torch.autograd.grad((loss.mean() * s["grad_output"].double()).sum(), sums)[0]
    per_row = torch.zeros_like(logp)
    for j, (a, b) in enumerate(zip(off[:-1], off[1:])):
        per_row[a:b] = per_seq[j]
    _, _, grad = _exact_logits(x, target, 1.0, lambda lo, hi, lp, en: (per_row[lo:hi], None))
    return {"loss": loss.mean().detach().reshape(1), "seq_logp": value.detach(), "grad": grad}
