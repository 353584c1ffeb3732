"""Cases that measure the operators of the 8-bit serving head: root-mean-square
norm with the residual's addition and an 8-bit output, quantising to 8 bits in
blocks, the matrix product of 8-bit operands with a scale for each block of
128, and the verification of drafted tokens against the target's
probabilities, each beside its plain form.

The plain forms are elementary torch operations in fp32 (running sums over a
vocabulary in fp64); ``exact`` holds the definitions in fp64. 8-bit values are
e4m3; ``exact`` gives them before their rounding.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
E4M3_MAX, MIN_SCALE, BLOCK = 448.0, 2.0 ** -126, 128


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # the final norm of one decoding step of four sequences: the smallest call
        dict(name="norm_step", op="norm", rows=4, hidden=4096, pad=0, dtype="bf16", residual=True, eps=1e-6),
        # the norm before the head over a prompt batch
        dict(name="norm_prompt", op="norm", rows=8192, hidden=4096, pad=0, dtype="bf16", residual=True, eps=1e-6),
        # fp32 rows of an odd width in a wider buffer, no residual
        dict(name="norm_ragged", op="norm", rows=1501, hidden=2570, pad=3, dtype="f32", residual=False, eps=1e-5),
        # activations on their way into an 8-bit product
        dict(name="quantize_rows", op="quantize", rows=4096, cols=8192, pad=0, dtype="bf16", tile=False),
        # a head's weights, laid out once after loading
        dict(name="quantize_weight", op="quantize", rows=128256, cols=4096, pad=0, dtype="bf16", tile=True),
        # the head for single tokens of four sequences: bound by the weights' bytes
        dict(name="gemm_step", op="gemm", m=4, n=128256, k=4096, dtype="bf16", bias=False),
        # a decoding batch through a square layer
        dict(name="gemm_batch", op="gemm", m=64, n=4096, k=4096, dtype="bf16", bias=False),
        # odd sizes on every side, biased, fp32 logits
        dict(name="gemm_ragged", op="gemm", m=300, n=50257, k=2050, dtype="f32", bias=True),
        # every logit of a prompt chunk
        dict(name="gemm_prompt", op="gemm", m=4096, n=128256, k=4096, dtype="bf16", bias=False),
        # one sequence with three drafts: latency
        dict(name="verify_step", op="verify", seqs=1, drafts=3, vocab=128256, pad=0, dtype="bf16", draft_model=True,
             temperature=1.0, mixed=False, noise=0.7, padded=0.0, accept=0.75),
        # a serving batch with a draft model
        dict(name="verify_batch", op="verify", seqs=128, drafts=4, vocab=128256, pad=0, dtype="bf16", draft_model=True,
             temperature=0.8, mixed=False, noise=0.7, padded=0.0, accept=0.65),
        # looked-up drafts of different lengths, a temperature for each request (greedy among them), fp32 logits, odd rows
        dict(name="verify_lookup", op="verify", seqs=48, drafts=6, vocab=50257, pad=5, dtype="f32", draft_model=False,
             temperature=1.0, mixed=True, noise=0.0, padded=0.4, accept=0.7),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "gemm", "verify"])
    if op == "norm":
        hidden = _log_int(rng, 64, 16384)
        return dict(op=op, rows=_log_int(rng, 1, max(1, min(8192, 8192 * 4096 // hidden))), hidden=hidden,
                    pad=rng.choice([0, 0, 3, 8]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    residual=rng.random() < 0.6, eps=rng.choice([1e-6, 1e-5]))
    if op == "quantize":
        cols, tile = _log_int(rng, 64, 16384), rng.random() < 0.5
        return dict(op=op, rows=_log_int(rng, 1, max(1, min(131072 if tile else 8192, 64000 * 4096 // cols))), cols=cols,
                    pad=rng.choice([0, 0, 3, 8]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), tile=tile)
    if op == "gemm":
        k, n = _log_int(rng, 128, 8192), _log_int(rng, 64, 131072)
        k = k if rng.random() < 0.3 else max(128, k // 128 * 128)
        return dict(op=op, m=_log_int(rng, 1, max(1, min(4096, 2 * 10 ** 12 // (n * k)))), n=n, k=k,
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), bias=rng.random() < 0.4)
    vocab, drafts = _log_int(rng, 1000, 256000), rng.choice([0, 1, 2, 3, 4, 5, 8])
    model = rng.random() < 0.6
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = 128 * 5 * 128256 * 2 // (vocab * (drafts + 1) * SIZES[dtype])
    return dict(op=op, seqs=_log_int(rng, 1, max(1, min(256, most))), drafts=drafts, vocab=vocab,
                pad=rng.choice([0, 0, 1, 8]), dtype=dtype, draft_model=model,
                temperature=rng.choice([1.0, 0.7, 1.2]), mixed=rng.random() < 0.4, noise=0.7 if model else 0.0,
                padded=rng.choice([0.0, 0.3]), accept=0.65 if model else 0.3)


# ---------------------------------------------------------------------- inputs
def _e4m3(x):
    """(e4m3 values, scales) of blocks of 128 columns; the values in a buffer whose rows start at multiples of 16 bytes."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    wide = torch.zeros(rows, blocks * BLOCK, device=x.device)
    wide[:, :cols] = x
    wide = wide.view(rows, blocks, BLOCK)
    scale = (wide.abs().amax(2) / E4M3_MAX).clamp_min(MIN_SCALE)
    q = (wide / scale[:, :, None]).view(rows, -1)[:, :-(-cols // 16) * 16].to(E4M3)
    return q[:, :cols], scale


def _e4m3_tiles(rows, cols, gen, std):
    """A weight's e4m3 values (rows at multiples of 16 bytes) and a scale for each 128 x 128, made block row by block row."""
    ld = -(-cols // 16) * 16
    q = torch.zeros(rows, ld, dtype=torch.uint8, device="cuda").view(E4M3)
    scale = torch.empty(-(-rows // BLOCK), -(-cols // BLOCK), device="cuda")
    step = 128 * BLOCK
    for r in range(0, rows, step):
        e = min(rows, r + step)
        w = torch.zeros(-(-(e - r) // BLOCK) * BLOCK, scale.shape[1] * BLOCK, device="cuda")
        w[:e - r, :cols].normal_(0.0, std, generator=gen)
        t = w.view(-1, BLOCK, scale.shape[1], BLOCK)
        s = (t.abs().amax((1, 3)) / E4M3_MAX).clamp_min(MIN_SCALE)
        q[r:e] = (t / s[:, None, :, None]).view(w.shape)[:e - r, :ld].to(E4M3)
        scale[r // BLOCK:-(-e // BLOCK)] = s
    return q[:, :cols], scale


def _activations(rows, cols, pad, dtype, gen):
    """Hidden states: rows of different size, a few columns far above the others."""
    x = torch.empty(rows, cols + pad, device="cuda").normal_(0.0, 1.0, generator=gen)
    x *= 0.5 + 2.0 * torch.rand(rows, 1, generator=gen, device="cuda")
    x[:, ::509] *= 12.0
    return x.to(DTYPES[dtype])[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case=case)
    if case["op"] == "norm":
        state["x"] = _activations(case["rows"], case["hidden"], case["pad"], case["dtype"], gen)
        state["residual"] = None
        if case["residual"]:
            state["residual"] = _activations(case["rows"], case["hidden"], case["pad"], case["dtype"], gen)
        state["weight"] = (1.0 + 0.2 * torch.randn(case["hidden"], generator=gen, device="cuda")).to(DTYPES[case["dtype"]])
    elif case["op"] == "quantize":
        x = torch.empty(case["rows"], case["cols"] + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
        x.normal_(0.0, 0.02 if case["tile"] else 1.0, generator=gen)
        state["x"] = x[:, :case["cols"]]
    elif case["op"] == "gemm":
        state["a"], state["a_scale"] = _e4m3(_activations(case["m"], case["k"], 0, "f32", gen))
        state["b"], state["b_scale"] = _e4m3_tiles(case["n"], case["k"], gen, 0.02)
        state["bias"] = 0.3 * torch.randn(case["n"], generator=gen, device="cuda") if case["bias"] else None
    else:
        _prepare_verify(case, gen, state)
    return state


def _prepare_verify(case, gen, state):
    seqs, k, vocab, dtype = case["seqs"], case["drafts"], case["vocab"], DTYPES[case["dtype"]]
    target = torch.empty(seqs, k + 1, vocab + case["pad"], device="cuda").normal_(0.0, 2.0, generator=gen)
    peaks = torch.randint(0, vocab, (seqs, k + 1, 24), generator=gen, device="cuda")
    target.scatter_(2, peaks, 9.0 + 6.0 * torch.rand(seqs, k + 1, 24, generator=gen, device="cuda"))
    temperature = torch.full((seqs,), case["temperature"], device="cuda")
    if case["mixed"]:
        temperature = 0.5 + torch.rand(seqs, generator=gen, device="cuda")
        temperature[::3] = 0.0
    t = torch.where(temperature > 0, temperature, torch.ones_like(temperature))[:, None, None]
    state["logits"] = target.to(dtype)[:, :, :vocab]
    state["draft_logits"] = None
    if case["draft_model"]:
        # a draft model that knows the target up to a noise on its logits
        draft = target[:, :k].clone()
        draft += case["noise"] * torch.randn(draft.shape, generator=gen, device="cuda")
        state["draft_logits"] = draft.to(dtype)[:, :, :vocab]
        spread = state["draft_logits"].float()
        del draft
    else:
        # drafts found by lookup: like the target's own tokens
        spread = state["logits"][:, :k].float() * 1.4
    del target
    race = torch.empty(spread.shape, device="cuda").exponential_(generator=gen).log_()
    greedy = (temperature == 0)[:, None, None]
    pick = torch.where(greedy, spread, spread / t - race)
    token = _first_max(pick)
    del race, pick, spread
    if case["padded"]:
        # shorter drafts end in -1
        length = torch.randint(0, k + 1, (seqs,), generator=gen, device="cuda")
        full = torch.rand(seqs, generator=gen, device="cuda") >= case["padded"]
        length = torch.where(full, torch.full_like(length, k), length)
        token = torch.where(torch.arange(k, device="cuda") < length[:, None], token, torch.full_like(token, -1))
    state["draft_token"] = token
    state["temperature"] = temperature if case["mixed"] else case["temperature"]
    state["accept_uniform"] = torch.rand(seqs, k, generator=gen, device="cuda")
    state["sample_uniform"] = torch.rand(seqs, generator=gen, device="cuda")
    # the random numbers keep off the borders, where either answer is right
    p = torch.softmax(state["logits"].double() / t, 2)
    q = None if state["draft_logits"] is None else torch.softmax(state["draft_logits"].double() / t, 2)
    at = token.clamp_min(0)[:, :, None]
    pt = p[:, :k].gather(2, at)[:, :, 0]
    qt = torch.ones_like(pt) if q is None else q.gather(2, at)[:, :, 0]
    u = state["accept_uniform"].double()
    u = torch.where((u * qt / pt - 1.0).abs() < 1e-4, u * 0.999, u)
    state["accept_uniform"] = u.float()
    count = _leading((state["accept_uniform"].double() * qt < pt) & (token >= 0))
    w = _left_over(p, q, token, count)
    total = w.sum(1)
    r = state["sample_uniform"].double()
    upto = w.cumsum(1)
    pick = (upto <= (r * total)[:, None]).sum(1).clamp_max(vocab - 1)
    size = w.gather(1, pick[:, None])[:, 0] / total
    pick = torch.where(size < 1e-4, _first_max(w), pick)
    size = w.gather(1, pick[:, None])[:, 0]
    below = upto.gather(1, pick[:, None])[:, 0] - size
    inside = ((r * total - below) / size).clamp(0.05, 0.95)
    state["sample_uniform"] = ((below + inside * size) / total).float()


# ---------------------------------------------------------------------- plain forms
def _first_max(z):
    """The lowest index of the largest value along the last axis."""
    index = torch.arange(z.shape[-1], device=z.device)
    return torch.where(z == z.amax(-1, keepdim=True), index, z.shape[-1]).amin(-1) if z.numel() else z.new_zeros(z.shape[:-1]).long()


def _leading(ok):
    """How many of every row's values are true before the first that is not."""
    return ok.long().cumprod(1).sum(1)


def _left_over(p, q, token, count):
    """What the token at position count is drawn from: max(p - q, 0) where a draft was turned down, p otherwise."""
    seqs, k = token.shape
    rows = torch.arange(seqs, device=p.device)
    base = p[rows, count]
    if not k:
        return base
    at = count.clamp_max(k - 1)
    drafted = token[rows, at]
    turned = ((count < k) & (drafted >= 0))[:, None]
    if q is None:
        less = base.clone()
        less[rows, drafted.clamp_min(0)] = 0.0
    else:
        less = (base - q[rows, at]).clamp_min(0.0)
    less = torch.where(turned, less, base)
    return torch.where(less.sum(1, keepdim=True) > 0, less, base)


def _blocks_of(x):
    """x (fp32) as [rows, blocks, 128], zeros past the last column."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    if cols == blocks * BLOCK:
        return x.view(rows, blocks, BLOCK)
    wide = torch.zeros(rows, blocks * BLOCK, device=x.device)
    wide[:, :cols] = x
    return wide.view(rows, blocks, BLOCK)


def _plain_rows(y):
    t = _blocks_of(y)
    scale = (t.abs().amax(2) / E4M3_MAX).clamp_min(MIN_SCALE)
    q = (t / scale[:, :, None]).to(E4M3).view(y.shape[0], -1)[:, :y.shape[1]]
    return q, scale


def _plain_norm(s, c):
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["residual_out"] = h.to(s["x"].dtype)
    y = h / ((h * h).mean(1, keepdim=True) + c["eps"]).sqrt() * s["weight"].float()
    out["q"], out["scale"] = _plain_rows(y)
    return out


def _plain_quantize(s, c):
    x = s["x"].float()
    if not c["tile"]:
        q, scale = _plain_rows(x)
        return {"q": q, "scale": scale}
    rows, cols = x.shape
    n, m = -(-rows // BLOCK), -(-cols // BLOCK)
    if (rows, cols) != (n * BLOCK, m * BLOCK):
        wide = torch.zeros(n * BLOCK, m * BLOCK, device=x.device)
        wide[:rows, :cols] = x
        x = wide
    t = x.view(n, BLOCK, m, BLOCK)
    scale = (t.abs().amax(3).amax(1) / E4M3_MAX).clamp_min(MIN_SCALE)
    q = (t / scale[:, None, :, None]).to(E4M3).view(n * BLOCK, m * BLOCK)[:rows, :cols]
    return {"q": q, "scale": scale}


def _plain_gemm(s, c):
    k, n = c["k"], c["n"]
    a = s["a"].float() * s["a_scale"].repeat_interleave(BLOCK, 1)[:, :k]
    b = s["b"].float() * s["b_scale"].repeat_interleave(BLOCK, 1)[:, :k].repeat_interleave(BLOCK, 0)[:n]
    out = a @ b.t()
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(DTYPES[c["dtype"]])


def _plain_softmax(x, t):
    z = x.float() / t
    z = z - z.amax(2, keepdim=True)
    e = z.exp()
    total = e.sum(2, keepdim=True)
    return e / total, z - total.log()


def _plain_verify(s, c):
    seqs, k, vocab = c["seqs"], c["drafts"], c["vocab"]
    given = s["temperature"] if c["mixed"] else torch.full((seqs,), c["temperature"], device="cuda")
    greedy = given == 0
    t = torch.where(greedy, torch.ones_like(given), given)[:, None, None]
    p, logp = _plain_softmax(s["logits"], t)
    q = None if s["draft_logits"] is None else _plain_softmax(s["draft_logits"], t)[0]
    token = s["draft_token"]
    there = token >= 0
    at = token.clamp_min(0)[:, :, None]
    pt = p[:, :k].gather(2, at)[:, :, 0]
    qt = torch.ones_like(pt) if q is None else q.gather(2, at)[:, :, 0]
    best = _first_max(s["logits"])
    ok = torch.where(greedy[:, None], token == best[:, :k], s["accept_uniform"] * qt < pt) & there
    count = _leading(ok)
    w = _left_over(p, q, token, count).double()
    upto = w.cumsum(1)
    drawn = (upto <= (s["sample_uniform"].double() * upto[:, -1])[:, None]).sum(1).clamp_max(vocab - 1)
    rows = torch.arange(seqs, device="cuda")
    drawn = torch.where(greedy, best[rows, count], drawn)
    place = torch.arange(k + 1, device="cuda")
    kept = torch.cat([token, token.new_zeros(seqs, 1)], 1)
    tokens = torch.where(place == count[:, None], drawn[:, None], kept)
    tokens = torch.where(place <= count[:, None], tokens, torch.full_like(tokens, -1))
    value = logp.gather(2, tokens.clamp_min(0)[:, :, None])[:, :, 0]
    return {"accepted": count.to(torch.int32), "tokens": tokens,
            "logp": torch.where(tokens >= 0, value, torch.zeros_like(value))}


# ---------------------------------------------------------------------- the framework's calls
def _own_norm(s, c):
    import softmax_cross_entropy_pass_gb300 as ce
    q, scale, residual = ce.ce_rms_norm_fp8(s["x"], s["weight"], residual=s["residual"], eps=c["eps"])
    out = {"q": q, "scale": scale}
    if residual is not None:
        out["residual_out"] = residual
    return out


def _own_quantize(s, c):
    import softmax_cross_entropy_pass_gb300 as ce
    q, scale = ce.ce_quantize_fp8(s["x"], block_rows=128 if c["tile"] else 1)
    return {"q": q, "scale": scale}


def _own_gemm(s, c):
    import softmax_cross_entropy_pass_gb300 as ce
    return ce.ce_gemm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], bias=s["bias"], out_dtype=DTYPES[c["dtype"]])


def _own_verify(s, c):
    import softmax_cross_entropy_pass_gb300 as ce
    accepted, tokens, logp = ce.ce_verify_drafts(s["logits"], s["draft_token"], s["accept_uniform"],
                                                 s["sample_uniform"], draft_logits=s["draft_logits"],
                                                 temperature=s["temperature"])
    return {"accepted": accepted, "tokens": tokens, "logp": logp}


def run(state):
    c = state["case"]
    if own:
        call = {"norm": _own_norm, "quantize": _own_quantize, "gemm": _own_gemm, "verify": _own_verify}
    else:
        call = {"norm": _plain_norm, "quantize": _plain_quantize, "gemm": _plain_gemm, "verify": _plain_verify}
    return call[c["op"]](state, c)


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] == "norm":
        n, h, size = case["rows"], case["hidden"], SIZES[case["dtype"]]
        streams = 3 if case["residual"] else 1
        return {"bytes": n * h * (streams * size + 1) + n * -(-h // BLOCK) * 4 + h * size, "flops": 10 * n * h}
    if case["op"] == "quantize":
        n, h = case["rows"], case["cols"]
        scales = (-(-n // BLOCK) if case["tile"] else n) * -(-h // BLOCK)
        return {"bytes": n * h * (SIZES[case["dtype"]] + 1) + 4 * scales, "flops": 3 * n * h}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-k // BLOCK)
        return {"bytes": (m + n) * k + 4 * blocks * (m + -(-n // BLOCK)) + m * n * SIZES[case["dtype"]]
                + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    # rows behind the first draft that is turned down need not be read
    k, a = case["drafts"], case["accept"]
    rows = sum(a ** i for i in range(k + 1)) * case["seqs"]
    drafts = sum(a ** i for i in range(k)) * case["seqs"] if case["draft_model"] else 0.0
    return {"bytes": (rows + drafts) * case["vocab"] * SIZES[case["dtype"]] + case["seqs"] * (k + 1) * 28,
            "flops": 5 * (rows + drafts) * case["vocab"]}


# ---------------------------------------------------------------------- the definitions in 64 bits
def _exact_blocks(y, tall):
    """(y / scale, scale) of fp64 blocks of `tall` rows and 128 columns."""
    rows, cols = y.shape
    up, across = -(-rows // tall), -(-cols // BLOCK)
    padded = torch.nn.functional.pad(y, (0, across * BLOCK - cols, 0, up * tall - rows))
    top = padded.reshape(up, tall, across, BLOCK).abs().permute(0, 2, 1, 3).flatten(2).max(2).values
    scale = torch.maximum(top / E4M3_MAX, torch.full_like(top, MIN_SCALE))
    each = scale.repeat_interleave(tall, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]
    return y / each, scale


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        h = s["x"].double() + (0.0 if s["residual"] is None else s["residual"].double())
        size = torch.linalg.vector_norm(h, dim=1, keepdim=True).square() / c["hidden"] + c["eps"]
        q, scale = _exact_blocks(h * size.rsqrt() * s["weight"].double()[None], 1)
        out = {"q": q, "scale": scale}
        if s["residual"] is not None:
            out["residual_out"] = h
        return out
    if c["op"] == "quantize":
        q, scale = _exact_blocks(s["x"].double(), BLOCK if c["tile"] else 1)
        return {"q": q, "scale": scale}
    if c["op"] == "gemm":
        if 2.0 * c["m"] * c["n"] * c["k"] > 1.2e13:
            return None
        out = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
        wide = 64 * BLOCK
        for lo in range(0, c["n"], wide):
            hi = min(c["n"], lo + wide)
            per_row = torch.arange(lo, hi, device="cuda") // BLOCK
            for j, k in enumerate(range(0, c["k"], BLOCK)):
                part = s["a"][:, k:k + BLOCK].double() @ s["b"][lo:hi, k:k + BLOCK].double().t()
                out[:, lo:hi] += part * s["a_scale"][:, j].double()[:, None] * s["b_scale"][per_row, j].double()
        return out if s["bias"] is None else out + s["bias"].double()
    accepted, tokens, values = [], [], []
    for b in range(c["seqs"]):
        t = float(s["temperature"][b]) if c["mixed"] else c["temperature"]
        z = s["logits"][b].double()
        logq = torch.log_softmax(z / (t or 1.0), 1)
        line, lp = [], []
        for i in range(c["drafts"] + 1):
            p = logq[i].exp()
            drafted = int(s["draft_token"][b, i]) if i < c["drafts"] else -1
            q = torch.zeros_like(p)
            if drafted >= 0:
                if s["draft_logits"] is None:
                    q[drafted] = 1.0
                else:
                    q = torch.softmax(s["draft_logits"][b, i].double() / (t or 1.0), 0)
                best = int((z[i] == z[i].max()).nonzero()[0])
                if (best == drafted) if t == 0 else float(s["accept_uniform"][b, i]) < float(p[drafted] / q[drafted]):
                    line.append(drafted)
                    lp.append(logq[i, drafted])
                    continue
            if t == 0:
                token = int((z[i] == z[i].max()).nonzero()[0])
            else:
                w = (p - q).clamp_min(0.0)
                upto = (w if float(w.sum()) > 0 else p).cumsum(0)
                token = int(torch.searchsorted(upto, float(s["sample_uniform"][b]) * upto[-1], right=True))
            line.append(token)
            lp.append(logq[i, token])
            break
        accepted.append(len(line) - 1)
        rest = c["drafts"] + 1 - len(line)
        tokens.append(line + [-1] * rest)
        values.append(torch.stack(lp + [torch.zeros_like(lp[0])] * rest))
    return {"accepted": torch.tensor(accepted, dtype=torch.int32, device="cuda"),
            "tokens": torch.tensor(tokens, device="cuda"), "logp": torch.stack(values)}
