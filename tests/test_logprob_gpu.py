"""Token log-probabilities, the policy loss and the preference loss on the
GPU against their fp64 forms (lp_check.py, which derives the tolerances)."""
import math

import pytest
import torch

import lp_check as L

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def ce():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import softmax_cross_entropy_pass_gb300 as ce
    return ce


def f32(v):
    """A constant as the kernels hold it."""
    return float(torch.tensor(v, dtype=torch.float32))


def make(n, v, dtype, seed, ld=None, off=0, sigma=2.0, ignored=0.2, int32=False):
    """Logits as a view of a wider buffer, targets with ignored rows; some rows peaked at their target or elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or v
    buf = torch.empty(n, ld + off, device="cuda").normal_(0, sigma, generator=g)
    x = buf[:, off:off + v]
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    rows = torch.arange(n, device="cuda")
    x[rows[::3], t[::3]] = 25.0
    if v > 4:
        x[rows[1::3], (t[1::3] + 3) % v] = 18.0
    buf = buf.to(DT[dtype])
    x = buf[:, off:off + v]
    if n > 2:
        t[1] = v - 1
        t[2] = 0
    drop = torch.rand(n, generator=g, device="cuda") < ignored
    drop[0] = False
    t[drop] = -100
    return g, buf, x, (t.int() if int32 else t)


def rnd(g, n, s=1.0):
    return torch.randn(n, generator=g, device="cuda") * s


SHAPES = [
    # rows, vocab, row stride, first column
    (1, 1, 1, 0), (3, 2, 2, 0), (5, 7, 7, 0), (17, 1000, 1000, 0), (6, 4099, 4103, 3), (9, 8192, 8200, 0),
    (5, 20000, 20011, 5), (300, 513, 513, 0), (7, 33000, 33000, 0), (4, 65537, 65537, 1), (3, 131077, 131080, 2),
    (460, 2048, 2048, 0), (2, 280001, 280001, 0), (1, 128256, 128256, 0), (40, 50257, 50257, 0), (2, 700000, 700000, 0),
]


def outside_unchanged(buf, before, off, v):
    keep = torch.ones(buf.shape[1], dtype=torch.bool, device="cuda")
    keep[off:off + v] = False
    assert torch.equal(buf[:, keep], before[:, keep])


# ---------------------------------------------------------------------- token log-probabilities
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}ld{s[2]}@{s[3]}")
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("entropy", [True, False])
def test_token_logprob(ce, shape, dtype, entropy):
    n, v, ld, off = shape
    temperature = f32(0.7) if n % 2 else 1.0
    g, buf, x, t = make(n, v, dtype, n * 31 + v, ld, off, int32=n % 3 == 0)
    before = buf.clone()
    logp, ent, stats = ce.ce_token_logprob(x, t, temperature=temperature, with_entropy=entropy)
    gl, gh = rnd(g, n), rnd(g, n) if entropy else None
    grad = ce.ce_token_logprob_backward(x, t, stats, gl, grad_entropy=gh, temperature=temperature,
                                        grad=torch.empty(n, v, dtype=DT[dtype], device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    valid, logq, want, want_h = L.rows_ref(x, t, temperature)
    d = L.delta(x, temperature)
    L.check(logp, want, L.tol_logp(d, want) * valid, "logp")
    assert (ent is not None) == entropy
    if entropy:
        L.check(ent, want_h, L.tol_entropy(d, want_h) * valid, "entropy")
    z = torch.zeros(n, device="cuda")
    h = gh if entropy else z
    ref = L.grad_ref(logq, valid, t, gl, h, temperature)
    tol = L.tol_grad(x, ref, logq, valid, t, gl, h, z, z, DT[dtype], temperature)
    L.check(grad, ref, tol, "gradient")
    # over the logits: the same values, and nothing outside the rows' columns
    same = ce.ce_token_logprob_backward(x, t, stats, gl, grad_entropy=gh, temperature=temperature)
    assert same.data_ptr() == x.data_ptr()
    L.check(x, ref, tol, "gradient in place")
    outside_unchanged(buf, before, off, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_token_logprob_special_rows(ce, dtype):
    """-inf columns, the type's lowest value as a mask, rows of one value, huge
    and tiny logits; rows that have no distribution come out NaN; NaN and inf
    on ignored rows do no harm; targets outside the vocabulary give NaN."""
    v, dt = 5003, DT[dtype]
    low = torch.finfo(dt).min
    x = torch.randn(16, v, device="cuda").to(dt)
    t = torch.arange(16, device="cuda") * 7
    x[0, 100:] = -math.inf
    x[1, 100:] = low
    x[2] = low                       # everything masked with the lowest value: uniform
    x[3] = -math.inf                 # no distribution
    x[3 + 1, 11] = math.nan
    x[5, 12] = math.inf
    x[6] = math.nan
    t[6] = -100
    x[7] = 0.0
    x[8] = 50000.0 if dtype == "f16" else 3e38
    x[9, :] = -40000.0
    x[9, 5] = 60000.0
    x[10, t[10]] = -math.inf         # the target itself masked
    t[11] = v                        # outside
    t[12] = -5                       # outside
    x[13] = -math.inf
    x[13, t[13]] = 1.0               # the target alone: log p = 0, H = 0
    x[14] = math.nan
    x[15, :9] = math.nan             # NaN among -inf
    x[15, 9:] = -math.inf
    logp, ent, stats = ce.ce_token_logprob(x, t)
    gl, gh = torch.randn(16, device="cuda"), torch.randn(16, device="cuda")
    grad = ce.ce_token_logprob_backward(x, t, stats, gl, grad_entropy=gh, grad=torch.empty_like(x))
    plain = ce.ce_token_logprob(x, t, with_entropy=False)[0]
    valid, logq, want, want_h = L.rows_ref(x, t)
    nan = torch.tensor([3, 4, 5, 14, 15], device="cuda")
    for name, val in (("logp", logp), ("entropy", ent), ("logp without entropy", plain)):
        assert val[nan].isnan().all(), name
        assert val[[11, 12]].isnan().all() and val[6] == 0, name
    assert logp[10] == -math.inf and plain[10] == -math.inf
    assert logp[13] == 0 and ent[13] == 0
    ok = torch.tensor([0, 1, 2, 7, 8, 9, 13], device="cuda")
    d = L.delta(x[ok])
    L.check(logp[ok], want[ok], L.tol_logp(d, want[ok]), "logp")
    L.check(plain[ok], want[ok], L.tol_logp(d, want[ok]), "logp without entropy")
    L.check(ent[ok], want_h[ok], L.tol_entropy(d, want_h[ok]), "entropy")
    z = torch.zeros(len(ok), device="cuda")
    ref = L.grad_ref(logq[ok], valid[ok], t[ok], gl[ok], gh[ok])
    L.check(grad[ok], ref, L.tol_grad(x[ok], ref, logq[ok], valid[ok], t[ok], gl[ok], gh[ok], z, z, dt), "gradient")
    assert (grad[[6, 11, 12]] == 0).all()
    assert grad[nan].isnan().any(1).all()


@pytest.mark.parametrize("v", [5003, 8192, 32000, 50257])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("share", [0.0005, 0.3])
def test_scattered_masked_columns(ce, v, dtype, share):
    """-inf anywhere in the rows, beside the target's vector as well: probability
    and gradient exactly 0 there, everything else as the fp64 form has it."""
    n, dt = 24, DT[dtype]
    g, _, x, t = make(n, v, dtype, v + int(share * 1e4), ignored=0.1)
    off = torch.rand(n, v, generator=g, device="cuda") < share
    rows = torch.arange(n, device="cuda")
    for d in range(1, 9):       # some of the target's neighbours
        off[rows[d % 3::3], (t[d % 3::3].long().clamp_min(0) + d) % v] = True
    off[rows, t.long().clamp_min(0)] = False
    x[off] = -math.inf
    valid, logq, want, want_h = L.rows_ref(x, t)
    d = L.delta(x)
    logp, ent, stats = ce.ce_token_logprob(x, t)
    L.check(logp, want, L.tol_logp(d, want) * valid, "logp")
    L.check(ent, want_h, L.tol_entropy(d, want_h) * valid, "entropy")
    gl, gh, z = rnd(g, n), rnd(g, n), torch.zeros(n, device="cuda")
    ref = L.grad_ref(logq, valid, t, gl, gh)
    tol = L.tol_grad(x, ref, logq, valid, t, gl, gh, z, z, dt)
    grad = ce.ce_token_logprob_backward(x, t, stats, gl, grad_entropy=gh, grad=torch.empty_like(x))
    L.check(grad, ref, tol, "gradient from statistics")
    adv = rnd(g, n)
    want = L.policy_ref(x, t, adv, None, None, None, 0.2, 0.2, 0.0, f32(0.05), 1.0, "sum", None)
    for grad in (torch.empty_like(x), torch.empty(n, v + 1, dtype=dt, device="cuda")[:, 1:]):
        _, grad = ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=f32(0.05), reduction="sum", grad=grad)
        L.check(grad, want["grad"], want["tol_grad"], "policy gradient")
        assert (grad[off & valid[:, None]] == 0).all()


@pytest.mark.parametrize("temperature", [1e-4, 0.02, 50.0, 1e4])
@pytest.mark.parametrize("v", [900, 40000])
def test_far_temperatures(ce, temperature, v):
    temperature = f32(temperature)
    g, _, x, t = make(12, v, "f32", 3, ignored=0.1)
    logp, ent, stats = ce.ce_token_logprob(x, t, temperature=temperature)
    valid, logq, want, want_h = L.rows_ref(x, t, temperature)
    d = L.delta(x, temperature)
    L.check(logp, want, L.tol_logp(d, want) * valid, "logp")
    L.check(ent, want_h, L.tol_entropy(d, want_h) * valid, "entropy")
    gl, gh, z = rnd(g, 12), rnd(g, 12), torch.zeros(12, device="cuda")
    ref = L.grad_ref(logq, valid, t, gl, gh, temperature)
    grad = ce.ce_token_logprob_backward(x, t, stats, gl, grad_entropy=gh, temperature=temperature, grad=torch.empty_like(x))
    L.check(grad, ref, L.tol_grad(x, ref, logq, valid, t, gl, gh, z, z, torch.float32, temperature), "gradient")


@pytest.mark.parametrize("shape", [(21000, 110001), (300000, 8000)])
def test_offsets_past_32_bits(ce, shape):
    """Elements past 2^31 and bytes past 2^32: the last rows as the first ones."""
    n, v = shape
    x = torch.empty(n, v, dtype=torch.bfloat16, device="cuda").normal_(0, 2)
    t = torch.randint(0, v, (n,), device="cuda")
    t[5:-5] = -100
    adv, pick = torch.randn(n, device="cuda"), torch.cat([torch.arange(5), torch.arange(n - 5, n)]).cuda()
    xs, ts = x[pick].clone(), t[pick].clone()
    want = L.policy_ref(xs, ts, adv[pick], None, None, None, 0.2, 0.2, 0.0, f32(0.01), 1.0, "sum", None)
    stats = torch.empty(n, 4, device="cuda")
    logp, ent, st = ce.ce_token_logprob(x, t)
    gl = torch.randn(n, device="cuda")
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=f32(0.01), reduction="sum", row_stats=stats, grad=torch.empty_like(x))
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(grad[pick], want["grad"], want["tol_grad"], "policy gradient")
    L.check(stats[pick], want["stats"], want["tol_stats"], "row statistics")
    L.check(logp[pick], want["stats"][:, 0], want["tol_stats"][:, 0], "logp")
    L.check(ent[pick], want["stats"][:, 1], want["tol_stats"][:, 1], "entropy")
    assert (grad[n // 2] == 0).all() and (logp[5:-5] == 0).all()
    ce.ce_token_logprob_backward(x, t, st, gl, grad=grad)
    valid, logq, _, _ = L.rows_ref(xs, ts)
    z = torch.zeros(10, device="cuda")
    ref = L.grad_ref(logq, valid, ts, gl[pick], z)
    L.check(grad[pick], ref, L.tol_grad(xs, ref, logq, valid, ts, gl[pick], z, z, z, torch.bfloat16), "gradient")
    off = torch.tensor([0, 5, n], device="cuda")
    loss, seq, grad = ce.ce_preference_fwd_bwd(x, t, off, grad=grad)
    assert abs(seq[1].item() - logp[-5:].double().sum().item()) < 1e-3 and loss.isfinite().all()
    assert (grad[n - 1] != 0).any() and (grad[n // 2] == 0).all()


@pytest.mark.parametrize("n,v", [(9001, 3000), (20000, 300), (17000, 9000)])
def test_many_rows(ce, n, v):
    """More rows than one window of the row kernel deals out, most of them without a target, at random."""
    g, _, x, t = make(n, v, "bf16", n, ignored=0.6)
    adv = rnd(g, n)
    stats = torch.full((n, 4), 9.0, device="cuda")
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=f32(0.01), row_stats=stats, grad=torch.empty_like(x))
    want = L.policy_ref(x, t, adv, None, None, None, 0.2, 0.2, 0.0, f32(0.01), 1.0, "mean", None)
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(grad, want["grad"], want["tol_grad"], "gradient")
    L.check(stats, want["stats"], want["tol_stats"], "row statistics")
    logp, ent, _ = ce.ce_token_logprob(x, t)
    L.check(logp, want["stats"][:, 0], want["tol_stats"][:, 0], "logp")
    L.check(ent, want["stats"][:, 1], want["tol_stats"][:, 1], "entropy")
    rows, _ = ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=f32(0.01), reduction="none", grad=torch.empty_like(x))
    assert (rows[t < 0] == 0).all()
    assert abs(rows.double().sum().item() / int((t >= 0).sum()) - loss.item()) < 1e-6 * (1 + rows.double().abs().mean().item())


def test_token_logprob_statistics_without_entropy_refuse_its_gradient(ce):
    x, t = torch.randn(3, 100, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    _, _, stats = ce.ce_token_logprob(x, t, with_entropy=False)
    one = torch.ones(3, device="cuda")
    assert ce.ce_token_logprob_backward(x, t, stats, one, grad_entropy=one, grad=torch.empty_like(x)).isnan().any()
    assert ce.ce_token_logprob_backward(x, t, stats, one, grad=torch.empty_like(x)).isfinite().all()


def test_token_logprob_autograd(ce):
    g, _, x, t = make(33, 3001, "f32", 5)
    a = x.clone().requires_grad_()
    logp, ent = ce.token_logprob(a, t, temperature=0.5, with_entropy=True)
    w, u = rnd(g, 33), rnd(g, 33)
    (logp * w + ent * u).sum().backward()
    valid, logq, _, _ = L.rows_ref(x, t, 0.5)
    z = torch.zeros(33, device="cuda")
    ref = L.grad_ref(logq, valid, t, w, u, 0.5)
    tol = L.tol_grad(x, ref, logq, valid, t, w, u, z, z, torch.float32, 0.5)
    L.check(a.grad, ref, tol, "gradient")
    assert torch.equal(a.detach(), x)
    # one of the two outputs only, and twice over the same graph
    a.grad = None
    logp, ent = ce.token_logprob(a, t, temperature=0.5, with_entropy=True)
    ent.sum().backward(retain_graph=True)
    ent.sum().backward()
    ref = L.grad_ref(logq, valid, t, z, z + 1, 0.5)
    L.check(a.grad / 2, ref, L.tol_grad(x, ref, logq, valid, t, z, z + 1, z, z, torch.float32, 0.5), "entropy gradient")
    # in place: the logits become the gradient, once
    b = x.clone().requires_grad_()
    logp = ce.token_logprob(b, t, inplace=True)
    (gb,) = torch.autograd.grad(logp.sum(), b, retain_graph=True)
    assert gb.data_ptr() == b.data_ptr()
    with pytest.raises(ce.CEError, match="used up"):
        torch.autograd.grad(logp.sum(), b)
    # a directional difference of the fp64 form
    d = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
    f = lambda y: (L.rows_ref(y, t, 0.5)[2] * w.double() + L.rows_ref(y, t, 0.5)[3] * u.double()).sum()  # noqa: E731
    num = float((f(x.double() + 1e-6 * d) - f(x.double() - 1e-6 * d)) / 2e-6)
    a.grad = None
    logp, ent = ce.token_logprob(a, t, temperature=0.5, with_entropy=True)
    (logp * w + ent * u).sum().backward()
    assert abs(float((a.grad.double() * d).sum()) - num) <= float((tol * d.abs()).sum()) + 1e-5 * (1 + abs(num))


# ---------------------------------------------------------------------- policy loss
def policy_inputs(g, x, t, temperature, lo, hi):
    n = x.shape[0]
    base = L.rows_ref(x, t, temperature)[2].float()
    shift = rnd(g, n, 0.3)
    for border in (math.log1p(-lo) if lo < 1 else -99.0, math.log1p(hi)):
        shift = torch.where((shift - border).abs() < 0.003, torch.full_like(shift, border + 0.005), shift)
    old, ref, adv = base - shift, base + rnd(g, n, 0.5), rnd(g, n)
    w = torch.rand(n, generator=g, device="cuda") + 0.1
    if n > 4:
        w[3] = 0.0
    # what a masked row carries is not read
    dead = (t < 0) | (w == 0)
    for v in (old, ref, adv):
        v[dead] = math.nan
    w[t < 0] = math.nan
    return old, ref, adv, w


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}ld{s[2]}@{s[3]}")
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("form", ["full", "plain", "stats"])
def test_policy(ce, shape, dtype, form):
    n, v, ld, off = shape
    full = form == "full"
    temperature = f32(1.3) if full else 1.0
    lo, hi = f32(0.2), f32(0.28)
    reduction = {"full": ["mean", "sum", "none"][n % 3], "plain": "mean", "stats": "sum"}[form]
    g, buf, x, t = make(n, v, dtype, n * 17 + v, ld, off, int32=n % 2 == 0)
    old, ref, adv, w = policy_inputs(g, x, t, temperature, lo, hi)
    kl, ent = (f32(0.05), f32(0.01)) if full else (0.0, 0.0)
    kw = dict(clip_low=lo, clip_high=hi, kl_coef=kl, entropy_coef=ent, temperature=temperature, reduction=reduction)
    up = (rnd(g, n if reduction == "none" else 1).abs() + 0.1) if full else None
    if dtype == "f16":
        up = torch.full((n if reduction == "none" else 1,), 64.0, device="cuda")
    if form == "plain":
        adv[(t < 0)] = math.nan
        want = L.policy_ref(x, t, adv, None, None, None, lo, hi, 0.0, 0.0, 1.0, reduction, up)
        adv[(t >= 0) & adv.isnan()] = 0.5     # weight-0 rows of policy_inputs take part without weights
        want = L.policy_ref(x, t, adv, None, None, None, lo, hi, 0.0, 0.0, 1.0, reduction, up)
        old = ref = w = None
        stats = None
    else:
        want = L.policy_ref(x, t, adv, old, ref, w, lo, hi, kl, ent, temperature, reduction, up)
        stats = torch.full((n, 4), 7.0, device="cuda")
    x_in = buf.clone()
    ws = torch.full((ce.ce_workspace_size(n),), 255, dtype=torch.uint8, device="cuda")
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, old_logp=old, ref_logp=ref, row_weight=w, grad_output=up, ws=ws,
                                      grad=torch.empty(n, v, dtype=DT[dtype], device="cuda"), row_stats=stats, **kw)
    torch.cuda.synchronize()
    assert torch.equal(buf, x_in)
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(grad, want["grad"], want["tol_grad"], "gradient")
    if stats is not None:
        L.check(stats, want["stats"], want["tol_stats"], "row statistics")
    assert ce.ce_get_status(ws) == (0 if want["live"].any() or reduction != "mean" else 2)
    loss2, same = ce.ce_policy_fwd_bwd(x, t, adv, old_logp=old, ref_logp=ref, row_weight=w, grad_output=up,
                                       row_stats=stats, **kw)
    assert same.data_ptr() == x.data_ptr()
    L.check(x, want["grad"], want["tol_grad"], "gradient in place")
    assert torch.equal(loss2, loss)
    outside_unchanged(buf, x_in, off, v)


@pytest.mark.parametrize("row_kb", [17, 24, 32, 33, 47.9, 48, 48.1, 60])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ignored", [0.0, 0.6])
def test_policy_rows_of_a_few_chunks(ce, row_kb, dtype, ignored):
    """Several rows a CTA, of one to four chunks, that take part and that do not in any order; other alignments too."""
    n, v = 1300, int(row_kb * 1024) // (4 if dtype == "f32" else 2)
    lo, hi, ent = f32(0.2), f32(0.28), f32(0.01)
    for ld, off, gld, goff in ((v, 0, v, 0), (v + 5, 3, v + 8, 2)):
        g, buf, x, t = make(n, v, dtype, v + off, ld, off, ignored=ignored, int32=off == 3)
        old, ref, adv, w = policy_inputs(g, x, t, 1.0, lo, hi)
        kw = dict(old_logp=old, ref_logp=ref, row_weight=w, clip_low=lo, clip_high=hi, kl_coef=f32(0.05), entropy_coef=ent,
                  reduction="sum")
        want = L.policy_ref(x, t, adv, old, ref, w, lo, hi, f32(0.05), ent, 1.0, "sum", None)
        out = torch.full((n, gld), 7.0, dtype=DT[dtype], device="cuda")
        stats = torch.full((n, 4), 7.0, device="cuda")
        loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, grad=out[:, goff:goff + v], row_stats=stats, **kw)
        L.check(loss, want["loss"], want["tol_loss"], "loss")
        L.check(grad, want["grad"], want["tol_grad"], "gradient")
        L.check(stats, want["stats"], want["tol_stats"], "row statistics")
        outside_unchanged(out, torch.full_like(out, 7.0), goff, v)
        before = buf.clone()
        loss2, _ = ce.ce_policy_fwd_bwd(x, t, adv, **kw)
        L.check(x, want["grad"], want["tol_grad"], "gradient in place")
        assert torch.equal(loss2, loss)
        outside_unchanged(buf, before, off, v)


def test_policy_on_the_clip_border_and_beyond(ce):
    """Ratio exactly 1 with a clip range of no width: the unclipped slope. Advantage 0: no gradient. Far ratios."""
    x = torch.randn(6, 1000, device="cuda")
    t = torch.arange(6, device="cuda")
    adv = torch.tensor([1.0, -1.0, 0.0, 1.0, -1.0, 2.0], device="cuda")
    logp = ce.ce_token_logprob(x, t)[0]
    old = logp.clone()
    old[3] -= 3.0     # ratio e^3, positive advantage: clipped, no gradient
    old[4] += 3.0     # ratio e^-3, negative advantage: clipped, no gradient
    old[5] += 40.0    # ratio e^-40: unclipped, gradient nearly 0
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, old_logp=old, clip_low=0.0, clip_high=0.0, reduction="none",
                                      grad=torch.empty_like(x))
    zeros = torch.zeros(6, device="cuda")
    _, logq, _, _ = L.rows_ref(x, t)
    ref = L.grad_ref(logq, t >= 0, t, torch.where(torch.arange(6, device="cuda") < 2, -adv, zeros), zeros)
    assert (grad[:2].double() - ref[:2]).abs().max() < 1e-5
    assert (grad[2:5] == 0).all() and grad[5].abs().max() < 1e-15
    assert (loss.double() - torch.tensor([-1.0, 1.0, 0.0, -1.0, 1.0, -2 * math.exp(-40)], device="cuda")).abs().max() < 1e-5


def test_policy_nothing_live_and_bad_targets(ce):
    x = torch.full((5, 300), math.nan, device="cuda")
    t = torch.full((5,), -100, device="cuda")
    adv = torch.full((5,), math.nan, device="cuda")
    ws = ce.workspace(5)
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, ws=ws, grad=torch.ones_like(x))
    assert loss.item() == 0 and (grad == 0).all() and ce.ce_get_status(ws) == 2
    y, t2, adv2 = torch.randn(5, 300, device="cuda"), torch.tensor([300, 2, -1, 4, -100], device="cuda"), torch.ones(5, device="cuda")
    loss, grad = ce.ce_policy_fwd_bwd(y, t2, adv2, ws=ws, grad=torch.ones_like(y))
    assert ce.ce_get_status(ws) == 1
    assert abs(loss.item() + 1.0) < 1e-6 and (grad[[0, 2, 4]] == 0).all() and (grad[[1, 3]] != 0).all()
    # no rows at all
    e = torch.empty(0, 300, device="cuda")
    z = torch.empty(0, device="cuda")
    loss, grad = ce.ce_policy_fwd_bwd(e, t[:0], z, ws=ws)
    assert loss.item() == 0 and grad.shape == (0, 300)
    assert ce.ce_token_logprob(e, t[:0])[0].shape == (0,)
    out = ce.ce_token_logprob_backward(e, t[:0], torch.empty(0, 4, device="cuda"), z)
    assert out.shape == (0, 300)
    loss, seq, grad = ce.ce_preference_fwd_bwd(e, t[:0], torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert loss.item() == 0 and (seq == 0).all()


def test_policy_autograd(ce):
    g, _, x, t = make(40, 2000, "f32", 9)
    old, ref, adv, w = policy_inputs(g, x, t, 1.0, 0.2, 0.2)
    lo = f32(0.2)
    kw = dict(old_logp=old, ref_logp=ref, row_weight=w, clip_low=lo, clip_high=lo, kl_coef=f32(0.1), entropy_coef=f32(0.02))
    for reduction in ("mean", "sum", "none"):
        a = x.clone().requires_grad_()
        loss = ce.policy_loss(a * 1.0, t, adv, reduction=reduction, **kw)
        up = torch.tensor(1.7, device="cuda") if reduction != "none" else rnd(g, 40)
        loss.backward(up)
        want = L.policy_ref(x, t, adv, old, ref, w, lo, lo, f32(0.1), f32(0.02), 1.0, reduction, up.reshape(-1))
        L.check(a.grad, want["grad"], want["tol_grad"] + 2.0 ** -23 * want["grad"].abs(), "gradient")
    h = (x * 1.0).requires_grad_()
    loss = ce.policy_loss(h, t, adv, inplace=True, **kw)
    (gh,) = torch.autograd.grad(loss, h, retain_graph=True)
    assert gh.data_ptr() == h.data_ptr()
    with pytest.raises(ce.CEError, match="used up"):
        loss.backward()


# ---------------------------------------------------------------------- preference loss
def pair_offsets(lengths, int32):
    o = torch.tensor([0] + lengths).cumsum(0).cuda()
    return o.int() if int32 else o


PAIRS = [
    # lengths of the 2 P sequences, rows after the last, vocab, row stride, first column
    ([1, 1], 0, 50, 50, 0), ([3, 2, 4, 1], 2, 1000, 1003, 1), ([5, 0, 2, 7, 3, 1], 3, 513, 513, 0),
    ([40, 30, 20, 50], 0, 8192, 8192, 0), ([300, 700], 5, 2001, 2001, 0), ([2, 3], 1, 131075, 131075, 0),
    ([0, 0, 0, 0], 4, 100, 100, 0), ([1] * 700, 0, 64, 64, 0),
]


@pytest.mark.parametrize("case", PAIRS, ids=lambda c: f"{len(c[0]) // 2}pairs{sum(c[0])}+{c[1]}x{c[2]}")
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
def test_preference(ce, case, dtype, kind):
    lengths, extra, v, ld, off = case
    n, pairs = sum(lengths) + extra, len(lengths) // 2
    i = PAIRS.index(case) + {"sigmoid": 0, "hinge": 1, "squared": 2}[kind]
    reduction, normalize = ["mean", "sum", "none"][i % 3], i % 2 == 1
    g, buf, x, t = make(n, v, dtype, 100 + i, ld, off, int32=i % 2 == 0)
    if extra:
        x[n - extra:] = math.nan      # rows of no sequence are not read
        t[n - extra:] = 0
    offsets = pair_offsets(lengths, i % 2 == 1)
    beta, eps = f32(0.3), f32(0.1) if kind == "sigmoid" else 0.0
    logp = torch.where(t >= 0, L.rows_ref(x, t)[2], 0.0)
    seq = torch.stack([logp[b:e].sum() for b, e in zip(offsets[:-1].tolist(), offsets[1:].tolist())])
    ref = (seq + rnd(g, 2 * pairs, 4.0)).float() if i % 4 != 3 else None
    up = None if i % 3 == 0 else rnd(g, pairs if reduction == "none" else 1).abs() + 0.2
    want = L.preference_ref(x, t, offsets, ref, kind, beta, eps, normalize, reduction, up)
    before = buf.clone()
    ws_size = 2 ** 12 + 20 * n + 8 * pairs
    ws = torch.full((ws_size,), 255, dtype=torch.uint8, device="cuda")
    kw = dict(ref_logp=ref, loss_kind=kind, beta=beta, label_smoothing=eps, length_normalize=normalize,
              reduction=reduction, grad_output=up, ws=ws)
    loss, got_seq, grad = ce.ce_preference_fwd_bwd(x, t, offsets, grad=torch.empty(n, v, dtype=DT[dtype], device="cuda"), **kw)
    torch.cuda.synchronize()
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(got_seq, want["seq"], want["tol_seq"], "sequence values")
    L.check(grad, want["grad"].nan_to_num(0.0), want["tol_grad"].nan_to_num(0.0), "gradient")
    live = any(a and b for a, b in zip(lengths[:pairs], lengths[pairs:]))
    flags = ce.ce_get_status(ws)
    assert flags in (0, 2) and (flags == 2 or live)
    loss2, _, same = ce.ce_preference_fwd_bwd(x, t, offsets, **kw)
    assert same.data_ptr() == x.data_ptr() and torch.equal(loss2, loss)
    assert torch.equal(same, grad)
    outside_unchanged(buf, before, off, v)


@pytest.mark.parametrize("offsets", [[0, 5, 3], [0, 3, 7], [-1, 2, 4], [3, 2, 1], [0, 2 ** 31, 4], [2 ** 40, 2 ** 41, 2 ** 42]])
def test_preference_bad_offsets(ce, offsets):
    """Offsets that fall or leave the rows: loss NaN, gradient 0, a status bit, no access outside."""
    x, t = torch.randn(6, 200, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    ws = torch.empty(8192, dtype=torch.uint8, device="cuda")
    for reduction in ("mean", "sum", "none"):
        loss, seq, grad = ce.ce_preference_fwd_bwd(x, t, torch.tensor(offsets, device="cuda"), ws=ws, reduction=reduction,
                                                   grad=torch.ones_like(x))
        assert loss.isnan().all() and seq.isnan().all() and (grad == 0).all()
        assert ce.ce_get_status(ws) == ce.CE_FLAG_BAD_OFFSETS


def test_preference_bad_targets_and_dead_pairs(ce):
    x = torch.randn(8, 100, device="cuda")
    t = torch.tensor([1, 2, -100, -100, 3, 100, 4, 5], device="cuda")
    off = torch.tensor([0, 2, 4, 6, 8], device="cuda")     # the second pair's preferred side is all ignored
    ws = torch.empty(8192, dtype=torch.uint8, device="cuda")
    loss, seq, grad = ce.ce_preference_fwd_bwd(x, t, off, ws=ws, grad=torch.ones_like(x))
    want = L.preference_ref(x, t, off, None, "sigmoid", f32(0.1), 0.0, False, "mean", None)
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(grad, want["grad"], want["tol_grad"], "gradient")
    assert (grad[[2, 3, 5, 6, 7]] == 0).all()
    assert ce.ce_get_status(ws) == 1


def test_preference_far_margins(ce):
    """A margin far on either side: the loss and slope saturate, nothing overflows."""
    x, t = torch.randn(4, 60, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    off = torch.tensor([0, 1, 2, 3, 4], device="cuda")
    ref = torch.tensor([5e3, -5e3, 0.0, 0.0], device="cuda")
    loss, _, grad = ce.ce_preference_fwd_bwd(x, t, off, ref_logp=ref, beta=1.0, reduction="none", grad=torch.empty_like(x))
    want = L.preference_ref(x, t, off, ref, "sigmoid", 1.0, 0.0, False, "none", None)
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(grad, want["grad"], want["tol_grad"], "gradient")
    assert (grad[1] == 0).all() and loss[1] == 0


def test_preference_autograd(ce):
    g, _, x, t = make(30, 900, "f32", 21)
    off = pair_offsets([6, 9, 5, 10], False)
    for reduction in ("mean", "sum"):
        a = x.clone().requires_grad_()
        seq = torch.empty(4, device="cuda")
        loss = ce.preference_loss(a * 1.0, t, off, beta=0.5, reduction=reduction, seq_logp=seq)
        (2.5 * loss).backward()
        want = L.preference_ref(x, t, off, None, "sigmoid", 0.5, 0.0, False, reduction, torch.tensor([2.5], device="cuda"))
        L.check(a.grad, want["grad"], want["tol_grad"] + 2.0 ** -23 * want["grad"].abs(), "gradient")
        L.check(seq, want["seq"], want["tol_seq"], "sequence values")


# ---------------------------------------------------------------------- together
def test_training_step_of_a_policy(ce):
    """The operators as a training step uses them: the old and the reference
    policy scored, the policy loss and its gradient, the same gradient from
    the log-probabilities and a loss written with torch."""
    g, _, x, t = make(96, 4001, "f32", 33)
    with torch.no_grad():
        old = ce.ce_token_logprob(x + 0.05 * torch.randn(x.shape, generator=g, device="cuda"), t, with_entropy=False)[0]
        ref = ce.ce_token_logprob(x + 0.1 * torch.randn(x.shape, generator=g, device="cuda"), t, with_entropy=False)[0]
    adv = rnd(g, 96)
    a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
    stats = torch.empty(96, 4, device="cuda")
    loss = ce.policy_loss(a, t, adv, old_logp=old, ref_logp=ref, kl_coef=0.1, entropy_coef=0.01, row_stats=stats)
    loss.backward()
    logp, ent = ce.token_logprob(b, t, with_entropy=True)
    ratio = (logp - old).exp()
    gap = ref - logp
    row = -torch.minimum(adv * ratio, adv * ratio.clamp(0.8, 1.2)) + 0.1 * (gap.exp() - gap - 1) - 0.01 * ent
    keep = t >= 0
    other = row[keep].sum() / keep.sum()
    other.backward()
    assert abs(loss.item() - other.item()) < 1e-5
    assert (a.grad - b.grad).abs().max() < 1e-6
    assert torch.equal(stats[:, 0], logp.detach()) and torch.equal(stats[:, 1], ent.detach())


def test_graph_replay_and_other_stream(ce):
    """Captured once and replayed on new inputs; and a call on a stream that is not the current one."""
    n, v = 24, 3000
    g, _, x, t = make(n, v, "bf16", 41)
    old, ref, adv, w = policy_inputs(g, x, t, 1.0, 0.2, 0.2)
    w = w.nan_to_num(1.0)
    off = pair_offsets([7, 5, 6, 6], False)
    buf, grad, pgrad = x.clone(), torch.empty_like(x), torch.empty_like(x)
    ws, pws = ce.workspace(n), torch.empty(2 ** 14, dtype=torch.uint8, device="cuda")

    def step():
        loss, _ = ce.ce_policy_fwd_bwd(buf, t, adv, old_logp=old, ref_logp=ref, row_weight=w, kl_coef=0.1, grad=grad, ws=ws)
        pl, seq, _ = ce.ce_preference_fwd_bwd(buf, t, off, grad=pgrad, ws=pws)
        logp, ent, _ = ce.ce_token_logprob(buf, t)
        return loss, pl, seq, logp, ent
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2):
        buf.copy_(make(n, v, "bf16", 41 + seed)[2])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs] + [grad.clone(), pgrad.clone()]
        want = [o.clone() for o in step()] + [grad.clone(), pgrad.clone()]
        for a, b in zip(got, want):
            assert torch.equal(a, b) or torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = ce.ce_policy_fwd_bwd(buf, t, adv, old_logp=old, ref_logp=ref, row_weight=w, kl_coef=0.1,
                               grad=torch.empty_like(x), stream=other)
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda.synchronize()
    want = ce.ce_policy_fwd_bwd(buf, t, adv, old_logp=old, ref_logp=ref, row_weight=w, kl_coef=0.1, grad=torch.empty_like(x))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gradient_beside_the_logits(ce):
    """The gradient in the other half of the same buffer's columns, and in a buffer of another alignment."""
    g, _, x, t = make(12, 1001, "bf16", 51)
    adv = rnd(g, 12)
    # the exponent takes one rounding more or less by where a row lies, so the two
    # gradients are each held to the fp64 form and not to one another's bits
    want = L.policy_ref(x, t, adv, None, None, None, 0.2, 0.2, 0.0, 0.0, 1.0, "mean", None)
    wide = torch.zeros(12, 2003, dtype=torch.bfloat16, device="cuda")
    wide[:, :1001] = x
    ce.ce_policy_fwd_bwd(wide[:, :1001], t, adv, grad=wide[:, 1002:])
    L.check(wide[:, 1002:], want["grad"], want["tol_grad"], "gradient beside the logits")
    assert torch.equal(wide[:, :1001], x) and (wide[:, 1001] == 0).all()
    L.check(ce.ce_policy_fwd_bwd(x, t, adv, grad=torch.empty_like(x))[1], want["grad"], want["tol_grad"], "gradient")
    with pytest.raises(ce.CEError):
        ce.ce_policy_fwd_bwd(wide[:, :1001], t, adv, grad=wide[:, 1000:2001])


def test_no_second_derivative(ce):
    """A second differentiation is refused, not answered with nothing."""
    x, t = torch.randn(4, 50, device="cuda", requires_grad=True), torch.zeros(4, dtype=torch.int64, device="cuda")
    (g,) = torch.autograd.grad(ce.token_logprob(x, t).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.square().sum().backward()
    (g,) = torch.autograd.grad(ce.policy_loss(x, t, torch.ones(4, device="cuda")), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.square().sum().backward()


def test_argument_errors(ce):
    x, t = torch.randn(4, 10, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    adv = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="advantage"):
        ce.ce_policy_fwd_bwd(x, t, adv[:3])
    with pytest.raises(ValueError, match="advantage"):
        ce.ce_policy_fwd_bwd(x, t, adv.double())
    with pytest.raises(ValueError, match="old_logp"):
        ce.ce_policy_fwd_bwd(x, t, adv, old_logp=adv.cpu())
    with pytest.raises(ValueError, match="live on"):
        ce.ce_policy_fwd_bwd(x, t.cpu(), adv)
    with pytest.raises(ce.CEError, match="INVALID_ARG"):
        ce.ce_policy_fwd_bwd(x, t, adv, kl_coef=0.1)
    with pytest.raises(ce.CEError, match="INVALID_ARG"):
        ce.ce_token_logprob(x, t, temperature=0.0)
    with pytest.raises(ce.CEError, match="WORKSPACE"):
        ce.ce_policy_fwd_bwd(x, t, adv, ws=torch.empty(128, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="ref_logp"):
        ce.ce_preference_fwd_bwd(x, t, torch.tensor([0, 2, 4], device="cuda"), ref_logp=adv)
