"""The log-probability operators on logits, margins and ratios far from the
ordinary: finite masks and maxima of any magnitude, gradients under a loss
scale, -inf on one side of a pair. Against the fp64 forms of lp_check.py, which
derives the tolerances."""
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


# ---------------------------------------------------------------------- finite logits of any magnitude
def masks(dtype):
    low = torch.finfo(DT[dtype]).min
    return (-1e4, low) if dtype == "f16" else (-1e4, -1e6, -1e9, -1e10, -1e12, -1e30, -1e37, low)


def far_rows(v, dtype, seed):
    """Rows whose leading columns, all but 500 columns, or all columns hold a
    finite mask; the same with the target masked, where its log-probability is
    one of fp32; rows far above 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, targets = [], []
    for m in masks(dtype):
        for form in ("leading", "few", "all", "target"):
            if form == "target" and m < -1e30:
                continue
            x = torch.randn(v, generator=g, device="cuda") * 2
            few = torch.randperm(v, generator=g, device="cuda")[:500]
            t = int(few[0])
            if form == "leading":
                x[:min(8192, v - 1)] = m
                t = v - 1
            elif form == "all":
                x[:] = m
            else:
                kept = x[few].clone()
                x[:] = m
                x[few] = kept
                if form == "target":
                    x[t] = m
            rows.append(x)
            targets.append(t)
    for shift in (100.0, -300.0, 5e3):
        rows.append(torch.randn(v, generator=g, device="cuda") + shift)
        targets.append(v // 2)
    return g, torch.stack(rows).to(DT[dtype]), torch.tensor(targets, device="cuda")


@pytest.mark.parametrize("row_kb", [12, 17, 50, 200])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("temperature", [1e-3, 0.01, 0.7, 1.0, 5.0, 10.0])
def test_far_logits(ce, row_kb, dtype, temperature):
    temperature = f32(temperature)
    v = int(row_kb * 1024) // (4 if dtype == "f32" else 2) - 3
    g, base, bt = far_rows(v, dtype, v)
    n = len(bt)
    valid, logq, want, want_h = L.rows_ref(base, bt, temperature)
    d = L.delta(base, temperature)
    gl, gh, z = (torch.randn(n, generator=g, device="cuda") for _ in range(3))
    z.zero_()
    ref = L.grad_ref(logq, valid, bt, gl, gh, temperature)
    tol = L.tol_grad(base, ref, logq, valid, bt, gl, gh, z, z, DT[dtype], temperature)
    ent_coef = f32(0.03)
    pol = L.policy_ref(base, bt, gl, None, None, None, 0.2, 0.2, 0.0, ent_coef, temperature, "none", None)
    bare = L.policy_ref(base, bt, gl, None, None, None, 0.2, 0.2, 0.0, 0.0, temperature, "none", None)
    # few rows (clusters of CTAs a row) and more rows than CTAs; rows that start anywhere
    for copies, off in ((1, 0), (320 // n + 1, 3)):
        x = torch.empty(n * copies, v + 2 * off, dtype=DT[dtype], device="cuda")[:, off:off + v]
        x.copy_(base.repeat(copies, 1))
        t, rep = bt.repeat(copies), lambda a: a.repeat(copies, *[1] * (a.dim() - 1))  # noqa: E731
        logp, ent, stats = ce.ce_token_logprob(x, t, temperature=temperature)
        L.check(logp, rep(want), L.tol_logp(rep(d), rep(want)), "logp")
        L.check(ent, rep(want_h), L.tol_entropy(rep(d), rep(want_h)), "entropy")
        plain = ce.ce_token_logprob(x, t, temperature=temperature, with_entropy=False)[0]
        L.check(plain, rep(want), L.tol_logp(rep(d), rep(want)), "logp without entropy")
        grad = ce.ce_token_logprob_backward(x, t, stats, rep(gl), grad_entropy=rep(gh), temperature=temperature,
                                            grad=torch.empty_like(x))
        L.check(grad, rep(ref), rep(tol), "gradient from statistics")
        kw = dict(temperature=temperature, reduction="none")
        loss, grad = ce.ce_policy_fwd_bwd(x, t, rep(gl), grad=torch.empty_like(x), **kw)
        L.check(loss, rep(bare["loss"]), rep(bare["tol_loss"]), "policy loss")
        L.check(grad, rep(bare["grad"]), rep(bare["tol_grad"]), "policy gradient")
        row = torch.empty(n * copies, 4, device="cuda")
        loss, grad = ce.ce_policy_fwd_bwd(x, t, rep(gl), entropy_coef=ent_coef, row_stats=row, **kw)
        L.check(loss, rep(pol["loss"]), rep(pol["tol_loss"]), "policy loss with the entropy")
        L.check(grad, rep(pol["grad"]), rep(pol["tol_grad"]), "policy gradient with the entropy")
        L.check(row, rep(pol["stats"]), rep(pol["tol_stats"]), "row statistics")


@pytest.mark.parametrize("row_kb", [12, 50, 200])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_far_logits_in_pairs(ce, row_kb, dtype):
    v = int(row_kb * 1024) // (4 if dtype == "f32" else 2)
    _, x, t = far_rows(v, dtype, v)
    keep = L.rows_ref(x, t)[2] > -1e3      # sums of ordinary size
    x, t = x[keep].contiguous(), t[keep].contiguous()
    n = len(t)
    off = torch.tensor([0, n // 4, n // 2, 3 * n // 4, n], device="cuda")
    beta = f32(0.02)
    want = L.preference_ref(x, t, off, None, "sigmoid", beta, 0.0, True, "mean", None)
    loss, seq, grad = ce.ce_preference_fwd_bwd(x, t, off, beta=beta, length_normalize=True, grad=torch.empty_like(x))
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(seq, want["seq"], want["tol_seq"], "sequence values")
    L.check(grad, want["grad"], want["tol_grad"], "gradient")


@pytest.mark.parametrize("v", [20000, 33000, 128256])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_special_long_rows(ce, v, dtype):
    """Rows without a distribution (NaN, +inf, all -inf) among ordinary ones, and
    rows of one value, longer than the register kernel takes."""
    dt = DT[dtype]
    low = torch.finfo(dt).min
    x = torch.randn(16, v, device="cuda").to(dt)
    t = torch.arange(16, device="cuda") * 7
    x[0, 100:] = -math.inf
    x[1, 100:] = low
    x[2] = low
    x[3] = -math.inf
    x[4, v // 2] = math.nan
    x[5, v - 2] = math.inf
    x[6] = math.nan
    t[6] = -100
    x[7] = 0.0
    x[8] = 50000.0 if dtype == "f16" else 3e38
    x[9, :] = -40000.0
    x[9, v // 3] = 60000.0
    x[10, t[10]] = -math.inf
    t[11] = v
    t[12] = -5
    x[13] = -math.inf
    x[13, t[13]] = 1.0
    x[14] = math.nan
    x[15, :9] = math.nan
    x[15, 9:] = -math.inf
    adv = torch.randn(16, device="cuda")
    logp, ent, _ = ce.ce_token_logprob(x, t)
    plain = ce.ce_token_logprob(x, t, with_entropy=False)[0]
    coef = f32(0.1)
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=coef, reduction="none", grad=torch.empty_like(x))
    _, _, want, want_h = L.rows_ref(x, t)
    nan = torch.tensor([3, 4, 5, 14, 15], device="cuda")
    for name, val in (("logp", logp), ("entropy", ent), ("logp without entropy", plain)):
        assert val[nan].isnan().all(), name
        assert val[[11, 12]].isnan().all() and val[6] == 0, name
    assert grad[nan].isnan().any(1).all() and loss[nan].isnan().all()
    assert (grad[[6, 11, 12]] == 0).all() and (loss[[6, 11, 12]] == 0).all()
    assert logp[10] == -math.inf and plain[10] == -math.inf and logp[13] == 0 and ent[13] == 0
    ok = torch.tensor([0, 1, 2, 7, 8, 9, 13], device="cuda")
    d = L.delta(x[ok])
    L.check(logp[ok], want[ok], L.tol_logp(d, want[ok]), "logp")
    L.check(plain[ok], want[ok], L.tol_logp(d, want[ok]), "logp without entropy")
    L.check(ent[ok], want_h[ok], L.tol_entropy(d, want_h[ok]), "entropy")
    ref = L.policy_ref(x[ok], t[ok], adv[ok], None, None, None, 0.2, 0.2, 0.0, coef, 1.0, "none", None)
    L.check(loss[ok], ref["loss"], ref["tol_loss"], "policy loss")
    L.check(grad[ok], ref["grad"], ref["tol_grad"], "policy gradient")


@pytest.mark.parametrize("row_kb", [12, 17, 50, 200])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mask,temperature", [(-1e38, 1.0), (-3.3e38, 5.0), (-2e34, 1e-4)])
def test_far_masks_under_a_large_entropy_gradient(ce, row_kb, dtype, mask, temperature):
    """Masks whose exponent is just within fp32's range, times the entropy's coefficient: probability and gradient 0."""
    n, v, temperature = 330, int(row_kb * 1024) // (4 if dtype == "f32" else 2), f32(temperature)
    g = torch.Generator(device="cuda").manual_seed(v)
    x = torch.randn(n, v, generator=g, device="cuda")
    x[:, 100:v - 100][torch.rand(n, v - 200, generator=g, device="cuda") < 0.3] = mask
    x = x.to(DT[dtype])
    t = torch.randint(0, 100, (n,), generator=g, device="cuda")
    adv, up = torch.randn(n, generator=g, device="cuda"), torch.full((1,), 65536.0, device="cuda")
    coef = f32(0.25)
    want = L.policy_ref(x, t, adv, None, None, None, 0.2, 0.2, 0.0, coef, temperature, "sum", up)
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=coef, temperature=temperature, reduction="sum", grad_output=up,
                                      grad=torch.empty_like(x))
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(grad, want["grad"], want["tol_grad"], "gradient")
    assert (grad[x < -1e30] == 0).all()
    # over the logits, and into rows that lie otherwise
    other = torch.empty(n, v + 3, dtype=DT[dtype], device="cuda")[:, 1:1 + v]
    ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=coef, temperature=temperature, reduction="sum", grad_output=up, grad=other)
    L.check(other, want["grad"], want["tol_grad"], "gradient at other offsets")


# ---------------------------------------------------------------------- margins and ratios at their ends
@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_rejected_sequence_of_probability_zero(ce, eps):
    """A rejected sequence whose target is masked with -inf: the margin is +inf,
    and without smoothing the loss and the gradient are 0."""
    x = torch.randn(4, 300, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    x[2, 0] = -math.inf
    off = torch.tensor([0, 1, 2, 3, 4], device="cuda")
    for reduction in ("none", "mean"):
        loss, seq, grad = ce.ce_preference_fwd_bwd(x, t, off, beta=1.0, label_smoothing=eps, reduction=reduction,
                                                   grad=torch.empty_like(x))
        want = L.preference_ref(x[[1, 3]], t[:2], off[:3], None, "sigmoid", 1.0, f32(eps), False, "none", None)
        assert seq[2] == -math.inf and seq[[0, 1, 3]].isfinite().all()
        if eps:
            assert loss[0] == math.inf     # -eps log sigmoid(-inf)
        elif reduction == "none":
            assert loss[0] == 0
            L.check(loss[1:], want["loss"], want["tol_loss"], "the other pair's loss")
        else:
            L.check(loss, want["loss"] / 2, want["tol_loss"], "loss")
        if not eps:
            assert (grad[[0, 2]] == 0).all()
        scale = 1.0 if reduction == "none" else 0.5
        L.check(grad[[1, 3]], want["grad"] * scale, want["tol_grad"], "the other pair's gradient")


@pytest.mark.parametrize("v", [300, 20000])
def test_policy_far_below_its_reference(ce, v):
    """d kl / d logp = 1 - e^(ref - logp) is 1 however far the reference lies below; its loss then is the gap."""
    gaps = [-30.0, -1e4, -1e6, -3e7, -1e9, -1e20, -math.inf, 20.0, 0.1]
    n = len(gaps)
    x, t = torch.randn(n, v, device="cuda"), torch.arange(n, device="cuda")
    adv = torch.randn(n, device="cuda")
    ref = (L.rows_ref(x, t)[2] + torch.tensor(gaps, dtype=torch.float64, device="cuda")).float()
    kl = f32(0.5)
    want = L.policy_ref(x, t, adv, None, ref, None, 0.2, 0.2, kl, 0.0, 1.0, "none", None)
    stats = torch.empty(n, 4, device="cuda")
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, ref_logp=ref, kl_coef=kl, reduction="none", row_stats=stats,
                                      grad=torch.empty_like(x))
    L.check(loss, want["loss"], want["tol_loss"], "loss")
    L.check(grad, want["grad"], want["tol_grad"], "gradient")
    L.check(stats[:, 3], want["stats"][:, 3], want["tol_stats"][:, 3], "kl")


@pytest.mark.parametrize("v", [300, 20000])
def test_policy_ratio_past_fp32(ce, v):
    """A ratio over fp32's largest value: clipped where the advantage is positive, no part where it is 0."""
    x, t = torch.randn(4, v, device="cuda"), torch.arange(4, device="cuda")
    adv = torch.tensor([0.0, 2.0, -0.0, 1.0], device="cuda")
    old = (L.rows_ref(x, t)[2] - torch.tensor([200.0, 200.0, 90.0, 0.3], device="cuda")).float()
    lo = f32(0.2)
    kw = dict(old_logp=old, clip_low=lo, clip_high=lo, reduction="none")
    want = L.policy_ref(x, t, adv, old, None, None, lo, lo, 0.0, 0.0, 1.0, "none", None)
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, grad=torch.empty_like(x), **kw)
    assert loss[0] == 0 and loss[2] == 0 and (grad[:3] == 0).all()
    assert abs(loss[1].item() + 2 * (1 + lo)) < 1e-6
    L.check(loss[3:], want["loss"][3:], want["tol_loss"][3:], "loss")
    stats = torch.empty(4, 4, device="cuda")
    coef = f32(0.1)
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=coef, row_stats=stats, grad=torch.empty_like(x), **kw)
    _, logq, _, ent = L.rows_ref(x, t)
    z = torch.zeros(4, device="cuda")
    ref = L.grad_ref(logq, t >= 0, t, z, z - coef)
    tol = L.tol_grad(x, ref, logq, t >= 0, t, z, z - coef, z, z, torch.float32)
    L.check(grad[:3], ref[:3], tol[:3], "the entropy's gradient")
    assert stats[0, 2] == math.inf and (loss[[0, 2]].double() + coef * ent[[0, 2]]).abs().max() < 1e-5
    # a token the old policy excluded: e^inf, of which 0 times is not a number
    old[0] = -math.inf
    assert ce.ce_policy_fwd_bwd(x, t, adv, grad=torch.empty_like(x), **kw)[0][0].isnan()


# ---------------------------------------------------------------------- a loss scale in the one rounding
def in_range(want, dtype):
    """A gradient as its type holds it: fp16 rounds from 65520 on (65504 is its
    largest, and the next value it could hold is 65536) to infinity."""
    if dtype != "f16":
        return want
    return torch.where(want.abs() >= 65520.0, torch.sign(want) * math.inf, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_policy_loss_under_a_scale(ce, dtype, reduction):
    """The upstream gradient given to the forward is in the gradient's one rounding: fp16 under a loss scale keeps what it holds."""
    n, v, lo = 4096, 700, f32(0.2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(n, v, generator=g, device="cuda") * 2).to(DT[dtype])
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[::7] = -100
    adv, ref = torch.randn(n, generator=g, device="cuda"), -torch.rand(n, generator=g, device="cuda") * 8
    kw = dict(ref_logp=ref, clip_low=lo, clip_high=lo, kl_coef=f32(0.05), entropy_coef=f32(0.01), reduction=reduction)
    scale = torch.full((n,) if reduction == "none" else (), 65536.0 if reduction == "mean" else 64.0, device="cuda")
    want = L.policy_ref(x, t, adv, None, ref, None, lo, lo, f32(0.05), f32(0.01), 1.0, reduction, scale.reshape(-1))
    want["grad"] = in_range(want["grad"], dtype)
    for inplace in (False, True):
        a = x.clone().requires_grad_()
        loss = ce.policy_loss(a * 1, t, adv, grad_output=scale, inplace=inplace, **kw)
        L.check(loss.detach().reshape(-1), want["loss"], want["tol_loss"], "loss")
        loss.backward(scale)
        L.check(a.grad, want["grad"], want["tol_grad"], "gradient")
    direct = ce.ce_policy_fwd_bwd(x, t, adv, grad_output=scale.reshape(-1), grad=torch.empty_like(x), **kw)[1]
    assert torch.equal(direct, a.grad)
    # an upstream gradient other than the one announced: by the quotient, a second rounding
    a = x.clone().requires_grad_()
    ce.policy_loss(a, t, adv, grad_output=scale, **kw).backward(scale / 4)
    off = torch.finfo(DT[dtype]).eps / 2 * want["grad"].abs().nan_to_num(posinf=0.0) / 4 + (2.0 ** -25 if dtype == "f16" else 0.0)
    L.check(a.grad, want["grad"] / 4, want["tol_grad"] / 4 + 1.01 * off, "gradient by the quotient")
    zero = torch.zeros_like(scale)
    a = x.clone().requires_grad_()
    ce.policy_loss(a, t, adv, grad_output=zero, **kw).backward(zero)
    assert (a.grad == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_preference_loss_under_a_scale(ce, dtype):
    n, v, pairs = 2048, 700, 32
    g = torch.Generator(device="cuda").manual_seed(4)
    x = (torch.randn(n, v, generator=g, device="cuda") * 2).to(DT[dtype])
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[::5] = -100
    off = torch.arange(2 * pairs + 1, device="cuda") * (n // (2 * pairs))
    scale = torch.full((1,), 65536.0, device="cuda")
    beta = f32(0.02)
    want = L.preference_ref(x, t, off, None, "sigmoid", beta, 0.0, True, "mean", scale)
    a = x.clone().requires_grad_()
    loss = ce.preference_loss(a, t, off, beta=beta, length_normalize=True, grad_output=scale)
    (loss * scale[0]).backward()
    L.check(loss.detach().reshape(1), want["loss"], want["tol_loss"], "loss")
    L.check(a.grad, want["grad"], want["tol_grad"], "gradient")


def test_refused_scales(ce):
    x, t, adv = torch.randn(4, 20, device="cuda"), torch.arange(4, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(ValueError, match="grad_output"):
        ce.policy_loss(x, t, adv, grad_output=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError, match="grad_output"):
        ce.policy_loss(x, t, adv, grad_output=torch.ones(1, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError, match="grad_output"):
        ce.policy_loss(x, t, adv, reduction="none", grad_output=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="grad_output"):
        ce.preference_loss(x, t, torch.tensor([0, 2, 4], device="cuda"), grad_output=torch.ones(1))
    with pytest.raises(TypeError, match="grad_output"):
        ce.policy_loss(x, t, adv, grad_output=2.0)


# ---------------------------------------------------------------------- windows of long rows
@pytest.mark.parametrize("ignored", [0.4, 0.6])
def test_windows_of_long_rows(ce, ignored):
    """More rows than one window of the row kernel deals out, each longer than the delayed second pass takes."""
    n, v = 9001, 33000
    g = torch.Generator(device="cuda").manual_seed(int(ignored * 10))
    x = torch.empty(n, v, dtype=torch.bfloat16, device="cuda").normal_(0, 2, generator=g)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[torch.rand(n, generator=g, device="cuda") < ignored] = -100
    adv = torch.randn(n, generator=g, device="cuda")
    stats = torch.full((n, 4), 9.0, device="cuda")
    coef = f32(0.01)
    loss, grad = ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=coef, reduction="sum", row_stats=stats, grad=torch.full_like(x, 3.0))
    total = tol = 0.0
    for r in range(0, n, 500):
        s = slice(r, min(r + 500, n))
        want = L.policy_ref(x[s], t[s], adv[s], None, None, None, 0.2, 0.2, 0.0, coef, 1.0, "sum", None)
        L.check(grad[s], want["grad"], want["tol_grad"], f"gradient of rows from {r}")
        L.check(stats[s], want["stats"], want["tol_stats"], f"row statistics from {r}")
        total, tol = total + float(want["loss"]), tol + float(want["tol_loss"])
    assert abs(loss.item() - total) <= tol + 2 * L.U * abs(total)
    kept = grad.clone()
    ce.ce_policy_fwd_bwd(x, t, adv, entropy_coef=coef, reduction="sum")
    assert torch.equal(x, kept)
