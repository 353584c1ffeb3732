"""Token log-probabilities of a linear head and their gradient on the GPU
against fp64.

Tolerances: a logit is a sum of H exact bf16 products in fp32, each addition
off by at most 2^-23 of the sum of magnitudes (the bound of the GEMM's own
tests): ez = H 2^-23 |h| |W|^T. log p moves by at most ez_t + max_c ez_c (LSE
is 1-Lipschitz in the maximum norm), H by sum p |log p + H| 2 ez, p relatively
by twice the largest ez; the row arithmetic adds what lp_check.py derives. dZ
is rounded once to bf16 (2^-9, doubled for the products' own sums) and each
output once to its type."""
import math

import pytest
import torch

import lp_check as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ce():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import softmax_cross_entropy_pass_gb300 as ce
    return ce


def f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


def make(n, H, V, seed, bias=False, ignored=0.3, int32=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(V, H, generator=g, device="cuda") * 0.05).bfloat16()
    h = torch.randn(n, H, generator=g, device="cuda")
    t = torch.randint(0, V, (n,), generator=g, device="cuda")
    h = (h + 3.0 * torch.rand(n, 1, generator=g, device="cuda") * w[t].float() / w[t].float().norm(dim=1, keepdim=True)).bfloat16()
    drop = torch.rand(n, generator=g, device="cuda") < ignored
    drop[0] = False
    if n > 2:
        t[1], t[2] = V - 1, 0
    t[drop] = -100
    h[drop] = math.nan      # masked rows may hold anything
    b = torch.randn(V, generator=g, device="cuda") if bias else None
    return g, h, w, (t.int() if int32 else t), b


def reference(h, w, t, b, temperature, gl, gh):
    ok = t >= 0
    hd = torch.where(ok[:, None], h.double(), 0.0)
    z = hd @ w.double().t()
    ez = (hd.abs() @ w.double().abs().t()) * (h.shape[1] * 2.0 ** -23) + 1e-30
    if b is not None:
        z = z + b.double()
        ez = ez + 2 * L.U * z.abs()
    valid, logq, logp, ent = L.rows_ref(z, t, temperature)
    e = ez / temperature
    d = L.delta(z, temperature)
    rows = torch.arange(len(t), device=t.device)
    e_t = e[rows, t.long().clamp_min(0)]
    p = logq.exp()
    out = dict(logp=logp, ent=ent)
    out["tol_logp"] = (L.tol_logp(d, logp) + e_t + e.amax(1)) * valid
    out["tol_ent"] = (L.tol_entropy(d, ent) + 2 * (p * (logq.abs() + ent[:, None]) * e).sum(1)) * valid
    dz = L.grad_ref(logq, valid, t, gl, gh, temperature)
    zero = torch.zeros_like(gl)
    td = L.tol_grad(z, dz, logq, valid, t, gl, gh, zero, zero, torch.bfloat16, temperature)
    size = L.tol_grad(z, dz * 0, logq, valid, t, gl, gh, gl * 0 + gl.abs(), gh.abs(), torch.float32, temperature)
    td = td + size * 4 * e.amax(1, keepdim=True)
    wd = w.double()
    out["gh"], out["tol_gh"] = dz @ wd, (td + 2.0 ** -9 * dz.abs()) @ wd.abs()
    out["gw"], out["tol_gw"] = dz.t() @ hd, (td + 2.0 ** -9 * dz.abs()).t() @ hd.abs()
    out["gb"], out["tol_gb"] = dz.sum(0), (td + 2.0 ** -9 * dz.abs()).sum(0) + 1e-30
    return out


SHAPES = [
    # rows, H, V
    (1, 64, 256), (1, 8, 1), (3, 72, 1001), (16, 128, 50257), (127, 64, 513), (128, 256, 300), (129, 256, 1000),
    (200, 136, 4099), (600, 128, 2051), (1100, 192, 777), (65, 64, 70000), (33, 72, 3001), (64, 200, 4097),
    (2, 1000, 999), (17, 2056, 33), (300, 2048, 520),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("entropy", [False, True])
def test_linear_token_logprob(ce, shape, bias, entropy):
    n, H, V = shape
    temperature = f32(0.8) if n % 2 else 1.0
    g, h, w, t, b = make(n, H, V, n + H + V, bias, int32=n % 3 == 0)
    gl = torch.randn(n, generator=g, device="cuda")
    gh = torch.randn(n, generator=g, device="cuda") if entropy else None
    ref = reference(h, w, t, b, temperature, gl, gh if entropy else gl * 0)
    logp, ent, stats = ce.flce_token_logprob(h, w, t, bias=b, temperature=temperature, with_entropy=entropy)
    L.check(logp, ref["logp"], ref["tol_logp"], "logp")
    if entropy:
        L.check(ent, ref["ent"], ref["tol_ent"], "entropy")
    for chunk, dtype in ((None, torch.float32), (None, torch.bfloat16), (max(1, n // 3 + 1), torch.float32), (64, torch.float32)):
        gw = torch.empty(V, H, dtype=dtype, device="cuda")
        a, gw, gb = ce.flce_token_logprob_backward(h, w, t, stats, gl, grad_entropy=gh, bias=b, temperature=temperature,
                                                   chunk_rows=chunk, grad_weight=gw)
        L.check(a, ref["gh"], ref["tol_gh"] + 2.0 ** -9 * ref["gh"].abs(), f"grad_hidden, chunk {chunk}")
        step = 2.0 ** -9 if dtype == torch.bfloat16 else n * 2.0 ** -24
        L.check(gw, ref["gw"], ref["tol_gw"] + step * ref["gw"].abs(), f"grad_weight {dtype}, chunk {chunk}")
        assert (gb is not None) == bias
        if bias:
            L.check(gb, ref["gb"], ref["tol_gb"], f"grad_bias, chunk {chunk}")
        assert (a[t < 0] == 0).all()


def test_linear_nothing_valid_and_no_rows(ce):
    _, h, w, t, b = make(140, 64, 300, 3, True)
    t[:] = -100
    t[5] = 300          # outside the vocabulary: NaN, without a gradient
    logp, ent, stats = ce.flce_token_logprob(h, w, t, bias=b)
    assert logp[5].isnan() and ent[5].isnan()
    assert (logp[t < 0] == 0).all() and (ent[t < 0] == 0).all()
    one = torch.ones(140, device="cuda")
    gh, gw, gb = ce.flce_token_logprob_backward(h, w, t, stats, one, grad_entropy=one, bias=b)
    assert (gh == 0).all() and (gw == 0).all() and (gb == 0).all()
    e, z = h[:0], torch.empty(0, device="cuda")
    assert ce.flce_token_logprob(e, w, t[:0])[0].shape == (0,)
    gh, gw, gb = ce.flce_token_logprob_backward(e, w, t[:0], torch.empty(0, 4, device="cuda"), z, bias=b)
    assert gh.shape == (0, 64) and (gw == 0).all() and (gb == 0).all()


def test_linear_special_bias(ce):
    """A bias of -inf masks columns of the vocabulary; the masked columns have no gradient."""
    g, h, w, t, b = make(9, 64, 700, 5, True, ignored=0.0)
    b[350:] = -math.inf
    t = t % 350
    logp, ent, stats = ce.flce_token_logprob(h, w, t, bias=b)
    want, want_h, _ = ce.flce_token_logprob(h, w[:350].contiguous(), t, bias=b[:350].contiguous())
    assert (logp - want).abs().max() < 1e-5 and (ent - want_h).abs().max() < 1e-5
    gl = torch.randn(9, generator=g, device="cuda")
    _, gw, gb = ce.flce_token_logprob_backward(h, w, t, stats, gl, grad_entropy=gl, bias=b)
    assert gw.isfinite().all() and (gw[350:] == 0).all() and (gb[350:] == 0).all()


def test_linear_autograd_and_differences(ce):
    n, H, V = 150, 64, 1003
    g, h, w, t, _ = make(n, H, V, 11)
    b = torch.randn(V, generator=g, device="cuda")
    ha, wa, ba = h.clone().requires_grad_(), w.clone().requires_grad_(), b.clone().requires_grad_()
    gl, ge = torch.randn(n, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda")
    logp, ent = ce.linear_token_logprob(ha, wa, t, bias=ba, with_entropy=True)
    (logp * gl + ent * ge).sum().backward()
    ref = reference(h, w, t, b, 1.0, gl, ge)
    assert ha.grad.dtype == wa.grad.dtype == torch.bfloat16 and ba.grad.dtype == torch.float32
    L.check(ha.grad, ref["gh"], ref["tol_gh"] + 2.0 ** -9 * ref["gh"].abs(), "grad_hidden")
    L.check(wa.grad, ref["gw"], ref["tol_gw"] + 2.0 ** -9 * ref["gw"].abs(), "grad_weight")
    L.check(ba.grad, ref["gb"], ref["tol_gb"], "grad_bias")
    # a difference of the fp64 form along a direction of the weights
    d = torch.randn(V, H, generator=g, device="cuda", dtype=torch.float64)
    hd = torch.where((t >= 0)[:, None], h.double(), 0.0)

    def f(wd):
        _, _, lp, en = L.rows_ref(hd @ wd.t() + b.double(), t)
        return (lp * gl.double() + en * ge.double()).sum()
    num = float((f(w.double() + 1e-6 * d) - f(w.double() - 1e-6 * d)) / 2e-6)
    got = float((wa.grad.double() * d).sum())
    assert abs(got - num) <= float(((ref["tol_gw"] + 2.0 ** -9 * ref["gw"].abs()) * d.abs()).sum()) + 1e-5 * (1 + abs(num))
    only = ce.linear_token_logprob(ha, wa, t)
    assert torch.autograd.grad(only.sum(), [ha, wa])[1].isfinite().all()


def test_linear_policy_step(ce):
    """A policy loss over a linear head: log-probabilities from the hidden
    states, the loss in torch, against the same loss over stored logits."""
    n, H, V = 96, 128, 2000
    g, h, w, t, _ = make(n, H, V, 13, ignored=0.2)
    keep = t >= 0
    adv, shift = torch.randn(n, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda") * 0.3
    h = torch.where(keep[:, None], h, torch.zeros_like(h))
    old = ce.flce_token_logprob(h, w, t, with_entropy=False)[0] - shift
    ha, wa = h.clone().requires_grad_(), w.clone().requires_grad_()
    logp, ent = ce.linear_token_logprob(ha, wa, t, with_entropy=True)
    ratio = (logp - old).exp()
    row = -torch.minimum(adv * ratio, adv * ratio.clamp(0.8, 1.2)) - 0.01 * ent
    loss = row[keep].sum() / keep.sum()
    loss.backward()
    logits = (h.float() @ w.float().t()).requires_grad_()
    other = ce.policy_loss(logits, t, adv, old_logp=old, entropy_coef=0.01)
    other.backward()
    assert abs(loss.item() - other.item()) < 1e-4
    dz = logits.grad.double()
    tol = (dz.abs() * 2.0 ** -7) @ w.double().abs() + 1e-6
    assert ((ha.grad.double() - dz @ w.double()).abs() <= tol).all()


def test_linear_graph_replay(ce):
    _, h, w, t, b = make(300, 64, 1000, 17, True)
    n = 300
    gl = torch.randn(n, device="cuda")
    hb = h.clone()

    def step():
        logp, ent, stats = ce.flce_token_logprob(hb, w, t, bias=b)
        return (logp, ent) + ce.flce_token_logprob_backward(hb, w, t, stats, gl, grad_entropy=gl, bias=b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    hb.copy_(make(300, 64, 1000, 18, True)[1].nan_to_num(0.5))
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    for a, c in zip(got, step()):
        assert torch.equal(a, c)


def test_linear_refusals(ce):
    _, h, w, t, b = make(8, 64, 100, 19, True, ignored=0.0)
    with pytest.raises(TypeError, match="bf16"):
        ce.flce_token_logprob(h.float(), w, t)
    with pytest.raises(ValueError, match="contiguous"):
        ce.flce_token_logprob(h[:, :32], w, t)
    with pytest.raises(ValueError, match="columns"):
        ce.flce_token_logprob(h[:, :32].contiguous(), w, t)
    with pytest.raises(ValueError, match="bias"):
        ce.flce_token_logprob(h, w, t, bias=b[:50])
    with pytest.raises(ce.CEError, match="UNSUPPORTED"):
        ce.flce_token_logprob(h[:, :60].contiguous(), w[:, :60].contiguous(), t)
    with pytest.raises(ce.CEError, match="WORKSPACE"):
        ce.flce_token_logprob(h, w, t, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    _, _, stats = ce.flce_token_logprob(h, w, t)
    one = torch.ones(8, device="cuda")
    with pytest.raises(ce.CEError, match="UNSUPPORTED"):
        ce.flce_token_logprob_backward(h, w, t, stats, one, chunk_rows=4,
                                       grad_weight=torch.empty(100, 64, dtype=torch.bfloat16, device="cuda"))
