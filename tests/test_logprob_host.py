"""CPU checks of the log-probability operators: the fp64 forms the GPU tests
compare with (against automatic differentiation and central differences) and
the refusals of the C ABI and of the Python entries before any CUDA call."""
import ctypes
import math

import pytest
import torch

import lp_check as L


@pytest.fixture(scope="module")
def ce():
    import softmax_cross_entropy_pass_gb300 as ce
    return ce


# ---------------------------------------------------------------------- the fp64 forms
def _case(n, v, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, v, generator=g, dtype=torch.float64) * 2
    t = torch.randint(0, v, (n,), generator=g)
    t[1] = -100
    return g, x, t


def _differences(f, x, grad, seed, rtol=1e-6):
    g = torch.Generator().manual_seed(seed)
    for _ in range(4):
        d = torch.randn(x.shape, generator=g, dtype=torch.float64)
        d = d / d.norm()
        eps = 1e-5
        num = (f(x + eps * d) - f(x - eps * d)) / (2 * eps)
        assert abs(float(num) - float((grad * d).sum())) <= rtol * (1 + abs(float(num)))


@pytest.mark.parametrize("temperature", [1.0, 0.6, 1.7])
def test_row_gradient_form(temperature):
    g, x, t = _case(7, 23, 1)
    gl, gh = torch.randn(7, generator=g, dtype=torch.float64), torch.randn(7, generator=g, dtype=torch.float64)

    def f(x):
        _, _, lp, h = L.rows_ref(x, t, temperature)
        return (lp * gl + h * gh).sum()
    valid, logq, _, _ = L.rows_ref(x, t, temperature)
    grad = L.grad_ref(logq, valid, t, gl, gh, temperature)
    xa = x.clone().requires_grad_()
    (auto,) = torch.autograd.grad(f(xa), xa)
    assert (auto - grad).abs().max() < 1e-12
    assert grad[1].abs().max() == 0
    _differences(f, x, grad, 2)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_policy_form(reduction):
    g, x, t = _case(9, 31, 3)
    rnd = lambda s=1.0: torch.randn(9, generator=g, dtype=torch.float64) * s  # noqa: E731
    base = L.rows_ref(x, t, 0.8)[2]
    old, ref, adv = base + rnd(0.3), base + rnd(0.4), rnd()
    w = torch.rand(9, generator=g, dtype=torch.float64) + 0.1
    w[3] = 0.0
    up = rnd().abs() if reduction == "none" else torch.tensor([0.7], dtype=torch.float64)

    def f(x):
        valid, _, lp, h = L.rows_ref(x, t, 0.8)
        r = (lp - old).exp()
        gap = ref - lp
        row = -torch.minimum(adv * r, adv * r.clamp(0.8, 1.3)) + 0.1 * (gap.exp() - gap - 1) - 0.05 * h
        row = torch.where(valid, w * row, 0.0)
        total = torch.where(valid, w, 0.0).sum() if reduction == "mean" else 1.0
        return (row / total * up).sum()
    out = L.policy_ref(x, t, adv, old, ref, w, 0.2, 0.3, 0.1, 0.05, 0.8, reduction, up)
    loss = out["loss"] * up if reduction != "none" else out["loss"] * up
    assert abs(float(loss.sum() - f(x))) < 1e-12
    xa = x.clone().requires_grad_()
    (auto,) = torch.autograd.grad(f(xa), xa)
    assert (auto - out["grad"]).abs().max() < 1e-12
    _differences(f, x, out["grad"], 4)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("normalize", [False, True])
def test_preference_form(kind, normalize):
    g, x, t = _case(16, 19, 5)
    off = torch.tensor([0, 3, 3, 7, 9, 12, 14])   # the second preferred sequence is empty
    ref = torch.randn(6, generator=g, dtype=torch.float64)
    eps = 0.1 if kind == "sigmoid" else 0.0

    def f(x):
        valid, _, lp, _ = L.rows_ref(x, t)
        v = []
        for b, e in zip(off[:-1].tolist(), off[1:].tolist()):
            n = max(1, int(valid[b:e].sum()))
            v.append(lp[b:e].sum() / (n if normalize else 1))
        loss = 0.0
        for p in (0, 2):
            h = (v[p] - v[p + 3]) - (ref[p] - ref[p + 3])
            loss = loss + L.pair_losses(h[None], kind, 0.3, eps)[0][0]
        return loss / 2 * 1.7
    out = L.preference_ref(x, t, off, ref, kind, 0.3, eps, normalize, "mean", torch.tensor([1.7], dtype=torch.float64))
    assert abs(float(out["loss"][0] * 1.7 - f(x))) < 1e-12
    xa = x.clone().requires_grad_()
    (auto,) = torch.autograd.grad(f(xa), xa)
    assert (auto - out["grad"]).abs().max() < 1e-12
    assert out["grad"][14:].abs().max() == 0
    _differences(f, x, out["grad"], 6)


# ---------------------------------------------------------------------- refusals of the C ABI
FAKE, WS, NB = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x4000000), 1 << 30


def _p(ce, **kw):
    p = ce.ce_params()
    p.n_rows, p.vocab, p.ld = kw.get("n_rows", 4), kw.get("vocab", 100), kw.get("ld", 100)
    p.dtype, p.reduction, p.ignore_index = kw.get("dtype", 1), kw.get("reduction", 1), -100
    p.target_is_int32, p.variant, p.reserved = kw.get("tgt", 0), kw.get("variant", 0), kw.get("reserved", 0)
    p.label_smoothing, p.softcap, p.z_loss = kw.get("eps", 0.0), kw.get("softcap", 0.0), kw.get("z_loss", 0.0)
    if kw.get("class_weight"):
        p.class_weight = 0x100000
    return p


def _logprob(ce, p, t=1.0, x=FAKE, tgt=FAKE, logp=FAKE, ent=FAKE, stats=FAKE):
    return ce._lib.ce_token_logprob(ctypes.byref(p), t, x, tgt, logp, ent, stats, None)


def _backward(ce, p, t=1.0, x=FAKE, tgt=FAKE, stats=FAKE, g=FAKE, h=None, grad=FAKE, ld=100):
    return ce._lib.ce_token_logprob_backward(ctypes.byref(p), t, x, tgt, stats, g, h, grad, ld, None)


def _policy(ce, p, q=(1.0, 0.2, 0.2, 0.0, 0.0, 0), x=FAKE, tgt=FAKE, adv=FAKE, old=None, ref=None, w=None, up=None, loss=FAKE,
            stats=None, grad=FAKE, ld=100, ws=WS, nb=NB):
    q = ce.ce_policy_params(*q)
    return ce._lib.ce_policy_fwd_bwd(ctypes.byref(p), ctypes.byref(q), x, tgt, adv, old, ref, w, up, loss, stats, grad,
                                     ld, ws, nb, None)


def _preference(ce, p, q=(2, 0, 0, 0, 0.1, 0.0, 0), x=FAKE, tgt=FAKE, off=FAKE, ref=None, loss=FAKE, grad=FAKE, ld=100, ws=WS,
                nb=NB):
    q = ce.ce_preference_params(*q)
    return ce._lib.ce_preference_fwd_bwd(ctypes.byref(p), ctypes.byref(q), x, tgt, off, ref, None, loss, None, grad, ld,
                                         ws, nb, None)


BAD_PARAMS = [dict(n_rows=-1), dict(vocab=0), dict(ld=99), dict(dtype=3), dict(reduction=5), dict(tgt=2),
              dict(variant=1), dict(variant=0x10000), dict(reserved=1)]
UNSUPPORTED = [dict(eps=0.1), dict(softcap=30.0), dict(z_loss=1e-4), dict(class_weight=True)]


@pytest.mark.parametrize("call", [_logprob, _backward, _policy, _preference])
def test_parameter_refusals(ce, call):
    for kw in BAD_PARAMS:
        assert call(ce, _p(ce, **kw)) == ce.CE_ERR_INVALID_ARG, kw
    for kw in UNSUPPORTED:
        assert call(ce, _p(ce, **kw)) == ce.CE_ERR_UNSUPPORTED, kw
    assert call(ce, _p(ce), x=ctypes.c_void_p(0x100001)) == ce.CE_ERR_INVALID_ARG   # not element aligned
    assert call(ce, _p(ce), x=None) == ce.CE_ERR_INVALID_ARG
    assert call(ce, _p(ce), tgt=None) == ce.CE_ERR_INVALID_ARG
    assert call(ce, _p(ce), tgt=ctypes.c_void_p(0x100004)) == ce.CE_ERR_INVALID_ARG   # int64 targets
    assert call(ce, _p(ce, tgt=1), tgt=ctypes.c_void_p(0x100002)) == ce.CE_ERR_INVALID_ARG


@pytest.mark.parametrize("t", [0.0, -1.0, math.nan, math.inf, 1e-5, 1e5])
def test_temperature_refusals(ce, t):
    assert _logprob(ce, _p(ce), t) == ce.CE_ERR_INVALID_ARG
    assert _backward(ce, _p(ce), t) == ce.CE_ERR_INVALID_ARG
    assert _policy(ce, _p(ce), q=(t, 0.2, 0.2, 0.0, 0.0, 0)) == ce.CE_ERR_INVALID_ARG


def test_pointer_refusals(ce):
    p, bad = _p(ce), ce.CE_ERR_INVALID_ARG
    assert _logprob(ce, p, logp=None, ent=None, stats=None) == bad
    assert _logprob(ce, p, stats=ctypes.c_void_p(0x100008)) == bad
    assert _logprob(ce, p, tgt=None) == bad
    assert _backward(ce, p, g=None) == bad
    assert _backward(ce, p, stats=None) == bad
    assert _backward(ce, p, grad=None, x=FAKE) == bad
    assert _policy(ce, p, adv=None) == bad
    assert _policy(ce, p, loss=None) == bad
    assert _policy(ce, p, stats=ctypes.c_void_p(0x100004)) == bad
    assert _preference(ce, p, off=None) == bad
    assert _preference(ce, p, off=ctypes.c_void_p(0x100004)) == bad     # int64 offsets, 4-byte aligned


@pytest.mark.parametrize("q", [(1.0, -0.1, 0.2, 0, 0, 0), (1.0, 1.1, 0.2, 0, 0, 0), (1.0, 0.2, -0.1, 0, 0, 0),
                               (1.0, 0.2, 0.2, -1.0, 0, 0), (1.0, 0.2, 0.2, math.nan, 0, 0),
                               (1.0, 0.2, 0.2, 0.1, 0, 0), (1.0, 0.2, 0.2, 0, math.inf, 0), (1.0, 0.2, 0.2, 0, 0, 1)])
def test_policy_refusals(ce, q):
    """(a KL coefficient without reference log-probabilities among them)"""
    assert _policy(ce, _p(ce), q=q) == ce.CE_ERR_INVALID_ARG


@pytest.mark.parametrize("q", [(-1, 0, 0, 0, 0.1, 0.0, 0), (2, 3, 0, 0, 0.1, 0.0, 0), (2, 0, 2, 0, 0.1, 0.0, 0),
                               (2, 0, 0, 2, 0.1, 0.0, 0), (2, 0, 0, 0, 0.0, 0.0, 0), (2, 0, 0, 0, math.nan, 0.0, 0),
                               (2, 0, 0, 0, 0.1, 0.6, 0), (2, 1, 0, 0, 0.1, 0.1, 0), (2, 0, 0, 0, 0.1, 0.0, 1)])
def test_preference_refusals(ce, q):
    assert _preference(ce, _p(ce), q=q) == ce.CE_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_policy, _preference])
def test_workspace_refusals(ce, call):
    p = _p(ce)
    assert call(ce, p, ws=None) == ce.CE_ERR_WORKSPACE
    assert call(ce, p, ws=ctypes.c_void_p(0x4000010)) == ce.CE_ERR_WORKSPACE
    assert call(ce, p, nb=64) == ce.CE_ERR_WORKSPACE


@pytest.mark.parametrize("call", [_backward, _policy, _preference])
def test_gradient_buffer_refusals(ce, call):
    """The gradient buffer is the logits with their stride, or shares no element with them."""
    p, bad = _p(ce, ld=300), ce.CE_ERR_INVALID_ARG
    at = lambda b: ctypes.c_void_p(0x100000 + b)  # noqa: E731
    assert call(ce, p, ld=99) == bad
    assert call(ce, p, ld=301) == bad                        # the same buffer, another stride
    assert call(ce, p, ld=300, grad=at(2)) == bad             # shifted by a column
    assert call(ce, p, ld=300, grad=at(2 * 300)) == bad       # shifted by a row
    assert call(ce, p, ld=300, grad=at(2 * 99)) == bad        # the last logits column
    assert call(ce, p, ld=300, grad=at(2 * 201)) == bad       # the next row's first column
    assert call(ce, p, ld=400, grad=at(2 * 100)) == bad       # beside it, but another stride
    assert call(ce, p, ld=300, grad=at(2 * 100 + 1)) == bad   # not element aligned


def test_preference_workspace_size(ce):
    out = ctypes.c_size_t()
    for n, pairs in ((0, 0), (1, 1), (1000, 37), (8192, 512)):
        p = _p(ce, n_rows=n)
        assert ce._lib.ce_preference_workspace_size(ctypes.byref(p), pairs, ctypes.byref(out)) == 0
        assert 20 * n + 8 * pairs <= out.value <= 20 * n + 8 * pairs + 1024
    assert ce._lib.ce_preference_workspace_size(ctypes.byref(_p(ce)), -1, ctypes.byref(out)) == ce.CE_ERR_INVALID_ARG


@pytest.mark.parametrize("n", [0, 1, 3, 63, 64, 65, 1000, 8191, 65536, 10 ** 7 + 1])
def test_python_workspaces_are_large_enough(ce, n):
    out = ctypes.c_size_t()
    p = _p(ce, n_rows=n)
    assert ce._lib.ce_workspace_size(ctypes.byref(p), ctypes.byref(out)) == 0
    assert out.value <= ce.logprob._policy_ws_bytes(n)
    for pairs in (0, 1, 31, 500):
        assert ce._lib.ce_preference_workspace_size(ctypes.byref(p), pairs, ctypes.byref(out)) == 0
        assert out.value <= ce.logprob._preference_ws_bytes(n, pairs)


def test_parameter_blocks(ce):
    assert ctypes.sizeof(ce.ce_policy_params) == 24 and ce.ce_policy_params.entropy_coef.offset == 16
    assert ctypes.sizeof(ce.ce_preference_params) == 32 and ce.ce_preference_params.beta.offset == 20


# ---------------------------------------------------------------------- refusals of the Python entries
def test_python_refusals(ce):
    x, t = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        ce.ce_token_logprob(x, t)
    with pytest.raises(ValueError, match="GPU"):
        ce.policy_loss(x, t, torch.zeros(4))
    with pytest.raises(ValueError, match="column stride"):
        ce.ce_token_logprob(torch.zeros(10, 4).t(), t)
    with pytest.raises(ValueError, match="one entry per row"):
        ce.ce_token_logprob(x, t[:3])
    with pytest.raises(ValueError, match="one entry per row"):
        ce.ce_token_logprob(x, torch.zeros(8, dtype=torch.int64)[::2])
    with pytest.raises(TypeError, match="int64"):
        ce.ce_token_logprob(x, t.float())
    with pytest.raises(TypeError, match="dtype"):
        ce.ce_token_logprob(x.double(), t)
    with pytest.raises(ValueError, match="reduction"):
        ce.ce_policy_fwd_bwd(x, t, torch.zeros(4), reduction="avg")
    with pytest.raises(ValueError, match="grad must"):
        ce.ce_policy_fwd_bwd(x, t, torch.zeros(4), grad=torch.zeros(4, 11))
    with pytest.raises(ValueError, match="2 P"):
        ce.ce_preference_fwd_bwd(x, t, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="loss_kind"):
        ce.ce_preference_fwd_bwd(x, t, torch.zeros(5, dtype=torch.int64), loss_kind="margin")
    with pytest.raises(ValueError, match="mean"):
        ce.preference_loss(x, t, torch.zeros(5, dtype=torch.int64), reduction="none")


# ---------------------------------------------------------------------- linear head
def _linear(ce, p, H=64, t=1.0, h=FAKE, w=FAKE, b=None, tgt=FAKE, logp=FAKE, stats=FAKE, ws=WS, nb=NB):
    return ce._lib.flce_token_logprob(ctypes.byref(p), H, t, h, w, b, tgt, logp, FAKE, stats, ws, nb, None)


def _linear_backward(ce, p, H=64, t=1.0, h=FAKE, w=FAKE, b=None, tgt=FAKE, logp=FAKE, stats=FAKE, gw=FAKE, dtype=0,
                     gb=None, chunk=4, ws=WS, nb=NB):
    return ce._lib.flce_token_logprob_backward(ctypes.byref(p), H, t, h, w, b, tgt, stats, logp, None, FAKE, gw, dtype, gb,
                                               chunk, ws, nb, None)


@pytest.mark.parametrize("call", [_linear, _linear_backward])
def test_linear_refusals_on_host(ce, call):
    bad, uns = ce.CE_ERR_INVALID_ARG, ce.CE_ERR_UNSUPPORTED
    for kw in (dict(n_rows=-1), dict(vocab=0), dict(tgt=2), dict(variant=1), dict(reserved=1)):
        assert call(ce, _p(ce, **kw)) == bad, kw
    for kw in UNSUPPORTED + [dict(dtype=0), dict(dtype=2), dict(n_rows=1 << 31)]:
        assert call(ce, _p(ce, **kw)) == uns, kw
    p = _p(ce)
    assert call(ce, p, H=0) == bad and call(ce, p, H=60) == uns
    assert call(ce, p, t=0.0) == bad and call(ce, p, t=math.nan) == bad
    odd = ctypes.c_void_p(0x100008)
    for kw in (dict(h=None), dict(w=None), dict(tgt=None), dict(tgt=ctypes.c_void_p(0x100004)), dict(h=odd), dict(w=odd), dict(b=odd), dict(stats=odd)):
        assert call(ce, p, **kw) == bad, kw
    assert call(ce, p, ws=None) == ce.CE_ERR_WORKSPACE
    assert call(ce, p, ws=ctypes.c_void_p(0x4000010)) == ce.CE_ERR_WORKSPACE
    assert call(ce, p, nb=512) == ce.CE_ERR_WORKSPACE


def test_linear_backward_refusals_on_host(ce):
    p, bad = _p(ce), ce.CE_ERR_INVALID_ARG
    assert _linear_backward(ce, p, chunk=0) == bad
    assert _linear_backward(ce, p, dtype=2) == bad
    assert _linear_backward(ce, p, dtype=1, chunk=3) == ce.CE_ERR_UNSUPPORTED
    assert _linear_backward(ce, p, gw=None) == bad
    assert _linear_backward(ce, p, gw=ctypes.c_void_p(0x100008)) == bad
    assert _linear_backward(ce, p, logp=None) == bad
    assert _linear_backward(ce, p, stats=None) == bad


def test_linear_workspace_sizes(ce):
    out = ctypes.c_size_t()
    size = lambda n, V, H, c: (ce._lib.flce_token_logprob_workspace_size(ctypes.byref(_p(ce, n_rows=n, vocab=V)), H, c,  # noqa: E731
                                                                        ctypes.byref(out)), out.value)[1]
    tiles = (128256 + 255) // 256 * 2
    assert 16 * tiles * 100 <= size(100, 128256, 4096, 0) <= 16 * tiles * 100 + 4096          # one row tile: no copy
    assert size(1, 128256, 4096, 0) <= 16384 and size(64, 128256, 4096, 0) <= 64 * 10240
    assert size(4096, 128256, 4096, 0) <= 4096 * (16 * tiles + 4096 * 2 + 16) + 16384
    assert size(4096, 128256, 4096, 4096) >= 4096 * 128256 * 2
    assert size(4096, 128256, 4096, 512) < size(4096, 128256, 4096, 4096)
    assert ce._lib.flce_token_logprob_workspace_size(ctypes.byref(_p(ce)), 64, -1, ctypes.byref(out)) == ce.CE_ERR_INVALID_ARG
