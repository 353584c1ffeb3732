"""CPU checks of the 8-bit serving head: its fp64 forms against loops over
single values, and the refusals of the C ABI and of the Python entries before
any CUDA call."""
import ctypes
import math

import pytest
import torch

import fp8_check as F


@pytest.fixture(scope="module")
def ce():
    import softmax_cross_entropy_pass_gb300 as ce
    return ce


# ---------------------------------------------------------------------- the fp64 forms
def test_block_form():
    g = torch.Generator().manual_seed(1)
    y = torch.randn(130, 200, generator=g, dtype=torch.float64)
    y[3, 128:] = 0
    for tall in (1, 128):
        s = F.block_scales(y, tall)
        each = F.spread(s, 130, 200, tall)
        for r, c in ((0, 0), (3, 130), (127, 127), (128, 128), (129, 199)):
            block = y[r // tall * tall:(r // tall + 1) * tall, c // 128 * 128:(c // 128 + 1) * 128]
            assert each[r, c] == max(float(block.abs().max()) / 448, 2.0 ** -126)
        q = F.e4m3(y / each)
        assert ((q * each - y).abs() <= each * (q.abs() * 2.0 ** -4 * 16 / 15 + 2.0 ** -10)).all()


def test_gemm_form():
    g = torch.Generator().manual_seed(2)
    a, b = (torch.randn(n, 130, generator=g).to(torch.float8_e4m3fn) for n in (3, 131))
    sa, sb = torch.rand(3, 2, generator=g), torch.rand(2, 2, generator=g)
    d, s = F.gemm_ref(a, sa, b, sb)
    for m, n in ((0, 0), (2, 127), (1, 128), (2, 130)):
        want = sum(float(a[m, k]) * float(sa[m, k // 128]) * float(b[n, k]) * float(sb[n // 128, k // 128]) for k in range(130))
        assert abs(float(d[m, n]) - want) < 1e-12 * float(s[m, n])


def test_drawn_tokens_follow_the_target():
    """The rule that check_sequence holds the kernels to leaves the target's distribution, whatever the draft's."""
    z, y = torch.tensor([[0.3, -1.0, 1.2, 0.0]] * 2), torch.tensor([[1.0, 0.5, -0.4, 0.1]])
    p, q = F.softmax(z[0], 1.0), F.softmax(y[0], 1.0)
    out = torch.zeros(4, dtype=torch.float64)
    for t in range(4):
        stay = min(1.0, float(p[t] / q[t]))
        out[t] += q[t] * stay
        left = (p - q).clamp_min(0)
        out += q[t] * (1 - stay) * left / left.sum()
    assert (out - p).abs().max() < 1e-12


# ---------------------------------------------------------------------- refusals of the C ABI
def at(a):
    return ctypes.c_void_p(a)


X, R, W, RO, Q, S = (at(0x1000000 * i) for i in range(1, 7))


def _norm(ce, x=X, residual=R, weight=W, residual_out=RO, q=Q, scale=S, **kw):
    d = dict(n_rows=4, cols=200, ld_x=200, ld_residual=200, ld_residual_out=200, ld_q=208, dtype=1, weight_dtype=1,
             eps=1e-6, reserved=0) | kw
    p = ce.ce_norm_params(*d.values())
    return ce._lib.ce_rms_norm_fp8(ctypes.byref(p), x, residual, weight, residual_out, q, scale, None)


def test_norm_refusals(ce):
    bad, uns = ce.CE_ERR_INVALID_ARG, ce.CE_ERR_UNSUPPORTED
    for kw in (dict(n_rows=-1), dict(cols=0), dict(ld_x=199), dict(ld_residual=199), dict(ld_residual_out=199),
               dict(ld_q=200), dict(ld_q=192), dict(dtype=3), dict(weight_dtype=2), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(reserved=1)):
        assert _norm(ce, **kw) == bad, kw
    assert _norm(ce, cols=32769, ld_x=40000, ld_residual=40000, ld_residual_out=40000, ld_q=40000) == uns
    assert _norm(ce, n_rows=1 << 31) == uns
    for name in ("x", "weight", "q", "scale"):
        assert _norm(ce, **{name: None}) == bad, name
    assert _norm(ce, residual=None) == bad                      # a sum without its second part
    assert _norm(ce, x=at(0x1000001)) == bad
    assert _norm(ce, weight=at(0x3000008)) == bad
    assert _norm(ce, q=at(0x5000008)) == bad
    assert _norm(ce, scale=at(0x6000002)) == bad
    # overlaps: an output over anything but, for the sum, the input it replaces
    assert _norm(ce, q=X) == bad and _norm(ce, q=R) == bad and _norm(ce, q=W) == bad
    assert _norm(ce, scale=X) == bad and _norm(ce, scale=Q) == bad
    assert _norm(ce, residual_out=Q) == bad and _norm(ce, residual_out=W) == bad
    assert _norm(ce, residual_out=R, ld_residual_out=208) == bad
    assert _norm(ce, residual_out=at(0x1000000 + 400)) == bad
    assert _norm(ce, n_rows=0, x=None, q=None, scale=None) == 0


def _quant(ce, rows=4, cols=200, x=X, ld=200, dtype=1, block=1, q=Q, ldq=208, scale=S):
    return ce._lib.ce_quantize_fp8(rows, cols, x, ld, dtype, block, q, ldq, scale, None)


def test_quantize_refusals(ce):
    bad = ce.CE_ERR_INVALID_ARG
    for kw in (dict(rows=-1), dict(cols=0), dict(ld=199), dict(ldq=199), dict(ldq=200), dict(dtype=3), dict(block=2),
               dict(block=0), dict(x=None), dict(q=None), dict(scale=None), dict(x=at(0x1000001)), dict(q=at(0x5000004)),
               dict(scale=at(0x6000001)), dict(q=X), dict(scale=X), dict(scale=Q)):
        assert _quant(ce, **kw) == bad, kw
    assert _quant(ce, rows=1 << 31) == ce.CE_ERR_UNSUPPORTED
    assert _quant(ce, rows=(1 << 31) - 1, cols=8192, ld=8192, ldq=8192) == ce.CE_ERR_UNSUPPORTED   # the grid
    assert _quant(ce, rows=0, x=None) == 0


def _gemm(ce, M=4, N=200, K=300, A=X, lda=304, sa=R, B=W, ldb=304, sb=RO, bias=None, dtype=1, D=Q, ldd=200):
    return ce._lib.ce_gemm_fp8(M, N, K, A, lda, sa, B, ldb, sb, bias, dtype, D, ldd, None)


def test_gemm_refusals(ce):
    bad = ce.CE_ERR_INVALID_ARG
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(lda=300), dict(lda=288), dict(ldb=300), dict(ldd=199), dict(dtype=3),
               dict(A=None), dict(B=None), dict(D=None), dict(sa=None), dict(sb=None), dict(A=at(0x1000008)),
               dict(B=at(0x3000008)), dict(D=at(0x5000001)), dict(sa=at(0x2000002)), dict(bias=at(0x6000002)),
               dict(D=X), dict(D=W), dict(D=R), dict(D=RO), dict(D=S, bias=S)):
        assert _gemm(ce, **kw) == bad, kw
    for kw in (dict(M=1 << 31), dict(N=1 << 31, ldd=1 << 31), dict(K=1 << 31, lda=1 << 31, ldb=1 << 31)):
        assert _gemm(ce, **kw) == ce.CE_ERR_UNSUPPORTED, kw
    assert _gemm(ce, M=0, A=None, D=None) == 0 and _gemm(ce, N=0, B=None) == 0


WS, NB = at(0x40000000), 1 << 28


def _verify(ce, x=X, y=R, draft=W, u=RO, r=Q, temps=None, acc=S, tok=at(0x7000000), logp=at(0x8000000), ws=WS, nb=NB, **kw):
    d = dict(n_seqs=2, n_drafts=3, vocab=100, seq_stride=400, ld=100, draft_seq_stride=300, ld_draft=100, dtype=1,
             token_is_int32=0, temperature=1.0, reserved=0) | kw
    p = ce.ce_verify_params(*d.values())
    return ce._lib.ce_verify_drafts(ctypes.byref(p), x, y, draft, u, r, temps, acc, tok, logp, ws, nb, None)


def test_verify_refusals(ce):
    bad, uns = ce.CE_ERR_INVALID_ARG, ce.CE_ERR_UNSUPPORTED
    for kw in (dict(n_seqs=-1), dict(n_drafts=-1), dict(vocab=0), dict(ld=99), dict(ld_draft=99), dict(seq_stride=-1),
               dict(draft_seq_stride=-1), dict(dtype=3), dict(token_is_int32=2), dict(temperature=-1.0),
               dict(temperature=math.nan), dict(temperature=1e-5), dict(temperature=math.inf), dict(reserved=1),
               dict(x=None), dict(draft=None), dict(u=None), dict(r=None), dict(acc=None), dict(tok=None),
               dict(logp=None), dict(x=at(0x1000001)), dict(y=at(0x2000001)), dict(draft=at(0x3000004)),
               dict(u=at(0x4000002)), dict(r=at(0x5000002)), dict(temps=at(0x9000002)), dict(acc=at(0x6000002)),
               dict(tok=at(0x7000004)), dict(logp=at(0x8000002)), dict(tok=W), dict(acc=S, logp=S), dict(logp=RO),
               dict(acc=X), dict(tok=WS), dict(logp=R)):
        assert _verify(ce, **kw) == bad, kw
    for kw in (dict(n_drafts=256), dict(vocab=1 << 31, ld=1 << 31, ld_draft=1 << 31), dict(n_seqs=1 << 30)):
        assert _verify(ce, **kw) == uns, kw
    for kw in (dict(ws=None), dict(ws=at(0x40000010)), dict(nb=256)):
        assert _verify(ce, **kw) == ce.CE_ERR_WORKSPACE, kw
    assert _verify(ce, n_seqs=0, x=None, ws=None) == 0


def test_verify_workspace_size(ce):
    out = ctypes.c_size_t()
    for B, K, V in ((1, 0, 1), (1, 3, 128256), (128, 4, 128256), (256, 8, 700), (3, 255, 50257)):
        p = ce.ce_verify_params(B, K, V, V * (K + 1), V, V * K, V, 1, 0, 1.0, 0)
        assert ce._lib.ce_verify_workspace_size(ctypes.byref(p), ctypes.byref(out)) == 0
        rows, parts = B * (2 * K + 1), -(-(V + 7) // 256)   # at most: parts of 512 bytes
        assert 16 * rows <= out.value - 256 <= 16 * rows * parts
        assert out.value == ce.serving._verify_ws_bytes(p)
    assert ce._lib.ce_verify_workspace_size(ctypes.byref(p), None) == ce.CE_ERR_INVALID_ARG


# ---------------------------------------------------------------------- refusals of the Python entries
def test_python_refusals(ce):
    x, w = torch.zeros(4, 64), torch.zeros(64)
    q, s = torch.zeros(4, 64).to(torch.float8_e4m3fn), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="GPU"):
        ce.ce_rms_norm_fp8(x, w)
    with pytest.raises(ValueError, match="GPU"):
        ce.ce_quantize_fp8(x)
    with pytest.raises(ValueError, match="GPU"):
        ce.ce_gemm_fp8(q, s, q, s[:1])
    with pytest.raises(ValueError, match="column stride"):
        ce.ce_rms_norm_fp8(torch.zeros(64, 4).t(), w)
    with pytest.raises(TypeError, match="dtype"):
        ce.ce_quantize_fp8(x.double())
    with pytest.raises(ValueError, match="block_rows"):
        ce.ce_quantize_fp8(x, block_rows=64)
    with pytest.raises(TypeError, match="float8"):
        ce.ce_gemm_fp8(x, s, q, s)
    with pytest.raises(ValueError, match="16 bytes"):
        ce.ce_gemm_fp8(torch.zeros(4, 60).to(torch.float8_e4m3fn), s, q, s)
    with pytest.raises(ValueError, match="inner"):
        ce.ce_gemm_fp8(q, s, torch.zeros(4, 48).to(torch.float8_e4m3fn), s)
    z, d = torch.zeros(2, 4, 10), torch.zeros(2, 3, dtype=torch.int64)
    u, r = torch.zeros(2, 3), torch.zeros(2)
    with pytest.raises(ValueError, match="GPU"):
        ce.ce_verify_drafts(z, d, u, r)
    with pytest.raises(ValueError, match="K . 1, V"):
        ce.ce_verify_drafts(z[0], d, u, r)
    with pytest.raises(TypeError, match="int64"):
        ce.ce_verify_drafts(z, d.float(), u, r)
    with pytest.raises(ValueError, match="draft_token"):
        ce.ce_verify_drafts(z, d[:, :2], u, r)
    with pytest.raises(ValueError, match="accept_uniform"):
        ce.ce_verify_drafts(z, d, u.double(), r)
    with pytest.raises(ValueError, match="sample_uniform"):
        ce.ce_verify_drafts(z, d, u, r[:1])
    with pytest.raises(ValueError, match="temperature"):
        ce.ce_verify_drafts(z, d, u, r, temperature=torch.ones(3))
    with pytest.raises(TypeError, match="dtype"):
        ce.ce_verify_drafts(z.double(), d, u, r)
