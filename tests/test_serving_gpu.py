"""The 8-bit serving head on the GPU against its fp64 forms (fp8_check.py,
which derives the tolerances)."""
import math

import pytest
import torch

import fp8_check as F

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def ce():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import softmax_cross_entropy_pass_gb300 as ce
    return ce


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def wide(rows, cols, pad, off, dtype, g, std=1.0):
    """A view into a wider buffer: row stride cols + pad + off, first column off."""
    buf = torch.empty(rows, cols + pad + off, device="cuda").normal_(0, std, generator=g)
    buf *= 0.1 + 3 * torch.rand(rows, 1, generator=g, device="cuda")
    return buf.to(DT[dtype])[:, off:off + cols]


# ---------------------------------------------------------------------- norm
NORMS = [
    # rows, cols, padding, first column
    (1, 1, 0, 0), (3, 7, 0, 0), (2, 128, 0, 0), (5, 129, 2, 1), (33, 1000, 0, 0), (4, 4096, 0, 0), (7, 4099, 5, 3),
    (3, 8192, 8, 8), (2, 8200, 0, 0), (2, 16384, 0, 0), (2, 20001, 0, 1), (1, 32768, 0, 0), (300, 256, 0, 0),
]


@pytest.mark.parametrize("shape", NORMS, ids=lambda s: f"{s[0]}x{s[1]}+{s[2]}@{s[3]}")
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(ce, shape, dtype, residual):
    n, cols, pad, off = shape
    g = gen(n * 7 + cols)
    x = wide(n, cols, pad, off, dtype, g)
    r = wide(n, cols, 0, 0, dtype, g) if residual else None
    w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(torch.float32 if n % 2 else DT[dtype])
    eps = float(torch.tensor(1e-5, dtype=torch.float32))
    kept = x.clone(), None if r is None else r.clone()
    q, scale, out = ce.ce_rms_norm_fp8(x, w, residual=r, eps=eps)
    torch.cuda.synchronize()
    F.rows8(q)
    h, y = F.norm_ref(x, w, r, eps)
    F.check_blocks(q, scale, y)
    assert torch.equal(x, kept[0])
    if residual:
        assert torch.equal(r, kept[1])
        tol = h.abs() * (F.HALF[DT[dtype]] * (1 + 2.0 ** -10) + 2 * F.U) + (2.0 ** -25 if dtype == "f16" else 0)
        assert ((out.double() - h).abs() <= tol).all()
    else:
        assert out is None


@pytest.mark.parametrize("shape", [(700, 4096, 0, 0), (4100, 2048, 0, 0), (9001, 200, 3, 1), (3001, 1030, 2, 0), (500, 12000, 0, 0),
                                   (310, 20000, 4, 4), (1300, 2056, 0, 0), (20000, 64, 0, 0)],
                         ids=lambda s: f"{s[0]}x{s[1]}+{s[2]}@{s[3]}")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_many_rows(ce, shape, dtype):
    """More rows than the GPU holds at once: every row as in a call of its own few."""
    n, cols, pad, off = shape
    g = gen(n + cols)
    x, r = wide(n, cols, pad, off, dtype, g), wide(n, cols, pad, off, dtype, g)
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    q, s, out = ce.ce_rms_norm_fp8(x, w, residual=r)
    assert torch.equal(out, (x.float() + r.float()).to(x.dtype))
    h = x.double() + r.double()
    y = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    up = torch.nn.functional.pad(y, (0, -cols % 128)).view(n, -1, 128)
    want = up.abs().amax(2) / 448
    # fp32: the sum of cols squares (pairwise over lanes: cols / 32 + 32 additions at most), a root, three products
    tol = (cols / 32 + 48) * F.U
    assert ((s.double() - want).abs() <= want * tol + 2.0 ** -126).all()
    value = torch.nn.functional.pad(q.float().double(), (0, -cols % 128)).view(n, -1, 128) * s.double()[:, :, None]
    # half a step of e4m3 (2^-4 relative, 2^-10 of the scale below its smallest normal), beside the roundings above
    assert ((value - up).abs() <= up.abs() * (2.0 ** -4 + 2 * tol) + 2.0 ** -10 * s.double()[:, :, None] * (1 + 2 * tol)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place_and_given_buffers(ce, dtype):
    g = gen(5)
    x, r, w = wide(9, 500, 4, 0, dtype, g), wide(9, 500, 4, 0, dtype, g), torch.ones(500, device="cuda")
    q0, s0, out = ce.ce_rms_norm_fp8(x, w, residual=r)
    buf = torch.full((9, 528), 7, dtype=torch.uint8, device="cuda")
    q, s = buf.view(torch.float8_e4m3fn)[:, :500], torch.empty(9, 4, device="cuda")
    for place in (r.clone(memory_format=torch.preserve_format), None):
        # r and x are views: take the place of their own buffers
        rr, xx = r.clone(), x.clone()
        target = rr if place is not None else xx
        got = ce.ce_rms_norm_fp8(xx, w, residual=rr, residual_out=target, q=q, scale=s)
        assert got[0] is q and got[1] is s and got[2] is target
        assert torch.equal(target, out) and torch.equal(s, s0)
        assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8))
        assert (buf[:, 500:] == 7).all()   # bytes between the columns and the stride are left alone
    q2, s2, none = ce.ce_rms_norm_fp8(x, w, residual=r, with_residual_out=False)
    assert none is None and torch.equal(s2, s0)


def test_norm_ends_of_the_range(ce):
    """Rows of zeros, tiny and huge ones, single values, NaN and infinities."""
    w = torch.ones(300, device="cuda")
    x = torch.zeros(8, 300, device="cuda")
    x[1] = 1e-30 * torch.randn(300, device="cuda")
    x[2] = 1e25 * torch.randn(300, device="cuda")
    x[3, 170] = 3.0
    x[4, 5] = math.nan
    x[5, 7] = math.inf
    x[6] = 1e-3
    x[7] = torch.randn(300, device="cuda")
    for eps in (0.0, 1e-6):
        e = float(torch.tensor(eps, dtype=torch.float32))
        q, s, _ = ce.ce_rms_norm_fp8(x, w, eps=eps)
        rows = [2, 3, 6, 7] + ([1] if eps == 0 else [0])
        _, y = F.norm_ref(x[rows], w, None, e)
        F.check_blocks(q[rows], s[rows], y)
        assert s[4].isnan().all() and q[4].float().isnan().all()
        assert q[5, 7].float().isnan()
        if eps:
            assert (q[0].float() == 0).all() and (s[0] == F.MIN_SCALE).all()


# ---------------------------------------------------------------------- quantising
@pytest.mark.parametrize("shape", [(1, 1, 0, 0), (3, 128, 0, 0), (130, 300, 1, 1), (128, 4096, 0, 0), (257, 1000, 8, 8),
                                   (500, 129, 0, 0), (1, 9000, 0, 0)], ids=lambda s: f"{s[0]}x{s[1]}+{s[2]}@{s[3]}")
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tall", [1, 128])
def test_quantize(ce, shape, dtype, tall):
    n, cols, pad, off = shape
    x = wide(n, cols, pad, off, dtype, gen(n + cols))
    if n > 100:
        x[:128, :128] = 0          # a block of zeros
        x[4, cols - 1] = -x[:, cols - 1].abs().max() * 2
    q, scale = ce.ce_quantize_fp8(x, block_rows=tall)
    torch.cuda.synchronize()
    F.rows8(q)
    F.check_blocks(q, scale, x.double(), tall, slack=2.0 ** -22)   # two divisions and a product, no sums


def test_quantize_special_values(ce):
    x = torch.ones(130, 260, device="cuda")
    x[0, 0], x[1, 129], x[2, 258] = math.nan, math.inf, -1e-44
    x[:, 200] = 0.0
    q, s = ce.ce_quantize_fp8(x)
    assert s[0, 0].isnan() and q[0, :128].float().isnan().all() and not s[0, 1:].isnan().any()
    assert s[1, 1].isinf() and q[1, 129].float().isnan()
    q, s = ce.ce_quantize_fp8(x, block_rows=128)
    assert s[0, 0].isnan() and q[:128, :128].float().isnan().all() and s[0, 1].isinf()
    assert not s[1].isnan().any() and (q[128:, 200].float() == 0).all()


# ---------------------------------------------------------------------- product
def operands(ce, m, n, k, seed, pad=0):
    g = gen(seed)
    a = wide(m, k, 0, 0, "f32", g)
    b = torch.empty(n, k, device="cuda").normal_(0, 0.05, generator=g)
    b *= (0.02 + torch.rand(-(-n // 128), -(-k // 128), generator=g, device="cuda")).repeat_interleave(128, 0)[:n] \
        .repeat_interleave(128, 1)[:, :k]
    qa, sa = ce.ce_quantize_fp8(a)
    qb, sb = ce.ce_quantize_fp8(b, block_rows=128)
    bias = torch.randn(n, generator=g, device="cuda")
    return qa, sa, qb, sb, bias


GEMMS = [
    # M, N, K
    (70, 1024, 1100), (129, 700, 2064), (40, 500, 5000), (16, 4096, 4096),
    (1, 1, 1), (1, 16, 128), (2, 17, 100), (16, 128, 256), (5, 300, 130), (17, 1000, 520), (32, 129, 4096), (33, 2433, 384),
    (64, 4096, 1024), (65, 515, 777), (100, 20000, 256), (128, 128, 128), (130, 300, 4224), (200, 2500, 640), (300, 1111, 300),
    (1, 50257, 512), (513, 260, 256), (1000, 1000, 1000), (256, 256, 8320), (700, 3000, 200), (4, 152 * 16 + 5, 9000),
]


@pytest.mark.parametrize("shape", GEMMS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_gemm(ce, shape, dtype):
    m, n, k = shape
    a, sa, b, sb, bias = operands(ce, m, n, k, m + n + k)
    bias = bias if (m + n) % 2 else None
    pad = [0, 3, 16][k % 3]
    buf = torch.full((m, n + pad), 99.0, dtype=DT[dtype], device="cuda")
    out = ce.ce_gemm_fp8(a, sa, b, sb, bias=bias, out=buf[:, :n])
    torch.cuda.synchronize()
    F.check_gemm(out, a, sa, b, sb, bias)
    assert (buf[:, n:] == 99).all()
    again = ce.ce_gemm_fp8(a, sa, b, sb, bias=bias, out_dtype=DT[dtype])
    assert torch.equal(out, again)   # the same bits every time


def test_gemm_reads_nothing_past_the_columns(ce):
    """Bytes between the last column and the row stride hold NaN, in both operands."""
    m, n, k = 20, 150, 200
    a, sa, b, sb, _ = operands(ce, m, n, k, 3)
    fill = []
    for t in (a, b):
        buf = torch.full((t.shape[0], 240), 0x7f, dtype=torch.uint8, device="cuda")
        buf[:, :k] = t.view(torch.uint8)
        fill.append(buf.view(torch.float8_e4m3fn)[:, :k])
    assert torch.equal(ce.ce_gemm_fp8(*fill[:1], sa, fill[1], sb), ce.ce_gemm_fp8(a, sa, b, sb))


def test_gemm_nan_and_large_scales(ce):
    a, sa, b, sb, _ = operands(ce, 70, 300, 260, 4)
    sa, sb = sa * 1e12, sb * 1e-14
    out = ce.ce_gemm_fp8(a, sa, b, sb, out_dtype=torch.float32)
    F.check_gemm(out, a, sa, b, sb)
    sa[3, 1] = math.nan
    out = ce.ce_gemm_fp8(a, sa, b, sb, out_dtype=torch.float32)
    assert out[3].isnan().all() and not out[:3].isnan().any() and not out[4:].isnan().any()


def test_gemm_empty(ce):
    a, sa, b, sb, _ = operands(ce, 4, 30, 64, 5)
    assert ce.ce_gemm_fp8(a[:0], sa[:0], b, sb).shape == (0, 30)
    assert ce.ce_gemm_fp8(a, sa, b[:0], sb[:0]).shape == (4, 0)
    q, s = ce.ce_quantize_fp8(torch.empty(0, 100, device="cuda"))
    assert q.shape == (0, 100) and s.shape == (0, 1)
    q, s, r = ce.ce_rms_norm_fp8(torch.empty(0, 100, device="cuda"), torch.ones(100, device="cuda"),
                                 residual=torch.empty(0, 100, device="cuda"))
    assert q.shape == (0, 100) and r.shape == (0, 100)


# ---------------------------------------------------------------------- verification
def verify_inputs(B, K, V, dtype, model, seed, pad=0, off=0, temps=None, padded=True, int32=False):
    g = gen(seed)
    z = torch.empty(B, K + 1, V + pad + off, device="cuda").normal_(0, 2, generator=g)
    if V > 20:
        z.scatter_(2, torch.randint(0, V, (B, K + 1, 8), generator=g, device="cuda") + off,
                   6 + 5 * torch.rand(B, K + 1, 8, generator=g, device="cuda"))
    y = z[:, :K] + 0.6 * torch.randn(B, K, V + pad + off, generator=g, device="cuda")
    z, y = z.to(DT[dtype])[:, :, off:off + V], y.to(DT[dtype])[:, :, off:off + V]
    base = (y if model else z[:, :K] * 1.3).float()
    draft = (base - torch.empty(base.shape, device="cuda").exponential_(generator=g).log()).argmax(-1) if K else \
        torch.empty(B, 0, dtype=torch.int64, device="cuda")
    if padded and K:
        length = torch.randint(0, K + 3, (B,), generator=g, device="cuda")
        draft = torch.where(torch.arange(K, device="cuda") < length[:, None], draft, -1)
    u, r = torch.rand(B, K, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    if temps == "mixed":
        temps = 0.4 + torch.rand(B, generator=g, device="cuda")
        temps[::3] = 0
    return z, y if model else None, draft.int() if int32 else draft, u, r, 1.0 if temps is None else temps


def many(times, *tensors):
    """The batch several times over: where a position's rows hold more than 8 MB another kernel verifies them."""
    return tuple(t.repeat(times, *[1] * (t.dim() - 1)) if torch.is_tensor(t) else t for t in tensors)


def check(z, y, draft, u, r, t, got):
    """Against fp64; of large batches every sequence of the first 24 and every 7th behind them."""
    B = z.shape[0]
    at = torch.tensor([b for b in range(B) if b < 24 or b % 7 == 0 or B <= 160], device=z.device)
    pick = lambda v: v[at] if torch.is_tensor(v) and v.dim() else v  # noqa: E731
    F.check_verify(pick(z), None if y is None else pick(y), pick(draft).cpu(), pick(u).cpu(), pick(r).cpu(),
                   pick(t).cpu() if torch.is_tensor(t) else t, tuple(pick(v) for v in got))


VERIFIES = [
    # B, K, V, padding, first column
    (1, 0, 1, 0, 0), (3, 2, 2, 0, 0), (2, 1, 7, 0, 0), (5, 3, 257, 0, 0), (4, 4, 1000, 0, 0), (2, 3, 4099, 3, 1),
    (9, 0, 5000, 0, 0), (1, 3, 128256, 0, 0), (3, 2, 50257, 0, 0), (40, 5, 3001, 7, 8), (2, 20, 300, 0, 0),
    (150, 3, 2050, 0, 0), (2, 1, 300001, 0, 0), (28, 0, 3, 0, 0), (29, 2, 8200, 0, 0), (33, 1, 9, 7, 3), (60, 3, 20011, 5, 1),
    (27, 4, 6000, 8, 8), (100, 1, 40000, 0, 0), (230, 6, 1000, 0, 0),
    # a position's rows above 8 MB
    (130, 3, 34001, 7, 3), (300, 2, 17003, 5, 1), (29, 1, 300001, 0, 0), (40, 0, 120001, 0, 0), (210, 9, 24000, 8, 8),
    (460, 1, 10007, 0, 1), (600, 2, 8192, 0, 0), (56, 4, 80000, 0, 0),
]


@pytest.mark.parametrize("shape", VERIFIES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}+{s[3]}@{s[4]}")
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("model", [True, False])
def test_verify(ce, shape, dtype, model):
    B, K, V, pad, off = shape
    temps = [None, "mixed", 0.7][(B + K + V) % 3]
    args = verify_inputs(B, K, V, dtype, model, B * 100 + V, pad, off, temps, int32=B % 2 == 0)
    z, y, draft, u, r, t = args
    got = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y, temperature=t)
    torch.cuda.synchronize()
    check(z, y, draft, u, r, t, got)
    again = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y, temperature=t)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("times", [1, 6, 80])
def test_verify_all_stay_or_none(ce, dtype, times):
    z, _, draft, u, r, _ = verify_inputs(6, 4, 5000, dtype, False, 8, padded=False)
    z, draft, u, r = many(times, z, draft, u, r)
    y = z[:, :4].clone()
    # the draft model is the target: every draft stays, whatever u
    got = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y)
    check(z, y, draft, u, r, 1.0, got)
    assert (got[0] == 4).all() and torch.equal(got[1][:, :4], draft)
    # drafts that the target masks: none stays
    z.scatter_(2, torch.nn.functional.pad(draft, (0, 1))[:, :, None], -math.inf)
    got = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y)
    check(z, y, draft, u, r, 1.0, got)
    assert (got[0] == 0).all() and (got[1][:, 1:] == -1).all()
    # u = 0 keeps any draft with a probability above 0
    got = ce.ce_verify_drafts(y.new_zeros(2, 2, 64), torch.tensor([[5], [-1]], device="cuda"), torch.zeros(2, 1, device="cuda"),
                              torch.zeros(2, device="cuda"))
    assert got[0].tolist() == [1, 0] and got[1].tolist() == [[5, 0], [0, -1]]


@pytest.mark.parametrize("times", [1, 10, 60])
def test_verify_greedy_ties_take_the_lowest_index(ce, times):
    for V in (64, 5003, 131072):
        z = torch.zeros(3, 3, V, device="cuda", dtype=torch.bfloat16)
        z[0, :, 9] = z[0, :, V - 1] = z[0, :, V // 2] = 4.0
        z[1, :, V - 2] = z[1, :, V - 1] = 4.0
        z[2, 0, 3] = 1.0
        draft = torch.tensor([[9, V - 1], [V - 2, V - 2], [3, 1]], device="cuda")
        z, draft = many(times, z, draft)
        got = ce.ce_verify_drafts(z, draft, torch.rand(3 * times, 2, device="cuda"), torch.rand(3 * times, device="cuda"), temperature=0.0)
        assert got[0].tolist() == [1, 2, 1] * times
        assert got[1].tolist() == [[9, 9, -1], [V - 2, V - 2, V - 2], [3, 0, -1]] * times


@pytest.mark.parametrize("times", [1, 4, 130])
def test_verify_masks(ce, times):
    """Most of the vocabulary masked (-inf, the type's lowest value), rows with one value left, equal rows."""
    for dtype, low in (("bf16", -math.inf), ("f32", -math.inf), ("bf16", float(torch.finfo(torch.bfloat16).min)),
                       ("f32", float(torch.finfo(torch.float32).min)), ("f16", -65504.0)):
        z, y, draft, u, r, _ = verify_inputs(8, 3, 4100, dtype, True, 21, padded=False)
        for t in (z, y):
            t[::2, :, 100:] = low
            t[1, :, :4000] = low
            t[3] = low
            t[3, :, 77] = 1.0
        draft = (draft % 100)
        draft[1] += 4000
        draft[3] = 77
        z, y, draft, u, r = many(times, z, y, draft, u, r)
        got = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y)
        check(z, y, draft, u, r, 1.0, got)
        assert got[0][3] == 3 and (got[1][3] == 77).all() and (got[2][3] == 0).all()
        got = ce.ce_verify_drafts(z, draft, u, r)
        check(z, None, draft, u, r, 1.0, got)


@pytest.mark.parametrize("times", [1, 4, 100])
def test_verify_undefined_rows(ce, times):
    """A row with nothing left, a NaN or +inf ends its sequence with -1; rows behind the decision may hold anything."""
    z, y, draft, u, r, _ = verify_inputs(9, 2, 3000, "bf16", True, 31, padded=False)
    y.copy_(z[:, :2])                      # all drafts stay where the rows allow it
    z[0, 0] = -math.inf
    z[1, 1, 5] = math.nan
    z[2, 2, 2999] = math.inf
    y[3, 0] = -math.inf
    y[4, 1, 17] = math.nan
    draft[5, 0] = -1
    z[5, 1:], y[5] = math.nan, math.nan     # behind the last draft: not read
    draft[6, 1] = 3000                      # outside of the vocabulary
    y[6, 1] = math.nan
    temps = torch.ones(9, device="cuda")
    temps[7], temps[8] = -1.0, math.nan
    z, y, draft, u, r, temps = many(times, z, y, draft, u, r, temps)
    n, tok, lp = (v.tolist() for v in ce.ce_verify_drafts(z, draft, u, r, draft_logits=y, temperature=temps))
    assert n == [0, 1, 2, 0, 1, 0, 1, 0, 0] * times
    at = [9 * i for i in range(times)]
    for b in [i + j for i in (0, 1, 2, 3, 4, 7, 8) for j in at]:
        assert tok[b][n[b]] == -1 and math.isnan(lp[b][n[b]]) and all(t == -1 for t in tok[b][n[b]:])
        assert all(v == 0 for v in lp[b][n[b] + 1:])
    for b in [i + j for i in (5, 6) for j in at]:
        assert 0 <= tok[b][n[b]] < 3000 and math.isfinite(lp[b][n[b]])
    greedy = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y, temperature=0.0)
    assert greedy[1][0, 0] == -1 and greedy[0][0] == 0


@pytest.mark.parametrize("B", [64, 500])
def test_verify_ends_of_the_random_numbers(ce, B):
    z, y, draft, u, _, _ = verify_inputs(B, 2, 6000, "bf16", True, 41, padded=False)
    for v in (0.0, 1.0 - 2.0 ** -24):
        r = torch.full((B,), v, device="cuda")
        got = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y)
        check(z, y, draft, u, r, 1.0, got)


@pytest.mark.parametrize("B", [5, 40, 640])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verify_far_logits(ce, B, dtype):
    """Drafts far below the row's maximum, maxima far from 0, low and high temperatures: references that do not hold
    the row's terms."""
    z, y, draft, u, r, _ = verify_inputs(B, 3, 7000, dtype, True, 91, padded=False)
    z[:, 0] += 300.0
    y[:, 1] -= 500.0
    rows = torch.arange(B, device="cuda")
    z[rows[::3], 1, draft[::3, 1]] = -200.0            # turned down: its probability is 0 in fp32
    y[rows[::4], 0, draft[::4, 0]] = -150.0            # a draft that its own model would hardly draw stays
    z[1, 2], y[1, 2] = -3e4, -3e4
    z[1, 2, 17] = 3e4
    for t in (1.0, 0.05, 30.0):
        got = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y, temperature=t)
        # 3 u |a| of an exponent relative to the reference or the maximum, |a| up to 60
        check(z, y, draft, u, r, t, got)
        check(z, None, draft, u, r, t, ce.ce_verify_drafts(z, draft, u, r, temperature=t))


@pytest.mark.parametrize("B", [3, 32, 260])
def test_verify_likely_tokens(ce, B):
    """log p of tokens with probabilities near 1 keeps its relative precision, staying, greedy or drawn."""
    z = torch.randn(B, 2, 9000, generator=gen(95), device="cuda")
    tops = 9.0 + 8.0 * torch.rand(B, 2, generator=gen(96), device="cuda") + 9.0
    z[:, :, 4321] = tops
    draft = torch.full((B, 1), 4321, device="cuda")
    u, r = torch.zeros(B, 1, device="cuda"), torch.full((B,), 0.5, device="cuda")
    for t in (1.0, 0.0):
        n, tok, lp = ce.ce_verify_drafts(z, draft, u, r, temperature=t)
        assert (n == 1).all() and (tok == 4321).all()
        want = torch.log_softmax(z.double(), 2)[:, :, 4321]
        # -log1p(s): s is off by rel(V), log1p by its own rounding; s itself is below 0.02 here
        assert ((lp.double() - want).abs() <= want.abs() * (F.rel(9000) + 4 * F.U)).all()


@pytest.mark.parametrize("B,V", [(2, 700), (60, 80000)])
def test_verify_as_many_drafts_as_there_may_be(ce, B, V):
    """255 drafts that all stay, one that is turned down in the middle, a batch whose sequences are one in memory."""
    K = 255
    z = torch.empty(1, K + 1, V, device="cuda", dtype=torch.bfloat16).normal_(0, 3, generator=gen(7)).expand(B, -1, -1)
    draft = z[:, :K].argmax(2).contiguous()
    u, r = torch.zeros(B, K, device="cuda"), torch.rand(B, generator=gen(8), device="cuda")
    draft[1, 100] = (draft[1, 100] + 1) % V
    u[1, 100] = 0.999
    n, tok, lp = ce.ce_verify_drafts(z, draft, u, r)
    assert n[0] == K and n[1] == 100 and (n[2:] == K).all() and torch.equal(tok[0, :K], draft[0]) and (tok[1, 101:] == -1).all()
    want = torch.log_softmax(z[0].double(), 1)
    for b in (0, 1, B - 1):
        i = torch.arange(int(n[b]) + 1, device="cuda")
        got = want[i, tok[b, i]]
        # a sum's relative error, and the roundings of exponents and log p of at most 64 in magnitude
        assert ((lp[b, i].double() - got).abs() <= F.rel(V) + 8 * F.U * 64).all()


def test_verify_strides_and_buffers(ce):
    z, y, draft, u, r, _ = verify_inputs(4, 3, 900, "bf16", True, 51)
    # (rows at another alignment are summed in another order: each answer is held to fp64, not to the other)
    zt = z.transpose(0, 1).contiguous().transpose(0, 1)          # position-major memory
    acc, tok, lp = (torch.full_like(v, 77) for v in ce.ce_verify_drafts(z, draft, u, r, draft_logits=y))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    got = ce.ce_verify_drafts(zt, draft, u, r, draft_logits=y, accepted=acc, tokens=tok, logp=lp, ws=ws)
    assert got[0] is acc and got[1] is tok and got[2] is lp
    F.check_verify(z, y, draft.cpu(), u.cpu(), r.cpu(), 1.0, got)
    with pytest.raises(ValueError):
        ce.ce_verify_drafts(z, draft, u, r, draft_logits=y.float())
    with pytest.raises(ce.CEError):
        ce.ce_verify_drafts(z, draft, u, r, ws=ws[:256])
    empty = ce.ce_verify_drafts(z[:0], draft[:0], u[:0], r[:0])
    assert empty[1].shape == (0, 4)


# ---------------------------------------------------------------------- together
def head(ce, d):
    """One step of the serving head: hidden states of drafted positions to verified tokens."""
    logits = ce.fp8_head_logits(d["x"], d["w"], d["q"], d["s"], residual=d["res"])
    return (logits,) + ce.ce_verify_drafts(logits, d["draft"], d["u"], d["r"], temperature=d["t"])


def head_inputs(ce, seed, B=6, K=3, H=640, V=5003):
    g = gen(seed)
    d = dict(x=torch.randn(B, K + 1, H, generator=g, device="cuda").bfloat16(), res=torch.randn(B, K + 1, H, generator=g, device="cuda").bfloat16(),
             w=1 + 0.2 * torch.randn(H, generator=g, device="cuda"))
    d["q"], d["s"] = ce.ce_quantize_fp8((torch.randn(V, H, generator=gen(1), device="cuda") * 0.15).bfloat16(), block_rows=128)
    d["draft"] = torch.randint(0, V, (B, K), generator=g, device="cuda")
    d["draft"][::2] = head_best(ce, d)[::2, :K]
    d["u"], d["r"] = torch.rand(B, K, generator=g, device="cuda") * 0.2, torch.rand(B, generator=g, device="cuda")
    d["t"] = torch.tensor([0.7, 0.0, 1.0, 0.9, 0.0, 1.3], device="cuda")[:B].contiguous()
    return d


def head_best(ce, d):
    return ce.fp8_head_logits(d["x"], d["w"], d["q"], d["s"], residual=d["res"]).float().argmax(-1)


def test_head_together(ce):
    d = head_inputs(ce, 61)
    logits, accepted, tokens, logp = head(ce, d)
    B, K1, H = d["x"].shape
    # the product of the dequantised operands, and the verification of those logits
    q, s, _ = ce.ce_rms_norm_fp8(d["x"].view(-1, H), d["w"], residual=d["res"].view(-1, H))
    F.check_gemm(logits.view(B * K1, -1), q, s, d["q"], d["s"])
    F.check_verify(logits, None, d["draft"].cpu(), d["u"].cpu(), d["r"].cpu(), d["t"].cpu(), (accepted, tokens, logp))
    # near the unquantised head: e4m3 steps of 2^-4 of each factor, averaged over the columns
    _, y = F.norm_ref(d["x"].view(-1, H), d["w"], d["res"].view(-1, H), 1e-6)
    full = y @ (d["q"].double() * F.spread(d["s"], *d["q"].shape, 128)).t()
    assert (logits.view(B * K1, -1).double() - full).norm() < 2.0 ** -4 * full.norm()
    # the log-probabilities are those of the framework's own operator on the same logits
    keep = tokens >= 0
    want, _, _ = ce.ce_token_logprob(logits.view(B * K1, -1), torch.where(keep, tokens, -100).view(-1))
    ones = (d["t"] == 1.0) | (d["t"] == 0.0)
    assert ((want.view(B, K1) - logp)[ones].abs() < 1e-5).all()
    assert accepted.max() > 0


def test_head_captured(ce):
    d = head_inputs(ce, 62)
    head(ce, d)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = head(ce, d)
    with torch.cuda.graph(second):
        outs2 = head(ce, d)
    for seed in (63, 64):
        for k, v in head_inputs(ce, seed).items():
            d[k].copy_(v)
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        want = head(ce, d)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(outs2, want))


def test_head_on_another_stream_and_threads(ce):
    import threading
    data = [head_inputs(ce, 70 + i) for i in range(4)]
    alone = [head(ce, d) for d in data]
    torch.cuda.synchronize()
    side, d = torch.cuda.Stream(), data[0]
    q, s, _ = ce.ce_rms_norm_fp8(d["x"].view(-1, 640), d["w"], residual=d["res"].view(-1, 640), stream=side)
    logits = ce.ce_gemm_fp8(q, s, d["q"], d["s"], stream=side).view(alone[0][0].shape)
    got = ce.ce_verify_drafts(logits, d["draft"], d["u"], d["r"], temperature=d["t"], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((logits,) + got, alone[0]))
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = head(ce, data[i])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, alone[i])):
                        failed.append(f"thread {i} differs")
        except BaseException as e:  # noqa: BLE001
            failed.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed, failed


def test_offsets_past_32_bits(ce):
    """Rows of logits, of a product's output and of 8-bit operands that start beyond 2^31 elements."""
    V, stride = 3001, 1 << 30
    buf = torch.empty(3 * stride + V, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(buf, (2, 2, V), (2 * stride, stride, 1))
    small, _, draft, u, r, _ = verify_inputs(2, 1, V, "bf16", False, 81, padded=False)
    z.copy_(small)
    F.check_verify(small, None, draft.cpu(), u.cpu(), r.cpu(), 1.0, ce.ce_verify_drafts(z, draft, u, r))
    a, sa, b, sb, _ = operands(ce, 4, 300, 256, 82)
    out = torch.as_strided(buf, (4, 300), (stride, 1))
    ce.ce_gemm_fp8(a, sa, b, sb, out=out)
    assert torch.equal(out, ce.ce_gemm_fp8(a, sa, b, sb))
    x = torch.as_strided(buf, (4, 300), (stride, 1))
    x.copy_(torch.randn(4, 300, device="cuda"))
    far = torch.empty(3 * stride + 304, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    q = torch.as_strided(far, (4, 300), (stride, 1))
    for call in (lambda **k: ce.ce_quantize_fp8(k.pop("x"), **k),
                 lambda **k: ce.ce_rms_norm_fp8(k.pop("x"), torch.ones(300, device="cuda"), **k)):
        got, want = call(x=x, q=q), call(x=x.contiguous())
        assert torch.equal(got[0].contiguous().view(torch.uint8), want[0].contiguous().view(torch.uint8))
        assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [131200, 131203])
def test_gemm_output_past_32_bits(ce, n, dtype):
    m, k = (17000, 100) if dtype == "bf16" else (16500, 100)
    a, sa, b, sb, _ = operands(ce, m, n, k, 5)
    out = ce.ce_gemm_fp8(a, sa, b, sb, out_dtype=DT[dtype])
    at = torch.tensor([0, 255, 256, 8191, 16383, 16384, 16400, m - 1], device="cuda")
    F.check_gemm(out[at], a.view(torch.uint8)[at].view(torch.float8_e4m3fn), sa[at], b, sb)


@pytest.mark.parametrize("shape", [(20000, 100, 256), (3000, 16, 130), (40000, 1, 128), (1, 300000, 16), (66, 9728, 384), (640, 640, 20000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gemm_long_sides(ce, shape):
    test_gemm(ce, shape, "bf16")


FIRST = """
import torch, softmax_cross_entropy_pass_gb300 as ce
x = torch.randn({B}, 4, 256, device="cuda").bfloat16()
w = torch.ones(256, device="cuda")
W = (torch.randn({V}, 256, device="cuda") * 0.1).bfloat16()
draft = torch.randint(0, {V}, ({B}, 3), device="cuda")
u, r = torch.rand({B}, 3, device="cuda"), torch.rand({B}, device="cuda")
ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
def step():
    W8, s = ce.ce_quantize_fp8(W, block_rows=128)
    z = ce.fp8_head_logits(x, w, W8, s)
    return (z,) + ce.ce_verify_drafts(z, draft, u, r, ws=ws)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, step()))
print("first calls captured")
"""


@pytest.mark.parametrize("size", [(2, 3001), (260, 20000)])
def test_first_calls_captured(size):
    """A process whose very first calls are captured into a graph."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-c", FIRST.format(B=size[0], V=size[1])], cwd=root, capture_output=True, text=True, timeout=200)
    assert got.returncode == 0 and "first calls captured" in got.stdout, got.stderr[-2000:]
