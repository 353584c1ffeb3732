"""The 8-bit serving head where roundings, scales, references and lifetimes
meet their ends: against the bytes' own rule, and against fp64 with the
tolerances of fp8_check.py."""
import math

import pytest
import torch

import fp8_check as F

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ce():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import softmax_cross_entropy_pass_gb300 as ce
    return ce


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---------------------------------------------------------------------- bytes
def nearest(y, tall=1):
    """(bytes, scales) of fp32 y on the CPU: one division a block for its scale, one an element, one rounding to e4m3."""
    rows, cols = y.shape
    n, m = -(-rows // tall), -(-cols // 128)
    wide = torch.zeros(n * tall, m * 128)
    wide[:rows, :cols] = y
    t = wide.view(n, tall, m, 128)
    scale = (t.abs().amax((1, 3)) / 448.0).clamp_min(2.0 ** -126)
    q = (t / scale[:, None, :, None]).view(n * tall, m * 128)[:rows, :cols].to(E4M3)
    return q.contiguous().view(torch.uint8), scale


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("shape", [(600, 1000), (130, 4096), (257, 129)], ids=lambda s: "x".join(map(str, s)))
def test_quantized_bytes_are_the_nearest(ce, dtype, tall, shape):
    """Every byte is the nearest e4m3 of the fp32 quotient y / scale, ties to even: 16-bit inputs meet many ties."""
    x = torch.empty(shape, device="cuda").normal_(0, 1, generator=gen(shape[0])).to(DT[dtype])
    q, s = ce.ce_quantize_fp8(x, block_rows=tall)
    want, scale = nearest(x.float().cpu(), tall)
    assert torch.equal(s.cpu(), scale)
    assert torch.equal(q.contiguous().view(torch.uint8).cpu(), want)


def test_quantized_bytes_of_any_magnitude(ce):
    """Blocks from the least fp32 numbers to the largest, scales whose reciprocal or remainders leave the normal range."""
    g = gen(2)
    for dtype, lo, hi in (("f32", -148, 126), ("bf16", -132, 126), ("f16", -23, 14)):
        x = torch.randn(hi - lo, 300, generator=g, device="cuda", dtype=torch.float64).clamp(-1.9, 1.9)
        x = (x * torch.exp2(torch.arange(lo, hi, device="cuda", dtype=torch.float64))[:, None]).to(DT[dtype])
        x[:, 7], x[:, 8] = 0.0, -0.0
        q, s = ce.ce_quantize_fp8(x)
        want, scale = nearest(x.float().cpu())
        assert torch.equal(s.cpu(), scale)
        assert torch.equal(q.contiguous().view(torch.uint8).cpu(), want)


def test_quantized_tie(ce):
    """-1.3671875 over a scale of 3.0625 / 448 is -200, between -192 and -208: the even one is -192."""
    x = torch.zeros(128, 128, device="cuda", dtype=torch.bfloat16)
    x[0, 0], x[0, 1] = 3.0625, -1.3671875
    for tall in (1, 128):
        q, _ = ce.ce_quantize_fp8(x, block_rows=tall)
        assert q[0, :2].float().tolist() == [448.0, -192.0]


@pytest.mark.parametrize("cols", [200, 1000, 4096, 9000, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_bytes_are_the_nearest(ce, cols, dtype):
    """Rows of 1 and -1 have a root mean square of exactly 1, so that y is the weight, with signs."""
    g = gen(cols)
    x = (torch.randint(0, 2, (40, cols), generator=g, device="cuda") * 2 - 1).to(DT[dtype])
    w = torch.randn(cols, generator=g, device="cuda").to(torch.bfloat16).to(DT[dtype])
    q, s, _ = ce.ce_rms_norm_fp8(x, w, eps=0.0)
    want, scale = nearest((x.float() * w.float()).cpu())
    assert torch.equal(s.cpu(), scale)
    assert torch.equal(q.contiguous().view(torch.uint8).cpu(), want)


# ---------------------------------------------------------------------- lifetimes
@pytest.mark.parametrize("residual", [True, False])
def test_head_of_strided_states_on_another_stream(ce, residual):
    """Hidden states that cannot be viewed as rows are copied. The copies live until the other stream has read them,
    whatever the current stream allocates meanwhile."""
    B, K1, H, V = 64, 4, 4096, 3001
    g = gen(11)
    x = torch.randn(K1, B, H, generator=g, device="cuda").bfloat16().transpose(0, 1)
    r = torch.randn(K1, B, H, generator=g, device="cuda").bfloat16().transpose(0, 1) if residual else None
    w = torch.ones(H, device="cuda")
    W8, ws = ce.ce_quantize_fp8(torch.randn(V, H, generator=g, device="cuda"), block_rows=128)
    want = ce.fp8_head_logits(x, w, W8, ws, residual=r)
    side, busy = torch.cuda.Stream(), torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    for handle in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                torch.mm(busy, busy)
        got = ce.fp8_head_logits(x, w, W8, ws, residual=r, stream=handle)
        # memory of the copies' size, written by the current stream at once
        over = [torch.full((B * K1, H), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del over, got


# ---------------------------------------------------------------------- ends of sequences
@pytest.mark.parametrize("size", [(5, 3, 5003), (200, 3, 30011), (200, 40, 17003)], ids=["at_once", "clusters", "many"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_verify_valid_drafts_behind_a_missing_one(ce, size, dtype):
    """Drafts like [7, -1, 5]: nothing behind the missing one counts, whatever its rows and random numbers hold."""
    B, K, V = size
    g = gen(13)
    z = torch.empty(B, K + 1, V, device="cuda").normal_(0, 2, generator=g).to(DT[dtype])
    y = (z[:, :K].float() + torch.empty(B, K, V, device="cuda").normal_(0, 0.5, generator=g)).to(DT[dtype])
    draft = y.argmax(2)
    u, r = torch.rand(B, K, generator=g, device="cuda") * 0.2, torch.rand(B, generator=g, device="cuda")
    at = torch.randint(0, K + 1, (B,), generator=g, device="cuda")
    place = torch.arange(K, device="cuda")
    draft = torch.where(place == at[:, None], -1, draft)
    cut = torch.where(place > at[:, None], -1, draft)
    for model in (y, None):
        for t in (1.0, 0.0):
            want = ce.ce_verify_drafts(z, cut, u, r, draft_logits=model, temperature=t)
            zz, yy, uu = z.clone(), y.clone(), u.clone()
            zz[torch.arange(K + 1, device="cuda") > at[:, None]] = math.nan
            yy[place >= at[:, None]] = math.nan
            uu[place >= at[:, None]] = math.nan
            got = ce.ce_verify_drafts(zz, draft, uu, r, draft_logits=None if model is None else yy, temperature=t)
            assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------- references
FAR = [
    # dtype, offset, step between logits, temperature
    ("f32", 2e7, 2.0, 1.0), ("f32", -2e7, 2.0, 2.0), ("f32", 1e12, 65536.0, 1e4), ("f32", 1e15, 2.0 ** 27, 1e4),
    ("f32", 1e6, 0.0625, 1e-4), ("f32", -3e37, 2.0 ** 102, 1.0), ("f32", 1.2e38, 2.0 ** 103, 0.5), ("bf16", 1e10, 2.0 ** 26, 1e4),
    ("bf16", 2.0 ** 33, 2.0 ** 26, 1.0), ("bf16", -1e38, 2.0 ** 119, 0.7), ("f16", 4e4, 32.0, 1e-4), ("f16", -4e4, 32.0, 30.0),
]


def far_inputs(B, K, V, dtype, offset, step, seed):
    """Rows of four neighbouring values around the offset, both models' alike but for some of their entries."""
    g = gen(seed)
    z = torch.randint(0, 4, (B, K + 1, V), generator=g, device="cuda")
    move = torch.rand(B, K, V, generator=g, device="cuda") < 0.2
    y = torch.where(move, torch.randint(0, 4, (B, K, V), generator=g, device="cuda"), z[:, :K])
    z, y = ((offset + step * v.double()).to(DT[dtype]) for v in (z, y))
    draft = torch.where(torch.rand(B, K, generator=g, device="cuda") < 0.8, y.argmax(2), torch.randint(0, V, (B, K), generator=g, device="cuda"))
    return z, y, draft, torch.rand(B, K, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")


@pytest.mark.parametrize("case", FAR, ids=lambda c: f"{c[0]}{c[1]:g}T{c[3]:g}")
@pytest.mark.parametrize("size", [(6, 2, 3001), (160, 1, 30011)], ids=["at_once", "clusters"])
def test_verify_rows_far_from_zero(ce, case, size):
    """Finite logits are defined wherever they lie: their exponents' reference times log2(e) / T may round by whole
    powers of two, or leave fp32's range."""
    dtype, offset, step, t = case
    z, y, draft, u, r = far_inputs(*size, dtype, offset, step, 5)
    pick = torch.arange(0, size[0], max(1, size[0] // 24), device="cuda")
    for model in (y, None):
        for temp in (t, 0.0):
            got = ce.ce_verify_drafts(z, draft, u, r, draft_logits=model, temperature=temp)
            assert (got[1][torch.arange(size[0], device="cuda"), got[0].long()] >= 0).all()
            F.check_verify(z[pick], None if model is None else y[pick], draft[pick].cpu(), u[pick].cpu(), r[pick].cpu(), temp,
                           tuple(v[pick] for v in got))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [(6, 2, 5000), (300, 2, 20000)], ids=["at_once", "clusters"])
def test_verify_wholly_masked_rows(ce, dtype, size):
    """A row wholly at its type's lowest value is uniform: index 0 for greedy, any token otherwise."""
    B, K, V = size
    low = torch.finfo(DT[dtype]).min
    g = gen(7)
    z = torch.full((B, K + 1, V), low, device="cuda", dtype=DT[dtype])
    z[::2, 0, 17] = 1.0                         # (the first draft of every second sequence is certain)
    draft = torch.randint(1, V, (B, K), generator=g, device="cuda")
    draft[::2, 0] = 17
    draft[1::3, 1] = 0
    u, r = torch.rand(B, K, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    y = z[:, :K].clone()
    y[::4, 1] = torch.randn(V, generator=g, device="cuda").to(DT[dtype])
    pick = torch.arange(0, B, max(1, B // 24), device="cuda")
    for model in (None, y):
        for t in (1.0, 0.5, 1e-4, 0.0):
            got = ce.ce_verify_drafts(z, draft, u, r, draft_logits=model, temperature=t)
            F.check_verify(z[pick], None if model is None else y[pick], draft[pick].cpu(), u[pick].cpu(), r[pick].cpu(), t,
                           tuple(v[pick] for v in got))


# ---------------------------------------------------------------------- nothing left over
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [(4, 2, 5000), (3, 1, 128256), (200, 2, 17003), (128, 1, 80000), (160, 1, 30011)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("shift", [0.0, 2.0])
def test_verify_equal_rows_draw_from_the_target(ce, dtype, size, shift):
    """Both models' rows are equal (or equal but for a constant), and a number above 1 turns the first draft down: there
    is nothing in max(p - q, 0), and the token is p's, at its place on p's cumulative sum."""
    B, K, V = size
    g = gen(V)
    # multiples of 1/16: adding the constant is exact in every type
    y = (torch.empty(B, K, V, device="cuda").normal_(0, 2, generator=g) * 16).round().div(16).clamp(-6, 6)
    z = torch.cat([y + shift, y[:, :1]], 1).to(DT[dtype])
    y = y.to(DT[dtype])
    draft = y.argmax(2)
    u, r = torch.full((B, K), 1.0 + 2.0 ** -10, device="cuda"), torch.rand(B, generator=g, device="cuda")
    n, tokens, logp = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y)
    assert (n == 0).all()
    p = torch.softmax(z[:, 0].double(), 1)
    upto = p.cumsum(1)
    at = tokens[:, :1]
    end = upto.gather(1, at)[:, 0]
    start = end - p.gather(1, at)[:, 0]
    assert ((start <= r + 4 * F.rel(V)) & (end >= r - 4 * F.rel(V))).all()


@pytest.mark.parametrize("size", [(4, 5003), (160, 30011)], ids=["at_once", "clusters"])
@pytest.mark.parametrize("part", [1e-4, 1e-6, 1e-8])
def test_verify_little_left_over(ce, size, part):
    """One token of the target above the draft model's by a small part of all probability: what is left over is that
    token's alone, however little it is beside the roundings of the others."""
    B, V = size
    g = gen(3)
    y = torch.empty(B, 1, V, device="cuda").normal_(0, 1, generator=g)
    at = torch.randint(0, V, (B,), generator=g, device="cuda")
    rows = torch.arange(B, device="cuda")
    total = torch.logsumexp(y[:, 0].double(), 1)
    y[rows, 0, at] = (total + math.log(part)).float()
    z = torch.cat([y, y], 1)
    z[rows, 0, at] += 1.0                                   # e times as likely, before the sum grows by as little
    draft = torch.where(y[:, 0].argmax(1) == at, 0, y[:, 0].argmax(1))[:, None]
    u, r = torch.full((B, 1), 1.25, device="cuda"), torch.rand(B, generator=g, device="cuda")
    n, tokens, _ = ce.ce_verify_drafts(z, draft, u, r, draft_logits=y)
    assert (n == 0).all() and torch.equal(tokens[:, 0], at)


# ---------------------------------------------------------------------- scales
SCALED = [(5, 300, 260), (40, 1000, 4500), (70, 300, 260), (130, 20000, 384), (300, 20003, 384)]


def scaled_operands(m, n, k, seed):
    g = gen(seed)
    a = torch.randn(m, -(-k // 16) * 16, generator=g, device="cuda").mul_(40).to(E4M3)[:, :k]
    b = torch.randn(n, -(-k // 16) * 16, generator=g, device="cuda").mul_(40).to(E4M3)[:, :k]
    blocks = -(-k // 128)
    return a, 1 + torch.rand(m, blocks, generator=g, device="cuda"), b, 1 + torch.rand(-(-n // 128), blocks, generator=g, device="cuda")


def check_scaled(out, a, sa, b, sb):
    """check_gemm's tolerance, and half a step of the least fp32 number for each block's addition."""
    d, s = F.gemm_ref(a, sa, b, sb)
    tol = s * (16 + sa.shape[1] + 3) * F.U + d.abs() * F.HALF[out.dtype] * (1 + 2.0 ** -10) + (d.abs() + s) * F.U
    tol = tol + (sa.shape[1] + 1) * 2.0 ** -149
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -134
    assert ((out.double() - d).abs() <= tol).all(), float(((out.double() - d).abs() / tol).max())


@pytest.mark.parametrize("shape", SCALED, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ends", [(1e-22, 1e-22), (2.0 ** -120, 1e-9), (1e-14, 2.0 ** -126), (2.0 ** -149, 2.0 ** 20), (1e19, 1e-40)],
                         ids=lambda e: f"{e[0]:.0e}x{e[1]:.0e}")
def test_gemm_scales_with_tiny_products(ce, shape, ends):
    """The product of two scales below fp32's normal range, their results in or near it."""
    a, sa, b, sb = scaled_operands(*shape, 3)
    sa, sb = (sa.double() * ends[0]).float(), (sb.double() * ends[1]).float()
    sa[::2, 1] = 1.5 / ends[1] * 1e-30                      # rows with ordinary blocks among them
    for dtype in (torch.float32, torch.bfloat16):
        check_scaled(ce.ce_gemm_fp8(a, sa, b, sb, out_dtype=dtype), a, sa, b, sb)


@pytest.mark.parametrize("shape", SCALED, ids=lambda s: "x".join(map(str, s)))
def test_gemm_scales_with_huge_products(ce, shape):
    """The product of two scales above fp32's range: blocks of zeros add 0, and small sums stay finite."""
    m, n, k = shape
    a, sa, b, sb = scaled_operands(m, n, k, 4)
    a, b = a.float(), b.float()
    a[1, :128] = 0                                          # row 1, block 0: zeros under a huge scale
    a[2, :128] = 0
    a[2, 3], b[:, 3] = 2.0 ** -9, 2.0 ** -9                 # row 2, block 0: a sum of 2^-18
    a, b = (padded8(v) for v in (a, b))
    sa[1, 0] = sa[2, 0] = 2.0 ** 67
    sb[:, 0] = 2.0 ** 63
    sa[0, 0] = 2.0 ** -63
    sa[3:, 0] = 2.0 ** -64
    out = ce.ce_gemm_fp8(a, sa, b, sb, out_dtype=torch.float32)
    assert out.isfinite().all()
    check_scaled(out, a, sa, b, sb)
    sa[1, 0] = math.inf                                     # an infinite scale is no number of its block's zeros
    out = ce.ce_gemm_fp8(a, sa, b, sb, out_dtype=torch.float32)
    assert out[1].isnan().all() and out[0].isfinite().all() and out[2:].isfinite().all()


def padded8(v):
    """e4m3 with rows at multiples of 16 bytes."""
    buf = torch.zeros(v.shape[0], -(-v.shape[1] // 16) * 16, device=v.device)
    buf[:, :v.shape[1]] = v
    return buf.to(E4M3)[:, :v.shape[1]]


@pytest.mark.parametrize("shape", [(40, 3000, 1024), (300, 20000, 384)], ids=lambda s: "x".join(map(str, s)))
def test_gemm_rows_of_zeros_leave_the_others_alone(ce, shape):
    """Rows of zeros carry the least scale, whose product with a weight's is below the normal range: they come out 0,
    and the others bit for bit as without them."""
    m, n, k = shape
    g = gen(6)
    x = torch.randn(m, k, generator=g, device="cuda")
    W8, sb = ce.ce_quantize_fp8(torch.randn(n, k, generator=g, device="cuda") * 0.02, block_rows=128)
    q, s = ce.ce_quantize_fp8(x)
    want = ce.ce_gemm_fp8(q, s, W8, sb, out_dtype=torch.float32)
    zero = torch.arange(m, device="cuda") % 3 == 1
    x[zero] = 0
    q, s = ce.ce_quantize_fp8(x)
    got = ce.ce_gemm_fp8(q, s, W8, sb, out_dtype=torch.float32)
    assert (got[zero] == 0).all() and torch.equal(got[~zero], want[~zero])


@pytest.mark.parametrize("shape", [(40, 700, 8320), (70, 9900, 8320), (300, 5003, 8320)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("kind", ["low behind zeros", "high behind low", "mixed", "zeros under high"])
def test_gemm_scales_that_change_along_k(ce, shape, kind):
    """65 blocks along K whose scales change their order of magnitude on the way."""
    m, n, k = shape
    a, sa, b, sb = scaled_operands(m, n, k, 8)
    a = a.float()
    if kind == "low behind zeros":
        a[:, :40 * 128] = 0
        sa[:, 40:] *= 2.0 ** -70
        sb[:, 40:] *= 2.0 ** -70
    elif kind == "high behind low":
        sa[:, :40] *= 2.0 ** -70
        sb[:, :40] *= 2.0 ** -65
        sa[1::2, 40:] = 0                                   # (half of the rows have the low ones alone)
    elif kind == "mixed":
        sa *= torch.exp2(torch.randint(-60, 60, sa.shape, generator=gen(9), device="cuda").float())
        sb *= torch.exp2(torch.randint(-60, 0, sb.shape, generator=gen(10), device="cuda").float())
    else:
        a[::2, 33 * 128:34 * 128] = 0
        sa[::2, 33] = 2.0 ** 70
        sb[:, 33] = 2.0 ** 62
        sa[1::2, 33] = 2.0 ** -62
    a = padded8(a)
    out = ce.ce_gemm_fp8(a, sa, b, sb, out_dtype=torch.float32)
    check_scaled(out, a, sa, b, sb)
