"""w4_rmsnorm against a 64-bit numpy implementation.

Tolerance.  The kernel computes y in fp32: h = x + r (one rounding), a sum of
squares whose every chain is shorter than 128 additions, and three operations
behind it, so y is within a factor 1 +- d of the exact value with
d < (128 / 2 + 1 + 1 + 3 + 2) * 2^-24 < 2^-16.  Rounding is monotone: the stored
value has to lie between the roundings of y (1 - d) and y (1 + d), which is the
exact rounding itself except next to a tie.
"""
import numpy as np
import pytest

from bit_gemm_quant_b200 import synth
from parity import dev_bf16, host_u16
from test_parity_mx import mma_layout

D = 2.0 ** -16
EPS = 1e-6


@pytest.fixture(scope="module")
def w4():
    from bit_gemm_quant_b200 import build
    build.build()
    import bit_gemm_quant_b200 as w4
    w4.lib()
    return w4


def bf16(a: np.ndarray) -> np.ndarray:
    """The nearest bf16 value, ties to even, of fp64 values (normal range, and zero)."""
    m, e = np.frexp(a)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def e4m3(a: np.ndarray) -> np.ndarray:
    """The nearest E4M3 value, ties to even, saturating at 448."""
    e = np.maximum(np.frexp(a)[1] - 1, -6)
    return np.clip(np.ldexp(np.rint(np.ldexp(a, 3 - e)), e - 3), -448.0, 448.0)


def f64(bits: np.ndarray) -> np.ndarray:
    return synth.bf16_bits_to_f32(bits).astype(np.float64)


def reference(x, r, gamma, eps=EPS):
    h = f64(x) + (f64(r) if r is not None else 0.0)
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * f64(gamma)


def between(got, exact, rnd, what):
    lo, hi = rnd(exact * (1 - D)), rnd(exact * (1 + D))
    ok = (np.minimum(lo, hi) <= got) & (got <= np.maximum(lo, hi))
    assert ok.all(), "%s: %d of %d outside, first %s: %r for %r" % (
        what, (~ok).sum(), ok.size, np.argwhere(~ok)[0], got[~ok][0], exact[~ok][0])


def check_codes(codes, scales, y):
    """codes uint8 [M, K] and scales uint8 [M, K/32] against the exact y."""
    M, K = y.shape
    block = np.abs(y).reshape(M, K // 32, 32).max(2)
    lo, hi = (np.where(b > 0, np.clip(np.frexp(b)[1] - 1 - 8, -127, 127), -127) + 127
              for b in (block * (1 - D), block * (1 + D)))
    assert ((lo <= scales) & (scales <= hi)).all(), "scales"
    s = np.ldexp(1.0, scales.astype(np.int32) - 127)
    sign, mag = codes >> 7, codes & 0x7F
    e, m = (mag >> 3).astype(np.int32), (mag & 7).astype(np.float64)
    v = np.where(e > 0, np.ldexp(1 + m / 8, e - 7), m * 2.0 ** -9) * np.where(sign, -1.0, 1.0)
    assert (mag != 0x7F).all()
    between(v, y / np.repeat(s, 32, axis=1), e4m3, "codes")


def inputs(M, K, seed=0, residual=True):
    x = synth.activations(seed + 1, M, K, outlier_frac=0.01, outlier_mult=40.0)
    r = synth.activations(seed + 2, M, K, outlier_frac=0.02, outlier_mult=9.0) if residual else None
    gamma = synth.to_bf16_bits(1 + 0.3 * np.random.default_rng(seed + 3).standard_normal(K))
    return x, r, gamma


def dev(a):
    return None if a is None else dev_bf16(a)


# one element; rows within a warp, one vector over it, over a CTA; the longest;
# rows that are no whole vectors; many short rows
SHAPES = [(1, 1), (3, 7), (5, 8), (2, 64), (9, 256), (17, 264), (3, 512), (4, 520), (1, 4096), (33, 4096), (2, 8192),
          (1, 8200), (2, 16384), (1, 32768), (2, 32767), (7, 1001), (300, 136), (1000, 96), (2, 4098), (700, 2048),
          (400, 12288)]


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", SHAPES)
def test_bf16_out(w4, M, K, residual):
    x, r, gamma = inputs(M, K, residual=residual)
    Y, H = w4.rmsnorm(dev(x), dev(gamma), EPS, residual=dev(r))
    h, y = reference(x, r, gamma)
    between(f64(host_u16(Y)), y, bf16, "Y")
    if residual:
        between(f64(host_u16(H)), h, bf16, "H")
    else:
        assert H is None


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,layout", [(1, 32, 0), (5, 96, 0), (3, 1056, 0), (1, 128, 1), (130, 256, 1), (37, 4096, 1),
                                        (128, 640, 1), (2, 8192, 0), (5, 16384, 1), (1, 32768, 1), (1000, 384, 1),
                                        (700, 2048, 1), (600, 992, 0)])
def test_mxfp8_out(w4, M, K, layout):
    x, r, gamma = inputs(M, K, 7)
    codes, scales, H = w4.rmsnorm_mxfp8(dev(x), dev(gamma), EPS, residual=dev(r), scale_layout=layout)
    h, y = reference(x, r, gamma)
    sc = scales.cpu().numpy()
    if layout == w4.MX_SCALES_MMA:
        rows = np.zeros((M, K // 32), np.uint8)
        at = mma_layout(np.arange(M * (K // 32)).reshape(M, -1) % 251 + 1, K)      # where each row's scales went
        want = mma_layout(np.ones((M, K // 32), np.uint8), K)
        assert (sc[want == 0] == 0).all(), "padding rows"
        kb = np.arange(K // 32)
        for i in range(M):
            off = ((i // 128) * (K // 128) + kb // 4) * 512 + (i % 32) * 16 + ((i % 128) // 32) * 4 + kb % 4
            assert (at[off] == (i * (K // 32) + kb) % 251 + 1).all()
            rows[i] = sc[off]
        sc = rows
    check_codes(codes.cpu().numpy(), sc, y)
    between(f64(host_u16(H)), h, bf16, "H")


@pytest.mark.gpu
def test_both_outputs_and_the_product_behind_them(w4):
    """Y and codes of one call agree with the calls for one of them, and the
    codes are what w4_mx_gemm reads."""
    import torch
    M, K, N = 20, 512, 256
    x, r, gamma = (dev(a) for a in inputs(M, K, 11))
    Y, H = w4.rmsnorm(x, gamma, EPS, residual=r)
    codes, scales, H2 = w4.rmsnorm_mxfp8(x, gamma, EPS, residual=r)
    Y2, H3 = torch.empty_like(Y), torch.empty_like(Y)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    p = lambda t: t.data_ptr()
    st = w4.w4_rmsnorm(p(x), p(r), p(gamma), M, K, EPS, p(H3), p(Y2), p(c2), p(s2), w4.MX_SCALES_MMA,
                       torch.cuda.current_stream().cuda_stream)
    assert st == w4.W4_OK
    for a, b in ((Y, Y2), (H, H2), (H, H3), (codes, c2), (scales, s2)):
        assert torch.equal(a, b)
    W = dev_bf16(synth.weights(3, N, K, 0.02))
    wc, ws = w4.fp4_quant(W, w4.MXFP4)
    out = w4.mx_gemm(codes, scales, wc, w4.mx_scale_layout(ws, K))
    xq, xs = w4.mxfp8_quant(Y, w4.MX_SCALES_MMA)
    other = w4.mx_gemm(xq, xs, wc, w4.mx_scale_layout(ws, K))
    # the second went through bf16 as well: each product term is off by its rounding (2^-8) and
    # by at most one E4M3 step that it tips (2^-3, rare); their norm is far below 2^-4 of the whole
    assert (out.float() - other.float()).norm() <= 2.0 ** -4 * other.float().norm()


@pytest.mark.gpu
@pytest.mark.parametrize("K", [512, 1003, 4096])
def test_in_place(w4, K):
    """H over the residual or over X, Y over X: the same bits."""
    import torch
    x, r, gamma = (dev(a) for a in inputs(9, K, 21))
    Y, H = w4.rmsnorm(x, gamma, EPS, residual=r)
    x1, r1 = x.clone(), r.clone()
    Y1, H1 = w4.rmsnorm(x1, gamma, EPS, residual=r1, out=(x1, r1))
    assert torch.equal(Y1, Y) and torch.equal(H1, H) and Y1.data_ptr() == x1.data_ptr()
    x2 = x.clone()
    Y2, _ = w4.rmsnorm(x2, gamma, EPS, residual=r, out=(torch.empty_like(x), x2))
    assert torch.equal(Y2, Y) and torch.equal(x2, H)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(9000, 7), (5000, 129), (3000, 1003), (700, 4098), (333, 32767), (2, 1001)])
def test_in_place_rows_that_share_vectors(w4, M, K):
    """Rows that are no whole vectors, in place: many at once on either side of every shared vector, and the
    arrays' own end."""
    import torch
    x, r, gamma = (dev(a) for a in inputs(M, K, 22))
    Y, H = w4.rmsnorm(x, gamma, EPS, residual=r)
    for _ in range(3):
        x1, r1 = x.clone(), r.clone()
        w4.rmsnorm(x1, gamma, EPS, residual=r1, out=(x1, r1))
        assert torch.equal(x1, Y) and torch.equal(r1, H)
    x2, Y2 = x.clone(), torch.empty_like(x)
    w4.rmsnorm(x2, gamma, EPS, residual=r, out=(Y2, x2))
    assert torch.equal(Y2, Y) and torch.equal(x2, H)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [256, 1024, 1003])
def test_zero_rows_and_extremes(w4, K):
    """An all-zero row gives zeros; x = -r gives zeros; tiny rows stand on eps;
    rows near the largest sum of squares stay finite.  No element outside the
    outputs is written."""
    import torch
    x = np.zeros((5, K), np.float32)
    r = np.zeros((5, K), np.float32)
    x[1] = np.linspace(-2, 2, K)
    r[1] = -synth.bf16_bits_to_f32(synth.to_bf16_bits(x[1]))
    x[2] = 1e-20
    x[3] = np.where(np.arange(K) % 2, 1e17, -1e17)
    x[4] = 1.0
    xb, rb = synth.to_bf16_bits(x), synth.to_bf16_bits(r)
    gamma = synth.to_bf16_bits(np.linspace(0.5, 1.5, K, dtype=np.float32))
    big = torch.full((7, K), 7.0, dtype=torch.bfloat16, device="cuda")
    Y, H = w4.rmsnorm(dev(xb), dev(gamma), EPS, residual=dev(rb), out=(big[1:6], torch.empty_like(big[1:6])))
    h, y = reference(xb, rb, gamma)
    between(f64(host_u16(Y)), y, bf16, "Y")
    assert (Y[:2] == 0).all() and (big[0] == 7).all() and (big[6] == 7).all()


@pytest.mark.gpu
def test_unaligned_pointers(w4):
    """2-byte aligned rows of whole vectors take the other kernel and agree."""
    import torch
    M, K = 6, 1024
    x, r, gamma = inputs(M, K, 31)
    buf = torch.zeros(M * K + 1, dtype=torch.bfloat16, device="cuda")
    xs = buf[1:].view(M, K)
    xs.copy_(dev(x))
    Y, H = w4.rmsnorm(xs, dev(gamma), EPS, residual=dev(r))
    h, y = reference(x, r, gamma)
    between(f64(host_u16(Y)), y, bf16, "Y")
    between(f64(host_u16(H)), h, bf16, "H")


@pytest.mark.gpu
@pytest.mark.parametrize("K", [8192, 8191])
def test_rows_past_32_bits(w4, K):
    """More than 2^31 elements: the last rows are as they are alone."""
    import torch
    M = 2 ** 31 // K + 50
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail, _, gamma = inputs(40, K, 41, residual=False)
    x[-40:] = dev(tail)
    x[0] = dev(tail)[0]
    Y, _ = w4.rmsnorm(x, dev(gamma), EPS)
    Z, _ = w4.rmsnorm(x[-40:].clone(), dev(gamma), EPS)
    assert (Y[1:-40] == 0).all() and torch.equal(Y[0], Z[0])
    _, y = reference(tail, None, gamma)
    between(f64(host_u16(Y[-40:])), y, bf16, "Y")


# ------------------------------------------------------------- refusals --

FAKE = 1 << 20


def call(w4, X=FAKE, r=FAKE, gamma=FAKE, M=4, K=256, eps=1e-6, H=FAKE + (1 << 16), Y=FAKE, codes=None, scales=None, layout=0):
    return w4.w4_rmsnorm(X, r, gamma, M, K, eps, H, Y, codes, scales, layout, None)


@pytest.mark.parametrize("bad", [
    dict(X=None), dict(gamma=None), dict(Y=None), dict(M=0), dict(M=-1), dict(K=0), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(r=None), dict(X=FAKE + 1), dict(Y=FAKE + 1), dict(H=FAKE + (1 << 16) + 1),
    dict(codes=FAKE), dict(scales=FAKE), dict(layout=2), dict(codes=FAKE, scales=FAKE, K=40),
    dict(codes=FAKE, scales=FAKE, K=96, layout=1), dict(codes=FAKE + 8, scales=FAKE),
    dict(codes=FAKE, scales=FAKE + 8, layout=1), dict(codes=FAKE, scales=FAKE, X=FAKE + 2),
    dict(codes=FAKE, scales=FAKE, gamma=FAKE + 8), dict(M=1 << 61, K=256), dict(H=FAKE + 4096, Y=FAKE + 4096)])
def test_refusals(w4, bad):
    assert call(w4, **bad) == w4.W4_ERR_INVALID_ARG


@pytest.mark.parametrize("big", [dict(K=32776), dict(M=1 << 31)])
def test_unsupported(w4, big):
    assert call(w4, **big) == w4.W4_ERR_UNSUPPORTED


def test_helper_refusals(w4):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    g = torch.zeros(64, dtype=torch.bfloat16)
    for args in ((x, g), (x.float(), g), (x[0], g), (x.t(), g)):
        with pytest.raises(ValueError):
            w4.rmsnorm(*args, 1e-6)
        with pytest.raises(ValueError):
            w4.rmsnorm_mxfp8(*args, 1e-6)
