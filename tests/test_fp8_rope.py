"""The block-scaled FP8 linear layer and the query/key norm with rotation,
against plain implementations in 64 bits.

Tolerances (u = 2^-24, half a step of fp32; half steps of the 16-bit types
2^-11 and 2^-8, of e4m3 2^-4):

* codes: the kernel's value before rounding differs from the exact one by a
  relative error `eps`; a code may differ from the exactly rounded one only
  where the exact value lies within eps of the middle between two codes, and
  then it is the other of the two.
* scales: relative error of the block's values plus u for the division.
* GEMM: the 128 products of a block are exact; their fp32 sum is held to
  2 * 128 u of the sum of magnitudes (any order, with a factor two for adders
  that truncate, as for the FP16-activation GEMMs), the scaling of a block and
  the sum over blocks to (4 + blocks) u of the scaled magnitudes (products of
  two scales, product with the block, one addition per block, the bias), and
  half a step of the output type for the one rounding.
* norm and rotation: sums of D values and their reciprocal root within
  (D + 8) u, sine and cosine within 4 u, then six roundings of fp32 and half a
  step of the output type.
"""
import math
import os
import subprocess
import sys
import threading
import unittest.mock as mock

import numpy as np
import pytest
import torch

F8 = torch.float8_e4m3fn
U = 2.0 ** -24
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half of the smallest subnormal
DTYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def zq():
    from int4_quantized_transformer_b200 import build

    build.build()
    from int4_quantized_transformer_b200 import zq as m

    return m


@pytest.fixture(autouse=True)
def _device_status_clean(zq, request):
    yield
    if "gpu" in request.keywords and torch.cuda.is_available():
        rc, detail = zq.device_status()
        assert rc == zq.ZQ_OK, f"device status {rc} ({zq.status_str(rc)}), wait site {detail}"


def blocks(n):
    return -(-n // 128)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------ plain forms, 64 bits

def gelu(v):
    return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))  # keeps its digits in the far tail

def e4m3_grid():
    """The 127 finite magnitudes of e4m3, ascending."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(F8).double()
    return codes


def block_max(y, rows):
    n, k = y.shape
    p = torch.nn.functional.pad(y, (0, -k % 128, 0, -n % rows))
    return p.view(p.shape[0] // rows, rows, p.shape[1] // 128, 128).abs().amax(dim=(1, 3))


def spread(s, rows, n, k):
    return s.repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :k]


def check_codes(codes, scales, y, rows, eps):
    """codes (e4m3) and scales of y (64 bits; values known to a relative eps
    plus, for cancelled values, eps of the block's maximum)."""
    n, k = y.shape
    codes, scales = codes.cpu().double(), scales.cpu().double()
    amax = block_max(y, rows)
    a = torch.where(amax > 0, amax.clamp_min(2.0 ** -110), amax)
    assert torch.all((scales - a / 448).abs() <= (eps + 2 * U) * a / 448)
    assert torch.all(scales[amax == 0] == 0)
    full = spread(a, rows, n, k)
    v = torch.where(full > 0, y * 448 / torch.where(full > 0, full, torch.ones_like(full)),
                    torch.zeros_like(y))
    grid = e4m3_grid()
    m = v.abs().clamp_max(448.0)
    hi = torch.searchsorted(grid, m.contiguous()).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    mid = (grid[lo] + grid[hi]) / 2
    # ties go to the even code; indices are the codes themselves
    nearest = torch.where((m > mid) | ((m == mid) & (hi % 2 == 0)), hi, lo)
    nearest = torch.where(m == grid[hi], hi, nearest)
    want = grid[nearest] * torch.sign(v)
    other = torch.where(nearest == hi, lo, hi)
    slack = (eps + 4 * U) * m + eps * 448
    near_tie = (m - mid).abs() <= slack
    ok = (codes == want) | (near_tie & (codes.abs() == grid[other]))
    # a value near zero may change its sign's code only by rounding to zero
    assert ok.all(), f"{(~ok).sum()} codes differ"


def dequantize(q, s, rows):
    return q.cpu().double() * spread(s.cpu().double(), rows, *q.shape)


def quantized(zq, t, rows, seed):
    """Codes and scales of a CPU matrix, by plain arithmetic (not the kernels)."""
    y = t.double()
    amax = block_max(y, rows)
    s = (amax / 448).float()
    safe = torch.where(s > 0, s, torch.ones_like(s)).double()
    q = (y / spread(safe, rows, *y.shape)).clamp(-448, 448).float().to(F8)
    return q.cuda(), s.cuda()


def check_gemm(zq, T, K, N, dtype, bias=True, seed=0, **opts):
    g = gen(seed + 7 * T + 3 * K + N)
    x = torch.randn(T, K, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    x[:, torch.randint(0, K, (max(1, K // 500),), generator=g)] *= 30
    w = torch.randn(N, K, generator=g) * 0.02
    xq, sx = quantized(zq, x, 1, 0)
    wq, sw = quantized(zq, w, 128, 0)
    b = (torch.randn(N, generator=g) * 0.1).to(dtype).cuda() if bias else None
    with zq.options(**opts):
        y = zq.gemm_fp8(xq, sx, wq, sw, b, out_dtype=dtype)
        again = zq.gemm_fp8(xq, sx, wq, sw, b, out_dtype=dtype)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))  # the same bits each time
    X, W = dequantize(xq, sx, 1), dequantize(wq, sw, 128)
    ref, mag = X @ W.T, X.abs() @ W.abs().T
    if bias:
        ref, mag = ref + b.cpu().double(), mag + b.cpu().double().abs()
    tol = (2 * 128 + 4 + blocks(K)) * U * mag
    tol = tol + HALF_STEP[dtype] * (ref.abs() + tol) + TINY[dtype]
    err = (y.cpu().double() - ref).abs()
    assert torch.all(err <= tol), f"worst {(err / tol).max().item():.2f} of the tolerance"
    return y


# ------------------------------------------------------------ quantizers

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (129, 144), (300, 2064), (8, 4096), (1000, 400)])
def test_weights(zq, dtype, N, K):
    w = (torch.randn(N, K, generator=gen(N + K)) * 0.02).to(dtype)
    w[: N // 3] *= 8
    if N > 200:
        w[128:256] = 0
    q, s = zq.quantize_weights_fp8(w.cuda())
    assert q.shape == (N, K) and s.shape == (blocks(N), blocks(K))
    check_codes(q, s, w.double(), 128, 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K", [(1, 16), (1, 128), (3, 144), (37, 4096), (5, 32768), (130, 1040),
                                 (700, 2048)])
def test_rows_as_they_are(zq, dtype, T, K):
    x = torch.randn(T, K, generator=gen(T + K)).to(dtype)
    x[:, 0] *= 100
    q, s = zq.bias_act_quant_fp8(x.cuda())
    check_codes(q, s, x.double(), 1, 0.0)
    y = torch.empty_like(x.cuda())
    q2, s2 = zq.ln_quant_fp8(x.cuda(), y_ln=y)  # gamma None: the same call
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    assert torch.equal(y.cpu(), x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K", [(1, 16), (3, 144), (37, 4096), (2, 32768), (130, 1040)])
@pytest.mark.parametrize("act", [0, 1])
def test_bias_and_gelu(zq, dtype, T, K, act):
    g = gen(T + K + act)
    x, b = (torch.randn(T, K, generator=g) * 2).to(dtype), torch.randn(K, generator=g).to(dtype)
    yd = torch.empty_like(x.cuda())
    q, s = zq.bias_act_quant_fp8(x.cuda(), b.cuda(), act, y=yd)
    v = (x.float() + b.float()).double()  # the add is one fp32 operation
    y = gelu(v) if act else v
    # GeLU in fp32, relative: 1.2e-7 for the polynomial, 2^-22 for the power of
    # two, 3 * 2^-23 for the reciprocal (as a factor and through the
    # polynomial) and some roundings, together below 1e-6.  The exponent
    # -v^2 log2(e) / 2 has three roundings (the square, the constant, the
    # sum), each u of it, and an error of d there is d ln 2 in the result:
    # 1.5 u v^2, which counts in the far tail of negative v.
    eps = 1e-6 if act else 0.0
    check_codes(q, s, y, 1, eps)
    tail = 1.5 * U * v.square() if act else 0.0
    tol = (eps + tail + U + HALF_STEP[dtype]) * y.abs() + TINY[dtype]
    assert torch.all((yd.cpu().double() - y).abs() <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K", [(1, 16), (5, 128), (3, 144), (37, 768), (300, 1024), (5, 1040),
                                 (33, 6144), (2, 16384), (2, 16400), (3, 32768)])
def test_layernorm(zq, dtype, T, K):
    g = gen(T + K)
    x = (torch.randn(T, K, generator=g) + 0.5).to(dtype)
    x[:, torch.randint(0, K, (max(1, K // 1000),), generator=g)] *= 30
    gamma = (1 + 0.1 * torch.randn(K, generator=g)).to(dtype)
    beta = (0.1 * torch.randn(K, generator=g)).to(dtype)
    for bt in (beta, None):
        yd = torch.empty_like(x.cuda())
        q, s = zq.ln_quant_fp8(x.cuda(), gamma.cuda(), None if bt is None else bt.cuda(), 1e-5,
                               y_ln=yd)
        xd = x.double()
        mean = xd.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt(xd.var(1, correction=0, keepdim=True) + 1e-5)
        y = (xd - mean) * rstd * gamma.double() + (0 if bt is None else beta.double())
        # mean: tree sums of at most 32 + 10 levels of fp32 additions, relative
        # to the mean magnitude; variance and its root likewise; then four
        # roundings of magnitudes up to |x - mean| rstd |gamma| + |beta|
        mag = ((xd.abs() + xd.abs().mean(1, keepdim=True)) * rstd * gamma.double().abs()
               + (0 if bt is None else beta.double().abs()))
        err = 64 * U * mag
        assert torch.all((yd.cpu().double() - y).abs() <= err + HALF_STEP[dtype] * (y.abs() + err)
                         + TINY[dtype])
        full = spread(block_max(y, 1), 1, T, K)
        check_codes(q, s, y, 1, float((err / full).max()))


@pytest.mark.gpu
def test_zero_tiny_and_non_finite_blocks(zq):
    x = torch.randn(6, 384, generator=gen(1)).bfloat16()
    x[0] = 0
    x[1, :128] = 2.0 ** -120  # below the floor: codes 448 * 2^-10, a normal scale
    x[2, 200] = float("inf")
    x[3, 200] = float("nan")
    x[4, 5] = 3.0e38
    q, s = zq.bias_act_quant_fp8(x.cuda())
    q, s = q.float().cpu(), s.cpu()
    assert torch.all(s[0] == 0) and torch.all(q[0] == 0)
    assert s[1, 0] == 2.0 ** -110 / 448 and torch.all(q[1, :128] == 448 * 2.0 ** -10)
    for r in (2, 3):
        assert not torch.isfinite(s[r, 1]) and torch.isnan(q[r, 128:256]).all()
        assert torch.isfinite(q[r, :128]).all() and torch.isfinite(s[r, [0, 2]]).all()
    assert abs(s[4, 0].item() * 448 / x[4, 5].item() - 1) < 1e-6 and q[4, 5] == 448
    # weights: a NaN stays inside its 128 x 128 block
    w = torch.randn(260, 256, generator=gen(2)).half()
    w[130, 5] = float("nan")
    q, s = zq.quantize_weights_fp8(w.cuda())
    bad = torch.isnan(q.float()).cpu()
    assert bad[128:256, :128].all() and bad.sum() == 128 * 128
    assert torch.isnan(s.cpu()).sum() == 1 and torch.isnan(s[1, 0])


# ------------------------------------------------------------ GEMM

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,N", [
    (1, 16, 8), (1, 128, 128), (1, 6144, 264), (2, 144, 24), (3, 1024, 1000), (8, 4096, 512),
    (16, 400, 136), (17, 2064, 520), (31, 1040, 640), (33, 768, 2304), (64, 512, 384),
    (65, 272, 136), (127, 128, 128), (128, 2048, 256), (129, 1024, 264), (257, 640, 1032),
    (600, 5008, 2120), (1030, 384, 4104)])
def test_gemm(zq, dtype, T, K, N):
    check_gemm(zq, T, K, N, dtype, bias=(T + K + N) % 3 != 0)


@pytest.mark.gpu
@pytest.mark.parametrize("opts", [
    dict(path=2), dict(path=2, split_k=1), dict(path=2, split_k=3), dict(path=2, split_k=8),
    dict(path=2, max_ctas=7), dict(path=1, bn=128, pair=1), dict(path=1, bn=256, pair=1),
    dict(path=1, bn=128, pair=2), dict(path=1, bn=256, pair=2), dict(path=1, split_k=2),
    dict(path=1, split_k=4), dict(path=1, split_k=8)])
@pytest.mark.parametrize("T,K,N", [(1, 1024, 136), (29, 2064, 520), (64, 1152, 776)])
def test_gemm_every_tiling(zq, opts, T, K, N):
    check_gemm(zq, T, K, N, torch.float16, **opts)


@pytest.mark.gpu
def test_gemm_many_waves(zq):
    # more tiles than CTAs: the persistent loops, their rings and buffers go round
    check_gemm(zq, 900, 272, 12000, torch.float16, path=1, bn=128, pair=1)
    check_gemm(zq, 900, 272, 12000, torch.bfloat16, path=1, bn=256, pair=2)
    check_gemm(zq, 64, 400, 40000, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 300])
def test_gemm_sums_blocks_in_32_bits(zq, T):
    """A large product and its negative in one block with small ones: what
    is left has to be right to the fp32 sum's bound, not to that of fewer bits."""
    K, N = 256, 136
    g = gen(T)
    x = torch.randint(-8, 9, (T, K), generator=g).float()
    w = torch.randint(-8, 9, (N, K), generator=g).float()
    x[:, 3], w[:, 3], x[:, 100], w[:, 100] = 448, 448, 448, -448
    ones = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    y = zq.gemm_fp8(x.to(F8).cuda(), ones(T, 2), w.to(F8).cuda(), ones(2, 2))
    # all products are integers and every partial sum fits 24 bits: exact sums
    ref = x.double() @ w.double().T
    assert ref.abs().max() < 65504
    assert torch.equal(y.cpu(), ref.half())


@pytest.mark.gpu
def test_gemm_nan_and_zero_scales(zq):
    T, K, N = 20, 384, 264
    x, w = torch.randn(T, K, generator=gen(3)), torch.randn(N, K, generator=gen(4))
    xq, sx = quantized(zq, x, 1, 0)
    wq, sw = quantized(zq, w, 128, 0)
    sx[3] = 0  # a zero row: the bias is left
    b = torch.randn(N, generator=gen(5)).half().cuda()
    sx[7, 1] = float("nan")
    for t in (T, 400):
        if t > T:  # the tiles for many tokens
            xq, sx = xq.repeat(20, 1), sx.repeat(20, 1)
        y = zq.gemm_fp8(xq, sx, wq, sw, b)
        assert torch.equal(y[3], b) and torch.isnan(y[7]).all()
        assert torch.isfinite(y[torch.arange(len(y)) % 20 != 7]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 200])
def test_gemm_writes_its_rows_alone(zq, T):
    K, N = 512, 264
    xq, sx = quantized(zq, torch.randn(T, K, generator=gen(1)), 1, 0)
    wq, sw = quantized(zq, torch.randn(N, K, generator=gen(2)), 128, 0)
    buf = torch.full((T + 40, N), 7.0, dtype=torch.float16, device="cuda")
    zq.gemm_fp8(xq, sx, wq, sw, Y=buf[20:20 + T])
    assert torch.all(buf[:20] == 7) and torch.all(buf[20 + T:] == 7)
    assert torch.equal(buf[20:20 + T], zq.gemm_fp8(xq, sx, wq, sw))


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(3, 2048, 1024), (300, 1024, 768)])
def test_streams_graphs_and_overlap(zq, T, K, N):
    """No workspace: calls on two streams, and two captured graphs replayed
    with other inputs, give what a call alone gives."""
    g = gen(T)
    ws = [quantized(zq, torch.randn(N, K, generator=g), 128, 0) for _ in range(2)]
    xs = [torch.randn(T, K, generator=g).half().cuda() for _ in range(4)]

    def layer(x, w):
        q, s = zq.ln_quant_fp8(x, gamma)
        return zq.gemm_fp8(q, s, *w)

    gamma = torch.ones(K, dtype=torch.float16, device="cuda")
    want = [[layer(x, w) for w in ws] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for i in range(20):
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[j].append(layer(xs[i % 4], ws[j]))
    torch.cuda.synchronize()
    for j in range(2):
        for i, y in enumerate(got[j]):
            assert torch.equal(y, want[i % 4][j])
    # `stream=` is the stream that runs the call
    side = torch.cuda.Stream()
    q, s = zq.ln_quant_fp8(xs[0], gamma)
    side.wait_stream(torch.cuda.current_stream())
    y = zq.gemm_fp8(q, s, *ws[0], stream=side)
    side.synchronize()
    assert torch.equal(y, want[0][0])
    bufs, graphs, outs = [x.clone() for x in xs[:2]], [], []
    for j in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(layer(bufs[j], ws[j]))
        graphs.append(gr)
    for i in range(4):
        for j in range(2):
            bufs[j].copy_(xs[(i + j) % 4])
        torch.cuda.synchronize()
        for j, st in enumerate(streams):  # both at once
            with torch.cuda.stream(st):
                graphs[j].replay()
        torch.cuda.synchronize()
        for j in range(2):
            assert torch.equal(outs[j], want[(i + j) % 4][j])


# ------------------------------------------------------------ norm and rotation

def rotate_ref(x, pos, f, layout, scale, norm, eps, w, b):
    """(result, bound on the fp32 error) in 64 bits."""
    D, R = x.shape[-1], 2 * f.numel()
    v = x.double()
    mag = v.abs()
    if norm == 2:
        mag = mag + v.abs().mean(-1, keepdim=True)
        v = v - v.mean(-1, keepdim=True)
    if norm:
        rstd = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
        wd = torch.ones(D, dtype=torch.float64) if w is None else w.double()
        bd = torch.zeros(D, dtype=torch.float64) if b is None else b.double()
        v, mag = v * rstd * wd + bd, mag * rstd * wd.abs() + bd.abs()
    ang = pos.double()[:, None] * f.double()
    c, s = (torch.cos(ang) * scale)[:, None], (torch.sin(ang) * scale)[:, None]
    y, m = v.clone(), mag.clone()
    i, j = (slice(0, R // 2), slice(R // 2, R)) if layout == 0 else (slice(0, R, 2), slice(1, R, 2))
    y[..., i], y[..., j] = v[..., i] * c - v[..., j] * s, v[..., j] * c + v[..., i] * s
    m[..., i] = m[..., j] = abs(scale) * (mag[..., i] + mag[..., j])
    return y, ((D + 8 if norm else 0) + 4 + 6) * U * m


def check_rope(zq, T, Hq, Hk, D, R, layout, norm, dtype, far=0, scale=1.0, in_place=False, fused=True,
               affine=True, seed=0):
    g = gen(seed + T + Hq * 3 + Hk * 5 + D * 7 + R)
    if fused:  # slices of a fused QKV output
        qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(dtype).cuda()
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    else:  # per head: q, k and v side by side
        qkv = torch.randn(T, max(Hq, Hk), 3, D, generator=g).to(dtype).cuda()
        q, k = qkv[:, :Hq, 0], qkv[:, :Hk, 1]
    before = qkv.clone()
    pos = torch.randint(0, far + 1, (T,), generator=g).int()
    f, _ = zq.rope_frequencies(R) if R >= 2 else (torch.empty(0), 1.0)
    par = {}
    if norm and affine:
        for n in ("q", "k"):
            par[n + "_weight"] = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda()
            par[n + "_bias"] = (0.2 * torch.randn(D, generator=g)).to(dtype).cuda()
    want = {n: rotate_ref(t.cpu(), pos, f, layout, scale, norm, 1e-6,
                          *(None if n + p not in par else par[n + p].cpu()
                            for p in ("_weight", "_bias"))) for n, t in (("q", q), ("k", k))}
    out = dict(q_out=q, k_out=k) if in_place else {}
    qo, ko = zq.qk_norm_rope(q, k, pos.cuda(), f.cuda(), layout, scale, norm, 1e-6, **par, **out)
    for n, t in (("q", qo), ("k", ko)):
        ref, err = want[n]
        tol = err + HALF_STEP[dtype] * (ref.abs() + err) + TINY[dtype]
        bad = (t.cpu().double() - ref).abs() > tol
        assert not bad.any(), f"{n}: {bad.sum()} values outside the tolerance"
    if in_place:
        assert qo.data_ptr() == q.data_ptr()
        rest = qkv[:, Hq + Hk:] if fused else qkv[:, :, 2]
        assert torch.equal(rest, before[:, Hq + Hk:] if fused else before[:, :, 2])
    else:
        assert torch.equal(qkv, before)


ROPE_SHAPES = [(1, 1, 1, 8, 8), (1, 64, 8, 128, 128), (5, 16, 16, 256, 64), (33, 12, 12, 96, 24),
               (40, 7, 1, 80, 20), (3, 4, 2, 64, 64), (17, 3, 3, 192, 96), (130, 8, 2, 128, 32),
               (9, 2, 2, 256, 252), (700, 5, 5, 40, 16), (4, 2, 2, 72, 44), (2, 3, 1, 248, 248)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("shape", ROPE_SHAPES)
def test_rope(zq, dtype, layout, norm, shape):
    check_rope(zq, *shape, layout, norm, dtype, far=4096)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("shape", ROPE_SHAPES[:8])
def test_rope_in_place_and_other_strides(zq, norm, shape):
    check_rope(zq, *shape, 0, norm, torch.float16, far=100, in_place=True, affine=False)
    check_rope(zq, *shape, 1, norm, torch.bfloat16, far=100, in_place=True, fused=False)
    check_rope(zq, *shape, 0, norm, torch.float16, far=100, fused=False, scale=1.2)


@pytest.mark.gpu
@pytest.mark.parametrize("R", [6, 14, 30])
def test_rope_neighbours_of_odd_width(zq, R):
    check_rope(zq, 11, 3, 2, 64, R, 1, 0, torch.float16, far=50)
    check_rope(zq, 11, 3, 2, 64, R, 1, 1, torch.float16, far=50, in_place=True)
    check_rope(zq, 11, 3, 2, 64, R, 1, 0, torch.float16, far=50, in_place=True)


@pytest.mark.gpu
def test_rope_norm_alone(zq):
    check_rope(zq, 11, 3, 2, 64, 0, 0, 1, torch.float16)
    check_rope(zq, 11, 3, 2, 64, 0, 1, 2, torch.bfloat16, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", [0, 1])
def test_rope_far_positions_are_exact(zq, layout):
    # an fp32 angle at 2^30 would be off by up to 64 radians
    check_rope(zq, 64, 2, 2, 64, 64, layout, 0, torch.float16, far=2 ** 31 - 2)
    check_rope(zq, 64, 2, 2, 128, 128, layout, 1, torch.bfloat16, far=2 ** 30)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_skips_negative_positions(zq, norm, in_place):
    T, H, D = 50, 6, 64
    x = torch.randn(T, H, D, generator=gen(1)).half().cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f, _ = zq.rope_frequencies(D)
    whole, _ = zq.qk_norm_rope(x, None, pos, f.cuda(), norm=norm)
    skip = torch.zeros(T, dtype=torch.bool, device="cuda")
    skip[[0, 7, 8, 9]] = True
    skip[31:] = True
    pos[skip] = -1
    before = x.clone()
    out = x if in_place else torch.full_like(x, 3.0)
    left = before if in_place else out.clone()
    got, none = zq.qk_norm_rope(x, None, pos, f.cuda(), norm=norm, q_out=out)
    assert none is None and got is out
    assert torch.equal(got[skip], left[skip]) and torch.equal(got[~skip], whole[~skip])
    if not in_place:
        assert torch.equal(x, before)


@pytest.mark.gpu
def test_rope_keeps_lengths_and_products(zq):
    """What a rotation is for: lengths stay, and the product of a query and a
    key depends on the distance of their positions alone."""
    D = 64
    q, k = torch.randn(1, 1, D, generator=gen(1)), torch.randn(1, 1, D, generator=gen(2))
    f, scale = zq.rope_frequencies(D)
    T = 40
    for layout in (0, 1):
        pos = torch.arange(T).int().cuda()
        qr, kr = zq.qk_norm_rope(q.repeat(T, 1, 1).half().cuda(), k.repeat(T, 1, 1).half().cuda(), pos,
                                 f.cuda(), layout, scale)
        qr, kr = qr[:, 0].double(), kr[:, 0].double()
        dots = qr @ kr.T
        # two roundings to fp16 per product of vectors
        tol = 3 * 2.0 ** -11 * float(qr.norm(dim=1).max() * kr.norm(dim=1).max())
        for d in (0, 1, 9):
            assert float(dots.diagonal(d).max() - dots.diagonal(d).min()) <= 2 * tol
        assert float((qr.norm(dim=1) - q.half().double().norm()).abs().max()) <= tol


@pytest.mark.gpu
def test_rope_head_major_output(zq):
    T, H, D = 9, 4, 64
    x = torch.randn(T, H, D, generator=gen(1)).half().cuda()
    pos = torch.arange(T).int().cuda()
    f = zq.rope_frequencies(32)[0].cuda()
    want, _ = zq.qk_norm_rope(x, None, pos, f)
    out = torch.empty(H, T, D, dtype=torch.float16, device="cuda").transpose(0, 1)
    zq.qk_norm_rope(x, None, pos, f, q_out=out)
    assert torch.equal(out, want)


# ------------------------------------------------------------ a run of them together

@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 150])
def test_layer_together(zq, T):
    """LayerNorm, QKV projection, norm and rotation, output projection, LayerNorm,
    FFN with GeLU: a transformer layer's linear parts with attention left to the
    caller, against the same in 64 bits.  Its error is that of the e4m3 codes:
    each of the four products has codes off by at most half a step (2^-4
    relative) on either side, independent of one another."""
    h, H, D, R, ffn = 512, 8, 64, 16, 2048
    g = gen(T)
    mk = lambda *s: torch.randn(*s, generator=g) * 0.05  # noqa: E731
    W = {"qkv": mk(3 * h, h), "out": mk(h, h), "up": mk(ffn, h), "down": mk(h, ffn)}
    Q = {n: zq.quantize_weights_fp8(w.half().cuda()) for n, w in W.items()}
    bias = {n: (torch.randn(w.shape[0], generator=g) * 0.1).half() for n, w in W.items()}
    gamma, beta = (1 + 0.1 * torch.randn(h, generator=g)).half(), (0.1 * torch.randn(h, generator=g)).half()
    x = torch.randn(T, h, generator=g).half()
    pos = torch.arange(100, 100 + T).int()
    f, scale = zq.rope_frequencies(R)
    cu = lambda t: t.cuda()  # noqa: E731

    def linear(q, s, n):
        return zq.gemm_fp8(q, s, *Q[n], cu(bias[n]))

    qkv = linear(*zq.ln_quant_fp8(cu(x), cu(gamma), cu(beta)), "qkv").view(T, 3, H, D)
    q, k = zq.qk_norm_rope(qkv[:, 0], qkv[:, 1], cu(pos), f.cuda(), zq.ROPE_INTERLEAVED, scale,
                           zq.NORM_RMS, q_out=qkv[:, 0], k_out=qkv[:, 1])
    mixed = (q + k + qkv[:, 2]).reshape(T, h).contiguous()  # in attention's place
    a = linear(*zq.bias_act_quant_fp8(mixed), "out") + cu(x)
    up = linear(*zq.ln_quant_fp8(a, cu(gamma), cu(beta)), "up")
    y = linear(*zq.bias_act_quant_fp8(up, None, zq.ACT_GELU), "down") + a

    d = lambda t: t.double()  # noqa: E731
    def ln(v):
        return torch.nn.functional.layer_norm(v, (h,), d(gamma), d(beta), 1e-5)
    def lin(v, n):
        return v @ d(W[n].half()).T + d(bias[n])
    rq = lin(ln(d(x)), "qkv").view(T, 3, H, D)
    rot = [rotate_ref(rq[:, i], pos, f, 1, scale, 1, 1e-6, None, None)[0] for i in (0, 1)]
    ra = lin((rot[0] + rot[1] + rq[:, 2]).reshape(T, h), "out") + d(x)
    rup = lin(ln(ra), "up")
    ry = lin(gelu(rup), "down") + ra
    # each product: both operands rounded by at most 2^-4 of a value, so a
    # relative error (2-norm) below 2 * 2^-4; four in a row, of which the
    # normed and residual parts only lower it
    rel = float((y.cpu().double() - ry).norm() / ry.norm())
    assert rel <= 4 * 2 * 2.0 ** -4, rel
    assert rel > 0


@pytest.mark.gpu
@pytest.mark.parametrize("K", [16, 272, 1024, 1040, 2048, 5120, 6160, 12288, 16400, 24576, 24592, 32768])
def test_layernorm_rows_do_not_depend_on_their_number(zq, K):
    """More rows than run at once, and each row's bits as in a call of its own
    few."""
    T = 148 * 24 * 4 // (1 if K <= 1024 else 4 * -(-K // 1024)) * 2 + 5
    x = torch.randn(T, K, generator=gen(K)).half().cuda()
    gamma = (1 + 0.1 * torch.randn(K, generator=gen(K + 1))).half().cuda()
    y = torch.empty_like(x)
    q, s = zq.ln_quant_fp8(x, gamma, gamma, y_ln=y)
    for a, b in ((0, 1), (1, 40), (T // 2, T // 2 + 9), (T - 7, T)):
        yc = torch.empty_like(x[a:b])
        qc, sc = zq.ln_quant_fp8(x[a:b], gamma, gamma, y_ln=yc)
        assert torch.equal(q[a:b].view(torch.uint8), qc.view(torch.uint8))
        assert torch.equal(s[a:b], sc) and torch.equal(y[a:b], yc)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [0, 1, 2])
@pytest.mark.parametrize("T,Hq,Hk,D,R,layout", [(6001, 2, 1, 64, 64, 0), (2011, 32, 8, 128, 128, 0),
                                                (700, 64, 64, 96, 24, 0), (3000, 16, 4, 256, 64, 1)])
def test_rope_tokens_do_not_depend_on_their_number(zq, norm, T, Hq, Hk, D, R, layout):
    g = gen(T)
    q, k = torch.randn(T, Hq, D, generator=g).half().cuda(), torch.randn(T, Hk, D, generator=g).half().cuda()
    pos = torch.randint(0, 100000, (T,), generator=g).int().cuda()
    f = zq.rope_frequencies(R)[0].cuda()
    qo, ko = zq.qk_norm_rope(q, k, pos, f, layout, norm=norm)
    for a, b in ((0, 1), (1, 30), (T // 2, T // 2 + 5), (T - 3, T)):
        qc, kc = zq.qk_norm_rope(q[a:b], k[a:b], pos[a:b], f, layout, norm=norm)
        assert torch.equal(qo[a:b], qc) and torch.equal(ko[a:b], kc)


@pytest.mark.gpu
def test_kernels_with_tensor_memory_side_by_side(zq):
    """FP8 GEMMs of few tokens (clusters along K), of some (clusters of tiles)
    and of many (CTA pairs), and the INT8 GEMM's pairs, on four streams at
    once: each gives what it gives alone."""
    g = gen(3)
    jobs = []
    for T, K, N in ((8, 4096, 1024), (200, 4096, 512), (2048, 2048, 2048)):
        x = quantized(zq, torch.randn(T, K, generator=g), 1, 0)
        w = quantized(zq, torch.randn(N, K, generator=g), 128, 0)
        jobs.append(lambda x=x, w=w: zq.gemm_fp8(*x, *w))
    X = torch.randn(2048, 2048, generator=g).half().cuda()
    Wq, sg = zq.quantize_weights_groupwise(torch.randn(2048, 2048, generator=g).half().cuda(), 16, 8)
    Xq, st = zq.ln_quant(X)
    Y8 = torch.empty(2048, 2048, dtype=torch.float16, device="cuda")
    jobs.append(lambda: zq.gemm_w8a8(Xq, st, Wq, sg, Y=Y8))
    want = [job().clone() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(30):
        for job, s, out in zip(jobs, streams, got):
            with torch.cuda.stream(s):
                out.append(job())
    torch.cuda.synchronize()
    for w, out in zip(want, got):
        assert all(torch.equal(w, y) for y in out)


@pytest.mark.gpu
def test_calls_from_several_threads(zq):
    """Host threads call at once, each on a stream of its own: each gets what a
    single thread gets."""
    g = gen(9)
    w = quantized(zq, torch.randn(768, 1024, generator=g), 128, 0)
    gamma = torch.ones(1024, dtype=torch.float16, device="cuda")
    pos, f = torch.arange(700, dtype=torch.int32, device="cuda"), zq.rope_frequencies(32)[0].cuda()
    xs = [torch.randn(T, 1024, generator=g).half().cuda() for T in (1, 30, 100, 700)]

    def layer(x):
        T = x.shape[0]
        y = zq.gemm_fp8(*zq.ln_quant_fp8(x, gamma), *w).view(T, 12, 64)
        q, k = zq.qk_norm_rope(y[:, :8], y[:, 8:], pos[:T], f, norm=zq.NORM_RMS)
        return y, q, k, *zq.bias_act_quant_fp8(x, None, zq.ACT_GELU)

    want = [layer(x) for x in xs]
    torch.cuda.synchronize()
    wrong, streams = [], [torch.cuda.Stream() for _ in xs]

    def work(i):
        with torch.cuda.stream(streams[i]):
            got = [layer(xs[(i + n) % 4]) for n in range(24)]
        streams[i].synchronize()
        for n, out in enumerate(got):
            if not all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                       for a, b in zip(out, want[(i + n) % 4])):
                wrong.append((i, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


_FIRST_CALLS_IN_A_CAPTURE = r"""
import sys, torch
sys.path.insert(0, {root!r})
from int4_quantized_transformer_b200 import zq
g = torch.Generator().manual_seed(1)
K, N = 2048, 1024
W = torch.randn(N, K, generator=g).half().cuda()
xs = [torch.randn(T, K, generator=g).half().cuda() for T in (1, 40, 200, 1500)]
gamma = torch.ones(K, dtype=torch.float16, device="cuda")
pos = torch.arange(1500, dtype=torch.int32, device="cuda")
f = zq.rope_frequencies(64)[0].cuda()
# the library's own CUDA runtime starts up at its first call: make that call
# (a status query) outside any capture
assert zq.device_status()[0] == zq.ZQ_OK

def run():
    w = zq.quantize_weights_fp8(W)
    out = []
    for x in xs:
        T = x.shape[0]
        y = zq.gemm_fp8(*zq.ln_quant_fp8(x, gamma), *w)
        out += [y, zq.gemm_fp8(*zq.bias_act_quant_fp8(x, None, zq.ACT_GELU), *w)]
        out += zq.qk_norm_rope(y.view(T, 16, 64)[:, :12], y.view(T, 16, 64)[:, 12:], pos[:T], f,
                               norm=zq.NORM_RMS)
        out += zq.qk_norm_rope(y.view(T, 16, 64)[:, :12], y.view(T, 16, 64)[:, 12:], pos[:T], f)
    return out

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, run()):
    assert torch.equal(a, b)
assert zq.device_status()[0] == zq.ZQ_OK
print("ok")
"""


@pytest.mark.gpu
def test_first_calls_in_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", _FIRST_CALLS_IN_A_CAPTURE.format(root=root)],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-3000:]
    assert out.stdout.split()[-1] == "ok"


# ------------------------------------------------------------ frequencies (host)

def freq(R, base):
    return base ** (-np.arange(0, R, 2) / R)


@pytest.mark.parametrize("R,base", [(2, 10000.0), (24, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1e6)])
def test_frequencies(zq, R, base):
    f, s = zq.rope_frequencies(R, base)
    assert s == 1.0 and np.allclose(f.numpy(), freq(R, base), rtol=2 * U, atol=0)
    f, s = zq.rope_frequencies(R, base, zq.ROPE_LINEAR, 4.0)
    assert s == 1.0 and np.allclose(f.numpy(), freq(R, base) / 4, rtol=2 * U, atol=0)
    if R > 2:
        f, s = zq.rope_frequencies(R, base, zq.ROPE_NTK, 4.0)
        assert s == 1.0 and np.allclose(f.numpy(), freq(R, base * 4 ** (R / (R - 2))), rtol=2 * U, atol=0)
        # the highest frequency is kept, the lowest divided by the factor
        assert f[0] == 1 and abs(f[-1].item() * 4 / freq(R, base)[-1] - 1) < 4 * U


def test_frequencies_by_bands(zq):
    R, base, n, lo, hi, factor = 128, 500000.0, 8192, 1.0, 4.0, 8.0
    f, s = zq.rope_frequencies(R, base, zq.ROPE_BANDS, factor, lo, hi, n)
    plain = freq(R, base)
    turns = n * plain / (2 * math.pi)
    assert s == 1.0
    want = []
    for p, t in zip(plain, turns):
        if t > hi:
            want.append(p)
        elif t < lo:
            want.append(p / factor)
        else:
            sm = (t - lo) / (hi - lo)
            want.append((1 - sm) * p / factor + sm * p)
    assert (turns > hi).any() and (turns < lo).any() and ((turns < hi) & (turns > lo)).any()
    assert np.allclose(f.numpy(), want, rtol=4 * U, atol=0)


def test_frequencies_yarn(zq):
    R, base, n, lo, hi, factor = 128, 10000.0, 4096, 1.0, 32.0, 16.0
    f, s = zq.rope_frequencies(R, base, zq.ROPE_YARN, factor, lo, hi, n)
    assert abs(s - (0.1 * math.log(factor) + 1)) < 1e-6
    dim = lambda t: R * math.log(n / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    a, b = max(math.floor(dim(hi)), 0), min(math.ceil(dim(lo)), R - 1)
    plain = freq(R, base)
    ramp = np.clip((np.arange(R // 2) - a) / (b - a), 0, 1)
    assert 0 < a < b < R // 2
    assert np.allclose(f.numpy(), plain * (1 - ramp) + plain / factor * ramp, rtol=4 * U, atol=0)
    assert np.allclose(zq.rope_frequencies(R, base, zq.ROPE_YARN, 1.0, lo, hi, n)[0], plain, rtol=4 * U)


@pytest.mark.parametrize("args,expect", [
    ((0,), "SHAPE"), ((3,), "SHAPE"), ((258,), "SHAPE"), ((64, 1.0), "SHAPE"),
    ((64, float("nan")), "SHAPE"), ((64, 1e4, 9), "UNSUPPORTED"), ((64, 1e4, 1, 0.5), "SHAPE"),
    ((2, 1e4, 2, 2.0), "SHAPE"), ((64, 1e4, 3, 2.0, 0.0, 4.0, 10), "SHAPE"),
    ((64, 1e4, 3, 2.0, 4.0, 4.0, 10), "SHAPE"), ((64, 1e4, 4, 2.0, 1.0, 4.0, 0), "SHAPE")])
def test_frequencies_refuse(zq, args, expect):
    with pytest.raises(zq.ZQError) as e:
        zq.rope_frequencies(*args)
    assert e.value.status == getattr(zq, "ZQ_ERR_" + expect)


# ------------------------------------------------------------ refusals (no GPU: nothing is launched)

FAKE = 1 << 40  # an aligned address that is never dereferenced


@pytest.mark.parametrize("args,expect", [
    # (W, dtype, N, K, Wq, s_blk)
    ((FAKE, 2, 256, 64, FAKE, FAKE), "UNSUPPORTED"), ((FAKE, 0, 0, 64, FAKE, FAKE), "SHAPE"),
    ((FAKE, 0, 256, 40, FAKE, FAKE), "SHAPE"), ((FAKE, 0, 256, 0, FAKE, FAKE), "SHAPE"),
    ((FAKE, 0, 2 ** 31 - 1, 2 ** 31 - 16, FAKE, FAKE), "SHAPE"),
    ((None, 0, 256, 64, FAKE, FAKE), "NULL"), ((FAKE, 0, 256, 64, FAKE, None), "NULL"),
    ((FAKE + 2, 0, 256, 64, FAKE, FAKE), "ALIGN"), ((FAKE, 1, 256, 64, FAKE + 8, FAKE), "ALIGN"),
    ((FAKE, 1, 256, 64, FAKE, FAKE + 2), "ALIGN")])
def test_weights_refuse(zq, args, expect):
    assert zq.lib().zq_quantize_weights_fp8(*args, None) == getattr(zq, "ZQ_ERR_" + expect)


@pytest.mark.parametrize("args,expect", [
    # (X, dtype, gamma, beta, T, K, eps, Xq, s_blk, Y)
    ((FAKE, 3, FAKE, None, 4, 64, 1e-5, FAKE, FAKE, None), "UNSUPPORTED"),
    ((FAKE, 0, FAKE, None, -1, 64, 1e-5, FAKE, FAKE, None), "SHAPE"),
    ((FAKE, 0, FAKE, None, 4, 40, 1e-5, FAKE, FAKE, None), "SHAPE"),
    ((FAKE, 0, FAKE, None, 4, 32784, 1e-5, FAKE, FAKE, None), "SHAPE"),
    ((FAKE, 0, None, None, 4, 0, 1e-5, FAKE, FAKE, None), "SHAPE"),
    ((None, 0, FAKE, None, 4, 64, 1e-5, FAKE, FAKE, None), "NULL"),
    ((FAKE, 0, None, None, 4, 64, 1e-5, None, FAKE, None), "NULL"),
    ((FAKE, 0, FAKE + 4, None, 4, 64, 1e-5, FAKE, FAKE, None), "ALIGN"),
    ((FAKE, 0, FAKE, FAKE + 4, 4, 64, 1e-5, FAKE, FAKE, None), "ALIGN"),
    ((FAKE, 0, FAKE, None, 4, 64, 1e-5, FAKE, FAKE + 1, None), "ALIGN"),
    ((FAKE, 0, FAKE, None, 4, 64, 1e-5, FAKE, FAKE, FAKE + 2), "ALIGN")])
def test_layernorm_refuses(zq, args, expect):
    assert zq.lib().zq_ln_quant_fp8(*args, None) == getattr(zq, "ZQ_ERR_" + expect)


@pytest.mark.parametrize("args,expect", [
    # (X, dtype, bias, T, K, act, Xq, s_blk, Y)
    ((FAKE, 0, None, 4, 64, 2, FAKE, FAKE, None), "UNSUPPORTED"),
    ((FAKE, -1, None, 4, 64, 0, FAKE, FAKE, None), "UNSUPPORTED"),
    ((FAKE, 0, None, 4, 72, 0, FAKE, FAKE, None), "SHAPE"),
    ((FAKE, 0, None, 4, 64, 0, FAKE, None, None), "NULL"),
    ((FAKE, 0, FAKE + 8, 4, 64, 1, FAKE, FAKE, None), "ALIGN")])
def test_bias_act_refuses(zq, args, expect):
    assert zq.lib().zq_bias_act_quant_fp8(*args, None) == getattr(zq, "ZQ_ERR_" + expect)


GEMM_OK = dict(Xq=FAKE, sx=FAKE, Wq=FAKE, sw=FAKE, bias=None, T=16, N=256, K=64, dtype=0, Y=FAKE)


@pytest.mark.parametrize("change,expect", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(T=-1), "SHAPE"), (dict(N=250), "SHAPE"), (dict(N=0), "SHAPE"),
    (dict(K=72), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=2 ** 20 + 16), "SHAPE"), (dict(Xq=None), "NULL"),
    (dict(sx=None), "NULL"), (dict(Wq=None), "NULL"), (dict(sw=None), "NULL"), (dict(Y=None), "NULL"),
    (dict(Xq=FAKE + 8), "ALIGN"), (dict(Wq=FAKE + 4), "ALIGN"), (dict(Y=FAKE + 2), "ALIGN"),
    (dict(bias=FAKE + 2), "ALIGN"), (dict(sx=FAKE + 2), "ALIGN"), (dict(sw=FAKE + 1), "ALIGN")])
def test_gemm_refuses(zq, change, expect):
    rc = zq.lib().zq_gemm_fp8(*{**GEMM_OK, **change}.values(), None)
    assert rc == getattr(zq, "ZQ_ERR_" + expect)


@pytest.mark.parametrize("opts,T", [(dict(path=3), 16), (dict(path=4), 16), (dict(path=2), 65),
                                    (dict(split_k=9), 16), (dict(split_k=2), 16), (dict(bn=192), 100)])
def test_gemm_refuses_options(zq, opts, T):
    # (K = 64 is one block: it cannot be split)
    with zq.options(**opts):
        rc = zq.lib().zq_gemm_fp8(*{**GEMM_OK, "T": T}.values(), None)
    assert rc == zq.ZQ_ERR_UNSUPPORTED


def rope_call(zq, q=None, k=None, dtype=0, T=4, D=64, norm=0, pos=FAKE, f=FAKE, R=64, layout=0):
    base = dict(i=FAKE, o=FAKE + (1 << 30), w=0, b=0, it=512, ih=64, ot=512, oh=64, n=8)
    mk = lambda c: None if c is None else zq._pack_heads(*{**base, **c}.values())  # noqa: E731
    return zq.lib().zq_qk_norm_rope(mk({} if q is None else q), mk(k), dtype, T, D, norm, 1e-6, pos, f,
                                    R, layout, 1.0, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(norm=3), "UNSUPPORTED"), (dict(layout=2), "UNSUPPORTED"),
    (dict(T=-1), "SHAPE"), (dict(D=60), "SHAPE"), (dict(D=264), "SHAPE"), (dict(D=0, R=0), "SHAPE"),
    (dict(R=65), "SHAPE"), (dict(R=66), "SHAPE"), (dict(R=-2), "SHAPE"), (dict(R=6), "SHAPE"),
    (dict(pos=None), "NULL"), (dict(f=None), "NULL"), (dict(pos=FAKE + 2), "ALIGN"),
    (dict(f=FAKE + 2), "ALIGN"), (dict(q=dict(n=-1)), "SHAPE"), (dict(q=dict(i=0)), "NULL"),
    (dict(q=dict(o=0)), "NULL"), (dict(k=dict(i=0)), "NULL"), (dict(q=dict(it=511)), "ALIGN"),
    (dict(q=dict(ih=-64)), "ALIGN"), (dict(q=dict(i=FAKE + 8)), "ALIGN"),
    (dict(q=dict(w=FAKE + 8), norm=1), "ALIGN"), (dict(k=dict(b=FAKE + 8), norm=1), "ALIGN"),
    (dict(q=dict(oh=56)), "SHAPE"),            # heads overlap
    (dict(q=dict(ot=0)), "SHAPE"),             # tokens overlap
    (dict(q=dict(ot=128, oh=64)), "SHAPE"),    # token 1 starts in head 2 of token 0
    (dict(k=dict(o=FAKE, ot=1024)), "SHAPE")])  # in place with other strides
def test_rope_refuses(zq, kw, expect):
    assert rope_call(zq, **kw) == getattr(zq, "ZQ_ERR_" + expect)


def test_nothing_to_do_is_fine(zq):
    L = zq.lib()
    assert L.zq_ln_quant_fp8(None, 0, None, None, 0, 64, 1e-5, None, None, None, None) == zq.ZQ_OK
    assert L.zq_bias_act_quant_fp8(None, 1, None, 0, 64, 1, None, None, None, None) == zq.ZQ_OK
    assert L.zq_gemm_fp8(None, None, None, None, None, 0, 256, 64, 0, None, None) == zq.ZQ_OK
    assert rope_call(zq, T=0, pos=None, f=None) == zq.ZQ_OK
    assert rope_call(zq, q=dict(n=0)) == zq.ZQ_OK
    # in place, no norm, nothing rotated: nothing changes
    assert rope_call(zq, q=dict(o=FAKE), R=0, f=None) == zq.ZQ_OK


def test_binding_refuses(zq):
    x = torch.zeros(4, 64, dtype=torch.float16)
    for call in (lambda: zq.ln_quant_fp8(x), lambda: zq.bias_act_quant_fp8(x),
                 lambda: zq.quantize_weights_fp8(x), lambda: zq.gemm_fp8(x, x, x, x),
                 lambda: zq.qk_norm_rope(x[:, None], None, x, x), lambda: zq.gemm_fp8(None, x, x, x),
                 lambda: zq.gemm_fp8(x, x, x, x, out_dtype=torch.float32)):
        with pytest.raises(TypeError):
            call()



def test_binding_refuses_another_device(zq):
    t = mock.MagicMock(spec=torch.Tensor)
    t.dtype, t.shape, t.device, t.is_cuda = torch.float16, torch.Size((4, 64)), "cuda:1", True
    t.is_contiguous.return_value, t.get_device.return_value = True, 1
    assert zq._ptr(t, torch.float16, (4, 64), "X", 1) is t.data_ptr.return_value
    with pytest.raises(ValueError, match="current device cuda:0"):
        zq._ptr(t, torch.float16, (4, 64), "X", 0)


def test_binding_refuses_sizes_past_an_int(zq):
    def huge(dtype, *shape):
        t = mock.MagicMock(spec=torch.Tensor)
        t.dtype, t.shape, t.is_cuda = dtype, torch.Size(shape), True
        t.dim.return_value = len(shape)
        return t

    n, f = 2**32 + 3, torch.zeros(4)
    x, w = huge(torch.float16, n, 64), huge(F8, 128, 64)
    for call in (lambda: zq.ln_quant_fp8(x), lambda: zq.bias_act_quant_fp8(x),
                 lambda: zq.quantize_weights_fp8(x), lambda: zq.gemm_fp8(huge(F8, n, 64), f, w, f),
                 lambda: zq.gemm_fp8(w, f, huge(F8, n, 64), f),
                 lambda: zq.qk_norm_rope(huge(torch.float16, n, 1, 64), None, f, f)):
        with pytest.raises(ValueError, match="too large"):
            call()


@pytest.mark.gpu
def test_binding_refuses_shapes_and_dtypes(zq):
    c = lambda *s, d=torch.float16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    x = c(4, 256)
    xq, sx = zq.bias_act_quant_fp8(x)
    wq, sw = zq.quantize_weights_fp8(c(128, 256))
    for call in (
            lambda: zq.bias_act_quant_fp8(c(4, 512)[:, ::2]),
            lambda: zq.bias_act_quant_fp8(x, c(128)),
            lambda: zq.bias_act_quant_fp8(c(4)),
            lambda: zq.ln_quant_fp8(x, c(256), c(255)),
            lambda: zq.ln_quant_fp8(x, c(256), s_blk=c(4, 3, d=torch.float32)),
            lambda: zq.gemm_fp8(xq, c(4, 3, d=torch.float32), wq, sw),
            lambda: zq.gemm_fp8(xq, sx, wq, sw[:, :1]),
            lambda: zq.gemm_fp8(xq, sx, wq, sw, c(127)),
            lambda: zq.gemm_fp8(xq, sx, wq, sw, Y=c(5, 128)),
            lambda: zq.qk_norm_rope(c(4, 2, 64), c(5, 2, 64), c(4, d=torch.int32), c(8, d=torch.float32)),
            lambda: zq.qk_norm_rope(c(4, 2, 64), None, c(5, d=torch.int32), c(8, d=torch.float32)),
            lambda: zq.qk_norm_rope(c(4, 2, 128)[..., ::2], None, c(4, d=torch.int32),
                                    c(8, d=torch.float32))):
        with pytest.raises(ValueError):
            call()
    for call in (
            lambda: zq.bias_act_quant_fp8(c(4, 256, d=torch.float32)),
            lambda: zq.ln_quant_fp8(x, c(256, d=torch.bfloat16)),
            lambda: zq.gemm_fp8(x, sx, wq, sw),
            lambda: zq.gemm_fp8(xq, sx.half(), wq, sw),
            lambda: zq.gemm_fp8(xq, sx, wq, sw, c(128, d=torch.bfloat16)),
            lambda: zq.qk_norm_rope(c(4, 2, 64), c(4, 2, 64, d=torch.bfloat16), c(4, d=torch.int32),
                                    c(8, d=torch.float32)),
            lambda: zq.qk_norm_rope(c(4, 2, 64), None, c(4, d=torch.int64), c(8, d=torch.float32)),
            lambda: zq.qk_norm_rope(c(4, 2, 64), None, None, c(8, d=torch.float32))):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_no_tokens_on_the_device(zq):
    x = torch.zeros(0, 256, dtype=torch.float16, device="cuda")
    xq, sx = zq.ln_quant_fp8(x, torch.ones(256, dtype=torch.float16, device="cuda"))
    wq, sw = zq.quantize_weights_fp8(torch.randn(128, 256, device="cuda").half())
    assert zq.gemm_fp8(xq, sx, wq, sw).shape == (0, 128)
    q, k = zq.qk_norm_rope(torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda"), None,
                           torch.zeros(0, dtype=torch.int32, device="cuda"),
                           torch.zeros(8, device="cuda"))
    assert q.shape == (0, 2, 64) and k is None
