"""Edges of the block-scaled FP8 linear layer and of the query/key norm with
rotation: ties between codes, values that are not finite, plans of the GEMM
that only some sizes or options take, outputs on another stream, and a layer
of the operators together with each stage left out in turn."""
import os
import subprocess
import sys
import unittest.mock as mock

import pytest
import torch

from test_fp8_rope import (DTYPES, F8, HALF_STEP, TINY, U, _device_status_clean, block_max, blocks,  # noqa: F401
                           check_gemm, e4m3_grid, gen, rope_call, rotate_ref, spread, zq)


# ------------------------------------------------------------ codes of 16-bit values, ties among them

def exact_codes(y, rows):
    """The e4m3 values nearest to y * 448 / a, halves to the even code, from
    16-bit values: |y| * 448 has at most 14 significant bits and the product of
    a 5-bit middle between two codes with a 16, so that both sides of every
    comparison are exact in 64 bits and nothing is divided."""
    y = y.double()
    amax = block_max(y, rows)
    a = spread(torch.where(amax > 0, amax.clamp_min(2.0 ** -110), amax), rows, *y.shape)
    num, grid = y.abs() * 448, e4m3_grid()
    hi = torch.searchsorted(grid, (num / torch.where(a > 0, a, torch.ones_like(a))).contiguous())
    hi = hi.clamp(1, 126)
    hi = torch.where((hi < 126) & (num > grid[hi] * a), hi + 1, hi)
    hi = torch.where((hi > 1) & (num <= grid[hi - 1] * a), hi - 1, hi)
    mid = (grid[hi - 1] + grid[hi]) / 2 * a
    code = torch.where((num > mid) | ((num == mid) & (hi % 2 == 0)), hi, hi - 1)
    return torch.where(a > 0, grid[code] * torch.sign(y), torch.zeros_like(y)), (num == mid) & (a > 0)


def tied(n, k, rows, dtype, seed):
    """A matrix whose every value is a tie (bar each block's largest): in a
    block with a = 7 j 2^e the middle m between two codes is met by
    y = m j 2^e / 64.  j odd, so that 448 / a = 64 / (j 2^e) has no short form."""
    g = gen(seed)
    js = torch.tensor([3, 5, 7] if dtype is torch.bfloat16 else [3, 5, 7, 9, 11, 13, 19, 21, 27, 45, 63])
    shape = (blocks(n) if rows > 1 else n, blocks(k))
    j = js[torch.randint(0, len(js), shape, generator=g)].double()
    e = torch.randint(-3, 4, shape, generator=g).double()
    unit = spread(j * 2.0 ** e, rows, n, k)
    grid = e4m3_grid()
    at = torch.randint(8, 126, (n, k), generator=g)  # codes of four significant bits: the middle has five
    y = (grid[at] + grid[at + 1]) / 2 * unit / 64
    y = torch.where(torch.rand(n, k, generator=g) < 0.5, y, -y)
    for r in range(shape[0]):
        for c in range(shape[1]):
            y[r * rows, c * 128] = 7 * j[r, c] * 2.0 ** e[r, c]
    return y


def test_tied_inputs_are_ties():
    for dtype in DTYPES:
        y = tied(256, 512, 128, dtype, 1)
        if dtype is torch.float16:  # small enough to be exact there too
            assert torch.equal(y.half().double()[y.abs() >= 2.0 ** -14], y[y.abs() >= 2.0 ** -14])
        t = y.to(dtype)
        want, tie = exact_codes(t, 128)
        assert tie.float().mean() > 0.9
        # one rounded factor 448 / a sends some of them to the other neighbour
        a = spread(block_max(t.double(), 128), 128, *t.shape).float()
        one = (t.float() * (448 / a)).to(F8).double()
        wrong = (one != want) & tie
        assert wrong.float().mean() > 0.001
        assert torch.all((one == want) | tie)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_even_code(zq, dtype):
    """Codes of weights and of rows as they are, bit for bit: blocks of ties,
    normal values, and blocks at both ends of the type's range."""
    y = torch.cat((tied(384, 1040, 128, dtype, 1), torch.randn(400, 1040, generator=gen(2)).double() * 0.02)).to(dtype)
    for got, rows in ((zq.quantize_weights_fp8(y.cuda()), 128), (zq.bias_act_quant_fp8(y.cuda()), 1),
                      (zq.ln_quant_fp8(y.cuda()), 1)):
        want, _ = exact_codes(y, rows)
        assert torch.equal(got[0].cpu().double(), want)
    rows = tied(300, 1040, 1, dtype, 3).to(dtype)
    far = torch.randn(64, 1040, generator=gen(4))
    far = torch.cat((far * 2.0 ** 125, far * 2.0 ** -108, far * 2.0 ** -130) if dtype is torch.bfloat16
                    else (far * 2.0 ** 13, far * 2.0 ** -16, far * 2.0 ** -22)).to(dtype)
    for x in (rows, far):
        q, s = zq.bias_act_quant_fp8(x.cuda())
        want, _ = exact_codes(x, 1)
        assert torch.equal(q.cpu().double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_the_same_codes_each_time(zq, dtype):
    x = torch.randn(600, 2064, generator=gen(5)).to(dtype).cuda()
    gamma = (1 + 0.1 * torch.randn(2064, generator=gen(6))).to(dtype).cuda()
    calls = (lambda: zq.quantize_weights_fp8(x), lambda: zq.bias_act_quant_fp8(x),
             lambda: zq.bias_act_quant_fp8(x, gamma, zq.ACT_GELU), lambda: zq.ln_quant_fp8(x, gamma, gamma))
    for call in calls:
        q, s = call()
        for _ in range(20):
            q2, s2 = call()
            assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


# ------------------------------------------------------------ values behind the rotated ones

def odd_rest(T, H, D, R, dtype, seed):
    """Heads whose values behind R hold infinities, NaN and zeros of either
    sign, next to finite ones, and the same heads with zeros there."""
    x = torch.randn(T, H, D, generator=gen(seed)).to(dtype)
    plain = x.clone()
    plain[..., R:] = 0
    odd = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0, -1.0, 1.0])
    at = torch.randint(0, len(odd), (T, H, D - R), generator=gen(seed + 1))
    x[..., R:] = torch.where(torch.rand(T, H, D - R, generator=gen(seed + 2)) < 0.7, odd[at],
                             x[..., R:].float()).to(dtype)
    x[:, 0, R], x[:, 0, R + 1] = 3.0, float("inf")  # the pair right behind R
    x[:, 1, R], x[:, 1, R + 1] = float("nan"), 2.0
    x[:, 2, R], x[:, 2, R + 1] = -0.0, -1.0
    return x.cuda(), plain.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,R", [(64, 4), (64, 12), (80, 20), (64, 6), (64, 30), (64, 62), (128, 64), (96, 24)])
def test_values_behind_the_rotation_are_copied(zq, dtype, layout, in_place, D, R):
    if layout == 0 and R % 4:
        pytest.skip("halves are rotated in multiples of four values")
    T, H = 19, 5
    x, plain = odd_rest(T, H, D, R, dtype, D + R)
    pos = torch.arange(3, 3 + T, dtype=torch.int32, device="cuda")
    f = zq.rope_frequencies(R)[0].cuda()
    want = zq.qk_norm_rope(plain, None, pos, f, layout)[0]
    before = x.clone()
    got = zq.qk_norm_rope(x, None, pos, f, layout, q_out=x if in_place else None)[0]
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(got[..., R:]), bits(before[..., R:]))
    assert torch.equal(bits(got[..., :R]), bits(want[..., :R]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("norm", [1, 2])
@pytest.mark.parametrize("D,R", [(64, 4), (64, 12), (80, 20), (64, 6), (64, 30), (64, 62), (128, 64)])
def test_values_behind_the_rotation_get_the_norm_alone(zq, dtype, layout, norm, D, R):
    """An infinite bias behind R (the head itself is finite) reaches its own
    value and no other: what the norm gives without any rotation."""
    if layout == 0 and R % 4:
        pytest.skip("halves are rotated in multiples of four values")
    T, H = 19, 5
    x = torch.randn(T, H, D, generator=gen(D + R)).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=gen(1))).to(dtype).cuda()
    b = torch.zeros(D, dtype=dtype, device="cuda")
    b[R + 1::2] = float("inf")
    w[R::4], b[R::4] = 0.0, -0.0
    pos = torch.arange(3, 3 + T, dtype=torch.int32, device="cuda")
    f = zq.rope_frequencies(R)[0].cuda()
    got = zq.qk_norm_rope(x, None, pos, f, layout, norm=norm, q_weight=w, q_bias=b)[0]
    v = x.double()
    v = v - (v.mean(-1, keepdim=True) if norm == 2 else 0)
    v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w.double() + b.double()
    rest, want = got[..., R:].double(), v[..., R:]
    assert torch.equal(torch.isinf(rest), torch.isinf(want)) and not torch.isnan(got).any()
    ok = torch.isfinite(want)
    # (D + 8) units of 2^-24 for the sums and two roundings, half a step of the
    # type; the mean is off by D units of the mean magnitude, which is at most
    # one standard deviation (and a little), times a weight below 2
    tol = ((D + 10) * 2.0 ** -24 + torch.finfo(dtype).eps / 2) * want[ok].abs() + 2 * (D + 10) * 2.0 ** -24
    assert torch.all((rest[ok] - want[ok]).abs() <= tol)
    zero = (w == 0)[R:].expand_as(rest)
    assert torch.all(rest[zero] == 0)
    assert torch.isfinite(got[..., :R]).all()


# ------------------------------------------------------------ GeLU at the ends of its range

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_gelu_of_values_that_are_not_finite(zq, dtype, with_bias):
    """GeLU(+Inf) is +Inf, and NaN stays NaN; -Inf times a probability of 0 is
    NaN, as in the definition taken literally.  The block that holds one of
    them has NaN codes, no other block does."""
    inf, big = float("inf"), torch.finfo(dtype).max
    x = torch.randn(5, 512, generator=gen(1)).to(dtype)
    x[0, 130], x[1, 131], x[2, 132], x[3, 133], x[3, 140] = inf, -inf, float("nan"), big, -big
    b = torch.zeros(512, dtype=dtype).cuda() if with_bias else None
    y = torch.empty_like(x.cuda())
    q, s = zq.bias_act_quant_fp8(x.cuda(), b, zq.ACT_GELU, y=y)
    y, q, s = y.cpu(), q.cpu().double(), s.cpu()
    assert y[0, 130] == inf and torch.isnan(y[1, 131]) and torch.isnan(y[2, 132])
    assert y[3, 133] == big and y[3, 140] == 0
    assert (~torch.isfinite(y)).sum() == 3
    for r in range(5):
        bad = torch.zeros(512, dtype=torch.bool)
        bad[128:256] = r < 3
        assert torch.equal(torch.isnan(q[r]), bad)
        assert torch.equal(torch.isfinite(s[r]), ~bad[::128])
    assert q[3, 133] == 448 and q[3, 140] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_gelu_of_every_value(zq, dtype):
    """Every finite value of the type, the far tail among them: 1e-6 for the
    approximation, 1.5 units of 2^-24 of v^2 for the exponent's roundings, a
    rounding of fp32 and half a step of the type.  A result below 7e-39 may be
    flushed to 0."""
    x = torch.arange(-2 ** 15, 2 ** 15).short().view(dtype)
    x = x[torch.isfinite(x)]
    x = torch.nn.functional.pad(x, (0, -len(x) % 128)).view(-1, 128)
    y = torch.empty_like(x.cuda())
    zq.bias_act_quant_fp8(x.cuda(), None, zq.ACT_GELU, y=y)
    v = x.double()
    want = 0.5 * v * torch.erfc(v * -(0.5 ** 0.5))
    tol = (1e-6 + U * (1 + 1.5 * v.square().clamp_max(400)) + HALF_STEP[dtype]) * want.abs() + TINY[dtype]
    tol += torch.where(want.abs() < 7e-39, want.abs(), torch.zeros_like(want))
    bad = (y.cpu().double() - want).abs() > tol
    assert not bad.any(), (x[bad][:5], y.cpu()[bad][:5])


# ------------------------------------------------------------ plans of the GEMM

_EVERY_PLAN = r"""
import itertools, sys
sys.path.insert(0, {root!r})
from int4_quantized_transformer_b200 import zq
L, A = zq.lib(), 1 << 40  # an aligned address that is never dereferenced: there is no device
for cap, split, bn, path, pair in itertools.product((0, 1, 2, 3, 7), (0, 1, 2, 3, 8), (0, 128, 256), (0, 1, 2),
                                                    (0, 1, 2)):
    with zq.options(max_ctas=cap, split_k=split, bn=bn, path=path, pair=pair):
        for T, N, K in ((1, 8, 16), (16, 48, 512), (64, 8, 4096), (16, 2**31 - 8, 1024), (65, 24576, 1024),
                        (300, 128, 24576), (2**31 - 1, 8, 16)):
            rc = L.zq_gemm_fp8(A, A, A, A, None, T, N, K, 0, A, None)
            assert rc in (zq.ZQ_ERR_UNSUPPORTED, zq.ZQ_ERR_CUDA), rc
print("ok")
"""


def test_gemm_plans_on_the_host():
    """Every plan is made without a division by zero (which would end the
    process, so a process of its own makes them, where no device is seen)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", _EVERY_PLAN.format(root=root)], capture_output=True, text=True,
                         timeout=300, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert out.returncode == 0 and out.stdout.split()[-1:] == ["ok"], (out.returncode, out.stderr[-2000:])


@pytest.mark.gpu
@pytest.mark.parametrize("max_ctas", [1, 2, 3])
@pytest.mark.parametrize("T,K,N", [(1, 1024, 8), (16, 2064, 48), (33, 1024, 48), (64, 4096, 136)])
def test_gemm_on_very_few_ctas(zq, max_ctas, T, K, N):
    check_gemm(zq, T, K, N, torch.float16, path=2, max_ctas=max_ctas)


# ------------------------------------------------------------ outputs on another stream

def output_calls(zq, T=300, K=1024, N=768):
    """Every call that makes its output: (bytes of an output, call with stream=)."""
    g = gen(1)
    x = torch.randn(T, K, generator=g).half().cuda()
    w = torch.randn(N, K, generator=g).half().cuda()
    b = torch.randn(K, generator=g).half().cuda()
    q8, s8 = zq.bias_act_quant_fp8(x)
    w8, sw = zq.quantize_weights_fp8(w)
    qi, si = zq.ln_quant(x)
    wi, sg = zq.quantize_weights_groupwise(w, 16, 8)
    w4, sg4 = zq.quantize_weights_groupwise(w, 16, 4)
    heads = torch.randn(T, 16, 64, generator=g).half().cuda()
    pos, f = torch.arange(T, dtype=torch.int32, device="cuda"), zq.rope_frequencies(64)[0].cuda()
    return {
        "quantize_weights_fp8": lambda s: zq.quantize_weights_fp8(w, stream=s),
        "ln_quant_fp8": lambda s: zq.ln_quant_fp8(x, b, b, stream=s),
        "bias_act_quant_fp8": lambda s: zq.bias_act_quant_fp8(x, b, zq.ACT_GELU, stream=s),
        "gemm_fp8": lambda s: zq.gemm_fp8(q8, s8, w8, sw, stream=s),
        "qk_norm_rope": lambda s: zq.qk_norm_rope(heads[:, :8], heads[:, 8:], pos, f, stream=s),
        "quantize_weights_groupwise": lambda s: zq.quantize_weights_groupwise(w, 16, 8, stream=s),
        "ln_quant": lambda s: zq.ln_quant(x, b, b, stream=s),
        "bias_act_quant": lambda s: zq.bias_act_quant(x, b, zq.ACT_GELU, stream=s),
        "static_quant": lambda s: zq.static_quant(x, 4.0, stream=s),
        "gemm_w8a8": lambda s: zq.gemm_w8a8(qi, si, wi, sg, stream=s),
        "gemm_w4a8": lambda s: zq.gemm_w4a8(qi, si, w4, sg4, stream=s),
        "gemm_w8a16": lambda s: zq.gemm_w8a16(x, wi, sg, stream=s),
        "widen_int4_weights": lambda s: zq.widen_int4_weights(w4, K, stream=s),
    }


CALLS = ["quantize_weights_fp8", "ln_quant_fp8", "bias_act_quant_fp8", "gemm_fp8", "qk_norm_rope",
         "quantize_weights_groupwise", "ln_quant", "bias_act_quant", "static_quant", "gemm_w8a8", "gemm_w4a8",
         "gemm_w8a16", "widen_int4_weights"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_outputs_are_memory_of_the_stream_that_writes_them(zq, name):
    """A block that the current stream has just let go of (and may still write)
    is not given to a call on another stream."""
    call = output_calls(zq)[name]
    tensors = lambda out: [t for t in (out if isinstance(out, tuple) else (out,))]  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = tensors(call(None))
    let_go = {t.data_ptr() for t in want}
    want = [t.cpu() for t in want]  # the device tensors go back to the current stream's memory
    again = tensors(call(None))
    assert {t.data_ptr() for t in again} & let_go  # which hands them out first
    again = None
    torch.cuda.synchronize()
    got = tensors(call(side))
    assert not {t.data_ptr() for t in got} & let_go
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


@pytest.mark.gpu
def test_a_side_stream_inside_a_capture(zq):
    calls = output_calls(zq)
    want = [calls[n](None) for n in CALLS[:5]]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = [calls[n](side) for n in CALLS[:5]]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    flat = lambda outs: [t for o in outs for t in (o if isinstance(o, tuple) else (o,))]  # noqa: E731
    for a, b in zip(flat(got), flat(want)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_stream_of_another_device_is_refused(zq):
    stream = mock.MagicMock()
    stream.device_index, stream.device, stream.cuda_stream = 1, "cuda:1", 0
    assert zq._raw(stream, 1) == 0
    with pytest.raises(ValueError, match="current device cuda:0"):
        zq._raw(stream, 0)
    with pytest.raises(ValueError, match="current device cuda:0"):
        zq._out((2, 2), (2, 1), torch.float16, 0, stream)


# ------------------------------------------------------------ plans of the GEMM that some sizes alone take

def check_gemm_on_device(zq, T, K, N, dtype, bias=True, seed=0, **opts):
    """As check_gemm, with the 64-bit reference on the device, for sizes that
    take long on the host.  The same tolerance."""
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + 3 * K + N)
    x = torch.randn(T, K, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    # scales that differ from block to block: a wrong block's scale shows
    sx = torch.exp(torch.randn(T, blocks(K), generator=g, device="cuda"))
    sw = torch.exp(torch.randn(blocks(N), blocks(K), generator=g, device="cuda"))
    xq, wq = (x * 20).clamp(-448, 448).to(F8), (w * 1000).clamp(-448, 448).to(F8)
    b = (torch.randn(N, generator=g, device="cuda") * 0.5).to(dtype) if bias else None
    sx *= 2.0 ** -12
    sw *= 2.0 ** -6
    with zq.options(**opts):
        y = zq.gemm_fp8(xq, sx, wq, sw, b, out_dtype=dtype)
        again = zq.gemm_fp8(xq, sx, wq, sw, b, out_dtype=dtype)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    X, W = xq.double() * spread(sx.double(), 1, T, K), wq.double() * spread(sw.double(), 128, N, K)
    ref, mag = X @ W.T, X.abs() @ W.abs().T
    if bias:
        ref, mag = ref + b.double(), mag + b.double().abs()
    u = 2.0 ** -24
    tol = (2 * 128 + 4 + blocks(K)) * u * mag
    half, tiny = (2.0 ** -11, 2.0 ** -25) if dtype is torch.float16 else (2.0 ** -8, 2.0 ** -134)
    tol = tol + half * (ref.abs() + tol) + tiny
    err = (y.double() - ref).abs()
    assert torch.all(err <= tol), f"worst {(err / tol).max().item():.2f} of the tolerance"
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("split", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("T,K,N,dtype", [(65, 1024, 136, torch.float16), (300, 2064, 520, torch.bfloat16),
                                         (129, 4096, 264, torch.float16), (257, 5008, 1032, torch.bfloat16)])
def test_gemm_tiles_shared_along_k(zq, split, T, K, N, dtype):
    """Every cluster size, also those that do not divide the 16 pieces of a
    warp's columns nor the blocks of K, with several rows of token tiles, cut
    off at the end of N and of T."""
    check_gemm_on_device(zq, T, K, N, dtype, bias=split % 2 == 0, path=1, split_k=split)


@pytest.mark.gpu
@pytest.mark.parametrize("split", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("T,K,N", [(1, 1024, 136), (20, 4112, 520), (64, 2064, 24)])
def test_gemm_weight_rows_shared_along_k(zq, split, T, K, N):
    check_gemm_on_device(zq, T, K, N, torch.float16 if split % 2 else torch.bfloat16, path=2, split_k=split)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(100, 2304, 768), (200, 4096, 2048), (200, 4096, 1536), (397, 5008, 2120),
                                   (160, 3584, 1280), (65, 12288, 640), (500, 1280, 896), (128, 2816, 2560)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gemm_plans_of_some_tokens(zq, T, K, N, dtype):
    check_gemm_on_device(zq, T, K, N, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("opts", [dict(bn=128, pair=1), dict(bn=256, pair=1), dict(bn=128, pair=2),
                                  dict(bn=256, pair=2), {}])
@pytest.mark.parametrize("T,K,N", [(1500, 4224, 6152), (3100, 8336, 2568)])
def test_gemm_tiles_with_several_groups_of_scales(zq, opts, T, K, N):
    """More than 32 blocks along K (two and three groups of scales per tile) and
    more tiles than CTAs, so that groups, bias and accumulator buffers go on
    from tile to tile."""
    opts = dict(path=1, **opts) if opts else {}
    for i, dtype in enumerate(DTYPES):
        check_gemm_on_device(zq, T, K, N, dtype, bias=i == 0, **opts)


@pytest.mark.gpu
@pytest.mark.parametrize("opts", [dict(bn=128, pair=1), dict(bn=256, pair=1), dict(bn=128, pair=2),
                                  dict(bn=256, pair=2)])
@pytest.mark.parametrize("T,K,N", [(1700, 65536, 520), (900, 180224, 264)])
def test_gemm_groups_of_token_tiles(zq, opts, T, K, N):
    """K so long that the token tiles run in groups (40 MB of activations
    each), the last of them shorter; and groups of a single tile."""
    check_gemm_on_device(zq, T, K, N, torch.bfloat16, path=1, **opts)


# ------------------------------------------------------------ a layer of the operators together

LAYER = dict(h=512, H=8, D=64, R=32, ffn=2048)
STAGES = ("qkv", "rotation", "out", "up", "down")


def layer_inputs(T, dtype):
    h, ffn, D = LAYER["h"], LAYER["ffn"], LAYER["D"]
    g = gen(T)
    r = lambda *s, by=1.0, add=0.0: (torch.randn(*s, generator=g) * by + add).to(dtype)  # noqa: E731
    W = {n: r(*s, by=0.05) for n, s in (("qkv", (3 * h, h)), ("out", (h, h)), ("up", (ffn, h)), ("down", (h, ffn)))}
    return dict(x=r(T, h), W=W, bias={n: r(w.shape[0], by=0.3) for n, w in W.items()},
                gamma=r(h, by=0.3, add=1.0), beta=r(h, by=0.3), qw=r(D, by=0.3, add=1.0), kw=r(D, by=0.3, add=1.0),
                pos=torch.arange(100, 100 + T).int())


def frequencies(zq):
    return zq.rope_frequencies(LAYER["R"], 10000.0, zq.ROPE_YARN, 8.0, 1.0, 32.0, 4096)


def codes_and_doubt(y, err):
    """Dequantized e4m3 values of rows whose values are known to within `err`,
    and by how much each may be off: its scale, and where the value lies next
    to the middle between two codes the step between them."""
    a = spread(block_max(y, 1), 1, *y.shape)
    ea = spread(block_max(err, 1), 1, *y.shape)  # of the block's largest value
    grid, v = e4m3_grid(), y.abs() * 448 / a
    hi = torch.searchsorted(grid, v.contiguous()).clamp(1, 126)
    mid, step = (grid[hi - 1] + grid[hi]) / 2, grid[hi] - grid[hi - 1]
    code = torch.where(v > mid, grid[hi], grid[hi - 1])  # (at a tie either: it is in doubt)
    slack = (err + y.abs() * (ea / a + 4 * U)) * 448 / a
    off = torch.where((v - mid).abs() <= slack, step, torch.zeros_like(step)) + code * (ea / a + 2 * U)
    return torch.sign(y) * code * a / 448, off * a / 448


def layer_stage(zq, p, stage, seen, without=""):
    """(result, bound on its error) of one stage in 64 bits, from what the
    stages before it gave (`seen`), so that a rounding that falls the other way
    there is not counted here.  `without` leaves a part out or puts a wrong one
    in its place.  Bounds: as in test_layernorm and test_bias_and_gelu for the
    values that are quantized, check_gemm's for the products, half a step of the
    16-bit type for each rounding to it."""
    D, R, dtype = LAYER["D"], LAYER["R"], p["x"].dtype
    half, tiny = HALF_STEP[dtype], TINY[dtype]

    def round16(v, e):
        return v, e + half * (v.abs() + e) + tiny

    def linear(y, err, n):
        X, dX = codes_and_doubt(y, err)
        W = exact_codes(p["W"][n], 128)[0] * spread(block_max(p["W"][n].double(), 128) / 448, 128, *p["W"][n].shape)
        b = torch.zeros(len(W), dtype=torch.float64) if without == "biases" else p["bias"][n].double()
        e = (dX + (2 * 128 + 8 + blocks(W.shape[1])) * U * (X.abs() + dX)) @ W.abs().T + 8 * U * b.abs()
        return round16(X @ W.T + b, e)

    def ln(v):
        gamma = 1.0 if without == "gamma" else p["gamma"].double()
        beta = 0.0 if without == "beta" else p["beta"].double()
        mean, rstd = v.mean(-1, keepdim=True), 1 / torch.sqrt(v.var(-1, correction=0, keepdim=True) + 1e-5)
        if without == "LayerNorm":
            mean, rstd = torch.zeros_like(mean), torch.ones_like(rstd)
        mag = (v.abs() + v.abs().mean(-1, keepdim=True)) * rstd * p["gamma"].double().abs() + p["beta"].double().abs()
        return (v - mean) * rstd * gamma + beta, 64 * U * mag

    def plus(ve, other):  # the residual, added to what was rounded
        return round16(ve[0] + other, ve[1])

    if stage == "qkv":
        return linear(*ln(p["x"].double()), "qkv")
    if stage == "rotation":
        f, scale = frequencies(zq)
        x = seen["qkv"].view(-1, 3, LAYER["H"], D)
        out, err = [], []
        for i, w in ((0, "qw"), (1, "kw")):
            pos = p["pos"] + (1 if without == "position" else 0)
            v, e = rotate_ref(x[:, i], pos, f * (0 if without == "rotation" else 1), 0 if without == "layout" else 1,
                              1.0 if without in ("scale", "rotation") else scale, 0 if without == "head norm" else 1,
                              1e-6, None if without == "head weight" else p[w], None)
            out.append(v), err.append(e)
        return round16(torch.cat(out, 1).flatten(1), torch.cat(err, 1).flatten(1))
    if stage == "out":
        y = seen["mixed"].double()
        return plus(linear(y, torch.zeros_like(y), "out"), p["x"].double())
    if stage == "up":
        return linear(*ln(seen["out"].double()), "up")
    v = seen["up"].double()
    y = 0.5 * v * torch.erfc(v * -(0.5 ** 0.5))
    err = (1e-6 + 1.5 * U * v.square()) * y.abs()
    if without in ("GeLU", "ReLU"):
        y = v if without == "GeLU" else v.clamp_min(0)
    res = plus(linear(y, err, "down"), seen["out"].double())
    return (res[0] - seen["out"].double(), res[1]) if without == "residual" else res


WITHOUT = {"biases": STAGES[:1] + STAGES[2:], "LayerNorm": ("qkv", "up"), "gamma": ("qkv", "up"), "beta": ("qkv", "up"),
           "head norm": STAGES[1:2], "head weight": STAGES[1:2], "rotation": STAGES[1:2], "layout": STAGES[1:2],
           "scale": STAGES[1:2], "position": STAGES[1:2], "GeLU": STAGES[4:], "ReLU": STAGES[4:],
           "residual": STAGES[4:]}


def layer_seen_by_definition(zq, p):
    seen = {}
    for stage in STAGES:
        if stage == "out":
            q, k = seen["rotation"].chunk(2, 1)
            seen["mixed"] = q + k + seen["qkv"].chunk(3, 1)[2]
        seen[stage] = layer_stage(zq, p, stage, seen)[0].to(p["x"].dtype)
    return seen


def outside(zq, p, stage, seen, without=""):
    """The share of a stage's values that lie outside their bound."""
    want, err = layer_stage(zq, p, stage, seen, without)
    return float(((seen[stage].double() - want).abs() > err).float().mean())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 7, 150])
def test_layer_bounds_tell_a_missing_part(zq, T, dtype):
    p = layer_inputs(T, dtype)
    seen = layer_seen_by_definition(zq, p)
    for stage in STAGES:
        assert outside(zq, p, stage, seen) == 0
    for part, stages in WITHOUT.items():
        for stage in stages:
            assert outside(zq, p, stage, seen, part) > 0.1, (part, stage)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 7, 150])
def test_layer_stage_by_stage(zq, T, dtype):
    """LayerNorm, QKV projection, norm and rotation of the heads (in place),
    output projection, LayerNorm, FFN with GeLU, run as a layer runs them:
    every value of every stage within its bound, and outside it for the stage
    with a part missing."""
    H, D = LAYER["H"], LAYER["D"]
    p = layer_inputs(T, dtype)
    Q = {n: zq.quantize_weights_fp8(w.cuda()) for n, w in p["W"].items()}
    linear = lambda q, s, n: zq.gemm_fp8(q, s, *Q[n], p["bias"][n].cuda(), out_dtype=dtype)  # noqa: E731
    f, scale = frequencies(zq)
    x, gamma, beta = p["x"].cuda(), p["gamma"].cuda(), p["beta"].cuda()
    qkv = linear(*zq.ln_quant_fp8(x, gamma, beta), "qkv")
    seen = {"qkv": qkv.clone()}
    heads = qkv.view(T, 3, H, D)
    q, k = zq.qk_norm_rope(heads[:, 0], heads[:, 1], p["pos"].cuda(), f.cuda(), zq.ROPE_INTERLEAVED, scale,
                           zq.NORM_RMS, q_weight=p["qw"].cuda(), k_weight=p["kw"].cuda(),
                           q_out=heads[:, 0], k_out=heads[:, 1])
    assert torch.equal(heads[:, 2], seen["qkv"].view(T, 3, H, D)[:, 2])
    seen["rotation"] = torch.cat((q, k), 1).flatten(1)
    seen["mixed"] = (q + k + heads[:, 2]).reshape(T, -1).contiguous()  # in attention's place
    seen["out"] = linear(*zq.bias_act_quant_fp8(seen["mixed"]), "out") + x
    seen["up"] = linear(*zq.ln_quant_fp8(seen["out"], gamma, beta), "up")
    seen["down"] = linear(*zq.bias_act_quant_fp8(seen["up"], None, zq.ACT_GELU), "down") + seen["out"]
    seen = {n: t.cpu() for n, t in seen.items()}
    for stage in STAGES:
        assert outside(zq, p, stage, seen) == 0, stage
    for part, stages in WITHOUT.items():
        for stage in stages:
            assert outside(zq, p, stage, seen, part) > 0.1, (part, stage)


# ------------------------------------------------------------ offsets past 32 bits, and heads that are not there

@pytest.mark.gpu
def test_quantizers_past_32_bits(zq):
    """More than 2^31 values: the last rows as in a call of their own."""
    T, K = 70016, 32768
    x = torch.randn(4096, K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    big = x.repeat(18, 1)[:T].contiguous()
    gamma = (1 + 0.1 * torch.randn(K, generator=gen(2))).half().cuda()
    assert T * K > 2 ** 31
    for call in (lambda v: zq.ln_quant_fp8(v, gamma, gamma), lambda v: zq.bias_act_quant_fp8(v, gamma, zq.ACT_GELU),
                 lambda v: zq.bias_act_quant_fp8(v)):
        q, s = call(big)
        for a, b in ((0, 3), (T // 2, T // 2 + 3), (T - 5, T)):
            qc, sc = call(big[a:b])
            assert torch.equal(q[a:b].view(torch.uint8), qc.view(torch.uint8)) and torch.equal(s[a:b], sc)
        del q, s
    q, s = zq.quantize_weights_fp8(big)
    for a in (0, 65536 - 128, T - 128):  # whole blocks of rows
        qc, sc = zq.quantize_weights_fp8(big[a:a + 128])
        assert torch.equal(q[a:a + 128].view(torch.uint8), qc.view(torch.uint8))
        assert torch.equal(s[a // 128:a // 128 + 1], sc)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(140000, 16, 16384), (70016, 32768, 16), (33, 32768, 70016), (3, 32768, 70016)])
def test_gemm_past_32_bits(zq, T, K, N):
    """More than 2^31 outputs, activations or weights: the last rows and columns
    against 64 bits (inputs of few values, so that every sum is exact)."""
    g = torch.Generator(device="cuda").manual_seed(T)
    mk = lambda r: torch.randint(-1, 2, (r, K), generator=g, device="cuda", dtype=torch.int8).to(F8)  # noqa: E731
    x, w = mk(T), mk(N)
    sx, sw = torch.ones(T, blocks(K), device="cuda"), torch.ones(blocks(N), blocks(K), device="cuda")
    assert max(T * K, N * K, T * N) > 2 ** 31
    y = zq.gemm_fp8(x, sx, w, sw)
    rows = torch.tensor(sorted({0, T // 2, T - 1} | {r for r in (T - 130, T - 129) if r >= 0}), device="cuda")
    cols = torch.tensor(sorted({0, N // 2, N - 1} | {c for c in (N - 130, N - 9) if c >= 0}), device="cuda")
    want = (x[rows].double() @ w.double().T if N * K < 2 ** 30 else None)
    if want is not None:
        assert torch.equal(y[rows].double(), want)
    want = x.double() @ w[cols].double().T if T * K < 2 ** 30 else x[rows].double() @ w[cols].double().T
    got = y[:, cols] if T * K < 2 ** 30 else y[rows][:, cols]
    assert want.abs().max() <= 2048  # exact in fp16
    assert torch.equal(got.double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [0, 1])
def test_rope_past_32_bits(zq, norm):
    T, H, D = 270000, 64, 128
    x = torch.randn(2000, H, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    x = x.repeat(135, 1, 1)
    assert T * H * D > 2 ** 31 and len(x) == T
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f = zq.rope_frequencies(D)[0].cuda()
    out = zq.qk_norm_rope(x[:, :40], x[:, 40:], pos, f, norm=norm)
    for a, b in ((0, 3), (T // 2, T // 2 + 3), (T - 5, T)):
        part = zq.qk_norm_rope(x[a:b, :40], x[a:b, 40:], pos[a:b], f, norm=norm)
        assert torch.equal(out[0][a:b], part[0]) and torch.equal(out[1][a:b], part[1])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("norm", [0, 1, 2])
def test_rope_without_queries_or_without_rotation(zq, layout, norm):
    x = torch.randn(21, 6, 72, generator=gen(1)).half().cuda()
    pos = torch.arange(21, dtype=torch.int32, device="cuda")
    f = zq.rope_frequencies(24)[0].cuda()
    want = zq.qk_norm_rope(x, None, pos, f, layout, norm=norm)[0]
    q, k = zq.qk_norm_rope(x[:, :0], x, pos, f, layout, norm=norm)
    assert q.shape == (21, 0, 72) and torch.equal(k, want)
    q, k = zq.qk_norm_rope(x, x[:, :0], pos, f, layout, norm=norm)
    assert k.shape == (21, 0, 72) and torch.equal(q, want)
    none = torch.empty(0, device="cuda")
    q, _ = zq.qk_norm_rope(x, None, pos, none, layout, norm=norm)
    if norm == 0:
        assert torch.equal(q, x)
    assert torch.equal(q[..., 24:], want[..., 24:])
    assert torch.equal(q[0], want[0])  # position 0


def test_rope_refuses_one_memory_for_queries_and_keys(zq):
    """Queries and keys written to the same place, or one of them over the
    other's input, while both are at work."""
    A, B, C = 1 << 40, 1 << 41, 1 << 42  # aligned addresses that are never dereferenced
    for q, k in ((dict(i=A, o=B), dict(i=C, o=B)), (dict(i=A, o=A), dict(i=C, o=A)),
                 (dict(i=A, o=C), dict(i=C, o=C)), (dict(i=A, o=B), dict(i=C, o=A)),
                 (dict(i=A, o=B), dict(i=A, o=A))):
        assert rope_call(zq, q=q, k=k) == zq.ZQ_ERR_SHAPE
    # no keys, no tokens: nothing to refuse
    assert rope_call(zq, q=dict(i=A, o=A), k=dict(i=A, o=A), T=0) == zq.ZQ_OK
    assert rope_call(zq, q=dict(n=0), k=dict(n=0)) == zq.ZQ_OK


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16, 40])
@pytest.mark.parametrize("N,K", [(5120, 5120), (2048, 12288), (8192, 4096), (1024, 24576), (4104, 8208), (24576, 1024),
                                 (20488, 272)])
def test_gemm_weight_rows_of_large_matrices(zq, T, N, K):
    """Two CTAs per SM, in clusters of one to eight."""
    check_gemm_on_device(zq, T, K, N, torch.bfloat16 if T == 16 else torch.float16)
