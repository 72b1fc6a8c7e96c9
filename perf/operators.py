"""The block-scaled FP8 linear layer and the query/key rotation, as a user calls them: cases, inputs, the plain form of
each operator, its definition in 64 bits, and the bytes and operations that it cannot do without.

Operators (the arithmetic is the one that include/zq.h states):

* ``gemm``    Y = sum over blocks of 128 k of s_x[t, kb] * s_w[nb, kb] * (x8 . w8) + bias, e4m3 codes
* ``act``     row quantization to e4m3 with one scale for each 128 values of a row, after a LayerNorm (``ln``), a
              bias-add and GeLU (``gelu``) or nothing (``plain``)
* ``weight``  weight quantization to e4m3 with one scale for each 128 x 128 block
* ``rope``    per-head norm of queries and keys and their rotation by position, in one pass
"""
import math

import torch

own = False  # False: plain torch operations; True: the framework's own entry points

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -110  # smaller non-zero block maxima are taken as this, so that 448 / amax stays finite
F8 = torch.float8_e4m3fn
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through the widest projection of a GPT-NeoX-sized layer: a decode step, bound by the weight stream
        {"name": "gemm_decode_1", "op": "gemm", "T": 1, "K": 6144, "N": 24576, "bias": True, "dtype": "fp16"},
        # a small batch of decoding sequences through a GPT-J-sized QKV projection
        {"name": "gemm_decode_24", "op": "gemm", "T": 24, "K": 4096, "N": 12288, "bias": False, "dtype": "bf16"},
        # a short ragged batch with odd sizes: blocks of 128 cut off at the end of K and of N
        {"name": "gemm_ragged", "op": "gemm", "T": 397, "K": 5008, "N": 2120, "bias": True, "dtype": "bf16"},
        # a prompt of 4096 tokens through the QKV projection of a GPT-NeoX-sized layer: bound by the tensor cores
        {"name": "gemm_prefill", "op": "gemm", "T": 4096, "K": 6144, "N": 18432, "bias": True, "dtype": "fp16"},
        # the LayerNorm in front of that projection, for the whole prompt
        {"name": "act_ln_prefill", "op": "act", "kind": "ln", "T": 4096, "K": 6144, "dtype": "fp16", "y": False},
        # GeLU and bias between the two FFN matrices of a GPT-J-sized layer, an odd number of tokens
        {"name": "act_gelu", "op": "act", "kind": "gelu", "T": 1531, "K": 16384, "dtype": "bf16", "y": False},
        # a decode step's attention output, quantized as it is: the smallest call, where latency counts
        {"name": "act_plain_decode", "op": "act", "kind": "plain", "T": 3, "K": 4096, "dtype": "fp16", "y": False},
        # one FFN matrix of a GPT-NeoX-sized layer, as a checkpoint loader quantizes it
        {"name": "weight_ffn", "op": "weight", "N": 24576, "K": 6144, "dtype": "bf16"},
        # a small matrix with cut-off blocks on both sides
        {"name": "weight_odd", "op": "weight", "N": 1032, "K": 1808, "dtype": "fp16"},
        # GPT-NeoX: a quarter of each head rotated, halves layout, no norm, a whole prompt
        {"name": "rope_prefill_partial", "op": "rope", "T": 4096, "Hq": 64, "Hk": 64, "D": 96, "R": 24,
         "layout": "half", "norm": "none", "scaling": "none", "far": 0, "dtype": "fp16"},
        # shared key heads, normed queries and keys, whole heads rotated at far positions of a stretched context
        {"name": "rope_norm_far", "op": "rope", "T": 2011, "Hq": 32, "Hk": 8, "D": 128, "R": 128,
         "layout": "half", "norm": "rms", "scaling": "yarn", "far": 900000, "dtype": "bf16"},
        # GPT-J: pairs of neighbours rotated in the first 64 of 256 dims, a decode step of a few sequences
        {"name": "rope_decode", "op": "rope", "T": 5, "Hq": 16, "Hk": 16, "D": 256, "R": 64,
         "layout": "interleaved", "norm": "none", "scaling": "none", "far": 2000, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _mult(v, m, lo, hi):
    return max(lo, min(hi, int(round(v / m)) * m))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "act", "weight", "rope"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "gemm":
        while True:
            T = _mult(_log(rng, 1, 4096), 1, 1, 4096)
            K = _mult(_log(rng, 64, 24576), 16, 64, 24576)
            N = _mult(_log(rng, 64, 24576), 8, 64, 24576)
            if T * K * N <= 4096 * 6144 * 18432 and N * K <= 24576 * 6144:
                return {"op": op, "T": T, "K": K, "N": N, "bias": rng.random() < 0.5, "dtype": dtype}
    if op == "act":
        while True:
            T = _mult(_log(rng, 1, 16384), 1, 1, 16384)
            K = _mult(_log(rng, 64, 24576), 16, 64, 24576)
            if T * K <= 4096 * 6144:
                return {"op": op, "kind": rng.choice(["ln", "gelu", "plain"]), "T": T, "K": K, "dtype": dtype,
                        "y": rng.random() < 0.3}
    if op == "weight":
        while True:
            N = _mult(_log(rng, 64, 24576), 8, 64, 24576)
            K = _mult(_log(rng, 64, 24576), 16, 64, 24576)
            if N * K <= 24576 * 6144:
                return {"op": op, "N": N, "K": K, "dtype": dtype}
    while True:
        T = _mult(_log(rng, 1, 8192), 1, 1, 8192)
        Hk = rng.choice([1, 2, 4, 8, 12, 16, 32, 64])
        Hq = min(64, Hk * rng.choice([1, 1, 2, 4, 7]))
        D = rng.choice([64, 80, 96, 128, 192, 256])
        R = rng.choice([D, D, D // 2, D // 4])
        if T * (Hq + Hk) * D <= 4096 * 128 * 96:
            return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R,
                    "layout": rng.choice(["half", "interleaved"]), "norm": rng.choice(["none", "rms", "layer"]),
                    "scaling": rng.choice(["none", "linear", "yarn"]),
                    "far": int(_log(rng, 1, 1000000)), "dtype": dtype}


# --------------------------------------------------------------------------- inputs

def _blocks(n):
    return -(-n // BLOCK)


def _pad(x, rows, cols):
    """x with zeros behind its rows and columns, up to whole multiples of rows and cols."""
    r, c = -x.shape[0] % rows, -x.shape[1] % cols
    return torch.nn.functional.pad(x, (0, c, 0, r)) if r or c else x


def _quantize(y, rows):
    """e4m3 codes and scales of a matrix in 32 bits: one scale for each `rows` x 128 values."""
    n, k = y.shape
    p = _pad(y, rows, BLOCK)
    b = p.view(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)
    amax = b.abs().amax(dim=(1, 3))
    a = amax.clamp_min(AMAX_FLOOR)
    inv = torch.where(amax > 0, E4M3_MAX / a, torch.zeros_like(a))
    scale = torch.where(amax > 0, a / E4M3_MAX, torch.zeros_like(a))
    q = (b * inv[:, None, :, None]).reshape(p.shape)[:n, :k]
    return q.to(F8).contiguous(), scale


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, T, K):
    """Normal values with a few outlier channels, as the inputs of transformer layers have."""
    x = _randn(g, T, K)
    ch = torch.randint(0, K, (max(1, K // 1000),), generator=g, device="cuda")
    x[:, ch] *= 30.0
    return x


def _inverse_frequencies(R, scaling):
    """Frequencies in 64 bits, rounded once, and the factor on cosine and sine.  `linear`: positions of a context
    stretched 8 times; `yarn`: stretched 8 times from 4096 positions, with the ramp between 32 and 1 turns."""
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if scaling == "linear":
        return (f / 8.0).float(), 1.0
    if scaling == "yarn":
        turns = 4096.0 * f / (2.0 * math.pi)
        # turns(i) falls with i: 1 = keep the frequency (many turns), 0 = divide it (few turns)
        dim = lambda n: R * math.log(4096.0 / (n * 2.0 * math.pi)) / (2.0 * math.log(10000.0))  # noqa: E731
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), R - 1)
        ramp = ((torch.arange(turns.numel(), dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return (f * (1.0 - ramp) + f / 8.0 * ramp).float(), 0.1 * math.log(8.0) + 1.0
    return f.float(), 1.0


def prepare(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    if case["op"] == "gemm":
        T, K, N = case["T"], case["K"], case["N"]
        xq, sx = _quantize(_activations(g, T, K), 1)
        wq, sw = _quantize(_randn(g, N, K) * 0.02, BLOCK)
        bias = (_randn(g, N) * 0.1).to(dt) if case["bias"] else None
        return {"case": case, "xq": xq, "sx": sx, "wq": wq, "sw": sw, "bias": bias, "dt": dt}
    if case["op"] == "act":
        T, K = case["T"], case["K"]
        x = _activations(g, T, K).to(dt)
        a = (1.0 + 0.1 * _randn(g, K)).to(dt)
        b = (0.1 * _randn(g, K)).to(dt)
        return {"case": case, "x": x, "gamma": a, "beta": b}
    if case["op"] == "weight":
        w = _randn(g, case["N"], case["K"]) * 0.02
        w *= torch.exp(_randn(g, case["N"], 1) * 0.5)  # rows of unequal range
        return {"case": case, "w": w.to(dt)}
    T, Hq, Hk, D, R = (case[k] for k in ("T", "Hq", "Hk", "D", "R"))
    qkv = _randn(g, T, Hq + 2 * Hk, D).to(dt)  # the output of the fused QKV projection
    inv_freq, factor = _inverse_frequencies(R, case["scaling"])
    pos = case["far"] + torch.arange(T, device="cuda")
    if T <= 64:  # decoding sequences of unequal length
        pos = torch.randint(0, case["far"] + T, (T,), generator=g, device="cuda")
    norm = {}
    if case["norm"] != "none":
        norm["q_weight"] = (1.0 + 0.1 * _randn(g, D)).to(dt)
        norm["k_weight"] = (1.0 + 0.1 * _randn(g, D)).to(dt)
    if case["norm"] == "layer":
        norm["q_bias"] = (0.1 * _randn(g, D)).to(dt)
        norm["k_bias"] = (0.1 * _randn(g, D)).to(dt)
    return {"case": case, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "pos": pos.to(torch.int32),
            "inv_freq": inv_freq.cuda(), "factor": factor, "norm": norm}


# --------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "gemm":
        y = _gemm(state, torch.float32)
        return y.to(state["dt"])
    if case["op"] == "act":
        y = _activate(state, torch.float32)
        q, s = _quantize(y, 1)
        return {"codes": q, "scales": s, "y": y.to(state["x"].dtype)} if case["y"] else {"codes": q, "scales": s}
    if case["op"] == "weight":
        q, s = _quantize(state["w"].float(), BLOCK)
        return {"codes": q, "scales": s}
    return {n: _rotate(state, n, torch.float32).to(state[n].dtype) for n in ("q", "k")}


def _run_own(state, case):
    from int4_quantized_transformer_b200 import zq

    if case["op"] == "gemm":
        return zq.gemm_fp8(state["xq"], state["sx"], state["wq"], state["sw"], state["bias"], out_dtype=state["dt"])
    if case["op"] == "act":
        x = state["x"]
        y = torch.empty_like(x) if case["y"] else None
        if case["kind"] == "ln":
            q, s = zq.ln_quant_fp8(x, state["gamma"], state["beta"], 1e-5, y_ln=y)
        elif case["kind"] == "gelu":
            q, s = zq.bias_act_quant_fp8(x, state["beta"], zq.ACT_GELU, y=y)
        else:
            q, s = zq.bias_act_quant_fp8(x, y=y)
        return {"codes": q, "scales": s, "y": y} if case["y"] else {"codes": q, "scales": s}
    if case["op"] == "weight":
        q, s = zq.quantize_weights_fp8(state["w"])
        return {"codes": q, "scales": s}
    norm = {"none": zq.NORM_NONE, "rms": zq.NORM_RMS, "layer": zq.NORM_LAYER}[case["norm"]]
    layout = zq.ROPE_HALF if case["layout"] == "half" else zq.ROPE_INTERLEAVED
    q, k = zq.qk_norm_rope(state["q"], state["k"], state["pos"], state["inv_freq"], layout=layout,
                           scale=state["factor"], norm=norm, eps=1e-6, **state["norm"])
    return {"q": q, "k": k}


def _gemm(state, ft):
    k, n = state["xq"].shape[1], state["wq"].shape[0]
    x = state["xq"].to(ft) * state["sx"].to(ft).repeat_interleave(BLOCK, 1)[:, :k]
    w = state["wq"].to(ft)
    w = w * state["sw"].to(ft).repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    y = x @ w.T
    return y if state["bias"] is None else y + state["bias"].to(ft)


def _activate(state, ft):
    kind, x = state["case"]["kind"], state["x"].to(ft)
    if kind == "ln":
        d = x - x.mean(dim=1, keepdim=True)
        y = d * torch.rsqrt((d * d).mean(dim=1, keepdim=True) + 1e-5)
        return y * state["gamma"].to(ft) + state["beta"].to(ft)
    if kind == "gelu":
        v = x + state["beta"].to(ft)
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    return x


def _rotate(state, name, ft):
    case, x = state["case"], state[name].to(ft)
    R, norm = case["R"], state["norm"]
    if case["norm"] == "layer":
        x = x - x.mean(dim=-1, keepdim=True)
    if case["norm"] != "none":
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * norm[name + "_weight"].to(ft)
    if case["norm"] == "layer":
        x = x + norm[name + "_bias"].to(ft)
    angle = state["pos"].double()[:, None] * state["inv_freq"].double()  # far positions: 64 bits
    cos, sin = ((fn(angle) * state["factor"]).to(ft)[:, None, :] for fn in (torch.cos, torch.sin))
    if case["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((turned, x[..., R:]), dim=-1)


# --------------------------------------------------------------------------- cost

def work(case):
    if case["op"] == "gemm":
        T, K, N = case["T"], case["K"], case["N"]
        scales = 4 * (T * _blocks(K) + _blocks(N) * _blocks(K))
        return {"bytes": T * K + N * K + scales + 2 * T * N + (2 * N if case["bias"] else 0), "flops": 2 * T * K * N}
    if case["op"] == "act":
        T, K = case["T"], case["K"]
        per = {"ln": 10, "gelu": 25, "plain": 3}[case["kind"]]
        params = {"ln": 4, "gelu": 2, "plain": 0}[case["kind"]] * K
        return {"bytes": T * K * (5 if case["y"] else 3) + 4 * T * _blocks(K) + params, "flops": per * T * K}
    if case["op"] == "weight":
        N, K = case["N"], case["K"]
        return {"bytes": 3 * N * K + 4 * _blocks(N) * _blocks(K), "flops": 3 * N * K}
    T, H, D, R = case["T"], case["Hq"] + case["Hk"], case["D"], case["R"]
    per = {"none": 0, "rms": 4, "layer": 7}[case["norm"]] * D + 3 * R
    return {"bytes": 4 * T * H * D + 4 * T + 2 * R, "flops": T * H * per}


# --------------------------------------------------------------------------- the definition in 64 bits

def _e4m3_64(v):
    """v (64 bits, at most 448 in magnitude) rounded to the nearest e4m3 value, halves to even."""
    m = v.abs()
    e = torch.frexp(m)[1].sub_(1).clamp_min_(-6)  # 2^e <= m < 2^(e+1); below 2^-6 the step stays 2^-9
    step = torch.ldexp(torch.ones_like(m), e - 3)
    return torch.round(v / step).mul_(step).clamp_(-E4M3_MAX, E4M3_MAX)


def _quantize_64(y, rows):
    q, s = torch.empty_like(y), torch.zeros(-(-y.shape[0] // rows), _blocks(y.shape[1]), dtype=y.dtype, device=y.device)
    for c in range(s.shape[1]):
        b = _pad(y[:, c * BLOCK:(c + 1) * BLOCK], rows, 1)
        amax = b.abs().reshape(s.shape[0], -1).max(dim=1).values
        s[:, c] = torch.where(amax > 0, amax.clamp_min(AMAX_FLOOR), amax) / E4M3_MAX
        by = s[:, c].repeat_interleave(rows)[:y.shape[0], None]
        q[:, c * BLOCK:(c + 1) * BLOCK] = torch.where(by > 0, b[:y.shape[0]] / by, torch.zeros_like(by))
    return _e4m3_64(q).to(F8), s


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "gemm":
        # block by block, as the definition says
        T, K, N = case["T"], case["K"], case["N"]
        y = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        for c in range(_blocks(K)):
            cols = slice(c * BLOCK, min(K, (c + 1) * BLOCK))
            part = state["xq"][:, cols].double() @ state["wq"][:, cols].double().T
            part *= state["sx"][:, c].double()[:, None]
            part *= state["sw"][:, c].double().repeat_interleave(BLOCK)[None, :N]
            y += part
        return y if state["bias"] is None else y + state["bias"].double()
    if case["op"] == "act":
        x, K = state["x"].double(), case["K"]
        if case["kind"] == "ln":
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            y = (x - mean) / torch.sqrt(var + 1e-5) * state["gamma"].double() + state["beta"].double()
        elif case["kind"] == "gelu":
            v = x + state["beta"].double()
            y = v * torch.special.ndtr(v)
        else:
            y = x
        q, s = _quantize_64(y, 1)
        return {"codes": q, "scales": s, "y": y} if case["y"] else {"codes": q, "scales": s}
    if case["op"] == "weight":
        q, s = _quantize_64(state["w"].double(), BLOCK)
        return {"codes": q, "scales": s}
    out = {}
    R, half = case["R"], case["R"] // 2
    turn = torch.polar(torch.full((case["T"], half), state["factor"], dtype=torch.float64, device="cuda"),
                       torch.outer(state["pos"].double(), state["inv_freq"].double()))[:, None, :]
    for n in ("q", "k"):
        x = state[n].double()
        if case["norm"] == "layer":
            x = torch.nn.functional.layer_norm(x, x.shape[-1:], state["norm"][n + "_weight"].double(),
                                               state["norm"][n + "_bias"].double(), 1e-6)
        elif case["norm"] == "rms":
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * state["norm"][n + "_weight"].double()
        y = x.clone()
        at = (slice(0, half), slice(half, R)) if case["layout"] == "half" else (slice(0, R, 2), slice(1, R, 2))
        z = torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous()) * turn
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        out[n] = y
    return out
