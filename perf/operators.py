"""Measured cases of the operators that serve a quantized layer.

  gemv   gptq_dequant_gemv       a few tokens through packed weights (decoding)
  norm   gptq_rms_norm_e4m3      residual addition, root-mean-square norm, e4m3 rows with a scale each
  quant  gptq_quantize_e4m3      e4m3 rows with a scale each
  gemm   gptq_dequant_gemm_e4m3  e4m3 rows through packed weights (prefill, large batches)

``run`` computes them with elementary torch operations where ``own`` is false, and calls the library
where it is true.  Packed layouts are the quantizer's: qweight int32 [ceil(d_in b / 32), d_out], scales
fp16 [n_groups, d_out], qzeros int32 [n_groups, ceil(d_out b / 32)], g_idx int32 [d_in].
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------ cases

def _product(op, M, d_out, d_in, bits, g, sym, x, y, act=False):
    return dict(op=op, M=M, d_out=d_out, d_in=d_in, bits=bits, g=g, sym=sym, x=x, y=y, act=act)


def listed():
    return [
        # one token through an attention projection of the 4096 x 4096 layer: launch latency counts
        dict(name="gemv_1_attn", **_product("gemv", 1, 4096, 4096, 4, 128, False, "bf16", "bf16")),
        # sixteen sequences through the 3-bit ffn_up layer, fp32 sums for a gate
        dict(name="gemv_16_up", **_product("gemv", 16, 11008, 4096, 3, 64, True, "bf16", "f32")),
        # two sequences through a down projection that was quantized in activation order
        dict(name="gemv_2_down_act", **_product("gemv", 2, 4096, 11008, 4, 128, False, "bf16", "bf16", True)),
        # a wide output head with an odd number of rows, eight e4m3 tokens: the weight stream counts
        dict(name="gemv_8_head", **_product("gemv", 8, 50001, 8192, 4, 128, False, "e4m3", "f32")),
        # the norm before a projection while decoding one token
        dict(name="norm_1", op="norm", M=1, d_in=4096, x="bf16", w="bf16", res=True),
        # the norm of a 2048-token prompt
        dict(name="norm_2048", op="norm", M=2048, d_in=4096, x="bf16", w="bf16", res=True),
        # a long batch of wide fp32 rows, odd number of rows, no residual
        dict(name="norm_8191_wide", op="norm", M=8191, d_in=16384, x="f32", w="f32", res=False),
        # the input of a down projection while decoding sixteen sequences
        dict(name="quant_16", op="quant", M=16, d_in=11008, x="bf16"),
        # the same for a batch of prompts
        dict(name="quant_4096", op="quant", M=4096, d_in=11008, x="bf16"),
        # a large decoding batch through the 2-bit down projection
        dict(name="gemm_96_down", **_product("gemm", 96, 4096, 11008, 2, 32, False, "e4m3", "f32")),
        # a 2048-token prompt through the attention layer
        dict(name="gemm_2048_attn", **_product("gemm", 2048, 4096, 4096, 4, 128, False, "e4m3", "f32")),
        # a long batch through an up projection
        dict(name="gemm_8192_up", **_product("gemm", 8192, 11008, 4096, 4, 128, True, "e4m3", "bf16")),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + step)))) // step * step)


def draw(rng):
    op = rng.choice(["gemv", "gemv", "norm", "quant", "gemm", "gemm"])
    if op in ("norm", "quant"):
        d = _log(rng, 8, 32768, 8)
        M = _log(rng, 1, min(16384, (1 << 27) // d))
        c = dict(op=op, M=M, d_in=d, x=rng.choice(["bf16", "f32"]))
        if op == "norm":
            c.update(w=rng.choice(["bf16", "f32"]), res=rng.random() < 0.7)
        return c
    sym = rng.random() < 0.4
    y = rng.choice(["bf16", "f32"])
    if op == "gemv":
        d_in = _log(rng, 64, 16384, 8)
        d_out = _log(rng, 1, min(65536, 4 * 10 ** 8 // d_in))
        return _product("gemv", _log(rng, 1, 64), d_out, d_in, rng.choice([2, 3, 4, 4, 8]),
                        rng.choice([-1, 16, 32, 64, 128, 128]), sym, rng.choice(["bf16", "bf16", "e4m3"]), y,
                        rng.random() < 0.25)
    g = rng.choice([-1, 32, 64, 128, 128])
    d_in = _log(rng, 128, 16384, max(g, 32))
    d_out = _log(rng, 8, 32768, 8)
    M = _log(rng, 1, max(1, min(8192, 8192 * 11008 * 4096 // (d_in * d_out))))
    return _product("gemm", M, d_out, d_in, rng.choice([2, 3, 4, 4]), g, sym, "e4m3", y)


def _groups(case):
    return 1 if case["g"] == -1 else -(-case["d_in"] // case["g"])


def work(case):
    n = case["M"] * case["d_in"]
    if case["op"] in ("norm", "quant"):
        e = 2 if case["x"] == "bf16" else 4
        b = n * (e + 1) + 4 * case["M"]
        if case["op"] == "norm":
            b += (2 if case["w"] == "bf16" else 4) * case["d_in"] + (2 * n * e if case["res"] else 0)
        return {"bytes": b, "flops": 6 * n}
    N, bits, ng = case["d_out"], case["bits"], _groups(case)
    b = 4 * (case["d_in"] * bits // 32) * N + 2 * ng * N + (0 if case["sym"] else ng * N * bits // 8)
    b += n * (2 if case["x"] == "bf16" else 1) + case["M"] * N * (2 if case["y"] == "bf16" else 4)
    b += (4 * case["M"] if case["x"] == "e4m3" else 0) + (4 * case["d_in"] if case["act"] else 0)
    return {"bytes": b, "flops": 2 * n * N}


# ----------------------------------------------------------------------------------------- inputs

def _activations(r, M, d):
    """Rows with lognormal channel magnitudes and half a percent of channels fifty times larger."""
    std = torch.exp(torch.randn(d, generator=r, device=DEV))
    std = std * torch.where(torch.rand(d, generator=r, device=DEV) < 0.005, 50.0, 1.0)
    return torch.randn((M, d), generator=r, device=DEV) * std


def _pack(codes, bits):
    """Little-endian stream of codes along the first axis of [k, n], as int32 words [ceil(k b / 32), n]."""
    k, n = codes.shape
    per = 32 if bits == 3 else 32 // bits           # codes in a whole number of words
    words = per * bits // 32
    pad = torch.zeros((-(-k // per) * per, n), dtype=torch.int64, device=codes.device)
    pad[:k] = codes
    pad = pad.view(-1, per, n)
    out = torch.zeros((pad.shape[0], words, n), dtype=torch.int64, device=codes.device)
    for j in range(per):
        w, sh = j * bits // 32, j * bits % 32
        out[:, w] |= (pad[:, j] << sh) & 0xFFFFFFFF
        if sh + bits > 32:
            out[:, w + 1] |= pad[:, j] >> (32 - sh)
    out = out.view(-1, n)[: (k * bits + 31) // 32]
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32).contiguous()


def prepare(case, seed):
    r = torch.Generator(device=DEV)
    r.manual_seed(seed)
    M, d = case["M"], case["d_in"]
    s = {"case": case}
    X = _activations(r, M, d)
    if case["op"] in ("norm", "quant"):
        s["X"] = X.to(TYPES[case["x"]])
        s["X8"] = torch.empty((M, d), dtype=torch.float8_e4m3fn, device=DEV)
        s["xs"] = torch.empty((M,), dtype=torch.float32, device=DEV)
        if case["op"] == "norm":
            s["w"] = (1 + 0.2 * torch.randn(d, generator=r, device=DEV)).to(TYPES[case["w"]])
            s["eps"] = 1e-6
            if case["res"]:
                s["R"] = (4 * torch.randn((M, d), generator=r, device=DEV)).to(TYPES[case["x"]])
                s["R2"] = torch.empty_like(s["R"])
        return s
    N, bits, ng = case["d_out"], case["bits"], _groups(case)
    mid = 1 << (bits - 1)
    # codes as the rounding of normal weights leaves them: around the zero point, both ends used
    codes = torch.empty((d, N), dtype=torch.uint8, device=DEV)
    for k in range(0, d, 2048):
        part = torch.randn((min(2048, d - k), N), generator=r, device=DEV)
        codes[k:k + 2048] = (part * (mid / 2.5) + mid).round_().clamp_(0, 2 * mid - 1).to(torch.uint8)
    s["qweight"] = _pack(codes, bits)
    s["scales"] = (0.01 * torch.exp(0.3 * torch.randn((ng, N), generator=r, device=DEV))).to(torch.float16)
    s["qzeros"] = None
    if not case["sym"]:
        z = (mid + 0.12 * mid * torch.randn((ng, N), generator=r, device=DEV)).round().clamp(0, 2 * mid - 1)
        s["qzeros"] = _pack(z.to(torch.uint8).t().contiguous(), bits).t().contiguous()
    s["g_idx"] = None
    if case["act"]:
        g = d if case["g"] == -1 else case["g"]
        s["g_idx"] = (torch.argsort(torch.rand(d, generator=r, device=DEV)) // g).to(torch.int32)
    if case["x"] == "e4m3":
        s["X"], s["xs"] = _quantize_rows(X.to(torch.bfloat16).float())
    else:
        s["X"], s["xs"] = X.to(TYPES[case["x"]]), None
    s["Y"] = torch.empty((M, N), dtype=TYPES[case["y"]], device=DEV)
    if own:
        from post_weight_quantization_14_b200 import make_config
        s["cfg"] = make_config(bits, case["g"], case["sym"], desc_act=1 if case["act"] else 0)
    return s


# ----------------------------------------------------------------------------------- plain forms

def _quantize_rows(y):
    scale = y.abs().amax(dim=1) / E4M3_MAX
    q = y / torch.where(scale == 0, 1.0, scale)[:, None]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _unpack(words, bits, count):
    """The first ``count`` codes along the first axis of int32 words [w, n], as fp32 [count, n]."""
    n = words.shape[1]
    if bits == 3:
        w = torch.nn.functional.pad(words, (0, 0, 0, -words.shape[0] % 3)).view(-1, 3, n).to(torch.int64) & 0xFFFFFFFF
        lo, hi = w[:, 0] | ((w[:, 1] & 0xFFFF) << 32), (w[:, 1] >> 16) | (w[:, 2] << 16)   # 16 codes each
        sh = torch.arange(0, 48, 3, device=words.device)[None, :, None]
        q = torch.cat([(lo[:, None] >> sh) & 7, (hi[:, None] >> sh) & 7], dim=1)
    else:
        sh = torch.arange(0, 32, bits, dtype=torch.int32, device=words.device)[None, :, None]
        q = (words[:, None] >> sh) & ((1 << bits) - 1)
    return q.reshape(-1, n)[:count].float()


def _plain_product(s):
    c = s["case"]
    d, N, bits = c["d_in"], c["d_out"], c["bits"]
    if s["g_idx"] is not None:
        gi = s["g_idx"].long()
    else:
        gi = torch.arange(d, device=DEV) // (d if c["g"] == -1 else c["g"])
    W = _unpack(s["qweight"], bits, d)
    if c["sym"]:
        W -= 1 << (bits - 1)
    else:
        W -= _unpack(s["qzeros"].t(), bits, N).t()[gi]
    W *= s["scales"].float()[gi]
    Y = s["X"].float() @ W
    if s["xs"] is not None:
        Y *= s["xs"][:, None]
    return Y.to(s["Y"].dtype)


def _plain_rows(s):
    h = s["X"].float()
    if s["case"]["op"] == "quant":
        q, scale = _quantize_rows(h)
        return {"X8": q, "xs": scale}
    out = {}
    if "R" in s:
        h = h + s["R"].float()
        out["R2"] = h.to(s["R"].dtype)
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + s["eps"]) * s["w"].float()
    out["X8"], out["xs"] = _quantize_rows(y)
    return out


def run(s):
    c = s["case"]
    if not own:
        return _plain_rows(s) if c["op"] in ("norm", "quant") else _plain_product(s)
    import post_weight_quantization_14_b200 as G
    if c["op"] == "norm":
        R2 = s.get("R2")
        G.gptq_rms_norm_e4m3(s["X"], s["w"], s["X8"], s["xs"], s.get("R"), R2, s["eps"])
        return {"X8": s["X8"], "xs": s["xs"]} if R2 is None else {"X8": s["X8"], "xs": s["xs"], "R2": R2}
    if c["op"] == "quant":
        G.gptq_quantize_e4m3(s["X"], s["X8"], s["xs"])
        return {"X8": s["X8"], "xs": s["xs"]}
    if c["op"] == "gemv":
        return G.gptq_dequant_gemv(s["X"], s["qweight"], s["scales"], s["qzeros"], c["d_out"], c["d_in"], s["cfg"],
                                   s["Y"], s["xs"], s["g_idx"])
    return G.gptq_dequant_gemm_e4m3(s["X"], s["xs"], s["qweight"], s["scales"], s["qzeros"], c["d_out"], c["d_in"],
                                    s["cfg"], s["Y"])


# ------------------------------------------------------------------------------ 64-bit definition

def _code64(words, stride_first, index, bits):
    """Code ``index`` of each little-endian stream, read bit position by bit position."""
    w = (words if stride_first else words.t()).to(torch.int64) & 0xFFFFFFFF
    bit = index * bits
    k, sh = bit // 32, bit % 32
    v = w[k] >> sh[:, None]
    nxt = w[(k + 1).clamp(max=w.shape[0] - 1)]
    v = torch.where((sh + bits > 32)[:, None], v | (nxt << (32 - sh)[:, None]), v)
    return (v & ((1 << bits) - 1)).double()


def _e4m3_of(v):
    """v rounded to the e4m3 grid (three fraction bits, smallest exponent -6), ties to even, in fp64."""
    a = v.abs().clamp(min=2.0 ** -20)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6.0) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d_in"]
    if case["op"] in ("norm", "quant"):
        h = s["X"].double()
        out = {}
        if case["op"] == "norm":
            if case["res"]:
                h = h + s["R"].double()
                out["R2"] = h
            h = s["w"].double() * (h / torch.sqrt(torch.sum(h * h, dim=1, keepdim=True) / d + s["eps"]))
        out["xs"] = torch.amax(torch.abs(h), dim=1) / E4M3_MAX
        out["X8"] = _e4m3_of(h / out["xs"][:, None])
        return out
    N, bits = case["d_out"], case["bits"]
    columns = torch.arange(d, device=DEV)
    group = s["g_idx"].long() if case["act"] else (torch.zeros_like(columns) if case["g"] == -1 else columns // case["g"])
    X = s["X"].double()
    Y = torch.zeros((case["M"], N), dtype=torch.float64, device=DEV)
    zeros = None if case["sym"] else _code64(s["qzeros"], False, torch.arange(N, device=DEV), bits).t()
    for k in range(0, d, 1024):
        part = columns[k:k + 1024]
        q = _code64(s["qweight"], True, part, bits)
        z = float(1 << (bits - 1)) if zeros is None else zeros[group[part]]
        Y += X[:, part] @ ((q - z) * s["scales"].double()[group[part]])
    return Y if s["xs"] is None else Y * s["xs"].double()[:, None]
