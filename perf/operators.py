"""Measured cases of the 8-bit feed-forward operators: the block quantiser, the
8-bit matrix product, the gated activation and its backward pass.

A block-scaled 8-bit matrix holds e4m3 codes (torch.float8_e4m3fn) and, for
every block of 128 values along a row (or every 128 x 128 block of a weight),
a power-of-two scale (torch.float8_e8m0fnu). The value of an entry is its code
times its block's scale. The scale is the smallest power of two that brings
the block's largest magnitude to 448, the largest e4m3 value, or less.

  quantize    x -> codes and scales along the rows, and/or of x transposed
              (blocks along x's columns), each in one pass over x; x may be an
              8-bit matrix itself (a kept activation), then only transposed
  mm          C = A B^T + bias, A (M, K) and B (N, K) block-scaled along K
  swiglu      h = silu(gate) * up in 8 bits; optionally gate and up are kept
              in 8 bits for the backward pass
  swiglu_bwd  from dh and the kept gate and up: their gradients in 8 bits, and
              with h again also transposed (operands of the weight gradients)

`run` gives the codes and scales as torch's 8-bit float types, so that what is
compared are the values they stand for.
"""
import math

import torch

own = False

BLK = 128
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # the activations of one token in front of a 4096-wide product: latency
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 4096, "dtype": "fp16", "block": 1,
         "straight": True, "transposed": False},
        # an output gradient, as the operand of the input's and of the weight's gradient
        {"name": "quantize_gradient", "op": "quantize", "rows": 4096, "cols": 4096, "dtype": "bf16", "block": 1,
         "straight": True, "transposed": True},
        # a weight after an optimizer step, for the forward and the backward product
        {"name": "quantize_weight", "op": "quantize", "rows": 11008, "cols": 4096, "dtype": "fp32", "block": 128,
         "straight": True, "transposed": True},
        # a kept 8-bit activation turned into the operand of the weight gradient, ragged token count
        {"name": "quantize_kept", "op": "quantize", "rows": 4095, "cols": 4096, "dtype": "e4m3", "block": 1,
         "straight": False, "transposed": True},
        # decoding one token through the gate projection (4096 x 11008): the weight's bytes
        {"name": "mm_token", "op": "mm", "M": 1, "N": 11008, "K": 4096, "dtype": "fp16", "block": 128, "bias": False},
        # a small serving batch through the down projection, odd rows
        {"name": "mm_batch", "op": "mm", "M": 33, "N": 4096, "K": 11008, "dtype": "bf16", "block": 128, "bias": False},
        # a training or prefill product at the size of the framework's square GEMM
        {"name": "mm_forward", "op": "mm", "M": 8192, "N": 8192, "K": 8192, "dtype": "fp16", "block": 128,
         "bias": True},
        # a weight gradient in fp32: the contraction runs over a ragged number of tokens
        {"name": "mm_weight_gradient", "op": "mm", "M": 11008, "N": 4096, "K": 4095, "dtype": "fp32", "block": 1,
         "bias": False},
        # decoding one token: nothing is kept
        {"name": "swiglu_token", "op": "swiglu", "rows": 1, "cols": 11008, "dtype": "fp16", "keep": False},
        # a training step's activation between the two products, gate and up kept
        {"name": "swiglu_train", "op": "swiglu", "rows": 4096, "cols": 11008, "dtype": "bf16", "keep": True},
        # the backward pass on one rank of eight (11008 / 8 = 1376 columns: a ragged last block), few odd rows
        {"name": "swiglu_bwd_shard", "op": "swiglu_bwd", "rows": 1001, "cols": 1376, "dtype": "fp16"},
        # the backward pass of a whole layer
        {"name": "swiglu_bwd_train", "op": "swiglu_bwd", "rows": 4096, "cols": 11008, "dtype": "bf16"},
    ]


def _size(rng, lo, hi):
    """A length between lo and hi, spread over its logarithm; about half of them multiples of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 32:
        v -= v % 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "mm", "mm", "swiglu", "swiglu_bwd"])
    if op == "quantize":
        dtype = rng.choice(["fp16", "bf16", "fp32", "e4m3"])
        block = 1 if dtype == "e4m3" else rng.choice([1, 1, 128])
        way = "transposed" if dtype == "e4m3" else rng.choice(["straight", "both", "both", "transposed"])
        return {"op": op, "rows": _size(rng, 1, 11008), "cols": _size(rng, 64, 11008), "dtype": dtype, "block": block,
                "straight": way != "transposed", "transposed": way != "straight"}
    if op == "mm":
        M, N, K = _size(rng, 1, 11008), _size(rng, 64, 11008), _size(rng, 64, 11008)
        while M * N * K > 8192 ** 3:
            M, N, K = (max(64, 3 * v // 4) for v in (M, N, K))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(["fp16", "bf16", "fp32"]),
                "block": rng.choice([1, 128]), "bias": rng.random() < 0.5}
    case = {"op": op, "rows": _size(rng, 1, 4096), "cols": _size(rng, 64, 11008), "dtype": rng.choice(["fp16", "bf16"])}
    if op == "swiglu":
        case["keep"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- the inputs

def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(rows, cols, gen):
    """Rows of different sizes, a few columns that stand out, and a last row of padding where there are several."""
    x = _normal((rows, cols), gen)
    x *= torch.exp(0.5 * _normal((rows, 1), gen))
    x *= 1.0 + 15.0 * (torch.rand((1, cols), generator=gen, device="cuda") < 0.004).float()
    if rows > 8:
        x[-1] = 0.0
    return x


def _blank8(rows, cols, block=1):
    """Memory of a block-scaled matrix: rows of codes start at multiples of 16 bytes, rows of scales at multiples of 4."""
    ld, ls = -(-cols // 16) * 16, -(-(-(-cols // BLK)) // 4) * 4
    codes = torch.zeros((rows, ld), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((-(-rows // block), ls), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    return codes[:, :cols], scales[:, :-(-cols // BLK)]


def _made8(x, block=1):
    q, s = _blank8(x.shape[0], x.shape[1], block)
    codes, scales = _quantized(x, block)
    q.copy_(codes)
    s.copy_(scales)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "mm":
        M, N, K, dt = case["M"], case["N"], case["K"], TYPES[case["dtype"]]
        s["A"] = _made8(_activations(M, K, gen))
        b = _normal((N, K), gen) / math.sqrt(K) if case["block"] == 128 else _activations(N, K, gen)
        s["B"] = _made8(b, case["block"])
        s["bias"] = (0.1 * _normal((N,), gen)).to(dt) if case["bias"] else None
        s["C"] = torch.empty((M, N), dtype=dt, device="cuda")
        names = {"A": 1, "B": case["block"]}
    else:
        rows, cols = case["rows"], case["cols"]
        if case["op"] == "quantize":
            x = _activations(rows, cols, gen)
            if case["block"] == 128:
                x = _normal((rows, cols), gen) / math.sqrt(cols)
            s["x"] = _made8(x) if case["dtype"] == "e4m3" else x.to(TYPES[case["dtype"]])
            s["q"] = _blank8(rows, cols, case["block"]) if case["straight"] else None
            s["qt"] = _blank8(cols, rows, case["block"]) if case["transposed"] else None
            names = {"q": case["block"], "qt": case["block"]}
            if case["dtype"] == "e4m3":
                names["x"] = 1
        elif case["op"] == "swiglu":
            s["gate"], s["up"] = (_activations(rows, cols, gen).to(TYPES[case["dtype"]]) for _ in range(2))
            s["h"] = _blank8(rows, cols)
            s["gate8"], s["up8"] = (_blank8(rows, cols) if case["keep"] else None for _ in range(2))
            names = {"h": 1, "gate8": 1, "up8": 1}
        else:
            s["dh"] = (_activations(rows, cols, gen) / 64).to(TYPES[case["dtype"]])
            s["gate8"], s["up8"] = (_made8(_activations(rows, cols, gen)) for _ in range(2))
            s["dgate"], s["dup"] = _blank8(rows, cols), _blank8(rows, cols)
            s["dgate_t"], s["dup_t"], s["h_t"] = (_blank8(cols, rows) for _ in range(3))
            names = {k: 1 for k in ("gate8", "up8", "dgate", "dup", "dgate_t", "dup_t", "h_t")}
    if own:  # the handles that a program keeps of its block-scaled buffers
        import gemm_collective_tile_amd as il
        s["il"] = il
        s["m"] = {k: None if s[k] is None else il.Fp8(*s[k], block=b) for k, b in names.items()}
    return s


# ------------------------------------------------------------ the plain forms

def _blocks(x, block):
    """x (rows, cols) padded with zeros and seen as (row blocks, block, column blocks, 128)."""
    r, c = -(-x.shape[0] // block) * block, -(-x.shape[1] // BLK) * BLK
    if (r, c) != tuple(x.shape):
        p = torch.zeros((r, c), dtype=x.dtype, device=x.device)
        p[:x.shape[0], :x.shape[1]] = x
        x = p
    return x.reshape(r // block, block, c // BLK, BLK)


def _quantized(x, block=1):
    """Codes and scales of a matrix of finite values, computed in 32 bits."""
    b = _blocks(x.float(), block)
    amax = b.abs().amax(dim=(1, 3), keepdim=True)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(-126, 127).to(torch.int32)
    codes = (b * ((127 - e) << 23).view(torch.float32)).reshape(-1, b.shape[2] * BLK)
    codes = codes[:x.shape[0], :x.shape[1]].to(torch.float8_e4m3fn)
    scales = (e + 127).to(torch.uint8).reshape(b.shape[0], b.shape[2]).view(torch.float8_e8m0fnu)
    return codes, scales


def _values(q, block=1):
    """The 32-bit values of a block-scaled matrix."""
    codes, scales = q
    b = _blocks(codes.float(), block)
    v = b * scales.float().reshape(b.shape[0], 1, b.shape[2], 1)
    return v.reshape(-1, b.shape[2] * BLK)[:codes.shape[0], :codes.shape[1]]


def _plain(s):
    case = s["case"]
    if case["op"] == "mm":
        c = torch.matmul(_values(s["A"]), _values(s["B"], case["block"]).t())
        if s["bias"] is not None:
            c = c + s["bias"].float()
        return c.to(TYPES[case["dtype"]])
    if case["op"] == "quantize":
        x = _values(s["x"]) if case["dtype"] == "e4m3" else s["x"].float()
        return [_quantized(x, case["block"]) if case["straight"] else None,
                _quantized(x.t(), case["block"]) if case["transposed"] else None]
    if case["op"] == "swiglu":
        g, u = s["gate"].float(), s["up"].float()
        h = g / (1.0 + torch.exp(-g)) * u
        return [_quantized(h)] + ([_quantized(g), _quantized(u)] if case["keep"] else [])
    g, u, dh = _values(s["gate8"]), _values(s["up8"]), s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = g * sig
    dg = dh * u * (sig * (1.0 + g * (1.0 - sig)))
    du = dh * silu
    return [_quantized(dg), _quantized(du), _quantized(dg.t()), _quantized(du.t()), _quantized((silu * u).t())]


def run(state):
    if not own:
        return _plain(state)
    s, il, m, case = state, state["il"], state["m"], state["case"]
    if case["op"] == "mm":
        il.iris_fp8_mm(s["C"], m["A"], m["B"], s["bias"])
        return s["C"]
    if case["op"] == "quantize":
        il.iris_fp8_quantize(m.get("x", s["x"]), m["q"], m["qt"])
        return [s["q"], s["qt"]]
    if case["op"] == "swiglu":
        il.iris_fp8_swiglu(m["h"], s["gate"], s["up"], m["gate8"], m["up8"])
        return [s["h"]] + ([s["gate8"], s["up8"]] if case["keep"] else [])
    il.iris_fp8_swiglu_bwd(m["dgate"], m["dup"], s["dh"], m["gate8"], m["up8"], m["dgate_t"], m["dup_t"], m["h_t"])
    return [s["dgate"], s["dup"], s["dgate_t"], s["dup_t"], s["h_t"]]


# ------------------------------------------------------- work, exact results

def _bytes8(rows, cols, block=1):
    return rows * cols + -(-rows // block) * -(-cols // BLK)


def work(case):
    if case["op"] == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        out = TYPES[case["dtype"]].itemsize
        return {"bytes": _bytes8(M, K) + _bytes8(N, K, case["block"]) + M * N * out + (N * out if case["bias"] else 0),
                "flops": 2 * M * N * K}
    r, c = case["rows"], case["cols"]
    if case["op"] == "quantize":
        b = _bytes8(r, c) if case["dtype"] == "e4m3" else r * c * TYPES[case["dtype"]].itemsize
        b += _bytes8(r, c, case["block"]) if case["straight"] else 0
        b += _bytes8(c, r, case["block"]) if case["transposed"] else 0
        return {"bytes": b, "flops": 4 * r * c}
    if case["op"] == "swiglu":
        return {"bytes": 4 * r * c + (3 if case["keep"] else 1) * _bytes8(r, c), "flops": 8 * r * c}
    return {"bytes": 2 * r * c + 4 * _bytes8(r, c) + 3 * _bytes8(c, r), "flops": 20 * r * c}


def _exact_scaled(x, block=1, given=True):
    """x / scale before the rounding to 8 bits, and the scales, both as 64-bit values: how far a code is from the first
    is its rounding, half an e4m3 step at most. Where x is computed and not given, the scales have no exact value: at
    a largest magnitude within rounding of 448 times a power of two, either neighbour is right."""
    rows, cols = x.shape
    top = torch.zeros((-(-rows // block), -(-cols // BLK)), dtype=torch.float64, device=x.device)
    for j in range(top.shape[1]):
        m = x[:, j * BLK:(j + 1) * BLK].abs().max(dim=1).values
        if block > 1:
            m = torch.stack([part.max() for part in m.split(block)])
        top[:, j] = m
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448.0)).clamp(-126, 127)
    scale = torch.pow(torch.full_like(e, 2.0), e)
    wide = scale.repeat_interleave(block, 0)[:rows].repeat_interleave(BLK, 1)[:, :cols]
    return x / wide, (scale if given else None)


def _exact_values(q, block=1):
    codes, scales = q
    rows, cols = codes.shape
    return codes.double() * scales.double().repeat_interleave(block, 0)[:rows].repeat_interleave(BLK, 1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "mm":
        c = _exact_values(s["A"]) @ _exact_values(s["B"], case["block"]).t().contiguous()
        return c if s["bias"] is None else c + s["bias"].double()
    if case["op"] == "quantize":
        x = _exact_values(s["x"]) if case["dtype"] == "e4m3" else s["x"].double()
        return [_exact_scaled(x, case["block"]) if case["straight"] else None,
                _exact_scaled(x.t(), case["block"]) if case["transposed"] else None]
    if case["op"] == "swiglu":
        g, u = s["gate"].double(), s["up"].double()
        h = g * torch.special.expit(g) * u
        return [_exact_scaled(h, given=False)] + ([_exact_scaled(g), _exact_scaled(u)] if case["keep"] else [])
    g, u, dh = _exact_values(s["gate8"]), _exact_values(s["up8"]), s["dh"].double()
    sig = torch.special.expit(g)
    dg = dh * u * sig * (1 + g * torch.special.expit(-g))
    du = dh * g * sig
    return [_exact_scaled(v, given=False) for v in (dg, du, dg.t(), du.t(), (g * sig * u).t())]
