"""Measured cases of the operators around the 8-bit products of a block: dropout,
the norms before and after a block with its gate and residual scale, and the
8-bit product with bias, activation, dropout and residual in its epilogue.

  dropout    out = residual + alpha m x. The mask m is not stored: m(i, j) is
             [u(i, j) >= t] / (1 - t / 65536), t = round(65536 p), and u(i, j) the
             16-bit half number j % 8 (the low half of a word first) of
             Philox4x32-10 at counter (j / 8, i, offset low, offset high) and key
             (seed low, seed high) (Salmon, Moraes, Dror, Shaw: Parallel random
             numbers: as easy as 1, 2, 3; SC 2011)
  norm       p = norm(y) post_w + post_b, or y;  r = x + alpha gate m p;
             n = norm(r) pre_w + pre_b in 16 bits and / or in 8
  norm_bwd   gradients of x, y, the weights and the gate, from those of n and r
  mm         z = A B^T + bias;  C = residual + alpha m act(z) in C's type and / or
             in 8 bits; z is kept if wanted
  mm_bwd     C = alpha m (A B^T) act'(z), and the bias's gradient in C's type, its
             column sums before C's rounding

A block-scaled 8-bit matrix holds e4m3 codes (torch.float8_e4m3fn) and, for
every 128 values along a row (or every 128 x 128 block of a weight), a power-of-two
scale (torch.float8_e8m0fnu), the smallest that brings the block's largest
magnitude to 448 or less. `run` gives codes and scales as torch's 8-bit float
types, so that what is compared are the values they stand for.
"""
import math

import torch

own = False

BLK = 128
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # the output gradient of one rank's shard (11008 / 8 columns) through a block's dropout: the backward pass
        {"name": "dropout_shard", "op": "dropout", "rows": 1001, "cols": 1376, "dtype": "fp16", "p": 0.1, "residual": False},
        # a training batch's block output, dropped out and added to the residual stream
        {"name": "dropout_train", "op": "dropout", "rows": 8192, "cols": 11008, "dtype": "bf16", "p": 0.1, "residual": True},
        # decoding one token: the block's output is added to the stream, and the norm goes to the next product in 8 bits
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "fp16", "stream": "fp16", "kind": "rms",
         "y": True, "post": False, "gate": 0, "p": 0.0, "bias": False, "out": "8", "stats": False},
        # training: norms on both sides of the block, its gate and dropout, a 32-bit stream, statistics kept
        {"name": "norm_train", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16", "stream": "fp32", "kind": "rms",
         "y": True, "post": True, "gate": 8192, "p": 0.1, "bias": False, "out": "plain+8", "stats": True},
        # a ragged batch with an odd width, layer norms, a gate for every sequence of 129 rows
        {"name": "norm_ragged", "op": "norm", "rows": 1023, "cols": 4093, "dtype": "fp16", "stream": "fp16", "kind": "layer",
         "y": True, "post": False, "gate": 129, "p": 0.0, "bias": True, "out": "plain", "stats": True},
        # the backward pass of norm_train's operator at half the rows
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 4096, "cols": 4096, "dtype": "bf16", "stream": "fp32", "kind": "rms",
         "y": True, "post": True, "gate": 4096, "p": 0.1, "bias": False},
        # few ragged rows of a shard, layer norm with biases, a gate for every 100 rows
        {"name": "norm_bwd_ragged", "op": "norm_bwd", "rows": 333, "cols": 1376, "dtype": "fp16", "stream": "fp16",
         "kind": "layer", "y": True, "post": True, "gate": 100, "p": 0.0, "bias": True},
        # decoding one token through the up projection of an ungated layer: the weight's bytes
        {"name": "mm_token", "op": "mm", "M": 1, "N": 11008, "K": 4096, "dtype": "fp16", "act": "gelu", "bias": True,
         "residual": False, "p": 0.0, "out": "plain", "z": False},
        # a training step's up projection: z kept for the backward pass, the activation as the next product's operand
        {"name": "mm_up_train", "op": "mm", "M": 8192, "N": 11008, "K": 4096, "dtype": "bf16", "act": "gelu_tanh", "bias": True,
         "residual": False, "p": 0.0, "out": "8", "z": True},
        # its down projection with dropout, added to the residual stream
        {"name": "mm_down_train", "op": "mm", "M": 4096, "N": 4096, "K": 11008, "dtype": "bf16", "act": "none", "bias": True,
         "residual": True, "p": 0.1, "out": "plain", "z": False},
        # a small serving batch's up projection straight to 8 bits, odd rows
        {"name": "mm_batch", "op": "mm", "M": 33, "N": 11008, "K": 4096, "dtype": "bf16", "act": "silu", "bias": True,
         "residual": False, "p": 0.0, "out": "8", "z": False},
        # the gradient through the activation of mm_up_train's kind, ragged rows, and the bias's gradient
        {"name": "mm_bwd_train", "op": "mm_bwd", "M": 4095, "N": 11008, "K": 4096, "dtype": "bf16", "act": "gelu_tanh", "p": 0.1},
    ]


def _size(rng, lo, hi):
    """A length between lo and hi, spread over its logarithm; about half of them multiples of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 32:
        v -= v % 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["dropout", "norm", "norm", "norm_bwd", "mm", "mm", "mm_bwd"])
    dtype = rng.choice(["fp16", "bf16"])
    p = rng.choice([0.0, 0.1, round(rng.uniform(0.01, 0.6), 3)])
    if op == "dropout":
        return {"op": op, "rows": _size(rng, 1, 8192), "cols": _size(rng, 64, 11008), "dtype": rng.choice(list(TYPES)),
                "p": max(p, 0.05), "residual": rng.random() < 0.5}
    if op in ("norm", "norm_bwd"):
        rows, y = _size(rng, 1, 8192 if op == "norm" else 4096), rng.random() < 0.8
        case = {"op": op, "rows": rows, "cols": _size(rng, 64, 8192 if op == "norm" else 4096), "dtype": dtype,
                "stream": rng.choice([dtype, "fp32"]), "kind": rng.choice(["rms", "rms", "layer"]), "y": y,
                "post": y and rng.random() < 0.5, "gate": rng.choice([0, rows, _size(rng, min(rows, 48), rows)]) if y else 0,
                "p": p if y else 0.0, "bias": rng.random() < 0.4}
        if op == "norm":
            case["out"] = rng.choice(["plain", "8", "plain+8"])
            case["stats"] = rng.random() < 0.5
        return case
    M, N, K = _size(rng, 1, 8192), _size(rng, 64, 11008), _size(rng, 64, 11008)
    while M * N * K > 4096 * 11008 * 4096:
        M, N, K = (max(64, 3 * v // 4) for v in (M, N, K))
    case = {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(["fp16", "bf16", "bf16", "fp32"]),
            "act": rng.choice(["relu", "gelu", "gelu_tanh", "silu"]), "p": p}
    if op == "mm":
        case["act"] = rng.choice(["none", case["act"]])
        case["residual"], case["bias"] = rng.random() < 0.4, rng.random() < 0.7
        case["out"] = rng.choice(["plain", "8", "plain+8"])
        case["z"] = case["act"] != "none" and rng.random() < 0.5
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
    """Memory of a block-scaled matrix: rows of codes start at multiples of 16 bytes (of 128 beyond 512 columns), rows of
    scales at multiples of 4."""
    unit = 128 if cols > 512 else 16
    ld, ls = -(-cols // unit) * unit, -(-(-(-cols // BLK)) // 4) * 4
    codes = torch.zeros((rows, ld), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((-(-rows // block), ls), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    return codes[:, :cols], scales[:, :-(-cols // BLK)]


def _made8(x, block=1):
    q, s = _blank8(x.shape[0], x.shape[1], block)
    codes, scales = _quantized(x, block)
    q.copy_(codes)
    s.copy_(scales)
    return q, s


def _groups(case):
    return -(-case["rows"] // case["gate"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "key": ((seed * 0x9E3779B97F4A7C15 + 0x1234567) % 2 ** 64, (seed * 0xD1B54A32D192ED03 + 7) % 2 ** 64)}
    op, dt = case["op"], TYPES[case["dtype"]]
    fp8 = {}
    if op == "dropout":
        r, c = case["rows"], case["cols"]
        s["alpha"] = 1.0
        s["x"] = _activations(r, c, gen).to(dt)
        s["residual"] = _activations(r, c, gen).to(dt) if case["residual"] else None
        s["out"] = torch.empty((r, c), dtype=dt, device="cuda")
    elif op in ("norm", "norm_bwd"):
        r, c, st = case["rows"], case["cols"], TYPES[case["stream"]]
        s["alpha"] = 0.5 if case["y"] else 1.0
        for side, wanted in (("pre", True), ("post", case["post"])):
            s[side + "_w"] = (1.0 + 0.1 * _normal((c,), gen)).to(dt) if wanted else None
            s[side + "_b"] = (0.1 * _normal((c,), gen)).to(dt) if wanted and case["bias"] else None
        s["gate"] = (0.5 * _normal((_groups(case), c), gen)).to(dt) if case["gate"] else None
        s["y"] = _activations(r, c, gen).to(dt) if case["y"] else None
        if op == "norm":
            s["x"] = _activations(r, c, gen).to(st)
            s["r"] = torch.empty((r, c), dtype=st, device="cuda") if case["y"] else None
            s["n"] = torch.empty((r, c), dtype=dt, device="cuda") if "plain" in case["out"] else None
            s["q"] = _blank8(r, c) if "8" in case["out"] else None
            s["stats"] = torch.empty((r, 4), dtype=torch.float32, device="cuda") if case["stats"] else None
            fp8 = {"q": 1}
        else:
            s["r"] = _activations(r, c, gen).to(st)
            s["dn"] = (_activations(r, c, gen) / 64).to(dt)
            s["dr"] = (_activations(r, c, gen) / 64).to(st)
            s["stats"] = torch.cat([_statistics(s["y"], case["kind"]) if case["post"] else torch.zeros((r, 2), device="cuda"),
                                    _statistics(s["r"], case["kind"])], 1)
            s["dx"] = torch.empty((r, c), dtype=st, device="cuda")
            s["dy"] = torch.empty((r, c), dtype=dt, device="cuda") if case["y"] else None
            for k in ("pre_w", "pre_b", "post_w", "post_b", "gate"):
                s["d" + k] = None if s[k] is None else torch.empty(s[k].shape, dtype=torch.float32, device="cuda")
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["alpha"] = 0.5 if case.get("residual") else 1.0
        a = _activations(M, K, gen)
        s["A"] = _made8(a / 64 if op == "mm_bwd" else a)
        s["B"] = _made8(_normal((N, K), gen) / math.sqrt(K), BLK)
        if op == "mm":
            s["bias"] = (0.1 * _normal((N,), gen)).to(dt) if case["bias"] else None
            s["residual"] = _activations(M, N, gen).to(dt) if case["residual"] else None
            s["z"] = torch.empty((M, N), dtype=dt, device="cuda") if case["z"] else None
            s["C"] = torch.empty((M, N), dtype=dt, device="cuda") if "plain" in case["out"] else None
            s["q"] = _blank8(M, N) if "8" in case["out"] else None
        else:
            s["z"] = _activations(M, N, gen).to(dt)
            s["C"] = torch.empty((M, N), dtype=dt, device="cuda")
            s["dbias"] = torch.empty((N,), dtype=dt, device="cuda")
        fp8 = {"A": 1, "B": BLK, "q": 1}
    if own:  # the handles that a program keeps: of its block-scaled buffers, of the generator's place, of a norm's parameters
        import gemm_collective_tile_amd as il
        s["il"] = il
        s["m"] = {k: None if s.get(k) is None else il.Fp8(*s[k], block=b) for k, b in fp8.items()}
        s["drop"] = il.Dropout(case["p"], *s["key"]) if case["p"] > 0 else None
        if op in ("norm", "norm_bwd"):
            s["norm"] = il.BlockNorm(kind=case["kind"], eps=EPS, pre_w=s["pre_w"], pre_b=s["pre_b"], post=case["post"],
                                     post_w=s["post_w"], post_b=s["post_b"], gate=s["gate"],
                                     rows_per_gate=case["gate"], alpha=s["alpha"], dropout=s["drop"])
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


def _mask(rows, cols, p, key):
    """The dropout factors (rows, cols): 0, or 1 / (1 - p) at p's nearest multiple of 2^-16. Words are kept in 64-bit
    integers; a product of two of them wraps, its low and high halves are what the generator asks for."""
    low = 0xFFFFFFFF
    seed, offset = key
    c0 = torch.arange(-(-cols // 8), device="cuda", dtype=torch.int64)[None, :].expand(rows, -1)
    c1 = torch.arange(rows, device="cuda", dtype=torch.int64)[:, None].expand_as(c0)
    c2, c3 = torch.full_like(c1, offset & low), torch.full_like(c1, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    u = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], -1)
    t = round(65536 * p)
    return (u.reshape(rows, -1)[:, :cols] >= t).float() * (65536.0 / (65536 - t))


def _statistics(v, kind):
    """(mean, 1 / sqrt(variance + eps)) of every row in 32 bits; mean 0 for the root-mean-square norm."""
    v = v.float()
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    return torch.cat([mean, 1.0 / torch.sqrt((v - mean).square().mean(1, keepdim=True) + EPS)], 1)


def _affine(v, w, b):
    v = v * w.float()
    return v if b is None else v + b.float()


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":  # z s(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3)
        k = 2.0 * math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-k * (z + 0.044715 * z * z * z)))
        return s + z * s * (1.0 - s) * k * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain_norm(s, case):
    stat = torch.zeros((case["rows"], 4), dtype=torch.float32, device="cuda")
    r = s["x"].float()
    if case["y"]:
        p = s["y"].float()
        if case["post"]:
            stat[:, :2] = _statistics(p, case["kind"])
            p = _affine((p - stat[:, :1]) * stat[:, 1:2], s["post_w"], s["post_b"])
        if case["p"] > 0:
            p = p * _mask(*p.shape, case["p"], s["key"])
        if case["gate"]:
            p = p * s["gate"].float().repeat_interleave(case["gate"], 0)[:case["rows"]]
        r = r + s["alpha"] * p
    stat[:, 2:] = _statistics(r, case["kind"])
    n = _affine((r - stat[:, 2:3]) * stat[:, 3:], s["pre_w"], s["pre_b"])
    return {"r": r.to(TYPES[case["stream"]]) if case["y"] else None,
            "n": n.to(TYPES[case["dtype"]]) if "plain" in case["out"] else None,
            "q": _quantized(n) if "8" in case["out"] else None, "stats": stat if case["stats"] else None}


def _by_group(v, every):
    """Sums over each `every` rows."""
    g = -(-v.shape[0] // every)
    whole = torch.zeros((g * every, v.shape[1]), dtype=v.dtype, device=v.device)
    whole[:v.shape[0]] = v
    return whole.reshape(g, every, -1).sum(1)


def _through_norm(d, hat, rstd, kind):
    """The gradient of v from that of hat = (v - mean) rstd."""
    g = d - hat * (d * hat).mean(1, keepdim=True)
    return rstd * (g - d.mean(1, keepdim=True) if kind == "layer" else g)


def _plain_norm_bwd(s, case):
    st = s["stats"]
    hat, dn = (s["r"].float() - st[:, 2:3]) * st[:, 3:], s["dn"].float()
    out = {"dpre_w": (dn * hat).sum(0), "dpre_b": dn.sum(0) if case["bias"] else None}
    t = s["dr"].float() + _through_norm(dn * s["pre_w"].float(), hat, st[:, 3:], case["kind"])
    out["dx"] = t.to(TYPES[case["stream"]])
    if not case["y"]:
        return out
    d = s["alpha"] * t
    if case["p"] > 0:
        d = d * _mask(*d.shape, case["p"], s["key"])
    p = s["y"].float()
    if case["post"]:
        hat = (p - st[:, :1]) * st[:, 1:2]
        p = _affine(hat, s["post_w"], s["post_b"])
    if case["gate"]:
        out["dgate"] = _by_group(d * p, case["gate"])
        d = d * s["gate"].float().repeat_interleave(case["gate"], 0)[:case["rows"]]
    if case["post"]:
        out["dpost_w"], out["dpost_b"] = (d * hat).sum(0), d.sum(0) if case["bias"] else None
        d = _through_norm(d * s["post_w"].float(), hat, st[:, 1:2], case["kind"])
    out["dy"] = d.to(TYPES[case["dtype"]])
    return out


def _plain(s):
    case = s["case"]
    op, dt = case["op"], TYPES[case["dtype"]]
    if op == "dropout":
        v = s["alpha"] * s["x"].float() * _mask(case["rows"], case["cols"], case["p"], s["key"])
        return (v if s["residual"] is None else v + s["residual"].float()).to(dt)
    if op == "norm":
        return _plain_norm(s, case)
    if op == "norm_bwd":
        return _plain_norm_bwd(s, case)
    v = torch.matmul(_values(s["A"]), _values(s["B"], BLK).t())
    m = _mask(case["M"], case["N"], case["p"], s["key"]) if case["p"] > 0 else 1.0
    if op == "mm_bwd":
        v = s["alpha"] * m * v * _act_slope(s["z"].float(), case["act"])
        return {"C": v.to(dt), "dbias": v.sum(0).to(dt)}
    z = v if s["bias"] is None else v + s["bias"].float()
    c = s["alpha"] * m * _act(z, case["act"])
    if s["residual"] is not None:
        c = c + s["residual"].float()
    return {"C": c.to(dt) if "plain" in case["out"] else None, "q": _quantized(c) if "8" in case["out"] else None,
            "z": z.to(dt) if case["z"] else None}


def run(state):
    if not own:
        return _plain(state)
    s, il, case = state, state["il"], state["case"]
    if case["op"] == "dropout":
        il.iris_dropout(s["out"], s["x"], s["drop"], residual=s["residual"], alpha=s["alpha"])
        return s["out"]
    if case["op"] == "norm":
        il.iris_block_norm(s["x"], s["norm"], y=s["y"], r=s["r"], n=s["n"], q=s["m"]["q"], stats=s["stats"])
        return {k: s[k] for k in ("r", "n", "q", "stats")}
    if case["op"] == "norm_bwd":
        il.iris_block_norm_bwd(s["dx"], s["r"], s["stats"], s["norm"], dn=s["dn"], dr=s["dr"], y=s["y"], dy=s["dy"],
                               dpre_w=s["dpre_w"], dpre_b=s["dpre_b"], dpost_w=s["dpost_w"], dpost_b=s["dpost_b"],
                               dgate=s["dgate"])
        return {k: s[k] for k in ("dx", "dy", "dpre_w", "dpre_b", "dpost_w", "dpost_b", "dgate")}
    if case["op"] == "mm":
        il.iris_fp8_mm_act(s["C"], s["m"]["A"], s["m"]["B"], act=case["act"], bias=s["bias"], z=s["z"],
                           residual=s["residual"], alpha=s["alpha"], dropout=s["drop"], q=s["m"]["q"],
                           dtype=TYPES[case["dtype"]])
        return {k: s[k] for k in ("C", "q", "z")}
    il.iris_fp8_mm_act_bwd(s["C"], s["m"]["A"], s["m"]["B"], s["z"], act=case["act"], alpha=s["alpha"], dropout=s["drop"],
                           dbias=s["dbias"])
    return {"C": s["C"], "dbias": s["dbias"]}


# ------------------------------------------------------- work, exact results

def _bytes8(rows, cols, block=1):
    return rows * cols + -(-rows // block) * -(-cols // BLK)


def work(case):
    op, size = case["op"], TYPES[case["dtype"]].itemsize
    if op == "dropout":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * size * (3 if case["residual"] else 2), "flops": 3 * r * c}
    if op in ("norm", "norm_bwd"):
        r, c, st = case["rows"], case["cols"], TYPES[case["stream"]].itemsize
        params = c * size * (1 + case["post"]) * (1 + case["bias"]) + (_groups(case) * c * size if case["gate"] else 0)
        if op == "norm":
            b = r * c * st * (2 if case["y"] else 1) + (r * c * size if case["y"] else 0) + params
            b += (r * c * size if "plain" in case["out"] else 0) + (_bytes8(r, c) if "8" in case["out"] else 0)
            return {"bytes": b + (16 * r if case["stats"] else 0), "flops": 12 * r * c}
        b = r * c * (3 * st + size) + 16 * r + params * (1 + 4 / size)
        return {"bytes": b + (2 * r * c * size if case["y"] else 0), "flops": 30 * r * c}
    M, N, K = case["M"], case["N"], case["K"]
    b = _bytes8(M, K) + _bytes8(N, K, BLK)
    if op == "mm_bwd":
        return {"bytes": b + 2 * M * N * size + N * size, "flops": 2 * M * N * K}
    b += (N * size if case["bias"] else 0) + M * N * size * (case["residual"] + case["z"] + ("plain" in case["out"]))
    return {"bytes": b + (_bytes8(M, N) if "8" in case["out"] else 0), "flops": 2 * M * N * K}


def _exact_scaled(x):
    """x / scale before the rounding to 8 bits, as 64-bit values: how far a code is from it is its rounding, half an e4m3
    step at most. The scales of computed values have no exact value: at a largest magnitude within rounding of 448 times
    a power of two, either neighbour is right."""
    rows, cols = x.shape
    nb = -(-cols // BLK)
    wide = torch.nn.functional.pad(x.abs(), (0, nb * BLK - cols)).reshape(rows, nb, BLK).max(dim=2).values
    e = torch.ceil(torch.log2(torch.where(wide > 0, wide, torch.full_like(wide, 448.0)) / 448.0)).clamp(-126, 127)
    return x / torch.pow(torch.full_like(e, 2.0), e).repeat_interleave(BLK, 1)[:, :cols], None


def _exact_values(q, block=1):
    codes, scales = q
    rows, cols = codes.shape
    return codes.double() * scales.double().repeat_interleave(block, 0)[:rows].repeat_interleave(BLK, 1)[:, :cols]


def _exact_mask(rows, cols, p, key):
    """The mask from the generator's definition, its 32 x 32-bit products in halves of 16 bits so that none exceeds 2^34,
    and a table of which half of which word a column takes."""
    def high_low(x, m):
        xl, xh, ml, mh = x & 0xFFFF, x >> 16, m & 0xFFFF, m >> 16
        mid = (xl * ml >> 16) + (xh * ml & 0xFFFF) + (xl * mh & 0xFFFF)
        return xh * mh + (xh * ml >> 16) + (xl * mh >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) | (xl * ml & 0xFFFF)

    n = -(-cols // 8)
    ctr = [torch.arange(n, device="cuda").repeat(rows), torch.arange(rows, device="cuda").repeat_interleave(n)]
    ctr += [torch.full_like(ctr[0], key[1] % 2 ** 32), torch.full_like(ctr[0], key[1] // 2 ** 32)]
    for i in range(10):
        k = [(key[0] + i * 0x9E3779B9) % 2 ** 32, (key[0] // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32]
        h0, l0 = high_low(ctr[0], 0xD2511F53)
        h1, l1 = high_low(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ k[0], l1, h0 ^ ctr[3] ^ k[1], l0]
    t = round(65536 * p)
    keep = torch.zeros((rows, n, 8), dtype=torch.float64, device="cuda")
    for j in range(8):
        keep[:, :, j] = ((ctr[j // 2] // 2 ** (16 * (j % 2)) % 65536) >= t).reshape(rows, n).double()
    return keep.reshape(rows, 8 * n)[:, :cols] / (1 - t / 65536)


def _exact_stats(v, kind):
    mean = v.mean(1) if kind == "layer" else torch.zeros_like(v[:, 0])
    return mean, (((v - mean[:, None]) ** 2).mean(1) + EPS) ** -0.5


def _exact_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if act == "silu" else z


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op, alpha = case["op"], s["alpha"]
    shape = (case["M"], case["N"]) if "M" in case else (case["rows"], case["cols"])
    m = _exact_mask(*shape, case["p"], s["key"]) if case["p"] > 0 else torch.ones((1, 1), dtype=torch.float64, device="cuda")
    if op == "dropout":
        return alpha * m * d["x"] + (0 if d["residual"] is None else d["residual"])
    if op in ("mm", "mm_bwd"):
        v = _exact_values(s["A"]) @ _exact_values(s["B"], BLK).t().contiguous()
        if op == "mm":
            z = v if d["bias"] is None else v + d["bias"]
            c = alpha * m * _exact_act(z, case["act"]) + (0 if d["residual"] is None else d["residual"])
            return {"C": c if "plain" in case["out"] else None, "q": _exact_scaled(c) if "8" in case["out"] else None,
                    "z": z if case["z"] else None}
        with torch.enable_grad():  # act' from torch's own derivative of the 64-bit function
            z = d["z"].requires_grad_()
            slope = torch.autograd.grad(_exact_act(z, case["act"]).sum(), z)[0]
        c = alpha * m * v * slope
        return {"C": c, "dbias": c.sum(0)}
    one = torch.ones((1, case["cols"]), dtype=torch.float64, device="cuda")
    zero = torch.zeros_like(one)

    def forward(x, y, pre_w, pre_b, post_w, post_b, gate, stats=None):
        """r, n and the statistics (mean and rstd of y and of r)."""
        p, sy = y, (torch.zeros_like(x[:, 0]),) * 2
        if case["post"]:
            sy = _exact_stats(y, case["kind"])
            p = (y - sy[0][:, None]) * sy[1][:, None] * post_w + post_b
        r = x if y is None else x + alpha * gate * m * p
        sr = _exact_stats(r, case["kind"])
        return r, (r - sr[0][:, None]) * sr[1][:, None] * pre_w + pre_b, torch.stack([*sy, *sr], 1)

    which = torch.arange(case["rows"], device="cuda") // max(1, case["gate"])
    wide = {k: v if d[k] is None else d[k].reshape(1, -1)
            for k, v in (("pre_w", one), ("pre_b", zero), ("post_w", one), ("post_b", zero))}
    gate = one if d["gate"] is None else d["gate"][which]
    if op == "norm":
        r, n, stats = forward(d["x"], d["y"], wide["pre_w"], wide["pre_b"], wide["post_w"], wide["post_b"], gate)
        return {"r": r if case["y"] else None, "n": n if "plain" in case["out"] else None,
                "q": _exact_scaled(n) if "8" in case["out"] else None, "stats": stats if case["stats"] else None}
    # The backward pass, given r and the statistics as they are: a norm v -> hat = (v - mean) rstd has the Jacobian
    # rstd (1 - 1 1^T / n - hat hat^T / n), without its middle term for the root-mean-square norm.
    def pull(g, v, mean, rstd):
        hat = (v - mean) * rstd
        centre = g.sum(1, keepdim=True) if case["kind"] == "layer" else 0
        return hat, rstd * (g - (centre + hat * (hat * g).sum(1, keepdim=True)) / g.shape[1])

    mu_y, rho_y, mu_r, rho_r = (d["stats"][:, i:i + 1] for i in range(4))
    hat, g = pull(d["dn"] * wide["pre_w"], d["r"], mu_r, rho_r)
    t = d["dr"] + g
    out = {"dx": t, "dpre_w": (d["dn"] * hat).sum(0), "dpre_b": d["dn"].sum(0) if case["bias"] else None}
    if not case["y"]:
        return out
    dp = alpha * gate * m * t
    p = d["y"]
    if case["post"]:
        hat, out["dy"] = pull(dp * wide["post_w"], d["y"], mu_y, rho_y)
        p = hat * wide["post_w"] + wide["post_b"]
        out["dpost_w"], out["dpost_b"] = (dp * hat).sum(0), dp.sum(0) if case["bias"] else None
    else:
        out["dy"] = dp
    if case["gate"]:
        out["dgate"] = torch.zeros_like(d["gate"]).index_add_(0, which, alpha * m * t * p)
    return out
