"""The 8-bit projection path of an attention layer: what is measured.

Four operators, used together around the attention kernels of this package:

  rmsnorm_fp8                    residual addition and root-mean-square norm, the result in E4M3 with scales
  fp8_quantize                   rows (activations) or weights in E4M3 with scales
  fp8_matmul                     y = x w^T of two such matrices
  grouped_output_projection_fp8  the heads' outputs, projected by groups and then to the model dim, in E4M3

One number format throughout: E4M3 codes, and for each block of 128 columns (of one row for activations, of 128 rows for
weights) one power-of-two scale, the smallest 2^e with every magnitude of the block at most 448 2^e.

``own`` false: the plain forms, elementary torch operations in 32 bits.  ``own`` true: the package's calls.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def listed():
    return [
        # the input norm of one generated token: one row, latency alone
        {"name": "norm_token", "op": "rmsnorm_fp8", "T": 1, "d": 4096, "dtype": "bf16", "residual": True, "gain": True},
        # a ragged chunk in float32, unit gain, a last block of 16 columns
        {"name": "norm_odd_f32", "op": "rmsnorm_fp8", "T": 1001, "d": 1040, "dtype": "f32", "residual": False, "gain": False},
        # the 8192-token prefill of the benchmark
        {"name": "norm_8k", "op": "rmsnorm_fp8", "T": 8192, "d": 4096, "dtype": "bf16", "residual": True, "gain": True},
        # the 65536-token prefill
        {"name": "norm_64k", "op": "rmsnorm_fp8", "T": 65536, "d": 4096, "dtype": "bf16", "residual": True, "gain": True},
        # the attention output of a decode batch of 32, 64 heads of 512
        {"name": "quantize_decode", "op": "fp8_quantize", "rows": 32, "d": 32768, "dtype": "bf16", "block_rows": 1},
        # a weight as it is loaded: the output projection's, float32
        {"name": "quantize_weight", "op": "fp8_quantize", "rows": 4096, "d": 8192, "dtype": "f32", "block_rows": 128},
        # the indexer's query projection (64 heads of 128) of one generated token
        {"name": "matmul_token", "op": "fp8_matmul", "M": 1, "N": 8192, "K": 4096, "out": "bf16"},
        # the same for the decode batch of 32
        {"name": "matmul_decode", "op": "fp8_matmul", "M": 32, "N": 8192, "K": 4096, "out": "bf16"},
        # ragged in every direction, compression logits kept in float32
        {"name": "matmul_odd_f32", "op": "fp8_matmul", "M": 777, "N": 1111, "K": 1040, "out": "f32"},
        # the prefill of 8192 tokens
        {"name": "matmul_8k", "op": "fp8_matmul", "M": 8192, "N": 8192, "K": 4096, "out": "bf16"},
        # the grouped output projection of the decode batch
        {"name": "project_decode", "op": "grouped_output_projection_fp8", "T": 32, "H": 64, "c": 512, "g": 8, "dg": 1024, "d": 4096},
        # and of the 8192-token prefill
        {"name": "project_8k", "op": "grouped_output_projection_fp8", "T": 8192, "H": 64, "c": 512, "g": 8, "dg": 1024, "d": 4096},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rmsnorm_fp8", "fp8_quantize", "fp8_matmul", "fp8_matmul", "grouped_output_projection_fp8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rmsnorm_fp8":
        d = 16 * spread(4, 1024)
        return {"op": op, "T": min(spread(1, 65536), 65536 * 4096 // d // (2 if dtype == "f32" else 1)), "d": d,
                "dtype": dtype, "residual": rng.random() < 0.7, "gain": rng.random() < 0.7}
    if op == "fp8_quantize":
        d = 16 * spread(1, 2048)
        return {"op": op, "rows": min(spread(1, 65536), 65536 * 2048 // d), "d": d, "dtype": dtype,
                "block_rows": rng.choice([1, 128])}
    if op == "fp8_matmul":
        M, N, K = spread(1, 16384), spread(16, 16384), 16 * spread(4, 1024)
        while M * N * K > 8192 * 8192 * 4096:
            M = (M + 1) // 2
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "bf16", "f32"])}
    H, c = rng.choice([8, 16, 32, 64]), rng.choice([64, 128, 256, 512])
    g = rng.choice([n for n in (1, 2, 4, 8) if H // n * c % 128 == 0])
    return {"op": op, "T": spread(1, 8192), "H": H, "c": c, "g": g, "dg": 128 * rng.randint(1, 8), "d": spread(64, 4096)}


# ---- the format, in 32 bits ---------------------------------------------------------------------------------------


def _blocks(y, block_rows):
    """y [R, d] as [rows of blocks, block_rows, columns of blocks, 128], filled up with zeros."""
    R, d = y.shape
    br, bc = -(-R // block_rows), -(-d // 128)
    if (br * block_rows, bc * 128) != (R, d):
        y = torch.nn.functional.pad(y, (0, bc * 128 - d, 0, br * block_rows - R))
    return y.view(br, block_rows, bc, 128)


def _exponents(amax):
    """The smallest e with amax <= 448 2^e: with amax = f 2^x, f in [1/2, 1), and 448 = 7/8 2^9."""
    f, x = torch.frexp(amax)
    e = x - 9 + (f > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(min=-127)


def _quantize(y, block_rows):
    """(codes [R, d] E4M3, scales [block rows, block columns] E8M0) of a float32 y."""
    R, d = y.shape
    b = _blocks(y, block_rows)
    e = _exponents(b.abs().amax(dim=(1, 3)))
    codes = torch.ldexp(b, -e[:, None, :, None]).view(-1, b.shape[2] * 128)[:R, :d].to(E4M3)
    return codes.contiguous(), (e + 127).to(torch.uint8).view(E8M0)


def _spread(codes, scales, block_rows):
    """The float32 values that codes and scales stand for."""
    R, d = codes.shape
    e = scales.view(torch.uint8).to(torch.int32) - 127
    return torch.ldexp(_blocks(codes.to(torch.float32), block_rows), e[:, None, :, None]).view(-1, e.shape[1] * 128)[:R, :d]


def _times(x, xs, w, ws):
    return _spread(x, xs, 1) @ _spread(w, ws, 128).t()


# ---- inputs ---------------------------------------------------------------------------------------------------------


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _stream_rows(gen, rows, d, dtype):
    """Rows as a residual stream has them: N(0, 1), a few channels an order of magnitude larger."""
    s = torch.ones(d, device=DEV)
    s[torch.randint(0, d, (max(1, d // 256),), generator=gen, device=DEV)] = 12.0
    return (torch.randn((rows, d), generator=gen, device=DEV) * s).to(dtype)


def _weight(gen, rows, cols):
    return _quantize(_normal(gen, (rows, cols), torch.float32, cols ** -0.5), 128)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "rmsnorm_fp8":
        dt = _dtype(case["dtype"])
        s["x"] = _stream_rows(gen, case["T"], case["d"], dt)
        s["r"] = _stream_rows(gen, case["T"], case["d"], dt) if case["residual"] else None
        s["w"] = 1.0 + 0.2 * _normal(gen, (case["d"],), torch.float32) if case["gain"] else None
    elif op == "fp8_quantize":
        scale = 1.0 if case["block_rows"] == 1 else case["d"] ** -0.5
        s["x"] = _normal(gen, (case["rows"], case["d"]), _dtype(case["dtype"]), scale)
    elif op == "fp8_matmul":
        s["x"], s["xs"] = _quantize(_stream_rows(gen, case["M"], case["K"], torch.float32), 1)
        s["w"], s["ws"] = _weight(gen, case["N"], case["K"])
    else:
        H, c, g, dg, d = (case[k] for k in ("H", "c", "g", "dg", "d"))
        s["o"] = torch.randn((case["T"], H, c), generator=gen, device=DEV, dtype=torch.bfloat16)
        w, ws = _weight(gen, g * dg, H // g * c)
        s["wg"], s["wgs"] = w.view(g, dg, -1), ws.view(g, dg // 128, -1)
        s["wo"], s["wos"] = _weight(gen, d, g * dg)
    if own and op in ("fp8_matmul", "grouped_output_projection_fp8"):
        import long_context_attention_csa_b200 as csa

        s["work"] = csa.workspace(csa.csa_workspace_bytes(csa.CSA_OP_FP8_MATMUL, torch.bfloat16, 1, case["M"])
                                  if op == "fp8_matmul" else
                                  csa.csa_workspace_bytes(csa.CSA_OP_OUT_PROJ_FP8, torch.bfloat16, 1, case["T"],
                                                          case["H"], case["c"], case["g"] * case["dg"]))
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------


def _plain(s):
    op = s["op"]
    if op == "rmsnorm_fp8":
        h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-6)
        if s["w"] is not None:
            y = y * s["w"]
        codes, scales = _quantize(y, 1)
        return (codes, scales) if s["r"] is None else (codes, scales, h.to(s["x"].dtype))
    if op == "fp8_quantize":
        return _quantize(s["x"].float(), s["block_rows"])
    if op == "fp8_matmul":
        return _times(s["x"], s["xs"], s["w"], s["ws"]).to(_dtype(s["out"]))
    g, dg = s["g"], s["dg"]
    o, os = _quantize(s["o"].float().view(s["T"], -1), 1)
    x = _spread(o, os, 1).view(s["T"], g, -1)
    w = _spread(s["wg"].view(g * dg, -1), s["wgs"].view(g * dg // 128, -1), 128).view(g, dg, -1)
    v = torch.bmm(x.transpose(0, 1), w.transpose(1, 2)).transpose(0, 1).reshape(s["T"], g * dg)
    v, vs = _quantize(v, 1)
    return _times(v, vs, s["wo"], s["wos"]).to(torch.bfloat16)


def run(state):
    if not own:
        return _plain(state)
    import long_context_attention_csa_b200 as csa

    s = state
    if s["op"] == "rmsnorm_fp8":
        return csa.rmsnorm_fp8(s["x"], residual=s["r"], gain=s["w"], eps=1e-6)
    if s["op"] == "fp8_quantize":
        return csa.fp8_quantize(s["x"], block_rows=s["block_rows"])
    if s["op"] == "fp8_matmul":
        return csa.fp8_matmul(s["x"], s["xs"], s["w"], s["ws"], out_dtype=_dtype(s["out"]), ws=s["work"])
    return csa.grouped_output_projection_fp8(s["o"], s["wg"], s["wgs"], s["wo"], s["wos"], ws=s["work"])


def work(case):
    op = case["op"]
    if op == "rmsnorm_fp8":
        n, e = case["T"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        streams = 3 if case["residual"] else 1
        return {"bytes": n * e * streams + n + case["T"] * -(-case["d"] // 128) + 4 * case["d"] * case["gain"],
                "flops": 6 * n}
    if op == "fp8_quantize":
        n, e = case["rows"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (e + 1) + -(-case["rows"] // case["block_rows"]) * -(-case["d"] // 128), "flops": 2 * n}
    if op == "fp8_matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        return {"bytes": M * (K + kb) + N * K + -(-N // 128) * kb + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    T, H, c, g, dg, d = (case[k] for k in ("T", "H", "c", "g", "dg", "d"))
    weights = dg * H * c + d * g * dg
    return {"bytes": 2 * T * H * c + weights + weights // 16384 + 2 * T * d, "flops": 2 * T * weights}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------------


def _scale64(y, rows):
    """2^e of every element's block, spread over y [R, d] (float64), and the exponents."""
    R, d = y.shape
    nr, nc = -(-R // rows), -(-d // 128)
    full = torch.zeros((nr * rows, nc * 128), dtype=torch.float64, device=y.device)
    full[:R, :d] = y.abs()
    top = full.view(nr, rows, nc, 128).amax(dim=3).amax(dim=1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)          # log2 rounded across a border
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 0, e, torch.full_like(e, -127.0)).clamp(min=-127.0)
    return torch.exp2(e).repeat_interleave(rows, 0).repeat_interleave(128, 1)[:R, :d], torch.exp2(e)


def _e4m3_64(r):
    """The E4M3 value nearest to r (|r| <= 448), ties to even: a step of 2^(exponent - 3), exponents from -6 on."""
    a = r.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(r) * torch.round(a / step) * step


def _held64(y):
    s, _ = _scale64(y, 1)
    return _e4m3_64(y / s) * s


def _value64(codes, scales, rows):
    R, d = codes.shape
    f = torch.exp2(scales.view(torch.uint8).to(torch.float64) - 127)
    return codes.to(torch.float64) * f.repeat_interleave(rows, 0).repeat_interleave(128, 1)[:R, :d]


def exact(case, seed):
    """What run() returns, in 64 bits; where it is held in E4M3, the number before that rounding."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rmsnorm_fp8", "fp8_quantize"):
        h = s["x"].double()
        if op == "fp8_quantize":
            scale, e = _scale64(h, case["block_rows"])
            return [h / scale, e]
        if s["r"] is not None:
            h = h + s["r"].double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["d"] + 1e-6)
        if s["w"] is not None:
            y = y * s["w"].double()
        scale, e = _scale64(y, 1)
        return [y / scale, e] + ([] if s["r"] is None else [h])
    if op == "fp8_matmul":
        return _value64(s["x"], s["xs"], 1).matmul(_value64(s["w"], s["ws"], 128).t())
    T, g, dg = case["T"], case["g"], case["dg"]
    o = _held64(s["o"].double().reshape(T, -1))
    n = o.shape[1] // g
    v = torch.cat([o[:, j * n:(j + 1) * n].matmul(_value64(s["wg"][j], s["wgs"][j], 128).t()) for j in range(g)], 1)
    return _held64(v).matmul(_value64(s["wo"], s["wos"], 128).t())
