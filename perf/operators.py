"""What is measured of the microscaled 4-bit floating-point operators (f4_*).

Formats: e2m1 codes, two to a byte (low nibble first), with a scale for each
block of k: "mx" has blocks of 32 with a power-of-two scale (e8m0), "nv" blocks
of 16 with an e4m3 scale and one fp32 scale for the tensor.  The scale plane is
laid out in tiles of 128 rows x 4 blocks (512 bytes): the byte of row r, block b
is byte (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4 of tile (r // 128, b // 4).

Operators: quantisation with its inverse (a quantised tensor is returned as the
values that it stands for), the product of two 4-bit matrices, the decode GEMV
of a 4-bit matrix with bf16 activations, and the lookup of rows of a 4-bit
table.  ``own`` selects the framework's kernels; otherwise everything is
elementary torch arithmetic in fp32.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = {"mx": 32, "nv": 16}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # activations of a 64-token chunk, calibrated tensor scale: the smallest calls
        {"name": "quantize_chunk_nv", "op": "quantize", "fmt": "nv", "R": 64, "K": 2560,
         "src": "bf16", "calibrated": True},
        # weights of the up-projection, quantised once and compared with the original
        {"name": "quantize_weights_mx", "op": "quantize", "fmt": "mx", "R": 19456, "K": 2560,
         "src": "f32", "calibrated": False},
        # odd row count, scale found by the call, fp16 checkpoint
        {"name": "quantize_odd_nv", "op": "quantize", "fmt": "nv", "R": 1237, "K": 9728,
         "src": "f16", "calibrated": False},
        # token embedding of a decode batch from the tied vocabulary table
        {"name": "embed_decode_mx", "op": "embed", "fmt": "mx", "V": 151936, "K": 2560, "T": 8,
         "out": "bf16"},
        # token embedding of a prompt, padding ids among them
        {"name": "embed_prompt_nv", "op": "embed", "fmt": "nv", "V": 50257, "K": 2560, "T": 2048,
         "out": "bf16"},
        # attention output projection of one token: latency counts
        {"name": "gemv_out_mx_m1", "op": "gemv", "fmt": "mx", "N": 2560, "K": 4096, "M": 1,
         "out": "bf16"},
        # down projection, eight tokens (speculative check of a draft)
        {"name": "gemv_down_nv_m8", "op": "gemv", "fmt": "nv", "N": 2560, "K": 9728, "M": 8,
         "out": "bf16"},
        # vocabulary logits of one token in fp32: the largest stream
        {"name": "gemv_lmhead_mx_m1", "op": "gemv", "fmt": "mx", "N": 151936, "K": 2560, "M": 1,
         "out": "f32"},
        # vocabulary logits of five tokens
        {"name": "gemv_lmhead_nv_m5", "op": "gemv", "fmt": "nv", "N": 151936, "K": 2560, "M": 5,
         "out": "bf16"},
        # ragged decode batch, odd row count and a K that ends inside a tile
        {"name": "mm_ragged_nv_m33", "op": "mm", "fmt": "nv", "N": 6151, "K": 2592, "M": 33,
         "out": "f32"},
        # down projection of a short prompt
        {"name": "mm_down_mx_m256", "op": "mm", "fmt": "mx", "N": 2560, "K": 9728, "M": 256,
         "out": "bf16"},
        # up projection of a long prompt: the largest product
        {"name": "mm_up_nv_m2048", "op": "mm", "fmt": "nv", "N": 19456, "K": 2560, "M": 2048,
         "out": "bf16"},
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _extent(rng, lo, hi):
    """A reduction length: a multiple of 32 of [lo, hi]."""
    return 32 * _spread(rng, lo // 32, hi // 32)


def draw(rng):
    op = rng.choice(["quantize", "embed", "gemv", "mm"])
    fmt = rng.choice(["mx", "nv"])
    if op == "quantize":
        k = _extent(rng, 32, 16384)
        r = _spread(rng, 1, min(32768, 19456 * 2560 // k))
        return {"op": op, "fmt": fmt, "R": r, "K": k, "src": rng.choice(["bf16", "f16", "f32"]),
                "calibrated": rng.random() < 0.5}
    if op == "embed":
        k = _extent(rng, 32, 8192)
        v = _spread(rng, 1, min(151936, 151936 * 2560 // k))
        t = _spread(rng, 1, min(8192, 2048 * 2560 // k))
        return {"op": op, "fmt": fmt, "V": v, "K": k, "T": t, "out": rng.choice(["bf16", "f32"])}
    if op == "gemv":
        k = _extent(rng, 32, 32768)
        n = _spread(rng, 1, min(151936, 151936 * 2560 // k))
        return {"op": op, "fmt": fmt, "N": n, "K": k, "M": rng.randint(1, 8),
                "out": rng.choice(["bf16", "f32"])}
    k = _extent(rng, 32, 16384)
    n = _spread(rng, 1, min(32768, 19456 * 2560 // k))
    m = _spread(rng, 1, 2048)
    return {"op": op, "fmt": fmt, "N": n, "K": k, "M": m, "out": rng.choice(["bf16", "f32"])}


def _planes_bytes(rows, k, fmt):
    return rows * k // 2 + rows * (k // BLOCK[fmt])


def work(case):
    op, fmt, k = case["op"], case["fmt"], case["K"]
    if op == "quantize":  # x in, planes out; then planes in, fp32 values out
        r = case["R"]
        return {"bytes": r * k * SIZES[case["src"]] + 2 * _planes_bytes(r, k, fmt) + r * k * 4,
                "flops": 3 * r * k}
    if op == "embed":
        t = case["T"]
        return {"bytes": 8 * t + _planes_bytes(t, k, fmt) + t * k * SIZES[case["out"]],
                "flops": 2 * t * k}
    n, m = case["N"], case["M"]
    x = m * k * 2 if op == "gemv" else _planes_bytes(m, k, fmt)
    return {"bytes": _planes_bytes(n, k, fmt) + x + m * n * SIZES[case["out"]],
            "flops": 2 * m * n * k}


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _e2m1_codes(v):
    """Nearest e2m1 code of fp32 values, ties to the even code, saturating at 6."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c | (torch.signbit(v).to(torch.uint8) << 3)


def _quantize(x, fmt, g):
    """Codes (one to a byte) and block scale bytes of x [R][K] (fp32)."""
    r, k = x.shape
    b = x.view(r, k // BLOCK[fmt], BLOCK[fmt])
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    amax = torch.where(bad, torch.zeros_like(amax), amax)
    if fmt == "mx":
        # floor(log2(amax)) - 2, the largest power of two of e2m1 being 4
        e = torch.frexp(amax)[1] - 3
        e = torch.where(amax == 0, -127, e.clamp(-127, 125)).to(torch.int32)
        scales = torch.where(bad, 255, e + 127).to(torch.uint8)
        inv = ((127 - e) << 23).view(torch.float32)
    else:
        s = (amax / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        den = s.float() * g
        inv = torch.where(den == 0, torch.zeros_like(den), 1.0 / den)
        scales = torch.where(bad, 127, s.view(torch.uint8)).to(torch.uint8)
    v = torch.where(bad[..., None], torch.zeros_like(b), b * inv[..., None])
    return _e2m1_codes(v).view(r, k), scales


def _tensor_scale(x):
    """max |x| over the finite elements / (6 * 448), at least 2^-100, as fp32 [1]."""
    a = x.abs()
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax().view(1)
    return (a / torch.full_like(a, 2688.0)).clamp(min=2.0 ** -100)


def _scale_values(scales, fmt):
    """fp32 values of block scale bytes."""
    if fmt == "mx":
        b = scales.to(torch.int32)
        bits = torch.where(b == 0, 0x400000, torch.where(b == 255, 0x7FC00000, b << 23))
        return bits.to(torch.int32).view(torch.float32)
    return scales.view(torch.float8_e4m3fn).float()


def _tiled(scales):
    """Row-major scale bytes [R][blocks] -> tiles [R/128][blocks/4][512], padded with zeros."""
    r, b = scales.shape
    rt, bt = -(-r // 128), -(-b // 4)
    full = torch.zeros(rt * 128, bt * 4, dtype=torch.uint8, device=scales.device)
    full[:r, :b] = scales
    return full.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).reshape(rt, bt, 512)


def _untiled(tiles, r, b):
    rt, bt, _ = tiles.shape
    rows = tiles.view(rt, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)
    return rows[:r, :b]


def _packed(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _values(codes, scales, fmt):
    """fp32 q * s of packed codes [R][K/2] and row-major scale bytes."""
    r, half = codes.shape
    levels = torch.tensor(LEVELS + [-v for v in LEVELS], device=codes.device)
    q = torch.stack((levels[(codes & 15).int()], levels[(codes >> 4).int()]), -1)
    s = _scale_values(scales, fmt)
    return (q.view(r, s.shape[1], -1) * s[..., None]).view(r, 2 * half)


def _dense(codes, tiles, fmt):
    r, half = codes.shape
    return _values(codes, _untiled(tiles, r, 2 * half // BLOCK[fmt]).contiguous(), fmt)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, r, k, std, outliers=False):
    x = torch.randn(r, k, device=DEVICE, generator=gen) * std
    if outliers:  # one element in a hundred twenty times larger, as in real activations
        x *= 1.0 + 19.0 * (torch.rand(r, k, device=DEVICE, generator=gen) < 0.01)
    return x


def _stored(x, fmt):
    """What a program keeps of a quantised matrix: packed codes, scale tiles, tensor scale."""
    g = _tensor_scale(x) if fmt == "nv" else None
    codes, tiles = [], []
    step = 16384  # rows at a time, a multiple of the 128-row tile
    for i in range(0, x.shape[0], step):
        c, s = _quantize(x[i:i + step], fmt, g)
        codes.append(_packed(c))
        tiles.append(_tiled(s))
    return torch.cat(codes), torch.cat(tiles), g


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, fmt, k = case["op"], case["fmt"], case["K"]
    if op == "quantize":
        x = _normal(gen, case["R"], k, 1.0, outliers=True)
        x[::61] = 0.0  # padding rows
        x = x.to(TYPES[case["src"]])
        g = None
        if fmt == "nv" and case["calibrated"]:  # as calibration leaves it: now and then too small
            g = torch.full((1,), 72.0 / 2688.0, device=DEVICE)
        return {"x": x, "g": g}
    if op == "embed":
        table = _stored(_normal(gen, case["V"], k, 0.02), fmt)
        ids = torch.randint(0, case["V"], (case["T"],), device=DEVICE, generator=gen)
        ids[7::64] = -1  # padding
        return {"w": table, "ids": ids, "alpha": math.sqrt(k)}
    w = _stored(_normal(gen, case["N"], k, 0.02), fmt)
    x = _normal(gen, case["M"], k, 1.0, outliers=True).to(torch.bfloat16)
    if op == "gemv":
        return {"w": w, "x": x}
    return {"w": w, "x": _stored(x.float(), fmt)}


def prepare(case, seed):
    return {"case": dict(case), **_inputs(case, seed)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(case, state):
    import w4_quant_matmul_b200 as w4
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        codes, scales, g = w4.f4_quantize(state["x"], fmt, tensor_scale=state["g"])
        return w4.f4_dequantize(codes, scales, g, out_dtype=torch.float32)
    out = TYPES[case["out"]]
    if op == "embed":
        return w4.f4_embed(*state["w"], state["ids"], scale=state["alpha"], out_dtype=out)
    if op == "gemv":
        return w4.f4_gemv(*state["w"], state["x"], out_dtype=out)
    return w4.f4_mm(*state["w"], *state["x"], out_dtype=out)


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        x = state["x"].float()
        g = state["g"]
        if fmt == "nv" and g is None:
            g = _tensor_scale(x)
        codes, scales = _quantize(x, fmt, g)
        v = _values(_packed(codes), scales, fmt)
        return v if g is None else v * g
    out = TYPES[case["out"]]
    codes, tiles, g = state["w"]
    if op == "embed":
        ids = state["ids"]
        live = (ids >= 0) & (ids < case["V"])
        at = torch.where(live, ids, torch.zeros_like(ids))
        blocks = case["K"] // BLOCK[fmt]
        b = torch.arange(blocks, device=DEVICE)
        byte = (at % 32 * 16 + at % 128 // 32 * 4)[:, None] + b % 4
        s = tiles[(at // 128)[:, None], b // 4, byte]
        v = _values(codes[at], s, fmt)
        c = state["alpha"] if g is None else g * state["alpha"]
        return torch.where(live[:, None], v * c, torch.zeros_like(v)).to(out)
    w = _dense(codes, tiles, fmt)
    if op == "gemv":
        y = state["x"].float() @ w.t()
    else:
        xc, xt, xg = state["x"]
        y = _dense(xc, xt, fmt) @ w.t()
        g = g if g is None else g * xg
    return (y if g is None else y * g).to(out)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_matrix(codes, tiles, fmt):
    """float64 values of a stored matrix, read element by element from the format's definition."""
    r, half = codes.shape
    c = torch.empty(r, 2 * half, dtype=torch.long, device=codes.device)
    c[:, 0::2] = codes % 16
    c[:, 1::2] = codes // 16
    mag, exp, man = c % 8, c % 8 // 2, c % 2
    v = torch.where(exp == 0, man.double() * 0.5,
                    torch.exp2(exp.double() - 1.0) * (1.0 + man.double() / 2.0))
    del mag, exp, man
    v = torch.where(c >= 8, -v, v)
    del c
    nb = 2 * half // BLOCK[fmt]
    row = torch.arange(r, device=codes.device)[:, None]
    blk = torch.arange(nb, device=codes.device)[None, :]
    at = (row // 128 * tiles.shape[1] + blk // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + blk % 4
    s = tiles.reshape(-1)[at.reshape(-1)].view(r, nb).double()
    if fmt == "mx":
        s = torch.exp2(s - 127.0)
    else:  # e4m3: four exponent bits (bias 7), three mantissa bits, subnormals
        e, f = torch.floor(s / 8.0), torch.remainder(s, 8.0)
        s = torch.where(e == 0, f * 2.0 ** -9, torch.exp2(e - 7.0) * (1.0 + f / 8.0))
    v = v.view(r, nb, BLOCK[fmt])
    v *= s[..., None]
    return v.view(r, 2 * half)


def _exact_product(x, codes, tiles, fmt):
    out = []
    for i in range(0, codes.shape[0], 16384):
        w = _exact_matrix(codes[i:i + 16384], tiles[i // 128:(i + 16384) // 128], fmt)
        out.append(x @ w.t())
    return torch.cat(out, 1)


def _round_to(v, mantissa, lowest):
    """v rounded to `mantissa` fraction bits, ties to even, steps no finer than 2**lowest."""
    e = torch.frexp(v)[1] - 1
    step = torch.exp2(torch.clamp(e - mantissa, min=lowest).double())
    return torch.round(v / step) * step


def exact(case, seed):
    state = _inputs(case, seed)
    op, fmt = case["op"], case["fmt"]
    if op == "quantize":
        x = state["x"].double()
        r, k = x.shape
        b = x.view(r, k // BLOCK[fmt], BLOCK[fmt])
        amax = b.abs().amax(-1)
        g = 1.0
        if fmt == "mx":
            top = torch.frexp(amax)[1] - 1  # floor of the logarithm, for amax != 0
            s = torch.exp2(torch.clamp(top - 2, -127, 125).double())
            s = torch.where(amax == 0, torch.full_like(s, 2.0 ** -127), s)
            v = b / s[..., None]
        else:
            # the format's scales are fp32 and e4m3 numbers: their roundings are part of it
            g = state["g"].double() if state["g"] is not None else \
                (x.abs().amax() / 2688.0).clamp(min=2.0 ** -100).float().double()
            t = (amax / (g * 6.0).float().double()).float().double()
            s = _round_to(t, 3, -9).clamp(max=448.0)
            den = (s * g).float().double()
            inv = torch.where(den == 0, torch.zeros_like(den), (1.0 / den).float().double())
            v = (b * inv[..., None]).float().double()
        q = _round_to(v, 1, -1).clamp(-6.0, 6.0)
        return (q * s[..., None] * g).view(r, k)
    codes, tiles, g = state["w"]
    g = 1.0 if g is None else g.double()
    if op == "embed":
        ids = state["ids"]
        live = (ids >= 0) & (ids < case["V"])
        rows = torch.where(live, ids, torch.zeros_like(ids))
        out = torch.empty(case["T"], case["K"], dtype=torch.float64, device=DEVICE)
        for i in range(0, case["V"], 16384):
            here = (rows >= i) & (rows < i + 16384)
            if bool(here.any()):
                w = _exact_matrix(codes[i:i + 16384], tiles[i // 128:(i + 16384) // 128], fmt)
                out[here] = w[rows[here] - i]
        return torch.where(live[:, None], out * (g * state["alpha"]), torch.zeros_like(out))
    if op == "gemv":
        return _exact_product(state["x"].double(), codes, tiles, fmt) * g
    xc, xt, xg = state["x"]
    xg = 1.0 if xg is None else xg.double()
    return _exact_product(_exact_matrix(xc, xt, fmt), codes, tiles, fmt) * (g * xg)
