"""The 8-bit and mixture-of-experts operators, as cases that can be measured.

Three operators: the E4M3 quantizer with one fp32 scale per 128 values (of a
row, or a 128 x 128 tile), the matrix product of two such operands, and a whole
mixture-of-experts layer over weights in MXFP4, NVFP4 or E4M3.  ``run`` computes
them in their plain form, or with ``own`` through the package's entry points.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)          # E2M1 magnitudes, by code
BLOCK = {"mxfp4": 32, "nvfp4": 16, "f8": 128}
LARGEST_GEMM = 8192 * 13824 * 5120
LARGEST_MOE = 64 * 3 * 5120 * 1792


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token's hidden state on its way into an 8-bit projection: pure latency
        {"name": "quantize 1x5120", "op": "quantize", "rows": 1, "cols": 5120, "grain": "row"},
        # a prompt's activations before a projection
        {"name": "quantize 8192x5120", "op": "quantize", "rows": 8192, "cols": 5120, "grain": "row"},
        # a gate projection's weights, laid out once per model load or per training step
        {"name": "quantize tiles 13824x5120", "op": "quantize", "rows": 13824, "cols": 5120, "grain": "tile"},
        # decoding one token: the gate projection, bound by its weights' bytes
        {"name": "gemm 1x13824x5120", "op": "gemm", "m": 1, "n": 13824, "k": 5120, "out": "bf16"},
        # a batch of decoded tokens through a down projection with a long k
        {"name": "gemm 37x3584x18944", "op": "gemm", "m": 37, "n": 3584, "k": 18944, "out": "bf16"},
        # nothing a multiple of the tiles, the last block of k short, fp32 results
        {"name": "gemm 777x1001x4112 f32", "op": "gemm", "m": 777, "n": 1001, "k": 4112, "out": "f32"},
        # a prompt through the gate projection: bound by the tensor cores
        {"name": "gemm 8192x13824x5120", "op": "gemm", "m": 8192, "n": 13824, "k": 5120, "out": "bf16"},
        # decoding one token through small experts: latency and a few experts' bytes
        {"name": "moe nvfp4 1 token", "op": "moe", "fmt": "nvfp4", "tokens": 1, "experts": 64, "top_k": 8,
         "hidden": 2048, "inter": 1024, "normalize": True, "routed": False},
        # a few decoded tokens over 8-bit experts, probabilities not renormalised
        {"name": "moe f8 5 tokens", "op": "moe", "fmt": "f8", "tokens": 5, "experts": 32, "top_k": 4,
         "hidden": 4096, "inter": 896, "normalize": False, "routed": False},
        # the router's choice made elsewhere, some choices on another device's experts, odd sizes
        {"name": "moe nvfp4 23 tokens routed", "op": "moe", "fmt": "nvfp4", "tokens": 23, "experts": 60,
         "top_k": 4, "hidden": 1440, "inter": 1376, "normalize": True, "routed": True},
        # a decoding batch over many small experts
        {"name": "moe mxfp4 64 tokens", "op": "moe", "fmt": "mxfp4", "tokens": 64, "experts": 128, "top_k": 8,
         "hidden": 2048, "inter": 768, "normalize": True, "routed": False},
        # the widest layer: every expert's weights are read
        {"name": "moe nvfp4 64 tokens wide", "op": "moe", "fmt": "nvfp4", "tokens": 64, "experts": 64,
         "top_k": 8, "hidden": 5120, "inter": 1792, "normalize": True, "routed": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "moe", "moe"))
    if op == "quantize":
        cols = 16 * _log(rng, 8, 1184)
        return {"op": op, "rows": _log(rng, 1, max(2, 13824 * 5120 // cols)), "cols": cols,
                "grain": rng.choice(("row", "tile"))}
    if op == "gemm":
        n, k = _log(rng, 128, 18944), 16 * _log(rng, 16, 1184)
        m = _log(rng, 1, min(8192, LARGEST_GEMM // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(("bf16", "bf16", "f32"))}
    fmt = rng.choice(("mxfp4", "nvfp4", "f8"))
    unit = 128 if fmt == "f8" else 32
    while True:
        experts = _log(rng, 8, 160)
        hidden, inter = unit * _log(rng, 512 // unit, 5120 // unit), unit * _log(rng, 256 // unit, 2048 // unit)
        if 3 * experts * hidden * inter * (2 if fmt == "f8" else 1) <= LARGEST_MOE:
            return {"op": op, "fmt": fmt, "tokens": _log(rng, 1, 64), "experts": experts,
                    "top_k": rng.randint(1, 8), "hidden": hidden, "inter": inter,
                    "normalize": rng.random() < 0.5, "routed": rng.random() < 0.25}


def _experts_hit(case):
    e, k, t = case["experts"], case["top_k"], case["tokens"]
    return e * (1.0 - (1.0 - k / e) ** t)


def work(case):
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        groups = (r if case["grain"] == "row" else -(-r // 128)) * -(-c // 128)
        return {"bytes": 3 * r * c + 4 * groups, "flops": 3 * r * c}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // 128)) + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    t, h, i = case["tokens"], case["hidden"], case["inter"]
    weights = 3 * h * i
    per = {"mxfp4": 0.5 + 1 / 32, "nvfp4": 0.5 + 1 / 16, "f8": 1 + 4 / 128 ** 2}[case["fmt"]]
    route = 8 * t * case["top_k"] + (0 if case["routed"] else 2 * case["experts"] * h)
    return {"bytes": int(_experts_hit(case) * weights * per + route + 4 * t * h),
            "flops": int(2 * t * case["top_k"] * weights + (0 if case["routed"] else 2 * t * case["experts"] * h))}


# ------------------------------------------------------------------ inputs
def _activations(rows, cols, g):
    """Heavy-tailed rows with a few outlier channels, as bf16."""
    z = torch.randn((rows, cols), generator=g, device="cuda")
    chi = torch.zeros((rows, cols), device="cuda")
    for _ in range(3):
        chi += torch.randn((rows, cols), generator=g, device="cuda").square_()
    x = z / torch.sqrt(chi)
    x[:, torch.randint(0, cols, (8,), generator=g, device="cuda")] *= 20.0
    return x.to(torch.bfloat16)


def _e4m3(x, grain):
    """Codes and scales of a 2-D tensor, for prepared operands."""
    r, c = x.shape
    h = 1 if grain == "row" else 128
    p = torch.zeros((-(-r // h) * h, -(-c // 128) * 128), device="cuda")
    p[:r, :c] = x
    t = p.view(p.shape[0] // h, h, p.shape[1] // 128, 128)
    a = t.abs().amax(dim=(1, 3))
    s = torch.where(a > 0, a / torch.full_like(a, E4M3_MAX), torch.ones_like(a))
    q = (t / s[:, None, :, None]).view(p.shape)[:r, :c].contiguous()
    return q.to(torch.float8_e4m3fn), s


def _fp4(w, fmt):
    """Codes and scale bytes of a 2-D tensor, and its per-tensor scale (or None), for prepared weights."""
    b = BLOCK[fmt]
    t = w.float().view(w.shape[0], -1, b)
    a = t.abs().amax(dim=2)
    g = None
    if fmt == "mxfp4":
        e = torch.floor(torch.log2(a.clamp(min=1e-30))) - 2
        s, bytes_ = torch.exp2(e), (e + 127).to(torch.uint8)
    else:
        g = (a.max() / (6 * E4M3_MAX)).reshape(1)
        f8 = (a / (6 * g)).to(torch.float8_e4m3fn)
        s, bytes_ = f8.float() * g, f8.view(torch.uint8)
    r = t / s.clamp(min=1e-30)[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(r.abs(), edges, out_int32=True).to(torch.uint8) + 8 * (r < 0).to(torch.uint8)
    code = code.view(w.shape)
    return code[:, 0::2] | (code[:, 1::2] << 4), bytes_.contiguous(), g


def _experts(case, rows, cols, sigma, g):
    """The experts' matrices [experts * rows][cols], normal, quantized expert by expert into whole buffers."""
    fmt, n = case["fmt"], case["experts"]
    codes, scales, gscale = [], [], []
    for _ in range(n):
        w = (torch.randn((rows, cols), generator=g, device="cuda") * sigma).to(torch.bfloat16)
        c, s, one = _e4m3(w.float(), "tile") + (None,) if fmt == "f8" else _fp4(w, fmt)
        codes.append(c.view(torch.uint8))
        scales.append(s)
        gscale.append(one)
    codes = torch.cat(codes)
    return (codes.view(torch.float8_e4m3fn) if fmt == "f8" else codes, torch.cat(scales),
            torch.cat(gscale) if fmt == "nvfp4" else None)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        s["x"] = (_activations(r, c, g) if case["grain"] == "row"
                  else (torch.randn((r, c), generator=g, device="cuda") * 0.02).to(torch.bfloat16))
        return s
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = _e4m3(_activations(m, k, g).float(), "row")
        s["b"] = _e4m3((torch.randn((n, k), generator=g, device="cuda") * 0.02).to(torch.bfloat16).float(), "tile")
        return s
    t, e, h, i, k = (case[n] for n in ("tokens", "experts", "hidden", "inter", "top_k"))
    s["x"] = torch.randn((t, h), generator=g, device="cuda").to(torch.bfloat16)
    s["up"] = _experts(case, 2 * i, h, h ** -0.5, g)
    s["down"] = _experts(case, h, i, i ** -0.5, g)
    s["router"] = s["ids"] = s["weights"] = None
    if case["routed"]:
        # distinct experts per token; an eighth of the choices live elsewhere (-1)
        ids = torch.rand((t, e), generator=g, device="cuda").argsort(dim=1)[:, :k].to(torch.int32)
        gone = torch.rand((t, k), generator=g, device="cuda") < 0.125
        s["ids"] = torch.where(gone, torch.full_like(ids, -1), ids).contiguous()
        s["weights"] = torch.softmax(torch.randn((t, k), generator=g, device="cuda"), dim=1)
    else:
        s["router"] = (torch.randn((e, h), generator=g, device="cuda") * h ** -0.5).to(torch.bfloat16)
    s["workspace"] = torch.zeros((48 << 20,), dtype=torch.uint8, device="cuda")   # kept between calls
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_quantize(x, grain):
    r, c = x.shape
    h = 1 if grain == "row" else 128
    p = torch.nn.functional.pad(x.float(), (0, -c % 128, 0, -r % h))
    t = p.view(p.shape[0] // h, h, p.shape[1] // 128, 128)
    a = t.abs().amax(dim=(1, 3))
    s = torch.where(a == 0, torch.ones_like(a), a / torch.full_like(a, E4M3_MAX))     # a quotient, not a * (1 / 448)
    return (t / s[:, None, :, None]).view(p.shape)[:r, :c].to(torch.float8_e4m3fn), s


def _widen(codes, scales, rows_per_scale):
    """fp32 values of E4M3 codes under scales of 128 columns by 1 or 128 rows."""
    s = scales.repeat_interleave(rows_per_scale, 0)[:codes.shape[0]]
    return codes.float() * s.repeat_interleave(128, 1)[:, :codes.shape[1]]


def _plain_gemm(a, b, out):
    y = _widen(*a, 1) @ _widen(*b, 128).T
    return y.to(torch.bfloat16) if out == "bf16" else y


def _matrices(w, fmt, experts):
    """fp32 [experts][rows][cols] of the experts' quantized matrices."""
    codes, scales, gscale = w
    if fmt == "f8":
        return _widen(codes, scales, 128).view(experts, -1, codes.shape[1])
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")
    pairs = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), dim=-1)
    s = (torch.exp2(scales.float() - 127) if fmt == "mxfp4" else scales.view(torch.float8_e4m3fn).float())
    v = pairs.view(codes.shape[0], -1, BLOCK[fmt]) * s[:, :, None]
    v = v.view(experts, -1, 2 * codes.shape[1])
    return v if gscale is None else v * gscale.view(-1, 1, 1)


def _plain_moe(s):
    t, e, k, i = s["tokens"], s["experts"], s["top_k"], s["inter"]
    x = s["x"].float()
    if s["router"] is None:
        ids, w = s["ids"], s["weights"]
    else:
        logits = x.double() @ s["router"].double().T            # 64 bits: which expert wins a near tie
        order = torch.sort(logits, dim=1, descending=True, stable=True)
        ids = order.indices[:, :k].to(torch.int32)
        w = torch.softmax(order.values[:, :k] if s["normalize"] else order.values, dim=1)[:, :k].float()
    share = torch.zeros((t, e + 1), device="cuda")              # the last column takes the choices that are elsewhere
    share.scatter_add_(1, torch.where(ids < 0, e, ids).long(), w)
    up = _matrices(s["up"], s["fmt"], e)
    gu = torch.matmul(x, up.transpose(1, 2))                    # [e][t][2 i]
    gate = gu[:, :, :i]
    h = gate / (1 + torch.exp(-gate)) * gu[:, :, i:] * share.T[:e, :, None]
    y = torch.matmul(h, _matrices(s["down"], s["fmt"], e).transpose(1, 2)).sum(0)
    return y.to(torch.bfloat16), ids, w


def run(state):
    s = state
    if own:
        import microscaling_fp4_quantization_block_b200 as fq
        if s["op"] == "quantize":
            return fq.fp4q_f8_quantize(s["x"], s["grain"])
        if s["op"] == "gemm":
            return fq.fp4q_f8_gemm(*s["a"], *s["b"], out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)
        return fq.fp4q_moe(s["x"], s["router"], s["top_k"], s["up"], s["down"], s["fmt"], normalize=s["normalize"],
                           ids=s["ids"], weights=s["weights"], workspace=s["workspace"])
    if s["op"] == "quantize":
        return _plain_quantize(s["x"], s["grain"])
    if s["op"] == "gemm":
        return _plain_gemm(s["a"], s["b"], s["out"])
    return _plain_moe(s)


# ------------------------------------------------------------------ 64 bits
def _exact_weight(w, fmt, expert, rows):
    """One expert's matrix in 64 bits."""
    codes, scales, gscale = w
    c = codes[expert * rows:(expert + 1) * rows]
    if fmt == "f8":
        sr = rows // 128
        s = scales[expert * sr:(expert + 1) * sr].double()
        return c.double() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :c.shape[1]]
    sc = scales[expert * rows:(expert + 1) * rows]
    if fmt == "mxfp4":
        s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), sc.double() - 127)
    else:
        s = sc.view(torch.float8_e4m3fn).double() * gscale[expert].double()
    v = torch.empty((rows, 2 * c.shape[1]), dtype=torch.float64, device="cuda")
    for half in range(2):
        n = (c >> 4 if half else c & 15).long()
        exp, man = (n >> 1) & 3, (n & 1).double()
        mag = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * torch.pow(2.0, exp.double() - 1))
        v[:, half::2] = torch.where(n >= 8, -mag, mag)
    return v * s.repeat_interleave(BLOCK[fmt], 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x, tile = s["x"].double(), case["grain"] == "tile"
        out = torch.empty_like(x)
        scales = []
        for c in range(0, x.shape[1], 128):
            part = x[:, c:c + 128]
            top = part.abs().amax(dim=1)
            if tile:
                top = torch.stack([v.max() for v in top.split(128)])
            one = torch.where(top == 0, torch.ones_like(top), top / E4M3_MAX).float().double()   # held in fp32
            scales.append(one)
            each = one.repeat_interleave(128)[:x.shape[0]] if tile else one
            out[:, c:c + 128] = (part / each[:, None]).float().double()                          # the fp32 quotient
        # the nearest E4M3 value of a quotient, ties to even: 3 mantissa bits down to 2^-6, then steps of 2^-9
        step = torch.exp2(torch.floor(torch.log2(out.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(out / step) * step, torch.stack(scales, 1)
    if case["op"] == "gemm":
        (a, sa), (b, sb) = s["a"], s["b"]
        y = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        columns = torch.arange(case["n"], device="cuda") // 128
        for i, c in enumerate(range(0, case["k"], 128)):
            part = a[:, c:c + 128].double() * sa[:, i, None].double()
            y += part @ (b[:, c:c + 128].double() * sb[columns, i, None].double()).T
        return y
    x, h, i, k = s["x"].double(), case["hidden"], case["inter"], case["top_k"]
    if case["routed"]:
        ids, w = s["ids"], s["weights"].double()
    else:
        logits = x @ s["router"].double().T
        left, ids, top = logits.clone(), [], []
        for _ in range(k):                                       # the largest left, the first of equals
            best = left.max(dim=1, keepdim=True).values
            at = (left == best).int().argmax(dim=1, keepdim=True)
            ids.append(at)
            top.append(logits.gather(1, at))
            left.scatter_(1, at, -math.inf)
        ids, top = torch.cat(ids, 1).to(torch.int32), torch.cat(top, 1)
        peak = logits.max(dim=1, keepdim=True).values
        below = torch.exp((top if case["normalize"] else logits) - peak).sum(dim=1, keepdim=True)
        w = torch.exp(top - peak) / below
    y = torch.zeros((case["tokens"], h), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if token.numel():
            gu = x[token] @ _exact_weight(s["up"], case["fmt"], e, 2 * i).T
            act = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
            y.index_add_(0, token, (act @ _exact_weight(s["down"], case["fmt"], e, h).T) * w[token, slot][:, None])
    return y, ids, w
