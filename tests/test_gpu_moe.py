"""The mixture-of-experts layer (fp4q_moe) over MXFP4, NVFP4 and E4M3 experts,
against the layer in 64 bits on the codes and scales that it reads.

Bars (u = 2^-24, s(.) sums of magnitudes):
- a logit differs from the exact one by at most d = (hidden / 32 + 8) u s(x r):
  256 / 8 products a lane, then five additions.  The chosen experts must be the
  top_k up to 2 d, in descending order up to 2 d; equal router rows give equal
  logits and the lower expert.  A weight exp(l_j - l_max) / sum differs by a
  factor of 1 + 4 d (two logits above, two below) and 2^-20 for expf and the sum.
- gate and up: E = (hidden / 64 + 24) u s(W x) + 2^-32 s(W) max|x|: each of the
  eight slices of k adds 16 products with one rounding, or truncation (2 u); a
  product's own alignment, scales and the slices take at most 24 more; x as fp16
  under its row's power of two is off by at most half of 2^-24 where the row's
  largest value is at least 2^7.
- h = silu(g) u has |silu'| <= 1.1 and is held as fp16: 11 significant bits, so
  its values lie 2^-10 of their power of two apart and rounding moves one by at
  most half of that, 2^-11 of itself; brought to the row's power a value may
  lose all below 2^-24 of the row's largest: Eh = 1.1 Eg (|u| + Eu) +
  |silu(g)| Eu + (2^-11 + 2^-20) |h| + 2^-24 max|h|.
- y: s(w D Eh) + (inter / 64 + 24 + top_k) u s(w D h) + half an ulp of bf16,
  with the weights the call returned.
"""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import microscaling_fp4_quantization_block_b200 as m
    m.lib()
    return m


def experts_of(fq, fmt, experts, rows, cols, sigma, seed, per_expert=False):
    """(codes, scales, gscale) of experts * rows Gaussian rows."""
    w = workloads.gaussian_bf16(experts * rows, cols, sigma, seed, device="cuda")
    if fmt == "f8":
        return fq.fp4q_f8_quantize(w, "tile")
    if fmt == "mxfp4":
        c, s, _ = fq.fp4q_quantize(w, "mxfp4", 32)
        return c, s, None
    if per_expert:
        parts = [fq.fp4q_quantize(w[e * rows:(e + 1) * rows] * (1 + e % 3), "nvfp4", 16, 0, "compute")
                 for e in range(experts)]
        return tuple(torch.cat([p[i] for p in parts]) for i in range(3))
    return fq.fp4q_quantize(w, "nvfp4", 16, 0, "compute")


def decode(w, fmt, experts):
    """float64 [experts][rows][cols] on the CPU."""
    codes, scales, g = (w[0], w[1], w[2] if len(w) > 2 else None)
    if fmt == "f8":
        v = codes.cpu().float().double()
        s = scales.cpu().double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return (v * s).view(experts, -1, v.shape[1])
    c = codes.cpu()
    n = torch.stack((c & 15, c >> 4), -1).view(c.shape[0], -1).long()
    v = GRID[n & 7] * torch.where(n >= 8, -1.0, 1.0).double()
    sc = scales.cpu()
    s = torch.exp2(sc.double() - 127) if fmt == "mxfp4" else sc.view(torch.float8_e4m3fn).float().double()
    v = (v * s.repeat_interleave(v.shape[1] // s.shape[1], 1)).view(experts, -1, v.shape[1])
    return v if g is None else v * g.cpu().double().view(-1, 1, 1)


def top_of(v):
    return v.abs().amax(1, keepdim=True)


def layer64(x, up, down, ids, weights):
    """y, and how far a result may be from it."""
    x, ids, w = x.cpu().double(), ids.cpu().long(), weights.cpu().double()
    y = torch.zeros((x.shape[0], down.shape[1]), dtype=torch.float64)
    far = torch.zeros_like(y)
    hidden, inter, top_k = x.shape[1], down.shape[2], ids.shape[1]
    for e in range(up.shape[0]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if not token.numel():
            continue
        xe, W, D, we = x[token], up[e], down[e], w[token, slot][:, None]
        v = xe @ W.T
        ev = (hidden / 64 + 24) * U * (xe.abs() @ W.abs().T) + 2.0 ** -32 * top_of(xe) * W.abs().sum(1)
        g, u, eg, eu = v[:, :inter], v[:, inter:], ev[:, :inter], ev[:, inter:]
        silu = g * torch.sigmoid(g)
        h = silu * u
        eh = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (2.0 ** -11 + 2.0 ** -20) * h.abs() + 2.0 ** -24 * top_of(h)
        y.index_add_(0, token, (h @ D.T) * we)
        far.index_add_(0, token, (eh @ D.abs().T + (inter / 64 + 24 + top_k) * U * ((h.abs() + eh) @ D.abs().T))
                       * we.abs())
    half = torch.finfo(torch.bfloat16).eps / 2
    return y, far * (1 + half) + half * y.abs()


def check_y(y, x, up, down, ids, weights):
    want, tol = layer64(x, up, down, ids, weights)
    err = (y.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300)).max())
    # and not merely inside worst-case sums: far below them in the mean
    assert float(err.norm()) <= 2.0 ** -8 * float(want.norm()) + 1e-30


def check_route(ids, weights, x, router, top_k, normalize):
    x, r = x.cpu().double(), router.cpu().double()
    l = x @ r.T
    d = (x.shape[1] / 32 + 8) * U * (x.abs() @ r.abs().T).amax(1, keepdim=True)
    ids = ids.cpu().long()
    assert bool(((ids >= 0) & (ids < r.shape[0])).all())
    assert all(len(set(row)) == top_k for row in ids.tolist())
    top = l.gather(1, ids)
    best = l.sort(dim=1, descending=True).values[:, :top_k]
    assert bool(((top - best).abs() <= 2 * d).all())
    peak = top[:, :1]
    below = torch.exp((top if normalize else l) - peak).sum(1, keepdim=True)
    want = torch.exp(top - peak) / below
    assert bool(((weights.cpu().double() - want).abs() <= want * (4 * d + 2.0 ** -20)).all())


CASES = [(1, 8, 2, 256, 128), (3, 5, 5, 128, 384), (7, 60, 4, 1440, 160), (64, 16, 8, 512, 256), (23, 6, 3, 96, 32),
         (64, 3, 1, 160, 416), (33, 40, 6, 1024, 544), (9, 512, 16, 128, 128), (64, 128, 8, 256, 128),
         (2, 4, 2, 5120, 1792), (16, 8, 2, 2048, 768)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", CASES)
def test_layer(fq, fmt, tokens, experts, top_k, hidden, inter):
    if fmt == "f8":
        hidden, inter = -(-hidden // 128) * 128, -(-inter // 128) * 128
    seed = tokens * 7 + experts * 3 + hidden
    up = experts_of(fq, fmt, experts, 2 * inter, hidden, hidden ** -0.5, seed)
    down = experts_of(fq, fmt, experts, hidden, inter, inter ** -0.5, seed + 1)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, seed + 2, device="cuda")
    router = workloads.gaussian_bf16(experts, hidden, hidden ** -0.5, seed + 3, device="cuda")
    normalize = bool(seed % 2)
    ws = torch.zeros((fq.fp4q_moe_workspace_size(tokens, hidden, inter, experts, top_k),), dtype=torch.uint8,
                     device="cuda")
    y, ids, w = fq.fp4q_moe(x, router, top_k, up, down, fmt, normalize, workspace=ws)
    torch.cuda.synchronize()
    assert fq.fp4q_device_fault() == 0
    assert not ws[:64].any()
    check_route(ids, w, x, router, top_k, normalize)
    check_y(y, x, decode(up, fmt, experts), decode(down, fmt, experts), ids, w)
    # the same again, over the workspace as it was left
    y2, ids2, w2 = fq.fp4q_moe(x, router, top_k, up, down, fmt, normalize, workspace=ws)
    assert torch.equal(y, y2) and torch.equal(ids, ids2) and torch.equal(w, w2)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
@pytest.mark.parametrize("kind", ["some gone", "all gone", "twice", "one expert"])
def test_choices_made_elsewhere(fq, fmt, kind):
    tokens, experts, top_k, hidden, inter = 37, 9, 4, 384, 256
    g = torch.Generator().manual_seed(11)
    ids = torch.randint(0, experts, (tokens, top_k), generator=g, dtype=torch.int32)
    if kind == "some gone":
        ids[torch.rand((tokens, top_k), generator=g) < 0.4] = -1
        ids[5] = -1                                         # a token that has nothing left
        ids[6, 1], ids[7, 2] = experts, 2 ** 31 - 1         # past the last expert
    elif kind == "all gone":
        ids.fill_(-1)
    elif kind == "one expert":
        ids.fill_(3)                                        # 148 pairs: ten groups, a token four times
    w = torch.rand((tokens, top_k), generator=g)
    up = experts_of(fq, fmt, experts, 2 * inter, hidden, 0.05, 1, per_expert=True)
    down = experts_of(fq, fmt, experts, hidden, inter, 0.06, 2, per_expert=True)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3, device="cuda")
    y, i2, w2 = fq.fp4q_moe(x, None, top_k, up, down, fmt, ids=ids.cuda(), weights=w.cuda())
    torch.cuda.synchronize()
    assert torch.equal(i2.cpu(), ids) and torch.equal(w2.cpu(), w) and fq.fp4q_device_fault() == 0
    check_y(y, x, decode(up, fmt, experts), decode(down, fmt, experts), ids, w)
    nothing = ((ids < 0) | (ids >= experts)).all(1)
    assert not y.cpu()[nothing].any()


@pytest.mark.parametrize("tokens,top_k", [(1, 1), (1, 16), (8, 4), (2, 16), (7, 4), (11, 3)])
@pytest.mark.parametrize("kind", ["any", "one expert", "some gone", "all gone"])
def test_few_pairs(fq, tokens, top_k, kind):
    """Up to 32 pairs, and just above: lists of one, of more than a group's 16, with gaps, empty."""
    experts, hidden, inter = 20, 160, 96
    g = torch.Generator().manual_seed(tokens * 31 + top_k)
    ids = torch.randint(0, experts, (tokens, top_k), generator=g, dtype=torch.int32)
    if kind == "one expert":
        ids.fill_(19)
    elif kind == "some gone":
        ids[torch.rand((tokens, top_k), generator=g) < 0.5] = -7
    elif kind == "all gone":
        ids.fill_(20)
    w = torch.rand((tokens, top_k), generator=g)
    up = experts_of(fq, "nvfp4", experts, 2 * inter, hidden, 0.05, 1)
    down = experts_of(fq, "nvfp4", experts, hidden, inter, 0.06, 2)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3, device="cuda")
    y, _, _ = fq.fp4q_moe(x, None, top_k, up, down, "nvfp4", ids=ids.cuda(), weights=w.cuda())
    torch.cuda.synchronize()
    assert fq.fp4q_device_fault() == 0
    check_y(y, x, decode(up, "nvfp4", experts), decode(down, "nvfp4", experts), ids, w)


def test_equal_logits_take_the_lower_expert(fq):
    tokens, experts, top_k, hidden, inter = 4, 70, 5, 256, 64
    up = experts_of(fq, "nvfp4", experts, 2 * inter, hidden, 0.05, 1)
    down = experts_of(fq, "nvfp4", experts, hidden, inter, 0.05, 2)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3, device="cuda")
    router = workloads.gaussian_bf16(1, hidden, 0.1, 4, device="cuda").repeat(experts, 1)
    _, ids, w = fq.fp4q_moe(x, router, top_k, up, down, "nvfp4")
    assert torch.equal(ids.cpu(), torch.arange(top_k, dtype=torch.int32).repeat(tokens, 1))
    assert bool((w == w[0, 0]).all())
    # zero tokens' logits tie as well; -0 and 0 do not differ
    router[::2] *= -1
    _, ids, _ = fq.fp4q_moe(torch.zeros_like(x), router, top_k, up, down, "nvfp4")
    assert torch.equal(ids.cpu(), torch.arange(top_k, dtype=torch.int32).repeat(tokens, 1))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
def test_scales_and_inputs_of_every_size(fq, fmt):
    """Rows of x from 2^-60 to 2^60 and values within a row that span the format; weights whose scales span it."""
    tokens, experts, hidden, inter = 12, 3, 256, 128
    g = torch.Generator().manual_seed(5)
    e = torch.randint(-12, 13, (2 * inter * experts, hidden // 128), generator=g).float()
    w = torch.randn((experts * 2 * inter, hidden), generator=g) * torch.exp2(e).repeat_interleave(128, 1) * 0.01
    if fmt == "f8":
        up = fq.fp4q_f8_quantize(w.bfloat16().cuda(), "tile")
    else:
        up = fq.fp4q_quantize(w.bfloat16().cuda(), fmt, 32 if fmt == "mxfp4" else 16, 0,
                              "none" if fmt == "mxfp4" else "compute")
    down = experts_of(fq, fmt, experts, hidden, inter, 0.05, 2)
    x = torch.randn((tokens, hidden), generator=g) * torch.exp2(torch.randint(-9, 10, (tokens, hidden), generator=g).float())
    x *= torch.exp2(torch.linspace(-60, 20, tokens))[:, None]
    x = x.bfloat16().cuda()
    ids = torch.arange(tokens * 2, dtype=torch.int32).view(tokens, 2) % experts
    wt = torch.rand((tokens, 2), generator=g)
    y, _, _ = fq.fp4q_moe(x, None, 2, up, down, fmt, ids=ids.cuda(), weights=wt.cuda())
    want, tol = layer64(x, decode(up, fmt, experts), decode(down, fmt, experts), ids, wt)
    err = (y.cpu().double() - want).abs()
    # products of powers far below the smallest normal fp32 value are not held: 2^-126 per value of h
    tol += 2.0 ** -120
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
def test_tokens_stay_apart(fq, fmt):
    """NaN or infinity in a token changes no other; the others' results do not depend on who else is there."""
    tokens, experts, top_k, hidden, inter = 20, 6, 2, 256, 128
    up = experts_of(fq, fmt, experts, 2 * inter, hidden, 0.06, 1)
    down = experts_of(fq, fmt, experts, hidden, inter, 0.09, 2)
    router = workloads.gaussian_bf16(experts, hidden, 0.06, 4, device="cuda")
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3, device="cuda")
    y, ids, w = fq.fp4q_moe(x, router, top_k, up, down, fmt)
    bad = x.clone()
    bad[4, 17], bad[9, 200] = float("nan"), float("inf")
    y2, ids2, w2 = fq.fp4q_moe(bad, router, top_k, up, down, fmt)
    torch.cuda.synchronize()
    keep = torch.ones(tokens, dtype=torch.bool)
    keep[[4, 9]] = False
    assert torch.equal(ids[keep], ids2[keep]) and torch.equal(w[keep], w2[keep])
    assert torch.equal(y[keep], y2[keep]) and bool(torch.isnan(y2[4]).all())
    assert bool(((ids2 >= 0) & (ids2 < experts)).all())
    alone, _, _ = fq.fp4q_moe(x[3:4], router, top_k, up, down, fmt)
    assert torch.equal(alone[0], y[3])
    assert fq.fp4q_device_fault() == 0


def test_workspace_graphs_streams_and_outputs(fq):
    """One workspace for layers of several sizes in turn; captured calls replayed on new
    inputs, two graphs sharing a workspace in turn; two streams at once with a
    workspace each; strided x; given outputs, rows behind them left as they were."""
    small = dict(tokens=3, experts=8, top_k=2, hidden=128, inter=64)
    large = dict(tokens=40, experts=16, top_k=4, hidden=1024, inter=256)
    made = []
    for i, c in enumerate((small, large)):
        up = experts_of(fq, "nvfp4", c["experts"], 2 * c["inter"], c["hidden"], c["hidden"] ** -0.5, 10 + i)
        down = experts_of(fq, "nvfp4", c["experts"], c["hidden"], c["inter"], c["inter"] ** -0.5, 20 + i)
        router = workloads.gaussian_bf16(c["experts"], c["hidden"], 0.05, 30 + i, device="cuda")
        x = workloads.gaussian_bf16(c["tokens"], c["hidden"], 1.0, 40 + i, device="cuda")
        x2 = workloads.gaussian_bf16(c["tokens"], c["hidden"], 1.0, 50 + i, device="cuda")
        made.append((c, x, x2, (router, c["top_k"], up, down, "nvfp4")))
    size = max(fq.fp4q_moe_workspace_size(c["tokens"], c["hidden"], c["inter"], c["experts"], c["top_k"])
               for c, _, _, _ in made)
    shared = torch.zeros((size,), dtype=torch.uint8, device="cuda")
    plain = [(fq.fp4q_moe(x, *a)[0], fq.fp4q_moe(x2, *a)[0]) for _, x, x2, a in made]
    for i in (0, 1, 0, 1, 1, 0):
        assert torch.equal(fq.fp4q_moe(made[i][1], *made[i][3], workspace=shared)[0], plain[i][0])
    graphs = []
    for c, x, x2, a in made:
        held = x.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fq.fp4q_moe(held, *a, workspace=shared)
        graphs.append((g, held, out))
    for turn in range(4):
        for i in (0, 1):
            g, held, out = graphs[i]
            held.copy_(made[i][1 + (turn + i) % 2])
            g.replay()
            assert torch.equal(out[0], plain[i][(turn + i) % 2])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [torch.zeros_like(shared), torch.zeros_like(shared)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(6):
        for i in (0, 1):
            outs[i].append(fq.fp4q_moe(made[i][1], *made[i][3], workspace=spaces[i], stream=streams[i])[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, plain[i][0]) for i in (0, 1) for o in outs[i])
    c, x, _, a = made[1]
    wide = torch.zeros((c["tokens"], c["hidden"] + 24), dtype=torch.bfloat16, device="cuda")
    wide[:, :c["hidden"]] = x
    y = torch.full((c["tokens"] + 5, c["hidden"]), 9.0, dtype=torch.bfloat16, device="cuda")
    fq.fp4q_moe(wide[:, :c["hidden"]], *a, y=y[:c["tokens"]])
    assert torch.equal(y[:c["tokens"]], plain[1][0]) and bool((y[c["tokens"]:] == 9.0).all())
    assert fq.fp4q_device_fault() == 0


def test_past_32_bits(fq):
    """Codes of more than 2^32 bytes: the first, a middle and the last of 512 wide experts."""
    experts, hidden, inter = 512, 5120, 2048
    g = torch.Generator(device="cuda").manual_seed(4)
    draw = lambda r, c: torch.randint(0, 256, (r, c), generator=g, device="cuda", dtype=torch.uint8)
    scale = lambda r, c: torch.randint(118, 124, (r, c), generator=g, device="cuda", dtype=torch.uint8)
    up = (draw(experts * 2 * inter, hidden // 2), scale(experts * 2 * inter, hidden // 32), None)
    down = (draw(experts * hidden, inter // 2), scale(experts * hidden, inter // 32), None)
    assert up[0].numel() > 2 ** 32
    ids = torch.tensor([[511, 0], [400, 511], [255, 409]], dtype=torch.int32)
    w = torch.tensor([[0.5, 0.25], [0.75, 1.0], [0.3, 0.6]])
    x = workloads.gaussian_bf16(3, hidden, 2.0 ** -6, 5, device="cuda")
    y, _, _ = fq.fp4q_moe(x, None, 2, up, down, "mxfp4", ids=ids.cuda(), weights=w.cuda())
    torch.cuda.synchronize()
    chosen = sorted(set(ids.flatten().tolist()))
    part = lambda m, r: tuple(t.view(experts, r, -1)[chosen].flatten(0, 1) for t in m[:2])
    few = torch.tensor([[chosen.index(e) for e in row] for row in ids.tolist()])
    check_y(y, x, decode(part(up, 2 * inter), "mxfp4", len(chosen)), decode(part(down, hidden), "mxfp4", len(chosen)),
            few, w)
    assert fq.fp4q_device_fault() == 0


def test_two_host_threads_on_two_streams(fq):
    """Layers, products for few and for many tokens, in turn on two streams of different
    priority, from two host threads at once, a workspace each."""
    import threading

    tokens, experts, top_k, hidden, inter = 24, 16, 4, 1024, 512
    up = experts_of(fq, "nvfp4", experts, 2 * inter, hidden, hidden ** -0.5, 1)
    down = experts_of(fq, "nvfp4", experts, hidden, inter, inter ** -0.5, 2)
    router = workloads.gaussian_bf16(experts, hidden, 0.05, 3, device="cuda")
    xs = [workloads.gaussian_bf16(tokens, hidden, 1.0, 4 + i, device="cuda") for i in range(2)]
    a, sa = fq.fp4q_f8_quantize(workloads.gaussian_bf16(700, 2048, 1.0, 9, device="cuda"))
    b, sb = fq.fp4q_f8_quantize(workloads.gaussian_bf16(4096, 2048, 0.02, 10, device="cuda"), "tile")
    layer = lambda i, ws, s: fq.fp4q_moe(xs[i], router, top_k, up, down, "nvfp4", workspace=ws, stream=s)[0]
    calls = [layer, lambda i, ws, s: fq.fp4q_f8_gemm(a, sa, b, sb, stream=s),
             lambda i, ws, s: fq.fp4q_f8_gemm(a[:5], sa[:5], b, sb, stream=s)]
    want = [[c(i, None, None).clone() for c in calls] for i in range(2)]
    torch.cuda.synchronize()
    wrong = [0, 0]

    def run(i):
        stream = torch.cuda.Stream(priority=-i)
        with torch.cuda.stream(stream):
            ws = torch.zeros((8 << 20,), dtype=torch.uint8, device="cuda")
        for n in range(60):
            y = calls[(n + i) % 3](i, ws, stream)
            with torch.cuda.stream(stream):
                wrong[i] += int(not torch.equal(y, want[i][(n + i) % 3]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0] and fq.fp4q_device_fault() == 0


def test_run_of_the_operators_together(fq):
    """A decoder layer's linear part as it would be used: activations quantized to 8 bits and
    multiplied, the result through the experts, and the experts' result multiplied again."""
    tokens, hidden, inter, experts = 24, 512, 256, 8
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 1, device="cuda")
    b, sb = fq.fp4q_f8_quantize(workloads.gaussian_bf16(hidden, hidden, hidden ** -0.5, 2, device="cuda"), "tile")
    up = experts_of(fq, "f8", experts, 2 * inter, hidden, hidden ** -0.5, 3)
    down = experts_of(fq, "f8", experts, hidden, inter, inter ** -0.5, 4)
    router = workloads.gaussian_bf16(experts, hidden, 0.05, 5, device="cuda")
    a, sa = fq.fp4q_f8_quantize(x)
    m = fq.fp4q_f8_gemm(a, sa, b, sb)
    y, ids, w = fq.fp4q_moe(m, router, 2, up, down, "f8")
    a2, sa2 = fq.fp4q_f8_quantize(y)
    z = fq.fp4q_f8_gemm(a2, sa2, b, sb, torch.float32)
    torch.cuda.synchronize()
    check_route(ids, w, m, router, 2, True)
    check_y(y, m, decode(up, "f8", experts), decode(down, "f8", experts), ids, w)
    wide = lambda c, s, r: c.cpu().float().double() * s.cpu().double().repeat_interleave(r, 0).repeat_interleave(128, 1)
    want = wide(a2, sa2, 1) @ wide(b, sb, 128).T
    mag = wide(a2, sa2, 1).abs() @ wide(b, sb, 128).abs().T
    assert bool(((z.cpu().double() - want).abs() <= (17 + hidden / 128) * U * mag + U * want.abs()).all())


def test_empty_and_refusals(fq):
    experts, top_k, hidden, inter = 4, 2, 128, 128
    up = experts_of(fq, "mxfp4", experts, 2 * inter, hidden, 0.05, 1)
    down = experts_of(fq, "mxfp4", experts, hidden, inter, 0.05, 2)
    router = workloads.gaussian_bf16(experts, hidden, 0.05, 3, device="cuda")
    x = workloads.gaussian_bf16(2, hidden, 1.0, 4, device="cuda")
    y, ids, w = fq.fp4q_moe(x[:0], router, top_k, up, down, "mxfp4")
    assert y.shape == (0, hidden) and ids.shape == (0, top_k) and w.shape == (0, top_k)
    many = workloads.gaussian_bf16(65, hidden, 1.0, 4, device="cuda")
    for bad in (lambda: fq.fp4q_moe(many, router, top_k, up, down, "mxfp4"),
                lambda: fq.fp4q_moe(x, router, 5, up, down, "mxfp4"),
                lambda: fq.fp4q_moe(x, router, 0, up, down, "mxfp4"),
                lambda: fq.fp4q_moe(x, router, top_k, up, down, "mxfp4",
                                    workspace=torch.zeros((64,), dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fq.Fp4qError):
            bad()
    for bad in (lambda: fq.fp4q_moe(x, router, top_k, up, down, "ue5m3"),
                lambda: fq.fp4q_moe(x, router, top_k, up, down, "nvfp4"),
                lambda: fq.fp4q_moe(x, None, top_k, up, down, "mxfp4"),
                lambda: fq.fp4q_moe(x.float(), router, top_k, up, down, "mxfp4"),
                lambda: fq.fp4q_moe(x, router[:, :64], top_k, up, down, "mxfp4"),
                lambda: fq.fp4q_moe(x, router, top_k, (up[0][:-2], up[1]), down, "mxfp4"),
                lambda: fq.fp4q_moe(x, router, top_k, up, (down[0], down[1][:-1]), "mxfp4"),
                lambda: fq.fp4q_moe(x, None, top_k, up, down, "mxfp4", ids=torch.zeros((2, 2), device="cuda"),
                                    weights=torch.zeros((2, 2), device="cuda"))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("fmt,experts,hidden,inter", [
    ("nvfp4", 64, 5120, 768), ("nvfp4", 60, 1440, 1376), ("mxfp4", 128, 2048, 768), ("mxfp4", 60, 1440, 1376),
    ("f8", 32, 4096, 896), ("f8", 24, 1408, 1664)])
def test_a_token_alone_and_among_others(fq, fmt, experts, hidden, inter):
    """A token's result does not depend on who else is there, bit for bit, where a CTA works through many items
    whose stages are no multiple of the slices of k."""
    tokens, top_k = 64, 8
    up = experts_of(fq, fmt, experts, 2 * inter, hidden, hidden ** -0.5, 1)
    down = experts_of(fq, fmt, experts, hidden, inter, inter ** -0.5, 2)
    router = workloads.gaussian_bf16(experts, hidden, hidden ** -0.5, 3, device="cuda")
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 4, device="cuda")
    y, ids, w = fq.fp4q_moe(x, router, top_k, up, down, fmt)
    differ = []
    for first, last in ((0, 1), (17, 18), (63, 64), (5, 7), (30, 41), (8, 48)):
        ya, ia, wa = fq.fp4q_moe(x[first:last], router, top_k, up, down, fmt)
        assert torch.equal(ia, ids[first:last]) and torch.equal(wa, w[first:last])
        differ.append(int((ya != y[first:last]).sum()))
    assert not any(differ), differ
    assert fq.fp4q_device_fault() == 0


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 70, 5), (5, 512, 16), (64, 70, 8), (64, 512, 16), (9, 13, 13)])
def test_close_logits_are_told_apart(fq, tokens, experts, top_k):
    """Rows of the router that hold the same integers times powers of two in another order: the exact logits are
    equal (42 bits, so 64-bit sums in any order are exact) where fp32 sums are not. Equal ones take the lower expert
    and the same weight; ones that differ by a few 2^-12 of sums near 2^20 are in their exact order."""
    hidden, inter = 2048, 32
    g = torch.Generator().manual_seed(tokens + experts)
    base = (2 * torch.randint(-64, 64, (hidden,), generator=g) + 1) * torch.exp2(torch.randint(-12, 13, (hidden,), generator=g).float())
    base[0] = 0.0
    sign = torch.where(torch.rand((hidden,), generator=g) < 0.5, -1.0, 1.0)
    rows = torch.stack([torch.cat([base[:1], base[1:][torch.randperm(hidden - 1, generator=g)]]) for _ in range(experts)])
    router = (rows * sign).bfloat16().cuda()
    x = (sign * torch.exp2(-torch.randint(0, 9, (tokens, 1), generator=g).float() - 12)).bfloat16().cuda()
    up = experts_of(fq, "mxfp4", experts, 2 * inter, hidden, 0.02, 1)
    down = experts_of(fq, "mxfp4", experts, hidden, inter, 0.02, 2)
    _, ids, w = fq.fp4q_moe(x, router, top_k, up, down, "mxfp4")
    assert torch.equal(ids.cpu(), torch.arange(top_k, dtype=torch.int32).repeat(tokens, 1))
    assert bool((w == w[0, 0]).all())
    # column 0, where the rows hold nothing: different small integers (at most 255, in bf16 exactly) over 2^12
    d = torch.randperm(experts, generator=g) % 256
    router[:, 0] = (d * 2.0 ** -12 * sign[0]).bfloat16().cuda()
    _, ids, _ = fq.fp4q_moe(x, router, top_k, up, down, "mxfp4")
    want = torch.sort(d, descending=True, stable=True).indices[:top_k].to(torch.int32)
    assert torch.equal(ids.cpu(), want.repeat(tokens, 1))
    assert torch.equal(router.double().cpu() @ x.double().cpu().T, router.double().cpu().flip(1) @ x.double().cpu().flip(1).T)
    assert fq.fp4q_device_fault() == 0


@pytest.mark.parametrize("fmt,nan,tiny,huge", [("mxfp4", (0xFF,), 0, 254), ("nvfp4", (0x7F, 0x80, 0xB5, 0xFF), 0, 0x7E)])
@pytest.mark.parametrize("tokens", [2, 40])
def test_scale_bytes_at_the_ends(fq, fmt, nan, tiny, huge, tokens):
    """The last scale bytes are NaN (as in fp4q_dequantize), the first the smallest scale, and the largest scale of a
    block of zeros adds nothing; in every block of a row, which changes its own results alone."""
    experts, top_k, hidden, inter = 3, 2, 544, 512
    block = 32 if fmt == "mxfp4" else 16
    up = experts_of(fq, fmt, experts, 2 * inter, hidden, 0.05, 1)
    down = experts_of(fq, fmt, experts, hidden, inter, 0.05, 2)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3, device="cuda")
    ids = (torch.arange(tokens * 2, dtype=torch.int32).view(tokens, 2) % experts).cuda()
    w = torch.full((tokens, 2), 0.5, device="cuda")
    run = lambda u, d: fq.fp4q_moe(x, None, top_k, u, d, fmt, ids=ids, weights=w)[0]
    clean = run(up, down)
    hit = (ids == 1).any(1)                                  # tokens that read expert 1
    blocks = inter // block
    for byte in nan:
        # row r of expert 1's down matrix, block r
        s = down[1].clone()
        at = torch.arange(blocks, device="cuda")
        s[hidden + at, at] = byte
        y = run(up, (down[0], s, down[2]))
        assert bool(torch.isnan(y[hit][:, :blocks]).all())
        assert torch.equal(y[~hit], clean[~hit]) and torch.equal(y[:, blocks:], clean[:, blocks:])
        values = fq.fp4q_dequantize(down[0], s, down[2], experts * hidden, inter, fmt, block, 0, torch.float32)
        assert bool(torch.isnan(values.view(-1, blocks, block)[hidden + at, at]).all())
        # one gate row's block, then one up row's: a value of h, and with it the tokens' whole rows
        for row in (2 * inter + 5, 3 * inter + 7):
            for b in (0, 1, 7, hidden // block - 1):
                s = up[1].clone()
                s[row, b] = byte
                y = run((up[0], s, up[2]), down)
                assert bool(torch.isnan(y[hit]).all()) and torch.equal(y[~hit], clean[~hit])
    # the smallest scales, and the largest over blocks of zeros
    c, s = down[0].clone(), down[1].clone()
    c.view(experts * hidden, blocks, block // 2)[hidden + at, at] = 0
    zero = run(up, (c, s, down[2]))
    s[hidden + at, at] = huge
    assert torch.equal(run(up, (c, s, down[2])), zero)
    s = down[1].clone()
    s[hidden + at, at] = tiny
    check_y(run(up, (down[0], s, down[2])), x, decode(up, fmt, experts), decode((down[0], s, down[2]), fmt, experts), ids, w)
    assert fq.fp4q_device_fault() == 0


@pytest.mark.parametrize("counter,value", [(0, 1), (0, 5), (0, 2 ** 31 - 1), (1, 3), (1, 1000), (2, 1), (2, 1000), (3, 1000)])
@pytest.mark.parametrize("tokens", [2, 20])
def test_a_workspace_in_use_is_reported(fq, counter, value, tokens):
    """Counters that were not zero let waits pass early (all accesses stay within bounds): the fault word tells, and
    a workspace filled with zeros serves again."""
    experts, top_k, hidden, inter = 6, 2, 256, 128
    up = experts_of(fq, "nvfp4", experts, 2 * inter, hidden, 0.06, 1)
    down = experts_of(fq, "nvfp4", experts, hidden, inter, 0.09, 2)
    router = workloads.gaussian_bf16(experts, hidden, 0.06, 4, device="cuda")
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3, device="cuda")
    want = fq.fp4q_moe(x, router, top_k, up, down, "nvfp4")
    ws = torch.zeros((fq.fp4q_moe_workspace_size(tokens, hidden, inter, experts, top_k),), dtype=torch.uint8, device="cuda")
    ws[:16].view(torch.int32)[counter] = value
    assert fq.fp4q_device_fault() == 0
    fq.fp4q_moe(x, router, top_k, up, down, "nvfp4", workspace=ws)
    assert fq.fp4q_device_fault(clear=True) == 1
    ws[:64].zero_()
    got = fq.fp4q_moe(x, router, top_k, up, down, "nvfp4", workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert fq.fp4q_device_fault() == 0 and not ws[:64].any()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
def test_rows_of_every_size(fq, fmt):
    """Rows of x from 2^-60 to 2^60: a row's values are kept under its own power of two."""
    tokens, experts, hidden, inter = 25, 3, 256, 128
    up = experts_of(fq, fmt, experts, 2 * inter, hidden, 0.02, 1)
    down = experts_of(fq, fmt, experts, hidden, inter, 0.05, 2)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3).float() * torch.exp2(torch.linspace(-60, 60, tokens))[:, None]
    x = x.bfloat16().cuda()
    ids = torch.arange(tokens * 2, dtype=torch.int32).view(tokens, 2) % experts
    w = torch.full((tokens, 2), 0.5)
    y, _, _ = fq.fp4q_moe(x, None, 2, up, down, fmt, ids=ids.cuda(), weights=w.cuda())
    want, tol = layer64(x, decode(up, fmt, experts), decode(down, fmt, experts), ids, w)
    assert bool(torch.isfinite(y).all()) and float(want.abs().max()) > 2.0 ** 110
    # products of powers far below the smallest normal fp32 value are not held: 2^-126 per value of h
    tol += 2.0 ** -120
    err = (y.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
def test_channels_far_above_the_rest(fq, fmt):
    """One channel of each token 2^12 to 2^30 above the others, and no weight on it: the small values decide the
    result, exact as long as they lie above 2^-24 of the row's largest, off by 2^-32 of it at most below."""
    tokens, experts, hidden, inter = 19, 3, 512, 128
    at = torch.arange(tokens) * 27 + 3
    w = workloads.gaussian_bf16(experts * 2 * inter, hidden, 0.05, 1, device="cuda")
    w[:, at.cuda()] = 0.0
    if fmt == "f8":
        up = fq.fp4q_f8_quantize(w, "tile")
    else:
        up = fq.fp4q_quantize(w, fmt, 32 if fmt == "mxfp4" else 16, 0, "none" if fmt == "mxfp4" else "compute")
    down = experts_of(fq, fmt, experts, hidden, inter, 0.05, 2)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3)
    power = torch.arange(tokens) + 12
    x[torch.arange(tokens), at] = torch.exp2(power.float()).bfloat16()
    x = x.cuda()
    ids = torch.arange(tokens * 2, dtype=torch.int32).view(tokens, 2) % experts
    wt = torch.full((tokens, 2), 0.5)
    y, _, _ = fq.fp4q_moe(x, None, 2, up, down, fmt, ids=ids.cuda(), weights=wt.cuda())
    U64, D64 = decode(up, fmt, experts), decode(down, fmt, experts)
    assert not U64[:, :, at].any()
    want, tol = layer64(x, U64, D64, ids, wt)
    err = (y.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    exact = power <= 16                                      # values down to 2^-8 of one keep their eight bits
    assert float(err[exact].norm()) <= 2.0 ** -8 * float(want[exact].norm())


def test_nvfp4_without_a_tensor_scale(fq):
    """NVFP4 operands quantized without a per-tensor scale, on either side or both."""
    tokens, experts, top_k, hidden, inter = 21, 5, 2, 544, 96
    router = workloads.gaussian_bf16(experts, hidden, 0.05, 3, device="cuda")
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 4, device="cuda")
    plain = [fq.fp4q_quantize(workloads.gaussian_bf16(experts * r, c, s, 5 + r, device="cuda"), "nvfp4", 16)
             for r, c, s in ((2 * inter, hidden, 0.05), (hidden, inter, 0.08))]
    scaled = [experts_of(fq, "nvfp4", experts, 2 * inter, hidden, 0.05, 6, per_expert=True),
              experts_of(fq, "nvfp4", experts, hidden, inter, 0.08, 7)]
    assert plain[0][2] is None and plain[1][2] is None
    for up, down in ((plain[0], plain[1]), (plain[0], scaled[1]), (scaled[0], plain[1][:2])):
        y, ids, w = fq.fp4q_moe(x, router, top_k, up, down, "nvfp4")
        check_route(ids, w, x, router, top_k, True)
        check_y(y, x, decode(up, "nvfp4", experts), decode(down, "nvfp4", experts), ids, w)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
def test_a_wide_layer_of_many_experts(fq, fmt):
    """256 experts of 7168 x 2048 and 512 pairs, each expert's matrices decoded to 64 bits on the GPU; the bars of the top."""
    tokens, experts, top_k, hidden, inter = 64, 256, 8, 7168, 2048
    g = torch.Generator(device="cuda").manual_seed(8)

    def matrix(rows, cols):
        draw = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8)
        if fmt == "f8":                                      # codes of 1/16 to 15, either sign
            codes = draw(0x18, 0x58, experts * rows, cols) | draw(0, 2, experts * rows, 1) << 7
            scales = torch.rand((experts * rows // 128, cols // 128), generator=g, device="cuda") * (0.2 / cols ** 0.5)
            return codes.view(torch.float8_e4m3fn), scales
        codes = draw(0, 256, experts * rows, cols // 2)
        if fmt == "mxfp4":
            return codes, draw(118, 121, experts * rows, cols // 32), None
        return codes, draw(0x28, 0x39, experts * rows, cols // 16), torch.rand((experts,), generator=g, device="cuda") * (0.7 / cols ** 0.5)

    grid = torch.cat((GRID, -GRID)).cuda()

    def expert(m, e, rows):
        c, s = m[0][e * rows:(e + 1) * rows], m[1].view(experts, -1, m[1].shape[1])[e].double()
        if fmt == "f8":
            return c.double() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)
        v = torch.stack((grid[(c & 15).long()], grid[(c >> 4).long()]), -1).view(rows, -1)
        s = torch.exp2(s - 127) if fmt == "mxfp4" else m[1].view(experts, rows, -1)[e].view(torch.float8_e4m3fn).double() * m[2][e].double()
        return v * s.repeat_interleave(v.shape[1] // s.shape[1], 1)

    up, down = matrix(2 * inter, hidden), matrix(hidden, inter)
    router = workloads.gaussian_bf16(experts, hidden, hidden ** -0.5, 3, device="cuda")
    x = workloads.gaussian_bf16(tokens, hidden, 1.0 if fmt != "mxfp4" else 0.5, 4, device="cuda")
    y, ids, w = fq.fp4q_moe(x, router, top_k, up, down, fmt)
    assert fq.fp4q_device_fault() == 0
    check_route(ids, w, x, router, top_k, True)
    xd, want = x.double(), torch.zeros((tokens, hidden), dtype=torch.float64, device="cuda")
    far = torch.zeros_like(want)
    for e in range(experts):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if not token.numel():
            continue
        xe, W, D, we = xd[token], expert(up, e, 2 * inter), expert(down, e, hidden), w.double()[token, slot][:, None]
        v = xe @ W.T
        ev = (hidden / 64 + 24) * U * (xe.abs() @ W.abs().T) + 2.0 ** -32 * top_of(xe) * W.abs().sum(1)
        gate, u, eg, eu = v[:, :inter], v[:, inter:], ev[:, :inter], ev[:, inter:]
        silu = gate * torch.sigmoid(gate)
        h = silu * u
        eh = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (2.0 ** -11 + 2.0 ** -20) * h.abs() + 2.0 ** -24 * top_of(h)
        want.index_add_(0, token, (h @ D.T) * we)
        far.index_add_(0, token, (eh @ D.abs().T + (inter / 64 + 24 + top_k) * U * ((h.abs() + eh) @ D.abs().T)) * we)
    half = torch.finfo(torch.bfloat16).eps / 2
    err, tol = (y.double() - want).abs(), far * (1 + half) + half * want.abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert float(err.norm()) <= 2.0 ** -8 * float(want.norm())
    assert len(set(ids.flatten().tolist())) > 180


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", [
    (3, 2, 1, 65536, 128), (3, 2, 2, 128, 65536), (5, 2, 2, 65408, 256), (64, 512, 16, 128, 128), (1, 1, 1, 128, 128)])
def test_sizes_at_the_limits(fq, fmt, tokens, experts, top_k, hidden, inter):
    """The longest rows, the most experts and choices, one of each; memory beside the results and the workspace kept."""
    up = experts_of(fq, fmt, experts, 2 * inter, hidden, hidden ** -0.5, 1)
    down = experts_of(fq, fmt, experts, hidden, inter, inter ** -0.5, 2)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3, device="cuda")
    router = workloads.gaussian_bf16(experts, hidden, hidden ** -0.5, 4, device="cuda")
    size = fq.fp4q_moe_workspace_size(tokens, hidden, inter, experts, top_k)
    ws = torch.zeros((size + 64,), dtype=torch.uint8, device="cuda")
    ws[size:] = 0xAB
    guard = torch.full((tokens + 2, hidden), 5.0, dtype=torch.bfloat16, device="cuda")
    y, ids, w = fq.fp4q_moe(x, router, top_k, up, down, fmt, False, workspace=ws[:size], y=guard[1:tokens + 1])
    assert fq.fp4q_device_fault() == 0
    assert bool((ws[size:] == 0xAB).all()) and bool((guard[0] == 5.0).all()) and bool((guard[-1] == 5.0).all())
    check_route(ids, w, x, router, top_k, False)
    check_y(y, x, decode(up, fmt, experts), decode(down, fmt, experts), ids, w)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4", "f8"])
def test_every_choice_on_one_expert(fq, fmt):
    """1024 pairs, 64 groups, of one expert among 20."""
    tokens, experts, top_k, hidden, inter = 64, 20, 16, 256, 384
    up = experts_of(fq, fmt, experts, 2 * inter, hidden, 0.05, 1)
    down = experts_of(fq, fmt, experts, hidden, inter, 0.05, 2)
    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 3, device="cuda")
    ids = torch.full((tokens, top_k), 19, dtype=torch.int32)
    w = torch.rand((tokens, top_k), generator=torch.Generator().manual_seed(4))
    y, _, _ = fq.fp4q_moe(x, None, top_k, up, down, fmt, ids=ids.cuda(), weights=w.cuda())
    assert fq.fp4q_device_fault() == 0
    check_y(y, x, decode(up, fmt, experts), decode(down, fmt, experts), ids, w)


def test_a_run_of_the_operators_captured(fq):
    """Quantizer, product, layer, quantizer and product twice over in one graph, replayed on new inputs."""
    tokens, hidden, inter, experts = 24, 512, 256, 8
    b, sb = fq.fp4q_f8_quantize(workloads.gaussian_bf16(hidden, hidden, hidden ** -0.5, 2, device="cuda"), "tile")
    up = experts_of(fq, "f8", experts, 2 * inter, hidden, hidden ** -0.5, 3)
    down = experts_of(fq, "f8", experts, hidden, inter, inter ** -0.5, 4)
    router = workloads.gaussian_bf16(experts, hidden, 0.05, 5, device="cuda")

    def chain(x):
        m = fq.fp4q_f8_gemm(*fq.fp4q_f8_quantize(x), b, sb)
        y, _, _ = fq.fp4q_moe(m, router, 2, up, down, "f8")
        return fq.fp4q_f8_gemm(*fq.fp4q_f8_quantize(y), b, sb)

    x = workloads.gaussian_bf16(tokens, hidden, 1.0, 1, device="cuda")
    chain(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(chain(x))
    for seed in (6, 7, 8):
        new = workloads.gaussian_bf16(tokens, hidden, 1.0, seed, device="cuda")
        x.copy_(new)
        graph.replay()
        assert torch.equal(out, chain(chain(new)))
    assert fq.fp4q_device_fault() == 0
