"""The microscaled 4-bit layer and the norm and rotation of queries and keys, as they are measured.

Two operators stand next to the 8-bit layer and the norms of perf/operators.py: a linear layer
whose weights and rows are 4-bit floating point with a power of two for every 32 of them, and what
an attention does to the rows that such a layer (or any other of the library) gives it:

  linear       y = r * (W q_b) + bias, q_b the 4-bit row of T x_b (T the lifted layer's block Hadamard
               transform and channel scales, or nothing): lq_mx4_linear
  gated        the same of x = act(gate) * up, the gate and up halves of one product:
               lq_mx4_linear with its gate, or lq_mx4_quant_rows and lq_mx4_gemm
  rope         the heads' norms and the rotation by position: lq_qk_norm_rope
  qkv          the layer that makes queries, keys and values, then the norms and the
               rotation in place: lq_mx4_linear, lq_qk_norm_rope

The format: of 32 values v with the largest magnitude m, the scale is 2^e with e = floor(log2 m) - 2
(-127 at least), and v 2^-e is rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives, ties to the even code, what is above 6 to 6.

Sizes are those of this repository's workloads (Llama-3-8B/70B and Qwen-2.5-32B layers, the 512-wide
layer, a 2048-token prefill; heads of 128), and odd ones.
"""
import math

import torch

own = False

ACTS = {
    "silu": lambda v: v / (1 + torch.exp(-v)),
    "gelu": lambda v: 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))),
}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
MOST = 2048 * 28672 * 8192        # multiply-adds of the largest listed product
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    lin = dict(op="linear", hb=1, x="bf16", y="bf16", bias=False, r=True)
    rope = dict(op="rope", x="bf16", norm=True, one_plus=False, interleaved=False, base=500000.0, far=8192)
    return [
        # one token through the 512-wide layer in fp32: launch latency
        dict(lin, name="mx4 512x512 b1 f32", B=1, N=512, K=512, x="f32", y="f32"),
        # one token through an attention projection: the weights' stream
        dict(lin, name="mx4 10240x8192 b1 T", B=1, N=10240, K=8192, hb=1024),
        # a small serving batch through a down projection, long reduction
        dict(lin, name="mx4 8192x28672 b16 T", B=16, N=8192, K=28672, hb=1024),
        # a larger batch through an up projection, with a bias and no scale for the rows
        dict(lin, name="mx4 27648x5120 b64", B=64, N=27648, K=5120, bias=True, r=False),
        # a packed batch of odd sizes, fp32 in and out
        dict(lin, name="mx4 5125x4099 b333 f32", B=333, N=5125, K=4099, x="f32", y="f32", bias=True),
        # a prompt of 2048 tokens through the widest layer
        dict(lin, name="mx4 28672x8192 b2048", B=2048, N=28672, K=8192),
        # one token through the end of an MLP, the gate within the layer's call
        dict(op="gated", name="mx4 gated 4096x14336 b1", B=1, N=4096, K=14336, act="silu", apart=False),
        # a prompt of 2048 tokens through the end of the largest MLP, rows and product apart
        dict(op="gated", name="mx4 gated 8192x28672 b2048", B=2048, N=8192, K=28672, act="silu", apart=True),
        # one token's queries and keys, rotation alone: launch latency
        dict(rope, name="rope 64+8x128 b1", B=1, q=64, k=8, d=128, rot=128, norm=False),
        # a prompt: norms and rotation
        dict(rope, name="norm rope 64+8x128 b2048", B=2048, q=64, k=8, d=128, rot=128),
        # odd sizes, fp32, neighbours paired, a part of the head rotated, far positions
        dict(rope, name="norm rope 40+8x80 b777 f32", B=777, q=40, k=8, d=80, rot=60, x="f32", one_plus=True,
             interleaved=True, far=1 << 20, base=10000.0),
        # a serving batch: the projection, then its queries and keys normed and rotated in place
        dict(rope, name="qkv 10240x8192 b64 T", op="qkv", B=64, K=8192, N=10240, hb=1024, q=64, k=8, d=128, rot=128),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Tokens 1..2048, outputs 16..28672, inputs 32..28672, heads 1..64 of 16..256, every option of the listed cases."""
    op = rng.choice(["linear", "linear", "gated", "rope", "rope", "qkv"])
    B, N, K = _log(rng, 1, 2048), _log(rng, 16, 28672), _log(rng, 32, 28672)
    hb = rng.choice([1, 1, 128, 512, 1024])
    if op in ("linear", "qkv"):
        K = max(hb, K // hb * hb)
    rope = {}
    if op in ("rope", "qkv"):
        d = rng.choice([64, 128, 128, 256, 2 * rng.randint(8, 128)])
        rope = dict(q=_log(rng, 1, 64), d=d, rot=rng.choice([d, d, d // 2 // 2 * 2]), one_plus=rng.random() < 0.3,
                    norm=rng.random() < 0.6, interleaved=rng.random() < 0.4, far=rng.choice([8192, 1 << 20]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]))
        rope["k"] = max(1, rope["q"] // rng.choice([1, 4, 8]))
    if op == "rope":
        return dict(rope, op=op, B=B, x=rng.choice(["f32", "bf16"]))
    if op == "qkv":
        N = (rope["q"] + 2 * rope["k"]) * rope["d"]
    B = max(1, min(B, MOST // (N * K)))
    if op == "qkv":
        return dict(rope, op=op, B=B, N=N, K=K, hb=hb, x="bf16")
    if op == "gated":
        return dict(op=op, B=B, N=N, K=K, act=rng.choice(["silu", "gelu"]), apart=rng.random() < 0.5)
    # T's sums round differently in another order, and a value next to the border of two codes
    # then takes the other one: those outputs are bf16. Without T the codes are exact.
    return dict(op=op, B=B, N=N, K=K, hb=hb, x=rng.choice(["f32", "bf16"]),
                y="bf16" if hb > 1 else rng.choice(["f32", "bf16"]), bias=rng.random() < 0.5, r=rng.random() < 0.7)


# ------------------------------------------------------------------- the format, in 32 bits

def _blocks(v):
    """v's rows in blocks of 32, the last filled up with zeros."""
    B, K = v.shape
    nb = -(-K // 32)
    if K % 32:
        v = torch.nn.functional.pad(v, (0, 32 * nb - K))
    return v.reshape(B, nb, 32)


def _mx4(v):
    """(the values as multiples of their scales, the scales' exponents) of rows in 32 bits."""
    v = _blocks(v)
    e = (torch.frexp(v.abs().amax(dim=2, keepdim=True)).exponent - 3).clamp_(min=-127)
    u = v * torch.exp2(-e.float())                      # exact
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp_(max=6), u), e[:, :, 0]


def _as_bytes(u):
    """Codes, the even of two values in a byte's low half."""
    a = u.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | torch.where(u < 0, 8, 0).to(torch.uint8)).reshape(u.shape[0], -1, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4)


def _panels(code):
    """Scale bytes (rows, blocks) as the library keeps them: panels of 16 rows, in each 128 bytes for
    every 8 blocks, row by row, and of a row's 8 the order 0 4 1 5 2 6 3 7."""
    n, nb = code.shape
    units = -(-nb // 8)
    code = torch.nn.functional.pad(code, (0, 8 * units - nb, 0, -n % 16))
    return code.reshape(-1, 16, units, 2, 4).permute(0, 2, 1, 4, 3).contiguous().reshape(-1)


def _values(w, scale, K):
    """The values that rows of codes stand for, in 32 bits."""
    n, nb = w.shape[0], -(-K // 32)
    half = torch.tensor(GRID + [-x for x in GRID], device="cuda")
    both = torch.stack((half.repeat(16), half.repeat_interleave(16)), dim=1)       # of a byte, low half first
    code = scale.reshape(-1, -(-nb // 8), 16, 4, 2).permute(0, 2, 1, 4, 3).reshape(-(-n // 16) * 16, -1)
    v = both[w.int()].reshape(n, nb, 32) * torch.exp2(code[:n, :nb, None].float() - 127)
    return v.reshape(n, -1)[:, :K]


# ------------------------------------------------------------------- inputs

def _activations(g, B, K, dtype):
    """Token rows with 1% of the channels 20 times as large, as trained models have them."""
    gain = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return (torch.randn(B, K, generator=g, device="cuda") * gain).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B = case["op"], case["B"]
    s = {"case": case, "c": None, "r": None, "bias": None}
    if op != "rope":
        N, K = case["N"], case["K"]
        if op == "gated":
            s["gate_up"] = torch.randn(B, 2 * K, generator=g, device="cuda").to(torch.bfloat16)
        else:
            s["x"] = _activations(g, B, K, DTYPES[case["x"]])
            s["c"] = 0.8 + 0.4 * torch.rand(K, generator=g, device="cuda") if case["hb"] > 1 else None
        nb = -(-K // 32)
        s["w"] = torch.empty(N, 16 * nb, dtype=torch.uint8, device="cuda")
        code = torch.empty(N, nb, dtype=torch.uint8, device="cuda")
        rows = max(1, (1 << 26) // K)
        for n in range(0, N, rows):
            u, e = _mx4(torch.randn(min(rows, N - n), K, generator=g, device="cuda") / math.sqrt(K))
            s["w"][n:n + rows] = _as_bytes(u)
            code[n:n + rows] = (e + 127).to(torch.uint8)
        s["w_scale"] = _panels(code)
        if case.get("r", True):
            s["r"] = 0.5 + torch.rand(N, generator=g, device="cuda")
        if case.get("bias"):
            s["bias"] = torch.randn(N, generator=g, device="cuda")
    if op in ("rope", "qkv"):
        H, d, rot = case["q"] + case["k"], case["d"], case["rot"]
        if op == "rope":
            # queries, keys and values of a token lie side by side
            s["qkv"] = (2 * torch.randn(B, (H + case["k"]) * d, generator=g, device="cuda")).to(DTYPES[case["x"]])
        s["pos"] = torch.randint(0, case["far"], (B,), generator=g, device="cuda")
        s["freq"] = case["base"] ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        base = 0.0 if case["one_plus"] else 1.0
        s["w_q"] = base + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None
        s["w_k"] = base + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None
    if own:
        _handles(s)
    return s


def _heads(case, rows):
    """The queries and the keys in rows of queries, keys and values."""
    q, k, d = case["q"], case["k"], case["d"]
    return rows[:, :q * d].unflatten(1, (q, d)), rows[:, q * d:(q + k) * d].unflatten(1, (k, d))


def _handles(s):
    """What a program keeps next to its data: the layer's description, outputs and workspace."""
    import bit_matmul_amd as lq
    case = s["case"]
    op, B = case["op"], case["B"]
    if op == "rope":
        dtype = DTYPES[case["x"]]
        s["q_out"] = torch.empty(B, case["q"], case["d"], dtype=dtype, device="cuda")
        s["k_out"] = torch.empty(B, case["k"], case["d"], dtype=dtype, device="cuda")
        return
    N, K = case["N"], case["K"]
    s["layer"] = lq.mx4_layer_struct(N, K, s["w"], s["w_scale"], s["r"], hb=case.get("hb", 1), c=s["c"], bias=s["bias"])
    s["out"] = torch.empty(B, N, dtype=DTYPES[case.get("y", "bf16")], device="cuda")
    if case.get("apart"):
        n = lq.lq_mx4_gemm_workspace_size(s["layer"], B)
        s["codes"] = torch.empty(B, -(-K // 32) * 16, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty(lq.lq_mx4_scale_size(B, K), dtype=torch.uint8, device="cuda")
    else:
        n = lq.lq_mx4_linear_workspace_size(s["layer"], B, torch.bfloat16 if op == "gated" else s["x"].dtype)
    s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
    if op == "gated":
        s["act"] = getattr(lq, "LQ_ACT_" + case["act"].upper())


def _run_own(s):
    import bit_matmul_amd as lq
    case = s["case"]
    op, B = case["op"], case["B"]
    if op == "linear":
        lq.lq_mx4_linear(s["layer"], s["x"], B, s["out"], s["ws"])
        return s["out"]
    if op == "gated":
        K = case["K"]
        gate, up = s["gate_up"][:, :K], s["gate_up"][:, K:]
        if case["apart"]:
            lq.lq_mx4_quant_rows(up, B, K, s["codes"], s["scale"], gate=gate, act=s["act"])
            lq.lq_mx4_gemm(s["layer"], s["codes"], s["scale"], B, s["out"], s["ws"])
        else:
            lq.lq_mx4_linear(s["layer"], up, B, s["out"], s["ws"], gate=gate, act=s["act"])
        return s["out"]
    how = dict(norm=case["norm"], w_q=s["w_q"], w_k=s["w_k"], one_plus=case["one_plus"], eps=EPS,
               interleaved=case["interleaved"])
    if op == "rope":
        q, k = _heads(case, s["qkv"])
        lq.lq_qk_norm_rope(s["pos"], s["freq"], q=q, k=k, q_out=s["q_out"], k_out=s["k_out"], **how)
        return {"q": s["q_out"], "k": s["k_out"]}
    lq.lq_mx4_linear(s["layer"], s["x"], B, s["out"], s["ws"])
    q, k = _heads(case, s["out"])
    lq.lq_qk_norm_rope(s["pos"], s["freq"], q=q, k=k, q_out=q, k_out=k, **how)
    return s["out"]


# ------------------------------------------------------------------- plain form

def _whiten(v, c, hb):
    """T v: the orthonormal Hadamard matrix of order hb on every run of hb scaled channels."""
    v = (v * c).reshape(v.shape[0], -1, hb)
    h = 1
    while h < hb:
        v = v.reshape(v.shape[0], -1, 2, h)
        v = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), dim=2)
        h *= 2
    return v.reshape(v.shape[0], -1) / math.sqrt(hb)


def _layer(s, v):
    """The layer's outputs for rows v, in 32 bits."""
    K = v.shape[1]
    u, e = _mx4(v)
    q = (u * torch.exp2(e[:, :, None].float())).reshape(v.shape[0], -1)[:, :K]
    y = q @ _values(s["w"], s["w_scale"], K).t()
    y = y if s["r"] is None else y * s["r"]
    return y if s["bias"] is None else y + s["bias"]


def _rope(s, x, w, cos, sin):
    """Norm and rotation of the heads x (tokens, heads, d), in 32 bits."""
    case = s["case"]
    rot = case["rot"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(dim=2, keepdim=True) + EPS) * (1 + w if case["one_plus"] else w)
    if case["interleaved"]:
        a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=3).flatten(2)
    else:
        a, b = x[:, :, :rot // 2], x[:, :, rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=2)
    return torch.cat((turned, x[:, :, rot:]), dim=2)


def _turn(s):
    angle = s["pos"].double()[:, None, None] * s["freq"]
    return torch.cos(angle).float(), torch.sin(angle).float()


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op = case["op"]
    if op == "gated":
        K = case["K"]
        return _layer(s, ACTS[case["act"]](s["gate_up"][:, :K].float()) * s["gate_up"][:, K:].float()).to(torch.bfloat16)
    if op == "rope":
        q, k = _heads(case, s["qkv"])
        turn = _turn(s)
        return {"q": _rope(s, q, s["w_q"], *turn).to(q.dtype), "k": _rope(s, k, s["w_k"], *turn).to(k.dtype)}
    v = s["x"].float()
    y = _layer(s, _whiten(v, s["c"], case["hb"]) if case["hb"] > 1 else v)
    if op == "linear":
        return y.to(DTYPES[case["y"]])
    y = y.to(torch.bfloat16)
    q, k = _heads(case, y)
    turn = _turn(s)
    both = torch.cat((_rope(s, q, s["w_q"], *turn), _rope(s, k, s["w_k"], *turn)), dim=1).flatten(1)
    return torch.cat((both.to(torch.bfloat16), y[:, both.shape[1]:]), dim=1)


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, B = case["op"], case["B"]
    grid = torch.tensor(GRID, dtype=torch.float64, device="cuda")

    def rounded(v):
        """What the 4-bit rows of v stand for."""
        K = v.shape[1]
        out = torch.zeros(B, -(-K // 32) * 32, dtype=torch.float64, device="cuda")
        out[:, :K] = v
        out = out.view(B, -1, 32)
        m = out.abs().max(dim=2).values[:, :, None]
        scale = torch.pow(2.0, (torch.floor(torch.log2(m.clamp(min=2.0 ** -149))) - 2).clamp(min=-127))
        a = out.abs() / scale
        mid = (grid[1:] + grid[:-1]) / 2
        low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
        near = grid[torch.where(low % 2 == 0, low, high)]
        return (torch.sign(out) * near * scale).reshape(B, -1)[:, :K]

    def weights():
        n, K = case["N"], case["K"]
        nb = -(-K // 32)
        block = torch.arange(nb, device="cuda")
        row = torch.arange(n, device="cuda")[:, None]
        unit, inside = block // 8, block % 8
        at = (row // 16) * (128 * (-(-nb // 8))) + 128 * unit + 8 * (row % 16) + 2 * (inside % 4) + inside // 4
        e = s["w_scale"][at].double() - 127
        code = torch.stack((s["w"] & 15, s["w"] >> 4), dim=2).reshape(n, nb, 32)
        w = grid[(code & 7).long()]
        return torch.where(code > 7, -w, w).mul_(torch.pow(2.0, e)[:, :, None]).reshape(n, -1)[:, :K].T.contiguous()

    def layer(v):
        y = torch.matmul(rounded(v), weights())
        y = y if s["r"] is None else y * s["r"].double()
        return y if s["bias"] is None else y + s["bias"].double()

    def turned(x, w):
        rot, half = case["rot"], case["rot"] // 2
        if w is not None:
            n = torch.sqrt((x * x).sum(dim=2) / case["d"] + EPS)[:, :, None]
            x = x / n * (w.double() + (1.0 if case["one_plus"] else 0.0))
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        z = torch.complex(x[:, :, first], x[:, :, second])
        angle = s["pos"].double()[:, None] * s["freq"][None, :]
        z = z * torch.polar(torch.ones_like(angle), angle)[:, None, :]
        out = x.clone()
        out[:, :, first], out[:, :, second] = z.real, z.imag
        return out

    if op == "rope":
        q, k = _heads(case, s["qkv"].double())
        return {"q": turned(q, s["w_q"]), "k": turned(k, s["w_k"])}
    if op == "gated":
        g, u = s["gate_up"].double().split(case["K"], dim=1)
        if case["act"] == "silu":
            return layer(g * torch.sigmoid(g) * u)
        return layer(g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)) * u)
    v = s["x"].double()
    if case["hb"] > 1:
        i = torch.arange(case["hb"], device="cuda")
        parity = i[:, None] & i[None, :]
        for b in (8, 4, 2, 1):
            parity = parity ^ (parity >> b)
        H = (1 - 2 * (parity & 1)).double() / math.sqrt(case["hb"])
        v = torch.matmul((v * s["c"].double()).reshape(-1, case["hb"]), H).reshape(B, case["K"])
    y = layer(v)
    if op == "linear":
        return y
    q, k = _heads(case, y)
    both = torch.cat((turned(q, s["w_q"]), turned(k, s["w_k"])), dim=1).flatten(1)
    return torch.cat((both, y[:, both.shape[1]:]), dim=1)


def work(case):
    """Each input read once, each output written once; two operations for a multiply-add."""
    op, B = case["op"], case["B"]
    size = {"f32": 4, "bf16": 2}
    nbytes = flops = 0
    if op != "rope":
        N, K = case["N"], case["K"]
        nbytes = N * K // 2 + N * -(-K // 32) + 4 * N * (case.get("r", True) + case.get("bias", False))
        nbytes += B * K * (4 if op == "gated" else size[case["x"]]) + B * N * size[case.get("y", "bf16")]
        hb = case.get("hb", 1)
        flops = 2 * B * N * K + B * K * (8 if op == "gated" else 3)
        if hb > 1:
            nbytes += 4 * K
            flops += B * K * (1 + math.log2(hb))
    if op in ("rope", "qkv"):
        heads, d = case["q"] + case["k"], case["d"]
        flops += B * heads * (3 * case["rot"] + (4 * d if case["norm"] else 0))
        nbytes += 8 * B + 4 * case["rot"] + (8 * d if case["norm"] else 0)
        if op == "rope":
            nbytes += 2 * B * heads * d * size[case["x"]]
    return {"bytes": nbytes, "flops": flops}
