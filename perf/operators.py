"""The 8-bit linear layer and the norms around it, as they are measured.

Three operators stand next to the lifted layer. They serve the layers of a
model that are kept at 8 bits (the output head, the first and last blocks,
any layer that the lifted code does not hold well enough) and the norms
between the linear layers of either kind:

  linear       y = r * s_b * (W q_b) + bias, with q_b, s_b the 8-bit row of
               T x_b (T the lifted layer's block Hadamard transform and channel
               scales, or nothing): lq_int8_linear
  gated        the same from the gate and up halves of one product,
               x = act(gate) * up, and then the product on the rows that are
               8 bits already: lq_quant_rows, lq_int8_gemm
  norm         norm after a block, gate, scaled residual, norm before the
               next block: lq_norm_block
  norm_linear  the same, writing 8-bit rows that the next product takes:
               lq_norm_block, lq_int8_gemm

The 8-bit row of v is s = max|v| / 127, q = v * 127 / max|v| rounded to the
nearest whole number, ties to even. Products of 8-bit rows are summed exactly.

Sizes are those of this repository's workloads (Llama-3-8B/70B and
Qwen-2.5-32B layers, the 512-wide layer, a 2048-token prefill), and odd ones.
"""
import math

import torch

own = False

ACTS = {
    "none": lambda v: v,
    "silu": lambda v: v / (1 + torch.exp(-v)),
    "gelu": lambda v: 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))),
    "sigmoid": lambda v: 1 / (1 + torch.exp(-v)),
    "tanh": torch.tanh,
}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
MOST = 2048 * 28672 * 8192        # multiply-adds of the largest listed product


def listed():
    lin = dict(op="linear", hb=1, x="bf16", y="bf16", bias=False)
    norm = dict(op="norm", y="bf16", h="bf16", a="bf16", post=True, pre=True, gate="none", act="none",
                first=False, one_plus=False, alpha=1.0)
    return [
        # one token through the 512-wide layer in fp32: launch latency
        dict(lin, name="linear 512x512 b1 f32", B=1, N=512, K=512, x="f32", y="f32"),
        # one token through an attention projection: the weights' stream
        dict(lin, name="linear 10240x8192 b1 T", B=1, N=10240, K=8192, hb=1024),
        # a small serving batch through a down projection, long reduction
        dict(lin, name="linear 8192x28672 b16 T", B=16, N=8192, K=28672, hb=1024),
        # a larger batch through an up projection, with a bias
        dict(lin, name="linear 27648x5120 b64", B=64, N=27648, K=5120, bias=True),
        # a packed batch of odd sizes, fp32 in and out
        dict(lin, name="linear 5125x4099 b333 f32", B=333, N=5125, K=4099, x="f32", y="f32", bias=True),
        # a prompt of 2048 tokens through the widest layer
        dict(lin, name="linear 28672x8192 b2048", B=2048, N=28672, K=8192),
        # one token through the end of an MLP
        dict(op="gated", name="gated 4096x14336 b1", B=1, N=4096, K=14336, act="silu"),
        # a prompt of 2048 tokens through the end of the largest MLP
        dict(op="gated", name="gated 8192x28672 b2048", B=2048, N=8192, K=28672, act="silu"),
        # one token: residual sum and the next block's norm
        dict(norm, name="norm 8192 b1", B=1, K=8192, post=False),
        # a prompt: norms on both sides of the block, a learned scale for each channel
        dict(norm, name="norm 8192 b2048 both", B=2048, K=8192, gate="vector", one_plus=True),
        # odd sizes, fp32, a gate for each token before the norm, a scaled residual
        dict(norm, name="norm 4099 b777 f32", B=777, K=4099, y="f32", h="f32", a="f32", gate="rows",
             act="silu", first=True, alpha=0.22),
        # a serving batch: residual, norm to 8 bits, and the projection that reads it
        dict(op="norm_linear", name="norm_linear 10240x8192 b64", B=64, N=10240, K=8192),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Tokens 1..2048, outputs 16..28672, inputs 64..28672, every option of the listed cases."""
    op = rng.choice(["linear", "linear", "gated", "norm", "norm", "norm_linear"])
    B, N, K = _log(rng, 1, 2048), _log(rng, 16, 28672), _log(rng, 64, 28672)
    if op == "norm":
        gate = rng.choice(["none", "vector", "rows"])
        return dict(op=op, B=B, K=K, y=rng.choice(["f32", "bf16"]), h=rng.choice(["f32", "bf16"]),
                    a=rng.choice(["f32", "bf16"]), post=rng.random() < 0.5, pre=rng.random() < 0.8, gate=gate,
                    act="none" if gate == "none" else rng.choice(list(ACTS)), first=rng.random() < 0.5,
                    one_plus=rng.random() < 0.3, alpha=rng.choice([1.0, 0.22]))
    if op == "linear":
        hb = rng.choice([1, 1, 128, 512, 1024])
        K = max(hb, K // hb * hb)
    B = max(1, min(B, MOST // (N * K)))
    if op == "gated":
        return dict(op=op, B=B, N=N, K=K, act=rng.choice(["silu", "gelu"]))
    if op == "norm_linear":
        return dict(op=op, B=B, N=N, K=K)
    # T's sums round differently in another order, and a value next to the border of two 8-bit codes
    # then takes the other one: those outputs are bf16. Without T the codes are exact.
    return dict(op=op, B=B, N=N, K=K, hb=hb, x=rng.choice(["f32", "bf16"]),
                y="bf16" if hb > 1 else rng.choice(["f32", "bf16"]), bias=rng.random() < 0.5)


def _activations(g, B, K, dtype):
    """Token rows with 1% of the channels 20 times as large, as trained models have them."""
    gain = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return (torch.randn(B, K, generator=g, device="cuda") * gain).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, K = case["op"], case["B"], case["K"]
    s = {"case": case}
    if op in ("norm", "norm_linear"):
        c = case if op == "norm" else dict(y="bf16", h="bf16", gate="none", act="none", post=True, pre=True,
                                           first=False, one_plus=False, alpha=1.0)
        s["opt"] = c
        s["y"] = _activations(g, B, K, DTYPES[c["y"]])
        s["h"] = (_activations(g, B, K, torch.float32) * 4).to(DTYPES[c["h"]])
        s["gate"] = None
        if c["gate"] == "vector":
            s["gate"] = torch.randn(K, generator=g, device="cuda").to(DTYPES[c["y"]])
        elif c["gate"] == "rows":
            s["gate"] = torch.randn(B, K, generator=g, device="cuda").to(DTYPES[c["y"]])
        base = 0.0 if c["one_plus"] else 1.0
        s["w_post"] = base + 0.1 * torch.randn(K, generator=g, device="cuda")
        s["w_pre"] = base + 0.1 * torch.randn(K, generator=g, device="cuda")
    elif op == "gated":
        s["gate_up"] = torch.randn(B, 2 * K, generator=g, device="cuda").to(torch.bfloat16)
    else:
        s["x"] = _activations(g, B, K, DTYPES[case["x"]])
        s["c"] = 0.8 + 0.4 * torch.rand(K, generator=g, device="cuda") if case["hb"] > 1 else None
    if op != "norm":
        # 8-bit weights, rows padded to 16 bytes
        N, ld = case["N"], -(-K // 16) * 16
        s["w"] = torch.zeros(N, ld, dtype=torch.int8, device="cuda")[:, :K]
        step = max(1, (1 << 26) // K)
        for n in range(0, N, step):
            m = min(step, N - n)
            s["w"][n:n + m] = (torch.randn(m, K, generator=g, device="cuda") * 32).round_().clamp_(-127, 127).to(torch.int8)
        s["r"] = (0.5 + torch.rand(N, generator=g, device="cuda")) / (32 * math.sqrt(K))
        s["bias"] = torch.randn(N, generator=g, device="cuda") if case.get("bias") else None
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps next to its data: the layer's description, outputs and workspace."""
    import bit_matmul_amd as lq
    case = s["case"]
    op, B, K = case["op"], case["B"], case["K"]
    s["act"] = getattr(lq, "LQ_ACT_" + case.get("act", "none").upper())
    if "opt" in s:
        s["h_out"] = torch.empty(B, K, dtype=DTYPES[s["opt"]["h"]], device="cuda")
    if op == "norm":
        s["a"] = torch.empty(B, K, dtype=DTYPES[case["a"]], device="cuda") if case["pre"] else None
        return
    s["out"] = torch.empty(B, case["N"], dtype=DTYPES[case.get("y", "bf16")], device="cuda")
    s["layer"] = lq.int8_layer_struct(case["N"], K, s["w"], s["r"], hb=case.get("hb", 1), c=s.get("c"), bias=s["bias"])
    if op == "linear":
        n = lq.lq_int8_linear_workspace_size(s["layer"], B, s["x"].dtype)
    else:
        n = lq.lq_int8_gemm_workspace_size(s["layer"], B)
        s["q"] = torch.empty(B, -(-K // 16) * 16, dtype=torch.int8, device="cuda")[:, :K]
        s["scale"] = torch.empty(B, dtype=torch.float32, device="cuda")
    s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None


def _run_own(s):
    import bit_matmul_amd as lq
    case = s["case"]
    op, B, K = case["op"], case["B"], case["K"]
    if op == "linear":
        lq.lq_int8_linear(s["layer"], s["x"], B, s["out"], s["ws"])
        return s["out"]
    if op == "gated":
        lq.lq_quant_rows(s["gate_up"][:, K:], B, K, s["q"], s["scale"], gate=s["gate_up"][:, :K], act=s["act"])
        lq.lq_int8_gemm(s["layer"], s["q"], s["scale"], B, s["out"], s["ws"])
        return s["out"]
    o = s["opt"]
    lq.lq_norm_block(B, K, y=s["y"], gate=s["gate"], act=s["act"], gate_first=o["first"], post=o["post"],
                     w_post=s["w_post"] if o["post"] else None, h=s["h"], alpha=o["alpha"], h_out=s["h_out"],
                     pre=o["pre"], w_pre=s["w_pre"] if o["pre"] else None, one_plus=o["one_plus"], eps=EPS,
                     a=s.get("a"), q=s.get("q"), scale=s.get("scale"))
    if op == "norm":
        return {"h": s["h_out"], "a": s["a"]}
    lq.lq_int8_gemm(s["layer"], s["q"], s["scale"], B, s["out"], s["ws"])
    return {"h": s["h_out"], "y": s["out"]}


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


def _rows8(v):
    top = v.abs().amax(dim=1, keepdim=True)
    return torch.round(v * 127 / top), (top / 127).float()


def _product(q, scale, s, dtype):
    y = (q.float() @ s["w"].float().t()) * scale * s["r"]
    return (y if s["bias"] is None else y + s["bias"]).to(dtype)


def _norm(v, w, one_plus):
    v = v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)
    return v * (1 + w) if one_plus else v * w


def _block(s, o, as_real):
    """(h', the next block's input) in the type that as_real gives."""
    u = as_real(s["y"])
    gate = None if s["gate"] is None else ACTS[o["act"]](as_real(s["gate"]))
    if gate is not None and o["first"]:
        u = u * gate
    if o["post"]:
        u = _norm(u, as_real(s["w_post"]), o["one_plus"])
    if gate is not None and not o["first"]:
        u = u * gate
    h = as_real(s["h"]) + o["alpha"] * u
    return h, _norm(h, as_real(s["w_pre"]), o["one_plus"]) if o["pre"] else None


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    op, K = case["op"], case["K"]
    if op == "linear":
        # an 8-bit code next to a border is decided in 64 bits where x has 24; bf16 rows are exact in 32
        v = s["x"].double() if case["x"] == "f32" and case["hb"] == 1 else s["x"].float()
        if case["hb"] > 1:
            v = _whiten(v, s["c"], case["hb"])
        return _product(*_rows8(v), s, DTYPES[case["y"]])
    if op == "gated":
        v = ACTS[case["act"]](s["gate_up"][:, :K].float()) * s["gate_up"][:, K:].float()
        return _product(*_rows8(v), s, torch.bfloat16)
    h, a = _block(s, s["opt"], torch.Tensor.float)
    if op == "norm":
        return {"h": h.to(s["h"].dtype), "a": None if a is None else a.to(DTYPES[case["a"]])}
    return {"h": h.to(s["h"].dtype), "y": _product(*_rows8(a), s, torch.bfloat16)}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, K = case["op"], case["K"]

    def codes(v):
        m = v.abs().max(dim=1).values[:, None]
        t = v * 127 / m
        low = torch.floor(t)
        up = (t - low > 0.5) | ((t - low == 0.5) & (low.remainder(2) == 1))
        return low + up, m / 127

    def product(q, m):
        y = torch.matmul(q, s["w"].double().T.contiguous()) * (m * s["r"].double()[None, :])
        return y if s["bias"] is None else y + s["bias"].double()

    def rms(v, w, one_plus):
        n = torch.sqrt((v * v).sum(dim=1) / K + EPS)[:, None]
        return v / n * (w.double() + (1.0 if one_plus else 0.0))

    if op == "linear":
        v = s["x"].double()
        if case["hb"] > 1:
            i = torch.arange(case["hb"], device="cuda")
            parity = i[:, None] & i[None, :]
            for b in (8, 4, 2, 1):
                parity = parity ^ (parity >> b)
            H = (1 - 2 * (parity & 1)).double() / math.sqrt(case["hb"])
            v = torch.matmul((v * s["c"].double()).reshape(-1, case["hb"]), H).reshape(case["B"], K)
        return product(*codes(v))
    if op == "gated":
        g, u = s["gate_up"].double().split(K, dim=1)
        if case["act"] == "silu":
            v = g * torch.sigmoid(g) * u
        else:
            v = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)) * u
        return product(*codes(v))
    o = s["opt"]
    u, scale = s["y"].double(), 1.0
    if s["gate"] is not None:
        g = s["gate"].double()
        scale = {"none": lambda: g, "silu": lambda: g * torch.sigmoid(g), "sigmoid": lambda: torch.sigmoid(g),
                 "tanh": lambda: 1 - 2 / (torch.exp(2 * g) + 1),
                 "gelu": lambda: g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))}[o["act"]]()
    if o["post"]:
        u = rms(u * scale, s["w_post"], o["one_plus"]) if o["first"] else rms(u, s["w_post"], o["one_plus"]) * scale
    else:
        u = u * scale
    h = s["h"].double() + o["alpha"] * u
    a = rms(h, s["w_pre"], o["one_plus"]) if o["pre"] else None
    return {"h": h, "a": a} if op == "norm" else {"h": h, "y": product(*codes(a))}


def work(case):
    """Each input read once, each output written once; two operations for a multiply-add."""
    op, B, K = case["op"], case["B"], case["K"]
    size = {"f32": 4, "bf16": 2}
    if op in ("norm", "norm_linear"):
        o = dict(y="bf16", h="bf16", a=None, gate="none", post=True, pre=True) if op == "norm_linear" else case
        nbytes = B * K * (size[o["y"]] + 2 * size[o["h"]]) + 4 * K * (o["post"] + o["pre"])
        nbytes += {"none": 0, "vector": K, "rows": B * K}[o["gate"]] * size[o["y"]]
        flops = B * K * (3 + 4 * o["post"] + 4 * o["pre"])
        if op == "norm":
            return {"bytes": nbytes + (B * K * size[o["a"]] if o["pre"] else 0), "flops": flops}
    elif op == "gated":
        nbytes, flops = 4 * B * K, 8 * B * K
    else:
        nbytes = B * K * size[case["x"]] + (4 * K if case["hb"] > 1 else 0)
        flops = B * K * (3 + (1 + math.log2(case["hb"]) if case["hb"] > 1 else 0))
    N = case["N"]
    nbytes += N * K + 4 * N * (2 if case.get("bias") else 1) + B * N * size[case.get("y", "bf16")]
    return {"bytes": nbytes, "flops": flops + 2 * B * N * K}
