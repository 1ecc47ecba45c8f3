"""Cases of the 8-bit token path: quantizing rows, the int8 product, and the norms around a block.

The sizes are those of the Qwen3-4B-shaped layer this repository is measured on (hidden 2560,
q 4096, k and v 1024 each, MLP 9728; q/k/v and gate/up each stacked into one matrix), and odd ones.
`own` chooses between the operators' plain form in torch and the calls of this library.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HIDDEN, MLP, QKV, ATT = 2560, 9728, 6144, 4096


# ---------------------------------------------------------------- cases

def _gemm(M, N, K, y="f32", bias=False):
    return {"op": "gemm", "M": M, "N": N, "K": K, "y": y, "bias": bias}


def _quantize(M, K, x="bf16", gate=False):
    return {"op": "quantize", "M": M, "K": K, "x": x, "gate": gate}


def _norm(M, D, block="f32", residual="bf16", y="bf16", post=True, gate="none", offset=0.0, scale=1.0):
    """post: a norm after the block; gate: none, row (one vector for all tokens) or token."""
    return {"op": "norm", "M": M, "D": D, "block": block, "residual": residual, "y": y, "post": post, "gate": gate,
            "offset": offset, "scale": scale}


def listed():
    return [
        # attention output of one decoded token: latency, and 10.5 MB of weights
        {"name": "gemm o, 1 token", **_gemm(1, HIDDEN, ATT)},
        # stacked q/k/v of a decoded batch
        {"name": "gemm qkv, 32 tokens", **_gemm(32, QKV, HIDDEN, "bf16")},
        # down projection of a ragged piece of a prompt, split along its long K
        {"name": "gemm down, 333 tokens", **_gemm(333, HIDDEN, MLP)},
        # stacked gate/up of a whole prompt: the largest product of a layer
        {"name": "gemm gate_up, 4096 tokens", **_gemm(4096, 2 * MLP, HIDDEN, "bf16")},
        # nothing a multiple of anything: a small head with a bias, padded rows
        {"name": "gemm odd", **_gemm(77, 1003, 1259, "f16", True)},
        # input of the down projection of one token, from the product's fp32 outputs
        {"name": "quantize silu, 1 token", **_quantize(1, MLP, "f32", True)},
        # the same for a prompt
        {"name": "quantize silu, 4096 tokens", **_quantize(4096, MLP, "bf16", True)},
        # a weight matrix to 8 bits, one scale for each output channel
        {"name": "quantize up weights", **_quantize(MLP, HIDDEN, "f32")},
        # between two blocks of one decoded token, ready for the next product
        {"name": "norm i8, 1 token", **_norm(1, HIDDEN, "f32", "bf16", "i8", False)},
        # a decoded batch with norms on both sides of the block, weights stored as w - 1
        {"name": "norm sandwich, 64 tokens", **_norm(64, HIDDEN, "bf16", "bf16", "bf16", True, "none", 1.0)},
        # a prompt, the block's output gated for each channel and the residual scaled
        {"name": "norm gated, 8192 tokens", **_norm(8192, HIDDEN, "f32", "bf16", "bf16", True, "row", 0.0, 0.75)},
        # odd width, a gate for each token, residual in 32 bits
        {"name": "norm odd i8, 1001 tokens", **_norm(1001, 1237, "f16", "f32", "i8", True, "token")},
    ]


def _size(rng, lo, hi, odd=0.5):
    """A size spread over the logarithm of [lo, hi]; about half of them as they come, the others even."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd and n >= 32:
        n -= n % 16
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(("gemm", "gemm", "quantize", "norm", "norm"))
    if op == "gemm":
        while True:
            c = _gemm(_size(rng, 1, 4096), _size(rng, 64, 2 * MLP), _size(rng, 64, 16384), rng.choice(("f32", "bf16", "f16")),
                      rng.random() < 0.3)
            if c["M"] * c["N"] * c["K"] <= 4096 * 2 * MLP * HIDDEN:
                return c
    if op == "quantize":
        while True:
            c = _quantize(_size(rng, 1, 16384), _size(rng, 64, 32768), rng.choice(("f32", "bf16", "f16")), rng.random() < 0.5)
            if c["M"] * c["K"] <= 4096 * MLP:
                return c
    while True:
        c = _norm(_size(rng, 1, 8192), _size(rng, 64, 16384), rng.choice(("f32", "bf16", "f16")), rng.choice(("f32", "bf16", "f16")),
                  rng.choice(("f32", "bf16", "f16", "i8")), rng.random() < 0.6, rng.choice(("none", "row", "token")),
                  rng.choice((0.0, 1.0)), rng.choice((1.0, 0.75)))
        if c["M"] * c["D"] <= 8192 * HIDDEN:
            return c


# ---------------------------------------------------------------- inputs

def _pad16(n):
    return (n + 15) // 16 * 16


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _codes(g, rows, cols):
    """int8 rows as a quantizer leaves them (largest value 127), in rows padded to 16 bytes."""
    buf = torch.zeros(rows, _pad16(cols), dtype=torch.int8, device="cuda")
    q = buf[:, :cols]
    q.copy_((_normal(g, rows, cols) * 32).round_().clamp_(-127, 127))
    q.scatter_(1, torch.randint(0, cols, (rows, 1), device="cuda", generator=g), 127)
    return q


def _tokens(g, rows, cols):
    """Activations: a few channels far larger than the rest, tokens of different size."""
    v = _normal(g, rows, cols)
    v *= torch.where(torch.rand(cols, device="cuda", generator=g) < 0.01, 12.0, 1.0)
    v *= torch.exp(0.5 * _normal(g, rows, 1))
    return v


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["w"] = _codes(g, M, K), _codes(g, N, K)
        s["x_scale"] = torch.exp(0.5 * _normal(g, M)) * 0.03
        if M > 8:
            s["x_scale"][torch.randint(0, M, (1,), device="cuda", generator=g)] = 0   # a padding token
        s["w_scale"] = torch.exp(0.2 * _normal(g, N)) * 6e-4
        s["bias"] = _normal(g, N) if case["bias"] else None
        s["y"] = torch.empty(M, N, dtype=TYPES[case["y"]], device="cuda")
        return s
    if case["op"] == "quantize":
        M, D = case["M"], case["K"]
        t = TYPES[case["x"]]
        if case["gate"]:
            # the stacked gate/up product: its two halves are views of one buffer
            half = _pad16(D)
            both = torch.empty(M, 2 * half, dtype=t, device="cuda")
            s["gate"], s["x"] = both[:, :D], both[:, half:half + D]
            s["gate"].copy_(_tokens(g, M, D))
            s["x"].copy_(_tokens(g, M, D))
        else:
            s["gate"], s["x"] = None, (_normal(g, M, D) * 0.02).to(t)
        if M > 8:
            s["x"][torch.randint(0, M, (1,), device="cuda", generator=g)] = 0   # a padding token, a dead channel
        to_codes = True
    else:
        M, D = case["M"], case["D"]
        s["block"] = (_tokens(g, M, D) * 0.5).to(TYPES[case["block"]])
        s["residual"] = (_tokens(g, M, D) * 2).to(TYPES[case["residual"]])
        s["norm_weight"] = (1 - case["offset"] + 0.2 * _normal(g, D)).bfloat16()
        s["post_weight"] = (1 - case["offset"] + 0.2 * _normal(g, D)).bfloat16() if case["post"] else None
        rows = {"none": 0, "row": 1, "token": M}[case["gate"]]
        s["gate"] = torch.tanh(_normal(g, rows, D)).bfloat16() if rows else None
        s["residual_out"] = torch.empty_like(s["residual"])
        to_codes = case["y"] == "i8"
        if not to_codes:
            s["y"] = torch.empty(M, D, dtype=TYPES[case["y"]], device="cuda")
    if to_codes:
        s["y"] = torch.empty(M, _pad16(D), dtype=torch.int8, device="cuda")[:, :D]
        s["y_scale"] = torch.empty(M, dtype=torch.float32, device="cuda")
        # what the codes stand for: in 32 bits where the rows are given, in 16 where they are computed
        # (a value next to the border of two codes goes by the last bits of the arithmetic before it)
        given = case["op"] == "quantize" and not case["gate"]
        s["values"] = torch.empty(M, D, dtype=torch.float32 if given else torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

EPS = 1e-6


def run(s):
    op = s["case"]["op"]
    return _run_gemm(s) if op == "gemm" else _run_quantize(s) if op == "quantize" else _run_norm(s)


def _type(wr, t):
    return {torch.float32: wr.WR_F32, torch.bfloat16: wr.WR_BF16, torch.float16: wr.WR_F16, torch.int8: wr.WR_I8}[t.dtype]


def _run_gemm(s):
    c, x, w, y = s["case"], s["x"], s["w"], s["y"]
    if own:
        import bit_weight_only_wr_b200 as wr
        M, N, K = c["M"], c["N"], c["K"]
        if "workspace" not in s:   # kept by a program for as long as it keeps the weights
            s["workspace_bytes"] = wr.wr_gemm_i8_workspace_bytes(M, N, K)
            s["workspace"] = torch.zeros(max(16, s["workspace_bytes"]), dtype=torch.uint8, device="cuda")
        wr.wr_gemm_i8(M, N, K, x, x.stride(0), s["x_scale"], w, w.stride(0), s["w_scale"], _type(wr, y), y, N,
                      s["workspace"], s["workspace_bytes"], bias=s["bias"])
        return y
    out = (x.float() @ w.float().t()) * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(y.dtype)


def _plain_codes(v):
    """The codes of the rows of v (fp32) and their scales; which of two codes is decided in 64 bits."""
    big = v.abs().amax(1, keepdim=True)
    return torch.round(v.double() * 127 / torch.where(big > 0, big, 1).double()).float(), big / 127


def _run_quantize(s):
    c, x, gate, y = s["case"], s["x"], s["gate"], s["y"]
    if own:
        import bit_weight_only_wr_b200 as wr
        wr.wr_quantize_rows(_type(wr, x), c["M"], c["K"], x, x.stride(0), y, y.stride(0), s["y_scale"], gate=gate,
                            ldg=0 if gate is None else gate.stride(0))
        return {"values": torch.mul(y, s["y_scale"][:, None], out=s["values"]), "scale": s["y_scale"]}
    v = x.float()
    if gate is not None:
        g = gate.float()
        v = g / (1 + torch.exp(-g)) * v
    q, scale = _plain_codes(v)
    return {"values": torch.mul(q, scale, out=s["values"]), "scale": scale[:, 0]}


def _run_norm(s):
    c, b, h, y, gate = s["case"], s["block"], s["residual"], s["y"], s["gate"]
    to_codes = c["y"] == "i8"
    if own:
        import bit_weight_only_wr_b200 as wr
        D = c["D"]
        wr.wr_residual_norm(c["M"], D, block=b, ld_block=D, block_type=_type(wr, b), residual=h, ld_residual=D,
                            residual_out=s["residual_out"], ld_residual_out=D, residual_type=_type(wr, h),
                            post_weight=s["post_weight"], norm_weight=s["norm_weight"], weight_type=wr.WR_BF16,
                            weight_offset=c["offset"], gate=gate, ld_gate=D if c["gate"] == "token" else 0,
                            gate_type=wr.WR_BF16, residual_scale=c["scale"], eps=EPS, y=y, ld_y=y.stride(0),
                            y_type=_type(wr, y), y_scale=s["y_scale"] if to_codes else None)
        if to_codes:
            return {"residual": s["residual_out"], "scale": s["y_scale"],
                    "values": torch.mul(y, s["y_scale"][:, None], out=s["values"])}
        return {"residual": s["residual_out"], "y": y}
    b = b.float()
    if s["post_weight"] is not None:
        b = b / torch.sqrt((b * b).mean(1, keepdim=True) + EPS) * (s["post_weight"].float() + c["offset"])
    if gate is not None:
        b = b * gate.float()
    r = h.float() * c["scale"] + b
    v = r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS) * (s["norm_weight"].float() + c["offset"])
    if to_codes:
        q, scale = _plain_codes(v)
        return {"residual": r.to(h.dtype), "scale": scale[:, 0], "values": torch.mul(q, scale, out=s["values"])}
    return {"residual": r.to(h.dtype), "y": v.to(y.dtype)}


# ---------------------------------------------------------------- what it takes, and the definition

def work(case):
    """Bytes: every input read once, every output written once. A transcendental counts as one operation."""
    size = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * size[case["y"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if case["op"] == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * size[case["x"]] * (2 if case["gate"] else 1) + n + 4 * case["M"],
                "flops": n * (7 if case["gate"] else 3)}
    M, D = case["M"], case["D"]
    n = M * D
    gate = {"none": 0, "row": D, "token": n}[case["gate"]]
    vectors = 2 * D * (2 if case["post"] else 1) + 2 * gate
    return {"bytes": n * (size[case["block"]] + 2 * size[case["residual"]] + size[case["y"]]) + vectors +
            (4 * M if case["y"] == "i8" else 0), "flops": n * 10}


def _exact_codes(v):
    """Row by row: scale = largest value / 127, codes the nearest whole numbers (a tie to the even one)."""
    scale = v.abs().max(dim=1).values / 127
    safe = torch.where(scale == 0, torch.ones_like(scale), scale)
    # v / scale as v * 127 / largest, so that the quotient of the given values is the one that is rounded
    q = (v * 127).div(safe[:, None] * 127).round()
    return q * scale[:, None], scale


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: t.to(torch.float64) for k, t in s.items() if torch.is_tensor(t)}
    if case["op"] == "gemm":
        y = torch.einsum("mk,nk->mn", wide["x"], wide["w"])
        y = y.mul_(wide["x_scale"].unsqueeze(1)).mul_(wide["w_scale"].unsqueeze(0))
        return y if s["bias"] is None else y + wide["bias"]
    if case["op"] == "quantize":
        v = wide["x"]
        if s["gate"] is not None:
            v = v * wide["gate"] * torch.sigmoid(wide["gate"])
        values, scale = _exact_codes(v)
        return {"values": values, "scale": scale}

    def rms(v, weight):
        return v * torch.rsqrt(v.pow(2).sum(dim=-1, keepdim=True) / v.shape[-1] + EPS) * (weight + case["offset"])

    branch = wide["block"] if s["post_weight"] is None else rms(wide["block"], wide["post_weight"])
    if s["gate"] is not None:
        branch = branch * wide["gate"]
    residual = case["scale"] * wide["residual"] + branch
    y = rms(residual, wide["norm_weight"])
    if case["y"] == "i8":
        values, scale = _exact_codes(y)
        return {"residual": residual, "scale": scale, "values": values}
    return {"residual": residual, "y": y}
