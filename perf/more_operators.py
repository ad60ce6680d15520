"""Cases of the dense products beside the routed experts: what is timed, and what their outputs have to be.

Three operators, as the dense feed-forward blocks, projections and heads around a routed layer use them:

  norm to 8 bits     the block's norms, gate and residual scale with the next block's input quantised to
                     MXFP8 (E4M3 codes, one power of two per 32 values)
  matrix product     with bias, activation and residual in its epilogue, for one token or a chunk, with its
                     backward pass; operands in the activations' type, or x and the weight in MXFP8
  gated block        h = act(x Wg^T) * (x Wu^T), the gate's and the up projection's rows in one weight, with
                     its backward pass; the same operands, and h in MXFP8 for the next product

``own`` selects the framework's entry points; otherwise ``run`` computes the same outputs from elementary
torch operations in 32 bits.  ``exact`` is the definition in 64 bits.
"""
import functools
import math

import torch

own = False

EPS = 1e-5
RESIDUAL_SCALE = 0.7


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _norm(T, d, act, gate="none", post=True):
    return {"op": "norm_mx8", "T": T, "d": d, "act": act, "gate": gate, "post": post}


def _product(op, T, rows, cols, act, fn, mx8=False, bias=False, residual=False, h8=False, train=False):
    return {"op": op, "T": T, "rows": rows, "cols": cols, "act": act, "fn": fn, "mx8": mx8, "bias": bias,
            "residual": residual, "h8": h8, "train": train}


def listed():
    named = [
        # one decoded token between two blocks: the smallest call, latency
        ("norm_mx8_token", _norm(1, 4096, "bf16")),
        # a prefill chunk with an elementwise output gate, its normed rows the input of 8-bit products
        ("norm_mx8_chunk", _norm(4096, 4096, "bf16", gate="element")),
        # a square projection of one decoded token, onto the residual stream
        ("matmul_token", _product("matmul", 1, 4096, 4096, "bf16", "none", residual=True)),
        # a prefill or training chunk through a projection with everything in its epilogue
        ("matmul_chunk", _product("matmul", 4096, 4096, 4096, "bf16", "gelu", bias=True, residual=True)),
        # an odd fp32 prompt
        ("matmul_odd_f32", _product("matmul", 333, 6144, 2048, "f32", "silu", bias=True)),
        # the down projection of a prefill chunk in 8 bits, onto the residual stream
        ("matmul_chunk_mx8", _product("matmul", 4096, 4096, 8192, "bf16", "none", mx8=True, residual=True)),
        # a training chunk's gradients: input, weight and bias
        ("matmul_backward_chunk", _product("matmul_backward", 4096, 4096, 4096, "bf16", "gelu", bias=True)),
        # one decoded token through a dense block's gate and up projections
        ("gated_token", _product("gated", 1, 8192, 4096, "bf16", "silu")),
        # a batch of decoded tokens in 8 bits, h ready for the next 8-bit product
        ("gated_batch_mx8", _product("gated", 64, 8192, 4096, "bf16", "silu", mx8=True, h8=True)),
        # a training chunk, with what its backward pass needs
        ("gated_chunk", _product("gated", 4096, 8192, 4096, "bf16", "silu", train=True)),
        # the backward pass of that chunk
        ("gated_backward_chunk", _product("gated_backward", 4096, 8192, 4096, "bf16", "silu")),
        # fp32 training of a short odd batch of a small model
        ("gated_backward_odd_f32", _product("gated_backward", 777, 1536, 640, "f32", "gelu")),
    ]
    return [{"name": n} | c for n, c in named]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: T * rows * cols at most: the largest listed case's, for each kind
_MOST = {"norm_mx8": 4096 * 4096, "matmul": 4096 * 4096 * 8192, "matmul_backward": 4096 * 4096 * 4096,
         "gated": 4096 * 8192 * 4096, "gated_backward": 4096 * 8192 * 4096}


def draw(rng):
    op = rng.choice(["norm_mx8", "matmul", "matmul", "matmul_backward", "gated", "gated", "gated_backward"])
    act = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "norm_mx8":
        d = 128 * rng.randint(1, 48)
        T = min(_log(rng, 1, 4096), _MOST[op] * 2 // (d * (4 if act == "f32" else 2)))
        return _norm(T, d, act, rng.choice(["none", "token", "element"]), rng.random() < 0.75)
    mx8 = op in ("matmul", "gated") and rng.random() < 0.4
    rows, cols = 32 * _log(rng, 1, 256), 32 * _log(rng, 1, 256)
    if not mx8:     # rows and columns that end inside a tile
        rows, cols = rows - 8 * rng.randint(0, 3), cols - 8 * rng.randint(0, 3)
    T = _log(rng, 1, 4096)
    most = _MOST[op] // (8 if act == "f32" and not mx8 else 1)
    T = max(1, min(T, most // (rows * cols)))
    gated = op.startswith("gated")
    return _product(op, T, rows, cols, act, rng.choice(["silu", "gelu", "sigmoid"] if gated else ["none", "silu", "gelu", "sigmoid"]),
                    mx8=mx8, bias=not gated and rng.random() < 0.5, residual=op == "matmul" and rng.random() < 0.5,
                    h8=gated and mx8 and rng.random() < 0.5, train=op == "gated" and not mx8 and rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["act"] == "bf16" else torch.float32


def _normal(g, *size, dtype=torch.float32, std=1.0):
    return (torch.randn(*size, generator=g, device="cuda") * std).to(dtype)


def _quantise(v):
    """MXFP8 of fp32 rows: E4M3 codes and scale bytes (2^(b - 127)), the scale of a block of 32 values
    2^(floor(log2 max) - 7), exponent at least -126."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top).exponent - 8, -126).clamp(min=-126)
    codes = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).reshape(v.shape)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    op, T, dt = case["op"], case["T"], _dtype(case)
    s = {"case": case}
    if op == "norm_mx8":
        d = case["d"]
        s["x"], s["y"] = _normal(g, T, d, dtype=dt, std=2.0), _normal(g, T, d, dtype=dt, std=0.5)
        s["pre_gamma"] = 1 + _normal(g, d, std=0.1)
        s["post_gamma"] = 1 + _normal(g, d, std=0.1) if case["post"] else None
        s["gate"] = {"none": lambda: None, "token": lambda: torch.sigmoid(_normal(g, T)),
                     "element": lambda: torch.sigmoid(_normal(g, T, d)).to(dt)}[case["gate"]]()
        s["x_out"] = torch.empty(T, d, dtype=dt, device="cuda")
        s["codes"] = torch.empty(T, d, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(T, d // 32, dtype=torch.float8_e8m0fnu, device="cuda")
        return s
    N, K = case["rows"], case["cols"]
    gated = op.startswith("gated")
    R = 2 * N if gated else N
    if case["mx8"]:
        s["x"], s["xs"] = _quantise(_normal(g, T, K))
        s["w"], s["ws"] = _quantise(_normal(g, R, K, std=0.02))
    else:
        s["x"], s["xs"] = _normal(g, T, K, dtype=dt), None
        s["w"], s["ws"] = _normal(g, R, K, dtype=dt, std=0.02), None
    s["bias"] = _normal(g, N, std=0.1) if case["bias"] else None
    if op in ("matmul", "gated"):
        s["residual"] = _normal(g, T, N, dtype=dt) if case["residual"] else None
        s["pre"] = torch.empty(T, R, dtype=dt, device="cuda") if case["train"] else None
        s["y"] = torch.empty(T, N, dtype=torch.float8_e4m3fn if case["h8"] else dt, device="cuda")
        s["ys"] = torch.empty(T, N // 32, dtype=torch.float8_e8m0fnu, device="cuda") if case["h8"] else None
        return s
    # what the forward pass kept: pre-activations of the products' usual size
    s["pre"] = _normal(g, T, R, dtype=dt) if gated or case["fn"] != "none" else None
    s["dy"] = _normal(g, T, N, dtype=dt)
    s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    s["d_bias"] = torch.empty(N, device="cuda") if case["bias"] else None
    return s


# ---------------------------------------------------------------------------------------------
# the operators: the framework's entry points
# ---------------------------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _shape(d, act):
    import routed_expert_ffn_router_amd as m
    return m.make_shape(d, 128, 1, 1, m.MOE_WF_MXFP4, m.MOE_DT_BF16 if act == "bf16" else m.MOE_DT_F32)


@functools.lru_cache(maxsize=8)
def _dense(op, T, rows, cols, act, fn, mx8):
    """The products' description, and a workspace for T tokens, which a program keeps."""
    import routed_expert_ffn_router_amd as m
    dense = m.make_dense(rows, cols, m.MOE_DT_BF16 if act == "bf16" else m.MOE_DT_F32,
                         m.MOE_OPERANDS_MXFP8 if mx8 else m.MOE_OPERANDS_ACT,
                         {"none": m.MOE_ACT_NONE, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU, "sigmoid": m.MOE_ACT_SIGMOID}[fn])
    return dense, m.dense_workspace(dense, T)


def _run_own(s):
    import routed_expert_ffn_router_amd as m
    c = s["case"]
    op, T = c["op"], c["T"]
    if op == "norm_mx8":
        kind = {"none": m.MOE_GATE_NONE, "token": m.MOE_GATE_TOKEN, "element": m.MOE_GATE_ELEMENT}[c["gate"]]
        m.moe_block_norm_mx8(_shape(c["d"], c["act"]), s["x"], s["y"], T, s["post_gamma"], s["pre_gamma"], s["gate"], kind,
                             RESIDUAL_SCALE, EPS, s["x_out"], s["codes"], s["scales"])
        return {"x_out": s["x_out"], "codes": s["codes"], "scales": s["scales"]}
    dense, scratch = _dense(op, T, c["rows"], c["cols"], c["act"], c["fn"], c["mx8"])
    if op == "matmul":
        m.moe_matmul(dense, s["x"], s["xs"], T, s["w"], s["ws"], s["bias"], s["residual"], None, s["y"], scratch)
        return s["y"]
    if op == "gated":
        m.moe_gated(dense, s["x"], s["xs"], T, s["w"], s["ws"], s["pre"], s["y"], s["ys"], scratch)
        return {"h": s["y"], "scales": s["ys"], "pre": s["pre"]}
    if op == "matmul_backward":
        m.moe_matmul_backward(dense, s["x"], T, s["w"], s["pre"], s["dy"], s["dx"], s["dw"], s["d_bias"], scratch)
        return {"dx": s["dx"], "dw": s["dw"], "d_bias": s["d_bias"]}
    m.moe_gated_backward(dense, s["x"], T, s["w"], s["pre"], s["dy"], s["dx"], s["dw"], scratch)
    return {"dx": s["dx"], "dw": s["dw"]}


# ---------------------------------------------------------------------------------------------
# the operators: plain form, 32 bits
# ---------------------------------------------------------------------------------------------

def _values(codes, scales):
    """fp32 values of an operand: as given, or MXFP8 codes times their blocks' scales."""
    if scales is None:
        return codes.float()
    return (codes.float().reshape(*scales.shape, 32) * scales.float()[..., None]).reshape(codes.shape)


def _activation(fn, v):
    if fn == "none":
        return v
    if fn == "silu":
        return v * torch.sigmoid(v)
    if fn == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return torch.sigmoid(v)


def _slope(fn, v):
    """The activation's derivative."""
    if fn == "none":
        return torch.ones_like(v)
    if fn == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    p = torch.sigmoid(v)
    return p * (1 + v * (1 - p)) if fn == "silu" else p * (1 - p)


def _plain_norm(s, dt):
    y = s["y"].float()
    z = y if s["post_gamma"] is None else y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["post_gamma"]
    if s["gate"] is not None:
        z = z * (s["gate"][:, None] if s["gate"].dim() == 1 else s["gate"].float())
    u = s["x"].float() + RESIDUAL_SCALE * z
    codes, scales = _quantise(u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s["pre_gamma"])
    return {"x_out": u.to(dt), "codes": codes, "scales": scales}


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op, dt, fn = c["op"], _dtype(c), c.get("fn")
    if op == "norm_mx8":
        return _plain_norm(s, dt)
    x, w = _values(s["x"], s["xs"]), _values(s["w"], s["ws"])
    N = c["rows"]
    if op == "matmul":
        v = x @ w.t()
        if s["bias"] is not None:
            v = v + s["bias"]
        v = _activation(fn, v)
        return (v if s["residual"] is None else v + s["residual"].float()).to(dt)
    if op == "gated":
        v = x @ w.t()
        h, scales = _activation(fn, v[:, :N]) * v[:, N:], None
        if c["h8"]:
            h, scales = _quantise(h)
        return {"h": h if c["h8"] else h.to(dt), "scales": scales, "pre": v.to(dt) if c["train"] else None}
    dy = s["dy"].float()
    if op == "matmul_backward":
        d = dy if fn == "none" else dy * _slope(fn, s["pre"].float())
    else:
        a, b = s["pre"][:, :N].float(), s["pre"][:, N:].float()
        d = torch.cat([dy * b * _slope(fn, a), dy * _activation(fn, a)], 1)
    out = {"dx": (d @ w).to(dt), "dw": (d.t() @ x).to(dt)}
    if op == "matmul_backward":
        out["d_bias"] = d.sum(0) if c["bias"] else None
    return out


# ---------------------------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    es = 2 if case["act"] == "bf16" else 4
    if op == "norm_mx8":
        d = case["d"]
        gate = {"none": 0, "token": 4 * T, "element": T * d * es}[case["gate"]]
        return {"bytes": 3 * T * d * es + T * d * (1 + 1 / 32) + gate + 4 * d * (2 if case["post"] else 1), "flops": 14.0 * T * d}
    N, K = case["rows"], case["cols"]
    R = 2 * N if op.startswith("gated") else N
    unit = 1 + 1 / 32 if case["mx8"] else es
    operands = (T * K + R * K) * unit
    flops = 2.0 * T * R * K
    if op in ("matmul", "gated"):
        out = T * N * (1 + 1 / 32 if case["h8"] else es) + (T * R * es if case["train"] else 0)
        return {"bytes": operands + out + (4 * N if case["bias"] else 0) + (T * N * es if case["residual"] else 0), "flops": flops}
    kept = T * R * es if R > N or case["fn"] != "none" else 0
    return {"bytes": 2 * operands + T * N * es + kept + (4 * N if case["bias"] else 0), "flops": 2 * flops}


def _exact_values(t, scales):
    """Values in 64 bits; MXFP8 from the bit fields of its codes and scales."""
    if scales is None:
        return t.double()
    q = t.view(torch.uint8).to(torch.int32)
    e, man = q // 8 % 16, (q % 8).double()
    v = torch.where(e == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * 2.0 ** (e.double() - 7)) * (1.0 - 2.0 * (q // 128).double())
    return v * (2.0 ** (scales.view(torch.uint8).double() - 127)).repeat_interleave(32, 1)


def _phi(v):
    return torch.special.ndtr(v)


def _logistic(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _exact_activation(fn, v):
    return {"none": lambda: v, "silu": lambda: v / (1 + torch.exp(-v)), "gelu": lambda: v * _phi(v), "sigmoid": lambda: _logistic(v)}[fn]()


def _exact_slope(fn, v):
    p = _logistic(v)
    return {"none": lambda: torch.ones_like(v), "silu": lambda: p + v * p * _logistic(-v),
            "gelu": lambda: _phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi), "sigmoid": lambda: p * _logistic(-v)}[fn]()


def _codes_before_rounding(v):
    """What the 8-bit codes stand for before they are rounded: the values over their blocks' scales."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 7
    return (b * 2.0 ** -e.clamp(min=-126)).reshape(v.shape)


def exact(case, seed):
    # (scales are powers of two, which a value next to one may turn over: they have no value to be near to)
    s = prepare(case, seed)
    op, fn = case["op"], case.get("fn")
    if op == "norm_mx8":
        x, y, d = s["x"].double(), s["y"].double(), case["d"]
        if s["post_gamma"] is not None:
            y = s["post_gamma"].double() * y / (y.square().sum(1, keepdim=True) / d + EPS).sqrt()
        gate = 1.0 if s["gate"] is None else s["gate"].double().reshape(case["T"], -1)
        u = x + RESIDUAL_SCALE * gate * y
        n = s["pre_gamma"].double() * u / (u.square().sum(1, keepdim=True) / d + EPS).sqrt()
        return {"x_out": u, "codes": _codes_before_rounding(n), "scales": None}
    x, w, N = _exact_values(s["x"], s["xs"]), _exact_values(s["w"], s["ws"]), case["rows"]
    if op in ("matmul", "gated"):
        v = torch.matmul(x, w.t().contiguous())
        if op == "matmul":
            v = _exact_activation(fn, v if s["bias"] is None else v + s["bias"].double())
            return v if s["residual"] is None else v + s["residual"].double()
        h = _exact_activation(fn, v[:, :N]) * v[:, N:]
        return {"h": _codes_before_rounding(h) if case["h8"] else h, "scales": None, "pre": v if case["train"] else None}
    dy = s["dy"].double()
    pre = None if s["pre"] is None else s["pre"].double()
    if op == "matmul_backward":
        d = dy if pre is None else dy * _exact_slope(fn, pre)
    else:
        d = torch.cat([dy * pre[:, N:] * _exact_slope(fn, pre[:, :N]), dy * _exact_activation(fn, pre[:, :N])], 1)
    out = {"dx": torch.matmul(d, w), "dw": torch.matmul(d.t().contiguous(), x)}
    if op == "matmul_backward":
        out["d_bias"] = d.sum(0) if case["bias"] else None
    return out
