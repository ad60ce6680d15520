"""Cases of the operators around the routed experts: what is timed, and what their outputs have to be.

Three groups, as a block of a mixture-of-experts model uses them:

  tokens by expert and back    dispatch (rows of x to the sorted positions), and the backward pass of
                               dispatch and of the route-weighted combine
  norms around the block       the block's post-norm with its gate and residual scale, and the next
                               pre-norm, alone or fused with the combine, and their backward pass
  4-bit matrix-vector products the dense projections beside the experts, in the experts' weight formats

``own`` selects the framework's entry points; otherwise ``run`` computes the same outputs from elementary
torch operations in 32 bits.  ``exact`` is the definition in 64 bits.
"""
import functools
import math

import torch

own = False

EPS = 1e-5
RESIDUAL_SCALE = 0.7
ROUTED_SCALING = 2.5


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _sort(op, T, d, k, E, act, shared=False, drop=False):
    return {"op": op, "T": T, "d": d, "k": k, "E": E, "act": act, "shared": shared, "drop": drop}


def _norm(op, T, d, act, gate="none", post=True):
    return {"op": op, "T": T, "d": d, "act": act, "gate": gate, "post": post}


def _linear(rows, cols, wf, act, T, bias=False):
    return {"op": "linear", "rows": rows, "cols": cols, "wf": wf, "act": act, "T": T, "bias": bias}


def listed():
    named = [
        # one decoded token's eight rows: the smallest call, launch latency
        ("dispatch_token", _sort("dispatch", 1, 4096, 8, 288, "bf16")),
        # a prefill or training chunk's rows, laid out for the experts
        ("dispatch_chunk", _sort("dispatch", 4096, 4096, 8, 288, "bf16")),
        # the backward pass over the same chunk
        ("sort_backward_chunk", _sort("sort_backward", 4096, 4096, 8, 288, "bf16")),
        # fp32 training on a short odd batch, with a shared expert and picks that the router dropped
        ("sort_backward_odd_f32", _sort("sort_backward", 333, 6144, 8, 256, "f32", shared=True, drop=True)),
        # one decoded token between two blocks: latency
        ("block_norm_token", _norm("block_norm", 1, 4096, "bf16")),
        # a prefill chunk with an elementwise output gate
        ("block_norm_chunk", _norm("block_norm", 4096, 4096, "bf16", gate="element")),
        # the end of the layer for a batch of decoded tokens: combine, post-norm, residual, next pre-norm
        ("combine_norm_batch", _sort("combine_norm", 64, 4096, 8, 288, "bf16", shared=True) | {"gate": "none", "post": True}),
        # the same for an odd fp32 prompt with a gate for each token and dropped picks
        ("combine_norm_odd_f32", _sort("combine_norm", 1001, 6144, 8, 256, "f32", drop=True) | {"gate": "token", "post": True}),
        # training chunk: gradients of both streams, the gate and both norm weights
        ("norm_backward_chunk", _norm("norm_backward", 4096, 4096, "bf16", gate="element")),
        # a short odd fp32 batch of a small model
        ("norm_backward_odd_f32", _norm("norm_backward", 77, 640, "f32", gate="token")),
        # a square projection for one decoded token
        ("linear_token_mxfp4", _linear(4096, 4096, "mxfp4", "bf16", 1)),
        # an output head for a small batch of decoded tokens
        ("linear_head_nvfp4", _linear(65536, 6144, "nvfp4", "bf16", 16)),
    ]
    return [{"name": n} | c for n, c in named]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "sort_backward", "block_norm", "combine_norm", "norm_backward", "linear"])
    act = rng.choice(["bf16", "bf16", "f32"])
    d = 128 * rng.randint(1, 48)
    if op == "linear":
        return _linear(_log(rng, 1, 65536), d, rng.choice(["mxfp4", "nvfp4"]), act, _log(rng, 1, 16), rng.random() < 0.5)
    size = 4 if act == "f32" else 2
    if op in ("block_norm", "norm_backward"):
        T = min(_log(rng, 1, 4096), 4096 * 4096 * 2 // (d * size))
        return _norm(op, T, d, act, rng.choice(["none", "token", "element"]), rng.random() < 0.75)
    k = rng.randint(1, 8)
    E = _log(rng, k, 512)
    most = 8 * 4096 * 4096 * 2 if op != "combine_norm" else 1000 * 6144 * 4 * 4
    T = max(1, min(_log(rng, 1, 4096), most // (d * size * (k + 1))))
    c = _sort(op, T, d, k, E, act, rng.random() < 0.4, rng.random() < 0.4)
    return c | {"gate": rng.choice(["none", "token", "element"]), "post": True} if op == "combine_norm" else c


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _dtype(case):
    return torch.bfloat16 if case["act"] == "bf16" else torch.float32


def _normal(g, *size, dtype=torch.float32, std=1.0):
    return (torch.randn(*size, generator=g, device="cuda") * std).to(dtype)


def _routing(case, g):
    """Distinct experts for each token, weights that sum to 1 and the grouping of the picks by expert, with
    the last ranks of some tokens dropped (id -1) where the case says so."""
    T, k, E = case["T"], case["k"], case["E"]
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k]
    w = torch.rand(T, k, generator=g, device="cuda") + 0.05
    if case["drop"]:
        kept = 1 + (7 * torch.arange(T, device="cuda")) % k
        gone = torch.arange(k, device="cuda")[None] >= kept[:, None]
        idx = torch.where(gone, -1, idx)
        w = torch.where(gone, 0.0, w)
    w = w / w.sum(1, keepdim=True)
    flat = torch.where(idx < 0, E, idx).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    real = flat[order] < E
    sorted_pick = torch.where(real, order, -1)
    pick_pos = torch.empty_like(order)
    pick_pos[order] = torch.where(real, torch.arange(T * k, device="cuda"), -1)
    return w, sorted_pick.to(torch.int32), pick_pos.to(torch.int32).reshape(T, k)


def _norm_inputs(case, g):
    T, d, dt = case["T"], case["d"], _dtype(case)
    s = {"pre_gamma": 1 + _normal(g, d, std=0.1), "post_gamma": 1 + _normal(g, d, std=0.1) if case["post"] else None, "gate": None}
    if case["gate"] == "token":
        s["gate"] = torch.sigmoid(_normal(g, T))
    elif case["gate"] == "element":
        s["gate"] = torch.sigmoid(_normal(g, T, d)).to(dt)
    return s


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantised(case, g):
    """Weights N(0, 0.02) in the block formats: packed codes, scale bytes, tensor scale."""
    N, K = case["rows"], case["cols"]
    B = 32 if case["wf"] == "mxfp4" else 16
    ts = 1.0 if B == 32 else 0.02 * 5.5 / (448 * 6)
    middles = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    q = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(N, K // B, dtype=torch.uint8, device="cuda")
    for a in range(0, N, 16384):
        v = _normal(g, min(16384, N - a), K // B, B, std=0.02)
        top = v.abs().amax(-1)
        if B == 32:
            e = torch.frexp(top).exponent - 1 - 2
            s[a:a + 16384] = (e + 127).clamp(0, 254).to(torch.uint8)
            scale = torch.ldexp(torch.ones_like(top), e)
        else:
            f8 = (top / (6 * ts)).clamp(max=448).to(torch.float8_e4m3fn)
            s[a:a + 16384] = f8.view(torch.uint8)
            scale = f8.float() * ts
        v = v / scale.clamp(min=1e-30)[..., None]
        code = torch.bucketize(v.abs(), middles).to(torch.uint8) | (v < 0).to(torch.uint8) << 3
        code = code.reshape(-1, K)
        q[a:a + 16384] = code[:, 0::2] | code[:, 1::2] << 4
    return q, s, ts


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    op, dt = case["op"], _dtype(case)
    s = {"case": case}
    if op == "linear":
        T, N, K = case["T"], case["rows"], case["cols"]
        s["q"], s["s"], s["ts"] = _quantised(case, g)
        s["x"] = _normal(g, T, K, dtype=dt)
        s["bias"] = _normal(g, N, std=0.1) if case["bias"] else None
        s["y"] = torch.empty(T, N, dtype=dt, device="cuda")
        return s
    T, d = case["T"], case["d"]
    if op in ("dispatch", "sort_backward", "combine_norm"):
        k = case["k"]
        rows = T * k + (T if case["shared"] else 0)
        s["w"], s["sorted_pick"], s["pick_pos"] = _routing(case, g)
        if op == "dispatch":
            s["x"] = _normal(g, T, d, dtype=dt)
            s["xs"] = torch.zeros(rows, d, dtype=dt, device="cuda")
            return s
        s["o"] = _normal(g, rows, d, std=0.5)
        if op == "sort_backward":
            s["dy"] = _normal(g, T, d, dtype=dt)
            s["dxs"] = _normal(g, rows, d, dtype=dt)
            s["dx"] = torch.empty(T, d, dtype=dt, device="cuda")
            s["d_o"] = torch.zeros(rows, d, device="cuda")
            s["d_w"] = torch.empty(T, k, device="cuda")
            return s
    s |= _norm_inputs(case, g)
    s["x"] = _normal(g, T, d, dtype=dt, std=2.0)
    if op != "combine_norm":
        s["y"] = _normal(g, T, d, dtype=dt, std=0.5)
    if op != "norm_backward":
        s["x_out"] = torch.empty(T, d, dtype=dt, device="cuda")
        s["normed"] = torch.empty(T, d, dtype=dt, device="cuda")
        return s
    s["d_x_out"] = _normal(g, T, d, dtype=dt)
    s["d_normed"] = _normal(g, T, d, dtype=dt)
    s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    s["d_gate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    s["d_pre"] = torch.empty(d, device="cuda")
    s["d_post"] = torch.empty(d, device="cuda") if case["post"] else None
    # the layer's workspace for this many tokens, with room to spare
    s["ws"] = torch.zeros((64 << 20) + 10 * T * d, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# the operators: the framework's entry points
# ---------------------------------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _shape(d, k, E, act, shared):
    import routed_expert_ffn_router_amd as m
    return m.make_shape(d, 128, E, k, m.MOE_WF_MXFP4, m.MOE_DT_BF16 if act == "bf16" else m.MOE_DT_F32,
                        routed_scaling=ROUTED_SCALING, n_shared=int(shared))


@functools.lru_cache(maxsize=None)
def _matrix(rows, cols, wf, act):
    import routed_expert_ffn_router_amd as m
    return m.make_matrix(rows, cols, m.MOE_WF_MXFP4 if wf == "mxfp4" else m.MOE_WF_NVFP4,
                         m.MOE_DT_BF16 if act == "bf16" else m.MOE_DT_F32)


def _run_own(s):
    import routed_expert_ffn_router_amd as m
    c = s["case"]
    op, T = c["op"], c["T"]
    if op == "linear":
        m.moe_linear(_matrix(c["rows"], c["cols"], c["wf"], c["act"]), s["q"], s["s"], s["ts"], s["x"], T, s["bias"], s["y"])
        return s["y"]
    sh = _shape(c["d"], c.get("k", 1), c.get("E", 1), c["act"], c.get("shared", False))
    if op == "dispatch":
        m.moe_dispatch(sh, s["x"], T, s["pick_pos"], s["xs"])
        return s["xs"]
    if op == "sort_backward":
        m.moe_combine_backward(sh, s["dy"], s["o"], s["w"], s["pick_pos"], T, s["d_o"], s["d_w"])
        m.moe_dispatch_backward(sh, s["dxs"], T, s["pick_pos"], s["dx"])
        return {"d_o": s["d_o"], "d_w": s["d_w"], "dx": s["dx"]}
    kind = {"none": m.MOE_GATE_NONE, "token": m.MOE_GATE_TOKEN, "element": m.MOE_GATE_ELEMENT}[c["gate"]]
    if op == "block_norm":
        m.moe_block_norm(sh, s["x"], s["y"], T, s["post_gamma"], s["pre_gamma"], s["gate"], kind, RESIDUAL_SCALE, EPS,
                         s["x_out"], s["normed"])
        return {"x_out": s["x_out"], "normed": s["normed"]}
    if op == "combine_norm":
        m.moe_combine_norm(sh, s["o"], s["w"], s["pick_pos"], s["x"], T, s["post_gamma"], s["pre_gamma"], s["gate"], kind,
                           RESIDUAL_SCALE, EPS, s["x_out"], s["normed"])
        return {"x_out": s["x_out"], "normed": s["normed"]}
    m.moe_block_norm_backward(sh, s["x"], s["y"], T, s["post_gamma"], s["pre_gamma"], s["gate"], kind, RESIDUAL_SCALE, EPS,
                              s["d_x_out"], s["d_normed"], s["dx"], s["dy"], s["d_gate"], s["d_post"], s["d_pre"], s["ws"])
    return {k: s[k] for k in ("dx", "dy", "d_gate", "d_post", "d_pre")}


# ---------------------------------------------------------------------------------------------
# the operators: plain form, 32 bits
# ---------------------------------------------------------------------------------------------

def _picked(rows, pick_pos):
    """[T, k, d] in 32 bits: the row at each pick's position, zero for a dropped pick."""
    got = rows.float()[pick_pos.long().clamp(min=0)]
    return torch.where((pick_pos >= 0)[..., None], got, 0.0)


def _rms(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _gate32(s):
    g = s["gate"]
    return 1.0 if g is None else g[:, None] if s["case"]["gate"] == "token" else g.float()


def _plain_norm(s, y, dt):
    z = y if s["post_gamma"] is None else y * _rms(y) * s["post_gamma"]
    u = s["x"].float() + RESIDUAL_SCALE * _gate32(s) * z
    return {"x_out": u.to(dt), "normed": (u * _rms(u) * s["pre_gamma"]).to(dt)}


def _plain_combine(s, c):
    y = ROUTED_SCALING * (s["w"][..., None] * _picked(s["o"], s["pick_pos"])).sum(1)
    return y + s["o"][c["T"] * c["k"]:] if c["shared"] else y


def _plain_linear(s, c, dt):
    N, K, B = c["rows"], c["cols"], 32 if c["wf"] == "mxfp4" else 16
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device="cuda")
    code = torch.stack([s["q"] & 15, s["q"] >> 4], -1).reshape(N, K // B, B)
    if B == 32:
        scale = torch.ldexp(torch.ones((), device="cuda"), s["s"].int() - 127)
    else:
        scale = s["s"].view(torch.float8_e4m3fn).float()
    weight = (table[code.int()] * scale[..., None]).reshape(N, K)
    y = s["x"].float() @ weight.t() * s["ts"]
    return (y if s["bias"] is None else y + s["bias"]).to(dt)


def _plain_norm_backward(s, c, dt):
    x, y, gate, a = s["x"].float(), s["y"].float(), _gate32(s), RESIDUAL_SCALE
    post = s["post_gamma"] is not None
    ry = _rms(y) if post else 1.0
    yn = y * ry
    z = yn * s["post_gamma"] if post else y
    u = x + a * gate * z
    ru = _rms(u)
    un = u * ru
    dn = s["d_normed"].float()
    dun = dn * s["pre_gamma"]
    du = s["d_x_out"].float() + ru * (dun - un * (dun * un).mean(-1, keepdim=True))
    dz = a * gate * du
    if post:
        dyn = dz * s["post_gamma"]
        dy = ry * (dyn - yn * (dyn * yn).mean(-1, keepdim=True))
    else:
        dy = dz
    d_gate = {"none": lambda: None, "token": lambda: a * (du * z).sum(-1), "element": lambda: (a * du * z).to(dt)}[c["gate"]]()
    return {"dx": du.to(dt), "dy": dy.to(dt), "d_gate": d_gate, "d_post": (dz * yn).sum(0) if post else None,
            "d_pre": (dn * un).sum(0)}


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op, dt = c["op"], _dtype(c)
    if op == "linear":
        return _plain_linear(s, c, dt)
    if op == "block_norm":
        return _plain_norm(s, s["y"].float(), dt)
    if op == "norm_backward":
        return _plain_norm_backward(s, c, dt)
    if op == "combine_norm":
        return _plain_norm(s, _plain_combine(s, c), dt)
    kept = (s["sorted_pick"] >= 0)[:, None]
    pick = s["sorted_pick"].long().clamp(min=0)
    token = pick // c["k"]
    if op == "dispatch":
        xs = torch.where(kept, s["x"][token], 0.0)
        return torch.cat([xs, s["x"]]) if c["shared"] else xs
    dy = s["dy"].float()
    d_o = torch.where(kept, ROUTED_SCALING * s["w"].reshape(-1)[pick][:, None] * dy[token], 0.0)
    d_w = ROUTED_SCALING * (_picked(s["o"], s["pick_pos"]) * dy[:, None]).sum(-1)
    dx = _picked(s["dxs"], s["pick_pos"]).sum(1)
    if c["shared"]:
        d_o = torch.cat([d_o, dy])
        dx = dx + s["dxs"][c["T"] * c["k"]:].float()
    return {"d_o": d_o, "d_w": d_w, "dx": dx.to(dt)}


# ---------------------------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    es = 2 if case["act"] == "bf16" else 4
    if op == "linear":
        N, K = case["rows"], case["cols"]
        per = 1 / 32 if case["wf"] == "mxfp4" else 1 / 16
        return {"bytes": N * K * (0.5 + per) + es * T * (K + N) + (4 * N if case["bias"] else 0), "flops": 2.0 * N * K * T}
    d = case["d"]
    row = d * es
    if "k" in case:
        k = case["k"]
        n = sum(1 + 7 * t % k for t in range(T)) if case["drop"] else T * k
        rows = n + (T if case["shared"] else 0)
        if op == "dispatch":
            return {"bytes": T * row + rows * row + 4 * T * k, "flops": 0}
        if op == "sort_backward":
            return {"bytes": 2 * T * row + rows * row + n * d * 4 + rows * d * 4 + 12 * T * k, "flops": 4.0 * n * d}
    gate = {"none": 0, "token": 4 * T, "element": T * row}[case["gate"]]
    gammas = 4 * d * (2 if case["post"] else 1)
    if op == "combine_norm":
        return {"bytes": rows * d * 4 + 8 * T * k + 3 * T * row + gate + gammas, "flops": 2.0 * rows * d + 12.0 * T * d}
    if op == "block_norm":
        return {"bytes": 4 * T * row + gate + gammas, "flops": 12.0 * T * d}
    return {"bytes": 6 * T * row + 2 * gate + 2 * gammas, "flops": 34.0 * T * d}


def _exact_weight(s, c, a, b):
    """Rows [a, b) of the weight matrix from the bit fields of its codes and scales."""
    q = s["q"][a:b].to(torch.int32)
    code = torch.empty(b - a, c["cols"], dtype=torch.int32, device="cuda")
    code[:, 0::2], code[:, 1::2] = q % 16, q // 16
    sign, ex, man = 1.0 - 2.0 * (code // 8).double(), code // 2 % 4, (code % 2).double()
    val = sign * torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * 2.0 ** (ex.double() - 1))
    byte = s["s"][a:b].to(torch.int32)
    if c["wf"] == "mxfp4":
        return val * (2.0 ** (byte.double() - 127)).repeat_interleave(32, 1)
    e8, m8 = byte // 8 % 16, (byte % 8).double()
    scale = torch.where(e8 == 0, m8 / 8 * 2.0 ** -6, (1 + m8 / 8) * 2.0 ** (e8.double() - 7)) * (1.0 - 2.0 * (byte // 128).double())
    return val * scale.repeat_interleave(16, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op == "linear":
        N, x = case["rows"], s["x"].double()
        cut = range(0, N, 4096)
        y = torch.cat([x @ _exact_weight(s, case, a, min(N, a + 4096)).t().contiguous() for a in cut], 1) * s["ts"]
        return y if s["bias"] is None else y + s["bias"].double()
    if "k" in case:
        k, pos = case["k"], s["pick_pos"].long().reshape(-1)
        p = (pos >= 0).nonzero().reshape(-1)        # the picks that have a position
        t, at, total = p // k, pos[p], ROUTED_SCALING
        tail = torch.arange(T, device="cuda") + T * k
        if op == "dispatch":
            xs = torch.zeros(s["xs"].shape, dtype=torch.float64, device="cuda").index_copy_(0, at, s["x"].double()[t])
            return xs.index_copy_(0, tail, s["x"].double()) if case["shared"] else xs
        w = s["w"].double().reshape(-1)
        if op == "sort_backward":
            dy = s["dy"].double()
            d_o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
            d_o.index_copy_(0, at, dy[t] * (total * w[p])[:, None])
            d_w = torch.zeros(T * k, dtype=torch.float64, device="cuda")
            d_w[p] = total * (s["o"].double()[at] * dy[t]).sum(1)
            dx = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda").index_add_(0, t, s["dxs"].double()[at])
            if case["shared"]:
                d_o.index_copy_(0, tail, dy)
                dx += s["dxs"].double()[tail]
            return {"d_o": d_o, "d_w": d_w.reshape(T, k), "dx": dx}
        y = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda").index_add_(0, t, s["o"].double()[at] * (total * w[p])[:, None])
        if case["shared"]:
            y += s["o"].double()[tail]
    else:
        y = s["y"].double()
    # rows as vectors: N(v) = gamma v / sqrt(|v|^2 / d + eps), whose gradient for an upstream g is
    # (gamma g - v (v . gamma g) / (d (|v|^2 / d + eps))) / sqrt(|v|^2 / d + eps)
    x, d, a = s["x"].double(), case["d"], RESIDUAL_SCALE
    gate = torch.ones(T, 1, dtype=torch.float64, device="cuda") if s["gate"] is None else s["gate"].double().reshape(T, -1)
    pre = s["pre_gamma"].double()
    post = None if s["post_gamma"] is None else s["post_gamma"].double()
    y2 = y.square().sum(1, keepdim=True) / d + EPS
    z = y if post is None else post * y / y2.sqrt()
    u = x + a * gate * z
    u2 = u.square().sum(1, keepdim=True) / d + EPS
    if op != "norm_backward":
        return {"x_out": u, "normed": pre * u / u2.sqrt()}

    def through(v, v2, g):
        return (g - v * (v * g).sum(1, keepdim=True) / (d * v2)) / v2.sqrt()

    up = s["d_normed"].double()
    du = s["d_x_out"].double() + through(u, u2, pre * up)
    dz = a * gate * du
    d_gate = {"none": lambda: None, "token": lambda: (a * du * z).sum(1), "element": lambda: a * du * z}[case["gate"]]()
    return {"dx": du, "dy": dz if post is None else through(y, y2, post * dz), "d_gate": d_gate,
            "d_post": None if post is None else (dz * y / y2.sqrt()).sum(0), "d_pre": (up * u / u2.sqrt()).sum(0)}
