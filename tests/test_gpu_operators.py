"""The operators around the experts on the GPU, through the binding, against plain float64 forms with an
error bound carried along (block_ref): dispatch by expert and its gradient, the gradient of the weighted
combine, the norms around the block with gate and residual scale (forward, fused with the combine,
backward), and 4-bit matrix-vector products."""
import ctypes

import numpy as np
import pytest
import torch

import block_ref as ref
import synth
from gpu_util import DeviceLayer, oracle_layer, rel_l2, small

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routed_expert_ffn_router_amd as m      # must load: no fallback path exists

F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *size, dtype=F32, std=1.0):
    return (torch.randn(*size, generator=g, device="cuda") * std).to(dtype)


def shape(d, k=2, E=16, act=BF16, **kw):
    return m.make_shape(d, 128, E, k, act_dtype=m.MOE_DT_BF16 if act == BF16 else m.MOE_DT_F32, **kw)


def routing(g, sh, T, drop):
    """Distinct ids, weights and moe_permute's grouping of them; drop: the last ranks of some tokens are -1,
    and (with a k that allows it) every rank of one token."""
    k, E = sh.top_k, sh.n_experts
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    if drop:
        kept = (torch.arange(T, device="cuda") * 5 + 1) % (k + 1)
        idx[torch.arange(k, device="cuda")[None] >= kept[:, None]] = -1
    w = torch.rand(T, k, generator=g, device="cuda") + 0.1
    w = torch.where(idx < 0, 0.0, w)
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    sp = torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos = torch.empty(T, k, dtype=torch.int32, device="cuda")
    m.moe_permute(sh, idx, T, off, sp, pos)
    return idx, w, off, sp, pos


SORT = [  # T, d, k, E, act, shared, drop
    (1, 128, 1, 1, BF16, 0, 0), (1, 4096, 8, 288, BF16, 0, 0), (3, 256, 2, 16, F32, 0, 0), (5, 640, 3, 7, BF16, 1, 1),
    (17, 2176, 9, 33, F32, 1, 1), (129, 384, 16, 64, BF16, 0, 1), (333, 1152, 8, 256, F32, 1, 0), (70, 4352, 8, 40, BF16, 1, 0),
    (2, 128, 300, 300, F32, 0, 1),
]


@pytest.mark.parametrize("T,d,k,E,act,shared,drop", SORT)
def test_dispatch(T, d, k, E, act, shared, drop):
    g, sh = gen(1), shape(d, k, E, act, n_shared=shared)
    _, _, _, sp, pos = routing(g, sh, T, drop)
    x = rand(g, T, d, dtype=act)
    xs = torch.full((T * (k + shared), d), 7.5, dtype=act, device="cuda")
    m.moe_dispatch(sh, x, T, pos, xs)
    want = torch.where((sp >= 0)[:, None], x[(sp.clamp(min=0) // k).long()], torch.tensor(7.5, dtype=act, device="cuda"))
    assert torch.equal(xs[:T * k], want)                    # rows without a pick as they were
    if shared:
        assert torch.equal(xs[T * k:], x)


@pytest.mark.parametrize("T,d,k,E,act,shared,drop", SORT)
def test_dispatch_backward(T, d, k, E, act, shared, drop):
    g, sh = gen(2), shape(d, k, E, act, n_shared=shared)
    pos = routing(g, sh, T, drop)[4]
    dxs = rand(g, T * (k + shared), d, dtype=act)
    dx = torch.full((T, d), float("nan"), dtype=act, device="cuda")
    m.moe_dispatch_backward(sh, dxs, T, pos, dx)
    ref.check(dx, ref.dispatch_backward(dxs, pos, shared), act, "dx")


@pytest.mark.parametrize("T,d,k,E,act,shared,drop", SORT)
def test_combine_backward(T, d, k, E, act, shared, drop):
    g, sh = gen(3), shape(d, k, E, act, n_shared=shared, routed_scaling=2.5)
    _, w, _, sp, pos = routing(g, sh, T, drop)
    rows = T * (k + shared)
    dy, o = rand(g, T, d, dtype=act), rand(g, rows, d)
    d_o = torch.full((rows, d), 7.5, device="cuda")
    d_w = torch.full((T, k), float("nan"), device="cuda")
    m.moe_combine_backward(sh, dy, o, w, pos, T, d_o, d_w)
    ref.check(d_w, ref.combine_backward_weights(dy, o, pos, 2.5), F32, "d_w")
    want = ref.combine_backward_rows(dy, w, 2.5)
    ok = pos >= 0
    ref.check(d_o[pos[ok].long()], want[ok], F32, "d_o")
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    left[pos[ok].long()] = False
    left[T * k:] = False
    assert (d_o[left] == 7.5).all()                         # rows without a pick as they were
    if shared:
        assert torch.equal(d_o[T * k:], dy.float())
    # each output alone, and in place of o, gives the same bits
    only_w, only_o, here = torch.empty_like(d_w), torch.full_like(d_o, 7.5), o.clone()
    m.moe_combine_backward(sh, dy, o, None, pos, T, None, only_w)
    m.moe_combine_backward(sh, dy, None, w, pos, T, only_o, None)
    m.moe_combine_backward(sh, dy, here, w, pos, T, here, d_w.zero_())
    assert torch.equal(only_w, d_w) and torch.equal(only_o, d_o)
    assert torch.equal(here[~left], d_o[~left]) and torch.equal(here[left], o[left])


def test_positions_out_of_range_have_no_row():
    """Positions that moe_permute never writes are left out like a dropped pick's -1."""
    T, d, k = 3, 256, 4
    g, sh = gen(4), shape(d, k, 16, F32)
    pos = routing(g, sh, T, False)[4]
    bad = pos.clone()
    bad[0, 1], bad[1, 0], bad[2, 3] = -7, T * k, 2 ** 31 - 1
    clean = torch.where((bad < 0) | (bad >= T * k), -1, bad).to(torch.int32)
    x, o, w = rand(g, T, d), rand(g, T * k, d), torch.rand(T, k, generator=g, device="cuda")
    got = []
    for p in (bad, clean):
        xs, d_o = torch.zeros(T * k, d, device="cuda"), torch.zeros(T * k, d, device="cuda")
        dx, d_w, n, x2 = torch.empty_like(x), torch.empty_like(w), torch.empty_like(x), torch.empty_like(x)
        m.moe_dispatch(sh, x, T, p, xs)
        m.moe_dispatch_backward(sh, o, T, p, dx)
        m.moe_combine_backward(sh, x, o, w, p, T, d_o, d_w)
        m.moe_combine_norm(sh, o, w, p, x, T, None, torch.ones(d, device="cuda"), None, 0, 1.0, 1e-5, x2, n)
        got.append((xs, dx, d_o, d_w, n, x2))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", [BF16, F32])
def test_offsets_past_32_bits(act):
    """65536 tokens, eight picks and a shared expert: expert-side arrays of more than 2^31 elements (the fp32
    case more than 2^32 bytes with fewer)."""
    T, k = 65536, 8
    d = 4352 if act == BF16 else 2176
    g, sh = gen(5), shape(d, k, 64, act, n_shared=1)
    _, w, _, _, pos = routing(g, sh, T, True)
    x = rand(g, T, d, dtype=act)
    xs = torch.zeros(T * (k + 1), d, dtype=act, device="cuda")
    m.moe_dispatch(sh, x, T, pos, xs)
    rows = torch.tensor([0, 1, 4093, T // 2, T - 2, T - 1], device="cuda")
    dx, d_w = torch.empty_like(x), torch.empty(T, k, device="cuda")
    m.moe_dispatch_backward(sh, xs, T, pos, dx)
    for t in rows.tolist():
        p = pos[t][pos[t] >= 0].long()
        assert torch.equal(xs[p], x[t].expand(len(p), d)) and torch.equal(xs[T * k + t], x[t])
        n = len(p) + 1
        ref.check(dx[t], ref.Val(x[t].double() * n, x[t].double().abs() * n * n * ref.U), act, "dx")
    if act == F32:                                           # in place: xs stands for o, then holds its gradient
        m.moe_combine_backward(sh, x, xs, w, pos, T, xs, d_w)
        for t in rows.tolist():
            p = pos[t] >= 0
            ref.check(xs[pos[t][p].long()], ref.combine_backward_rows(x[t:t + 1], w[t:t + 1], 1.0)[0][p], F32, "d_o")
            sq = (x[t].double() ** 2).sum()
            ref.check(d_w[t], ref.Val(torch.where(p, sq, 0.0), torch.where(p, sq * (-(-d // 256) + 10) * ref.U, 0.0)), F32,
                      "d_w")


# ---------------------------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------------------------

NORM = [  # T, d, act, gate, post, y
    (1, 4096, BF16, 0, 1, 1), (1, 128, F32, 0, 0, 1), (2, 256, BF16, 0, 0, 0), (3, 640, F32, 1, 1, 1), (65, 384, BF16, 2, 1, 1),
    (7, 6144, F32, 2, 0, 1), (5, 8192, BF16, 1, 1, 1), (4, 8320, F32, 2, 1, 1), (3, 16384, BF16, 2, 1, 1),
    (2, 16384, F32, 1, 0, 1), (513, 256, F32, 1, 1, 1), (1030, 1152, BF16, 2, 1, 1), (9, 2176, F32, 0, 1, 1),
]
ALPHA, EPS = 0.7, 1e-5


def norm_inputs(g, T, d, act, gate, post, y):
    i = {"x": rand(g, T, d, dtype=act, std=2.0), "y": rand(g, T, d, dtype=act, std=0.5) if y else None,
         "post": 1 + rand(g, d, std=0.1) if post else None, "pre": 1 + rand(g, d, std=0.1),
         "gate": None if not gate else torch.sigmoid(rand(g, T)) if gate == 1 else torch.sigmoid(rand(g, T, d)).to(act)}
    return i, None if not gate else i["gate"][:, None] if gate == 1 else i["gate"]


@pytest.mark.parametrize("T,d,act,gate,post,y", NORM)
def test_block_norm(T, d, act, gate, post, y):
    sh = shape(d, act=act)
    i, wide = norm_inputs(gen(6), T, d, act, gate, post, y)
    args = (i["post"], i["pre"], i["gate"], gate, ALPHA, EPS)
    x_out, normed = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    m.moe_block_norm(sh, i["x"], i["y"], T, *args, x_out, normed)
    u, n = ref.norm_forward(i["x"], ref.Val(i["y"]) if y else None, i["post"], i["pre"], wide, ALPHA, EPS)
    ref.check(x_out, u, act, "x_out")
    ref.check(normed, n, act, "normed")
    # each output alone, and written over the inputs, gives the same bits
    a, b = torch.empty_like(x_out), torch.empty_like(x_out)
    m.moe_block_norm(sh, i["x"], i["y"], T, i["post"], None, *args[2:], a, None)
    m.moe_block_norm(sh, i["x"], i["y"], T, *args, None, b)
    assert torch.equal(a, x_out) and torch.equal(b, normed)
    x2, y2 = i["x"].clone(), i["y"].clone() if y else None
    m.moe_block_norm(sh, x2, y2, T, *args, x2, y2 if y else b)
    assert torch.equal(x2, x_out) and torch.equal(y2 if y else b, normed)
    if gate == 2:
        g2 = i["gate"].clone()
        m.moe_block_norm(sh, i["x"], i["y"], T, i["post"], i["pre"], g2, gate, ALPHA, EPS, x_out, g2)
        assert torch.equal(g2, normed)


def test_block_norm_keeps_rows_apart():
    """Rows of zeros give zeros (eps), and NaN or infinity in one row stays there."""
    T, d, sh = 5, 640, shape(640, act=F32)
    g = gen(7)
    x, y, w = rand(g, T, d), rand(g, T, d), torch.ones(d, device="cuda")
    x[1], y[1] = 0.0, 0.0
    clean = [torch.empty_like(x) for _ in range(2)]
    m.moe_block_norm(sh, x, y, T, w, w, None, 0, 1.0, EPS, *clean)
    assert (clean[0][1] == 0).all() and (clean[1][1] == 0).all()
    y[3, 17], x[0, 600] = float("nan"), float("inf")
    got = [torch.empty_like(x) for _ in range(2)]
    m.moe_block_norm(sh, x, y, T, w, w, None, 0, 1.0, EPS, *got)
    for a, b in zip(got, clean):
        assert torch.equal(a[[1, 2, 4]], b[[1, 2, 4]])
    assert torch.isnan(got[0][3]).all() and torch.isinf(got[0][0, 600]) and torch.isnan(got[1][0, 600])


def norm_gradients(sh, i, T, d, act, gate, post, y, d_x_out, d_normed, ws=None, want=("dx", "dy", "d_gate", "d_post", "d_pre")):
    out = {"dx": torch.empty_like(i["x"]), "dy": torch.empty_like(i["x"]) if y else None,
           "d_gate": None if not gate else torch.empty_like(i["gate"]), "d_post": torch.empty(d, device="cuda") if post else None,
           "d_pre": torch.empty(d, device="cuda") if d_normed is not None else None}
    out = {k: v if k in want else None for k, v in out.items()}
    m.moe_block_norm_backward(sh, i["x"], i["y"], T, i["post"], i["pre"] if d_normed is not None else None, i["gate"], gate, ALPHA,
                              EPS, d_x_out, d_normed, out["dx"], out["dy"], out["d_gate"], out["d_post"], out["d_pre"],
                              m.workspace(sh, T) if ws is None else ws)
    return out


def check_gradients(out, want, act, gate):
    for k, v in out.items():
        if v is not None:
            ref.check(v, want[k], F32 if k in ("d_post", "d_pre") or (k == "d_gate" and gate == 1) else act, k)


@pytest.mark.parametrize("T,d,act,gate,post,y", NORM)
def test_block_norm_backward(T, d, act, gate, post, y):
    g, sh = gen(8), shape(d, act=act)
    i, wide = norm_inputs(g, T, d, act, gate, post, y)
    dxo, dn = rand(g, T, d, dtype=act), rand(g, T, d, dtype=act)
    ws = m.workspace(sh, T)
    full = None
    for a, b in ((dxo, dn), (None, dn), (dxo, None)):
        out = norm_gradients(sh, i, T, d, act, gate, post, y, a, b, ws)
        check_gradients(out, ref.norm_backward(i["x"], i["y"], i["post"], i["pre"], wide, ALPHA, EPS, a, b, gate == 1), act, gate)
        full = full or out
    # again, each output alone, and written over the upstream gradients and inputs: the same bits
    for k, v in full.items():
        if v is not None:
            one = norm_gradients(sh, i, T, d, act, gate, post, y, dxo, dn, ws, want=(k,))
            assert torch.equal(one[k], v), k
    over = {k: v.clone() if v is not None else None for k, v in i.items()} | {"a": dxo.clone(), "b": dn.clone()}
    m.moe_block_norm_backward(sh, over["x"], over["y"], T, over["post"], over["pre"], over["gate"], gate, ALPHA, EPS, over["a"],
                              over["b"], over["a"], over["b"] if y else None, over["gate"], None, None, ws)
    assert torch.equal(over["a"], full["dx"]) and (not y or torch.equal(over["b"], full["dy"]))
    assert not gate or torch.equal(over["gate"], full["d_gate"])
    assert m.workspace_status(ws) == 0


def test_block_norm_backward_against_differences():
    """Central differences of the float64 forward form, for a loss that weighs both outputs."""
    T, d, h = 2, 128, 1e-4
    g, sh = gen(9), shape(d, act=F32)
    i, _ = norm_inputs(g, T, d, F32, 1, 1, 1)
    dxo, dn = rand(g, T, d), rand(g, T, d)
    out = norm_gradients(sh, i, T, d, F32, 1, 1, 1, dxo, dn)
    names = {"x": "dx", "y": "dy", "gate": "d_gate", "post": "d_post", "pre": "d_pre"}
    base = {k: i[k].double() for k in names}

    def loss(v):
        y = v["y"] * (v["y"].square().mean(1, keepdim=True) + EPS).rsqrt() * v["post"]
        u = v["x"] + ref.alpha32(ALPHA) * v["gate"][:, None] * y
        n = u * (u.square().mean(1, keepdim=True) + EPS).rsqrt() * v["pre"]
        return (u * dxo.double()).sum() + (n * dn.double()).sum()

    for k, name in names.items():
        flat = out[name].double().reshape(-1)
        for at in range(0, flat.numel(), max(1, flat.numel() // 24)):
            v = base[k].clone()
            step = []
            for s in (h, -h):
                w = v.clone()
                w.view(-1)[at] += s
                step.append(loss(base | {k: w}))
            num = (step[0] - step[1]).item() / (2 * h)
            # h^2 times a third derivative of order one, 2^-52 |loss| / h, and fp32 sums of up to 128 terms
            assert abs(num - flat[at].item()) <= 1e-5 * max(1.0, abs(num)), (name, at, num, flat[at].item())


def test_gradient_sums_of_no_tokens_are_zero():
    sh = shape(640, act=F32)
    a, b = torch.full((640,), 3.0, device="cuda"), torch.full((640,), 3.0, device="cuda")
    m.moe_block_norm_backward(sh, None, None, 0, None, None, None, 0, 1.0, EPS, None, None, None, None, None, a, b, None)
    assert (a == 0).all() and (b == 0).all()


COMBINE = [  # T, d, k, E, act, shared, drop, gate, post
    (1, 4096, 8, 288, BF16, 1, 0, 0, 1), (1, 128, 1, 1, F32, 0, 0, 0, 0), (64, 640, 8, 32, BF16, 1, 1, 2, 1),
    (33, 2176, 9, 40, F32, 0, 1, 1, 1), (5, 8320, 3, 16, BF16, 0, 0, 1, 1), (3, 16384, 17, 20, F32, 1, 1, 2, 0),
    (700, 256, 2, 16, F32, 0, 1, 0, 1),
]


@pytest.mark.parametrize("T,d,k,E,act,shared,drop,gate,post", COMBINE)
def test_combine_norm(T, d, k, E, act, shared, drop, gate, post):
    g, sh = gen(10), shape(d, k, E, act, n_shared=shared, routed_scaling=2.5)
    _, w, _, _, pos = routing(g, sh, T, drop)
    o = rand(g, T * (k + shared), d, std=0.5)
    i, wide = norm_inputs(g, T, d, act, gate, post, 1)
    x_out, normed = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    m.moe_combine_norm(sh, o, w, pos, i["x"], T, i["post"], i["pre"], i["gate"], gate, ALPHA, EPS, x_out, normed)
    u, n = ref.norm_forward(i["x"], ref.combine(o, w, pos, 2.5, shared), i["post"], i["pre"], wide, ALPHA, EPS)
    ref.check(x_out, u, act, "x_out")
    ref.check(normed, n, act, "normed")
    x2 = i["x"].clone()
    m.moe_combine_norm(sh, o, w, pos, x2, T, i["post"], i["pre"], i["gate"], gate, ALPHA, EPS, x2, normed)
    assert torch.equal(x2, x_out)
    if act == F32:                                           # an fp32 y is not rounded between: the same bits in two calls
        y = torch.empty_like(i["x"])
        m.moe_combine(sh, o, w, pos, T, None, y)
        a, b = torch.empty_like(y), torch.empty_like(y)
        m.moe_block_norm(sh, i["x"], y, T, i["post"], i["pre"], i["gate"], gate, ALPHA, EPS, a, b)
        assert torch.equal(a, x_out) and torch.equal(b, normed)


@pytest.mark.parametrize("act,T", [(BF16, 4099), (F32, 2051)])
def test_rows_larger_than_the_caches(act, T):
    """Arrays past the sizes from which the row kernels go round the caches: every operator on rows, in full."""
    d, k = 4096, 8
    g, sh = gen(17), shape(d, k, 64, act, n_shared=1, routed_scaling=2.5)
    _, w, _, sp, pos = routing(g, sh, T, True)
    i, wide = norm_inputs(g, T, d, act, 2, 1, 1)
    o = rand(g, T * (k + 1), d, std=0.5)
    tail = (i["post"], i["pre"], i["gate"], 2, ALPHA, EPS)
    xs = torch.full((T * (k + 1), d), 7.5, dtype=act, device="cuda")
    m.moe_dispatch(sh, i["x"], T, pos, xs)
    want = torch.where((sp >= 0)[:, None], i["x"][(sp.clamp(min=0) // k).long()], torch.tensor(7.5, dtype=act, device="cuda"))
    assert torch.equal(xs[:T * k], want) and torch.equal(xs[T * k:], i["x"])
    del want
    xs.mul_(torch.rand(T * (k + 1), 1, generator=g, device="cuda"))
    dx = torch.empty_like(i["x"])
    m.moe_dispatch_backward(sh, xs, T, pos, dx)
    ref.check(dx, ref.dispatch_backward(xs, pos, 1), act, "dx")
    del xs
    d_o, d_w = torch.full_like(o, 7.5), torch.empty_like(w)
    m.moe_combine_backward(sh, i["y"], o, w, pos, T, d_o, d_w)
    ref.check(d_w, ref.combine_backward_weights(i["y"], o, pos, 2.5), F32, "d_w")
    ok = pos >= 0
    ref.check(d_o[pos[ok].long()], ref.combine_backward_rows(i["y"], w, 2.5)[ok], F32, "d_o")
    assert torch.equal(d_o[T * k:], i["y"].float())
    left = torch.ones(T * (k + 1), dtype=torch.bool, device="cuda")
    left[pos[ok].long()], left[T * k:] = False, False
    assert (d_o[left] == 7.5).all()
    del d_o
    a, b = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    m.moe_combine_norm(sh, o, w, pos, i["x"], T, *tail, a, b)
    u, n = ref.norm_forward(i["x"], ref.combine(o, w, pos, 2.5, 1), i["post"], i["pre"], wide, ALPHA, EPS)
    ref.check(a, u, act, "x_out of the combine")
    ref.check(b, n, act, "normed of the combine")
    del o
    m.moe_block_norm(sh, i["x"], i["y"], T, *tail, a, b)
    u, n = ref.norm_forward(i["x"], ref.Val(i["y"]), i["post"], i["pre"], wide, ALPHA, EPS)
    ref.check(a, u, act, "x_out")
    ref.check(b, n, act, "normed")
    out = norm_gradients(sh, i, T, d, act, 2, 1, 1, a, b)
    check_gradients(out, ref.norm_backward(i["x"], i["y"], i["post"], i["pre"], wide, ALPHA, EPS, a, b, False), act, 2)


# ---------------------------------------------------------------------------------------------
# 4-bit matrix-vector products
# ---------------------------------------------------------------------------------------------

def quantised(g, N, K, wf):
    """Random codes and scales around 2^-6 (every code and many scales, not a quantiser's output)."""
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if wf == 0:
        return q, torch.randint(115, 128, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8), 1.0
    s = torch.randint(0, 127, (N, K // 16), generator=g, device="cuda", dtype=torch.uint8)       # 127 is NaN
    return q, s | torch.randint(0, 2, s.shape, generator=g, device="cuda", dtype=torch.uint8) << 7, 0.0123


LINEAR = [  # N, K, T
    (1, 128, 1), (15, 256, 1), (16, 128, 2), (33, 384, 3), (128, 4096, 1), (100, 1152, 5), (257, 640, 16), (64, 2048, 17),
    (48, 512, 33), (31, 896, 64), (5000, 256, 7), (2048, 6144, 4), (4096, 512, 12), (40000, 128, 1), (9000, 384, 40), (515, 8192, 9),
    (20000, 640, 6), (16399, 8192, 13), (16384, 6144, 5), (33000, 256, 16), (300, 8320, 5), (16400, 8320, 3),
    (17000, 256, 20), (17000, 256, 40), (32770, 4096, 3), (300, 8320, 20), (300, 8320, 40),
    (4100, 512, 64), (4099, 256, 16), (5000, 8448, 33), (16390, 1024, 16), (16400, 8320, 16), (17003, 1152, 40), (33001, 640, 25),
    (32900, 256, 64), (65540, 384, 33), (65539, 128, 20), (32771, 8320, 9), (32768, 2432, 49), (16390, 2176, 8),
]


@pytest.mark.parametrize("wf", [0, 1])
@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("N,K,T", LINEAR)
def test_linear(N, K, T, act, wf):
    g = gen(N + K + T)
    q, s, ts = quantised(g, N, K, wf)
    x, bias = rand(g, T, K, dtype=act), rand(g, N)
    mat = m.make_matrix(N, K, wf, m.MOE_DT_BF16 if act == BF16 else m.MOE_DT_F32)
    for b in (None, bias):
        y = torch.full((T * N + 64,), 7.5, dtype=act, device="cuda")
        m.moe_linear(mat, q, s, ts, x, T, b, y)
        ref.check(y[:T * N].view(T, N), ref.linear(q, s, wf, ts, x, b), act, "y")
        assert (y[T * N:] == 7.5).all()                      # nothing behind the last row


@pytest.mark.parametrize("N,K,T,act", [(256, 128, 16, BF16), (256, 128, 16, F32), (16640, 128, 16, BF16), (16640, 128, 8, F32),
                                       (256, 8320, 16, BF16), (256, 8320, 16, F32), (4352, 128, 32, BF16), (4352, 128, 16, F32),
                                       (16640, 128, 16, F32), (32768, 8320, 16, BF16), (16640, 128, 48, BF16),
                                       (16640, 128, 20, F32), (65536, 128, 40, BF16), (65536, 128, 32, F32),
                                       (16640, 2048, 8, F32)])
def test_linear_scale_bytes(N, K, T, act):
    """Every code under every E8M0 byte whose weights are below 2^128, subnormal ones among them, and the NaN
    byte: row n has all codes in block 1 under byte n, token t one value at code t % 16, so y is that product (exact
    where it is a normal number of the type)."""
    q = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    s[:, 1] = (torch.arange(N, device="cuda") % 256).to(torch.uint8)
    for j in range(8):
        q[:, 16 + j] = 2 * j | (2 * j + 1) << 4              # elements 32 .. 47: codes 0 .. 15
    values = torch.tensor(ref.E2M1 + tuple(-v for v in ref.E2M1), dtype=torch.float64, device="cuda")[torch.arange(T) % 16, None]
    weight = values * torch.ldexp(torch.ones(N, dtype=torch.float64, device="cuda"), s[:, 1].int() - 127)
    for e in (60, -60):
        x = torch.zeros(T, K, dtype=act, device="cuda")
        x[torch.arange(T), 32 + torch.arange(T) % 16] = 2.0 ** e
        y = torch.empty(T, N, dtype=act, device="cuda")
        m.moe_linear(m.make_matrix(N, K, 0, m.MOE_DT_BF16 if act == BF16 else m.MOE_DT_F32), q, s, 1.0, x, T, None, y)
        want = weight * 2.0 ** e
        sure = (s[:, 1] < 253) & ((want == 0) | (want.abs() >= 2.0 ** -126))
        assert torch.equal(y[sure], want.to(act)[sure])
        assert torch.isnan(y[:, s[:, 1] == 255]).all()


def test_linear_values_outside_the_numbers():
    """Infinity and NaN in x reach the rows whose weights see them, in that token alone."""
    g = gen(12)
    for N, K, T, act in ((40, 256, 3, BF16), (40, 256, 3, F32), (16390, 256, 3, BF16), (16390, 256, 3, F32), (40, 8320, 3, BF16),
                         (40, 8320, 3, F32), (4352, 256, 20, BF16), (4352, 256, 16, F32), (16390, 256, 16, F32),
                         (16390, 256, 40, BF16), (16390, 256, 20, F32), (16390, 2048, 16, BF16), (16390, 2048, 8, F32)):
        q, s, _ = quantised(g, N, K, 0)
        x = rand(g, T, K, dtype=act)
        mat = m.make_matrix(N, K, 0, m.MOE_DT_BF16 if act == BF16 else m.MOE_DT_F32)
        y, z = torch.empty(T, N, dtype=act, device="cuda"), torch.empty(T, N, dtype=act, device="cuda")
        m.moe_linear(mat, q, s, 1.0, x, T, None, y)
        x[0, 200], x[2, 3] = float("inf"), float("nan")
        m.moe_linear(mat, q, s, 1.0, x, T, None, z)
        assert torch.equal(z[1], y[1]) and torch.equal(z[3:], y[3:]) and torch.isnan(z[2]).all()
        if act == F32:                                       # a NaN whose payload lies in the lower half
            x.view(torch.int32)[2, 3] = 0x7f800001
            m.moe_linear(mat, q, s, 1.0, x, T, None, z)
            assert torch.equal(z[1], y[1]) and torch.equal(z[3:], y[3:]) and torch.isnan(z[2]).all()
        w = ref.weights(q, s, 0)[:, 200]
        assert torch.equal(torch.isnan(z[0]), w == 0)        # 0 times infinity
        assert torch.equal(z[0][w != 0], (torch.sign(w) * float("inf")).to(act)[w != 0])
        # the largest finite values stay finite on the way
        if act == F32 and T == 3 and K == 256 and N == 40:
            x = torch.zeros(1, K, device="cuda")
            x[0, 7] = torch.finfo(F32).max
            small_s = torch.full_like(s, 100)
            m.moe_linear(mat, q, small_s, 1.0, x, 1, None, z[:1])
            ref.check(z[:1], ref.linear(q, small_s, 0, 1.0, x, None), F32, "y")


# ---------------------------------------------------------------------------------------------
# streams, graphs, repeats
# ---------------------------------------------------------------------------------------------

def everything(T=70, d=640, k=4, act=BF16):
    """One call of each operator on inputs of its own: (run(), outputs)."""
    g, sh = gen(13), shape(d, k, 24, act, n_shared=1)
    _, w, _, _, pos = routing(g, sh, T, True)
    i, _ = norm_inputs(g, T, d, act, 2, 1, 1)
    o, dxs = rand(g, T * (k + 1), d), rand(g, T * (k + 1), d, dtype=act)
    q, s, ts = quantised(g, 300, d, 1)
    dxo, dn = rand(g, T, d, dtype=act), rand(g, T, d, dtype=act)
    mat, ws = m.make_matrix(300, d, 1, sh.act_dtype), m.workspace(sh, T)
    out = {n: torch.zeros_like(v) for n, v in dict(
        xs=dxs, dx0=dxo, d_o=o, d_w=w, x_out=dxo, normed=dxo, x_out2=dxo, normed2=dxo, dx=dxo, dy=dxo, d_gate=dxo,
        d_post=i["post"], d_pre=i["pre"]).items()}
    out["lin"] = torch.zeros(16, 300, dtype=act, device="cuda")
    tail = (i["post"], i["pre"], i["gate"], 2, ALPHA, EPS)

    def run():
        m.moe_dispatch(sh, i["x"], T, pos, out["xs"])
        m.moe_dispatch_backward(sh, dxs, T, pos, out["dx0"])
        m.moe_combine_backward(sh, i["x"], o, w, pos, T, out["d_o"], out["d_w"])
        m.moe_block_norm(sh, i["x"], i["y"], T, *tail, out["x_out"], out["normed"])
        m.moe_combine_norm(sh, o, w, pos, i["x"], T, *tail, out["x_out2"], out["normed2"])
        m.moe_block_norm_backward(sh, i["x"], i["y"], T, *tail, dxo, dn, out["dx"], out["dy"], out["d_gate"], out["d_post"],
                                  out["d_pre"], ws)
        m.moe_linear(mat, q, s, ts, i["x"], 16, None, out["lin"])
    return run, out, (i, o, dxs, dxo, dn)


def test_repeats_streams_and_graph_replays_give_the_same_bits():
    run, out, inputs = everything()
    run()
    torch.cuda.synchronize()
    first = {n: v.clone() for n, v in out.items()}

    def same(what):
        torch.cuda.synchronize()
        for n, v in out.items():
            assert torch.equal(v, first[n]), (what, n)
            v.zero_()
        torch.cuda.synchronize()

    run()
    same("repeat")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    same("another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        graph.replay()
        same("replay")
        run()                                                # eager work of the same kernels between replays
        same("eager between replays")
    # a replay reads the inputs as they are then
    i = inputs[0]
    i["x"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = {n: v.clone() for n, v in out.items()}
    run()
    torch.cuda.synchronize()
    for n, v in out.items():
        assert torch.equal(v, got[n]), n
    assert not torch.equal(got["xs"], first["xs"])


def test_layer_runs_on_the_workspace_of_a_gradient():
    """The norms' gradient leaves the workspace's status and hand-over slots alone: the few-token router still
    routes on it, and gives the same bits as on a fresh one."""
    dl = DeviceLayer(m, synth.WORKLOADS["tiny"])
    wl, T = dl.wl, 4
    x = synth.make_x(wl, 0, "cpu").to("cuda").contiguous()
    ws, y = m.workspace(dl.shape, T), [torch.empty_like(x) for _ in range(2)]
    m.moe_layer(dl.shape, x, T, dl.router, None, dl.table, None, None, y[0], ws=m.workspace(dl.shape, T))
    dp = torch.empty(wl.d_model, device="cuda")
    one = torch.ones(wl.d_model, device="cuda")
    m.moe_block_norm_backward(dl.shape, x, x, T, one, one, None, 0, 1.0, EPS, x, x, None, torch.empty_like(x), None, dp, None, ws)
    m.moe_layer(dl.shape, x, T, dl.router, None, dl.table, None, None, y[1], ws=ws)
    assert m.workspace_status(ws) == 0 and torch.equal(y[0], y[1])


def test_binding_refuses_strided_and_short_tensors():
    sh, T = shape(256, act=F32), 4
    x, out = torch.zeros(T, 512, device="cuda"), torch.zeros(T, 256, device="cuda")
    one = torch.ones(256, device="cuda")
    for bad in (x[:, ::2], x[:, :256], out[:3], out.bfloat16(), out.cpu()):
        with pytest.raises(m.MoeError):
            m.moe_block_norm(sh, bad, None, T, None, one, None, 0, 1.0, EPS, None, out)
    with pytest.raises(m.MoeError):
        m.moe_dispatch(sh, out, T, torch.zeros(T, 2, dtype=torch.int64, device="cuda"), torch.zeros(T * 2, 256, device="cuda"))


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------

def test_training_step_through_the_block():
    """pre-norm, routing, dispatch, dense experts (torch), combine, post-norm with gate and residual, and the
    whole way back, against autograd of the same block in float64 on the CPU."""
    T, d, k, E = 37, 256, 2, 8
    g, sh = gen(14), shape(d, k, E, F32, routed_scaling=1.5)
    i, _ = norm_inputs(g, T, d, F32, 1, 1, 1)
    x, pre, post, gate = i["x"], i["pre"], i["post"], i["gate"]
    wr, we = rand(g, E, d, std=0.05), rand(g, E, d, d, std=d ** -0.5)
    n, x_out, n2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    m.moe_block_norm(sh, x, None, T, None, pre, None, 0, 1.0, EPS, None, n)
    ws = m.workspace(sh, T)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    m.moe_route(sh, n, T, wr, None, idx, w, ws)
    off, sp = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos = torch.empty(T, k, dtype=torch.int32, device="cuda")
    m.moe_permute(sh, idx, T, off, sp, pos, ws, ws.numel())
    xs, y = torch.empty(T * k, d, device="cuda"), torch.empty_like(x)
    m.moe_dispatch(sh, n, T, pos, xs)
    cut = off.tolist()
    act = torch.cat([xs[a:b] @ we[e] for e, (a, b) in enumerate(zip(cut, cut[1:]))])
    o = torch.tanh(act).contiguous()
    m.moe_combine(sh, o, w, pos, T, None, y)
    m.moe_block_norm(sh, x, y, T, post, pre, gate, 1, ALPHA, EPS, x_out, n2)
    # upstream gradients, and back
    up_x, up_n = rand(g, T, d), rand(g, T, d)
    dx, dy, dgate = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gate)
    dpost, dpre, dpre0 = (torch.empty(d, device="cuda") for _ in range(3))
    m.moe_block_norm_backward(sh, x, y, T, post, pre, gate, 1, ALPHA, EPS, up_x, up_n, dx, dy, dgate, dpost, dpre, ws)
    d_o, d_w = torch.empty_like(o), torch.empty_like(w)
    m.moe_combine_backward(sh, dy, o, w, pos, T, d_o, d_w)
    da = d_o * (1 - o * o)
    dxs = torch.cat([da[a:b] @ we[e].t().contiguous() for e, (a, b) in enumerate(zip(cut, cut[1:]))])
    dn = torch.empty_like(x)
    m.moe_dispatch_backward(sh, dxs, T, pos, dn)
    dx0 = torch.empty_like(x)
    m.moe_block_norm_backward(sh, x, None, T, None, pre, None, 0, 1.0, EPS, dx, dn, dx0, None, None, None, dpre0, ws)

    t = {a: v.double().cpu().requires_grad_() for a, v in dict(x=x, pre=pre, post=post, gate=gate, w=w).items()}
    ids, we64 = idx.cpu().long(), we.double().cpu()

    def rms(v):
        return v * (v.square().mean(1, keepdim=True) + EPS).rsqrt()

    h = rms(t["x"]) * t["pre"]
    outs = torch.stack([torch.stack([torch.tanh(h[a] @ we64[ids[a, j]]) for j in range(k)]) for a in range(T)])
    yy = 1.5 * (t["w"][..., None] * outs).sum(1)
    u = t["x"] + ref.alpha32(ALPHA) * t["gate"][:, None] * rms(yy) * t["post"]
    nn = rms(u) * t["pre"]
    ((u * up_x.double().cpu()).sum() + (nn * up_n.double().cpu()).sum()).backward()
    # fp32 throughout: products over 256 columns, sums over 37 tokens; 1e-5 of each gradient's own norm is
    # about eighty fp32 steps
    for got, want in ((x_out, u), (n2, nn), (dx0, t["x"].grad), (dpost, t["post"].grad), (dpre + dpre0, t["pre"].grad),
                      (dgate, t["gate"].grad), (d_w, t["w"].grad)):
        assert rel_l2(got.double().cpu().numpy(), want.detach().numpy()) <= 1e-5


def test_decode_step_around_the_layer():
    """A 4-bit projection, the pre-norm, the routed layer's own steps and the fused combine with post-norm and next
    pre-norm, for one token and for a few: against the oracle's layer and the norms in float64."""
    wl = small("tiny")
    dl = DeviceLayer(m, wl)
    d, k, sh = wl.d_model, wl.top_k, dl.shape
    for T in (1, 5, 40):
        g = gen(15 + T)
        q, s, ts = quantised(g, d, 384, 0)
        a = rand(g, T, 384, std=0.01)
        h, n = torch.empty(T, d, device="cuda"), torch.empty(T, d, device="cuda")
        pre, post = 1 + rand(g, d, std=0.1), 1 + rand(g, d, std=0.1)
        m.moe_linear(m.make_matrix(d, 384, 0, m.MOE_DT_F32), q, s, ts, a, T, None, h)
        m.moe_block_norm(sh, h, None, T, None, pre, None, 0, 1.0, EPS, None, n)
        ws = m.workspace(sh, T)
        idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        off = torch.empty(wl.n_experts + 1, dtype=torch.int32, device="cuda")
        sp, pos = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
        o = torch.empty(T * k, d, device="cuda")
        m.moe_route(sh, n, T, dl.router, None, idx, w, ws)
        m.moe_permute(sh, idx, T, off, sp, pos)
        m.moe_expert_ffn(sh, dl.table, n, T, off, sp, o, ws)
        x_out, n2 = torch.empty_like(h), torch.empty_like(h)
        m.moe_combine_norm(sh, o, w, pos, h, T, post, pre, None, 0, ALPHA, EPS, x_out, n2)
        ref.check(h, ref.linear(q, s, 0, ts, a, None), F32, "projection")
        _, n64 = ref.norm_forward(h, None, None, pre, None, 1.0, EPS)
        ref.check(n, n64, F32, "pre-norm")
        oy, oidx, _, _ = oracle_layer(dl, n, idx_hint=idx.cpu().numpy())
        np.testing.assert_array_equal(idx.cpu().numpy(), oidx)
        y64 = torch.from_numpy(np.asarray(oy)).to("cuda")
        u, nn = ref.norm_forward(h, ref.Val(y64), post, pre, None, ALPHA, EPS)
        # the layer's own bar for fp32 output, on what it contributes
        assert rel_l2((x_out - h).double().cpu().numpy(), (u.v - h.double()).cpu().numpy()) <= 1e-4
        assert rel_l2(n2.double().cpu().numpy(), nn.v.cpu().numpy()) <= 1e-4


def test_no_tokens_is_a_no_op():
    sh = shape(256, act=F32)
    p = m.library()
    st = torch.cuda.current_stream().cuda_stream
    b = ctypes.byref(sh)
    assert p.moe_dispatch(b, None, 0, None, None, st) == 0 and p.moe_dispatch_backward(b, None, 0, None, None, st) == 0
    assert p.moe_combine_backward(b, None, None, None, None, 0, None, None, st) == 0
    assert p.moe_block_norm(b, None, None, 0, None, None, None, 0, 1.0, EPS, None, None, st) == 0
