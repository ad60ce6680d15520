"""The operators around the experts where their loops run past the first fill: products whose rings and stages wrap, in
integers that every order of summing gives exactly; norm gradients of many rows to a workgroup; values outside the numbers in
the gradients; and what no pick has, which must not reach any result."""
import pytest
import torch

import block_ref as ref
import test_gpu_operators as ops

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import routed_expert_ffn_router_amd as m      # must load: no fallback path exists

F32, BF16 = torch.float32, torch.bfloat16
EPS = ops.EPS

# N, K, T: one to sixteen row tiles to a workgroup, one to 65 steps of 128 columns, waves with unequal shares of them
DEEP = [
    (16390, 8192, 5), (16390, 7040, 9), (16390, 4736, 3), (16390, 8192, 16), (20011, 5888, 12), (65540, 2432, 5), (65540, 2432, 9),
    (65540, 2432, 16), (65540, 2432, 20), (65540, 2432, 33), (65540, 2432, 49), (32900, 2432, 64), (16400, 4224, 40),
    (16400, 8448, 16), (33001, 8320, 24), (9000, 4224, 40), (4099, 4224, 16), (4099, 4224, 33), (515, 8192, 64), (300, 16384, 2),
    (300, 16384, 7), (16384, 8320, 5), (24580, 4224, 7), (12290, 4224, 22), (12290, 4224, 30), (12300, 4096, 20), (49160, 5504, 2),
    (49155, 512, 1), (49155, 512, 4), (4100, 512, 40), (6150, 640, 33), (4099, 4224, 17), (16390, 1152, 3), (12300, 1152, 9),
    (6150, 4096, 13), (24600, 8320, 13), (8200, 1024, 48), (98310, 640, 7), (4090, 4224, 16), (2048, 8320, 64), (12300, 8192, 12),
    (9000, 7168, 4), (16400, 2688, 8),
]


def matrix(N, K, wf, act):
    return m.make_matrix(N, K, wf, m.MOE_DT_BF16 if act == BF16 else m.MOE_DT_F32)


def linear_bound(q, s, wf, ts, x, bias):
    """The float64 product with the bound of any order of summing: a product passes at most one addition for every column and
    term (fp32 x has three terms), and sixteen more where waves share out the columns."""
    W, x64 = ref.weights(q, s, wf), x.double()
    depth = W.shape[1] * (3 if x.dtype == F32 else 1) + 16
    y, mag = x64 @ W.t().contiguous(), x64.abs() @ W.abs().t().contiguous()
    r = ref.Val(y, depth * ref.U * mag) * ref.alpha32(ts)
    return r if bias is None else r + ref.Val(bias)


@pytest.mark.parametrize("wf", [0, 1])
@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("N,K,T", DEEP)
def test_linear_past_the_first_fill(N, K, T, act, wf):
    """Random values within the bound, and integers to the bit: weights are multiples of 1/2 up to 12, so 16384 of them times
    integers up to 7, or 64 of them times integers up to 4095 (two terms of an fp32 x; bf16 takes those up to 255), sum to
    multiples of 1/2 below 2^23: exact in fp32 in any order."""
    g = ops.gen(N + K + T)
    q, s, ts = ops.quantised(g, N, K, wf)
    x, bias, mat = ops.rand(g, T, K, dtype=act), ops.rand(g, N), matrix(N, K, wf, act)
    y = torch.empty(T, N, dtype=act, device="cuda")
    m.moe_linear(mat, q, s, ts, x, T, bias, y)
    ref.check(y, linear_bound(q, s, wf, ts, x, bias), act, "y")
    one, two = (127, 128) if wf == 0 else (0x38, 0x40)
    s = torch.where(s % 2 == 0, one, two).to(torch.uint8)
    W = ref.weights(q, s, wf)
    dense = torch.randint(-7, 8, (T, K), generator=g, device="cuda")
    most = 4095 if act == F32 else 255
    big = torch.randint(-most, most + 1, (T, K), generator=g, device="cuda")
    sparse = torch.where(torch.rand(T, K, generator=g, device="cuda").argsort(1) < 64, big, 0)
    for xi in (dense, sparse):
        m.moe_linear(mat, q, s, 1.0, xi.to(act), T, None, y)
        want = xi.double() @ W.t().contiguous()
        assert want.abs().max() < 2.0 ** 23
        assert torch.equal(y, want.float().to(act))


@pytest.mark.parametrize("N,K,T", [(40, 256, 1), (40, 256, 3), (4352, 256, 16), (16390, 256, 3), (16390, 2048, 5), (16390, 256, 16),
                                   (16390, 256, 20), (65540, 256, 33), (9000, 256, 40)])
def test_linear_smallest_inputs(N, K, T):
    """fp32 x near the smallest normal numbers: its bf16 terms end at 2^-133, so each value is cut by less than that; and weights of
    2^128 or more, which are infinite, leave no finite result."""
    g = ops.gen(31)
    q, s, _ = ops.quantised(g, N, K, 0)
    s += 60                                                  # weights around 2^60
    x = ops.rand(g, T, K) * 2.0 ** -120
    mat, y = matrix(N, K, 0, F32), torch.empty(T, N, device="cuda")
    m.moe_linear(mat, q, s, 1.0, x, T, None, y)
    want = linear_bound(q, s, 0, 1.0, x, None)
    want.e += 2.0 ** -133 * ref.weights(q, s, 0).abs().sum(1)[None]
    ref.check(y, want, F32, "y")
    q[3] = 0x77                                              # every code 6
    s[3] = 254
    for act in (F32, BF16):
        xa = ops.rand(g, T, K, dtype=act)
        xa[xa == 0] = 1.0
        y, clean = torch.empty(T, N, dtype=act, device="cuda"), torch.empty(T, N, dtype=act, device="cuda")
        m.moe_linear(matrix(N, K, 0, act), q, s - 60, 1.0, xa, T, None, clean)
        s2 = s - 60
        s2[3] = 254
        m.moe_linear(matrix(N, K, 0, act), q, s2, 1.0, xa, T, None, y)
        rest = torch.arange(N, device="cuda") != 3
        assert not torch.isfinite(y[:, 3]).any() and torch.equal(y[:, rest], clean[:, rest])


# sizes at which each kernel takes a call: N, K, T, activations
KERNELS = [(256, 1152, 3, F32), (256, 1152, 8, F32), (4090, 1152, 16, F32), (16640, 1152, 3, F32), (16640, 4224, 5, F32),
           (9000, 7168, 4, F32), (24580, 4224, 7, F32), (16640, 512, 2, F32), (8448, 1152, 8, F32), (12300, 2176, 16, F32),
           (12300, 4224, 20, F32), (16640, 1152, 20, F32), (65540, 256, 33, F32), (256, 1152, 3, BF16), (256, 1152, 7, BF16),
           (256, 1152, 16, BF16), (4352, 1152, 33, BF16), (12300, 1152, 9, BF16), (16640, 2176, 7, BF16), (12300, 5120, 16, BF16),
           (16640, 7168, 12, BF16), (24580, 384, 7, BF16), (16640, 1152, 20, BF16), (16640, 1152, 40, BF16), (65540, 256, 40, BF16)]


@pytest.mark.parametrize("N,K,T,act", KERNELS)
def test_linear_scale_bytes_in_every_kernel(N, K, T, act):
    ops.test_linear_scale_bytes(N, K, T, act)


@pytest.mark.parametrize("N,K,T,act", KERNELS)
def test_linear_outside_the_numbers_in_every_kernel(N, K, T, act):
    """Infinity and NaN in x, a NaN whose payload lies in the lower half among them, reach that token alone, and the largest
    finite value stays finite on the way."""
    g = ops.gen(35)
    q, s, _ = ops.quantised(g, N, K, 0)
    x, mat = ops.rand(g, T, K, dtype=act), matrix(N, K, 0, act)
    y, z = torch.empty(T, N, dtype=act, device="cuda"), torch.empty(T, N, dtype=act, device="cuda")
    m.moe_linear(mat, q, s, 1.0, x, T, None, y)
    w = ref.weights(q, s, 0)[:, 200]
    for t, bits in ((0, None), (T - 1, float("nan")), (T // 2, 0x7f800001), (T // 2, -0x7ffff0)):
        if isinstance(bits, int) and act != F32:
            continue
        x2 = x.clone()
        if isinstance(bits, int):
            x2.view(torch.int32)[t, 200] = bits
        else:
            x2[t, 200] = float("inf") if bits is None else bits
        m.moe_linear(mat, q, s, 1.0, x2, T, None, z)
        rest = torch.arange(T, device="cuda") != t
        assert torch.equal(z[rest], y[rest])
        if bits is None:
            assert torch.equal(torch.isnan(z[t]), w == 0)    # 0 times infinity
            assert torch.equal(z[t][w != 0], (torch.sign(w) * float("inf")).to(act)[w != 0])
        else:
            assert torch.isnan(z[t]).all()
    x2 = torch.zeros_like(x)
    x2[:, 7] = torch.finfo(act).max
    low = torch.full_like(s, 100)
    m.moe_linear(mat, q, low, 1.0, x2, T, None, z)
    ref.check(z, linear_bound(q, low, 0, 1.0, x2, None), act, "y")


# ---------------------------------------------------------------------------------------------
# norm gradients
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,d,act,gate,post,y", [
    (601, 6144, BF16, 2, 1, 1), (601, 6144, F32, 1, 1, 1), (300, 8192, F32, 1, 1, 1), (520, 8320, BF16, 2, 1, 1), (520, 8320, F32, 0, 1, 1),
    (300, 16384, BF16, 1, 1, 1), (300, 16384, F32, 2, 1, 1), (2801, 6144, BF16, 2, 1, 1), (1401, 6144, F32, 2, 1, 1), (1400, 4224, BF16, 0, 0, 1),
    (2049, 640, BF16, 1, 1, 1), (5000, 128, F32, 2, 1, 1), (700, 8192, BF16, 0, 0, 0),
])
def test_norm_gradients_of_many_rows(T, d, act, gate, post, y):
    """Two to nineteen rows to a workgroup, so that its sums pass from row to row, with and without the next row requested ahead,
    through the caches and past them."""
    g, sh = ops.gen(32), ops.shape(d, act=act)
    i, wide = ops.norm_inputs(g, T, d, act, gate, post, y)
    dxo, dn = ops.rand(g, T, d, dtype=act), ops.rand(g, T, d, dtype=act)
    ws = m.workspace(sh, T)
    for a, b in ((dxo, dn), (dxo, None)) if y else ((dxo, dn),):
        out = ops.norm_gradients(sh, i, T, d, act, gate, post, y, a, b, ws)
        ops.check_gradients(out, ref.norm_backward(i["x"], i["y"], i["post"], i["pre"], wide, ops.ALPHA, EPS, a, b, gate == 1), act, gate)


@pytest.mark.parametrize("T,d", [(5, 640), (600, 1152), (300, 8320)])
@pytest.mark.parametrize("act", [BF16, F32])
def test_norm_gradients_keep_rows_apart(T, d, act):
    """A row of zeros has finite gradients, and NaN or infinity in one row of any input reaches that row of the row gradients, the
    gammas' gradients and nothing else."""
    g, sh = ops.gen(33), ops.shape(d, act=act)
    i, _ = ops.norm_inputs(g, T, d, act, 2, 1, 1)
    up = {"a": ops.rand(g, T, d, dtype=act), "b": ops.rand(g, T, d, dtype=act)}
    i["x"][1], i["y"][1] = 0.0, 0.0

    def run(i, up):
        return ops.norm_gradients(sh, i, T, d, act, 2, 1, 1, up["a"], up["b"])

    clean = run(i, up)
    assert all(torch.isfinite(v).all() for v in clean.values())
    bad = 3
    rest = torch.arange(T, device="cuda") != bad
    for name in ("x", "y", "gate", "a", "b"):
        for value in (float("nan"), float("inf")):
            i2, up2 = dict(i), dict(up)
            src = i2 if name in i2 else up2
            src[name] = src[name].clone()
            src[name][bad, 17] = value
            out = run(i2, up2)
            for k in ("dx", "dy", "d_gate"):
                assert torch.equal(out[k][rest], clean[k][rest]), (name, value, k)
            assert not torch.isfinite(out["dx"][bad, 17]), (name, value)


@pytest.mark.parametrize("T,d,act", [(4099, 4096, BF16), (2100, 8192, BF16), (2051, 4096, F32)])
def test_rows_larger_than_the_caches_in_place(T, d, act):
    """Each value is read before its place is written, past the caches too: outputs over the inputs, and over the upstream
    gradients, have the bits of outputs of their own, eagerly and replayed."""
    g, sh = ops.gen(36), ops.shape(d, act=act)
    i, _ = ops.norm_inputs(g, T, d, act, 2, 1, 1)
    up = [ops.rand(g, T, d, dtype=act) for _ in range(2)]
    tail = (i["post"], i["pre"], i["gate"], 2, ops.ALPHA, EPS)
    want = [torch.empty_like(i["x"]) for _ in range(2)]
    m.moe_block_norm(sh, i["x"], i["y"], T, *tail, *want)
    grads = ops.norm_gradients(sh, i, T, d, act, 2, 1, 1, *up)
    x, y, gate, a, b = (torch.empty_like(i["x"]) for _ in range(5))
    ws, sums = m.workspace(sh, T), [torch.empty(d, device="cuda") for _ in range(2)]

    def fill():
        for dst, src in ((x, i["x"]), (y, i["y"]), (gate, i["gate"]), (a, up[0]), (b, up[1])):
            dst.copy_(src)

    def forward():
        m.moe_block_norm(sh, x, y, T, i["post"], i["pre"], gate, 2, ops.ALPHA, EPS, x, y)

    def backward():
        m.moe_block_norm_backward(sh, x, y, T, i["post"], i["pre"], gate, 2, ops.ALPHA, EPS, a, b, a, b, gate, *sums, ws)

    for run, out in ((forward, ((x, want[0]), (y, want[1]))),
                     (backward, ((a, grads["dx"]), (b, grads["dy"]), (gate, grads["d_gate"]), (sums[0], grads["d_post"]),
                                 (sums[1], grads["d_pre"])))):
        fill()
        run()
        torch.cuda.synchronize()
        for got, ref_bits in out:
            assert torch.equal(got, ref_bits)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(3):
            fill()
            graph.replay()
            torch.cuda.synchronize()
            for got, ref_bits in out:
                assert torch.equal(got, ref_bits)


# ---------------------------------------------------------------------------------------------
# tokens by expert
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,d,k,E,act,shared", [(5, 640, 3, 7, BF16, 1), (129, 384, 16, 64, F32, 0), (333, 1152, 8, 256, F32, 1),
                                                (70, 4352, 8, 40, BF16, 0), (260, 256, 9, 33, BF16, 1)])
def test_what_no_pick_has_reaches_no_result(T, d, k, E, act, shared):
    """Rows past the last pick and the weights of dropped picks may hold anything: NaN there changes nothing, and NaN in a
    row that a pick has stays with its token."""
    g, sh = ops.gen(34), ops.shape(d, k, E, act, n_shared=shared, routed_scaling=2.5)
    _, w, _, sp, pos = ops.routing(g, sh, T, True)
    rows = T * (k + shared)
    o, dxs, x = ops.rand(g, rows, d), ops.rand(g, rows, d, dtype=act), ops.rand(g, T, d, dtype=act)
    pre = torch.ones(d, device="cuda")

    def run(o, dxs, w):
        out = {n: torch.zeros(s, dtype=t, device="cuda") for n, s, t in (("dx", (T, d), act), ("d_o", (rows, d), F32), ("d_w", (T, k), F32),
                                                                           ("u", (T, d), act), ("n", (T, d), act), ("y", (T, d), act))}
        m.moe_dispatch_backward(sh, dxs, T, pos, out["dx"])
        m.moe_combine_backward(sh, x, o, w, pos, T, out["d_o"], out["d_w"])
        m.moe_combine_norm(sh, o, w, pos, x, T, pre, pre, None, 0, 1.0, EPS, out["u"], out["n"])
        m.moe_combine(sh, o, w, pos, T, None, out["y"])
        return out

    clean = run(o, dxs, w)
    empty = torch.zeros(rows, dtype=torch.bool, device="cuda")
    empty[:T * k] = sp < 0
    assert empty.any() and not (pos < 0).all()
    o2, dxs2, w2 = o.clone(), dxs.clone(), w.clone()
    o2[empty], dxs2[empty], w2[pos < 0] = float("nan"), float("nan"), float("nan")
    out = run(o2, dxs2, w2)
    for n, v in clean.items():
        assert torch.equal(out[n], v), n
    at = (pos >= 0).nonzero()[-1]                             # the last kept pick's row
    t, row = int(at[0]), int(pos[at[0], at[1]])
    rest = torch.arange(T, device="cuda") != t
    o2[row, 5], dxs2[row, 5] = float("nan"), float("nan")
    out = run(o2, dxs2, w2)
    for n in ("dx", "d_w", "u", "n", "y"):
        assert torch.equal(out[n][rest], clean[n][rest]), n
    assert torch.equal(out["d_o"], clean["d_o"]) and torch.isnan(out["dx"][t, 5]) and torch.isnan(out["d_w"][t, at[1]])
    assert torch.isnan(out["u"][t]).all() and torch.isnan(out["y"][t, 5])
