"""Plain float64 forms of the operators around the experts, with a bound on the error of an fp32
evaluation carried along: every value is a pair (v, e) of the exact result for the given inputs and a
bound on how far a computation that rounds each step to fp32 may be from it.  No code is shared with the
library.

One rounding to fp32 is off by at most u = 2^-24 of the rounded value, and a sum of n values in which
no value passes more than `depth` additions by at most depth * u * sum |v| (to first order; the second-order
terms are covered by the 1 + 2^-10 that every bound is widened by at the end)."""
import torch

U = 2.0 ** -24


class Val:
    def __init__(self, v, e=None):
        self.v = v.double()
        self.e = torch.zeros_like(self.v) if e is None else e

    def _r(v, e):                            # one rounding of v, known to within e
        return Val(v, e + U * (v.abs() + e))

    def __mul__(a, b):
        b = b if isinstance(b, Val) else Val(torch.as_tensor(b, dtype=torch.float64, device=a.v.device))
        return Val._r(a.v * b.v, a.v.abs() * b.e + b.v.abs() * a.e + a.e * b.e)

    def __add__(a, b):
        return Val._r(a.v + b.v, a.e + b.e)

    def __neg__(a):
        return Val(-a.v, a.e)

    def sum(self, dim, depth, keepdim=True):
        return Val(self.v.sum(dim, keepdim), (self.e + depth * U * (self.v.abs() + self.e)).sum(dim, keepdim))

    def __getitem__(self, at):
        return Val(self.v[at], self.e[at])

    def bound(self, dtype):
        """How far the value may be once rounded to dtype: half a step more."""
        half = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
        return (self.e + half * (self.v.abs() + self.e)) * (1 + 2.0 ** -10) + 1e-37


def check(got, want, dtype, what):
    assert got.dtype == dtype, (what, got.dtype)
    g, v, b = got.double(), want.v, want.bound(dtype)
    nan = torch.isnan(v)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    off = ((g - v).abs() - b)[~nan]
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} beyond the bound; off by {(g - v).abs()[~nan].max().item():.3e}"


def row_depth(d):
    """Additions that a value passes in a row sum: eight columns per thread and vector (at most two
    vectors), six steps over a wave, sixteen waves."""
    return 16 + 6 + 16


def inv_rms(v, eps):
    """1 / sqrt(mean v^2 + eps): a relative error of the mean counts half, then the division by d, the
    added eps, the root and the division (two units each for root and division)."""
    d = v.v.shape[-1]
    s = (v * v).sum(-1, row_depth(d))
    mean, rel = s.v / d + eps, s.e / d / (s.v / d + eps) + 2 * U
    r = mean.rsqrt()
    return Val(r, r * (rel / 2 + 4 * U))


def norm_forward(x, y, post, pre, gate, alpha, eps):
    """(u, normed) of the block norm; gate broadcast to [T, d] or None; y a Val or None."""
    u = Val(x)
    if y is not None:
        z = y if post is None else y * inv_rms(y, eps) * Val(post)
        if gate is not None:
            z = z * Val(gate)
        u = u + z * alpha32(alpha)
    normed = None if pre is None else u * inv_rms(u, eps) * Val(pre)
    return u, normed


def alpha32(a):
    return float(torch.tensor(a, dtype=torch.float32))


def norm_backward(x, y, post, pre, gate, alpha, eps, d_x_out, d_normed, token_gate):
    """dict of Val: dx, dy, d_gate, d_post, d_pre (None where there is no such input)."""
    T, d = x.shape
    alpha = alpha32(alpha)
    one = Val(torch.ones(1, dtype=torch.float64, device=x.device))
    g = one if gate is None else Val(gate)
    ag = g * alpha
    u, yn, z, ry = Val(x), None, None, one
    if y is not None:
        if post is not None:
            ry = inv_rms(Val(y), eps)
        yn = Val(y) * ry if post is not None else Val(y)
        z = yn * (one if post is None else Val(post))
        u = u + z * ag
    du = Val(torch.zeros_like(x) if d_x_out is None else d_x_out)
    out = dict.fromkeys(("dx", "dy", "d_gate", "d_post", "d_pre"))
    # a sum over the tokens: the rows of one group (of at least 256), at most 2048 groups by 32 threads, 32 sums
    cols = -(-T // 256) + 64 + 32
    if d_normed is not None:
        dn = Val(d_normed)
        ru = inv_rms(u, eps)
        un = u * ru
        gn = dn * Val(pre)
        q = (gn * u).sum(-1, row_depth(d)) * ru * (1.0 / d)
        du = du + ru * (gn + -(un * q))
        out["d_pre"] = (dn * un).sum(0, cols, False)
    out["dx"] = du
    if y is None:
        return out
    dz = ag * du
    if gate is not None:
        dg = du * z
        out["d_gate"] = dg.sum(-1, row_depth(d), False) * alpha if token_gate else dg * alpha
    if post is not None:
        out["d_post"] = (dz * yn).sum(0, cols, False)
        t = dz * Val(post)
        m = (t * yn).sum(-1, row_depth(d)) * (1.0 / d)
        out["dy"] = ry * (t + -(yn * m))
    else:
        out["dy"] = dz
    return out


def picked(rows, pick_pos):
    """[T, k, d]: the row of each pick, zeros for a pick without one."""
    T, k = pick_pos.shape
    ok = (pick_pos >= 0) & (pick_pos < T * k)
    r = rows.double()[torch.where(ok, pick_pos, 0).long()]
    return torch.where(ok[..., None], r, 0.0)


def combine(o, w, pick_pos, scaling, shared):
    T, k = pick_pos.shape
    y = (Val(w[..., None].double().expand(T, k, o.shape[1])) * Val(picked(o, pick_pos))).sum(1, k + 1, False)
    y = y * alpha32(scaling)
    return y + Val(o[T * k:]) if shared else y


def dispatch_backward(dxs, pick_pos, shared):
    T, k = pick_pos.shape
    dx = Val(picked(dxs, pick_pos)).sum(1, k, False)
    return dx + Val(dxs[T * k:]) if shared else dx


def combine_backward_rows(dy, w, scaling):
    """[T, k, d]: each pick's row of d_o."""
    f = Val(w) * alpha32(scaling)
    return Val(f.v[..., None], f.e[..., None]) * Val(dy[:, None])


def combine_backward_weights(dy, o, pick_pos, scaling):
    d = dy.shape[1]
    dot = (Val(dy[:, None].double()) * Val(picked(o, pick_pos))).sum(-1, -(-d // 256) + 8, False)
    return dot * alpha32(scaling)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def weights(q, s, wformat):
    """float64 weight matrix without the tensor scale, from codes and scale bytes."""
    N, K = q.shape[0], q.shape[1] * 2
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=q.device)
    code = torch.stack([q & 15, q >> 4], -1).reshape(N, K).long()
    if wformat == 0:
        scale = torch.where(s == 255, float("nan"), torch.ldexp(torch.ones((), dtype=torch.float64, device=q.device),
                                                              s.int() - 127))
        block = 32
    else:
        scale, block = s.view(torch.float8_e4m3fn).double(), 16
    return table[code] * scale.repeat_interleave(block, 1)


def linear(q, s, wformat, ts, x, bias):
    """A product passes at most 32 additions in each of its wave's MFMAs (four per 128 columns, three
    times as many for fp32 x; the columns are shared out over at least four waves) and 16 over the waves."""
    W, x64 = weights(q, s, wformat), x.double()
    K = W.shape[1]
    steps = -(-(K // 128) // 4)
    depth = 32 * 4 * steps * (3 if x.dtype == torch.float32 else 1) + 16
    y, mag = x64 @ W.t().contiguous(), x64.abs() @ W.abs().t().contiguous()
    r = Val(y, depth * U * mag) * alpha32(ts)
    return r if bias is None else r + Val(bias)
