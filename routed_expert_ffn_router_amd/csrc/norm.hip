// The norms before and after a block, fused with its gate and residual scale, alone or with the
// weighted combine, and their gradient.
//
//   N(v; g) = g v r(v), r(v) = 1 / sqrt(mean v^2 + eps);   z = N(y; post) or y;
//   u = x + a gate z;   x_out = u;   normed = N(u; pre).
//
// A workgroup holds one row in registers, eight columns per thread and vector, so each row is read
// once and written once; the row sums go through DPP and LDS in a fixed order.  Bound by HBM where there
// are many rows (d 4096, bf16, with a gate: 4096 rows 31 us, 168 MB at 5.5 TB/s), by the chain load, sum,
// sum, store where there are few (one row 2.6 us).  Two vectors per thread and half the threads, tried for
// d 4096 to 8192, were slower (35 -> 39 us; the combine 45 -> 50).
#include "block_ops.h"

namespace moe {

// Sums of NS values over the workgroup, in every thread.  `slot` (16 waves x NS floats in LDS) must
// not be the one of the reduction before it: a wave may still read that one.
template <int NS>
__device__ __forceinline__ void block_sums(float (&v)[NS], float* slot) {
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = wave_sum_f32(v[i]);
    const int nw = blockDim.x >> 6;
    if (nw == 1) return;
    const int wv = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < NS; ++i) slot[wv * NS + i] = v[i];
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = 0.0f;
    for (int w = 0; w < nw; ++w) {
#pragma unroll
        for (int i = 0; i < NS; ++i) v[i] += slot[w * NS + i];
    }
}

__device__ __forceinline__ float inv_rms(float sum_sq, int d, float eps) {
    return 1.0f / sqrtf(sum_sq / (float)d + eps);
}

// the combine's sum for columns c .. c + 7 of token t, in k_combine's order
template <int MAXN>
__device__ __forceinline__ f32x8 combine8(const NormArgs& a, int t, int c) {
    const int P = a.T * a.k;
    f32x8 acc = {};
    for_picks<MAXN>(a.pick_pos + (size_t)t * a.k, a.k, P, [&](auto n, const int (&row)[MAXN], const bool (&has)[MAXN], int j0) {
        constexpr int N = decltype(n)::value;
        Raw8<float> v[N];
        float w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i].load(a.o, (size_t)row[i] * a.d + c);
            w[i] = a.w[(size_t)t * a.k + (j0 + i < a.k ? j0 + i : j0)];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const f32x8 o = v[i].values();
#pragma unroll
            for (int e = 0; e < 8; ++e) acc.v[e] = has[i] ? fmaf(w[i], o.v[e], acc.v[e]) : acc.v[e];
        }
    });
#pragma unroll
    for (int e = 0; e < 8; ++e) acc.v[e] *= a.scaling;
    if (a.shared) {
        const f32x8 v = load_act8(a.o, ((size_t)P + t) * a.d + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc.v[e] += v.v[e];
    }
    return acc;
}

// One row per workgroup; thread i holds columns 8 (i + n blockDim) .. + 7 for n < VPT.
// COMBINE: 0, or the picks whose rows are loaded together.  LATE: the gate and the gammas are loaded when
// they are used, which saves registers for more rows per CU (with eight picks and early loads one row of
// d 6144 fits on a CU, so two); else with the row, before the first sum waits.
// Combined, 8 picks: 64 tokens, d 4096 5.7 us; 1001 tokens, d 6144, fp32, one to eight picks kept at random 44 us
// (185 MB at 4.2 TB/s: two rows at a time on a CU do not cover each other's sums); kept 1, 8, 7, .. 2 in turn
// 46, since workgroups go to the eight XCDs in turn.
// MX8: the normed row goes out as MXFP8, a block of 32 columns in four neighbouring lanes.  4096 rows of 4096, bf16, gate
// per element, 30.7 us (151 MB at 4.9 TB/s), fp32 51 (286 MB at 5.6 TB/s); one row 7.1, the call's host time.
template <typename XT, int VPT, int COMBINE, bool LATE, bool NT, bool MX8 = false>
__global__ __launch_bounds__(1024) void k_block_norm(NormArgs a) {
    __shared__ float s_post[16], s_pre[16];
    const int t = blockIdx.x;
    const size_t base = (size_t)t * a.d;
    const bool has_y = COMBINE || a.y, element = a.gate_kind == MOE_GATE_ELEMENT;
    auto col = [&](int n) { return 8 * (int)(threadIdx.x + n * blockDim.x); };
    f32x8 u[VPT], z[VPT], pre[VPT], post[VPT];
    Raw8<XT> gate[VPT];
    auto load_after = [&](int n) {            // what multiplies z
        if (element) gate[n].template load<NT>((const XT*)a.gate, base + col(n));
        if (a.post) post[n] = load_act8(a.post, (size_t)col(n));
    };
    float sum[1] = {0.0f};
#pragma unroll
    for (int n = 0; n < VPT; ++n) {
        u[n] = z[n] = f32x8{};
        if (col(n) >= a.d) continue;
        u[n] = load_act8<NT>((const XT*)a.x, base + col(n));
        if constexpr (!LATE) {
            load_after(n);
            if (a.pre) pre[n] = load_act8(a.pre, (size_t)col(n));
        }
        if constexpr (COMBINE > 0) z[n] = combine8<COMBINE>(a, t, col(n));
        else if (has_y) z[n] = load_act8<NT>((const XT*)a.y, base + col(n));
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(z[n].v[e], z[n].v[e], sum[0]);
    }
    if (has_y) {
        float r = 1.0f;
        if (a.post) {
            block_sums(sum, s_post);
            r = inv_rms(sum[0], a.d, a.eps);
        }
        const float gt = a.alpha * (a.gate_kind == MOE_GATE_TOKEN ? ((const float*)a.gate)[t] : 1.0f);
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            if (col(n) >= a.d) continue;
            if constexpr (LATE) load_after(n);
            if (a.post) {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[n].v[e] *= r * post[n].v[e];
            }
            if (element) {
                const f32x8 g = gate[n].values();
#pragma unroll
                for (int e = 0; e < 8; ++e) z[n].v[e] *= g.v[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) u[n].v[e] = fmaf(gt, z[n].v[e], u[n].v[e]);
        }
    }
    sum[0] = 0.0f;
#pragma unroll
    for (int n = 0; n < VPT; ++n) {
        if (col(n) >= a.d) continue;
        if (a.x_out) store_act8<NT>((XT*)a.x_out, base + col(n), u[n]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(u[n].v[e], u[n].v[e], sum[0]);
    }
    if (!MX8 && !a.normed) return;
    float r = 1.0f;
    if (!MX8 || a.pre) {
        block_sums(sum, s_pre);
        r = inv_rms(sum[0], a.d, a.eps);
    }
#pragma unroll
    for (int n = 0; n < VPT; ++n) {
        if (col(n) >= a.d) continue;
        if (LATE && (!MX8 || a.pre)) pre[n] = load_act8(a.pre, (size_t)col(n));
        if (!MX8 || a.pre) {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[n].v[e] *= r * pre[n].v[e];
        }
        if constexpr (MX8) {
            uint8_t scale;
            const uint2 c = mx8_codes(u[n], quad_max(mx8_amax(u[n])), &scale);
            *(uint2*)(a.codes + base + col(n)) = c;
            if (threadIdx.x % 4 == 0) a.scales[(base + col(n)) / 32] = scale;
        } else {
            store_act8((XT*)a.normed, base + col(n), u[n]);    // the next kernel reads it
        }
    }
}

// Bytes of one row array from which bf16 rows go past the caches (the eight L2s together), but for normed, which the
// router or dispatch reads next.  4096 rows, d 4096, gate per element: the norm alone 32.2 us, all of it through the
// caches 33.4; then route and dispatch (4 picks) 134.5, 142.9, with normed past the caches too 138.5; 16384 rows 112 and
// 484, 122 and 489, 116 and 507.  fp32 rows stay in the caches: 4096 rows 62 us, past them 68, with route and dispatch
// 185, 196.
constexpr size_t kStreamRows = (size_t)32 << 20;
template <typename XT>
static bool past_caches(int T, int d) {
    return sizeof(XT) == 2 && (size_t)T * d * sizeof(XT) >= kStreamRows;
}

// threads of a workgroup for rows of d columns, eight per thread and vector
static int norm_threads(int d, int* vpt) {
    const int nv = d / 8;
    *vpt = nv <= 1024 ? 1 : 2;                 // d <= 16384
    const int per = (nv + *vpt - 1) / *vpt;
    return (per + 63) / 64 * 64;
}

template <typename XT>
static void norm_launch(const NormArgs& a, hipStream_t st) {
    int vpt;
    const dim3 grid(a.T), block(norm_threads(a.d, &vpt));
    if (a.o) {
        // the combine: with more rows than CUs, four picks at a time and late loads.  Never past the caches: 4096 tokens,
        // d 4096, bf16 127 us, past them 135, 16384 502 for 556 (fp32 569 for 655); after a kernel that writes o 854 for
        // 895 (914 for 983; only there, with 384 to 768 MB of o and bf16 rows, past them gained: 4096 tokens 222 for 233).
        if (vpt == 2) MOE_LAUNCH((k_block_norm<XT, 2, 4, true, false>), grid, block, 0, st, a);
        else if (a.T > 256) MOE_LAUNCH((k_block_norm<XT, 1, 4, true, false>), grid, block, 0, st, a);
        else MOE_LAUNCH((k_block_norm<XT, 1, 8, false, false>), grid, block, 0, st, a);
    } else if (vpt == 2) {
        MOE_LAUNCH((k_block_norm<XT, 2, 0, true, false>), grid, block, 0, st, a);
    } else if (past_caches<XT>(a.T, a.d)) {
        MOE_LAUNCH((k_block_norm<XT, 1, 0, false, sizeof(XT) == 2>), grid, block, 0, st, a);
    } else {
        MOE_LAUNCH((k_block_norm<XT, 1, 0, false, false>), grid, block, 0, st, a);
    }
}

template <typename XT>
static void norm_mx8_launch(const NormArgs& a, hipStream_t st) {
    int vpt;
    const dim3 grid(a.T), block(norm_threads(a.d, &vpt));
    if (vpt == 2) MOE_LAUNCH((k_block_norm<XT, 2, 0, true, false, true>), grid, block, 0, st, a);
    else MOE_LAUNCH((k_block_norm<XT, 1, 0, false, false, true>), grid, block, 0, st, a);
}

hipError_t launch_block_norm(const moe_shape* s, const NormArgs& a, hipStream_t st) {
    const char* name = a.o ? "combine_norm" : a.codes ? "block_norm_mx8" : "block_norm";
    trace(name, 0, st);
    if (a.codes && s->act_dtype == MOE_DT_BF16) norm_mx8_launch<uint16_t>(a, st);
    else if (a.codes) norm_mx8_launch<float>(a, st);
    else if (s->act_dtype == MOE_DT_BF16) norm_launch<uint16_t>(a, st);
    else norm_launch<float>(a, st);
    trace(name, 1, st);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// gradient: with yn = y r(y), un = u r(u), gn = d_normed pre and q = mean(gn un),
//   du = d_x_out + r(u) (gn - un q);   dx = du;   d_pre = sum_t d_normed un;
//   dz = a gate du;   d_gate = a du z (its row sum for a gate per token);   d_post = sum_t dz yn;
//   dy = r(y) (dz post - yn mean(dz post yn)),  or dz without a post-norm.
// A workgroup takes rows b, b + G, ... (G workgroups) and keeps its columns' sums of d_post and d_pre
// itself; k_norm_grad_sums adds the workgroups' sums in order.  Bound by HBM: 4096 rows, d 4096, bf16, with a
// gate per element: 51 us, 277 MB at 5.4 TB/s, and 4.7 us for the sums; fp32 112 us at 5.0 TB/s, with 20 bytes of a lane
// spilled.  Requesting the next row before the sums of this one needs its registers: the gammas wait in LDS (72 -> 54 us
// with both, fewer groups, and rows past the caches).  Past 8192 columns a CU holds one row and none ahead: 2048 bf16
// rows of 12288 113 us at 3.6 TB/s (28 bytes spilled, fp32 72).
// ---------------------------------------------------------------------------------------------
// Groups: a row's chain of three sums takes about 2 us, so a CU needs some 64 KB of rows at once to keep its
// share of HBM busy: one workgroup per CU for long rows, up to eight for short ones.  More only add partial sums
// to write and read (4096 rows, 256 / 512 groups: d 4096 bf16 55 / 60 us, d 1024 41 / 28).  Up to two
// rows one workgroup takes them all and no second kernel runs (d 4096 bf16: 2, 3, 4 rows 7.2, 9.5, 11.8 us, in
// groups 7.7).
static int norm_groups_cap(const moe_shape* s) {
    const int row = 8 * s->d_model * (s->act_dtype == MOE_DT_BF16 ? 2 : 4);       // bytes of a row, in and out
    return 256 * (row >= 65536 ? 1 : 65536 / row < 8 ? (65536 + row - 1) / row : 8);
}

static int norm_grad_groups(const moe_shape* s, int T) {
    if (T <= 2) return 1;
    const int cap = norm_groups_cap(s), rows = (T + cap - 1) / cap;
    return (T + rows - 1) / rows;
}

int norm_grad_groups_most(const moe_shape* s, int T) {
    const int cap = norm_groups_cap(s);
    return T <= 2 ? 1 : T < cap ? T : cap;
}

// One row's loads, as they come: requested for the next row while this one is worked on
template <typename XT, int VPT>
struct NormRow {
    Raw8<XT> x[VPT], y[VPT], du[VPT], dn[VPT], gate[VPT];
};

template <typename XT, int VPT, int THREADS, bool NT>
__global__ __launch_bounds__(THREADS, 4) void k_block_norm_backward(NormArgs a, NormGradArgs g) {
    constexpr bool AHEAD = VPT == 1;          // (two vectors per thread leave no registers for the next row)
    // two sets, for odd and even rows: with one sum a row, a wave may still read the last row's
    __shared__ float s_y[2][16], s_u[2][32], s_d[2][32];
    const bool element = a.gate_kind == MOE_GATE_ELEMENT, token = a.gate_kind == MOE_GATE_TOKEN;
    auto col = [&](int n) { return 8 * (int)(threadIdx.x + n * blockDim.x); };
    auto load_row = [&](int t, NormRow<XT, VPT>& r) {
        const size_t base = (size_t)t * a.d;
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            r.x[n].clear();
            r.y[n].clear();
            r.du[n].clear();
            r.dn[n].clear();
            r.gate[n].clear();
            if (col(n) >= a.d) continue;
            const size_t i = base + col(n);
            r.x[n].template load<NT>((const XT*)a.x, i);
            if (a.y) r.y[n].template load<NT>((const XT*)a.y, i);
            if (g.d_x_out) r.du[n].template load<NT>((const XT*)g.d_x_out, i);
            if (g.d_normed) r.dn[n].template load<NT>((const XT*)g.d_normed, i);
            if (element) r.gate[n].template load<NT>((const XT*)a.gate, i);
        }
    };
    auto gamma = [&](const float* p, int n) {
        f32x8 r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = 1.0f;
        if (p && col(n) < a.d) r = load_act8(p, (size_t)col(n));
        return r;
    };
    // LDS that only its own thread reads and writes: the gammas of its columns, or, with two vectors per
    // thread, their sums (the sums of one vector stay in registers)
    __shared__ float s_own[2][8 * THREADS * VPT];
    auto own = [&](int w, int n) { return &s_own[w][8 * (threadIdx.x + n * THREADS)]; };
    auto get = [&](int w, int n) {
        const float4 p = *(const float4*)own(w, n), q = *(const float4*)(own(w, n) + 4);
        return f32x8{{p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w}};
    };
    auto put = [&](int w, int n, const f32x8& r) {
        *(float4*)own(w, n) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
        *(float4*)(own(w, n) + 4) = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
    };
    auto post_of = [&](int n) { return VPT == 1 ? get(0, n) : gamma(a.post, n); };
    auto pre_of = [&](int n) { return VPT == 1 ? get(1, n) : gamma(a.pre, n); };
    f32x8 acc_post = {}, acc_pre = {};
    if constexpr (VPT == 1) {
        put(0, 0, gamma(a.post, 0));
        put(1, 0, gamma(a.pre, 0));
    } else {
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            put(0, n, f32x8{});
            put(1, n, f32x8{});
        }
    }
    auto add_post = [&](int n, const f32x8& p, const f32x8& q) {          // sums += p q
        f32x8 s = VPT == 1 ? acc_post : get(0, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) s.v[e] = fmaf(p.v[e], q.v[e], s.v[e]);
        if constexpr (VPT == 1) acc_post = s;
        else put(0, n, s);
    };
    auto add_pre = [&](int n, const f32x8& p, const f32x8& q) {
        f32x8 s = VPT == 1 ? acc_pre : get(1, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) s.v[e] = fmaf(p.v[e], q.v[e], s.v[e]);
        if constexpr (VPT == 1) acc_pre = s;
        else put(1, n, s);
    };
    NormRow<XT, VPT> row;
    if (AHEAD) load_row(blockIdx.x, row);
    int odd = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, odd ^= 1) {
        const size_t base = (size_t)t * a.d;
        if (!AHEAD) load_row(t, row);
        f32x8 x[VPT], y[VPT], du[VPT], dn[VPT];
        Raw8<XT> gate_raw[VPT];
        const float gt = a.alpha * (token ? ((const float*)a.gate)[t] : 1.0f);
        float sy[1] = {0.0f};
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            x[n] = row.x[n].values();
            y[n] = row.y[n].values();
            du[n] = row.du[n].values();
            dn[n] = row.dn[n].values();
            gate_raw[n] = row.gate[n];
#pragma unroll
            for (int e = 0; e < 8; ++e) sy[0] = fmaf(y[n].v[e], y[n].v[e], sy[0]);
        }
        if (AHEAD && t + (int)gridDim.x < a.T) load_row(t + gridDim.x, row);
        // a gate of column vector n
        auto gate_of = [&](int n) {
            f32x8 r = gate_raw[n].values();
#pragma unroll
            for (int e = 0; e < 8; ++e) r.v[e] = element ? a.alpha * r.v[e] : gt;
            return r;
        };
        float ry = 1.0f;
        if (a.post) {
            block_sums(sy, s_y[odd]);
            ry = inv_rms(sy[0], a.d, a.eps);
        }
        // y becomes yn (or stays y), x becomes u, dn becomes gn
        float su[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            const f32x8 post = post_of(n), pre = pre_of(n);
            const f32x8 ag = gate_of(n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[n].v[e] *= ry;
                x[n].v[e] = fmaf(ag.v[e], y[n].v[e] * post.v[e], x[n].v[e]);
                su[0] = fmaf(x[n].v[e], x[n].v[e], su[0]);
                su[1] = fmaf(dn[n].v[e] * pre.v[e], x[n].v[e], su[1]);
            }
        }
        if (g.d_normed) {
            block_sums(su, s_u[odd]);
            const float ru = inv_rms(su[0], a.d, a.eps);
            const float q = su[1] * ru / (float)a.d;
#pragma unroll
            for (int n = 0; n < VPT; ++n) {
                const f32x8 pre = pre_of(n);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[n].v[e] *= ru;                 // un
                add_pre(n, dn[n], x[n]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    du[n].v[e] = fmaf(ru, fmaf(-x[n].v[e], q, dn[n].v[e] * pre.v[e]), du[n].v[e]);
            }
        }
        // dn becomes dz post; sums of dz post yn and of du z
        float sd[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            const f32x8 post = post_of(n), ag = gate_of(n);
            f32x8 dg, dz;
#pragma unroll
            for (int e = 0; e < 8; ++e) dz.v[e] = ag.v[e] * du[n].v[e];
            add_post(n, dz, y[n]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dn[n].v[e] = dz.v[e] * post.v[e];
                sd[0] = fmaf(dn[n].v[e], y[n].v[e], sd[0]);
                dg.v[e] = du[n].v[e] * (y[n].v[e] * post.v[e]);
                sd[1] += dg.v[e];
            }
            if (col(n) >= a.d) continue;
            if (g.dx) store_act8<NT>((XT*)g.dx, base + col(n), du[n]);
            if (g.d_gate && element) {
#pragma unroll
                for (int e = 0; e < 8; ++e) dg.v[e] *= a.alpha;
                store_act8<NT>((XT*)g.d_gate, base + col(n), dg);
            }
        }
        if (!a.y) continue;
        float m = 0.0f;
        if (a.post || (g.d_gate && token)) {
            block_sums(sd, s_d[odd]);
            m = a.post ? sd[0] / (float)a.d : 0.0f;
            if (g.d_gate && token && threadIdx.x == 0) ((float*)g.d_gate)[t] = a.alpha * sd[1];
        }
        if (!g.dy) continue;
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            if (col(n) >= a.d) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) dn[n].v[e] = ry * fmaf(-y[n].v[e], m, dn[n].v[e]);
            store_act8<NT>((XT*)g.dy, base + col(n), dn[n]);
        }
    }
    if (!g.d_post && !g.d_pre) return;
    // one group's sums are the gradients; the others' go to the workspace
    float* part = g.part + (size_t)blockIdx.x * 2 * a.d;
    float* post_out = gridDim.x == 1 ? g.d_post : part;
    float* pre_out = gridDim.x == 1 ? g.d_pre : part + a.d;
#pragma unroll
    for (int n = 0; n < VPT; ++n) {
        if (col(n) >= a.d) continue;
        if (g.d_post) store_act8(post_out, (size_t)col(n), VPT == 1 ? acc_post : get(0, n));
        if (g.d_pre) store_act8(pre_out, (size_t)col(n), VPT == 1 ? acc_pre : get(1, n));
    }
}

// d_post and d_pre from the groups' sums: a workgroup adds 32 columns (four per thread), 32 threads each
// every 32nd group, eight loads in flight, and then those 32 sums, in order
__global__ __launch_bounds__(256) void k_norm_grad_sums(const float* __restrict__ part, int groups, int d,
                                                        float* __restrict__ d_post, float* __restrict__ d_pre) {
    __shared__ float4 s_sum[32][8];
    const int col = (threadIdx.x & 7) * 4 + blockIdx.x * 32;          // of the 2 d columns; d % 32 = 0
    const int q = threadIdx.x >> 3;
    float* out = blockIdx.x * 32 < (unsigned)d ? d_post : d_pre;
    if (!out) return;                                                  // uniform
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b0 = q; b0 < groups; b0 += 256) {
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *(const float4*)(part + (size_t)(b0 + 32 * i < groups ? b0 + 32 * i : q) * 2 * d + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = b0 + 32 * i < groups;
            s.x += in ? v[i].x : 0.0f;
            s.y += in ? v[i].y : 0.0f;
            s.z += in ? v[i].z : 0.0f;
            s.w += in ? v[i].w : 0.0f;
        }
    }
    s_sum[q][threadIdx.x & 7] = s;
    __syncthreads();
    if (q) return;
    for (int i = 1; i < 32; ++i) {
        const float4 v = s_sum[i][threadIdx.x];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    *(float4*)(out + (col < d ? col : col - d)) = s;
}

template <typename XT>
static void norm_backward_launch(const NormArgs& a, const NormGradArgs& g, int groups, hipStream_t st) {
    int vpt;
    const int threads = norm_threads(a.d, &vpt);
    const dim3 grid(groups);
    // as the forward pass; dy, which the combine's gradient reads next, past the caches too (d 4096, gate per element, 2
    // picks: 8192 bf16 rows 98 us, with the combine's gradient 238, through the caches 104 and 239; 4096 fp32 rows 122 and
    // 197, 113 and 187)
    const bool nt = past_caches<XT>(a.T, a.d);
    constexpr bool NT = sizeof(XT) == 2;
    if (vpt == 2) MOE_LAUNCH((k_block_norm_backward<XT, 2, 1024, false>), grid, dim3(threads), 0, st, a, g);
    else if (threads > 512 && nt) MOE_LAUNCH((k_block_norm_backward<XT, 1, 1024, NT>), grid, dim3(threads), 0, st, a, g);
    else if (threads > 512) MOE_LAUNCH((k_block_norm_backward<XT, 1, 1024, false>), grid, dim3(threads), 0, st, a, g);
    else if (nt) MOE_LAUNCH((k_block_norm_backward<XT, 1, 512, NT>), grid, dim3(threads), 0, st, a, g);
    else MOE_LAUNCH((k_block_norm_backward<XT, 1, 512, false>), grid, dim3(threads), 0, st, a, g);
}

hipError_t launch_block_norm_backward(const moe_shape* s, const NormArgs& a, const NormGradArgs& g, hipStream_t st) {
    trace("block_norm_backward", 0, st);
    const int groups = a.T > 0 ? norm_grad_groups(s, a.T) : 0;
    if (groups > 0) {
        if (s->act_dtype == MOE_DT_BF16) norm_backward_launch<uint16_t>(a, g, groups, st);
        else norm_backward_launch<float>(a, g, groups, st);
    }
    if ((g.d_post || g.d_pre) && groups != 1)
        MOE_LAUNCH(k_norm_grad_sums, dim3(2 * a.d / 32), dim3(256), 0, st, (const float*)g.part, groups, a.d, g.d_post,
                   g.d_pre);
    trace("block_norm_backward", 1, st);
    return hipGetLastError();
}

}  // namespace moe
