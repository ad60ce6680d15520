// The norms before and after a block, fused with its gate and residual scale, alone or with the
// weighted combine, and their gradient.
//
//   N(v; g) = g v r(v), r(v) = 1 / sqrt(mean v^2 + eps);   z = N(y; post) or y;
//   u = x + a gate z;   x_out = u;   normed = N(u; pre).
//
// A workgroup holds one row in registers, eight columns per thread and vector, so each row is read
// once and written once; the row sums go through DPP and LDS in a fixed order.
#include "moe_internal.h"

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
__device__ __forceinline__ f32x8 combine8(const NormArgs& a, int t, int c) {
    const int P = a.T * a.k;
    f32x8 acc = {};
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        int row[8];
        float wj[8];
        f32x8 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const size_t p = (size_t)t * a.k + j0 + i;
            row[i] = j0 + i < a.k ? a.pick_pos[p] : -1;
            wj[i] = j0 + i < a.k ? a.w[p] : 0.0f;
            if ((unsigned)row[i] >= (unsigned)P) row[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = load_act8(a.o, (size_t)(row[i] >= 0 ? row[i] : 0) * a.d + c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc.v[e] = row[i] >= 0 ? fmaf(wj[i], v[i].v[e], acc.v[e]) : acc.v[e];
    }
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
template <typename XT, int VPT, bool COMBINE>
__global__ __launch_bounds__(1024) void k_block_norm(NormArgs a) {
    __shared__ float s_post[16], s_pre[16];
    const int t = blockIdx.x;
    const size_t base = (size_t)t * a.d;
    const bool has_y = COMBINE || a.y;
    f32x8 u[VPT], z[VPT], gate[VPT], post[VPT], pre[VPT];
    float sum[1] = {0.0f};
    // every load of the row is requested before the first sum waits
#pragma unroll
    for (int n = 0; n < VPT; ++n) {
        const int c = 8 * (threadIdx.x + n * blockDim.x);
        u[n] = z[n] = gate[n] = post[n] = pre[n] = f32x8{};
        if (c >= a.d) continue;
        u[n] = load_act8((const XT*)a.x, base + c);
        if (a.gate_kind == MOE_GATE_ELEMENT) gate[n] = load_act8((const XT*)a.gate, base + c);
        if (a.post) post[n] = load_act8(a.post, (size_t)c);
        if (a.pre) pre[n] = load_act8(a.pre, (size_t)c);
        if constexpr (COMBINE) z[n] = combine8(a, t, c);
        else if (has_y) z[n] = load_act8((const XT*)a.y, base + c);
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
            const int c = 8 * (threadIdx.x + n * blockDim.x);
            if (c >= a.d) continue;
            if (a.post) {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[n].v[e] *= r * post[n].v[e];
            }
            if (a.gate_kind == MOE_GATE_ELEMENT) {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[n].v[e] *= gate[n].v[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) u[n].v[e] = fmaf(gt, z[n].v[e], u[n].v[e]);
        }
    }
    sum[0] = 0.0f;
#pragma unroll
    for (int n = 0; n < VPT; ++n) {
        const int c = 8 * (threadIdx.x + n * blockDim.x);
        if (c >= a.d) continue;
        if (a.x_out) store_act8((XT*)a.x_out, base + c, u[n]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(u[n].v[e], u[n].v[e], sum[0]);
    }
    if (!a.normed) return;
    block_sums(sum, s_pre);
    const float r = inv_rms(sum[0], a.d, a.eps);
#pragma unroll
    for (int n = 0; n < VPT; ++n) {
        const int c = 8 * (threadIdx.x + n * blockDim.x);
        if (c >= a.d) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) u[n].v[e] *= r * pre[n].v[e];
        store_act8((XT*)a.normed, base + c, u[n]);
    }
}

// threads of a workgroup for rows of d columns, eight per thread and vector
static int norm_threads(int d, int* vpt) {
    const int nv = d / 8;
    *vpt = nv <= 1024 ? 1 : 2;                 // d <= 16384
    const int per = (nv + *vpt - 1) / *vpt;
    return (per + 63) / 64 * 64;
}

template <typename XT, int VPT>
static void norm_launch(const NormArgs& a, int threads, hipStream_t st) {
    if (a.o) MOE_LAUNCH((k_block_norm<XT, VPT, true>), dim3(a.T), dim3(threads), 0, st, a);
    else MOE_LAUNCH((k_block_norm<XT, VPT, false>), dim3(a.T), dim3(threads), 0, st, a);
}

hipError_t launch_block_norm(const moe_shape* s, const NormArgs& a, hipStream_t st) {
    const char* name = a.o ? "combine_norm" : "block_norm";
    trace(name, 0, st);
    int vpt;
    const int threads = norm_threads(a.d, &vpt);
    const bool bf = s->act_dtype == MOE_DT_BF16;
    if (vpt == 1) bf ? norm_launch<uint16_t, 1>(a, threads, st) : norm_launch<float, 1>(a, threads, st);
    else bf ? norm_launch<uint16_t, 2>(a, threads, st) : norm_launch<float, 2>(a, threads, st);
    trace(name, 1, st);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// gradient: with yn = y r(y), un = u r(u), gn = d_normed pre and q = mean(gn un),
//   du = d_x_out + r(u) (gn - un q);   dx = du;   d_pre = sum_t d_normed un;
//   dz = a gate du;   d_gate = a du z (its row sum for a gate per token);   d_post = sum_t dz yn;
//   dy = r(y) (dz post - yn mean(dz post yn)),  or dz without a post-norm.
// A workgroup takes rows b, b + G, ... (G workgroups) and keeps its columns' sums of d_post and d_pre
// in registers; k_norm_grad_sums adds the workgroups' sums in order.
// ---------------------------------------------------------------------------------------------
constexpr int kNormGroups = 512;

int norm_grad_groups(int T) { return T < kNormGroups ? T : kNormGroups; }

template <typename XT, int VPT>
__global__ __launch_bounds__(1024) void k_block_norm_backward(NormArgs a, NormGradArgs g) {
    // two sets, for odd and even rows: with one sum a row, a wave may still read the last row's
    __shared__ float s_y[2][16], s_u[2][32], s_d[2][32];
    int odd = 0;
    f32x8 acc_post[VPT], acc_pre[VPT];
#pragma unroll
    for (int n = 0; n < VPT; ++n) acc_post[n] = acc_pre[n] = f32x8{};
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, odd ^= 1) {
        const size_t base = (size_t)t * a.d;
        f32x8 x[VPT], y[VPT], du[VPT], dn[VPT], gate[VPT], pre[VPT], post[VPT];
        float sy[1] = {0.0f};
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            const int c = 8 * (threadIdx.x + n * blockDim.x);
            x[n] = y[n] = du[n] = dn[n] = gate[n] = pre[n] = post[n] = f32x8{};
            if (c >= a.d) continue;
            x[n] = load_act8((const XT*)a.x, base + c);
            if (a.y) y[n] = load_act8((const XT*)a.y, base + c);
            if (g.d_x_out) du[n] = load_act8((const XT*)g.d_x_out, base + c);
            if (g.d_normed) dn[n] = load_act8((const XT*)g.d_normed, base + c);
            if (a.gate_kind == MOE_GATE_ELEMENT) gate[n] = load_act8((const XT*)a.gate, base + c);
            if (a.pre) pre[n] = load_act8(a.pre, (size_t)c);
            if (a.post) post[n] = load_act8(a.post, (size_t)c);
#pragma unroll
            for (int e = 0; e < 8; ++e) sy[0] = fmaf(y[n].v[e], y[n].v[e], sy[0]);
        }
        const float gt = a.gate_kind == MOE_GATE_TOKEN ? ((const float*)a.gate)[t] : 1.0f;
        float ry = 1.0f;
        if (a.post) {
            block_sums(sy, s_y[odd]);
            ry = inv_rms(sy[0], a.d, a.eps);
        }
        // y becomes yn (or stays y), x becomes u, gate becomes a gate
        float su[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[n].v[e] *= ry;
                if (!a.post) post[n].v[e] = 1.0f;
                gate[n].v[e] = a.alpha * (a.gate_kind == MOE_GATE_ELEMENT ? gate[n].v[e] : gt);
                x[n].v[e] = fmaf(gate[n].v[e], y[n].v[e] * post[n].v[e], x[n].v[e]);
                su[0] = fmaf(x[n].v[e], x[n].v[e], su[0]);
                su[1] = fmaf(dn[n].v[e] * pre[n].v[e], x[n].v[e], su[1]);
            }
        }
        if (g.d_normed) {
            block_sums(su, s_u[odd]);
            const float ru = inv_rms(su[0], a.d, a.eps);
            const float q = su[1] * ru / (float)a.d;
#pragma unroll
            for (int n = 0; n < VPT; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float un = x[n].v[e] * ru;
                    acc_pre[n].v[e] = fmaf(dn[n].v[e], un, acc_pre[n].v[e]);
                    du[n].v[e] = fmaf(ru, fmaf(-un, q, dn[n].v[e] * pre[n].v[e]), du[n].v[e]);
                }
        }
        // dn becomes dz post; sums of dz post yn and of du z
        float sd[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            const int c = 8 * (threadIdx.x + n * blockDim.x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dz = gate[n].v[e] * du[n].v[e];
                acc_post[n].v[e] = fmaf(dz, y[n].v[e], acc_post[n].v[e]);
                dn[n].v[e] = dz * post[n].v[e];
                sd[0] = fmaf(dn[n].v[e], y[n].v[e], sd[0]);
                gate[n].v[e] = du[n].v[e] * (y[n].v[e] * post[n].v[e]);
                sd[1] += gate[n].v[e];
            }
            if (c >= a.d) continue;
            if (g.dx) store_act8((XT*)g.dx, base + c, du[n]);
            if (g.d_gate && a.gate_kind == MOE_GATE_ELEMENT) {
#pragma unroll
                for (int e = 0; e < 8; ++e) gate[n].v[e] *= a.alpha;
                store_act8((XT*)g.d_gate, base + c, gate[n]);
            }
        }
        if (!a.y) continue;
        float m = 0.0f;
        if (a.post || (g.d_gate && a.gate_kind == MOE_GATE_TOKEN)) {
            block_sums(sd, s_d[odd]);
            m = a.post ? sd[0] / (float)a.d : 0.0f;
            if (g.d_gate && a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0) ((float*)g.d_gate)[t] = a.alpha * sd[1];
        }
        if (!g.dy) continue;
#pragma unroll
        for (int n = 0; n < VPT; ++n) {
            const int c = 8 * (threadIdx.x + n * blockDim.x);
            if (c >= a.d) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) dn[n].v[e] = ry * fmaf(-y[n].v[e], m, dn[n].v[e]);
            store_act8((XT*)g.dy, base + c, dn[n]);
        }
    }
    if (!g.d_post && !g.d_pre) return;
    float* part = g.part + (size_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int n = 0; n < VPT; ++n) {
        const int c = 8 * (threadIdx.x + n * blockDim.x);
        if (c >= a.d) continue;
        if (g.d_post) store_act8(part, (size_t)c, acc_post[n]);
        if (g.d_pre) store_act8(part, (size_t)a.d + c, acc_pre[n]);
    }
}

// d_post and d_pre from the groups' sums: a workgroup adds 64 columns (four per thread), sixteen
// threads each a sixteenth of the groups, and then those sixteen sums, in order
__global__ __launch_bounds__(256) void k_norm_grad_sums(const float* __restrict__ part, int groups, int d,
                                                        float* __restrict__ d_post, float* __restrict__ d_pre) {
    __shared__ float4 s_sum[16][16];
    const int col = (threadIdx.x & 15) * 4 + blockIdx.x * 64;         // of the 2 d columns; d % 64 = 0
    const int q = threadIdx.x >> 4;
    float* out = blockIdx.x * 64 < (unsigned)d ? d_post : d_pre;
    if (!out) return;                                                  // uniform
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = q; b < groups; b += 16) {
        const float4 v = *(const float4*)(part + (size_t)b * 2 * d + col);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    s_sum[q][threadIdx.x & 15] = s;
    __syncthreads();
    if (q) return;
    for (int i = 1; i < 16; ++i) {
        const float4 v = s_sum[i][threadIdx.x];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    *(float4*)(out + (col < d ? col : col - d)) = s;
}

template <typename XT>
static void norm_backward_launch(const NormArgs& a, const NormGradArgs& g, int vpt, int threads, hipStream_t st) {
    const dim3 grid(norm_grad_groups(a.T));
    if (vpt == 1) MOE_LAUNCH((k_block_norm_backward<XT, 1>), grid, dim3(threads), 0, st, a, g);
    else MOE_LAUNCH((k_block_norm_backward<XT, 2>), grid, dim3(threads), 0, st, a, g);
}

hipError_t launch_block_norm_backward(const moe_shape* s, const NormArgs& a, const NormGradArgs& g, hipStream_t st) {
    trace("block_norm_backward", 0, st);
    int vpt;
    const int threads = norm_threads(a.d, &vpt);
    if (a.T > 0) {
        if (s->act_dtype == MOE_DT_BF16) norm_backward_launch<uint16_t>(a, g, vpt, threads, st);
        else norm_backward_launch<float>(a, g, vpt, threads, st);
    }
    if (g.d_post || g.d_pre)
        MOE_LAUNCH(k_norm_grad_sums, dim3(2 * a.d / 64), dim3(256), 0, st, (const float*)g.part, norm_grad_groups(a.T),
                   a.d, g.d_post, g.d_pre);
    trace("block_norm_backward", 1, st);
    return hipGetLastError();
}

}  // namespace moe
