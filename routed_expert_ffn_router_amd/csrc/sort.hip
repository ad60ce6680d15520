// Tokens laid out by expert (dispatch), and the gradients of the dispatch and of the weighted combine.
#include "moe_internal.h"

namespace moe {

// Workgroups of a launch over `jobs` of them: a launch has fewer than 2^32 threads per dimension, so
// the kernels step through their jobs by the grid.
static dim3 job_grid(size_t jobs) { return dim3((unsigned)(jobs < (1u << 22) ? jobs : (1u << 22))); }

// a pick's row, or -1: positions outside [0, P) (a dropped pick's is -1) have none
__device__ __forceinline__ int pick_row(const int32_t* __restrict__ pick_pos, size_t p, int P) {
    const int pos = pick_pos[p];
    return (unsigned)pos < (unsigned)P ? pos : -1;
}

// xs[pick_pos[t,j]] = x[t]: one thread per 16 bytes of a token's row, which it reads once and stores
// for every pick.
__global__ __launch_bounds__(256) void k_dispatch(const uint8_t* __restrict__ x, int T, int k, size_t row_bytes,
                                                  int chunks, int shared, const int32_t* __restrict__ pick_pos,
                                                  uint8_t* __restrict__ xs) {
    const int P = T * k;
    for (size_t job = blockIdx.x; job < (size_t)T * chunks; job += gridDim.x) {
        const int t = (int)(job / chunks);
        const size_t c = (job % chunks * 256 + threadIdx.x) * 16;
        if (c >= row_bytes) continue;
        const uint4 v = *(const uint4*)(x + (size_t)t * row_bytes + c);
        for (int j = 0; j < k; ++j) {
            const int r = pick_row(pick_pos, (size_t)t * k + j, P);
            if (r >= 0) *(uint4*)(xs + (size_t)r * row_bytes + c) = v;
        }
        if (shared) *(uint4*)(xs + ((size_t)P + t) * row_bytes + c) = v;
    }
}

hipError_t launch_dispatch(const moe_shape* s, const void* x, int T, const int32_t* pick_pos, void* xs,
                           hipStream_t st) {
    trace("dispatch", 0, st);
    const size_t row = (size_t)s->d_model * (s->act_dtype == MOE_DT_BF16 ? 2 : 4);
    const int chunks = (int)((row + 4095) / 4096);
    MOE_LAUNCH(k_dispatch, job_grid((size_t)T * chunks), dim3(256), 0, st, (const uint8_t*)x, T, s->top_k, row, chunks,
               s->n_shared, pick_pos, (uint8_t*)xs);
    trace("dispatch", 1, st);
    return hipGetLastError();
}

// dx[t] = sum_j dxs[pick_pos[t,j]] (+ dxs[P + t]): one thread per 8 columns, eight picks' rows in
// flight at a time, added in rank order in fp32.  A pick without a row reads row 0 and adds nothing.
template <typename XT>
__global__ __launch_bounds__(256) void k_dispatch_backward(const XT* __restrict__ dxs, int T, int k, int d,
                                                           int chunks, int shared,
                                                           const int32_t* __restrict__ pick_pos,
                                                           XT* __restrict__ dx) {
    const int P = T * k;
    for (size_t job = blockIdx.x; job < (size_t)T * chunks; job += gridDim.x) {
        const int t = (int)(job / chunks);
        const int c = ((int)(job % chunks) * 256 + threadIdx.x) * 8;
        if (c >= d) continue;
        f32x8 acc = {};
        for (int j0 = 0; j0 < k; j0 += 8) {
            int row[8];
            f32x8 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) row[i] = j0 + i < k ? pick_row(pick_pos, (size_t)t * k + j0 + i, P) : -1;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = load_act8(dxs, (size_t)(row[i] >= 0 ? row[i] : 0) * d + c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc.v[e] = row[i] >= 0 ? acc.v[e] + v[i].v[e] : acc.v[e];
        }
        if (shared) {
            const f32x8 v = load_act8(dxs, ((size_t)P + t) * d + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc.v[e] += v.v[e];
        }
        store_act8(dx, (size_t)t * d + c, acc);
    }
}

hipError_t launch_dispatch_backward(const moe_shape* s, const void* dxs, int T, const int32_t* pick_pos, void* dx,
                                    hipStream_t st) {
    trace("dispatch_backward", 0, st);
    const int d = s->d_model, chunks = (d + 2047) / 2048;
    const dim3 grid = job_grid((size_t)T * chunks);
    if (s->act_dtype == MOE_DT_BF16)
        MOE_LAUNCH(k_dispatch_backward<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)dxs, T, s->top_k, d, chunks,
                   s->n_shared, pick_pos, (uint16_t*)dx);
    else
        MOE_LAUNCH(k_dispatch_backward<float>, grid, dim3(256), 0, st, (const float*)dxs, T, s->top_k, d, chunks,
                   s->n_shared, pick_pos, (float*)dx);
    trace("dispatch_backward", 1, st);
    return hipGetLastError();
}

// One wave per (token, pick): d_o[pos] = s w dy[t] and d_w = s <dy[t], o[pos]>, the products summed per
// lane in fp32 and over the lanes in a fixed order.  With a shared expert each token has one wave more,
// which copies dy[t] to row P + t.  d_o may be o: a lane reads its values of o before it writes them.
template <typename XT>
__global__ __launch_bounds__(256) void k_combine_backward(const XT* __restrict__ dy, const float* o,
                                                          const float* __restrict__ w,
                                                          const int32_t* __restrict__ pick_pos, int T, int k, int d,
                                                          int shared, float scaling, float* d_o,
                                                          float* __restrict__ d_w) {
    const int lane = threadIdx.x & 63;
    const int kk = k + shared, P = T * k;
    const size_t jobs = (size_t)T * kk;
    for (size_t job = (size_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); job < jobs;
         job += (size_t)gridDim.x * 4) {
        const int t = (int)(job / kk), j = (int)(job % kk);
        const bool routed = j < k;
        const size_t p = (size_t)t * k + j;
        const int row = routed ? pick_row(pick_pos, p, P) : P + t;
        if (row < 0) {
            if (d_w && lane == 0) d_w[p] = 0.0f;
            continue;
        }
        const bool dot = routed && d_w;
        const float f = routed ? (d_o ? scaling * w[p] : 0.0f) : 1.0f;
        const XT* g = dy + (size_t)t * d;
        const float* orow = dot ? o + (size_t)row * d : nullptr;
        float* drow = d_o ? d_o + (size_t)row * d : nullptr;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // four loads of each row in flight before any store; columns past the row read its last ones
        // and add nothing
        for (int c0 = lane * 4; c0 < d; c0 += 1024) {
            float4 v[4], ov[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = load_act4(g, c0 + 256 * u < d ? c0 + 256 * u : d - 4);
            if (dot) {
#pragma unroll
                for (int u = 0; u < 4; ++u) ov[u] = *(const float4*)(orow + (c0 + 256 * u < d ? c0 + 256 * u : d - 4));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (c0 + 256 * u >= d) continue;
                    acc.x = fmaf(v[u].x, ov[u].x, acc.x);
                    acc.y = fmaf(v[u].y, ov[u].y, acc.y);
                    acc.z = fmaf(v[u].z, ov[u].z, acc.z);
                    acc.w = fmaf(v[u].w, ov[u].w, acc.w);
                }
            }
            if (d_o) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (c0 + 256 * u < d)
                        *(float4*)(drow + c0 + 256 * u) = make_float4(f * v[u].x, f * v[u].y, f * v[u].z, f * v[u].w);
            }
        }
        if (dot) {
            const float sum = wave_sum_f32((acc.x + acc.y) + (acc.z + acc.w));
            if (lane == 0) d_w[p] = scaling * sum;
        }
    }
}

hipError_t launch_combine_backward(const moe_shape* s, const void* dy, const float* o, const float* w,
                                   const int32_t* pick_pos, int T, float* d_o, float* d_w, hipStream_t st) {
    trace("combine_backward", 0, st);
    const size_t jobs = (size_t)T * (s->top_k + s->n_shared);
    const dim3 grid = job_grid((jobs + 3) / 4);
    if (s->act_dtype == MOE_DT_BF16)
        MOE_LAUNCH(k_combine_backward<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)dy, o, w, pick_pos, T, s->top_k,
                   s->d_model, s->n_shared, s->routed_scaling, d_o, d_w);
    else
        MOE_LAUNCH(k_combine_backward<float>, grid, dim3(256), 0, st, (const float*)dy, o, w, pick_pos, T, s->top_k,
                   s->d_model, s->n_shared, s->routed_scaling, d_o, d_w);
    trace("combine_backward", 1, st);
    return hipGetLastError();
}

}  // namespace moe
