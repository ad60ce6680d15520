// Tokens laid out by expert (dispatch), and the gradients of the dispatch and of the weighted combine.
#include "block_ops.h"

namespace moe {

// Workgroups of a launch over `jobs` of them: a launch has fewer than 2^32 threads per dimension, so
// the kernels step through their jobs by the grid.
static dim3 job_grid(size_t jobs) { return dim3((unsigned)(jobs < (1u << 22) ? jobs : (1u << 22))); }

// Jobs up to which four waves share one: a wave alone on its SIMD steps through a row a round trip at a time.
constexpr size_t kFewJobs = 512;

// a pick's row, or -1: positions outside [0, P) (a dropped pick's is -1) have none
__device__ __forceinline__ int pick_row(const int32_t* __restrict__ pick_pos, size_t p, int P) {
    const int pos = pick_pos[p];
    return (unsigned)pos < (unsigned)P ? pos : -1;
}

// workgroups of at most `most` threads over a row of `units` 8-column or 16-byte units, and their threads:
// whole waves, spread evenly
static int row_chunks(size_t units, int most) { return (int)((units + most - 1) / most); }
static int row_threads(size_t units, int most) {
    const int chunks = row_chunks(units, most);
    return (int)(((units + chunks - 1) / chunks + 63) / 64 * 64);
}

// xs[pick_pos[t,j]] = x[t]: one thread per 16 bytes of a token's row, which it reads once and stores for
// every pick (the other way round, a read per sorted row, would read x k times).  Bound by its stores:
// 4096 tokens, d 4096, 8 picks, bf16: 54 us, 302 MB at 5.6 TB/s, the rate of a large copy; one token 2.0 us.
template <bool NT>
__global__ __launch_bounds__(512) void k_dispatch(const uint8_t* __restrict__ x, int T, int k, size_t row_bytes,
                                                  int chunks, int shared, const int32_t* __restrict__ pick_pos,
                                                  uint8_t* __restrict__ xs) {
    const int P = T * k;
    for (size_t job = blockIdx.x; job < (size_t)T * chunks; job += gridDim.x) {
        const int t = (int)(job / chunks);
        const size_t c = (job % chunks * blockDim.x + threadIdx.x) * 16;
        if (c >= row_bytes) continue;
        const u32x4_t v = *(const u32x4_t*)(x + (size_t)t * row_bytes + c);
        for (int j = 0; j < k; ++j) {
            const int r = pick_row(pick_pos, (size_t)t * k + j, P);
            if (r >= 0) store16<NT>(xs + (size_t)r * row_bytes + c, v);
        }
        if (shared) store16<NT>(xs + ((size_t)P + t) * row_bytes + c, v);
    }
}

hipError_t launch_dispatch(const moe_shape* s, const void* x, int T, const int32_t* pick_pos, void* xs,
                           hipStream_t st) {
    trace("dispatch", 0, st);
    const size_t row = (size_t)s->d_model * (s->act_dtype == MOE_DT_BF16 ? 2 : 4);
    const int threads = row_threads(row / 16, 512), chunks = row_chunks(row / 16, 512);
    const dim3 grid = job_grid((size_t)T * chunks);
    if (row * T * (s->top_k + s->n_shared) >= kStreamBytes)
        MOE_LAUNCH(k_dispatch<true>, grid, dim3(threads), 0, st, (const uint8_t*)x, T, s->top_k, row, chunks, s->n_shared,
                   pick_pos, (uint8_t*)xs);
    else
        MOE_LAUNCH(k_dispatch<false>, grid, dim3(threads), 0, st, (const uint8_t*)x, T, s->top_k, row, chunks, s->n_shared,
                   pick_pos, (uint8_t*)xs);
    trace("dispatch", 1, st);
    return hipGetLastError();
}

// dx[t] = sum_j dxs[pick_pos[t,j]] (+ dxs[P + t]): one thread per 8 columns, added in rank order in fp32;
// read by token, so there are no atomics.  Bound by its loads, up to eight rows in flight; workgroups of two
// waves, because larger ones leave CUs uneven when there are few tokens (333 tokens, d 6144, fp32: 13 us,
// 384 threads 14).  4096 tokens, d 4096, 8 picks, bf16: 52 us, 302 MB at 5.8 TB/s.
template <typename XT, bool NT>
__global__ __launch_bounds__(128) void k_dispatch_backward(const XT* __restrict__ dxs, int T, int k, int d,
                                                           int chunks, int shared,
                                                           const int32_t* __restrict__ pick_pos,
                                                           XT* __restrict__ dx) {
    const int P = T * k;
    for (size_t job = blockIdx.x; job < (size_t)T * chunks; job += gridDim.x) {
        const int t = (int)(job / chunks);
        const int c = ((int)(job % chunks) * blockDim.x + threadIdx.x) * 8;
        if (c >= d) continue;
        f32x8 acc = {};
        for_picks<8>(pick_pos + (size_t)t * k, k, P, [&](auto n, const int (&row)[8], const bool (&has)[8], int) {
            constexpr int N = decltype(n)::value;
            Raw8<XT> v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) v[i].template load<NT>(dxs, (size_t)row[i] * d + c);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const f32x8 g = v[i].values();
#pragma unroll
                for (int e = 0; e < 8; ++e) acc.v[e] = has[i] ? acc.v[e] + g.v[e] : acc.v[e];
            }
        });
        if (shared) {
            const f32x8 v = load_act8<NT>(dxs, ((size_t)P + t) * d + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc.v[e] += v.v[e];
        }
        store_act8<NT>(dx, (size_t)t * d + c, acc);
    }
}

template <typename XT>
static void dispatch_backward_launch(const moe_shape* s, const XT* dxs, int T, const int32_t* pick_pos, XT* dx,
                                     hipStream_t st) {
    const int d = s->d_model, threads = row_threads(d / 8, 128), chunks = row_chunks(d / 8, 128);
    const dim3 grid = job_grid((size_t)T * chunks);
    if (sizeof(XT) * d * T * (s->top_k + s->n_shared) >= kStreamBytes)
        MOE_LAUNCH((k_dispatch_backward<XT, true>), grid, dim3(threads), 0, st, dxs, T, s->top_k, d, chunks, s->n_shared,
                   pick_pos, dx);
    else
        MOE_LAUNCH((k_dispatch_backward<XT, false>), grid, dim3(threads), 0, st, dxs, T, s->top_k, d, chunks, s->n_shared,
                   pick_pos, dx);
}

hipError_t launch_dispatch_backward(const moe_shape* s, const void* dxs, int T, const int32_t* pick_pos, void* dx,
                                    hipStream_t st) {
    trace("dispatch_backward", 0, st);
    if (s->act_dtype == MOE_DT_BF16)
        dispatch_backward_launch(s, (const uint16_t*)dxs, T, pick_pos, (uint16_t*)dx, st);
    else
        dispatch_backward_launch(s, (const float*)dxs, T, pick_pos, (float*)dx, st);
    trace("dispatch_backward", 1, st);
    return hipGetLastError();
}

// W waves (1, or 4 when there are few picks) per (token, pick): d_o[pos] = s w dy[t] and
// d_w = s <dy[t], o[pos]>, the products summed per lane in fp32 and over lanes and waves in a fixed order.
// With a shared expert each token has one job more, which copies dy[t] to row P + t.  d_o may be o: a lane
// reads its values of o before it writes them.  Bound by HBM: o read and d_o written once, 4096 tokens,
// d 4096, 8 picks: 220 us, 1.14 GB at 5.2 TB/s (dy comes twice, its eight picks lying in two workgroups;
// one of eight waves took as long, and requesting the next loads before the stores gained 3% there and lost
// 6% on short rows).
template <typename XT, int W, bool NT>
__global__ __launch_bounds__(256) void k_combine_backward(const XT* __restrict__ dy, const float* o,
                                                          const float* __restrict__ w,
                                                          const int32_t* __restrict__ pick_pos, int T, int k, int d,
                                                          int shared, float scaling, float* d_o,
                                                          float* __restrict__ d_w) {
    __shared__ float s_dot[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kk = k + shared, P = T * k;
    const size_t jobs = (size_t)T * kk;
    for (size_t job = W == 1 ? (size_t)blockIdx.x * 4 + wave : blockIdx.x; job < jobs;
         job += W == 1 ? (size_t)gridDim.x * 4 : gridDim.x) {
        const int t = (int)(job / kk), j = (int)(job % kk);
        const bool routed = j < k;
        const size_t p = (size_t)t * k + j;
        const int row = routed ? pick_row(pick_pos, p, P) : P + t;
        if (row < 0) {
            if (d_w && lane == 0 && (W == 1 || wave == 0)) d_w[p] = 0.0f;
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
        for (int c0 = (W == 1 ? lane : (int)threadIdx.x) * 4; c0 < d; c0 += 1024 * W) {
            float4 v[4];
            u32x4_t ov[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = load_act4(g, c0 + 256 * W * u < d ? c0 + 256 * W * u : d - 4);
            if (dot) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    ov[u] = load16<NT>(orow + (c0 + 256 * W * u < d ? c0 + 256 * W * u : d - 4));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (c0 + 256 * W * u >= d) continue;
                    acc.x = fmaf(v[u].x, __uint_as_float(ov[u][0]), acc.x);
                    acc.y = fmaf(v[u].y, __uint_as_float(ov[u][1]), acc.y);
                    acc.z = fmaf(v[u].z, __uint_as_float(ov[u][2]), acc.z);
                    acc.w = fmaf(v[u].w, __uint_as_float(ov[u][3]), acc.w);
                }
            }
            if (d_o) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (c0 + 256 * W * u < d)
                        store16<NT>(drow + c0 + 256 * W * u,
                                    u32x4_t{__float_as_uint(f * v[u].x), __float_as_uint(f * v[u].y),
                                            __float_as_uint(f * v[u].z), __float_as_uint(f * v[u].w)});
            }
        }
        if (!dot) continue;                                    // (the same for the whole job)
        float sum = wave_sum_f32((acc.x + acc.y) + (acc.z + acc.w));
        if constexpr (W > 1) {
            if (lane == 0) s_dot[wave] = sum;
            __syncthreads();
            sum = (s_dot[0] + s_dot[1]) + (s_dot[2] + s_dot[3]);
            __syncthreads();                                   // the next job overwrites the sums
        }
        if (lane == 0 && (W == 1 || wave == 0)) d_w[p] = scaling * sum;
    }
}

template <typename XT>
static void combine_backward_launch(const moe_shape* s, const XT* dy, const float* o, const float* w,
                                    const int32_t* pick_pos, int T, float* d_o, float* d_w, hipStream_t st) {
    const size_t jobs = (size_t)T * (s->top_k + s->n_shared);
    if (jobs <= kFewJobs)
        MOE_LAUNCH((k_combine_backward<XT, 4, false>), dim3((unsigned)jobs), dim3(256), 0, st, dy, o, w, pick_pos, T,
                   s->top_k, s->d_model, s->n_shared, s->routed_scaling, d_o, d_w);
    else if (jobs * s->d_model * 4 >= kStreamBytes)
        MOE_LAUNCH((k_combine_backward<XT, 1, true>), job_grid((jobs + 3) / 4), dim3(256), 0, st, dy, o, w, pick_pos, T,
                   s->top_k, s->d_model, s->n_shared, s->routed_scaling, d_o, d_w);
    else
        MOE_LAUNCH((k_combine_backward<XT, 1, false>), job_grid((jobs + 3) / 4), dim3(256), 0, st, dy, o, w, pick_pos, T,
                   s->top_k, s->d_model, s->n_shared, s->routed_scaling, d_o, d_w);
}

hipError_t launch_combine_backward(const moe_shape* s, const void* dy, const float* o, const float* w,
                                   const int32_t* pick_pos, int T, float* d_o, float* d_w, hipStream_t st) {
    trace("combine_backward", 0, st);
    if (s->act_dtype == MOE_DT_BF16)
        combine_backward_launch(s, (const uint16_t*)dy, o, w, pick_pos, T, d_o, d_w, st);
    else
        combine_backward_launch(s, (const float*)dy, o, w, pick_pos, T, d_o, d_w, st);
    trace("combine_backward", 1, st);
    return hipGetLastError();
}

}  // namespace moe
