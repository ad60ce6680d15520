// Dense products beside the experts, on the bf16 and the scaled FP8 matrix cores:
//
//   out[i][j] = sum_k P[i][k] Q[j][k]  and an epilogue (bias, activation, residual; or gate and up projection
//   multiplied), which serves the forward products (P the tokens, Q the weight), the input's gradient (Q the weight
//   stored k-major) and the weight's gradient (both stored k-major: k runs over the tokens).
//
// fp32 operands are split into three bf16 planes first (8 + 8 + 8 bits of mantissa), and six products of planes
// are summed in fp32; the three left out are below 2^-24 of the whole.
//
// A tile of P and Q advances by 128 bytes of k a step through a ring in LDS, filled by direct loads.  The matrix
// instruction's rows are Q's, so that a lane ends with 16 consecutive columns of one output row: row i of
// fragment f is column 16 (i / 4) + 4 f + i % 4 of the wave's 64.
#include "dense.h"

namespace moe {

typedef __bf16 pr_bf16x8 __attribute__((ext_vector_type(8)));
typedef float pr_f32x4 __attribute__((ext_vector_type(4)));
typedef int pr_i32x8 __attribute__((ext_vector_type(8)));
typedef short pr_i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t* pr_lds_t;

constexpr int kStepBytes = 128;              // of a row and step: 64 bf16, 128 codes
constexpr uint32_t kNowhere = 0x80000000u;   // past every descriptor's end: a load from there brings zeros

// planes of the six products of fp32 operands
constexpr uint32_t kPlaneP = 0x021100u, kPlaneQ = 0x200110u;   // (0,0) (0,1) (1,1) (1,0) (2,0) (0,2), four bits each

// one wave's 16 bytes per lane, lane l's to lds + 16 l
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t off, uint8_t* lds) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 0x7fffffff, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (dma_dst_t)lds, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void load_lds4(const uint8_t* base, uint32_t off, uint8_t* lds) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 0x7fffffff, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (dma_dst_t)lds, 4, off, 0, 0, 0);
}

// Place of a row's 16-byte chunk in LDS: chunk ^ key(row).  The sixteen rows that a fragment reads at once are
// 0 .. 15 of P and 16 a + b (a, b < 4) of Q; two rows fill the 64 banks, so eight keys are needed.
template <bool Q>
__device__ __forceinline__ int row_key(int r) {
    return Q ? ((r >> 1) & 1) | ((r >> 3) & 6) : (r >> 1) & 7;
}
// the same of a k-major tile: a read takes four rows k of 32 bytes (P), or of four 8-byte pieces 32 bytes apart (Q)
template <bool Q>
__device__ __forceinline__ int kmajor_key(int k) {
    return Q ? (k & 1) | ((k << 2) & 8) : ((k & 3) << 1) | (k & 8);
}

// One operand's tile of B rows: the lane's share of a step's loads.
template <bool Q, bool KMAJOR, int B, int N, bool GATED>
struct TileLoads {
    uint32_t off[N];         // from the step's first byte; kNowhere outside the matrix
    const uint8_t* base;
    size_t step, upper;      // bytes from one step to the next; from the gate's rows to the up projection's
    int left;                // bytes of a row (k-major: rows) from the step on

    // first: the tile's first row (gated: h column); rows: rows of the matrix; ld: its rows' bytes; K: length of the sum
    __device__ __forceinline__ void init(const uint8_t* p, int first, int rows, int ld, int K, int esize, int wave, int lane) {
        if constexpr (KMAJOR) {
            constexpr int C = B / 8;                        // chunks of a k
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int unit = (wave * N + n) * 64 + lane, k = unit / C;
                const int c = (unit % C) ^ kmajor_key<Q>(k);
                off[n] = first + c * 8 < rows ? (uint32_t)(k * ld + c * 16) : kNowhere;
            }
            base = p + (size_t)first * 2;
            step = (size_t)ld * 64;
            left = K;
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int r = (wave * N + n) * 8 + (lane >> 3), c = (lane & 7) ^ row_key<Q>(r);
                // gated: rows 16 q + 4 f + e of each 64 are columns 8 q + 4 (f % 2) + e of 32, f / 2 the half
                const int row = GATED ? (r & ~63) / 2 + ((r >> 4) & 3) * 8 + (r & 7) : r;
                off[n] = first + row < rows ? (uint32_t)(row * ld + c * 16) : kNowhere;
            }
            base = p + (size_t)first * ld;
            step = kStepBytes;
            left = K * esize;
            upper = (size_t)rows * ld;
        }
    }
    // step s of plane `plane` bytes on
    __device__ __forceinline__ void load(int s, size_t plane, uint8_t* lds, int wave, int lane) const {
        const uint8_t* b = base + (size_t)s * step + plane;
        const int here = left - s * (KMAJOR ? 64 : kStepBytes);
        const bool whole = here >= (KMAJOR ? 64 : kStepBytes);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint32_t o = off[n];
            if (!whole) {
                int at;
                if constexpr (KMAJOR) at = ((wave * N + n) * 64 + lane) / (B / 8);
                else at = ((lane & 7) ^ row_key<Q>((wave * N + n) * 8 + (lane >> 3))) * 16;
                if (at >= here) o = kNowhere;
            }
            // gated: eight rows are all the gate's (even n) or all the up projection's
            load_lds16(GATED && (n & 1) ? b + upper : b, o, lds + (wave * N + n) * 1024);
        }
    }
};

// fragment f (P: rows 16 f .. of the wave's; Q: see above) of 32 k from 32 h on
template <bool Q, bool KMAJOR, int B>
__device__ __forceinline__ pr_bf16x8 fragment(const uint8_t* tile, int first, int f, int h, int lane) {
    const int i = lane & 15, g = lane >> 4;
    pr_bf16x8 r;
    if constexpr (KMAJOR) {
        const int k = 32 * h + 8 * g + (i >> 2);
        const int m = first + (Q ? (i & 3) * 16 + f * 4 : f * 16 + (i & 3) * 4);
        pr_i16x4 v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int kk = k + 4 * e;
            const uint8_t* p = tile + kk * (2 * B) + (((m >> 3) ^ kmajor_key<Q>(kk)) << 4) + (m & 4) * 2;
            v[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) pr_i16x4*)p);
        }
        __builtin_memcpy(&r, v, 16);
    } else {
        const int row = first + (Q ? (i >> 2) * 16 + f * 4 + (i & 3) : f * 16 + i);
        r = *(const pr_bf16x8*)(tile + row * kStepBytes + (((4 * h + g) ^ row_key<Q>(row)) << 4));
    }
    return r;
}
// of 128 codes: lane group g holds k 16 g .. and 64 + 16 g ..
template <bool Q>
__device__ __forceinline__ pr_i32x8 fragment8(const uint8_t* tile, int first, int f, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const int row = first + (Q ? (i >> 2) * 16 + f * 4 + (i & 3) : f * 16 + i);
    const uint4 a = *(const uint4*)(tile + row * kStepBytes + ((g ^ row_key<Q>(row)) << 4));
    const uint4 b = *(const uint4*)(tile + row * kStepBytes + (((4 + g) ^ row_key<Q>(row)) << 4));
    return pr_i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Tile of BI rows and 64 WJ columns; WI x WJ waves, each BI / WI rows by 64 columns.  ST stages.
template <bool MX8, bool PK, bool QK, int BI, int WI, int WJ, int ST, bool GATED>
__global__ __launch_bounds__(64 * WI * WJ) void k_product(ProductArgs a) {
    constexpr int W = WI * WJ, BJ = 64 * WJ, FI = BI / WI / 16;
    constexpr int NP = BI / 8 / W, NQ = BJ / 8 / W;
    constexpr int PB = BI * kStepBytes, QB = BJ * kStepBytes, SB = MX8 ? W * 256 : 0, STG = PB + QB + SB;
    static_assert(!GATED || NQ % 2 == 0, "even loads are the gate's");
    static_assert(!MX8 || W * 64 >= BI + BJ, "one load brings a step's scales");
    __shared__ __align__(1024) uint8_t ring[ST * STG];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int JH = GATED ? a.J / 2 : a.J, BH = GATED ? BJ / 2 : BJ;
    const int tj = (JH + BH - 1) / BH;
    const int tile = blockIdx.x;
    const int i0 = tile / tj * BI, j0 = tile % tj * BH;
    TileLoads<false, PK, BI, NP, false> lp;
    TileLoads<true, QK, BJ, NQ, GATED> lq;
    lp.init(a.p, i0, a.I, a.p_ld, a.K, MX8 ? 1 : 2, wave, lane);
    lq.init(a.q, j0, JH, a.q_ld, a.K, MX8 ? 1 : 2, wave, lane);
    uint32_t soff = kNowhere;
    const uint8_t* sbase = a.p_scales;
    if constexpr (MX8) {
        const int ld = a.K / 32, r = wave * 64 + lane;
        if (wave * 64 < BI) {
            if (i0 + r < a.I) soff = (uint32_t)(r * ld);
            sbase = a.p_scales + (size_t)i0 * ld;
        } else {
            const int w = r - BI;
            const int row = GATED ? (w & ~63) / 2 + ((w >> 4) & 3) * 8 + (w & 7) : w;
            if (w < BJ && j0 + row < JH) soff = (uint32_t)((row + (GATED && (w & 8) ? JH : 0)) * ld);
            sbase = a.q_scales + (size_t)j0 * ld;
        }
    }
    const int ksteps = (a.K + (MX8 ? 127 : 63)) / (MX8 ? 128 : 64);
    const int total = ksteps * a.pairs;
    const int s0 = (int)((long long)blockIdx.y * total / a.splits), s1 = (int)((long long)(blockIdx.y + 1) * total / a.splits);
    auto load = [&](int s) {
        uint8_t* st = ring + (s - s0) % ST * STG;
        int k = s;
        size_t pp = 0, qp = 0;
        if (a.pairs > 1) {
            const int pair = s % 6;
            k = s / 6;
            pp = ((kPlaneP >> (4 * pair)) & 15) * a.p_plane;
            qp = ((kPlaneQ >> (4 * pair)) & 15) * a.q_plane;
        }
        lp.load(k, pp, st, wave, lane);
        lq.load(k, qp, st + PB, wave, lane);
        if constexpr (MX8) load_lds4(sbase + 4 * (size_t)k, soff, st + PB + QB + wave * 256);
    };
    constexpr int PER = NP + NQ + (MX8 ? 1 : 0);
    const int wi = wave / WJ * (BI / WI), wj = wave % WJ * 64;
    pr_f32x4 acc[FI][4];
#pragma unroll
    for (int f = 0; f < FI; ++f)
#pragma unroll
        for (int g = 0; g < 4; ++g) acc[f][g] = pr_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
        if (s0 + s < s1) load(s0 + s);
    for (int s = s0; s < s1; ++s) {
        if (s + ST - 2 < s1) wait_vm<(ST - 2) * PER>();
        else wait_vm<0>();
        ring_barrier();
        if (s + ST - 1 < s1) load(s + ST - 1);
        const uint8_t* st = ring + (s - s0) % ST * STG;
        if constexpr (MX8) {
            pr_i32x8 q[4];
            int qs[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                q[f] = fragment8<true>(st + PB, wj, f, lane);
                qs[f] = st[PB + QB + 4 * (BI + wj + ((lane & 15) >> 2) * 16 + f * 4 + (lane & 3)) + (lane >> 4)];
            }
#pragma unroll
            for (int fi = 0; fi < FI; ++fi) {
                const pr_i32x8 p = fragment8<false>(st, wi, fi, lane);
                const int ps = st[PB + QB + 4 * (wi + fi * 16 + (lane & 15)) + (lane >> 4)];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    acc[fi][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[f], p, acc[fi][f], 0, 0, 0, qs[f], 0, ps);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                pr_bf16x8 q[4], p[FI];
#pragma unroll
                for (int f = 0; f < 4; ++f) q[f] = fragment<true, QK, BJ>(st + PB, wj, f, h, lane);
#pragma unroll
                for (int fi = 0; fi < FI; ++fi) p[fi] = fragment<false, PK, BI>(st, wi, fi, h, lane);
#pragma unroll
                for (int fi = 0; fi < FI; ++fi)
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        acc[fi][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[f], p[fi], acc[fi][f], 0, 0, 0);
            }
        }
    }
    const int g = lane >> 4;
#pragma unroll
    for (int fi = 0; fi < FI; ++fi) {
#pragma unroll
        for (int f = 0; f < 4; ++f) mfma_results_here(acc[fi][f]);
        const int i = i0 + wi + fi * 16 + (lane & 15);
        f32x8 v[2];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e / 8].v[e % 8] = acc[fi][e / 4][e % 4];
        if constexpr (GATED) {
            const int n = j0 + wj / 2 + g * 8;
            const bool valid = i < a.I && n < JH;
            if (a.splits > 1) {
                if (valid) {
                    float* part = a.part + ((size_t)blockIdx.y * a.I + i) * a.J + n;
                    store_act8(part, 0, v[0]);
                    store_act8(part, (size_t)JH, v[1]);
                }
            } else {
                gated_out8(a, i, n, valid, v[0], v[1], [](float m) { return max_xor32(max_xor16(m)); });
            }
        } else {
            const int j = j0 + wj + g * 16;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (i >= a.I || j + 8 * c >= a.J) continue;
                if (a.splits > 1) store_act8(a.part, ((size_t)blockIdx.y * a.I + i) * a.J + j + 8 * c, v[c]);
                else product_out8(a, i, j + 8 * c, v[c]);
            }
        }
    }
}

// the parts' sums in order, then the epilogue; eight columns per thread (gated: of h)
template <bool GATED>
__global__ __launch_bounds__(256) void k_product_finish(ProductArgs a) {
    const int N = GATED ? a.J / 2 : a.J, per = (N + 7) / 8;
    const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x, all = (size_t)a.I * per;
    const bool valid = at < all;
    const int i = valid ? (int)(at / per) : 0, n = valid ? (int)(at % per) * 8 : 0;
    auto sum = [&](int j) {
        const size_t from = (size_t)i * a.J + j;
        f32x8 v = load_act8(a.part, from);
        for (int s = 1; s < a.splits; ++s) {
            const f32x8 w = load_act8(a.part, (size_t)s * a.I * a.J + from);
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] += w.v[e];
        }
        return v;
    };
    if constexpr (GATED) {
        // (with 8-bit outputs N is a multiple of 32, so a block's four lanes are a quad)
        gated_out8(a, i, n, valid, sum(n), sum(N + n), [](float m) { return quad_max(m); });
    } else {
        if (valid) product_out8(a, i, n, sum(n));
    }
}

constexpr size_t kPartBytes = (size_t)64 << 20;
constexpr int kMostSplits = 16;
size_t product_part_bytes(size_t I, size_t J) {
    const size_t all = kMostSplits * I * J * 4;
    return all < kPartBytes ? all : kPartBytes;
}

template <bool MX8, bool PK, bool QK, bool GATED>
static void product_launch(ProductArgs& a, hipStream_t st) {
    constexpr int BI = 128, WI = 2, WJ = 2;
    const int JH = GATED ? a.J / 2 : a.J, BH = GATED ? 32 * WJ : 64 * WJ;
    const int tiles = (a.I + BI - 1) / BI * ((JH + BH - 1) / BH);
    const int steps = (a.K + (MX8 ? 127 : 63)) / (MX8 ? 128 : 64) * a.pairs;
    int splits = 512 / tiles;
    if (splits > steps / 4) splits = steps / 4;
    if (splits > kMostSplits) splits = kMostSplits;
    while (splits > 1 && (size_t)splits * a.I * a.J * 4 > product_part_bytes(a.I, a.J)) --splits;
    a.splits = splits < 1 ? 1 : splits;
    MOE_LAUNCH((k_product<MX8, PK, QK, BI, WI, WJ, 2, GATED>), dim3(tiles, a.splits), dim3(64 * WI * WJ), 0, st, a);
}

hipError_t launch_product(ProductArgs a, bool mx8, bool p_kmajor, bool q_kmajor, bool gated, hipStream_t st) {
    trace("product", 0, st);
    if (mx8) {
        if (gated) product_launch<true, false, false, true>(a, st);
        else product_launch<true, false, false, false>(a, st);
    } else if (gated) {
        product_launch<false, false, false, true>(a, st);
    } else if (p_kmajor) {
        product_launch<false, true, true, false>(a, st);
    } else if (q_kmajor) {
        product_launch<false, false, true, false>(a, st);
    } else {
        product_launch<false, false, false, false>(a, st);
    }
    trace("product", 1, st);
    if (a.splits > 1) {
        const size_t n = (size_t)a.I * (((gated ? a.J / 2 : a.J) + 7) / 8);
        const dim3 grid((uint32_t)((n + 255) / 256));
        trace("product_finish", 0, st);
        if (gated) MOE_LAUNCH((k_product_finish<true>), grid, dim3(256), 0, st, a);
        else MOE_LAUNCH((k_product_finish<false>), grid, dim3(256), 0, st, a);
        trace("product_finish", 1, st);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// three bf16 planes of fp32 values: each the nearest bf16 to what the planes before it leave.  A value whose
// nearest bf16 would be infinite is cut instead; an infinity or a NaN is its own first plane, the others zero.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void planes8(const f32x8& v, uint4 (&out)[3]) {
    f32x8 rest = v;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float r = rest.v[e];
            uint32_t b = f32_to_bf16_bits(r);
            const bool finite = __builtin_isfinite(r);
            if (finite && (b & 0x7fffu) == 0x7f80u) b = __float_as_uint(r) >> 16;
            w[e] = b;
            rest.v[e] = finite ? r - bf16_bits_to_f32((uint16_t)b) : 0.0f;
        }
        out[p] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}
__device__ __forceinline__ void store_planes8(uint16_t* planes, size_t plane, size_t i, const f32x8& v) {
    uint4 w[3];
    planes8(v, w);
#pragma unroll
    for (int p = 0; p < 3; ++p) *(uint4*)(planes + p * plane + i) = w[p];
}

__global__ __launch_bounds__(256) void k_planes(const float* __restrict__ x, size_t n, uint16_t* __restrict__ planes) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i < n) store_planes8(planes, n, i, load_act8(x, i));
}

hipError_t launch_planes(const float* x, size_t n, uint16_t* planes, hipStream_t st) {
    trace("planes", 0, st);
    MOE_LAUNCH(k_planes, dim3((uint32_t)((n / 8 + 255) / 256)), dim3(256), 0, st, x, n, planes);
    trace("planes", 1, st);
    return hipGetLastError();
}

// A scale byte b stands for 2^(b - 127); codes of blocks under 2^-117 that pass bf16's smallest number are rounded.
__global__ __launch_bounds__(256) void k_unpack(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, size_t n,
                                                uint16_t* __restrict__ values) {
    const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    const uint2 c = *(const uint2*)(codes + i);
    const int b = scales[i / 32];
    const float sc = b == 255 ? __builtin_nanf("") : ldexpf(1.0f, b - 127);
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t w = e ? c.y : c.x;
        const v2f_t lo = fp8x2_decode<false>(w, 1.0f), hi = fp8x2_decode<true>(w, 1.0f);
        v.v[4 * e] = lo[0] * sc;
        v.v[4 * e + 1] = lo[1] * sc;
        v.v[4 * e + 2] = hi[0] * sc;
        v.v[4 * e + 3] = hi[1] * sc;
    }
    store_act8(values, i, v);
}

hipError_t launch_unpack(const uint8_t* codes, const uint8_t* scales, size_t n, uint16_t* values, hipStream_t st) {
    trace("unpack", 0, st);
    MOE_LAUNCH(k_unpack, dim3((uint32_t)((n / 8 + 255) / 256)), dim3(256), 0, st, codes, scales, n, values);
    trace("unpack", 1, st);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// gradient of the pre-activations, rounded for the products behind it, and its column sums in fp32 before that
// rounding (the bias's gradient: row chunks apart, then added in order).  A workgroup takes 256 columns, 32 threads
// of eight, and every eighth row of its chunk per thread row.
// ---------------------------------------------------------------------------------------------
template <typename XT, bool GATED>
__global__ __launch_bounds__(256) void k_pre_grad(PreGradArgs a) {
    __shared__ f32x8 part[8][32];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5, n = blockIdx.x * 256 + c * 8;
    const int t0 = (int)((long long)blockIdx.y * a.T / gridDim.y), t1 = (int)((long long)(blockIdx.y + 1) * a.T / gridDim.y);
    const int ld = GATED ? 2 * a.N : a.N;
    f32x8 sum = {};
    if (n < a.N) {
        for (int t = t0 + r; t < t1; t += 8) {
            const f32x8 dy = load_act8((const XT*)a.dy, (size_t)t * a.N + n);
            const size_t at = (size_t)t * ld + n;
            f32x8 d = dy, du;
            if constexpr (GATED) {
                const f32x8 g = load_act8((const XT*)a.pre, at), u = load_act8((const XT*)a.pre, at + a.N);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    d.v[e] = dy.v[e] * u.v[e] * slope(a.activation, g.v[e]);
                    du.v[e] = dy.v[e] * activate(a.activation, g.v[e]);
                }
            } else if (a.activation != MOE_ACT_NONE) {
                const f32x8 v = load_act8((const XT*)a.pre, at);
#pragma unroll
                for (int e = 0; e < 8; ++e) d.v[e] = dy.v[e] * slope(a.activation, v.v[e]);
            }
            if (a.d) {
                if constexpr (sizeof(XT) == 4) {
                    store_planes8(a.d, (size_t)a.T * ld, at, d);
                    if constexpr (GATED) store_planes8(a.d, (size_t)a.T * ld, at + a.N, du);
                } else {
                    store_act8(a.d, at, d);
                    if constexpr (GATED) store_act8(a.d, at + a.N, du);
                }
            }
            if constexpr (!GATED) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum.v[e] += d.v[e];
            }
        }
    }
    if (!a.bias_part) return;
    part[r][c] = sum;
    __syncthreads();
    if (r == 0 && n < a.N) {
        for (int k = 1; k < 8; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum.v[e] += part[k][c].v[e];
        store_act8(a.bias_part, (size_t)blockIdx.y * a.N + n, sum);
    }
}
__global__ __launch_bounds__(256) void k_bias_sums(PreGradArgs a, int chunks) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.N) return;
    float s = 0.0f;
    for (int c = 0; c < chunks; ++c) s += a.bias_part[(size_t)c * a.N + n];
    a.d_bias[n] = s;
}

hipError_t launch_pre_grad(const PreGradArgs& a, bool f32, hipStream_t st) {
    int chunks = (a.T + 31) / 32;
    if (chunks > kBiasChunks) chunks = kBiasChunks;
    const dim3 grid((a.N + 255) / 256, chunks);
    trace("pre_grad", 0, st);
    if (a.gated) {
        if (f32) MOE_LAUNCH((k_pre_grad<float, true>), grid, dim3(256), 0, st, a);
        else MOE_LAUNCH((k_pre_grad<uint16_t, true>), grid, dim3(256), 0, st, a);
    } else {
        if (f32) MOE_LAUNCH((k_pre_grad<float, false>), grid, dim3(256), 0, st, a);
        else MOE_LAUNCH((k_pre_grad<uint16_t, false>), grid, dim3(256), 0, st, a);
    }
    trace("pre_grad", 1, st);
    if (a.bias_part) {
        trace("bias_sums", 0, st);
        MOE_LAUNCH(k_bias_sums, dim3((a.N + 255) / 256), dim3(256), 0, st, a, chunks);
        trace("bias_sums", 1, st);
    }
    return hipGetLastError();
}

}  // namespace moe
