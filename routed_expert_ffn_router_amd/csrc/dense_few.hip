// Dense products of up to 64 tokens: the weight is read once, and HBM bounds the call.
//
// A workgroup takes 16 F rows of the weight and all tokens (16 C of them), tile after tile, and its waves share out k.
// Each wave has a ring of its own in LDS, filled by direct loads in row order (in the matrix instructions' operand layout
// a lane quad would lie on four rows, at four times the cost in the vector L1); the ring runs on from one tile to the
// next, so that only the sums at a tile's end are waited for.  The waves' sums are added through LDS in a fixed order, and
// go through the epilogue eight columns at a time.
//
// A step is 128 bytes of a row.  bf16: chunks g and 4 + g of 16 bytes for lane group g, in two products.  fp32 values enter
// fp32 matrix products as they are: the same chunks, four values each, in eight products.  MXFP8: block g, whose
// codes times their scale are exact in bf16 (but for the ends of its range), in four products.
//
// bf16, 4096 x 4096, one token 8.1 us (33.6 MB at 4.1 TB/s; 2 us of it are the launch and the first step's way), gated 8192 x
// 4096 26.9 us (134 MB at 5.0 TB/s); fp32 4096 x 4096 12.8 us (5.2 TB/s); 64 tokens, bf16, 4096 x 4096 10.5 us; MXFP8,
// 4096 x 4096, one token 7.6 us (17.3 MB).
#include "dense_tile.h"

namespace moe {

// eight codes times their block's scale (the E8M0 byte as the exponent of a float), in bf16: exact from 2^-133 to 2^128
__device__ __forceinline__ pr_bf16x8 few_mx8(uint32_t a, uint32_t b, float scale) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    const v2 w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false), x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true),
             y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false), z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
    return pr_bf16x8{w[0], w[1], x[0], x[1], y[0], y[1], z[0], z[1]};
}

// gated: of a tile's 16 F rows the first half are the gate's of 8 F columns of h, the others the up projection's
template <int FMT, int F, int C, int W, int ST, bool GATED>
__global__ __launch_bounds__(64 * W) void k_product_few(ProductArgs a, int tiles) {
    constexpr bool MX8 = FMT == kMx8;
    constexpr int ES = kSize<FMT>, COLS = GATED ? 8 * F : 16 * F, SL = MX8 ? 2 : 0;
    constexpr int QB = 2048 * F, PB = 2048 * C, STG = QB + PB + 256 * SL, PER = 2 * F + 2 * C + SL;
    static_assert((ST - 1) * PER < 64, "vmcnt holds 6 bits");
    static_assert(W * (ST * STG + F * C * 1024) <= 160 << 10, "LDS");
    __shared__ __align__(1024) uint8_t rings[W * (ST * STG + F * C * 1024)];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int N = GATED ? a.J / 2 : a.J, ld = a.K * ES, NS = (ld + kStepBytes - 1) / kStepBytes;
    const int s0 = wave * NS / W, s1 = (wave + 1) * NS / W;
    uint8_t* mine = rings + wave * ST * STG;
    // the lane's part of every load: row r8 of eight, its chunk exchanged by the row
    const int r8 = lane >> 3, at = ((lane & 7) ^ row_key(r8)) * 16;
    uint32_t qoff[2 * F], poff[2 * C], qsoff = kNowhere, psoff = kNowhere;
    const uint8_t* qbase;
    int lt = blockIdx.x, ls = s0;                            // the next load's tile and step
    auto new_tile = [&] {
        const int n0 = lt * COLS;
        qbase = a.q + (size_t)(lt < tiles ? n0 : 0) * ld;
#pragma unroll
        for (int u = 0; u < 2 * F; ++u) {
            const int r = (GATED ? u % F : u) * 8 + r8;
            qoff[u] = lt < tiles && n0 + r < N ? (uint32_t)(r * ld + at) : kNowhere;
        }
        if constexpr (MX8) {                                 // a row's four scale bytes, a row per lane
            const int q = GATED ? lane % (8 * F) : lane;
            qsoff = lt < tiles && lane < 16 * F && n0 + q < N
                        ? (uint32_t)((size_t)(n0 + q + (GATED && lane >= 8 * F ? N : 0)) * scale_row(a.K)) : kNowhere;
        }
    };
#pragma unroll
    for (int u = 0; u < 2 * C; ++u) poff[u] = u * 8 + r8 < a.I ? (uint32_t)((u * 8 + r8) * ld + at) : kNowhere;
    if constexpr (MX8) psoff = lane < 16 * C && lane < a.I ? (uint32_t)(lane * scale_row(a.K)) : kNowhere;
    new_tile();
    auto load = [&](uint8_t* st) {
        const size_t k = (size_t)ls * kStepBytes;
        const int here = ld - ls * kStepBytes;
        const bool more = lt < tiles;
#pragma unroll
        for (int u = 0; u < 2 * F; ++u)
            load_lds16(qbase + k + (GATED && u >= F ? (size_t)N * ld : 0), at < here ? qoff[u] : kNowhere, st + u * 1024);
#pragma unroll
        for (int u = 0; u < 2 * C; ++u) load_lds16(a.p + k, more && at < here ? poff[u] : kNowhere, st + QB + u * 1024);
        if constexpr (MX8) {
            load_lds4(a.q_scales + k / 32, qsoff, st + QB + PB);
            load_lds4(a.p_scales + k / 32, more ? psoff : kNowhere, st + QB + PB + 256);
        }
        if (++ls == s1) {
            ls = s0;
            lt += gridDim.x;
            new_tile();
        }
    };
    pr_f32x4* const part = (pr_f32x4*)(rings + W * ST * STG);
    if (s1 > s0) {
#pragma unroll
        for (int t = 0; t < ST; ++t) load(mine + t * STG);
    }
    int slot = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        pr_f32x4 acc[F][C];
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int c = 0; c < C; ++c) acc[f][c] = pr_f32x4{0.f, 0.f, 0.f, 0.f};
        for (int s = s0; s < s1; ++s) {
            uint8_t* st = mine + slot * STG;
            slot = slot + 1 == ST ? 0 : slot + 1;
            wait_vm<(ST - 1) * PER>();
            asm volatile("" ::: "memory");
            // a lane's two chunks of a row, and its block's scale
            auto chunk = [&](int base, int f, int h) {
                return *(const pr_u32x4*)(st + base + (f * 16 + i) * kStepBytes + (((MX8 ? 2 * g + h : 4 * h + g) ^ row_key(i)) << 4));
            };
            auto scale = [&](int base, int f) { return __uint_as_float((uint32_t)st[base + 4 * (f * 16 + i) + g] << 23); };
            pr_u32x4 q[F][2], p[C][2];
            float qs[F], ps[C];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int f = 0; f < F; ++f) q[f][h] = chunk(0, f, h);
#pragma unroll
                for (int c = 0; c < C; ++c) p[c][h] = chunk(QB, c, h);
            }
            if constexpr (MX8) {
#pragma unroll
                for (int f = 0; f < F; ++f) qs[f] = scale(QB + PB, f);
#pragma unroll
                for (int c = 0; c < C; ++c) ps[c] = scale(QB + PB + 256, c);
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0): the step is in registers, and its place free
            asm volatile("" ::: "memory");
            load(st);
            if constexpr (MX8) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    pr_bf16x8 x[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) x[c] = few_mx8(p[c][h / 2][h % 2 * 2], p[c][h / 2][h % 2 * 2 + 1], ps[c]);
#pragma unroll
                    for (int f = 0; f < F; ++f) {
                        const pr_bf16x8 w = few_mx8(q[f][h / 2][h % 2 * 2], q[f][h / 2][h % 2 * 2 + 1], qs[f]);
#pragma unroll
                        for (int c = 0; c < C; ++c) acc[f][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[c], acc[f][c], 0, 0, 0);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int f = 0; f < F; ++f)
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            if constexpr (FMT == kF32) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    acc[f][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(q[f][h][e]), __uint_as_float(p[c][h][e]),
                                                                                     acc[f][c], 0, 0, 0);
                            } else {
                                acc[f][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(pr_bf16x8, q[f][h]),
                                                                                    __builtin_bit_cast(pr_bf16x8, p[c][h]), acc[f][c], 0, 0, 0);
                            }
                        }
            }
        }
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                mfma_results_here(acc[f][c]);
                part[((wave * F + f) * C + c) * 64 + lane] = acc[f][c];
            }
        ring_barrier();
        // eight rows of the tile from `row` on for token t, the waves' sums in their order
        auto sum8 = [&](int t, int row) {
            const pr_f32x4* from = part + (row / 16 * C + t / 16) * 64 + t % 16 + row % 16 / 4 * 16;
            pr_f32x4 x = from[0], y = from[16];
#pragma unroll
            for (int w = 1; w < W; ++w) {
                x += from[w * F * C * 64];
                y += from[w * F * C * 64 + 16];
            }
            return f32x8{{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}};
        };
        with_activation(a.activation, [&](auto fn) {
            constexpr int FN = decltype(fn)::value;
            for (int x = threadIdx.x; x < 16 * C * COLS / 8; x += 64 * W) {
                const int t = x / (COLS / 8), c = x % (COLS / 8) * 8, n = tile * COLS + c;
                if constexpr (GATED) gated_out8<FN>(a, t, n, t < a.I && n < N, sum8(t, c), sum8(t, 8 * F + c));
                else if (t < a.I && n < N) product_out8<FN>(a, t, n, sum8(t, c));
            }
        });
        ring_barrier();                                      // the next tile's sums go to the same place
    }
    wait_vm<0>();                                            // no direct load outlives the workgroup
}

template <int FMT, int F, int C, int W, int ST, bool GATED>
static void few_launch_as(const ProductArgs& a, hipStream_t st) {
    const int N = GATED ? a.J / 2 : a.J, cols = GATED ? 8 * F : 16 * F, tiles = (N + cols - 1) / cols;
    MOE_LAUNCH((k_product_few<FMT, F, C, W, ST, GATED>), dim3(tiles < 256 ? tiles : 256), dim3(64 * W), 0, st, a, tiles);
}

template <int FMT, bool GATED>
static void few_launch(const ProductArgs& a, hipStream_t st) {
    if (GATED && a.out_scales) {                             // 32 columns of h in a tile: whole blocks
        if (a.I <= 16) few_launch_as<FMT, 4, 1, 4, 3, GATED>(a, st);
        else few_launch_as<FMT, 4, 2, 4, 2, GATED>(a, st);
    } else {
        if (a.I <= 16) few_launch_as<FMT, 1, 1, 8, 4, GATED>(a, st);
        else if (a.I <= 32) few_launch_as<FMT, 1, 2, 4, 5, GATED>(a, st);
        else few_launch_as<FMT, 1, 4, 4, 3, GATED>(a, st);
    }
}

hipError_t launch_product_few(const ProductArgs& a, int bytes, bool gated, hipStream_t st) {
    trace("product_few", 0, st);
    if (bytes == 2) {
        if (gated) few_launch<kBf16, true>(a, st);
        else few_launch<kBf16, false>(a, st);
    } else if (bytes == 4) {
        if (gated) few_launch<kF32, true>(a, st);
        else few_launch<kF32, false>(a, st);
    } else {
        if (gated) few_launch<kMx8, true>(a, st);
        else few_launch<kMx8, false>(a, st);
    }
    trace("product_few", 1, st);
    return hipGetLastError();
}

}  // namespace moe
