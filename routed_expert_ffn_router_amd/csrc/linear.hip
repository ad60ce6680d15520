// Matrix-vector products of up to 64 vectors with a dense weight in the experts' 4-bit formats.
//
//   y[t,n] = ts sum_k W[n,k] x[t,k] (+ bias[n]),   W[n,k] = E2M1 code x block scale.
//
// A code times its block scale is exact in bf16 (one bit of mantissa times a power of two, or times
// the four bits of an E4M3 scale), so the weights enter the bf16 matrix cores exactly; a bf16 x does
// too, and an fp32 x is the sum of three bf16 terms cut from it (8 + 8 + 8 bits; exact but for bits below
// 2^-133, bf16's smallest number), each one more MFMA column or MFMA into the same fp32 sums.  Subnormal terms
// and weights count in full.  A weight that passes the type (E8M0 bytes 253 and 254) is infinite, and NaN times a
// term that is zero.
//
// V_MFMA_F32_16X16X32_BF16: lane l supplies 8 consecutive K of weight row (A) or token (B) l % 16;
// any assignment of K to the lane groups works when both operands share it.  A step covers 128 K of a
// row: lane group g takes elements [32 g, 32 g + 32), 16 code bytes, and MFMA h of the step their
// elements [8 h, 8 h + 8).  C: lane l, register r is weight row 4 (l / 16) + r, token l % 16.
//
// Four kernels.  The bytes are the weights', read once, so HBM is the floor; what a straight kernel
// meets first is the vector L1, which serves a load one lane quad at a time: in the operand layout the
// lanes of a quad hold four different rows, so a load of 16 bytes per lane costs as much as four that
// are laid out along the rows, and a load of one scale byte per lane as much as one of 16 (taking the
// scale or the x loads out of k_linear each saved 20 of 84 us at 65536 x 6144, 16 tokens).
//   k_linear_ring    few rows, and few tokens: codes, scales and x go straight to LDS
//                    (global_load_lds) in row order, each wave into its own ring, so no wave waits for
//                    another before the sums;
//   k_linear_stream  many long rows: each wave keeps its K slice of x in registers for all the row tiles that
//                    its workgroup takes, so x is read once per CU;
//   k_linear_tile    many rows that are short, or too long for the registers, or with many tokens: the waves
//                    of a workgroup share x's step in LDS;
//   k_linear         6 to 16 fp32 tokens, or fewer with short rows, of many rows, straight from global memory
//                    to registers.
// Which one takes a call: lin_kernel_bf16 and lin_kernel_f32.
#include "block_ops.h"

namespace moe {

typedef __bf16 lin_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 lin_bf16x2 __attribute__((ext_vector_type(2)));
typedef float lin_f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t lin_u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ lin_bf16x8 lin_as_bf16x8(const uint4& v) {
    lin_bf16x8 r;
    __builtin_memcpy(&r, &v, 16);
    return r;
}

// 8 codes (one dword, element 2i in the low nibble of byte i) times their block scale, exact in bf16.
// MXFP4: the conversion unit's scale operand is a float read as a power of two (its exponent field, the
// E8M0 byte; 255 makes every value NaN).
__device__ __forceinline__ lin_bf16x8 lin_weights_mx(uint32_t codes, float scale) {
    const lin_bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0),
                     b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1),
                     c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2),
                     d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return lin_bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// NVFP4: codes at scale 1, times the E4M3 scale in fp32, rounded to bf16 (all exact)
__device__ __forceinline__ lin_bf16x8 lin_weights_nv(uint32_t codes, float scale) {
    const v2f_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0),
                b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
                c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2),
                d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
    return lin_bf16x8{(__bf16)(a[0] * scale), (__bf16)(a[1] * scale), (__bf16)(b[0] * scale), (__bf16)(b[1] * scale),
                      (__bf16)(c[0] * scale), (__bf16)(c[1] * scale), (__bf16)(d[0] * scale), (__bf16)(d[1] * scale)};
}

// The three bf16 terms of 8 fp32 values.  Cut, not rounded: the first term of a large value never becomes infinite;
// an infinite value is its own first term, and a NaN is made quiet, so that the cut leaves one (0x7f800001 is cut
// to infinity).
__device__ __forceinline__ void lin_f32_terms(const lin_u32x4& a, const lin_u32x4& b, lin_bf16x8 (&t)[3]) {
    uint32_t w[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float rest = __builtin_canonicalizef(__uint_as_float(e < 4 ? a[e] : b[e - 4]));
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t cut = __float_as_uint(rest) & 0xffff0000u;
            w[i][e] = cut;
            rest = (cut & 0x7fffffffu) == 0x7f800000u ? 0.0f : rest - __uint_as_float(cut);
        }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        t[i] = lin_as_bf16x8(make_uint4(w[i][0] >> 16 | w[i][1], w[i][2] >> 16 | w[i][3], w[i][4] >> 16 | w[i][5],
                                        w[i][6] >> 16 | w[i][7]));
}

// a step's scale byte(s) as factors of its first and last 16 elements
template <int WF>
__device__ __forceinline__ void lin_scales(uint32_t raw, float (&s)[2]) {
    if constexpr (WF == MOE_WF_MXFP4) {
        s[0] = s[1] = __uint_as_float(raw << 23);
    } else {
        const v2f_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(raw, 1.0f, false);
        s[0] = v[0];
        s[1] = v[1];
    }
}
template <int WF>
__device__ __forceinline__ lin_bf16x8 lin_weights(uint32_t codes, float scale) {
    if constexpr (WF == MOE_WF_MXFP4) return lin_weights_mx(codes, scale);
    else return lin_weights_nv(codes, scale);
}

struct LinArgs {
    int N, K, T;
    const uint8_t* q;
    const uint8_t* s;
    float ts;
    const void* x;
    const float* bias;
    void* y;
};

// rows row .. row + 3 of token t
template <typename XT>
__device__ __forceinline__ void lin_store(const LinArgs& a, int t, int row, const lin_f32x4& v) {
    float o[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = fmaf(v[r], a.ts, a.bias && row + r < a.N ? a.bias[row + r] : 0.0f);
    XT* y = (XT*)a.y + (size_t)t * a.N + row;
    if ((a.N & 3) == 0 && row < a.N) {           // row is a multiple of four: the four are there, and aligned
        if constexpr (sizeof(XT) == 4) *(float4*)y = make_float4(o[0], o[1], o[2], o[3]);
        else *(uint2*)y = make_uint2(f32_to_bf16_bits(o[0]) | (uint32_t)f32_to_bf16_bits(o[1]) << 16,
                                     f32_to_bf16_bits(o[2]) | (uint32_t)f32_to_bf16_bits(o[3]) << 16);
        return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (row + r < a.N) store_act(y, (size_t)r, o[r]);
}

// A workgroup of eight waves owns 64 rows and 16 fp32 tokens; its waves share out K, and their sums are added
// through LDS in wave order.  65536 x 6144 MXFP4, 16 tokens: 111 us, 16384 x 4096 22 (k_linear_tile 97 and 45,
// k_linear_ring 227 and 43); one or two rows' fragments per wave and deeper prefetch were slower.
template <int WF>
__global__ __launch_bounds__(512) void k_linear(LinArgs a) {
    constexpr int F = 4, W = 8;
    __shared__ lin_f32x4 part[W][F][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16 * F;
    const int NS = a.K / 128;
    const int s0 = wave * NS / W, n = (wave + 1) * NS / W - s0;
    constexpr int SB = WF == MOE_WF_MXFP4 ? 32 : 16;          // weights per scale
    const uint8_t* q[F];
    const uint8_t* s[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const int row = n0 + 16 * f + li < a.N ? n0 + 16 * f + li : a.N - 1;
        q[f] = a.q + (size_t)row * (a.K / 2) + (size_t)s0 * 64 + lg * 16;
        s[f] = a.s + (size_t)row * (a.K / SB) + (size_t)s0 * (128 / SB) + lg * (32 / SB);
    }
    const float* x = (const float*)a.x + (size_t)(li < a.T ? li : a.T - 1) * a.K + (size_t)s0 * 128 + lg * 32;
    lin_f32x4 acc[F];
#pragma unroll
    for (int f = 0; f < F; ++f) acc[f] = lin_f32x4{0.f, 0.f, 0.f, 0.f};

    uint4 code[F], xr[8];
    uint32_t sc[F];
    auto request = [&](int k) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            code[f] = gload16(q[f] + (size_t)k * 64);
            if constexpr (WF == MOE_WF_MXFP4) sc[f] = *(__attribute__((address_space(1))) const uint8_t*)(s[f] + (size_t)k * 4);
            else sc[f] = *(__attribute__((address_space(1))) const uint16_t*)(s[f] + (size_t)k * 8);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) xr[i] = gload16(x + (size_t)k * 128 + 4 * i);
    };
    auto multiply = [&]() {
        float s2[F][2];
#pragma unroll
        for (int f = 0; f < F; ++f) lin_scales<WF>(sc[f], s2[f]);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            lin_bf16x8 xt[3];
            lin_f32_terms(lin_u32x4{xr[2 * h].x, xr[2 * h].y, xr[2 * h].z, xr[2 * h].w},
                          lin_u32x4{xr[2 * h + 1].x, xr[2 * h + 1].y, xr[2 * h + 1].z, xr[2 * h + 1].w}, xt);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const uint32_t word = h == 0 ? code[f].x : h == 1 ? code[f].y : h == 2 ? code[f].z : code[f].w;
                const lin_bf16x8 w = lin_weights<WF>(word, s2[f][h / 2]);
#pragma unroll
                for (int i = 0; i < 3; ++i) acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xt[i], acc[f], 0, 0, 0);
            }
        }
    };
    if (n > 0) {
        request(0);
        for (int k = 1; k < n; ++k) {      // each register is requested again once its product is under way
            multiply();
            request(k);
        }
        multiply();
    }
#pragma unroll
    for (int f = 0; f < F; ++f) {
        mfma_results_here(acc[f]);
        part[wave][f][lane] = acc[f];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < F * 64; i += 64 * W) {
        const int f = i >> 6, l = i & 63;
        if ((l & 15) >= a.T) continue;
        lin_f32x4 v = part[0][f][l];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w][f][l];
        lin_store<float>(a, l & 15, n0 + 16 * f + 4 * (l >> 4), v);
    }
}

// ---------------------------------------------------------------------------------------------
// direct loads to LDS.  A row fragment's step is 16 rows x 64 code bytes, one instruction of 16 bytes
// per lane, a lane quad per row; its 16-byte parts are swizzled by row so that the operand reads meet no
// bank conflict.  Scales: 16 rows x 16 bytes, one instruction of 4 bytes per lane, for 2 (NVFP4) or 4
// (MXFP4) steps.  Rows past the last repeat it, and so do scale bytes past a row's end.
//
// The loads in flight are counted by hand (wait_vm), and LDS is read in asm blocks that wait for their
// own reads: a read that the compiler sees would make it wait for every direct load.
// ---------------------------------------------------------------------------------------------
// Term i (0, 1, 2) of 8 fp32 values as bf16, m1 = i > 0 and m2 = i > 1 as masks of the upper half: what the
// terms before it leave, cut off.  Terms 1 and 2 of an infinite or NaN value come out NaN; the sum over
// term 0 is then not finite and alone gives the result (lin_sum_terms).
__device__ __forceinline__ lin_bf16x8 lin_f32_term(const lin_u32x4& a, const lin_u32x4& b, uint32_t m1, uint32_t m2) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t v = e < 4 ? a[e] : b[e - 4];
        const float r = __uint_as_float(v) - __uint_as_float(v & m1);
        w[e] = __float_as_uint(r - __uint_as_float(__float_as_uint(r) & m2));
    }
    return lin_as_bf16x8(make_uint4(__builtin_amdgcn_perm(w[1], w[0], 0x07060302), __builtin_amdgcn_perm(w[3], w[2], 0x07060302),
                                    __builtin_amdgcn_perm(w[5], w[4], 0x07060302), __builtin_amdgcn_perm(w[7], w[6], 0x07060302)));
}
__device__ __forceinline__ lin_f32x4 lin_sum_terms(const lin_f32x4& s0, const lin_f32x4& s1, const lin_f32x4& s2) {
    lin_f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __builtin_isfinite(s0[i]) ? s0[i] + (s1[i] + s2[i]) : s0[i];
    return r;
}
// tokens of one pass over the weights (blockIdx.y): sixteen columns, or five tokens of three columns
// (column 3 t + i is term i of token t)
template <typename XT>
constexpr int kLinPass = sizeof(XT) == 4 ? 5 : 16;

constexpr int kLinStreamMaxK = 8192;      // x in registers: 8 steps for each of 8 waves
typedef __attribute__((address_space(3))) uint8_t* lin_lds_t;

__device__ __forceinline__ uint32_t lin_lds_offset(const uint8_t* p) { return (uint32_t)(uintptr_t)(lin_lds_t)p; }
__device__ __forceinline__ int lin_swz(int r) { return ((r >> 2) ^ (r >> 1)) & 3; }

template <int WF>
struct LinFmt {
    static constexpr int UB = WF == MOE_WF_MXFP4 ? 4 : 8;      // scale bytes of a row and step
    static constexpr int SPD = 16 / UB;                        // steps of one scale load
};

// wait until at most `left` of this wave's vector-memory operations are in flight
template <int M>
__device__ __forceinline__ void lin_wait_upto(int left) {
    if constexpr (M > 0) {
        if (left < M) {
            lin_wait_upto<M - 1>(left);
            return;
        }
    }
    wait_vm<M>();
}

// the source of a lane's direct loads of codes: its part of its row, from step s0 on
__device__ __forceinline__ const uint8_t* lin_src(const LinArgs& a, int tile, int s0, int lane) {
    const int r = lane >> 2, row = tile * 16 + r < a.N ? tile * 16 + r : a.N - 1;
    return a.q + (size_t)row * (a.K / 2) + (size_t)s0 * 64 + ((lane & 3) ^ lin_swz(r)) * 16;
}
template <int WF>
__device__ __forceinline__ void lin_dma_scales(const LinArgs& a, int tile, int s0, int i, int lane, uint8_t* dst) {
    const int SR = a.K / 128 * LinFmt<WF>::UB;
    const int r = lane >> 2, row = tile * 16 + r < a.N ? tile * 16 + r : a.N - 1;
    const int off = s0 * LinFmt<WF>::UB + i * 16 + (lane & 3) * 4;
    dma4(a.s + (size_t)row * SR + (off < SR ? off : SR - 4), dst);
}

// the waves' sums of a tile, in wave order, and over a token's terms where those are columns: a lane's rows of
// token lane % 16
template <bool TERMS, int W>
__device__ __forceinline__ lin_f32x4 lin_sum_waves(const lin_f32x4* part, int lane) {
    if constexpr (!TERMS) {
        lin_f32x4 v = part[lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w * 64 + lane];
        return v;
    } else {
        const int at = (lane & 48) + 3 * (lane & 15);          // lanes of tokens 0 .. 4
        lin_f32x4 v[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            v[i] = part[at + i];
#pragma unroll
            for (int w = 1; w < W; ++w) v[i] += part[w * 64 + at + i];
        }
        return lin_sum_terms(v[0], v[1], v[2]);
    }
}

// One tile of 16 rows per workgroup, K shared out over W waves.  NX direct loads bring x's step (four bf16 or two
// fp32 tokens each), swizzled by token.  Two steps of codes and x in flight, scales with the first step that
// they serve.  bf16: 16 columns of tokens, or twice 16 (NX = 8).  fp32: up to five tokens of three columns, or
// (NX = 8) 16 columns of tokens, multiplied by each term in turn.
// 4096 x 4096 MXFP4, one token: 4.0 us (8.9 MB; a kernel of one round trip to memory takes 2.0), 16 tokens 5.4, 32
// 7.2; 4096 x 16384 8.6, 14.7 and 20.  Eight waves and two steps were as fast or faster than 4 or 16 waves and one
// to four steps up to 4096 rows.  With many rows x is what costs (65536 x 6144, 16 tokens: 92 us).
template <typename XT, int WF, int NX, int W>
__global__ __launch_bounds__(64 * W) void k_linear_ring(LinArgs a) {
    constexpr int UB = LinFmt<WF>::UB, SPD = LinFmt<WF>::SPD;
    constexpr int STG = (1 + NX) * 1024, SCB = 2 * 256, WB = SCB + 2 * STG;
    constexpr bool F32 = sizeof(XT) == 4, TERMS = F32 && NX <= 3;
    constexpr int TB = 128 * (int)sizeof(XT), TPL = 1024 / TB;  // bytes of a token's step, tokens of one load
    constexpr int C = !F32 && NX > 4 ? 2 : 1, PASS = TERMS ? 5 : 16 * C;
    static_assert(SPD >= 2 && WB >= 1024 * C, "scales outlast the steps in flight; a wave's sums fit into its ring");
    __shared__ __align__(32) uint8_t ring[W * WB];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int tile = blockIdx.x, NS = a.K / 128;
    const int s0 = wave * NS / W, n = (wave + 1) * NS / W - s0;
    const int t0 = blockIdx.y * PASS, nt = a.T - t0 < PASS ? a.T - t0 : PASS;
    uint8_t* mine = ring + wave * WB;
    const uint8_t* qs = lin_src(a, tile, s0, lane);
    const uint8_t* xs[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int t = TPL * i + lane / (64 / TPL), tok = t0 + (t < nt ? t : nt - 1);
        xs[i] = (const uint8_t*)a.x + ((size_t)tok * a.K + (size_t)s0 * 128) * sizeof(XT) + ((lane % (64 / TPL)) ^ (t & 15)) * 16;
    }
    auto issue = [&](int k) {
        uint8_t* st = mine + SCB + (k & 1) * STG;
        if (k % SPD == 0) lin_dma_scales<WF>(a, tile, s0, k / SPD, lane, mine + (k / SPD & 1) * 256);
        dma16(qs + (size_t)k * 64, st);
#pragma unroll
        for (int i = 0; i < NX; ++i) dma16(xs[i] + (size_t)k * TB, st + (1 + i) * 1024);
    };
    if (n > 0) issue(0);
    if (n > 1) issue(1);
    const uint32_t base = lin_lds_offset(mine);
    const uint32_t qa = base + SCB + li * 64 + (lg ^ lin_swz(li)) * 16, sa = base + li * 16 + lg * (UB / 4);
    uint32_t xa[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {                              // columns past the last repeat a token
        const int t = TERMS ? li / 3 % (TPL * NX) : li % (TPL * NX);
        xa[h] = base + SCB + 1024 + t * TB + ((F32 ? 8 * lg + 2 * h : 4 * lg + h) ^ t) * 16;
    }
    const uint32_t m1 = li % 3 > 0 ? 0xffff0000u : 0u, m2 = li % 3 > 1 ? 0xffff0000u : 0u;
    lin_f32x4 acc[C][2];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c][0] = acc[c][1] = lin_f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < n; ++k) {
        if (k + 1 == n) wait_vm<0>();                          // all but the next step's loads are here
        else if ((k + 1) % SPD == 0) wait_vm<2 + NX>();
        else wait_vm<1 + NX>();
        lin_u32x4 code, x[4], x2[4];
        uint32_t sc;
        const uint32_t so = (k & 1) * STG, sk = sa + (k / SPD & 1) * 256 + k % SPD * UB;
        if constexpr (F32 || C == 2) {
            // the other 16 bytes of a lane's 8 fp32 values are in the neighbouring slot, the other 16 tokens a
            // step of 16 tokens on
            const uint32_t f = F32 ? 16 : 0, o = so + (C == 2 ? 16 * TB : 0);
            asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\tds_read_b128 %3, %7\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(x2[0]), "=&v"(x2[1]), "=&v"(x2[2]), "=&v"(x2[3])
                         : "v"((xa[0] + o) ^ f), "v"((xa[1] + o) ^ f), "v"((xa[2] + o) ^ f), "v"((xa[3] + o) ^ f)
                         : "memory");
        }
        if constexpr (WF == MOE_WF_MXFP4)
            asm volatile("ds_read_b128 %0, %6\n\tds_read_u8 %1, %7\n\tds_read_b128 %2, %8\n\tds_read_b128 %3, %9\n\t"
                         "ds_read_b128 %4, %10\n\tds_read_b128 %5, %11\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(code), "=&v"(sc), "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
                         : "v"(qa + so), "v"(sk), "v"(xa[0] + so), "v"(xa[1] + so), "v"(xa[2] + so), "v"(xa[3] + so)
                         : "memory");
        else
            asm volatile("ds_read_b128 %0, %6\n\tds_read_u16 %1, %7\n\tds_read_b128 %2, %8\n\tds_read_b128 %3, %9\n\t"
                         "ds_read_b128 %4, %10\n\tds_read_b128 %5, %11\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(code), "=&v"(sc), "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
                         : "v"(qa + so), "v"(sk), "v"(xa[0] + so), "v"(xa[1] + so), "v"(xa[2] + so), "v"(xa[3] + so)
                         : "memory");
        if (k + 2 < n) issue(k + 2);
        float s2[2];
        lin_scales<WF>(sc, s2);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const lin_bf16x8 w = lin_weights<WF>(code[h], s2[h / 2]);
            if constexpr (TERMS) {
                acc[0][h & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, lin_f32_term(x[h], x2[h], m1, m2), acc[0][h & 1], 0, 0, 0);
            } else if constexpr (F32) {
                lin_bf16x8 t[3];
                lin_f32_terms(x[h], x2[h], t);
#pragma unroll
                for (int i = 0; i < 3; ++i) acc[0][h & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, t[i], acc[0][h & 1], 0, 0, 0);
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    lin_bf16x8 xv;
                    __builtin_memcpy(&xv, c ? &x2[h] : &x[h], 16);
                    acc[c][h & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xv, acc[c][h & 1], 0, 0, 0);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        acc[c][0] += acc[c][1];
        mfma_results_here(acc[c][0]);
    }
    __syncthreads();
    lin_f32x4* part = (lin_f32x4*)ring;
#pragma unroll
    for (int c = 0; c < C; ++c) part[(c * W + wave) * 64 + lane] = acc[c][0];
    __syncthreads();
    if (wave < C && 16 * wave + li < nt)
        lin_store<XT>(a, t0 + 16 * wave + li, tile * 16 + 4 * lg, lin_sum_waves<TERMS, W>(part + wave * W * 64, lane));
}

// Tiles of 16 rows blockIdx.x, blockIdx.x + G, .. (G workgroups); wave w of 8 takes K slice w of every
// tile and keeps x's slice in registers.  A wave's ring holds two tiles of its slice.  The waves' sums of
// kLinRound tiles meet in LDS between two barriers, one wave adding up each tile in wave order.
// Rounds: sums of 1, 2, 3 tiles at a time in two buffers, one barrier a round, took 65, 56 and 53 us at
// 65536 x 6144 NVFP4 and 16 tokens; one buffer of 4 tiles with two barriers 53, one of 6 52.
// Now 50 us there, 228 MB at 4.5 TB/s (MXFP4 43): bringing x's 196 KB to every CU takes about 5 of them before
// the first product.  The decode does not bound it: fp16 weights at half the instructions took as long.
constexpr int kLinWaves = 8;

template <typename XT, int WF, int NSW>
__global__ __launch_bounds__(64 * kLinWaves) void k_linear_stream(LinArgs a, int ntiles) {
    constexpr int W = kLinWaves, R = NSW <= 6 ? 4 : 2;          // (8 steps leave LDS for the sums of two)
    constexpr int UB = LinFmt<WF>::UB, SPD = LinFmt<WF>::SPD, NSC = (NSW + SPD - 1) / SPD;
    constexpr int STG = NSW * 1024 + NSC * 256;
    constexpr bool F32 = sizeof(XT) == 4;
    static_assert(NSW % 2 == 0 && STG >= 4096, "steps are read in pairs; a slot of the ring holds a step of x");
    __shared__ __align__(16) uint8_t ring[W * 2 * STG];
    __shared__ lin_f32x4 part[R][W][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int NS = a.K / 128, G = gridDim.x;
    const int s0 = wave * NS / W, n = (wave + 1) * NS / W - s0, nsc = (n + SPD - 1) / SPD;
    const int t0 = blockIdx.y * kLinPass<XT>, nt = a.T - t0 < kLinPass<XT> ? a.T - t0 : kLinPass<XT>;
    uint8_t* mine = ring + wave * 2 * STG;
    auto issue = [&](int tile, int slot) {
        const uint8_t* q = lin_src(a, tile, s0, lane);
        uint8_t* st = mine + slot * STG;
#pragma unroll
        for (int i = 0; i < NSW; ++i)
            if (i < n) dma16(q + i * 64, st + i * 1024);
#pragma unroll
        for (int i = 0; i < NSC; ++i)
            if (i < nsc) lin_dma_scales<WF>(a, tile, s0, i, lane, st + NSW * 1024 + i * 256);
    };
    int tile = blockIdx.x;
    issue(tile, 0);
    lin_bf16x8 x[NSW][4];
    if constexpr (F32) {
        // this lane's token and term
        const int t = t0 + (li / 3 < nt ? li / 3 : nt - 1);
        const float* xr = (const float*)a.x + (size_t)t * a.K + lg * 32;
        const uint32_t m1 = li % 3 > 0 ? 0xffff0000u : 0u, m2 = li % 3 > 1 ? 0xffff0000u : 0u;
#pragma unroll
        for (int i = 0; i < NSW; ++i) {
            const int k = s0 + i < NS ? s0 + i : NS - 1;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                lin_u32x4 v[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 u = gload16(xr + (size_t)k * 128 + 8 * h + 4 * j);
                    v[j] = lin_u32x4{u.x, u.y, u.z, u.w};
                }
                x[i][h] = lin_f32_term(v[0], v[1], m1, m2);
            }
        }
    } else {
        // in row order (four tokens x 256 bytes a load), then through the ring's second slot to the
        // operand layout
        uint4 raw[NSW][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * j + lg, tok = t < nt ? t : nt - 1;
            const uint16_t* xr = (const uint16_t*)a.x + (size_t)(t0 + tok) * a.K + (li ^ t) * 8;
#pragma unroll
            for (int i = 0; i < NSW; ++i) raw[i][j] = gload16(xr + (size_t)(s0 + i < NS ? s0 + i : NS - 1) * 128);
        }
        uint4* stage = (uint4*)(mine + STG);
#pragma unroll
        for (int i = 0; i < NSW; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) stage[j * 64 + lane] = raw[i][j];
            asm volatile("" ::: "memory");                    // one wave's own reads and writes, in order
#pragma unroll
            for (int h = 0; h < 4; ++h) x[i][h] = lin_as_bf16x8(stage[li * 16 + ((lg * 4 + h) ^ li)]);
            asm volatile("" ::: "memory");
        }
    }
    // x is here (and the first tile) before the loop, whose waits count the ring's loads alone
    wait_vm<0>();
#pragma unroll
    for (int i = 0; i < NSW; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h) asm volatile("" : "+v"(x[i][h]));
    if (tile + G < ntiles) issue(tile + G, 1);                 // the slot's reads are over: their values are used above

    const uint32_t base = lin_lds_offset(mine);
    const uint32_t qa = base + li * 64 + (lg ^ lin_swz(li)) * 16, sa = base + NSW * 1024 + li * 16 + lg * (UB / 4);
    for (int it = 0; tile < ntiles; tile += G, ++it) {
        const bool more = tile + G < ntiles;
        // the next tile's loads may be in flight (a store of y counts as one more, which only waits longer)
        lin_wait_upto<NSW + NSC>(more ? n + nsc : 0);
        const uint32_t so = (it & 1) * STG;
        lin_u32x4 code[NSW];
        uint32_t sc[NSW];
#pragma unroll
        for (int i = 0; i < NSW; i += 2) {
            const uint32_t sk = sa + so + (i / SPD) * 256 + (i % SPD) * UB;
            if constexpr (WF == MOE_WF_MXFP4)
                asm volatile("ds_read_b128 %0, %4\n\tds_read_u8 %2, %5\n\tds_read_b128 %1, %4 offset:1024\n\t"
                             "ds_read_u8 %3, %5 offset:4\n\ts_waitcnt lgkmcnt(0)"
                             : "=&v"(code[i]), "=&v"(code[i + 1]), "=&v"(sc[i]), "=&v"(sc[i + 1])
                             : "v"(qa + so + i * 1024), "v"(sk) : "memory");
            else
                asm volatile("ds_read_b128 %0, %4\n\tds_read_u16 %2, %5\n\tds_read_b128 %1, %4 offset:1024\n\t"
                             "ds_read_u16 %3, %5 offset:8\n\ts_waitcnt lgkmcnt(0)"
                             : "=&v"(code[i]), "=&v"(code[i + 1]), "=&v"(sc[i]), "=&v"(sc[i + 1])
                             : "v"(qa + so + i * 1024), "v"(sk) : "memory");
        }
        if (tile + 2 * G < ntiles) issue(tile + 2 * G, it & 1);
        lin_f32x4 acc[2] = {lin_f32x4{0.f, 0.f, 0.f, 0.f}, lin_f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < NSW; ++i) {
            if (i >= n) continue;
            float s2[2];
            lin_scales<WF>(sc[i], s2);
#pragma unroll
            for (int h = 0; h < 4; ++h)
                acc[h & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lin_weights<WF>(code[i][h], s2[h / 2]), x[i][h],
                                                                     acc[h & 1], 0, 0, 0);
        }
        acc[0] += acc[1];
        mfma_results_here(acc[0]);
        part[it % R][wave][lane] = acc[0];
        if (it % R != R - 1 && more) continue;
        lds_barrier();
        const int j = it / R * R + wave;                       // the round's tile that this wave adds up
        if (j <= it && wave < R && li < nt)
            lin_store<XT>(a, t0 + li, (blockIdx.x + j * G) * 16 + 4 * lg, lin_sum_waves<F32, W>(&part[wave][0][0], lane));
        lds_barrier();                                         // the next round overwrites the sums
    }
}

// N 16-byte reads of LDS, STRIDE apart
template <int N, int STRIDE>
__device__ __forceinline__ void lin_read(uint32_t at, lin_u32x4 (&v)[N]) {
    static_assert(N == 2 || N == 4 || N == 6, "numbers of reads that the tile kernel makes");
    if constexpr (N == 2)
        asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0]), "=&v"(v[1]) : "v"(at), "n"(STRIDE) : "memory");
    else if constexpr (N == 4)
        asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:%5\n\tds_read_b128 %2, %4 offset:%6\n\t"
                     "ds_read_b128 %3, %4 offset:%7\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
                     : "v"(at), "n"(STRIDE), "n"(2 * STRIDE), "n"(3 * STRIDE) : "memory");
    else
        asm volatile("ds_read_b128 %0, %6\n\tds_read_b128 %1, %6 offset:%7\n\tds_read_b128 %2, %6 offset:%8\n\t"
                     "ds_read_b128 %3, %6 offset:%9\n\tds_read_b128 %4, %6 offset:%10\n\tds_read_b128 %5, %6 offset:%11\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5])
                     : "v"(at), "n"(STRIDE), "n"(2 * STRIDE), "n"(3 * STRIDE), "n"(4 * STRIDE), "n"(5 * STRIDE) : "memory");
}

// Many rows and many tokens: 16 F rows per wave, eight waves over rows, and 16 C tokens, whose step of x the
// waves share in LDS; each wave has its own ring of codes and scales.  S steps alive, one barrier a step.
// fp32 x is cut into its terms once per workgroup and step, each wave the part that it loaded.
// 65536 x 6144 MXFP4, bf16: 32 tokens 54 us, 64 70; fp32: 102 and 190 (at the matrix cores' 1.23 PFLOP/s 63 and
// 126).  16384 rows are 128 workgroups on 256 CUs: 19 and 28 us with 4096 columns.  With the workgroups' rows on few CUs a step's chain of LDS reads, decode, products and barrier (0.5 us)
// bounds it: steps of 256 K, all of a step's reads at once or four stages for three took as long; sixteen waves
// that share out a step's K took 22 us for 27 at 16384 x 4096 and 64 tokens, but 82 for 68 at 65536 x 6144.
template <typename XT, int WF, int C, int F, int S>
__global__ __launch_bounds__(512) void k_linear_tile(LinArgs a) {
    constexpr int UB = LinFmt<WF>::UB, SPD = LinFmt<WF>::SPD, W = 8;
    constexpr bool F32 = sizeof(XT) == 4;
    constexpr int NT = F32 ? 3 : 1;
    constexpr int TB = 128 * (int)sizeof(XT), TPL = 1024 / TB;  // bytes of a token's step, tokens of one load
    constexpr int XL = 16 * C / TPL / W;                        // loads of x per wave and step
    constexpr int XSTG = 16 * C * TB, TERMS = F32 ? NT * C * 4096 : 0;
    constexpr int SL = S == 3 ? 2 : 4;                          // loads of scales that are alive
    constexpr int CW = S * F * 1024 + SL * F * 256, P = F + XL;
    static_assert(XL >= 1 && (!F32 || XL == 2) && SPD >= 2 && (S == 3 || S == 4), "shares of the loads; scales outlast them");
    __shared__ __align__(1024) uint8_t lds[S * XSTG + 2 * TERMS + W * CW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int tile = (blockIdx.x * W + wave) * F, n = a.K / 128;
    const int t0 = blockIdx.y * 16 * C, nt = a.T - t0 < 16 * C ? a.T - t0 : 16 * C;
    uint8_t* mine = lds + S * XSTG + 2 * TERMS + wave * CW;
    const uint8_t* qs[F];
    const uint8_t* xs[XL];
#pragma unroll
    for (int f = 0; f < F; ++f) qs[f] = lin_src(a, tile + f, 0, lane);
#pragma unroll
    for (int i = 0; i < XL; ++i) {                              // fp32 in order, bf16 swizzled by token
        const int t = (wave * XL + i) * TPL + lane / (64 / TPL), tok = t0 + (t < nt ? t : nt - 1);
        xs[i] = (const uint8_t*)a.x + (size_t)tok * a.K * sizeof(XT) + (F32 ? lane % 32 : (lane % 16) ^ (t & 15)) * 16;
    }
    int slot_in = 0;                                           // of the next step to request
    auto issue = [&](int k) {
        if (k % SPD == 0)
#pragma unroll
            for (int f = 0; f < F; ++f)
                lin_dma_scales<WF>(a, tile + f, 0, k / SPD, lane, mine + S * F * 1024 + ((k / SPD % SL) * F + f) * 256);
#pragma unroll
        for (int f = 0; f < F; ++f) dma16(qs[f] + (size_t)k * 64, mine + (slot_in * F + f) * 1024);
#pragma unroll
        for (int i = 0; i < XL; ++i) dma16(xs[i] + (size_t)k * TB, lds + slot_in * XSTG + (wave * XL + i) * 1024);
        slot_in = slot_in + 1 == S ? 0 : slot_in + 1;
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k)
        if (k < n) issue(k);
    const uint32_t base = lin_lds_offset(lds), my = lin_lds_offset(mine);
    const uint32_t qa = my + li * 64 + (lg ^ lin_swz(li)) * 16, sa = my + S * F * 1024 + li * 16 + lg * (UB / 4);
    uint32_t xa[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) xa[h] = base + (F32 ? S * XSTG : 0) + li * 256 + ((4 * lg + h) ^ li) * 16;
    lin_f32x4 acc[F][C];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[f][c] = lin_f32x4{0.f, 0.f, 0.f, 0.f};
    int slot = 0;
    for (int k = 0; k < n; ++k) {
        if (k + S - 2 >= n) wait_vm<0>();                      // all but the loads of the steps behind are here
        else if constexpr (S == 3) {
            if ((k + 1) % SPD == 0) wait_vm<P + F>();
            else wait_vm<P>();
        } else {
            if ((k + 1) % SPD == 0 || (k + 2) % SPD == 0) wait_vm<2 * P + F>();
            else wait_vm<2 * P>();
        }
        if constexpr (F32) {
            const uint32_t raw = base + slot * XSTG + wave * 2048 + lane * 32;
            lin_u32x4 v[2];
            lin_read<2, 16>(raw, v);
            lin_bf16x8 t[3];
            lin_f32_terms(v[0], v[1], t);
            const int tk = 4 * wave + lg;                      // the lane's token and 8 values
            const uint32_t to = base + S * XSTG + (k & 1) * TERMS + tk * 256 + (li ^ (tk & 15)) * 16;
            lin_u32x4 w[3];
            __builtin_memcpy(w, t, 48);
            asm volatile("ds_write_b128 %0, %1\n\tds_write_b128 %0, %2 offset:%4\n\tds_write_b128 %0, %3 offset:%5\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         :: "v"(to), "v"(w[0]), "v"(w[1]), "v"(w[2]), "n"(C * 4096), "n"(2 * C * 4096) : "memory");
        }
        lds_barrier();
        if (k + S - 1 < n) issue(k + S - 1);
        const uint32_t xo = F32 ? (k & 1) * TERMS : slot * XSTG;
        lin_u32x4 code[F];
        float s2[F][2];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            uint32_t sc;
            const uint32_t sk = sa + ((k / SPD % SL) * F + f) * 256 + k % SPD * UB;
            if constexpr (WF == MOE_WF_MXFP4)
                asm volatile("ds_read_b128 %0, %2\n\tds_read_u8 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                             : "=&v"(code[f]), "=&v"(sc) : "v"(qa + (slot * F + f) * 1024), "v"(sk) : "memory");
            else
                asm volatile("ds_read_b128 %0, %2\n\tds_read_u16 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                             : "=&v"(code[f]), "=&v"(sc) : "v"(qa + (slot * F + f) * 1024), "v"(sk) : "memory");
            lin_scales<WF>(sc, s2[f]);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            lin_u32x4 x[C * NT];
            lin_read<C * NT, 4096>(xa[h] + xo, x);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const lin_bf16x8 w = lin_weights<WF>(code[f][h], s2[f][h / 2]);
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        lin_bf16x8 xv;
                        __builtin_memcpy(&xv, &x[i * C + c], 16);
                        acc[f][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xv, acc[f][c], 0, 0, 0);
                    }
            }
        }
        slot = slot + 1 == S ? 0 : slot + 1;
    }
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            mfma_results_here(acc[f][c]);
            if (16 * c + li < nt) lin_store<XT>(a, t0 + 16 * c + li, (tile + f) * 16 + 4 * lg, acc[f][c]);
        }
}

template <typename XT, int WF, int NX>
static void ring_launch(const LinArgs& a, int passes, hipStream_t st) {
    MOE_LAUNCH((k_linear_ring<XT, WF, NX, 8>), dim3((a.N + 15) / 16, passes), dim3(512), 0, st, a);
}

template <typename XT, int WF>
static void stream_launch(const LinArgs& a, int passes, hipStream_t st) {
    const int ntiles = (a.N + 15) / 16, n = (a.K / 128 + kLinWaves - 1) / kLinWaves;
    const dim3 grid(ntiles < 256 ? ntiles : 256, passes), block(64 * kLinWaves);          // a workgroup per CU
    if (n <= 4) MOE_LAUNCH((k_linear_stream<XT, WF, 4>), grid, block, 0, st, a, ntiles);
    else if (n <= 6) MOE_LAUNCH((k_linear_stream<XT, WF, 6>), grid, block, 0, st, a, ntiles);
    else MOE_LAUNCH((k_linear_stream<XT, WF, 8>), grid, block, 0, st, a, ntiles);
}

template <typename XT, int WF, int C, int S>
static void tile_launch_columns(const LinArgs& a, hipStream_t st) {
    const int passes = (a.T + 16 * C - 1) / (16 * C);
    // two fragments of 16 rows per wave once one would take more than a workgroup per CU, but for 32 bf16 tokens, whose
    // step is short: 49152 x 4096, 64 bf16 tokens 45 us for 55, 32 fp32 tokens 67 for 95; 32 bf16 tokens 33 for 34, with 98304
    // rows 64 for 53
    if constexpr (sizeof(XT) == 4 || C == 4) {
        if ((long long)(a.N + 127) / 128 * passes > 256) {
            MOE_LAUNCH((k_linear_tile<XT, WF, C, 2, S>), dim3((a.N + 255) / 256, passes), dim3(512), 0, st, a);
            return;
        }
    }
    MOE_LAUNCH((k_linear_tile<XT, WF, C, 1, S>), dim3((a.N + 127) / 128, passes), dim3(512), 0, st, a);
}
template <typename XT, int WF>
static void tile_launch(const LinArgs& a, hipStream_t st) {
    if constexpr (sizeof(XT) == 4) tile_launch_columns<XT, WF, 2, 3>(a, st);
    else if (a.T <= 32) tile_launch_columns<XT, WF, 2, 4>(a, st);
    else tile_launch_columns<XT, WF, 4, 4>(a, st);
}

enum class LinKernel { ring, stream, tile, straight };

// The kernel for N rows, K columns and T tokens.  Each boundary stands where the times of two kernels cross, over 6300
// timings (1024 to 131072 rows by 512 to 12288 columns, 1 to 64 tokens, both formats, the weights in memory and not in
// the caches).  At 3300 other sizes at random between them the choice takes at most 10% longer than the best kernel in
// 95% of the bf16 ones and 99% of the fp32 ones, and on average 1%.  Some of the timings, us, MXFP4:
//   the stream against the ring: x in registers pays once a CU has several tiles of long rows.  bf16: 8192 x 4096,
//   16 tokens 8.0, 10.8; 16384 x 4096, 2 tokens 10.7, 10.0, 8 tokens 10.8, 12.8; 65536 x 6144, 1 token 41.7, 45.8;
//   16384 x 1024, 4 tokens 7.0, 4.5.  fp32, 5 tokens: 12288 x 4096 11.4, 14.3; 8192 x 2048 8.3, 6.5.
//   the tile against the ring or the stream: x shared by 128 or 256 rows pays with short rows, rows past the
//   registers and more than 16 tokens.  bf16: 65536 x 512, 16 tokens 8.2, 15.5; 32768 x 12288, 8 tokens 52, 63;
//   12288 x 2048, 64 tokens 15.7, 22.5; 8192 x 4096, 32 tokens 18.6, 12.7.
//   k_linear (straight) against the stream in two passes and the ring, fp32: 65536 x 2048, 8 tokens 32, 36;
//   65536 x 6144 88, 77 (NVFP4 93, 96); 20239 x 3200, 9 tokens 25, 23; 12288 x 4096, 16 tokens 21, 33; 4096 x 4096 18, 13.
//   k_linear against the tile, fp32, 16 tokens: 65536 x 6144 111, 97, but 98304 x 4096 107, 125 and 49152 x 4096 56, 64,
//   whose workgroups leave CUs idle at the end: k_linear throughout.
static LinKernel lin_kernel_bf16(int N, int K, int T) {
    const long long NK = (long long)N * K;
    const bool fit = K <= kLinStreamMaxK, deep = fit && K > 2560;
    bool tile, stream;
    if (T <= 4) {
        stream = T > 2 ? deep && NK >= 1 << 27 : K > 4096 && K <= 6144 && NK >= 1 << 28;
        tile = N >= 49152 && K <= 512;
    } else if (T <= 8) {
        const int wgs = (N + 127) / 128, rounds = (wgs + 255) / 256;
        stream = deep ? N >= 12288 : fit && K >= 1536 && N >= (K >= 2048 ? 16384 : 49152);
        tile = K <= 512 ? N >= 24576 : N >= 32768 && (K <= 1024 || (!fit && 4 * wgs >= 3 * 256 * rounds));
    } else if (T <= 16) {
        stream = deep ? N >= 6144 : fit && K > 1024 && N > 8192;
        tile = K <= 512 ? N >= 8192 : K <= 1024 ? N >= 12288 : !fit && N >= 24576;
    } else if (T <= 32) {
        stream = K >= 4096 && K <= 6144 && N >= 12288 && N < 16384;
        tile = N >= 16384 || (N >= 9216 && K <= 1536) || (N >= 12288 && K < 4096);
    } else {
        stream = fit && K >= 4096 && T <= 48 && N >= 8192 && N < 16384;
        tile = N >= 12288 || (N >= 8192 && K <= 2048) || (N >= 6144 && K <= 512);
    }
    return stream ? LinKernel::stream : tile ? LinKernel::tile : LinKernel::ring;
}

// mx: MXFP4 (NVFP4 takes longer to decode, and the stream decodes once a pass)
static LinKernel lin_kernel_f32(int N, int K, int T, bool mx) {
    const bool fit = K <= kLinStreamMaxK, deep = fit && K > 2560;
    if (T <= 5) {
        if (deep ? N >= 8192 : fit && K > 1024 && N >= 16384) return LinKernel::stream;
        return K <= 1024 && N >= 16384 ? LinKernel::straight : LinKernel::ring;
    }
    if (T <= 10) {
        if (mx && deep && N > 16384) return LinKernel::stream;
        return N > 8192 || (N == 8192 && K <= 2048) ? LinKernel::straight : LinKernel::ring;
    }
    if (T <= 16) return N >= 5632 ? LinKernel::straight : LinKernel::ring;
    if (deep && T <= 24 && N >= 12288 && N < 16384) return LinKernel::stream;
    // the ring's time grows with rows times passes, the tile's steps by rounds of the chip
    const int passes = (T + 4) / 5, least = K <= 512 ? 24576 : K <= 1024 ? 43008 : 49152;
    return (long long)N * passes >= least ? LinKernel::tile : LinKernel::ring;
}

template <typename XT, int WF>
static void linear_launch(const LinArgs& a, hipStream_t st) {
    constexpr bool F32 = sizeof(XT) == 4;
    const int tiles = (a.N + 15) / 16, passes = (a.T + kLinPass<XT> - 1) / kLinPass<XT>;
    const LinKernel kernel = F32 ? lin_kernel_f32(a.N, a.K, a.T, WF == MOE_WF_MXFP4) : lin_kernel_bf16(a.N, a.K, a.T);
    if (kernel == LinKernel::tile) return tile_launch<XT, WF>(a, st);
    if (kernel == LinKernel::stream) return stream_launch<XT, WF>(a, passes, st);
    if constexpr (F32) {
        if (kernel == LinKernel::straight) {
            MOE_LAUNCH((k_linear<WF>), dim3((a.N + 63) / 64), dim3(512), 0, st, a);
            return;
        }
        // 16 tokens in one pass (their terms in turn), a workgroup per CU, take as long as three rounds of 256 workgroups
        // of five, of which two share a CU: 4096 x 4096, 16 tokens 12.7 us for 16.1, 20 tokens 23 for 16.2; 4220 x 4992, 15
        // tokens 26.8 for 18.5; 1024 x 2048, 16 tokens 7.5 for 5.0
        const int wgs5 = tiles * passes, passes16 = (a.T + 15) / 16, rounds16 = (tiles * passes16 + 255) / 256;
        if (a.T <= 2) ring_launch<XT, WF, 1>(a, 1, st);
        else if (a.T <= 4) ring_launch<XT, WF, 2>(a, 1, st);
        else if (a.T <= 10 || wgs5 <= 512 || (rounds16 > 1 && wgs5 < 3 * 256 * rounds16)) ring_launch<XT, WF, 3>(a, passes, st);
        else ring_launch<XT, WF, 8>(a, passes16, st);
    } else {
        // 32 tokens in one pass once two of 16 no longer run side by side: 4096 x 4096 7.2 us for 8.5; 2048 x 4096 6.8 for 5.4
        if (a.T <= 4) ring_launch<XT, WF, 1>(a, 1, st);
        else if (a.T <= 8) ring_launch<XT, WF, 2>(a, 1, st);
        else if (a.T <= 16 || tiles * passes <= 256) ring_launch<XT, WF, 4>(a, passes, st);
        else ring_launch<XT, WF, 8>(a, (a.T + 31) / 32, st);
    }
}

hipError_t launch_linear(const moe_matrix* m, const uint8_t* q, const uint8_t* s, float ts, const void* x, int T,
                         const float* bias, void* y, hipStream_t st) {
    trace("linear", 0, st);
    const LinArgs a = {m->rows, m->cols, T, q, s, ts, x, bias, y};
    const bool bf = m->act_dtype == MOE_DT_BF16;
    if (m->wformat == MOE_WF_MXFP4)
        bf ? linear_launch<uint16_t, MOE_WF_MXFP4>(a, st) : linear_launch<float, MOE_WF_MXFP4>(a, st);
    else
        bf ? linear_launch<uint16_t, MOE_WF_NVFP4>(a, st) : linear_launch<float, MOE_WF_NVFP4>(a, st);
    trace("linear", 1, st);
    return hipGetLastError();
}

}  // namespace moe
