// Matrix-vector products of up to 64 vectors with a dense weight in the experts' 4-bit formats.
//
//   y[t,n] = ts sum_k W[n,k] x[t,k] (+ bias[n]),   W[n,k] = E2M1 code x block scale.
//
// A code times its block scale is exact in bf16 (one bit of mantissa times a power of two, or times
// the four bits of an E4M3 scale), so the weights enter the bf16 matrix cores exactly; a bf16 x does
// too, and an fp32 x is the sum of three bf16 terms cut from it (8 + 8 + 8 bits, exact), each one more
// MFMA into the same fp32 sums.
//
// V_MFMA_F32_16X16X32_BF16: lane l supplies 8 consecutive K of weight row (A) or token (B) l % 16;
// any assignment of K to the lane groups works when both operands share it.  A step covers 128 K of a
// row: lane group g takes elements [32 g, 32 g + 32), 16 code bytes in one load, and MFMA h of the step
// their elements [8 h, 8 h + 8).  C: lane l, register r is weight row 4 (l / 16) + r, token l % 16.
#include "moe_internal.h"

namespace moe {

typedef __bf16 lin_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 lin_bf16x2 __attribute__((ext_vector_type(2)));
typedef float lin_f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ lin_bf16x8 lin_as_bf16x8(const uint4& v) {
    lin_bf16x8 r;
    __builtin_memcpy(&r, &v, 16);
    return r;
}

// 8 codes (one dword, element 2i in the low nibble of byte i) times a scale, exact in bf16
__device__ __forceinline__ lin_bf16x8 lin_weights(uint32_t codes, float scale) {
    lin_bf16x8 r;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const v2f_t v = b == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0)
                      : b == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1)
                      : b == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2)
                               : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
        r[2 * b] = (__bf16)(v[0] * scale);
        r[2 * b + 1] = (__bf16)(v[1] * scale);
    }
    return r;
}

// E8M0 byte -> 2^(b - 127) (b = 0 is a subnormal float; b = 255 is NaN)
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
    return __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
}

// x's operand of one MFMA: NT bf16 terms of 8 consecutive elements
template <typename XT>
struct LinX {
    static constexpr int NT = sizeof(XT) == 4 ? 3 : 1;
    lin_bf16x8 t[NT];
};

template <typename XT>
__device__ __forceinline__ LinX<XT> lin_load_x(const XT* p, bool valid) {
    LinX<XT> r;
    if constexpr (sizeof(XT) == 2) {
        r.t[0] = lin_as_bf16x8(valid ? *(const uint4*)p : make_uint4(0, 0, 0, 0));
    } else {
        // cut, not rounded: the first term of a large value never becomes infinite; an infinite
        // value is its own first term
        f32x8 v = {};
        if (valid) v = load_act8(p, 0);
        uint32_t w[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float rest = v.v[e];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const uint32_t cut = __float_as_uint(rest) & 0xffff0000u;
                w[i][e] = cut;
                rest = (cut & 0x7fffffffu) == 0x7f800000u ? 0.0f : rest - __uint_as_float(cut);
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
            r.t[i] = lin_as_bf16x8(make_uint4(w[i][0] >> 16 | w[i][1], w[i][2] >> 16 | w[i][3], w[i][4] >> 16 | w[i][5],
                                              w[i][6] >> 16 | w[i][7]));
    }
    return r;
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

// A workgroup of W waves owns 16 F rows and 16 C tokens; its waves share out K, and their sums are
// added through LDS in wave order.
template <typename XT, int WF, int F, int C, int W>
__global__ __launch_bounds__(64 * W) void k_linear(LinArgs a) {
    __shared__ lin_f32x4 part[W][F * C][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16 * F, t0 = blockIdx.y * 16 * C;
    const int NS = a.K / 128;
    const int s0 = wave * NS / W, s1 = (wave + 1) * NS / W;
    constexpr int SB = WF == MOE_WF_MXFP4 ? 32 : 16;          // weights per scale
    const uint8_t* q[F];
    const uint8_t* s[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const int row = n0 + 16 * f + li < a.N ? n0 + 16 * f + li : a.N - 1;
        q[f] = a.q + (size_t)row * (a.K / 2) + lg * 16;
        s[f] = a.s + (size_t)row * (a.K / SB) + lg * (32 / SB);
    }
    const XT* x[C];
    bool tok[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        tok[c] = t0 + 16 * c + li < a.T;
        x[c] = (const XT*)a.x + (size_t)(tok[c] ? t0 + 16 * c + li : 0) * a.K + lg * 32;
    }
    lin_f32x4 acc[F][C];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[f][c] = lin_f32x4{0.f, 0.f, 0.f, 0.f};
    for (int ks = s0; ks < s1; ++ks) {
        uint4 code[F];
        float sc[F][2];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            code[f] = gload16(q[f] + (size_t)ks * 64);
            if constexpr (WF == MOE_WF_MXFP4) {
                sc[f][0] = sc[f][1] = e8m0_to_f32(s[f][(size_t)ks * 4]);
            } else {
                const v2f_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(*(const uint16_t*)(s[f] + (size_t)ks * 8), 1.0f, false);
                sc[f][0] = v[0];
                sc[f][1] = v[1];
            }
        }
        LinX<XT> xv[C][4];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int h = 0; h < 4; ++h) xv[c][h] = lin_load_x(x[c] + (size_t)ks * 128 + 8 * h, tok[c]);
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const uint32_t word = h == 0 ? code[f].x : h == 1 ? code[f].y : h == 2 ? code[f].z : code[f].w;
                const lin_bf16x8 wv = lin_weights(word, sc[f][h / 2]);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < LinX<XT>::NT; ++i)
                        acc[f][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xv[c][h].t[i], acc[f][c], 0, 0, 0);
            }
    }
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            mfma_results_here(acc[f][c]);
            part[wave][f * C + c][lane] = acc[f][c];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < F * C * 64; i += 64 * W) {
        const int fc = i >> 6, l = i & 63;
        const int t = t0 + 16 * (fc % C) + (l & 15), n = n0 + 16 * (fc / C) + 4 * (l >> 4);
        if (t >= a.T) continue;
        lin_f32x4 v = part[0][fc][l];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w][fc][l];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < a.N)
                store_act((XT*)a.y, (size_t)t * a.N + n + r, fmaf(v[r], a.ts, a.bias ? a.bias[n + r] : 0.0f));
    }
}

template <typename XT, int WF>
static void linear_launch(const LinArgs& a, hipStream_t st) {
    MOE_LAUNCH((k_linear<XT, WF, 1, 1, 8>), dim3((a.N + 15) / 16, (a.T + 15) / 16), dim3(512), 0, st, a);
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
