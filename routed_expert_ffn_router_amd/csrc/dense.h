// Declarations of the dense products (dense.hip, dense_few.hip): the products' arguments, the
// epilogue shared by the kernels, and the launchers.
#pragma once

#include "block_ops.h"
#include "dense_rule.h"

namespace moe {

// bytes of a row of scales in the products of MXFP8: a step's four are read at once
constexpr int scale_row(int K) { return (K + 127) / 128 * 4; }

// One product out[i][j] = sum_k P[i][k] Q[j][k], i < I, j < J, with its epilogue.  P and Q are bf16, fp32 or MXFP8
// codes; each is stored with k along its rows ([i][k]) or, "k-major", across them ([k][i]).
struct ProductArgs {
    int I, J, K;
    const uint8_t *p, *q;
    int p_ld, q_ld;               // bytes of a stored row
    const uint8_t *p_scales, *q_scales;   // MXFP8: a byte for each 32 of k, rows of scale_row(K) bytes (past K/32: no NaN's)
    int splits;                   // parts of the sum over k; more than one: fp32 sums to part, [splits][I][J]
    float* part;
    // epilogue; the outputs' rows are J long (gated: N = J / 2)
    int activation;
    int out_f32;                  // type of residual, pre and out: fp32 or bf16
    const float* bias;            // or null
    const void* residual;         // or null
    void* pre;                    // or null: the activation's argument (gated: both halves, [I][J])
    void* out;
    uint8_t* out_scales;          // or null; gated only: out in MXFP8
};

// ---------------------------------------------------------------------------------------------
// activations, in fp32
// ---------------------------------------------------------------------------------------------
// 1 / d for d of ordinary size, to a rounding: a bare reciprocal instruction is a unit off
__device__ __forceinline__ float reciprocal(float d) {
    const float r = __builtin_amdgcn_rcpf(d);
    return fmaf(fmaf(-d, r, 1.0f), r, r);
}
// The logistic function of v and of -v, each right relative to itself: 1 - p has lost q where p is next to 1.
struct Logistic {
    float p, q;
};
__device__ __forceinline__ Logistic logistic(float v) {
    const float e = expf(-fabsf(v)), large = reciprocal(1.0f + e), small = e * large;
    return v < 0.0f ? Logistic{small, large} : Logistic{large, small};
}
// The normal distribution's function, and exp(-v^2 / 2).  With x = |v|, Phi(-x) = exp(-x^2 / 2) R(x): R = 1/2 + u S(u) with
// u = x / (x + 9/4), S the polynomial of degree 8 whose largest relative error of R over 0 .. 13.4 is least (half of 2^-24; a
// fit to the scaled complementary error function by reweighted least squares).  Past 13.2 the exponential is zero.  Its
// argument is carried in two parts, since a rounding of x^2 / 2 = 80 is one of 80 units of the result.  Evaluated in fp32
// Phi(-x) is right to 33 * 2^-24 of itself and Phi to 1.7 * 2^-24.  4096^3 with bias and residual: 148.7 us; 145 with a
// formula that is right to 8 * 2^-24 of 1 only.
struct Normal {
    float cdf, density;
};
__device__ __forceinline__ Normal normal(float v) {
    const float x = fabsf(v) > 32.0f ? 32.0f : fabsf(v), u = x * reciprocal(x + 2.25f);        // (a NaN stays)
    float p = fmaf(u, -0.0354012474f, 0.104736947f);
    p = fmaf(u, p, -0.0872863159f);
    p = fmaf(u, p, 0.0347602181f);
    p = fmaf(u, p, -0.0652041808f);
    p = fmaf(u, p, -0.0407651812f);
    p = fmaf(u, p, 0.118775897f);
    p = fmaf(u, p, 0.367995501f);
    p = fmaf(u, p, -0.897619307f);
    constexpr float C = -0.72134752044448170f, CL = (float)(-0.72134752044448170 - (double)C);     // -log2(e) / 2
    const float s = x * x, hi = s * C, lo = fmaf(fmaf(x, x, -s), C, fmaf(s, CL, fmaf(s, C, -hi)));
    const float e0 = __builtin_amdgcn_exp2f(hi), e = fmaf(e0, lo * 0.69314718055994531f, e0);
    const float tail = fmaf(u, p, 0.5f) * e;
    return {v < 0.0f ? tail : 1.0f - tail, e};
}

template <int F>
__device__ __forceinline__ float activate(float v) {
    if constexpr (F == MOE_ACT_SILU) return v * logistic(v).p;
    if constexpr (F == MOE_ACT_GELU) return v * normal(v).cdf;
    if constexpr (F == MOE_ACT_SIGMOID) return logistic(v).p;
    return v;
}
__device__ __forceinline__ float activate(int f, float v) {
    switch (f) {
        case MOE_ACT_SILU: return activate<MOE_ACT_SILU>(v);
        case MOE_ACT_GELU: return activate<MOE_ACT_GELU>(v);
        case MOE_ACT_SIGMOID: return activate<MOE_ACT_SIGMOID>(v);
        default: return v;
    }
}
// f(StepPos<F>{}) for the activation F: one branch, outside the loops over rows, so that the code that runs is short
template <typename Fn>
__device__ __forceinline__ void with_activation(int activation, Fn&& f) {
    switch (activation) {
        case MOE_ACT_SILU: f(StepPos<MOE_ACT_SILU>{}); break;
        case MOE_ACT_GELU: f(StepPos<MOE_ACT_GELU>{}); break;
        case MOE_ACT_SIGMOID: f(StepPos<MOE_ACT_SIGMOID>{}); break;
        default: f(StepPos<MOE_ACT_NONE>{});
    }
}
// the activation's derivative
__device__ __forceinline__ float slope(int f, float v) {
    switch (f) {
        case MOE_ACT_SILU: {
            const Logistic l = logistic(v);
            return l.p * fmaf(v, l.q, 1.0f);
        }
        case MOE_ACT_GELU: {
            const Normal n = normal(v);
            return n.cdf + v * 0.39894228040143268f * n.density;
        }
        case MOE_ACT_SIGMOID: {
            const Logistic l = logistic(v);
            return l.p * l.q;
        }
        default: return 1.0f;
    }
}

// ---------------------------------------------------------------------------------------------
// epilogues of eight consecutive columns of one row
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void store_out8(const ProductArgs& a, void* p, size_t i, const f32x8& v) {
    if (a.out_f32) store_act8((float*)p, i, v);
    else store_act8((uint16_t*)p, i, v);
}
__device__ __forceinline__ f32x8 residual8(const ProductArgs& a, size_t at) {
    return a.out_f32 ? load_act8((const float*)a.residual, at) : load_act8((const uint16_t*)a.residual, at);
}
// bias and r: the columns' bias and residual, or zeros
template <int F>
__device__ __forceinline__ void product_out8(const ProductArgs& a, size_t at, f32x8 v, const f32x8& bias, const f32x8& r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v.v[e] += bias.v[e];
    if (a.pre) store_out8(a, a.pre, at, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v.v[e] = activate<F>(v.v[e]) + r.v[e];
    store_out8(a, a.out, at, v);
}
template <int F>
__device__ __forceinline__ void product_out8(const ProductArgs& a, int i, int j, const f32x8& v) {
    const size_t at = (size_t)i * a.J + j;
    f32x8 bias = {}, r = {};
    if (a.bias) bias = load_act8(a.bias, (size_t)j);
    if (a.residual) r = residual8(a, at);
    product_out8<F>(a, at, v, bias, r);
}
// gate g and up projection u of columns n .. n + 7 of h's row i; a block of 32 columns is in four neighbouring lanes, and
// every lane of them calls this, valid or not
template <int F>
__device__ __forceinline__ void gated_out8(const ProductArgs& a, int i, int n, bool valid, const f32x8& g, const f32x8& u) {
    const int N = a.J / 2;
    if (valid && a.pre) {
        store_out8(a, a.pre, (size_t)i * a.J + n, g);
        store_out8(a, a.pre, (size_t)i * a.J + N + n, u);
    }
    f32x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h.v[e] = activate<F>(g.v[e]) * u.v[e];
    if (a.out_scales) {
        uint8_t scale;
        const uint2 c = mx8_codes(h, quad_max(mx8_amax(h)), &scale);
        if (!valid) return;
        *(uint2*)((uint8_t*)a.out + (size_t)i * N + n) = c;
        if (n % 32 == 0) a.out_scales[(size_t)i * (N / 32) + n / 32] = scale;
    } else if (valid) {
        store_out8(a, a.out, (size_t)i * N + n, h);
    }
}

// ---------------------------------------------------------------------------------------------
// launchers; all return hipGetLastError() of their launches
// ---------------------------------------------------------------------------------------------
// bytes: of an operand's value (2 bf16, 4 fp32, 1 MXFP8); p_kmajor, q_kmajor: stored [k][i], [k][j] (not MXFP8); gated: Q
// holds the gate's rows, then the up projection's.  Chooses a.splits, given a.part with part_bytes(I, J) bytes.
hipError_t launch_product(ProductArgs a, int bytes, bool p_kmajor, bool q_kmajor, bool gated, hipStream_t st);

// few_rows(...) of P, neither operand k-major
hipError_t launch_product_few(const ProductArgs& a, int bytes, bool gated, hipStream_t st);

// Rows of K/32 scale bytes to rows of scale_row(K), filled up with 2^0 (beside codes of zero): scales_p [I], then scales_q
// [J], to `padded`.
hipError_t launch_pad_scales(const uint8_t* scales_p, int I, const uint8_t* scales_q, int J, int K, uint8_t* padded, hipStream_t st);

// MXFP8 [n] as bf16, which holds every code times its scale but for the ends of the range: bits below 2^-133 are rounded off,
// and 2^128 and more is infinite
hipError_t launch_unpack(const uint8_t* codes, const uint8_t* scales, size_t n, uint16_t* values, hipStream_t st);

constexpr int kBiasChunks = 64;   // row chunks of the bias gradient's sums, at most
struct PreGradArgs {
    int T, N;                     // gated: pre and d are [T][2 N]
    int activation, gated;
    const void *dy, *pre;
    void* d;                      // the pre-activations' gradient in bf16 or fp32; or null
    float* bias_part;             // or null: [chunks][N]
    float* d_bias;
};
hipError_t launch_pre_grad(const PreGradArgs& a, bool f32, hipStream_t st);

}  // namespace moe
