// Declarations of the operators around the experts (sort.hip, norm.hip, linear.hip): row accesses, the walk
// over a token's picks, and the launchers.
#pragma once

#include "moe_internal.h"

namespace moe {

template <int CTRL, int ROWMASK>
__device__ __forceinline__ float dpp_add_f32(float v) {
    return v + __uint_as_float(dpp_u32<CTRL, ROWMASK>(0u, __float_as_uint(v)));
}

// sum over the 64 lanes of a wave in fp32, returned in every lane (wave_sum_f64's order)
__device__ __forceinline__ float wave_sum_f32(float v) {
    v = dpp_add_f32<kDppXor1, 0xF>(v);
    v = dpp_add_f32<kDppXor2, 0xF>(v);
    v = dpp_add_f32<kDppHalfMirror, 0xF>(v);
    v = dpp_add_f32<kDppMirror, 0xF>(v);
    v = dpp_add_f32<kDppBcast15, 0xA>(v);
    v = dpp_add_f32<kDppBcast31, 0xC>(v);
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// eight consecutive activations at a multiple of eight, as one or two 16-byte accesses (the hardware's
// bf16 conversion rounds to nearest even and keeps NaN).  NT: a non-temporal access, for arrays that
// are larger than the caches (kStreamBytes) and touched once.
struct f32x8 {
    float v[8];
};
template <bool NT>
__device__ __forceinline__ u32x4_t load16(const void* p) {
    if constexpr (NT) return __builtin_nontemporal_load((const u32x4_t*)p);
    else return *(const u32x4_t*)p;
}
template <bool NT>
__device__ __forceinline__ void store16(void* p, u32x4_t v) {
    if constexpr (NT) __builtin_nontemporal_store(v, (u32x4_t*)p);
    else *(u32x4_t*)p = v;
}
// as loaded, until the values are wanted
template <typename XT>
struct Raw8 {
    u32x4_t w[sizeof(XT) / 2];
    __device__ __forceinline__ void clear() {
        for (auto& q : w) q = u32x4_t{0, 0, 0, 0};
    }
    template <bool NT = false>
    __device__ __forceinline__ void load(const XT* p, size_t i) {
        w[0] = load16<NT>(p + i);
        if constexpr (sizeof(XT) == 4) w[1] = load16<NT>(p + i + 4);
    }
    __device__ __forceinline__ f32x8 values() const {
        f32x8 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(XT) == 4) {
                r.v[j] = __uint_as_float(w[0][j]);
                r.v[4 + j] = __uint_as_float(w[1][j]);
            } else {
                r.v[2 * j] = __uint_as_float(w[0][j] << 16);
                r.v[2 * j + 1] = __uint_as_float(w[0][j] & 0xffff0000u);
            }
        }
        return r;
    }
};
template <bool NT = false, typename XT>
__device__ __forceinline__ f32x8 load_act8(const XT* p, size_t i) {
    Raw8<XT> r;
    r.template load<NT>(p, i);
    return r.values();
}
template <bool NT = false, typename XT>
__device__ __forceinline__ void store_act8(XT* p, size_t i, const f32x8& r) {
    u32x4_t w[sizeof(XT) / 2];
    if constexpr (sizeof(XT) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j / 4][j % 4] = __float_as_uint(r.v[j]);
        store16<NT>(p + i + 4, w[1]);
    } else {
        typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
        bf16x8 b;
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = (__bf16)r.v[j];
        __builtin_memcpy(&w[0], &b, 16);
    }
    store16<NT>(p + i, w[0]);
}
// Bytes of an expert-side array from which the dispatch's and the gradients' rows go past the caches: the last-level
// cache's size.  Below it the next kernel finds them there: 128 MB (2048 tokens, d 4096, 8 picks, bf16) dispatched
// and read again 53 us, past the caches 63.  Above it, d 4096, us, past the caches and through them: dispatch of 256 MB 55,
// 58, with a matrix product behind it 164, 181 (512 MB 108, 119 and 325, 341); its gradient 50, 59, behind a kernel
// that writes the rows 124, 130 (512 MB 100, 117 and 258, 297; fp32 256 MB 59, 60 and 148, 135, 512 MB 117, 116 and 281, 296);
// the combine's gradient 116, 129, with a reader of d_o 167, 174 (2 GB 867, 894 and 1220, 1242).
constexpr size_t kStreamBytes = (size_t)256 << 20;

// A token's picks in rank order, in groups whose rows are loaded together: f(N, row, has, j0) with N = MAXN
// (8 or 4), half or a quarter of it (at least 2) picks j0 .. j0 + N - 1 (a StepPos).  pos: the token's k
// positions, the same in every lane of the wave; positions outside [0, P) have no row.  Dropped picks are
// the last ranks, so the groups end with the last pick that has one; a pick without a row inside a group
// (has false) stands on another pick's row, which it reads from the cache and must not use.  The positions
// themselves are waited for one after the other, before the first row is requested.
template <int MAXN, typename F>
__device__ __forceinline__ void for_picks(const int32_t* __restrict__ pos, int k, int P, F&& f) {
    for (int j0 = 0; j0 < k; j0 += MAXN) {
        int row[MAXN], last = -1, any = 0;
        bool has[MAXN];
#pragma unroll
        for (int i = 0; i < MAXN; ++i) {
            row[i] = __builtin_amdgcn_readfirstlane(pos[j0 + i < k ? j0 + i : k - 1]);
            has[i] = j0 + i < k && (unsigned)row[i] < (unsigned)P;
            if (has[i]) {
                last = i;
                any = row[i];
            }
        }
#pragma unroll
        for (int i = 0; i < MAXN; ++i) row[i] = has[i] ? row[i] : any;
        if (MAXN > 4 && last >= 4) f(StepPos<MAXN>{}, row, has, j0);
        else if (last >= 2) f(StepPos<4>{}, row, has, j0);
        else if (last >= 0) f(StepPos<2>{}, row, has, j0);
    }
}

// ---------------------------------------------------------------------------------------------
// launchers; all return hipGetLastError() of their launches
// ---------------------------------------------------------------------------------------------
hipError_t launch_dispatch(const moe_shape* s, const void* x, int T, const int32_t* pick_pos, void* xs,
                           hipStream_t st);
hipError_t launch_dispatch_backward(const moe_shape* s, const void* dxs, int T, const int32_t* pick_pos, void* dx,
                                    hipStream_t st);
hipError_t launch_combine_backward(const moe_shape* s, const void* dy, const float* o, const float* w,
                                   const int32_t* pick_pos, int T, float* d_o, float* d_w, hipStream_t st);

constexpr int kNormMaxD = 16384;
struct NormArgs {
    int T, d;
    const void* x;
    const void* y;            // or null; in the fused combine, o, w and pick_pos stand for it
    const float* o;
    const float* w;
    const int32_t* pick_pos;
    int k, shared;
    float scaling;
    const float* post;        // or null
    const float* pre;         // or null
    const void* gate;         // or null
    int gate_kind;
    float alpha, eps;         // residual scale, eps
    void* x_out;              // or null
    void* normed;             // or null
};
hipError_t launch_block_norm(const moe_shape* s, const NormArgs& a, hipStream_t st);   // a.o: fused with the combine

struct NormGradArgs {
    const void* d_x_out;      // or null
    const void* d_normed;     // or null
    void* dx;                 // outputs: each may be null
    void* dy;
    void* d_gate;
    float* d_post;
    float* d_pre;
    float* part;              // [groups][2][d] in the workspace
};
// groups of rows whose parameter gradients are summed apart, at most, for up to T tokens
int norm_grad_groups_most(const moe_shape* s, int T);
hipError_t launch_block_norm_backward(const moe_shape* s, const NormArgs& a, const NormGradArgs& g, hipStream_t st);

constexpr int kLinearMaxT = 64;
hipError_t launch_linear(const moe_matrix* m, const uint8_t* q, const uint8_t* s, float ts, const void* x, int T,
                         const float* bias, void* y, hipStream_t st);

}  // namespace moe
