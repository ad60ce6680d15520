// Dense products beside the experts, on the bf16 and the scaled FP8 matrix cores:
//
//   out[i][j] = sum_k P[i][k] Q[j][k]  and an epilogue (bias, activation, residual; or gate and up projection
//   multiplied), which serves the forward products (P the tokens, Q the weight), the input's gradient (Q the weight
//   stored k-major) and the weight's gradient (both stored k-major: k runs over the tokens).
//
// An fp32 value becomes three bf16 terms on its way from LDS to the matrix cores (8 + 8 + 8 bits of mantissa), and six
// products of terms are summed in fp32; the three left out are below 2^-24 of the whole.  (The fp32 matrix instructions
// have a sixteenth of bf16's rate: 4096^3 takes 602 us here, 228 TFLOP/s, where their peak is 157.)  An infinity has no
// such terms: a tile with one is summed again by the fp32 matrix instructions.
//
// Roundings: sums and epilogues are fp32; y, pre, h and the gradients are rounded once.  The pre-activations' gradient is
// rounded to the activations' type, so that its two products run at bf16's rate.  MXFP8 sums with bf16 outputs are the
// scaled matrix cores', which cut eight neighbouring products to 2^-13 of the largest: 7 * 2^-13 of sum |x| |w| at most,
// under bf16's half step in a typical sum.
//
// A tile of P and Q advances by 128 bytes of k a step through a ring in LDS, filled by direct loads.  The matrix
// instruction's rows are Q's, so that a lane ends with four consecutive columns of one output row.
#include <type_traits>

#include "dense_tile.h"

namespace moe {

// Place of a k-major tile's 16-byte chunk, as row_key: sixteen lanes read 32 bytes of each of four rows k; of fp32, 64 bytes
// of each of two
template <int FMT, int B>
__device__ __forceinline__ int kmajor_key(int k) {
    return FMT == kF32 ? (k >> 1) & 4 : (((k & 3) << 1) | (k & 8)) & (B / 8 - 1);
}

// gated: of each 64 rows of Q's tile, the first 32 are the gate's of 32 columns of h, the others the up projection's
__device__ __forceinline__ int gated_row(int r) { return (r & ~63) / 2 + (r & 31); }

// Where an operand's next step is.  Scalar state that is moved on by a step at a time, since the products wait for what
// computes their loads' addresses.
struct Walk {
    const uint8_t* at;
    size_t step;
    int unit, left, steps;   // units (bytes of a row; k-major: rows) of a step, and left of the sum

    // the steps [s, end) are walked
    __device__ __forceinline__ void init(const uint8_t* p, size_t step_, int left_, int unit_, int s, int end) {
        step = step_;
        unit = unit_;
        at = p + (size_t)s * step;
        left = left_ - s * unit;
        steps = end - s;
    }
    // units of the step that there are; none past the last step
    __device__ __forceinline__ int here() const { return steps > 0 ? left : 0; }
    __device__ __forceinline__ void next() {
        --steps;
        at += step;
        left -= unit;
    }
};

// One operand's tile of B rows: the lane's share of a step's loads.
template <int FMT, bool KMAJOR, int B, int N, bool GATED>
struct TileLoads {
    static constexpr int ES = kSize<FMT>, C = B * ES / 16;  // chunks of a row k of a k-major tile
    uint32_t off[N];         // from the step's first byte; kNowhere outside the matrix
    size_t upper;            // bytes from the gate's rows to the up projection's
    Walk walk;

    // first: the tile's first row (gated: h column); rows: rows of the matrix; ld: its rows' bytes; K: length of the sum;
    // [s, end): the steps
    __device__ __forceinline__ void init(const uint8_t* p, int first, int rows, int ld, int K, int s, int end, int wave, int lane) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if constexpr (KMAJOR) {
                const int unit = (wave * N + n) * 64 + lane, k = unit / C;
                const int c = (unit % C) ^ kmajor_key<FMT, B>(k);
                off[n] = first + c * (16 / ES) < rows ? (uint32_t)(k * ld + c * 16) : kNowhere;
            } else {
                const int r = (wave * N + n) * 8 + (lane >> 3), c = (lane & 7) ^ row_key(r);
                const int row = GATED ? gated_row(r) : r;
                off[n] = first + row < rows ? (uint32_t)(row * ld + c * 16) : kNowhere;
            }
        }
        upper = (size_t)rows * ld;
        if constexpr (KMAJOR) walk.init(p + (size_t)first * ES, (size_t)ld * kStep<FMT>, K, kStep<FMT>, s, end);
        else walk.init(p + (size_t)first * ld, kStepBytes, K * ES, kStepBytes, s, end);
    }
    // load n of the walk's step; zeros past the end of the sum
    __device__ __forceinline__ void load(int n, uint8_t* lds, int wave, int lane) const {
        int at;
        if constexpr (KMAJOR) at = ((wave * N + n) * 64 + lane) / C;
        else at = ((lane & 7) ^ row_key((wave * N + n) * 8 + (lane >> 3))) * 16;
        load_lds16(GATED && ((wave * N + n) & 4) ? walk.at + upper : walk.at, at < walk.here() ? off[n] : kNowhere,
                   lds + (wave * N + n) * 1024);
    }
};

// rows first + 16 f .. of 32 k from 32 h on
template <bool KMAJOR, int B>
__device__ __forceinline__ pr_bf16x8 fragment(const uint8_t* tile, int first, int f, int h, int lane) {
    const int i = lane & 15, g = lane >> 4;
    pr_bf16x8 r;
    if constexpr (KMAJOR) {
        const int k = 32 * h + 8 * g + (i >> 2);
        const int m = first + f * 16 + (i & 3) * 4;
        pr_i16x4 v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int kk = k + 4 * e;
            const uint8_t* p = tile + kk * (2 * B) + (((m >> 3) ^ kmajor_key<kBf16, B>(kk)) << 4) + (m & 4) * 2;
            v[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) pr_i16x4*)p);
        }
        __builtin_memcpy(&r, v, 16);
    } else {
        const int row = first + f * 16 + i;
        r = *(const pr_bf16x8*)(tile + row * kStepBytes + (((4 * h + g) ^ row_key(row)) << 4));
    }
    return r;
}
// the same of fp32 (a step is one fragment of 32 k)
struct Values {
    float v[8];
};
template <bool KMAJOR, int B>
__device__ __forceinline__ Values fragment_f32(const uint8_t* tile, int first, int f, int lane) {
    const int i = lane & 15, g = lane >> 4, m = first + f * 16 + i;
    Values r;
    if constexpr (KMAJOR) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = 8 * g + e;
            r.v[e] = *(const float*)(tile + k * (4 * B) + (((m >> 2) ^ kmajor_key<kF32, B>(k)) << 4) + (m & 3) * 4);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const pr_f32x4 x = *(const pr_f32x4*)(tile + m * kStepBytes + (((2 * g + h) ^ row_key(m)) << 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) r.v[4 * h + e] = x[e];
        }
    }
    return r;
}
// its three bf16 terms: each the nearest to what the terms before it leave.  Two values at a time, taken back to fp32 as
// bits: from the bf16 values the compiler would round each one a second time.
struct Terms {
    pr_bf16x8 t[3];
};
__device__ __forceinline__ Terms split_terms(Values x) {
    Terms r;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            typedef __bf16 v2 __attribute__((ext_vector_type(2)));
            w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f_t{x.v[2 * e], x.v[2 * e + 1]}, v2));
            if (t < 2) {
                x.v[2 * e] -= __uint_as_float(w[e] << 16);
                x.v[2 * e + 1] -= __uint_as_float(w[e] & 0xffff0000u);
            }
        }
        __builtin_memcpy(&r.t[t], w, 16);
    }
    return r;
}
// acc[f] += the six largest products of terms, the smallest first
__device__ __forceinline__ void multiply_f32(pr_f32x4 (&acc)[4], const Terms (&q)[4], const Terms& p) {
    constexpr int TQ[6] = {2, 0, 1, 1, 0, 0}, TP[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
    for (int n = 0; n < 6; ++n)
#pragma unroll
        for (int f = 0; f < 4; ++f)
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[f].t[TQ[n]], p.t[TP[n]], acc[f], 0, 0, 0);
}

// The steps [first, end) of a workgroup's part of the sum
struct Steps {
    int first, end;
    template <int FMT>
    __device__ __forceinline__ void init(const ProductArgs& a) {
        const int total = (a.K + kStep<FMT> - 1) / kStep<FMT>;
        first = 0;
        end = total;
        if (a.splits > 1) {                                  // (K up to 2^21, the gated block's rows: 32 bits hold the products)
            first = (int)((uint32_t)(blockIdx.y * total) / (uint32_t)a.splits);
            end = (int)((uint32_t)((blockIdx.y + 1) * total) / (uint32_t)a.splits);
        }
    }
};

// One load of 64 rows' scale bytes of a step, the lane's row four of them
struct ScaleLoads {
    uint32_t off;
    const uint8_t* at;
    int steps;
    // rows first + from + lane of a tile from `first` on (gated: rows from + lane of Q's tile)
    template <bool GATED>
    __device__ __forceinline__ void init(const uint8_t* scales, int first, int from, int rows, int K, const Steps& s, int lane) {
        const int ld = scale_row(K), r = from + lane, row = GATED ? gated_row(r) : r;
        off = first + row < rows ? (uint32_t)((row + (GATED && (r & 32) ? rows : 0)) * ld) : kNowhere;
        at = scales + (size_t)first * ld + 4 * (size_t)s.first;
        steps = s.end - s.first;
    }
    // of the n-th step from here
    __device__ __forceinline__ void load(uint8_t* lds, int n = 0) const { load_lds4(at + 4 * n, steps > n ? off : kNowhere, lds); }
    __device__ __forceinline__ void next(int n = 1) {
        at += 4 * n;
        steps -= n;
    }
};

// The lane's share of every load of a tile's step.
template <int FMT, bool PK, bool QK, int BI, int BJ, int W, bool GATED>
struct StepLoads {
    static constexpr bool MX8 = FMT == kMx8;
    static constexpr int NP = BI / 8 / W, NQ = BJ / 8 / W, NS = MX8 ? ((BI + BJ) / 64 + W - 1) / W : 0, PER = NP + NQ + NS;
    static constexpr int PB = BI * kStepBytes, QB = BJ * kStepBytes, BYTES = PB + QB + NS * W * 256;
    static_assert(BI % 64 == 0, "whole loads of scales");
    TileLoads<FMT, PK, BI, NP, false> p;
    TileLoads<FMT, QK, BJ, NQ, GATED> q;
    ScaleLoads sc[NS > 0 ? NS : 1];

    __device__ __forceinline__ void init(const ProductArgs& a, const Steps& s, int i0, int j0, int wave, int lane) {
        const int JH = GATED ? a.J / 2 : a.J;
        p.init(a.p, i0, a.I, a.p_ld, a.K, s.first, s.end, wave, lane);
        q.init(a.q, j0, JH, a.q_ld, a.K, s.first, s.end, wave, lane);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int at = (wave * NS + n) * 64;
            if (at < BI) sc[n].template init<false>(a.p_scales, i0, at, a.I, a.K, s, lane);
            else sc[n].template init<GATED>(a.q_scales, j0, at - BI, at < BI + BJ ? JH : 0, a.K, s, lane);
        }
    }
    // the next step
    __device__ __forceinline__ void load(uint8_t* st, int wave, int lane) {
#pragma unroll
        for (int n = 0; n < NP; ++n) p.load(n, st, wave, lane);
        p.walk.next();
#pragma unroll
        for (int n = 0; n < NQ; ++n) q.load(n, st + PB, wave, lane);
        q.walk.next();
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            sc[n].load(st + PB + QB + (wave * NS + n) * 256);
            sc[n].next();
        }
    }
};

// A wave's sums go through its own LDS, 256 bytes for each row of 64 columns, from where a lane takes eight columns of a
// row, and a store 128 bytes of it.  The 16-byte chunks of a row are exchanged by the row's number, which keeps the writes,
// many rows at once, on different banks.
__device__ __forceinline__ pr_f32x4* sums_chunk(uint8_t* mine, int r, int c) {
    return (pr_f32x4*)(mine + r * 256 + ((c ^ (r & 15)) << 4));
}
// ROWS rows from `row` on and 64 columns from `column` on (gated: 32 columns of h, the gate's and the up projection's)
template <int ROWS, bool GATED>
__device__ __forceinline__ void write_rows(const ProductArgs& a, uint8_t* mine, int row, int column, int lane) {
    constexpr int PER_ROW = GATED ? 4 : 8;                   // lanes of a row
    const int N = GATED ? a.J / 2 : a.J, c = lane % PER_ROW, n = column + 8 * c;
    auto read8 = [&](int r, int c) {
        const pr_f32x4 x = *sums_chunk(mine, r, c), y = *sums_chunk(mine, r, c + 1);
        return f32x8{{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}};
    };
    asm volatile("" ::: "memory");                           // one wave's own writes and reads, in order
    if (a.splits > 1) {
#pragma unroll 2
        for (int r = lane / PER_ROW; r < ROWS; r += 64 / PER_ROW) {
            const int i = row + r;
            if (i >= a.I || n >= N) continue;
            float* sums = a.part + ((size_t)blockIdx.y * a.I + i) * a.J + n;
            store_act8(sums, 0, read8(r, 2 * c));
            if (GATED) store_act8(sums, (size_t)N, read8(r, 8 + 2 * c));
        }
    } else {
        f32x8 bias = {};
        if (!GATED && a.bias && n < N) bias = load_act8(a.bias, (size_t)n);
        with_activation(a.activation, [&](auto f) {
            constexpr int F = decltype(f)::value;
            if constexpr (GATED) {
#pragma unroll 4
                for (int r = lane / PER_ROW; r < ROWS; r += 64 / PER_ROW)
                    gated_out8<F>(a, row + r, n, row + r < a.I && n < N, read8(r, 2 * c), read8(r, 8 + 2 * c));
            } else {
                // four rows at a time, their residuals in flight together
#pragma unroll 1
                for (int r0 = lane / PER_ROW; r0 < ROWS; r0 += 32) {
                    f32x8 res[ROWS < 32 ? ROWS / 8 : 4];
                    constexpr int R = sizeof(res) / sizeof(res[0]);
#pragma unroll
                    for (int u = 0; u < R; ++u) {
                        const int i = row + r0 + 8 * u;
                        res[u] = f32x8{};
                        if (a.residual && i < a.I && n < N) res[u] = residual8(a, (size_t)i * a.J + n);
                    }
#pragma unroll
                    for (int u = 0; u < R; ++u) {
                        const int i = row + r0 + 8 * u;
                        if (i < a.I && n < N) product_out8<F>(a, (size_t)i * a.J + n, read8(r0 + 8 * u, 2 * c), bias, res[u]);
                    }
                }
            }
        });
    }
    asm volatile("" ::: "memory");
}

// Workgroups go to the eight XCDs in turn: an XCD takes a run of tiles, in panels of eight tile rows, so that the tiles
// it works on at once share their operands in its L2.
__device__ __forceinline__ void tile_place(int b, int tiles, int ti, int tj, int* i, int* j) {
    const int x = b & 7, per = tiles >> 3, more = tiles & 7;
    const uint32_t t = x * per + (x < more ? x : more) + (b >> 3);
    const int panel = t / (uint32_t)(8 * tj), r = t - panel * 8 * tj, rows = ti - panel * 8 < 8 ? ti - panel * 8 : 8;
    *j = rows == 8 ? r >> 3 : (int)((uint32_t)r / (uint32_t)rows);
    *i = panel * 8 + r - *j * rows;
}

// scale bytes of four fragments, rows first + 16 f .., for this lane's block
__device__ __forceinline__ int four_scales(const uint8_t* scales, int first, int lane) {
    const uint8_t* p = scales + 4 * (first + (lane & 15)) + (lane >> 4);
    return p[0] | p[64] << 8 | p[128] << 16 | p[192] << 24;
}
// acc[f] += P's fragment FI times Q's fragment f, their scales in byte FI % 4 of ps and f of qs
template <int FI>
__device__ __forceinline__ void multiply_mx8(pr_f32x4 (&acc)[4], const pr_i32x8& p, const pr_i32x8 (&q)[4], int ps, int qs) {
    acc[0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[0], p, acc[0], 0, 0, 0, qs, FI % 4, ps);
    acc[1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[1], p, acc[1], 0, 0, 1, qs, FI % 4, ps);
    acc[2] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[2], p, acc[2], 0, 0, 2, qs, FI % 4, ps);
    acc[3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[3], p, acc[3], 0, 0, 3, qs, FI % 4, ps);
}

// Tile of BI rows and 64 WJ columns; WI x WJ waves, each BI / WI rows by 64 columns.  ST stages.
// Small tiles fill the CUs, two workgroups on one covering each other's waits; what bounds them is a step's chain of
// barrier, LDS reads and products.  bf16, 4096 x 4096: 256 tokens 20.0 us and 4.2 of k_product_finish, 1024 tokens 42.2
// (814 TFLOP/s).  fp32, 333 tokens, 6144 x 2048: 71.5 us and 6.6 (matrix cores 46% busy where there is a workgroup: the
// terms' vector instructions, five for each product, take the other half).  MXFP8 gated, 64 tokens, 8192 x 4096: 14.7
// us a call where the last-level cache holds the weight (69 MB, 4.7 TB/s), 20 and more where it comes from HBM.
template <int FMT, bool PK, bool QK, int BI, int WI, int WJ, int ST, bool GATED>
__global__ __launch_bounds__(64 * WI * WJ) void k_product(ProductArgs a) {
    constexpr int W = WI * WJ, BJ = 64 * WJ, FI = BI / WI / 16, BH = GATED ? BJ / 2 : BJ;
    typedef StepLoads<FMT, PK, QK, BI, BJ, W, GATED> Loads;
    constexpr int STG = Loads::BYTES, PB = Loads::PB, PER = Loads::PER;
    __shared__ __align__(1024) uint8_t ring[ST * STG];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ti = (a.I + BI - 1) / BI, tj = ((GATED ? a.J / 2 : a.J) + BH - 1) / BH;
    int i0, j0;
    tile_place(blockIdx.x, gridDim.x, ti, tj, &i0, &j0);
    i0 *= BI;
    j0 *= BH;
    Steps steps;
    steps.init<FMT>(a);
    const int wi = wave / WJ * (BI / WI), wj = wave % WJ * 64;
    pr_f32x4 acc[FI][4];
    // The tile's sums; exact: fp32 values as they are, in fp32 matrix products.
    auto sums = [&](auto exact) {
        Loads loads;
        loads.init(a, steps, i0, j0, wave, lane);
#pragma unroll
        for (int f = 0; f < FI; ++f)
#pragma unroll
            for (int g = 0; g < 4; ++g) acc[f][g] = pr_f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < ST - 1; ++s) loads.load(ring + s * STG, wave, lane);
        int at = 0;
        for (int s = steps.first; s < steps.end; ++s) {
            wait_vm<(ST - 2) * PER>();
            ring_barrier();
            loads.load(ring + (at == 0 ? ST - 1 : at - 1) * STG, wave, lane);
            const uint8_t* st = ring + at * STG;
            at = at + 1 == ST ? 0 : at + 1;
            if constexpr (FMT == kMx8) {
                pr_i32x8 p[FI], q[4];
                int ps[(FI + 3) / 4];                            // (fewer fragments: the other bytes are not used)
                const int qs = four_scales(st + PB + Loads::QB + 4 * BI, wj, lane);
#pragma unroll
                for (int f = 0; f < (FI + 3) / 4; ++f) ps[f] = four_scales(st + PB + Loads::QB, wi + 64 * f, lane);
#pragma unroll
                for (int f = 0; f < 4; ++f) q[f] = fragment8(st + PB, wj, f, lane);
#pragma unroll
                for (int f = 0; f < FI; ++f) p[f] = fragment8(st, wi, f, lane);
                for_steps<0>([&](auto n) {
                    constexpr int fi = decltype(n)::value;
                    multiply_mx8<fi>(acc[fi], p[fi], q, ps[fi / 4], qs);
                }, std::make_integer_sequence<int, FI>{});
            } else if constexpr (decltype(exact)::value) {
                Values q[4];
#pragma unroll
                for (int f = 0; f < 4; ++f) q[f] = fragment_f32<QK, BJ>(st + PB, wj, f, lane);
#pragma unroll
                for (int fi = 0; fi < FI; ++fi) {
                    const Values p = fragment_f32<PK, BI>(st, wi, fi, lane);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int f = 0; f < 4; ++f) acc[fi][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(q[f].v[e], p.v[e], acc[fi][f], 0, 0, 0);
                }
            } else if constexpr (FMT == kF32) {
                Values pv[FI];
                Terms q[4];
#pragma unroll
                for (int f = 0; f < 4; ++f) q[f] = split_terms(fragment_f32<QK, BJ>(st + PB, wj, f, lane));
#pragma unroll
                for (int fi = 0; fi < FI; ++fi) pv[fi] = fragment_f32<PK, BI>(st, wi, fi, lane);
                Terms p = split_terms(pv[0]);
#pragma unroll
                for (int fi = 0; fi < FI; ++fi) {                // one fragment's products over the next one's terms
                    const Terms now = p;
                    if (fi + 1 < FI) p = split_terms(pv[fi + 1]);
                    multiply_f32(acc[fi], q, now);
#pragma unroll
                    for (int n = 0; n < 24; ++n) {
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x2, 2, 0);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    pr_bf16x8 q[4], p[FI];
#pragma unroll
                    for (int f = 0; f < 4; ++f) q[f] = fragment<QK, BJ>(st + PB, wj, f, h, lane);
#pragma unroll
                    for (int fi = 0; fi < FI; ++fi) p[fi] = fragment<PK, BI>(st, wi, fi, h, lane);
#pragma unroll
                    for (int fi = 0; fi < FI; ++fi)
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            acc[fi][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[f], p[fi], acc[fi][f], 0, 0, 0);
                }
            }
        }
        wait_vm<0>();                                        // no direct load is under way
        ring_barrier();
    };
    sums(StepPos<0>{});
    if constexpr (FMT == kF32) {
        // A value without finite terms (an infinity, or one that bf16 rounds to it) leaves every sum that it enters infinite or
        // NaN, and so does a sum past the type's end: then the tile's sums are taken again, of the values themselves.  (To look at
        // the sums takes 0.2 us at 128 tokens, 1024 x 1024, and 3 of 601 at 4096^3; an infinity in every tile doubles a call's time.)
        float none = 0.0f;
#pragma unroll
        for (int fi = 0; fi < FI; ++fi)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                mfma_results_here(acc[fi][f]);
#pragma unroll
                for (int e = 0; e < 4; ++e) none = fmaf(acc[fi][f][e], 0.0f, none);
            }
        uint32_t* bad = (uint32_t*)ring;
        const bool mine_bad = __ballot(none != 0.0f) != 0;   // (a NaN is unequal to everything)
        if (lane == 0) bad[wave] = mine_bad;
        ring_barrier();
        uint32_t any = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) any |= bad[w];
        ring_barrier();
        if (__builtin_amdgcn_readfirstlane((int)any)) sums(StepPos<1>{});
    }
    constexpr int RF = FI > 4 ? 4 : FI;                      // 16 RF rows at a time
    static_assert(ST * STG >= W * RF * 4096, "the waves' sums fit into the ring");
    uint8_t* mine = ring + wave * RF * 4096;
#pragma unroll
    for (int f0 = 0; f0 < FI; f0 += RF) {
#pragma unroll
        for (int fi = 0; fi < RF; ++fi)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                mfma_results_here(acc[f0 + fi][f]);
                *sums_chunk(mine, fi * 16 + (lane & 15), f * 4 + (lane >> 4)) = acc[f0 + fi][f];
            }
        write_rows<RF * 16, GATED>(a, mine, i0 + wi + f0 * 16, GATED ? j0 + wj / 2 : j0 + wj, lane);
    }
}

// of 32 rows, first + 32 f ..: 16 k from 16 j on
template <bool KMAJOR, int B>
__device__ __forceinline__ pr_bf16x8 fragment32(const uint8_t* tile, int first, int f, int j, int lane) {
    const int g = lane >> 5;
    pr_bf16x8 r;
    if constexpr (KMAJOR) {
        const int i = lane & 15, k = 16 * j + 8 * g + (i >> 2), m = first + f * 32 + (lane & 16) + (i & 3) * 4;
        pr_i16x4 v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int kk = k + 4 * e;
            const uint8_t* p = tile + kk * (2 * B) + (((m >> 3) ^ kmajor_key<kBf16, B>(kk)) << 4) + (m & 4) * 2;
            v[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) pr_i16x4*)p);
        }
        __builtin_memcpy(&r, v, 16);
    } else {
        const int row = first + f * 32 + (lane & 31);
        r = *(const pr_bf16x8*)(tile + row * kStepBytes + (((2 * j + g) ^ row_key(row)) << 4));
    }
    return r;
}

// Half steps of MXFP8: 64 codes of a row, 64 bytes.  Eight lanes, on eight rows, are served at once.
constexpr int kHalfBytes = kStepBytes / 2;
__device__ __forceinline__ int half_key(int r) { return (r >> 1) & 3; }
// of 32 rows, first + 32 f ..: lane group g holds k 16 g .. and 32 + 16 g ..
__device__ __forceinline__ pr_i32x8 fragment8_half(const uint8_t* tile, int first, int f, int lane) {
    const int row = first + f * 32 + (lane & 31), g = lane >> 5;
    const uint4 a = *(const uint4*)(tile + row * kHalfBytes + ((g ^ half_key(row)) << 4));
    const uint4 b = *(const uint4*)(tile + row * kHalfBytes + (((2 + g) ^ half_key(row)) << 4));
    return pr_i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}
// one operand's 256 rows: the lane's share of a half step's loads, four for each of four waves
template <bool GATED>
struct HalfLoads {
    uint32_t off[4];
    size_t upper;
    Walk walk;
    // as TileLoads; [s, end) are half steps, the last of which may lie past the end of the sum
    __device__ __forceinline__ void init(const uint8_t* p, int first, int rows, int ld, int s, int end, int wave, int lane) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int r = (wave * 4 + n) * 16 + (lane >> 2), c = (lane & 3) ^ half_key(r), row = GATED ? gated_row(r) : r;
            off[n] = first + row < rows ? (uint32_t)(row * ld + c * 16) : kNowhere;
        }
        upper = (size_t)rows * ld;
        walk.init(p + (size_t)first * ld, kHalfBytes, ld, kHalfBytes, s, end);
    }
    __device__ __forceinline__ void load(int n, uint8_t* lds, int wave, int lane) const {
        const int at = ((lane & 3) ^ half_key(lane >> 2)) * 16;      // (the key of 16 rows on is the same)
        load_lds16(GATED && (n & 2) ? walk.at + upper : walk.at, at < walk.here() ? off[n] : kNowhere, lds + (wave * 4 + n) * 1024);
    }
};
// the row's four scale bytes, moved so that bytes 0 and 2 are those of the lane group's blocks
__device__ __forceinline__ int scales32(const uint8_t* scales, int first, int f, int lane) {
    return (int)(*(const uint32_t*)(scales + 4 * (first + f * 32 + (lane & 31))) >> (8 * (lane >> 5)));
}

// The sums of four waves' 128 x 128, acc[i][j] of 32 x 32, through LDS and the epilogue.
template <bool GATED>
__device__ __forceinline__ void write_large(const ProductArgs& a, uint8_t* lds, const pr_f32x16 (&acc)[4][4], int i0, int j0, int wave, int lane) {
    wait_vm<0>();                                            // no direct load is under way
    ring_barrier();
    const int wi = wave / 2 * 128, wj = wave % 2 * 128;
    uint8_t* mine = lds + wave * 32768;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int fi = 0; fi < 4; ++fi)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const pr_f32x16& v = acc[fi][2 * c + f];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const pr_f32x4 w = {v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]};
                    mfma_results_here(w);
                    *sums_chunk(mine, fi * 32 + (lane & 31), f * 8 + 2 * e + (lane >> 5)) = w;
                }
            }
        write_rows<128, GATED>(a, mine, i0 + wi, GATED ? j0 + wj / 2 + 32 * c : j0 + wj + 64 * c, lane);
    }
}
__device__ __forceinline__ void clear(pr_f32x16 (&acc)[4][4]) {
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[f][g][e] = 0.0f;
}

// Tile of 256 x 256 for large bf16 products: four waves of 128 x 128, each alone on its SIMD.  A step is four parts of 16 k;
// while the matrix cores work on one, the next one's fragments come from LDS, and the direct loads are handed out between
// the products (a burst of them would hold the products up).  One barrier a step, before its last part: every wave has
// the whole step in registers then, and the next one has landed.  P has two places in LDS, whose loads follow that
// barrier; Q three, and its loads a step more to land.
// 4096^3 112 us (1228 TFLOP/s; dx 116, dw 118), 8192^3 802 us (1370): the matrix cores are busy 81% of its cycles, at a
// clock that falls to 1.6 GHz under the load.
template <bool PK, bool QK, bool GATED>
__global__ __launch_bounds__(256, 1) void k_product_large(ProductArgs a) {
    constexpr int B = 256, BH = GATED ? B / 2 : B, TB = B * kStepBytes, QS = 3, QAT = 2 * TB;
    __shared__ __align__(1024) uint8_t lds[QAT + QS * TB];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int JH = GATED ? a.J / 2 : a.J;
    int i0, j0;
    tile_place(blockIdx.x, gridDim.x, (a.I + B - 1) / B, (JH + BH - 1) / BH, &i0, &j0);
    i0 *= B;
    j0 *= BH;
    Steps steps;
    steps.init<kBf16>(a);
    TileLoads<kBf16, PK, B, 8, false> lp;
    TileLoads<kBf16, QK, B, 8, GATED> lq;
    lp.init(a.p, i0, a.I, a.p_ld, a.K, steps.first, steps.end, wave, lane);
    lq.init(a.q, j0, JH, a.q_ld, a.K, steps.first, steps.end, wave, lane);
    const int wi = wave / 2 * 128, wj = wave % 2 * 128;
    pr_f32x16 acc[4][4];
    clear(acc);
    // the places where the next loads go, and of the step that is read
    int p_to = 0, q_to = QAT, p_at = 0, q_at = QAT;
    auto q_after = [](int q) { return q == QAT + (QS - 1) * TB ? QAT : q + TB; };
    auto load_p = [&](int n) { lp.load(n, lds + p_to, wave, lane); };
    auto load_q = [&](int n) { lq.load(n, lds + q_to, wave, lane); };
    auto p_next = [&] {
        p_to ^= TB;
        lp.walk.next();
    };
    auto q_next = [&] {
        q_to = q_after(q_to);
        lq.walk.next();
    };
    pr_bf16x8 p[2][4], q[2][4];
    // fragment n of part j: Q's, then P's
    auto read = [&](int j, int n) {
        if (n < 4) q[j & 1][n] = fragment32<QK, B>(lds + q_at, wj, n, j, lane);
        else p[j & 1][n - 4] = fragment32<PK, B>(lds + p_at, wi, n - 4, j, lane);
    };
    auto multiply = [&](int j, int n) {                      // products 2 n and 2 n + 1 of a part
#pragma unroll
        for (int f = n % 2 * 2; f < n % 2 * 2 + 2; ++f)
            acc[n / 2][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[j & 1][f], p[j & 1][n / 2], acc[n / 2][f], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto load_all = [&](bool with_p, bool with_q) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            if (with_p) load_p(n);
            if (with_q) load_q(n);
        }
        if (with_p) p_next();
        if (with_q) q_next();
    };
    load_all(true, true);
    load_all(false, true);
    load_all(true, false);
    wait_vm<16>();
    ring_barrier();
#pragma unroll
    for (int n = 0; n < 8; ++n) read(0, n);
    for (int s = steps.first; s < steps.end; ++s) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n < 4) {
                    read(j + 1, 2 * n);
                    read(j + 1, 2 * n + 1);
                }
                if (j == 0) load_q(n);
                multiply(j, n);
            }
            if (j == 0) q_next();
        }
        wait_vm<8>();
        __builtin_amdgcn_sched_barrier(0);
        ring_barrier();
        __builtin_amdgcn_sched_barrier(0);
        p_at ^= TB;
        q_at = q_after(q_at);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            if (n < 4) {
                read(0, 2 * n);
                read(0, 2 * n + 1);
            }
            load_p(n);
            multiply(3, n);
        }
        p_next();
    }
    write_large<GATED>(a, lds, acc, i0, j0, wave, lane);
}

// The same tile of MXFP8, in half steps of 64 codes with four places in LDS.  While the matrix cores work on half step h,
// fragments of h + 1 come from LDS and loads of h + 4 go to the place of h, which every wave has in registers; one barrier
// at its end, by when h + 2 has landed: a load has two to three half steps for that.  Scales are loaded for four steps
// at a time: each load of them touches a line for every row, and step by step the lines' way through L2 took as long as
// the operands' (8192^3 600 us so, 534 now).
// 4096 x 4096 x 8192 136 us (2020 TFLOP/s; two whole steps in LDS, whose loads have half a step to land, 145), 8192^3 517
// (2130): counters show the matrix cores busy for 46% of either's cycles, and 4.5 vector instructions for each matrix one; the
// scales' lines, one for each row, are the likely rest.  Rows that end inside a line cost more than that: 4096 x 8224 180 us.
template <bool GATED>
__global__ __launch_bounds__(256, 1) void k_product_large_mx8(ProductArgs a) {
    constexpr int B = 256, BH = GATED ? B / 2 : B, TB = B * kHalfBytes, STG = 2 * TB, SAT = 4 * STG, SB = 8 * B;
    __shared__ __align__(1024) uint8_t lds[SAT + 8 * SB];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int JH = GATED ? a.J / 2 : a.J;
    int i0, j0;
    tile_place(blockIdx.x, gridDim.x, (a.I + B - 1) / B, (JH + BH - 1) / BH, &i0, &j0);
    i0 *= B;
    j0 *= BH;
    Steps steps;
    steps.init<kMx8>(a);
    HalfLoads<false> lp;
    HalfLoads<GATED> lq;
    ScaleLoads ls[2];
    lp.init(a.p, i0, a.I, a.p_ld, 2 * steps.first, 2 * steps.end, wave, lane);
    lq.init(a.q, j0, JH, a.q_ld, 2 * steps.first, 2 * steps.end, wave, lane);
    ls[0].init<false>(a.p_scales, i0, wave * 64, a.I, a.K, steps, lane);
    ls[1].init<GATED>(a.q_scales, j0, wave * 64, JH, a.K, steps, lane);
    const int wi = wave / 2 * 128, wj = wave % 2 * 128;
    pr_f32x16 acc[4][4];
    clear(acc);
    int to = 0, s_to = 0, at = 0, s_at = 0;              // the places of the next loads, and of the next reads
    auto load = [&](int n) {
        if (n < 4) lp.load(n, lds + to, wave, lane);
        else lq.load(n - 4, lds + to + TB, wave, lane);
    };
    auto load_scales = [&] {                                 // of four steps
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int u = 0; u < 4; ++u) ls[n].load(lds + SAT + s_to + u * SB + n * 4 * B + wave * 256, u);
            ls[n].next(4);
        }
        s_to ^= 4 * SB;
    };
    auto next = [&] {
        to = (to + STG) & (4 * STG - 1);
        lp.walk.next();
        lq.walk.next();
    };
    pr_i32x8 p[2][4], q[2][4];
    int ps[4], qs[4], ps_next[4], qs_next[4];
    auto read = [&](int j, int n) {                          // fragment n of half j: Q's, then P's
        if (n < 4) q[j][n] = fragment8_half(lds + at + TB, wj, n, lane);
        else p[j][n - 4] = fragment8_half(lds + at, wi, n - 4, lane);
    };
    auto read_scales = [&](int f) {
        ps_next[f] = scales32(lds + SAT + s_at, wi, f, lane);
        qs_next[f] = scales32(lds + SAT + s_at + 4 * B, wj, f, lane);
    };
    auto take_scales = [&] {
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            ps[f] = ps_next[f];
            qs[f] = qs_next[f];
        }
        s_at = (s_at + SB) & (8 * SB - 1);
    };
    static_assert((4 * STG & (4 * STG - 1)) == 0 && (8 * SB & (8 * SB - 1)) == 0, "places by a mask");
    load_scales();
    for (int h = 0; h < 4; ++h) {
#pragma unroll
        for (int n = 0; n < 8; ++n) load(n);
        next();
    }
    wait_vm<16>();                                           // the first two half steps
    ring_barrier();
#pragma unroll
    for (int n = 0; n < 8; ++n) read(0, n);
#pragma unroll
    for (int f = 0; f < 4; ++f) read_scales(f);
    take_scales();
    at = STG;
    ring_barrier();
    for (int s = steps.first; s < steps.end; ++s) {
        for_steps<0>([&](auto half) {
            constexpr int j = decltype(half)::value;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n < 4) {
                    read(j ^ 1, 2 * n);
                    read(j ^ 1, 2 * n + 1);
                }
                load(n);
                if (j == 0 && n == 7 && (s - steps.first) % 4 == 0) load_scales();
                if (j == 1 && n >= 4) read_scales(n - 4);
#pragma unroll
                for (int f = n % 2 * 2; f < n % 2 * 2 + 2; ++f) {
                    pr_f32x16& c = acc[n / 2][f];
                    c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(q[j][f], p[j][n / 2], c, 0, 0, 2 * j, qs[f], 2 * j, ps[n / 2]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            next();
            at = (at + STG) & (4 * STG - 1);
            if (j == 1) take_scales();
            wait_vm<16>();                                   // at most this half step's loads and the one's before are under way
            __builtin_amdgcn_sched_barrier(0);
            ring_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }, std::make_integer_sequence<int, 2>{});
    }
    write_large<GATED>(a, lds, acc, i0, j0, wave, lane);
}

// the parts' sums in order, then the epilogue; eight columns per thread (gated: of h).  Out of L2 and the last-level
// cache: 4.2 us for 256 tokens, 4096 columns, two parts; 6.7 for 333 tokens, 6144 columns, three.
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
    with_activation(a.activation, [&](auto f) {
        constexpr int F = decltype(f)::value;
        // (with 8-bit outputs N is a multiple of 32, so a block's four lanes are a quad)
        if constexpr (GATED) gated_out8<F>(a, i, n, valid, sum(n), sum(N + n));
        else if (valid) product_out8<F>(a, i, n, sum(n));
    });
}

template <int FMT, bool PK, bool QK, bool GATED, int BI, int WI, int WJ, int ST>
static void product_launch_as(const ProductArgs& a, hipStream_t st) {
    const int JH = GATED ? a.J / 2 : a.J, BH = GATED ? 32 * WJ : 64 * WJ, tiles = (a.I + BI - 1) / BI * ((JH + BH - 1) / BH);
    MOE_LAUNCH((k_product<FMT, PK, QK, BI, WI, WJ, ST, GATED>), dim3(tiles, a.splits), dim3(64 * WI * WJ), 0, st, a);
}

template <int FMT, bool PK, bool QK, bool GATED>
static void product_launch(ProductArgs& a, hipStream_t st) {
    switch (choose_tile(a.I, a.J, a.K, FMT, &a.splits)) {
        case 0: product_launch_as<FMT, PK, QK, GATED, 64, 4, 1, 4>(a, st); break;
        case 1: product_launch_as<FMT, PK, QK, GATED, 64, 2, 2, 3>(a, st); break;
        case 2: product_launch_as<FMT, PK, QK, GATED, 128, 2, 4, 3>(a, st); break;
        default:
            if constexpr (FMT == kF32) {
                product_launch_as<FMT, PK, QK, GATED, 256, 2, 4, 2>(a, st);
            } else {
                const int JH = GATED ? a.J / 2 : a.J, BH = GATED ? 128 : 256, tiles = (a.I + 255) / 256 * ((JH + BH - 1) / BH);
                if constexpr (FMT == kMx8) MOE_LAUNCH((k_product_large_mx8<GATED>), dim3(tiles, a.splits), dim3(256), 0, st, a);
                else MOE_LAUNCH((k_product_large<PK, QK, GATED>), dim3(tiles, a.splits), dim3(256), 0, st, a);
            }
    }
}
template <int FMT>
static void product_launch(ProductArgs& a, bool p_kmajor, bool q_kmajor, bool gated, hipStream_t st) {
    if (gated) {
        product_launch<FMT, false, false, true>(a, st);
        return;
    }
    if constexpr (FMT != kMx8) {
        if (p_kmajor) {
            product_launch<FMT, true, true, false>(a, st);
            return;
        }
        if (q_kmajor) {
            product_launch<FMT, false, true, false>(a, st);
            return;
        }
    }
    product_launch<FMT, false, false, false>(a, st);
}

hipError_t launch_product(ProductArgs a, int bytes, bool p_kmajor, bool q_kmajor, bool gated, hipStream_t st) {
    trace("product", 0, st);
    if (bytes == 2) product_launch<kBf16>(a, p_kmajor, q_kmajor, gated, st);
    else if (bytes == 4) product_launch<kF32>(a, p_kmajor, q_kmajor, gated, st);
    else product_launch<kMx8>(a, p_kmajor, q_kmajor, gated, st);
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

// Four bytes of a row per thread, 3.3 us for a token and 4096 rows of 129 bytes.  Direct loads to LDS take whole aligned
// words, which rows of K/32 bytes are not made of unless K is a multiple of 128.  2.5 us of a call: 4096 x 4128, one token
// 10.3 us, 4096 x 4096 7.6.
__global__ __launch_bounds__(256) void k_pad_scales(const uint8_t* __restrict__ scales_p, const uint8_t* __restrict__ scales_q, int I, int J,
                                                    int blocks, uint32_t* __restrict__ padded) {
    const int words = (blocks + 3) / 4;
    const size_t all = (size_t)(I + J) * words;
    for (size_t at = (size_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (size_t)gridDim.x * 256) {
        const int row = (int)(at / words), b = (int)(at % words) * 4;
        const uint8_t* from = row < I ? scales_p + (size_t)row * blocks : scales_q + (size_t)(row - I) * blocks;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= (uint32_t)(b + e < blocks ? from[b + e] : 127) << (8 * e);
        padded[at] = w;
    }
}

hipError_t launch_pad_scales(const uint8_t* scales_p, int I, const uint8_t* scales_q, int J, int K, uint8_t* padded, hipStream_t st) {
    const size_t blocks = ((size_t)(I + J) * (scale_row(K) / 4) + 255) / 256;
    trace("pad_scales", 0, st);
    MOE_LAUNCH(k_pad_scales, dim3((uint32_t)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, scales_p, scales_q, I, J, K / 32,
               (uint32_t*)padded);
    trace("pad_scales", 1, st);
    return hipGetLastError();
}

// MXFP8 to bf16, for products whose sums have to be right to fp32.  A scale byte b stands for 2^(b - 127); codes of blocks
// under 2^-117 that pass bf16's smallest number are rounded.  A stream of three bytes a code.
__global__ __launch_bounds__(256) void k_unpack(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, size_t n,
                                                uint16_t* __restrict__ values) {
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (size_t)gridDim.x * 2048) {
        const uint2 c = *(const uint2*)(codes + i);
        const float sc = mx8_scale(scales[i / 32]);
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
}

hipError_t launch_unpack(const uint8_t* codes, const uint8_t* scales, size_t n, uint16_t* values, hipStream_t st) {
    trace("unpack", 0, st);
    const size_t blocks = (n / 8 + 255) / 256;
    MOE_LAUNCH(k_unpack, dim3((uint32_t)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, codes, scales, n, values);
    trace("unpack", 1, st);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// gradient of the pre-activations, rounded for the products behind it, and its column sums in fp32 before that
// rounding (the bias's gradient: row chunks apart, then added in order).  A workgroup takes 256 columns, 32 threads
// of eight, and every eighth row of its chunk per thread row.  A stream: gated, 4096 x 8192, bf16, 336 MB in 59 us (5.7
// TB/s); fp32, 777 x 1536, 8.3 us.  Formed inside the products instead, it would be computed again for every tile that
// reads it, 16 and 64 times here.  With a bias's gradient, 4096 x 4096, bf16, GELU: 31 us (100 MB at 3.2 TB/s, in 1024
// workgroups of serial sums), and 20 for the 64 chunks' sums, sixteen workgroups that wait for one load after another.
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
                store_act8((XT*)a.d, at, d);
                if constexpr (GATED) store_act8((XT*)a.d, at + a.N, du);
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
    int chunks = a.bias_part ? (a.T + 31) / 32 : (a.T + 7) / 8;
    const int most = a.bias_part ? kBiasChunks : 1024;
    if (chunks > most) chunks = most;
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
