// Which kernel a dense product runs in: rules on its sizes, in plain C++, so that a host test can hold its sizes against them.
#pragma once

#include <stddef.h>

namespace moe {

// formats of the operands, as the kernels number them
enum { kBf16 = 0, kF32 = 1, kMx8 = 2 };

// Few rows of P, neither operand k-major: k_product_few.  Up to kFewTokens every product; beyond, up to 64, by rule.  Each
// workgroup reads all tokens again for each of its 16 F rows of the weight, which up to 32 tokens hides behind the weight's own
// bytes.  Beyond, tiles of 64 tokens win once they fill the CUs.  us, this kernel and the tiles, 64 tokens, bf16,
// 4096 columns: 4096 rows 10.6, 14.0; 16384 rows 56, 37.  fp32 stays here (1024 x 1024: 9, 22: no terms, no parts).  A
// block of 32 outputs in MXFP8 (h8) needs four fragments of rows, for which LDS has no room with more than 32 tokens.
constexpr int kFewTokens = 32;
inline bool few_rows(int I, int J, int format, bool h8) {
    if (I <= kFewTokens) return true;
    if (I > 64 || h8) return false;
    return format == kF32 || J <= 6144;
}

// bytes for the parts' sums
constexpr size_t kPartBytes = (size_t)64 << 20;
constexpr int kMostSplits = 16;
inline size_t part_bytes(size_t I, size_t J) {
    const size_t all = kMostSplits * I * J * 4;
    return all < kPartBytes ? all : kPartBytes;
}

// Which tile, and how many parts of the sum: the least time by a model of each tile's own measurements.  A workgroup takes
// `start` and `step` for each 128 bytes of k, `step2` where two share a CU; parts cost a second kernel, that adds them.
// us, model and measured (bf16): 256 tokens, 4096 x 4096 64 x 128 in two parts 21, 21.6 (128 x 256 26); 1024 tokens 64 x 128
// 42, 42.0 (128 x 256 48); 2048 tokens 128 x 256 64, 64.1 (64 x 128 80); 4096 tokens 256 x 256 106, 110 (128 x 256 125);
// 512 tokens, 1024 x 1024 64 x 64 9.4, 9.3 (64 x 128 9.8).  Steps of fp32 and MXFP8 are taken to be longer by one factor each:
// fp32, 333 tokens, 6144 x 2048 128 x 256 in three parts 70, 72; MXFP8, 256 tokens, 4096 x 4096 64 x 64 16.2, 16.1 (kernel),
// 4096 tokens, 4096 x 8192 256 x 256 140, 136.
struct TileChoice {
    int bi, bj, per_cu;
    float start, step, step2;
};
static const TileChoice kTiles[] = {
    {64, 64, 2, 5.4f, 0.25f, 0.42f}, {64, 128, 2, 5.7f, 0.32f, 0.57f}, {128, 256, 1, 5.2f, 0.92f, 0.92f}, {256, 256, 1, 6.2f, 1.55f, 1.55f}};
static constexpr struct {
    int step;                     // values of 128 bytes
    float slower;
} kFormats[] = {{64, 1.0f}, {32, 2.9f}, {128, 1.35f}};

inline int choose_tile(int I, int J, int K, int format, int* parts) {
    const int steps = (K + kFormats[format].step - 1) / kFormats[format].step;
    float least = 0.0f;
    int best = -1;
    for (int t = 0; t < 4; ++t) {
        const TileChoice& c = kTiles[t];
        const long long tiles = (long long)((I + c.bi - 1) / c.bi) * ((J + c.bj - 1) / c.bj);
        for (int splits = 1; splits <= kMostSplits; ++splits) {
            const size_t part = (size_t)splits * I * J * 4;
            if (splits > 1 && (splits * 4 > steps || part > part_bytes(I, J) || tiles * splits > 256 * c.per_cu)) break;
            const long long groups = tiles * splits, rounds = (groups + 256 * c.per_cu - 1) / (256 * c.per_cu);
            const float step = (groups <= 256 ? c.step : c.step2) * kFormats[format].slower;
            float us = rounds * (steps / (float)splits) * step + c.start * (rounds < 2 ? 1.0f : 0.5f + 0.5f * rounds);
            if (splits > 1) us += 4.0f + part * 1.5e-7f;
            if (best < 0 || us < least) {
                least = us;
                best = t;
                *parts = splits;
            }
        }
    }
    return best;
}

}  // namespace moe
