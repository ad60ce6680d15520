// Device pieces of the dense products' kernels: types, direct loads to LDS, and fragments.
#pragma once

#include "dense.h"

namespace moe {

typedef __bf16 pr_bf16x8 __attribute__((ext_vector_type(8)));
typedef float pr_f32x4 __attribute__((ext_vector_type(4)));
typedef float pr_f32x16 __attribute__((ext_vector_type(16)));
typedef int pr_i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t pr_u32x4 __attribute__((ext_vector_type(4)));
typedef short pr_i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t* pr_lds_t;

constexpr int kStepBytes = 128;              // of a row and step: 64 bf16, 128 codes
constexpr uint32_t kNowhere = 0x80000000u;   // past every descriptor's end: a load from there brings zeros
// A row is 2^23 bytes long at most (2^21 fp32 values of the gated block's gradient), and a tile's last row is its 256th: every
// offset from a tile's first byte stays below the descriptors' 2^31 - 1 bytes.
static_assert(255ull * (1 << 23) + kStepBytes < 0x7fffffffu, "offsets in a tile");

// values of a step, bytes of a value
template <int FMT>
constexpr int kStep = FMT == kBf16 ? 64 : FMT == kF32 ? 32 : 128;
template <int FMT>
constexpr int kSize = kStepBytes / kStep<FMT>;
static_assert(kStep<kBf16> == kFormats[kBf16].step && kStep<kF32> == kFormats[kF32].step && kStep<kMx8> == kFormats[kMx8].step,
              "the rule counts the kernels' steps");

// Direct loads to LDS: 16 (4) bytes per lane from base + off, lane l's to lds + 16 l (4 l); an offset past the descriptor's
// end brings zeros.  In assembly, because the compiler has every transposing read of LDS wait for all direct loads that
// it knows of; they have no result in registers, and are waited for by count (wait_vm).
__device__ __forceinline__ pr_u32x4 load_rsrc(const uint8_t* base) {
    const uint64_t p = (uint64_t)base;                       // the same in every lane
    return pr_u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                    (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32)) & 0xffffu, 0x7fffffffu, 0x00020000u};
}
// (m0 is reserved: the compiler sets it right before each use of its own, and warns of its name among what is overwritten)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t off, uint8_t* lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"((uint32_t)(uintptr_t)(pr_lds_t)lds),
                 "v"(off), "s"(load_rsrc(base)) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(const uint8_t* base, uint32_t off, uint8_t* lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"((uint32_t)(uintptr_t)(pr_lds_t)lds),
                 "v"(off), "s"(load_rsrc(base)) : "memory", "m0");
}
#pragma clang diagnostic pop

// Place of a row's 16-byte chunk in LDS: chunk ^ key(row).  Eight lanes, on eight rows, are served at once, from 32 banks.
__device__ __forceinline__ int row_key(int r) { return r & 7; }
// of 128 codes: lane group g holds k 16 g .. and 64 + 16 g ..
__device__ __forceinline__ pr_i32x8 fragment8(const uint8_t* tile, int first, int f, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const int row = first + f * 16 + i;
    const uint4 a = *(const uint4*)(tile + row * kStepBytes + ((g ^ row_key(row)) << 4));
    const uint4 b = *(const uint4*)(tile + row * kStepBytes + (((4 + g) ^ row_key(row)) << 4));
    return pr_i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

}  // namespace moe
