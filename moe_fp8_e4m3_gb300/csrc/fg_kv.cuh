// fg_kv.cuh - the 4-bit key/value cache: where an element stands, and the device codes of the
// calls around it.
//
// A cache of one kind (keys or values) is codes [pages][heads][page_size][D / 2] and scales
// [pages][heads][page_size][D / 32]: a row holds one token of one head.  With B = D / 32 blocks of 32
// elements, element 32 b + 8 c + j of a key is nibble (c B + b) 8 + j of its row, element
// 32 b + 4 g + j of a value is nibble (g B + b) 4 + j (nibble 2i: bits 0-3 of byte i).  So the lane that
// holds column group c (keys) or row group g (values) of a tensor-core operand finds its codes of
// every block side by side, in one load.
#pragma once

#include <cuda_fp4.h>
#include <cstdint>

#include "fg_ptx.cuh"

namespace fg {

enum : int {
    kKvErrPages = 0x107,        // block tables: lengths, pages or free list
    kKvErrSlot = 0x108,         // a slot outside the cache
    kKvErrPosition = 0x109,     // a position outside the rotation table
    kKvErrAttention = 0x10A,    // attention: query_start, seq_lens or a page outside their range
};

__device__ __forceinline__ void kv_record(int* status, int code) { atomicCAS(status, 0, code); }

// Scales stay within 2^-64 and 2^63, so that a product of two of them, and of a scale and a weight, stays
// finite in FP32.
constexpr int kKvMinExp = -64, kKvMaxExp = 63;

// Value of a UE8M0 byte (0 stands for 0 here: 2^-127 is below everything a cache holds).
__device__ __forceinline__ float ue8m0(uint32_t u) { return __uint_as_float(u << 23); }

// Eight E2M1 codes to four FP16 pairs, exactly; pair i holds codes 2i (low) and 2i + 1.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}

}  // namespace fg
