// sv_kv8.cuh -- the 8-bit paged cache: its byte layout, and what its append, read and attention share.
//
// Layout of one page and head, for P slots of D dimensions (see spec_serve.h):
//   keys    P D codes, values P D codes: code d of slot t in byte t / 8 * 8 D + d / 16 * 128 + t % 8 * 16 + d % 16.
//           Eight slots by 16 bytes are 128 contiguous bytes, the unit from which the fifth-generation tensor cores
//           read 8-bit operands without a swizzle: the keys as a K-major operand (slots are rows), the values
//           as an M-major one (dimensions are rows), both as they lie in memory.  Copies into shared memory are plain.
//   blocks  16 bytes for each 16 slots: a word for the keys, one for the values, 8 unused bytes.  A word's upper half is the scale
//           as a bfloat16 (a power of two), bit t % 16 of its lower half says that slot t's vector is held as NaN.
#pragma once

#include "sv_kv.cuh"

namespace sv {

constexpr int kKv8Block = 16;                      // slots that share a scale
constexpr int kKv8Least = -40, kKv8Most = 40;      // exponents of scales
constexpr int kKv8Top = 8;                         // the largest code of a block is in 2^7 .. 2^8

__host__ __device__ inline int kv8_page_bytes(int page, int D) { return page * (2 * D + 1); }
// within the keys' or the values' codes (these begin at page * D)
__host__ __device__ inline int kv8_code_byte(int D, int slot, int d) {
    return slot / 8 * (8 * D) + d / 16 * 128 + slot % 8 * 16 + d % 16;
}
__host__ __device__ inline int kv8_word_byte(int page, int D, int slot, int values) {
    return 2 * page * D + slot / kKv8Block * 16 + values * 4;
}

// The exponent of a word's scale, within the range that scales have (whatever the word holds).
__device__ __forceinline__ int kv8_exponent(uint32_t word) {
    const int e = int(word >> 23 & 255u) - 127;
    return e < kKv8Least ? kKv8Least : (e > kKv8Most ? kKv8Most : e);
}
__device__ __forceinline__ float kv8_power(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127

// Codes nearest to four numbers (ties to even, at most 448 in magnitude), x in the lowest byte.
__device__ __forceinline__ uint32_t kv8_codes(float x, float y, float z, float w) {
    uint32_t c;
    asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\tmov.b32 %0, {a, b};\n\t}"
        : "=r"(c)
        : "f"(x), "f"(y), "f"(z), "f"(w));
    return c;
}
// What the two codes in the low half of w stand for.
__device__ __forceinline__ float2 kv8_numbers(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// Four codes with those of -0 replaced by +0.
__device__ __forceinline__ uint32_t kv8_no_minus_zero(uint32_t w) {
    return w & (((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | 0x7F7F7F7Fu);
}

// Two numbers rounded to the type, the first in the low half.
template <bool kBF16>
__device__ __forceinline__ uint32_t kv8_pack(float x, float y) {
    if (kBF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 16 numbers of a row, of an address on the 16-byte grid; `whole`: on the 32-byte grid, where one instruction takes a sector (as two halves of
// sectors a row costs twice the wavefronts: reading a prefix back took 89 us for 74, an append of a long one 59 for 50).
__device__ __forceinline__ void kv8_load_row(const uint16_t *p, uint32_t (&w)[8], bool whole) {
    if (whole) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(__cvta_generic_to_global(p)));
    } else {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p)), y = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
    }
}
__device__ __forceinline__ void kv8_store_row(uint16_t *p, const uint32_t (&o)[8], bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(p)), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                     "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace sv
