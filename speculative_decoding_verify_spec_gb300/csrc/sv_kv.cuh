// sv_kv.cuh -- the 4-bit paged cache: its byte layout, the rotation and the type helpers that
// the append and the attention share.
//
// Layout of one page and head, for P slots of D dimensions (see spec_serve.h):
//   keys    row-major, dimension d of slot t in byte t D / 2 + d / 2, the lower half first.  Read
//           as an MMA operand, lane t % 4 of a quad takes a quarter of a token's row in one load.
//   values  blocks of 16 slots, 8 D bytes each: [D / 32][8: d % 32 / 4][4: t % 8 / 2][2: t % 16 / 8]
//           [2: t % 2][2 bytes: d % 4].  The 8 bytes of a (slice of 32 dimensions, lane) are the four
//           dimensions that the lane feeds to four n-tiles, for the two token pairs of a k16 step:
//           one conflict-free 8-byte load per lane and 16 tokens, and each 32-bit word unpacks to
//           half2 registers that already hold a token pair.
//   scales  (scale, zero) fp16 pairs per slot, keys then values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "spec_serve.h"

namespace sv {

__host__ __device__ inline int kv_page_bytes(int page, int D) { return page * (D + 8); }
__host__ __device__ inline int kv_key_byte(int D, int slot, int d) { return slot * (D / 2) + d / 2; }
// within the values' codes (which start at page * D / 2)
__host__ __device__ inline int kv_value_byte(int D, int slot, int d) {
    return slot / 16 * (8 * D) + d / 32 * 256 + (d % 32 / 4 * 4 + slot % 8 / 2) * 8 + slot % 16 / 8 * 4 + slot % 2 * 2 +
           d % 4 / 2;
}
__host__ __device__ inline int kv_key_scale_byte(int page, int D, int slot) { return page * D + slot * 4; }
__host__ __device__ inline int kv_value_scale_byte(int page, int D, int slot) { return page * (D + 4) + slot * 4; }

struct Rotation {
    const float *cos, *sin;  // [len][pairs], NULL: none
    int len, pairs;
    int interleaved;
    const int32_t *positions;  // [B][T] or NULL
};

inline bool kv_head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }
inline bool kv_page_size_ok(int p) { return p >= 16 && p <= 1024 && p % 16 == 0; }

// A sequence's tokens in the cache before the step, and its new ones, clamped.
__device__ __forceinline__ void kv_lengths(const int32_t *start, const int32_t *new_lens, int64_t b, int T,
                                           int64_t capacity, int &before, int &fresh) {
    const int s = start[b];
    before = s < 0 ? 0 : (s > capacity ? int(capacity) : s);
    int n = new_lens ? new_lens[b] : T;
    fresh = n < 0 ? 0 : (n > T ? T : n);
}

// Where the angles of a sequence's new token t begin.
__device__ __forceinline__ int64_t kv_rotation_row(const Rotation &r, int64_t bt, int before, int t) {
    const int64_t p = r.positions ? r.positions[bt] : int64_t(before) + t;  // (the sum may pass 31 bits)
    return (p < 0 ? 0 : (p >= r.len ? r.len - 1 : p)) * r.pairs;
}

// Dimension d's partner, angle index and the sign of the sine: rotated = x c + sign partner s.
// False: d is not rotated.
__device__ __forceinline__ bool kv_partner(const Rotation &r, int d, int &partner, int &angle, float &sign) {
    if (d >= 2 * r.pairs) return false;
    if (r.interleaved) {
        partner = d ^ 1, angle = d >> 1, sign = d & 1 ? 1.f : -1.f;
    } else {
        const bool low = d < r.pairs;
        partner = low ? d + r.pairs : d - r.pairs, angle = low ? d : d - r.pairs, sign = low ? -1.f : 1.f;
    }
    return true;
}

__device__ __forceinline__ float kv_to_float(uint16_t u, bool bf16) {
    return bf16 ? __uint_as_float(uint32_t(u) << 16) : __half2float(__ushort_as_half(u));
}
__device__ __forceinline__ uint16_t kv_from_float(float x, bool bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

}  // namespace sv
