// sv_kv8_append.cu -- the new tokens' keys and values into the 8-bit paged cache, the position rotation of the keys
// applied on the way.
//
// A block of 16 slots has one scale, so D / 64 warps take a block of one sequence and head, its keys or its values: they load
// the new tokens' vectors, rotate keys, reduce the largest magnitude, and from it have the scale (a power of two) and the
// codes; the block's older codes are read only if the scale grows.  A lane has a slot and two pieces of 16 dimensions: a piece of eight
// slots is 128 contiguous bytes of the cache, and the two pieces are those that the rotation joins, so that an angle is loaded
// once for both.  The rotated numbers stay in registers from the reduction to the codes.
//
// The result is that of the exact rule.  fp32 leaves a rotated key off by at most 2^-23 (|a cos| + |b sin|), and with D the
// largest such bound of the block (for its scale) or of a lane's numbers (for their codes), a scale or a code is settled if x - D and x + D
// have the same one.  What is left (a code in some ten thousand, a scale in a million) is computed in 64 bits, where a 16-bit number
// times an fp32 angle is exact and one subtraction rounds; a lane collects its codes in doubt first, so that the lanes' ones go side by side.
//
// Everything is read once and written once; 16 bits in, 8 out (and 16 where the values held are wanted).  Measured, with the values held:
// 8 prompts of up to 2001 tokens, 16 heads of 64, fp16, 41 us (3.5 TB/s); one of 16384 tokens, 4 heads of 256, bf16, 46 us (4.0 TB/s), 38 without a rotation;
// 256 x 9 drafts, 8 heads of 128, 16 us.  It waits for loads (a block's lengths, then its page and rows, then its angles) with 18 and 24 warps
// an SM under way, and issues 2 instructions a clock.  Blocks that take several items in turn were slower (88 us for 59, before rows went in 32 bytes).
#include <cstdint>

#include "sv_checks.cuh"
#include "sv_device.cuh"
#include "sv_kv8.cuh"

namespace sv {
namespace {

constexpr int kApp8Threads = 128;

struct Append8Args {
    const uint16_t *k, *v;
    int64_t k_bs, k_ts, k_hs, v_bs, v_ts, v_hs;
    uint32_t items, blocks;  // B * blocks * H * 2; blocks a sequence
    int T, H;
    uint8_t *cache;
    int num_pages, page, width;
    const int32_t *table, *start, *new_lens;
    Rotation rot;
    uint16_t *k_values, *v_values;
    bool whole_in, whole, whole_angles;  // all rows of k and v, of k_values and v_values, of the angles are on the 32-byte grid
};

// How rows and rotation lie: any way; on the 16-byte grid, and the rotation's partners whole pieces apart (or no rotation);
// on the grid, and the partners neighbours.
enum Layout8 { kAny8, kHalves8, kNeighbours8 };

// A pair's two pieces of 16 dimensions each, of a row.
template <int D, Layout8 kLayout>
__device__ __forceinline__ void pieces_of(int pairs, int unit, int &lo, int &hi) {
    const int p = kLayout == kHalves8 ? pairs / 16 : 0;  // pieces of a half
    if (unit < p) {
        lo = unit, hi = unit + p;
    } else {
        lo = 2 * unit, hi = 2 * unit + 1;  // (those behind the rotated ones: 2 p + 2 (unit - p))
    }
}

template <Layout8 kLayout>
__device__ __forceinline__ void load_piece(const uint16_t *p, uint32_t (&w)[8], bool whole) {
    if (kLayout != kAny8) {
        kv8_load_row(p, w, whole);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = uint32_t(__ldg(p + 2 * i)) | uint32_t(__ldg(p + 2 * i + 1)) << 16;
    }
}
template <bool kBF16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
    if (kBF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Eight angles.  (Those of neighbours are taken by fours: by eights, prompts of 64 dimensions took 41.9 us for 41.0.)
__device__ __forceinline__ void load_angles(const float *p, bool whole, float (&x)[8]) {
    uint32_t w[8];
    kv8_load_row(reinterpret_cast<const uint16_t *>(p), w, whole);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}

// The raw pair w (piece lo, piece hi) as floats, rotated; `most` takes the largest |a cos| + |b sin|.
template <Layout8 kLayout, bool kBF16>
__device__ __forceinline__ void rotated(const Rotation &rot, const uint16_t *row, int64_t angles, int lo, int hi, const uint32_t (&w)[2][8],
                                        float (&x)[2][16], float &most, bool whole) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = widen2<kBF16>(w[p][i]);
            x[p][2 * i] = f.x, x[p][2 * i + 1] = f.y;
        }
    if (!rot.cos) return;
    const float *cp = rot.cos + angles, *sp = rot.sin + angles;
    if constexpr (kLayout == kHalves8) {
        if (lo * 16 >= rot.pairs) return;
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            float c[8], s[8];
            load_angles(cp + lo * 16 + i, whole, c), load_angles(sp + lo * 16 + i, whole, s);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = x[0][i + j], b = x[1][i + j];
                most = fmaxf(most, (fabsf(a) + fabsf(b)) * fmaxf(fabsf(c[j]), fabsf(s[j])));
                x[0][i + j] = fmaf(a, c[j], -b * s[j]), x[1][i + j] = fmaf(b, c[j], a * s[j]);
            }
        }
    } else if constexpr (kLayout == kNeighbours8) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int d0 = (p ? hi : lo) * 16;
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                if (d0 + i >= 2 * rot.pairs) break;  // (pairs is a multiple of four)
                const float4 cv = __ldg(reinterpret_cast<const float4 *>(cp + (d0 + i) / 2)), sv = __ldg(reinterpret_cast<const float4 *>(sp + (d0 + i) / 2));
                const float c[4] = {cv.x, cv.y, cv.z, cv.w}, s[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = x[p][i + 2 * j], b = x[p][i + 2 * j + 1];
                    most = fmaxf(most, (fabsf(a) + fabsf(b)) * fmaxf(fabsf(c[j]), fabsf(s[j])));
                    x[p][i + 2 * j] = fmaf(a, c[j], -b * s[j]), x[p][i + 2 * j + 1] = fmaf(b, c[j], a * s[j]);
                }
            }
        }
    } else {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                int partner, angle;
                float sign;
                if (kv_partner(rot, (p ? hi : lo) * 16 + i, partner, angle, sign)) {
                    const float a = x[p][i], b = kv_to_float(__ldg(row + partner), kBF16), c = __ldg(cp + angle), s = __ldg(sp + angle);
                    most = fmaxf(most, (fabsf(a) + fabsf(b)) * fmaxf(fabsf(c), fabsf(s)));
                    x[p][i] = fmaf(a, c, sign * b * s);
                }
            }
    }
}

// Dimension d of a row, rotated, in 64 bits: both products exact, one rounding.
template <bool kBF16>
__device__ __noinline__ double rotated_exactly(const Rotation &rot, const uint16_t *row, int64_t angles, int d) {
    const double x = kv_to_float(row[d], kBF16);
    int partner, angle;
    float sign;
    if (!rot.cos || !kv_partner(rot, d, partner, angle, sign)) return x;
    const double p = x * double(rot.cos[angles + angle]), q = double(kv_to_float(row[partner], kBF16)) * double(rot.sin[angles + angle]);
    return sign < 0 ? p - q : p + q;
}

// The least e with 2^e >= |x|, far below every scale for 0; x finite.
__device__ __forceinline__ int ceil_exponent(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    return u < 0x00800000u ? -126 : int(u >> 23) - 127 + ((u & 0x7FFFFFu) != 0);
}
__device__ __forceinline__ int ceil_exponent(double x) {
    const uint64_t u = __double_as_longlong(x) & 0x7FFFFFFFFFFFFFFFull;
    return u < 0x0010000000000000ull ? -1022 : int(u >> 52) - 1023 + ((u & 0xFFFFFFFFFFFFFull) != 0);
}

// The code nearest to x, finite (ties to the even one).
__device__ __noinline__ uint32_t code_exactly(double x) {
    const double m = fmin(fabs(x), 448.0);
    const int e = max(int(uint64_t(__double_as_longlong(m)) >> 52) - 1023, -6);
    const int n = __double2int_rn(m * __longlong_as_double(int64_t(1023 + 3 - e) << 52));  // 8 .. 16; less at the lowest exponent
    return uint32_t(n >= 8 ? (e + 6) * 8 + n : n) | (x < 0 ? 128u : 0u);                    // (16: the next exponent's first)
}

// The larger one, NaN if there is one.
__device__ __forceinline__ float max_or_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

template <int D, Layout8 kLayout, bool kBF16>
__global__ void __launch_bounds__(kApp8Threads) kv8_append_kernel(const Append8Args a) {
    constexpr int W = D / 64, kItems = kApp8Threads / 32 / W;  // warps of a block of slots, and those blocks of a thread block
    __shared__ uint32_t red[kItems][2][W], bad_s[kItems];
    __shared__ int e_s[kItems];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, part = warp % W, mine = warp / W;
    const uint32_t item0 = blockIdx.x * kItems + mine, item = item0 < a.items ? item0 : a.items - 1;
    griddep_launch_next();
    griddep_wait();
    const int values = int(item & 1u);
    const uint32_t bjh = item >> 1, bj = bjh / uint32_t(a.H), h = bjh - bj * uint32_t(a.H), b = bj / a.blocks;
    const int64_t capacity = int64_t(a.width) * a.page;
    int before, fresh;
    kv_lengths(a.start, a.new_lens, b, a.T, capacity, before, fresh);
    const int64_t first = int64_t(before / kKv8Block) * kKv8Block + int64_t(bj - b * a.blocks) * kKv8Block;  // the block's first slot
    // the block's slots from `lo` on are tokens t0 + slot; those below `end` are new
    const int64_t t0 = first - before;
    const int lo = item0 < a.items ? (t0 < 0 ? int(-t0) : 0) : kKv8Block;  // (past the last item: nothing)
    const int end = int(fresh - t0 < 0 ? 0 : (fresh - t0 < kKv8Block ? fresh - t0 : kKv8Block));
    uint16_t *held = values ? a.v_values : a.k_values;
    const uint16_t *in = values ? a.v + b * a.v_bs + h * a.v_hs : a.k + b * a.k_bs + h * a.k_hs;
    Rotation rot = a.rot;
    if (values) rot.cos = nullptr, rot.pairs = 0;
    int pg = -1, s0 = 0;  // page, and the block's first slot in it
    if (first < capacity && end > lo) {
        const uint32_t pi = uint32_t(first) / uint32_t(a.page);
        s0 = int(uint32_t(first) - pi * uint32_t(a.page));
        pg = __ldg(a.table + int64_t(b) * a.width + pi);
    }
    // this lane's slot and its two pieces of the row
    const int slot = D == 64 ? lane & 15 : (lane & 7) + (part & 1) * 8;
    const int unit = D == 64 ? lane >> 4 : (lane >> 3) + part / 2 * 4;
    int p, q;
    pieces_of<D, kLayout>(rot.pairs, unit, p, q);
    const int64_t t = t0 + slot;
    const bool live = slot >= lo && slot < end;
    const uint16_t *row = in + t * (values ? a.v_ts : a.k_ts);
    float x[2][16], largest = 0.f, most = 0.f;
    int64_t angles = 0;
    bool fine = true;
    if (live) {
        uint32_t raw[2][8];
        load_piece<kLayout>(row + p * 16, raw[0], a.whole_in), load_piece<kLayout>(row + q * 16, raw[1], a.whole_in);
        if (rot.cos) angles = kv_rotation_row(rot, int64_t(b) * a.T + t, before, int(t));
        rotated<kLayout, kBF16>(rot, row, angles, p, q, raw, x, most, a.whole_angles);
#pragma unroll
        for (int j = 0; j < 16; ++j) largest = max_or_nan(max_or_nan(largest, fabsf(x[0][j])), fabsf(x[1][j]));
        fine = largest < INFINITY && most < INFINITY;
    }
    const bool here = pg >= 0 && pg < a.num_pages && SV_IN(kv8_code_byte(D, s0 + kKv8Block - 1, D - 1), a.page * D);
    uint8_t *base = here ? a.cache + (int64_t(pg) * a.H + h) * kv8_page_bytes(a.page, D) : nullptr;
    uint8_t *codes = base + values * a.page * D;
    uint32_t *word = reinterpret_cast<uint32_t *>(base + kv8_word_byte(a.page, D, s0, values));
    uint32_t old = 0;
    if (here && lo > 0) old = __ldcg(word);

    uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(largest)), bound = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    if (W > 1) {
        if (lane == 0) red[mine][0][part] = top, red[mine][1][part] = bound;
    }
    if (threadIdx.x < kItems) bad_s[threadIdx.x] = 0, e_s[threadIdx.x] = -1022;
    const bool odd = __syncthreads_or(!fine);  // (some number here is not finite, or not in 32 bits: all in 64)
    if (W > 1) {
#pragma unroll
        for (int i = 0; i < W; ++i) top = max(top, red[mine][0][i]), bound = max(bound, red[mine][1][i]);
    }
    const float off = __uint_as_float(bound) * 2.4e-7f;  // 2^-22 and a little: two roundings, and those of the sums that make `most`
    int e = ceil_exponent(fmaxf(__uint_as_float(top) - off, 0.f));  // (if !odd) that of the largest magnitude, or less
    uint32_t bad = 0;  // slots with a NaN or an infinity
    if (odd) {  // first which vectors are to be left out, then the largest magnitude of the others
        for (int round = 0; round < 2; ++round) {
            e = -1022;
            if (live && !(bad >> slot & 1u)) {
                bool out = false;
#pragma unroll 1
                for (int j = 0; j < 32; ++j) {
                    const double y = rotated_exactly<kBF16>(rot, row, angles, (j < 16 ? p : q) * 16 + j % 16);
                    if (!(fabs(y) < INFINITY)) out = true;
                    else e = max(e, ceil_exponent(y));
                }
                if (out) atomicOr(&bad_s[mine], 1u << slot);
                if (round == 1) atomicMax(&e_s[mine], e);
            }
            __syncthreads();
            bad = bad_s[mine];
        }
        e = e_s[mine];
    } else if (__syncthreads_or(e != ceil_exponent(__uint_as_float(top) + off))) {
        // the numbers that may be above 2^e, in 64 bits.  (A power of two itself, not turned, is in doubt: one largest magnitude in 200.)
        uint32_t doubt = 0;
        if (live) {
#pragma unroll
            for (int j = 0; j < 32; ++j) doubt |= uint32_t(fabsf(x[j / 16][j % 16]) + off > kv8_power(e)) << j;
        }
#pragma unroll 1
        while (doubt) {
            const int j = __ffs(doubt) - 1;
            doubt &= doubt - 1;
            atomicMax(&e_s[mine], ceil_exponent(rotated_exactly<kBF16>(rot, row, angles, (j < 16 ? p : q) * 16 + j % 16)));
        }
        __syncthreads();
        e = max(e, e_s[mine]);
    }
    e = min(max(e - kKv8Top, kKv8Least), kKv8Most);
    if (here && lo > 0) e = max(e, kv8_exponent(old));
    const float inv = kv8_power(-e), scale = kv8_power(e);
    // this lane's numbers are off by 2^-23 of its own `most`, and the sums below by half of that
    const float o_turned = most * 1.85e-7f * inv;

    if (slot >= lo && t < a.T) {
        const bool nan = bad >> slot & 1u;
        uint32_t c[2][4] = {}, doubt = 0;  // bit 16 k + i: element i of piece k
        if (live && !nan) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float y[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) y[n] = x[k][4 * j + n] * inv;
                    const bool turned = rot.cos && (k ? q : p) * 16 + 4 * j < 2 * rot.pairs;
                    const float o = turned ? o_turned : 0.f;
                    c[k][j] = kv8_codes(y[0] - o, y[1] - o, y[2] - o, y[3] - o);
                    if (turned) {
                        const uint32_t u = kv8_codes(y[0] + o, y[1] + o, y[2] + o, y[3] + o) ^ c[k][j];
                        if (u || odd) {
#pragma unroll
                            for (int n = 0; n < 4; ++n) doubt |= uint32_t(odd || (u >> (8 * n) & 255u)) << (16 * k + 4 * j + n);
                        }
                    }
                }
#pragma unroll 1
            while (doubt) {  // (the lanes' ones side by side)
                const int i = __ffs(doubt) - 1, d = (i < 16 ? p : q) * 16 + (i & 15), shift = 8 * (i & 3);
                doubt &= doubt - 1;
                const uint32_t one = code_exactly(rotated_exactly<kBF16>(rot, row, angles, d) * double(inv));
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (i / 4 == k) c[k / 4][k % 4] = (c[k / 4][k % 4] & ~(255u << shift)) | one << shift;
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int piece = k ? q : p;
#pragma unroll
            for (int j = 0; j < 4; ++j) c[k][j] = kv8_no_minus_zero(c[k][j]);
            if (live && here)
                *reinterpret_cast<uint4 *>(codes + kv8_code_byte(D, s0 + slot, piece * 16)) = make_uint4(c[k][0], c[k][1], c[k][2], c[k][3]);
            if (held) {
                const float s = nan ? NAN : scale;
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 u = kv8_numbers(c[k][j]), v = kv8_numbers(c[k][j] >> 16);
                    o[2 * j] = kv8_pack<kBF16>(u.x * s, u.y * s), o[2 * j + 1] = kv8_pack<kBF16>(v.x * s, v.y * s);
                }
                kv8_store_row(held + ((int64_t(b) * a.T + t) * a.H + h) * D + piece * 16, o, a.whole);
            }
        }
    }
    if (!here) return;
    if (lo > 0 && e > kv8_exponent(old)) {  // the older codes, to the new scale
        const float shrink = kv8_power(max(kv8_exponent(old) - e, -100));
#pragma unroll 1
        for (int i = part * 32 + lane; i < kKv8Block * (D / 16); i += 32 * W) {
            const int sl = i & 15, piece = i >> 4;
            if (sl >= lo) continue;
            uint4 *at = reinterpret_cast<uint4 *>(codes + kv8_code_byte(D, s0 + sl, piece * 16));
            const uint4 was = __ldcg(at);
            uint32_t w[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = kv8_numbers(w[j]), v = kv8_numbers(w[j] >> 16);
                w[j] = kv8_no_minus_zero(kv8_codes(u.x * shrink, u.y * shrink, v.x * shrink, v.y * shrink));
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if (lane == 0 && part == 0) *word = (__float_as_uint(scale) & 0xFFFF0000u) | (old & ((1u << lo) - 1)) | bad;
}

template <int D>
cudaError_t launch_append8(const Append8Args &a, Layout8 layout, bool bf16, cudaStream_t s) {
    constexpr unsigned kItems = kApp8Threads / 32 / (D / 64);
    const unsigned blocks = (a.items + kItems - 1) / kItems;
    auto go = [&](auto kernel) { return launch_after(kernel, blocks, unsigned(kApp8Threads), 0, s, a); };
    switch (layout) {
    case kHalves8: return bf16 ? go(kv8_append_kernel<D, kHalves8, true>) : go(kv8_append_kernel<D, kHalves8, false>);
    case kNeighbours8: return bf16 ? go(kv8_append_kernel<D, kNeighbours8, true>) : go(kv8_append_kernel<D, kNeighbours8, false>);
    default: return bf16 ? go(kv8_append_kernel<D, kAny8, true>) : go(kv8_append_kernel<D, kAny8, false>);
    }
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_kv8_append(const void *k, int64_t k_batch_stride, int64_t k_token_stride, int64_t k_head_stride,
                                     const void *v, int64_t v_batch_stride, int64_t v_token_stride, int64_t v_head_stride,
                                     sv_kv_dtype dtype, int B, int T, int kv_heads, int head_dim, void *cache, int num_pages,
                                     int page_size, const int32_t *page_table, int table_width, const int32_t *start,
                                     const int32_t *new_lens, const float *cos, const float *sin, int table_len, int pairs,
                                     int interleaved, const int32_t *positions, void *k_values, void *v_values, void *stream) {
    if (dtype != SV_KV_BF16 && dtype != SV_KV_FP16) return SV_ERR_UNSUPPORTED;
    if (!sv::kv_head_dim_ok(head_dim) || !sv::kv_page_size_ok(page_size)) return SV_ERR_UNSUPPORTED;
    if (B < 0 || T < 0 || kv_heads < 1 || num_pages < 0 || table_width < 0) return SV_ERR_INVALID_ARG;
    if (k_batch_stride < 0 || k_token_stride < 0 || k_head_stride < 0 || v_batch_stride < 0 || v_token_stride < 0 ||
        v_head_stride < 0)
        return SV_ERR_INVALID_ARG;
    if (int64_t(table_width) * page_size > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;
    if (!cos != !sin) return SV_ERR_INVALID_ARG;
    if (cos && (table_len < 1 || pairs < 1 || pairs > head_dim / 2)) return SV_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return SV_OK;
    if (!k || !v || !start || (table_width > 0 && !page_table) || (num_pages > 0 && !cache)) return SV_ERR_INVALID_ARG;
    // blocks of 16 slots that T tokens touch, wherever the first one lies
    const int64_t blocks = (int64_t(T) + 30) / sv::kKv8Block, warps = 2 * blocks * kv_heads;
    if (warps > 0x7FFFFFF0 || warps * B > 0x7FFFFFF0) return SV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(k) % 2 || reinterpret_cast<uintptr_t>(v) % 2 ||
        reinterpret_cast<uintptr_t>(k_values) % 16 || reinterpret_cast<uintptr_t>(v_values) % 16)
        return SV_ERR_INVALID_ARG;
    const int64_t all = k_batch_stride | k_token_stride | k_head_stride | v_batch_stride | v_token_stride | v_head_stride;
    sv::Append8Args a{};
    a.k = static_cast<const uint16_t *>(k), a.v = static_cast<const uint16_t *>(v);
    a.k_bs = k_batch_stride, a.k_ts = k_token_stride, a.k_hs = k_head_stride;
    a.v_bs = v_batch_stride, a.v_ts = v_token_stride, a.v_hs = v_head_stride;
    const bool grid = all % 8 == 0 && (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 16 == 0 &&
                      (!cos || (pairs % 4 == 0 && (reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) % 16 == 0));
    const sv::Layout8 layout = !grid                    ? sv::kAny8
                               : cos && interleaved     ? sv::kNeighbours8
                               : cos && pairs % 16 != 0 ? sv::kAny8
                                                        : sv::kHalves8;
    a.items = uint32_t(warps * B), a.blocks = uint32_t(blocks), a.T = T, a.H = kv_heads;
    a.cache = static_cast<uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.table = page_table, a.start = start, a.new_lens = new_lens;
    a.rot = sv::Rotation{cos, sin, table_len, cos ? pairs : 0, interleaved != 0, positions};
    a.k_values = static_cast<uint16_t *>(k_values), a.v_values = static_cast<uint16_t *>(v_values);
    a.whole = (reinterpret_cast<uintptr_t>(k_values) | reinterpret_cast<uintptr_t>(v_values)) % 32 == 0;
    a.whole_angles = pairs % 8 == 0 && (reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) % 32 == 0;
    a.whole_in = all % 16 == 0 && (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == SV_KV_BF16;
    const cudaError_t e = head_dim == 64    ? sv::launch_append8<64>(a, layout, bf16, s)
                          : head_dim == 128 ? sv::launch_append8<128>(a, layout, bf16, s)
                                            : sv::launch_append8<256>(a, layout, bf16, s);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
