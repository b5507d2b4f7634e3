// sv_kv_append.cu -- the new tokens' keys and values into the 4-bit paged cache, the position
// rotation of the keys applied on the way.
//
// D / 8 lanes take a (token, head): eight dimensions of its key and of its value each, one 16-byte load a
// row.  They rotate the key, reduce minimum and maximum over their lanes, and write the codes.  The result is
// that of the exact rule: rotated keys are double-float (a 16-bit input times an fp32 cosine is exact in
// two floats), and whatever lies so near a rounding border that 32 bits cannot tell -- about one scale
// in two thousand, one code in 100,000 -- is decided on exact differences.  Everything is read once and written
// once.  The variants are by what the loads can be: rows and angles on the 16-byte grid with the rotation's
// partners eight dimensions apart in one place (halves) or in the lane itself (neighbours), else any.
//
// Measured: 256 x 9 tokens of 8 heads of 128 dimensions 11.7 us (1.9 TB/s), 8 prompts of up to 2001 tokens, 16 heads
// of 64, 52 us (2.5 TB/s).  The two-float rotation, the extremes and the codes keep the ALU pipe at 60 %: the
// largest part of what bounds it, at about 25 instructions a dimension.
#include <cstdint>

#include "sv_checks.cuh"
#include "sv_device.cuh"
#include "sv_kv.cuh"

namespace sv {
namespace {

constexpr int kAppThreads = 256;

struct AppendArgs {
    const uint16_t *k, *v;
    int64_t k_bs, k_ts, k_hs, v_bs, v_ts, v_hs;
    uint32_t items;  // B * T * H
    int T, H;
    uint8_t *cache;
    int num_pages, page, width;
    const int32_t *table, *start, *new_lens;
    Rotation rot;
    uint16_t *k_values, *v_values;
};

__device__ __forceinline__ float saturate(float x) { return fminf(fmaxf(x, -65504.f), 65504.f); }

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 1.5 * 2^23: added to a float of less than 2^22 it leaves the nearest integer (ties to even) in the low bits.
constexpr float kRound = 12582912.f;

// Quantises one head vector of 8 L dimensions, held as hi + lo by L lanes (eight each): the lane's codes, 4 bits
// each, and the scale and zero as fp16 bits in one word (scale low).
template <int L, bool kLow>
__device__ __forceinline__ uint32_t quantise(const float (&hi)[8], const float (&lo)[8], uint32_t &meta) {
    float low = hi[0], high = hi[0];  // (a NaN stays)
#pragma unroll
    for (int i = 1; i < 8; ++i) low = min_nan(low, hi[i]), high = max_nan(high, hi[i]);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) {
        low = min_nan(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
        high = max_nan(high, __shfl_xor_sync(0xFFFFFFFFu, high, o));
    }
    const bool bad = !(high <= 3.4e38f && low >= -3.4e38f);
    // zero = fp16(fp32(min)): the least hi is that fp32 number
    const float range = high - low, t = range * (1.f / 15.f);
    // scale = fp16(fp32(range / 15)): t is off by three roundings, and by what the low parts add (each at most 2^-24
    // of its high part); where that may matter, the quotient of the exact range in 64 bits
    float off = t * 2.4e-7f;
    if constexpr (kLow) off = fmaf(fmaxf(fabsf(low), fabsf(high)), 1e-8f, off);
    const __half2 ends = __floats2half2_rn(saturate(t - off), saturate(t + off));
    uint32_t sb = __half_as_ushort(__low2half(ends));
    const bool doubt = !bad && sb != __half_as_ushort(__high2half(ends));
    if (__any_sync(0xFFFFFFFFu, doubt)) {  // (all lanes take part in the reductions)
        float least = 0.f, most = 0.f;  // the low parts of the extremes
        if constexpr (kLow) {
            least = INFINITY, most = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (hi[i] == low) least = fminf(least, lo[i]);
                if (hi[i] == high) most = fmaxf(most, lo[i]);
            }
#pragma unroll
            for (int o = L / 2; o; o >>= 1) {
                least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
            }
        }
        if (doubt) {
            const double exact = ((double(high) - double(low)) + (double(most) - double(least))) / 15.0;
            sb = __half_as_ushort(__float2half_rn(saturate(__double2float_rn(exact))));
        }
    }
    uint32_t zb = __half_as_ushort(__float2half_rn(saturate(low)));
    if (sb == 0) sb = 1;          // 2^-24
    if (zb == 0x8000u) zb = 0;
    if (bad) {
        meta = 0x7E007E00u;  // NaN, NaN
        return 0;
    }
    meta = zb << 16 | sb;
    const float z = __half2float(__ushort_as_half(uint16_t(zb))), s = __half2float(__ushort_as_half(uint16_t(sb)));
    const float inv = __frcp_rn(s);
    uint32_t codes = 0;
    bool near = false;
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // clamped before rounding, which changes no code; |q| <= 15 and four roundings of 2^-24: in doubt within
        // 3.6e-6 of a border (a saturated zero or scale only meets the clamp)
        const float q = fminf(fmaxf(((hi[i] - z) + (kLow ? lo[i] : 0.f)) * inv, 0.f), 15.f);
        c[i] = q + kRound;
        near |= fabsf(q - (c[i] - kRound)) > 0.499995f;
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = fminf(fmaxf(((hi[i] - z) + (kLow ? lo[i] : 0.f)) * inv, 0.f), 15.f), f = floorf(q);
            if (fabsf(q - (f + 0.5f)) < 1e-4f) {
                // the sign of x - z - s (f + 1/2), exact: s (f + 1/2) has 16 bits, and each difference keeps its error
                const float sb2 = s * (f + 0.5f), u = __fsub_rn(hi[i], z), ub = __fsub_rn(u, hi[i]);
                const float ue = __fsub_rn(__fsub_rn(hi[i], __fsub_rn(u, ub)), __fadd_rn(z, ub));
                const float d = __fsub_rn(u, sb2), db = __fsub_rn(d, u);
                const float de = __fsub_rn(__fsub_rn(u, __fsub_rn(d, db)), __fadd_rn(sb2, db));
                const float t2 = __fadd_rn(d, __fadd_rn(__fadd_rn(de, ue), kLow ? lo[i] : 0.f));
                const bool odd = (int(f) & 1) != 0;
                c[i] = (t2 > 0.f || (t2 == 0.f && odd) ? f + 1.f : f) + kRound;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= (__float_as_uint(c[i]) & 15u) << (4 * i);
    return codes;
}

enum Layout { kAny, kHalves, kNeighbours };  // how rows and rotation lie, see above

// Eight 16-bit numbers.
template <bool kVec>
__device__ __forceinline__ uint4 load_row(const uint16_t *p) {
    if (kVec) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = uint32_t(__ldg(p + 2 * i)) | uint32_t(__ldg(p + 2 * i + 1)) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool kBF16>
__device__ __forceinline__ void widen(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBF16) {
            x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

// What the codes stand for.
template <bool kBF16>
__device__ __forceinline__ void store_values(uint16_t *p, uint32_t codes, uint32_t meta, bool live) {
    const float s = __half2float(__ushort_as_half(uint16_t(meta))), z = __half2float(__ushort_as_half(uint16_t(meta >> 16)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // s code is exact: one rounding, then that to the type
        const float x = fmaf(s, float(codes >> (8 * i) & 15u), z), y = fmaf(s, float(codes >> (8 * i + 4) & 15u), z);
        if (kBF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x, y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    *reinterpret_cast<uint4 *>(p) = live ? make_uint4(w[0], w[1], w[2], w[3]) : make_uint4(0, 0, 0, 0);
}

// Rotates eight dimensions from d0 on of the key row kp, x, in two floats: both products exact, their sum exact, then
// the rest.
template <Layout kLayout, bool kBF16>
__device__ __forceinline__ void rotate(const AppendArgs &a, const uint16_t *kp, int d0, int64_t row, float (&x)[8], float (&lo)[8]) {
    const int pairs = a.rot.pairs;
    const float *cp = a.rot.cos + row, *sp = a.rot.sin + row;
    float y[8], c[8], s[8];
    if constexpr (kLayout == kHalves) {  // the eight lie within one half
        const bool low = d0 < pairs;
        const int e0 = low ? d0 : d0 - pairs;
        widen<kBF16>(load_row<true>(kp + (low ? d0 + pairs : e0)), y);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 u = __ldg(reinterpret_cast<const float4 *>(cp + e0 + i)), v = __ldg(reinterpret_cast<const float4 *>(sp + e0 + i));
            c[i] = u.x, c[i + 1] = u.y, c[i + 2] = u.z, c[i + 3] = u.w;
            s[i] = v.x, s[i + 1] = v.y, s[i + 2] = v.z, s[i + 3] = v.w;
        }
        if (low) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = -s[i];
        }
    } else if constexpr (kLayout == kNeighbours) {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(cp + d0 / 2)), v = __ldg(reinterpret_cast<const float4 *>(sp + d0 / 2));
        c[0] = c[1] = u.x, c[2] = c[3] = u.y, c[4] = c[5] = u.z, c[6] = c[7] = u.w;
        s[1] = v.x, s[3] = v.y, s[5] = v.z, s[7] = v.w;
#pragma unroll
        for (int i = 0; i < 8; i += 2) s[i] = -s[i + 1], y[i] = x[i + 1], y[i + 1] = x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int partner, angle;
            float sign;
            if (kv_partner(a.rot, d0 + i, partner, angle, sign)) {
                y[i] = kv_to_float(__ldg(kp + partner), kBF16);
                c[i] = __ldg(cp + angle), s[i] = sign * __ldg(sp + angle);
            } else {
                y[i] = 0.f, c[i] = 1.f, s[i] = 0.f;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float p = __fmul_rn(x[i], c[i]), pe = __fmaf_rn(x[i], c[i], -p);
        const float r = __fmul_rn(y[i], s[i]), re = __fmaf_rn(y[i], s[i], -r);
        const float sum = __fadd_rn(p, r), bb = __fsub_rn(sum, p);
        const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, bb)), __fsub_rn(r, bb));
        const float rest = __fadd_rn(e, __fadd_rn(pe, re));
        y[i] = __fadd_rn(sum, rest);
        lo[i] = __fsub_rn(rest, __fsub_rn(y[i], sum));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i];
}

template <int D, Layout kLayout, bool kBF16>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const AppendArgs a) {
    constexpr int L = D / 8, kItems = kAppThreads / L;
    const uint32_t item = blockIdx.x * kItems + threadIdx.x / L;
    griddep_launch_next();
    griddep_wait();
    const bool there = item < a.items;  // (the others only take part in the warp's reductions)
    const uint32_t it = there ? item : 0;
    const int d0 = int(threadIdx.x % L) * 8;
    const uint32_t bt = it / uint32_t(a.H), h = it - bt * uint32_t(a.H), b = bt / uint32_t(a.T);
    const int t = int(bt - b * uint32_t(a.T));
    const int64_t capacity = int64_t(a.width) * a.page;
    int before, fresh;
    kv_lengths(a.start, a.new_lens, b, a.T, capacity, before, fresh);
    const bool live = there && t < fresh;
    uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
    const uint16_t *kp = a.k + b * a.k_bs + t * a.k_ts + h * a.k_hs, *vp = a.v + b * a.v_bs + t * a.v_ts + h * a.v_hs;
    int pg = -1, sl = 0;
    if (live) {
        kv = load_row<kLayout != kAny>(kp + d0), vv = load_row<kLayout != kAny>(vp + d0);
        const int64_t slot = int64_t(before) + t;
        if (slot < capacity) {
            const uint32_t pi = uint32_t(slot) / uint32_t(a.page);
            sl = int(uint32_t(slot) - pi * uint32_t(a.page));
            pg = __ldg(a.table + int64_t(b) * a.width + pi);
        }
    }
    if (!__any_sync(0xFFFFFFFFu, live)) {  // tokens past the new ones
        const uint4 none = make_uint4(0, 0, 0, 0);
        if (there && a.k_values) *reinterpret_cast<uint4 *>(a.k_values + int64_t(item) * D + d0) = none;
        if (there && a.v_values) *reinterpret_cast<uint4 *>(a.v_values + int64_t(item) * D + d0) = none;
        return;
    }
    float x[8], lo[8];
    uint32_t km, vm, kc, vc;
    widen<kBF16>(kv, x);
    if (a.rot.cos) {
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = 0.f;
        if (live && d0 < 2 * a.rot.pairs) rotate<kLayout, kBF16>(a, kp, d0, kv_rotation_row(a.rot, bt, before, t), x, lo);
        kc = quantise<L, true>(x, lo, km);
    } else {
        kc = quantise<L, false>(x, x, km);
    }
    widen<kBF16>(vv, x);
    vc = quantise<L, false>(x, x, vm);
    if (!there) return;
    if (live && pg >= 0 && pg < a.num_pages && SV_IN(kv_value_byte(D, sl, d0 + 7), a.page * D / 2)) {
        uint8_t *base = a.cache + (int64_t(pg) * a.H + h) * kv_page_bytes(a.page, D);
        *reinterpret_cast<uint32_t *>(base + kv_key_byte(D, sl, d0)) = kc;
        uint8_t *vd = base + a.page * D / 2 + kv_value_byte(D, sl, d0);
        *reinterpret_cast<uint16_t *>(vd) = uint16_t(vc);
        *reinterpret_cast<uint16_t *>(vd + 32) = uint16_t(vc >> 16);  // the next four dimensions
        if (d0 == 0) {
            *reinterpret_cast<uint32_t *>(base + kv_key_scale_byte(a.page, D, sl)) = km;
            *reinterpret_cast<uint32_t *>(base + kv_value_scale_byte(a.page, D, sl)) = vm;
        }
    }
    if (a.k_values) store_values<kBF16>(a.k_values + int64_t(item) * D + d0, kc, km, live);
    if (a.v_values) store_values<kBF16>(a.v_values + int64_t(item) * D + d0, vc, vm, live);
}

template <int D>
cudaError_t launch_append(const AppendArgs &a, Layout layout, bool bf16, unsigned blocks, cudaStream_t s) {
    auto go = [&](auto kernel) { return launch_after(kernel, blocks, unsigned(kAppThreads), 0, s, a); };
    switch (layout) {
    case kHalves: return bf16 ? go(kv_append_kernel<D, kHalves, true>) : go(kv_append_kernel<D, kHalves, false>);
    case kNeighbours: return bf16 ? go(kv_append_kernel<D, kNeighbours, true>) : go(kv_append_kernel<D, kNeighbours, false>);
    default: return bf16 ? go(kv_append_kernel<D, kAny, true>) : go(kv_append_kernel<D, kAny, false>);
    }
}

}  // namespace
}  // namespace sv

extern "C" {

size_t spec_kv_page_bytes(int page_size, int head_dim) {
    if (!sv::kv_page_size_ok(page_size) || !sv::kv_head_dim_ok(head_dim)) return 0;
    return size_t(sv::kv_page_bytes(page_size, head_dim));
}

int64_t spec_kv_code_offset(int page_size, int head_dim, int values, int token, int dim) {
    if (!sv::kv_page_size_ok(page_size) || !sv::kv_head_dim_ok(head_dim) || token < 0 || token >= page_size || dim < 0 ||
        dim >= head_dim)
        return -1;
    const int byte = values ? page_size * head_dim / 2 + sv::kv_value_byte(head_dim, token, dim)
                            : sv::kv_key_byte(head_dim, token, dim);
    return 2 * int64_t(byte) + (dim & 1);
}

sv_status spec_kv_append(const void *k, int64_t k_batch_stride, int64_t k_token_stride, int64_t k_head_stride,
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
    if (int64_t(T) * kv_heads > 0x7FFFFFFF || int64_t(T) * kv_heads * B > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;
    const int64_t items = int64_t(B) * T * kv_heads, per = sv::kAppThreads / (head_dim / 8);
    if (reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(k) % 2 || reinterpret_cast<uintptr_t>(v) % 2 ||
        reinterpret_cast<uintptr_t>(k_values) % 16 || reinterpret_cast<uintptr_t>(v_values) % 16)
        return SV_ERR_INVALID_ARG;
    const int64_t all = k_batch_stride | k_token_stride | k_head_stride | v_batch_stride | v_token_stride | v_head_stride;
    sv::AppendArgs a{};
    a.k = static_cast<const uint16_t *>(k), a.v = static_cast<const uint16_t *>(v);
    a.k_bs = k_batch_stride, a.k_ts = k_token_stride, a.k_hs = k_head_stride;
    a.v_bs = v_batch_stride, a.v_ts = v_token_stride, a.v_hs = v_head_stride;
    const bool bf16 = dtype == SV_KV_BF16;
    const bool grid = all % 8 == 0 && (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 16 == 0 &&
                      (!cos || (pairs % 4 == 0 && (reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) % 16 == 0));
    const sv::Layout layout = !grid ? sv::kAny : cos && interleaved ? sv::kNeighbours : cos && pairs % 8 ? sv::kAny : sv::kHalves;
    a.items = uint32_t(items), a.T = T, a.H = kv_heads;
    a.cache = static_cast<uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.table = page_table, a.start = start, a.new_lens = new_lens;
    a.rot = sv::Rotation{cos, sin, table_len, cos ? pairs : 0, interleaved != 0, positions};
    a.k_values = static_cast<uint16_t *>(k_values), a.v_values = static_cast<uint16_t *>(v_values);
    const unsigned blocks = unsigned((items + per - 1) / per);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (head_dim) {
    case 64: e = sv::launch_append<64>(a, layout, bf16, blocks, s); break;
    case 128: e = sv::launch_append<128>(a, layout, bf16, blocks, s); break;
    default: e = sv::launch_append<256>(a, layout, bf16, blocks, s); break;
    }
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
