// sv_kv_append.cu -- the new tokens' keys and values into the 4-bit paged cache, the position
// rotation of the keys applied on the way.
//
// D / 8 lanes take a (token, head): eight dimensions of its key and of its value each, one 16-byte load a
// row.  They rotate the key, reduce minimum and maximum over their lanes, and write the codes.  The result is
// that of the exact rule: rotated keys are double-float (a 16-bit input times an fp32 cosine is exact in
// two floats), and whatever lies so near a rounding border that 32 bits cannot tell -- about one scale
// in a thousand, one code in 50,000 -- is decided in 64.  Everything is read once and written once.
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
    int bf16, vec, rot_vec;  // rows, and the angles' rows, lie on the 16-byte grid
    int64_t items;  // B * T * H
    int T, H;
    uint8_t *cache;
    int num_pages, page, width;
    const int32_t *table, *start, *new_lens;
    Rotation rot;
    uint16_t *k_values, *v_values;
};

__device__ __forceinline__ float saturate(float x) { return fminf(fmaxf(x, -65504.f), 65504.f); }

// 1.5 * 2^23: added to a float of less than 2^22 it leaves the nearest integer (ties to even) in the low bits.
constexpr float kRound = 12582912.f;

// Quantises one head vector of 8 L dimensions, held as hi + lo by L lanes (eight each): the lane's codes, 4 bits
// each, and the scale and zero as fp16 bits in one word (scale low).
template <int L, bool kLow>
__device__ __forceinline__ uint32_t quantise(const float (&hi)[8], const float (&lo)[8], uint32_t &meta) {
    float low = hi[0], high = hi[0], size = fabsf(hi[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) low = fminf(low, hi[i]), high = fmaxf(high, hi[i]);
    bool bad = false;  // (fminf and fmaxf drop a NaN)
#pragma unroll
    for (int i = 0; i < 8; ++i) bad |= !(fabsf(hi[i]) <= 3.4e38f);
    if (bad) high = INFINITY;
#pragma unroll
    for (int o = L / 2; o; o >>= 1) {
        low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
        high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, o));
    }
    bad = !(high <= 3.4e38f);
    // zero = fp16(fp32(min)): the least hi is that fp32 number
    const float range = high - low, t = range * (1.f / 15.f);
    // scale = fp16(fp32(range / 15)): t is off by a few units of its last place, and by what the low parts
    // add; where that may matter, the quotient in 64 bits
    float off = t * 4.8e-7f;
    if (kLow) size = fmaxf(fabsf(low), fabsf(high)), off = fmaf(size, 2.4e-8f, off);
    const __half2 ends = __floats2half2_rn(saturate(t - off), saturate(t + off));
    uint32_t sb = __half_as_ushort(__low2half(ends));
    const bool doubt = !bad && sb != __half_as_ushort(__high2half(ends));
    if (__any_sync(0xFFFFFFFFu, doubt)) {  // (all lanes take part in the reductions)
        double least = 1e300, most = -1e300;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double x = double(hi[i]) + double(lo[i]);
            least = fmin(least, x), most = fmax(most, x);
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) {
            least = fmin(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
            most = fmax(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        }
        if (doubt) sb = __half_as_ushort(__float2half_rn(saturate(__double2float_rn((most - least) / 15.0))));
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
        // clamped before rounding, which changes no code; |q| <= 16 and a few roundings of 2^-24 each: in doubt
        // within 1e-5 of a border (a saturated zero or scale only meets the clamp)
        const float q = fminf(fmaxf(((hi[i] - z) + (kLow ? lo[i] : 0.f)) * inv, 0.f), 15.f);
        c[i] = q + kRound;
        near |= fabsf(q - (c[i] - kRound)) > 0.49999f;
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double q = ((double(hi[i]) - double(z)) + (kLow ? double(lo[i]) : 0.0)) / double(s);
            c[i] = float(rint(fmin(fmax(q, 0.0), 15.0))) + kRound;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= (__float_as_uint(c[i]) & 15u) << (4 * i);
    return codes;
}

// Eight 16-bit numbers (vec: 16-byte aligned).
__device__ __forceinline__ uint4 load_row(const uint16_t *p, bool vec) {
    if (vec) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = uint32_t(__ldg(p + 2 * i)) | uint32_t(__ldg(p + 2 * i + 1)) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void widen(const uint4 &v, bool bf16, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

// What the codes stand for.
__device__ __forceinline__ void store_values(uint16_t *p, uint32_t codes, uint32_t meta, bool live, bool bf16) {
    const float s = __half2float(__ushort_as_half(uint16_t(meta))), z = __half2float(__ushort_as_half(uint16_t(meta >> 16)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // s code is exact: one rounding, then that to the type
        const float x = fmaf(s, float(codes >> (8 * i) & 15u), z), y = fmaf(s, float(codes >> (8 * i + 4) & 15u), z);
        if (bf16) {
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
__device__ __forceinline__ void rotate(const AppendArgs &a, const uint16_t *kp, int d0, int64_t row, float (&x)[8], float (&lo)[8]) {
    const int pairs = a.rot.pairs;
    const float *cp = a.rot.cos + row, *sp = a.rot.sin + row;
    float y[8], c[8], s[8];
    if (!a.rot.interleaved && pairs % 8 == 0) {  // the eight lie within one half
        const bool low = d0 < pairs;
        const int e0 = low ? d0 : d0 - pairs;
        widen(load_row(kp + (low ? d0 + pairs : e0), a.vec), a.bf16, y);
        if (a.rot_vec) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(cp + e0 + i)), v = __ldg(reinterpret_cast<const float4 *>(sp + e0 + i));
                c[i] = u.x, c[i + 1] = u.y, c[i + 2] = u.z, c[i + 3] = u.w;
                s[i] = v.x, s[i + 1] = v.y, s[i + 2] = v.z, s[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = __ldg(cp + e0 + i), s[i] = __ldg(sp + e0 + i);
        }
        if (low) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = -s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int partner, angle;
            float sign;
            if (kv_partner(a.rot, d0 + i, partner, angle, sign)) {
                y[i] = a.rot.interleaved ? x[i ^ 1] : kv_to_float(__ldg(kp + partner), a.bf16);
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

template <int D>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const AppendArgs a) {
    constexpr int L = D / 8, kItems = kAppThreads / L;
    const int64_t item = int64_t(blockIdx.x) * kItems + threadIdx.x / L;
    griddep_launch_next();
    griddep_wait();
    const bool there = item < a.items;  // (the others only take part in the warp's reductions)
    const int64_t it = there ? item : 0;
    const int d0 = int(threadIdx.x % L) * 8;
    const uint32_t bt = uint32_t(it / a.H), h = uint32_t(it - int64_t(bt) * a.H);  // (the host has checked that B T fits)
    const uint32_t b = bt / uint32_t(a.T);
    const int t = int(bt - b * uint32_t(a.T));
    const int64_t capacity = int64_t(a.width) * a.page;
    int before, fresh;
    kv_lengths(a.start, a.new_lens, b, a.T, capacity, before, fresh);
    const bool live = there && t < fresh;
    uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
    const uint16_t *kp = a.k + b * a.k_bs + t * a.k_ts + h * a.k_hs, *vp = a.v + b * a.v_bs + t * a.v_ts + h * a.v_hs;
    int pg = -1, sl = 0;
    if (live) {
        kv = load_row(kp + d0, a.vec), vv = load_row(vp + d0, a.vec);
        const int64_t slot = int64_t(before) + t;
        if (slot < capacity) {
            const uint32_t pi = uint32_t(slot) / uint32_t(a.page);
            sl = int(uint32_t(slot) - pi * uint32_t(a.page));
            pg = __ldg(a.table + int64_t(b) * a.width + pi);
        }
    }
    float x[8], lo[8];
    uint32_t km, vm, kc, vc;
    widen(kv, a.bf16, x);
    if (a.rot.cos) {
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = 0.f;
        if (live && d0 < 2 * a.rot.pairs) rotate(a, kp, d0, kv_rotation_row(a.rot, bt, before + t), x, lo);
        kc = quantise<L, true>(x, lo, km);
    } else {
        kc = quantise<L, false>(x, x, km);
    }
    widen(vv, a.bf16, x);
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
    if (a.k_values) store_values(a.k_values + item * D + d0, kc, km, live, a.bf16);
    if (a.v_values) store_values(a.v_values + item * D + d0, vc, vm, live, a.bf16);
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
    if (int64_t(T) * kv_heads > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;  // (so that the next product fits 64 bits)
    if (int64_t(B) * T > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;
    const int64_t items = int64_t(B) * T * kv_heads, per = sv::kAppThreads / (head_dim / 8);
    if ((items + per - 1) / per > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(k) % 2 || reinterpret_cast<uintptr_t>(v) % 2 ||
        reinterpret_cast<uintptr_t>(k_values) % 16 || reinterpret_cast<uintptr_t>(v_values) % 16)
        return SV_ERR_INVALID_ARG;
    const int64_t all = k_batch_stride | k_token_stride | k_head_stride | v_batch_stride | v_token_stride | v_head_stride;
    sv::AppendArgs a{};
    a.k = static_cast<const uint16_t *>(k), a.v = static_cast<const uint16_t *>(v);
    a.k_bs = k_batch_stride, a.k_ts = k_token_stride, a.k_hs = k_head_stride;
    a.v_bs = v_batch_stride, a.v_ts = v_token_stride, a.v_hs = v_head_stride;
    a.bf16 = dtype == SV_KV_BF16;
    a.vec = all % 8 == 0 && (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 16 == 0;
    a.rot_vec = pairs % 4 == 0 && (reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) % 16 == 0;
    a.items = items, a.T = T, a.H = kv_heads;
    a.cache = static_cast<uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.table = page_table, a.start = start, a.new_lens = new_lens;
    a.rot = sv::Rotation{cos, sin, table_len, cos ? pairs : 0, interleaved != 0, positions};
    a.k_values = static_cast<uint16_t *>(k_values), a.v_values = static_cast<uint16_t *>(v_values);
    const unsigned blocks = unsigned((items + per - 1) / per);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (head_dim) {
    case 64: e = sv::launch_after(sv::kv_append_kernel<64>, blocks, sv::kAppThreads, 0, s, a); break;
    case 128: e = sv::launch_after(sv::kv_append_kernel<128>, blocks, sv::kAppThreads, 0, s, a); break;
    default: e = sv::launch_after(sv::kv_append_kernel<256>, blocks, sv::kAppThreads, 0, s, a); break;
    }
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
