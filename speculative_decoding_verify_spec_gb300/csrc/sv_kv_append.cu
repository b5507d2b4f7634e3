// sv_kv_append.cu -- the new tokens' keys and values into the 4-bit paged cache, the position
// rotation of the keys applied on the way.
//
// One warp per (token, head): it loads the key and the value (D / 32 dimensions a lane), rotates
// the key, reduces minimum and maximum with one warp reduction each, and writes the codes.  The
// result is that of the exact rule: rotated keys are double-float (a 16-bit input times an fp32
// cosine is exact in two floats), and whatever lies so near a rounding border that 32 bits cannot
// tell -- about one scale in a thousand, one code in 50,000 -- is decided in 64.  Everything is
// read once and written once.
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
    int bf16, vec;  // vec: rows lie on the lanes' vector grid
    int64_t items;  // B * T * H
    int T, H;
    uint8_t *cache;
    int num_pages, page, width;
    const int32_t *table, *start, *new_lens;
    Rotation rot;
    uint16_t *k_values, *v_values;
};

// Order-preserving map of floats to unsigned.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

__device__ __forceinline__ uint16_t half_sat(float x) {
    return __half_as_ushort(__float2half_rn(fminf(fmaxf(x, -65504.f), 65504.f)));
}
__device__ __noinline__ uint16_t scale_exact(double x) { return half_sat(__double2float_rn(x)); }

// Quantises one head vector held as hi + lo (E dimensions a lane): the lane's codes (4 bits each),
// and the scale and zero as fp16 bits in one word (scale low).
template <int E>
__device__ __forceinline__ uint32_t quantise(const float (&hi)[E], const float (&lo)[E], bool two, uint32_t &meta) {
    float mnh = hi[0], mnl = lo[0], mxh = hi[0], mxl = lo[0];
    bool bad = !(fabsf(hi[0]) <= 3.4e38f);
#pragma unroll
    for (int i = 1; i < E; ++i) {
        bad |= !(fabsf(hi[i]) <= 3.4e38f);
        if (hi[i] < mnh || (hi[i] == mnh && lo[i] < mnl)) mnh = hi[i], mnl = lo[i];
        if (hi[i] > mxh || (hi[i] == mxh && lo[i] > mxl)) mxh = hi[i], mxl = lo[i];
    }
    if (__any_sync(0xFFFFFFFFu, bad)) {
        meta = 0x7E007E00u;  // NaN, NaN
        return 0;
    }
    const uint32_t kn = __reduce_min_sync(0xFFFFFFFFu, key_of(mnh)), kx = __reduce_max_sync(0xFFFFFFFFu, key_of(mxh));
    if (two) {
        const uint32_t ln = __reduce_min_sync(0xFFFFFFFFu, key_of(mnh) == kn ? key_of(mnl) : 0xFFFFFFFFu);
        const uint32_t lx = __reduce_max_sync(0xFFFFFFFFu, key_of(mxh) == kx ? key_of(mxl) : 0u);
        mnl = of_key(ln), mxl = of_key(lx);
    } else {
        mnl = mxl = 0.f;
    }
    mnh = of_key(kn), mxh = of_key(kx);
    // zero = fp16(fp32(min)): hi is that fp32 number
    uint16_t zb = half_sat(mnh);
    // scale = fp16(fp32(range / 15)): the fp32 quotient below is off by a few units of its last
    // place at most, which matters next to a midpoint of fp16
    const float range = (mxh - mnh) + (mxl - mnl);
    const float t = range * (1.f / 15.f);
    uint16_t sb = half_sat(t);
    const int low = int(__float_as_uint(t) & 0x1FFFu) - 0x1000;
    if ((low >= -8 && low <= 8) || t < 6.2e-5f || !(t < 65000.f))
        sb = scale_exact(((double(mxh) - double(mnh)) + (double(mxl) - double(mnl))) / 15.0);
    if (sb == 0) sb = 1;  // 2^-24
    if (zb == 0x8000u) zb = 0;
    meta = uint32_t(zb) << 16 | sb;
    const float z = __half2float(__ushort_as_half(zb)), s = __half2float(__ushort_as_half(sb));
    const float inv = __frcp_rn(s);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float q = ((hi[i] - z) + lo[i]) * inv;
        float c = rintf(q);
        // |q| <= 16 and a few roundings of 2^-24 each: in doubt within 1e-5 of a border (a saturated
        // zero or scale only meets the clamp)
        if (fabsf(fabsf(q - c) - 0.5f) < 1e-5f)
            c = float(rint(((double(hi[i]) - double(z)) + double(lo[i])) / double(s)));
        c = fminf(fmaxf(c, 0.f), 15.f);
        codes |= uint32_t(int(c)) << (4 * i);
    }
    return codes;
}

template <int E>
__device__ __forceinline__ void load_row(const uint16_t *p, int d0, int vec, uint16_t (&x)[E]) {
    if (vec) {
        if constexpr (E == 8) {
            const uint4 w = *reinterpret_cast<const uint4 *>(p + d0);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = uint16_t(u[i / 2] >> (16 * (i & 1)));
        } else if constexpr (E == 4) {
            const uint2 w = *reinterpret_cast<const uint2 *>(p + d0);
            x[0] = uint16_t(w.x), x[1] = uint16_t(w.x >> 16), x[2] = uint16_t(w.y), x[3] = uint16_t(w.y >> 16);
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(p + d0);
            x[0] = uint16_t(w), x[1] = uint16_t(w >> 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = p[d0 + i];
    }
}

template <int E>
__device__ __forceinline__ void store_values(uint16_t *p, int d0, uint32_t codes, uint32_t meta, bool live, bool bf16) {
    const float s = __half2float(__ushort_as_half(uint16_t(meta))), z = __half2float(__ushort_as_half(uint16_t(meta >> 16)));
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float x = live ? fmaf(s, float(codes >> (4 * i) & 15u), z) : 0.f;  // s code is exact: one rounding
        const uint32_t u = kv_from_float(x, bf16);
        w[i / 2] = i & 1 ? w[i / 2] | u << 16 : u;
    }
    if constexpr (E == 8) *reinterpret_cast<uint4 *>(p + d0) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (E == 4) *reinterpret_cast<uint2 *>(p + d0) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(p + d0) = w[0];
}

template <int D>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const AppendArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = int64_t(blockIdx.x) * (kAppThreads / 32) + (threadIdx.x >> 5);
    griddep_launch_next();
    griddep_wait();
    if (item >= a.items) return;
    const int h = int(item % a.H);
    const int64_t bt = item / a.H;
    const int t = int(bt % a.T);
    const int64_t b = bt / a.T;
    const int d0 = lane * E;
    const int64_t capacity = int64_t(a.width) * a.page;
    int before, fresh;
    kv_lengths(a.start, a.new_lens, b, a.T, capacity, before, fresh);
    const bool live = t < fresh;
    uint32_t kc = 0, km = 0, vc = 0, vm = 0;
    if (live) {
        const uint16_t *kp = a.k + b * a.k_bs + t * a.k_ts + h * a.k_hs, *vp = a.v + b * a.v_bs + t * a.v_ts + h * a.v_hs;
        uint16_t kx[E], vx[E];
        load_row<E>(kp, d0, a.vec, kx);
        load_row<E>(vp, d0, a.vec, vx);
        float hi[E], lo[E];
        bool two = false;
        if (a.rot.cos) {
            two = true;
            const int64_t row = kv_rotation_row(a.rot, bt, before + t);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float x = kv_to_float(kx[i], a.bf16);
                int partner, angle;
                float sign;
                if (kv_partner(a.rot, d0 + i, partner, angle, sign)) {
                    const float c = __ldg(a.rot.cos + row + angle), s = sign * __ldg(a.rot.sin + row + angle);
                    const float y = kv_to_float(__ldg(kp + partner), a.bf16);
                    // x c + y s in two floats: both products exact, their sum exact, then the rest
                    const float p = __fmul_rn(x, c), pe = __fmaf_rn(x, c, -p);
                    const float r = __fmul_rn(y, s), re = __fmaf_rn(y, s, -r);
                    const float sum = __fadd_rn(p, r), bb = __fsub_rn(sum, p);
                    const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, bb)), __fsub_rn(r, bb));
                    const float rest = __fadd_rn(e, __fadd_rn(pe, re));
                    hi[i] = __fadd_rn(sum, rest);
                    lo[i] = __fsub_rn(rest, __fsub_rn(hi[i], sum));
                } else {
                    hi[i] = x, lo[i] = 0.f;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) hi[i] = kv_to_float(kx[i], a.bf16), lo[i] = 0.f;
        }
        kc = quantise<E>(hi, lo, two, km);
#pragma unroll
        for (int i = 0; i < E; ++i) hi[i] = kv_to_float(vx[i], a.bf16), lo[i] = 0.f;
        vc = quantise<E>(hi, lo, false, vm);
        const int64_t slot = int64_t(before) + t;
        if (slot < capacity) {
            const int pg = __ldg(a.table + b * a.width + slot / a.page);
            const int sl = int(slot % a.page);
            if (pg >= 0 && pg < a.num_pages && SV_IN(kv_value_byte(D, sl, d0) + (E == 8 ? 33 : E / 2 - 1), a.page * D / 2)) {
                uint8_t *base = a.cache + (int64_t(pg) * a.H + h) * kv_page_bytes(a.page, D);
                uint8_t *kd = base + kv_key_byte(D, sl, d0), *vd = base + a.page * D / 2 + kv_value_byte(D, sl, d0);
                if constexpr (E == 8) {
                    *reinterpret_cast<uint32_t *>(kd) = kc;
                    *reinterpret_cast<uint16_t *>(vd) = uint16_t(vc);
                    *reinterpret_cast<uint16_t *>(vd + 32) = uint16_t(vc >> 16);  // the next four dimensions
                } else if constexpr (E == 4) {
                    *reinterpret_cast<uint16_t *>(kd) = uint16_t(kc);
                    *reinterpret_cast<uint16_t *>(vd) = uint16_t(vc);
                } else {
                    *kd = uint8_t(kc);
                    *vd = uint8_t(vc);
                }
                if (lane == 0) {
                    *reinterpret_cast<uint32_t *>(base + kv_key_scale_byte(a.page, D, sl)) = km;
                    *reinterpret_cast<uint32_t *>(base + kv_value_scale_byte(a.page, D, sl)) = vm;
                }
            }
        }
    }
    if (a.k_values) store_values<E>(a.k_values + item * D, d0, kc, km, live, a.bf16);
    if (a.v_values) store_values<E>(a.v_values + item * D, d0, vc, vm, live, a.bf16);
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
    const int64_t items = int64_t(B) * T * kv_heads, per = sv::kAppThreads / 32;
    if ((items + per - 1) / per > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(k) % 2 || reinterpret_cast<uintptr_t>(v) % 2 ||
        reinterpret_cast<uintptr_t>(k_values) % 16 || reinterpret_cast<uintptr_t>(v_values) % 16)
        return SV_ERR_INVALID_ARG;
    const int64_t grid = head_dim / 32;  // elements of a lane's vector
    const int64_t all = k_batch_stride | k_token_stride | k_head_stride | v_batch_stride | v_token_stride | v_head_stride;
    sv::AppendArgs a{};
    a.k = static_cast<const uint16_t *>(k), a.v = static_cast<const uint16_t *>(v);
    a.k_bs = k_batch_stride, a.k_ts = k_token_stride, a.k_hs = k_head_stride;
    a.v_bs = v_batch_stride, a.v_ts = v_token_stride, a.v_hs = v_head_stride;
    a.bf16 = dtype == SV_KV_BF16;
    a.vec = all % grid == 0 && (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % (2 * grid) == 0;
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
