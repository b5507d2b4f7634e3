// sv_kv8_attention.cu -- the new tokens' attention over the 8-bit paged cache: C entry and kernel.
//
// A warp takes a query row (one new token's one head) and goes over the cached tokens with the running maximum and sum of
// the softmax; lanes have D / 32 dimensions each.
#include <cstdint>

#include "sv_checks.cuh"
#include "sv_device.cuh"
#include "sv_kv8.cuh"

namespace sv {
namespace {

struct Att8Args {
    const uint16_t *q;
    int64_t q_bs, q_ts, q_hs;
    int bf16, B, T, H, G;
    const uint8_t *cache;
    int num_pages, page, width;
    const int32_t *table, *start, *new_lens, *parent;
    float scale;
    Rotation rot;
    uint16_t *out;
};

template <int D>
__global__ void __launch_bounds__(128) kv8_attention_kernel(const Att8Args a, int64_t rows) {
    constexpr int E = D / 32;
    const int64_t item = int64_t(blockIdx.x) * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    griddep_launch_next();
    griddep_wait();
    if (item >= rows) return;
    const int heads = a.H * a.G, head = int(item % heads), t = int(item / heads % a.T), b = int(item / heads / a.T), h = head / a.G;
    const int64_t capacity = int64_t(a.width) * a.page;
    int before, fresh;
    kv_lengths(a.start, a.new_lens, b, a.T, capacity, before, fresh);
    const int64_t len = min(int64_t(before) + fresh, capacity);
    float q[E], o[E], m = -INFINITY, l = 0.f;
    const uint16_t *qp = a.q + b * a.q_bs + t * a.q_ts + head * a.q_hs;
    for (int i = 0; i < E; ++i) {
        const int d = lane * E + i;
        q[i] = kv_to_float(qp[d], a.bf16), o[i] = 0.f;
        int partner, angle;
        float sign;
        if (a.rot.cos && kv_partner(a.rot, d, partner, angle, sign)) {
            const int64_t at = kv_rotation_row(a.rot, int64_t(b) * a.T + t, before, t) + angle;
            q[i] = fmaf(q[i], a.rot.cos[at], sign * kv_to_float(qp[partner], a.bf16) * a.rot.sin[at]);
        }
        q[i] *= a.scale;
    }
    for (int64_t j = 0; j < len && t < fresh; ++j) {
        const int x = int(j - before);  // among the new tokens
        bool see = x < 0 || x == t;
        if (x >= 0 && !see) {
            if (!a.parent) {
                see = x < t;
            } else {
                for (int v = t; v > x;) {
                    const int up = a.parent[v];
                    v = up < v ? up : -1;
                    see |= v == x;
                }
            }
        }
        if (!see) continue;
        const int pg = a.table[int64_t(b) * a.width + j / a.page], sl = int(j % a.page);
        if (pg < 0 || pg >= a.num_pages) continue;
        const uint8_t *base = a.cache + (int64_t(pg) * a.H + h) * kv8_page_bytes(a.page, D);
        const uint32_t *w = reinterpret_cast<const uint32_t *>(base + kv8_word_byte(a.page, D, sl, 0));
        const float ks = (w[0] | w[1]) >> (sl & 15) & 1u ? NAN : __uint_as_float(w[0] & 0xFFFF0000u), vs = __uint_as_float(w[1] & 0xFFFF0000u);
        float s = 0.f;
        for (int i = 0; i < E; ++i) s = fmaf(q[i], kv8_numbers(base[kv8_code_byte(D, sl, lane * E + i)]).x, s);
        for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
        s *= ks;
        const float top = fmaxf(m, s), keep = m == -INFINITY ? 1.f : expf(m - top), p = expf(s - (top == -INFINITY ? 0.f : top));
        l = fmaf(l, keep, p);
        for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], keep, p * vs * kv8_numbers(base[a.page * D + kv8_code_byte(D, sl, lane * E + i)]).x);
        m = top;
    }
    uint16_t *out = a.out + ((int64_t(b) * a.T + t) * heads + head) * D + lane * E;
    for (int i = 0; i < E; ++i) out[i] = kv_from_float(l == 0.f ? 0.f : o[i] / l, a.bf16);
}

}  // namespace
}  // namespace sv

extern "C" {

size_t spec_kv8_attention_workspace_size(int B, int T, int heads, int kv_heads, int head_dim) {
    if (B <= 0 || T <= 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || !sv::kv_head_dim_ok(head_dim)) return 0;
    return 256;
}

sv_status spec_kv8_attention(const void *q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
                             sv_kv_dtype dtype, int B, int T, int heads, int kv_heads, int head_dim, const void *cache,
                             int num_pages, int page_size, const int32_t *page_table, int table_width,
                             const int32_t *start, const int32_t *new_lens, const int32_t *parent, float scale,
                             const float *cos, const float *sin, int table_len, int pairs, int interleaved,
                             const int32_t *positions, void *out, void *workspace, size_t workspace_bytes, void *stream) {
    if (dtype != SV_KV_BF16 && dtype != SV_KV_FP16) return SV_ERR_UNSUPPORTED;
    if (!sv::kv_head_dim_ok(head_dim) || !sv::kv_page_size_ok(page_size)) return SV_ERR_UNSUPPORTED;
    if (B < 0 || T < 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || num_pages < 0 || table_width < 0)
        return SV_ERR_INVALID_ARG;
    if (q_batch_stride < 0 || q_token_stride < 0 || q_head_stride < 0) return SV_ERR_INVALID_ARG;
    if (int64_t(table_width) * page_size > 0x7FFFFF80) return SV_ERR_INVALID_ARG;  // (rounded up to a unit of 128: 31 bits)
    if (parent && T > SV_MAX_TREE_NODES) return SV_ERR_INVALID_ARG;
    if (int64_t(T) * heads > 0x3FFFFFFF) return SV_ERR_INVALID_ARG;
    if (!(scale - scale == 0.f)) return SV_ERR_INVALID_ARG;
    if (!cos != !sin) return SV_ERR_INVALID_ARG;
    if (cos && (table_len < 1 || pairs < 1 || pairs > head_dim / 2)) return SV_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return SV_OK;
    if (!q || !out || !start || (table_width > 0 && !page_table) || (num_pages > 0 && !cache)) return SV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(q) % 2 || reinterpret_cast<uintptr_t>(out) % 16)
        return SV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < 256 || reinterpret_cast<uintptr_t>(workspace) % 16) return SV_ERR_WORKSPACE;
    const int64_t rows = int64_t(T) * heads * B;
    if (rows > 0x7FFFFFF0) return SV_ERR_INVALID_ARG;
    sv::Att8Args a{};
    a.q = static_cast<const uint16_t *>(q);
    a.q_bs = q_batch_stride, a.q_ts = q_token_stride, a.q_hs = q_head_stride;
    a.bf16 = dtype == SV_KV_BF16;
    a.B = B, a.T = T, a.H = kv_heads, a.G = heads / kv_heads;
    a.cache = static_cast<const uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.table = page_table, a.start = start, a.new_lens = new_lens, a.parent = parent;
    a.scale = scale;
    a.rot = sv::Rotation{cos, sin, table_len, cos ? pairs : 0, interleaved != 0, positions};
    a.out = static_cast<uint16_t *>(out);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned blocks = unsigned((rows + 3) / 4);
    if (cudaMemsetAsync(workspace, 0, 4, s) != cudaSuccess) return SV_ERR_CUDA;
    const cudaError_t e = head_dim == 64    ? sv::launch_after(sv::kv8_attention_kernel<64>, blocks, 128u, 0, s, a, rows)
                          : head_dim == 128 ? sv::launch_after(sv::kv8_attention_kernel<128>, blocks, 128u, 0, s, a, rows)
                                            : sv::launch_after(sv::kv8_attention_kernel<256>, blocks, 128u, 0, s, a, rows);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
