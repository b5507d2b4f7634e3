// sv_kv8_read.cu -- tokens of the 8-bit paged cache back in 16 bits.
//
// A warp takes eight tokens of a sequence and one head, keys and values: lane l token l % 8 and the 16-byte pieces
// l / 8, l / 8 + 4, ..  Of a range of tokens the eight are those of one group in the cache, so that a load of the warp is four runs of 128
// bytes; every lane writes 32 bytes of a row.  All loads go out before the first conversion.  Each byte is read and
// written once: the copy bandwidth is what bounds it.  Measured: 4 x 20001 tokens, 8 heads of 128, 74 us, 6.6 TB/s (98 % of a plain copy's rate).
#include <cstdint>

#include "sv_checks.cuh"
#include "sv_device.cuh"
#include "sv_kv8.cuh"

namespace sv {
namespace {

constexpr int kReadThreads = 256;

struct ReadArgs {
    const uint8_t *cache;
    int num_pages, page, width;
    const int32_t *table, *start, *lens, *slots;
    int T, H;
    uint32_t groups, items;  // groups of eight tokens a sequence; B * groups * H
    uint16_t *k, *v;
    bool whole;  // k and v on the 32-byte grid
};

template <int D, bool kBF16>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(const ReadArgs a) {
    constexpr int N = D / 64;
    const uint32_t item = blockIdx.x * (kReadThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x & 31, tok = lane & 7;
    griddep_launch_next();
    griddep_wait();
    if (item >= a.items) return;
    const uint32_t bg = item / uint32_t(a.H), h = item - bg * uint32_t(a.H), b = bg / a.groups;
    const int g = int(bg - b * a.groups);
    const int64_t capacity = int64_t(a.width) * a.page;
    int before, count;
    kv_lengths(a.start, a.lens, b, a.T, capacity, before, count);
    const int t = a.slots ? 8 * g + tok : 8 * g + tok - (before & 7);
    if (t < 0 || t >= a.T) return;
    int64_t slot = -1;
    if (t < count) slot = a.slots ? int64_t(a.slots[int64_t(b) * a.T + t]) : int64_t(before) + t;
    int pg = -1, sl = 0;
    if (slot >= 0 && slot < capacity) {
        const uint32_t pi = uint32_t(slot) / uint32_t(a.page);
        sl = int(uint32_t(slot) - pi * uint32_t(a.page));
        pg = __ldg(a.table + int64_t(b) * a.width + pi);
    }
    const bool here = pg >= 0 && pg < a.num_pages && SV_IN(kv8_code_byte(D, sl, D - 1), a.page * D);
    const int d0 = lane / 8 * 16;
    uint4 code[2][N];
    uint2 word = make_uint2(0, 0);
    if (here) {
        const uint8_t *base = a.cache + (int64_t(pg) * a.H + h) * kv8_page_bytes(a.page, D);
        word = __ldcg(reinterpret_cast<const uint2 *>(base + kv8_word_byte(a.page, D, sl, 0)));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < N; ++n)
                code[i][n] = __ldcg(reinterpret_cast<const uint4 *>(base + i * a.page * D + kv8_code_byte(D, sl, d0 + 64 * n)));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < N; ++n) code[i][n] = make_uint4(0, 0, 0, 0);
    }
    const int64_t at = ((int64_t(b) * a.T + t) * a.H + h) * D + d0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w = i ? word.y : word.x;
        const float s = w >> (sl & 15) & 1u ? NAN : __uint_as_float(w & 0xFFFF0000u);
        uint16_t *out = (i ? a.v : a.k) + at;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t c[4] = {code[i][n].x, code[i][n].y, code[i][n].z, code[i][n].w};
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = kv8_numbers(c[j]), y = kv8_numbers(c[j] >> 16);
                o[2 * j] = kv8_pack<kBF16>(x.x * s, x.y * s), o[2 * j + 1] = kv8_pack<kBF16>(y.x * s, y.y * s);
            }
            kv8_store_row(out + 64 * n, o, a.whole);
        }
    }
}

template <int D>
cudaError_t launch_read(const ReadArgs &a, bool bf16, cudaStream_t s) {
    const unsigned blocks = (a.items + kReadThreads / 32 - 1) / (kReadThreads / 32);
    return bf16 ? launch_after(kv8_read_kernel<D, true>, blocks, unsigned(kReadThreads), 0, s, a)
                : launch_after(kv8_read_kernel<D, false>, blocks, unsigned(kReadThreads), 0, s, a);
}

}  // namespace
}  // namespace sv

extern "C" {

size_t spec_kv8_page_bytes(int page_size, int head_dim) {
    if (!sv::kv_page_size_ok(page_size) || !sv::kv_head_dim_ok(head_dim)) return 0;
    return size_t(sv::kv8_page_bytes(page_size, head_dim));
}

int64_t spec_kv8_code_offset(int page_size, int head_dim, int values, int token, int dim) {
    if (!sv::kv_page_size_ok(page_size) || !sv::kv_head_dim_ok(head_dim) || token < 0 || token >= page_size || dim < 0 ||
        dim >= head_dim)
        return -1;
    return int64_t(values ? page_size * head_dim : 0) + sv::kv8_code_byte(head_dim, token, dim);
}

sv_status spec_kv8_read(const void *cache, int num_pages, int page_size, int B, int T, int kv_heads, int head_dim,
                        const int32_t *page_table, int table_width, const int32_t *start, const int32_t *lens,
                        const int32_t *slots, sv_kv_dtype dtype, void *k, void *v, void *stream) {
    if (dtype != SV_KV_BF16 && dtype != SV_KV_FP16) return SV_ERR_UNSUPPORTED;
    if (!sv::kv_head_dim_ok(head_dim) || !sv::kv_page_size_ok(page_size)) return SV_ERR_UNSUPPORTED;
    if (B < 0 || T < 0 || kv_heads < 1 || num_pages < 0 || table_width < 0) return SV_ERR_INVALID_ARG;
    if (int64_t(table_width) * page_size > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return SV_OK;
    if (!k || !v || !start || (table_width > 0 && !page_table) || (num_pages > 0 && !cache)) return SV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(k) % 16 || reinterpret_cast<uintptr_t>(v) % 16)
        return SV_ERR_INVALID_ARG;
    const int64_t groups = (int64_t(T) + 14) / 8;  // (a range may begin at a group's last slot)
    if (groups * kv_heads > 0x7FFFFFF0 || groups * kv_heads * B > 0x7FFFFFF0) return SV_ERR_INVALID_ARG;
    sv::ReadArgs a{};
    a.cache = static_cast<const uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.table = page_table, a.start = start, a.lens = lens, a.slots = slots;
    a.T = T, a.H = kv_heads, a.groups = uint32_t(groups), a.items = uint32_t(groups * kv_heads * B);
    a.k = static_cast<uint16_t *>(k), a.v = static_cast<uint16_t *>(v);
    a.whole = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 32 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == SV_KV_BF16;
    const cudaError_t e = head_dim == 64    ? sv::launch_read<64>(a, bf16, s)
                          : head_dim == 128 ? sv::launch_read<128>(a, bf16, s)
                                            : sv::launch_read<256>(a, bf16, s);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
