// sv_kv_attention.cu -- the C entry of the attention over the 4-bit paged cache: argument checks and
// workspace layout.
#include "sv_kv_wide.cuh"

namespace sv {

#ifdef SV_CHECKS
__device__ int g_kv_lose = -1;
#endif

template <>
cudaError_t launch_attention_rows<64, false>(const AttArgs &a, int nr, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention_rows<64, true>(const AttArgs &a, int nr, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention_rows<128, false>(const AttArgs &a, int nr, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention_rows<128, true>(const AttArgs &a, int nr, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention_rows<256, false>(const AttArgs &a, int nr, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention_rows<256, true>(const AttArgs &a, int nr, int grid, cudaStream_t s);

template <int D, bool kExact>
cudaError_t launch_wide_of(const AttArgs &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_wide_of<64, false>(const AttArgs &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_wide_of<64, true>(const AttArgs &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_wide_of<128, false>(const AttArgs &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_wide_of<128, true>(const AttArgs &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_wide_of<256, false>(const AttArgs &a, int grid, cudaStream_t s);

namespace {

// More rows than this a kv head go to the kernel for many rows.  64 sequences of up to 2047 cached tokens, 4 query heads a kv head, us in
// tiles of up to 48 rows and in one of 128: 64 dimensions, bf16, 56 rows 67 and 64, 72 rows 75 and 67; 128 dimensions, bf16, 64 rows 90 and
// 120, 72 rows 107 and 122, 96 rows 161 and 122; the same, rotated fp16, 56 rows 137 and 145, 72 rows 185 and 150, 256 rows 608 and 291;
// 256 dimensions, bf16, 48 rows 147 and 194, 64 rows 184 and 200, 72 rows 216 and 206, 256 rows 717 and 402, but 26 and 36 for one
// sequence alone, whose blocks have a unit or two each.
constexpr int kNarrowRows = 64;
// Both parts of rotated fp16 queries of 256 dimensions do not fit its shared memory.
bool att_wide(int64_t rows, int D, bool exact) { return rows > kNarrowRows && !(D == 256 && exact); }

struct AttLayout {
    size_t desc, ml, acc, total;
    int grid;
};
AttLayout att_layout(int64_t rows, int D, bool wide) {
    const int nr = att_nr(rows, D), R = wide ? kWideRows : 8 * nr;
    AttLayout L;
    L.grid = kAttSMs * (wide ? wide_occupancy(D) : att_occupancy(D, nr));
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    L.desc = 256;
    L.ml = up(L.desc + size_t(L.grid) * sizeof(AttDesc));
    L.acc = up(L.ml + size_t(2) * L.grid * R * 8);
    L.total = up(L.acc + size_t(2) * L.grid * R * D * 4);
    return L;
}

}  // namespace
}  // namespace sv

extern "C" {

size_t spec_kv_attention_workspace_size(int B, int T, int heads, int kv_heads, int head_dim) {
    if (B <= 0 || T <= 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || !sv::kv_head_dim_ok(head_dim)) return 0;
    const int64_t rows = int64_t(T) * (heads / kv_heads);
    const size_t plain = sv::att_layout(rows, head_dim, sv::att_wide(rows, head_dim, false)).total;
    const size_t exact = sv::att_layout(rows, head_dim, sv::att_wide(rows, head_dim, true)).total;
    return plain > exact ? plain : exact;
}

sv_status spec_kv_attention(const void *q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
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
    const int G = heads / kv_heads;
    const int64_t rows = int64_t(T) * G;
    // rotated fp16 queries are multiplied in two parts
    const bool exact = cos && dtype == SV_KV_FP16, wide = sv::att_wide(rows, head_dim, exact);
    const sv::AttLayout L = sv::att_layout(rows, head_dim, wide);
    if (!workspace || workspace_bytes < L.total || reinterpret_cast<uintptr_t>(workspace) % 16) return SV_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    const int nr = sv::att_nr(rows, head_dim), R = wide ? sv::kWideRows : 8 * nr;
    const int unit = wide ? sv::kWideTokens : sv::att_tokens(head_dim, nr);
    const int64_t row_tiles = (rows + R - 1) / R, tokens = int64_t(table_width) * page_size;
    const int64_t most = row_tiles * (tokens / unit + 1);  // units of a sequence and head
    if (most > 0x7FFFFFFF / kv_heads || most * kv_heads > 0x7FFFFFFF / B) return SV_ERR_INVALID_ARG;
    // no more CTAs than the page tables have room for units: empty shares would only lengthen the joins
    const int64_t units = most * kv_heads * B;
    const int grid = units < L.grid ? int(units) : L.grid;
    sv::AttArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.q_bs = q_batch_stride, a.q_ts = q_token_stride, a.q_hs = q_head_stride;
    a.bf16 = dtype == SV_KV_BF16;
    a.B = B, a.T = T, a.H = kv_heads, a.G = G;
    a.cache = static_cast<const uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.granule = 16;
    while (a.granule < unit && page_size % (2 * a.granule) == 0) a.granule *= 2;
    a.vec = (q_batch_stride | q_token_stride | q_head_stride) % 8 == 0 && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    a.rot_vec = cos && pairs % 4 == 0 && (reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) % 16 == 0;
    a.table = page_table, a.start = start, a.new_lens = new_lens, a.parent = parent;
    a.scale = scale;
    a.rot = sv::Rotation{cos, sin, table_len, cos ? pairs : 0, interleaved != 0, positions};
    a.out = static_cast<uint16_t *>(out);
    a.row_tiles = int(row_tiles);
    a.status = reinterpret_cast<int *>(ws);
    a.desc = reinterpret_cast<sv::AttDesc *>(ws + L.desc);
    a.ml = reinterpret_cast<float2 *>(ws + L.ml);
    a.acc = reinterpret_cast<float *>(ws + L.acc);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (wide)
        e = head_dim == 256 ? sv::launch_wide_of<256, false>(a, grid, s)
            : head_dim == 128 ? exact ? sv::launch_wide_of<128, true>(a, grid, s) : sv::launch_wide_of<128, false>(a, grid, s)
            : exact         ? sv::launch_wide_of<64, true>(a, grid, s)
                            : sv::launch_wide_of<64, false>(a, grid, s);
    else if (head_dim == 64)
        e = exact ? sv::launch_attention_rows<64, true>(a, nr, grid, s) : sv::launch_attention_rows<64, false>(a, nr, grid, s);
    else if (head_dim == 128)
        e = exact ? sv::launch_attention_rows<128, true>(a, nr, grid, s) : sv::launch_attention_rows<128, false>(a, nr, grid, s);
    else
        e = exact ? sv::launch_attention_rows<256, true>(a, nr, grid, s) : sv::launch_attention_rows<256, false>(a, nr, grid, s);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

sv_status spec_kv_lose_unit(int unit) {
#ifdef SV_CHECKS
    return cudaMemcpyToSymbol(sv::g_kv_lose, &unit, sizeof(unit)) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
#else
    (void)unit;
    return SV_ERR_UNSUPPORTED;
#endif
}

}  // extern "C"
