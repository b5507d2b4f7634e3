// sv_kv8_attention.cu -- the C entry of the attention over the 8-bit paged cache: argument checks and workspace layout.
#include "sv_kv8_wide.cuh"

namespace sv {

template <>
cudaError_t launch_attention8_rows<64, 3>(const Att8Args &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention8_rows<64, 4>(const Att8Args &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention8_rows<128, 3>(const Att8Args &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention8_rows<128, 4>(const Att8Args &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention8_rows<256, 3>(const Att8Args &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_attention8_rows<256, 4>(const Att8Args &a, int grid, cudaStream_t s);

template <>
cudaError_t launch_wide8_of<64>(const Att8Args &a, int grid, cudaStream_t s);
template <>
cudaError_t launch_wide8_of<128>(const Att8Args &a, int grid, cudaStream_t s);

namespace {

// More rows than this a kv head go to the kernel for many rows.  4 kv heads, us in tiles of up to 64 rows and in one of 128; 64 sequences of up to 2047
// cached tokens: 64 dimensions 48 rows 57 and 66, 64 rows 68 and 66, 80 rows 99 and 73 (fp16 72 and 65, 104 and 71 for the last two); 128 dimensions 64 rows
// 75 and 90, 80 rows 107 and 91 (fp16 78 and 88, 115 and 89).  8 sequences of up to 8192: 64 dimensions 64 rows 38 and 41, 80 rows 48 and 45; 128 dimensions
// 64 rows 40 and 49, 80 rows 50 and 50.  One of 16384 has too few segments for tiles of 128 rows, 22 and 33, 23 and 31 for 96 rows, but how
// long the sequences are is on the GPU.  (bf16, rotated, unless it says fp16.)
constexpr int64_t kNarrowRows8 = 64;

struct Att8Layout {
    size_t desc, ml, acc, parts, see, total;
    int grid, nr, tile, see_words;  // blocks at most, rows and tokens a tile
    bool wide;
};
Att8Layout att8_layout(int B, int T, int H, int64_t rows, int D) {
    Att8Layout L;
    L.wide = wide8_has(D) && rows > kNarrowRows8;
    L.nr = L.wide ? kWideRows8 : att8_rows(rows, D);
    L.tile = L.wide ? wide8_tile(D) : kTile8;
    L.grid = kAttSMs * (L.wide ? wide8_occupancy(D) : att8_occupancy(D, L.nr));
    L.see_words = L.wide ? (T + 31) / 32 : (L.nr + 31) / 32;
    const int nr = L.nr;
    const size_t row_tiles = size_t((rows + nr - 1) / nr);
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    L.desc = 256;
    L.ml = up(L.desc + size_t(L.grid) * sizeof(AttDesc));
    L.acc = up(L.ml + size_t(2) * L.grid * nr * 8);
    L.parts = up(L.acc + size_t(2) * L.grid * nr * D * 4);
    L.see = up(L.parts + size_t(B) * H * row_tiles * query_bytes8(D, nr));
    L.total = up(L.see + (T <= SV_MAX_TREE_NODES ? row_tiles * (L.wide ? nr : T) * L.see_words * 4 : 0));
    return L;
}

}  // namespace
}  // namespace sv

extern "C" {

size_t spec_kv8_attention_workspace_size(int B, int T, int heads, int kv_heads, int head_dim) {
    if (B <= 0 || T <= 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || !sv::kv_head_dim_ok(head_dim)) return 0;
    return sv::att8_layout(B, T, kv_heads, int64_t(T) * (heads / kv_heads), head_dim).total;
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
    if (int64_t(table_width) * page_size > 0x7FFFFF80) return SV_ERR_INVALID_ARG;  // (rounded up to a tile of 128: 31 bits)
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
    const sv::Att8Layout L = sv::att8_layout(B, T, kv_heads, int64_t(T) * G, head_dim);
    if (!workspace || workspace_bytes < L.total || reinterpret_cast<uintptr_t>(workspace) % 16) return SV_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    const int nr = L.nr;
    const int64_t row_tiles = (int64_t(T) * G + nr - 1) / nr, tokens = int64_t(table_width) * page_size;
    const int64_t most = row_tiles * (tokens / L.tile + 1);  // units of a sequence and head
    if (most > 0x7FFFFFFF / kv_heads || most * kv_heads > 0x7FFFFFFF / B) return SV_ERR_INVALID_ARG;
    // no more blocks than the page tables have room for units: empty shares would only lengthen the joins
    const int64_t units = most * kv_heads * B;
    const int grid = units < L.grid ? int(units) : L.grid;
    const int64_t query_blocks = (int64_t(B) * kv_heads * row_tiles * nr * (head_dim / 8) + sv::kQueryThreads8 - 1) / sv::kQueryThreads8;
    if (query_blocks + row_tiles > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;
    sv::Att8Args a{};
    a.q = static_cast<const uint16_t *>(q);
    a.q_bs = q_batch_stride, a.q_ts = q_token_stride, a.q_hs = q_head_stride;
    a.bf16 = dtype == SV_KV_BF16;
    a.B = B, a.T = T, a.H = kv_heads, a.G = G;
    a.cache = static_cast<const uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.granule = 16;
    while (a.granule < L.tile && page_size % (2 * a.granule) == 0) a.granule *= 2;
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
    a.nr = nr, a.wide = L.wide, a.see_words = L.see_words, a.query_blocks = query_blocks;
    a.parts = reinterpret_cast<uint8_t *>(ws + L.parts), a.see = reinterpret_cast<uint32_t *>(ws + L.see);
    // a bf16 query has 8 bits, which two parts hold; what the rotation makes of it, and an fp16 one, takes three
    a.nq = cos || !a.bf16 ? 3 : 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (L.wide)
        e = head_dim == 64 ? sv::launch_wide8_of<64>(a, grid, s) : sv::launch_wide8_of<128>(a, grid, s);
    else if (head_dim == 64)
        e = a.bf16 ? sv::launch_attention8_rows<64, 3>(a, grid, s) : sv::launch_attention8_rows<64, 4>(a, grid, s);
    else if (head_dim == 128)
        e = a.bf16 ? sv::launch_attention8_rows<128, 3>(a, grid, s) : sv::launch_attention8_rows<128, 4>(a, grid, s);
    else
        e = a.bf16 ? sv::launch_attention8_rows<256, 3>(a, grid, s) : sv::launch_attention8_rows<256, 4>(a, grid, s);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
