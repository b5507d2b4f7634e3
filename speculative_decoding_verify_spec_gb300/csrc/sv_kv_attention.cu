// sv_kv_attention.cu -- the new tokens' attention over the 4-bit paged cache.
//
// For a query row q (one of the T x G rows that share a kv head) and cached tokens j with key
// k_j = z_j + s_j code_j and value likewise,
//   x_j = scale (s_j (q . code_j) + z_j sum(q)),  p_j = exp(x_j - m),
//   out = [ sum_j (p_j s'_j) code'_j + sum_j p_j z'_j ] / sum_j p_j,
// so the matrix products run on the bare codes (exact in fp16) and each token's scale and zero
// cost a multiply-add per score instead of one per dimension.
//
// Work: a unit is 64 tokens for one (sequence, kv head, tile of 16 MT rows).  All units of the
// batch form one list; each CTA takes an equal, contiguous share of it, so ragged lengths balance
// by themselves and a long context spreads over the card.  A segment (one sequence, head, row
// tile) that ends up whole in a CTA is written out there; the others leave partial results
// that combine_kernel joins.
//
// A CTA has D / 32 warps.  Each scores its part of the 64 tokens for all rows, the weights go
// through shared memory, and each warp accumulates its own 32 dimensions over all 64 tokens: a
// key or value code is unpacked once per row tile and the accumulators need no joining.  The
// running maximum moves only when a score passes it by 2^8 (the weights fit fp16 either way),
// which leaves one barrier per unit.
#include <cstdint>

#include "sv_checks.cuh"
#include "sv_device.cuh"
#include "sv_grid.cuh"
#include "sv_kv.cuh"

namespace sv {
namespace {

constexpr int kNT = 64;                 // tokens per unit
constexpr int kStages = 4;              // units in flight per CTA
constexpr float kLazy = 8.f;            // log2 of how far a weight may pass 1
constexpr uint64_t kCopyLimitNs = 1000000000ull;
constexpr int kAttSMs = 152;

constexpr int att_occupancy(int D, int MT) {  // CTAs per SM: by registers and shared memory
    return D == 64 ? (MT == 4 ? 4 : 8) : D == 128 ? (MT == 1 ? 4 : MT == 2 ? 3 : 2) : (MT == 4 ? 1 : 2);
}
inline int att_mt(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

struct AttArgs {
    const uint16_t *q;
    int64_t q_bs, q_ts, q_hs;
    int bf16;
    int B, T, H, G;  // H kv heads, G query heads each
    const uint8_t *cache;
    int num_pages, page, width, granule;  // granule: tokens per copy, a power of two dividing page and 64
    const int32_t *table, *start, *new_lens, *parent;
    float scale;
    Rotation rot;
    uint16_t *out;
    int row_tiles;
    int *status;
    struct AttDesc *desc;  // [grid]
    float2 *ml;            // [2 grid][R] running maximum (log2) and sum
    float *acc;            // [2 grid][R][D]
};

// The first segment of a CTA's share, for the joining kernel.
struct AttDesc {
    int64_t lo, hi, total;  // the segment's units, and all units
    int b, h, rt, fresh;
};

// Where a CTA's share begins.
__host__ __device__ inline int64_t share_begin(int64_t total, int64_t c, int64_t n) { return c * total / n; }
__device__ __forceinline__ int64_t share_owner(int64_t total, int64_t u, int64_t n) { return ((u + 1) * n - 1) / total; }

struct SeqWork {
    int before, fresh, len;
    int tiles;       // units of a live segment
    int live;        // row tiles with a live row
    int64_t units;   // of the whole sequence
};
__device__ __forceinline__ SeqWork seq_work(const AttArgs &a, int64_t b, int R) {
    SeqWork w;
    const int64_t capacity = int64_t(a.width) * a.page;
    kv_lengths(a.start, a.new_lens, b, a.T, capacity, w.before, w.fresh);
    const int64_t len = int64_t(w.before) + w.fresh;
    w.len = int(len < capacity ? len : capacity);
    w.tiles = w.len > 0 ? (w.len + kNT - 1) / kNT : 1;
    w.live = int((int64_t(w.fresh) * a.G + R - 1) / R);
    w.units = int64_t(a.H) * (int64_t(w.live) * w.tiles + (a.row_tiles - w.live));
    return w;
}

// A position in the list of units.
struct Cursor {
    SeqWork w;
    int64_t base;  // first unit of sequence b
    int b, h, rt, tile;
    bool live;
    __device__ __forceinline__ void place(const AttArgs &a, int64_t u) {  // base <= u < base + w.units
        int64_t i = u - base;
        const int64_t lives = int64_t(a.H) * w.live * w.tiles;
        live = i < lives;
        if (live) {
            tile = int(i % w.tiles);
            i /= w.tiles;
            rt = int(i % w.live), h = int(i / w.live);
        } else {
            i -= lives;
            const int dead = a.row_tiles - w.live;
            tile = 0, rt = w.live + int(i % dead), h = int(i / dead);
        }
    }
    __device__ __forceinline__ int tiles() const { return live ? w.tiles : 1; }
    __device__ __forceinline__ void next(const AttArgs &a, int R) {
        if (++tile < tiles()) return;
        const int64_t u = base + (live ? (int64_t(h) * w.live + rt + 1) * w.tiles
                                       : int64_t(a.H) * w.live * w.tiles + int64_t(h) * (a.row_tiles - w.live) +
                                             (rt - w.live) + 1);
        if (u == base + w.units) {
            base += w.units;
            if (++b >= a.B) return;
            w = seq_work(a, b, R);
        }
        place(a, u);
    }
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for a phase; false after kCopyLimitNs.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0;; ++i) {
        if (mbar_try(bar, parity)) return true;
        if ((i & 63) == 63 && global_ns() - t0 > kCopyLimitNs) return false;
    }
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The codes in half-bytes 0 and 4 of w as fp16 (1024 + code has its code in the low bits), and 16
// times those in half-bytes 1 and 5: both exact.  (The factor is in the queries, or taken out of the
// output.)
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
    uint32_t r = (w & 0x000F000Fu) | 0x64006400u;
    asm("sub.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x64006400u));
    return r;
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
    uint32_t r = (w & 0x00F000F0u) | 0x64006400u;
    asm("sub.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x64006400u));
    return r;
}

template <int D, int MT>
struct AttShared {
    static constexpr int R = 16 * MT, NW = D / 32;
    static constexpr int kStageBytes = kNT * (D + 8);
    static constexpr int kQStride = D + 8, kPStride = kNT + 8;  // halves; 16 bytes past a multiple of 128: no bank conflicts
    alignas(128) uint8_t stage[kStages][kStageBytes];
    alignas(16) __half q[R * kQStride];
    alignas(16) __half p[2][R * kPStride];
    float row_c[R], row_qs[R];  // log2 scale of a row's scores; the sum of its queries
    float red[2][NW][R];
    int row_node[R];  // the row's new token, -1: no live row
    alignas(8) uint64_t full[kStages];
    uint32_t granules[kStages];  // bit 4 g: granule g of the unit was loaded
    int64_t find[2];
    int64_t scan[NW];
};

template <int D, int MT>
__global__ void __launch_bounds__(D, att_occupancy(D, MT)) kv_attention_kernel(const AttArgs a) {
    using Sh = AttShared<D, MT>;
    constexpr int R = Sh::R, NW = Sh::NW, TW = kNT / NW, NJ = TW / 8, KS = D / 16, E = D / 32;
    constexpr int kThreads = D;
    constexpr bool kQRegs = MT == 1 && D <= 128;
    extern __shared__ __align__(128) unsigned char raw[];
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    int *parent_s = reinterpret_cast<int *>(raw + sizeof(Sh));
    const int anc_words = (a.T + 31) / 32;
    uint32_t *anc_s = reinterpret_cast<uint32_t *>(parent_s + (a.parent ? a.T : 0));  // [R][anc_words]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int64_t ncta = gridDim.x, cta = blockIdx.x;

    griddep_launch_next();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&sh.full[i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    griddep_wait();
    if (cta == 0 && tid == 0) *a.status = SV_OK;
    if (a.parent)
        for (int i = tid; i < a.T; i += kThreads) parent_s[i] = a.parent[i];

    // all units, then the sequence where this CTA's share begins
    int64_t mine = 0;
    for (int b = tid; b < a.B; b += kThreads) mine += seq_work(a, b, R).units;
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    if (lane == 0) sh.scan[warp] = mine;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < NW; ++w) total += sh.scan[w];
    const int64_t ubegin = share_begin(total, cta, ncta), uend = share_begin(total, cta + 1, ncta);
    if (ubegin >= uend) return;
    {
        int64_t run = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            const int b = b0 + tid;
            const int64_t u = b < a.B ? seq_work(a, b, R).units : 0;
            int64_t inc = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += v;
            }
            __syncthreads();
            if (lane == 31) sh.scan[warp] = inc;
            __syncthreads();
            int64_t off = run;
            for (int w = 0; w < warp; ++w) off += sh.scan[w];
            const int64_t lo = off + inc - u;
            if (ubegin >= lo && ubegin < lo + u) sh.find[0] = b, sh.find[1] = lo;
            for (int w = 0; w < NW; ++w) run += sh.scan[w];
            if (run > ubegin) break;  // uniform
        }
        __syncthreads();
    }
    Cursor cur;
    cur.b = int(sh.find[0]), cur.base = sh.find[1];
    cur.w = seq_work(a, cur.b, R);
    cur.place(a, ubegin);
    Cursor ahead = cur;  // of the copies (warp 0)
    int64_t uahead = ubegin;

    const int64_t page_bytes = kv_page_bytes(a.page, D);
    auto issue = [&](int stage) {  // warp 0: the copies of unit uahead
        if (uahead >= uend) return;
        const int gi = lane >> 2, piece = lane & 3;
        const int64_t tok = int64_t(ahead.tile) * kNT + gi * a.granule;
        const uint8_t *src = nullptr;
        const int slot = int(tok % a.page);
        if (gi * a.granule < kNT && ahead.live && tok < ahead.w.len) {
            const int pg = __ldg(a.table + int64_t(ahead.b) * a.width + tok / a.page);
            if (pg >= 0 && pg < a.num_pages && SV_IN(slot + a.granule - 1, a.page))
                src = a.cache + (int64_t(pg) * a.H + ahead.h) * page_bytes;
        }
        const uint32_t bytes = src == nullptr ? 0 : piece < 2 ? a.granule * (D / 2) : a.granule * 4;
        const uint32_t sum = __reduce_add_sync(0xFFFFFFFFu, bytes);
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, src != nullptr && piece == 0);
        const uint32_t bar = smem_u32(&sh.full[stage]);
        if (lane == 0) {
            sh.granules[stage] = have;
            mbar_expect(bar, sum);
        }
        __syncwarp();
        if (src) {
            const uint32_t dst = smem_u32(sh.stage[stage]);
            if (piece < 2)
                bulk_load(dst + (piece * kNT + gi * a.granule) * (D / 2), src + (piece * a.page + slot) * (D / 2), bytes, bar);
            else
                bulk_load(dst + kNT * D + ((piece - 2) * kNT + gi * a.granule) * 4,
                          src + a.page * D + ((piece - 2) * a.page + slot) * 4, bytes, bar);
        }
        ++uahead;
        if (uahead < uend) ahead.next(a, R);
    };
    if (warp == 0)
        for (int i = 0; i < kStages - 1; ++i) issue(i);

    uint32_t qf[kQRegs ? KS : 1][4];
    float acc[MT][4][4];
    float m[MT][2], thr[MT][2], l[MT][2], z[MT][2], ym[MT][2];
    int kexp = 1;  // values' scales are divided by 2^(kexp - 14): all are below 1 then
    bool fresh_segment = true, waits = true;
    int64_t seg_lo = ubegin - cur.tile;
    const uint32_t all_granules = 0x11111111u & (kNT / a.granule == 8 ? 0xFFFFFFFFu : (1u << (4 * (kNT / a.granule))) - 1);

    for (int64_t u = ubegin; u < uend; ++u) {
        const int it = int(u - ubegin), stage = it % kStages, buf = it & 1;
        const uint32_t parity = uint32_t(it / kStages) & 1;
        if (fresh_segment) {
            // the rows' queries: rotated, scaled by a power of two into fp16's range (exact for 16-bit
            // inputs but for values 2^-25 of the row's largest; a rotated value is rounded to 11 bits),
            // columns in the order in which the codes unpack
            __syncthreads();
            for (int r = warp; r < R; r += NW) {
                const int64_t row = int64_t(cur.rt) * R + r;
                const int node = int(row / a.G), head = cur.h * a.G + int(row % a.G);
                const bool on = cur.live && node < cur.w.fresh;
                const int d0 = lane * E;
                float x[E];
#pragma unroll
                for (int i = 0; i < E; ++i) x[i] = 0.f;
                if (on) {
                    const uint16_t *qp = a.q + cur.b * a.q_bs + node * a.q_ts + head * a.q_hs;
                    const int64_t arow = a.rot.cos ? kv_rotation_row(a.rot, int64_t(cur.b) * a.T + node, cur.w.before + node) : 0;
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        x[i] = kv_to_float(__ldg(qp + d0 + i), a.bf16);
                        int partner, angle;
                        float sign;
                        if (a.rot.cos && kv_partner(a.rot, d0 + i, partner, angle, sign)) {
                            const float y = kv_to_float(__ldg(qp + partner), a.bf16);
                            x[i] = fmaf(x[i], __ldg(a.rot.cos + arow + angle), sign * y * __ldg(a.rot.sin + arow + angle));
                        }
                    }
                }
                float big = 0.f;
#pragma unroll
                for (int i = 0; i < E; ++i) big = fmaxf(big, fabsf(x[i]));
                const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(big));
                const int e2 = top == 0 ? 0 : int(top >> 23) - 127 - 10;  // the largest becomes 2^10 .. 2^11
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int d = d0 + i, quad = d / (D / 4), dd = d % (D / 4), n = dd % 8, ii = n & 3;
                    const float v = __half2float(__float2half_rn(ldexpf(a.scale < 0.f ? -x[i] : (a.scale == 0.f ? 0.f : x[i]), -e2)));
                    sum += v;
                    const int col = (2 * (dd / 8) + (ii >> 1)) * 16 + (ii & 1) * 8 + 2 * quad + (n >> 2);
                    sh.q[r * Sh::kQStride + col] = __float2half_rn(ii & 1 ? v * 0.0625f : v);
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                if (lane == 0) {
                    sh.row_c[r] = a.scale == 0.f ? 1.f : ldexpf(fabsf(a.scale) * 1.4426950408889634f, e2);
                    sh.row_qs[r] = sum;
                    sh.row_node[r] = on ? node : -1;
                }
                if (a.parent && lane == 0) {
                    uint32_t *anc = anc_s + r * anc_words;
                    for (int i = 0; i < anc_words; ++i) anc[i] = 0;
                    for (int v = on ? node : -1; v >= 0;) {
                        anc[v >> 5] |= 1u << (v & 31);
                        const int up = parent_s[v];
                        v = up < v ? up : -1;
                    }
                }
            }
            __syncthreads();
            if constexpr (kQRegs) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    ldmatrix4(qf[s], smem_u32(&sh.q[(lane & 15) * Sh::kQStride + s * 16 + (lane >> 4) * 8]));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[i][j][k] = 0.f;
#pragma unroll
                for (int k = 0; k < 2; ++k) m[i][k] = thr[i][k] = -INFINITY, l[i][k] = z[i][k] = 0.f;
            }
            kexp = 1;
            seg_lo = u - cur.tile;
            fresh_segment = false;
        }

        if (waits && !mbar_wait(smem_u32(&sh.full[stage]), parity)) {
            waits = false;  // reported; no further waits
            atomicExch(a.status, int(SV_ERR_TIMEOUT));
        }
        const uint8_t *kc = sh.stage[stage], *vc = kc + kNT * (D / 2);
        const uint32_t *km = reinterpret_cast<const uint32_t *>(kc + kNT * D), *vm = km + kNT;
        const uint32_t have = sh.granules[stage];
        const int tok0 = cur.tile * kNT;  // (fits: a table spans less than 2^31 tokens)
        const bool masked = tok0 + kNT > cur.w.before || have != all_granules;
        auto loaded = [&](int col) { return tok0 + col < cur.w.len && (have >> (4 * (col / a.granule)) & 1u); };

        // scores of this warp's tokens
        float s[MT][NJ][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[i][j][k] = 0.f;
        uint32_t kw[NJ][E];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint8_t *p = kc + (warp * TW + j * 8 + g) * (D / 2) + t4 * (D / 8);
            if constexpr (E == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                kw[j][0] = v.x, kw[j][1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
                    kw[j][4 * i] = v.x, kw[j][4 * i + 1] = v.y, kw[j][4 * i + 2] = v.z, kw[j][4 * i + 3] = v.w;
                }
            }
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t b0[NJ], b1[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint32_t w = ks & 1 ? kw[j][ks / 2] >> 8 : kw[j][ks / 2];
                b0[j] = codes_even(w), b1[j] = codes_odd(w);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t af[4];
                if constexpr (kQRegs) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) af[k] = qf[ks][k];
                } else {
                    ldmatrix4(af, smem_u32(&sh.q[(i * 16 + (lane & 15)) * Sh::kQStride + ks * 16 + (lane >> 4) * 8]));
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j) mma16816(s[i][j], af, b0[j], b1[j]);
            }
        }

        // y = s_j (q . code_j) + z_j sum(q); masked scores are -inf
        float vs[NJ][2], vz[NJ][2];
        uint32_t see[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) see[i] = 0xFFFFFFFFu, ym[i][0] = ym[i][1] = -INFINITY;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int col = warp * TW + j * 8 + 2 * t4;
            const uint2 kk = *reinterpret_cast<const uint2 *>(km + col), vv = *reinterpret_cast<const uint2 *>(vm + col);
            const float ks0 = __half2float(__ushort_as_half(uint16_t(kk.x))), kz0 = __half2float(__ushort_as_half(uint16_t(kk.x >> 16)));
            const float ks1 = __half2float(__ushort_as_half(uint16_t(kk.y))), kz1 = __half2float(__ushort_as_half(uint16_t(kk.y >> 16)));
            vs[j][0] = __half2float(__ushort_as_half(uint16_t(vv.x))), vz[j][0] = __half2float(__ushort_as_half(uint16_t(vv.x >> 16)));
            vs[j][1] = __half2float(__ushort_as_half(uint16_t(vv.y))), vz[j][1] = __half2float(__ushort_as_half(uint16_t(vv.y >> 16)));
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float q0 = sh.row_qs[i * 16 + g], q1 = sh.row_qs[i * 16 + g + 8];
                s[i][j][0] = fmaf(s[i][j][0], ks0, q0 * kz0);
                s[i][j][1] = fmaf(s[i][j][1], ks1, q0 * kz1);
                s[i][j][2] = fmaf(s[i][j][2], ks0, q1 * kz0);
                s[i][j][3] = fmaf(s[i][j][3], ks1, q1 * kz1);
            }
        }
        // the largest scale of the unit's values (a NaN one spoils only the rows that see it)
        auto scale_bits = [&](int col) { return (vm[col] & 0xFFFFu) < 0x7C00u ? vm[col] & 0xFFFFu : 0u; };
        uint32_t top;
        if (!masked) {
            top = max(scale_bits(lane), scale_bits(lane + 32));
        } else {
            top = max(loaded(lane) ? scale_bits(lane) : 0u, loaded(lane + 32) ? scale_bits(lane + 32) : 0u);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                see[i] = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = i * 16 + g + (k >> 1) * 8, node = sh.row_node[r];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int col = warp * TW + j * 8 + 2 * t4 + (k & 1);
                        const int idx = tok0 + col - cur.w.before;  // below 0: before the new tokens
                        bool v = node >= 0 && loaded(col);
                        if (v && idx >= 0 && SV_IN(idx, a.T)) v = a.parent ? anc_s[r * anc_words + (idx >> 5)] >> (idx & 31) & 1u : idx <= node;
                        if (v) see[i] |= 1u << (j * 4 + k);
                        else s[i][j][k] = -INFINITY;
                    }
                }
            }
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        const int knew = max(kexp, int(top >> 10));
        bool need = knew != kexp;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                ym[i][0] = fmaxf(ym[i][0], fmaxf(s[i][j][0], s[i][j][1]));
                ym[i][1] = fmaxf(ym[i][1], fmaxf(s[i][j][2], s[i][j][3]));
            }
            need |= ym[i][0] > thr[i][0] || ym[i][1] > thr[i][1];
        }
        // weights: p for the sums (this warp's tokens), p s' for the product
        auto weigh = [&](float (&dl)[MT][2], float (&dz)[MT][2]) {
            const float down = ldexpf(1.f, 14 - kexp);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float c0 = sh.row_c[i * 16 + g], c1 = sh.row_c[i * 16 + g + 8];
                const float m0 = m[i][0] == -INFINITY ? 0.f : m[i][0], m1 = m[i][1] == -INFINITY ? 0.f : m[i][1];
                dl[i][0] = dl[i][1] = dz[i][0] = dz[i][1] = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    float p[4], w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        p[k] = ex2(fmaf(s[i][j][k], k < 2 ? c0 : c1, k < 2 ? -m0 : -m1));
                        const float sc = vs[j][k & 1] * down, ze = vz[j][k & 1];
                        dl[i][k >> 1] += p[k];
                        if (masked) {  // a masked token's own scale and zero (NaN, or not loaded) must not matter
                            const bool v = see[i] >> (j * 4 + k) & 1u;
                            dz[i][k >> 1] += v ? p[k] * ze : 0.f;
                            w[k] = v ? p[k] * sc : 0.f;
                        } else {
                            dz[i][k >> 1] = fmaf(p[k], ze, dz[i][k >> 1]);
                            w[k] = p[k] * sc;
                        }
                    }
                    __half *dst = &sh.p[buf][(i * 16 + g) * Sh::kPStride + warp * TW + j * 8 + 2 * t4];
                    *reinterpret_cast<__half2 *>(dst) = __floats2half2_rn(w[0], w[1]);
                    *reinterpret_cast<__half2 *>(dst + 8 * Sh::kPStride) = __floats2half2_rn(w[2], w[3]);
                }
            }
        };
        float dl[MT][2], dz[MT][2];
        weigh(dl, dz);
        if (__syncthreads_or(need)) {  // some row's maximum moves (the first unit's always does), or the values' exponent
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y = ym[i][k];
                    y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 1));
                    y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 2));
                    if (t4 == 0) sh.red[0][warp][i * 16 + g + 8 * k] = y;
                }
            __syncthreads();
            const float kfac = ldexpf(1.f, kexp - knew);
            kexp = knew;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = i * 16 + g + 8 * k;
                    float y = sh.red[0][0][r];
#pragma unroll
                    for (int w = 1; w < NW; ++w) y = fmaxf(y, sh.red[0][w][r]);
                    const float c = sh.row_c[r], mn = fmaxf(m[i][k], y * c);
                    const float al = mn == -INFINITY ? 1.f : ex2(m[i][k] - mn);
                    m[i][k] = mn;
                    thr[i][k] = (mn + kLazy) / c;
                    l[i][k] *= al, z[i][k] *= al;
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j][2 * k] *= al * kfac, acc[i][j][2 * k + 1] *= al * kfac;
                }
            weigh(dl, dz);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) l[i][k] += dl[i][k], z[i][k] += dz[i][k];

        // every warp is past the last unit's values: their stage takes the copies of the unit after the next ones
        if (warp == 0) issue((it + kStages - 1) % kStages);

        // this warp's 32 dimensions
#pragma unroll
        for (int kk = 0; kk < kNT / 16; ++kk) {
            const uint2 w = *reinterpret_cast<const uint2 *>(vc + kk * 8 * D + warp * 256 + lane * 8);
            uint32_t b0[4], b1[4];
            b0[0] = codes_even(w.x), b0[1] = codes_odd(w.x), b0[2] = codes_even(w.x >> 8), b0[3] = codes_odd(w.x >> 8);
            b1[0] = codes_even(w.y), b1[1] = codes_odd(w.y), b1[2] = codes_even(w.y >> 8), b1[3] = codes_odd(w.y >> 8);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t af[4];
                ldmatrix4(af, smem_u32(&sh.p[buf][(i * 16 + (lane & 15)) * Sh::kPStride + kk * 16 + (lane >> 4) * 8]));
#pragma unroll
                for (int j = 0; j < 4; ++j) mma16816(acc[i][j], af, b0[j], b1[j]);
            }
        }

        const bool seg_end = cur.tile + 1 == cur.tiles();
        if (seg_end || u + 1 == uend) {
            // the rows' sums over lanes and warps
            __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x = l[i][k], y = z[i][k];
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 1), y += __shfl_xor_sync(0xFFFFFFFFu, y, 1);
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 2), y += __shfl_xor_sync(0xFFFFFFFFu, y, 2);
                    if (t4 == 0) sh.red[0][warp][i * 16 + g + 8 * k] = x, sh.red[1][warp][i * 16 + g + 8 * k] = y;
                }
            __syncthreads();
            const bool whole = seg_end && seg_lo >= ubegin;
            const int64_t slot = 2 * cta + (seg_lo >= ubegin && u - cur.tile != ubegin ? 1 : 0);
            const float up = ldexpf(1.f, kexp - 14);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = i * 16 + g + 8 * k;
                    float sl = 0.f, sz = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) sl += sh.red[0][w][r], sz += sh.red[1][w][r];
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float f = j & 1 ? up * 0.0625f : up;
                        o[j] = fmaf(acc[i][j][2 * k], f, sz), o[4 + j] = fmaf(acc[i][j][2 * k + 1], f, sz);
                    }
                    const int d0 = warp * 32 + 8 * t4;
                    if (whole) {
                        const int64_t row = int64_t(cur.rt) * R + r, node = row / a.G;
                        if (node < a.T) {
                            const bool zero = sh.row_node[r] < 0 || sl == 0.f;
                            const float inv = 1.f / sl;
                            uint32_t w4[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                w4[j] = uint32_t(kv_from_float(zero ? 0.f : o[2 * j] * inv, a.bf16)) |
                                        uint32_t(kv_from_float(zero ? 0.f : o[2 * j + 1] * inv, a.bf16)) << 16;
                            const int64_t head = int64_t(cur.h) * a.G + row % a.G;
                            *reinterpret_cast<uint4 *>(a.out + ((cur.b * int64_t(a.T) + node) * a.H * a.G + head) * D + d0) =
                                make_uint4(w4[0], w4[1], w4[2], w4[3]);
                        }
                    } else if (SV_IN(slot, 2 * ncta)) {
                        float4 *dst = reinterpret_cast<float4 *>(a.acc + (slot * R + r) * D + d0);
                        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                        if (warp == 0 && t4 == 0) a.ml[slot * R + r] = make_float2(m[i][k], sl);
                    }
                }
            if (tid == 0 && u - cur.tile <= ubegin)  // the share's first segment
                a.desc[cta] = AttDesc{u - cur.tile, u - cur.tile + cur.tiles(), total, cur.b, cur.h, cur.rt, cur.live ? cur.w.fresh : 0};
            fresh_segment = true;
        }
        if (u + 1 < uend) cur.next(a, R);
    }
}

// Joins a segment that several CTAs share: out = sum_c 2^(m_c - M) acc_c / sum_c 2^(m_c - M) l_c.
// Block (c, y) acts if CTA c's share begins inside a segment whose previous owner held its start;
// y takes four of the segment's rows.
constexpr int kJoinThreads = 128, kJoinRows = 4;

template <int D, int MT>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join_kernel(const AttArgs a, int ncta) {
    constexpr int R = 16 * MT;
    __shared__ float weight[kJoinRows][kAttSMs * 8 + 8];
    __shared__ float inv_s[kJoinRows];
    griddep_launch_next();
    griddep_wait();
    const int64_t c = int64_t(blockIdx.x) / (R / kJoinRows) + 1;
    const int r0 = int(blockIdx.x % (R / kJoinRows)) * kJoinRows;
    if (c >= ncta) return;
    // (CTA 0's share is empty only if all are; a CTA with an empty share wrote no descriptor)
    const int64_t total = a.desc[ncta - 1].total;  // the last share is never empty
    const int64_t begin = share_begin(total, c, ncta);
    if (begin >= share_begin(total, c + 1, ncta)) return;
    const AttDesc d = a.desc[c];
    if (begin <= d.lo) return;
    const int64_t c0 = share_owner(total, d.lo, ncta), c1 = share_owner(total, d.hi - 1, ncta);
    // the first non-empty share after the start's owner joins the segment
    if (share_owner(total, begin - 1, ncta) != c0) return;
    if (d.fresh <= 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // c0's part lies in its second slot unless its share begins with the segment
    auto slot_of = [&](int64_t k) { return 2 * k + (k == c0 && share_begin(total, c0, ncta) != d.lo ? 1 : 0); };
    for (int q = warp; q < kJoinRows; q += kJoinThreads / 32) {
        const int r = r0 + q;
        float big = -INFINITY;
        for (int64_t k = c0 + lane; k <= c1; k += 32)
            if (share_begin(total, k, ncta) < share_begin(total, k + 1, ncta)) big = fmaxf(big, a.ml[slot_of(k) * R + r].x);
        for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
        float sum = 0.f;
        for (int64_t k = c0 + lane; k <= c1; k += 32) {
            float w = 0.f;
            if (share_begin(total, k, ncta) < share_begin(total, k + 1, ncta)) {
                const float2 ml = a.ml[slot_of(k) * R + r];
                w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - big);
                sum += w * ml.y;
            }
            if (SV_IN(k - c0, kAttSMs * 8 + 8)) weight[q][k - c0] = w;
        }
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) inv_s[q] = sum == 0.f ? 0.f : 1.f / sum;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kJoinRows * D / 4; i += kJoinThreads) {
        const int q = i / (D / 4), d4 = i % (D / 4) * 4, r = r0 + q;
        const int64_t row = int64_t(d.rt) * R + r, node = row / a.G;
        if (node >= a.T) continue;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (node < d.fresh) {
#pragma unroll 4
            for (int64_t k = c0; k <= c1; ++k) {
                const float w = weight[q][k - c0];
                if (w == 0.f) continue;  // also: parts of empty shares, never written
                const float4 v = *reinterpret_cast<const float4 *>(a.acc + (slot_of(k) * R + r) * D + d4);
                o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
            }
            const float inv = inv_s[q];
            o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
        }
        const int64_t head = int64_t(d.h) * a.G + row % a.G;
        uint2 w;
        w.x = uint32_t(kv_from_float(o.x, a.bf16)) | uint32_t(kv_from_float(o.y, a.bf16)) << 16;
        w.y = uint32_t(kv_from_float(o.z, a.bf16)) | uint32_t(kv_from_float(o.w, a.bf16)) << 16;
        *reinterpret_cast<uint2 *>(a.out + ((d.b * int64_t(a.T) + node) * a.H * a.G + head) * D + d4) = w;
    }
}

struct AttLayout {
    size_t desc, ml, acc, total;
    int grid;
};
AttLayout att_layout(int64_t rows, int D) {
    const int mt = att_mt(rows), R = 16 * mt;
    AttLayout L;
    L.grid = kAttSMs * att_occupancy(D, mt);
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    L.desc = 256;
    L.ml = up(L.desc + size_t(L.grid) * sizeof(AttDesc));
    L.acc = up(L.ml + size_t(2) * L.grid * R * 8);
    L.total = up(L.acc + size_t(2) * L.grid * R * D * 4);
    return L;
}

template <int D, int MT>
cudaError_t launch_attention(const AttArgs &a, int grid, cudaStream_t s) {
    const size_t smem = sizeof(AttShared<D, MT>) + (a.parent ? size_t(a.T) * 4 + size_t(16 * MT) * ((a.T + 31) / 32) * 4 : 0);
    cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    e = launch_after(kv_attention_kernel<D, MT>, unsigned(grid), unsigned(D), smem, s, a);
    if (e != cudaSuccess) return e;
    return launch_after(kv_attention_join_kernel<D, MT>, unsigned((grid - 1) * (16 * MT / kJoinRows)), unsigned(kJoinThreads), 0, s, a, grid);
}

template <int D>
cudaError_t launch_attention_rows(const AttArgs &a, int mt, int grid, cudaStream_t s) {
    return mt == 1 ? launch_attention<D, 1>(a, grid, s) : mt == 2 ? launch_attention<D, 2>(a, grid, s) : launch_attention<D, 4>(a, grid, s);
}

}  // namespace
}  // namespace sv

extern "C" {

size_t spec_kv_attention_workspace_size(int B, int T, int heads, int kv_heads, int head_dim) {
    if (B <= 0 || T <= 0 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || !sv::kv_head_dim_ok(head_dim)) return 0;
    return sv::att_layout(int64_t(T) * (heads / kv_heads), head_dim).total;
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
    if (int64_t(table_width) * page_size > 0x7FFFFFC0) return SV_ERR_INVALID_ARG;
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
    const sv::AttLayout L = sv::att_layout(rows, head_dim);
    if (!workspace || workspace_bytes < L.total || reinterpret_cast<uintptr_t>(workspace) % 16) return SV_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    const int mt = sv::att_mt(rows);
    sv::AttArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.q_bs = q_batch_stride, a.q_ts = q_token_stride, a.q_hs = q_head_stride;
    a.bf16 = dtype == SV_KV_BF16;
    a.B = B, a.T = T, a.H = kv_heads, a.G = G;
    a.cache = static_cast<const uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.granule = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
    a.table = page_table, a.start = start, a.new_lens = new_lens, a.parent = parent;
    a.scale = scale;
    a.rot = sv::Rotation{cos, sin, table_len, cos ? pairs : 0, interleaved != 0, positions};
    a.out = static_cast<uint16_t *>(out);
    a.row_tiles = int((rows + 16 * mt - 1) / (16 * mt));
    a.status = reinterpret_cast<int *>(ws);
    a.desc = reinterpret_cast<sv::AttDesc *>(ws + L.desc);
    a.ml = reinterpret_cast<float2 *>(ws + L.ml);
    a.acc = reinterpret_cast<float *>(ws + L.acc);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = head_dim == 64    ? sv::launch_attention_rows<64>(a, mt, L.grid, s)
                          : head_dim == 128 ? sv::launch_attention_rows<128>(a, mt, L.grid, s)
                                            : sv::launch_attention_rows<256>(a, mt, L.grid, s);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
