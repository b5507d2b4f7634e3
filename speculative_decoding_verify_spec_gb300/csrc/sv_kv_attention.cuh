// sv_kv_attention.cuh -- the new tokens' attention over the 4-bit paged cache: the kernels, instantiated
// per head dimension by the translation units sv_kv_attention*.cu.
//
// For a query row q (one of the T x G rows that share a kv head) and cached tokens j with key
// k_j = z_j + s_j code_j and value likewise,
//   x_j = scale (s_j (q . (code_j - 8)) + (z_j + 8 s_j) sum(q)),  p_j = exp(x_j - m),
//   out = [ sum_j (p_j s'_j) (code'_j - 8) + sum_j p_j (z'_j + 8 s'_j) ] / sum_j p_j,
// so the matrix products run on the bare codes (exact in fp16) and each token's scale and zero
// cost a multiply-add per score instead of one per dimension.
//
// The second product's weights w_j = p_j s'_j are fp16, so their own maximum is what counts: with
// X_j = x_j log2(e) + log2(s'_j) and m near the row's largest X_j of the tokens that it sees, w_j = 2^(X_j - m), p_j =
// w_j / s'_j, and m cancels in the quotient.  Neither a token that the row does not see nor one of little weight then takes
// bits from the others, however large its values are.  m lies so that the largest weight is 2^7 to 2^15: a weight keeps fp16's 11
// bits down to 2^-21 of the largest at least, and is off by 2^-32 of that below.
//
// Work: a unit is 32 to 128 tokens for one (sequence, kv head, tile of 8 NR rows).  All units of the
// batch form one list; each CTA takes an equal, contiguous share of it, so ragged lengths balance
// by themselves and a long context spreads over the card.  A segment (one sequence, head, row
// tile) that ends up whole in a CTA is written out there; the others leave partial results
// that the join kernel adds up.
//
// A CTA has a warp that copies units into a ring in shared memory, and consumer warps.  Each
// consumer scores its part of a unit's tokens for all rows, the weights go through shared
// memory, and each warp accumulates its own 16 or 32 dimensions over all the tokens: a key or value code
// is unpacked once (or twice) per row tile and the accumulators need no joining.  Both products have
// the cache as the 16-row operand (tokens x dimensions, dimensions x tokens) and the queries or
// weights as the 8-column one, so that a single token's few heads are padded to 8 rows, not 16.  A
// unit's scores are computed two units ahead of its product, which leaves one barrier per unit and
// straight-line code between two of them.  m moves only when a weight passes 2^15, to where it is 2^7 (the weights fit
// fp16 either way).
//
// What bounds it.  The cache is read once per row tile: for few rows a byte of it needs about one instruction
// slot a lane (unpacking, one HMMA per 16 tokens and 16 dimensions, the scores), and the warps that fit
// the registers issue 2.4 instructions a clock: 256 single tokens with 8 heads a kv head over 4600 cached ones
// on average take 0.31 ms, 4.2 TB/s of the cache.  For many rows the HMMA rate (one m16n8k16 in 2 clocks a
// SM) and the scores' exponentials join in: 64 x 9 drafts with 4 heads a kv head take 0.16 ms, 140 TFLOP/s.
#pragma once

#include <cstdint>

#include "sv_checks.cuh"
#include "sv_device.cuh"
#include "sv_grid.cuh"
#include "sv_kv.cuh"
#include "sv_launch.cuh"

namespace sv {

constexpr float kTop = 7.f, kMost = 15.f;  // log2 of the largest weight where m moves, and of the largest there may be
constexpr uint64_t kCopyLimitNs = 1000000000ull;
constexpr int kAttSMs = 152;

// 16-row tiles of dimensions per consumer warp: 64 dimensions are shared by four warps too.
__host__ __device__ constexpr int att_mh(int D, int NR) { return D == 64 ? 1 : 2; }
// Tokens per unit, 16 or 32 a warp: as many as the registers for their scores allow.
__host__ __device__ constexpr int att_tokens(int D, int NR) { return D == 256 || (D == 128 && NR == 1) ? 128 : 64; }
// Units in the ring: one whose product runs, one that has its weights, one whose scores run, one on its way.
__host__ __device__ constexpr int att_stages(int D, int NR) { return 4; }
// CTAs per SM, by registers and shared memory.
__host__ __device__ constexpr int att_occupancy(int D, int NR) { return D == 256 ? 1 : D == 128 ? (NR <= 5 ? 3 : 2) : (NR <= 2 ? 4 : 3); }
// Tiles of 8 NR rows: as few as there have to be and no larger than they need be.  At most 48 rows, for more spill
// (64 rows of 128 dimensions do, by 250 bytes a thread); 32 of 64 dimensions, where 64 x 64 tree nodes with 4 query heads a
// kv head took 253 us in tiles of 32 rows (255 now), 267 in tiles of 64 and 276 in tiles of 16; 40 of 256, by shared memory.
constexpr int att_cap(int D) { return D == 64 ? 32 : D == 128 ? 48 : 40; }
inline int att_nr(int64_t rows, int D) {
    const int64_t tiles = (rows + att_cap(D) - 1) / att_cap(D);
    return int(((rows + tiles - 1) / tiles + 7) / 8);
}

struct AttArgs {
    const uint16_t *q;
    int64_t q_bs, q_ts, q_hs;
    int bf16, vec, rot_vec;  // query rows, and the angles' rows, lie on the 16-byte grid
    int B, T, H, G;  // H kv heads, G query heads each
    const uint8_t *cache;
    int num_pages, page, width, granule;  // granule: tokens per copy, a power of two dividing page and a unit
    const int32_t *table, *start, *new_lens, *parent;
    float scale;
    Rotation rot;
    uint16_t *out;
    int row_tiles;
    int *status;
    struct AttDesc *desc;  // [grid]
    float2 *ml;            // [2 grid][R] m (-inf: no score was seen) and the sum of w / s'
    float *acc;            // [2 grid][R][D]
};

// What the joining kernel has to do for the segment inside which a CTA's share begins.
struct alignas(16) AttDesc {
    int join;           // 1: this share is the one after that of the segment's start; 0: nothing to do
    int first, last;    // the shares that hold parts of the segment, 2 first + 1: the first one's part lies in its second slot
    int total;          // all units: if they are fewer than the shares, some shares are empty
    int b, h, rt, fresh;
};

// Where a CTA's share begins.
__device__ __forceinline__ int share_begin(int total, int c, int n) { return int(int64_t(c) * total / n); }
__device__ __forceinline__ int share_owner(int total, int u, int n) { return int((int64_t(u + 1) * n - 1) / total); }

// Written once by every CTA: seg_lo and seg_hi bound the units of the share's first segment.
__device__ __forceinline__ AttDesc describe(int total, int cta, int ncta, int ubegin, int seg_lo, int seg_hi, int b, int h, int rt, int fresh) {
    if (seg_lo >= ubegin || fresh <= 0) return AttDesc{0, 0, 0, 0, 0, 0, 0, 0};
    const int first = share_owner(total, seg_lo, ncta);
    return AttDesc{share_owner(total, ubegin - 1, ncta) == first, 2 * first + (share_begin(total, first, ncta) != seg_lo),
                   share_owner(total, seg_hi - 1, ncta), total, b, h, rt, fresh};
}

struct SeqWork {
    int before, fresh, len;
    int tiles;       // units of a live segment
    int live;        // row tiles with a live row
    int units;       // of the whole sequence (the host has checked that all fit 31 bits)
};
template <int NT>
__device__ __forceinline__ SeqWork seq_work(const AttArgs &a, int64_t b, int R) {
    SeqWork w;
    const int64_t capacity = int64_t(a.width) * a.page;
    kv_lengths(a.start, a.new_lens, b, a.T, capacity, w.before, w.fresh);
    const int64_t len = int64_t(w.before) + w.fresh;
    w.len = int(len < capacity ? len : capacity);
    w.tiles = w.len > 0 ? (w.len + NT - 1) / NT : 1;
    w.live = int((int64_t(w.fresh) * a.G + R - 1) / R);
    w.units = a.H * (w.live * w.tiles + (a.row_tiles - w.live));
    return w;
}

// A position in the list of units.
template <int NT>
struct Cursor {
    SeqWork w;
    int base;  // first unit of sequence b
    int b, h, rt, tile;
    bool live;
    __device__ __forceinline__ void place(const AttArgs &a, int u) {  // base <= u < base + w.units
        int i = u - base;
        const int lives = a.H * w.live * w.tiles;
        live = i < lives;
        if (live) {
            tile = i % w.tiles;
            i /= w.tiles;
            rt = i % w.live, h = i / w.live;
        } else {
            i -= lives;
            const int dead = a.row_tiles - w.live;
            tile = 0, rt = w.live + i % dead, h = i / dead;
        }
    }
    __device__ __forceinline__ int tiles() const { return live ? w.tiles : 1; }
    // to unit u, the one after the current
    __device__ __forceinline__ void next(const AttArgs &a, int R, int u) {
        if (++tile < tiles()) return;
        if (u == base + w.units) {
            base += w.units;
            if (++b >= a.B) return;
            w = seq_work<NT>(a, b, R);
        }
        place(a, u);
    }
};

// What the consumers know of a unit; written by the copying warp.
struct alignas(16) Unit {
    int b, h, rt, tile, tiles;
    int before, len, fresh;   // tokens before the step; all; new ones (0: no live row)
    uint32_t have;            // bit 4 g: granule g was loaded
    int masked;               // not every token is seen by every row
    int unused[2];
};
static_assert(sizeof(Unit) == 48, "");

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
                 : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldmatrix2_trans(uint32_t &r0, uint32_t &r1, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with sums that start from nothing.
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// The codes in half-bytes 0 and 4 of w, less 8, as fp16 (1024 + code has its code in the low bits), and
// 16 times those in half-bytes 1 and 5: all exact.  (The factor is in the queries, or taken out of the
// output.)  Centred, so that sums over thousands of tokens do not cancel against the zeros' part.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
    uint32_t r;  // (w & 0x000F000F) | 0x64006400 in one instruction
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(0x000F000Fu), "r"(0x64006400u));
    asm("sub.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x64086408u));
    return r;
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(0x00F000F0u), "r"(0x64006400u));
    asm("sub.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x64806480u));
    return r;
}

__host__ __device__ constexpr int att_threads(int D, int NR) { return D * 2 / att_mh(D, NR) + 32; }

template <int D, int NR>
struct AttShared {
    static constexpr int R = 8 * NR, NW = D / 16 / att_mh(D, NR), kConsumers = 32 * NW;
    static constexpr int NT = att_tokens(D, NR), kStages = att_stages(D, NR);
    static constexpr int kStageBytes = NT * (D + 8);
    static constexpr int kQStride = D + 8;        // halves; 16 bytes past a multiple of 128: no bank conflicts
    static constexpr int kPStride = 8 * (NR | 1);  // an odd number of 16-byte columns: none here either
    alignas(128) uint8_t stage[kStages][kStageBytes];
    alignas(16) __half q[R * kQStride];
    alignas(16) __half p[2][NT * kPStride];       // [token][row]
    // per pair of rows: their queries' sums and the log2 scales of their scores; what moves m (-inf until a score was
    // seen), and -m (0 until then)
    alignas(16) float row_y[R / 2][4];
    alignas(16) float row_p[R / 2][4];
    alignas(16) float alpha[R];
    float red[2][NW][R];
    alignas(8) int row_node[R];  // the row's new token, -1: no live row
    alignas(8) uint64_t full[kStages], empty[kStages];
    Unit unit[kStages];
};

// All units, and this CTA's share of them: where it begins and ends, and the cursor at its beginning (every warp for
// itself).  False: the share is empty.
template <int NT>
__device__ __forceinline__ bool find_share(const AttArgs &a, int R, int lane, int cta, int ncta, Cursor<NT> &cur, int &total,
                                           int &ubegin, int &uend) {
    total = 0;
    SeqWork w0{};  // of sequence `lane`
    for (int b = lane; b < a.B; b += 32) {
        const SeqWork w = seq_work<NT>(a, b, R);
        if (b == lane) w0 = w;
        total += w.units;
    }
    total = __reduce_add_sync(0xFFFFFFFFu, total);
    ubegin = share_begin(total, cta, ncta), uend = share_begin(total, cta + 1, ncta);
    if (ubegin >= uend) return false;
    for (int b0 = 0, run = 0;; b0 += 32) {  // (ubegin < total: some sequence holds it)
        const int b = b0 + lane;
        if (b0 > 0) w0 = b < a.B ? seq_work<NT>(a, b, R) : SeqWork{};
        int inc = w0.units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        const int lo = run + inc - w0.units;
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, ubegin >= lo && ubegin < run + inc);
        if (hit) {
            const int l = __ffs(hit) - 1;
            cur.b = b0 + l;
            cur.base = __shfl_sync(0xFFFFFFFFu, lo, l);
            int *to = reinterpret_cast<int *>(&cur.w);
            const int *from = reinterpret_cast<const int *>(&w0);
#pragma unroll
            for (int i = 0; i < int(sizeof(SeqWork) / 4); ++i) to[i] = __shfl_sync(0xFFFFFFFFu, from[i], l);
            break;
        }
        run += __shfl_sync(0xFFFFFFFFu, inc, 31);
        if (b0 + 32 >= a.B) return false;  // never
    }
    cur.place(a, ubegin);
    return true;
}

#ifdef SV_CHECKS
extern __device__ int g_kv_lose;  // see spec_kv_lose_unit
#endif

// The copying warp: the units of the share into the ring, up to kStages ahead of the consumers.  Returns when all copies
// that it has begun are there (waiting as long as it may): a block must not end with copies under way into its shared memory.
template <int D, int NT, int kStages, typename Shared>
__device__ __forceinline__ void copy_units(const AttArgs &a, Shared &sh, Cursor<NT> &cur, int ubegin, int uend, int R, int lane) {
    // Lanes take (granule, piece) pairs: keys,
    // values and their scales; a page that is a unit is one piece.
    const bool whole = a.page == NT;
    const int gi = lane >> 2, piece = lane & 3, granules = NT / a.granule;
    const bool busy = whole ? lane == 0 : gi < granules;
    const uint32_t bytes = !busy ? 0 : whole ? NT * (D + 8) : piece < 2 ? a.granule * (D / 2) : a.granule * 4;
    const int to = piece < 2 ? (piece * NT + gi * a.granule) * (D / 2) : NT * D + ((piece - 2) * NT + gi * a.granule) * 4;
    const int from = piece < 2 ? piece * a.page * (D / 2) : a.page * D + (piece - 2) * a.page * 4, each = piece < 2 ? D / 2 : 4;
    const uint32_t all_granules = granules == 8 ? 0x11111111u : 0x11111111u & ((1u << (4 * granules)) - 1);
    const uint32_t all_bytes = __reduce_add_sync(0xFFFFFFFFu, bytes);
    const int64_t page_bytes = kv_page_bytes(a.page, D), head_step = int64_t(a.H) * page_bytes;
    int pi = 0, slot = 0, stage = 0, wrap = 0;  // this lane's granule: page of the sequence, slot in it
    uint32_t phase = 1;
    int begun = 0;
    bool placed = false;
    for (int u = ubegin; u < uend; ++u) {
        if (!placed) {
            const int tok = cur.tile * NT + gi * a.granule;
            pi = tok / a.page, slot = tok - pi * a.page;
            placed = true;
        }
        const bool inside = busy && cur.live && cur.tile * NT + gi * a.granule < cur.w.len;
        const int pg = inside ? __ldg(a.table + int64_t(cur.b) * a.width + pi) : -1;
        const bool here = pg >= 0 && pg < a.num_pages && SV_IN(slot + a.granule - 1, a.page);
        const uint32_t got = __ballot_sync(0xFFFFFFFFu, here), have = got & 0x11111111u;
        const uint32_t sum = have == all_granules ? all_bytes : __reduce_add_sync(0xFFFFFFFFu, here ? bytes : 0u);
        if (wrap > 0 && !mbar_wait(smem_u32(&sh.empty[stage]), phase)) {
            atomicExch(a.status, int(SV_ERR_TIMEOUT));
            break;  // (the consumers' waits give up too)
        }
#ifdef SV_CHECKS
        if (u - ubegin == g_kv_lose) break;
#endif
        const uint32_t bar = smem_u32(&sh.full[stage]);
        if (lane == 0) {
            int4 *un = reinterpret_cast<int4 *>(&sh.unit[stage]);
            un[0] = make_int4(cur.b, cur.h, cur.rt, cur.tile);
            un[1] = make_int4(cur.tiles(), cur.w.before, cur.w.len, cur.live ? cur.w.fresh : 0);
            un[2] = make_int4(int(have), int((cur.tile + 1) * NT > cur.w.before || have != all_granules), 0, 0);
            mbar_expect(bar, sum);
        }
        __syncwarp();
        if (here)
            bulk_load(smem_u32(sh.stage[stage]) + to, a.cache + pg * head_step + cur.h * page_bytes + from + slot * each, bytes, bar);
        ++begun;
        if (++stage == kStages) stage = 0, phase ^= 1, wrap = 1;
        if (cur.tile + 1 < cur.tiles()) {
            ++cur.tile;
            slot += NT;
            while (slot >= a.page) slot -= a.page, ++pi;
        } else if (u + 1 < uend) {
            cur.next(a, R, u + 1);
            placed = false;
        }
    }
    for (int i = max(0, begun - kStages); i < begun; ++i)
        if (!mbar_wait(smem_u32(&sh.full[i % kStages]), uint32_t(i / kStages) & 1u)) atomicExch(a.status, int(SV_ERR_TIMEOUT));
}

// Two fp32 numbers in a register pair, worked on by one instruction.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float x, float y) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 split(Two a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float power2(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127
// Barriers of the N consumer threads, whole warps: each warp is together afterwards, as the matrix instructions need it.
template <int N>
__device__ __forceinline__ void consumers_sync() {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory");
    __syncwarp();
}
template <int N>
__device__ __forceinline__ bool consumers_or(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(x)), "n"(N)
        : "memory");
    __syncwarp();
    return r != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Eight 16-bit numbers from p (vec: 16-byte aligned) as floats.
__device__ __forceinline__ void load8(const uint16_t *p, bool vec, bool bf16, float (&x)[8]) {
    if (vec) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = kv_to_float(uint16_t(u[i / 2] >> (16 * (i & 1))), bf16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = kv_to_float(__ldg(p + i), bf16);
    }
}

// A value's scale s' and zero z', from their fp16 words, as the weights need them.
struct ValueScale {
    float log2, inverse, shift;  // log2(s'), 1 / s', (z' + 8 s') / s'
    bool finite;
};
__device__ __forceinline__ ValueScale value_scale(uint32_t word) {
    // at least 2^-24, as all are that were appended (so that slots of zeros have a logarithm too); NaN stays
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(word) : "r"(0xFC000001u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&word));
    ValueScale v;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(v.log2) : "f"(f.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v.inverse) : "f"(f.x));
    v.shift = fmaf(f.y, v.inverse, 8.f);
    v.finite = fabsf(f.x) < INFINITY && fabsf(f.y) < INFINITY;
    return v;
}

// The power of two that is taken out of a row whose largest number has the bits `top`: that number becomes 2^10 .. 2^11
// (less for rows below 2^-100).
__device__ __forceinline__ int query_exponent(uint32_t top) { return top == 0 ? 0 : max(int(top >> 23) - 127 - 10, -110); }

// Eight dimensions from d0 on of a query row, rotated.
__device__ __forceinline__ void query_chunk(const AttArgs &a, const Unit &un, int node, int head, int d0, float (&x)[8]) {
    const uint16_t *qp = a.q + un.b * a.q_bs + node * a.q_ts + head * a.q_hs;
    load8(qp + d0, a.vec, a.bf16, x);
    if (a.rot.cos && d0 < 2 * a.rot.pairs) {
        const int64_t arow = kv_rotation_row(a.rot, int64_t(un.b) * a.T + node, un.before, node);
        const float *cp = a.rot.cos + arow, *sp = a.rot.sin + arow;
        float y[8], cs[8], sn[8];
        if (!a.rot.interleaved && a.rot.pairs % 8 == 0) {  // the chunk lies within one half
            const int e0 = d0 < a.rot.pairs ? d0 : d0 - a.rot.pairs;
            load8(qp + (d0 < a.rot.pairs ? d0 + a.rot.pairs : e0), a.vec, a.bf16, y);
            if (a.rot_vec) {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 u = __ldg(reinterpret_cast<const float4 *>(cp + e0 + i)), v = __ldg(reinterpret_cast<const float4 *>(sp + e0 + i));
                    cs[i] = u.x, cs[i + 1] = u.y, cs[i + 2] = u.z, cs[i + 3] = u.w;
                    sn[i] = v.x, sn[i + 1] = v.y, sn[i + 2] = v.z, sn[i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) cs[i] = __ldg(cp + e0 + i), sn[i] = __ldg(sp + e0 + i);
            }
            const float sign = d0 < a.rot.pairs ? -1.f : 1.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sn[i] *= sign;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                int partner, angle;
                float sign;
                if (kv_partner(a.rot, d0 + i, partner, angle, sign)) {
                    y[i] = kv_to_float(__ldg(qp + partner), a.bf16);
                    cs[i] = __ldg(cp + angle), sn[i] = sign * __ldg(sp + angle);
                } else {
                    y[i] = 0.f, cs[i] = 1.f, sn[i] = 0.f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], cs[i], y[i] * sn[i]);
    }
}

// The queries of a segment's rows into shared memory: rotated, scaled by a power of two into fp16's
// range (exact for 16-bit inputs but for values 2^-25 of the row's largest), columns in the order in which the
// codes unpack.  A rotated value is rounded to 11 bits: for bf16 outputs that is a tenth of their own
// rounding; for fp16 ones it would be as large, so that what the rounding took (rest) is multiplied too, in a second
// product.  Eight dimensions a thread.
template <int D, int NR, bool kExact>
__device__ __forceinline__ void load_queries(const AttArgs &a, AttShared<D, NR> &sh, const Unit &un, int tid, bool rest, __half *out) {
    using Sh = AttShared<D, NR>;
    constexpr int R = Sh::R, L = D / 8, P = Sh::kConsumers / L;  // lanes of a row, rows at a time
    const int c = tid % L, d0 = c * 8;
#pragma unroll 2
    for (int r0 = 0; r0 < R; r0 += P) {
        const int r = r0 + tid / L;
        const int row = un.rt * R + r;
        const int node = row / a.G, head = un.h * a.G + row - node * a.G;
        const bool on = r < R && node < un.fresh;
        float x[8];
        query_chunk(a, un, on ? node : 0, on ? head : 0, d0, x);  // (no branch: the rows' loads go out together)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = on ? x[i] : 0.f;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(fabsf(x[i])));
#pragma unroll
        for (int o = L / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const int e2 = query_exponent(top);
        const float shrink = power2(-e2);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = a.scale < 0.f ? -x[i] : (a.scale == 0.f ? 0.f : x[i]);
            const float y = v * shrink, r = __half2float(__float2half_rn(y));
            x[i] = rest ? y - r : r;
            sum += kExact ? y : r;
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (R % P != 0 && r >= R) continue;
        // dimension 8 w + n of quad's quarter: k-step 2 w + (n % 4) / 2, the odd n scaled by 1 / 16
        __half *dst = &out[r * Sh::kQStride + 2 * (d0 / (D / 4)) + 2 * (d0 % (D / 4) / 8) * 16];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float f = n & 1 ? 0.0625f : 1.f;
            *reinterpret_cast<__half2 *>(dst + (n >> 1) * 16 + (n & 1) * 8) = __floats2half2_rn(x[n] * f, x[n + 4] * f);
        }
        if (c == 0 && !rest) {
            const float c2 = a.scale == 0.f ? 1.f : fmaxf(fabsf(a.scale) * 1.4426950408889634f * power2(e2), 1.2e-38f);
            sh.row_y[r / 2][r & 1] = sum, sh.row_y[r / 2][2 + (r & 1)] = c2;
            sh.row_p[r / 2][r & 1] = -INFINITY, sh.row_p[r / 2][2 + (r & 1)] = 0.f;
            sh.row_node[r] = on ? node : -1;
        }
    }
}

// kExact: queries have a second fp16 part (see load_queries).
template <int D, int NR, bool kExact>
__global__ void __launch_bounds__(att_threads(D, NR), att_occupancy(D, NR)) kv_attention_kernel(const AttArgs a) {
    using Sh = AttShared<D, NR>;
    constexpr int R = Sh::R, NW = Sh::NW, NT = Sh::NT, TW = NT / NW, NG = TW / 16, kStages = Sh::kStages, KS = D / 16, E = D / 32;
    constexpr int MH = att_mh(D, NR), kThreads = att_threads(D, NR), C = Sh::kConsumers;
    constexpr bool kQRegs = NR * KS <= 16;  // the queries' fragments stay in registers (as launch_attention knows)
    static_assert(NG >= 1 && TW % 16 == 0 && NT <= 128 && NT % 32 == 0 && NG * NR <= 8, "");
    extern __shared__ __align__(128) unsigned char raw[];
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    // the queries' second part takes the first one's place where that is in registers
    __half *q_rest = kQRegs ? sh.q : reinterpret_cast<__half *>(raw + sizeof(Sh));
    int *parent_s = reinterpret_cast<int *>(raw + sizeof(Sh) + (kQRegs || !kExact ? 0 : sizeof(sh.q)));
    const int anc_words = (a.T + 31) / 32;
    uint32_t *anc_s = reinterpret_cast<uint32_t *>(parent_s + (a.parent ? a.T : 0));  // [R][anc_words]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int ncta = int(gridDim.x), cta = int(blockIdx.x);

    griddep_launch_next();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&sh.full[i]), 1), mbar_init(smem_u32(&sh.empty[i]), NW);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    griddep_wait();
    if (cta == 0 && tid == 0) *a.status = SV_OK;
    if (a.parent)
        for (int i = tid; i < a.T; i += kThreads) parent_s[i] = a.parent[i];

    Cursor<NT> cur;
    int total, ubegin, uend;
    if (!find_share<NT>(a, R, lane, cta, ncta, cur, total, ubegin, uend)) {
        if (tid == 0) a.desc[cta] = AttDesc{0, 0, 0, 0, 0, 0, 0, 0};
        return;
    }
    __syncthreads();

    if (warp == NW) {
        copy_units<D, NT, kStages>(a, sh, cur, ubegin, uend, R, lane);
        return;
    }

    // MH 16-row tiles of dimensions x R rows: dimension 4 g + 2 h (+ 1, times 16) of the slice, rows 2 t4, 2 t4 + 1
    float acc[MH][NR][4];
    Two l[NR], z[NR];     // of rows 2 t4, 2 t4 + 1
    float s[NG][NR][4];   // X of tokens g, g + 8 of each group, rows 2 t4, 2 t4 + 1
    float vi[NG][2], vz[NG][2];  // of those tokens' values: 1 / s', (z' + 8 s') / s'
    uint32_t qf[kQRegs ? KS : 2][kQRegs ? NR : 1][2];
    bool waits = true;
    int stage = 0;
    uint32_t phase = 0;
    const int units = uend - ubegin;
    const int slice = warp % (D / 32), part = warp / (D / 32);  // this warp's dimensions

    auto wait_unit = [&](int st, uint32_t ph) {
        if (waits && !mbar_wait(smem_u32(&sh.full[st]), ph)) {
            waits = false;  // reported; no further waits
            atomicExch(a.status, int(SV_ERR_TIMEOUT));
        }
        __syncwarp();  // (lanes may leave the wait at different times, and matrix instructions follow)
    };
    // X of this warp's tokens of a unit; whether they move some row's m.
    auto score = [&](int st) -> bool {
        const Unit &un = sh.unit[st];
        const uint8_t *kc = sh.stage[st];
        const uint32_t *km = reinterpret_cast<const uint32_t *>(kc + NT * D) + warp * TW + g, *vm = km + NT;
        uint32_t kw[NG][2][E];
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *p = kc + (warp * TW + i * 16 + h * 8 + g) * (D / 2) + t4 * (D / 8);
                if constexpr (E == 2) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(p);
                    kw[i][h][0] = v.x, kw[i][h][1] = v.y;
                } else {
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) {
                        const uint4 v = reinterpret_cast<const uint4 *>(p)[e];
                        kw[i][h][4 * e] = v.x, kw[i][h][4 * e + 1] = v.y, kw[i][h][4 * e + 2] = v.z, kw[i][h][4 * e + 3] = v.w;
                    }
                }
            }
        // few independent sums: the odd k-steps have their own, so that products do not wait for one another
        constexpr bool kTwo = NG * NR <= 2;
        float s2[kTwo ? NG : 1][kTwo ? NR : 1][4];
#pragma unroll
        for (int w = 0; w < E; ++w) {  // a word of codes: two k-steps
            uint32_t af[2][NG][4];
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = kw[i][h][w], y = x >> 8;
                    af[0][i][h] = codes_even(x), af[0][i][2 + h] = codes_odd(x);
                    af[1][i][h] = codes_even(y), af[1][i][2 + h] = codes_odd(y);
                }
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                uint32_t b[4];
                if constexpr (kQRegs) {
                    b[0] = qf[2 * w][n][0], b[1] = qf[2 * w][n][1], b[2] = qf[2 * w + 1][n][0], b[3] = qf[2 * w + 1][n][1];
                } else {
                    ldmatrix4(b, smem_u32(&sh.q[(n * 8 + (lane & 7)) * Sh::kQStride + w * 32 + (lane >> 3) * 8]));
                }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if (w == 0) mma16816_first(s[i][n], af[0][i], b[0], b[1]);
                    else mma16816(s[i][n], af[0][i], b[0], b[1]);
                    if constexpr (!kTwo) mma16816(s[i][n], af[1][i], b[2], b[3]);
                    else if (w == 0) mma16816_first(s2[i][n], af[1][i], b[2], b[3]);
                    else mma16816(s2[i][n], af[1][i], b[2], b[3]);
                }
            }
        }
        if constexpr (kTwo) {
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[i][n][k] += s2[i][n][k];
        }
        if constexpr (kExact) {
#pragma unroll
            for (int w = 0; w < E; ++w)
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    uint32_t b[4];
                    ldmatrix4(b, smem_u32(&q_rest[(n * 8 + (lane & 7)) * Sh::kQStride + w * 32 + (lane >> 3) * 8]));
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        const uint32_t x = kw[i][0][w], y = kw[i][1][w];
                        const uint32_t even[4] = {codes_even(x), codes_even(y), codes_odd(x), codes_odd(y)};
                        const uint32_t odd[4] = {codes_even(x >> 8), codes_even(y >> 8), codes_odd(x >> 8), codes_odd(y >> 8)};
                        mma16816(s[i][n], even, b[0], b[1]);
                        mma16816(s[i][n], odd, b[2], b[3]);
                    }
                }
        }
        // y = s_j (q . (code_j - 8)) + (z_j + 8 s_j) sum(q)
        float ks[NG][2], kz[NG][2], vl[NG][2];
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t kk = km[i * 16 + h * 8], vv = vm[i * 16 + h * 8];
                const float2 kf = __half22float2(*reinterpret_cast<const __half2 *>(&kk));
                ks[i][h] = kf.x, kz[i][h] = fmaf(8.f, kf.x, kf.y);
                const ValueScale v = value_scale(vv);
                vl[i][h] = v.log2, vi[i][h] = v.inverse, vz[i][h] = v.shift;
            }
        uint32_t see = 0xFFFFFFFFu;
        if (un.masked) {
            const int tok0 = un.tile * NT;  // (fits: a table spans less than 2^31 tokens)
            auto loaded = [&](int col) { return tok0 + col < un.len && (un.have >> (4 * (col / a.granule)) & 1u); };
            // bit (i NR + n) 4 + k: that score's token is seen by its row
            see = 0;
            int idx[NG][2];  // of the tokens among the new ones; -1: before them, T: not there
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = warp * TW + i * 16 + h * 8 + g;
                    idx[i][h] = loaded(col) ? max(-1, tok0 + col - un.before) : a.T;
                }
#pragma unroll 1
            for (int n = 0; n < NR; ++n) {
                const int2 node = *reinterpret_cast<const int2 *>(&sh.row_node[n * 8 + 2 * t4]);
                const uint32_t *anc = anc_s + (n * 8 + 2 * t4) * anc_words;
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int x = idx[i][k >> 1], own = k & 1 ? node.y : node.x;
                        bool v = own >= 0 && x <= own;  // a row's ancestors come before it
                        if (a.parent && v && x >= 0 && SV_IN(x, a.T)) v = anc[(k & 1) * anc_words + (x >> 5)] >> (x & 31) & 1u;
                        see |= uint32_t(v) << ((i * NR + n) * 4 + k);
                    }
            }
            // A masked token's weight is 0, and its scale and zero must not matter, whatever they are.  A
            // NaN value reaches the rows that see it by their score instead.
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool here = loaded(warp * TW + i * 16 + h * 8 + g);
                    if (!here || !value_scale(vm[i * 16 + h * 8]).finite) {
                        vl[i][h] = vi[i][h] = vz[i][h] = 0.f;
                        ks[i][h] = NAN;
                    }
                }
        }
        bool need = false;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float4 ry = *reinterpret_cast<const float4 *>(sh.row_y[n * 4 + t4]);
            const Two qs = two(ry.x, ry.y), c = two(ry.z, ry.w);
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float *y = s[i][n] + 2 * h;
                    const Two x = fma2(two(y[0], y[1]), two(ks[i][h], ks[i][h]), mul2(qs, two(kz[i][h], kz[i][h])));
                    const float2 r = split(fma2(x, c, two(vl[i][h], vl[i][h])));
                    y[0] = r.x, y[1] = r.y;
                }
        }
        if (un.masked) {
            __syncwarp();  // (a branch, not a select on every unit's scores)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (!(see >> ((i * NR + n) * 4 + k) & 1u)) s[i][n][k] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float2 most = *reinterpret_cast<const float2 *>(sh.row_p[n * 4 + t4]);
            float y0 = -INFINITY, y1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < NG; ++i) y0 = fmaxf(y0, fmaxf(s[i][n][0], s[i][n][2])), y1 = fmaxf(y1, fmaxf(s[i][n][1], s[i][n][3]));
            need |= y0 > most.x || y1 > most.y;
        }
        return need;
    };
    // Some row's m moves (the first unit's always does).  The weights of the unit before, in buffer buf (-1: none), move
    // along.
    auto update = [&](int buf) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float y = -INFINITY;
#pragma unroll
                for (int i = 0; i < NG; ++i) y = fmaxf(y, fmaxf(s[i][n][k], s[i][n][2 + k]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, o));
                if (g == 0) sh.red[0][warp][n * 8 + 2 * t4 + k] = y;
            }
        consumers_sync<C>();
        for (int r = tid; r < R; r += C) {
            float y = sh.red[0][0][r];
#pragma unroll
            for (int w = 1; w < NW; ++w) y = fmaxf(y, sh.red[0][w][r]);
            const float seen = sh.row_p[r / 2][r & 1] == -INFINITY ? -INFINITY : -sh.row_p[r / 2][2 + (r & 1)], mn = fmaxf(seen, y - kTop);
            sh.alpha[r] = seen == -INFINITY ? 0.f : ex2(seen - mn);
            if (mn != -INFINITY) sh.row_p[r / 2][r & 1] = mn + kMost, sh.row_p[r / 2][2 + (r & 1)] = -mn;
        }
        consumers_sync<C>();
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float2 al = *reinterpret_cast<const float2 *>(&sh.alpha[n * 8 + 2 * t4]);
            l[n] = mul2(l[n], two(al.x, al.y)), z[n] = mul2(z[n], two(al.x, al.y));
#pragma unroll
            for (int h = 0; h < MH; ++h) {
                acc[h][n][0] *= al.x, acc[h][n][1] *= al.y;
                acc[h][n][2] *= al.x, acc[h][n][3] *= al.y;
            }
        }
        if (buf >= 0) {
            for (int i = tid; i < NT * NR * 4; i += C) {
                const int tok = i / (NR * 4), r = i % (NR * 4) * 2;
                __half2 *w = reinterpret_cast<__half2 *>(&sh.p[buf][tok * Sh::kPStride + r]);
                const float2 v = __half22float2(*w);
                *w = __floats2half2_rn(v.x * sh.alpha[r], v.y * sh.alpha[r + 1]);
            }
            consumers_sync<C>();
        }
    };
    // Weights: w / s' and w (z' + 8 s') / s' for the sums (this warp's tokens), w for the product, rounded to fp16.
    auto weigh = [&](int buf) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float2 rp = *reinterpret_cast<const float2 *>(&sh.row_p[n * 4 + t4][2]);
            const Two minus = two(rp.x, rp.y);
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 x = split(add2(two(s[i][n][2 * h], s[i][n][2 * h + 1]), minus));
                    const float w0 = ex2(x.x), w1 = ex2(x.y);
                    const Two w = two(w0, w1);
                    l[n] = fma2(w, two(vi[i][h], vi[i][h]), l[n]);
                    z[n] = fma2(w, two(vz[i][h], vz[i][h]), z[n]);
                    *reinterpret_cast<__half2 *>(&sh.p[buf][(warp * TW + i * 16 + h * 8 + g) * Sh::kPStride + n * 8 + 2 * t4]) =
                        __floats2half2_rn(w0, w1);
                }
        }
    };
    // This warp's dimensions of a unit's product.
    auto product = [&](int st, int buf) {
        const uint8_t *vc = sh.stage[st] + NT * (D / 2) + slice * 256 + lane * 8;
#pragma unroll
        for (int kk = 0; kk < NT / 16; ++kk) {
            const uint2 w = *reinterpret_cast<const uint2 *>(vc + kk * 8 * D);
            uint32_t af[MH][4];
#pragma unroll
            for (int h = 0; h < MH; ++h) {
                const int shift = MH == 2 ? 8 * h : 8 * part;
                const uint32_t x = w.x >> shift, y = w.y >> shift;
                af[h][0] = codes_even(x), af[h][1] = codes_odd(x), af[h][2] = codes_even(y), af[h][3] = codes_odd(y);
            }
            const uint32_t row = smem_u32(&sh.p[buf][(kk * 16 + (lane & 15)) * Sh::kPStride]);
#pragma unroll
            for (int n = 0; n < NR; n += 2) {
                if (n + 1 < NR) {
                    uint32_t b[4];
                    ldmatrix4_trans(b, row + (n * 8 + (lane >> 4) * 8) * 2);
#pragma unroll
                    for (int h = 0; h < MH; ++h) mma16816(acc[h][n], af[h], b[0], b[1]), mma16816(acc[h][n + 1], af[h], b[2], b[3]);
                } else {
                    uint32_t b0, b1;
                    ldmatrix2_trans(b0, b1, row + n * 16);
#pragma unroll
                    for (int h = 0; h < MH; ++h) mma16816(acc[h][n], af[h], b0, b1);
                }
            }
        }
    };

    // the first segment is known already, and its queries load while its first unit is on its way
    Unit seg{cur.b, cur.h, cur.rt, cur.tile, cur.tiles(), cur.w.before, cur.w.len, cur.live ? cur.w.fresh : 0, 0, 0, {0, 0}};
    for (int it = 0;;) {  // segments
        const int last = min(units, it + seg.tiles - seg.tile);  // past the segment's last unit here
        if (consumers_or<C>(!waits)) break;  // a wait gave up, some thread's at least: `seg` may not be there
        load_queries<D, NR, kExact>(a, sh, seg, tid, false, sh.q);
        if (a.parent)
            for (int r = tid; r < R; r += C) {
                uint32_t *anc = anc_s + r * anc_words;
                for (int i = 0; i < anc_words; ++i) anc[i] = 0;
                const int node = (seg.rt * R + r) / a.G;
                for (int v = node < seg.fresh ? node : -1; v >= 0;) {
                    anc[v >> 5] |= 1u << (v & 31);
                    const int up = parent_s[v];
                    v = up < v ? up : -1;
                }
            }
        consumers_sync<C>();
        if constexpr (kQRegs) {
#pragma unroll
            for (int w = 0; w < E; ++w)
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    uint32_t b[4];
                    ldmatrix4(b, smem_u32(&sh.q[(n * 8 + (lane & 7)) * Sh::kQStride + w * 32 + (lane >> 3) * 8]));
                    qf[2 * w][n][0] = b[0], qf[2 * w][n][1] = b[1], qf[2 * w + 1][n][0] = b[2], qf[2 * w + 1][n][1] = b[3];
                }
        }
        if constexpr (kExact) {
            consumers_sync<C>();
            load_queries<D, NR, kExact>(a, sh, seg, tid, true, q_rest);
            consumers_sync<C>();
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            l[n] = z[n] = 0;  // (two zeros)
#pragma unroll
            for (int h = 0; h < MH; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[h][n][k] = 0.f;
        }
        const int seg_lo = ubegin + it - seg.tile;
        const bool whole = it >= seg.tile && it + seg.tiles - seg.tile <= units;

        // Three units are under way: one's product, the next one's weights, and the scores of the one after.  One
        // barrier per unit, and between two of them straight-line code without a dependence from part to part.
        auto advance = [&]() {
            if (++stage == kStages) stage = 0, phase ^= 1;
        };
        auto nothing = [&]() {  // scores of no token
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                vi[i][0] = vi[i][1] = vz[i][0] = vz[i][1] = 0.f;
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[i][n][k] = -INFINITY;
            }
        };
        int here = stage;  // of the unit whose product is next; `stage` runs ahead
        if (it == 0) wait_unit(stage, phase);
        bool need = score(stage);
        advance();
        if (consumers_or<C>(need)) update(-1);
        weigh(0);
        need = false;
        if (it + 1 < last) {
            wait_unit(stage, phase);
            need = score(stage);
            advance();
        } else {
            nothing();
        }
        for (int buf = 0; it < last; ++it, buf ^= 1) {
            if (consumers_or<C>(need)) update(buf);  // and this unit's weights are in place
            const bool more = it + 2 < last;
            if (more) wait_unit(stage, phase);
            product(here, buf);
            weigh(buf ^ 1);
            need = false;
            if (more) {
                need = score(stage);
                advance();
            } else {
                nothing();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.empty[here]));
            if (++here == kStages) here = 0;
        }

        // the rows' sums over lanes and warps
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x = k ? split(l[n]).y : split(l[n]).x, y = k ? split(z[n]).y : split(z[n]).x;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o), y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
                if (g == 0) sh.red[0][warp][n * 8 + 2 * t4 + k] = x, sh.red[1][warp][n * 8 + 2 * t4 + k] = y;
            }
        consumers_sync<C>();
        const int64_t slot = 2 * cta + (seg_lo > ubegin ? 1 : 0);
        const int d0 = slice * 32 + 4 * g + 2 * part;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = n * 8 + 2 * t4 + k;
                float sl = 0.f, sz = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) sl += sh.red[0][w][r], sz += sh.red[1][w][r];
                float o[2 * MH];
#pragma unroll
                for (int h = 0; h < MH; ++h) o[2 * h] = acc[h][n][k] + sz, o[2 * h + 1] = fmaf(acc[h][n][2 + k], 0.0625f, sz);
                if (whole) {
                    const int row = seg.rt * R + r, node = row / a.G;
                    if (node < a.T) {
                        const float inv = sh.row_node[r] < 0 || sl == 0.f ? 0.f : 1.f / sl;
                        const int64_t head = seg.h * a.G + row % a.G;
                        uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + ((seg.b * int64_t(a.T) + node) * a.H * a.G + head) * D + d0);
#pragma unroll
                        for (int h = 0; h < MH; ++h) {
                            const float x = inv == 0.f ? 0.f : o[2 * h] * inv, y = inv == 0.f ? 0.f : o[2 * h + 1] * inv;
                            dst[h] = uint32_t(kv_from_float(x, a.bf16)) | uint32_t(kv_from_float(y, a.bf16)) << 16;
                        }
                    }
                } else if (SV_IN(slot, 2 * ncta)) {
                    float2 *dst = reinterpret_cast<float2 *>(a.acc + (slot * R + r) * D + d0);
#pragma unroll
                    for (int h = 0; h < MH; ++h) dst[h] = make_float2(o[2 * h], o[2 * h + 1]);
                    if (warp == 0 && g == 0)
                        a.ml[slot * R + r] = make_float2(sh.row_p[r / 2][k] == -INFINITY ? -INFINITY : -sh.row_p[r / 2][2 + k], sl);
                }
            }
        if (tid == 0 && seg_lo <= ubegin)  // the share's first segment
            a.desc[cta] = describe(total, cta, ncta, ubegin, seg_lo, seg_lo + seg.tiles, seg.b, seg.h, seg.rt, seg.fresh);
        if (it == units) break;
        wait_unit(stage, phase);
        seg = sh.unit[stage];
    }
}

// Joins a segment that several CTAs share: out = sum_c 2^(m_c - M) acc_c / sum_c 2^(m_c - M) l_c, in one pass with a
// running M.  Block (c, y) acts if CTA c's share is the second one with a part of a segment; y takes the rows that 256
// threads hold at four dimensions a thread.  What bounds it is the latency of three dependent reads.
constexpr int kJoinThreads = 256;
__host__ __device__ constexpr int join_rows(int D) { return kJoinThreads * 4 / D; }

template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join_kernel(const AttArgs a, int ncta, int R, int groups) {
    // (no griddep_launch_next: the next call's kernel, resident early beside this one's waiting blocks, would not find
    // all its places; 256 single tokens took 389 us so, and 299 without)
    griddep_wait();
    const int c = int(blockIdx.x) / groups + 1, r = int(blockIdx.x) % groups * join_rows(D) + threadIdx.x / (D / 4);
    const AttDesc d = a.desc[c];
    if (!d.join || r >= R) return;
    const int d4 = threadIdx.x % (D / 4) * 4, row = d.rt * R + r, node = row / a.G;
    if (node >= a.T) return;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (node < d.fresh) {
        float m = -INFINITY, l = 0.f;
        constexpr int kAhead = 4;
        for (int k0 = d.first / 2; k0 <= d.last; k0 += kAhead) {
            float2 ml[kAhead];
            float4 v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = k0 + i;
                const int64_t slot = k == d.first / 2 ? d.first : int64_t(2) * k;
                ml[i] = make_float2(-INFINITY, 0.f), v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                const bool wrote = k <= d.last && (d.total >= ncta || share_begin(d.total, k, ncta) < share_begin(d.total, k + 1, ncta));
                if (wrote && SV_IN(slot, 2 * ncta)) {
                    ml[i] = a.ml[slot * R + r];
                    v[i] = *reinterpret_cast<const float4 *>(a.acc + (slot * R + r) * D + d4);
                }
            }
            float most = m;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) most = fmaxf(most, ml[i].x);
            const float keep = most == -INFINITY ? 1.f : ex2(m - most);
            l *= keep, o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                // a part that saw no score, or only NaN, has no maximum: its sums are 0, or NaN and to be kept
                const float w = ml[i].x == -INFINITY ? 1.f : ex2(ml[i].x - most);
                l = fmaf(w, ml[i].y, l);
                o.x = fmaf(w, v[i].x, o.x), o.y = fmaf(w, v[i].y, o.y), o.z = fmaf(w, v[i].z, o.z), o.w = fmaf(w, v[i].w, o.w);
            }
            m = most;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        o.x = l == 0.f ? 0.f : o.x * inv, o.y = l == 0.f ? 0.f : o.y * inv;
        o.z = l == 0.f ? 0.f : o.z * inv, o.w = l == 0.f ? 0.f : o.w * inv;
    }
    uint2 w;
    w.x = uint32_t(kv_from_float(o.x, a.bf16)) | uint32_t(kv_from_float(o.y, a.bf16)) << 16;
    w.y = uint32_t(kv_from_float(o.z, a.bf16)) | uint32_t(kv_from_float(o.w, a.bf16)) << 16;
    const int64_t head = d.h * a.G + row - node * a.G;
    *reinterpret_cast<uint2 *>(a.out + ((d.b * int64_t(a.T) + node) * a.H * a.G + head) * D + d4) = w;
}

template <int D>
cudaError_t launch_join(const AttArgs &a, int grid, int R, cudaStream_t s) {
    const int groups = (R + join_rows(D) - 1) / join_rows(D);
    if (grid < 2) return cudaSuccess;  // nothing is shared
    return launch_after(kv_attention_join_kernel<D>, unsigned((grid - 1) * groups), unsigned(kJoinThreads), 0, s, a, grid, R, groups);
}

template <int D, int NR, bool kExact>
cudaError_t launch_attention(const AttArgs &a, int grid, cudaStream_t s) {
    constexpr size_t fixed = sizeof(AttShared<D, NR>) + (kExact && NR * (D / 16) > 16 ? sizeof(AttShared<D, NR>::q) : 0);
    static_assert(fixed + (1 + NR / 4.0) * 4 * SV_MAX_TREE_NODES <= 227 * 1024, "");
    const size_t smem = fixed + (a.parent ? size_t(a.T) * 4 + size_t(8 * NR) * ((a.T + 31) / 32) * 4 : 0);
    static std::atomic<int> allowed[64];
    cudaError_t e = allow_shared(kv_attention_kernel<D, NR, kExact>, int(smem), allowed);
    if (e != cudaSuccess) return e;
    e = launch_after(kv_attention_kernel<D, NR, kExact>, unsigned(grid), unsigned(att_threads(D, NR)), smem, s, a);
    if (e != cudaSuccess) return e;
    return launch_join<D>(a, grid, 8 * NR, s);
}

// The attention kernels of a head dimension, each instantiated in its own translation unit.
template <int D, bool kExact>
cudaError_t launch_attention_rows(const AttArgs &a, int nr, int grid, cudaStream_t s);

template <int D, bool kExact>
cudaError_t launch_attention_of(const AttArgs &a, int nr, int grid, cudaStream_t s) {
    if constexpr (att_cap(D) >= 40) {
        if (nr == 5) return launch_attention<D, 5, kExact>(a, grid, s);
    }
    if constexpr (att_cap(D) >= 48) {
        if (nr == 6) return launch_attention<D, 6, kExact>(a, grid, s);
    }
    switch (nr) {
    case 1: return launch_attention<D, 1, kExact>(a, grid, s);
    case 2: return launch_attention<D, 2, kExact>(a, grid, s);
    case 3: return launch_attention<D, 3, kExact>(a, grid, s);
    default: return launch_attention<D, 4, kExact>(a, grid, s);
    }
}

#define SV_KV_ATTENTION_INSTANTIATE(D, EXACT)                                                          \
    template <>                                                                                       \
    cudaError_t launch_attention_rows<D, EXACT>(const AttArgs &a, int nr, int grid, cudaStream_t s) {   \
        return launch_attention_of<D, EXACT>(a, nr, grid, s);                                         \
    }

}  // namespace sv
