// sv_kv8_attention.cuh -- the new tokens' attention over the 8-bit paged cache: the kernel, instantiated per head
// dimension by the translation units sv_kv8_attention_*.cu.
//
// For a query row q (one of the T x G rows that share a kv head) and cached tokens j with keys s_j c_j and values s'_j c'_j,
//   t_j = log2(e) scale s_j (q . c_j) + log2(s'_j),  w_j = 2^(t_j - m) = p_j s'_j,  out = sum_j w_j c'_j / sum_j (w_j / s'_j).
// Both products run on the fifth-generation tensor cores with the cache's bytes as they lie in memory as the 128-row operand,
// so that no code is ever unpacked:
//   S [128 tokens x rows]     = K codes [128 x D]  times  q^T          D / 32 steps a part of q
//   O [D (128) x rows]        = V codes^T [D x 128]  times  w          4 steps a part of w
// The other operands are 8-bit floats too, so a query and a weight are held as sums of parts, each the rounding of what the parts
// before it left.  A query's have 4 bits each: two hold the 8 bits of a bfloat16, three 12.  A part's products are summed in fp32 with the others', which
// costs no more than one product in 16 bits would.
//
// Weights span far more than such floats do: next to a token with nearly all of the probability, or in a tile with a block whose scale is
// 2^30 above its neighbours', it is the small ones that may make the result, for nothing says that the large one's value is not 0.  So
// their parts have 5 bits of exponent and 3 bits each (three hold 11 bits, for bf16 outputs, four 15, for fp16 ones), and two ranges: weights from
// 2^-23 of the tile's largest on (2^-20 with four parts), and those below, times 2^23 (2^20), in columns of their own, whose sums come back times
// 2^-23.  A weight is off by 2^-11 of itself (2^-15), near a range's lower end by 2^-8.6 (2^-12), and below both by 2^-51.5 of the largest at most.
//
// Every tile of 128 tokens has its own m, a whole number (the rounded largest t of the row's tokens that it sees, less 15), and its own O, which is added
// to the row's sums in registers times 2^(m - M), with M the row's first m; M moves only when a later m is 60 above it.
//
// The queries' parts come from a kernel of their own.  A block of the attention has a warp that copies tiles and queries into rings in
// shared memory (keys and values apart: a key's place is free once its scores are there), a thread that issues the
// products as their operands come, and a group of four warps for the softmax for each 16 rows.  A thread of those has one
// token's scores for the group's rows, and one or two dimensions of their output: maxima are one reduction over the warp and one
// barrier, the weights' sums stay in the thread until the segment ends, and a token's weights are stored in 16 bytes a part and range
// (rows are the operand's contiguous axis).  Scores and outputs have two places each in tensor memory, so that the next tile's
// scores are computed during this one's softmax, and its output is taken up after the next one's weights.
//
// Work: all tiles of the batch form one list that is cut into equal shares, as in sv_kv_attention.cuh, whose list, descriptors
// and join of split segments these are.
//
// Measured, and what bounds it.  256 single tokens with 8 heads a kv head over 4600 cached ones on average: 392 us in a graph, 6.2 TB/s, 92 % of
// a plain copy's rate.  6 drafts over 200001 tokens, 256 dimensions: 99 us, 4.1 TB/s; there and with more rows the path of a
// tile through a block counts, which one block an SM does not cover: 64 x 9 drafts with 4 heads a kv head (36 rows) take 147 us, 2.4 us a
// tile, 54 instructions for each row and token, 2.1 a clock, the tensor pipe at 44 %.  (With two parts of 4 bits a weight and one range, which lost weights of 2^-18 of the largest, these took 372, 85 and 128 us.)  A product of 128 x N x 32
// takes 45 clocks up to N = 48, 48 for 64, 56 for 96 and 65 for 128 columns, measured, so that parts and ranges cost little there.
#pragma once

#include "sv_kv8.cuh"
#include "sv_kv_wide.cuh"

namespace sv {

constexpr int kTile8 = 128;
constexpr int kGroupRows8 = 16;  // query rows of a softmax group
__host__ __device__ constexpr int att8_groups(int NR) { return NR / kGroupRows8; }
__host__ __device__ constexpr int att8_threads(int NR) { return 64 + 128 * att8_groups(NR); }
// Tiles in the rings, places for queries, and blocks an SM: by shared memory and registers.
__host__ __device__ constexpr int att8_stages(int D, int NR) { return D == 64 ? (NR == 16 ? 5 : NR == 32 ? 4 : 6) : D == 128 ? (NR <= 32 ? 2 : 3) : (NR == 16 ? 3 : 2); }
__host__ __device__ constexpr int att8_value_stages(int D, int NR) {
    return D == 256 ? (NR == 48 ? 2 : 3) : D == 128 && NR == 16 ? 3 : D == 64 && NR == 32 ? 3 : att8_stages(D, NR);
}
__host__ __device__ constexpr int att8_q_places(int D, int NR) { return D == 256 || (D == 128 && NR == 32) ? 1 : 2; }
__host__ __device__ constexpr int att8_occupancy(int D, int NR) { return D == 256 || NR >= 48 ? 1 : 2; }
// Rows a tile, by the rows that share a kv head: as few tiles as there have to be, and no larger than they need be.  At most 64; 48 of 256
// dimensions, by tensor memory.
constexpr int att8_cap(int D) { return D == 256 ? 48 : 64; }
inline int att8_rows(int64_t rows, int D) {
    const int64_t tiles = (rows + att8_cap(D) - 1) / att8_cap(D);
    return int((rows + tiles * kGroupRows8 - 1) / (tiles * kGroupRows8)) * kGroupRows8;
}

constexpr float kTop8 = 15.f;  // log2 of the largest weight
enum : int { kMasked8 = 1, kRagged8 = 2, kFirst8 = 4, kLast8 = 8 };  // in Unit::masked: not every row sees every token; not every token is there; of a segment

// Bytes of a segment's queries: three parts, laid out as the keys, and the rows' factors.
__host__ __device__ constexpr int query_bytes8(int D, int NR) { return 3 * NR * D + 4 * NR; }

struct Att8Args : AttArgs {
    int nr, nq;            // rows a tile, parts of a query
    int wide;              // the kernel for many rows
    int see_words;         // a new token's words in `see`; of the kernel for many rows: a row's
    int64_t query_blocks;
    uint8_t *parts;        // [B][H][row_tiles][query_bytes8]
    uint32_t *see;         // [row_tiles][T][see_words]: the rows that see a new token of a tree; or [row_tiles][nr][see_words], the other way round
};

struct alignas(16) Info8 {
    Unit unit;
    uint32_t word[kTile8 / kKv8Block][4];
};

template <int D, int NR, int NP>
struct Att8Shared {
    static constexpr int kDims = D, kRows = NR, kTile = kTile8, W = att8_groups(NR), RW = kGroupRows8, SW = (NR + 31) / 32, kStages = att8_stages(D, NR), kValues = att8_value_stages(D, NR), kInfos = kStages + 2;
    static constexpr int kQ = att8_q_places(D, NR), MB = D == 256 ? 2 : 1;
    // Few rows: a product reads the cache's operand at its full width whatever the columns, so the parts are columns of
    // one product and are added up afterwards.
    static constexpr bool kStackQ = NR == 16 || (D == 256 && NR == 32);
    // A part of the weights has the rows' columns twice (one of a weight's two is 0).  16 rows: the first two parts side by side.
    static constexpr int kStackP = NR == 16 ? 2 : 1;
    static constexpr int kScoreCols = kStackQ ? (NR == 16 ? 64 : 96) : NR == 32 ? 32 : 64, kOutEach = 2 * kStackP * NR, kOutCols = MB * kOutEach;
    static constexpr int kUsed = 2 * (kScoreCols + kOutCols), kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    alignas(128) uint8_t k[kStages][kTile8 * D];
    uint8_t v[kValues][kTile8 * D];       // (64 dimensions: a product's upper 64 rows read past the end, into w)
    uint8_t w[NP][2][NR * kTile8];        // [part][of the upper range, of the lower one][16 rows][token][16 bytes]
    struct Queries {
        uint8_t part[3][NR * D];
        float factor[NR];                 // log2(e) scale times the power of two taken out of the row
    };
    Queries q[kQ];
    Info8 info[kInfos];
    alignas(16) float red[W][2][4][RW];        // maxima of a warp's 32 tokens
    alignas(16) float sums[W][4][RW];
    alignas(16) float4 move[W][4][2][RW / 2];  // of a row pair: -m, then 2^(m - M); every warp has its own
    // Each is waited for before what it tells of can come about once more, so that a phase's parity is enough: a unit's place in `info`
    // is taken again after the scores of two units later, which wait for the softmax to have read this one's.
    alignas(8) uint64_t full_k[kStages], full_v[kValues], empty_k[kStages], empty_v[kValues], full_i[kInfos];
    uint64_t full_s[2], free_s[2], full_o[2], free_o[2], full_w[2], full_q[kQ], free_q[kQ], done;
    uint32_t tmem;
};

// A shared-memory operand without a swizzle: blocks of 8 x 16 bytes, `along_k` and `across` bytes apart.  Its words: the address and the
// first distance, and the second.  Later steps are sums with the first word (computed anew, a descriptor cost the issuing thread 150 clocks a product).
__device__ __forceinline__ uint32_t operand8(uint32_t addr, uint32_t along_k) { return (addr & 0x3FFFF) >> 4 | along_k >> 4 << 16; }
__host__ __device__ constexpr uint32_t operand8_high(uint32_t across) { return across >> 4 | 1u << 14; }
// 8-bit floats (4 bits of exponent; `five`: 5 in the second operand) into fp32, 128 rows, N columns; `turned`: both operands have their rows contiguous.
__device__ __forceinline__ constexpr uint32_t kind8(int N, bool turned, bool five = false) { return 1u << 4 | (five ? 1u << 10 : 0u) | (turned ? 3u << 15 : 0u) | uint32_t(N / 8) << 17 | 8u << 24; }
__device__ __forceinline__ void mma8(uint32_t d, uint32_t a, uint32_t a_high, uint32_t b, uint32_t b_high, uint32_t kind, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(kind), "r"(uint32_t(add))
        : "memory");
}
// Eight columns of this warp's 32 rows, there after tmem_loaded().
__device__ __forceinline__ void tmem_get8(float (&x)[8], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// (what follows uses x after the wait)
__device__ __forceinline__ void tmem_here(float (&x)[8]) {
    asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]));
}
__device__ __forceinline__ float warp_largest(float x) {  // NaN left out
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
// mbar_wait by a whole warp: true for all its lanes or none.
static __device__ __noinline__ bool warp_wait_long(uint32_t bar, uint32_t parity) {
    const bool there = mbar_wait(bar, parity);
    return __all_sync(0xFFFFFFFFu, there);
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, mbar_try(smem_u32(bar), parity)) || warp_wait_long(smem_u32(bar), parity);
}
// Barrier kId of N threads; true if x is for any of them.
template <int kId, int N>
__device__ __forceinline__ bool group_or(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(x)), "n"(kId), "n"(N)
        : "memory");
    __syncwarp();
    return r != 0;
}

// The three parts of two pairs of numbers, four codes each (the first number's in the lowest byte).  A part is the number rounded to 4 bits, by
// the difference with a multiple of it (Dekker's splitting): the conversion to a code then rounds only what is below 2^-6, and a
// conversion back would cost four times a conversion there.
__device__ __forceinline__ void parts8(Two v, Two w, uint32_t (&c)[3]) {
    const Two minus = two(-1.f, -1.f), split4 = two(1048577.f, 1048577.f);  // 2^20 + 1
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const float2 f = split(v), g = split(w);
        c[i] = kv8_codes(f.x, f.y, g.x, g.y);
        if (i < 2) {
            const Two m = mul2(v, split4), o = mul2(w, split4);
            v = fma2(fma2(fma2(v, minus, m), minus, m), minus, v);  // v - (m - (m - v))
            w = fma2(fma2(fma2(w, minus, o), minus, o), minus, w);
        }
    }
}

// The parts of four weights, the first one's in the lowest byte, a word for a part in the upper range and one in the lower range.  Weights are at most 2^15.5; those of
// 2^-kLow on are taken as they are, those below times 2^kLift, into the parts of the lower range; a weight's parts in the other range are 0.  A part has
// 3 bits and 5 of exponent: the upper byte of a 16-bit float, so that a part is one addition (to the nearest) and the next ones' sum one
// exact subtraction there.  Three parts hold the 11 bits of such a float; the fourth is what the float left of the weight.
template <int NP>
struct Weights8 {
    static constexpr int kLow = NP == 3 ? 8 : 5, kLift = int(kTop8) + kLow;
};
__device__ __forceinline__ uint32_t half2_of(float2 x) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x.y), "f"(x.x));
    return h;
}
__device__ __forceinline__ uint32_t half2_minus(uint32_t x, uint32_t y) {
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
    return x;
}
template <int NP>
__device__ __forceinline__ void weight_parts8(const Two (&w)[2], uint32_t (&upper)[NP], uint32_t (&lower)[NP]) {
    constexpr float lift = float(1 << Weights8<NP>::kLift);
    constexpr uint32_t border = uint32_t(15 - Weights8<NP>::kLow) << 10 /* 2^-kLow */, nearest = 0x00800080u, high = 0xFF00FF00u;
    uint32_t h[2], mask[2], part[2];
    float2 rest[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Two lifted = mul2(w[i], two(lift, lift));
        const uint32_t up = half2_of(split(w[i])), low = half2_of(split(lifted));
        asm("set.ge.u32.f16x2 %0, %1, %2;" : "=r"(mask[i]) : "r"(up), "r"(border << 16 | border));
        h[i] = (up & mask[i]) | (low & ~mask[i]);
        if (NP > 3) {
            const __half2 h2 = *reinterpret_cast<const __half2 *>(&h[i]);
            const float2 a = split(w[i]), b = split(lifted), f = __half22float2(h2);
            rest[i] = make_float2((mask[i] & 1u ? a.x : b.x) - f.x, (mask[i] >> 16 ? a.y : b.y) - f.y);
        }
    }
    const uint32_t which = __byte_perm(mask[0], mask[1], 0x7531);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint32_t round[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            round[i] = h[i] + nearest;
            part[i] = round[i] & high;
            if (k < 2) h[i] = half2_minus(h[i], part[i]);
        }
        const uint32_t code = __byte_perm(round[0], round[1], 0x7531);
        upper[k] = code & which, lower[k] = code & ~which;
    }
    if (NP > 3) {
        uint32_t code;
        asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e5m2x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e5m2x2.f32 b, %4, %3;\n\tmov.b32 %0, {a, b};\n\t}"
            : "=r"(code)
            : "f"(rest[0].x), "f"(rest[0].y), "f"(rest[1].x), "f"(rest[1].y));
        upper[NP - 1] = code & which, lower[NP - 1] = code & ~which;
    }
}

// Whether a phase is over, without a wait.
__device__ __forceinline__ bool mbar_test(const uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Asleep until a phase is over, or some 200 ns.
__device__ __forceinline__ void mbar_doze(const uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(200)
        : "memory");
}
// Between two looks at several barriers: false when nothing has come for as long as a wait may take.
struct Patience {
    uint64_t since = 0;
    uint32_t looks = 0;
    __device__ __forceinline__ void reset() { looks = 0; }
    __device__ __forceinline__ bool go_on() {
        if (looks++ == 0) since = global_ns();
        return (looks & 63) != 0 || global_ns() - since <= kCopyLimitNs;
    }
};

// Where a unit's pieces lie for a lane of the copying warp: a granule's keys or values and words.
struct Source8 {
    const uint8_t *at;
    uint32_t bytes, sum, have;  // this lane's bytes, those of all granules (of codes), bit 4 g: granule g is there
};
// The units of the share in turn, each with a lane's piece (0: keys, 1: values, 2: words).
template <typename Sh>
struct Walk8 {
    Cursor<Sh::kTile> cur;
    int u, pi = 0, slot = 0;
    bool placed = false;
    __device__ __forceinline__ Source8 source(const Att8Args &a, int gi, int piece, bool busy) {
        constexpr int D = Sh::kDims;
        const int tok = cur.tile * Sh::kTile + gi * a.granule;
        if (!placed) pi = tok / a.page, slot = tok - pi * a.page, placed = true;
        const bool inside = busy && cur.live && tok < cur.w.len;
        const int pg = inside ? __ldg(a.table + int64_t(cur.b) * a.width + pi) : -1;
        const bool here = pg >= 0 && pg < a.num_pages && SV_IN(slot + a.granule - 1, a.page);
        const int there = here ? min(a.granule, (cur.w.len - tok + kKv8Block - 1) / kKv8Block * kKv8Block) : 0;  // tokens of whole blocks
        const int each = piece < 2 ? D : 1;  // bytes a slot
        const int64_t page_bytes = kv8_page_bytes(a.page, D);
        Source8 r;
        r.at = a.cache + (here ? (int64_t(pg) * a.H + cur.h) * page_bytes + min(piece, 2) * a.page * D + int64_t(slot) * each : 0);
        r.bytes = uint32_t(there * each);
        r.sum = __reduce_add_sync(0xFFFFFFFFu, piece < 2 ? r.bytes : 0u);
        r.have = __ballot_sync(0xFFFFFFFFu, here);
        return r;
    }
    __device__ __forceinline__ void advance(const Att8Args &a, int uend) {
        ++u;
        if (cur.tile + 1 < cur.tiles()) {
            ++cur.tile;
            slot += Sh::kTile;
            while (slot >= a.page) slot -= a.page, ++pi;
        } else if (u < uend) {
            cur.next(a, Sh::kRows, u);
            placed = false;
        }
    }
};

// The copying warp.  Keys and words, values, and segments' queries each go as far ahead as their rings have room.  Returns when all that it has begun is there.
template <typename Sh>
__device__ __forceinline__ void copy_tiles8(const Att8Args &a, Sh &sh, Cursor<Sh::kTile> &cur, int ubegin, int uend, int lane) {
    constexpr int NT = Sh::kTile, D = Sh::kDims, NR = Sh::kRows, kStages = Sh::kStages, kValues = Sh::kValues;
    const int gi = lane & 7, piece = lane >> 3, granules = NT / a.granule;  // lanes 0 .. 7 keys, 8 .. 15 words, 16 .. 23 values
    const uint32_t all = (1u << granules) - 1;
    const int units = uend - ubegin;
    int keys = 0, values = 0;  // begun
    int queries = 0, qu = ubegin;  // segments whose queries are begun, and the unit with which the next one begins
    Walk8<Sh> kw{cur, ubegin}, vw{cur, ubegin};
    Cursor<NT> qc = cur;
    const uint32_t part_bytes = uint32_t(a.nq) * NR * D;
    Patience patience;
#ifdef SV_CHECKS
    const int most = g_kv_lose < 0 ? units : min(units, g_kv_lose);
#else
    const int most = units;
#endif
    while (keys < most || values < most || (qu < uend && most == units)) {
        bool did = false;
        if (qu < uend && __all_sync(0xFFFFFFFFu, queries < Sh::kQ || mbar_test(&sh.free_q[queries % Sh::kQ], uint32_t(queries / Sh::kQ - 1) & 1u))) {
            const int at = queries % Sh::kQ;
            if (lane == 0) {
                const uint8_t *src = a.parts + ((int64_t(qc.b) * a.H + qc.h) * a.row_tiles + qc.rt) * query_bytes8(D, NR);
                const uint32_t bar = smem_u32(&sh.full_q[at]);
                mbar_expect(bar, part_bytes + 4 * NR);
                bulk_load(smem_u32(sh.q[at].part), src, part_bytes, bar);
                bulk_load(smem_u32(sh.q[at].factor), src + 3 * NR * D, 4 * NR, bar);
            }
            __syncwarp();
            ++queries;
            qu += qc.tiles() - qc.tile;
            if (qu < uend) {
                qc.tile = qc.tiles() - 1;
                qc.next(a, NR, qu);
            }
            did = true;
        }
        // (a warp looks as one: the lanes' looks may differ)
        if (keys < most && __all_sync(0xFFFFFFFFu, keys < kStages || mbar_test(&sh.empty_k[keys % kStages], uint32_t(keys / kStages - 1) & 1u))) {
            const int s = keys % kStages, at = keys % Sh::kInfos;
            const Source8 src = kw.source(a, gi, piece == 1 ? 2 : 0, piece < 2 && gi < granules);
            const uint32_t have = src.have & all;
            Info8 &in = sh.info[at];
            if (lane == 0) {
                const Cursor<NT> &c = kw.cur;
                int4 *un = reinterpret_cast<int4 *>(&in.unit);
                const bool ragged = (c.tile + 1) * NT > c.w.len || have != all;
                const int flags = (ragged || (c.tile + 1) * NT > c.w.before ? kMasked8 : 0) | (ragged ? kRagged8 : 0) |
                                  (keys == 0 || c.tile == 0 ? kFirst8 : 0) | (keys + 1 == units || c.tile + 1 == c.tiles() ? kLast8 : 0);
                un[0] = make_int4(c.b, c.h, c.rt, c.tile);
                un[1] = make_int4(c.tiles(), c.w.before, c.w.len, c.live ? c.w.fresh : 0);
                un[2] = make_int4(int(have), flags, 0, 0);
                mbar_expect(smem_u32(&sh.full_i[at]), src.sum / D);  // a byte of words for D of codes
                mbar_expect(smem_u32(&sh.full_k[s]), src.sum);
            }
            __syncwarp();
            if (src.bytes && piece == 0) bulk_load(smem_u32(sh.k[s]) + gi * a.granule * D, src.at, src.bytes, smem_u32(&sh.full_k[s]));
            if (src.bytes && piece == 1) bulk_load(smem_u32(in.word) + gi * a.granule, src.at, src.bytes, smem_u32(&sh.full_i[at]));
            ++keys;
            kw.advance(a, uend);
            did = true;
        }
        if (values < most && __all_sync(0xFFFFFFFFu, values < kValues || mbar_test(&sh.empty_v[values % kValues], uint32_t(values / kValues - 1) & 1u))) {
            const int s = values % kValues;
            const Source8 src = vw.source(a, gi, 1, piece == 2 && gi < granules);
            if (lane == 0) mbar_expect(smem_u32(&sh.full_v[s]), src.sum);
            __syncwarp();
            if (src.bytes) bulk_load(smem_u32(sh.v[s]) + gi * a.granule * D, src.at, src.bytes, smem_u32(&sh.full_v[s]));
            ++values;
            vw.advance(a, uend);
            did = true;
        }
        if (did) {
            patience.reset();
        } else if (!__all_sync(0xFFFFFFFFu, patience.go_on())) {
            atomicExch(a.status, int(SV_ERR_TIMEOUT));
            break;
        } else {
            __nanosleep(100);  // (looks take instruction slots from the softmax)
        }
    }
    for (int i = max(0, keys - kStages); i < keys; ++i)
        if (!mbar_wait(smem_u32(&sh.full_k[i % kStages]), uint32_t(i / kStages) & 1u) ||
            !mbar_wait(smem_u32(&sh.full_i[i % Sh::kInfos]), uint32_t(i / Sh::kInfos) & 1u))
            atomicExch(a.status, int(SV_ERR_TIMEOUT));
    for (int i = max(0, queries - Sh::kQ); i < queries; ++i)
        if (!mbar_wait(smem_u32(&sh.full_q[i % Sh::kQ]), uint32_t(i / Sh::kQ) & 1u)) atomicExch(a.status, int(SV_ERR_TIMEOUT));
    for (int i = max(0, values - kValues); i < values; ++i)
        if (!mbar_wait(smem_u32(&sh.full_v[i % kValues]), uint32_t(i / kValues) & 1u)) atomicExch(a.status, int(SV_ERR_TIMEOUT));
}

// The issuing thread.
template <int D, int NR, int NP>
__device__ __forceinline__ void issue_products8(const Att8Args &a, Att8Shared<D, NR, NP> &sh, int units, int nq) {
    using Sh = Att8Shared<D, NR, NP>;
    constexpr int kStages = Sh::kStages, kValues = Sh::kValues, MB = Sh::MB;
    const uint32_t tmem = sh.tmem;
    int segment = -1, flags = 0;  // of the next scores' unit, once its keys are there
    bool known = false;
    auto scores = [&](int n) {
        const int s = n % kStages;
        if (!known) {
            if (!mbar_test(&sh.full_k[s], uint32_t(n / kStages) & 1u)) return false;
            flags = sh.info[n % Sh::kInfos].unit.masked;
            if (flags & kFirst8) ++segment;
            known = true;
        }
        if ((flags & kFirst8) && !mbar_test(&sh.full_q[segment % Sh::kQ], uint32_t(segment / Sh::kQ) & 1u)) return false;
        if (n >= 2 && !mbar_test(&sh.free_s[n & 1], uint32_t((n >> 1) - 1) & 1u)) return false;
        known = false;
        fence_after();
        constexpr uint32_t high = operand8_high(8 * D);
        const uint32_t d = tmem + (n & 1) * Sh::kScoreCols, k = operand8(smem_u32(sh.k[s]), 128);
        uint32_t q = operand8(smem_u32(sh.q[segment % Sh::kQ].part), 128);
        if constexpr (Sh::kStackQ) {
            const uint32_t kind = kind8(NR, false) + uint32_t((nq - 1) * NR / 8) * (1u << 17);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) mma8(d, k + i * 16, high, q + i * 16, high, kind, i > 0);
        } else {
#pragma unroll
            for (int p = 0; p < 3; ++p, q += NR * D / 16)
                if (p < 2 || nq > 2) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) mma8(d, k + i * 16, high, q + i * 16, high, kind8(NR, false), p > 0 || i > 0);
                }
        }
        wide_commit(&sh.empty_k[s]);
        wide_commit(&sh.full_s[n & 1]);
        if (flags & kLast8) wide_commit(&sh.free_q[segment % Sh::kQ]);
        return true;
    };
    auto products = [&](int n) {
        const int s = n % kValues;
        if (!mbar_test(&sh.full_w[n & 1], uint32_t(n >> 1) & 1u) || !mbar_test(&sh.full_v[s], uint32_t(n / kValues) & 1u)) return false;
        if (n >= 2 && !mbar_test(&sh.free_o[n & 1], uint32_t((n >> 1) - 1) & 1u)) return false;
        fence_after();
        const uint32_t d = tmem + 2 * Sh::kScoreCols + (n & 1) * Sh::kOutCols;
        const uint32_t v = operand8(smem_u32(sh.v[s]), 8 * D), w = operand8(smem_u32(sh.w), 128);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int p = 0; p < NP; p += Sh::kStackP)
#pragma unroll
                for (int i = 0; i < kTile8 / 32; ++i)
                    mma8(d + mb * Sh::kOutEach, v + mb * 64 + i * 2 * D, operand8_high(128), w + p * 2 * NR * kTile8 / 16 + i * 32, operand8_high(2048),
                         kind8(2 * NR * (p + Sh::kStackP <= NP ? Sh::kStackP : 1), true, true), p > 0 || i > 0);
        wide_commit(&sh.empty_v[s]);
        wide_commit(&sh.full_o[n & 1]);
        return true;
    };
    Patience patience;
    for (int ns = 0, np = 0; np < units;) {
        if (np < ns && products(np)) {
            ++np, patience.reset();
        } else if (ns < units && scores(ns)) {
            ++ns, patience.reset();
        } else if (!patience.go_on()) {  // nothing more is issued; the other warps' waits give up too
            atomicExch(a.status, int(SV_ERR_TIMEOUT));
            break;
        } else if (np < ns) {  // asleep until what comes next is likely there
            mbar_doze(&sh.full_w[np & 1], uint32_t(np >> 1) & 1u);
        } else {
            mbar_doze(&sh.full_k[ns % kStages], uint32_t(ns / kStages) & 1u);
        }
    }
    // nothing may be under way when the block ends
    wide_commit(&sh.done);
    if (!mbar_wait(smem_u32(&sh.done), 0)) atomicExch(a.status, int(SV_ERR_TIMEOUT));
}

// The queries in parts, for all segments (sequence, kv head, row tile): each row rotated, times a power of two that brings its largest number to
// 2^7 .. 2^8.  A row with a NaN or an infinity is NaN throughout.  D / 8 lanes a row.  The blocks behind those have a row tile each
// of a tree's words (which rows see a new token).  A kernel of its own: two warps of the attention's blocks took 20 us a segment for it, beside
// instructions that the softmax then had to fetch again.
constexpr int kQueryThreads8 = 256;

template <int D>
__global__ void __launch_bounds__(kQueryThreads8) kv8_queries_kernel(const Att8Args a) {
    constexpr int L = D / 8;
    extern __shared__ uint32_t see_s[];
    const int tid = threadIdx.x;
    griddep_launch_next();
    griddep_wait();
    if (int64_t(blockIdx.x) >= a.query_blocks) {
        const int rt = int(blockIdx.x - a.query_blocks), words = (a.wide ? a.nr : a.T) * a.see_words;
        for (int i = tid; i < words; i += kQueryThreads8) see_s[i] = 0;
        __syncthreads();
        if (tid < a.nr) {
            const int64_t node = (int64_t(rt) * a.nr + tid) / a.G;
            for (int v = node < a.T ? int(node) : -1; v >= 0;) {
                if (a.wide)
                    see_s[tid * a.see_words + v / 32] |= 1u << (v & 31);
                else
                    atomicOr(see_s + v * a.see_words + tid / 32, 1u << (tid & 31));
                const int up = __ldg(a.parent + v);
                v = up < v ? up : -1;
            }
        }
        __syncthreads();
        for (int i = tid; i < words; i += kQueryThreads8) a.see[int64_t(rt) * words + i] = see_s[i];
        return;
    }
    const int64_t row = (int64_t(blockIdx.x) * kQueryThreads8 + tid) / L;
    const int64_t tile = row / a.nr;
    const int r = int(row - tile * a.nr), c = tid % L, d0 = c * 8;
    const bool inside = tile < int64_t(a.B) * a.H * a.row_tiles;
    Unit un{};
    int node = 0, head = 0;
    bool on = false;
    if (inside) {
        const int64_t bh = tile / a.row_tiles;
        un.rt = int(tile - bh * a.row_tiles), un.b = int(bh / a.H), un.h = int(bh - int64_t(un.b) * a.H);
        kv_lengths(a.start, a.new_lens, un.b, a.T, int64_t(a.width) * a.page, un.before, un.fresh);
        const int at = un.rt * a.nr + r;
        node = at / a.G, head = un.h * a.G + at - node * a.G;
        on = node < un.fresh;
    }
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (on) query_chunk(a, un, node, head, d0, x);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = a.scale == 0.f ? x[i] * 0.f : a.scale < 0.f ? -x[i] : x[i];  // (factors are above 0)
        top = max(top, __float_as_uint(fabsf(x[i])));
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (!inside) return;
    const int e2 = top == 0 ? 0 : max(int(top >> 23) - 127 - 7, -110);
    const bool odd = top >= 0x7F800000u;
    const float shrink = power2(odd ? 0 : -e2);
    uint32_t code[2][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = odd ? NAN : x[i] * shrink;
#pragma unroll
    for (int i = 0; i < 2; ++i) parts8(two(x[4 * i], x[4 * i + 1]), two(x[4 * i + 2], x[4 * i + 3]), code[i]);
    uint8_t *q = a.parts + tile * query_bytes8(D, a.nr);
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < a.nq) *reinterpret_cast<uint2 *>(q + kv8_code_byte(D, k * a.nr + r, d0)) = make_uint2(code[0][k], code[1][k]);
    if (c == 0) reinterpret_cast<float *>(q + 3 * a.nr * D)[r] =
            a.scale == 0.f ? 1.f : fmaxf(fabsf(a.scale) * 1.4426950408889634f * power2(odd ? 0 : e2), 1.2e-38f);
}

template <int D, int NR, int NP>
__global__ void __launch_bounds__(att8_threads(NR), att8_occupancy(D, NR)) kv8_attention_kernel(const Att8Args a) {
    using Sh = Att8Shared<D, NR, NP>;
    constexpr int W = Sh::W, RW = Sh::RW, MB = Sh::MB, kValues = Sh::kValues;
    extern __shared__ unsigned char raw0[];
    unsigned char *raw = raw0 + ((128 - (smem_u32(raw0) & 127)) & 127);
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = int(gridDim.x), cta = int(blockIdx.x);

    griddep_launch_next();
    if (tid == 0) {
        for (int i = 0; i < Sh::kStages; ++i) mbar_init(smem_u32(&sh.full_k[i]), 1), mbar_init(smem_u32(&sh.empty_k[i]), 1);
        for (int i = 0; i < kValues; ++i) mbar_init(smem_u32(&sh.full_v[i]), 1), mbar_init(smem_u32(&sh.empty_v[i]), 1);
        for (int i = 0; i < 2; ++i)
            mbar_init(smem_u32(&sh.full_s[i]), 1), mbar_init(smem_u32(&sh.free_s[i]), 4 * W), mbar_init(smem_u32(&sh.full_o[i]), 1),
                mbar_init(smem_u32(&sh.free_o[i]), 4 * W), mbar_init(smem_u32(&sh.full_w[i]), 4 * W);
        for (int i = 0; i < Sh::kQ; ++i) mbar_init(smem_u32(&sh.full_q[i]), 1), mbar_init(smem_u32(&sh.free_q[i]), 4 * W + 1);
        for (int i = 0; i < Sh::kInfos; ++i) mbar_init(smem_u32(&sh.full_i[i]), 1);
        mbar_init(smem_u32(&sh.done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    griddep_wait();
    if (cta == 0 && tid == 0) *a.status = SV_OK;
    Cursor<kTile8> cur;
    int total, ubegin, uend;
    if (!find_share<kTile8>(a, NR, lane, cta, ncta, cur, total, ubegin, uend)) {
        if (tid == 0) a.desc[cta] = AttDesc{0, 0, 0, 0, 0, 0, 0, 0};
        return;
    }
    if (tid == 0)  // the share's first segment (at once: the join reads this whether or not a wait gives up)
        a.desc[cta] = describe(total, cta, ncta, ubegin, ubegin - cur.tile, ubegin - cur.tile + cur.tiles(), cur.b, cur.h, cur.rt, cur.live ? cur.w.fresh : 0);
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"(Sh::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        fence_before();
    }
    __syncthreads();
    fence_after();
    const int units = uend - ubegin;
    if (warp == 0) {
        copy_tiles8(a, sh, cur, ubegin, uend, lane);
    } else if (warp == 1) {
        if (lane == 0) issue_products8<D, NR, NP>(a, sh, units, a.nq);
        __syncwarp();
    } else {
        const int wg = (warp - 2) / 4, quarter = warp & 3, nq = a.nq, token = quarter * 32 + lane;
        const int r0 = wg * RW;  // the group's first row
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const uint32_t tmem_s = sh.tmem + lanes + r0, tmem_o = sh.tmem + lanes + 2 * Sh::kScoreCols + r0;
        const bool writes = D >= 128 || quarter < 2;  // has a dimension
        int granule_log2 = 4;
        while (1 << granule_log2 < a.granule) ++granule_log2;
        auto any = [&](bool x) {
            if (W > 3 && wg == 3) return group_or<4, 128>(x);
            if (W > 2 && wg == 2) return group_or<5, 128>(x);
            if (W > 1 && wg == 1) return group_or<2, 128>(x);
            return group_or<1, 128>(x);
        };
        bool failed = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!warp_wait(bar, parity) && !failed) {
                failed = true;
                atomicExch(a.status, int(SV_ERR_TIMEOUT));
            }
        };
        Unit seg{};
        int seg_lo = 0, segment = -1, live = 0;  // live: rows of this group
        Two l[RW / 2], acc[MB][RW / 2];
        float M = -INFINITY;  // of row lane % 16 of the group
        // the output of unit n, which is of the segment at hand
        auto take_up = [&](int n) {
            wait(&sh.full_o[n & 1], uint32_t(n >> 1) & 1u);
            if (failed) return;
            fence_after();
            if (writes) {
                constexpr int cols = 2 * Sh::kStackP;  // of a row: the ranges' parts
                constexpr float lowered = 1.f / (1 << Weights8<NP>::kLift);
                const uint32_t o_at = tmem_o + (n & 1) * Sh::kOutCols;
#pragma unroll
                for (int c = 0; c < RW / 8; ++c) {
                    if (8 * c >= live) continue;
                    float o[MB][cols][8];
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                        for (int p = 0; p < cols; ++p) tmem_get8(o[mb][p], o_at + mb * Sh::kOutEach + p * NR + 8 * c);
                    tmem_loaded();
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                        for (int p = 0; p < cols; ++p) tmem_here(o[mb][p]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 mv = sh.move[wg][quarter][n & 1][4 * c + j];
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb) {
                            Two x = two(o[mb][0][2 * j], o[mb][0][2 * j + 1]), y = two(o[mb][1][2 * j], o[mb][1][2 * j + 1]);
                            if (Sh::kStackP == 2)
                                x = add2(x, two(o[mb][cols - 2][2 * j], o[mb][cols - 2][2 * j + 1])), y = add2(y, two(o[mb][cols - 1][2 * j], o[mb][cols - 1][2 * j + 1]));
                            x = fma2(y, two(lowered, lowered), x);
                            acc[mb][4 * c + j] = fma2(x, two(mv.z, mv.w), acc[mb][4 * c + j]);
                        }
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.free_o[n & 1]));
        };

        for (int n = 0; n < units; ++n) {
            const Info8 &in = sh.info[n % Sh::kInfos];
            wait(&sh.full_i[n % Sh::kInfos], uint32_t(n / Sh::kInfos) & 1u);
            int flags = 0;
            float t[RW], inv = 0.f;  // inv: 1 / s', 0: not there
            if (!failed) {
                flags = in.unit.masked;
                if (flags & kFirst8) {
                    seg = in.unit;
                    ++segment;
                    seg_lo = ubegin + n - seg.tile;
                    live = min(max(seg.fresh * a.G - seg.rt * NR - r0, 0), RW);
                    M = -INFINITY;
#pragma unroll
                    for (int j = 0; j < RW / 2; ++j) l[j] = acc[0][j] = acc[MB - 1][j] = 0;
                    wait(&sh.full_q[segment % Sh::kQ], uint32_t(segment / Sh::kQ) & 1u);
                }
                // the scale of this thread's token, and the rows that see it
                const int at = segment % Sh::kQ;
                float ks = 0.f, log2vs = 0.f;
                uint32_t see = 0xFFFFu;
                bool there = true;
                if (flags & kMasked8) {
                    const int j = in.unit.tile * kTile8 + token, x = j - seg.before;  // among the new tokens
                    there = j < seg.len && (in.unit.have >> (token >> granule_log2) & 1u);
                    see = there ? (1u << live) - 1 : 0u;
                    if (there && x >= 0) {
                        if (a.parent) {
                            see &= __ldcg(a.see + (int64_t(seg.rt) * a.T + x) * Sh::SW + wg / 2) >> (16 * (wg & 1));
                        } else {
                            see &= 0xFFFFu << min(max(x * a.G - seg.rt * NR - r0, 0), 16);  // not the rows of earlier tokens
                        }
                    }
                }
                if (there) {
                    const uint2 word = *reinterpret_cast<const uint2 *>(in.word[token / kKv8Block]);
                    const int e = kv8_exponent(word.y);
                    ks = (word.x | word.y) >> (token & 15) & 1u ? NAN : __uint_as_float(word.x & 0xFFFF0000u);
                    log2vs = float(e), inv = kv8_power(-e);
                }
                if (flags & kRagged8) wait(&sh.full_v[n % kValues], uint32_t(n / kValues) & 1u);
                wait(&sh.full_s[n & 1], uint32_t(n >> 1) & 1u);
                fence_after();
                const Two ks2 = two(ks, ks), vs2 = two(log2vs, log2vs);
                const uint32_t s_at = tmem_s + (n & 1) * Sh::kScoreCols;
                constexpr int parts = Sh::kStackQ ? 3 : 1;
#pragma unroll
                for (int c = 0; c < RW / 8; ++c) {
                    if (8 * c >= live) continue;
                    float x[parts][8], most[8];
                    tmem_get8(x[0], s_at + 8 * c);
                    if constexpr (parts > 1) {
                        tmem_get8(x[1], s_at + NR + 8 * c);
                        tmem_get8(x[2], s_at + (nq > 2 ? 2 * NR : NR) + 8 * c);
                    }
                    tmem_loaded();
#pragma unroll
                    for (int p = 0; p < parts; ++p) tmem_here(x[p]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = *reinterpret_cast<const float2 *>(&sh.q[at].factor[r0 + 8 * c + 2 * j]);
                        Two y = two(x[0][2 * j], x[0][2 * j + 1]);
                        if constexpr (parts > 1) {
                            const Two z = two(x[1][2 * j], x[1][2 * j + 1]);
                            y = add2(y, nq > 2 ? add2(z, two(x[2][2 * j], x[2][2 * j + 1])) : z);
                        }
                        const float2 u = split(fma2(mul2(y, two(f.x, f.y)), ks2, vs2));
                        t[8 * c + 2 * j] = u.x, t[8 * c + 2 * j + 1] = u.y;
                    }
                    if (flags & kMasked8) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (!(see >> (8 * c + j) & 1u)) t[8 * c + j] = -INFINITY;
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) most[j] = warp_largest(t[8 * c + j]);
                    if (lane == 0) {
                        float4 *to = reinterpret_cast<float4 *>(&sh.red[wg][n & 1][quarter][8 * c]);
                        to[0] = make_float4(most[0], most[1], most[2], most[3]), to[1] = make_float4(most[4], most[5], most[6], most[7]);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) {  // the scores and what is known of the unit are read
                    mbar_arrive(smem_u32(&sh.free_s[n & 1]));
                    if (flags & kLast8) mbar_arrive(smem_u32(&sh.free_q[at]));
                }
            }
            if (any(failed)) break;
            {  // each warp for itself: m, and what it makes of M (lane: row)
                const int row = lane & 15;
                const float(*red)[RW] = sh.red[wg][n & 1];
                const float m = fmaxf(fmaxf(red[0][row], red[1][row]), fmaxf(red[2][row], red[3][row]));
                const float whole = rintf(m);
                float f = 1.f, g = 1.f, minus = m == INFINITY ? -INFINITY : 0.f;
                if (row < live && fabsf(whole) < INFINITY) {
                    if (M == -INFINITY) M = whole;
                    if (whole > M + 60.f) g = ex2(fmaxf(M - whole, -126.f)), M = whole;
                    f = ex2(fmaxf(whole - M, -127.f));
                    minus = kTop8 - whole;
                }
                float *mv = reinterpret_cast<float *>(&sh.move[wg][quarter][n & 1][row / 2]);
                if (lane < 16) mv[row & 1] = minus, mv[2 + (row & 1)] = f;
                if (__any_sync(0xFFFFFFFFu, g != 1.f)) {  // (rare; the last unit's output, not taken up yet, is to move too)
                    if (lane < 16) reinterpret_cast<float *>(&sh.move[wg][quarter][(n & 1) ^ 1][row / 2])[2 + (row & 1)] *= g;
#pragma unroll
                    for (int j = 0; j < RW / 2; ++j) {
                        const Two g2 = two(__shfl_sync(0xFFFFFFFFu, g, 2 * j), __shfl_sync(0xFFFFFFFFu, g, 2 * j + 1));
                        l[j] = mul2(l[j], g2);
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb) acc[mb][j] = mul2(acc[mb][j], g2);
                    }
                }
                __syncwarp();
            }
            // the weights
            const bool first = (flags & kFirst8) != 0, last = (flags & kLast8) != 0;
            if (!first) wait(&sh.full_o[(n & 1) ^ 1], uint32_t((n - 1) >> 1) & 1u);  // the last unit's weights are in the place of these
            if (!failed) {
                const Two inv2 = two(inv, inv);
                uint8_t *to = sh.w[0][0] + wg * 2048 + token * 16;
#pragma unroll
                for (int c = 0; c < RW / 8; ++c) {
                    if (8 * c >= live) continue;
                    uint32_t upper[2][NP], lower[2][NP];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        Two w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int at = 4 * c + 2 * j + i;  // the pair of rows
                            const float4 mv = sh.move[wg][quarter][n & 1][at];
                            const float2 x = split(add2(two(t[2 * at], t[2 * at + 1]), two(mv.x, mv.y)));
                            w[i] = two(ex2(x.x), ex2(x.y));
                            l[at] = fma2(mul2(w[i], inv2), two(mv.z, mv.w), l[at]);
                        }
                        weight_parts8<NP>(w, upper[j], lower[j]);
                    }
#pragma unroll
                    for (int k = 0; k < NP; ++k) {  // (both halves of 16 bytes at once were slower: their registers spill)
                        *reinterpret_cast<uint2 *>(to + 2 * k * NR * kTile8 + 8 * c) = make_uint2(upper[0][k], upper[1][k]);
                        *reinterpret_cast<uint2 *>(to + (2 * k + 1) * NR * kTile8 + 8 * c) = make_uint2(lower[0][k], lower[1][k]);
                    }
                }
                if ((flags & kRagged8) && wg == 0 && inv == 0.f) {  // a code that is not there may be a NaN, which no weight of 0 takes away
                    uint8_t *v = sh.v[n % kValues];
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) *reinterpret_cast<uint4 *>(v + kv8_code_byte(D, token, 16 * j)) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_operands();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.full_w[n & 1]));
            // the last unit's output, and at the segment's end this one's
#pragma unroll 1
            for (int j = first ? n : n - 1; j <= (last ? n : n - 1); ++j) take_up(j);
            if (!last) continue;

            // the segment's end
            {  // the weights' sums over the warp: at each step a lane keeps half of the rows, in the end row lane / 2
                float x[RW];
#pragma unroll
                for (int i = 0; i < RW; ++i) x[i] = i & 1 ? split(l[i / 2]).y : split(l[i / 2]).x;
#pragma unroll
                for (int o = 16, rows = RW / 2; o > 1; o >>= 1, rows >>= 1) {
                    const bool up = lane & o;
#pragma unroll
                    for (int i = 0; i < RW / 2; ++i)
                        if (i < rows) {
                            const float give = up ? x[i] : x[i + rows];
                            x[i] = (up ? x[i + rows] : x[i]) + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                        }
                }
                x[0] += __shfl_xor_sync(0xFFFFFFFFu, x[0], 1);
                if (!(lane & 1)) sh.sums[wg][quarter][lane / 2] = x[0];
            }
            if (any(failed)) break;
            const bool whole = seg_lo >= ubegin && seg_lo + seg.tiles <= uend;
            const int64_t slot = 2 * cta + (seg_lo > ubegin ? 1 : 0);
            const int row = lane & 15;
            const float sum = (sh.sums[wg][0][row] + sh.sums[wg][1][row]) + (sh.sums[wg][2][row] + sh.sums[wg][3][row]);
            const float part = row >= live || sum == 0.f ? 0.f : 1.f / sum;
            if (!whole && token < RW && SV_IN(slot, 2 * ncta)) a.ml[slot * NR + r0 + row] = make_float2(M, sum);
            const int first_row = seg.rt * NR + r0;
            int node = first_row / a.G, head = first_row - node * a.G;
            uint16_t *out = a.out + (seg.b * int64_t(a.T) * a.H + seg.h) * a.G * D + token;  // of token 0's first head
            float *part_out = a.acc + (slot * NR + r0) * D + token;
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const float scale = __shfl_sync(0xFFFFFFFFu, part, i);
                if (node < a.T && writes) {
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb) {
                        const float2 x2 = split(acc[mb][i / 2]);
                        const float x = i & 1 ? x2.y : x2.x;
                        if (whole)
                            out[(int64_t(node) * a.H * a.G + head) * D + mb * 128] = kv_from_float(scale == 0.f ? 0.f : x * scale, a.bf16);
                        else if (SV_IN(slot, 2 * ncta))
                            part_out[i * D + mb * 128] = x;
                    }
                }
                if (++head == a.G) head = 0, ++node;
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(Sh::kCols));
}

template <int D>
cudaError_t launch_queries8(const Att8Args &a, cudaStream_t s) {
    const size_t smem = a.parent ? size_t(a.wide ? a.nr : a.T) * a.see_words * 4 : 0;  // at most 17 KB
    const unsigned blocks = unsigned(a.query_blocks + (a.parent ? a.row_tiles : 0));
    return launch_after(kv8_queries_kernel<D>, blocks, unsigned(kQueryThreads8), smem, s, a);
}

template <int D, int NR, int NP>
cudaError_t launch_attention8(const Att8Args &a, int grid, cudaStream_t s) {
    using Sh = Att8Shared<D, NR, NP>;
    constexpr size_t smem = sizeof(Sh) + 128;
    static_assert(smem <= 227 * 1024 && (smem + 1024) * att8_occupancy(D, NR) <= 228 * 1024, "");
    static_assert(sizeof(typename Sh::Queries) == query_bytes8(D, NR) && Sh::kUsed <= Sh::kCols && Sh::kCols * att8_occupancy(D, NR) <= 512, "");
    static std::atomic<int> allowed[64];
    cudaError_t e = allow_shared(kv8_attention_kernel<D, NR, NP>, int(smem), allowed);
    if (e != cudaSuccess) return e;
    e = launch_after(kv8_attention_kernel<D, NR, NP>, unsigned(grid), unsigned(att8_threads(NR)), smem, s, a);
    if (e != cudaSuccess) return e;
    return launch_join<D>(a, grid, NR, s);
}

// The kernels of a head dimension and number of weights' parts, each in its own translation unit.
template <int D, int NP>
cudaError_t launch_attention8_rows(const Att8Args &a, int grid, cudaStream_t s);

#define SV_KV8_ATTENTION_INSTANTIATE(D, NP)                                                                   \
    template <>                                                                                              \
    cudaError_t launch_attention8_rows<D, NP>(const Att8Args &a, int grid, cudaStream_t s) {    \
        cudaError_t e = launch_queries8<D>(a, s);                                                              \
        if (e != cudaSuccess) return e;                                                                       \
        if constexpr (att8_cap(D) >= 64) {                                                                    \
            if (a.nr == 64) return launch_attention8<D, 64, NP>(a, grid, s);                                   \
        }                                                                                                     \
        return a.nr == 16   ? launch_attention8<D, 16, NP>(a, grid, s)                                         \
               : a.nr == 32 ? launch_attention8<D, 32, NP>(a, grid, s)                                         \
                            : launch_attention8<D, 48, NP>(a, grid, s);                                        \
    }

}  // namespace sv
