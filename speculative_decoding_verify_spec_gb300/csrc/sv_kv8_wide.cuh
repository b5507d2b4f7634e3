// sv_kv8_wide.cuh -- the attention over the 8-bit paged cache for many query rows a kv head (drafts, token trees): 128 rows
// a tile, a thread of the softmax has one row.
//
// The sums are those of sv_kv8_attention.cuh, and so are the queries' parts, the copying warp, the list of units and the join.  Here
// the rows are the products' 128-row operand and the cache's bytes the other one:
//   S [128 rows x tokens] = q [128 x D]  times  K codes^T         8-bit floats, D / 32 steps a part of q
//   O [128 rows x D]      = w [128 x tokens]  times  V codes      bfloat16, a step for 16 tokens and part of w
// so that a row's maximum and sum need no reduction over lanes, a block of 16 tokens has its scales in registers, and m is taken out in the
// multiplication that scales a score.  Two or four groups of 128 threads have the 128 rows each, and their share of
// the tile's tokens and of the output's dimensions.  The scores are read from tensor memory twice, for the maximum and for the weights, 16 tokens
// at a time, instead of kept.  As there, every tile has its own m and output, which is added up in registers.
//
// A weight is held in two bfloat16 parts: off by 2^-17 of itself however far below the tile's largest it is, for bfloat16 has the exponents of fp32.  The
// value codes are widened for that once a tile, by the softmax's threads: once for 128 rows.  (In parts of 8 bits and one
// range, against the codes as they lie, two parts took 116 and three 130 us in the first case below, and lost weights of 2^-18 of the largest.)
//
// Measured: 64 x 64 tree nodes with 4 query heads a kv head over up to 2047 tokens, us: 64 dimensions 129 to 132, 27 instructions
// for each row and token, 2.3 a clock, the tensor pipe at 33 %; 128 dimensions 165 to 174.  A tile's path
// through a block (scores, maximum, barrier, weights, product) is covered by the other block of the SM only in part, and at 128 dimensions by none.
// 256 dimensions, whose queries leave shared memory for a tile of 64 tokens and one place for all else, took 242, 435 and 457 us
// for 128, 192 and 256 rows where tiles of 48 rows of the other kernel take 229, 296 and 435 (bf16, rotated): they go there.
#pragma once

#include "sv_kv8_attention.cuh"

namespace sv {

constexpr int kWideRows8 = 128;
__host__ __device__ constexpr bool wide8_has(int D) { return D <= 128; }  // (256: above)
// Softmax groups of a block and blocks an SM: two blocks hide each other's waits where registers and shared memory admit them.
__host__ __device__ constexpr int wide8_groups(int D) { return D == 64 ? 2 : 4; }
__host__ __device__ constexpr int wide8_occupancy(int D) { return D == 64 ? 2 : 1; }
__host__ __device__ constexpr int wide8_threads(int D) { return 64 + 128 * wide8_groups(D); }
__host__ __device__ constexpr int wide8_tile(int D) { return D == 64 ? 64 : 128; }  // by shared memory

template <int D>
struct Wide8Shared {
    static constexpr int kDims = D, kRows = kWideRows8, kTile = wide8_tile(D);
    static constexpr int kStages = D == 64 ? 3 : 2, kValues = kStages, kInfos = kStages + 2, kQ = 1, kGroups = wide8_groups(D);
    static constexpr int kS = 2, kO = 2;  // scores and outputs in tensor memory
    static constexpr int kUsed = kS * kTile + kO * D, kCols = kUsed <= 256 ? 256 : 512;
    alignas(128) uint8_t k[kStages][kTile * D];
    uint8_t v[kValues][kTile * D];
    uint16_t wide[kTile * D];      // the values' codes as bfloat16
    uint16_t w[2][kRows * kTile];  // [part][8 tokens][row][8]
    struct Queries {
        uint8_t part[3][kRows * D];
        float factor[kRows];
    };
    Queries q[kQ];
    Info8 info[kInfos];
    float red[2][kGroups][kRows], sums[kGroups][kRows];
    alignas(8) uint64_t full_k[kStages], full_v[kValues], empty_k[kStages], empty_v[kValues], full_i[kInfos];
    uint64_t full_s[kS], free_s[kS], full_o[kO], free_o[kO], full_w[2], full_q[kQ], free_q[kQ], done;
    uint32_t tmem;
};

// bfloat16 into fp32, 128 rows, N columns, and a product of them (its operands as those in 8 bits).
__device__ __forceinline__ constexpr uint32_t kind16(int N) { return 1u << 4 | 1u << 7 | 1u << 10 | uint32_t(N / 8) << 17 | 8u << 24; }
__device__ __forceinline__ void mma16(uint32_t d, uint32_t a, uint32_t a_high, uint32_t b, uint32_t b_high, uint32_t kind, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(kind), "r"(uint32_t(add))
        : "memory");
}

// The values' codes as bfloat16: a code's exponent and mantissa in the place of those stand for 2^-120 times its number, the smallest codes
// (no exponent) as numbers without one too.  What the factor lacks is in the weights (2^76) and in what takes up the output.
constexpr int kWidened8 = 120, kLifted8 = 76;
__device__ __forceinline__ uint2 widened4(uint32_t c) {
    const uint32_t high = (c & 0x80808080u) | (c >> 4 & 0x07070707u), low = c << 4 & 0xF0F0F0F0u;  // each code's bytes
    return make_uint2(__byte_perm(low, high, 0x5140), __byte_perm(low, high, 0x7362));
}
// A tile's values, from eight tokens by 16 bytes a block to eight by 8 numbers; by kThreads threads.  there(i): whether token i is there (a
// code that is not may be a NaN, which no weight of 0 takes away).
template <int D, int kTokens, int kThreads, typename There>
__device__ __forceinline__ void widen8(const uint8_t *v, uint16_t *wide, int thread, bool ragged, There there) {
    constexpr int kEach = kTokens * D / 16 / kThreads;
    static_assert(kEach * kThreads * 16 == kTokens * D, "");
    uint4 c[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) c[i] = reinterpret_cast<const uint4 *>(v)[thread + i * kThreads];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = thread + i * kThreads;
        if (ragged && !there(at / (D / 2) * 8 + at % 8)) c[i] = make_uint4(0, 0, 0, 0);
        const uint2 x = widened4(c[i].x), y = widened4(c[i].y), z = widened4(c[i].z), w = widened4(c[i].w);
        uint4 *to = reinterpret_cast<uint4 *>(wide) + at / 8 * 16 + at % 8;
        to[0] = make_uint4(x.x, x.y, y.x, y.y), to[8] = make_uint4(z.x, z.y, w.x, w.y);
    }
}
// Two weights times 2^76 in two parts, the first one's in the lower half: bfloat16 has the exponents of fp32, so that a weight keeps 16 bits
// whatever the others are.
__device__ __forceinline__ void weight_parts16(Two w, uint32_t &first, uint32_t &rest) {
    constexpr float lift = 75557863725914323419136.f;
    w = mul2(w, two(lift, lift));
    const float2 f = split(w);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(first) : "f"(f.y), "f"(f.x));
    const float2 r = split(fma2(two(__uint_as_float(first << 16), __uint_as_float(first & 0xFFFF0000u)), two(-1.f, -1.f), w));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(r.y), "f"(r.x));
}

// The issuing thread.
template <int D>
__device__ __forceinline__ void issue_wide8(const Att8Args &a, Wide8Shared<D> &sh, int units) {
    using Sh = Wide8Shared<D>;
    constexpr int kStages = Sh::kStages, NT = Sh::kTile;
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
        if (n >= Sh::kS && !mbar_test(&sh.free_s[n % Sh::kS], uint32_t(n / Sh::kS - 1) & 1u)) return false;
        known = false;
        fence_after();
        constexpr uint32_t high = operand8_high(8 * D);
        const uint32_t d = tmem + n % Sh::kS * NT, k = operand8(smem_u32(sh.k[s]), 128);
        uint32_t q = operand8(smem_u32(sh.q[segment % Sh::kQ].part), 128);
#pragma unroll
        for (int p = 0; p < 3; ++p, q += kWideRows8 * D / 16)
            if (p < 2 || a.nq > 2) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) mma8(d, q + i * 16, high, k + i * 16, high, kind8(NT, false), p > 0 || i > 0);
            }
        wide_commit(&sh.empty_k[s]);
        wide_commit(&sh.full_s[n % Sh::kS]);
        if (flags & kLast8) wide_commit(&sh.free_q[segment % Sh::kQ]);
        return true;
    };
    auto products = [&](int n) {
        const int at = n % Sh::kO;
        if (!mbar_test(&sh.full_w[n & 1], uint32_t(n >> 1) & 1u)) return false;  // (the values are there as well)
        if (n >= Sh::kO && !mbar_test(&sh.free_o[at], uint32_t(n / Sh::kO - 1) & 1u)) return false;
        fence_after();
        const uint32_t d = tmem + Sh::kS * NT + at * D, v = operand8(smem_u32(sh.wide), 16 * D), w = operand8(smem_u32(sh.w), 2048);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < NT / 16; ++i)
                mma16(d, w + (p * kWideRows8 * NT * 2 + i * 4096) / 16, operand8_high(128), v + i * 2 * D, operand8_high(128),
                      kind16(D) | 1u << 16, p > 0 || i > 0);  // (the values have their rows contiguous)
        wide_commit(&sh.full_o[at]);
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

template <int D>
__global__ void __launch_bounds__(wide8_threads(D), wide8_occupancy(D)) kv8_wide_kernel(const Att8Args a) {
    using Sh = Wide8Shared<D>;
    constexpr int NT = Sh::kTile, NR = kWideRows8, kValues = Sh::kValues, kGroups = Sh::kGroups, TW = NT / kGroups, CW = D / kGroups;  // a thread's tokens and dimensions
    extern __shared__ unsigned char raw0[];
    Sh &sh = *reinterpret_cast<Sh *>(raw0 + ((128 - (smem_u32(raw0) & 127)) & 127));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = int(gridDim.x), cta = int(blockIdx.x);

    griddep_launch_next();
    if (tid == 0) {
        for (int i = 0; i < Sh::kStages; ++i) mbar_init(smem_u32(&sh.full_k[i]), 1), mbar_init(smem_u32(&sh.empty_k[i]), 1);
        constexpr int kWarps = 4 * kGroups;
        for (int i = 0; i < kValues; ++i) mbar_init(smem_u32(&sh.full_v[i]), 1), mbar_init(smem_u32(&sh.empty_v[i]), kWarps);
        for (int i = 0; i < Sh::kS; ++i) mbar_init(smem_u32(&sh.full_s[i]), 1), mbar_init(smem_u32(&sh.free_s[i]), kWarps);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.full_w[i]), kWarps);
        for (int i = 0; i < Sh::kO; ++i) mbar_init(smem_u32(&sh.full_o[i]), 1), mbar_init(smem_u32(&sh.free_o[i]), kWarps);
        for (int i = 0; i < Sh::kQ; ++i) mbar_init(smem_u32(&sh.full_q[i]), 1), mbar_init(smem_u32(&sh.free_q[i]), kWarps + 1);
        for (int i = 0; i < Sh::kInfos; ++i) mbar_init(smem_u32(&sh.full_i[i]), 1);
        mbar_init(smem_u32(&sh.done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    griddep_wait();
    if (cta == 0 && tid == 0) *a.status = SV_OK;
    Cursor<NT> cur;
    int total, ubegin, uend;
    if (!find_share<NT>(a, NR, lane, cta, ncta, cur, total, ubegin, uend)) {
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
        if (lane == 0) issue_wide8<D>(a, sh, units);
        __syncwarp();
    } else {
        const int group = (warp - 2) / 4, quarter = warp & 3, r = quarter * 32 + lane;  // this thread's row
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        const uint32_t tmem_s = sh.tmem + lanes + group * TW, tmem_o = sh.tmem + lanes + Sh::kS * NT + group * CW;
        int granule_log2 = 4;
        while (1 << granule_log2 < a.granule) ++granule_log2;
        bool failed = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!warp_wait(bar, parity) && !failed) {
                failed = true;
                atomicExch(a.status, int(SV_ERR_TIMEOUT));
            }
        };
        Unit seg{};
        int seg_lo = 0, segment = -1, node = -1;
        bool warp_on = false;  // some row of the warp is live
        float factor = 1.f, M = -INFINITY, l = 0.f, f_last = 1.f;
        Two acc[CW / 2];
        // the output of unit n, which is of the segment at hand
        auto take_up = [&](int n, float f) {
            wait(&sh.full_o[n % Sh::kO], uint32_t(n / Sh::kO) & 1u);
            if (failed) return;
            fence_after();
            if (warp_on) {
                const float f44 = f * kv8_power(kWidened8 - kLifted8);
#pragma unroll
                for (int c = 0; c < CW; c += 16) {
                    float o[2][8];
                    tmem_get8(o[0], tmem_o + n % Sh::kO * D + c), tmem_get8(o[1], tmem_o + n % Sh::kO * D + c + 8);
                    tmem_loaded();
                    tmem_here(o[0]), tmem_here(o[1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[c / 2 + j] = fma2(two(o[j / 4][2 * (j % 4)], o[j / 4][2 * (j % 4) + 1]), two(f44, f44), acc[c / 2 + j]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.free_o[n % Sh::kO]));
        };

        for (int n = 0; n < units; ++n) {
            const Info8 &in = sh.info[n % Sh::kInfos];
            wait(&sh.full_i[n % Sh::kInfos], uint32_t(n / Sh::kInfos) & 1u);
            int flags = 0, left = 0;  // left: the sequence's tokens from the tile on
            uint32_t have = 0;
            uint32_t see[(TW + 31) / 32];
#pragma unroll
            for (int i = 0; i < (TW + 31) / 32; ++i) see[i] = 0xFFFFFFFFu;
            const uint32_t s_at = tmem_s + n % Sh::kS * NT;
            // 16 tokens' scores, as they are to be seen, and their scales: t = score * scale + shift, w / s' = w * inv
            auto scores = [&](int b, float (&s)[16], float &scale, float &shift, float &inv) {
                tmem_get8(*reinterpret_cast<float(*)[8]>(s), s_at + 16 * b), tmem_get8(*reinterpret_cast<float(*)[8]>(s + 8), s_at + 16 * b + 8);
                const int token = group * TW + 16 * b;  // in the tile
                uint2 word = *reinterpret_cast<const uint2 *>(in.word[token / kKv8Block]);
                // (what is not there has no scale; its tokens are not seen)
                if ((flags & kRagged8) && (token >= left || !(have >> (token >> granule_log2) & 1u)))
                    word = make_uint2(0x3F800000u, 0x3F800000u);
                const int e = kv8_exponent(word.y);
                scale = fmaxf(factor * __uint_as_float(word.x & 0xFFFF0000u), 1.2e-38f), shift = float(e), inv = kv8_power(-e);
                const uint32_t bad = (word.x | word.y) & 0xFFFFu;
                tmem_loaded();
                tmem_here(*reinterpret_cast<float(*)[8]>(s)), tmem_here(*reinterpret_cast<float(*)[8]>(s + 8));
                if ((flags & kMasked8) || bad) {  // (the same for the whole warp)
                    const uint32_t seen = (TW > 32 && b >= 2 ? see[(TW + 31) / 32 - 1] : see[0]) >> (16 * (b & 1));
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (bad >> j & 1u) s[j] = NAN;
                        if (!(seen >> j & 1u)) s[j] = -INFINITY;
                    }
                    __syncwarp();  // (a branch, not 32 selections in every block)
                }
            };
            if (!failed) {
                flags = in.unit.masked, left = in.unit.len - in.unit.tile * NT, have = in.unit.have;
                if (flags & kFirst8) {
                    seg = in.unit;
                    ++segment;
                    seg_lo = ubegin + n - seg.tile;
                    node = (seg.rt * NR + r) / a.G;
                    if (node >= seg.fresh) node = -1;
                    warp_on = __any_sync(0xFFFFFFFFu, node >= 0);
                    M = -INFINITY, l = 0.f;
#pragma unroll
                    for (int j = 0; j < CW / 2; ++j) acc[j] = 0;
                    wait(&sh.full_q[segment % Sh::kQ], uint32_t(segment / Sh::kQ) & 1u);
                    factor = sh.q[segment % Sh::kQ].factor[r];
                }
                if (flags & kMasked8) {  // which of its tokens the row sees
#pragma unroll
                    for (int i = 0; i < (TW + 31) / 32; ++i) {
                        const int in_tile = group * TW + 32 * i, tok0 = in.unit.tile * NT + in_tile;  // the first of up to 32 tokens
                        uint32_t there = 0, row = 0xFFFFFFFFu;
#pragma unroll
                        for (int b = 0; b < (TW < 32 ? TW : 32); b += 16) {  // (granules are 16 tokens at least)
                            const int more = left - (in_tile + b);
                            if (more > 0 && (have >> ((in_tile + b) >> granule_log2) & 1u)) there |= (more >= 16 ? 0xFFFFu : (1u << more) - 1) << b;
                        }
                        const int x = tok0 - seg.before;  // the first one among the new tokens
                        if (x > -32 && node >= 0) {
                            if (a.parent) {
                                const uint32_t *words = a.see + (int64_t(seg.rt) * NR + r) * a.see_words;
                                const int w = max(x, 0) >> 5;
                                const uint32_t low = w < a.see_words ? __ldcg(words + w) : 0u, high = w + 1 < a.see_words ? __ldcg(words + w + 1) : 0u;
                                row = x >= 0 ? __funnelshift_r(low, high, x & 31) : low << -x | ((1u << -x) - 1);
                            } else {
                                const int count = node + 1 - x;
                                row = count >= 32 ? 0xFFFFFFFFu : count <= 0 ? 0u : (1u << count) - 1;
                            }
                        }
                        see[i] = row & there;
                    }
                }
                wait(&sh.full_s[n % Sh::kS], uint32_t(n / Sh::kS) & 1u);
                fence_after();
                if (warp_on) {
                    float most = -INFINITY;
#pragma unroll 2
                    for (int b = 0; b < TW / 16; ++b) {
                        float s[16], scale, shift, inv;
                        scores(b, s, scale, shift, inv);
                        float top = s[0];
#pragma unroll
                        for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
                        most = fmaxf(most, fmaf(top, scale, shift));
                    }
                    sh.red[n & 1][group][r] = most;
                }
            }
            if (group_or<1, 128 * kGroups>(failed)) break;
            const bool first = (flags & kFirst8) != 0, last = (flags & kLast8) != 0;
            float f = 1.f;
            if (!first) wait(&sh.full_o[(n - 1) % Sh::kO], uint32_t((n - 1) / Sh::kO) & 1u);  // the last unit's weights and values are in the place of these
            if (warp_on && !failed) {
                float m = sh.red[n & 1][0][r];
#pragma unroll
                for (int i = 1; i < kGroups; ++i) m = fmaxf(m, sh.red[n & 1][i][r]);
                const float whole = rintf(m);
                float g = 1.f, minus = m == INFINITY ? -INFINITY : 0.f;
                if (fabsf(whole) < INFINITY) {
                    if (M == -INFINITY) M = whole;
                    if (whole > M + 60.f) g = ex2(fmaxf(M - whole, -126.f)), M = whole;
                    f = ex2(fmaxf(whole - M, -127.f));
                    minus = float(kKv8Top) - whole;
                }
                if (__any_sync(0xFFFFFFFFu, g != 1.f)) {  // (rare; the last unit's output, not taken up yet, is to move too)
                    l *= g, f_last *= g;
#pragma unroll
                    for (int j = 0; j < CW / 2; ++j) acc[j] = mul2(acc[j], two(g, g));
                }
#pragma unroll 2
                for (int b = 0; b < TW / 16; ++b) {
                    float s[16], scale, shift, inv;
                    scores(b, s, scale, shift, inv);
                    const Two a2 = two(scale, scale), b2 = two(shift + minus, shift + minus);
                    Two sum = 0;
                    uint32_t bits[2][8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 x = split(fma2(two(s[2 * j], s[2 * j + 1]), a2, b2));
                        const Two w = two(ex2(x.x), ex2(x.y));
                        sum = add2(sum, w);
                        weight_parts16(w, bits[0][j], bits[1][j]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            *reinterpret_cast<uint4 *>(sh.w[k] + (group * (TW / 8) + 2 * b + c) * (8 * NR) + r * 8) =
                                make_uint4(bits[k][4 * c], bits[k][4 * c + 1], bits[k][4 * c + 2], bits[k][4 * c + 3]);
                    const float2 both = split(sum);
                    l = fmaf((both.x + both.y) * inv, f, l);
                }
            }
            wait(&sh.full_v[n % kValues], uint32_t(n / kValues) & 1u);
            if (!failed)
                widen8<D, NT, 128 * kGroups>(sh.v[n % kValues], sh.wide, tid - 64, (flags & kRagged8) != 0,
                                             [&](int token) { return token < left && (have >> (token >> granule_log2) & 1u); });
            fence_before();
            __syncwarp();
            if (lane == 0) {  // the scores and what is known of the unit are read
                mbar_arrive(smem_u32(&sh.free_s[n % Sh::kS]));
                if (last) mbar_arrive(smem_u32(&sh.free_q[segment % Sh::kQ]));
            }
            fence_operands();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.empty_v[n % kValues])), mbar_arrive(smem_u32(&sh.full_w[n & 1]));
            // the last unit's output, and at the segment's end this one's
#pragma unroll 1
            for (int j = first ? n : n - 1; j <= (last ? n : n - 1); ++j) take_up(j, j == n ? f : f_last);
            f_last = f;
            if (!last) continue;

            // the segment's end
            sh.sums[group][r] = l;
            if (group_or<1, 128 * kGroups>(failed)) break;
            const bool whole = seg_lo >= ubegin && seg_lo + seg.tiles <= uend;
            const int64_t slot = 2 * cta + (seg_lo > ubegin ? 1 : 0);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) sum += sh.sums[i][r];
            const float part = node < 0 || sum == 0.f ? 0.f : 1.f / sum;
            const int row = seg.rt * NR + r, at = row / a.G;
            if (whole) {
                if (at < a.T) {
                    uint16_t *out = a.out + ((seg.b * int64_t(a.T) + at) * a.H * a.G + seg.h * a.G + row - at * a.G) * D + group * CW;
#pragma unroll
                    for (int c = 0; c < CW; c += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = split(acc[c / 2 + j]);
                            w[j] = uint32_t(kv_from_float(part == 0.f ? 0.f : x.x * part, a.bf16)) | uint32_t(kv_from_float(part == 0.f ? 0.f : x.y * part, a.bf16)) << 16;
                        }
                        *reinterpret_cast<uint4 *>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            } else if (SV_IN(slot, 2 * ncta)) {
                float4 *dst = reinterpret_cast<float4 *>(a.acc + (slot * NR + r) * D + group * CW);
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    const float2 x = split(acc[c / 2]), y = split(acc[c / 2 + 1]);
                    dst[c / 4] = make_float4(x.x, x.y, y.x, y.y);
                }
                if (group == 0) a.ml[slot * NR + r] = make_float2(M, sum);
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
cudaError_t launch_wide8(const Att8Args &a, int grid, cudaStream_t s) {
    using Sh = Wide8Shared<D>;
    constexpr size_t smem = sizeof(Sh) + 128;
    static_assert((smem + 1024) * wide8_occupancy(D) <= 228 * 1024 && Sh::kCols * wide8_occupancy(D) <= 512 && sizeof(typename Sh::Queries) == query_bytes8(D, kWideRows8) && Sh::kUsed <= 512, "");
    static std::atomic<int> allowed[64];
    cudaError_t e = launch_queries8<D>(a, s);
    if (e != cudaSuccess) return e;
    e = allow_shared(kv8_wide_kernel<D>, int(smem), allowed);
    if (e != cudaSuccess) return e;
    e = launch_after(kv8_wide_kernel<D>, unsigned(grid), unsigned(wide8_threads(D)), smem, s, a);
    if (e != cudaSuccess) return e;
    return launch_join<D>(a, grid, kWideRows8, s);
}

template <int D>
cudaError_t launch_wide8_of(const Att8Args &a, int grid, cudaStream_t s);

}  // namespace sv
