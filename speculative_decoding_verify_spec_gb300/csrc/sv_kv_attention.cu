// sv_kv_attention.cu -- the new tokens' attention over the 4-bit paged cache.
//
// For a query row q (one of the T x G rows that share a kv head) and cached tokens j with key
// k_j = z_j + s_j code_j and value likewise,
//   x_j = scale (s_j (q . (code_j - 8)) + (z_j + 8 s_j) sum(q)),  p_j = exp(x_j - m),
//   out = [ sum_j (p_j s'_j) (code'_j - 8) + sum_j p_j (z'_j + 8 s'_j) ] / sum_j p_j,
// so the matrix products run on the bare codes (exact in fp16) and each token's scale and zero
// cost a multiply-add per score instead of one per dimension.
//
// Work: a unit is 32 to 128 tokens for one (sequence, kv head, tile of 16 MT rows).  All units of the
// batch form one list; each CTA takes an equal, contiguous share of it, so ragged lengths balance
// by themselves and a long context spreads over the card.  A segment (one sequence, head, row
// tile) that ends up whole in a CTA is written out there; the others leave partial results
// that combine_kernel joins.
//
// A CTA has D / 32 consumer warps, and one that copies units into a ring in shared memory.  Each
// consumer scores its part of a unit's tokens for all rows, the weights go through shared
// memory, and each warp accumulates its own 32 dimensions over all the tokens: a
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

constexpr int kStages = 3;              // units in flight per CTA
constexpr float kLazy = 8.f;            // log2 of how far a weight may pass 1
constexpr uint64_t kCopyLimitNs = 1000000000ull;
constexpr int kAttSMs = 152;

// Tokens per unit: as many as the registers for their scores allow.
constexpr int att_tokens(int D, int MT) { return MT >= 3 ? (D == 64 ? 32 : 64) : D == 64 ? 64 : 128; }
constexpr int att_occupancy(int D, int MT) {  // CTAs per SM: by registers and shared memory
    return D == 64 ? (MT == 1 ? 6 : MT == 2 ? 5 : 4) : D == 128 ? (MT == 1 ? 3 : 2) : 1;
}
// Tiles of at most 64 rows, as few as there have to be and no larger than they need be.
inline int att_mt(int64_t rows) {
    const int64_t tiles = (rows + 63) / 64;
    return int(((rows + tiles - 1) / tiles + 15) / 16);
}

struct AttArgs {
    const uint16_t *q;
    int64_t q_bs, q_ts, q_hs;
    int bf16, vec;  // vec: query rows lie on the 16-byte grid
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
    float2 *ml;            // [2 grid][R] running maximum (log2) and sum
    float *acc;            // [2 grid][R][D]
};

// The first segment of a CTA's share, for the joining kernel.
struct AttDesc {
    int lo, hi, total;  // the segment's units, and all units
    int b, h, rt, fresh;
};

// Where a CTA's share begins.
__device__ __forceinline__ int share_begin(int total, int c, int n) { return int(int64_t(c) * total / n); }
__device__ __forceinline__ int share_owner(int total, int u, int n) { return int((int64_t(u + 1) * n - 1) / total); }

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
struct Unit {
    int b, h, rt, tile, tiles;
    int before, len, fresh;   // tokens before the step; all; new ones (0: no live row)
    uint32_t have;            // bit 4 g: granule g was loaded
    int masked;               // not every token is seen by every row
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
// The codes in half-bytes 0 and 4 of w, less 8, as fp16 (1024 + code has its code in the low bits), and
// 16 times those in half-bytes 1 and 5: all exact.  (The factor is in the queries, or taken out of the
// output.)  Centred, so that sums over thousands of tokens do not cancel against the zeros' part.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
    uint32_t r = (w & 0x000F000Fu) | 0x64006400u;
    asm("sub.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x64086408u));
    return r;
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
    uint32_t r = (w & 0x00F000F0u) | 0x64006400u;
    asm("sub.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x64806480u));
    return r;
}

template <int D, int MT>
struct AttShared {
    static constexpr int R = 16 * MT, NW = D / 32, NT = att_tokens(D, MT);
    static constexpr int kStageBytes = NT * (D + 8);
    static constexpr int kQStride = D + 8, kPStride = NT + 8;  // halves; 16 bytes past a multiple of 64: no bank conflicts
    alignas(128) uint8_t stage[kStages][kStageBytes];
    alignas(16) __half q[R * kQStride];
    alignas(16) __half p[2][R * kPStride];
    float row_c[R], row_qs[R];  // log2 scale of a row's scores; the sum of its queries
    float red[2][NW][R];
    int row_node[R];  // the row's new token, -1: no live row
    alignas(8) uint64_t full[kStages], empty[kStages];
    Unit unit[kStages];
};

__device__ __forceinline__ float power2(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127
// Barriers of the D consumer threads.
template <int N>
__device__ __forceinline__ void consumers_sync() {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ bool consumers_or(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(x)), "n"(N)
        : "memory");
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

// The queries of a segment's rows into shared memory: rotated, scaled by a power of two into fp16's
// range (exact for 16-bit inputs but for values 2^-25 of the row's largest; a rotated value is
// rounded to 11 bits), columns in the order in which the codes unpack.  D consumer threads, eight
// rows at a time, eight dimensions a thread.
template <int D, int MT>
__device__ __forceinline__ void load_queries(const AttArgs &a, AttShared<D, MT> &sh, const Unit &un, int tid) {
    using Sh = AttShared<D, MT>;
    constexpr int R = Sh::R, L = D / 8;  // lanes of a row
    const int c = tid % L, d0 = c * 8;
#pragma unroll 2
    for (int r0 = 0; r0 < R; r0 += 8) {
        const int r = r0 + tid / L;
        const int row = un.rt * R + r;
        const int node = row / a.G, head = un.h * a.G + row % a.G;
        const bool on = node < un.fresh;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (on) {
            const uint16_t *qp = a.q + un.b * a.q_bs + node * a.q_ts + head * a.q_hs;
            load8(qp + d0, a.vec, a.bf16, x);
            if (a.rot.cos && d0 < 2 * a.rot.pairs) {
                const int64_t arow = kv_rotation_row(a.rot, int64_t(un.b) * a.T + node, un.before + node);
                const float *cp = a.rot.cos + arow, *sp = a.rot.sin + arow;
                float y[8], cs[8], sn[8];
                if (!a.rot.interleaved && a.rot.pairs % 8 == 0) {  // the chunk lies within one half
                    const int e0 = d0 < a.rot.pairs ? d0 : d0 - a.rot.pairs;
                    load8(qp + (d0 < a.rot.pairs ? d0 + a.rot.pairs : e0), a.vec, a.bf16, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        cs[i] = __ldg(cp + e0 + i);
                        sn[i] = d0 < a.rot.pairs ? -__ldg(sp + e0 + i) : __ldg(sp + e0 + i);
                    }
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
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(fabsf(x[i])));
#pragma unroll
        for (int o = L / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const int e2 = top == 0 ? 0 : int(top >> 23) - 127 - 10;  // the largest becomes 2^10 .. 2^11
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = a.scale < 0.f ? -x[i] : (a.scale == 0.f ? 0.f : x[i]);
            x[i] = __half2float(__float2half_rn(ldexpf(v, -e2)));
            sum += x[i];
        }
        // dimension 8 w + n of quad's quarter: k-step 2 w + (n % 4) / 2, the odd n scaled by 1 / 16
        __half *dst = &sh.q[r * Sh::kQStride + 2 * (d0 / (D / 4)) + 2 * (d0 % (D / 4) / 8) * 16];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float f = n & 1 ? 0.0625f : 1.f;
            *reinterpret_cast<__half2 *>(dst + (n >> 1) * 16 + (n & 1) * 8) = __floats2half2_rn(x[n] * f, x[n + 4] * f);
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (c == 0) {
            sh.row_c[r] = a.scale == 0.f ? 1.f : ldexpf(fabsf(a.scale) * 1.4426950408889634f, e2);
            sh.row_qs[r] = sum;
            sh.row_node[r] = on ? node : -1;
        }
    }
}

template <int D, int MT>
__global__ void __launch_bounds__(D + 32, att_occupancy(D, MT)) kv_attention_kernel(const AttArgs a) {
    using Sh = AttShared<D, MT>;
    constexpr int R = Sh::R, NW = Sh::NW, NT = Sh::NT, TW = NT / NW, NJ = TW / 8, KS = D / 16, E = D / 32;
    constexpr int kThreads = D + 32;
    constexpr bool kQRegs = MT == 1 && D == 64;
    static_assert(NJ >= 1 && NJ <= 8 && NT <= 128 && NT % 32 == 0, "");
    extern __shared__ __align__(128) unsigned char raw[];
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    int *parent_s = reinterpret_cast<int *>(raw + sizeof(Sh));
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

    // all units, then the sequence where this CTA's share begins (every warp for itself)
    int total = 0;
    for (int b = lane; b < a.B; b += 32) total += seq_work<NT>(a, b, R).units;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    const int ubegin = share_begin(total, cta, ncta), uend = share_begin(total, cta + 1, ncta);
    if (ubegin >= uend) return;
    Cursor<NT> cur;
    {
        int run = 0;
        for (int b0 = 0;; b0 += 32) {  // (ubegin < total: some sequence holds it)
            const int b = b0 + lane;
            const int u = b < a.B ? seq_work<NT>(a, b, R).units : 0;
            int inc = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += v;
            }
            const int lo = run + inc - u;
            const uint32_t hit = __ballot_sync(0xFFFFFFFFu, ubegin >= lo && ubegin < lo + u);
            if (hit) {
                const int l = __ffs(hit) - 1;
                cur.b = b0 + l;
                cur.base = __shfl_sync(0xFFFFFFFFu, lo, l);
                break;
            }
            run += __shfl_sync(0xFFFFFFFFu, inc, 31);
            if (b0 + 32 >= a.B) return;  // never
        }
    }
    cur.w = seq_work<NT>(a, cur.b, R);
    cur.place(a, ubegin);
    __syncthreads();

    if (warp == NW) {
        // the copies, up to kStages units ahead of the consumers
        const int64_t page_bytes = kv_page_bytes(a.page, D);
        const int gi = lane >> 2, piece = lane & 3;
        const uint32_t all_granules = NT / a.granule == 8 ? 0x11111111u : 0x11111111u & ((1u << (4 * (NT / a.granule))) - 1);
        for (int u = ubegin; u < uend; ++u) {
            const int it = u - ubegin, stage = it % kStages;
            const int tok = cur.tile * NT + gi * a.granule;
            const uint8_t *src = nullptr;
            int slot = 0;
            if (gi * a.granule < NT && cur.live && tok < cur.w.len) {
                const int pi = tok / a.page, pg = __ldg(a.table + int64_t(cur.b) * a.width + pi);
                slot = tok - pi * a.page;
                if (pg >= 0 && pg < a.num_pages && SV_IN(slot + a.granule - 1, a.page))
                    src = a.cache + (int64_t(pg) * a.H + cur.h) * page_bytes;
            }
            const uint32_t bytes = src == nullptr ? 0 : piece < 2 ? a.granule * (D / 2) : a.granule * 4;
            const uint32_t sum = __reduce_add_sync(0xFFFFFFFFu, bytes);
            const uint32_t have = __ballot_sync(0xFFFFFFFFu, src != nullptr && piece == 0);
            if (it >= kStages && !mbar_wait(smem_u32(&sh.empty[stage]), uint32_t(it / kStages - 1) & 1)) {
                atomicExch(a.status, int(SV_ERR_TIMEOUT));
                return;  // (the consumers' waits give up too)
            }
            const uint32_t bar = smem_u32(&sh.full[stage]);
            if (lane == 0) {
                sh.unit[stage] = Unit{cur.b, cur.h, cur.rt, cur.tile, cur.tiles(), cur.w.before, cur.w.len, cur.live ? cur.w.fresh : 0, have,
                                      int((cur.tile + 1) * NT > cur.w.before || have != all_granules)};
                mbar_expect(bar, sum);
            }
            __syncwarp();
            if (src) {
                const uint32_t dst = smem_u32(sh.stage[stage]);
                if (piece < 2)
                    bulk_load(dst + (piece * NT + gi * a.granule) * (D / 2), src + (piece * a.page + slot) * (D / 2), bytes, bar);
                else
                    bulk_load(dst + NT * D + ((piece - 2) * NT + gi * a.granule) * 4,
                              src + a.page * D + ((piece - 2) * a.page + slot) * 4, bytes, bar);
            }
            if (u + 1 < uend) cur.next(a, R, u + 1);
        }
        return;
    }

    uint32_t qf[kQRegs ? KS : 1][4];
    float acc[MT][4][4];
    float m[MT][2], thr[MT][2], l[MT][2], z[MT][2];  // m: running maximum in log2, 0 until a score was seen
    int kexp = 1;  // values' scales are divided by 2^(kexp - 14): all are below 1 then
    bool fresh_segment = true, waits = true;

    int stage = 0;
    uint32_t phase = 0;
    const int units = uend - ubegin;
    for (int it = 0; it < units; ++it) {
        const int buf = it & 1;
        if (waits && !mbar_wait(smem_u32(&sh.full[stage]), phase)) {
            waits = false;  // reported; no further waits
            atomicExch(a.status, int(SV_ERR_TIMEOUT));
        }
        const Unit &un = sh.unit[stage];
        if (fresh_segment) {
            consumers_sync<D>();
            load_queries<D, MT>(a, sh, un, tid);
            if (a.parent)
                for (int r = tid; r < R; r += D) {
                    uint32_t *anc = anc_s + r * anc_words;
                    for (int i = 0; i < anc_words; ++i) anc[i] = 0;
                    const int node = (un.rt * R + r) / a.G;
                    for (int v = node < un.fresh ? node : -1; v >= 0;) {
                        anc[v >> 5] |= 1u << (v & 31);
                        const int up = parent_s[v];
                        v = up < v ? up : -1;
                    }
                }
            consumers_sync<D>();
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
                for (int k = 0; k < 2; ++k) m[i][k] = 0.f, thr[i][k] = -INFINITY, l[i][k] = z[i][k] = 0.f;
            }
            kexp = 1;
            fresh_segment = false;
        }

        const uint8_t *kc = sh.stage[stage], *vc = kc + NT * (D / 2);
        const uint32_t *km = reinterpret_cast<const uint32_t *>(kc + NT * D), *vm = km + NT;
        const bool masked = un.masked != 0;
        const int tok0 = un.tile * NT;  // (fits: a table spans less than 2^31 tokens)
        auto loaded = [&](int col) { return tok0 + col < un.len && (un.have >> (4 * (col / a.granule)) & 1u); };

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

        // y = s_j (q . (code_j - 8)) + (z_j + 8 s_j) sum(q); masked scores are -inf
        float vs[NJ][2], vz[NJ][2], ym[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i) ym[i][0] = ym[i][1] = -INFINITY;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int col = warp * TW + j * 8 + 2 * t4;
            const uint2 kk = *reinterpret_cast<const uint2 *>(km + col), vv = *reinterpret_cast<const uint2 *>(vm + col);
            const float2 k0 = __half22float2(*reinterpret_cast<const __half2 *>(&kk.x)), k1 = __half22float2(*reinterpret_cast<const __half2 *>(&kk.y));
            const float2 v0 = __half22float2(*reinterpret_cast<const __half2 *>(&vv.x)), v1 = __half22float2(*reinterpret_cast<const __half2 *>(&vv.y));
            const float z0 = fmaf(8.f, k0.x, k0.y), z1 = fmaf(8.f, k1.x, k1.y);
            vs[j][0] = v0.x, vs[j][1] = v1.x;
            vz[j][0] = fmaf(8.f, v0.x, v0.y), vz[j][1] = fmaf(8.f, v1.x, v1.y);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float q0 = sh.row_qs[i * 16 + g], q1 = sh.row_qs[i * 16 + g + 8];
                s[i][j][0] = fmaf(s[i][j][0], k0.x, q0 * z0);
                s[i][j][1] = fmaf(s[i][j][1], k1.x, q0 * z1);
                s[i][j][2] = fmaf(s[i][j][2], k0.x, q1 * z0);
                s[i][j][3] = fmaf(s[i][j][3], k1.x, q1 * z1);
            }
        }
        // the largest scale of the unit's values (a NaN one spoils only the rows that see it)
        auto scale_bits = [&](int col) { return (vm[col] & 0xFFFFu) < 0x7C00u ? vm[col] & 0xFFFFu : 0u; };
        uint32_t top = 0;
        if (!masked) {
#pragma unroll
            for (int c = 0; c < NT; c += 32) top = max(top, scale_bits(c + lane));
        } else {
#pragma unroll 1
            for (int c = 0; c < NT; c += 32)
                if (loaded(c + lane)) top = max(top, scale_bits(c + lane));
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = i * 16 + g + (k >> 1) * 8, node = sh.row_node[r];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int col = warp * TW + j * 8 + 2 * t4 + (k & 1);
                        const int idx = tok0 + col - un.before;  // below 0: before the new tokens
                        bool v = node >= 0 && loaded(col);
                        if (v && idx >= 0 && SV_IN(idx, a.T)) v = a.parent ? anc_s[r * anc_words + (idx >> 5)] >> (idx & 31) & 1u : idx <= node;
                        if (!v) s[i][j][k] = -INFINITY;
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
        // weights: p for the sums (this warp's tokens), p s' for the product, rounded to fp16
        float dl[MT][2], dz[MT][2];
        auto weigh = [&]() {
            const float down = power2(14 - kexp);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float c0 = sh.row_c[i * 16 + g], c1 = sh.row_c[i * 16 + g + 8];
                dl[i][0] = dl[i][1] = dz[i][0] = dz[i][1] = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    float w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float p = ex2(fmaf(s[i][j][k], k < 2 ? c0 : c1, -m[i][k >> 1]));
                        const float sc = vs[j][k & 1] * down, ze = vz[j][k & 1];
                        dl[i][k >> 1] += p;
                        if (masked) {  // a masked token's own scale and zero (NaN, or not loaded) must not matter
                            const bool v = s[i][j][k] != -INFINITY;
                            dz[i][k >> 1] += v ? p * ze : 0.f;
                            w[k] = v ? p * sc : 0.f;
                        } else {
                            dz[i][k >> 1] = fmaf(p, ze, dz[i][k >> 1]);
                            w[k] = p * sc;
                        }
                    }
                    __half *dst = &sh.p[buf][(i * 16 + g) * Sh::kPStride + warp * TW + j * 8 + 2 * t4];
                    *reinterpret_cast<__half2 *>(dst) = __floats2half2_rn(w[0], w[1]);
                    *reinterpret_cast<__half2 *>(dst + 8 * Sh::kPStride) = __floats2half2_rn(w[2], w[3]);
                }
            }
        };
        weigh();
        if (consumers_or<D>(need)) {  // some row's maximum moves (the first unit's always does), or the values' exponent
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y = ym[i][k];
                    y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 1));
                    y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 2));
                    if (t4 == 0) sh.red[0][warp][i * 16 + g + 8 * k] = y;
                }
            consumers_sync<D>();
            const float kfac = power2(kexp - knew);
            kexp = knew;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = i * 16 + g + 8 * k;
                    float y = sh.red[0][0][r];
#pragma unroll
                    for (int w = 1; w < NW; ++w) y = fmaxf(y, sh.red[0][w][r]);
                    // thr is -inf until the row has seen a score
                    const float c = sh.row_c[r], seen = thr[i][k] == -INFINITY ? -INFINITY : m[i][k], mn = fmaxf(seen, y * c);
                    const float al = seen == -INFINITY ? 0.f : ex2(seen - mn);
                    if (mn != -INFINITY) m[i][k] = mn, thr[i][k] = (mn + kLazy) / c;
                    l[i][k] *= al, z[i][k] *= al;
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j][2 * k] *= al * kfac, acc[i][j][2 * k + 1] *= al * kfac;
                }
            weigh();
            consumers_sync<D>();
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) l[i][k] += dl[i][k], z[i][k] += dz[i][k];

        // this warp's 32 dimensions
#pragma unroll
        for (int kk = 0; kk < NT / 16; ++kk) {
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

        const bool seg_end = un.tile + 1 == un.tiles;
        if (seg_end || it + 1 == units) {
            // the rows' sums over lanes and warps
            consumers_sync<D>();
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x = l[i][k], y = z[i][k];
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 1), y += __shfl_xor_sync(0xFFFFFFFFu, y, 1);
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, 2), y += __shfl_xor_sync(0xFFFFFFFFu, y, 2);
                    if (t4 == 0) sh.red[0][warp][i * 16 + g + 8 * k] = x, sh.red[1][warp][i * 16 + g + 8 * k] = y;
                }
            consumers_sync<D>();
            const int seg_lo = ubegin + it - un.tile;
            const bool whole = seg_end && seg_lo >= ubegin;
            const int64_t slot = 2 * cta + (seg_lo > ubegin ? 1 : 0);
            const float up = power2(kexp - 14);
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
                        const int row = un.rt * R + r, node = row / a.G;
                        if (node < a.T) {
                            const bool zero = sh.row_node[r] < 0 || sl == 0.f;
                            const float inv = 1.f / sl;
                            uint32_t w4[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                w4[j] = uint32_t(kv_from_float(zero ? 0.f : o[2 * j] * inv, a.bf16)) |
                                        uint32_t(kv_from_float(zero ? 0.f : o[2 * j + 1] * inv, a.bf16)) << 16;
                            const int64_t head = un.h * a.G + row % a.G;
                            *reinterpret_cast<uint4 *>(a.out + ((un.b * int64_t(a.T) + node) * a.H * a.G + head) * D + d0) =
                                make_uint4(w4[0], w4[1], w4[2], w4[3]);
                        }
                    } else if (SV_IN(slot, 2 * ncta)) {
                        float4 *dst = reinterpret_cast<float4 *>(a.acc + (slot * R + r) * D + d0);
                        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                        if (warp == 0 && t4 == 0) a.ml[slot * R + r] = make_float2(thr[i][k] == -INFINITY ? -INFINITY : m[i][k], sl);
                    }
                }
            if (tid == 0 && seg_lo <= ubegin)  // the share's first segment
                a.desc[cta] = AttDesc{seg_lo, seg_lo + un.tiles, total, un.b, un.h, un.rt, un.fresh};
            fresh_segment = true;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.empty[stage]));
        if (++stage == kStages) stage = 0, phase ^= 1;
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
    const int c = int(blockIdx.x) / (R / kJoinRows) + 1;
    const int r0 = int(blockIdx.x % (R / kJoinRows)) * kJoinRows;
    if (c >= ncta) return;
    // (CTA 0's share is empty only if all are; a CTA with an empty share wrote no descriptor)
    const int total = a.desc[ncta - 1].total;  // the last share is never empty
    const int begin = share_begin(total, c, ncta);
    if (begin >= share_begin(total, c + 1, ncta)) return;
    const AttDesc d = a.desc[c];
    if (begin <= d.lo) return;
    const int c0 = share_owner(total, d.lo, ncta), c1 = share_owner(total, d.hi - 1, ncta);
    // the first non-empty share after the start's owner joins the segment
    if (share_owner(total, begin - 1, ncta) != c0) return;
    if (d.fresh <= 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // c0's part lies in its second slot unless its share begins with the segment
    auto slot_of = [&](int k) { return int64_t(2) * k + (k == c0 && share_begin(total, c0, ncta) != d.lo ? 1 : 0); };
    for (int q = warp; q < kJoinRows; q += kJoinThreads / 32) {
        const int r = r0 + q;
        float big = -INFINITY;
        for (int k = c0 + lane; k <= c1; k += 32)
            if (share_begin(total, k, ncta) < share_begin(total, k + 1, ncta)) big = fmaxf(big, a.ml[slot_of(k) * R + r].x);
        for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
        float sum = 0.f;
        for (int k = c0 + lane; k <= c1; k += 32) {
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
        const int row = d.rt * R + r, node = row / a.G;
        if (node >= a.T) continue;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (node < d.fresh) {
#pragma unroll 4
            for (int k = c0; k <= c1; ++k) {
                const float w = weight[q][k - c0];
                if (w == 0.f) continue;  // also: parts of empty shares, never written
                const float4 v = *reinterpret_cast<const float4 *>(a.acc + (slot_of(k) * R + r) * D + d4);
                o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
            }
            const float inv = inv_s[q];
            o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
        }
        const int64_t head = d.h * a.G + row % a.G;
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
    e = launch_after(kv_attention_kernel<D, MT>, unsigned(grid), unsigned(D + 32), smem, s, a);
    if (e != cudaSuccess) return e;
    return launch_after(kv_attention_join_kernel<D, MT>, unsigned((grid - 1) * (16 * MT / kJoinRows)), unsigned(kJoinThreads), 0, s, a, grid);
}

template <int D>
cudaError_t launch_attention_rows(const AttArgs &a, int mt, int grid, cudaStream_t s) {
    switch (mt) {
    case 1: return launch_attention<D, 1>(a, grid, s);
    case 2: return launch_attention<D, 2>(a, grid, s);
    case 3: return launch_attention<D, 3>(a, grid, s);
    default: return launch_attention<D, 4>(a, grid, s);
    }
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
    const int64_t row_tiles = (rows + 16 * mt - 1) / (16 * mt), tokens = int64_t(table_width) * page_size;
    const int64_t most = row_tiles * (tokens / sv::att_tokens(head_dim, mt) + 1);  // units of a sequence and head
    if (most > 0x7FFFFFFF / kv_heads || most * kv_heads > 0x7FFFFFFF / B) return SV_ERR_INVALID_ARG;
    sv::AttArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.q_bs = q_batch_stride, a.q_ts = q_token_stride, a.q_hs = q_head_stride;
    a.bf16 = dtype == SV_KV_BF16;
    a.B = B, a.T = T, a.H = kv_heads, a.G = G;
    a.cache = static_cast<const uint8_t *>(cache), a.num_pages = num_pages, a.page = page_size, a.width = table_width;
    a.granule = 16;
    while (a.granule < sv::att_tokens(head_dim, mt) && page_size % (2 * a.granule) == 0) a.granule *= 2;
    a.vec = (q_batch_stride | q_token_stride | q_head_stride) % 8 == 0 && reinterpret_cast<uintptr_t>(q) % 16 == 0;
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
    const cudaError_t e = head_dim == 64    ? sv::launch_attention_rows<64>(a, mt, L.grid, s)
                          : head_dim == 128 ? sv::launch_attention_rows<128>(a, mt, L.grid, s)
                                            : sv::launch_attention_rows<256>(a, mt, L.grid, s);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
