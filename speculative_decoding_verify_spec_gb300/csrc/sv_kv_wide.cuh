// sv_kv_wide.cuh -- the attention over the 4-bit paged cache for many query rows a kv head (token trees, long
// drafts): 128 rows a tile on the fifth-generation tensor cores.
//
// The sums are those of sv_kv_attention.cuh, and so are the list of units (64 tokens of a sequence, kv head and row
// tile), its equal shares and the join of split segments.  Here a unit's codes are unpacked once for 128 rows, into
// shared memory in the operand layout (K-major, 128-byte swizzle), and both products run from there with their sums in
// tensor memory:
//   S [128 rows x 64 tokens]   = Q [128 x D] (code - 8)^T            one thread issues, D / 16 steps
//   O [128 rows x D] += W [128 x 64] (code' - 8)                     W: the weights p s', fp16
// Eight warps unpack and take the scores: a warp reads 32 rows of tensor memory, a thread one row's 32 tokens, so a
// row's maximum and sums need no shuffles.  A ninth warp copies units into the ring.  Within a unit the value codes
// are unpacked while S is computed, and the next unit's key codes while O is.
//
// Measured: 64 x 64 tree nodes with 4 query heads a kv head over up to 2047 tokens 123 us (255 in tiles of 32 rows); a unit
// takes a block 2.0 us at 64 dimensions, two blocks an SM, and 1.7 at 128 and 2.5 at 256, one block an SM, whatever its rows:
// the chain of unpacking, product, scores, weights, product and its two barriers.
//
// Why: with eight rows a tile column, 256 rows unpack every code eight times and spend most of their instructions
// around the products; here what is left a row and token is the exponential and a few more instructions.
#pragma once

#include "sv_kv_attention.cuh"

namespace sv {

constexpr int kWideRows = 128, kWideTokens = 64, kWideThreads = 288, kWideStages = 3;
// CTAs per SM.  64 x 64 tree nodes as above, us: 128 dimensions 241 with one and 260 with two (one sequence: 25 and 41), 64
// dimensions 159 and 124 (20 and 29).  One leaves a thread 164 registers instead of 96 and halves the split segments; the
// unpacking of 128 dimensions is long enough to fill the waits by itself.
__host__ __device__ constexpr int wide_occupancy(int D) { return D == 64 ? 2 : 1; }
__host__ __device__ constexpr int wide_columns(int D) { return D == 64 ? 128 : D == 128 ? 256 : 512; }  // of tensor memory: S, then O

template <int D, bool kExact>
struct WideShared {
    static constexpr int kStageBytes = kWideTokens * (D + 8), kPanels = D / 64;
    alignas(1024) uint8_t q[(kExact ? 2 : 1) * kPanels][kWideRows * 128];  // panels of 64 columns; then the rest's
    alignas(1024) uint8_t k[kPanels][kWideTokens * 128];
    alignas(1024) uint8_t v[D * 128];           // [dimension][64 tokens]
    alignas(1024) uint8_t w[kWideRows * 128];   // [row][64 tokens]
    alignas(128) uint8_t stage[kWideStages][kStageBytes];
    alignas(16) float key_of[kWideTokens / 2][4];    // of a token pair: scales, zeros + 8 scales
    alignas(16) float value_of[kWideTokens / 2][4];  // 1 / s', (z' + 8 s') / s'
    alignas(8) float log2_of[kWideTokens / 2][2];    // log2(s')
    float row_c[kWideRows], row_q[kWideRows];
    int row_node[kWideRows];
    float red[2][2][kWideRows];
    alignas(8) uint64_t full[kWideStages], empty[kWideStages], scores, products;
    alignas(16) Unit unit[kWideStages];
    uint32_t tmem;
};

// 16-byte chunk c of row r in a panel of 128-byte rows, swizzled.
__device__ __forceinline__ uint32_t wide_chunk(int r, int c) { return uint32_t(r * 128 + ((c ^ (r & 7)) << 4)); }
// A shared-memory operand: K-major, 128-byte swizzle, groups of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t wide_operand(uint32_t addr) {
    return uint64_t((addr & 0x3FFFF) >> 4) | uint64_t(1) << 16 | uint64_t(64) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// fp16 x fp16 into fp32, 128 rows, N columns.
__device__ __forceinline__ constexpr uint32_t wide_kind(int N) { return 1u << 4 | uint32_t(N / 8) << 17 | uint32_t(kWideRows / 16) << 24; }
__device__ __forceinline__ void wide_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"(uint32_t(add))
        : "memory");
}
__device__ __forceinline__ void wide_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_operands() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 columns of this warp's 32 rows (a lane a row).
__device__ __forceinline__ void tmem_load16(float (&x)[16], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]),
          "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
        : "r"(addr)
        : "memory");
}
// 32 columns of this warp's 32 rows (a lane a row).
__device__ __forceinline__ void tmem_load32(float (&x)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]),
          "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]), "=f"(x[18]),
          "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]), "=f"(x[25]), "=f"(x[26]), "=f"(x[27]),
          "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_store32(const float (&x)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};\n\ttcgen05.wait::st.sync.aligned;" ::"f"(x[0]),
        "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "f"(x[8]), "f"(x[9]), "f"(x[10]), "f"(x[11]),
        "f"(x[12]), "f"(x[13]), "f"(x[14]), "f"(x[15]), "f"(x[16]), "f"(x[17]), "f"(x[18]), "f"(x[19]), "f"(x[20]), "f"(x[21]),
        "f"(x[22]), "f"(x[23]), "f"(x[24]), "f"(x[25]), "f"(x[26]), "f"(x[27]), "f"(x[28]), "f"(x[29]), "f"(x[30]), "f"(x[31]),
        "r"(addr)
        : "memory");
}

// The queries of a segment, as load_queries, into the operand panels.  256 threads, eight dimensions a thread.
template <int D, bool kExact>
__device__ __forceinline__ void wide_queries(const AttArgs &a, WideShared<D, kExact> &sh, const Unit &un, int tid) {
    constexpr int L = D / 8, P = 256 / L;
    const int c = tid % L, d0 = c * 8;
#pragma unroll 2
    for (int r0 = 0; r0 < kWideRows; r0 += P) {
        const int r = r0 + tid / L, row = un.rt * kWideRows + r;
        const int node = row / a.G, head = un.h * a.G + row - node * a.G;
        const bool on = node < un.fresh;
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
        float sum = 0.f, rest[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = a.scale < 0.f ? -x[i] : (a.scale == 0.f ? 0.f : x[i]);
            const float y = v * shrink, f = __half2float(__float2half_rn(y));
            x[i] = f, rest[i] = y - f;
            sum += kExact ? y : f;
        }
#pragma unroll
        for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        // in the order in which a word of codes unpacks, the odd ones scaled by 1 / 16
        auto chunk = [](const float (&v)[8]) {
            uint32_t w[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float f = n & 1 ? 0.0625f : 1.f;
                const __half2 h = __floats2half2_rn(v[n] * f, v[n + 4] * f);
                w[n] = *reinterpret_cast<const uint32_t *>(&h);
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        const uint32_t at = wide_chunk(r, c % 8);
        *reinterpret_cast<uint4 *>(sh.q[c / 8] + at) = chunk(x);
        if constexpr (kExact) *reinterpret_cast<uint4 *>(sh.q[D / 64 + c / 8] + at) = chunk(rest);
        if (c == 0) {
            sh.row_c[r] = a.scale == 0.f ? 1.f : fmaxf(fabsf(a.scale) * 1.4426950408889634f * power2(e2), 1.2e-38f);
            sh.row_q[r] = sum;
            sh.row_node[r] = on ? node : -1;
        }
    }
}

template <int D, bool kExact>
__global__ void __launch_bounds__(kWideThreads, wide_occupancy(D)) kv_wide_kernel(const AttArgs a) {
    using Sh = WideShared<D, kExact>;
    constexpr int R = kWideRows, NT = kWideTokens, NW = 8, C = 32 * NW, kStages = kWideStages;
    extern __shared__ unsigned char raw0[];
    unsigned char *raw = raw0 + ((1024 - (smem_u32(raw0) & 1023)) & 1023);
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    int *parent_s = reinterpret_cast<int *>(raw + sizeof(Sh));
    const int anc_words = (a.T + 31) / 32 + 1;  // a word past the end, for windows that reach over it
    uint32_t *anc_s = reinterpret_cast<uint32_t *>(parent_s + (a.parent ? a.T : 0));  // [R][anc_words]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncta = int(gridDim.x), cta = int(blockIdx.x);

    griddep_launch_next();
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&sh.full[i]), 1), mbar_init(smem_u32(&sh.empty[i]), NW);
        mbar_init(smem_u32(&sh.scores), 1), mbar_init(smem_u32(&sh.products), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    griddep_wait();
    if (cta == 0 && tid == 0) *a.status = SV_OK;
    if (a.parent)
        for (int i = tid; i < a.T; i += kWideThreads) parent_s[i] = a.parent[i];
    Cursor<NT> cur;
    int total, ubegin, uend;
    if (!find_share<NT>(a, R, lane, cta, ncta, cur, total, ubegin, uend)) {
        if (tid == 0) a.desc[cta] = AttDesc{0, 0, 0, 0, 0, 0, 0, 0};
        return;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"(wide_columns(D))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        fence_before();
    }
    __syncthreads();
    fence_after();

    if (warp == NW) {
        copy_units<D, NT, kStages>(a, sh, cur, ubegin, uend, R, lane);
    } else {
        const uint32_t tmem = sh.tmem, tmem_s = tmem + (uint32_t(warp % 4 * 32) << 16), tmem_o = tmem_s + NT;
        const int r = warp % 4 * 32 + lane, half = warp / 4;  // this thread's row, and which 32 of a unit's tokens
        bool waits = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (waits && !mbar_wait(smem_u32(bar), parity)) {
                waits = false;  // reported; no further waits
                atomicExch(a.status, int(SV_ERR_TIMEOUT));
            }
            __syncwarp();  // (lanes may leave the wait at different times, and loads from tensor memory follow)
        };
        int stage = 0;
        uint32_t phase = 0, turn = 0;  // turn: parity of this unit's products
        const int units = uend - ubegin;
        Unit seg{cur.b, cur.h, cur.rt, cur.tile, cur.tiles(), cur.w.before, cur.w.len, cur.live ? cur.w.fresh : 0, 0, 0, {0, 0}};
        for (int it = 0;;) {  // segments
            const int last = min(units, it + seg.tiles - seg.tile), first = it;
            if (consumers_or<C>(!waits)) break;  // a wait gave up, some thread's at least: `seg` may not be there
            wide_queries<D, kExact>(a, sh, seg, tid);
            if (a.parent && tid < R) {
                uint32_t *anc = anc_s + tid * anc_words;
                for (int i = 0; i < anc_words; ++i) anc[i] = 0;
                const int node = (seg.rt * R + tid) / a.G;
                for (int v = node < seg.fresh ? node : -1; v >= 0;) {
                    anc[v >> 5] |= 1u << (v & 31);
                    const int up = parent_s[v];
                    v = up < v ? up : -1;
                }
            }
            consumers_sync<C>();
            const float c2 = sh.row_c[r], qsum = sh.row_q[r];
            const int node = sh.row_node[r];
            const bool warp_on = __any_sync(0xFFFFFFFFu, node >= 0);  // rows past the last one: nothing to score
            const Two qs = two(qsum, qsum), cc = two(c2, c2);
            Two l = 0, z = 0;
            float m = 0.f, thr = -INFINITY;  // m, 0 until a score was seen, and what moves it
            const int seg_lo = ubegin + it - seg.tile;
            const bool whole = it >= seg.tile && it + seg.tiles - seg.tile <= units;

            for (; it < last; ++it) {
                wait(&sh.full[stage], phase);
                const Unit &un = sh.unit[stage];
                const uint8_t *kc = sh.stage[stage], *vc = kc + NT * (D / 2);
                const uint32_t *km = reinterpret_cast<const uint32_t *>(kc + NT * D), *vm = km + NT;
                const bool masked = un.masked != 0;
                const int tok0 = un.tile * NT;
                auto loaded = [&](int col) { return tok0 + col < un.len && (un.have >> (4 * (col / a.granule)) & 1u); };
                // key codes: a thread takes a quarter of a token's words
                {
                    const int t = tid >> 2, w0 = (tid & 3) * (D / 32);
                    uint32_t kw[D / 32];
                    if constexpr (D == 64) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(kc + t * (D / 2) + w0 * 4);
                        kw[0] = x.x, kw[1] = x.y;
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 32; i += 4) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(kc + t * (D / 2) + (w0 + i) * 4);
                            kw[i] = x.x, kw[i + 1] = x.y, kw[i + 2] = x.z, kw[i + 3] = x.w;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint32_t x = kw[i], y = x >> 8;
                        *reinterpret_cast<uint4 *>(sh.k[(w0 + i) / 8] + wide_chunk(t, (w0 + i) % 8)) =
                            make_uint4(codes_even(x), codes_odd(x), codes_even(y), codes_odd(y));
                    }
                }
                if (tid < NT) {  // scales and zeros; of tokens that are not there, nothing
                    const float2 kf = __half22float2(*reinterpret_cast<const __half2 *>(km + tid));
                    float ks = kf.x, kz = fmaf(8.f, kf.x, kf.y);
                    ValueScale v = value_scale(vm[tid]);
                    // a NaN value reaches the rows that see it by their score
                    if ((masked && !loaded(tid)) || !v.finite) v.log2 = v.inverse = v.shift = 0.f, ks = NAN;
                    sh.key_of[tid / 2][tid & 1] = ks, sh.key_of[tid / 2][2 + (tid & 1)] = kz;
                    sh.value_of[tid / 2][tid & 1] = v.inverse, sh.value_of[tid / 2][2 + (tid & 1)] = v.shift;
                    sh.log2_of[tid / 2][tid & 1] = v.log2;
                }
                fence_operands();
                fence_before();
                consumers_sync<C>();
                if (tid == 0) {
                    fence_after();
#pragma unroll
                    for (int s = 0; s < (kExact ? 2 : 1) * D / 16; ++s) {
                        const int panel = s / 4, step = s % 4 * 32;  // bytes along a 128-byte row
                        wide_mma(tmem, wide_operand(smem_u32(sh.q[panel]) + step), wide_operand(smem_u32(sh.k[panel % (D / 64)]) + step),
                                 wide_kind(NT), s > 0);
                    }
                    wide_commit(&sh.scores);
                }
                // value codes, once the last unit's product has been read: (chunk of 8 tokens, group of 4 dimensions)
                if (it > first) wait(&sh.products, turn ^ 1);
#pragma unroll
                for (int at = tid; at < 2 * D; at += C) {
                    const int c = at & 7, group = at >> 3;  // tokens 8 c .. ; dimensions 4 group ..
                    const uint4 *src = reinterpret_cast<const uint4 *>(vc + c / 2 * 8 * D + group / 8 * 256 + group % 8 * 32);
                    const uint4 x = src[0], y = src[1];
                    const bool j = c & 1;
                    const uint32_t w[4] = {j ? x.y : x.x, j ? x.w : x.z, j ? y.y : y.x, j ? y.w : y.z};  // token pairs
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t s = i < 2 ? w[t] : w[t] >> 8;
                            h[t] = i & 1 ? codes_odd(s) : codes_even(s);
                        }
                        *reinterpret_cast<uint4 *>(sh.v + wide_chunk(4 * group + i, c)) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
                // which of this thread's tokens its row sees
                uint32_t see = node >= 0 ? 0xFFFFFFFFu : 0u;
                if (masked) {
                    const int x = tok0 + half * 32 - un.before;  // the first one among the new tokens
                    if (x > -32 && node >= 0) {
                        uint32_t fresh;
                        if (a.parent) {
                            const uint32_t *anc = anc_s + r * anc_words;
                            if (x >= 0) {
                                const int w = x >> 5, words = anc_words - 1;
                                fresh = w < words ? __funnelshift_r(anc[w], anc[w + 1], x & 31) : 0u;
                            } else {
                                fresh = anc[0] << -x | ((1u << -x) - 1);
                            }
                        } else {
                            const int count = node + 1 - x;
                            fresh = count >= 32 ? 0xFFFFFFFFu : count <= 0 ? 0u : (1u << count) - 1;
                        }
                        see = fresh;
                    }
                    uint32_t there = 0;
                    for (int j = 0; j < 32; j += 16) {  // (granules are 16 tokens at least)
                        const int col = half * 32 + j, left = un.len - (tok0 + col);
                        if (loaded(col)) there |= (left >= 16 ? 0xFFFFu : (1u << left) - 1) << j;
                    }
                    see &= there;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.empty[stage]));  // (nothing more of the stage, or `un`, is read)
                wait(&sh.scores, turn);
                fence_after();
                bool weighed = it > first;  // a segment's first unit moves m: no use in weights before
                bool need = !weighed, again = false;
                Two dl = 0, dz = 0;
                while (true) {
                    if (warp_on) {
                        const Two minus = two(-m, -m);
                        float most = -INFINITY;
                        dl = 0, dz = 0;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {  // 16 tokens at a time
                            float s[16];
                            tmem_load16(s, tmem_s + half * 32 + 16 * c);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 k = *reinterpret_cast<const float4 *>(sh.key_of[half * 16 + 8 * c + j]);
                                const float2 v = *reinterpret_cast<const float2 *>(sh.log2_of[half * 16 + 8 * c + j]);
                                const Two y = fma2(two(s[2 * j], s[2 * j + 1]), two(k.x, k.y), mul2(qs, two(k.z, k.w)));
                                const float2 x = split(fma2(y, cc, two(v.x, v.y)));
                                s[2 * j] = x.x, s[2 * j + 1] = x.y;
                            }
                            if (masked) {
                                __syncwarp();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    if (!(see >> (16 * c + j) & 1u)) s[j] = -INFINITY;
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) most = fmaxf(most, s[j]);
                            if (weighed) {
#pragma unroll
                                for (int d = 0; d < 2; ++d) {
                                    uint32_t w[4];
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const int j = 4 * d + i;
                                        const float4 v = *reinterpret_cast<const float4 *>(sh.value_of[half * 16 + 8 * c + j]);
                                        const float2 x = split(add2(two(s[2 * j], s[2 * j + 1]), minus));
                                        const float p0 = ex2(x.x), p1 = ex2(x.y);
                                        dl = fma2(two(p0, p1), two(v.x, v.y), dl);
                                        dz = fma2(two(p0, p1), two(v.z, v.w), dz);
                                        const __half2 h = __floats2half2_rn(p0, p1);
                                        w[i] = *reinterpret_cast<const uint32_t *>(&h);
                                    }
                                    *reinterpret_cast<uint4 *>(sh.w + wide_chunk(r, half * 4 + 2 * c + d)) = make_uint4(w[0], w[1], w[2], w[3]);
                                }
                            }
                        }
                        sh.red[0][half][r] = most;
                        need |= !again && most > thr;  // (a second pass is the last one, whatever the scores are)
                    }
                    fence_operands();
                    fence_before();
                    if (!consumers_or<C>(need)) break;
                    // some row's m moves (the first unit's always does): again
                    if (warp_on) {
                        const float y = fmaxf(sh.red[0][0][r], sh.red[0][1][r]);
                        const float seen = thr == -INFINITY ? -INFINITY : m, mn = fmaxf(seen, y - kTop);
                        const float al = seen == -INFINITY ? 0.f : ex2(seen - mn);
                        if (mn != -INFINITY) m = mn, thr = mn + kMost;
                        l = mul2(l, two(al, al)), z = mul2(z, two(al, al));
                        if (it > first) {  // (the last unit's product is done: its codes' place has been taken)
                            fence_after();
#pragma unroll 1
                            for (int col = half * (D / 2); col < (half + 1) * (D / 2); col += 32) {
                                float o[32];
                                tmem_load32(o, tmem_o + col);
#pragma unroll
                                for (int j = 0; j < 32; ++j) o[j] *= al;
                                tmem_store32(o, tmem_o + col);
                            }
                        }
                    }
                    need = false, weighed = again = true;
                    consumers_sync<C>();  // (the maxima are read)
                }
                if (warp_on) l = add2(l, dl), z = add2(z, dz);
                if (tid == 0) {
                    fence_after();
#pragma unroll
                    for (int kk = 0; kk < NT / 16; ++kk)
                        wide_mma(tmem + NT, wide_operand(smem_u32(sh.w) + kk * 32), wide_operand(smem_u32(sh.v) + kk * 32), wide_kind(D),
                                 it > first || kk > 0);
                    wide_commit(&sh.products);
                }
                turn ^= 1;
                if (++stage == kStages) stage = 0, phase ^= 1;
            }

            // the rows' sums over both halves, then the output
            const float2 l2 = split(l), z2 = split(z);
            consumers_sync<C>();
            sh.red[0][half][r] = l2.x + l2.y, sh.red[1][half][r] = z2.x + z2.y;
            consumers_sync<C>();
            wait(&sh.products, turn ^ 1);
            fence_after();
            const float sl = sh.red[0][0][r] + sh.red[0][1][r], sz = sh.red[1][0][r] + sh.red[1][1][r];
            const int row = seg.rt * R + r, at = row / a.G;
            const int64_t slot = 2 * cta + (seg_lo > ubegin ? 1 : 0);
            const float inv = node < 0 || sl == 0.f ? 0.f : 1.f / sl;
            uint16_t *out = a.out + ((seg.b * int64_t(a.T) + at) * a.H * a.G + seg.h * a.G + row % a.G) * D;
#pragma unroll 1
            for (int col = half * (D / 2); col < (half + 1) * (D / 2); col += 32) {
                float o[32];
                tmem_load32(o, tmem_o + col);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = warp_on ? fmaf(o[j], j & 1 ? 0.0625f : 1.f, sz) : 0.f;
                if (whole) {
                    if (at < a.T) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float x = inv == 0.f ? 0.f : o[j + 2 * i] * inv, y = inv == 0.f ? 0.f : o[j + 2 * i + 1] * inv;
                                w[i] = uint32_t(kv_from_float(x, a.bf16)) | uint32_t(kv_from_float(y, a.bf16)) << 16;
                            }
                            *reinterpret_cast<uint4 *>(out + col + j) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                } else if (SV_IN(slot, 2 * ncta)) {
                    float4 *dst = reinterpret_cast<float4 *>(a.acc + (slot * R + r) * D + col);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    if (col == 0) a.ml[slot * R + r] = make_float2(thr == -INFINITY ? -INFINITY : m, sl);
                }
            }
            fence_before();
            if (tid == 0 && seg_lo <= ubegin)  // the share's first segment
                a.desc[cta] = describe(total, cta, ncta, ubegin, seg_lo, seg_lo + seg.tiles, seg.b, seg.h, seg.rt, seg.fresh);
            if (it == units) break;
            wait(&sh.full[stage], phase);
            seg = sh.unit[stage];
        }
        // where a wait gave up, products may still be under way: the last chance that they get before their operands' place goes
        if (tid == 0 && !waits) mbar_wait(smem_u32(&sh.scores), turn ^ 1), mbar_wait(smem_u32(&sh.products), turn ^ 1);
    }
    __syncthreads();
    fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(wide_columns(D)));
}

template <int D, bool kExact>
cudaError_t launch_wide(const AttArgs &a, int grid, cudaStream_t s) {
    constexpr size_t fixed = sizeof(WideShared<D, kExact>) + 1024;
    static_assert(fixed + SV_MAX_TREE_NODES * 4 + kWideRows * (SV_MAX_TREE_NODES / 32 + 1) * 4 <= 227 * 1024, "the largest tree");
    const size_t smem = fixed + (a.parent ? size_t(a.T) * 4 + size_t(kWideRows) * ((a.T + 31) / 32 + 1) * 4 : 0);
    static std::atomic<int> allowed[64];
    cudaError_t e = allow_shared(kv_wide_kernel<D, kExact>, int(smem), allowed);
    if (e != cudaSuccess) return e;
    e = launch_after(kv_wide_kernel<D, kExact>, unsigned(grid), unsigned(kWideThreads), smem, s, a);
    if (e != cudaSuccess) return e;
    return launch_join<D>(a, grid, kWideRows, s);
}

}  // namespace sv
