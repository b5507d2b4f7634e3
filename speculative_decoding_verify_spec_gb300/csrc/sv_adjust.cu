// sv_adjust.cu -- penalties, biases and grammar masks on the verified rows' logits.
//
// For token t of row i, with n its occurrences in the output part of the row's context and s
// whether the context holds it at all:
//   l := s ? (l > 0 ? l / r : l r) : l;  l -= f n + p (n > 0);  l += bias(t);  masked: -inf
// in fp32, rounded once to the logits' type.  One pass: every logit is read once and written
// once (in place: only the 16-byte groups that change are written), so DRAM bounds it.
//
// A CTA owns TV consecutive tokens of one sequence for all its rows.  Its warps take 2 KB chunks of the
// rows through a ring of buffers in shared memory, filled by asynchronous copies (and each chunk's mask
// words with it), so that loads are under way from the first moment on.  Meanwhile the CTA counts the
// history's tokens of its range (a table in shared memory, integer atomics: the order does not matter)
// and lists the tokens that the history, the drafts or the bias list touch.  A chunk that has arrived is
// adjusted in place at its listed tokens, which the lanes share out (text repeats few tokens: an
// arithmetic branch in the stream itself would leave most lanes idle most of the time), and then
// masked on its way from shared memory to the output.  The history is read once per token range from L2,
// the price of needing no second kernel and no table in DRAM.
//
// Measured: 256 x 9 rows of 128256 bf16 logits with masks, histories of up to 1500 tokens and 16 biases 251 us, 4.9 TB/s
// read and written (a copy 175 us; masks alone 182; histories alone 226: counting them is instruction-bound and overlaps the
// stream only in part); 64 x 64 tree rows of 50257 fp32 logits 303 us, 5.5 TB/s (a copy 240 us).
#include <cstdint>

#include "spec_serve.h"
#include "sv_checks.cuh"
#include "sv_device.cuh"
#include "sv_launch.cuh"

namespace sv {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjWarps = kAdjThreads / 32;

struct AdjustArgs {
    const void *in;
    void *out;
    int64_t in_bs, in_rs, out_bs, out_rs;
    int rows, V;
    const int32_t *history, *lengths, *prompt_lengths;
    int64_t history_stride;
    const int32_t *drafts, *parent;
    int ndraft;  // draft tokens per sequence (0: none counted)
    const float *repetition, *frequency, *presence;
    const int32_t *bias_tokens;
    const float *bias_values;
    int nbias;
    const uint32_t *allowed;
    bool in_place;
};

constexpr uint32_t kPrompt = 0x80000000u;  // table word: the prompt holds the token; low bits: output count

constexpr int kVecs = 4, kChunkVecs = 32 * kVecs;  // 16-byte vectors per lane and per chunk
constexpr int kRing = 3;                           // chunks of a warp in shared memory (4: 255 us for 251 below)

template <int TV>
struct AdjustShared {
    uint4 chunk[kAdjWarps][kRing][kChunkVecs];
    uint32_t mask[kAdjWarps][kRing][36];           // the chunk's words of the allowed mask
    alignas(16) uint32_t count[TV];                // of a listed token that is no draft: what its logit gains, as a float
    alignas(16) uint32_t winner[TV / 2];                       // 16 bits each: 1 + index of the token's last bias entry, 0: none
    uint16_t list[TV];                             // the touched tokens in order, and two flags
    uint32_t touched[TV / 32], drafted[TV / 32];   // tokens of history, drafts or bias list; of the drafts
    int before[TV / 32];                           // listed tokens before each word of `touched`
};
constexpr uint32_t kSeen = 0x4000u, kDrafted = 0x8000u;  // flags of a listed token
static_assert(SV_MAX_BIAS < 65535, "");

// Four bits as byte masks' top bits: bit j to bit 8 j + 7.
__device__ __forceinline__ uint32_t spread4(uint32_t bits) { return (bits * 0x10204080u) & 0x80808080u; }
// Bytes of v by prmt's selector: 8 + j is byte j's sign, eight times over.
template <uint32_t S>
__device__ __forceinline__ uint32_t pick(uint32_t v) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(v), "n"(S));
    return r;
}
__device__ __forceinline__ uint32_t keep(uint32_t v, uint32_t m, uint32_t other) { return (v & m) | (other & ~m); }

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int per = 4;
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float round(float x) { return x; }
    // -inf where the bit of an element is clear
    static __device__ __forceinline__ void mask(uint4 &v, uint32_t ok) {
        v.x = ok & 1 ? v.x : 0xFF800000u, v.y = ok & 2 ? v.y : 0xFF800000u;
        v.z = ok & 4 ? v.z : 0xFF800000u, v.w = ok & 8 ? v.w : 0xFF800000u;
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int per = 8;
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ void mask(uint4 &v, uint32_t ok) {
        const uint32_t a = spread4(ok & 15), b = spread4(ok >> 4);  // a byte's sign selects a half-word
        v.x = keep(v.x, pick<0x9988u>(a), 0xFF80FF80u), v.y = keep(v.y, pick<0xBBAAu>(a), 0xFF80FF80u);
        v.z = keep(v.z, pick<0x9988u>(b), 0xFF80FF80u), v.w = keep(v.w, pick<0xBBAAu>(b), 0xFF80FF80u);
    }
};

__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Walks the drafts of row r's context, nearest first: f(draft index).
template <typename F>
__device__ __forceinline__ void for_path(const int *parent_s, int r, F f) {
    if (parent_s == nullptr) {
        for (int j = r - 1; j >= 0; --j) f(j);
    } else {
        for (int v = r; v > 0;) {  // strictly falling: a parent that is not before its node ends the walk
            f(v);
            const int u = parent_s[v];
            v = u < v ? u : 0;
        }
    }
}

template <typename T, int TV>
__global__ void __launch_bounds__(kAdjThreads, 2) adjust_kernel(const AdjustArgs a, int batch) {
    extern __shared__ __align__(16) unsigned char raw[];
    using Sh = AdjustShared<TV>;
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    int *draft_s = reinterpret_cast<int *>(raw + sizeof(Sh));
    int *parent_s = a.parent ? draft_s + a.ndraft : nullptr;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // low ranges first: they hold a vocabulary's frequent tokens, and with them most of the arithmetic
    const int64_t b = blockIdx.x % batch;
    const int t0 = int(blockIdx.x / batch) * TV;
    const int n = min(TV, a.V - t0);  // tokens of this range
    using E = Elem<T>;
    constexpr int per = E::per;
    constexpr uint32_t kAll = (1u << per) - 1;
    // warps step through the rows, each time at the next place in the range (the arithmetic is uneven over it)
    constexpr int kChunks = (TV / per + kChunkVecs - 1) / kChunkVecs, kRowStep = kAdjWarps / kChunks;
    static_assert(kChunks * kRowStep == kAdjWarps, "");
    const int first_row = warp / kChunks;
    const int64_t words = (int64_t(a.V) + 31) / 32;

    griddep_launch_next();
    for (int i = tid; i < TV / 4; i += kAdjThreads) reinterpret_cast<uint4 *>(sh.count)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < TV / 8; i += kAdjThreads) reinterpret_cast<uint4 *>(sh.winner)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < TV / 32; i += kAdjThreads) sh.touched[i] = 0, sh.drafted[i] = 0;
    griddep_wait();

    // Elements before the 16-byte grid, and this warp's vectors after them, of a row that begins at p.
    auto head_of = [&](const T *p) { return min(n, int((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / int(sizeof(T))); };
    auto vectors_of = [&](int head, int v0) { return max(0, min((n - head) / per - v0, kChunkVecs)); };
    const T *src = static_cast<const T *>(a.in) + b * a.in_bs + first_row * a.in_rs + t0;
    T *dst = static_cast<T *>(a.out) + b * a.out_bs + first_row * a.out_rs + t0;
    const uint32_t *mask = a.allowed ? a.allowed + (b * a.rows + first_row) * words : nullptr;
    // the copies run kRing - 1 rows ahead
    const T *src_ahead = src;
    const uint32_t *mask_ahead = mask;
    int row_ahead = first_row, v0_ahead = warp % kChunks * kChunkVecs;
    auto step = [](int v0) { return v0 + kChunkVecs == kChunks * kChunkVecs ? 0 : v0 + kChunkVecs; };
    auto fetch = [&](int slot) {
        if (row_ahead < a.rows) {
            const int v0 = v0_ahead, head = head_of(src_ahead), count = vectors_of(head, v0);
            const uint4 *from = reinterpret_cast<const uint4 *>(src_ahead + head) + v0 + lane;
            uint4 *to = &sh.chunk[warp][slot][lane];
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
                if (u * 32 + lane < count) copy_async16(to + u * 32, from + u * 32);
            if (mask_ahead && count > 0) {  // at most 33 words
                const int e0 = t0 + head + v0 * per, w0 = e0 >> 5, w1 = (e0 + count * per - 1) >> 5;
                if (w0 + lane <= w1) copy_async4(&sh.mask[warp][slot][lane], mask_ahead + w0 + lane);
                if (lane == 0 && w0 + 32 <= w1) copy_async4(&sh.mask[warp][slot][32], mask_ahead + w0 + 32);
            }
            row_ahead += kRowStep, v0_ahead = step(v0), src_ahead += kRowStep * a.in_rs;
            if (mask_ahead) mask_ahead += kRowStep * words;
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(i);

    // the tokens of this range that the history, the drafts and the bias list hold
    for (int i = tid; i < a.ndraft; i += kAdjThreads) draft_s[i] = a.drafts[b * a.ndraft + i];
    if (parent_s)
        for (int i = tid; i < a.rows; i += kAdjThreads) parent_s[i] = a.parent[i];
    __syncthreads();
    if (a.history) {
        const int stride = int(a.history_stride);
        const int L = min(max(a.lengths[b], 0), stride), P = a.prompt_lengths ? a.prompt_lengths[b] : 0;
        const int32_t *h = a.history + b * a.history_stride;
        auto note = [&](int32_t tok, int i) {
            const uint32_t k = uint32_t(tok) - uint32_t(t0);
            if (k < uint32_t(n)) {
                if (i < P) atomicOr(&sh.count[k], kPrompt);
                else atomicAdd(&sh.count[k], 1u);
                atomicOr(&sh.touched[k >> 5], 1u << (k & 31));
            }
        };
        int i = 0;
        if ((reinterpret_cast<uintptr_t>(h) & 15) == 0) {
            const int4 *h4 = reinterpret_cast<const int4 *>(h);
            i = L & ~3;
            for (int q = tid; q < L / 4; q += 2 * kAdjThreads) {  // two loads in flight
                const int q2 = q + kAdjThreads;
                const int4 none = make_int4(-1, -1, -1, -1), v = __ldg(h4 + q), w = q2 < L / 4 ? __ldg(h4 + q2) : none;
                const uint32_t z = uint32_t(t0), m = uint32_t(n);
                if ((uint32_t(v.x) - z < m) | (uint32_t(v.y) - z < m) | (uint32_t(v.z) - z < m) | (uint32_t(v.w) - z < m))
                    note(v.x, 4 * q), note(v.y, 4 * q + 1), note(v.z, 4 * q + 2), note(v.w, 4 * q + 3);
                if ((uint32_t(w.x) - z < m) | (uint32_t(w.y) - z < m) | (uint32_t(w.z) - z < m) | (uint32_t(w.w) - z < m))
                    note(w.x, 4 * q2), note(w.y, 4 * q2 + 1), note(w.z, 4 * q2 + 2), note(w.w, 4 * q2 + 3);
            }
        }
        for (i += tid; i < L; i += kAdjThreads) note(__ldg(h + i), i);
    }
    for (int i = tid; i < a.nbias; i += kAdjThreads) {
        const uint32_t k = uint32_t(__ldg(a.bias_tokens + b * a.nbias + i)) - uint32_t(t0);
        if (k < uint32_t(n)) {
            uint32_t *word = &sh.winner[k >> 1], old = *word;
            const uint32_t shift = 16 * (k & 1), mine = uint32_t(i + 1);
            while ((old >> shift & 0xFFFFu) < mine) {  // the largest index stays, whatever the order
                const uint32_t was = atomicCAS(word, old, (old & ~(0xFFFFu << shift)) | mine << shift);
                if (was == old) break;
                old = was;
            }
            atomicOr(&sh.touched[k >> 5], 1u << (k & 31));
        }
    }
    for (int i = tid; i < a.ndraft; i += kAdjThreads) {
        const uint32_t k = uint32_t(draft_s[i]) - uint32_t(t0);
        if (k < uint32_t(n)) {
            atomicOr(&sh.drafted[k >> 5], 1u << (k & 31));
            atomicOr(&sh.touched[k >> 5], 1u << (k & 31));
        }
    }
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        for (int i0 = 0; i0 < TV / 32; i0 += 32) {
            const int c = __popc(sh.touched[i0 + lane]);
            int inc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += v;
            }
            sh.before[i0 + lane] = run + inc - c;
            run += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
    }
    __syncthreads();
    // the list; a token that is no draft has the same penalties and bias in every row
    const float rep = a.repetition ? a.repetition[b] : 1.f, inverse = 1.f / rep;
    const float freq = a.frequency ? a.frequency[b] : 0.f;
    const float pres = a.presence ? a.presence[b] : 0.f;
    auto gain = [&](uint32_t word, int k) {  // of token k with a count word
        const uint32_t c = word & ~kPrompt, won = sh.winner[k >> 1] >> (16 * (k & 1)) & 0xFFFFu;
        const float penalty = fmaf(freq, float(c), c ? pres : 0.f);
        return (won && SV_IN(won - 1, a.nbias) ? __ldg(a.bias_values + b * a.nbias + won - 1) : 0.f) - penalty;
    };
    for (int i = tid; i < TV / 32; i += kAdjThreads) {
        const uint32_t drafts = sh.drafted[i];
        int at = sh.before[i];
        for (uint32_t w = sh.touched[i]; w; w &= w - 1) {
            const int j = __ffs(w) - 1, k = i * 32 + j;
            const uint32_t word = sh.count[k];
            uint32_t flags = word ? kSeen : 0;
            if (drafts >> j & 1) flags = kDrafted;
            else sh.count[k] = __float_as_uint(gain(word, k));
            sh.list[at++] = uint16_t(uint32_t(k) | flags);
        }
    }
    __syncthreads();

    // Penalties and bias of a touched token in row r (a division by the repetition penalty is a product with
    // its reciprocal: one more rounding of 2^-24).
    auto adjust = [&](float l, int r, uint32_t entry) {
        const int k = entry & 0x3FFFu;
        if (!SV_IN(k, n)) return l;
        uint32_t word = sh.count[k];
        float g = __uint_as_float(word);
        bool seen = entry & kSeen;
        if (entry & kDrafted) {
            if (r > 0) for_path(parent_s, r, [&](int j) { word += draft_s[j] == t0 + k; });
            g = gain(word, k), seen = word != 0;
        }
        if (seen) l *= l > 0.f ? inverse : rep;
        return l + g;
    };
    auto is_touched = [&](int k) { return sh.touched[k >> 5] >> (k & 31) & 1u; };
    auto listed_before = [&](int k) { return sh.before[k >> 5] + __popc(sh.touched[k >> 5] & ((1u << (k & 31)) - 1)); };

    int slot = 0, v0 = warp % kChunks * kChunkVecs;
    for (int r = first_row; r < a.rows; r += kRowStep) {
        fetch(slot == 0 ? kRing - 1 : slot - 1);
        const int head = head_of(src), count = vectors_of(head, v0);
        auto scalar = [&](int k) {
            const bool ok = mask == nullptr || (__ldg(mask + ((t0 + k) >> 5)) >> ((t0 + k) & 31) & 1u), mine = is_touched(k);
            if (a.in_place && ok && !mine) return;
            const T v = src[k];
            dst[k] = !ok ? E::round(-__int_as_float(0x7f800000)) : mine ? E::round(adjust(E::get(v), r, sh.list[listed_before(k)])) : v;
        };
        copy_wait<kRing - 1>();
        __syncwarp();
        if (((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15) != 0) {
            // the two rows lie differently on the 16-byte grid
            const int k1 = min(n, (v0 + kChunkVecs) * per);
            for (int k = v0 * per + lane; k < k1; k += 32) scalar(k);
        } else {
            if (v0 == 0 && (head > 0 || (n - head) % per != 0)) {  // the row's ends off the grid
                const int tail = head + (n - head) / per * per;
                if (lane < head) scalar(lane);
                if (lane < n - tail) scalar(tail + lane);
            }
            uint4 *mine = &sh.chunk[warp][slot][0];
            const int k0 = head + v0 * per;  // the chunk's first token
            if (count > 0) {
                const int last = k0 + count * per - 1, e0 = listed_before(k0), e1 = listed_before(last) + int(is_touched(last));
                if (e0 < e1) {
                    T *elems = reinterpret_cast<T *>(mine);
                    for (int e = e0 + lane; e < e1; e += 32) {
                        const uint32_t entry = sh.list[e];
                        const int k = int(entry & 0x3FFFu) - k0;
                        if (SV_IN(k, count * per)) elems[k] = E::round(adjust(E::get(elems[k]), r, entry));
                    }
                    __syncwarp();
                }
            }
            uint4 *to = reinterpret_cast<uint4 *>(dst + head) + v0 + lane;
            const uint32_t first = (uint32_t(t0 + k0) & 31) + lane * per;
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                if (u * 32 + lane >= count) continue;
                uint32_t ok = kAll;
                if (mask) {
                    const uint32_t e = first + u * 32 * per;
                    const uint32_t *m = &sh.mask[warp][slot][e >> 5];
                    ok = __funnelshift_r(m[0], m[1], e & 31) & kAll;  // (m[1] unread bits: any)
                }
                if (a.in_place && ok == kAll) {  // only what changes is written
                    const int k = k0 + (u * 32 + lane) * per;
                    const uint32_t s = uint32_t(k) & 31, hi = s + per > 32 ? sh.touched[(k >> 5) + 1] : 0u;
                    if ((__funnelshift_r(sh.touched[k >> 5], hi, s) & kAll) == 0) continue;
                }
                uint4 x = mine[u * 32 + lane];
                if (ok != kAll) E::mask(x, ok);
                to[u * 32] = x;
            }
        }
        __syncwarp();  // the buffer may be filled again
        src += kRowStep * a.in_rs, dst += kRowStep * a.out_rs;
        if (mask) mask += kRowStep * words;
        slot = slot + 1 == kRing ? 0 : slot + 1;
        v0 = step(v0);
    }
    copy_wait<0>();
}

template <typename T, int TV>
cudaError_t launch_adjust(const AdjustArgs &a, int B, int tiles, cudaStream_t s) {
    const size_t smem = sizeof(AdjustShared<TV>) + (size_t(a.ndraft) + (a.parent ? a.rows : 0)) * 4;
    static std::atomic<int> allowed[64];
    const cudaError_t e = allow_shared(adjust_kernel<T, TV>, int(smem), allowed);
    if (e != cudaSuccess) return e;
    return launch_after(adjust_kernel<T, TV>, unsigned(int64_t(B) * tiles), kAdjThreads, smem, s, a, B);
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_logit_adjust(const void *logits, int64_t batch_stride, int64_t row_stride, void *out,
                                       int64_t out_batch_stride, int64_t out_row_stride, sv_dtype dtype, int B,
                                       int rows, int V, const int32_t *history, int64_t history_stride,
                                       const int32_t *lengths, const int32_t *prompt_lengths,
                                       const int32_t *draft_tokens, const int32_t *parent, const float *repetition,
                                       const float *frequency, const float *presence, const int32_t *bias_tokens,
                                       const float *bias_values, int nbias, const int32_t *allowed, void *stream) {
    if (dtype != SV_FP32 && dtype != SV_BF16) return SV_ERR_UNSUPPORTED;
    if (B < 0 || rows < 0 || V < 1 || V > SV_MAX_VOCAB || nbias < 0 || nbias > SV_MAX_BIAS) return SV_ERR_INVALID_ARG;
    if (rows > (parent ? SV_MAX_TREE_NODES : SV_MAX_GAMMA + 1)) return SV_ERR_INVALID_ARG;
    if (batch_stride < 0 || row_stride < 0 || out_batch_stride < 0 || out_row_stride < 0) return SV_ERR_INVALID_ARG;
    if (history_stride < 0 || history_stride > SV_MAX_HISTORY) return SV_ERR_INVALID_ARG;
    if (B == 0 || rows == 0) return SV_OK;
    if (!logits || !out || (history && !lengths) || (parent && !draft_tokens)) return SV_ERR_INVALID_ARG;
    if (nbias > 0 && (!bias_tokens || !bias_values)) return SV_ERR_INVALID_ARG;
    // distinct output rows must not share memory
    if ((rows > 1 && out_row_stride < V) || (B > 1 && out_batch_stride < V)) return SV_ERR_INVALID_ARG;
    if (out == logits && ((rows > 1 && out_row_stride != row_stride) || (B > 1 && out_batch_stride != batch_stride)))
        return SV_ERR_INVALID_ARG;
    const size_t es = dtype == SV_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(out) % es) return SV_ERR_INVALID_ARG;
    sv::AdjustArgs a{};
    a.in = logits, a.out = out;
    a.in_bs = batch_stride, a.in_rs = row_stride, a.out_bs = out_batch_stride, a.out_rs = out_row_stride;
    a.rows = rows, a.V = V;
    a.history = history_stride > 0 ? history : nullptr;
    a.lengths = lengths, a.prompt_lengths = prompt_lengths, a.history_stride = history_stride;
    a.drafts = draft_tokens, a.parent = parent;
    a.ndraft = draft_tokens ? (parent ? rows : rows - 1) : 0;
    a.repetition = repetition, a.frequency = frequency, a.presence = presence;
    a.bias_tokens = bias_tokens, a.bias_values = bias_values, a.nbias = nbias;
    a.allowed = reinterpret_cast<const uint32_t *>(allowed);
    a.in_place = out == logits;
    // small batches: shorter token ranges, so that every SM has work
    const int64_t big = (int64_t(V) + 4095) / 4096, small = (int64_t(V) + 1023) / 1024;
    const bool wide = int64_t(B) * big >= 304;
    const int64_t tiles = wide ? big : small;
    if (int64_t(B) * tiles > 0x7FFFFFFF) return SV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == SV_BF16)
        e = wide ? sv::launch_adjust<__nv_bfloat16, 4096>(a, B, int(tiles), s)
                 : sv::launch_adjust<__nv_bfloat16, 1024>(a, B, int(tiles), s);
    else
        e = wide ? sv::launch_adjust<float, 4096>(a, B, int(tiles), s)
                 : sv::launch_adjust<float, 1024>(a, B, int(tiles), s);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
