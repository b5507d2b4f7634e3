// sv_adjust.cu -- penalties, biases and grammar masks on the verified rows' logits.
//
// For token t of row i, with n its occurrences in the output part of the row's context and s
// whether the context holds it at all:
//   l := s ? (l > 0 ? l / r : l r) : l;  l -= f n + p (n > 0);  l += bias(t);  masked: -inf
// in fp32, rounded once to the logits' type.  One pass: every logit is read once and written
// once (in place: only the 16-byte groups that change are written), so DRAM bounds it.
//
// A CTA owns TV consecutive tokens of one sequence for all its rows.  It streams its part of every
// row through registers, masked, 16 bytes a lane and eight loads in flight; meanwhile it counts
// the history's tokens of its range (a table in shared memory, integer atomics: the order does
// not matter).  The few tokens that the history, the drafts or the bias list touch are compacted into
// a list, and after the stream each (row, listed token) pair is computed from its logit, one
// thread each, and stored over the streamed one.  So the long part does no arithmetic on
// logits, and the part with arithmetic has no idle lanes.  The history is read once per token range
// from L2, the price of needing no second kernel and no table in DRAM.
#include <cstdint>

#include "spec_serve.h"
#include "sv_checks.cuh"
#include "sv_device.cuh"

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

template <int TV>
struct AdjustShared {
    uint32_t count[TV];
    uint32_t winner[TV];      // 1 + index of the last bias entry of the token, 0: none
    uint32_t touched[TV / 32];  // tokens of the history, the drafts or the bias list
    uint32_t drafted[TV / 32];  // tokens of the drafts
    uint16_t list[TV];        // the touched tokens
    int listed;
};

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
    static __device__ __forceinline__ uint32_t two(uint32_t v, uint32_t ok) {
        const uint32_t m = (ok & 1 ? 0xFFFFu : 0u) | (ok & 2 ? 0xFFFF0000u : 0u);
        return (v & m) | (0xFF80FF80u & ~m);
    }
    static __device__ __forceinline__ void mask(uint4 &v, uint32_t ok) {
        v.x = two(v.x, ok), v.y = two(v.y, ok >> 2), v.z = two(v.z, ok >> 4), v.w = two(v.w, ok >> 6);
    }
};

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
__global__ void __launch_bounds__(kAdjThreads)
    adjust_kernel(const AdjustArgs a, int tiles) {
    extern __shared__ __align__(16) unsigned char raw[];
    using Sh = AdjustShared<TV>;
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    int *draft_s = reinterpret_cast<int *>(raw + sizeof(Sh));
    int *parent_s = a.parent ? draft_s + a.ndraft : nullptr;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x / tiles;
    const int t0 = int(blockIdx.x % tiles) * TV;
    const int n = min(TV, a.V - t0);  // tokens of this range
    using E = Elem<T>;
    constexpr int per = E::per;

    griddep_launch_next();
    for (int i = tid; i < TV; i += kAdjThreads) sh.count[i] = 0, sh.winner[i] = 0;
    for (int i = tid; i < TV / 32; i += kAdjThreads) sh.touched[i] = 0, sh.drafted[i] = 0;
    if (tid == 0) sh.listed = 0;
    griddep_wait();
    const int64_t words = (int64_t(a.V) + 31) / 32;
    const T *in = static_cast<const T *>(a.in) + b * a.in_bs + t0;
    T *out = static_cast<T *>(a.out) + b * a.out_bs + t0;
    const uint32_t *allowed = a.allowed ? a.allowed + b * a.rows * words : nullptr;
    auto is_allowed = [&](int r, int k) {
        return allowed == nullptr || (__ldg(allowed + r * words + ((t0 + k) >> 5)) >> ((t0 + k) & 31) & 1u);
    };

    // the stream: warps take (row, chunk) pairs
    constexpr int U = 8, kChunk = 32 * U;
    const int chunks = (TV / per + kChunk - 1) / kChunk;
    for (int item = warp; item < a.rows * chunks; item += kAdjWarps) {
        const int r = item / chunks, part = item % chunks;
        const T *src = in + r * a.in_rs;
        T *dst = out + r * a.out_rs;
        auto scalar = [&](int k) {
            const bool ok = is_allowed(r, k);
            if (a.in_place && ok) return;
            dst[k] = ok ? src[k] : E::round(-__int_as_float(0x7f800000));
        };
        const uintptr_t ai = reinterpret_cast<uintptr_t>(src), ao = reinterpret_cast<uintptr_t>(dst);
        if (((ai ^ ao) & 15) != 0) {  // the two rows lie differently on the 16-byte grid
            const int k1 = min(n, (part + 1) * kChunk * per);
            for (int k = part * kChunk * per + lane; k < k1; k += 32) scalar(k);
            continue;
        }
        const int head = min(n, int((16 - (ai & 15)) & 15) / int(sizeof(T)));
        const int nv = (n - head) / per, tail = head + nv * per;
        if (part == 0) {  // the row's ends off the grid
            if (lane < head) scalar(lane);
            if (lane < n - tail) scalar(tail + lane);
        }
        const uint4 *src4 = reinterpret_cast<const uint4 *>(src + head);
        uint4 *dst4 = reinterpret_cast<uint4 *>(dst + head);
        const uint32_t *mask = allowed ? allowed + r * words : nullptr;
        constexpr uint32_t kAll = (1u << per) - 1;
        uint4 x[U];
        uint32_t ok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = part * kChunk + u * 32 + lane;
            ok[u] = kAll;
            if (v < nv) {
                x[u] = __ldcs(src4 + v);
                if (mask) {
                    const uint32_t e = uint32_t(t0 + head + v * per), s = e & 31;
                    const uint32_t lo = __ldg(mask + (e >> 5)), hi = s + per > 32 ? __ldg(mask + (e >> 5) + 1) : 0u;
                    ok[u] = __funnelshift_r(lo, hi, s) & kAll;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = part * kChunk + u * 32 + lane;
            if (v < nv && !(a.in_place && ok[u] == kAll)) {
                if (mask) E::mask(x[u], ok[u]);
                dst4[v] = x[u];
            }
        }
    }
    if (!a.history && a.ndraft == 0 && a.nbias == 0) return;

    // the tokens of this range that the history, the drafts and the bias list hold
    for (int i = tid; i < a.ndraft; i += kAdjThreads) draft_s[i] = a.drafts[b * a.ndraft + i];
    if (parent_s)
        for (int i = tid; i < a.rows; i += kAdjThreads) parent_s[i] = a.parent[i];
    __syncthreads();
    if (a.history) {
        const int64_t Lr = a.lengths[b];
        const int64_t L = Lr < 0 ? 0 : (Lr > a.history_stride ? a.history_stride : Lr);
        const int64_t P = a.prompt_lengths ? a.prompt_lengths[b] : 0;
        const int32_t *h = a.history + b * a.history_stride;
        auto note = [&](int32_t tok, int64_t i) {
            const uint32_t k = uint32_t(tok) - uint32_t(t0);
            if (k < uint32_t(n)) {
                if (i < P) atomicOr(&sh.count[k], kPrompt);
                else atomicAdd(&sh.count[k], 1u);
                atomicOr(&sh.touched[k >> 5], 1u << (k & 31));
            }
        };
        int64_t i = 0;
        if ((reinterpret_cast<uintptr_t>(h) & 15) == 0) {
            const int4 *h4 = reinterpret_cast<const int4 *>(h);
            for (int64_t q = tid; q < L / 4; q += kAdjThreads) {
                const int4 v = __ldg(h4 + q);
                note(v.x, 4 * q), note(v.y, 4 * q + 1), note(v.z, 4 * q + 2), note(v.w, 4 * q + 3);
            }
            i = L / 4 * 4;
        }
        for (i += tid; i < L; i += kAdjThreads) note(__ldg(h + i), i);
    }
    for (int i = tid; i < a.nbias; i += kAdjThreads) {
        const uint32_t k = uint32_t(__ldg(a.bias_tokens + b * a.nbias + i)) - uint32_t(t0);
        if (k < uint32_t(n)) {
            atomicMax(&sh.winner[k], uint32_t(i + 1));
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
    for (int i = tid; i < TV / 32; i += kAdjThreads) {
        uint32_t w = sh.touched[i];
        int at = w ? atomicAdd(&sh.listed, __popc(w)) : 0;
        for (; w; w &= w - 1) sh.list[at++] = uint16_t(i * 32 + __ffs(w) - 1);
    }
    __syncthreads();  // (and the streamed logits are in place for this CTA's threads)

    const float rep = a.repetition ? a.repetition[b] : 1.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f;
    const float pres = a.presence ? a.presence[b] : 0.f;
    const int listed = sh.listed;
    // threads take listed tokens, and of each the rows in turn (four loads in flight)
    const int groups = max(1, kAdjThreads / max(1, listed));  // threads that share a token
    for (int e = tid; e < listed * groups; e += kAdjThreads) {
        const int k = sh.list[e % listed], r0 = e / listed;
        if (!SV_IN(k, n)) continue;
        const uint32_t base = sh.count[k], won = sh.winner[k];
        const bool drafted = sh.drafted[k >> 5] >> (k & 31) & 1u;
        const float bias = won && SV_IN(won - 1, a.nbias) ? __ldg(a.bias_values + b * a.nbias + won - 1) : 0.f;
#pragma unroll 4
        for (int r = r0; r < a.rows; r += groups) {
            if (!is_allowed(r, k)) continue;
            uint32_t w = base;
            if (drafted) for_path(parent_s, r, [&](int j) { w += draft_s[j] == t0 + k; });
            const uint32_t c = w & ~kPrompt;
            float l = E::get(in[r * a.in_rs + k]);
            if (w) l = l > 0.f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
            l = __fsub_rn(__fsub_rn(l, __fmul_rn(freq, float(c))), c ? pres : 0.f);
            if (won) l = __fadd_rn(l, bias);
            out[r * a.out_rs + k] = E::round(l);
        }
    }
}

template <typename T, int TV>
cudaError_t launch_adjust(const AdjustArgs &a, int B, int tiles, cudaStream_t s) {
    const size_t smem = sizeof(AdjustShared<TV>) + (size_t(a.ndraft) + (a.parent ? a.rows : 0)) * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(adjust_kernel<T, TV>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    return launch_after(adjust_kernel<T, TV>, unsigned(int64_t(B) * tiles), kAdjThreads, smem, s, a, tiles);
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
