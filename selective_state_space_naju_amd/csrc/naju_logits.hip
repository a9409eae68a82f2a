// naju_logits.hip -- logits made ready for the choice of a token: penalties for
// tokens that occurred before, biases, a grammar's mask, and the best token.
//
// Per row, with c_v the occurrences of v among the row's earlier tokens:
//     x = l_v
//     if c_v > 0:  x = x > 0 ? x / r : x r;   x = x - f c_v;   x = x - a
//     x = x + bias_v                     (the first listed pair of v)
//     x = -inf where the mask does not allow v
// and best = the lowest index of the largest x, -1 where nothing is above -inf.
//
// Few tokens of a row are penalised or biased, so the arithmetic is done for
// those alone.  A workgroup owns a tile of one row's vocabulary and keeps one
// LDS word per token of it: the row's bias list and history are scanned and
// counted there, the tokens that were touched are listed, their values are
// computed once each into their words, and the dense pass that follows only
// selects between a word and the logit.  It reads every logit and writes every
// result once.  256 x 131072 bf16 with 4096 tokens of history, 300 biases and a
// mask: 50 us (4.2 TB/s); the dense pass alone is 35 us, the rest is the lists'
// latency between barriers.
#include "naju_device.h"
#include "naju_host.h"
#include "naju_launch.h"
#include "naju_vec.h"

namespace naju {

constexpr int kLogThreads = 1024;
constexpr int kLogTile = 16384;        // most tokens of a workgroup
constexpr int kLogSmallTile = 4096;
constexpr int kLogRuns = kLogTile / (4 * kLogThreads);  // accesses of 4 tokens per thread
constexpr int kCountBits = 20;         // a word: list place (12 bits) | count (20 bits)
constexpr uint32_t kCountMask = (1u << kCountBits) - 1;
constexpr int kPlaces = 4095;          // biases of a row
constexpr int64_t kMostHistory = kCountMask;

struct LogitsArgs {
    int64_t B, V;
    int tile;
    int64_t n_tiles;
    int64_t ld;
    const int32_t *history;       // [B][H] or null
    int64_t H;
    const int32_t *lengths;       // [B] or null (= H)
    const float *rep, *pres, *freq;  // [B] or null
    const int32_t *bias_ids;      // [B][nb] or null
    const float *bias;
    int nb;
    const uint32_t *mask;         // [B][ceil(V / 32)] or null
    float *out;                   // [B][V]
    int32_t *best;                // [B] or null
    char *ws;                     // RowBest[B]
};

// the best token over the tiles of a row, and the tiles that have reported
struct RowBest {
    uint64_t key;
    uint32_t done, pad;
};

// Order-preserving key of (value, index): larger values first, then lower
// indices; 0 stands for nothing above -inf.
__device__ __forceinline__ uint64_t best_key(float v, int32_t idx)
{
    if (idx < 0) return 0;
    const uint32_t b = __float_as_uint(v + 0.f);  // (-0 and 0 are equal)
    const uint32_t o = (b >> 31) ? ~b : b | 0x80000000u;
    return ((uint64_t)o << 32) | (uint32_t)~(uint32_t)idx;
}
__device__ __forceinline__ int32_t key_index(uint64_t k)
{
    return k ? (int32_t)~(uint32_t)k : -1;
}

// A touched token's value.  Every operation rounds by itself, as written.
__device__ __forceinline__ float penalised(float x, uint32_t count, const LogitsArgs &g, int64_t b)
{
#pragma clang fp contract(off)
    if (count > 0) {
        if (g.rep) {
            const float r = g.rep[b];
            x = x > 0.f ? x / r : x * r;
        }
        if (g.freq) {
            const float f = g.freq[b] * (float)count;
            x = x - f;
        }
        if (g.pres) x = x - g.pres[b];
    }
    return x;
}

template <typename IO>
__global__ __launch_bounds__(kLogThreads, 8) void logits_kernel(const LogitsArgs g,
                                                                const IO *__restrict__ logits,
                                                                const int64_t first)
{
    // word[tile], then the list of touched tokens, at most H + nb of them
    extern __shared__ __attribute__((aligned(16))) uint32_t word[];
    uint16_t *list = (uint16_t *)(word + g.tile);
    __shared__ uint32_t n_list;
    __shared__ uint64_t wave_best[kLogThreads / 64];
    const int tid = threadIdx.x;
    const bool touched = g.H > 0 || g.nb > 0;
    const int64_t b = first + blockIdx.x / (uint32_t)g.n_tiles;
    const int64_t v0 = (int64_t)(blockIdx.x % (uint32_t)g.n_tiles) * g.tile;
    const int nv = g.V - v0 < g.tile ? (int)(g.V - v0) : g.tile;
    const IO *row = logits + b * g.ld + v0;
    const uint32_t *mrow = g.mask ? g.mask + b * ((g.V + 31) / 32) + v0 / 32 : nullptr;
    // the first of the lists, then the tile's logits and mask words, all in flight while the
    // lists are counted (loads return in order: the lists would wait behind the logits)
    const int32_t *bi = g.bias_ids + b * g.nb, *h = g.history + b * g.H;
    int32_t bias0 = tid < g.nb ? bi[tid] : -1;
    Run<IO, 4> in[kLogRuns];
    uint32_t allowed[kLogRuns];
#pragma unroll
    for (int i = 0; i < kLogRuns; ++i) {
        const int c = (i * kLogThreads + tid) * 4;
        in[i].zero();
        allowed[i] = ~0u;
        if (c + 4 <= nv) {
            in[i].load(row + c);
            if (mrow) allowed[i] = mrow[c >> 5];
        }
    }
    if (touched) {
        for (int i = tid * 4; i < g.tile; i += kLogThreads * 4)
            *(uint4 *)&word[i] = make_uint4(0, 0, 0, 0);
        if (tid == 0) n_list = 0;
        __syncthreads();
        // bias list: the first pair that names a token has the highest mark
        for (int j = tid; j < g.nb; j += kLogThreads) {
            const int64_t v = (j == tid ? bias0 : bi[j]) - v0;
            if (v >= 0 && v < nv) atomicMax(&word[v], (uint32_t)(kPlaces - j) << kCountBits);
        }
        __syncthreads();
        for (int j = tid; j < g.nb; j += kLogThreads) {
            const int64_t v = bi[j] - v0;
            if (v >= 0 && v < nv && (word[v] >> kCountBits) == (uint32_t)(kPlaces - j))
                list[atomicAdd(&n_list, 1u)] = (uint16_t)v;
        }
        // history: whoever counts a token first lists it
        int64_t len = g.H;
        if (g.lengths) {
            len = g.lengths[b];
            len = len < 0 ? 0 : len > g.H ? g.H : len;
        }
        for (int64_t i = (int64_t)tid * 4; i < len; i += kLogThreads * 4) {
            Run<float, 4> r;
            const int m = len - i < 4 ? (int)(len - i) : 4;
            if (m == 4) r.load((const float *)h + i);
            else r.load_part((const float *)h + i, m);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t v = (int32_t)r.w[q] - v0;
                if (q < m && v >= 0 && v < nv)
                    if (atomicAdd(&word[v], 1u) == 0) list[atomicAdd(&n_list, 1u)] = (uint16_t)v;
            }
        }
        __syncthreads();
        const int n = (int)n_list;
        for (int i = tid; i < n; i += kLogThreads) {
            const int v = list[i];
            const uint32_t w = word[v];
            float x = penalised(to_f(row[v]), w & kCountMask, g, b);
            if (w >> kCountBits) x = x + g.bias[b * g.nb + (kPlaces - (w >> kCountBits))];
            if (x != x) x = __uint_as_float(0x7fc00000u);
            word[v] = ~__float_as_uint(x);  // (0 only for a NaN pattern that is not used)
        }
        __syncthreads();
    }
    // dense pass
    float top = -__builtin_huge_valf();
    int32_t at = -1;
    float *out = g.out + b * g.V + v0;
#pragma unroll
    for (int i = 0; i < kLogRuns; ++i) {
        const int c = (i * kLogThreads + tid) * 4;
        if (c + 4 > nv) continue;
        float x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = in[i].get(q);
        if (touched) {
            const uint4 w = *(const uint4 *)&word[c];
            x[0] = w.x ? __uint_as_float(~w.x) : x[0];
            x[1] = w.y ? __uint_as_float(~w.y) : x[1];
            x[2] = w.z ? __uint_as_float(~w.z) : x[2];
            x[3] = w.w ? __uint_as_float(~w.w) : x[3];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (!((allowed[i] >> ((c & 31) + q)) & 1u)) x[q] = -__builtin_huge_valf();
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (x[q] > top) {
                top = x[q];
                at = c + q;
            }
        round_run<float, 4>(x).store(out + c);
    }
    // the last one to three tokens
    if (tid < (nv & 3)) {
        const int c = (nv & ~3) + tid;
        float x = to_f(row[c]);
        if (touched && word[c]) x = __uint_as_float(~word[c]);
        if (mrow && !((mrow[c >> 5] >> (c & 31)) & 1u)) x = -__builtin_huge_valf();
        if (x > top) {
            top = x;
            at = c;
        }
        out[c] = x;
    }
    if (g.best) {
        uint64_t k = best_key(top, at < 0 ? -1 : (int32_t)(v0 + at));
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const uint64_t x = __shfl_xor(k, o);
            k = x > k ? x : k;
        }
        if ((tid & 63) == 0) wave_best[tid >> 6] = k;
        __syncthreads();
        if (tid == 0) {
            for (int i = 1; i < kLogThreads / 64; ++i) k = wave_best[i] > k ? wave_best[i] : k;
            if (g.n_tiles == 1) {
                g.best[b] = key_index(k);
            } else {
                // the last tile of the row to report reads the row's key and clears
                // the record for the next call.  Only the record's own words pass
                // between workgroups, all by agent-scope atomics, so their order
                // (the wait) is enough: a release here would write every dirty line
                // of the L2 back first (243 us against 80 us at 256 x 131072)
                RowBest *rb = (RowBest *)g.ws + b;
                __hip_atomic_fetch_max(&rb->key, k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                wait_mem();
                const uint32_t d = add_agent(&rb->done, 1u);
                if (d + 1 == (uint32_t)g.n_tiles) {
                    k = __hip_atomic_exchange(&rb->key, (uint64_t)0, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
                    st_agent(&rb->done, 0u);
                    g.best[b] = key_index(k);
                }
            }
        }
    }
}

static size_t logits_ws_bytes(int64_t rows) { return align256(sizeof(RowBest) * (size_t)rows); }

template <typename IO>
static hipError_t launch_logits(const LogitsArgs &g, const void *logits, hipStream_t st)
{
    size_t lds = 0;
    if (g.H > 0 || g.nb > 0) {
        const int64_t most = g.H + g.nb;
        lds = (size_t)g.tile * 4 + (size_t)(most < g.tile ? most : g.tile) * 2;
    }
    // (above 64 KB a kernel has to ask for its LDS)
    if (lds > (64 << 10)) {
        const hipError_t e = hipFuncSetAttribute(
            (const void *)logits_kernel<IO>, hipFuncAttributeMaxDynamicSharedMemorySize, 128 << 10);
        if (e != hipSuccess) return e;
    }
    const int64_t most = ((int64_t)1 << 21) / g.n_tiles + 1;  // rows of a launch
    for (int64_t r = 0; r < g.B; r += most) {
        const int64_t rows = g.B - r < most ? g.B - r : most;
        hipLaunchKernelGGL(logits_kernel<IO>, dim3((unsigned)(rows * g.n_tiles)), dim3(kLogThreads),
                           lds, st, g, (const IO *)logits, r);
    }
    return hipGetLastError();
}

static naju_status_t check_logits(int64_t rows, int64_t vocab)
{
    if (rows < 0 || vocab < 0)
        return fail(NAJU_EINVAL, "negative size (rows=%lld vocab=%lld)", (long long)rows,
                    (long long)vocab);
    if (rows > ((int64_t)1 << 24) || vocab > ((int64_t)1 << 30))
        return fail(NAJU_EINVAL, "rows (2^24 max) or vocab (2^30 max) too large");
    return NAJU_OK;
}

}  // namespace naju

using namespace naju;

extern "C" {

size_t naju_logits_workspace_bytes(int64_t rows)
{
    if (check_logits(rows, 1) != NAJU_OK) return 0;
    return logits_ws_bytes(rows);
}

naju_status_t naju_logits_process(int64_t rows, int64_t vocab, int32_t io, const void *logits,
                                  int64_t ld, const int32_t *history, int64_t history_len,
                                  const int32_t *lengths, const float *repetition,
                                  const float *presence, const float *frequency,
                                  const int32_t *bias_ids, const float *bias, int64_t n_bias,
                                  const uint32_t *mask, float *out, int32_t *best, void *ws,
                                  size_t ws_bytes, void *stream)
{
    NAJU_TRY(check_logits(rows, vocab));
    if (io != NAJU_F32 && io != NAJU_BF16)
        return fail(NAJU_EINVAL, "io dtype %d is neither NAJU_F32 nor NAJU_BF16", (int)io);
    if (history_len < 0 || n_bias < 0)
        return fail(NAJU_EINVAL, "negative size (history_len=%lld n_bias=%lld)",
                    (long long)history_len, (long long)n_bias);
    if (history_len > kMostHistory)
        return fail(NAJU_EUNSUPPORTED, "history_len %lld (%lld max)", (long long)history_len,
                    (long long)kMostHistory);
    if (n_bias >= kPlaces)
        return fail(NAJU_EUNSUPPORTED, "n_bias %lld (%d max)", (long long)n_bias, kPlaces - 1);
    if (rows == 0 || vocab == 0) return NAJU_OK;
    if (ld < vocab || ld > ((int64_t)1 << 31))
        return fail(NAJU_EINVAL, "row stride of logits %lld (vocab is %lld)", (long long)ld,
                    (long long)vocab);
    NAJU_TRY(need(logits, "logits", io == NAJU_F32 ? 4 : 2));
    NAJU_TRY(need(out, "out", 4));
    if (history_len > 0) NAJU_TRY(need(history, "history", 4));
    NAJU_TRY(opt(lengths, "lengths", 4));
    NAJU_TRY(opt(repetition, "repetition", 4));
    NAJU_TRY(opt(presence, "presence", 4));
    NAJU_TRY(opt(frequency, "frequency", 4));
    if (n_bias > 0) {
        NAJU_TRY(need(bias_ids, "bias_ids", 4));
        NAJU_TRY(need(bias, "bias", 4));
    }
    NAJU_TRY(opt(mask, "mask", 4));
    NAJU_TRY(opt(best, "best", 4));
    if (best) NAJU_TRY(need_ws(ws, ws_bytes, logits_ws_bytes(rows)));
    LogitsArgs g{};
    g.B = rows;
    g.V = vocab;
    // small tiles only where large ones leave most CUs idle (2048 tokens of history, 16 biases and
    // a mask, large and small, us: 1 x 32000 7.6 and 7.4, 8 x 50001 8.7 and 7.4, 16 x 131072 9.6
    // and 12.6, 256 x 131072 48 and 108)
    g.tile = rows * ((vocab + kLogTile - 1) / kLogTile) >= 64 ? kLogTile : kLogSmallTile;
    g.n_tiles = (vocab + g.tile - 1) / g.tile;
    g.ld = ld;
    g.history = history;
    g.H = history_len;
    g.lengths = lengths;
    g.rep = repetition;
    g.pres = presence;
    g.freq = frequency;
    g.bias_ids = bias_ids;
    g.bias = bias;
    g.nb = (int)n_bias;
    g.mask = mask;
    g.out = out;
    g.best = best;
    g.ws = (char *)ws;
    hipStream_t st = (hipStream_t)stream;
    return hip_status(io == NAJU_F32 ? launch_logits<float>(g, logits, st)
                                     : launch_logits<bf16>(g, logits, st),
                      "logits launch");
}

}  // extern "C"
