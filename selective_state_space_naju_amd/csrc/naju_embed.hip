// naju_embed.hip -- token embedding with scaling, and its gradient.
//
//     out[t]  = scale W[ids[t]]                 (0 where ids[t] is outside [0, V))
//     dW[v]  (+)= scale sum_{t : ids[t] = v} dout[t]
//
// The gradient sums each token's rows in the order of their positions, with no
// floating-point atomics, so equal inputs give equal bits: the positions are
// sorted by token (a stable radix sort), and the sorted list is cut into blocks
// of kBlk positions whose runs of equal tokens are summed in registers.  A run
// inside one block goes straight to dW; a run that crosses blocks leaves one
// partial row per block in the workspace, and a last kernel adds those in
// order.  Sums are fp32.  dW is dense: rows of tokens that do not occur are
// zero-filled (kept, when accumulating).
//
// Bound by the bytes of dout and dW: 65536 x 2048 fp32 over 100003 rows take
// 343 us (1356 MB, 4.0 TB/s; a copy reaches 4.8), 16384 x 768 bf16 over 50000
// rows 61 us, of which the sums are 14.
#include "naju_device.h"
#include "naju_host.h"
#include "naju_launch.h"
#include "naju_vec.h"

namespace naju {

// ---------------------------------------------------------------- forward
// One wave per (token, 256 accesses of 16 bytes): the token id is uniform over
// the wave, and its row moves as four 16-byte accesses per lane in flight.
// Bound by the bytes: the row is read and written once, and nothing else is
// (65536 x 768 bf16 26 us, 4.8 TB/s; 65536 x 2048 77 us).
template <typename IO>
__global__ __launch_bounds__(256) void embed_fwd_kernel(
    const int64_t T, const int64_t V, const int64_t d, const int32_t *__restrict__ ids,
    const IO *__restrict__ W, const float scale, IO *__restrict__ out)
{
    constexpr int n = kPer16<IO>;
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = ((int64_t)blockIdx.y * 256 + lane) * n;
    for (int64_t t = wave; t < T; t += (int64_t)gridDim.x * 4) {
        const int32_t id = ids[t];
        const bool there = id >= 0 && id < V;
        const IO *src = W + (there ? (int64_t)id : 0) * d;
        IO *dst = out + t * d;
        Run<IO, n> r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t c = c0 + (int64_t)q * 64 * n;
            if (!there || c >= d) r[q].zero();
            else if (c + n <= d) r[q].load(src + c);
            else r[q].load_part(src + c, (int)(d - c));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t c = c0 + (int64_t)q * 64 * n;
            if (c >= d) continue;
            float f[n];
#pragma unroll
            for (int i = 0; i < n; ++i) f[i] = scale * r[q].get(i);
            if (!there) {  // (0 * inf would not be 0)
#pragma unroll
                for (int i = 0; i < n; ++i) f[i] = 0.f;
            }
            const Run<IO, n> o = round_run<IO, n>(f);
            if (c + n <= d) o.store(dst + c);
            else o.store_part(dst + c, (int)(d - c));
        }
    }
}

// Rows of at most 32 accesses: 1 << lanes_log2 lanes a row, so that a wave takes
// several (65536 x 96 bf16: 17.2 us with a wave a row, 10.1 us so).
template <typename IO>
__global__ __launch_bounds__(256) void embed_fwd_short_kernel(
    const int64_t T, const int64_t V, const int d, const int lanes_log2,
    const int32_t *__restrict__ ids, const IO *__restrict__ W, const float scale,
    IO *__restrict__ out)
{
    constexpr int n = kPer16<IO>;
    const int c = (threadIdx.x & ((1 << lanes_log2) - 1)) * n;
    const int64_t rows = (int64_t)gridDim.x * (256 >> lanes_log2);
    for (int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lanes_log2; t < T; t += rows) {
        if (c >= d) continue;
        const int32_t id = ids[t];
        const bool there = id >= 0 && id < V;
        const IO *src = W + (there ? (int64_t)id : 0) * d + c;
        Run<IO, n> r;
        if (!there) r.zero();
        else if (c + n <= d) r.load(src);
        else r.load_part(src, d - c);
        float f[n];
#pragma unroll
        for (int i = 0; i < n; ++i) f[i] = there ? scale * r.get(i) : 0.f;
        const Run<IO, n> o = round_run<IO, n>(f);
        if (c + n <= d) o.store(out + t * d + c);
        else o.store_part(out + t * d + c, d - c);
    }
}

template <typename IO>
static hipError_t launch_embed_fwd(int64_t T, int64_t V, int64_t d, const int32_t *ids,
                                   const void *W, float scale, void *out, hipStream_t st)
{
    if (d <= 32 * kPer16<IO>) {
        int lg = 0;
        while ((1 << lg) * kPer16<IO> < d) ++lg;
        const int64_t blocks = (T + (256 >> lg) - 1) / (256 >> lg);
        hipLaunchKernelGGL(embed_fwd_short_kernel<IO>,
                           dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, T,
                           V, (int)d, lg, ids, (const IO *)W, scale, (IO *)out);
        return hipGetLastError();
    }
    const int64_t bx = (T + 3) / 4, by = (d + 256 * kPer16<IO> - 1) / (256 * kPer16<IO>);
    const dim3 grid((unsigned)(bx < 65536 ? bx : 65536), (unsigned)by);
    hipLaunchKernelGGL(embed_fwd_kernel<IO>, grid, dim3(256), 0, st, T, V, d, ids, (const IO *)W,
                       scale, (IO *)out);
    return hipGetLastError();
}

// ------------------------------------------------------------------- sort
// Stable least-significant-digit radix sort of (token, position), up to 9 bits
// a pass.  Tokens outside [0, V) get the key V: they end up last and are
// dropped there.  A pass is two kernels: every tile of 1024 ROUNDS keys counts its
// digits, then every tile ranks its keys (in its own order) behind the smaller
// digits of all tiles and the equal digits of the tiles before it.
constexpr int kDigits = 512;  // most values of a digit
// keys of a tile: 1024 while that leaves a tile few others to look at, else 4096 (sort and fill
// with tiles of 1024 and 4096: 16384 tokens, 50000 x 768 rows 38 and 43 us; 65536 tokens, 100003 x
// 2048 rows 148 and 146 us).  Every tile reads the counts of all, so the sort grows with the
// square of the tokens in the end: a pass takes 25 us at 2^18 tokens, 76 us at 2^20, 526 us at
// 2^22.
static int tile_rounds(int64_t T) { return T <= 16384 ? 1 : 4; }

__device__ __forceinline__ uint32_t key_of(const int32_t *ids, const uint32_t *keys, int64_t i,
                                           uint32_t V)
{
    if (keys) return keys[i];
    const uint32_t id = (uint32_t)ids[i];
    return id < V ? id : V;  // (a negative id is a large unsigned one)
}

// The zero fill of dW needs nothing from the sort, whose kernels leave most of
// the device idle: each launch of the sort carries workgroups that fill a slice.
// (16384 x 768 tokens over 50000 rows: 72 us with the fill in front of the
// sort, 61 us beside it; the fill alone is 21 us, the sort 27 us.)
struct Fill {
    float *p;       // null: nothing to fill
    int64_t n;      // floats of this launch's slice
    int blocks;     // workgroups that share it
};

__device__ __forceinline__ void fill_slice(const Fill &f, int block)
{
    const int64_t per = (f.n + f.blocks - 1) / f.blocks;
    const int64_t lo = per * block, hi = lo + per < f.n ? lo + per : f.n;
    Run<float, 4> z;
    z.zero();
    for (int64_t i = lo + threadIdx.x * 4; i < hi; i += blockDim.x * 4) {
        if (i + 4 <= hi) z.store(f.p + i);
        else z.store_part(f.p + i, (int)(hi - i));
    }
}

template <int ROUNDS>
__global__ __launch_bounds__(1024) void radix_count_kernel(
    const int64_t T, const uint32_t V, const int32_t *__restrict__ ids,
    const uint32_t *__restrict__ keys, const int shift, const int digits, const int n_tiles,
    uint32_t *__restrict__ counts, const Fill fill)
{
    __shared__ uint32_t hist[kDigits];
    const int tid = threadIdx.x;
    if ((int)blockIdx.x >= n_tiles) {
        fill_slice(fill, (int)blockIdx.x - n_tiles);
        return;
    }
    if (tid < kDigits) hist[tid] = 0u;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * (1024 * ROUNDS);
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
        const int64_t i = base + q * 1024 + tid;
        if (i < T) atomicAdd(&hist[(key_of(ids, keys, i, V) >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    if (tid < digits) counts[(int64_t)blockIdx.x * kDigits + tid] = hist[tid];
}

// Inclusive sum over the wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane)
{
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const uint32_t o = __shfl_up(v, s);
        if (lane >= s) v += o;
    }
    return v;
}

// Ranks 64 keys of equal digit in lane order: the lanes whose digit equals
// this lane's, as a mask.
__device__ __forceinline__ uint64_t same_digit(uint32_t dg, int bits, bool valid)
{
    uint64_t m = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((dg >> b) & 1u);
        m &= ((dg >> b) & 1u) ? one : ~one;
    }
    return m;
}

template <int ROUNDS>
__global__ __launch_bounds__(1024) void radix_scatter_kernel(
    const int64_t T, const uint32_t V, const int32_t *__restrict__ ids,
    const uint32_t *__restrict__ keys, const int32_t *__restrict__ pos, const int shift,
    const int bits, const int n_tiles, const uint32_t *__restrict__ counts,
    uint32_t *__restrict__ out_keys, int32_t *__restrict__ out_pos, const Fill fill)
{
    // cnt[w][digit]: the keys of wave w with this digit, then where its first one goes
    __shared__ uint32_t cnt[16][kDigits];
    __shared__ uint32_t wsum[16];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    if ((int)blockIdx.x >= n_tiles) {
        fill_slice(fill, (int)blockIdx.x - n_tiles);
        return;
    }
    const int digits = 1 << bits;
    for (int i = tid; i < 16 * kDigits; i += 1024) (&cnt[0][0])[i] = 0u;
    // digit tid: keys of the tiles before this one, and of all tiles
    uint32_t before = 0, total = 0;
    if (tid < digits) {
        for (int b = 0; b < n_tiles; ++b) {
            const uint32_t c = counts[(int64_t)b * kDigits + tid];
            before += b < (int)blockIdx.x ? c : 0u;
            total += c;
        }
    }
    const uint32_t incl = wave_scan(total, lane);
    if (lane == 63) wsum[w] = incl;
    __syncthreads();
    uint32_t start = incl - total + before;
    for (int i = 0; i < w; ++i) start += wsum[i];

    // each wave ranks its consecutive keys, 64 at a time
    const int64_t base = (int64_t)blockIdx.x * (1024 * ROUNDS) + w * (64 * ROUNDS);
    uint32_t key[ROUNDS], rank[ROUNDS];
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
        const int64_t i = base + q * 64 + lane;
        key[q] = i < T ? key_of(ids, keys, i, V) : 0u;
    }
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
        const bool valid = base + q * 64 + lane < T;
        const uint32_t dg = (key[q] >> shift) & (digits - 1);
        const uint64_t m = same_digit(dg, bits, valid);
        const uint32_t below = __popcll(m & ((1ull << lane) - 1));
        uint32_t c = 0;
        if (valid) c = cnt[w][dg];
        rank[q] = c + below;
        // (only this wave touches cnt[w]: its LDS accesses stay in program order,
        // every lane's read before the write, the write before the next round)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (valid && below == 0) cnt[w][dg] = c + (uint32_t)__popcll(m);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (tid < digits) {
        uint32_t at = start;
        for (int i = 0; i < 16; ++i) {
            const uint32_t c = cnt[i][tid];
            cnt[i][tid] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < ROUNDS; ++q) {
        const int64_t i = base + q * 64 + lane;
        if (i >= T) continue;
        const uint32_t dg = (key[q] >> shift) & (digits - 1);
        const uint32_t at = cnt[w][dg] + rank[q];
        out_keys[at] = key[q];
        out_pos[at] = pos ? pos[i] : (int32_t)i;
    }
}

// Up to kSmallTokens tokens: one workgroup sorts them in LDS, a word holding
// key << 12 | position, while the others fill.  One launch in place of two per
// digit.  (With four times the tokens the one CU takes 110 us; several tiles
// take 25.)
constexpr int kSmallTokens = 4096;
constexpr int64_t kSmallVocab = ((int64_t)1 << 20) - 1;  // keys 0 .. V in 20 bits

__global__ __launch_bounds__(1024) void small_sort_kernel(
    const int T, const uint32_t V, const int32_t *__restrict__ ids, const int passes,
    const int bits, uint32_t *__restrict__ out_keys, int32_t *__restrict__ out_pos,
    const Fill fill)
{
    __shared__ uint32_t buf[kSmallTokens];
    __shared__ uint32_t cnt[16][kDigits];
    __shared__ uint32_t wsum[16];
    constexpr int kMostRounds = kSmallTokens / 1024;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    if (blockIdx.x > 0) {
        fill_slice(fill, (int)blockIdx.x - 1);
        return;
    }
    // each wave holds `rounds` x 64 consecutive words
    const int rounds = (T + 1023) / 1024, base = w * rounds * 64 + lane;
    const uint32_t digits = 1u << bits;
    uint32_t word[kMostRounds], at[kMostRounds];
#pragma unroll
    for (int q = 0; q < kMostRounds; ++q) {
        const int i = base + q * 64;
        word[q] = 0;
        if (q < rounds && i < T) word[q] = key_of(ids, nullptr, i, V) << 12 | (uint32_t)i;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = 12 + p * bits;
        for (int i = tid; i < 16 * kDigits; i += 1024) (&cnt[0][0])[i] = 0u;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kMostRounds; ++q) {
            if (q < rounds) {
                const bool valid = base + q * 64 < T;
                const uint32_t dg = (word[q] >> shift) & (digits - 1);
                const uint64_t m = same_digit(dg, bits, valid);
                const uint32_t below = __popcll(m & ((1ull << lane) - 1));
                const uint32_t c = valid ? cnt[w][dg] : 0u;
                at[q] = c + below;
                // (only this wave touches cnt[w], as in radix_scatter_kernel)
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (valid && below == 0) cnt[w][dg] = c + (uint32_t)__popcll(m);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        }
        __syncthreads();
        // where each wave's first word of each digit goes
        uint32_t total = 0;
        if (tid < (int)digits)
            for (int i = 0; i < 16; ++i) total += cnt[i][tid];
        const uint32_t incl = wave_scan(total, lane);
        if (lane == 63) wsum[w] = incl;
        __syncthreads();
        if (tid < (int)digits) {
            uint32_t start = incl - total;
            for (int i = 0; i < w; ++i) start += wsum[i];
            for (int i = 0; i < 16; ++i) {
                const uint32_t c = cnt[i][tid];
                cnt[i][tid] = start;
                start += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kMostRounds; ++q) {
            if (q < rounds && base + q * 64 < T)
                buf[cnt[w][(word[q] >> shift) & (digits - 1)] + at[q]] = word[q];
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kMostRounds; ++q) {
            const int i = base + q * 64;
            if (q < rounds && i < T) word[q] = buf[i];
        }
    }
#pragma unroll
    for (int q = 0; q < kMostRounds; ++q) {
        const int i = base + q * 64;
        if (q < rounds && i < T) {
            out_keys[i] = word[q] >> 12;
            out_pos[i] = (int32_t)(word[q] & 4095u);
        }
    }
}

// -------------------------------------------------------------- gradient
constexpr int kSeg = 16;             // sorted positions of a wave
constexpr int kSumWaves = 8;
constexpr int kBlk = kSeg * kSumWaves;
constexpr int kCols = 256;           // columns of a workgroup: 4 per lane

__device__ __forceinline__ void add4(float (&a)[4], const float4 v)
{
    a[0] += v.x;
    a[1] += v.y;
    a[2] += v.z;
    a[3] += v.w;
}

// dW[key][col..] = (or +=) scale * acc, nc of 4 columns
template <bool ACC>
__device__ __forceinline__ void write_row(float *dW, int64_t key, int64_t d, int64_t col, int nc,
                                          float scale, const float (&acc)[4])
{
    if (nc <= 0) return;
    float *p = dW + key * d + col;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = scale * acc[i];
    Run<float, 4> r;
    if (ACC) {
        if (nc == 4) r.load(p);
        else r.load_part(p, nc);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] += r.get(i);
    }
    r = round_run<float, 4>(f);
    if (nc == 4) r.store(p);
    else r.store_part(p, nc);
}

// One workgroup sums the runs of kBlk sorted positions over kCols columns;
// wave w takes kSeg of them.  All row loads of a wave are issued before the
// first is used.  The keys are uniform over the wave.  (Waves side by side over
// 1024 columns of fewer positions read no faster, and left more partial rows.)
template <typename IO, bool ACC>
__global__ __launch_bounds__(64 * kSumWaves) void embed_sum_kernel(
    const int64_t T, const int64_t V, const int64_t d, const int64_t first, const uint32_t n_cols,
    const uint32_t *__restrict__ skey, const int32_t *__restrict__ spos,
    const IO *__restrict__ dout, const float scale, float *__restrict__ dW,
    float *__restrict__ part)
{
    __shared__ float4 head[kSumWaves][64], tail[kSumWaves][64];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // (the column tiles of a block run next to each other: whole rows are read at a time)
    const int64_t ib = first + blockIdx.x / n_cols;
    const uint32_t ic = blockIdx.x % n_cols;
    const int64_t blk = ib * kBlk, base = blk + w * kSeg;
    const int64_t col = (int64_t)ic * kCols + lane * 4;
    const int nc = d - col >= 4 ? 4 : d > col ? (int)(d - col) : 0;
    const int n = T - base >= kSeg ? kSeg : T > base ? (int)(T - base) : 0;

    Run<IO, 4> v[kSeg];
    uint32_t key[kSeg];
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
        v[i].zero();
        key[i] = (uint32_t)V;
        if (i < n) {
            key[i] = skey[base + i];
            const IO *p = dout + (int64_t)spos[base + i] * d + col;
            if (key[i] < V) {
                if (nc == 4) v[i].load(p);
                else v[i].load_part(p, nc);
            }
        }
    }
    const uint32_t prev = n > 0 && base > 0 ? skey[base - 1] : (uint32_t)V;
    const uint32_t next = n > 0 && base + n < T ? skey[base + n] : (uint32_t)V;

    // acc: the current run; at its end it is written, or parked for the
    // neighbours: `head` if it began before this wave's positions, `tail` if it
    // begins here and goes on after them
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    bool from_before = n > 0 && prev == key[0];
    bool has_tail = false;
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
        if (i >= n || key[i] >= V) continue;  // (dropped tokens are sorted last)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] += v[i].get(q);
        const bool last = i == n - 1;
        const uint32_t after = last ? next : key[i < kSeg - 1 ? i + 1 : i];
        if (last || after != key[i]) {
            const bool goes_on = after == key[i];
            if (from_before) {
                head[w][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            } else if (goes_on) {
                tail[w][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                has_tail = true;
            } else {
                write_row<ACC>(dW, key[i], d, col, nc, scale, acc);
            }
            from_before = false;
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = 0.f;
        }
    }
    __syncthreads();

    // a run that begins in this wave and goes on, or (first waves) the one that
    // began before this block: add the later waves' heads in order
    const int64_t slot = ib * 2;
    if (has_tail) {
        const uint32_t k = skey[base + n - 1];
        const float4 t = tail[w][lane];
        float s[4] = {t.x, t.y, t.z, t.w};
        int j = w + 1;
        for (; j < kSumWaves && blk + j * kSeg < T && skey[blk + j * kSeg] == k; ++j)
            add4(s, head[j][lane]);
        if (j == kSumWaves && blk + kBlk < T && skey[blk + kBlk] == k) {
            if (nc > 0) {
                Run<float, 4> r = round_run<float, 4>(s);
                float *p = part + (slot + 1) * d + col;
                if (nc == 4) r.store(p);
                else r.store_part(p, nc);
            }
        } else {
            write_row<ACC>(dW, k, d, col, nc, scale, s);
        }
    }
    if (w == 0 && n > 0 && prev == key[0] && key[0] < V) {
        const uint32_t k = key[0];
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < kSumWaves && blk + j * kSeg < T && skey[blk + j * kSeg] == k; ++j)
            add4(s, head[j][lane]);
        if (nc > 0) {
            Run<float, 4> r = round_run<float, 4>(s);
            float *p = part + slot * d + col;
            if (nc == 4) r.store(p);
            else r.store_part(p, nc);
        }
    }
}

// A run that begins in block i and goes on into block i + 1: its partial row
// there plus the first partial rows of the blocks that it covers or ends in.
// The waves take every eighth of them; their sums are added in wave order.
template <bool ACC>
__global__ __launch_bounds__(512) void embed_join_kernel(
    const int64_t T, const int64_t V, const int64_t d, const int64_t first,
    const uint32_t n_cols, const uint32_t *__restrict__ skey, const float scale, const float *__restrict__ part,
    float *__restrict__ dW)
{
    __shared__ float4 sum[8][64];
    const int64_t ib = first + blockIdx.x / n_cols;
    const uint32_t ic = blockIdx.x % n_cols;
    const int64_t blk = ib * kBlk, end = blk + kBlk;
    const uint32_t k = skey[end - 1];  // (the grid has no last block: end < T)
    if (k >= V || skey[end] != k || (blk > 0 && skey[blk - 1] == k)) return;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t col = (int64_t)ic * kCols + lane * 4;
    const int nc = d - col >= 4 ? 4 : d > col ? (int)(d - col) : 0;
    // blocks whose first key is still k: (ib, hi]
    int64_t lo = ib + 1, hi = (T - 1) / kBlk;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (skey[mid * kBlk] == k) lo = mid;
        else hi = mid - 1;
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (nc > 0) {
        for (int64_t j = ib + 1 + w; j <= hi; j += 8 * 4) {
            Run<float, 4> r[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                r[q].zero();
                if (j + 8 * q <= hi) {
                    const float *p = part + (j + 8 * q) * 2 * d + col;
                    if (nc == 4) r[q].load(p);
                    else r[q].load_part(p, nc);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] += r[q].get(i);
        }
    }
    sum[w][lane] = make_float4(s[0], s[1], s[2], s[3]);
    __syncthreads();
    if (w != 0 || nc <= 0) return;
    Run<float, 4> r;
    const float *p = part + (ib * 2 + 1) * d + col;
    if (nc == 4) r.load(p);
    else r.load_part(p, nc);
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = r.get(i);
    for (int j = 0; j < 8; ++j) add4(a, sum[j][lane]);
    write_row<ACC>(dW, k, d, col, nc, scale, a);
}

struct EmbedPlan {
    int passes, bits;   // radix passes and digit width
    int n_tiles;        // sort tiles
    int64_t n_blk;      // blocks of kBlk sorted positions
    size_t off_keys[2], off_pos[2], off_counts, off_part, bytes;
};

static EmbedPlan embed_plan(int64_t T, int64_t V, int64_t d)
{
    EmbedPlan p{};
    int bits = 1;
    while (((uint64_t)V >> bits) != 0) ++bits;  // keys 0 .. V (at least one digit)
    p.passes = (bits + 8) / 9;
    p.bits = (bits + p.passes - 1) / p.passes;
    const int64_t tile = 1024 * tile_rounds(T);
    p.n_tiles = (int)((T + tile - 1) / tile);
    p.n_blk = (T + kBlk - 1) / kBlk;
    size_t at = 256;
    for (int i = 0; i < 2; ++i) {
        p.off_keys[i] = at;
        at = align256(at + 4 * (size_t)T);
        p.off_pos[i] = at;
        at = align256(at + 4 * (size_t)T);
    }
    p.off_counts = at;
    at = align256(at + 4 * (size_t)kDigits * (size_t)p.n_tiles);
    p.off_part = at;
    p.bytes = align256(at + (p.n_blk > 1 ? 2 * 4 * (size_t)p.n_blk * (size_t)d : 0));
    return p;
}

template <typename IO, bool ACC>
static hipError_t launch_embed_sum(const EmbedPlan &pl, int64_t T, int64_t V, int64_t d,
                                   const uint32_t *skey, const int32_t *spos, const void *dout,
                                   float scale, float *dW, float *part, hipStream_t st)
{
    const int64_t cols = (d + kCols - 1) / kCols;
    const int64_t most = ((int64_t)1 << 22) / cols;  // blocks of a launch
    for (int64_t i = 0; i < pl.n_blk; i += most) {
        const int64_t n = pl.n_blk - i < most ? pl.n_blk - i : most;
        hipLaunchKernelGGL((embed_sum_kernel<IO, ACC>), dim3((unsigned)(n * cols)),
                           dim3(64 * kSumWaves), 0, st, T, V, d, i, (uint32_t)cols, skey, spos,
                           (const IO *)dout, scale, dW, part);
    }
    for (int64_t i = 0; i < pl.n_blk - 1; i += most) {
        const int64_t n = pl.n_blk - 1 - i < most ? pl.n_blk - 1 - i : most;
        hipLaunchKernelGGL(embed_join_kernel<ACC>, dim3((unsigned)(n * cols)), dim3(512), 0, st, T,
                           V, d, i, (uint32_t)cols, skey, scale, part, dW);
    }
    return hipGetLastError();
}

static hipError_t launch_embed_bwd(int64_t T, int64_t V, int64_t d, int io, const int32_t *ids,
                                   const void *dout, float scale, bool acc, float *dW, char *ws,
                                   hipStream_t st)
{
    if (T == 0) return launch_zero(dW, (size_t)V * (size_t)d * 4, st);
    const EmbedPlan pl = embed_plan(T, V, d);
    uint32_t *keys[2] = {(uint32_t *)(ws + pl.off_keys[0]), (uint32_t *)(ws + pl.off_keys[1])};
    int32_t *pos[2] = {(int32_t *)(ws + pl.off_pos[0]), (int32_t *)(ws + pl.off_pos[1])};
    uint32_t *counts = (uint32_t *)(ws + pl.off_counts);
    const uint32_t *ik = nullptr;
    const int32_t *ip = nullptr;
    // slices of the fill: all of it beside the small sort; else as the launches last, a count
    // about a third of a scatter
    const bool small = T <= kSmallTokens && V <= kSmallVocab;
    const int64_t all = acc ? 0 : V * d;
    const int units = small ? 1 : 4 * pl.passes;
    int64_t filled = 0;
    int done = 0;
    auto slice = [&](int weight) {
        done += weight;
        const int64_t to = done == units ? all : all / units * done;
        Fill f{dW + filled, to - filled, 0};
        const int64_t blocks = (f.n + 16383) / 16384;
        f.blocks = (int)(blocks < 4096 ? blocks : 4096);
        filled = to;
        return f;
    };
    if (small) {
        const Fill f = slice(1);
        hipLaunchKernelGGL(small_sort_kernel, dim3(1 + f.blocks), dim3(1024), 0, st, (int)T,
                           (uint32_t)V, ids, pl.passes, pl.bits, keys[0], pos[0], f);
        ik = keys[0];
        ip = pos[0];
    }
    for (int q = 0; !small && q < pl.passes; ++q) {
        const Fill f1 = slice(1), f2 = slice(3);
        const bool one = tile_rounds(T) == 1;
        hipLaunchKernelGGL(one ? radix_count_kernel<1> : radix_count_kernel<4>,
                           dim3(pl.n_tiles + f1.blocks), dim3(1024), 0, st, T, (uint32_t)V, ids,
                           ik, q * pl.bits, 1 << pl.bits, pl.n_tiles, counts, f1);
        hipLaunchKernelGGL(one ? radix_scatter_kernel<1> : radix_scatter_kernel<4>,
                           dim3(pl.n_tiles + f2.blocks), dim3(1024), 0, st, T, (uint32_t)V, ids,
                           ik, ip, q * pl.bits, pl.bits, pl.n_tiles, counts, keys[q & 1],
                           pos[q & 1], f2);
        ik = keys[q & 1];
        ip = pos[q & 1];
    }
    float *part = (float *)(ws + pl.off_part);
    if (io == NAJU_F32)
        return acc ? launch_embed_sum<float, true>(pl, T, V, d, ik, ip, dout, scale, dW, part, st)
                   : launch_embed_sum<float, false>(pl, T, V, d, ik, ip, dout, scale, dW, part, st);
    return acc ? launch_embed_sum<bf16, true>(pl, T, V, d, ik, ip, dout, scale, dW, part, st)
               : launch_embed_sum<bf16, false>(pl, T, V, d, ik, ip, dout, scale, dW, part, st);
}

static naju_status_t check_embed(int64_t T, int64_t V, int64_t d, int32_t io)
{
    if (T < 0 || V < 0 || d < 0)
        return fail(NAJU_EINVAL, "negative size (tokens=%lld vocab=%lld d_model=%lld)",
                    (long long)T, (long long)V, (long long)d);
    if (io != NAJU_F32 && io != NAJU_BF16)
        return fail(NAJU_EINVAL, "io dtype %d is neither NAJU_F32 nor NAJU_BF16", (int)io);
    // positions and tokens are 32-bit in the sort, and the grids stay below 2^32 threads
    if (T > ((int64_t)1 << 28) || V > ((int64_t)1 << 30) || d > ((int64_t)1 << 20))
        return fail(NAJU_EINVAL, "tokens (2^28 max), vocab (2^30 max) or d_model (2^20 max) "
                                 "too large");
    return NAJU_OK;
}

}  // namespace naju

using namespace naju;

extern "C" {

naju_status_t naju_embed_fwd(int64_t tokens, int64_t vocab, int64_t d_model, int32_t io,
                             const int32_t *ids, const void *W, float scale, void *out,
                             void *stream)
{
    NAJU_TRY(check_embed(tokens, vocab, d_model, io));
    if (tokens == 0 || d_model == 0) return NAJU_OK;
    const size_t e = io == NAJU_F32 ? 4 : 2;
    NAJU_TRY(need(ids, "ids", 4));
    if (vocab > 0) NAJU_TRY(need(W, "W", e));
    NAJU_TRY(need(out, "out", e));
    hipStream_t st = (hipStream_t)stream;
    return hip_status(
        io == NAJU_F32 ? launch_embed_fwd<float>(tokens, vocab, d_model, ids, W, scale, out, st)
                       : launch_embed_fwd<bf16>(tokens, vocab, d_model, ids, W, scale, out, st),
        "embedding launch");
}

size_t naju_embed_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t d_model)
{
    if (check_embed(tokens, vocab, d_model, NAJU_F32) != NAJU_OK) return 0;
    return embed_plan(tokens, vocab, d_model).bytes;
}

naju_status_t naju_embed_bwd(int64_t tokens, int64_t vocab, int64_t d_model, int32_t io,
                             const int32_t *ids, const void *dout, float scale,
                             int32_t accumulate, float *dW, void *ws, size_t ws_bytes,
                             void *stream)
{
    NAJU_TRY(check_embed(tokens, vocab, d_model, io));
    if (vocab == 0 || d_model == 0) return NAJU_OK;
    NAJU_TRY(need(dW, "dW", 4));
    if (tokens > 0) {
        NAJU_TRY(need(ids, "ids", 4));
        NAJU_TRY(need(dout, "dout", io == NAJU_F32 ? 4 : 2));
        NAJU_TRY(need_ws(ws, ws_bytes, embed_plan(tokens, vocab, d_model).bytes));
    } else if (accumulate) {
        return NAJU_OK;
    }
    return hip_status(launch_embed_bwd(tokens, vocab, d_model, io, ids, dout, scale,
                                       accumulate != 0, dW, (char *)ws, (hipStream_t)stream),
                      "embedding gradient launch");
}

}  // extern "C"
