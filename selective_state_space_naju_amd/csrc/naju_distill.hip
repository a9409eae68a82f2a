// naju_distill.hip -- distillation of a student's logits from a teacher's top
// logits: the loss of each row, its gradient, or both in one call.
//
// With temperature tau, student logits s_v, teacher entries (i_j, t_j):
//     x_v = s_v / tau,  lse = log sum_v exp x_v,  q_v = exp(x_v - lse)
//     p = softmax over the valid entries of t_j / tau
//     loss = tau^2 sum_j p_j (log p_j - (x_{i_j} - lse))
//     dloss/ds_v = tau ([any valid] q_v - sum_{j : i_j = v} p_j)
// An entry is valid when its index lies in [0, V) and t_j is not -inf.  One
// entry and tau = 1 make the loss the cross entropy of a hard label.
//
// The rows are long (tens of thousands of logits) and the entries few, so a
// workgroup takes a row, streams it with 16-byte accesses and keeps one entry
// per thread; statistics and sums are fp32, each rounded once on output.
//
// Bound by the bytes of the logits.  16384 x 32000 bf16, kernel times: loss 179 us
// (5.9 TB/s of reads), gradient 413 us, both in one call 426 us (4.9 TB/s; a large
// copy reaches 4.8).
#include <math.h>

#include "naju_device.h"
#include "naju_host.h"
#include "naju_launch.h"
#include "naju_vec.h"

namespace naju {

constexpr int kMostEntries = 512;  // entries of a row: one per thread of a large workgroup
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.6931471805599453f;

// Maximum of some logits, and the sum of exp((. - maximum) / tau) over them.
// The maximum is kept as it was read and taken off before the difference is
// scaled: scaled by itself, a logit near the type's lowest or largest value
// would leave fp32's range.  c2 = log2(e) / tau.  The maximum passes NaN over, the
// sum does not: a row of -inf alone is the one whose sum is 0, and a row with NaN
// has the sum NaN, whatever its maximum.
struct MaxSum {
    float m, s;
};

__device__ __forceinline__ float exp_nat(float d) { return ex2(d * kLog2e); }
// what is taken off where there is no value above -inf is 0, not -inf
__device__ __forceinline__ float base_of(float m) { return m == kNegInf ? 0.f : m; }

__device__ __forceinline__ MaxSum wave_maxsum(MaxSum a, float c2)
{
    float M = a.m;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
    float s = a.s * ex2((a.m - base_of(M)) * c2);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    return {M, s};
}

template <int kWaves> __device__ __forceinline__ MaxSum join_maxsum(const MaxSum *w, float c2)
{
    float M = w[0].m;
#pragma unroll
    for (int i = 1; i < kWaves; ++i) M = fmaxf(M, w[i].m);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) s += w[i].s * ex2((w[i].m - base_of(M)) * c2);
    return {M, s};
}

// One teacher entry per thread.
struct Entry {
    int id;      // -1: not valid
    float t;     // -inf if not valid
};

__device__ __forceinline__ Entry load_entry(const int32_t *t_ids, const float *t_logits, int k,
                                            int64_t V)
{
    Entry e{-1, kNegInf};
    if ((int)threadIdx.x < k) {
        const int id = t_ids[threadIdx.x];
        if (id >= 0 && id < V) {
            // (kept behind the id: with both asked for at once the rows' loads of a CU's workgroups
            // fall together, 16384 x 32000 bf16 loss and gradient 437 us in place of 430)
            asm volatile("");
            const float t = t_logits[threadIdx.x];
            if (t != kNegInf) {
                e.id = id;
                e.t = t;
            }
        }
    }
    return e;
}
__device__ __forceinline__ MaxSum entry_maxsum(const Entry &e, float c2)
{
    // (1, or NaN for an infinite or NaN entry)
    return wave_maxsum({e.t, e.id >= 0 ? ex2((e.t - base_of(e.t)) * c2) : 0.f}, c2);
}

// elements between p and the 16-byte boundary before it
template <typename IO> __device__ __forceinline__ int past_boundary(const IO *p)
{
    return (int)((uintptr_t)p % 16 / sizeof(IO));
}

template <typename IO> __device__ __forceinline__ IO neg_inf_raw();
template <> __device__ __forceinline__ float neg_inf_raw<float>() { return kNegInf; }
template <> __device__ __forceinline__ bf16 neg_inf_raw<bf16>() { return 0xff80; }

// ------------------------------------------------------------------ loss
// Reads the row once, kLossRuns accesses per thread in flight, with a running
// maximum and sum per thread.  Accesses start at a 16-byte boundary; one that
// would leave the row is moved inside it, and what it holds of its neighbours is
// taken for -inf.
constexpr int kLossRuns = 4;

template <typename IO, int BS>
__global__ __launch_bounds__(BS) void distill_loss_kernel(
    const int64_t R, const int64_t V, const int k, const IO *__restrict__ logits,
    const int64_t ld, const int32_t *__restrict__ t_ids, const float *__restrict__ t_logits,
    const float tau, const float inv_tau, float *__restrict__ loss, float *__restrict__ lse)
{
    constexpr int n = kPer16<IO>;
    constexpr int per = BS * n * kLossRuns;
    __shared__ MaxSum row_ms[BS / 64], ent_ms[BS / 64];
    __shared__ float sum[BS / 64];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const float c2 = inv_tau * kLog2e;
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const IO *row = logits + r * ld;
        const Entry e = load_entry(t_ids + r * k, t_logits + r * k, k, V);
        const float at = e.id >= 0 ? to_f(row[e.id]) : 0.f;
        float m = kNegInf, s = 0.f;
        if (V >= n) {
            for (int64_t c0 = -past_boundary(row); c0 < V; c0 += per) {
                Run<IO, n> v[kLossRuns];
#pragma unroll
                for (int i = 0; i < kLossRuns; ++i) {
                    const int64_t c = c0 + (i * BS + tid) * n;
                    v[i].load(row + (c < 0 ? 0 : c > V - n ? V - n : c));
                }
#pragma unroll
                for (int i = 0; i < kLossRuns; ++i) {
                    if ((i == 0 && c0 < 0) || c0 + (i + 1) * (BS * n) > V) {  // (uniform)
                        const int64_t c = c0 + (i * BS + tid) * n;
                        const int64_t in = c < 0 ? 0 : c > V - n ? V - n : c;
#pragma unroll
                        for (int j = 0; j < n; ++j)
                            if (in + j < c || in + j >= c + n) v[i].set_raw(j, neg_inf_raw<IO>());
                    }
                }
                float top = m;
#pragma unroll
                for (int i = 0; i < kLossRuns; ++i) {
                    if (c0 + i * (BS * n) < V) {
#pragma unroll
                        for (int j = 0; j < n; ++j) top = fmaxf(top, v[i].get(j));
                    }
                }
                const float b = base_of(top);
                s *= ex2((m - b) * c2);
                m = top;
#pragma unroll
                for (int i = 0; i < kLossRuns; ++i) {
                    if (c0 + i * (BS * n) < V) {
                        v[i].repack();
#pragma unroll
                        for (int j = 0; j < n; ++j) s += ex2((v[i].get(j) - b) * c2);
                    }
                }
            }
        } else if (tid < V) {  // (shorter than an access)
            m = to_f(row[tid]);
            s = m == kNegInf ? 0.f : fabsf(m) < -kNegInf ? 1.f : __builtin_nanf("");
        }
        const MaxSum rs = wave_maxsum({m, s}, c2);
        const MaxSum es = entry_maxsum(e, c2);
        if (lane == 0) {
            row_ms[w] = rs;
            ent_ms[w] = es;
        }
        __syncthreads();
        const MaxSum ts = join_maxsum<BS / 64>(ent_ms, c2), row_s = join_maxsum<BS / 64>(row_ms, c2);
        const float b = base_of(row_s.m), log2_s = log2f(row_s.s);
        float term = 0.f;
        if (e.id >= 0) {
            const float gap = (e.t - base_of(ts.m)) * c2;  // (in base 2, as log2 q)
            const float p = ex2(gap) / ts.s;
            const float log2_q =
                at == kNegInf && log2_s == log2_s ? kNegInf : (at - b) * c2 - log2_s;
            // 0 log 0 = 0; NaN goes on
            if (!(p == 0.f)) term = p * (((gap - log2f(ts.s)) - log2_q) * kLn2);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) term += __shfl_xor(term, o);
        if (lane == 0) sum[w] = term;
        __syncthreads();
        if (tid == 0) {
            float t = 0.f;
            for (int i = 0; i < BS / 64; ++i) t += sum[i];
            loss[r] = tau * tau * t;
            lse[r] = fmaf(b, inv_tau, log2_s * kLn2);
        }
        // (the next row writes row_ms and ent_ms: every thread has read them by now)
    }
}

// -------------------------------------------------------------- gradient
// A workgroup takes NV accesses per thread of one row, all loads issued before
// the first is used.  The dense part g tau q_v is stored first; then the
// elements that the entries name are written again with their share of p, by
// the first entry that names each.  The accesses are laid out from a 16-byte
// boundary of the gradient's row at or before its start (rows of an odd
// vocabulary start anywhere).
//
// q_v is exp(x_v - lse), with the rounding of lse in it: |lse| 2^-24 relative,
// up to kFineLse a quarter of a bf16 rounding.  A row beyond it (logits near the
// type's lowest or largest value have no usable lse at all) has its maximum and
// sum formed again, by every workgroup of the row.
constexpr float kFineLse = 16384.f;

template <typename IO, int NV, int BS>
__global__ __launch_bounds__(BS, 6) void distill_grad_kernel(
    const int64_t V, const int k, const int n_chunks, const IO *__restrict__ logits,
    const int64_t ld, const int32_t *__restrict__ t_ids, const float *__restrict__ t_logits,
    const float tau, const float inv_tau, const float *__restrict__ lse,
    const float *__restrict__ g, IO *__restrict__ dlogits, const int64_t ldd)
{
    constexpr int n = kPer16<IO>;
    constexpr int chunk = BS * n * NV;
    __shared__ MaxSum row_ms[BS / 64], ent_ms[BS / 64];
    __shared__ int ids[BS];
    __shared__ float ps[BS];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const float c2 = inv_tau * kLog2e;
    const int64_t r = blockIdx.x / (unsigned)n_chunks;
    const int part = (int)(blockIdx.x - (unsigned)r * (unsigned)n_chunks);
    const IO *row = logits + r * ld;
    IO *out = dlogits + r * ldd;
    // this chunk: elements [c0, c0 + chunk) of the row, c0 on a boundary; the last chunk also
    // takes the few that the shift pushes past it
    const int64_t c0 = (int64_t)part * chunk - past_boundary(out);
    const bool is_last = part == n_chunks - 1;
    const int64_t lo = c0 > 0 ? c0 : 0, hi = is_last ? V : c0 + chunk;
    const Entry e = load_entry(t_ids + r * k, t_logits + r * k, k, V);
    const float L = lse[r], gr = g[r];
    Run<IO, n> v[NV];
    if (V >= n) {
        const IO *at_c0 = row + c0;  // (the accesses are moved into the row)
        const int least = c0 < 0 ? (int)-c0 : 0;
        const int most = V - n - c0 < chunk ? (int)(V - n - c0) : chunk;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * BS + tid) * n;
            const int in = c < least ? least : c > most ? most : c;
            v[i].load(at_c0 + in);
        }
    }
    const bool mine = e.id >= lo && e.id < hi;
    const float at = mine ? to_f(row[e.id]) : 0.f;
    const MaxSum es = entry_maxsum(e, c2);
    if (lane == 0) ent_ms[w] = es;
    __syncthreads();
    const MaxSum ts = join_maxsum<BS / 64>(ent_ms, c2);
    // no valid entry: no loss to descend; weight 0: a row that does not count
    const bool some = !(ts.s == 0.f) && gr != 0.f;  // (a list of NaN has the sum NaN)
    const float f = some ? gr * tau : 0.f;
    ids[tid] = e.id;
    ps[tid] = e.id >= 0 ? ex2((e.t - base_of(ts.m)) * c2) / ts.s : 0.f;
    float dense_at;  // the dense part at this thread's entry
    if (fabsf(L) <= kFineLse || L != L || !some) {
        auto dense = [&](float x) { return f * exp_nat(fmaf(x, inv_tau, -L)); };
        if (V >= n) {
            IO *out_c0 = out + c0;
            const int64_t left = V - c0;  // elements from c0 to the row's end
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * BS + tid) * n;
                float d[n];
#pragma unroll
                for (int j = 0; j < n; ++j) d[j] = dense(v[i].get(j));
                Run<IO, n> o = round_run<IO, n>(d);
                if (!some) o.zero();
                if (c0 + c >= 0 && c + n <= left) {
                    o.store(out_c0 + c);
                } else if (c0 + c > -n && c < left) {
                    // the row's first or last access, moved inside it: its own elements
                    const int in = c0 + c < 0 ? (int)-c0 : (int)(left - n);
#pragma unroll
                    for (int j = 0; j < n; ++j)
                        if (in + j >= c && in + j < c + n) out_c0[in + j] = o.get_raw(j);
                }
            }
            const int64_t rest = c0 + chunk + tid;
            if (is_last && tid < n && rest < V) {
                const float d = dense(to_f(row[rest]));
                out[rest] = from_f<IO>(some ? d : 0.f);
            }
        } else if (tid < V) {  // (shorter than an access)
            const float d = dense(to_f(row[tid]));
            out[tid] = from_f<IO>(some ? d : 0.f);
        }
        dense_at = dense(at);
    } else {  // (uniform)
        MaxSum rs{kNegInf, 0.f};
#pragma unroll 1
        for (uint32_t c = tid; c < (uint32_t)V; c += BS) rs.m = fmaxf(rs.m, to_f(row[c]));
#pragma unroll 1
        for (uint32_t c = tid; c < (uint32_t)V; c += BS) rs.s += ex2((to_f(row[c]) - base_of(rs.m)) * c2);
        rs = wave_maxsum(rs, c2);
        if (lane == 0) row_ms[w] = rs;
        __syncthreads();
        rs = join_maxsum<BS / 64>(row_ms, c2);
        const float base = base_of(rs.m), fq = rs.s == 0.f ? 0.f : f / rs.s;
        auto dense = [&](float x) { return fq * ex2((x - base) * c2); };
#pragma unroll 1
        for (uint32_t c = (uint32_t)lo + tid; c < (uint32_t)hi; c += BS) {
            const float d = dense(to_f(row[c]));
            out[c] = from_f<IO>(some ? d : 0.f);
        }
        dense_at = dense(at);
    }
    // the dense stores are done before an element is written again
    wait_mem();
    __syncthreads();
    if (some && mine) {
        float p = 0.f;
        bool first = true;
        for (int j = 0; j < k; ++j)
            if (ids[j] == e.id) {
                first = first && j >= tid;
                p += ps[j];
            }
        if (first) out[e.id] = from_f<IO>(dense_at - f * p);
    }
}

// ------------------------------------------------- loss and gradient at once
// The row stays in registers between its statistics and its gradient, NV
// accesses per thread: every logit is read once and every gradient written
// once.  Exponents are formed with the maximum of the wave, so one barrier joins
// the row's and the list's statistics; q is exp((s - m) / tau) over the row's
// sum, with no rounded lse in between.  Places past the row hold -inf, which
// adds nothing.
//
// (s - m) c2 is formed as one multiply-add, s c - b with b = m c rounded; what
// that rounding took, m c - b, is the same for every logit and comes off the sum.
// (Subtracted first, an operation more per logit, 8192 x 50001 bf16 takes 3 %
// longer.)  c is c2 unless m c2 would pass 2^30, or fp32's range: there it
// is made smaller.  Numbers of that size lie 64 or more apart in units of 1 / c,
// so either way all but the largest weigh nothing, and b's rounding, up to 64,
// leaves the exponential in range.
struct Exponent {
    float m, c, b, rest;
    __device__ __forceinline__ Exponent(float max, float c2)
        : m(base_of(max)), c(fabsf(m) * c2 <= 0x1p30f ? c2 : 0x1p30f / fabsf(m)), b(m * c),
          rest(fmaf(m, c, -b))
    {
    }
    __device__ __forceinline__ float operator()(float s) const { return fmaf(s, c, -b); }
};

// The waves per SIMD that the launch bounds ask for keep the row's packed words
// (4 NV registers) and little else live, so that several workgroups share a CU
// and one loads while another computes.
template <typename IO, int NV, int BS>
__global__ __launch_bounds__(BS, NV <= 8 ? 6 : NV <= 16 ? 4 : 2) void distill_step_kernel(
    const uint32_t V, const int k, const IO *__restrict__ logits, const int64_t ld,
    const int32_t *__restrict__ t_ids, const float *__restrict__ t_logits, const float tau,
    const float inv_tau, const float *__restrict__ g, float *__restrict__ loss,
    float *__restrict__ lse, IO *__restrict__ dlogits, const int64_t ldd)
{
    constexpr int n = kPer16<IO>;
    constexpr uint32_t per = BS * n;
    __shared__ MaxSum row_ms[BS / 64], ent_ms[BS / 64];
    __shared__ float sum[BS / 64];
    __shared__ int ids[BS];
    __shared__ float ps[BS];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const float c2 = inv_tau * kLog2e;
    const int64_t r = blockIdx.x;
    const IO *row = logits + r * ld;
    IO *out = dlogits + r * ldd;
    const Entry e = load_entry(t_ids + r * k, t_logits + r * k, k, V);
    const float gr = g[r];
    // accesses from the 16-byte boundary `before` elements ahead of the gradient's row, moved
    // into the row at its ends: no load waits on a branch
    const int before = past_boundary(out), last = (int)V - n;
    const int c0 = tid * n - before;
    Run<IO, n> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * (int)per + c0;
        const int in = c < 0 ? 0 : c < last ? c : last;
        v[i].load_at(row, (uint32_t)in * (uint32_t)sizeof(IO));
    }
    const float at = e.id >= 0 ? to_f(row[e.id]) : 0.f;
    const MaxSum es = entry_maxsum(e, c2);
    // what a moved access holds of its neighbours is taken for -inf
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((i == 0 && before > 0) || (i + 1) * per > V + before) {  // (uniform)
            const int c = i * (int)per + c0;
            const int in = c < 0 ? 0 : c < last ? c : last;
#pragma unroll
            for (int j = 0; j < n; ++j)
                if (in + j < c || in + j >= c + n) v[i].set_raw(j, neg_inf_raw<IO>());
        }
    }
    // maximum of the wave, sum of exp((. - maximum) / tau)
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i * per < V + before) {
#pragma unroll
            for (int j = 0; j < n; ++j) top = fmaxf(top, v[i].get(j));
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const Exponent xw(top, c2);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i * per < V + before) {
            v[i].repack();
#pragma unroll
            for (int j = 0; j < n; ++j) s += ex2(xw(v[i].get(j)));
            v[i].repack();
        }
    }
    s *= ex2(-xw.rest);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) {
        row_ms[w] = {top, s};
        ent_ms[w] = es;
    }
    __syncthreads();
    const MaxSum ts = join_maxsum<BS / 64>(ent_ms, c2), row_s = join_maxsum<BS / 64>(row_ms, c2);
    const Exponent xr(row_s.m, c2);
    // the entries: their probabilities and their terms of the loss
    const float log2_s = log2f(row_s.s), log2_t = log2f(ts.s);
    float p = 0.f, term = 0.f;
    if (e.id >= 0) {
        const float gap = (e.t - base_of(ts.m)) * c2;  // (in base 2, as log2 q)
        p = ex2(gap) / ts.s;
        const float log2_q =
            at == kNegInf && log2_s == log2_s ? kNegInf : (at - xr.m) * c2 - log2_s;
        if (!(p == 0.f)) term = p * (((gap - log2_t) - log2_q) * kLn2);
    }
    ids[tid] = e.id;
    ps[tid] = p;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) term += __shfl_xor(term, o);
    if (lane == 0) sum[w] = term;
    // the dense part of the gradient: f q_v (a row of -inf alone has q = 0)
    const bool some = !(ts.s == 0.f) && gr != 0.f;  // (a list of NaN has the sum NaN)
    const float f = some ? gr * tau : 0.f;
    const float fq = row_s.s == 0.f ? 0.f : f / row_s.s * ex2(-xr.rest);
    int c1 = c0;
    asm volatile("" : "+v"(c1));  // (offsets formed anew, not kept since the loads)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i * per < V + before) {
            const int c = i * (int)per + c1;
            float d[n];
#pragma unroll
            for (int j = 0; j < n; ++j) d[j] = fq * ex2(xr(v[i].get(j)));
            Run<IO, n> o = round_run<IO, n>(d);
            if (!some) o.zero();
            if (c >= 0 && c <= last) {
                o.store_at(out, (uint32_t)c * (uint32_t)sizeof(IO));
            } else if (c > -n && c < (int)V) {
                const int in = c < 0 ? 0 : last;
#pragma unroll
                for (int j = 0; j < n; ++j)
                    if (in + j >= c && in + j < c + n) out[in + j] = o.get_raw(j);
            }
        }
    }
    // the dense stores are done before an element is written again
    wait_mem();
    __syncthreads();
    if (tid == 0) {
        float t = 0.f;
        for (int i = 0; i < (BS / 64); ++i) t += sum[i];
        loss[r] = tau * tau * t;
        lse[r] = fmaf(xr.m, inv_tau, log2_s * kLn2);
    }
    if (some && e.id >= 0) {
        float all = 0.f;
        bool first = true;
        for (int j = 0; j < k; ++j)
            if (ids[j] == e.id) {
                first = first && j >= tid;
                all += ps[j];
            }
        if (first) {
            const float q = row_s.s == 0.f ? 0.f : ex2((at - xr.m) * c2) / row_s.s;
            out[e.id] = from_f<IO>(f * (q - all));
        }
    }
}

struct DistillArgs {
    int64_t R, V;
    int k;
    const void *logits;
    int64_t ld;
    const int32_t *t_ids;
    const float *t_logits;
    float tau;
    float *loss, *lse;          // forward
    const float *g;             // backward
    void *dlogits;
    int64_t ldd;
};

// Short rows take workgroups of two waves: the rows, not the logits, are then what there are
// many of (65536 x 1000 fp32, loss and gradient: 367 us with eight waves a row, 184 us with
// two).
constexpr int kSmallBS = 128, kLargeBS = 512;
template <typename IO> static bool short_rows(const DistillArgs &a)
{
    return a.V <= (int64_t)kSmallBS * kPer16<IO> * 4 && a.k <= kSmallBS;
}

template <typename IO, int BS> static hipError_t launch_loss_t(const DistillArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)(a.R < (1 << 22) ? a.R : 1 << 22);
    hipLaunchKernelGGL((distill_loss_kernel<IO, BS>), dim3(grid), dim3(BS), 0, st, a.R, a.V, a.k,
                       (const IO *)a.logits, a.ld, a.t_ids, a.t_logits, a.tau, 1.f / a.tau, a.loss,
                       a.lse);
    return hipGetLastError();
}
template <typename IO> static hipError_t launch_loss(const DistillArgs &a, hipStream_t st)
{
    return short_rows<IO>(a) ? launch_loss_t<IO, kSmallBS>(a, st)
                             : launch_loss_t<IO, kLargeBS>(a, st);
}

template <typename IO, int NV, int BS>
static hipError_t launch_grad_t(const DistillArgs &a, hipStream_t st)
{
    constexpr int64_t chunk = (int64_t)BS * kPer16<IO> * NV;
    const int64_t n_chunks = (a.V + chunk - 1) / chunk;
    const int64_t most = ((int64_t)1 << 22) / n_chunks + 1;  // rows of a launch
    for (int64_t r = 0; r < a.R; r += most) {
        const int64_t rows = a.R - r < most ? a.R - r : most;
        hipLaunchKernelGGL((distill_grad_kernel<IO, NV, BS>), dim3((unsigned)(rows * n_chunks)),
                           dim3(BS), 0, st, a.V, a.k, (int)n_chunks,
                           (const IO *)a.logits + r * a.ld, a.ld, a.t_ids + r * a.k,
                           a.t_logits + r * a.k, a.tau, 1.f / a.tau, a.lse + r, a.g + r,
                           (IO *)a.dlogits + r * a.ldd, a.ldd);
    }
    return hipGetLastError();
}
template <typename IO> static hipError_t launch_grad(const DistillArgs &a, hipStream_t st)
{
    if (short_rows<IO>(a)) return launch_grad_t<IO, 4, kSmallBS>(a, st);
    // eight accesses a thread amortise the entries' part of a workgroup; few rows are cut finer
    // (eight and two, us, 131072 bf16 logits: 1 row 9.2 and 7.4, 64 rows 13.9 and 13.6, 128 rows
    // 18.8 and 19.0, 256 rows 31.1 and 31.3)
    constexpr int64_t per = kLargeBS * kPer16<IO>;
    return a.R * ((a.V + 8 * per - 1) / (8 * per)) >= 512 ? launch_grad_t<IO, 8, kLargeBS>(a, st)
                                                          : launch_grad_t<IO, 2, kLargeBS>(a, st);
}

template <typename IO, int NV, int BS>
static hipError_t launch_step_t(const DistillArgs &a, hipStream_t st)
{
    constexpr int64_t most = 1 << 22;  // rows of a launch
    for (int64_t r = 0; r < a.R; r += most) {
        const int64_t rows = a.R - r < most ? a.R - r : most;
        hipLaunchKernelGGL((distill_step_kernel<IO, NV, BS>), dim3((unsigned)rows), dim3(BS), 0, st,
                           (uint32_t)a.V, a.k, (const IO *)a.logits + r * a.ld, a.ld,
                           a.t_ids + r * a.k, a.t_logits + r * a.k, a.tau, 1.f / a.tau, a.g + r,
                           a.loss + r, a.lse + r, (IO *)a.dlogits + r * a.ldd, a.ldd);
    }
    return hipGetLastError();
}

template <typename IO> static hipError_t launch_step(const DistillArgs &a, hipStream_t st)
{
    constexpr int n = kPer16<IO>;
    if (a.V < n) {  // (shorter than an access)
        const hipError_t e = launch_loss<IO>(a, st);
        return e == hipSuccess ? launch_grad<IO>(a, st) : e;
    }
    // logits and what may lie between them and a 16-byte boundary of the gradient's row
    const bool aligned = (uintptr_t)a.dlogits % 16 == 0 && a.ldd % n == 0;
    const int64_t span = a.V + (aligned ? 0 : n - 1);
    if (span <= kSmallBS * n * 4 && a.k <= kSmallBS)
        return span <= kSmallBS * n ? launch_step_t<IO, 1, kSmallBS>(a, st)
                                   : launch_step_t<IO, 4, kSmallBS>(a, st);
    constexpr int64_t per = kLargeBS * n;  // logits of one access each
    if (span <= 2 * per) return launch_step_t<IO, 2, kLargeBS>(a, st);
    if (span <= 4 * per) return launch_step_t<IO, 4, kLargeBS>(a, st);
    if (span <= 8 * per) return launch_step_t<IO, 8, kLargeBS>(a, st);
    if (span <= 16 * per) return launch_step_t<IO, 16, kLargeBS>(a, st);
    if (span <= 32 * per) return launch_step_t<IO, 32, kLargeBS>(a, st);
    // the row does not fit the registers: it is read again for the gradient
    const hipError_t e = launch_loss<IO>(a, st);
    return e == hipSuccess ? launch_grad<IO>(a, st) : e;
}

static naju_status_t check_distill(int64_t R, int64_t V, int64_t k, int32_t io, const void *logits,
                                   int64_t ld, const void *t_ids, const void *t_logits, float tau)
{
    if (R < 0 || V < 0 || k < 0)
        return fail(NAJU_EINVAL, "negative size (rows=%lld vocab=%lld k=%lld)", (long long)R,
                    (long long)V, (long long)k);
    if (io != NAJU_F32 && io != NAJU_BF16)
        return fail(NAJU_EINVAL, "io dtype %d is neither NAJU_F32 nor NAJU_BF16", (int)io);
    if (R > ((int64_t)1 << 30) || V > ((int64_t)1 << 30))
        return fail(NAJU_EINVAL, "rows or vocab too large (2^30 max)");
    if (k > kMostEntries)
        return fail(NAJU_EUNSUPPORTED, "k %lld teacher entries a row (%d max)", (long long)k,
                    kMostEntries);
    if (!(tau > 0.f) || !(tau < __builtin_huge_valf()))
        return fail(NAJU_EINVAL, "temperature must be positive and finite");
    // (exponents are scaled by it, and 0 times infinity would be NaN)
    if (!(1.f / tau * kLog2e < __builtin_huge_valf()))
        return fail(NAJU_EINVAL, "temperature is too small for its reciprocal");
    if (R == 0 || V == 0) return NAJU_OK;
    if (ld < V) return fail(NAJU_EINVAL, "row stride of logits %lld is less than vocab %lld",
                            (long long)ld, (long long)V);
    if (ld > ((int64_t)1 << 31)) return fail(NAJU_EINVAL, "row stride of logits too large");
    NAJU_TRY(need(logits, "logits", io == NAJU_F32 ? 4 : 2));
    if (k > 0) {
        NAJU_TRY(need(t_ids, "t_ids", 4));
        NAJU_TRY(need(t_logits, "t_logits", 4));
    }
    return NAJU_OK;
}

static naju_status_t check_dlogits(int64_t V, int32_t io, const float *g, const void *dlogits,
                                   int64_t ldd)
{
    if (ldd < V) return fail(NAJU_EINVAL, "row stride of dlogits %lld is less than vocab %lld",
                             (long long)ldd, (long long)V);
    if (ldd > ((int64_t)1 << 31)) return fail(NAJU_EINVAL, "row stride of dlogits too large");
    NAJU_TRY(need(g, "g", 4));
    return need(dlogits, "dlogits", io == NAJU_F32 ? 4 : 2);
}

}  // namespace naju

using namespace naju;

extern "C" {

naju_status_t naju_distill_fwd(int64_t rows, int64_t vocab, int64_t k, int32_t io,
                               const void *logits, int64_t ld, const int32_t *t_ids,
                               const float *t_logits, float temperature, float *loss, float *lse,
                               void *stream)
{
    NAJU_TRY(check_distill(rows, vocab, k, io, logits, ld, t_ids, t_logits, temperature));
    if (rows == 0 || vocab == 0) return NAJU_OK;
    NAJU_TRY(need(loss, "loss", 4));
    NAJU_TRY(need(lse, "lse", 4));
    const DistillArgs a{rows, vocab, (int)k, logits, ld, t_ids, t_logits, temperature,
                        loss, lse, nullptr, nullptr, 0};
    hipStream_t st = (hipStream_t)stream;
    return hip_status(io == NAJU_F32 ? launch_loss<float>(a, st) : launch_loss<bf16>(a, st),
                      "distillation loss launch");
}

naju_status_t naju_distill_bwd(int64_t rows, int64_t vocab, int64_t k, int32_t io,
                               const void *logits, int64_t ld, const int32_t *t_ids,
                               const float *t_logits, float temperature, const float *lse,
                               const float *g, void *dlogits, int64_t ld_d, void *stream)
{
    NAJU_TRY(check_distill(rows, vocab, k, io, logits, ld, t_ids, t_logits, temperature));
    if (rows == 0 || vocab == 0) return NAJU_OK;
    NAJU_TRY(need(lse, "lse", 4));
    NAJU_TRY(check_dlogits(vocab, io, g, dlogits, ld_d));
    const DistillArgs a{rows, vocab, (int)k, logits, ld, t_ids, t_logits, temperature,
                        nullptr, const_cast<float *>(lse), g, dlogits, ld_d};
    hipStream_t st = (hipStream_t)stream;
    return hip_status(io == NAJU_F32 ? launch_grad<float>(a, st) : launch_grad<bf16>(a, st),
                      "distillation gradient launch");
}

naju_status_t naju_distill_fwd_bwd(int64_t rows, int64_t vocab, int64_t k, int32_t io,
                                   const void *logits, int64_t ld, const int32_t *t_ids,
                                   const float *t_logits, float temperature, const float *g,
                                   float *loss, float *lse, void *dlogits, int64_t ld_d,
                                   void *stream)
{
    NAJU_TRY(check_distill(rows, vocab, k, io, logits, ld, t_ids, t_logits, temperature));
    if (rows == 0 || vocab == 0) return NAJU_OK;
    NAJU_TRY(need(loss, "loss", 4));
    NAJU_TRY(need(lse, "lse", 4));
    NAJU_TRY(check_dlogits(vocab, io, g, dlogits, ld_d));
    const DistillArgs a{rows, vocab, (int)k, logits, ld, t_ids, t_logits, temperature,
                        loss, lse, g, dlogits, ld_d};
    hipStream_t st = (hipStream_t)stream;
    return hip_status(io == NAJU_F32 ? launch_step<float>(a, st) : launch_step<bf16>(a, st),
                      "distillation launch");
}

}  // extern "C"
