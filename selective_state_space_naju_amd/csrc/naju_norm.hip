// naju_norm.hip -- the norms before and after a block, fused with the block's
// gate and its residual scale, and their gradients.
//
// Per token, with the residual stream x, the block's output y, a gate
// pre-activation z and per-channel vectors s, w_post, w_pre:
//     n  = y * rsqrt(mean y^2 + eps) * w_post       (y itself without w_post)
//     x' = x + s n SiLU(z)
//     xn = x' * rsqrt(mean x'^2 + eps) * w_pre
// and backwards, for the gradients dxn of xn and dx' of x':
//     r = rsqrt(mean x'^2 + eps), xh = x' r, e = dxn w_pre
//     dx = dx' + r (e - xh mean(e xh)),   dw_pre = sum_t dxn xh
//     f = dx s SiLU(z),  dz = dx s n SiLU'(z),  ds = sum_t dx n SiLU(z)
//     dw_post = sum_t f yh,  dy = r_y (f w_post - yh mean(f w_post yh))
//
// Bound by bytes: every tensor is read or written once, the row's means are
// taken from registers.  A row belongs to one wave (up to 1024 channels), or to
// a workgroup of 4, 8 or 16 waves; workgroups walk over rows with the per-channel
// vectors, and the gradient's per-channel sums, in registers, and the next row's
// loads in flight while one is worked on.  Statistics and sums are fp32; each
// output is rounded once.
//
// 16384 x 768, all of it: forward in bf16 with an fp32 stream 35.8 us (4.9 TB/s, a large
// copy's rate), gradient with an fp32 stream gradient 60 us (4.6 TB/s); 65536 x 2048,
// gradient 342 us (5.5 TB/s).  Rows that do not fill a wave's or a workgroup's threads
// waste them (300 channels 3.7 TB/s, 64 channels 1.5), and the gradient beyond 4096
// channels is bound by its registers (8192 channels, below).
#include <math.h>

#include "naju_device.h"
#include "naju_host.h"
#include "naju_launch.h"
#include "naju_vec.h"

namespace naju {

constexpr int kNormMost = 8192;  // channels of a row

struct NormArgs {
    int64_t R;
    int d;
    float eps, inv_d;
    const void *x, *y, *z;               // x: the stream before (forward), after (backward)
    const float *scale, *w_post, *w_pre;
    void *x_new, *xn;                    // forward
    const void *dxn, *dx_new;            // backward
    void *dx, *dy, *dz;
    float *part;                         // [workgroups][3][d]: dw_pre, dw_post, dscale
};

// Sum over the wave's 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float v)
{
    v = quad_sum(v);
    v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x124,
                                                            0xF, 0xF, false));  // row_ror:4
    v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x128,
                                                            0xF, 0xF, false));  // row_ror:8
    const uint32_t a = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const uint32_t b = __float_as_uint(v);
    const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Sums of N values over a row's W waves, in every lane.  `slot` alternates between
// calls, so that a wave may write the next sums while another still reads these.
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[4][16], int slot, int w,
                                         int lane)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (lane == i) red[slot][i][w] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = red[slot][i][0];
#pragma unroll
            for (int j = 1; j < W; ++j) v[i] += red[slot][i][j];
        }
    }
}

// Where a thread's K runs of 4 channels lie.  The last run of a row that is no
// multiple of 4 is moved back to end with the row: its first `skip` channels
// belong to the run before it, are computed twice and counted once.  A run past
// the row's end repeats the last one and counts nothing (skip 4).
template <int T, int K> struct Runs {
    int at[K], skip[K];
    __device__ __forceinline__ Runs(int t, int d)
    {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * T + t) * 4;
            at[k] = c <= d - 4 ? c : d - 4;
            skip[k] = c - at[k] < 4 ? c - at[k] : 4;
        }
    }
    __device__ __forceinline__ bool counts(int k, int i) const { return i >= skip[k]; }
};

template <typename IO, int T, int K>
__device__ __forceinline__ void load_runs(Run<IO, 4> (&r)[K], const void *p, int64_t row, int d,
                                          const Runs<T, K> &at)
{
    const IO *base = (const IO *)p + row * d;
#pragma unroll
    for (int k = 0; k < K; ++k) r[k].load_at(base, (uint32_t)at.at[k] * (uint32_t)sizeof(IO));
}

template <typename IO, int T, int K>
__device__ __forceinline__ void load_or_zero(Run<IO, 4> (&r)[K], bool given, const void *p,
                                             int64_t row, int d, const Runs<T, K> &at)
{
    if (given) {
        load_runs<IO, T, K>(r, p, row, d, at);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) r[k].zero();
    }
}

// (channels that two runs share get the same bits from both)
template <typename IO, int T, int K>
__device__ __forceinline__ void store_runs(const float (&v)[K][4], void *p, int64_t row, int d,
                                           const Runs<T, K> &at)
{
    IO *base = (IO *)p + row * d;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (at.skip[k] < 4)
            round_run<IO, 4>(v[k]).store_at(base, (uint32_t)at.at[k] * (uint32_t)sizeof(IO));
}

template <int T, int K>
__device__ __forceinline__ void load_vector(float (&v)[K][4], const float *p, const Runs<T, K> &at)
{
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] = p != nullptr ? p[at.at[k] + i] : 1.f;
}

// ------------------------------------------------------------------- forward
template <typename IO, typename XIO, int W, int K>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_fwd_kernel(const NormArgs g)
{
    constexpr int T = 64 * W, kRows = W == 1 ? 4 : 1;
    __shared__ float red[2][4][16];
    const int lane = threadIdx.x & 63, d = g.d;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int w = W == 1 ? 0 : wave;
    const Runs<T, K> at(w * 64 + lane, d);
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + (W == 1 ? wave : 0);
    if (row >= g.R) return;  // (a row's waves leave together)

    const bool has_y = g.y != nullptr, has_z = g.z != nullptr;
    float s[K][4], wo[K][4], wi[K][4];
    load_vector(s, g.scale, at);
    load_vector(wo, g.w_post, at);
    load_vector(wi, g.w_pre, at);
    Run<XIO, 4> xr[K];
    Run<IO, 4> yr[K], zr[K];
    auto fetch = [&](int64_t r) {
        load_runs<XIO, T, K>(xr, g.x, r, d, at);
        if (has_y) load_runs<IO, T, K>(yr, g.y, r, d, at);
        if (has_z) load_runs<IO, T, K>(zr, g.z, r, d, at);
    };
    fetch(row);
    int slot = 0;
    for (; row < g.R; row += step) {
        float x[K][4], n[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[k][i] = xr[k].get(i);
                n[k][i] = 0.f;
                if (has_y) n[k][i] = yr[k].get(i);
            }
        float gate[K][4];
        if (has_z) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float z = zr[k].get(i);
                    gate[k][i] = z * sigm(z);
                }
        }
        const int64_t next = row + step;
        if (next < g.R) fetch(next);
        if (has_y) {
            float ry = 1.f;
            if (g.w_post != nullptr) {
                float sum[1] = {0.f};
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (at.counts(k, i)) sum[0] = __builtin_fmaf(n[k][i], n[k][i], sum[0]);
                row_sums<W, 1>(sum, red, slot, w, lane);
                slot ^= 1;
                ry = rsqrtf(sum[0] * g.inv_d + g.eps);
            }
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = n[k][i] * ry * wo[k][i] * s[k][i];
                    if (has_z) v *= gate[k][i];
                    x[k][i] += v;
                }
            store_runs<XIO, T, K>(x, g.x_new, row, d, at);
        }
        if (g.w_pre != nullptr) {
            float sum[1] = {0.f};
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at.counts(k, i)) sum[0] = __builtin_fmaf(x[k][i], x[k][i], sum[0]);
            row_sums<W, 1>(sum, red, slot, w, lane);
            slot ^= 1;
            const float r = rsqrtf(sum[0] * g.inv_d + g.eps);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[k][i] *= r * wi[k][i];
            store_runs<IO, T, K>(x, g.xn, row, d, at);
        }
    }
}

// ------------------------------------------------------------------ backward
// AHEAD: the next row's loads are in flight while a row is worked on.  Beyond 4096 channels that
// does not fit the registers; a row then stays packed, unpacked once for the sums and again for the
// outputs (4882 x 8192: bf16 225 us, fp32 351; with 16 waves and the next row ahead 297 and 480).
template <typename IO, typename XIO, typename GIO, int W, int K, bool AHEAD>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_bwd_kernel(const NormArgs g)
{
    constexpr int T = 64 * W, kRows = W == 1 ? 4 : 1;
    __shared__ float red[2][4][16];
    const int lane = threadIdx.x & 63, d = g.d;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int w = W == 1 ? 0 : wave;
    const Runs<T, K> at(w * 64 + lane, d);
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + (W == 1 ? wave : 0);

    const bool pre = g.w_pre != nullptr, has_dx = g.dx_new != nullptr;
    const bool has_y = g.y != nullptr, has_z = g.z != nullptr, post = g.w_post != nullptr;
    float s[K][4], wo[K][4], wi[K][4];
    load_vector(s, g.scale, at);
    load_vector(wo, g.w_post, at);
    load_vector(wi, g.w_pre, at);
    float a_pre[K][4], a_post[K][4], a_scale[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) a_pre[k][i] = a_post[k][i] = a_scale[k][i] = 0.f;

    // (what is not given is zero, not left from the row before: nothing lives on)
    Run<XIO, 4> xr[K];
    Run<GIO, 4> er[K], dr[K];
    Run<IO, 4> yr[K], zr[K];
    auto fetch = [&](int64_t r) {
        load_or_zero<XIO, T, K>(xr, pre, g.x, r, d, at);
        load_or_zero<GIO, T, K>(er, pre, g.dxn, r, d, at);
        load_or_zero<GIO, T, K>(dr, has_dx, g.dx_new, r, d, at);
        load_or_zero<IO, T, K>(yr, has_y, g.y, r, d, at);
        load_or_zero<IO, T, K>(zr, has_z, g.z, r, d, at);
    };
    if (AHEAD && row < g.R) fetch(row);
    int slot = 0;
    for (; row < g.R; row += step) {
        if (!AHEAD) fetch(row);
        Run<XIO, 4> xc[K];
        Run<GIO, 4> ec[K], dc[K];
        Run<IO, 4> yc[K], zc[K];
        float sum[3] = {0.f, 0.f, 0.f};  // x'^2, dxn w_pre x', y^2
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xc[k] = xr[k];
            ec[k] = er[k];
            dc[k] = dr[k];
            yc[k] = yr[k];
            zc[k] = zr[k];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!at.counts(k, i)) continue;
                if (pre) {
                    const float x = xc[k].get(i);
                    sum[0] = __builtin_fmaf(x, x, sum[0]);
                    sum[1] = __builtin_fmaf(ec[k].get(i) * wi[k][i], x, sum[1]);
                }
                if (post) sum[2] = __builtin_fmaf(yc[k].get(i), yc[k].get(i), sum[2]);
            }
        }
        const int64_t next = row + step;
        if (AHEAD && next < g.R) fetch(next);
        if (pre || post) {
            row_sums<W, 3>(sum, red, slot, w, lane);
            slot ^= 1;
        }
        float dx[K][4];
        const float r = pre ? rsqrtf(sum[0] * g.inv_d + g.eps) : 0.f;
        const float mean = sum[1] * r * g.inv_d;  // of e xh
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!AHEAD) xc[k].repack();
            if (!AHEAD) ec[k].repack();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dx[k][i] = has_dx ? dc[k].get(i) : 0.f;
                if (pre) {
                    const float xh = xc[k].get(i) * r, e = ec[k].get(i);
                    a_pre[k][i] = __builtin_fmaf(e, xh, a_pre[k][i]);
                    dx[k][i] += r * (e * wi[k][i] - xh * mean);
                }
            }
        }
        store_runs<GIO, T, K>(dx, g.dx, row, d, at);
        if (!has_y) continue;
        const float ry = post ? rsqrtf(sum[2] * g.inv_d + g.eps) : 1.f;
        float dot[1] = {0.f};  // of f w_post and y
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float dz[4];
            if (!AHEAD) yc[k].repack();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float gate = 1.f, slope = 0.f;
                if (has_z) {
                    const float z = zc[k].get(i), sig = sigm(z);
                    gate = z * sig;
                    slope = sig * __builtin_fmaf(z, 1.f - sig, 1.f);
                }
                const float yh = yc[k].get(i) * ry, n = yh * wo[k][i];
                const float t = dx[k][i] * s[k][i];
                a_scale[k][i] = __builtin_fmaf(dx[k][i] * gate, n, a_scale[k][i]);
                dz[i] = t * n * slope;
                const float f = t * gate;
                a_post[k][i] = __builtin_fmaf(f, yh, a_post[k][i]);
                dx[k][i] = f * wo[k][i];
                if (at.counts(k, i)) dot[0] = __builtin_fmaf(dx[k][i], yh, dot[0]);
            }
            if (has_z && at.skip[k] < 4)
                round_run<IO, 4>(dz).store_at((IO *)g.dz + row * d,
                                              (uint32_t)at.at[k] * (uint32_t)sizeof(IO));
        }
        if (post) {
            row_sums<W, 1>(dot, red, slot, w, lane);
            slot ^= 1;
            const float m = dot[0] * g.inv_d;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!AHEAD) yc[k].repack();
#pragma unroll
                for (int i = 0; i < 4; ++i) dx[k][i] = ry * (dx[k][i] - yc[k].get(i) * ry * m);
            }
        }
        store_runs<IO, T, K>(dx, g.dy, row, d, at);
    }

    // this workgroup's sums; with a wave for each row, the four waves' first added up
    float *part = g.part + (int64_t)blockIdx.x * 3 * d;
    if constexpr (W == 1) {
        __shared__ float join[4][K * 256];
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at.counts(k, i))
                        join[wave][at.at[k] + i] =
                            q == 0 ? a_pre[k][i] : q == 1 ? a_post[k][i] : a_scale[k][i];
            __syncthreads();
            for (int c = threadIdx.x; c < d; c += 256)
                part[q * d + c] = (join[0][c] + join[1][c]) + (join[2][c] + join[3][c]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at.counts(k, i)) {
                    part[at.at[k] + i] = a_pre[k][i];
                    part[d + at.at[k] + i] = a_post[k][i];
                    part[2 * d + at.at[k] + i] = a_scale[k][i];
                }
    }
}

// out[q][c] = sum over the workgroups' partial sums, in a fixed order: 32 rows of
// threads take every 32nd workgroup.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float *part, int groups, int d,
                                                         float *dw_pre, float *dw_post,
                                                         float *dscale)
{
    __shared__ float sum[32][33];
    float *out = blockIdx.y == 0 ? dw_pre : blockIdx.y == 1 ? dw_post : dscale;
    if (out == nullptr) return;
    const int x = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    const float *p = part + (int64_t)blockIdx.y * d + c;
    float v = 0.f;
    if (c < d) {
#pragma unroll 4
        for (int i = r; i < groups; i += 32) v += p[(int64_t)i * 3 * d];
    }
    sum[r][x] = v;
    __syncthreads();
    if (r == 0 && c < d) {
#pragma unroll 8
        for (int i = 1; i < 32; ++i) v += sum[i][x];
        out[c] = v;
    }
}

// ---------------------------------------------------------------------- host
template <typename IO, typename XIO, int W, int K>
static hipError_t launch_fwd(const NormArgs &g, hipStream_t st)
{
    const int64_t blocks = W == 1 ? (g.R + 3) / 4 : g.R;
    const int64_t most = W == 1 ? 2048 : W == 4 ? 2048 : 512;
    hipLaunchKernelGGL((norm_fwd_kernel<IO, XIO, W, K>), dim3((unsigned)(blocks < most ? blocks : most)),
                       dim3(W == 1 ? 256 : 64 * W), 0, st, g);
    return hipGetLastError();
}

template <typename IO, typename XIO> static hipError_t pick_fwd(const NormArgs &g, hipStream_t st)
{
    if (g.d <= 256) return launch_fwd<IO, XIO, 1, 1>(g, st);
    if (g.d <= 512) return launch_fwd<IO, XIO, 1, 2>(g, st);
    if (g.d <= 768) return launch_fwd<IO, XIO, 1, 3>(g, st);
    if (g.d <= 1024) return launch_fwd<IO, XIO, 1, 4>(g, st);
    if (g.d <= 2048) return launch_fwd<IO, XIO, 4, 2>(g, st);
    if (g.d <= 4096) return launch_fwd<IO, XIO, 4, 4>(g, st);
    return launch_fwd<IO, XIO, 16, 2>(g, st);
}

// Workgroups of the gradient, each with a row of partial sums: as many as are resident.
static int bwd_groups(int64_t R, int64_t d)
{
    const int64_t blocks = d <= 1024 ? (R + 3) / 4 : R;
    const int64_t most = d <= 256 ? 1536 : d <= 2048 ? 512 : 256;
    return (int)(blocks < most ? blocks : most);
}

template <typename IO, typename XIO, typename GIO, int W, int K>
static hipError_t launch_bwd(const NormArgs &g, hipStream_t st)
{
    hipLaunchKernelGGL((norm_bwd_kernel<IO, XIO, GIO, W, K, (W * K < 32)>), dim3(bwd_groups(g.R, g.d)),
                       dim3(W == 1 ? 256 : 64 * W), 0, st, g);
    return hipGetLastError();
}

template <typename IO, typename XIO, typename GIO>
static hipError_t pick_bwd(const NormArgs &g, hipStream_t st)
{
    if (g.d <= 256) return launch_bwd<IO, XIO, GIO, 1, 1>(g, st);
    if (g.d <= 512) return launch_bwd<IO, XIO, GIO, 1, 2>(g, st);
    if (g.d <= 768) return launch_bwd<IO, XIO, GIO, 1, 3>(g, st);
    if (g.d <= 1024) return launch_bwd<IO, XIO, GIO, 1, 4>(g, st);
    if (g.d <= 2048) return launch_bwd<IO, XIO, GIO, 4, 2>(g, st);
    if (g.d <= 4096) return launch_bwd<IO, XIO, GIO, 8, 2>(g, st);
    return launch_bwd<IO, XIO, GIO, 8, 4>(g, st);
}

static naju_status_t check_norm(int64_t R, int64_t d, int32_t io, int32_t x_io, int32_t g_io,
                                float eps)
{
    if (R < 0 || d < 0)
        return fail(NAJU_EINVAL, "negative size (tokens=%lld d_model=%lld)", (long long)R,
                    (long long)d);
    for (int32_t t : {io, x_io, g_io})
        if (t != NAJU_F32 && t != NAJU_BF16)
            return fail(NAJU_EINVAL, "io dtype %d is neither NAJU_F32 nor NAJU_BF16", (int)t);
    if (io == NAJU_F32 && (x_io != NAJU_F32 || g_io != NAJU_F32))
        return fail(NAJU_EUNSUPPORTED, "an fp32 block needs an fp32 residual stream and fp32 "
                                       "gradients");
    if (R > ((int64_t)1 << 40)) return fail(NAJU_EINVAL, "tokens (2^40 max) too large");
    if (d != 0 && (d < 4 || d > kNormMost))
        return fail(NAJU_EUNSUPPORTED, "d_model %lld is not from 4 to %d", (long long)d, kNormMost);
    if (!(eps >= 0.f) || eps > 1e30f)
        return fail(NAJU_EINVAL, "eps must be finite and not negative");
    return NAJU_OK;
}

// what goes with y: nothing of it may be given alone
static naju_status_t check_block(const void *y, const void *z, const float *scale,
                                 const float *w_post, size_t e)
{
    if (y == nullptr && (z != nullptr || scale != nullptr || w_post != nullptr))
        return fail(NAJU_EINVAL, "z, scale and w_post need y");
    NAJU_TRY(opt(y, "y", e));
    NAJU_TRY(opt(z, "z", e));
    NAJU_TRY(opt(scale, "scale", 4));
    return opt(w_post, "w_post", 4);
}

}  // namespace naju

using namespace naju;

extern "C" {

naju_status_t naju_res_norm_fwd(int64_t tokens, int64_t d_model, int32_t io, int32_t x_io,
                                const void *x, const void *y, const void *z, const float *scale,
                                const float *w_post, const float *w_pre, float eps, void *x_new,
                                void *xn, void *stream)
{
    NAJU_TRY(check_norm(tokens, d_model, io, x_io, io, eps));
    const size_t e = io == NAJU_F32 ? 4 : 2, ex = x_io == NAJU_F32 ? 4 : 2;
    if (tokens == 0 || d_model == 0) return NAJU_OK;
    NAJU_TRY(check_block(y, z, scale, w_post, e));
    if ((w_pre != nullptr) != (xn != nullptr))
        return fail(NAJU_EINVAL, "w_pre and xn go together");
    if ((y != nullptr) != (x_new != nullptr))
        return fail(NAJU_EINVAL, "y and x_new go together");
    if (y == nullptr && w_pre == nullptr)
        return fail(NAJU_EINVAL, "neither y nor w_pre is given: nothing to compute");
    NAJU_TRY(need(x, "x", ex));
    NAJU_TRY(opt(w_pre, "w_pre", 4));
    NAJU_TRY(opt(x_new, "x_new", ex));
    NAJU_TRY(opt(xn, "xn", e));
    NormArgs g{};
    g.R = tokens;
    g.d = (int)d_model;
    g.eps = eps;
    g.inv_d = 1.f / (float)d_model;
    g.x = x;
    g.y = y;
    g.z = z;
    g.scale = scale;
    g.w_post = w_post;
    g.w_pre = w_pre;
    g.x_new = x_new;
    g.xn = xn;
    hipStream_t st = (hipStream_t)stream;
    return hip_status(io == NAJU_F32     ? pick_fwd<float, float>(g, st)
                      : x_io == NAJU_F32 ? pick_fwd<bf16, float>(g, st)
                                         : pick_fwd<bf16, bf16>(g, st),
                      "norm launch");
}

size_t naju_res_norm_bwd_workspace_bytes(int64_t tokens, int64_t d_model)
{
    if (check_norm(tokens, d_model, NAJU_F32, NAJU_F32, NAJU_F32, 0.f) != NAJU_OK) return 0;
    return align256(256 + (size_t)bwd_groups(tokens, d_model) * 3 * (size_t)d_model * 4);
}

naju_status_t naju_res_norm_bwd(int64_t tokens, int64_t d_model, int32_t io, int32_t x_io,
                                int32_t g_io, const void *dxn, const void *dx_new,
                                const void *x_new, const void *y, const void *z,
                                const float *scale, const float *w_post, const float *w_pre,
                                float eps, void *dx, void *dy, void *dz, float *dscale,
                                float *dw_post, float *dw_pre, void *ws, size_t ws_bytes,
                                void *stream)
{
    NAJU_TRY(check_norm(tokens, d_model, io, x_io, g_io, eps));
    const size_t e = io == NAJU_F32 ? 4 : 2, ex = x_io == NAJU_F32 ? 4 : 2;
    const size_t eg = g_io == NAJU_F32 ? 4 : 2;
    if (d_model == 0) return NAJU_OK;
    NAJU_TRY(opt(dscale, "dscale", 4));
    NAJU_TRY(opt(dw_post, "dw_post", 4));
    NAJU_TRY(opt(dw_pre, "dw_pre", 4));
    hipStream_t st = (hipStream_t)stream;
    if (tokens > 0) {
        NAJU_TRY(check_block(y, z, scale, w_post, e));
        if ((w_pre != nullptr) != (dxn != nullptr))
            return fail(NAJU_EINVAL, "w_pre and dxn go together");
        if (dscale != nullptr && scale == nullptr)
            return fail(NAJU_EINVAL, "dscale needs scale");
        if (dw_post != nullptr && w_post == nullptr)
            return fail(NAJU_EINVAL, "dw_post needs w_post");
        if (dw_pre != nullptr && w_pre == nullptr)
            return fail(NAJU_EINVAL, "dw_pre needs w_pre");
        if (dxn == nullptr && dx_new == nullptr)
            return fail(NAJU_EINVAL, "neither dxn nor dx_new is given: no gradient to pass on");
        NAJU_TRY(opt(w_pre, "w_pre", 4));
        NAJU_TRY(opt(dxn, "dxn", eg));
        NAJU_TRY(opt(dx_new, "dx_new", eg));
        if (w_pre != nullptr) NAJU_TRY(need(x_new, "x_new", ex));
        NAJU_TRY(need(dx, "dx", eg));
        if (y != nullptr) NAJU_TRY(need(dy, "dy", e));
        if (z != nullptr) NAJU_TRY(need(dz, "dz", e));
        NAJU_TRY(need_ws(ws, ws_bytes, naju_res_norm_bwd_workspace_bytes(tokens, d_model)));
    }
    NormArgs g{};
    g.R = tokens;
    g.d = (int)d_model;
    g.eps = eps;
    g.inv_d = 1.f / (float)d_model;
    g.x = x_new;
    g.y = y;
    g.z = z;
    g.scale = scale;
    g.w_post = w_post;
    g.w_pre = w_pre;
    g.dxn = dxn;
    g.dx_new = dx_new;
    g.dx = dx;
    g.dy = dy;
    g.dz = dz;
    g.part = (float *)ws;
    if (tokens > 0) {
        const hipError_t err =
            io == NAJU_F32 ? pick_bwd<float, float, float>(g, st)
            : x_io == NAJU_F32
                ? (g_io == NAJU_F32 ? pick_bwd<bf16, float, float>(g, st)
                                    : pick_bwd<bf16, float, bf16>(g, st))
                : (g_io == NAJU_F32 ? pick_bwd<bf16, bf16, float>(g, st)
                                    : pick_bwd<bf16, bf16, bf16>(g, st));
        NAJU_TRY(hip_status(err, "norm gradient launch"));
    }
    if (dscale == nullptr && dw_post == nullptr && dw_pre == nullptr) return NAJU_OK;
    // (no tokens: no partial sums, zeros)
    hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((d_model + 31) / 32), 3), dim3(1024), 0,
                       st, (const float *)ws, bwd_groups(tokens, d_model), (int)d_model, dw_pre,
                       dw_post, dscale);
    return hip_status(hipGetLastError(), "norm gradient sums launch");
}

}  // extern "C"
