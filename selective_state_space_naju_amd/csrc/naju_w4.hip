// naju_w4.hip -- linear layer with 4-bit weights and one scale per group of
// inputs, for the few rows of a decode step, and the quantisation of weights
// into its layout.
//
//     y[r][n] = sum_k x[r][k] (q[n][k] - z[n][k / G]) s[n][k / G] + bias[n] + res[r][n]
//
// The codes are read once and everything else is small, so the bytes of the
// codes bound it as long as unpacking keeps up: one VALU instruction per two
// weights.  (d >> 4 i) & 0x000f000f puts two codes into the low bits of two
// halves, and or-ing 0x4300 into each makes them the bf16 numbers 128 + q,
// exactly.  The matrix cores multiply those with x (fp32 sums), and
//     sum x (q - z) = sum x (128 + q) - (128 + z) sum x
// per group, with sum x formed in fp32 once per workgroup.  The subtraction
// costs at most about 2^-17 of sum |x| max|q - z|, far below the bf16 rounding
// of y.
//
// v_mfma_f32_16x16x32_bf16: 16 rows of x by 16 outputs, 32 inputs.  A lane
// (output l % 16, quarter l / 16) loads 16 bytes, 32 codes of one row; a 4 x 4
// transpose between the quarters (two lane-swap steps) makes each of the four
// products cover 32 consecutive inputs, so a product never spans two groups.
// The order of the 8 inputs inside a quarter is that of the unpacking; x is
// staged in LDS in the same order.
#include "naju_device.h"
#include "naju_host.h"
#include "naju_launch.h"
#include "naju_vec.h"

namespace naju {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kW4Threads = 512;
constexpr int kW4Waves = 8;

struct W4Args {
    int64_t R, K, N, ng;
    const bf16 *x;             // [R][K]
    const uint8_t *q;          // [N][K / 2]
    const bf16 *scales;        // [N][ng]
    const uint8_t *zeros;      // [N][ng] or null (= 8)
    const float *bias;         // [N] or null
    const bf16 *res;           // [R][N] or null
    bf16 *y;                   // [R][N]
};

// 16 bytes of a weight row from byte `off`, zeros past its `bytes`
__device__ __forceinline__ u32x4 load_codes(const uint8_t *row, int64_t off, int64_t bytes)
{
    u32x4 d = {0, 0, 0, 0};
    if (off + 16 <= bytes) {
        __builtin_memcpy(&d, row + off, 16);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (off + j < bytes) d[j / 4] |= (uint32_t)row[off + j] << (8 * (j % 4));
    }
    return d;
}

// 4 x 4 transpose of dwords between the wave's quarters: afterwards dword j of
// quarter h is what dword h of quarter j was.
__device__ __forceinline__ u32x4 transpose_quarters(u32x4 d)
{
    const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], e[0], e[1]};
}

// 8 codes as the bf16 numbers 128 + q, in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ bf16x8 unpack(uint32_t d)
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ((d >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    return __builtin_bit_cast(bf16x8, r);
}

// RT: tiles of 16 rows of x; G: inputs of a group; WK: waves that share an
// output tile and split the inputs between them (the other kW4Waves / WK take
// neighbouring tiles).
template <int RT, int G, int WK>
__global__ __launch_bounds__(kW4Threads) void w4_kernel(const W4Args g)
{
    constexpr int WN = kW4Waves / WK;
    constexpr int NB = WK >= 4 ? 1 : 4;           // blocks of 128 inputs per wave and stage
    constexpr int SC = NB * WK * 128;             // inputs of a stage
    constexpr int kRow = SC + 32;                 // staged row, padded to spread the banks
    constexpr int NG = 128 / G;                   // groups of a block
    constexpr int kRed = WK > 1 ? kW4Waves * RT * 256 : 0;  // floats of the final sums
    constexpr int kStage = RT * 16 * kRow / 2;    // 32-bit words of the staged x
    __shared__ __attribute__((aligned(16))) uint32_t lds[kStage > kRed ? kStage : kRed];
    __shared__ __attribute__((aligned(16))) float sx[SC / 32][RT * 16];
    bf16 *xs = (bf16 *)lds;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = w % WK, wn = w / WK, col = lane & 15, quarter = lane >> 4;
    const int64_t n = ((int64_t)blockIdx.x * WN + wn) * 16 + col;
    const int64_t nc = n < g.N ? n : g.N - 1;     // (lanes past the last output repeat it)
    const int64_t r0 = (int64_t)blockIdx.y * (RT * 16);
    const int64_t row_bytes = g.K / 2;
    const uint8_t *qrow = g.q + nc * row_bytes;
    const bf16 *srow = g.scales + nc * g.ng;
    const uint8_t *zrow = g.zeros ? g.zeros + nc * g.ng : nullptr;

    f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    u32x4 d[NB];
    float s[NB][NG], z[NB][NG];
    auto fetch = [&](int64_t k0) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int64_t k = k0 + (b * WK + wk) * 128;
            d[b] = load_codes(qrow, k / 2 + quarter * 16, row_bytes);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int64_t gi = k / G + i;
                s[b][i] = gi < g.ng ? to_f(srow[gi]) : 0.f;
                z[b][i] = zrow && gi < g.ng ? 128.f + (float)zrow[gi] : 136.f;
            }
        }
    };
    fetch(0);
    for (int64_t k0 = 0; k0 < g.K; k0 += SC) {
        if (k0) __syncthreads();
        // stage x[r0 .. ][k0 .. k0 + SC): 8 inputs a thread, and the sums of 32
        for (int i = tid; i < RT * 16 * (SC / 8); i += kW4Threads) {
            const int m = i / (SC / 8), c = (i % (SC / 8)) * 8;
            Run<bf16, 8> v;
            const int64_t left = g.K - k0 - c;
            if (r0 + m >= g.R || left <= 0) v.zero();
            else if (left >= 8) v.load(g.x + (r0 + m) * g.K + k0 + c);
            else v.load_part(g.x + (r0 + m) * g.K + k0 + c, (int)left);
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) sum += v.get(q);
            sum = quad_sum(sum);
            u32x4 o;  // pairs (0, 4) (1, 5) (2, 6) (3, 7)
            o[0] = __builtin_amdgcn_perm(v.w[2], v.w[0], 0x05040100);
            o[1] = __builtin_amdgcn_perm(v.w[2], v.w[0], 0x07060302);
            o[2] = __builtin_amdgcn_perm(v.w[3], v.w[1], 0x05040100);
            o[3] = __builtin_amdgcn_perm(v.w[3], v.w[1], 0x07060302);
            *(u32x4 *)(xs + m * kRow + c) = o;
            if ((i & 3) == 0) sx[c / 32][m] = sum;
        }
        __syncthreads();
        u32x4 cur[NB];
        float cs[NB][NG], cz[NB][NG];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            cur[b] = d[b];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                cs[b][i] = s[b][i];
                cz[b][i] = z[b][i];
            }
        }
        if (k0 + SC < g.K) fetch(k0 + SC);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const u32x4 t4 = transpose_quarters(cur[b]);
            const int c0 = (b * WK + wk) * 128;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                f32x4 p[RT];
                f32x4 tot[RT];
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    p[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                    tot[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
#pragma unroll
                for (int j = i * (G / 32); j < (i + 1) * (G / 32); ++j) {
                    const bf16x8 wv = unpack(t4[j]);
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const bf16x8 xv = *(const bf16x8 *)(xs + (t * 16 + col) * kRow + c0 +
                                                            j * 32 + quarter * 8);
                        p[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, wv, p[t], 0, 0, 0);
                        tot[t] += *(const f32x4 *)&sx[c0 / 32 + j][t * 16 + quarter * 4];
                    }
                }
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[t][q] = fmaf(cs[b][i], fmaf(-cz[b][i], tot[t][q], p[t][q]), acc[t][q]);
            }
        }
    }

    // the waves of an output tile add their sums in order
    if constexpr (WK > 1) {
        float *red = (float *)lds;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; ++t) *(f32x4 *)&red[((w * RT + t) * 64 + lane) * 4] = acc[t];
        __syncthreads();
        if (wk != 0) return;
#pragma unroll
        for (int i = 1; i < WK; ++i)
#pragma unroll
            for (int t = 0; t < RT; ++t)
                acc[t] += *(const f32x4 *)&red[(((w + i) * RT + t) * 64 + lane) * 4];
    }
    if (n >= g.N) return;
    const float bias = g.bias ? g.bias[n] : 0.f;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t r = r0 + t * 16 + quarter * 4 + q;
            if (r >= g.R) continue;
            float v = acc[t][q] + bias;
            if (g.res) v += to_f(g.res[r * g.N + n]);
            g.y[r * g.N + n] = from_f<bf16>(v);
        }
}

template <int RT, int G, int WK> static hipError_t launch_w4_t(const W4Args &g, hipStream_t st)
{
    constexpr int per = (kW4Waves / WK) * 16;
    const dim3 grid((unsigned)((g.N + per - 1) / per), (unsigned)((g.R + RT * 16 - 1) / (RT * 16)));
    hipLaunchKernelGGL((w4_kernel<RT, G, WK>), grid, dim3(kW4Threads), 0, st, g);
    return hipGetLastError();
}

template <int G> static hipError_t launch_w4(const W4Args &g, hipStream_t st)
{
    // few outputs: the waves of a workgroup split the inputs of one tile
    const bool split = g.N < 16 * 8 * 512;
    if (g.R <= 16) return split ? launch_w4_t<1, G, 8>(g, st) : launch_w4_t<1, G, 1>(g, st);
    if (g.R <= 32) return split ? launch_w4_t<2, G, 4>(g, st) : launch_w4_t<2, G, 1>(g, st);
    return split ? launch_w4_t<4, G, 4>(g, st) : launch_w4_t<4, G, 1>(g, st);
}

// ------------------------------------------------------------ quantisation
// One thread per (output, group): the extremes of its inputs, then its codes.
// Neighbouring threads take neighbouring outputs (coalesced reads of W).
template <typename IO>
__global__ __launch_bounds__(256) void w4_quantize_kernel(
    const int64_t K, const int64_t N, const int G, const int64_t ng, const IO *__restrict__ W,
    uint8_t *__restrict__ qw, bf16 *__restrict__ scales, uint8_t *__restrict__ zeros)
{
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    for (int64_t gi = blockIdx.y; gi < ng; gi += gridDim.y) {
        const int64_t k0 = gi * G, k1 = k0 + G < K ? k0 + G : K;
        float lo = 0.f, hi = 0.f;
        for (int64_t k = k0; k < k1; ++k) {
            const float v = to_f(W[k * N + n]);
            lo = fminf(lo, v);
            hi = fmaxf(hi, v);
        }
        // codes -7 .. 7 around 8 without zeros, 0 .. 15 between the extremes with them
        const bf16 sb = from_f<bf16>(zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f);
        const float s = to_f(sb);
        float z = 8.f;
        if (zeros) z = s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 8.f;
        scales[n * ng + gi] = sb;
        if (zeros) zeros[n * ng + gi] = (uint8_t)z;
        for (int64_t k = k0; k < k1; k += 2) {
            uint32_t b = 0;
            for (int j = 0; j < 2; ++j) {
                const float v = to_f(W[(k + j) * N + n]);
                const float c = s > 0.f ? fminf(fmaxf(rintf(v / s) + z, 0.f), 15.f) : z;
                b |= (uint32_t)c << (4 * j);
            }
            qw[n * (K / 2) + k / 2] = (uint8_t)b;
        }
    }
}

static naju_status_t check_w4(int64_t K, int64_t N, int64_t G)
{
    if (K < 0 || N < 0) return fail(NAJU_EINVAL, "negative size (d_in=%lld d_out=%lld)",
                                    (long long)K, (long long)N);
    if (G != 32 && G != 64 && G != 128)
        return fail(NAJU_EUNSUPPORTED, "group %lld not built (32, 64 and 128 are)", (long long)G);
    if (K % 2) return fail(NAJU_EUNSUPPORTED, "d_in %lld is odd (two codes share a byte)",
                           (long long)K);
    if (K > ((int64_t)1 << 24) || N > ((int64_t)1 << 26))
        return fail(NAJU_EINVAL, "d_in (2^24 max) or d_out (2^26 max) too large");
    return NAJU_OK;
}

}  // namespace naju

using namespace naju;

extern "C" {

naju_status_t naju_w4_quantize(int64_t d_in, int64_t d_out, int64_t group, int32_t io,
                               const void *W, uint8_t *qweight, void *scales, uint8_t *zeros,
                               void *stream)
{
    NAJU_TRY(check_w4(d_in, d_out, group));
    if (io != NAJU_F32 && io != NAJU_BF16)
        return fail(NAJU_EINVAL, "io dtype %d is neither NAJU_F32 nor NAJU_BF16", (int)io);
    if (d_in == 0 || d_out == 0) return NAJU_OK;
    NAJU_TRY(need(W, "W", io == NAJU_F32 ? 4 : 2));
    NAJU_TRY(need(qweight, "qweight", 1));
    NAJU_TRY(need(scales, "scales", 2));
    const int64_t ng = (d_in + group - 1) / group;
    const dim3 grid((unsigned)((d_out + 255) / 256), (unsigned)(ng < 16384 ? ng : 16384));
    hipStream_t st = (hipStream_t)stream;
    if (io == NAJU_F32)
        hipLaunchKernelGGL(w4_quantize_kernel<float>, grid, dim3(256), 0, st, d_in, d_out,
                           (int)group, ng, (const float *)W, qweight, (bf16 *)scales, zeros);
    else
        hipLaunchKernelGGL(w4_quantize_kernel<bf16>, grid, dim3(256), 0, st, d_in, d_out,
                           (int)group, ng, (const bf16 *)W, qweight, (bf16 *)scales, zeros);
    return hip_status(hipGetLastError(), "quantisation launch");
}

naju_status_t naju_w4_linear(int64_t rows, int64_t d_in, int64_t d_out, int64_t group,
                             const void *x, const uint8_t *qweight, const void *scales,
                             const uint8_t *zeros, const float *bias, const void *res, void *y,
                             void *stream)
{
    NAJU_TRY(check_w4(d_in, d_out, group));
    if (rows < 0) return fail(NAJU_EINVAL, "negative size (rows=%lld)", (long long)rows);
    if (rows > ((int64_t)1 << 20)) return fail(NAJU_EINVAL, "rows too large (2^20 max)");
    if (rows == 0 || d_out == 0) return NAJU_OK;
    if (d_in > 0) {
        NAJU_TRY(need(x, "x", 2));
        NAJU_TRY(need(qweight, "qweight", 1));
        NAJU_TRY(need(scales, "scales", 2));
    }
    NAJU_TRY(opt(bias, "bias", 4));
    NAJU_TRY(opt(res, "res", 2));
    NAJU_TRY(need(y, "y", 2));
    const W4Args g{rows, d_in, d_out, (d_in + group - 1) / group, (const bf16 *)x, qweight,
                   (const bf16 *)scales, zeros, bias, (const bf16 *)res, (bf16 *)y};
    hipStream_t st = (hipStream_t)stream;
    return hip_status(group == 32 ? launch_w4<32>(g, st)
                                  : group == 64 ? launch_w4<64>(g, st) : launch_w4<128>(g, st),
                      "4-bit linear launch");
}

}  // extern "C"
