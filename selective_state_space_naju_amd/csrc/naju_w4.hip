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

// One workgroup: WN = kW4Waves / WK tiles of 16 outputs; the WK waves of a tile
// take every WK-th block of 128 inputs.  RT: tiles of 16 rows of x; G: inputs of
// a group; D: blocks whose codes a wave holds or has in flight; Z: zeros are
// given.
//
// x and the outputs' scales and zeros are staged in LDS, `stage` inputs at a time
// (a multiple of 128 WK D): all of them where they fit, so that nothing but the
// codes is waited for.  Rows past the last one are not staged: lanes that stand
// for them compute what nobody stores.
//
// Four neighbouring lanes load the 64 bytes of one weight row, and the block
// passes through 1 KB of LDS of its wave into the product's layout (a lane for
// each output and quarter).  Loaded in that layout directly, every lane of a
// quarter wave touches a line of its own, and address processing bounds the
// kernel (one row of x, 4096 -> 131072: 76 us, the address units 80 % busy).
//
// The loads of whole blocks are unconditional (past the last one they repeat
// it): a load that is issued under a condition makes the compiler wait for the
// ones in flight where the branches meet.
template <int RT, int G, int WK, int D, bool Z>
__global__ __launch_bounds__(kW4Threads) void w4_kernel(const W4Args g, const int stage)
{
    constexpr int WN = kW4Waves / WK;
    constexpr int NG = 128 / G;  // groups of a block
    constexpr int NR = WN * 16;  // outputs of the workgroup
    extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = w % WK, wn = w / WK, col = lane & 15, quarter = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * NR;  // first output
    const int64_t n = n0 + wn * 16 + col;
    const int64_t r0 = (int64_t)blockIdx.y * (RT * 16);
    const int rows = g.R - r0 < RT * 16 ? (int)(g.R - r0) : RT * 16;
    const int outs = g.N - n0 < NR ? (int)(g.N - n0) : NR;
    const int pitch = stage + 8;               // of a staged row: the pad spreads the banks
    const int groups = stage / G;              // of a stage
    uint32_t *slot = lds + w * 256;            // this wave's block of codes
    bf16 *xs = (bf16 *)(lds + kW4Waves * 256);            // [rows][pitch]
    float *sx = (float *)(xs + rows * pitch);             // [groups][RT * 16]: sums of x
    bf16 *sl = (bf16 *)(sx + groups * (RT * 16));         // [groups][NR]: scales
    uint8_t *zl = (uint8_t *)(sl + groups * NR);          // [groups][NR]: zeros

    f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    int xrow[RT];  // where this lane's row of a tile is staged
#pragma unroll
    for (int t = 0; t < RT; ++t)
        xrow[t] = (t * 16 + col < rows ? t * 16 + col : rows - 1) * pitch + quarter * 8;

    // codes: lane l loads 16 bytes of row l / 4 of the tile (past the last output: of that one)
    const int lrow = wn * 16 + (lane >> 2) < outs ? wn * 16 + (lane >> 2) : outs - 1;
    const uint32_t loff = (uint32_t)lrow * (uint32_t)(g.K / 2) + (lane & 3) * 16;
    const uint8_t *qtile = g.q + n0 * (g.K / 2);
    const int64_t whole = g.K / 128 * 128;  // inputs in whole blocks
    u32x4 d[D];
    auto fetch = [&](int u, int64_t k) {
        k = k < whole ? k : whole - 128;
        __builtin_memcpy(&d[u], qtile + k / 2 + loff, 16);
    };
    // a loaded block in the product's layout; within the slot a row's four parts are rotated by
    // a quarter of its number, which spreads the banks of the read
    const int put = (lane >> 2) * 4 + (((lane & 3) + (lane >> 4)) & 3);
    const int get = col * 4 + ((quarter + (col >> 2)) & 3);
    auto arrange = [&](const u32x4 v) {
        ((u32x4 *)slot)[put] = v;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const u32x4 r = ((const u32x4 *)slot)[get];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        return transpose_quarters(r);
    };
    // the products of a block of 128 inputs, c0 inputs into the stage
    auto block = [&](const u32x4 t4, int c0) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            f32x4 p[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) p[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = i * (G / 32); j < (i + 1) * (G / 32); ++j) {
                const bf16x8 wv = unpack(t4[j]);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const bf16x8 xv = *(const bf16x8 *)(xs + xrow[t] + c0 + j * 32);
                    p[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, wv, p[t], 0, 0, 0);
                }
            }
            const int gi = c0 / G + i;
            const float sc = to_f(sl[gi * NR + wn * 16 + col]);
            const float cz = Z ? 128.f + (float)zl[gi * NR + wn * 16 + col] : 136.f;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const f32x4 tot = *(const f32x4 *)&sx[gi * (RT * 16) + t * 16 + quarter * 4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[t][q] = fmaf(sc, fmaf(-cz, tot[q], p[t][q]), acc[t][q]);
            }
        }
    };
    if (whole > 0) {
#pragma unroll
        for (int u = 0; u < D; ++u) fetch(u, (int64_t)(u * WK + wk) * 128);
    }
    constexpr int turn = 128 * WK * D;
    for (int64_t s0 = 0; s0 < g.K; s0 += stage) {
        if (s0) __syncthreads();
        // stage x[r0 ..][s0 .. s0 + stage), and its sums over the groups; zeros past the inputs
        const int64_t avail = (g.K - s0 + 127) / 128 * 128;
        const int runs = (int)(avail < stage ? avail : stage) / 8;
        for (int i = tid; i < rows * runs; i += kW4Threads) {
            const int m = i / runs, c = (i - m * runs) * 8;
            Run<bf16, 8> v;
            const bf16 *src = g.x + (r0 + m) * g.K + s0 + c;
            const int64_t left = g.K - s0 - c;
            if (left >= 8) v.load(src);
            else if (left > 0) v.load_part(src, (int)left);
            else v.zero();
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) sum += v.get(q);
            sum = quad_sum(sum);
            if constexpr (G >= 64) sum += __shfl_xor(sum, 4);
            if constexpr (G >= 128) sum += __shfl_xor(sum, 8);
            u32x4 o;  // pairs (0, 4) (1, 5) (2, 6) (3, 7)
            o[0] = __builtin_amdgcn_perm(v.w[2], v.w[0], 0x05040100);
            o[1] = __builtin_amdgcn_perm(v.w[2], v.w[0], 0x07060302);
            o[2] = __builtin_amdgcn_perm(v.w[3], v.w[1], 0x05040100);
            o[3] = __builtin_amdgcn_perm(v.w[3], v.w[1], 0x07060302);
            *(u32x4 *)(xs + m * pitch + c) = o;
            if (c % G == 0) sx[c / G * (RT * 16) + m] = sum;
        }
        // the outputs' scales and zeros, 8 groups a thread; none past the last group
        const int g0 = (int)(s0 / G), sets = (runs * 8 / G + 7) / 8;
        for (int i = tid; i < outs * sets; i += kW4Threads) {
            const int m = i / sets, c = (i - m * sets) * 8;
            const int64_t at = (n0 + m) * g.ng + g0 + c;
            const int left = (int)(g.ng - g0) - c;
            Run<bf16, 8> v;
            Run<uint8_t, 8> zv;
            v.zero();
            zv.zero();
            if (left >= 8) {
                v.load(g.scales + at);
                if (Z) zv.load(g.zeros + at);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (c + q >= groups) continue;
                const bool alone = left < 8 && q < left;
                sl[(c + q) * NR + m] = alone ? g.scales[at + q] : v.get_raw(q);
                if (Z)
                    zl[(c + q) * NR + m] =
                        alone ? g.zeros[at + q] : (uint8_t)(zv.w[q / 4] >> (8 * (q % 4)));
            }
        }
        __syncthreads();
        const int64_t s1 = s0 + stage < g.K ? s0 + stage : g.K;
        int64_t k1 = s0;
        for (; k1 + turn <= whole && k1 < s1; k1 += turn) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                const int64_t k = k1 + (u * WK + wk) * 128;
                const u32x4 t4 = arrange(d[u]);
                // what the next load overwrites is used up, and it is issued here: left to
                // itself the scheduler collects the loads at the end of the loop and waits there
                __builtin_amdgcn_sched_barrier(0);
                fetch(u, k + turn);
                __builtin_amdgcn_sched_barrier(0);
                block(t4, (int)(k - s0));
            }
        }
        if (k1 >= s1) continue;
        // the last turn: the blocks in hand, and the one cut short by the end of the inputs,
        // of which nothing past that end is read
#pragma unroll
        for (int u = 0; u < D; ++u) {
            const int64_t k = k1 + (u * WK + wk) * 128;
            if (k < whole) {
                block(arrange(d[u]), (int)(k - s0));
            } else if (k < g.K) {
                u32x4 t = {0, 0, 0, 0};
                const int left = (int)(g.K - k) / 2 - (lane & 3) * 16;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < left) t[j / 4] |= (uint32_t)qtile[k / 2 + loff + j] << (8 * (j % 4));
                block(arrange(t), (int)(k - s0));
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

template <int RT, int G, int WK, int D, bool Z>
static hipError_t launch_w4_t(const W4Args &g, hipStream_t st)
{
    constexpr int per = (kW4Waves / WK) * 16;
    constexpr int64_t unit = 128 * WK * D;  // inputs of a turn of the ring
    constexpr int64_t budget = 78 << 10;    // two workgroups on a CU
    const int64_t rows = g.R < RT * 16 ? g.R : RT * 16;
    // LDS of `s` staged inputs: the waves' blocks; rows of x; per group RT * 16 sums and `per`
    // scales and zeros
    auto bytes = [&](int64_t s) {
        return 1024 * kW4Waves + rows * (s + 8) * 2 + s / G * (RT * 16 * 4 + per * (Z ? 3 : 2));
    };
    const int64_t all = (g.K + unit - 1) / unit * unit;
    int64_t stage = unit;
    while (stage < all && bytes(stage + unit) <= budget) stage += unit;
    int64_t lds = bytes(stage);
    const int64_t red = WK > 1 ? kW4Waves * RT * 256 * 4 : 0;
    if (lds < red) lds = red;
    // (above 64 KB a kernel has to ask for its LDS)
    if (lds > (64 << 10)) {
        const hipError_t e =
            hipFuncSetAttribute((const void *)w4_kernel<RT, G, WK, D, Z>,
                                hipFuncAttributeMaxDynamicSharedMemorySize, 160 << 10);
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)((g.N + per - 1) / per), (unsigned)((g.R + RT * 16 - 1) / (RT * 16)));
    hipLaunchKernelGGL((w4_kernel<RT, G, WK, D, Z>), grid, dim3(kW4Threads), (size_t)lds, st, g,
                       (int)stage);
    return hipGetLastError();
}

template <int G, bool Z> static hipError_t launch_w4_z(const W4Args &g, hipStream_t st)
{
    // few outputs: the waves of a workgroup split the inputs of a tile
    const bool split = g.N < 16 * 8 * 512;
    if (g.R <= 16)
        return split ? launch_w4_t<1, G, 4, 4, Z>(g, st) : launch_w4_t<1, G, 1, 4, Z>(g, st);
    if (g.R <= 32)
        return split ? launch_w4_t<2, G, 4, 2, Z>(g, st) : launch_w4_t<2, G, 1, 4, Z>(g, st);
    return split ? launch_w4_t<4, G, 2, 2, Z>(g, st) : launch_w4_t<4, G, 1, 4, Z>(g, st);
}
template <int G> static hipError_t launch_w4(const W4Args &g, hipStream_t st)
{
    return g.zeros ? launch_w4_z<G, true>(g, st) : launch_w4_z<G, false>(g, st);
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
