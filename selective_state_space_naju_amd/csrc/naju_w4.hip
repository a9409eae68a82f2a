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
//
// 4096 -> 131072, groups of 128: one row 51 us (5.3 TB/s of codes), 32 rows
// 79 us and 64 rows 157 us, where unpacking and the LDS reads of x come to more
// than the codes.
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

// 8 codes as the bf16 numbers 128 + q, in the order 0 4 1 5 2 6 3 7.  `ones` holds
// 0x43004300 in a register: with one constant of its own the instruction can
// mask and or at once.
__device__ __forceinline__ bf16x8 unpack(uint32_t d, uint32_t ones)
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ((d >> (4 * i)) & 0x000f000fu) | ones;
    return __builtin_bit_cast(bf16x8, r);
}

// One workgroup: WN = kW4Waves / WK sets of 16 NT outputs; the WK waves of a set
// take every WK-th block of 128 inputs.  RT: tiles of 16 rows of x; P: rows of x
// that LDS has room for (lanes that stand for more repeat some); NT: tiles of
// 16 outputs that a wave multiplies with the same x; G: inputs of a group; D: blocks whose codes a wave holds or has in flight; Z: zeros are
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
template <int RT, int P, int G, int WK, int NT, int D, bool Z>
__global__ __launch_bounds__(kW4Threads, 4) void w4_kernel(const W4Args g, const int stage,
                                                           const FastDiv by_rows)
{
    constexpr int WN = kW4Waves / WK;
    constexpr int NG = 128 / G;  // groups of a block
    constexpr int NR = WN * NT * 16;  // outputs of the workgroup
    extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = w % WK, wn = w / WK, col = lane & 15, quarter = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * NR;  // first output
    const int o0 = wn * NT * 16;                  // the wave's first among them
    const int64_t r0 = (int64_t)blockIdx.y * (RT * 16);
    const int rows = g.R - r0 < RT * 16 ? (int)(g.R - r0) : RT * 16;
    const int outs = g.N - n0 < NR ? (int)(g.N - n0) : NR;
    const int groups = stage / G;              // of a stage
    uint32_t *slot = lds + w * 256;            // this wave's block of codes
    // staged x: [stage / 8][P][8].  Row m of the 8 inputs from c stands at m ^ (c / 32 % 4): the
    // lanes of a staging write, one row's neighbouring inputs, would otherwise all meet one bank
    bf16 *xs = (bf16 *)(lds + kW4Waves * 256);
    float *sx = (float *)(xs + P * stage);                // [groups][P]: sums of x
    bf16 *sl = (bf16 *)(sx + groups * P);         // [groups][NR]: scales
    uint8_t *zl = (uint8_t *)(sl + groups * NR);          // [groups][NR]: zeros

    f32x4 acc[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int v = 0; v < NT; ++v) acc[t][v] = f32x4{0.f, 0.f, 0.f, 0.f};
    int xrow[4];  // where this lane's row and quarter of the j-th 32 inputs is staged
#pragma unroll
    for (int j = 0; j < 4; ++j) xrow[j] = ((j * 4 + quarter) * P + ((col & (P - 1)) ^ j)) * 8;

    // codes: lane l loads 16 bytes of row l / 4 of the tile (past the last output: of that one)
    uint32_t loff[NT];
#pragma unroll
    for (int v = 0; v < NT; ++v) {
        const int o = o0 + v * 16 + (lane >> 2);
        loff[v] = (uint32_t)(o < outs ? o : outs - 1) * (uint32_t)(g.K / 2) + (lane & 3) * 16;
    }
    const uint8_t *qtile = g.q + n0 * (g.K / 2);
    const int64_t whole = g.K / 128 * 128;  // inputs in whole blocks
    u32x4 d[D][NT];
    auto fetch = [&](int u, int64_t k) {
        k = k < whole ? k : whole - 128;
#pragma unroll
        for (int v = 0; v < NT; ++v) __builtin_memcpy(&d[u][v], qtile + k / 2 + loff[v], 16);
    };
    // a loaded block in the product's layout.  Within the slot a row's four parts are exchanged
    // by the row's number / 4, so that neither the write nor the read meets a bank twice
    auto part = [](int row, int p) { return row * 4 + ((row >> 2) ^ (p & 1 ? 3 : 0) ^ (p >> 1)); };
    const int put = part(lane >> 2, lane & 3), get = part(col, quarter);
    auto arrange = [&](u32x4 (&r)[NT], const u32x4 (&in)[NT]) {
#pragma unroll
        for (int v = 0; v < NT; ++v) {
            ((u32x4 *)slot)[put] = in[v];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            r[v] = ((const u32x4 *)slot)[get];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    };
    uint32_t ones = 0x43004300u;
    asm volatile("" : "+v"(ones));
    // the products of a block of 128 inputs, c0 inputs into the stage
    auto block = [&](const u32x4 (&t4)[NT], int c0) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            f32x4 p[RT][NT];
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int v = 0; v < NT; ++v) p[t][v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = i * (G / 32); j < (i + 1) * (G / 32); ++j) {
                bf16x8 wv[NT];
#pragma unroll
                for (int v = 0; v < NT; ++v) wv[v] = unpack(t4[v][j], ones);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const bf16x8 xv = *(const bf16x8 *)(xs + c0 * P + xrow[j] + t * 128);
#pragma unroll
                    for (int v = 0; v < NT; ++v)
                        p[t][v] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, wv[v], p[t][v], 0, 0, 0);
                }
            }
            const int gi = c0 / G + i;
            float sc[NT], cz[NT];
#pragma unroll
            for (int v = 0; v < NT; ++v) {
                sc[v] = to_f(sl[gi * NR + o0 + v * 16 + col]);
                cz[v] = Z ? 128.f + (float)zl[gi * NR + o0 + v * 16 + col] : 136.f;
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const f32x4 tot = *(const f32x4 *)&sx[gi * P + t * 16 + (quarter * 4 & (P - 1))];
#pragma unroll
                for (int v = 0; v < NT; ++v)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        acc[t][v][q] =
                            fmaf(sc[v], fmaf(-cz[v], tot[q], p[t][v][q]), acc[t][v][q]);
            }
        }
    };
    if (whole > 0) {
#pragma unroll
        for (int u = 0; u < D; ++u) fetch(u, (int64_t)(u * WK + wk) * 128);
    }
    constexpr int turn = 128 * WK * D;
    // the block that comes next is passed through the slot while one is multiplied
    u32x4 next[NT] = {};
    if (whole > 0) arrange(next, d[0]);
    for (int64_t s0 = 0; s0 < g.K; s0 += stage) {
        if (s0) __syncthreads();
        // stage x[r0 ..][s0 .. s0 + stage), and its sums over the groups; zeros past the inputs
        const int64_t avail = (g.K - s0 + 127) / 128 * 128;
        const int runs = (int)(avail < stage ? avail : stage) / 8;
        // Rows of 512 inputs are dealt out to the waves, F of them in flight.  Where the waves
        // split the inputs, a stage is most of a call: four rows, and the first scales and zeros
        // asked for before them (5 x 4100 -> 7001: 13.9 -> 13.0 us; elsewhere the registers cost
        // more: 16 x 4096 -> 131072 took 6 % longer).
        constexpr bool kAhead = WK > 1;
        constexpr int F = RT == 1 && kAhead ? 4 : 2 * RT;
        const int g0 = (int)(s0 / G), sets = (runs * 8 / G + 7) / 8;
        Run<bf16, 8> sv;
        Run<uint8_t, 8> zv;
        auto ask = [&](int i) {
            sv.zero();
            zv.zero();
            const int m = i / sets, c = (i - m * sets) * 8;
            const int64_t at = (n0 + m) * g.ng + g0 + c;
            if (i < outs * sets && g.ng - g0 - c >= 8) {
                sv.load(g.scales + at);
                if (Z) zv.load(g.zeros + at);
            }
        };
        if (kAhead) ask(tid);
        const int64_t left = g.K - s0;
        const int parts = (int)by_rows.d * ((runs + 63) / 64);
        const bf16 *src = g.x + r0 * g.K + s0;
        for (int p0 = w; p0 < parts; p0 += kW4Waves * F) {
            Run<bf16, 8> v[F];
            int m[F], c[F];
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const int p = p0 + i * kW4Waves < parts ? p0 + i * kW4Waves : p0;
                const int cb = (int)fdiv((uint32_t)p, by_rows);
                m[i] = p - cb * (int)by_rows.d;
                c[i] = cb * 512 + lane * 8;
                const bf16 *at = src + m[i] * g.K;
                if (m[i] >= rows) v[i].zero();  // (the last rows' workgroups have fewer)
                else if (c[i] + 8 <= left) v[i].load(at + c[i]);
                else if (c[i] < left) v[i].load_part(at + c[i], (int)(left - c[i]));
                else v[i].zero();
            }
#pragma unroll
            for (int i = 0; i < F; ++i) {
                if (p0 + i * kW4Waves >= parts) break;  // (uniform)
                float sum = 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q) sum += v[i].get(q);
                sum = quad_sum(sum);
                if constexpr (G >= 64) sum += __shfl_xor(sum, 4);
                if constexpr (G >= 128) sum += __shfl_xor(sum, 8);
                if (c[i] >= runs * 8 || m[i] >= rows) continue;
                u32x4 o;  // pairs (0, 4) (1, 5) (2, 6) (3, 7)
                o[0] = __builtin_amdgcn_perm(v[i].w[2], v[i].w[0], 0x05040100);
                o[1] = __builtin_amdgcn_perm(v[i].w[2], v[i].w[0], 0x07060302);
                o[2] = __builtin_amdgcn_perm(v[i].w[3], v[i].w[1], 0x05040100);
                o[3] = __builtin_amdgcn_perm(v[i].w[3], v[i].w[1], 0x07060302);
                *(u32x4 *)(xs + c[i] * P + (m[i] ^ ((c[i] >> 5) & 3)) * 8) = o;
                if (c[i] % G == 0) sx[c[i] / G * P + m[i]] = sum;
            }
        }
        // the outputs' scales and zeros, 8 groups a thread; none past the last group
        for (int i = tid; i < outs * sets; i += kW4Threads) {
            if (!kAhead || i != tid) ask(i);
            const int m = i / sets, c = (i - m * sets) * 8;
            const int64_t at = (n0 + m) * g.ng + g0 + c;
            const int left = (int)(g.ng - g0) - c;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (c + q >= groups) continue;
                const bool alone = left < 8 && q < left;
                sl[(c + q) * NR + m] = alone ? g.scales[at + q] : sv.get_raw(q);
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
                u32x4 t4[NT];
#pragma unroll
                for (int v = 0; v < NT; ++v) t4[v] = transpose_quarters(next[v]);
                arrange(next, d[(u + 1) % D]);
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
                u32x4 t4[NT];
#pragma unroll
                for (int v = 0; v < NT; ++v) t4[v] = transpose_quarters(next[v]);
                if (u + 1 < D) arrange(next, d[u + 1 < D ? u + 1 : 0]);
                block(t4, (int)(k - s0));
            } else if (k < g.K) {
                u32x4 t4[NT] = {};
                const int left = (int)(g.K - k) / 2 - (lane & 3) * 16;
#pragma unroll
                for (int v = 0; v < NT; ++v)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < left)
                            t4[v][j / 4] |= (uint32_t)qtile[k / 2 + loff[v] + j] << (8 * (j % 4));
                arrange(t4, t4);
#pragma unroll
                for (int v = 0; v < NT; ++v) t4[v] = transpose_quarters(t4[v]);
                block(t4, (int)(k - s0));
            }
        }
    }

    // the waves of an output tile add their sums in order
    if constexpr (WK > 1) {
        f32x4 *red = (f32x4 *)lds;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int v = 0; v < NT; ++v) red[((w * RT + t) * NT + v) * 64 + lane] = acc[t][v];
        __syncthreads();
        if (wk != 0) return;
#pragma unroll
        for (int i = 1; i < WK; ++i)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int v = 0; v < NT; ++v)
                    acc[t][v] += red[(((w + i) * RT + t) * NT + v) * 64 + lane];
    }
#pragma unroll
    for (int v = 0; v < NT; ++v) {
        const int64_t n = n0 + o0 + v * 16 + col;
        if (n >= g.N) continue;
        const float bias = g.bias ? g.bias[n] : 0.f;
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t r = r0 + t * 16 + quarter * 4 + q;
                if (r >= g.R) continue;
                float y = acc[t][v][q] + bias;
                if (g.res) y += to_f(g.res[r * g.N + n]);
                g.y[r * g.N + n] = from_f<bf16>(y);
            }
    }
}

// LDS of `s` staged inputs: the waves' blocks; P rows of x; per group P sums, and scales and
// zeros of the workgroup's outputs
constexpr int64_t w4_lds(int P, int G, int WK, int NT, bool Z, int64_t s)
{
    const int per = (kW4Waves / WK) * NT * 16;
    return 1024 * kW4Waves + P * s * 2 + s / G * (P * 4 + per * (Z ? 3 : 2));
}
constexpr int64_t kHalfLds = 80 << 10;

// DEPTH: blocks whose codes a wave holds, or half of them where a turn of that many would not
// leave a CU room for a second workgroup (groups of 32 with zeros, four and two, us: 64 x 4096 ->
// 131072 268 and 250, 64 x 1000 -> 33000 46 and 38, 16 x 4096 -> 16384 27 and 22)
template <int RT, int P, int G, int WK, int NT, int DEPTH, bool Z>
static hipError_t launch_w4_t(const W4Args &g, hipStream_t st)
{
    constexpr int per = (kW4Waves / WK) * NT * 16;
    constexpr int D = w4_lds(P, G, WK, NT, Z, 128 * WK * DEPTH) <= kHalfLds ? DEPTH : DEPTH / 2;
    constexpr int64_t unit = 128 * WK * D;  // inputs of a turn of the ring
    static_assert(w4_lds(P, G, WK, NT, Z, unit) <= kHalfLds, "two workgroups share a CU");
    const int64_t rows = g.R < RT * 16 ? g.R : RT * 16;
    const int64_t wgs = (g.N + per - 1) / per * ((g.R + RT * 16 - 1) / (RT * 16));
    // two workgroups on a CU, or one where there are not more than that
    const int64_t budget = wgs <= device_cu_count() ? 150 << 10 : kHalfLds;
    auto bytes = [](int64_t s) { return w4_lds(P, G, WK, NT, Z, s); };
    // all inputs at once if they fit, else whole turns of the ring
    int64_t stage = (g.K + 127) / 128 * 128;
    if (stage == 0) stage = 128;
    if (bytes(stage) > budget) {
        stage = unit;
        while (bytes(stage + unit) <= budget) stage += unit;
    }
    int64_t lds = bytes(stage);
    const int64_t red = WK > 1 ? kW4Waves * RT * NT * 256 * 4 : 0;
    if (lds < red) lds = red;
    // (above 64 KB a kernel has to ask for its LDS)
    if (lds > (64 << 10)) {
        const hipError_t e =
            hipFuncSetAttribute((const void *)w4_kernel<RT, P, G, WK, NT, D, Z>,
                                hipFuncAttributeMaxDynamicSharedMemorySize, 160 << 10);
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)((g.N + per - 1) / per), (unsigned)((g.R + RT * 16 - 1) / (RT * 16)));
    hipLaunchKernelGGL((w4_kernel<RT, P, G, WK, NT, D, Z>), grid, dim3(kW4Threads), (size_t)lds, st, g,
                       (int)stage, make_fastdiv((uint32_t)rows));
    return hipGetLastError();
}

template <int G, bool Z> static hipError_t launch_w4_z(const W4Args &g, hipStream_t st)
{
    // few outputs: the waves of a workgroup split the inputs of a tile (4096 inputs, groups of
    // 128, split and not, us:
    //   rows    14336 outputs    24576          32000          131072
    //    1      11 and 15        17 and 17      20 and 17      65 and 51
    //    8      14 and 18        22 and 20      26 and 20      92 and 63
    //   16      19 and 21        29 and 23      35 and 24      124 and 65
    //   32      29 and 40        47 and 43      55 and 44      202 and 78
    //   64      42 and 49        62 and 51      63 and 53      228 and 157)
    const bool split = g.N < 24576;
    if (g.R <= 4)
        return split ? launch_w4_t<1, 4, G, 4, 1, 4, Z>(g, st)
                     : launch_w4_t<1, 4, G, 1, 1, 4, Z>(g, st);
    if (g.R <= 8)
        return split ? launch_w4_t<1, 8, G, 4, 1, 4, Z>(g, st)
                     : launch_w4_t<1, 8, G, 1, 1, 4, Z>(g, st);
    if (g.R <= 16)
        return split ? launch_w4_t<1, 16, G, 4, 1, 4, Z>(g, st)
                     : launch_w4_t<1, 16, G, 1, 1, 4, Z>(g, st);
    if (g.R <= 32)
        return split ? launch_w4_t<2, 32, G, 4, 1, 2, Z>(g, st)
                     : launch_w4_t<2, 32, G, 1, 2, 2, Z>(g, st);
    return split ? launch_w4_t<4, 64, G, 2, 1, 2, Z>(g, st)
                 : launch_w4_t<4, 64, G, 1, 1, 4, Z>(g, st);
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
        // (divided first where the difference would leave fp32)
        const float span = hi - lo;
        const float step = span < __builtin_huge_valf() ? span / 15.f : hi / 15.f - lo / 15.f;
        const bf16 sb = from_f<bf16>(zeros ? step : fmaxf(hi, -lo) / 7.f);
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
