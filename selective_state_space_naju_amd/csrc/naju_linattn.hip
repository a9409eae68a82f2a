// naju_linattn.hip -- linear attention with a decay for each head: chunked for
// prompts and training (forward and gradients), recurrent for single tokens.
//
//     S_t = l S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   l = exp(log_decay)
// Over a chunk of tokens that the state S enters, i and j counted from 0:
//     O_i = scale ( sum_{j <= i} l^{i-j} (q_i . k_j) v_j + l^{i+1} S^T q_i )
//     S'  = l^T S + sum_j l^{T-1-j} k_j v_j^T
// so all of it is matrix products; powers of l are formed from differences of
// positions and never exceed 1 for l <= 1.
//
// The gradients are the same walk with other operands.  With G = dO:
//     dq_i = scale sum_{j <= i} l^{i-j} (G_i . v_j) k_j + ...   (G, v, k), state S^T
//     dv_j = scale sum_{i >= j} l^{i-j} (k_j . q_i) G_i + ...   (k, q, G), back in time
//     dk_j = scale sum_{i >= j} l^{i-j} (v_j . G_i) q_i + ...   (v, G, q), back in time
// where the state walking back is M <- l (M + scale q_t G_t^T), from the gradient of
// the last state to that of the first: it enters a chunk already decayed, so its
// powers of l are one lower than the forward walk's (`late` 0 in place of 1).
//
// One workgroup walks one head of one batch row over a stretch of chunks, for 64 or
// 128 of the value columns, with its part of the state in the accumulators of its
// four waves from chunk to chunk.  A wave owns 16 CT columns: the state's tiles come
// out of the matrix instruction with a column in each lane and four rows in its
// registers, which is also the layout of an operand, so the product with q reads the
// state from registers.  Scores are shared through LDS.  Where heads and rows are too
// few for the CUs the sequence is cut into segments: their own contributions to the
// state first, the entering states from those, then the walk over all segments at
// once.
//
// bf16: v_mfma_f32_16x16x32_bf16 with fp32 sums; scores and state enter products as
// bf16 hi + lo (2^-16), the decayed values of the state's sum in three bf16 parts
// (fp32's precision: the state is an fp32 output).  fp32: v_mfma_f32_16x16x4_f32.
//
// Bound by a chunk's length in time: its loads, two barriers and three rounds of
// products follow one another, and registers leave room for two workgroups a CU to
// cover that.  8 x 2048 x 64 heads x 128 (a full chip) forward 290 us, 3.7 TB/s of its
// inputs and outputs; few heads are cut into segments, which read k and v twice (both
// times from beyond L2, by counter): 65536 x 16 x 128 forward 422 us (2.5 TB/s), 8 x 2048 x
// 12 x 128 gradient 224 us (its three walks read 348 MB from beyond L2, the four tensors
// once are 201); fp32 3 x 333 x 5 heads of 40 and 72 forward 17 us in a graph.  Not faster in
// the same place (the base there 282 us, or as given): eight waves of 16 columns (330 us, one
// workgroup a CU), LDS reads a step ahead of the products (345, one workgroup a CU; two
// spill), splitting values by hand between the products (334), loads that bypass the
// caches (332 to 341).
#include <math.h>

#include "naju_device.h"
#include "naju_host.h"
#include "naju_launch.h"
#include "naju_vec.h"

namespace naju {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kLinMost = 256;      // elements of a head's keys or values
constexpr int kLinThreads = 256;
constexpr int64_t kLinStride = (int64_t)1 << 20;  // elements from token to token: a chunk's tokens
                                                  // span 2^28 bytes at most

// A number as if it were new: what was formed from it before is not kept in registers for later.
__device__ __forceinline__ int anew(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// One walk.  The names are the forward's: q reads, k and v are summed into the state.
struct LinJob {
    const void *q, *k, *v;
    void *o;
    const float *enter;      // states entering the segments, or the first; null: zeros
    float *leave;            // segments' contributions, or the last state; may be null
    int64_t ldq, ldk, ldv, ldo;         // elements from token to token
    int64_t bq, bk, bv;                 // from batch row to batch row
    int64_t enter_bh, enter_seg, leave_bh, leave_seg;
    int enter_r, enter_c, leave_r, leave_c;  // element (row, column) of a state
    int D1, D2;              // rows (q's and k's elements) and columns (v's) of the state
    int gq, gk, gv;          // heads that share one of q, k, v
    float s_row, s_pair, s_tok;         // scales of S^T q, of the scores, of k v^T
    int late;
    int back;                // 1: from each row's last token to its first
};

struct LinArgs {
    LinJob job[3];
    const float *log_decay;
    const int32_t *lengths;
    int B, H, slices, nseg, seg;        // seg: tokens of a segment
    int jobs, items;                    // walks, and workgroups of each
    int64_t L;
};

// ------------------------------------------------------- operands of the products
// An operand in a lane: row l % 16 of 16, and 8 of 32 elements, those in the slots 8 h .. 8 h + 7 of
// its quarter h = l / 16.  Both operands of a product put the same elements into the same slots,
// in any order: where elements are tokens, and in products with the state, slot 8 h + j holds
// element slot_step(j) + 4 h, the order in which the matrix instruction leaves two tiles of 16
// rows in a lane's registers.
//
// Rows of LDS tiles lie 32 bytes further in the 64 banks than the one before.  Cycles of one
// wave's access with eight waves at it: transposing reads 7 whichever columns the lanes take,
// 16-byte reads of 16 rows 8; two 8-byte reads of 16 rows (slot_step's order) 32, and 16 where rows
// lie 16 bytes further.  Those read q alone; rows 16 bytes further, or 16-byte reads of a second
// order of k, made the walk slower all the same (362 to 390 us against 366).
__device__ __forceinline__ constexpr int slot_step(int j) { return 16 * (j >> 2) + (j & 3); }

template <typename T> struct Frag;

template <> struct Frag<bf16> {
    bf16x8 f;
    // 8 neighbouring elements of the 32 from p on
    __device__ __forceinline__ void row(const bf16 *p, int h) { f = *(const bf16x8 *)(p + 8 * h); }
    __device__ __forceinline__ void scores(const bf16 *p, int h) { row(p, h); }
    // those of slot_step
    __device__ __forceinline__ void split_row(const bf16 *p, int h)
    {
        const bf16x4 a = *(const bf16x4 *)(p + 4 * h), b = *(const bf16x4 *)(p + 4 * h + 16);
        f = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // Transposed: element j of the lane is its column of row slot_step(j) behind the first.
    // ds_read_tr16_b64: lane i of 16 hands in row i / 4 (of four) and columns
    // 4 (i % 4) .. + 3 of its choice, and receives column i of all four rows.
    __device__ __forceinline__ void cols(const bf16 *p, int stride)
    {
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds4 *)(__attribute__((address_space(3))) const bf16 *)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds4 *)(__attribute__((address_space(3))) const bf16 *)(p + 16 * stride));
        const bf16x4 x = __builtin_bit_cast(bf16x4, a), y = __builtin_bit_cast(bf16x4, b);
        f = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    __device__ __forceinline__ float get(int i) const
    {
        const u32x4 w = __builtin_bit_cast(u32x4, f);
        return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};
template <> struct Frag<float> {
    float f[8];
    __device__ __forceinline__ void split_row(const float *p, int h)
    {
        const f32x4 a = *(const f32x4 *)(p + 4 * h), b = *(const f32x4 *)(p + 4 * h + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    }
    __device__ __forceinline__ void row(const float *p, int h) { split_row(p, h); }
    __device__ __forceinline__ void scores(const float *p, int h) { split_row(p, h); }
    // (no transposing read for 32-bit elements: the lane reads its own column)
    __device__ __forceinline__ void cols(const float *p, int stride)
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = p[slot_step(j) * stride];
    }
    __device__ __forceinline__ float get(int i) const { return f[i]; }
};

__device__ __forceinline__ f32x4 mma(const Frag<bf16> &a, const Frag<bf16> &b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.f, b.f, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float> &a, const Frag<float> &b, f32x4 c)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.f[j], b.f[j], c, 0, 0, 0);
    return c;
}

// fp32 values as an operand: P bf16 parts whose sum holds 8 P bits (the first ones cut off, the
// last one rounded), or fp32 as they are
template <typename T, int P> struct Parts;
template <int P> struct Parts<bf16, P> {
    Frag<bf16> p[P];
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        float r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
        for (int n = 0; n < P; ++n) {
            if (n == P - 1) {
                Run<bf16, 8> w = round_run<bf16, 8>(r);
                p[n].f = __builtin_bit_cast(bf16x8, w.w);
            } else {
                u32x4 h;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b0 = __float_as_uint(r[2 * i]);
                    const uint32_t b1 = __float_as_uint(r[2 * i + 1]);
                    h[i] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
                    r[2 * i] -= __uint_as_float(b0 & 0xffff0000u);
                    r[2 * i + 1] -= __uint_as_float(b1 & 0xffff0000u);
                }
                p[n].f = __builtin_bit_cast(bf16x8, h);
            }
        }
    }
};
template <int P> struct Parts<float, P> {
    Frag<float> p[1];
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[0].f[i] = v[i];
    }
};
template <typename T, int P>
__device__ __forceinline__ f32x4 mma(const Parts<T, P> &a, const Frag<T> &b, f32x4 c)
{
    constexpr int n = sizeof(T) == 2 ? P : 1;
#pragma unroll
    for (int i = n - 1; i >= 0; --i) c = mma(a.p[i], b, c);
    return c;
}
template <typename T, int P>
__device__ __forceinline__ f32x4 mma(const Frag<T> &a, const Parts<T, P> &b, f32x4 c)
{
    constexpr int n = sizeof(T) == 2 ? P : 1;
#pragma unroll
    for (int i = n - 1; i >= 0; --i) c = mma(a, b.p[i], c);
    return c;
}

// A raw buffer over [p, p + bytes): loads past the end read 0, stores past the end are dropped (the
// check covers every dword's whole offset).
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes,
                                             0x00020000);
}
// An offset past every buffer here, also with a chunk's length taken off or added
// (a chunk's rows span less than 2^29 bytes).
constexpr uint32_t kPast = 0x80000000u;

// A tile of rows on its way from HBM to LDS, 16 bytes at a time.  Rows are a chunk's tokens in the
// order of the walk; a buffer over the chunk's tokens that there are gives zeros for the others.
template <typename T, int ROWS, int COLS> struct Stage {
    static constexpr int E = 16 / (int)sizeof(T);
    static constexpr int kPerRow = COLS / E;
    static constexpr int N = ROWS * kPerRow / kLinThreads;  // accesses of a thread
    static_assert(ROWS * kPerRow % kLinThreads == 0, "whole accesses");
    static constexpr int kStride = COLS + 2 * E;  // (32 bytes further in the banks)
    static constexpr int kRows = kLinThreads / kPerRow;     // rows from one access to the next
    u32x4 r[N];
    uint32_t off;   // of the first access, in a chunk of ROWS tokens
    uint32_t step;  // to the next (negative where the walk goes back)

    __device__ __forceinline__ void init(int64_t ld, bool back, int D, int tid)
    {
        const uint32_t row_bytes = (uint32_t)ld * (uint32_t)sizeof(T);
        const int row = tid / kPerRow, col = tid % kPerRow * E;
        off = (uint32_t)(back ? ROWS - 1 - row : row) * row_bytes + col * (uint32_t)sizeof(T);
        if (col >= D) off = kPast;
        step = (uint32_t)(back ? -kRows : kRows) * row_bytes;
    }
    // lo: the chunk's lowest token; there: its tokens; moved: offsets' change in a short chunk
    __device__ __forceinline__ void fetch(const T *lo, int64_t ld, int there, uint32_t moved, int tid)
    {
        const rsrc_t b = make_rsrc(lo, (uint32_t)there * (uint32_t)ld * (uint32_t)sizeof(T));
        const int row = tid / kPerRow;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t at = off + moved + i * step;
            if (row + i * kRows >= there) at = kPast;  // (walking back it is below the buffer)
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, 0, 0);
        }
    }
    // zeros in place of what is neither a number nor finite; from[c]: the first row where column c
    // had it, and what was there before if that is less
    __device__ __forceinline__ void clean(int *from, int tid)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int at = e * (int)sizeof(T) / 4;
                const uint32_t own = sizeof(T) == 4 ? ~0u : e % 2 ? 0xffff0000u : 0xffffu;
                const uint32_t exponent = 0x7f807f80u & own & (sizeof(T) == 4 ? 0x7f800000u : ~0u);
                if ((r[i][at] & exponent) == exponent) {
                    r[i][at] &= ~own;
                    atomicMin(from + tid % kPerRow * E + e, tid / kPerRow + i * kRows);
                }
            }
    }
    __device__ __forceinline__ void put(T *lds, int tid) const
    {
        T *to = lds + tid / kPerRow * kStride + tid % kPerRow * E;
#pragma unroll
        for (int i = 0; i < N; ++i) *(u32x4 *)(to + i * kRows * kStride) = r[i];
    }
};

template <typename T, int KD, int CT> struct LinShape {
    static constexpr int TT = sizeof(T) == 2 ? 64 : 32;  // tokens of a chunk
    static constexpr int VC = 64 * CT;                   // columns of a workgroup
    using SK = Stage<T, TT, KD>;
    using SV = Stage<T, TT, VC>;
    static constexpr int E = 16 / (int)sizeof(T);
    static constexpr int kScores = TT + 2 * E;           // stride of the scores
    static constexpr int kParts = sizeof(T) == 2 ? 2 : 1;
    static constexpr size_t bytes(bool out)
    {
        return sizeof(T) * ((out ? 2 : 1) * TT * SK::kStride + TT * SV::kStride +
                            (out ? kParts * TT * kScores : 0)) +
               (out ? sizeof(int) * VC : 0);
    }
};

// One workgroup's walk.  OT: the outputs' type; void: none, a segment's contribution to the state
// alone.  Returns whether it has to be done again with care.
//
// A score of 0 times a value that is not finite is NaN, which so reaches the tokens before it in
// its chunk.  In the state such a value leaves its whole column not finite for good: one look at it
// behind the walk tells, and then the walk is done again: with care, each chunk's bad values are
// taken as 0, and the outputs of their columns from the first of them on are NaN, as is the
// column's last state.  (The loop has nothing of it but one branch behind a barrier, where few
// registers hold anything: 3 % slower to 5 % faster than without it, by what the scheduler makes of
// each form.  Looked for in each chunk's products, or in a second form of the walk in the same
// kernel, it made heads of 128 15 to 25 % slower, in registers that spill.)
template <typename T, int KD, int CT, typename OT>
__device__ __forceinline__ bool linattn_walk(const LinArgs &g, char *lds, const bool care)
{
    using Sh = LinShape<T, KD, CT>;
    constexpr bool OUT = !__is_same(OT, void), wide_out = __is_same(OT, float);
    constexpr int TT = Sh::TT, VC = Sh::VC, IT = TT / 16, KS = TT / 32, KB = KD / 32;
    constexpr int QS = Sh::SK::kStride, VS = Sh::SV::kStride, PS = Sh::kScores;
    T *vs = (T *)lds, *ks = vs + TT * VS, *qs = ks + TT * QS;
    T *ps = qs + TT * QS;  // [parts][TT][PS]
    int *from = (int *)(ps + Sh::kParts * TT * PS);  // [VC] first token whose value is bad

    const int tid = anew(threadIdx.x);
    const int lane = tid & 63, m = lane & 15, h4 = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // jobs of the same segment run on the same XCD (workgroups go round robin over 8 of them)
    int id = blockIdx.x;
    const int jobs = g.jobs;
    const int job = id / 8 % jobs;
    id = id / (8 * jobs) * 8 + id % 8;
    if (id >= g.items) return false;
    const LinJob &J = g.job[job];
    const int slice = id % g.slices;
    id /= g.slices;
    const int seg = id % g.nseg;
    id /= g.nseg;
    const int hd = id % g.H, b = id / g.H;
    const int c0 = slice * VC;
    if (c0 >= J.D2) return false;
    const int D1 = J.D1, D2 = J.D2 - c0 < VC ? J.D2 - c0 : VC;  // of this workgroup
    const int64_t L = g.L;
    int len_i = g.lengths != nullptr ? g.lengths[b] : (int)L;
    len_i = len_i < 0 ? 0 : len_i < (int)L ? len_i : (int)L;
    const int64_t len = __builtin_amdgcn_readfirstlane(len_i);
    const bool back = J.back != 0;
    const int late = J.late;
    const float s_pair = J.s_pair, s_tok = J.s_tok;
    // log2 of the decay; below -1e30 it is 0 after one step, and 0 * -1e30 stays 0
    float a2 = g.log_decay[hd];
    a2 = (a2 < -1e30f ? -1e30f : a2) * kLog2e;

    const int64_t ldq = J.ldq, ldk = J.ldk, ldv = J.ldv;
    const T *q = (const T *)J.q + (int64_t)b * J.bq + (int64_t)(hd / J.gq) * D1;
    const T *k = (const T *)J.k + (int64_t)b * J.bk + (int64_t)(hd / J.gk) * D1;
    const T *v = (const T *)J.v + (int64_t)b * J.bv + (int64_t)(hd / J.gv) * J.D2 + c0;
    const uint32_t out_row = (uint32_t)J.ldo * (wide_out ? 4u : 2u);  // bytes
    char *out = (char *)J.o + (int64_t)b * L * out_row +
                ((int64_t)hd * J.D2 + c0) * (wide_out ? 4 : 2);

    // this lane's columns of the state: 4 CT neighbouring lanes' tiles interleave, so that a
    // lane's outputs of one token are 4 CT consecutive elements
    auto column = [&](int m, int ct) {
        return 16 * CT * w + 4 * CT * (m >> 2) + 4 * ct + (m & 3);
    };
    // rows of the state: register r of tile kt is row 16 kt + 4 h4 + r
    f32x4 S[CT][2 * KB];
    {
        const int ln = anew(lane), m = ln & 15, h4 = ln >> 4;
        const float *e = J.enter;
        if (e != nullptr)
            e += (int64_t)(b * g.H + hd) * J.enter_bh + (int64_t)seg * J.enter_seg;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int kt = 0; kt < 2 * KB; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * kt + 4 * h4 + r;
                    const int col = column(m, ct);
                    float s = 0.f;
                    if (OUT && e != nullptr && row < D1 && col < D2)
                        s = e[(int64_t)row * J.enter_r + (int64_t)(c0 + col) * J.enter_c];
                    S[ct][kt][r] = s;
                }
    }
    // Powers of the decay that every whole chunk takes.
    float lead[IT];     // of S^T q, for this lane's token of each tile
    // scores come in tiles of 16 tokens i by 16 tokens j <= i, dealt out to the waves; then the
    // tiles above the diagonal that a product of 32 tokens takes in, which are zeros
    constexpr int kTiles = IT * (IT + 1) / 2, kAll = kTiles + IT / 2, kOwn = (kAll + 3) / 4;
    float pair[kOwn][4];  // of the scores: scale and power, 0 above the diagonal
    auto tile = [&](int n, int &it, int &jt) {
        const int t = w + 4 * n;
        it = t < kTiles ? (t >= 1) + (t >= 3) + (t >= 6) : 2 * (t - kTiles);
        jt = t < kTiles ? t - it * (it + 1) / 2 : it + 1;
    };
    float tok[8], tok0[KS];  // of k v^T: a product of two, neither exponent negative
#pragma unroll
    for (int j = 0; j < 8; ++j) tok[j] = ex2(a2 * (float)(19 - slot_step(j)));
#pragma unroll
    for (int s = 0; s < KS; ++s) tok0[s] = s_tok * ex2(a2 * (float)(TT - late - 32 * s - 4 * h4 - 19));
    if constexpr (OUT) {
#pragma unroll
        for (int n = 0; n < kOwn; ++n) {
            int it, jt;
            tile(n, it, jt);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int gap = 16 * (it - jt) + m - (4 * h4 + r);
                pair[n][r] = gap >= 0 ? s_pair * ex2(a2 * (float)gap) : 0.f;
            }
        }
#pragma unroll
        for (int it = 0; it < IT; ++it) lead[it] = J.s_row * ex2(a2 * (float)(16 * it + m + late));
    }

    const int64_t first = (int64_t)seg * g.seg;
    const int64_t end = first + g.seg < L ? first + g.seg : L;      // tokens of this segment
    const int64_t stop = end < len ? end : len;                     // those that there are
    typename Sh::SK rq, rk;
    typename Sh::SV rv;
    if constexpr (OUT) rq.init(ldq, back, D1, tid);
    rk.init(ldk, back, D1, tid);
    rv.init(ldv, back, D2, tid);
    auto fetch = [&](int64_t n0) {
        const int there = stop - n0 < TT ? (int)(stop - n0) : TT;
        const int64_t lo = back ? len - n0 - there : n0;
        const uint32_t moved = back ? (uint32_t)(there - TT) : 0u;
        if constexpr (OUT) rq.fetch(q + lo * ldq, ldq, there, moved * (uint32_t)ldq * sizeof(T), tid);
        rk.fetch(k + lo * ldk, ldk, there, moved * (uint32_t)ldk * sizeof(T), tid);
        rv.fetch(v + lo * ldv, ldv, there, moved * (uint32_t)ldv * sizeof(T), tid);
    };
    // where this lane's outputs go, in a chunk of TT tokens: 4 CT elements of tokens m, m + 16, ..
    const int ocol = 16 * CT * w + 4 * CT * h4;
    uint32_t ooff = (uint32_t)(back ? TT - 1 - m : m) * out_row + ocol * (wide_out ? 4 : 2);
    if (ocol >= D2) ooff = kPast;
    const uint32_t ostep = (back ? -16u : 16u) * out_row;

    // with care: the bad outputs of the chunk at n0 (by the lane that stored them)
    auto patch = [&](int64_t n0) {
        const int there = stop - n0 < TT ? (int)(stop - n0) : TT;
        const int ln = anew(lane), from_c = 16 * CT * w + 4 * CT * (ln >> 4);
#pragma unroll 1
        for (int c = from_c; c < from_c + 4 * CT && c < D2; ++c)
#pragma unroll 1
            for (int i = ln & 15; i < there; i += 16) {
                if (i < from[c]) continue;
                const int64_t t = back ? len - 1 - n0 - i : n0 + i;
                if constexpr (wide_out) *(float *)(out + t * out_row + c * 4) = NAN;
                else *(bf16 *)(out + t * out_row + c * 2) = (bf16)0x7fc0;
            }
    };
    if (first < stop) fetch(first);
    for (int64_t n0 = first; n0 < stop; n0 += TT) {
        __syncthreads();  // (the chunk before has been read)
        if (OUT && __builtin_expect(care, 0)) {
            if (n0 > first) patch(n0 - TT);
            __syncthreads();
            const int c = anew(tid);
            if (c < VC) from[c] = n0 > first && from[c] < TT ? 0 : TT;
            __syncthreads();
            rv.clean(from, c);
        }
        if constexpr (OUT) rq.put(qs, tid);
        rk.put(ks, tid);
        rv.put(vs, tid);
        if (n0 + TT < stop) fetch(n0 + TT);
        __syncthreads();
        const int there = stop - n0 < TT ? (int)(stop - n0) : TT;

        if constexpr (OUT) {
            // (transposed: positions of tokens j in a lane's registers)
            f32x4 acc[kOwn];
#pragma unroll
            for (int n = 0; n < kOwn; ++n) {
                acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
                int it, jt;
                tile(n, it, jt);
                if (w + 4 * n < kTiles) {
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        Frag<T> fq, fk;
                        fq.row(qs + (16 * it + m) * QS + 32 * kb, h4);
                        fk.row(ks + (16 * jt + m) * QS + 32 * kb, h4);
                        acc[n] = mma(fk, fq, acc[n]);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < kOwn; ++n) {
                int it, jt;
                tile(n, it, jt);
                if (w + 4 * n < kAll) {
                    float s[4];
                    const int i = 16 * it + m;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        s[r] = pair[n][r] != 0.f ? acc[n][r] * pair[n][r] : 0.f;
                    // (bf16: in the order of the slots, to be read as one run)
                    T *to = ps + i * PS + (sizeof(T) == 2 ? 32 * (jt / 2) + 8 * h4 + 4 * (jt & 1)
                                                          : 16 * jt + 4 * h4);
                    if constexpr (sizeof(T) == 2) {
                        float lo[4];
                        uint32_t hi[2];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            lo[r] = s[r] - __uint_as_float(__float_as_uint(s[r]) & 0xffff0000u);
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            hi[r] = __builtin_amdgcn_perm(__float_as_uint(s[2 * r + 1]),
                                                          __float_as_uint(s[2 * r]), 0x07060302u);
                        __builtin_memcpy(__builtin_assume_aligned(to, 8), hi, 8);
                        const Run<bf16, 4> l = round_run<bf16, 4>(lo);
                        __builtin_memcpy(__builtin_assume_aligned(to + TT * PS, 8), l.w, 8);
                    } else {
                        *(f32x4 *)to = f32x4{s[0], s[1], s[2], s[3]};
                    }
                }
            }
        }

        // values: this wave's columns, slots = tokens
        Frag<T> fv[CT][KS];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if constexpr (sizeof(T) == 2)
                    fv[ct][s].cols(vs + (32 * s + 4 * h4 + (m >> 2)) * VS + 16 * CT * w +
                                       4 * CT * (m & 3) + 4 * ct, VS);
                else
                    fv[ct][s].cols(vs + (32 * s + 4 * h4) * VS + column(m, ct), VS);
            }

        if constexpr (OUT) {
            const int64_t lo = back ? len - n0 - there : n0;
            const rsrc_t ob = make_rsrc(out + lo * out_row, (uint32_t)there * out_row);
            const uint32_t omoved = back ? (uint32_t)(there - TT) * out_row : 0u;
            f32x4 o[IT][CT];
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                Parts<T, 2> st[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    float x[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) x[r] = S[ct][2 * kb + r / 4][r % 4];
                    st[ct].set(x);
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    Frag<T> fq;
                    fq.split_row(qs + (16 * it + m) * QS + 32 * kb, h4);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) o[it][ct] = mma(st[ct], fq, o[it][ct]);
                }
            }
            // (the scores of the other waves: waited for behind the products that do without them)
            __syncthreads();
#pragma unroll
            for (int it = 0; it < IT; ++it) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[it][ct] *= lead[it];
#pragma unroll
                for (int s = 0; s <= it / 2; ++s) {
                    Parts<T, 2> fp;
#pragma unroll
                    for (int n = 0; n < Sh::kParts; ++n)
                        fp.p[n].scores(ps + n * TT * PS + (16 * it + m) * PS + 32 * s, h4);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) o[it][ct] = mma(fv[ct][s], fp, o[it][ct]);
                }
                // (tokens that there are none of lie past the buffer's end)
                const uint32_t at = 16 * it + m < there ? ooff + it * ostep + omoved : kPast;
                if constexpr (wide_out) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(u32x4, o[it][ct]), ob, (int)(at + 16 * ct), 0, 0);
                } else {
                    float x[4 * CT];
#pragma unroll
                    for (int i = 0; i < 4 * CT; ++i) x[i] = o[it][i / 4][i % 4];
                    const Run<bf16, 4 * CT> run = round_run<bf16, 4 * CT>(x);
                    if constexpr (CT == 2)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            u32x4{run.w[0], run.w[1], run.w[2], run.w[3]}, ob, (int)at, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b64(
                            u32x2{run.w[0], run.w[1]}, ob, (int)at, 0, 0);
                }
            }
        }

        // the state behind the chunk
        const float fade = ex2(a2 * (float)there);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int kt = 0; kt < 2 * KB; ++kt) S[ct][kt] *= fade;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            Parts<T, 3> vd[CT];
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = tok0[s] * tok[j];
            if (there < TT) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int left = there - late - (32 * s + 4 * h4 + slot_step(j));
                    f[j] = s_tok * ex2(a2 * (float)(left > 0 ? left : 0));
                }
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = fv[ct][s].get(j) * f[j];
                vd[ct].set(x);
            }
#pragma unroll
            for (int kt = 0; kt < 2 * KB; ++kt) {
                Frag<T> fk;
                if constexpr (sizeof(T) == 2)
                    fk.cols(ks + (32 * s + 4 * h4 + (m >> 2)) * QS + 16 * kt + 4 * (m & 3), QS);
                else
                    fk.cols(ks + (32 * s + 4 * h4) * QS + 16 * kt + m, QS);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[ct][kt] = mma(fk, vd[ct], S[ct][kt]);
            }
        }
    }

    if constexpr (OUT) {
        if (care) {
            if (first < stop) patch(first + (stop - 1 - first) / TT * TT);
        } else if (first < stop) {
            // (one row of the state says it for all: no key makes a bad value good)
            float sum = 0.f;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) sum = __builtin_fmaf(S[ct][0][0], 0.f, sum);
            const bool bad = __builtin_amdgcn_ballot_w64(sum != 0.f) != 0;
            if (lane == 0) from[w] = bad;
            __syncthreads();
            const int again = from[0] | from[1] | from[2] | from[3];
            if (__builtin_expect(__builtin_amdgcn_readfirstlane(again) != 0, 0)) return true;
        }
        // rows behind a sequence's last token
        const int64_t z0 = first > len ? first : len;
        if (z0 < end) {
            const int per = D2 / 8;
            for (int64_t i = tid; i < (end - z0) * per; i += kLinThreads) {
                const int64_t t = z0 + i / per;
                u32x4 *at = (u32x4 *)(out + t * out_row + i % per * (wide_out ? 32 : 16));
                const u32x4 zero = {0u, 0u, 0u, 0u};
                at[0] = zero;
                if (wide_out) at[1] = zero;
            }
        }
    }
    if (J.leave == nullptr || (OUT && seg != g.nseg - 1)) return false;
    const int ln = anew(lane);
    float *e = J.leave + (int64_t)(b * g.H + hd) * J.leave_bh + (int64_t)seg * J.leave_seg;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int kt = 0; kt < 2 * KB; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * kt + 4 * (ln >> 4) + r, col = column(ln & 15, ct);
                if (row < D1 && col < D2)
                    e[(int64_t)row * J.leave_r + (int64_t)(c0 + col) * J.leave_c] =
                        OUT && care && from[col] < TT ? NAN : S[ct][kt][r];
            }
    return false;
}

template <typename T, int KD, int CT, typename OT>
__global__ __launch_bounds__(kLinThreads, KD <= 128 ? 2 : 1) void linattn_kernel(const LinArgs g)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    bool care = false;
    while (linattn_walk<T, KD, CT, OT>(g, lds, care)) care = true;  // (twice at most)
}

// Segments' contributions -> the states that enter them, in place: [B H][nseg][D1 D2].
struct LinJoin {
    float *seg[2];
    const float *enter[2];   // the first state, or null
    int enter_r[2], enter_c[2];
    int cols[2];             // D2: elements of a row
};
__global__ __launch_bounds__(256) void linattn_join_kernel(const LinJoin j, const float *log_decay,
                                                           const int32_t *lengths, int H, int n,
                                                           int nseg, int seg, int64_t L)
{
    const int i = (blockIdx.x * 256 + threadIdx.x) * 4, bh = blockIdx.y, q = blockIdx.z;
    if (i >= n) return;
    const int b = bh / H;
    int64_t len = lengths != nullptr ? lengths[b] : L;
    len = len < 0 ? 0 : len < L ? len : L;
    float a2 = log_decay[bh % H];
    a2 = (a2 < -1e30f ? -1e30f : a2) * kLog2e;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (j.enter[q] != nullptr) {
        const float *e = j.enter[q] + (int64_t)bh * n + (int64_t)(i / j.cols[q]) * j.enter_r[q] +
                         (int64_t)(i % j.cols[q]) * j.enter_c[q];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = e[r * j.enter_c[q]];
    }
    float *p = j.seg[q] + (int64_t)bh * nseg * n + i;
    for (int s0 = 0; s0 < nseg; s0 += 8) {  // (eight at a time: loads ahead of the stores)
        f32x4 own[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            own[r] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (s0 + r < nseg - 1) own[r] = *(const f32x4 *)(p + (int64_t)(s0 + r) * n);
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int64_t left = len - (int64_t)(s0 + r) * seg;
            const int64_t there = left < 0 ? 0 : left < seg ? left : seg;
            if (s0 + r < nseg) *(f32x4 *)(p + (int64_t)(s0 + r) * n) = x;
            x = x * ex2(a2 * (float)there) + own[r];
        }
    }
}

// Sums over the heads that share a key or a value: [tokens][Hk][group][D] -> [tokens][Hk][D].
template <typename T>
__global__ __launch_bounds__(256) void linattn_group_kernel(const float *x, T *out, int64_t n,
                                                            int group, int D)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;  // of the output
    if (i >= n) return;
    const int64_t row = i / D;
    const float *p = x + row * group * D + i % D;
    f32x4 s = *(const f32x4 *)p;
    for (int g = 1; g < group; ++g) s += *(const f32x4 *)(p + (int64_t)g * D);
    const float f[4] = {s[0], s[1], s[2], s[3]};
    round_run<T, 4>(f).store(out + i);
}

// --------------------------------------------------------------------- one token
// A workgroup takes 32 columns of one head's state: 8 lanes of 4 columns, 32 rows at a time.
template <typename T>
__global__ __launch_bounds__(256) void linattn_step_kernel(int H, int group, int D1, int D2,
                                                           const T *q, const T *k, const T *v,
                                                           const float *log_decay, float scale,
                                                           const float *state, float *state_out,
                                                           T *o)
{
    __shared__ f32x4 part[4][8];
    const int tid = threadIdx.x, c4 = tid & 7, r0 = tid >> 3;
    const int hd = blockIdx.y % H, b = blockIdx.y / H, Hk = H / group;
    const int col = blockIdx.x * 32 + 4 * c4;
    const bool in = col < D2;
    const int64_t bh = (int64_t)b * H + hd, kv = (int64_t)b * Hk + hd / group;
    const float lam = ex2(log_decay[hd] * kLog2e);
    f32x4 x = {0.f, 0.f, 0.f, 0.f}, acc = x;
    const int64_t base = bh * D1 * D2 + col;
    if (in) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = to_f(v[kv * D2 + col + i]);
    }
    f32x4 s[kLinMost / 32];
    float kf[kLinMost / 32], qf[kLinMost / 32];
#pragma unroll
    for (int i = 0; i < kLinMost / 32; ++i) {
        const int row = r0 + 32 * i;
        if (in && row < D1) {
            s[i] = *(const f32x4 *)(state + base + (int64_t)row * D2);
            kf[i] = to_f(k[kv * D1 + row]);
            qf[i] = to_f(q[bh * D1 + row]);
        }
    }
#pragma unroll
    for (int i = 0; i < kLinMost / 32; ++i) {
        const int row = r0 + 32 * i;
        if (in && row < D1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[i][e] = __builtin_fmaf(s[i][e], lam, kf[i] * x[e]);
                acc[e] = __builtin_fmaf(qf[i], s[i][e], acc[e]);
            }
            *(f32x4 *)(state_out + base + (int64_t)row * D2) = s[i];
        }
    }
    // over the rows: lanes 8, 16 and 32 apart, then the waves
#pragma unroll
    for (int d = 8; d < 64; d <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], d);
    if ((tid & 63) < 8) part[tid >> 6][c4] = acc;
    __syncthreads();
    if (tid < 8 && in) {
        const f32x4 y = ((part[0][c4] + part[1][c4]) + (part[2][c4] + part[3][c4])) * scale;
        const float f[4] = {y[0], y[1], y[2], y[3]};
        round_run<T, 4>(f).store(o + bh * D2 + col);
    }
}

// ---------------------------------------------------------------------- host
template <typename T, int KD, int CT, typename OT>
static hipError_t launch_walk(LinArgs &g, hipStream_t st)
{
    g.items = g.B * g.H * g.slices * g.nseg;
    const int n = (g.items + 7) / 8 * 8 * g.jobs;
    constexpr size_t bytes = LinShape<T, KD, CT>::bytes(!__is_same(OT, void));
    if constexpr (bytes > 65536) {  // (more than a kernel may take unasked)
        const hipError_t e = hipFuncSetAttribute((const void *)linattn_kernel<T, KD, CT, OT>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((linattn_kernel<T, KD, CT, OT>), dim3(n), dim3(kLinThreads), bytes,
                       st, g);
    return hipGetLastError();
}

template <typename T, typename OT>
static hipError_t pick_walk(LinArgs &g, int rows, bool wide, hipStream_t st)
{
    if (rows <= 32 && !wide) return launch_walk<T, 32, 1, OT>(g, st);
    if (rows <= 64)
        return wide ? launch_walk<T, 64, 2, OT>(g, st) : launch_walk<T, 64, 1, OT>(g, st);
    if (rows <= 128)
        return wide ? launch_walk<T, 128, 2, OT>(g, st) : launch_walk<T, 128, 1, OT>(g, st);
    return wide ? launch_walk<T, 256, 2, OT>(g, st) : launch_walk<T, 256, 1, OT>(g, st);
}

struct LinPlan {
    int rows, slices, nseg, seg;
    bool wide;
    size_t off_seg[2], off_dk, off_dv, bytes;
};

// How wide a workgroup's part of the state is, 128 or 64 columns, and how the sequence is cut into
// segments: what costs least, in chunks of 64 tokens that a workgroup of 128 columns walks alone on
// its CU (4.9 us with heads of 128 in bf16).  With 64 columns a chunk takes 0.7; two workgroups on
// each CU 1.8 each, 1.05 with 64 columns (with keys beyond 128 a CU holds one).  1 more for the state
// that it starts and ends with, 2 with keys beyond 128; what a segment adds to the state costs 0.53
// of a walk, 0.45 with 64 columns; the launches and the joining 1, 1.5 with keys up to 64, whose
// chunks are shorter, and 0.1 a segment.  Measured against other choices, the rule's in brackets (us,
// columns x segments).  Forward, heads of 128: 8 rows x 2048 tokens x 12 heads 128x1: 150, [128x4:
// 112], 128x5: 102, 64x1: 111, 64x4: 115; 4 x 2048 x 64 [128x1: 165], 64x1: 179, 128x2: 195; 65536 x
// 16 128x16: 449, [128x32: 421], 64x32: 514; 2 x 4096 x 32 64x4: 133, [128x8: 121], 128x1: 286; 2048
// x 4 128x16: 37, 64x8: 35, [64x16: 29]; heads of 256, 4 x 1024 x 16 [64x1: 105], 128x1: 134; heads
// of 64, 2 x 4096 x 8 1: 138, 8: 39, [16: 30], 24: 32; fp32, 3 x 333 x 5 heads of 40 and 72 128x6: 22,
// [64x6: 17], 64x1: 29.  Gradient: 8 x 2048 x 12 [128x1: 214], 128x3: 208, 64x1: 251; 2 x 4096 x 32
// 128x1: 297, 128x4: 257, [64x1: 308]; 1000 x 12 128x6: 44, [64x6: 39], 64x1: 58; heads of 256, 4 x
// 1024 x 16 [128x1: 252], 64x1: 296, 128x2: 308.  So it misses by up to a fifth: it averages over the
// CUs where the fullest one ends the call, and takes a chunk of fp32 for one of bf16.
static double lin_rounds(int64_t groups, bool wide, int rows)
{
    const double lone = wide ? 1. : 0.7, two = rows > 128 ? 2. * lone : wide ? 1.8 : 1.05;
    const int64_t full = groups / 512, left = groups % 512;
    const double part = rows > 128 ? (left > 256 ? 1. : 0.) : (left - 256) / 256.;
    return two * (double)full +
           (left == 0 ? 0. : left <= 256 ? lone : lone + (two - lone) * part);
}
struct LinCut {
    int64_t n;
    double cost;
};
// heads: walks of the call, adds: those whose segments add to the state first
static LinCut lin_segments(int64_t heads, int64_t adds, int64_t L, bool wide, int rows)
{
    static const int kCounts[] = {2,  3,  4,  5,  6,  7,  8,  10, 12,  14,  16,  20, 24,
                                  28, 32, 40, 48, 64, 80, 96, 128, 192, 256, 384, 512};
    const int64_t chunks = (L + 63) / 64;
    const int64_t ends = rows > 128 ? 2 : 1;
    LinCut best{1, (double)(chunks + ends) * lin_rounds(heads, wide, rows)};
    for (int n : kCounts) {
        if (n > chunks || heads > ((int64_t)1 << 20)) break;
        const int64_t per = (chunks + n - 1) / n;
        const double t = (double)(per + ends) * (lin_rounds(heads * n, wide, rows) +
                                                 (wide ? 0.53 : 0.45) *
                                                     lin_rounds(adds * (n - 1), wide, rows)) +
                         (rows > 64 ? 1. : 1.5) + 0.1 * n;
        if (t < best.cost) best = {n, t};
    }
    return best;
}

static LinPlan lin_plan(int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv,
                        bool bwd)
{
    LinPlan p{};
    const int64_t most = dk > dv ? dk : dv, cols = bwd ? most : dv;
    p.rows = (int)(bwd ? most : dk);
    int64_t n = 0;
    double least = 0.;
    for (const bool wide : {false, true}) {
        if (wide && cols <= 64) break;
        const int64_t slices = wide ? (cols + 127) / 128 : (cols + 63) / 64, groups = B * H * slices;
        const LinCut cut = lin_segments(groups * (bwd ? 3 : 1), groups * (bwd ? 2 : 1), L, wide,
                                        p.rows);
        if (n > 0 && cut.cost > least) break;
        n = cut.n;
        least = cut.cost;
        p.wide = wide;
        p.slices = (int)slices;
    }
    int64_t seg = ((L + n - 1) / n + 63) / 64 * 64;
    if (seg < 64) seg = 64;
    p.seg = (int)(seg < ((int64_t)1 << 30) ? seg : (int64_t)1 << 30);
    p.nseg = (int)((L + p.seg - 1) / p.seg);
    if (p.nseg < 1) p.nseg = 1;
    size_t at = 0;
    if (p.nseg > 1)
        for (int i = 0; i < (bwd ? 2 : 1); ++i) {
            p.off_seg[i] = at;
            at = align256(at + (size_t)(B * H * p.nseg) * (size_t)(dk * dv) * 4);
        }
    if (bwd && H > Hk) {
        p.off_dk = at;
        at = align256(at + (size_t)(B * L * H) * (size_t)dk * 4);
        p.off_dv = at;
        at = align256(at + (size_t)(B * L * H) * (size_t)dv * 4);
    }
    p.bytes = at;
    return p;
}

static naju_status_t check_lin(int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv,
                               int32_t io, float scale)
{
    if (B < 0 || L < 0 || H < 0 || Hk < 0 || dk < 0 || dv < 0)
        return fail(NAJU_EINVAL, "negative size (batch=%lld seqlen=%lld heads=%lld kv_heads=%lld "
                                 "d_key=%lld d_value=%lld)",
                    (long long)B, (long long)L, (long long)H, (long long)Hk, (long long)dk,
                    (long long)dv);
    if (io != NAJU_F32 && io != NAJU_BF16)
        return fail(NAJU_EINVAL, "io dtype %d is neither NAJU_F32 nor NAJU_BF16", (int)io);
    if (H > 0 && (Hk == 0 || H % Hk != 0))
        return fail(NAJU_EINVAL, "heads %lld is no multiple of kv_heads %lld", (long long)H,
                    (long long)Hk);
    if (H > 0 && (dk < 8 || dv < 8 || dk % 8 || dv % 8 || dk > kLinMost || dv > kLinMost))
        return fail(NAJU_EUNSUPPORTED, "d_key %lld and d_value %lld must be multiples of 8 up to %d",
                    (long long)dk, (long long)dv, kLinMost);
    if (B > (1 << 20) || H > 65535 || B * H > (1 << 20) || L > ((int64_t)1 << 30))
        return fail(NAJU_EINVAL, "batch * heads (2^20 max), heads (65535 max) or seqlen (2^30 max) "
                                 "too large");
    if (H * dk > kLinStride || H * dv > kLinStride)
        return fail(NAJU_EINVAL, "heads * d_key or heads * d_value (2^20 max) too large");
    if (!(scale >= -1e30f && scale <= 1e30f)) return fail(NAJU_EINVAL, "scale must be finite");
    return NAJU_OK;
}

// (one token a row: the rows' distance, which no chunk spans)
static naju_status_t check_ld(int64_t ld, int64_t least, int64_t L, size_t e, const char *name)
{
    const int64_t most = L == 1 ? (int64_t)1 << 40 : kLinStride;
    if (ld < least || ld > most || ld * (int64_t)e % 16 != 0)
        return fail(NAJU_EINVAL, "token stride of %s (%lld) must be from %lld to %lld elements and a "
                                 "multiple of 16 bytes",
                    name, (long long)ld, (long long)least, (long long)most);
    return NAJU_OK;
}

// The kernel's tokens lie in chunks, and its rows where J.bq, .. say: with one token a row the
// distance from token to token is that of a contiguous one.
static int64_t token_ld(int64_t ld, int64_t least, int64_t L) { return L == 1 ? least : ld; }

// the walks g.job[from] .. g.job[to - 1]
static hipError_t walk(LinArgs g, int from, int to, const LinPlan &p, int32_t io, bool wide_out,
                       hipStream_t st)
{
    for (int i = from; i < to; ++i) g.job[i - from] = g.job[i];
    g.jobs = to - from;
    return io == NAJU_F32 ? pick_walk<float, float>(g, p.rows, p.wide, st)
           : wide_out     ? pick_walk<bf16, float>(g, p.rows, p.wide, st)
                          : pick_walk<bf16, bf16>(g, p.rows, p.wide, st);
}

// the entering states of all segments, for the first `jobs` of g's walks
static hipError_t enter_segments(LinArgs g, int jobs, const LinPlan &p, char *ws, int n, int32_t io,
                                 hipStream_t st)
{
    LinJoin j{};
    for (int i = 0; i < jobs; ++i) {
        LinJob &J = g.job[i];
        j.seg[i] = (float *)(ws + p.off_seg[i]);
        j.enter[i] = J.enter;
        j.enter_r[i] = J.enter_r;
        j.enter_c[i] = J.enter_c;
        j.cols[i] = J.D2;
        J.enter = nullptr;
        J.leave = j.seg[i];
        J.leave_bh = (int64_t)p.nseg * n;
        J.leave_seg = n;
        J.leave_r = J.D2;
        J.leave_c = 1;
    }
    LinArgs w = g;
    w.jobs = jobs;
    w.nseg -= 1;  // (what the last segment adds enters none)
    const hipError_t e = io == NAJU_F32 ? pick_walk<float, void>(w, p.rows, p.wide, st)
                                        : pick_walk<bf16, void>(w, p.rows, p.wide, st);
    if (e != hipSuccess) return e;
    // (a launch holds whole batch rows, so that heads and lengths keep their places)
    const int rows = 65535 / g.H * g.H;
    for (int at = 0; at < g.B * g.H; at += rows) {
        const int now = g.B * g.H - at < rows ? g.B * g.H - at : rows;
        LinJoin part = j;
        for (int i = 0; i < jobs; ++i) {
            part.seg[i] += (int64_t)at * p.nseg * n;
            if (part.enter[i] != nullptr) part.enter[i] += (int64_t)at * n;
        }
        hipLaunchKernelGGL(linattn_join_kernel, dim3((n + 1023) / 1024, now, jobs), dim3(256), 0, st,
                           part, g.log_decay, g.lengths != nullptr ? g.lengths + at / g.H : nullptr,
                           g.H, n, p.nseg, p.seg, g.L);
        const hipError_t f = hipGetLastError();
        if (f != hipSuccess) return f;
    }
    return hipSuccess;
}

}  // namespace naju

using namespace naju;

extern "C" {

size_t naju_linattn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                        int64_t kv_heads, int64_t d_key, int64_t d_value)
{
    if (check_lin(batch, seqlen, heads, kv_heads, d_key, d_value, NAJU_F32, 1.f) != NAJU_OK ||
        batch == 0 || heads == 0)  // (without heads the other sizes are not looked at)
        return 0;
    return lin_plan(batch, seqlen, heads, kv_heads, d_key, d_value, false).bytes;
}

naju_status_t naju_linattn_fwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads,
                               int64_t d_key, int64_t d_value, int32_t io, const void *q,
                               int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                               const float *log_decay, const float *state, const int32_t *lengths,
                               float scale, void *o, float *state_out, void *ws, size_t ws_bytes,
                               void *stream)
{
    NAJU_TRY(check_lin(batch, seqlen, heads, kv_heads, d_key, d_value, io, scale));
    if (batch == 0 || heads == 0) return NAJU_OK;
    const size_t e = io == NAJU_F32 ? 4 : 2;
    if (seqlen > 0) {
        NAJU_TRY(check_ld(ldq, heads * d_key, seqlen, e, "q"));
        NAJU_TRY(check_ld(ldk, kv_heads * d_key, seqlen, e, "k"));
        NAJU_TRY(check_ld(ldv, kv_heads * d_value, seqlen, e, "v"));
        NAJU_TRY(need(q, "q", 16));
        NAJU_TRY(need(k, "k", 16));
        NAJU_TRY(need(v, "v", 16));
        NAJU_TRY(need(o, "o", 16));
    }
    NAJU_TRY(need(log_decay, "log_decay", 4));
    NAJU_TRY(opt(state, "state", 4));
    NAJU_TRY(opt(state_out, "state_out", 4));
    NAJU_TRY(opt(lengths, "lengths", 4));
    const LinPlan p = lin_plan(batch, seqlen, heads, kv_heads, d_key, d_value, false);
    if (p.bytes > 0) NAJU_TRY(need_ws(ws, ws_bytes, p.bytes));
    if (batch * heads * p.slices * p.nseg > ((int64_t)1 << 22))
        return fail(NAJU_EINVAL, "batch * heads too large for this sequence length");
    const int n = (int)(d_key * d_value);
    LinArgs g{};
    g.log_decay = log_decay;
    g.lengths = lengths;
    g.B = (int)batch;
    g.H = (int)heads;
    g.L = seqlen;
    g.slices = p.slices;
    g.nseg = p.nseg;
    g.seg = p.seg;
    LinJob &J = g.job[0];
    J.q = q;
    J.k = k;
    J.v = v;
    J.o = o;
    J.ldq = token_ld(ldq, heads * d_key, seqlen);
    J.ldk = token_ld(ldk, kv_heads * d_key, seqlen);
    J.ldv = token_ld(ldv, kv_heads * d_value, seqlen);
    J.ldo = heads * d_value;
    J.bq = seqlen * ldq;
    J.bk = seqlen * ldk;
    J.bv = seqlen * ldv;
    J.enter = state;
    J.enter_bh = n;
    J.enter_r = (int)d_value;
    J.enter_c = 1;
    J.leave = state_out;
    J.leave_bh = n;
    J.leave_r = (int)d_value;
    J.leave_c = 1;
    J.D1 = (int)d_key;
    J.D2 = (int)d_value;
    J.gq = 1;
    J.gk = J.gv = (int)(heads / kv_heads);
    J.s_row = J.s_pair = scale;
    J.s_tok = 1.f;
    J.late = 1;
    hipStream_t st = (hipStream_t)stream;
    if (p.nseg > 1) {
        NAJU_TRY(hip_status(enter_segments(g, 1, p, (char *)ws, n, io, st),
                            "linear attention segments launch"));
        J.enter = (const float *)((char *)ws + p.off_seg[0]);
        J.enter_bh = (int64_t)p.nseg * n;
        J.enter_seg = n;
    }
    return hip_status(walk(g, 0, 1, p, io, false, st), "linear attention launch");
}

size_t naju_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                        int64_t kv_heads, int64_t d_key, int64_t d_value)
{
    if (check_lin(batch, seqlen, heads, kv_heads, d_key, d_value, NAJU_F32, 1.f) != NAJU_OK ||
        batch == 0 || heads == 0)  // (without heads the other sizes are not looked at)
        return 0;
    return lin_plan(batch, seqlen, heads, kv_heads, d_key, d_value, true).bytes;
}

naju_status_t naju_linattn_bwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t kv_heads,
                               int64_t d_key, int64_t d_value, int32_t io, const void *q,
                               int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                               const float *log_decay, const float *state, const int32_t *lengths,
                               float scale, const void *dout, const float *dstate_out, void *dq,
                               void *dk, void *dv, float *dstate, void *ws, size_t ws_bytes,
                               void *stream)
{
    NAJU_TRY(check_lin(batch, seqlen, heads, kv_heads, d_key, d_value, io, scale));
    if (batch == 0 || heads == 0) return NAJU_OK;
    const size_t e = io == NAJU_F32 ? 4 : 2;
    if (seqlen > 0) {
        NAJU_TRY(check_ld(ldq, heads * d_key, seqlen, e, "q"));
        NAJU_TRY(check_ld(ldk, kv_heads * d_key, seqlen, e, "k"));
        NAJU_TRY(check_ld(ldv, kv_heads * d_value, seqlen, e, "v"));
        NAJU_TRY(need(q, "q", 16));
        NAJU_TRY(need(k, "k", 16));
        NAJU_TRY(need(v, "v", 16));
        NAJU_TRY(need(dout, "dout", 16));
        NAJU_TRY(need(dq, "dq", 16));
        NAJU_TRY(need(dk, "dk", 16));
        NAJU_TRY(need(dv, "dv", 16));
    }
    NAJU_TRY(need(log_decay, "log_decay", 4));
    NAJU_TRY(opt(state, "state", 4));
    NAJU_TRY(opt(dstate_out, "dstate_out", 4));
    NAJU_TRY(opt(dstate, "dstate", 4));
    NAJU_TRY(opt(lengths, "lengths", 4));
    const LinPlan p = lin_plan(batch, seqlen, heads, kv_heads, d_key, d_value, true);
    if (p.bytes > 0) NAJU_TRY(need_ws(ws, ws_bytes, p.bytes));
    if (batch * heads * p.slices * p.nseg > ((int64_t)1 << 22))
        return fail(NAJU_EINVAL, "batch * heads too large for this sequence length");
    const int n = (int)(d_key * d_value), group = (int)(heads / kv_heads);
    char *base = (char *)ws;
    LinArgs g{};
    g.log_decay = log_decay;
    g.lengths = lengths;
    g.B = (int)batch;
    g.H = (int)heads;
    g.L = seqlen;
    g.slices = p.slices;
    g.nseg = p.nseg;
    g.seg = p.seg;
    const int64_t ldg = heads * d_value, bg = seqlen * ldg;
    const int64_t bq = seqlen * ldq, bk = seqlen * ldk, bv = seqlen * ldv;
    ldq = token_ld(ldq, heads * d_key, seqlen);
    ldk = token_ld(ldk, kv_heads * d_key, seqlen);
    ldv = token_ld(ldv, kv_heads * d_value, seqlen);
    // dq: the forward's state transposed, from dout, v and k
    LinJob &A = g.job[0];
    A.q = dout;
    A.ldq = ldg;
    A.bq = bg;
    A.gq = 1;
    A.k = v;
    A.ldk = ldv;
    A.bk = bv;
    A.v = k;
    A.ldv = ldk;
    A.bv = bk;
    A.gk = A.gv = group;
    A.o = dq;
    A.ldo = heads * d_key;
    A.D1 = (int)d_value;
    A.D2 = (int)d_key;
    A.enter = state;
    A.enter_bh = n;
    A.enter_r = 1;
    A.enter_c = (int)d_value;
    A.s_row = A.s_pair = scale;
    A.s_tok = 1.f;
    A.late = 1;
    // dv, and the state's gradient: back in time from k, q and dout
    LinJob &V = g.job[1];
    V.q = k;
    V.ldq = ldk;
    V.bq = bk;
    V.gq = group;
    V.k = q;
    V.ldk = ldq;
    V.bk = bq;
    V.v = dout;
    V.ldv = ldg;
    V.bv = bg;
    V.gk = V.gv = 1;
    V.o = group > 1 ? (void *)(base + p.off_dv) : dv;
    V.ldo = heads * d_value;
    V.D1 = (int)d_key;
    V.D2 = (int)d_value;
    V.enter = dstate_out;
    V.enter_bh = n;
    V.enter_r = (int)d_value;
    V.enter_c = 1;
    V.leave = dstate;
    V.leave_bh = n;
    V.leave_r = (int)d_value;
    V.leave_c = 1;
    V.s_row = 1.f;
    V.s_pair = V.s_tok = scale;
    V.late = 0;
    V.back = 1;
    hipStream_t st = (hipStream_t)stream;
    if (p.nseg > 1) {
        NAJU_TRY(hip_status(enter_segments(g, 2, p, base, n, io, st),
                            "linear attention segments launch"));
        A.enter = (const float *)(base + p.off_seg[0]);
        A.enter_r = (int)d_key;
        A.enter_c = 1;
        V.enter = (const float *)(base + p.off_seg[1]);
        A.enter_bh = V.enter_bh = (int64_t)p.nseg * n;
        A.enter_seg = V.enter_seg = n;
    }
    // dk: the same state as dv's, transposed, from v, dout and q
    LinJob &K = g.job[2];
    K = V;
    K.q = v;
    K.ldq = ldv;
    K.bq = bv;
    K.k = dout;
    K.ldk = ldg;
    K.bk = bg;
    K.v = q;
    K.ldv = ldq;
    K.bv = bq;
    K.o = group > 1 ? (void *)(base + p.off_dk) : dk;
    K.ldo = heads * d_key;
    K.D1 = (int)d_value;
    K.D2 = (int)d_key;
    K.enter_r = 1;
    K.enter_c = (int)d_value;
    K.leave = nullptr;
    if (group == 1 || io == NAJU_F32) {
        NAJU_TRY(hip_status(walk(g, 0, 3, p, io, false, st), "linear attention gradient launch"));
    } else {  // (those of shared heads are summed before they are rounded)
        NAJU_TRY(hip_status(walk(g, 0, 1, p, io, false, st), "linear attention gradient launch"));
        NAJU_TRY(hip_status(walk(g, 1, 3, p, io, true, st), "linear attention gradient launch"));
    }
    if (group == 1 || seqlen == 0) return NAJU_OK;
    for (int i = 0; i < 2; ++i) {
        const int64_t D = i ? d_value : d_key, total = batch * seqlen * kv_heads * D;
        const float *x = (const float *)(base + (i ? p.off_dv : p.off_dk));
        void *out = i ? dv : dk;
        const int64_t most = (int64_t)1 << 32;  // elements of a launch, a multiple of every D's row
        for (int64_t at = 0; at < total;) {
            const int64_t step = most / D * D, now = total - at < step ? total - at : step;
            const dim3 grid((unsigned)((now + 1023) / 1024));
            if (io == NAJU_F32)
                hipLaunchKernelGGL(linattn_group_kernel<float>, grid, dim3(256), 0, st,
                                   x + at * group, (float *)out + at, now, group, (int)D);
            else
                hipLaunchKernelGGL(linattn_group_kernel<bf16>, grid, dim3(256), 0, st,
                                   x + at * group, (bf16 *)out + at, now, group, (int)D);
            NAJU_TRY(hip_status(hipGetLastError(), "linear attention head sums launch"));
            at += now;
        }
    }
    return NAJU_OK;
}

naju_status_t naju_linattn_step(int64_t batch, int64_t heads, int64_t kv_heads, int64_t d_key,
                                int64_t d_value, int32_t io, const void *q, const void *k,
                                const void *v, const float *log_decay, const float *state,
                                float scale, void *o, float *state_out, void *stream)
{
    NAJU_TRY(check_lin(batch, 1, heads, kv_heads, d_key, d_value, io, scale));
    if (batch == 0 || heads == 0) return NAJU_OK;
    const size_t e = io == NAJU_F32 ? 4 : 2;
    NAJU_TRY(need(q, "q", e));
    NAJU_TRY(need(k, "k", e));
    NAJU_TRY(need(v, "v", e));
    NAJU_TRY(need(o, "o", e));
    NAJU_TRY(need(log_decay, "log_decay", 4));
    NAJU_TRY(need(state, "state", 16));
    NAJU_TRY(need(state_out, "state_out", 16));
    const int64_t per = 65535 / heads;  // batch rows of a launch
    const int group = (int)(heads / kv_heads);
    for (int64_t b = 0; b < batch; b += per) {
        const int64_t now = batch - b < per ? batch - b : per;
        const dim3 grid((unsigned)((d_value + 31) / 32), (unsigned)(now * heads));
        const int64_t s = b * heads * d_key * d_value;
        const int64_t bq = b * heads * d_key, bo = b * heads * d_value;
        const int64_t bk = b * kv_heads * d_key, bv = b * kv_heads * d_value;
        if (io == NAJU_F32)
            hipLaunchKernelGGL(linattn_step_kernel<float>, grid, dim3(256), 0, (hipStream_t)stream,
                               (int)heads, group, (int)d_key, (int)d_value, (const float *)q + bq,
                               (const float *)k + bk, (const float *)v + bv, log_decay, scale,
                               state + s, state_out + s, (float *)o + bo);
        else
            hipLaunchKernelGGL(linattn_step_kernel<bf16>, grid, dim3(256), 0, (hipStream_t)stream,
                               (int)heads, group, (int)d_key, (int)d_value, (const bf16 *)q + bq,
                               (const bf16 *)k + bk, (const bf16 *)v + bv, log_decay, scale,
                               state + s, state_out + s, (bf16 *)o + bo);
        NAJU_TRY(hip_status(hipGetLastError(), "linear attention step launch"));
    }
    return NAJU_OK;
}

}  // extern "C"
