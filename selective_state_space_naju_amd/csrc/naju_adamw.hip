// naju_adamw.hip -- one AdamW step over many tensors, optimizer states in 32 or 8
// bits.
//
// Per element, with gradient g, coefficient c, step t:
//     g = c g,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//     p = p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
// 8-bit states hold m and sqrt(v) as e4m3 numbers (3 mantissa bits, 2^-9 to 448)
// times one fp32 scale for every 256 elements, the block's largest magnitude over
// 448: the root's range is half as many powers of two as v's, which that type
// holds.  Rounding moves a value by at most 2^-4 of itself down to 2^-6 of the scale
// (1 / 28672 of the block's largest), and by 2^-10 of the scale below that.  The step
// itself uses the unrounded m and v.  m may be small against its block where the root
// is smaller still: a root lost beside a first moment that is kept would leave the next
// step eps alone to divide by, so there it is stored as the smallest code, 2^-9 of its
// scale (gradients of 1 beside sparse ones of 1e-5 move the latter by 3 lr at most, in
// place of 900).
//
// Rounded to nearest, a state that a step changes by less than half a code stays where it
// was, however many steps: a root at b2 = 0.999 cannot fall (gradients that fall to a tenth
// beside others that do not: 5.4 times its value 4000 steps later, in the median).  The
// stochastic form rounds up with the probability of the value's distance from the code
// below, so the mean of what is stored is the value: 1.00 times, eight of ten roots within
// 25 %.  Its random number is the step's, mixed, plus the element's place in the sequence
// of the golden ratio's multiples: independent from step to step for each element, and
// spread evenly over a step's elements, for one addition an element.
//
// Bound by bytes: 28 an element with fp32 gradients and 32-bit states, 16 with
// 8-bit ones.  A wave takes 256 consecutive elements at a time, 4 a lane, so a
// block of the 8-bit states is one wave's and its maximum a reduction inside the
// wave.  The tensors' addresses travel in the kernel's arguments, as many as fit: no
// table in device memory, which would have to be kept in step with gradients that
// move, and nothing to copy before the launch.  A workgroup finds its tensor by
// bisection over the first units of each.
//
// 138 M parameters with bf16 gradients and copies 738 us (28 bytes each, 5.2 TB/s, a large
// copy's rate); 200 M with 8-bit states and fp32 gradients 642 us (16 bytes, 5.0 TB/s), with
// stochastic rounding 734 us (4.4 TB/s: 23 vector instructions an element on top of 118, four cycles
// of a SIMD each, which then take longer than the loads).
#include <math.h>
#include <stdlib.h>

#include "naju_device.h"
#include "naju_host.h"
#include "naju_launch.h"
#include "naju_vec.h"

namespace naju {

constexpr int kBlock8 = 256;              // elements that share a scale
constexpr int kUnit = 4096;               // elements of a workgroup: 4 waves x 4 x 256
constexpr float kE4m3Most = 448.f;
constexpr float kE4m3Tiny = 0x1p-120f;    // scales below this are taken as 0

struct AdamTensor {
    const float *p;
    const void *g, *m, *v;
    const float *ms, *vs;
    float *p_out;
    void *m_out, *v_out;
    float *ms_out, *vs_out;
    bf16 *copy;
    int64_t n;
    uint32_t at;                          // first element's index in its tensor, low bits
};
constexpr int kTensors = 32;              // of a launch: 3.5 KB of the 4 KB of arguments

enum Store { kF32, kNearest, kStochastic };  // the states' type, and how they are rounded

struct AdamArgs {
    AdamTensor t[kTensors];
    uint32_t first[kTensors + 1];         // first unit of each tensor, and their number
    int count;
    float b1, c1, b2, c2;                 // betas and 1 - betas
    float lr, wd, eps;
    float bc1, bc2;                       // 1 - b^t, where the step is the host's
    float ln1, ln2;                       // log of the betas
    const int32_t *step;                  // or null
    uint32_t step_host;
    const float *lr_dev, *grad_scale;     // or null
};

// Multiples of the golden ratio's fraction lie evenly in [0, 1), the first n for every n.
constexpr uint32_t kGolden = 0x9E3779B9u;

// A step's random number, one for each of its two states.  (Products with the fractions of
// the golden ratio, of sqrt 2 and of sqrt 3; their upper halves folded down in between.)
__device__ __forceinline__ uint32_t step_noise(uint32_t step, uint32_t which)
{
    uint32_t x = (2u * step + which + 1u) * kGolden;
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ x >> 16;
}

// v_cvt_*_fp8 converts e4m3 on gfx950, to nearest even
__device__ __forceinline__ uint32_t to_e4m3x4(const float (&f)[4])
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], r, true);
}
__device__ __forceinline__ void from_e4m3x4(uint32_t w, float (&f)[4])
{
    f[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
    f[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
    f[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
    f[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
}

// the largest of the wave's values, in every lane (NaN is passed over)
__device__ __forceinline__ float wave_most(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

// f, at most kE4m3Most, as one of the two codes' values around it: 20 bits of noise are added to
// the bits that a code does not hold, which are then cut off.  Below 2^-6 codes lie 2^-9 apart, as
// they do from 2^-6 on: values are moved up there and back.
__device__ __forceinline__ float spread(float f, uint32_t noise)
{
    const float a = fabsf(f), up = a < 0x1p-6f ? 0x1p-6f : 0.f;
    const float r = __uint_as_float((__float_as_uint(a + up) + (noise >> 12)) & 0xfff00000u) - up;
    return f == f ? copysignf(r, f) : f;
}

// 4 of a block's values as codes of 8 bits; the scale is the block's.  noise: the first one's
template <bool STOCHASTIC>
__device__ __forceinline__ uint32_t encode(const float (&x)[4], float &scale, uint32_t noise)
{
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(x[i]));
    scale = wave_most(most) / kE4m3Most;
    if (scale < kE4m3Tiny) scale = 0.f;
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = x[i] * inv;  // (selects, so that NaN stays)
        f[i] = f[i] > kE4m3Most ? kE4m3Most : f[i] < -kE4m3Most ? -kE4m3Most : f[i];
        if constexpr (STOCHASTIC) f[i] = spread(f[i], noise + (uint32_t)i * kGolden);
    }
    return to_e4m3x4(f);
}

// the codes of roots with the smallest one in place of each 0 beside a first moment that is not 0
__device__ __forceinline__ uint32_t keep_roots(uint32_t v, uint32_t m)
{
    const uint32_t low = 0x7f7f7f7fu;  // (bits below the sign: a sum past them says not 0)
    const uint32_t has_m = (m & low) + low, has_v = (v & low) + low;
    return v | (has_m & ~has_v & ~low) >> 7;
}

struct AdamCoef {
    float b1, c1, b2, c2, lr, shrink, eps, inv1, bc2, gs;
    uint32_t noise_m, noise_v;
};

__device__ __forceinline__ void adam_element(const AdamCoef &c, float g, float &p, float &m,
                                             float &v)
{
    g *= c.gs;
    m = c.b1 * m + c.c1 * g;
    v = c.b2 * v + c.c2 * g * g;
    p = p * c.shrink - c.lr * (m * c.inv1) / (sqrtf(v / c.bc2) + c.eps);
}

// a lane's 4 elements of a wave's block of 256 from b on; FULL: the tensor has them all
template <typename GIO, Store ST> struct Elements {
    static constexpr bool S8 = ST != kF32;
    Run<float, 4> p, m, v;
    Run<GIO, 4> g;
    uint32_t m8, v8;
    float ms, vs;

    template <bool FULL>
    __device__ __forceinline__ void load(const AdamTensor &t, int64_t b, int lane)
    {
        const int64_t e = b + lane * 4;
        const int left = FULL ? 4 : t.n - e < 4 ? (int)(t.n - e) : 4;  // (none: 0 or less)
        if constexpr (S8) {
            ms = t.ms[b / kBlock8];
            vs = t.vs[b / kBlock8];
        }
        if (FULL || left == 4) {
            p.load(t.p + e);
            g.load((const GIO *)t.g + e);
            if constexpr (S8) {
                __builtin_memcpy(&m8, (const uint8_t *)t.m + e, 4);
                __builtin_memcpy(&v8, (const uint8_t *)t.v + e, 4);
            } else {
                m.load((const float *)t.m + e);
                v.load((const float *)t.v + e);
            }
        } else {
            p.load_part(t.p + e, left);
            g.load_part((const GIO *)t.g + e, left);
            if constexpr (S8) {
                m8 = v8 = 0u;
                for (int i = 0; i < left; ++i) {
                    m8 |= (uint32_t)((const uint8_t *)t.m)[e + i] << (8 * i);
                    v8 |= (uint32_t)((const uint8_t *)t.v)[e + i] << (8 * i);
                }
            } else {
                m.load_part((const float *)t.m + e, left);
                v.load_part((const float *)t.v + e, left);
            }
        }
    }

    template <bool FULL>
    __device__ __forceinline__ void step(const AdamTensor &t, int64_t b, int lane,
                                         const AdamCoef &c) const
    {
        const int64_t e = b + lane * 4;
        const int left = FULL ? 4 : t.n - e < 4 ? (int)(t.n - e) : 4;
        float pf[4], mf[4], vf[4];
        if constexpr (S8) {
            from_e4m3x4(m8, mf);
            from_e4m3x4(v8, vf);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pf[i] = p.get(i);
            if constexpr (S8) {
                mf[i] *= ms;
                vf[i] *= vs;
                vf[i] *= vf[i];
            } else {
                mf[i] = m.get(i);
                vf[i] = v.get(i);
            }
            adam_element(c, g.get(i), pf[i], mf[i], vf[i]);
            if constexpr (S8) {  // (elements that there are none of count nothing)
                mf[i] = i < left ? mf[i] : 0.f;
                vf[i] = i < left ? sqrtf(vf[i]) : 0.f;
            }
        }
        uint32_t cm = 0, cv = 0;
        if constexpr (S8) {
            float sm, sv;
            const uint32_t place = (t.at + (uint32_t)e) * kGolden;
            cm = encode<ST == kStochastic>(mf, sm, c.noise_m + place);
            cv = encode<ST == kStochastic>(vf, sv, c.noise_v + place);
            if (sv > 0.f && sv < INFINITY) cv = keep_roots(cv, cm);
            if (lane == 0) {
                t.ms_out[b / kBlock8] = sm;
                t.vs_out[b / kBlock8] = sv;
            }
        }
        const Run<float, 4> po = round_run<float, 4>(pf);
        const Run<bf16, 4> co = round_run<bf16, 4>(pf);
        if (FULL || left == 4) {
            po.store(t.p_out + e);
            if (t.copy != nullptr) co.store(t.copy + e);
            if constexpr (S8) {
                __builtin_memcpy((uint8_t *)t.m_out + e, &cm, 4);
                __builtin_memcpy((uint8_t *)t.v_out + e, &cv, 4);
            } else {
                round_run<float, 4>(mf).store((float *)t.m_out + e);
                round_run<float, 4>(vf).store((float *)t.v_out + e);
            }
        } else if (left > 0) {
            po.store_part(t.p_out + e, left);
            if (t.copy != nullptr) co.store_part(t.copy + e, left);
            if constexpr (S8) {
                for (int i = 0; i < left; ++i) {
                    ((uint8_t *)t.m_out)[e + i] = (uint8_t)(cm >> (8 * i));
                    ((uint8_t *)t.v_out)[e + i] = (uint8_t)(cv >> (8 * i));
                }
            } else {
                round_run<float, 4>(mf).store_part((float *)t.m_out + e, left);
                round_run<float, 4>(vf).store_part((float *)t.v_out + e, left);
            }
        }
    }
};

template <typename GIO, Store ST>
__global__ __launch_bounds__(256) void adamw_kernel(const AdamArgs a)
{
    // the tensor that holds this workgroup's unit
    int lo = 0, hi = a.count;  // first[lo] <= unit < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.first[mid] <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const AdamTensor &t = a.t[lo];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t e0 = (int64_t)(blockIdx.x - a.first[lo]) * kUnit + wave * 256;

    AdamCoef c{a.b1, a.c1, a.b2, a.c2, a.lr, 0.f, a.eps, 0.f, a.bc2, 1.f, 0u, 0u};
    float bc1 = a.bc1;
    if (a.lr_dev != nullptr) c.lr = *a.lr_dev;
    if (a.grad_scale != nullptr) c.gs = *a.grad_scale;
    if (a.step != nullptr) {
        const float s = (float)*a.step;
        bc1 = -expm1f(s * a.ln1);
        c.bc2 = -expm1f(s * a.ln2);
    }
    if constexpr (ST == kStochastic) {
        const uint32_t n = a.step != nullptr ? (uint32_t)*a.step : a.step_host;
        c.noise_m = step_noise(n, 0);
        c.noise_v = step_noise(n, 1);
    }
    c.inv1 = 1.f / bc1;
    c.shrink = 1.f - c.lr * a.wd;

    constexpr int J = kUnit / 1024;  // blocks of 256 elements of a wave
    if (e0 - wave * 256 + kUnit <= t.n) {
        Elements<GIO, ST> x[J];
#pragma unroll
        for (int j = 0; j < J; ++j) x[j].template load<true>(t, e0 + j * 1024, lane);
#pragma unroll
        for (int j = 0; j < J; ++j) x[j].template step<true>(t, e0 + j * 1024, lane, c);
        return;
    }
    // the tensor's last unit: whole blocks, then what is left
    for (int j = 0; j < J; ++j) {
        const int64_t b = e0 + j * 1024;
        if (b >= t.n) break;
        Elements<GIO, ST> x;
        if (b + 256 <= t.n) {
            x.template load<true>(t, b, lane);
            x.template step<true>(t, b, lane, c);
        } else {
            x.template load<false>(t, b, lane);
            x.template step<false>(t, b, lane, c);
        }
    }
}

// ---------------------------------------------------------------------- host
template <typename GIO> static void launch(const AdamArgs &a, unsigned units, Store st, hipStream_t s)
{
    if (st == kF32) hipLaunchKernelGGL((adamw_kernel<GIO, kF32>), dim3(units), dim3(256), 0, s, a);
    else if (st == kNearest)
        hipLaunchKernelGGL((adamw_kernel<GIO, kNearest>), dim3(units), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((adamw_kernel<GIO, kStochastic>), dim3(units), dim3(256), 0, s, a);
}

static int by_address(const void *a, const void *b)
{
    const naju_adamw_tensor_t *x = *(naju_adamw_tensor_t *const *)a;
    const naju_adamw_tensor_t *y = *(naju_adamw_tensor_t *const *)b;
    return x->p < y->p ? -1 : x->p > y->p;
}

}  // namespace naju

using namespace naju;

extern "C" naju_status_t naju_adamw_step(int64_t n_tensors, const naju_adamw_tensor_t *tensors,
                                         int32_t g_io, int32_t state_bits, double lr,
                                         double beta1, double beta2, double eps,
                                         double weight_decay, int64_t step,
                                         const int32_t *step_dev, const float *lr_dev,
                                         const float *grad_scale, void *stream)
{
    if (n_tensors < 0) return fail(NAJU_EINVAL, "negative size (n_tensors=%lld)",
                                   (long long)n_tensors);
    if (n_tensors > (1 << 24)) return fail(NAJU_EINVAL, "n_tensors (2^24 max) too large");
    if (g_io != NAJU_F32 && g_io != NAJU_BF16)
        return fail(NAJU_EINVAL, "io dtype %d is neither NAJU_F32 nor NAJU_BF16", (int)g_io);
    if (state_bits != 32 && state_bits != 8 && state_bits != 8 + NAJU_STOCHASTIC)
        return fail(NAJU_EUNSUPPORTED, "state_bits %d is neither 32 nor 8 nor 8 + NAJU_STOCHASTIC",
                    (int)state_bits);
    if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1))
        return fail(NAJU_EINVAL, "beta1 and beta2 must lie in [0, 1)");
    if (!(eps >= 0) || eps > 1e30) return fail(NAJU_EINVAL, "eps must be finite and not negative");
    if (!(lr >= -1e30 && lr <= 1e30) || !(weight_decay >= -1e30 && weight_decay <= 1e30))
        return fail(NAJU_EINVAL, "lr and weight_decay must be finite");
    if (step_dev == nullptr && step < 1)
        return fail(NAJU_EINVAL, "step %lld: steps count from 1", (long long)step);
    NAJU_TRY(opt(step_dev, "step_dev", 4));
    NAJU_TRY(opt(lr_dev, "lr_dev", 4));
    NAJU_TRY(opt(grad_scale, "grad_scale", 4));
    if (n_tensors == 0) return NAJU_OK;
    NAJU_TRY(need(tensors, "tensors", 8));
    const Store store = state_bits == 32 ? kF32 : state_bits == 8 ? kNearest : kStochastic;
    const bool s8 = store != kF32;
    const size_t eg = g_io == NAJU_F32 ? 4 : 2, es = s8 ? 1 : 4;
    for (int64_t i = 0; i < n_tensors; ++i) {
        const naju_adamw_tensor_t &t = tensors[i];
        if (t.n < 0 || t.n > ((int64_t)1 << 42))
            return fail(NAJU_EINVAL, "tensor %lld: %lld elements (0 to 2^42)", (long long)i,
                        (long long)t.n);
        if (t.n == 0) continue;
        NAJU_TRY(need(t.p, "p", 4));
        NAJU_TRY(need(t.g, "g", eg));
        NAJU_TRY(need(t.m, "m", es));
        NAJU_TRY(need(t.v, "v", es));
        NAJU_TRY(opt(t.p_out, "p_out", 4));
        NAJU_TRY(opt(t.m_out, "m_out", es));
        NAJU_TRY(opt(t.v_out, "v_out", es));
        NAJU_TRY(opt(t.copy, "copy", 2));
        if (s8) {
            NAJU_TRY(need(t.m_scale, "m_scale", 4));
            NAJU_TRY(need(t.v_scale, "v_scale", 4));
            NAJU_TRY(opt(t.m_scale_out, "m_scale_out", 4));
            NAJU_TRY(opt(t.v_scale_out, "v_scale_out", 4));
        }
    }
    // a parameter listed twice would be updated by two workgroups at once
    if (n_tensors > 1) {
        const naju_adamw_tensor_t **order =
            (const naju_adamw_tensor_t **)malloc(sizeof(*order) * (size_t)n_tensors);
        if (order == nullptr) return fail(NAJU_EINVAL, "out of host memory");
        int64_t used = 0;
        for (int64_t i = 0; i < n_tensors; ++i)
            if (tensors[i].n > 0) order[used++] = &tensors[i];
        qsort(order, (size_t)used, sizeof(*order), by_address);
        int64_t bad = -1;
        for (int64_t i = 1; i < used && bad < 0; ++i)
            if ((uintptr_t)order[i - 1]->p + 4 * (uintptr_t)order[i - 1]->n >
                (uintptr_t)order[i]->p)
                bad = order[i] - tensors;
        free(order);
        if (bad >= 0)
            return fail(NAJU_EINVAL, "tensor %lld: its parameters overlap another's",
                        (long long)bad);
    }

    AdamArgs a{};
    a.b1 = (float)beta1;
    a.c1 = (float)(1.0 - beta1);
    a.b2 = (float)beta2;
    a.c2 = (float)(1.0 - beta2);
    a.lr = (float)lr;
    a.wd = (float)weight_decay;
    a.eps = (float)eps;
    a.ln1 = (float)log(beta1);
    a.ln2 = (float)log(beta2);
    if (step_dev == nullptr) {
        a.bc1 = (float)-expm1((double)step * log(beta1));
        a.bc2 = (float)-expm1((double)step * log(beta2));
    }
    a.step = step_dev;
    a.step_host = (uint32_t)step;
    a.lr_dev = lr_dev;
    a.grad_scale = grad_scale;
    hipStream_t st = (hipStream_t)stream;
    const int64_t most = (int64_t)1 << 23;  // units of a launch (a grid stays below 2^32 threads)
    int64_t i = 0, done = 0;                // next tensor, and units of it already launched
    while (i < n_tensors) {
        a.count = 0;
        int64_t units = 0;
        while (i < n_tensors && a.count < kTensors && units < most) {
            const naju_adamw_tensor_t &t = tensors[i];
            const int64_t all = (t.n + kUnit - 1) / kUnit, left = all - done;
            const int64_t now = left < most - units ? left : most - units;
            if (now > 0) {
                const int64_t e = done * kUnit, b = e / kBlock8;
                const int64_t end = (done + now) * kUnit;
                AdamTensor &o = a.t[a.count];
                o.n = (end < t.n ? end : t.n) - e;
                o.at = (uint32_t)e;
                o.p = t.p + e;
                o.g = (const char *)t.g + e * (int64_t)eg;
                o.m = (const char *)t.m + e * (int64_t)es;
                o.v = (const char *)t.v + e * (int64_t)es;
                o.p_out = (t.p_out != nullptr ? t.p_out : t.p) + e;
                o.m_out = (char *)(t.m_out != nullptr ? t.m_out : t.m) + e * (int64_t)es;
                o.v_out = (char *)(t.v_out != nullptr ? t.v_out : t.v) + e * (int64_t)es;
                o.copy = t.copy != nullptr ? (bf16 *)t.copy + e : nullptr;
                if (s8) {
                    o.ms = t.m_scale + b;
                    o.vs = t.v_scale + b;
                    o.ms_out = (t.m_scale_out != nullptr ? t.m_scale_out : t.m_scale) + b;
                    o.vs_out = (t.v_scale_out != nullptr ? t.v_scale_out : t.v_scale) + b;
                }
                a.first[a.count] = (uint32_t)units;
                units += now;
                a.first[++a.count] = (uint32_t)units;
                done += now;
            }
            if (done == all) {
                ++i;
                done = 0;
            }
        }
        if (units == 0) break;
        if (g_io == NAJU_F32) launch<float>(a, (unsigned)units, store, st);
        else launch<bf16>(a, (unsigned)units, store, st);
        NAJU_TRY(hip_status(hipGetLastError(), "AdamW launch"));
    }
    return NAJU_OK;
}
