// naju_vec.h -- short runs of elements moved as one wide access.
//
// Rows of odd length start at any element, so the accesses are declared with
// the element's own alignment: gfx950 serves a 16-byte global access at any
// byte address, and one that crosses a 128-byte line costs a second request.
#pragma once

#include "naju_device.h"

namespace naju {

// n elements (a power of two, at most 16 bytes in all) as raw words
template <typename IO, int n> struct Run {
    static constexpr int kWords = n * (int)sizeof(IO) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const IO *p) { __builtin_memcpy(w, p, sizeof(w)); }
    __device__ __forceinline__ void store(IO *p) const { __builtin_memcpy(p, w, sizeof(w)); }
    // at a 32-bit byte offset from an address that the wave shares
    __device__ __forceinline__ void load_at(const IO *base, uint32_t bytes) {
        __builtin_memcpy(w, (const char *)base + bytes, sizeof(w));
    }
    __device__ __forceinline__ void store_at(IO *base, uint32_t bytes) const {
        __builtin_memcpy((char *)base + bytes, w, sizeof(w));
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // the first m elements, zeros after them (0 <= m < n)
    __device__ __forceinline__ void load_part(const IO *p, int m) {
        zero();
#pragma unroll
        for (int i = 0; i < n - 1; ++i)
            if (i < m) put_raw(i, p[i]);
    }
    __device__ __forceinline__ void store_part(IO *p, int m) const {
#pragma unroll
        for (int i = 0; i < n - 1; ++i)
            if (i < m) p[i] = get_raw(i);
    }
    __device__ __forceinline__ IO get_raw(int i) const;
    __device__ __forceinline__ void put_raw(int i, IO v);
    __device__ __forceinline__ float get(int i) const { return to_f(get_raw(i)); }
    // The packed words as if they were new: what was unpacked from them before is
    // not kept in registers for a later use.
    __device__ __forceinline__ void repack() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
    }
    // replaces an element
    __device__ __forceinline__ void set_raw(int i, IO v) {
        if constexpr (sizeof(IO) == 2) w[i / 2] &= 0xffff0000u >> (16 * (i % 2));
        else w[i] = 0u;
        put_raw(i, v);
    }
};

template <typename IO, int n> __device__ __forceinline__ IO Run<IO, n>::get_raw(int i) const
{
    if constexpr (sizeof(IO) == 4) return __builtin_bit_cast(IO, w[i]);
    else return (IO)(w[i / 2] >> (16 * (i % 2)));
}
template <typename IO, int n> __device__ __forceinline__ void Run<IO, n>::put_raw(int i, IO v)
{
    if constexpr (sizeof(IO) == 4) w[i] = __builtin_bit_cast(uint32_t, v);
    else w[i / 2] |= (uint32_t)v << (16 * (i % 2));  // (its half is zero)
}

// n floats rounded to the io type
template <typename IO, int n> __device__ __forceinline__ Run<IO, n> round_run(const float *f)
{
    Run<IO, n> r;
#pragma unroll
    for (int i = 0; i < Run<IO, n>::kWords; ++i) {
        if constexpr (sizeof(IO) == 4) {
            r.w[i] = __float_as_uint(f[i]);
        } else {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            const bf16x2 v = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
            r.w[i] = __builtin_bit_cast(uint32_t, v);
        }
    }
    return r;
}

// elements in a 16-byte access
template <typename IO> constexpr int kPer16 = 16 / (int)sizeof(IO);

}  // namespace naju
