// Runs of consecutive channels of a row as the element-wise kernels load, hold and store them, and row sums over
// groups of lanes. Included only by the .hip sources of this library.
#pragma once

#include "gdn_device.h"

namespace gdn {

// Eight consecutive channels as they lie in memory, and as fp32: rows wait for their turn as loaded, which halves the
// registers of bf16 rows in flight.
// hide(): the compiler is made to assume that the words may have changed, so that a later get() unpacks them again instead of keeping fp32 values
// from an earlier one, twice the registers, all the way.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void hide() {}
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <> struct Raw8<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(a.x), "+v"(a.y), "+v"(a.z), "+v"(a.w)); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16_lo_half(w[e]);
            x[2 * e + 1] = bf16_hi_half(w[e]);
        }
    }
};
// NT: past the caches.
template <bool NT, typename T>
__device__ __forceinline__ void store_piece(void* p, const T& x) {
    if constexpr (NT) __builtin_nontemporal_store(x, static_cast<T*>(p));
    else *static_cast<T*>(p) = x;
}
template <bool NT>
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    store_piece<NT>(p, f32x4_t{x[0], x[1], x[2], x[3]});
    store_piece<NT>(p + 4, f32x4_t{x[4], x[5], x[6], x[7]});
}
template <bool NT>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    store_piece<NT>(p, u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                               pack_bf16x2(x[6], x[7])});
}

// The same for four channels.
template <typename T> struct Raw4;
template <> struct Raw4<float> {
    float4 a;
    __device__ __forceinline__ void load(const float* p) { a = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; }
    __device__ __forceinline__ void put(float* p) const { *reinterpret_cast<float4*>(p) = a; }
};
template <> struct Raw4<uint16_t> {
    uint2 a;
    __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float (&x)[4]) const {
        x[0] = bf16_lo_half(a.x); x[1] = bf16_hi_half(a.x); x[2] = bf16_lo_half(a.y); x[3] = bf16_hi_half(a.y);
    }
    __device__ __forceinline__ void put(uint16_t* p) const { *reinterpret_cast<uint2*>(p) = a; }
};
__device__ __forceinline__ void store4c(float* p, const float (&x)[4]) { store_piece<false>(p, f32x4_t{x[0], x[1], x[2], x[3]}); }
__device__ __forceinline__ void store4c(uint16_t* p, const float (&x)[4]) {
    store_piece<false>(p, u32x2_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])});
}

// A row at a scalar address (the same in every lane) and a lane's byte offset in it: the empty asm keeps the compiler from adding the two
// parts the other way round, which costs a pair of registers and an addition a load.
typedef __attribute__((address_space(1))) char* global_char_ptr;
template <typename T> __device__ __forceinline__ T* at_byte(T* row, unsigned byte) {
    uint64_t r = reinterpret_cast<uint64_t>(row);
    asm("" : "+s"(r));
    return (T*)((global_char_ptr)r + byte);
}

// Sum over groups of G lanes, in every lane.
template <int G>
__device__ __forceinline__ float row_sum(float x) {
    x += dpp_f32<0xB1>(x);    // quad_perm [1,0,3,2]
    x += dpp_f32<0x4E>(x);    // quad_perm [2,3,0,1]
    x += dpp_f32<0x141>(x);   // row_half_mirror
    if constexpr (G >= 16) x += dpp_f32<0x140>(x);   // row_mirror
    if constexpr (G >= 32) x += __shfl_xor(x, 16, 64);
    if constexpr (G >= 64) x += __shfl_xor(x, 32, 64);
    return x;
}

}  // namespace gdn
