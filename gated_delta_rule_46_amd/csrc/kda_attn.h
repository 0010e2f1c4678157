// Fragments, results and exponentials on 32x32 MFMA tiles, 16 deep, shared by the
// window-attention and the paged-attention kernels (bf16; fp32: eight 32x32x2 steps):
// lane l = 32 h + n holds row (column) n of an operand at 8 of the 16 contracted
// places, and column n of the result at rows 8 (r / 4) + 4 h + r % 4.
#pragma once

#include "kda_tiles.h"

typedef float f32x16 __attribute__((ext_vector_type(16)));

namespace kda {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ __forceinline__ f32x16 mma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(const f32x8& a, const f32x8& b, f32x16 c) {
#pragma unroll
    for (int m = 0; m < 8; ++m) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[m], b[m], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = 0.f;
    return z;
}

// rows r0 + n, columns k0 + 8 h + (0..7)
template <class T>
__device__ __forceinline__ typename Frag<T>::V nat32(const T* t, int st, int r0, int k0, int n, int h) {
    return frag_nat(t, st, r0 + n, k0, h);
}
// column c0 + n, rows r0 + 4 h + (0..3) and r0 + 8 + 4 h + (0..3)
__device__ __forceinline__ bf16x8 tr32(const uint16_t* t, int st, int r0, int c0, int lane) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int i = lane & 15, b = (lane >> 4) & 1, h = lane >> 5;
    const uint16_t* p = t + (r0 + 4 * h + (i >> 2)) * st + c0 + 16 * b + 4 * (i & 3);
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 8 * st));
    const auto u = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, u);
}
__device__ __forceinline__ f32x8 tr32(const float* t, int st, int r0, int c0, int lane) {
    const float* p = t + (r0 + 4 * (lane >> 5)) * st + c0 + (lane & 31);
    f32x8 r;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        r[m] = p[m * st];
        r[4 + m] = p[(8 + m) * st];
    }
    return r;
}
// half b of a result tile's rows as an operand (rows contracted)
template <class T> __device__ __forceinline__ typename Frag<T>::V rows16(const f32x16& x, int b) {
    f32x8 y;
#pragma unroll
    for (int m = 0; m < 8; ++m) y[m] = x[8 * b + m];
    return narrow<T>(y);
}
__device__ __forceinline__ int result_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// A lane's values of a result tile, times f, to 32 consecutive columns of a row:
// bf16 halves of 8 columns are swapped with the other half of the wave first, so
// that they go out 16 bytes a lane instead of 8.
template <class T> __device__ __forceinline__ void store_tile(T* row, const f32x16& y, float f, int h) {
#pragma unroll
    for (int r = 0; r < 4; r += 2) {
        const f32x4 a = f32x4{y[4 * r], y[4 * r + 1], y[4 * r + 2], y[4 * r + 3]} * f;
        const f32x4 b = f32x4{y[4 * r + 4], y[4 * r + 5], y[4 * r + 6], y[4 * r + 7]} * f;
        if constexpr (sizeof(T) == 2) {
            u32x2 u, v;
            store4(reinterpret_cast<T*>(&u), a);
            store4(reinterpret_cast<T*>(&v), b);
            const auto s0 = __builtin_amdgcn_permlane32_swap(u[0], v[0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(u[1], v[1], false, false);
            *reinterpret_cast<uint4*>(row + 8 * (r + h)) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
        } else {
            store4(row + 8 * r + 4 * h, a);
            store4(row + 8 * r + 8 + 4 * h, b);
        }
    }
}

// 8 consecutive elements of a row in global memory, or zeros
template <class T> __device__ __forceinline__ typename Frag<T>::V load8(const T* p, bool in) {
    constexpr int N = sizeof(T) / 2;
    uint4 u[N];
#pragma unroll
    for (int m = 0; m < N; ++m) u[m] = in ? reinterpret_cast<const uint4*>(p)[m] : make_uint4(0u, 0u, 0u, 0u);
    typename Frag<T>::V r;
    __builtin_memcpy(&r, u, sizeof(r));
    return r;
}

__device__ __forceinline__ float swap_max(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float swap_sum(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// largest of 16 values (IEEE maximum: takes a product's result as it is, where
// fmaxf would first quiet every operand with an instruction of its own)
__device__ __forceinline__ float tree_max(const f32x16& x) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m[i] = __builtin_elementwise_maximum(__builtin_elementwise_maximum(x[4 * i], x[4 * i + 1]),
                                             __builtin_elementwise_maximum(x[4 * i + 2], x[4 * i + 3]));
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(m[0], m[1]), __builtin_elementwise_maximum(m[2], m[3]));
}

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }   // 1 ulp, no range fix-up

}  // namespace kda
