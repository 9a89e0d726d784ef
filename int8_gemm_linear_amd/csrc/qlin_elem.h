// The element types of plain rows (fp32, bf16 bits, fp16) as fp32 values.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qlin_device.h"

namespace qlin {

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ inline float get(float v) { return v; }
    static __device__ inline float put(float v) { return v; }
};
template <> struct Elem<__half> {
    static __device__ inline float get(__half v) { return __half2float(v); }
    static __device__ inline __half put(float v) { return __float2half(v); }
};
template <> struct Elem<uint16_t> {                // bf16 bits
    static __device__ inline float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ inline uint16_t put(float v) { return bf16_bits(v); }
};

// Piece of 16 bytes at an element's alignment (the hardware loads and stores 16
// bytes at any address).
template <typename T>
__device__ inline v4i load_piece(const T *p)
{
    v4i v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// The fp32 values of a piece.
template <typename T, int E = 16 / sizeof(T)>
__device__ inline void piece_values(float (&f)[E], v4i v)
{
    T t[E];
    __builtin_memcpy(t, &v, 16);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = Elem<T>::get(t[i]);
}

// The piece of fp32 values, each rounded to T once.
template <typename T, int E = 16 / sizeof(T)>
__device__ inline v4i value_piece(const float (&f)[E])
{
    T t[E];
#pragma unroll
    for (int i = 0; i < E; ++i) t[i] = Elem<T>::put(f[i]);
    v4i v;
    __builtin_memcpy(&v, t, 16);
    return v;
}

}  // namespace qlin
