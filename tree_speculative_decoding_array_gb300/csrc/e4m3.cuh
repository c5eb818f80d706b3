// 8-bit rows: e4m3 codes with one fp32 scale per 128 features, and the row types around them.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace tsv {

constexpr int kE4Block = 128;      // features per scale of a row; rows and features per scale of a weight
constexpr float kE4Inv = 1.f / 448.f;  // 448: the largest e4m3 value

__host__ __device__ constexpr int e4_blocks(int n) { return n / kE4Block + (n % kE4Block != 0); }

// 8 consecutive features of a row as fp32, and back (rounded once).  T: uint16_t-sized bf16 / fp16 or float; `n` of the 8
// are inside the row; VEC: all 8 are and the address is a multiple of the vector's bytes.
template <typename T>
struct RowType;
template <>
struct RowType<__nv_bfloat16> {
    static __device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ void unpack(uint32_t u, float& a, float& b) { a = bf16_lo(u); b = bf16_hi(u); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct RowType<__half> {
    static __device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
    static __device__ __forceinline__ void unpack(uint32_t u, float& a, float& b) {
        const float2 f = f16x2_to_f32x2(u);
        a = f.x;
        b = f.y;
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct RowType<float> {
    static __device__ __forceinline__ float to_f32(float x) { return x; }
    static __device__ __forceinline__ float from_f32(float x) { return x; }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? RowType<T>::to_f32(p[j]) : 0.f;
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        RowType<T>::unpack(u.x, v[0], v[1]);
        RowType<T>::unpack(u.y, v[2], v[3]);
        RowType<T>::unpack(u.z, v[4], v[5]);
        RowType<T>::unpack(u.w, v[6], v[7]);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[8]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = RowType<T>::from_f32(v[j]);
    } else if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(RowType<T>::pack(v[0], v[1]), RowType<T>::pack(v[2], v[3]),
                                                  RowType<T>::pack(v[4], v[5]), RowType<T>::pack(v[6], v[7]));
    }
}

// The 16 lanes of a half-warp hold the 128 features of one group, 8 each (zeros past the row's end): codes and scale.
// The maximum is taken over the bits of |y|, so that a NaN, whose bits are above infinity's, is not lost.
__device__ __forceinline__ float group_scale(const float (&y)[8]) {
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return __fmul_rn(__uint_as_float(m), kE4Inv);
}

__device__ __forceinline__ uint2 group_codes(const float (&y)[8], float scale) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 q = scale == 0.f ? make_float2(0.f, 0.f)
                                      : make_float2(__fdiv_rn(y[2 * j], scale), __fdiv_rn(y[2 * j + 1], scale));
        w[j] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint2 c) {
    if constexpr (VEC) {
        *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = (uint8_t)((j < 4 ? c.x >> (8 * j) : c.y >> (8 * (j - 4))) & 0xFFu);
    }
}

// Bytes of an 8-bit copy of `rows` rows of H features: codes, then scales, each rounded up to 256.
inline size_t e4_codes_bytes(int rows, int H) { return ((size_t)rows * H + 255) & ~(size_t)255; }
inline size_t e4_rows_bytes(int rows, int H) {
    return e4_codes_bytes(rows, H) + (((size_t)rows * e4_blocks(H) * 4 + 255) & ~(size_t)255);
}

// Defined in norm.cu and matmul_e4m3.cu; arguments already checked.
tsv_status launch_quantize_e4m3(const void* x, int rows, int H, int dtype, void* out8, float* out8_scale, cudaStream_t stream);

struct E4Product {
    const void* a;
    const float* a_scale;
    const void* w;
    const float* w_scale;
    int rows, K, N;
    void* out;      // [rows, N] of out_dtype, or NULL
    int out_dtype;
    unsigned long long* best;  // packed (value, ~index) per row, raised by the products, or NULL
};
tsv_status launch_matmul_e4m3(const char* name, const E4Product& p, cudaStream_t stream);

}  // namespace tsv
