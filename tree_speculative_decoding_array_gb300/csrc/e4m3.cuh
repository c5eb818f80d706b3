// 8-bit rows: e4m3 codes with one fp32 scale per 128 features, and the row types around them.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace tsv {

constexpr int kE4Block = 128;      // features per scale of a row; rows and features per scale of a weight
constexpr float kE4Inv = 1.f / 448.f;  // 448: the largest e4m3 value

__host__ __device__ constexpr int e4_blocks(int n) { return n / kE4Block + (n % kE4Block != 0); }

// Row types: to and from fp32 (rounded once), one by one and, 16-bit types, two at a time.
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

// 8 features from an address that is a multiple of 16 bytes.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
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

// 8 features, VEC: to an address that is a multiple of 16 bytes; else the first n of them, one by one.
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float* v) {
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

// The larger magnitude of two values, with some sign; a NaN if either is one.
__device__ __forceinline__ float larger_magnitude(float a, float b) {
    float m;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
// A group's scale from its largest magnitude.
__device__ __forceinline__ float e4_scale(float largest) { return __fmul_rn(fabsf(largest), kE4Inv); }
__device__ __forceinline__ bool e4_ordinary(float scale) { return scale >= 0x1p-100f && scale <= 0x1p100f; }

// y / scale in fp32, rounded to nearest, for N of a group's values.  Where scale is an ordinary number the quotient is y r with one
// residual step, r the rounded reciprocal: correctly rounded unless scale's significand is all ones (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990), and three instructions where a division takes about ten.  A
// residual that underflows belongs to a quotient far below the smallest code.
template <int N>
__device__ __forceinline__ void group_quotients(const float* y, float scale, float* q) {
    if (e4_ordinary(scale) && (__float_as_uint(scale) & 0x7FFFFFu) != 0x7FFFFFu) {
        const float r = __frcp_rn(scale);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float p = __fmul_rn(y[j], r);
            q[j] = fmaf(fmaf(-p, scale, y[j]), r, p);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = scale == 0.f ? 0.f : __fdiv_rn(y[j], scale);
    }
}

// Two quotients' codes, the first in the low byte.
__device__ __forceinline__ uint32_t e4_pair(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
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
