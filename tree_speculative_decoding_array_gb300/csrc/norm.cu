// tsv_add_rms_norm, tsv_quantize_e4m3: the residual's addition and the root-mean-square norm ahead of a product, with
// the normed rows in 16 bits, in 8 bits with a scale per 128 features, or both.
//
//   h = x + residual;  y = h / sqrt(mean(h^2) + eps) * (weight_offset + weight)
//
// Bound by HBM: x and residual are read once, h, y and the codes written once.  A row stays in its CTA's registers
// between the sum of squares and the outputs.  A thread takes 8 consecutive features at a time (16-byte accesses), so
// the 16 lanes of a half-warp hold exactly one group of 128 and its maximum needs four shuffles and no shared memory.
#include "e4m3.cuh"

namespace tsv {

struct NormParams {
    const void *x, *residual, *weight;
    void *residual_out, *out;
    uint8_t* out8;
    float* out8_scale;
    int rows, H;
    float eps, weight_offset;
};

constexpr int kNormMaxThreads = 1024;

// Sum over the CTA, the same in every thread and every run: warps by shuffles, then the warps in order.
__device__ __forceinline__ float cta_sum(float v, float* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += s[w];
    __syncthreads();
    return t;
}

// VPT vectors of 8 features per thread.  VEC: H % 8 == 0 and every row 16-byte aligned.
template <typename T, int VPT, bool VEC>
__global__ void __launch_bounds__(kNormMaxThreads) rms_norm_kernel(const NormParams p) {
    griddep_begin();
    __shared__ float s[32];
    const T *x = (const T*)p.x, *res = (const T*)p.residual, *wt = (const T*)p.weight;
    const size_t row = blockIdx.x, at = row * p.H;
    float h[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * 8, n = p.H - c;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] = 0.f;
        if (n <= 0) continue;
        load8<T, VEC>(x + at + c, n, h[k]);
        if (res) {
            float r[8];
            load8<T, VEC>(res + at + c, n, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] += r[j];
        }
        if (p.residual_out) store8<T, VEC>((T*)p.residual_out + at + c, n, h[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[k][j], h[k][j], ss);
    }
    if (!p.out && !p.out8) return;
    ss = cta_sum(ss, s);
    float eps = p.eps;
    if (ss == INFINITY) {
        // squares beyond fp32: once more with the row's largest value scaled to 2^50 by a power of two, eps with it
        // (values that leave fp32's normal numbers by that are zero after the norm)
        uint32_t m = 0u;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(h[k][j]) & 0x7FFFFFFFu);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        uint32_t* su = reinterpret_cast<uint32_t*>(s);
        if ((threadIdx.x & 31) == 0) su[threadIdx.x >> 5] = m;
        __syncthreads();
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) m = max(m, su[w]);
        __syncthreads();
        if (m < 0x7F800000u) {  // an infinity stays: its row's sum of squares is infinite
            const float scale = exp2f((float)(177 - (int)(m >> 23)));
            ss = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[k][j] *= scale;
                    ss = fmaf(h[k][j], h[k][j], ss);
                }
            ss = cta_sum(ss, s);
            eps *= scale * scale;
        }
    }
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(ss, (float)p.H) + eps));
    const int groups = e4_blocks(p.H);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * 8, n = p.H - c;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
        if (n > 0) {
            float w[8];
            load8<T, VEC>(wt + c, n, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = VEC || j < n ? h[k][j] * rstd * (p.weight_offset + w[j]) : 0.f;
            if (p.out) store8<T, VEC>((T*)p.out + at + c, n, y);
        }
        if (p.out8) {  // the same for the whole CTA
            const float scale = group_scale(y);
            if (n > 0) {
                store_codes<VEC>(p.out8 + at + c, n, group_codes(y, scale));
                if ((threadIdx.x & 15) == 0) p.out8_scale[row * groups + c / kE4Block] = scale;
            }
        }
    }
}

// A half-warp per group of 128 features.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_e4m3_kernel(const T* __restrict__ x, uint8_t* __restrict__ out8,
                                                            float* __restrict__ out8_scale, int rows, int H) {
    griddep_begin();
    const int groups = e4_blocks(H);
    const size_t total = (size_t)rows * groups, step = (size_t)gridDim.x * (blockDim.x >> 4);
    const int l = threadIdx.x & 15;
    // both halves of a warp take part in every shuffle
    for (size_t g0 = (size_t)blockIdx.x * (blockDim.x >> 4) + ((threadIdx.x >> 5) << 1); g0 < total; g0 += step) {
        const size_t g = g0 + ((threadIdx.x >> 4) & 1);
        const size_t row = g / groups;
        const int c = (int)(g - row * groups) * kE4Block + l * 8;
        const int n = g < total ? H - c : 0;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
        if (n > 0) load8<T, VEC>(x + row * H + c, n, y);
        const float scale = group_scale(y);
        if (n > 0) store_codes<VEC>(out8 + row * H + c, n, group_codes(y, scale));
        if (l == 0 && g < total) out8_scale[g] = scale;
    }
}

static bool row_type(int dtype) { return dtype == TSV_F16 || dtype == TSV_BF16 || dtype == TSV_F32; }

template <typename T, bool VEC>
static void launch_norm(const NormParams& p, cudaStream_t stream) {
    const int vecs = (p.H + 7) / 8;
    const int vpt = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
    const int threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
    if (vpt == 1) launch_pdl(rms_norm_kernel<T, 1, VEC>, p.rows, threads, 0, stream, p);
    else if (vpt == 2) launch_pdl(rms_norm_kernel<T, 2, VEC>, p.rows, threads, 0, stream, p);
    else launch_pdl(rms_norm_kernel<T, 4, VEC>, p.rows, threads, 0, stream, p);
}

template <typename T>
static void launch_quantize(const void* x, int rows, int H, uint8_t* out8, float* out8_scale, cudaStream_t stream) {
    const size_t pairs = ((size_t)rows * e4_blocks(H) + 15) / 16;  // CTAs of 16 groups
    const int grid = (int)std::min<size_t>(pairs, (size_t)sm_count() * 8);
    if (H % 8 == 0 && (((uintptr_t)x & 15) | ((uintptr_t)out8 & 7)) == 0)
        launch_pdl(quantize_e4m3_kernel<T, true>, grid, 256, 0, stream, (const T*)x, out8, out8_scale, rows, H);
    else
        launch_pdl(quantize_e4m3_kernel<T, false>, grid, 256, 0, stream, (const T*)x, out8, out8_scale, rows, H);
}

tsv_status launch_quantize_e4m3(const void* x, int rows, int H, int dtype, void* out8, float* out8_scale, cudaStream_t stream) {
    uint8_t* o = (uint8_t*)out8;
    if (dtype == TSV_BF16) launch_quantize<__nv_bfloat16>(x, rows, H, o, out8_scale, stream);
    else if (dtype == TSV_F16) launch_quantize<__half>(x, rows, H, o, out8_scale, stream);
    else launch_quantize<float>(x, rows, H, o, out8_scale, stream);
    return check_launch("quantize_e4m3");
}

}  // namespace tsv

extern "C" tsv_status tsv_add_rms_norm(const void* x, const void* residual, const void* weight, int32_t rows, int32_t H,
                                       int32_t dtype, float eps, float weight_offset, void* residual_out, void* out,
                                       void* out8, float* out8_scale, cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    if (rows < 0 || H < 1) return fail(TSV_EINVAL, "add_rms_norm: rows=%d H=%d", rows, H);
    if (H > 32768) return fail(TSV_ECAPACITY, "add_rms_norm: H=%d above 32768", H);
    if (!row_type(dtype)) return fail(TSV_EUNSUPPORTED, "add_rms_norm: type %d (fp16, bf16 or fp32 only)", dtype);
    if (!(eps >= 1e-30f && eps < INFINITY) || !(fabsf(weight_offset) < INFINITY))
        return fail(TSV_EINVAL, "add_rms_norm: eps=%g (at least 1e-30) weight_offset=%g (finite)", eps, weight_offset);
    if (!residual_out && !out && !out8) return fail(TSV_EINVAL, "add_rms_norm: no output");
    if (rows == 0) return TSV_OK;
    if (!x || !weight) return fail(TSV_EINVAL, "add_rms_norm: null pointer argument");
    if ((out8 != nullptr) != (out8_scale != nullptr)) return fail(TSV_EINVAL, "add_rms_norm: out8 and out8_scale belong together");
    const uintptr_t elt = dtype == TSV_F32 ? 4 : 2;
    const uintptr_t all = (uintptr_t)x | (uintptr_t)residual | (uintptr_t)weight | (uintptr_t)residual_out | (uintptr_t)out;
    if (all & (elt - 1) || (uintptr_t)out8_scale & 3) return fail(TSV_EINVAL, "add_rms_norm: a buffer is not aligned to its elements");
    const NormParams p = {x, residual, weight, residual_out, out, (uint8_t*)out8, out8_scale, rows, H, eps, weight_offset};
    const bool vec = H % 8 == 0 && ((all & 15) | ((uintptr_t)out8 & 7)) == 0;
    if (dtype == TSV_BF16) vec ? launch_norm<__nv_bfloat16, true>(p, stream) : launch_norm<__nv_bfloat16, false>(p, stream);
    else if (dtype == TSV_F16) vec ? launch_norm<__half, true>(p, stream) : launch_norm<__half, false>(p, stream);
    else vec ? launch_norm<float, true>(p, stream) : launch_norm<float, false>(p, stream);
    return check_launch("add_rms_norm");
}

extern "C" tsv_status tsv_quantize_e4m3(const void* x, int32_t rows, int32_t H, int32_t dtype, void* out8, float* out8_scale,
                                        cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    if (rows < 0 || H < 1) return fail(TSV_EINVAL, "quantize_e4m3: rows=%d H=%d", rows, H);
    if (!row_type(dtype)) return fail(TSV_EUNSUPPORTED, "quantize_e4m3: type %d (fp16, bf16 or fp32 only)", dtype);
    if (rows == 0) return TSV_OK;
    if (!x || !out8 || !out8_scale) return fail(TSV_EINVAL, "quantize_e4m3: null pointer argument");
    if ((uintptr_t)x & (dtype == TSV_F32 ? 3 : 1) || (uintptr_t)out8_scale & 3)
        return fail(TSV_EINVAL, "quantize_e4m3: a buffer is not aligned to its elements");
    return launch_quantize_e4m3(x, rows, H, dtype, out8, out8_scale, stream);
}
