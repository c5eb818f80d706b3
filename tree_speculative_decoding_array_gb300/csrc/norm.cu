// tsv_add_rms_norm, tsv_quantize_e4m3: the residual's addition and the root-mean-square norm ahead of a product, with
// the normed rows in 16 bits, in 8 bits with a scale per 128 features, or both.
//
//   h = x + residual;  y = h / sqrt(mean(h^2) + eps) * (weight_offset + weight)
//
// Bound by HBM: x and residual are read once, h, y and the codes written once.  A row stays in its threads' registers between the
// sum of squares and the outputs.  Where every row is 16-byte aligned a thread takes 8 consecutive features at a time, and the 16 lanes
// of a half-warp hold one group of 128; else a warp takes two groups at a time, its lanes neighbouring features (8 in a row per
// thread, one by one, had cost three times as much).  Either way a group's maximum needs shuffles and no shared memory.  Short rows share a
// CTA.
#include <algorithm>
#include <atomic>

#include "e4m3.cuh"

namespace tsv {

struct NormParams {
    const void *x, *residual, *weight;
    void *residual_out, *out;
    uint8_t* out8;
    float* out8_scale;
    int rows, H;
    float eps, weight_offset, inv_h;
};

// Where the 8 features of a thread's k-th portion of a row are, and the groups of 128 among them.
template <bool VEC>
struct Portion {
    static constexpr int kGroups = VEC ? 1 : 2, kPer = 8 / kGroups;  // groups that a thread has features of, features in each
    int c;  // the first feature
    __device__ __forceinline__ Portion(int k, int thread, int threads) {
        if constexpr (VEC) c = (k * threads + thread) * 8;
        else c = ((k * threads + thread) / 32) * 256 + (thread & 31);
    }
    __device__ __forceinline__ int at(int j) const { return VEC ? c + j : c + j * 32; }  // of feature j
    // largest magnitude in group g, from every lane that has a part of it
    __device__ __forceinline__ float largest(const float (&y)[8], int g) const {
        float m = y[g * kPer];
#pragma unroll
        for (int j = 1; j < kPer; ++j) m = larger_magnitude(m, y[g * kPer + j]);
#pragma unroll
        for (int o = VEC ? 8 : 16; o > 0; o >>= 1) m = larger_magnitude(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        return m;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T* row, int H, float (&v)[8]) const {
        if constexpr (VEC) {
            load8(row + c, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = at(j) < H ? RowType<T>::to_f32(row[at(j)]) : 0.f;
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, int H, const float (&v)[8]) const {
        if constexpr (VEC) {
            store8<T, true>(row + c, 8, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at(j) < H) row[at(j)] = RowType<T>::from_f32(v[j]);
        }
    }
    // Codes and scales of the groups; every lane of the warp takes part.  EXACT: the quotients rounded to nearest; else within two units
    // in the last place, of values that are no more exact themselves.
    template <bool EXACT>
    __device__ __forceinline__ void quantize(const float (&y)[8], uint8_t* codes, float* scales, int H) const {
        float q[8];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const float scale = e4_scale(largest(y, g));
            if (!EXACT && e4_ordinary(scale)) {
                const float r = __frcp_rn(scale);
#pragma unroll
                for (int j = 0; j < kPer; ++j) q[g * kPer + j] = y[g * kPer + j] * r;
            } else {
                group_quotients<kPer>(y + g * kPer, scale, q + g * kPer);
            }
            const int f = at(g * kPer);
            if ((threadIdx.x & (VEC ? 15 : 31)) == 0 && f < H) scales[f / kE4Block] = scale;
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = e4_pair(q[2 * j], q[2 * j + 1]);
        if constexpr (VEC) {
            if (c < H) *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at(j) < H) codes[at(j)] = (uint8_t)(w[j / 2] >> (8 * (j & 1)));
        }
    }
};

// Sum over the `warps` warps of a row (this one is number `warp` of the CTA, the row's first is `first`), the same in every thread and
// every run.  The whole CTA calls it together, and not again with the same s before its next barrier.
__device__ __forceinline__ float warp_sum1(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float row_sum(float v, float* s, int warp, int warps, int first) {
    v = warp_sum1(v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    return warp_sum1(lane < warps ? s[first + lane] : 0.f);
}

// How a row is spread.  kAhead: a thread asks for its part of the next row before it works on this one, and keeps its weights in
// registers (16391 rows of 5120, sum and 16-bit output: 111 -> 103 us; 4096 rows of 12288: 141 -> 98).  One portion per thread where 1024
// threads suffice: two had cost 121 us, since the warps that an SM holds hide each other's barriers and shuffles.
template <int VPT, int THREADS, bool VEC>
struct NormShape {
    static constexpr bool kAhead = VEC && (VPT == 1 || THREADS <= 512);
    static constexpr int kPerSm = THREADS == 256 ? 4 : THREADS == 640 ? 2 : 1;  // CTAs of THREADS that an SM has to hold
};

// 8 features of a row as they came from memory.
template <typename T>
struct Raw {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) u[i] = ldg_stream16(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const { load8(reinterpret_cast<const T*>(u), v); }
};

// VPT portions per thread; `threads` threads (whole warps) per row, as many rows at a time as fit the CTA.  VEC: H % 8 == 0 and every
// row 16-byte aligned (codes: 8-byte).
template <typename T, int VPT, int THREADS, bool VEC>
__global__ void __launch_bounds__(THREADS, NormShape<VPT, THREADS, VEC>::kPerSm) rms_norm_kernel(const NormParams p, int threads) {
    griddep_begin();
    constexpr bool kAhead = NormShape<VPT, THREADS, VEC>::kAhead;
    constexpr int RAW = kAhead ? VPT : 1;
    __shared__ float s[3][32];
    const int thread = threadIdx.x % threads, warp = threadIdx.x >> 5, warps = threads >> 5, together = blockDim.x / threads;
    const bool sums = p.out || p.out8;
    const int first_warp = warp / warps * warps;  // once: the division in every row cost up to 7 % (8192 rows of 8192: 90 us, 84 without)
    const T *x = (const T*)p.x, *res = (const T*)p.residual, *wt = (const T*)p.weight;
    Raw<T> xr[RAW], rr[RAW], wr[RAW];
    auto ask = [&](long long row) {
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = (k * threads + thread) * 8;
                if (row >= p.rows || c >= p.H) continue;
                xr[k].load(x + row * p.H + c);
                if (res) rr[k].load(res + row * p.H + c);
            }
        }
    };
    const long long sub = threadIdx.x / threads, step = (long long)gridDim.x * together;
    ask((long long)blockIdx.x * together + sub);
    if constexpr (kAhead)
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            if ((k * threads + thread) * 8 < p.H && sums) wr[k].load(wt + (k * threads + thread) * 8);
    int turn = 0;
    for (long long base = (long long)blockIdx.x * together; base < p.rows; base += step, turn ^= 1) {
        const long long row = base + sub;
        const bool real = row < p.rows;
        const size_t at = (size_t)(real ? row : 0) * p.H;
        float h[VPT][8];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const Portion<VEC> part(k, thread, threads);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[k][j] = 0.f;
            if (!real || part.c >= p.H) continue;
            if constexpr (kAhead) xr[k].values(h[k]);
            else part.load(x + at, p.H, h[k]);
            if (res) {
                float r[8];
                if constexpr (kAhead) rr[k].values(r);
                else part.load(res + at, p.H, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[k][j] += r[j];
            }
        }
        ask(row + step);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const Portion<VEC> part(k, thread, threads);
            if (p.residual_out && real && part.c < p.H) part.store((T*)p.residual_out + at, p.H, h[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(h[k][j], h[k][j], ss);
        }
        if (!sums) continue;
        ss = row_sum(ss, s[turn], warp, warps, first_warp);
        float eps = p.eps;
        // the same for the whole CTA where it takes part in a barrier
        if (warps == 1 || together == 1 ? ss == INFINITY : __syncthreads_or(ss == INFINITY)) {
            // squares beyond fp32: once more with the row's largest value scaled to 2^50 by a power of two, eps with it
            // (values that leave fp32's normal numbers by that are zero after the norm)
            uint32_t m = 0u;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(h[k][j]) & 0x7FFFFFFFu);
            m = __reduce_max_sync(0xFFFFFFFFu, m);
            if (warps > 1) {
                uint32_t* su = reinterpret_cast<uint32_t*>(s[2]);
                __syncthreads();
                if ((threadIdx.x & 31) == 0) su[warp] = m;
                __syncthreads();
                for (int w = first_warp; w < first_warp + warps; ++w) m = max(m, su[w]);
            }
            // rows of finite sums stay as they are, and an infinity stays: its row's sum of squares is infinite
            const float scale = ss == INFINITY && m < 0x7F800000u ? exp2f((float)(177 - (int)(m >> 23))) : 1.f;
            ss = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[k][j] *= scale;
                    ss = fmaf(h[k][j], h[k][j], ss);
                }
            if (warps > 1) __syncthreads();
            ss = row_sum(ss, s[turn], warp, warps, first_warp);
            eps *= scale * scale;
        }
        const float rstd = rsqrtf(fmaf(ss, p.inv_h, eps));  // within 2 ulp; IEEE root and quotients had cost more than the row's sums
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const Portion<VEC> part(k, thread, threads);
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = 0.f;
            if (real && part.c < p.H) {
                float w[8];
                if constexpr (kAhead) wr[k].values(w);
                else part.load(wt, p.H, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (p.weight_offset != 0.f) w[j] += p.weight_offset;
                    y[j] = VEC || part.at(j) < p.H ? h[k][j] * rstd * w[j] : 0.f;
                }
                if (p.out) part.store((T*)p.out + at, p.H, y);
            }
            if (p.out8) part.template quantize<false>(y, p.out8 + at, p.out8_scale + (real ? row : 0) * e4_blocks(p.H), real ? p.H : 0);
        }
    }
}

// VEC: a half-warp per group of 128 features, both halves of a warp in every shuffle.  Else a warp per two groups of a row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_e4m3_kernel(const T* __restrict__ x, uint8_t* __restrict__ out8,
                                                            float* __restrict__ out8_scale, int rows, int H) {
    griddep_begin();
    const int groups = e4_blocks(H), units = VEC ? groups : (groups + 1) / 2;  // of a row
    const size_t total = (size_t)rows * units, step = (size_t)gridDim.x * (VEC ? 16 : 8);
    for (size_t u0 = (size_t)blockIdx.x * (VEC ? 16 : 8) + (threadIdx.x >> 5) * (VEC ? 2 : 1); u0 < total; u0 += step) {
        const size_t u = u0 + (VEC ? (threadIdx.x >> 4) & 1 : 0), row = u / units;
        Portion<VEC> part(0, 0, 0);
        part.c = (int)(u - row * units) * (VEC ? kE4Block : 2 * kE4Block) + (VEC ? (threadIdx.x & 15) * 8 : threadIdx.x & 31);
        const bool mine = u < total && part.c < H;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
        if (mine) part.load(x + row * H, H, y);
        part.template quantize<true>(y, out8 + row * H, out8_scale + row * groups, u < total ? H : 0);
    }
}

static bool row_type(int dtype) { return dtype == TSV_F16 || dtype == TSV_BF16 || dtype == TSV_F32; }

template <typename T, int VPT, int THREADS, bool VEC>
static void launch_norm_as(const NormParams& p, int vecs, cudaStream_t stream) {
    const int threads = ((vecs + VPT - 1) / VPT + 31) / 32 * 32, together = std::max(1, 256 / threads), block = threads * together;
    const auto kernel = rms_norm_kernel<T, VPT, THREADS, VEC>;
    static std::atomic<int> per_sm[THREADS / 32 + 1];  // CTAs resident on an SM, by the CTA's warps (the same on every GPU of the build's kind)
    int fit = per_sm[block / 32].load(std::memory_order_relaxed);
    if (fit == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, block, 0) != cudaSuccess || fit < 1) fit = 1;
        per_sm[block / 32].store(fit, std::memory_order_relaxed);
    }
    const long long ctas = ((long long)p.rows + together - 1) / together;
    launch_pdl(kernel, (int)std::min<long long>(ctas, (long long)sm_count() * fit), block, 0, stream, p, threads);
}

template <typename T, bool VEC>
static void launch_norm(const NormParams& p, cudaStream_t stream) {
    const int vecs = VEC ? p.H / 8 : (p.H + 255) / 256 * 32;  // threads, with 8 features each; short rows share a CTA
    if (vecs <= 256) launch_norm_as<T, 1, 256, VEC>(p, vecs, stream);
    else if (vecs <= 640) launch_norm_as<T, 1, 640, VEC>(p, vecs, stream);
    else if (vecs <= 1024) launch_norm_as<T, 1, 1024, VEC>(p, vecs, stream);
    else if (vecs <= 2048) launch_norm_as<T, 4, 512, VEC>(p, vecs, stream);
    else launch_norm_as<T, 4, 1024, VEC>(p, vecs, stream);
}

template <typename T>
static void launch_quantize(const void* x, int rows, int H, uint8_t* out8, float* out8_scale, cudaStream_t stream) {
    const bool vec = H % 8 == 0 && (((uintptr_t)x & 15) | ((uintptr_t)out8 & 7)) == 0;
    const size_t per = vec ? 16 : 8, units = (size_t)rows * (vec ? e4_blocks(H) : (e4_blocks(H) + 1) / 2);
    const int grid = (int)std::min<size_t>((units + per - 1) / per, (size_t)sm_count() * 8);
    if (vec) launch_pdl(quantize_e4m3_kernel<T, true>, grid, 256, 0, stream, (const T*)x, out8, out8_scale, rows, H);
    else launch_pdl(quantize_e4m3_kernel<T, false>, grid, 256, 0, stream, (const T*)x, out8, out8_scale, rows, H);
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
    const NormParams p = {x, residual, weight, residual_out, out, (uint8_t*)out8, out8_scale, rows, H, eps, weight_offset, 1.f / H};
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
