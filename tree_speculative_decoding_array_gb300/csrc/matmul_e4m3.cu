// tsv_matmul_e4m3, tsv_matmul_e4m3_argmax: rows in 8 bits times weights in 8 bits.
//
//   out[m, n] = sum over blocks b of a_scale[m, b] w_scale[n / 128, b] (sum over the 128 features k of b of a[m, k] w[n, k])
#include "e4m3.cuh"

namespace tsv {

constexpr int kTile = 64, kChunk = 32;

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
}

__global__ void __launch_bounds__(256) matmul_e4m3_kernel(const E4Product p) {
    griddep_begin();
    __shared__ float sa[kChunk][kTile + 1], sw[kChunk][kTile + 1];
    const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int blocks = e4_blocks(p.K);
    const uint8_t *a = (const uint8_t*)p.a, *w = (const uint8_t*)p.w;
    float acc[4][4] = {}, part[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += kChunk) {
        for (int e = threadIdx.x; e < kTile * kChunk; e += 256) {
            const int r = e / kChunk, k = e % kChunk;
            sa[k][r] = m0 + r < p.rows && k0 + k < p.K ? e4m3_to_f32(a[(size_t)(m0 + r) * p.K + k0 + k]) : 0.f;
            sw[k][r] = n0 + r < p.N && k0 + k < p.K ? e4m3_to_f32(w[(size_t)(n0 + r) * p.K + k0 + k]) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < kChunk; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[k][ty * 4 + i], sw[k][tx * 4 + j], part[i][j]);
        __syncthreads();
        if ((k0 + kChunk) % kE4Block == 0 || k0 + kChunk >= p.K) {
            const int b = k0 / kE4Block;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
                    if (m < p.rows && n < p.N)
                        acc[i][j] = fmaf(p.a_scale[(size_t)m * blocks + b] * p.w_scale[(size_t)(n / kE4Block) * blocks + b],
                                         part[i][j], acc[i][j]);
                    part[i][j] = 0.f;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= p.rows || n >= p.N) continue;
            const size_t o = (size_t)m * p.N + n;
            if (p.best) atomicMax(&p.best[m], pack_best(acc[i][j], (uint32_t)n));
            else if (p.out_dtype == TSV_F32) ((float*)p.out)[o] = acc[i][j];
            else if (p.out_dtype == TSV_BF16) ((__nv_bfloat16*)p.out)[o] = __float2bfloat16_rn(acc[i][j]);
            else ((__half*)p.out)[o] = __float2half_rn(acc[i][j]);
        }
}

tsv_status launch_matmul_e4m3(const char* name, const E4Product& p, cudaStream_t stream) {
    launch_pdl(matmul_e4m3_kernel, dim3((p.N + kTile - 1) / kTile, (p.rows + kTile - 1) / kTile), 256, 0, stream, p);
    return check_launch(name);
}

// What both entry points ask of their operands.
static tsv_status check_product(const char* name, const E4Product& p) {
    if (p.rows < 0 || p.K < 1 || p.N < 1) return fail(TSV_EINVAL, "%s: rows=%d K=%d N=%d", name, p.rows, p.K, p.N);
    if (p.K % 16) return fail(TSV_EINVAL, "%s: K=%d not a multiple of 16", name, p.K);
    if (p.rows == 0) return TSV_OK;
    if (!p.a || !p.a_scale || !p.w || !p.w_scale) return fail(TSV_EINVAL, "%s: null pointer argument", name);
    if (((uintptr_t)p.a | (uintptr_t)p.w) & 15) return fail(TSV_EINVAL, "%s: a or w not 16-byte aligned", name);
    if (((uintptr_t)p.a_scale | (uintptr_t)p.w_scale) & 3) return fail(TSV_EINVAL, "%s: scales not 4-byte aligned", name);
    return TSV_OK;
}

}  // namespace tsv

extern "C" tsv_status tsv_matmul_e4m3(const void* a, const float* a_scale, int32_t rows, int32_t K, const void* w,
                                      const float* w_scale, int32_t N, void* out, int32_t out_dtype, cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    const E4Product p = {a, a_scale, w, w_scale, rows, K, N, out, out_dtype, nullptr};
    if (out_dtype != TSV_F32 && out_dtype != TSV_BF16 && out_dtype != TSV_F16)
        return fail(TSV_EUNSUPPORTED, "matmul_e4m3: output type %d (fp32, bf16 or fp16 only)", out_dtype);
    const tsv_status st = check_product("matmul_e4m3", p);
    if (st != TSV_OK || rows == 0) return st;
    if (!out) return fail(TSV_EINVAL, "matmul_e4m3: null pointer argument");
    if ((uintptr_t)out & (out_dtype == TSV_F32 ? 3 : 1)) return fail(TSV_EINVAL, "matmul_e4m3: out is not aligned to its elements");
    return launch_matmul_e4m3("matmul_e4m3", p, stream);
}

namespace tsv {
// Defined in lm_head.cu: the running bests of a call, cleared and unpacked on its stream.
size_t lm_best_bytes(int rows);
void launch_lm_best_clear(unsigned long long* best, int rows, cudaStream_t stream);
tsv_status launch_lm_best_unpack(const char* name, const unsigned long long* best, int rows, int32_t* argmax, float* maxval,
                                 cudaStream_t stream);
}  // namespace tsv

extern "C" size_t tsv_matmul_e4m3_argmax_workspace_size(int32_t rows) { return rows < 1 ? 0 : tsv::lm_best_bytes(rows); }

extern "C" tsv_status tsv_matmul_e4m3_argmax(const void* a, const float* a_scale, int32_t rows, int32_t K, const void* w,
                                             const float* w_scale, int32_t N, int32_t* argmax, float* maxval, void* workspace,
                                             size_t ws_bytes, cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    E4Product p = {a, a_scale, w, w_scale, rows, K, N, nullptr, TSV_F32, (unsigned long long*)workspace};
    const tsv_status st = check_product("matmul_e4m3_argmax", p);
    if (st != TSV_OK || rows == 0) return st;
    if (!argmax || !workspace) return fail(TSV_EINVAL, "matmul_e4m3_argmax: null pointer argument");
    if ((uintptr_t)workspace & 15) return fail(TSV_EINVAL, "matmul_e4m3_argmax: workspace not 16-byte aligned");
    if (ws_bytes < lm_best_bytes(rows))
        return fail(TSV_ECAPACITY, "matmul_e4m3_argmax: workspace %zu < %zu bytes", ws_bytes, lm_best_bytes(rows));
    launch_lm_best_clear(p.best, rows, stream);
    const tsv_status done = launch_matmul_e4m3("matmul_e4m3_argmax", p, stream);
    return done != TSV_OK ? done : launch_lm_best_unpack("matmul_e4m3_argmax", p.best, rows, argmax, maxval, stream);
}
