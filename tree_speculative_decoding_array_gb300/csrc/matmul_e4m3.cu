// tsv_matmul_e4m3, tsv_matmul_e4m3_argmax: rows in 8 bits times weights in 8 bits.
//
//   out[m, n] = sum over blocks b of a_scale[m, b] w_scale[n / 128, b] (sum over the 128 features k of b of a[m, k] w[n, k])
//
// One kernel for every size.  A CTA's tile is 128 rows of a (TMEM lanes) x BN weights (TMEM columns); per block of 128 features four
// tcgen05 MMAs (K = 32) sum the products of codes, which are exact, into one of NB accumulators in TMEM.  The scales differ
// from block to block, so the epilogue warps take every block's sums out of TMEM and add them, scaled, to fp32 sums in
// registers.  A thread holds one row, so its scale is one number per block; and since BN is a power of two, no warp's columns
// cross a block of 128 weights.  The argmax of a row is then a thread's own loop, without shuffles.
//
// Few rows (rows <= 128): bound by reading the weights once.  The MMA's 128 rows are padded, which costs nothing: 16 KB of
// weights take 745 SM clocks from HBM and 270 on the tensor pipe.  Many rows: CTA pairs share MMAs of 256 x 256, each CTA with its
// own 128 rows and half of the weights in shared memory (32 KB per block instead of the 48 KB of a CTA alone, which L2 does not
// deliver in the 512 clocks that its MMAs take).
#include <cuda.h>

#include <algorithm>

#include "e4m3.cuh"
#include "tc.cuh"

namespace tsv {

constexpr int kMmRows = 128;  // rows of a per CTA
constexpr int kMmMaxStages = 24;

struct MmParams {
    CUtensorMap amap, wmap;  // uint8 [rows][K] box 128 x abox; uint8 [N][K] box 128 x wbox; both 128-byte swizzled
    E4Product p;
    int blocks;              // of 128 features
    int mtiles, ntiles;      // of 128 rows (pairs: 256), of BN weights
    int panel;               // row tiles that are walked together, so that their weights are read from L2
    int stages, stage_bytes, a_bytes;
};

template <int BN, bool PAIR>
struct MmShape {
    static constexpr int kEpiWarps = BN >= 128 ? 8 : 4;
    static constexpr int kCols = BN / (kEpiWarps / 4);     // columns of an epilogue thread
    static constexpr int kBufs = BN == 256 ? 2 : 256 / BN;  // accumulators in TMEM
    static constexpr int kThreads = (kEpiWarps + 2) * 32;
    static constexpr int kPerSm = BN >= 128 ? 1 : 2;
    static constexpr int kSmem = kPerSm == 1 ? 224 * 1024 : 110 * 1024;
};

// acc += s * d, two fp32 numbers at a time.
__device__ __forceinline__ void fma2(unsigned long long& acc, uint32_t d0, uint32_t d1, unsigned long long s) {
    asm("{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n fma.rn.f32x2 %0, d, %3, %0;\n}" : "+l"(acc) : "r"(d0), "r"(d1), "l"(s));
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(MmShape<BN, PAIR>::kThreads, MmShape<BN, PAIR>::kPerSm)
    matmul_e4m3_kernel(const __grid_constant__ MmParams q) {
    griddep_begin();
    using S = MmShape<BN, PAIR>;
    constexpr int CTAS = PAIR ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMmMaxStages], empty[kMmMaxStages], acc_full[S::kBufs], acc_empty[S::kBufs], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? tc::cluster_rank() : 0;
    const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS, tiles = q.mtiles * q.ntiles;
    const int KB = q.blocks, ST = q.stages;
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < S::kBufs; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            tc::mbar_init(&acc_empty[b], S::kEpiWarps * CTAS);
        }
        tc::mbar_init(&drain, 1);
        abort_word = 0;
        tc::fence_mbar_init();
    }
    constexpr uint32_t kTmemCols = S::kBufs * BN;
    if (warp == S::kEpiWarps + 1) {
        if constexpr (PAIR) {
            tc::tmem_alloc_pair(&tmem_slot, kTmemCols);
        } else {
            tc::tmem_alloc(&tmem_slot, kTmemCols);
            tc::tmem_relinquish();
        }
    }
    __syncthreads();
    if constexpr (PAIR) tc::cluster_sync();  // both CTAs' barriers exist before either's copies or MMAs reach them
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // tile -> (row tile, weight tile): panels of row tiles, within a panel the row tile changes first
    auto place = [&](int t, int& m, int& n) {
        const int per = q.panel * q.ntiles, p0 = t / per * q.panel, r = t - t / per * per;
        const int wide = min(q.panel, q.mtiles - p0);
        n = r / wide;
        m = p0 + r - n * wide;
    };

    if (warp == S::kEpiWarps) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tc::tma_prefetch_desc(&q.amap);
            tc::tma_prefetch_desc(&q.wmap);
            int st = 0, issued = 0;
            uint32_t fill = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                int m, n;
                place(t, m, n);
                const int arow = (m * CTAS + rank) * kMmRows, wrow = n * BN + rank * (BN / CTAS);
                for (int kb = 0; kb < KB; ++kb) {
                    if (issued >= ST && !tc::mbar_wait(&empty[st], fill ^ 1u, abort_flag, 256)) { ok = false; break; }
                    uint8_t* a = ring + (size_t)st * q.stage_bytes;
                    if constexpr (PAIR) {
                        const uint32_t bar = tc::cluster_addr(&full[st], 0);
                        if (rank == 0) tc::mbar_expect_tx(&full[st], 2u * q.stage_bytes);
                        tc::tma_load_2d_pair(a, &q.amap, bar, kb * kE4Block, arow);
                        tc::tma_load_2d_pair(a + q.a_bytes, &q.wmap, bar, kb * kE4Block, wrow);
                    } else {
                        tc::mbar_expect_tx(&full[st], q.stage_bytes);
                        tc::tma_load_2d(a, &q.amap, &full[st], kb * kE4Block, arow);
                        tc::tma_load_2d(a + q.a_bytes, &q.wmap, &full[st], kb * kE4Block, wrow);
                    }
                    ++issued;
                    if (++st == ST) { st = 0; fill ^= 1u; }
                }
            }
            if (*abort_flag && rank == 0)  // let the copies in flight land (bounded) before the CTA goes away
                for (int i = max(0, issued - ST); i < issued; ++i) tc::mbar_drain(&full[i % ST], (i / ST) & 1);
        }
    } else if (warp == S::kEpiWarps + 1) {
        // ------------------------------------------------------------ MMA issuer (of a pair: its first CTA's)
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = tc::idesc_e4m3(kMmRows * CTAS, BN);
            const uint64_t d0 = tc::sdesc_sw128(tc::smem_u32(ring), 16, 1024);
            int st = 0, buf = 0;
            uint32_t ph = 0, use = 0;  // parities of the stage's fill and of the accumulator's use
            bool ok = true, reused = false;
            for (int t = first; ok && t < tiles; t += step) {
                for (int kb = 0; kb < KB; ++kb) {
                    if (reused && !tc::mbar_wait_spin(&acc_empty[buf], use ^ 1u, abort_flag)) { ok = false; break; }
                    if (!tc::mbar_wait_spin(&full[st], ph, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
                    const uint64_t da = tc::sdesc_add(d0, (uint32_t)st * q.stage_bytes), db = tc::sdesc_add(da, q.a_bytes);
#pragma unroll
                    for (int k = 0; k < kE4Block / 32; ++k)
                        tc::mma_e4m3<PAIR>(tmem + buf * BN, tc::sdesc_add(da, k * 32), tc::sdesc_add(db, k * 32), idesc, k > 0);
                    if constexpr (PAIR) {
                        tc::mma_commit_pair(&empty[st]);
                        tc::mma_commit_pair(&acc_full[buf]);
                    } else {
                        tc::mma_commit(&empty[st]);
                        tc::mma_commit(&acc_full[buf]);
                    }
                    if (++st == ST) { st = 0; ph ^= 1u; }
                    if (++buf == S::kBufs) { buf = 0; use ^= 1u; reused = true; }
                }
            }
            if constexpr (PAIR) tc::mma_commit_pair(&drain);
            else tc::mma_commit(&drain);
            tc::mbar_drain(&drain, 0);
        }
    } else {
        // ------------------------------------------------------------ epilogue: scale and add up, then write out
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + half * S::kCols;
        const uint32_t bar0 = tc::cluster_addr(&acc_empty[0], 0);
        const E4Product& p = q.p;
        int buf = 0;
        uint32_t use = 0;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
            int m, n;
            place(t, m, n);
            const int row = (m * CTAS + rank) * kMmRows + quarter * 32 + lane, col = n * BN + half * S::kCols;
            const bool live = row < p.rows;
            const float* as = p.a_scale + (size_t)(live ? row : 0) * KB;
            const float* ws = p.w_scale + (size_t)(min(col, p.N - 1) / kE4Block) * KB;
            unsigned long long acc[S::kCols / 2];
#pragma unroll
            for (int c = 0; c < S::kCols / 2; ++c) acc[c] = 0ull;
            float sa = __ldg(as), sw = __ldg(ws);
            for (int kb = 0; kb < KB; ++kb) {
                const float sc = sa * sw;
                const unsigned long long s2 = (unsigned long long)__float_as_uint(sc) << 32 | __float_as_uint(sc);
                if (kb + 1 < KB) sa = __ldg(as + kb + 1), sw = __ldg(ws + kb + 1);
                if (!__all_sync(0xFFFFFFFFu, tc::mbar_wait(&acc_full[buf], use, abort_flag))) { ok = false; break; }
                tc::tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < S::kCols; c0 += 32) {
                    uint32_t d[32];
                    tc::tmem_ld32(taddr + buf * BN + c0, d);
                    tc::tmem_wait_ld();
                    if (c0 + 32 == S::kCols) {
                        tc::tc_fence_before();
                        __syncwarp();
                        if constexpr (PAIR) tc::mbar_arrive_one_cluster(bar0 + buf * 8);
                        else tc::mbar_arrive_one(&acc_empty[buf]);
                    }
#pragma unroll
                    for (int c = 0; c < 32; c += 2) fma2(acc[(c0 + c) / 2], d[c], d[c + 1], s2);
                }
                if (++buf == S::kBufs) { buf = 0; use ^= 1u; }
            }
            if (!ok || !live) continue;
            if (p.best) {
                float best = 0.f;
                int at = -1;
#pragma unroll
                for (int c = 0; c < S::kCols; ++c) {
                    const float2 v2 = unpack2(acc[c / 2]);
                    const float v = c & 1 ? v2.y : v2.x;
                    if (col + c < p.N && (at < 0 || orderable(v) > orderable(best))) best = v, at = col + c;
                }
                if (at >= 0) atomicMax(&p.best[row], pack_best(best, (uint32_t)at));
            } else {
#pragma unroll
                for (int c = 0; c < S::kCols; ++c) {
                    const float2 v2 = unpack2(acc[c / 2]);
                    const float v = c & 1 ? v2.y : v2.x;
                    const size_t o = (size_t)row * p.N + col + c;
                    if (col + c >= p.N) continue;
                    if (p.out_dtype == TSV_F32) ((float*)p.out)[o] = v;
                    else if (p.out_dtype == TSV_BF16) ((__nv_bfloat16*)p.out)[o] = __float2bfloat16_rn(v);
                    else ((__half*)p.out)[o] = __float2half_rn(v);
                }
            }
        }
    }
    __syncthreads();
    // the pair's second CTA: the last arrivals of the first one's commits have to come in as well
    if (PAIR && rank == 1 && threadIdx.x == 0) tc::mbar_drain(&drain, 0);
    if constexpr (PAIR) tc::cluster_sync();  // neither CTA's memory goes while the other's copies, MMAs or arrivals use it
    if (warp == S::kEpiWarps + 1) {
        tc::tc_fence_after();
        if constexpr (PAIR) tc::tmem_dealloc_pair(tmem, kTmemCols);
        else tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*MmEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static MmEncodeFn mm_encode_fn() {
    static MmEncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<MmEncodeFn>(f) : nullptr;
    }();
    return fn;
}

// Codes [rows][K], in boxes of 128 features x `box` rows.
static bool mm_map(CUtensorMap* m, const void* base, int rows, int K, int box) {
    const MmEncodeFn enc = mm_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K};
    cuuint32_t boxes[2] = {kE4Block, (cuuint32_t)box};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool PAIR>
static tsv_status launch_mm(const char* name, const E4Product& p, cudaStream_t stream) {
    using S = MmShape<BN, PAIR>;
    constexpr int CTAS = PAIR ? 2 : 1;
    MmParams q;
    q.p = p;
    q.blocks = e4_blocks(p.K);
    q.mtiles = (p.rows + kMmRows * CTAS - 1) / (kMmRows * CTAS);
    q.ntiles = (p.N + BN - 1) / BN;
    q.panel = std::min(q.mtiles, 8);
    // rows of a in shared memory: as many as there are, in whole swizzle atoms of 8.  The MMA reads 128 rows, so a stage's
    // weights, or the next stage's bytes, stand in for missing ones and end in accumulator rows that nothing reads.
    const int arows = std::min(kMmRows, (p.rows + 7) / 8 * 8), wrows = BN / CTAS;
    q.a_bytes = arows * kE4Block;
    q.stage_bytes = q.a_bytes + wrows * kE4Block;
    // the last stage's 128 rows have to end inside the ring as well
    const int slack = std::max(0, kMmRows * kE4Block - q.stage_bytes);
    q.stages = std::min((int)kMmMaxStages, (S::kSmem - 1024 - slack) / q.stage_bytes);
    if (!mm_map(&q.amap, p.a, p.rows, p.K, arows) || !mm_map(&q.wmap, p.w, p.N, p.K, wrows))
        return fail(TSV_ECUDA, "%s: tensor map encoding failed", name);
    const long long tiles = (long long)q.mtiles * q.ntiles;
    if (tiles > INT_MAX / 2) return fail(TSV_ECAPACITY, "%s: %lld tiles", name, tiles);
    const int places = sm_count() * S::kPerSm / CTAS;
    const int grid = (int)std::min<long long>(tiles, places) * CTAS;
    cudaFuncSetAttribute(matmul_e4m3_kernel<BN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    launch_pdl_cluster(matmul_e4m3_kernel<BN, PAIR>, grid, S::kThreads, S::kSmem, stream, CTAS, q);
    return check_launch(name);
}

tsv_status launch_matmul_e4m3(const char* name, const E4Product& p, cudaStream_t stream) {
    if (p.rows > kMmRows && (long long)p.N * p.rows >= 256ll * 256 * 76) return launch_mm<256, true>(name, p, stream);
    const long long mt = (p.rows + kMmRows - 1) / kMmRows;
    if (mt * p.N >= 256ll * sm_count() && p.rows > kMmRows) return launch_mm<256, false>(name, p, stream);
    if (mt * p.N >= 128ll * sm_count() && p.rows > 64) return launch_mm<128, false>(name, p, stream);
    if (mt * p.N >= 64ll * sm_count()) return launch_mm<64, false>(name, p, stream);
    return launch_mm<32, false>(name, p, stream);
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
