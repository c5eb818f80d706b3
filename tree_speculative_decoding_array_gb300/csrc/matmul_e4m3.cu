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
    int split;               // CTAs of a cluster that share a tile's blocks (1: none; more: one tile per cluster)
    bool vec;                // every 16-byte piece of an output row is aligned
};

template <int BN, bool PAIR>
struct MmShape {
    static constexpr int kEpiWarps = BN == 256 ? 16 : BN == 128 ? 8 : 4;
    static constexpr int kCols = BN / (kEpiWarps / 4);  // columns of an epilogue thread
    static constexpr int kPerSm = BN >= 128 ? 1 : 3;
    // A tile's columns are kParts MMAs of kPart columns, each with accumulators, barriers, an issuing warp and a warpgroup of its
    // own: the shorter an accumulator's way round (products, read out, free again), the less the two of TMEM are waited for.
    static constexpr int kParts = BN == 256 ? 2 : 1, kPart = BN / kParts;
    static constexpr int kBufs = BN == 128 ? 4 : 2;  // accumulators of a part in TMEM
    static constexpr int kBox = kPart / (PAIR ? 2 : 1);  // weights of a part in a CTA's shared memory
    // 256 columns: an epilogue thread holds 64 sums and 16 warps have to share the registers, so they take some over from the last
    // warpgroup (producer, two issuers, scales): 512 x 104 + 128 x 64 = 640 x 96.  A warp of its own reads the scales ahead
    // of the epilogue, which has neither the registers nor the time.  (Eight epilogue warps with 128 sums each: 346 us against
    // 337 for 4096 x 5120 x 20480.)
    static constexpr bool kWide = BN == 256;
    static constexpr int kIssuers = BN >= 128 ? 2 : 1, kTurns = kParts > 1 ? 1 : kIssuers;  // issuers that take turns with the blocks
    static constexpr int kThreads = (kEpiWarps + (kWide ? 4 : 1 + kIssuers)) * 32;
    static constexpr int kScaleBytes = kWide ? 2 * 4 * 2 * 128 * 4 : 0;   // two groups of 4 blocks, two weight blocks, 128 rows
    static constexpr int kPiece = kWide ? 64 : 128;                        // bytes of an output row that a warp gathers
    static constexpr int kOutBytes = BN >= 128 ? kEpiWarps * 32 * kPiece : 0;
    static constexpr bool kAhead = BN == 128;
    static constexpr int kSmem = (kPerSm == 1 ? 225 : 72) * 1024;
    static constexpr int kRing = kSmem - 1024 - kScaleBytes - kOutBytes;
};

// a += s x, b += s y, in one instruction.
__device__ __forceinline__ void add_scaled(float& a, float& b, uint32_t x, uint32_t y, float s) {
    asm("{\n .reg .b64 d, t, f;\n mov.b64 d, {%2, %3};\n mov.b64 t, {%0, %1};\n mov.b64 f, {%4, %4};\n"
        " fma.rn.f32x2 t, d, f, t;\n mov.b64 {%0, %1}, t;\n}"
        : "+f"(a), "+f"(b)
        : "r"(x), "r"(y), "f"(s));
}

// Bits of the largest of a thread's sums in the order of orderable(): a NaN without a sign above everything, one with a sign
// below everything, -0 below 0.  Bits of numbers without a sign are ordered as integers; where all have one, the other way round.
template <int COLS>
__device__ __forceinline__ uint32_t largest(const float (&acc)[COLS]) {
    int m = __float_as_int(acc[0]);
#pragma unroll
    for (int c = 1; c < COLS; ++c) m = max(m, __float_as_int(acc[c]));
    if (__any_sync(0xFFFFFFFFu, m < 0)) {
        uint32_t u = __float_as_uint(acc[0]);
#pragma unroll
        for (int c = 1; c < COLS; ++c) u = min(u, __float_as_uint(acc[c]));
        m = m < 0 ? (int)u : m;
    }
    return (uint32_t)m;
}

// A thread's COLS sums to `n` places of its output row.
template <typename T, int COLS>
__device__ __forceinline__ void store_row(T* o, const float (&acc)[COLS], int n, bool vec) {
#pragma unroll
    for (int c = 0; c < COLS; c += 8) {
        if (vec && c + 8 <= n) store8<T, true>(o + c, 8, acc + c);
        else store8<T, false>(o + c, n - c, acc + c);
    }
}

// A warp's 32 rows of COLS sums through its shared memory, BYTES of every row at a time, so that a store covers whole 64- or 128-byte
// pieces of rows (a thread's own row, written by itself, costs a 32-byte sector for every 16 bytes: 10,000 SM clocks for a tile of
// 128 x 256 bf16, half of what its products take).  `rows`, `n`: what is left of the matrix from o on.
template <typename T, int COLS, int BYTES>
__device__ __forceinline__ void store_rows(T* o, const float (&acc)[COLS], size_t ld, int rows, int n, bool vec, uint8_t* buf, int lane) {
    constexpr int P = BYTES / sizeof(T), V = 16 / sizeof(T), J = BYTES / 16;  // elements of a piece, of a 16-byte vector, vectors of a piece
    // vector j of row r: no two of 8 lanes in one bank, as they write (a row each) and as they read (J to a row)
    const auto place = [&](int r, int j) { return buf + r * BYTES + ((j ^ (r * J / 8 & (J - 1))) << 4); };
#pragma unroll
    for (int c = 0; c < COLS; c += P) {
        if (c >= n) break;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            uint4 u;
            if constexpr (sizeof(T) == 4) {
                const float* x = acc + c + 4 * j;
                u = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            } else {
                const float* x = acc + c + 8 * j;
                u = make_uint4(RowType<T>::pack(x[0], x[1]), RowType<T>::pack(x[2], x[3]), RowType<T>::pack(x[4], x[5]),
                               RowType<T>::pack(x[6], x[7]));
            }
            *reinterpret_cast<uint4*>(place(lane, j)) = u;
        }
        __syncwarp();
        if (vec) {
#pragma unroll
            for (int i = 0; i < J; ++i) {
                const int r = (i * 32 + lane) / J, j = lane % J, at = c + j * V;
                const uint4 u = *reinterpret_cast<const uint4*>(place(r, j));
                if (r < rows && at < n) *reinterpret_cast<uint4*>(o + (size_t)r * ld + at) = u;  // n is a multiple of V
            }
        } else {  // rows at any address: neighbouring lanes write neighbouring elements
            for (int r = 0; r < min(rows, 32); ++r)
#pragma unroll
                for (int k = lane; k < P; k += 32)
                    if (c + k < n) o[(size_t)r * ld + c + k] = *reinterpret_cast<const T*>(place(r, k / V) + k % V * sizeof(T));
        }
        __syncwarp();
    }
}

// One element of the output.
__device__ __forceinline__ void put(const E4Product& p, size_t at, float x) {
    if (p.out_dtype == TSV_F32) ((float*)p.out)[at] = x;
    else if (p.out_dtype == TSV_BF16) ((__nv_bfloat16*)p.out)[at] = __float2bfloat16_rn(x);
    else ((__half*)p.out)[at] = __float2half_rn(x);
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(MmShape<BN, PAIR>::kThreads, MmShape<BN, PAIR>::kPerSm)
    matmul_e4m3_kernel(const __grid_constant__ MmParams q) {
    griddep_begin();
    using S = MmShape<BN, PAIR>;
    constexpr int CTAS = PAIR ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMmMaxStages], empty[kMmMaxStages], acc_full[S::kBufs * S::kParts], acc_empty[S::kBufs * S::kParts], sc_full[2], sc_empty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    uint8_t* outbuf = ring + S::kRing;
    float* scales = reinterpret_cast<float*>(outbuf + S::kOutBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? tc::cluster_rank() : 0;
    const int split = PAIR ? 1 : q.split, share = split > 1 ? (int)tc::cluster_rank() : 0;
    const int first = blockIdx.x / (CTAS * split), step = gridDim.x / (CTAS * split), tiles = q.mtiles * q.ntiles;
    const int KB = q.blocks, ST = q.stages;
    const int k0 = (int)((long long)KB * share / split), k1 = (int)((long long)KB * (share + 1) / split);  // this CTA's blocks
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], S::kParts);
        }
        for (int b = 0; b < S::kBufs * S::kParts; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            // of a single row tile, the warps that have rows
            tc::mbar_init(&acc_empty[b], CTAS * S::kEpiWarps / 4 / S::kParts * (!PAIR && q.mtiles == 1 ? min(4, (q.p.rows + 31) / 32) : 4));
        }
        for (int g = 0; g < 2; ++g) {
            tc::mbar_init(&sc_full[g], 1);
            tc::mbar_init(&sc_empty[g], S::kEpiWarps);
        }
        tc::mbar_init(&drain, S::kIssuers);
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

    if (warp >= S::kEpiWarps) {
        if constexpr (S::kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == S::kEpiWarps) {
            // -------------------------------------------------------- producer
            int st = 0, issued = 0;
            uint32_t fill = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                int m, n;
                place(t, m, n);
                const int arow = (m * CTAS + rank) * kMmRows, wrow = n * BN + rank * S::kBox;
                for (int kb = k0; kb < k1; ++kb) {
                    if (!tc::mbar_wait_warp(&empty[st], fill ^ 1u, abort_flag)) { ok = false; break; }
                    uint8_t* a = ring + (size_t)st * q.stage_bytes;
                    const uint32_t bar = PAIR ? tc::cluster_addr(&full[st], 0) : tc::smem_u32(&full[st]);
                    // a pair's bytes, of both CTAs, are expected by its first CTA
                    tc::mbar_expect_tx_one(&full[st], rank == 0 ? CTAS * q.stage_bytes : 0u);
                    tc::tma_load_2d_one<PAIR>(a, &q.amap, bar, kb * kE4Block, arow);
#pragma unroll
                    for (int h = 0; h < S::kParts; ++h)
                        tc::tma_load_2d_one<PAIR>(a + q.a_bytes + h * S::kBox * kE4Block, &q.wmap, bar, kb * kE4Block, wrow + h * S::kPart);
                    ++issued;
                    if (++st == ST) { st = 0; fill ^= 1u; }
                }
            }
            if (*abort_flag && rank == 0)  // let the copies in flight land (bounded) before the CTA goes away
                for (int i = max(0, issued - ST); i < issued; ++i) tc::mbar_drain(&full[i % ST], (i / ST) & 1);
        } else if (warp <= S::kEpiWarps + S::kIssuers && rank == 0) {
            // -------------------------------------------------------- MMA issuers (of a pair: its first CTA's)
            // An issuer's waits, MMAs and commits follow one another and take as long as the MMAs of 128 columns run, so there are
            // two: with two parts, one for each; else they take turns.
            const int i = warp - S::kEpiWarps - 1;
            constexpr int kTurns = S::kTurns;
            const int h = S::kParts > 1 ? i : 0;
            const uint32_t idesc = tc::idesc_e4m3(kMmRows * CTAS, S::kPart);
            const uint64_t d0 = tc::sdesc_sw128(tc::smem_u32(ring), 16, 1024);
            const uint32_t b_off = q.a_bytes + h * S::kBox * kE4Block, tm = tmem + h * S::kPart;
            uint64_t *part_full = acc_full + h * S::kBufs, *part_empty = acc_empty + h * S::kBufs;
            const long long todo = (long long)(first < tiles ? (tiles - 1 - first) / step + 1 : 0) * (k1 - k0);
            int st = kTurns > 1 ? i : 0, buf = kTurns > 1 ? i : 0;  // both counts are multiples of kTurns
            uint32_t ph = 0, use = 0;  // parities of the stage's fill and of the accumulator's use
            for (long long g = kTurns > 1 ? i : 0; g < todo; g += kTurns) {
                if (!tc::mbar_wait_warp(tc::smem_u32(&full[st]), ph, tc::smem_u32(&part_empty[buf]), use ^ 1u, abort_flag)) break;
                tc::tc_fence_after();
                const uint64_t da = tc::sdesc_add(d0, (uint32_t)st * q.stage_bytes), db = tc::sdesc_add(da, b_off);
                tc::mma_e4m3_block<PAIR>(tm + buf * BN, da, db, idesc, &empty[st], &part_full[buf]);
                st += kTurns;
                if (st >= ST) { st -= ST; ph ^= 1u; }
                buf += kTurns;
                if (buf >= S::kBufs) { buf -= S::kBufs; use ^= 1u; }
            }
            tc::mma_commit_elect<PAIR>(&drain);
            tc::mbar_drain(&drain, 0);
        } else if (S::kWide && warp == S::kEpiWarps + 3) {
            // -------------------------------------------------------- scales: a_scale w_scale of 128 rows, two weight blocks, 4 blocks
            const E4Product& p = q.p;
            const int wlast = e4_blocks(p.N) - 1;
            int g = 0, groups = 0;
            uint32_t use = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                int m, n;
                place(t, m, n);
                const int row0 = (m * CTAS + rank) * kMmRows + lane;
                const float* w0 = p.w_scale + (size_t)min(n * 2, wlast) * KB;
                const float* w1 = p.w_scale + (size_t)min(n * 2 + 1, wlast) * KB;
                for (int kb = 0; kb < KB; kb += 4) {
                    float a[4][4], w[2][4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float* as = p.a_scale + (size_t)min(row0 + r * 32, p.rows - 1) * KB + kb;
#pragma unroll
                        for (int k = 0; k < 4; ++k) a[r][k] = kb + k < KB ? __ldg(as + k) : 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        w[0][k] = kb + k < KB ? __ldg(w0 + kb + k) : 0.f;
                        w[1][k] = kb + k < KB ? __ldg(w1 + kb + k) : 0.f;
                    }
                    if (groups >= 2 && !tc::mbar_wait_warp(&sc_empty[g], use ^ 1u, abort_flag)) { ok = false; break; }
                    float* to = scales + g * 4 * 256 + lane;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            to[k * 256 + r * 32] = a[r][k] * w[0][k];
                            to[k * 256 + 128 + r * 32] = a[r][k] * w[1][k];
                        }
                    __syncwarp();
                    tc::mbar_arrive_one(&sc_full[g]);
                    ++groups;
                    if (++g == 2) { g = 0; use ^= 1u; }
                }
            }
        }
    } else {
        if constexpr (S::kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        // ------------------------------------------------------------ epilogue: scale and add up, then write out
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + half * S::kCols;
        const int which = half * S::kCols / S::kPart;  // the part that this warp's columns are of
        const uint32_t part = which * S::kBufs * 8;
        const uint32_t full0 = tc::smem_u32(acc_full) + part, empty0 = PAIR ? tc::cluster_addr(acc_empty, 0) + part : tc::smem_u32(acc_empty) + part;
        const uint32_t sc0 = tc::smem_u32(scales) + (half * S::kCols / kE4Block * 128 + quarter * 32 + lane) * 4;
        const E4Product& p = q.p;
        int buf = 0, g = 0;
        uint32_t use = 0, gph = 0;
        bool ok = true;
        // a warp without rows has no part in a single row tile's barriers
        for (int t = !PAIR && q.mtiles == 1 && quarter * 32 >= p.rows ? tiles : first; ok && t < tiles; t += step) {
            int m, n;
            place(t, m, n);
            const int row0 = (m * CTAS + rank) * kMmRows + quarter * 32, row = row0 + lane, col = n * BN + half * S::kCols;
            float acc[S::kCols];
#pragma unroll
            for (int c = 0; c < S::kCols; ++c) acc[c] = 0.f;
            const float* as = p.a_scale + (size_t)min(row, p.rows - 1) * KB;
            const float* ws = p.w_scale + (size_t)(min(col, p.N - 1) / kE4Block) * KB;
            float sa = 0.f, sw = 0.f;
            unsigned long long seen = 0ull;  // the row's best so far, or an older one
            if (p.best && row < p.rows) seen = *(volatile unsigned long long*)&p.best[row];
            if constexpr (!S::kWide) sa = __ldg(as + k0), sw = __ldg(ws + k0);
            // kAhead: 16 columns are on their way out of TMEM while the 16 before them are added up, from one block to the next
            uint32_t d[S::kAhead ? 2 : 1][16];
            if constexpr (S::kAhead) {
                ok = tc::mbar_wait_warp(full0 + buf * 8, use, abort_flag);
                tc::tc_fence_after();
                if (ok) tc::tmem_ld16(taddr + buf * BN, d[0]);
            }
            for (int kb = k0; ok && kb < k1; ++kb) {
                bool there = false;  // the next block's sums, looked at ahead of the wait
                float sc;
                if constexpr (S::kWide) {
                    if ((kb & 3) == 0) ok = tc::mbar_wait_warp(tc::smem_u32(&sc_full[g]), gph, abort_flag);
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sc) : "r"(sc0 + (g * 4 + (kb & 3)) * 1024));
                } else {
                    sc = sa * sw;
                    if (kb + 1 < k1) sa = __ldg(as + kb + 1), sw = __ldg(ws + kb + 1);
                }
                if constexpr (!S::kAhead) {
                    ok = tc::mbar_wait_warp(full0 + buf * 8, use, abort_flag);
                    tc::tc_fence_after();
                }
#pragma unroll
                for (int c = 0; c < S::kCols / 16; ++c) {
                    uint32_t(&now)[16] = d[S::kAhead ? c & 1 : 0];
                    if (S::kAhead && c == S::kCols / 16 - 1) there = __all_sync(0xFFFFFFFFu, tc::mbar_test(full0 + (buf + 1 == S::kBufs ? 0 : buf + 1) * 8, buf + 1 == S::kBufs ? use ^ 1u : use));
                    if constexpr (!S::kAhead) tc::tmem_ld16(taddr + buf * BN + c * 16, now);
                    tc::tmem_wait_ld16(now);
                    if (c + 1 == S::kCols / 16) {
                        tc::tc_fence_before();
                        tc::mbar_arrive_lane0<PAIR>(empty0 + buf * 8, lane);
                        if (++buf == S::kBufs) { buf = 0; use ^= 1u; }
                        if (S::kAhead && kb + 1 < k1) {
                            if (!there) ok = ok && tc::mbar_wait_warp(full0 + buf * 8, use, abort_flag);
                            tc::tc_fence_after();
                            tc::tmem_ld16(taddr + buf * BN, d[0]);
                        }
                    } else if constexpr (S::kAhead) {
                        tc::tmem_ld16(taddr + buf * BN + (c + 1) * 16, d[(c + 1) & 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 2) add_scaled(acc[c * 16 + i], acc[c * 16 + i + 1], now[i], now[i + 1], sc);
                }
                if (S::kWide && ((kb & 3) == 3 || kb + 1 == k1)) {
                    __syncwarp();
                    tc::mbar_arrive_one(&sc_empty[g]);
                    if (++g == 2) { g = 0; gph ^= 1u; }
                }
            }
            tc::tmem_wait_ld();
            if (!ok || row0 >= p.rows || col >= p.N) continue;
            if (!PAIR && split > 1) {
                // this CTA's sums to its own shared memory, where the stages were; 16-byte pieces swizzled against bank conflicts
                float* to = reinterpret_cast<float*>(ring) + (quarter * 32 + lane) * BN;
                const int c4 = half * S::kCols / 4;
                if (row < p.rows)
#pragma unroll
                    for (int c = 0; c < S::kCols / 4; ++c)
                        *reinterpret_cast<float4*>(to + (((c4 + c) ^ (lane & 7)) << 2)) = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
            } else if (p.best) {
                if (col + S::kCols > p.N)  // columns behind the last one: the bits that rank below every number's
#pragma unroll
                    for (int c = 0; c < S::kCols; ++c) acc[c] = col + c < p.N ? acc[c] : __uint_as_float(0xFFFFFFFFu);
                const uint32_t top = largest<S::kCols>(acc);
                // most tiles do not hold their rows' best: `seen`, read a tile's time ago, tells
                const bool wins = row < p.rows && orderable(__uint_as_float(top)) >= (uint32_t)(seen >> 32);
                if (__any_sync(0xFFFFFFFFu, wins)) {
                    int at = 0;
#pragma unroll
                    for (int c = S::kCols - 1; c >= 0; --c) at = __float_as_uint(acc[c]) == top ? c : at;
                    if (wins) atomicMax(&p.best[row], pack_best(__uint_as_float(top), (uint32_t)(col + at)));
                }
            } else if constexpr (S::kOutBytes > 0) {
                uint8_t* piece = outbuf + warp * 32 * S::kPiece;
                const size_t o = (size_t)row0 * p.N + col;
                const int rows = p.rows - row0, cols = p.N - col;
                if (p.out_dtype == TSV_F32) store_rows<float, S::kCols, S::kPiece>((float*)p.out + o, acc, p.N, rows, cols, q.vec, piece, lane);
                else if (p.out_dtype == TSV_BF16) store_rows<__nv_bfloat16, S::kCols, S::kPiece>((__nv_bfloat16*)p.out + o, acc, p.N, rows, cols, q.vec, piece, lane);
                else store_rows<__half, S::kCols, S::kPiece>((__half*)p.out + o, acc, p.N, rows, cols, q.vec, piece, lane);
            } else if (row < p.rows) {
                const size_t o = (size_t)row * p.N + col;
                if (p.out_dtype == TSV_F32) store_row<float, S::kCols>((float*)p.out + o, acc, p.N - col, q.vec);
                else if (p.out_dtype == TSV_BF16) store_row<__nv_bfloat16, S::kCols>((__nv_bfloat16*)p.out + o, acc, p.N - col, q.vec);
                else store_row<__half, S::kCols>((__half*)p.out + o, acc, p.N - col, q.vec);
            }
        }
    }
    __syncthreads();
    // A wait of this CTA ran out (its copies and MMAs have ended, or had their time to): NaN is what its tiles hold, or what it adds to
    // the cluster's sums, so that no reader takes what is missing for a product.  By the epilogue's warps, which have registers for it.
    if (*abort_flag && warp < S::kEpiWarps) {
        constexpr int kThreads = S::kEpiWarps * 32;
        const float nan = __int_as_float(0x7FFFFFFF);
        if (!PAIR && split > 1)
            for (int e = threadIdx.x; e < kMmRows * BN; e += kThreads) reinterpret_cast<float*>(ring)[e] = nan;
        else
            for (int t = first; t < tiles; t += step) {
                int m, n;
                place(t, m, n);
                const int row0 = (m * CTAS + rank) * kMmRows, rows = min(kMmRows, q.p.rows - row0), cols = min(BN, q.p.N - n * BN);
                for (int r = 0; r < rows; ++r) {
                    if (q.p.best && threadIdx.x == 0) atomicMax(&q.p.best[row0 + r], pack_best(nan, (uint32_t)(n * BN)));
                    if (!q.p.best)
                        for (int c = threadIdx.x; c < cols; c += kThreads) put(q.p, (size_t)(row0 + r) * q.p.N + n * BN + c, nan);
                }
            }
    }
    if (!PAIR && split > 1) {
        // every CTA of the cluster adds up, share by share, its part of the tile's columns, and writes them
        tc::cluster_sync();
        int m, n;
        place(first, m, n);
        const int row0 = m * kMmRows, rows = min(kMmRows, q.p.rows - row0), per = BN / 4 / split;
        for (int e = threadIdx.x; e < rows * per; e += blockDim.x) {
            const int r = e / per, c = share * per + e - r * per, col = n * BN + c * 4;
            const float* from = reinterpret_cast<const float*>(ring) + r * BN + ((c ^ (r & 7)) << 2);
            float4 part[8], v = make_float4(0.f, 0.f, 0.f, 0.f);  // asked for together, added up in order
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s < split) part[s] = tc::ld_cluster_f4(tc::cluster_addr(from, s));
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s < split) v = make_float4(v.x + part[s].x, v.y + part[s].y, v.z + part[s].z, v.w + part[s].w);
            const size_t o = (size_t)(row0 + r) * q.p.N + col;
            const float x[4] = {v.x, v.y, v.z, v.w};
            if (q.p.best) {
                unsigned long long key = 0ull;
                for (int j = 0; j < 4 && col + j < q.p.N; ++j) key = max(key, pack_best(x[j], (uint32_t)(col + j)));
                if (key) atomicMax(&q.p.best[row0 + r], key);
                continue;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (col + j >= q.p.N) break;
                put(q.p, o + j, x[j]);
            }
        }
        tc::cluster_sync();  // no CTA goes while another reads its sums
    }
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
static tsv_status launch_mm(const char* name, const E4Product& p, int split, cudaStream_t stream) {
    using S = MmShape<BN, PAIR>;
    constexpr int CTAS = PAIR ? 2 : 1;
    MmParams q;
    q.p = p;
    q.blocks = e4_blocks(p.K);
    q.mtiles = (p.rows + kMmRows * CTAS - 1) / (kMmRows * CTAS);
    q.ntiles = (p.N + BN - 1) / BN;
    q.panel = std::min(q.mtiles, 8);
    q.split = split;
    // rows of a in shared memory: as many as there are, in whole swizzle atoms of 8.  The MMA reads 128 rows, so a stage's
    // weights, or the next stage's bytes, stand in for missing ones and end in accumulator rows that nothing reads.
    const int arows = std::min(kMmRows, (p.rows + 7) / 8 * 8);
    q.a_bytes = arows * kE4Block;
    q.stage_bytes = q.a_bytes + S::kParts * S::kBox * kE4Block;
    // the last stage's 128 rows have to end inside the ring as well
    const int slack = std::max(0, kMmRows * kE4Block - q.stage_bytes);
    q.stages = std::min((int)kMmMaxStages, (S::kRing - slack) / q.stage_bytes);
    // Issuers that take turns need every stage to be one issuer's: a parity does not tell a filling from the last but one, so whoever
    // waits for a filling has to have seen the one before.  (That a freed accumulator implies the one before does not help: a
    // suspended test of one barrier ends after the test of another that was issued behind it.)
    q.stages -= q.stages % S::kTurns;
    if (!mm_map(&q.amap, p.a, p.rows, p.K, arows) || !mm_map(&q.wmap, p.w, p.N, p.K, S::kBox))
        return fail(TSV_ECUDA, "%s: tensor map encoding failed", name);
    q.vec = ((uintptr_t)p.out & 15) == 0 && p.N % (p.out_dtype == TSV_F32 ? 4 : 8) == 0;
    const long long tiles = (long long)q.mtiles * q.ntiles;
    if (tiles > INT_MAX / 2) return fail(TSV_ECAPACITY, "%s: %lld tiles", name, tiles);
    const int places = sm_count() * S::kPerSm / CTAS;
    const int grid = split > 1 ? (int)tiles * split : (int)std::min<long long>(tiles, places) * CTAS;
    cudaFuncSetAttribute(matmul_e4m3_kernel<BN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    launch_pdl_cluster(matmul_e4m3_kernel<BN, PAIR>, grid, S::kThreads, S::kSmem, stream, CTAS * split, q);
    return check_launch(name);
}

// The kernel for a product, by an estimate of each one's microseconds.  A block of 128 features takes a CTA 0.28 us (a pair: 0.5)
// wherever its operands come from, since that is what its hand-offs and 66 bytes per SM clock from L2 cost; rounds of CTAs
// follow one another; HBM delivers 6.5 bytes per nanosecond at most; a launch costs 3.5 us, sharing a tile's features between the CTAs of a
// cluster 2.5 and 0.035 per row (their sums go through shared memory).  Measured (us: estimate's choice, others), K = 5120:
//   1 x 1024: 64 columns shared by 8 6.5, by 4 7.0, 128 shared by 4 7.4   1 x 20480: 64 columns 21.3, 128 27.8
//   1 x 6144: 64 shared by 4 11.6, 128 by 2 11.2, 64 alone 13.9           1 x 248320: 128 columns 183 (the HBM rate), 64 195
//   128 x 6144: 128 columns 14.3, 64 shared by 4 16.2                     128 x 248320: 128 columns 207, 64 273
//   512 x 5120: pairs 23.1, 128 columns 24.0                              2048 x 5120: 128 columns 54.0, pairs 60.7
//   1024 x 5120: 128 columns 34.0, pairs 41.6                             4096 x 20480: pairs 329, 128 columns 364
tsv_status launch_matmul_e4m3(const char* name, const E4Product& p, cudaStream_t stream) {
    const int sms = sm_count(), blocks = e4_blocks(p.K);
    const long long mt = (p.rows + kMmRows - 1) / kMmRows, n64 = mt * ((p.N + 63) / 64), n128 = mt * ((p.N + 127) / 128);
    const long long pairs = (mt + 1) / 2 * ((p.N + 255) / 256);
    const float stream_us = ((float)p.N + p.rows) * p.K / 6.5e6f;
    const auto rounds = [](long long tiles, int places) { return (float)((tiles + places - 1) / places); };
    float best = 1e30f;
    int columns = 0, split = 1;
    const auto offer = [&](float us, int c, int s) {
        if (us < best) best = us, columns = c, split = s;
    };
    if (mt > 1) offer(std::max(rounds(pairs, sms / 2) * blocks * 0.5f, stream_us), 256, 1);
    for (int s = 1; s <= 8 && s <= std::max(1, blocks / 2); s *= 2) {
        const float share = (float)((blocks + s - 1) / s), joined = s > 1 ? 2.5f + 0.035f * std::min(p.rows, kMmRows) : 0.f;
        if (s == 1 || n128 * s <= sms) offer(std::max(rounds(n128 * s, sms) * share * 0.28f, stream_us) + joined, 128, s);
        if (s == 1 || n64 * s <= sms * 3) {
            const float beside = std::min(3.f, std::max(1.f, (float)(n64 * s) / sms));  // CTAs on an SM
            const float block = std::max(0.28f, beside * (std::min(p.rows, kMmRows) * 128 + 8192) / 85e3f);
            offer(std::max(rounds(n64 * s, sms * 3) * share * block, stream_us) + joined, 64, s);
        }
    }
    if (columns == 256) return launch_mm<256, true>(name, p, 1, stream);
    if (columns == 128) return launch_mm<128, false>(name, p, split, stream);
    return launch_mm<64, false>(name, p, split, stream);
}

// What both entry points ask of their operands.
static tsv_status check_product(const char* name, const E4Product& p) {
    if (p.rows < 0 || p.K < 1 || p.N < 1) return fail(TSV_EINVAL, "%s: rows=%d K=%d N=%d", name, p.rows, p.K, p.N);
    if (p.K % 16) return fail(TSV_EINVAL, "%s: K=%d not a multiple of 16", name, p.K);
    if (p.rows > 1 << 30 || p.N > 1 << 30) return fail(TSV_ECAPACITY, "%s: rows=%d N=%d above 2^30", name, p.rows, p.N);
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
