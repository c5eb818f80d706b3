// tsv_gdn_tree_verify: every node of a draft tree through the recurrent layers, from one read of the state.
//
// mlxcel issue #1204 and Splash issue #728 ("What it does"): recurrent layers cannot take a mask and a flattened tree
// would leak state between siblings, so each node runs from its own parent's state.  The recurrence along a node's
// ancestors unrolls into one triangular system over the tree (gdn_tc.cuh), in which the state appears only in the
// products S k_i and S q_i: no node's state is ever formed.
//
// One CTA per (layer, sequence, some value heads of one key head): K and Q are staged and [K; Q] K^T taken once, then
// the value heads follow one another.  Each warp owns 16 value features and takes their rows of S from global memory
// to fp16 pairs in TMEM, fetches their columns of V and writes their columns of o; the next head's state and V are
// fetched while this head is computed, and a head's matrices are built while the tensor cores work on its S [K; Q]^T.
// The warps of a head only meet to hand over S and the matrices.  48 layers x 48 heads of 128 x 128: trees of 3 nodes 35 us,
// of 16 nodes 37 us (4.7 TB/s), 32 trees of 64 nodes 1.99 ms (4.1 TB/s): two CTAs fit an SM, so what bounds it is the chain
// of a head's steps, and at 64 nodes its 15,000 warp instructions (45 % of the issue slots).
//
// K, Q and S are kept with the columns of every 16 in the order 0 1 4 5 8 9 12 13 2 3 6 7 10 11 14 15, in which a thread's four
// values of a fragment are neighbours in memory.
#include <math.h>

#include "gdn_tc.cuh"

namespace tsv {

constexpr int kMaxHeads = 4;  // value heads of one CTA

template <int DK, int DV, int NB>
struct TreeSmem {
    static constexpr int T = 16 * NB;
    static constexpr int kq = 0;                       // K rows [T], Q rows [T], DK fp16 each
    static constexpr int v = kq + 2 * T * DK * 2;      // two buffers of V rows [T], DV bf16 each; o over them
    static constexpr int a16 = v + 2 * T * DV * 2;     // [T][64] fp16: -A below the diagonal blocks, inverses on them
    static constexpr int p16 = a16 + T * 128;          // [T][64] fp16: P
    static constexpr int diag = p16 + T * 128;         // [NB][16][kDiag] fp32: A of the diagonal blocks
    static constexpr int keys = diag + NB * 16 * kDiag * 4;
    static constexpr int rows = keys + (int)sizeof(GdnKeys);  // per value head
    static constexpr int bars = rows + kMaxHeads * (int)sizeof(GdnRows);  // two barriers, TMEM address, abort flag
    // [K; Q] K^T takes 128 rows of the K and Q tile, whatever lies behind them
    static constexpr int reach = (DK / 64 - 1) * 2 * T * 128 + 128 * 128;
    static constexpr int total = bars + 32 > reach ? bars + 32 : reach;
    // TMEM columns: S as fp16 pairs, S [K; Q]^T, [K; Q] K^T
    static constexpr int col_s = 0, col_d = DK / 2, col_g = col_d + 2 * T, cols_used = col_g + T;
    static constexpr int cols = cols_used <= 64 ? 64 : cols_used <= 128 ? 128 : 256;
    // the fp32 path: u [T][DV] over v, one node's k and q over a16, its ancestors' products over p16
    static_assert(T * DV * 4 <= a16 - v && 2 * DK * 4 <= T * 128 && 2 * 64 * 4 <= T * 128, "fp32 path does not fit");
};

// The whole tree of one head in fp32, node by node: taken when an operand left fp16's range (an infinity or a NaN in
// the inputs, keys that are not of unit length with large writes, values far above those that another node sees).  Only a
// node's ancestors are ever read, so what is not finite stays with its node and the node's descendants.  Thread = value
// feature.
template <int DK, int DV, int NB>
__device__ __noinline__ void tree_fp32(const tsv_gdn_desc& d, const uint64_t* anc, int layer, int b, int h, char* sm, const GdnRows& rw) {
    using M = TreeSmem<DK, DV, NB>;
    float* u = reinterpret_cast<float*>(sm + M::v);
    float* kk = reinterpret_cast<float*>(sm + M::a16);   // k_i, then q_i
    float* wk = reinterpret_cast<float*>(sm + M::p16);   // e^{G_i - G_j} (k_i . k_j), then (q_i . k_j)
    const GdnKeys& ky = *reinterpret_cast<const GdnKeys*>(sm + M::keys);
    const int T = d.T, hk = h / (d.HV / d.HK), warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x;
    const uint16_t* K = reinterpret_cast<const uint16_t*>(d.k[layer]);
    const uint16_t* Q = reinterpret_cast<const uint16_t*>(d.q[layer]);
    for (int i = 0; i < T; ++i) {
        const size_t row = (size_t)b * T + i;
        float ki[DK / 32], qi[DK / 32];
        unit_row<DK>(K + (row * d.HK + hk) * DK, d.norm_eps, 1.f, lane, ki);
        unit_row<DK>(Q + (row * d.HK + hk) * DK, d.norm_eps, d.scale, lane, qi);
        __syncthreads();  // the node before is done with kk and wk
        if (warp == 0)
#pragma unroll
            for (int e = 0; e < DK / 32; ++e) {
                kk[lane + 32 * e] = ki[e];
                kk[DK + lane + 32 * e] = qi[e];
            }
        int at = 0;
        for (uint64_t a = ky.before[i] | (1ull << i); a; a &= a - 1, ++at) {
            if (at % (DV / 16) != warp) continue;
            const int j = __ffsll((long long)a) - 1;
            float kj[DK / 32], x = 0.f, y = 0.f;
            unit_row<DK>(K + (((size_t)b * T + j) * d.HK + hk) * DK, d.norm_eps, 1.f, lane, kj);
#pragma unroll
            for (int e = 0; e < DK / 32; ++e) {
                x = fmaf(ki[e], kj[e], x);
                y = fmaf(qi[e], kj[e], y);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
            }
            const float w = exp2f((rw.g_hi[i] - rw.g_hi[j]) + (rw.g_lo[i] - rw.g_lo[j]));
            if (lane == 0) {
                wk[j] = w * x;
                wk[64 + j] = w * y;
            }
        }
        __syncthreads();
        if (r < DV) {
            const float* S = d.state[layer] + (((size_t)b * d.HV + h) * DV + r) * DK;
            float sk = 0.f, sq = 0.f;
            for (int e = 0; e < DK; ++e) {
                sk = fmaf(S[e], kk[e], sk);
                sq = fmaf(S[e], kk[DK + e], sq);
            }
            const float w = exp2f(rw.g_hi[i] + rw.g_lo[i]);
            const size_t ov = (row * d.HV + h) * DV + r;
            float x = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(d.v[layer])[ov]) - w * sk, y = w * sq;
            for (uint64_t a = ky.before[i]; a; a &= a - 1) {
                const int j = __ffsll((long long)a) - 1;
                x = fmaf(-wk[j], u[j * DV + r], x);
                y = fmaf(wk[64 + j], u[j * DV + r], y);
            }
            x *= rw.beta[i];
            u[i * DV + r] = x;
            reinterpret_cast<__nv_bfloat16*>(d.o[layer])[ov] = __float2bfloat16(fmaf(wk[64 + i], x, y));
        }
    }
}

// Row of the K and Q tile that holds row r of [K; Q].
template <int NB>
__device__ __forceinline__ int row_pos(int r) {
    const int q = r >= 16 * NB ? 16 * NB : 0, i = r - q;
    return q + 16 * block_pos<NB>(i >> 4) + (i & 15);
}

template <int DK, int DV, int NB>
__global__ void __launch_bounds__(2 * DV, 2) gdn_tree_kernel(const __grid_constant__ tsv_gdn_desc d,
                                                             const uint64_t* __restrict__ anc, int heads, int big, int32_t* status) {
    griddep_begin();
    using M = TreeSmem<DK, DV, NB>;
    constexpr int kThreads = 2 * DV, kWarps = DV / 16;
    constexpr int KS = DK / 16;
    constexpr int T16 = M::T;
    extern __shared__ __align__(1024) char sm[];
    GdnKeys& ky = *reinterpret_cast<GdnKeys*>(sm + M::keys);
    GdnRows* rows = reinterpret_cast<GdnRows*>(sm + M::rows);
    const uint32_t s0 = tc::smem_u32(sm);
    const int T = d.T;
    int item = blockIdx.x;
    if (item < big) {  // CTAs of `heads` heads, then of one
        item *= heads;
    } else {
        item = big * heads + (item - big);
        heads = 1;
    }
    const int h0 = item % d.HV;
    item /= d.HV;
    const int b = item % d.B, layer = item / d.B;
    const int hk = h0 / (d.HV / d.HK);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const size_t row0 = (size_t)b * T;
    // this warp's TMEM lanes and value features (16 of each); 64 features leave the upper half of each quarter unused
    const int lane0 = (warp & 3) * 32 + (warp >> 2) * 16, fb = DV == 128 ? lane0 : warp * 16;

    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + M::bars);  // [K; Q] K^T done, S [K; Q]^T done
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 3);
    int* redo_s = reinterpret_cast<int*>(bars + 3) + 1;
    if (threadIdx.x == 0) {
        tc::mbar_init(&bars[0], 1);
        tc::mbar_init(&bars[1], 1);
        *abort_flag = 0;
        *redo_s = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, M::cols);
        tc::tmem_relinquish();
    }

    // K, Q and the first V rows; rows beyond T are zero
    constexpr int LPR = DK / 8;                      // lanes that share a K or Q row
    constexpr int KQ = 2 * T16 * LPR / kThreads;     // its chunks per thread
    static_assert(KQ * kThreads == 2 * T16 * LPR, "uneven staging");
    const int chunk = threadIdx.x % LPR;
#pragma unroll
    for (int x = 0; x < KQ; ++x) {
        const int r = threadIdx.x / LPR + x * (kThreads / LPR), i = r >= T16 ? r - T16 : r;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(r >= T16 ? d.q[layer] : d.k[layer]);
        cp16(kq_at<2 * T16>(s0 + M::kq, row_pos<NB>(r), chunk), src + ((row0 + (i < T ? i : 0)) * d.HK + hk) * DK + chunk * 8, i < T);
    }
    cp_commit();
    // this warp's columns of V, and of o over them: 32 bytes of every row, a 16-byte chunk per lane and NB
    const int vc = fb / 8 + (lane & 1), vr = lane >> 1;
    const size_t vo0 = (row0 * d.HV + h0) * DV + vc * 8;  // + (row * HV + head) * DV
    auto fetch_v = [&](int k) {
#pragma unroll
        for (int x = 0; x < NB; ++x) {
            const int i = vr + 16 * x;
            cp16(tile_at<DV * 2>(s0 + M::v + (k & 1) * T16 * DV * 2, i, vc),
                 reinterpret_cast<const uint16_t*>(d.v[layer]) + vo0 + ((size_t)(i < T ? i : 0) * d.HV + k) * DV, i < T);
        }
        cp_commit();
    };
    fetch_v(0);
    // the state's loads: features (rows) fb + g and fb + g + 8, columns 16 j + 4 t .. + 3
    const float* S = d.state[layer] + (((size_t)b * d.HV + h0) * DV + fb + g) * DK + 4 * t;
    float4 raw[2][KS];
    auto fetch_s = [&](int k) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int j = 0; j < KS; ++j)
                raw[half][j] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)k * DV * DK + half * 8 * DK + 16 * j));
    };
    // G of every head, a warp each, two nodes per lane: pointer doubling over the parents (the highest strict ancestor)
    static_assert(kMaxHeads <= kWarps, "a warp per head");
    if (const int k = warp; k < heads) {
        Pair G[2];
        int p[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = lane + 32 * x;
            uint64_t before = 0;
            float gi = 0.f, bi = 0.f;
            if (i < T) {
                before = anc[row0 + i] & ((1ull << i) - 1ull);
                gi = d.g[layer][(row0 + i) * d.HV + h0 + k];
                bi = d.beta[layer][(row0 + i) * d.HV + h0 + k];
            }
            if (k == 0) ky.before[i] = before;
            rows[k].beta[i] = bi;
            G[x] = log2_decay(gi);
            p[x] = before ? 63 - __clzll((long long)before) : -1;
        }
        while (__any_sync(0xFFFFFFFFu, p[0] >= 0 || p[1] >= 0)) {  // each round halves every remaining chain
            Pair more[2];
            int np[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int src = p[x] & 31;
                Pair q[2];
                int pp[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    q[y].hi = __shfl_sync(0xFFFFFFFFu, G[y].hi, src);
                    q[y].lo = __shfl_sync(0xFFFFFFFFu, G[y].lo, src);
                    pp[y] = __shfl_sync(0xFFFFFFFFu, p[y], src);
                }
                more[x] = p[x] >= 32 ? q[1] : q[0];
                np[x] = p[x] >= 32 ? pp[1] : pp[0];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (p[x] >= 0) {
                    G[x] = add(G[x], more[x]);
                    p[x] = np[x];
                }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            rows[k].g_hi[lane + 32 * x] = G[x].hi;
            rows[k].g_lo[lane + 32 * x] = G[x].lo;
        }
        __syncwarp();
    }
    // The next head's state is fetched ahead: to registers where they are free, else (four blocks) to L2, 128 bytes per
    // prefetch.  48 layers, registers against L2: 3 nodes 35.3 and 38.9 us, 16 nodes 38.9 and 41.5, 4 trees of 20 nodes 166 and
    // 171, of 40 nodes 215 and 213; 8 trees of 64 nodes 514 and 509.
    constexpr bool kAhead = NB < 4;
    auto ahead_s = [&](int k) {
        const char* p = reinterpret_cast<const char*>(d.state[layer] + ((size_t)b * d.HV + h0 + k) * DV * DK);
#pragma unroll
        for (int x = 0; x < DV * DK * 4 / 128 / kThreads; ++x)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (threadIdx.x + x * kThreads) * 128));
    };
    if (kAhead) fetch_s(0);
    else ahead_s(0);
    if (warp < heads) {  // the largest and smallest G and the smallest write, while K and Q arrive
        GdnRows& rw = rows[warp];
        const float g0 = lane < T ? rw.g_hi[lane] : rw.g_hi[0], g1 = lane + 32 < T ? rw.g_hi[lane + 32] : g0;
        const float e = fade_exponent((float)__reduce_max_sync(0xFFFFFFFFu, __float2int_rd(fmaxf(g0, g1))));
        const int least = __reduce_min_sync(0xFFFFFFFFu, __float2int_rd(fminf(g0, g1)));
        const float write = least_write(rw, T, lane);
        if (lane == 0) {
            rw.e = e;
            rw.fade = pow2_of(e);
            rw.seen = tc::ex2_approx((float)least - e);
            rw.write = write;
        }
    }
    uint32_t flag_kq = 0;
    cp_wait<1>();  // this thread's own chunks of K and Q: converted in place
    constexpr int KH = KQ >= 4 ? KQ / 4 : 1;
#pragma unroll
    for (int x0 = 0; x0 < KQ; x0 += KH) {
        uint4 w[KH];
        float f[KH];
#pragma unroll
        for (int x = 0; x < KH; ++x)
            w[x] = *reinterpret_cast<const uint4*>(sm + kq_at<2 * T16>(M::kq, row_pos<NB>(threadIdx.x / LPR + (x0 + x) * (kThreads / LPR)), chunk));
        stage_chunks<DK, KH>(w, f, d.norm_eps, flag_kq);
#pragma unroll
        for (int x = 0; x < KH; ++x) {
            const int r = threadIdx.x / LPR + (x0 + x) * (kThreads / LPR);
            // columns 0 1 4 5 (or 8 9 12 13) of the 16 to their first chunk, 2 3 6 7 (10 11 14 15) to the second
            const int p = row_pos<NB>(r), at = 8 * (chunk & 1);
            *reinterpret_cast<uint2*>(sm + kq_at<2 * T16>(M::kq, p, chunk & ~1) + at) = make_uint2(w[x].x, w[x].z);
            *reinterpret_cast<uint2*>(sm + kq_at<2 * T16>(M::kq, p, chunk | 1) + at) = make_uint2(w[x].y, w[x].w);
            if (chunk == 0) (r >= T16 ? ky.fq : ky.fk)[r >= T16 ? r - T16 : r] = r >= T16 ? f[x] * kOutLift : f[x];
        }
    }
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();

    const uint64_t kq_desc = tc::sdesc_sw128(s0 + M::kq, 16, 1024);
    const int vrow = ((lane >> 4) << 3) + (lane & 7), vchunk = fb / 8 + ((lane >> 3) & 1);
    float* diag = reinterpret_cast<float*>(sm + M::diag);
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (threadIdx.x == 0) {  // [K; Q] K^T
        const uint32_t id = tc::idesc_f16(false, false, false, 128, T16);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const uint64_t at = tc::sdesc_add(kq_desc, (ks >> 2) * 2 * T16 * 128 + (ks & 3) * 32);
            tc::mma_f16(tmem + M::col_g, at, at, id, ks > 0);
        }
        tc::mma_commit(&bars[0]);
    }
    if (threadIdx.x < 2 * T16) {
        const int r = threadIdx.x, i = r >= T16 ? r - T16 : r;
        const float x = (r >= T16 ? ky.fq : ky.fk)[i];
        for (int y = 0; y < heads; ++y)
            (r >= T16 ? rows[y].cq : rows[y].ck)[i] = tc::ex2_approx((rows[y].g_hi[i] - rows[y].e) + rows[y].g_lo[i]) * x;
    }
    uint32_t redo = 0;  // heads in which this thread saw an operand that is not finite
    bool ok = true;
    for (int k = 0; k < heads; ++k) {
        const GdnRows& rw = rows[k];
        const int vt = M::v + (k & 1) * T16 * DV * 2;
        uint32_t flag = flag_kq;
        if (!kAhead) {
            fetch_s(k);
            if (k + 1 < heads) ahead_s(k + 1);
        }
        cp_wait<0>();
        __syncwarp();  // this warp's V is here
        if (k + 1 < heads) fetch_v(k + 1);
        // this warp's features: a power-of-two scale each, from the largest of the state's row and of v
        float down[2], up[2], sd = INFINITY;  // up: with o's scale
        {
            uint32_t top[2] = {0, 0};
#pragma unroll
            for (int bb = 0; bb < NB; ++bb) {
                uint32_t w[4];
                ldsm4_t(w, tile_at<DV * 2>(s0 + vt, bb * 16 + vrow, vchunk));
#pragma unroll
                for (int x = 0; x < 4; ++x) top[x & 1] = abs_max2(top[x & 1], w[x]);
            }
            uint32_t Sf[4 * KS];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float sx = 0.f, mx = fmaxf(bf16_lo(top[half]), bf16_hi(top[half]));
#pragma unroll
                for (int j = 0; j < KS; ++j)
                    sx = fmaxf(fmaxf(sx, fmaxf(fabsf(raw[half][j].x), fabsf(raw[half][j].y))), fmaxf(fabsf(raw[half][j].z), fabsf(raw[half][j].w)));
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    sx = fmaxf(sx, __shfl_xor_sync(0xFFFFFFFFu, sx, x));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
                }
                sx *= rw.fade;
                mx = fmaxf(8.f * sx, mx);
                pow2_scale(mx * (1.f / kLift), down[half], up[half]);
                // the smaller of the two features' largest state, faded and scaled, where a feature is not empty
                sd = fminf(sd, mx == 0.f ? INFINITY : sx * down[half]);
                up[half] *= d.scale / kOutLift;
                const float2 d2 = make_float2(rw.fade * down[half], rw.fade * down[half]);
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const float2 x = mul2(make_float2(raw[half][j].x, raw[half][j].y), d2), y = mul2(make_float2(raw[half][j].z, raw[half][j].w), d2);
                    Sf[4 * j + half] = f16x2(x.x, x.y);
                    Sf[4 * j + 2 + half] = f16x2(y.x, y.y);
                }
            }
#pragma unroll
            for (int x = 0; x < KS / 4; ++x)
                tc::tmem_st_frag8(tmem + ((uint32_t)lane0 << 16) + M::col_s + x * 32, Sf + 16 * x);
            tc::tmem_wait_st();
        }
        if (kAhead && k + 1 < heads) fetch_s(k + 1);
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
        if (threadIdx.x == 0) {  // S [K; Q]^T
            const uint32_t id = tc::idesc_f16(false, false, false, 128, 2 * T16);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                tc::mma_f16_ts(tmem + M::col_d, tmem + M::col_s + ks * 8,
                               tc::sdesc_add(kq_desc, (ks >> 2) * 2 * T16 * 128 + (ks & 3) * 32), id, ks > 0);
            tc::mma_commit(&bars[1]);
        }
        __syncwarp();
        if (__any_sync(0xFFFFFFFFu, sd * rw.seen < kFaint))
            if (faint_rows<DV * 2, NB>(sm + vt, fb, down[0], down[1], sd, sd, rw, ky, T)) flag = 0x7FFF7FFFu;
        __syncwarp();
        // the system's matrices
        ok = warp_wait(&bars[0], 0, abort_flag);
        tc::tc_fence_after();
        if (ok) {
            for (int hf = warp >> 2; hf < 2; hf += kWarps / 4)
                warp_matrices<NB, 1>(warp & 3, hf, tmem + M::col_g, sm + M::a16, sm + M::p16, diag, ky, rw, flag, lane);
            ok = warp_wait(&bars[1], k & 1, abort_flag);
        }
        ok = __syncthreads_and(ok);
        tc::tc_fence_after();
        if (!ok) break;

        uint32_t Uf[NB][1][4];
#pragma unroll
        for (int bb = 0; bb < NB; ++bb) {
            float dk[8], dq[8], ak[2][4], aq[2][4], u[2][4];  // this block's columns of S K^T and S Q^T
            tc::tmem_ld_frag2(tmem + ((uint32_t)lane0 << 16) + M::col_d + 16 * block_pos<NB>(bb), dk);
            tc::tmem_ld_frag2(tmem + ((uint32_t)lane0 << 16) + M::col_d + T16 + 16 * block_pos<NB>(bb), dq);
            uint32_t w[4];
            ldsm4_t(w, tile_at<DV * 2>(s0 + vt, bb * 16 + vrow, vchunk));
            tc::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                ak[x >> 2][x & 3] = dk[x];
                aq[x >> 2][x & 3] = dq[x];
            }
            block_rhs<1>(bb, ak, w, down, rw, t);
#pragma unroll
            for (int c = 0; c < bb; ++c) block_update<NB, 1>(bb, c, ak, Uf[c], s0 + M::a16, lane);
            block_solve<NB, 1>(bb, ak, Uf[bb], u, s0 + M::a16, flag, lane);
            block_rhs_q(bb, aq, rw, t);
#pragma unroll
            for (int c = 0; c <= bb; ++c) block_out(bb, c, aq, Uf[c][0], s0 + M::p16, lane);
            // o over v's place
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    w[2 * n + half] = bf16x2(aq[n][2 * half] * up[half], aq[n][2 * half + 1] * up[half]);
            stsm4_t(tile_at<DV * 2>(s0 + vt, bb * 16 + vrow, vchunk), w);
        }
        tc::tc_fence_before();
        redo |= (uint32_t)watched(flag) << k;
        __syncwarp();
#pragma unroll
        for (int x = 0; x < NB; ++x) {
            const int i = vr + 16 * x;
            if (i < T)
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(d.o[layer]) + vo0 + ((size_t)i * d.HV + k) * DV) =
                    *reinterpret_cast<const uint4*>(sm + tile_at<DV * 2>(vt, i, vc));
        }
        __syncwarp();  // before V is fetched over it
    }
    if (redo) atomicOr(redo_s, (int)redo);
    cp_wait<0>();
    __syncthreads();
    redo = *redo_s;
    if (warp == 1) {
        tc::tc_fence_after();
        if (!ok)  // let the MMAs end before their TMEM goes
            for (int x = 0; x < 2; ++x) tc::mbar_drain(&bars[x], 0);
        tc::tmem_dealloc(tmem, M::cols);
    }
    if (!ok) {
        if (threadIdx.x == 0) dev_fail(status, TSV_DEV_TIMEOUT, b, h0);
        return;
    }
    for (int k = 0; k < heads; ++k)
        if (redo & (1u << k)) tree_fp32<DK, DV, NB>(d, anc, layer, b, h0 + k, sm, rows[k]);
}

template <int DK, int DV, int NB>
static void launch_tree_nb(const tsv_gdn_desc& d, const uint64_t* anc, int32_t* status, cudaStream_t stream) {
    constexpr int sm = TreeSmem<DK, DV, NB>::total;
    cudaFuncSetAttribute(gdn_tree_kernel<DK, DV, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
    // Value heads per CTA: as many as share a key head (up to kMaxHeads) as long as every SM gets CTAs for two rounds;
    // fewer, larger CTAs save the staging but leave SMs idle on small batches.  48 layers x 48 heads, one tree of 3 nodes:
    // three heads per CTA 35.4 us, one 50.0.
    const int per = d.HV / d.HK;
    int heads = 1;
    for (int x = 2; x <= kMaxHeads; ++x)
        if (per % x == 0 && (long long)d.n_layers * d.B * d.HV / x >= 4LL * sm_count()) heads = x;
    // The last heads, four for every three SMs, have a CTA each: the call ends sooner than with large CTAs alone (3 nodes 35.4
    // against 37.6 us, 16 nodes 38.8 against 40.6; twice as many 36.9 and 40.5, half as many 35.5 and 38.9).
    const long long all = (long long)d.n_layers * d.B * d.HV;
    const long long big = heads > 1 ? (all - sm_count() * 4 / 3) / heads : all;
    launch_pdl(gdn_tree_kernel<DK, DV, NB>, (unsigned)(big + (all - big * heads)), 2 * DV, sm, stream, d, anc, heads, (int)big, status);
}

template <int DK, int DV>
static void launch_tree_dims(const tsv_gdn_desc& d, const uint64_t* anc, int32_t* status, cudaStream_t stream) {
    if (d.T <= 16) launch_tree_nb<DK, DV, 1>(d, anc, status, stream);
    else if (d.T <= 32) launch_tree_nb<DK, DV, 2>(d, anc, status, stream);
    else if (d.T <= 48) launch_tree_nb<DK, DV, 3>(d, anc, status, stream);
    else launch_tree_nb<DK, DV, 4>(d, anc, status, stream);
}

void launch_gdn_tree(const tsv_gdn_desc& d, const uint64_t* anc, int32_t* status, cudaStream_t stream) {
    if (d.DK == 64 && d.DV == 64) launch_tree_dims<64, 64>(d, anc, status, stream);
    else if (d.DK == 64) launch_tree_dims<64, 128>(d, anc, status, stream);
    else if (d.DV == 64) launch_tree_dims<128, 64>(d, anc, status, stream);
    else launch_tree_dims<128, 128>(d, anc, status, stream);
}

}  // namespace tsv
