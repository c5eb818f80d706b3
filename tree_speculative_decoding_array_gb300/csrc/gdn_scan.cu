// tsv_gdn_scan over many tokens: the gated delta rule in chunks of 64.
//
// A chunk is one triangular system (gdn_tc.cuh) whose rows are consecutive tokens, and the state moves on by
//     S <- e^{G_n} S + sum_j e^{G_n - G_j} u_j k_j^T        (n: the chunk's last token)
// One persistent CTA per (layer, sequence, value head) walks its chunks - or two, of half the value features each, where
// the heads alone would leave half of the SMs idle.  Two groups of warps work a chunk apart:
//   8 preparing warps   stage K, Q, V and the gates of a chunk, take [K; Q] K^T on the tensor cores and build the
//                       system's matrices; two buffers, so they run up to two chunks ahead.  A chunk's global loads
//                       are issued while the one before is prepared.
//   DV / 16 state warps 16 value features each: split the state into fp16 hi + lo pairs (TMEM), S [K; Q]^T on the
//                       tensor cores (the lo pieces for K only: what reaches o alone is rounded to bf16 anyway), solve
//                       the system in mma fragments, write u as hi + lo pairs to TMEM, and let the tensor cores add
//                       their product with K onto the decayed state, which stays in TMEM in fp32.
// The system is solved right-looking: U_b is applied to every block after b at once, so that the products of different
// blocks are independent.
// 16391 tokens, 48 heads of 128 x 128: 1.21 ms alone, 1.34 among others, about 5 us a chunk, where reading and writing
// everything once would take 81 us: bound by the two groups' chains of steps (split, product, solve, o and the new state;
// staging, product, matrices), which are of equal length.  24 prompts of 5 to 4001 tokens 0.47 ms.
// What reaches the state is kept to 2^-22 (fp16 pairs; K's values are exact), what reaches o alone to 2^-12.
#include <math.h>

#include "gdn_tc.cuh"

namespace tsv {

constexpr int kScanPrep = 8;  // preparing warps
constexpr int kScanT = 64;    // tokens per chunk
constexpr int kScanNB = 4;
constexpr float kFaintState = 0x1p-6f;  // a write's pair holds 2^-25 of the scale, 2^-19 of this
constexpr int kScanSort = 32 * (kScanPrep + 4);  // sequences that can be sorted: a thread each

template <int DK, int DV>
struct ScanSmem {
    static constexpr int T = kScanT;
    // per buffer
    static constexpr int kq = 0;                    // K rows [64], Q rows [64], DK fp16 each
    static constexpr int v = kq + 2 * T * DK * 2;   // V rows [64], DV bf16 each; o over them
    static constexpr int a16 = v + T * DV * 2;      // hi and lo tiles of -A and the diagonal blocks' inverses
    static constexpr int p16 = a16 + 2 * T * 128;   // P
    static constexpr int keys = p16 + T * 128;
    static constexpr int rows = keys + (int)sizeof(GdnKeys);
    static constexpr int dj = rows + (int)sizeof(GdnRows);  // e^{G_n - G_j} times k_j's factor, then e^{G_n}
    static constexpr int buffer = (dj + 65 * 4 + 1023) / 1024 * 1024;
    static constexpr int diag = 2 * buffer;                        // [4][16][kDiag] fp32
    static constexpr int slow = diag + kScanNB * 16 * kDiag * 4;   // fp32 path: one token's k and q, and k . q
    static constexpr int bars = slow + (2 * 128 + 4) * 4;
    static constexpr int total = bars + 16 * 8;
    // [K; Q] K^T reads 128 rows per 64-feature block: exactly the tile
    // TMEM columns: the state (fp32), its hi and lo pieces (then u's), S [K; Q]^T, [K; Q] K^T
    static constexpr int col_s = 0, col_hi = DK, col_lo = col_hi + DK / 2, col_d = col_lo + DK / 2, col_g = col_d + 128;
    static constexpr int cols = 512;
    static_assert(col_g + T <= 512, "TMEM");
};

// Barriers of one CTA.
struct ScanBars {
    uint64_t full[2], empty[2], gram, prod, state, drain_s, drain_p;
    uint32_t tmem;
    int abort, bad[2], said[2][2];
};

// One of the CTA's two groups of warps (hardware barrier 1 + which, `threads` threads).  Only the group's first warp
// polls a barrier; the others wait for it at the group's own barrier and take its answer, so every warp of a group
// takes the same decisions, always meets the others, and waits without spending issue slots.
struct Group {
    int which, threads;
    bool lead;
    volatile int* said;  // [2]
    volatile int* abort;
    uint32_t turn;
    __device__ __forceinline__ void sync() { asm volatile("bar.sync %0, %1;" ::"r"(1 + which), "r"(threads) : "memory"); }
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
        const int slot = turn++ & 1;
        if (lead) {
            const bool ok = warp_wait(bar, parity, abort);
            if ((threadIdx.x & 31) == 0) said[slot] = ok;
        }
        sync();
        return said[slot] != 0;
    }
};

// A chunk token by token in fp32, by the state warps: the state in TMEM times un0 / un1 (features g, g + 8 of the warp's
// 16) is advanced over rows row .. row + nt - 1 and written back unscaled; o goes to global memory.
template <int DK>
__device__ __noinline__ void chunk_fp32(const tsv_gdn_desc& d, int layer, int h, size_t row, int nt, uint32_t state, int fb, float un0,
                                        float un1, float* tk, Group& group) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, hk = h / (d.HV / d.HK);
    float S[DK / 2];  // S[32 x + 4 n + 2 half + e]: feature fb + g + 8 half, column 64 x + 8 n + 2 t + e
#pragma unroll
    for (int x = 0; x < DK / 64; ++x) tc::tmem_ld_frag8(state + 64 * x, S + 32 * x);
    tc::tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < DK / 2; ++x) S[x] *= (x >> 1) & 1 ? un1 : un0;
    for (int i = 0; i < nt; ++i, ++row) {
        if (warp == 0) {
            float kx[DK / 32], qx[DK / 32], kq = 0.f;
            unit_row<DK>(reinterpret_cast<const uint16_t*>(d.k[layer]) + (row * d.HK + hk) * DK, d.norm_eps, 1.f, lane, kx);
            unit_row<DK>(reinterpret_cast<const uint16_t*>(d.q[layer]) + (row * d.HK + hk) * DK, d.norm_eps, d.scale, lane, qx);
#pragma unroll
            for (int e = 0; e < DK / 32; ++e) {
                tk[lane + 32 * e] = kx[e];
                tk[128 + lane + 32 * e] = qx[e];
                kq = fmaf(kx[e], qx[e], kq);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(0xFFFFFFFFu, kq, o);
            if (lane == 0) tk[256] = kq;
        }
        group.sync();
        const float a = expf(d.g[layer][row * d.HV + h]), be = d.beta[layer][row * d.HV + h];
        float sk[2] = {0.f, 0.f}, sq[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < DK / 2; ++x) {
            const int e = (x >> 5) * 64 + ((x & 31) >> 2) * 8 + 2 * t + (x & 1);
            sk[(x >> 1) & 1] = fmaf(S[x], tk[e], sk[(x >> 1) & 1]);
            sq[(x >> 1) & 1] = fmaf(S[x], tk[128 + e], sq[(x >> 1) & 1]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                sk[half] += __shfl_xor_sync(0xFFFFFFFFu, sk[half], o);
                sq[half] += __shfl_xor_sync(0xFFFFFFFFu, sq[half], o);
            }
            const size_t at = (row * d.HV + h) * d.DV + fb + g + 8 * half;
            const float u = be * (bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(d.v[layer])[at]) - a * sk[half]);
            if (t == 0) reinterpret_cast<__nv_bfloat16*>(d.o[layer])[at] = __float2bfloat16(fmaf(a, sq[half], u * tk[256]));
            sk[half] = u;
        }
#pragma unroll
        for (int x = 0; x < DK / 2; ++x) {
            const int e = (x >> 5) * 64 + ((x & 31) >> 2) * 8 + 2 * t + (x & 1);
            S[x] = fmaf(sk[(x >> 1) & 1], tk[e], a * S[x]);
        }
        group.sync();
    }
#pragma unroll
    for (int x = 0; x < DK / 64; ++x) tc::tmem_st_frag8f(state + 64 * x, S + 32 * x);
}

// Whether one of this warp's features needs the fp32 path for a chunk: for what faint_rows() says, or because the state (x:
// the largest of its row) lies outside what fp32 holds at the chunk's scale (d; c: from the scale that it is held at).
constexpr float kScaleMax = 0x1p100f, kStateMin = 0x1p-40f;
template <int BYTES, int NB>
__device__ __noinline__ bool scan_redo(const char* v, int fb, float d0, float d1, float s0, float s1, float x0, float x1, float c0, float c1,
                                       const GdnRows& rw, const GdnKeys& ky, int n) {
    bool redo = faint_rows<BYTES, NB>(v, fb, d0, d1, s0, s1, rw, ky, n);
    redo = redo || (x0 > 0.f && !(x0 * d0 >= kStateMin && c0 <= kScaleMax)) || (x1 > 0.f && !(x1 * d1 >= kStateMin && c1 <= kScaleMax));
    return __any_sync(0xFFFFFFFFu, redo);
}

// DV: value features of one CTA, d.DV or half of it.
template <int DK, int DV>
__global__ void __launch_bounds__((kScanPrep + DV / 16) * 32, 1)
    gdn_scan_kernel(const __grid_constant__ tsv_gdn_desc d, const int32_t* __restrict__ cu_len, int max_len, int sorted, int32_t* status) {
    griddep_begin();
    using M = ScanSmem<DK, DV>;
    constexpr int SW = DV / 16;  // state warps
    constexpr int KS = DK / 16;
    constexpr int NB = kScanNB;
    extern __shared__ __align__(1024) char sm[];
    ScanBars& br = *reinterpret_cast<ScanBars*>(sm + M::bars);
    static_assert(sizeof(ScanBars) <= 128, "barriers");
    volatile int* abort_flag = &br.abort;
    const uint32_t s0 = tc::smem_u32(sm);
    const int slices = d.DV / DV;
    int item = blockIdx.x;
    const int f0 = item % slices * DV;  // this CTA's first value feature
    item /= slices;
    const int h = item % d.HV;
    item /= d.HV;
    const int layer = item % d.n_layers;
    int b = item / d.n_layers;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int row0, row1;
    if (sorted) {
        // CTAs start in the order of their index: this one takes the sequence of b-th most chunks (ties by index), its
        // number of chunks found bit by bit, a count of the batch each.
        int* equal = reinterpret_cast<int*>(sm + M::diag);
        int* pick = equal + 32;
        int mine = -1;
        row0 = row1 = 0;
        if (threadIdx.x < d.B) {
            row0 = cu_len[threadIdx.x];
            row1 = cu_len[threadIdx.x + 1];
            const long long len = (long long)row1 - row0;
            mine = len < 0 ? 0 : (int)((len > max_len ? max_len : len) + kScanT - 1) / kScanT;
        }
        int want = 0;
        for (int bit = 31 - __clz((max_len - 1) / kScanT + 1); bit >= 0; --bit)
            if (__syncthreads_count(mine >= (want | 1 << bit)) > b) want |= 1 << bit;
        const int more = __syncthreads_count(mine > want);
        const uint32_t same = __ballot_sync(0xFFFFFFFFu, mine == want);
        if (lane == 0) equal[warp] = __popc(same);
        __syncthreads();
        int before = more + __popc(same & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) before += equal[w];
        if (mine == want && before == b) {
            pick[0] = threadIdx.x;
            pick[1] = row0;
            pick[2] = row1;
        }
        __syncthreads();
        b = pick[0];
        row0 = pick[1];
        row1 = pick[2];
    } else {
        row0 = cu_len[b];
        row1 = cu_len[b + 1];
    }
    const int hk = h / (d.HV / d.HK);
    const int g = lane >> 2, t = lane & 3;

    if (row0 < 0 || row1 < row0 || row1 > d.T || row1 - row0 > max_len) {
        if (h == 0 && layer == 0 && f0 == 0 && threadIdx.x == 0) dev_fail(status, TSV_DEV_BAD_SEQ_LEN, b, row1);
        return;
    }
    const int n = row1 - row0;
    const size_t state0 = (((size_t)b * d.HV + h) * d.DV + f0) * DK;
    if (n == 0) {  // the state as it was
        if (d.state_out[layer] != d.state[layer])
            for (int e = threadIdx.x; e < DV * DK / 4; e += blockDim.x)
                reinterpret_cast<float4*>(d.state_out[layer] + state0)[e] = reinterpret_cast<const float4*>(d.state[layer] + state0)[e];
        return;
    }
    const int chunks = (n + kScanT - 1) / kScanT;

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(&br.full[x], 1);
            tc::mbar_init(&br.empty[x], 1);
            br.bad[x] = 0;
        }
        tc::mbar_init(&br.gram, 1);
        tc::mbar_init(&br.prod, 1);
        tc::mbar_init(&br.state, 1);
        tc::mbar_init(&br.drain_s, 1);
        tc::mbar_init(&br.drain_p, 1);
        br.abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&br.tmem, M::cols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = br.tmem;

    if (warp >= SW) {
        // ------------------------------------------------------------ preparing warps
        const int pw = warp - SW, pt = threadIdx.x - SW * 32;
        constexpr int PT = kScanPrep * 32;
        constexpr int LPR = DK / 8, CPR = DV / 8;
        constexpr int KQ = 2 * kScanT * LPR / PT, VC = kScanT * CPR / PT;
        const int chunk = pt % LPR;
        uint4 kq[KQ];
        float gi[2] = {0.f, 0.f}, bi[2] = {0.f, 0.f};
        auto fetch = [&](int c) {
            const int t0 = c * kScanT;
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int x = 0; x < KQ; ++x) {
                const int r = pt / LPR + x * (PT / LPR), i = t0 + (r & 63);
                const uint16_t* src = reinterpret_cast<const uint16_t*>(r >= kScanT ? d.q[layer] : d.k[layer]);
                kq[x] = i < n ? *reinterpret_cast<const uint4*>(src + ((size_t)(row0 + i) * d.HK + hk) * DK + chunk * 8) : zero;
            }
            if (pw == 1) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = t0 + 2 * lane + x;
                    gi[x] = i < n ? d.g[layer][(size_t)(row0 + i) * d.HV + h] : 0.f;
                    bi[x] = i < n ? d.beta[layer][(size_t)(row0 + i) * d.HV + h] : 0.f;
                }
            }
        };
        Group group = {1, PT, pw == 0, br.said[1], abort_flag, 0};
        // G of the fetched chunk: tokens 2 lane, 2 lane + 1 of one warp; inclusive scan over the lanes
        Pair G[2];
        auto sum_gates = [&]() {
            G[0] = log2_decay(gi[0]);
            Pair run = add(G[0], log2_decay(gi[1])), before;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                Pair y;
                y.hi = __shfl_up_sync(0xFFFFFFFFu, run.hi, o);
                y.lo = __shfl_up_sync(0xFFFFFFFFu, run.lo, o);
                if (lane >= o) run = add(run, y);
            }
            before.hi = __shfl_up_sync(0xFFFFFFFFu, run.hi, 1);
            before.lo = __shfl_up_sync(0xFFFFFFFFu, run.lo, 1);
            if (lane > 0) G[0] = add(G[0], before);
            G[1] = run;
        };
        fetch(0);
        if (pw == 1) sum_gates();
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const int buf = c & 1;
            char* bs = sm + buf * M::buffer;
            const uint32_t bs32 = s0 + buf * M::buffer;
            GdnKeys& ky = *reinterpret_cast<GdnKeys*>(bs + M::keys);
            GdnRows& rw = *reinterpret_cast<GdnRows*>(bs + M::rows);
            float* dj = reinterpret_cast<float*>(bs + M::dj);
            if (c >= 2 && !(ok = group.wait(&br.empty[buf], ((c >> 1) - 1) & 1))) break;
            if (pt == 0) br.bad[buf] = 0;  // read by the state warps before they gave the buffer back; set again after sync()
            uint32_t flag = 0;
#pragma unroll
            for (int x = 0; x < VC; ++x) {
                const int e = pt + x * PT, i = c * kScanT + e / CPR;
                cp16(bs32 + tile_at<DV * 2>(M::v, e / CPR, e % CPR),
                     reinterpret_cast<const uint16_t*>(d.v[layer]) + ((size_t)(row0 + min(i, n - 1)) * d.HV + h) * d.DV + f0 + e % CPR * 8, i < n);
            }
            cp_commit();
            constexpr int KH = KQ / 2;  // half of a thread's chunks at a time
#pragma unroll
            for (int x0 = 0; x0 < KQ; x0 += KH) {
                uint4 w[KH];
                float f[KH];
#pragma unroll
                for (int x = 0; x < KH; ++x) w[x] = kq[x0 + x];
                stage_chunks<DK, KH>(w, f, d.norm_eps, flag);
#pragma unroll
                for (int x = 0; x < KH; ++x) {
                    const int r = pt / LPR + (x0 + x) * (PT / LPR), i = r & 63;
                    *reinterpret_cast<uint4*>(bs + kq_at<2 * kScanT>(M::kq, (r & 64) + 16 * block_pos<NB>(i >> 4) + (i & 15), chunk)) = w[x];
                    if (chunk == 0) (r >= kScanT ? ky.fq : ky.fk)[i] = r >= kScanT ? f[x] * kOutLift : f[x];
                }
            }
            if (pw == 1) {
                *reinterpret_cast<float2*>(&rw.g_hi[2 * lane]) = make_float2(G[0].hi, G[1].hi);
                *reinterpret_cast<float2*>(&rw.g_lo[2 * lane]) = make_float2(G[0].lo, G[1].lo);
                *reinterpret_cast<float2*>(&rw.beta[2 * lane]) = make_float2(bi[0], bi[1]);
                ky.before[2 * lane] = (1ull << (2 * lane)) - 1ull;
                ky.before[2 * lane + 1] = (1ull << (2 * lane + 1)) - 1ull;
            }
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            group.sync();
            tc::tc_fence_after();
            if (pt == 6 * 32) {  // [K; Q] K^T, by a warp with a small share of the matrices
                const uint32_t id = tc::idesc_f16(false, false, false, 128, kScanT);
                const uint64_t desc = tc::sdesc_sw128(bs32 + M::kq, 16, 1024);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint64_t at = tc::sdesc_add(desc, (ks >> 2) * 2 * kScanT * 128 + (ks & 3) * 32);
                    tc::mma_f16(tmem + M::col_g, at, at, id, ks > 0);
                }
                tc::mma_commit(&br.gram);
            }
            __syncwarp();
            if (c + 1 < chunks) fetch(c + 1);
            if (pt >= 2 * kScanT) {  // for the state warps
                const int i = pt & 63;
                const bool q = pt >= 3 * kScanT;
                const float x = (q ? ky.fq : ky.fk)[i], gh = rw.g_hi[i], gl = rw.g_lo[i];
                (q ? rw.cq : rw.ck)[i] = tc::ex2_approx((gh - fade_exponent(rw.g_hi[0])) + gl) * x;
                if (!q) dj[i] = tc::ex2_approx((rw.g_hi[63] - gh) + (rw.g_lo[63] - gl)) * x;
                else if (i == 63) dj[64] = tc::ex2_approx(gh + gl);
            } else if (pw == 2) {
                const float write = least_write(rw, min(kScanT, n - c * kScanT), lane), e = fade_exponent(rw.g_hi[0]);
                if (lane == 0) {  // G falls from token to token
                    rw.e = e;
                    rw.fade = pow2_of(e);
                    rw.seen = tc::ex2_approx(rw.g_hi[63] - e);
                    rw.write = write;
                }
            }
            __syncwarp();
            if (!(ok = group.wait(&br.gram, c & 1))) break;
            tc::tc_fence_after();
            warp_matrices<NB, 2>(pw & 3, pw >> 2, tmem + M::col_g, bs + M::a16, bs + M::p16, reinterpret_cast<float*>(sm + M::diag), ky, rw, flag,
                                 lane);
            if (watched(flag)) br.bad[buf] = 1;
            tc::tc_fence_before();
            cp_wait<0>();  // V
            group.sync();
            if (pt == 0) tc::mbar_arrive(&br.full[buf]);
            if (pw == 1) sum_gates();
        }
        if (!ok && pt == 6 * 32) {  // let this thread's MMAs end
            tc::mma_commit(&br.drain_p);
            tc::mbar_drain(&br.drain_p, 0);
        }
    } else {
        // ------------------------------------------------------------ state warps
        const int lane0 = DV == 128 ? (warp & 3) * 32 + (warp >> 2) * 16 : warp * 32;  // TMEM lanes (16 of them)
        const int fb = DV == 128 ? lane0 : warp * 16;                                  // value features
        const uint32_t la = tmem + ((uint32_t)lane0 << 16);
        const int vrow = ((lane >> 4) << 3) + (lane & 7), vchunk = fb / 8 + ((lane >> 3) & 1);
        Group group = {0, SW * 32, warp == 0, br.said[0], abort_flag, 0};
        // 64 columns of the state at a time: r[4 n + 2 half + e] = S[fb + g + 8 half][64 x + 8 n + 2 t + e]
        float r[32];
        const float* S = d.state[layer] + state0 + (size_t)(fb + g) * DK + 2 * t;
#pragma unroll 1
        for (int x = 0; x < DK / 64; ++x) {
#pragma unroll
            for (int nn = 0; nn < 8; ++nn)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float2 y = __ldcs(reinterpret_cast<const float2*>(S + half * 8 * DK + 64 * x + 8 * nn));
                    r[4 * nn + 2 * half] = y.x;
                    r[4 * nn + 2 * half + 1] = y.y;
                }
            tc::tmem_st_frag8f(la + M::col_s + 64 * x, r);
        }
        tc::tmem_wait_st();
        float up[2] = {1.f, 1.f};  // the state is what TMEM holds times up
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const int buf = c & 1;
            char* bs = sm + buf * M::buffer;
            const uint32_t bs32 = s0 + buf * M::buffer;
            const GdnKeys& ky = *reinterpret_cast<const GdnKeys*>(bs + M::keys);
            const GdnRows& rw = *reinterpret_cast<const GdnRows*>(bs + M::rows);
            const float* dj = reinterpret_cast<const float*>(bs + M::dj);
            const int nt = min(kScanT, n - c * kScanT);
            uint32_t flag = 0;
            if (!(ok = group.wait(&br.full[buf], (c >> 1) & 1))) break;
            // each feature's power-of-two scale from the largest of its state row and v
            float sx[2] = {0.f, 0.f}, down[2], sc[2];
            uint32_t vf[NB][4], top[2] = {0, 0}, low[2] = {kInf2, kInf2};
#pragma unroll
            for (int bb = 0; bb < NB; ++bb) {
                ldsm4_t(vf[bb], tile_at<DV * 2>(bs32 + M::v, bb * 16 + vrow, vchunk));
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    top[x & 1] = abs_max2(top[x & 1], vf[bb][x]);
                    low[x & 1] = abs_min2(low[x & 1], vf[bb][x]);
                }
            }
            const float e_n = dj[64];
            tc::tc_fence_after();
            float S2[32];  // 64 columns of this thread's part of the state (all of it would crowd registers and instruction cache)
#pragma unroll 1
            for (int x = 0; x < DK / 64; ++x) {
                tc::tmem_ld_frag8(la + M::col_s + 64 * x, S2);
                tc::tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; y += 4)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        sx[half] = fmaxf(sx[half], fmaxf(fabsf(S2[y + 2 * half]), fabsf(S2[y + 2 * half + 1])));
            }
            const float fade = rw.fade, seen = rw.seen;
            // sd: the feature's largest state, faded and scaled; the smaller of both features' (fade_s), of the state as it is
            // (full_s) and of all v (least), where a feature is not empty
            float up_new[2], sd[2], fade_s = INFINITY, full_s = INFINITY, least = INFINITY;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float m = fmaxf(bf16_lo(top[half]), bf16_hi(top[half]));
                sx[half] *= up[half];
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    sx[half] = fmaxf(sx[half], __shfl_xor_sync(0xFFFFFFFFu, sx[half], x));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
                }
                m = fmaxf(8.f * (sx[half] * fade), m);
                pow2_scale(m * (1.f / kLift), down[half], up_new[half]);
                sd[half] = sx[half] * fade * down[half];
                sc[half] = fminf(up[half] * down[half], 2.f * kScaleMax);
                const float empty = m == 0.f ? INFINITY : 0.f;
                fade_s = fminf(fade_s, sd[half] + empty);
                full_s = fminf(full_s, sx[half] * down[half] + empty);
                least = fminf(least, fminf(bf16_lo(low[half]), bf16_hi(low[half])) * down[half] + empty);
            }
            // hardly ever: where the state fades out of sight, and where it cannot be held in fp32 at v's scale
            const bool check = (fade_s * seen < kFaint && (least * rw.write < kFaint || full_s < kStateMin)) || !(fmaxf(sc[0], sc[1]) <= kScaleMax);
            bool redo = false;
            if (__any_sync(0xFFFFFFFFu, check))
                redo = scan_redo<DV * 2, NB>(bs + M::v, fb, down[0], down[1], sd[0], sd[1], sx[0], sx[1], sc[0], sc[1], rw, ky, nt);
            if (redo) {  // this chunk is for the fp32 path: the state stays as it is
                flag = 0x7FFF7FFFu;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    up_new[half] = up[half];
                    down[half] = 1.f / up[half];
                    sc[half] = 1.f;
                }
            }
            up[0] = up_new[0];
            up[1] = up_new[1];
            // Unless the decay over the chunk is next to nothing (its inverse then still is far inside fp32) the state is decayed
            // (and scaled) in TMEM at once: should the chunk have to be done again in fp32, the state can be had back.
            const bool early = e_n >= 0x1p-60f && !redo;
            const float se[2] = {sc[0] * e_n, sc[1] * e_n}, sf[2] = {sc[0] * fade, sc[1] * fade};
            float last[2] = {sd[0] * seen, sd[1] * seen};  // what the feature's new state is made of, its largest
#pragma unroll 1
            for (int x = DK / 64 - 1; x >= 0; --x) {
                uint32_t hi[16], lo[16];
                if (x != DK / 64 - 1) {
                    tc::tmem_ld_frag8(la + M::col_s + 64 * x, S2);
                    tc::tmem_wait_ld();
                }
#pragma unroll
                for (int y = 0; y < 16; ++y) {  // y = 2 n + half
                    const float2 s = make_float2(S2[2 * y], S2[2 * y + 1]);
                    const float2 z = mul2(s, make_float2(sf[y & 1], sf[y & 1]));
                    split2(z.x, z.y, hi[y], lo[y]);
                    if (early) {
                        const float2 ze = mul2(s, make_float2(se[y & 1], se[y & 1]));
                        S2[2 * y] = ze.x;
                        S2[2 * y + 1] = ze.y;
                    }
                }
                if (early) tc::tmem_st_frag8f(la + M::col_s + 64 * x, S2);
                tc::tmem_st_frag8(la + M::col_hi + 32 * x, hi);
                tc::tmem_st_frag8(la + M::col_lo + 32 * x, lo);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            group.sync();
            const uint64_t desc = tc::sdesc_sw128(bs32 + M::kq, 16, 1024);
            if (threadIdx.x == 0) {  // S [K; Q]^T
                tc::tc_fence_after();
                const uint32_t id = tc::idesc_f16(false, false, false, 128, 2 * kScanT), idk = tc::idesc_f16(false, false, false, 128, kScanT);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    tc::mma_f16_ts(tmem + M::col_d, tmem + M::col_hi + ks * 8,
                                   tc::sdesc_add(desc, (ks >> 2) * 2 * kScanT * 128 + (ks & 3) * 32), id, ks > 0);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    tc::mma_f16_ts(tmem + M::col_d, tmem + M::col_lo + ks * 8,
                                   tc::sdesc_add(desc, (ks >> 2) * 2 * kScanT * 128 + (ks & 3) * 32), idk, 1);
                tc::mma_commit(&br.prod);
            }
            __syncwarp();
            if (!(ok = group.wait(&br.prod, c & 1))) break;
            tc::tc_fence_after();

            float ak[NB][2][4];
#pragma unroll
            for (int bb = 0; bb < NB; ++bb) {
                float x8[8];
                tc::tmem_ld_frag2(la + M::col_d + 16 * block_pos<NB>(bb), x8);
#pragma unroll
                for (int x = 0; x < 8; ++x) ak[bb][x >> 2][x & 3] = x8[x];
            }
            tc::tmem_wait_ld();
#pragma unroll
            for (int bb = 0; bb < NB; ++bb) {
                ldsm4_t(vf[bb], tile_at<DV * 2>(bs32 + M::v, bb * 16 + vrow, vchunk));
                block_rhs<2>(bb, ak[bb], vf[bb], down, rw, t);
            }
            uint32_t Uh[NB][4];
#pragma unroll
            for (int bb = 0; bb < NB; ++bb) {
                uint32_t Uf[2][4];
                float u[2][4];
                block_solve<NB, 2>(bb, ak[bb], Uf, u, bs32 + M::a16, flag, lane);
#pragma unroll
                for (int bn = bb + 1; bn < NB; ++bn) block_update<NB, 2>(bn, bb, ak[bn], Uf, bs32 + M::a16, lane);
                // u for the state, over the state's pieces
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) Uh[bb][x] = Uf[0][x];
#pragma unroll
                for (int nn = 0; nn < 2; ++nn) {
                    const float2 z = *reinterpret_cast<const float2*>(&dj[bb * 16 + nn * 8 + 2 * t]);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float2 y = mul2(make_float2(u[nn][2 * half], u[nn][2 * half + 1]), z);
                        split2(y.x, y.y, hi[2 * nn + half], lo[2 * nn + half]);
                        last[half] = fmaxf(fmaxf(last[half], fabsf(y.x)), fabsf(y.y));
                        watch(flag, hi[2 * nn + half]);
                    }
                }
                tc::tmem_st_frag2(la + M::col_hi + 8 * block_pos<NB>(bb), hi);
                tc::tmem_st_frag2(la + M::col_lo + 8 * block_pos<NB>(bb), lo);
            }
            // a new state whose every part fp16 holds by its last bits only
            if (__any_sync(0xFFFFFFFFu, fminf(last[0], last[1]) < kFaintState)) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int x = 1; x < 4; x <<= 1) last[half] = fmaxf(last[half], __shfl_xor_sync(0xFFFFFFFFu, last[half], x));
                    if (last[half] > 0.f && last[half] < kFaintState) flag = 0x7FFF7FFFu;
                }
            }
            if (watched(flag)) br.bad[buf] = 1;
            tc::tmem_wait_st();
            tc::tc_fence_before();
            group.sync();
            const bool bad = *reinterpret_cast<volatile int*>(&br.bad[buf]) != 0;
            if (bad) {
                // fp32, token by token: an operand left fp16's range.  Not finite inputs then reach what the recurrence
                // lets them reach: later tokens, and with v only their own feature.  What TMEM holds times un is the
                // state ahead of the chunk.
                const float un0 = early ? up[0] / e_n : sc[0] * up[0], un1 = early ? up[1] / e_n : sc[1] * up[1];
                chunk_fp32<DK>(d, layer, h, (size_t)row0 + (size_t)c * kScanT, nt, la + M::col_s, f0 + fb, un0, un1,
                               reinterpret_cast<float*>(sm + M::slow), group);
                up[0] = up[1] = 1.f;
            } else if (!early) {
#pragma unroll 1
                for (int x = 0; x < DK / 64; ++x) {
                    tc::tmem_ld_frag8(la + M::col_s + 64 * x, S2);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int y = 0; y < 32; ++y) S2[y] *= sc[(y >> 1) & 1] * e_n;
                    tc::tmem_st_frag8f(la + M::col_s + 64 * x, S2);
                }
            }
            if (bad || !early) {
                tc::tmem_wait_st();
                tc::tc_fence_before();
                group.sync();
            }
            if (threadIdx.x == 0) {  // S += U'^T K
                tc::tc_fence_after();
                if (!bad) {
                    const uint32_t id = tc::idesc_f16(false, false, true, 128, DK);
                    const uint64_t kd = tc::sdesc_sw128(bs32 + M::kq, 2 * kScanT * 128, 1024);
#pragma unroll
                    for (int ks = 0; ks < kScanT / 16; ++ks)
                        tc::mma_f16_ts(tmem + M::col_s, tmem + M::col_hi + ks * 8, tc::sdesc_add(kd, ks * 2048), id, 1);
#pragma unroll
                    for (int ks = 0; ks < kScanT / 16; ++ks)
                        tc::mma_f16_ts(tmem + M::col_s, tmem + M::col_lo + ks * 8, tc::sdesc_add(kd, ks * 2048), id, 1);
                }
                tc::mma_commit(&br.state);
            }
            __syncwarp();
            if (!bad) {  // o while the tensor cores work on the state
                const float oscale = d.scale / kOutLift, uo[2] = {up[0] * oscale, up[1] * oscale};
                // o over v's place
#pragma unroll
                for (int bb = 0; bb < NB; ++bb) {
                    float x8[8], aq[2][4];
                    uint32_t w[4];
                    tc::tmem_ld_frag2(la + M::col_d + kScanT + 16 * block_pos<NB>(bb), x8);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 8; ++x) aq[x >> 2][x & 3] = x8[x];
                    block_rhs_q(bb, aq, rw, t);
#pragma unroll
                    for (int cc = 0; cc <= bb; ++cc) block_out(bb, cc, aq, Uh[cc], bs32 + M::p16, lane);
#pragma unroll
                    for (int nn = 0; nn < 2; ++nn)
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            w[2 * nn + half] = bf16x2(aq[nn][2 * half] * uo[half], aq[nn][2 * half + 1] * uo[half]);
                    stsm4_t(tile_at<DV * 2>(bs32 + M::v, bb * 16 + vrow, vchunk), w);
                }
                group.sync();
                constexpr int CPR = DV / 8;
                for (int e = threadIdx.x; e < nt * CPR; e += SW * 32) {
                    const int i = e / CPR, cc = e % CPR;
                    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(d.o[layer]) +
                                              ((size_t)(row0 + c * kScanT + i) * d.HV + h) * d.DV + f0 + cc * 8) =
                        *reinterpret_cast<const uint4*>(bs + tile_at<DV * 2>(M::v, i, cc));
                }
            }
            // the new state, with which the buffer is free
            if (!(ok = group.wait(&br.state, c & 1))) break;
            if (threadIdx.x == 0) tc::mbar_arrive(&br.empty[buf]);
        }
        if (ok) {
            tc::tc_fence_after();
            float* out = d.state_out[layer] + state0 + (size_t)(fb + g) * DK + 2 * t;
#pragma unroll 1
            for (int x = 0; x < DK / 64; ++x) {
                tc::tmem_ld_frag8(la + M::col_s + 64 * x, r);
                tc::tmem_wait_ld();
#pragma unroll
                for (int nn = 0; nn < 8; ++nn)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        *reinterpret_cast<float2*>(out + half * 8 * DK + 64 * x + 8 * nn) =
                            make_float2(r[4 * nn + 2 * half] * up[half], r[4 * nn + 2 * half + 1] * up[half]);
            }
        } else if (threadIdx.x == 0) {  // let this thread's MMAs end
            tc::mma_commit(&br.drain_s);
            tc::mbar_drain(&br.drain_s, 0);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) dev_fail(status, TSV_DEV_TIMEOUT, b, h);
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, M::cols);
    }
}

template <int DK, int DV>
static void launch_scan_dims(const tsv_gdn_desc& d, const int32_t* cu_len, int max_len, int32_t* status, cudaStream_t stream) {
    constexpr int sm = ScanSmem<DK, DV>::total;
    cudaFuncSetAttribute(gdn_scan_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
    // The longest sequences first, where one of the longest, started last, would add more than a sixteenth to the whole
    // (max_len rows of one head against every SM's share of all rows).  24 prompts of 5 to 4001 tokens: 0.465 ms, in the
    // order given 0.516; finding its place costs a CTA up to 0.9 us: 256 prompts of 17 to 400 tokens 1.77 ms, in the order
    // given 1.73.
    const int sorted = d.B > 1 && d.B <= kScanSort && max_len > kScanT &&
                       16LL * max_len * sm_count() > (long long)d.T * d.n_layers * d.HV;
    launch_pdl(gdn_scan_kernel<DK, DV>, (unsigned)((long long)d.n_layers * d.B * d.HV * (d.DV / DV)), (kScanPrep + DV / 16) * 32, sm,
               stream, d, cu_len, max_len, sorted, status);
}

void launch_gdn_scan(const tsv_gdn_desc& d, const int32_t* cu_len, int max_len, int32_t* status, cudaStream_t stream) {
    // Half heads while both halves of every head find an SM: the preparation is done twice, but a half's warps have more
    // of their SM to themselves.  48 heads, 16391 tokens: 1.33 ms, whole heads 1.42 (alone 1.20 and 1.42); two prompts of 4096:
    // 0.61 ms, whole heads 0.39.
    const bool half = d.DV == 64 || 2LL * d.n_layers * d.B * d.HV <= sm_count();
    if (d.DK == 64) half ? launch_scan_dims<64, 64>(d, cu_len, max_len, status, stream) : launch_scan_dims<64, 128>(d, cu_len, max_len, status, stream);
    else half ? launch_scan_dims<128, 64>(d, cu_len, max_len, status, stream) : launch_scan_dims<128, 128>(d, cu_len, max_len, status, stream);
}

}  // namespace tsv
