// Attention of few query rows over a 4-bit cache (single tokens, short chains, head sizes the tcgen05 kernel lacks).
//
// Same operation as attention.cu.  With up to 16 query rows per K/V stream the work is reading the cache (288 bytes per
// position, head and 256 features) and taking its codes apart; a tcgen05 tile of 128 rows would spend more on empty rows
// than the cache takes to arrive.  So the codes go from shared memory to mma.sync operands in registers, one mask each:
// a code in the low bits of an fp16 is a subnormal, q * 2^-24 (or q * 2^-20 four bits higher), exact, and the tensor
// cores multiply subnormals exactly.  No code is ever converted, scaled or biased:
//   scores   S^T = K Q^T, 16 keys x 8 query rows per MMA, one accumulator per group of 64 features; the group's scale and
//            bias meet the accumulator: s_g acc_g 2^24 + b_g sum_{f in g} q_f
//   output   O^T = V^T P^T, 16 features x 8 rows per MMA over 16 keys: every group's P carries the keys' scales of that
//            group (P s_g as fp16), the biases are summed beside it (sum_c p_c b_gc)
// Q takes the order and the power of two of the masks when it is loaded, the output's when it is written.
//
// A warp takes 16 keys at a time through a private ring of cp.async stages, all rows, all features; the four warps of a
// CTA interleave over one key range and merge their partials through shared memory at its end.  32 tokens over up to 32768
// keys, 4 layers x 4 heads of 256: 668 us, 5.4 TB/s (720 us with scales above 3.9 in every step); about 25 instructions per
// key and warp take 62 % of the issue slots, half of them masks on the half-rate integer pipe.
#include <math.h>

#include "common.cuh"
#include "gdn_tc.cuh"

namespace tsv {

constexpr int kFewWarps = 4;
constexpr int kFewKeys = 16;  // keys per warp and step
// P s_g goes through fp16, whose smallest value is 2^-24: with scales of 2^-7 (values of 0.06) a key 2^17 behind the
// maximum would be lost, and a long cache holds many such keys behind an early one that draws most of the weight.  So
// P is lifted by 2^12, but for a group in steps where one of its scales is above 3.9 (4 x 2^12 x 3.9 < 65504): its part of O
// is brought to the other unit where such steps begin and end, and the other groups keep their lift.
constexpr float kFewLift = 4096.f;

// Lanes whose group (lane % NG) is 0; what takes the lift off group j, given the lanes that saw a large scale of theirs.
template <int NG>
constexpr uint32_t few_lanes() {
    return NG == 4 ? 0x11111111u : NG == 2 ? 0x55555555u : 0xFFFFFFFFu;
}
template <int NG>
__device__ __forceinline__ float few_unit(uint32_t wide, int j) {
    return wide & (few_lanes<NG>() << j) ? 1.f / kFewLift : 1.f;
}

template <int D>
struct FewTile {
    static constexpr int groups = D / 64;
    static constexpr int row = D / 2;                 // bytes of codes per key
    static constexpr int pairs = 4 * groups;          // bytes of (scale, bias) pairs per key
    static constexpr int k = 0, v = kFewKeys * row, ks = 2 * v, vs = ks + kFewKeys * pairs;
    static constexpr int bytes = vs + kFewKeys * pairs;
    // Which 16-byte chunk of a row a chunk is kept in, so that the reads of 8 keys' 32-byte groups (K) and of 4 keys'
    // (V) fall into different banks.
    static __device__ __forceinline__ int k_swizzle(int key) {
        return D == 256 ? ((key & 3) << 1) | ((key >> 2) & 1) : D == 128 ? ((key >> 1) & 1) << 1 : 0;
    }
    static __device__ __forceinline__ int v_swizzle(int key) {
        return D == 256 ? ((key >> 1) & 3) << 1 : D == 128 ? ((key >> 1) & 1) << 1 : 0;
    }
};
template <int D, int NT>
constexpr int few_stages() {
    return D == 256 ? (NT == 1 ? 4 : 5) : 6;
}
template <int D, int NT>
constexpr int few_smem() {
    constexpr int ring = few_stages<D, NT>() * kFewWarps * FewTile<D>::bytes;
    constexpr int merge = kFewWarps * 8 * NT * (D + 4) * 4;
    return (ring > merge ? ring : merge) + (NT == 1 ? 0 : FewTile<D>::groups * 4 * NT * 32 * 8);
}

template <int BYTES>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src, bool real) {
    if constexpr (BYTES == 16)
        cp16(dst, src, real);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(real ? BYTES : 0) : "memory");
}

// 8 x 8 16-bit values across a warp, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int NT>
__global__ void __launch_bounds__(kFewWarps * 32, NT == 1 ? 3 : 2)
    attn_few_kernel(const __grid_constant__ tsv_attn_desc d, int splits, int chunk, float* __restrict__ ws_o, float* __restrict__ ws_ml,
                    int32_t* status) {
    griddep_begin();
    using F = FewTile<D>;
    constexpr int NG = F::groups, ST = few_stages<D, NT>();
    extern __shared__ __align__(128) char sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = d.HQ / d.HKV, T = d.T, rows_unit = G * T;
    const int unit = blockIdx.z, split = blockIdx.x, row0 = blockIdx.y * 8 * NT;
    const int kvh = unit % d.HKV, b = (unit / d.HKV) % d.B, layer = unit / (d.HKV * d.B);
    const int kvl = d.kv_len[b];
    if (kvl < T || kvl > d.max_kv_len || (int64_t)kvl > d.s_cap) {
        if (split == 0 && row0 == 0 && kvh == 0 && layer == 0 && threadIdx.x == 0) dev_fail(status, TSV_DEV_BAD_KV_LEN, b, kvl);
        return;
    }
    const int S = kvl - T, win = d.window[layer];
    int k_begin = split * chunk;
    const int k_end = min(kvl, k_begin + chunk);
    // Sliding-window layer: node i keeps keys c >= S + i - win + 1; whole steps below the first row's bound are skipped.
    const int lo_first = win > 0 ? S + row0 / G - win + 1 : INT_MIN;
    const int lo_last = win > 0 ? S + (min(rows_unit, row0 + 8 * NT) - 1) / G - win + 1 : INT_MIN;
    if (lo_first > k_begin) k_begin += (lo_first - k_begin) / kFewKeys * kFewKeys;
    const int steps = k_end > k_begin ? (k_end - k_begin + kFewKeys - 1) / kFewKeys : 0;

    // rows 8 nt + 2 t + e of this lane's score columns
    uint64_t anc[NT][2];
    int lo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = row0 + 8 * nt + 2 * t + e, node = r / G;
            anc[nt][e] = r < rows_unit ? d.anc[(size_t)b * T + node] : 0ull;
            lo[nt][e] = win > 0 ? S + node - win + 1 : INT_MIN;
        }
    // Q as B operands: group j, step s: features f0 + 8 (s / 2) + 2 (s % 2) + {0, 4} and, divided by 16, + {1, 5} of row
    // 8 nt + g, f0 = 64 j + 16 t: the order in which the masks take a key's 16 codes.  Beside them the rows' sums per
    // group for the biases, times the scores' scale.
    const float qscale = kLog2e * rsqrtf((float)D);
    uint2 qf[NT == 1 ? NG * 4 : 1];
    uint2* q_s = reinterpret_cast<uint2*>(sm + few_smem<D, NT>() - (NT == 1 ? 0 : NG * 4 * NT * 32 * 8));
    float qsum[NG][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + 8 * nt + g;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(d.q[layer]) +
                              ((size_t)(b * T + (r < rows_unit ? r / G : 0)) * d.HQ + kvh * G + (r < rows_unit ? r % G : 0)) * D + 16 * t;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            float x[16], sum = 0.f;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint4 w = r < rows_unit ? *reinterpret_cast<const uint4*>(src + 64 * j + 8 * y) : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    x[8 * y + 2 * z] = bf16_lo(u[z]);
                    x[8 * y + 2 * z + 1] = bf16_hi(u[z]);
                    sum += x[8 * y + 2 * z] + x[8 * y + 2 * z + 1];
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int f = 8 * (s / 2) + 2 * (s % 2);
                const uint2 w = make_uint2(f16x2(x[f], x[f + 4]), f16x2(x[f + 1] * 0.0625f, x[f + 5] * 0.0625f));
                if constexpr (NT == 1) qf[4 * j + s] = w;
                else if (warp == 0) q_s[((4 * j + s) * NT + nt) * 32 + lane] = w;
            }
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);  // row g, on its four lanes
#pragma unroll
            for (int e = 0; e < 2; ++e) qsum[j][nt][e] = qscale * __shfl_sync(0xFFFFFFFFu, sum, 4 * (2 * t + e));
        }
    }
    if constexpr (NT > 1) __syncthreads();

    // ring: this warp's stages
    const size_t seq0 = ((size_t)b * d.HKV + kvh) * (size_t)d.s_cap;
    const char* Kp = reinterpret_cast<const char*>(d.k[layer]) + seq0 * F::row;
    const char* Vp = reinterpret_cast<const char*>(d.v[layer]) + seq0 * F::row;
    const char* KSp = reinterpret_cast<const char*>(d.k_scale[layer]) + seq0 * F::pairs;
    const char* VSp = reinterpret_cast<const char*>(d.v_scale[layer]) + seq0 * F::pairs;
    char* ring = sm + warp * ST * F::bytes;
    const uint32_t ring32 = tc::smem_u32(ring);
    auto fetch = [&](int i, int slot) {  // step warp + 4 i
        const int kt = k_begin + (warp + kFewWarps * i) * kFewKeys;
        if (warp + kFewWarps * i < steps) {
            const uint32_t dst = ring32 + slot * F::bytes;
            constexpr int CPK = F::row / 16;  // chunks per key
#pragma unroll
            for (int x = 0; x < kFewKeys * CPK / 32; ++x) {
                const int key = lane / CPK + x * (32 / CPK), c = lane % CPK;
                const bool real = kt + key < k_end;
                const size_t at = (size_t)(real ? kt + key : k_begin) * F::row + c * 16;
                cp16(dst + F::k + key * F::row + ((c ^ F::k_swizzle(key)) << 4), Kp + at, real);
                cp16(dst + F::v + key * F::row + ((c ^ F::v_swizzle(key)) << 4), Vp + at, real);
            }
            const int key = lane & 15;
            const bool real = kt + key < k_end;
            cp_small<F::pairs>(dst + (lane < 16 ? F::ks : F::vs) + key * F::pairs,
                               (lane < 16 ? KSp : VSp) + (size_t)(real ? kt + key : k_begin) * F::pairs, real);
        }
        cp_commit();
    };

    float m[NT][2], l[NT][2], ob[NG][NT][2];
    float o[NG][4][NT][4];  // [group][tile of 16 features][rows' tile][feature g or g + 8, row 2 t or 2 t + 1]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[nt][e] = -INFINITY;
            l[nt][e] = 0.f;
#pragma unroll
            for (int j = 0; j < NG; ++j) ob[j][nt][e] = 0.f;
        }
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) o[j][i][nt][0] = o[j][i][nt][1] = o[j][i][nt][2] = o[j][i][nt][3] = 0.f;

    uint32_t wide = 0;  // lanes' groups with a scale above 3.9 in the step before: O of such a group is not lifted
    const int mine = steps > warp ? (steps - warp + kFewWarps - 1) / kFewWarps : 0;
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(i, i);
    int slot = 0, ahead = ST - 1;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        cp_wait<ST - 2>();
        __syncwarp();  // everyone's part of this stage is here, and everyone is done with the one before
        fetch(i + ST - 1, ahead);
        const char* st = ring + slot * F::bytes;
        slot = slot + 1 == ST ? 0 : slot + 1;
        ahead = ahead + 1 == ST ? 0 : ahead + 1;
        const int kt = k_begin + (warp + kFewWarps * i) * kFewKeys;

        // scores of keys g, g + 8 and rows 2 t, 2 t + 1, in the log2 domain
        float x[NT][4], bx[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nt][e] = bx[nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
            uint2 w[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int key = g + 8 * half;
                w[half] = *reinterpret_cast<const uint2*>(st + F::k + key * F::row + (((2 * j + (t >> 1)) ^ F::k_swizzle(key)) << 4) + 8 * (t & 1));
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t c0 = y ? w[0].y : w[0].x, c1 = y ? w[1].y : w[1].x;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t a[4] = {c0 & 0x000F000Fu, c1 & 0x000F000Fu, c0 & 0x00F000F0u, c1 & 0x00F000F0u};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint2 q = NT == 1 ? qf[NT == 1 ? 4 * j + 2 * y + s : 0] : q_s[((4 * j + 2 * y + s) * NT + nt) * 32 + lane];
                        mma_16816(acc[nt], a, q.x, q.y);
                    }
                    c0 >>= 8;
                    c1 >>= 8;
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float2 sb = f16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(st + F::ks + (g + 8 * half) * F::pairs + 4 * j));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[nt][2 * half + e] = fmaf(acc[nt][2 * half + e], sb.x, x[nt][2 * half + e]);
                        bx[nt][2 * half + e] = fmaf(sb.y, qsum[j][nt][e], bx[nt][2 * half + e]);
                    }
            }
        }
        const float up = qscale * 16777216.f;  // 2^24
        const bool plain = kt + kFewKeys <= k_end && kt + kFewKeys <= S && kt >= lo_last;
        bool grow = false, large = false;  // large: a scale of this lane's group, lane % NG
        const uint32_t* pairs = reinterpret_cast<const uint32_t*>(st + F::vs);
#pragma unroll
        for (int y = 0; y < (NG > 2 ? NG / 2 : 1); ++y)
            large = large || fabsf(f16x2_to_f32x2(pairs[(lane + 32 * y) & (kFewKeys * NG - 1)]).x) > 3.9f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y = fmaf(x[nt][e], up, bx[nt][e]);
                if (!plain) {
                    const int key = kt + g + 8 * (e >> 1);
                    bool v = key < k_end && key >= lo[nt][e & 1];
                    if (key >= S) v = v && ((anc[nt][e & 1] >> ((key - S) & 63)) & 1ull);
                    y = v ? y : -INFINITY;
                }
                x[nt][e] = y;
                grow = grow || y > m[nt][e & 1] + 2.f;
            }
        // The reference follows a row's maximum only when it is exceeded by more than 2 (p <= 4): then the sums and O are
        // brought to the new one.
        if (__any_sync(0xFFFFFFFFu, grow || large || wide != 0)) {
            const uint32_t now = __ballot_sync(0xFFFFFFFFu, large);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                constexpr uint32_t kLanes = few_lanes<NG>();
                const uint32_t lanes = kLanes << j;
                if (((now & lanes) != 0) != ((wide & lanes) != 0)) {
                    const float f = (now & lanes) != 0 ? 1.f / kFewLift : kFewLift;
#pragma unroll
                    for (int z = 0; z < 4; ++z)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[j][z][nt][e] *= f;
                }
            }
            wide = now;
            if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y = fmaxf(x[nt][e], x[nt][e + 2]);
#pragma unroll
                        for (int z = 4; z < 32; z <<= 1) y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, z));
                        // by the row alone: its result does not depend on its neighbours
                        if (y > m[nt][e] + 2.f) {
                            const float a = tc::ex2_approx(m[nt][e] - y);
                            m[nt][e] = y;
                            l[nt][e] *= a;
#pragma unroll
                            for (int j = 0; j < NG; ++j) {
                                ob[j][nt][e] *= a;
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    o[j][z][nt][e] *= a;
                                    o[j][z][nt][e + 2] *= a;
                                }
                            }
                        }
                    }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // every key masked so far: nothing; a score that is NaN (q is, or left fp16's range) stays NaN
                const float mr = m[nt][e & 1];
                x[nt][e] = tc::ex2_approx(x[nt][e] - (mr == -INFINITY ? 0.f : mr));
            }
        // O^T += V^T P^T
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[nt][e] *= kFewLift;
                l[nt][e & 1] += x[nt][e];
            }
        auto add_values = [&](auto any_wide) {
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                uint32_t p[NT][2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float2 sb = f16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(st + F::vs + (g + 8 * half) * F::pairs + 4 * j));
                    if constexpr (decltype(any_wide)::value) sb.x *= few_unit<NG>(wide, j);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        p[nt][half] = transposed(f16x2(x[nt][2 * half] * sb.x, x[nt][2 * half + 1] * sb.x));
                        ob[j][nt][0] = fmaf(x[nt][2 * half], sb.y, ob[j][nt][0]);
                        ob[j][nt][1] = fmaf(x[nt][2 * half + 1], sb.y, ob[j][nt][1]);
                    }
                }
                // features 64 j + 8 g .. + 7 of keys 2 t, 2 t + 1 (first) and 2 t + 8, 2 t + 9 (second), keys side by side
                uint32_t c[2][2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int key = 2 * t + 8 * half;
                    const char* at = st + F::v + key * F::row + (((2 * j + (g >> 2)) ^ F::v_swizzle(key)) << 4) + 4 * (g & 3);
                    const uint32_t w0 = *reinterpret_cast<const uint32_t*>(at), w1 = *reinterpret_cast<const uint32_t*>(at + F::row);
                    c[half][0] = __byte_perm(w0, w1, 0x5410);
                    c[half][1] = __byte_perm(w0, w1, 0x7632);
                }
#pragma unroll
                for (int z = 0; z < 4; ++z) {  // features 2 z (rows g) and 2 z + 1 (rows g + 8, times 16) of the 8
                    const uint32_t c0 = c[0][z >> 1] >> (8 * (z & 1)), c1 = c[1][z >> 1] >> (8 * (z & 1));
                    const uint32_t a[4] = {c0 & 0x000F000Fu, c0 & 0x00F000F0u, c1 & 0x000F000Fu, c1 & 0x00F000F0u};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816(o[j][z][nt], a, p[nt][0], p[nt][1]);
                }
            }
        };
        if (wide == 0) add_values(std::false_type{});
        else add_values(std::true_type{});
    }
    cp_wait<0>();

    // merge the four warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) {
                l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], z);
#pragma unroll
                for (int j = 0; j < NG; ++j) ob[j][nt][e] += __shfl_xor_sync(0xFFFFFFFFu, ob[j][nt][e], z);
            }
    __shared__ float ml[2][kFewWarps][8 * NT];
    if (g == 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ml[0][warp][8 * nt + 2 * t + e] = m[nt][e];
                ml[1][warp][8 * nt + 2 * t + e] = l[nt][e] / kFewLift;
            }
    __syncthreads();  // and the rings are free
    float* part = reinterpret_cast<float*>(sm);  // [warp][row][D + 4]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * nt + 2 * t + e;
            float top = ml[0][0][r];
#pragma unroll
            for (int w = 1; w < kFewWarps; ++w) top = fmaxf(top, ml[0][w][r]);
            const float f = m[nt][e] == -INFINITY ? 0.f : tc::ex2_approx(m[nt][e] - top) / kFewLift;
            float* dst = part + ((size_t)warp * 8 * NT + r) * (D + 4) + 8 * g;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                float y[8];
                const float unit = 1.f / few_unit<NG>(wide, j);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    y[2 * z] = f * fmaf(o[j][z][nt][e], 16777216.f * unit, ob[j][nt][e]);
                    y[2 * z + 1] = f * fmaf(o[j][z][nt][e + 2], 1048576.f * unit, ob[j][nt][e]);
                }
                *reinterpret_cast<float4*>(dst + 64 * j) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(dst + 64 * j + 4) = make_float4(y[4], y[5], y[6], y[7]);
            }
        }
    __syncthreads();
    constexpr int Q4 = D / 4;
    for (int e = threadIdx.x; e < 8 * NT * Q4; e += kFewWarps * 32) {
        const int r = e / Q4, c = e % Q4 * 4, gr = row0 + r;
        if (gr >= rows_unit) continue;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float4 z = *reinterpret_cast<const float4*>(part + ((size_t)w * 8 * NT + r) * (D + 4) + c);
            y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
        }
        float top = ml[0][0][r], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kFewWarps; ++w) top = fmaxf(top, ml[0][w][r]);
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w)  // no maximum: the sum is 0, or NaN
            sum += ml[0][w][r] == -INFINITY ? ml[1][w][r] : tc::ex2_approx(ml[0][w][r] - top) * ml[1][w][r];
        if (splits == 1) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(d.o[layer]) + ((size_t)(b * T + gr / G) * d.HQ + kvh * G + gr % G) * D + c) =
                make_uint2(bf16x2(y.x * inv, y.y * inv), bf16x2(y.z * inv, y.w * inv));
        } else {
            const size_t at = ((size_t)unit * splits + split) * rows_unit + gr;
            *reinterpret_cast<float4*>(ws_o + at * D + c) = y;
            if (c == 0) {
                ws_ml[2 * at] = top;
                ws_ml[2 * at + 1] = sum;
            }
        }
    }
}

// Rows of one CTA's tile: one MMA column tile of 8 or two.
int few_rows(const tsv_attn_desc* d) { return (d->HQ / d->HKV) * d->T <= 8 ? 8 : 16; }

template <int D, int NT>
static void launch_few_nt(const tsv_attn_desc* d, int splits, int chunk, float* ws_o, float* ws_ml, int32_t* status, cudaStream_t stream) {
    constexpr int sm = few_smem<D, NT>();
    cudaFuncSetAttribute(attn_few_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
    const int rows = (d->HQ / d->HKV) * d->T;
    const dim3 grid(splits, (rows + 8 * NT - 1) / (8 * NT), d->n_layers * d->B * d->HKV);
    launch_pdl(attn_few_kernel<D, NT>, grid, kFewWarps * 32, sm, stream, *d, splits, chunk, ws_o, ws_ml, status);
}

void launch_few(const tsv_attn_desc* d, int splits, int chunk, float* ws_o, float* ws_ml, int32_t* status, cudaStream_t stream) {
    const bool one = few_rows(d) == 8;
    if (d->D == 256) one ? launch_few_nt<256, 1>(d, splits, chunk, ws_o, ws_ml, status, stream) : launch_few_nt<256, 2>(d, splits, chunk, ws_o, ws_ml, status, stream);
    else if (d->D == 128) one ? launch_few_nt<128, 1>(d, splits, chunk, ws_o, ws_ml, status, stream) : launch_few_nt<128, 2>(d, splits, chunk, ws_o, ws_ml, status, stream);
    else one ? launch_few_nt<64, 1>(d, splits, chunk, ws_o, ws_ml, status, stream) : launch_few_nt<64, 2>(d, splits, chunk, ws_o, ws_ml, status, stream);
}

}  // namespace tsv
