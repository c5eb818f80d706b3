// tsv_token_logprobs: log probability and rank of a given token, entropy and the likeliest tokens of every row of logits.
//
//   z = logits / T;  logp(t) = z_t - log sum exp z;  entropy = log sum exp z - sum p z
//
// Bound by HBM: every logit is read once.  A CTA walks a part of a row in tiles of 4096 logits, 16 in a thread's registers; a
// row is one part where there are rows enough to fill the GPU, else up to 64, whose results a second kernel joins (one warp per
// row).  Sums are kept per thread against the thread's own running maximum (rescaled when it rises) and joined at the end, in the
// same order in every run.
//
// The top k are exact.  The k-th largest of the 256 threads' maxima over the first tile is a bound below which no logit of the top k
// lies, and at most k threads hold anything above it: at most 16 k candidates go to shared memory.  From then on a logit is a
// candidate if it is larger than the k-th best known, which few are; the list is cut back to k whenever it might overflow, and
// a tile in which too many logits still qualify (an ascending row) is bounded like the first one.  Candidates are 64-bit keys (value, then
// lower index), so ties need no care.
#include <algorithm>

#include "e4m3.cuh"
#include "tc.cuh"

namespace tsv {

constexpr int kLpThreads = 256;
constexpr int kLpPer = 16;                       // logits per thread and tile
constexpr int kLpTile = kLpThreads * kLpPer;
constexpr int kLpMaxTop = 64;
constexpr int kLpMaxParts = 64;
constexpr int kLpList = 2048;                    // candidates; 16 x 64 + 64 at least
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LogprobParams {
    const void* logits;
    const int32_t* targets;
    int rows, V, K, parts;
    float inv_t;
    float *logp, *entropy, *top_logp;
    int32_t *rank, *top_tokens;
    float4* part_sums;               // [rows][parts]: maximum, sum, weighted sum, tokens ahead of the target (bits)
    unsigned long long* part_top;    // [rows][parts][K]
};

// What is known of some of a row's logits: their maximum m, the sum of 2^d and of d 2^d with d = (x - m) log2(e) / T, and how
// many rank ahead of the target.
struct Sums {
    float m, s, w;
    int ahead;
};

__device__ __forceinline__ Sums joined(Sums a, Sums b, float c) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, a.s + b.s, a.w + b.w, a.ahead + b.ahead};  // nothing but -infinity (or NaN, which s keeps)
    const float da = fmaxf((a.m - m) * c, -1000.f), db = fmaxf((b.m - m) * c, -1000.f);
    const float fa = tc::ex2_approx(da), fb = tc::ex2_approx(db);
    return {m, fmaf(a.s, fa, b.s * fb), fmaf(a.w + a.s * da, fa, (b.w + b.s * db) * fb), a.ahead + b.ahead};
}

__device__ __forceinline__ Sums joined_warp(Sums v, float c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Sums u = {__shfl_xor_sync(0xFFFFFFFFu, v.m, o), __shfl_xor_sync(0xFFFFFFFFu, v.s, o),
                        __shfl_xor_sync(0xFFFFFFFFu, v.w, o), __shfl_xor_sync(0xFFFFFFFFu, v.ahead, o)};
        v = (threadIdx.x & o) ? joined(u, v, c) : joined(v, u, c);  // both lanes add in the same order
    }
    return v;
}

__device__ __forceinline__ int power_of_two(int n) { return 1 << (32 - __clz(n - 1)); }  // at least n >= 1

// Sorts n keys (a power of two) in shared memory, largest first; the whole CTA.
__device__ __forceinline__ void sort_keys(unsigned long long* key, int n) {
    for (int size = 2; size <= n; size <<= 1)
        for (int step = size >> 1; step > 0; step >>= 1) {
            for (int e = threadIdx.x; e < n / 2; e += kLpThreads) {
                const int i = ((e & ~(step - 1)) << 1) | (e & (step - 1)), j = i | step;
                const unsigned long long a = key[i], b = key[j];
                if ((a < b) == ((i & size) == 0)) key[i] = b, key[j] = a;
            }
            __syncthreads();
        }
}

// 16 bytes of logits as fp32.
template <typename T>
__device__ __forceinline__ void unpack16(uint4 u, float* x) {
    if constexpr (sizeof(T) == 4) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    } else {
        RowType<T>::unpack(u.x, x[0], x[1]);
        RowType<T>::unpack(u.y, x[2], x[3]);
        RowType<T>::unpack(u.z, x[4], x[5]);
        RowType<T>::unpack(u.w, x[6], x[7]);
    }
}

// + 0 turns -0 into 0, which is no smaller a logit.
__device__ __forceinline__ unsigned long long logit_key(float x, int i) { return pack_best(x + 0.f, (uint32_t)i); }
__device__ __forceinline__ int key_token(unsigned long long k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }
__device__ __forceinline__ float key_logit(unsigned long long k) { return unorderable((uint32_t)(k >> 32)); }

// A row's numbers, by one thread; NaN and -1 where the row has no distribution.  Returns log sum exp((x - m) / T), or NaN.
__device__ __forceinline__ float row_results(const LogprobParams& p, size_t row, Sums v, int target, float t) {
    const bool bad = !(v.s < INFINITY) || v.m == -INFINITY, has = target >= 0 && target < p.V;
    const float nan = __int_as_float(0x7FFFFFFF), lse = bad ? nan : logf(v.s);
    if (p.logp) p.logp[row] = bad || !has ? nan : (t - v.m) * p.inv_t - lse;
    if (p.rank) p.rank[row] = bad || !has ? -1 : v.ahead;
    if (p.entropy) p.entropy[row] = bad ? nan : lse - kLn2 * v.w / v.s;
    return lse;
}

template <typename T>
__device__ __forceinline__ float target_logit(const LogprobParams& p, size_t row, int target) {
    return target >= 0 && target < p.V ? RowType<T>::to_f32(((const T*)p.logits)[row * p.V + target]) : 0.f;
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_kernel(const LogprobParams p) {
    griddep_begin();
    constexpr int W = 16 / sizeof(T), NV = kLpPer / W;
    __shared__ unsigned long long list[kLpList], maxima[kLpThreads];
    __shared__ Sums warps[kLpThreads / 32];
    __shared__ int filled;
    const int tid = threadIdx.x, lane = tid & 31, K = p.K;
    const size_t row = blockIdx.x / p.parts;
    const int part = blockIdx.x - (int)row * p.parts;
    const T* x0 = (const T*)p.logits + row * p.V;
    // a row may start anywhere: tiles are counted from the 16-byte boundary at or before its start
    const int lead = (int)(((uintptr_t)x0 & 15) / sizeof(T));
    const int tiles = (int)(((long long)p.V + lead + kLpTile - 1) / kLpTile);
    const int t0 = (int)((long long)tiles * part / p.parts), t1 = (int)((long long)tiles * (part + 1) / p.parts);
    const float c = p.inv_t * kLog2e;
    const int target = p.targets ? p.targets[row] : -1;
    const float t = target_logit<T>(p, row, target);
    const bool ranked = p.rank && target >= 0 && target < p.V;
    // a logit before the target ranks ahead if it is larger than `below`, the next number under t: an equal one does
    const float below = nextafterf(t, -INFINITY);

    Sums v = {-INFINITY, 0.f, 0.f, 0};
    float kth = -INFINITY;   // the k-th best of the list when it was last cut back
    int room_used = 0;       // an upper bound of `filled`, the same in every thread
    if (tid == 0) filled = 0;
    for (int tile = t0; tile < t1; ++tile) {
        float x[kLpPer];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = tile * kLpTile + (j * kLpThreads + tid) * W - lead;
            if (i >= 0 && i + W <= p.V) {
                unpack16<T>(ldg_stream16(x0 + i), x + j * W);
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) x[j * W + k] = i + k >= 0 && i + k < p.V ? RowType<T>::to_f32(x0[i + k]) : -INFINITY;
            }
        }
        float most = x[0];
#pragma unroll
        for (int k = 1; k < kLpPer; ++k) most = fmaxf(most, x[k]);
        if (most > v.m) {
            if (v.m > -INFINITY) {
                const float d = fmaxf((v.m - most) * c, -1000.f), f = tc::ex2_approx(d);
                v.w = (v.w + v.s * d) * f;
                v.s *= f;
            }
            v.m = most;
        }
        const float m = v.m > -INFINITY ? v.m : 0.f;
#pragma unroll
        for (int k = 0; k < kLpPer; ++k) {
            const float d = (x[k] - m) * c, e = tc::ex2_approx(d);
            v.s += e;                              // a NaN stays
            v.w = fmaf(e, fmaxf(d, -1000.f), v.w);  // 0 for -infinity
        }
        if (ranked) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = tile * kLpTile + (j * kLpThreads + tid) * W - lead;
                if (i + W <= target || i > target) {
                    const float over = i > target ? t : below;
                    if (t > -INFINITY || i > target) {
#pragma unroll
                        for (int k = 0; k < W; ++k) v.ahead += x[j * W + k] > over;
                    } else {
                        v.ahead += W - max(0, -i);  // every logit is at least -infinity
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        v.ahead += i + k >= 0 && i + k < p.V && (x[j * W + k] > t || (x[j * W + k] == t && i + k < target));
                }
            }
        }
        if (K == 0) continue;
        // ---- the top k
        auto index = [&](int k) { return tile * kLpTile + ((k / W) * kLpThreads + tid) * W + k % W - lead; };
        auto append = [&](auto&& wanted) {
#pragma unroll
            for (int k = 0; k < kLpPer; ++k) {
                const int i = index(k);
                if (i >= 0 && i < p.V && wanted(x[k], i)) {
                    const int at = atomicAdd(&filled, 1);
                    if (at < kLpList) list[at] = logit_key(x[k], i);  // more than that only where NaNs are, whose row has no top k
                }
            }
        };
        auto cut = [&] {  // the list back to its best K, sorted
            __syncthreads();
            const int have = min(filled, kLpList);
            const int n = power_of_two(max(have, K));
            for (int e = have + tid; e < n; e += kLpThreads) list[e] = 0ull;
            __syncthreads();
            sort_keys(list, n);
            if (tid == 0) filled = min(have, K);
            room_used = min(have, K);
            if (have >= K) kth = key_logit(list[K - 1]);
            __syncthreads();
        };
        bool all_above = tile == t0;
        if (!all_above) {
            int holders = __syncthreads_count(most > kth);
            if (room_used + holders * kLpPer > kLpList) {
                cut();
                holders = __syncthreads_count(most > kth);
                all_above = room_used + holders * kLpPer > kLpList;
            }
            if (!all_above) {
                room_used += holders * kLpPer;
                if (most > kth) append([&](float y, int) { return y > kth; });
            }
        }
        if (all_above) {
            unsigned long long mine = 0ull;
#pragma unroll
            for (int k = 0; k < kLpPer; ++k) {
                const int i = index(k);
                if (i >= 0 && i < p.V && x[k] == x[k]) mine = max(mine, logit_key(x[k], i));
            }
            __syncthreads();
            maxima[tid] = mine;
            __syncthreads();
            sort_keys(maxima, kLpThreads);
            const unsigned long long bound = maxima[K - 1];
            room_used += K * kLpPer;
            if (mine >= bound) append([&](float y, int i) { return logit_key(y, i) >= bound && y >= kth; });
            cut();
        }
    }
    // ---- the part's results
    v = joined_warp(v, c);
    if (lane == 0) warps[tid >> 5] = v;
    __syncthreads();
    v = warps[0];
#pragma unroll
    for (int w = 1; w < kLpThreads / 32; ++w) v = joined(v, warps[w], c);
    if (K > 0) {
        __syncthreads();
        const int have = min(filled, kLpList);
        const int n = power_of_two(max(have, K));
        for (int e = have + tid; e < n; e += kLpThreads) list[e] = 0ull;
        __syncthreads();
        sort_keys(list, n);
    }
    if (p.parts > 1) {
        if (tid == 0) p.part_sums[blockIdx.x] = make_float4(v.m, v.s, v.w, __int_as_float(v.ahead));
        for (int k = tid; k < K; k += kLpThreads) p.part_top[(size_t)blockIdx.x * K + k] = list[k];
        return;
    }
    const bool bad = !(v.s < INFINITY) || v.m == -INFINITY;
    const float nan = __int_as_float(0x7FFFFFFF), lse = bad ? nan : logf(v.s);
    if (tid == 0) row_results(p, row, v, target, t);
    for (int k = tid; k < K; k += kLpThreads) {
        p.top_tokens[row * K + k] = bad ? -1 : key_token(list[k]);
        p.top_logp[row * K + k] = bad ? nan : (key_logit(list[k]) - v.m) * p.inv_t - lse;
    }
}

// Largest 64-bit key of the warp (keys are unique, but for 0).
__device__ __forceinline__ unsigned long long warp_largest(unsigned long long k) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((unsigned long long)hi << 32) | lo;
}

// One warp per row joins its parts: the sums in the parts' order, the sorted lists by taking the largest head K times.  A lane
// holds the parts `lane` and `lane + 32`.
template <typename T>
__global__ void __launch_bounds__(128) logprobs_join_kernel(const LogprobParams p) {
    griddep_begin();
    const int lane = threadIdx.x & 31;
    const size_t row = (size_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const float c = p.inv_t * kLog2e;
    Sums v = {-INFINITY, 0.f, 0.f, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (lane + h * 32 < p.parts) {
            const float4 f = p.part_sums[row * p.parts + lane + h * 32];
            const Sums u = {f.x, f.y, f.z, __float_as_int(f.w)};
            v = h ? joined(v, u, c) : u;
        }
    v = joined_warp(v, c);
    const bool bad = !(v.s < INFINITY) || v.m == -INFINITY;
    const float nan = __int_as_float(0x7FFFFFFF), lse = bad ? nan : logf(v.s);
    if (lane == 0) {
        const int target = p.targets ? p.targets[row] : -1;
        row_results(p, row, v, target, target_logit<T>(p, row, target));
    }
    const unsigned long long* tops = p.part_top + row * p.parts * p.K;
    int at[2] = {0, 0};
    unsigned long long head[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) head[h] = p.K > 0 && lane + h * 32 < p.parts ? tops[(size_t)(lane + h * 32) * p.K] : 0ull;
    for (int k = 0; k < p.K; ++k) {
        const unsigned long long best = warp_largest(max(head[0], head[1]));
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (head[h] == best && best != 0ull) head[h] = ++at[h] < p.K ? tops[(size_t)(lane + h * 32) * p.K + at[h]] : 0ull;
        if (lane == 0) {
            p.top_tokens[row * p.K + k] = bad ? -1 : key_token(best);
            p.top_logp[row * p.K + k] = bad ? nan : (key_logit(best) - v.m) * p.inv_t - lse;
        }
    }
}

// Parts of a row: enough CTAs for eight per SM, a tile at least in each.
static int logprob_parts(int rows, int V) {
    const int tiles = (V + kLpTile - 1) / kLpTile, want = (int)(((long long)sm_count() * 4 + rows - 1) / rows);
    return std::max(1, std::min({want, tiles, kLpMaxParts}));
}

template <typename T>
static void launch_logprobs(const LogprobParams& p, cudaStream_t stream) {
    launch_pdl(logprobs_kernel<T>, p.rows * p.parts, kLpThreads, 0, stream, p);
    if (p.parts > 1) launch_pdl(logprobs_join_kernel<T>, (p.rows + 3) / 4, 128, 0, stream, p);
}

}  // namespace tsv

extern "C" size_t tsv_token_logprobs_workspace_size(int32_t rows, int32_t V, int32_t top_k) {
    using namespace tsv;
    if (rows < 1 || V < 1 || top_k < 0 || top_k > kLpMaxTop) return 0;
    const size_t parts = logprob_parts(rows, V);
    return parts > 1 ? (rows * parts * (16 + 8 * (size_t)top_k) + 255) & ~(size_t)255 : 0;
}

extern "C" tsv_status tsv_token_logprobs(const void* logits, int32_t logits_dtype, int32_t rows, int32_t V,
                                         const int32_t* targets, float temperature, int32_t top_k, float* logp, int32_t* rank,
                                         float* entropy, int32_t* top_tokens, float* top_logp, void* workspace,
                                         size_t ws_bytes, cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    if (rows < 0 || V < 1 || V > (1 << 24)) return fail(TSV_EINVAL, "token_logprobs: rows=%d V=%d (1 .. 2^24)", rows, V);
    if (logits_dtype != TSV_F32 && logits_dtype != TSV_BF16 && logits_dtype != TSV_F16)
        return fail(TSV_EUNSUPPORTED, "token_logprobs: logits of type %d (fp32, bf16 or fp16 only)", logits_dtype);
    if (top_k < 0 || top_k > kLpMaxTop || top_k > V)
        return fail(TSV_EUNSUPPORTED, "token_logprobs: top_k=%d outside [0, min(%d, V)]", top_k, kLpMaxTop);
    if (!(temperature >= 1e-6f && temperature <= 1e6f))
        return fail(TSV_EINVAL, "token_logprobs: temperature=%g outside [1e-6, 1e6]", temperature);
    if (rows == 0) return TSV_OK;
    if (!logits) return fail(TSV_EINVAL, "token_logprobs: null pointer argument");
    if ((targets != nullptr) != (logp != nullptr) || (rank && !targets))
        return fail(TSV_EINVAL, "token_logprobs: targets and logp belong together, and rank needs them");
    if (top_k > 0 && (!top_tokens || !top_logp)) return fail(TSV_EINVAL, "token_logprobs: top_k=%d without top_tokens and top_logp", top_k);
    if (top_k == 0 && (top_tokens || top_logp)) return fail(TSV_EINVAL, "token_logprobs: top_tokens or top_logp with top_k=0");
    if (!logp && !entropy && !top_k) return fail(TSV_EINVAL, "token_logprobs: no output");
    if ((uintptr_t)logits & (logits_dtype == TSV_F32 ? 3 : 1)) return fail(TSV_EINVAL, "token_logprobs: logits not aligned to their elements");
    const size_t need = tsv_token_logprobs_workspace_size(rows, V, top_k);
    if (need && !workspace) return fail(TSV_EINVAL, "token_logprobs: null workspace");
    if ((uintptr_t)workspace & 15) return fail(TSV_EINVAL, "token_logprobs: workspace not 16-byte aligned");
    if (ws_bytes < need) return fail(TSV_ECAPACITY, "token_logprobs: workspace %zu < %zu bytes", ws_bytes, need);
    if ((long long)rows * logprob_parts(rows, V) > INT_MAX) return fail(TSV_ECAPACITY, "token_logprobs: rows=%d", rows);
    LogprobParams p = {logits, targets, rows, V, top_k, logprob_parts(rows, V), 1.f / temperature, logp, entropy, top_logp, rank, top_tokens};
    p.part_sums = (float4*)workspace;
    p.part_top = (unsigned long long*)(p.part_sums + (size_t)rows * p.parts);
    if (logits_dtype == TSV_F32) launch_logprobs<float>(p, stream);
    else if (logits_dtype == TSV_BF16) launch_logprobs<__nv_bfloat16>(p, stream);
    else launch_logprobs<__half>(p, stream);
    return check_launch("token_logprobs");
}
