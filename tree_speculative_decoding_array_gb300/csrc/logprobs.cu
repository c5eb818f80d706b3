// tsv_token_logprobs: log probability and rank of a given token, entropy and the likeliest tokens of every row of logits.
//
//   z = logits / T;  logp(t) = z_t - log sum exp z;  entropy = log sum exp z - sum p z
//
// Bound by HBM: every logit is read once.  A CTA walks a part of a row in tiles of 4096 logits, 16 in a thread's registers; a
// row is one part where there are rows enough to fill the GPU, else up to 64, whose results a second kernel joins.  Sums are kept
// per thread against the thread's own maximum so far (the sums are rescaled when it rises) and joined at the
// end, in the same order in every run.
//
// The top k are exact.  Logits above a bound that k logits are known to reach go to a list in shared memory: in the first tile the
// bound is the smallest over the 8 warps of each one's ceil(k / 8)-th largest thread maximum (where there are too few, the k-th largest
// of all 256), then the k-th best of the list as it was cut last.  The list is looked at between groups of 1, 2, 6, 16, 16 ... tiles (no
// barrier inside a group: one per tile cost a third of the time), and cut back to k where more than k + k / 2 stand in it.  Of logits in no
// particular order a few hundred pass.  Where a group's do not fit (an ascending row, many equal ones), what stood in the list ahead
// of it is kept and its tiles are read again, each bounded by the k-th largest of the 256 threads' maxima, above which no more
// than 16 k logits can lie.  Candidates are 64-bit keys (value, then lower index), so ties need no care.
//
// 2048 rows of 248320 with ranks of likely tokens: fp32 338 us with 20 alternatives (0.89 of HBM), 304 without; bf16 286 and 222, of
// random tokens 304 and 227, 14 to 17 instructions per logit at 76 % of the issue slots.  -infinity as any other logit: 2 % of them
// masked 340 us in fp32 (393 where a tile that has one was summed again).
#include <algorithm>

#include "e4m3.cuh"
#include "tc.cuh"

namespace tsv {

constexpr int kLpThreads = 256;
constexpr int kLpPer = 16;                       // logits per thread and tile
constexpr int kLpTile = kLpThreads * kLpPer;
constexpr int kLpMaxTop = 64;
constexpr int kLpMaxParts = 64;
constexpr int kLpList = 2048;                    // candidates; 16 x 64 + 96 at least
constexpr int kLpGroup = 16;                     // tiles between two looks at the list
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// CTAs resident on an SM, and whether a thread asks for its next tile before it works on this one.  16-bit logits, whose tiles are 8
// registers: four CTAs that look ahead (2048 rows of 248320, an earlier build: 292 us, five without 328); fp32, near HBM's rate as it is:
// five (346; four that look ahead 401).
template <typename T>
struct LpShape {
    static constexpr bool kAhead = sizeof(T) == 2;
    static constexpr int kPerSm = kAhead ? 4 : 5;
};

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

// What is known of some of a row's logits x: their maximum m, the sums of 2^d and of d 2^d with d = (x - m) c, c = log2(e) / T, and
// how many rank ahead of the target.  (x - m) c in two steps, not x c - m c in one: a rounded m c would shift every d of a thread alike,
// and overflow where a mask's lowest value is all there is.
struct Sums {
    float m, s, w;
    int ahead;
};

// Two fp32 numbers in one register pair, and operations on both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float first_of(uint64_t p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float second_of(uint64_t p) { return __uint_as_float((uint32_t)(p >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// At least -1000, whose power of two is 0 as -infinity's is, but whose product with it is a number; a NaN stays.
__device__ __forceinline__ float clamped(float d) {
    float r;
    asm("max.NaN.f32 %0, %1, 0fC47A0000;" : "=f"(r) : "f"(d));
    return r;
}

// 1 where a > b, else 0.
__device__ __forceinline__ float larger(float a, float b) {
    float r;
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

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

// Sorts n keys (a power of two) in shared memory, largest first.  A barrier follows.
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

// The best K of 0 to 256 keys, no two alike, to the front, largest first, and 0 where there are fewer: each key's place is how many
// are larger, counted by as many neighbouring lanes as there are threads for it.  (Sorting 64 keys took one warp 4600 SM clocks.)
__device__ __forceinline__ void place_keys(unsigned long long* key, int have, int K) {
    const int lanes = min(32, kLpThreads / power_of_two(max(have, 1))), e = threadIdx.x / lanes;
    const unsigned long long mine = e < have ? key[e] : 0ull;
    int larger = 0;
    if (e < have)
#pragma unroll 4
        for (int j = threadIdx.x & (lanes - 1); j < have; j += lanes) larger += key[j] > mine;
    for (int o = lanes >> 1; o > 0; o >>= 1) larger += __shfl_xor_sync(0xFFFFFFFFu, larger, o);
    __syncthreads();
    if (e < have && larger < K) key[larger] = mine;  // the same from all of the key's lanes
    if (threadIdx.x >= have && threadIdx.x < K) key[threadIdx.x] = 0ull;
    __syncthreads();
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

// A row's results, once its sums are known.
struct RowResults {
    bool bad;         // a NaN or +infinity, or nothing but -infinity: no distribution
    float inv_t, m, lse;  // 1 / T, the largest logit, log sum exp((x - m) / T)
    __device__ __forceinline__ RowResults(Sums v, float inv_t)
        : bad(!(v.s < INFINITY) || v.m == -INFINITY), inv_t(inv_t), m(v.m), lse(bad ? 0.f : logf(v.s)) {}
    __device__ __forceinline__ float logp(float x) const { return bad ? __int_as_float(0x7FFFFFFF) : (x - m) * inv_t - lse; }
    // by one thread
    __device__ __forceinline__ void write(const LogprobParams& p, size_t row, Sums v, int target, float t) const {
        const bool has = target >= 0 && target < p.V;
        const float nan = __int_as_float(0x7FFFFFFF);
        if (p.logp) p.logp[row] = has ? logp(t) : nan;
        if (p.rank) p.rank[row] = bad || !has ? -1 : v.ahead;
        if (p.entropy) p.entropy[row] = bad ? nan : lse - kLn2 * v.w / v.s;
    }
    __device__ __forceinline__ void write_top(const LogprobParams& p, size_t row, int k, unsigned long long key) const {
        p.top_tokens[row * p.K + k] = bad ? -1 : key_token(key);
        p.top_logp[row * p.K + k] = logp(key_logit(key));
    }
};

template <typename T>
__device__ __forceinline__ float target_logit(const LogprobParams& p, size_t row, int target) {
    return target >= 0 && target < p.V ? RowType<T>::to_f32(((const T*)p.logits)[row * p.V + target]) : 0.f;
}

// A thread's 16 logits of a tile as they come from memory.
template <typename T>
struct RawTile {
    static constexpr int W = 16 / sizeof(T), NV = kLpPer / W;
    uint4 u[NV];
    __device__ __forceinline__ void load(const T* x0, int at) {
#pragma unroll
        for (int j = 0; j < NV; ++j) u[j] = ldg_stream16(x0 + at + j * kLpThreads * W);
    }
};

// As numbers, -infinity where the row has none.  inside: `raw` holds them.
template <typename T>
__device__ __forceinline__ void load_tile(const T* x0, int at, int V, bool inside, const RawTile<T>& raw, float (&x)[kLpPer]) {
    constexpr int W = 16 / sizeof(T), NV = kLpPer / W;
    if (inside) {
#pragma unroll
        for (int j = 0; j < NV; ++j) unpack16<T>(raw.u[j], x + j * W);
        return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const int i = at + j * kLpThreads * W + k;
            x[j * W + k] = i >= 0 && i < V ? RowType<T>::to_f32(x0[i]) : -INFINITY;
        }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, LpShape<T>::kPerSm) logprobs_kernel(const LogprobParams p) {
    griddep_begin();
    constexpr int W = 16 / sizeof(T);
    __shared__ unsigned long long list[kLpList], maxima[kLpThreads];
    __shared__ Sums warps[kLpThreads / 32];
    __shared__ float bounds[kLpThreads / 32];
    __shared__ int filled;
    __shared__ int stood;  // of the list's candidates, those of earlier groups of tiles: kept ones, and uncut ones behind them (thread 0's alone)
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
    // a logit ahead of the target outranks it if it is larger than `below`, the next number under t: an equal one does
    const float below = nextafterf(t, -INFINITY);

    // element k of this thread's 16 in a tile is logit first(tile) + (k / W) * 256 W + k % W
    auto first = [&](int tile) { return tile * kLpTile + tid * W - lead; };
    auto inside = [&](int tile) { return tile * kLpTile >= lead && (tile + 1) * kLpTile - lead <= p.V; };
    // candidates among a thread's 16
    auto append = [&](const float (&x)[kLpPer], int at, auto&& wanted) {
        uint32_t mask = 0u;
#pragma unroll
        for (int k = 0; k < kLpPer; ++k) mask |= wanted(x[k], at + (k / W) * kLpThreads * W + k % W) ? 1u << k : 0u;
        while (mask) {
            const int k = __ffs(mask) - 1, i = at + (k / W) * kLpThreads * W + k % W;
            mask &= mask - 1;
            if (i < 0 || i >= p.V) continue;
            float y = x[0];
#pragma unroll
            for (int j = 1; j < kLpPer; ++j) y = j == k ? x[j] : y;
            const int to = atomicAdd(&filled, 1);
            if (to < kLpList) list[to] = logit_key(y, i);
        }
    };
    Sums v = {-INFINITY, 0.f, 0.f, 0};
    float kth = -INFINITY;  // what a logit has to exceed to be a candidate; in the first tile, to reach
    int kept = 0;           // candidates that stood in the list, sorted, after the last cut
    if (tid == 0) filled = stood = 0;
    auto cut = [&](int have) {  // the list's `have` candidates back to the best K, sorted; after a barrier
        if (have <= kLpThreads) {
            place_keys(list, have, K);
        } else {
            const int n = power_of_two(have);
            for (int e = have + tid; e < n; e += kLpThreads) list[e] = 0ull;
            __syncthreads();
            sort_keys(list, n);
        }
        kept = min(have, K);
        if (tid == 0) filled = stood = kept;
        if (have >= K) kth = key_logit(list[K - 1]);
        __syncthreads();
    };
    // Candidates of a tile by the K-th largest of the threads' maxima; the whole CTA.
    auto append_bounded = [&](const float (&x)[kLpPer], int at) {
        unsigned long long mine = tid;  // below every logit's key, and no two alike
#pragma unroll
        for (int k = 0; k < kLpPer; ++k) {
            const int i = at + (k / W) * kLpThreads * W + k % W;
            if (i >= 0 && i < p.V && x[k] == x[k]) mine = max(mine, logit_key(x[k], i));
        }
        // the threads that have a logit; up to K of them hold no more than the list takes
        const int left = p.V - at + tid * W, holders = min(kLpThreads, (left + W - 1) / W);
        unsigned long long bound = 0ull;
        if (holders > K) {
            maxima[tid] = mine;
            __syncthreads();
            place_keys(maxima, holders, K);
            bound = maxima[K - 1];
        }
        if (mine >= bound) append(x, at, [&](float y, int i) { return logit_key(y, i) >= bound; });
    };
    RawTile<T> raw;
    if (LpShape<T>::kAhead && inside(t0)) raw.load(x0, first(t0));
    for (int next = t0, group = 1; next < t1;) {
        const int end = min(t1, next + group);
        for (int tile = next; tile < end; ++tile) {
            float x[kLpPer];
            const int at = first(tile);
            if (!LpShape<T>::kAhead && inside(tile)) raw.load(x0, at);
            load_tile<T>(x0, at, p.V, inside(tile), raw, x);
            if (LpShape<T>::kAhead && tile + 1 < t1 && inside(tile + 1)) raw.load(x0, first(tile + 1));
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
            // two logits at a time; a NaN stays in both sums
            uint64_t s2 = 0ull, w2 = 0ull;
            const uint64_t less = pair(-m, -m), scale = pair(c, c);
#pragma unroll
            for (int k = 0; k < kLpPer; k += 2) {
                const uint64_t d = mul2(add2(pair(x[k], x[k + 1]), less), scale);
                const float da = clamped(first_of(d)), db = clamped(second_of(d));
                const uint64_t e = pair(tc::ex2_approx(da), tc::ex2_approx(db));
                s2 = add2(s2, e);
                w2 = fma2(e, pair(da, db), w2);
            }
            const float w = first_of(w2) + second_of(w2);
            v.s += first_of(s2) + second_of(s2);
            v.w += w;
            if (ranked) {
                const bool after = tile * kLpTile - lead > target, before = (tile + 1) * kLpTile - lead <= target;
                if (before && t == -INFINITY && inside(tile)) {
                    v.ahead += kLpPer;
                } else if (after || (before && t > -INFINITY)) {
                    const float over = after ? t : below;
                    if (most > over) {
                        uint64_t n2 = 0ull;  // in fp32: a comparison gives 1 or 0 in one instruction
#pragma unroll
                        for (int k = 0; k < kLpPer; k += 2) n2 = add2(n2, pair(larger(x[k], over), larger(x[k + 1], over)));
                        v.ahead += (int)(first_of(n2) + second_of(n2));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kLpPer; ++k) {
                        const int i = at + (k / W) * kLpThreads * W + k % W;
                        v.ahead += i >= 0 && i < p.V && (x[k] > t || (x[k] == t && i < target));
                    }
                }
            }
            if (K == 0) continue;
            if (tile == t0) {
                uint32_t m = orderable(most), q = 0u;
                for (int n = 0; n < (K + kLpThreads / 32 - 1) / (kLpThreads / 32); ++n) {
                    q = __reduce_max_sync(0xFFFFFFFFu, m);
                    if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, m == q)) - 1) m = 0u;
                }
                if (lane == 0) bounds[tid >> 5] = q > 0u ? unorderable(q) : -INFINITY;
                __syncthreads();
                float bound = bounds[0];
#pragma unroll
                for (int w = 1; w < kLpThreads / 32; ++w) bound = fminf(bound, bounds[w]);
                if (bound == -INFINITY) append_bounded(x, at);  // threads without a logit, or masked ones
                else if (most >= bound) append(x, at, [&](float y, int) { return y >= bound; });
            } else if (most > kth) {
                append(x, at, [&](float y, int) { return y > kth; });
            }
        }
        if (K > 0) {
            __syncthreads();
            const int have = filled;
            __syncthreads();
            if (have > kLpList) {
                if (tid == 0) filled = stood;  // these are still there: a group's candidates go behind them
                for (int tile = next; tile < end; ++tile) {
                    float x[kLpPer];
                    const int at = first(tile);
                    RawTile<T> again;
                    if (inside(tile)) again.load(x0, at);
                    load_tile<T>(x0, at, p.V, inside(tile), again, x);
                    append_bounded(x, at);
                    __syncthreads();
                    cut(min(filled, kLpList));  // beyond the list only where NaNs are, and such a row has no top k
                }
            } else if (next == t0 || have > K + K / 2) {
                cut(have);
            } else if (tid == 0) {
                stood = have;
            }
        }
        group = next == t0 ? 2 : min(kLpGroup, 3 * group);
        next = end;
    }
    // ---- the part's results
    v = joined_warp(v, c);
    if (lane == 0) warps[tid >> 5] = v;
    __syncthreads();
    v = warps[0];
#pragma unroll
    for (int w = 1; w < kLpThreads / 32; ++w) v = joined(v, warps[w], c);
    if (K > 0 && filled > kept) {  // the same in every thread: the last appends lie behind barriers
        const int have = filled;
        __syncthreads();
        cut(have);
    }
    if (p.parts > 1) {
        if (tid == 0) p.part_sums[blockIdx.x] = make_float4(v.m, v.s, v.w, __int_as_float(v.ahead));
        for (int k = tid; k < K; k += kLpThreads) p.part_top[(size_t)blockIdx.x * K + k] = list[k];
        return;
    }
    const RowResults res(v, p.inv_t);
    if (tid == 0) res.write(p, row, v, target, t);
    for (int k = tid; k < K; k += kLpThreads) res.write_top(p, row, k, list[k]);
}

// Largest 64-bit key of the warp (keys are unique, but for 0).
__device__ __forceinline__ unsigned long long warp_largest(unsigned long long k) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((unsigned long long)hi << 32) | lo;
}

// A CTA per row joins its parts: the sums in the parts' order, the sorted lists (brought to shared memory first) by taking the
// largest head K times.  Lane l of the first warp holds the parts l and l + 32.  (Counting places among the keys that reach a bound takes
// longer up to 20 alternatives: 3 rows of 248320 with 5 9.8 us instead of 8.8; with 64 it is 16.3 instead of 18.8.)
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_join_kernel(const LogprobParams p) {
    griddep_begin();
    __shared__ unsigned long long tops[kLpMaxParts * kLpMaxTop];
    const int lane = threadIdx.x & 31;
    const size_t row = blockIdx.x;
    const unsigned long long* from = p.part_top + row * p.parts * p.K;
    for (int e = threadIdx.x; e < p.parts * p.K; e += 8 * kLpThreads) {  // eight loads under way
        unsigned long long key[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) key[j] = e + j * kLpThreads < p.parts * p.K ? from[e + j * kLpThreads] : 0ull;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e + j * kLpThreads < p.parts * p.K) tops[e + j * kLpThreads] = key[j];
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
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
    const RowResults res(v, p.inv_t);
    if (lane == 0) {
        const int target = p.targets ? p.targets[row] : -1;
        res.write(p, row, v, target, target_logit<T>(p, row, target));
    }
    int at[2] = {0, 0};
    unsigned long long head[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) head[h] = p.K > 0 && lane + h * 32 < p.parts ? tops[(lane + h * 32) * p.K] : 0ull;
    unsigned long long mine[2] = {0ull, 0ull};  // lane l keeps the l-th and the (l + 32)-th best
    for (int k = 0; k < p.K; ++k) {
        const unsigned long long best = warp_largest(max(head[0], head[1]));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (head[h] == best && best != 0ull) head[h] = ++at[h] < p.K ? tops[(lane + h * 32) * p.K + at[h]] : 0ull;
            if (k == lane + h * 32) mine[h] = best;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (lane + h * 32 < p.K) res.write_top(p, row, lane + h * 32, mine[h]);
}

// The greedy token and its logit of every row, where the row's likeliest token is known: that one.  A row without a distribution has none, and
// a CTA looks for the largest of its logits in the order of the LM heads' argmax (as pack_best() ranks them), so that a round's
// tokens do not depend on whether it asks for log probabilities.  Two loads and two stores per row (2048 rows 1.9 us), but for such rows (one of
// 248320 57 us: its CTA's loads, latency; 2048 of them 386, near HBM's rate).
__global__ void __launch_bounds__(kLpThreads) greedy_tokens_kernel(const float* __restrict__ logits, int rows, int V,
                                                                   const int32_t* __restrict__ top_tokens, int K,
                                                                   int32_t* __restrict__ argmax, float* __restrict__ maxlogit) {
    griddep_begin();
    __shared__ unsigned long long bests[kLpThreads / 32];
    for (int row = blockIdx.x; row < rows; row += gridDim.x) {
        const float* x = logits + (size_t)row * V;
        int token = top_tokens[(size_t)row * K];
        float value;
        if (token >= 0 && token < V) {
            value = x[token];
        } else {
            unsigned long long best = 0ull;
#pragma unroll 4
            for (int i = threadIdx.x; i < V; i += kLpThreads) best = max(best, pack_best(x[i], (uint32_t)i));
            best = warp_largest(best);
            __syncthreads();  // of a row before this one, every thread has read its bests
            if ((threadIdx.x & 31) == 0) bests[threadIdx.x >> 5] = best;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kLpThreads / 32; ++w) best = max(best, bests[w]);
            token = key_token(best);
            value = key_logit(best);
        }
        if (threadIdx.x == 0) {
            argmax[row] = token;
            if (maxlogit) maxlogit[row] = value;
        }
    }
}

// Parts of a row, half a tile at least in each (every thread then has a logit, and the first bound comes from the warps): as many as fill the
// GPU once, or twice where once would leave more than a quarter of its places empty (400 rows of 248320: 3 parts 98 us, one 126; 512: 2
// parts 124, one 130; 300 rows, which fill 0.79: 2 parts 82, 5 parts 83).
template <typename T>
static int logprob_parts(int rows, int V) {
    const int places = sm_count() * LpShape<T>::kPerSm, once = places / rows, tiles = (V + kLpTile / 2) / kLpTile;
    const int want = once * rows < places * 3 / 4 ? 2 * places / rows : once;
    return std::max(1, std::min({want, tiles, kLpMaxParts}));
}

template <typename T>
static void launch_logprobs(LogprobParams p, void* workspace, cudaStream_t stream) {
    p.parts = logprob_parts<T>(p.rows, p.V);
    p.part_sums = (float4*)workspace;
    p.part_top = (unsigned long long*)(p.part_sums + (size_t)p.rows * p.parts);
    launch_pdl(logprobs_kernel<T>, p.rows * p.parts, kLpThreads, 0, stream, p);
    if (p.parts > 1) launch_pdl(logprobs_join_kernel<T>, p.rows, kLpThreads, 0, stream, p);
}

}  // namespace tsv

extern "C" size_t tsv_token_logprobs_workspace_size(int32_t rows, int32_t V, int32_t top_k) {
    using namespace tsv;
    if (rows < 1 || V < 1 || top_k < 0 || top_k > kLpMaxTop) return 0;
    const size_t parts = std::max(logprob_parts<float>(rows, V), logprob_parts<__half>(rows, V));  // for any type
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
    if ((long long)rows * std::max(logprob_parts<float>(rows, V), logprob_parts<__half>(rows, V)) > INT_MAX)
        return fail(TSV_ECAPACITY, "token_logprobs: rows=%d", rows);
    const LogprobParams p = {logits, targets, rows, V, top_k, 1, 1.f / temperature, logp, entropy, top_logp, rank, top_tokens};
    if (logits_dtype == TSV_F32) launch_logprobs<float>(p, workspace, stream);
    else if (logits_dtype == TSV_BF16) launch_logprobs<__nv_bfloat16>(p, workspace, stream);
    else launch_logprobs<__half>(p, workspace, stream);
    return check_launch("token_logprobs");
}

extern "C" tsv_status tsv_greedy_tokens(const float* logits, int32_t rows, int32_t V, const int32_t* top_tokens, int32_t top_k,
                                        int32_t* argmax, float* maxlogit, cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    if (rows < 0 || V < 1 || V > (1 << 24) || top_k < 1)
        return fail(TSV_EINVAL, "greedy_tokens: rows=%d V=%d (1 .. 2^24) top_k=%d", rows, V, top_k);
    if (rows == 0) return TSV_OK;
    if (!logits || !top_tokens || !argmax) return fail(TSV_EINVAL, "greedy_tokens: null pointer argument");
    if (((uintptr_t)logits | (uintptr_t)top_tokens | (uintptr_t)argmax | (uintptr_t)maxlogit) & 3)
        return fail(TSV_EINVAL, "greedy_tokens: a buffer is not aligned to its elements");
    launch_pdl(greedy_tokens_kernel, std::min(rows, sm_count() * 8), kLpThreads, 0, stream, logits, rows, V, top_tokens, top_k, argmax, maxlogit);
    return check_launch("greedy_tokens");
}
