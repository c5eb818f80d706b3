// tsv_token_logprobs: log probability and rank of a given token, entropy and the likeliest tokens of every row of logits.
//
//   z = logits / T;  logp(t) = z_t - log sum exp z;  entropy = log sum exp z - sum p z
#include "e4m3.cuh"

namespace tsv {

constexpr int kLpThreads = 1024;
constexpr int kLpMaxTop = 64;

struct LogprobParams {
    const void* logits;
    const int32_t* targets;
    int rows, V, K;
    float inv_t;
    float *logp, *entropy, *top_logp;
    int32_t *rank, *top_tokens;
};

template <typename F>
__device__ __forceinline__ unsigned long long lp_cta_max(unsigned long long v, unsigned long long* s, F) {
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    for (int w = 0; w < kLpThreads / 32; ++w) v = max(v, s[w]);
    __syncthreads();
    return v;
}

__device__ __forceinline__ float lp_cta_sum(float v, float* s) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kLpThreads / 32; ++w) v += s[w];
    __syncthreads();
    return v;
}

// A CTA per row.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LogprobParams p) {
    griddep_begin();
    __shared__ unsigned long long s[kLpThreads / 32];
    float* sf = reinterpret_cast<float*>(s);
    const size_t row = blockIdx.x;
    const T* x = (const T*)p.logits + row * p.V;
    // + 0 turns -0 into 0, which is no smaller a logit
    auto at = [&](int i) { return RowType<T>::to_f32(x[i]) + 0.f; };
    unsigned long long best = 0ull;
    float bad = 0.f;
    for (int i = threadIdx.x; i < p.V; i += kLpThreads) {
        const float v = at(i);
        if (!(v < INFINITY)) bad = 1.f;
        best = max(best, pack_best(v, (uint32_t)i));
    }
    bad = lp_cta_sum(bad, sf);
    best = lp_cta_max(best, s, 0);
    const float m = unorderable((uint32_t)(best >> 32));
    if (bad > 0.f || m == -INFINITY) {
        const float nan = __int_as_float(0x7FFFFFFF);
        for (int k = threadIdx.x; k < p.K; k += kLpThreads) p.top_tokens[row * p.K + k] = -1, p.top_logp[row * p.K + k] = nan;
        if (threadIdx.x == 0) {
            if (p.logp) p.logp[row] = nan;
            if (p.rank) p.rank[row] = -1;
            if (p.entropy) p.entropy[row] = nan;
        }
        return;
    }
    const int target = p.targets ? p.targets[row] : -1;
    const bool has = target >= 0 && target < p.V;
    const float t = has ? at(target) : 0.f;
    float sum = 0.f, mean = 0.f, rank = 0.f;
    int above = 0;
    for (int i = threadIdx.x; i < p.V; i += kLpThreads) {
        const float v = at(i), z = (v - m) * p.inv_t, e = expf(z);
        sum += e;
        if (e > 0.f) mean = fmaf(e, z, mean);
        if (has && (v > t || (v == t && i < target))) ++above;
    }
    sum = lp_cta_sum(sum, sf);
    mean = lp_cta_sum(mean, sf);
    rank = lp_cta_sum((float)above, sf);  // whole numbers below 2^24
    const float lse = logf(sum);
    if (threadIdx.x == 0) {
        if (p.logp) p.logp[row] = has ? (t - m) * p.inv_t - lse : __int_as_float(0x7FFFFFFF);
        if (p.rank) p.rank[row] = has ? (int)rank : -1;
        if (p.entropy) p.entropy[row] = lse - mean / sum;
    }
    for (int k = 0; k < p.K; ++k) {
        if (threadIdx.x == 0) {
            p.top_tokens[row * p.K + k] = (int32_t)(0xFFFFFFFFu - (uint32_t)best);
            p.top_logp[row * p.K + k] = (unorderable((uint32_t)(best >> 32)) - m) * p.inv_t - lse;
        }
        unsigned long long next = 0ull;
        for (int i = threadIdx.x; i < p.V; i += kLpThreads) {
            const unsigned long long key = pack_best(at(i), (uint32_t)i);
            if (key < best) next = max(next, key);
        }
        best = lp_cta_max(next, s, 0);
    }
}

}  // namespace tsv

extern "C" size_t tsv_token_logprobs_workspace_size(int32_t rows, int32_t V, int32_t top_k) {
    (void)V, (void)top_k;
    return rows < 1 ? 0 : 16;
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
    const LogprobParams p = {logits, targets, rows, V, top_k, 1.f / temperature, logp, entropy, top_logp, rank, top_tokens};
    if (logits_dtype == TSV_F32) launch_pdl(logprobs_kernel<float>, rows, kLpThreads, 0, stream, p);
    else if (logits_dtype == TSV_BF16) launch_pdl(logprobs_kernel<__nv_bfloat16>, rows, kLpThreads, 0, stream, p);
    else launch_pdl(logprobs_kernel<__half>, rows, kLpThreads, 0, stream, p);
    return check_launch("token_logprobs");
}
