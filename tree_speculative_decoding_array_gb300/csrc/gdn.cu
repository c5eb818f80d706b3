// The gated delta rule of a hybrid target's recurrent layers: tsv_gdn_tree_verify, tsv_gdn_commit, tsv_gdn_scan.
//
// mlxcel issue #1204 and Splash issue #728 ("What it does") name the need: recurrent layers cannot take a mask, a
// flattened tree would leak state between siblings, so every node has to run from its own parent's state and the
// accepted path's state is the one that is kept.  The pages do not spell the recurrence out; the arithmetic here is
// the published gated delta rule.  For one value head with state S [DV, DK], log decay g and write strength beta:
//
//     S <- e^g S;   u = beta (v - S k);   S <- S + u k^T;   o = S q * scale
//
// This file holds the CUDA-core kernels and the dispatch:
//   gdn_recur_kernel   token by token (short scans, commits): the state stays in registers, one pass over it
// tsv_gdn_tree_verify is in gdn_tree.cu, scans of more tokens in gdn_scan.cu.
#include <math.h>

#include "gdn_tc.cuh"

namespace tsv {

constexpr int kGdnRows = 64;      // state rows (value features) per CTA
constexpr int kGdnThreads = 128;  // 4 warps of 16 rows; 8 lanes share a row, 4 rows to a lane
constexpr int kGdnR = 4;
constexpr int kGdnBatch = 8;      // tokens whose q and k rows are in shared memory together

// One bf16 row of DK features, read by a whole warp, normalised and written to shared memory as fp32.
template <int DK>
__device__ __forceinline__ void stage_row(const uint16_t* src, float* dst, float norm_eps, float scale, int lane) {
    constexpr int E = DK / 32;  // 2 or 4 features per lane
    float x[E];
    if constexpr (E == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(src + lane * 4);
        x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(src + lane * 2);
        x[0] = bf16_lo(w); x[1] = bf16_hi(w);
    }
    float f = scale;
    if (norm_eps > 0.f) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        f = scale / sqrtf(ss + norm_eps);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) dst[lane * E + e] = x[e] * f;
}

// This lane's part of kGdnR state rows: features 4 (lane % 8) + 32 c .. + 3 of rows 4 r + lane / 8, as pairs.
template <int DK>
__device__ __forceinline__ void load_state(const float* base, float2 (&s)[kGdnR][DK / 16], int lane) {
#pragma unroll
    for (int r = 0; r < kGdnR; ++r)
#pragma unroll
        for (int c = 0; c < DK / 32; ++c) {
            const float4 w = __ldcs(reinterpret_cast<const float4*>(base + (size_t)(r * 4 + lane / 8) * DK + 32 * c + 4 * (lane % 8)));
            s[r][2 * c] = make_float2(w.x, w.y);
            s[r][2 * c + 1] = make_float2(w.z, w.w);
        }
}

// Advances the state token by token; COMMIT takes a tree block's rows along `path` and writes no outputs, otherwise
// the packed rows cu_len[b] .. cu_len[b + 1].  grid: (layer, sequence, value head, slice of kGdnRows state rows).
//
// Per token and state element: one FMA for S k, one for S q, a multiply for the decay and an FMA for the write, two
// elements to an instruction, with o = e^g (S q) + u (k . q) so that both products read the state before the write.  The
// state is read and written once per call, so few tokens are bound by HBM (128 KB per 128 x 128 head).  64 rows per CTA:
// a small CTA's loads, steps and stores overlap with those of the four others on its SM (128 rows: 74.6 us for 64 single
// tokens of 48 heads; 64 rows: 62 us, 6.5 TB/s).  Commit of up to 9 nodes, 32 sequences x 48 layers x 48 heads: 1.78 ms,
// 5.5 TB/s (four CTAs per SM: 1.85 ms); what is missing is the time of the steps between a CTA's loads and its stores.
template <int DK, bool COMMIT>
__global__ void __launch_bounds__(kGdnThreads, 5) gdn_recur_kernel(const __grid_constant__ tsv_gdn_desc d,
                                                                const int32_t* __restrict__ cu_len, int max_len,
                                                                const int32_t* __restrict__ path,
                                                                const int32_t* __restrict__ path_len, int32_t* status) {
    griddep_begin();
    __shared__ float ks[kGdnBatch][DK], qs[kGdnBatch][DK];
    __shared__ float vs[kGdnBatch][kGdnRows];
    __shared__ float al[kGdnBatch], be[kGdnBatch], kq[kGdnBatch];
    __shared__ int row_s[TSV_MAX_T];
    __shared__ int bad_s;
    const int slices = d.DV / kGdnRows;
    int item = blockIdx.x;
    const int slice = item % slices;
    item /= slices;
    const int h = item % d.HV;
    const int b = (item / d.HV) % d.B;
    const int layer = item / (d.HV * d.B);
    const int hk = h / (d.HV / d.HK);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool first_cta = slice == 0 && h == 0 && layer == 0;

    int n;
    size_t row0;  // first row of this sequence in the [rows, heads, features] inputs
    if (COMMIT) {
        n = path_len[b];
        row0 = (size_t)b * d.T;
        if (threadIdx.x == 0) bad_s = n < 1 || n > d.T;
        __syncthreads();
        if (!bad_s)
            for (int j = threadIdx.x; j < n; j += kGdnThreads) {
                const int p = path[(size_t)b * d.T + j];
                const int before = j > 0 ? path[(size_t)b * d.T + j - 1] : -1;
                if (p <= before || p >= d.T || (j == 0 && p != 0)) bad_s = 1;
                row_s[j] = p;
            }
        __syncthreads();
        if (bad_s) {
            if (first_cta && threadIdx.x == 0) dev_fail(status, TSV_DEV_BAD_PATH, b, 0);
            return;
        }
    } else {
        const int a = cu_len[b], e = cu_len[b + 1];
        n = e - a;
        row0 = (size_t)a;
        if (a < 0 || e < a || e > d.T || n > max_len) {
            if (first_cta && threadIdx.x == 0) dev_fail(status, TSV_DEV_BAD_SEQ_LEN, b, e);
            return;
        }
    }

    const size_t s0 = (((size_t)b * d.HV + h) * d.DV + slice * kGdnRows + warp * 4 * kGdnR) * DK;
    float2 s[kGdnR][DK / 16];
    load_state<DK>(d.state[layer] + s0, s, lane);
    const uint16_t* Q = reinterpret_cast<const uint16_t*>(d.q[layer]);
    const uint16_t* K = reinterpret_cast<const uint16_t*>(d.k[layer]);
    const uint16_t* V = reinterpret_cast<const uint16_t*>(d.v[layer]);
    __nv_bfloat16* O = reinterpret_cast<__nv_bfloat16*>(d.o[layer]);

    for (int t0 = 0; t0 < n; t0 += kGdnBatch) {
        const int nt = min(kGdnBatch, n - t0);
        __syncthreads();
        for (int j = warp; j < nt; j += kGdnThreads / 32) {
            const size_t row = row0 + (COMMIT ? row_s[t0 + j] : t0 + j);
            stage_row<DK>(K + (row * d.HK + hk) * DK, ks[j], d.norm_eps, 1.f, lane);
            if (!COMMIT) stage_row<DK>(Q + (row * d.HK + hk) * DK, qs[j], d.norm_eps, d.scale, lane);
            const uint32_t v2 = *reinterpret_cast<const uint32_t*>(V + (row * d.HV + h) * d.DV + slice * kGdnRows + 2 * lane);
            *reinterpret_cast<float2*>(&vs[j][2 * lane]) = make_float2(bf16_lo(v2), bf16_hi(v2));
            if (lane == 0) {
                al[j] = expf(d.g[layer][row * d.HV + h]);
                be[j] = d.beta[layer][row * d.HV + h];
            }
            if (!COMMIT) {
                __syncwarp();
                float p = 0.f;
#pragma unroll
                for (int e = lane; e < DK; e += 32) p = fmaf(ks[j][e], qs[j][e], p);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) p += __shfl_xor_sync(0xFFFFFFFFu, p, o);
                if (lane == 0) kq[j] = p;
            }
        }
        __syncthreads();
        for (int j = 0; j < nt; ++j) {
            float2 kk[DK / 16], sk2[kGdnR], sq2[kGdnR];
#pragma unroll
            for (int r = 0; r < kGdnR; ++r) sk2[r] = sq2[r] = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < DK / 32; ++c) {
                const float4 w = *reinterpret_cast<const float4*>(&ks[j][32 * c + 4 * (lane % 8)]);
                kk[2 * c] = make_float2(w.x, w.y);
                kk[2 * c + 1] = make_float2(w.z, w.w);
#pragma unroll
                for (int r = 0; r < kGdnR; ++r) sk2[r] = fma2(s[r][2 * c], kk[2 * c], fma2(s[r][2 * c + 1], kk[2 * c + 1], sk2[r]));
                if (!COMMIT) {
                    const float4 y = *reinterpret_cast<const float4*>(&qs[j][32 * c + 4 * (lane % 8)]);
#pragma unroll
                    for (int r = 0; r < kGdnR; ++r)
                        sq2[r] = fma2(s[r][2 * c], make_float2(y.x, y.y), fma2(s[r][2 * c + 1], make_float2(y.z, y.w), sq2[r]));
                }
            }
            float sk[kGdnR], sq[kGdnR];
#pragma unroll
            for (int r = 0; r < kGdnR; ++r) {
                sk[r] = sk2[r].x + sk2[r].y;
                sq[r] = sq2[r].x + sq2[r].y;
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                for (int r = 0; r < kGdnR; ++r) {
                    sk[r] += __shfl_xor_sync(0xFFFFFFFFu, sk[r], o);
                    if (!COMMIT) sq[r] += __shfl_xor_sync(0xFFFFFFFFu, sq[r], o);
                }
            const float a = al[j], bt = be[j];
#pragma unroll
            for (int r = 0; r < kGdnR; ++r) {
                const int vr = warp * 4 * kGdnR + r * 4 + lane / 8;
                const float u = bt * (vs[j][vr] - a * sk[r]);
#pragma unroll
                for (int c = 0; c < DK / 16; ++c) s[r][c] = fma2(make_float2(u, u), kk[c], mul2(make_float2(a, a), s[r][c]));
                if (!COMMIT && lane % 8 == 0)
                    O[((row0 + t0 + j) * d.HV + h) * d.DV + slice * kGdnRows + vr] = __float2bfloat16(fmaf(a, sq[r], u * kq[j]));
            }
        }
    }
    float* out = d.state_out[layer] + s0;
#pragma unroll
    for (int r = 0; r < kGdnR; ++r)
#pragma unroll
        for (int c = 0; c < DK / 32; ++c)
            __stcs(reinterpret_cast<float4*>(out + (size_t)(r * 4 + lane / 8) * DK + 32 * c + 4 * (lane % 8)),
                   make_float4(s[r][2 * c].x, s[r][2 * c].y, s[r][2 * c + 1].x, s[r][2 * c + 1].y));
}

// Defined in gdn_tree.cu and gdn_scan.cu.
void launch_gdn_tree(const tsv_gdn_desc& d, const uint64_t* anc, int32_t* status, cudaStream_t stream);
void launch_gdn_scan(const tsv_gdn_desc& d, const int32_t* cu_len, int max_len, int32_t* status, cudaStream_t stream);

// Sequences of up to this many tokens are advanced token by token, longer ones in chunks of 64 (whose time hardly depends on
// the length up to 64; the more heads there are, the better the recurrence hides its latency).  48 heads of 128, token by token
// against in chunks: 1 sequence of 8 tokens 10.2 and 12.0 us, of 12 13.9 and 12.0; 8 sequences of 12 tokens 34.9 and 38.1, of
// 16 44.2 and 38.2; 64 sequences of 16 tokens 233 and 256, of 18 268 and 256.
static int recur_max(const tsv_gdn_desc* d) {
    const long long units = (long long)d->n_layers * d->B * d->HV;
    return units < 2LL * sm_count() ? 10 : units < 8LL * sm_count() ? 14 : 17;
}

enum GdnCall { kGdnVerify, kGdnCommit, kGdnScan };

static tsv_status check_gdn(const tsv_gdn_desc* d, GdnCall call, const char* name) {
    if (!d) return fail(TSV_EINVAL, "%s: null descriptor", name);
    if (d->n_layers < 1 || d->n_layers > TSV_MAX_LAYERS)
        return fail(TSV_ECAPACITY, "%s: n_layers=%d outside [1, %d]", name, d->n_layers, TSV_MAX_LAYERS);
    if (call == kGdnScan ? d->T < 0 : (d->T < 1 || d->T > TSV_MAX_T))
        return fail(TSV_ECAPACITY, "%s: T=%d outside [%d, %d]", name, d->T, call == kGdnScan ? 0 : 1,
                    call == kGdnScan ? 0x7FFFFFFF : TSV_MAX_T);
    if (d->B < 0 || d->HK < 1 || d->HV < 1 || d->HV % d->HK)
        return fail(TSV_EINVAL, "%s: B=%d HK=%d HV=%d", name, d->B, d->HK, d->HV);
    if ((d->DK != 64 && d->DK != 128) || (d->DV != 64 && d->DV != 128))
        return fail(TSV_EUNSUPPORTED, "%s: head dims DK=%d DV=%d are not 64 or 128", name, d->DK, d->DV);
    if (!(d->norm_eps >= 0.f) || d->norm_eps > 1e30f) return fail(TSV_EINVAL, "%s: norm_eps=%g", name, (double)d->norm_eps);
    if (!(fabsf(d->scale) <= 1e30f)) return fail(TSV_EINVAL, "%s: scale=%g", name, (double)d->scale);
    if ((long long)d->n_layers * d->B * d->HV * (d->DV / kGdnRows) > 0x7FFFFFFFLL)
        return fail(TSV_ECAPACITY, "%s: too many (layer, sequence, head) units", name);
    if (d->B == 0) return TSV_OK;  // an empty batch: no pointer is read
    const bool out = call != kGdnCommit, wr = call != kGdnVerify;
    for (int l = 0; l < d->n_layers; ++l) {
        if (!d->state[l] || (wr && !d->state_out[l])) return fail(TSV_EINVAL, "%s: layer %d has a null state", name, l);
        if (((uintptr_t)d->state[l] | (wr ? (uintptr_t)d->state_out[l] : 0)) & 15)
            return fail(TSV_EINVAL, "%s: layer %d state not 16-byte aligned", name, l);
        if (d->T == 0) continue;  // a scan without new rows reads no inputs
        if (!d->k[l] || !d->v[l] || !d->g[l] || !d->beta[l] || (out && (!d->q[l] || !d->o[l])))
            return fail(TSV_EINVAL, "%s: layer %d has a null pointer", name, l);
        if (((uintptr_t)d->k[l] | (uintptr_t)d->v[l] | (out ? (uintptr_t)d->q[l] | (uintptr_t)d->o[l] : 0)) & 15)
            return fail(TSV_EINVAL, "%s: layer %d q/k/v/o not 16-byte aligned", name, l);
        if (((uintptr_t)d->g[l] | (uintptr_t)d->beta[l]) & 3)
            return fail(TSV_EINVAL, "%s: layer %d g/beta not 4-byte aligned", name, l);
    }
    return TSV_OK;
}

// The caller's descriptor with the default scale filled in.
static tsv_gdn_desc with_scale(const tsv_gdn_desc* d) {
    tsv_gdn_desc x = *d;
    if (x.scale == 0.f) x.scale = (float)(1.0 / sqrt((double)d->DK));
    return x;
}

}  // namespace tsv

extern "C" tsv_status tsv_gdn_tree_verify(const tsv_gdn_desc* d, const uint64_t* anc, int32_t* dev_status,
                                          cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    tsv_status st = check_gdn(d, kGdnVerify, "gdn_tree_verify");
    if (st != TSV_OK || d->B == 0) return st;
    if (!anc) return fail(TSV_EINVAL, "gdn_tree_verify: anc must be non-null");
    const tsv_gdn_desc x = with_scale(d);
    launch_gdn_tree(x, anc, dev_status, stream);
    return check_launch("gdn_tree_verify");
}

extern "C" tsv_status tsv_gdn_commit(const tsv_gdn_desc* d, const int32_t* path, const int32_t* path_len,
                                     int32_t* dev_status, cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    tsv_status st = check_gdn(d, kGdnCommit, "gdn_commit");
    if (st != TSV_OK || d->B == 0) return st;
    if (!path || !path_len) return fail(TSV_EINVAL, "gdn_commit: path and path_len must be non-null");
    const tsv_gdn_desc x = with_scale(d);
    const unsigned grid = (unsigned)((long long)d->n_layers * d->B * d->HV * (d->DV / kGdnRows));
    const int32_t* none = nullptr;
    if (d->DK == 64) launch_pdl(gdn_recur_kernel<64, true>, grid, kGdnThreads, 0, stream, x, none, 0, path, path_len, dev_status);
    else launch_pdl(gdn_recur_kernel<128, true>, grid, kGdnThreads, 0, stream, x, none, 0, path, path_len, dev_status);
    return check_launch("gdn_commit");
}

extern "C" tsv_status tsv_gdn_scan(const tsv_gdn_desc* d, const int32_t* cu_len, int32_t max_len, int32_t* dev_status,
                                   cudaStream_t stream) {
    using namespace tsv;
    clear_error();
    tsv_status st = check_gdn(d, kGdnScan, "gdn_scan");
    if (st != TSV_OK || d->B == 0) return st;
    if (!cu_len) return fail(TSV_EINVAL, "gdn_scan: cu_len must be non-null");
    if (max_len < 0 || max_len > d->T) return fail(TSV_EINVAL, "gdn_scan: max_len=%d outside [0, T=%d]", max_len, d->T);
    const tsv_gdn_desc x = with_scale(d);
    if (max_len > recur_max(d)) {
        launch_gdn_scan(x, cu_len, max_len, dev_status, stream);
        return check_launch("gdn_scan");
    }
    const unsigned grid = (unsigned)((long long)d->n_layers * d->B * d->HV * (d->DV / kGdnRows));
    const int32_t* none = nullptr;
    if (d->DK == 64) launch_pdl(gdn_recur_kernel<64, false>, grid, kGdnThreads, 0, stream, x, cu_len, max_len, none, none, dev_status);
    else launch_pdl(gdn_recur_kernel<128, false>, grid, kGdnThreads, 0, stream, x, cu_len, max_len, none, none, dev_status);
    return check_launch("gdn_scan");
}
