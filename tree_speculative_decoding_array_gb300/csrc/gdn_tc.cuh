// Building blocks of the gated delta rule's tensor-core kernels: fp16 fragments of mma.sync, rows staged with an
// exact power-of-two scale, the block's triangular system.
//
// A block of up to 64 rows (a tree's nodes, or consecutive tokens) is one triangular system.  With G_i the log decay
// summed over i's ancestors and itself, unit rows k_i, q_i and the state S [DV, DK] ahead of the block,
//     u_i = beta_i (v_i - e^{G_i} S k_i - sum_{j before i} e^{G_i - G_j} (k_i . k_j) u_j)
//     o_i = e^{G_i} S q_i + sum_{j before i, or i} e^{G_i - G_j} (q_i . k_j) u_j
// ("before": strict ancestor, or earlier token).  Every value feature (row of S, column of u and o) is a system of
// its own with the same matrices.  The large products run on the 5th-generation tensor cores: [K; Q] K^T (rows in the
// TMEM lanes) and S [K; Q]^T (value features in the lanes, S as fp16 pairs in TMEM).  Both are read back from TMEM in
// the layout of mma.sync fragments, in which a warp owns 16 value features and solves their systems in registers, 16
// rows of the block at a time: R_b from S and the blocks before, U_b = (I + A_bb)^-1 R_b with that 16 x 16 inverse,
// then O_b.  Only the matrices, K, Q and V pass through shared memory.
//
// Operands are fp16 with power-of-two scales, which cost nothing in accuracy: K and Q rows hold bf16 values (8 bits,
// exact in fp16 once the row's norm is scaled to about 1; what falls below 2^-24 of it is lost), S, R and U of one
// value feature share a scale (their equations are linear in them).  An fp16 operand is within 2^-12 of its value; an
// hi + lo pair within 2^-22 (either: or 2^-37 of the feature's largest value).  Accumulation is fp32.
#pragma once

#include "common.cuh"
#include "tc.cuh"

namespace tsv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLogDecay = -150.f;  // e^-150 is 0 in fp32: a smaller (or infinite) log decay means the same
// P and e^G S q are computed without q's scale and times this, and o is multiplied with scale / kOutLift in fp32: an fp16
// P then holds weights down to 2^-33 whatever the scale, and q rows of up to 2^8 times unit length.
constexpr float kOutLift = 256.f;
// A feature's S, R and U are scaled until the largest of 8 max |S row| and max |v| is in [2^12, 2^13): fp16 then holds them
// down to 2^-37 of it.  Room above: with unit keys and 0 <= beta <= 1 a write v adds at most v^2 to |S row|^2, so 64 writes
// reach 2^16 only where each is orthogonal to those before; what does leave the range is seen (watch()).
constexpr float kLift = 4096.f;
// The system's matrix (its blocks ahead of the diagonal and the inverses on it) is held down to 2^-37, so that a large write
// which decays by much is as exact as what it is added to.  One piece: the matrix is held times kMatLift, with room for keys
// of up to four times unit length, and R on its way to U as well.  Two pieces: the lo piece is held times kMatLift and meets
// the operand divided by it.
constexpr float kMatLift = 4096.f;
template <int PIECES>
constexpr float kHiLift = PIECES == 1 ? kMatLift : 1.f;

__device__ __forceinline__ float clamp_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }  // keeps NaN

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// hi + lo fp16 pieces of two values.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = f16x2(a, b);
    const float2 h = f16x2_to_f32x2(hi);
    lo = f16x2(a - h.x, b - h.y);
}
// NaN in `flag` once any half of x is an infinity or a NaN.
__device__ __forceinline__ void watch(uint32_t& flag, uint32_t x) {
    const __half2 z = __floats2half2_rn(0.f, 0.f);
    const __half2 f = __hfma2(*reinterpret_cast<const __half2*>(&x), z, *reinterpret_cast<const __half2*>(&flag));
    flag = *reinterpret_cast<const uint32_t*>(&f);
}
__device__ __forceinline__ bool watched(uint32_t flag) {
    const float2 f = f16x2_to_f32x2(flag);
    return !(f.x == 0.f && f.y == 0.f);
}
// Two fp32 products or sums per instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 c;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}"
        : "=f"(c.x), "=f"(c.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return c;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 d) {
    float2 c;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n fma.rn.f32x2 z, x, y, z;\n"
        " mov.b64 {%0, %1}, z;\n}"
        : "=f"(c.x), "=f"(c.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(d.x), "f"(d.y));
    return c;
}
// hi + lo fp16 pieces of two values, lo times kMatLift.
__device__ __forceinline__ void split2_lifted(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = f16x2(a, b);
    const float2 y = fma2(f16x2_to_f32x2(hi), make_float2(-kMatLift, -kMatLift), mul2(make_float2(a, b), make_float2(kMatLift, kMatLift)));
    lo = f16x2(y.x, y.y);
}
// An operand for a lifted lo piece.
__device__ __forceinline__ uint32_t lowered(uint32_t x) {
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x), __floats2half2_rn(1.f / kMatLift, 1.f / kMatLift));
    return *reinterpret_cast<const uint32_t*>(&y);
}
// 2^-e and 2^e for m in [2^e, 2^(e+1)); 1 for 0, infinities and NaN.
__device__ __forceinline__ void pow2_scale(float m, float& down, float& up) {
    uint32_t e = (__float_as_uint(m) >> 23) & 255u;
    if (e == 255u || m == 0.f) e = 127u;
    e = min(max(e, 1u), 253u);
    down = __uint_as_float((254u - e) << 23);
    up = __uint_as_float(e << 23);
}

// A whole warp's bounded wait: the poll inline, the sleeping loop (tc::mbar_wait) out of line, once per kernel.
static __device__ __noinline__ bool wait_out_of_line(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xFFFFFFFFu, tc::mbar_wait(bar, parity, abort));
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (__all_sync(0xFFFFFFFFu, tc::mbar_test(bar, parity))) return true;
    return wait_out_of_line(bar, parity, abort);
}

// 16 bytes from global to shared memory, asynchronously; zeros when !real (src is then not read).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A sum of log decays in units of ln 2 as an unevaluated pair: differences of far sums keep fp32 accuracy.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair log2_decay(float g) {
    const float c = clamp_decay(g);
    Pair p;
    p.hi = c * kLog2e;
    p.lo = fmaf(c, kLog2e, -p.hi) + c * 1.925963033500e-8f;  // log2(e) - fp32(log2(e))
    return p;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {  // two-sum, then renormalised
    const float s = a.hi + b.hi, z = s - a.hi;
    const float e = ((a.hi - (s - z)) + (b.hi - z)) + (a.lo + b.lo);
    Pair p;
    p.hi = s + e;
    p.lo = e - (p.hi - s);
    return p;
}

// Shared-memory tiles: rows of BYTES bytes, 16-byte chunk c of row r at chunk c ^ (r & 7), so that the 8 rows of an
// ldmatrix fall into different banks.
template <int BYTES>
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int row, int chunk) {
    return base + (uint32_t)(row * BYTES + ((chunk ^ (row & 7)) << 4));
}

// Per-row scalars of a block: those of the key head, and those of one value head.
struct GdnKeys {
    uint64_t before[64];   // rows ahead of i in its system (strict ancestors, or earlier tokens)
    float fk[64], fq[64];  // what a staged row's products are multiplied with: its scale and norm (q: and kOutLift)
};
struct GdnRows {
    float g_hi[64], g_lo[64];  // G in units of ln 2, as hi + lo (differences of far sums keep fp32 accuracy)
    float beta[64];
    float ck[64], cq[64];      // 2^(G - e) fk, 2^(G - e) fq
    // e: the floor of the largest G (within fp32's exponents).  The state enters as 2^e S (fade = 2^e), so that what no row
    // sees of it - a state that the block's first row forgets - has no part in the scale.  seen, write: smallest 2^(G - e)
    // (rounded down) and |beta|.
    float e, fade, seen, write;
};

// N chunks of 8 bf16 values, each of a K or Q row of its own -> fp16 in place, scaled by a power of two that brings the
// row's norm to [1, 2); DK / 8 consecutive lanes share a row.  f: what the row's products are to be multiplied with,
// its scale over its norm.  The chunks go through each step together: their shuffles overlap, and there is no branch.
template <int DK, int N>
__device__ __forceinline__ void stage_chunks(uint4 (&w)[N], float (&f)[N], float norm_eps, uint32_t& flag) {
    float ss[N];
#pragma unroll
    for (int x = 0; x < N; ++x) {
        const uint32_t y[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 z = make_float2(bf16_lo(y[e]), bf16_hi(y[e]));
            s2 = fma2(z, z, s2);
        }
        ss[x] = s2.x + s2.y;
    }
#pragma unroll
    for (int o = DK / 16; o > 0; o >>= 1)
#pragma unroll
        for (int x = 0; x < N; ++x) ss[x] += __shfl_xor_sync(0xFFFFFFFFu, ss[x], o);
#pragma unroll
    for (int x = 0; x < N; ++x) {
        const int es = (int)(__float_as_uint(ss[x]) >> 23);
        const int e = es == 0 || es >= 255 ? 0 : (es - 127) >> 1;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
        f[x] = norm_eps > 0.f ? up * rsqrtf(ss[x] + norm_eps) : up;
        // squares that underflowed, or a row so short (norm_eps 0, or far above its squares) that P would be: the fp32 path
        flag = (ss[x] < 1e-30f || f[x] < 0x1p-8f) && ((w[x].x | w[x].y | w[x].z | w[x].w) & 0x7FFF7FFFu) ? 0x7FFF7FFFu : flag;
        const uint32_t y[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
        uint32_t z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 a = mul2(make_float2(bf16_lo(y[k]), bf16_hi(y[k])), make_float2(down, down));
            z[k] = f16x2(a.x, a.y);
        }
        w[x] = make_uint4(z[0], z[1], z[2], z[3]);
    }
}

// Largest (smallest) |v| as pairs of bf16, NaN passed over, two values of v at a time.
constexpr uint32_t kInf2 = 0x7F807F80u;
__device__ __forceinline__ uint32_t abs_max2(uint32_t top, uint32_t v) {
    const uint32_t a = v & 0x7FFF7FFFu;
    const __nv_bfloat162 x = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&top), *reinterpret_cast<const __nv_bfloat162*>(&a));
    return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint32_t abs_min2(uint32_t low, uint32_t v) {
    const uint32_t a = v & 0x7FFF7FFFu;
    const __nv_bfloat162 x = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&low), *reinterpret_cast<const __nv_bfloat162*>(&a));
    return *reinterpret_cast<const uint32_t*>(&x);
}

// The exponent that the state enters a block with, from the largest G, and its power of two.
__device__ __forceinline__ float fade_exponent(float g) { return fminf(fmaxf(floorf(g), -126.f), 127.f); }
__device__ __forceinline__ float pow2_of(float e) { return __uint_as_float((uint32_t)((int)e + 127) << 23); }

// Smallest |beta| of a block's first n rows, by one warp.
__device__ __forceinline__ float least_write(const GdnRows& rw, int n, int lane) {
    uint32_t x = lane < n ? __float_as_uint(fabsf(rw.beta[lane])) : 0x7F800000u;
    if (lane + 32 < n) x = min(x, __float_as_uint(fabsf(rw.beta[lane + 32])));
    return __uint_as_float(__reduce_min_sync(0xFFFFFFFFu, x));
}

// What fp16 loses at its lower end.  S, R and U of a feature share a scale, so next to a value at the scale's top (2^13) a
// value below kFaint = 2^-12 is held by its last 13 bits or fewer, and next to a far larger one it is 0.  That only matters
// where a row sees nothing larger.  True if one of the block's first n rows sees less than kFaint in one of this thread's
// features f and f + 8, and not nothing: for what it sees this takes its own write, that of the row just before it (its
// parent) and the state, decayed to it.  The block is then for the fp32 path.
// Called by whole warps, where the state fades below kFaint (s * rw.seen).  Rows 8 m + 2 t, + 1 are this thread's, and the
// product of their smallest v and the smallest beta is looked at first: in a block of ordinary values it is hardly ever
// faint.  v: V tile, rows of BYTES bytes; d: what v is scaled with; s: the largest of the state's row, faded and scaled.
constexpr float kFaint = 0x1p-12f;
template <int BYTES, int NB>
__device__ __noinline__ bool faint_rows(const char* v, int fb, float d0, float d1, float s0, float s1, const GdnRows& rw, const GdnKeys& ky,
                                        int n) {
    const int lane = threadIdx.x & 31;
    uint32_t low[2] = {kInf2, kInf2};
#pragma unroll
    for (int bb = 0; bb < NB; ++bb) {
        uint32_t w[4];
        ldsm4_t(w, tile_at<BYTES>(tc::smem_u32(v), bb * 16 + ((lane >> 4) << 3) + (lane & 7), fb / 8 + ((lane >> 3) & 1)));
#pragma unroll
        for (int x = 0; x < 4; ++x) low[x & 1] = abs_min2(low[x & 1], w[x]);
    }
    if (fminf(fminf(bf16_lo(low[0]), bf16_hi(low[0])) * d0, fminf(bf16_lo(low[1]), bf16_hi(low[1])) * d1) * rw.write >= kFaint) return false;
    const int f = fb + (lane >> 2);
    bool faint = false;
    for (int j = 2 * (lane & 3); j < n; j += (j & 1) ? 7 : 1) {
        const float G = rw.g_hi[j], W = tc::ex2_approx(G - rw.e);
        const int p = ky.before[j] ? 63 - __clzll((long long)ky.before[j]) : -1;
        const float be = fabsf(rw.beta[j]), bp = p < 0 ? 0.f : fabsf(rw.beta[p]) * tc::ex2_approx(G - rw.g_hi[p]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int at = (f >> 3) + half;
            const float x = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(v + tile_at<BYTES>(0, j, at) + 2 * (f & 7)));
            const float y = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(v + tile_at<BYTES>(0, p < 0 ? j : p, at) + 2 * (f & 7)));
            const float sees = fmaxf(fmaxf(be * fabsf(x), bp * fabsf(y)) * (half ? d1 : d0), (half ? s1 : s0) * W);
            faint = faint || (sees > 0.f && sees < kFaint);
        }
    }
    return faint;
}

// K and Q as operand tiles: DK / 64 blocks of [ROWS][128 B], 128-byte swizzled; chunk 0 .. DK / 8 - 1 of a row.
template <int ROWS>
__device__ __forceinline__ uint32_t kq_at(uint32_t base, int row, int chunk) {
    return base + (uint32_t)((chunk >> 3) * ROWS * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// Where 16-row block b of K (and of Q, NB blocks on) sits in the tile, its TMEM lanes and the products' columns.  A
// quarter of the TMEM lanes belongs to two warps; four blocks in the order 0 3 1 2 give every quarter five block
// products (block b has b + 1).
template <int NB>
__host__ __device__ constexpr int block_pos(int b) {
    return NB == 4 ? (b == 0 ? 0 : b == 3 ? 1 : b + 1) : b;
}

// Products of one 16-row block with the K rows of blocks c0 .. c1 - 1, none of them after its own (TMEM columns
// 16 block_pos(c) of `taddr`, the block's rows in its lanes), decayed and masked:
//   q == false: rows K_b; -A kHiLift (fp16 pieces) for the blocks before, A itself (fp32) for the block's own
//   q == true:  rows Q_b; P (fp16)
// a16 / p16: [T rows][128 B] tiles; diag: this block's [16][kDiag] fp32.
constexpr int kDiag = 20;  // fp32 row stride of a diagonal block: 16-byte aligned, rows in different banks
template <int NB, int PIECES>
__device__ __forceinline__ void block_matrices(bool q, int b, int c0, int c1, uint32_t taddr, char* a16, char* p16, float* diag,
                                               const GdnKeys& ky, const GdnRows& rw, uint32_t& flag, int lane) {
    constexpr int T = 16 * NB;
    const int g = lane >> 2, t = lane & 3;
    float gh[2], gl[2], f[2];
    uint64_t seen[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = b * 16 + g + 8 * half;
        gh[half] = rw.g_hi[i];
        gl[half] = rw.g_lo[i];
        f[half] = q ? ky.fq[i] : rw.beta[i] * ky.fk[i];
        seen[half] = q ? ky.before[i] | (1ull << i) : ky.before[i];
    }
    float next[8];
    tc::tmem_ld_frag2(taddr + 16 * block_pos<NB>(c0), next);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {  // rolled: a kernel's warps run different parts at once and share the instruction cache
        float x[8];
        float2 jh[2], jl[2], jf[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int j0 = c * 16 + n * 8 + 2 * t;
            jh[n] = *reinterpret_cast<const float2*>(&rw.g_hi[j0]);
            jl[n] = *reinterpret_cast<const float2*>(&rw.g_lo[j0]);
            jf[n] = *reinterpret_cast<const float2*>(&ky.fk[j0]);
        }
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = next[e];
        if (c + 1 < c1) tc::tmem_ld_frag2(taddr + 16 * block_pos<NB>(c + 1), next);
        float y[2][2][2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float fc = q || c == b ? f[half] : -kHiLift<PIECES> * f[half];
            const uint32_t bits = (uint32_t)(seen[half] >> (c * 16)) >> (2 * t);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float w0 = tc::ex2_approx((gh[half] - jh[n].x) + (gl[half] - jl[n].x));
                const float w1 = tc::ex2_approx((gh[half] - jh[n].y) + (gl[half] - jl[n].y));
                const float y0 = x[4 * n + 2 * half] * jf[n].x * (fc * w0);
                const float y1 = x[4 * n + 2 * half + 1] * jf[n].y * (fc * w1);
                y[half][n][0] = (bits & (1u << (n * 8))) ? y0 : 0.f;
                y[half][n][1] = (bits & (2u << (n * 8))) ? y1 : 0.f;
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int il = g + 8 * half, i = b * 16 + il;
                const float y0 = y[half][n][0], y1 = y[half][n][1];
                if (q) {
                    const uint32_t h = f16x2(y0, y1);
                    watch(flag, h);
                    *reinterpret_cast<uint32_t*>(p16 + tile_at<128>(0, i, 2 * c + n) + 4 * t) = h;
                } else if (c == b) {
                    *reinterpret_cast<float2*>(diag + il * kDiag + n * 8 + 2 * t) = make_float2(y0, y1);
                } else {
                    uint32_t hi, lo;
                    split2_lifted(y0, y1, hi, lo);
                    *reinterpret_cast<uint32_t*>(a16 + tile_at<128>(0, i, 2 * c + n) + 4 * t) = hi;
                    if (PIECES == 2) *reinterpret_cast<uint32_t*>(a16 + T * 128 + tile_at<128>(0, i, 2 * c + n) + 4 * t) = lo;
                }
            }
    }
}

// kHiLift (I + A_bb)^-1 of one block by forward substitution, a column per lane (both half-warps do the same), stored over
// block (b, b) of the a16 tile.
template <int NB, int PIECES>
__device__ __forceinline__ void block_inverse(int b, char* a16, const float* diag, int lane) {
    constexpr int T = 16 * NB;
    const int c = lane & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s0 = i == c ? kHiLift<PIECES> : 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < i; j += 4) {
            const float4 a = *reinterpret_cast<const float4*>(diag + i * kDiag + j);
            s0 = fmaf(-a.x, x[j], s0);
            if (j + 1 < i) s1 = fmaf(-a.y, x[j + 1], s1);
            if (j + 2 < i) s0 = fmaf(-a.z, x[j + 2], s0);
            if (j + 3 < i) s1 = fmaf(-a.w, x[j + 3], s1);
        }
        x[i] = s0 + s1;
    }
    if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            uint32_t hi, lo;
            split2_lifted(x[i], x[i + 1], hi, lo);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = b * 16 + i + e, col = b * 16 + c;
                char* at = a16 + tile_at<128>(0, row, col >> 3) + 2 * (col & 7);
                *reinterpret_cast<uint16_t*>(at) = (uint16_t)(hi >> (16 * e));
                if (PIECES == 2) *reinterpret_cast<uint16_t*>(at + T * 128) = (uint16_t)(lo >> (16 * e));
            }
        }
    }
}

// One warp's share of a block's matrices: quarter qt of the TMEM lanes, its first or second warp m.  gram: TMEM address
// of [K; Q] K^T.
template <int NB, int PIECES>
__device__ __forceinline__ void warp_matrices(int qt, int m, uint32_t gram, char* a16, char* p16, float* diag, const GdnKeys& ky,
                                              const GdnRows& rw, uint32_t& flag, int lane) {
    const bool q = NB == 4 ? qt >= 2 : 2 * qt + m >= NB;
    int b, c0 = 0, c1, parts = 1;
    if constexpr (NB == 4) {
        b = qt & 1 ? m + 1 : (m == 0 ? 0 : 3);  // blocks 1 and 2, or 0 with the first product of 3 and the rest of 3
        c0 = b == 3 ? 1 : 0;
        parts = b == 0 ? 2 : 1;
    } else {
        b = q ? 2 * qt + m - NB : 2 * qt + m;
        if (b >= NB) return;
    }
    c1 = b + 1;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) {
        const int row = 16 * ((q ? NB : 0) + block_pos<NB>(b));
        block_matrices<NB, PIECES>(q, b, c0, c1, gram + ((uint32_t)row << 16), a16, p16, diag + b * 16 * kDiag, ky, rw, flag, lane);
        if (!q && p == 0) {
            __syncwarp();
            block_inverse<NB, PIECES>(b, a16, diag + b * 16 * kDiag, lane);
        }
        b = 3;  // the second part: the first product of block 3
        c0 = 0;
        c1 = 1;
    }
}

// One block and value feature pair in mma fragments (features g, g + 8; rows 8 n + 2 t, + 1): S k_i -> kHiLift R_b ahead
// of the blocks before, from v's fragments and the features' scales; and S q_i -> e^{G_i} S q_i.
template <int PIECES>
__device__ __forceinline__ void block_rhs(int bb, float (&ak)[2][4], const uint32_t (&v)[4], const float (&down)[2], const GdnRows& rw, int t) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int i = bb * 16 + n * 8 + 2 * t;
        float2 be = *reinterpret_cast<const float2*>(&rw.beta[i]);
        if constexpr (PIECES == 1) be = mul2(be, make_float2(kMatLift, kMatLift));
        const float2 ck = *reinterpret_cast<const float2*>(&rw.ck[i]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t v2 = v[2 * n + half];
            ak[n][2 * half] = be.x * (bf16_lo(v2) * down[half] - ck.x * ak[n][2 * half]);
            ak[n][2 * half + 1] = be.y * (bf16_hi(v2) * down[half] - ck.y * ak[n][2 * half + 1]);
        }
    }
}
__device__ __forceinline__ void block_rhs_q(int bb, float (&aq)[2][4], const GdnRows& rw, int t) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const float2 cq = *reinterpret_cast<const float2*>(&rw.cq[bb * 16 + n * 8 + 2 * t]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            aq[n][2 * half] *= cq.x;
            aq[n][2 * half + 1] *= cq.y;
        }
    }
}

// kHiLift R_b -> U_b: pieces in Uf, fp32 in u.  a16: shared address of the tiles.
template <int NB, int PIECES>
__device__ __forceinline__ void block_solve(int bb, const float (&ak)[2][4], uint32_t (&Uf)[PIECES][4], float (&u)[2][4], uint32_t a16,
                                            uint32_t& flag, int lane) {
    const int brow = ((lane >> 4) << 3) + (lane & 7), bch = (lane >> 3) & 1;
    constexpr int kLo = 16 * NB * 128;  // the lo pieces' tile
    uint32_t w[4], r[PIECES][4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const float a = ak[x >> 1][2 * (x & 1)], b = ak[x >> 1][2 * (x & 1) + 1];
        if constexpr (PIECES == 2) split2(a, b, r[0][x], r[1][x]);
        else r[0][x] = f16x2(a * (1.f / kMatLift), b * (1.f / kMatLift));
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[n][e] = 0.f;
    ldsm4(w, tile_at<128>(a16, bb * 16 + brow, 2 * bb + bch));
    mma_16816(u[0], r[0], w[0], w[1]);
    mma_16816(u[1], r[0], w[2], w[3]);
    if constexpr (PIECES == 2) {
        float v[2][4] = {};
        uint32_t w2[4];
        ldsm4(w2, tile_at<128>(a16 + kLo, bb * 16 + brow, 2 * bb + bch));
        mma_16816(v[0], r[1], w[0], w[1]);
        mma_16816(v[1], r[1], w[2], w[3]);
#pragma unroll
        for (int x = 0; x < 4; ++x) r[0][x] = lowered(r[0][x]);
        mma_16816(v[0], r[0], w2[0], w2[1]);
        mma_16816(v[1], r[0], w2[2], w2[3]);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[n][e] += v[n][e];
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const float a = u[x >> 1][2 * (x & 1)], b = u[x >> 1][2 * (x & 1) + 1];
        if constexpr (PIECES == 2) split2(a, b, Uf[0][x], Uf[1][x]);
        else Uf[0][x] = f16x2(a * (1.f / kMatLift), b * (1.f / kMatLift));
        watch(flag, Uf[0][x]);  // an R, A or inverse that is not finite ends here
    }
}
// acc -= kHiLift A_bc U_c for a block b after c (the tile holds -kHiLift A).
template <int NB, int PIECES>
__device__ __forceinline__ void block_update(int b, int c, float (&acc)[2][4], const uint32_t (&Uf)[PIECES][4], uint32_t a16, int lane) {
    const int brow = ((lane >> 4) << 3) + (lane & 7), bch = (lane >> 3) & 1;
    constexpr int kLo = 16 * NB * 128;
    uint32_t w[4];
    ldsm4(w, tile_at<128>(a16, b * 16 + brow, 2 * c + bch));
    mma_16816(acc[0], Uf[0], w[0], w[1]);
    mma_16816(acc[1], Uf[0], w[2], w[3]);
    if constexpr (PIECES == 2) {
        uint32_t w2[4];
        ldsm4(w2, tile_at<128>(a16 + kLo, b * 16 + brow, 2 * c + bch));
        mma_16816(acc[0], Uf[1], w[0], w[1]);
        mma_16816(acc[1], Uf[1], w[2], w[3]);
        uint32_t y[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) y[x] = lowered(Uf[0][x]);
        mma_16816(acc[0], y, w2[0], w2[1]);
        mma_16816(acc[1], y, w2[2], w2[3]);
    }
}
// acc += P_bc U_c.
__device__ __forceinline__ void block_out(int b, int c, float (&acc)[2][4], const uint32_t (&U)[4], uint32_t p16, int lane) {
    uint32_t w[4];
    ldsm4(w, tile_at<128>(p16, b * 16 + ((lane >> 4) << 3) + (lane & 7), 2 * c + ((lane >> 3) & 1)));
    mma_16816(acc[0], U, w[0], w[1]);
    mma_16816(acc[1], U, w[2], w[3]);
}

// One bf16 row of DK features, read by a whole warp, normalised: this lane's values of features lane + 32 e.
template <int DK>
__device__ __forceinline__ void unit_row(const uint16_t* src, float norm_eps, float scale, int lane, float (&x)[DK / 32]) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < DK / 32; ++e) {
        x[e] = bf16_bits_to_f32(src[lane + 32 * e]);
        ss = fmaf(x[e], x[e], ss);
    }
    float f = scale;
    if (norm_eps > 0.f) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        f = scale / sqrtf(ss + norm_eps);
    }
#pragma unroll
    for (int e = 0; e < DK / 32; ++e) x[e] *= f;
}

}  // namespace tsv
