// Causal softmax attention on the CUDA cores (fp32 arithmetic throughout):
// fp32 inputs, and bf16 inputs whose groups are too large for a tensor-core
// tile.  Also the kernels that every path uses: the check and item tables of
// packed sequences, the join of a split key axis, the backward pass's row
// sums.
//
//   forward   s = scale q k^T, p = exp(s - m), o = p v / l, lse = m + log l,
//             with the running maximum m and sum l over tiles of 64 keys
//   backward  p = exp(s - lse), dp = go v^T, ds = p (dp - sum go o) scale,
//             dv = p^T go, dk = ds^T q (a block per key tile), dq = ds k (a
//             block per query tile): no atomics, a result does not depend on
//             the order of blocks
//
// 256 threads as 16 x 16; thread (ty, tx) holds the scores of rows ty + 16 i
// and keys tx + 16 j, and of the outputs rows ty + 16 i, features 4 tx + 64 j.
// Rows in shared memory are 4 floats longer than d, so that the 16-byte reads
// of 8 neighbouring keys fall into different banks.  A tile's rows are read
// from memory into registers a step ahead.  Bound by the issue of the products
// and by the reads of shared memory between them (a 16-byte read for 4 packed
// multiply-adds); few blocks: by the steps' latency, 4 to 5 us each.  fp32,
// forward and backward: B 1, T 256, 2 heads of 64 16 and 37 us; B 4, T 2048, 8
// heads of 64 0.49 and 1.66 ms (35 and 26 TFLOP/s); B 2, T 2048, 8 + 4 heads of
// 128 0.49 and 1.69 ms; single tokens of B 16, 16 + 4 heads of 128 over 4096
// keys 178 us.
//
// Blocks an SM, as measured (B 4, T 2048, 8 heads of 64 or B 2, 8 + 4 heads of
// 128): forward, tiles of 64 rows, d 64: one, 494 us (two 453, but 100 against
// 76 where there are fewer blocks than places), d 128: two, 491 (one 559; two cost
// fp32 172 bytes of spilled registers a thread and bf16 60, and pay all the same);
// backward, d 64: two, 1660 (one 2115), d 128: one, 1690 (two 2100).  Tiles of
// 16 rows: three at d 64 (one: 64 single tokens over 700 keys 244 us against 213), two
// at d 128 (backward, T 82 over 694 keys: 295 us against 315).
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "kla_attn.cuh"

namespace kla {
namespace {

using attn::Args;
using attn::Item;
using attn::Seq;

constexpr int kT = 256;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void st4(__nv_bfloat16 *p, float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(reinterpret_cast<const uint32_t &>(a),
                                               reinterpret_cast<const uint32_t &>(b));
}

// ROWS rows of a tile on their way to shared memory, a part of them in each
// thread's registers: asked for a step ahead, so that the wait for memory runs
// under the products of the step before.
template <typename T, int D, int ROWS>
struct Ahead {
    using Raw = std::conditional_t<sizeof(T) == 4, float4, uint2>;      // 4 features
    static constexpr int N = ROWS * D / 4 / kT;
    static_assert(N * kT * 4 == ROWS * D, "whole parts");
    Raw x[N];

    __device__ __forceinline__ void take(int z, const T *p, bool on) {
        x[z] = Raw{};
        if (on) x[z] = *reinterpret_cast<const Raw *>(p);
    }
    // Query-side rows (packed); zero past the sequence's last.
    __device__ __forceinline__ void rows(const T *src, long long stride, const Args &a,
                                         const Seq &q, int head, int row0) {
#pragma unroll
        for (int z = 0; z < N; ++z) {
            const int i = threadIdx.x + z * kT, row = row0 + i / (D / 4), c = i % (D / 4) * 4;
            const int tok = (int)((unsigned)row / (unsigned)a.G), g = row - tok * a.G;
            take(z, src + (q.q0 + tok) * stride + (long long)(head * a.G + g) * D + c, tok < q.lq);
        }
    }
    // Keys or values from j0; zero past the last.
    __device__ __forceinline__ void keys(const T *src, long long stride, const Seq &q, int head,
                                         int j0) {
#pragma unroll
        for (int z = 0; z < N; ++z) {
            const int i = threadIdx.x + z * kT, r = i / (D / 4), c = i % (D / 4) * 4;
            take(z, src + (q.k0 + j0 + r) * stride + (long long)head * D + c, j0 + r < q.lk);
        }
    }
    // Into dst[ROWS][D + 4].
    __device__ __forceinline__ void put(float *dst) const {
#pragma unroll
        for (int z = 0; z < N; ++z) {
            const int i = threadIdx.x + z * kT;
            *reinterpret_cast<float4 *>(dst + i / (D / 4) * (D + 4) + i % (D / 4) * 4) =
                ld4(reinterpret_cast<const T *>(&x[z]));
        }
    }
};

// acc[i][j] += sum_c A[ty + 16 i][c] B[tx + 16 j][c] over the D features, two
// products an instruction: even and odd features are summed apart.
template <int D, int MI, int NJ>
__device__ __forceinline__ void dots(const float *A, const float *B, float (&acc)[MI][NJ]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float2 s[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[i][j] = make_float2(acc[i][j], 0.f);
#pragma unroll 8
    for (int c = 0; c < D; c += 4) {
        float4 x[MI], y[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) x[i] = ld4(A + (ty + 16 * i) * (D + 4) + c);
#pragma unroll
        for (int j = 0; j < NJ; ++j) y[j] = ld4(B + (tx + 16 * j) * (D + 4) + c);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                s[i][j] = __ffma2_rn(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), s[i][j]);
                s[i][j] = __ffma2_rn(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), s[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = s[i][j].x + s[i][j].y;
}
// acc[i][:] += sum_n W[ty + 16 i][n] X[n][:], features 4 tx + 64 j; W has LD
// floats a row, N terms.
template <int D, int MI, int N, int LD>
__device__ __forceinline__ void mix(const float *W, const float *X, float4 (&acc)[MI][D / 64]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 4
    for (int n = 0; n < N; n += 4) {
        float4 w[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) w[i] = ld4(W + (ty + 16 * i) * LD + n);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const float4 x = ld4(X + (n + m) * (D + 4) + 4 * tx + 64 * j);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const float f = m == 0 ? w[i].x : m == 1 ? w[i].y : m == 2 ? w[i].z : w[i].w;
                    const float2 lo = __ffma2_rn(make_float2(f, f), make_float2(x.x, x.y),
                                                 make_float2(acc[i][j].x, acc[i][j].y));
                    const float2 hi = __ffma2_rn(make_float2(f, f), make_float2(x.z, x.w),
                                                 make_float2(acc[i][j].z, acc[i][j].w));
                    acc[i][j] = make_float4(lo.x, lo.y, hi.x, hi.y);
                }
            }
        }
    }
}

template <int D, int BM>
constexpr size_t fwd_smem() {
    return ((size_t)BM * (D + 4) + 64 * (D + 4) + BM * 68) * 4;
}

template <typename T, int D, int BM>
__global__ void __launch_bounds__(kT, D == 128 ? 2 : BM == 16 ? 3 : 1)
attn_simt_fwd_kernel(const __grid_constant__ Args a) {
    constexpr int MI = BM / 16;
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *KV = Q + BM * (D + 4), *P = KV + 64 * (D + 4);
    attn::clear_status(a);
    Item it;
    if (!attn::item_of(a, blockIdx.x, true, it)) return;
    const Seq s = attn::sequence(a, it.seq);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int row0 = it.tile * BM, rows = s.lq * a.G;
    const int seen = (min(row0 + BM, rows) - 1) / a.G + 1 + s.lk - s.lq;      // keys of the last row
    int begin, end;
    attn::split_range(seen > 0 ? (seen + 63) / 64 : 0, a.splits, it.split, begin, end);
    const T *key = static_cast<const T *>(a.k), *value = static_cast<const T *>(a.v);
    Ahead<T, D, BM> q;
    Ahead<T, D, 64> kv;
    q.rows(static_cast<const T *>(a.q), a.q_stride, a, s, it.head, row0);
    if (begin < end) kv.keys(key, a.k_stride, s, it.head, begin * 64);
    q.put(Q);
    int limit[MI];                                             // last key of each row
    float m[MI], l[MI];
    float4 acc[MI][D / 64];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int r = row0 + ty + 16 * i;
        limit[i] = r < rows ? r / a.G + s.lk - s.lq : -1;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int kb = begin; kb < end; ++kb) {
        __syncthreads();
        kv.put(KV);
        __syncthreads();
        kv.keys(value, a.v_stride, s, it.head, kb * 64);
        float x[MI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
        dots<D, MI, 4>(Q, KV, x);
        __syncthreads();
        kv.put(KV);
        if (kb + 1 < end) kv.keys(key, a.k_stride, s, it.head, kb * 64 + 64);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool on = kb * 64 + tx + 16 * j <= limit[i];
                x[i][j] = on ? x[i][j] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, x[i][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float base = mx == -INFINITY ? 0.f : mx;     // nothing seen yet
            const float shrink = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(x[i][j] - base);
                sum += p;
                P[(ty + 16 * i) * 68 + tx + 16 * j] = p;
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[i] = l[i] * shrink + sum;
            m[i] = mx;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                acc[i][j].x *= shrink; acc[i][j].y *= shrink;
                acc[i][j].z *= shrink; acc[i][j].w *= shrink;
            }
        }
        __syncthreads();
        mix<D, MI, 64, 68>(P, KV, acc);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int r = row0 + ty + 16 * i;
        if (r >= rows) continue;
        const long long tok = s.q0 + r / a.G;
        const int head = it.head * a.G + r % a.G;
        const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
        const float lse = l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
        long long at = (tok * a.Hq + head) * D;
        if (a.splits > 1) at += (long long)it.split * a.total_q * a.Hq * D;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            float4 x = acc[i][j];
            x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
            if (a.splits > 1) st4(a.o_part + at + 4 * tx + 64 * j, x);
            else st4(static_cast<T *>(a.out) + at + 4 * tx + 64 * j, x);
        }
        if (tx == 0) {
            if (a.splits > 1)
                a.lse_part[((long long)it.split * a.total_q + tok) * a.Hq + head] = lse;
            else if (a.lse)
                a.lse[tok * a.Hq + head] = lse;
        }
    }
}

// Scores and their gradients of BM rows by BN keys into P (p) and S (ds); the
// caller has the four tiles in shared memory.  Row r's lse and delta.
template <int D, int MI, int NJ>
__device__ __forceinline__ void grads_tile(const float *Q, const float *K, const float *G,
                                           const float *V, const int (&limit)[MI],
                                           const float (&lse2)[MI], const float (&delta)[MI],
                                           int j0, const Args &a, float (&p)[MI][NJ],
                                           float (&ds)[MI][NJ]) {
    const int tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) p[i][j] = ds[i][j] = 0.f;
    dots<D, MI, NJ>(Q, K, p);
    dots<D, MI, NJ>(G, V, ds);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const bool on = j0 + tx + 16 * j <= limit[i];
            p[i][j] = on ? exp2f(p[i][j] * a.scale_log2 - lse2[i]) : 0.f;
            ds[i][j] = on ? p[i][j] * (ds[i][j] - delta[i]) * a.scale : 0.f;
        }
}

template <int D, int BM>
constexpr size_t dq_smem() {
    return ((size_t)2 * BM * (D + 4) + 2 * 32 * (D + 4) + BM * 36) * 4;
}

template <typename T, int D, int BM>
__device__ void attn_simt_dq(const Args &a, int block, float *sm) {
    constexpr int MI = BM / 16;
    float *Q = sm, *G = Q + BM * (D + 4), *K = G + BM * (D + 4), *V = K + 32 * (D + 4),
          *S = V + 32 * (D + 4);
    Item it;
    if (!attn::item_of(a, block, true, it)) return;
    const Seq s = attn::sequence(a, it.seq);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int row0 = it.tile * BM, rows = s.lq * a.G;
    const int seen = (min(row0 + BM, rows) - 1) / a.G + 1 + s.lk - s.lq;
    const int tiles = seen > 0 ? (seen + 31) / 32 : 0;
    const T *key = static_cast<const T *>(a.k), *value = static_cast<const T *>(a.v);
    Ahead<T, D, BM> own;
    Ahead<T, D, 32> k, v;
    if (tiles > 0) {
        k.keys(key, a.k_stride, s, it.head, 0);
        v.keys(value, a.v_stride, s, it.head, 0);
    }
    own.rows(static_cast<const T *>(a.q), a.q_stride, a, s, it.head, row0);
    own.put(Q);
    own.rows(static_cast<const T *>(a.go), a.go_stride, a, s, it.head, row0);
    own.put(G);
    int limit[MI];
    float lse2[MI], delta[MI];
    float4 acc[MI][D / 64];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int r = row0 + ty + 16 * i;
        const bool on = r < rows;
        limit[i] = on ? r / a.G + s.lk - s.lq : -1;
        const long long at = (s.q0 + r / a.G) * a.Hq + it.head * a.G + r % a.G;
        lse2[i] = on ? a.lse_in[at] / kLn2 : 0.f;
        delta[i] = on ? attn::delta_of(a, at, limit[i] + 1) : 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int kb = 0; kb < tiles; ++kb) {
        __syncthreads();
        k.put(K);
        v.put(V);
        __syncthreads();
        if (kb + 1 < tiles) {
            k.keys(key, a.k_stride, s, it.head, kb * 32 + 32);
            v.keys(value, a.v_stride, s, it.head, kb * 32 + 32);
        }
        float p[MI][2], ds[MI][2];
        grads_tile<D, MI, 2>(Q, K, G, V, limit, lse2, delta, kb * 32, a, p, ds);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) S[(ty + 16 * i) * 36 + tx + 16 * j] = ds[i][j];
        __syncthreads();
        mix<D, MI, 32, 36>(S, K, acc);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int r = row0 + ty + 16 * i;
        if (r >= rows) continue;
        const long long at = ((s.q0 + r / a.G) * a.Hq + it.head * a.G + r % a.G) * D;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            st4(static_cast<T *>(a.dq) + at + 4 * tx + 64 * j, acc[i][j]);
    }
}

template <int D, int BN>
constexpr size_t dkv_smem() {
    return ((size_t)2 * BN * (D + 4) + 2 * 32 * (D + 4) + 2 * BN * 36) * 4;
}

// A block per key tile: all rows of the group that see one of its keys.  Here
// the tile's keys are the 16-row side: thread (ty, tx) has keys ty + 16 i and
// rows tx + 16 j.
template <typename T, int D, int BN>
__device__ void attn_simt_dkv(const Args &a, int block, float *sm) {
    constexpr int MI = BN / 16;
    float *K = sm, *V = K + BN * (D + 4), *Q = V + BN * (D + 4), *G = Q + 32 * (D + 4),
          *P = G + 32 * (D + 4), *S = P + BN * 36;
    Item it;
    if (!attn::item_of(a, block, false, it)) return;
    const Seq s = attn::sequence(a, it.seq);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int j0 = it.tile * BN;
    const T *query = static_cast<const T *>(a.q), *grad = static_cast<const T *>(a.go);
    const int rows = s.lq * a.G;
    const int first = max(0, j0 + s.lq - s.lk) * a.G / 32 * 32;   // rows of the first query that sees key j0
    Ahead<T, D, BN> own;
    Ahead<T, D, 32> q, g;
    float lse2[2], delta[2];
    int limit[2];
    const auto fetch = [&](int row0) {
        if (row0 >= rows) return;
        q.rows(query, a.q_stride, a, s, it.head, row0);
        g.rows(grad, a.go_stride, a, s, it.head, row0);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = row0 + tx + 16 * j, tok = r / a.G;
            const bool on = r < rows;
            limit[j] = on ? tok + s.lk - s.lq : -1;
            const long long at = (s.q0 + tok) * a.Hq + it.head * a.G + r % a.G;
            lse2[j] = on ? a.lse_in[at] / kLn2 : 0.f;
            delta[j] = on ? attn::delta_of(a, at, limit[j] + 1) : 0.f;
        }
    };
    fetch(first);
    own.keys(static_cast<const T *>(a.k), a.k_stride, s, it.head, j0);
    own.put(K);
    own.keys(static_cast<const T *>(a.v), a.v_stride, s, it.head, j0);
    own.put(V);
    float4 dk[MI][D / 64], dv[MI][D / 64];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < D / 64; ++j) dk[i][j] = dv[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int row0 = first; row0 < rows; row0 += 32) {
        __syncthreads();
        q.put(Q);
        g.put(G);
        __syncthreads();
        const float l[2] = {lse2[0], lse2[1]}, dl[2] = {delta[0], delta[1]};
        const int last[2] = {limit[0], limit[1]};
        fetch(row0 + 32);
        float p[MI][2], ds[MI][2];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) p[i][j] = ds[i][j] = 0.f;
        dots<D, MI, 2>(K, Q, p);
        dots<D, MI, 2>(V, G, ds);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int key = j0 + ty + 16 * i;
                const bool on = key <= last[j] && key < s.lk;
                const float pv = on ? exp2f(p[i][j] * a.scale_log2 - l[j]) : 0.f;
                P[(ty + 16 * i) * 36 + tx + 16 * j] = pv;
                S[(ty + 16 * i) * 36 + tx + 16 * j] =
                    on ? pv * (ds[i][j] - dl[j]) * a.scale : 0.f;
            }
        }
        __syncthreads();
        mix<D, MI, 32, 36>(P, G, dv);
        mix<D, MI, 32, 36>(S, Q, dk);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int key = j0 + ty + 16 * i;
        if (key >= s.lk) continue;
        const long long at = ((s.k0 + key) * a.Hk + it.head) * D;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            st4(static_cast<T *>(a.dk) + at + 4 * tx + 64 * j, dk[i][j]);
            st4(static_cast<T *>(a.dv) + at + 4 * tx + 64 * j, dv[i][j]);
        }
    }
}

// Both sides in one launch: the blocks of the key tiles first.
template <typename T, int D, int B>
__global__ void __launch_bounds__(kT, D == 64 || B == 16 ? 2 : 1)
attn_simt_bwd_kernel(const __grid_constant__ Args keys, const __grid_constant__ Args rows,
                     int key_blocks) {
    extern __shared__ __align__(16) float sm[];
    if ((int)blockIdx.x < key_blocks) attn_simt_dkv<T, D, B>(keys, blockIdx.x, sm);
    else attn_simt_dq<T, D, B>(rows, blockIdx.x - key_blocks, sm);
}

// ------------------------------------------------------- shared by all paths
// 16 bytes of a row, and what two such parts add to a dot product.
template <typename T>
__device__ __forceinline__ uint4 ld16(const T *p) { return *reinterpret_cast<const uint4 *>(p); }
template <typename T>
__device__ __forceinline__ float dot16(const uint4 &a, const uint4 &b, float sum) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            sum = fmaf(__uint_as_float(x[i]), __uint_as_float(y[i]), sum);
        } else {
            sum = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), sum);
            sum = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), sum);
        }
    }
    return sum;
}

constexpr int kDeltaRows = 2;
template <typename T, int D>
struct DeltaShape {
    static constexpr int V = 16 / (int)sizeof(T), L = D / V, ROWS = 256 / L * kDeltaRows;
};
// The sum over the L lanes of a row.
template <int L>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// delta = sum go o of every row: 16 bytes of it a lane, kDeltaRows rows a
// thread; bound by the bytes of o and go.
template <typename T, int D>
__device__ __forceinline__ void delta_rows(const Args &a, int block_index) {
    using S = DeltaShape<T, D>;
    const long long n = (long long)a.total_q * a.Hq;
    const long long block = (long long)block_index * S::ROWS;
    const int block_tok = n <= 0xffffffffll ? (int)((unsigned)block / (unsigned)a.Hq)
                                            : (int)(block / a.Hq);
    const int block_head = (int)(block - (long long)block_tok * a.Hq);
    const int lane = threadIdx.x % S::L;
    uint4 o[kDeltaRows], g[kDeltaRows];
    long long row[kDeltaRows];            // behind the last one: that one
#pragma unroll
    for (int r = 0; r < kDeltaRows; ++r) {
        row[r] = min(block + threadIdx.x / S::L + 256 / S::L * r, n - 1);
        const int x = block_head + (int)(row[r] - block);
        const long long at = (block_tok + x / a.Hq) * a.go_stride + (long long)(x % a.Hq) * D;
        o[r] = ld16(static_cast<const T *>(a.o) + row[r] * D + lane * S::V);
        g[r] = ld16(static_cast<const T *>(a.go) + at + lane * S::V);
    }
#pragma unroll
    for (int r = 0; r < kDeltaRows; ++r) {
        const float sum = sum_lanes<S::L>(dot16<T>(o[r], g[r], 0.f));
        if (lane == 0) a.delta[row[r]] = sum;
    }
}

// The same of the rows with few keys, as sum p dp.
template <typename T, int D>
__device__ __forceinline__ void few_rows(const Args &a, int block, int blocks) {
    using S = DeltaShape<T, D>;
    constexpr int GROUPS = 256 / S::L;
    const long long n = (long long)a.n_seq * attn::kFewKeys * a.Hq;
    const int lane = threadIdx.x % S::L;
    for (long long x0 = (long long)block * GROUPS; x0 < n; x0 += (long long)blocks * GROUPS) {
        const long long x = min(x0 + threadIdx.x / S::L, n - 1), y = x / a.Hq;
        const int head = (int)(x % a.Hq);
        const Seq q = attn::sequence(a, (int)(y / attn::kFewKeys));
        const int shift = q.lk - q.lq, i = (int)(y % attn::kFewKeys) + max(0, -shift);
        int keys = i + shift + 1;
        if (i >= q.lq || keys > attn::kFewKeys) keys = 0;
        const int most = __reduce_max_sync(0xffffffffu, keys);
        const long long row = (q.q0 + i) * a.Hq + head;
        const long long own = (long long)head * D + lane * S::V;
        const long long shared = (long long)(head / a.G) * D + lane * S::V;
        uint4 qx = make_uint4(0, 0, 0, 0), gx = qx;
        float l = 0.f, sum = 0.f;
        if (keys > 0) {
            qx = ld16(static_cast<const T *>(a.q) + (q.q0 + i) * a.q_stride + own);
            gx = ld16(static_cast<const T *>(a.go) + (q.q0 + i) * a.go_stride + own);
            l = a.lse_in[row] * 1.4426950408889634f;
        }
        for (int j = 0; j < most; ++j) {
            float score = 0.f, dp = 0.f;
            if (j < keys) {
                const T *k = static_cast<const T *>(a.k) + (q.k0 + j) * a.k_stride + shared;
                const T *v = static_cast<const T *>(a.v) + (q.k0 + j) * a.v_stride + shared;
                score = dot16<T>(qx, ld16(k), 0.f);
                dp = dot16<T>(gx, ld16(v), 0.f);
            }
            score = sum_lanes<S::L>(score);
            dp = sum_lanes<S::L>(dp);
            if (j < keys) sum = fmaf(exp2f(fmaf(score, a.scale_log2, -l)), dp, sum);
        }
        if (keys > 0 && lane == 0) a.delta_few[row] = sum;
    }
}

// The first blocks take the rows with few keys: their keys one after another
// take about as long as all other rows, and behind them (or looked for by the
// blocks of all rows, a search in packed sequences) they would come on top:
// 131072 rows of 128 take 16 us, 302316 of 64 18 us, against 25 and 30.  Six
// blocks an SM (40 registers): 16 us against 19 with 37 % of the threads.
template <typename T, int D>
__global__ void __launch_bounds__(256, 6) attn_delta_kernel(const __grid_constant__ Args a,
                                                         int few_blocks) {
    attn::clear_status(a);
    if (attn::rejected(a)) return;
    if ((int)blockIdx.x < few_blocks) few_rows<T, D>(a, blockIdx.x, few_blocks);
    else delta_rows<T, D>(a, blockIdx.x - few_blocks);
}

// o = sum_s exp(lse_s - lse) o_s, lse = log sum_s exp(lse_s): 16 lanes read a
// part's row, `per` such groups (a power of two up to 16) a row's parts, so that
// few rows of many parts do not wait for one read after another; the groups'
// sums meet in shared memory in a fixed order.  Bound by the latency of those
// reads: 16 tokens of 16 heads of 128 in 7 parts take 4.3 us, one in 38 parts 4.3
// (with one group a row 7.7 and 10.3).  Nothing is joined where the tables were
// refused or a wait ran out: parts are missing then.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ Args a, int per) {
    const unsigned status = *a.status;        // looked at last: its read runs under the others
    constexpr int MOST = attn::kMaxSplits / 16;
    __shared__ __align__(16) float part[16][D];
    const long long n = (long long)a.total_q * a.Hq;
    const int group = threadIdx.x / 16, lane = threadIdx.x % 16, sub = group % per;
    const long long row = (long long)blockIdx.x * (16 / per) + group / per, i = min(row, n - 1);
    float w[MOST], top = -INFINITY;
#pragma unroll
    for (int z = 0; z < MOST; ++z) {
        const int s = lane + 16 * z;
        w[z] = s < a.splits ? a.lse_part[s * n + i] : -INFINITY;
        top = fmaxf(top, w[z]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int z = 0; z < MOST; ++z) {
        w[z] = exp2f((w[z] - base) / kLn2);
        sum += w[z];
    }
    sum = sum_lanes<16>(sum);
    float4 acc[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    // the block's groups walk the same count of parts, so the shuffles are whole
    for (int s0 = 0; s0 < a.splits; s0 += per) {
        const int s = s0 + sub;
        float f = 0.f;
#pragma unroll
        for (int z = 0; z < MOST; ++z) {
            const float x = __shfl_sync(0xffffffffu, w[z], s % 16, 16);
            if (s / 16 == z) f = x;
        }
        if (s >= a.splits) continue;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const float4 v = ld4(a.o_part + (s * n + i) * D + 4 * lane + 64 * j);
            acc[j].x = fmaf(f, v.x, acc[j].x); acc[j].y = fmaf(f, v.y, acc[j].y);
            acc[j].z = fmaf(f, v.z, acc[j].z); acc[j].w = fmaf(f, v.w, acc[j].w);
        }
    }
    if (per > 1) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            *reinterpret_cast<float4 *>(&part[group][4 * lane + 64 * j]) = acc[j];
        __syncthreads();
        if (sub != 0) return;
        for (int x = 1; x < per; ++x)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const float4 v = ld4(&part[group + x][4 * lane + 64 * j]);
                acc[j].x += v.x; acc[j].y += v.y; acc[j].z += v.z; acc[j].w += v.w;
            }
    }
    if (row >= n || status != kDevOk) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        acc[j].x *= inv; acc[j].y *= inv; acc[j].z *= inv; acc[j].w *= inv;
        st4(static_cast<T *>(a.out) + i * D + 4 * lane + 64 * j, acc[j]);
    }
    if (lane == 0 && a.lse) a.lse[i] = sum == 0.f ? -INFINITY : base + logf(sum);
}

// One block: the check of both tables, then the items of up to two.  5 to 6 us,
// the latency of its reads and barriers.
__global__ void __launch_bounds__(1024)
attn_prep_kernel(const int *cu_q, const int *cu_k, int n, int total_q, int total_k, AttnTable t0,
                 AttnTable t1, unsigned *status) {
    __shared__ int base, warp_sum[32], off[1024], cnt[1024];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    int wrong = 0;                  // bits, not branches: the reads go out together
    if (tid == 0)
        wrong = (cu_q[0] != 0) | (cu_k[0] != 0) | (cu_q[n] != total_q) | (cu_k[n] != total_k);
    for (int i = tid; i < n; i += 1024)
        wrong |= (cu_q[i] > cu_q[i + 1]) | (cu_k[i] > cu_k[i + 1]);
    const bool bad = __syncthreads_or(wrong) != 0;
    if (tid == 0) *status = bad ? (unsigned)kDevBadSeqlens : (unsigned)kDevOk;
    if (bad) return;
    for (int z = 0; z < 2; ++z) {
        const AttnTable t = z == 0 ? t0 : t1;
        if (t.items == nullptr) continue;
        __syncthreads();
        if (tid == 0) base = 0;
        __syncthreads();
        for (int c = 0; c < n; c += 1024) {
            const int i = c + tid;
            int tiles = 0;
            if (i < n) {
                const long long len = t.cu[i + 1] - t.cu[i];
                tiles = (int)((len * t.mult + t.per - 1) / t.per);
            }
            int sum = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            if (lane == 31) warp_sum[warp] = sum;
            __syncthreads();
            if (warp == 0) {
                int w = warp_sum[lane];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, w, o);
                    if (lane >= o) w += up;
                }
                warp_sum[lane] = w;
            }
            __syncthreads();
            off[tid] = base + sum - tiles + (warp ? warp_sum[warp - 1] : 0);
            cnt[tid] = tiles;
            __syncthreads();
            if (tid == 0) base += warp_sum[31];
            for (int x = warp; x < 1024 && c + x < n; x += 32)
                for (int j = lane; j < cnt[x]; j += 32)
                    if (off[x] + j < t.entries)
                        t.items[off[x] + j] = make_int2(c + x, t.last_first ? cnt[x] - 1 - j : j);
            __syncthreads();
        }
        for (int j = base + tid; j < t.entries; j += 1024) t.items[j] = make_int2(-1, 0);
    }
}

// Key gradients of packed sequences without queries, if their tables passed.
__global__ void __launch_bounds__(256)
attn_zero_kernel(uint4 *dk, uint4 *dv, long long n, const unsigned *status) {
    if (*status != kDevOk) return;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        dk[i] = zero;
        dv[i] = zero;
    }
}

template <typename K, typename... A>
cudaError_t launch(K *kernel, long long blocks, size_t smem, cudaStream_t s, const A &...args) {
    if (blocks == 0) return cudaSuccess;
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)blocks, kT, smem, s>>>(args...);
    note_launch();
    return cudaGetLastError();
}

template <typename T, int D, int B>
cudaError_t launch_fwd(const Args &a, cudaStream_t s) {
    return launch(attn_simt_fwd_kernel<T, D, B>, (long long)a.items * a.splits * a.Hk,
                  fwd_smem<D, B>(), s, a);
}
template <typename T, int D, int B>
cudaError_t launch_bwd(const Args &keys, const Args &rows, cudaStream_t s) {
    const long long kb = (long long)keys.items * keys.Hk, rb = (long long)rows.items * rows.Hk;
    constexpr size_t smem = dkv_smem<D, B>() > dq_smem<D, B>() ? dkv_smem<D, B>() : dq_smem<D, B>();
    return launch(attn_simt_bwd_kernel<T, D, B>, kb + rb, smem, s, keys, rows, (int)kb);
}

}  // namespace

#define KLA_BY_TYPE(d, dtype, CALL)                                        \
    do {                                                                   \
        if ((dtype) == 1) {                                                \
            if ((d) == 128) { using T = __nv_bfloat16; constexpr int D = 128; CALL; } \
            else { using T = __nv_bfloat16; constexpr int D = 64; CALL; }  \
        } else {                                                           \
            if ((d) == 128) { using T = float; constexpr int D = 128; CALL; } \
            else { using T = float; constexpr int D = 64; CALL; }          \
        }                                                                  \
    } while (0)

cudaError_t launch_attn_simt_fwd(const Args &a, int rows, int d, int dtype, cudaStream_t s) {
    if (rows == 16) KLA_BY_TYPE(d, dtype, return (launch_fwd<T, D, 16>(a, s)));
    KLA_BY_TYPE(d, dtype, return (launch_fwd<T, D, 64>(a, s)));
}

cudaError_t launch_attn_simt_bwd(const Args &keys, const Args &rows, int tile, int d, int dtype,
                                 cudaStream_t s) {
    if (tile == 16) KLA_BY_TYPE(d, dtype, return (launch_bwd<T, D, 16>(keys, rows, s)));
    KLA_BY_TYPE(d, dtype, return (launch_bwd<T, D, 64>(keys, rows, s)));
}

cudaError_t launch_attn_delta(const Args &a, int d, int dtype, cudaStream_t s) {
    // 16-byte parts of a row; groups of lanes of a block, see DeltaShape
    const int parts = d * (dtype == 1 ? 2 : 4) / 16, groups = 256 / parts;
    const long long rows = (long long)a.total_q * a.Hq;
    const long long blocks = (rows + groups * kDeltaRows - 1) / (groups * kDeltaRows);
    long long few = 0;
    if (a.delta_few != a.delta && (a.cu_q || a.Tk - a.Tq < attn::kFewKeys))
        few = min(((long long)a.n_seq * attn::kFewKeys * a.Hq + groups - 1) / groups, 4096ll);
    KLA_BY_TYPE(d, dtype, (attn_delta_kernel<T, D><<<(unsigned)(few + blocks), 256, 0, s>>>(a, (int)few)));
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_attn_join(const Args &a, int d, int dtype, cudaStream_t s) {
    int per = 1;
    while (per < a.splits && per < 16) per *= 2;
    const long long blocks = ((long long)a.total_q * a.Hq * per + 15) / 16;
    KLA_BY_TYPE(d, dtype, (attn_join_kernel<T, D><<<(unsigned)blocks, 256, 0, s>>>(a, per)));
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_attn_zero(void *dk, void *dv, long long bytes, const unsigned *status,
                             cudaStream_t s) {
    const long long n = bytes / 16, blocks = (n + 255) / 256;
    attn_zero_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(
        static_cast<uint4 *>(dk), static_cast<uint4 *>(dv), n, status);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_attn_prep(const int *cu_q, const int *cu_k, int n, int total_q, int total_k,
                             const AttnTable &t0, const AttnTable &t1, unsigned *status,
                             cudaStream_t s) {
    attn_prep_kernel<<<1, 1024, 0, s>>>(cu_q, cu_k, n, total_q, total_k, t0, t1, status);
    note_launch();
    return cudaGetLastError();
}

}  // namespace kla
