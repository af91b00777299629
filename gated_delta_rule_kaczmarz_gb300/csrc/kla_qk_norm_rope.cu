// Query and key conditioning: a norm of every head's row and the rotary
// positions, in one pass over q and k, and its backward pass.
//
//   r = 1 / sqrt(mean x^2 + eps)  (rms),  1 / sqrt(sum x^2 + eps)  (l2),  1
//   y = x r w                     (w: a weight per feature, or none)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for pair i of rot/2,
//   angle = position of i's axis * inv_freq_i; features from rot on pass
//
// and with g the rotated-back gradient R^T dy:
//   dw = sum g x r,  u = g w,  dx = r (u - x r^2 c sum(u x)),  c = 1/d or 1.
//
// The pass is bound by HBM: every row is read once and written once (backward:
// x and dy read, dx written).  A row of d features is held by d/16 lanes, 16
// features each as two runs of 8 (16-byte accesses in bf16), so that a warp
// works on 512/d rows at a time, both features of every rotated pair lie in
// one lane, and a norm costs log2(d/16) shuffles.  A warp takes a token (or a
// part of its heads, when there are too few tokens to fill the GPU): the
// cosines and sines are computed once for it, spread over the lanes, and
// shared by its heads through shared memory.
//
// Angles: inv_freq / 2 pi is formed as the sum of two fp32 numbers (products
// by fma, 48 bits) and kept as a 64-bit fixed-point fraction of a turn; the
// integer position multiplies it modulo 2^64, and the upper 32 bits of that are
// rounded to fp32 and go to sincospif.  The fraction is off by less than 2^-49
// inv_freq turns per position (of the second number the rounding of its sum
// 2^-49.9, of its product 2^-51.2, of its constant 2^-52) and 2^-61: 1.2e-8
// radians at one radian and position 10^6, 2.4e-5 at the ends of int32.  The
// rounding adds 1e-7 radians at any position.  An fp32 product would be off by
// 0.03 at position 10^6.  (With 1 / 2 pi to 192 bits nothing but that rounding
// would be left, but each launch starts 0.5 us later.)  No fp64 instruction.
#include <cuda_bf16.h>

#include <cstdlib>

#include "kla_internal.h"
#include "kla_tc.cuh"

namespace kla {
namespace {

constexpr int kWarps = 4;          // warps of a block, forward and backward
constexpr int kThreads = kWarps * 32;

struct QkArgs {
    const void *x[2], *g[2];       // q, k; backward: gradients of the outputs
    void *y[2];                    // outputs; backward: dq, dk
    const float *w[2];
    float *dw;                     // backward: partial sums [blocks][2][d]
    const int *pos;                // [n_axes][tokens]
    const float *freq;             // [rot / 2]
    long long xs[2], gs[2], ys[2]; // elements between token rows
    int heads[2];
    int norm[2];
    int tokens, pairs, pair_style, parts;
    int end[3];                    // first pair of axes 1, 2 and 3
    float eps;
};

// 8 features as loaded and as four pairs for the packed fp32 instructions: the
// pass executes about 90 instructions for 1 KB of bf16 with them and 170
// without, where it was bound by their issue.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        v = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void get(float2 *x) const {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
};
template <>
struct Raw<float> {
    float4 u, v;
    __device__ __forceinline__ void zero() { u = v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p) {
        u = *reinterpret_cast<const float4 *>(p);
        v = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void get(float2 *x) const {
        x[0] = make_float2(u.x, u.y); x[1] = make_float2(u.z, u.w);
        x[2] = make_float2(v.x, v.y); x[3] = make_float2(v.z, v.w);
    }
};
__device__ __forceinline__ void st8(__nv_bfloat16 *p, const float2 *x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
        u[i] = reinterpret_cast<const uint32_t &>(h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void st8(float *p, const float2 *x) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}

// inv_freq / 2 pi, modulo one turn, as a 64-bit fraction; up to 2^26 radians (e
// stays below 2).
__device__ __forceinline__ unsigned long long turns_per_position(float f) {
    constexpr float kHi = 0x1.45f306p-3f, kLo = 0x1.b9391p-28f;   // 1 / 2 pi
    float p = f * kHi;
    const float e = fmaf(f, kHi, -p) + f * kLo;
    p -= rintf(p);
    const long long h = (long long)(p * 0x1p62f) + (long long)(e * 0x1p62f);
    return (unsigned long long)h << 2;
}

// What a lane holds of its rows, and where the pairs of those features are.
template <int D>
struct Lane {
    int row, col0, col1;     // row of the warp's group; first feature of each run
    int pair0, pair1;        // pair of the first feature of each run (pairs style)
    bool rotated;
    __device__ Lane(int lane, int pairs) {
        constexpr int LG = D / 16;
        const int j = lane % LG, m = pairs / 8;
        row = lane / LG;
        rotated = j < m;
        col0 = rotated ? 8 * j : 2 * pairs + 16 * (j - m);
        col1 = rotated ? pairs + 8 * j : col0 + 8;
        pair0 = col0 / 2;
        pair1 = col1 / 2;
    }
};

// Cosines and sines of a token: each lane computes those of two pairs and
// takes from the warp's array those of its own features, once for all heads.
struct Angles {
    unsigned long long step[2];
    long long at[2];          // of the pair's axis in the positions
    int pos[2];               // of the token to come, read ahead
    float2 c[4], s[4];        // of the lane's eight pairs
    __device__ void init(const QkArgs &a, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int p = lane + 32 * i;
            step[i] = p < a.pairs ? turns_per_position(a.freq[p]) : 0ull;
            at[i] = (long long)((p >= a.end[0]) + (p >= a.end[1]) + (p >= a.end[2])) * a.tokens;
        }
    }
    __device__ __forceinline__ void read(const QkArgs &a, int lane, int t) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 32 * i < a.pairs) pos[i] = a.pos[at[i] + t];
    }
    template <int D>
    __device__ __forceinline__ void turn(const QkArgs &a, int lane, const Lane<D> &l, float2 *cs) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int p = lane + 32 * i;
            if (p < a.pairs) {
                const int top = (int)((step[i] * (unsigned long long)(long long)pos[i]) >> 32);
                float sn, cn;
                sincospif((float)top * 0x1p-31f, &sn, &cn);
                cs[p] = make_float2(cn, sn);
            }
        }
        __syncwarp();
        if (!l.rotated) return;
        // half: pairs col0 .. col0 + 7; pairs: four from each run
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = a.pair_style == 0 ? l.col0 + 2 * i : i < 2 ? l.pair0 + 2 * i : l.pair1 + 2 * i - 4;
            const float4 v = *reinterpret_cast<const float4 *>(cs + p);
            c[i] = make_float2(v.x, v.z);
            s[i] = make_float2(v.y, v.w);
        }
    }
};

// x: a lane's two runs of four pairs; BACK turns back.
template <int D, bool BACK>
__device__ __forceinline__ void rotate(float2 (&x)[8], const Lane<D> &l, const Angles &g,
                                       int pair_style) {
    if (!l.rotated) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 c = g.c[i], m = make_float2(-g.s[i].x, -g.s[i].y);
        const float2 s = BACK ? m : g.s[i], n = BACK ? g.s[i] : m;      // sine, -sine
        if (pair_style == 0) {
            const float2 u = x[i], v = x[4 + i];
            x[i] = __ffma2_rn(v, n, __fmul2_rn(u, c));
            x[4 + i] = __ffma2_rn(u, s, __fmul2_rn(v, c));
        } else {
            const float2 u = x[2 * i], v = x[2 * i + 1];
            x[2 * i] = __ffma2_rn(make_float2(u.y, u.x), make_float2(n.x, s.x), __fmul2_rn(u, both(c.x)));
            x[2 * i + 1] = __ffma2_rn(make_float2(v.y, v.x), make_float2(n.y, s.y), __fmul2_rn(v, both(c.y)));
        }
    }
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int D>
__device__ __forceinline__ float row_dot(const float2 (&x)[8], const float2 (&y)[8]) {
    float2 a = __fmul2_rn(x[0], y[0]), b = __fmul2_rn(x[1], y[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        a = __ffma2_rn(x[i], y[i], a);
        b = __ffma2_rn(x[i + 1], y[i + 1], b);
    }
    a = __fadd2_rn(a, b);
    return row_sum<D>(a.x + a.y);
}
template <int D>
__device__ __forceinline__ float inv_norm(const float2 (&x)[8], int mode, float eps) {
    if (mode == 0) return 1.f;
    const float n2 = row_dot<D>(x, x), m = (mode == 1 ? n2 * (1.f / D) : n2) + eps;
    return m == 0.f ? 0.f : rsqrtf(m);      // a zero row with eps = 0 stays zero
}
// The weights of a lane's features.
template <int D>
__device__ __forceinline__ void load_weight(float2 (&w)[8], const float *p, const Lane<D> &l) {
    Raw<float> a, b;
    a.load(p + l.col0);
    b.load(p + l.col1);
    a.get(w);
    b.get(w + 4);
}

// The heads of one tensor (z: q, k) of a token: groups of 512 / D rows, `parts`
// apart, U of them loaded ahead.  x and y may be the same rows.
template <typename T, int D, int U>
__device__ __forceinline__ void forward_rows(const QkArgs &a, int z, const T *x, T *y, int part,
                                             int parts, const Lane<D> &l, const Angles &ang) {
    constexpr int RW = 512 / D;
    const int H = a.heads[z], mode = a.norm[z];
    float2 w[8];
    const bool weighted = a.w[z] != nullptr;
    if (weighted) load_weight<D>(w, a.w[z], l);
    for (int h0 = part * RW; h0 < H; h0 += U * parts * RW) {
        Raw<T> r0[U], r1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * parts * RW + l.row;
            if (h < H) {
                r0[u].load(x + h * D + l.col0);
                r1[u].load(x + h * D + l.col1);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u * parts * RW >= H) break;            // the warp's whole group
            const int h = h0 + u * parts * RW + l.row;
            float2 v[8];
            r0[u].get(v);
            r1[u].get(v + 4);
            if (mode != 0) {
                const float2 r = both(inv_norm<D>(v, mode, a.eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __fmul2_rn(v[i], r);
            }
            if (weighted) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __fmul2_rn(v[i], w[i]);
            }
            rotate<D, false>(v, l, ang, a.pair_style);
            if (h < H) {
                st8(y + h * D + l.col0, v);
                st8(y + h * D + l.col1, v + 4);
            }
        }
    }
}
// Their gradients: x and g into y, the weight's into acc.
template <typename T, int D, int U>
__device__ __forceinline__ void backward_rows(const QkArgs &a, int z, const T *x, const T *g, T *y,
                                              int part, int parts, const Lane<D> &l,
                                              const Angles &ang, float2 (&acc)[8]) {
    constexpr int RW = 512 / D;
    const int H = a.heads[z], mode = a.norm[z];
    float2 w[8];
    const bool weighted = a.w[z] != nullptr;
    if (weighted) load_weight<D>(w, a.w[z], l);
    for (int h0 = part * RW; h0 < H; h0 += U * parts * RW) {
        Raw<T> x0[U], x1[U], g0[U], g1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * parts * RW + l.row;
            if (h < H) {
                x0[u].load(x + h * D + l.col0);
                x1[u].load(x + h * D + l.col1);
                g0[u].load(g + h * D + l.col0);
                g1[u].load(g + h * D + l.col1);
            } else {                  // no row: adds nothing to the weights' gradients
                x0[u].zero(); x1[u].zero(); g0[u].zero(); g1[u].zero();
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u * parts * RW >= H) break;
            const int h = h0 + u * parts * RW + l.row;
            float2 v[8], d[8];
            x0[u].get(v);
            x1[u].get(v + 4);
            g0[u].get(d);
            g1[u].get(d + 4);
            rotate<D, true>(d, l, ang, a.pair_style);
            const float r = inv_norm<D>(v, mode, a.eps);
            if (weighted) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i] = __ffma2_rn(d[i], __fmul2_rn(v[i], both(r)), acc[i]);
                    d[i] = __fmul2_rn(d[i], w[i]);
                }
            }
            if (mode != 0) {
                float dot = row_dot<D>(d, v) * r * r;
                if (mode == 1) dot *= 1.f / D;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = __fmul2_rn(__ffma2_rn(v[i], both(-dot), d[i]), both(r));
            }
            if (h < H) {
                st8(y + h * D + l.col0, d);
                st8(y + h * D + l.col1, d + 4);
            }
        }
    }
}
// A block's sums of the weights' gradients, warp by warp in part_w, to its
// place among the partial sums.  No atomics: a result does not depend on the
// order in which blocks run.
template <int D>
__device__ __forceinline__ void leave_partial_sums(const QkArgs &a, const float2 (&acc)[2][8],
                                                   const Lane<D> &l, float *part_w, int warp,
                                                   int warps, int block) {
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i % 2 ? acc[z][i / 2].y : acc[z][i / 2].x;
#pragma unroll
            for (int o = 16; o >= D / 16; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (l.row == 0) part_w[(warp * 2 + z) * D + (i < 8 ? l.col0 + i : l.col1 + i - 8)] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += part_w[w * 2 * D + i];
        a.dw[(size_t)block * 2 * D + i] = v;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 4)
qk_fwd_kernel(const __grid_constant__ QkArgs a) {
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    __shared__ __align__(16) float2 cs_all[kWarps][64];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const Lane<D> l(lane, a.pairs);
    Angles ang;
    ang.init(a, lane);
    const int stride = gridDim.x * kWarps;
    int t = blockIdx.x * kWarps + warp;
    if (t < a.tokens) ang.read(a, lane, t);
    // (unsigned: the last step may pass 2^31)
    for (; (unsigned)t < (unsigned)a.tokens; t = (int)((unsigned)t + stride)) {
        ang.turn(a, lane, l, cs_all[warp]);
        if ((unsigned)t + stride < (unsigned)a.tokens) ang.read(a, lane, t + stride);
#pragma unroll 1
        for (int z = 0; z < 2; ++z)
            forward_rows<T, D, U>(a, z, static_cast<const T *>(a.x[z]) + (long long)t * a.xs[z],
                                  static_cast<T *>(a.y[z]) + (long long)t * a.ys[z], blockIdx.y,
                                  a.parts, l, ang);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 3)
qk_bwd_kernel(const __grid_constant__ QkArgs a) {
    constexpr int U = sizeof(T) == 2 ? 2 : 1;
    __shared__ __align__(16) float2 cs_all[kWarps][64];
    __shared__ float part_w[kWarps * 2 * D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const Lane<D> l(lane, a.pairs);
    Angles ang;
    ang.init(a, lane);
    float2 acc[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = both(0.f);
    const int stride = gridDim.x * kWarps;
    int t = blockIdx.x * kWarps + warp;
    if (t < a.tokens) ang.read(a, lane, t);
    for (; (unsigned)t < (unsigned)a.tokens; t = (int)((unsigned)t + stride)) {
        ang.turn(a, lane, l, cs_all[warp]);
        if ((unsigned)t + stride < (unsigned)a.tokens) ang.read(a, lane, t + stride);
#pragma unroll
        for (int z = 0; z < 2; ++z)
            backward_rows<T, D, U>(a, z, static_cast<const T *>(a.x[z]) + (long long)t * a.xs[z],
                                   static_cast<const T *>(a.g[z]) + (long long)t * a.gs[z],
                                   static_cast<T *>(a.y[z]) + (long long)t * a.ys[z], blockIdx.y,
                                   a.parts, l, ang, acc[z]);
    }
    if (a.dw != nullptr)
        leave_partial_sums<D>(a, acc, l, part_w, warp, kWarps, blockIdx.y * gridDim.x + blockIdx.x);
}

// ------------------------------------------------------------ many tokens
// A warp walks whole tokens; their rows come by bulk copies into a ring of
// stages of its own in shared memory, are worked on in place and leave by bulk
// copies, so that HBM is busy while a warp computes.  The kernels above keep a
// token's rows in registers: a warp's loads then wait for its arithmetic.
struct Pipe {
    int warps, stages;               // of a block
    uint32_t bytes[2];               // a token's rows of q and of k
    uint32_t stage;                  // bytes of a stage: x, and for the backward g
    bool lost_wait;                  // test hook: as if every warp's first wait had run out
};
constexpr int kPipeMost = 16;        // warps of a block, forward; backward 12 (registers)
constexpr size_t kPipeSmem = 200 * 1024;

// A copy did not come within the bound: there is no status word, so the rows that
// are left to the warp become NaN (as do the weights' gradients).
template <typename T, int D>
__device__ __noinline__ void lost_rows(const QkArgs &a, int lane, long long t, unsigned stride) {
    const float2 nan = both(__int_as_float(0x7fffffff)), row[4] = {nan, nan, nan, nan};
    for (; t < a.tokens; t += stride)
        for (int z = 0; z < 2; ++z)
            for (int c = lane * 8; c < a.heads[z] * D; c += 256)
                st8(static_cast<T *>(a.y[z]) + t * a.ys[z] + c, row);
}

template <typename T, int D, bool BACK>
__global__ void __launch_bounds__(BACK ? 384 : kPipeMost * 32, 1)
qk_pipe_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ Pipe p) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kPipeMost][4];
    __shared__ __align__(16) float2 cs_all[kPipeMost][64];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, S = p.stages;
    unsigned char *ring = smem + (size_t)warp * S * p.stage;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) tc::mbar_init(&full[warp][i], 1);
        tc::fence_mbar_init();
    }
    __syncwarp();
    const Lane<D> l(lane, a.pairs);
    Angles ang;
    ang.init(a, lane);
    float2 acc[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = both(0.f);
    const unsigned first = blockIdx.x * p.warps + warp, stride = gridDim.x * p.warps;
    const unsigned tokens = a.tokens;
    const int n = first < tokens ? (int)((tokens - 1 - first) / stride) + 1 : 0;   // of this warp

    const auto load = [&](int i, int s) {       // one lane: the warp's i-th token
        const long long t = first + (long long)i * stride;
        unsigned char *dst = ring + (size_t)s * p.stage;
        tc::mbar_expect_tx(&full[warp][s], p.stage);
#pragma unroll
        for (int g = 0; g < (BACK ? 2 : 1); ++g)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                if (p.bytes[z] == 0) continue;
                const T *src = g ? static_cast<const T *>(a.g[z]) + t * a.gs[z]
                                 : static_cast<const T *>(a.x[z]) + t * a.xs[z];
                tc::bulk_load(dst, src, p.bytes[z], &full[warp][s]);
                dst += p.bytes[z];
            }
    };
    if (lane == 0)
        for (int i = 0; i < S - 1 && i < n; ++i) load(i, i);
    if (n > 0) ang.read(a, lane, (int)first);
    int s = 0, use = 0, i = 0;
    const int walk = p.lost_wait ? 0 : n;
    for (; i < walk; ++i) {
        const long long t = first + (long long)i * stride;
        ang.turn(a, lane, l, cs_all[warp]);
        if (i + 1 < n) ang.read(a, lane, (int)(t + stride));
        // the warp's own copy: it comes, and the bound is not met
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[warp][s], use & 1))) break;
        unsigned char *row = ring + (size_t)s * p.stage;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            T *x = reinterpret_cast<T *>(row + (z ? p.bytes[0] : 0));
            if (BACK)
                backward_rows<T, D, 1>(a, z, x,
                                       reinterpret_cast<T *>(reinterpret_cast<unsigned char *>(x) +
                                                             p.bytes[0] + p.bytes[1]),
                                       x, 0, 1, l, ang, acc[z]);
            else
                forward_rows<T, D, 2>(a, z, x, x, 0, 1, l, ang);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
            for (int z = 0; z < 2; ++z)
                if (p.bytes[z])
                    tc::bulk_store(static_cast<T *>(a.y[z]) + t * a.ys[z],
                                   row + (z ? p.bytes[0] : 0), p.bytes[z]);
            tc::bulk_commit_group();
            // the stage of the token before is free once its rows have left
            if (i + S - 1 < n) {
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                load(i + S - 1, s == 0 ? S - 1 : s - 1);
            }
        }
        if (++s == S) {
            s = 0;
            ++use;
        }
    }
    if (lane == 0) {
        for (int j = i; j < n && j < i + S - 1; ++j)       // a copy that had not come
            (void)tc::mbar_wait(&full[warp][j % S], (j / S) & 1);
        tc::bulk_wait_group0();
    }
    if (i < n) {
        lost_rows<T, D>(a, lane, first + (long long)i * stride, stride);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[0][j] = acc[1][j] = both(__int_as_float(0x7fffffff));
    }
    if (BACK && a.dw != nullptr) {
        __syncthreads();       // the rings are done with: the warps' sums take their place
        leave_partial_sums<D>(a, acc, l, reinterpret_cast<float *>(smem), warp, p.warps, blockIdx.x);
    }
}

// dw[i] = sum over the blocks' partial sums, in a fixed order.
__global__ void __launch_bounds__(1024)
qk_dw_kernel(const float *part, int blocks, int d, float *dwq, float *dwk) {
    __shared__ float s[32][33];
    const int col = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    for (int b = threadIdx.y; b < blocks; b += 32) v += part[(size_t)b * 2 * d + col];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += s[i][threadIdx.x];
        float *dw = col < d ? dwq : dwk;
        if (dw) dw[col < d ? col : col - d] = v;
    }
}

// Blocks of a launch: as many as are resident at once, so that none starts late
// and a warp's start is paid once.  30011 tokens of 16 + 16 heads of 128 in bf16
// take 93 us (backward 160), with three (four) times as many blocks 95 (170).
// The partial sums of the backward pass are sized by it, so it depends on the
// problem alone.
constexpr int kBlocksFwd = 152 * 4, kBlocksBwd = 152 * 3;

// A warp takes a token's heads in `parts` parts: one when the tokens alone
// give every SM 32 warps (the cosines are then computed once a token), else as
// many as there are groups of rows, so that a decode batch spreads over the SMs.
int parts_for(const QkProblem &p) {
    if (p.tokens >= 152 * 32) return 1;
    const int rw = 512 / p.d;
    const int groups = ((p.Hq > p.Hk ? p.Hq : p.Hk) + rw - 1) / rw;
    const int want = (152 * 32 + p.tokens - 1) / p.tokens;
    return want < groups ? want : groups;
}

QkArgs make_args(const QkProblem &p) {
    QkArgs a{};
    a.x[0] = p.q; a.x[1] = p.k; a.g[0] = p.gq; a.g[1] = p.gk;
    a.y[0] = p.q_out; a.y[1] = p.k_out; a.w[0] = p.wq; a.w[1] = p.wk;
    a.xs[0] = p.q_stride; a.xs[1] = p.k_stride; a.gs[0] = p.gq_stride; a.gs[1] = p.gk_stride;
    a.ys[0] = p.qo_stride; a.ys[1] = p.ko_stride;
    a.heads[0] = p.Hq; a.heads[1] = p.Hk; a.norm[0] = p.norm_q; a.norm[1] = p.norm_k;
    a.pos = p.positions; a.freq = p.inv_freq; a.tokens = p.tokens; a.pairs = p.rot / 2;
    a.pair_style = p.style; a.eps = p.eps; a.parts = parts_for(p);
    int end = 0;
    for (int i = 0; i < 3; ++i) {
        end = i < p.n_axes ? end + p.sections[i] : a.pairs;
        a.end[i] = i + 1 < p.n_axes ? end : 1 << 30;     // no axis beyond the last
    }
    return a;
}

// Blocks over the tokens, and their parts beside.
dim3 blocks_for(const QkArgs &a, bool back) {
    const int want = (a.tokens - 1) / kWarps + 1;
    const int most = ((back ? kBlocksBwd : kBlocksFwd) - 1) / a.parts + 1;
    return dim3((unsigned)(want < most ? want : most), (unsigned)a.parts);
}

// The pipelined kernel's shape, or warps = 0 where it does not pay: it wants 12
// warps of three stages in a block's shared memory (backward: 8 of two), and 4
// tokens for each.  32768 tokens of 16 + 4 heads of 128 in bf16 take 70 us with
// it and 74 without (backward 114 and 123), of head size 64 46 and 55 (66 and
// 80); 65536 of 12 + 12 heads of 128, the backward's 8 warps, 260 and 284; with
// rows of 16 + 16 heads, where it has 8 warps, 106 and 93 (backward, 6 warps,
// 196 and 160).  Both are bound by the warps' own latency, at about half of the
// issue slots; a copy alone would take 51 us.
Pipe pipe_for(const QkProblem &p, bool back) {
    Pipe r{};
    const uint32_t row = (uint32_t)p.d * (p.dtype == 1 ? 2 : 4);
    r.bytes[0] = p.Hq * row;
    r.bytes[1] = p.Hk * row;
    r.stage = (r.bytes[0] + r.bytes[1]) * (back ? 2 : 1);
    const int most = back ? 12 : kPipeMost;
    for (r.stages = 3; r.stages >= (back ? 2 : 3); --r.stages) {
        const size_t fit = kPipeSmem / ((size_t)r.stages * r.stage);
        r.warps = fit < (size_t)most ? (int)fit : most;
        if (r.warps >= (r.stages == 3 ? 12 : 8)) {
            if (p.tokens < 4 * 152 * r.warps) break;
            return r;
        }
    }
    r.warps = 0;
    return r;
}

template <typename T, int D, bool BACK>
cudaError_t launch_pipe(const QkArgs &a, const Pipe &p, cudaStream_t s) {
    const void *kernel = reinterpret_cast<const void *>(qk_pipe_kernel<T, D, BACK>);
    cudaError_t e = allow_dynamic_smem(kernel, kPipeSmem);
    if (e != cudaSuccess) return e;
    size_t smem = (size_t)p.warps * p.stages * p.stage;
    const size_t sums = (size_t)p.warps * 2 * D * sizeof(float);
    if (BACK && smem < sums) smem = sums;
    Pipe q = p;
    q.lost_wait = std::getenv("KLA_TEST_LOST_WAIT") != nullptr;
    qk_pipe_kernel<T, D, BACK><<<152, p.warps * 32, smem, s>>>(a, q);
    note_launch();
    return cudaGetLastError();
}
template <typename T, int D, bool BACK>
cudaError_t launch_rows(const QkArgs &a, cudaStream_t s) {
    if (BACK) qk_bwd_kernel<T, D><<<blocks_for(a, BACK), kThreads, 0, s>>>(a);
    else qk_fwd_kernel<T, D><<<blocks_for(a, BACK), kThreads, 0, s>>>(a);
    note_launch();
    return cudaGetLastError();
}
template <bool BACK>
cudaError_t launch_qk(const QkProblem &p, const QkArgs &a, const Pipe &pipe, cudaStream_t s) {
    const bool on = pipe.warps > 0;
    if (p.dtype == 1) {
        using T = __nv_bfloat16;
        if (p.d == 128) return on ? launch_pipe<T, 128, BACK>(a, pipe, s) : launch_rows<T, 128, BACK>(a, s);
        return on ? launch_pipe<T, 64, BACK>(a, pipe, s) : launch_rows<T, 64, BACK>(a, s);
    }
    if (p.d == 128) return on ? launch_pipe<float, 128, BACK>(a, pipe, s) : launch_rows<float, 128, BACK>(a, s);
    return on ? launch_pipe<float, 64, BACK>(a, pipe, s) : launch_rows<float, 64, BACK>(a, s);
}

}  // namespace

// Partial sums of the weights' gradients.  The pipelined kernel's 152 blocks
// need no more than the others' over as many tokens.
size_t qk_bwd_workspace_bytes(const QkProblem &p) {
    if (p.tokens == 0) return 0;
    const dim3 b = blocks_for(make_args(p), true);
    return (size_t)b.x * b.y * 2 * p.d * sizeof(float);
}

cudaError_t launch_qk_fwd(const QkProblem &p, cudaStream_t s) {
    return launch_qk<false>(p, make_args(p), pipe_for(p, false), s);
}

cudaError_t launch_qk_bwd(const QkProblem &p, cudaStream_t s) {
    QkArgs a = make_args(p);
    const bool weights = p.dwq != nullptr || p.dwk != nullptr;
    a.dw = weights ? static_cast<float *>(p.ws) : nullptr;
    const Pipe pipe = pipe_for(p, true);
    cudaError_t e = launch_qk<true>(p, a, pipe, s);
    if (e != cudaSuccess || !weights) return e;
    const dim3 b = blocks_for(a, true);
    qk_dw_kernel<<<2 * p.d / 32, dim3(32, 32), 0, s>>>(a.dw, pipe.warps ? 152 : (int)(b.x * b.y), p.d,
                                                       p.dwq, p.dwk);
    note_launch();
    return cudaGetLastError();
}

}  // namespace kla
