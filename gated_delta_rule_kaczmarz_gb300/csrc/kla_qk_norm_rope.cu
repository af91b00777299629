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
// by fma, 48 bits) and kept as a 64-bit fixed-point fraction of a turn;
// multiplied by the integer position modulo 2^64 it loses nothing at any
// position, and its upper 32 bits go to sincospif.  The error is below
// 2^-47 turns per position, that is 1e-8 radians at position 10^6, where an
// fp32 product would be off by 0.03.  No fp64 instruction is used.
#include <cuda_bf16.h>

#include "kla_internal.h"

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

__device__ __forceinline__ void ld8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void unpack(const uint4 &v, float (&x)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// 8 features as loaded: one or two 16-byte words.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        v = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const { unpack(v, x); }
};
template <>
struct Raw<float> {
    float x[8];
    __device__ __forceinline__ void load(const float *p) { ld8(p, x); }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = x[i];
    }
};
__device__ __forceinline__ void st8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = reinterpret_cast<const uint32_t &>(h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void st8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// inv_freq / 2 pi, modulo one turn, as a 64-bit fraction.
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

// Cosines and sines of the token into cs[pair] (the warp's own array).
struct Angles {
    unsigned long long step[2];
    int axis[2];
    __device__ void init(const QkArgs &a, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int p = lane + 32 * i;
            step[i] = p < a.pairs ? turns_per_position(a.freq[p]) : 0ull;
            axis[i] = (p >= a.end[0]) + (p >= a.end[1]) + (p >= a.end[2]);
        }
    }
    __device__ __forceinline__ void write(const QkArgs &a, int lane, int t, float2 *cs) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int p = lane + 32 * i;
            if (p < a.pairs) {
                const long long pos = a.pos[(long long)axis[i] * a.tokens + t];
                const int top = (int)((step[i] * (unsigned long long)pos) >> 32);
                float s, c;
                sincospif((float)top * 0x1p-31f, &s, &c);
                cs[p] = make_float2(c, s);
            }
        }
    }
};

// (x0, x1): a lane's two runs; dir 1 turns forward, -1 back.
template <int D>
__device__ __forceinline__ void rotate(float (&x0)[8], float (&x1)[8], const Lane<D> &l,
                                       const float2 *cs, int pair_style, float dir) {
    if (!l.rotated) return;
    if (pair_style == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 c = cs[l.col0 + i];
            const float s = dir * c.y, u = x0[i], v = x1[i];
            x0[i] = u * c.x - v * s;
            x1[i] = v * c.x + u * s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 c = cs[l.pair0 + i];
            float s = dir * c.y, u = x0[2 * i], v = x0[2 * i + 1];
            x0[2 * i] = u * c.x - v * s;
            x0[2 * i + 1] = v * c.x + u * s;
            c = cs[l.pair1 + i];
            s = dir * c.y; u = x1[2 * i]; v = x1[2 * i + 1];
            x1[2 * i] = u * c.x - v * s;
            x1[2 * i + 1] = v * c.x + u * s;
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
__device__ __forceinline__ float inv_norm(float n2, int mode, float eps) {
    if (mode == 0) return 1.f;
    const float m = (mode == 1 ? n2 * (1.f / D) : n2) + eps;
    return m == 0.f ? 0.f : 1.f / sqrtf(m);      // a zero row with eps = 0 stays zero
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
qk_fwd_kernel(const __grid_constant__ QkArgs a) {
    constexpr int RW = 512 / D;                       // rows of a warp's group
    constexpr int U = sizeof(T) == 2 ? 4 : 2;         // groups loaded ahead
    __shared__ __align__(16) float2 cs_all[kWarps][64];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float2 *cs = cs_all[warp];
    const Lane<D> l(lane, a.pairs);
    Angles ang;
    ang.init(a, lane);
    const long long items = (long long)a.tokens * a.parts;
    for (long long it = (long long)blockIdx.x * kWarps + warp; it < items;
         it += (long long)gridDim.x * kWarps) {
        const int t = (int)(it / a.parts), part = (int)(it % a.parts);
        __syncwarp();
        ang.write(a, lane, t, cs);
        __syncwarp();
#pragma unroll 1
        for (int z = 0; z < 2; ++z) {
            const int H = a.heads[z];
            if (H == 0) continue;
            float w0[8], w1[8];
            const bool weighted = a.w[z] != nullptr;
            if (weighted) {
                ld8(a.w[z] + l.col0, w0);
                ld8(a.w[z] + l.col1, w1);
            }
            const T *x = static_cast<const T *>(a.x[z]) + (long long)t * a.xs[z];
            T *y = static_cast<T *>(a.y[z]) + (long long)t * a.ys[z];
            const int mode = a.norm[z];
            for (int h0 = part * RW; h0 < H; h0 += U * a.parts * RW) {
                Raw<T> r0[U], r1[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * a.parts * RW + l.row;
                    if (h < H) {
                        r0[u].load(x + h * D + l.col0);
                        r1[u].load(x + h * D + l.col1);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h0 + u * a.parts * RW >= H) break;      // the warp's whole group
                    const int h = h0 + u * a.parts * RW + l.row;
                    float x0[8], x1[8];
                    r0[u].get(x0);
                    r1[u].get(x1);
                    if (mode != 0) {
                        float n2 = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) n2 += x0[i] * x0[i] + x1[i] * x1[i];
                        const float r = inv_norm<D>(row_sum<D>(n2), mode, a.eps);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x0[i] *= r;
                            x1[i] *= r;
                        }
                    }
                    if (weighted) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x0[i] *= w0[i];
                            x1[i] *= w1[i];
                        }
                    }
                    rotate<D>(x0, x1, l, cs, a.pair_style, 1.f);
                    if (h < H) {
                        st8(y + h * D + l.col0, x0);
                        st8(y + h * D + l.col1, x1);
                    }
                }
            }
        }
    }
}

// The weight gradients are summed in registers over a warp's rows, then over
// the block, and leave as one partial sum per block: no atomics, so a result
// does not depend on the order in which blocks run.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
qk_bwd_kernel(const __grid_constant__ QkArgs a) {
    constexpr int RW = 512 / D;
    constexpr int U = sizeof(T) == 2 ? 2 : 1;
    __shared__ __align__(16) float2 cs_all[kWarps][64];
    __shared__ float part_w[kWarps][2][D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float2 *cs = cs_all[warp];
    const Lane<D> l(lane, a.pairs);
    Angles ang;
    ang.init(a, lane);
    float acc[2][16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.f;
    const long long items = (long long)a.tokens * a.parts;
    for (long long it = (long long)blockIdx.x * kWarps + warp; it < items;
         it += (long long)gridDim.x * kWarps) {
        const int t = (int)(it / a.parts), part = (int)(it % a.parts);
        __syncwarp();
        ang.write(a, lane, t, cs);
        __syncwarp();
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int H = a.heads[z];
            if (H == 0) continue;
            float w0[8], w1[8];
            const bool weighted = a.w[z] != nullptr;
            if (weighted) {
                ld8(a.w[z] + l.col0, w0);
                ld8(a.w[z] + l.col1, w1);
            }
            const T *x = static_cast<const T *>(a.x[z]) + (long long)t * a.xs[z];
            const T *g = static_cast<const T *>(a.g[z]) + (long long)t * a.gs[z];
            T *y = static_cast<T *>(a.y[z]) + (long long)t * a.ys[z];
            const int mode = a.norm[z];
            for (int h0 = part * RW; h0 < H; h0 += U * a.parts * RW) {
                Raw<T> rx0[U], rx1[U], rg0[U], rg1[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * a.parts * RW + l.row;
                    if (h < H) {
                        rx0[u].load(x + h * D + l.col0);
                        rx1[u].load(x + h * D + l.col1);
                        rg0[u].load(g + h * D + l.col0);
                        rg1[u].load(g + h * D + l.col1);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h0 + u * a.parts * RW >= H) break;
                    const int h = h0 + u * a.parts * RW + l.row;
                    float x0[8], x1[8], g0[8], g1[8];
                    rx0[u].get(x0);
                    rx1[u].get(x1);
                    rg0[u].get(g0);
                    rg1[u].get(g1);
                    rotate<D>(g0, g1, l, cs, a.pair_style, -1.f);
                    float r = 1.f;
                    if (mode != 0) {
                        float n2 = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) n2 += x0[i] * x0[i] + x1[i] * x1[i];
                        r = inv_norm<D>(row_sum<D>(n2), mode, a.eps);
                    }
                    if (weighted) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (h < H) {
                                acc[z][i] = fmaf(g0[i], x0[i] * r, acc[z][i]);
                                acc[z][8 + i] = fmaf(g1[i], x1[i] * r, acc[z][8 + i]);
                            }
                            g0[i] *= w0[i];
                            g1[i] *= w1[i];
                        }
                    }
                    if (mode != 0) {
                        float dot = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot += g0[i] * x0[i] + g1[i] * x1[i];
                        dot = row_sum<D>(dot) * r * r;
                        if (mode == 1) dot *= 1.f / D;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            g0[i] = r * (g0[i] - x0[i] * dot);
                            g1[i] = r * (g1[i] - x1[i] * dot);
                        }
                    }
                    if (h < H) {
                        st8(y + h * D + l.col0, g0);
                        st8(y + h * D + l.col1, g1);
                    }
                }
            }
        }
    }
    if (a.dw == nullptr) return;
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = acc[z][i];
#pragma unroll
            for (int o = 16; o >= D / 16; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (l.row == 0) part_w[warp][z][i < 8 ? l.col0 + i : l.col1 + i - 8] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += part_w[w][i / D][i % D];
        a.dw[(size_t)blockIdx.x * 2 * D + i] = v;
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

// Blocks that a launch may use: the partial sums of the backward pass are
// sized by it, so it depends on the problem alone.
constexpr int kMaxBlocks = 152 * 8;

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

int blocks_for(const QkArgs &a) {
    const long long want = ((long long)a.tokens * a.parts + kWarps - 1) / kWarps;
    return (int)(want < kMaxBlocks ? want : kMaxBlocks);
}

}  // namespace

size_t qk_bwd_workspace_bytes(const QkProblem &p) {
    if (p.tokens == 0) return 0;
    return (size_t)blocks_for(make_args(p)) * 2 * p.d * sizeof(float);
}

cudaError_t launch_qk_fwd(const QkProblem &p, cudaStream_t s) {
    const QkArgs a = make_args(p);
    const int blocks = blocks_for(a);
    if (p.dtype == 1) {
        if (p.d == 128) qk_fwd_kernel<__nv_bfloat16, 128><<<blocks, kThreads, 0, s>>>(a);
        else qk_fwd_kernel<__nv_bfloat16, 64><<<blocks, kThreads, 0, s>>>(a);
    } else {
        if (p.d == 128) qk_fwd_kernel<float, 128><<<blocks, kThreads, 0, s>>>(a);
        else qk_fwd_kernel<float, 64><<<blocks, kThreads, 0, s>>>(a);
    }
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_qk_bwd(const QkProblem &p, cudaStream_t s) {
    QkArgs a = make_args(p);
    const bool weights = p.dwq != nullptr || p.dwk != nullptr;
    a.dw = weights ? static_cast<float *>(p.ws) : nullptr;
    const int blocks = blocks_for(a);
    if (p.dtype == 1) {
        if (p.d == 128) qk_bwd_kernel<__nv_bfloat16, 128><<<blocks, kThreads, 0, s>>>(a);
        else qk_bwd_kernel<__nv_bfloat16, 64><<<blocks, kThreads, 0, s>>>(a);
    } else {
        if (p.d == 128) qk_bwd_kernel<float, 128><<<blocks, kThreads, 0, s>>>(a);
        else qk_bwd_kernel<float, 64><<<blocks, kThreads, 0, s>>>(a);
    }
    note_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !weights) return e;
    qk_dw_kernel<<<2 * p.d / 32, dim3(32, 32), 0, s>>>(a.dw, blocks, p.d, p.dwq, p.dwk);
    note_launch();
    return cudaGetLastError();
}

}  // namespace kla
