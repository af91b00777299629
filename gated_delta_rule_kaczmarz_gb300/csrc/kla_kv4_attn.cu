// Causal attention of few query rows over the 4-bit paged cache.
//
//   s = scale <q, k>,  p = exp2(s log2 e - base),  o = sum p v / sum p
//
// Work.  Keys go in tiles of 64 (four blocks of the cache).  A work item is a
// sequence, key head and group of 8 or 16 query rows (the heads of a key head and
// the call's tokens, packed); all items' tiles in a row are cut into equal parts,
// one for each warp of one CTA an SM, so lengths may differ as they like.  A warp
// keeps its own running base, sums and outputs and brings its tiles by bulk copies
// through a ring of its own: warps wait for nobody.  What the warps of a CTA hold of
// the same item is joined in shared memory, a warp for each row; items that reach
// over a CTA's edge, at most one for each CTA, are left to a second kernel.
//
// Products.  S^T = K Q^T and O^T = V^T P^T as m16n8k16: 16 keys (16 features)
// against 8 query rows, so that 4 rows of a decode batch fill half of an operand
// where 16 rows a tile would leave it to a quarter.  16 bytes of shared memory are a
// thread's part of the operand for all products of a block, whichever features the
// hardware takes them for: Q is laid out, and O written back, in the same order.
// Codes become fp16 by the hardware's conversion and one multiplication by the
// scale, exactly.  q is one (bf16) or two (fp32) fp16 terms after a power of two for
// each row, p is rounded to fp16 once (bf16) or split in two (fp32); sums are fp32.
//
// Measured (16 + 4 heads of 128, bf16, one token): 16 contexts of 16384 to 32768
// 45.5 us, 256 of up to 4096 58.0, 0.78 and 0.79 of measured HBM bandwidth.  The tiles
// themselves run at 6.8 TB/s; the first are asked for 1.8 us after the start (length,
// table: reads that wait for each other, and the place between them), a CTA's last warp is
// done 2 to 3 us behind the others (a tile is a warp's), the CTA's join takes 1.2 to 2 and
// the second kernel 2.5.  What runs once is bound by fetching its instructions, so it is short.
// 221 KB of ring in flight an SM are needed: 147 KB took 56 us, 110 KB 61, where this took
// 50.5 (an earlier form, as are the next figures).  12 warps of 64 keys and
// two stages; 16 warps of 32 keys 53.0, 11 of 64 53.0.  tcgen05 takes e2m1 with its
// scales along the contracted axis: that is so of the keys, not of the values.
#include <cuda_bf16.h>

#include <atomic>
#include <cstdlib>

#include "kla_attn.cuh"
#include "kla_kv4.cuh"
#include "kla_launch.cuh"
#include "kla_tc.cuh"

namespace kla {
namespace {

using kv4::kBlock;
using kv4::divided;
using kv4::Divisor;
using kv4::divisor;
using kv4::Layout;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
// p = 2^(s - m + kTop) with a base m that follows the maximum only when that is
// kLag above it: a row's largest p is 2^7 to 2^15 (fp16 ends at 2^16), what is 2^-21 of
// it is still a normal number, and below that p is off by 2^-32 of it at most.
constexpr float kTop = 7.f, kLag = 8.f;
// From so many tiles to a warp on an item counts as a tile more in the split.  Both, in us:
// 16 contexts (14 tiles a warp) 46.9 and 47.1, 256 contexts (19) 61.7 and 60.0, drafted tokens
// (4) 24.7 and 23.5; a tile a warp 6.4 and 6.7.  Two tiles more: 47.1, 60.2 and 23.2, three
// 47.8, 61.8 and 23.1.
constexpr unsigned kMany = 2;

// NT: tiles of 8 query rows.
template <int D, int NT, bool F32>
struct Config {
    static constexpr int kWarps = F32 || NT > 1 ? 8 : 12;        // as the registers allow
    static constexpr int kTile = 64;                             // keys of a stage
    static constexpr int kKeys = 32;                             // of a step of the softmax
    static constexpr int kBlocks = kTile / kBlock;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRows = 8 * NT;
    static constexpr int kStage = kBlocks * Layout<D>::kBytes;
    static constexpr int kFit = 221184 / kWarps / kStage, kStages = kFit < 6 ? kFit : 6;
    static constexpr int kRing = kStages * kStage;               // of a warp
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kStages >= 2 && kStage >= (kRows * (D + 2) + 3) * 4, "a part lies in a stage");
};

// An item that began in CTA `from` and ends in this one: joined by the second kernel.
struct Owner {
    int seq, item, from;         // seq < 0: none
};

struct Args {
    const void *q;
    long long q_stride;
    const unsigned char *pool;
    const int *table, *lens;
    void *o;
    float *lse;
    int B, Tq, Hq, Hk, G, d, blocks, n_pages, columns;     // blocks: of 16 tokens in a page
    int rows, groups, items;     // query rows of a key head, their groups, items of a sequence
    Divisor by_G, by_groups, by_items, by_blocks;
    float scale_log2, v_unit;
    int part_rows;               // rows of a part: of a group, as far as there are
    int part_size;               // floats of a part, in whole 16 bytes
    unsigned *status;
    unsigned *cta_status;        // [CTAs]
    Owner *owners;               // [CTAs]
    float *part;                 // [CTAs][2 + warps][part_size]: of the CTA's first and last item,
                                 // and what each warp closed
    int ctas;
    bool lost_wait;              // test hook
};

// ------------------------------------------------------------------ the split
// Tile u of all (fewer than 2^31): items in order, their tiles in order.
struct Split {
    unsigned total;
    int ctas;
    unsigned each, rest;         // floor(total c / ctas) = each c + floor(rest c / ctas)
    __device__ unsigned cta(int c) const { return each * (unsigned)c + rest * (unsigned)c / (unsigned)ctas; }
};
template <int WARPS>
__device__ __forceinline__ Split split_of(const Args &a, unsigned tiles) {
    Split s;
    s.total = tiles * (unsigned)a.items;
    const unsigned most = (s.total + WARPS - 1) / WARPS;        // a tile for each warp at least
    s.ctas = most < (unsigned)a.ctas ? (most > 0 ? (int)most : 1) : a.ctas;
    s.each = s.total / (unsigned)s.ctas;
    s.rest = s.total - s.each * (unsigned)s.ctas;
    return s;
}
__device__ __forceinline__ int length(const Args &a, int b) {
    const int n = a.lens[b], most = a.columns * a.blocks * kBlock;
    return n < 0 ? 0 : (n < most ? n : most);
}
template <int TILE>
__device__ __forceinline__ int tiles_of(int len) { return (len + TILE - 1) / TILE; }

// ------------------------------------------------------------------ products
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return reinterpret_cast<const uint32_t &>(h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t h) {
    return __half22float2(reinterpret_cast<const __half2 &>(h));
}

// A bulk copy of what is read once (`once`), which need not push anything out of L2, or of
// what other groups of rows read too.
__device__ __forceinline__ uint64_t policy_of(bool once) {
    uint64_t first, normal;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
    return once ? first : normal;
}
__device__ __forceinline__ void load_block(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
        ::"r"(tc::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(tc::smem_u32(bar)),
        "l"(policy)
        : "memory");
}

template <int N>
__device__ __forceinline__ void load_words(const unsigned char *p, uint32_t (&w)[N]) {
    if (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[N - 2] = v.z; w[N - 1] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    }
}

__device__ __forceinline__ void store2(float *p, float x, float y) {
    *reinterpret_cast<float2 *>(p) = make_float2(x, y);
}
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float x, float y) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}
// A fourth of a query row.
template <typename T, int D>
struct Query {
    uint4 w[D / 16 * sizeof(T) / 4];
    __device__ __forceinline__ void load(const T *p, bool there) {
#pragma unroll
        for (int i = 0; i < D / 16 * (int)sizeof(T) / 4; ++i)
            w[i] = there ? reinterpret_cast<const uint4 *>(p)[i] : make_uint4(0, 0, 0, 0);
    }
    // four features from 4 j on
    __device__ __forceinline__ void get(int j, float (&x)[4]) const {
        if (sizeof(T) == 4) {
            const uint4 v = w[j];
            x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
            x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
        } else {
            const uint4 v = w[j / 2];
            const uint32_t lo = j % 2 ? v.z : v.x, hi = j % 2 ? v.w : v.y;
            x[0] = __uint_as_float(lo << 16); x[1] = __uint_as_float(lo & 0xffff0000u);
            x[2] = __uint_as_float(hi << 16); x[3] = __uint_as_float(hi & 0xffff0000u);
        }
    }
};

// Output row of row n of a group: its offset in [B, Tq, Hq], or -1 behind the last.
__device__ __forceinline__ long long out_row(const Args &a, int seq, int head, int n) {
    if (n >= a.rows) return -1;
    const int token = divided(n, a.by_G), g = n - token * a.G;
    return ((long long)seq * a.Tq + token) * a.Hq + head * a.G + g;
}

// Row n of a key head's query rows.
template <typename T>
__device__ __forceinline__ const T *query(const Args &a, int seq, int head, int n) {
    const int token = divided(n, a.by_G);
    return static_cast<const T *>(a.q) + ((long long)seq * a.Tq + token) * a.q_stride +
           (long long)(head * a.G + n - token * a.G) * a.d;
}

// What a warp holds of an item.  Thread (r, c) = (lane / 4, lane % 4) has query
// rows 8 nt + 2c, + 1 and of their outputs the features r D / 8 + 2 mt, + 1.
template <int D, int NT, bool F32>
struct State {
    static constexpr int kSteps = D / 16, kKeys = Config<D, NT, F32>::kKeys;
    uint32_t q[F32 ? 2 : 1][NT][kSteps][2];
    float o[NT][kSteps][4];
    float m[NT][2], l[NT][2], mul[NT][2];
    int limit[NT][2];            // keys below it are seen
    int full;                    // keys below it are seen by all rows

    // This thread's part of the query rows, as it lies in memory.
    template <typename T>
    __device__ __forceinline__ void fetch(const Args &a, int seq, int head, int group, Query<T, D> (&x)[NT]) const {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int n = group * 8 * NT + nt * 8 + r;
            x[nt].load(query<T>(a, seq, head, n) + c * (D / 4), n < a.rows);
        }
    }
    template <typename T>
    __device__ __forceinline__ void begin(const Args &a, int group, int len, const Query<T, D> (&given)[NT]) {
        const int lane = threadIdx.x % 32, c = lane % 4;
        const int first = len - a.Tq + 1;
        full = first + divided(group * 8 * NT, a.by_G);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[D / 4], top = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                float y[4];
                given[nt].get(j, y);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    x[4 * j + z] = y[z];
                    top = fmaxf(top, fabsf(y[z]));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the row times a power of two that takes its largest to 2^14 and above
            int e = 268 - (int)(__float_as_uint(top) >> 23);
            e = e < 253 ? e : 253;
            const float up = __uint_as_float((unsigned)e << 23);
            // (never 0: hidden scores are -infinity times it)
            const float down = fmaxf(__uint_as_float((unsigned)(254 - e) << 23) * a.scale_log2, 1.2e-38f);
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float u = x[4 * j + 2 * z] * up, v = x[4 * j + 2 * z + 1] * up;
                    q[0][nt][j][z] = pack_half(u, v);
                    if (F32) {
                        const float2 h = unpack_half(q[0][nt][j][z]);
                        q[F32 ? 1 : 0][nt][j][z] = pack_half(u - h.x, v - h.y);
                    }
                }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                mul[nt][z] = __shfl_sync(0xffffffffu, down, (2 * c + z) * 4);
                // (rows behind the last would see keys that are not there: what their scores
                // are then must not move the base)
                limit[nt][z] = min(first + divided(group * 8 * NT + nt * 8 + 2 * c + z, a.by_G), len);
                m[nt][z] = -INFINITY;
                l[nt][z] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int z = 0; z < 4; ++z) o[nt][j][z] = 0.f;
        }
    }

    // Scores of a block: s[nt][0..1] key r, s[nt][2..3] key r + 8.
    __device__ __forceinline__ void scores(const unsigned char *block, float (&s)[NT][4]) {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
        uint32_t wa[D / 32], wb[D / 32];
        load_words(block + r * (D / 2) + c * (D / 8), wa);
        load_words(block + (r + 8) * (D / 2) + c * (D / 8), wb);
        const unsigned char *ks = block + Layout<D>::kKs;
        uint32_t sa, sb;
        if (D == 128) {
            sa = kv4::scales_to_half2(*reinterpret_cast<const unsigned short *>(ks + r * 8 + 2 * c));
            sb = kv4::scales_to_half2(*reinterpret_cast<const unsigned short *>(ks + (r + 8) * 8 + 2 * c));
        } else {
            sa = kv4::scales_to_half2(ks[r * 4 + c] * 0x101u);
            sb = kv4::scales_to_half2(ks[(r + 8) * 4 + c] * 0x101u);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 4; ++z) s[nt][z] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            const uint32_t fa = __byte_perm(sa, 0, x < 2 ? 0x1010 : 0x3232);
            const uint32_t fb = __byte_perm(sb, 0, x < 2 ? 0x1010 : 0x3232);
            uint32_t ha[4], hb[4];
            kv4::codes_to_half2(wa[x], ha);
            kv4::codes_to_half2(wb[x], hb);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint32_t k[4] = {kv4::mul_half2(ha[2 * y], fa), kv4::mul_half2(hb[2 * y], fb),
                                       kv4::mul_half2(ha[2 * y + 1], fa), kv4::mul_half2(hb[2 * y + 1], fb)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma(s[nt], k, q[0][nt][2 * x + y]);
                    if (F32) mma(s[nt], k, q[F32 ? 1 : 0][nt][2 * x + y]);
                }
            }
        }
    }

    // o += p v over a block; p as operands.  EDGE: values of keys from `left` on are zeros.
    template <bool EDGE>
    __device__ __forceinline__ void mix(const unsigned char *block, const uint32_t (&p)[F32 ? 2 : 1][NT][2],
                                        int left, float (&apart)[F32 ? NT : 1][F32 ? kSteps : 1][4]) {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
        uint32_t w0[D / 32], w1[D / 32];
        load_words(block + Layout<D>::kV + c * D + r * (D / 8), w0);
        load_words(block + Layout<D>::kV + (c + 4) * D + r * (D / 8), w1);
        const unsigned char *vs = block + Layout<D>::kVs + r * (D / 8) / 16 * kBlock + 2 * c;
        uint32_t f0 = kv4::scales_to_half2(*reinterpret_cast<const unsigned short *>(vs));
        uint32_t f1 = kv4::scales_to_half2(*reinterpret_cast<const unsigned short *>(vs + 8));
        if (EDGE && left < kBlock) { // what lies behind the last key may be anything
            f0 = 2 * c + 1 < left ? f0 : (2 * c < left ? f0 & 0xffffu : 0u);
            f1 = 2 * c + 9 < left ? f1 : (2 * c + 8 < left ? f1 & 0xffffu : 0u);
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            uint32_t h0[4], h1[4];
            kv4::codes_to_half2(w0[x], h0);
            kv4::codes_to_half2(w1[x], h1);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint32_t v[4] = {kv4::mul_half2(h0[2 * y], f0), kv4::mul_half2(h0[2 * y + 1], f0),
                                       kv4::mul_half2(h1[2 * y], f1), kv4::mul_half2(h1[2 * y + 1], f1)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (F32) {
                        mma(apart[F32 ? nt : 0][F32 ? 2 * x + y : 0], v, p[0][nt]);
                        mma(apart[F32 ? nt : 0][F32 ? 2 * x + y : 0], v, p[F32 ? 1 : 0][nt]);
                    } else {
                        mma(o[nt][2 * x + y], v, p[0][nt]);
                    }
                }
            }
        }
    }

    // kKeys keys from key0 on, those below len.  EDGE: some of them may not be there, or
    // not be seen by all rows.
    template <bool EDGE>
    __device__ __forceinline__ void keys(const unsigned char *stage, int key0, int len) {
        const int r = threadIdx.x % 32 / 4;
        constexpr int N = kKeys / kBlock;
        float s[N][NT][4];
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (!EDGE || key0 + i * kBlock < len) scores(stage + i * Layout<D>::kBytes, s[i]);
        if (EDGE) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (key0 + i * kBlock + z / 2 * 8 + r >= limit[nt][z % 2]) s[i][nt][z] = -INFINITY;
        }
        float top[NT][2];
        bool above = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                float t = -INFINITY;
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        t = fmaxf(t, s[i][nt][2 * j + z]);
                    }
                top[nt][z] = t * mul[nt][z];             // mul is positive
                above = above || top[nt][z] > m[nt][z] + kLag;
            }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    float t = top[nt][z];
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    t = fmaxf(t, m[nt][z]);
                    const float f = m[nt][z] == t ? 1.f : exp2_of(m[nt][z] - t);
                    m[nt][z] = t;
                    l[nt][z] *= f;
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        o[nt][j][z] *= f;
                        o[nt][j][2 + z] *= f;
                    }
                }
        }
        uint32_t p[N][F32 ? 2 : 1][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float base[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) base[z] = m[nt][z] == -INFINITY ? 0.f : kTop - m[nt][z];
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float u = exp2_of(fmaf(s[i][nt][2 * j], mul[nt][0], base[0])),
                                v = exp2_of(fmaf(s[i][nt][2 * j + 1], mul[nt][1], base[1]));
                    l[nt][0] += u;
                    l[nt][1] += v;
                    const uint32_t h = pack_half(u, v);
                    p[i][0][nt][j] = transposed(h);
                    if (F32) {
                        const float2 g = unpack_half(h);
                        p[i][F32 ? 1 : 0][nt][j] = transposed(pack_half(u - g.x, v - g.y));
                    }
                }
        }
        // fp32: the tensor cores' sums are cut, not rounded, so a tile's are added to the others
        // by an addition that rounds (16 contexts of 32768 keys: 3.7e-6 of o, all of one sign,
        // and 5.3e-7 so)
        float apart[F32 ? NT : 1][F32 ? kSteps : 1][4] = {};
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (!EDGE || key0 + i * kBlock < len)
                mix<EDGE>(stage + i * Layout<D>::kBytes, p[i], len - key0 - i * kBlock, apart);
        if (F32) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
#pragma unroll
                    for (int z = 0; z < 4; ++z) o[nt][j][z] += apart[F32 ? nt : 0][F32 ? j : 0][z];
        }
    }

    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                float &x = l[nt][z];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
            }
    }
    // Outputs of an item that this warp had alone.
    template <typename T>
    __device__ __forceinline__ void write(const Args &a, int seq, int head, int group) const {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const long long row = out_row(a, seq, head, group * 8 * NT + nt * 8 + 2 * c + z);
                if (row < 0) continue;
                const float sum = l[nt][z], f = sum == 0.f ? 0.f : a.v_unit / sum;
                T *to = static_cast<T *>(a.o) + row * D + r * (D / 8);
#pragma unroll
                for (int j = 0; j < kSteps; ++j) store2(to + 2 * j, o[nt][j][z] * f, o[nt][j][2 + z] * f);
                if (r == 0 && a.lse)
                    a.lse[row] = sum == 0.f ? -INFINITY : (m[nt][z] - kTop + log2f(sum)) * kLn2;
            }
    }
    // A part: outputs [part_rows][D], then bases, then sums.
    __device__ __forceinline__ void put(const Args &a, float *part) const {
        const int lane = threadIdx.x % 32, r = lane / 4, c = lane % 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int n = nt * 8 + 2 * c + z;
                if (n >= a.part_rows) continue;
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
                    *reinterpret_cast<float2 *>(part + n * D + r * (D / 8) + 2 * j) =
                        make_float2(o[nt][j][z], o[nt][j][2 + z]);
                if (r == 0) {
                    part[a.part_rows * D + n] = m[nt][z] - kTop;
                    part[a.part_rows * D + a.part_rows + n] = l[nt][z];
                }
            }
    }
};

// ------------------------------------------------------------------ the kernel
// A place among all tiles.
struct Place {
    int seq, len, item, tile;
};
// lens: the lengths in shared memory where they fit there, else nullptr.
__device__ __forceinline__ int length(const Args &a, const int *lens, int b) { return lens ? lens[b] : length(a, b); }
__device__ __forceinline__ void next_item(const Args &a, const int *lens, Place &p) {
    p.tile = 0;
    if (++p.item < a.items) return;
    p.item = 0;
    do {
        ++p.seq;
        p.len = p.seq < a.B ? length(a, lens, p.seq) : 1;
    } while (p.len == 0);
}

// A part of an item that a warp did not have alone: where in shared memory or
// the workspace it lies, for the CTA's own join.
struct Part {
    int seq, item;       // seq < 0: none
    bool first, end;     // has the item's first tile, its last
    int at;              // in shared memory
};

// Parts of a row: a lane brings a part's base, -infinity where it has none; returns its
// weight, and the row's base.
__device__ __forceinline__ float join_weight(float m, float &base) {
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(base) : "f"(m));
    return m == base ? 1.f : exp2_of(m - base);
}

template <int N>
__device__ __forceinline__ void load_row(const float *p, float (&v)[N]) {
    if (N == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        v[0] = x.x; v[1] = x.y; v[N - 2] = x.z; v[N - 1] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        v[0] = x.x; v[1] = x.y;
    }
}
template <int N>
__device__ __forceinline__ void store_row(float *p, const float (&v)[N]) {
    if (N == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[N - 2], v[N - 1]);
    else *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float (&v)[N]) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = reinterpret_cast<const uint32_t &>(b);
    }
    if (N == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[N / 2 - 1]);
    else *reinterpret_cast<uint32_t *>(p) = w[0];
}

// A row's result: lane's N features of it.
template <typename T, int D, int N>
__device__ __forceinline__ void write_row(const Args &a, long long row, float (&v)[N], float base, float l) {
    const int lane = threadIdx.x % 32;
    const float f = l == 0.f ? 0.f : a.v_unit / l;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= f;
    store_row(static_cast<T *>(a.o) + row * D + N * lane, v);
    if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (base + log2f(l)) * kLn2;
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(Config<D, NT, F32>::kThreads, 1)
kv4_attn_kernel(const __grid_constant__ Args a) {
    using C = Config<D, NT, F32>;
    using T = std::conditional_t<F32, float, __nv_bfloat16>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t bars[C::kWarps][C::kStages];
    __shared__ unsigned sums[C::kThreads], warp_sums[C::kWarps], warp_some[C::kWarps];
    __shared__ int all_lens[C::kThreads];
    __shared__ Part parts[2 * C::kWarps];       // of each warp: what it closed, what it had last
    __shared__ unsigned trouble;
    __shared__ int from;                        // the CTA in which this one's first item begins
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, cta = blockIdx.x;
    unsigned char *ring = smem + warp * C::kRing;
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i) tc::mbar_init(&bars[warp][i], 1);
        tc::fence_mbar_init();
        parts[2 * warp].seq = parts[2 * warp + 1].seq = -1;
    }
    if (tid == 0) trouble = kDevOk;
    after_previous();
    let_next_start();

    // tiles before each thread's share of the sequences
    const int share = (a.B + C::kThreads - 1) / C::kThreads, b0 = tid * share;
    unsigned mine = 0;
    for (int b = b0; b < b0 + share && b < a.B; ++b) {
        const int n = length(a, b);
        all_lens[tid] = n;
        mine += tiles_of<C::kTile>(n);
    }
    const int *const lens = share == 1 ? all_lens : nullptr;
    unsigned sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    const unsigned some = __ballot_sync(0xffffffffu, mine > 0);
    if (lane == 31) {
        warp_sums[warp] = sum;
        warp_some[warp] = __popc(some);
    }
    __syncthreads();
    unsigned tiles = 0, held = 0, before = __popc(some & ((1u << lane) - 1));
    for (int w = 0; w < C::kWarps; ++w) {
        if (w == warp) {
            sum += tiles;
            before += held;
        }
        tiles += warp_sums[w];
        held += warp_some[w];
    }
    // An item counts as a tile more than it has, for its begin and end, where warps have
    // so many tiles that one does not matter.
    const int extra = share == 1 && tiles * (unsigned)a.items >= kMany * (unsigned)(C::kWarps * a.ctas) ? 1 : 0;
    sums[tid] = sum - mine + (extra ? before : 0u);
    if (extra) tiles += held;
    __syncthreads();

    const Split split = split_of<C::kWarps>(a, tiles);
    const unsigned cta0 = split.cta(cta);
    unsigned u = 0, end = 0;
    if (cta < split.ctas) {
        const unsigned size = split.cta(cta + 1) - cta0;
        u = cta0 + size / C::kWarps * warp + size % C::kWarps * warp / C::kWarps;
        end = cta0 + size / C::kWarps * (warp + 1) + size % C::kWarps * (warp + 1) / C::kWarps;
    }
    bool ok = true, bad = false;
    float *const mine_at = a.part + (size_t)cta * (2 + C::kWarps) * a.part_size;
    if (u < end) {
        // where the warp's tiles begin
        Place at;
        {
            const unsigned x = (unsigned)divided((int)u, a.by_items);
            // the last share that begins at x or before: sums do not fall
            constexpr int kStep = C::kThreads / 32;
            static_assert(kStep <= 32, "a lane for each of a step's sums");
            int lo = (31 - __clz(__ballot_sync(0xffffffffu, sums[lane * kStep] <= x))) * kStep;
            lo += 31 - __clz(__ballot_sync(0xffffffffu, lane < kStep && sums[lo + lane % kStep] <= x));
            unsigned y = sums[lo];
            at.seq = lo * share;
            at.len = length(a, lens, at.seq);
            while (y + tiles_of<C::kTile>(at.len) + extra <= x) {
                y += tiles_of<C::kTile>(at.len) + extra;
                at.len = length(a, lens, ++at.seq);
            }
            const unsigned rest = u - y * (unsigned)a.items, of = (unsigned)(tiles_of<C::kTile>(at.len) + extra);
            at.item = (int)(rest / of);
            at.tile = (int)(rest - (unsigned)at.item * of);
        }
        // its tiles, without those that count and are none
        int n = (int)(end - u);
        const bool leads_cta = u == cta0;
        if (extra) {
            int left = n;
            n = 0;
            if (at.tile == tiles_of<C::kTile>(at.len)) {
                ++u;
                if (--left > 0) next_item(a, lens, at);
            }
            for (Place p = at; left > 0;) {
                const int some = min(left, tiles_of<C::kTile>(p.len) - p.tile);
                n += some;
                left -= some + 1;
                if (left > 0) next_item(a, lens, p);
            }
        }
        const int first_tile = at.tile;

        // Copies.  The lanes look up the blocks of kAhead tiles at once.  (A lookup ahead of
        // its use, too, does not pay: 256 contexts 67.4 us, 65.9 without.)
        constexpr int kAhead = 32 / C::kBlocks;
        const uint64_t policy = policy_of(a.groups == 1);
        Place ahead = at;                            // of the tile to be asked for
        int issued = 0, looked = -kAhead;
        unsigned block = 0;                          // this lane's, of the tiles from `looked` on
        bool fresh = true;                           // the tile begins an item
        auto issue = [&](int slot) {
            if (fresh || ahead.tile >= looked + kAhead) {
                looked = ahead.tile;
                const int nb = C::kBlocks * looked + lane, column = divided(nb, a.by_blocks);
                int page = 0;
                if (nb * kBlock < ahead.len) page = a.table[(long long)ahead.seq * a.columns + column];
                if (page < 0 || page >= a.n_pages) {
                    bad = true;
                    page = 0;
                }
                block = ((unsigned)page * a.Hk + divided(ahead.item, a.by_groups)) * a.blocks + nb - column * a.blocks;
            }
            const int from_lane = C::kBlocks * (ahead.tile - looked) + lane % C::kBlocks;
            const unsigned src = __shfl_sync(0xffffffffu, block, from_lane);
            const int there = min(C::kBlocks, (ahead.len - ahead.tile * C::kTile + kBlock - 1) / kBlock);
            if (lane == 0) tc::mbar_expect_tx(&bars[warp][slot], there * Layout<D>::kBytes);
            __syncwarp();
            if (lane < there)
                load_block(ring + slot * C::kStage + lane * Layout<D>::kBytes,
                           a.pool + (unsigned long long)src * Layout<D>::kBytes, Layout<D>::kBytes,
                           &bars[warp][slot], policy);
            if (fresh && issued > 0) {               // its query rows into L1
                const int head = divided(ahead.item, a.by_groups);
                const int row = (ahead.item - head * a.groups) * C::kRows + lane % C::kRows;
                if (row < a.rows) {
                    const T *q = query<T>(a, ahead.seq, head, row);
                    const int i = lane / C::kRows * 128;
                    unsigned x;
                    const char *at_q = reinterpret_cast<const char *>(q) + i;
                    if (i < D * (int)sizeof(T)) asm volatile("ld.global.ca.b32 %0, [%1];" : "=r"(x) : "l"(at_q));
                }
            }
            ++issued;
            fresh = ++ahead.tile == tiles_of<C::kTile>(ahead.len);
            if (fresh && issued < n) next_item(a, lens, ahead);
        };

        // the first item's queries, before the copies: behind them they would take 4000 cycles
        State<D, NT, F32> st;
        Query<T, D> given[NT];
        st.template fetch<T>(a, at.seq, divided(at.item, a.by_groups),
                             at.item - divided(at.item, a.by_groups) * a.groups, given);
        for (; issued < C::kStages && issued < n;) issue(issued);
        int slot = 0, parity = 0, begin = first_tile;
        st.template begin<T>(a, at.item - divided(at.item, a.by_groups) * a.groups, at.len, given);
        bool start = false, closed = false, back = false;
        for (int done = 0; done < n; ++done) {
            const int free_slot = slot + 1 == C::kStages ? 0 : slot + 1;
            if (done + 1 == n && closed) {
                // the part that the warp closed comes back, into a stage that is free: its
                // way to memory and back runs under the last tile
                if (lane == 0) {
                    tc::mbar_expect_tx(&bars[warp][free_slot], a.part_size * 4);
                    tc::bulk_load(ring + free_slot * C::kStage, mine_at + (2 + warp) * a.part_size, a.part_size * 4,
                                  &bars[warp][free_slot]);
                    parts[2 * warp].at = warp * C::kRing + free_slot * C::kStage;
                }
                back = true;
                __syncwarp();
            }
            const int head = divided(at.item, a.by_groups), group = at.item - head * a.groups;
            if (start) {
                Query<T, D> given[NT];
                st.template fetch<T>(a, at.seq, head, group, given);
                st.template begin<T>(a, group, at.len, given);
            }
            start = false;
            ok = tc::mbar_wait(&bars[warp][slot], parity) && !a.lost_wait;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const unsigned char *stage = ring + slot * C::kStage;
#pragma unroll 1
            for (int i = 0; i < C::kTile; i += C::kKeys) {
                const int key0 = at.tile * C::kTile + i;
                const unsigned char *keys = stage + i / kBlock * Layout<D>::kBytes;
                if (key0 + C::kKeys <= st.full) st.template keys<false>(keys, key0, at.len);
                else if (key0 < at.len) st.template keys<true>(keys, key0, at.len);
            }
            __syncwarp();
            if (issued < n) issue(slot);
            if (++slot == C::kStages) {
                slot = 0;
                parity ^= 1;
            }
            const bool whole = ++at.tile == tiles_of<C::kTile>(at.len), last = done + 1 == n;
            if (!whole && !last) continue;
            // the end of the warp's part of an item
            st.finish();
            if (begin == 0 && whole) {
                st.template write<T>(a, at.seq, head, group);
            } else {
                // (the last tile's stage is free)
                const int last_slot = slot == 0 ? C::kStages - 1 : slot - 1;
                st.put(a, last ? reinterpret_cast<float *>(ring + last_slot * C::kStage)
                               : mine_at + (2 + warp) * a.part_size);
                if (lane == 0)
                    parts[2 * warp + last] = {at.seq, at.item, begin == 0, whole,
                                              warp * C::kRing + last_slot * C::kStage};
                if (!last) {
                    closed = true;
                    tc::fence_proxy_async_global();
                    __syncwarp();
                }
            }
            if (last) break;
            next_item(a, lens, at);
            begin = 0;
            start = true;
        }
        // the stage that the closed part came back to: behind the last tile's
        const int free_slot = !back ? -1 : ok ? slot : (slot + 1 == C::kStages ? 0 : slot + 1);
        if (back) {
            const int turns = n > free_slot ? (n - 1 - free_slot) / C::kStages + 1 : 0;
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[warp][free_slot], turns & 1)) && ok;
        }
        if (!ok) {
            // what was asked for arrives by itself; the ring must outlive it
            for (int i = 0; i < C::kStages && i < issued; ++i)
                if (i != free_slot)
                    tc::mbar_wait(&bars[warp][i], (issued - 1 - i) / C::kStages & 1);    // its last phase
            if (lane == 0) atomicMax(&trouble, (unsigned)kDevTimeout);
        }
        if (bad) atomicMax(&trouble, (unsigned)kDevBadTable);
        if (lane == 0 && leads_cta) {                // the CTA's first tile
            const unsigned x = u - first_tile;
            int c = min((int)((float)x / (float)split.total * split.ctas), cta);
            while (c > 0 && split.cta(c) > x) --c;
            while (split.cta(c + 1) <= x) ++c;
            from = c;
        }
    }
    __syncthreads();

    // Items that several of the CTA's warps had.  Lane i has part i; parts of an item
    // follow each other, and the lane of its first has the item.  Rows of all items in a
    // row are the warps' in turn.  (Few instructions: they are fetched anew here.)
    {
        constexpr int N = D / 32;
        Part x{-1, 0, false, false, 0};
        if (lane < 2 * C::kWarps) x = parts[lane];
        const unsigned all = __ballot_sync(0xffffffffu, x.seq >= 0), lower = all & ((1u << lane) - 1);
        const int prev = lower ? 31 - __clz(lower) : lane;
        const int pseq = __shfl_sync(0xffffffffu, x.seq, prev), pitem = __shfl_sync(0xffffffffu, x.item, prev);
        const bool leads = x.seq >= 0 && (!lower || pseq != x.seq || pitem != x.item);
        const unsigned leaders = __ballot_sync(0xffffffffu, leads), above = leaders & ~((2u << lane) - 1);
        const unsigned parts_of = all & (above ? (1u << (__ffs(above) - 1)) - 1 : 0xffffffffu) & ~((1u << lane) - 1);
        const bool whole = __shfl_sync(0xffffffffu, (int)x.end, parts_of ? 31 - __clz(parts_of) : 0);
        const int x_head = divided(x.item, a.by_groups), x_row = (x.item - x_head * a.groups) * C::kRows;
        const int rows = leads ? min(C::kRows, a.rows - x_row) : 0;
        int behind = rows;                           // rows of the items up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, behind, o);
            if (lane >= o) behind += y;
        }
        // an item that began in an earlier CTA: this CTA's first, if any
        const unsigned owned = __ballot_sync(0xffffffffu, leads && !x.first && whole);
        if (warp == 0 && (owned ? lane == __ffs(owned) - 1 : lane == 0))
            a.owners[cta] = owned ? Owner{x.seq, x.item, from} : Owner{-1, 0, 0};
        const int total = __shfl_sync(0xffffffffu, behind, 31), pr = a.part_rows;
#pragma unroll 1
        for (int p = warp; p < total; p += C::kWarps) {
            const int of = __ffs(__ballot_sync(0xffffffffu, p < behind)) - 1;
            const int turn = p - __shfl_sync(0xffffffffu, behind - rows, of);
            const unsigned members = __shfl_sync(0xffffffffu, parts_of, of);
            const bool here = members >> lane & 1;
            const float *part = reinterpret_cast<const float *>(smem + x.at) + pr * D + turn;
            const float m = here ? part[0] : -INFINITY, t = here ? part[pr] : 0.f;
            int k = of;
            float y[N], v[N] = {}, base, l = 0.f;
            auto load = [&](float (&to)[N]) {
                const int at = __shfl_sync(0xffffffffu, x.at, k);
                load_row(reinterpret_cast<const float *>(smem + at) + turn * D + N * lane, to);
            };
            load(y);
            const float w = join_weight(m, base), wt = w * t;
            for (unsigned left = members;;) {
                const int now = k;
                left &= left - 1;
                k = left ? __ffs(left) - 1 : now;    // (behind the last, that again)
                float z[N];
                load(z);
                const float f = __shfl_sync(0xffffffffu, w, now);
                l += __shfl_sync(0xffffffffu, wt, now);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    v[i] = fmaf(f, y[i], v[i]);
                    y[i] = z[i];
                }
                if (!left) break;
            }
            const bool first = __shfl_sync(0xffffffffu, (int)x.first, of);
            const bool end = __shfl_sync(0xffffffffu, (int)whole, of);
            const int seq = __shfl_sync(0xffffffffu, x.seq, of), head = __shfl_sync(0xffffffffu, x_head, of);
            const int row = __shfl_sync(0xffffffffu, x_row, of) + turn;
            if (first && end) {
                write_row<T, D>(a, out_row(a, seq, head, row), v, base, l);
            } else {
                float *out = mine_at + (first ? 1 : 0) * a.part_size;
                store_row(out + turn * D + N * lane, v);
                if (lane == 0) {
                    out[pr * D + turn] = base;
                    out[pr * D + pr + turn] = l;
                }
            }
        }
    }
    if (tid == 0) *(a.ctas == 1 ? a.status : a.cta_status + cta) = trouble;

    // rows of empty caches
    for (int b = cta; b < a.B; b += gridDim.x) {
        if (length(a, lens, b) > 0) continue;
        const long long row0 = (long long)b * a.Tq * a.Hq;
        const long long n = (long long)a.Tq * a.Hq;
        for (long long i = tid; i < n * (D / 4); i += C::kThreads) {
            const float zero[4] = {};
            store_row(static_cast<T *>(a.o) + row0 * D + 4 * i, zero);
        }
        if (a.lse)
            for (long long i = tid; i < n; i += C::kThreads) a.lse[row0 + i] = -INFINITY;
    }
}

// Joins the parts of the item that began in an earlier CTA and ends in CTA
// blockIdx.x; PER warps to a row.  The first block writes the status word.
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(512) kv4_join_kernel(const __grid_constant__ Args a) {
    using C = Config<D, NT, F32>;
    using T = std::conditional_t<F32, float, __nv_bfloat16>;
    constexpr int N = D / 32, kPer = 16 / C::kRows;
    __shared__ __align__(16) float shared_v[16][D];
    __shared__ float shared_m[16], shared_l[16];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, n = warp % C::kRows, sub = warp / C::kRows;
    after_previous();
    let_next_start();
    const Owner own = a.owners[blockIdx.x];
    if (blockIdx.x == 0 && warp == 0) {
        unsigned x = kDevOk;
        for (int c = lane; c < a.ctas; c += 32) x = max(x, a.cta_status[c]);
        x = __reduce_max_sync(0xffffffffu, x);
        if (lane == 0) *a.status = x;
    }
    if (own.seq < 0) return;
    const int head = divided(own.item, a.by_groups), group = own.item - head * a.groups;
    const bool there = group * C::kRows + n < a.rows;
    // parts: of its first CTA the last item's, of the others the first item's
    const int count = (int)blockIdx.x - own.from + 1, stride = (2 + C::kWarps) * a.part_size;
    const float *const parts = a.part + (size_t)own.from * stride + n * D + N * lane;      // (fewer than 2^31)
    const int sums = a.part_rows * D + n - (n * D + N * lane);
    float base = -INFINITY, l = 0.f, v[N] = {};
    for (int k0 = 32 * sub; k0 < count && there; k0 += 32 * kPer) {
        const int k = k0 + lane;
        const bool here = k < count;
        const float *part = parts + (here ? k : 0) * stride + (k == 0 ? a.part_size : 0) + sums;
        const float m = here ? part[0] : -INFINITY, sum = here ? part[a.part_rows] : 0.f;
        const int most = min(32, count - k0);
        float y[4][N] = {};                          // four parts are asked for ahead
        auto ask = [&](int j0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j0 + j < most)
                    load_row(parts + (k0 + j0 + j) * stride + (k0 + j0 + j == 0 ? a.part_size : 0), y[j]);
        };
        ask(0);
        float top;
        const float w = join_weight(m, top);
        float t = w * sum;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        const float both = fmaxf(base, top);
        const float f0 = base == both ? 1.f : exp2_of(base - both), f1 = top == both ? 1.f : exp2_of(top - both);
        base = both;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= f0;
#pragma unroll 1
        for (int j0 = 0; j0 < most; j0 += 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f = __shfl_sync(0xffffffffu, w, (j0 + j) & 31) * f1;
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = j0 + j < most ? fmaf(f, y[j][i], v[i]) : v[i];
            }
            ask(j0 + 4);
        }
        l = l * f0 + t * f1;
    }
    if (kPer > 1 && count > 32) {                    // (the same for all of the block)
        store_row(&shared_v[warp][N * lane], v);
        if (lane == 0) {
            shared_m[warp] = base;
            shared_l[warp] = l;
        }
        __syncthreads();
        if (sub != 0) return;
        for (int z = 1; z < kPer; ++z) {
            const int y = warp + z * C::kRows;
            const float m = shared_m[y], both = fmaxf(base, m);
            const float f0 = base == both ? 1.f : exp2_of(base - both), f1 = m == both ? 1.f : exp2_of(m - both);
            base = both;
            l = l * f0 + shared_l[y] * f1;
            float t[N];
            load_row(&shared_v[y][N * lane], t);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = v[i] * f0 + t[i] * f1;
        }
    } else if (sub != 0) {
        return;
    }
    if (there) write_row<T, D>(a, out_row(a, own.seq, head, group * C::kRows + n), v, base, l);
}

// The unpacked path's check of the table, after the attention that writes the status word,
// or cta_status where that is not the call's.
__global__ void kv4_check_kernel(const __grid_constant__ Args a) {
    after_previous();
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.cta_status) atomicMax(a.status, *a.cta_status);
    const int b = blockIdx.x, page = a.blocks * kBlock, held = (int)(((long long)length(a, b) + page - 1) / page);
    for (int c = threadIdx.x; c < held; c += blockDim.x) {
        const int x = a.table[(long long)b * a.columns + c];
        if (x < 0 || x >= a.n_pages) atomicMax(a.status, (unsigned)kDevBadTable);
    }
}

// Without any key: zeros, from a launch that has no table to read.  lens: of a table
// with columns, whose entries name no page then.
__global__ void kv4_no_keys_kernel(uint4 *o, long long n, float *lse, long long rows, unsigned *status,
                                   const int *lens, int B) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (blockIdx.x == 0) {
        bool some = false;
        for (int b = threadIdx.x; lens && b < B; b += blockDim.x) some = some || lens[b] > 0;
        some = __syncthreads_or(some);
        if (i == 0) *status = some ? kDevBadTable : kDevOk;
    }
    if (i < n) o[i] = make_uint4(0, 0, 0, 0);
    if (lse && i < rows) lse[i] = -INFINITY;
}

// ------------------------------------------------------------------ host
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev < 64 && (n = known[dev].load()) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();     // no device: sizes are still wanted
        return 152;
    }
    if (dev < 64) known[dev].store(n);
    return n;
}

// Many query rows: the cache's rows are unpacked into the workspace once and go
// through the attention of dense rows, where that runs on the tensor cores (bf16, up
// to 128 query heads to a key head; the CUDA cores take 4 to 8 times as long as the
// kernel here in fp32, and 569 us for 49 with 256 + 1 heads of 128, a token over 65536
// keys), whose tcgen05 products take 128 rows, and where there is enough to do for that
// way's launches.  Both, in us, with 16 + 4 heads of 128 over 32768 keys, by tokens: 24
// 38 and 38, 32 46 and 40, 64 78 and 48, 512 529 and 157; over 4096 keys: 32 18 and 19,
// 64 21 and 25, 128 29 and 29, 256 47 and 32; over 8 caches of 4096: 24 39 and 40, 32 47 and 42; 16 + 2 of
// 64 over 4 caches of 16384: 12 28 and 28, 16 33 and 30, 64 100 and 54; 8 + 8 of 64 over 1024 keys: 64
// 10 and 15, 256 15 and 18, 512 19 and 20.  They are the same at 8 to 13 million pairs of a row and a key.
constexpr int kUnpackRows = 128;
constexpr long long kUnpackPairs = 12LL << 20;
// The unpacked rows, of the table's whole width: of as many sequences at a time as fit into
// these bytes; not where one does not.  (A quarter of them: 8 sequences of 64 tokens, 32 + 8
// heads of 128 over 32768 keys, 548 us in four turns and 444 in one; over 1000 keys in tables
// as wide 184 and 111.)
constexpr long long kUnpackBytes = 1LL << 30;
// The n sequences from b0 on, unpacked (the workspace's places are not in it).
void unpack_part(const Kv4Attn &p, int b0, int n, AttnProblem &x, Kv4Rows &r) {
    const size_t es = p.dtype == 1 ? 2 : 4;
    const long long row0 = (long long)b0 * p.Tq;
    x.q = static_cast<const unsigned char *>(p.q) + row0 * p.q_stride * es;
    x.out = static_cast<unsigned char *>(p.o) + row0 * p.Hq * p.d * es;
    x.lse = p.lse ? p.lse + row0 * p.Hq : nullptr;
    x.q_stride = p.q_stride;
    x.k_stride = x.v_stride = (long long)p.Hk * p.d;
    x.n_seq = n; x.Tq = p.Tq; x.Tk = p.columns * p.page; x.total_q = n * p.Tq; x.total_k = n * x.Tk;
    x.Hq = p.Hq; x.Hk = p.Hk; x.d = p.d; x.dtype = p.dtype;
    // keys without their unit, which goes with the scale (both ways exact): fp32 holds the
    // products of rows whose scores are in its range, whatever the unit
    x.scale = p.scale * p.k_unit;
    r.k_stride = x.k_stride; r.v_stride = x.v_stride; r.from_start = true;
    r.pool = const_cast<void *>(p.pool); r.table = p.table + (long long)b0 * p.columns; r.lens = p.lens + b0;
    x.k_lens = r.lens;
    r.B = n; r.T = x.Tk; r.Hk = p.Hk; r.d = p.d; r.page = p.page; r.n_pages = p.n_pages; r.columns = p.columns;
    r.dtype = p.dtype; r.k_unit = 1.f; r.v_unit = p.v_unit;
}
// How it is unpacked: `each` sequences at a time (0: it is not), and in the workspace the
// attention's (its status word first), the keys and the values.
struct Unpack {
    int each;
    size_t attn, k, v, bytes;
};
Unpack unpack_of(const Kv4Attn &p) {
    Unpack u{};
    const long long rows = (long long)p.columns * p.page, bytes = rows * p.Hk * p.d * 4;
    if (rows == 0 || (long long)p.Hq / p.Hk * p.Tq < kUnpackRows || bytes > kUnpackBytes) return u;
    if (rows * ((long long)p.B * p.Tq * p.Hq) < kUnpackPairs) return u;     // (of the tables' whole width)
    const long long fit = kUnpackBytes / bytes, turns = (p.B + fit - 1) / fit;
    const int each = (int)((p.B + turns - 1) / turns), last = (p.B - 1) % each + 1;
    AttnProblem x{};
    Kv4Rows r{};
    unpack_part(p, 0, each, x, r);
    if (!attn_on_tensor_cores(x) || attn_too_large(x) || kv4_rows_too_large(r)) return u;
    size_t need = attn_fwd_workspace_bytes(x);
    const size_t part = up256((size_t)each * bytes / 2);
    unpack_part(p, 0, last, x, r);                   // (fewer sequences may have more parts)
    if (attn_fwd_workspace_bytes(x) > need) need = attn_fwd_workspace_bytes(x);
    u.each = each;
    u.attn = each < p.B ? up256(kWsHeader) : 0;      // one turn: its status word is the call's
    u.k = u.attn + up256(need);
    u.v = u.k + part;
    u.bytes = u.v + part;
    return u;
}

struct Plan {
    int ctas, rows, groups, part_rows, part_size;
    long long tiles;             // at most, of all sequences and key heads
    size_t cta_status, owners, part, bytes;
    cudaError_t (*run)(const Args &, cudaStream_t);
};
template <int D, int NT, bool F32>
cudaError_t launch(const Args &a, cudaStream_t s);

template <int D, int NT, bool F32>
void sizes(Plan &p) {
    using C = Config<D, NT, F32>;
    p.run = launch<D, NT, F32>;
    p.groups = (p.rows + C::kRows - 1) / C::kRows;
    p.part_rows = p.rows < C::kRows ? p.rows : C::kRows;
    p.part_size = (p.part_rows * (D + 2) + 3) & ~3;
    // no more CTAs than there can be tiles for their warps
    const long long wanted = (p.tiles * p.groups + C::kWarps - 1) / C::kWarps;
    if (wanted < p.ctas) p.ctas = wanted > 0 ? (int)wanted : 1;
    p.bytes = up256(p.part + (size_t)p.ctas * (2 + C::kWarps) * p.part_size * sizeof(float));
}
Plan plan_of(const Kv4Attn &p) {
    Plan x{};
    x.ctas = sm_count();
    x.rows = p.Hq / p.Hk * p.Tq;
    x.tiles = (long long)p.B * p.Hk * (((long long)p.columns * p.page + 63) / 64);
    x.cta_status = kWsHeader;
    x.owners = up256(x.cta_status + x.ctas * sizeof(unsigned));
    x.part = up256(x.owners + x.ctas * sizeof(Owner));
    const bool two = x.rows > 8;
    if (p.d == 64) {
        if (p.dtype == 0) sizes<64, 1, true>(x);
        else two ? sizes<64, 2, false>(x) : sizes<64, 1, false>(x);
    } else {
        if (p.dtype == 0) sizes<128, 1, true>(x);
        else two ? sizes<128, 2, false>(x) : sizes<128, 1, false>(x);
    }
    return x;
}

template <int D, int NT, bool F32>
cudaError_t launch(const Args &a, cudaStream_t s) {
    using C = Config<D, NT, F32>;
    cudaError_t e = allow_dynamic_smem((const void *)kv4_attn_kernel<D, NT, F32>, C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_next(kv4_attn_kernel<D, NT, F32>, a.ctas, C::kThreads, C::kSmem, 1, a, s);
    note_launch();
    if (e != cudaSuccess || a.ctas == 1) return e;      // one CTA joins what there is
    e = launch_next(kv4_join_kernel<D, NT, F32>, a.ctas, 512, 0, 1, a, s);
    note_launch();
    return e;
}

}  // namespace

size_t kv4_attn_workspace_bytes(const Kv4Attn &p) {
    const Unpack u = unpack_of(p);
    return u.each ? u.bytes : plan_of(p).bytes;
}

bool kv4_attn_too_large(const Kv4Attn &p) {
    const long long rows = (long long)p.B * p.Tq * p.Hq;
    const long long tiles = (long long)p.B * ((long long)p.columns * p.page / 64 + 2);
    const long long items = (long long)p.Hk * ((p.Hq / p.Hk * (long long)p.Tq + 7) / 8);
    return rows > INT32_MAX || items > INT32_MAX || (items > 0 && tiles > INT32_MAX / items);
}

namespace {
cudaError_t launch_unpacked(const Kv4Attn &p, const Unpack &u, cudaStream_t s) {
    unsigned char *ws = static_cast<unsigned char *>(p.ws);
    cudaError_t e = u.attn ? cudaMemsetAsync(ws, 0, sizeof(unsigned), s) : cudaSuccess;
    for (int b0 = 0; b0 < p.B && e == cudaSuccess; b0 += u.each) {
        const int n = p.B - b0 < u.each ? p.B - b0 : u.each;
        AttnProblem x{};
        Kv4Rows r{};
        unpack_part(p, b0, n, x, r);
        x.ws = ws + u.attn;
        x.k = r.k_out = ws + u.k;
        x.v = r.v_out = ws + u.v;
        if ((e = launch_kv4_rows(r, true, s)) != cudaSuccess || (e = launch_attn_fwd(x, s)) != cudaSuccess) break;
        Args a{};
        a.table = r.table; a.lens = r.lens; a.columns = p.columns; a.blocks = p.page / kBlock;
        a.n_pages = p.n_pages; a.status = static_cast<unsigned *>(p.ws);
        a.cta_status = u.attn ? static_cast<unsigned *>(x.ws) : nullptr;
        e = launch_next(kv4_check_kernel, n, 256, 0, 1, a, s);
        note_launch();
    }
    return e;
}
}  // namespace

cudaError_t launch_kv4_attn(const Kv4Attn &p, cudaStream_t s) {
    unsigned char *ws = static_cast<unsigned char *>(p.ws);
    if (p.n_pages == 0 || p.columns == 0) {
        const long long rows = (long long)p.B * p.Tq * p.Hq, n = rows * p.d * (p.dtype == 1 ? 2 : 4) / 16;
        kv4_no_keys_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(static_cast<uint4 *>(p.o), n, p.lse, rows,
                                                                      static_cast<unsigned *>(p.ws),
                                                                      p.columns > 0 ? p.lens : nullptr, p.B);
        note_launch();
        return cudaGetLastError();
    }
    const Unpack u = unpack_of(p);
    if (u.each) return launch_unpacked(p, u, s);
    const Plan x = plan_of(p);
    Args a{};
    a.q = p.q; a.q_stride = p.q_stride; a.pool = static_cast<const unsigned char *>(p.pool);
    a.table = p.table; a.lens = p.lens; a.o = p.o; a.lse = p.lse;
    a.B = p.B; a.Tq = p.Tq; a.Hq = p.Hq; a.Hk = p.Hk; a.G = p.Hq / p.Hk; a.d = p.d;
    a.blocks = p.page / kBlock; a.n_pages = p.n_pages; a.columns = p.columns;
    a.rows = x.rows;
    a.groups = x.groups;
    a.items = p.Hk * x.groups;
    a.by_G = divisor(a.G); a.by_groups = divisor(a.groups); a.by_items = divisor(a.items);
    a.by_blocks = divisor(a.blocks);
    a.part_rows = x.part_rows; a.part_size = x.part_size;
    a.scale_log2 = p.scale * p.k_unit * kLog2e;
    a.v_unit = p.v_unit;
    a.status = static_cast<unsigned *>(p.ws);
    a.cta_status = reinterpret_cast<unsigned *>(ws + x.cta_status);
    a.owners = reinterpret_cast<Owner *>(ws + x.owners);
    a.part = reinterpret_cast<float *>(ws + x.part);
    a.ctas = x.ctas;
    // test hook: every warp takes its first wait for one that ran out
    a.lost_wait = std::getenv("KLA_TEST_LOST_WAIT") != nullptr;
    return x.run(a, s);
}

}  // namespace kla
