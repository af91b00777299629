// Causal softmax attention, backward, on the tensor cores (bf16, head sizes 64
// and 128):
//
//   p = exp2(c s - lse log2 e),  ds = p (dp - delta),  dp = go v^T,
//   dv = p^T go,  dk = scale ds^T q,  dq = scale ds k,  delta = sum go o
//
// One launch has two kinds of CTAs, each on 128 x 128 tiles of (packed rows,
// keys) with scores, probabilities and sums in tensor memory:
//
//   a key tile:  S^T = K Q^T, dP^T = V dO^T over the row tiles that see it;
//                P^T and dS^T (bf16, tensor memory) are the A operands of
//                dV += P^T dO and dK += dS^T Q
//   a row tile:  S = Q K^T, dP = dO V^T over its keys; dS is the A operand of
//                dQ += dS K
//
// Scores are computed twice (7 products where 5 would do with dQ summed by
// atomics), so that no sum depends on the order of CTAs and no fp32 copy of dQ
// passes through memory.  Two warpgroups share a tile's columns; one warp each
// issues the products, the loads (TMA) and, for key tiles, the rows' lse and
// delta.  p and ds are rounded to bf16 as operands; sums are fp32.
//
// Tensor memory, key tiles: four blocks of 64 columns hold S^T and dP^T (two
// each) while P^T and dS^T of the same tile take one block of each once they
// are read; the two blocks left take the next S^T.  By this the product dV
// runs under the dS step and dK, dP^T of the next under the exponentials:
//
//     S' (next)   dK   dP'   dV'
//     [ds done]        [exp: P']   [ds']
#include "kla_attn_tc.cuh"

namespace kla {
namespace {

using namespace tc;
using attn::Args;
using attn::Item;
using attn::kSlab;
using attn::kTile;
using attn::Seq;

constexpr int kThreads = 384;            // 8 softmax warps, products, loads, row statistics
constexpr int kSoftmax = 256;

template <int D>
struct Cfg {
    static constexpr int SLABS = D / 64;
    static constexpr uint32_t TILE = SLABS * kSlab;
    static constexpr size_t SMEM = (size_t)TILE * 7 + 1024;
    static constexpr uint32_t TM_COLS = 512;
};

struct Shared {
    uint64_t fix;                        // the CTA's own tiles landed
    uint64_t full[5], empty[5];          // ring slots
    uint64_t s[2], dp, p, ds;            // products ready; operands ready
    uint64_t st[2], read[2];             // row statistics ready, and read
    uint64_t tail[2], fin;
    uint32_t tmem;
    volatile int abort;
};

struct Maps {
    CUtensorMap q, go, k, v;
    int tokens;                          // of a row tile
};

// Blocks of 64 columns of iteration i of a key tile: S^T's halves, dP^T's
// halves, and the block of each that P^T and dS^T take.
struct Blocks {
    uint32_t s0, s1, d0, d1, p, ds;
};
__device__ __forceinline__ Blocks blocks_of(int i) {
    switch (i & 3) {
        case 0: return {0, 64, 128, 192, 0, 192};
        case 1: return {64, 128, 0, 192, 64, 0};
        case 2: return {128, 192, 0, 64, 192, 0};
        default: return {64, 128, 0, 192, 128, 192};
    }
}

__device__ __forceinline__ void mul2(float &x0, float &x1, float y0, float y1) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(y0), "f"(y1));
}
__device__ __forceinline__ void fma2v(float &x0, float &x1, float a, float b0, float b1) {
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %4};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(a), "f"(b0), "f"(b1));
}

// A row of D features from tensor memory, times f, to global memory (zeros
// where there was no product).  Warp-wide; `on`: this lane's row is stored.
template <int D>
__device__ __forceinline__ void store_row(uint32_t tmem, __nv_bfloat16 *dst, float f, bool any,
                                          bool on) {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        uint32_t y[16];
        if (any) {
            tmem_ld16(tmem + 16u * j, y);
            tmem_ld_wait();
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = 0;
        }
        if (on) {
            uint4 *p = reinterpret_cast<uint4 *>(dst + 16 * j);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t u[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    u[z] = attn::pack2(__uint_as_float(y[8 * k + 2 * z]) * f,
                                       __uint_as_float(y[8 * k + 2 * z + 1]) * f);
                p[k] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
        __syncwarp();
    }
}

template <int D>
struct Cta {
    using C = Cfg<D>;
    const Args &a;
    const Maps &maps;
    Shared &sh;
    unsigned char *base;      // 7 tiles: two of the CTA, five of the rings
    uint32_t tb;
    int warp, lane;
    Item it;
    Seq seq;

    __device__ void give_up() {
        sh.abort = 1;
        *a.status = kDevTimeout;
    }
    // One lane's wait, and a warp's.
    __device__ bool wait(uint64_t *bar, int phase) {
        return mbar_wait_or_abort(bar, (uint32_t)phase & 1u, &sh.abort);
    }
    __device__ bool wait_warp(uint64_t *bar, int phase) {
        return __all_sync(0xffffffffu, wait(bar, phase));
    }
    __device__ void load(int tile, const CUtensorMap *m, uint64_t *bar, int y, int z) {
        for (int c = 0; c < C::SLABS; ++c)
            tma_load_3d(base + tile * C::TILE + c * kSlab, m, bar, c * 64, y, z);
    }
    __device__ uint32_t addr(int tile) { return smem_u32(base + tile * C::TILE); }

    // ------------------------------------------------------------- key tile
    // Tiles: 0 K, 1 V; ring slots 2 + i: Q_0 dO_0 Q_1 dO_1 ..; statistics in
    // the seventh.
    __device__ void keys() {
        const int j0 = it.tile * kTile, TT = maps.tokens, R = TT * a.G;
        const int shift = seq.lk - seq.lq;
        const int first = max(0, j0 - shift) / TT, last = (seq.lq + TT - 1) / TT;
        const int n = max(0, last - first);
        float *stats = reinterpret_cast<float *>(base + 6 * C::TILE);   // [2][2][128]
        constexpr uint32_t TM_V = 256, TM_K = 256 + D;
        if (n > 0 && warp == 9) {
            bool ok = true;
            if (lane == 0) {
                mbar_expect_tx(&sh.fix, 2 * C::TILE);
                load(0, &maps.k, &sh.fix, it.head, (int)(seq.k0 + j0));
                load(1, &maps.v, &sh.fix, it.head, (int)(seq.k0 + j0));
                int j = 0;
                for (; j < 2 * n; ++j) {
                    const int slot = j % 4, use = j / 4;
                    if (use > 0 && !mbar_wait_or_abort(&sh.empty[slot], (uint32_t)((use - 1) & 1),
                                                       &sh.abort)) {
                        give_up();
                        break;
                    }
                    mbar_expect_tx(&sh.full[slot], (uint32_t)R * 128u * C::SLABS);
                    load(2 + slot, j % 2 ? &maps.go : &maps.q, &sh.full[slot], it.head * a.G,
                         (int)(seq.q0 + (long long)(first + j / 2) * TT));
                }
                ok = j == 2 * n;
                if (!ok) {
                    for (int i = max(0, j - 4); i < j; ++i)
                        (void)mbar_wait(&sh.full[i % 4], (uint32_t)((i / 4) & 1));
                    (void)mbar_wait(&sh.fix, 0u);
                }
            }
            const int valid = (seq.lq - (last - 1) * TT) * a.G;
            if (__all_sync(0xffffffffu, ok) && valid < R)
                for (int j = 2 * n - 2; j < 2 * n; ++j) {
                    (void)mbar_wait(&sh.full[j % 4], (uint32_t)((j / 4) & 1));
                    attn::zero_rows<C::SLABS>(base + (2 + j % 4) * C::TILE, valid, lane);
                    if (lane == 0) mbar_arrive(&sh.tail[j & 1]);
                }
        } else if (n > 0 && warp == 8) {
            constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t id_h = idesc_bf16_f32(128, 64, false, false);
            constexpr uint32_t id_g = idesc_bf16_f32(128, D, false, true);
            // D (two halves of 64 columns) = tile A x rows of the slot
            const auto product = [&](int A, int slot, uint32_t c0, uint32_t c1, uint64_t *bar) {
                const uint32_t x = addr(A), y = addr(2 + slot);
                if (c1 == c0 + 64) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_bf16(tb + c0, attn::kdesc(x, ks), attn::kdesc(y, ks), id_s, ks > 0);
                } else {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_bf16(tb + c0, attn::kdesc(x, ks), attn::kdesc(y, ks), id_h, ks > 0);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)         // rows 64 .. 127 of each slab
                        mma_bf16(tb + c1, attn::kdesc(x, ks), attn::kdesc(y + 8192, ks), id_h,
                                 ks > 0);
                }
                mma_commit(bar);
            };
            const auto gather = [&](uint32_t out, uint32_t block, int slot, bool acc) {
                const uint32_t y = addr(2 + slot);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    mma_bf16_ts(tb + out, tb + block + 8u * ks, attn::mdesc(y, ks), id_g,
                                acc || ks > 0);
                mma_commit(&sh.empty[slot]);
            };
            // the last row tile may end inside: the loads' warp zeroes what
            // follows, which is a neighbour's
            const bool ragged = last * TT > seq.lq;
            const auto landed = [&](int j) {
                return wait(&sh.full[j % 4], j / 4) &&
                       (!ragged || j < 2 * n - 2 || wait(&sh.tail[j & 1], 0));
            };
            if (lane == 0) {
            bool ok = wait(&sh.fix, 0) && landed(0);
            if (ok) {
                const Blocks b = blocks_of(0);
                product(0, 0, b.s0, b.s1, &sh.s[0]);
                ok = landed(1);
                if (ok) product(1, 1, b.d0, b.d1, &sh.dp);
                ok = ok && wait(&sh.p, 0);
                if (ok) {
                    tc_fence_after();
                    gather(TM_V, b.p, 1, false);
                }
            }
            for (int i = 0; ok && i < n; ++i) {
                const Blocks b = blocks_of(i), c = blocks_of(i + 1);
                const bool more = i + 1 < n;
                ok = wait(&sh.ds, i) && (!more || landed(2 * i + 2));
                if (!ok) break;
                tc_fence_after();
                if (more) product(0, (2 * i + 2) % 4, c.s0, c.s1, &sh.s[0]);
                gather(TM_K, b.ds, (2 * i) % 4, i > 0);
                if (more) {
                    ok = landed(2 * i + 3);
                    if (!ok) break;
                    product(1, (2 * i + 3) % 4, c.d0, c.d1, &sh.dp);
                    ok = wait(&sh.p, i + 1);
                    if (!ok) break;
                    tc_fence_after();
                    gather(TM_V, c.p, (2 * i + 3) % 4, true);
                }
            }
            if (!ok) give_up();
            mma_commit(&sh.fin);
            (void)mbar_wait(&sh.fin, 0u);
            }
            __syncwarp();
        } else if (n > 0 && warp == 10) {
            // -lse log2 e and -delta of the tile's rows; a row that is none, or
            // saw no key, gets p = exp2(-inf) = 0
            for (int i = 0; i < n; ++i) {
                if (i >= 2 && !wait_warp(&sh.read[i & 1], i / 2 - 1)) break;
                float *dst = stats + (i & 1) * 256;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int r = lane + 32 * z, tok = (first + i) * TT + r / a.G;
                    float nl = -INFINITY, nd = 0.f;
                    if (r < R && tok < seq.lq) {
                        const long long at = (seq.q0 + tok) * a.Hq + it.head * a.G + r % a.G;
                        const float l = a.lse_in[at];
                        nl = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
                        nd = -a.delta[at];
                    }
                    dst[r] = nl;
                    dst[128 + r] = nd;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.st[i & 1]);
            }
        } else if (warp < 8) {
            const int half = warp / 4, w = warp % 4, key = j0 + 32 * w + lane;
            const uint32_t lanes = (uint32_t)(32 * w) << 16;
            const float c = a.scale_log2;
            bool ok = true;
            for (int i = 0; i < n; ++i) {
                const Blocks b = blocks_of(i);
                float p[64];
                const float *st = stats + (i & 1) * 256 + 64 * half;
                ok = ok && wait_warp(&sh.st[i & 1], i / 2) && wait_warp(&sh.s[0], i);
                if (ok) {
                    tc_fence_after();
                    uint32_t x[2][32];
                    const uint32_t tS = tb + (half ? b.s1 : b.s0) + lanes;
                    tmem_ld32(tS, x[0]);
                    tmem_ld32(tS + 32, x[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 64; k += 4) {
                        const float4 nl = *reinterpret_cast<const float4 *>(st + k);
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            p[k + z] = __uint_as_float(x[k / 32][k % 32 + z]);
                        fma2v(p[k], p[k + 1], c, nl.x, nl.y);
                        fma2v(p[k + 2], p[k + 3], c, nl.z, nl.w);
#pragma unroll
                        for (int z = 0; z < 4; ++z) p[k + z] = attn::ex2(p[k + z]);
                    }
                    const int tok0 = (first + i) * TT;
                    if (tok0 + shift < j0 + kTile - 1) {
                        // the rows are in the order of their tokens: those from
                        // `from` on see this key
                        const int from = min(max(key - shift - tok0, 0), TT) * a.G - 64 * half;
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (k < from) p[k] = 0.f;
                    }
                }
                tc_fence_before();
                named_sync(1, kSoftmax);      // both halves of S^T are read
                if (ok) {
                    tc_fence_after();
                    uint32_t y[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) y[k] = attn::pack2(p[2 * k], p[2 * k + 1]);
                    attn::tmem_st32(tb + b.p + 32u * half + lanes, y);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p);
                    ok = wait_warp(&sh.dp, i);
                }
                if (ok) {
                    tc_fence_after();
                    uint32_t x[2][32];
                    const uint32_t tD = tb + (half ? b.d1 : b.d0) + lanes;
                    tmem_ld32(tD, x[0]);
                    tmem_ld32(tD + 32, x[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 64; k += 4) {
                        const float4 nd = *reinterpret_cast<const float4 *>(st + 128 + k);
                        float d[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) d[z] = __uint_as_float(x[k / 32][k % 32 + z]);
                        attn::add2(d[0], d[1], nd.x, nd.y);
                        attn::add2(d[2], d[3], nd.z, nd.w);
                        mul2(p[k], p[k + 1], d[0], d[1]);
                        mul2(p[k + 2], p[k + 3], d[2], d[3]);
                    }
                }
                tc_fence_before();
                named_sync(1, kSoftmax);      // both halves of dP^T are read
                if (ok) {
                    tc_fence_after();
                    uint32_t y[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) y[k] = attn::pack2(p[2 * k], p[2 * k + 1]);
                    attn::tmem_st32(tb + b.ds + 32u * half + lanes, y);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh.ds);
                        mbar_arrive(&sh.read[i & 1]);
                    }
                }
            }
            if (n > 0) ok = ok && wait_warp(&sh.fin, 0);
            if (!ok) {
                give_up();
            } else {
                tc_fence_after();
                const long long at = ((seq.k0 + key) * a.Hk + it.head) * D;
                store_row<D>(tb + (half ? TM_K : TM_V) + lanes,
                             static_cast<__nv_bfloat16 *>(half ? a.dk : a.dv) + at,
                             half ? a.scale : 1.f, n > 0, key < seq.lk);
            }
        }
    }

    // ------------------------------------------------------------- row tile
    // Tiles: 0 Q, 1 dO; 2, 3, 4 the ring of K; 5, 6 of V.  Ring barriers: K 0
    // to 2, V 3 and 4.
    __device__ void rows() {
        const int TT = maps.tokens, R = TT * a.G, tok0 = it.tile * TT;
        const int shift = seq.lk - seq.lq;
        const int seen = min(tok0 + TT, seq.lq) + shift;
        const int n = seen > 0 ? (seen + kTile - 1) / kTile : 0;
        constexpr uint32_t TM_P = 256, TM_Q = 384;
        if (n > 0 && warp == 9) {
            bool ok = true;
            if (lane == 0) {
                const uint32_t box = (uint32_t)R * 128u * C::SLABS;
                mbar_expect_tx(&sh.fix, 2 * box);
                load(0, &maps.q, &sh.fix, it.head * a.G, (int)(seq.q0 + tok0));
                load(1, &maps.go, &sh.fix, it.head * a.G, (int)(seq.q0 + tok0));
                int nk = 0, nv = 0;           // tiles asked for
                const auto next = [&](bool value, int i) {
                    const int slot = value ? 3 + i % 2 : i % 3, use = value ? i / 2 : i / 3;
                    if (use > 0 && !mbar_wait_or_abort(&sh.empty[slot], (uint32_t)((use - 1) & 1),
                                                       &sh.abort)) {
                        ok = false;
                        return;
                    }
                    mbar_expect_tx(&sh.full[slot], C::TILE);
                    load(2 + slot, value ? &maps.v : &maps.k, &sh.full[slot], it.head,
                         (int)(seq.k0 + (long long)i * kTile));
                    ++(value ? nv : nk);
                };
                next(false, 0);
                for (int i = 0; ok && i < n; ++i) {      // in the order of their first use
                    if (i + 1 < n) next(false, i + 1);
                    if (ok) next(true, i);
                }
                if (!ok) {
                    give_up();
                    for (int i = max(0, nk - 3); i < nk; ++i)
                        (void)mbar_wait(&sh.full[i % 3], (uint32_t)((i / 3) & 1));
                    for (int i = max(0, nv - 2); i < nv; ++i)
                        (void)mbar_wait(&sh.full[3 + i % 2], (uint32_t)((i / 2) & 1));
                    (void)mbar_wait(&sh.fix, 0u);
                }
            }
            const int valid = seq.lk - (n - 1) * kTile;
            if (__all_sync(0xffffffffu, ok) && valid < kTile) {
                const int slot = (n - 1) % 3;
                (void)mbar_wait(&sh.full[slot], (uint32_t)(((n - 1) / 3) & 1));
                attn::zero_rows<C::SLABS>(base + (2 + slot) * C::TILE, valid, lane);
                if (lane == 0) mbar_arrive(&sh.tail[0]);
            }
        } else if (n > 0 && warp == 8) {
            constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t id_g = idesc_bf16_f32(128, D, false, true);
            const auto product = [&](int A, int tile, uint32_t out, uint64_t *bar) {
                const uint32_t x = addr(A), y = addr(tile);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16(tb + out, attn::kdesc(x, ks), attn::kdesc(y, ks), id_s, ks > 0);
                mma_commit(bar);
            };
            // the keys' rows are summed over in dQ: those behind the last are a
            // neighbour's, and the loads' warp zeroes them
            const bool ragged = n * kTile > seq.lk;
            const auto scores = [&](int i) {
                if (!wait(&sh.full[i % 3], i / 3)) return false;
                if (ragged && i == n - 1 && !wait(&sh.tail[0], 0)) return false;
                product(0, 2 + i % 3, 128u * (i & 1), &sh.s[i & 1]);
                return true;
            };
            const auto grads = [&](int i) {
                if (!wait(&sh.full[3 + i % 2], i / 2)) return false;
                product(1, 5 + i % 2, TM_P, &sh.dp);
                mma_commit(&sh.empty[3 + i % 2]);
                return true;
            };
            if (lane == 0) {
            bool ok = wait(&sh.fix, 0) && scores(0) && grads(0) && (n < 2 || scores(1));
            for (int i = 0; ok && i < n; ++i) {
                ok = wait(&sh.ds, i);
                tc_fence_after();
                ok = ok && (i + 1 >= n || grads(i + 1));
                if (!ok) break;
                const uint32_t y = addr(2 + i % 3);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)          // dS: 32 columns in each half of S's
                    mma_bf16_ts(tb + TM_Q, tb + 128u * (i & 1) + 64u * (ks / 4) + 8u * (ks % 4),
                                attn::mdesc(y, ks), id_g, i > 0 || ks > 0);
                mma_commit(&sh.empty[i % 3]);
                if (i + 2 < n) ok = scores(i + 2);
            }
            if (!ok) give_up();
            mma_commit(&sh.fin);
            (void)mbar_wait(&sh.fin, 0u);
            }
            __syncwarp();
        } else if (warp < 8) {
            const int half = warp / 4, w = warp % 4, r = 32 * w + lane;
            const int tok = tok0 + r / a.G;
            const bool row = r < R && tok < seq.lq;
            const int limit = row ? tok + shift : -1, full = tok0 + shift;
            const long long at = (seq.q0 + tok) * a.Hq + it.head * a.G + r % a.G;
            const uint32_t lanes = (uint32_t)(32 * w) << 16;
            const float c = a.scale_log2;
            float nl = -INFINITY, nd = 0.f;
            if (row) {
                const float l = a.lse_in[at];
                nl = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
                nd = -a.delta[at];
            }
            bool ok = true;
            for (int i = 0; ok && i < n; ++i) {
                ok = wait_warp(&sh.s[i & 1], i / 2);
                if (!ok) break;
                tc_fence_after();
                const uint32_t tS = tb + 128u * (i & 1) + 64u * half + lanes;
                float p[64];
                {
                    uint32_t x[2][32];
                    tmem_ld32(tS, x[0]);
                    tmem_ld32(tS + 32, x[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 64; k += 2) {
                        p[k] = __uint_as_float(x[k / 32][k % 32]);
                        p[k + 1] = __uint_as_float(x[k / 32][k % 32 + 1]);
                        attn::fma2(p[k], p[k + 1], c, nl);
                        p[k] = attn::ex2(p[k]);
                        p[k + 1] = attn::ex2(p[k + 1]);
                    }
                }
                ok = wait_warp(&sh.dp, i);
                if (!ok) break;
                tc_fence_after();
                uint32_t x[2][32];
                const uint32_t tD = tb + TM_P + 64u * half + lanes;
                tmem_ld32(tD, x[0]);
                tmem_ld32(tD + 32, x[1]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 64; k += 2) {
                    float d0 = __uint_as_float(x[k / 32][k % 32]);
                    float d1 = __uint_as_float(x[k / 32][k % 32 + 1]);
                    attn::add2(d0, d1, nd, nd);
                    mul2(p[k], p[k + 1], d0, d1);
                }
                if (i * kTile + kTile - 1 > full) {
                    const int rel = limit - i * kTile - 64 * half;
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (k > rel) p[k] = 0.f;
                }
                uint32_t y[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) y[k] = attn::pack2(p[2 * k], p[2 * k + 1]);
                attn::tmem_st32(tS, y);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.ds);
            }
            if (n > 0) ok = ok && wait_warp(&sh.fin, 0);
            if (!ok) {
                give_up();
            } else {
                tc_fence_after();
                // the halves of the row's features to the two warpgroups
                store_row<D / 2>(tb + TM_Q + (uint32_t)(D / 2 * half) + lanes,
                                 static_cast<__nv_bfloat16 *>(a.dq) + at * D + D / 2 * half,
                                 a.scale, n > 0, row);
            }
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_bwd_kernel(const __grid_constant__ Args ak, const __grid_constant__ Args ar,
                   const __grid_constant__ Maps maps, int key_blocks) {
    using C = Cfg<D>;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const bool key_tile = (int)blockIdx.x < key_blocks;
    const Args &a = key_tile ? ak : ar;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    Item it;
    if (!attn::item_of(a, key_tile ? blockIdx.x : blockIdx.x - key_blocks, !key_tile, it)) return;
    const Seq seq = attn::sequence(a, it.seq);

    if (threadIdx.x == 0) {
        mbar_init(&sh.fix, 1);
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s[i], 1);
            mbar_init(&sh.tail[i], 1);
            mbar_init(&sh.st[i], 1);
            mbar_init(&sh.read[i], 8);
        }
        mbar_init(&sh.dp, 1);
        mbar_init(&sh.p, 8);
        mbar_init(&sh.ds, 8);
        mbar_init(&sh.fin, 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    // rows that no copy fills (the group does not divide 128) are summed over
    // by a key tile's products
    const int R = maps.tokens * a.G;
    if (key_tile && R < kTile && warp < 8 && warp / 2 < 4 && warp % 2 == 0)
        attn::zero_rows<C::SLABS>(base + (2 + warp / 2) * C::TILE, R, lane);
    if (warp == 8) tmem_alloc(&sh.tmem, C::TM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    Cta<D> cta{a, maps, sh, base, sh.tmem, warp, lane, it, seq};
    if (key_tile) cta.keys();
    else cta.rows();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) {
        tmem_relinquish();
        tmem_dealloc(sh.tmem, C::TM_COLS);
    }
}

template <int D>
cudaError_t launch_bwd(const Args &keys, const Args &rows, const Maps &maps, cudaStream_t s) {
    const long long kb = (long long)keys.items * keys.Hk, rb = (long long)rows.items * rows.Hk;
    if (kb + rb == 0) return cudaSuccess;
    cudaError_t e = attn_allow_smem(reinterpret_cast<const void *>(attn_tc_bwd_kernel<D>), Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    attn_tc_bwd_kernel<D><<<(unsigned)(kb + rb), kThreads, Cfg<D>::SMEM, s>>>(keys, rows, maps,
                                                                              (int)kb);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc_bwd(const Args &keys, const Args &rows, int d, int total_k,
                               cudaStream_t s) {
    Maps maps;
    maps.tokens = attn::tile_tokens(rows.G);
    if (!attn::map_rows(&maps.q, rows.q, d, rows.Hq, rows.total_q, rows.q_stride, rows.G,
                        maps.tokens) ||
        !attn::map_rows(&maps.go, rows.go, d, rows.Hq, rows.total_q, rows.go_stride, rows.G,
                        maps.tokens) ||
        !attn::map_rows(&maps.k, rows.k, d, rows.Hk, total_k, rows.k_stride, 1, kTile) ||
        !attn::map_rows(&maps.v, rows.v, d, rows.Hk, total_k, rows.v_stride, 1, kTile))
        return cudaErrorInvalidValue;
    return d == 128 ? launch_bwd<128>(keys, rows, maps, s) : launch_bwd<64>(keys, rows, maps, s);
}

}  // namespace kla
