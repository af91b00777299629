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
// Order of a key tile's products: dV runs under the dS step, dK and the next
// dP^T under the exponentials.  P^T takes the columns of S^T, dS^T those of
// dP^T:
//
//     S' (next)   dK   dP'   dV'
//     [ds done]        [exp: P']   [ds']
//
// A wait takes 100 to 150 cycles even where there is nothing to wait for, and
// the queue of issued products about 300: two warps issue, one lane each, so
// that one's waits run under the other's products.  Products that overwrite
// what an earlier one reads are the same lane's (dV, then S^T; dK, then dP^T;
// dQ, then S), so they run in order.
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
    uint64_t s[2], dp, p, ds[2];         // products ready; operands ready
    uint64_t turn[2];                    // of the second warp of products
    uint64_t st[2], read[2];             // row statistics ready, and read
    uint64_t tail[2], fin;
    uint32_t tmem;
    volatile int abort;
};

struct Maps {
    CUtensorMap q, go, k, v;
    int tokens;                          // of a row tile
};

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
    int TT, R, shift;         // tokens and rows of a row tile; lk - lq
    int j0, tok0;             // key tile: its first key; row tile: its first token
    int first, last, n;       // tiles of the other side: first .. last, how many
    float *stats;             // key tiles: [2][-lse log2 e, -delta][128]

    // Tensor memory of a key tile: S^T, dP^T, dV, dK; of a row tile: S twice, dP, dQ.
    static constexpr uint32_t TM_S = 0, TM_P = 128, TM_V = 256, TM_K = 256 + D;
    static constexpr uint32_t TM_DP = 256, TM_Q = 384;

    __device__ Cta(const Args &a_, const Maps &maps_, Shared &sh_, unsigned char *base_, int warp_,
                   int lane_, const Item &it_, const Seq &seq_, bool key_tile)
        : a(a_), maps(maps_), sh(sh_), base(base_), tb(sh_.tmem), warp(warp_), lane(lane_),
          it(it_), seq(seq_) {
        TT = maps.tokens;
        R = TT * a.G;
        shift = seq.lk - seq.lq;
        j0 = it.tile * kTile;
        tok0 = it.tile * TT;
        stats = reinterpret_cast<float *>(base + 6 * C::TILE);
        first = 0;
        if (key_tile) {
            first = max(0, j0 - shift) / TT;
            last = (seq.lq + TT - 1) / TT;
        } else {
            const int seen = min(tok0 + TT, seq.lq) + shift;
            last = seen > 0 ? (seen + kTile - 1) / kTile : 0;
        }
        n = max(0, last - first);
    }
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
    // K step ks of an operand in the columns of the product it came from, 32
    // columns in each half (a warpgroup's own).
    static __device__ uint32_t operand(uint32_t col, int ks) {
        return col + 64u * (ks / 4) + 8u * (ks % 4);
    }
    __device__ uint32_t addr(int tile) { return smem_u32(base + tile * C::TILE); }

    // ------------------------------------------------------------- key tile
    // Tiles: 0 K, 1 V; ring slots 2 + i: Q_0 dO_0 Q_1 dO_1 ..; statistics in
    // the seventh.
    // Loads, products and statistics (warps 8 to 10).
    __device__ void keys_work() {
        if (n == 0) return;
        if (warp == 9) {
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
        } else if (warp == 8 || warp == 11) {
            // two warps, a lane each: S^T and dV, dP^T and dK
            if (lane == 0) {
                constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
                constexpr uint32_t id_g = idesc_bf16_f32(128, D, false, true);
                // tile A (K or V) x the rows of a slot
                const auto product = [&](int A, int j, uint32_t out, uint64_t *bar) {
                    const uint32_t x = addr(A), y = addr(2 + j % 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_bf16(tb + out, attn::kdesc(x, ks), attn::kdesc(y, ks), id_s, ks > 0);
                    mma_commit(bar);
                };
                // P^T or dS^T x the rows of a slot
                const auto gather = [&](uint32_t from, int j, uint32_t out, bool acc) {
                    const uint32_t y = addr(2 + j % 4);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_bf16_ts(tb + out, tb + operand(from, ks), attn::mdesc(y, ks), id_g,
                                    acc || ks > 0);
                    mma_commit(&sh.empty[j % 4]);
                };
                // the last row tile may end inside: the loads' warp zeroes what
                // follows, which is a neighbour's
                const bool ragged = last * TT > seq.lq;
                const auto landed = [&](int j) {
                    return wait(&sh.full[j % 4], j / 4) &&
                           (!ragged || j < 2 * n - 2 || wait(&sh.tail[j & 1], 0));
                };
                bool ok = wait(&sh.fix, 0);
                if (warp == 8) {
                    ok = ok && landed(0);
                    if (ok) product(0, 0, TM_S, &sh.s[0]);
                    for (int i = 0; ok && i < n; ++i) {
                        ok = wait(&sh.p, i);
                        if (!ok) break;
                        tc_fence_after();
                        gather(TM_S, 2 * i + 1, TM_V, i > 0);
                        if (i + 1 == n) break;
                        ok = landed(2 * i + 2) && wait(&sh.ds[i & 1], i / 2);
                        if (!ok) break;
                        product(0, 2 * i + 2, TM_S, &sh.s[0]);
                        mbar_arrive(&sh.turn[0]);
                    }
                } else {
                    ok = ok && landed(1);
                    if (ok) {
                        product(1, 1, TM_P, &sh.dp);
                        mma_commit(&sh.empty[1]);
                    }
                    for (int i = 0; ok && i < n; ++i) {
                        const bool more = i + 1 < n;
                        ok = (!more || landed(2 * i + 3)) && wait(&sh.ds[i & 1], i / 2) &&
                             (!more || wait(&sh.turn[0], i));
                        if (!ok) break;
                        tc_fence_after();
                        gather(TM_P, 2 * i, TM_K, i > 0);
                        if (!more) break;
                        product(1, 2 * i + 3, TM_P, &sh.dp);
                        mma_commit(&sh.empty[(2 * i + 3) % 4]);
                    }
                }
                if (!ok) give_up();
                mma_commit(&sh.fin);
                (void)mbar_wait(&sh.fin, 0u);
            }
            __syncwarp();
        } else if (warp == 10) {
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
        }
    }
    __device__ void keys_softmax() {
        {
            const int half = warp / 4, w = warp % 4, key = j0 + 32 * w + lane;
            const uint32_t at_s = tb + TM_S + 64u * half + ((uint32_t)(32 * w) << 16);
            const uint32_t at_p = at_s + (TM_P - TM_S);
            const float c = a.scale_log2;
            bool ok = true;
            for (int i = 0; ok && i < n; ++i) {
                // the rows' statistics into registers ahead of the waits: the
                // products hold shared memory busy, and a read takes its time
                const float4 *st = reinterpret_cast<const float4 *>(stats + (i & 1) * 256 + 64 * half);
                ok = wait_warp(&sh.st[i & 1], i / 2);
                if (!ok) break;
                float p[64];
                {
                    float4 nl[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) nl[k] = st[k];
                    ok = wait_warp(&sh.s[0], i);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t x[2][32];
                    tmem_ld32(at_s, x[0]);
                    tmem_ld32(at_s + 32, x[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 64; k += 4) {
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            p[k + z] = __uint_as_float(x[k / 32][k % 32 + z]);
                        fma2v(p[k], p[k + 1], c, nl[k / 4].x, nl[k / 4].y);
                        fma2v(p[k + 2], p[k + 3], c, nl[k / 4].z, nl[k / 4].w);
#pragma unroll
                        for (int z = 0; z < 4; ++z) p[k + z] = attn::ex2(p[k + z]);
                    }
                }
                const int t0 = (first + i) * TT;
                if (t0 + shift < j0 + kTile - 1) {
                    // the rows are in the order of their tokens: those from
                    // `from` on see this key
                    const int from = min(max(key - shift - t0, 0), TT) * a.G - 64 * half;
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (k < from) p[k] = 0.f;
                }
                {
                    uint32_t y[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) y[k] = attn::pack2(p[2 * k], p[2 * k + 1]);
                    attn::tmem_st32(at_s, y);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p);
                float4 nd[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) nd[k] = st[32 + k];
                ok = wait_warp(&sh.dp, i);
                if (!ok) break;
                tc_fence_after();
                uint32_t x[2][32];
                tmem_ld32(at_p, x[0]);
                tmem_ld32(at_p + 32, x[1]);
                tmem_ld_wait();
                uint32_t y[32];
#pragma unroll
                for (int k = 0; k < 64; k += 4) {
                    float d[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) d[z] = __uint_as_float(x[k / 32][k % 32 + z]);
                    attn::add2(d[0], d[1], nd[k / 4].x, nd[k / 4].y);
                    attn::add2(d[2], d[3], nd[k / 4].z, nd[k / 4].w);
                    mul2(d[0], d[1], p[k], p[k + 1]);
                    mul2(d[2], d[3], p[k + 2], p[k + 3]);
                    y[k / 2] = attn::pack2(d[0], d[1]);
                    y[k / 2 + 1] = attn::pack2(d[2], d[3]);
                }
                attn::tmem_st32(at_p, y);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.ds[i & 1]);
                    mbar_arrive(&sh.read[i & 1]);
                }
            }
            if (n > 0) ok = ok && wait_warp(&sh.fin, 0);
            if (!ok) {
                give_up();
            } else {
                tc_fence_after();
                const long long at = ((seq.k0 + key) * a.Hk + it.head) * D;
                store_row<D>(tb + (half ? TM_K : TM_V) + ((uint32_t)(32 * w) << 16),
                             static_cast<__nv_bfloat16 *>(half ? a.dk : a.dv) + at,
                             half ? a.scale : 1.f, n > 0, key < seq.lk);
            }
        }
    }

    // ------------------------------------------------------------- row tile
    // Tiles: 0 Q, 1 dO; 2, 3, 4 the ring of K; 5, 6 of V.  Ring barriers: K 0
    // to 2, V 3 and 4.
    __device__ void rows_work() {
        if (n == 0) return;
        if (warp == 9) {
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
        } else if (warp == 8 || warp == 11) {
            // two warps, a lane each: S and dQ, dP
            if (lane == 0) {
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
                const auto key_landed = [&](int i) {
                    return wait(&sh.full[i % 3], i / 3) &&
                           (!ragged || i < n - 1 || wait(&sh.tail[0], 0));
                };
                const auto value_landed = [&](int i) { return wait(&sh.full[3 + i % 2], i / 2); };
                const auto scores = [&](int i) { product(0, 2 + i % 3, 128u * (i & 1), &sh.s[i & 1]); };
                const auto grads = [&](int i) {
                    product(1, 5 + i % 2, TM_DP, &sh.dp);
                    mma_commit(&sh.empty[3 + i % 2]);
                };
                bool ok = wait(&sh.fix, 0);
                if (warp == 8) {
                    for (int i = 0; ok && i < 2 && i < n; ++i) {
                        ok = key_landed(i);
                        if (ok) scores(i);
                    }
                    for (int i = 0; ok && i < n; ++i) {
                        ok = (i + 2 >= n || key_landed(i + 2)) && wait(&sh.ds[i & 1], i / 2) &&
                             (i + 1 >= n || wait(&sh.turn[i & 1], i / 2));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t y = addr(2 + i % 3);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_bf16_ts(tb + TM_Q, tb + operand(128u * (i & 1), ks),
                                        attn::mdesc(y, ks), id_g, i > 0 || ks > 0);
                        mma_commit(&sh.empty[i % 3]);
                        if (i + 2 < n) scores(i + 2);
                    }
                } else {
                    for (int i = 0; ok && i < n; ++i) {
                        ok = value_landed(i) && (i == 0 || wait(&sh.ds[(i - 1) & 1], (i - 1) / 2));
                        if (!ok) break;
                        grads(i);
                        if (i > 0) mbar_arrive(&sh.turn[(i - 1) & 1]);
                    }
                }
                if (!ok) give_up();
                mma_commit(&sh.fin);
                (void)mbar_wait(&sh.fin, 0u);
            }
            __syncwarp();
        }
    }
    __device__ void rows_softmax() {
        {
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
                const uint32_t tD = tb + TM_DP + 64u * half + lanes;
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
                if (lane == 0) mbar_arrive(&sh.ds[i & 1]);
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
            // a key tile's dO slots are read by both warps of products
            mbar_init(&sh.empty[i], key_tile && i % 2 == 1 ? 2 : 1);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s[i], 1);
            mbar_init(&sh.ds[i], 8);
            mbar_init(&sh.turn[i], 1);
            mbar_init(&sh.tail[i], 1);
            mbar_init(&sh.st[i], 1);
            mbar_init(&sh.read[i], 8);
        }
        mbar_init(&sh.dp, 1);
        mbar_init(&sh.p, 8);
        mbar_init(&sh.fin, 2);
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
    Cta<D> cta(a, maps, sh, base, warp, lane, it, seq, key_tile);
    // Registers of a thread: 128 x 88 + 256 x 208 = 384 x 168.
    if (warp >= 8) {
        attn::fewer_registers<88>();
        if (key_tile) cta.keys_work();
        else cta.rows_work();
    } else {
        attn::more_registers<208>();
        if (key_tile) cta.keys_softmax();
        else cta.rows_softmax();
    }
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
