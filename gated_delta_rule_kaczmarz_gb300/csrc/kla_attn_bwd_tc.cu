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
// Order of the products.  A key tile's next scores do not wait for dS: P is in
// registers for that step, and S^T's columns are free after dV.  So the dS step
// runs under dV and S^T, the exponentials under dK and dP^T:
//
//     dK   dP^T   |  dV   S^T (next)  |  dK   dP^T
//     [exp: P]    |  [dS]             |  [exp: P]
//
// P^T takes the columns of S^T, dS^T those of dP^T.  A row tile has dP twice:
// S and dP of the next tile run under the dS step, then dQ.
//
// A wait takes 100 to 150 cycles even where there is nothing to wait for, and
// the queue of issued products about 300: one lane waits and issues, and a key
// tile has two such warps, so that one's waits run under the other's products.
// Products that overwrite what an earlier one reads are the same lane's (dV,
// then S^T; dK, then dP^T), so they run in order.
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

struct Shared {
    uint64_t fix;                        // the CTA's own tiles landed
    uint64_t full[5], empty[5];          // ring slots
    uint64_t s, dp[2];                   // scores and dP ready
    uint64_t s_read, p, ds[2];           // scores read; P and dS in place
    uint64_t st[2], read[2];             // row statistics ready, and read
    uint64_t tail[2], fin;
    uint32_t tmem;
    volatile int abort;
};

template <int D>
struct Cfg {
    static constexpr int SLABS = D / 64;
    static constexpr uint32_t TILE = SLABS * kSlab;
    // seven tiles, the row statistics of two, the barriers; what is left of a
    // block's 227 KB covers the alignment
    static constexpr size_t STATS = (size_t)TILE * 7, BARS = STATS + 2048;
    static constexpr size_t USED = BARS + 256;
    static constexpr size_t SMEM = USED + 768;
    static constexpr uint32_t TM_COLS = 512;
    static_assert(sizeof(Shared) <= 256 && SMEM <= 227 * 1024, "shared memory");
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
    unsigned char *base;      // tiles 0, 1: the CTA's own; 2 to 4: ring X; 5, 6: ring Y
    uint32_t tb;
    int warp, lane;
    bool key_tile;
    Item it;
    Seq seq;
    int TT, R, shift;         // tokens and rows of a row tile; lk - lq
    int j0, tok0;             // key tile: its first key; row tile: its first token
    int first, last, n;       // tiles of the other side: first .. last, how many
    int valid;                // rows of the last of them that are the sequence's own
    float *stats;             // key tiles: [2][-lse log2 e, -delta][128]

    // Tensor memory of a key tile: S^T, dP^T, dV, dK; of a row tile: S, dP twice, dQ.
    static constexpr uint32_t TM_S = 0, TM_P = 128, TM_V = 256, TM_K = 256 + D, TM_Q = 384;

    __device__ Cta(const Args &a_, const Maps &maps_, Shared &sh_, unsigned char *base_, int warp_,
                   int lane_, const Item &it_, const Seq &seq_, bool key_tile_)
        : a(a_), maps(maps_), sh(sh_), base(base_), tb(sh_.tmem), warp(warp_), lane(lane_),
          key_tile(key_tile_), it(it_), seq(seq_) {
        TT = maps.tokens;
        R = TT * a.G;
        shift = seq.lk - seq.lq;
        j0 = it.tile * kTile;
        tok0 = it.tile * TT;
        stats = reinterpret_cast<float *>(base + C::STATS);
        if (key_tile) {
            first = max(0, j0 - shift) / TT;
            last = (seq.lq + TT - 1) / TT;
            valid = min((seq.lq - (last - 1) * TT) * a.G, R);
        } else {
            const int seen = min(tok0 + TT, seq.lq) + shift;
            first = 0;
            last = seen > 0 ? (seen + kTile - 1) / kTile : 0;
            valid = min(seq.lk - (last - 1) * kTile, kTile);
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
    __device__ uint32_t addr(int tile) { return smem_u32(base + tile * C::TILE); }
    // K step ks of an operand in the columns of the product it came from, 32
    // columns in each half (a warpgroup's own).
    static __device__ uint32_t operand(uint32_t col, int ks) {
        return col + 64u * (ks / 4) + 8u * (ks % 4);
    }

    // Ring slots of the i-th tile of the other side: Q (key tile) or K in X, dO
    // or V in Y.  Those of the last tile's rows that are a neighbour's are
    // zeroed before they are summed over.
    static __device__ int slot_x(int i) { return i % 3; }
    static __device__ int slot_y(int i) { return 3 + i % 2; }
    __device__ bool ragged() const { return valid < (key_tile ? R : kTile); }
    __device__ bool landed_x(int i) {
        return wait(&sh.full[slot_x(i)], i / 3) &&
               (i < n - 1 || !ragged() || wait(&sh.tail[0], 0));
    }
    __device__ bool landed_y(int i) {
        return wait(&sh.full[slot_y(i)], i / 2) &&
               (i < n - 1 || !ragged() || !key_tile || wait(&sh.tail[1], 0));
    }
    __device__ void load(int tile, const CUtensorMap *m, uint64_t *bar, int y, int z) {
        for (int c = 0; c < C::SLABS; ++c)
            tma_load_3d(base + tile * C::TILE + c * kSlab, m, bar, c * 64, y, z);
    }
    __device__ void loads() {
        bool ok = true;
        if (lane == 0) {
            const uint32_t rows = (uint32_t)R * 128u * C::SLABS, keys = C::TILE;
            const int hq = it.head * a.G, hk = it.head;
            const int q0 = (int)seq.q0, k0 = (int)seq.k0;
            mbar_expect_tx(&sh.fix, 2 * (key_tile ? keys : rows));
            load(0, key_tile ? &maps.k : &maps.q, &sh.fix, key_tile ? hk : hq,
                 key_tile ? k0 + j0 : q0 + tok0);
            load(1, key_tile ? &maps.v : &maps.go, &sh.fix, key_tile ? hk : hq,
                 key_tile ? k0 + j0 : q0 + tok0);
            const CUtensorMap *mx = key_tile ? &maps.q : &maps.k, *my = key_tile ? &maps.go : &maps.v;
            int nx = 0, ny = 0;           // tiles asked for
            const auto next = [&](bool y, int i) {
                const int slot = y ? slot_y(i) : slot_x(i), use = y ? i / 2 : i / 3;
                ok = use == 0 || wait(&sh.empty[slot], use - 1);
                if (!ok) return;
                mbar_expect_tx(&sh.full[slot], key_tile ? rows : keys);
                load(2 + slot, y ? my : mx, &sh.full[slot], key_tile ? hq : hk,
                     key_tile ? q0 + (first + i) * TT : k0 + i * kTile);
                ++(y ? ny : nx);
            };
            next(false, 0);
            for (int i = 0; ok && i < n; ++i) {      // in the order of their first use
                next(true, i);
                if (ok && i + 1 < n) next(false, i + 1);
            }
            if (!ok) {     // given up: the copies in flight land before the CTA leaves
                give_up();
                for (int i = max(0, nx - 3); i < nx; ++i)
                    (void)mbar_wait(&sh.full[slot_x(i)], (uint32_t)((i / 3) & 1));
                for (int i = max(0, ny - 2); i < ny; ++i)
                    (void)mbar_wait(&sh.full[slot_y(i)], (uint32_t)((i / 2) & 1));
                (void)mbar_wait(&sh.fix, 0u);
            }
        }
        if (!__all_sync(0xffffffffu, ok) || !ragged()) return;
        for (int y = 0; y < (key_tile ? 2 : 1); ++y) {
            const int slot = y ? slot_y(n - 1) : slot_x(n - 1), use = y ? (n - 1) / 2 : (n - 1) / 3;
            (void)mbar_wait(&sh.full[slot], (uint32_t)(use & 1));
            attn::zero_rows<C::SLABS>(base + (2 + slot) * C::TILE, valid, lane);
            if (lane == 0) mbar_arrive(&sh.tail[y]);
        }
    }

    // ---------------------------------------------------------- products
    // Tensor memory (128 columns at out) = own tile x the rows of a slot's tile.
    __device__ void product(int own, int slot, uint32_t out, uint64_t *bar) {
        constexpr uint32_t id = idesc_bf16_f32(128, 128, false, false);
        const uint32_t x = addr(own), y = addr(2 + slot);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
            mma_bf16(tb + out, attn::kdesc(x, ks), attn::kdesc(y, ks), id, ks > 0);
        mma_commit(bar);
    }
    // Tensor memory (D columns at out) += operand in tensor memory x a slot's tile.
    __device__ void gather(uint32_t from, int slot, uint32_t out, bool acc) {
        constexpr uint32_t id = idesc_bf16_f32(128, D, false, true);
        const uint32_t y = addr(2 + slot);
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
            mma_bf16_ts(tb + out, tb + operand(from, ks), attn::mdesc(y, ks), id, acc || ks > 0);
        mma_commit(&sh.empty[slot]);
    }
    __device__ void finish(bool ok) {
        if (!ok) give_up();
        mma_commit(&sh.fin);
        (void)mbar_wait(&sh.fin, 0u);
    }
    // S^T and dV of a key tile.
    __device__ void key_products_v() {
        bool ok = wait(&sh.fix, 0) && landed_x(0);
        if (ok) product(0, slot_x(0), TM_S, &sh.s);
        for (int i = 0; ok && i < n; ++i) {
            ok = landed_y(i) && wait(&sh.p, i);
            if (!ok) break;
            gather(TM_S, slot_y(i), TM_V, i > 0);
            if (i + 1 == n) break;
            ok = landed_x(i + 1);
            if (ok) product(0, slot_x(i + 1), TM_S, &sh.s);
        }
        finish(ok);
    }
    // dP^T and dK of a key tile.
    __device__ void key_products_k() {
        bool ok = wait(&sh.fix, 0) && landed_y(0);
        if (ok) {
            product(1, slot_y(0), TM_P, &sh.dp[0]);
            mma_commit(&sh.empty[slot_y(0)]);
        }
        for (int i = 0; ok && i < n; ++i) {
            ok = wait(&sh.ds[i & 1], i / 2);
            if (!ok) break;
            gather(TM_P, slot_x(i), TM_K, i > 0);
            if (i + 1 == n) break;
            ok = landed_y(i + 1);
            if (!ok) break;
            product(1, slot_y(i + 1), TM_P, &sh.dp[0]);
            mma_commit(&sh.empty[slot_y(i + 1)]);
        }
        finish(ok);
    }
    // All of a row tile.
    __device__ void row_products() {
        bool ok = wait(&sh.fix, 0);
        for (int i = 0; ok && i <= n; ++i) {
            if (i < n) {
                ok = landed_x(i) && (i == 0 || wait(&sh.s_read, i - 1));
                if (!ok) break;
                product(0, slot_x(i), TM_S, &sh.s);
                ok = landed_y(i);
                if (!ok) break;
                product(1, slot_y(i), TM_P + 128u * (i & 1), &sh.dp[i & 1]);
                mma_commit(&sh.empty[slot_y(i)]);
            }
            if (i > 0) {
                ok = wait(&sh.ds[(i - 1) & 1], (i - 1) / 2);
                if (ok) gather(TM_P + 128u * ((i - 1) & 1), slot_x(i - 1), TM_Q, i > 1);
            }
        }
        finish(ok);
    }

    // Warps 8 to 11.
    __device__ void work() {
        if (n == 0) return;
        if (warp == 9) {
            loads();
        } else if (key_tile && warp == 10) {
            statistics();
        } else if (warp == 8 || (key_tile && warp == 11)) {
            if (lane == 0) {
                if (!key_tile) row_products();
                else if (warp == 8) key_products_v();
                else key_products_k();
            }
            __syncwarp();
        }
    }
    // -lse log2 e and -delta of a row; a row that is none, or saw no key, gets
    // p = exp2(-inf) = 0.
    __device__ void row_statistics(int r, int tok, float &nl, float &nd) {
        nl = -INFINITY;
        nd = 0.f;
        if (r < R && tok < seq.lq) {
            const long long at = (seq.q0 + tok) * a.Hq + it.head * a.G + r % a.G;
            const float l = a.lse_in[at];
            nl = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
            nd = -a.delta[at];
        }
    }
    __device__ void statistics() {
        for (int i = 0; i < n; ++i) {
            float nl[4], nd[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int r = lane + 32 * z;
                row_statistics(r, (first + i) * TT + r / a.G, nl[z], nd[z]);
            }
            if (i >= 2 && !wait_warp(&sh.read[i & 1], i / 2 - 1)) break;
            float *dst = stats + (i & 1) * 256;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                dst[lane + 32 * z] = nl[z];
                dst[128 + lane + 32 * z] = nd[z];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.st[i & 1]);
        }
    }

    // ------------------------------------------------------- softmax, warps 0 to 7
    __device__ void key_softmax() {
        const int half = warp / 4, w = warp % 4, key = j0 + 32 * w + lane;
        const uint32_t lanes = tb + ((uint32_t)(32 * w) << 16);
        const uint32_t at_s = lanes + TM_S + 64u * half, at_p = lanes + TM_P + 64u * half;
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
                ok = wait_warp(&sh.s, i);
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
                // the rows are in the order of their tokens: those from `from`
                // on see this key
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
            ok = wait_warp(&sh.dp[0], i);
            if (!ok) break;
            tc_fence_after();
            uint32_t x[2][32], y[32];
            tmem_ld32(at_p, x[0]);
            tmem_ld32(at_p + 32, x[1]);
            tmem_ld_wait();
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
            return;
        }
        tc_fence_after();
        const long long at = ((seq.k0 + key) * a.Hk + it.head) * D;
        store_row<D>(lanes + (half ? TM_K : TM_V),
                     static_cast<__nv_bfloat16 *>(half ? a.dk : a.dv) + at, half ? a.scale : 1.f,
                     n > 0, key < seq.lk);
    }
    __device__ void row_softmax() {
        const int half = warp / 4, w = warp % 4, r = 32 * w + lane;
        const int tok = tok0 + r / a.G;
        const bool row = r < R && tok < seq.lq;
        const int limit = row ? tok + shift : -1, full = tok0 + shift;
        const long long at = (seq.q0 + tok) * a.Hq + it.head * a.G + r % a.G;
        const uint32_t lanes = tb + ((uint32_t)(32 * w) << 16);
        const uint32_t at_s = lanes + TM_S + 64u * half;
        const float c = a.scale_log2;
        float nl, nd;
        row_statistics(r, tok, nl, nd);
        bool ok = true;
        for (int i = 0; ok && i < n; ++i) {
            ok = wait_warp(&sh.s, i);
            if (!ok) break;
            tc_fence_after();
            uint32_t x[2][32];
            tmem_ld32(at_s, x[0]);
            tmem_ld32(at_s + 32, x[1]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_read);
            float p[64];
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                p[k] = __uint_as_float(x[k / 32][k % 32]);
                p[k + 1] = __uint_as_float(x[k / 32][k % 32 + 1]);
                attn::fma2(p[k], p[k + 1], c, nl);
                p[k] = attn::ex2(p[k]);
                p[k + 1] = attn::ex2(p[k + 1]);
            }
            ok = wait_warp(&sh.dp[i & 1], i / 2);
            if (!ok) break;
            tc_fence_after();
            const uint32_t at_p = lanes + TM_P + 128u * (i & 1) + 64u * half;
            tmem_ld32(at_p, x[0]);
            tmem_ld32(at_p + 32, x[1]);
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
            attn::tmem_st32(at_p, y);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.ds[i & 1]);
        }
        if (n > 0) ok = ok && wait_warp(&sh.fin, 0);
        if (!ok) {
            give_up();
            return;
        }
        tc_fence_after();
        // the halves of the row's features to the two warpgroups
        store_row<D / 2>(lanes + TM_Q + (uint32_t)(D / 2 * half),
                         static_cast<__nv_bfloat16 *>(a.dq) + at * D + D / 2 * half, a.scale,
                         n > 0, row);
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_bwd_kernel(const __grid_constant__ Args ak, const __grid_constant__ Args ar,
                   const __grid_constant__ Maps maps, int key_blocks) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const bool key_tile = (int)blockIdx.x < key_blocks;
    const Args &a = key_tile ? ak : ar;
    if (base + C::USED > raw + C::SMEM) {      // not where the array's alignment is kept
        *a.status = kDevTimeout;
        return;
    }
    Shared &sh = *reinterpret_cast<Shared *>(base + C::BARS);
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
            mbar_init(&sh.empty[i], key_tile && i >= 3 ? 2 : 1);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.dp[i], 1);
            mbar_init(&sh.ds[i], 8);
            mbar_init(&sh.st[i], 1);
            mbar_init(&sh.read[i], 8);
            mbar_init(&sh.tail[i], 1);
        }
        mbar_init(&sh.s, 1);
        mbar_init(&sh.s_read, 8);
        mbar_init(&sh.p, 8);
        mbar_init(&sh.fin, key_tile ? 2 : 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    // rows that no copy fills (the group does not divide 128) are summed over
    // by a key tile's products
    if (key_tile && maps.tokens * a.G < kTile && warp < 5)
        attn::zero_rows<C::SLABS>(base + (2 + warp) * C::TILE, maps.tokens * a.G, lane);
    if (warp == 8) tmem_alloc(&sh.tmem, C::TM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    Cta<D> cta(a, maps, sh, base, warp, lane, it, seq, key_tile);
    // Registers of a thread: 128 x 88 + 256 x 208 = 384 x 168.
    if (warp >= 8) {
        attn::fewer_registers<88>();
        cta.work();
    } else {
        attn::more_registers<208>();
        if (key_tile) cta.key_softmax();
        else cta.row_softmax();
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
