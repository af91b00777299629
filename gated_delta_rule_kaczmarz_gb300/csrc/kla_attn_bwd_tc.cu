// Causal softmax attention, backward, on the tensor cores (bf16, head sizes 64
// and 128):
//
//   p = exp2(c s - lse log2 e),  ds = p (dp - delta),  dp = go v^T,
//   dv = p^T go,  dk = scale ds^T q,  dq = scale ds k,  delta = sum go o
// (what delta is of rows with few keys: delta_of)
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
// There is a block per tile, key tiles first; a running CTA takes over blocks
// that have not started, so that an item's loads and first scores run under the
// end of the one before (its start and end cost about 6 us, a step 1.5 to 2).
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
//
// Head size 64 leaves room for a second S^T, so the next scores go ahead of
// the wait for P^T.  A barrier that another role may pass twice before a waiter
// looks comes in pairs, for odd and even steps.
//
// The barriers' phases are modelled in tests/test_attention_roles_cpu.py, by hand: a
// change of the order of waits and arrivals here is made there too.
//
// Bound: the chain of a step, through its products and the softmax, at half of
// the tensor cores' cycles (ncu: 51%).  16 + 4 heads in bf16, with the row sums:
// B 4, T 2048, d 128 224 us; B 1, T 32768 11.1 ms, 0.99 PFLOP/s of the five
// products it needs (1.38 of the seven it does); d 64, B 4, T 2048 177 us.
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

// An item: one tile of keys or of rows, and the tiles of the other side.
struct Work {
    int key_tile;
    int q0, k0, lq, lk;                  // the sequence: first rows and lengths
    int at, head;                        // first key or token of the tile; key head
    int first, n;                        // tiles of the other side: the first, how many
    int valid;                           // rows of the last of them that are the sequence's own
    int any;                             // 0: there is no more work
};

struct Shared {
    uint64_t full[5], empty[5];          // ring slots
    uint64_t fix, fix_read;              // the item's own tiles landed, and no longer read
    uint64_t s[2], dp[2];                // scores and dP ready
    uint64_t s_read, p[2], ds[2];        // scores read; P and dS in place
    uint64_t st[2], read[2];             // row statistics ready, and read
    uint64_t raw[2], zeroed;             // last tiles with a neighbour's rows landed, and cleaned
    uint64_t fin, drained;               // an item's products complete, its sums read
    uint64_t work[2], work_read[2], asked, done;
    uint4 answer;
    Work item[2];
    uint32_t tmem;
    volatile int abort;
    bool rejected;                       // the status word as the CTA's first thread read it
};

template <int D>
struct Cfg {
    static constexpr int SLABS = D / 64;
    static constexpr uint32_t TILE = SLABS * kSlab;
    // seven tiles, the row statistics of two, the barriers; what is left of a
    // block's 227 KB covers the alignment
    static constexpr size_t STATS = (size_t)TILE * 7, BARS = STATS + 2048;
    static constexpr size_t USED = BARS + 512;
    static constexpr size_t SMEM = USED + 512;
    static constexpr uint32_t TM_COLS = 512;
    static_assert(sizeof(Shared) <= 512 && SMEM <= 227 * 1024, "shared memory");
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
            uint32_t u[8];
#pragma unroll
            for (int z = 0; z < 8; ++z)
                u[z] = attn::pack2(__uint_as_float(y[2 * z]) * f, __uint_as_float(y[2 * z + 1]) * f);
            attn::store16(dst + 16 * j, u);
        }
        __syncwarp();
    }
}

template <int D>
struct Cta {
    using C = Cfg<D>;
    const Args &ak, &ar;      // key tiles and row tiles
    const Maps &maps;
    const int key_blocks;
    Shared &sh;
    unsigned char *base;      // tiles 0, 1: the item's own; 2 to 4: ring X; 5, 6: ring Y
    const uint32_t tb;
    const int warp, lane;
    const int TT, R;          // tokens and rows of a row tile
    float *stats;             // key tiles: [2][-lse log2 e, -delta][128]

    // Tensor memory of a key tile: S^T, dP^T, dV, dK; of a row tile: S, dP twice, dQ.
    static constexpr uint32_t TM_S = 0, TM_P = 128, TM_V = 256, TM_K = 256 + D, TM_Q = 384;
    static constexpr uint32_t TM_S2 = 384;      // head size 64: S^T of every second step

    // Where an item begins in the barriers' phases: steps of all items, of key
    // and of row tiles, items with steps.  Every role counts the same.
    struct Count {
        int g = 0, key = 0, row = 0, items = 0;
        __device__ void add(const Work &w) {
            g += w.n;
            (w.key_tile ? key : row) += w.n;
            items += w.n > 0;
        }
    };

    __device__ Cta(const Args &ak_, const Args &ar_, const Maps &maps_, int key_blocks_,
                   Shared &sh_, unsigned char *base_, int warp_, int lane_)
        : ak(ak_), ar(ar_), maps(maps_), key_blocks(key_blocks_), sh(sh_), base(base_),
          tb(sh_.tmem), warp(warp_), lane(lane_), TT(maps_.tokens), R(maps_.tokens * ar_.G),
          stats(reinterpret_cast<float *>(base_ + C::STATS)) {}
    __device__ void give_up() {
        sh.abort = 1;
        *ar.status = kDevTimeout;
    }
    // One lane's wait, and a warp's.
    __device__ bool wait(uint64_t *bar, int phase) {
        return mbar_wait_or_abort(bar, (uint32_t)phase & 1u, &sh.abort);
    }
    __device__ bool wait_warp(uint64_t *bar, int phase) {
        return __all_sync(0xffffffffu, wait(bar, phase));
    }
    // The m-th item for a reader: a lane, or a warp.
    __device__ bool item(int m, Work &w) {
        if (!wait(&sh.work[m & 1], m / 2)) return false;
        w = sh.item[m & 1];
        mbar_arrive(&sh.work_read[m & 1]);
        return true;
    }
    __device__ bool item_warp(int m, Work &w) {
        if (!wait_warp(&sh.work[m & 1], m / 2)) return false;
        w = sh.item[m & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.work_read[m & 1]);
        return true;
    }
    __device__ uint32_t addr(int tile) { return smem_u32(base + tile * C::TILE); }
    // K step ks of an operand in the columns of the product it came from, 32
    // columns in each half (a warpgroup's own).
    static __device__ uint32_t operand(uint32_t col, int ks) {
        return col + 64u * (ks / 4) + 8u * (ks % 4);
    }
    // Ring slots of step g of all items: Q (key tile) or K in X, dO or V in Y.
    static __device__ int slot_x(int g) { return g % 3; }
    static __device__ int slot_y(int g) { return 3 + (g & 1); }
    __device__ bool landed_y(int g) { return wait(&sh.full[slot_y(g)], g >> 1); }
    // The last tile of the other side holds rows that are a neighbour's: they
    // are zeroed before they are summed over.
    __device__ bool ragged(const Work &w) const {
        return w.n > 0 && w.valid < (w.key_tile ? R : kTile);
    }

    // ---------------------------------------------------------- items and their loads
    __device__ Work decode(int block) {
        Work w{};
        if (block < 0) return w;
        w.key_tile = block < key_blocks;
        const Args &a = w.key_tile ? ak : ar;
        Item it;
        if (!attn::item_of(a, w.key_tile ? block : block - key_blocks, !w.key_tile, it)) return w;
        const Seq seq = attn::sequence(a, it.seq);
        const int shift = seq.lk - seq.lq;
        w.q0 = (int)seq.q0; w.k0 = (int)seq.k0; w.lq = seq.lq; w.lk = seq.lk;
        w.head = it.head;
        int last;
        if (w.key_tile) {
            w.at = it.tile * kTile;
            w.first = max(0, w.at - shift) / TT;
            last = (seq.lq + TT - 1) / TT;
            w.valid = min((seq.lq - (last - 1) * TT) * a.G, R);
        } else {
            w.at = it.tile * TT;
            const int seen = min(w.at + TT, seq.lq) + shift;
            last = seen > 0 ? (seen + kTile - 1) / kTile : 0;
            w.valid = min(seq.lk - (last - 1) * kTile, kTile);
        }
        w.n = max(0, last - w.first);
        w.any = 1;
        return w;
    }
    __device__ void load(int tile, const CUtensorMap *m, uint64_t *bar, int y, int z) {
        for (int c = 0; c < C::SLABS; ++c)
            tma_load_3d(base + tile * C::TILE + c * kSlab, m, bar, c * 64, y, z);
    }
    __device__ void loads() {
        const uint32_t row_bytes = (uint32_t)R * 128u * C::SLABS, key_bytes = C::TILE;
        Count at;
        int block = blockIdx.x, raws = 0, raws_y = 0, fixed = 0, gx = 0, gy = 0;
        uint32_t raw_slots = 0;              // slots whose last load went by way of sh.raw
        bool ok = true, rows_before = false;
        for (int m = 0; ok; ++m) {
            Work w{};
            if (lane == 0) {
                w = decode(block);
                ok = m < 2 || wait(&sh.work_read[m & 1], m / 2 - 1);
                if (m == 1 && ar.lost_wait) ok = mbar_try_wait(&sh.work_read[1], 0);   // not published yet
                if (ok) {
                    sh.item[m & 1] = w;
                    mbar_arrive(&sh.work[m & 1]);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            __syncwarp();
            w = sh.item[m & 1];
            if (!ok || !w.any) break;
            // Rows that no copy of a row tile fills (the group does not divide
            // 128) were zeroed at the start.  Key tiles come before row tiles;
            // if one came after, the key rows that are in the slots by then go.
            if (w.key_tile && rows_before && R < kTile) {
                for (int i = 0; i < 3 && i < at.g; ++i)
                    ok = ok && wait_warp(&sh.empty[slot_x(at.g - 1 - i)], (at.g - 1 - i) / 3);
                for (int i = 0; i < 2 && i < at.g; ++i)
                    ok = ok && wait_warp(&sh.empty[slot_y(at.g - 1 - i)], (at.g - 1 - i) / 2);
                for (int i = 0; ok && i < 5; ++i)
                    attn::zero_rows<C::SLABS>(base + (2 + i) * C::TILE, R, lane);
            }
            rows_before = !w.key_tile;
            if (lane == 0) {
                const bool key = w.key_tile;
                const int hq = w.head * ar.G, hk = w.head;
                const CUtensorMap *mx = key ? &maps.q : &maps.k, *my = key ? &maps.go : &maps.v;
                // a last tile with a neighbour's rows goes to the cleaning warp,
                // which completes the slot; one item's at a time
                const auto next = [&](bool y, int i) {
                    const int g = at.g + i, slot = y ? slot_y(g) : slot_x(g), use = y ? g / 2 : g / 3;
                    ok = use == 0 || wait(&sh.empty[slot], use - 1);
                    uint64_t *bar = &sh.full[slot];
                    const bool raw = i == w.n - 1 && ragged(w) && (key || !y);
                    if (ok && raw) {
                        if (!y) {
                            ok = raws == 0 || wait(&sh.zeroed, raws - 1);
                            raws += ok;
                        } else {
                            ++raws_y;
                        }
                        bar = &sh.raw[y];
                    }
                    if (!ok) return;
                    raw_slots = (raw_slots & ~(1u << slot)) | ((raw ? 1u : 0u) << slot);
                    mbar_expect_tx(bar, key ? row_bytes : key_bytes);
                    load(2 + slot, y ? my : mx, bar, key ? hq : hk,
                         key ? w.q0 + (w.first + i) * TT : w.k0 + i * kTile);
                    ++(y ? gy : gx);
                };
                // In the order of their first use; the own tiles after the first
                // of each ring, because the item before reads its own until its
                // last scores.  The next block is asked for a few tiles before
                // the end: earlier, a CTA would hold what another could start.
                bool asked = false;
                for (int i = 0; ok && i <= w.n; ++i) {
                    if (i == max(0, w.n - 4)) {
                        mbar_expect_tx(&sh.asked, 16);
                        attn::ask_block(&sh.answer, &sh.asked);
                        asked = true;
                    }
                    if (i == w.n) break;
                    if (i == 0) next(false, 0);
                    if (ok) next(true, i);
                    if (ok && i == 0) {
                        ok = fixed == 0 || wait(&sh.fix_read, fixed - 1);
                        if (!ok) break;
                        ++fixed;
                        mbar_expect_tx(&sh.fix, 2 * (key ? key_bytes : row_bytes));
                        load(0, key ? &maps.k : &maps.q, &sh.fix, key ? hk : hq,
                             (key ? w.k0 : w.q0) + w.at);
                        load(1, key ? &maps.v : &maps.go, &sh.fix, key ? hk : hq,
                             (key ? w.k0 : w.q0) + w.at);
                    }
                    if (ok && i + 1 < w.n) next(false, i + 1);
                }
                if (asked) {
                    ok = mbar_wait(&sh.asked, (uint32_t)(m & 1)) && ok;
                    block = attn::answered_block(&sh.answer);
                    fence_async_smem();        // read before the next answer is written
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            at.add(w);
        }
        if (!ok && lane == 0) {    // given up: the copies in flight land before the CTA leaves
            give_up();
            for (int i = max(0, gx - 3); i < gx; ++i)
                if (!(raw_slots >> slot_x(i) & 1u))
                    (void)mbar_wait(&sh.full[slot_x(i)], (uint32_t)((i / 3) & 1));
            for (int i = max(0, gy - 2); i < gy; ++i)
                if (!(raw_slots >> slot_y(i) & 1u))
                    (void)mbar_wait(&sh.full[slot_y(i)], (uint32_t)((i / 2) & 1));
            if (raws > 0) (void)mbar_wait(&sh.raw[0], (uint32_t)((raws - 1) & 1));
            if (raws_y > 0) (void)mbar_wait(&sh.raw[1], (uint32_t)((raws_y - 1) & 1));
            if (fixed > 0) (void)mbar_wait(&sh.fix, (uint32_t)((fixed - 1) & 1));
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
    // The sums of the item before are read, and with them all it had in tensor
    // memory is free.
    __device__ bool drained(const Count &at) {
        return at.items == 0 || wait(&sh.drained, at.items - 1);
    }
    // Ring X walked without divisions: a step's instructions on the issuing
    // lanes are part of its latency.
    struct RingX {
        int slot, use;
        __device__ RingX(int g) : slot(g % 3), use(g / 3) {}
        __device__ void next() {
            if (++slot == 3) {
                slot = 0;
                ++use;
            }
        }
    };
    // Where a key tile has S^T of its step i (and P^T after it): at head size
    // 64 tensor memory has room for two.
    static __device__ uint32_t key_scores(int i) { return D == 64 && (i & 1) ? TM_S2 : TM_S; }
    // S^T and dV of a key tile.  With one S^T the next takes its columns after
    // dV; with two it goes ahead of the wait for P^T.
    __device__ bool key_products_v(const Work &w, const Count &at) {
        const int n = w.n;
        RingX x(at.g);
        const auto scores = [&](int i) {
            if (!wait(&sh.full[x.slot], x.use)) return false;
            product(0, x.slot, key_scores(i), &sh.s[(at.g + i) & 1]);
            if (i + 1 == n) mma_commit(&sh.fix_read);
            x.next();
            return true;
        };
        if (!wait(&sh.fix, at.items) || !scores(0) || !drained(at)) return false;
        for (int i = 0; i < n; ++i) {
            const int g = at.g + i;
            if (D == 64 && i + 1 < n && !scores(i + 1)) return false;
            // one barrier for odd and one for even steps: with two S^T the next
            // step's P can be in place before this wait is looked at
            const int gk = at.key + i;
            if (!landed_y(g) || !wait(&sh.p[gk & 1], gk >> 1)) return false;
            gather(key_scores(i), slot_y(g), TM_V, i > 0);
            if (D != 64 && i + 1 < n && !scores(i + 1)) return false;
        }
        mma_commit(&sh.fin);
        return true;
    }
    // dP^T and dK of a key tile.
    __device__ bool key_products_k(const Work &w, const Count &at) {
        const int n = w.n;
        RingX x(at.g);
        if (!wait(&sh.fix, at.items) || !landed_y(at.g) || !drained(at)) return false;
        product(1, slot_y(at.g), TM_P, &sh.dp[at.g & 1]);
        mma_commit(&sh.empty[slot_y(at.g)]);
        if (n == 1) mma_commit(&sh.fix_read);
        for (int i = 0;; ++i) {
            const int g = at.g + i;
            if (!wait(&sh.ds[g & 1], g >> 1)) return false;
            gather(TM_P, x.slot, TM_K, i > 0);
            if (i + 1 == n) break;
            x.next();
            if (!landed_y(g + 1)) return false;
            product(1, slot_y(g + 1), TM_P, &sh.dp[(g + 1) & 1]);
            mma_commit(&sh.empty[slot_y(g + 1)]);
            if (i + 2 == n) mma_commit(&sh.fix_read);
        }
        mma_commit(&sh.fin);
        return true;
    }
    // All of a row tile.  What both warps release at a key tile is released
    // twice here.
    __device__ bool row_products(const Work &w, const Count &at) {
        const int n = w.n;
        RingX x(at.g), before(at.g);
        if (!wait(&sh.fix, at.items)) return false;
        for (int i = 0; i <= n; ++i) {
            const int g = at.g + i;
            if (i < n) {
                if (!wait(&sh.full[x.slot], x.use)) return false;
                if (i > 0 && !wait(&sh.s_read, at.row + i - 1)) return false;
                product(0, x.slot, TM_S, &sh.s[g & 1]);
                x.next();
                if (!landed_y(g) || (i == 0 && !drained(at))) return false;
                product(1, slot_y(g), TM_P + 128u * (g & 1), &sh.dp[g & 1]);
                mma_commit(&sh.empty[slot_y(g)]);
                mma_commit(&sh.empty[slot_y(g)]);
                if (i + 1 == n) {
                    mma_commit(&sh.fix_read);
                    mma_commit(&sh.fix_read);
                }
            }
            if (i > 0) {
                if (!wait(&sh.ds[(g - 1) & 1], (g - 1) >> 1)) return false;
                gather(TM_P + 128u * ((g - 1) & 1), before.slot, TM_Q, i > 1);
                before.next();
            }
        }
        mma_commit(&sh.fin);
        return wait(&sh.s_read, at.row + n - 1);
    }
    // One lane of warp 8 (second = false) and of warp 11.
    __device__ void products(bool second) {
        Count at;
        bool ok = true;
        for (int m = 0; ok; ++m) {
            Work w;
            ok = item(m, w);
            if (!ok || !w.any) break;
            if (w.n > 0) {
                if (w.key_tile) {
                    ok = second ? key_products_k(w, at) : key_products_v(w, at);
                } else if (!second) {
                    ok = row_products(w, at);
                } else {
                    // not needed; it stays with the item, so that the barriers
                    // that it waits on next are in the phase before
                    // (and not ahead: its arrival would count for the item before)
                    ok = at.items == 0 || wait(&sh.fin, at.items - 1);
                    if (ok) mbar_arrive(&sh.fin);
                    ok = ok && wait(&sh.fin, at.items);
                }
            }
            at.add(w);
        }
        if (!ok) give_up();
    }

    // ------------------------------------------------ row statistics, cleaning
    // lse and delta of a row as they are, and what the exponentials and dS take:
    // -lse log2 e and -delta; a row that is none, or saw no key, gets p =
    // exp2(-inf) = 0.
    __device__ float2 read_statistics(const Work &w, int r, int tok) {
        if (r >= R || tok >= w.lq) return make_float2(-INFINITY, 0.f);
        const long long at = (long long)(w.q0 + tok) * ar.Hq + w.head * ar.G + r % ar.G;
        return make_float2(ar.lse_in[at], attn::delta_of(ar, at, tok + w.lk - w.lq + 1));
    }
    static __device__ float2 row_statistics(float2 x) {
        return make_float2(x.x == -INFINITY ? -INFINITY : -x.x * 1.4426950408889634f, -x.y);
    }
    __device__ void statistics() {
        Count at;
        int raws[2] = {0, 0};
        bool ok = true;
        for (int m = 0; ok; ++m) {
            Work w;
            ok = item_warp(m, w);
            if (!ok || !w.any) break;
            if (w.key_tile && w.n > 0) {
                // read two tiles ahead: a read takes about as long as a step
                float2 x[2][4];
                int tok[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) tok[z] = (lane + 32 * z) / ar.G;
                const auto fetch = [&](int i, float2 (&x)[4]) {
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        x[z] = read_statistics(w, lane + 32 * z, (w.first + i) * TT + tok[z]);
                };
                const auto store = [&](int i, const float2 (&x)[4]) {
                    const int g = at.key + i;
                    if (g >= 2 && !wait_warp(&sh.read[g & 1], (g >> 1) - 1)) return false;
                    float *dst = stats + (g & 1) * 256;
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float2 v = row_statistics(x[z]);
                        dst[lane + 32 * z] = v.x;
                        dst[128 + lane + 32 * z] = v.y;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.st[g & 1]);
                    return true;
                };
                fetch(0, x[0]);
                if (w.n > 1) fetch(1, x[1]);
                for (int i = 0; ok && i < w.n; i += 2) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        if (!ok || i + z >= w.n) break;
                        ok = store(i + z, x[z]);
                        if (i + z + 2 < w.n) fetch(i + z + 2, x[z]);
                    }
                }
            }
            if (ok && ragged(w)) {
                const int g = at.g + w.n - 1;
                for (int y = 0; ok && y < (w.key_tile ? 2 : 1); ++y) {
                    const int slot = y ? slot_y(g) : slot_x(g);
                    ok = wait_warp(&sh.raw[y], raws[y]++);
                    if (!ok) break;
                    attn::zero_rows<C::SLABS>(base + (2 + slot) * C::TILE, w.valid, lane);
                    if (lane == 0) mbar_arrive(&sh.full[slot]);
                }
                if (ok && lane == 0) mbar_arrive(&sh.zeroed);
            }
            at.add(w);
        }
        if (!ok) give_up();
    }

    // ------------------------------------------------------- softmax, warps 0 to 7
    __device__ bool key_softmax(const Work &w, const Count &at) {
        const int half = warp / 4, key = w.at + 32 * (warp % 4) + lane;
        const int shift = w.lk - w.lq;
        const uint32_t lanes = tb + ((uint32_t)(32 * (warp % 4)) << 16);
        const uint32_t at_p = lanes + TM_P + 64u * half;
        const float c = ak.scale_log2;
        for (int i = 0; i < w.n; ++i) {
            const int g = at.g + i, gk = at.key + i;
            const uint32_t at_s = lanes + key_scores(i) + 64u * half;
            // the rows' statistics into registers ahead of the waits: the
            // products hold shared memory busy, and a read takes its time
            const float4 *st = reinterpret_cast<const float4 *>(stats + (gk & 1) * 256 + 64 * half);
            if (!wait_warp(&sh.st[gk & 1], gk >> 1)) return false;
            float p[64];
            {
                float4 nl[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) nl[k] = st[k];
                if (!wait_warp(&sh.s[g & 1], g >> 1)) return false;
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
            const int t0 = (w.first + i) * TT;
            if (t0 + shift < w.at + kTile - 1) {
                // the rows are in the order of their tokens: those from `from`
                // on see this key
                const int from = min(max(key - shift - t0, 0), TT) * ak.G - 64 * half;
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
            if (lane == 0) mbar_arrive(&sh.p[gk & 1]);
            float4 nd[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) nd[k] = st[32 + k];
            if (!wait_warp(&sh.dp[g & 1], g >> 1)) return false;
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
                mbar_arrive(&sh.ds[g & 1]);
                mbar_arrive(&sh.read[gk & 1]);
            }
        }
        if (w.n > 0 && !wait_warp(&sh.fin, at.items)) return false;
        tc_fence_after();
        const long long row = ((long long)(w.k0 + key) * ak.Hk + w.head) * D;
        store_row<D>(lanes + (half ? TM_K : TM_V),
                     static_cast<__nv_bfloat16 *>(half ? ak.dk : ak.dv) + row,
                     half ? ak.scale : 1.f, w.n > 0, key < w.lk);
        return true;
    }
    __device__ bool row_softmax(const Work &w, const Count &at) {
        const int half = warp / 4, r = 32 * (warp % 4) + lane;
        const int tok = w.at + r / ar.G, shift = w.lk - w.lq;
        const bool row = r < R && tok < w.lq;
        const int limit = row ? tok + shift : -1, full = w.at + shift;
        const uint32_t lanes = tb + ((uint32_t)(32 * (warp % 4)) << 16);
        const uint32_t at_s = lanes + TM_S + 64u * half;
        const float c = ar.scale_log2;
        const float2 stat = row_statistics(read_statistics(w, r, tok));
        const float nl = stat.x, nd = stat.y;
        for (int i = 0; i < w.n; ++i) {
            const int g = at.g + i;
            if (!wait_warp(&sh.s[g & 1], g >> 1)) return false;
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
            if (!wait_warp(&sh.dp[g & 1], g >> 1)) return false;
            tc_fence_after();
            const uint32_t at_p = lanes + TM_P + 128u * (g & 1) + 64u * half;
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
            if (lane == 0) mbar_arrive(&sh.ds[g & 1]);
        }
        if (w.n > 0 && !wait_warp(&sh.fin, at.items)) return false;
        tc_fence_after();
        // the halves of the row's features to the two warpgroups
        const long long out = ((long long)(w.q0 + tok) * ar.Hq + w.head * ar.G + r % ar.G) * D;
        store_row<D / 2>(lanes + TM_Q + (uint32_t)(D / 2 * half),
                         static_cast<__nv_bfloat16 *>(ar.dq) + out + D / 2 * half, ar.scale,
                         w.n > 0, row);
        return true;
    }
    __device__ void softmax() {
        Count at;
        bool ok = true;
        for (int m = 0; ok; ++m) {
            Work w;
            ok = item_warp(m, w);
            if (!ok || !w.any) break;
            ok = w.key_tile ? key_softmax(w, at) : row_softmax(w, at);
            if (!ok) break;
            if (w.n > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.drained);
            }
            at.add(w);
        }
        if (!ok) give_up();
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
    if (base + C::USED > raw + C::SMEM) {      // not where the array's alignment is kept
        *ar.status = kDevTimeout;
        return;
    }
    Shared &sh = *reinterpret_cast<Shared *>(base + C::BARS);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], i >= 3 ? 2 : 1);     // dO is read by both product warps
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s[i], 1);
            mbar_init(&sh.dp[i], 1);
            mbar_init(&sh.p[i], 8);
            mbar_init(&sh.ds[i], 8);
            mbar_init(&sh.st[i], 1);
            mbar_init(&sh.read[i], 8);
            mbar_init(&sh.raw[i], 1);
            mbar_init(&sh.work[i], 1);
            mbar_init(&sh.work_read[i], 11);             // products (2), statistics, softmax (8)
        }
        mbar_init(&sh.fix, 1);
        mbar_init(&sh.fix_read, 2);
        mbar_init(&sh.s_read, 8);
        mbar_init(&sh.zeroed, 1);
        mbar_init(&sh.fin, 2);
        mbar_init(&sh.drained, 8);
        mbar_init(&sh.asked, 1);
        mbar_init(&sh.done, 2);
        sh.abort = 0;
        sh.rejected = attn::rejected(ar);
        fence_mbar_init();
    }
    // rows that no copy fills (the group does not divide 128) are summed over
    // by a key tile's products
    if (maps.tokens * ar.G < kTile && warp < 5)
        attn::zero_rows<C::SLABS>(base + (2 + warp) * C::TILE, maps.tokens * ar.G, lane);
    if (warp == 8) tmem_alloc(&sh.tmem, C::TM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh.rejected) {
        if (warp == 8) {
            tmem_relinquish();
            tmem_dealloc(sh.tmem, C::TM_COLS);
        }
        return;
    }
    Cta<D> cta(ak, ar, maps, key_blocks, sh, base, warp, lane);
    // Registers of a thread: 128 x 88 + 256 x 208 = 384 x 168.
    if (warp >= 8) {
        attn::fewer_registers<88>();
        if (warp == 9) {
            cta.loads();
        } else if (warp == 10) {
            cta.statistics();
        } else {
            if (lane == 0) {
                cta.products(warp == 11);
                // every product issued has completed before the tensor memory is released
                mma_commit(&sh.done);
                (void)mbar_wait(&sh.done, 0u);
            }
            __syncwarp();
        }
    } else {
        attn::more_registers<208>();
        cta.softmax();
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
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(attn_tc_bwd_kernel<D>), Cfg<D>::SMEM);
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
