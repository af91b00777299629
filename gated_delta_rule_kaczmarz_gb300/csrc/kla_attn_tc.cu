// Causal softmax attention, forward, on the tensor cores (bf16, head sizes 64
// and 128).
//
//   s = q k^T,  p = exp2(c (s - m)),  o = (sum p v) / l,  l = sum p,
//   lse = (c m + log2 l) ln 2,  c = scale log2 e
//
// An item is two tiles of up to 128 packed rows (token x group head) of one key
// head, walked over the keys in tiles of 128.  There is a block per item, the
// longest first; a running CTA takes over blocks that have not started, so
// that one item's start runs under the end of the one before.  Scores,
// probabilities and outputs stay in tensor memory: S_t = Q_t K^T (128 columns
// each), P_t as bf16 over S_t's columns, from where it is the A operand of O_t
// += P_t V.  A warp loads (TMA, a ring of slots that holds K and V tiles in the
// order of their use), each tile has a warp that issues its products and four
// softmax warps with one row per thread, and one warp zeroes a neighbour's rows
// in a last V tile.  The two tiles alternate: while one's softmax runs,
// the tensor cores work on the other's products.
//
// The running maximum m is raised only where a row's grew by more than 8 (in
// log2 units): p then stays below 2^8, which costs no accuracy in fp32 sums
// and bf16 mantissas, and the rescaling of O in tensor memory, a round trip of
// its whole row, happens in the first tiles only.  p is rounded to bf16 as an
// operand; the sum l is of the unrounded values.
//
// The barriers' phases are modelled in tests/test_attention_roles_cpu.py, by hand: a
// change of the order of waits and arrivals here is made there too.
//
// Bound: the tensor cores over a prompt (4 d flops a pair and head), HBM for
// single tokens over a cache (the key tiles pass once for all heads of a
// group).  16 + 4 heads of 128 in bf16: B 1, T 32768 2.73 ms, 1.61 PFLOP/s, by itself
// (2.89 ms, 1.52, at the clock of a busy GPU); B 4, T 2048 66 us, 1.04 (three to
// four items a CTA, and each costs about 3 us at its ends); single tokens of B 16
// over 32768 keys 169 us, 6.4 TB/s.  Head size 64, B 1, T 8192 186 us, 0.74
// PFLOP/s: its P V has 64 columns, which take the tensor cores as long as 128, and
// the softmax does not shrink with the head.
// The exponentials are not the bound: a part of them as polynomials on the
// multiply-add units made every size slower (T 32768: an eighth 5%).
#include "kla_attn_tc.cuh"

namespace kla {
namespace {

using namespace tc;
using attn::Args;
using attn::Item;
using attn::kSlab;
using attn::kTile;
using attn::Seq;

constexpr int kThreads = 384;            // 8 softmax warps, 2 of products, loads, zeroing
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kGrow = 8.f;             // see above

template <int D>
struct Cfg {
    static constexpr int SLABS = D / 64;
    static constexpr uint32_t TILE = SLABS * kSlab;
    static constexpr int SLOTS = D == 128 ? 4 : 6;
    static constexpr size_t SMEM = (size_t)TILE * (2 + SLOTS) + 1024;
    static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
};

// An item's rows, its key tiles and where they lie.
struct Work {
    int q0, k0, lq, lk;                  // the sequence: first rows and lengths
    int tok0, head, split;               // first token of the two row tiles, key head
    int b0, b1, e[2];                    // key tiles b0 .. b1; row tile t: b0 .. e[t]
    int any;                             // 0: there is no more work
};

struct Shared {
    uint64_t full[8], empty[8];          // ring slots
    uint64_t q[2], q_read[2];            // Q tiles landed, and no longer read
    uint64_t s[2], p[2], o[2];           // scores ready, probabilities ready, product done
    uint64_t work[2], work_read[2];      // items published, and read
    uint64_t turn[2];
    uint64_t raw, zeroed;                // a ragged V tile landed, and cleaned
    uint64_t asked, fin;
    uint4 answer;
    Work item[2];
    uint32_t tmem;
    volatile int abort;
    bool rejected;                       // the status word as the CTA's first thread read it
};

// Maps of a launch and its row tiling.
struct Maps {
    CUtensorMap q, k, v;
    int tokens;                          // of a tile
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_fwd_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps) {
    using C = Cfg<D>;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *sQ = base, *sKV = base + 2 * C::TILE;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    attn::clear_status(a);
    const int TT = maps.tokens, R = TT * a.G;

    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 2);          // both tiles' products
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.q[t], 1);
            mbar_init(&sh.q_read[t], 1);
            mbar_init(&sh.s[t], 1);
            mbar_init(&sh.p[t], 4);
            mbar_init(&sh.o[t], 1);
            mbar_init(&sh.work[t], 1);
            mbar_init(&sh.work_read[t], 11);     // products (2), zeroing and softmax (8)
            mbar_init(&sh.turn[t], 1);
        }
        mbar_init(&sh.raw, 1);
        mbar_init(&sh.zeroed, 1);
        mbar_init(&sh.asked, 1);
        mbar_init(&sh.fin, 2);
        sh.abort = 0;
        sh.rejected = attn::rejected(a);
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&sh.tmem, C::TM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = sh.tmem;
    if (sh.rejected) {
        if (warp == 8) {
            tmem_relinquish();
            tmem_dealloc(tb, C::TM_COLS);
        }
        return;
    }
    const auto give_up = [&] {
        sh.abort = 1;
        *a.status = kDevTimeout;
    };
    const auto wait = [&](uint64_t *bar, int phase) {
        return mbar_wait_or_abort(bar, (uint32_t)(phase & 1), &sh.abort);
    };
    const auto wait_warp = [&](uint64_t *bar, int phase) {
        return __all_sync(0xffffffffu, wait(bar, phase));
    };

    // Registers of a thread: 128 x 88 + 256 x 208 = 384 x 168.
    if (warp >= 8) {
        attn::fewer_registers<88>();
        if (warp == 9) {
            // ------------------------------------------- items and their loads
            int j = 0, used[2] = {0, 0}, raws = 0, block = blockIdx.x;
            uint32_t raw_slots = 0;     // slots whose last load went by way of sh.raw
            bool ok = true;
            for (int m = 0; ok; ++m) {
                // publish item m (the consumers may be an item behind)
                if (lane == 0) {
                    Work w{};
                    Item it;
                    if (block >= 0 && attn::item_of(a, block, true, it)) {
                        const Seq seq = attn::sequence(a, it.seq);
                        const int shift = seq.lk - seq.lq;
                        w.q0 = (int)seq.q0; w.k0 = (int)seq.k0; w.lq = seq.lq; w.lk = seq.lk;
                        w.tok0 = it.tile * 2 * TT; w.head = it.head; w.split = it.split;
                        int n[2];      // key tiles of a row tile; none without tokens
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int first = w.tok0 + t * TT, last = min(first + TT, seq.lq);
                            const int seen = last > first ? last + shift : 0;
                            n[t] = seen > 0 ? (seen + kTile - 1) / kTile : 0;
                        }
                        attn::split_range(max(n[0], n[1]), a.splits, it.split, w.b0, w.b1);
                        w.e[0] = min(n[0], w.b1);
                        w.e[1] = min(n[1], w.b1);
                        w.any = 1;
                    }
                    ok = m < 2 || wait(&sh.work_read[m & 1], m / 2 - 1);
                    if (m == 1 && a.lost_wait) ok = mbar_try_wait(&sh.work_read[1], 0);   // not published yet
                    if (ok) {
                        sh.item[m & 1] = w;
                        mbar_arrive(&sh.work[m & 1]);
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                __syncwarp();
                const Work w = sh.item[m & 1];
                if (!ok || !w.any) break;
                const int nb = w.b1 - w.b0;
                bool asked = false;
                if (lane == 0) {
                    const uint32_t box = (uint32_t)R * 128u;
                    // The next block is asked for four key tiles before the end:
                    // the answer and the item's rows are there when the last
                    // load is under way.  (Earlier, a CTA would hold what
                    // another could start.)  Q's tiles are free only after the
                    // item before has its last scores, so the first key and
                    // value tile go ahead of them.
                    const int ask_at = max(0, 2 * nb - 8);
                    for (int i = 0; ok && i <= 2 * nb; ++i) {
                        if (i == ask_at) {
                            mbar_expect_tx(&sh.asked, 16);
                            attn::ask_block(&sh.answer, &sh.asked);
                            asked = true;
                        }
                        if (i == 2) {
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                if (w.e[t] <= w.b0) continue;
                                ok = ok && (used[t] == 0 || wait(&sh.q_read[t], used[t] - 1));
                                if (!ok) break;
                                ++used[t];
                                mbar_expect_tx(&sh.q[t], box * C::SLABS);
                                for (int c = 0; c < C::SLABS; ++c)
                                    tma_load_3d(sQ + t * C::TILE + c * kSlab, &maps.q, &sh.q[t],
                                                c * 64, w.head * a.G, w.q0 + w.tok0 + t * TT);
                            }
                        }
                        if (!ok || i == 2 * nb) break;
                        const int slot = j % C::SLOTS, use = j / C::SLOTS;
                        ok = use == 0 || wait(&sh.empty[slot], use - 1);
                        if (!ok) break;
                        // a last V tile that holds a neighbour's rows goes to
                        // the zeroing warp, which completes the slot; one at a time
                        uint64_t *bar = &sh.full[slot];
                        if (i == 2 * nb - 1 && w.b1 * kTile > w.lk) {
                            bar = &sh.raw;
                            ok = raws == 0 || wait(&sh.zeroed, raws - 1);
                            if (!ok) break;
                            ++raws;
                        }
                        raw_slots = (raw_slots & ~(1u << slot)) | (bar == &sh.raw ? 1u << slot : 0u);
                        ++j;
                        mbar_expect_tx(bar, C::TILE);
                        const int row = w.k0 + (w.b0 + i / 2) * kTile;
                        for (int c = 0; c < C::SLABS; ++c)
                            tma_load_3d(sKV + slot * C::TILE + c * kSlab, i % 2 ? &maps.v : &maps.k,
                                        bar, c * 64, w.head, row);
                    }
                    if (asked) {
                        ok = mbar_wait(&sh.asked, (uint32_t)(m & 1)) && ok;
                        block = attn::answered_block(&sh.answer);
                        fence_async_smem();        // read before the next answer is written
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!ok && lane == 0) {    // given up: the copies in flight land before the CTA leaves
                give_up();
                for (int i = max(0, j - C::SLOTS); i < j; ++i)
                    if (!(raw_slots >> (i % C::SLOTS) & 1u))
                        (void)mbar_wait(&sh.full[i % C::SLOTS], (uint32_t)((i / C::SLOTS) & 1));
                if (raws > 0) (void)mbar_wait(&sh.raw, (uint32_t)((raws - 1) & 1));
                for (int t = 0; t < 2; ++t)
                    if (used[t] > 0) (void)mbar_wait(&sh.q[t], (uint32_t)((used[t] - 1) & 1));
            }
        } else if (warp == 11) {
            // -------------- rows of a last V tile that are a neighbour's: zeroed
            int j = 0, raws = 0;
            bool ok = true;
            for (int m = 0; ok; ++m) {
                ok = wait_warp(&sh.work[m & 1], m / 2);
                if (!ok) break;
                const Work w = sh.item[m & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.work_read[m & 1]);
                if (!w.any) break;
                j += 2 * (w.b1 - w.b0);
                const int valid = w.lk - (w.b1 - 1) * kTile, slot = (j - 1) % C::SLOTS;
                if (w.b1 == w.b0 || valid >= kTile) continue;
                ok = wait_warp(&sh.raw, raws++);
                if (!ok) break;
                attn::zero_rows<C::SLABS>(sKV + slot * C::TILE, valid, lane);
                if (lane == 0) {
                    mbar_arrive(&sh.full[slot]);
                    mbar_arrive(&sh.zeroed);
                }
            }
            if (!ok) give_up();
        } else if (warp == 8 || warp == 10) {
            // ---------------------------------------------------------- products
            // A warp per row tile, one lane of which waits and issues: a wait
            // takes about 100 cycles even where there is nothing to wait for,
            // and the queue of issued products is shorter than the six of a
            // step, so one tile's waits have to run under the other's issue.
            // The tiles' batches (O += P V, then the next scores) take turns;
            // without them both tiles' products run at the same time and
            // their softmax too, with the tensor cores idle.
            constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t id_o = idesc_bf16_f32(128, D, false, true);
            const int t = warp == 8 ? 0 : 1;
            const uint32_t aQ = smem_u32(sQ) + t * C::TILE, aKV = smem_u32(sKV);
            const uint32_t tS = tb + C::TM_S + 128u * t, tO = tb + C::TM_O + (uint32_t)(D * t);
            const auto landed = [&](int j) { return wait(&sh.full[j % C::SLOTS], j / C::SLOTS); };
            const auto scores = [&](int j, int ks0, int ks1) {
#pragma unroll
                for (int ks = ks0; ks < ks1; ++ks)
                    mma_bf16(tS, attn::kdesc(aQ, ks),
                             attn::kdesc(aKV + (j % C::SLOTS) * C::TILE, ks), id_s, ks > 0);
            };
            if (lane == 0) {
                int j = 0, used = 0, step = 0, turns = 0;
                bool ok = true;
                for (int m = 0; ok; ++m) {
                    ok = wait(&sh.work[m & 1], m / 2);
                    if (!ok) break;
                    const Work w = sh.item[m & 1];
                    mbar_arrive(&sh.work_read[m & 1]);
                    if (!w.any) break;
                    const int nb = w.b1 - w.b0;
                    if (nb == 0) continue;
                    const int mine = max(0, w.e[t] - w.b0), other = max(0, w.e[1 - t] - w.b0);
                    ok = landed(j);
                    if (ok && mine > 0) {
                        ok = wait(&sh.q[t], used++);
                        if (!ok) break;
                        scores(j, 0, D / 16);
                        mma_commit(&sh.s[t]);
                        if (mine == 1) mma_commit(&sh.q_read[t]);
                        mma_commit(&sh.empty[j % C::SLOTS]);
                    } else if (ok) {
                        mbar_arrive(&sh.empty[j % C::SLOTS]);
                    }
                    for (int n = 0; ok && n < nb; ++n) {
                        const int jv = j + 2 * n + 1, jk = j + 2 * n + 2, sv = jv % C::SLOTS;
                        ok = landed(jv) && (n + 1 == nb || landed(jk));
                        if (!ok) break;
                        if (n >= mine) {       // the other tile's keys
                            mbar_arrive(&sh.empty[sv]);
                            if (n + 1 < nb) mbar_arrive(&sh.empty[jk % C::SLOTS]);
                            continue;
                        }
                        // strictly in turn over all items, where both tiles have a batch
                        const bool both = n < other;
                        if (both && (t == 1 || turns > 0))
                            ok = ok && wait(&sh.turn[t], t == 1 ? turns : turns - 1);
                        turns += both;
                        ok = ok && wait(&sh.p[t], step);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_bf16_ts(tO, tS + 8u * ks, attn::mdesc(aKV + sv * C::TILE, ks),
                                        id_o, n > 0 || ks > 0);
                        ++step;
                        mma_commit(&sh.o[t]);
                        mma_commit(&sh.empty[sv]);
                        // the turn passes on while the queue still holds products
                        if (n + 1 < mine) {
                            scores(jk, 0, D / 32);
                            if (both) mbar_arrive(&sh.turn[1 - t]);
                            scores(jk, D / 32, D / 16);
                            mma_commit(&sh.s[t]);
                            if (n + 2 == mine) mma_commit(&sh.q_read[t]);
                            mma_commit(&sh.empty[jk % C::SLOTS]);
                        } else {
                            if (both) mbar_arrive(&sh.turn[1 - t]);
                            if (n + 1 < nb) mbar_arrive(&sh.empty[jk % C::SLOTS]);
                        }
                    }
                    j += 2 * nb;
                }
                if (!ok) give_up();
                // every product issued has completed before the tensor memory is released
                mma_commit(&sh.fin);
                (void)mbar_wait(&sh.fin, 0u);
            }
            __syncwarp();
        }
    } else {
        // ----------------------------------------------------------- softmax
        attn::more_registers<208>();
        const int t = warp / 4, w = warp % 4, r = 32 * w + lane;
        const uint32_t lanes = (uint32_t)(32 * w) << 16;
        const uint32_t tS = tb + C::TM_S + 128u * t + lanes;
        const uint32_t tO = tb + C::TM_O + (uint32_t)(D * t) + lanes;
        const int tok_r = t * TT + r / a.G, head_r = r % a.G;
        const float c = a.scale_log2;
        int step = 0;                                         // of this row tile, over all items
        bool ok = true;
        for (int it = 0; ok; ++it) {
            ok = wait_warp(&sh.work[it & 1], it / 2);
            if (!ok) break;
            const Work k = sh.item[it & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.work_read[it & 1]);
            if (!k.any) break;
            const int shift = k.lk - k.lq, e = k.e[t];
            const int tok = k.tok0 + tok_r, head = k.head * a.G + head_r;
            const bool row = r < R && tok < k.lq;
            const int limit = row ? tok + shift : -1;         // last key of the row
            const int full = k.tok0 + t * TT + shift;         // last key that every row sees
            const bool work = __any_sync(0xffffffffu, row);   // a warp without rows only arrives
            float m = -INFINITY, l = 0.f, mc = 0.f;           // mc = c m (0 while m is -inf)
            for (int n = k.b0; n < e; ++n, ++step) {
                ok = wait_warp(&sh.s[t], step);
                if (!ok) break;
                tc_fence_after();
                if (work) {
                    uint32_t x[4][32];
#pragma unroll
                    for (int j = 0; j < 4; ++j) tmem_ld32(tS + 32u * j, x[j]);
                    tmem_ld_wait();
                    if (n * kTile + kTile - 1 > full) {
                        const int rel = limit - n * kTile;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * j + i > rel) x[j][i] = 0xff800000u;      // -infinity
                    }
                    float mx[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) mx[j] = __uint_as_float(x[0][j]);
#pragma unroll
                    for (int i = 8; i < 128; i += 16)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int u = i + j, v = i + 8 + j;
                            const float f = __uint_as_float(x[u / 32][u % 32]);
                            mx[j] = v < 128
                                        ? attn::max3(mx[j], f, __uint_as_float(x[v / 32 % 4][v % 32]))
                                        : fmaxf(mx[j], f);
                        }
                    const float top = fmaxf(attn::max3(mx[0], mx[1], mx[2]),
                                            attn::max3(attn::max3(mx[3], mx[4], mx[5]), mx[6], mx[7]));
                    const bool grow = row && (top - m) * c > kGrow;
                    if (n == k.b0) {
                        m = top;
                        mc = top == -INFINITY ? 0.f : top * c;
                    } else if (__any_sync(0xffffffffu, grow)) {
                        // O holds the products up to the last tile: they have to be complete
                        ok = wait_warp(&sh.o[t], step - 1);
                        if (!ok) break;
                        tc_fence_after();
                        float f = 1.f;
                        if (grow) {
                            f = m == -INFINITY ? 0.f : attn::ex2((m - top) * c);
                            m = top;
                            mc = top * c;
                        }
                        __syncwarp();
                        l *= f;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            uint32_t y[16];
                            tmem_ld16(tO + 16u * j, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                            tmem_st16(tO + 16u * j, y);
                        }
                    }
                    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t y[32];
#pragma unroll
                        for (int i = 0; i < 64; i += 4) {
                            float p[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                p[z] = __uint_as_float(x[2 * h + (i + z) / 32][(i + z) % 32]);
                            attn::fma2(p[0], p[1], c, -mc);
                            attn::fma2(p[2], p[3], c, -mc);
#pragma unroll
                            for (int z = 0; z < 4; ++z) p[z] = attn::ex2(p[z]);
                            attn::add2(s0, s1, p[0], p[1]);
                            attn::add2(s2, s3, p[2], p[3]);
                            y[i / 2] = attn::pack2(p[0], p[1]);
                            y[i / 2 + 1] = attn::pack2(p[2], p[3]);
                        }
                        attn::tmem_st32(tS + 32u * h, y);
                    }
                    l += (s0 + s1) + (s2 + s3);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&sh.p[t]);
            }
            if (ok && e > k.b0) {
                ok = wait_warp(&sh.o[t], step - 1);
                tc_fence_after();
            }
            if (!ok) break;
            if (work) {
                // a row that saw no key has l = 0: o = 0 and lse = -infinity
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const long long at = (long long)(k.q0 + tok) * a.Hq + head;
                const bool parts = a.splits > 1;
                const long long n_rows = (long long)a.total_q * a.Hq;
                if (row) {
                    const float lse = l == 0.f ? -INFINITY : (mc + log2f(l)) * kLn2;
                    if (parts) a.lse_part[k.split * n_rows + at] = lse;
                    else if (a.lse) a.lse[at] = lse;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t y[16];
                    if (e > k.b0) {
                        tmem_ld16(tO + 16u * j, y);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = 0;
                    }
                    float f[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[i] = l == 0.f ? 0.f : __uint_as_float(y[i]) * inv;
                    if (row && parts) {
                        float4 *dst = reinterpret_cast<float4 *>(
                            a.o_part + (k.split * n_rows + at) * D + 16 * j);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                    } else if (row) {
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + at * D + 16 * j;
                        uint32_t u[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = attn::pack2(f[2 * i], f[2 * i + 1]);
                        attn::store16(dst, u);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok) give_up();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) {
        tmem_relinquish();
        tmem_dealloc(tb, C::TM_COLS);
    }
}

template <int D>
cudaError_t launch_fwd(const Args &a, const Maps &maps, cudaStream_t s) {
    const long long blocks = (long long)a.items * a.splits * a.Hk;
    if (blocks == 0) return cudaSuccess;
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(attn_tc_fwd_kernel<D>), Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    attn_tc_fwd_kernel<D><<<(unsigned)blocks, kThreads, Cfg<D>::SMEM, s>>>(a, maps);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

bool attn_tc_ready() { return tmap::encode_fn() != nullptr; }

cudaError_t launch_attn_tc_fwd(const Args &a, int d, int total_k, cudaStream_t s) {
    Maps maps;
    maps.tokens = attn::tile_tokens(a.G);
    if (!attn::map_rows(&maps.q, a.q, d, a.Hq, a.total_q, a.q_stride, a.G, maps.tokens) ||
        !attn::map_rows(&maps.k, a.k, d, a.Hk, total_k, a.k_stride, 1, kTile) ||
        !attn::map_rows(&maps.v, a.v, d, a.Hk, total_k, a.v_stride, 1, kTile))
        return cudaErrorInvalidValue;
    return d == 128 ? launch_fwd<128>(a, maps, s) : launch_fwd<64>(a, maps, s);
}

}  // namespace kla
