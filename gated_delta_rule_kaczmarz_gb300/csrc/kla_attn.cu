// Causal attention, host side: which kernels a call runs, its workspace and
// its launches.  The kernels and their reasons are in kla_attn_tc.cu and
// kla_attn_bwd_tc.cu (tensor cores) and kla_attn_simt.cu (CUDA cores).
#include <atomic>
#include <cstdlib>
#include <mutex>

#include "kla_attn_tc.cuh"

namespace kla {
namespace {

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Of the current device; a device's count is asked for once.
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

// Items of one side: tiles of ceil(len * mult / per) per sequence.
struct Side {
    int mult, per, tiles;
    long long items;
};
Side side(const AttnProblem &p, bool keys, int mult, int per) {
    Side r{mult, per, 0, 0};
    const int len = keys ? p.Tk : p.Tq, total = keys ? p.total_k : p.total_q;
    if (p.cu_q) {
        // a sequence adds at most one partial tile, and has none without tokens
        r.items = (long long)total * mult / per + (p.n_seq < total ? p.n_seq : total);
    } else {
        r.tiles = (int)ceil_div((long long)len * mult, per);
        r.items = (long long)p.n_seq * r.tiles;
    }
    return r;
}

// Rows of a CUDA-core tile: 64 reuses a loaded key four times as often as 16,
// but leaves SMs empty where there are few rows and wastes them where a
// sequence has fewer (a decode batch).
int simt_rows(const AttnProblem &p, bool keys) {
    const int mult = keys ? 1 : p.Hq / p.Hk, total = keys ? p.total_k : p.total_q;
    const long long each = ceil_div((long long)total * mult, p.n_seq);
    return each <= 16 || side(p, keys, mult, 64).items * p.Hk < sm_count() ? 16 : 64;
}

// The number of parts of `tiles` key tiles that makes a launch shortest, each
// part of at least `least` tiles: waves of blocks, `slots` at a time, times the
// tiles that each walks and `extra` tiles' time for its start and end; a join
// takes `extra` tiles' time too.  Only where there are under two waves.
int cheapest_splits(long long blocks, long long tiles, int slots, int extra, int least) {
    if (blocks < 1 || blocks >= 2 * slots) return 1;
    int best = 1;
    long long cost = 0;
    for (int n = 1; n <= attn::kMaxSplits && n * least < tiles + least; ++n) {
        const long long c = ceil_div(blocks * n, slots) * (ceil_div(tiles, n) + extra) +
                            (n > 1 ? extra : 0);
        if (n == 1 || c < cost) {
            cost = c;
            best = n;
        }
    }
    return best;
}

// Parts of the key axis on the CUDA cores: as on the tensor cores below, with
// two places an SM, tiles of 64 keys, and a tile's time for a block's start and
// end and for the join.  In fp32, one part and the
// chosen: B 1, T 256, 2 heads of 64 18 and 16 us; one token over 32768 keys of 8
// heads of 64 1544 and 96 us; of B 16 over 4096 keys of 4 heads of 128 367 and 181.
// Two places whatever the kernel: the blocks that an SM holds (1, 2 or 3, by head
// size and rows) moved 46 of 68 sizes with heads of 64, to between 0.77 (B 2,
// T 2048, one head: 131 and 101 us) and 1.17 of their time (40 tokens over 700 keys
// of 8 heads: 83 and 96; B 4, T 2048, 2 heads: 141 and 164), because the model takes
// all blocks for equally long.
int simt_splits(const AttnProblem &p, long long blocks) {
    return cheapest_splits(blocks, ceil_div(p.total_k, (long long)p.n_seq * 64), 2 * sm_count(), 1, 1);
}

// The tensor cores take bf16 with groups that fit into a tile's 128 rows.
bool on_tensor_cores(const AttnProblem &p) {
    return p.dtype == 1 && p.Hq / p.Hk <= attn::kTile && p.total_k > 0 && attn_tc_ready();
}

// Parts of the key axis on the tensor cores, one CTA per SM: the number that
// makes the whole launch shortest, counted in key tiles walked one after
// another (waves of CTAs times the tiles of each, and 4 tiles' time for a
// CTA's start and end).  Only where the unsplit launch has under two waves of
// CTAs that all walk about the same tiles, that is few query rows.
int tc_splits(const AttnProblem &p, long long blocks) {
    const long long tiles = ceil_div(p.total_k, (long long)p.n_seq * attn::kTile);
    return cheapest_splits(blocks, tiles, sm_count(), 4, 2);
}

struct FwdPlan {
    bool tc;
    Side q;
    int rows, splits;
    size_t table, o_part, lse_part, bytes;    // offsets and size of the workspace
};
FwdPlan fwd_plan(const AttnProblem &p) {
    FwdPlan f{};
    const int G = p.Hq / p.Hk;
    f.tc = on_tensor_cores(p);
    if (f.tc) {
        f.q = side(p, false, 1, 2 * attn::tile_tokens(G));
        f.splits = tc_splits(p, f.q.items * p.Hk);
    } else {
        f.rows = simt_rows(p, false);
        f.q = side(p, false, G, f.rows);
        f.splits = simt_splits(p, f.q.items * p.Hk);
    }
    size_t at = kWsHeader;
    f.table = at;
    if (p.cu_q) at = up256(at + f.q.items * sizeof(int2));
    f.o_part = at;
    if (f.splits > 1) {
        const size_t rows = (size_t)f.splits * p.total_q * p.Hq;
        at = up256(at + rows * p.d * sizeof(float));
        f.lse_part = at;
        at = up256(at + rows * sizeof(float));
    }
    f.bytes = at;
    return f;
}

struct BwdPlan {
    bool tc;
    Side q, k;
    int tile;
    size_t table_q, table_k, delta, delta_few, bytes;
};
BwdPlan bwd_plan(const AttnProblem &p) {
    BwdPlan b{};
    const int G = p.Hq / p.Hk;
    b.tc = on_tensor_cores(p);
    if (b.tc) {
        b.q = side(p, false, 1, attn::tile_tokens(G));
        b.k = side(p, true, 1, attn::kTile);
    } else {
        b.tile = simt_rows(p, false);
        if (p.total_k == 0 || simt_rows(p, true) == 16) b.tile = 16;
        b.q = side(p, false, G, b.tile);
        b.k = side(p, true, 1, b.tile);
    }
    size_t at = kWsHeader;
    b.table_q = at;
    if (p.cu_q) at = up256(at + b.q.items * sizeof(int2));
    b.table_k = at;
    if (p.cu_q) at = up256(at + b.k.items * sizeof(int2));
    b.delta = at;
    const size_t rows = up256((size_t)p.total_q * p.Hq * sizeof(float));
    b.delta_few = p.dtype == 1 ? at + rows : at;
    b.bytes = b.delta_few + rows;
    return b;
}

attn::Args make_args(const AttnProblem &p) {
    attn::Args a{};
    a.q = p.q; a.k = p.k; a.v = p.v; a.o = p.o; a.go = p.go; a.out = p.out;
    a.dq = p.dq; a.dk = p.dk; a.dv = p.dv; a.lse_in = p.lse_in; a.lse = p.lse;
    a.q_stride = p.q_stride; a.k_stride = p.k_stride; a.v_stride = p.v_stride;
    a.go_stride = p.go_stride; a.cu_q = p.cu_q; a.cu_k = p.cu_k; a.k_lens = p.k_lens;
    a.status = static_cast<unsigned *>(p.ws);
    a.n_seq = p.n_seq; a.Tq = p.Tq; a.Tk = p.Tk; a.Hq = p.Hq; a.Hk = p.Hk; a.G = p.Hq / p.Hk;
    a.splits = 1; a.total_q = p.total_q; a.scale = p.scale;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    // Test hook: with KLA_TEST_LOST_WAIT set, every tensor-core CTA takes a wait
    // under way of its first item for one that ran out.
    a.lost_wait = std::getenv("KLA_TEST_LOST_WAIT") != nullptr;
    return a;
}

unsigned char *at(const AttnProblem &p, size_t offset) {
    return static_cast<unsigned char *>(p.ws) + offset;
}

// Of packed sequences: the check, the status word and the item tables.
cudaError_t prepare(const AttnProblem &p, const AttnTable &t0, const AttnTable &t1,
                    cudaStream_t s) {
    if (!p.cu_q) return cudaSuccess;
    return launch_attn_prep(p.cu_q, p.cu_k, p.n_seq, p.total_q, p.total_k, t0, t1,
                            static_cast<unsigned *>(p.ws), s);
}

void take(attn::Args &a, const Side &x, int2 *table) {
    a.items = (int)x.items;
    a.tiles = x.tiles;
    a.table = table;
}

}  // namespace

// The setting stays with the device's context, so each kernel asks once per
// device (a few kernels: a short list of what was asked for).
cudaError_t allow_dynamic_smem(const void *kernel, size_t bytes) {
    struct Asked {
        const void *kernel;
        int device;
    };
    constexpr int kMost = 256;
    static Asked asked[kMost];
    static int n = 0;
    static std::mutex lock;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> hold(lock);
    for (int i = 0; i < n; ++i)
        if (asked[i].kernel == kernel && asked[i].device == dev) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && n < kMost) asked[n++] = {kernel, dev};
    return e;
}

size_t attn_fwd_workspace_bytes(const AttnProblem &p) { return fwd_plan(p).bytes; }
size_t attn_bwd_workspace_bytes(const AttnProblem &p) { return bwd_plan(p).bytes; }

bool attn_too_large(const AttnProblem &p) {
    const int G = p.Hq / p.Hk;
    const long long q = side(p, false, G, 16).items, k = side(p, true, 1, 16).items;
    // rows are counted in 32 bits, up to a tile past the last (as many of the
    // smallest size are 275 GB)
    const long long rows = (long long)p.total_q * p.Hq + attn::kTile;
    return q * p.Hk > INT32_MAX || k * p.Hk > INT32_MAX || rows > INT32_MAX;
}

cudaError_t launch_attn_no_queries(const AttnProblem &p, cudaStream_t s) {
    const cudaError_t e = prepare(p, {}, {}, s);
    const long long bytes = (long long)p.total_k * p.Hk * p.d * (p.dtype == 1 ? 2 : 4);
    if (e != cudaSuccess || !p.dk || bytes == 0) return e;
    return launch_attn_zero(p.dk, p.dv, bytes, static_cast<unsigned *>(p.ws), s);
}

cudaError_t launch_attn_fwd(const AttnProblem &p, cudaStream_t s) {
    const FwdPlan f = fwd_plan(p);
    attn::Args a = make_args(p);
    int2 *table = p.cu_q ? reinterpret_cast<int2 *>(at(p, f.table)) : nullptr;
    cudaError_t e = prepare(p, {table, p.cu_q, f.q.mult, f.q.per, (int)f.q.items, true}, {}, s);
    if (e != cudaSuccess) return e;
    take(a, f.q, table);
    a.splits = f.splits;
    if (f.splits > 1) {
        a.o_part = reinterpret_cast<float *>(at(p, f.o_part));
        a.lse_part = reinterpret_cast<float *>(at(p, f.lse_part));
    }
    e = f.tc ? launch_attn_tc_fwd(a, p.d, p.total_k, s)
             : launch_attn_simt_fwd(a, f.rows, p.d, p.dtype, s);
    if (e != cudaSuccess || f.splits == 1) return e;
    return launch_attn_join(a, p.d, p.dtype, s);
}

cudaError_t launch_attn_bwd(const AttnProblem &p, cudaStream_t s) {
    const BwdPlan b = bwd_plan(p);
    attn::Args a = make_args(p);
    int2 *tq = p.cu_q ? reinterpret_cast<int2 *>(at(p, b.table_q)) : nullptr;
    int2 *tk = p.cu_q ? reinterpret_cast<int2 *>(at(p, b.table_k)) : nullptr;
    cudaError_t e = prepare(p, {tq, p.cu_q, b.q.mult, b.q.per, (int)b.q.items, true},
                            {tk, p.cu_k, b.k.mult, b.k.per, (int)b.k.items, false}, s);
    if (e != cudaSuccess) return e;
    a.delta = reinterpret_cast<float *>(at(p, b.delta));
    a.delta_few = reinterpret_cast<float *>(at(p, b.delta_few));
    e = launch_attn_delta(a, p.d, p.dtype, s);
    if (e != cudaSuccess) return e;
    attn::Args keys = a;
    take(keys, b.k, tk);
    take(a, b.q, tq);
    return b.tc ? launch_attn_tc_bwd(keys, a, p.d, p.total_k, s)
                : launch_attn_simt_bwd(keys, a, b.tile, p.d, p.dtype, s);
}

}  // namespace kla
