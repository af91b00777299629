// What the attention kernels share: the request, where a sequence's rows are,
// the tables that map a launch's blocks to tiles, and the join of partial
// results over a split key axis.
//
// Rows are packed: the G = Hq / Hk query heads of a key head read the same
// keys and values, so a tile's row r is token r / G, head r % G of the group,
// and one load of a key tile serves all of them, in a prompt as for the single
// tokens of a decode batch.  Query i of lq sees the keys j <= i + lk - lq.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "kla_internal.h"

namespace kla {
namespace attn {

// One launch's tables and problem, passed by value to every kernel.
struct Args {
    const void *q, *k, *v, *o, *go;       // o, go: backward
    void *out, *dq, *dk, *dv;
    const float *lse_in;
    float *lse;
    float *delta, *delta_few;             // backward: [total_q][Hq], see delta_of
    long long q_stride, k_stride, v_stride, go_stride;
    const int *cu_q, *cu_k, *k_lens;      // device; cu_*: packed, k_lens: padded keys
    unsigned *status;                     // device status word
    const int2 *table;                    // packed: (sequence, tile) of every item
    int n_seq, Tq, Tk, Hq, Hk, G;
    int items;                            // fixed: n_seq * tiles, packed: table entries
    int tiles;                            // fixed: tiles of a sequence
    int splits;
    float *o_part, *lse_part;             // splits > 1: [splits][total_q][Hq][d], [..][Hq]
    int total_q;
    float scale, scale_log2;
    bool lost_wait;                       // test hook: a wait of every CTA runs out (tensor cores)
};

struct Seq {
    long long q0, k0;    // first row
    int lq, lk;
};

__device__ __forceinline__ Seq sequence(const Args &a, int s) {
    Seq r;
    if (a.cu_q) {
        r.q0 = a.cu_q[s];
        r.lq = a.cu_q[s + 1] - a.cu_q[s];
        r.k0 = a.cu_k[s];
        r.lk = a.cu_k[s + 1] - a.cu_k[s];
    } else {
        r.q0 = (long long)s * a.Tq;
        r.lq = a.Tq;
        r.k0 = (long long)s * a.Tk;
        r.lk = a.Tk;
        if (a.k_lens) {          // outside 0..Tk: clamped, every access stays in bounds
            const int n = a.k_lens[s];
            r.lk = n < 0 ? 0 : (n < a.Tk ? n : a.Tk);
        }
    }
    return r;
}

// delta of a row is sum go o.  bf16 rows that see at most kFewKeys keys take
// sum p dp instead, which is the same sum before o was rounded: with few keys p
// is near 1, and what the rounding of o adds to delta is larger than the
// rounding of ds (of a row with one key, whose ds is 0, it would be all there
// is).  Of a sequence of 4 tokens the relative error of dq and dk is 2.3e-3
// instead of 3.2e-3, of 128 tokens 2.4e-3 instead of 2.6e-3; more than 8 keys
// change it by less than 0.1e-3.  fp32: delta_few is delta.  (Rows without keys
// have a delta, 0, but no entry in delta_few.)
constexpr int kFewKeys = 8;
// Parts of a split key axis, at most (a multiple of the 16 lanes that join a row).
constexpr int kMaxSplits = 64;
__device__ __forceinline__ float delta_of(const Args &a, long long row, int keys) {
    return (keys >= 1 && keys <= kFewKeys ? a.delta_few : a.delta)[row];
}

// Packed sequences whose tables the check refused: nothing is done.  In the
// tensor-core kernels other CTAs of the launch write the word where a wait runs
// out, so there one thread reads it for all of its CTA.
__device__ __forceinline__ bool rejected(const Args &a) { return a.cu_q && *a.status != kDevOk; }

// Fixed lengths have no check before them: the first block of a call's first
// kernel clears the status word (blocks start in the order of their numbers, so it
// is none of those that a running CTA takes over).  What else writes it is a wait
// that ran out, a second and more after that block started.
__device__ __forceinline__ void clear_status(const Args &a) {
    if (!a.cu_q && blockIdx.x == 0 && threadIdx.x == 0) *a.status = kDevOk;
}

// The item of a block: sequence, tile, key head and split.  Fixed lengths:
// the last tiles first (they see the most keys, so the longest blocks start
// first), key heads and sequences innermost.  False: nothing to do.
struct Item {
    int seq, tile, head, split;
};
__device__ __forceinline__ bool item_of(const Args &a, int block, bool last_first, Item &it) {
    if (rejected(a)) return false;
    it.head = block % a.Hk;
    int x = block / a.Hk;
    if (a.table) {
        it.split = x % a.splits;
        const int2 e = a.table[x / a.splits];
        it.seq = e.x;
        it.tile = e.y;
        return e.x >= 0;
    }
    it.seq = x % a.n_seq;
    x /= a.n_seq;
    it.split = x % a.splits;
    x /= a.splits;
    it.tile = last_first ? a.tiles - 1 - x : x;
    return true;
}

// The key tiles of a split: [begin, end) of those of `n` that it takes.
__device__ __forceinline__ void split_range(int n, int splits, int split, int &begin, int &end) {
    const int per = (n + splits - 1) / splits;
    begin = split * per;
    end = begin + per < n ? begin + per : n;
    if (begin > end) begin = end;
}

}  // namespace attn

// A table that maps items to (sequence, tile): sequence n has
// ceil(len * mult / per) tiles; entries past the last item hold -1.
struct AttnTable {
    int2 *items;
    const int *cu;
    int mult, per, entries;
    bool last_first;      // a sequence's last tile first
};
// Checks the packed sequences' tables (writes *status) and fills up to two
// item tables (items nullptr: none).
cudaError_t launch_attn_prep(const int *cu_q, const int *cu_k, int n, int total_q, int total_k,
                             const AttnTable &t0, const AttnTable &t1, unsigned *status,
                             cudaStream_t s);
// Zeroes dk and dv (bytes each, a multiple of 16) where *status is OK.
cudaError_t launch_attn_zero(void *dk, void *dv, long long bytes, const unsigned *status,
                             cudaStream_t s);
cudaError_t launch_attn_join(const attn::Args &a, int d, int dtype, cudaStream_t s);
cudaError_t launch_attn_delta(const attn::Args &a, int d, int dtype, cudaStream_t s);

// CUDA-core kernels: any G.  rows / tile: rows of a tile, 16 or 64.
cudaError_t launch_attn_simt_fwd(const attn::Args &a, int rows, int d, int dtype, cudaStream_t s);
cudaError_t launch_attn_simt_bwd(const attn::Args &keys, const attn::Args &rows, int tile, int d,
                                 int dtype, cudaStream_t s);

}  // namespace kla
