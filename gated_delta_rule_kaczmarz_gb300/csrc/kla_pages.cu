// The pages of a cache: who holds them, and what is moved when that changes.
//
// The book of a cache is a table [S][columns] of page numbers, the lengths [S] and
// a count of holders for each page; a page without holders is free.  Nothing else is kept, so
// any order of calls, captured ones too, finds the state that the last one left.
//
// Each operator is one CTA, or one cluster of 8, that reads and changes the book
// (its phases part at barriers, what they hand over goes through the workspace), and
// where pages move a second kernel that copies those that the first listed.  The
// first is bound by latency, a barrier and a round trip to L2 for each phase: 2 to 9
// us.  The second is bound by HBM: 2060 pages of 36 KB in 4 layers 99 us behind the
// first, 0.91 of measured bandwidth (92 and 0.97 by itself, cold).
#include "kla_internal.h"
#include "kla_launch.cuh"

namespace kla {
namespace {

constexpr int kCtas = 8, kThreads = 1024;
constexpr int kMostSequences = 1 << 18;

// The workspace: status word, what the phases share, then arrays.
struct Shared {
    unsigned status;
    int copies;                  // pages that the copy kernel moves
    alignas(16) int sums[4][kCtas];
};
static_assert(sizeof(Shared) <= kWsHeader, "fits the header");

struct Book {
    Pages p;
    Shared *sh;
    int *from, *to;              // [n] pages that move
    int *a, *b, *c;              // [n] scratch
    int *rows;                   // [n][columns + 1]
};

// All threads of the launch, which is one cluster or one CTA.
__device__ __forceinline__ void all_barrier() {
    if (gridDim.x == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cta_of_all() { return blockIdx.x; }
__device__ __forceinline__ int thread_of_all() { return blockIdx.x * kThreads + threadIdx.x; }
__device__ __forceinline__ int threads_of_all() { return gridDim.x * kThreads; }

// What other CTAs of the cluster wrote: from L2.  (Volatile reads would wait for one
// another: the sums below took 8000 cycles so.)
__device__ __forceinline__ int at(const int *p) { return __ldcg(p); }

__device__ __forceinline__ int length_of(const Book &k, int s) {
    const long long most = (long long)k.p.columns * k.p.page;
    const int n = k.p.lens[s];
    return n < 0 ? 0 : (n < most ? n : (int)most);
}
__device__ __forceinline__ int pages_of(const Book &k, int len) {
    return (int)(((long long)len + k.p.page - 1) / k.p.page);
}
__device__ __forceinline__ bool is_page(const Book &k, int p) { return p >= 0 && p < k.p.n_pages; }

// Sums of N numbers over the CTA, and of the threads before this one.
template <int N>
__device__ __forceinline__ void cta_scan(const int (&x)[N], int (&before)[N], int (&all)[N], int (*warps)[32]) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = x[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int y = __shfl_up_sync(0xffffffffu, s[i], o);
            if (lane >= o) s[i] += y;
        }
    __syncthreads();
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < N; ++i) warps[i][warp] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int w = warps[i][lane];
        int t = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        before[i] = s[i] - x[i] + __shfl_sync(0xffffffffu, t - w, warp);
        all[i] = __shfl_sync(0xffffffffu, t, 31);
    }
}

// The share of n things that a CTA takes, in multiples of 4.
__device__ __forceinline__ void share_of(int n, int &a, int &e) {
    const int each = ((n + (int)gridDim.x - 1) / (int)gridDim.x + 3) & ~3;
    const long long x = (long long)each * cta_of_all();
    a = x < n ? (int)x : n;
    e = x + each < n ? (int)(x + each) : n;
}

// The sum of the shares' counts, of which this CTA's is `own`, and of those before it.
__device__ __forceinline__ int total_of(const int *sums, int own, int &before) {
    static_assert(kCtas == 8, "two reads");
    if (gridDim.x == 1) {
        before = 0;
        return own;
    }
    const int4 u = __ldcg(reinterpret_cast<const int4 *>(sums)), v = __ldcg(reinterpret_cast<const int4 *>(sums) + 1);
    const int x[kCtas] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    int t = 0;
    before = 0;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
        if (c < cta_of_all()) before += x[c];
        if (c < (int)gridDim.x) t += x[c];
    }
    return t;
}

// Entries of a row are taken by a warp kRow at a time: what is read of them is asked
// for at once, before anything is written.
constexpr int kEntries = 4, kRow = 32 * kEntries;

// ------------------------------------------------------------------ fork, free
// Sequence dst[f] becomes what src[f] was (src NULL or -1: empty), all at once.
__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    __shared__ unsigned seen[kMostSequences / 32];       // a bit for each target
    const int tid = threadIdx.x, lane = tid % 32, warp = thread_of_all() / 32;
    after_previous();
    let_next_start();
    // every CTA looks the whole list over
    for (int i = tid; i < (p.S + 31) / 32; i += kThreads) seen[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int f = tid; f < p.n; f += kThreads) {
        const int d = p.dst[f], s = p.src ? p.src[f] : -1;
        bad = bad || d < 0 || d >= p.S || s < -1 || s >= p.S ||
              (atomicOr(&seen[d / 32], 1u << d % 32) >> d % 32 & 1);
    }
    if (__syncthreads_or(bad)) {                         // nothing is changed
        if (thread_of_all() == 0) k.sh->status = kDevBadTable;
        return;
    }
    // what the rows will be, and the counts: the tables are still as they were
    const int pieces = p.columns / kRow + 1;             // (a row of no columns has a length)
    const unsigned work = (unsigned)p.n * (unsigned)pieces;
    for (unsigned x = warp; x < work; x += threads_of_all() / 32) {
        const int f = (int)(x / pieces), c0 = (int)(x % pieces) * kRow + lane;
        const int s = p.src ? p.src[f] : -1, d = p.dst[f], len = s < 0 ? 0 : length_of(k, s);
        const int held = pages_of(k, len), had = pages_of(k, length_of(k, d));
        int *row = k.rows + (long long)f * (p.columns + 1);
        int now[kEntries], old[kEntries];
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
            const int c = c0 + 32 * i;
            now[i] = c < held ? p.table[(long long)s * p.columns + c] : -1;
            old[i] = c < had ? p.table[(long long)d * p.columns + c] : -1;
        }
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
            const int c = c0 + 32 * i;
            if (c < held) {
                if (is_page(k, now[i])) atomicAdd(&p.refs[now[i]], 1);
                else bad = true;
            }
            if (c < had) {
                if (is_page(k, old[i])) atomicAdd(&p.refs[old[i]], -1);
                else bad = true;
            }
            if (c < p.columns) row[c] = now[i];
        }
        if (c0 == 0) row[p.columns] = len;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) k.sh->sums[0][cta_of_all()] = bad;
    all_barrier();
    for (unsigned x = warp; x < work; x += threads_of_all() / 32) {
        const int f = (int)(x / pieces), c0 = (int)(x % pieces) * kRow + lane, d = p.dst[f];
        const int *row = k.rows + (long long)f * (p.columns + 1);
        int now[kEntries];
#pragma unroll
        for (int i = 0; i < kEntries; ++i) now[i] = c0 + 32 * i < p.columns ? at(row + c0 + 32 * i) : 0;
#pragma unroll
        for (int i = 0; i < kEntries; ++i)
            if (c0 + 32 * i < p.columns) p.table[(long long)d * p.columns + c0 + 32 * i] = now[i];
        if (c0 == 0) p.lens[d] = at(row + p.columns);
    }
    int before;
    if (thread_of_all() == 0) k.sh->status = total_of(k.sh->sums[0], bad, before) ? kDevBadTable : kDevOk;
}

// ------------------------------------------------------------------ growth
// What a sequence needs: pages [first, first + pages) of its row, the first of
// them a copy of `last`, the one that is there, where `copy`.
struct Need {
    int len, more, first, pages, last;
    bool copy, bad;
};
__device__ __forceinline__ Need need_of(const Book &k, int s) {
    const Pages &p = k.p;
    Need x{length_of(k, s), p.more[s], 0, 0, 0, false, false};
    x.bad = x.more < 0 || (long long)x.len + x.more > (long long)p.columns * p.page;
    if (x.more <= 0 || x.bad) return x;
    if (x.len % p.page != 0) {
        x.last = p.table[(long long)s * p.columns + x.len / p.page];
        x.bad = !is_page(k, x.last);
        x.copy = !x.bad && p.refs[x.last] > 1;
    }
    x.first = pages_of(k, x.len) - x.copy;
    x.pages = pages_of(k, x.len + x.more) - x.first;
    return x;
}
// The share of a .. e - 1 that a thread takes, and how many at most: few of them lie
// in as many warps as they can.
__device__ __forceinline__ int share_of_thread(int a, int e, int &x, int &y) {
    const int gap = kThreads / max(e - a, 1), each = (e - a + kThreads - 1) / kThreads;
    if (gap > 1) {
        const int tid = threadIdx.x;
        x = min(a + tid / gap, e);
        y = tid % gap == 0 ? min(x + 1, e) : x;
    } else {
        x = min(a + (int)threadIdx.x * each, e);
        y = min(x + each, e);
    }
    return each;
}

// A thread has sequences that follow each other, a warp pages, so one scan tells them
// the places of all; what a thread found of its first sequence it keeps.
__global__ void __launch_bounds__(kThreads) pages_grow_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    __shared__ int warps[4][32];
    const int tid = threadIdx.x, lane = tid % 32, cta = cta_of_all();
    after_previous();
    let_next_start();
    int s0, s1, r0, r1;
    share_of(p.S, s0, s1);
    const int turns = share_of_thread(s0, s1, s0, s1);
    share_of(p.n_pages, r0, r1);
    const int per_warp = ((r1 - r0 + kThreads - 1) / kThreads) * 32;
    r0 = min(r0 + tid / 32 * per_warp, r1);
    r1 = min(r0 + per_warp, r1);
    // pages needed and copies, free pages
    int count[4] = {}, before[4], all[4];                // needed, copies, free, bad
#pragma unroll 4
    for (int r = r0 + lane; r < r1; r += 32) count[2] += p.refs[r] == 0;
    Need own{};
    for (int s = s0; s < s1; ++s) {
        const Need x = need_of(k, s);
        if (s == s0) own = x;
        count[0] += x.pages;
        count[1] += x.copy;
        count[3] += x.bad;
    }
    cta_scan(count, before, all, warps);
    if (tid < 4) k.sh->sums[tid][cta] = tid == 0 ? all[0] : tid == 1 ? all[1] : tid == 2 ? all[2] : all[3];
    all_barrier();
    int rank, number, place, none;
    const int need = total_of(k.sh->sums[0], all[0], rank), copies = total_of(k.sh->sums[1], all[1], number);
    const int spare = total_of(k.sh->sums[2], all[2], place), bad = total_of(k.sh->sums[3], all[3], none);
    if (thread_of_all() == 0) {
        k.sh->status = bad ? kDevBadTable : need > spare ? kDevNoPages : kDevOk;
        k.sh->copies = bad || need > spare ? 0 : copies;
    }
    if (bad || need > spare) return;                     // nothing is changed
    // the free pages, in order, as far as they are needed
    place += __shfl_sync(0xffffffffu, before[2], 0);
    for (int r = r0; r < r1 && place < need; r += 32) {
        const bool free = r + lane < r1 && p.refs[r + lane] == 0;
        const unsigned frees = __ballot_sync(0xffffffffu, free);
        const int rank_of = place + __popc(frees & ((1u << lane) - 1));
        if (free && rank_of < need) k.a[rank_of] = r + lane;
        place += __popc(frees);
    }
    // where each sequence's begin in that order, and its copy's number
    rank += before[0];
    number += before[1];
    int own_rank = rank, own_number = own.copy ? number : -1;
    for (int s = s0; s < s1; ++s) {
        const Need x = s == s0 ? own : need_of(k, s);
        if (s > s0) {
            k.b[s] = rank;
            k.c[s] = x.copy ? number : -1;
        }
        rank += x.pages;
        number += x.copy;
    }
    all_barrier();                                       // (counts change from here on)
    for (int i = 0; i < turns; ++i) {
        const int s = s0 + i;
        if (i > 0) {
            own.pages = own.more = 0;
            if (s < s1) {
                own.more = p.more[s];
                own.len = length_of(k, s);
                own_rank = k.b[s];
                own_number = k.c[s];
                own.first = pages_of(k, own.len) - (own_number >= 0);
                own.pages = own.more > 0 ? pages_of(k, own.len + own.more) - own.first : 0;
                if (own_number >= 0) own.last = p.table[(long long)s * p.columns + own.first];
            }
        }
        if (own.pages > 0) {
            const int page = at(k.a + own_rank);
            p.table[(long long)s * p.columns + own.first] = page;
            p.refs[page] = 1;
            if (own_number >= 0) {
                k.to[own_number] = page;
                k.from[own_number] = own.last;
                atomicAdd(&p.refs[own.last], -1);
            }
        }
        if (own.more > 0) p.lens[s] = own.len + own.more;
        // more pages than one: by the warp
        for (unsigned left = __ballot_sync(0xffffffffu, own.pages > 1); left; left &= left - 1) {
            const int of = __ffs(left) - 1;
            const int seq = __shfl_sync(0xffffffffu, s, of), pages = __shfl_sync(0xffffffffu, own.pages, of);
            const int first = __shfl_sync(0xffffffffu, own.first, of);
            const int at0 = __shfl_sync(0xffffffffu, own_rank, of);
            for (int x = 1 + lane; x < pages; x += kRow) {
                int page[kEntries];
#pragma unroll
                for (int y = 0; y < kEntries; ++y) page[y] = x + 32 * y < pages ? at(k.a + at0 + x + 32 * y) : -1;
#pragma unroll
                for (int y = 0; y < kEntries; ++y)
                    if (page[y] >= 0) {
                        p.table[(long long)seq * p.columns + first + x + 32 * y] = page[y];
                        p.refs[page[y]] = 1;
                    }
            }
        }
    }
}

// ------------------------------------------------------------------ trimming
// The last more[s] positions of a sequence are given up, with the pages behind those
// that are left: one page of a sequence by its thread, more by the warp.
__global__ void __launch_bounds__(kThreads) pages_trim_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    const int tid = threadIdx.x, lane = tid % 32;
    after_previous();
    let_next_start();
    int s0, s1, none;
    share_of(p.S, s0, s1);
    const int turns = share_of_thread(s0, s1, s0, s1);
    bool bad = false;
    for (int s = s0; s < s1; ++s) bad = bad || p.more[s] < 0 || p.more[s] > length_of(k, s);
    bad = __syncthreads_or(bad);
    if (tid == 0) k.sh->sums[0][cta_of_all()] = bad;
    all_barrier();
    if (total_of(k.sh->sums[0], bad, none)) {                 // nothing is changed
        if (thread_of_all() == 0) k.sh->status = kDevBadTable;
        return;
    }
    bad = false;
    for (int i = 0; i < turns; ++i) {
        const int s = s0 + i, n = s < s1 ? p.more[s] : 0;
        int first = 0, held = 0;
        if (n > 0) {
            const int len = length_of(k, s);
            first = pages_of(k, len - n);
            held = pages_of(k, len);
            p.lens[s] = len - n;
        }
        auto drop = [&](int page) {
            if (is_page(k, page)) atomicAdd(&p.refs[page], -1);
            else bad = true;
        };
        if (held > first) {
            int &entry = p.table[(long long)s * p.columns + first];
            drop(entry);
            entry = -1;
        }
        for (unsigned left = __ballot_sync(0xffffffffu, held > first + 1); left; left &= left - 1) {
            const int of = __ffs(left) - 1;
            const int seq = __shfl_sync(0xffffffffu, s, of), end = __shfl_sync(0xffffffffu, held, of);
            int *row = p.table + (long long)seq * p.columns;
            for (int c = __shfl_sync(0xffffffffu, first, of) + 1 + lane; c < end; c += kRow) {
                int page[kEntries];
#pragma unroll
                for (int y = 0; y < kEntries; ++y) page[y] = c + 32 * y < end ? row[c + 32 * y] : 0;
#pragma unroll
                for (int y = 0; y < kEntries; ++y)
                    if (c + 32 * y < end) {
                        drop(page[y]);
                        row[c + 32 * y] = -1;
                    }
            }
        }
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) k.sh->sums[1][cta_of_all()] = bad;
    all_barrier();
    if (thread_of_all() == 0) k.sh->status = total_of(k.sh->sums[1], bad, none) ? kDevBadTable : kDevOk;
}

// ------------------------------------------------------------------ compaction
__global__ void __launch_bounds__(kThreads) pages_compact_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    __shared__ int warps[1][32];
    const int tid = threadIdx.x, cta = cta_of_all();
    after_previous();
    let_next_start();
    if (thread_of_all() == 0) k.sh->status = kDevOk;     // (reports come behind the barriers)
    int r0, r1, before;
    share_of(p.n_pages, r0, r1);
    int used[1] = {}, rank[1], all[1];
    for (int r = r0 + tid; r < r1; r += kThreads) used[0] += p.refs[r] > 0;
    cta_scan(used, rank, all, warps);
    if (tid == 0) k.sh->sums[0][cta] = all[0];
    all_barrier();
    const int n_used = total_of(k.sh->sums[0], all[0], before);
    // holes below n_used in order (a), used pages from there on in reverse order (b)
    int holes[1] = {};
    for (int r = r0; r < r1; r += 4 * kThreads) {
        int on[4], n[1] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = r + 4 * tid + i;
            on[i] = x < r1 && p.refs[x] > 0;
            n[0] += on[i];
        }
        cta_scan(n, rank, all, warps);
        rank[0] += before;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = r + 4 * tid + i;
            if (x >= r1) break;
            if (on[i] && x >= n_used) {
                k.b[n_used - 1 - rank[0]] = x;
            } else {
                if (!on[i] && x < n_used) {
                    k.a[x - rank[0]] = x;
                    ++holes[0];
                }
                p.page_map[x] = on[i] ? x : -1;
            }
            rank[0] += on[i];
        }
        before += all[0];
    }
    cta_scan(holes, rank, all, warps);
    if (tid == 0) k.sh->sums[1][cta] = all[0];
    all_barrier();
    const int moved = total_of(k.sh->sums[1], all[0], before);
    for (int i = thread_of_all(); i < moved; i += threads_of_all()) {
        const int from = at(k.b + moved - 1 - i), to = at(k.a + i);
        p.page_map[from] = to;
        p.refs[to] = p.refs[from];
        p.refs[from] = 0;
        k.from[i] = from;
        k.to[i] = to;
    }
    if (thread_of_all() == 0) {
        k.sh->copies = moved;
        *p.n_used = n_used;
    }
    all_barrier();
    const int lane = tid % 32, pieces = (p.columns + kRow - 1) / kRow;
    const unsigned long long work = (unsigned long long)p.S * (unsigned)pieces;
    for (unsigned long long w = thread_of_all() / 32; w < work; w += threads_of_all() / 32) {
        const int s = (int)(w / (unsigned)pieces), c0 = (int)(w % (unsigned)pieces) * kRow + lane;
        const int held = pages_of(k, length_of(k, s));
        int *row = p.table + (long long)s * p.columns;
        int from[kEntries], to[kEntries];
#pragma unroll
        for (int i = 0; i < kEntries; ++i) from[i] = c0 + 32 * i < held ? row[c0 + 32 * i] : -1;
#pragma unroll
        for (int i = 0; i < kEntries; ++i) to[i] = is_page(k, from[i]) ? at(p.page_map + from[i]) : -1;
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
            if (c0 + 32 * i >= held) continue;
            if (to[i] < 0) atomicMax(&k.sh->status, (unsigned)kDevBadTable);  // no page, or a free one: left
            else if (to[i] != from[i]) row[c0 + 32 * i] = to[i];
        }
    }
}

// ------------------------------------------------------------------ copies
// The lists of a copy that the caller gives: every page once among the targets,
// none of them a source of another.
__global__ void __launch_bounds__(kThreads) pages_check_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    const int tid = thread_of_all();
    after_previous();
    let_next_start();
    for (int i = tid; i < p.n; i += threads_of_all()) {
        if (is_page(k, p.src[i])) k.a[p.src[i]] = -1;
        if (is_page(k, p.dst[i])) k.a[p.dst[i]] = -1;
    }
    all_barrier();
    bool bad = false;
    for (int i = tid; i < p.n; i += threads_of_all()) {
        bad = bad || !is_page(k, p.src[i]) || !is_page(k, p.dst[i]) || atomicCAS(&k.a[p.dst[i]], -1, i) != -1;
        k.from[i] = p.src[i];
        k.to[i] = p.dst[i];
    }
    all_barrier();
    for (int i = tid; i < p.n; i += threads_of_all())
        if (is_page(k, p.src[i])) {
            const int other = at(k.a + p.src[i]);
            bad = bad || (other != -1 && other != i);
        }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) k.sh->sums[0][cta_of_all()] = bad;
    all_barrier();
    if (tid == 0) {
        int before;
        bad = total_of(k.sh->sums[0], bad, before) != 0;
        k.sh->status = bad ? kDevBadTable : kDevOk;
        k.sh->copies = bad ? 0 : p.n;
    }
}

constexpr int kCopyThreads = 256, kEach = 4;
constexpr long long kPiece = (long long)kCopyThreads * kEach * 16;      // bytes

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ Book k) {
    after_previous();
    let_next_start();
    const Pages &p = k.p;
    const int copies = k.sh->copies;
    const unsigned pieces = (unsigned)((p.page_bytes + kPiece - 1) / kPiece);
    const unsigned long long all = (unsigned long long)copies * (unsigned)p.layers * pieces;
    for (unsigned long long x = blockIdx.x; x < all; x += gridDim.x) {
        const unsigned piece = (unsigned)(x % pieces);
        const unsigned long long y = x / pieces;
        const int i = (int)(y % (unsigned)copies), layer = (int)(y / (unsigned)copies);
        const int from = k.from[i], to = k.to[i];
        char *base = static_cast<char *>(p.pool) + (long long)layer * p.n_pages * p.page_bytes;
        const char *src = base + (long long)from * p.page_bytes;
        char *dst = base + (long long)to * p.page_bytes;
        int4 v[kEach];
#pragma unroll
        for (int z = 0; z < kEach; ++z) {
            const long long at = piece * kPiece + ((long long)z * kCopyThreads + threadIdx.x) * 16;
            if (at < p.page_bytes) v[z] = __ldcs(reinterpret_cast<const int4 *>(src + at));
        }
#pragma unroll
        for (int z = 0; z < kEach; ++z) {
            const long long at = piece * kPiece + ((long long)z * kCopyThreads + threadIdx.x) * 16;
            if (at < p.page_bytes) __stcs(reinterpret_cast<int4 *>(dst + at), v[z]);
        }
    }
}

// ------------------------------------------------------------------ host
size_t most(int S, int n_pages, int n) {
    size_t x = (size_t)(S > n_pages ? S : n_pages);
    x = x > (size_t)n ? x : (size_t)n;
    return (x + 63) & ~(size_t)63;
}

Book book_of(const Pages &p) {
    Book k{p, static_cast<Shared *>(p.ws), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    const size_t n = most(p.S, p.n_pages, p.n);
    k.from = reinterpret_cast<int *>(static_cast<unsigned char *>(p.ws) + kWsHeader);
    k.to = k.from + n;
    k.a = k.to + n;
    k.b = k.a + n;
    k.c = k.b + n;
    k.rows = k.c + n;
    return k;
}

// One CTA up to `most` units of work, whose barriers are cheaper, else the cluster,
// which has more hands.  Both in us.  Forks, by rows times pieces of kRow entries: 32 rows
// of 64 entries 4.6 and 5.4, 40 5.9 and 5.3, 8 of 500 4.9 and 5.8.  Growth, by pages and
// 128 for a sequence: 128 sequences among 16384 pages 5.7 and 6.8, 1024 among 131072 11.0
// and 8.3; 256 that take 32 pages each among 16384, with the trimming behind it, 20.5 and 17.7.
// Trimming, by sequences: 256 that lose a page or none 2.9 and 4.8, 25 pages each 8.1
// and 6.1; 64 of 25 pages 3.8 and 5.4, 512 12.6 and 6.1.  Compaction, by pages and
// entries: 2048 pages with 32 x 64 6.4 and 8.8, 4096 with 64 x 64 8.2 and 9.1, 8192 with
// 64 x 64 9.9 and 9.2.
constexpr long long kForkPieces = 32, kGrowEntries = 32768, kCompactEntries = 8192, kCopyEntries = 4096,
                    kTrimEntries = 256;

cudaError_t run(void (*kernel)(const Book), const Book &k, long long work, long long most, cudaStream_t s) {
    const bool one = work <= most;
    const cudaError_t e = launch_next(kernel, one ? 1 : kCtas, kThreads, 0, one ? 1 : kCtas, k, s);
    note_launch();
    return e;
}

// The pages that the kernel before it listed.
cudaError_t copy(const Book &k, long long copies, cudaStream_t s) {
    const Pages &p = k.p;
    if (p.layers == 0 || p.page_bytes == 0 || copies == 0) return cudaSuccess;
    const long long pieces = (p.page_bytes + kPiece - 1) / kPiece;
    const long long most = copies * p.layers;
    const long long blocks = most > 152 * 8 / pieces ? 152 * 8 : most * pieces;
    const cudaError_t e = launch_next(pages_copy_kernel, (unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), kCopyThreads,
                                      0, 1, k, s);
    note_launch();
    return e;
}

}  // namespace

bool pages_too_many(int S) { return S > kMostSequences; }

size_t pages_workspace_bytes(int S, int columns, int n_pages, int n) {
    const size_t x = most(S, n_pages, n);
    const size_t rows = (size_t)n * ((size_t)columns + 1);
    return (kWsHeader + (5 * x + rows) * sizeof(int) + 255) & ~(size_t)255;
}

cudaError_t launch_pages_fork(const Pages &p, cudaStream_t s) {
    return run(pages_fork_kernel, book_of(p), (long long)p.n * (p.columns / kRow + 1), kForkPieces, s);
}
cudaError_t launch_pages_grow(const Pages &p, cudaStream_t s) {
    const Book k = book_of(p);
    const cudaError_t e = run(pages_grow_kernel, k, p.n_pages + 128LL * p.S, kGrowEntries, s);
    return e != cudaSuccess ? e : copy(k, p.S, s);
}
cudaError_t launch_pages_trim(const Pages &p, cudaStream_t s) {
    return run(pages_trim_kernel, book_of(p), p.S, kTrimEntries, s);
}
cudaError_t launch_pages_compact(const Pages &p, cudaStream_t s) {
    const Book k = book_of(p);
    const cudaError_t e = run(pages_compact_kernel, k, p.n_pages + (long long)p.S * p.columns, kCompactEntries, s);
    return e != cudaSuccess ? e : copy(k, p.n_pages / 2, s);
}
cudaError_t launch_pages_copy(const Pages &p, cudaStream_t s) {
    const Book k = book_of(p);
    const cudaError_t e = run(pages_check_kernel, k, p.n, kCopyEntries, s);
    return e != cudaSuccess ? e : copy(k, p.n, s);
}

}  // namespace kla
