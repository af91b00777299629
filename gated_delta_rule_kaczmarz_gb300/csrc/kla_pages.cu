// The pages of a cache: who holds them, and what is moved when that changes.
//
// The book of a cache is a table [S][columns] of page numbers, the lengths [S] and
// a count of holders for each page; a page without holders is free.  Nothing else is kept, so
// any order of calls, captured ones too, finds the state that the last one left.
//
// Each operator is one CTA, or one cluster of 8, that reads and changes the book
// (its phases part at barriers, what they hand over goes through the workspace), and
// where pages move a second kernel that copies those that the first listed.  The
// first is bound by latency, a barrier and a round trip to L2 for each phase: 4 to 9
// us.  The second is bound by HBM: 2048 pages of 36 KB in 4 layers 89 us, 0.99 of
// measured bandwidth.
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

// The sum of the shares' counts, and of those before this CTA's.
__device__ __forceinline__ int total_of(const int *sums, int &before) {
    static_assert(kCtas == 8, "two reads");
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
    for (int f = warp; f < p.n; f += threads_of_all() / 32) {
        const int s = p.src ? p.src[f] : -1, d = p.dst[f], len = s < 0 ? 0 : length_of(k, s);
        const int held = pages_of(k, len), had = pages_of(k, length_of(k, d));
        int *row = k.rows + (long long)f * (p.columns + 1);
        for (int c = lane; c < p.columns; c += 32) {
            int x = -1;
            if (c < held) {
                x = p.table[(long long)s * p.columns + c];
                if (is_page(k, x)) atomicAdd(&p.refs[x], 1);
                else bad = true;
            }
            row[c] = x;
            if (c < had) {
                const int y = p.table[(long long)d * p.columns + c];
                if (is_page(k, y)) atomicAdd(&p.refs[y], -1);
                else bad = true;
            }
        }
        if (lane == 0) row[p.columns] = len;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) k.sh->sums[0][cta_of_all()] = bad;
    all_barrier();
    for (int f = warp; f < p.n; f += threads_of_all() / 32) {
        const int d = p.dst[f];
        const int *row = k.rows + (long long)f * (p.columns + 1);
        for (int c = lane; c < p.columns; c += 32) p.table[(long long)d * p.columns + c] = at(row + c);
        if (lane == 0) p.lens[d] = at(row + p.columns);
    }
    int before;
    if (thread_of_all() == 0) k.sh->status = total_of(k.sh->sums[0], before) ? kDevBadTable : kDevOk;
}

// ------------------------------------------------------------------ growth
// What a sequence needs: pages [first, first + need) of its row, the first of
// them a copy of the one that is there where `copy`.
struct Need {
    int first, pages;
    bool copy, bad;
};
__device__ __forceinline__ Need need_of(const Book &k, int s) {
    const Pages &p = k.p;
    const int len = length_of(k, s), n = p.more[s];
    Need x{pages_of(k, len), 0, false, n < 0 || (long long)len + n > (long long)p.columns * p.page};
    if (n <= 0 || x.bad) return x;
    if (len % p.page != 0) {
        const int last = p.table[(long long)s * p.columns + len / p.page];
        x.bad = !is_page(k, last);
        x.copy = !x.bad && p.refs[last] > 1;
    }
    x.first -= x.copy;
    x.pages = pages_of(k, len + n) - x.first;
    return x;
}

__global__ void __launch_bounds__(kThreads) pages_grow_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    __shared__ int warps[4][32];
    const int tid = threadIdx.x, cta = cta_of_all();
    after_previous();
    let_next_start();
    // pages needed and copies, of this CTA's sequences; free pages of its share
    int s0, s1, r0, r1;
    share_of(p.S, s0, s1);
    share_of(p.n_pages, r0, r1);
    int count[4] = {};           // needed, copies, free, bad
    for (int s = s0 + tid; s < s1; s += kThreads) {
        const Need x = need_of(k, s);
        count[0] += x.pages;
        count[1] += x.copy;
        count[3] += x.bad;
    }
    for (int r = r0 + tid; r < r1; r += kThreads) count[2] += p.refs[r] == 0;
    {
        int before[4], all[4];
        cta_scan(count, before, all, warps);
        if (tid < 4) k.sh->sums[tid][cta] = tid == 0 ? all[0] : tid == 1 ? all[1] : tid == 2 ? all[2] : all[3];
    }
    all_barrier();
    int need0, copies0, spare0, none;
    const int need = total_of(k.sh->sums[0], need0), copies = total_of(k.sh->sums[1], copies0);
    const int spare = total_of(k.sh->sums[2], spare0), bad = total_of(k.sh->sums[3], none);
    if (thread_of_all() == 0) {
        k.sh->status = bad ? kDevBadTable : need > spare ? kDevNoPages : kDevOk;
        k.sh->copies = bad || need > spare ? 0 : copies;
    }
    if (bad || need > spare) return;                     // nothing is changed
    // the free pages, in order, as far as they are needed
    for (int r = r0; r < r1 && spare0 < need; r += 4 * kThreads) {
        int free[4], n[1] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = r + 4 * tid + i;
            free[i] = x < r1 && p.refs[x] == 0;
            n[0] += free[i];
        }
        int rank[1], all[1];
        cta_scan(n, rank, all, warps);
        rank[0] += spare0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (free[i] && rank[0] < need) k.a[rank[0]] = r + 4 * tid + i;
            rank[0] += free[i];
        }
        spare0 += all[0];
    }
    // where each sequence's begin in that order, and its copy's number
    for (int s = s0; s < s1; s += kThreads) {
        Need x{0, 0, false, false};
        if (s + tid < s1) x = need_of(k, s + tid);
        const int n[2] = {x.pages, x.copy};
        int rank[2], all[2];
        cta_scan(n, rank, all, warps);
        if (s + tid < s1) {
            k.b[s + tid] = need0 + rank[0];
            k.c[s + tid] = x.copy ? copies0 + rank[1] : -1;
        }
        need0 += all[0];
        copies0 += all[1];
    }
    all_barrier();
    const int warp = thread_of_all() / 32, lane = tid % 32;
    for (int s = warp; s < p.S; s += threads_of_all() / 32) {
        const int n = p.more[s];
        if (n == 0) continue;
        const int len = length_of(k, s), number = at(k.c + s);
        const int first = pages_of(k, len) - (number >= 0), pages = pages_of(k, len + n) - first;
        const int rank = at(k.b + s);
        int *row = p.table + (long long)s * p.columns;
        int old = 0;
        if (number >= 0) old = row[first];
        __syncwarp();
        for (int i = lane; i < pages; i += 32) {
            const int page = at(k.a + rank + i);
            row[first + i] = page;
            p.refs[page] = 1;
            if (i == 0 && number >= 0) {
                k.to[number] = page;
                k.from[number] = old;
                atomicAdd(&p.refs[old], -1);
            }
        }
        __syncwarp();
        if (lane == 0) p.lens[s] = len + n;
    }
}

// ------------------------------------------------------------------ trimming
// The last more[s] positions of a sequence are given up, with the pages behind those
// that are left: a warp to a sequence.
__global__ void __launch_bounds__(kThreads) pages_trim_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    const int tid = threadIdx.x, lane = tid % 32;
    after_previous();
    let_next_start();
    bool bad = false;                                    // every CTA looks all of them over
    for (int s = tid; s < p.S; s += kThreads) {
        const int n = p.more[s];
        bad = bad || n < 0 || n > length_of(k, s);
    }
    bad = __syncthreads_or(bad);
    all_barrier();                                       // (before a length changes)
    if (bad) {
        if (thread_of_all() == 0) k.sh->status = kDevBadTable;
        return;
    }
    for (int s = thread_of_all() / 32; s < p.S; s += threads_of_all() / 32) {
        const int n = p.more[s];
        if (n == 0) continue;
        const int len = length_of(k, s), held = pages_of(k, len);
        int *row = p.table + (long long)s * p.columns;
        for (int c = pages_of(k, len - n) + lane; c < held; c += 32) {
            const int x = row[c];
            if (is_page(k, x)) atomicAdd(&p.refs[x], -1);
            else bad = true;
            row[c] = -1;
        }
        __syncwarp();
        if (lane == 0) p.lens[s] = len - n;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) k.sh->sums[0][cta_of_all()] = bad;
    all_barrier();
    int before;
    if (thread_of_all() == 0) k.sh->status = total_of(k.sh->sums[0], before) ? kDevBadTable : kDevOk;
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
    const int n_used = total_of(k.sh->sums[0], before);
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
    const int moved = total_of(k.sh->sums[1], before);
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
    const int warp = thread_of_all() / 32, lane = tid % 32;
    for (int s = warp; s < p.S; s += threads_of_all() / 32) {
        const int held = pages_of(k, length_of(k, s));
        int *row = p.table + (long long)s * p.columns;
        for (int c = lane; c < held; c += 32) {
            const int x = row[c];
            const int y = is_page(k, x) ? at(p.page_map + x) : -1;
            if (y < 0) atomicMax(&k.sh->status, (unsigned)kDevBadTable);     // no page, or a free one: left
            else if (y != x) row[c] = y;
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
        bad = total_of(k.sh->sums[0], before) != 0;
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

// One CTA up to `most` entries, whose barriers are cheaper (1.0 to 2.6 us a call),
// else the cluster, which has more hands.  Both in us: a fork of 32 rows of 64 pages 5.8
// and 6.3, of 64 8.6 and 6.2; growth among 16384 pages 7.4 and 8.1, 32768 7.9 and 8.0,
// 131072 13.4 and 9.5 (a sequence that grows counts as 128 of them: of 256 that do among
// 3200 pages 18.5 and 11.5); compaction of 2048 pages with a table of 32 x 64 7.1 and 8.6, 4096
// with 64 x 64 8.7 and 8.7, 8192 with 128 x 64 12.3 and 8.9; trimming 64 sequences 2.1 and 2.5,
// 256 5.9 and 3.1.
constexpr long long kForkEntries = 2048, kGrowEntries = 32768, kCompactEntries = 8192, kCopyEntries = 4096,
                    kTrimEntries = 64;

cudaError_t run(void (*kernel)(const Book), const Book &k, long long entries, long long most, cudaStream_t s) {
    const bool one = entries <= most;
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
    return run(pages_fork_kernel, book_of(p), (long long)p.n * p.columns + p.S / 32, kForkEntries, s);
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
