// The pages of a cache: who holds them, and what is moved when that changes.
//
// The book of a cache is a table [S][columns] of page numbers, the lengths [S] and
// a count of holders for each page; a page without holders is free.  Nothing else is kept, so
// any order of calls, captured ones too, finds the state that the last one left.
//
// Each operator is one cluster of 8 CTAs that reads and changes the book (its
// phases part at cluster barriers, what they hand over goes through the
// workspace), and where pages move a second kernel that copies those that the
// first listed.  The first is bound by latency: a barrier and a round trip to L2 for
// each phase.  The second is bound by HBM.
#include "kla_internal.h"

namespace kla {
namespace {

constexpr int kCtas = 8, kThreads = 1024, kAll = kCtas * kThreads;

// The workspace: status word, what the phases share, then arrays.
struct Shared {
    unsigned status;
    unsigned trouble;            // set by any thread; cleared in the first phase
    unsigned late;               // what is found once changes have begun: reported alone
    int copies;                  // pages that the copy kernel moves
    int sums[3][kCtas];
};
static_assert(sizeof(Shared) <= kWsHeader, "fits the header");

struct Book {
    Pages p;
    Shared *sh;
    int *from, *to;              // [n] pages that move
    int *a, *b;                  // [n] scratch
    int *rows;                   // [n][columns + 1]
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cta_of_cluster() { return blockIdx.x; }      // one cluster a launch
__device__ __forceinline__ int thread_of_all() { return blockIdx.x * kThreads + threadIdx.x; }
// Before a phase that looks whether to go on; and after it.
__device__ __forceinline__ void report(const Book &k, unsigned what) { atomicMax(&k.sh->trouble, what); }
__device__ __forceinline__ void report_late(const Book &k) { atomicMax(&k.sh->late, (unsigned)kDevBadTable); }
__device__ __forceinline__ unsigned look(const unsigned *p) { return *(const volatile unsigned *)p; }

// Entries are written by other CTAs of the cluster: not through the read-only path.
__device__ __forceinline__ int at(const int *p) { return *(const volatile int *)p; }

__device__ __forceinline__ int length_of(const Book &k, int s) {
    const long long most = (long long)k.p.columns * k.p.page;
    const int n = k.p.lens[s];
    return n < 0 ? 0 : (n < most ? n : (int)most);
}
__device__ __forceinline__ int pages_of(const Book &k, int len) { return (int)(((long long)len + k.p.page - 1) / k.p.page); }
__device__ __forceinline__ bool is_page(const Book &k, int p) { return p >= 0 && p < k.p.n_pages; }

// Sum over the CTA, and of the threads before this one.
__device__ __forceinline__ int cta_scan(int x, int &before, int *warps) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    int w = warps[lane], t = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += y;
    }
    before = s - x + __shfl_sync(0xffffffffu, t - w, warp);
    return __shfl_sync(0xffffffffu, t, 31);
}

// The share of n things that a CTA takes, in multiples of 4.
__device__ __forceinline__ void share_of(int n, int &a, int &e) {
    const int each = ((n + kCtas - 1) / kCtas + 3) & ~3;
    const long long x = (long long)each * cta_of_cluster();
    a = x < n ? (int)x : n;
    e = x + each < n ? (int)(x + each) : n;
}

// The sum of a share's counts, and of those before it.
__device__ __forceinline__ int total_of(const int *sums, int &before) {
    int t = 0;
    before = 0;
    for (int c = 0; c < kCtas; ++c) {
        const int x = at(sums + c);
        if (c < (int)cta_of_cluster()) before += x;
        t += x;
    }
    return t;
}

__device__ __forceinline__ void start(const Book &k) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");     // the copies' launch
    if (thread_of_all() == 0) {
        k.sh->trouble = k.sh->late = kDevOk;
        k.sh->copies = 0;
    }
}
__device__ __forceinline__ void finish(const Book &k) {
    cluster_barrier();
    if (thread_of_all() == 0) k.sh->status = max(look(&k.sh->trouble), look(&k.sh->late));
}

// ------------------------------------------------------------------ fork, free
// Sequence dst[f] becomes what src[f] was (src NULL or -1: empty), all at once.
__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    const int tid = thread_of_all(), lane = tid % 32, warp = tid / 32;
    start(k);
    for (int f = tid; f < p.n; f += kAll)
        if (p.dst[f] >= 0 && p.dst[f] < p.S) k.a[p.dst[f]] = -1;
    cluster_barrier();
    for (int f = tid; f < p.n; f += kAll) {
        const int d = p.dst[f], s = p.src ? p.src[f] : -1;
        if (d < 0 || d >= p.S || s < -1 || s >= p.S || atomicCAS(&k.a[d], -1, f) != -1)
            report(k, kDevBadTable);
    }
    cluster_barrier();
    if (look(&k.sh->trouble) != kDevOk) {        // nothing is changed
        finish(k);
        return;
    }
    // what the rows will be, and the counts: the tables are still as they were
    for (int f = warp; f < p.n; f += kAll / 32) {
        const int s = p.src ? p.src[f] : -1, d = p.dst[f], len = s < 0 ? 0 : length_of(k, s);
        const int held = pages_of(k, len), had = pages_of(k, length_of(k, d));
        int *row = k.rows + (long long)f * (p.columns + 1);
        for (int c = lane; c < p.columns; c += 32) {
            int x = -1;
            if (c < held) {
                x = p.table[(long long)s * p.columns + c];
                if (is_page(k, x)) atomicAdd(&p.refs[x], 1);
                else report_late(k);
            }
            row[c] = x;
            if (c < had) {
                const int y = p.table[(long long)d * p.columns + c];
                if (is_page(k, y)) atomicAdd(&p.refs[y], -1);
                else report_late(k);
            }
        }
        if (lane == 0) row[p.columns] = len;
    }
    cluster_barrier();
    for (int f = warp; f < p.n; f += kAll / 32) {
        const int d = p.dst[f];
        const int *row = k.rows + (long long)f * (p.columns + 1);
        for (int c = lane; c < p.columns; c += 32) p.table[(long long)d * p.columns + c] = at(row + c);
        if (lane == 0) p.lens[d] = at(row + p.columns);
    }
    finish(k);
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
    __shared__ int warps[32];
    const int tid = threadIdx.x, cta = cta_of_cluster();
    start(k);
    // pages needed and copies, of this CTA's sequences; free pages of its share
    int s0, s1, r0, r1, before;
    share_of(p.S, s0, s1);
    share_of(p.n_pages, r0, r1);
    int need = 0, copies = 0, spare = 0;
    bool bad = false;
    for (int s = s0 + tid; s < s1; s += kThreads) {
        const Need x = need_of(k, s);
        need += x.pages;
        copies += x.copy;
        bad = bad || x.bad;
    }
    for (int r = r0 + tid; r < r1; r += kThreads) spare += p.refs[r] == 0;
    need = cta_scan(need, before, warps);
    copies = cta_scan(copies, before, warps);
    spare = cta_scan(spare, before, warps);
    if (tid == 0) {
        k.sh->sums[0][cta] = need;
        k.sh->sums[1][cta] = copies;
        k.sh->sums[2][cta] = spare;
    }
    cluster_barrier();           // (trouble is cleared)
    if (bad) report(k, kDevBadTable);
    int need0, copies0, spare0;
    need = total_of(k.sh->sums[0], need0);
    copies = total_of(k.sh->sums[1], copies0);
    spare = total_of(k.sh->sums[2], spare0);
    if (need > spare && tid == 0) report(k, kDevNoPages);
    // the free pages, in order, as far as they are needed
    for (int r = r0; r < r1 && spare0 < need; r += 4 * kThreads) {
        int free[4], n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = r + 4 * tid + i;
            free[i] = x < r1 && p.refs[x] == 0;
            n += free[i];
        }
        int rank;
        const int all = cta_scan(n, rank, warps);
        rank += spare0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (free[i] && rank < need) k.a[rank] = r + 4 * tid + i;
            rank += free[i];
        }
        spare0 += all;
    }
    // where each sequence's begin in that order
    for (int s = s0; s < s1; s += kThreads) {
        Need x{0, 0, false, false};
        if (s + tid < s1) x = need_of(k, s + tid);
        int rank, crank;
        const int all = cta_scan(x.pages, rank, warps), call = cta_scan(x.copy, crank, warps);
        if (s + tid < s1) {
            k.b[s + tid] = need0 + rank;
            k.to[s + tid] = x.copy ? copies0 + crank : -1;       // its number among the copies, for now
        }
        need0 += all;
        copies0 += call;
    }
    cluster_barrier();
    if (look(&k.sh->trouble) != kDevOk) {        // nothing is changed
        finish(k);
        return;
    }
    // what a sequence copies: read before any count changes
    const int warp = thread_of_all() / 32, lane = tid % 32;
    for (int s = warp; s < p.S; s += kAll / 32) {
        const int n = p.more[s];
        if (n == 0) continue;
        const int len = length_of(k, s), number = at(k.to + s);
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
                k.rows[number] = page;
                k.from[number] = old;
                atomicAdd(&p.refs[old], -1);
            }
        }
        if (lane == 0) p.lens[s] = len + n;
    }
    cluster_barrier();
    for (int i = thread_of_all(); i < copies; i += kAll) k.to[i] = at(k.rows + i);
    if (thread_of_all() == 0) k.sh->copies = copies;
    finish(k);
}

// ------------------------------------------------------------------ compaction
__global__ void __launch_bounds__(kThreads) pages_compact_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    __shared__ int warps[32];
    const int tid = threadIdx.x, cta = cta_of_cluster();
    start(k);
    int r0, r1, before;
    share_of(p.n_pages, r0, r1);
    int used = 0;
    for (int r = r0 + tid; r < r1; r += kThreads) used += p.refs[r] > 0;
    used = cta_scan(used, before, warps);
    if (tid == 0) k.sh->sums[0][cta] = used;
    cluster_barrier();
    const int n_used = total_of(k.sh->sums[0], before);
    // holes below n_used in order (a), used pages from there on in reverse order (b)
    int holes = 0;
    for (int r = r0; r < r1; r += 4 * kThreads) {
        int on[4], n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = r + 4 * tid + i;
            on[i] = x < r1 && p.refs[x] > 0;
            n += on[i];
        }
        int rank;
        const int all = cta_scan(n, rank, warps);
        rank += before;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int x = r + 4 * tid + i;
            if (x >= r1) break;
            if (on[i] && x >= n_used) {
                k.b[n_used - 1 - rank] = x;
            } else {
                if (!on[i] && x < n_used) {
                    k.a[x - rank] = x;
                    ++holes;
                }
                p.page_map[x] = on[i] ? x : -1;
            }
            rank += on[i];
        }
        before += all;
    }
    holes = cta_scan(holes, before, warps);
    if (tid == 0) k.sh->sums[1][cta] = holes;
    cluster_barrier();
    holes = total_of(k.sh->sums[1], before);
    for (int i = thread_of_all(); i < holes; i += kAll) {
        const int from = at(k.b + holes - 1 - i), to = at(k.a + i);
        p.page_map[from] = to;
        p.refs[to] = p.refs[from];
        p.refs[from] = 0;
        k.from[i] = from;
        k.to[i] = to;
    }
    cluster_barrier();
    const int warp = thread_of_all() / 32, lane = tid % 32;
    for (int s = warp; s < p.S; s += kAll / 32) {
        const int held = pages_of(k, length_of(k, s));
        int *row = p.table + (long long)s * p.columns;
        for (int c = lane; c < held; c += 32) {
            const int x = row[c];
            const int y = is_page(k, x) ? at(p.page_map + x) : -1;
            if (y < 0) report_late(k);                           // no page, or a free one: left
            else if (y != x) row[c] = y;
        }
    }
    if (thread_of_all() == 0) {
        k.sh->copies = holes;
        *p.n_used = n_used;
    }
    finish(k);
}

// ------------------------------------------------------------------ copies
// The lists of a copy that the caller gives: every page once among the targets,
// none of them a source of another.
__global__ void __launch_bounds__(kThreads) pages_check_kernel(const __grid_constant__ Book k) {
    const Pages &p = k.p;
    const int tid = thread_of_all();
    start(k);
    for (int i = tid; i < p.n; i += kAll) {
        if (is_page(k, p.src[i])) k.a[p.src[i]] = -1;
        if (is_page(k, p.dst[i])) k.a[p.dst[i]] = -1;
    }
    cluster_barrier();
    for (int i = tid; i < p.n; i += kAll)
        if (!is_page(k, p.src[i]) || !is_page(k, p.dst[i]) || atomicCAS(&k.a[p.dst[i]], -1, i) != -1)
            report(k, kDevBadTable);
    cluster_barrier();
    for (int i = tid; i < p.n; i += kAll)
        if (is_page(k, p.src[i])) {
            const int other = at(k.a + p.src[i]);
            if (other != -1 && other != i) report(k, kDevBadTable);
        }
    cluster_barrier();
    if (look(&k.sh->trouble) == kDevOk) {
        for (int i = tid; i < p.n; i += kAll) {
            k.from[i] = p.src[i];
            k.to[i] = p.dst[i];
        }
        if (tid == 0) k.sh->copies = p.n;
    }
    finish(k);
}

constexpr int kCopyThreads = 256, kEach = 4;
constexpr long long kPiece = (long long)kCopyThreads * kEach * 16;      // bytes

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ Book k) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    Book k{p, static_cast<Shared *>(p.ws), nullptr, nullptr, nullptr, nullptr, nullptr};
    const size_t n = most(p.S, p.n_pages, p.n);
    k.from = reinterpret_cast<int *>(static_cast<unsigned char *>(p.ws) + kWsHeader);
    k.to = k.from + n;
    k.a = k.to + n;
    k.b = k.a + n;
    k.rows = k.b + n;
    return k;
}

cudaError_t run(void (*kernel)(const Book), const Book &k, cudaStream_t s) {
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = kCtas;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, k);
    note_launch();
    return e;
}

// The pages that the kernel before it listed.
cudaError_t copy(const Book &k, long long copies, cudaStream_t s) {
    const Pages &p = k.p;
    if (p.layers == 0 || p.page_bytes == 0 || copies == 0) return cudaSuccess;
    const long long pieces = (p.page_bytes + kPiece - 1) / kPiece;
    const long long most = copies * p.layers;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    const long long blocks = most > 152 * 8 / pieces ? 152 * 8 : most * pieces;
    cfg.gridDim = dim3((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pages_copy_kernel, k);
    note_launch();
    return e;
}

}  // namespace

size_t pages_workspace_bytes(int S, int columns, int n_pages, int n) {
    const size_t x = most(S, n_pages, n);
    const size_t rows = (size_t)n * ((size_t)columns + 1);
    return (kWsHeader + (4 * x + (rows > x ? rows : x)) * sizeof(int) + 255) & ~(size_t)255;
}

cudaError_t launch_pages_fork(const Pages &p, cudaStream_t s) {
    return run(pages_fork_kernel, book_of(p), s);
}
cudaError_t launch_pages_grow(const Pages &p, cudaStream_t s) {
    const Book k = book_of(p);
    const cudaError_t e = run(pages_grow_kernel, k, s);
    return e != cudaSuccess ? e : copy(k, p.S, s);
}
cudaError_t launch_pages_compact(const Pages &p, cudaStream_t s) {
    const Book k = book_of(p);
    const cudaError_t e = run(pages_compact_kernel, k, s);
    return e != cudaSuccess ? e : copy(k, p.n_pages / 2, s);
}
cudaError_t launch_pages_copy(const Pages &p, cudaStream_t s) {
    const Book k = book_of(p);
    const cudaError_t e = run(pages_check_kernel, k, s);
    return e != cudaSuccess ? e : copy(k, p.n, s);
}

}  // namespace kla
