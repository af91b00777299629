// Rows of keys and values into the 4-bit cache and out of it.
//
//   scale = e4m3(min(max |x| * (1/6), 448)) over 16 features of x / unit, 1/6 in fp32
//   code  = e2m1(x / unit / scale), nearest, ties to even, saturated at 6
//
// A thread takes 16 features of one head of a pair of tokens (an even position
// and the next): the pair's values share bytes, so no byte has two writers, and
// of a pair with one new token the other's codes are kept.  Bound by HBM, the append
// by the issue of its conversions too (0.68 of the slots): 306282 packed rows of 4 heads
// of 128 in bf16 133 and 122 us, 0.89 and 0.97 of measured HBM bandwidth.  A thread
// that goes on to 2, 4 or 8 pairs goes through the three reads before the first
// (sequence, length, page) once, but keeps fewer under way: the read 172, 183, 176
// where one pair took 164.  Rows are read and, where they lie so, written 32 bytes a
// thread at once (the read 164 -> 122).  Single tokens are bound by latency: 256 of 4
// heads of 128 2.5 us each way.
#include <cuda_bf16.h>

#include "kla_kv4.cuh"
#include "kla_launch.cuh"

namespace kla {
namespace {

using kv4::Layout;

constexpr int kThreads = 256;

// The rows of a sequence and the first one's position.
struct Span {
    long long row0;
    int rows, pos0;
};

struct Work {
    Kv4Rows p;
    int slots;           // pairs of positions, all sequences'
    int per_seq;         // pairs of a sequence, not packed
    kv4::Divisor by_each, by_seq, by_page;
};

// Sequence and pair of a slot; false: a table that does not hold.  n rows lie in
// n / 2 + 1 pairs at most, wherever they begin.  WRITES: rows keep the positions that the
// length gives them, and those behind the table's end are none; for reading a length is
// clamped to what the table has.
template <bool WRITES>
__device__ __forceinline__ bool span_of(const Work &w, int slot, int &seq, int &pair, Span &s) {
    const Kv4Rows &p = w.p;
    if (p.cu) {
        // sequence n's slots begin at cu[n] / 2 + n
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if ((p.cu[mid] >> 1) + mid <= slot) lo = mid; else hi = mid - 1;
        }
        seq = lo;
        const int a = p.cu[lo], e = p.cu[lo + 1];
        pair = slot - (a >> 1) - lo;
        s.row0 = a;
        s.rows = e - a;
        if (a < 0 || e < a || e > p.total || pair < 0) return false;
    } else {
        seq = kv4::divided(slot, w.by_seq);
        pair = slot - seq * w.per_seq;
        s.row0 = (long long)seq * p.T;
        s.rows = p.T;
    }
    const int most = p.columns * p.page;
    int len = p.lens[seq];
    len = len < 0 ? 0 : len;
    const int past = len > most ? len - most : 0;
    if (!WRITES) len -= past;
    if (p.from_start) {
        s.pos0 = 0;
        s.rows = len < p.T ? len : p.T;
    } else {
        s.pos0 = len - s.rows;
        if (WRITES) s.rows = s.rows > past ? s.rows - past : 0;
    }
    return true;
}

// The block of a position, or nullptr where the table names no page of the pool.
template <int D>
__device__ __forceinline__ unsigned char *block_of(const Work &w, int seq, int pos, int head) {
    const Kv4Rows &p = w.p;
    const int column = kv4::divided(pos, w.by_page), in = pos - column * p.page;
    const int page = p.table[(long long)seq * p.columns + column];
    if (page < 0 || page >= p.n_pages) return nullptr;
    const long long block = ((long long)page * p.Hk + head) * (p.page / kv4::kBlock) + in / kv4::kBlock;
    return static_cast<unsigned char *>(p.pool) + block * Layout<D>::kBytes;
}

// 16 features as they lie in memory, and as fp32.
template <typename T>
struct Raw {
    uint4 x[sizeof(T)];
    __device__ __forceinline__ void load(const T *p, bool on) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i)
            x[i] = on ? __ldcs(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&y)[16]) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (sizeof(T) == 4) {
                    y[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    y[(8 * i + 2 * j) % 16] = __uint_as_float(w[j] << 16);
                    y[(8 * i + 2 * j + 1) % 16] = __uint_as_float(w[j] & 0xffff0000u);
                }
            }
        }
    }
};
// 32 bytes in one store where they lie on such a boundary (rows may begin on any of
// 16), else in two.
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
__device__ __forceinline__ void store16(float *p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[8 * i + j]);
        store32(p + 8 * i, w);
    }
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&x)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = reinterpret_cast<const uint32_t &>(b);
    }
    store32(p, w);
}

// a / b, given r = 1 / b within 2^-22: the product, corrected once by its exact
// remainder, which leaves less than 2^-44 before the rounding.
__device__ __forceinline__ float quotient(float a, float b, float r) {
    const float q = a * r;
    return fmaf(fmaf(-q, b, a), r, q);
}
// x / unit in units of its scale; returns the scale's code (0, and what is not
// finite: the codes have no meaning).  Such quotients decide a code's border cases as
// exact ones do: a border of e2m1 times a scale has at most 8 bits, so an x that is not
// just that is a step of fp32 or more away, and its quotient by the scale, whose
// significand is at most 15/8, at least 8/15 of a step.
__device__ __forceinline__ unsigned scaled(float (&x)[16], float unit, float inv_unit) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)            // a NaN stays
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x[i])));
    const bool fine = top < INFINITY;
    top *= inv_unit;
    uint32_t code;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
        : "=r"(code) : "f"(0.f), "f"(top * (1.f / 6.f)));
    if (!fine) return 0x7f;                 // the 16 read as NaN
    const uint32_t h = kv4::scales_to_half2(code);
    const float s = __half2float(__ushort_as_half((unsigned short)h)) * unit;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    if (top > 8.f * 448.f) {                // far beyond the largest code: the quotients stay finite
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -8.f * s), 8.f * s);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = quotient(x[i], s, r);
    return code;
}
// Whether a scale's codes are to be written as zeros.
__device__ __forceinline__ bool no_codes(unsigned scale) { return scale == 0 || scale == 0x7f; }
// Codes of four bytes: lo[i] in the low four bits of byte i, hi[i] in the high.
__device__ __forceinline__ uint32_t codes(const float (&lo)[4], const float (&hi)[4]) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %5, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %6, %2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %7, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %4;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(lo[0]), "f"(lo[1]), "f"(lo[2]), "f"(lo[3]), "f"(hi[0]), "f"(hi[1]), "f"(hi[2]), "f"(hi[3]));
    return w;
}

// The first block looks the packed sequences' table over.
__device__ __forceinline__ void check_table(const Kv4Rows &p) {
    if (!p.cu || !p.status || blockIdx.x != 0) return;
    bool fine = threadIdx.x != 0 || (p.cu[0] == 0 && p.cu[p.B] == p.total);
    for (int n = threadIdx.x; n < p.B; n += kThreads) fine = fine && p.cu[n] <= p.cu[n + 1];
    if (!fine) *p.status = kDevBadSeqlens;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const __grid_constant__ Work w) {
    const Kv4Rows &p = w.p;
    after_previous();
    let_next_start();
    check_table(p);
    const int i = blockIdx.x * kThreads + threadIdx.x, each = p.Hk * (D / 16);
    const int slot = kv4::divided(i, w.by_each), unit = i - slot * each, head = unit / (D / 16), f = unit % (D / 16);
    if (slot >= w.slots) return;
    int seq, pair;
    Span s;
    if (!span_of<true>(w, slot, seq, pair, s)) {
        if (p.status) *p.status = kDevBadSeqlens;
        return;
    }
    if (pair > s.rows / 2) return;               // (a table that does not hold may ask for any)
    // the pair that holds the sequence's first new position, and those behind it
    const int first = s.pos0 < 0 ? 0 : s.pos0, pos = (first & ~1) + 2 * pair, end = s.pos0 + s.rows;
    const bool even = pos >= first && pos < end, odd = pos + 1 < end;
    if (!even && !odd) return;
    unsigned char *block = block_of<D>(w, seq, pos, head);
    if (!block) {
        if (p.status) *p.status = kDevBadTable;
        return;
    }
    const long long at = head * D + f * 16;
    const int t = pos % kv4::kBlock;
    const long long row = s.row0 + (pos - s.pos0);
    Raw<T> k[2], v[2];                           // all that is read is asked for at once
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        k[z].load(static_cast<const T *>(p.k) + (row + z) * p.k_stride + at, z ? odd : even);
        v[z].load(static_cast<const T *>(p.v) + (row + z) * p.v_stride + at, z ? odd : even);
    }
    float x[2][16];
    unsigned code[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        if (!(z ? odd : even)) continue;
        k[z].get(x[0]);
        const unsigned scale = scaled(x[0], p.k_unit, p.k_inv);
        uint32_t c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            c[j] = codes({x[0][8 * j], x[0][8 * j + 2], x[0][8 * j + 4], x[0][8 * j + 6]},
                         {x[0][8 * j + 1], x[0][8 * j + 3], x[0][8 * j + 5], x[0][8 * j + 7]});
        if (no_codes(scale)) c[0] = c[1] = 0;
        *reinterpret_cast<uint2 *>(block + (t + z) * (D / 2) + 8 * f) = make_uint2(c[0], c[1]);
        block[Layout<D>::kKs + (t + z) * (D / 16) + f] = (unsigned char)scale;
    }
    // values: of a token that is not there zeros
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        v[z].get(x[z]);
        code[z] = scaled(x[z], p.v_unit, p.v_inv);
    }
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = codes({x[0][4 * j], x[0][4 * j + 1], x[0][4 * j + 2], x[0][4 * j + 3]},
                     {x[1][4 * j], x[1][4 * j + 1], x[1][4 * j + 2], x[1][4 * j + 3]});
    const uint32_t mask = (no_codes(code[0]) ? 0u : 0x0f0f0f0fu) | (no_codes(code[1]) ? 0u : 0xf0f0f0f0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] &= mask;
    uint4 *to = reinterpret_cast<uint4 *>(block + Layout<D>::kV + (t / 2) * D + 16 * f);
    unsigned char *vs = block + Layout<D>::kVs + f * kv4::kBlock + t;
    if (even && odd) {
        *to = make_uint4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<unsigned short *>(vs) = (unsigned short)(code[0] | code[1] << 8);
    } else {                        // the other token's codes stay
        const uint32_t keep = even ? 0xf0f0f0f0u : 0x0f0f0f0fu;
        const uint4 old = *to;
        *to = make_uint4((old.x & keep) | (c[0] & ~keep), (old.y & keep) | (c[1] & ~keep),
                         (old.z & keep) | (c[2] & ~keep), (old.w & keep) | (c[3] & ~keep));
        vs[even ? 0 : 1] = (unsigned char)(even ? code[0] : code[1]);
    }
}

__device__ __forceinline__ float2 to_float2(uint32_t h) {
    return __half22float2(reinterpret_cast<const __half2 &>(h));
}

// The inverse.  Rows before a sequence's first position are zeros, rows of a
// table entry that names no page too.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Work w) {
    const Kv4Rows &p = w.p;
    after_previous();
    let_next_start();
    check_table(p);
    const int i = blockIdx.x * kThreads + threadIdx.x, each = p.Hk * (D / 16);
    const int slot = kv4::divided(i, w.by_each), unit = i - slot * each, head = unit / (D / 16), f = unit % (D / 16);
    if (slot >= w.slots) return;
    int seq, pair;
    Span s;
    if (!span_of<false>(w, slot, seq, pair, s)) {
        if (p.status) *p.status = kDevBadSeqlens;
        return;
    }
    if (pair > s.rows / 2) return;
    const int pos = (s.pos0 & ~1) + 2 * pair, end = s.pos0 + s.rows;
    if (pos >= end) return;
    const bool want[2] = {pos >= s.pos0, pos + 1 < end};
    const long long row = s.row0 + (pos - s.pos0);
    const unsigned char *block = nullptr;
    if (pos >= 0) {
        block = block_of<D>(w, seq, pos, head);
        if (!block && p.status) *p.status = kDevBadTable;
    }
    const int t = pos & (kv4::kBlock - 1);
    const long long at = head * D + f * 16;
    uint2 kc[2] = {};
    uint4 vc = {};
    uint32_t ks[2] = {}, vs = 0;
    if (block) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            kc[z] = *reinterpret_cast<const uint2 *>(block + (t + z) * (D / 2) + 8 * f);
            ks[z] = block[Layout<D>::kKs + (t + z) * (D / 16) + f];
        }
        vc = *reinterpret_cast<const uint4 *>(block + Layout<D>::kV + (t / 2) * D + 16 * f);
        vs = *reinterpret_cast<const unsigned short *>(block + Layout<D>::kVs + f * kv4::kBlock + t);
    }
    float x[2][16];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const float unit_of = to_float2(kv4::scales_to_half2(ks[z])).x * p.k_unit;
        const uint32_t c[2] = {kc[z].x, kc[z].y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t h[4];
            kv4::codes_to_half2(c[j], h);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float2 two = to_float2(h[y]);
                x[z][8 * j + 2 * y] = two.x * unit_of;
                x[z][8 * j + 2 * y + 1] = two.y * unit_of;
            }
        }
        if (want[z]) store16(static_cast<T *>(p.k_out) + (row + z) * p.k_stride + at, x[z]);
    }
    const float2 units = to_float2(kv4::scales_to_half2(vs));
    const uint32_t c[4] = {vc.x, vc.y, vc.z, vc.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h[4];
        kv4::codes_to_half2(c[j], h);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const float2 two = to_float2(h[y]);
            x[0][4 * j + y] = two.x * (units.x * p.v_unit);
            x[1][4 * j + y] = two.y * (units.y * p.v_unit);
        }
    }
#pragma unroll
    for (int z = 0; z < 2; ++z)
        if (want[z]) store16(static_cast<T *>(p.v_out) + (row + z) * p.v_stride + at, x[z]);
}

template <typename T, int D>
cudaError_t launch(const Work &w, bool read, cudaStream_t s) {
    const long long n = (long long)w.slots * w.p.Hk * (D / 16), blocks = (n + kThreads - 1) / kThreads;
    const cudaError_t e = launch_next(read ? kv4_read_kernel<T, D> : kv4_append_kernel<T, D>, (unsigned)blocks,
                                      kThreads, 0, 1, w, s);
    note_launch();
    return e;
}

long long slots_of(const Kv4Rows &p) {
    return p.cu ? (long long)p.total / 2 + p.B : (long long)p.B * (p.T / 2 + 1);
}

}  // namespace

bool kv4_rows_too_large(const Kv4Rows &p) {
    return slots_of(p) * p.Hk * (p.d / 16) + kThreads > INT32_MAX;
}

cudaError_t launch_kv4_rows(const Kv4Rows &p, bool read, cudaStream_t s) {
    const int per_seq = p.T / 2 + 1;
    const Work w{p, (int)slots_of(p), per_seq, kv4::divisor(p.Hk * (p.d / 16)), kv4::divisor(per_seq),
                 kv4::divisor(p.page)};
    if (p.dtype == 1)
        return p.d == 64 ? launch<__nv_bfloat16, 64>(w, read, s) : launch<__nv_bfloat16, 128>(w, read, s);
    return p.d == 64 ? launch<float, 64>(w, read, s) : launch<float, 128>(w, read, s);
}

}  // namespace kla
