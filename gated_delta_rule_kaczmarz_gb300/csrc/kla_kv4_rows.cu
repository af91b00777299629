// Rows of keys and values into the 4-bit cache and out of it.
//
//   scale = e4m3(min(max |x| / 6, 448)) over 16 features of x / unit
//   code  = e2m1(x / unit / scale), nearest, ties to even, saturated at 6
//
// A thread takes 16 features of one head of a pair of tokens (an even position
// and the next): the pair's values share bytes, so no byte has two writers, and
// of a pair with one new token the other's codes are kept.  Bound by HBM for
// prompts and by latency for single tokens.
#include <cuda_bf16.h>

#include "kla_kv4.cuh"

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
    long long slots;     // pairs of positions, all sequences'
    int per_seq;         // pairs of a sequence, not packed
};

// Sequence and pair of a slot; false: a table that does not hold.
__device__ __forceinline__ bool span_of(const Work &w, long long slot, int &seq, int &pair, Span &s) {
    const Kv4Rows &p = w.p;
    if (p.cu) {
        // sequence n's slots begin at cu[n] / 2 + n
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if ((long long)(p.cu[mid] >> 1) + mid <= slot) lo = mid; else hi = mid - 1;
        }
        seq = lo;
        const int a = p.cu[lo], e = p.cu[lo + 1];
        pair = (int)(slot - (a >> 1) - lo);
        s.row0 = a;
        s.rows = e - a;
        if (a < 0 || e < a || e > p.total) return false;
    } else {
        seq = (int)(slot / w.per_seq);
        pair = (int)(slot - (long long)seq * w.per_seq);
        s.row0 = (long long)seq * p.T;
        s.rows = p.T;
    }
    const int most = p.columns * p.page;
    int len = p.lens[seq];
    len = len < 0 ? 0 : (len < most ? len : most);
    if (p.from_start) {
        s.pos0 = 0;
        s.rows = len < p.T ? len : p.T;
    } else {
        s.pos0 = len - s.rows;
    }
    return true;
}

// The block of a position, or nullptr where the table names no page of the pool.
template <int D>
__device__ __forceinline__ unsigned char *block_of(const Kv4Rows &p, int seq, int pos, int head) {
    const int column = pos / p.page, in = pos - column * p.page;
    const int page = p.table[(long long)seq * p.columns + column];
    if (page < 0 || page >= p.n_pages) return nullptr;
    const long long block = ((long long)page * p.Hk + head) * (p.page / kv4::kBlock) + in / kv4::kBlock;
    return static_cast<unsigned char *>(p.pool) + block * Layout<D>::kBytes;
}

__device__ __forceinline__ void load16(const float *p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = reinterpret_cast<const float4 *>(p)[i];
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16 *p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ void store16(float *p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
            w[j] = reinterpret_cast<const uint32_t &>(b);
        }
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// x in units of its scale; returns the scale's code.  The scale's border cases
// are decided by amax / 6 correctly rounded (a midpoint of e4m3 times 6 has at
// most 8 bits, so no other quotient rounds to it).  x / scale is x times the
// reciprocal, corrected once by the exact remainder, which leaves less than 2^-45
// before the rounding; a quotient that is no border of e2m1 is at least 8/15 of a
// step of fp32 from one (a border times a scale has 8 bits, so x is a step or more
// from it, and a scale's significand is at most 15/8), so ties are ties.
__device__ __forceinline__ unsigned scaled(float (&x)[16], float inv_unit) {
    float top = 0.f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] *= inv_unit;
        top = fmaxf(top, fabsf(x[i]));
        fine = fine && fabsf(x[i]) < INFINITY;
    }
    uint32_t code;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
        : "=r"(code) : "f"(0.f), "f"(__fdiv_rn(top, 6.f)));
    if (!fine) code = 0x7f;                                  // the block reads as NaN
    const uint32_t h = kv4::scales_to_half2(code);
    const float s = __half2float(__ushort_as_half((unsigned short)h));
    const bool none = !fine || s == 0.f;
    const float r = none ? 0.f : __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float a = none ? 0.f : x[i], y = a * r;
        x[i] = fmaf(fmaf(-y, s, a), r, y);
    }
    return code;
}
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
    check_table(p);
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int each = p.Hk * (D / 16), unit = (int)(i % each), head = unit / (D / 16), f = unit % (D / 16);
    const long long slot = i / each;
    if (slot >= w.slots) return;
    int seq, pair;
    Span s;
    if (!span_of(w, slot, seq, pair, s)) {
        if (p.status) *p.status = kDevBadSeqlens;
        return;
    }
    // the pair that holds the sequence's first new position, and those behind it
    const int first = s.pos0 < 0 ? 0 : s.pos0, pos = (first & ~1) + 2 * pair;
    const int end = s.pos0 + s.rows;
    if (pos >= end) return;
    const bool even = pos >= first, odd = pos + 1 < end;
    if (!even && !odd) return;                      // no new rows behind an odd length
    unsigned char *block = block_of<D>(p, seq, pos, head);
    if (!block) {
        if (p.status) *p.status = kDevBadTable;
        return;
    }
    const int t = pos % kv4::kBlock;
    const long long row = s.row0 + (pos - s.pos0);
    float x[2][16];
    unsigned code[2];
    // keys
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        if (!(z ? odd : even)) continue;
        load16(static_cast<const T *>(p.k) + (row + z) * p.k_stride + head * D + f * 16, x[z]);
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        if (!(z ? odd : even)) continue;
        code[z] = scaled(x[z], p.k_inv);
        uint32_t c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            c[j] = codes({x[z][8 * j], x[z][8 * j + 2], x[z][8 * j + 4], x[z][8 * j + 6]},
                         {x[z][8 * j + 1], x[z][8 * j + 3], x[z][8 * j + 5], x[z][8 * j + 7]});
        *reinterpret_cast<uint2 *>(block + (t + z) * (D / 2) + 8 * f) = make_uint2(c[0], c[1]);
        block[Layout<D>::kKs + (t + z) * (D / 16) + f] = (unsigned char)code[z];
    }
    // values
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        if (z ? odd : even) {
            load16(static_cast<const T *>(p.v) + (row + z) * p.v_stride + head * D + f * 16, x[z]);
            code[z] = scaled(x[z], p.v_inv);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[z][j] = 0.f;
        }
    }
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = codes({x[0][4 * j], x[0][4 * j + 1], x[0][4 * j + 2], x[0][4 * j + 3]},
                     {x[1][4 * j], x[1][4 * j + 1], x[1][4 * j + 2], x[1][4 * j + 3]});
    uint4 *to = reinterpret_cast<uint4 *>(block + Layout<D>::kV + (t / 2) * D + 16 * f);
    unsigned char *vs = block + Layout<D>::kVs + f * kv4::kBlock + t;
    if (even && odd) {
        *to = make_uint4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<unsigned short *>(vs) = (unsigned short)(code[0] | code[1] << 8);
    } else {                            // the other token's codes stay
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
    check_table(p);
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int each = p.Hk * (D / 16), unit = (int)(i % each), head = unit / (D / 16), f = unit % (D / 16);
    const long long slot = i / each;
    if (slot >= w.slots) return;
    int seq, pair;
    Span s;
    if (!span_of(w, slot, seq, pair, s)) {
        if (p.status) *p.status = kDevBadSeqlens;
        return;
    }
    const int pos = (s.pos0 & ~1) + 2 * pair, end = s.pos0 + s.rows;
    if (pos >= end) return;
    const bool want[2] = {pos >= s.pos0, pos + 1 < end};
    const long long row = s.row0 + (pos - s.pos0);
    const unsigned char *block = nullptr;
    if (pos >= 0) {
        block = block_of<D>(p, seq, pos, head);
        if (!block && p.status) *p.status = kDevBadTable;
    }
    const int t = pos & (kv4::kBlock - 1);
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
        if (want[z])
            store16(static_cast<T *>(p.k_out) + (row + z) * p.k_stride + head * D + f * 16, x[z]);
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
        if (want[z])
            store16(static_cast<T *>(p.v_out) + (row + z) * p.v_stride + head * D + f * 16, x[z]);
}

template <typename T, int D>
cudaError_t launch(const Work &w, bool read, cudaStream_t s) {
    const long long n = w.slots * w.p.Hk * (D / 16), blocks = (n + kThreads - 1) / kThreads;
    if (read) kv4_read_kernel<T, D><<<(unsigned)blocks, kThreads, 0, s>>>(w);
    else kv4_append_kernel<T, D><<<(unsigned)blocks, kThreads, 0, s>>>(w);
    note_launch();
    return cudaGetLastError();
}

Work work_of(const Kv4Rows &p) {
    Work w{p, 0, p.T / 2 + 1};
    w.slots = p.cu ? (long long)p.total / 2 + p.B : (long long)p.B * w.per_seq;
    return w;
}

}  // namespace

bool kv4_rows_too_large(const Kv4Rows &p) {
    return work_of(p).slots * p.Hk * (p.d / 16) / kThreads >= INT32_MAX;
}

cudaError_t launch_kv4_rows(const Kv4Rows &p, bool read, cudaStream_t s) {
    const Work w = work_of(p);
    if (p.dtype == 1)
        return p.d == 64 ? launch<__nv_bfloat16, 64>(w, read, s) : launch<__nv_bfloat16, 128>(w, read, s);
    return p.d == 64 ? launch<float, 64>(w, read, s) : launch<float, 128>(w, read, s);
}

}  // namespace kla
