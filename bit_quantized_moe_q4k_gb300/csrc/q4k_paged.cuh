// q4k_paged.cuh -- what the attention-side kernels share: the sequences of a batch, the paged
// 8-bit cache's addresses and scales, and the position rotation's angles.
//
// The cache: codes in e4m3, [num_pages][kv_heads][page_size][head_dim], one scale per (page, kv
// head); value = code * scale. Sequence i's cached tokens lie in the pages table[i][0], table[i][1],
// ... in order; its new tokens are rows q_start[i] .. q_start[i+1] of the inputs and the last ones
// of its seq_lens[i] cached tokens.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "q4k_internal.cuh"

namespace q4k {

struct PagedBatch {
    const int32_t* q_start;
    const int32_t* seq_lens;
    const int32_t* table;
    int batch, m, max_pages, page_shift, num_pages;
};

// Sequence i's new rows [start, start + n) and cached length; the first new token's position is
// len - n (negative: the first rows have no token). Values that leave their ranges are clamped
// (no access leaves its buffer) and `bad` is set.
struct SeqSpan {
    int start, n, len;
};
__device__ __forceinline__ SeqSpan seq_span(const PagedBatch& B, int i, bool* bad) {
    const int a = __ldcg(B.q_start + i), b = __ldcg(B.q_start + i + 1), l = __ldcg(B.seq_lens + i);
    SeqSpan s;
    s.start = min(max(a, 0), B.m);
    s.n = min(max(b, s.start), B.m) - s.start;
    s.len = min(max(l, 0), B.max_pages << B.page_shift);
    *bad = s.start != a || s.start + s.n != b || s.len != l || s.len < s.n;
    return s;
}

// Page of the sequence, or -1 (flag raised) when the table holds an id outside [0, num_pages). The
// read and the check apart, for callers with other reads to issue in between.
__device__ __forceinline__ int page_entry(const PagedBatch& B, int seq, int page) {
    return __ldcg(B.table + (int64_t)seq * B.max_pages + page);
}
__device__ __forceinline__ int page_checked(const PagedBatch& B, int p, int* err_flag) {
    if ((unsigned)p < (unsigned)B.num_pages) return p;
    raise_flag(err_flag, Q4K_ERR_PAGE);
    return -1;
}
__device__ __forceinline__ int page_id(const PagedBatch& B, int seq, int page, int* err_flag) {
    return page_checked(B, page_entry(B, seq, page), err_flag);
}

// ---- element access -----------------------------------------------------------------------------
// What an earlier kernel of the stream may have written is read through L2 (ld.global.cg) here and
// in the kernels: a programmatic dependent launch starts before that kernel ends, so its SM's L1
// may hold lines from before the writes.
template <typename T> struct Vec;  // N consecutive elements of an input row as fp32
template <> struct Vec<float> {
    using Four = float4;  // four elements as they are in memory
    static __device__ __forceinline__ void unpack(const Four& f, float* v) {
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    }
    template <int N> static __device__ __forceinline__ void load(const float* p, float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 a = __ldcg(reinterpret_cast<const float4*>(p + i));
            v[i] = a.x; v[i + 1] = a.y; v[i + 2] = a.z; v[i + 3] = a.w;
        }
    }
    template <int N> static __device__ __forceinline__ void store(float* p, const float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
};
template <> struct Vec<__nv_bfloat16> {
    using Four = uint2;
    static __device__ __forceinline__ void unpack(const Four& f, float* v) {
        v[0] = __uint_as_float(f.x << 16); v[1] = __uint_as_float(f.x & 0xFFFF0000u);
        v[2] = __uint_as_float(f.y << 16); v[3] = __uint_as_float(f.y & 0xFFFF0000u);
    }
    template <int N> static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[N]) {
        uint32_t w[N / 2];
        if constexpr (N == 4) {
            const uint2 a = __ldcg(reinterpret_cast<const uint2*>(p));
            w[0] = a.x; w[1] = a.y;
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 8) {
                const uint4 a = __ldcg(reinterpret_cast<const uint4*>(p + i));
                w[i / 2] = a.x; w[i / 2 + 1] = a.y; w[i / 2 + 2] = a.z; w[i / 2 + 3] = a.w;
            }
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    template <int N> static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[N]) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if constexpr (N == 4) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 8)
                *reinterpret_cast<uint4*>(p + i) = make_uint4(w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3]);
        }
    }
};

// ---- rotation -----------------------------------------------------------------------------------
// The angle pos * f is needed only modulo one turn. With F = f / 2pi mod 1 as a 64-bit fraction,
// pos * F mod 2^64 is that fraction of a turn: integer wrap-around is the range reduction, exact
// but for F's own rounding (|pos| * 2^-53 of f, below 2^-22 of a turn at pos = 2^31 for f <= 1).
// F comes from f's 53 significant bits by one 64 x 64 bit product with 2/pi * 2^64 (fp64
// arithmetic is two orders of magnitude slower than integers here).
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    const uint64_t bits = (uint64_t)__double_as_longlong(f);
    const int e = (int)((bits >> 52) & 0x7FF);                             // f = M * 2^(e - 1086)
    const uint64_t M = ((bits & 0xFFFFFFFFFFFFFull) | (e ? 1ull << 52 : 0)) << 11;
    const uint64_t hi = __umul64hi(M, 0xA2F9836E4E441529ull);              // M * 2/pi
    const int sh = 1024 - e;                                               // turns * 2^64 = hi * 2^(e - 1024)
    uint64_t F = sh >= 64 ? 0 : sh >= 0 ? hi >> sh : sh > -64 ? hi << -sh : 0;
    return (bits >> 63) ? 0 - F : F;
}
// Sine and cosine of pos * F turns. The top bits choose the quadrant and leave |x| <= pi/4, where the
// Taylor polynomials to x^9 and x^10 are within 2^-28 and 2^-29 of the functions: rounding is all the error.
__device__ __forceinline__ void turn_sincos(int pos, uint64_t F, float* s, float* c) {
    const uint32_t t = (uint32_t)(((uint64_t)(int64_t)pos * F) >> 32);     // turn * 2^32
    const uint32_t q = (t + 0x20000000u) >> 30;                            // quarter turns, rounded
    const float x = (float)(int)(t - (q << 30)) * 1.46291807926715968e-9f; // 2 pi / 2^32
    const float z = x * x;
    float a = fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
    a = fmaf(z, a, 1.0f / 120.0f);
    a = fmaf(z, a, -1.0f / 6.0f);
    a = fmaf(x * z, a, x);
    float b = fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    b = fmaf(z, b, -1.0f / 720.0f);
    b = fmaf(z, b, 1.0f / 24.0f);
    b = fmaf(z, b, -0.5f);
    b = fmaf(z, b, 1.0f);
    const float u = (q & 1) ? b : a, v = (q & 1) ? a : b;
    *s = __uint_as_float(__float_as_uint(u) ^ (q & 2) << 30);
    *c = __uint_as_float(__float_as_uint(v) ^ ((q + 1) & 2) << 30);
}

// A head spread over D/8 lanes, 8 dims a lane in two runs of 4, so that a lane holds four whole
// pairs: (v[i], v[4 + i]) with "halves", (v[2i], v[2i + 1]) with "pairs". 32 / (D/8) heads a warp.
template <int D>
struct HeadLane {
    static constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    int c0, c1;   // first dim of each run
    int j0;       // first of the four pairs
    bool turns, pairs;

    __device__ __forceinline__ HeadLane(int rot_dim, int pairs_mode) {
        const int q = threadIdx.x & (kLanes - 1);
        pairs = pairs_mode != 0;
        j0 = 4 * q;
        turns = 8 * q < rot_dim;
        if (!pairs && turns) {
            c0 = 4 * q;
            c1 = c0 + (rot_dim >> 1);
        } else {  // "pairs", and the dims that do not turn (8 q >= rot_dim in either order)
            c0 = 8 * q;
            c1 = c0 + 4;
        }
    }
    __device__ __forceinline__ void shared(const float* head, float (&v)[8]) const {  // of a head in shared memory
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = head[c0 + i]; v[4 + i] = head[c1 + i]; }
    }
    template <typename T> __device__ __forceinline__ void load(const T* head, float (&v)[8]) const {
        float a[4], b[4];
        Vec<T>::load(head + c0, a);
        Vec<T>::load(head + c1, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    }
    // The same in two steps, for loads that are to be in flight while other work goes on.
    template <typename T> struct Raw {
        typename Vec<T>::Four a{}, b{};
    };
    template <typename T> __device__ __forceinline__ void load(const T* head, Raw<T>& r) const {
        r.a = __ldcg(reinterpret_cast<const typename Vec<T>::Four*>(head + c0));
        r.b = __ldcg(reinterpret_cast<const typename Vec<T>::Four*>(head + c1));
    }
    template <typename T> __device__ __forceinline__ static void unpack(const Raw<T>& r, float (&v)[8]) {
        Vec<T>::unpack(r.a, v);
        Vec<T>::unpack(r.b, v + 4);
    }
    template <typename T> __device__ __forceinline__ void store(T* head, const float (&v)[8]) const {
        const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
        Vec<T>::store(head + c0, a);
        Vec<T>::store(head + c1, b);
    }
    __device__ __forceinline__ void frequencies(const double* inv_freq, double (&f)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = turns ? __ldcg(inv_freq + j0 + i) : 0.0;
    }
    __device__ __forceinline__ void angles(int pos, const uint64_t (&F)[4], float (&sn)[4], float (&cs)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn_sincos(pos, F[i], &sn[i], &cs[i]);
    }
    // (a, b) -> (a cos - b sin, b cos + a sin)
    __device__ __forceinline__ void rotate(const float (&sn)[4], const float (&cs)[4], float (&v)[8]) const {
        if (!turns) return;
        if (pairs) {
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(sn[i], cs[i], v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(sn[i], cs[i], v[i], v[4 + i]);
        }
    }
    __device__ __forceinline__ static void turn(float sn, float cs, float& a, float& b) {
        const float x = a * cs - b * sn;
        b = b * cs + a * sn;
        a = x;
    }
    // 1 / sqrt(mean v^2 + eps), the mean over the head's lanes (the whole warp calls it): the hardware's estimate and one
    // Newton step, half the instructions of a root and a quotient. (0: infinite, as the quotient would be.)
    __device__ __forceinline__ static float inv_rms(float eps, const float (&v)[8]) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float a = fmaf(ss, 1.0f / (float)D, eps), r = rsqrtf(a);
        const float n = r * fmaf(-0.5f * a * r, r, 1.5f);
        return a > 1e-37f && a < 1e37f ? n : r;
    }
    __device__ __forceinline__ static void norm(const float (&w)[8], float eps, float (&v)[8]) {
        const float r = inv_rms(eps, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
    }
};

// ---- e4m3 ---------------------------------------------------------------------------------------
// Two e4m3 codes (low byte first) to two halves, and back (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t lo16) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(lo16));
    return r;
}
// All four codes of a word: bytes 0 and 1, bytes 2 and 3.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t* lo, uint32_t* hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(*lo), "=r"(*hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

constexpr int kMinScaleExp = -64;  // the scale of a page of zeros, and the smallest one

// The least e >= kMinScaleExp with amax <= 448 * 2^e; amax finite and >= 0. (448 = 1.75 * 2^8.)
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(e, kMinScaleExp);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // |e| <= 126

}  // namespace q4k
