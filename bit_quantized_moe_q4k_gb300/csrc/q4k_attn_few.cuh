// q4k_attn_few.cuh -- what the kernels of attention for few query rows share (q4k_attn.cu: whole sequences; q4k_prefix.cu: what
// sequences do not share): fragments of mma.m16n8k16, packed arithmetic, and a warp's ring of cache chunks in shared memory.
#pragma once

#include "q4k_paged.cuh"

namespace q4k {
namespace few {

constexpr int kChunk = 16;                    // tokens a warp takes at a time

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16816_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// Two fp32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ void add2(float2& a, float x, float y) {
    float2 b = make_float2(x, y);
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(reinterpret_cast<uint64_t&>(a)) : "l"(reinterpret_cast<uint64_t&>(b)));
}
__device__ __forceinline__ void fma2(float2& a, float x, float y, float scale) {  // a += (x, y) * scale
    float2 b = make_float2(x, y), c = make_float2(scale, scale);
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<uint64_t&>(a))
        : "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
}
__device__ __forceinline__ void mul2(float2& a, float x) {
    float2 b = make_float2(x, x);
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(reinterpret_cast<uint64_t&>(a)) : "l"(reinterpret_cast<uint64_t&>(b)));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 0x80 in each byte that is one of e4m3's two NaN codes (0x7F, 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) { return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// The ring of a warp: kRing stages of kPair chunks, and each chunk's page: K's scale, V's scale as
// log2 and reciprocal, whether there is such a page.
constexpr int kRing = 2, kPair = 2;
template <int D> constexpr int kSlot = 2 * kChunk * D;        // a chunk: K's rows, then V's
template <int D> constexpr int kStage = kPair * kSlot<D>;

// Where 16-byte unit `u` of row `r` lies in a chunk's K or V part, as 128-byte lines of 8 units: the
// unit's place in its line is xored with the row's parity times 4 (K at head_dim 128: a read
// meets rows of both parities) or with twice the row's group of four (V: a read meets all four groups).
template <int D> __device__ __forceinline__ int k_unit(int r, int u) {
    return 16 * (D == 128 ? 8 * r + (u ^ ((r & 1) << 2)) : 4 * r + u);
}
template <int D> __device__ __forceinline__ int v_unit(int r, int u) {
    const int x = D / 16 * r + u;
    return 16 * (x ^ ((r >> 2) << 1));
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

struct ChunkMeta {
    float ks, ev, inv;
    int ok;
};

// The pages of a warp's chunks, 32 at a time: lane i holds those of chunks i, 32 + i, ... Page ids are
// read two batches ahead and scales one, so that no issue waits for them.
struct PageAhead {
    int p0, p1, p2;
    float ks0, vs0, ks1, vs1;
};

// log2 of a page's V scale: exact for the powers of two that the append writes.
__device__ __forceinline__ float scale_log2_of(float s) {
    const uint32_t b = __float_as_uint(s);
    const float e = (float)((int)(b >> 23) - 127);
    return (b & 0x7FFFFFu) ? e + log2f(__uint_as_float((b & 0x7FFFFFu) | 0x3F800000u)) : e;
}

}  // namespace few
}  // namespace q4k
