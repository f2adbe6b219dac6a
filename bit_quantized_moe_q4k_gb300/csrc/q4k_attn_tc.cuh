// q4k_attn_tc.cuh -- what the tensor-core attention kernels share (prompts: q4k_attn_tc.cu; rows behind a shared prefix:
// q4k_prefix.cu): the cache's tiles expanded to fp16 operands, pages and scales looked up ahead, and the softmax of a row of S in
// tensor memory. The mathematics: x_j = c (code_k . q) + e_j, P_j = 2^(x_j - M + B).
#pragma once

#include "q4k_paged.cuh"
#include "q4k_sm100.cuh"
#include "q4k_sync.cuh"

namespace q4k {
namespace tc {
using namespace sm100;

constexpr int kRows = 128;   // query rows of a CTA
constexpr int kToks = 128;   // tokens of a tile
constexpr int kGroups = kToks / 16;
constexpr int kMetaRing = 4;

struct PromptParams {
    PagedBatch B;
    const void* q;
    void* out;
    int64_t q_stride, out_stride;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int kv_heads, group, window;
    int min_rows;       // sequences with fewer query rows per kv head are not this kernel's
    float scale_log2;   // |softmax scale| * log2(e)
    float sign;         // its sign, multiplied into the queries
    int* err_flag;
    uint64_t wait_ns;
};

// A tile's 16-token groups: where their rows begin in the cache (-1: no such page), K's scale, V's as
// log2 and reciprocal.
struct TileMeta {
    int64_t at[kGroups];
    float ks[kGroups], ev[kGroups], inv[kGroups];
    int all_ok;
};

template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_scale(float s) {  // exact for powers of two
    const uint32_t b = __float_as_uint(s);
    const float e = (float)((int)(b >> 23) - 127);
    return (b & 0x7FFFFFu) ? e + log2f(__uint_as_float((b & 0x7FFFFFu) | 0x3F800000u)) : e;
}
// Two fp32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// 16 codes to 16 halves.
__device__ __forceinline__ void expand16(const uint4& c, uint32_t (&h)[8]) {
    e4m3x4_to_f16x4(c.x, &h[0], &h[1]);
    e4m3x4_to_f16x4(c.y, &h[2], &h[3]);
    e4m3x4_to_f16x4(c.z, &h[4], &h[5]);
    e4m3x4_to_f16x4(c.w, &h[6], &h[7]);
}

// A wait of a whole warp, bounded in time: its lanes go on, or give up, together. The clock is looked at every 64 tries.
// A try suspends the thread, maybe for longer than a limit below a millisecond, so with SHORT such a limit is polled
// for; the page warp does, whose abort ends the others' waits (in all roles it took the bf16 prompt above 7 us more).
template <bool SHORT = false>
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    const bool poll = SHORT && limit_ns < 1000000;
    bool done = poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
    uint64_t t0 = 0;
    for (uint32_t i = 1; !done; ++i) {
        if (*abort) break;
        if (poll || (i & 63) == 0) {
            const uint64_t t = global_timer_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > limit_ns) break;
        }
        done = poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
    }
    return __all_sync(0xffffffffu, done) != 0;
}

// A warp's one arrival, once each of its lanes has read what the barrier gives back.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Expands half tiles (64 rows) of the cache. A thread reads 16 codes of rows 32 x + rs, in each 64-dim panel,
// and writes them as two 16-byte units of the panel's 128-byte rows; the eight threads of a store's phase
// hold two rows of different parity, so their units lie on different banks.
template <int D>
struct Loader {
    static constexpr int kPanels = D / 64, kLoads = 2 * kPanels;
    const uint8_t* cache;
    int rs;
    uint32_t u0, u1;
    __device__ __forceinline__ Loader(const uint8_t* codes, int i) : rs(i >> 2) {
        const int c = i & 3;
        cache = codes + (rs & 15) * D + 16 * c;
        u0 = rs * 128 + (((2 * c) ^ (rs & 7)) << 4);
        u1 = rs * 128 + (((2 * c + 1) ^ (rs & 7)) << 4);
    }
    // left: tokens of the tile that are there
    __device__ __forceinline__ void fetch(const TileMeta& meta, int half, int left, uint4 (&r)[kLoads]) const {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int64_t at = meta.at[4 * half + 2 * x + (rs >> 4)];
            const bool there = at >= 0 && 64 * half + 32 * x + rs < left;
#pragma unroll
            for (int p = 0; p < kPanels; ++p) {
                r[x * kPanels + p] = make_uint4(0, 0, 0, 0);
                if (there) r[x * kPanels + p] = __ldcg(reinterpret_cast<const uint4*>(cache + at + 64 * p));
            }
        }
    }
    // NaN on V's side is written as 0 (0 * NaN would reach rows that do not see it), and tile j noted among the first
    // and last that hold any.
    __device__ __forceinline__ void put(uint8_t* base, bool v_side, const uint4 (&r)[kLoads], int j, int* nan_tiles) const {
        __half2 acc[2] = {__float2half2_rn(0.0f), __float2half2_rn(0.0f)};
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            uint32_t h[8];
            expand16(r[x], h);
            if (v_side) {
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 0 * NaN: NaN if any of them is
                    acc[k & 1] = __hfma2(*reinterpret_cast<const __half2*>(&h[k]), __float2half2_rn(0.0f), acc[k & 1]);
            }
            const int off = (x % kPanels) * (kToks * 128) + (x / kPanels) * (32 * 128);
            *reinterpret_cast<uint4*>(base + u0 + off) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(base + u1 + off) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        const __half2 a = __hadd2(acc[0], acc[1]);
        if (v_side && (__hisnan(__low2half(a)) || __hisnan(__high2half(a)))) {  // written again with 0 in NaN's place
            atomicMin(&nan_tiles[0], j);
            atomicMax(&nan_tiles[1], j);
#pragma unroll 1
            for (int x = 0; x < kLoads; ++x) {
                const int off = (x % kPanels) * (kToks * 128) + (x / kPanels) * (32 * 128);
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {
                    uint16_t* w = reinterpret_cast<uint16_t*>(base + (k < 8 ? u0 : u1) + off) + (k & 7);
                    if ((*w & 0x7FFFu) > 0x7C00u) *w = 0;
                }
            }
        }
    }
};

// The page warp: pages and scales of the tiles, up to kMetaRing ahead. j0: tiles that the CTA has taken before.
template <int D>
__device__ __forceinline__ bool page_ahead(const PromptParams& A, int seq, int head, int kv0, int kv_hi, int n, TileMeta* metas,
                                           uint64_t* meta_full, uint64_t* meta_empty, volatile int* abort, int j0 = 0) {
    const int lane = threadIdx.x & 31;
    auto page_of = [&](int j) {  // lanes 0-7: the page of each 16-token group
        const int tok = kv0 + kToks * j + 16 * lane;
        return lane < kGroups && j < n && tok < kv_hi ? page_id(A.B, seq, tok >> A.B.page_shift, A.err_flag) : -1;
    };
    int next = page_of(0);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const int pid = next, tok = kv0 + kToks * j + 16 * lane;
        next = page_of(j + 1);
        const int64_t ph = (int64_t)pid * A.kv_heads + head;
        float ks = 1.0f, vs = 1.0f;
        if (pid >= 0) {
            ks = __ldcg(A.k_scale + ph);
            vs = __ldcg(A.v_scale + ph);
        }
        const bool all = __all_sync(0xffffffffu, lane >= kGroups || pid >= 0 || tok >= kv_hi);
        const int slot = (j0 + j) % kMetaRing;
        if (!wait_all<true>(&meta_empty[slot], (((j0 + j) / kMetaRing) & 1) ^ 1, abort, A.wait_ns)) return false;
        TileMeta& m = metas[slot];
        if (lane < kGroups) {
            m.at[lane] = pid < 0 ? (int64_t)-1 : ((ph << A.B.page_shift) + (tok & ((1 << A.B.page_shift) - 1))) * D;
            m.ks[lane] = ks;
            m.ev[lane] = log2_scale(vs);
            m.inv[lane] = 1.0f / vs;
        }
        if (lane == 0) m.all_ok = all;
        warp_arrive(&meta_full[slot]);
    }
    return true;
}

// One side (K or V) of all tiles of an item, by a warpgroup: half a tile at a time, the other half's reads in flight.
// entry(j): tile j's place in the order in which the products take the slots; j0: tiles that the CTA has taken before.
template <int D, int kSlots, typename Entry>
__device__ __forceinline__ bool expand_side(const PromptParams& A, bool v_side, int toks, int n, Entry entry, uint8_t* s_kv,
                                            const TileMeta* metas, uint64_t* meta_full, uint64_t* meta_empty, uint64_t* full,
                                            uint64_t* empty, int* nan_tiles, volatile int* abort, int j0 = 0) {
    Loader<D> ld(v_side ? A.v_cache : A.k_cache, threadIdx.x & 127);
    uint4 ra[Loader<D>::kLoads], rb[Loader<D>::kLoads];
    if (n > 0) {
        if (!wait_all(&meta_full[j0 % kMetaRing], (j0 / kMetaRing) & 1, abort, A.wait_ns)) return false;
        ld.fetch(metas[j0 % kMetaRing], 0, toks, ra);
    }
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const int e = entry(j), slot = e % kSlots, m = (j0 + j) % kMetaRing;
        ld.fetch(metas[m], 1, toks - kToks * j, rb);
        warp_arrive(&meta_empty[m]);
        if (!wait_all(&empty[slot], ((e / kSlots) & 1) ^ 1, abort, A.wait_ns)) return false;
        uint8_t* base = s_kv + slot * (kToks * D * 2);
        ld.put(base, v_side, ra, j, nan_tiles);
        if (j + 1 < n) {
            const int next = j0 + j + 1;
            if (!wait_all(&meta_full[next % kMetaRing], (next / kMetaRing) & 1, abort, A.wait_ns)) return false;
            ld.fetch(metas[next % kMetaRing], 0, toks - kToks * (j + 1), ra);
        }
        ld.put(base + 64 * 128, v_side, rb, j, nan_tiles);
        fence_proxy_async_smem();
        mbar_arrive(&full[slot]);
    }
    return true;
}

// Largest x = c s + e of a row of S (tensor memory columns at ..): whole when the row sees every token.
__device__ __forceinline__ float row_max(uint32_t at, const TileMeta& meta, float crow, int t0, int lo, int hi, bool whole) {
    float top = -INFINITY;
    if (whole) {
#pragma unroll 1
        for (int q = 0; q < kToks / 32; ++q) {
            uint32_t v[32];
            tmem_ld32(at + 32 * q, v);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int g = 2 * q + h;
                float x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t* w = &v[16 * h + 4 * c];
                    x[c] = fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])),
                                 fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
                }
                top = fmaxf(top, fmaf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), crow * meta.ks[g], meta.ev[g]));
            }
        }
        return top;
    }
#pragma unroll 1
    for (int g = 0; g < kGroups; ++g) {
        uint32_t v[16];
        tmem_ld16(at + 16 * g, v);
        tmem_wait_ld();
        float x = -INFINITY;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const int tok = t0 + 16 * g + c;
            if (meta.at[g] >= 0 && tok >= lo && tok < hi) x = fmaxf(x, __uint_as_float(v[c]));
        }
        if (x > -INFINITY) top = fmaxf(top, fmaf(x, crow * meta.ks[g], meta.ev[g]));
    }
    return top;
}

constexpr float kTop = 15.0f;  // log2 of the largest P

// What x is taken from in the exponent of P, with references up to kNear and so with x - base in one rounding; further off
// than that x is rounded first, as its maximum was (x <= M, and base is rounded up), so that P stays below 2^16 still.
constexpr float kNear = 1048576.0f;
__device__ __forceinline__ float weight_base(float ref, float bits) { return __fadd_ru(ref, -bits); }
__device__ __forceinline__ bool all_near(float ref) { return __all_sync(0xffffffffu, fabsf(ref) < kNear) != 0; }

// P of one group's 16 tokens, packed to fp16 (and what that leaves times 2^11, packed to fp16: lo8, where wanted), and its
// sum. plain: the row sees them all, and its reference is near.
__device__ __forceinline__ float group_weights(const uint32_t* v, const TileMeta& meta, int g, float crow, float base, int t0,
                                               int lo, int hi, bool plain, uint32_t* hi8, uint32_t* lo8) {
    const float c = crow * meta.ks[g], e = plain ? meta.ev[g] - base : meta.ev[g];
    float2 p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        p[k] = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), make_float2(c, c), make_float2(e, e));
    if (!plain) {
        const int tok = t0 + 16 * g, from = meta.at[g] >= 0 ? lo - tok : 16, to = hi - tok;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            p[k] = add2(p[k], make_float2(-base, -base));
            if (2 * k < from || 2 * k >= to) p[k].x = -INFINITY;
            if (2 * k + 1 < from || 2 * k + 1 >= to) p[k].y = -INFINITY;
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = make_float2(ex2(p[k].x), ex2(p[k].y));
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const __half2 h = __floats2half2_rn(p[k].x, p[k].y);
        hi8[k] = h2_bits(h);
        if (lo8) {
            const float2 f = fma2(__half22float2(h), make_float2(-2048.0f, -2048.0f), mul2(p[k], make_float2(2048.0f, 2048.0f)));
            lo8[k] = h2_bits(__floats2half2_rn(f.x, f.y));
        }
    }
    const float2 sum = add2(add2(add2(p[0], p[1]), add2(p[2], p[3])), add2(add2(p[4], p[5]), add2(p[6], p[7])));
    return sum.x + sum.y;
}
// P = 2^(x - base) of a row in the place of its S, and the row's share of the denominator: 32 tokens' P take 16
// columns (one fp16 term), columns of S that have been read.
__device__ __forceinline__ float weights(uint32_t at, const TileMeta& meta, float crow, float base, int t0, int lo, int hi) {
    float l = 0.0f;
#pragma unroll 1
    for (int q = 0; q < kToks / 32; ++q) {
        uint32_t v[32], pk[16];
        tmem_ld32(at + 32 * q, v);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 2; ++h) l = fmaf(group_weights(&v[16 * h], meta, 2 * q + h, crow, base, t0, lo, hi, false, &pk[8 * h], nullptr),
                                             meta.inv[2 * q + h], l);
        tmem_st16(at + 16 * q, pk);
    }
    return l;
}
// The same in two fp16 terms: 32 tokens' P take the 32 columns of their S, 16 high, then 16 low. The next group's S
// is read before this one's P is written (over part of it).
__device__ __forceinline__ float weights2(uint32_t at, const TileMeta& meta, float crow, float base, int t0, int lo, int hi,
                                          bool plain) {
    float l = 0.0f;
    uint32_t v[2][16];
    tmem_ld16(at, v[0]);
    tmem_wait_ld();
    auto step = [&](int g, uint32_t (&now)[16], uint32_t (&next)[16], bool all) {
        uint32_t hi8[8], lo8[8];
        if (g + 1 < kGroups) tmem_ld16(at + 16 * (g + 1), next);
        l = fmaf(group_weights(now, meta, g, crow, base, t0, lo, hi, all, hi8, lo8), meta.inv[g], l);
        tmem_wait_ld();
        tmem_st8(at + 32 * (g >> 1) + 8 * (g & 1), hi8);
        tmem_st8(at + 32 * (g >> 1) + 8 * (g & 1) + 16, lo8);
    };
    if (plain) {
#pragma unroll 1
        for (int g = 0; g < kGroups; g += 2) {
            step(g, v[0], v[1], true);
            step(g + 1, v[1], v[0], true);
        }
    } else {
#pragma unroll 1
        for (int g = 0; g < kGroups; g += 2) {
            step(g, v[0], v[1], false);
            step(g + 1, v[1], v[0], false);
        }
    }
    return l;
}

// The same in one pass with the largest x - base, for a tile that the row sees whole, P left in registers (one
// term): S stays as it is until the caller knows that the reference held.
__device__ __forceinline__ float weights_and_max(uint32_t at, const TileMeta& meta, float crow, float base,
                                                 uint32_t (&pk)[2][32], float* top_out) {
    float l = 0.0f, top[2] = {-INFINITY, -INFINITY};
    uint32_t v[2][16];
    tmem_ld16(at, v[0]);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        tmem_wait_ld();
        if (g + 1 < kGroups) tmem_ld16(at + 16 * (g + 1), v[(g + 1) & 1]);
        const float c = crow * meta.ks[g], e = meta.ev[g] - base;
        float2 p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            p[k] = fma2(make_float2(__uint_as_float(v[g & 1][2 * k]), __uint_as_float(v[g & 1][2 * k + 1])), make_float2(c, c),
                        make_float2(e, e));
#pragma unroll
        for (int k = 0; k < 8; ++k) top[k % 2] = fmaxf(fmaxf(top[k % 2], p[k].x), p[k].y);
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = make_float2(ex2(p[k].x), ex2(p[k].y));
#pragma unroll
        for (int k = 0; k < 8; ++k) pk[g >> 2][8 * (g & 3) + k] = h2_bits(__floats2half2_rn(p[k].x, p[k].y));
        const float2 sum = add2(add2(add2(p[0], p[1]), add2(p[2], p[3])), add2(add2(p[4], p[5]), add2(p[6], p[7])));
        l = fmaf(sum.x + sum.y, meta.inv[g], l);
    }
    *top_out = fmaxf(top[0], top[1]);
    return l;
}

// Some V of the tokens [from, to] holds NaN (expanded as 0): dims [c0, c0 + N) of a row that sees tokens [lo, pos]
// are NaN where one of those is.
template <int D, int N>
__device__ __forceinline__ void mark_nan(const PromptParams& A, int seq, int head, int lo, int pos, int from, int to, int c0,
                                         float (&y)[N]) {
    lo = max(lo, from);
    pos = min(pos, to);
    int p = -1;
#pragma unroll 1
    for (int tok = lo; tok <= pos; ++tok) {
        if (tok == lo || (tok & 15) == 0) p = page_id(A.B, seq, tok >> A.B.page_shift, nullptr);
        if (p < 0) continue;
        const uint4* v = reinterpret_cast<const uint4*>(
            A.v_cache + ((((int64_t)p * A.kv_heads + head) << A.B.page_shift) + (tok & ((1 << A.B.page_shift) - 1))) * D + c0);
#pragma unroll
        for (int u = 0; u < N / 16; ++u) {
            const uint4 w = __ldcg(v + u);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (((x[k >> 2] >> (8 * (k & 3))) & 0x7Fu) == 0x7Fu) y[16 * u + k] = __int_as_float(0x7FC00000);
        }
    }
}

}  // namespace tc
}  // namespace q4k
