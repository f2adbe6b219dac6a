// q4k_attn_tc.cu -- attention over the paged 8-bit cache for many query rows per kv head (prompts), on the
// tensor cores.
//
// The mathematics of q4k_attn.cu: x_j = c (code_k . q) + e_j, P_j = 2^(x_j - M + B), out = sum P_j code_v,j /
// sum 2^(-e_j) P_j, with the codes of both sides exact in fp16, bf16 queries in one fp16 term and fp32
// queries (and their P) in two. P is 2^15 at most, fp16's largest power of two: B is 15, or 9 where M may be behind by
// 2^6 (bf16). So P_j keeps its 11 bits down to 2^-23 of the largest and 2^-34 of it below (bf16), its 22 bits down to
// 2^-29 and 2^-51 of it below (fp32, whose low term is held times 2^11).
//
// A CTA takes 128 (fp32) or 256 (bf16) query rows of one kv head (row r: token r / group, head r % group, so the
// heads of a group share each K and V tile) and walks over the tokens that some row sees, 128 at a time:
//   S = Q K^T   tcgen05.mma, Q and K from shared memory (K-major, 128-byte swizzle)
//   P in place of S in tensor memory, the A operand of
//   O = P V     V from shared memory as it lies in the cache, d contiguous (N-major)
// Roles by warp: softmax (thread = row), for fp32 the sums, expanding K, expanding V, issuing the products, and
// looking pages and scales up. Every wait is bounded; an abort flag lets all roles leave together. The
// loops are kept short: the roles share a scheduler and its instruction cache, and unrolled further they waited for
// instructions (the bf16 prompt below took 1863 us with the first, fully unrolled ones).
//
// Bound by the chain S, largest value, exponentials, P, product, which is serial within a row tile and which the two row
// tiles of a CTA do not cover: the tensor pipe is active 45% of the time and issue 49%. A 128 x 128 x 128 product
// takes 512 cycles of the tensor core, four a tile of fp32 rows. 8192 tokens, 32 / 8 heads, head_dim 128: bf16 518 us,
// 1061 TFLOP/s of the pairs that are seen (55% of the card's measured dense rate); fp32 1039 us, 529 TFLOP/s, with twice
// the products. Items are not cut along the tokens, so few of them leave SMs idle: 256 new tokens behind 131000 are 32 items
// (bf16) and take 1.9 ms.
#include <atomic>

#include "q4k_paged.cuh"
#include "q4k_sm100.cuh"
#include "q4k_sync.cuh"

namespace q4k {
using namespace sm100;
namespace {

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

// The block's item among two to 32 sequences (lane i holds the i-th): the items in falling order of the tokens that
// they walk over, in steps of 128, since the last ones to start decide when the kernel ends. A sequence's tiles
// that walk over L tokens or more are its last ones, so their number is a quotient, and L is found by bisection.
// (Sequence by sequence, six ragged chunks of fp32 took 178 us instead of 158.)
__device__ __forceinline__ void find_by_length(const PromptParams& A, int tile_rows, const SeqSpan& s, int tiles, int* item) {
    const int lane = threadIdx.x & 31, most = A.window > 0 ? A.window + tile_rows / A.group : 0x7FFFFFFF;
    auto count = [&](int step) {  // this sequence's items of at least 128 * step tokens
        const int tokens = 128 * step;
        if (step == 0) return tiles * A.kv_heads;
        if (tokens > s.len || tokens > most) return 0;
        const int before = max(tokens - 1 - (s.len - s.n), 0) * A.group / tile_rows;
        return max(tiles - before, 0) * A.kv_heads;
    };
    const int at = blockIdx.x;
    int lo = 0, hi = (__reduce_max_sync(0xffffffffu, tiles ? s.len : 0) >> 7) + 1;  // count(lo) > at >= count(hi)
    if ((int)__reduce_add_sync(0xffffffffu, count(0)) <= at) {
        if (lane == 0) item[0] = -1;
        return;
    }
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int)__reduce_add_sync(0xffffffffu, count(mid)) > at) lo = mid;
        else hi = mid;
    }
    const int above = count(hi), own = count(lo) - above;
    int inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    const int rest = at - (int)__reduce_add_sync(0xffffffffu, above) - (inc - own);
    if (rest >= 0 && rest < own) {  // one lane
        item[0] = lane;
        item[1] = tiles * A.kv_heads - above - 1 - rest;
        item[2] = s.start;
        item[3] = s.n;
        item[4] = s.len;
    }
}

// The block's item: sequence, row tile * kv_heads + kv head, its first row, new tokens and length; -1 past
// the last. Otherwise from the last row tile of the last sequence down.
__device__ __forceinline__ void find_item(const PromptParams& A, int tile_rows, int* item) {
    const int lane = threadIdx.x & 31;
    if (A.B.batch > 1 && A.B.batch <= 32) {
        SeqSpan s{0, 0, 0};
        int tiles = 0;
        if (lane < A.B.batch) {
            bool bad;
            s = seq_span(A.B, lane, &bad);
            if (bad) raise_flag(A.err_flag, Q4K_ERR_SEQ);
            const int rows = s.n * A.group;
            if (rows >= A.min_rows) tiles = (rows + tile_rows - 1) / tile_rows;
        }
        find_by_length(A, tile_rows, s, tiles, item);
        return;
    }
    int at = blockIdx.x;
    for (int top = A.B.batch; top > 0; top -= 32) {
        const int i = top - 1 - lane;  // lane 0: the last sequence
        SeqSpan s{0, 0, 0};
        int n = 0;
        if (i >= 0) {
            bool bad;
            s = seq_span(A.B, i, &bad);
            if (bad) raise_flag(A.err_flag, Q4K_ERR_SEQ);
            const int rows = s.n * A.group;
            if (rows >= A.min_rows) n = (rows + tile_rows - 1) / tile_rows * A.kv_heads;
        }
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, at < inc);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                item[0] = i;
                item[1] = n - 1 - (at - (inc - n));
                item[2] = s.start;
                item[3] = s.n;
                item[4] = s.len;
            }
            return;
        }
        at -= __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) item[0] = -1;
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

// The page warp: pages and scales of the tiles, up to kMetaRing ahead.
template <int D>
__device__ __forceinline__ bool page_ahead(const PromptParams& A, int seq, int head, int kv0, int kv_hi, int n, TileMeta* metas,
                                           uint64_t* meta_full, uint64_t* meta_empty, volatile int* abort) {
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
        if (!wait_all<true>(&meta_empty[j % kMetaRing], ((j / kMetaRing) & 1) ^ 1, abort, A.wait_ns)) return false;
        TileMeta& m = metas[j % kMetaRing];
        if (lane < kGroups) {
            m.at[lane] = pid < 0 ? (int64_t)-1 : ((ph << A.B.page_shift) + (tok & ((1 << A.B.page_shift) - 1))) * D;
            m.ks[lane] = ks;
            m.ev[lane] = log2_scale(vs);
            m.inv[lane] = 1.0f / vs;
        }
        if (lane == 0) m.all_ok = all;
        warp_arrive(&meta_full[j % kMetaRing]);
    }
    return true;
}

// One side (K or V) of all tiles of an item, by a warpgroup: half a tile at a time, the other half's reads in flight.
// entry(j): tile j's place in the order in which the products take the slots.
template <int D, int kSlots, typename Entry>
__device__ __forceinline__ bool expand_side(const PromptParams& A, bool v_side, int toks, int n, Entry entry, uint8_t* s_kv,
                                            const TileMeta* metas, uint64_t* meta_full, uint64_t* meta_empty, uint64_t* full,
                                            uint64_t* empty, int* nan_tiles, volatile int* abort) {
    Loader<D> ld(v_side ? A.v_cache : A.k_cache, threadIdx.x & 127);
    uint4 ra[Loader<D>::kLoads], rb[Loader<D>::kLoads];
    if (n > 0) {
        if (!wait_all(&meta_full[0], 0, abort, A.wait_ns)) return false;
        ld.fetch(metas[0], 0, toks, ra);
    }
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const int e = entry(j), slot = e % kSlots, m = j % kMetaRing;
        ld.fetch(metas[m], 1, toks - kToks * j, rb);
        warp_arrive(&meta_empty[m]);
        if (!wait_all(&empty[slot], ((e / kSlots) & 1) ^ 1, abort, A.wait_ns)) return false;
        uint8_t* base = s_kv + slot * (kToks * D * 2);
        ld.put(base, v_side, ra, j, nan_tiles);
        if (j + 1 < n) {
            if (!wait_all(&meta_full[(j + 1) % kMetaRing], ((j + 1) / kMetaRing) & 1, abort, A.wait_ns)) return false;
            ld.fetch(metas[(j + 1) % kMetaRing], 0, toks - kToks * (j + 1), ra);
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

// ---------------------------------------------------------------------------------------------------
// Both kernels: warps 0-7 softmax or sums, 8-11 expand K, 12-15 V, warp 16 issues the products, warp 17 looks the
// pages and scales up (18-19 idle).
constexpr int kThreads = 640;
constexpr int kKWarp = 8, kVWarp = 12, kMmaWarp = 16, kPageWarp = 17;
constexpr int kRegsAll = 5 * (65536 / kThreads / 8 * 8);  // what a launch gives a thread, times the warpgroups

// fp32 rows: 128 a CTA, queries and P in two fp16 terms. S and O have two tiles each in tensor memory, so that S of
// the next tokens is multiplied while the softmax of these is computed. O of each 128 tokens is a fresh
// accumulator that warps 4-7 add to fp32 sums in registers: the tensor core's own accumulation does not round to
// nearest, and the running maximum's correction costs nothing more there. They also find the maximum of the next S, while
// warps 0-3 make P of this one, the longest step. Order of the slots: K0, K1, V0, K2,
// V1, ..., V(n-1).
constexpr int kRegsSoftmax1 = 104, kRegsSums1 = 176, kRegsLoad1 = 72, kRegsCtrl1 = 56;
static_assert(kRegsSoftmax1 + kRegsSums1 + 2 * kRegsLoad1 + kRegsCtrl1 <= kRegsAll, "register split");

template <int D>
struct Layout1 {
    static constexpr int kTile = kToks * D * 2;  // a K or V tile, and one term of the queries
    static constexpr int kSlots = 4;             // at most 6: kMetaRing holds what is in flight
    static constexpr int kBytes = 1024 + 2 * kTile + kSlots * kTile;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const __grid_constant__ PromptParams A) {
    using L = Layout1<D>;
    constexpr uint32_t kColS = 0, kColO = 256;  // tensor memory: two S tiles, two O tiles
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* s_q = smem;
    uint8_t* s_kv = smem + 2 * L::kTile;
    __shared__ __align__(8) uint64_t full[L::kSlots], empty[L::kSlots], meta_full[kMetaRing], meta_empty[kMetaRing];
    __shared__ __align__(8) uint64_t s_full[2], max_full[2], p_full[2], o_full[2], fin, drain;
    __shared__ TileMeta s_meta[kMetaRing];
    __shared__ float s_c[kRows], s_ref[2][kRows], s_inv[kRows];
    __shared__ uint32_t s_tmem;
    __shared__ int s_item[5], s_nan[2];
    __shared__ volatile int s_abort;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5;
    if (warp == 0) find_item(A, kRows, s_item);
    if (tid == 32) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kMetaRing; ++i) {
            mbar_init(&meta_full[i], 1);
            mbar_init(&meta_empty[i], 16);  // the warps of the softmax, of the sums and of the loaders
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
            mbar_init(&max_full[i], 128);
        }
        mbar_init(&fin, 256);
        mbar_init(&drain, 1);
        fence_mbar_init();
        s_abort = 0;
        s_nan[0] = 0x7FFFFFFF;
        s_nan[1] = -1;
    }
    __syncthreads();
    const int seq = s_item[0];
    if (seq < 0) return;  // the whole CTA, before any allocation
    const int head = s_item[1] % A.kv_heads, tile = s_item[1] / A.kv_heads;
    const int start = s_item[2], rows = s_item[3] * A.group, first = s_item[4] - s_item[3];
    const int r0 = tile * kRows, last = min(rows, r0 + kRows) - 1;
    // positions: some row sees tokens in [kv_lo, kv_hi), every row those in [full_lo, full_hi)
    const int pf = first + r0 / A.group, pl = first + last / A.group;
    const int kv_hi = max(pl + 1, 0), full_hi = max(pf + 1, 0);
    const int kv_lo = A.window > 0 ? max(pf - A.window + 1, 0) : 0;
    const int full_lo = A.window > 0 ? max(pl - A.window + 1, 0) : 0;
    const int kv0 = kv_lo & ~15;
    const int n = (kv_hi - kv0 + kToks - 1) / kToks;  // tiles; 0: no row sees anything

    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    // queries: four threads a row, D/4 dims each, scaled by a power of two into fp16's range
    if (tid < 4 * kRows) {
        const int row = tid >> 2, part = tid & 3, r = r0 + row;
        const bool valid = r < rows;
        const float* p = static_cast<const float*>(A.q) + (int64_t)(start + (valid ? r / A.group : 0)) * A.q_stride +
                         (int64_t)(head * A.group + (valid ? r % A.group : 0)) * D + part * (D / 4);
        float x[D / 4];
        Vec<float>::load(p, x);
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) {
            if (!valid) x[i] = 0.0f;
            const float a = fabsf(x[i]);
            if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = amax > 0.0f ? min(max(134 - (int)(__float_as_uint(amax) >> 23), -120), 120) : 0;
        const float up = A.sign * exp2_int(e);
        if (part == 0) s_c[row] = A.scale_log2 * exp2_int(-e);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {  // 8 dims a unit
            const int unit = part * (D / 32) + u;
            uint8_t* dst = s_q + (unit >> 3) * (kRows * 128) + row * 128 + (((unit & 7) ^ (row & 7)) << 4);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[8 * u + 2 * i] * up, b = x[8 * u + 2 * i + 1] * up;
                const __half2 h = __floats2half2_rn(a, b);
                const float2 f = __half22float2(h);
                hi[i] = h2_bits(h);
                lo[i] = h2_bits(__floats2half2_rn(a - f.x, b - f.y));
            }
            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + L::kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(bar, parity, &s_abort, A.wait_ns); };
    // the place of tile j's K and V in the order of the slots
    auto k_entry = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto v_entry = [n](int j) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; };

    if (warp >= kMmaWarp) {
        regs_dec<kRegsCtrl1>();
        if (warp == kMmaWarp) {
            // ---------------- products, issued by one elected lane of the warp
            const uint32_t idesc_s = idesc_f16_f32(kRows, kToks);
            const uint32_t idesc_o = idesc_f16_f32(kRows, D) | kIdescBMnMajor;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t q_at = __shfl_sync(0xffffffffu, smem_u32(s_q), 0), kv_at = q_at + 2 * L::kTile;
            bool issued = false;
#pragma unroll 1
            for (int j = -1; j < n && ok && n > 0; ++j) {
                if (j + 1 < n) {
                    const int e = k_entry(j + 1), slot = e % L::kSlots;
                    ok = wait(&full[slot], (e / L::kSlots) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t b = desc_sw128_kmajor(kv_at + slot * L::kTile);
                    // the low term first, into small sums: the tensor core's additions truncate
#pragma unroll
                    for (int t = 1; t >= 0; --t) {
                        const uint64_t a = desc_sw128_kmajor(q_at + t * L::kTile);
#pragma unroll
                        for (int k = 0; k < D / 64; ++k)
                            mma_f16_ss_elect4(tm + kColS + ((j + 1) & 1) * kToks, a + ((k * kToks * 128) >> 4),
                                              b + ((k * kToks * 128) >> 4), 2, 2, idesc_s, 1 - t + k);
                    }
                    mma_commit_elect(&s_full[(j + 1) & 1]);
                    mma_commit_elect(&empty[slot]);
                    issued = true;
                }
                if (j < 0) continue;
                // P of these tokens; O of the tile two before has been taken (its reader found this one's maximum after)
                const int e = v_entry(j), slot = e % L::kSlots;
                ok = wait(&p_full[j & 1], (j >> 1) & 1) && wait(&full[slot], (e / L::kSlots) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t p = tm + kColS + (j & 1) * kToks, d = tm + kColO + (j & 1) * D;
                const uint64_t b = desc_sw128_mnmajor(kv_at + slot * L::kTile, kToks * 128);
                // 32 tokens' P in the 32 columns of their S: 16 of the high term, 16 of the low. The low one first; its
                // sums lose their 2^11 with the high term's first product. k steps 0, 2, 4, 6, then 1, 3, 5, 7: 32 columns apart.
                const uint64_t b1 = b + ((16 * 128) >> 4);
                mma_f16_ts_elect4(d, p + 16, b, 32, (32 * 128) >> 4, idesc_o, 0);
                mma_f16_ts_elect4(d, p + 24, b1, 32, (32 * 128) >> 4, idesc_o, 1);
                mma_f16_ts_elect4<11>(d, p, b, 32, (32 * 128) >> 4, idesc_o, 1);
                mma_f16_ts_elect4(d, p + 8, b1, 32, (32 * 128) >> 4, idesc_o, 1);
                mma_commit_elect(&o_full[j & 1]);
                mma_commit_elect(&empty[slot]);
            }
            if (issued) {  // whichever role gave up: outstanding products finish before tensor memory is freed
                volatile int never = 0;
                mma_commit_elect(&drain);
                mbar_wait(&drain, 0, &never);
            }
            __syncwarp();
        } else if (warp == kPageWarp) {
            ok = page_ahead<D>(A, seq, head, kv0, kv_hi, n, s_meta, meta_full, meta_empty, &s_abort);
        }
    } else if (warp >= kKWarp) {
        regs_dec<kRegsLoad1>();
        const bool v_side = warp >= kVWarp;
        ok = expand_side<D, L::kSlots>(A, v_side, kv_hi - kv0, n, [&](int j) { return v_side ? v_entry(j) : k_entry(j); }, s_kv,
                                       s_meta, meta_full, meta_empty, full, empty, s_nan, &s_abort);
        if (v_side) mbar_arrive(&fin);
    } else if (warp < 4) {
        // ---------------- softmax: thread = row = tensor memory lane
        regs_inc<kRegsSoftmax1>();
        const int r = r0 + tid;
        const bool valid = r < rows;
        const int pos = first + (valid ? r / A.group : 0);
        const int hi = valid ? pos + 1 : 0, lo = A.window > 0 ? max(pos - A.window + 1, 0) : 0;
        const float crow = s_c[tid];
        const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
        float ref = -INFINITY, l = 0.0f;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            const int b = j & 1;
            ok = wait(&max_full[b], (j >> 1) & 1);  // S and its scales, too
            if (!ok) break;
            tc_fence_after();
            const TileMeta& meta = s_meta[j % kMetaRing];
            const int t0 = kv0 + kToks * j;
            const bool whole = meta.all_ok && t0 >= full_lo && t0 + kToks <= full_hi;
            const float r_new = s_ref[b][tid];  // -inf while the row has seen nothing
            const float use = r_new == -INFINITY ? 0.0f : r_new;
            l *= ex2(ref - use);
            ref = r_new;
            const bool plain = all_near(use) && whole;
            l += weights2(tmem + lane_base + kColS + b * kToks, meta, crow, weight_base(use, kTop), t0, lo, hi, plain);
            warp_arrive(&meta_empty[j % kMetaRing]);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[b]);
        }
        s_inv[tid] = l == 0.0f ? 0.0f : 1.0f / l;  // 0: the row sees nothing
        mbar_arrive(&fin);
    } else {
        // ---------------- maxima and sums: thread = row
        regs_inc<kRegsSums1>();
        const int row = tid - 128, r = r0 + row;
        const bool valid = r < rows;
        const int pos = first + (valid ? r / A.group : 0);
        const int hi = valid ? pos + 1 : 0, lo = A.window > 0 ? max(pos - A.window + 1, 0) : 0;
        const float crow = s_c[row];
        const uint32_t lane_at = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        float m = -INFINITY, corr = 0.0f, corr_last = 0.0f;
        float2 acc[D / 2];
#pragma unroll
        for (int c = 0; c < D / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
#pragma unroll 1
        for (int j = 0; j <= n && n > 0; ++j) {
            if (j < n) {
                const int b = j & 1;
                ok = wait(&meta_full[j % kMetaRing], (j / kMetaRing) & 1) && wait(&s_full[b], (j >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const TileMeta& meta = s_meta[j % kMetaRing];
                const int t0 = kv0 + kToks * j;
                const bool whole = meta.all_ok && t0 >= full_lo && t0 + kToks <= full_hi;
                const float m_new = fmaxf(m, row_max(lane_at + kColS + b * kToks, meta, crow, t0, lo, hi, whole));
                corr_last = corr;
                corr = ex2(m - (m_new == -INFINITY ? 0.0f : m_new));
                m = m_new;
                s_ref[b][row] = m_new;
                warp_arrive(&meta_empty[j % kMetaRing]);
                tc_fence_before();
                mbar_arrive(&max_full[b]);
            } else {
                corr_last = corr;
            }
            if (j == 0) continue;
            ok = wait(&o_full[(j - 1) & 1], ((j - 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t at = lane_at + kColO + ((j - 1) & 1) * D;
            uint32_t v[2][16];
            tmem_ld16(at, v[0]);
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
                tmem_wait_ld();
                if (q + 1 < D / 16) tmem_ld16(at + 16 * (q + 1), v[(q + 1) & 1]);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    acc[8 * q + c] = fma2(acc[8 * q + c], make_float2(corr_last, corr_last),
                                          make_float2(__uint_as_float(v[q & 1][2 * c]), __uint_as_float(v[q & 1][2 * c + 1])));
            }
            tc_fence_before();
        }
        ok = ok && wait(&fin, 0);  // the denominators, and the loaders' report of NaN
        if (ok && valid) {
            const float inv = s_inv[row];
            float* o = static_cast<float*>(A.out) + (int64_t)(start + r / A.group) * A.out_stride +
                       (int64_t)(head * A.group + r % A.group) * D;
#pragma unroll
            for (int c = 0; c < D; c += 16) {
                float y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = (k & 1 ? acc[(c + k) / 2].y : acc[(c + k) / 2].x) * inv;  // sees nothing: 0 * 0
                if (s_nan[1] >= 0)
                    mark_nan<D, 16>(A, seq, head, lo, pos, kv0 + kToks * s_nan[0],
                                    kv0 + kToks * (s_nan[1] + 1) - 1, c, y);
                Vec<float>::store(o + c, y);
            }
        }
    }
    if (!ok) {
        s_abort = 1;
        raise_flag(A.err_flag, Q4K_ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// bf16 rows: 256 query rows a CTA, two tiles of 128 that share every K and V tile, so the cache is
// expanded to fp16 half as often, and one tile's softmax runs while the other's products do. The sums stay
// in tensor memory over all tokens (the tensor core adds each 16 tokens' product truncated, 2^-23 of the sum at most: 2^-10
// of it over 131072 tokens, a quarter of a bf16 step), scaled again only when a row's
// maximum has grown by more than 2^6 since its reference was taken: P then stays within fp16.
//
// Warps 0-3 and 4-7 are the softmax of a tile each (thread = row) and its store.
constexpr int kRegsSoftmax2 = 136, kRegsLoad2 = 72, kRegsCtrl2 = 64;
static_assert(2 * kRegsSoftmax2 + 2 * kRegsLoad2 + kRegsCtrl2 <= kRegsAll, "register split");
// log2 growth of a row's maximum before its sums are scaled again. What it grows by is taken from the bits of small weights;
// the bf16 prompt above takes 579 us with 4, 537 with 5, 517 with 6, 510 with 8.
constexpr float kSlack = 6.0f;

template <int D>
struct Layout2 {
    static constexpr int kTile = kToks * D * 2;            // a K or V tile, and the queries of a row tile
    static constexpr int kSlots = 4;
    static constexpr int kBytes = 1024 + 2 * kTile + kSlots * kTile;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt2_kernel(const __grid_constant__ PromptParams A) {
    using L = Layout2<D>;
    constexpr uint32_t kColS = 0, kColO = 256;  // tensor memory: S (then P) and O of both row tiles
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* s_q = smem;
    uint8_t* s_kv = smem + 2 * L::kTile;
    __shared__ __align__(8) uint64_t full[L::kSlots], empty[L::kSlots], meta_full[kMetaRing], meta_empty[kMetaRing];
    __shared__ __align__(8) uint64_t s_full[2], p_full[2], o_full[2], fin, drain;
    __shared__ TileMeta s_meta[kMetaRing];
    __shared__ float s_c[2 * kRows];
    __shared__ uint32_t s_tmem;
    __shared__ int s_item[5], s_nan[2];
    __shared__ volatile int s_abort;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5;
    if (warp == 0) find_item(A, 2 * kRows, s_item);
    if (tid == 32) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kMetaRing; ++i) {
            mbar_init(&meta_full[i], 1);
            mbar_init(&meta_empty[i], 16);  // the warps of both softmaxes and of the loaders
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
        }
        mbar_init(&fin, 128);
        mbar_init(&drain, 1);
        fence_mbar_init();
        s_abort = 0;
        s_nan[0] = 0x7FFFFFFF;
        s_nan[1] = -1;
    }
    __syncthreads();
    const int seq = s_item[0];
    if (seq < 0) return;  // the whole CTA, before any allocation
    const int head = s_item[1] % A.kv_heads, tile = s_item[1] / A.kv_heads;
    const int start = s_item[2], rows = s_item[3] * A.group, first = s_item[4] - s_item[3];
    const int r0 = tile * 2 * kRows, last = min(rows, r0 + 2 * kRows) - 1;
    // positions: some row sees tokens in [kv_lo, kv_hi)
    const int pf = first + r0 / A.group, pl = first + last / A.group;
    const int kv_hi = max(pl + 1, 0), kv_lo = A.window > 0 ? max(pf - A.window + 1, 0) : 0;
    const int kv0 = kv_lo & ~15;
    const int n = (kv_hi - kv0 + kToks - 1) / kToks;  // tiles; 0: no row sees anything

    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    // queries: two threads a row, D/2 dims each, scaled by a power of two into fp16's range (exact there)
    if (tid < 512) {
        const int row = tid >> 1, half = tid & 1, r = r0 + row;
        const bool valid = r < rows;
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(A.q) +
                                 (int64_t)(start + (valid ? r / A.group : 0)) * A.q_stride +
                                 (int64_t)(head * A.group + (valid ? r % A.group : 0)) * D + half * (D / 2);
        uint4 x[D / 16];
        uint32_t top = 0;  // largest finite magnitude's bits
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            x[i] = __ldcg(reinterpret_cast<const uint4*>(p) + i);
            if (!valid) x[i] = make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = w[k] & 0x7FFFu, b = (w[k] >> 16) & 0x7FFFu;
                if (a < 0x7F80u) top = max(top, a);
                if (b < 0x7F80u) top = max(top, b);
            }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const int e = top > 0 ? min(max(134 - (int)(top >> 7), -120), 120) : 0;
        const float up = A.sign * exp2_int(e);
        if (half == 0) s_c[row] = A.scale_log2 * exp2_int(-e);
        uint8_t* base = s_q + (row >> 7) * L::kTile + (row & 127) * 128;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {  // 8 dims a unit
            const int unit = half * (D / 16) + i;
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[k] = h2_bits(__floats2half2_rn(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up));
            *reinterpret_cast<uint4*>(base + (unit >> 3) * (kRows * 128) + (((unit & 7) ^ (row & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(bar, parity, &s_abort, A.wait_ns); };

    if (warp >= kMmaWarp) {
        regs_dec<kRegsCtrl2>();
        if (warp == kMmaWarp) {
            // ---------------- products, issued by one elected lane of the warp
            const uint32_t idesc_s = idesc_f16_f32(kRows, kToks);
            const uint32_t idesc_o = idesc_f16_f32(kRows, D) | kIdescBMnMajor;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t q_at = __shfl_sync(0xffffffffu, smem_u32(s_q), 0), kv_at = q_at + 2 * L::kTile;
            bool issued = false;
            // slot 2 j: K of tile j, slot 2 j + 1: V
#pragma unroll 1
            for (int j = -1; j < n && ok && n > 0; ++j) {
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    if (j >= 0) {
                        const int sv = 2 * j + 1;
                        ok = wait(&p_full[x], j & 1) && (x > 0 || wait(&full[sv % L::kSlots], (sv / L::kSlots) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t p = tm + kColS + x * kToks, d = tm + kColO + x * D;
                        const uint64_t b = desc_sw128_mnmajor(kv_at + sv % L::kSlots * L::kTile, kToks * 128);
                        mma_f16_ts_elect4(d, p, b, 8, (16 * 128) >> 4, idesc_o, j > 0);
                        mma_f16_ts_elect4(d, p + 32, b + ((64 * 128) >> 4), 8, (16 * 128) >> 4, idesc_o, 1);
                        if (x) mma_commit_elect(&empty[sv % L::kSlots]);
                        if (j == n - 1) mma_commit_elect(&o_full[x]);
                    }
                    if (j + 1 < n) {
                        const int sk = 2 * j + 2;
                        if (x == 0 && !(ok = wait(&full[sk % L::kSlots], (sk / L::kSlots) & 1))) break;
                        tc_fence_after();
                        const uint64_t a = desc_sw128_kmajor(q_at + x * L::kTile);
                        const uint64_t b = desc_sw128_kmajor(kv_at + sk % L::kSlots * L::kTile);
#pragma unroll
                        for (int k = 0; k < D / 64; ++k)
                            mma_f16_ss_elect4(tm + kColS + x * kToks, a + ((k * kToks * 128) >> 4), b + ((k * kToks * 128) >> 4), 2,
                                              2, idesc_s, k);
                        mma_commit_elect(&s_full[x]);
                        if (x) mma_commit_elect(&empty[sk % L::kSlots]);
                        issued = true;
                    }
                }
            }
            if (issued) {  // whichever role gave up: outstanding products finish before tensor memory is freed
                volatile int never = 0;
                mma_commit_elect(&drain);
                mbar_wait(&drain, 0, &never);
            }
            __syncwarp();
        } else if (warp == kPageWarp) {
            ok = page_ahead<D>(A, seq, head, kv0, kv_hi, n, s_meta, meta_full, meta_empty, &s_abort);
        }
    } else if (warp >= kKWarp) {
        regs_dec<kRegsLoad2>();
        const bool v_side = warp >= kVWarp;
        ok = expand_side<D, L::kSlots>(A, v_side, kv_hi - kv0, n, [&](int j) { return 2 * j + v_side; }, s_kv, s_meta, meta_full,
                                       meta_empty, full, empty, s_nan, &s_abort);
        if (v_side) mbar_arrive(&fin);
    } else {
        regs_inc<kRegsSoftmax2>();
        // ---------------- softmax: thread = row = tensor memory lane
        const int x = warp >> 2, row = tid & 127, r = r0 + x * kRows + row;
        const bool valid = r < rows;
        const int pos = first + (valid ? r / A.group : 0);
        const int hi = valid ? pos + 1 : 0, lo = A.window > 0 ? max(pos - A.window + 1, 0) : 0;
        // every row of the tile sees [full_lo, full_hi)
        const int t_last = min(rows, r0 + (x + 1) * kRows) - 1, t_first = min(r0 + x * kRows, t_last);
        const int full_hi = max(first + t_first / A.group + 1, 0);
        const int full_lo = A.window > 0 ? max(first + t_last / A.group - A.window + 1, 0) : 0;
        const float crow = s_c[x * kRows + row];
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t at = tmem + lane_base + kColS + x * kToks, o_at = tmem + lane_base + kColO + x * D;
        float ref = -INFINITY, l = 0.0f;  // the reference of P and of the sums
        bool near = false;                // all rows of the warp have one, and near
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            ok = wait(&meta_full[j % kMetaRing], (j / kMetaRing) & 1) && wait(&s_full[x], j & 1);
            if (!ok) break;
            tc_fence_after();
            const TileMeta& meta = s_meta[j % kMetaRing];
            const int t0 = kv0 + kToks * j;
            const bool whole = meta.all_ok && t0 >= full_lo && t0 + kToks <= full_hi;
            // P under the reference so far, in one pass, where every row sees the whole tile and no maximum outgrows
            // its reference; else the maximum first, a new reference, and the sums so far (all products
            // before this S are complete) scaled to it.
            bool done = false;
            if (whole && near) {
                uint32_t pk[2][32];
                float top;
                const float sum = weights_and_max(at, meta, crow, weight_base(ref, kTop - kSlack), pk, &top);
                if (!__any_sync(0xffffffffu, top > kTop)) {
                    l += sum;
                    tmem_st32(at, pk[0]);
                    tmem_st32(at + 32, pk[1]);
                    done = true;
                }
            }
            if (!done) {
                const float top = row_max(at, meta, crow, t0, lo, hi, whole);
                if (__any_sync(0xffffffffu, top - ref > kSlack)) {
                    const float m_new = fmaxf(ref, top);
                    const float corr = ex2(ref - (m_new == -INFINITY ? 0.0f : m_new));
                    ref = m_new;
                    near = all_near(ref);
                    l *= corr;
                    if (j > 0) {
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t v[32];
                            tmem_ld32(o_at + 32 * q, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * corr);
                            tmem_st32(o_at + 32 * q, v);
                        }
                    }
                }
                l += weights(at, meta, crow, weight_base(ref == -INFINITY ? 0.0f : ref, kTop - kSlack), t0, lo, hi);
            }
            warp_arrive(&meta_empty[j % kMetaRing]);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[x]);
        }
        ok = ok && wait(&fin, 0) && (n == 0 || wait(&o_full[x], 0));
        if (ok) {
            tc_fence_after();
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // 0: the row sees nothing
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(A.out) + (int64_t)(start + r / A.group) * A.out_stride +
                               (int64_t)(head * A.group + r % A.group) * D;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t v[32];
                float y[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = 0;
                if (n > 0) {
                    tmem_ld32(o_at + 32 * q, v);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) y[c] = inv == 0.0f ? 0.0f : __uint_as_float(v[c]) * inv;
                if (s_nan[1] >= 0 && valid)
                    mark_nan<D, 32>(A, seq, head, lo, pos, kv0 + kToks * s_nan[0], kv0 + kToks * (s_nan[1] + 1) - 1, 32 * q, y);
                if (valid) Vec<__nv_bfloat16>::store(o + 32 * q, y);
            }
        }
    }
    if (!ok) {
        s_abort = 1;
        raise_flag(A.err_flag, Q4K_ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <typename T, int D>
cudaError_t launch_typed(const PromptParams& P, cudaStream_t stream) {
    constexpr bool HL = sizeof(T) == 4;
    void (*kern)(PromptParams);
    int bytes, rows;
    if constexpr (HL) {
        kern = attn_prompt_kernel<D>;
        bytes = Layout1<D>::kBytes;
        rows = kRows;
    } else {
        kern = attn_prompt2_kernel<D>;
        bytes = Layout2<D>::kBytes;
        rows = 2 * kRows;
    }
    // every CTA holds all of its SM's tensor memory: enough shared memory that one fits
    const int smem = bytes < 144 * 1024 ? 144 * 1024 : bytes;
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        allowed[dev].store(true, std::memory_order_relaxed);
    }
    // an upper bound of the row tiles: a sequence's last one may be part filled
    const int64_t items = ((int64_t)P.B.m * P.group / rows + (P.B.m < P.B.batch ? P.B.m : P.B.batch)) * P.kv_heads;
    if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)items);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P);
}

}  // namespace

cudaError_t launch_attention_prompt(const PagedBatch& B, const void* q, int dtype, int64_t q_stride, int q_heads,
                                    int kv_heads, int head_dim, const uint8_t* k_cache, const uint8_t* v_cache,
                                    const float* k_scale, const float* v_scale, int min_rows, float scale, int window,
                                    void* out, int64_t out_stride, int* err_flag, cudaStream_t stream) {
    PromptParams P{};
    P.B = B; P.q = q; P.out = out; P.q_stride = q_stride; P.out_stride = out_stride;
    P.k_cache = k_cache; P.v_cache = v_cache; P.k_scale = k_scale; P.v_scale = v_scale;
    P.kv_heads = kv_heads; P.group = q_heads / kv_heads; P.window = window; P.min_rows = min_rows;
    P.scale_log2 = (scale < 0.0f ? -scale : scale) * 1.44269504088896340736f;
    P.sign = scale < 0.0f ? -1.0f : 1.0f;
    P.err_flag = err_flag;
    P.wait_ns = wait_limit_ns();
    if (dtype == Q4K_F32)
        return head_dim == 64 ? launch_typed<float, 64>(P, stream) : launch_typed<float, 128>(P, stream);
    return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(P, stream) : launch_typed<__nv_bfloat16, 128>(P, stream);
}

}  // namespace q4k
