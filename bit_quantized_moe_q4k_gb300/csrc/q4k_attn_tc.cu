// q4k_attn_tc.cu -- attention over the paged 8-bit cache for many query rows per kv head (prompts), on the
// tensor cores.
//
// The mathematics of q4k_attn.cu: x_j = c (code_k . q) + e_j, P_j = 2^(x_j - M + 7), out = sum P_j code_v,j /
// sum 2^(-e_j) P_j, with the codes of both sides exact in fp16, bf16 queries in one fp16 term and fp32
// queries (and their P) in two.
//
// A CTA takes 128 query rows of one kv head (row r: token r / group, head r % group, so the heads of a
// group share each K and V tile) and walks over the tokens that some row sees, 128 at a time:
//   S = Q K^T   tcgen05.mma, Q and K from shared memory (K-major, 128-byte swizzle)
//   P in place of S in tensor memory, the A operand of
//   O = P V     V from shared memory as it lies in the cache, d contiguous (N-major)
// S and O have two tiles each in tensor memory, so that S of the next tokens is multiplied while the
// softmax of these is computed. O of each 128 tokens is a fresh accumulator that is added to fp32 sums in
// registers: the tensor core's own accumulation does not round to nearest, and the running maximum's
// correction costs nothing more there.
//
// Roles: warps 0-3 softmax (thread = row), 4-7 the sums (thread = row) and the store, 8-11 read the
// cache and write fp16 tiles, warp 12 issues the products, warp 13 looks the pages and scales up (14-15
// idle). Every wait is bounded; an abort flag lets all roles leave together. The loops are kept
// short: four roles share a scheduler, and unrolled further they waited for instructions.
//
// Bound by shared memory and the tensor core together: a tile of 128 x 128 x 128 takes 512 cycles for
// each product, reads 96 KB of operands and writes 64 KB of converted K and V at 128 bytes a cycle.
#include "q4k_paged.cuh"
#include "q4k_sm100.cuh"
#include "q4k_sync.cuh"

namespace q4k {
using namespace sm100;
namespace {

constexpr int kRows = 128;   // query rows of a CTA
constexpr int kToks = 128;   // tokens of a tile
constexpr int kGroups = kToks / 16;
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 12, kPageWarp = 13;
// Registers a thread of each warpgroup after the split; their sum is four times what the launch gives.
constexpr int kRegsSoftmax = 152, kRegsSums = 184, kRegsLoad = 104, kRegsMma = 72;
static_assert(kRegsSoftmax + kRegsSums + kRegsLoad + kRegsMma <= 4 * (65536 / kThreads), "register split");
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

template <bool HL, int D>
struct Layout {
    static constexpr int kTerms = HL ? 2 : 1;
    static constexpr int kTile = kToks * D * 2;            // a K or V tile (and one term of Q)
    static constexpr int kSlots = HL ? 4 : 5;              // at most 6: kMetaRing holds what is in flight
    static constexpr int kQ = kTerms * kTile;
    static constexpr int kBytes = 1024 + kQ + kSlots * kTile;
};

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
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// 16 codes to 16 halves.
__device__ __forceinline__ void expand16(const uint4& c, uint32_t (&h)[8]) {
    e4m3x4_to_f16x4(c.x, &h[0], &h[1]);
    e4m3x4_to_f16x4(c.y, &h[2], &h[3]);
    e4m3x4_to_f16x4(c.z, &h[4], &h[5]);
    e4m3x4_to_f16x4(c.w, &h[6], &h[7]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const __grid_constant__ PromptParams A) {
    constexpr bool HL = sizeof(T) == 4;
    using L = Layout<HL, D>;
    constexpr uint32_t kColS = 0, kColO = 256;  // tensor memory: two S tiles, two O tiles
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* s_q = smem;
    uint8_t* s_kv = smem + L::kQ;
    __shared__ __align__(8) uint64_t full[L::kSlots], empty[L::kSlots], meta_full[kMetaRing], meta_empty[kMetaRing];
    __shared__ __align__(8) uint64_t s_full[2], p_full[2], o_full[2], o_empty[2], fin, drain;
    __shared__ TileMeta s_meta[kMetaRing];
    __shared__ float s_c[kRows], s_corr[2][kRows], s_inv[kRows];
    __shared__ uint32_t s_tmem;
    __shared__ int s_item[5];
    __shared__ volatile int s_abort;
    __shared__ volatile int s_nan;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // the item: blocks are taken from the last row tile down, the longest first
    if (warp == 0) {
        int at = blockIdx.x;
        bool found = false;
        for (int top = A.B.batch; top > 0 && !found; top -= 32) {
            const int i = top - 1 - lane;  // lane 0: the last sequence
            SeqSpan s{0, 0, 0};
            int n = 0;
            if (i >= 0) {
                bool bad;
                s = seq_span(A.B, i, &bad);
                if (bad) raise_flag(A.err_flag, Q4K_ERR_SEQ);
                const int rows = s.n * A.group;
                if (rows >= A.min_rows) n = (rows + kRows - 1) / kRows * A.kv_heads;
            }
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, at < inc);
            if (hit) {
                const int src = __ffs(hit) - 1;
                if (lane == src) {
                    s_item[0] = i;
                    s_item[1] = n - 1 - (at - (inc - n));  // row tile * kv_heads + kv head
                    s_item[2] = s.start;
                    s_item[3] = s.n;
                    s_item[4] = s.len;
                }
                found = true;
            }
            at -= __shfl_sync(0xffffffffu, inc, 31);
        }
        if (!found && lane == 0) s_item[0] = -1;
    }
    if (tid == 32) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kMetaRing; ++i) {
            mbar_init(&meta_full[i], 1);
            mbar_init(&meta_empty[i], 8);  // the warps of the softmax and of the loaders
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 128);
        }
        mbar_init(&fin, 256);
        mbar_init(&drain, 1);
        fence_mbar_init();
        s_abort = 0;
        s_nan = 0;
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
    // queries: two threads a row, D/2 dims each, scaled by a power of two into fp16's range
    if (tid < 256) {
        const int row = tid >> 1, half = tid & 1, r = r0 + row;
        const bool valid = r < rows;
        const T* p = static_cast<const T*>(A.q) + (int64_t)(start + (valid ? r / A.group : 0)) * A.q_stride +
                     (int64_t)(head * A.group + (valid ? r % A.group : 0)) * D + half * (D / 2);
        float x[D / 2];
        Vec<T>::load(p, x);
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 2; ++i) {
            if (!valid) x[i] = 0.0f;
            const float a = fabsf(x[i]);
            if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const int e = amax > 0.0f ? min(max(134 - (int)(__float_as_uint(amax) >> 23), -120), 120) : 0;
        const float up = A.sign * exp2_int(e);
        if (half == 0) s_c[row] = A.scale_log2 * exp2_int(-e);
#pragma unroll
        for (int u = 0; u < D / 16; ++u) {  // 8 dims a unit
            const int unit = half * (D / 16) + u;
            uint8_t* dst = s_q + (unit >> 3) * (kRows * 128) + row * 128 + (((unit & 7) ^ (row & 7)) << 4);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[8 * u + 2 * i] * up, b = x[8 * u + 2 * i + 1] * up;
                const __half2 h = __floats2half2_rn(a, b);
                hi[i] = h2_bits(h);
                if (HL) {
                    const float2 f = __half22float2(h);
                    lo[i] = h2_bits(__floats2half2_rn(a - f.x, b - f.y));
                }
            }
            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (HL) *reinterpret_cast<uint4*>(dst + L::kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    // a wait of a whole warp: its lanes go on, or give up, together
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_for(bar, parity, &s_abort, A.wait_ns)) != 0;
    };

    if (warp >= kLoadWarp && warp < kMmaWarp) {
        regs_dec<kRegsLoad>();
        // ---------------- cache to fp16 tiles. Order of the slots: K0, K1, V0, K2, V1, ..., V(n-1). A thread
        // reads 16 codes of rows 32 x + rs, in each 64-dim panel, and writes them as two 16-byte units of the
        // panel's 128-byte rows; the eight threads of a store's phase hold two rows of different parity,
        // so their units lie on different banks.
        constexpr int kPanels = D / 64, kLoads = 4 * kPanels;
        const int i = tid - 32 * kLoadWarp, rs = i >> 2, c = i & 3;
        const uint8_t* k_at = A.k_cache + (rs & 15) * D + 16 * c;
        const uint8_t* v_at = A.v_cache + (rs & 15) * D + 16 * c;
        auto fetch = [&](const uint8_t* cache, int j, uint4 (&r)[kLoads]) {
            const int left = kv_hi - (kv0 + kToks * j);  // tokens of the tile that are there
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int64_t at = s_meta[j % kMetaRing].at[2 * x + (rs >> 4)];
                const bool there = at >= 0 && 32 * x + rs < left;
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    r[x * kPanels + p] = make_uint4(0, 0, 0, 0);
                    if (there) r[x * kPanels + p] = __ldcg(reinterpret_cast<const uint4*>(cache + at + 64 * p));
                }
            }
        };
        int slot = 0, uses = 0;
        bool nan = false;
        uint8_t* const dst = s_kv + rs * 128 + (((2 * c) ^ (rs & 7)) << 4);
        auto put = [&](bool v_side, const uint4 (&r)[kLoads]) {
            if (!wait(&empty[slot], (uses & 1) ^ 1)) return false;
            uint8_t* base = dst + slot * L::kTile;
            uint8_t* base1 = s_kv + slot * L::kTile + rs * 128 + (((2 * c + 1) ^ (rs & 7)) << 4);
            __half2 acc[2] = {__float2half2_rn(0.0f), __float2half2_rn(0.0f)};
#pragma unroll
            for (int x = 0; x < kLoads; ++x) {
                uint32_t h[8];
                expand16(r[x], h);
                if (v_side) {  // 0 * NaN: NaN if any of them is
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        acc[k & 1] = __hfma2(*reinterpret_cast<const __half2*>(&h[k]), __float2half2_rn(0.0f), acc[k & 1]);
                }
                const int off = (x % kPanels) * (kToks * 128) + (x / kPanels) * (32 * 128);
                *reinterpret_cast<uint4*>(base + off) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(base1 + off) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            if (v_side) {
                const __half2 a = __hadd2(acc[0], acc[1]);
                if (__hisnan(__low2half(a)) || __hisnan(__high2half(a))) {  // written again with 0 in NaN's place
                    nan = true;
#pragma unroll 1
                    for (int x = 0; x < kLoads; ++x) {
                        const int off = (x % kPanels) * (kToks * 128) + (x / kPanels) * (32 * 128);
#pragma unroll 1
                        for (int k = 0; k < 16; ++k) {
                            uint16_t* w = reinterpret_cast<uint16_t*>((k < 8 ? base : base1) + off) + (k & 7);
                            if ((*w & 0x7FFFu) > 0x7C00u) *w = 0;
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&full[slot]);
            if (++slot == L::kSlots) { slot = 0; ++uses; }
            return true;
        };
        uint4 ra[kLoads], rb[kLoads];  // K of tile j + 1, V of tile j
#pragma unroll 1
        for (int j = -2; j < n && ok && n > 0; ++j) {
            if (j + 1 >= 0 && j + 1 < n) ok = put(false, ra);
            if (ok && j + 2 < n) {
                ok = wait(&meta_full[(j + 2) % kMetaRing], ((j + 2) / kMetaRing) & 1);
                if (ok) fetch(k_at, j + 2, ra);
            }
            if (ok && j >= 0) ok = put(true, rb);
            if (ok && j + 1 >= 0 && j + 1 < n) {
                fetch(v_at, j + 1, rb);
                if (lane == 0) mbar_arrive(&meta_empty[(j + 1) % kMetaRing]);
            }
        }
        if (nan) s_nan = 1;
        mbar_arrive(&fin);
    } else if (warp >= kMmaWarp) {
        regs_dec<kRegsMma>();
        if (warp == kMmaWarp) {
        // ---------------- products, issued by one elected lane of the warp
        const uint32_t idesc_s = idesc_f16_f32(kRows, kToks);
        const uint32_t idesc_o = idesc_f16_f32(kRows, D) | kIdescBMnMajor;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t q_at = __shfl_sync(0xffffffffu, smem_u32(s_q), 0), kv_at = q_at + L::kQ;
        int slot = 0, uses = 0;
        bool issued = false;
        auto next_slot = [&]() { if (++slot == L::kSlots) { slot = 0; ++uses; } };
        auto scores = [&](int j) {
            if (!wait(&full[slot], uses & 1)) return false;
            tc_fence_after();
            const uint32_t d = tm + kColS + (j & 1) * kToks;
            const uint64_t b = desc_sw128_kmajor(kv_at + slot * L::kTile);
#pragma unroll
            for (int t = 0; t < L::kTerms; ++t) {
                const uint64_t a = desc_sw128_kmajor(q_at + t * L::kTile);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * (kToks * 128) + (k & 3) * 32) >> 4;
                    mma_f16_ss_elect(d, a + off, b + off, idesc_s, t > 0 || k > 0);
                }
            }
            mma_commit_elect(&s_full[j & 1]);
            mma_commit_elect(&empty[slot]);
            issued = true;
            next_slot();
            return true;
        };
#pragma unroll 1
        for (int j = -1; j < n && ok; ++j) {
            if (j + 1 < n && !(ok = scores(j + 1))) break;
            if (j < 0) continue;
            // P of these tokens (o_empty of the tile two before is implied: the softmax waited for it)
            ok = wait(&p_full[j & 1], (j >> 1) & 1) && wait(&full[slot], uses & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t p = tm + kColS + (j & 1) * kToks, d = tm + kColO + (j & 1) * D;
            const uint64_t b = desc_sw128_mnmajor(kv_at + slot * L::kTile, kToks * 128);
#pragma unroll
            for (int t = 0; t < L::kTerms; ++t)
#pragma unroll
                for (int k = 0; k < kToks / 16; ++k) {
                    const uint32_t a = HL ? p + 32 * (k >> 1) + 8 * (k & 1) + 16 * t : p + 8 * k;
                    mma_f16_ts_elect(d, a, b + ((k * 16 * 128) >> 4), idesc_o, t > 0 || k > 0);
                }
            mma_commit_elect(&o_full[j & 1]);
            mma_commit_elect(&empty[slot]);
            next_slot();
        }
        if (!ok && issued) {  // outstanding products finish before tensor memory is freed
            volatile int never = 0;
            mma_commit_elect(&drain);
            mbar_wait(&drain, 0, &never);
        }
        __syncwarp();
        } else if (warp == kPageWarp) {
            // ---------------- pages and scales, up to kMetaRing tiles ahead
            auto page_of = [&](int j) {  // lanes 0-7: the page of each 16-token group
                const int tok = kv0 + kToks * j + 16 * lane;
                return lane < kGroups && j < n && tok < kv_hi ? page_id(A.B, seq, tok >> A.B.page_shift, A.err_flag) : -1;
            };
            int next = page_of(0);
#pragma unroll 1
            for (int j = 0; j < n && ok; ++j) {
                const int pid = next, tok = kv0 + kToks * j + 16 * lane;
                next = page_of(j + 1);
                const int64_t ph = (int64_t)pid * A.kv_heads + head;
                float ks = 1.0f, vs = 1.0f;
                if (pid >= 0) {
                    ks = __ldcg(A.k_scale + ph);
                    vs = __ldcg(A.v_scale + ph);
                }
                const bool all = __all_sync(0xffffffffu, lane >= kGroups || pid >= 0 || tok >= kv_hi);
                ok = wait(&meta_empty[j % kMetaRing], ((j / kMetaRing) & 1) ^ 1);
                if (!ok) break;
                TileMeta& m = s_meta[j % kMetaRing];
                if (lane < kGroups) {
                    m.at[lane] = pid < 0 ? (int64_t)-1 : ((ph << A.B.page_shift) + (tok & ((1 << A.B.page_shift) - 1))) * D;
                    m.ks[lane] = ks;
                    m.ev[lane] = log2_scale(vs);
                    m.inv[lane] = 1.0f / vs;
                }
                if (lane == 0) m.all_ok = all;
                __syncwarp();
                if (lane == 0) mbar_arrive(&meta_full[j % kMetaRing]);
            }
        }
    } else if (warp < 4) {
        regs_inc<kRegsSoftmax>();
        // ---------------- softmax: thread = row = tensor memory lane
        const int r = r0 + tid;
        const bool valid = r < rows;
        const int pos = first + (valid ? r / A.group : 0);
        const int hi = valid ? pos + 1 : 0, lo = A.window > 0 ? max(pos - A.window + 1, 0) : 0;
        const float crow = s_c[tid];
        const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
        float m = -INFINITY, l = 0.0f;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            const int b = j & 1;
            ok = wait(&meta_full[j % kMetaRing], (j / kMetaRing) & 1) && wait(&s_full[b], (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const TileMeta& meta = s_meta[j % kMetaRing];
            const int t0 = kv0 + kToks * j;
            const bool whole = meta.all_ok && t0 >= full_lo && t0 + kToks <= full_hi;
            const uint32_t at = tmem + lane_base + kColS + b * kToks;
            float top = -INFINITY;
            if (whole) {
#pragma unroll 1
                for (int q = 0; q < kToks / 32; q += 2) {
                    uint32_t v[2][32];
                    tmem_ld32(at + 32 * q, v[0]);
                    tmem_ld32(at + 32 * q + 32, v[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int g = 2 * q + h;
                        float x[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t* w = &v[h >> 1][16 * (h & 1) + 4 * c];
                            x[c] = fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])),
                                         fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
                        }
                        top = fmaxf(top, fmaf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), crow * meta.ks[g], meta.ev[g]));
                    }
                }
            } else {
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
            }
            const float m_new = fmaxf(m, top), m_use = m_new == -INFINITY ? 0.0f : m_new;
            const float corr = ex2(m - m_use);
            m = m_new;
            l *= corr;
            // the sums have taken the tile two before this one
            if (j >= 2) ok = wait(&o_empty[b], ((j >> 1) - 1) & 1);
            if (!ok) break;
            s_corr[b][tid] = corr;
            // P over columns of S that have been read. One term: 8 columns for 16 tokens, packed; two: hi
            // and lo of 32 tokens in the 32 columns of their S.
#pragma unroll 1
            for (int q0 = 0; q0 < kToks / 32; q0 += 2) {
                uint32_t v[2][32], pk[32];
                tmem_ld32(at + 32 * q0, v[0]);
                tmem_wait_ld();
                tmem_ld32(at + 32 * q0 + 32, v[1]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (q) tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int g = 2 * (q0 + q) + h;
                        const float c = crow * meta.ks[g], e = meta.ev[g] - (m_use - 7.0f);
                        float2 p[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t* w = &v[q][16 * h + 2 * k];
                            p[k] = fma2(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), make_float2(c, c), make_float2(e, e));
                        }
                        if (!whole) {
                            const int tok = t0 + 16 * g, from = meta.at[g] >= 0 ? lo - tok : 16, to = hi - tok;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                if (2 * k < from || 2 * k >= to) p[k].x = -INFINITY;
                                if (2 * k + 1 < from || 2 * k + 1 >= to) p[k].y = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) p[k] = make_float2(ex2(p[k].x), ex2(p[k].y));
                        const float2 sum = add2(add2(add2(p[0], p[1]), add2(p[2], p[3])), add2(add2(p[4], p[5]), add2(p[6], p[7])));
                        l = fmaf(sum.x + sum.y, meta.inv[g], l);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const __half2 hh = __floats2half2_rn(p[k].x, p[k].y);
                            if constexpr (HL) {
                                const float2 f = __half22float2(hh);
                                pk[8 * h + k] = h2_bits(hh);
                                pk[16 + 8 * h + k] = h2_bits(__floats2half2_rn(p[k].x - f.x, p[k].y - f.y));
                            } else {
                                pk[16 * q + 8 * h + k] = h2_bits(hh);
                            }
                        }
                    }
                    if (HL) tmem_st32(at + 32 * (q0 + q), pk);
                    else if (q) tmem_st32(at + 16 * q0, pk);
                }
            }
            if (lane == 0) mbar_arrive(&meta_empty[j % kMetaRing]);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[b]);
        }
        s_inv[tid] = m == -INFINITY ? 0.0f : 1.0f / l;
        mbar_arrive(&fin);
    } else {
        regs_inc<kRegsSums>();
        // ---------------- sums: thread = row
        const int row = tid - 128, r = r0 + row;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        float2 acc[D / 2];
#pragma unroll
        for (int c = 0; c < D / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            const int b = j & 1;
            ok = wait(&p_full[b], (j >> 1) & 1) && wait(&o_full[b], (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const float corr = s_corr[b][row];
            const uint32_t at = tmem + lane_base + kColO + b * D;
            uint32_t v[2][16];
            tmem_ld16(at, v[0]);
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
                tmem_wait_ld();
                if (q + 1 < D / 16) tmem_ld16(at + 16 * (q + 1), v[(q + 1) & 1]);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    acc[8 * q + c] = fma2(acc[8 * q + c], make_float2(corr, corr),
                                          make_float2(__uint_as_float(v[q & 1][2 * c]), __uint_as_float(v[q & 1][2 * c + 1])));
            }
            tc_fence_before();
            mbar_arrive(&o_empty[b]);
        }
        ok = ok && wait(&fin, 0);  // the denominators, and the loaders' report of NaN
        if (ok && s_nan && r < rows) {
            // some V holds NaN (written as 0 above): the dims of the rows that see it are NaN
            const int pos = first + r / A.group;
            for (int tok = A.window > 0 ? max(pos - A.window + 1, 0) : 0; tok <= pos; ++tok) {
                const int p = page_id(A.B, seq, tok >> A.B.page_shift, nullptr);
                if (p < 0) continue;
                const uint4* v = reinterpret_cast<const uint4*>(
                    A.v_cache + ((((int64_t)p * A.kv_heads + head) << A.B.page_shift) + (tok & ((1 << A.B.page_shift) - 1))) * D);
#pragma unroll
                for (int u = 0; u < D / 16; ++u) {
                    const uint4 w = __ldcg(v + u);
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (((x[k >> 2] >> (8 * (k & 3))) & 0x7Fu) == 0x7Fu)
                            (k & 1 ? acc[8 * u + k / 2].y : acc[8 * u + k / 2].x) = __int_as_float(0x7FC00000);
                }
            }
        }
        if (ok && r < rows) {
            const float inv = s_inv[row];
            T* o = static_cast<T*>(A.out) + (int64_t)(start + r / A.group) * A.out_stride +
                   (int64_t)(head * A.group + r % A.group) * D;
#pragma unroll
            for (int c = 0; c < D; c += 8) {
                float y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float x = k & 1 ? acc[(c + k) / 2].y : acc[(c + k) / 2].x;
                    y[k] = x * inv;  // a row that sees nothing: 0 * 0
                }
                Vec<T>::store(o + c, y);
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
    // every CTA holds all of its SM's tensor memory: enough shared memory that one fits
    const int smem = Layout<HL, D>::kBytes < 144 * 1024 ? 144 * 1024 : Layout<HL, D>::kBytes;
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev]) {
        e = cudaFuncSetAttribute(attn_prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        set[dev] = true;
    }
    // an upper bound of the row tiles: a sequence's last one may be part filled
    const int64_t items = ((int64_t)P.B.m * P.group / kRows + (P.B.m < P.B.batch ? P.B.m : P.B.batch)) * P.kv_heads;
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
    return cudaLaunchKernelEx(&cfg, attn_prompt_kernel<T, D>, P);
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
