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

#include "q4k_attn_tc.cuh"

namespace q4k {
using namespace tc;
namespace {

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
