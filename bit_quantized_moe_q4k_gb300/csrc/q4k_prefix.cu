// q4k_prefix.cu -- attention over prefixes that the sequences of a group share, on the tensor cores: the rows of all of a group's
// sequences against one reading of the prefix.
//
//   out_r = (sum over shared j + sum over own j) P_j v_j / (the same of P_j),
// a sum of two parts that are each relative to a reference of their own, 2^(x - M), and joined by 2^(M_part - M).
// The shared part is made here, the sequences' own one by q4k_attn.cu, which joins them as it stores.
//
// prefix_plan_kernel lays the work out (q4k_prefix.cuh): one CTA, since it has to see every group before it can cut the line.
// prefix_kernel<D> (fp32 rows, 128 a row tile) and prefix2_kernel<D> (bf16, 256) then are the prompt kernels of
// q4k_attn_tc.cu without the diagonal: the same roles and the same tiles, but a CTA walks over its piece of the line, item after
// item, and leaves sums, references and denominators in fp32. No row sees less than the whole shared part unless there is a
// window, so nearly every tile is of the kind that is multiplied whole.
#include <atomic>

#include "q4k_attn_tc.cuh"
#include "q4k_prefix.cuh"

namespace q4k {
using namespace tc;
namespace {

// ---- the plan -----------------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 512;

struct PlanParams {
    PagedBatch B;
    const int32_t *group_start, *prefix_lens;
    PrefixPlan plan;
    int kv_heads, rep, window, max_rows;
    int* err_flag;
};

__device__ __forceinline__ int64_t block_exclusive(int64_t v, int64_t* total, int64_t* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    const int64_t x = lane < kPlanThreads / 32 ? s_warp[lane] : 0;
    int64_t before = lane < warp ? x : 0, all = x;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    __syncthreads();
    *total = all;
    return before + inc - v;
}

// Piece c of `ctas` begins at unit c * units / ctas.
__device__ __forceinline__ int64_t cut(int64_t units, int ctas, int64_t c) { return units * c / ctas; }
__device__ __forceinline__ int piece_of(int64_t units, int ctas, int64_t u) {  // the last c with cut(c) <= u
    return (int)(((u + 1) * ctas - 1) / units);
}

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ PlanParams A) {
    __shared__ int64_t s_warp[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int groups = A.plan.groups, batch = A.B.batch, shift = A.B.page_shift;
    // Starts that do not rise would let groups share rows: then nothing is shared.
    bool bad = false;
    for (int i = tid; i < batch; i += kPlanThreads) {
        const int a = __ldcg(A.B.q_start + i), b = __ldcg(A.B.q_start + i + 1);
        if (a < 0 || b < a || b > A.B.m) bad = true;
        A.plan.seq[i] = make_int2(-1, 0);
    }
    for (int g = tid; g < groups; g += kPlanThreads) {
        const int a = __ldcg(A.group_start + g), b = __ldcg(A.group_start + g + 1), p = __ldcg(A.prefix_lens + g);
        if (a < 0 || b < a || b > batch) bad = true;
        if (p < 0 || p > (A.B.max_pages << shift)) raise_flag(A.err_flag, Q4K_ERR_SEQ);
    }
    if (bad) raise_flag(A.err_flag, Q4K_ERR_SEQ);
    const bool none = __syncthreads_or(bad) != 0;  // the sequences' entries are written, too

    for (int g = warp; g < groups; g += kPlanThreads / 32) {
        PrefixGroup G{};
        if (!none) {
            const int a = __ldcg(A.group_start + g), b = __ldcg(A.group_start + g + 1);
            const int prefix = min(max(__ldcg(A.prefix_lens + g), 0), A.B.max_pages << shift);
            int least = 0x7FFFFFFF, most = -1, live = 0, rows = 0;
            for (int i = a + lane; i < b; i += 32) {
                bool odd;
                const SeqSpan s = seq_span(A.B, i, &odd);
                if (s.n == 0) continue;
                least = min(least, s.len - s.n);
                most = max(most, s.len - 1);
                rows = max(rows, s.n);
                ++live;
            }
            least = __reduce_min_sync(0xffffffffu, least);
            most = __reduce_max_sync(0xffffffffu, most);
            rows = __reduce_max_sync(0xffffffffu, rows);
            live = __reduce_add_sync(0xffffffffu, live);
            G.leader = a;
            if (live > 1 && (int64_t)rows * A.rep <= A.max_rows) {
                G.row0 = __ldcg(A.B.q_start + a);
                G.n = __ldcg(A.B.q_start + b) - G.row0;
                G.from = min(prefix, max(least, 0)) >> shift << shift;
                G.lo = A.window > 0 ? max(least - A.window + 1, 0) & ~15 : 0;
                G.full_lo = A.window > 0 ? max(most - A.window + 1, 0) : 0;
                if (G.from > G.lo) {
                    G.tiles = (G.from - G.lo + kToks - 1) / kToks;
                    G.rows = (int)(((int64_t)G.n * A.rep + A.plan.tile_rows - 1) / A.plan.tile_rows);
                    for (int i = a + lane; i < b; i += 32) {
                        A.plan.seq[i] = make_int2(g, G.from);
                        if (A.window > 0) {
                            bool odd;
                            const SeqSpan s = seq_span(A.B, i, &odd);
                            for (int t = 0; t < s.n; ++t) A.plan.pos[s.start + t] = s.len - s.n + t;
                        }
                    }
                }
            }
        }
        if (lane == 0) A.plan.group[g] = G;
    }
    __syncthreads();
    // places on the line of work, of each thread's run of groups
    const int per = (groups + kPlanThreads - 1) / kPlanThreads, lo = min(tid * per, groups), hi = min(lo + per, groups);
    int64_t items = 0, units = 0, all_items, all_units;
    for (int g = lo; g < hi; ++g) {
        const int64_t n = (int64_t)A.plan.group[g].rows * A.kv_heads;
        items += n;
        units += n * A.plan.group[g].tiles;
    }
    items = block_exclusive(items, &all_items, s_warp);
    units = block_exclusive(units, &all_units, s_warp);
    for (int g = lo; g < hi; ++g) {
        PrefixGroup* G = A.plan.group + g;
        const int64_t n = (int64_t)G->rows * A.kv_heads;
        G->item0 = items;
        G->unit0 = units;
        items += n;
        units += n * G->tiles;
    }
    all_items = min(all_items, A.plan.items);
    const int ctas = (int)min(all_units, (int64_t)kPrefixCtas);
    if (tid == 0) *A.plan.head = PrefixHead{all_units, all_items, ctas, 0};
    __syncthreads();
    for (int64_t i = tid; i < all_items; i += kPlanThreads) {
        int a = 0, b = groups;  // the last group that begins at or before item i
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (A.plan.group[mid].item0 <= i) a = mid;
            else b = mid;
        }
        const PrefixGroup& G = A.plan.group[a];
        const int64_t u = G.unit0 + (i - G.item0) * G.tiles;
        const int c0 = piece_of(all_units, ctas, u), c1 = piece_of(all_units, ctas, u + G.tiles - 1);
        A.plan.piece[i] = make_int2((int)(c0 + i), c1 - c0 + 1);
    }
}

// ---- the shared part ----------------------------------------------------------------------------------------------
struct PrefixParams : PromptParams {  // window: the attention's; out, out_stride, min_rows: not used
    PrefixPlan plan;
};

// What a CTA does next: an item's units, or nothing (n 0).
struct Segment {
    int n;                    // units (tiles of 128 tokens)
    int leader, head;         // whose pages, which kv head
    int row0, r0, rows;       // the group's first row of the inputs; the row tile's first query row; the group's query rows
    int kv0, kv_hi, full_lo;  // tokens
    int slot;
};
// The warp finds the segment at unit s_u[0] of piece c, which ends at s_u[1], and goes past it. None once a role has given up.
__device__ __forceinline__ void find_segment(const PrefixParams& A, int c, int64_t* s_u, volatile int* abort, Segment* out) {
    const int lane = threadIdx.x & 31;
    const int64_t u = s_u[0], end = s_u[1];
    __syncwarp();
    if (u >= end || *abort) {
        if (lane == 0) out->n = 0;
        return;
    }
    int lo = 0, hi = A.plan.groups - 1;  // the last group that begins at or before u (one without units begins where the next does)
    while (hi - lo >= 32) {
        const int step = (hi - lo) / 32 + 1, i = lo + lane * step;
        const unsigned hit = __ballot_sync(0xffffffffu, i <= hi && __ldcg(&A.plan.group[i].unit0) <= u);
        lo += (31 - __clz(hit)) * step;
        hi = min(hi, lo + step - 1);
    }
    const unsigned hit = __ballot_sync(0xffffffffu, lo + lane <= hi && __ldcg(&A.plan.group[lo + lane].unit0) <= u);
    lo += 31 - __clz(hit);
    if (lane) return;
    const int4* p = reinterpret_cast<const int4*>(A.plan.group + lo);
    const int4 f[3] = {__ldcg(p), __ldcg(p + 1), __ldcg(p + 2)};
    PrefixGroup G;
    memcpy(&G, f, sizeof G);
    // Two calls at once on one workspace write over each other's plans. Nothing of one is believed as far as addresses go.
    G.tiles = min(max(G.tiles, 1), (A.B.max_pages << A.B.page_shift) / kToks + 1);
    G.leader = min(max(G.leader, 0), A.B.batch - 1);
    G.from = min(max(G.from, 0), A.B.max_pages << A.B.page_shift);
    G.lo = min(max(G.lo, 0), G.from) & ~15;
    G.row0 = min(max(G.row0, 0), A.B.m);
    G.n = min(max(G.n, 0), A.B.m - G.row0);
    const int64_t rel = max(u - G.unit0, (int64_t)0);
    const int64_t item = min(rel / G.tiles, A.plan.items - 1);
    const int t = (int)(rel % G.tiles), tile = (int)(item / A.kv_heads);
    out->n = (int)min((int64_t)(G.tiles - t), end - u);
    s_u[0] = u + out->n;
    out->leader = G.leader;
    out->head = (int)(item - (int64_t)tile * A.kv_heads);
    out->row0 = G.row0;
    out->r0 = tile * A.plan.tile_rows;
    out->rows = G.n * A.group;
    out->kv0 = G.lo + kToks * t;
    out->kv_hi = min(G.from, out->kv0 + kToks * out->n);
    out->full_lo = G.full_lo;
    out->slot = (int)min(max(c + G.item0 + item, (int64_t)0), A.plan.slots - 1);
}
static_assert(sizeof(PrefixGroup) == 48, "read as three 16-byte words");

constexpr int kThreads = 640;
constexpr int kKWarp = 8, kVWarp = 12, kMmaWarp = 16, kPageWarp = 17;  // as in the prompt kernels
constexpr int kRegsAll = 5 * (65536 / kThreads / 8 * 8);

__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }  // warps 0-7

// fp32 rows: the pipeline of attn_prompt_kernel.
constexpr int kRegsSoftmax1 = 104, kRegsSums1 = 176, kRegsLoad1 = 72, kRegsCtrl1 = 56;
static_assert(kRegsSoftmax1 + kRegsSums1 + 2 * kRegsLoad1 + kRegsCtrl1 <= kRegsAll, "register split");

template <int D>
struct Layout {
    static constexpr int kTile = kToks * D * 2;  // a K or V tile, one term of 128 fp32 queries, 128 bf16 queries
    static constexpr int kSlots = 4;
    static constexpr int kBytes = 1024 + 2 * kTile + kSlots * kTile;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ PrefixParams A) {
    using L = Layout<D>;
    constexpr uint32_t kColS = 0, kColO = 256;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* s_q = smem;
    uint8_t* s_kv = smem + 2 * L::kTile;
    __shared__ __align__(8) uint64_t full[L::kSlots], empty[L::kSlots], meta_full[kMetaRing], meta_empty[kMetaRing];
    __shared__ __align__(8) uint64_t q_full, s_full[2], max_full[2], p_full[2], o_full[2], fin, drain;
    __shared__ TileMeta s_meta[kMetaRing];
    __shared__ float s_c[kRows], s_ref[2][kRows], s_l[kRows];
    __shared__ uint32_t s_tmem;
    __shared__ Segment s_seg;
    __shared__ int64_t s_u[2];
    __shared__ int s_nan[2];
    __shared__ volatile int s_abort;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t units = __ldcg(&A.plan.head->units);
    const int ctas = __ldcg(&A.plan.head->ctas), cta = blockIdx.x;
    if (cta >= ctas || ctas > kPrefixCtas || units < ctas || units > A.plan.units) return;  // the whole CTA, before any allocation
    if (tid < 2) s_u[tid] = cut(units, ctas, cta + tid);
    if (tid == 32) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kMetaRing; ++i) {
            mbar_init(&meta_full[i], 1);
            mbar_init(&meta_empty[i], 16);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
            mbar_init(&max_full[i], 128);
        }
        mbar_init(&q_full, 256);
        mbar_init(&fin, 256);
        mbar_init(&drain, 1);
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(bar, parity, &s_abort, A.wait_ns); };
    int j0 = 0, seg = 0;  // tiles and segments before this one
    bool issued = false;
    // Every role's loop: the segment before is done with by all, the next one is known to all (false: there is none).
    auto next = [&]() {
        tc_fence_before();
        __syncthreads();
        if (warp == 0) find_segment(A, cta, s_u, &s_abort, &s_seg);
        if (tid == 32) {
            s_nan[0] = 0x7FFFFFFF;
            s_nan[1] = -1;
        }
        __syncthreads();
        tc_fence_after();
        return s_seg.n > 0;  // not s_abort: a role that is already ahead may set it while others look
    };
    auto done = [&](bool ok) {
        if (!ok) {
            s_abort = 1;
            raise_flag(A.err_flag, Q4K_ERR_TIMEOUT);
        }
        j0 += s_seg.n;
        ++seg;
    };
    // The first token that query row `tid % 128` of the row tile sees.
    auto first_seen = [&](bool valid) {
        if (A.window <= 0) return 0;
        const int r = valid ? s_seg.r0 + (tid & 127) : 0;
        return max(__ldcg(A.plan.pos + s_seg.row0 + r / A.group) - A.window + 1, 0);
    };
    // Queries, by warps 0-7: four threads a row, D/4 dims each, 64 rows at a time, scaled by a power of two into fp16's range.
    auto load_queries = [&]() {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            const int qrow = 64 * half + (tid >> 2), part = tid & 3, qr = s_seg.r0 + qrow;
            const bool there = qr < s_seg.rows;
            const float* p = static_cast<const float*>(A.q) + (int64_t)(s_seg.row0 + (there ? qr / A.group : 0)) * A.q_stride +
                             (int64_t)(s_seg.head * A.group + (there ? qr % A.group : 0)) * D + part * (D / 4);
            float x[D / 4];
            Vec<float>::load(p, x);
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) {
                if (!there) x[i] = 0.0f;
                const float a = fabsf(x[i]);
                if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int e = amax > 0.0f ? min(max(134 - (int)(__float_as_uint(amax) >> 23), -120), 120) : 0;
            const float up = A.sign * exp2_int(e);
            if (part == 0) s_c[qrow] = A.scale_log2 * exp2_int(-e);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {  // 8 dims a unit
                const int unit = part * (D / 32) + k;
                uint8_t* dst = s_q + (unit >> 3) * (kRows * 128) + qrow * 128 + (((unit & 7) ^ (qrow & 7)) << 4);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = x[8 * k + 2 * i] * up, b = x[8 * k + 2 * i + 1] * up;
                    const __half2 h = __floats2half2_rn(a, b);
                    const float2 f = __half22float2(h);
                    hi[i] = h2_bits(h);
                    lo[i] = h2_bits(__floats2half2_rn(a - f.x, b - f.y));
                }
                *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(dst + L::kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_full);
        sync_softmax();
    };
    // the place of tile j's K and V in the order of the slots
    auto k_entry = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto v_entry = [](int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; };

    if (warp >= kMmaWarp) {
        regs_dec<kRegsCtrl1>();
        while (next()) {
            bool ok = true;
            const int n = s_seg.n;
            if (warp == kMmaWarp) {
                const uint32_t idesc_s = idesc_f16_f32(kRows, kToks);
                const uint32_t idesc_o = idesc_f16_f32(kRows, D) | kIdescBMnMajor;
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                const uint32_t q_at = __shfl_sync(0xffffffffu, smem_u32(s_q), 0), kv_at = q_at + 2 * L::kTile;
                ok = wait(&q_full, seg & 1);
#pragma unroll 1
                for (int j = -1; j < n && ok; ++j) {
                    if (j + 1 < n) {
                        const int e = 2 * j0 + k_entry(j + 1), slot = e % L::kSlots, b2 = (j0 + j + 1) & 1;
                        ok = wait(&full[slot], (e / L::kSlots) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t b = desc_sw128_kmajor(kv_at + slot * L::kTile);
#pragma unroll
                        for (int t = 1; t >= 0; --t) {  // the low term first, into small sums
                            const uint64_t a = desc_sw128_kmajor(q_at + t * L::kTile);
#pragma unroll
                            for (int k = 0; k < D / 64; ++k)
                                mma_f16_ss_elect4(tm + kColS + b2 * kToks, a + ((k * kToks * 128) >> 4), b + ((k * kToks * 128) >> 4), 2, 2,
                                                  idesc_s, 1 - t + k);
                        }
                        mma_commit_elect(&s_full[b2]);
                        mma_commit_elect(&empty[slot]);
                        issued = true;
                    }
                    if (j < 0) continue;
                    const int e = 2 * j0 + v_entry(j, n), slot = e % L::kSlots, jj = j0 + j;
                    ok = wait(&p_full[jj & 1], (jj >> 1) & 1) && wait(&full[slot], (e / L::kSlots) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t p = tm + kColS + (jj & 1) * kToks, d = tm + kColO + (jj & 1) * D;
                    const uint64_t b = desc_sw128_mnmajor(kv_at + slot * L::kTile, kToks * 128);
                    const uint64_t b1 = b + ((16 * 128) >> 4);
                    mma_f16_ts_elect4(d, p + 16, b, 32, (32 * 128) >> 4, idesc_o, 0);
                    mma_f16_ts_elect4(d, p + 24, b1, 32, (32 * 128) >> 4, idesc_o, 1);
                    mma_f16_ts_elect4<11>(d, p, b, 32, (32 * 128) >> 4, idesc_o, 1);
                    mma_f16_ts_elect4(d, p + 8, b1, 32, (32 * 128) >> 4, idesc_o, 1);
                    mma_commit_elect(&o_full[jj & 1]);
                    mma_commit_elect(&empty[slot]);
                }
            } else if (warp == kPageWarp) {
                ok = page_ahead<D>(A, s_seg.leader, s_seg.head, s_seg.kv0, s_seg.kv_hi, n, s_meta, meta_full, meta_empty, &s_abort, j0);
            }
            done(ok);
        }
    } else if (warp >= kKWarp) {
        regs_dec<kRegsLoad1>();
        while (next()) {
            const bool v_side = warp >= kVWarp;
            const int n = s_seg.n;
            const bool ok = expand_side<D, L::kSlots>(A, v_side, s_seg.kv_hi - s_seg.kv0, n,
                                                      [&](int j) { return 2 * j0 + (v_side ? v_entry(j, n) : k_entry(j)); }, s_kv, s_meta,
                                                      meta_full, meta_empty, full, empty, s_nan, &s_abort, j0);
            if (v_side) mbar_arrive(&fin);
            done(ok);
        }
    } else if (warp < 4) {
        regs_inc<kRegsSoftmax1>();
        const int row = tid;
        const uint32_t lane_at = tmem + ((uint32_t)(32 * warp) << 16);
        while (next()) {
            bool ok = true;
            const int n = s_seg.n, kv0 = s_seg.kv0, kv_hi = s_seg.kv_hi, full_lo = s_seg.full_lo;
            load_queries();
            const bool valid = s_seg.r0 + row < s_seg.rows;
            const int lo = first_seen(valid), hi = valid ? kv_hi : 0;
            const float crow = s_c[row];
            // ---------------- softmax: thread = row = tensor memory lane
            float ref = -INFINITY, l = 0.0f;
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const int jj = j0 + j, b = jj & 1;
                ok = wait(&max_full[b], (jj >> 1) & 1);  // S and its scales, too
                if (!ok) break;
                tc_fence_after();
                const TileMeta& meta = s_meta[jj % kMetaRing];
                const int t0 = kv0 + kToks * j;
                const bool whole = meta.all_ok && t0 >= full_lo && t0 + kToks <= kv_hi;
                const float r_new = s_ref[b][row];  // -inf while the row has seen nothing
                const float use = r_new == -INFINITY ? 0.0f : r_new;
                l *= ex2(ref - use);
                ref = r_new;
                const bool plain = all_near(use) && whole;
                l += weights2(lane_at + kColS + b * kToks, meta, crow, weight_base(use, kTop), t0, lo, hi, plain);
                warp_arrive(&meta_empty[jj % kMetaRing]);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[b]);
            }
            s_l[row] = l;
            mbar_arrive(&fin);
            done(ok);
        }
    } else {
        regs_inc<kRegsSums1>();
        const int row = tid - 128;
        const uint32_t lane_at = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        while (next()) {
            bool ok = true;
            const int n = s_seg.n, kv0 = s_seg.kv0, kv_hi = s_seg.kv_hi, full_lo = s_seg.full_lo;
            load_queries();
            const bool valid = s_seg.r0 + row < s_seg.rows;
            const int lo = first_seen(valid), hi = valid ? kv_hi : 0;
            const float crow = s_c[row];
            // ---------------- maxima and sums: thread = row
            float m = -INFINITY, corr = 0.0f, corr_last = 0.0f;
            float2 acc[D / 2];
#pragma unroll
            for (int c = 0; c < D / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
#pragma unroll 1
            for (int j = 0; j <= n; ++j) {
                const int jj = j0 + j;
                if (j < n) {
                    const int b = jj & 1;
                    ok = wait(&meta_full[jj % kMetaRing], (jj / kMetaRing) & 1) && wait(&s_full[b], (jj >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const TileMeta& meta = s_meta[jj % kMetaRing];
                    const int t0 = kv0 + kToks * j;
                    const bool whole = meta.all_ok && t0 >= full_lo && t0 + kToks <= kv_hi;
                    const float m_new = fmaxf(m, row_max(lane_at + kColS + b * kToks, meta, crow, t0, lo, hi, whole));
                    corr_last = corr;
                    corr = ex2(m - (m_new == -INFINITY ? 0.0f : m_new));
                    m = m_new;
                    s_ref[b][row] = m_new;
                    warp_arrive(&meta_empty[jj % kMetaRing]);
                    tc_fence_before();
                    mbar_arrive(&max_full[b]);
                } else {
                    corr_last = corr;
                }
                if (j == 0) continue;
                ok = wait(&o_full[(jj - 1) & 1], ((jj - 1) >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = lane_at + kColO + ((jj - 1) & 1) * D;
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
            ok = ok && wait(&fin, seg & 1);  // the denominators, and the loaders' report of NaN
            if (ok && valid) {
                const int64_t place = (int64_t)s_seg.slot * kRows + row;
                float* o = A.plan.sums + place * D;
#pragma unroll
                for (int c = 0; c < D; c += 16) {
                    float y[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k] = k & 1 ? acc[(c + k) / 2].y : acc[(c + k) / 2].x;
                    if (s_nan[1] >= 0)
                        mark_nan<D, 16>(A, s_seg.leader, s_seg.head, lo, kv_hi - 1, kv0 + kToks * s_nan[0],
                                        kv0 + kToks * (s_nan[1] + 1) - 1, c, y);
                    Vec<float>::store(o + c, y);
                }
                A.plan.refs[place] = make_float2(m == -INFINITY ? m : weight_base(m, kTop), s_l[row]);
            }
            done(ok);
        }
    }
    // every role has left its loop behind the barrier in next()
    if (warp == kMmaWarp) {
        if (s_abort && issued) {  // whichever role gave up: outstanding products finish before tensor memory is freed
            volatile int never = 0;
            mma_commit_elect(&drain);
            mbar_wait(&drain, 0, &never);
        }
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

// bf16 rows: the pipeline of attn_prompt2_kernel, two row tiles that share every K and V tile.
constexpr int kRegsSoftmax2 = 136, kRegsLoad2 = 72, kRegsCtrl2 = 64;
static_assert(2 * kRegsSoftmax2 + 2 * kRegsLoad2 + kRegsCtrl2 <= kRegsAll, "register split");
constexpr float kSlack = 6.0f;  // growth of a row's maximum, in powers of two, before its sums are scaled again

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefix2_kernel(const __grid_constant__ PrefixParams A) {
    using L = Layout<D>;
    constexpr uint32_t kColS = 0, kColO = 256;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* s_q = smem;
    uint8_t* s_kv = smem + 2 * L::kTile;
    __shared__ __align__(8) uint64_t full[L::kSlots], empty[L::kSlots], meta_full[kMetaRing], meta_empty[kMetaRing];
    __shared__ __align__(8) uint64_t q_full, s_full[2], p_full[2], o_full[2], fin, drain;
    __shared__ TileMeta s_meta[kMetaRing];
    __shared__ float s_c[2 * kRows];
    __shared__ uint32_t s_tmem;
    __shared__ Segment s_seg;
    __shared__ int64_t s_u[2];
    __shared__ int s_nan[2];
    __shared__ volatile int s_abort;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t units = __ldcg(&A.plan.head->units);
    const int ctas = __ldcg(&A.plan.head->ctas), cta = blockIdx.x;
    if (cta >= ctas || ctas > kPrefixCtas || units < ctas || units > A.plan.units) return;  // the whole CTA, before any allocation
    if (tid < 2) s_u[tid] = cut(units, ctas, cta + tid);
    if (tid == 32) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(&full[i], 128);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kMetaRing; ++i) {
            mbar_init(&meta_full[i], 1);
            mbar_init(&meta_empty[i], 16);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
        }
        mbar_init(&q_full, 256);
        mbar_init(&fin, 128);
        mbar_init(&drain, 1);
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(bar, parity, &s_abort, A.wait_ns); };
    int j0 = 0, seg = 0;  // tiles and segments before this one
    bool issued = false;
    // Every role's loop: the segment before is done with by all, the next one is known to all (false: there is none).
    auto next = [&]() {
        tc_fence_before();
        __syncthreads();
        if (warp == 0) find_segment(A, cta, s_u, &s_abort, &s_seg);
        if (tid == 32) {
            s_nan[0] = 0x7FFFFFFF;
            s_nan[1] = -1;
        }
        __syncthreads();
        tc_fence_after();
        return s_seg.n > 0;  // not s_abort: a role that is already ahead may set it while others look
    };
    auto done = [&](bool ok) {
        if (!ok) {
            s_abort = 1;
            raise_flag(A.err_flag, Q4K_ERR_TIMEOUT);
        }
        j0 += s_seg.n;
        ++seg;
    };

    if (warp >= kMmaWarp) {
        regs_dec<kRegsCtrl2>();
        while (next()) {
            bool ok = true;
            const int n = s_seg.n;
            if (warp == kMmaWarp) {
                const uint32_t idesc_s = idesc_f16_f32(kRows, kToks);
                const uint32_t idesc_o = idesc_f16_f32(kRows, D) | kIdescBMnMajor;
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                const uint32_t q_at = __shfl_sync(0xffffffffu, smem_u32(s_q), 0), kv_at = q_at + 2 * L::kTile;
                ok = wait(&q_full, seg & 1);
                // slot 2 jj: K of tile jj, slot 2 jj + 1: V
#pragma unroll 1
                for (int j = -1; j < n && ok; ++j) {
                    const int jj = j0 + j;
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        if (j >= 0) {
                            const int sv = 2 * jj + 1;
                            ok = wait(&p_full[x], jj & 1) && (x > 0 || wait(&full[sv % L::kSlots], (sv / L::kSlots) & 1));
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
                            const int sk = 2 * jj + 2;
                            if (x == 0 && !(ok = wait(&full[sk % L::kSlots], (sk / L::kSlots) & 1))) break;
                            tc_fence_after();
                            const uint64_t a = desc_sw128_kmajor(q_at + x * L::kTile);
                            const uint64_t b = desc_sw128_kmajor(kv_at + sk % L::kSlots * L::kTile);
#pragma unroll
                            for (int k = 0; k < D / 64; ++k)
                                mma_f16_ss_elect4(tm + kColS + x * kToks, a + ((k * kToks * 128) >> 4), b + ((k * kToks * 128) >> 4), 2, 2,
                                                  idesc_s, k);
                            mma_commit_elect(&s_full[x]);
                            if (x) mma_commit_elect(&empty[sk % L::kSlots]);
                            issued = true;
                        }
                    }
                }
            } else if (warp == kPageWarp) {
                ok = page_ahead<D>(A, s_seg.leader, s_seg.head, s_seg.kv0, s_seg.kv_hi, n, s_meta, meta_full, meta_empty, &s_abort, j0);
            }
            done(ok);
        }
    } else if (warp >= kKWarp) {
        regs_dec<kRegsLoad2>();
        while (next()) {
            const bool v_side = warp >= kVWarp;
            const bool ok = expand_side<D, L::kSlots>(A, v_side, s_seg.kv_hi - s_seg.kv0, s_seg.n,
                                                      [&](int j) { return 2 * (j0 + j) + v_side; }, s_kv, s_meta, meta_full, meta_empty,
                                                      full, empty, s_nan, &s_abort, j0);
            if (v_side) mbar_arrive(&fin);
            done(ok);
        }
    } else {
        regs_inc<kRegsSoftmax2>();
        // ---------------- softmax: thread = row = tensor memory lane
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t at = tmem + lane_base + kColS + x * kToks, o_at = tmem + lane_base + kColO + x * D;
        while (next()) {
            bool ok = true;
            const int n = s_seg.n, kv0 = s_seg.kv0, kv_hi = s_seg.kv_hi, r0 = s_seg.r0, rows = s_seg.rows, full_lo = s_seg.full_lo;
            // queries: two threads a row, D/2 dims each, 128 rows at a time, scaled by a power of two into fp16's range (exact there)
#pragma unroll 1
            for (int y = 0; y < 2; ++y) {
                const int qrow = tid >> 1, half = tid & 1, qr = r0 + y * kRows + qrow;
                const bool there = qr < rows;
                const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(A.q) +
                                         (int64_t)(s_seg.row0 + (there ? qr / A.group : 0)) * A.q_stride +
                                         (int64_t)(s_seg.head * A.group + (there ? qr % A.group : 0)) * D + half * (D / 2);
                uint4 w4[D / 16];
                uint32_t top = 0;  // largest finite magnitude's bits
#pragma unroll
                for (int i = 0; i < D / 16; ++i) w4[i] = there ? __ldcg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t w[4] = {w4[i].x, w4[i].y, w4[i].z, w4[i].w};
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
                if (half == 0) s_c[y * kRows + qrow] = A.scale_log2 * exp2_int(-e);
                uint8_t* base = s_q + y * L::kTile + qrow * 128;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {  // 8 dims a unit
                    const int unit = half * (D / 16) + i;
                    const uint32_t w[4] = {w4[i].x, w4[i].y, w4[i].z, w4[i].w};
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = h2_bits(__floats2half2_rn(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up));
                    *reinterpret_cast<uint4*>(base + (unit >> 3) * (kRows * 128) + (((unit & 7) ^ (qrow & 7)) << 4)) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&q_full);
            sync_softmax();
            const int r = r0 + x * kRows + row;
            const bool valid = r < rows;
            int lo = 0;
            if (A.window > 0) lo = max(__ldcg(A.plan.pos + s_seg.row0 + (valid ? r / A.group : 0)) - A.window + 1, 0);
            const int hi = valid ? kv_hi : 0;
            const float crow = s_c[x * kRows + row];
            float ref = -INFINITY, l = 0.0f;  // the reference of P and of the sums
            bool near = false;                // all rows of the warp have one, and near
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const int jj = j0 + j;
                ok = wait(&meta_full[jj % kMetaRing], (jj / kMetaRing) & 1) && wait(&s_full[x], jj & 1);
                if (!ok) break;
                tc_fence_after();
                const TileMeta& meta = s_meta[jj % kMetaRing];
                const int t0 = kv0 + kToks * j;
                const bool whole = meta.all_ok && t0 >= full_lo && t0 + kToks <= kv_hi;
                bool one_pass = false;
                if (whole && near) {
                    uint32_t pk[2][32];
                    float top;
                    const float sum = weights_and_max(at, meta, crow, weight_base(ref, kTop - kSlack), pk, &top);
                    if (!__any_sync(0xffffffffu, top > kTop)) {
                        l += sum;
                        tmem_st32(at, pk[0]);
                        tmem_st32(at + 32, pk[1]);
                        one_pass = true;
                    }
                }
                if (!one_pass) {
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
                warp_arrive(&meta_empty[jj % kMetaRing]);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[x]);
            }
            ok = ok && wait(&fin, seg & 1) && wait(&o_full[x], seg & 1);
            if (ok) {
                tc_fence_after();
                const int64_t place = (int64_t)s_seg.slot * (2 * kRows) + x * kRows + row;
                float* o = A.plan.sums + place * D;
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t v[32];
                    float y[32];
                    tmem_ld32(o_at + 32 * q, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) y[c] = __uint_as_float(v[c]);
                    if (s_nan[1] >= 0 && valid)
                        mark_nan<D, 32>(A, s_seg.leader, s_seg.head, lo, kv_hi - 1, kv0 + kToks * s_nan[0],
                                        kv0 + kToks * (s_nan[1] + 1) - 1, 32 * q, y);
                    if (valid) Vec<float>::store(o + 32 * q, y);
                }
                if (valid) A.plan.refs[place] = make_float2(ref == -INFINITY ? ref : weight_base(ref, kTop - kSlack), l);
            }
            done(ok);
        }
    }
    // every role has left its loop behind the barrier in next()
    if (warp == kMmaWarp) {
        if (s_abort && issued) {  // whichever role gave up: outstanding products finish before tensor memory is freed
            volatile int never = 0;
            mma_commit_elect(&drain);
            mbar_wait(&drain, 0, &never);
        }
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int D>
cudaError_t launch_typed(const PrefixParams& P, int ctas, cudaStream_t stream) {
    void (*kern)(PrefixParams);
    if constexpr (sizeof(T) == 4) kern = prefix_kernel<D>;
    else kern = prefix2_kernel<D>;
    // every CTA holds all of its SM's tensor memory: enough shared memory that one fits
    constexpr int smem = Layout<D>::kBytes < 144 * 1024 ? 144 * 1024 : Layout<D>::kBytes;
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
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
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

// Row tiles of all groups at most: a group's last one may be part filled.
int64_t most_items(int batch, int groups, int m, int rep, int kv_heads, int tile_rows) {
    const int some = groups < batch ? groups : batch;
    return ((int64_t)m * rep / tile_rows + (some < m ? some : m)) * kv_heads;
}

// Where the plan's parts lie in the workspace; the bytes of them all.
size_t layout(int batch, int groups, int m, int rep, int kv_heads, int head_dim, int tile_rows, uint8_t* base, PrefixPlan* plan) {
    size_t at = 0;
    auto part = [&](size_t bytes) {
        uint8_t* p = base + at;
        at += (bytes + 255) & ~size_t(255);
        return p;
    };
    const int64_t items = most_items(batch, groups, m, rep, kv_heads, tile_rows), slots = items + kPrefixCtas;
    plan->head = reinterpret_cast<PrefixHead*>(part(sizeof(PrefixHead)));
    plan->group = reinterpret_cast<PrefixGroup*>(part(sizeof(PrefixGroup) * (size_t)groups));
    plan->seq = reinterpret_cast<int2*>(part(sizeof(int2) * (size_t)batch));
    plan->piece = reinterpret_cast<int2*>(part(sizeof(int2) * (size_t)items));
    plan->pos = reinterpret_cast<int*>(part(sizeof(int) * (size_t)m));
    plan->refs = reinterpret_cast<float2*>(part(sizeof(float2) * (size_t)slots * tile_rows));
    plan->sums = reinterpret_cast<float*>(part(sizeof(float) * (size_t)slots * tile_rows * head_dim));
    plan->tile_rows = tile_rows;
    plan->groups = groups;
    plan->items = items;
    plan->slots = slots;
    return at;
}

}  // namespace

size_t prefix_workspace_bytes(int batch, int groups, int m, int q_heads, int kv_heads, int head_dim) {
    if (groups == 0 || m == 0 || batch == 0 || (int64_t)m * q_heads > kPrefixMaxRows) return 0;
    PrefixPlan plan;
    const size_t a = layout(batch, groups, m, q_heads / kv_heads, kv_heads, head_dim, kRows, nullptr, &plan);
    const size_t b = layout(batch, groups, m, q_heads / kv_heads, kv_heads, head_dim, 2 * kRows, nullptr, &plan);
    return a > b ? a : b;
}

cudaError_t launch_prefix(const PagedBatch& B, const void* q, int dtype, int64_t q_stride, int q_heads, int kv_heads,
                          int head_dim, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                          const float* v_scale, const int32_t* group_start, const int32_t* prefix_lens, int groups,
                          int max_prefix, int max_rows, float scale, int window, void* workspace, int* err_flag,
                          PrefixPlan* plan, cudaStream_t stream) {
    const int rep = q_heads / kv_heads, tile_rows = dtype == Q4K_F32 ? kRows : 2 * kRows;
    layout(B.batch, groups, B.m, rep, kv_heads, head_dim, tile_rows, static_cast<uint8_t*>(workspace), plan);
    plan->units = plan->items * (((int64_t)B.max_pages << B.page_shift) / kToks + 1);
    PlanParams L{};
    L.B = B; L.group_start = group_start; L.prefix_lens = prefix_lens; L.plan = *plan;
    L.kv_heads = kv_heads; L.rep = rep; L.window = window; L.max_rows = max_rows; L.err_flag = err_flag;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, prefix_plan_kernel, L);
    if (e != cudaSuccess) return e;
    PrefixParams P{};
    P.B = B; P.q = q; P.q_stride = q_stride; P.k_cache = k_cache; P.v_cache = v_cache; P.k_scale = k_scale; P.v_scale = v_scale;
    P.kv_heads = kv_heads; P.group = rep; P.window = window;
    P.scale_log2 = (scale < 0.0f ? -scale : scale) * 1.44269504088896340736f;
    P.sign = scale < 0.0f ? -1.0f : 1.0f;
    P.err_flag = err_flag;
    P.wait_ns = wait_limit_ns();
    P.plan = *plan;
    const int ctas = kPrefixCtas;
    if (dtype == Q4K_F32) return head_dim == 64 ? launch_typed<float, 64>(P, ctas, stream) : launch_typed<float, 128>(P, ctas, stream);
    return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(P, ctas, stream) : launch_typed<__nv_bfloat16, 128>(P, ctas, stream);
}

}  // namespace q4k
