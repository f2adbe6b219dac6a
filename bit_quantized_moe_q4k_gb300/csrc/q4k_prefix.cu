// q4k_prefix.cu -- attention over prefixes that the sequences of a group share, on the tensor cores: the rows of all of a group's
// sequences against one reading of the prefix.
//
//   out_r = (sum over shared j + sum over own j) P_j v_j / (the same of P_j),
// a sum of two parts that are each relative to a reference of their own, 2^(x - M), and joined by 2^(M_part - M).
// The shared part is made here; the sequences' own one in q4k_own.cu, beside it where SMs are free, and there both are joined.
//
// prefix_plan_kernel lays the work out (q4k_prefix.cuh): one CTA, since it has to see every group before it can cut the line.
// prefix_kernel<D> (fp32 rows, 128 a row tile) and prefix2_kernel<D> (bf16, 256) then are the prompt kernels of
// q4k_attn_tc.cu without the diagonal: the same roles and the same tiles, but a CTA walks over its piece of the line, item after
// item, and leaves sums, references and denominators in fp32. No row sees less than the whole shared part unless there is a
// window, so nearly every tile is of the kind that is multiplied whole.
//
// Bound by the softmax chain of the prompt kernels, 1.9 us for 256 rows and 128 tokens, and by a piece's start and end, about 15 us (its
// queries, their conversion, the first scores, the sums' way out). The plan takes 8 us, 13 with several groups or hundreds of sequences. 64 sequences behind 8192 tokens, 8 kv heads of 128, bf16: 47 us
// in all; 256 behind 32768: 215 us, 186 of them this kernel's on 96 SMs beside the own parts. q4k_paged_attention takes 145 and 1970 us.
#include <atomic>
#include <cstdlib>

#include "q4k_attn_tc.cuh"
#include "q4k_prefix.cuh"

namespace q4k {
using namespace tc;
namespace {

// ---- the plan -----------------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanSeqs = 2048, kPlanGroups = 128;  // whose lengths, and plans, are looked up in shared memory
// What a piece's start and end cost, in units (1.9 us each, 128 tokens of a row tile); what an own piece and 64 of its tokens cost of an SM.
constexpr float kPieceCost = 6.0f, kOwnCost = 0.2f, kOwnTokensCost = 0.2f;
// What a unit, and a piece's start, of a row tile of the shared part cost, in units of an own tile (8 rows). 64 groups of 2 sequences behind
// 2048 tokens, 8 kv heads, shared 190 us and not 134; 32 of 3 behind 2048 and 8192 109 and 104, 275 and 304; 32 of 4 behind 512 and 2048
// 65 and 60, 113 and 130; 24 of 6 behind 512 and 2048 64 and 64, 102 and 140.
constexpr float kShareUnit = 2.0f, kShareStart = 16.0f;

int share_setting() {
    const char* s = getenv("Q4K_SHARE_PREFIX");
    return s ? (atoi(s) != 0 ? 1 : 0) : -1;
}

struct PlanParams {
    PagedBatch B;
    const int32_t *group_start, *prefix_lens;
    PrefixPlan plan;
    int kv_heads, rep, window, max_rows;
    bool always;  // share whatever can be
    int* err_flag;
};

__device__ __forceinline__ int64_t warp_exclusive(int64_t v, int64_t* total) {
    const int lane = threadIdx.x & 31;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    *total = __shfl_sync(0xffffffffu, inc, 31);
    return inc - v;
}

// Piece c of `ctas` of the line begins at unit c * units / ctas.
__device__ __forceinline__ int64_t cut(int64_t units, int ctas, int64_t c) { return units * c / ctas; }
__device__ __forceinline__ int piece_of(int64_t units, int ctas, int64_t u) {  // the last c with cut(c) <= u
    return (int)(((u + 1) * ctas - 1) / units);
}

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const __grid_constant__ PlanParams A) {
    __shared__ int64_t s_own_tokens[kPlanWarps];
    __shared__ int s_own[kPlanWarps], s_pieces[kPlanWarps];
    __shared__ PrefixHead s_head;
    __shared__ int s_start[kPlanSeqs + 1], s_len[kPlanSeqs], s_from[kPlanSeqs], s_piece0[kPlanSeqs];
    __shared__ PrefixGroup s_group[kPlanGroups];
    __shared__ int s_each;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int groups = A.plan.groups, batch = A.B.batch, shift = A.B.page_shift, cap = A.B.max_pages << shift;
    const bool near = batch <= kPlanSeqs;
    PrefixGroup* const plan = groups <= kPlanGroups ? s_group : A.plan.group;  // while it is made
    // Starts that do not rise would let groups share rows: then nothing is shared.
    bool bad = false;
    for (int i = tid; i < batch; i += kPlanThreads) {
        const int a = __ldcg(A.B.q_start + i), b = __ldcg(A.B.q_start + i + 1), l = __ldcg(A.B.seq_lens + i);
        if (a < 0 || b < a || b > A.B.m) bad = true;
        if (l < 0 || l > cap || l < b - a) raise_flag(A.err_flag, Q4K_ERR_SEQ);
        if (near) {
            s_start[i] = a;
            if (i == batch - 1) s_start[batch] = b;
            s_len[i] = l;
            s_from[i] = 0;
        }
        A.plan.seq[i] = make_int2(-1, 0);
    }
    for (int g = tid; g < groups; g += kPlanThreads) {
        const int a = __ldcg(A.group_start + g), b = __ldcg(A.group_start + g + 1), p = __ldcg(A.prefix_lens + g);
        if (a < 0 || b < a || b > batch) bad = true;
        if (p < 0 || p > cap) raise_flag(A.err_flag, Q4K_ERR_SEQ);
        plan[g].leader = a;
        plan[g].n = b;
        plan[g].from = min(max(p, 0), cap);
    }
    if (bad) raise_flag(A.err_flag, Q4K_ERR_SEQ);
    const bool none = __syncthreads_or(bad) != 0;  // what the threads wrote is seen by all, too
    auto span = [&](int i) {  // seq_span of the batch
        if (!near) {
            bool odd;
            return seq_span(A.B, i, &odd);
        }
        SeqSpan s;
        s.start = min(max(s_start[i], 0), A.B.m);
        s.n = min(max(s_start[i + 1], s.start), A.B.m) - s.start;
        s.len = min(max(s_len[i], 0), cap);
        return s;
    };

    for (int g = warp; g < groups; g += kPlanWarps) {
        const int a = plan[g].leader, b = plan[g].n, prefix = plan[g].from;
        __syncwarp();
        PrefixGroup G{};
        if (!none) {
            int least = 0x7FFFFFFF, most = -1, live = 0, rows = 0, tiles = 0, lead = 0x7FFFFFFF;
            for (int i = a + lane; i < b; i += 32) {
                const SeqSpan s = span(i);
                if (s.n == 0) continue;   // nothing of such a sequence is believed: it may have ended
                lead = min(lead, i);
                least = min(least, s.len - s.n);
                most = max(most, s.len - 1);
                rows = max(rows, s.n);
                tiles += (int)(((int64_t)s.n * A.rep + kOwnRows - 1) / kOwnRows);
                ++live;
            }
            least = __reduce_min_sync(0xffffffffu, least);
            most = __reduce_max_sync(0xffffffffu, most);
            rows = __reduce_max_sync(0xffffffffu, rows);
            live = __reduce_add_sync(0xffffffffu, live);
            tiles = __reduce_add_sync(0xffffffffu, tiles);
            G.leader = __reduce_min_sync(0xffffffffu, lead);
            if (live > 1 && (int64_t)rows * A.rep <= A.max_rows) {
                G.row0 = span(a).start;
                G.n = span(b - 1).start + span(b - 1).n - G.row0;
                G.from = min(prefix, max(least, 0)) >> shift << shift;
                G.lo = A.window > 0 ? max(least - A.window + 1, 0) & ~15 : 0;
                G.full_lo = A.window > 0 ? max(most - A.window + 1, 0) : 0;
                const int row_tiles = (int)(((int64_t)G.n * A.rep + A.plan.tile_rows - 1) / A.plan.tile_rows);
                const int units = (G.from - G.lo + kToks - 1) / kToks;
                if (units > 0 && (A.always || (float)tiles * units > (float)row_tiles * (kShareUnit * units + kShareStart))) {
                    G.tiles = units;
                    G.rows = row_tiles;
                    for (int i = a + lane; i < b; i += 32) {
                        A.plan.seq[i] = make_int2(g, G.from);
                        if (near) s_from[i] = G.from;
                        if (A.window > 0) {
                            const SeqSpan s = span(i);
                            for (int t = 0; t < s.n; ++t) A.plan.pos[s.start + t] = s.len - s.n + t;
                        }
                    }
                }
            }
        }
        if (lane == 0) plan[g] = G;
    }
    __syncthreads();
    // The sequences' own row tiles and their tokens, counted by all warps but the first; it meanwhile finds the groups' places.
    struct Own { SeqSpan s; int from, tiles; };
    auto own_of = [&](int i) {
        Own w{};
        w.s = span(i);
        if (w.s.n == 0 || (int64_t)w.s.n * A.rep > A.max_rows) return w;
        w.from = near ? s_from[i] : A.plan.seq[i].y;
        w.tiles = (w.s.n * A.rep + kOwnRows - 1) / kOwnRows;
        return w;
    };
    auto tokens_of = [&](const Own& w, int tile) {  // [x, y): what some row of the tile sees
        const int first = w.s.len - w.s.n, pf = first + tile * kOwnRows / A.rep;
        const int pl = first + (min(w.s.n * A.rep, (tile + 1) * kOwnRows) - 1) / A.rep;
        const int lo = max(A.window > 0 ? max(pf - A.window + 1, 0) & ~15 : 0, w.from);
        return make_int2(lo, max(max(pl + 1, 0), lo));
    };
    constexpr int kOwnThreads = kPlanThreads - 32;
    const int runs = (batch + kOwnThreads - 1) / kOwnThreads, s0 = min(max(tid - 32, 0) * runs, batch), s1 = warp ? min(s0 + runs, batch) : s0;
    int tiles_before = 0;   // of this thread's run of sequences, within its warp
    if (warp == 0) {
        int64_t items = 0, units = 0;
        int most = 1;
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int g = g0 + lane;
            const int64_t n = g < groups ? (int64_t)plan[g].rows * A.kv_heads : 0, t = g < groups ? plan[g].tiles : 0;
            int64_t ti, tu;
            const int64_t i0 = warp_exclusive(n, &ti), v0 = warp_exclusive(n * t, &tu);
            if (g < groups) {
                plan[g].item0 = items + i0;
                plan[g].unit0 = units + v0;
            }
            most = max(most, (int)t);
            items += ti;
            units += tu;
        }
        items = min(items, A.plan.items);
        asm volatile("bar.sync 1, %0;" ::"n"(kPlanThreads) : "memory");
        int64_t tokens = lane > 0 && lane < kPlanWarps ? s_own_tokens[lane] : 0;
#pragma unroll
        for (int o = 16; o; o >>= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
        const int own_tiles = __reduce_add_sync(0xffffffffu, lane > 0 && lane < kPlanWarps ? s_own[lane] : 0);
        // Own pieces: one and a half for each warp that works on them, but not shorter than is worth a start.
        const int length = own_length(tokens, A.kv_heads);
        // How many CTAs: the sequences' own tiles run on the SMs that these leave free, and on all when they are done. Candidates in steps
        // of a sixteenth, the cheapest by estimate.
        const float own_work = (float)A.kv_heads * (kOwnCost * ((float)own_tiles + (float)tokens / (float)length) +
                                                     kOwnTokensCost / 64.0f * (float)tokens);
        const int candidate = max(kPrefixCtas * (lane < 16 ? lane + 1 : 16) / 16, 1);
        const float shared_time = kPieceCost + ceilf((float)units / (float)candidate);
        const float left = fmaxf(own_work - (float)(kPrefixCtas - candidate) * shared_time, 0.0f) / (float)kPrefixCtas;
        // (the estimate's bits order as it does; the least by the lowest lane)
        const unsigned best = __reduce_min_sync(0xffffffffu, (__float_as_uint(shared_time + left) & ~31u) | (unsigned)lane) & 31u;
        const int most_ctas = __shfl_sync(0xffffffffu, candidate, (int)best);
        // Pieces of `each` units at most, none of two items, where that takes not much longer than equal pieces of the line of all
        // units, of which many consist of two parts.
        int each = 0;
        const int equal = (int)((units + most_ctas - 1) / most_ctas);
        int64_t ctas = min(units, (int64_t)most_ctas);
        if (items > 0 && items <= kPrefixCtas) {
            int64_t pieces = 0;
            for (each = max(equal, 1); each <= equal + (int)kPieceCost; each += 1 + each / 16) {
                pieces = 0;
                for (int g0 = 0; g0 < groups; g0 += 32) {
                    const int g = g0 + lane;
                    int64_t more;
                    const int64_t before = warp_exclusive(g < groups ? plan[g].rows * A.kv_heads * ((plan[g].tiles + each - 1) / each) : 0, &more);
                    if (g < groups) plan[g].cta0 = (int)min(pieces + before, (int64_t)0x7FFFFFFF);
                    pieces += more;
                }
                if (pieces <= most_ctas || pieces <= items) break;   // (an item is a piece at least)
            }
            if (pieces <= max((int64_t)most_ctas, items) && pieces <= kPrefixCtas) ctas = pieces;
            else each = 0;
        }
        if (lane == 0) {
            s_each = each;
            s_head = PrefixHead{units, items, (int)ctas, own_tiles, 0, length, 0, {0, 0, 0}};
        }
    } else {
        int tiles = 0;
        int64_t tokens = 0;
        for (int i = s0; i < s1; ++i) {
            const Own w = own_of(i);
            tiles += w.tiles;
            for (int t = 0; t < w.tiles; ++t) {
                const int2 x = tokens_of(w, t);
                tokens += x.y - x.x;
            }
        }
        int inc = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        tiles_before = inc - tiles;
#pragma unroll
        for (int o = 16; o; o >>= 1) tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
        if (lane == 31) s_own[warp] = inc;
        if (lane == 0) s_own_tokens[warp] = tokens;
        asm volatile("bar.arrive 1, %0;" ::"n"(kPlanThreads) : "memory");
    }
    __syncthreads();
    const int each = s_each, ctas = s_head.ctas;
    const int64_t all_items = s_head.items, all_units = s_head.units;
    if (plan == s_group)
        for (int g = tid; g < groups; g += kPlanThreads) A.plan.group[g] = plan[g];
    auto group_of = [&](int64_t item) {  // the last group that begins at or before it
        int a = 0, b = groups;
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (plan[mid].item0 <= item) a = mid;
            else b = mid;
        }
        return a;
    };
    auto item_at = [&](const PrefixGroup& G, int64_t item, int slot, int slots) {
        const int rel = (int)(item - G.item0), tile = rel / A.kv_heads;
        return PrefixItem{slot, slots, G.row0, tile * A.plan.tile_rows, G.n * A.rep, rel - tile * A.kv_heads, {0, 0}};
    };
    auto piece_at = [&](const PrefixGroup& G, int64_t item, int t, int n, int slot, int next) {
        const int rel = (int)(item - G.item0), tile = rel / A.kv_heads;
        PrefixPiece p;
        p.n = n;
        p.leader = G.leader;
        p.head = rel - tile * A.kv_heads;
        p.row0 = G.row0;
        p.r0 = tile * A.plan.tile_rows;
        p.rows = G.n * A.rep;
        p.kv0 = G.lo + kToks * t;
        p.kv_hi = min(G.from, p.kv0 + kToks * n);
        p.full_lo = G.full_lo;
        p.slot = slot;
        p.next = next;
        p.pad = 0;
        return p;
    };
    for (int64_t i = tid; i < all_items; i += kPlanThreads) {
        const PrefixGroup& G = plan[group_of(i)];
        if (each > 0) {  // the item's pieces, a CTA each
            const int k = (G.tiles + each - 1) / each;
            A.plan.item[i] = item_at(G, i, G.cta0 + (int)(i - G.item0) * k, k);
        } else {
            // the CTAs that share it: one that begins within it (or at its start) has it as its first piece, the one before it as a later one
            const int64_t u = G.unit0 + (i - G.item0) * G.tiles, end = u + G.tiles;
            const int c0 = piece_of(all_units, ctas, u), c1 = piece_of(all_units, ctas, end - 1);
            A.plan.item[i] = item_at(G, i, (int)(c0 + i), c1 - c0 + 1);
            for (int c = c0; c <= c1; ++c) {
                const int64_t a = cut(all_units, ctas, c), b = cut(all_units, ctas, c + 1), from = max(a, u);
                const int next = b > end ? (int)(kPrefixCtas + i + 1) : -1;
                A.plan.piece[a >= u ? c : (int)(kPrefixCtas + i)] =
                    piece_at(G, i, (int)(from - u), (int)(min(b, end) - from), (int)(c + i), next);
            }
        }
    }
    if (each > 0 && tid < ctas) {
        int a = 0, b = groups;  // the last group whose pieces begin at or before CTA tid
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (plan[mid].cta0 <= tid) a = mid;
            else b = mid;
        }
        const PrefixGroup& G = plan[a];
        const int k = (G.tiles + each - 1) / each, rel = tid - G.cta0, item = rel / k, j = rel - item * k;
        const int t = G.tiles * j / k;
        A.plan.piece[tid] = piece_at(G, G.item0 + item, t, G.tiles * (j + 1) / k - t, tid, -1);
    }
    // the sequences' own row tiles, then their pieces
    const int length = s_head.own_length, counted = lane > 0 && lane < kPlanWarps ? s_own[lane] : 0;
    int at = tiles_before + __reduce_add_sync(0xffffffffu, lane < warp ? counted : 0);
    auto pieces_of = [&](const int2& x) { return pieces_of_tile(x.y - x.x, length); };
    int pieces = 0;
    for (int i = s0; i < s1; ++i) {
        const Own w = own_of(i);
        for (int t = 0; t < w.tiles; ++t) pieces += pieces_of(tokens_of(w, t));
    }
    int inc = pieces;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) s_pieces[warp] = inc;
    __syncthreads();
    const int counted_pieces = lane < kPlanWarps ? s_pieces[lane] : 0;
    const int all_pieces = __reduce_add_sync(0xffffffffu, counted_pieces);
    int piece = inc - pieces + __reduce_add_sync(0xffffffffu, lane < warp ? counted_pieces : 0);
    for (int i = s0; i < s1; ++i) {
        const Own w = own_of(i);
        const int g = w.tiles ? A.plan.seq[i].x : -1;
        for (int t = 0; t < w.tiles; ++t, ++at) {
            const int2 x = tokens_of(w, t);
            const int k = pieces_of(x);
            const int first = g < 0 ? -1 : (w.s.start - plan[g].row0) * A.rep + t * kOwnRows;
            if (at < A.plan.owns) A.plan.own[at] = OwnTile{i, w.s.start, w.s.n, w.s.len, x.x, x.y, t, piece, k, first, g < 0 ? 0 : plan[g].item0};
            if (at < kPlanSeqs) s_piece0[at] = piece;
            piece += k;
        }
    }
    __syncthreads();
    const int all_tiles = (int)min((int64_t)s_head.own_tiles, A.plan.owns);  // (less only where starts fall)
    const int most = (int)min((int64_t)all_pieces, A.plan.own_pieces);
    for (int p = tid; p < most && all_tiles; p += kPlanThreads) {
        int a = 0, b = all_tiles;  // the last tile that begins at or before piece p
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if ((mid < kPlanSeqs ? s_piece0[mid] : A.plan.own[mid].piece0) <= p) a = mid;
            else b = mid;
        }
        const int first = a < kPlanSeqs ? s_piece0[a] : A.plan.own[a].piece0;
        A.plan.own_piece[p] = make_int2(a, (p - first) * length);
    }
    if (tid == 0) {
        if (s_head.own_tiles > A.plan.owns || all_pieces > A.plan.own_pieces) raise_flag(A.err_flag, Q4K_ERR_SEQ);
        PrefixHead H = s_head;
        H.own_tiles = all_tiles;
        H.own_pieces = all_tiles ? most : 0;
        *A.plan.head = H;
    }
}

// ---- the shared part ----------------------------------------------------------------------------------------------
struct PrefixParams : PromptParams {  // window: the attention's; out, out_stride, min_rows: not used
    PrefixPlan plan;
};

// The CTA's next piece, by a warp: number `at` of the list. None once a role has given up. Two calls at once on one workspace write over
// each other's plans: nothing of one is believed as far as addresses go.
__device__ __forceinline__ void read_piece(const PrefixParams& A, int at, volatile int* abort, PrefixPiece* out) {
    const int lane = threadIdx.x & 31;
    __syncwarp();  // `at` may come from where the piece goes
    if (at < 0 || at >= kPrefixCtas + A.plan.items || (abort && *abort)) {
        if (lane == 0) out->n = 0;
        return;
    }
    if (lane < 3) reinterpret_cast<int4*>(out)[lane] = __ldcg(reinterpret_cast<const int4*>(A.plan.piece + at) + lane);
    __syncwarp();
    if (lane) return;
    PrefixPiece p = *out;
    p.leader = min(max(p.leader, 0), A.B.batch - 1);
    p.head = min(max(p.head, 0), A.kv_heads - 1);
    p.row0 = min(max(p.row0, 0), A.B.m - 1);
    p.rows = (int)min((int64_t)max(p.rows, 1), (int64_t)(A.B.m - p.row0) * A.group);
    p.r0 = min(max(p.r0, 0), p.rows - 1);
    p.kv0 = max(p.kv0, 0) & ~15;
    p.kv_hi = min(p.kv_hi, A.B.max_pages << A.B.page_shift) & ~15;
    p.n = p.kv_hi > p.kv0 ? (p.kv_hi - p.kv0 + kToks - 1) / kToks : 0;
    p.slot = (int)min((int64_t)max(p.slot, 0), A.plan.slots - 1);
    p.next = p.next > at ? p.next : -1;
    *out = p;
}
static_assert(sizeof(PrefixPiece) == 48, "read as three 16-byte words");

constexpr int kThreads = 640;
constexpr int kKWarp = 8, kVWarp = 12, kMmaWarp = 16, kPageWarp = 17;  // as in the prompt kernels
constexpr int kRegsAll = 5 * (65536 / kThreads / 8 * 8);

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// The rows first, first + step, .. below `count` of a piece's row tile, a thread's part of each at `q` + its place: take(row, where, or null
// past the group's last).
template <typename T, typename F>
__device__ __forceinline__ void copy_rows(const T* q, const PrefixParams& A, const PrefixPiece& seg, int d, int first, int step, int count,
                                          F take) {
    const int group = A.group, rows = seg.rows - seg.r0, r = seg.r0 + first;
    int h = r % group;
    const T* p = q + (int64_t)(seg.row0 + r / group) * A.q_stride + (int64_t)(seg.head * group + h) * d;
    const int64_t move = (int64_t)(step / group) * A.q_stride + (step % group) * d, wrap = A.q_stride - (int64_t)group * d;
    const int h_step = step % group;
#pragma unroll 4
    for (int row = first; row < count; row += step) {
        take(row, row < rows ? p : nullptr);
        p += move;
        h += h_step;
        if (h >= group) {
            h -= group;
            p += wrap;
        }
    }
}
// A row of partial sums, which the thread has put into shared memory, to global memory: a copy that runs by itself. The rows lie kRowBytes
// apart there, so that a warp's writes meet all banks.
template <int D> constexpr int kRowBytes = D * 4 + 16;
template <int D>
__device__ __forceinline__ void store_row_async(float* dst, const uint8_t* src) {
    fence_proxy_async_smem();
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "n"(D * 4) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// .. until shared memory may be written again
__device__ __forceinline__ void stored() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// NaN where the row's tokens hold it, in a row of sums in shared memory. Rare, and kept out of the code that runs.
template <int D>
__device__ __noinline__ void mark_row(const PromptParams& A, int seq, int head, int lo, int hi, int from, int to, float* row) {
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
        float y[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) y[k] = row[c + k];
        mark_nan<D, 16>(A, seq, head, lo, hi, from, to, c, y);
#pragma unroll
        for (int k = 0; k < 16; ++k) row[c + k] = y[k];
    }
}

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
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset, so that accesses are known to be to shared memory)
    uint8_t* s_q = smem;
    uint8_t* s_kv = smem + 2 * L::kTile;
    __shared__ __align__(8) uint64_t full[L::kSlots], empty[L::kSlots], meta_full[kMetaRing], meta_empty[kMetaRing];
    __shared__ __align__(8) uint64_t q_full, s_full[2], max_full[2], p_full[2], o_full[2], fin, drain;
    __shared__ TileMeta s_meta[kMetaRing];
    __shared__ float s_c[kRows], s_ref[2][kRows], s_l[kRows];
    __shared__ uint32_t s_tmem;
    __shared__ PrefixPiece s_seg;
    __shared__ int s_nan[2];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5;
    // what needs no results of the plan goes before the wait for it
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
        s_nan[0] = 0x7FFFFFFF;
        s_nan[1] = -1;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) read_piece(A, (int)blockIdx.x < __ldcg(&A.plan.head->ctas) ? (int)blockIdx.x : -1, nullptr, &s_seg);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(bar, parity, &s_abort, A.wait_ns); };
    int j0 = 0, seg = 0;  // tiles and segments before this one
    bool issued = false;
    // Every role's loop: the segment before is done with by all, the next one is known to all (false: there is none).
    auto next = [&]() {
        if (seg > 0) {
            tc_fence_before();
            __syncthreads();
            if (warp == 0) read_piece(A, s_seg.next, &s_abort, &s_seg);
            if (tid == 32) {
                s_nan[0] = 0x7FFFFFFF;
                s_nan[1] = -1;
            }
            __syncthreads();
            tc_fence_after();
        }
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
    // Queries, by warps 0-7: sixteen (or eight) lanes a row of D dims, eight dims a lane. The rows are copied to where their two terms
    // will lie, and turned into them there, scaled by a power of two into fp16's range.
    auto load_queries = [&]() {
        constexpr int kLanes = D / 8, kStep = 256 / kLanes;   // lanes of a row, rows at a time
        const int u = tid % kLanes;
        uint8_t* const at = s_q + (u >> 3) * (kRows * 128);
        auto place_of = [&](int row) { return at + row * 128 + (((u & 7) ^ (row & 7)) << 4); };
        copy_rows(static_cast<const float*>(A.q) + 8 * u, A, s_seg, D, tid / kLanes, kStep, kRows, [&](int row, const float* p) {
            if (p) {
                copy16(place_of(row), p);
                copy16(place_of(row) + L::kTile, p + 4);
            } else {
                *reinterpret_cast<uint4*>(place_of(row)) = *reinterpret_cast<uint4*>(place_of(row) + L::kTile) = make_uint4(0, 0, 0, 0);
            }
        });
        asm volatile("cp.async.wait_all;" ::: "memory");
        constexpr int kBatch = 4;  // rows read before the first is written: the chain of one is some hundred cycles long
#pragma unroll 1
        for (int row0 = tid / kLanes; row0 < kRows; row0 += kBatch * kStep) {
            float x[kBatch][8], amax[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const uint8_t* p = place_of(row0 + b * kStep);
                *reinterpret_cast<float4*>(x[b]) = *reinterpret_cast<const float4*>(p);
                *reinterpret_cast<float4*>(x[b] + 4) = *reinterpret_cast<const float4*>(p + L::kTile);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                amax[b] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a = fabsf(x[b][i]);
                    if (a <= 3.402823466e38f) amax[b] = fmaxf(amax[b], a);
                }
            }
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1)
#pragma unroll
                for (int b = 0; b < kBatch; ++b) amax[b] = fmaxf(amax[b], __shfl_xor_sync(0xffffffffu, amax[b], o));
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int row = row0 + b * kStep;
                const int e = amax[b] > 0.0f ? min(max(134 - (int)(__float_as_uint(amax[b]) >> 23), -120), 120) : 0;
                const float up = A.sign * exp2_int(e);
                if (u == 0) s_c[row] = A.scale_log2 * exp2_int(-e);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = x[b][2 * i] * up, q = x[b][2 * i + 1] * up;
                    const __half2 t = __floats2half2_rn(p, q);
                    const float2 f = __half22float2(t);
                    hi[i] = h2_bits(t);
                    lo[i] = h2_bits(__floats2half2_rn(p - f.x, q - f.y));
                }
                *reinterpret_cast<uint4*>(place_of(row)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(place_of(row) + L::kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
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
                // all products are done: the queries' and the tiles' place is free
                uint8_t* const mine = s_q + row * kRowBytes<D>;
#pragma unroll
                for (int c = 0; c < D; c += 16) {
                    float y[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k] = k & 1 ? acc[(c + k) / 2].y : acc[(c + k) / 2].x;
                    Vec<float>::store(reinterpret_cast<float*>(mine) + c, y);
                }
                if (s_nan[1] >= 0)
                    mark_row<D>(A, s_seg.leader, s_seg.head, lo, kv_hi - 1, kv0 + kToks * s_nan[0], kv0 + kToks * (s_nan[1] + 1) - 1,
                                reinterpret_cast<float*>(mine));
                store_row_async<D>(A.plan.sums + place * D, mine);
                A.plan.refs[place] = make_float2(m == -INFINITY ? m : weight_base(m, kTop), s_l[row]);
                stored();
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
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset, so that accesses are known to be to shared memory)
    uint8_t* s_q = smem;
    uint8_t* s_kv = smem + 2 * L::kTile;
    __shared__ __align__(8) uint64_t full[L::kSlots], empty[L::kSlots], meta_full[kMetaRing], meta_empty[kMetaRing];
    __shared__ __align__(8) uint64_t q_full, s_full[2], p_full[2], o_full[2], fin, drain;
    __shared__ TileMeta s_meta[kMetaRing];
    __shared__ float s_c[2 * kRows];
    __shared__ uint32_t s_tmem;
    __shared__ PrefixPiece s_seg;
    __shared__ int s_nan[2];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5;
    // what needs no results of the plan goes before the wait for it
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
        s_nan[0] = 0x7FFFFFFF;
        s_nan[1] = -1;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) read_piece(A, (int)blockIdx.x < __ldcg(&A.plan.head->ctas) ? (int)blockIdx.x : -1, nullptr, &s_seg);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(bar, parity, &s_abort, A.wait_ns); };
    int j0 = 0, seg = 0;  // tiles and segments before this one
    bool issued = false;
    // Every role's loop: the segment before is done with by all, the next one is known to all (false: there is none).
    auto next = [&]() {
        if (seg > 0) {
            tc_fence_before();
            __syncthreads();
            if (warp == 0) read_piece(A, s_seg.next, &s_abort, &s_seg);
            if (tid == 32) {
                s_nan[0] = 0x7FFFFFFF;
                s_nan[1] = -1;
            }
            __syncthreads();
            tc_fence_after();
        }
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
            // queries: sixteen (or eight) lanes a row, eight dims a lane, as in prefix_kernel; exact in one fp16 term
            {
                constexpr int kLanes = D / 8, kStep = 256 / kLanes;
                const int u = tid % kLanes;
                uint8_t* const q_at = s_q + (u >> 3) * (kRows * 128);
                auto place_of = [&](int row) {
                    return q_at + (row >> 7) * L::kTile + (row & 127) * 128 + (((u & 7) ^ (row & 7)) << 4);
                };
                copy_rows(static_cast<const __nv_bfloat16*>(A.q) + 8 * u, A, s_seg, D, tid / kLanes, kStep, 2 * kRows,
                          [&](int qrow, const __nv_bfloat16* p) {
                              if (p) copy16(place_of(qrow), p);
                              else *reinterpret_cast<uint4*>(place_of(qrow)) = make_uint4(0, 0, 0, 0);
                          });
                asm volatile("cp.async.wait_all;" ::: "memory");
                constexpr int kBatch = 4;
#pragma unroll 1
                for (int row0 = tid / kLanes; row0 < 2 * kRows; row0 += kBatch * kStep) {
                    uint4 v[kBatch];
                    uint32_t top[kBatch];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) v[b] = *reinterpret_cast<const uint4*>(place_of(row0 + b * kStep));
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        // largest finite magnitude's bits
                        const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
                        top[b] = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t lo16 = w[k] & 0x7FFFu, hi16 = w[k] >> 16 & 0x7FFFu;
                            if (lo16 < 0x7F80u) top[b] = max(top[b], lo16);
                            if (hi16 < 0x7F80u) top[b] = max(top[b], hi16);
                        }
                    }
#pragma unroll
                    for (int o = kLanes / 2; o; o >>= 1)
#pragma unroll
                        for (int b = 0; b < kBatch; ++b) top[b] = max(top[b], __shfl_xor_sync(0xffffffffu, top[b], o));
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int qrow = row0 + b * kStep;
                        const int e = top[b] > 0 ? min(max(134 - (int)(top[b] >> 7), -120), 120) : 0;
                        const float up = A.sign * exp2_int(e);
                        if (u == 0) s_c[qrow] = A.scale_log2 * exp2_int(-e);
                        uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = h2_bits(__floats2half2_rn(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up));
                        *reinterpret_cast<uint4*>(place_of(qrow)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
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
            ok = ok && wait(&fin, seg & 1) && wait(&o_full[x], seg & 1) && wait(&o_full[x ^ 1], seg & 1);
            if (ok) {
                tc_fence_after();
                const int64_t place = (int64_t)s_seg.slot * (2 * kRows) + x * kRows + row;
                // all products of both row tiles are done: the queries' and the tiles' place is free
                uint8_t* const mine = s_q + (x * kRows + row) * kRowBytes<D>;
                uint32_t v[2][32];
                tmem_ld32(o_at, v[0]);
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    tmem_wait_ld();
                    if (q + 1 < D / 32) tmem_ld32(o_at + 32 * (q + 1), v[(q + 1) & 1]);
#pragma unroll
                    for (int c = 0; c < 32; c += 4)
                        *reinterpret_cast<uint4*>(mine + 128 * q + 4 * c) =
                            make_uint4(v[q & 1][c], v[q & 1][c + 1], v[q & 1][c + 2], v[q & 1][c + 3]);
                }
                if (valid) {
                    if (s_nan[1] >= 0)
                        mark_row<D>(A, s_seg.leader, s_seg.head, lo, kv_hi - 1, kv0 + kToks * s_nan[0],
                                    kv0 + kToks * (s_nan[1] + 1) - 1, reinterpret_cast<float*>(mine));
                    store_row_async<D>(A.plan.sums + place * D, mine);
                    A.plan.refs[place] = make_float2(ref == -INFINITY ? ref : weight_base(ref, kTop - kSlack), l);
                    stored();
                }
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
    // row tiles, a sequence's last part filled; a piece of each kv head
    const int64_t owns = (int64_t)m * rep / kOwnRows + (m < batch ? m : batch), own_pieces = most_own_pieces(owns, kv_heads);
    plan->head = reinterpret_cast<PrefixHead*>(part(sizeof(PrefixHead)));
    plan->group = reinterpret_cast<PrefixGroup*>(part(sizeof(PrefixGroup) * (size_t)groups));
    plan->seq = reinterpret_cast<int2*>(part(sizeof(int2) * (size_t)batch));
    plan->piece = reinterpret_cast<PrefixPiece*>(part(sizeof(PrefixPiece) * (size_t)slots));
    plan->item = reinterpret_cast<PrefixItem*>(part(sizeof(PrefixItem) * (size_t)items));
    plan->own = reinterpret_cast<OwnTile*>(part(sizeof(OwnTile) * (size_t)owns));
    plan->own_piece = reinterpret_cast<int2*>(part(sizeof(int2) * (size_t)own_pieces));
    plan->pos = reinterpret_cast<int*>(part(sizeof(int) * (size_t)m));
    plan->refs = reinterpret_cast<float2*>(part(sizeof(float2) * (size_t)slots * tile_rows));
    plan->sums = reinterpret_cast<float*>(part(sizeof(float) * (size_t)slots * tile_rows * head_dim));
    const int64_t own_slots = own_pieces * kv_heads;
    plan->own_refs = reinterpret_cast<float2*>(part(sizeof(float2) * (size_t)own_slots * kOwnRows));
    plan->own_sums = reinterpret_cast<float*>(part(sizeof(float) * (size_t)own_slots * kOwnRows * head_dim));
    plan->tile_rows = tile_rows;
    plan->groups = groups;
    plan->items = items;
    plan->slots = slots;
    plan->owns = owns;
    plan->own_pieces = own_pieces;
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

// Whether a call is worth the plan, the shared kernel and the join: by how many units of 128 tokens, of a row tile as q4k_paged_attention
// cuts them and a kv head, fewer it would read if its groups were equally large. On both sides of the bound, shared and not (bf16, 8 kv
// heads, one new token each): a group of 32 behind 2048 tokens (3600) 33 and 34 us, 8 behind 8192 (2448) 36 and 32, 4 behind 512 25 and 9,
// 16 groups of 16 behind 512 (4864) 68 and 77, 24 of 6 behind 2048 (6528) 102 and 110, 24 of 5 (3456) 105 and 93.
// The sequences' own units cost more here, each 9/32 of one: 64 sequences with 8000 tokens of their own behind 2048 take 222 and 182 us, 32 with up to
// 30000 behind 8192 191 and 171, 128 with up to 2000 behind 4096 95 and 182. max_len tells how many they may be; where that is more than
// eight times the prefix, it is taken for a bound that says nothing, since sharing in vain loses less than not sharing.
// Switch (environment, read at every call): Q4K_SHARE_PREFIX=1 shares whatever can be, 0 nothing.
constexpr int64_t kShareLeast = 4500;
bool prefix_pays(const PagedBatch& B, int dtype, int q_heads, int kv_heads, int groups, int max_q_len, int max_len, int max_prefix, int window) {
    if (share_setting() >= 0) return share_setting() > 0;
    int64_t tokens = (int64_t)B.max_pages << B.page_shift;
    int64_t own = max_len < tokens ? max_len : tokens;
    tokens = max_prefix < tokens ? max_prefix : tokens;
    own = own > tokens && own - tokens <= 8 * tokens ? own - tokens : 0;
    if (window > 0) {
        tokens = window < tokens ? window : tokens;
        own = window < own ? window : own;
    }
    const int64_t rep = q_heads / kv_heads, units = (tokens + kToks - 1) / kToks, rows = B.m * rep;
    const int64_t own_rows = dtype == Q4K_F32 || max_q_len * rep <= 8 ? 8 : 16, shared_rows = dtype == Q4K_F32 ? kRows : 2 * kRows;
    const int64_t live = B.batch < B.m ? B.batch : B.m, by_rows = (rows + own_rows - 1) / own_rows;
    const int64_t tiles = live > by_rows ? live : by_rows, row_tiles = (groups < live ? groups : live) + rows / shared_rows;
    return (tiles * units - row_tiles * (3 * units + 14) - tiles * (own / kToks) * 9 / 32) * kv_heads >= kShareLeast;
}

cudaError_t launch_prefix(const PagedBatch& B, const void* q, int dtype, int64_t q_stride, int q_heads, int kv_heads,
                          int head_dim, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                          const float* v_scale, const SharedPrefix& shared, int max_rows, float scale, int window, void* out,
                          int64_t out_stride, int* err_flag, cudaStream_t stream) {
    const int rep = q_heads / kv_heads, tile_rows = dtype == Q4K_F32 ? kRows : 2 * kRows, groups = shared.groups;
    PrefixPlan plan;
    layout(B.batch, groups, B.m, rep, kv_heads, head_dim, tile_rows, static_cast<uint8_t*>(shared.workspace), &plan);
    PlanParams L{};
    L.B = B; L.group_start = shared.group_start; L.prefix_lens = shared.prefix_lens; L.plan = plan;
    L.kv_heads = kv_heads; L.rep = rep; L.window = window; L.max_rows = max_rows; L.always = share_setting() > 0; L.err_flag = err_flag;
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
    P.plan = plan;
    const int ctas = kPrefixCtas;
    if (dtype == Q4K_F32) e = head_dim == 64 ? launch_typed<float, 64>(P, ctas, stream) : launch_typed<float, 128>(P, ctas, stream);
    else e = head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(P, ctas, stream) : launch_typed<__nv_bfloat16, 128>(P, ctas, stream);
    if (e != cudaSuccess) return e;
    OwnParams O{B, plan, q, out, q_stride, out_stride, k_cache, v_cache, k_scale, v_scale, kv_heads, rep, window,
                scale * 1.44269504088896340736f, err_flag};
    e = launch_own(O, dtype, head_dim, stream);
    return e != cudaSuccess ? e : launch_join(O, dtype, head_dim, stream);
}

}  // namespace q4k
