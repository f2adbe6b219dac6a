// q4k_attn.cu -- attention over the paged 8-bit cache for few query rows per kv head (decoding).
//
//   out[r] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q_r . k_j)  over the tokens j that row r sees
//
// With everything in powers of two and V's page scale 2^e_j inside the exponent,
//   x_j = c * (code_k . q) * ks_j + e_j,   P_j = 2^(x_j - M + 15),  M the running maximum of x,
//   l = sum_j 2^(-e_j) P_j,   out = sum_j P_j code_v,j / l,
// so the codes of both sides enter the matrix products as they are: e4m3 is exact in fp16. Query
// rows are the M side of mma.m16n8k16: fp32 queries are split into two fp16 halves (hi in rows 0-7,
// lo in rows 8-15, scaled by a power of two so that 22 bits survive) and so are their P; bf16
// queries are exact in one half and P is rounded to fp16 (2^-11), so 16 rows fill the tile. 2^15 is
// the largest power of two in fp16, and the low half of P is held times 2^11, so that small weights (all of them where
// one token without value dominates) stay normal numbers: P_j keeps its 11 or 22 bits down to 2^-29 of the
// largest, below that 2^-40 or 2^-51 of it.
//
// Bound by the cache's bytes. Each warp owns a ring of stages in shared memory, a stage being two chunks
// of 16 tokens (2 KB of K and 2 KB of V each at head_dim 128), which its lanes fill by 16-byte
// asynchronous copies one stage ahead (bulk copies, five a chunk, took 223 us for the batch below where these then
// took 199). The copies place 16-byte units so that the fragment reads meet different banks.
//
// The work (sequence, kv head, row tile, 64 tokens) is laid out on one line and cut into equal pieces, one per CTA,
// whatever the lengths. The CTAs that share a tile leave partial results in the workspace; the last one to arrive
// joins them, in two levels where there are many. (A second kernel for that found no room beside the first, so it began
// to look for its tile only when the first had ended: 8 us of 49 for the long sequence below.) Where there are few
// tiles, clusters of eight CTAs work as one, 512 tokens a unit, and join their tiles through distributed shared
// memory: an eighth of the pieces, and reads of a few hundred cycles instead of the thousand and more through L2.
//
// 64 ragged sequences of up to 8192 tokens, 8 kv heads of 128, 514 MB: 96 us, 5.3 TB/s. One of 131071, 4 kv heads,
// 134 MB: 39 us, 20 of them bytes at the copy rate. One of 509: 8.4 us, the chain of launch, lengths, pages, queries, first copies and
// the joins of warps and cluster; what the long one takes beyond both is not broken down.
#include <atomic>
#include <chrono>

#include "q4k_paged.cuh"

namespace q4k {
namespace {

constexpr int kAttnWarps = 4;
constexpr int kChunk = 16;                    // tokens a warp takes at a time
constexpr int kUnit = kChunk * kAttnWarps;    // tokens of one unit of work
// Units that starting and ending a tile are worth. Ragged batches of 64 up to 8192 tokens, 256 up to 2000, 40 up to
// 30000: 102, 87, 184 us with 4; 96, 76, 174 with 10; 97, 79, 173 with 16.
constexpr int kTileCost = 10;
constexpr int kCtasPerSm = 3;
// A sequence is worked on here up to kFewRows query rows per kv head, and a whole batch up to kFewTiles tiles of 8 rows,
// else by the prompt kernel, whose tiles hold 128 or 256 rows and are not split along the axis. fp32, 4 kv heads, here
// and there: 16 sequences of 2000 tokens with 48 rows 43 and 45 us, with 64 51 and 46 (bf16 42 and 43), with 96 71 and
// 48 (bf16 49 and 44); one of 4000 with 64 rows 16 and 70, with 256 34 and 73.
constexpr int kFewRows = 64, kFewTiles = 450;
constexpr int kLeast = 4;                      // units of a cluster's part of a tile, at least (8: 8000 tokens 15.4 -> 16.5 us)
constexpr int kMaxParts = 512;                // CTAs that the workspace serves
constexpr int kJoinCost = 8;                  // units that joining a tile is worth (16: 8000 tokens 15.4 -> 17.5 us)
static_assert(kJoinCost >= kLeast, "a tile that is shared has a unit for each cluster");
constexpr int kOneLevel = 16;                 // up to this many pieces of a tile are joined at once (4: 16000 tokens 17 -> 21 us)
constexpr int kTickets = 2 * kMaxParts;       // arrival counters before the partial results: by group of pieces, by tile

struct AttnParams {
    PagedBatch B;
    const void* q;
    void* out;
    int64_t q_stride, out_stride;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int kv_heads, group;
    int window;
    int max_rows;       // sequences with more query rows per kv head are the prompt kernel's
    float scale_log2;   // softmax scale * log2(e)
    float* part;        // partial results: per CTA two slots of [rows][D] sums, rows M, rows l
    unsigned long long* tickets;
    unsigned long long tag;  // this launch's counters carry it in their high 48 bits: others count as 0
    int parts;          // CTAs the partial buffer holds
    int* err_flag;
};

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

// The work of one sequence: `tiles` row tiles per kv head, each kTileCost units of nothing (so that a
// piece of many short tiles is not longer than one of a few long ones) and `units` units of kUnit
// tokens, from token `lo` (a multiple of kChunk: the first one any of its rows sees).
struct SeqWork {
    SeqSpan s;
    int lo, tiles, units;
    int64_t total;
};
template <int RT, int CL>
__device__ __forceinline__ SeqWork seq_work(const AttnParams& A, int i) {
    SeqWork w{};
    if (i >= A.B.batch) return w;
    bool bad;
    w.s = seq_span(A.B, i, &bad);
    if (bad) raise_flag(A.err_flag, Q4K_ERR_SEQ);
    if (w.s.n == 0 || (int64_t)w.s.n * A.group > A.max_rows) return w;
    const int first = max(w.s.len - w.s.n, 0);
    w.lo = A.window > 0 ? (max(first - A.window + 1, 0) & ~(kChunk - 1)) : 0;
    w.tiles = (w.s.n * A.group + RT - 1) / RT;
    w.units = max((w.s.len - w.lo + CL * kUnit - 1) / (CL * kUnit), 1);  // an empty sequence: its rows are zeroed
    w.total = (int64_t)w.tiles * A.kv_heads * (kTileCost + w.units);
    return w;
}

// A place on the line of work: the sequence that holds it and the line's position where that
// sequence begins. Every lane of the warp holds the same values.
struct Cursor {
    int seq;
    int64_t begin;
    SeqWork w;
};
__device__ __forceinline__ int64_t warp_scan(int64_t v) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}
// Move the cursor to the sequence that holds u (u >= c.begin; false past the end). `mine`: the work
// of sequence `lane`, read once (it is all there is up to 32 sequences).
template <int RT>
__device__ __forceinline__ bool seek(const AttnParams& A, int64_t u, const SeqWork& mine, Cursor* c) {
    const int lane = threadIdx.x & 31;
    int64_t acc = c->begin;
    for (int base = c->seq & ~31; base < A.B.batch; base += 32) {
        SeqWork w = base == 0 ? mine : seq_work<RT, 1>(A, base + lane);
        if (base + lane < c->seq) w.total = 0;
        const int64_t inc = warp_scan(w.total);
        const unsigned hit = __ballot_sync(0xffffffffu, u < acc + inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            c->seq = base + src;
            c->begin = acc + __shfl_sync(0xffffffffu, inc - w.total, src);
            c->w.s.start = __shfl_sync(0xffffffffu, w.s.start, src);
            c->w.s.n = __shfl_sync(0xffffffffu, w.s.n, src);
            c->w.s.len = __shfl_sync(0xffffffffu, w.s.len, src);
            c->w.lo = __shfl_sync(0xffffffffu, w.lo, src);
            c->w.tiles = __shfl_sync(0xffffffffu, w.tiles, src);
            c->w.units = __shfl_sync(0xffffffffu, w.units, src);
            c->w.total = __shfl_sync(0xffffffffu, w.total, src);
            return true;
        }
        acc += __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}
template <int RT>
__device__ __forceinline__ int64_t total_work(const AttnParams& A, const SeqWork& mine) {
    int64_t t = mine.total;
    for (int i = 32 + (threadIdx.x & 31); i < A.B.batch; i += 32) t += seq_work<RT, 1>(A, i).total;
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}
// 64-bit values that mostly fit 32: the short division where they do.
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// What cluster (or CTA) `c` of `clusters` works on, `mine` being the work of sequence `lane`: a tile's units are shared by k clusters, k in proportion to its length but
// at least one, and at least kLeast units a cluster; no cluster takes a part of two tiles.
struct TilePart {
    int index, k;  // the tile among its sequence's (row tile, kv head), and its clusters
    int first, j;  // its first cluster; this one's number among them
    bool more;     // there are more tiles than clusters, which then walk over them, a whole one at a time
};
template <int RT, int CL>
__device__ __forceinline__ bool tile_part(const AttnParams& A, const SeqWork& mine, int c, int clusters, Cursor* cur, TilePart* p) {
    const int lane = threadIdx.x & 31;
    int64_t tiles = (int64_t)mine.tiles * A.kv_heads, units = tiles * mine.units;
    for (int i = 32 + lane; i < A.B.batch; i += 32) {
        const SeqWork w = seq_work<RT, CL>(A, i);
        tiles += (int64_t)w.tiles * A.kv_heads;
        units += (int64_t)w.tiles * A.kv_heads * w.units;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        units += __shfl_xor_sync(0xffffffffu, units, o);
    }
    const int64_t spare = max(clusters - tiles, (int64_t)0);
    p->more = tiles > clusters;
    int64_t acc = 0;
    for (int base = 0; base < A.B.batch; base += 32) {
        const SeqWork w = base == 0 ? mine : seq_work<RT, CL>(A, base + lane);
        const int k = w.tiles ? min(1 + (int)div_pos(w.units * spare, units), w.units <= kJoinCost ? 1 : w.units / kLeast) : 1;
        const int64_t own = (int64_t)w.tiles * A.kv_heads * k, inc = warp_scan(own);
        const unsigned hit = __ballot_sync(0xffffffffu, c < acc + inc);
        if (hit) {
            const int src = __ffs(hit) - 1, begin = (int)(acc + __shfl_sync(0xffffffffu, inc - own, src));
            cur->seq = base + src;
            cur->w.s.start = __shfl_sync(0xffffffffu, w.s.start, src);
            cur->w.s.n = __shfl_sync(0xffffffffu, w.s.n, src);
            cur->w.s.len = __shfl_sync(0xffffffffu, w.s.len, src);
            cur->w.lo = __shfl_sync(0xffffffffu, w.lo, src);
            cur->w.tiles = __shfl_sync(0xffffffffu, w.tiles, src);
            cur->w.units = __shfl_sync(0xffffffffu, w.units, src);
            p->k = __shfl_sync(0xffffffffu, k, src);
            p->index = (c - begin) / p->k;
            p->j = (c - begin) - p->index * p->k;
            p->first = c - p->j;
            return true;
        }
        acc += __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}
// First unit of piece c when `total` units are cut into `pieces`.
__device__ __forceinline__ int64_t piece_begin(int64_t total, int pieces, int c) {
    const int64_t q = div_pos(total, pieces);
    return q * c + min((int64_t)c, total - q * pieces);
}
__device__ __forceinline__ int piece_of(int64_t total, int pieces, int64_t u) {
    const int64_t q = div_pos(total, pieces), r = total - q * pieces;
    return (int)(u < r * (q + 1) ? div_pos(u, q + 1) : r + div_pos(u - r * (q + 1), q));
}

// A counter of this launch, whatever an earlier one or anything else left in its word (`seen`): 48 bits of the launch's
// tag, 16 of count. Every CTA that will arrive sees to the tag before (only this launch's CTAs change the word, all to
// the same, so the second look finds it), so that arriving is one addition.
__device__ __forceinline__ void open_counter(unsigned long long* w, unsigned long long tag, unsigned long long seen) {
    while ((seen >> 16) != tag) {
        const unsigned long long was = atomicCAS(w, seen, tag << 16);
        if (was == seen) return;
        seen = was;
    }
}
__device__ __forceinline__ int arrive(unsigned long long* w) {  // how many had arrived before
    return (int)(atomicAdd(w, 1ull) & 0xFFFFu);
}

// Clusters (CL CTAs that work as one).
__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
template <int CL> __device__ __forceinline__ void sync_all() {  // the CTA, or the cluster's CTAs
    if constexpr (CL == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A word of the shared memory of CTA `rank` of the cluster, at the place of `p` in this one's.
__device__ __forceinline__ float peer_f32(const float* p, int rank) {
    float v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
        : "=f"(v)
        : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank)
        : "memory");
    return v;
}

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

// RT: query rows of a tile. fp32: 8 (two fp16 terms fill the 16 rows); bf16: 8 where a tile has no
// more rows, else 16.
template <typename T, int D, int RT, int CL>
__global__ void __launch_bounds__(32 * kAttnWarps, kCtasPerSm) attn_kernel(const __grid_constant__ AttnParams A) {
    constexpr bool HL = sizeof(T) == 4;           // two fp16 terms
    constexpr int NR = RT / 8;                    // rows of a thread: g, and g + 8
    static_assert(RT == 8 || (RT == 16 && !HL), "rows");
    constexpr int NT = D / 8;                     // output column tiles
    extern __shared__ __align__(128) uint8_t s_mem[];
    float* s_o = reinterpret_cast<float*>(s_mem); // [warps][RT][D], over the rings once they are read
    __shared__ float s_m[kAttnWarps * RT], s_l[kAttnWarps * RT];
    __shared__ ChunkMeta s_meta[kAttnWarps][kRing * kPair];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int rank = CL > 1 ? cluster_rank() : 0, my_piece = CL > 1 ? (int)blockIdx.x / CL : (int)blockIdx.x;
    __shared__ float s_xm[RT], s_xl[RT];  // the CTA's share of a tile, for its cluster: maxima, denominators, sums
    float* s_x = s_o + kAttnWarps * RT * D;
    // The first warp finds the piece and its segments; what the main loop does not need stays in
    // shared memory.
    __shared__ SeqWork s_work[32];
    __shared__ uint4 s_q[D / 16][32];  // the tile's query fragments, a 16-dim step of a lane each
    __shared__ Cursor s_cur;
    __shared__ int64_t s_u[2], s_total;
    __shared__ int s_pieces;
    __shared__ TilePart s_tile;
    __shared__ bool s_by_tile;
    __shared__ struct { int c0, slot0, size, groups, first, count, last; } s_join;
    if (warp == 0) {
        const SeqWork mine = seq_work<RT, CL>(A, lane);
        int longest = mine.units;
        int64_t tiles = (int64_t)mine.tiles * A.kv_heads;
        for (int i = 32 + lane; CL == 1 && i < A.B.batch; i += 32) {
            const SeqWork w = seq_work<RT, CL>(A, i);
            longest = max(longest, w.units);
            tiles += (int64_t)w.tiles * A.kv_heads;
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
        for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        // Joining a tile costs about as much as eight of its units: where no tile is longer, a CTA takes a whole one if
        // there are enough (128 tiles of up to 400 tokens: 13 us, cut into equal pieces 24).
        const bool by_tile = CL > 1 || (longest <= kJoinCost && tiles <= gridDim.x);
        if (lane == 0) s_by_tile = by_tile;
        if (by_tile) {
            Cursor c{};
            TilePart p{};
            const bool any = tile_part<RT, CL>(A, mine, my_piece, gridDim.x / CL, &c, &p);
            if (lane == 0) {
                s_cur = c;
                s_tile = p;
                s_u[0] = 0;
                s_u[1] = any;
            }
        } else {
            s_work[lane] = mine;
            const int64_t total = total_work<RT>(A, mine);
            // more such tiles than CTAs: pieces are not shorter than a whole one
            const int64_t least = longest <= kJoinCost ? kTileCost + longest : 1;
            const int pieces = (int)min((int64_t)min((int)gridDim.x, A.parts), div_pos(total + least - 1, least));
            const bool any = my_piece < pieces;
            const int64_t u0 = any ? piece_begin(total, pieces, my_piece) : 0;
            const int64_t u1 = any ? piece_begin(total, pieces, my_piece + 1) : 0;
            Cursor c{};
            if (any) seek<RT>(A, u0, mine, &c);
            if (lane == 0) {
                s_cur = c;
                s_u[0] = u0;
                s_u[1] = u1;
                s_total = total;
                s_pieces = pieces;
            }
        }
    }
    __syncthreads();
    uint8_t* ring = s_mem + warp * (kRing * kStage<D>);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    bool not_first = false;
    while (s_u[0] < s_u[1]) {
        const SeqSpan sp = s_cur.w.s;
        const int w_lo = s_cur.w.lo, seq = s_cur.seq;
        int tile, head, ua, ub, step = 0;
        const bool by_tile = CL > 1 || s_by_tile;
        if (by_tile) {
            ua = (int)((int64_t)s_cur.w.units * s_tile.j / s_tile.k);
            ub = (int)((int64_t)s_cur.w.units * (s_tile.j + 1) / s_tile.k);
            tile = s_tile.index / A.kv_heads;
            head = s_tile.index - tile * A.kv_heads;
        } else {
            const int64_t at = s_u[0] - s_cur.begin;
            const int length = kTileCost + s_cur.w.units;
            const int seg = (int)div_pos(at, length);  // (row tile, kv head) of the sequence
            const int va = (int)(at - (int64_t)seg * length);
            const int vb = (int)min((int64_t)length, va + (s_u[1] - s_u[0]));
            step = vb - va;
            ua = max(va - kTileCost, 0);
            ub = vb - kTileCost;  // <= 0: the piece ends before the tile's first unit
            tile = seg / A.kv_heads;
            head = seg - tile * A.kv_heads;
        }
        if (ub <= 0) break;
        const int rows = sp.n * A.group, first = sp.len - sp.n;
        const bool whole = ua == 0 && ub == s_cur.w.units;
        if (!whole && threadIdx.x == 32) {
            // the tile's pieces c0 .. c1, in groups of about the root of their number where they are many
            int c0, c1, slot0 = 0;
            if (by_tile) {
                c0 = s_tile.first;
                c1 = c0 + s_tile.k - 1;
            } else {
                const int length = kTileCost + s_cur.w.units;
                const int64_t begin = s_cur.begin + (int64_t)(tile * A.kv_heads + head) * length;
                c0 = piece_of(s_total, s_pieces, begin + kTileCost);
                c1 = piece_of(s_total, s_pieces, begin + length - 1);
                slot0 = piece_begin(s_total, s_pieces, c0) >= begin ? 0 : 1;
            }
            const int np = c1 - c0 + 1, size = np <= kOneLevel ? np : (int)ceilf(sqrtf((float)np)), of = (my_piece - c0) / size;
            s_join.c0 = c0;
            s_join.slot0 = slot0;
            s_join.size = size;
            s_join.groups = (np + size - 1) / size;
            s_join.first = c0 + of * size;
            s_join.count = min(size, c1 + 1 - s_join.first);
        }

        // positions: some row of the tile sees tokens below tile_hi, all see those in [full_lo, full_hi)
        const int pf = first + tile * RT / A.group, pl = first + (min(rows, tile * RT + RT) - 1) / A.group;
        const int tile_hi = max(pl + 1, 0), full_hi = max(pf + 1, 0);
        const int full_lo = A.window > 0 ? max(pl - A.window + 1, 0) : 0;

        // this warp's chunks: base0 + kStep i, i < n
        constexpr int kStep = CL * kUnit;
        const int c_end = min(w_lo + ub * kStep, tile_hi);
        const int base0 = w_lo + ua * kStep + rank * kUnit + warp * kChunk;
        const int n = base0 < c_end ? (c_end - base0 + kStep - 1) / kStep : 0;
        auto entry_of = [&](int i) { return i < n ? page_entry(A.B, seq, (base0 + kStep * i) >> A.B.page_shift) : -1; };
        auto checked = [&](int i, int p) { return i < n ? page_checked(A.B, p, A.err_flag) : -1; };
        auto scales_of = [&](int pid, float& ks, float& vs) {
            ks = vs = 1.0f;
            if (pid >= 0) {
                ks = __ldcg(A.k_scale + (int64_t)pid * A.kv_heads + head);
                vs = __ldcg(A.v_scale + (int64_t)pid * A.kv_heads + head);
            }
        };
        // What a segment begins with is a chain of reads through L2, so each is issued before an earlier one is
        // looked at: page ids, the tile's queries, the counters, the first copies, scales.
        PageAhead ah{entry_of(lane), entry_of(32 + lane), entry_of(64 + lane), 1.f, 1.f, 1.f, 1.f};
        float x[NR][D / 64][16];
        // a row's token, its dims 64 h + 16 t ..; rows past the last one read the first one's
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const int r = tile * RT + g + 8 * j < rows ? tile * RT + g + 8 * j : 0;
            const T* p = static_cast<const T*>(A.q) + (int64_t)(sp.start + r / A.group) * A.q_stride +
                         (int64_t)(head * A.group + r % A.group) * D + 16 * t;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) Vec<T>::load(p + 64 * h, x[j][h]);
        }
        unsigned long long seen[2] = {};
        const bool opens = !whole && threadIdx.x == 32 && rank == 0;
        if (opens) {
            seen[0] = *reinterpret_cast<volatile unsigned long long*>(A.tickets + s_join.first);
            seen[1] = *reinterpret_cast<volatile unsigned long long*>(A.tickets + kMaxParts + s_join.c0);
        }
        ah.p0 = checked(lane, ah.p0);
        ah.p1 = checked(32 + lane, ah.p1);
        ah.p2 = checked(64 + lane, ah.p2);
        const int n_st = (n + kPair - 1) / kPair;
        auto issue = [&](int k) {  // the copies of stage k (a group of its own, empty past the last stage)
#pragma unroll
            for (int c = 0; c < kPair; ++c) {
                const int i = kPair * k + c;
                if (i > 0 && (i & 31) == 0) {
                    ah.p0 = ah.p1; ah.ks0 = ah.ks1; ah.vs0 = ah.vs1;
                    ah.p1 = ah.p2;
                    scales_of(ah.p1, ah.ks1, ah.vs1);
                    ah.p2 = checked(i + 64 + lane, entry_of(i + 64 + lane));
                }
                const int pid = __shfl_sync(0xffffffffu, ah.p0, i & 31);  // -1 past the last chunk
                if (pid < 0) continue;
                const int slot = (base0 + kStep * i) & ((1 << A.B.page_shift) - 1);
                const int64_t at = ((((int64_t)pid * A.kv_heads + head) << A.B.page_shift) + slot) * D + 16 * lane;
                const uint32_t dst = ring_at + k % kRing * kStage<D> + c * kSlot<D>;
                constexpr int kUnits = D / 16, kRows = 32 / kUnits;  // a row's units; rows of one copy instruction
#pragma unroll
                for (int j = 0; j < kChunk / kRows; ++j) {
                    const int r = kRows * j + lane / kUnits, u = lane % kUnits;
                    copy16(dst + k_unit<D>(r, u), A.k_cache + at + 512 * j);
                    copy16(dst + kChunk * D + v_unit<D>(r, u), A.v_cache + at + 512 * j);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto note = [&](int k) {  // their scales, after the copies are on their way
            const int c = (lane - kPair * k) & 31;
            if (c < kPair)
                s_meta[warp][k % kRing * kPair + c] = ChunkMeta{ah.ks0, scale_log2_of(ah.vs0), 1.0f / ah.vs0, ah.p0 >= 0};
        };
        for (int k = 0; k < kRing; ++k) issue(k);
        scales_of(ah.p0, ah.ks0, ah.vs0);
        scales_of(ah.p1, ah.ks1, ah.vs1);

        // the thread's rows: position limits and query fragments
        int hi[NR], lo[NR];
        float crow[NR];
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const int r = tile * RT + g + 8 * j;
            const bool valid = r < rows;
            const int tok = valid ? r / A.group : 0;
            const int pos = first + tok;
            hi[j] = valid ? pos + 1 : 0;
            lo[j] = A.window > 0 ? max(pos - A.window + 1, 0) : 0;
            float amax = 0.0f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (!valid) x[j][h][i] = 0.0f;
                    const float a = fabsf(x[j][h][i]);
                    if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // power of two that brings the row's largest magnitude to [2^7, 2^8)
            const int e = amax > 0.0f ? min(max(134 - (int)(__float_as_uint(amax) >> 23), -120), 120) : 0;
            const float up = exp2_int(e);
            crow[j] = A.scale_log2 * exp2_int(-e);
            // the warps share the packing: a fourth of the steps each
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i != warp) continue;
                    const float a0 = x[j][h][4 * i] * up, a1 = x[j][h][4 * i + 1] * up;
                    const float a2 = x[j][h][4 * i + 2] * up, a3 = x[j][h][4 * i + 3] * up;
                    uint4 f;
                    if constexpr (HL) {
                        const __half2 h01 = __floats2half2_rn(a0, a1), h23 = __floats2half2_rn(a2, a3);
                        const float2 b01 = __half22float2(h01), b23 = __half22float2(h23);
                        f.x = *reinterpret_cast<const uint32_t*>(&h01);
                        f.z = *reinterpret_cast<const uint32_t*>(&h23);
                        f.y = pack_f16(a0 - b01.x, a1 - b01.y);
                        f.w = pack_f16(a2 - b23.x, a3 - b23.y);
                        s_q[4 * h + i][lane] = f;
                    } else if (RT == 8) {  // rows 8-15 of the products are not used
                        s_q[4 * h + i][lane] = make_uint4(pack_f16(a0, a1), 0, pack_f16(a2, a3), 0);
                    } else if (j == 0) {
                        s_q[4 * h + i][lane].x = pack_f16(a0, a1);
                        s_q[4 * h + i][lane].z = pack_f16(a2, a3);
                    } else {
                        s_q[4 * h + i][lane].y = pack_f16(a0, a1);
                        s_q[4 * h + i][lane].w = pack_f16(a2, a3);
                    }
                }
        }
        static_assert(kAttnWarps == 4, "a step of each 64 dims a warp");
        for (int k = 0; k < kRing; ++k) note(k);
        if (opens) {
            if (s_join.count > 1) open_counter(A.tickets + s_join.first, A.tag, seen[0]);
            if (s_join.groups > 1) open_counter(A.tickets + kMaxParts + s_join.c0, A.tag, seen[1]);
        }
        __syncthreads();

        float2 o[NT][NR];
        float mx[NR], l[NR];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < NR; ++j) o[n][j] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < NR; ++j) { mx[j] = -INFINITY; l[j] = 0.0f; }

        // a stage at a time: one maximum, one correction and one flush of the sums for its chunks
        constexpr int S = kPair;
        for (int k_st = 0; k_st < n_st; ++k_st) {
            const int stage = k_st % kRing, i = S * k_st;
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();
            // Tokens: lane t's of a chunk are 4 t + {0, 1, 2, 3}, columns 2 t, 2 t + 1 of score tiles 0 and 1, so
            // column c of tile j is token 4 (c / 2) + 2 j + c % 2.
            float x[S][NR][4];
            float inv[S];
            bool full[S], held[S];
            float s[S][2][4];
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                uint4 kf[S][2];
#pragma unroll
                for (int c = 0; c < S; ++c)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        kf[c][j] = *reinterpret_cast<const uint4*>(ring + stage * kStage<D> + c * kSlot<D> +
                                                                   k_unit<D>(4 * (g >> 1) + (g & 1) + 2 * j, 4 * h + t));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 qf = s_q[4 * h + q][lane];
                    const uint32_t qa[4] = {qf.x, qf.y, qf.z, qf.w};
#pragma unroll
                    for (int c = 0; c < S; ++c)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t kw[4] = {kf[c][j].x, kf[c][j].y, kf[c][j].z, kf[c][j].w};
                            uint32_t b0, b1;
                            e4m3x4_to_f16x4(kw[q], &b0, &b1);
                            if (h == 0 && q == 0) mma_16816_zero(s[c][j], qa, b0, b1);
                            else mma_16816(s[c][j], qa, b0, b1);
                        }
                }
            }
#pragma unroll
            for (int c = 0; c < S; ++c) {
                const int base = base0 + kStep * (i + c);
                const ChunkMeta meta = s_meta[warp][stage * S + c];
                // x = c * s + e, masked
                inv[c] = meta.inv;
                held[c] = meta.ok;
                full[c] = meta.ok && base >= full_lo && base + kChunk <= full_hi;
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    const float cr = crow[j] * meta.ks;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float sv = HL ? s[c][k >> 1][k & 1] + s[c][k >> 1][2 + (k & 1)] : s[c][k >> 1][2 * j + (k & 1)];
                        x[c][j][k] = fmaf(sv, cr, meta.ev);
                    }
                }
                if (!full[c]) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = base + 4 * t + k;
#pragma unroll
                        for (int j = 0; j < NR; ++j)
                            if (!meta.ok || tok < lo[j] || tok >= hi[j]) x[c][j][k] = -INFINITY;
                    }
                }
            }
            uint32_t pa[S][4];
            bool grew = false;
            float corr[NR];
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                float top = x[0][j][0];
#pragma unroll
                for (int c = 0; c < S; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k) top = fmaxf(top, x[c][j][k]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float m_new = fmaxf(mx[j], top);
                grew = grew || m_new > mx[j];
                const float m_use = m_new == -INFINITY ? 0.0f : m_new;
                const float base = __fadd_ru(m_use, -15.0f);  // rounded up: x - base is 15 at most
                corr[j] = ex2(mx[j] - m_use);
                mx[j] = m_new;
                l[j] *= corr[j];
#pragma unroll
                for (int c = 0; c < S; ++c) {
                    float sum = 0.0f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[c][j][k] = ex2(x[c][j][k] - base);
                        sum += x[c][j][k];
                    }
                    l[j] = fmaf(sum, inv[c], l[j]);
                }
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int j = 0; j < NR; ++j)
#pragma unroll
                    for (int k = 0; k < NT; ++k) mul2(o[k][j], corr[j]);
            }
            uint32_t vf[S][4][D / 32];
#pragma unroll
            for (int c = 0; c < S; ++c) {
                const uint8_t* vp = ring + stage * kStage<D> + c * kSlot<D> + kChunk * D;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (D == 128) {
                        const uint4 a = *reinterpret_cast<const uint4*>(vp + v_unit<D>(4 * t + r, g));
                        vf[c][r][0] = a.x; vf[c][r][1] = a.y; vf[c][r][2] = a.z; vf[c][r][3] = a.w;
                    } else {
                        const uint2 a = *reinterpret_cast<const uint2*>(vp + v_unit<D>(4 * t + r, g >> 1) + 8 * (g & 1));
                        vf[c][r][0] = a.x; vf[c][r][1] = a.y;
                    }
                }
            }
            __syncwarp();
            issue(k_st + kRing);
            note(k_st + kRing);
#pragma unroll
            for (int c = 0; c < S; ++c) {
                if constexpr (HL) {
                    const __half2 h0 = __floats2half2_rn(x[c][0][0], x[c][0][1]), h1 = __floats2half2_rn(x[c][0][2], x[c][0][3]);
                    const float2 b0 = __half22float2(h0), b1 = __half22float2(h1);
                    pa[c][0] = *reinterpret_cast<const uint32_t*>(&h0);
                    pa[c][2] = *reinterpret_cast<const uint32_t*>(&h1);
                    float2 r0 = make_float2(x[c][0][0], x[c][0][1]), r1 = make_float2(x[c][0][2], x[c][0][3]);
                    mul2(r0, 2048.0f);
                    mul2(r1, 2048.0f);
                    fma2(r0, b0.x, b0.y, -2048.0f);
                    fma2(r1, b1.x, b1.y, -2048.0f);
                    pa[c][1] = pack_f16(r0.x, r0.y);
                    pa[c][3] = pack_f16(r1.x, r1.y);
                } else {
                    pa[c][0] = pack_f16(x[c][0][0], x[c][0][1]);
                    pa[c][2] = pack_f16(x[c][0][2], x[c][0][3]);
                    pa[c][1] = RT == 8 ? 0 : pack_f16(x[c][NR - 1][0], x[c][NR - 1][1]);
                    pa[c][3] = RT == 8 ? 0 : pack_f16(x[c][NR - 1][2], x[c][NR - 1][3]);
                }
                if (!full[c]) {
                    // tokens that no row of the tile sees hold anything: NaN codes too
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = base0 + kStep * (i + c) + 4 * t + k;
                        if (!held[c] || tok >= tile_hi || tok < w_lo)
#pragma unroll
                            for (int q = 0; q < D / 32; ++q) vf[c][k][q] = 0;
                    }
                    // a token that only some rows see may hold NaN, which 0 * NaN would spread
                    uint32_t bad = 0;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int q = 0; q < D / 32; ++q) bad |= nan_bytes(vf[c][r][q]);
                    if (__any_sync(0xffffffffu, bad != 0)) {
                        // which rows see which tokens, times which codes are NaN: NaN where the product counts one
                        uint32_t see[4] = {};
#pragma unroll
                        for (int j = 0; j < NR; ++j)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int tok = base0 + kStep * (i + c) + 4 * t + k;
                                if (tok >= lo[j] && tok < hi[j]) see[2 * (k >> 1) + j] |= 0x3C00u << (16 * (k & 1));
                            }
#pragma unroll
                        for (int q = 0; q < D / 32; ++q)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t b[2];
#pragma unroll
                                for (int r = 0; r < 2; ++r)
                                    b[r] = ((nan_bytes(vf[c][2 * r][q]) >> (8 * k + 7) & 1u) ? 0x3C00u : 0u) |
                                           ((nan_bytes(vf[c][2 * r + 1][q]) >> (8 * k + 7) & 1u) ? 0x3C000000u : 0u);
                                float acc[4] = {};
                                mma_16816(acc, see, b[0], b[1]);
#pragma unroll
                                for (int j = 0; j < NR; ++j) {
                                    if (acc[2 * j] > 0.0f) o[4 * q + k][j].x = __int_as_float(0x7FC00000);
                                    if (acc[2 * j + 1] > 0.0f) o[4 * q + k][j].y = __int_as_float(0x7FC00000);
                                }
                            }
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int q = 0; q < D / 32; ++q) vf[c][r][q] &= ~((nan_bytes(vf[c][r][q]) >> 7) * 0xFFu);
                    }
                }
            }
            // sums: column tile 4 q + {0..3}, this lane's dims D/8 g + 4 q ..
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t b0[S][4], b1[S][4];
#pragma unroll
                for (int c = 0; c < S; ++c) {
                    e4m3x4_to_f16x4(__byte_perm(vf[c][0][q], vf[c][1][q], 0x5140), &b0[c][0], &b0[c][1]);
                    e4m3x4_to_f16x4(__byte_perm(vf[c][0][q], vf[c][1][q], 0x7362), &b0[c][2], &b0[c][3]);
                    e4m3x4_to_f16x4(__byte_perm(vf[c][2][q], vf[c][3][q], 0x5140), &b1[c][0], &b1[c][1]);
                    e4m3x4_to_f16x4(__byte_perm(vf[c][2][q], vf[c][3][q], 0x7362), &b1[c][2], &b1[c][3]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // A fresh accumulator for each stage, added in fp32: the tensor core's own accumulation does
                    // not round to nearest, which shows over long caches; and rows 8-15 hold the low terms
                    // of the same rows (fp32) or nothing (RT 8), so half the registers carry the sums.
                    float acc[4];
                    mma_16816_zero(acc, pa[0], b0[0][k], b1[0][k]);
#pragma unroll
                    for (int c = 1; c < S; ++c) mma_16816(acc, pa[c], b0[c][k], b1[c][k]);
                    add2(o[4 * q + k][0], acc[0], acc[1]);
                    if (HL) fma2(o[4 * q + k][0], acc[2], acc[3], 1.0f / 2048.0f);
                    if (RT == 16) add2(o[4 * q + k][NR - 1], acc[2], acc[3]);
                }
            }
        }
        // join the warps: each row's maximum, then the weighted sums
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
            if (t == 0) {
                s_m[warp * RT + g + 8 * j] = mx[j];
                s_l[warp * RT + g + 8 * j] = l[j];
            }
            // this lane's dims: D/8 (2 t) + n and D/8 (2 t + 1) + n, n = 0 .. NT - 1; 16-byte units xored with the
            // lane, or the eight lanes of a store would meet the same banks
            float4* d0 = reinterpret_cast<float4*>(s_o + (warp * RT + g + 8 * j) * D);
#pragma unroll
            for (int n = 0; n < NT; n += 4) {
                const int u = D / 16 * t + n / 4, x = (2 * t + (g & 1)) & 7;
                d0[u ^ x] = make_float4(o[n][j].x, o[n + 1][j].x, o[n + 2][j].x, o[n + 3][j].x);
                d0[(u + D / 32) ^ x] = make_float4(o[n][j].y, o[n + 1][j].y, o[n + 2][j].y, o[n + 3][j].y);
            }
        }
        __syncthreads();
        // a tile that begins in this piece, but not at its start, goes to the second slot
        constexpr int kPart = RT * (D + 2);
        float* part = A.part + ((int64_t)my_piece * 2 + (not_first ? 1 : 0)) * kPart;
        auto store_row = [&](int r, int c, const float4& acc, float den) {
            const int row = tile * RT + r;
            if (row >= rows) return;
            const float iv = den == 0.0f ? 0.0f : 1.0f / den;  // 0: the row sees nothing
            const float y[4] = {acc.x * iv, acc.y * iv, acc.z * iv, acc.w * iv};
            Vec<T>::store(static_cast<T*>(A.out) + (int64_t)(sp.start + row / A.group) * A.out_stride +
                              (int64_t)(head * A.group + row % A.group) * D + c,
                          y);
        };
        for (int i = threadIdx.x; i < RT * D / 4; i += 32 * kAttnWarps) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4));
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) m = fmaxf(m, s_m[k * RT + r]);
            const float mu = m == -INFINITY ? 0.0f : m;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float den = 0.0f;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) {
                const float wt = ex2(s_m[k * RT + r] - mu);
                const int u = c / 4, x = (2 * (u / (D / 16)) + (r & 1)) & 7;
                const float4 v = reinterpret_cast<const float4*>(s_o + (k * RT + r) * D)[u ^ x];
                den = fmaf(wt, s_l[k * RT + r], den);
                acc.x = fmaf(wt, v.x, acc.x); acc.y = fmaf(wt, v.y, acc.y);
                acc.z = fmaf(wt, v.z, acc.z); acc.w = fmaf(wt, v.w, acc.w);
            }
            if constexpr (CL > 1) {
                *reinterpret_cast<float4*>(s_x + r * D + c) = acc;
                if (c == 0) {
                    s_xm[r] = m;
                    s_xl[r] = den;
                }
                continue;
            }
            if (whole) {
                store_row(r, c, acc, den);
            } else {
                *reinterpret_cast<float4*>(part + r * D + c) = acc;
                if (c == 0) {
                    part[RT * D + r] = m;
                    part[RT * D + RT + r] = den;
                }
            }
        }
        auto peer_or_own = [&](const float* x) {  // the cluster's first CTA's
            if constexpr (CL > 1) return peer_f32(x, 0);
            else return *x;
        };
        if constexpr (CL > 1) {
            // the cluster's shares: CTA `rank` joins rows rank, rank + CL, ...
            sync_all<CL>();
            for (int i = threadIdx.x; i < RT / CL * D; i += 32 * kAttnWarps) {
                const int r = rank + CL * (i / D), c = i % D;
                float xm[CL], xl[CL], xv[CL], m = -INFINITY;
#pragma unroll
                for (int k = 0; k < CL; ++k) {
                    xm[k] = peer_f32(s_xm + r, k);
                    xl[k] = peer_f32(s_xl + r, k);
                    xv[k] = peer_f32(s_x + r * D + c, k);
                }
#pragma unroll
                for (int k = 0; k < CL; ++k) m = fmaxf(m, xm[k]);
                const float mu = m == -INFINITY ? 0.0f : m;
                float acc = 0.0f, den = 0.0f;
#pragma unroll
                for (int k = 0; k < CL; ++k) {
                    const float wt = ex2(xm[k] - mu);
                    den = fmaf(wt, xl[k], den);
                    acc = fmaf(wt, xv[k], acc);
                }
                if (!whole) {
                    part[r * D + c] = acc;
                    if (c == 0) {
                        part[RT * D + r] = m;
                        part[RT * D + RT + r] = den;
                    }
                } else if (const int row = tile * RT + r; row < rows) {
                    const float y = den == 0.0f ? 0.0f : acc / den;  // 0: the row sees nothing
                    T* o = static_cast<T*>(A.out) + (int64_t)(sp.start + row / A.group) * A.out_stride +
                           (int64_t)(head * A.group + row % A.group) * D + c;
                    if constexpr (HL) *o = y;
                    else *o = __float2bfloat16_rn(y);
                }
            }
        }
        if (!whole) {
            auto last_to_arrive = [&](unsigned long long* w, int count) {  // every thread's results, then the counter
                sync_all<CL>();
                if (threadIdx.x == 0 && rank == 0) {
                    __threadfence();
                    s_join.last = arrive(w) == count - 1;
                    if (s_join.last) {
                        *reinterpret_cast<volatile unsigned long long*>(w) = A.tag << 16;  // for a replay of this launch
                        __threadfence();
                    }
                }
                sync_all<CL>();
                return __float_as_int(peer_or_own(reinterpret_cast<const float*>(&s_join.last))) != 0;
            };
            auto piece = [&](int i) { return A.part + ((int64_t)i * 2 + (i == s_join.c0 ? s_join.slot0 : 0)) * kPart; };
            // pieces first, first + step, ..: their weighted sum to the first one's slot, or to the output
            auto join = [&](int first, int step, int count, bool to_out) {
                float* pm = reinterpret_cast<float*>(s_mem);  // maxima, then denominators, [count][RT]
                float* pl = pm + count * RT;
                for (int i = threadIdx.x; i < count * RT; i += 32 * kAttnWarps) {
                    const float* x = piece(first + i / RT * step) + RT * D + i % RT;
                    pm[i] = __ldcg(x);
                    pl[i] = __ldcg(x + RT);
                }
                sync_all<CL>();  // the first piece's maxima and denominators are written over below: the whole cluster has them
                // a cluster's CTAs take the 16-byte units in turn
#pragma unroll 1
                for (int i = threadIdx.x * CL + rank; i < RT * D / 4; i += 32 * kAttnWarps * CL) {
                    const int r = i / (D / 4), c = 4 * (i % (D / 4));
                    float m = -INFINITY, den = 0.0f;
                    for (int k = 0; k < count; ++k) m = fmaxf(m, pm[k * RT + r]);
                    const float mu = m == -INFINITY ? 0.0f : m;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int k = 0; k < count; ++k) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(piece(first + k * step) + r * D + c));
                        const float wt = ex2(pm[k * RT + r] - mu);
                        den = fmaf(wt, pl[k * RT + r], den);
                        acc.x = fmaf(wt, v.x, acc.x); acc.y = fmaf(wt, v.y, acc.y);
                        acc.z = fmaf(wt, v.z, acc.z); acc.w = fmaf(wt, v.w, acc.w);
                    }
                    if (to_out) {
                        store_row(r, c, acc, den);
                        continue;
                    }
                    float* x = piece(first);
                    *reinterpret_cast<float4*>(x + r * D + c) = acc;
                    if (c == 0) {
                        x[RT * D + r] = m;
                        x[RT * D + RT + r] = den;
                    }
                }
            };
            // A group of one has no counter: its piece may be the next tile's first, whose counter is at the same place.
            if (s_join.count == 1 || last_to_arrive(A.tickets + s_join.first, s_join.count)) {
                if (s_join.count > 1) join(s_join.first, 1, s_join.count, s_join.groups == 1);
                if (s_join.groups > 1 && last_to_arrive(A.tickets + kMaxParts + s_join.c0, s_join.groups))
                    join(s_join.c0, s_join.size, s_join.groups, true);
            }
        }
        not_first = true;
        sync_all<CL>();  // what lies over the rings has been read, by the cluster too
        if (by_tile) {
            if (!s_tile.more) break;
            if (warp == 0) {
                Cursor c{};
                TilePart p{};
                const int clusters = gridDim.x / CL, next = s_tile.first + clusters;
                const bool any = tile_part<RT, CL>(A, seq_work<RT, CL>(A, lane), next, clusters, &c, &p);
                if (lane == 0) {
                    s_cur = c;
                    s_tile = p;
                    s_u[1] = any;
                }
            }
        } else if (warp == 0) {
            const int64_t u = s_u[0] + step;
            Cursor c = s_cur;
            __syncwarp();
            const bool more = u < s_u[1] && (u < c.begin + c.w.total || seek<RT>(A, u, s_work[lane], &c));
            if (lane == 0) {
                s_cur = c;
                s_u[0] = more ? u : s_u[1];
            }
        }
        __syncthreads();
    }
}

constexpr int kCluster = 8;

template <typename T, int D, int RT, int CL>
cudaError_t launch_cluster(const AttnParams& P, int max_len, cudaStream_t stream, int64_t segs, bool* fits) {
    const size_t rings = (size_t)kAttnWarps * kRing * kStage<D>, join = (size_t)(kAttnWarps + 1) * RT * D * sizeof(float);
    const size_t smem = rings > join ? rings : join;
    static std::atomic<int> clusters[64];  // what the device holds at once; 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(32 * kAttnWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    int most = clusters[dev].load(std::memory_order_relaxed);
    if (most == 0) {
        e = cudaFuncSetAttribute(attn_kernel<T, D, RT, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        most = P.parts;
        if (CL > 1) {
            cfg.gridDim = dim3(CL);
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, attn_kernel<T, D, RT, CL>, &cfg);
            if (e != cudaSuccess) return e;
            most = n < 1 ? 1 : n < P.parts ? n : P.parts;
        }
        clusters[dev].store(most, std::memory_order_relaxed);
    }
    if (CL > 1 && segs > most) {
        *fits = false;
        return cudaSuccess;
    }
    // no more CTAs or clusters than can share the tiles: the others would only look for work
    const int units = max_len / (CL * kUnit) + 1;
    int64_t grid = segs * (units <= kJoinCost ? 1 : CL > 1 ? units / kLeast : kTileCost + units);
    if (grid > most) grid = most;
    cfg.gridDim = dim3((unsigned)(grid * CL));
    return cudaLaunchKernelEx(&cfg, attn_kernel<T, D, RT, CL>, P);
}

template <typename T, int D, int RT>
cudaError_t launch_typed(const AttnParams& P, int64_t max_rows, int max_len, cudaStream_t stream) {
    const int64_t held = (int64_t)P.B.max_pages << P.B.page_shift;  // no sequence is longer than its table's row
    if (max_len > held) max_len = (int)held;
    // An upper bound of the row tiles: each sequence's last one may be part filled, and none has more than max_rows.
    const int64_t seqs = P.B.m < P.B.batch ? P.B.m : P.B.batch, full = (int64_t)P.B.m * P.group / RT;
    const int64_t each = max_rows > RT ? (max_rows + RT - 1) / RT : 1;
    const int64_t segs = (full + seqs < seqs * each ? full + seqs : seqs * each) * P.kv_heads;
    // Clusters where each tile finds one (51 at once on a GB300). 4 kv heads of 8 rows of fp32: one sequence of 1000 tokens
    // 8.5 us with, 12.9 without; of 16000 17.3 and 22.7; ten of 2000 13.0 and 17.6; 64 tiles of 1000 20.6 and 17.6.
    bool fits = true;
    const cudaError_t e = launch_cluster<T, D, RT, kCluster>(P, max_len, stream, segs, &fits);
    if (e != cudaSuccess || fits) return e;
    return launch_cluster<T, D, RT, 1>(P, max_len, stream, segs, nullptr);
}

// A value that no other launch of the process has (and, from a start that differs, hardly any other process's).
unsigned long long next_tag() {
    static std::atomic<unsigned long long> n{0};
    static const unsigned long long start =
        (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15ull ^
        reinterpret_cast<uintptr_t>(&n);
    return (start + n.fetch_add(1, std::memory_order_relaxed)) & 0xFFFFFFFFFFFFull;
}

}  // namespace

size_t attn_workspace_bytes(int head_dim) {  // the counters, then two slots of up to 16 rows per CTA
    return kTickets * sizeof(unsigned long long) + (size_t)kMaxParts * 2 * 16 * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_attention(const PagedBatch& B, const void* q, int dtype, int64_t q_stride, int q_heads, int kv_heads,
                             int head_dim, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                             const float* v_scale, int max_q_len, int max_len, float scale, int window, void* out,
                             int64_t out_stride, void* workspace, int* err_flag, cudaStream_t stream) {
    if (window >= 1 << 30) window = 0;  // no sequence is longer: every row sees all before it
    // Which kernel a sequence takes goes by its query rows per kv head; max_q_len says which kernels can
    // be needed, and a kernel that is launched alone takes every sequence.
    const int64_t most = (int64_t)max_q_len * (q_heads / kv_heads);
    const bool prompts = most > kFewRows && (int64_t)B.m * q_heads > 8 * kFewTiles;
    const bool few = !prompts || !(B.batch == 1 || B.m == (int64_t)B.batch * max_q_len);
    if (prompts) {
        const cudaError_t e = launch_attention_prompt(B, q, dtype, q_stride, q_heads, kv_heads, head_dim, k_cache, v_cache,
                                                      k_scale, v_scale, few ? kFewRows + 1 : 1, scale, window, out,
                                                      out_stride, err_flag, stream);
        if (e != cudaSuccess || !few) return e;
    }
    AttnParams P{};
    P.B = B; P.q = q; P.out = out; P.q_stride = q_stride; P.out_stride = out_stride;
    P.k_cache = k_cache; P.v_cache = v_cache; P.k_scale = k_scale; P.v_scale = v_scale;
    P.kv_heads = kv_heads; P.group = q_heads / kv_heads; P.window = window;
    P.scale_log2 = scale * 1.44269504088896340736f;
    P.tickets = static_cast<unsigned long long*>(workspace);
    P.tag = next_tag();
    P.part = reinterpret_cast<float*>(P.tickets + kTickets);
    P.parts = num_sms() * kCtasPerSm < kMaxParts ? num_sms() * kCtasPerSm : kMaxParts;
    P.err_flag = err_flag;
    P.max_rows = prompts ? kFewRows : 0x7FFFFFFF;
    const int64_t rows = prompts ? kFewRows : most;  // of a sequence, per kv head
    if (dtype == Q4K_F32)
        return head_dim == 64 ? launch_typed<float, 64, 8>(P, rows, max_len, stream) : launch_typed<float, 128, 8>(P, rows, max_len, stream);
    // bf16: tiles of 8 rows where a sequence's rows fit one (half the softmax), else 16; next to prompts
    // the other sequences mostly decode
    if ((prompts ? P.group : most) <= 8)
        return head_dim == 64 ? launch_typed<__nv_bfloat16, 64, 8>(P, rows, max_len, stream)
                              : launch_typed<__nv_bfloat16, 128, 8>(P, rows, max_len, stream);
    return head_dim == 64 ? launch_typed<__nv_bfloat16, 64, 16>(P, rows, max_len, stream)
                          : launch_typed<__nv_bfloat16, 128, 16>(P, rows, max_len, stream);
}

}  // namespace q4k
