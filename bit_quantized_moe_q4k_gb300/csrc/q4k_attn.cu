// q4k_attn.cu -- attention over the paged 8-bit cache for few query rows per kv head (decoding).
//
//   out[r] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q_r . k_j)  over the tokens j that row r sees
//
// With everything in powers of two and V's page scale 2^e_j inside the exponent,
//   x_j = c * (code_k . q) * ks_j + e_j,   P_j = 2^(x_j - M),  M the running maximum of x,
//   l = sum_j 2^(-e_j) P_j,   out = sum_j P_j code_v,j / l,
// so the codes of both sides enter the matrix products as they are: e4m3 is exact in fp16. Query
// rows are the M side of mma.m16n8k16: fp32 queries are split into two fp16 halves (hi in rows 0-7,
// lo in rows 8-15, scaled by a power of two so that 22 bits survive) and so are their P; bf16
// queries are exact in one half and P is rounded to fp16 (2^-12), so 16 rows fill the tile.
//
// Bound by the cache's bytes. Each warp reads 16 tokens of a page at a time straight into the
// fragments (16-byte loads, whole 128-byte lines) while the previous 16 are multiplied; nothing goes
// through shared memory. The work (sequence, kv head, row tile, 64 tokens) is laid out on one line and cut
// into equal pieces, one per CTA, whatever the lengths; a second kernel joins the pieces of a tile.
#include "q4k_paged.cuh"

namespace q4k {
namespace {

constexpr int kAttnWarps = 4;
constexpr int kChunk = 16;                    // tokens a warp takes at a time
constexpr int kUnit = kChunk * kAttnWarps;    // tokens of one piece of work
constexpr int kCtasPerSm = 3;
constexpr int kMaxParts = 512;                // CTAs that the workspace serves

struct AttnParams {
    PagedBatch B;
    const void* q;
    void* out;
    int64_t q_stride, out_stride;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int q_heads, kv_heads, group;
    int window;
    float scale_log2;   // softmax scale * log2(e)
    float* part;        // partial results: per CTA two slots of [rows][D] sums, rows M, rows l
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

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 0x80 in each byte that is one of e4m3's two NaN codes (0x7F, 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) { return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// The work of one sequence: `tiles` row tiles per kv head, `units` pieces of kUnit tokens each,
// from token `lo` (a multiple of kChunk: the first one any of its rows sees).
struct SeqWork {
    SeqSpan s;
    int lo, tiles, units;
    int64_t total;
};
template <int RT>
__device__ __forceinline__ SeqWork seq_work(const AttnParams& A, int i) {
    SeqWork w{};
    if (i >= A.B.batch) return w;
    bool bad;
    w.s = seq_span(A.B, i, &bad);
    if (bad) raise_flag(A.err_flag, Q4K_ERR_SEQ);
    if (w.s.n == 0) return w;
    const int first = max(w.s.len - w.s.n, 0);
    w.lo = A.window > 0 ? (max(first - A.window + 1, 0) & ~(kChunk - 1)) : 0;
    w.tiles = (w.s.n * A.group + RT - 1) / RT;
    w.units = max((w.s.len - w.lo + kUnit - 1) / kUnit, 1);  // an empty sequence: its rows are zeroed
    w.total = (int64_t)w.tiles * A.kv_heads * w.units;
    return w;
}

// A place on the line of work: the sequence that holds it and the line's position where that
// sequence begins. Every lane of the warp holds the same values.
struct Cursor {
    int seq;
    int64_t begin;
    SeqWork w;
};
// Move the cursor to the sequence that holds u (u >= c.begin; false past the end).
template <int RT>
__device__ __forceinline__ bool seek(const AttnParams& A, int64_t u, Cursor* c) {
    const int lane = threadIdx.x & 31;
    int64_t acc = c->begin;
    for (int base = c->seq; base < A.B.batch; base += 32) {
        const SeqWork w = seq_work<RT>(A, base + lane);
        int64_t inc = w.total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
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
__device__ __forceinline__ int64_t total_work(const AttnParams& A) {
    int64_t t = 0;
    for (int i = threadIdx.x & 31; i < A.B.batch; i += 32) t += seq_work<RT>(A, i).total;
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}
// First unit of piece c when `total` units are cut into `pieces`.
__device__ __forceinline__ int64_t piece_begin(int64_t total, int pieces, int c) {
    return total / pieces * c + min((int64_t)c, total % pieces);
}
__device__ __forceinline__ int piece_of(int64_t total, int pieces, int64_t u) {
    const int64_t q = total / pieces, r = total % pieces;
    return (int)(u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q);
}

// What a warp loads for 16 tokens: K words of its token rows, V words, and the page's scales.
template <int D>
struct Frag {
    uint4 k[2][D / 64];
    uint32_t v[4][D / 32];
    float ks, vs;
    bool ok;
};

template <int D>
__device__ __forceinline__ void load_frag(const AttnParams& A, int seq, int head, int base, int len, Frag<D>& f) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    f.ok = false;
    f.ks = f.vs = 1.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) f.k[i][h] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) f.v[i][j] = 0;
    if (base >= len) return;
    const int pid = page_id(A.B, seq, base >> A.B.page_shift, A.err_flag);
    if (pid < 0) return;
    f.ok = true;
    const int64_t ph = (int64_t)pid * A.kv_heads + head;
    f.ks = __ldcg(A.k_scale + ph);
    f.vs = __ldcg(A.v_scale + ph);
    const int slot = base & ((1 << A.B.page_shift) - 1);
    const int64_t at = ((ph << A.B.page_shift) + slot) * D;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            f.k[i][h] = __ldcg(reinterpret_cast<const uint4*>(A.k_cache + at + (8 * i + g) * D + 64 * h + 16 * t));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t* p = A.v_cache + at + (2 * t + (i & 1) + 8 * (i >> 1)) * D + D / 8 * g;
        if constexpr (D == 128) {
            const uint4 x = __ldcg(reinterpret_cast<const uint4*>(p));
            f.v[i][0] = x.x; f.v[i][1] = x.y; f.v[i][2] = x.z; f.v[i][3] = x.w;
        } else {
            const uint2 x = __ldcg(reinterpret_cast<const uint2*>(p));
            f.v[i][0] = x.x; f.v[i][1] = x.y;
        }
    }
}

// log2 of a page's V scale: exact for the powers of two that the append writes.
__device__ __forceinline__ float scale_log2_of(float s) {
    const uint32_t b = __float_as_uint(s);
    const float e = (float)((int)(b >> 23) - 127);
    return (b & 0x7FFFFFu) ? e + log2f(__uint_as_float((b & 0x7FFFFFu) | 0x3F800000u)) : e;
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kAttnWarps, kCtasPerSm) attn_kernel(const __grid_constant__ AttnParams A) {
    constexpr bool HL = sizeof(T) == 4;           // two fp16 terms
    constexpr int RT = HL ? 8 : 16;               // query rows of a tile
    constexpr int NR = HL ? 1 : 2;                // rows of a thread: g, and g + 8
    constexpr int NT = D / 8;                     // output column tiles
    extern __shared__ __align__(16) float s_mem[];
    float* s_o = s_mem;                           // [warps][RT][D]
    float* s_m = s_o + kAttnWarps * RT * D;       // [warps][RT]
    float* s_l = s_m + kAttnWarps * RT;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int64_t total = total_work<RT>(A);
    const int pieces = (int)min((int64_t)min((int)gridDim.x, A.parts), total);
    if ((int)blockIdx.x >= pieces) return;
    const int64_t u0 = piece_begin(total, pieces, blockIdx.x), u1 = piece_begin(total, pieces, blockIdx.x + 1);
    Cursor cur{};
    for (int64_t u = u0; u < u1;) {
        if (!seek<RT>(A, u, &cur)) return;
        const SeqWork w = cur.w;
        const int seg = (int)((u - cur.begin) / w.units);      // (row tile, kv head) of the sequence
        const int ua = (int)((u - cur.begin) % w.units);
        const int ub = (int)min((int64_t)w.units, ua + (u1 - u));
        const int tile = seg / A.kv_heads, head = seg % A.kv_heads;
        const int rows = w.s.n * A.group, first = w.s.len - w.s.n;

        // the thread's rows: position limits and query fragments
        int hi[NR], lo[NR];
        float crow[NR];
        uint32_t qa[D / 16][4];
        int tile_hi = 0, full_lo = 0, full_hi = 0x7FFFFFFF;
        {
            const int r0 = tile * RT, r1 = min(rows, r0 + RT) - 1;
            const int pf = first + r0 / A.group, pl = first + r1 / A.group;
            tile_hi = max(pl + 1, 0);
            full_hi = max(pf + 1, 0);
            full_lo = A.window > 0 ? max(pl - A.window + 1, 0) : 0;
        }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const int r = tile * RT + g + 8 * j;
            const bool valid = r < rows;
            const int tok = valid ? r / A.group : 0;
            const int pos = first + tok;
            hi[j] = valid ? pos + 1 : 0;
            lo[j] = A.window > 0 ? max(pos - A.window + 1, 0) : 0;
            float x[D / 64][16];
            float amax = 0.0f;
            const T* p = static_cast<const T*>(A.q) + (int64_t)(w.s.start + tok) * A.q_stride +
                         (int64_t)(head * A.group + (valid ? r % A.group : 0)) * D + 16 * t;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                Vec<T>::load(p + 64 * h, x[h]);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (!valid) x[h][i] = 0.0f;
                    const float a = fabsf(x[h][i]);
                    if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
                }
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // power of two that brings the row's largest magnitude to [2^7, 2^8)
            const int e = amax > 0.0f ? min(max(134 - (int)(__float_as_uint(amax) >> 23), -120), 120) : 0;
            const float up = exp2_int(e);
            crow[j] = A.scale_log2 * exp2_int(-e);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a0 = x[h][4 * i] * up, a1 = x[h][4 * i + 1] * up;
                    const float a2 = x[h][4 * i + 2] * up, a3 = x[h][4 * i + 3] * up;
                    uint32_t (&f)[4] = qa[4 * h + i];
                    if constexpr (HL) {
                        const __half2 h01 = __floats2half2_rn(a0, a1), h23 = __floats2half2_rn(a2, a3);
                        const float2 b01 = __half22float2(h01), b23 = __half22float2(h23);
                        f[0] = *reinterpret_cast<const uint32_t*>(&h01);
                        f[2] = *reinterpret_cast<const uint32_t*>(&h23);
                        f[1] = pack_f16(a0 - b01.x, a1 - b01.y);
                        f[3] = pack_f16(a2 - b23.x, a3 - b23.y);
                    } else {
                        f[j] = pack_f16(a0, a1);
                        f[2 + j] = pack_f16(a2, a3);
                    }
                }
        }

        float o[NT][HL ? 2 : 4];
        float mx[NR], l[NR];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < (HL ? 2 : 4); ++i) o[n][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < NR; ++j) { mx[j] = -INFINITY; l[j] = 0.0f; }

        const int c_end = min(w.lo + ub * kUnit, tile_hi);
        int base = w.lo + ua * kUnit + warp * kChunk;
        Frag<D> f;
        load_frag<D>(A, cur.seq, head, base, c_end, f);
        for (; base < c_end; base += kUnit) {
            Frag<D> nx;
            load_frag<D>(A, cur.seq, head, base + kUnit, c_end, nx);
            // scores: two tiles of 8 tokens
            float s[2][4] = {};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    const uint32_t kw[4] = {f.k[i][h].x, f.k[i][h].y, f.k[i][h].z, f.k[i][h].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mma_16816(s[i], qa[4 * h + q], e4m3x2_to_f16x2(kw[q] & 0xFFFFu), e4m3x2_to_f16x2(kw[q] >> 16));
                }
            // x = c * s + e, masked: this lane's tokens base + 8 i + 2 t + {0, 1}
            const float ev = scale_log2_of(f.vs), inv = 1.0f / f.vs;
            const bool full = f.ok && base >= full_lo && base + kChunk <= full_hi;
            float x[NR][4];
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const float c = crow[j] * f.ks;
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float sv = HL ? s[i >> 1][i & 1] + s[i >> 1][2 + (i & 1)] : s[i >> 1][2 * j + (i & 1)];
                    x[j][i] = fmaf(sv, c, ev);
                    if (!full) {
                        const int tok = base + 8 * (i >> 1) + 2 * t + (i & 1);
                        if (!f.ok || tok < lo[j] || tok >= hi[j]) x[j][i] = -INFINITY;
                    }
                    top = fmaxf(top, x[j][i]);
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float m_new = fmaxf(mx[j], top);
                const float m_use = m_new == -INFINITY ? 0.0f : m_new;
                const float corr = ex2(mx[j] - m_use);
                mx[j] = m_new;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[j][i] = ex2(x[j][i] - m_use + 7.0f);  // P * 2^7: fp16 keeps more of the small ones
                    sum += x[j][i];
                }
                l[j] = fmaf(l[j], corr, sum * inv);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][HL ? 0 : 2 * j] *= corr;
                    o[n][HL ? 1 : 2 * j + 1] *= corr;
                }
            }
            uint32_t pa[4];
            if constexpr (HL) {
                const __half2 h0 = __floats2half2_rn(x[0][0], x[0][1]), h1 = __floats2half2_rn(x[0][2], x[0][3]);
                const float2 b0 = __half22float2(h0), b1 = __half22float2(h1);
                pa[0] = *reinterpret_cast<const uint32_t*>(&h0);
                pa[2] = *reinterpret_cast<const uint32_t*>(&h1);
                pa[1] = pack_f16(x[0][0] - b0.x, x[0][1] - b0.y);
                pa[3] = pack_f16(x[0][2] - b1.x, x[0][3] - b1.y);
            } else {
                pa[0] = pack_f16(x[0][0], x[0][1]);
                pa[1] = pack_f16(x[NR - 1][0], x[NR - 1][1]);
                pa[2] = pack_f16(x[0][2], x[0][3]);
                pa[3] = pack_f16(x[NR - 1][2], x[NR - 1][3]);
            }
            // tokens that no row of the tile sees hold anything: NaN codes too
            if (!full) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = base + 2 * t + (i & 1) + 8 * (i >> 1);
                    if (tok >= tile_hi || tok < w.lo)
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) f.v[i][j] = 0;
                }
                // and a token that only some rows see may hold NaN, which 0 * NaN would spread
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) bad |= nan_bytes(f.v[i][j]);
                if (__any_sync(0xffffffffu, bad != 0)) {
                    // which rows see which tokens, times which codes are NaN: NaN where the product counts one
                    uint32_t see[4] = {};
#pragma unroll
                    for (int j = 0; j < NR; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int tok = base + 8 * (i >> 1) + 2 * t + (i & 1);
                            if (tok >= lo[j] && tok < hi[j]) see[2 * (i >> 1) + j] |= 0x3C00u << (16 * (i & 1));
                        }
#pragma unroll
                    for (int wd = 0; wd < D / 32; ++wd)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t b[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                b[k] = ((nan_bytes(f.v[2 * k][wd]) >> (8 * i + 7) & 1u) ? 0x3C00u : 0u) |
                                       ((nan_bytes(f.v[2 * k + 1][wd]) >> (8 * i + 7) & 1u) ? 0x3C000000u : 0u);
                            float acc[4] = {};
                            mma_16816(acc, see, b[0], b[1]);
                            float (&oo)[HL ? 2 : 4] = o[4 * wd + i];
#pragma unroll
                            for (int k = 0; k < (HL ? 2 : 4); ++k)
                                if (acc[k] > 0.0f) oo[k] = __int_as_float(0x7FC00000);
                        }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) f.v[i][j] &= ~((nan_bytes(f.v[i][j]) >> 7) * 0xFFu);
                }
            }
            // sums: column tile 4 w + {0..3}, this lane's dims D/8 g + 4 w ..
#pragma unroll
            for (int wd = 0; wd < D / 32; ++wd) {
                const uint32_t a = __byte_perm(f.v[0][wd], f.v[1][wd], 0x5140), b = __byte_perm(f.v[0][wd], f.v[1][wd], 0x7362);
                const uint32_t c = __byte_perm(f.v[2][wd], f.v[3][wd], 0x5140), d = __byte_perm(f.v[2][wd], f.v[3][wd], 0x7362);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t p0 = i < 2 ? a : b, p1 = i < 2 ? c : d;
                    const uint32_t b0 = e4m3x2_to_f16x2((i & 1) ? p0 >> 16 : p0 & 0xFFFFu);
                    const uint32_t b1 = e4m3x2_to_f16x2((i & 1) ? p1 >> 16 : p1 & 0xFFFFu);
                    if constexpr (HL) {
                        // a zero accumulator for each 16 tokens, added in fp32: the tensor core's own
                        // accumulation does not round to nearest, which shows over long caches
                        float acc[4] = {};
                        mma_16816(acc, pa, b0, b1);
                        o[4 * wd + i][0] += acc[0] + acc[2];
                        o[4 * wd + i][1] += acc[1] + acc[3];
                    } else {
                        mma_16816(*reinterpret_cast<float (*)[4]>(&o[4 * wd + i][0]), pa, b0, b1);
                    }
                }
            }
            f = nx;
        }

        // join the warps: each row's maximum, then the weighted sums
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
            if (t == 0) {
                s_m[warp * RT + g + 8 * j] = mx[j];
                s_l[warp * RT + g + 8 * j] = l[j];
            }
            // this lane's dims: D/8 (2 t) + n and D/8 (2 t + 1) + n, n = 0 .. NT - 1
            float* d0 = s_o + (warp * RT + g + 8 * j) * D + D / 8 * 2 * t;
#pragma unroll
            for (int n = 0; n < NT; n += 4) {
                *reinterpret_cast<float4*>(d0 + n) =
                    make_float4(o[n][HL ? 0 : 2 * j], o[n + 1][HL ? 0 : 2 * j], o[n + 2][HL ? 0 : 2 * j], o[n + 3][HL ? 0 : 2 * j]);
                *reinterpret_cast<float4*>(d0 + D / 8 + n) =
                    make_float4(o[n][HL ? 1 : 2 * j + 1], o[n + 1][HL ? 1 : 2 * j + 1], o[n + 2][HL ? 1 : 2 * j + 1], o[n + 3][HL ? 1 : 2 * j + 1]);
            }
        }
        __syncthreads();
        const bool whole = ua == 0 && ub == w.units;
        float* part = A.part + ((int64_t)blockIdx.x * 2 + (ua == 0 && u > u0 ? 1 : 0)) * (RT * (D + 2));
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
                const float4 v = *reinterpret_cast<const float4*>(s_o + (k * RT + r) * D + c);
                den = fmaf(wt, s_l[k * RT + r], den);
                acc.x = fmaf(wt, v.x, acc.x); acc.y = fmaf(wt, v.y, acc.y);
                acc.z = fmaf(wt, v.z, acc.z); acc.w = fmaf(wt, v.w, acc.w);
            }
            if (whole) {
                const int row = tile * RT + r;
                if (row < rows) {
                    // a row that sees nothing has m = -inf: zero
                    const float iv = m == -INFINITY ? 0.0f : 1.0f / den;
                    const float y[4] = {m == -INFINITY ? 0.0f : acc.x * iv, m == -INFINITY ? 0.0f : acc.y * iv,
                                        m == -INFINITY ? 0.0f : acc.z * iv, m == -INFINITY ? 0.0f : acc.w * iv};
                    Vec<T>::store(static_cast<T*>(A.out) + (int64_t)(w.s.start + row / A.group) * A.out_stride +
                                      (int64_t)(head * A.group + row % A.group) * D + c,
                                  y);
                }
            } else {
                *reinterpret_cast<float4*>(part + r * D + c) = acc;
                if (c == 0) {
                    part[RT * D + r] = m;
                    part[RT * D + RT + r] = den;
                }
            }
        }
        u += ub - ua;
    }
}

// Join the pieces of every tile that was cut: grid (tiles of all sequences, an upper bound; rows).
template <typename T, int D>
__global__ void __launch_bounds__(D) attn_join_kernel(const __grid_constant__ AttnParams A, int pieces_max) {
    constexpr int RT = sizeof(T) == 4 ? 8 : 16;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the segment: sequence of the blockIdx.x-th (tile, head) pair
    const int lane = threadIdx.x & 31;
    int64_t total = total_work<RT>(A);
    const int pieces = (int)min((int64_t)pieces_max, total);
    if (pieces == 0) return;
    int seg = blockIdx.x;
    int64_t begin = 0;
    for (int base = 0; base < A.B.batch; base += 32) {
        const SeqWork w = seq_work<RT>(A, base + lane);
        const int n = w.tiles * A.kv_heads;
        int inc = n;
        int64_t inw = w.total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            const int64_t y = __shfl_up_sync(0xffffffffu, inw, o);
            if (lane >= o) { inc += x; inw += y; }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, seg < inc);
        if (!hit) {
            seg -= __shfl_sync(0xffffffffu, inc, 31);
            begin += __shfl_sync(0xffffffffu, inw, 31);
            continue;
        }
        const int src = __ffs(hit) - 1;
        const int local = seg - __shfl_sync(0xffffffffu, inc - n, src);
        const int units = __shfl_sync(0xffffffffu, w.units, src);
        const int start = __shfl_sync(0xffffffffu, w.s.start, src), cnt = __shfl_sync(0xffffffffu, w.s.n, src);
        const int64_t a = begin + __shfl_sync(0xffffffffu, inw - w.total, src) + (int64_t)local * units;
        const int c0 = piece_of(total, pieces, a), c1 = piece_of(total, pieces, a + units - 1);
        const int tile = local / A.kv_heads, head = local % A.kv_heads, r = blockIdx.y;
        const int row = tile * RT + r;
        if (c0 == c1 || row >= cnt * A.group) return;  // written by its one CTA
        const int slot0 = piece_begin(total, pieces, c0) == a ? 0 : 1;
        const int64_t step = 2 * RT * (D + 2);
        const float* p = A.part + c0 * step + slot0 * (RT * (D + 2));
        const float* p1 = A.part + (int64_t)(c0 + 1) * step;
        const int c = threadIdx.x;
        float m = p[RT * D + r];
        for (int i = 0; i < c1 - c0; ++i) m = fmaxf(m, p1[i * step + RT * D + r]);
        const float mu = m == -INFINITY ? 0.0f : m;
        const float w0 = ex2(p[RT * D + r] - mu);
        float acc = w0 * p[r * D + c], den = w0 * p[RT * D + RT + r];
        for (int i = 0; i < c1 - c0; ++i) {
            const float* x = p1 + i * step;
            const float wt = ex2(x[RT * D + r] - mu);
            acc = fmaf(wt, x[r * D + c], acc);
            den = fmaf(wt, x[RT * D + RT + r], den);
        }
        const float y = m == -INFINITY ? 0.0f : acc / den;
        T* out = static_cast<T*>(A.out) + (int64_t)(start + row / A.group) * A.out_stride +
                 (int64_t)(head * A.group + row % A.group) * D + c;
        if constexpr (sizeof(T) == 4) *out = y;
        else *out = __float2bfloat16_rn(y);
        return;
    }
}

template <typename T, int D>
cudaError_t launch_typed(const AttnParams& P, int64_t segs, int64_t units, cudaStream_t stream) {
    constexpr int RT = sizeof(T) == 4 ? 8 : 16;
    const size_t smem = (size_t)kAttnWarps * RT * (D + 2) * sizeof(float);
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev]) {
        e = cudaFuncSetAttribute(attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        set[dev] = true;
    }
    int64_t grid = segs * units;
    if (grid > P.parts) grid = P.parts;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(32 * kAttnWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_kernel<T, D>, P);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)segs, RT);
    cfg.blockDim = dim3(D);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<T, D>, P, (int)grid);
}

}  // namespace

size_t attn_workspace_bytes(int head_dim) {  // two slots of up to 16 rows per CTA
    return (size_t)kMaxParts * 2 * 16 * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_attention(const PagedBatch& B, const void* q, int dtype, int64_t q_stride, int q_heads, int kv_heads,
                             int head_dim, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                             const float* v_scale, int max_len, float scale, int window, void* out, int64_t out_stride,
                             void* workspace, int* err_flag, cudaStream_t stream) {
    AttnParams P{};
    P.B = B; P.q = q; P.out = out; P.q_stride = q_stride; P.out_stride = out_stride;
    P.k_cache = k_cache; P.v_cache = v_cache; P.k_scale = k_scale; P.v_scale = v_scale;
    P.q_heads = q_heads; P.kv_heads = kv_heads; P.group = q_heads / kv_heads; P.window = window;
    P.scale_log2 = scale * 1.44269504088896340736f;
    P.part = static_cast<float*>(workspace);
    P.parts = num_sms() * kCtasPerSm < kMaxParts ? num_sms() * kCtasPerSm : kMaxParts;
    P.err_flag = err_flag;
    const int rt = dtype == Q4K_F32 ? 8 : 16;
    // upper bounds: row tiles (a sequence's last one may be part filled), pieces of a tile
    int64_t segs = ((int64_t)B.m * P.group / rt + min(B.m, B.batch)) * kv_heads;
    const int64_t units = (max_len + kUnit - 1) / kUnit + 1;
    if (dtype == Q4K_F32)
        return head_dim == 64 ? launch_typed<float, 64>(P, segs, units, stream) : launch_typed<float, 128>(P, segs, units, stream);
    return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(P, segs, units, stream)
                          : launch_typed<__nv_bfloat16, 128>(P, segs, units, stream);
}

}  // namespace q4k
