// q4k_own.cu -- attention behind shared prefixes: what each sequence sees of its own tokens, and the join of that with what
// its group shares (q4k_prefix.cu; the plan: q4k_prefix.cuh).
//
// The mathematics of q4k_attn.cu, and its fragments: query rows are the M side of mma.m16n8k16, eight of them a tile; fp32 rows in two fp16 terms.
// But a piece (a row tile of a kv head, over some hundred tokens) is one warp's, from its list entry to its sums in the workspace, and warps
// share nothing: while one looks up pages or writes its sums, the other eleven of the SM stream. Own parts are short, so that in the kernel for
// whole sequences, where four warps share a tile and wait for one another at its start, in its join and at its end, starts and ends
// were two thirds of the time. Bound by each warp's chain of copies, products and exponentials, twelve warps an SM: 256 sequences of up to 1000
// tokens, 8 kv heads of 128, bf16, 262 MB: 70 us alone, 3.8 TB/s. Looking a piece up while the one before it streams, and longest pieces
// first, gave nothing (215 us for the whole call behind 32768 shared tokens, and 219).
#include <atomic>

#include "q4k_attn_few.cuh"
#include "q4k_prefix.cuh"

namespace q4k {
using namespace few;
namespace {

// What P and so the sums are relative to, for the running maximum m (x - reference is 15 at most).
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? m : __fadd_ru(m, -15.0f); }

template <typename T, int D>
__global__ void __launch_bounds__(32 * kOwnWarps, 3) own_kernel(const __grid_constant__ OwnParams A) {
    constexpr bool HL = sizeof(T) == 4;           // two fp16 terms
    constexpr int NT = D / 8;                     // output column tiles
    constexpr int S = kPair;
    extern __shared__ __align__(128) uint8_t s_mem[];
    __shared__ ChunkMeta s_meta[kOwnWarps][kRing * kPair];
    // The shared part's kernel, before this one in the stream, waited for the plan, so the plan is there; nothing else of
    // it is read here, and it is waited for at the end only, for the sake of what comes after.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint8_t* const ring = s_mem + warp * (kRing * kStage<D>);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    const int4* const head_at = reinterpret_cast<const int4*>(&A.plan.head->ctas);
    const int4 counts = __ldcg(head_at);   // ctas, own_tiles, own_pieces, own_length
    const int tiles = (int)min((int64_t)max(counts.y, 0), A.plan.owns), length = max(counts.w, kChunk);
    const int64_t pieces = min((int64_t)max(counts.z, 0), A.plan.own_pieces) * A.kv_heads;
    unsigned next = 0;
    if (lane == 0) next = atomicAdd(&A.plan.head->next, 1u);
    for (;;) {
        const int64_t at = __shfl_sync(0xffffffffu, next, 0);
        if (at >= pieces || tiles == 0) break;
        if (lane == 0) next = atomicAdd(&A.plan.head->next, 1u);   // looked at when this piece is done
        const int pc = (int)(at / A.kv_heads), head = (int)(at - (int64_t)pc * A.kv_heads);
        const int2 which = __ldcg(A.plan.own_piece + pc);
        // (no number of the plan is believed as far as addresses go: two calls at once on one workspace write over it)
        const int4* const entry = reinterpret_cast<const int4*>(A.plan.own + min(max(which.x, 0), tiles - 1));
        const int4 ea = __ldcg(entry), eb = __ldcg(entry + 1);
        const int seq = min(max(ea.x, 0), A.B.batch - 1), start = min(max(ea.y, 0), A.B.m - 1), n_new = min(max(ea.z, 0), A.B.m - start);
        const int len = min(max(ea.w, 0), A.B.max_pages << A.B.page_shift), rows = n_new * A.group, first = len - n_new, tile = max(eb.z, 0);
        const int t0 = (max(eb.x, 0) + max(which.y, 0)) & ~(kChunk - 1), tile_hi = min(eb.y, len);
        const int n = min(max((min(tile_hi - t0, length) + kChunk - 1) / kChunk, 0), 1 << 26);   // chunks

        auto entry_of = [&](int i) { return i < n ? page_entry(A.B, seq, (t0 + kChunk * i) >> A.B.page_shift) : -1; };
        auto checked = [&](int i, int p) { return i < n ? page_checked(A.B, p, A.err_flag) : -1; };
        auto scales_of = [&](int pid, float& ks, float& vs) {
            ks = vs = 1.0f;
            if (pid >= 0) {
                ks = __ldcg(A.k_scale + (int64_t)pid * A.kv_heads + head);
                vs = __ldcg(A.v_scale + (int64_t)pid * A.kv_heads + head);
            }
        };
        PageAhead ah{entry_of(lane), entry_of(32 + lane), entry_of(64 + lane), 1.f, 1.f, 1.f, 1.f};
        // the lane's row, its dims 64 h + 16 t ..; a row past the last one reads the first one's
        const int row = tile * kOwnRows + g;
        const bool valid = row < rows;
        const int tok_of_row = valid ? row / A.group : 0, pos = first + tok_of_row;
        float x[D / 64][16];
        {
            const T* p = static_cast<const T*>(A.q) + (int64_t)(start + tok_of_row) * A.q_stride +
                         (int64_t)(head * A.group + (valid ? row - tok_of_row * A.group : 0)) * D + 16 * t;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) Vec<T>::load(p + 64 * h, x[h]);
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
                const int slot = (t0 + kChunk * i) & ((1 << A.B.page_shift) - 1);
                const int64_t from = ((((int64_t)pid * A.kv_heads + head) << A.B.page_shift) + slot) * D + 16 * lane;
                const uint32_t dst = ring_at + k % kRing * kStage<D> + c * kSlot<D>;
                constexpr int kUnits = D / 16, kRows = 32 / kUnits;  // a row's units; rows of one copy instruction
#pragma unroll
                for (int j = 0; j < kChunk / kRows; ++j) {
                    const int r = kRows * j + lane / kUnits, u = lane % kUnits;
                    copy16(dst + k_unit<D>(r, u), A.k_cache + from + 512 * j);
                    copy16(dst + kChunk * D + v_unit<D>(r, u), A.v_cache + from + 512 * j);
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

        // the row's limits and its fragments: 16-dim steps, four dims of the lane each
        const int hi = valid ? pos + 1 : 0, lo = A.window > 0 ? max(pos - A.window + 1, 0) : 0;
        const int pf = first + tile * kOwnRows / A.group, pl = first + (min(rows, tile * kOwnRows + kOwnRows) - 1) / A.group;
        const int full_hi = max(pf + 1, 0), full_lo = A.window > 0 ? max(pl - A.window + 1, 0) : 0;
        uint32_t qf[D / 16][HL ? 4 : 2];
        float crow;
        {
            float amax = 0.0f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (!valid) x[h][i] = 0.0f;
                    const float a = fabsf(x[h][i]);
                    if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // power of two that brings the row's largest magnitude to [2^7, 2^8)
            const int e = amax > 0.0f ? min(max(134 - (int)(__float_as_uint(amax) >> 23), -120), 120) : 0;
            const float up = exp2_int(e);
            crow = A.scale_log2 * exp2_int(-e);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a0 = x[h][4 * i] * up, a1 = x[h][4 * i + 1] * up, a2 = x[h][4 * i + 2] * up, a3 = x[h][4 * i + 3] * up;
                    uint32_t(&f)[HL ? 4 : 2] = qf[4 * h + i];
                    if constexpr (HL) {
                        const __half2 h01 = __floats2half2_rn(a0, a1), h23 = __floats2half2_rn(a2, a3);
                        const float2 b01 = __half22float2(h01), b23 = __half22float2(h23);
                        f[0] = *reinterpret_cast<const uint32_t*>(&h01);
                        f[2] = *reinterpret_cast<const uint32_t*>(&h23);
                        f[1] = pack_f16(a0 - b01.x, a1 - b01.y);
                        f[3] = pack_f16(a2 - b23.x, a3 - b23.y);
                    } else {
                        f[0] = pack_f16(a0, a1);
                        f[1] = pack_f16(a2, a3);
                    }
                }
        }
        for (int k = 0; k < kRing; ++k) note(k);

        float2 o[NT];
        float mx = -INFINITY, l = 0.0f;
#pragma unroll
        for (int k = 0; k < NT; ++k) o[k] = make_float2(0.0f, 0.0f);
        // a stage at a time: one maximum, one correction and one flush of the sums for its chunks
#pragma unroll 1
        for (int k_st = 0; k_st < n_st; ++k_st) {
            const int stage = k_st % kRing, i0 = S * k_st;
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();
            // Tokens: lane t's of a chunk are 4 t + {0, 1, 2, 3}, columns 2 t, 2 t + 1 of score tiles 0 and 1, so
            // column c of tile j is token 4 (c / 2) + 2 j + c % 2.
            float xs[S][4], inv[S];
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
                    const uint32_t(&f)[HL ? 4 : 2] = qf[4 * h + q];
                    const uint32_t qa[4] = {f[0], HL ? f[1] : 0u, HL ? f[HL ? 2 : 0] : f[1], HL ? f[HL ? 3 : 0] : 0u};
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
                const int base = t0 + kChunk * (i0 + c);
                const ChunkMeta meta = s_meta[warp][stage * S + c];
                // x = c * s + e, masked
                inv[c] = meta.inv;
                held[c] = meta.ok;
                full[c] = meta.ok && base >= full_lo && base + kChunk <= full_hi;
                const float cr = crow * meta.ks;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float sv = HL ? s[c][k >> 1][k & 1] + s[c][k >> 1][2 + (k & 1)] : s[c][k >> 1][k & 1];
                    xs[c][k] = fmaf(sv, cr, meta.ev);
                }
                if (!full[c]) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = base + 4 * t + k;
                        if (!meta.ok || tok < lo || tok >= hi) xs[c][k] = -INFINITY;
                    }
                }
            }
            float top = xs[0][0];
#pragma unroll
            for (int c = 0; c < S; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, xs[c][k]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float m_new = fmaxf(mx, top);
            const bool grew = m_new > mx;
            const float m_use = m_new == -INFINITY ? 0.0f : m_new, base15 = __fadd_ru(m_use, -15.0f);
            const float corr = ex2(mx - m_use);
            mx = m_new;
            l *= corr;
#pragma unroll
            for (int c = 0; c < S; ++c) {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    xs[c][k] = ex2(xs[c][k] - base15);
                    sum += xs[c][k];
                }
                l = fmaf(sum, inv[c], l);
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int k = 0; k < NT; ++k) mul2(o[k], corr);
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
            uint32_t pa[S][4];
#pragma unroll
            for (int c = 0; c < S; ++c) {
                if constexpr (HL) {
                    const __half2 h0 = __floats2half2_rn(xs[c][0], xs[c][1]), h1 = __floats2half2_rn(xs[c][2], xs[c][3]);
                    const float2 b0 = __half22float2(h0), b1 = __half22float2(h1);
                    pa[c][0] = *reinterpret_cast<const uint32_t*>(&h0);
                    pa[c][2] = *reinterpret_cast<const uint32_t*>(&h1);
                    float2 r0 = make_float2(xs[c][0], xs[c][1]), r1 = make_float2(xs[c][2], xs[c][3]);
                    mul2(r0, 2048.0f);
                    mul2(r1, 2048.0f);
                    fma2(r0, b0.x, b0.y, -2048.0f);
                    fma2(r1, b1.x, b1.y, -2048.0f);
                    pa[c][1] = pack_f16(r0.x, r0.y);
                    pa[c][3] = pack_f16(r1.x, r1.y);
                } else {
                    pa[c][0] = pack_f16(xs[c][0], xs[c][1]);
                    pa[c][2] = pack_f16(xs[c][2], xs[c][3]);
                    pa[c][1] = pa[c][3] = 0;
                }
                if (!full[c]) {
                    // tokens that no row of the tile sees hold anything: NaN codes too
                    const int base = t0 + kChunk * (i0 + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = base + 4 * t + k;
                        if (!held[c] || tok >= tile_hi)
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
                        for (int k = 0; k < 4; ++k) {
                            const int tok = base + 4 * t + k;
                            if (tok >= lo && tok < hi) see[2 * (k >> 1)] |= 0x3C00u << (16 * (k & 1));
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
                                if (acc[0] > 0.0f) o[4 * q + k].x = __int_as_float(0x7FC00000);
                                if (acc[1] > 0.0f) o[4 * q + k].y = __int_as_float(0x7FC00000);
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
                    // a fresh accumulator for each stage, added in fp32: the tensor core's own accumulation does not round to nearest
                    float acc[4];
                    mma_16816_zero(acc, pa[0], b0[0][k], b1[0][k]);
#pragma unroll
                    for (int c = 1; c < S; ++c) mma_16816(acc, pa[c], b0[c][k], b1[c][k]);
                    add2(o[4 * q + k], acc[0], acc[1]);
                    if (HL) fma2(o[4 * q + k], acc[2], acc[3], 1.0f / 2048.0f);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (valid) {
            // this lane's dims: D/8 (2 t) + k and D/8 (2 t + 1) + k, k = 0 .. NT - 1
            const int64_t place = at * kOwnRows + g;
            float* const d0 = A.plan.own_sums + place * D + D / 8 * (2 * t);
#pragma unroll
            for (int k = 0; k < NT; k += 4) {
                *reinterpret_cast<float4*>(d0 + k) = make_float4(o[k].x, o[k + 1].x, o[k + 2].x, o[k + 3].x);
                *reinterpret_cast<float4*>(d0 + D / 8 + k) = make_float4(o[k].y, o[k + 1].y, o[k + 2].y, o[k + 3].y);
            }
            if (t == 0) A.plan.own_refs[place] = make_float2(reference(mx), l);
        }
        __syncwarp();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what comes after this kernel comes after the shared part's, too
}

// Each row's sums over its own pieces and over the pieces of what its group shares, to the largest of their references. A CTA a row
// tile and kv head; D / 4 lanes a row, four dims a lane. Bound by reading the pieces, from L2.
template <typename T, int D>
__global__ void __launch_bounds__(kOwnRows * D / 4) join_kernel(const __grid_constant__ OwnParams A) {
    constexpr int kLanes = D / 4;
    __shared__ float s_w[kOwnRows][kLanes];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, local = tid / kLanes, u = tid % kLanes, c = 4 * u;
    const int64_t i = blockIdx.x / A.kv_heads;
    const int head = (int)(blockIdx.x - i * A.kv_heads);
    const int4* const entry = reinterpret_cast<const int4*>(A.plan.own + min(i, A.plan.owns - 1));
    const int4 ea = __ldcg(entry), eb = __ldcg(entry + 1), ec = __ldcg(entry + 2);
    if (i >= min((int64_t)__ldcg(&A.plan.head->own_tiles), A.plan.owns)) return;
    OwnTile W;
    memcpy(&W, &ea, 16);
    memcpy(reinterpret_cast<char*>(&W) + 16, &eb, 16);
    memcpy(reinterpret_cast<char*>(&W) + 32, &ec, 16);
    const int row = W.tile * kOwnRows + local;
    const int tok = W.start + row / A.group;
    // (no number of the plan is believed as far as addresses go: two calls at once on one workspace write over it)
    const bool there = W.tile >= 0 && row >= 0 && row < W.n * A.group && tok >= 0 && tok < A.B.m;
    const int own = there && W.piece0 >= 0 && W.pieces > 0 && (int64_t)W.piece0 + W.pieces <= A.plan.own_pieces ? W.pieces : 0;
    const int64_t own_at = ((int64_t)W.piece0 * A.kv_heads + head) * kOwnRows + local, own_step = (int64_t)A.kv_heads * kOwnRows;
    int shared = 0;
    int64_t shared_at = 0;
    if (there && W.first >= 0) {
        const int r = W.first + local, row_tile = r / A.plan.tile_rows;
        const int64_t item = W.item0 + (int64_t)row_tile * A.kv_heads + head;
        if (item >= 0 && item < A.plan.items) {
            const int2 s = __ldcg(reinterpret_cast<const int2*>(A.plan.item + item));
            if (s.x >= 0 && s.y > 0 && s.y <= kPrefixCtas && s.x + s.y <= A.plan.slots) {
                shared = s.y;
                shared_at = (int64_t)s.x * A.plan.tile_rows + (r - row_tile * A.plan.tile_rows);
            }
        }
    }
    const int all = own + shared;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.0f, ref = -INFINITY;   // den: the lane's pieces
    // the rows of a warp go on together
    for (int k0 = 0; __any_sync(0xffffffffu, k0 < all); k0 += kLanes) {
        const int k = k0 + u;
        float2 f = make_float2(-INFINITY, 0.0f);
        if (k < own) f = __ldcg(A.plan.own_refs + own_at + k * own_step);
        else if (k < all) f = __ldcg(A.plan.refs + shared_at + (int64_t)(k - own) * A.plan.tile_rows);
        float top = fmaxf(ref, f.x);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float use = top == -INFINITY ? 0.0f : top, keep = ex2(ref - use), w = ex2(f.x - use);
        acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
        den = fmaf(w, f.y, den * keep);
        ref = top;
        __syncwarp();
        s_w[local][u] = w;
        __syncwarp();
        const int here = min(all - k0, kLanes);
#pragma unroll 8
        for (int j = 0; j < here; ++j) {
            const float* p = k0 + j < own ? A.plan.own_sums + (own_at + (k0 + j) * own_step) * D
                                          : A.plan.sums + (shared_at + (int64_t)(k0 + j - own) * A.plan.tile_rows) * D;
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p + c));
            const float x = s_w[local][j];
            acc.x = fmaf(x, v.x, acc.x); acc.y = fmaf(x, v.y, acc.y);
            acc.z = fmaf(x, v.z, acc.z); acc.w = fmaf(x, v.w, acc.w);
        }
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (!there) return;
    const float iv = den == 0.0f ? 0.0f : 1.0f / den;  // 0: the row sees nothing
    const float y[4] = {acc.x * iv, acc.y * iv, acc.z * iv, acc.w * iv};
    Vec<T>::store(static_cast<T*>(A.out) + (int64_t)tok * A.out_stride + (int64_t)(head * A.group + row % A.group) * D + c, y);
}

cudaLaunchConfig_t config(int64_t grid, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <typename T, int D>
cudaError_t launch_own_typed(const OwnParams& P, cudaStream_t stream) {
    constexpr int smem = kOwnWarps * kRing * kStage<D>;
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(own_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        allowed[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr;
    const int64_t most = (P.plan.own_pieces * P.kv_heads + kOwnWarps - 1) / kOwnWarps;
    const cudaLaunchConfig_t cfg = config(most < kOwnCtas ? most : kOwnCtas, 32 * kOwnWarps, smem, stream, &attr);
    return cudaLaunchKernelEx(&cfg, own_kernel<T, D>, P);
}
template <typename T, int D>
cudaError_t launch_join_typed(const OwnParams& P, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(P.plan.owns * P.kv_heads, kOwnRows * D / 4, 0, stream, &attr);
    return cudaLaunchKernelEx(&cfg, join_kernel<T, D>, P);
}

}  // namespace

cudaError_t launch_own(const OwnParams& P, int dtype, int head_dim, cudaStream_t stream) {
    if (dtype == Q4K_F32) return head_dim == 64 ? launch_own_typed<float, 64>(P, stream) : launch_own_typed<float, 128>(P, stream);
    return head_dim == 64 ? launch_own_typed<__nv_bfloat16, 64>(P, stream) : launch_own_typed<__nv_bfloat16, 128>(P, stream);
}
cudaError_t launch_join(const OwnParams& P, int dtype, int head_dim, cudaStream_t stream) {
    if (dtype == Q4K_F32) return head_dim == 64 ? launch_join_typed<float, 64>(P, stream) : launch_join_typed<float, 128>(P, stream);
    return head_dim == 64 ? launch_join_typed<__nv_bfloat16, 64>(P, stream) : launch_join_typed<__nv_bfloat16, 128>(P, stream);
}

}  // namespace q4k
