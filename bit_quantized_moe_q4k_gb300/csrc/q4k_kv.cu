// q4k_kv.cu -- appending keys and values to the paged 8-bit cache, keys normed and rotated on the way.
//
// A work item is one page that receives tokens, one kv head and one side (keys or values), so each
// scale has one writer. It holds the page's new rows in registers (head_dim / 8 lanes a row), takes
// their largest finite magnitude, and writes e4m3 codes under the scale 2^e, the least power of two
// that maps it into e4m3's range. A page that held tokens already keeps the larger of its scale and
// the new one; when its scale grows, its codes are read and rounded again under it. The scale
// being a power of two, that changes a value only where its code becomes subnormal, so what a page
// holds hardly depends on how many calls filled it.
//
// Bound by latency for single tokens (a chain of four dependent reads: lengths, page, scale, row)
// and by bytes for prompts. Item i < batch is sequence i's first page, so a decode batch finds its
// work without a search; further pages are found by a scan over the sequences.
#include "q4k_paged.cuh"

namespace q4k {
namespace {

struct AppendParams {
    PagedBatch B;
    const void *k, *v;
    int64_t k_stride, v_stride;
    const uint16_t* w_k;
    const double* inv_freq;
    float eps;
    int rot_dim, pairs_mode;
    uint8_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int* err_flag;
};

// Pages of sequence i that receive tokens: the first and their number.
__device__ __forceinline__ int touched_pages(const PagedBatch& B, int i, int* err_flag, SeqSpan* s, int* p0) {
    bool bad;
    *s = seq_span(B, i, &bad);
    if (bad) raise_flag(err_flag, Q4K_ERR_SEQ);
    const int lo = max(s->len - s->n, 0);
    *p0 = lo >> B.page_shift;
    return s->n > 0 && s->len > lo ? ((s->len - 1) >> B.page_shift) - *p0 + 1 : 0;
}

// The w-th page beyond the sequences' first ones (every warp finds it by itself); false past the last.
__device__ __forceinline__ bool further_page(const PagedBatch& B, int w, int* err_flag, int* seq, int* page, SeqSpan* span) {
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < B.batch; base += 32) {
        int cnt = 0, p0 = 0;
        SeqSpan s{0, 0, 0};
        if (base + lane < B.batch) cnt = max(touched_pages(B, base + lane, err_flag, &s, &p0) - 1, 0);
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, w < inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            *seq = base + src;
            *page = __shfl_sync(0xffffffffu, p0 + 1 + w - (inc - cnt), src);
            span->start = __shfl_sync(0xffffffffu, s.start, src);
            span->n = __shfl_sync(0xffffffffu, s.n, src);
            span->len = __shfl_sync(0xffffffffu, s.len, src);
            return true;
        }
        w -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

// One (page, head, side) by W warps (W == 1: warps of a CTA work on items of their own). Rows are
// taken in sets of W * heads-per-warp * HELD; the rows of a single set stay in registers between
// the two passes (largest magnitude, codes), more sets are read and computed again.
template <typename T, int D, int P, int W, int HELD>
__device__ __forceinline__ void append_page(const AppendParams& A, int seq, int page, const SeqSpan& s, int head,
                                            int heads, bool keys, float* s_max) {
    using Lane = HeadLane<D>;
    constexpr int kSet = W * Lane::kHeads * HELD;
    const int entry = page_entry(A.B, seq, page);  // looked at once the rows are on their way
    const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5, sub = lane / Lane::kLanes;
    const int first = s.len - s.n;                          // position of the first new row
    const int lo = max(max(first, 0) - page * P, 0);        // slots [lo, hi) of the page are new
    const int hi = min(s.len - page * P, P);
    const Lane ln(keys ? A.rot_dim : 0, A.pairs_mode);
    const int64_t stride = keys ? A.k_stride : A.v_stride;
    const T* x = static_cast<const T*>(keys ? A.k : A.v) + (int64_t)(s.start + page * P - first) * stride + head * D;
    float w[8];
    uint64_t F[4];
    const bool norm = keys && A.w_k != nullptr, rot = keys && A.rot_dim;
    float v[HELD][8];
    auto read = [&](int set) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int slot = set * kSet + (i * W + warp) * Lane::kHeads + sub;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            if (slot >= lo && slot < hi) ln.load(x + slot * stride, v[i]);
        }
    };
    auto turn = [&](int set) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int slot = set * kSet + (i * W + warp) * Lane::kHeads;
            if (slot >= hi || slot + Lane::kHeads <= lo) continue;  // the same in all lanes
            if (norm) Lane::norm(w, A.eps, v[i]);
            if (rot) {
                float sn[4], cs[4];
                ln.angles(page * P + slot + sub, F, sn, cs);
                ln.rotate(sn, cs, v[i]);
            }
        }
    };
    const int set0 = lo / kSet, set1 = (hi - 1) / kSet;
    read(set0);
    if (norm) ln.load(reinterpret_cast<const __nv_bfloat16*>(A.w_k), w);
    if (rot) ln.fractions(A.inv_freq, F);
    const int pid = page_checked(A.B, entry, A.err_flag);
    if (pid < 0) return;  // the same in all threads
    float* sp = (keys ? A.k_scale : A.v_scale) + (int64_t)pid * heads + head;
    uint8_t* codes = (keys ? A.k_cache : A.v_cache) + ((int64_t)pid * heads + head) * (P * D);
    const float old = lo > 0 ? __ldcg(sp) : 0.0f;
    float amax = 0.0f;
    for (int set = set0; set <= set1; ++set) {
        if (set != set0) read(set);
        turn(set);
#pragma unroll
        for (int i = 0; i < HELD; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = fabsf(v[i][j]);
                if (a <= 3.402823466e38f) amax = fmaxf(amax, a);  // infinities saturate, NaN stays NaN
            }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (W > 1) {
        if (lane == 0) s_max[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) amax = fmaxf(amax, s_max[i]);
    }
    const float scale = fmaxf(exp2_int(scale_exponent(amax)), old);
    if (W == 1 ? lane == 0 : threadIdx.x == 0) *sp = scale;  // every thread has read the old one
    const float inv = 1.0f / scale;  // exact: a power of two
    for (int set = set0; set <= set1; ++set) {
        if (set0 != set1) {
            read(set);
            turn(set);
        }
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int slot = set * kSet + (i * W + warp) * Lane::kHeads + sub;
            if (slot < lo || slot >= hi) continue;
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = f32x2_to_e4m3x2(v[i][2 * j] * inv, v[i][2 * j + 1] * inv);
            *reinterpret_cast<uint32_t*>(codes + slot * D + ln.c0) = q[0] | (q[1] << 16);
            *reinterpret_cast<uint32_t*>(codes + slot * D + ln.c1) = q[2] | (q[3] << 16);
        }
    }
    if (lo == 0 || scale == old) return;
    const float ratio = old * inv;
    for (int i = 16 * (32 * warp + lane); i < lo * D; i += 16 * 32 * W) {  // slots 0 .. lo - 1 lie in a row
        uint4* p = reinterpret_cast<uint4*>(codes + i);
        const uint4 c = __ldcg(p);
        uint32_t r[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t o = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t h = e4m3x2_to_f16x2((r[j] >> (16 * k)) & 0xFFFFu);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                o |= f32x2_to_e4m3x2(f.x * ratio, f.y * ratio) << (16 * k);
            }
            r[j] = o;
        }
        *p = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

constexpr int kPageWarps = 8, kTokenWarps = 4;

// A CTA per (page, head, side): grid (batch first pages, then CTAs that walk over further pages; heads; 2).
template <typename T, int D, int P>
__global__ void __launch_bounds__(32 * kPageWarps) append_pages_kernel(const __grid_constant__ AppendParams A) {
    constexpr int kRows = kPageWarps * HeadLane<D>::kHeads;
    __shared__ float s_max[kPageWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int seq = blockIdx.x, page;
    SeqSpan s;
    if (seq < A.B.batch) {
        if (touched_pages(A.B, seq, A.err_flag, &s, &page) == 0) return;
        append_page<T, D, P, kPageWarps, (P + kRows - 1) / kRows>(A, seq, page, s, blockIdx.y, gridDim.y, blockIdx.z == 0, s_max);
        return;
    }
    for (int w = blockIdx.x - A.B.batch; further_page(A.B, w, A.err_flag, &seq, &page, &s); w += gridDim.x - A.B.batch) {
        append_page<T, D, P, kPageWarps, (P + kRows - 1) / kRows>(A, seq, page, s, blockIdx.y, gridDim.y, blockIdx.z == 0, s_max);
        __syncthreads();  // s_max is free again
    }
}

// A warp per (page, head, side): grid (as above; 2 * heads / kTokenWarps).
template <typename T, int D, int P>
__global__ void __launch_bounds__(32 * kTokenWarps) append_tokens_kernel(const __grid_constant__ AppendParams A, int heads) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int hs = blockIdx.y * kTokenWarps + (threadIdx.x >> 5);
    if (hs >= 2 * heads) return;
    int seq = blockIdx.x, page;
    SeqSpan s;
    if (seq < A.B.batch) {
        if (touched_pages(A.B, seq, A.err_flag, &s, &page) == 0) return;
        append_page<T, D, P, 1, 2>(A, seq, page, s, hs >> 1, heads, (hs & 1) == 0, nullptr);
        return;
    }
    for (int w = blockIdx.x - A.B.batch; further_page(A.B, w, A.err_flag, &seq, &page, &s); w += gridDim.x - A.B.batch)
        append_page<T, D, P, 1, 2>(A, seq, page, s, hs >> 1, heads, (hs & 1) == 0, nullptr);
}

template <typename T, int D, int P>
cudaError_t launch_page(const AppendParams& A, int kv_heads, cudaStream_t stream) {
    // CTAs for the pages beyond each sequence's first: as many as the tokens fill; where ragged
    // sequences touch more, the CTAs walk on.
    const int items = A.B.batch + ((A.B.m - 1) >> A.B.page_shift) + 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // Mostly single tokens: a warp an item; else the CTA that shares a page's rows.
    if (A.B.m <= 2 * (int64_t)A.B.batch) {
        cfg.gridDim = dim3((unsigned)items, (unsigned)((2 * kv_heads + kTokenWarps - 1) / kTokenWarps));
        cfg.blockDim = dim3(32 * kTokenWarps);
        return cudaLaunchKernelEx(&cfg, append_tokens_kernel<T, D, P>, A, kv_heads);
    }
    cfg.gridDim = dim3((unsigned)items, (unsigned)kv_heads, 2);
    cfg.blockDim = dim3(32 * kPageWarps);
    return cudaLaunchKernelEx(&cfg, append_pages_kernel<T, D, P>, A);
}

template <typename T, int D>
cudaError_t launch_dim(const AppendParams& A, int kv_heads, cudaStream_t stream) {
    switch (A.B.page_shift) {
        case 4: return launch_page<T, D, 16>(A, kv_heads, stream);
        case 5: return launch_page<T, D, 32>(A, kv_heads, stream);
        case 6: return launch_page<T, D, 64>(A, kv_heads, stream);
        default: return launch_page<T, D, 128>(A, kv_heads, stream);
    }
}

}  // namespace

cudaError_t launch_kv_append(const PagedBatch& B, const void* k, const void* v, int dtype, int64_t k_stride,
                             int64_t v_stride, int kv_heads, int head_dim, const uint16_t* w_k, float eps,
                             const double* inv_freq, int rot_dim, int rope_mode, uint8_t* k_cache, uint8_t* v_cache,
                             float* k_scale, float* v_scale, int* err_flag, cudaStream_t stream) {
    AppendParams A{};
    A.B = B; A.k = k; A.v = v; A.k_stride = k_stride; A.v_stride = v_stride; A.w_k = w_k; A.inv_freq = inv_freq;
    A.eps = eps; A.rot_dim = rot_dim; A.pairs_mode = rope_mode == Q4K_ROPE_PAIRS; A.k_cache = k_cache;
    A.v_cache = v_cache; A.k_scale = k_scale; A.v_scale = v_scale; A.err_flag = err_flag;
    if (dtype == Q4K_F32)
        return head_dim == 64 ? launch_dim<float, 64>(A, kv_heads, stream) : launch_dim<float, 128>(A, kv_heads, stream);
    return head_dim == 64 ? launch_dim<__nv_bfloat16, 64>(A, kv_heads, stream)
                          : launch_dim<__nv_bfloat16, 128>(A, kv_heads, stream);
}

}  // namespace q4k
