// q4k_kv.cu -- appending keys and values to the paged 8-bit cache, keys normed and rotated on the way.
//
// A work item is one page that receives tokens, one kv head and one side (keys or values), so each
// scale has one writer. Its CTA holds the page's new rows in registers (one warp per row, head_dim /
// 32 dims a lane), takes their largest finite magnitude, and writes e4m3 codes under the scale 2^e,
// the least power of two that maps it into e4m3's range. A page that held tokens already keeps the
// larger of its scale and the new one; when its scale grows, its codes are read and rounded again
// under it. The scale being a power of two, that changes a value only where its code becomes
// subnormal, so what a page holds hardly depends on how many calls filled it.
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

constexpr int kAppendWarps = 8;

// Sequence and page of work item w (every warp finds them by itself); false past the last item.
__device__ __forceinline__ bool append_item(const PagedBatch& B, int w, int* err_flag, int* seq, int* page, SeqSpan* span) {
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < B.batch; base += 32) {
        int cnt = 0, p0 = 0;
        SeqSpan s{0, 0, 0};
        if (base + lane < B.batch) {
            bool bad;
            s = seq_span(B, base + lane, &bad);
            if (bad) raise_flag(err_flag, Q4K_ERR_SEQ);
            const int lo = max(s.len - s.n, 0);
            p0 = lo >> B.page_shift;
            if (s.n > 0 && s.len > lo) cnt = ((s.len - 1) >> B.page_shift) - p0 + 1;
        }
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
            *page = __shfl_sync(0xffffffffu, p0 + w - (inc - cnt), src);
            span->start = __shfl_sync(0xffffffffu, s.start, src);
            span->n = __shfl_sync(0xffffffffu, s.n, src);
            span->len = __shfl_sync(0xffffffffu, s.len, src);
            return true;
        }
        w -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

// Grid (items, kv heads, 2). P: page size.
template <typename T, int N, int P>
__global__ void __launch_bounds__(32 * kAppendWarps) kv_append_kernel(const __grid_constant__ AppendParams A) {
    constexpr int D = 32 * N, RPW = P / kAppendWarps;  // rows of the page a warp holds
    __shared__ float s_max[kAppendWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int seq, page;
    SeqSpan s;
    if (!append_item(A.B, blockIdx.x, A.err_flag, &seq, &page, &s)) return;
    const int pid = page_id(A.B, seq, page, A.err_flag);
    if (pid < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = N * lane;
    const int head = blockIdx.y, heads = gridDim.y;
    const bool keys = blockIdx.z == 0;
    const int first = s.len - s.n;                          // position of the first new row
    const int lo = max(max(first, 0) - page * P, 0);        // slots [lo, hi) of the page are new
    const int hi = min(s.len - page * P, P);
    const T* x = static_cast<const T*>(keys ? A.k : A.v) + head * D + c0;
    const int64_t stride = keys ? A.k_stride : A.v_stride;
    float w[N];
    const bool norm = keys && A.w_k != nullptr;
    if (norm) Vec<__nv_bfloat16>::load(reinterpret_cast<const __nv_bfloat16*>(A.w_k) + c0, w);
    float v[RPW][N];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        const int slot = warp + kAppendWarps * i;
        if (slot < lo || slot >= hi) continue;
        const int pos = page * P + slot;
        Vec<T>::load(x + (int64_t)(s.start + pos - first) * stride, v[i]);
        if (norm) lane_norm<N>(w, D, A.eps, v[i]);
        if (keys && A.rot_dim) {
            float sn[N], cs[N];
            lane_angles<N>(c0, pos, A.inv_freq, A.rot_dim, A.pairs_mode, sn, cs);
            lane_rotate<N>(c0, A.rot_dim, A.pairs_mode, sn, cs, v[i]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float a = fabsf(v[i][j]);
            if (a <= 3.402823466e38f) amax = fmaxf(amax, a);  // infinities saturate, NaN stays NaN
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAppendWarps; ++i) amax = fmaxf(amax, s_max[i]);
    float* sp = (keys ? A.k_scale : A.v_scale) + (int64_t)pid * heads + head;
    uint8_t* codes = (keys ? A.k_cache : A.v_cache) + ((int64_t)pid * heads + head) * (P * D) + c0;
    const float fresh = exp2_int(scale_exponent(amax));
    const float old = lo > 0 ? __ldcg(sp) : 0.0f;
    const float scale = fmaxf(fresh, old);
    __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0) *sp = scale;
    const float inv = 1.0f / scale;  // exact: a power of two
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        const int slot = warp + kAppendWarps * i;
        if (slot < lo || slot >= hi) continue;
        uint32_t q[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) q[j] = f32x2_to_e4m3x2(v[i][2 * j] * inv, v[i][2 * j + 1] * inv);
        if constexpr (N == 4)
            *reinterpret_cast<uint32_t*>(codes + slot * D) = q[0] | (q[1] << 16);
        else
            *reinterpret_cast<uint16_t*>(codes + slot * D) = (uint16_t)q[0];
    }
    if (lo == 0 || scale == old) return;
    const float ratio = old * inv;
    for (int slot = warp; slot < lo; slot += kAppendWarps) {
        uint16_t* p = reinterpret_cast<uint16_t*>(codes + slot * D);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const uint32_t h = e4m3x2_to_f16x2(__ldcg(p + j));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            p[j] = (uint16_t)f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
        }
    }
}

template <typename T, int N, int P>
cudaError_t launch_page(const AppendParams& A, int items, int kv_heads, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)items, (unsigned)kv_heads, 2);
    cfg.blockDim = dim3(32 * kAppendWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<T, N, P>, A);
}

template <typename T, int N>
cudaError_t launch_dim(const AppendParams& A, int items, int kv_heads, cudaStream_t stream) {
    switch (A.B.page_shift) {
        case 4: return launch_page<T, N, 16>(A, items, kv_heads, stream);
        case 5: return launch_page<T, N, 32>(A, items, kv_heads, stream);
        case 6: return launch_page<T, N, 64>(A, items, kv_heads, stream);
        default: return launch_page<T, N, 128>(A, items, kv_heads, stream);
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
    // A sequence of n new tokens touches at most (n - 1) / page + 2 pages, and at most n.
    const int64_t most = (int64_t)(B.m >> B.page_shift) + 2 * (int64_t)B.batch;
    const int items = (int)(most < B.m ? most : B.m);
    if (dtype == Q4K_F32)
        return head_dim == 64 ? launch_dim<float, 2>(A, items, kv_heads, stream)
                              : launch_dim<float, 4>(A, items, kv_heads, stream);
    return head_dim == 64 ? launch_dim<__nv_bfloat16, 2>(A, items, kv_heads, stream)
                          : launch_dim<__nv_bfloat16, 4>(A, items, kv_heads, stream);
}

}  // namespace q4k
