// q4k_qkrope.cu -- the norm of each query and key head with the position rotation in the same pass.
//
//   y = x * w / sqrt(mean_c x_c^2 + eps)   (per head; no weight: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin) over the first rot_dim dims, angle pos[t] * inv_freq[j]
// One warp per head and token, head_dim / 32 consecutive dims a lane, everything in fp32 and
// rounded once at the store.
#include "q4k_paged.cuh"

namespace q4k {
namespace {

struct NormRopeParams {
    const void *q, *k;
    void *q_out, *k_out;
    const uint16_t *w_q, *w_k;
    const int32_t* pos;
    const double* inv_freq;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;
    int m, q_heads, heads, rot_dim, pairs_mode;
    float eps;
};

constexpr int kRopeWarps = 4;

template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(32 * kRopeWarps) norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = blockIdx.x, lane = threadIdx.x & 31, c0 = N * lane;
    float sn[N], cs[N];
    if (P.rot_dim) lane_angles<N>(c0, __ldcg(P.pos + t), P.inv_freq, P.rot_dim, P.pairs_mode, sn, cs);
    for (int h = blockIdx.y * kRopeWarps + (threadIdx.x >> 5); h < P.heads; h += gridDim.y * kRopeWarps) {
        const bool is_q = h < P.q_heads;
        const int hh = is_q ? h : h - P.q_heads;
        const TI* x = static_cast<const TI*>(is_q ? P.q : P.k) + t * (is_q ? P.q_stride : P.k_stride) + hh * 32 * N + c0;
        TO* o = static_cast<TO*>(is_q ? P.q_out : P.k_out) + t * (is_q ? P.q_out_stride : P.k_out_stride) + hh * 32 * N + c0;
        float v[N];
        Vec<TI>::load(x, v);
        const uint16_t* wp = is_q ? P.w_q : P.w_k;
        if (wp) {
            float w[N];
            Vec<__nv_bfloat16>::load(reinterpret_cast<const __nv_bfloat16*>(wp) + c0, w);
            lane_norm<N>(w, 32 * N, P.eps, v);
        }
        if (P.rot_dim) lane_rotate<N>(c0, P.rot_dim, P.pairs_mode, sn, cs, v);
        Vec<TO>::store(o, v);
    }
}

template <typename TI, typename TO>
cudaError_t launch_typed(const NormRopeParams& P, int head_dim, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)P.m, (unsigned)((P.heads + kRopeWarps - 1) / kRopeWarps));
    cfg.blockDim = dim3(32 * kRopeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (head_dim == 64) return cudaLaunchKernelEx(&cfg, norm_rope_kernel<TI, TO, 2>, P);
    if (head_dim == 128) return cudaLaunchKernelEx(&cfg, norm_rope_kernel<TI, TO, 4>, P);
    return cudaLaunchKernelEx(&cfg, norm_rope_kernel<TI, TO, 8>, P);
}

}  // namespace

cudaError_t launch_norm_rope(const void* q, const void* k, int dtype, int out_dtype, int m, int q_heads, int kv_heads,
                             int head_dim, int64_t q_stride, int64_t k_stride, const uint16_t* w_q,
                             const uint16_t* w_k, float eps, const int32_t* pos, const double* inv_freq, int rot_dim,
                             int rope_mode, void* q_out, void* k_out, int64_t q_out_stride, int64_t k_out_stride,
                             cudaStream_t stream) {
    NormRopeParams P{};
    P.q = q; P.k = k; P.q_out = q_out; P.k_out = k_out; P.w_q = w_q; P.w_k = w_k; P.pos = pos; P.inv_freq = inv_freq;
    P.q_stride = q_stride; P.k_stride = k_stride; P.q_out_stride = q_out_stride; P.k_out_stride = k_out_stride;
    P.m = m; P.q_heads = q_heads; P.heads = q_heads + kv_heads; P.rot_dim = rot_dim;
    P.pairs_mode = rope_mode == Q4K_ROPE_PAIRS; P.eps = eps;
    if (dtype == Q4K_F32)
        return out_dtype == Q4K_F32 ? launch_typed<float, float>(P, head_dim, stream)
                                    : launch_typed<float, __nv_bfloat16>(P, head_dim, stream);
    return out_dtype == Q4K_F32 ? launch_typed<__nv_bfloat16, float>(P, head_dim, stream)
                                : launch_typed<__nv_bfloat16, __nv_bfloat16>(P, head_dim, stream);
}

}  // namespace q4k
