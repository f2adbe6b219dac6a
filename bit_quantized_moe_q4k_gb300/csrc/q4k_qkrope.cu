// q4k_qkrope.cu -- the norm of each query and key head with the position rotation in the same pass.
//
//   y = x * w / sqrt(mean_c x_c^2 + eps)   (per head; no weight: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin) over the first rot_dim dims, angle pos[t] * inv_freq[j]
// head_dim / 8 lanes hold a head (8 dims each, whole pairs, so the rotation needs no exchange), everything
// in fp32 and rounded once at the store. A warp computes its token's angles once and walks over heads,
// two loads ahead: with one head a warp the sines cost more than the bytes.
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

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(32 * kRopeWarps) norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
    using Lane = HeadLane<D>;
    constexpr int kAhead = 2;  // steps whose loads are in flight together
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = blockIdx.x, sub = (threadIdx.x & 31) / Lane::kLanes;
    const Lane ln(P.rot_dim, P.pairs_mode);
    const int stride = gridDim.y * kRopeWarps * Lane::kHeads;
    float sn[4], cs[4], wq[8], wk[8];
    if (P.rot_dim) {
        uint64_t F[4];
        ln.fractions(P.inv_freq, F);
        ln.angles(__ldcg(P.pos + t), F, sn, cs);
    }
    // a side without weights multiplies by nothing: its norm is computed (the warp's lanes stay together) and dropped
#pragma unroll
    for (int i = 0; i < 8; ++i) wq[i] = wk[i] = 1.0f;
    if (P.w_q) ln.load(reinterpret_cast<const __nv_bfloat16*>(P.w_q), wq);
    if (P.w_k) ln.load(reinterpret_cast<const __nv_bfloat16*>(P.w_k), wk);
    const TI* q = static_cast<const TI*>(P.q) + t * P.q_stride;
    const TI* k = static_cast<const TI*>(P.k) + t * P.k_stride;
    TO* qo = static_cast<TO*>(P.q_out) + t * P.q_out_stride;
    TO* ko = static_cast<TO*>(P.k_out) + t * P.k_out_stride;
    // h0 is the same in all lanes of a warp; a lane's head is h0 + its group
    for (int h0 = (blockIdx.y * kRopeWarps + (threadIdx.x >> 5)) * Lane::kHeads; h0 < P.heads; h0 += kAhead * stride) {
        float v[kAhead][8] = {};
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int h = h0 + a * stride + sub;
            if (h < P.q_heads) ln.load(q + h * D, v[a]);
            else if (h < P.heads) ln.load(k + (h - P.q_heads) * D, v[a]);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int h = h0 + a * stride + sub;
            const bool is_q = h < P.q_heads;
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = is_q ? wq[i] : wk[i];
            const float s[8] = {v[a][0], v[a][1], v[a][2], v[a][3], v[a][4], v[a][5], v[a][6], v[a][7]};
            Lane::norm(w, P.eps, v[a]);
            if (!(is_q ? P.w_q : P.w_k)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[a][i] = s[i];
            }
            ln.rotate(sn, cs, v[a]);
            if (is_q) ln.store(qo + h * D, v[a]);
            else if (h < P.heads) ln.store(ko + (h - P.q_heads) * D, v[a]);
        }
    }
}

template <typename TI, typename TO, int D>
cudaError_t launch_dim(const NormRopeParams& P, cudaStream_t stream) {
    // One token's heads over as many CTAs as bring about four warps to each scheduler: a single
    // token wants every head at once, a prompt the angles computed once.
    const int steps = (P.heads + HeadLane<D>::kHeads - 1) / HeadLane<D>::kHeads;
    const int most = (steps + kRopeWarps - 1) / kRopeWarps;
    const int want = (16 * num_sms() + kRopeWarps * P.m - 1) / (kRopeWarps * P.m);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)P.m, (unsigned)(want < most ? want : most));
    cfg.blockDim = dim3(32 * kRopeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_kernel<TI, TO, D>, P);
}

template <typename TI, typename TO>
cudaError_t launch_typed(const NormRopeParams& P, int head_dim, cudaStream_t stream) {
    if (head_dim == 64) return launch_dim<TI, TO, 64>(P, stream);
    if (head_dim == 128) return launch_dim<TI, TO, 128>(P, stream);
    return launch_dim<TI, TO, 256>(P, stream);
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
