// q4k_qkrope.cu -- the norm of each query and key head with the position rotation in the same pass.
//
//   y = x * w / sqrt(mean_c x_c^2 + eps)   (per head; no weight: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin) over the first rot_dim dims, angle pos[t] * inv_freq[j]
// head_dim / 8 lanes hold a head (8 dims each, whole pairs, so the rotation needs no exchange), everything
// in fp32 and rounded once at the store. A CTA is one token's heads, or a share of them where tokens are few:
// its sines, cosines and weights go to shared memory once (a warp's own cost more than the bytes: 62 us for the
// prompt below), and a warp takes one step of heads after the other.
//
// Bound by bytes: 8192 tokens of 40 heads of 128 in bf16, 168 MB, 35 us, 4.8 TB/s. What hides the latency is
// warps, 64 an SM at 32 registers: two to four steps in flight per warp, at 70 to 114 registers, took 50 to 78 us.
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
constexpr int kRopeCtas = 16;  // of an SM: all its warps, at 32 registers

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeCtas) norm_rope_kernel(const __grid_constant__ NormRopeParams P) {
    using Lane = HeadLane<D>;
    __shared__ __align__(16) float s_sn[D / 2], s_cs[D / 2], s_w[2][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = blockIdx.x, sub = (threadIdx.x & 31) / Lane::kLanes;
    const Lane ln(P.rot_dim, P.pairs_mode);
    const int stride = gridDim.y * kRopeWarps * Lane::kHeads;
    const TI* q = static_cast<const TI*>(P.q) + t * P.q_stride;
    const TI* k = static_cast<const TI*>(P.k) + t * P.k_stride;
    TO* qo = static_cast<TO*>(P.q_out) + t * P.q_out_stride;
    TO* ko = static_cast<TO*>(P.k_out) + t * P.k_out_stride;
    // h0 is the same in all lanes of a warp; a lane's head is h0 + its group
    int h0 = (blockIdx.y * kRopeWarps + (threadIdx.x >> 5)) * Lane::kHeads;
    auto take = [&](int h, float (&v)[8]) {
        if (h < P.q_heads) ln.load(q + h * D, v);
        else if (h < P.heads) ln.load(k + (h - P.q_heads) * D, v);
    };
    float v[8] = {};
    take(h0 + sub, v);
    // every read is on its way before the first is looked at
    static_assert(D / 2 <= 32 * kRopeWarps, "an angle a thread");
    constexpr int kEach = D > 32 * kRopeWarps ? D / (32 * kRopeWarps) : 1;
    const int i = threadIdx.x;
    const bool turns = 2 * i < P.rot_dim;
    const int pos = turns ? __ldcg(P.pos + t) : 0;
    const double f = turns ? __ldcg(P.inv_freq + i) : 0.0;
    uint16_t w[2][kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (const int c = i + 32 * kRopeWarps * j; c < D) {
            w[0][j] = P.w_q ? __ldcg(P.w_q + c) : 0x3F80;  // a side without weights multiplies by ones
            w[1][j] = P.w_k ? __ldcg(P.w_k + c) : 0x3F80;
        }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (const int c = i + 32 * kRopeWarps * j; c < D) {
            s_w[0][c] = __uint_as_float((uint32_t)w[0][j] << 16);
            s_w[1][c] = __uint_as_float((uint32_t)w[1][j] << 16);
        }
    if (turns) turn_sincos(pos, turn_fraction(f), &s_sn[i], &s_cs[i]);
    __syncthreads();
    float sn[4], cs[4];
    if (ln.turns) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sn[j] = s_sn[ln.j0 + j];
            cs[j] = s_cs[ln.j0 + j];
        }
    }
#pragma unroll 1
    for (; h0 < P.heads; h0 += stride) {
        const int h = h0 + sub;
        const bool is_q = h < P.q_heads;
        // the norm is computed for a side without weights too (the warp's lanes stay together), and dropped
        float r = Lane::inv_rms(P.eps, v), g[8];
        if (!(is_q ? P.w_q : P.w_k)) r = 1.0f;
        ln.shared(is_q ? s_w[0] : s_w[1], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * r * g[i];
        ln.rotate(sn, cs, v);
        if (is_q) ln.store(qo + h * D, v);
        else if (h < P.heads) ln.store(ko + (h - P.q_heads) * D, v);
        take(h + stride, v);
    }
}

template <typename TI, typename TO, int D>
cudaError_t launch_dim(const NormRopeParams& P, cudaStream_t stream) {
    // One token's heads over as many CTAs as bring about four warps to each scheduler: a single
    // token wants every head at once, a prompt the angles computed once.
    const int steps = (P.heads + HeadLane<D>::kHeads - 1) / HeadLane<D>::kHeads;
    const int most = (steps + kRopeWarps - 1) / kRopeWarps;
    const int64_t want = (16 * num_sms() + kRopeWarps * (int64_t)P.m - 1) / (kRopeWarps * (int64_t)P.m);
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
