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
// Single tokens (up to two a sequence): a warp per item, bound by latency, a chain of lengths, page and row, scale:
// 2.6 us for one sequence, 6.7 for 256 of 8 heads. Item i < batch is sequence i's first page, so a decode batch
// finds its work without a search; further pages are found by a scan over the sequences. Prompts: a CTA per
// (page, side) that takes heads one after the other, the next one's rows on their way, so that the chain and the
// sines are paid once: 8191 tokens of 8 heads of 128 in bf16, 50 MB, 23 us, 2.2 TB/s (a CTA per head: 28). Each
// head still waits for its largest magnitude before its codes can be written, about 1.5 us with two CTAs an SM.
#include <atomic>

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

// The w-th page beyond the sequences' first ones (every warp finds it by itself); false past the last. A lane takes
// kEach sequences at a time, so that their reads are in flight together: one by one, the CTAs that find nothing were
// the last to end (7.2 us for 256 sequences of a token each).
__device__ __forceinline__ bool further_page(const PagedBatch& B, int w, int* err_flag, int* seq, int* page, SeqSpan* span) {
    constexpr int kEach = 8;
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < B.batch; base += 32 * kEach) {
        int cnt[kEach], p0[kEach], sum = 0;
        SeqSpan s[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = base + lane * kEach + j;
            cnt[j] = p0[j] = 0;
            s[j] = SeqSpan{0, 0, 0};
            if (i < B.batch) cnt[j] = max(touched_pages(B, i, err_flag, &s[j], &p0[j]) - 1, 0);
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) sum += cnt[j];
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, w < inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            int rest = w - (inc - sum), at = 0, from = 0, first = 0;  // in lane src: which of its sequences, which page
            SeqSpan f{0, 0, 0};
            bool found = false;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                if (!found && rest < cnt[j]) {
                    found = true;
                    at = j;
                    from = rest;
                    first = p0[j];
                    f = s[j];
                }
                if (!found) rest -= cnt[j];
            }
            *seq = base + src * kEach + __shfl_sync(0xffffffffu, at, src);
            *page = __shfl_sync(0xffffffffu, first + 1 + from, src);
            span->start = __shfl_sync(0xffffffffu, f.start, src);
            span->n = __shfl_sync(0xffffffffu, f.n, src);
            span->len = __shfl_sync(0xffffffffu, f.len, src);
            return true;
        }
        w -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

// What one (page, head, side) is made of: its new slots [lo, hi), where its codes and scale lie, its input rows.
template <typename T, int D, int P>
struct Side {
    int lo, hi;
    int64_t stride;
    const T* x;  // slot s's row of head h: x + s * stride + h * D
    bool keys;
    __device__ __forceinline__ Side(const AppendParams& A, int page, const SeqSpan& s, bool k) {
        const int first = s.len - s.n;  // position of the first new row
        lo = max(max(first, 0) - page * P, 0);
        hi = min(s.len - page * P, P);
        keys = k;
        stride = k ? A.k_stride : A.v_stride;
        x = static_cast<const T*>(k ? A.k : A.v) + (int64_t)(s.start + page * P - first) * stride;
    }
    __device__ __forceinline__ uint8_t* codes(const AppendParams& A, int pid, int head, int heads) const {
        return (keys ? A.k_cache : A.v_cache) + ((int64_t)pid * heads + head) * (P * D);
    }
    __device__ __forceinline__ float* scale(const AppendParams& A, int pid, int head, int heads) const {
        return (keys ? A.k_scale : A.v_scale) + (int64_t)pid * heads + head;
    }
};

__device__ __forceinline__ float finite_amax(const float (&v)[8], float amax) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = fabsf(v[j]);
        if (a <= 3.402823466e38f) amax = fmaxf(amax, a);  // infinities saturate, NaN stays NaN
    }
    return amax;
}
__device__ __forceinline__ float warp_max(float a) {  // a >= 0
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
}
template <int D>
__device__ __forceinline__ void put_codes(uint8_t* row, const HeadLane<D>& ln, const float (&v)[8], float inv) {
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = f32x2_to_e4m3x2(v[2 * j] * inv, v[2 * j + 1] * inv);
    *reinterpret_cast<uint32_t*>(row + ln.c0) = q[0] | (q[1] << 16);
    *reinterpret_cast<uint32_t*>(row + ln.c1) = q[2] | (q[3] << 16);
}
// The n codes that the page held, rounded again under its grown scale (a power of two: ratio is exact).
__device__ __forceinline__ void round_again(uint8_t* codes, int n, float ratio, int thread, int threads) {
    for (int i = 16 * thread; i < n; i += 16 * threads) {
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

// One (page, head, side) by one warp. Rows are taken in sets of heads-per-warp * HELD; the rows of a single
// set stay in registers between the two passes (largest magnitude, codes), more sets are read and computed again.
template <typename T, int D, int P, int HELD>
__device__ __forceinline__ void append_tokens(const AppendParams& A, int seq, int page, const SeqSpan& s, int head,
                                              int heads, bool keys) {
    using Lane = HeadLane<D>;
    constexpr int kSet = Lane::kHeads * HELD;
    const int entry = page_entry(A.B, seq, page);  // looked at once the rows are on their way
    const int lane = threadIdx.x & 31, sub = lane / Lane::kLanes;
    const Side<T, D, P> S(A, page, s, keys);
    const Lane ln(keys ? A.rot_dim : 0, A.pairs_mode);
    float w[8];
    uint64_t F[4];
    const bool norm = keys && A.w_k != nullptr, rot = keys && A.rot_dim;
    float v[HELD][8];
    auto read = [&](int set) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int slot = set * kSet + i * Lane::kHeads + sub;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            if (slot >= S.lo && slot < S.hi) ln.load(S.x + slot * S.stride + head * D, v[i]);
        }
    };
    auto turn = [&](int set) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int slot = set * kSet + i * Lane::kHeads;
            if (slot >= S.hi || slot + Lane::kHeads <= S.lo) continue;  // the same in all lanes
            if (norm) Lane::norm(w, A.eps, v[i]);
            if (rot) {
                float sn[4], cs[4];
                ln.angles(page * P + slot + sub, F, sn, cs);
                ln.rotate(sn, cs, v[i]);
            }
        }
    };
    const int set0 = S.lo / kSet, set1 = (S.hi - 1) / kSet;
    read(set0);
    if (norm) ln.load(reinterpret_cast<const __nv_bfloat16*>(A.w_k), w);
    double f[4];
    if (rot) ln.frequencies(A.inv_freq, f);
    const int pid = page_checked(A.B, entry, A.err_flag);
    if (pid < 0) return;  // the same in all lanes
    float* sp = S.scale(A, pid, head, heads);
    uint8_t* codes = S.codes(A, pid, head, heads);
    const float old = S.lo > 0 ? __ldcg(sp) : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) F[i] = rot ? turn_fraction(f[i]) : 0;
    float amax = 0.0f;
    for (int set = set0; set <= set1; ++set) {
        if (set != set0) read(set);
        turn(set);
#pragma unroll
        for (int i = 0; i < HELD; ++i) amax = finite_amax(v[i], amax);
    }
    const float scale = fmaxf(exp2_int(scale_exponent(warp_max(amax))), old);
    if (lane == 0) *sp = scale;  // every lane has read the old one
    const float inv = 1.0f / scale;  // exact: a power of two
    for (int set = set0; set <= set1; ++set) {
        if (set0 != set1) {
            read(set);
            turn(set);
        }
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int slot = set * kSet + i * Lane::kHeads + sub;
            if (slot >= S.lo && slot < S.hi) put_codes<D>(codes + slot * D, ln, v[i], inv);
        }
    }
    if (S.lo > 0 && scale != old) round_again(codes, S.lo * D, old * inv, lane, 32);
}

constexpr int kTokenWarps = 4;
constexpr int kFill = 4;  // CTAs an SM that a page's heads are shared out for (2 to 4: 23 us; 6: 25; 12, a head each: 35)
template <int D, int P> constexpr int kPageWarps = D * P > 8192 ? 16 : 8;  // four rows a lane, at most

// One (page, side) by a CTA, heads blockIdx.y, blockIdx.y + gridDim.y, ..: every row stays in registers between the
// passes, and the rotation's sines and cosines are computed once for all heads.
template <typename T, int D, int P>
__device__ __forceinline__ void append_page(const AppendParams& A, int seq, int page, const SeqSpan& s, int heads, bool keys) {
    using Lane = HeadLane<D>;
    constexpr int W = kPageWarps<D, P>, kRows = W * Lane::kHeads, kHeld = (P + kRows - 1) / kRows;
    extern __shared__ __align__(16) float s_turn[];  // [P][sines D / 2, cosines D / 2]
    __shared__ float s_max[2][W];
    const int entry = page_entry(A.B, seq, page);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / Lane::kLanes;
    const Side<T, D, P> S(A, page, s, keys);
    const Lane ln(keys ? A.rot_dim : 0, A.pairs_mode);
    const bool norm = keys && A.w_k != nullptr, rot = keys && A.rot_dim;
    float w[8];
    typename Lane::template Raw<T> next[kHeld];
    auto read = [&](int head) {
        if (head >= heads) return;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int slot = (i * W + warp) * Lane::kHeads + sub;
            if (slot >= S.lo && slot < S.hi) ln.load(S.x + slot * S.stride + head * D, next[i]);  // else it stays 0
        }
    };
    read(blockIdx.y);
    if (norm) ln.load(reinterpret_cast<const __nv_bfloat16*>(A.w_k), w);
    if (rot) {
        const int pair = threadIdx.x % (D / 2);
        if (2 * pair < A.rot_dim) {
            const uint64_t F = turn_fraction(__ldcg(A.inv_freq + pair));
            for (int slot = S.lo + threadIdx.x / (D / 2); slot < S.hi; slot += 32 * W / (D / 2))
                turn_sincos(page * P + slot, F, s_turn + slot * D + pair, s_turn + slot * D + D / 2 + pair);
        }
    }
    const int pid = page_checked(A.B, entry, A.err_flag);
    if (pid < 0) return;  // the same in all threads
    __syncthreads();
    int turn = 0;
    for (int head = blockIdx.y; head < heads; head += gridDim.y, turn ^= 1) {
        float v[kHeld][8];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) Lane::unpack(next[i], v[i]);
        read(head + gridDim.y);  // on its way while this head's rows are worked on
        float* sp = S.scale(A, pid, head, heads);
        uint8_t* codes = S.codes(A, pid, head, heads);
        const float old = S.lo > 0 ? __ldcg(sp) : 0.0f;
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int slot = (i * W + warp) * Lane::kHeads;
            if (slot >= S.hi || slot + Lane::kHeads <= S.lo) continue;  // the same in all lanes
            if (norm) Lane::norm(w, A.eps, v[i]);
            if (rot && ln.turns) {
                const float* at = s_turn + (slot + sub) * D + ln.j0;  // slots outside [lo, hi): not written, not used
                float sn[4], cs[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) { sn[j] = at[j]; cs[j] = at[D / 2 + j]; }
                if (slot + sub >= S.lo && slot + sub < S.hi) ln.rotate(sn, cs, v[i]);
            }
            amax = finite_amax(v[i], amax);
        }
        amax = warp_max(amax);
        if (lane == 0) s_max[turn][warp] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) amax = fmaxf(amax, s_max[turn][i]);
        const float scale = fmaxf(exp2_int(scale_exponent(amax)), old);
        if (threadIdx.x == 0) *sp = scale;  // every thread has read the old one
        const float inv = 1.0f / scale;     // exact: a power of two
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int slot = (i * W + warp) * Lane::kHeads + sub;
            if (slot >= S.lo && slot < S.hi) put_codes<D>(codes + slot * D, ln, v[i], inv);
        }
        if (S.lo > 0 && scale != old) round_again(codes, S.lo * D, old * inv, threadIdx.x, 32 * W);
    }
}

// A CTA per (page, side) and share of the heads: grid (batch first pages, then CTAs that walk over further pages;
// shares; 2).
template <typename T, int D, int P>
__global__ void __launch_bounds__(32 * kPageWarps<D, P>) append_pages_kernel(const __grid_constant__ AppendParams A, int heads) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int seq = blockIdx.x, page;
    SeqSpan s;
    if (seq < A.B.batch) {
        if (touched_pages(A.B, seq, A.err_flag, &s, &page) == 0) return;
        append_page<T, D, P>(A, seq, page, s, heads, blockIdx.z == 0);
        return;
    }
    for (int w = blockIdx.x - A.B.batch; further_page(A.B, w, A.err_flag, &seq, &page, &s); w += gridDim.x - A.B.batch) {
        append_page<T, D, P>(A, seq, page, s, heads, blockIdx.z == 0);
        __syncthreads();  // the shared memory is free again
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
        append_tokens<T, D, P, 2>(A, seq, page, s, hs >> 1, heads, (hs & 1) == 0);
        return;
    }
    for (int w = blockIdx.x - A.B.batch; further_page(A.B, w, A.err_flag, &seq, &page, &s); w += gridDim.x - A.B.batch)
        append_tokens<T, D, P, 2>(A, seq, page, s, hs >> 1, heads, (hs & 1) == 0);
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
    // Mostly single tokens: a warp an item; else the CTA that shares a page's rows. 64 sequences of 1 token 3.8 us and
    // 6.7, of 4 4.2 and 9.8; 8 of 16 tokens 9.7 and 4.2. The mean is all the host knows, and a prompt among single
    // tokens costs a warp up to 64 rounds of reads a page, so the bound is low.
    if (A.B.m <= 2 * (int64_t)A.B.batch) {
        cfg.gridDim = dim3((unsigned)items, (unsigned)((2 * kv_heads + kTokenWarps - 1) / kTokenWarps));
        cfg.blockDim = dim3(32 * kTokenWarps);
        return cudaLaunchKernelEx(&cfg, append_tokens_kernel<T, D, P>, A, kv_heads);
    }
    // The heads of a page in as many shares as fill the SMs once.
    const int fill = kFill * num_sms() / (2 * items), shares = fill < 1 ? 1 : fill < kv_heads ? fill : kv_heads;
    const size_t smem = (size_t)P * D * sizeof(float);
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(append_pages_kernel<T, D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        allowed[dev].store(true, std::memory_order_relaxed);
    }
    cfg.gridDim = dim3((unsigned)items, (unsigned)shares, 2);
    cfg.blockDim = dim3(32 * kPageWarps<D, P>);
    cfg.dynamicSmemBytes = A.rot_dim ? smem : 0;
    return cudaLaunchKernelEx(&cfg, append_pages_kernel<T, D, P>, A, kv_heads);
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
