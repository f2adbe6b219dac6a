// q4k_verify.cu -- drafted tokens against the target's distribution, from given random numbers.
//
//   p_r = softmax(logits_r / T); draft d after row r, drawn from q_r, is accepted while u_r q_r(d) < p_r(d).
//   The token after the last accepted one is drawn from max(p_r - q_r, 0) where a draft was rejected, else from p_r:
//   the first j whose cumulative sum exceeds u times the whole.
//
// Whether u lies below a ratio, and between which of some 10^5 cumulative sums, is decided by bits that fp32 sums do not
// have (a vocabulary of 131072 with sums off by 1e-8 would give another token in one draw of a thousand). So only what
// decides is computed precisely, and the whole is read in fp32:
//   1. verify_stats_kernel: each row's largest logit and its sum of 2^(c (x - max)), c = log2(e) / T, in fp32, by chunks of
//      rows over all SMs. Bound by the logits' bytes.
//   2. verify_pick_kernel: a cluster of eight CTAs a sequence. An acceptance whose two sides differ by more than 2^-14 stands;
//      another is computed again from weights good to 2^-41. The token is drawn in such weights, as 64-bit integers in units of
//      2^-b of the row's largest, b = 63 - log2(vocabulary): their sums are exact in any order. One row of logits, and of the drafts' probabilities, is read up to three times, the
//      second and third time from L2.
#include <atomic>

#include "q4k_paged.cuh"

namespace q4k {
namespace {

constexpr int kStatThreads = 256, kStatUnits = 4;   // 16-byte units of a thread in flight
constexpr int kPickThreads = 512, kPickWarps = kPickThreads / 32, kPickCluster = 8, kAllWarps = kPickWarps * kPickCluster;
constexpr float kGreedy = 5.421010862427522e-20f;   // 2^-64: temperatures not above choose the largest logit
constexpr float kLargest = 3.402823466e38f;
// Above the relative error of a decision's two sides in fp32: exponents of up to 100 rounded three times (1.3e-5), ex2, a
// few hundred additions a thread (1.2e-5).
constexpr double kClose = 1.0 / 16384.0;

struct VerifyParams {
    const void* logits;
    const float* probs;
    int64_t logits_stride, probs_stride;
    const int32_t *tokens, *q_start, *seq_lens;
    const float *temperature, *u_accept, *u_sample;
    int32_t *accepted, *next, *kept;
    float4* stats;   // [m][chunks]: largest, sum, its index (bits)
    int batch, m, vocab, chunks;
    int bits;        // weights are integers in units of 2^-bits: 2^(63 - bits) of them add up to less than 2^64
    int* err_flag;
};

// NaN as -inf (such a token has no probability), +inf as the largest finite number.
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, -INFINITY), kLargest); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float one(const float* p) { return __ldcg(p); }
__device__ __forceinline__ float one(const __nv_bfloat16* p) {
    return __uint_as_float((uint32_t)__ldcg(reinterpret_cast<const unsigned short*>(p)) << 16);
}
template <typename T, int V> __device__ __forceinline__ void unpack(const uint4& w, float (&x)[V]) {
    const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(b[i]);
        else { x[2 * i] = __uint_as_float(b[i] << 16); x[2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u); }
    }
}
// The sequence that holds row r, or -1; the whole warp calls it.
__device__ __forceinline__ int sequence_of(const VerifyParams& A, int r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = A.batch;  // the last start <= r is one of lo .. hi
    while (hi - lo >= 32) {
        const int step = (hi - lo) / 32 + 1, i = lo + lane * step;
        const unsigned hit = __ballot_sync(0xffffffffu, i <= hi && __ldcg(A.q_start + i) <= r);
        if (!hit) return -1;
        lo += (31 - __clz(hit)) * step;
        hi = min(hi, lo + step - 1);
    }
    const unsigned hit = __ballot_sync(0xffffffffu, lo + lane <= hi && __ldcg(A.q_start + lo + lane) <= r);
    if (!hit) return -1;
    lo += 31 - __clz(hit);
    return lo < A.batch ? lo : -1;
}

// ---- the rows in fp32 ---------------------------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kStatThreads) verify_stats_kernel(const __grid_constant__ VerifyParams A) {
    constexpr int V = 16 / (int)sizeof(T), W = kStatThreads / 32;
    __shared__ float s_m[W], s_s[W], s_t;
    __shared__ int s_i[W], s_seq;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / A.chunks, chunk = blockIdx.x - row * A.chunks;
    const T* x = static_cast<const T*>(A.logits) + (int64_t)row * A.logits_stride;
    // 16-byte units from the aligned address at or below the row; only units that lie inside the row are read whole
    const int shift = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int units = (A.vocab + shift + V - 1) / V;
    const int u0 = (int)((int64_t)units * chunk / A.chunks), u1 = (int)((int64_t)units * (chunk + 1) / A.chunks);
    auto load = [&](int u, float (&v)[V]) {
        const int e = u * V - shift;
        if (u < u1 && e >= 0 && e + V <= A.vocab) {
            unpack<T, V>(__ldcg(reinterpret_cast<const uint4*>(x + e)), v);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = u < u1 && e + k >= 0 && e + k < A.vocab ? one(x + e + k) : -INFINITY;
        }
    };
    float v[kStatUnits][V];
    auto fetch = [&](int u) {
#pragma unroll
        for (int j = 0; j < kStatUnits; ++j) load(u + j * kStatThreads + tid, v[j]);
    };
    fetch(u0);
    if (warp == 0) {
        const int seq = sequence_of(A, row);
        if (lane == 0) {
            s_seq = seq;
            s_t = seq >= 0 && A.temperature ? __ldcg(A.temperature + seq) : 1.0f;
        }
    }
    __syncthreads();
    if (s_seq < 0) return;
    const bool greedy = !(s_t > kGreedy);
    const float c = 1.44269504088896340736f / s_t;
    float m = -INFINITY, s = 0.0f;
    int best = 0x7FFFFFFF;
    bool tamed = false;
    for (int u = u0;;) {
        if (greedy) {
#pragma unroll
            for (int j = 0; j < kStatUnits; ++j)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float y = tame(v[j][k]);
                    if (y > m) {
                        m = y;
                        best = (u + j * kStatThreads + tid) * V - shift + k;
                    }
                }
        } else {
            float top = m;
#pragma unroll
            for (int j = 0; j < kStatUnits; ++j)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (tamed) v[j][k] = tame(v[j][k]);
                    top = fmaxf(top, v[j][k]);
                }
            if (top > -INFINITY) {
                s *= ex2((m - top) * c);
                if (m == -INFINITY) s = 0.0f;
                m = top;
#pragma unroll
                for (int j = 0; j < kStatUnits; ++j) {
                    float part = 0.0f;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const float w = ex2((v[j][k] - m) * c);
                        part += tamed && v[j][k] == -INFINITY ? 0.0f : w;
                    }
                    s += part;
                }
            }
        }
        u += kStatUnits * kStatThreads;
        if (u >= u1) {
            // NaN, +inf or a c of 0 among them: once more with every logit tamed
            if (tamed || greedy || (s < INFINITY && m < INFINITY)) break;
            tamed = true;
            m = -INFINITY;
            s = 0.0f;
            u = u0;
        }
        fetch(u);
    }
    // the block's
    float top = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (greedy) {
        if (m != top) best = 0x7FFFFFFF;
        best = __reduce_min_sync(0xffffffffu, best);
    } else {
        s = m > -INFINITY ? s * ex2((m - top) * c) : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    if (lane == 0) {
        s_m[warp] = top;
        s_s[warp] = s;
        s_i[warp] = best;
    }
    __syncthreads();
    if (tid) return;
    float all = -INFINITY, sum = 0.0f;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int w = 0; w < W; ++w) all = fmaxf(all, s_m[w]);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (s_m[w] == -INFINITY) continue;
        if (!greedy) sum += s_s[w] * ex2((s_m[w] - all) * c);
        else if (s_m[w] == all) at = min(at, s_i[w]);
    }
    A.stats[blockIdx.x] = make_float4(all, sum, __int_as_float(at), 0.0f);
}

// ---- precise weights ----------------------------------------------------------------------------------------------
// 2^(i/256), i < 256, as two floats: products of the square roots of square roots of 2.
struct Powers {
    float hi[256], lo[256];
};
constexpr Powers make_powers() {
    constexpr double root[8] = {1.414213562373095048801689, 1.189207115002721066717500, 1.090507732665257659207010,
                                1.044273782427413840321966, 1.021897148654116678234480, 1.010889286051700460020410,
                                1.005429901112802821351384, 1.002711275050202485430746};
    Powers p{};
    for (int i = 0; i < 256; ++i) {
        double x = 1.0;
        for (int k = 0; k < 8; ++k)
            if (i >> (7 - k) & 1) x *= root[k];
        p.hi[i] = (float)x;
        p.lo[i] = (float)(x - (double)p.hi[i]);
    }
    return p;
}
__device__ const Powers kPowers = make_powers();

// The weight 2^(c (x - top)) of a logit, relative error 2^-41: the exponent in two floats (2^-46 of itself), cut
// into 256ths and a rest r of at most 2^-9; 2^r = 1 + a + a^2/2 + a^3/6, a = r ln 2, whose next term is below 2^-42.
struct Weigher {
    const float2* pow;   // in shared memory
    float top, c_hi, c_lo;
    int bits;
    __device__ __forceinline__ Weigher(const float2* p, float t, float temperature, int b) : pow(p), top(t), bits(b) {
        const double c = 1.4426950408889634074 / (double)temperature;
        c_hi = (float)c;
        c_lo = (float)(c - (double)c_hi);
    }
    // mantissa in [2^43, 2^44) and exponent: weight = mant 2^(e - 43). False: below 2^-1000, or no probability.
    __device__ __forceinline__ bool parts(float x, uint64_t* mant, int* e) const {
        // x - top in two floats, then times c
        const float d = x - top, b = d - x, dl = (x - (d - b)) + (-top - b);
        const float y = d * c_hi;
        if (!(y > -1000.0f)) return false;
        const float yl = fmaf(d, c_hi, -y) + fmaf(d, c_lo, dl * c_hi);
        const float k = rintf(y * 256.0f);
        const int n = (int)k;
        const float r = fmaf(k, -1.0f / 256.0f, y);   // exact
        const float a = r * 0.693147180559945309417f;  // ln 2 = this float and the one below
        const float al = fmaf(r, 0.693147180559945309417f, -a) + fmaf(r, -1.904654299957768e-9f, yl * 0.693147180559945309417f);
        const float z = a + al, s = fmaf(z * z, fmaf(z, 1.0f / 6.0f, 0.5f), al);   // al has the exponent's second float, too: up to 2^-19
        const float2 t = pow[n & 255];
        const float b1 = t.x * a;
        const float b2 = fmaf(t.x, s, fmaf(t.y, a, t.y + fmaf(t.x, a, -b1)));
        // t.x + b1 + b2 in units of 2^-43: |b1| below 2^-8, |b2| below 2^-18
        *mant = ((uint64_t)((__float_as_uint(t.x) & 0x7FFFFFu) | 0x800000u) << 20) + __float2ll_rn(b1 * 8796093022208.0f) +
                __float2int_rn(b2 * 8796093022208.0f);
        *e = n >> 8;
        return true;
    }
    __device__ __forceinline__ uint64_t operator()(float x) const {  // in units of 2^-bits, rounded; 0 for tokens without probability
        uint64_t mant;
        int e;
        if (!parts(x, &mant, &e)) return 0;
        const int up = e + bits - 43;
        return up >= 0 ? mant << up : up < -45 ? 0 : ((mant >> (-up - 1)) + 1) >> 1;
    }
};
// floor(f * s) for f in [0, 1] (above: s, below or NaN: 0), s < 2^63.
__device__ __forceinline__ uint64_t portion(float f, uint64_t s) {
    if (!(f > 0.0f)) return 0;
    if (f >= 1.0f) return s;
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const uint64_t m = e ? (b & 0x7FFFFFu) | 0x800000u : (uint64_t)(b & 0x7FFFFFu) << 1;  // f = m 2^(e - 150)
    const int down = 126 - (int)e;
    return down >= 64 ? 0 : __umul64hi(m << 40, s) >> down;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ uint64_t peer_u64(const uint64_t* p, int rank) {
    uint64_t v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u64 %0, [a];\n\t}"
                 : "=l"(v)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sync_cluster() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// VEC: the rows of logits and probabilities are 16-byte aligned, so a lane takes 16 bytes of logits at a time, else one element.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kPickThreads) verify_pick_kernel(const __grid_constant__ VerifyParams A) {
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
    __shared__ float2 s_pow[256];
    __shared__ uint64_t s_part[2][kPickWarps], s_all[kAllWarps];
    __shared__ int s_stop, s_close;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, seq = blockIdx.x / kPickCluster;
    const int rank = blockIdx.x - seq * kPickCluster;
    if (tid < 256) s_pow[tid] = make_float2(kPowers.hi[tid], kPowers.lo[tid]);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int a = __ldcg(A.q_start + seq), b = __ldcg(A.q_start + seq + 1);
    const int start = min(max(a, 0), A.m), n = min(max(b, start), A.m) - start;
    const bool writes = rank == 0 && tid == 0;
    if (writes && (start != a || start + n != b)) raise_flag(A.err_flag, Q4K_ERR_SEQ);
    const int len = A.seq_lens ? __ldcg(A.seq_lens + seq) : 0;
    if (n == 0) {
        if (writes) {
            A.accepted[seq] = 0;
            A.next[seq] = -1;
            if (A.kept) A.kept[seq] = len;
        }
        return;
    }
    const float temperature = A.temperature ? __ldcg(A.temperature + seq) : 1.0f;
    const bool greedy = !(temperature > kGreedy);
    const float c = 1.44269504088896340736f / temperature;

    // A row's largest logit, its sum in fp32 and the largest's index, over its chunks; the whole warp calls it.
    struct Row { float top, sum; int best; };
    auto row_of = [&](int r) {
        Row R{-INFINITY, 0.0f, 0x7FFFFFFF};
        for (int k = lane; k < A.chunks; k += 32) {
            const float4 f = __ldcg(A.stats + (int64_t)r * A.chunks + k);
            if (f.x > R.top) {
                R.sum = R.sum * ex2((R.top - f.x) * c);
                if (R.top == -INFINITY) R.sum = 0.0f;
                R.top = f.x;
                R.best = __float_as_int(f.z);
                R.sum += f.y;
            } else if (f.x > -INFINITY) {
                R.sum += f.y * ex2((f.x - R.top) * c);   // an equal one of a later chunk has the higher index
            }
        }
        float top = R.top;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        R.sum = R.top > -INFINITY ? R.sum * ex2((R.top - top) * c) : 0.0f;
        if (R.top != top || top == -INFINITY) R.best = 0x7FFFFFFF;
        R.top = top;
#pragma unroll
        for (int o = 16; o; o >>= 1) R.sum += __shfl_xor_sync(0xffffffffu, R.sum, o);
        R.best = __reduce_min_sync(0xffffffffu, R.best);
        return R;
    };
    auto logit = [&](int r, int d) { return tame(one(static_cast<const T*>(A.logits) + (int64_t)r * A.logits_stride + d)); };
    // u q(d): what p(d) has to exceed
    auto bar = [&](int r, int d) {
        const double u = fmaxf(__ldcg(A.u_accept + r), 0.0f);
        return A.probs ? u * (double)fmaxf(__ldcg(A.probs + (int64_t)r * A.probs_stride + d), 0.0f) : u;
    };
    enum { kYes, kNo, kAsk };
    auto decide = [&](int r) {
        const Row R = row_of(r);
        const int d = __ldcg(A.tokens + r + 1);
        if ((unsigned)d >= (unsigned)A.vocab) {
            if (rank == 0 && lane == 0) raise_flag(A.err_flag, Q4K_ERR_TOKEN);
            return (int)kNo;
        }
        const float x = logit(r, d);
        const double need = bar(r, d);
        if (x == -INFINITY) return (int)kNo;
        if (greedy) return (int)(d == R.best && need < 1.0 ? kYes : kNo);
        if (need == 0.0) return (int)kYes;
        const float w = ex2((x - R.top) * c);
        const double l = need * (double)R.sum;
        if (w < 1e-30f) return (int)kAsk;
        return (int)(l * (1.0 + kClose) < (double)w ? kYes : l * (1.0 - kClose) >= (double)w ? kNo : kAsk);
    };

    // this warp's part of a row, in the order of the tokens: 32 lanes of V at a time
    const int all_warp = rank * kPickWarps + warp;
    const int seg = ((A.vocab + kAllWarps - 1) / kAllWarps + 32 * V - 1) / (32 * V) * (32 * V);
    const int e0 = min(all_warp * seg, A.vocab), e1 = min(e0 + seg, A.vocab);
    auto logits_at = [&](const T* x, int e, float (&v)[V]) {
        if (VEC && e + V <= A.vocab) {
            if constexpr (VEC) unpack<T, V>(__ldcg(reinterpret_cast<const uint4*>(x + e)), v);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = e + k < A.vocab ? one(x + e + k) : -INFINITY;
        }
    };
    auto probs_at = [&](const float* q, int e, float (&v)[V]) {
        if (VEC && e + V <= A.vocab) {
            if constexpr (VEC) {
#pragma unroll
                for (int k = 0; k < V; k += 4) {
                    const float4 f = __ldcg(reinterpret_cast<const float4*>(q + e + k));
                    v[k] = f.x; v[k + 1] = f.y; v[k + 2] = f.z; v[k + 3] = f.w;
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = e + k < A.vocab ? __ldcg(q + e + k) : 0.0f;
        }
    };
    // every warp's sum of the cluster's 128, in s_all, and their total
    int turn = 0;
    bool gathered = false;
    auto gather = [&](uint64_t mine) {
        gathered = true;
        if (lane == 0) s_part[turn][warp] = mine;
        sync_cluster();
        if (tid < kAllWarps) s_all[tid] = peer_u64(&s_part[turn][tid % kPickWarps], tid / kPickWarps);
        __syncthreads();
        turn ^= 1;   // written again only after the next gather's barrier
        uint64_t t = 0;
        for (int k = lane; k < kAllWarps; k += 32) t += s_all[k];
        return warp_sum(t);
    };
    auto weights_of = [&](const Weigher& W, int r) {
        const T* x = static_cast<const T*>(A.logits) + (int64_t)r * A.logits_stride;
        uint64_t t = 0;
        for (int e = e0 + lane * V; e < e1; e += 32 * V) {
            float v[V];
            logits_at(x, e, v);
#pragma unroll
            for (int k = 0; k < V; ++k) t += W(tame(v[k]));
        }
        return warp_sum(t);
    };

    // how many drafts are accepted
    int at = 0;
    uint64_t whole = 0;      // the row's sum, once it is known
    bool rejected = false;
    while (at < n - 1) {
        if (tid == 0) s_stop = s_close = 0x7FFFFFFF;
        __syncthreads();
        for (int j = at + warp; j < n - 1; j += kPickWarps) {
            const int said = decide(start + j);
            if (said == kYes) continue;
            if (lane == 0) {
                atomicMin(&s_stop, j);
                if (said == kAsk) atomicMin(&s_close, j);
            }
            break;
        }
        __syncthreads();
        const int stop = s_stop, close = s_close;
        __syncthreads();
        whole = 0;
        if (stop == 0x7FFFFFFF) {
            at = n - 1;
            break;
        }
        at = stop;
        rejected = true;
        if (close != stop) break;
        const int r = start + stop, d = __ldcg(A.tokens + r + 1);
        const Weigher W(s_pow, row_of(r).top, temperature, A.bits);
        whole = gather(weights_of(W, r));
        uint64_t mant;
        int e;
        const bool some = W.parts(logit(r, d), &mant, &e);
        if (!some || !(bar(r, d) * (double)whole < scalbn((double)mant, e + A.bits - 43))) break;
        rejected = false;
        whole = 0;
        ++at;
    }
    // the token after them
    const int r = start + at;
    const Row R = row_of(r);
    if (writes) {
        A.accepted[seq] = at;
        if (A.kept) A.kept[seq] = len - n + 1 + at;
    }
    if (greedy || R.top == -INFINITY) {
        if (writes) {
            A.next[seq] = R.top == -INFINITY ? -1 : R.best;
            if (R.top == -INFINITY) raise_flag(A.err_flag, Q4K_ERR_TOKEN);
        }
        if (gathered) sync_cluster();   // no CTA leaves while another reads its sums
        return;
    }
    const Weigher W(s_pow, R.top, temperature, A.bits);
    __syncthreads();   // s_pow, where no draft was looked at
    if (!whole) whole = gather(weights_of(W, r));
    const T* x = static_cast<const T*>(A.logits) + (int64_t)r * A.logits_stride;
    const float* q = A.probs ? A.probs + (int64_t)r * A.probs_stride : nullptr;
    const int drafted = rejected ? __ldcg(A.tokens + r + 1) : -1;
    // what is left of a token's weight
    bool minus = rejected;
    auto left = [&](int e, float y, float qe) {
        const uint64_t w = W(tame(y));
        if (!minus) return w;
        if (!q) return e == drafted ? (uint64_t)0 : w;
        const uint64_t away = portion(qe, whole);
        return w > away ? w - away : (uint64_t)0;
    };
    uint64_t rest = whole;
    if (rejected) {
        uint64_t t = 0;
        for (int e = e0 + lane * V; e < e1; e += 32 * V) {
            float v[V], p[V];
            logits_at(x, e, v);
            if (q) probs_at(q, e, p);
#pragma unroll
            for (int k = 0; k < V; ++k) t += left(e + k, v[k], q ? p[k] : 0.0f);
        }
        rest = gather(warp_sum(t));
        if (rest == 0) {   // nothing is left: from the distribution itself
            minus = false;
            rest = gather(weights_of(W, r));
        }
    }
    // the first token whose cumulative sum exceeds u * rest: the warp that holds it, then its place there
    const uint64_t goal = min(portion(__ldcg(A.u_sample + seq), rest), rest - 1);
    uint64_t before = 0;
    for (int k = lane; k < all_warp; k += 32) before += s_all[k];
    before = warp_sum(before);
    if (goal >= before && goal - before < s_all[all_warp]) {
        for (int base = e0; base < e1; base += 32 * V) {
            const int e = base + lane * V;
            float v[V], p[V];
            uint64_t w[V], own = 0;
            logits_at(x, e, v);
            if (q) probs_at(q, e, p);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                w[k] = e + k < e1 ? left(e + k, v[k], q ? p[k] : 0.0f) : 0;
                own += w[k];
            }
            uint64_t inc = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, before + inc > goal);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    uint64_t cum = before + inc - own;
                    int found = -1;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        cum += w[k];
                        if (found < 0 && cum > goal) found = e + k;
                    }
                    A.next[seq] = found;
                }
                break;
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    sync_cluster();
}

int chunks_of(int m, int vocab) {
    // Eight CTAs on each of 152 SMs where there are few rows (but 4096 logits a CTA at least), pieces of up to 16384 where there
    // are many.
    const int64_t want = (8 * 152 + (int64_t)m - 1) / (m < 1 ? 1 : m), most = (vocab + 4095) / 4096, least = (vocab + 16383) / 16384;
    return (int)(want > most ? most : want < least ? least : want);
}

template <typename T>
cudaError_t launch_typed(const VerifyParams& P, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)P.m * P.chunks));
    cfg.blockDim = dim3(kStatThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kPickCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (P.m > 0) {
        const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_stats_kernel<T>, P);
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3((unsigned)P.batch * kPickCluster);
    cfg.blockDim = dim3(kPickThreads);
    cfg.numAttrs = 2;
    const auto even = [](const void* p, int64_t stride, int size) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * size % 16 == 0;
    };
    const bool vec = even(P.logits, P.logits_stride, (int)sizeof(T)) && even(P.probs, P.probs ? P.probs_stride : 0, 4);
    return vec ? cudaLaunchKernelEx(&cfg, verify_pick_kernel<T, true>, P) : cudaLaunchKernelEx(&cfg, verify_pick_kernel<T, false>, P);
}

}  // namespace

size_t verify_workspace_bytes(int m, int vocab) { return sizeof(float4) * (size_t)m * chunks_of(m, vocab); }

cudaError_t launch_verify(const void* logits, int dtype, int m, int vocab, int64_t logits_stride, const float* probs,
                          int64_t probs_stride, const int32_t* tokens, const int32_t* q_start, int batch,
                          const float* temperature, const float* u_accept, const float* u_sample, const int32_t* seq_lens,
                          int32_t* accepted, int32_t* next, int32_t* kept, void* workspace, int* err_flag, cudaStream_t stream) {
    VerifyParams P{};
    P.logits = logits; P.probs = probs; P.logits_stride = logits_stride; P.probs_stride = probs_stride;
    P.tokens = tokens; P.q_start = q_start; P.seq_lens = seq_lens; P.temperature = temperature;
    P.u_accept = u_accept; P.u_sample = u_sample; P.accepted = accepted; P.next = next; P.kept = kept;
    P.stats = static_cast<float4*>(workspace);
    P.batch = batch; P.m = m; P.vocab = vocab; P.chunks = chunks_of(m, vocab); P.err_flag = err_flag;
    P.bits = 63;
    while ((int64_t)1 << (63 - P.bits) < vocab) --P.bits;
    return dtype == Q4K_F32 ? launch_typed<float>(P, stream) : launch_typed<__nv_bfloat16>(P, stream);
}

}  // namespace q4k
