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
//   2. verify_pick_kernel: a cluster of up to eight CTAs a sequence. An acceptance whose two sides differ by more than 2^-14 stands;
//      another is computed again from weights good to 2^-41. The token is drawn in weights good to 2^-31, as 64-bit integers in units of
//      2^-b of the row's largest, b = 62 - log2(vocabulary): their sums are exact in any order. One row of logits, and of the drafts' probabilities, is read once.
//      Bound by instructions, 58 a token, where there are many sequences, by each CTA's chain of loads, sums and barriers where there are few.
// 256 sequences of 4 rows of 131072 fp32: 85 us (6.3 TB/s) and 96; 64 of up to 6 rows in bf16: 57 together; one of 5 rows of 32000: 11.5.
// Both in one kernel, a cluster going through its rows one after another: 172 to 177, 62 and 15 us.
#include <atomic>

#include "q4k_paged.cuh"

namespace q4k {
namespace {

constexpr int kStatThreads = 256;
constexpr int kPickThreads = 256, kPickWarps = kPickThreads / 32, kMostCluster = 8;
constexpr int kSeg = 512;                           // tokens of a segment, whose sum is kept
constexpr float kGreedy = 5.421010862427522e-20f;   // 2^-64: temperatures not above choose the largest logit
constexpr float kLargest = 3.402823466e38f;
// The relative error of a decision's two sides in fp32 is below (1.4 |y| + 94) 2^-23, y the draft's exponent: four roundings of y
// (4 ln 2 2^-24 |y|), the same in the sum, where the mean of |y| is the distribution's entropy at most (20 bits), ex2 (2 2^-23), up to
// thirteen changes of a thread's largest (26 2^-23), and some sixty additions one after another (30 2^-23).
__device__ __forceinline__ float closeness(float y) { return fmaf(fabsf(y), 1.5f, 96.0f) * 1.1920929e-7f; }
// And where it is computed from the draw's weights: 2^-31 of themselves (the sum and the draft's, 32 times that here), and each cut to the
// sums' unit, so that a sum of n may be n units short.
constexpr double kCloseFine = 1.0 / 67108864.0;
// The precise sum has this many more bits behind the unit: all its weights together are short by one unit at most.
constexpr int kFineBits = 20;

struct VerifyParams {
    const void* logits;
    const float* probs;
    int64_t logits_stride, probs_stride;
    const int32_t *tokens, *q_start, *seq_lens;
    const float *temperature, *u_accept, *u_sample;
    int32_t *accepted, *next, *kept;
    float4* stats;   // [m][chunks]: largest, sum, its index (bits), the sequence whose temperature it was (bits; -1: none holds the row)
    int batch, m, vocab, chunks;
    int bits;        // weights are integers in units of 2^-bits: the row's add up to 2^62 at most
    int* err_flag;
};

// NaN as -inf (such a token has no probability), +inf as the largest finite number.
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, -INFINITY), kLargest); }
// +inf as the largest finite number, NaN as it is.
__device__ __forceinline__ float below_inf(float x) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(kLargest));
    return y;
}
// Shifts of which amounts from the type's width on, negative ones among them, leave nothing.
__device__ __forceinline__ uint32_t shr(uint32_t x, int by) {
    uint32_t y;
    asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(by));
    return y;
}
__device__ __forceinline__ uint64_t shr(uint64_t x, int by) {
    uint64_t y;
    asm("shr.u64 %0, %1, %2;" : "=l"(y) : "l"(x), "r"(by));
    return y;
}
__device__ __forceinline__ uint32_t shl(uint32_t x, int by) {
    uint32_t y;
    asm("shl.b32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(by));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(c d) for a difference d of logits; -inf (no probability, or further apart than numbers go) gives 0 at c = 0, too.
__device__ __forceinline__ float power(float d, float c) { return d > -INFINITY ? ex2(d * c) : 0.0f; }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two fp32 operations in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
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
__global__ void __launch_bounds__(kStatThreads, 6) verify_stats_kernel(const __grid_constant__ VerifyParams A) {
    constexpr int V = 16 / (int)sizeof(T), W = kStatThreads / 32;
    constexpr int kUnits = 2;  // 16-byte units a thread and batch (4, with 4 CTAs an SM: 64 sequences of 131072 in bf16 58.4 us, with 2 and 6 56.8)
    __shared__ float s_m[W], s_s[W], s_t;
    __shared__ int s_i[W], s_seq;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / A.chunks, chunk = blockIdx.x - row * A.chunks;
    const T* x = static_cast<const T*>(A.logits) + (int64_t)row * A.logits_stride;
    // 16-byte units from the aligned address at or below the row. Whole ones lie inside it; the two ends are read by element.
    const int shift = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int units = (A.vocab + shift + V - 1) / V;
    const int u0 = (int)((int64_t)units * chunk / A.chunks), u1 = (int)((int64_t)units * (chunk + 1) / A.chunks);
    const int w0 = max(u0, shift ? 1 : 0), w1 = min(u1, (A.vocab + shift) / V);   // the chunk's whole units
    const uint4* const xu = reinterpret_cast<const uint4*>(x - shift);
    constexpr int kStep = kUnits * kStatThreads;
    uint4 raw[2][kUnits];  // two batches, one under way while another is worked on
    auto fetch = [&](int u, uint4 (&to)[kUnits]) {
        if (u + kStep <= w1) {
#pragma unroll
            for (int j = 0; j < kUnits; ++j) to[j] = __ldcg(xu + u + j * kStatThreads + tid);
        }
    };
    fetch(w0, raw[0]);
    if (warp == 0) {
        const int seq = sequence_of(A, row);
        if (lane == 0) {
            s_seq = seq;
            s_t = seq >= 0 && A.temperature ? __ldcg(A.temperature + seq) : 1.0f;
        }
    }
    __syncthreads();
    if (s_seq < 0) {
        if (tid == 0) A.stats[blockIdx.x] = make_float4(-INFINITY, 0.0f, __int_as_float(0x7FFFFFFF), __int_as_float(-1));
        return;
    }
    const bool greedy = !(s_t > kGreedy);
    const float c = 1.44269504088896340736f / s_t;
    float m = -INFINITY, s = 0.0f;
    int best = 0x7FFFFFFF;
    // One unit: its elements begin at token e.
    auto choose = [&](int e, const float (&v)[V]) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float y = tame(v[k]);
            if (y > m || (y == m && e + k < best && y > -INFINITY)) {
                m = y;
                best = e + k;
            }
        }
    };
    auto rise = [&](float top) {  // the sum's reference
        s = m > -INFINITY ? s * ex2((m - top) * c) : 0.0f;
        m = top;
    };
    auto add = [&](const float (&v)[V]) {
        float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            float2 y = add2(make_float2(v[k], v[k + 1]), make_float2(-m, -m));
            y = mul2(y, make_float2(c, c));
            part = add2(part, make_float2(ex2(y.x), ex2(y.y)));
        }
        s += part.x + part.y;
    };
    auto take = [&](int u, const uint4 (&from)[kUnits]) {
        if (greedy) {
#pragma unroll
            for (int j = 0; j < kUnits; ++j) {
                float v[V];
                unpack<T, V>(from[j], v);
                choose((u + j * kStatThreads + tid) * V - shift, v);
            }
            return;
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            float v[V];
            unpack<T, V>(from[j], v);
#pragma unroll
            for (int k = 0; k < V; k += 2) top = max3(top, v[k], v[k + 1]);
        }
        if (top > m) rise(top);
        if (m == -INFINITY) return;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            float v[V];
            unpack<T, V>(from[j], v);
            add(v);
        }
    };
    int u = w0;
    for (; u + 2 * kStep <= w1; u += 2 * kStep) {
        fetch(u + kStep, raw[1]);
        take(u, raw[0]);
        fetch(u + 2 * kStep, raw[0]);
        take(u + kStep, raw[1]);
    }
    if (u + kStep <= w1) {
        take(u, raw[0]);
        u += kStep;
    }
    // what is left of the whole units, then the ends
    auto few = [&](int e, const float (&v)[V]) {
        if (greedy) return choose(e, v);
        float top = m;
#pragma unroll
        for (int k = 0; k < V; ++k) top = fmaxf(top, v[k]);
        if (top > m) rise(top);
        if (m > -INFINITY) add(v);
    };
    auto at_end = [&](int un, float (&v)[V]) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int e = un * V - shift + k;
            v[k] = e >= 0 && e < A.vocab ? one(x + e) : -INFINITY;
        }
    };
    for (int v0 = u + tid; v0 < w1; v0 += kStatThreads) {
        float v[V];
        unpack<T, V>(__ldcg(xu + v0), v);
        few(v0 * V - shift, v);
    }
    const int end = tid ? u1 - 1 : u0;   // threads 0 and 1: an end of the chunk that is no whole unit
    const bool has_end = tid < 2 && end >= u0 && end < u1 && (end < w0 || end >= w1) && (tid == 0 || u1 - 1 != u0);
    if (has_end) {
        float v[V];
        at_end(end, v);
        few(end * V - shift, v);
    }
    if (!greedy && !(s < INFINITY && m < INFINITY)) {  // NaN, +inf or a c of 0 among them: this thread's units once more, with every logit tamed
        m = -INFINITY;
        s = 0.0f;
        auto again = [&](int un, bool sums) {
            float v[V];
            at_end(un, v);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float y = tame(v[k]);
                if (!sums) m = fmaxf(m, y);
                else s += y > -INFINITY ? power(y - m, c) : 0.0f;
            }
        };
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
            for (int un = w0 + tid; un < w1; un += kStatThreads) again(un, pass);
            if (has_end) again(end, pass);
        }
    }
    // The next kernel's large CTAs are let in only now: they would take the place of this one's.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the block's
    float top = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (greedy) {
        if (m != top) best = 0x7FFFFFFF;
        best = __reduce_min_sync(0xffffffffu, best);
    } else {
        s = m > -INFINITY ? s * power(m - top, c) : 0.0f;
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
        if (!greedy) sum += s_s[w] * power(s_m[w] - all, c);
        else if (s_m[w] == all) at = min(at, s_i[w]);
    }
    A.stats[blockIdx.x] = make_float4(all, sum, __int_as_float(at), __int_as_float(s_seq));
}

// ---- weights of more than 24 bits ---------------------------------------------------------------------------------
// The weight 2^y of a logit, y = c (x - top), relative to the row's largest: y in two floats (2^-46 of itself), cut into
// multiples of a table's step and a rest r; 2^r = 1 + a + a^2/2 + .., a = r ln 2.
//   Weigher: 1024 steps, 32 bits of the power in an integer, a^2/2 the last term: off by 2^-31 of itself at most
//            (half a unit of 2^-31 in the table, half in the product, 2^-37 from the next term), 34 instructions. For the draw.
//   precise: 256 steps, two floats, a^3/6: 2^-41. For an acceptance too close to call in fp32.
constexpr double kRoots[10] = {  // 2^(1/2), 2^(1/4), ..
    1.414213562373095048801689, 1.189207115002721066717500, 1.090507732665257659207010, 1.044273782427413840321966,
    1.021897148654116678234480, 1.010889286051700460020410, 1.005429901112802821351384, 1.002711275050202485430746,
    1.001354719892108205880882, 1.000677130693066356678173};
constexpr double power_of_two(int i, int bits) {  // 2^(i / 2^bits)
    double x = 1.0;
    for (int k = 0; k < bits; ++k)
        if (i >> (bits - 1 - k) & 1) x *= kRoots[k];
    return x;
}
constexpr int kTable = 1024;
struct Powers {
    uint32_t fix[kTable];  // 2^(i/1024) 2^31
    float hi[256], lo[256];
};
constexpr Powers make_powers() {
    Powers p{};
    for (int i = 0; i < kTable; ++i) p.fix[i] = (uint32_t)(power_of_two(i, 10) * 2147483648.0 + 0.5);
    for (int i = 0; i < 256; ++i) {
        const double x = power_of_two(i, 8);
        p.hi[i] = (float)x;
        p.lo[i] = (float)(x - (double)p.hi[i]);
    }
    return p;
}
__device__ const Powers kPowers = make_powers();

struct Weigher {
    const uint2* table;   // in shared memory: the integer, and the same as a float
    float top, c_hi, c_lo;
    int down;             // 63 - bits: the sums' unit is 2^-bits
    __device__ __forceinline__ Weigher(const uint2* t, float largest, float temperature, int bits) : table(t), top(largest), down(63 - bits) {
        // log2(e) / T in two floats (fp64 has no rate worth the name here: one quotient a thread took 8 us a CTA)
        constexpr float l_hi = 1.442695040888963407f, l_lo = (float)(1.4426950408889634074 - (double)l_hi);
        c_hi = l_hi / temperature;
        c_lo = temperature < INFINITY ? (fmaf(-c_hi, temperature, l_hi) + l_lo) / temperature : 0.0f;   // +inf: c is 0
    }
    __device__ __forceinline__ void exponent(float x, float* y, float* yl) const {
        const float d = x - top, b = d - x, dl = (x - (d - b)) + (-top - b);  // x - top in two floats
        *y = d * c_hi;
        *yl = fmaf(d, c_lo, fmaf(dl, c_hi, fmaf(d, c_hi, -*y)));
    }
    // Mantissa in [2^31, 2^32) and exponent: weight = mant 2^(e - 31), off by 2^-31 of itself. No probability, or below 2^-200: e < -190.
    __device__ __forceinline__ void parts(float x, uint32_t* mant, int* e) const {
        constexpr float kRound = 12582912.0f;  // 1.5 2^23: adding it rounds to an integer, which the low bits hold
        constexpr int kRoundBits = 0x4B400000;
        float y, yl;
        exponent(x, &y, &yl);
        y = fmaxf(y, -200.0f);   // -inf and NaN (no probability), too: far below the unit
        const float kf = fmaf(y, (float)kTable, kRound);
        const int n = __float_as_int(kf) - kRoundBits;
        const float r = fmaf(kf - kRound, -1.0f / kTable, y) + yl;
        const float p = r * fmaf(r, 0.240226506959100712f, 0.693147180559945309f);  // (ln 2)^2 / 2, ln 2
        const uint2 t = table[n & (kTable - 1)];
        *mant = t.x + (uint32_t)(__float_as_int(fmaf(__uint_as_float(t.y), p, kRound)) - kRoundBits);
        *e = n >> 10;
    }
    // In units of 2^-bits, cut off; 0 for tokens without probability (their exponent is -200).
    __device__ __forceinline__ uint64_t operator()(float x) const {
        uint32_t w;
        int e;
        parts(x, &w, &e);
        const int shift = down - e;   // w 2^-31 2^e in that unit: w 2^32 to the right, by 64 and more to nothing
        return (uint64_t)shr(w, shift) << 32 | (shl(w, 32 - shift) | shr(w, shift - 32));
    }
    // mantissa in [2^43, 2^44) and exponent: weight = mant 2^(e - 43). False: below 2^-1000, or no probability.
    __device__ __noinline__ bool precise(float x, uint64_t* mant, int* e) const {
        float y, yl;
        exponent(x, &y, &yl);
        if (!(y > -1000.0f)) return false;
        const float k = rintf(y * 256.0f);
        const int n = (int)k;
        const float r = fmaf(k, -1.0f / 256.0f, y);   // exact
        const float a = r * 0.693147180559945309417f;  // ln 2 = this float and the one below
        const float al = fmaf(r, 0.693147180559945309417f, -a) + fmaf(r, -1.904654299957768e-9f, yl * 0.693147180559945309417f);
        const float z = a + al, s = fmaf(z * z, fmaf(z, 1.0f / 6.0f, 0.5f), al);   // al has the exponent's second float, too: up to 2^-19
        const float hi = kPowers.hi[n & 255], lo = kPowers.lo[n & 255];
        const float b1 = hi * a;
        const float b2 = fmaf(hi, s, fmaf(lo, a, lo + fmaf(hi, a, -b1)));
        // hi + b1 + b2 in units of 2^-43: |b1| below 2^-8, |b2| below 2^-18
        *mant = ((uint64_t)((__float_as_uint(hi) & 0x7FFFFFu) | 0x800000u) << 20) + __float2ll_rn(b1 * 8796093022208.0f) +
                __float2int_rn(b2 * 8796093022208.0f);
        *e = n >> 8;
        return true;
    }
    // Adds it to sums of whole units of 2^-bits and of 2^-kFineBits of them, cut off there.
    __device__ __forceinline__ void add_precise(float x, uint64_t* units, uint64_t* parts) const {
        uint64_t mant;
        int e;
        if (!precise(x, &mant, &e)) return;
        const int by = down - 20 - e;   // mant 2^(e - 43) is mant 2^-by units; by is -19 at least
        if (by <= 0) {
            *units += mant << -by;
        } else {
            *units += shr(mant, by);
            *parts += (by < 64 ? mant << (64 - by) : shr(mant, by - 64)) >> (64 - kFineBits);
        }
    }
};
// f * s for a sum s < 2^63, of which it keeps 32 bits (2^-31 of itself), and f in [0, 1], cut off.
struct Portion {
    uint32_t top;
    int down;
    __device__ __forceinline__ explicit Portion(uint64_t s) {
        const int lead = __clzll((int64_t)(s | 1));
        top = (uint32_t)((s << lead) >> 32);
        down = 126 + lead;
    }
    __device__ __forceinline__ uint64_t operator()(float f) const {
        const uint32_t b = __float_as_uint(f);   // f = (b << 8 | 2^31) 2^(b >> 23 - 158); zero and denormal numbers give less than 1
        return shr((uint64_t)(b << 8 | 0x80000000u) * top, down - (int)(b >> 23));
    }
};
// A probability as it counts: above 1 as 1, below 0 and NaN as 0.
__device__ __forceinline__ float fraction(float f) { return fminf(fmaxf(f, 0.0f), 1.0f); }
// floor(f * s), exactly.
__device__ __forceinline__ uint64_t portion(float f, uint64_t s) {
    const uint32_t b = __float_as_uint(fraction(f));
    const uint32_t m8 = b << 8 | 0x80000000u;   // f = m8 2^(e - 158), but for zero and denormal numbers, whose product is below 1
    const uint64_t hi = (uint64_t)m8 * (uint32_t)(s >> 32) + (((uint64_t)m8 * (uint32_t)s) >> 32);  // m8 s / 2^32
    const int down = 126 - (int)(b >> 23);
    return down > 63 ? 0 : down >= 0 ? hi >> down : s;   // down is -1 for f = 1 alone
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

// A cluster of one to eight CTAs a sequence; a CTA's part of the vocabulary is cut into segments of kSeg tokens.
// VEC: the rows of logits and probabilities are 16-byte aligned, so a lane takes 16 bytes of logits at a time, else one element.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kPickThreads, 4) verify_pick_kernel(const __grid_constant__ VerifyParams A) {
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, kSteps = kSeg / (32 * V), kAhead = kSteps < 4 ? kSteps : 4;
    extern __shared__ __align__(16) uint64_t s_sum[];   // [segments of the CTA]: what is left of their weights, then ..
    __shared__ uint2 s_pow[kTable];
    __shared__ uint64_t s_part[2][3], s_warp[kPickWarps];
    __shared__ int s_stop, s_close;
    __shared__ float s_top[kPickWarps], s_row_sum[kPickWarps];  // of the row at which a warp stopped
    __shared__ int s_best[kPickWarps];
    uint32_t rank, ranks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, seq = blockIdx.x / ranks;
    const int segs = (A.vocab + kSeg - 1) / kSeg, per = (segs + ranks - 1) / ranks;
    const int seg0 = min((int)rank * per, segs), seg1 = min(seg0 + per, segs);
    float* s_share = reinterpret_cast<float*>(s_sum + per);  // .. the drafts' probability among those that are left something
    for (int i = tid; i < kTable; i += kPickThreads) s_pow[i] = make_uint2(kPowers.fix[i], __float_as_uint((float)kPowers.fix[i]));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int a = __ldcg(A.q_start + seq), b = __ldcg(A.q_start + seq + 1);
    const int start = min(max(a, 0), A.m), n = min(max(b, start), A.m) - start;
    const float temperature = A.temperature ? __ldcg(A.temperature + seq) : 1.0f;
    const float u_sample = __ldcg(A.u_sample + seq);
    const int len = A.seq_lens ? __ldcg(A.seq_lens + seq) : 0;
    const bool writes = rank == 0 && tid == 0;
    if (writes && (start != a || start + n != b)) raise_flag(A.err_flag, Q4K_ERR_SEQ);
    if (n == 0) {
        if (writes) {
            A.accepted[seq] = 0;
            A.next[seq] = -1;
            if (A.kept) A.kept[seq] = len;
        }
        return;
    }
    const bool greedy = !(temperature > kGreedy);
    const float c = 1.44269504088896340736f / temperature;

    // A row's largest logit, its sum in fp32 and the largest's index, over its chunks; the whole warp calls it.
    struct Row { float top, sum; int best; };
    auto row_of = [&](int r) {
        Row R{-INFINITY, 0.0f, 0x7FFFFFFF};
        for (int k = lane; k < A.chunks; k += 32) {
            float4 f = __ldcg(A.stats + (int64_t)r * A.chunks + k);
            if (__float_as_int(f.w) != seq) f.x = -INFINITY;   // (where starts fall, a row that two sequences have is one's)
            if (f.x > R.top) {
                R.sum *= power(R.top - f.x, c);
                R.top = f.x;
                R.best = __float_as_int(f.z);
                R.sum += f.y;
            } else if (f.x > -INFINITY) {
                R.sum += f.y * power(f.x - R.top, c);   // an equal one of a later chunk has the higher index
            }
        }
        float top = R.top;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        R.sum = R.top > -INFINITY ? R.sum * power(R.top - top, c) : 0.0f;
        if (R.top != top || top == -INFINITY) R.best = 0x7FFFFFFF;
        R.top = top;
#pragma unroll
        for (int o = 16; o; o >>= 1) R.sum += __shfl_xor_sync(0xffffffffu, R.sum, o);
        R.best = __reduce_min_sync(0xffffffffu, R.best);
        return R;
    };
    auto logit = [&](int r, int d) { return tame(one(static_cast<const T*>(A.logits) + (int64_t)r * A.logits_stride + d)); };
    auto chance = [&](int r) { return fmaxf(__ldcg(A.u_accept + r), 0.0f); };
    auto drafts = [&](int r, int d) { return A.probs ? fmaxf(__ldcg(A.probs + (int64_t)r * A.probs_stride + d), 0.0f) : 1.0f; };
    enum { kYes, kNo, kAsk };
    auto decide = [&](int r) {
        if (r == start + n - 1) {  // no draft behind it
            const Row R = row_of(r);
            if (lane == 0) {
                s_top[warp] = R.top;
                s_row_sum[warp] = R.sum;
                s_best[warp] = R.best;
            }
            return (int)kNo;
        }
        const int d = __ldcg(A.tokens + r + 1);
        const bool there = (unsigned)d < (unsigned)A.vocab;
        const float x = there ? logit(r, d) : -INFINITY, u = chance(r), q = there ? drafts(r, d) : 0.0f;
        const Row R = row_of(r);
        if (lane == 0) {
            s_top[warp] = R.top;
            s_row_sum[warp] = R.sum;
            s_best[warp] = R.best;
        }
        if (!there && rank == 0 && lane == 0) raise_flag(A.err_flag, Q4K_ERR_TOKEN);
        if (x == -INFINITY || R.top == -INFINITY) return (int)kNo;
        if (u == 0.0f || q == 0.0f) return (int)(!greedy || d == R.best ? kYes : kNo);
        const float need = u * q;
        if (greedy) return (int)(d == R.best && need < 1.0f ? kYes : kNo);
        const float y = (x - R.top) * c, w = ex2(y), l = need * R.sum, band = closeness(y);
        if (w < 1e-30f || need < 1e-30f) return (int)kAsk;
        return (int)(l * (1.0f + band) < w ? kYes : l * (1.0f - band) >= w ? kNo : kAsk);
    };

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
    // A value of every warp: the CTA's sum, in every thread.
    auto block_sum = [&](uint64_t v) {
        v = warp_sum(v);
        __syncthreads();
        if (lane == 0) s_warp[warp] = v;
        __syncthreads();
        return warp_sum(lane < kPickWarps ? s_warp[lane] : 0);
    };
    // Values of every CTA, lane k's those of CTA k.
    int turn = 0;
    bool gathered = false;
    struct Values { uint64_t a, b, c; };
    auto gather = [&](uint64_t a, uint64_t b, uint64_t c) {
        gathered = true;
        if (tid == 0) {
            s_part[turn][0] = a;
            s_part[turn][1] = b;
            s_part[turn][2] = c;
        }
        sync_cluster();
        Values v{};
        if (lane < (int)ranks) v = Values{peer_u64(&s_part[turn][0], lane), peer_u64(&s_part[turn][1], lane), peer_u64(&s_part[turn][2], lane)};
        turn ^= 1;   // written again only after the next gather's barrier
        return v;
    };

    // How many drafts are accepted. A decision too close to call in fp32 counts as a rejection until the draw's first pass has
    // given the row's sum; should the draft pass after all, the search goes on behind it.
    int at = 0;
    bool rejected, asked;
    Row R;
    auto search = [&]() {
        if (tid == 0) s_stop = s_close = 0x7FFFFFFF;
        __syncthreads();
        for (int j = at + warp; j < n; j += kPickWarps) {
            const int said = decide(start + j);
            if (said == kYes) continue;
            if (lane == 0) {
                atomicMin(&s_stop, j);
                if (said == kAsk) atomicMin(&s_close, j);
            }
            break;
        }
        __syncthreads();
        const int by = (s_stop - at) % kPickWarps;
        R = Row{s_top[by], s_row_sum[by], s_best[by]};
        at = s_stop;
        rejected = at < n - 1;
        asked = rejected && s_close == at;
        __syncthreads();
    };
    // The row behind them: a pass over it, which gives every segment's sum and the row's.
    int r;
    const T* x;
    const float* q;
    int drafted;
    uint64_t whole, about, left_of, share_of;   // left_of, share_of: of CTA `lane`
    for (;;) {
        search();
        r = start + at;
        if (R.top == -INFINITY || greedy) {
            if (writes) {
                A.accepted[seq] = at;
                if (A.kept) A.kept[seq] = len - n + 1 + at;
                A.next[seq] = R.top == -INFINITY ? -1 : R.best;
                if (R.top == -INFINITY) raise_flag(A.err_flag, Q4K_ERR_TOKEN);
            }
            if (gathered) sync_cluster();   // no CTA leaves while another reads its sums
            return;
        }
        const Weigher W(s_pow, R.top, temperature, A.bits);
        x = static_cast<const T*>(A.logits) + (int64_t)r * A.logits_stride;
        q = rejected && A.probs ? A.probs + (int64_t)r * A.probs_stride : nullptr;
        drafted = rejected && !A.probs ? __ldcg(A.tokens + r + 1) : -1;  // only it has nothing left
        // One pass with the sum S that fp32 gave: what is left is max(w - q S, 0), and where S is off by s, the sum of that over a
        // segment is off by s times the q of the tokens that are left something (which those are, S decides well enough: a token that
        // changes sides has at most s q left). So each segment keeps both sums, and the precise S comes in afterwards.
        about = __float2ull_rn(R.sum * __int_as_float((127 + A.bits) << 23));
        const Portion away_of(about);
        uint64_t cta_whole = 0, cta_left = 0, cta_share = 0;   // shares in units of 2^-40
        for (int sg = seg0 + warp; sg < seg1; sg += kPickWarps) {
            uint64_t all = 0, left = 0;
            float share = 0.0f;
#pragma unroll
            for (int i0 = 0; i0 < kSteps; i0 += kAhead) {
                float v[kAhead][V], p[kAhead][V];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int e = sg * kSeg + (i0 + i) * 32 * V + lane * V;
                    logits_at(x, e, v[i]);
                    if (q) probs_at(q, e, p[i]);
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const uint64_t w = W(below_inf(v[i][k]));
                        all += w;
                        if (q) {
                            const float f = fraction(p[i][k]);
                            const uint64_t away = away_of(f);
                            if (w > away) {
                                left += w - away;
                                share += f;
                            }
                        } else if (sg * kSeg + (i0 + i) * 32 * V + lane * V + k != drafted) {
                            left += w;
                        }
                    }
            }
            all = warp_sum(all);
            left = warp_sum(left);
            if (q) {
#pragma unroll
                for (int o = 16; o; o >>= 1) share += __shfl_xor_sync(0xffffffffu, share, o);
            }
            if (lane == 0) {
                s_sum[sg - seg0] = left;
                s_share[sg - seg0] = share;
                cta_whole += all;
                cta_left += left;
                cta_share += __float2ull_rn(share * 1099511627776.0f);
            }
        }
        const uint64_t a0 = block_sum(cta_whole), b0 = block_sum(cta_left), c0 = block_sum(cta_share);
        const Values sums = gather(a0, b0, c0);
        whole = warp_sum(sums.a);
        left_of = sums.b;
        share_of = sums.c;
        if (!asked) break;
        // u q(d) S against w(d)
        const int d = __ldcg(A.tokens + r + 1);
        uint32_t m32;
        int e;
        W.parts(logit(r, d), &m32, &e);
        const double need = (double)chance(r) * (double)drafts(r, d), l = need * (double)whole, w = scalbn((double)m32, e + A.bits - 31);
        bool passes = l < w;
        if (!(fabs(l - w) > kCloseFine * w + need * (double)A.vocab) || e < -190) {  // closer still (or a draft below 2^-190): all to 2^-41
            uint64_t units = 0, parts = 0, mant;
#pragma unroll 1
            for (int i = seg0 * kSeg + tid; i < min(seg1 * kSeg, A.vocab); i += kPickThreads) W.add_precise(tame(one(x + i)), &units, &parts);
            const uint64_t a1 = block_sum(units), b1 = block_sum(parts);
            const Values all = gather(a1, b1, 0);
            const double fine = (double)warp_sum(all.a) + (double)warp_sum(all.b) * (1.0 / (1 << kFineBits));
            passes = W.precise(logit(r, d), &mant, &e) && need * fine < scalbn((double)mant, e + A.bits - 43);
        }
        if (!passes) break;
        ++at;
        __syncthreads();
    }
    const Weigher W(s_pow, R.top, temperature, A.bits);
    if (writes) {
        A.accepted[seq] = at;
        if (A.kept) A.kept[seq] = len - n + 1 + at;
    }
    // what is left, with the precise S: of the CTAs, and of this one's segments as they are looked at
    const float off = q ? (float)(int64_t)(whole - about) : 0.0f;
    auto corrected = [&](uint64_t left, float share) {
        const int64_t v = (int64_t)left - __float2ll_rn(off * share);
        return v > 0 ? (uint64_t)v : 0;
    };
    left_of = corrected(left_of, (float)share_of * 9.094947e-13f);
    bool minus = rejected;
    auto left_with = [&](int e, float logit_e, float prob_e) {   // what is left of token e, past the last one's -inf and 0
        const uint64_t w = W(tame(logit_e)), away = portion(prob_e, whole);   // (a portion of 0 is 0)
        return minus && e == drafted ? 0 : w > away ? w - away : 0;
    };
    auto logit_at = [&](int e) { return e < A.vocab ? one(x + e) : -INFINITY; };
    auto prob_at = [&](int e) { return minus && q && e < A.vocab ? __ldcg(q + e) : 0.0f; };
    auto left_at = [&](int e) { return left_with(e, logit_at(e), prob_at(e)); };
    auto recount = [&]() {   // the segments' sums with the precise S
        uint64_t cta_left = 0;
        for (int sg = seg0 + warp; sg < seg1; sg += kPickWarps) {
            uint64_t t = 0;
#pragma unroll 1
            for (int e = sg * kSeg + lane; e < (sg + 1) * kSeg; e += 32) t += left_at(e);
            t = warp_sum(t);
            if (lane == 0) {
                s_sum[sg - seg0] = t;
                s_share[sg - seg0] = 0.0f;
                cta_left += t;
            }
        }
        return gather(block_sum(cta_left), 0, 0).a;
    };
    // Where target and draft nearly agree, the tokens that change sides are many and what is left is as little as they have: counted once
    // more. (A draft is rejected with the probability of what is left, so this is rare where the random numbers are fair: one row of 1024 at
    // most.) Where nothing is left, the token is drawn from the distribution itself.
    uint64_t rest = warp_sum(left_of);
    if (rest < (q ? whole >> 10 : 1)) {
        bool again = q != nullptr;
        for (;;) {
            if (!again) minus = false;
            left_of = recount();
            rest = warp_sum(left_of);
            if (rest != 0 || !again) break;
            again = false;
        }
    }
    const uint64_t cta_before = warp_sum(lane < (int)rank ? left_of : 0);
    const uint64_t cta_rest = __shfl_sync(0xffffffffu, left_of, (int)rank);
    // the first token whose cumulative sum exceeds u * rest: the CTA's segment that holds it, then its place there
    const uint64_t goal = min(portion(u_sample, rest), rest - 1);
    if (goal >= cta_before && goal - cta_before < cta_rest) {
        // every warp finds the segment, then takes a part of it: its tokens' sums, then the place in the part that holds the goal
        uint64_t before = cta_before;
        int sg = -1, last_sg = 0;   // last_sg: the last with something left, should rounding put the goal behind all of them
        for (int base = 0; base < seg1 - seg0 && sg < 0; base += 32) {
            const uint64_t v = base + lane >= seg1 - seg0 ? 0
                               : minus && q              ? corrected(s_sum[base + lane], s_share[base + lane])
                                                         : s_sum[base + lane];
            uint64_t inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, before + inc > goal), some = __ballot_sync(0xffffffffu, v != 0);
            if (some) last_sg = base + 31 - __clz(some);
            if (hit) {
                const int src = __ffs(hit) - 1;
                sg = base + src;
                before += __shfl_sync(0xffffffffu, inc - v, src);
            } else {
                before += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        const bool past = sg < 0;
        sg = seg0 + (past ? last_sg : sg);
        constexpr int kMine = kSeg / kPickThreads;   // tokens of a lane, one after another
        const int e = sg * kSeg + (warp * 32 + lane) * kMine;
        uint64_t w[kMine], own = 0;
        float v[kMine], p[kMine];
        int mine = -1;
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
            v[k] = logit_at(e + k);
            p[k] = prob_at(e + k);
        }
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
            w[k] = left_with(e + k, v[k], p[k]);
            if (w[k]) mine = e + k;
            own += w[k];
        }
        uint64_t inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) s_warp[warp] = inc;
        mine = __reduce_max_sync(0xffffffffu, mine);
        if (lane == 0) s_best[warp] = mine;
        __syncthreads();
        const uint64_t part = lane < kPickWarps ? s_warp[lane] : 0;
        before += warp_sum(lane < warp ? part : 0);
        const unsigned hit = __ballot_sync(0xffffffffu, !past && before + inc > goal);
        const uint64_t end = before + __shfl_sync(0xffffffffu, inc, 31);
        if (hit && before <= goal) {
            if (lane == __ffs(hit) - 1) {
                uint64_t cum = before + inc - own;
                int found = -1;
#pragma unroll
                for (int k = 0; k < kMine; ++k) {
                    cum += w[k];
                    if (found < 0 && cum > goal) found = e + k;
                }
                A.next[seq] = found;
            }
        } else if (warp == kPickWarps - 1 && (past || end <= goal)) {
            int found = -1;
#pragma unroll
            for (int k = 0; k < kPickWarps; ++k) found = max(found, s_best[k]);
            // a segment whose sum was rounding alone: the next token that is left something, or the last one
#pragma unroll 1
            for (int e0 = (sg + 1) * kSeg; found < 0 && e0 < A.vocab; e0 += 32) {
                const unsigned some = __ballot_sync(0xffffffffu, left_at(e0 + lane) != 0);
                if (some) found = e0 + __ffs(some) - 1;
            }
#pragma unroll 1
            for (int e0 = sg * kSeg - 32; found < 0 && e0 >= 0; e0 -= 32) {
                const unsigned some = __ballot_sync(0xffffffffu, left_at(e0 + lane) != 0);
                if (some) found = e0 + 31 - __clz(some);
            }
            if (lane == 0) A.next[seq] = found;
        }
    }
    sync_cluster();
}

// Pieces of a row: five CTAs on each of 152 SMs, one wave, where there are few rows (but 4096 logits a CTA at least), pieces of up to 16384
// where there are many. 150 rows of 50001 logits, whole call: 20.8 us, with eight 25.7, with four 21.9.
constexpr int kWave = 5 * 152;
int most_chunks(int vocab) { return (vocab + 4095) / 4096; }
int least_chunks(int vocab) { return (vocab + 16383) / 16384; }
int chunks_of(int m, int vocab) {
    const int64_t want = (kWave + (int64_t)m - 1) / (m < 1 ? 1 : m), most = most_chunks(vocab), least = least_chunks(vocab);
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
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (P.m > 0) {
        const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_stats_kernel<T>, P);
        if (e != cudaSuccess) return e;
    }
    // Up to eight CTAs a sequence, four an SM at once, and not many more than twice that in all: a CTA's chain of reads and barriers is
    // some microseconds long, whatever its part of the vocabulary.
    int ranks = kMostCluster;
    while (ranks > 1 && (int64_t)P.batch * ranks > 8 * 152) ranks /= 2;
    attr[1].val.clusterDim.x = ranks;
    const int segs = (P.vocab + kSeg - 1) / kSeg, per = (segs + ranks - 1) / ranks;
    cfg.gridDim = dim3((unsigned)P.batch * ranks);
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = (size_t)per * (sizeof(uint64_t) + sizeof(float));  // 24 KB at most
    cfg.numAttrs = 2;
    const auto even = [](const void* p, int64_t stride, int size) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * size % 16 == 0;
    };
    const bool vec = even(P.logits, P.logits_stride, (int)sizeof(T)) && even(P.probs, P.probs ? P.probs_stride : 0, 4);
    return vec ? cudaLaunchKernelEx(&cfg, verify_pick_kernel<T, true>, P) : cudaLaunchKernelEx(&cfg, verify_pick_kernel<T, false>, P);
}

}  // namespace

// m * chunks_of(m, vocab) at most, and of no fewer rows more: m ceil(kWave / m) is below kWave + m.
size_t verify_workspace_bytes(int m, int vocab) {
    const int64_t most = (int64_t)m * most_chunks(vocab), least = (int64_t)m * least_chunks(vocab), wave = kWave + (int64_t)m;
    const int64_t some = least > wave ? least : wave;
    return sizeof(float4) * (size_t)(most < some ? most : some);
}

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
    P.bits = 62;
    while ((int64_t)1 << (62 - P.bits) < vocab) --P.bits;
    return dtype == Q4K_F32 ? launch_typed<float>(P, stream) : launch_typed<__nv_bfloat16>(P, stream);
}

}  // namespace q4k
