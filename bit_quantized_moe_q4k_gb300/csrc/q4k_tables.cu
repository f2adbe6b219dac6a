// q4k_tables.cu -- a step's page tables, starts, positions and slots, made on the device from the sequences' lengths.
//
//   need_i = max(ceil((kept_i + new_i) / page) - fixed_i, 0)   pages of its own that sequence i has to hold
//   take_i = max(need_i - held_i, 0),  give_i = max(held_i - need_i, 0)
// The free pages are a stack; what is given back goes on top of it in the order of sequences and table entries, and the
// k-th page taken (same order) is the k-th from the top. So every place follows from exclusive sums over the sequences:
// no atomics, the same tables at every call.
//
// Bound by latency: one CTA, or one cluster of eight where there is more to write (and a second kernel for the rows of
// long prompts). Every CTA forms the sums over all sequences itself in shared memory (a few KB of lengths), and writes
// its share of the entries and rows, finding the sequence of each by bisection of the sums. The cluster's barrier between
// the last read of the lengths and the first write lets results take the place of inputs.
// A step of 7 sequences takes 3.2 us, one of 1000 with up to 6 new tokens and 6300 pages given back 7.6, prompts of 121000
// tokens in all 8.0. The code is small on purpose: a version with all of a thread's entries and rows looked up in one
// unrolled pass waited for instructions (9.2 us for the 1000).
#include <atomic>

#include "q4k_paged.cuh"

namespace q4k {
namespace {

constexpr int kFewThreads = 256, kManyThreads = 1024, kTablesCluster = 8;
constexpr int kSumThreads = 256;  // that add the sequences up
constexpr int kRun = 4;           // rows of a thread at a time, where there are more rows than threads
// More rows than this are written by a kernel of their own, on all SMs. 40 sequences, in the cluster and apart: 8000 rows 5.3 and 6.2 us, 16000 6.7
// and 6.2, 121000 13.1 and 8.0; 1000 sequences, 15000 rows 8.4 and 8.1.
constexpr int kRowsTogether = 16384;
constexpr int kRowsThreads = 512;
constexpr int kArrays = 6;        // of batch + 1 words in shared memory

struct TablesParams {
    const int32_t *kept, *fresh, *fixed, *held, *count;
    int32_t *free_pages, *table, *held_out, *count_out, *q_start, *seq_lens, *pos;
    int64_t* slots;
    int batch, m, max_pages, page_shift, num_pages;
    bool rows_apart;  // positions and slots are rows_kernel's
    int* err_flag;
};

// Exclusive sums of three values a thread over the first kSumThreads threads, and their totals for all. (Shuffles bound it: by all 32 warps of a
// CTA, a sequence a lane, it took 2.1 us.)
__device__ __forceinline__ void block_sums(int64_t (&v)[3], int64_t (&total)[3], int64_t (*s_warp)[kSumThreads / 32 + 1]) {
    constexpr int kWarps = kSumThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < kWarps) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            int64_t inc = v[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            if (lane == 31) s_warp[k][warp] = inc;
            v[k] = inc - v[k];
        }
    }
    __syncthreads();
    if (warp < 3) {  // the warps' sums, of one value a warp
        int64_t x = lane < kWarps ? s_warp[warp][lane] : 0, inc = x;
#pragma unroll
        for (int o = 1; o <= kWarps; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane <= kWarps) s_warp[warp][lane] = inc - x;  // the total last
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (warp < kWarps) v[k] += s_warp[k][warp];
        total[k] = s_warp[k][kWarps];
    }
    __syncthreads();  // s_warp may be written again
}

// The last i with a[i] <= x, of a[0] = 0 <= a[1] <= .. a[n] and 0 <= x < a[n].
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
    int lo = 0, hi = n;  // a[lo] <= x < a[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Positions and slots of the rows, R consecutive ones a thread at a time (R 4: 16-byte stores, to outputs that begin at such a boundary). Returns
// the flag to raise, or 0.
template <int R>
__device__ __forceinline__ int write_rows(const TablesParams& A, const int* s_kept, const int* s_start, int rows, int most, int at, int step) {
    int bad = 0;
#pragma unroll 1
    for (int r0 = at * R; r0 < most; r0 += step * R) {
        int pos[R], id[R];
        int i = r0 < rows ? last_at_most(s_start, A.batch, r0) : 0, last = -1;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const int r = r0 + u;
            pos[u] = 0;
            id[u] = -1;
            if (r >= rows) continue;
            while (r >= s_start[i + 1]) {  // (sequences without rows are passed over)
                ++i;
                last = -1;
            }
            const int e = (pos[u] = s_kept[i] + (r - s_start[i])) >> A.page_shift;
            if (A.slots) {
                if (u > 0 && e == last) id[u] = -2;  // the page of the row before
                else id[u] = __ldcg(A.table + (int64_t)i * A.max_pages + e);
                last = e;
            }
        }
        int64_t slot[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (u > 0 && id[u] == -2) id[u] = id[u - 1];
            const bool known = (unsigned)id[u] < (unsigned)A.num_pages;
            if (r0 + u < rows && A.slots && !known) bad = Q4K_ERR_PAGE;
            slot[u] = known ? ((int64_t)id[u] << A.page_shift) + (pos[u] & ((1 << A.page_shift) - 1)) : -1;
        }
        if (R == 4 && r0 + R <= most) {
            if (A.pos) *reinterpret_cast<int4*>(A.pos + r0) = make_int4(pos[0], pos[1 % R], pos[2 % R], pos[3 % R]);
            if (A.slots) {
                reinterpret_cast<longlong2*>(A.slots + r0)[0] = make_longlong2(slot[0], slot[1 % R]);
                reinterpret_cast<longlong2*>(A.slots + r0)[1] = make_longlong2(slot[2 % R], slot[3 % R]);
            }
        } else {
#pragma unroll
            for (int u = 0; u < R; ++u) {
                if (r0 + u >= most) continue;
                if (A.pos) A.pos[r0 + u] = pos[u];
                if (A.slots) A.slots[r0 + u] = slot[u];
            }
        }
    }
    return bad;
}

template <int T>
__global__ void __launch_bounds__(T) tables_kernel(const __grid_constant__ TablesParams A) {
    extern __shared__ int s_mem[];
    __shared__ int64_t s_warp[3][kSumThreads / 32 + 1];
    const int n = A.batch, width = n + 1;
    int* s_kept = s_mem;             // tokens that stay
    int* s_start = s_mem + width;    // new tokens, then their exclusive sum
    int* s_base = s_mem + 2 * width; // table entries held: those of others and its own
    int* s_need = s_mem + 3 * width; // table entries needed
    int* s_take = s_mem + 4 * width; // exclusive sums of pages taken and given back
    int* s_give = s_mem + 5 * width;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int cap = A.max_pages << A.page_shift, tid = threadIdx.x;
    const int count_in = __ldcg(A.count), count = min(max(count_in, 0), A.num_pages);
    int bad = count != count_in ? Q4K_ERR_PAGE : 0;
    auto entries = [&](int i, int tokens, int fixed) {  // needed for that many tokens
        return max((int)(((int64_t)tokens + (1 << A.page_shift) - 1) >> A.page_shift), fixed);
    };
    for (int i = tid; i < n; i += T) {
        const int k_in = __ldcg(A.kept + i), w_in = __ldcg(A.fresh + i), h_in = __ldcg(A.held + i);
        const int f_in = A.fixed ? __ldcg(A.fixed + i) : 0;
        const int k = min(max(k_in, 0), cap), f = min(max(f_in, 0), A.max_pages), h = min(max(h_in, 0), A.max_pages - f);
        const int w = w_in < 0 || w_in > cap - k ? 0 : w_in;  // more than its row of the table holds: none
        if (k != k_in || f != f_in || h != h_in || w != w_in) bad = Q4K_ERR_SEQ;
        s_kept[i] = k;
        s_start[i] = w;
        s_base[i] = f + h;
        s_need[i] = entries(i, k + w, f);
        s_take[i] = f;  // until the sums
    }
    __syncthreads();
    // each thread's run of sequences, an odd number of them for the banks
    const int per = (n + kSumThreads - 1) / kSumThreads | 1, lo = tid < kSumThreads ? min(tid * per, n) : n, hi = min(lo + per, n);
    int64_t sum[3], total[3];
    auto sums = [&]() {
        sum[0] = sum[1] = sum[2] = 0;
        for (int i = lo; i < hi; ++i) {
            sum[0] += s_start[i];
            sum[1] += max(s_need[i] - s_base[i], 0);
            sum[2] += max(s_base[i] - s_need[i], 0);
        }
        block_sums(sum, total, s_warp);
    };
    sums();
    if (total[0] > A.m) {  // more rows than the outputs have: sequences in order, while they fit
        int64_t before = sum[0];
        for (int i = lo; i < hi; ++i) {
            const int w = s_start[i];
            before += w;
            if (before <= A.m || w == 0) continue;
            bad = Q4K_ERR_SEQ;
            s_start[i] = 0;
            s_need[i] = entries(i, s_kept[i], s_take[i]);
        }
        __syncthreads();
        sums();
    }
    int64_t available = count + total[2];
    if (available > A.num_pages) {  // some page is held twice
        available = A.num_pages;
        bad = Q4K_ERR_PAGE;
    }
    if (total[1] > available) {  // more pages than there are: sequences in order, up to the first that lacks one
        int64_t before = sum[1];
        for (int i = lo; i < hi; ++i) {
            const int t = max(s_need[i] - s_base[i], 0);
            before += t;
            if (before <= available || t == 0) continue;
            bad = Q4K_ERR_PAGE;
            s_start[i] = 0;
            s_need[i] = s_base[i];
        }
        __syncthreads();
        sums();
    }
    for (int i = lo; i < hi; ++i) {
        const int w = s_start[i], t = max(s_need[i] - s_base[i], 0), g = max(s_base[i] - s_need[i], 0);
        s_start[i] = (int)sum[0];
        s_take[i] = (int)sum[1];
        s_give[i] = (int)min(sum[2], (int64_t)0x7FFFFFFF);
        sum[0] += w;
        sum[1] += t;
        sum[2] += g;
    }
    if (tid == 0) {
        s_start[n] = (int)total[0];
        s_take[n] = (int)total[1];
        s_give[n] = (int)min(total[2], (int64_t)0x7FFFFFFF);
    }
    // every CTA has read the lengths: they may be written over
    int rank, ranks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    if (ranks > 1) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    else __syncthreads();

    const int taken = s_take[n], rows = s_start[n], top = (int)available, left = top - taken;
    const int at = rank * T + tid, step = ranks * T;
    for (int i = at; i <= n; i += step) {
        A.q_start[i] = s_start[i];
        if (i == n) continue;
        const int f = A.fixed ? min(max(__ldcg(A.fixed + i), 0), A.max_pages) : 0;
        A.seq_lens[i] = s_kept[i] + s_start[i + 1] - s_start[i];
        A.held_out[i] = s_need[i] - f;
    }
    if (at == 0) *A.count_out = left;
    // Pages: the k-th taken is the one at place top - 1 - k of the stack, and what stays on it above `count` is the pages given back that nobody took.
    // Entries taken are written where no entry is read: given-back ones lie in other sequences' rows, free pages below `count`.
#pragma unroll 1
    for (int64_t y = at; y < max(taken, left - count); y += step) {
        const int x = (int)y;
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            if (x >= (side ? left - count : taken)) continue;
            const int p = side ? count + x : top - 1 - x;
            const int32_t* from = A.free_pages + p;
            if (p >= count) {
                const int i = last_at_most(s_give, n, p - count);
                from = A.table + (int64_t)i * A.max_pages + s_need[i] + (p - count - s_give[i]);
            }
            const int id = __ldcg(from);
            if (side) {
                A.free_pages[p] = id;
            } else {
                const int i = last_at_most(s_take, n, x);
                if ((unsigned)id >= (unsigned)A.num_pages) bad = Q4K_ERR_PAGE;
                A.table[(int64_t)i * A.max_pages + s_base[i] + (x - s_take[i])] = id;
            }
        }
    }
    const int most = (A.pos || A.slots) && !A.rows_apart ? A.m : 0;
    if (most > 0) {
        if (A.slots) {  // the tables are complete
            if (ranks > 1) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
            else __syncthreads();
        }
        const bool wide = most > step && ((reinterpret_cast<uintptr_t>(A.pos) | reinterpret_cast<uintptr_t>(A.slots)) & 15) == 0;
        if (wide) bad = max(bad, write_rows<kRun>(A, s_kept, s_start, rows, most, at, step));
        else bad = max(bad, write_rows<1>(A, s_kept, s_start, rows, most, at, step));
    }
    if (bad) raise_flag(A.err_flag, bad);
}

// Positions and slots from the results of the other kernel.
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const __grid_constant__ TablesParams A) {
    extern __shared__ int s_mem[];
    const int n = A.batch;
    int *s_start = s_mem, *s_kept = s_mem + n + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = threadIdx.x; i <= n; i += kRowsThreads) {
        const int a = __ldcg(A.q_start + i);
        s_start[i] = a;
        if (i < n) s_kept[i] = __ldcg(A.seq_lens + i) - (__ldcg(A.q_start + i + 1) - a);
    }
    __syncthreads();
    const bool wide = ((reinterpret_cast<uintptr_t>(A.pos) | reinterpret_cast<uintptr_t>(A.slots)) & 15) == 0;
    const int at = blockIdx.x * kRowsThreads + threadIdx.x, step = gridDim.x * kRowsThreads, rows = s_start[n];
    const int bad = wide ? write_rows<kRun>(A, s_kept, s_start, rows, A.m, at, step) : write_rows<1>(A, s_kept, s_start, rows, A.m, at, step);
    if (bad) raise_flag(A.err_flag, bad);
}

cudaError_t launch_rows(const TablesParams& P, cudaStream_t stream) {
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * (kTablesMaxBatch + 1) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
        allowed[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    const int ctas = (P.m + kRun * kRowsThreads - 1) / (kRun * kRowsThreads);
    cfg.gridDim = dim3(ctas < 2 * num_sms() ? ctas : 2 * num_sms());
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = (size_t)2 * (P.batch + 1) * sizeof(int);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rows_kernel, P);
}

template <int T>
cudaError_t launch_tables(const TablesParams& P, int cluster, cudaStream_t stream) {
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(tables_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kArrays * (kTablesMaxBatch + 1) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
        allowed[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = (size_t)kArrays * (P.batch + 1) * sizeof(int);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, tables_kernel<T>, P);
}

}  // namespace

cudaError_t launch_page_tables(const int32_t* kept, const int32_t* fresh, const int32_t* fixed, int batch, int m,
                               int max_pages, int page_shift, int num_pages, const int32_t* held, int32_t* free_pages,
                               const int32_t* count, int32_t* table, int32_t* held_out, int32_t* count_out,
                               int32_t* q_start, int32_t* seq_lens, int32_t* pos, int64_t* slots, int* err_flag,
                               cudaStream_t stream) {
    TablesParams P{};
    P.kept = kept; P.fresh = fresh; P.fixed = fixed; P.held = held; P.count = count;
    P.free_pages = free_pages; P.table = table; P.held_out = held_out; P.count_out = count_out;
    P.q_start = q_start; P.seq_lens = seq_lens; P.pos = pos; P.slots = slots;
    P.batch = batch; P.m = m; P.max_pages = max_pages; P.page_shift = page_shift; P.num_pages = num_pages;
    P.err_flag = err_flag;
    if (batch <= kFewThreads && m <= 4 * kFewThreads) return launch_tables<kFewThreads>(P, 1, stream);
    P.rows_apart = (pos || slots) && m > kRowsTogether;
    const cudaError_t e = launch_tables<kManyThreads>(P, kTablesCluster, stream);
    return e != cudaSuccess || !P.rows_apart ? e : launch_rows(P, stream);
}

}  // namespace q4k
