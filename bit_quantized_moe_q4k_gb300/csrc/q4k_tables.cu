// q4k_tables.cu -- a step's page tables, starts, positions and slots, made on the device from the sequences' lengths.
//
//   need_i = max(ceil((kept_i + new_i) / page) - fixed_i, 0)   pages of its own that sequence i has to hold
//   take_i = max(need_i - held_i, 0),  give_i = max(held_i - need_i, 0)
// The free pages are a stack; what is given back goes on top of it in the order of sequences and table entries, and the
// k-th page taken (same order) is the k-th from the top. So every place follows from exclusive sums over the sequences:
// no atomics, the same tables at every call.
//
// Bound by latency: one launch of one CTA, or of one cluster of eight where there is more to write. Every CTA forms the
// sums over all sequences itself in shared memory (a few KB of lengths), and writes its share of the entries and rows,
// finding the sequence of each by bisection of the sums. The cluster's barrier between the last read of the lengths and
// the first write lets results take the place of inputs.
#include <atomic>

#include "q4k_paged.cuh"

namespace q4k {
namespace {

constexpr int kFewThreads = 256, kManyThreads = 1024, kTablesCluster = 8;
constexpr int kArrays = 6;  // of batch + 1 words in shared memory

struct TablesParams {
    const int32_t *kept, *fresh, *fixed, *held, *count;
    int32_t *free_pages, *table, *held_out, *count_out, *q_start, *seq_lens, *pos;
    int64_t* slots;
    int batch, m, max_pages, page_shift, num_pages;
    int* err_flag;
};

// Exclusive sums of three values a thread over the block, and their totals.
template <int T>
__device__ __forceinline__ void block_sums(int64_t (&v)[3], int64_t (&total)[3], int64_t (*s_warp)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        inc[k] = v[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc[k], o);
            if (lane >= o) inc[k] += x;
        }
        if (lane == 31) s_warp[k][warp] = inc[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int64_t x = lane < T / 32 ? s_warp[k][lane] : 0;
        int64_t before = lane < warp ? x : 0, all = x;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, o);
            all += __shfl_xor_sync(0xffffffffu, all, o);
        }
        total[k] = all;
        v[k] = before + inc[k] - v[k];
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

template <int T>
__global__ void __launch_bounds__(T) tables_kernel(const __grid_constant__ TablesParams A) {
    extern __shared__ int s_mem[];
    __shared__ int64_t s_warp[3][32];
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
    // each thread's run of sequences
    const int per = (n + T - 1) / T, lo = min(tid * per, n), hi = min(lo + per, n);
    int64_t sum[3], total[3];
    auto sums = [&]() {
        sum[0] = sum[1] = sum[2] = 0;
        for (int i = lo; i < hi; ++i) {
            sum[0] += s_start[i];
            sum[1] += max(s_need[i] - s_base[i], 0);
            sum[2] += max(s_base[i] - s_need[i], 0);
        }
        block_sums<T>(sum, total, s_warp);
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
    auto given = [&](int p) {  // the page at place p >= count of the stack
        const int i = last_at_most(s_give, n, p - count);
        return __ldcg(A.table + (int64_t)i * A.max_pages + s_need[i] + (p - count - s_give[i]));
    };
    auto taken_page = [&](int t) {
        const int p = top - 1 - t;
        return p < count ? __ldcg(A.free_pages + p) : given(p);
    };
    for (int i = at; i <= n; i += step) {
        A.q_start[i] = s_start[i];
        if (i == n) continue;
        const int f = A.fixed ? min(max(__ldcg(A.fixed + i), 0), A.max_pages) : 0;
        A.seq_lens[i] = s_kept[i] + s_start[i + 1] - s_start[i];
        A.held_out[i] = s_need[i] - f;
    }
    if (at == 0) *A.count_out = left;
    // Entries taken are written where no entry is read: given-back ones lie in other sequences' rows, free pages below `count`.
    for (int t = at; t < taken; t += step) {
        const int i = last_at_most(s_take, n, t), id = taken_page(t);
        if ((unsigned)id >= (unsigned)A.num_pages) bad = Q4K_ERR_PAGE;
        A.table[(int64_t)i * A.max_pages + s_base[i] + (t - s_take[i])] = id;
    }
    for (int p = count + at; p < left; p += step) A.free_pages[p] = given(p);
    if (A.pos || A.slots) {
#pragma unroll 4
        for (int r = at; r < A.m; r += step) {
            int pos = 0;
            int64_t slot = -1;
            if (r < rows) {
                const int i = last_at_most(s_start, n, r);
                pos = s_kept[i] + (r - s_start[i]);
                if (A.slots) {
                    const int e = pos >> A.page_shift;
                    const int id = e < s_base[i] ? __ldcg(A.table + (int64_t)i * A.max_pages + e)
                                                 : taken_page(s_take[i] + (e - s_base[i]));
                    if ((unsigned)id < (unsigned)A.num_pages)
                        slot = ((int64_t)id << A.page_shift) + (pos & ((1 << A.page_shift) - 1));
                    else
                        bad = Q4K_ERR_PAGE;
                }
            }
            if (A.pos) A.pos[r] = pos;
            if (A.slots) A.slots[r] = slot;
        }
    }
    if (bad) raise_flag(A.err_flag, bad);
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
    return launch_tables<kManyThreads>(P, kTablesCluster, stream);
}

}  // namespace q4k
