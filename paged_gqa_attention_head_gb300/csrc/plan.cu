// The page plan of a serving step: from the requests' lengths and a list of free pages, on the
// device, the new block-table entries, each packed token's position and slot in the cache, the
// prefix sums of the lengths and the lengths after the step; and finished requests' pages back to
// the list.
//
// The list is a stack: entries [0, num_free) of free_pages, taken from its top.  With need_i the
// pages that request i's new tokens begin and off_i their exclusive prefix sum, its k-th new page is
// free_pages[num_free - 1 - (off_i + k)], so no request waits for another: every block sums the
// lengths for itself (B 4-byte loads, L2 after the first) and then works out its own tokens.  A
// token that begins a page writes the page's table entry.  Releases push in the opposite order, so
// that releasing what the last plan took leaves the list as it was.
//
// Both are bound by latency: the lengths, the list's entry and the stores one after the other.  Measured: 24
// prompts with 43 k new tokens 4.5 us, 256 single tokens 4.6 us, 64 requests' 104 k pages released 3.6 us.
// A captured step carries the lengths and the list's size on from replay to replay, so their new
// values may lie where the old ones are.  Then the blocks are one cluster, and its barrier lies
// between the reads and the writes; otherwise they are a plain grid, which is launched sooner (a cluster's
// launch takes some 6 us more of host time) and may be wider.  In place, inside a graph: the prompts 8.8 us, the long
// release 9.3 (eight blocks, a cluster launch), the single tokens 4.3 (one block).
#include "internal.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCluster = 8;    // blocks of a call that updates in place at most (the portable cluster size)
constexpr int kPlanBlocks = 152;   // blocks of another at most

__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();  // .aligned: a warp's threads come together
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive sums over the block's threads, in thread order, of (x, y); the totals in *tx, *ty.
__device__ __forceinline__ void block_scan(int64_t &x, int64_t &y, int64_t *tx, int64_t *ty) {
    __shared__ int64_t s_x[32], s_y[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
    int64_t ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ax = __shfl_up_sync(0xffffffffu, ix, o), ay = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) {
            ix += ax;
            iy += ay;
        }
    }
    if (lane == 31) {
        s_x[warp] = ix;
        s_y[warp] = iy;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t wx = lane < warps ? s_x[lane] : 0, wy = lane < warps ? s_y[lane] : 0;
        const int64_t ox = wx, oy = wy;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t ax = __shfl_up_sync(0xffffffffu, wx, o), ay = __shfl_up_sync(0xffffffffu, wy, o);
            if (lane >= o) {
                wx += ax;
                wy += ay;
            }
        }
        s_x[lane] = wx - ox;
        s_y[lane] = wy - oy;
        if (lane == 31) {
            *tx = wx;
            *ty = wy;
        }
    }
    __syncthreads();
    x = ix - x + s_x[warp];
    y = iy - y + s_y[warp];
}

// Entries of a list whose size reads n, held to what it can be.
__device__ __forceinline__ int list_size(const PlanArgs &a, int n, uint32_t &bad) {
    if (n >= 0 && n <= a.num_pages) return n;
    bad |= SINKATTN_STATUS_BAD_LENGTH;
    return n < 0 ? 0 : a.num_pages;
}

// Largest i < n with s[i] <= x (s not decreasing, s[0] <= x).
__device__ __forceinline__ int last_at_most(const int *s, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The same from an i that is not past it: mostly that one or the next.
__device__ __forceinline__ int next_at_most(const int *s, int n, int i, int x) {
    if (i + 1 >= n || s[i + 1] > x) return i;
    ++i;
    return i + 1 >= n || s[i + 1] > x ? i : last_at_most(s, n, x);
}

__device__ __forceinline__ int pages_of(int64_t tokens) { return (int)((tokens + kPageSize - 1) / kPageSize); }

__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(const PlanArgs a) {
    extern __shared__ int s_plan[];
    int *s_cu = s_plan;            // [B + 1] first token of each request, at most max_tokens
    int *s_len = s_cu + a.B + 1;   // [B] tokens held before the step
    int *s_off = s_len + a.B;      // [B] place of the first new page in what is taken; -1: not served
    __shared__ int64_t s_total[2];
    __shared__ int s_taken;
    const int tid = threadIdx.x, rank = blockIdx.x;
    const int64_t cap = min((int64_t)a.max_pages * kPageSize, (int64_t)INT32_MAX);
    const int free_now = *a.num_free;  // on its way while the lengths are read
    if (tid == 0) s_taken = 0;

    // Every request's tokens and new pages; a thread sums a run of requests.
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t tokens = 0, pages = 0;
    for (int b = b0; b < b1; ++b) {
        const int raw = a.new_lens[b], L = a.seq_lens[b], n = max(raw, 0);
        s_off[b] = raw;
        s_len[b] = L;
        tokens += n;
        if (L >= 0 && (int64_t)L + n <= cap) pages += pages_of((int64_t)L + n) - pages_of(L);
    }
    block_scan(tokens, pages, &s_total[0], &s_total[1]);
    uint32_t bad = 0;
    const int nfree = list_size(a, free_now, bad);
    int taken = 0;
    for (int b = b0; b < b1; ++b) {
        const int raw = s_off[b], n = max(raw, 0), L = s_len[b];
        const bool fits = L >= 0 && (int64_t)L + n <= cap;
        const int need = fits ? pages_of((int64_t)L + n) - pages_of(L) : 0;
        const bool rows = n == 0 || tokens + n <= a.max_tokens;
        if (raw < 0 || !fits || !rows) bad |= SINKATTN_STATUS_BAD_LENGTH;
        const bool paid = need == 0 || pages + need <= nfree;
        if (fits && rows && !paid) bad |= SINKATTN_STATUS_NO_PAGES;
        const bool served = fits && rows && paid;
        // the served requests that need pages are the first of those that do: what they take has no gaps
        if (served && need > 0) taken = (int)pages + need;
        s_cu[b] = (int)min(tokens, (int64_t)a.max_tokens);
        s_off[b] = served ? (int)min(pages, (int64_t)nfree) : -1;
        tokens += n;
        pages += need;
    }
    if (taken > 0) atomicMax(&s_taken, taken);
    if (tid == 0) s_cu[a.B] = (int)min(s_total[0], (int64_t)a.max_tokens);
    if (rank == 0 && bad) set_status(a.status, bad);
    __syncthreads();
    cluster_barrier();  // in place: every block has read what may be written now

    if (rank == 0) {
        for (int b = tid; b < a.B; b += blockDim.x) {
            const int L = s_len[b];
            a.cu_seqlens[b] = s_cu[b];
            if (a.start_pos) a.start_pos[b] = L;
            a.seq_lens_out[b] = s_off[b] >= 0 ? L + (s_cu[b + 1] - s_cu[b]) : L;  // served: its rows fit
        }
        if (tid == 0) {
            a.cu_seqlens[a.B] = s_cu[a.B];
            *a.num_free_out = nfree - s_taken;
        }
    }

    // Four tokens a thread and step: one look-up, the pages' loads side by side, wide stores.
    const int total = s_cu[a.B];
    for (int64_t t0 = 4 * ((int64_t)rank * blockDim.x + tid); t0 < a.max_tokens;
         t0 += 4 * (int64_t)gridDim.x * blockDim.x) {
        int pos[4], pg[4];
        const int32_t *from[4];
        int32_t *begins[4];  // the table's entry of a page that begins with the token
        int i = t0 < total ? last_at_most(s_cu, a.B, (int)t0) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t t = t0 + e;
            pos[e] = -1;
            from[e] = nullptr;
            begins[e] = nullptr;
            if (t >= total) continue;
            i = next_at_most(s_cu, a.B, i, (int)t);
            const int off = s_off[i], L = s_len[i];
            if (off < 0) continue;
            const int p = L + (int)(t - s_cu[i]);
            const int page = p / kPageSize, first_new = pages_of(L);
            int32_t *entry = a.block_table + (int64_t)i * a.max_pages + page;
            from[e] = page < first_new ? entry : a.free_pages + (nfree - 1 - (off + page - first_new));
            if (page >= first_new && p % kPageSize == 0) begins[e] = entry;
            pos[e] = p;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) pg[e] = from[e] ? *from[e] : 0;
        int64_t slot[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            slot[e] = -1;
            if (!from[e]) continue;
            if (begins[e]) *begins[e] = pg[e];
            if (pg[e] >= 0 && pg[e] < a.num_pages)
                slot[e] = (int64_t)pg[e] * kPageSize + pos[e] % kPageSize;
            else
                set_status(a.status, SINKATTN_STATUS_BAD_PAGE);
        }
        if (t0 + 3 < a.max_tokens) {
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<longlong2 *>(a.slots + t0) = make_longlong2(slot[0], slot[1]);
            *reinterpret_cast<longlong2 *>(a.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (t0 + e < a.max_tokens) {
                    a.positions[t0 + e] = pos[e];
                    a.slots[t0 + e] = slot[e];
                }
        }
    }
}

__global__ void __launch_bounds__(kPlanThreads) release_pages_kernel(const PlanArgs a) {
    extern __shared__ int s_plan[];
    int *s_off = s_plan;          // [B] place of the request's first page in what is released
    int *s_len = s_off + a.B;     // [B] tokens held afterwards
    __shared__ int64_t s_total[2];
    const int tid = threadIdx.x, rank = blockIdx.x;
    const int64_t cap = (int64_t)a.max_pages * kPageSize;
    const int free_now = *a.num_free;
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t pages = 0, none = 0;
    uint32_t bad = 0;
    for (int b = b0; b < b1; ++b) {
        const int L = a.seq_lens[b];
        int n = 0;  // pages of the request to push
        if (a.done[b]) {
            if (L < 0 || L > cap) bad |= SINKATTN_STATUS_BAD_LENGTH;
            else n = pages_of(L);
        }
        s_off[b] = n;
        s_len[b] = a.done[b] ? 0 : L;
        pages += n;
    }
    const int nfree = list_size(a, free_now, bad);
    block_scan(pages, none, &s_total[0], &s_total[1]);
    for (int b = b0; b < b1; ++b) {
        const int n = s_off[b];
        s_off[b] = (int)pages;
        pages += n;
    }
    __syncthreads();
    const int total = (int)s_total[0];
    if (nfree + (int64_t)total > a.num_pages) bad |= SINKATTN_STATUS_BAD_LENGTH;  // more than there are
    if (rank == 0 && bad) set_status(a.status, bad);
    cluster_barrier();  // every block has read what may be written now
    if (rank == 0) {
        for (int b = tid; b < a.B; b += blockDim.x) a.seq_lens_out[b] = s_len[b];
        if (tid == 0) *a.num_free_out = (int)min((int64_t)nfree + total, (int64_t)a.num_pages);
    }
    // the pages' places from the list's new top down, a run of four a thread and step
    for (int64_t o0 = 4 * ((int64_t)rank * blockDim.x + tid); o0 < total; o0 += 4 * (int64_t)gridDim.x * blockDim.x) {
        int i = last_at_most(s_off, a.B, (int)o0);
        const int32_t *from[4];
        int pg[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int o = (int)min(o0 + e, (int64_t)total - 1);
            i = next_at_most(s_off, a.B, i, o);
            from[e] = a.block_table + (int64_t)i * a.max_pages + (o - s_off[i]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) pg[e] = *from[e];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t at = (int64_t)nfree + total - 1 - (o0 + e);
            if (o0 + e >= total) continue;
            if (pg[e] < 0 || pg[e] >= a.num_pages) set_status(a.status, SINKATTN_STATUS_BAD_PAGE);
            if (at < a.num_pages) a.free_pages_w[at] = pg[e];
        }
    }
}

// Shared memory of a plan's and of a release's lengths and offsets.
constexpr int plan_smem(int B) { return (3 * B + 1) * 4; }
constexpr int release_smem(int B) { return 2 * B * 4; }

template <typename Kernel>
cudaError_t launch_plan(Kernel kernel, const PlanArgs &a, bool in_place, int64_t items, int smem, cudaStream_t stream) {
    // Up to 48 KB, static and dynamic together, need no leave.  What is asked for is the most that any call takes, so
    // that no call lowers what another thread is about to launch with.
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, plan_smem(kPlanMaxSeqs));
        if (e != cudaSuccess) return e;
    }
    // Few requests, few threads: they are set up sooner.  Four items a thread.
    const int threads = a.B <= 512 ? 256 : kPlanThreads;
    int64_t blocks = (items + 4 * threads - 1) / (4 * threads);
    blocks = blocks < 1 ? 1 : blocks > kPlanBlocks ? kPlanBlocks : blocks;
    if (!in_place || blocks == 1) {  // one block is a cluster of its own
        kernel<<<(unsigned)blocks, threads, smem, stream>>>(a);
        return cudaGetLastError();
    }
    // values updated in place: the blocks wait for one another before they write
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks > kPlanCluster ? kPlanCluster : blocks));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cfg.gridDim.x;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Whether the outputs lie on the values that every block reads first (the only inputs that they may lie on).
bool in_place(const PlanArgs &a) { return a.num_free == a.num_free_out || a.seq_lens == a.seq_lens_out; }

}  // namespace

cudaError_t launch_plan_step(const PlanArgs &a, cudaStream_t stream) {
    return launch_plan(plan_step_kernel, a, in_place(a), a.max_tokens, plan_smem(a.B), stream);
}

cudaError_t launch_release_pages(const PlanArgs &a, cudaStream_t stream) {
    // how many pages there are to release only the device knows: at most every page
    const int64_t most = (int64_t)a.B * a.max_pages;
    return launch_plan(release_pages_kernel, a, in_place(a), most < a.num_pages ? most : a.num_pages, release_smem(a.B), stream);
}

}  // namespace sinkattn
