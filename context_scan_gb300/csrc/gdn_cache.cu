// gdn_cache.cu -- pages of a state cache: copying, forking, freeing and compacting them
// (gdn_cache_copy, gdn_cache_fork, gdn_cache_free, gdn_cache_compact).
//
// A cache is `layers` arrays of num_pages pages; a page number names one page in every layer.
// Which pages are in use stands in an array of reference counts on the device, so that no call
// reads anything back to the host and each can be captured in a graph. A call is two launches: one
// block turns the caller's page numbers into a list of jobs (page src to page dst, or zeros to page
// dst) and updates the counts; move_kernel, its programmatic dependent, carries the bytes out, which
// are the work: each moved byte read once and written once.
#include <algorithm>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 1024;   // of the blocks that make the job lists
constexpr int kItems = 8;        // pages a thread of them looks at in one round
// detail words of GDN_ERR_INVALID_ARG and GDN_ERR_NO_PAGE
constexpr unsigned kTagPage = 0x51, kTagSharedPage = 0x52, kTagFreePage = 0x53, kTagFull = 0x54;
constexpr int kNobody = -1, kShared = -2;
constexpr int kMostCount = 1 << 30;   // pages of a cache, entries of a list: the kernels' int steps stay below 2^31

struct Job {
    int src, dst;   // src < 0: zeros; dst < 0: nothing to do
};

__device__ __forceinline__ void report(DeviceError* e, unsigned code, unsigned detail) {
    if (atomicCAS(&e->code, 0u, code) == 0u) atomicExch(&e->detail, detail);
}

// Exclusive prefix sum of x over the block and the block's total; every thread calls it.
__device__ __forceinline__ int block_scan(int x, int& sum) {
    __shared__ int part[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int run = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += y;
    }
    __syncthreads();   // the last round's reads of part are over
    if (lane == 31) part[warp] = run;
    __syncthreads();
    int w = part[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += y;
    }
    sum = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    return run - x + (warp ? before : 0);
}

__device__ __forceinline__ bool in_range(int p, int n) { return p >= 0 && p < n; }

// Jobs of a copy: every pair at once, as if all pages were read before any is written. That holds
// when no pair's dst is another pair's dst or src; a pair that breaks it is left out. Pairs with dst < 0 read nothing.
// `owner`: for every page the pair that writes it, of which only the entries that the other pairs name are touched.
__global__ void __launch_bounds__(kThreads)
    copy_jobs_kernel(int num_pages, int n, const int* src, const int* dst, int* owner, Job* jobs,
                     DeviceError* err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = threadIdx.x; i < n; i += kThreads) {
        if (dst[i] < 0) continue;
        if (in_range(src[i], num_pages)) owner[src[i]] = kNobody;
        if (in_range(dst[i], num_pages)) owner[dst[i]] = kNobody;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (in_range(dst[i], num_pages) && atomicCAS(owner + dst[i], kNobody, i) != kNobody)
            atomicExch(owner + dst[i], kShared);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (dst[i] >= 0 && in_range(src[i], num_pages)) {
            const int was = atomicAdd(owner + src[i], 0);
            if (was != kNobody && was != i) atomicExch(owner + src[i], kShared);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        Job j{src[i], dst[i]};
        if (j.src >= num_pages || j.dst >= num_pages) {
            j.dst = -1;
            report(err, GDN_ERR_INVALID_ARG, kTagPage);
        } else if (j.dst >= 0 && __ldcg(owner + j.dst) != i) {
            j.dst = -1;
            report(err, GDN_ERR_INVALID_ARG, kTagSharedPage);
        }
        if (j.src == j.dst) j.dst = -1;
        jobs[i] = j;
    }
}

// Jobs of a fork: request i, when its parent is in use (or negative: a page of zeros), gets the next
// of the lowest-numbered free pages; `list` takes their numbers. With share no page is taken: the
// parent's count goes up.
__global__ void __launch_bounds__(kThreads)
    fork_jobs_kernel(int num_pages, int* refs, int n, const int* parents, int* children, int share,
                     Job* jobs, int* list, DeviceError* err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x;
    int wanted = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + t;
        const int parent = i < n ? parents[i] : 0;
        const bool used = i < n && in_range(parent, num_pages) && __ldcg(refs + parent) > 0;
        const bool ok = i < n && (used || (parent < 0 && !share));
        int sum;
        const int rank = wanted + block_scan(ok, sum);
        wanted += sum;
        if (i < n) {
            jobs[i] = Job{parent, ok ? rank : -1};
            if (!ok) report(err, GDN_ERR_INVALID_ARG, parent < num_pages ? kTagFreePage : kTagPage);
        }
    }
    int found = 0;
    if (share) {
        __syncthreads();   // every parent's count has been looked at
        for (int i = t; i < n; i += kThreads) {
            const bool ok = jobs[i].dst >= 0;
            if (ok) atomicAdd(refs + jobs[i].src, 1);
            children[i] = ok ? jobs[i].src : -1;
        }
        return;
    }
    for (int p0 = 0; p0 < num_pages && found < wanted; p0 += kThreads * kItems) {
        const int mine = p0 + t * kItems;
        unsigned free = 0;
#pragma unroll
        for (int j = 0; j < kItems; ++j)
            if (mine + j < num_pages && refs[mine + j] <= 0) free |= 1u << j;
        int sum;
        int rank = found + block_scan(__popc(free), sum);
        found += sum;
        for (; free && rank < wanted; free &= free - 1, ++rank) {
            const int page = mine + __ffs(free) - 1;
            list[rank] = page;
            refs[page] = 1;
        }
    }
    __syncthreads();
    for (int i = t; i < n; i += kThreads) {
        const int rank = jobs[i].dst;
        const int child = rank >= 0 && rank < found ? list[rank] : -1;
        if (rank >= found) report(err, GDN_ERR_NO_PAGE, kTagFull);
        jobs[i].dst = child;
        children[i] = child;
    }
}

// Jobs of a compaction: the `live` pages in use that lie at or behind page `live` go, in order, to the
// free pages in front of it (there are as many). remap: the new number of every page, -1 for free ones.
__global__ void __launch_bounds__(kThreads)
    compact_jobs_kernel(int num_pages, int* refs, int n, int* table, int* remap, int* live_out,
                        Job* jobs, int* count, DeviceError* err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x;
    int live = 0;
    for (int p0 = 0; p0 < num_pages; p0 += kThreads * kItems) {
        int used = 0, sum;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int p = p0 + t * kItems + j;
            used += p < num_pages && refs[p] > 0;
        }
        block_scan(used, sum);
        live += sum;
    }
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < num_pages; p0 += kThreads * kItems) {
        const int mine = p0 + t * kItems;
        unsigned hole = 0, mover = 0;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int p = mine + j;
            if (p >= num_pages) continue;
            const bool used = refs[p] > 0;
            remap[p] = used ? p : -1;
            if (!used && p < live) hole |= 1u << j;
            if (used && p >= live) mover |= 1u << j;
        }
        int sum;
        int h = holes + block_scan(__popc(hole), sum);
        holes += sum;
        int m = movers + block_scan(__popc(mover), sum);
        movers += sum;
        for (; hole; hole &= hole - 1) jobs[h++].dst = mine + __ffs(hole) - 1;
        for (; mover; mover &= mover - 1) jobs[m++].src = mine + __ffs(mover) - 1;
    }
    __syncthreads();
    for (int j = t; j < movers; j += kThreads) {
        const Job job = jobs[j];
        remap[job.src] = job.dst;
        refs[job.dst] = refs[job.src];
        refs[job.src] = 0;
    }
    if (t == 0) {
        *count = movers;
        if (live_out) *live_out = live;
    }
    __syncthreads();
    for (int i = t; i < n; i += kThreads) {
        const int p = table[i];
        if (p < 0) continue;
        const int to = p < num_pages ? remap[p] : -1;
        if (to < 0) report(err, GDN_ERR_INVALID_ARG, p < num_pages ? kTagFreePage : kTagPage);
        table[i] = to;
    }
}

// Counts of the pages in `list` go down by one each time they are named; one that would fall below zero
// is put back (so it ends at zero however often it is named).
__global__ void __launch_bounds__(256)
    free_kernel(int num_pages, int* refs, int n, const int* list, DeviceError* err) {
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
        const int p = list[i];
        if (p < 0) continue;
        if (p >= num_pages) {
            report(err, GDN_ERR_INVALID_ARG, kTagPage);
        } else if (atomicSub(refs + p, 1) <= 0) {
            atomicAdd(refs + p, 1);
            report(err, GDN_ERR_INVALID_ARG, kTagFreePage);
        }
    }
}

// The bytes. A piece of 64 KB is read whole into the registers of a block and then written, one block an SM: long
// runs of reads and of writes, which memory turns between less often. 48 pages of 2 MB in 12 layers, 256
// threads with 16 loads of 16 bytes each: one block an SM 348 us (42 pages read, 48 written: 6.5 TB/s, 96 % of
// a large copy), two 369; 8 loads each: two blocks 369, four 379-385 us; 2 loads each: 600 us; bulk copies through
// shared memory, 16 or 32 KB a stage: 380 us. Pages of less than 64 KB go to as few warps each as hold them.
constexpr int kMoveThreads = 256, kUnroll = 16;
__global__ void __launch_bounds__(kMoveThreads)
    move_kernel(char* pages, int layers, int num_pages, size_t page_bytes, int threads, const Job* jobs, int n,
                const int* count) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (count) n = min(n, __ldcg(count));
    const int piece = threads * kUnroll * 16, t = threadIdx.x % threads, sets = kMoveThreads / threads;
    const long long pieces = (long long)((page_bytes + piece - 1) / piece);
    const long long total = (long long)n * layers * pieces;
    for (long long item = (long long)blockIdx.x * sets + threadIdx.x / threads; item < total;
         item += (long long)gridDim.x * sets) {
        const long long jl = item / pieces;
        const int j = (int)(jl / layers), layer = (int)(jl - (long long)j * layers);
        const size_t off = (size_t)(item - jl * pieces) * piece;
        const Job job{__ldcg(&jobs[j].src), __ldcg(&jobs[j].dst)};
        if (job.dst < 0) continue;
        const size_t base = (size_t)layer * num_pages;
        const uint4* src = reinterpret_cast<const uint4*>(pages + (base + max(job.src, 0)) * page_bytes + off);
        uint4* dst = reinterpret_cast<uint4*>(pages + (base + job.dst) * page_bytes + off);
        const int units = (int)(min((size_t)piece, page_bytes - off) / 16);
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int at = u * threads + t;
            x[u] = make_uint4(0, 0, 0, 0);
            if (job.src >= 0 && at < units) x[u] = src[at];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int at = u * threads + t;
            if (at < units) dst[at] = x[u];
        }
    }
}

struct CacheLayout {
    size_t off_owner, off_jobs, off_list, total;
};

// [header | a page number (or pair) per page | jobs | free pages found]
CacheLayout cache_layout(int num_pages, int n) {
    CacheLayout w{};
    w.off_owner = kWsHeader;
    w.off_jobs = w.off_owner + ws_round(sizeof(int) * (size_t)num_pages);
    w.off_list = w.off_jobs + ws_round(sizeof(Job) * std::max((size_t)n, (size_t)num_pages / 2 + 1));
    w.total = w.off_list + ws_round(sizeof(int) * (size_t)n);
    return w;
}

struct Pages {
    void* pages;
    int layers, num_pages;
    size_t page_bytes;
};

cudaError_t launch_move(const Pages& c, const Job* jobs, int n, const int* count, cudaStream_t s) {
    // threads of a piece: fewer where they hold a whole page (finer pieces of large pages made no difference)
    int threads = kMoveThreads;
    while (threads > 32 && (size_t)(threads / 2) * kUnroll * 16 >= c.page_bytes) threads /= 2;
    const size_t piece = (size_t)threads * kUnroll * 16, sets = kMoveThreads / threads;
    const size_t most = (size_t)n * (size_t)c.layers * ((c.page_bytes + piece - 1) / piece);
    const size_t blocks = std::min<size_t>((most + sets - 1) / sets, (size_t)std::max(1, current_sm_count()));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::max<size_t>(1, blocks));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;   // the dependent of the launch that makes the jobs
    return cudaLaunchKernelEx(&cfg, move_kernel, (char*)c.pages, c.layers, c.num_pages, c.page_bytes,
                              threads, jobs, n, count);
}

bool off_int(const void* ptr) { return reinterpret_cast<uintptr_t>(ptr) & 3u; }

gdn_status check_pages(const Pages& c, int n) {
    if (c.layers < 1 || c.num_pages < 1 || n < 0 || !c.pages) return GDN_ERR_INVALID_ARG;
    if (c.num_pages > kMostCount || n > kMostCount) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (c.page_bytes == 0 || c.page_bytes % 16 != 0 || c.page_bytes >= ((size_t)1 << 40))
        return GDN_ERR_UNSUPPORTED_SHAPE;
    if (reinterpret_cast<uintptr_t>(c.pages) & 15u) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

gdn_status check_ws(int num_pages, int n, const void* ws, size_t bytes) {
    if (!ws || bytes < cache_layout(num_pages, n).total) return GDN_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 15u) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_cache_workspace_bytes(int num_pages, int n) {
    if (num_pages < 1 || n < 0 || num_pages > kMostCount || n > kMostCount) return 0;
    return cache_layout(num_pages, n).total;
}

gdn_status gdn_cache_copy(void* pages, int layers, int num_pages, size_t page_bytes, int n,
                          const int* src, const int* dst, void* workspace, size_t workspace_bytes,
                          void* stream) {
    const Pages c{pages, layers, num_pages, page_bytes};
    gdn_status st = check_pages(c, n);
    if (st != GDN_OK) return st;
    if (n > 0 && (!src || !dst)) return GDN_ERR_INVALID_ARG;
    if (off_int(src) || off_int(dst)) return GDN_ERR_MISALIGNED;
    if ((st = check_ws(num_pages, n, workspace, workspace_bytes)) != GDN_OK) return st;
    if ((st = current_device_status()) != GDN_OK) return st;
    if (n == 0) return GDN_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = reinterpret_cast<char*>(workspace);
    const CacheLayout w = cache_layout(num_pages, n);
    Job* jobs = reinterpret_cast<Job*>(ws + w.off_jobs);
    copy_jobs_kernel<<<1, kThreads, 0, s>>>(num_pages, n, src, dst, reinterpret_cast<int*>(ws + w.off_owner),
                                            jobs, reinterpret_cast<DeviceError*>(ws));
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    return launch_move(c, jobs, n, nullptr, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_cache_fork(void* pages, int layers, int num_pages, size_t page_bytes, int* refs, int n,
                          const int* parents, int* children, int share, void* workspace,
                          size_t workspace_bytes, void* stream) {
    const Pages c{pages, layers, num_pages, page_bytes};
    gdn_status st = check_pages(c, n);
    if (st != GDN_OK) return st;
    if (!refs || (n > 0 && (!parents || !children)) || (share != 0 && share != 1)) return GDN_ERR_INVALID_ARG;
    if (off_int(refs) || off_int(parents) || off_int(children)) return GDN_ERR_MISALIGNED;
    if ((st = check_ws(num_pages, n, workspace, workspace_bytes)) != GDN_OK) return st;
    if ((st = current_device_status()) != GDN_OK) return st;
    if (n == 0) return GDN_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = reinterpret_cast<char*>(workspace);
    const CacheLayout w = cache_layout(num_pages, n);
    Job* jobs = reinterpret_cast<Job*>(ws + w.off_jobs);
    fork_jobs_kernel<<<1, kThreads, 0, s>>>(num_pages, refs, n, parents, children, share, jobs,
                                            reinterpret_cast<int*>(ws + w.off_list),
                                            reinterpret_cast<DeviceError*>(ws));
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    if (share) return GDN_OK;
    return launch_move(c, jobs, n, nullptr, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_cache_free(int num_pages, int* refs, int n, const int* list, void* workspace,
                          size_t workspace_bytes, void* stream) {
    if (num_pages < 1 || n < 0 || !refs || (n > 0 && !list)) return GDN_ERR_INVALID_ARG;
    if (num_pages > kMostCount || n > kMostCount) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (off_int(refs) || off_int(list)) return GDN_ERR_MISALIGNED;
    gdn_status st = check_ws(num_pages, 0, workspace, workspace_bytes);
    if (st != GDN_OK) return st;
    if ((st = current_device_status()) != GDN_OK) return st;
    if (n == 0) return GDN_OK;
    const int blocks = std::min((n + 255) / 256, 1024);
    free_kernel<<<blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        num_pages, refs, n, list, reinterpret_cast<DeviceError*>(workspace));
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_cache_compact(void* pages, int layers, int num_pages, size_t page_bytes, int* refs,
                             int n, int* table, int* remap, int* live, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const Pages c{pages, layers, num_pages, page_bytes};
    gdn_status st = check_pages(c, n);
    if (st != GDN_OK) return st;
    if (!refs || (n > 0 && !table)) return GDN_ERR_INVALID_ARG;
    if (off_int(refs) || off_int(table) || off_int(remap) || off_int(live)) return GDN_ERR_MISALIGNED;
    if ((st = check_ws(num_pages, 0, workspace, workspace_bytes)) != GDN_OK) return st;
    if ((st = current_device_status()) != GDN_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = reinterpret_cast<char*>(workspace);
    const CacheLayout w = cache_layout(num_pages, 0);
    Job* jobs = reinterpret_cast<Job*>(ws + w.off_jobs);
    int* count = reinterpret_cast<int*>(ws + kWsVerdict);
    compact_jobs_kernel<<<1, kThreads, 0, s>>>(num_pages, refs, n, table,
                                               remap ? remap : reinterpret_cast<int*>(ws + w.off_owner), live,
                                               jobs, count, reinterpret_cast<DeviceError*>(ws));
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    return launch_move(c, jobs, num_pages / 2, count, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
