// fg_pages.cu - block tables, slots and positions of a step's tokens from the requests' lengths.
//
// Every CTA scans all requests (three sums: tokens, pages given back, pages taken), so that none waits
// for another's result; the work behind the scan (pages pushed and popped, one slot and position a
// token) is dealt over the CTAs of one cluster.  A cluster barrier stands between what is read of the
// caller's arrays and what is written over them, and between the pages pushed and the pages popped.
// Bound: latency (256 requests of a token each, or 48 of up to 512 tokens: 4.8 us).
#include <cuda_runtime.h>

#include "fg.h"
#include "fg_host.h"
#include "fg_kv.cuh"

namespace {

using fg::al;

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
constexpr int kPer = 4;                       // requests a thread scans
constexpr int kMaxRequests = 4000;             // three words each in 48 KB, and at most kThreads * kPer
static_assert(kMaxRequests <= kThreads * kPer, "requests that a CTA scans");
constexpr int kMaxTokens = 1 << 18, kMaxTable = 1 << 18;   // sums over all requests stay below 2^31

struct PagesParams {
    int S, T, page, max_pages, num_pages, free_len;
    const int32_t *context, *fresh;
    int32_t* free;
    const int32_t* count;
    int32_t *count_out, *table, *start, *lens, *slots, *positions;
    int* status;
};

struct Sums {
    int tokens, back, more;
};

__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return Sums{a.tokens + b.tokens, a.back + b.back, a.more + b.more}; }

__device__ __forceinline__ Sums shfl_up(Sums v, int o) {
    return Sums{__shfl_up_sync(0xffffffffu, v.tokens, o), __shfl_up_sync(0xffffffffu, v.back, o),
                __shfl_up_sync(0xffffffffu, v.more, o)};
}

// Pages of n >= 0 tokens.  Unsigned: n + page - 1 may pass 2^31 (a page holds up to 2^31 - 1 tokens), and not 2^32.
__device__ __forceinline__ int pages_of(int n, int page) {
    return static_cast<int>((static_cast<unsigned>(n) + static_cast<unsigned>(page) - 1) / static_cast<unsigned>(page));
}

// Last r with a[r] <= i, a[0] == 0, over n entries.
__device__ __forceinline__ int find(const int* a, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <bool kClustered>
__global__ void __launch_bounds__(kThreads) pages_kernel(const PagesParams p) {
    extern __shared__ int sm[];
    int* s_start = sm;                        // [S] tokens before a request
    int* s_more = sm + p.S;                   // [S] pages given back before it, then pages taken before it
    int* s_context = sm + 2 * p.S;            // [S]
    __shared__ Sums s_warp[32];
    __shared__ int s_bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x, ctas = gridDim.x;
    if (tid == 0) s_bad = 0;
    fg::grid_dependency_wait();
    if (tid == 0) fg::grid_launch_dependents();
    __syncthreads();

    int context[kPer], fresh[kPer];
    Sums mine{0, 0, 0}, each[kPer];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int r = tid * kPer + i;
        const bool in = r < p.S;
        context[i] = in ? p.context[r] : 0;
        fresh[i] = in ? p.fresh[r] : 0;
        each[i] = Sums{0, 0, 0};
        if (!in) continue;
        const int most = p.max_pages * p.page;             // within int32 (checked by the caller)
        if (context[i] < 0 || context[i] > most || fresh[i] < -1 || fresh[i] > p.T || fresh[i] > most - context[i]) {
            bad = true;
            continue;
        }
        const int held = pages_of(context[i], p.page);
        if (fresh[i] < 0) each[i].back = held;
        else {
            each[i].tokens = fresh[i];
            each[i].more = pages_of(context[i] + fresh[i], p.page) - held;
        }
        mine = mine + each[i];
    }
    if (bad) s_bad = 1;
    const int count = *p.count;
    Sums incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums y = shfl_up(incl, o);
        if (lane >= o) incl = incl + y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        Sums v = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums y = shfl_up(v, o);
            if (lane >= o) v = v + y;
        }
        s_warp[lane] = v;
    }
    __syncthreads();
    const Sums total = s_warp[kThreads / 32 - 1];
    bad = s_bad || total.tokens > p.T || count < 0 || count > p.free_len || total.back > p.free_len - count ||
          total.more > count + total.back;
    Sums at = warp ? s_warp[warp - 1] + incl : incl;        // inclusive
    at = Sums{at.tokens - mine.tokens, at.back - mine.back, at.more - mine.more};
    const Sums before = at;
    const int step = ctas * kThreads, first = rank * kThreads + tid;
    if (!bad && total.back > 0) {                           // the same for all: finished requests' pages, dealt by the page
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = tid * kPer + i;
            if (r < p.S) s_more[r] = at.back;
            at = at + each[i];
        }
        __syncthreads();
        for (int i = first; i < total.back; i += step) {
            const int r = find(s_more, p.S, i);
            p.free[count + i] = p.table[(long long)r * p.max_pages + i - s_more[r]];
        }
        __syncthreads();
        at = before;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int r = tid * kPer + i;
        if (r < p.S) {
            s_start[r] = at.tokens;
            s_more[r] = at.more;
            s_context[r] = context[i];
        }
        at = at + each[i];
    }
    if constexpr (kClustered) {
        __threadfence();
        __syncthreads();
        fg::cluster_sync();
    } else {
        __syncthreads();
    }
    const int top = count + total.back;                     // pages to take from
    if (rank == 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = tid * kPer + i;
            if (r >= p.S) break;
            p.start[r] = bad ? 0 : s_start[r];
            p.lens[r] = bad ? max(context[i], 0) : fresh[i] < 0 ? 0 : context[i] + fresh[i];
        }
        if (tid == 0) {
            p.start[p.S] = bad ? 0 : total.tokens;
            *p.count_out = bad ? count : top - total.more;
            if (bad) fg::kv_record(p.status, fg::kKvErrPages);
        }
    }
    if (!bad) {
        for (int i = first; i < total.more; i += step) {    // new pages into the table
            const int r = find(s_more, p.S, i);
            const int held = pages_of(s_context[r], p.page);
            p.table[(long long)r * p.max_pages + held + i - s_more[r]] = __ldcg(p.free + top - 1 - i);
        }
    }
    for (int i = first; i < p.T; i += step) {
        int slot = -1, pos = -1;
        if (!bad && i < total.tokens) {
            const int r = find(s_start, p.S, i);
            pos = s_context[r] + i - s_start[r];
            const int held = pages_of(s_context[r], p.page), j = pos / p.page;
            const int id = j < held ? __ldcg(p.table + (long long)r * p.max_pages + j)
                                    : __ldcg(p.free + top - 1 - (s_more[r] + j - held));
            if (id >= 0 && id < p.num_pages) slot = id * p.page + pos % p.page;
            else fg::kv_record(p.status, fg::kKvErrPages);
        }
        p.slots[i] = slot;
        p.positions[i] = pos;
    }
}

}  // namespace

extern "C" int fg_build_block_tables(int S, int T, int page_size, int num_pages, int max_pages, int free_len,
                                     const int32_t* context_lens, const int32_t* new_lens, int32_t* free_pages,
                                     const int32_t* free_count, int32_t* block_table, int32_t* query_start,
                                     int32_t* seq_lens, int32_t* slots, int32_t* positions, int32_t* free_count_out,
                                     fg_stream_t stream) {
    if (S < 0 || T < 0 || page_size < 1 || num_pages < 1 || max_pages < 1 || free_len < 0 ||
        (long long)page_size * num_pages > 0x7fffffffLL || (long long)page_size * max_pages > 0x7fffffffLL)
        return FG_ERR_INVALID_ARG;
    if (S > kMaxRequests || T > kMaxTokens || max_pages > kMaxTable || free_len > 1 << 30) return FG_ERR_UNSUPPORTED;
    if (!free_count || !query_start || !free_count_out || !al(free_count, 4) || !al(query_start, 4) || !al(free_count_out, 4) ||
        (S > 0 && (!context_lens || !new_lens || !block_table || !seq_lens)) || (T > 0 && (!slots || !positions)) ||
        (free_len > 0 && !free_pages) || !al(context_lens, 4) || !al(new_lens, 4) || !al(free_pages, 4) || !al(block_table, 4) ||
        !al(seq_lens, 4) || !al(slots, 4) || !al(positions, 4))
        return FG_ERR_INVALID_ARG;
    fg::HostState st;
    if (const int rc = fg::host_state(&st)) return rc;
    const PagesParams p{S, T, page_size, max_pages, num_pages, free_len, context_lens, new_lens, free_pages, free_count,
                        free_count_out, block_table, query_start, seq_lens, slots, positions, st.status};
    // one CTA does a decode step's tokens in one go; a prompt's are dealt over a cluster
    const bool clustered = T > kThreads;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(clustered ? kCluster : 1);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 3 * S * sizeof(int);             // at most 48000 bytes
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    if (clustered) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = kCluster;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (st.pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    const cudaError_t e = clustered ? cudaLaunchKernelEx(&cfg, pages_kernel<true>, p) : cudaLaunchKernelEx(&cfg, pages_kernel<false>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    return FG_OK;
}
