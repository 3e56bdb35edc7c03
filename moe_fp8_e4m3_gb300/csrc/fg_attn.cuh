// fg_attn.cuh - what the attention kernels over the 4-bit cache share: a launch's parameters, the cut of all
// items into equal shares, and the join of an item's pieces.
//
// An item is (request, chunk of kRows rows, kv head); its keys are cut into blocks of kBlock tokens.  The blocks of all
// items stand in one line that is cut into equal shares, one per CTA, from lengths that only the device knows; an
// item that crosses a cut leaves partial results (a row's maximum, sum and unscaled output) in the workspace, and
// the CTA that arrives last joins them in the items' order, so results do not depend on the order of arrival.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "fg_kv.cuh"

namespace fg {

constexpr int kAttnMaxCtas = 640;             // shares of a launch, at most
constexpr int kAttnMaxRequests = 4096;
constexpr float kAttnEmpty = -3e38f;          // maximum of a row without a key: below every score, and finite
constexpr uint32_t kAllLanes = 0xffffffffu;

struct AttnParams {
    const uint16_t* q;
    const uint8_t *kc, *ks, *vc, *vs;
    const int32_t *table, *start, *lens;
    uint16_t* out;
    int T, S, heads, group, page, pages, max_pages, window;
    float scale_log2;                          // scale * log2(e)
    unsigned* ctr;                             // [3 * kAttnMaxCtas]: per item, then per eight pieces
    float* part;                               // [2 * kAttnMaxCtas][kRows][D + 2]: M, l, O
    int* status;
    unsigned long long timeout_ns;
    int stall;                                 // for tests: a key tile that is never announced
};


__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One request as the kernels see it (n == 0: nothing to do, or its lengths are wrong; then t0 < 0: query_start falls).
struct AttnRequest {
    int n, len, t0;
};
__device__ __forceinline__ AttnRequest attn_request(const AttnParams& p, int r) {
    const int t0 = __ldcg(p.start + r), t1 = __ldcg(p.start + r + 1), len = __ldcg(p.lens + r);
    const bool ok = t0 >= 0 && t1 >= t0 && t1 <= p.T && len >= 0 && len <= (long long)p.max_pages * p.page;
    return ok ? AttnRequest{t1 - t0, len, t0} : AttnRequest{0, 0, t1 < t0 ? -1 : 0};
}
// Whether a request's rows begin before those of an earlier one end, so that two might write the same ones.  Where
// query_start does not fall there is none.
__device__ __forceinline__ bool attn_claimed_twice(const AttnParams& p) {
    int end = 0;
#pragma unroll 1
    for (int q = 0; q < p.S; ++q) {
        const AttnRequest x = attn_request(p, q);
        if (x.n == 0) continue;
        if (x.t0 < end) return true;
        end = x.t0 + x.n;
    }
    return false;
}
// First key that a row at position hi - 1 looks at.  A row before position 0 has a negative hi, of which a window as large
// as its type is not taken away: the difference would wrap.
__device__ __forceinline__ int attn_from(const AttnParams& p, int hi) {
    return p.window > 0 ? max(0, max(hi, 0) - p.window) : 0;
}
// The same where nothing depends on it for hi <= 0, and what is below 0 counts as 0: without a comparison, and allowed to wrap.
__device__ __forceinline__ int attn_back(const AttnParams& p, int hi) {
    return p.window > 0 ? static_cast<int>(static_cast<unsigned>(hi) - static_cast<unsigned>(p.window)) : 0;
}
// Keys [lo, hi) that some row of a chunk looks at; hi <= lo: none.
struct AttnKeys {
    int lo, hi;
};

// Shared memory of a plan.
template <int kThreads>
struct AttnPlanSmem {
    unsigned long long warp[kThreads / 32], strip[kThreads];
    volatile unsigned long long line[4];       // shares, blocks of all items, this share's end, where the current item begins
    int last;
};

// Where a CTA stands in the line.
// kByRequest: requests bring few chunks (and a CTA's blocks are short).
template <int kRows, int kBlock, int kThreads, bool kByRequest>
struct AttnCursor {
    AttnRequest rq;
    AttnKeys keys;
    int r, ch, h, cost, off0;                  // request, chunk (of all), head, the item's cost, the share's begin within it
    unsigned long long begin;                  // where the item begins; the next one's while next() runs

    // What every item takes besides its keys (its q, filling the pipeline, the join), in blocks.
    static constexpr int kStart = kByRequest ? 5 : 3;
    static constexpr unsigned long long kCostMask = (1ull << 40) - 1;

    static __device__ __forceinline__ void complain(const AttnParams& p, int q) {   // of a request without rows: are its lengths right?
        const int t0 = __ldcg(p.start + q), t1 = __ldcg(p.start + q + 1), len = __ldcg(p.lens + q);
        if (t0 != t1 || t0 < 0 || t0 > p.T || len < 0 || len > (long long)p.max_pages * p.page) kv_record(p.status, kKvErrAttention);
    }
    __device__ __forceinline__ void look(const AttnParams& p, const int* s_pre) {
        rq = attn_request(p, r);
        look_at(p, ch - s_pre[r]);
    }
    __device__ __forceinline__ void look_at(const AttnParams& p, int chunk) {
        const int i0 = chunk * kRows / p.group, i1 = min(rq.n - 1, (chunk * kRows + kRows - 1) / p.group);
        keys.hi = rq.len - rq.n + i1 + 1;
        keys.lo = attn_from(p, rq.len - rq.n + i0 + 1);
        cost = kStart + (keys.hi > keys.lo ? (keys.hi + kBlock - 1) / kBlock - keys.lo / kBlock : 1);
    }

    // Sum of v over the threads before this one, and of all.
    static __device__ __forceinline__ unsigned long long scan(unsigned long long v, unsigned long long* s_warp, unsigned long long& total) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        unsigned long long incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(kAllLanes, incl, o);
            if (lane >= o) incl += y;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        unsigned long long before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            total += s_warp[w];
        }
        return before + incl - v;
    }

    // Last entry of a with a[i] <= x, a[0] == 0, over n entries.
    static __device__ __forceinline__ int find(const int* a, int n, int x) {
        int lo = 0, hi = n;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a[mid] <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }

    // Works out this CTA's share and its first item; false: there is none.  All threads call it.  Chunks per request,
    // then blocks per chunk, are scanned in strips of consecutive entries.
    __device__ __forceinline__ bool open(const AttnParams& p, AttnPlanSmem<kThreads>& sm, int* s_pre) {
        const int tid = threadIdx.x;
        unsigned long long total_blocks;
        constexpr int kFew = 64;                               // chunks that a thread walks
        if (kByRequest && p.S <= kThreads) {
            // few chunks a request, a request a thread: chunks and costs in one scan
            unsigned long long sum = 0, total;
            int n = 0;
            ch = 0;
            r = 0;
            rq.t0 = 0;
            if (tid < p.S) {
                rq = attn_request(p, tid);
                n = static_cast<int>(((long long)rq.n * p.group + kRows - 1) / kRows);
            }
            if (!__syncthreads_or(n > kFew || rq.t0 < 0)) {
                if (blockIdx.x == 0 && tid < p.S && rq.n == 0) complain(p, tid);
                for (int i = 0; i < n; ++i) {
                    look_at(p, i);
                    sum += cost;
                }
                sum |= static_cast<unsigned long long>(n) << 40;   // costs stay below 2^39: kThreads x kFew chunks of at most 2^24 blocks
                static_assert(kThreads * kFew <= 1 << 14 || !kByRequest, "room for both");
                const unsigned long long at = scan(sum, sm.warp, total);
                sm.strip[tid] = at & kCostMask;
                if (tid <= p.S) s_pre[tid] = static_cast<int>(at >> 40);
                if (tid == 0 && p.S == kThreads) s_pre[kThreads] = static_cast<int>(total >> 40);
                total_blocks = total & kCostMask;
                __syncthreads();
                return settle(p, sm, s_pre, total_blocks, true);
            }
        }
        const int per_r = (p.S + kThreads - 1) / kThreads;
        {
            constexpr unsigned long long kFalls = 1ull << 48;      // of query_start, counted above the chunks (below 2^36)
            unsigned long long sum = 0, total;
            for (int i = 0; i < per_r; ++i) {
                const int q = tid * per_r + i;
                if (q >= p.S) break;
                const AttnRequest x = attn_request(p, q);
                if (blockIdx.x == 0 && x.n == 0) complain(p, q);
                sum += ((long long)x.n * p.group + kRows - 1) / kRows + (x.t0 < 0 ? kFalls : 0);
            }
            unsigned long long at = scan(sum, sm.warp, total) % kFalls;
            if (total >= kFalls && attn_claimed_twice(p)) return false;    // the fall is on record
            for (int i = 0; i < per_r; ++i) {
                const int q = tid * per_r + i;
                if (q >= p.S) break;
                s_pre[q] = static_cast<int>(at);
                at += ((long long)attn_request(p, q).n * p.group + kRows - 1) / kRows;
            }
            if (tid == 0) s_pre[p.S] = static_cast<int>(total % kFalls);
        }
        __syncthreads();
        const int chunks = s_pre[p.S];
        const int per_c = (chunks + kThreads - 1) / kThreads;
        {
            unsigned long long sum = 0;
            ch = tid * per_c;
            if (ch < chunks) {
                r = find(s_pre, p.S, ch);
                for (int i = 0; i < per_c && ch < chunks; ++i, ++ch) {
                    while (s_pre[r + 1] <= ch) ++r;
                    look(p, s_pre);
                    sum += cost;
                }
            }
            const unsigned long long at = scan(sum, sm.warp, total_blocks);
            sm.strip[tid] = at;
        }
        __syncthreads();
        return settle(p, sm, s_pre, total_blocks, false);
    }

    // Finds this CTA's share and its first item.  by_request: the strips are requests, else per_c chunks each.
    __device__ __forceinline__ bool settle(const AttnParams& p, AttnPlanSmem<kThreads>& sm, const int* s_pre, unsigned long long total_blocks,
                                           bool by_request) {
        const unsigned long long all = total_blocks * p.heads;
        // a share is worth an item's start
        const unsigned long long shares = min(static_cast<unsigned long long>(gridDim.x), (all + kStart) / (kStart + 1));
        if (blockIdx.x >= shares) return false;
        const unsigned long long u = all * blockIdx.x / shares;
        if (threadIdx.x == 0) { sm.line[0] = shares; sm.line[1] = all; sm.line[2] = all * (blockIdx.x + 1) / shares; }
        __syncthreads();
        // the chunk that holds u: its strip, then the strip's chunks one by one
        int lo = 0, hi = by_request ? p.S : kThreads;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.strip[mid] * p.heads <= u) lo = mid;
            else hi = mid;
        }
        begin = sm.strip[lo] * p.heads;
        if (by_request) {
            r = lo;
            ch = s_pre[lo];
        } else {
            ch = lo * ((s_pre[p.S] + kThreads - 1) / kThreads);
            r = find(s_pre, p.S, ch);
        }
        while (s_pre[r + 1] <= ch) ++r;
        look(p, s_pre);
        while (begin + (unsigned long long)cost * p.heads <= u) {
            begin += (unsigned long long)cost * p.heads;
            ++ch;
            while (s_pre[r + 1] <= ch) ++r;
            look(p, s_pre);
        }
        h = static_cast<int>((u - begin) / cost);
        begin += (unsigned long long)h * cost;
        off0 = static_cast<int>(u - begin);
        return true;
    }

    // Blocks [b0, b1) of the current item that are this share's; false: none of them, and the share ends here.
    __device__ __forceinline__ bool piece(AttnPlanSmem<kThreads>& sm, int& b0, int& b1) const {
        const int off1 = static_cast<int>(min(static_cast<unsigned long long>(cost), sm.line[2] - begin));
        if (off1 <= kStart) return false;
        if (threadIdx.x == 0) sm.line[3] = begin;            // read again behind the piece's first barrier
        const int block0 = keys.hi > keys.lo ? keys.lo / kBlock : 0;
        b0 = block0 + max(off0 - kStart, 0);
        b1 = block0 + off1 - kStart;
        return true;
    }

    // The CTAs that hold pieces of the current item, first and last.
    __device__ __forceinline__ void holders(AttnPlanSmem<kThreads>& sm, int& a, int& z) const {
        const unsigned long long at = sm.line[3], shares = sm.line[0], all = sm.line[1];
        a = static_cast<int>(((at + kStart + 1) * shares - 1) / all);
        z = static_cast<int>(((at + cost) * shares - 1) / all);
    }

    // On to the next item; false: the share ends with this one.  Every thread calls it, and a barrier stands between it
    // and the next piece().
    __device__ __forceinline__ bool next(const AttnParams& p, AttnPlanSmem<kThreads>& sm, const int* s_pre) {
        begin = sm.line[3] + cost;
        if (begin >= sm.line[2]) return false;
        off0 = 0;
        if (++h == p.heads) {
            h = 0;
            ++ch;
            while (s_pre[r + 1] <= ch) ++r;
            look(p, s_pre);
        }
        return true;
    }
};

// Floats of a partial result: kRows maxima, kRows sums, kRows x D outputs (rows outermost, or kByColumn: groups of four
// columns outermost, for writers that hold a row a thread).
template <int kRows, int D>
__host__ __device__ constexpr int attn_slot() { return kRows * (D + 2); }

// Where CTA k keeps its piece of the item that begins at CTA a.
template <int kRows, int D>
__device__ __forceinline__ float* attn_piece(const AttnParams& p, int k, int a) {
    return p.part + (long long)(2 * k + (k == a ? 1 : 0)) * attn_slot<kRows, D>();
}

template <int D>
__device__ __forceinline__ void attn_store(const AttnParams& p, int t0, int h, int row, int d4, float4 v) {
    const int i = row / p.group, hq = h * p.group + row % p.group;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p.out + ((long long)(t0 + i) * p.heads * p.group + hq) * D + 4 * d4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Joins `count` pieces of the item that begins at CTA a, those of CTAs k0, k0 + stride, ...; kFlight of them and kSame
// quarters of rows a thread in flight together.  done(it, maximum, sum, four outputs) takes each quarter row.
template <int kRows, int D, int kThreads, bool kByColumn, int kFlight, int kSame, class F>
__device__ __forceinline__ void attn_join_rows(const AttnParams& p, int a, int k0, int count, int stride, int rows, const F& done) {
    const int end = (kByColumn ? kRows : rows) * (D / 4);
    for (int it0 = threadIdx.x; it0 < end; it0 += kThreads * kSame) {
        float top[kSame], sum[kSame];
        float4 acc[kSame];
#pragma unroll
        for (int q = 0; q < kSame; ++q) {
            top[q] = kAttnEmpty;
            sum[q] = 0.0f;
            acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int x = 0; x < count; x += kFlight) {
            float mk[kSame][kFlight], lk[kSame][kFlight];
            float4 v[kSame][kFlight];
#pragma unroll
            for (int q = 0; q < kSame; ++q) {
                const int it = min(it0 + q * kThreads, end - 1);
                const int j = kByColumn ? it % kRows : it / (D / 4);
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const float* s = attn_piece<kRows, D>(p, k0 + min(x + i, count - 1) * stride, a);
                    mk[q][i] = __ldcg(s + j);
                    lk[q][i] = __ldcg(s + kRows + j);
                    v[q][i] = __ldcg(reinterpret_cast<const float4*>(s + 2 * kRows) + it);
                }
            }
#pragma unroll
            for (int q = 0; q < kSame; ++q) {
                float t = top[q];
#pragma unroll
                for (int i = 0; i < kFlight; ++i) t = fmaxf(t, mk[q][i]);
                const float f = ex2(top[q] - t);
                top[q] = t;
                sum[q] *= f;
                acc[q].x *= f; acc[q].y *= f; acc[q].z *= f; acc[q].w *= f;
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const float e = x + i < count ? ex2(mk[q][i] - t) : 0.0f;
                    sum[q] = fmaf(lk[q][i], e, sum[q]);
                    acc[q].x = fmaf(v[q][i].x, e, acc[q].x); acc[q].y = fmaf(v[q][i].y, e, acc[q].y);
                    acc[q].z = fmaf(v[q][i].z, e, acc[q].z); acc[q].w = fmaf(v[q][i].w, e, acc[q].w);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kSame; ++q)
            if (it0 + q * kThreads < end) done(it0 + q * kThreads, top[q], sum[q], acc[q]);
    }
}

// Whether this CTA is the last of `count` to arrive at a counter, which is left at zero.  All threads call it, behind
// what they have written for the others.
template <int kThreads>
__device__ __forceinline__ bool attn_last(AttnPlanSmem<kThreads>& sm, unsigned* ctr, int count) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        sm.last = atomicAdd(ctr, 1u) == static_cast<unsigned>(count - 1);
        if (sm.last) *ctr = 0;
    }
    __syncthreads();
    if (!sm.last) return false;
    __threadfence();
    return true;
}

// Called by all threads once this CTA's piece is written: the CTA that arrives last joins the pieces of CTAs a to z, in
// their order, and stores rows [row0, row0 + rows).  Many pieces of few rows are joined eight at a time first, each
// eight by its own last CTA.
template <int kRows, int D, int kThreads, bool kByColumn>
__device__ __forceinline__ void attn_join(const AttnParams& p, AttnPlanSmem<kThreads>& sm, int a, int z, int t0, int h, int row0, int rows) {
    auto store = [&](int it, float, float sum, const float4& v) {
        const int j = kByColumn ? it % kRows : it / (D / 4), d4 = kByColumn ? it / kRows : it % (D / 4);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (j < rows) attn_store<D>(p, t0, h, row0 + j, d4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    };
    const int n = z - a + 1;
    if (!kByColumn && n > 12) {
        const int k0 = a + (static_cast<int>(blockIdx.x) - a) / 8 * 8, eight = min(8, z - k0 + 1);
        if (!attn_last<kThreads>(sm, p.ctr + kAttnMaxCtas + 2 * k0 + (k0 == a), eight)) return;
        float* slot = attn_piece<kRows, D>(p, k0, a);
        float* tops = reinterpret_cast<float*>(sm.strip);    // the plan is done with it: the joined maxima and sums
        static_assert(sizeof(sm.strip) >= 2 * kRows * sizeof(float) || kByColumn, "room for them");
        attn_join_rows<kRows, D, kThreads, kByColumn, 8, 1>(p, a, k0, eight, 1, rows, [&](int it, float top, float sum, const float4& v) {
            reinterpret_cast<float4*>(slot + 2 * kRows)[it] = v;
            if (it % (D / 4) == 0) {
                tops[it / (D / 4)] = top;
                tops[kRows + it / (D / 4)] = sum;
            }
        });
        __syncthreads();                                     // every thread has read the pieces' own
        for (int j = threadIdx.x; j < rows; j += kThreads) {
            slot[j] = tops[j];
            slot[kRows + j] = tops[kRows + j];
        }
        if (!attn_last<kThreads>(sm, p.ctr + a, (n + 7) / 8)) return;
        attn_join_rows<kRows, D, kThreads, kByColumn, 8, 1>(p, a, a, (n + 7) / 8, 8, rows, store);
        return;
    }
    if (!attn_last<kThreads>(sm, p.ctr + a, n)) return;
    // pieces in flight together, times rows where there are many: most items are cut once, long ones many times
    if (n <= 2) attn_join_rows<kRows, D, kThreads, kByColumn, 2, (kRows * D / 4) / kThreads >= 4 ? 3 : 1>(p, a, a, n, 1, rows, store);
    else attn_join_rows<kRows, D, kThreads, kByColumn, 8, 1>(p, a, a, n, 1, rows, store);
}

// Launches the kernel for many rows a request (fg_attn_prompt.cu).
// rows: of an item, 128 or (D <= 128) 256.
int launch_attn_prompt(const AttnParams& p, int D, int rows, int sms, int pdl, cudaStream_t stream);
constexpr int kAttnPromptCtas = 152, kAttnPromptRequests = 1024;

}  // namespace fg
