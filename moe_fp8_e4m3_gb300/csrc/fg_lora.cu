// fg_lora.cu - an FP8 projection shared by all tokens plus each token's own low-rank adapter,
// in two launches: v = scaling * x @ A^T per token and adapter (here), then the projection's
// K-groups and the adapters' B against v in one accumulator (fg_stream.cuh).
// Bound: a decode batch by the launch chain and by reading A and B of its distinct adapters, a
// prompt by the projection's units (0.33 us each where nothing waits, their products' time).
// Measured on GB300, both launches: 1 token x 4096 x 4096, rank 16 10.2 us; 64 x 7168 x 4096 with
// 52 adapters of rank 16 21.2 us (2.2 TB/s); 33 x 1008 x 2048, rank 8, FP32 10.6 us; 2048 x 4096 x
// 4096, rank 64, five prompts 61 us, 42 of them the projection (1.7 PFLOP/s).
#include <cuda_bf16.h>

#include <cstdio>
#include <cstring>

#include "fg.h"
#include "fg_host.h"
#include "fg_stream.cuh"

namespace {

using fg::al;
using fg::align4;
using fg::up256;
int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Rank columns as the tensor core takes them: 16 per step, whole or half adapters per unit.
int padded_rank(int r) { return r <= 16 ? 16 : (r <= 32 ? 32 : (r <= 64 ? 64 : 128)); }

struct Layout {
    int bn, rp, tiles;                    // token columns, padded rank, token tiles
    int slots, parts;                     // adapters that a tile may use; BF16 parts of x @ A^T
    long long ids, count, v, part, bytes; // behind the counters (fg_stream.cuh)
};
// Parts of x @ lora_a^T: 16 mantissa bits under a BF16 result, 24 under an FP32 one.
Layout layout(int M, int R, int L, int d_dtype) {
    Layout l;
    l.bn = fg::stream_bn(M);
    l.rp = padded_rank(R);
    l.tiles = ceil_div(M, l.bn);
    l.slots = L < l.bn ? L : l.bn;
    l.parts = d_dtype == FG_F32 ? 3 : 2;
    l.ids = fg::kCounterBytes;
    l.count = l.ids + up256((long long)l.tiles * l.bn * 4);
    l.v = l.count + up256((long long)l.tiles * 4);
    l.part = l.v + up256((long long)l.tiles * l.slots * l.parts * l.bn * l.rp * 2);
    l.bytes = l.part + (long long)fg::kMaxStreamCtas * 2 * 2 * l.bn * 128 * 4;
    return l;
}

bool shapes_ok(int M, int N, int K, int R) {
    if (M < 0 || N < 16 || N % 16 != 0 || K < 128 || K % 128 != 0 || R < 8 || R % 8 != 0 || R > 128) return false;
    const Layout l = layout(M > 0 ? M : 1, R, fg::kMaxListed, FG_F32);
    return l.tiles <= fg::kMaxTokenTiles &&
           (long long)l.tiles * ceil_div(N, 256) * (K / 128 + 8 * l.bn) < (1LL << 31) &&
           (long long)l.tiles * l.bn * 3 * l.bn < (1LL << 31);
}

// ---------------------------------------------------------------- v = scaling * x @ A^T
// Two ways through one kernel, taken per token tile by how many tokens share an adapter.
//
// Few (a decode batch): a work item is (distinct adapter, 8 of the tokens that use it), dealt to the
// tile's CTAs; where there are CTAs to spare, its rank rows are dealt to several (4 x 1072 x 2816,
// rank 128 18.3 -> 9.8 us; always, 113 adapters in 180 tokens 45.7 -> 50.5).  The adapter's rows are
// the M operand of mma.sync (MB blocks of 16), its tokens the N operand, gathered by their row
// numbers.  The 16 warps split K and read both operands straight into registers, 16 bytes (8
// consecutive k) per row and lane: k is summed over, so a lane's 8 values may stand for any k as
// long as A and x agree; they feed two 16-wide steps.  There is nothing to stage: each A element is
// used once (latency-bound: its bytes in flight are what counts, U blocks of 32 k per warp), and
// tcgen05's 128 rows would be mostly empty.  The partial sums meet in shared memory, in warp order.
//
// Many (a prompt's tile of 128 tokens, from 8 tokens per adapter): tcgen05 with the tokens as 128
// rows and up to 256 rank columns of the tile's adapters.  K is split over a cluster of CTAs
// (each streams its few 64-wide chunks through a TMA ring), the partial sums meet through
// distributed shared memory: the CTAs take four tokens in turn and add them up in rank order.  (2048 tokens x
// 4096, rank 64, five prompts: 36 us by the first way, each 32 tokens re-reading their adapter.)
struct ShrinkParams {
    int tokens, bn, K, R, rp, L, max_slots, parts;
    const int32_t* ids;
    const uint16_t* x;          // [tokens][K] BF16
    const uint16_t* lora_a;     // [L][R][K] BF16
    const float* scaling;
    uint16_t* v;                // [token tile][slot][parts][bn][rp] BF16
    int* slot_ids;
    int* slot_count;
    int* status;
    unsigned long long timeout_ns;
};
struct ShrinkMaps {
    CUtensorMap x;              // [tokens][K], boxes of 128 rows x 64
    CUtensorMap a;              // [L][R][K], boxes of rp rows x 64
};

constexpr int kShrinkWarps = 16;
constexpr int kShrinkCluster = 6;                 // measured on GB300: of 16 clusters of 8 one waits for SMs, of 6 none
constexpr int kTcStages = 4, kTcXBytes = 128 * 128, kTcABytes = 256 * 128;
constexpr int kTcPitch = 132;                     // floats per column of the exchange buffer (128 tokens + 4)
constexpr int kTcSmem = kTcStages * (kTcXBytes + kTcABytes) + 1024;
static_assert(256 * kTcPitch * 4 <= kTcStages * (kTcXBytes + kTcABytes), "the exchange buffer takes the ring's place");

__device__ __forceinline__ void mma_bf16_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x as a sum of BF16 parts: each holds what the parts before it leave.  A finite x that would round
// to infinity (above 3.396e38) is cut instead; the next part takes the rest.
__device__ __forceinline__ void store_parts(uint16_t* dst, long long stride, int parts, float x) {
    for (int o = 0; o < parts; ++o) {
        uint32_t h = __bfloat16_as_ushort(__float2bfloat16(x));
        if ((h & 0x7fffu) == 0x7f80u && x - x == 0.0f) --h;      // the largest BF16
        dst[o * stride] = static_cast<uint16_t>(h);
        x -= __uint_as_float(h << 16);
        if (!(x == x)) x = 0.0f;       // an infinite or NaN part leaves nothing
    }
}

// What both ways know of the tile: its distinct adapters and each token's place among them.
struct TileShared {
    alignas(16) uint8_t marks[fg::kMaxListed];
    uint16_t list[fg::kMaxListed];
    int listed;
    int16_t slot_of[128];               // of each token of the tile, -1 without an adapter
    int count[128], first_item[129];    // tokens of each slot, work items before it
    int16_t member[128];                // tokens that use the item's adapter, in order
    float scale[128];                   // of each slot's adapter
};

// The few-tokens way: items first, first + stride, ...
template <int MB, int U>
__device__ __forceinline__ void shrink_items(const ShrinkParams& p, TileShared& sh,
                                             float (&red)[kShrinkWarps / 2][MB * 16][8], int tt, int n, int first_of_cta,
                                             int stride) {
    constexpr int kTok = 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slots = sh.listed;
    if (warp == 0) {                              // items of each slot, four slots a lane, and their prefix sums
        int c[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = (sh.count[4 * lane + i] + kTok - 1) / kTok;
            sum += c[i];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        int at = incl - sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sh.first_item[4 * lane + i] = at;
            at += c[i];
        }
        if (lane == 31) sh.first_item[128] = at;
    }
    __syncthreads();
    // an item's rank rows (rp, a power of two) in halves or quarters, as far as the CTAs go
    const int whole_items = sh.first_item[128];
    int parted = 0;
    while (p.rp >> parted > 16 * MB && whole_items << (parted + 1) <= stride) ++parted;
    const int rows = p.rp >> parted, items = whole_items << parted;
    const long long part = (long long)p.bn * p.rp;
    const int g = lane >> 2, q = lane & 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int i = first_of_cta; i < items; i += stride) {
        const int item = i >> parted, m_first = (i - (item << parted)) * rows, m_end = m_first + rows;
        int slot = 0;
        for (int lo = 0, hi = slots; lo < hi;) {      // the last slot whose first item is not behind `item`
            const int mid = (lo + hi) / 2;
            if (sh.first_item[mid] <= item) { slot = mid; lo = mid + 1; }
            else hi = mid;
        }
        const int first = (item - sh.first_item[slot]) * kTok, id = sh.list[slot];
        uint16_t* v = p.v + ((long long)tt * p.max_slots + slot) * p.parts * p.bn * p.rp;
        __syncthreads();                              // the item before is done with member
        if (warp == 0) {
            int members = 0;
            for (int t0 = 0; t0 < p.bn; t0 += 32) {
                const bool mine = t0 + lane < n && sh.slot_of[t0 + lane] == slot;
                const uint32_t m = __ballot_sync(0xffffffffu, mine);
                if (mine) sh.member[members + __popc(m & ((1u << lane) - 1))] = static_cast<int16_t>(t0 + lane);
                members += __popc(m);
            }
        } else if (first == 0 && m_first == 0) {
            // the other tokens' rows are zero: they are multiplied with this adapter's B too
            const int per = p.rp / 8;                 // 16-byte pieces of a row
            for (int i = threadIdx.x - 32; i < p.parts * p.bn * per; i += blockDim.x - 32) {
                const int t = i / per % p.bn;
                if (t >= n || sh.slot_of[t] != slot) *reinterpret_cast<uint4*>(v + (long long)i * 8) = zero;
            }
        }
        __syncthreads();
        const int mine = min(kTok, sh.count[slot] - first);
        const float scale = sh.scale[slot];
        // rows by their offset in 16-byte pieces from the tile's and the adapter's first, -1: none
        const uint4* xb = reinterpret_cast<const uint4*>(p.x + (long long)tt * p.bn * p.K) + q;
        const uint4* ab = reinterpret_cast<const uint4*>(p.lora_a + (long long)id * p.R * p.K) + q;
        const int xrow = g < mine ? sh.member[first + g] * (p.K / 8) : -1;
        const int blocks = p.K / 32;                  // 64 bytes of a row each: four lanes' 16
        for (int m0 = m_first; m0 < m_end; m0 += 16 * MB) {
            float acc[MB][4] = {};
            int arow[MB][2];
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = m0 + 16 * i + 8 * h + g;
                    arow[i][h] = r < p.R ? r * (p.K / 8) : -1;
                }
            for (int b0 = warp; b0 < blocks; b0 += kShrinkWarps * U) {
                uint4 a[U][MB][2], x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int b = b0 + u * kShrinkWarps;
                    const bool in = b < blocks;
#pragma unroll
                    for (int i = 0; i < MB; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) a[u][i][h] = in && arow[i][h] >= 0 ? __ldg(ab + arow[i][h] + b * 4) : zero;
                    x[u] = in && xrow >= 0 ? __ldg(xb + xrow + b * 4) : zero;
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < MB; ++i) {
                        mma_bf16_16x8x16(acc[i], a[u][i][0].x, a[u][i][1].x, a[u][i][0].y, a[u][i][1].y, x[u].x, x[u].y);
                        mma_bf16_16x8x16(acc[i], a[u][i][0].z, a[u][i][1].z, a[u][i][0].w, a[u][i][1].w, x[u].z, x[u].w);
                    }
            }
            // the upper eight warps' sums first, then the lower eight add theirs
#pragma unroll
            for (int pass = 1; pass >= 0; --pass) {
                if (warp / 8 == pass) {
#pragma unroll
                    for (int i = 0; i < MB; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            float& at = red[warp & 7][16 * i + g + 8 * (c >> 1)][2 * q + (c & 1)];
                            at = pass ? acc[i][c] : at + acc[i][c];
                        }
                }
                __syncthreads();
            }
            for (int o = threadIdx.x; o < MB * 16 * mine; o += blockDim.x) {
                const int r = o % (MB * 16), t = o / (MB * 16);
                float sum = red[0][r][t];
#pragma unroll
                for (int w = 1; w < kShrinkWarps / 2; ++w) sum += red[w][r][t];
                if (m0 + r < p.rp) store_parts(v + (long long)sh.member[first + t] * p.rp + m0 + r, part, p.parts, scale * sum);
            }
            __syncthreads();
        }
    }
}

// The many-tokens way: groups of up to 256 rank columns, one per cluster and round.
__device__ __forceinline__ void shrink_tcgen05(const ShrinkParams& p, const ShrinkMaps& maps, TileShared& sh, uint8_t* ring,
                                               uint64_t* bars, uint32_t* tmem_slot, int* abort_word, int tt) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slots = sh.listed;
    const int rank = static_cast<int>(fg::cluster_ctarank()), cluster = blockIdx.x / kShrinkCluster;
    const int clusters = gridDim.x / kShrinkCluster;
    const int per_group = 256 / p.rp, groups = (slots + per_group - 1) / per_group;
    const int nk = p.K / 64, k0 = rank * nk / kShrinkCluster, k1 = (rank + 1) * nk / kShrinkCluster;
    const uint32_t rbase = fg::smem_u32(ring), b0 = fg::smem_u32(bars);
    auto full_bar = [&](int s) { return b0 + 8u * s; };
    auto empty_bar = [&](int s) { return b0 + 8u * (kTcStages + s); };
    const uint32_t done_bar = b0 + 8u * (2 * kTcStages);
    volatile int* abort_flag = abort_word;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kTcStages; ++s) {
            fg::mbar_init(full_bar(s), 1);
            fg::mbar_init(empty_bar(s), 1);
        }
        fg::mbar_init(done_bar, 1);
        *abort_flag = 0;
        fg::fence_mbar_init();
        fg::tma_prefetch_map(&maps.x);
        fg::tma_prefetch_map(&maps.a);
    }
    if (warp == 1) {
        fg::tmem_alloc(fg::smem_u32(tmem_slot), 256);
        fg::tmem_relinquish();
    }
    fg::tc_fence_before();
    __syncthreads();
    fg::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const fg::WaitCtl wctl{abort_flag, p.status, p.timeout_ns};
    // four TMA producers (warps 0, 2, 3, 8; one thread's loads complete one after another), one per stage
    const int producer = warp == 0 ? 0 : (warp == 2 || warp == 3 ? warp - 1 : (warp == 8 ? 3 : -1));
    int s = 0, loads = 0;
    uint32_t ph = 0, done_ph = 0;
    int before = 0;                                   // chunks of the groups before: stage of chunk c is (before + c) mod 4
    for (int grp = cluster; grp < groups; grp += clusters) {
        const int slot0 = grp * per_group, cnt = min(per_group, slots - slot0), cols = cnt * p.rp;
        if (producer >= 0) {
            if (lane == 0 && !*abort_flag)
                for (int k = k0; k < k1; ++k) {
                    if (((before + k - k0) & (kTcStages - 1)) != producer) continue;
                    if (!fg::wait_bar(empty_bar(producer), (loads & 1) ^ 1, wctl, fg::kWaitProducer)) break;
                    const uint32_t dst = rbase + producer * (kTcXBytes + kTcABytes), fb = full_bar(producer);
                    fg::mbar_arrive_expect_tx(fb, kTcXBytes + cols * 128);
                    fg::tma_load_2d(dst, &maps.x, fb, k * 64, tt * p.bn);
                    for (int i = 0; i < cnt; ++i)
                        fg::tma_load_3d(dst + kTcXBytes + i * p.rp * 128, &maps.a, fb, k * 64, 0, sh.list[slot0 + i]);
                    ++loads;
                }
            __syncwarp();
        } else if (warp == 1) {
            const uint32_t idesc = fg::make_idesc_bf16(128, 0) | static_cast<uint32_t>(cols >> 3) << 17;
            bool ok = true;
            for (int k = k0; k < k1; ++k) {
                ok = __all_sync(0xffffffffu, fg::wait_bar(full_bar(s), ph, wctl, fg::kWaitMma)) != 0;
                if (!ok) break;
                fg::tc_fence_after();
                if (fg::elect_one()) {
                    const uint32_t at = rbase + s * (kTcXBytes + kTcABytes);
                    const uint64_t xd = fg::make_sdesc(at, 0, 1024, fg::kLayoutSw128);
                    const uint64_t ad = fg::make_sdesc(at + kTcXBytes, 0, 1024, fg::kLayoutSw128);
#pragma unroll
                    for (int j = 0; j < 4; ++j) fg::tc_mma_bf16(tmem, xd + 2 * j, ad + 2 * j, idesc, (k > k0 || j) ? 1u : 0u);
                    fg::tc_commit(empty_bar(s));
                }
                __syncwarp();
                if (++s == kTcStages) { s = 0; ph ^= 1u; }
            }
            // also on the way out: no product of this CTA is in flight behind this
            if (fg::elect_one()) fg::tc_commit(done_bar);
            __syncwarp();
        }
        before += k1 - k0;
        const bool ok = fg::wait_bar(done_bar, done_ph, wctl, fg::kWaitEpilogue);
        done_ph ^= 1u;
        (void)ok;                                     // on a time-out the sums are wrong, and reported
        fg::tc_fence_after();
        float* xch = reinterpret_cast<float*>(ring);  // [column][token], pitch kTcPitch
        if (warp >= 4 && warp < 8 && k1 > k0) {
            const int row = (warp & 3) * 32 + lane;
            for (int c0 = 0; c0 < cols; c0 += 16) {
                uint32_t r[16];
                fg::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0, r);
                fg::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) xch[(c0 + i) * kTcPitch + row] = __uint_as_float(r[i]);
            }
        }
        fg::tc_fence_before();
        __syncwarp();
        fg::cluster_sync();
        // four tokens at a time, rank's: thread = (column, four tokens), the partials in rank order
        const uint32_t xbase = fg::smem_u32(xch);
        const long long part = (long long)p.bn * p.rp;
        for (int o = threadIdx.x; o < cols * ((31 - rank) / kShrinkCluster + 1); o += blockDim.x) {
            const int col = o % cols, t0 = (rank + o / cols * kShrinkCluster) * 4;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float4 x[kShrinkCluster];
#pragma unroll
            for (int r = 0; r < kShrinkCluster; ++r)
                x[r] = r * nk / kShrinkCluster < (r + 1) * nk / kShrinkCluster
                           ? fg::ld_dsmem_f32x4(fg::map_shared_rank(xbase + (col * kTcPitch + t0) * 4, r))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < kShrinkCluster; ++r) {
                sum.x += x[r].x; sum.y += x[r].y; sum.z += x[r].z; sum.w += x[r].w;
            }
            const int i = col / p.rp, rr = col - i * p.rp, slot = slot0 + i;
            const float scale = sh.scale[slot];
            const float val[4] = {sum.x, sum.y, sum.z, sum.w};
            uint16_t* v = p.v + ((long long)tt * p.max_slots + slot) * p.parts * part + rr;
#pragma unroll
            for (int t = 0; t < 4; ++t)               // another adapter's tokens are zero rows
                store_parts(v + (long long)(t0 + t) * p.rp, part, p.parts, sh.slot_of[t0 + t] == slot ? scale * val[t] : 0.0f);
        }
        fg::fence_proxy_async_smem();                 // the ring is TMA's again
        __syncwarp();
        fg::cluster_sync();
    }
    if (producer >= 0 && lane == 0 && *abort_flag && loads > 0)
        fg::drain_bar(full_bar(producer), (loads - 1) & 1, 20000000ull);
    __syncthreads();
    if (warp == 1) {
        fg::tc_fence_after();
        fg::tmem_dealloc(tmem, 256);
    }
}

template <int MB, int U, bool kClusters>
__global__ void __launch_bounds__(32 * kShrinkWarps) lora_shrink_kernel(const ShrinkParams p, const __grid_constant__ ShrinkMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ TileShared sh;
    __shared__ float red[kShrinkWarps / 2][MB * 16][8];
    __shared__ uint64_t bars[2 * kTcStages + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    const int tt = blockIdx.y;
    const int n = min(p.bn, p.tokens - tt * p.bn);
    const int32_t* ids = p.ids + (long long)tt * p.bn;
    if (threadIdx.x < 128) sh.count[threadIdx.x] = 0;
    fg::clear_marks(sh.marks);
    fg::grid_dependency_wait();
    if (threadIdx.x == 0) fg::grid_launch_dependents();
    const int my_id = fg::load_id(ids, n);
    __syncthreads();
    fg::mark_ids(ids, n, my_id, 0, p.L, sh.marks);
    if (threadIdx.x < 32) {
        const int found = fg::list_marked(sh.marks, sh.list);
        if (threadIdx.x == 0) sh.listed = found;
    }
    __syncthreads();
    const int slots = sh.listed;
    if (threadIdx.x < 128) {
        int slot = -1;
        if (my_id >= 0 && my_id < p.L)            // its rank in the list
            for (int lo = 0, hi = slots; lo < hi;) {
                const int mid = (lo + hi) / 2;
                if (sh.list[mid] <= my_id) { slot = mid; lo = mid + 1; }
                else hi = mid;
            }
        sh.slot_of[threadIdx.x] = static_cast<int16_t>(slot);
        if (slot >= 0) atomicAdd(sh.count + slot, 1);
        if (static_cast<int>(threadIdx.x) < slots) sh.scale[threadIdx.x] = __ldg(p.scaling + sh.list[threadIdx.x]);
    }
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < slots; i += blockDim.x) p.slot_ids[tt * p.max_slots + i] = sh.list[i];
        if (threadIdx.x == 0) p.slot_count[tt] = slots;
        if (my_id >= p.L) fg::record_status(p.status, fg::kErrContract | fg::kChkAdapter);
    }
    __syncthreads();
    if (kClusters && n >= 8 * slots) {
        uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
        shrink_tcgen05(p, maps, sh, ring, bars, &tmem_slot, &abort_word, tt);
    } else {
        shrink_items<MB, U>(p, sh, red, tt, n, blockIdx.x, gridDim.x);
    }
    fg::fence_proxy_async_global();
}

template <int MB, int U, bool kClusters>
cudaError_t launch_shrink_as(const ShrinkParams& p, const ShrinkMaps& maps, dim3 grid, int pdl, cudaStream_t stream) {
    static bool configured[256] = {};        // set once per device; setting it again is harmless
    const int smem = kClusters ? kTcSmem : 0;
    if (kClusters) {
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        if (dev < 0 || dev >= 256) return cudaErrorInvalidDevice;
        if (!configured[dev]) {
            err = cudaFuncSetAttribute(lora_shrink_kernel<MB, U, kClusters>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (err != cudaSuccess) return err;
            configured[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kShrinkWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (kClusters) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = kShrinkCluster;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, lora_shrink_kernel<MB, U, kClusters>, p, maps);
}

// sms: how many the launch may take.
cudaError_t launch_shrink(const ShrinkParams& p, const ShrinkMaps& maps, int tiles, int sms, int pdl, cudaStream_t stream) {
    if (tiles > 1) {                              // whole clusters per tile, as far as one wave of SMs goes
        const int clusters = sms / (kShrinkCluster * tiles) > 1 ? sms / (kShrinkCluster * tiles) : 1;
        const dim3 grid(static_cast<unsigned>(clusters * kShrinkCluster), static_cast<unsigned>(tiles));
        return p.rp <= 16 ? launch_shrink_as<1, 8, true>(p, maps, grid, pdl, stream)
                          : launch_shrink_as<2, 4, true>(p, maps, grid, pdl, stream);
    }
    // one CTA an item, of which there are at most min(bn, L) + bn / 8 per block of rank rows
    const int most = ((p.L < p.bn ? p.L : p.bn) + p.bn / 8) * ceil_div(p.rp, p.rp <= 16 ? 16 : 32);
    const dim3 grid(static_cast<unsigned>(most < sms ? most : sms));
    return p.rp <= 16 ? launch_shrink_as<1, 8, false>(p, maps, grid, pdl, stream)
                      : launch_shrink_as<2, 4, false>(p, maps, grid, pdl, stream);
}

}  // namespace

extern "C" {

long long fg_lora_workspace(int M, int N, int K, int R) {
    return fg_lora_workspace_for(M, N, K, fg::kMaxListed, R, FG_F32);
}

long long fg_lora_workspace_for(int M, int N, int K, int L, int R, int d_dtype) {
    if (!shapes_ok(M, N, K, R) || L < 1 || L > fg::kMaxListed || (d_dtype != FG_BF16 && d_dtype != FG_F32)) return -1;
    return layout(M > 0 ? M : 1, R, L, d_dtype).bytes;
}

int fg_fp8_gemm_nt_lora(int M, int N, int K, int L, int R, const uint8_t* a, const int32_t* sfa, const uint8_t* b,
                        const int32_t* sfb, const void* x, const void* lora_a, const void* lora_b,
                        const float* scaling, const int32_t* ids, void* d, int d_dtype, void* workspace,
                        fg_stream_t stream) {
    if (!shapes_ok(M, N, K, R) || L < 1 || (d_dtype != FG_BF16 && d_dtype != FG_F32)) return FG_ERR_INVALID_ARG;
    if (L > fg::kMaxListed) return FG_ERR_UNSUPPORTED;
    if (M == 0) return FG_OK;
    if (!a || !sfa || !b || !sfb || !x || !lora_a || !lora_b || !scaling || !ids || !d || !workspace || !al(a, 16) ||
        !al(sfa, 16) || !al(b, 16) || !al(sfb, 16) || !al(x, 16) || !al(lora_a, 16) || !al(lora_b, 16) ||
        !al(scaling, 4) || !al(ids, 4) || !al(d, 16) || !al(workspace, 256))
        return FG_ERR_INVALID_ARG;
    fg::HostState st;
    if (const int rc = fg::host_state(&st)) return rc;
    const Layout l = layout(M, R, L, d_dtype);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int grid = st.sms < fg::kMaxStreamCtas ? st.sms : fg::kMaxStreamCtas;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    // an adapter unit's parts x columns fit the stage's token area
    const int parts = l.parts, unit_cols = parts == 3 ? 16 : 32;
    if (fg::print_configs_enabled())
        std::fprintf(stderr, "[fg] fp8_gemm_nt_lora M=%d N=%d K=%d L=%d R=%d BN=%d rank=%d grid=%d\n", M, N, K, L, R, l.bn,
                     l.rp, grid);
    const ShrinkParams sp{M, l.bn, K, R, l.rp, L, l.slots, parts, ids, static_cast<const uint16_t*>(x),
                          static_cast<const uint16_t*>(lora_a), scaling, reinterpret_cast<uint16_t*>(ws + l.v),
                          reinterpret_cast<int*>(ws + l.ids), reinterpret_cast<int*>(ws + l.count), st.status, st.timeout_ns};
    ShrinkMaps sm;
    std::memset(&sm, 0, sizeof(sm));
    if (l.tiles > 1) {
        const uint64_t xd[2] = {(uint64_t)K, (uint64_t)M}, xp[1] = {(uint64_t)K * 2};
        const uint64_t ad[3] = {(uint64_t)K, (uint64_t)R, (uint64_t)L}, ap[2] = {(uint64_t)K * 2, (uint64_t)K * 2 * R};
        const uint32_t xb[2] = {64, 128}, ab[3] = {64, (uint32_t)l.rp, 1};
        if (!fg::encode_tiled(&sm.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, xd, xp, xb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !fg::encode_tiled(&sm.a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, lora_a, ad, ap, ab, CU_TENSOR_MAP_SWIZZLE_128B))
            return FG_ERR_INVALID_ARG;
    }
    // Where a tile's pieces find SMs, the projection runs in clusters that start beside this launch,
    // stream the FP8 weights meanwhile and join the pieces: this launch leaves them their SMs, they
    // leave it 40.  Measured on GB300, one token tile: 64 x 7168 x 4096, 52 adapters 21.0 us with 4 CTAs a
    // cluster and 40 SMs here, 22.4 with 72 here (some clusters start late), 25.0 without clusters; 64 x
    // 4096 16.4 with 6, 23.0 without.  Several: 275 x 464 x 2304, rank 8 16.0 with 8, 22.1 in whole
    // tiles, 54.6 in equal shares; 221 x 1984 x 2432, one adapter 17.8 with 7, 24.2, 40.4; 180 x 544 x
    // 640, 113 adapters of rank 128 47 with 8, 177, 94.
    const int row_tiles = ceil_div(N, 256);
    const int cluster = fg::stream_cluster<fg::kProj, false>(l.bn, row_tiles * l.tiles, grid - 40);
    const int beside = cluster > 1 ? cluster * row_tiles * l.tiles : 0;
    if (launch_shrink(sp, sm, l.tiles, beside ? grid - beside : st.sms, st.pdl, s) != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    fg::StreamParams p{};
    p.tokens = M;
    p.ids = ids;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.lora_rp = l.rp; p.lora_count = L;
    p.max_slots = l.slots; p.token_tiles = l.tiles;
    p.parts = parts; p.unit_cols = unit_cols;
    p.slot_ids = sp.slot_ids;
    p.slot_count = sp.slot_count;
    p.status = st.status; p.timeout_ns = st.timeout_ns; p.pdl = st.pdl;
    fg::StreamMaps m;
    std::memset(&m, 0, sizeof(m));
    {   // the projection and the adapters' B
        const uint64_t wd[3] = {(uint64_t)K, (uint64_t)N, 1}, wp[2] = {(uint64_t)K, (uint64_t)K * N};
        const uint32_t wb[3] = {128, 256, 1};
        const uint64_t xd[2] = {(uint64_t)K, (uint64_t)M}, xp[1] = {(uint64_t)K};
        const uint32_t xb[2] = {128, (uint32_t)l.bn};
        const uint32_t cols = l.rp < p.unit_cols ? l.rp : p.unit_cols;
        const CUtensorMapSwizzle sw = cols == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B;
        const uint64_t ld[3] = {(uint64_t)R, (uint64_t)N, (uint64_t)L}, lp[2] = {(uint64_t)R * 2, (uint64_t)R * 2 * N};
        const uint32_t lb[3] = {cols, 256, 1};
        const uint64_t vd[2] = {(uint64_t)l.rp, (uint64_t)l.tiles * l.slots * parts * l.bn}, vp[1] = {(uint64_t)l.rp * 2};
        const int v_rows = (unit_cols / l.rp > 1 ? unit_cols / l.rp : 1) * parts * l.bn;   // of a unit
        const uint32_t vb[2] = {cols, (uint32_t)(v_rows <= 256 ? v_rows : v_rows / 2)};
        if (!fg::encode_tiled(&m.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, b, wd, wp, wb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !fg::encode_tiled(&m.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a, xd, xp, xb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !fg::encode_tiled(&m.lb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, lora_b, ld, lp, lb, sw) ||
            !fg::encode_tiled(&m.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, sp.v, vd, vp, vb, sw))
            return FG_ERR_INVALID_ARG;
        p.nk = K / 128; p.row_tiles = row_tiles; p.out_rows = N;
        p.sfw = sfb;
        p.sfw_rows = ceil_div(N, 128);
        p.sfw_ld = align4(p.sfw_rows);
        p.sft = sfa; p.sft_ld = align4(M);
        p.ctr = reinterpret_cast<unsigned*>(ws) + fg::kMaxCounters;
        p.d = d; p.d_f32 = d_dtype == FG_F32;
        p.debug_stall = st.debug_stall;
        p.w_raw = b; p.x_raw = a;
        p.lb_raw = static_cast<const uint16_t*>(lora_b); p.v_raw = sp.v;
        p.lora_r = R;
        p.cluster = cluster;
        const dim3 ctas(p.cluster > 1 ? p.cluster * p.row_tiles * l.tiles : grid);
        if (fg::launch_stream<fg::kProj, false>(l.bn, p, m, ctas, s) != cudaSuccess) {
            cudaGetLastError();
            return FG_ERR_CUDA;
        }
    }
    return FG_OK;
}

}  // extern "C"
