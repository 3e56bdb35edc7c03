// fg_lora.cu - an FP8 projection shared by all tokens plus each token's own low-rank adapter,
// in two launches: v = scaling * x @ A^T per token and adapter (here), then the projection's
// K-groups and the adapters' B against v in one accumulator (fg_stream.cuh).
#include <cuda_bf16.h>

#include <cstdio>
#include <cstring>

#include "fg.h"
#include "fg_host.h"
#include "fg_stream.cuh"

namespace {

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int align4(int x) { return (x + 3) / 4 * 4; }
int ceil_div(int a, int b) { return (a + b - 1) / b; }
long long up256(long long x) { return (x + 255) / 256 * 256; }

// Rank columns as the tensor core takes them: 16 per step, whole or half adapters per unit.
int padded_rank(int r) { return r <= 16 ? 16 : (r <= 32 ? 32 : (r <= 64 ? 64 : 128)); }

struct Layout {
    int bn, rp, tiles;                    // token columns, padded rank, token tiles
    long long ids, count, v, part, bytes; // behind the counters (fg_stream.cuh)
};
Layout layout(int M, int R) {
    Layout l;
    l.bn = fg::stream_bn(M);
    l.rp = padded_rank(R);
    l.tiles = ceil_div(M, l.bn);
    l.ids = fg::kCounterBytes;
    l.count = l.ids + up256((long long)l.tiles * l.bn * 4);
    l.v = l.count + up256((long long)l.tiles * 4);
    l.part = l.v + up256((long long)l.tiles * l.bn * 3 * l.bn * l.rp * 2);
    l.bytes = l.part + (long long)fg::kMaxStreamCtas * 2 * 2 * l.bn * 128 * 4;
    return l;
}

bool shapes_ok(int M, int N, int K, int R) {
    if (M < 0 || N < 16 || N % 16 != 0 || K < 128 || K % 128 != 0 || R < 8 || R % 8 != 0 || R > 128) return false;
    const Layout l = layout(M > 0 ? M : 1, R);
    return l.tiles <= fg::kMaxTokenTiles &&
           (long long)l.tiles * ceil_div(N, 256) * (K / 128 + 8 * l.bn) < (1LL << 31) &&
           (long long)l.tiles * l.bn * 3 * l.bn < (1LL << 31);
}

// ---------------------------------------------------------------- v = scaling * x @ A^T
// A work item is (distinct adapter of a token tile, 8 * NB of the tokens that use it); a token
// tile's CTAs share its items.  The adapter's rows are the M operand of mma.sync (MB blocks of
// 16), its tokens the N operand (NB blocks of 8), gathered by their row numbers.  The 16 warps split K and read both operands
// straight into registers, 16 bytes (8 consecutive k) per row and lane: k is summed over, so a
// lane's 8 values may stand for any k as long as A and x agree; they feed two 16-wide steps.
// There is nothing to stage: each A element is used by one CTA (latency-bound: its bytes in
// flight are what counts, U blocks of 32 k per warp), and tcgen05's 128 rows would be mostly
// empty.  The partial sums meet in shared memory, in warp order.
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
};

constexpr int kShrinkWarps = 16;

__device__ __forceinline__ void mma_bf16_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x as a sum of BF16 parts: each holds what the parts before it leave.
__device__ __forceinline__ void store_parts(uint16_t* dst, long long stride, int parts, float x) {
    for (int o = 0; o < parts; ++o) {
        const __nv_bfloat16 h = __float2bfloat16(x);
        dst[o * stride] = __bfloat16_as_ushort(h);
        x -= __bfloat162float(h);
        if (!(x == x)) x = 0.0f;       // an infinite or NaN part leaves nothing
    }
}

template <int MB, int NB, int U>
__global__ void __launch_bounds__(32 * kShrinkWarps) lora_shrink_kernel(const ShrinkParams p) {
    constexpr int kTok = 8 * NB;
    __shared__ uint32_t bits[32];
    __shared__ uint16_t list[fg::kMaxListed];
    __shared__ int listed;
    __shared__ int16_t slot_of[128];              // of each token of the tile, -1 without an adapter
    __shared__ int count[128], first_item[129];   // tokens of each slot, items before it
    __shared__ int16_t member[128];               // tokens that use the item's adapter, in order
    __shared__ float red[kShrinkWarps / 2][MB * 16][kTok];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tt = blockIdx.y;
    fg::grid_dependency_wait();
    if (threadIdx.x == 0) fg::grid_launch_dependents();
    const int n = min(p.bn, p.tokens - tt * p.bn);
    const int32_t* ids = p.ids + (long long)tt * p.bn;
    const int my_id = threadIdx.x < static_cast<unsigned>(n) ? __ldcg(ids + threadIdx.x) : -1;
    if (threadIdx.x < 128) count[threadIdx.x] = 0;
    fg::list_distinct(ids, n, 0, p.L, bits, list, &listed);
    const int slots = listed;
    if (threadIdx.x < 128) {
        int slot = -1;
        if (my_id >= 0 && my_id < p.L)            // its rank in the list
            for (int lo = 0, hi = slots; lo < hi;) {
                const int mid = (lo + hi) / 2;
                if (list[mid] <= my_id) { slot = mid; lo = mid + 1; }
                else hi = mid;
            }
        slot_of[threadIdx.x] = static_cast<int16_t>(slot);
        if (slot >= 0) atomicAdd(count + slot, 1);
    }
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < slots; i += blockDim.x) p.slot_ids[tt * p.max_slots + i] = list[i];
        if (threadIdx.x == 0) p.slot_count[tt] = slots;
        if (my_id >= p.L) fg::record_status(p.status, fg::kErrContract | fg::kChkAdapter);
    }
    __syncthreads();
    if (warp == 0) {                              // items of each slot, four slots a lane, and their prefix sums
        int c[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = (count[4 * lane + i] + kTok - 1) / kTok;
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
            first_item[4 * lane + i] = at;
            at += c[i];
        }
        if (lane == 31) first_item[128] = at;
    }
    __syncthreads();
    const int items = first_item[128];
    const long long part = (long long)p.bn * p.rp;
    const int g = lane >> 2, q = lane & 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int slot = 0;
    for (int lo = 0, hi = slots; lo < hi;) {      // the last slot whose first item is not behind `item`
        const int mid = (lo + hi) / 2;
        if (first_item[mid] <= item) { slot = mid; lo = mid + 1; }
        else hi = mid;
    }
    const int first = (item - first_item[slot]) * kTok, id = list[slot];
    uint16_t* v = p.v + ((long long)tt * p.max_slots + slot) * p.parts * p.bn * p.rp;
    __syncthreads();                              // the item before is done with member
    if (warp == 0) {
        int members = 0;
        for (int t0 = 0; t0 < p.bn; t0 += 32) {
            const bool mine = t0 + lane < n && slot_of[t0 + lane] == slot;
            const uint32_t m = __ballot_sync(0xffffffffu, mine);
            if (mine) member[members + __popc(m & ((1u << lane) - 1))] = static_cast<int16_t>(t0 + lane);
            members += __popc(m);
        }
    } else {
        // the other tokens' rows are zero: they are multiplied with this adapter's B too
        if (first == 0) {
            const int per = p.rp / 8;             // 16-byte pieces of a row
            for (int i = threadIdx.x - 32; i < p.parts * p.bn * per; i += blockDim.x - 32) {
                const int row = i / per, t = row % p.bn;
                if (t >= n || slot_of[t] != slot) *reinterpret_cast<uint4*>(v + (long long)i * 8) = zero;
            }
        }
    }
    __syncthreads();
    const int mine = min(kTok, count[slot] - first);
    const float scale = __ldg(p.scaling + id);
    // rows by their offset in 16-byte pieces from the tile's and the adapter's first, -1: none
    const uint4* xb = reinterpret_cast<const uint4*>(p.x + (long long)tt * p.bn * p.K) + q;
    const uint4* ab = reinterpret_cast<const uint4*>(p.lora_a + (long long)id * p.R * p.K) + q;
    int xrow[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) xrow[j] = 8 * j + g < mine ? member[first + 8 * j + g] * (p.K / 8) : -1;
    const int blocks = p.K / 32;                   // 64 bytes of a row each: four lanes' 16
    for (int m0 = 0; m0 < p.rp; m0 += 16 * MB) {
        float acc[MB][NB][4] = {};
        int arow[MB][2];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = m0 + 16 * i + 8 * h + g;
                arow[i][h] = r < p.R ? r * (p.K / 8) : -1;
            }
        for (int b0 = warp; b0 < blocks; b0 += kShrinkWarps * U) {
            uint4 a[U][MB][2], x[U][NB];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = b0 + u * kShrinkWarps;
                const bool in = b < blocks;
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) a[u][i][h] = in && arow[i][h] >= 0 ? __ldg(ab + arow[i][h] + b * 4) : zero;
#pragma unroll
                for (int j = 0; j < NB; ++j) x[u][j] = in && xrow[j] >= 0 ? __ldg(xb + xrow[j] + b * 4) : zero;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        mma_bf16_16x8x16(acc[i][j], a[u][i][0].x, a[u][i][1].x, a[u][i][0].y, a[u][i][1].y, x[u][j].x, x[u][j].y);
                        mma_bf16_16x8x16(acc[i][j], a[u][i][0].z, a[u][i][1].z, a[u][i][0].w, a[u][i][1].w, x[u][j].z, x[u][j].w);
                    }
        }
        // the upper eight warps' sums first, then the lower eight add theirs
#pragma unroll
        for (int pass = 1; pass >= 0; --pass) {
            if (warp / 8 == pass) {
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            float& at = red[warp & 7][16 * i + g + 8 * (c >> 1)][8 * j + 2 * q + (c & 1)];
                            at = pass ? acc[i][j][c] : at + acc[i][j][c];
                        }
            }
            __syncthreads();
        }
        for (int o = threadIdx.x; o < MB * 16 * mine; o += blockDim.x) {
            const int r = o % (MB * 16), t = o / (MB * 16);
            float sum = red[0][r][t];
#pragma unroll
            for (int w = 1; w < kShrinkWarps / 2; ++w) sum += red[w][r][t];
            if (m0 + r < p.rp) store_parts(v + (long long)member[first + t] * p.rp + m0 + r, part, p.parts, scale * sum);
        }
        __syncthreads();
    }
    }
    fg::fence_proxy_async_global();
}

cudaError_t launch_shrink(const ShrinkParams& p, int tiles, int sms, int pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.blockDim = dim3(32 * kShrinkWarps);
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    auto go = [&](auto kernel, int tok) {
        // a tile has at most min(bn, L) + bn / tok items; one CTA an item, as far as one wave of SMs goes
        const int most = (p.L < p.bn ? p.L : p.bn) + p.bn / tok;
        const int share = sms / tiles > 1 ? sms / tiles : 1;
        cfg.gridDim = dim3(static_cast<unsigned>(most < share ? most : share), static_cast<unsigned>(tiles));
        return cudaLaunchKernelEx(&cfg, kernel, p);
    };
    // 8 tokens at a time where there are few per adapter (small tiles), 32 in a prompt's tiles
    if (p.bn <= 64)
        return p.rp <= 16 ? go(lora_shrink_kernel<1, 1, 8>, 8) : go(lora_shrink_kernel<2, 1, 4>, 8);
    return p.rp <= 16 ? go(lora_shrink_kernel<1, 4, 2>, 32) : go(lora_shrink_kernel<2, 4, 2>, 32);
}

}  // namespace

extern "C" {

long long fg_lora_workspace(int M, int N, int K, int R) {
    if (!shapes_ok(M, N, K, R)) return -1;
    return layout(M > 0 ? M : 1, R).bytes;
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
    const Layout l = layout(M, R);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int grid = st.sms < fg::kMaxStreamCtas ? st.sms : fg::kMaxStreamCtas;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    // parts of x @ lora_a^T: 16 mantissa bits under a BF16 result, 24 under an FP32 one; an adapter
    // unit's parts x columns fit the stage's token area
    const int parts = d_dtype == FG_F32 ? 3 : 2, unit_cols = d_dtype == FG_F32 ? 16 : 32;
    if (fg::print_configs_enabled())
        std::fprintf(stderr, "[fg] fp8_gemm_nt_lora M=%d N=%d K=%d L=%d R=%d BN=%d rank=%d grid=%d\n", M, N, K, L, R, l.bn,
                     l.rp, grid);
    const ShrinkParams sp{M, l.bn, K, R, l.rp, L, l.bn, parts, ids, static_cast<const uint16_t*>(x),
                          static_cast<const uint16_t*>(lora_a), scaling, reinterpret_cast<uint16_t*>(ws + l.v),
                          reinterpret_cast<int*>(ws + l.ids), reinterpret_cast<int*>(ws + l.count), st.status};
    if (launch_shrink(sp, l.tiles, st.sms, st.pdl, s) != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    fg::StreamParams p{};
    p.tokens = M;
    p.ids = ids;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.lora_rp = l.rp; p.lora_count = L;
    p.max_slots = l.bn; p.token_tiles = l.tiles;
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
        const CUtensorMapSwizzle sw = cols == 16 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                 : (cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
        const uint64_t ld[3] = {(uint64_t)R, (uint64_t)N, (uint64_t)L}, lp[2] = {(uint64_t)R * 2, (uint64_t)R * 2 * N};
        const uint32_t lb[3] = {cols, 256, 1};
        const uint64_t vd[2] = {(uint64_t)l.rp, (uint64_t)l.tiles * l.bn * p.parts * l.bn}, vp[1] = {(uint64_t)l.rp * 2};
        const uint32_t vb[2] = {cols, (uint32_t)l.bn};
        if (!fg::encode_tiled(&m.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, b, wd, wp, wb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !fg::encode_tiled(&m.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a, xd, xp, xb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !fg::encode_tiled(&m.lb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, lora_b, ld, lp, lb, sw) ||
            !fg::encode_tiled(&m.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, sp.v, vd, vp, vb, sw))
            return FG_ERR_INVALID_ARG;
        p.nk = K / 128; p.row_tiles = ceil_div(N, 256); p.out_rows = N;
        p.sfw = sfb;
        p.sfw_rows = ceil_div(N, 128);
        p.sfw_ld = align4(p.sfw_rows);
        p.sft = sfa; p.sft_ld = align4(M);
        p.ctr = reinterpret_cast<unsigned*>(ws) + fg::kMaxCounters;
        p.d = d; p.d_f32 = d_dtype == FG_F32;
        p.debug_stall = st.debug_stall;
        if (fg::launch_stream<fg::kProj, false>(l.bn, p, m, dim3(grid), s) != cudaSuccess) {
            cudaGetLastError();
            return FG_ERR_CUDA;
        }
    }
    return FG_OK;
}

}  // extern "C"
