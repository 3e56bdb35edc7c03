// fg_lora.cu - an FP8 projection shared by all tokens plus each token's own low-rank adapter,
// in two launches (fg_stream.cuh): x times the adapters' A, then the projection's K-groups and
// the adapters' B in one accumulator.
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
    const long long ctas = l.tiles > fg::kMaxStreamCtas ? l.tiles : fg::kMaxStreamCtas;
    l.bytes = l.part + ctas * 2 * 2 * l.bn * 128 * 4;
    return l;
}

bool shapes_ok(int M, int N, int K, int R) {
    if (M < 0 || N < 16 || N % 16 != 0 || K < 128 || K % 128 != 0 || R < 8 || R % 8 != 0 || R > 128) return false;
    const Layout l = layout(M > 0 ? M : 1, R);
    return l.tiles <= fg::kMaxTokenTiles &&
           (long long)l.tiles * ceil_div(N, 256) * (K / 128 + 4 * l.bn) < (1LL << 31) &&
           (long long)l.tiles * l.bn * 3 * l.bn < (1LL << 31);
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

    fg::StreamParams p{};
    p.tokens = M;
    p.ids = ids;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.lora_r = R; p.lora_rp = l.rp; p.lora_k = K; p.lora_count = L;
    p.max_slots = l.bn; p.token_tiles = l.tiles;
    // parts of x @ lora_a^T: 16 mantissa bits under a BF16 result, 24 under an FP32 one
    p.parts = d_dtype == FG_F32 ? 3 : 2;
    p.unit_cols = d_dtype == FG_F32 ? 32 : 64;        // parts x columns fit the stage's token area
    p.lora_a = static_cast<const uint16_t*>(lora_a);
    p.scaling = scaling;
    p.v = reinterpret_cast<uint16_t*>(ws + l.v);
    p.slot_ids = reinterpret_cast<int*>(ws + l.ids);
    p.slot_count = reinterpret_cast<int*>(ws + l.count);
    p.min_units = 4;
    p.status = st.status; p.timeout_ns = st.timeout_ns; p.pdl = st.pdl;
    fg::StreamMaps m;
    std::memset(&m, 0, sizeof(m));
    if (fg::print_configs_enabled())
        std::fprintf(stderr, "[fg] fp8_gemm_nt_lora M=%d N=%d K=%d L=%d R=%d BN=%d rank=%d grid=%d\n", M, N, K, L, R, l.bn,
                     l.rp, grid);
    {   // x times the distinct adapters' A, token tile by token tile
        const uint64_t xd[2] = {(uint64_t)K, (uint64_t)M}, xp[1] = {(uint64_t)K * 2};
        const uint32_t xb[2] = {64, (uint32_t)l.bn};
        if (!fg::encode_tiled(&m.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, xd, xp, xb, CU_TENSOR_MAP_SWIZZLE_128B))
            return FG_ERR_INVALID_ARG;
        p.nk = K / 64;
        p.ctr = reinterpret_cast<unsigned*>(ws);
        const int per_tile = grid / l.tiles > 0 ? grid / l.tiles : 1;
        if (fg::launch_stream<fg::kShrink, false>(l.bn, p, m, dim3(per_tile, l.tiles), s) != cudaSuccess) {
            cudaGetLastError();
            return FG_ERR_CUDA;
        }
    }
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
            !fg::encode_tiled(&m.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.v, vd, vp, vb, sw))
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
