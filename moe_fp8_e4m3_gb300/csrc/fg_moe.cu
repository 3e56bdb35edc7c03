// fg_moe.cu - the whole MoE MLP of a decode step in two launches (fg_stream.cuh): gate-up +
// SwiGLU + requantisation, then the down projection summed over the experts (from 33 tokens on a
// third one adds up its parts).  Two, because every down product needs the scale of 128 gate-up
// outputs and the sum of all experts: between them lies a wait for the whole grid, which the second
// launch's CTAs spend with their first weight tiles on the way.
#include <climits>
#include <cstdio>
#include <cstring>

#include "fg.h"
#include "fg_host.h"
#include "fg_stream.cuh"

namespace {

constexpr int kMaxTokens = 128, kMaxTopk = 32;

using fg::al;
using fg::align4;
using fg::up256;

// Workspace: the counters (zero between calls; at the same place for every size, so that a
// workspace can serve calls of several), then what the first launch leaves for the second (codes
// and scales of every listed expert's activations), then the partial tiles.
struct Layout {
    long long sfh, hq, part, bytes;
};
Layout layout(int T, int I, int E) {
    const long long bn = fg::stream_bn(T);
    const long long slots = (long long)T * kMaxTopk < E ? (long long)T * kMaxTopk : E;
    Layout l;
    l.sfh = fg::kCounterBytes;
    l.hq = l.sfh + up256(slots * ((I + 511) / 512) * bn * 4);
    l.part = l.hq + up256(slots * bn * I);
    l.bytes = l.part + (long long)fg::kMaxStreamCtas * 2 * 2 * bn * 128 * 4;
    return l;
}

bool shapes_ok(int T, int H, int I, int E) {
    return T >= 0 && H >= 128 && H % 128 == 0 && I >= 128 && I % 128 == 0 && E >= 1 &&
           (long long)E * (I / 128) * (H / 128) < (1LL << 31) && (long long)E * 2 * I < (1LL << 31) &&
           (long long)E * fg::kMaxListed < (1LL << 31);
}

template <bool kFp4>
int moe_mlp(int T, int H, int I, int E, int topk, int expert_base, const uint8_t* a, const int32_t* sfa,
            const uint8_t* w13, const int32_t* sf13, const uint8_t* w2, const int32_t* sf2, const int32_t* ids,
            const float* weights, void* d, int d_dtype, void* workspace, fg_stream_t stream) {
    if (!shapes_ok(T, H, I, E) || topk < 1 || expert_base < 0 || expert_base > INT_MAX - E || (d_dtype != FG_BF16 && d_dtype != FG_F32))
        return FG_ERR_INVALID_ARG;
    if (T > kMaxTokens || E > fg::kMaxListed || topk > kMaxTopk) return FG_ERR_UNSUPPORTED;
    if (T == 0) return FG_OK;
    const uintptr_t wa = kFp4 ? 32 : 16;
    if (!a || !sfa || !w13 || !sf13 || !w2 || !sf2 || !ids || !weights || !d || !workspace || !al(a, 16) || !al(sfa, 16) ||
        !al(w13, wa) || !al(w2, wa) || !al(sf13, 16) || !al(sf2, 16) || !al(ids, 4) || !al(weights, 4) || !al(d, 16) ||
        !al(workspace, 256))
        return FG_ERR_INVALID_ARG;
    fg::HostState st;
    if (const int rc = fg::host_state(&st)) return rc;
    const int bn = fg::stream_bn(T);
    const Layout l = layout(T, I, E);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const long long slots = (long long)T * topk < E ? (long long)T * topk : E;
    const int grid = st.sms < fg::kMaxStreamCtas ? st.sms : fg::kMaxStreamCtas;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const CUtensorMapDataType wtype = kFp4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8;

    fg::StreamParams p{};
    p.tokens = T;
    p.experts = E; p.expert_base = expert_base; p.topk = topk;
    p.ids = ids; p.weights = weights;
    p.cluster = 1;
    p.hq = ws + l.hq; p.sfh = ws + l.sfh;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.status = st.status; p.timeout_ns = st.timeout_ns; p.pdl = st.pdl; p.debug_stall = st.debug_stall;
    fg::StreamMaps m;
    std::memset(&m, 0, sizeof(m));
    if (fg::print_configs_enabled())
        std::fprintf(stderr, "[fg] moe_mlp%s T=%d H=%d I=%d E=%d topk=%d BN=%d grid=%d\n", kFp4 ? "_fp4" : "", T, H, I, E,
                     topk, bn, grid);
    {   // gate-up: weights seen as [2E halves][I][H], a box = 128 gate rows and their up rows
        const uint64_t row = kFp4 ? H / 2 : H;
        const uint64_t wd[3] = {(uint64_t)H, (uint64_t)I, 2ull * E}, wp[2] = {row, row * I};
        const uint32_t wb[3] = {128, 128, 2};
        const uint64_t xd[2] = {(uint64_t)H, (uint64_t)T}, xp[1] = {(uint64_t)H};
        const uint32_t xb[2] = {128, (uint32_t)bn};
        if (!fg::encode_tiled(&m.w, wtype, 3, w13, wd, wp, wb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !fg::encode_tiled(&m.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a, xd, xp, xb, CU_TENSOR_MAP_SWIZZLE_128B))
            return FG_ERR_INVALID_ARG;
        p.nk = H / 128; p.row_tiles = I / 128; p.out_rows = I;
        p.sfw = sf13;
        p.sfw_rows = kFp4 ? 2 * I : 2 * I / 128;
        p.sfw_ld = align4(p.sfw_rows);
        p.sfw_gstride = (long long)p.sfw_ld * (kFp4 ? H / 128 : (H + 511) / 512);
        p.sft = sfa; p.sft_ld = align4(T);
        p.ctr = reinterpret_cast<unsigned*>(ws);
        if (fg::launch_stream<fg::kGateUp, kFp4>(bn, p, m, dim3(grid), s) != cudaSuccess) {
            cudaGetLastError();
            return FG_ERR_CUDA;
        }
    }
    {   // down: weights [E][H][I], a box = 256 output rows of one expert
        const uint64_t row = kFp4 ? I / 2 : I;
        const uint64_t wd[3] = {(uint64_t)I, (uint64_t)H, (uint64_t)E}, wp[2] = {row, row * H};
        const uint32_t wb[3] = {128, 256, 1};
        const uint64_t xd[2] = {(uint64_t)I, (uint64_t)slots * bn}, xp[1] = {(uint64_t)I};
        const uint32_t xb[2] = {128, (uint32_t)bn};
        if (!fg::encode_tiled(&m.w, wtype, 3, w2, wd, wp, wb, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !fg::encode_tiled(&m.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.hq, xd, xp, xb, CU_TENSOR_MAP_SWIZZLE_128B))
            return FG_ERR_INVALID_ARG;
        p.nk = I / 128; p.row_tiles = (H + 255) / 256; p.out_rows = H;
        p.sfw = sf2;
        p.sfw_rows = kFp4 ? H : H / 128;
        p.sfw_ld = align4(p.sfw_rows);
        p.sfw_gstride = (long long)p.sfw_ld * (kFp4 ? I / 128 : (I + 511) / 512);
        p.sft = reinterpret_cast<const int32_t*>(p.sfh);
        p.w_raw = w2; p.x_raw = p.hq; p.w_fp4 = kFp4;
        p.ctr = reinterpret_cast<unsigned*>(ws) + fg::kMaxCounters;
        p.d = d; p.d_f32 = d_dtype == FG_F32;
        p.debug_stall = 0;
        // Up to 32 tokens a tile's pieces meet in a cluster, on three quarters of the SMs (of more, some
        // clusters wait for SMs of one GPC).  Wider parts take the third launch.  Measured on GB300, us
        // in clusters (CTAs each), through the workspace: 1 x 1024 11.0 (8), 12.8; 1 x 4096 34.4 (6),
        // 39.2; 16 x 4096 49.7 (6), 53.0; 4 x 7168 127.1 (4), 140.9 (5), 129.6; 128 x 7168 276 (4), 255
        // with the third launch.
        p.cluster = bn <= 32 ? fg::stream_cluster<fg::kDown, kFp4>(bn, p.row_tiles, grid * 3 / 4) : 1;
        if (p.cluster == 1 && bn >= 64 && p.row_tiles <= grid) p.spread = reinterpret_cast<int*>(ws) + 2 * fg::kMaxCounters;
        const dim3 ctas(p.cluster > 1 ? p.cluster * p.row_tiles : grid);
        if (fg::launch_stream<fg::kDown, kFp4>(bn, p, m, ctas, s) != cudaSuccess ||
            (p.spread && fg::launch_reduce(bn, p, s) != cudaSuccess)) {
            cudaGetLastError();
            return FG_ERR_CUDA;
        }
    }
    return FG_OK;
}

}  // namespace

extern "C" {

long long fg_moe_mlp_workspace(int T, int H, int I, int E) {
    if (!shapes_ok(T, H, I, E) || T > kMaxTokens || E > fg::kMaxListed) return -1;
    return layout(T, I, E).bytes;
}

int fg_fp8_moe_mlp(int T, int H, int I, int E, int topk, int expert_base, const uint8_t* a, const int32_t* sfa,
                   const uint8_t* w13, const int32_t* sf13, const uint8_t* w2, const int32_t* sf2,
                   const int32_t* topk_ids, const float* topk_weights, void* d, int d_dtype, void* workspace,
                   fg_stream_t stream) {
    return moe_mlp<false>(T, H, I, E, topk, expert_base, a, sfa, w13, sf13, w2, sf2, topk_ids, topk_weights, d, d_dtype,
                          workspace, stream);
}

int fg_fp8_fp4_moe_mlp(int T, int H, int I, int E, int topk, int expert_base, const uint8_t* a, const int32_t* sfa,
                       const uint8_t* w13, const int32_t* sf13, const uint8_t* w2, const int32_t* sf2,
                       const int32_t* topk_ids, const float* topk_weights, void* d, int d_dtype, void* workspace,
                       fg_stream_t stream) {
    return moe_mlp<true>(T, H, I, E, topk, expert_base, a, sfa, w13, sf13, w2, sf2, topk_ids, topk_weights, d, d_dtype,
                         workspace, stream);
}

}  // extern "C"
