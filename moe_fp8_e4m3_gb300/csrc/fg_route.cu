// fg_route.cu - MoE router: logits -> top-k expert ids and routing weights.
//
// One warp per token, the token's E logits in its registers (E / 32 per lane) as keys whose
// unsigned order is the floats'.  The k-th best expert is found k times: each lane keeps its best
// key, one warp-wide integer maximum finds the winner, the lowest of the winners' indices breaks a
// tie, and the winning lane looks for its next best.  Scores of all experts are worked out only
// where something needs them (a bias, or softmax weights that are not renormalised): else the
// chosen logits, one per lane, are enough, since a common factor cancels.
// Bound: latency, for few tokens and for many: a warp's topk rounds are one chain of reductions behind
// the load of its 4 E bytes.  Measured on GB300: 1 token x 256 experts, 8 groups, top 8 5.1 us, of which an
// empty launch takes 3; 8192 x 256, top 6 7.8 us (1.1 TB/s; the bytes alone 1.3 us), where a scheduler
// issues in 47 % of the cycles with 7 warps on it, a third of whose waits are for the logits.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "fg.h"
#include "fg_host.h"
#include "fg_ptx.cuh"

namespace {

constexpr int kWarps = 4;
constexpr float kNegInf = -__builtin_huge_valf();

struct RouteParams {
    const float* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int T, E, topk, groups, keep, sigmoid, renormalize;
    float scale;
};

// Unsigned order of floats; 0 stands for "never": -inf and NaN.  (x + 0 makes -0 equal to +0.)
__device__ __forceinline__ uint32_t ordered(float x) {
    if (!(x > kNegInf)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// Two largest of a group, as one order with -inf allowed.
__device__ __forceinline__ uint32_t ordered_any(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t k) {
    return k == 0 ? kNegInf : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// kScores: every expert's score is needed (see above).
template <int V, bool kScores>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const RouteParams p) {
    extern __shared__ float keys_s[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + warp;
    fg::grid_dependency_wait();
    if (threadIdx.x == 0) fg::grid_launch_dependents();
    if (t >= p.T) return;
    constexpr uint32_t kAll = 0xffffffffu;
    float s[V];
    uint32_t key[V];
    const float* row = p.logits + (long long)t * p.E;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        s[i] = e < p.E ? __ldcg(row + e) : kNegInf;
    }
    float bias[V];                                            // loaded beside the logits
    if (kScores && p.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = i * 32 + lane < p.E ? __ldg(p.bias + i * 32 + lane) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = ordered(s[i]);       // NaN and -inf: never chosen
    if constexpr (kScores) {
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = key[i] ? 1.0f / (1.0f + expf(-s[i])) : 0.0f;
        } else {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) best = max(best, key[i]);
            const float top = value_of(__reduce_max_sync(kAll, best));
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = key[i] ? expf(s[i] - top) : 0.0f;
                sum += s[i];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = sum > 0.0f ? s[i] / sum : (sum == sum ? 0.0f : sum);
        }
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i]) key[i] = ordered(s[i] + bias[i]);
        }
    }
    if (p.groups > 1) {
        // group score: its largest key, or with a bias the sum of its two largest.  `per_lanes` lanes
        // (a power of two) share a group and join their two largest.
        uint32_t* ks = reinterpret_cast<uint32_t*>(keys_s) + warp * p.E;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * 32 + lane < p.E) ks[i * 32 + lane] = key[i];
        __syncwarp();
        const int per = p.E / p.groups;
        const int per_lanes = 1 << (31 - __clz(32 / p.groups));
        const int g = lane / per_lanes;
        uint32_t a = 0, b = 0;                                // two largest
        if (g < p.groups)
            for (int j = lane & (per_lanes - 1); j < per; j += per_lanes) {
                const uint32_t k = ks[g * per + j];
                b = max(b, min(a, k));
                a = max(a, k);
            }
        for (int o = 1; o < per_lanes; o <<= 1) {
            const uint32_t a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
            b = max(min(a, a2), max(b, b2));
            a = max(a, a2);
        }
        const uint32_t score = ordered_any(p.bias && per > 1 ? value_of(a) + value_of(b) : value_of(a));
        int rank = 0;
        for (int h = 0; h < p.groups; ++h) {
            const uint32_t other = __shfl_sync(kAll, score, h * per_lanes);
            rank += other > score || (other == score && h < g);
        }
        const uint32_t kept = __ballot_sync(kAll, g < p.groups && rank < p.keep);   // bit g * per_lanes: group g
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * 32 + lane < p.E && !(kept >> ((i * 32 + lane) / per * per_lanes) & 1u)) key[i] = 0;
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    int my_id = -1;
    uint32_t my_key = 0;
    float my_w = 0.0f;
    for (int j = 0; j < p.topk; ++j) {
        const uint32_t m = __reduce_max_sync(kAll, best);
        if (m == 0) break;                                    // nothing left: the slots stay -1
        const uint32_t who = __ballot_sync(kAll, best == m);
        int e = 0x7fffffff;
        if (best == m) {
#pragma unroll
            for (int i = V - 1; i >= 0; --i)
                if (key[i] == m) e = i * 32 + lane;
        }
        const int win = (who & (who - 1)) == 0 ? __shfl_sync(kAll, e, __ffs(who) - 1) : __reduce_min_sync(kAll, e);
        float w = 0.0f;
        if (e == win) {
            best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (i * 32 + lane == win) {
                    if (kScores) w = s[i];
                    key[i] = 0;
                }
                best = max(best, key[i]);
            }
        }
        if (kScores) w = __shfl_sync(kAll, w, win & 31);
        if (lane == j) { my_id = win; my_key = m; my_w = w; }
    }
    if constexpr (!kScores) {
        // the key is the logit; the first chosen one is the largest
        const float l = value_of(my_key), top = value_of(__shfl_sync(kAll, my_key, 0));
        if (my_id >= 0) my_w = p.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top);
    }
    // Chosen scores below FP32's normal range (a sigmoid of -88, a softmax that the bias chose far below the
    // row's largest) have lost bits or are 0, their ratios have not: the scores again, over the largest
    // chosen one's e^min(l, 0) or e^l.
    if (p.renormalize && (kScores || p.sigmoid) && __any_sync(kAll, my_id >= 0 && my_w < FLT_MIN)) {
        const float l = my_id >= 0 ? __ldcg(p.logits + (long long)t * p.E + my_id) : kNegInf;
        const float top = value_of(__reduce_max_sync(kAll, ordered(l)));
        if (my_id >= 0) my_w = p.sigmoid ? expf(fminf(l, 0.0f) - fminf(top, 0.0f)) / (1.0f + expf(-fabsf(l))) : expf(l - top);
    }
    if (p.renormalize) {
        float sum = my_w;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        my_w = sum > 0.0f ? my_w / sum : (sum == sum ? 0.0f : sum);
    }
    if (lane < p.topk) {
        p.ids[(long long)t * p.topk + lane] = my_id;
        p.weights[(long long)t * p.topk + lane] = my_id >= 0 ? my_w * p.scale : 0.0f;
    }
}

template <int V>
cudaError_t launch(const RouteParams& p, int pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.T + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = p.groups > 1 ? kWarps * p.E * sizeof(float) : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return p.bias || !(p.sigmoid || p.renormalize) ? cudaLaunchKernelEx(&cfg, route_kernel<V, true>, p)
                                                   : cudaLaunchKernelEx(&cfg, route_kernel<V, false>, p);
}

bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" int fg_moe_route(int T, int E, int topk, int n_group, int topk_group, int score, int renormalize, float scale,
                            const float* logits, const float* bias, int32_t* topk_ids, float* topk_weights,
                            fg_stream_t stream) {
    if (T < 0 || E < 1 || topk < 1 || topk > E || n_group < 1 || E % n_group != 0 || topk_group < 1 ||
        topk_group > n_group || topk > topk_group * (E / n_group) || (score != FG_SCORE_SOFTMAX && score != FG_SCORE_SIGMOID))
        return FG_ERR_INVALID_ARG;
    if (E > 1024 || topk > 32 || n_group > 32) return FG_ERR_UNSUPPORTED;
    if (T == 0) return FG_OK;
    if (!logits || !topk_ids || !topk_weights || !al4(logits) || !al4(topk_ids) || !al4(topk_weights) || !al4(bias))
        return FG_ERR_INVALID_ARG;
    fg::HostState st;
    if (const int rc = fg::host_state(&st)) return rc;
    const RouteParams p{logits, bias, topk_ids, topk_weights, T, E, topk, n_group, topk_group,
                        score == FG_SCORE_SIGMOID, renormalize != 0, scale};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int v = (E + 31) / 32;
    const cudaError_t e = v <= 1 ? launch<1>(p, st.pdl, s) : v <= 2 ? launch<2>(p, st.pdl, s)
                        : v <= 4 ? launch<4>(p, st.pdl, s) : v <= 8 ? launch<8>(p, st.pdl, s)
                        : v <= 16 ? launch<16>(p, st.pdl, s) : launch<32>(p, st.pdl, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    return FG_OK;
}
