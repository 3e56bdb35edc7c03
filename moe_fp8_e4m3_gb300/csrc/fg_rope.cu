// fg_rope.cu - norms of queries and keys for each head with the position rotation, in one pass.
//
// A head of D elements is held by L lanes of eight consecutive elements each (L: D / 8 rounded up to a
// power of two), in registers from its one read to its one write: sum of squares over the lanes, then
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
// in FP32, rounded once.  Pairs are neighbours, which a lane holds itself, or halves of the rotated part,
// where a lane takes its partner's four words by shuffles (and the partner's weights from memory).
// Bound: HBM bytes for many tokens (each element read and written once), launch latency for few.  The
// rotation's FP32 cosines and sines take four times the bytes of a lane's elements, so a lane keeps them
// for kHeads heads of its token, whose loads are all in flight together.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fg.h"
#include "fg_host.h"
#include "fg_kv.cuh"

namespace {

using fg::al;

constexpr int kThreads = 128;

struct RopeParams {
    const uint16_t *q, *k, *qw, *kw;
    uint16_t *qo, *ko;
    long long q_ld, k_ld, qo_ld, ko_ld;      // elements between tokens
    const int32_t* positions;
    const float* cos_sin;
    int T, Hq, Hkv, D, rot, max_pos, q_chunks, chunks;
    float eps;
    int* status;
};

__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// One (token, chunk of kHeads query or key heads) per group of L lanes; all lanes of the warp stay for
// the shuffles.
template <int L, int kHeads, bool kPairs>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
    constexpr uint32_t kAll = 0xffffffffu;
    fg::grid_dependency_wait();
    if (threadIdx.x == 0) fg::grid_launch_dependents();
    const long long item = ((long long)blockIdx.x * kThreads + threadIdx.x) / L;
    const int l = threadIdx.x % L;
    bool live = item < (long long)p.T * p.chunks;
    const int t = live ? static_cast<int>(item / p.chunks) : 0;
    const int chunk = live ? static_cast<int>(item % p.chunks) : 0;
    const bool is_q = chunk < p.q_chunks;
    const int h0 = (is_q ? chunk : chunk - p.q_chunks) * kHeads;
    const int heads = is_q ? p.Hq : p.Hkv;
    const int e0 = 8 * l;                                     // first element of this lane
    const int pos = live ? __ldg(p.positions + t) : -1;
    if (pos >= p.max_pos && l == 0) fg::kv_record(p.status, fg::kKvErrPosition);
    live = live && pos >= 0 && pos < p.max_pos && e0 < p.D;

    const uint16_t* src = (is_q ? p.q + t * p.q_ld : p.k + t * p.k_ld) + (long long)h0 * p.D + e0;
    uint16_t* dst = (is_q ? p.qo + t * p.qo_ld : p.ko + t * p.ko_ld) + (long long)h0 * p.D + e0;
    uint4 x[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (live && h0 + i < heads) x[i] = *reinterpret_cast<const uint4*>(src + (long long)i * p.D);
    }
    const int half = p.rot / 2;
    const bool turned = live && e0 < p.rot;
    const bool second = !kPairs && e0 >= half;                // this lane's elements are the pairs' b
    const int partner = (threadIdx.x & 31) - l + (turned && !kPairs ? (second ? l - half / 8 : l + half / 8) : l);
    float cs[8], sn[8];                                       // pairs: four of each
#pragma unroll
    for (int i = 0; i < 8; ++i) { cs[i] = 1.0f; sn[i] = 0.0f; }
    if (turned) {
        const float* row = p.cos_sin + (long long)pos * p.rot + (kPairs ? e0 / 2 : (second ? e0 - half : e0));
#pragma unroll
        for (int i = 0; i < (kPairs ? 4 : 8); i += 4) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(row + i));
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i));
            cs[i] = c.x; cs[i + 1] = c.y; cs[i + 2] = c.z; cs[i + 3] = c.w;
            sn[i] = s.x; sn[i + 1] = s.y; sn[i + 2] = s.z; sn[i + 3] = s.w;
        }
    }
    const uint16_t* w = is_q ? p.qw : p.kw;
    float wt[8], wp[8];                                       // this lane's weights, its partner's
#pragma unroll
    for (int i = 0; i < 8; ++i) wt[i] = wp[i] = 1.0f;
    if (w && live) {
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + e0)), wt);
        if (!kPairs && turned) unpack8(__ldg(reinterpret_cast<const uint4*>(w + (second ? e0 - half : e0 + half))), wp);
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        float f[8], g[8];
        unpack8(x[i], f);
        float r = 1.0f;
        if (p.qw || p.kw) {                                   // the same for the whole grid
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
#pragma unroll
            for (int o = L / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            if (w) r = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
        }
        if constexpr (!kPairs) {
            uint4 y;
            y.x = __shfl_sync(kAll, x[i].x, partner);
            y.y = __shfl_sync(kAll, x[i].y, partner);
            y.z = __shfl_sync(kAll, x[i].z, partner);
            y.w = __shfl_sync(kAll, x[i].w, partner);
            unpack8(y, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = g[j] * r * wp[j];
        }
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * r * wt[j];
        if constexpr (kPairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[2 * j] = f[2 * j] * cs[j] - f[2 * j + 1] * sn[j];
                o[2 * j + 1] = f[2 * j + 1] * cs[j] + f[2 * j] * sn[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = second ? f[j] * cs[j] + g[j] * sn[j] : f[j] * cs[j] - g[j] * sn[j];
        }
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = turned ? __floats2bfloat162_rn(o[2 * j], o[2 * j + 1]) : __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            out[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        if (live && h0 + i < heads) *reinterpret_cast<uint4*>(dst + (long long)i * p.D) = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

template <int L, int kHeads>
int launch(RopeParams p, bool pairs, int pdl, cudaStream_t stream) {
    p.q_chunks = (p.Hq + kHeads - 1) / kHeads;
    p.chunks = p.q_chunks + (p.Hkv + kHeads - 1) / kHeads;
    const long long blocks = ((long long)p.T * p.chunks * L + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return FG_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t e = pairs ? cudaLaunchKernelEx(&cfg, rope_kernel<L, kHeads, true>, p)
                                : cudaLaunchKernelEx(&cfg, rope_kernel<L, kHeads, false>, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    return FG_OK;
}

// Several heads a lane only where the launch fills the GPU without it.
template <int L>
int launch_heads(const RopeParams& p, bool pairs, int sms, int pdl, cudaStream_t stream) {
    const long long warps = (long long)p.T * (p.Hq + p.Hkv) * L / 32;
    return warps >= (long long)sms * 64 ? launch<L, 4>(p, pairs, pdl, stream) : launch<L, 1>(p, pairs, pdl, stream);
}

}  // namespace

extern "C" int fg_qk_norm_rope(int T, int Hq, int Hkv, int D, int rot, int max_pos, const void* q, long long q_stride,
                               const void* k, long long k_stride, const void* q_weight, const void* k_weight, float eps,
                               const int32_t* positions, const float* cos_sin, int interleaved, void* q_out,
                               long long q_out_stride, void* k_out, long long k_out_stride, fg_stream_t stream) {
    if (T < 0 || Hq < 1 || Hkv < 0 || D < 8 || D % 8 || rot < 0 || rot > D || rot % 16 || max_pos < 1 || !(eps >= 0.0f) ||
        Hq > 65536 || Hkv > 65536 || q_stride < (long long)Hq * D || q_out_stride < (long long)Hq * D ||
        k_stride < (long long)Hkv * D || k_out_stride < (long long)Hkv * D || q_stride % 8 || k_stride % 8 ||
        q_out_stride % 8 || k_out_stride % 8)
        return FG_ERR_INVALID_ARG;
    if (D > 256) return FG_ERR_UNSUPPORTED;
    if (T == 0) return FG_OK;
    if (!q || !q_out || !positions || (rot > 0 && !cos_sin) || (Hkv > 0 && (!k || !k_out)) || !al(q, 16) || !al(k, 16) ||
        !al(q_out, 16) || !al(k_out, 16) || !al(q_weight, 16) || !al(k_weight, 16) || !al(positions, 4) || !al(cos_sin, 16))
        return FG_ERR_INVALID_ARG;
    fg::HostState st;
    if (const int rc = fg::host_state(&st)) return rc;
    const RopeParams p{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(q_weight),
                       static_cast<const uint16_t*>(k_weight), static_cast<uint16_t*>(q_out), static_cast<uint16_t*>(k_out),
                       q_stride, k_stride, q_out_stride, k_out_stride, positions, cos_sin, T, Hq, Hkv, D, rot, max_pos, 0, 0,
                       eps, st.status};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool pairs = interleaved != 0;
    return D <= 64 ? launch_heads<8>(p, pairs, st.sms, st.pdl, s)
         : D <= 128 ? launch_heads<16>(p, pairs, st.sms, st.pdl, s) : launch_heads<32>(p, pairs, st.sms, st.pdl, s);
}
