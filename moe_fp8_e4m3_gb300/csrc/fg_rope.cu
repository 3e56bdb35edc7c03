// fg_rope.cu - norms of queries and keys for each head with the position rotation, in one pass.
//
// A head of D elements is held by L lanes (L: D / 8 rounded up to a power of two), eight elements each, in
// registers from its one read to its one write: sum of squares over the lanes, then
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
// in FP32, rounded once.  A lane holds both elements of its four pairs (two runs of four elements, from the two halves
// of the rotated part or side by side), so that it needs four cosines and sines and nothing of its neighbours; lanes
// behind the rotated part hold eight elements that stay.
// Bound: HBM bytes for many tokens (each element read and written once), launch latency for few.  A lane keeps its
// cosines, sines and weights for kHeads heads of its token, whose loads are all in flight together: 8192 tokens of 64 + 8
// heads of 128 take 51.9 us (306 MB, 5.9 TB/s; 64.4 with fewer in flight and pairs met by shuffles), one token 1.6 us.
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

__device__ __forceinline__ void unpack4(const uint2& x, float (&f)[4]) {
    f[0] = __uint_as_float(x.x << 16);
    f[1] = __uint_as_float(x.x & 0xFFFF0000u);
    f[2] = __uint_as_float(x.y << 16);
    f[3] = __uint_as_float(x.y & 0xFFFF0000u);
}
__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// One (token, chunk of kHeads query or key heads) per group of L lanes; all lanes of the warp stay for
// the shuffles.
template <int L, int kHeads, bool kPairs>
__global__ void __launch_bounds__(kThreads, 7) rope_kernel(const RopeParams p) {
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
    const int pos = live ? __ldcg(p.positions + t) : -1;
    if (pos >= p.max_pos && l == 0) fg::kv_record(p.status, fg::kKvErrPosition);
    const bool turned = 8 * l < p.rot;
    const int ea = kPairs ? 8 * l : turned ? 4 * l : p.rot + 8 * (l - p.rot / 8);      // this lane's two runs of four
    const int eb = !kPairs && turned ? p.rot / 2 + 4 * l : ea + 4;
    live = live && pos >= 0 && pos < p.max_pos && 8 * l < p.D;

    const uint16_t* src = (is_q ? p.q + t * p.q_ld : p.k + t * p.k_ld) + (long long)h0 * p.D;
    uint16_t* dst = (is_q ? p.qo + t * p.qo_ld : p.ko + t * p.ko_ld) + (long long)h0 * p.D;
    uint2 xa[kHeads], xb[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        xa[i] = xb[i] = make_uint2(0, 0);
        if (live && h0 + i < heads) {
            xa[i] = *reinterpret_cast<const uint2*>(src + i * p.D + ea);
            xb[i] = *reinterpret_cast<const uint2*>(src + i * p.D + eb);
        }
    }
    float4 cs = make_float4(1.0f, 1.0f, 1.0f, 1.0f), sn = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (live && turned) {
        const float* row = p.cos_sin + (long long)pos * p.rot + 4 * l;
        cs = __ldcg(reinterpret_cast<const float4*>(row));
        sn = __ldcg(reinterpret_cast<const float4*>(row + p.rot / 2));
    }
    const uint16_t* w = is_q ? p.qw : p.kw;
    uint2 wa = make_uint2(0, 0), wb = wa;                     // as they are stored: registers hold more heads
    if (w && live) {
        wa = __ldcg(reinterpret_cast<const uint2*>(w + ea));
        wb = __ldcg(reinterpret_cast<const uint2*>(w + eb));
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        float a[4], b[4];
        unpack4(xa[i], a);
        unpack4(xb[i], b);
        if (p.qw || p.kw) {                                   // the same for the whole grid
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum = fmaf(a[j], a[j], fmaf(b[j], b[j], sum));
#pragma unroll
            for (int o = L / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            if (w) {
                const float r = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
                float fa[4], fb[4];
                unpack4(wa, fa);
                unpack4(wb, fb);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[j] = a[j] * r * fa[j];
                    b[j] = b[j] * r * fb[j];
                }
            }
        }
        uint2 ya, yb;
        if constexpr (kPairs) {
            ya = pack4(a[0] * cs.x - a[1] * sn.x, a[1] * cs.x + a[0] * sn.x, a[2] * cs.y - a[3] * sn.y, a[3] * cs.y + a[2] * sn.y);
            yb = pack4(b[0] * cs.z - b[1] * sn.z, b[1] * cs.z + b[0] * sn.z, b[2] * cs.w - b[3] * sn.w, b[3] * cs.w + b[2] * sn.w);
        } else {
            ya = pack4(a[0] * cs.x - b[0] * sn.x, a[1] * cs.y - b[1] * sn.y, a[2] * cs.z - b[2] * sn.z, a[3] * cs.w - b[3] * sn.w);
            yb = pack4(b[0] * cs.x + a[0] * sn.x, b[1] * cs.y + a[1] * sn.y, b[2] * cs.z + a[2] * sn.z, b[3] * cs.w + a[3] * sn.w);
        }
        if (live && h0 + i < heads) {
            // an element that is not turned keeps its value, also where its partner in the lane is not finite
            *reinterpret_cast<uint2*>(dst + i * p.D + ea) = turned ? ya : pack4(a[0], a[1], a[2], a[3]);
            *reinterpret_cast<uint2*>(dst + i * p.D + eb) = turned ? yb : pack4(b[0], b[1], b[2], b[3]);
        }
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
    return warps >= (long long)sms * 64 ? launch<L, 8>(p, pairs, pdl, stream) : launch<L, 1>(p, pairs, pdl, stream);
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
