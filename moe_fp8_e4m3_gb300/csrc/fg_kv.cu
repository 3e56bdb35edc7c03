// fg_kv.cu - keys and values into the 4-bit cache (append) and out of it (gather).
//
// D / 8 lanes hold one token's row of one head, eight consecutive elements each: a block of 32 is four
// neighbouring lanes, and the eight elements of lane 4 b + c are the word (b, c) of a key row.  A value
// row wants half words (b, 2c) and (b, 2c + 1) instead, the first of block b beside the first of block
// b + 1: lanes of neighbouring blocks trade one half word each, so every lane stores one whole word.
// Bound: HBM bytes for many tokens, launch latency for few.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fg.h"
#include "fg_host.h"
#include "fg_kv.cuh"

namespace {

using fg::al;

constexpr int kThreads = 256;

struct KvParams {
    const uint16_t* k_in;         // append
    const uint16_t* v_in;
    uint16_t* k_out;              // gather
    uint16_t* v_out;
    long long k_ld, v_ld;         // elements between tokens
    const int32_t* slots;
    uint8_t *kc, *ks, *vc, *vs;
    int T, heads, page, slots_total;
    int* status;
};

// Scale exponent of a block: the smallest e with amax <= 6 * 2^e, within the cache's range (0 for a
// block of zeros).  amax = m * 2^E, m in [1, 2): m * 4 <= 6 iff m <= 1.5.
__device__ __forceinline__ int kv_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    if (b == 0) return 0;
    const int e = static_cast<int>(b >> 23) - 127 - 2 + ((b & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    return max(fg::kKvMinExp, min(fg::kKvMaxExp, e));
}

__device__ __forceinline__ float2 bf2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Codes of a lane's eight elements (code i at bits 4i) and its block's scale exponent.
__device__ __forceinline__ uint32_t encode8(const uint4& x, int& e) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf2(w[i]);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    e = kv_exponent(amax);
    const float sc = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf2(w[i]);
        codes |= (static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(f.x * sc, f.y * sc), __NV_E2M1, cudaRoundNearest)) & 0xFFu)
                 << (8 * i);
    }
    return codes;
}

struct Item {
    int t, h, l;                  // token, head, lane within the row
    bool live;
    long long row;                // row of the cache, -1: none
};

// L = D / 8 lanes per (token, head); every lane of the warp stays for the shuffles.
template <int L>
__device__ __forceinline__ Item item_of(const KvParams& p) {
    Item it;
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) / L;
    it.l = threadIdx.x % L;
    it.live = i < (long long)p.T * p.heads;
    it.t = it.live ? static_cast<int>(i / p.heads) : 0;
    it.h = it.live ? static_cast<int>(i % p.heads) : 0;
    it.row = -1;
    if (it.live) {
        const int slot = __ldg(p.slots + it.t);
        if (slot >= p.slots_total) {
            if (it.l == 0) fg::kv_record(p.status, fg::kKvErrSlot);
        } else if (slot >= 0) {
            it.row = ((long long)(slot / p.page) * p.heads + it.h) * p.page + slot % p.page;
        }
    }
    return it;
}

template <int L>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvParams p) {
    constexpr int B = L / 4;
    fg::grid_dependency_wait();
    if (threadIdx.x == 0) fg::grid_launch_dependents();
    const Item it = item_of<L>(p);
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (it.row >= 0) {
        k = __ldg(reinterpret_cast<const uint4*>(p.k_in + it.t * p.k_ld + it.h * (8 * L)) + it.l);
        v = __ldg(reinterpret_cast<const uint4*>(p.v_in + it.t * p.v_ld + it.h * (8 * L)) + it.l);
    }
    int ek, ev;
    const uint32_t ck = encode8(k, ek), cv = encode8(v, ev);
    const int b = it.l / 4, c = it.l % 4;
    // an even block's lane gives its second half word and takes the odd block's first one
    const uint32_t other = __shfl_xor_sync(0xffffffffu, (b & 1) ? cv & 0xFFFFu : cv >> 16, 4);
    const uint32_t wv = (b & 1) ? other | (cv & 0xFFFF0000u) : (cv & 0xFFFFu) | other << 16;
    if (it.row < 0) return;
    reinterpret_cast<uint32_t*>(p.kc + it.row * (4 * L))[c * B + b] = ck;
    reinterpret_cast<uint32_t*>(p.vc + it.row * (4 * L))[((2 * c + (b & 1)) * B + (b & ~1)) / 2] = wv;
    if (c == 0) {
        p.ks[it.row * B + b] = static_cast<uint8_t>(ek + 127);
        p.vs[it.row * B + b] = static_cast<uint8_t>(ev + 127);
    }
}

// Values of eight codes as BF16 (E2M1 times a power of two within the cache's range: exact).
__device__ __forceinline__ uint4 decode8(uint32_t codes, uint32_t u) {
    uint32_t h[4], o[4];
    fg::e2m1x8_f16(codes, h);
    const float s = fg::ue8m0(u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h[i]));
        const __nv_bfloat162 w = __floats2bfloat162_rn(lo * s, hi * s);
        o[i] = *reinterpret_cast<const uint32_t*>(&w);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int L>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const KvParams p) {
    constexpr int B = L / 4;
    fg::grid_dependency_wait();
    if (threadIdx.x == 0) fg::grid_launch_dependents();
    const Item it = item_of<L>(p);
    const int b = it.l / 4, c = it.l % 4;
    uint32_t ck = 0, wv = 0, uk = 0, uv = 0;
    if (it.row >= 0) {
        ck = __ldcg(reinterpret_cast<const uint32_t*>(p.kc + it.row * (4 * L)) + c * B + b);
        wv = __ldcg(reinterpret_cast<const uint32_t*>(p.vc + it.row * (4 * L)) + ((2 * c + (b & 1)) * B + (b & ~1)) / 2);
        uk = __ldcg(p.ks + it.row * B + b);
        uv = __ldcg(p.vs + it.row * B + b);
    }
    const uint32_t other = __shfl_xor_sync(0xffffffffu, (b & 1) ? wv & 0xFFFFu : wv >> 16, 4);
    const uint32_t cv = (b & 1) ? other | (wv & 0xFFFF0000u) : (wv & 0xFFFFu) | other << 16;
    if (it.row < 0) return;
    reinterpret_cast<uint4*>(p.k_out + it.t * p.k_ld + it.h * (8 * L))[it.l] = decode8(ck, uk);
    reinterpret_cast<uint4*>(p.v_out + it.t * p.v_ld + it.h * (8 * L))[it.l] = decode8(cv, uv);
}

template <class F>
int launch(F kernel, int L, const KvParams& p, int pdl, cudaStream_t stream) {
    const long long blocks = ((long long)p.T * p.heads * L + kThreads - 1) / kThreads;
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
    if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    return FG_OK;
}

// The arguments that append and gather share; rows = k and v.
int check(int T, int heads, int D, int page_size, int num_pages, const void* k, long long k_stride, const void* v,
          long long v_stride, const int32_t* slots, const void* kc, const void* ks, const void* vc, const void* vs) {
    if (T < 0 || heads < 1 || D < 1 || page_size < 1 || num_pages < 1 || (long long)page_size * num_pages > 0x7fffffffLL ||
        heads > 65536 || k_stride < (long long)heads * D || v_stride < (long long)heads * D || k_stride % 8 || v_stride % 8)
        return FG_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || page_size % 16) return FG_ERR_UNSUPPORTED;
    if (T == 0) return FG_OK;
    if (!k || !v || !slots || !kc || !ks || !vc || !vs || !al(k, 16) || !al(v, 16) || !al(slots, 4) || !al(kc, 16) ||
        !al(ks, 16) || !al(vc, 16) || !al(vs, 16))
        return FG_ERR_INVALID_ARG;
    return FG_OK;
}

}  // namespace

extern "C" {

int fg_kv_append_mxfp4(int T, int heads, int D, int page_size, int num_pages, const void* k, long long k_stride,
                       const void* v, long long v_stride, const int32_t* slots, uint8_t* k_cache, uint8_t* k_sf,
                       uint8_t* v_cache, uint8_t* v_sf, fg_stream_t stream) {
    if (const int rc = check(T, heads, D, page_size, num_pages, k, k_stride, v, v_stride, slots, k_cache, k_sf, v_cache, v_sf))
        return rc;
    if (T == 0) return FG_OK;
    fg::HostState st;
    if (const int rc = fg::host_state(&st)) return rc;
    const KvParams p{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), nullptr, nullptr, k_stride, v_stride,
                     slots, k_cache, k_sf, v_cache, v_sf, T, heads, page_size, page_size * num_pages, st.status};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return D == 64 ? launch(kv_append_kernel<8>, 8, p, st.pdl, s)
         : D == 128 ? launch(kv_append_kernel<16>, 16, p, st.pdl, s) : launch(kv_append_kernel<32>, 32, p, st.pdl, s);
}

int fg_kv_gather_mxfp4(int T, int heads, int D, int page_size, int num_pages, const int32_t* slots, const uint8_t* k_cache,
                       const uint8_t* k_sf, const uint8_t* v_cache, const uint8_t* v_sf, void* k, long long k_stride,
                       void* v, long long v_stride, fg_stream_t stream) {
    if (const int rc = check(T, heads, D, page_size, num_pages, k, k_stride, v, v_stride, slots, k_cache, k_sf, v_cache, v_sf))
        return rc;
    if (T == 0) return FG_OK;
    fg::HostState st;
    if (const int rc = fg::host_state(&st)) return rc;
    const KvParams p{nullptr, nullptr, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), k_stride, v_stride, slots,
                     const_cast<uint8_t*>(k_cache), const_cast<uint8_t*>(k_sf), const_cast<uint8_t*>(v_cache),
                     const_cast<uint8_t*>(v_sf), T, heads, page_size, page_size * num_pages, st.status};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return D == 64 ? launch(kv_gather_kernel<8>, 8, p, st.pdl, s)
         : D == 128 ? launch(kv_gather_kernel<16>, 16, p, st.pdl, s) : launch(kv_gather_kernel<32>, 32, p, st.pdl, s);
}

}  // extern "C"
