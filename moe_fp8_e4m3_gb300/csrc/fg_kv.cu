// fg_kv.cu - keys and values into the 4-bit cache (append) and out of it (gather).
//
// D / 8 lanes hold one token's row of one head, eight consecutive elements each: a block of 32 is four
// neighbouring lanes, and the eight elements of lane 4 b + c are the word (b, c) of a key row.  A value
// row wants half words (b, 2c) and (b, 2c + 1) instead, the first of block b beside the first of block
// b + 1: lanes of neighbouring blocks trade one half word each, so every lane stores one whole word.
// A thread has its part of one or two heads of a token in flight, keys and values both.
// Bound: HBM bytes and, near them, instructions for many tokens (8192 tokens of 8 heads of 128 in and out
// again, 85 MB: 17.3 us, 4.9 TB/s, 9.5 of them the append, which runs some 200 instructions per 16 lanes' row; 15.4 where
// the same arrays are still in L2), launch latency for few (37 tokens: 3.5 us for both calls).
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

__device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }

// Codes of a lane's eight elements (code i at bits 4i) and its block's scale exponent.
__device__ __forceinline__ uint32_t encode8(const uint4& x, int& e) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    __nv_bfloat162 most = __habs2(pair(w[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i) most = __hmax2(most, __habs2(pair(w[i])));
    float amax = fmaxf(__low2float(most), __high2float(most));       // NaN is passed over
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

// What a thread works on: its part of up to kRows heads of one token.
struct Item {
    int t, h, n;                  // token, first head, heads; n < 0: the slot is outside the cache
    long long row;                // the first head's row of the cache, the next one's p.page rows on
};

// L = D / 8 lanes per token and kRows heads; every lane of the warp stays for the shuffles.  A thread without work gets
// a place that it may read.
template <int L, int kRows>
__device__ __forceinline__ Item item_of(const KvParams& p) {
    const unsigned x = blockIdx.x * static_cast<unsigned>(kThreads / L) + threadIdx.x / L;
    const unsigned groups = (static_cast<unsigned>(p.heads) + kRows - 1) / kRows, t = x / groups;
    if (t >= static_cast<unsigned>(p.T)) return Item{0, 0, 0, 0};
    const int slot = __ldcg(p.slots + t), h = static_cast<int>(x - t * groups) * kRows;
    if (slot < 0 || slot >= p.slots_total) return Item{static_cast<int>(t), h, slot < 0 ? 0 : -1, 0};
    const unsigned page = static_cast<unsigned>(slot) / static_cast<unsigned>(p.page);
    return Item{static_cast<int>(t), h, min(kRows, p.heads - h),
                ((long long)page * p.heads + h) * p.page + (slot - page * static_cast<unsigned>(p.page))};
}
template <int L>
__device__ __forceinline__ void complain(const KvParams& p, const Item& it) {
    if (it.n < 0 && it.h == 0 && threadIdx.x % L == 0) fg::kv_record(p.status, fg::kKvErrSlot);
}

template <int L, int kRows>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvParams p) {
    constexpr int B = L / 4;
    fg::grid_dependency_wait();
    if (threadIdx.x == 0) fg::grid_launch_dependents();
    const Item it = item_of<L, kRows>(p);
    const int l = threadIdx.x % L, b = l / 4, c = l % 4;
    const uint4* kin = reinterpret_cast<const uint4*>(p.k_in + it.t * p.k_ld + it.h * (8 * L)) + l;
    const uint4* vin = reinterpret_cast<const uint4*>(p.v_in + it.t * p.v_ld + it.h * (8 * L)) + l;
    uint4 k[kRows], v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int j = max(min(i, it.n - 1), 0);               // a head that is there, so that no branch parts the loads
        k[i] = __ldcg(kin + j * L);
        v[i] = __ldcg(vin + j * L);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        int ek, ev;
        const uint32_t ck = encode8(k[i], ek), cv = encode8(v[i], ev);
        // an even block's lane gives its second half word and takes the odd block's first one
        const uint32_t other = __shfl_xor_sync(0xffffffffu, (b & 1) ? cv & 0xFFFFu : cv >> 16, 4);
        const uint32_t wv = (b & 1) ? other | (cv & 0xFFFF0000u) : (cv & 0xFFFFu) | other << 16;
        if (i < it.n) {
            const long long row = it.row + (long long)i * p.page;
            reinterpret_cast<uint32_t*>(p.kc)[row * L + c * B + b] = ck;
            reinterpret_cast<uint32_t*>(p.vc)[row * L + ((2 * c + (b & 1)) * B + (b & ~1)) / 2] = wv;
            if (c == 0) {
                p.ks[row * B + b] = static_cast<uint8_t>(ek + 127);
                p.vs[row * B + b] = static_cast<uint8_t>(ev + 127);
            }
        }
    }
    complain<L>(p, it);
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

template <int L, int kRows>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const KvParams p) {
    constexpr int B = L / 4;
    fg::grid_dependency_wait();
    if (threadIdx.x == 0) fg::grid_launch_dependents();
    const Item it = item_of<L, kRows>(p);
    const int l = threadIdx.x % L, b = l / 4, c = l % 4;
    uint32_t ck[kRows], wv[kRows], uk[kRows], uv[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const long long row = it.row + (long long)max(min(i, it.n - 1), 0) * p.page;
        ck[i] = __ldcg(reinterpret_cast<const uint32_t*>(p.kc) + row * L + c * B + b);
        wv[i] = __ldcg(reinterpret_cast<const uint32_t*>(p.vc) + row * L + ((2 * c + (b & 1)) * B + (b & ~1)) / 2);
        uk[i] = __ldcg(p.ks + row * B + b);
        uv[i] = __ldcg(p.vs + row * B + b);
    }
    uint4* ko = reinterpret_cast<uint4*>(p.k_out + it.t * p.k_ld + it.h * (8 * L)) + l;
    uint4* vo = reinterpret_cast<uint4*>(p.v_out + it.t * p.v_ld + it.h * (8 * L)) + l;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, (b & 1) ? wv[i] & 0xFFFFu : wv[i] >> 16, 4);
        const uint32_t cv = (b & 1) ? other | (wv[i] & 0xFFFF0000u) : (wv[i] & 0xFFFFu) | other << 16;
        if (i < it.n) {
            ko[i * L] = decode8(ck[i], uk[i]);
            vo[i * L] = decode8(cv, uv[i]);
        }
    }
    complain<L>(p, it);
}

template <class F>
int launch(F kernel, int rows, int per_block, const KvParams& p, int pdl, cudaStream_t stream) {
    const long long blocks = ((long long)p.T * ((p.heads + rows - 1) / rows) + per_block - 1) / per_block;
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
// One head a thread where the device holds all their threads at once (37 tokens of 8 heads of 128 in and out again: 3.5
// us, with two 3.9; 1024: 4.8 either way), two where it does not (2048: 6.3 us, with one 7.4; 8192: 17.3 and 20.5; with
// four 18.8).
template <int L>
int launch(bool append, const KvParams& p, const fg::HostState& st, cudaStream_t stream) {
    constexpr int kGroups = kThreads / L;
    const bool two = (long long)p.T * p.heads * L > st.sms * 1024LL;
    if (append)
        return two ? launch(kv_append_kernel<L, 2>, 2, kGroups, p, st.pdl, stream) : launch(kv_append_kernel<L, 1>, 1, kGroups, p, st.pdl, stream);
    return two ? launch(kv_gather_kernel<L, 2>, 2, kGroups, p, st.pdl, stream) : launch(kv_gather_kernel<L, 1>, 1, kGroups, p, st.pdl, stream);
}
int launch(bool append, int D, const KvParams& p, const fg::HostState& st, cudaStream_t stream) {
    return D == 64 ? launch<8>(append, p, st, stream) : D == 128 ? launch<16>(append, p, st, stream) : launch<32>(append, p, st, stream);
}

// The arguments that append and gather share; rows = k and v.
int check(int T, int heads, int D, int page_size, int num_pages, const void* k, long long k_stride, const void* v,
          long long v_stride, const int32_t* slots, const void* kc, const void* ks, const void* vc, const void* vs) {
    if (T < 0 || heads < 1 || D < 1 || page_size < 1 || num_pages < 1 || (long long)page_size * num_pages > 0x7fffffffLL ||
        heads > 65536 || k_stride < (long long)heads * D || v_stride < (long long)heads * D || k_stride % 8 || v_stride % 8)
        return FG_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || page_size % 16 || (long long)T * heads > 0x7fffffffLL) return FG_ERR_UNSUPPORTED;
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
    return launch(true, D, p, st, reinterpret_cast<cudaStream_t>(stream));
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
    return launch(false, D, p, st, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
