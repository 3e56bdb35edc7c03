// fg_attn_prompt.cu - attention of many new tokens a request over its 4-bit key/value cache, on the tensor
// cores of the fifth generation.
//
// An item is 128 rows (new tokens x the query heads that share a kv head) of one request; per tile of kTok keys
//   S = Q K^T       tcgen05.mma, BF16, FP32 in tensor memory (two tiles of it, so the next product runs while a
//                   tile's exponentials are taken)
//   P = 2^(S - m)   two threads a row, half of the keys each, in registers; m a running maximum that moves only when a score passes it by 2^8, because
//                   moving it scales O, which lives in tensor memory; P rounded once, to BF16
//   O += P V        tcgen05.mma, BF16, FP32 in tensor memory
// Keys and values become BF16 tiles in shared memory once per item tile, exactly (a code has two significant bits,
// its scale is a power of two): 256 threads decode what 128 rows use.  Keys, values and Q stand as rows of 64
// elements in 128-byte swizzled atoms; a value tile is the product's MN-major operand as it is.
//
// Warps: 0-7 softmax and output (warps w and w + 4 share 32 rows), 8 the MMA issuer, 9-16 the decoders.  They meet at
// mbarriers (every wait is bounded, as in the GEMMs); a row's two threads meet at a barrier of their two warps,
// which both reach on every tile, also after a wait that ran out; pieces of items follow one another with a CTA
// barrier between.
#include <cuda_runtime.h>

#include <cstdio>

#include "fg.h"
#include "fg_host.h"
#include "fg_attn.cuh"
#include "fg_gemm_kernel.cuh"

namespace {

using fg::AttnParams;
using fg::ex2;

constexpr int kRows = fg::kPromptRows;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kDecodeWarp0 = 9, kDecodeWarps = 8;
constexpr int kThreads = 32 * (kDecodeWarp0 + kDecodeWarps);
constexpr int kWaitPrompt = 12;                // status code of a wait that ran out
constexpr float kSlack = 8.0f;                 // scores above m by at most this (log2): P <= 2^8
constexpr uint32_t kAll = fg::kAllLanes;

template <int B>
struct Cfg {
    static constexpr int D = 32 * B, kSub = B / 2;               // sub-tiles of 64 elements
    static constexpr int kTok = B == 8 ? 64 : 128;               // keys of a tile
    static constexpr int kTile = kTok * 128 * kSub;              // bytes of a key or value tile
    static constexpr int kQ = kRows * 128 * kSub, kP = kRows * kTok * 2;
    static constexpr int kOffK = kQ, kOffV = kOffK + 2 * kTile, kOffP = kOffV + 2 * kTile, kOffBar = kOffP + kP;
    static constexpr int kNumBars = 14;
    static constexpr int kOffMisc = kOffBar + 8 * kNumBars;      // tensor memory address, abort flag, drain barrier
    static constexpr int kOffPre = kOffMisc + 16;
    static constexpr int kSmem = 1024 + kOffPre;                 // then [S + 1] int
    static constexpr int kCols = 256;                            // O's first column (S: 0 and 128)
    // a decoder thread: one token, kC of the four column groups
    static constexpr int kC = 4 * kTok / (32 * kDecodeWarps);
};
constexpr int kMaxRequests = 1024;

__device__ __forceinline__ void tc_mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// kind::f16 with BF16 operands (format 1 at bits 7 and 10), FP32 accumulator, A K-major, B K- or MN-major (bit 16).
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool b_mn) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn ? 1u : 0u) << 16 | static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(m >> 4) << 24;
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
        " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
          "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
          "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_shared_16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Barrier of the 64 threads of two warps; returns whether the predicate holds for any of them.
__device__ __forceinline__ bool pair_any(int id, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, %1, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"(pred ? 1u : 0u) : "memory");
    return r != 0;
}

// What a decoder thread holds of a tile: its column groups of one token's key and value rows, and their scales.
template <int B>
struct Raw {
    uint32_t k[Cfg<B>::kC][B], v[Cfg<B>::kC][B];
    uint32_t ks[(B + 3) / 4], vs[(B + 3) / 4];
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&r)[N], const uint8_t* p) {
    if constexpr (N == 1) {
        r[0] = __ldcg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (N == 2) {
        const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
        r[0] = v.x; r[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p) + i / 4);
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    }
}

template <int B>
__device__ __forceinline__ float scale_of(const uint32_t (&s)[(B + 3) / 4], int b) {
    const uint32_t w = s[b / 4];
    const int sh = 8 * (b % 4);
    return __uint_as_float((sh <= 23 ? w << (23 - sh) : w >> (sh - 23)) & 0x7F800000u);
}

template <int B>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const AttnParams p) {
    using C = Cfg<B>;
    constexpr int D = C::D, kTok = C::kTok;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = fg::smem_u32(smem);
    __shared__ fg::AttnPlanSmem<kThreads> s_plan;
    __shared__ float s_top[2][kRows], s_l[2][kRows];           // of a row's two halves
    __shared__ int s_dead[kSoftWarps];
    __shared__ fg::AttnCursor<kRows, C::kTok, kThreads> s_cur;  // while the roles run, out of their registers
    const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
    const uint32_t bar = sbase + C::kOffBar;
    const uint32_t k_full = bar, k_empty = bar + 16, v_full = bar + 32, v_empty = bar + 48, s_full = bar + 64, s_empty = bar + 80,
                   p_full = bar + 96, p_empty = bar + 104;                 // two of each but the last two
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    uint64_t* drain = reinterpret_cast<uint64_t*>(smem + C::kOffMisc + 8);
    int* s_pre = reinterpret_cast<int*>(smem + C::kOffPre);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            fg::mbar_init(k_full + 8 * i, kDecodeWarps);
            fg::mbar_init(k_empty + 8 * i, 1);
            fg::mbar_init(v_full + 8 * i, kDecodeWarps);
            fg::mbar_init(v_empty + 8 * i, 1);
            fg::mbar_init(s_full + 8 * i, 1);
            fg::mbar_init(s_empty + 8 * i, kSoftWarps);
        }
        fg::mbar_init(p_full, kSoftWarps);
        fg::mbar_init(p_empty, 1);
        fg::mbar_init(fg::smem_u32(drain), 1);
        *abort_flag = 0;
        fg::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        fg::tmem_alloc(fg::smem_u32(tmem_slot), 512);
        fg::tmem_relinquish();
    }
    fg::tc_fence_before();
    __syncthreads();
    fg::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    fg::grid_dependency_wait();
    if (tid == 0) fg::grid_launch_dependents();
    const fg::WaitCtl wctl{abort_flag, p.status, p.timeout_ns};
    auto wait = [&](uint32_t b, uint32_t parity) { return fg::wait_bar(b, parity, wctl, kWaitPrompt); };

    fg::AttnCursor<kRows, kTok, kThreads> cur;
    const bool any = cur.open(p, s_plan, s_pre);
    uint32_t n0 = 0;                                           // tiles of the pieces before this one
    while (any) {
        int b0, b1;
        if (!cur.piece(s_plan, b0, b1)) break;
        const int h = cur.h;
        const int row0 = (cur.ch - s_pre[cur.r]) * kRows, rows = min(kRows, cur.rq.n * p.group - row0);
        const int first = cur.rq.len - cur.rq.n;               // position of new token 0
        const int* table = p.table + (long long)cur.r * p.max_pages;
        const bool empty = cur.keys.hi <= cur.keys.lo;
        const int t0 = cur.rq.t0, keys_lo = cur.keys.lo;
        if (tid == 0) s_cur = cur;
        const int tok0 = b0 * kTok, tok1 = empty ? tok0 : min(b1 * kTok, cur.keys.hi);
        const int tiles = (tok1 - tok0 + kTok - 1) / kTok;     // 0 where no row of the item has a key

        // Q: 16-byte chunks of the 128 rows, zeros behind the last
        if (warp >= kDecodeWarp0) {
            const int t = tid - 32 * kDecodeWarp0, j = t % kRows;
            const int i = (row0 + j) / p.group, hq = h * p.group + (row0 + j) % p.group;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + ((long long)(t0 + i) * p.heads * p.group + hq) * D);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                const int ch = (t / kRows) * (D / 16) + x;      // chunk of eight elements
                const uint4 v = j < rows ? __ldcg(src + ch) : make_uint4(0, 0, 0, 0);
                st_shared_16(sbase + (ch / 8) * (kRows * 128) + j * 128 + (((ch % 8) ^ (j & 7)) << 4), v);
            }
            fg::fence_proxy_async_smem();
        }
        __syncthreads();

        float m = fg::kAttnEmpty, l = 0.0f;                    // of this thread's row, and of its half (softmax warps)
        if (warp >= kDecodeWarp0) {
            // ------------------------------------------------------------- decoders
            const int t = tid - 32 * kDecodeWarp0, my = t % kTok, c0 = t / kTok * C::kC;
            int page_i = (tok0 + my) / p.page, page_off = (tok0 + my) % p.page;
            const int step_page = kTok / p.page, step_off = kTok % p.page;
            auto next_page = [&](int tok) {                     // the page of token tok (its row's offset in `off`); -1: none
                const int group = tok & ~15;
                const bool wanted = tok < tok1 && group + 16 > keys_lo;
                const int id = wanted ? __ldg(table + page_i) : -1;
                return id >= 0 && id < p.pages ? id : -1;
            };
            auto load = [&](Raw<B>& x, int page, int off) {
                if (page >= 0) {
                    const long long row = ((long long)page * p.heads + h) * p.page + off;
#pragma unroll
                    for (int i = 0; i < C::kC; ++i) {
                        load_words(x.k[i], p.kc + row * (16 * B) + (c0 + i) * (4 * B));
                        load_words(x.v[i], p.vc + row * (16 * B) + (c0 + i) * (4 * B));
                    }
                    if constexpr (B == 2) {
                        x.ks[0] = __ldcg(reinterpret_cast<const uint16_t*>(p.ks + row * B));
                        x.vs[0] = __ldcg(reinterpret_cast<const uint16_t*>(p.vs + row * B));
                    } else {
                        load_words(x.ks, p.ks + row * B);
                        load_words(x.vs, p.vs + row * B);
                    }
                } else {                                       // absent: zeros, which the softmax masks
#pragma unroll
                    for (int i = 0; i < C::kC; ++i)
#pragma unroll
                        for (int j = 0; j < B; ++j) x.k[i][j] = x.v[i][j] = 0;
#pragma unroll
                    for (int i = 0; i < (B + 3) / 4; ++i) x.ks[i] = x.vs[i] = 0;
                }
            };
            auto advance = [&]() {
                page_i += step_page;
                page_off += step_off;
                if (page_off >= p.page) { page_off -= p.page; ++page_i; }
            };
            auto decode = [&](uint32_t codes, float s) {
                uint32_t f[4], o[4];
                fg::e2m1x8_f16(codes, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(f[i]));
                    const __nv_bfloat162 w = __floats2bfloat162_rn(lo * s, hi * s);
                    o[i] = *reinterpret_cast<const uint32_t*>(&w);
                }
                return make_uint4(o[0], o[1], o[2], o[3]);
            };
            // place of chunk (b, c) of this token's row in a tile
            auto place = [&](int b, int c) { return static_cast<uint32_t>((b / 2) * (kTok * 128) + my * 128 + ((((b & 1) * 4 + c) ^ (my & 7)) << 4)); };
            auto fill = [&](const Raw<B>& x, uint32_t n) {
                const uint32_t st = n & 1, ph = (n >> 1) & 1;
                bool ok = wait(k_empty + 8 * st, ph ^ 1);
                if (!__all_sync(kAll, ok)) return false;
                const uint32_t kt = sbase + C::kOffK + st * C::kTile, vt = sbase + C::kOffV + st * C::kTile;
#pragma unroll
                for (int i = 0; i < C::kC; ++i)
#pragma unroll
                    for (int b = 0; b < B; ++b) st_shared_16(kt + place(b, c0 + i), decode(x.k[i][b], scale_of<B>(x.ks, b)));
                fg::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) fg::mbar_arrive(k_full + 8 * st);
                ok = wait(v_empty + 8 * st, ph ^ 1);
                if (!__all_sync(kAll, ok)) return false;
#pragma unroll
                for (int i = 0; i < C::kC; ++i)
#pragma unroll
                    for (int b = 0; b < B; ++b)
                        st_shared_16(vt + place(b, c0 + i), decode(__byte_perm(x.v[i][b / 2], x.v[i][B / 2 + b / 2], (b & 1) ? 0x7632 : 0x5410),
                                                                   scale_of<B>(x.vs, b)));
                fg::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) fg::mbar_arrive(v_full + 8 * st);
                return true;
            };
            Raw<B> x, ahead;                                    // a tile, and the next one on its way
            int tok = tok0 + my, off = page_off, page = next_page(tok);
            load(x, page, off);
            auto look = [&]() {                                 // the page of the tile after the last one looked up
                advance();
                tok += kTok;
                off = page_off;
                page = next_page(tok);
            };
            look();
#pragma unroll 1
            for (int i = 0; i < tiles; ++i) {
                load(ahead, page, off);
                look();
                if (!fill(x, n0 + i)) break;
                x = ahead;
            }
        } else if (warp == kMmaWarp) {
            // ----------------------------------------------------------- MMA issuer
            if (lane == 0) {
                constexpr uint32_t kIdS = idesc_bf16(kRows, kTok, false), kIdO = idesc_bf16(kRows, D, true);
                const uint64_t dq = fg::make_sdesc(sbase, 0, 1024, fg::kLayoutSw128);
                const uint64_t dk = fg::make_sdesc(sbase + C::kOffK, 0, 1024, fg::kLayoutSw128);
                const uint64_t dv = fg::make_sdesc(sbase + C::kOffV, kTok * 128, 1024, fg::kLayoutSw128);
                const uint64_t dp = fg::make_sdesc(sbase + C::kOffP, 0, 1024, fg::kLayoutSw128);
                for (int i = 0; i <= tiles; ++i) {
                    const uint32_t n = n0 + i;
                    if (i < tiles) {
                        const uint32_t st = n & 1, ph = (n >> 1) & 1;
                        if (!wait(k_full + 8 * st, ph) || !wait(s_empty + 8 * st, ph ^ 1)) break;
                        fg::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4 * C::kSub; ++k)
                            tc_mma_bf16(tmem + st * 128, dq + (k / 4) * (kRows * 128 / 16) + (k % 4) * 2,
                                        dk + st * (C::kTile / 16) + (k / 4) * (kTok * 128 / 16) + (k % 4) * 2, kIdS, k != 0);
                        fg::tc_commit(s_full + 8 * st);
                        fg::tc_commit(k_empty + 8 * st);
                    }
                    if (i > 0) {
                        const uint32_t q = n - 1, st = q & 1, ph = (q >> 1) & 1;
                        if (!wait(v_full + 8 * st, ph) || !wait(p_full, q & 1)) break;
                        fg::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kTok / 16; ++k)
                            tc_mma_bf16(tmem + C::kCols, dp + (k / 4) * (kRows * 128 / 16) + (k % 4) * 2,
                                        dv + st * (C::kTile / 16) + k * (2048 / 16), kIdO, i > 1 || k != 0);
                        fg::tc_commit(v_empty + 8 * st);
                        fg::tc_commit(p_empty);
                    }
                }
            }
            __syncwarp();
        } else {
            // ------------------------------------------- softmax, half a row's keys a thread
            constexpr int kHalf = kTok / 2;
            const int half = warp >> 2, my = (warp & 3) * 32 + lane, col0 = half * kHalf;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const int hi = first + (row0 + my) / p.group + 1, lo = p.window > 0 ? hi - p.window : 0;
            // keys that every row of the chunk looks at
            const int all_hi = first + row0 / p.group + 1;
            const int all_lo = p.window > 0 ? max(0, first + (row0 + rows - 1) / p.group + 1 - p.window) : 0;
            const uint32_t p_row = sbase + C::kOffP + (col0 / 64) * (kRows * 128) + my * 128;
            for (int i = 0; i < tiles; ++i) {
                const uint32_t n = n0 + i, st = n & 1, ph = (n >> 1) & 1;
                const int base = tok0 + i * kTok;
                // sixteen-token groups whose page is outside the cache
                uint32_t absent = 0;
                {
                    const int at = base + 16 * lane;
                    bool bad = false;
                    if (lane < kTok / 16 && at < tok1 && at + 16 > keys_lo) {
                        const int id = __ldg(table + at / p.page);
                        bad = id < 0 || id >= p.pages;
                    }
                    absent = __ballot_sync(kAll, bad);
                    if (absent && lane == 0) fg::kv_record(p.status, fg::kKvErrAttention);
                }
                bool dead = !__all_sync(kAll, wait(s_full + 8 * st, ph));
                fg::tc_fence_after();
                const uint32_t at_s = tmem + lanes + st * 128 + col0;
                const bool border = absent != 0 || base < all_lo || base + kTok > all_hi;
                auto scores = [&](int c, uint32_t (&r)[32]) {   // columns col0 + c .. + 31, masked at a border
                    fg::tmem_ld_32x32b_x32(at_s + c, r);
                    fg::tmem_wait_ld();
                    if (border) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            const int tok = base + col0 + c + x;
                            if (tok < lo || tok >= hi || (absent >> ((col0 + c + x) >> 4) & 1u)) r[x] = 0xFF800000u;
                        }
                    }
                };
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < kHalf; c += 32) {
                    uint32_t r[32];
                    scores(c, r);
#pragma unroll
                    for (int x = 0; x < 32; ++x) top = fmaxf(top, __uint_as_float(r[x]));
                }
                top *= p.scale_log2;
                // the last tile's P has been read, and O is whole, once its product is done
                if (n > 0) dead = dead || !__all_sync(kAll, wait(p_empty, (n - 1) & 1));
                if (pair_any(1 + (warp & 3), dead || top > m + kSlack)) {
                    s_top[half][my] = top;
                    if (lane == 0) s_dead[warp] = dead;
                    pair_any(1 + (warp & 3), false);
                    const float both = fmaxf(top, s_top[half ^ 1][my]);
                    if (dead || s_dead[warp ^ 4]) break;
                    const float now = both > m + kSlack ? both : m, f = ex2(m - now);
                    m = now;
                    l *= f;
                    if (i > 0) {
                        fg::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 32) {
                            uint32_t x[32];
                            const uint32_t at = tmem + lanes + C::kCols + half * (D / 2) + c;
                            fg::tmem_ld_32x32b_x32(at, x);
                            fg::tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 32; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * f);
                            tmem_st_32x32b_x32(at, x);
                        }
                        tmem_wait_st();
                        fg::tc_fence_before();
                    }
                    pair_any(1 + (warp & 3), false);            // both have read before either writes again
                }
                const float shift = -m;
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < kHalf; c += 32) {
                    uint32_t r[32];
                    scores(c, r);
#pragma unroll
                    for (int x = 0; x < 32; x += 8) {
                        uint32_t o[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float w0 = ex2(fmaf(__uint_as_float(r[x + 2 * y]), p.scale_log2, shift));
                            const float w1 = ex2(fmaf(__uint_as_float(r[x + 2 * y + 1]), p.scale_log2, shift));
                            part[y] += w0 + w1;
                            const __nv_bfloat162 w = __floats2bfloat162_rn(w0, w1);
                            o[y] = *reinterpret_cast<const uint32_t*>(&w);
                        }
                        st_shared_16(p_row + (((((col0 + c) % 64 + x) / 8) ^ (my & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
                    }
                }
                l += (part[0] + part[1]) + (part[2] + part[3]);
                fg::tc_fence_before();
                fg::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    fg::mbar_arrive(s_empty + 8 * st);
                    fg::mbar_arrive(p_full);
                }
            }
            if (tiles > 0) {
                const bool ok = wait(p_empty, (n0 + tiles - 1) & 1);
                (void)ok;                                       // on a time-out the abort flag is up: the output is not stored
                __syncwarp();
                fg::tc_fence_after();
            }
            s_l[half][my] = l;
        }
        __syncthreads();
        if (*abort_flag) break;
        n0 += tiles;
        cur = s_cur;

        // ------------------------------------------------------------------ output
        int a, z;
        cur.holders(s_plan, a, z);
        const bool whole = a == z;
        if (warp < kSoftWarps) {
            const int half = warp >> 2, my = (warp & 3) * 32 + lane;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const float sum = s_l[0][my] + s_l[1][my];
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            float* slot = fg::attn_piece<kRows, D>(p, blockIdx.x, a);
            if (!whole && half == 0 && my < rows) {
                slot[my] = m;
                slot[kRows + my] = sum;
            }
            const int i = (row0 + my) / p.group, hq = h * p.group + (row0 + my) % p.group;
            uint16_t* out = p.out + ((long long)(cur.rq.t0 + i) * p.heads * p.group + hq) * D;
#pragma unroll 1
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
                uint32_t r[32];
                if (tiles > 0) {
                    fg::tmem_ld_32x32b_x32(tmem + lanes + C::kCols + c, r);
                    fg::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) r[x] = 0;
                }
                if (my < rows && whole) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t o[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const __nv_bfloat162 w = __floats2bfloat162_rn(__uint_as_float(r[8 * x + 2 * y]) * inv, __uint_as_float(r[8 * x + 2 * y + 1]) * inv);
                            o[y] = *reinterpret_cast<const uint32_t*>(&w);
                        }
                        *reinterpret_cast<uint4*>(out + c + 8 * x) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                } else if (my < rows) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        *reinterpret_cast<float4*>(slot + 2 * kRows + my * D + c + 4 * x) =
                            make_float4(__uint_as_float(r[4 * x]), __uint_as_float(r[4 * x + 1]), __uint_as_float(r[4 * x + 2]), __uint_as_float(r[4 * x + 3]));
                }
            }
            fg::tc_fence_before();
        }
        if (!whole) fg::attn_join<kRows, D, kThreads>(p, s_plan, a, z, cur.rq.t0, h, row0, rows);
        if (!cur.next(p, s_plan, s_pre)) break;
        __syncthreads();                                        // Q and O are written again
        fg::tc_fence_after();
    }

    // Every product is done (bounded) before tensor memory goes back.
    if (warp == kMmaWarp && lane == 0) {
        fg::tc_commit(fg::smem_u32(drain));
        const uint64_t t0 = fg::globaltimer_ns();
        while (!fg::mbar_try_wait(fg::smem_u32(drain), 0))
            if (fg::globaltimer_ns() - t0 > p.timeout_ns) { fg::record_status(p.status, fg::kErrTimeout | fg::kWaitDrain); break; }
    }
    fg::tc_fence_before();
    __syncthreads();
    fg::tc_fence_after();
    if (warp == kMmaWarp) fg::tmem_dealloc(tmem, 512);
}

template <int B>
int launch(const AttnParams& p, int sms, int pdl, cudaStream_t stream) {
    using C = Cfg<B>;
    static bool configured[256] = {};        // set once per device; setting it again is harmless
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(attn_prompt_kernel<B>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem + (kMaxRequests + 1) * 4) !=
            cudaSuccess) {
            cudaGetLastError();
            return FG_ERR_CUDA;
        }
        configured[dev] = true;
    }
    const int ctas = sms < fg::kAttnPromptCtas ? sms : fg::kAttnPromptCtas;
    if (fg::print_configs_enabled())
        std::fprintf(stderr, "[fg] paged_attention_mxfp4 T=%d S=%d heads=%d x %d D=%d rows=%d grid=%d (tcgen05)\n", p.T, p.S, p.heads,
                     p.group, C::D, kRows, ctas);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem + (p.S + 1) * 4;
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&cfg, attn_prompt_kernel<B>, p) != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    return FG_OK;
}

}  // namespace

namespace fg {

int launch_attn_prompt(const AttnParams& p, int D, int sms, int pdl, cudaStream_t stream) {
    static_assert(kMaxRequests == kAttnPromptRequests, "requests of a launch");
    return D == 64 ? launch<2>(p, sms, pdl, stream) : D == 128 ? launch<4>(p, sms, pdl, stream) : launch<8>(p, sms, pdl, stream);
}

}  // namespace fg
