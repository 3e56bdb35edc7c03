// fg_attn_prompt.cu - attention of many new tokens a request over its 4-bit key/value cache, on the tensor
// cores of the fifth generation.
//
// An item (fg_attn.cuh) is 128 rows (new tokens x the query heads that share a kv head) of one request, or 256 in two row
// tiles of 128; per row tile and tile of kTok keys
//   S = Q K^T       tcgen05.mma, BF16, FP32 in tensor memory (two tiles of it, so the next product runs while a
//                   tile's exponentials are taken)
//   P = 2^(S - m)   in registers: two threads a row, half of the keys each, or a thread a row where there are two row
//                   tiles; m a running maximum that moves only when a score passes it by 2^8, because moving it
//                   scales O, which lives in tensor memory; P rounded once, to BF16 (2^-8 relative; no sum goes through it:
//                   l adds the unrounded weights)
//   O += P V        tcgen05.mma, BF16, FP32 in tensor memory
// Keys and values become BF16 tiles in shared memory once per item tile, exactly (a code has two significant bits,
// its scale is a power of two): 256 threads decode what 128 or 256 rows use.  Keys, values and Q stand as rows of 64
// elements in 128-byte swizzled atoms; a value tile is the product's MN-major operand as it is.
//
// Warps: 0-7 softmax and output (one row tile: warps w and w + 4 share 32 rows), 8 the MMA issuer, 9-16 the decoders.
// They meet at mbarriers (every wait is bounded, as in the GEMMs); a row's two threads meet at a barrier of their two
// warps, which both reach on every tile, also after a wait that ran out; pieces of items follow one another with a CTA
// barrier between.
//
// Bound: latency.  4 prompts of up to 512 tokens over 6000, 32 query heads on 4 of 128: 117 us (449 TFLOP/s; with
// other lengths of that range 87 to 148; items of one row tile 131), 2.9 us a key tile and pair of row tiles, with the tensor pipe at work in 27 % of it: decode, product,
// exponentials, product are one chain over four hand-offs, and each role's warps issue once in 4 clocks.  Without
// the decoders' arithmetic, the exponentials or half of the products a call is at most 8 % shorter, without all three 17 %.
#include <cuda_runtime.h>

#include <cstdio>
#include <type_traits>

#include "fg.h"
#include "fg_host.h"
#include "fg_attn.cuh"
#include "fg_gemm_kernel.cuh"

namespace {

using fg::AttnParams;
using fg::ex2;

constexpr int kSoftWarps = 8, kMmaWarp = 8, kDecodeWarp0 = 9, kDecodeWarps = 8;
constexpr int kThreads = 32 * (kDecodeWarp0 + kDecodeWarps);
constexpr int kWaitPrompt = 12;                // status code of a wait that ran out
constexpr float kSlack = 8.0f;                 // scores above m by at most this (log2): P <= 2^8
constexpr uint32_t kAll = fg::kAllLanes;

// RT row tiles of 128 rows: two share what is decoded (where tensor memory holds two O, and shared memory two Q).
template <int B, int RT>
struct Cfg {
    static constexpr int D = 32 * B, kSub = B / 2;               // sub-tiles of 64 elements
    static constexpr int kRows = 128 * RT;
    static_assert(RT == 1 || B <= 4, "tensor memory: two S of 128 columns, RT x D of O");
    static constexpr int kTok = B == 8 ? 64 : 128;               // keys of a tile
    static constexpr int kTile = kTok * 128 * kSub;              // bytes of a key or value tile
    static constexpr int kQ = 128 * 128 * kSub, kP = 128 * kTok * 2;      // of one row tile
    // one key tile (its product comes long before the next one is wanted), two of P; a second value tile where it fits
    static constexpr int kVStages = RT == 1 ? 2 : 1;
    static constexpr int kOffK = RT * kQ, kOffV = kOffK + kTile, kOffP = kOffV + kVStages * kTile, kOffBar = kOffP + 2 * kP;
    static constexpr int kNumBars = 14;
    static constexpr int kOffMisc = kOffBar + 8 * kNumBars;      // tensor memory address, abort flag, drain barrier
    static constexpr int kOffPre = kOffMisc + 16;
    static constexpr int kSmem = 1024 + kOffPre;                 // then [S + 1] int
    static constexpr int kCols = 256;                            // O's first column (S: 0 and 128)
    // columns of S of a softmax thread: RT == 1: warps w and w + 4 share 32 rows; RT == 2: a thread has a row
    static constexpr int kWide = RT == 1 ? kTok / 2 : kTok;
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
    uint32_t k[Cfg<B, 1>::kC][B], v[Cfg<B, 1>::kC][B];
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

template <int B, int RT>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const AttnParams p) {
    using C = Cfg<B, RT>;
    constexpr int D = C::D, kTok = C::kTok, kRows = C::kRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = fg::smem_u32(smem);
    __shared__ fg::AttnPlanSmem<kThreads> s_plan;
    __shared__ float s_top[2][128], s_l[2][128];               // of a row's two halves, or of two row tiles
    __shared__ int s_dead[kSoftWarps];
    __shared__ uint32_t s_absent[4][kDecodeWarps];             // of tile n in [n & 3], a decoder warp's tokens that have no page
    __shared__ fg::AttnCursor<kRows, C::kTok, kThreads, false> s_cur;  // while the roles run, out of their registers
    const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
    const uint32_t bar = sbase + C::kOffBar;
    const uint32_t k_full = bar, k_empty = bar + 8, v_full = bar + 16, v_empty = bar + 32, s_full = bar + 48, s_empty = bar + 64,
                   p_full = bar + 80, p_empty = bar + 96;                  // two of each but the first two
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    uint64_t* drain = reinterpret_cast<uint64_t*>(smem + C::kOffMisc + 8);
    int* s_pre = reinterpret_cast<int*>(smem + C::kOffPre);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            fg::mbar_init(v_full + 8 * i, kDecodeWarps);
            fg::mbar_init(v_empty + 8 * i, 1);
            fg::mbar_init(s_full + 8 * i, 1);
            fg::mbar_init(s_empty + 8 * i, kSoftWarps / RT);
            fg::mbar_init(p_full + 8 * i, kSoftWarps / RT);
            fg::mbar_init(p_empty + 8 * i, 1);
        }
        fg::mbar_init(k_full, kDecodeWarps);
        fg::mbar_init(k_empty, 1);
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
    auto wait = [&](uint32_t b, uint32_t parity) { return fg::wait_bar<false, false>(b, parity, wctl, kWaitPrompt); };

    fg::AttnCursor<kRows, kTok, kThreads, false> cur;
    const bool any = cur.open(p, s_plan, s_pre);
    uint32_t n0 = 0;                                           // tiles of the pieces before this one
    while (any) {
        int b0, b1;
        if (!cur.piece(s_plan, b0, b1)) break;
        const int h = cur.h, row0 = (cur.ch - s_pre[cur.r]) * kRows, rows = min(kRows, cur.rq.n * p.group - row0);
        const int first = cur.rq.len - cur.rq.n;               // position of new token 0
        const int* table = p.table + (long long)cur.r * p.max_pages;
        const bool empty = cur.keys.hi <= cur.keys.lo;
        const int t0 = cur.rq.t0, keys_lo = cur.keys.lo;
        if (tid == 0) s_cur = cur;
        const int tok0 = b0 * kTok, tok1 = empty ? tok0 : min(b1 * kTok, cur.keys.hi);
        const int tiles = (tok1 - tok0 + kTok - 1) / kTok;     // 0 where no row of the item has a key

        // Q: 16-byte chunks of the rows, zeros behind the last; all threads, four loads in flight
#pragma unroll 4
        for (int it = tid; it < kRows * (D / 8); it += kThreads) {
            const int j = it / (D / 8), ch = it % (D / 8);
            const int i = (row0 + j) / p.group, hq = h * p.group + (row0 + j) % p.group;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + ((long long)(t0 + i) * p.heads * p.group + hq) * D);
            const uint4 v = j < rows ? __ldcg(src + ch) : make_uint4(0, 0, 0, 0);
            st_shared_16(sbase + (j / 128) * C::kQ + (ch / 8) * (128 * 128) + (j % 128) * 128 + (((ch % 8) ^ (j & 7)) << 4), v);
        }
        fg::fence_proxy_async_smem();
        __syncthreads();

        float m = fg::kAttnEmpty, l = 0.0f;                    // of this thread's row, and of its half (softmax warps)
        if (warp >= kDecodeWarp0) {
            // ------------------------------------------------------------- decoders
            const int t = tid - 32 * kDecodeWarp0, my = t % kTok, c0 = t / kTok * C::kC;
            int page_i = (tok0 + my) / p.page, page_off = (tok0 + my) % p.page;
            const int step_page = kTok / p.page, step_off = kTok % p.page;
            // whether token tok's page is wanted, and its id (looked at only a tile later: nothing waits for it here)
            auto wanted = [&](int tok) { return tok < tok1 && (tok & ~15) + 16 > keys_lo; };
            auto page_at = [&](int tok) { return wanted(tok) ? static_cast<uint32_t>(table[page_i]) : ~0u; };
            auto load = [&](Raw<B>& x, uint32_t page, int off) {
                if (page < static_cast<uint32_t>(p.pages)) {
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
            auto fill = [&](const Raw<B>& x, uint32_t n, bool bad) {
                const uint32_t st = RT == 1 ? n & 1 : 0, ph = RT == 1 ? (n >> 1) & 1 : n & 1;   // of the value tiles
                const uint32_t absent = __ballot_sync(kAll, bad);
                if (absent && lane == 0) fg::kv_record(p.status, fg::kKvErrAttention);
                bool ok = wait(k_empty, (n & 1) ^ 1);
                if (!__all_sync(kAll, ok)) return false;
                if (lane == 0) s_absent[n & 3][warp - kDecodeWarp0] = absent;
                const uint32_t kt = sbase + C::kOffK, vt = sbase + C::kOffV + st * C::kTile;
#pragma unroll
                for (int i = 0; i < C::kC; ++i)
#pragma unroll
                    for (int b = 0; b < B; ++b) st_shared_16(kt + place(b, c0 + i), decode(x.k[i][b], scale_of<B>(x.ks, b)));
                fg::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && !(p.stall != 0 && n == 0 && warp == kDecodeWarp0)) fg::mbar_arrive(k_full);   // stalled: the MMA issuer times out
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
            int tok = tok0 + my, off = page_off;
            uint32_t page = page_at(tok);
            load(x, page, off);
            bool bad = wanted(tok) && page >= static_cast<uint32_t>(p.pages);
            auto look = [&]() {                                 // the page of the tile after the last one looked up
                advance();
                tok += kTok;
                off = page_off;
                page = page_at(tok);
            };
            look();
#pragma unroll 1
            for (int i = 0; i < tiles; ++i) {
                load(ahead, page, off);
                const bool bad_ahead = wanted(tok) && page >= static_cast<uint32_t>(p.pages);
                look();
                if (!fill(x, n0 + i, bad)) break;
                x = ahead;
                bad = bad_ahead;
            }
        } else if (warp == kMmaWarp) {
            // ----------------------------------------------------------- MMA issuer
            if (lane == 0) {
                constexpr uint32_t kIdS = idesc_bf16(128, kTok, false), kIdO = idesc_bf16(128, D, true);
                const uint64_t dq = fg::make_sdesc(sbase, 0, 1024, fg::kLayoutSw128);
                const uint64_t dk = fg::make_sdesc(sbase + C::kOffK, 0, 1024, fg::kLayoutSw128);
                const uint64_t dv = fg::make_sdesc(sbase + C::kOffV, kTok * 128, 1024, fg::kLayoutSw128);
                const uint64_t dp = fg::make_sdesc(sbase + C::kOffP, 0, 1024, fg::kLayoutSw128);
                // units: (tile, row tile); S and P of unit u stand in place u mod 2.  A unit's score product goes
                // ahead of the output product of the unit before it.
                for (int i = 0; i <= RT * tiles; ++i) {
                    if (i < RT * tiles) {
                        const uint32_t n = n0 + i / RT, u = RT * n0 + i, st = u & 1, ph = (u >> 1) & 1;
                        const int rt = i % RT;
                        if ((rt == 0 && !wait(k_full, n & 1)) || !wait(s_empty + 8 * st, ph ^ 1)) break;
                        fg::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4 * C::kSub; ++k)
                            tc_mma_bf16(tmem + st * 128, dq + rt * (C::kQ / 16) + (k / 4) * (128 * 128 / 16) + (k % 4) * 2,
                                        dk + (k / 4) * (kTok * 128 / 16) + (k % 4) * 2, kIdS, k != 0);
                        fg::tc_commit(s_full + 8 * st);
                        if (rt == RT - 1) fg::tc_commit(k_empty);
                    }
                    if (i > 0) {
                        const uint32_t n = n0 + (i - 1) / RT, u = RT * n0 + i - 1, st = u & 1, ph = (u >> 1) & 1;
                        const uint32_t vs = RT == 1 ? n & 1 : 0, vp = RT == 1 ? (n >> 1) & 1 : n & 1;
                        const int rt = (i - 1) % RT;
                        if ((rt == 0 && !wait(v_full + 8 * vs, vp)) || !wait(p_full + 8 * st, ph)) break;
                        fg::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kTok / 16; ++k)
                            tc_mma_bf16(tmem + C::kCols + rt * D, dp + st * (C::kP / 16) + (k / 4) * (128 * 128 / 16) + (k % 4) * 2,
                                        dv + vs * (C::kTile / 16) + k * (2048 / 16), kIdO, i > RT || k != 0);
                        if (rt == RT - 1) fg::tc_commit(v_empty + 8 * vs);
                        fg::tc_commit(p_empty + 8 * st);
                    }
                }
            }
            __syncwarp();
        } else {
            // ------------------------------- softmax: half a row's keys a thread, or (RT == 2) a row
            const int group = warp >> 2, my = (warp & 3) * 32 + lane;
            const int rt = RT == 1 ? 0 : group, col0 = RT == 1 ? group * C::kWide : 0;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const int hi = first + (row0 + rt * 128 + my) / p.group + 1, lo = fg::attn_from(p, hi);
            // keys that every row of the chunk looks at
            const int all_hi = first + row0 / p.group + 1;
            const int all_lo = fg::attn_from(p, first + (row0 + rows - 1) / p.group + 1);
            const uint32_t p_row = sbase + C::kOffP + (col0 / 64) * (128 * 128) + my * 128;
            for (int i = 0; i < tiles; ++i) {
                const uint32_t n = n0 + i, u = RT * n + rt, st = u & 1, ph = (u >> 1) & 1;
                const int base = tok0 + i * kTok;
                bool dead = !__all_sync(kAll, wait(s_full + 8 * st, ph));
                fg::tc_fence_after();
                const uint32_t at_s = tmem + lanes + st * 128 + col0;
                // tokens whose page is outside the cache (32 a decoder warp; a place is written again four tiles on, which
                // takes a key product that waits for this tile)
                uint32_t absent = 0;
#pragma unroll
                for (int x = 0; x < kTok / 32; ++x) absent |= s_absent[n & 3][x];
                const bool border = absent != 0 || base < all_lo || base + kTok > all_hi;
                // P's place is free once the product of the tile before the last is done
                dead = dead || !__all_sync(kAll, wait(p_empty + 8 * st, ph ^ 1));
                // One pass over the scores, 16 columns ahead on their way: weights under the present m, their sum, the
                // largest score.  Where that one passes m by more than kSlack, m moves and the pass is done again.
                float top, sum;
                auto weights = [&](auto rounded, int c, uint32_t (&r)[16]) {
                    constexpr bool kRounded = decltype(rounded)::value;
                    if (border) {                               // bit x: column c + x counts
                        const int at = base + col0 + c;
                        const int from = min(max(lo - at, 0), 16), to = min(max(hi - at, 0), 16);
                        const uint32_t keep = (1u << to) - (1u << min(from, to)) & ~(s_absent[n & 3][(col0 + c) / 32] >> ((col0 + c) & 31));
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (!(keep >> x & 1u)) r[x] = 0xFF800000u;
                    }
                    float part[2] = {0.0f, 0.0f}, most[2] = {__uint_as_float(r[0]), __uint_as_float(r[1])};
#pragma unroll
                    for (int x = 0; x < 16; x += 8) {
                        uint32_t o[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float s0 = __uint_as_float(r[x + 2 * y]), s1 = __uint_as_float(r[x + 2 * y + 1]);
                            most[0] = fmaxf(most[0], s0);
                            most[1] = fmaxf(most[1], s1);
                            const float w0 = ex2(kRounded ? __fmul_rn(s0, p.scale_log2) - m : fmaf(s0, p.scale_log2, -m));
                            const float w1 = ex2(kRounded ? __fmul_rn(s1, p.scale_log2) - m : fmaf(s1, p.scale_log2, -m));
                            part[0] += w0;
                            part[1] += w1;
                            const __nv_bfloat162 w = __floats2bfloat162_rn(w0, w1);
                            o[y] = *reinterpret_cast<const uint32_t*>(&w);
                        }
                        st_shared_16(p_row + st * C::kP + (c / 64) * (128 * 128) + (((((col0 + c) % 64 + x) / 8) ^ (my & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
                    }
                    sum += part[0] + part[1];
                    top = fmaxf(top, fmaxf(most[0], most[1]));
                };
                auto pass = [&](auto rounded) {
                    top = -INFINITY;
                    sum = 0.0f;
                    uint32_t ra[16], rb[16];
                    fg::tmem_ld_32x32b_x16(at_s, ra);
                    fg::tmem_wait_ld();
#pragma unroll 1
                    for (int c = 0; c < C::kWide; c += 32) {
                        fg::tmem_ld_32x32b_x16(at_s + c + 16, rb);
                        weights(rounded, c, ra);
                        fg::tmem_wait_ld();
                        if (c + 32 < C::kWide) fg::tmem_ld_32x32b_x16(at_s + c + 32, ra);
                        weights(rounded, c + 16, rb);
                        fg::tmem_wait_ld();
                    }
                    top *= p.scale_log2;
                };
                pass(std::false_type{});
                // m is rounded, which a large score minus m would be off by (past 2^30 beyond what a weight holds): then the pass
                // is done again with rounded scores.  That costs every pass 4 us of 116 where it is always done.
                const bool large = fabsf(m) > 0x1p20f && m > fg::kAttnEmpty;
                const bool rise = dead || large || top > m + kSlack;
                if (RT == 1 ? pair_any(1 + (warp & 3), rise) : __any_sync(kAll, rise)) {
                    float both = top;
                    if constexpr (RT == 1) {
                        // O is whole once the last tile's product is done (RT == 2: that is the wait above)
                        if (n > 0) dead = dead || !__all_sync(kAll, wait(p_empty + 8 * (st ^ 1), ((n - 1) >> 1) & 1));
                        s_top[group][my] = top;
                        if (lane == 0) s_dead[warp] = dead;
                        pair_any(1 + (warp & 3), false);
                        both = fmaxf(top, s_top[group ^ 1][my]);
                        dead = dead || s_dead[warp ^ 4];
                    }
                    if (dead) break;
                    const float now = both > m + kSlack ? both : m, f = ex2(m - now);
                    m = now;
                    l *= f;
                    if (i > 0) {
                        fg::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D * RT / 2; c += 32) {
                            uint32_t x[32];
                            const uint32_t at = tmem + lanes + C::kCols + group * (D * RT / 2) + c;   // RT == 1: a half each
                            fg::tmem_ld_32x32b_x32(at, x);
                            fg::tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 32; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * f);
                            tmem_st_32x32b_x32(at, x);
                        }
                        tmem_wait_st();
                    }
                    if (RT == 1) pair_any(1 + (warp & 3), false);   // both have read before either writes again
                    pass(std::true_type{});
                }
                l += sum;
                fg::tc_fence_before();
                fg::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    fg::mbar_arrive(s_empty + 8 * st);
                    fg::mbar_arrive(p_full + 8 * st);
                }
            }
            if (tiles > 0) {
                const uint32_t u = RT * (n0 + tiles - 1) + rt;
                const bool ok = wait(p_empty + 8 * (u & 1), (u >> 1) & 1);
                (void)ok;                                       // on a time-out the abort flag is up: the output is not stored
                __syncwarp();
                fg::tc_fence_after();
            }
            s_l[group][my] = l;
        }
        __syncthreads();
        if (*abort_flag) break;
        n0 += tiles;
        cur = s_cur;
        const int row_0 = (cur.ch - s_pre[cur.r]) * kRows, rows_ = min(kRows, cur.rq.n * p.group - row_0);
        const bool none = cur.keys.hi <= cur.keys.lo;

        // ------------------------------------------------------------------ output
        int a, z;
        cur.holders(s_plan, a, z);
        const bool whole = a == z;
        if (warp < kSoftWarps) {
            const int group = warp >> 2, at = (warp & 3) * 32 + lane, my = RT == 1 ? at : group * 128 + at;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const float sum = RT == 1 ? s_l[0][at] + s_l[1][at] : l;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            float* slot = fg::attn_piece<kRows, D>(p, blockIdx.x, a);
            if (!whole && (RT == 2 || group == 0) && my < rows_) {
                slot[my] = m;
                slot[kRows + my] = sum;
            }
            const int i = (row_0 + my) / p.group, hq = cur.h * p.group + (row_0 + my) % p.group;
            uint16_t* out = p.out + ((long long)(cur.rq.t0 + i) * p.heads * p.group + hq) * D;
#pragma unroll 1
            for (int x0 = 0; x0 < D * RT / 2; x0 += 32) {
                const int c = RT == 1 ? group * (D / 2) + x0 : x0;
                uint32_t r[32];
                if (!none) {
                    fg::tmem_ld_32x32b_x32(tmem + lanes + C::kCols + (RT == 1 ? 0 : group * D) + c, r);
                    fg::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) r[x] = 0;
                }
                if (my < rows_ && whole) {
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
                } else if (my < rows_) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        *reinterpret_cast<float4*>(slot + 2 * kRows + ((c / 4 + x) * kRows + my) * 4) =
                            make_float4(__uint_as_float(r[4 * x]), __uint_as_float(r[4 * x + 1]), __uint_as_float(r[4 * x + 2]), __uint_as_float(r[4 * x + 3]));
                }
            }
            fg::tc_fence_before();
        }
        if (!whole) fg::attn_join<kRows, D, kThreads, true>(p, s_plan, a, z, cur.rq.t0, cur.h, row_0, rows_);
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

template <int B, int RT>
int launch(const AttnParams& p, int sms, int pdl, cudaStream_t stream) {
    using C = Cfg<B, RT>;
    static bool configured[256] = {};        // set once per device; setting it again is harmless
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(attn_prompt_kernel<B, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem + (kMaxRequests + 1) * 4) !=
            cudaSuccess) {
            cudaGetLastError();
            return FG_ERR_CUDA;
        }
        configured[dev] = true;
    }
    const int ctas = sms < fg::kAttnPromptCtas ? sms : fg::kAttnPromptCtas;
    if (fg::print_configs_enabled())
        std::fprintf(stderr, "[fg] paged_attention_mxfp4 T=%d S=%d heads=%d x %d D=%d rows=%d grid=%d (tcgen05)\n", p.T, p.S, p.heads,
                     p.group, C::D, C::kRows, ctas);
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
    if (cudaLaunchKernelEx(&cfg, attn_prompt_kernel<B, RT>, p) != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    return FG_OK;
}

}  // namespace

namespace fg {

int launch_attn_prompt(const AttnParams& p, int D, int rows, int sms, int pdl, cudaStream_t stream) {
    static_assert(kMaxRequests == kAttnPromptRequests, "requests of a launch");
    if (rows == 128)
        return D == 64 ? launch<2, 1>(p, sms, pdl, stream) : D == 128 ? launch<4, 1>(p, sms, pdl, stream) : launch<8, 1>(p, sms, pdl, stream);
    return D == 64 ? launch<2, 2>(p, sms, pdl, stream) : launch<4, 2>(p, sms, pdl, stream);
}

}  // namespace fg
