// fg_attn.cu - attention of each request's new tokens over its 4-bit key/value cache.
//
// Mathematics.  For the R = group x new-token rows that share a kv head, with keys k_j = sum over blocks b of
// s_jb * (codes), per 16 tokens:
//   S^T = K Q^T      16 tokens x 8 rows per mma (m16n8k16, FP16 codes, FP16 q scaled to [2^8, 2^9) by a
//                    power of two per row: exact down to 2^-22 of the row's largest element, off by up to 2^-33 of it
//                    below); one FP32 accumulator per block of 32, then times s_jb
//   w_jb = 2^(S_j - M) * t_jb      t_jb: the value's block scale; M follows the maximum of S_j + max_b log2 t_jb,
//                    so that w <= 2^15 in FP16 however far the scales of different tokens lie apart
//   O^T += V^T W^T   32 elements of block b x 16 tokens x 8 rows, FP16 codes, FP32 accumulators
//   l   += 2^(S_j - M),   o = O / l
// M moves only when some w might pass 2^15 (a vote a tile), to where the largest is 2^8; then O and l are scaled.
// A weight is rounded once, to FP16: by 2^-11 of itself, or by 2^-33 of the row's largest w where that is more.  M
// speaks for all blocks, so that is 2^-25 of a block's own largest w as long as the scales of a token lie within 2^8 of each
// other.  From the first tile on in which they do not (the same vote), or in which a score passes 2^20 (whose rounding then
// is more than FP16's range takes), a warp multiplies its piece's weights and values in FP32 on the CUDA cores, M the largest
// score: called alone, 64 requests of up to 8192 tokens then take 233 us for 69, one of 131072 129 for 44.
// The looks cost 0.7 of 67.7 us (D = 64: 1.1 of 46.2); with the FP32 products in the same loop it was 4.3 (registers).
//
// Work.  An item (fg_attn.cuh: request, chunk of kRows rows, kv head) is walked in blocks of 128 tokens, of which each of
// a CTA's eight warps takes 16 with accumulators of its own, joined at the end through shared memory.  Codes and scales
// come through a ring of kStages tiles of 16 tokens that each warp has to itself (asynchronous 16-byte copies, no
// barrier of the CTA); the cache's order puts what a lane needs of a row into one load, and sixteen tokens never
// cross a page.  Three stages: with four 64 requests of up to 8192 tokens, 64 query heads on 8 of 128, took 0.3 us longer,
// with five 1.9; one of 131072 0.5 and 1.6.
//
// Bound: the ALU pipe (conversions of codes, which take 52 % of it over a launch and more inside the loop) beside HBM
// bytes: the loop streams at 6.3 TB/s, all of a launch at 4.2 (64 requests of up to 8192 tokens 67.7 us, one of 131072
// 38.4); the rest is the cut (2.2 us: every CTA scans the lengths), q and the first pages (3), joins (1 to 4) and the last
// CTAs' tail.  FP16 codes on mma.sync: its 1022 products a clock and SM suffice for few rows, and E4M3 operands would leave
// a weight four significant bits.
#include <cuda_runtime.h>

#include <cstdio>
#include <type_traits>

#include "fg.h"
#include "fg_host.h"
#include "fg_attn.cuh"

namespace {

using fg::al;
using fg::AttnParams;
using fg::ex2;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlock = 16 * kWarps;           // tokens of a block
constexpr float kEmpty = fg::kAttnEmpty;
constexpr float kBias = 8.0f, kMostW = 32768.0f;   // w: 2^8 where M has just moved, at most 2^15
constexpr uint32_t kAll = fg::kAllLanes;

template <int B, int NT>
struct Cfg {
    static constexpr int D = 32 * B, kRows = 8 * NT;
    static constexpr int kPad = D + 4;         // floats of a row in shared memory: conflict-free 16-byte stores
    static constexpr int kJoin = kWarps * kRows * kPad * 4;
    // a warp's ring: per tile 16 key rows, 16 value rows, their scales
    static constexpr int kStages = 3;
    static constexpr int kTileV = 16 * 16 * B, kTileKs = 2 * kTileV, kTileVs = kTileKs + 16 * B, kTile = kTileVs + 16 * B;
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kMain = kJoin > kRing ? kJoin : kRing;          // the join comes when the ring is empty
    static constexpr int kPerSm = NT * B <= 4 ? 2 : 1;                   // CTAs: 128 registers a thread
    static constexpr bool kParked = NT > 1 && kPerSm == 2;
    static constexpr bool kQShared = NT > 1;                             // q in shared memory: registers hold O
    static constexpr int kQ = kQShared ? NT * B * 32 * 16 : 0;
    static constexpr int kSmem = kMain + kQ;                             // then [S + 1] int
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same without a sum before it.
__device__ __forceinline__ void mma_f16_new(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Byte i (two codes) of w as an FP16 pair.
__device__ __forceinline__ uint32_t e2m1x2_f16(uint32_t w, int i) {
    uint32_t r;
    if (i == 0) asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if (i == 1) asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if (i == 2) asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ void f16x2_f32(uint32_t h, float& lo, float& hi) {
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h));
}
// Transposes an 8 x 8 matrix of 16-bit values (row i / 4, columns 2 (i mod 4) and + 1 in lane i).
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// A tile's token that stands in row g (and, plus 8, in row g + 8) of the products, and the swizzle of a row's
// 16-byte chunks: chosen so that the lanes which a shared-memory phase serves together, those of two (D = 64:
// four) neighbouring g of a key row and those of four c of a value row, find their words in different banks.
template <int B>
__device__ __forceinline__ int token_of(int g) {
    if (B == 2) return (g & 1) ? 4 + (((g >> 1) + 2) & 3) : g >> 1;
    if (B == 4) return g ^ (g >> 2 & 1);
    return g;
}
template <int B>
__device__ __forceinline__ int swizzle(int t) {
    return B == 2 ? 0 : B == 4 ? (t & 2) : (t & 7);
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&r)[N], uint32_t addr) {
    if constexpr (N == 1) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(addr) : "memory");
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
    } else {
        static_assert(N == 4, "one load");
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    }
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Key words (column group c of the row at `row`): B of them.
template <int B>
__device__ __forceinline__ void load_key(uint32_t (&r)[B], uint32_t row, int sw, int c) {
    if constexpr (B == 8) {
        uint32_t lo[4], hi[4];
        load_words(lo, row + 16 * ((2 * c) ^ sw));
        load_words(hi, row + 16 * ((2 * c + 1) ^ sw));
#pragma unroll
        for (int i = 0; i < 4; ++i) { r[i] = lo[i]; r[4 + i] = hi[i]; }
    } else {
        load_words(r, B == 4 ? row + 16 * (c ^ sw) : row + 8 * c);
    }
}
// Value words (row group g of the row at `row`): B / 2 of them.
template <int B>
__device__ __forceinline__ void load_value(uint32_t (&r)[B / 2], uint32_t row, int sw, int g) {
    load_words(r, row + (B == 8 ? 16 * (g ^ sw) : B == 4 ? 16 * ((g >> 1) ^ sw) + 8 * (g & 1) : 4 * g));
}
template <int B>
__device__ __forceinline__ void load_scales(uint32_t (&r)[(B + 3) / 4], uint32_t addr) {
    if constexpr (B == 2) {
        uint16_t h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr) : "memory");
        r[0] = h;
    } else {
        load_words(r, addr);
    }
}

// The B scales of a token as floats.  A byte's exponent as BF16 is byte << 7, so a mask and a product give two
// at once (products and sums run beside the ALU pipe, which the conversions fill).
template <int B>
__device__ __forceinline__ void scales_of(float (&f)[B], const uint32_t (&s)[(B + 3) / 4]) {
#pragma unroll
    for (int i = 0; i < B; i += 4) {
        const uint32_t w = s[i / 4], even = (w & 0x00FF00FFu) * 128u, odd = (w >> 1) & 0x7F807F80u;
        f[i] = __uint_as_float(even * 65536u);
        f[i + 1] = __uint_as_float(odd * 65536u);
        if (B > 2) {
            f[i + 2] = __uint_as_float(even & 0xFFFF0000u);
            f[i + 3] = __uint_as_float(odd & 0xFFFF0000u);
        }
    }
}
// Exponent of a token's largest scale (at least the smallest that the cache holds).
template <int B>
__device__ __forceinline__ float top_exponent(const float (&f)[B]) {
    float m = f[0];
#pragma unroll
    for (int b = 1; b < B; ++b) m = fmaxf(m, f[b]);
    const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
    return static_cast<float>(max(e, fg::kKvMinExp));
}

// Whether a token's B scales are more than 2^8 apart, at the latest: B sum e^2 - (sum e)^2, the squared differences of its
// exponents over all pairs, is at least B / 2 times the largest of them.
template <int B>
__device__ __forceinline__ bool scales_apart(const uint32_t (&s)[(B + 3) / 4]) {
    uint32_t sum = 0, squares = 0;
#pragma unroll
    for (int i = 0; i < (B + 3) / 4; ++i) {
        sum = __dp4a(s[i], 0x01010101u, sum);
        squares = __dp4a(s[i], s[i], squares);
    }
    return B * squares > sum * sum + 32 * B;
}

template <int B, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<B, NT>::kPerSm) attn_kernel(const AttnParams p) {
    using C = Cfg<B, NT>;
    constexpr int D = C::D, kRows = C::kRows, kPad = C::kPad;
    extern __shared__ __align__(16) uint8_t smem[];
    float* s_join = reinterpret_cast<float*>(smem);                       // [kWarps][kRows][kPad]
    uint4* s_q = reinterpret_cast<uint4*>(smem + C::kMain);               // [NT][B][32]
    int* s_pre = reinterpret_cast<int*>(smem + C::kSmem);                 // [S + 1] chunks before a request
    __shared__ float s_qs[kRows];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ fg::AttnPlanSmem<kThreads> s_plan;
    __shared__ fg::AttnCursor<kRows, kBlock, kThreads, true> s_cur;       // kParked: out of the tiles' registers
    const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31, g = lane >> 2, c = lane & 3;
    const uint32_t smem_base = fg::smem_u32(smem);
    fg::grid_dependency_wait();
    if (tid == 0) fg::grid_launch_dependents();

    fg::AttnCursor<kRows, kBlock, kThreads, true> cur;
    if (!cur.open(p, s_plan, s_pre)) return;

    // what a lane copies of a tile (16-byte chunk `lane`, and every 32nd on) and where it finds its operands in one
    const uint32_t page_rows = static_cast<uint32_t>(p.heads) * p.page;
    const int step_page = kBlock / p.page, step_off = kBlock % p.page;
    const uint32_t ring = smem_base + warp * (C::kStages * C::kTile);
    const uint32_t cp_dst = ring + (lane / B) * (16 * B) + 16 * ((lane % B) ^ swizzle<B>(lane / B));
    const uint32_t cp_dst_odd = ring + (lane / B) * (16 * B) + 16 * ((lane % B) ^ swizzle<B>(lane / B) ^ 4);
    const uint32_t cp_sf = ring + C::kTileKs + 16 * lane;
    const uint8_t* sf_lane = lane < B ? p.ks + 16 * lane : p.vs + 16 * (lane - B);
    const int tau = token_of<B>(g), tau0 = token_of<B>(2 * c), tau1 = token_of<B>(2 * c + 1);
    const uint32_t at_sf = ring + C::kTileKs + tau * B;
    const uint32_t at_k = ring + tau * (16 * B), at_v0 = ring + C::kTileV + tau0 * (16 * B), at_v1 = ring + C::kTileV + tau1 * (16 * B);

    // ---------------------------------------------------------------- pieces of items
    while (true) {
        int b0, b1;
        if (!cur.piece(s_plan, b0, b1)) break;
        const int h = cur.h;
        const int row0 = (cur.ch - s_pre[cur.r]) * kRows, rows = min(kRows, cur.rq.n * p.group - row0);
        const int first = cur.rq.len - cur.rq.n;                               // position of new token 0
        const int* table = p.table + (long long)cur.r * p.max_pages;
        const uint32_t head_row = static_cast<uint32_t>(h) * p.page;
        const int keys_lo = cur.keys.lo, keys_hi = cur.keys.hi, row_t0 = cur.rq.t0;
        if (C::kParked && tid == 0) s_cur = cur;

        // keys that every row of the chunk looks at: tiles inside need no mask
        const int i_first = row0 / p.group, i_last = (row0 + rows - 1) / p.group;
        const int all_hi = first + i_first + 1, all_lo = max(0, fg::attn_back(p, first + i_last + 1));
        // this warp's tiles: tokens 16 * (8 * block + warp)
        int base = b0 * kBlock + 16 * warp;
        const int base_end = keys_hi > keys_lo ? min(b1 * kBlock, keys_hi) : 0;
        if (base + 16 <= keys_lo) base += kBlock;
        // page and offset of the next tile to look up: a warp's tiles are kBlock tokens apart
        int look_page = base / p.page, look_off = base % p.page;
        auto next_page = [&](int tok, uint32_t& page, uint32_t& off) {
            page = tok < base_end ? static_cast<uint32_t>(table[look_page]) : ~0u;
            off = head_row + look_off;
            look_page += step_page;
            look_off += step_off;
            if (look_off >= p.page) { look_off -= p.page; ++look_page; }
        };
        // copies of a tile into a stage; a page outside the cache is not read and counts as masked
        auto issue = [&](uint32_t page, uint32_t off, int stage, bool wanted) {
            const bool ok = page < static_cast<uint32_t>(p.pages);
            if (ok) {
                // row of the tile's first token: (page * heads + h) * page_size + offset
                const unsigned long long row = (unsigned long long)page * page_rows + off;
                const unsigned long long at = row * (16 * B) + 16 * lane;
                const uint8_t *k = p.kc + at, *v = p.vc + at;
#pragma unroll
                for (int i = 0; i < B / 2; ++i) {
                    // 32 chunks on, 32 / B tokens: B = 8 swizzles four tokens on with another bit
                    const uint32_t dst = (B == 8 && (i & 1) ? cp_dst_odd : cp_dst) + stage * C::kTile + 512 * i;
                    cp_async_16(dst, k + 512 * i);
                    cp_async_16(dst + C::kTileV, v + 512 * i);
                }
                if (lane < 2 * B) cp_async_16(cp_sf + stage * C::kTile, sf_lane + row * B);
            } else if (wanted && lane == 0) {
                fg::kv_record(p.status, fg::kKvErrAttention);
            }
            cp_async_commit();
            return ok;
        };
        // q of row tile nt: rows nt * 8 + g, elements 32 b + 8 c .. + 7; then as FP16 times 2^x, with 2^-x * scale
        auto load_q = [&](int nt, uint4 (&raw)[B]) {
            const int j = row0 + nt * 8 + g;
#pragma unroll
            for (int b = 0; b < B; ++b) raw[b] = make_uint4(0, 0, 0, 0);
            if (nt * 8 + g < rows) {
                const int i = j / p.group, hq = h * p.group + j % p.group;
                const uint16_t* src = p.q + ((long long)(row_t0 + i) * p.heads * p.group + hq) * D + 8 * c;
#pragma unroll
                for (int b = 0; b < B; ++b) raw[b] = __ldcg(reinterpret_cast<const uint4*>(src + 32 * b));
            }
        };
        auto convert_q = [&](const uint4 (&raw)[B], uint32_t (&f)[B][4]) {
            float amax = 0.0f;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
            }
            amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
            const int x = min(126, 8 + 127 - static_cast<int>(__float_as_uint(amax) >> 23));
            const float up = __uint_as_float(static_cast<uint32_t>(x + 127) << 23);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[b][i] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
            }
            // never 0, which a masked score's -inf must not meet; below 2^-126 no score (at most 2^82 before) counts
            return fmaxf(__uint_as_float(static_cast<uint32_t>(127 - x) << 23) * p.scale_log2, 0x1p-126f);
        };
        // One after another in flight: q, the pages of the first tiles, those tiles.
        uint4 raw[B];
        if (!C::kQShared || warp < NT) load_q(C::kQShared ? warp : 0, raw);
        uint32_t absent = 0;                                // bit: the stage's tile has no page; a tile left to the FP32 loop: its stage + 1, from bit 8 on
        uint32_t page, off;
        {
            uint32_t pages[C::kStages - 1], offs[C::kStages - 1];
#pragma unroll
            for (int i = 0; i < C::kStages - 1; ++i) next_page(base + i * kBlock, pages[i], offs[i]);
            next_page(base + (C::kStages - 1) * kBlock, page, off);
#pragma unroll
            for (int i = 0; i < C::kStages - 1; ++i)
                if (!issue(pages[i], offs[i], i, base + i * kBlock < base_end)) absent |= 1u << i;
        }
        uint32_t qf[C::kQShared ? 1 : B][4];
        float qs1[C::kQShared ? 1 : NT][2];
        auto qs = [&](int nt, int k) { return C::kQShared ? s_qs[nt * 8 + 2 * c + k] : qs1[C::kQShared ? 0 : nt][k]; };
        if constexpr (C::kQShared) {
            static_assert(NT <= kWarps, "a row tile a warp");
            if (warp < NT) {
                uint32_t f[B][4];
                const float down = convert_q(raw, f);
#pragma unroll
                for (int b = 0; b < B; ++b) s_q[(warp * B + b) * 32 + lane] = make_uint4(f[b][0], f[b][1], f[b][2], f[b][3]);
                if (c == 0) s_qs[warp * 8 + g] = down;
            }
            __syncthreads();
        } else {
            const float down = convert_q(raw, qf);
            qs1[0][0] = __shfl_sync(kAll, down, 8 * c);
            qs1[0][1] = __shfl_sync(kAll, down, 8 * c + 4);
        }

        float o[NT][2 * B][4], l[NT][2], m[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2 * B; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
            l[nt][0] = l[nt][1] = 0.0f;
            m[nt][0] = m[nt][1] = kEmpty;
        }

        // A tile.  False: a token's value scales are far apart, nothing is done yet, and kApart has to do it.
        // M up to the largest of the lanes' `top`, where that is more.
        auto move = [&](int nt, int k, float top) {
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, i));
            top = fmaxf(top, m[nt][k]);
            const float f = ex2(m[nt][k] - top);
            m[nt][k] = top;
            l[nt][k] *= f;
#pragma unroll
            for (int i = 0; i < 2 * B; ++i) {
                o[nt][i][k] *= f;
                o[nt][i][2 + k] *= f;
            }
        };
        auto compute = [&](auto is_apart, int stage, int tok0, bool ok) {
            constexpr bool kApart = decltype(is_apart)::value;
            const uint32_t at = stage * C::kTile;
            uint32_t ks0[(B + 3) / 4], ks1[(B + 3) / 4], vs0[(B + 3) / 4], vs1[(B + 3) / 4];
            load_scales<B>(ks0, at_sf + at);
            load_scales<B>(ks1, at_sf + at + 8 * B);
            load_scales<B>(vs0, at_sf + at + 16 * B);
            load_scales<B>(vs1, at_sf + at + 24 * B);
            uint32_t k0[B], k1[B];
            load_key<B>(k0, at_k + at, swizzle<B>(tau), c);
            load_key<B>(k1, at_k + at + 128 * B, swizzle<B>(tau), c);
            float s[NT][4];
            float f0[B], f1[B];
            scales_of<B>(f0, ks0);
            scales_of<B>(f1, ks1);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                uint32_t a[4], e[4];
                fg::e2m1x8_f16(k0[b], a);
                fg::e2m1x8_f16(k1[b], e);
                const float s0 = f0[b], s1 = f1[b];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x[4];
                    uint4 f;
                    if constexpr (C::kQShared) f = s_q[(nt * B + b) * 32 + lane];
                    else f = make_uint4(qf[b][0], qf[b][1], qf[b][2], qf[b][3]);
                    mma_f16_new(x, a[0], e[0], a[1], e[1], f.x, f.y);
                    mma_f16(x, a[2], e[2], a[3], e[3], f.z, f.w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[nt][i] = b == 0 ? x[i] * (i < 2 ? s0 : s1) : fmaf(x[i], i < 2 ? s0 : s1, s[nt][i]);
                }
            }
            if (!ok || tok0 < all_lo || tok0 + 16 > all_hi) {                  // a border: mask
                const int t0 = tok0 + tau, t1 = t0 + 8;
                const bool in0 = ok && t0 >= keys_lo && t0 < keys_hi, in1 = ok && t1 >= keys_lo && t1 < keys_hi;
#pragma unroll
                for (int i = 0; i < (B + 3) / 4; ++i) {                        // scales behind the keys may be anything
                    if (!in0) vs0[i] = 0;
                    if (!in1) vs1[i] = 0;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int i = (row0 + nt * 8 + 2 * c + k) / p.group;
                        const int hi = first + i + 1, lo = fg::attn_back(p, hi);
                        if (!(in0 && t0 >= lo && t0 < hi)) s[nt][k] = -INFINITY;
                        if (!(in1 && t1 >= lo && t1 < hi)) s[nt][2 + k] = -INFINITY;
                    }
            }
            uint32_t mine[(B + 3) / 4];                         // two of the four lanes that have a token's scales look at them
#pragma unroll
            for (int i = 0; i < (B + 3) / 4; ++i) mine[i] = (c & 1) ? vs1[i] : vs0[i];
            bool far = scales_apart<B>(mine);
            scales_of<B>(f0, vs0);
            scales_of<B>(f1, vs1);
            float w[NT][4];
            if constexpr (kApart) {                             // as usual: M is the largest score
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // rounded before the difference, so that it is 0 for the largest, whatever its size
                        const float s0 = __fmul_rn(s[nt][k], qs(nt, k)), s1 = __fmul_rn(s[nt][2 + k], qs(nt, k));
                        move(nt, k, fmaxf(s0, s1));
                        w[nt][k] = ex2(s0 - m[nt][k] + kBias);
                        w[nt][2 + k] = ex2(s1 - m[nt][k] + kBias);
                    }
            } else {
                auto weights = [&]() {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            w[nt][k] = ex2(fmaf(s[nt][k], qs(nt, k), kBias - m[nt][k]));
                            w[nt][2 + k] = ex2(fmaf(s[nt][2 + k], qs(nt, k), kBias - m[nt][k]));
                        }
                };
                weights();
                // no weight times scale is above the sum of all
                float sum0 = f0[0], sum1 = f1[0];
#pragma unroll
                for (int b = 1; b < B; ++b) { sum0 += f0[b]; sum1 += f1[b]; }
                bool over = far;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    over |= !(fmaf(w[nt][0], sum0, fmaf(w[nt][1], sum0, fmaf(w[nt][2], sum1, w[nt][3] * sum1))) <= kMostW);
                if (__any_sync(kAll, over)) {
                    // a score past 2^20 leaves no room for the scales in M, nor FP16's range to what M is rounded by
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x = s[nt][i] * qs(nt, i & 1);
                            far |= fabsf(x) > 0x1p20f && x > -INFINITY;
                        }
                    if (__any_sync(kAll, far)) return false;
                    const float e0 = top_exponent<B>(f0), e1 = top_exponent<B>(f1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) move(nt, k, fmaxf(fmaf(s[nt][k], qs(nt, k), e0), fmaf(s[nt][2 + k], qs(nt, k), e1)));
                    weights();
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                l[nt][0] += w[nt][0] + w[nt][2];
                l[nt][1] += w[nt][1] + w[nt][3];
            }
            if constexpr (kApart) {
#pragma unroll 1
                for (int t = 0; t < 8; ++t) {
                    const int from = 4 * t + c, row = token_of<B>(t);     // the lane that has this token's weights
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t v[B / 2];
                        load_value<B>(v, ring + at + C::kTileV + row * (16 * B) + 128 * B * i, swizzle<B>(row), g);
                        float u[NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int k = 0; k < 2; ++k) u[nt][k] = __shfl_sync(kAll, w[nt][2 * i + k], from);
#pragma unroll
                        for (int b = 0; b < B; ++b) {
                            const float f = __shfl_sync(kAll, i ? f1[b] : f0[b], from);
                            float x[4];
                            f16x2_f32(e2m1x2_f16(v[b / 2], 2 * (b & 1)), x[0], x[1]);
                            f16x2_f32(e2m1x2_f16(v[b / 2], 2 * (b & 1) + 1), x[2], x[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float uf = u[nt][k] * f;
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        o[nt][2 * b + j / 2][2 * (j & 1) + k] = fmaf(uf, x[j], o[nt][2 * b + j / 2][2 * (j & 1) + k]);
                                }
                        }
                    }
                }
                return true;
            }
            uint32_t even[2][B / 2], odd[2][B / 2];            // row group g of tokens 2c and 2c + 1, 2c + 8 and 2c + 9
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t v0[B / 2], v1[B / 2];
                load_value<B>(v0, at_v0 + at + 128 * B * i, swizzle<B>(tau0), g);
                load_value<B>(v1, at_v1 + at + 128 * B * i, swizzle<B>(tau1), g);
#pragma unroll
                for (int j = 0; j < B / 2; ++j) {
                    even[i][j] = (v0[j] & 0x0F0F0F0Fu) | (v1[j] * 16u & 0xF0F0F0F0u);
                    odd[i][j] = (v0[j] >> 4 & 0x0F0F0F0Fu) | (v1[j] & 0xF0F0F0F0u);
                }
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                uint32_t wb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    wb[nt][0] = movmatrix(pack_f16(w[nt][0] * f0[b], w[nt][1] * f0[b]));
                    wb[nt][1] = movmatrix(pack_f16(w[nt][2] * f1[b], w[nt][3] * f1[b]));
                }
                // half word b of the four tokens, zipped: byte 2 (b mod 2) + i holds code 2 i (even) or 2 i + 1
                // (odd) of a pair of tokens, which one conversion makes an operand's pair
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int at = 2 * (b & 1) + i;
                    const uint32_t a0 = e2m1x2_f16(even[0][b / 2], at), a1 = e2m1x2_f16(odd[0][b / 2], at);
                    const uint32_t a2 = e2m1x2_f16(even[1][b / 2], at), a3 = e2m1x2_f16(odd[1][b / 2], at);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][2 * b + i], a0, a1, a2, a3, wb[nt][0], wb[nt][1]);
                }
            }
            return true;
        };
        // Waits for the tile in `stage` and sends for the one kAhead tiles on.
        constexpr int kAhead = C::kStages - 1;
        auto advance = [&](int stage) {
            constexpr uint32_t kBits = (1u << C::kStages) - 1;
            const int next = (stage + kAhead) % C::kStages;
            const bool ok = issue(page, off, next, base + kAhead * kBlock < base_end);
            absent = (absent & (kBits ^ 1u << next)) | (ok ? 0u : 1u << next);
            next_page(base + C::kStages * kBlock, page, off);
            cp_async_wait<kAhead>();
            __syncwarp();
        };

        while (base < base_end) {
#pragma unroll
            for (int i = 0; i < C::kStages; ++i) {          // stages at fixed places
                advance(i);
                if (!compute(std::false_type{}, i, base, !(absent >> i & 1u))) {
                    absent |= (i + 1u) << 8;
                    break;
                }
                __syncwarp();                               // every lane has read the stage that is filled next
                base += kBlock;
                if (base >= base_end) break;
            }
            if (absent >> 8) break;
        }
        if (absent >> 8) {                                  // this tile and all that follow
            int stage = static_cast<int>(absent >> 8) - 1;
            while (true) {
                compute(std::true_type{}, stage, base, !(absent >> stage & 1u));
                __syncwarp();
                base += kBlock;
                if (base >= base_end) break;
                stage = stage + 1 == C::kStages ? 0 : stage + 1;
                advance(stage);
            }
        }
        cp_async_wait<0>();
        __syncthreads();                                    // the rings are empty: their place takes the join
        if (C::kParked) cur = s_cur;
        const int row0_ = (cur.ch - s_pre[cur.r]) * kRows, rows_ = min(kRows, cur.rq.n * p.group - row0_);

        // ---------------------------------------------------------- join the warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int i = 4; i < 32; i <<= 1) l[nt][k] += __shfl_xor_sync(kAll, l[nt][k], i);
                if (g == 0) {
                    s_m[warp][nt * 8 + 2 * c + k] = m[nt][k];
                    s_l[warp][nt * 8 + 2 * c + k] = l[nt][k];
                }
                float* dst = s_join + (warp * kRows + nt * 8 + 2 * c + k) * kPad + 4 * g;
#pragma unroll
                for (int b = 0; b < B; ++b)
                    *reinterpret_cast<float4*>(dst + 32 * b) =
                        make_float4(o[nt][2 * b][k], o[nt][2 * b][2 + k], o[nt][2 * b + 1][k], o[nt][2 * b + 1][2 + k]);
            }
        __syncthreads();
        int a, z;
        cur.holders(s_plan, a, z);
        const bool whole = a == z;
        float* slot = fg::attn_piece<kRows, D>(p, blockIdx.x, a);
        for (int it = tid; it < rows_ * (D / 4); it += kThreads) {
            const int j = it / (D / 4), d4 = it % (D / 4);
            float top = s_m[0][j];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][j]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(s_m[w][j] - top);
                const float4 v = *reinterpret_cast<const float4*>(s_join + (w * kRows + j) * kPad + 4 * d4);
                sum = fmaf(s_l[w][j], f, sum);
                acc.x = fmaf(v.x, f, acc.x); acc.y = fmaf(v.y, f, acc.y);
                acc.z = fmaf(v.z, f, acc.z); acc.w = fmaf(v.w, f, acc.w);
            }
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                fg::attn_store<D>(p, cur.rq.t0, cur.h, row0_ + j, d4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
            } else {
                if (d4 == 0) {
                    slot[j] = top;
                    slot[kRows + j] = sum;
                }
                *reinterpret_cast<float4*>(slot + 2 * kRows + j * D + 4 * d4) = acc;
            }
        }
        if (!whole) fg::attn_join<kRows, D, kThreads, false>(p, s_plan, a, z, cur.rq.t0, cur.h, row0_, rows_);
        if (!cur.next(p, s_plan, s_pre)) break;
        __syncthreads();                                    // s_join is written again
    }
}

template <int B, int NT>
int launch(const AttnParams& p, int sms, int pdl, cudaStream_t stream) {
    using C = Cfg<B, NT>;
    const int smem = C::kSmem + (p.S + 1) * 4;
    static bool configured[256] = {};        // set once per device; setting it again is harmless
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(attn_kernel<B, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem + (fg::kAttnMaxRequests + 1) * 4) != cudaSuccess) {
            cudaGetLastError();
            return FG_ERR_CUDA;
        }
        configured[dev] = true;
    }
    const int ctas = sms * C::kPerSm < fg::kAttnMaxCtas ? sms * C::kPerSm : fg::kAttnMaxCtas;
    if (fg::print_configs_enabled())
        std::fprintf(stderr, "[fg] paged_attention_mxfp4 T=%d S=%d heads=%d x %d D=%d rows=%d grid=%d\n", p.T, p.S, p.heads,
                     p.group, C::D, C::kRows, ctas);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    if (pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&cfg, attn_kernel<B, NT>, p) != cudaSuccess) {
        cudaGetLastError();
        return FG_ERR_CUDA;
    }
    return FG_OK;
}

// Rows of an average request's kv head.
long long rows_of(int T, int S, int group) { return ((long long)T + S - 1) / S * group; }
// Row tiles of eight: as many as those rows fill, and as many as registers hold the accumulators of.  16 requests of
// 8192 tokens, 4 kv heads, us with one, two and four tiles: D = 64, 8 rows 16.7, 21.9, 28.7; 16 rows 25.8, 22.3, 28.7;
// 32 rows 42.5, 35.8, 30.1; D = 128, 8 rows 23.6, 30.3; 16 rows 37.2, 31.7.
int row_tiles(int T, int S, int group, int D) {
    const long long rows = rows_of(T, S, group);
    const int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    const int most = D == 64 ? 4 : D == 128 ? 2 : 1;
    return nt < most ? nt : most;
}
// Whether a call takes the kernel for many rows a request: where its work, in blocks of 128 keys times chunks of rows
// and each chunk's start, is less by more than it takes to begin and end (some 12 us).  Lengths are known on the device
// only; max_pages stands for them.  Measured, us here and there, 4 kv heads, 8192 keys: 16 requests, D = 64, 64 rows 50
// and 54, 128 rows 90 and 56; D = 128, 48 rows 73 and 76, 64 rows 93 and 76, 128 rows 176 and 80; 4 requests, D = 256,
// 64 rows 65 and 71, 128 rows 119 and 80.  One request of 1024 keys, D = 128: 64 rows 13 and 25, 512 rows 25.2 and 28.3;
// 64 requests of 512 keys: 64 rows 52 and 37.
constexpr int kFewestMany = 33;               // no call of fewer rows meets that
bool many_rows(int T, int S, int heads, int group, int D, long long keys, int window) {
    const long long rows = rows_of(T, S, group);
    if (S > fg::kAttnPromptRequests || rows < kFewestMany) return false;
    if (window > 0 && keys > window + rows / group) keys = window + rows / group;
    const double blocks = static_cast<double>(keys / kBlock + 1), items = static_cast<double>(S) * heads;
    const int few = 8 * row_tiles(T, S, group, D);
    const double a_block = D == 64 ? 2.1 : D == 128 ? 3.2 : 9.0;     // of 128 rows there, in blocks of `few` rows here
    return items * ((rows + few - 1) / few) * (5 + blocks) > a_block * items * ((rows + 127) / 128) * (3 + blocks) + 2300;
}
// Rows of its items (16 requests of 8192 tokens, D = 128, us with 128 and 256: 256 rows 133.5 and 136.3, 320 rows 190 and
// 217, 512 rows 242 and 220).
int prompt_rows(int T, int S, int group, int D) { return D <= 128 && rows_of(T, S, group) >= 512 ? 256 : 128; }

bool shapes_ok(int T, int S, int Hq, int Hkv, int D) {
    return T >= 0 && S >= 0 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq <= 65536 && D >= 1;
}

// Floats of the largest partial result of this file's variants.
constexpr int kMaxSlot = fg::attn_slot<32, 64>();
static_assert(fg::attn_slot<16, 128>() <= kMaxSlot && fg::attn_slot<8, 256>() <= kMaxSlot, "largest partial result");
constexpr long long kCtrBytes = (3 * fg::kAttnMaxCtas * 4 + 255) / 256 * 256;

}  // namespace

extern "C" {

long long fg_paged_attention_workspace(int T, int S, int Hq, int Hkv, int D) {
    if (!shapes_ok(T, S, Hq, Hkv, D) || (D != 64 && D != 128 && D != 256)) return -1;
    // enough for any fewer rows and requests too
    const bool many = rows_of(T, 1, Hq / Hkv) >= kFewestMany;
    const long long slot = (long long)prompt_rows(T, 1, Hq / Hkv, D) * (D + 2);
    const long long few = 2LL * fg::kAttnMaxCtas * kMaxSlot * 4, most = 2LL * fg::kAttnPromptCtas * slot * 4;
    return kCtrBytes + (many && most > few ? most : few);
}

int fg_paged_attention_mxfp4(int T, int S, int Hq, int Hkv, int D, int page_size, int num_pages, int max_pages,
                             const void* q, const uint8_t* k_cache, const uint8_t* k_sf, const uint8_t* v_cache,
                             const uint8_t* v_sf, const int32_t* block_table, const int32_t* query_start,
                             const int32_t* seq_lens, float scale, int window, void* out, void* workspace,
                             fg_stream_t stream) {
    if (!shapes_ok(T, S, Hq, Hkv, D) || page_size < 1 || num_pages < 1 || max_pages < 1 || window < 0 ||
        (long long)page_size * num_pages > 0x7fffffffLL || (long long)page_size * max_pages > 0x7fffffffLL - 4096 ||
        !(scale > 0.0f) || !(scale <= 3.402823466e38f))
        return FG_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || page_size % 16 || S > fg::kAttnMaxRequests || T > 1 << 18 || Hq / Hkv > 256 ||
        (long long)Hkv * page_size > 0x7fffffffLL)
        return FG_ERR_UNSUPPORTED;
    if (T == 0 || S == 0) return FG_OK;
    if (!q || !k_cache || !k_sf || !v_cache || !v_sf || !block_table || !query_start || !seq_lens || !out || !workspace ||
        !al(q, 16) || !al(k_cache, 16) || !al(k_sf, 16) || !al(v_cache, 16) || !al(v_sf, 16) || !al(block_table, 4) ||
        !al(query_start, 4) || !al(seq_lens, 4) || !al(out, 16) || !al(workspace, 256))
        return FG_ERR_INVALID_ARG;
    fg::HostState st;
    if (const int rc = fg::host_state(&st)) return rc;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const AttnParams p{static_cast<const uint16_t*>(q), k_cache, k_sf, v_cache, v_sf, block_table, query_start, seq_lens,
                       static_cast<uint16_t*>(out), T, S, Hkv, Hq / Hkv, page_size, num_pages, max_pages, window,
                       scale * 1.4426950408889634f, reinterpret_cast<unsigned*>(ws), reinterpret_cast<float*>(ws + kCtrBytes),
                       st.status, st.timeout_ns, st.debug_stall};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (many_rows(T, S, Hkv, Hq / Hkv, D, (long long)max_pages * page_size, window))
        return fg::launch_attn_prompt(p, D, prompt_rows(T, S, Hq / Hkv, D), st.sms, st.pdl, s);
    const int nt = row_tiles(T, S, Hq / Hkv, D);
    switch (D) {
        case 64: return nt == 1 ? launch<2, 1>(p, st.sms, st.pdl, s) : nt == 2 ? launch<2, 2>(p, st.sms, st.pdl, s) : launch<2, 4>(p, st.sms, st.pdl, s);
        case 128: return nt == 1 ? launch<4, 1>(p, st.sms, st.pdl, s) : launch<4, 2>(p, st.sms, st.pdl, s);
        default: return launch<8, 1>(p, st.sms, st.pdl, s);
    }
}

}  // extern "C"
