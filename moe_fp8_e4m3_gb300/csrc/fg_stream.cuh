// fg_stream.cuh - weight-streaming kernels for few tokens: one kernel template behind the
// whole-layer MoE MLP (fg_moe.cu) and the projection with per-token adapters (fg_lora.cu).
//
// With few tokens every product is bound by reading its weights once, so the operands swap
// places: the weights are the tensor core's M operand (two blocks of 128 rows per tile, 32 KB
// of a K-group of 128 per ring stage) and the tokens its N operand (BN = 16, 32, 64 or 128
// columns; the host takes the smallest that holds them).  Every token is multiplied with
// every weight block read; a token that does not use it is masked where the result is
// formed.  The tensor core has room for that (a 256 x 128 x 128 K-group takes ~0.3 us of it,
// reading its weights from HBM takes an SM 0.7 us), and no token is gathered or sorted.
//
// Work split: the units of one launch - (tile, K-group) pairs, tile by tile - form one line
// that is cut into equal shares, one per CTA, wherever the cuts fall ("stream-K"): every SM
// streams the same number of bytes whatever the number of experts, tiles and K-groups.  Where
// cuts cost more than they balance, whole tiles or equal pieces of each are dealt instead
// (plan_shares, plan_prompt).
// A cut tile is accumulated by several CTAs, whose FP32 parts are added up in share order (so
// the result does not depend on who comes last), in one of three ways that the host chooses:
//   through the workspace: each CTA writes its part and counts itself in, the last to arrive
//     adds them up and finishes the tile; no CTA waits for another, and the counters wrap to
//     zero by themselves (atomicInc);
//   in a cluster (few columns or a prompt's few tiles, tiles x pieces within the SMs): the parts stay
//     in the CTAs' shared memory, and each CTA adds up its share of the tile over the cluster;
//   spread (kDown with 64 or more columns): all parts go to the workspace and a third launch adds
//     them up on all SMs (stream_reduce_kernel).
//
// Bound: HBM, whose time for the weights is the floor.  Measured on GB300, the whole MoE MLP, its
// launches included: 128 tokens x 7168 x 2048, 32 experts, E4M3 253 us (5.6 TB/s, 0.82 of a copy's
// 6.8), 16 x 4096 49.8 us (0.75), 37 x 4096 with FP4 weights 93 us (0.68; half the bytes in the
// same ring), 1 x 4096 34 us (0.65).  Within a launch the weights stream at 6.3 to 6.6 TB/s; what
// is left are the ends: 3 us until the first loads are out and 2 us until they are back, 4 to 5 us
// from the first launch's last product to the second's first, and the joins.
//
// Modes
//   kGateUp  tile = 128 gate rows + the 128 up rows of one expert; epilogue: SiLU(gate) * up *
//            routing weight, per token and 128 outputs one UE8M0 scale, E4M3 codes -> workspace
//   kDown    tile = 256 output rows; its K axis runs over all active experts one after
//            another, so the sum over experts happens in the FP32 accumulator
//   kProj    tile = 256 output rows; K-groups of the shared FP8 weights, then units of the
//            adapters' B matrices (BF16, against x @ A^T from fg_lora.cu), in one accumulator
//
// Warp roles: 0, 2 TMA producers of the weight tiles (even / odd stages); 1 TMEM owner and
// MMA issuer of the tile's first block, 9 of the second; 3 TMA producer of the token operand;
// 8, 10 scale loaders; 4-7 and 12-15 epilogue, the first four on the first half of the tile's
// token columns, the others on the second.
// Every wait is bounded: on expiry the CTA records a time-out in the status word, all its
// roles wind down and the kernel returns.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>

#include "fg_gemm_kernel.cuh"

namespace fg {

enum StreamMode : int { kGateUp = 0, kDown = 1, kProj = 2 };

enum : int { kChkAdapter = 6 };          // an adapter id >= L

constexpr int kMaxListed = 1024;         // experts of a shard, adapters of a call
constexpr int kMaxTokenTiles = 512;      // kProj: token tiles of one call
constexpr int kMaxStreamCtas = 256;      // shares of a launch (partial slots in the workspace)
constexpr int kMaxCounters = 512;        // of one launch: two per share, one for each half of the columns
// head of a workspace: both launches' counters, a spread plan with its list of experts
constexpr int kCounterBytes = 2 * kMaxCounters * 4 + 256 + 2 * kMaxListed;

struct StreamMaps {
    CUtensorMap w;       // weights
    CUtensorMap x;       // token operand
    CUtensorMap lb;      // kProj: adapters' B
    CUtensorMap v;       // kProj: x @ A^T, [token tile][slot][part][BN][rp]
};

struct StreamParams {
    int tokens;                  // rows of the token operand
    int nk;                      // K-groups of one tile (kDown: of one expert)
    int row_tiles;               // kGateUp: I / 128 per expert; kDown, kProj: ceil(rows / 256)
    int out_rows;                // kGateUp: I; kDown: H; kProj: N (row length of d)
    int experts, expert_base, topk;
    const int32_t* ids;          // MoE: [tokens][topk]; LoRA: [tokens]
    const float* weights;        // routing weights [tokens][topk]
    const int32_t* sfw;          // weight scales
    int sfw_ld, sfw_rows;        // words per word row; words of it that exist
    long long sfw_gstride;       // words between experts
    const int32_t* sft;          // token scales
    int sft_ld;
    uint8_t* hq;                 // kGateUp out: [slot][BN][I] E4M3
    uint8_t* sfh;                // and its scale words [slot][ceil(I/512)][BN]
    float* part;                 // [CTA][2][2][BN][128] partial tiles
    unsigned* ctr;               // [kMaxCounters]
    void* d;
    int d_f32;
    int* spread;                 // not null: every tile's parts go to the workspace, and a third launch adds
                                 // them up (stream_reduce_kernel), told here how the units were dealt
    // adapters
    int lora_rp, lora_count, max_slots, token_tiles;
    int parts, unit_cols;        // BF16 parts of x @ A^T; rank columns of a unit
    const int* slot_ids;         // [token tile][max_slots] distinct adapters, ascending
    const int* slot_count;       // [token tile]
    int* status;
    unsigned long long timeout_ns;
    int debug_stall, pdl;
    int cluster;                 // kDown, kProj: > 1: a tile's pieces, one a CTA of a cluster that joins them itself
    // the operands as plain arrays (mend_outputs): weights, token codes, adapters' B and x @ A^T
    const uint8_t* w_raw;
    const uint8_t* x_raw;
    const uint16_t* lb_raw;
    const uint16_t* v_raw;
    int lora_r, w_fp4;
};

// D(tmem) (+)= A(smem) x B(smem)^T, BF16 inputs, FP32 accumulation in TMEM.
__device__ __forceinline__ void tc_mma_bf16(uint32_t d_taddr, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_taddr), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor of kind::f16: FP32 accumulator (1 at bits 4-5), BF16 A and B (1 at
// bits 7-9 and 10-12), K-major operands, N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t make_idesc_bf16(int m, int n) {
    return 1u << 4 | 1u << 7 | 1u << 10 | static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(m >> 4) << 24;
}
// mxf8f6f4 with E2M1 A (the swapped operand order): format code at bits 7-9.
__host__ __device__ constexpr uint32_t make_idesc_stream(int n, bool fp4) {
    return make_idesc_mxf8(128, n, false, false) | (fp4 ? kFmtE2M1 << 7 : 0u);
}
// 8 consecutive 32-bit TMEM columns of this warp's 32 lanes (one column per register).
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// True in one lane of the converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// Bulk copy of [src, src + bytes) to shared memory (16-byte aligned, bytes a multiple of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// Maximum over the warp's lanes of each of C columns (C = 8 or 16 values per lane): halves of the
// columns are exchanged until a lane holds one column, then its copies are joined.  Returns the
// maximum of column_of<C>(lane).
template <int C>
__device__ __forceinline__ uint32_t column_max(uint32_t (&m)[C], int lane) {
    int o = 16;
#pragma unroll
    for (int n = C / 2; n >= 1; n /= 2, o /= 2) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? m[i] : m[i + n], o);
            m[i] = max(up ? m[i + n] : m[i], got);
        }
    }
    for (; o >= 1; o /= 2) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    return m[0];
}
template <int C>
__device__ __forceinline__ int column_of(int lane) {
    return lane / (32 / C);          // the lane bits from the top choose the halves in turn
}
__device__ __forceinline__ float ld_dsmem_f32(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}
// Orders generic-proxy global writes (the codes that the next kernel loads by TMA).
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

template <int kMode, int BN>
struct StreamCfg {
    static constexpr int kABytes = 32768;                                   // two 128-row blocks x 128 bytes
    static constexpr int kBBytes = BN * 128;                                // kProj: also the parts of an adapter unit
    static constexpr int kSfBytes = 3 * 512;                                // weight block 0, 1, tokens
    static constexpr int kStageBytes = kABytes + kBBytes + kSfBytes;
    static constexpr int kMiscBytes = 512 + 1024 + BN * 8 + kMaxListed + 128 + 2 * kMaxListed +
                                      (kMode == kProj ? 4 * (kMaxTokenTiles + 1) : 0) + (kMode == kGateUp && BN >= 32 ? 2 * 16 * 128 : 0);
    static constexpr int kStages0 = (kSmemLimit - 1024 - kMiscBytes) / kStageBytes;
    static constexpr int kStages = kStages0 > 8 ? 8 : kStages0;
    static constexpr int kNumAcc = BN <= 64 ? 2 : 1;
    static constexpr int kSfCol0 = kNumAcc * 2 * BN;
    static constexpr int kTmemCols = kSfCol0 + 64 <= 128 ? 128 : (kSfCol0 + 64 <= 256 ? 256 : 512);
    static constexpr int kThreads = 512;
    // join of a share's last tile: partials through the idle ring, kJoinSlots pieces per group
    static constexpr int kChunk = BN >= 32 ? 16 : 8;                        // token columns an epilogue group takes at a time
    static constexpr int kChunks = BN / 2 / kChunk;                         // of a group
    static constexpr int kJoin = 16 / kChunk;                               // partials it loads at a time
    static constexpr int kPieceBytes = kChunk * 2 * 128 * 4;                // a chunk of one partial
    static constexpr int kJoinSlots = kStages * kABytes / 2 / kPieceBytes > 10 ? 10 : kStages * kABytes / 2 / kPieceBytes;
    static constexpr int kOffB = kStages * kABytes;
    static constexpr int kOffSf = kOffB + kStages * kBBytes;
    static constexpr int kOffBar = kOffSf + kStages * kSfBytes;
    static constexpr int kNumBars = 2 * kStages + 2 * kNumAcc + 5 + 2 * kJoinSlots;
    static constexpr int kOffMisc = kOffBar + 512 - 64;                     // TMEM address, abort flag, count, last flag
    static constexpr int kOffRed = kOffBar + 512;                           // [group][2][4 warps][16] amax words
    static constexpr int kOffTok = kOffRed + 1024;                          // [BN] routing weights, [BN] flags
    static constexpr int kOffBits = kOffTok + BN * 8;
    static constexpr int kOffSetup = kOffBits + kMaxListed;
    static constexpr int kOffList = kOffSetup + 128;
    static constexpr int kOffPre = kOffList + 2 * kMaxListed;
    static constexpr int kOffCodes = kOffPre;                               // kGateUp, BN >= 32: [group][16 columns][128 rows] E4M3
    static constexpr int kSmemBytes = kOffBar + kMiscBytes + 1024;          // + alignment slack
    static_assert(kNumBars * 8 <= 512 - 64, "barrier area");
    static_assert(kSfCol0 + 64 <= 512, "TMEM columns");
    static_assert(kStages >= 3 && kSmemBytes <= kSmemLimit, "shared memory");
};

// One share's piece of one tile: units [k0, k1) of nk.  kProj deals a tile's FP8 units and its
// adapter units to its pieces separately (the adapter units wait for x @ A^T and take longer):
// unit k0 + j is FP8 unit f0 + j for j < nf, then adapter unit l0 + j - nf.
struct StreamSeg {
    int tile, tt, k0, k1, nk;
    int first_unit;      // of the tile
    int f0, nf, l0;
    bool whole;
};

struct StreamPlan {
    int units, shares, nk, row_tiles;
    int pieces;          // > 0: every tile is cut into that many pieces, one a share; 0: equal shares;
                         // -1: whole tiles, equally many to a share
    int q, r;            // the last two: r shares of q + 1 units (tiles), then shares of q
    int fp8;             // kProj: FP8 units of a tile
    const int* pre;      // kProj: units before each token tile
};

// Units of a tile before its piece i.
__device__ __forceinline__ int piece_begin(const StreamPlan& pl, int i) {
    return i == 0 ? 0 : i * pl.fp8 / pl.pieces + (pl.nk == pl.fp8 ? 0 : i * (pl.nk - pl.fp8) / pl.pieces);
}
__device__ __forceinline__ int share_begin(const StreamPlan& pl, int c) {
    if (pl.pieces > 0) {
        const int t = c / pl.pieces;
        return t * pl.nk + piece_begin(pl, c - t * pl.pieces);
    }
    return c * pl.q + min(c, pl.r);
}
// The first and the last share of the tile of units [u0, u0 + nk).
__device__ __forceinline__ void shares_of(const StreamPlan& pl, int u0, int nk, int& first, int& last) {
    if (pl.pieces > 0) {
        first = u0 / pl.nk * pl.pieces;
        last = first + pl.pieces - 1;
        return;
    }
    auto of = [&](int u) {
        const int big = (pl.q + 1) * pl.r;
        return u < big ? u / (pl.q + 1) : pl.r + (u - big) / pl.q;
    };
    first = of(u0);
    last = of(u0 + nk - 1);
}

__device__ __forceinline__ void deal_shares(StreamPlan& pl, int tiles, int grid) {
    pl.shares = max(1, pl.pieces > 0 ? pl.pieces * tiles : min(grid, pl.pieces < 0 ? tiles : pl.units));
    const int n = pl.pieces < 0 ? tiles : pl.units;
    pl.q = n / pl.shares;
    pl.r = n - pl.q * pl.shares;
}
// How `tiles` tiles of nk units each become shares for at most `grid` CTAs: s pieces per tile
// (s = 1: no cut), where all pieces find a CTA, whole tiles in several rounds, or equal shares cut
// anywhere.  The time is the larger of a CTA's units at the pace of its MMA issuers and all units
// at HBM's (less `early` units per share, which stream before the launch can begin; in the last
// round of whole tiles only some CTAs ask for theirs), plus the join of a cut tile.  Equal shares
// cut a tile at both ends of a share; with more than a tile to a share the join hides behind the
// rest of it.  Measured on GB300: a unit takes an SM 0.3 us when HBM keeps up, all SMs together
// 4.75 ns (E4M3) or 2.5 ns (FP4) of HBM; counting in takes 2 us and a partial's chunk 0.25 us, and
// what equal shares lose against whole tiles with the same bytes 8 us at 64 columns and 11 us of
// streaming, 6 at 128 and 19, 4 at 128 and 46, nothing at 128 and 136, 3 to 4 at 32 and 15.  The
// whole MoE MLP, equal shares and whole tiles: 59 x 1408 x 1280, 24 experts 52.6 and 44.6 us; 88 x
// 2048 x 1920, 17 experts 71.1 and 65.0; 29 x 1920 x 1536, 37 experts, FP4 54.8 and 51.6; 128 x 7168
// x 2048, 32 experts 255 and 263; 37 x 4096 x 2048, 32 experts, FP4 94.4 and 98.7.
__device__ __forceinline__ void plan_shares(StreamPlan& pl, int tiles, int grid, bool fp4, int chunks, int early, bool spread) {
    const float unit_hbm = fp4 ? 0.0025f : 0.00475f;
    const float units = pl.units, nk = pl.nk;
    auto time = [&](float shares, float per, float n) {
        const float t = fmaxf(per * 0.3f, fmaxf(units - early * shares, 0.0f) * unit_hbm);
        return t + (spread ? 0.1f * n : n > 1.0f ? 2.0f + 0.25f * n * chunks : 0.0f);
    };
    // lane s > 0 looks at s pieces per tile, lane 0 at equal shares, lane 31 at whole tiles; the least
    // time (its bits, the lane in the low five) wins
    const int s = static_cast<int>(threadIdx.x & 31);
    float t = 1e30f;
    if (s == 0) {
        const float per = fmaxf(__fdividef(units, static_cast<float>(grid)), 1.0f);
        const float n = __fdividef(nk, per) + 1.0f, all = time(fminf(grid, units), per, 1.0f);
        t = spread ? time(fminf(grid, units), per, n)
                   : all + fmaxf(n > 2.0f ? 4.0f + 0.25f * n * chunks : 0.0f, (chunks > 1 ? 9.0f : 5.0f) - 0.125f * all);
    } else if (s <= 16 && s * tiles <= grid && s <= pl.fp8) {                 // (no piece is empty)
        t = time(s * tiles, __fdividef(nk, static_cast<float>(s)), s);
    } else if (s == 31 && tiles > grid) {
        const int rounds = tiles / grid;
        t = nk * (rounds * fmaxf(0.3f, grid * unit_hbm) +
                  (tiles > rounds * grid ? fmaxf(0.33f, (tiles - rounds * grid) * unit_hbm) : 0.0f));
    }
    const uint32_t best = __reduce_min_sync(0xffffffffu, (__float_as_uint(t) & ~31u) | s);
    pl.pieces = (best & 31u) == 31u ? -1 : static_cast<int>(best & 31u);
    deal_shares(pl, tiles, grid);
}
// The same for a projection of several token tiles (128 columns each, `most` units in the largest
// one), whose products bound it: whole tiles, or equal shares where that leaves too many CTAs idle in
// the last round.  Measured on GB300: a unit takes 0.33 us, a tile's epilogue or part 3 us, counting
// in and waiting for the last arrival 6, adding a part of 128 KB 2.2.  Whole tiles and equal shares:
// 2048 x 4096 x 4096, rank 64 60.4 and 66.8 us; 664 x 4224 x 1280 23.4 and 35.2; 1037 x 416 x 1408
// 28.2 and 51.0; 180 x 544 x 640, 113 adapters of rank 128 177 and 93.7.
__device__ __forceinline__ void plan_prompt(StreamPlan& pl, int tiles, int grid, int most) {
    const float nk = __fdividef(pl.units, tiles), per = __fdividef(pl.units, static_cast<float>(min(grid, pl.units)));
    const float whole = ((tiles + grid - 1) / grid) * (0.33f * most + 3.0f);
    const float equal = 0.33f * per + 3.0f * (__fdividef(per, nk) + 1.0f) + 6.0f + 2.2f * (__fdividef(nk, per) + 1.0f);
    pl.pieces = whole <= equal ? -1 : 0;
    deal_shares(pl, tiles, grid);
}

// What stream_reduce_kernel has to know of a plan.
enum : int { kSpreadUnits = 0, kSpreadShares, kSpreadNk, kSpreadPieces, kSpreadListed, kSpreadWords = 8 };

// The pieces of one share: first the tile that goes on into the next share, then the others in
// order (so a tile that the share before began comes next, whole tiles last).  A cut tile's parts
// are then the first thing its shares do, and joining them hides behind the whole tiles.
template <int kMode>
struct StreamWalk {
    int u, end, tail, tail_end;          // [u, end) is left; before it [tail, tail_end) if tail >= 0
    int tile, tt, first, nk;             // the tile of unit u
    int tail_tile, tail_tt, tail_nk;
    StreamWalk() = default;
    __device__ __forceinline__ StreamWalk(const StreamPlan& pl, int share)
        : u(0), end(0), tail(-1), tail_end(0), tile(0), tt(0), first(0), nk(1), tail_tile(0), tail_tt(0), tail_nk(1) {
        if (share >= pl.shares) return;
        if (pl.pieces < 0) {
            auto first_of = [&](int t) {
                tile = t;
                nk = pl.nk;
                if (kMode != kProj) return t * nk;
                tt = t / pl.row_tiles;
                tile = t - tt * pl.row_tiles;
                nk = (pl.pre[tt + 1] - pl.pre[tt]) / pl.row_tiles;
                return pl.pre[tt] + tile * nk;
            };
            const int t = share * pl.q + min(share, pl.r);
            const int last = first_of(t + pl.q - (share < pl.r ? 0 : 1));
            end = last + nk;
            u = first = first_of(t);
            return;
        }
        if (pl.pieces > 0) {              // one piece of one tile
            tile = pl.pieces == 1 ? share : share / pl.pieces;
            const int i = share - tile * pl.pieces;
            if (kMode == kProj) {         // (in a cluster, pl.nk is this tile's)
                tt = tile / pl.row_tiles;
                tile -= tt * pl.row_tiles;
            }
            nk = pl.nk;
            first = tile * nk;
            u = first + piece_begin(pl, i);
            end = first + (i + 1 == pl.pieces ? nk : piece_begin(pl, i + 1));
            return;
        }
        u = share_begin(pl, share);
        end = tail_end = share_begin(pl, share + 1);
        int a = 0, base = 0;
        auto locate = [&](int v, int& at_tile, int& at_tt, int& at_nk) {
            at_nk = pl.nk;
            if (kMode == kProj) {
                while (v >= pl.pre[a + 1]) ++a;
                base = pl.pre[a];
                at_nk = (pl.pre[a + 1] - base) / pl.row_tiles;
            }
            at_tt = a;
            at_tile = (v - base) / at_nk;
            return base + at_tile * at_nk;
        };
        if (u >= end) return;
        first = locate(u, tile, tt, nk);
        const int last = locate(end - 1, tail_tile, tail_tt, tail_nk);
        if (last + tail_nk != end && last > u) end = tail = last;
    }
    __device__ __forceinline__ bool next(const StreamPlan& pl, StreamSeg& s) {
        if (tail >= 0) {
            s.tile = tail_tile; s.tt = tail_tt; s.nk = tail_nk; s.first_unit = tail;
            s.k0 = 0;
            s.k1 = tail_end - tail;
            s.whole = false;
            tail = -1;
            deal(pl, s);
            return true;
        }
        if (u >= end) return false;
        s.tile = tile; s.tt = tt; s.nk = nk; s.first_unit = first;
        s.k0 = u - first;
        s.k1 = min(nk, s.k0 + (end - u));
        s.whole = s.k0 == 0 && s.k1 == nk;
        u += s.k1 - s.k0;
        deal(pl, s);
        // the tile behind it
        first += nk;
        if (++tile == pl.row_tiles && kMode == kProj) {
            tile = 0;
            ++tt;
            if (u < end) nk = (pl.pre[tt + 1] - pl.pre[tt]) / pl.row_tiles;
        }
        return true;
    }
    __device__ __forceinline__ void deal(const StreamPlan& pl, StreamSeg& s) const {
        if (kMode != kProj) return;
        if (pl.pieces > 0) {
            // k0 is the sum of both kinds' shares before piece i (the share is one piece)
            const int i = static_cast<int>(blockIdx.x) % pl.pieces;
            s.f0 = i * pl.fp8 / pl.pieces;
            s.nf = (i + 1) * pl.fp8 / pl.pieces - s.f0;
            s.l0 = i * (pl.nk - pl.fp8) / pl.pieces;
        } else {
            s.f0 = min(s.k0, pl.fp8);
            s.nf = min(s.k1, pl.fp8) - s.f0;
            s.l0 = max(s.k0, pl.fp8) - pl.fp8;
        }
    }
    __device__ __forceinline__ bool done() const { return tail < 0 && u >= end; }
};

// Walks a share unit by unit.  k: K-group, from `fp8` on adapter units (kProj).  li, kl: kDown's
// expert (list index) and K-group within it (else kl == k); no division per unit.
template <int kMode>
struct StreamCursor {
    StreamWalk<kMode> walk;
    StreamSeg sg;
    int at, k, li, kl, per;
    bool valid;
    __device__ __forceinline__ StreamCursor(const StreamPlan& pl, const StreamWalk<kMode>& from, int per_expert)
        : walk(from), at(0), k(0), li(0), kl(0), per(per_expert) { enter(pl); }
    __device__ __forceinline__ void enter(const StreamPlan& pl) {
        valid = walk.next(pl, sg);
        if (!valid) return;
        at = k = kl = sg.k0;
        if (kMode == kDown) { li = k / per; kl = k - li * per; }
        if (kMode == kProj) { at = 0; k = kl = sg.nf > 0 ? sg.f0 : pl.fp8 + sg.l0; }
    }
    __device__ __forceinline__ void step(const StreamPlan& pl) {
        ++at;
        ++k;
        ++kl;
        if (kMode == kDown && kl == per) { kl = 0; ++li; }
        if (kMode == kProj && at == sg.nf) k = kl = pl.fp8 + sg.l0;
        if (at == (kMode == kProj ? sg.k1 - sg.k0 : sg.k1)) enter(pl);
    }
    // the unit brings new scale words: FP4 weights every K-group, else at the segment's first and
    // every fourth K-group
    __device__ __forceinline__ bool new_words(bool fp4, int fp8_units) const {
        return (kMode != kProj || k < fp8_units) && (fp4 || at == (kMode == kProj ? 0 : sg.k0) || (kl & 3) == 0);
    }
};

// Marks the byte of every id in [base, base + count) among ids[0, n) (plain stores: with few
// experts, atomics on one word's bits would queue up); all threads, behind a barrier after
// clear_marks.  own: what load_id gave the thread, so that the load can run ahead of the barrier.
__device__ __forceinline__ void clear_marks(uint8_t* marks) {
    for (int i = threadIdx.x; i < kMaxListed / 4; i += blockDim.x) reinterpret_cast<uint32_t*>(marks)[i] = 0;
}
__device__ __forceinline__ int load_id(const int32_t* ids, int n) {
    return static_cast<int>(threadIdx.x) < n ? __ldcg(ids + threadIdx.x) : -1;
}
__device__ __forceinline__ void mark_ids(const int32_t* ids, int n, int own, int base, int count, uint8_t* marks) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const unsigned v = static_cast<unsigned>(own) - static_cast<unsigned>(base);
        if (v < static_cast<unsigned>(count)) marks[v] = 1;
        if (i + blockDim.x < n) own = __ldcg(ids + i + blockDim.x);
    }
    __syncthreads();
}
// The marked ids in ascending order, and their number; one warp.
__device__ __forceinline__ int list_marked(const uint8_t* marks, uint16_t* list) {
    const int lane = threadIdx.x & 31;
    // lane's 32 bytes to bits: four at a time, byte k of a word to bit k
    uint32_t m = 0;
    const uint4* own = reinterpret_cast<const uint4*>(marks) + lane * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 w = own[i];
        m |= ((w.x * 0x10204080u) >> 28) << (16 * i) | ((w.y * 0x10204080u) >> 28) << (16 * i + 4) |
             ((w.z * 0x10204080u) >> 28) << (16 * i + 8) | ((w.w * 0x10204080u) >> 28) << (16 * i + 12);
    }
    const int c = __popc(m);
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    int pos = incl - c;
    for (; m; m &= m - 1) list[pos++] = static_cast<uint16_t>(lane * 32 + __ffs(m) - 1);
    return __shfl_sync(0xffffffffu, incl, 31);
}

// What warp 0 works out for a CTA before its roles begin.
template <int kMode>
struct StreamSetup {
    StreamPlan pl;
    int listed;              // distinct experts or adapters
    StreamWalk<kMode> walk;
};

// ---------------------------------------------------------------- outputs that are not finite
// Every weight tile is multiplied with every token of its tile, so a NaN weight or scale, or a
// non-finite element of an adapter's B, makes a NaN of 0 * NaN for tokens that do not use it.  An
// output that is not finite is therefore worked out again, from what its token uses alone: one
// thread an output, the same products in FP32, in K order.  Slow, and only ever there (a NaN in every
// row of one expert's w2: 16 x 4096 0.4 ms, 128 x 7168 26 ms; in all of one adapter's B: 64 x 7168 5 ms,
// 2048 x 4096 86 ms, far inside the 4 s of a bounded wait).  Where all is finite it costs an FMA an
// output, whose zero becomes a NaN behind an infinity or a NaN (1 x 4096 34.4 -> 34.6 us, 64 x 7168 with
// adapters 21.55 -> 21.75, 2048 x 4096 with adapters 60.1 -> 60.8).  One function for both
// weight types: with one each, the reduce kernel beside the FP4 one gets 48 registers instead of 61 and
// keeps fewer loads in flight (37 x 4096 FP4 93.9 us instead of 92.9).
__device__ __forceinline__ float ue8m0(uint32_t b) {
    return b == 255u ? __int_as_float(0x7fc00000) : __uint_as_float(b ? b << 23 : 0x00400000u);
}
__device__ __forceinline__ uint32_t scale_byte(const int32_t* word, int i) {
    return static_cast<uint32_t>(__ldcg(word)) >> (8 * i) & 255u;
}
// One row of nk K-groups: x and w point at its codes, xs at its scale words (xs_ld words apart), ws
// at the weight row's (FP4: a word a K-group, ws_ld apart; E4M3: one for four).
__device__ __forceinline__ float exact_dot(bool fp4, const uint8_t* x, const uint8_t* w, const int32_t* xs, int xs_ld,
                                           const int32_t* ws, int ws_ld, int nk) {
    float sum = 0.0f;
#pragma unroll 1
    for (int g = 0; g < nk && sum == sum; ++g) {                        // (a NaN stays one)
        const float sx = ue8m0(scale_byte(xs + (long long)(g >> 2) * xs_ld, g & 3));
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {                                   // 32 elements
            const uint32_t* x4 = reinterpret_cast<const uint32_t*>(x + g * 128 + b * 32);
            float part = 0.0f;
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const uint32_t xc = __ldcg(x4 + i);
                const uint32_t wc = fp4 ? __ldg(reinterpret_cast<const uint16_t*>(w + g * 64 + b * 16) + i)
                                         : __ldg(reinterpret_cast<const uint32_t*>(w + g * 128 + b * 32) + i);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const __half_raw wv = fp4 ? __nv_cvt_fp4_to_halfraw(static_cast<__nv_fp4_storage_t>(wc >> (4 * c) & 15u), __NV_E2M1)
                                               : __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(wc >> (8 * c)), __NV_E4M3);
                    const __half_raw xv = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(xc >> (8 * c)), __NV_E4M3);
                    part += __half2float(__half(xv)) * __half2float(__half(wv));
                }
            }
            const float sw = ue8m0(fp4 ? scale_byte(ws + (long long)g * ws_ld, b) : scale_byte(ws + (long long)(g >> 2) * ws_ld, g & 3));
            sum += part * sx * sw;
        }
    }
    return sum;
}
__device__ __forceinline__ int place_of(const uint16_t* list, int n, int id) {
    int lo = 0;
    for (int hi = n; lo < hi;) {
        const int mid = (lo + hi) / 2;
        if (list[mid] < id) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}
// Row r of D's tokens [t0, t0 + n) of token tile tt, where the stored value is not finite.
template <int kMode, int BN>
__device__ __noinline__ void mend_outputs(const StreamParams& p, const uint16_t* list, int nlist, int tt, int t0, int n, int r) {
    const bool fp4 = kMode == kDown && p.w_fp4;
    for (int t = t0; t < t0 + n; ++t) {
        const int m = tt * BN + t;
        const long long at = (long long)m * p.out_rows + r;
        const float old = p.d_f32 ? static_cast<float*>(p.d)[at] : __bfloat162float(static_cast<__nv_bfloat16*>(p.d)[at]);
        if (old - old == 0.0f) continue;
        float sum = 0.0f;
        if (kMode == kDown) {
            const int32_t* ids = p.ids + (long long)m * p.topk;
            for (int j = 0; j < p.topk; ++j) {
                const int id = __ldg(ids + j), e = id - p.expert_base;
                bool again = static_cast<unsigned>(e) >= static_cast<unsigned>(p.experts);
                for (int i = 0; i < j; ++i) again |= __ldg(ids + i) == id;
                if (again) continue;
                const int li = place_of(list, nlist, e), words = (p.nk + 3) / 4;
                const long long k = (long long)p.nk * 128, row = (long long)e * p.out_rows + r;
                sum += exact_dot(fp4, p.x_raw + ((long long)li * BN + t) * k, p.w_raw + (fp4 ? row * k / 2 : row * k),
                                       p.sft + (long long)li * words * BN + t, BN,
                                       p.sfw + e * p.sfw_gstride + (fp4 ? r : r >> 7), p.sfw_ld, p.nk);
            }
        } else {
            const long long k = (long long)p.nk * 128;
            sum = exact_dot(false, p.x_raw + m * k, p.w_raw + r * k, p.sft + m, p.sft_ld, p.sfw + (r >> 7), p.sfw_ld, p.nk);
            const int id = __ldg(p.ids + m);
            if (id >= 0 && id < p.lora_count) {
                int slot = 0;                     // its place among the tile's adapters
                if (nlist > 0) slot = place_of(list, nlist, id);
                else while (slot + 1 < p.max_slots && __ldcg(p.slot_ids + tt * p.max_slots + slot) != id) ++slot;
                const long long part = (long long)BN * p.lora_rp;
                const uint16_t* v = p.v_raw + ((long long)tt * p.max_slots + slot) * p.parts * part + (long long)t * p.lora_rp;
                const uint16_t* lb = p.lb_raw + ((long long)id * p.out_rows + r) * p.lora_r;
                for (int c = 0; c < p.lora_r; ++c)
                    for (int o = 0; o < p.parts; ++o)
                        sum += __bfloat162float(__ushort_as_bfloat16(__ldcg(v + o * part + c))) *
                               __bfloat162float(__ushort_as_bfloat16(__ldg(lb + c)));
            }
        }
        if (p.d_f32) static_cast<float*>(p.d)[at] = sum;
        else static_cast<__nv_bfloat16*>(p.d)[at] = __float2bfloat16(sum);
    }
}

template <int kMode, int BN, bool kFp4>
__global__ void __launch_bounds__(StreamCfg<kMode, BN>::kThreads, 1)
fg_stream_kernel(const __grid_constant__ StreamParams p, const __grid_constant__ StreamMaps maps) {
    using C = StreamCfg<kMode, BN>;
    static_assert(sizeof(StreamSetup<kMode>) <= 128, "set-up area");
    constexpr bool kMoe = kMode == kGateUp || kMode == kDown;
    constexpr bool kClusters = kMode == kProj || (kMode == kDown && BN <= 32);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    // the warp's number from a shuffle and the plan's below: what follows is uniform over a warp
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t bar0 = sbase + C::kOffBar;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (C::kStages + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * C::kStages + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * C::kStages + C::kNumAcc + b); };
    // per issuer: its MMAs done, on the way out and before products of another kind
    auto drain_of = [&](int b) { return bar0 + 8u * (2 * C::kStages + 2 * C::kNumAcc + b); };
    auto turn_of = [&](int b) { return bar0 + 8u * (2 * C::kStages + 2 * C::kNumAcc + 2 + b); };
    const uint32_t xfull_bar = bar0 + 8u * (2 * C::kStages + 2 * C::kNumAcc + 4 + 2 * C::kJoinSlots);   // cluster: all parts ready
    const int cl = kClusters ? p.cluster : 1;
    // a group's pieces of partials on their way into the ring
    auto join_bar = [&](int g, int i) { return bar0 + 8u * (2 * C::kStages + 2 * C::kNumAcc + 4 + g * C::kJoinSlots + i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 16);     // [2]
    // per token: routing weight of the tile's expert, 1 where the token uses it
    float2* tok = reinterpret_cast<float2*>(smem + C::kOffTok);
    uint8_t* marks = smem + C::kOffBits;
    uint16_t* list = reinterpret_cast<uint16_t*>(smem + C::kOffList);
    int* pre = reinterpret_cast<int*>(smem + C::kOffPre);

    // kDown runs behind its own kGateUp launch, and kProj behind x @ A^T, which let it start only
    // after their own wait: the ids, weights and adapters they read before this launch's wait were
    // complete before that.  Only the roles that touch what the launch before writes wait.
    // A CTA of one token tile (the only one, or its cluster's) finds its adapters by itself; one whose
    // share crosses tiles reads what the launch before found.
    const bool own_tile = kMode == kProj && (p.token_tiles == 1 || cl > 1);
    const int own_tt = own_tile && p.token_tiles > 1 ? static_cast<int>(blockIdx.x) / cl / p.row_tiles : 0;
    const int32_t* ids = p.ids + own_tt * BN;
    const int n_ids = kMoe ? p.tokens * p.topk : (own_tile ? min(BN, p.tokens - own_tt * BN) : 0);
    int own_id = kMode == kGateUp ? -1 : load_id(ids, n_ids);
    clear_marks(marks);
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full_bar(s), 66);          // two TMA producers; the lanes of the scale loader and of warp 3
            mbar_init(empty_bar(s), 2);          // both issuers' commits
        }
        for (int b = 0; b < C::kNumAcc; ++b) {
            mbar_init(accf_bar(b), 2);
            mbar_init(acce_bar(b), 8);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(drain_of(b), 1);
            mbar_init(turn_of(b), 1);
            for (int i = 0; i < C::kJoinSlots; ++i) mbar_init(join_bar(b, i), 1);
        }
        mbar_init(xfull_bar, 8 * cl);             // every epilogue warp of the cluster
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&maps.w);
        tma_prefetch_map(&maps.x);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    // a cluster's barriers are initialised before any CTA of it arrives on them from afar
    if (cl > 1) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (kMode == kGateUp || (kMode == kProj && !own_tile)) {
        grid_dependency_wait();
        if (threadIdx.x == 0) grid_launch_dependents();
    }
    if (kMode == kGateUp) own_id = load_id(ids, n_ids);
    if (kMoe || own_tile) mark_ids(ids, n_ids, own_id, kMoe ? p.expert_base : 0, kMoe ? p.experts : p.lora_count, marks);
    StreamSetup<kMode>& setup = *reinterpret_cast<StreamSetup<kMode>*>(smem + C::kOffSetup);
    const int share = static_cast<int>(blockIdx.x);
    if (warp == 0) {
        StreamPlan pl;
        int nlist = 0, most = 0;              // (units of the largest token tile)
        pl.row_tiles = p.row_tiles;
        pl.pre = pre;
        pl.nk = p.nk;
        if (kMoe || own_tile) nlist = list_marked(marks, list);
        auto tile_units = [&](int adapters) { return p.nk + (adapters * p.lora_rp + p.unit_cols - 1) / p.unit_cols; };
        if constexpr (kMoe) {
            pl.nk = kMode == kDown ? nlist * p.nk : p.nk;
            pl.units = kMode == kDown ? p.row_tiles * pl.nk : nlist * p.row_tiles * pl.nk;
        } else if (own_tile) {
            pl.nk = tile_units(nlist);
            pl.units = p.row_tiles * pl.nk;
            if (lane < 2) pre[lane] = lane * pl.units;
        } else {
            // units of a token tile: row tiles x (K-groups + adapter units of unit_cols rank columns)
            int run = 0;
            for (int i0 = 0; i0 < p.token_tiles; i0 += 32) {
                const int i = i0 + lane;
                const int v = i < p.token_tiles ? p.row_tiles * tile_units(__ldcg(p.slot_count + i)) : 0;
                most = max(most, static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v))));
                int incl = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                if (i < p.token_tiles) pre[i] = run + incl - v;
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) pre[p.token_tiles] = run;
            __syncwarp();
            pl.units = run;
        }
        pl.fp8 = kMode == kProj ? p.nk : pl.nk;
        if (cl > 1) {
            pl.pieces = cl;
            pl.shares = cl * p.row_tiles * (kMode == kProj ? p.token_tiles : 1);
            pl.q = pl.r = 0;
        } else if (kMode == kProj && !own_tile) {
            plan_prompt(pl, p.token_tiles * p.row_tiles, static_cast<int>(gridDim.x), most / p.row_tiles);
        } else {
            const int tiles = kMode == kGateUp ? nlist * p.row_tiles : p.row_tiles;
            plan_shares(pl, tiles, static_cast<int>(gridDim.x), kFp4, C::kChunks, kMode == kDown ? C::kStages : 0,
                        p.spread != nullptr);
            // no token uses an expert of this shard: no tile, so no share that would read or count one
            if (kMode == kGateUp && nlist == 0) pl.shares = 0;
        }
        __syncwarp();
        if (lane == 0) {
            setup.pl = pl;
            setup.listed = nlist;
            setup.walk = StreamWalk<kMode>(pl, share);
        }
    }
    __syncthreads();
    const StreamPlan pl = setup.pl;
    const StreamWalk<kMode>& share_walk = setup.walk;      // each role's copy starts from it
    const int nlist = setup.listed;
    auto slots_of = [&](int tt) { return own_tile ? nlist : __ldcg(p.slot_count + tt); };
    auto adapter_of = [&](int tt, int slot) { return own_tile ? static_cast<int>(list[slot]) : __ldcg(p.slot_ids + tt * p.max_slots + slot); };
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const WaitCtl wctl{abort_flag, p.status, p.timeout_ns};
    // kProj: adapter units behind the K-groups
    const int ucols = min(p.lora_rp, p.unit_cols), rb = ucols * 2;           // rank columns of an adapter in a unit, bytes
    const int per_unit = kMode == kProj ? max(1, p.unit_cols / p.lora_rp) : 1;   // adapters in a unit
    const int pieces = kMode == kProj ? max(1, p.lora_rp / p.unit_cols) : 1;     // units of one adapter

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ weight tiles
        if (lane == 0) {
            const uint32_t par = warp == 0 ? 0u : 1u;
            int s = 0;
            uint32_t ph = 0, n = 0, armed = 0, armed_par = 0;
            bool stall = p.debug_stall != 0 && par == 0, aborted = false;
            StreamCursor<kMode> c(pl, share_walk, p.nk);
            for (; c.valid; c.step(pl), ++n) {
                if ((n & 1u) == par) {
                    if (!wait_bar(empty_bar(s), ph ^ 1u, wctl, kWaitProducer)) { aborted = true; break; }
                    if (stall) {
                        stall = false;       // this stage stays unfilled: the MMA issuer times out
                    } else {
                        const uint32_t fb = full_bar(s), dst = sbase + s * C::kABytes;
                        armed |= 1u << s;
                        armed_par = (armed_par & ~(1u << s)) | (ph << s);
                        if (kMode == kProj && c.k >= p.nk) {
                            const int u = c.k - p.nk;
                            const int nslots = slots_of(c.sg.tt);
                            const int s0 = pieces > 1 ? u / pieces : u * per_unit;
                            const int cnt = min(per_unit, nslots - s0);
                            mbar_arrive_expect_tx(fb, static_cast<uint32_t>(cnt * 256 * rb));
                            for (int j = 0; j < cnt; ++j)
                                tma_load_3d(dst + j * 256 * rb, &maps.lb, fb, pieces > 1 ? (u % pieces) * ucols : 0,
                                            c.sg.tile * 256, adapter_of(c.sg.tt, s0 + j));
                        } else {
                            // packed FP4: the transaction counts the bytes read, half of those filled
                            mbar_arrive_expect_tx(fb, kFp4 ? C::kABytes / 2 : C::kABytes);
                            if constexpr (kMode == kGateUp) {
                                const int e = list[c.sg.tile / p.row_tiles];
                                tma_load_3d(dst, &maps.w, fb, c.k * 128, c.sg.tile % p.row_tiles * 128, 2 * e);
                            } else if constexpr (kMode == kDown) {
                                tma_load_3d(dst, &maps.w, fb, c.kl * 128, c.sg.tile * 256, list[c.li]);
                            } else {
                                tma_load_3d(dst, &maps.w, fb, c.k * 128, c.sg.tile * 256, 0);
                            }
                        }
                    }
                }
                if (++s == C::kStages) { s = 0; ph ^= 1u; }
            }
            if (aborted || *abort_flag)
                for (int i = 0; i < C::kStages; ++i)
                    if (armed >> i & 1u) drain_bar(full_bar(i), armed_par >> i & 1u, 20000000ull);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ----------------------------------------------- token operand and its scale words
        // Only this warp (and the epilogue) waits for the launch before: in kDown and kProj the
        // weights and their scales stream meanwhile.
        if (kMode == kDown) {
            grid_dependency_wait();
            if (lane == 0) {
                grid_launch_dependents();
                fence_proxy_async_global();
            }
        }
        int s = 0;
        uint32_t ph = 0, armed = 0, armed_par = 0;
        bool aborted = false, waited = !own_tile;
        StreamCursor<kMode> c(pl, share_walk, p.nk);
        for (; c.valid; c.step(pl)) {
            if (kMode == kProj && !waited && c.k >= p.nk) {      // x @ A^T from here on
                grid_dependency_wait();
                fence_proxy_async_global();
                waited = true;
            }
            const bool go = wait_bar(empty_bar(s), ph ^ 1u, wctl, kWaitProducerB);
            if (!__all_sync(0xffffffffu, go)) { aborted = true; break; }
            const uint32_t fb = full_bar(s), dst = sbase + C::kOffB + s * C::kBBytes;
            if (lane == 0) {
                armed |= 1u << s;
                armed_par = (armed_par & ~(1u << s)) | (ph << s);
                if (kMode == kProj && c.k >= p.nk) {
                    const int u = c.k - p.nk;
                    const int s0 = pieces > 1 ? u / pieces : u * per_unit;
                    // an adapter's parts follow one another, and the adapters: one piece of v (past
                    // the last adapter it is not used)
                    const int rows = per_unit * p.parts * BN, box = rows <= 256 ? rows : rows / 2;
                    mbar_arrive_expect_tx(fb, static_cast<uint32_t>(rows * rb));
                    for (int j = 0; j < rows; j += box)
                        tma_load_2d(dst + j * rb, &maps.v, fb, pieces > 1 ? (u % pieces) * ucols : 0,
                                    (c.sg.tt * p.max_slots + s0) * p.parts * BN + j);
                } else {
                    mbar_arrive_expect_tx(fb, BN * 128);
                    if constexpr (kMode == kDown) tma_load_2d(dst, &maps.x, fb, c.kl * 128, c.li * BN);
                    else tma_load_2d(dst, &maps.x, fb, c.k * 128, c.sg.tt * BN);
                }
            }
            __syncwarp();
            if (c.new_words(kFp4, p.nk)) {
                const uint32_t dt = sbase + C::kOffSf + s * C::kSfBytes + 1024 + lane * 16;
                const int32_t* pt;
                if (kMode == kDown) pt = p.sft + ((long long)c.li * ((p.nk + 3) / 4) + (c.kl >> 2)) * BN;
                else pt = p.sft + (long long)(c.kl >> 2) * p.sft_ld + c.sg.tt * BN;
                const int nt = kMode == kDown ? BN : min(BN, p.tokens - c.sg.tt * BN);
#pragma unroll
                for (int j = 0; j < (BN + 31) / 32; ++j) {
                    const int i = j * 32 + lane;
                    const bool in = i < nt;
                    cp_async_4(dt + 4 * j, in ? pt + i : pt, in ? 4u : 0u);
                }
            }
            cp_async_mbar_arrive(fb);
            if (++s == C::kStages) { s = 0; ph ^= 1u; }
        }
        cp_async_wait_all();
        if (lane == 0 && (aborted || *abort_flag))
            for (int i = 0; i < C::kStages; ++i)
                if (armed >> i & 1u) drain_bar(full_bar(i), armed_par >> i & 1u, 20000000ull);
        __syncwarp();
    } else if (warp == 1 || warp == 9) {
        // ------------------------------------------------------------- MMA issuers
        // One for each 128-row block of the tile.  The whole warp takes the loop and the waits, one
        // elected lane issues: measured 0.14 us for a unit's four products and copies where a
        // single-lane loop takes 0.29, which, twice for one issuer, would pace the FP4 weights
        // (HBM 0.38 us a unit).
        {
            const int blk = warp == 1 ? 0 : 1;
            constexpr uint32_t kIdesc = make_idesc_stream(BN, kFp4);
            constexpr uint32_t kIdescBf16 = make_idesc_bf16(128, BN);
            // scale slots in rotation (this issuer's: its block's words, the tokens' words): FP4
            // weights bring new words every K-group, E4M3 every fourth
            constexpr uint32_t kSfSlots = kFp4 ? 4u : 2u;
            const uint32_t sf0 = tmem_base + C::kSfCol0 + 8 * blk;
            const uint64_t a0 = make_sdesc(sbase + blk * 16384, 0, 1024, kLayoutSw128);
            const uint64_t b0 = make_sdesc(sbase + C::kOffB, 0, 1024, kLayoutSw128);
            const uint64_t w0 = make_sdesc(sbase + C::kOffSf + 512 * blk, 0, 128, kLayoutNone);
            const uint64_t t0w = make_sdesc(sbase + C::kOffSf + 1024, 0, 128, kLayoutNone);
            // adapter units: an adapter's rows are rb bytes long, swizzled over as many
            const uint32_t layout = rb == 64 ? 4u : 6u;
            const uint64_t la0 = make_sdesc(sbase + blk * 128 * rb, 0, 8 * rb, layout);
            const uint64_t lb0 = make_sdesc(sbase + C::kOffB, 0, 8 * rb, layout);
            int s = 0, acc = 0;
            uint32_t ph = 0, acc_ph = 0, kcount = 0, turn_ph = 0;
            bool aborted = false;
            auto wait_all = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, wait_bar(bar, parity, wctl, kWaitMma)) != 0;
            };
            StreamWalk<kMode> walk(share_walk);
            StreamSeg sg;
            while (!aborted && walk.next(pl, sg)) {
                if (!wait_all(acce_bar(acc), acc_ph ^ 1u)) { aborted = true; break; }
                tc_fence_after();
                const uint32_t dt = tmem_base + (acc * 2 + blk) * BN;
                uint32_t add = 0;                     // 0: the first product of the segment overwrites
                int kl = kMode == kDown ? sg.k0 % p.nk : (kMode == kProj ? sg.f0 : sg.k0);   // K-group (kDown: within the expert)
                for (int i = 0; i < sg.k1 - sg.k0; ++i) {
                    const bool lora_unit = kMode == kProj && i >= sg.nf;
                    if (!wait_all(full_bar(s), ph)) { aborted = true; break; }
                    tc_fence_after();
                    const uint64_t ad = a0 + static_cast<uint64_t>((s * C::kABytes) >> 4);
                    const uint64_t bd = b0 + static_cast<uint64_t>((s * C::kBBytes) >> 4);
                    if (lora_unit) {
                        if (i == sg.nf && add) {
                            // let the scaled FP8 products finish before another kind adds to their sums
                            if (elect_one()) tc_commit(turn_of(blk));
                            __syncwarp();
                            if (!wait_all(turn_of(blk), turn_ph)) { aborted = true; break; }
                            turn_ph ^= 1u;
                            tc_fence_after();
                        }
                        const int u = sg.l0 + i - sg.nf;
                        const int nslots = slots_of(sg.tt);
                        const int cnt = pieces > 1 ? 1 : min(per_unit, nslots - u * per_unit);
                        if (elect_one()) {
                            uint64_t aj = la0 + static_cast<uint64_t>((s * C::kABytes) >> 4);
                            uint64_t bj = lb0 + static_cast<uint64_t>((s * C::kBBytes) >> 4);
                            uint32_t keep = add;
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                if (n >= cnt) break;
#pragma unroll
                                for (int o = 0; o < 3; ++o) {
                                    if (o >= p.parts) break;
#pragma unroll
                                    for (int c = 0; c < 2; ++c) {
                                        if (c >= rb / 32) break;
                                        tc_mma_bf16(dt, aj + 2 * c, bj + 2 * c, kIdescBf16, keep);
                                        keep = 1;
                                    }
                                    bj += BN / 16 * rb;
                                }
                                aj += 16 * rb;
                            }
                            tc_commit(empty_bar(s));
                        }
                        add = 1;
                    } else {
                        const uint32_t sf_id = static_cast<uint32_t>(kl) & 3u;
                        const bool words = kFp4 || i == 0 || sf_id == 0;
                        if (words) ++kcount;
                        const uint32_t t = sf0 + (kcount % kSfSlots) * 16;
                        if (elect_one()) {
                            if (words) {
                                const uint32_t so = static_cast<uint32_t>(s * C::kSfBytes) >> 4;
                                fence_proxy_async_smem();   // scale words written by cp.async
                                tc_cp_32x128b_warpx4(t, w0 + so);
                                tc_cp_32x128b_warpx4(t + 4, t0w + so);
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tc_mma_mxf8(dt, ad + 2 * j, bd + 2 * j,
                                            idesc_sf_ids(kIdesc, kFp4 ? static_cast<uint32_t>(j) : sf_id, sf_id), t, t + 4,
                                            j ? 1u : add);
                            tc_commit(empty_bar(s));
                        }
                        add = 1;
                    }
                    __syncwarp();
                    if (++s == C::kStages) { s = 0; ph ^= 1u; }
                    if (++kl == p.nk && kMode == kDown) kl = 0;
                }
                if (aborted) break;
                if (elect_one()) tc_commit(accf_bar(acc));
                __syncwarp();
                if (++acc == C::kNumAcc) { acc = 0; acc_ph ^= 1u; }
            }
            if (elect_one()) tc_commit(drain_of(blk));
            __syncwarp();
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(drain_of(blk), 0)) {
                if (globaltimer_ns() - t0 > p.timeout_ns) { record_status(p.status, kErrTimeout | kWaitDrain); break; }
            }
        }
        __syncwarp();
    } else if (warp == 8 || warp == 10) {
        // -------------------------------------------------------- scale loaders
        // Warp 8 fills the even stages of the unit sequence, warp 10 the odd ones.  Word (lane, j)
        // of a 512-byte atom holds row j * 32 + lane, the form tcgen05.cp reads.  The weights'
        // words are asked into L2 kAhead units early: a unit's words are a few short pieces of
        // the array, which come from HBM later than the unit's weight tile would.
        constexpr int kAhead = C::kStages + 6;
        const uint32_t par = warp == 8 ? 0u : 1u;
        int s = 0;
        uint32_t ph = 0, n = 0;
        StreamCursor<kMode> c(pl, share_walk, p.nk), ahead(c);
        auto words_of = [&](const StreamCursor<kMode>& at) {
            const int e = kMode == kGateUp ? list[at.sg.tile / p.row_tiles] : (kMode == kDown ? list[at.li] : 0);
            return p.sfw + e * p.sfw_gstride + (long long)(kFp4 ? at.kl : at.kl >> 2) * p.sfw_ld;
        };
        // first row of the tile's weight block b
        auto row_of = [&](const StreamCursor<kMode>& at, int b) {
            return kMode == kGateUp ? at.sg.tile % p.row_tiles * 128 + b * p.out_rows : at.sg.tile * 256 + b * 128;
        };
        auto prefetch = [&]() {
            if (ahead.new_words(kFp4, p.nk) && lane < 2) {
                const int i = kFp4 ? row_of(ahead, lane) : row_of(ahead, lane) >> 7;
                if (i < p.sfw_rows) prefetch_l2_bulk(words_of(ahead) + (i & ~3), kFp4 ? 512u : 16u);
            }
        };
        for (int i = 0; i < kAhead && ahead.valid; ++i, ahead.step(pl))
            if ((static_cast<uint32_t>(i) & 1u) == par) prefetch();
        for (; c.valid; c.step(pl), ++n) {
            if ((n & 1u) == par) {
                const bool go = wait_bar(empty_bar(s), ph ^ 1u, wctl, kWaitScales);
                if (!__all_sync(0xffffffffu, go)) break;
                if (c.new_words(kFp4, p.nk)) {
                    const uint32_t da = sbase + C::kOffSf + s * C::kSfBytes + lane * 16;
                    const int32_t* pw = words_of(c);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int row = row_of(c, b);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int i = kFp4 ? row + j * 32 + lane : row >> 7;
                            const bool in = i < p.sfw_rows;
                            cp_async_4(da + 512 * b + 4 * j, in ? pw + i : pw, in ? 4u : 0u);
                        }
                    }
                }
                cp_async_mbar_arrive(full_bar(s));
            }
            if (ahead.valid) {
                if (((n + kAhead) & 1u) == par) prefetch();
                ahead.step(pl);
            }
            if (++s == C::kStages) { s = 0; ph ^= 1u; }
        }
        cp_async_wait_all();
        __syncwarp();
    } else if (warp >= 4 && warp != 11) {
        // ----------------------------------------------------------------- epilogue
        // Group g's four warps hold the tile's 2 x 128 rows (thread = row of both blocks) and take
        // columns [g * BN/2, (g + 1) * BN/2), kChunk at a time.  The groups share nothing but the
        // accumulator's release: each joins, counts and finishes its own half of a cut tile.
        constexpr int kHalf = BN / 2, kChunk = C::kChunk, kJoin = C::kJoin;
        const int q = warp & 3, row = q * 32 + lane, grp = warp >= 8 ? 1 : 0;
        const int te = row;                                            // 0..127 over the group
        if (kMode == kDown || own_tile) grid_dependency_wait();
        if (own_tile && threadIdx.x == 128) grid_launch_dependents();
        if (p.spread && share == 0 && threadIdx.x == 128) {
            p.spread[kSpreadUnits] = pl.units;
            p.spread[kSpreadShares] = pl.shares;
            p.spread[kSpreadNk] = pl.nk;
            p.spread[kSpreadPieces] = pl.pieces;
            p.spread[kSpreadListed] = nlist;
        }
        if (p.spread && share == 0 && grp == 0)
            for (int i = te; i < nlist; i += 128) reinterpret_cast<uint16_t*>(p.spread + kSpreadWords)[i] = list[i];
        if (kMode == kDown && nlist == 0 && !p.spread && cl == 1) {
            // no token uses an expert of this shard: the sum is empty
            const long long n = (long long)p.tokens * p.out_rows;
            for (long long i = ((long long)blockIdx.x * 2 + grp) * 128 + te; i < n; i += (long long)gridDim.x * 256) {
                if (p.d_f32) static_cast<float*>(p.d)[i] = 0.0f;
                else static_cast<__nv_bfloat16*>(p.d)[i] = __float2bfloat16(0.0f);
            }
        }
        // The group's four warps.  Whether to give up is voted once per tile, so all four take the
        // same path and every barrier below is reached by all of them.
        auto esync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory"); };
        auto evote = [&](bool ok) {
            uint32_t r;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                         "bar.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(r) : "r"(ok ? 1u : 0u), "r"(1 + grp) : "memory");
            return r != 0;
        };
        uint32_t* red = reinterpret_cast<uint32_t*>(smem + C::kOffRed) + grp * 128;
        int red_at = 0;                                                // alternates: one wait per chunk
        constexpr long long part_tile = 2LL * BN * 128;                // floats of one partial
        // a partial: [half][chunk of columns][block][column][row]
        const int my_part = grp * 2 * kHalf * 128 + row;
        int acc = 0;
        uint32_t acc_ph = 0;
        StreamWalk<kMode> walk(share_walk);
        StreamSeg sg;
        if (kClusters && cl > 1) {
            // A tile's pieces are the CTAs of a cluster: each leaves its part in its own ring (idle: its
            // only tile's products are done), and each adds up every cl-th (column, 32 rows) of the
            // tile over the cluster, in piece order.
            float* xch = reinterpret_cast<float*>(smem);               // [column][block][row]
            const int rank = static_cast<int>(cluster_ctarank()), tile = share_walk.tile, token0 = share_walk.tt * BN;
            const int cols_all = min(BN, p.tokens - token0);
            uint32_t full = 0;                                         // pieces that are not empty
            for (int c = 0; c < cl; ++c)
                if (pl.fp8 >= cl || (c + 1 == cl ? pl.nk : piece_begin(pl, c + 1)) > piece_begin(pl, c)) full |= 1u << c;
            bool ok = true;
            if (walk.next(pl, sg)) {
                ok = evote(wait_bar(accf_bar(acc), acc_ph, wctl, kWaitEpilogue));
                tc_fence_after();
                if (ok) {
                    const uint32_t ta = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + grp * kHalf;
                    const int cols = min(kHalf, cols_all - grp * kHalf);
                    for (int c0 = 0; c0 < cols; c0 += kChunk) {
                        uint32_t r0[kChunk], r1[kChunk];
                        if constexpr (kChunk == 16) {
                            tmem_ld_32x32b_x16(ta + c0, r0);
                            tmem_ld_32x32b_x16(ta + BN + c0, r1);
                        } else {
                            tmem_ld_32x32b_x8(ta + c0, r0);
                            tmem_ld_32x32b_x8(ta + BN + c0, r1);
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            if (c0 + i >= cols) break;
                            xch[(grp * kHalf + c0 + i) * 256 + row] = __uint_as_float(r0[i]);
                            xch[(grp * kHalf + c0 + i) * 256 + 128 + row] = __uint_as_float(r1[i]);
                        }
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane < cl) mbar_arrive_remote(map_shared_rank(xfull_bar, lane));
            ok = wait_bar<true>(xfull_bar, 0, wctl, kWaitExchange) && ok;
            const uint32_t xbase = smem_u32(xch) + lane * 4;
            const int w = grp * 4 + q;
            if (__all_sync(0xffffffffu, ok)) {
                constexpr int kItems = BN >= 64 ? 4 : 1;               // at a time
                float bad = 0.0f;                                      // NaN behind a value that is not finite
                for (int i0 = rank + cl * w; i0 < cols_all * 8; i0 += cl * 8 * kItems) {
                    float v[kItems], x[kItems][8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
#pragma unroll
                        for (int n = 0; n < kItems; ++n) {
                            const int it = i0 + cl * 8 * n;
                            x[n][c] = (full >> c & 1u) && it < cols_all * 8 ? ld_dsmem_f32(map_shared_rank(xbase + it * 128, c)) : 0.0f;
                        }
#pragma unroll
                    for (int n = 0; n < kItems; ++n) {
                        v[n] = x[n][0];
#pragma unroll
                        for (int c = 1; c < 8; ++c) v[n] += x[n][c];
                        const int it = i0 + cl * 8 * n, t = it >> 3, r = tile * 256 + (it & 7) * 32 + lane;
                        if (it < cols_all * 8 && r < p.out_rows) {
                            const long long at = (long long)(token0 + t) * p.out_rows + r;
                            if (p.d_f32) static_cast<float*>(p.d)[at] = v[n];
                            else static_cast<__nv_bfloat16*>(p.d)[at] = __float2bfloat16(v[n]);
                            bad = fmaf(v[n], 0.0f, bad);
                        }
                    }
                }
                if (__builtin_expect(bad != 0.0f, 0) && cols_all > 1) {
#pragma unroll 1
                    for (int it = rank + cl * w; it < cols_all * 8; it += cl * 8) {
                        const int r = tile * 256 + (it & 7) * 32 + lane;
                        if (r < p.out_rows) mend_outputs<kMode, BN>(p, list, nlist, share_walk.tt, it >> 3, 1, r);
                    }
                }
            }
        }
        while (walk.next(pl, sg)) {
            if constexpr (kMode == kGateUp) {
                // the tile's routing weights, while its weights stream
                const int expert = p.expert_base + list[sg.tile / p.row_tiles];
                if (te < kHalf) {
                    const int t = grp * kHalf + te;
                    float w = 0.0f, on = 0.0f;
                    if (t < p.tokens) {
                        const int32_t* ids = p.ids + (long long)t * p.topk;
                        const float* weights = p.weights + (long long)t * p.topk;
                        for (int j0 = 0; j0 < p.topk; j0 += 8) {
                            int id[8];
                            float x[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const bool in = j0 + j < p.topk;
                                id[j] = in ? __ldg(ids + j0 + j) : -1;
                                x[j] = in ? __ldg(weights + j0 + j) : 0.0f;
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (id[j] == expert && j0 + j < p.topk) { w += x[j]; on = 1.0f; }
                        }
                    }
                    tok[t] = make_float2(w, on);
                }
            }
            if (!evote(wait_bar(accf_bar(acc), acc_ph, wctl, kWaitEpilogue))) break;
            tc_fence_after();
            // token columns of this group that exist
            const int cols = min(kHalf, min(BN, p.tokens - sg.tt * BN) - grp * kHalf);
            const uint32_t ta = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 2 * BN + grp * kHalf;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce_bar(acc));
            };
            // columns c0.. of both blocks from the accumulator
            auto load_acc = [&](int c0, float (&v0)[kChunk], float (&v1)[kChunk]) {
                uint32_t r0[kChunk], r1[kChunk];
                if constexpr (kChunk == 16) {
                    tmem_ld_32x32b_x16(ta + c0, r0);
                    tmem_ld_32x32b_x16(ta + BN + c0, r1);
                } else {
                    tmem_ld_32x32b_x8(ta + c0, r0);
                    tmem_ld_32x32b_x8(ta + BN + c0, r1);
                }
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < kChunk; ++i) { v0[i] = __uint_as_float(r0[i]); v1[i] = __uint_as_float(r1[i]); }
            };
            int c_first = share, c_last = share;
            if (!sg.whole || p.spread) {
                // this share's part of the tile: 0 where the tile began in an earlier share, else 1
                float* mine = p.part + (2LL * share + (sg.k0 > 0 ? 0 : 1)) * part_tile + my_part;
                for (int c0 = 0; c0 < cols; c0 += kChunk) {
                    float v0[kChunk], v1[kChunk];
                    load_acc(c0, v0, v1);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        if (c0 + i >= cols) break;
                        __stcg(mine + (2 * c0 + i) * 128, v0[i]);
                        __stcg(mine + (2 * c0 + kChunk + i) * 128, v1[i]);
                    }
                }
                release();
                if (cols <= 0 || p.spread) {
                    if (++acc == C::kNumAcc) { acc = 0; acc_ph ^= 1u; }
                    continue;
                }
                shares_of(pl, sg.first_unit, sg.nk, c_first, c_last);
                esync();
                if (te == 0) {
                    // only the last tile that begins in a share goes on into the next one, so a cut
                    // tile is told by its first share; the count wraps to 0 with the last arrival
                    const unsigned n = static_cast<unsigned>(c_last - c_first);
                    __threadfence();                     // this group's stores, ordered by the barrier
                    last_flag[grp] = atomicInc(p.ctr + 2 * c_first + grp, n) == n;
                    __threadfence();
                }
                esync();
                if (!last_flag[grp]) {
                    if (++acc == C::kNumAcc) { acc = 0; acc_ph ^= 1u; }
                    continue;
                }
            }
            // ---- finish the tile
            // Partials of the share's last tile come through the ring, idle by now (this tile's
            // products were its last): pieces (chunk, share) in order, kJoinSlots in flight, issued by
            // the four warps in turn (one thread's bulk copies complete one after another).  Those of
            // an earlier tile, joined while others stream, come into registers.
            const bool few = cols <= 2;
            const bool by_ring = !sg.whole && !few && walk.done();
            const int n_parts = c_last - c_first + 1;
            const int pieces_all = by_ring ? (cols + kChunk - 1) / kChunk * n_parts : 0;
            const uint32_t jbuf = sbase + grp * C::kJoinSlots * C::kPieceBytes;
            const float* jsmem = reinterpret_cast<const float*>(smem + grp * C::kJoinSlots * C::kPieceBytes);
            auto part_of = [&](int c) {
                return p.part + (2LL * c + (share_begin(pl, c) > sg.first_unit ? 0 : 1)) * part_tile + grp * 2 * kHalf * 128;
            };
            int fetched = 0;
            auto fetch = [&](int i) {                    // piece i of the join; lane 0 of warp i mod 4
                fetched = i + 1;
                const int ch = i / n_parts, slot = i % C::kJoinSlots;
                mbar_arrive_expect_tx(join_bar(grp, slot), C::kPieceBytes);
                bulk_load(jbuf + slot * C::kPieceBytes, part_of(c_first + i - ch * n_parts) + ch * 2 * kChunk * 128,
                          C::kPieceBytes, join_bar(grp, slot));
            };
            if (by_ring && lane == 0) {
                fence_proxy_async_global();
                for (int i = q; i < min(pieces_all, C::kJoinSlots); i += 4) fetch(i);
            }
            int piece = 0;
            bool lost = false;
            float bad = 0.0f, bad2 = 0.0f;               // NaN behind a value that is not finite
            for (int c0 = 0; c0 < cols; c0 += kChunk) {
                const int t0 = grp * kHalf + c0;                       // first token column
                float v0[kChunk], v1[kChunk];
                if (sg.whole) {
                    load_acc(c0, v0, v1);
                    if (c0 + kChunk >= cols) release();
                } else if (by_ring) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v0[i] = v1[i] = 0.0f;
                    for (int c = 0; c < n_parts; ++c, ++piece) {
                        const int slot = piece % C::kJoinSlots;
                        if (!wait_bar(join_bar(grp, slot), (piece / C::kJoinSlots) & 1, wctl, kWaitExchange)) lost = true;
                        const float* src = jsmem + slot * (C::kPieceBytes / 4) + row;
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            v0[i] += src[i * 128];
                            v1[i] += src[(kChunk + i) * 128];
                        }
                        if (piece + C::kJoinSlots < pieces_all) {
                            esync();                                   // the slot is free
                            if (lane == 0 && ((piece + C::kJoinSlots) & 3) == q && !lost) fetch(piece + C::kJoinSlots);
                        }
                    }
                } else if (few) {
                    // one or two columns: eight partials in flight
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v0[i] = v1[i] = 0.0f;
                    for (int c = c_first; c <= c_last; c += 8) {
                        float x[8][4];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float* src = part_of(min(c + u, c_last)) + row;
                            x[u][0] = __ldcg(src);
                            x[u][1] = __ldcg(src + kChunk * 128);
                            x[u][2] = __ldcg(src + (cols - 1) * 128);
                            x[u][3] = __ldcg(src + (kChunk + cols - 1) * 128);
                        }
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            if (c + u <= c_last) {
                                v0[0] += x[u][0];
                                v1[0] += x[u][1];
                                v0[1] += x[u][2];
                                v1[1] += x[u][3];
                            }
                    }
                } else {
                    // the partials in share order, kJoin of them in flight
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v0[i] = v1[i] = 0.0f;
                    for (int c = c_first; c <= c_last; c += kJoin) {
                        float x0[kJoin][kChunk], x1[kJoin][kChunk];
#pragma unroll
                        for (int u = 0; u < kJoin; ++u) {
                            const float* src = part_of(min(c + u, c_last)) + 2 * c0 * 128 + row;
#pragma unroll
                            for (int i = 0; i < kChunk; ++i) {
                                x0[u][i] = __ldcg(src + i * 128);
                                x1[u][i] = __ldcg(src + (kChunk + i) * 128);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < kJoin; ++u)
                            if (c + u <= c_last) {
#pragma unroll
                                for (int i = 0; i < kChunk; ++i) { v0[i] += x0[u][i]; v1[i] += x1[u][i]; }
                            }
                    }
                }
                if constexpr (kMode == kGateUp) {
                    // y = w * SiLU(gate) * up, then one scale for each token's 128 values (the rows of
                    // this block): maximum of |y| over the warp's lanes, then over the four warps.
                    // Lane i of every warp works out column i's scale for the others.  The exponential and the
                    // division are the fast ones: with expf and a rounded division 128 x 7168 takes 257.7
                    // us instead of 253.8, 1 x 4096 37.2 instead of 35.5, and the same 26 of 1.6 million
                    // codes fall to the other side of a rounding than in FP64 (the sums over K decide; 6
                    // with an FP32 matrix product).
                    uint32_t* rd = red + red_at;
                    red_at ^= 64;
                    uint32_t m[kChunk];
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        const float2 w = tok[t0 + i];
                        const float y = swiglu_value(__float_as_uint(v0[i]), __float_as_uint(v1[i])) * w.x;
                        v0[i] = w.y != 0.0f ? y : 0.0f;
                        m[i] = __float_as_uint(v0[i]) & 0x7fffffffu;
                    }
                    const uint32_t top = column_max<kChunk>(m, lane);
                    if ((lane & (32 / kChunk - 1)) == 0) rd[q * 16 + column_of<kChunk>(lane)] = top;
                    esync();
                    const int li = sg.tile / p.row_tiles, it = sg.tile % p.row_tiles;
                    const int lc = lane & (kChunk - 1);
                    const uint32_t all = max(max(rd[lc], rd[16 + lc]), max(rd[32 + lc], rd[48 + lc]));
                    const bool finite = all < 0x7f800000u;
                    const int e = finite ? scale_exponent(__uint_as_float(all)) : 0;
                    const float sc = finite ? pow2_neg(e) : __int_as_float(0x7fc00000);   // not finite: NaN codes
                    if (q == 0 && lane < kChunk && c0 + lane < cols)
                        p.sfh[(((long long)li * ((p.row_tiles + 3) / 4) + (it >> 2)) * BN + t0 + lane) * 4 + (it & 3)] =
                            static_cast<uint8_t>(e + 127);
                    uint8_t* hq = p.hq + ((long long)li * BN + t0) * p.out_rows + it * 128;
                    if constexpr (BN >= 32) {
                        // the codes by way of shared memory, 16 bytes of a token a thread: a byte a row and
                        // token takes 0.6 us of stores a chunk, of 1.7 (128 x 7168 255.5 -> 253.4 us; 1 x
                        // 4096, where few columns are stored, 34.4 -> 34.5)
                        uint8_t* codes = smem + C::kOffCodes + grp * 16 * 128;
#pragma unroll
                        for (int i = 0; i < kChunk; i += 2) {
                            const float x = v0[i] * __shfl_sync(0xffffffffu, sc, i), y = v0[i + 1] * __shfl_sync(0xffffffffu, sc, i + 1);
                            const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
                            codes[i * 128 + row] = static_cast<uint8_t>(two);
                            codes[(i + 1) * 128 + row] = static_cast<uint8_t>(two >> 8);
                        }
                        esync();
                        const int ct = te >> 3, cr = (te & 7) * 16;
                        if (c0 + ct < cols)
                            *reinterpret_cast<uint4*>(hq + (long long)ct * p.out_rows + cr) =
                                *reinterpret_cast<const uint4*>(codes + ct * 128 + cr);
                    } else {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            const float x = v0[i] * __shfl_sync(0xffffffffu, sc, i);
                            if (c0 + i < cols) hq[(long long)i * p.out_rows + row] = static_cast<uint8_t>(e4m3(x));
                        }
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int r = sg.tile * 256 + b * 128 + row;
                        if (r < p.out_rows) {
                            const long long at = ((long long)sg.tt * BN + t0) * p.out_rows + r;
#pragma unroll
                            for (int i = 0; i < kChunk; ++i) {
                                if (c0 + i >= cols) break;
                                const float x = b ? v1[i] : v0[i];
                                if (p.d_f32) static_cast<float*>(p.d)[at + (long long)i * p.out_rows] = x;
                                else static_cast<__nv_bfloat16*>(p.d)[at + (long long)i * p.out_rows] = __float2bfloat16(x);
                                if (i & 1) bad = fmaf(x, 0.0f, bad);
                                else bad2 = fmaf(x, 0.0f, bad2);
                            }
                        }
                    }
                }
            }
            if (sg.whole && cols <= 0) release();
            if (kMode != kGateUp && __builtin_expect(bad + bad2 != 0.0f, 0) && p.tokens > 1) {
#pragma unroll 1
                for (int r = sg.tile * 256 + row; r < min(p.out_rows, (sg.tile + 1) * 256); r += 128)
                    mend_outputs<kMode, BN>(p, list, nlist, sg.tt, grp * kHalf, cols, r);
            }
            if (lost && lane == 0)     // pieces that may still be landing
                for (int i = fetched - 1; i >= 0 && i >= fetched - C::kJoinSlots; i -= 4)
                    drain_bar(join_bar(grp, i % C::kJoinSlots), (i / C::kJoinSlots) & 1, 20000000ull);
            if (!evote(!lost)) break;
            if (++acc == C::kNumAcc) { acc = 0; acc_ph ^= 1u; }
        }
        if (kMode == kGateUp) fence_proxy_async_global();
    }
    tc_fence_before();
    // a cluster's parts stay in place until all its CTAs have read them
    __syncwarp();
    if (cl > 1) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
}

// Adds up the parts of every tile (spread joins).  With 64 or more token columns a part is 64 KB or
// more, and one SM reads about 55 GB/s: the last arrival of nine would take 11 us to join them,
// while all SMs together read all tiles' parts in about 2.  One CTA per (tile, kSpreadCols columns),
// thread = row of the tile; the parts are added in share order, eight in flight.
constexpr int kSpreadCols = 4;
template <int BN>
__global__ void __launch_bounds__(256) stream_reduce_kernel(const __grid_constant__ StreamParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int* spread = p.spread;
    const float* part = p.part;
    const int tokens = p.tokens, out_rows = p.out_rows;
    constexpr int kChunk = 16, kHalf = BN / 2;
    StreamPlan pl;
    pl.units = __ldcg(spread + kSpreadUnits);
    pl.shares = __ldcg(spread + kSpreadShares);
    pl.nk = __ldcg(spread + kSpreadNk);
    pl.pieces = __ldcg(spread + kSpreadPieces);
    pl.q = pl.units / pl.shares;
    pl.r = pl.units - pl.q * pl.shares;
    pl.fp8 = pl.nk;
    const int tile = blockIdx.x, c0 = blockIdx.y * kSpreadCols;
    const int row = threadIdx.x & 127, blk = threadIdx.x >> 7;
    const int cols = min(kSpreadCols, tokens - c0);
    float v[kSpreadCols] = {};
    if (pl.units > 0) {
        int first, last;
        const int first_unit = tile * pl.nk;
        shares_of(pl, first_unit, pl.nk, first, last);
        // [half][chunk][block][column][row] within a part
        const int in_half = c0 % kHalf;
        const float* at = part + (c0 / kHalf) * 2 * kHalf * 128 +
                          (2 * (in_half / kChunk * kChunk) + blk * kChunk + in_half % kChunk) * 128 + row;
        for (int c = first; c <= last; c += 8) {
            float x[8][kSpreadCols];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int cc = min(c + u, last);
                const float* src = at + (2LL * cc + (share_begin(pl, cc) > first_unit ? 0 : 1)) * 2 * BN * 128;
#pragma unroll
                for (int i = 0; i < kSpreadCols; ++i) x[u][i] = i < cols ? __ldcg(src + i * 128) : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (c + u <= last) {
#pragma unroll
                    for (int i = 0; i < kSpreadCols; ++i) v[i] += x[u][i];
                }
        }
    }
    const int r = tile * 256 + blk * 128 + row;
    if (r >= out_rows) return;
    const long long out = (long long)c0 * out_rows + r;
    float bad = 0.0f;                             // NaN behind a value that is not finite
#pragma unroll
    for (int i = 0; i < kSpreadCols; ++i) {
        if (i >= cols) break;
        if (p.d_f32) static_cast<float*>(p.d)[out + (long long)i * out_rows] = v[i];
        else static_cast<__nv_bfloat16*>(p.d)[out + (long long)i * out_rows] = __float2bfloat16(v[i]);
        bad = fmaf(v[i], 0.0f, bad);
    }
    if (__builtin_expect(bad != 0.0f, 0)) {
        const uint16_t* list = reinterpret_cast<const uint16_t*>(spread + kSpreadWords);
        const int nlist = __ldcg(spread + kSpreadListed);
        mend_outputs<kDown, BN>(p, list, nlist, 0, c0, cols, r);
    }
}

inline cudaError_t launch_reduce(int bn, const StreamParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.row_tiles), static_cast<unsigned>((p.tokens + kSpreadCols - 1) / kSpreadCols));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (p.pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return bn == 64 ? cudaLaunchKernelEx(&cfg, stream_reduce_kernel<64>, p)
                    : cudaLaunchKernelEx(&cfg, stream_reduce_kernel<128>, p);
}

template <int kMode, int BN, bool kFp4>
struct StreamLaunch {
    using C = StreamCfg<kMode, BN>;
    // The current device, its kernel's shared memory allowed (again is harmless).
    static cudaError_t device(int* dev) {
        static bool configured[256] = {};
        cudaError_t err = cudaGetDevice(dev);
        if (err != cudaSuccess) return err;
        if (*dev < 0 || *dev >= 256) return cudaErrorInvalidDevice;
        if (!configured[*dev]) {
            err = cudaFuncSetAttribute(fg_stream_kernel<kMode, BN, kFp4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmemBytes);
            if (err != cudaSuccess) return err;
            configured[*dev] = true;
        }
        return cudaSuccess;
    }
    static void config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, dim3 grid, int cluster, int pdl, cudaStream_t stream) {
        cfg.gridDim = grid;
        cfg.blockDim = dim3(C::kThreads);
        cfg.dynamicSmemBytes = C::kSmemBytes;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 0;
        if (cluster > 1) {
            attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
            attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(cluster);
            attr[cfg.numAttrs].val.clusterDim.y = 1;
            attr[cfg.numAttrs].val.clusterDim.z = 1;
            ++cfg.numAttrs;
        }
        if (pdl) {
            attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
            ++cfg.numAttrs;
        }
    }
    static cudaError_t launch(const StreamParams& p, const StreamMaps& maps, dim3 grid, cudaStream_t stream) {
        int dev = 0;
        const cudaError_t err = device(&dev);
        if (err != cudaSuccess) return err;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        config(cfg, attr, grid, p.cluster, p.pdl, stream);
        return cudaLaunchKernelEx(&cfg, fg_stream_kernel<kMode, BN, kFp4>, p, maps);
    }
    // How many clusters of `cluster` CTAs run at once (0: unknown).
    static int resident(int cluster) {
        static int known[256][9] = {};           // + 1; asked again at worst
        int dev = 0;
        if (device(&dev) != cudaSuccess) return 0;
        if (!known[dev][cluster]) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[2];
            int n = 0;
            config(cfg, attr, dim3(static_cast<unsigned>(cluster)), cluster, 0, nullptr);
            if (cudaOccupancyMaxActiveClusters(&n, fg_stream_kernel<kMode, BN, kFp4>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            known[dev][cluster] = n + 1;
        }
        return known[dev][cluster] - 1;
    }
};

template <int kMode, bool kFp4>
cudaError_t launch_stream(int bn, const StreamParams& p, const StreamMaps& maps, dim3 grid, cudaStream_t stream) {
    switch (bn) {
        case 16: return StreamLaunch<kMode, 16, kFp4>::launch(p, maps, grid, stream);
        case 32: return StreamLaunch<kMode, 32, kFp4>::launch(p, maps, grid, stream);
        case 64: return StreamLaunch<kMode, 64, kFp4>::launch(p, maps, grid, stream);
        default: return StreamLaunch<kMode, 128, kFp4>::launch(p, maps, grid, stream);
    }
}

// CTAs that share a tile of `tiles` as a cluster: the most whose clusters are all resident at once
// on `sms` SMs; 1 where not even three are (the shares are then dealt and joined through the
// workspace).
template <int kMode, bool kFp4>
int stream_cluster(int bn, int tiles, int sms) {
    for (int s = 8; s > 2; --s) {
        if (tiles * s > sms) continue;
        int n = 0;
        switch (bn) {
            case 16: n = StreamLaunch<kMode, 16, kFp4>::resident(s); break;
            case 32: n = StreamLaunch<kMode, 32, kFp4>::resident(s); break;
            case 64: n = StreamLaunch<kMode, 64, kFp4>::resident(s); break;
            default: n = StreamLaunch<kMode, 128, kFp4>::resident(s); break;
        }
        if (tiles <= n) return s;
    }
    return 1;
}

// Token columns of a tile: the smallest width that holds them.
inline int stream_bn(int tokens) { return tokens <= 16 ? 16 : (tokens <= 32 ? 32 : (tokens <= 64 ? 64 : 128)); }

}  // namespace fg
