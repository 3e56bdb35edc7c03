
#include <cstdio>
#include <cstdint>
#include <cstring>
#include <cmath>
#include <algorithm>
using std::min; using std::max;
#define __device__
#define __forceinline__ inline
struct D3 { int x; } threadIdx, blockIdx, gridDim;
static uint32_t lanes[32]; static int passno;
static uint32_t __reduce_min_sync(uint32_t, uint32_t v) { if (!passno) { lanes[threadIdx.x] = v; return v; } uint32_t m = ~0u; for (auto l : lanes) m = std::min(m, l); return m; }
static float __fdividef(float a, float b) { return a / b; }
static uint32_t __float_as_uint(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
enum StreamMode : int { kGateUp = 0, kDown = 1, kProj = 2 };
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
    if (pl.units == 0) {      // no token uses an expert of this shard: no share, so nothing is read or counted
        pl.pieces = pl.shares = pl.q = pl.r = 0;
        return;
    }
    pl.shares = pl.pieces > 0 ? pl.pieces * tiles : min(grid, pl.pieces < 0 ? tiles : pl.units);
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


int main() {
  int bad = 0;
  for (int H : {256, 1408, 2048, 4096, 7168}) for (int I : {512, 2048}) for (int nlist : {0, 1, 3, 32}) for (int fp4 = 0; fp4 < 2; ++fp4)
  for (int mode = 0; mode < 2; ++mode) for (int grid : {1, 3, 152}) for (int spread = 0; spread <= (mode == 1); ++spread) {
    StreamPlan pl{}; int nkp = mode ? I / 128 : H / 128; pl.row_tiles = mode ? (H + 255) / 256 : I / 128;
    if (spread && pl.row_tiles > grid) continue;
    pl.nk = mode ? nlist * nkp : nkp;
    pl.units = mode ? pl.row_tiles * pl.nk : nlist * pl.row_tiles * pl.nk; pl.fp8 = pl.nk;
    StreamPlan p0 = pl;
    int tiles = mode ? pl.row_tiles : nlist * pl.row_tiles;
    for (passno = 0; passno < 2; ++passno) for (int l = 31; l >= 0; --l) { threadIdx.x = l; pl = p0; plan_shares(pl, tiles, grid, fp4, 1, mode ? 8 : 0, spread); }
    long got = 0; int counted = 0, segs = 0;
    for (int c = 0; c < grid; ++c) {
      blockIdx.x = c;
      auto go = [&](auto w) { StreamSeg s; while (w.next(pl, s)) { ++segs; got += s.k1 - s.k0; if (!s.whole) ++counted; } };
      if (mode) go(StreamWalk<kDown>(pl, c)); else go(StreamWalk<kGateUp>(pl, c));
    }
    if (got != pl.units) { ++bad; printf("H %d I %d listed %d fp4 %d mode %d grid %d spread %d: units %d, dealt %ld in %d segments (%d cut), pieces %d shares %d\n", H, I, nlist, fp4, mode, grid, spread, pl.units, got, segs, counted, pl.pieces, pl.shares); }
  }
  printf("%d wrong\n", bad); return bad != 0;
}
