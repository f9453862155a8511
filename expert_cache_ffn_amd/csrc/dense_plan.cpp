// Which kernel a dense product takes, and how it is cut: host code without HIP calls.
#include <algorithm>

#include "dense_internal.h"

namespace ecf {
namespace {

// A tile of the output and what it costs: `us` per k-tile of 64 with per_cu blocks
// on every CU (measured, K 4096), `us1` with one, `fixed` per block for filling the
// pipeline and the epilogue.  us1 and fixed are fitted to every tile and split of
// 6000 products of 1 to 8192 tokens and up to 40 GFLOP: the choice takes 1.7% longer
// than the best of them on the geometric mean.
struct TileCost {
    int bm, bn, per_cu;
    double us, us1, fixed;
};
const TileCost kTilesDma[] = {{256, 256, 1, 1.78, 1.78, 10.9}, {128, 256, 1, 0.98, 0.98, 5.7},
                              {128, 128, 2, 1.05, 0.74, 5.3}, {64, 128, 2, 0.66, 0.34, 5.1},
                              {64, 64, 2, 0.45, 0.25, 2.5}};
const TileCost kTilesReg[] = {{256, 256, 1, 1.92, 1.92, 13.6}, {128, 256, 1, 1.14, 1.14, 8.0},
                              {128, 128, 2, 1.25, 0.83, 7.6}, {64, 64, 2, 0.64, 0.45, 2.8}};
const TileCost kTilesF32[] = {{128, 128, 1, 2.70, 2.70, 5.9}, {64, 128, 1, 1.75, 1.75, 6.3}, {64, 64, 1, 1.00, 1.00, 5.8}};
constexpr int kShortK = 32;

const TileCost *tiles_of(int dtype, bool dma) { return dtype == ECF_F32 ? kTilesF32 : dma ? kTilesDma : kTilesReg; }
int tile_count(int dtype, bool dma) { return dtype == ECF_F32 ? 3 : dma ? 5 : 4; }

bool aligned16(const void *p, int64_t ld, int dtype)
{
    return (uintptr_t)p % 16 == 0 && ld * (int64_t)dense_esize(dtype) % 16 == 0;
}

constexpr int kMaxSplits = 16;
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, kMaxSplits};
constexpr int kSplitTiles = 2;  // least k-tiles of a split
constexpr double kLaunchUs = 5.0;  // one launch more, host and device

// Rows at 16-byte boundaries and whole 16-byte chunks: operands can go straight to LDS.
bool dma_ok(const DenseGemm &g)
{
    if (g.dtype == ECF_F32)
        return false;
    for (int s = 0; s < g.ksegs || s < g.mhalves; ++s)
        if (!aligned16(g.a[s], g.lda, g.dtype))
            return false;
    for (int s = 0; s < (g.gated || g.ksegs == 2 ? 2 : 1); ++s)
        if (!aligned16(g.b[s], g.ldb, g.dtype))
            return false;
    return (g.a_padded || (g.a_t ? g.M : g.K) % 8 == 0) && (g.b_t ? g.N : g.K) % 8 == 0;
}

// Rows too short for the MFMA tiles' chunks, or (fp32) a reduction too short to be worth them.
bool short_rows(const DenseGemm &g)
{
    return (g.a_t ? g.M : g.K) < 8 || (g.b_t ? g.N : g.K) < 8 || (g.dtype == ECF_F32 && g.K < kShortK);
}

int ktiles(const DenseGemm &g) { return (g.K + 63) / 64 * g.ksegs; }
int64_t out_tiles(const DenseGemm &g, const TileCost &c)
{
    const int bn = c.bn / (g.gated ? 2 : 1);
    return (int64_t)((g.M + c.bm - 1) / c.bm) * g.mhalves * ((g.N + bn - 1) / bn);
}
// Bytes of the partial sums, and the join's time for them.
double partial_bytes(const DenseGemm &g, int splits)
{
    return splits > 1 ? (double)splits * (g.gated ? 2 : g.mhalves) * g.M * ((g.N + 7) / 8 * 8) * 4 : 0.0;
}
double join_us(const DenseGemm &g, int splits) { return splits > 1 ? 3.0 + partial_bytes(g, splits) * 2 / 5e6 : 0.0; }
bool may_split(const DenseGemm &g, int splits, size_t room)
{
    return splits == 1 || (ktiles(g) / splits >= kSplitTiles && partial_bytes(g, splits) <= (double)room);
}

// The tile and the splits of K with the least estimated time: rounds of blocks
// over the CUs times the k-tiles each walks, plus the join of the splits.
DensePlan plan_gemm(const DenseGemm &g, int cus, size_t room, double *us_out)
{
    DensePlan best{0, 1, dma_ok(g)};
    const int n_tiles = tile_count(g.dtype, best.dma), kt = ktiles(g);
    const TileCost *tiles = tiles_of(g.dtype, best.dma);
    *us_out = 1e300;
    for (int t = 0; t < n_tiles; ++t) {
        const TileCost &c = tiles[t];
        for (const int s : kSplits) {
            if (!may_split(g, s, room))
                break;
            // full rounds of per_cu blocks on every CU, then what is left
            const int64_t blocks = out_tiles(g, c) * s, round = (int64_t)cus * c.per_cu, rest = blocks % round;
            const double walk = (double)((kt + s - 1) / s);
            const double tail = rest == 0 ? 0.0 : walk * (rest <= cus ? c.us1 : c.us) + c.fixed;
            const double us = (double)(blocks / round) * (walk * c.us + c.fixed) + tail + join_us(g, s);
            if (us < *us_out) {
                *us_out = us;
                best.tile = t;
                best.splits = s;
            }
        }
    }
    return best;
}

// When the last of n1 blocks that take k1 and, behind them, n2 that take k2 (k1 >= k2)
// is done, on `slots` slots that each take the next block when they are free.
double makespan(int64_t n1, double k1, int64_t n2, double k2, int64_t slots)
{
    const int64_t left = n1 % slots;  // slots that start one more long block at t0
    const double t0 = (double)(n1 / slots) * k1;
    double t = left ? t0 + k1 : t0;
    if (n2 == 0)
        return t;
    // the others go on with short blocks at t0, those `left` at t0 + k1
    int64_t early = 0, late = 0;
    while (early * (slots - left) + late * left < n2) {
        const double next_early = t0 + (double)(early + 1) * k2, next_late = t0 + k1 + (double)(late + 1) * k2;
        if (left == 0 || (left < slots && next_early <= next_late)) {
            ++early;
            t = std::max(t, next_early);
        } else {
            ++late;
            t = std::max(t, next_late);
        }
        if (early + late > 64)  // many rounds: the work over all slots says it well enough
            return std::max(t, ((double)n1 * k1 + (double)n2 * k2) / (double)slots);
    }
    return t;
}

// The same for two products in one launch.
DensePair plan_pair(const DenseGemm &gx, const DenseGemm &gw, int cus, size_t room, double *us_out)
{
    DensePair best{{0, 1, dma_ok(gx) && dma_ok(gw)}, 1, 0};
    const size_t each = kDensePartialBytes / 2;  // and both together within the room
    const int n_tiles = tile_count(gx.dtype, best.x.dma);
    const TileCost *tiles = tiles_of(gx.dtype, best.x.dma);
    *us_out = 1e300;
    for (int t = gx.dtype == ECF_F32 ? 0 : 2; t < n_tiles; ++t) {  // (the large 16-bit tiles: apart)
        const TileCost &c = tiles[t];
        const int64_t slots = (int64_t)cus * c.per_cu;
        for (const int sx : kSplits) {
            if (!may_split(gx, sx, std::min(each, room)))
                break;
            const size_t at_w = (dense_partials(gx, sx) + 255) & ~(size_t)255;
            for (const int sw : kSplits) {
                // (one of the two reductions is long, and splitting the short one too
                // gains nothing)
                if ((sx > 2 && sw > 2) || !may_split(gw, sw, std::min(each, room - std::min(at_w, room))))
                    break;
                const int64_t bx = out_tiles(gx, c) * sx, bw = out_tiles(gw, c) * sw;
                const double us_k = bx + bw <= cus ? c.us1 : c.us;
                const double tx = (double)((ktiles(gx) + sx - 1) / sx) * us_k + c.fixed;
                const double tw = (double)((ktiles(gw) + sw - 1) / sw) * us_k + c.fixed;
                const double us = (tx >= tw ? makespan(bx, tx, bw, tw, slots) : makespan(bw, tw, bx, tx, slots)) +
                                  join_us(gx, sx) + join_us(gw, sw);
                if (us < *us_out) {
                    *us_out = us;
                    best.x.tile = t;
                    best.x.splits = sx;
                    best.splits_w = sw;
                    best.at_w = at_w;
                }
            }
        }
    }
    return best;
}

// 16-bit rows that start at odd elements.
bool odd_rows(const DenseGemm &g)
{
    const uintptr_t at = (uintptr_t)g.a[0] | (uintptr_t)g.b[0] | (uintptr_t)(g.gated ? g.b[1] : nullptr);
    return g.dtype != ECF_F32 && (g.lda % 2 || g.ldb % 2 || at % 4);
}

// Rows per block (4, 8 or 16; at most four groups of tokens) with the least time, and
// that time in us.  A CU takes in about 40 KB/us of weights and x together, whatever
// it is (4096 x 4096 bf16: 8 tokens 9.9 us, 64 tokens 21 us; 1024 x 4096: 4.4 and 7.6),
// and 17 KB/us where 16-bit rows start at odd elements, whose loads the hardware
// splits (7353 x 2048 bf16, 8 tokens: 20.8 us).  Fitted against the tiles on 840 calls
// of up to 64 tokens: the choice between the two costs 1.5% over the better one.
int few_rows(const DenseGemm &g, int cus, double *us)
{
    const int es = (int)dense_esize(g.dtype), h = g.gated ? 2 : 1;
    const bool odd = odd_rows(g);
    int best = 16;
    *us = 1e300;
    for (int rt = 4; rt <= 16; rt *= 2) {
        const int64_t blocks = (g.N + rt - 1) / rt, tokens = (g.M + rt - 1) / rt * rt;
        if (tokens > 4 * rt)
            continue;
        const double t = (es == 2 ? 4.0 : 2.5) +
                         (double)((blocks + cus - 1) / cus) * (rt * h + tokens) * g.K * es / (odd ? 17e3 : es == 2 ? 42e3 : 38e3);
        if (t < *us) {
            *us = t;
            best = rt;
        }
    }
    return best;
}

DenseFew plan_few(const DenseGemm &g, int cus, double *us)
{
    DenseFew f;
    f.rows = few_rows(g, cus, us);
    const int groups = (g.M + f.rows - 1) / f.rows;
    f.groups = groups > 2 ? 4 : groups;
    const int step = 16 / (int)dense_esize(g.dtype) * 64 / f.rows, steps = (g.K + step - 1) / step;
    f.waves = steps >= 2 * kFewWaves ? kFewWaves : steps >= 4 ? 4 : 1;
    return f;
}

}  // namespace

size_t dense_partials(const DenseGemm &g, int splits) { return (size_t)partial_bytes(g, splits); }

DenseTile dense_tile(int dtype, bool dma, int tile)
{
    const TileCost &t = tiles_of(dtype, dma)[tile];
    return DenseTile{t.bm, t.bn};
}

bool few_needs_no_room(int64_t T, int64_t in) { return T <= kAlwaysFew && T * in < kAlwaysFewX; }

DenseChoice choose_gemm(const DenseGemm &g, int cus, size_t room)
{
    DenseChoice c{};
    const bool few = !g.a_t && !g.b_t && g.M <= kFewTokens;
    double few_us = 1e300, us;
    if (few)
        c.few = plan_few(g, cus, &few_us);
    const bool always = few && few_needs_no_room(g.M, g.K);
    if ((always && !odd_rows(g)) || (few && short_rows(g))) {
        c.kind = DenseChoice::kFew;
    } else if (short_rows(g)) {
        c.kind = DenseChoice::kShort;
    } else {
        c.tiles = plan_gemm(g, cus, room, &us);
        // Rows at odd elements: 16 x 2048 to 65536 200 us streamed, 76 in tiles; 8 x 8192
        // to 16384 199 and 105; 2 x 128 to 256 2.5 and 4.2.  (Calls of few tokens have no
        // room to split K, and their tiles wait for loads that the estimate takes for
        // hidden: 16 x 4096 to 8192, estimated at 32 us, takes 54, streamed 52.  Over 34
        // sizes the factor costs at most 1.2 us against streaming.)
        c.kind = few_us <= us * (always ? 1.5 : 1.0) ? DenseChoice::kFew : DenseChoice::kTiles;
    }
    return c;
}

bool choose_pair(const DenseGemm &gx, const DenseGemm &gw, int cus, size_t room, DensePair *out)
{
    if (short_rows(gx) || short_rows(gw))
        return false;
    double ux, uw, both;
    plan_gemm(gx, cus, room, &ux);
    plan_gemm(gw, cus, room, &uw);
    *out = plan_pair(gx, gw, cus, room, &both);
    return both < ux + uw + kLaunchUs;
}

size_t dense_gemm_ws(int64_t M, int64_t N, int64_t K, int ksegs, int planes)
{
    const int64_t kt = (K + 63) / 64 * ksegs;
    int most = 1;
    for (const int s : kSplits)
        if (kt / s >= kSplitTiles)
            most = s;
    if (most == 1)
        return 0;
    const size_t all = (size_t)most * planes * M * ((N + 7) / 8 * 8) * 4;
    return (std::min(all, kDensePartialBytes) + 255) & ~(size_t)255;
}

}  // namespace ecf
