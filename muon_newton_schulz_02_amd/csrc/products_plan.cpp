// Which kernel and which tiles a product runs on, and how its sum is cut: host code, which
// every product's launch and workspace go by.
#include <algorithm>
#include <cmath>

#include "products_internal.h"

namespace muon {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The fastest plan by a model of the time, in us: full rounds of tiles over the GPU and a
// last one that fills a part of it, a stage of k (64 of bfloat16, 32 of binary32) measured
// for each shape with every workgroup busy (`stage`) and with a quarter of them
// (`alone`), a tile's start and end, and the partial sums' way to memory and back at 5 TB/s.
struct Kind {
  int shape, bm, bn, per_cu;
  double stage, alone, ends;
};
// The narrow shape, for few columns: TN dl^T x of 2341 x 15034 and 25 33 us (52 without it), 2868
// x 18624 and 97 43 (54), 8192 x 32768 and 64 107 (161); NN and NT, where it is taken up to its 64
// columns (beyond them it lost up to a tenth): 16384 rows of eight groups, 4096 to 64 37 (44), 3394
// rows of three, 4291 to 45 25 (32).
constexpr Kind KINDS[] = {{SHAPE_LARGE, 256, 256, 1, 1.80, 1.10, 9.0},
                          {SHAPE_MEDIUM, 128, 128, 2, 1.10, 0.54, 7.0},
                          {SHAPE_SMALL, 32, 128, 3, 0.88, 0.43, 5.0},
                          {SHAPE_NARROW, 128, 64, 2, 0.63, 0.40, 5.0}};
constexpr Kind KINDS_TN[] = {{SHAPE_LARGE, 256, 256, 1, 1.72, 1.15, 11.0},
                             {SHAPE_MEDIUM, 128, 256, 1, 0.98, 0.72, 8.0},
                             {SHAPE_NARROW, 128, 64, 2, 0.63, 0.40, 5.0}};
constexpr Kind KINDS_F32[] = {{SHAPE_LARGE, 256, 128, 1, 2.58, 2.05, 7.0},
                              {SHAPE_MEDIUM, 128, 128, 1, 1.42, 1.10, 5.0},
                              {SHAPE_SMALL, 32, 128, 2, 1.10, 0.70, 5.0}};
constexpr Kind KINDS_F32_TN[] = {{SHAPE_LARGE, 256, 128, 1, 2.62, 2.10, 8.0}, {SHAPE_MEDIUM, 128, 128, 1, 1.45, 1.15, 6.0}};

// `tiles` tiles of `stages` stages each.
double tiles_us(const Kind& s, double tiles, double stages, int cus) {
  const double slots = double(cus) * s.per_cu, rounds = std::floor(tiles / slots), rest = tiles / slots - rounds;
  double us = rounds * (stages * s.stage + s.ends);
  if (rest > 0) us += stages * (s.alone + (s.stage - s.alone) * std::max(0.0, (rest - 0.25) / 0.75)) + s.ends;
  return us;
}

// Few rows, where Q's way from memory is most of a product: the stream (product_stream.hip)
// or tiles that are not cut.  Up to 16 rows a group on average, the stream where it is
// faster by this: the turns of its workgroups (1024 at a time), Q from memory, and from the
// caches x once for every 32 columns and Q again for every further 16 rows of a group; tiles
// take 8 us and Q from memory at least.  Measured, stream and tiles, us, the rows spread
// evenly / at random / all to one expert:
//   bfloat16  64 experts, 1536 to 2048, a row each       86 /  43 /  17     73 /  42 /  12
//                                       16 rows         110 / 133 /  89     77 /  86 /  19
//             8 experts, 1536 to 6144,  a row each       29 /  21 /   9     32 /  24 /  21
//                                       4 rows           30 /  30 /  13     25 /  25 /  12
//             32 experts, 768 to 256,   8 rows            8 /  10 /   8     12 /  17 /  39
//             32 experts, 6144 to 1536, 3 rows           90                112
//             one, 1536 to 6144,        1 to 16 rows      7 to 8            13
//   binary32  64 experts, 1536 to 2048, a row each      170 /  95 /  22    177 / 119 /  36
//                                       16 rows         208 / 236 / 151    176 / 191 /  64
//             8 experts, 1536 to 6144,  8 rows           64 /  60 /  32     69 /  64 /  40
//             32 experts, 768 to 256,   16 rows          11 /  16 /  10     18 /  26 /  47
// With more than 16 rows tiles are faster (64 experts, bfloat16, 24 rows 78 and 167).
constexpr int64_t STREAM_ROWS = 16;
struct StreamRates {
  double turn, once, again, tiles;     // us, and bytes a us
};
constexpr StreamRates STREAM_BF16 = {6.5, 7.2e6, 7.2e6, 6.0e6}, STREAM_F32 = {8.5, 6.4e6, 11.0e6, 4.8e6};
bool stream_rows(const ProductArgs& a, double tiles_us) {
  const StreamRates& s = a.f32 ? STREAM_F32 : STREAM_BF16;
  const double rows = a.rows, used = std::min(rows, double(std::max(1, a.groups)));
  const double units = std::max(used, rows / 16 + used / 2), nt = double(ceil_div(a.n, STREAM_TILE_N));
  const double row = double(a.k) * (a.f32 ? 4 : 2), once = used * a.n * row;
  const double again = (units - used) * a.n * row + nt * rows * row;
  return std::max(5.0, s.turn * units * nt / 1024) + once / s.once + again / s.again < std::max(tiles_us, 8.0 + once / s.tiles);
}

}  // namespace

ProductPlan product_plan(int form, int epi, const ProductArgs& a, int cus) {
  const int64_t esz = a.f32 ? 4 : 2, ke = 128 / esz;
  // 16-byte loads (product_tile.h)
  if (a.p_elems * esz < 16 || a.q_elems * esz < 16 || (form == FORM_TN && a.ld_p * esz < 16) ||
      (form != FORM_NT && a.ld_q * esz < 16))
    return {SHAPE_NAIVE, 0, 0, 0};
  // (a launch takes fewer than 2^32 threads)
  const bool few = form == FORM_NT && epi != EPI_DZ && a.k % (16 / esz) == 0 && a.rows <= STREAM_ROWS * std::max(1, a.groups) &&
                   (epi != EPI_STORE || (!a.add && !a.map && a.out_f32 == a.f32)) &&
                   ceil_div(a.n, STREAM_TILE_N) * (a.rows / 16 + std::min(a.groups, a.rows)) <= (1 << 22);
  const bool tn = form == FORM_TN;
  const Kind* kinds = a.f32 ? (tn ? KINDS_F32_TN : KINDS_F32) : (tn ? KINDS_TN : KINDS);
  const int nkinds = a.f32 ? (tn ? 2 : 3) : tn ? 3 : epi == EPI_STORE ? 4 : 3;
  const int64_t groups = std::max(1, a.groups);
  const size_t queue = (size_t(QUEUE_PRE) + 3 * size_t(groups) + 1 + 63) / 64 * 256;
  ProductPlan best = {kinds[0].shape, 1 << 30, 0, 0};
  double least = 1e30;
  auto offer = [&](int shape, int64_t chunk, size_t bytes, double us, bool queued) {
    if (bytes > (size_t(2) << 30) || us >= least) return;
    least = us;
    best = {shape, int32_t(chunk), bytes + (queued ? queue : 0), queued ? queue : 0};
  };
  for (int i = 0; i < nkinds; ++i) {
    const Kind& s = kinds[i];
    if (s.shape == SHAPE_NARROW && !tn && a.n > s.bn) continue;
    const int64_t nt = ceil_div(a.n, s.bn);
    if (!tn) {
      // tiles of rows: a group's rows fill all but half of its last one
      const int64_t mt = groups == 1 ? ceil_div(a.rows, s.bm)
                                     : std::max<int64_t>(std::min<int64_t>(groups, a.rows), a.rows / s.bm + groups / 2);
      const int64_t stages = ceil_div(a.k, ke);
      if (mt * nt > (int64_t(1) << 30)) continue;        // tiles are counted in 31 bits
      offer(s.shape, 1 << 30, 0, tiles_us(s, double(mt * nt), double(stages), cus), false);
      for (int cut = 2; cut <= 32 && epi == EPI_STORE && !few && mt * nt < 2 * cus * s.per_cu; ++cut) {
        const int64_t each = ceil_div(stages, cut);
        if (each < 4) break;
        if (ceil_div(stages, each) != cut) continue;
        const size_t bytes = size_t(cut) * size_t(a.rows) * size_t(part_ld(a.n)) * 4;
        offer(s.shape, each * ke, bytes, tiles_us(s, double(mt * nt * cut), double(each), cus) + 3.0 + 2e-6 / 5.0 * double(bytes), false);
      }
    } else {
      // Groups of very different lengths: on average a tile has `stages` stages, but one
      // group may have half of all.
      const int64_t mt = ceil_div(a.m, s.bm), all = ceil_div(a.rows, ke);
      const double tiles = double(groups * mt * nt), stages = double(std::max<int64_t>(1, all / groups));
      for (int step = 0; step < 8; ++step) {
        const int64_t chunk = step == 0 ? int64_t(1) << 30 : int64_t(32768) >> (step - 1);
        if (step > 0 && chunk >= a.rows) continue;
        const bool cut = chunk < a.rows;
        const int64_t longest = std::min(groups > 1 ? all / 2 + 1 : std::max<int64_t>(all, 1), ceil_div(chunk, ke));
        const int64_t pieces = cut ? a.rows / chunk : 0;
        const double count = tiles + double(pieces * mt * nt), each = cut || groups > 1 ? (tiles * stages) / count : stages;
        const size_t bytes = 2 * size_t(pieces) * size_t(a.m) * size_t(part_ld(a.n)) * 4;
        const double sums = cut ? 5.0 + 1e-6 / 5.0 * double(bytes) : 0.0, alone = double(longest) * s.alone + s.ends;
        // A queue keeps every workgroup busy until the last tiles, and costs a launch and
        // what an idle GPU takes to start (12 us).  Without one, groups whose lengths differ
        // leave some workgroups waiting: 15 % in the middle.  (16384 rows to 32 groups of 1536
        // x 1536, shares e^N(0, 1): 147 us without, 113 with; to eight groups of 1536 x 6144:
        // shares e^N(0, 1) 368 to 435 and 332 to 427, e^N(0, 2) 388 to 427 and 315 to 340,
        // equal shares 315 and 330.)
        const double slots = double(cus) * s.per_cu;
        if (groups > 1 && count > slots)
          offer(s.shape, chunk, bytes, 12.0 + sums + std::max(count / slots * (each * s.stage + s.ends) + 0.3 * each * s.stage, alone), true);
        double us = sums + std::max(tiles_us(s, count, each, cus), alone);
        if (groups > 1 && count > slots) us *= 1.15;
        offer(s.shape, chunk, bytes, us, false);
      }
    }
  }
  if (few && stream_rows(a, least)) return {SHAPE_STREAM, 0, 0, 0};
  return best;
}

int product_epilogue(int epi, const ProductArgs& a) {
  if (epi == EPI_STORE) return a.rest ? EPI_STORE_TARGET : EPI_STORE;
  if (a.cap == 0.f) return epi;
  const bool large = !a.f32 && a.cap > FAST_CAP;
  return epi == EPI_LSE ? (large ? EPI_LSE_LARGE_CAP : EPI_LSE_CAP) : (large ? EPI_DZ_LARGE_CAP : EPI_DZ_CAP);
}

int32_t product_tile_n(int form, int epi, const ProductArgs& a, int cus) {
  switch (product_plan(form, epi, a, cus).shape) {
    case SHAPE_NAIVE: return NAIVE_TILE_N;
    case SHAPE_STREAM: return STREAM_TILE_N;
    case SHAPE_LARGE: return a.f32 ? 128 : 256;
    default: return 128;
  }
}

}  // namespace muon
