// group_norm_cut.cpp -- how calls of the group norm are cut up.  Host code only.
#include "group_norm_cut.h"

namespace adamw {
namespace {

constexpr int kGnTiles = 65535;          // of a grid's second axis

bool on_grid(const void* p, int64_t sample, int64_t position, const GroupNormArgs& a, int size, int bytes) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (a.samples < 2 || sample * size % bytes == 0) &&
                          (a.positions < 2 || position * size % bytes == 0));
}
int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Tiles of whole groups for the small kernels: as few as may be, but up to three more where
// narrower ones leave fewer of the 256 threads without a piece (160 pieces: two tiles of 80,
// three rows at once).  False where a group fits none.
bool cut_whole(GnCut* c) {
  const int q = c->group_pieces;
  if (q > kGnThreads) return false;
  const int64_t least = up(c->pieces, kGnThreads / q * q);
  double best = 0.0;
  for (int64_t t = least; t < least + 4 && t <= c->pieces / q; ++t) {
    const int64_t wide = up(up(c->pieces, t), q) * q;
    if (wide > kGnThreads) continue;
    const int64_t tiles = up(c->pieces, wide);
    const double use = static_cast<double>(c->pieces) / static_cast<double>(tiles * kGnThreads) * static_cast<double>(kGnThreads / wide);
    if (use > 1.05 * best) {
      best = use;
      c->wide = static_cast<int32_t>(wide);
      c->tiles = static_cast<int32_t>(tiles);
    }
  }
  c->at_once = kGnThreads / c->wide;
  return best > 0.0;
}

// Tiles of the fused kernels, narrow ones of whole groups: at least 256 bytes of a row, and
// of those the one that leaves the fewest threads and CTAs without work.  At most `most`
// tiles; where no such tile will do, any 256 pieces.
void cut_narrow(GnCut* c, int piece_bytes, int64_t most, int ctas) {
  const int q = c->group_pieces;
  if (most > ctas) most = ctas;
  double best = 0.0;
  for (int wide = q; wide <= kGnThreads; wide += q) {
    const int64_t tiles = up(c->pieces, wide);
    if (tiles > most || (wide * piece_bytes < 256 && tiles > 1)) continue;
    const double use = static_cast<double>(c->pieces) / static_cast<double>(tiles * kGnThreads) * (kGnThreads / wide) *
                       static_cast<double>(ctas / tiles * tiles) / ctas;
    if (use > 1.03 * best) {
      best = use;
      c->wide = wide;
      c->tiles = static_cast<int32_t>(tiles);
    }
    if (tiles == 1) break;
  }
  c->aligned = best > 0.0;
  if (!c->aligned) {
    c->wide = c->pieces < kGnThreads ? c->pieces : kGnThreads;
    c->tiles = static_cast<int32_t>(up(c->pieces, c->wide));
  }
  c->at_once = kGnThreads / c->wide;
}

// Tiles and clusters of the cluster kernels: of all that fit, the one that the model likes best.
// False where nothing fits, or takes more than `limit` ns.
bool cut_cluster(GnCut* c, const GroupNormArgs& a, int piece, int sms, double limit) {
  const int groups = a.groups;
  GnCut best = *c, k = *c;
  double least = 0.0;
  for (int m = 1; m <= kGnTileGroups && m * c->group_pieces <= kGnThreads; m = 2 * m < groups ? 2 * m : groups) {
    for (int cluster = 1; cluster <= kGnClusterMax; cluster *= 2) {
      const double time = gn_cluster_time(a, piece, sms, m, cluster, &k);
      if (time > 0.0 && (least == 0.0 || time < least)) {
        least = time;
        best = k;
      }
    }
    if (m == groups) break;
  }
  if (least == 0.0 || least > limit) return false;
  *c = best;
  return true;
}

// Bytes that an item of the fused kernels reads, if there is enough for every CTA: 16 x 4096 x
// 1024 bf16 forward 159 us with 48 KB, 73 with 96, 66 with 160, 70 with 192 (backward 130, 130,
// 113, 122): short items leave the waits bare, long ones lose the L2.
constexpr int64_t kItemBytes = 160 << 10;

}  // namespace

int gn_piece(const GroupNormArgs& a, int size) {
  const int per = a.channels / a.groups;
  for (int bytes = 16; bytes > size; bytes = bytes == 16 ? 4 : 0) {
    const int n = bytes / size;
    if (per % n == 0 && on_grid(a.x, a.x_sample, a.x_position, a, size, bytes) &&
        on_grid(a.dy, a.dy_sample, a.dy_position, a, size, bytes) &&
        on_grid(a.out, a.out_sample, a.out_position, a, size, bytes))
      return n;
  }
  return 1;
}

// A sample takes 3 us, 0.4 more for each CTA of a cluster, and the larger of its copies
// (5.5 bytes/ns in all) and its instructions (8 (8 N + 60) per warp, row and tensor for pieces
// of N), and half the smaller one.  Off by a factor of 1.29 over the 251 choices that were measured
// (tests/golden/group_norm_cuts.json); the choices taken by it take at most 1.26 times the best one's
// time (pieces of one 16-bit element backward: 1.44).
double gn_cluster_time(const GroupNormArgs& a, int piece, int sms, int m, int cluster, GnCut* c) {
  const int tensors = a.dy != nullptr ? 2 : 1, wide = m * c->group_pieces;
  const int64_t tiles = up(a.groups, m), tile_bytes = static_cast<int64_t>(wide) * piece * a.size;
  const int64_t rows = up(a.positions, cluster), bytes = rows * tile_bytes * tensors;
  if (wide > kGnThreads || tiles > kGnTiles || bytes > kGnClusterBytes || (cluster > 1 && rows * (cluster - 1) >= a.positions)) return 0.0;
  const int at_once = kGnThreads / wide;
  int64_t per_sm = (224 << 10) / (bytes + (12 << 10));
  if (per_sm > 3) per_sm = 3;
  const double slots = static_cast<double>(per_sm * sms);
  int64_t clusters = per_sm * sms / cluster / tiles;
  if (clusters < 1) clusters = 1;
  if (clusters > a.samples) clusters = a.samples;
  const double busy = static_cast<double>(clusters * cluster * tiles), waves = busy > slots ? busy / slots : 1.0;
  const double ctas = busy < slots ? busy : slots, on_sm = ctas > sms ? ctas / sms : 1.0;
  const double compute = static_cast<double>(up(rows, at_once) * 8 * (8 * piece + 60) * tensors) * on_sm / 7.6;
  const double copies = static_cast<double>(bytes) * (1.0 + 1.0 / tensors) * ctas / 5500.0;
  c->wide = wide;
  c->tiles = static_cast<int32_t>(tiles);
  c->at_once = at_once;
  c->cluster = cluster;
  c->part_rows = static_cast<int32_t>(rows);
  c->ctas = static_cast<int32_t>(clusters * cluster);
  return static_cast<double>(up(a.samples, clusters)) * waves *
         (3000.0 + (cluster > 1 ? 400.0 * cluster : 0.0) + (compute > copies ? compute + 0.5 * copies : copies + 0.5 * compute));
}

// 13 us a batch, or 1.7 times the floor (3 and 14 times with pieces of 4 and 2 bytes: 300 x 100 x 1000
// fp16 in 8 groups, backward, takes 384 us so and 85 by clusters), and 8 us for the first statistics
// and the last results.
double gn_parts_time(const GroupNormArgs& a, int piece, const GnCut& c) {
  const int bytes = piece * a.size;
  const double floor = static_cast<double>(a.samples) * static_cast<double>(a.positions) * a.channels * a.size * (a.dy != nullptr ? 3 : 2) / 6800.0;
  const double work = floor * (bytes == 16 ? 1.7 : (bytes == 4 ? 3.0 : 14.0)), turns = 13000.0 * static_cast<double>(up(a.samples, c.batch));
  return 8000.0 + (work > turns ? work : turns);
}

GnCut gn_cut(const GroupNormArgs& a, int piece, int sms) {
  const int most = a.dy != nullptr ? kSmallBackward : kSmallForward;
  GnCut c{};
  c.per = a.channels / a.groups;
  c.pieces = a.channels / piece;
  c.group_pieces = c.per / piece;
  const bool lanes = c.group_pieces <= 32 && (c.group_pieces & (c.group_pieces - 1)) == 0;
  if (cut_whole(&c) && a.positions <= static_cast<int64_t>(most) * c.at_once) {
    // with samples enough for every CTA's threads, as few threads a sample as hold it;
    // else as many as it has work for
    const int64_t resident = static_cast<int64_t>(a.dy != nullptr ? 3 : kSmallCtasPerSm) * sms;
    const bool many = a.samples * c.tiles >= resident * c.at_once;
    const int64_t rows = many ? up(a.positions, most) : (a.positions < c.at_once ? a.positions : c.at_once);
    c.by_lanes = lanes;
    c.team_rows = static_cast<int32_t>(rows);
    c.teams = c.at_once / c.team_rows;
    int64_t ctas = up(a.samples, c.teams), all = resident / c.tiles;
    if (all < 1) all = 1;
    c.ctas = static_cast<int32_t>(ctas < all ? ctas : all);
    return c;
  }
  const int64_t samples = a.samples > 0 ? a.samples : 1;
  const int resident = kGnCtasPerSm * sms;
  cut_narrow(&c, piece * a.size, resident, resident);
  c.by_lanes = c.aligned && lanes;
  // the batch whose parts come closest to an item's bytes, one part for each of a tile's CTAs
  const int64_t ctas = resident / c.tiles > 0 ? resident / c.tiles : 1;
  const int64_t row_bytes = static_cast<int64_t>(c.wide) * piece * a.size * (a.dy != nullptr ? 2 : 1);
  const int64_t rows = kItemBytes / row_bytes > c.at_once ? kItemBytes / row_bytes : c.at_once;
  int64_t batch = ctas / up(a.positions, rows);
  if (batch < 1) batch = 1;
  batch = up(samples, up(samples, batch));        // as many in the last one, or nearly
  int64_t parts = ctas / batch;
  const int64_t most_parts = up(a.positions, c.at_once);
  if (parts > most_parts) parts = most_parts;
  c.part_rows = static_cast<int32_t>(up(a.positions, parts));
  c.parts = static_cast<int32_t>(up(a.positions, c.part_rows));
  c.batch = static_cast<int32_t>(batch);
  c.ctas = c.batch * c.parts;
  GnCut k = c;
  if (a.samples > 0 && cut_cluster(&k, a, piece, sms, gn_parts_time(a, piece, c))) {
    k.by_lanes = lanes;
    const int64_t step = static_cast<int64_t>(k.wide) * piece * a.size;     // bytes from tile to tile
    k.unit = a.size;
    for (int unit : {16, 4}) {
      if (unit > a.size && step % unit == 0 && static_cast<int64_t>(a.channels) * a.size % unit == 0 &&
          on_grid(a.x, a.x_sample, a.x_position, a, a.size, unit) && on_grid(a.dy, a.dy_sample, a.dy_position, a, a.size, unit)) {
        k.unit = unit;
        break;
      }
    }
    return k;
  }
  return c;
}

GnKind gn_kind(const GroupNormArgs& a, const GnCut& c) {
  if (c.cluster > 0) return kGnCluster;
  if (c.team_rows == 0) return kGnFused;
  if (a.positions == 1 && c.by_lanes && c.teams == c.at_once) return kGnLanes;
  return a.positions <= c.team_rows ? kGnRow : kGnSmall;
}

int gn_cluster_bytes(const GroupNormArgs& a, const GnCut& c, int piece) {
  const int bytes = c.part_rows * c.wide * piece * a.size * (a.dy != nullptr ? 2 : 1);
  // the threads' column sums take the elements' place at the end
  const int columns = a.dy != nullptr ? 2 * ((piece + 1) / 2) * kGnThreads * static_cast<int>(sizeof(float2)) : 0;
  return bytes > columns ? bytes : columns;
}

GroupNormSpace group_norm_space(int32_t channels, int32_t groups, int64_t max_samples, int sms) {
  GroupNormSpace n{};
  const int64_t resident = static_cast<int64_t>(kGnCtasPerSm) * sms;
  n.joined = max_samples * groups * 2;
  n.words = kGnWords * resident;
  // of the CTAs of a tile, the most where tiles are widest: fused ones leave statistics, all
  // leave a row of column sums
  const int64_t rows = (kSmallCtasPerSm > kGnCtasPerSm ? kSmallCtasPerSm : kGnCtasPerSm) * static_cast<int64_t>(sms);
  for (int piece : {1, 2, 4, 8}) {
    if (channels / groups % piece != 0) continue;
    const int64_t tiles = up(channels / piece, kGnThreads);
    const int64_t parts = resident / tiles > 1 ? resident / tiles : 1;
    const int64_t stats = kGnKept * parts * (groups + tiles) * 2;
    const int64_t ctas = rows / tiles > kGnClusterMax ? rows / tiles : kGnClusterMax;
    if (stats > n.stats) n.stats = stats;
    if (2 * ctas * channels > n.columns) n.columns = 2 * ctas * channels;
  }
  return n;
}

}  // namespace adamw
