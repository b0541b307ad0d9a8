// group_norm_cuts.cpp -- test harness: how the group norm's calls are cut up (group_norm_cut.cpp), for the
// host alone.
#include <cmath>
#include <cstdio>
#include <random>

#include "group_norm_cut.h"

using namespace adamw;

namespace {

constexpr uintptr_t kBase = 1 << 16;

// Tensors of the call: `shift` elements off the grid, `pad` elements behind a position's channels, samples
// inside positions with `swap`.
GroupNormArgs call(int64_t samples, int64_t positions, int channels, int groups, int size, bool backward, int shift, int pad, bool swap) {
  GroupNormArgs a{};
  a.samples = samples;
  a.positions = positions;
  a.channels = channels;
  a.groups = groups;
  a.size = size;
  const int64_t row = channels + pad;
  const void* at = reinterpret_cast<const void*>(kBase + static_cast<uintptr_t>(shift * size));
  a.x = at;
  a.dy = backward ? at : nullptr;
  a.out = const_cast<void*>(at);
  a.x_sample = a.dy_sample = a.out_sample = swap ? row : positions * row;
  a.x_position = a.dy_position = a.out_position = swap ? samples * row : row;
  return a;
}

// What a cut must keep to: the first rule it breaks, or null.
const char* broken(const GroupNormArgs& a, const GnCut& c, int piece, int sms) {
  const GroupNormSpace s = group_norm_space(a.channels, a.groups, a.samples, sms);
  const bool backward = a.dy != nullptr;
#define RULE(x) if (!(x)) return #x
  RULE(c.tiles <= 65535);
  RULE(c.ctas >= 1);
  RULE(c.wide <= kGnThreads);
  RULE(static_cast<int64_t>(c.wide) * c.tiles >= c.pieces);
  RULE(static_cast<int64_t>(c.wide) * (c.tiles - 1) < c.pieces);
  RULE(c.at_once >= 1 && c.at_once * c.wide <= kGnThreads);
  if (backward) RULE(2 * static_cast<int64_t>(c.ctas) * a.channels <= s.columns);
  switch (gn_kind(a, c)) {
    case kGnCluster:
      RULE(c.cluster <= kGnClusterMax && c.ctas % c.cluster == 0);
      RULE(c.ctas / c.cluster <= a.samples);
      RULE(static_cast<int64_t>(c.part_rows) * c.cluster >= a.positions);
      RULE(static_cast<int64_t>(c.part_rows) * (c.cluster - 1) < a.positions);
      RULE(gn_cluster_bytes(a, c, piece) <= kGnClusterBytes);
      RULE(c.wide % c.group_pieces == 0 && c.wide / c.group_pieces <= kGnTileGroups);
      RULE(static_cast<int64_t>(c.wide) * piece * a.size % c.unit == 0 && static_cast<int64_t>(a.channels) * a.size % c.unit == 0);
      break;
    case kGnFused: {
      const int64_t pitch = a.groups + (c.aligned ? 0 : c.tiles);
      RULE(c.ctas == c.batch * c.parts);
      RULE(static_cast<int64_t>(kGnKept) * c.batch * c.parts * pitch * 2 <= s.stats);
      RULE(static_cast<int64_t>(kGnWords) * c.batch * (c.aligned ? c.tiles : 1) <= s.words);
      RULE(static_cast<int64_t>(c.ctas) * c.tiles <= kGnCtasPerSm * sms);       // all resident
      RULE(static_cast<int64_t>(c.parts) * c.part_rows >= a.positions);
      RULE(static_cast<int64_t>(c.parts - 1) * c.part_rows < a.positions);
      RULE(!c.aligned || c.wide % c.group_pieces == 0);
      break;
    }
    default:
      RULE(c.team_rows * c.teams <= c.at_once);
      RULE(static_cast<int64_t>(c.team_rows) * (backward ? kSmallBackward : kSmallForward) >= a.positions);
      RULE(c.wide % c.group_pieces == 0);
  }
#undef RULE
  return nullptr;
}

}  // namespace

extern "C" {

struct Cut {
  int32_t kind, piece, tiles, wide, cluster, part_rows, parts, batch, aligned, ctas;
};
Cut group_norm_cut(int64_t samples, int64_t positions, int channels, int groups, int size, int backward, int shift, int pad, int swap) {
  const GroupNormArgs a = call(samples, positions, channels, groups, size, backward != 0, shift, pad, swap != 0);
  const int piece = gn_piece(a, size);
  const GnCut c = gn_cut(a, piece, 152);
  return {gn_kind(a, c), piece, c.tiles, c.wide, c.cluster, c.part_rows, c.parts, c.batch, c.aligned, c.ctas};
}

// The model's time in ns of the cluster kernels with m groups a tile and `cluster` CTAs a sample (0: does not fit).
double group_norm_cluster_ns(int64_t samples, int64_t positions, int channels, int groups, int size, int backward, int m, int cluster) {
  const GroupNormArgs a = call(samples, positions, channels, groups, size, backward != 0, 0, 0, false);
  GnCut c{};
  const int piece = gn_piece(a, size);
  c.group_pieces = channels / groups / piece;
  return gn_cluster_time(a, piece, 152, m, cluster, &c);
}

// And of the kernels for parts of samples, in batches of `batch`.
double group_norm_parts_ns(int64_t samples, int64_t positions, int channels, int groups, int size, int backward, int batch) {
  const GroupNormArgs a = call(samples, positions, channels, groups, size, backward != 0, 0, 0, false);
  GnCut c{};
  c.batch = batch;
  return gn_parts_time(a, gn_piece(a, size), c);
}

// Cuts `n` random calls; returns how many broke a rule, and says which in `why`; `kinds` counts the kernels.
int64_t group_norm_check(uint64_t seed, int64_t n, int64_t* kinds, char* why, int length) {
  std::mt19937_64 g(seed);
  const auto spread = [&](double lo, double hi) {       // over the logarithm, without the library's own distributions
    return static_cast<int64_t>(std::exp(std::log(lo) + (std::log(hi) - std::log(lo)) * static_cast<double>(g() >> 11) / 9007199254740992.0));
  };
  int64_t bad = 0;
  for (int64_t i = 0; i < n; ++i) {
    const int sms = i % 11 == 0 ? 132 : 152;
    const int64_t groups = spread(1, 65537);
    const int64_t per = i % 3 == 0 ? int64_t{1} << (g() % 10) : spread(1, 65537.0 / static_cast<double>(groups) + 1);
    if (groups * per > kMaxChannels) continue;
    const int64_t samples = spread(1, i % 5 == 0 ? 1e6 : 2000), positions = spread(1, i % 7 == 0 ? 2147483647.0 : 1e5);
    const int size = g() % 2 != 0 ? 2 : 4;
    const bool backward = g() % 2 != 0;
    for (int piece : {16 / size, 4 / size, 1}) {
      if (per % piece != 0) continue;
      const GroupNormArgs a = call(samples, positions, static_cast<int>(groups * per), static_cast<int>(groups), size, backward, 0, 0, false);
      const GnCut c = gn_cut(a, piece, sms);
      ++kinds[gn_kind(a, c)];
      const char* rule = broken(a, c, piece, sms);
      if (rule != nullptr && bad++ == 0)
        std::snprintf(why, static_cast<size_t>(length), "%s: %lld x %lld x %lld in %lld groups of %d bytes, backward %d, pieces of %d, %d SMs", rule,
                      (long long)samples, (long long)positions, (long long)(groups * per), (long long)groups, size, backward, piece, sms);
    }
  }
  return bad;
}

}  // extern "C"
