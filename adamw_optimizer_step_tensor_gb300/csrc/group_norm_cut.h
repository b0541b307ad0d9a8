// group_norm_cut.h -- how a call of the group norm is cut up, and which of its kernels takes it.
// Host code and constants that the kernels share; no kernels.
#pragma once

#include <cstdint>

#include "block_ops.h"

namespace adamw {

// How a call is cut up.
struct GnCut {
  int32_t pieces, wide, tiles;   // of a row; of a tile; tiles of a row
  int32_t at_once;               // rows a CTA takes at once
  int32_t per;                   // channels of a group
  int32_t group_pieces;          // pieces of a group
  int32_t by_lanes;              // a group's pieces are a power of two of neighbouring lanes
  // small kernels
  int32_t team_rows;             // rows of threads per sample
  int32_t teams;                 // samples a CTA takes at once
  // cluster kernels
  int32_t cluster;               // CTAs that share a sample's tile; 0: other kernels
  int32_t unit;                  // bytes of a copy
  // fused kernels
  int32_t aligned;               // tiles are of whole groups: each of a sample's is open by itself
  int32_t parts;                 // of a sample
  int32_t batch;                 // samples of a batch
  int32_t part_rows;
  int32_t ctas;                  // per tile; fused kernels: batch x parts
};

constexpr int kGnThreads = 256;
constexpr int kGnCtasPerSm = 2;          // of the fused kernels
constexpr int kSmallForward = 8;         // pieces a thread of the small kernel holds
constexpr int kSmallBackward = 4;        // of x and of dy
constexpr int kSmallCtasPerSm = 4;       // of the small kernels forward, on which their grid goes; backward 3
constexpr int kGnTileGroups = 64;        // groups of a cluster kernel's tile, at most
constexpr int kGnClusterMax = 8;
constexpr int kGnClusterBytes = 208 << 10;   // of a CTA's elements, at most

// Statistics of parts and means of samples are kept for three batches: a CTA leaves those of
// batch j + 3 after its results of batch j + 1, whose sample was opened when all parts of
// batch j had been joined.
constexpr int kGnKept = 3;
// Words of the CTAs that share a sample: one for each batch kept, and the batches that are open.
constexpr int kGnWords = kGnKept + 1;

// The widest piece of the call, in elements of `size` bytes.
int gn_piece(const GroupNormArgs& a, int size);
// Cuts a call up (a.dy: the backward pass) in pieces of `piece` elements.
GnCut gn_cut(const GroupNormArgs& a, int piece, int sms);
// The model's time, in ns, of the cluster kernels with `m` groups a tile and `cluster` CTAs a sample,
// and their cut (c: with its group_pieces); 0 where they do not fit.
double gn_cluster_time(const GroupNormArgs& a, int piece, int sms, int m, int cluster, GnCut* c);
// And of the kernels that cut samples into parts, in batches of c.batch.
double gn_parts_time(const GroupNormArgs& a, int piece, const GnCut& c);
// What takes a call: lone positions on neighbouring lanes; samples in a CTA's registers, one piece
// a thread or several; samples in the shared memory of a cluster; parts of samples, read twice.
enum GnKind { kGnLanes, kGnRow, kGnSmall, kGnCluster, kGnFused };
GnKind gn_kind(const GroupNormArgs& a, const GnCut& c);
// Shared memory of a CTA of the cluster kernels, for its elements.
int gn_cluster_bytes(const GroupNormArgs& a, const GnCut& c, int piece);

}  // namespace adamw
