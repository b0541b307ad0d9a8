// token_loss.cu -- the token losses' row kernel, and the pairs of the
// preference loss.
//
// One cluster of C CTAs (C = 1, 2, 4, 8) works through rows of logits; each CTA
// has its share of every row pass through a ring of shared-memory slots:
//   loader (one thread)     bulk copies (TMA engine) of 16 KB pieces into free
//                           slots
//   scheduler (one warp)    walks the rows' labels and weights ahead of the
//                           others, deals live rows (and the rows that only
//                           need zeros) out to the clusters in turn, and hands
//                           each of its cluster's rows on with everything the
//                           row's arithmetic reads from memory
//   summing warps           sum the exponentials of a row's pieces
//   finisher (one warp)     joins the sums over the CTA and the cluster, and
//                           turns them into the row's outputs and slope
//   gradient warps          turn the same pieces, still in shared memory, into
//                           gradients in place
//   storer (one thread)     bulk copies of finished slots out to dlogits; a slot
//                           is free once its copy has read it
// A policy-loss row is so read once and its gradient written once.  Summing and
// gradient warps are apart so that the next row is summed while one row's sum
// is joined and differentiated; with one set of warps for both, every row paid
// the join's latency and 8192 rows of 128,256 bf16 logits took 727 us.
#include <cmath>

#include "cluster.cuh"
#include "token_rows.cuh"

namespace adamw {
namespace {

constexpr int kSlotWords = kPieceWords;
constexpr int kSlotBytes = kSlotWords * 16;
constexpr int kMaxSlots = 13;
constexpr int kWorkers = 16;                    // summing and gradient warps together
constexpr int kFirstWorker = 4;                 // after loader, scheduler, finisher, storer
constexpr int kRingThreads = (kFirstWorker + kWorkers) * 32;
constexpr int kQueue = 16;                      // rows handed on ahead
// Cluster-wide sums under way: a finisher is through with sum n only after the
// others have taken it up, and they do that after they are through with n - 1,
// so two places are enough.
constexpr int kJoins = 2;
constexpr int kStoresOut = 3;                   // copies out whose slots may be awaited later
constexpr int kMaxCluster = 8;
constexpr int kRowsPerLane = 8;                 // rows the scheduler looks at per lane and step
constexpr int kBatch = 2;                       // rows whose inputs it fetches together
constexpr int kSharePieces = 7;                 // of a row that waits for its sum, at most

// Warps of either kind; a pass with one kind gives it all of them.
__host__ __device__ constexpr int sum_warps(int pass) {
  return !sums(pass) ? 0 : (writes_gradient(pass) ? kWorkers / 2 : kWorkers);
}
__host__ __device__ constexpr int grad_warps(int pass) { return kWorkers - sum_warps(pass); }
// Workers form teams, and the teams take a row's pieces in turn.  Where nothing
// waits for a row as a whole, teams of 4 warps: a warp then waits once for 8
// words per lane instead of once for every two, and the teams' waits overlap
// (6080 rows of 50,257: 128 -> 108 us).  Where the gradient waits for the sum,
// all summing warps take every piece, so that the row's sum is there sooner
// (8192 rows of 128,256: 595 us against 683).  The slots are a multiple of the
// teams: a team meets a slot's uses one after the other, as the parity of its
// barrier needs.
__host__ __device__ constexpr int team_warps(int pass) {
  return sums(pass) && writes_gradient(pass) ? kWorkers / 2 : 4;
}
__host__ __device__ constexpr int slots(int pass) {
  return sums(pass) && writes_gradient(pass) ? kMaxSlots : kMaxSlots / (kWorkers / 4) * (kWorkers / 4);
}
static_assert(kWorkers % 8 == 0, "whole teams");

// A live row whose sum is a far row's (see token_math.cuh) becomes kRowFar for the
// gradient warps, by the finisher, or with known sums by the scheduler; the other
// roles need not see the difference.
enum RowKind { kRowLive, kRowZero, kRowStop, kRowFar };
// A row's inputs, one per scheduler lane: its elements off the 16-byte grid (the
// first ones on lanes 0.., the last ones on lanes 8..), then
enum Input {
  kInToken = 16,                          // the token's logit
  kInWeight, kInAdvantage, kInOld, kInRef,
  kInReference, kInSum, kInSlope,         // kPassGrad
  kInputs
};
struct DealtRow {
  int64_t row;
  int32_t kind;
  int32_t y;                  // the row's token
};
struct QueueRow : DealtRow {
  float in[kInputs];
};

struct RingShared {
  alignas(128) unsigned char slot[kMaxSlots][kSlotBytes];
  QueueRow queue[kQueue];
  DealtRow dealt[kBatch + 32 * kRowsPerLane];   // this cluster's next rows, scheduler only
  float2 part[kQueue][kWorkers];          // (c, s) of every summing warp
  float2 cross[kJoins][kMaxCluster];      // (c, s) of every CTA of the cluster
  struct {
    float c, f, coef, pad;
  } result[kQueue];                       // what the gradient warps need of a row
  uint64_t full[kMaxSlots];      // a slot's copy has landed
  uint64_t done[kMaxSlots];      // a slot's gradients are in place
  uint64_t empty[kMaxSlots];     // a slot may be filled again
  uint64_t queue_full[kQueue], queue_empty[kQueue];
  uint64_t summed[kQueue];    // a row's `part` is complete
  uint64_t joined[kJoins];    // a row's `cross` is complete
  uint64_t ready[kQueue];     // a row's `result` is there
  uint32_t gave_up;
};

// A bounded wait of a whole warp, the same answer in every lane: lanes that each timed
// their own could part at the limit, and those that went on would wait for the others
// at the next shuffle.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, mbar_wait(bar, parity));
}

// ---- scheduler

// Lane `lane`'s input of a row.
template <typename T, int PASS>
__device__ __forceinline__ float row_input(const LossArgs& a, const DealtRow& d, int lane,
                                           uint32_t rank, uint32_t ranks) {
  const T* const z = static_cast<const T*>(a.logits) + d.row * a.stride;
  const float* from = nullptr;
  if (lane <= kInToken) {
    const RowShare<T> share(z, a.vocab, rank, ranks);
    const int e = lane == kInToken ? (PASS != kPassGrad ? d.y : -1)
                                   : ragged_element(share, a.vocab, lane);
    return e >= 0 ? to_f32(z[e]) : 0.0f;
  }
  if (policy_pass(PASS)) {
    if (lane == kInWeight) from = a.weights;
    if (lane == kInAdvantage) from = a.advantages;
    if (lane == kInOld) from = a.old_logps;
    if (lane == kInRef) from = a.ref_logps;
  }
  if (PASS == kPassGrad) {
    const float2 st = a.row_stat[d.row];
    if (lane == kInReference) return st.x;
    if (lane == kInSum) return st.y;
    if (lane == kInSlope) from = a.row_coef;
  }
  return from != nullptr ? from[d.row] : 0.0f;
}

template <typename T, int PASS>
__device__ void schedule(const LossArgs& a, RingShared& sh) {
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const uint32_t me = blockIdx.x / ranks, clusters = gridDim.x / ranks;
  const int lane = threadIdx.x & 31;
  uint32_t live_turn = 0, zero_turn = 0;       // whose turn the next live / zero row is
  uint32_t sent = 0;
  int64_t base = 0;                            // rows looked at
  int held = 0, next = 0;                      // rows in sh.dealt, and the first not sent yet
  // labels and weights of the next step's rows (kRowsPerLane neighbours on each
  // lane), on their way while this step's rows are dealt
  int64_t ahead_y[kRowsPerLane];
  float ahead_w[kRowsPerLane];
  // gradients of known rows run from the last row to the first: the pass before
  // ended there, so the end of the logits is still in L2
  auto row_at = [&](int64_t i) { return PASS == kPassGrad ? a.rows - 1 - i : i; };
  auto look = [&](int64_t at) {
    const float* const weights = PASS == kPassGrad ? a.row_coef : a.weights;
#pragma unroll
    for (int u = 0; u < kRowsPerLane; ++u) {
      const int64_t i = at + lane * kRowsPerLane + u;
      ahead_y[u] = i < a.rows ? label_of(a, row_at(i)) : -1;
      ahead_w[u] = i < a.rows && weights != nullptr ? weights[row_at(i)] : 1.0f;
    }
  };
  look(0);
  for (;;) {
    if (next == held) next = held = 0;
    while (held - next < kBatch && held <= kBatch && base < a.rows) {
      int32_t y[kRowsPerLane];
      uint32_t live = 0u;                      // bit u: row u of this lane is live
#pragma unroll
      for (int u = 0; u < kRowsPerLane; ++u) {
        y[u] = static_cast<int32_t>(ahead_y[u]);
        if (ahead_w[u] != 0.0f && ahead_y[u] >= 0 && ahead_y[u] < a.vocab) live |= 1u << u;
      }
      look(base + 32 * kRowsPerLane);
      const int64_t first = base + lane * kRowsPerLane;
      const int mine_in = static_cast<int>(max(min(a.rows - first, (int64_t)kRowsPerLane), (int64_t)0));
      const uint32_t dead = ((1u << mine_in) - 1u) & ~live;
      // counts of live and dead rows before this lane's, packed in one scan
      uint32_t scan = __popc(live) | __popc(dead) << 16;
      const uint32_t own = scan;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(kFull, scan, o);
        if (lane >= o) scan += up;
      }
      const uint32_t total = __shfl_sync(kFull, scan, 31);
      uint32_t live_at = (live_turn + ((scan - own) & 0xFFFFu)) % clusters;
      uint32_t dead_at = (zero_turn + ((scan - own) >> 16)) % clusters;
      live_turn = (live_turn + (total & 0xFFFFu)) % clusters;
      zero_turn = (zero_turn + (total >> 16)) % clusters;
      uint32_t send = 0u;
#pragma unroll
      for (int u = 0; u < kRowsPerLane; ++u) {
        const bool on = (live >> u) & 1u;
        bool mine;
        if (on) {
          mine = live_at == me;
          live_at = live_at + 1 == clusters ? 0 : live_at + 1;
        } else {
          mine = ((dead >> u) & 1u) && dead_at == me;
          dead_at = dead_at + 1 == clusters ? 0 : dead_at + 1;
        }
        if (mine && (on || writes_gradient(PASS))) send |= 1u << u;
        if (mine && rank == 0) {
          const int64_t t = row_at(first + u);
          if (PASS == kPassPrefer) a.row_coef[t] = 0.0f;
          if (PASS != kPassGrad && !on) {
            a.logps[t] = 0.0f;
            if (a.lse != nullptr) a.lse[t] = 0.0f;
          }
        }
      }
      int place = __popc(send);
      const int count = place;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFull, place, o);
        if (lane >= o) place += up;
      }
      const int sends = __shfl_sync(kFull, place, 31);
      place += held - count;
#pragma unroll
      for (int u = 0; u < kRowsPerLane; ++u)
        if ((send >> u) & 1u)
          sh.dealt[place++] = {row_at(first + u), (live >> u) & 1u ? kRowLive : kRowZero, y[u]};
      held += sends;
      base += 32 * kRowsPerLane;
      __syncwarp();
    }
    const int n = min(kBatch, held - next);
    float in[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      in[i] = i < n && sh.dealt[next + i].kind == kRowLive
                  ? row_input<T, PASS>(a, sh.dealt[next + i], lane, rank, ranks)
                  : 0.0f;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i > n || (i == n && n != 0)) break;
      // with nothing left, one last row says so
      const DealtRow d = n == 0 ? DealtRow{0, kRowStop, 0} : sh.dealt[next + i];
      const uint32_t q = sent % kQueue;
      if (sent >= kQueue && !warp_wait(&sh.queue_empty[q], (sent / kQueue - 1) & 1u)) {
        atomicOr(&sh.gave_up, 1u);
        return;
      }
      if (lane < kInputs) sh.queue[q].in[lane] = in[i];
      const bool far = PASS == kPassGrad && __any_sync(kFull, lane == kInSum && in[i] < 0.0f);
      if (lane == 0) static_cast<DealtRow&>(sh.queue[q]) = {d.row, far ? kRowFar : d.kind, d.y};
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.queue_full[q]);
      ++sent;
      if (n == 0) return;
    }
    next += n;
    __syncwarp();
  }
}

// ---- loader and storer

// Waits for the next row of the queue; false if the wait gave up.
template <bool WARP = true>
__device__ __forceinline__ bool take_row(RingShared& sh, uint32_t n, uint32_t site) {
  uint64_t* const bar = &sh.queue_full[n % kQueue];
  const uint32_t parity = (n / kQueue) & 1u;
  if (WARP ? warp_wait(bar, parity) : mbar_wait(bar, parity)) return true;
  atomicOr(&sh.gave_up, site);
  return false;
}

template <typename T, int PASS>
__device__ void load_rows(const LossArgs& a, RingShared& sh) {
  constexpr int kSlots = slots(PASS);
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  uint32_t use = 0;
  bool ok = true;
  for (uint32_t n = 0; ok && take_row<false>(sh, n, 2u); ++n) {
    const int64_t row = sh.queue[n % kQueue].row;
    const int kind = sh.queue[n % kQueue].kind;
    mbar_arrive(&sh.queue_empty[n % kQueue]);
    if (kind == kRowStop) break;
    if (kind == kRowZero) continue;
    const RowShare<T> share(static_cast<const T*>(a.logits) + row * a.stride, a.vocab, rank, ranks);
    for (int j = 0; j < share.pieces; ++j, ++use) {
      const uint32_t s = use % kSlots;
      if (use >= kSlots && !mbar_wait(&sh.empty[s], (use / kSlots - 1) & 1u)) {
        atomicOr(&sh.gave_up, 2u);
        ok = false;
        break;
      }
      const uint32_t bytes = 16u * share.piece_words(j);
      mbar_expect_tx(&sh.full[s], bytes);
      bulk_g2s(sh.slot[s], share.base + static_cast<int64_t>(j) * kSlotBytes, bytes, &sh.full[s]);
    }
  }
  // the copies in flight land before the CTA may leave, whichever role it is whose
  // wait gave up (otherwise they have all been waited for by now)
  for (uint32_t u = use > kSlots ? use - kSlots : 0; u < use; ++u)
    mbar_wait(&sh.full[u % kSlots], (u / kSlots) & 1u);
}

template <typename T, int PASS>
__device__ void store_rows(const LossArgs& a, RingShared& sh, bool bulk_out) {
  constexpr int kSlots = slots(PASS);
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  uint32_t stores = 0, released = 0;
  auto release_to = [&](uint32_t upto) {
    for (; released < upto; ++released) mbar_arrive(&sh.empty[released % kSlots]);
  };
  // Waits on `bar`; where it is not ready at once, the copies still out are
  // awaited first, so that nobody waits for a slot that this thread holds back.
  auto await = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    bulk_wait_read_all();
    release_to(stores);
    if (mbar_wait(bar, parity)) return true;
    atomicOr(&sh.gave_up, 512u);
    return false;
  };
  for (uint32_t n = 0; await(&sh.queue_full[n % kQueue], (n / kQueue) & 1u); ++n) {
    const int64_t row = sh.queue[n % kQueue].row;
    const int kind = sh.queue[n % kQueue].kind;
    mbar_arrive(&sh.queue_empty[n % kQueue]);
    if (kind == kRowStop) break;
    if (kind == kRowZero) continue;
    const RowShare<T> share(static_cast<const T*>(a.logits) + row * a.stride, a.vocab, rank, ranks);
    unsigned char* const out = reinterpret_cast<unsigned char*>(static_cast<T*>(a.dlogits) +
                                                                row * a.dstride + share.first);
    bool ok = true;
    for (int j = 0; ok && j < share.pieces; ++j) {
      const uint32_t s = stores % kSlots;
      if (!(ok = await(&sh.done[s], (stores / kSlots) & 1u))) break;
      if (bulk_out) {
        bulk_s2g(out + static_cast<int64_t>(j) * kSlotBytes, sh.slot[s], 16u * share.piece_words(j));
        bulk_commit();
      }
      ++stores;
      if (stores - released > kStoresOut) {
        bulk_wait_read_but<kStoresOut>();
        release_to(stores - kStoresOut);
      }
    }
    if (!ok) break;
  }
  bulk_wait_all();
}

// ---- workers

__device__ __forceinline__ void leave_row(RingShared& sh, uint32_t n) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.queue_empty[n % kQueue]);
}

template <typename T, int PASS>
__device__ void sum_rows(const LossArgs& a, RingShared& sh, int warp) {
  constexpr int kTeam = team_warps(PASS), kTeams = sum_warps(PASS) / kTeam;
  constexpr int kThreadsHere = kTeam * 32;
  constexpr int kSlots = slots(PASS);
  constexpr int kRun = 2;                                // words summed together
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const uint32_t team = warp / kTeam;
  const int lane = threadIdx.x & 31, tid = (warp % kTeam) * 32 + lane;
  uint32_t use = 0;
  for (uint32_t n = 0; take_row(sh, n, 4u); ++n) {
    const QueueRow& q = sh.queue[n % kQueue];
    if (q.kind == kRowStop) return;
    if (q.kind == kRowLive) {
      const RowShare<T> share(static_cast<const T*>(a.logits) + q.row * a.stride, a.vocab, rank,
                              ranks);
      RowSum r{-kFar, 0.0f};
      for (int j = 0; j < share.pieces; ++j, ++use) {
        if (use % kTeams != team) continue;
        const uint32_t slot = use % kSlots;
        if (!warp_wait(&sh.full[slot], (use / kSlots) & 1u)) {
          atomicOr(&sh.gave_up, 8u);
          return;
        }
        const uint4* const w = reinterpret_cast<const uint4*>(sh.slot[slot]) + tid;
        const int words = share.piece_words(j);
        if (words == kSlotWords) {
#pragma unroll
          for (int i = 0; i < kSlotWords / kThreadsHere; i += kRun) {
            uint4 v[kRun];
#pragma unroll
            for (int m = 0; m < kRun; ++m) v[m] = w[(i + m) * kThreadsHere];
            add_words<T, kRun>(a, v, r);
          }
        } else {
          for (int i = 0; tid + i < words; i += kThreadsHere) {
            const uint4 v[1] = {w[i]};
            add_words<T, 1>(a, v, r);
          }
        }
        if (!writes_gradient(PASS)) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.empty[slot]);
        }
      }
      if (rank == 0 && warp == 0 && ragged_element(share, a.vocab, lane) >= 0) {
        const float x = q.in[lane];
        r.raise(x * a.k);
        r.s += exp2_fast(arg(a, x, r.c));
      }
      r.join_lanes();
      if (lane == 0) {
        sh.part[n % kQueue][warp] = make_float2(r.c, r.s);
        mbar_arrive(&sh.summed[n % kQueue]);
      }
    } else if (lane == 0) {
      mbar_arrive(&sh.summed[n % kQueue]);               // keeps the phases in step
    }
    leave_row(sh, n);
  }
}

// Gives the other CTAs of the cluster x; lane i gets what CTA i gave (lanes past
// the cluster keep theirs).  False if the wait gave up.
__device__ __forceinline__ bool exchange(RingShared& sh, RowSum& x, uint32_t join, uint32_t rank,
                                         uint32_t ranks) {
  const uint32_t lane = threadIdx.x & 31;
  const int b = join % kJoins;
  if (lane < ranks) {
    cluster_store2(cluster_map(&sh.cross[b][rank], lane), x.c, x.s);
    cluster_arrive(cluster_map(&sh.joined[b], lane));
  }
  if (!__all_sync(kFull, mbar_wait_cluster(&sh.joined[b], (join / kJoins) & 1u))) {
    atomicOr(&sh.gave_up, 64u);
    return false;
  }
  if (lane < ranks) x = RowSum{sh.cross[b][lane].x, sh.cross[b][lane].y};
  return true;
}

// A far row's sum (see token_math.cuh), from two more passes over the row in memory;
// 1 if a wait gave up.  Called by the finisher; far rows are rare, and a function of
// its own leaves the other rows' code alone.
template <typename T>
__device__ __noinline__ RowSum far_sums(const LossArgs& a, RingShared& sh, int64_t row, uint32_t join) {
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int lane = threadIdx.x & 31;
  const T* const z = static_cast<const T*>(a.logits) + row * a.stride;
  RowSum r{lanes_max(far_max<T>(z, a.vocab, rank, ranks, lane, 32)), 0.0f};
  if (ranks > 1) {
    if (!exchange(sh, r, join, rank, ranks)) return RowSum{0.0f, 1.0f};
    r.c = lanes_max(lane < static_cast<int>(ranks) ? r.c : -INFINITY);
  }
  const float top = r.c;
  r.s = lanes_sum(far_sum<T>(z, a.vocab, rank, ranks, lane, 32, top, a.k, a.k_lo));
  if (ranks > 1) {
    if (!exchange(sh, r, join + 1, rank, ranks)) return RowSum{0.0f, 1.0f};
    r.s = lanes_sum(lane < static_cast<int>(ranks) ? r.s : 0.0f);
  }
  return RowSum{top, -r.s};
}

template <typename T, int PASS>
__device__ void finish_rows(const LossArgs& a, RingShared& sh, double (&acc)[4]) {
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int lane = threadIdx.x & 31;
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  uint32_t joins = 0;
  for (uint32_t n = 0; take_row(sh, n, 16u); ++n) {
    const QueueRow& q = sh.queue[n % kQueue];
    const int64_t row = q.row;
    if (q.kind == kRowStop) return;
    const int e = n % kQueue;
    if (q.kind == kRowLive) {
      if (!warp_wait(&sh.summed[e], (n / kQueue) & 1u)) {
        atomicOr(&sh.gave_up, 32u);
        return;
      }
      RowSum r{-kFar, 0.0f};
      if (lane < sum_warps(PASS)) r = RowSum{sh.part[e][lane].x, sh.part[e][lane].y};
      r.join_lanes();
      if (ranks > 1) {
        if (!exchange(sh, r, joins++, rank, ranks)) return;
        if (lane >= static_cast<int>(ranks)) r = RowSum{-kFar, 0.0f};
        r.join_lanes();
      }
      RowLog l;
      if (r.ordinary()) {                  // the same in every CTA of the cluster
        l = row_log(a, r, q.in[kInToken]);
      } else {
        if (!r.undefined()) {
          r = far_sums<T>(a, sh, row, joins);
          if (ranks > 1) joins += 2;
          if (r.s > 0.0f) return;          // a wait gave up
        }
        if (r.far() && lane == 0) sh.queue[e].kind = kRowFar;
        l = far_row_log(a, r, q.in[kInToken]);
      }
      PolicyTerm p{0.0f, 0.0f, 0.0f, 0.0f};
      if (policy_pass(PASS))
        p = policy_term(a, {q.in[kInWeight], q.in[kInAdvantage], q.in[kInOld], q.in[kInRef]}, l.logp);
      if (lane == 0) {
        if (writes_gradient(PASS)) {
          // first of all: the gradient warps wait for it
          const float coef = p.slope * out_scale;
          sh.result[e] = {r.c, grad_factor<T>(a, r, coef), coef, 0.0f};
          mbar_arrive(&sh.ready[e]);
        }
        if (rank == 0) {
          a.logps[row] = l.logp;
          if (a.lse != nullptr) a.lse[row] = l.lse;
          if ((PASS == kPassPrefer || PASS == kPassPolicy) && a.row_stat != nullptr) {
            a.row_stat[row] = make_float2(r.c, r.s);
            if (PASS == kPassPolicy) a.row_coef[row] = p.slope;
          }
        }
      }
      if (policy_pass(PASS)) {
        acc[1] += p.policy;
        acc[2] += p.kl;
        acc[3] += p.clipped;
      }
    } else if (writes_gradient(PASS) && lane == 0) {
      mbar_arrive(&sh.ready[e]);                         // keeps the phases in step
    }
    leave_row(sh, n);
  }
}

// A far row's gradient, by the warp `warp` of the gradient warps; false if a wait
// gave up.
template <typename T, int PASS>
__device__ __forceinline__ bool far_pieces(const LossArgs& a, RingShared& sh, uint32_t n, int warp,
                                           uint32_t& use, bool bulk_out) {
  constexpr int kTeam = team_warps(PASS), kTeams = grad_warps(PASS) / kTeam;
  constexpr int kThreadsHere = kTeam * 32, kSlots = slots(PASS);
  const QueueRow& q = sh.queue[n % kQueue];
  const uint32_t team = warp / kTeam;
  const int lane = threadIdx.x & 31, tid = (warp % kTeam) * 32 + lane;
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  const float c = sums(PASS) ? sh.result[n % kQueue].c : q.in[kInReference];
  const float coef = sums(PASS) ? sh.result[n % kQueue].coef : q.in[kInSlope] * out_scale;
  const float f = sums(PASS) ? sh.result[n % kQueue].f : coef / q.in[kInSum];
  T* const dz = static_cast<T*>(a.dlogits) + q.row * a.dstride;
  const RowShare<T> share(static_cast<const T*>(a.logits) + q.row * a.stride, a.vocab, cluster_rank(),
                          cluster_size());
#pragma unroll 1
  for (int j = 0; j < share.pieces; ++j, ++use) {
    if (use % kTeams != team) continue;
    const uint32_t slot = use % kSlots;
    if (!sums(PASS) && !warp_wait(&sh.full[slot], (use / kSlots) & 1u)) {
      atomicOr(&sh.gave_up, 8u);
      return false;
    }
    uint4* const w = reinterpret_cast<uint4*>(sh.slot[slot]);
    const int64_t from = share.first + static_cast<int64_t>(j) * kSlotWords * kPerWord<T>;
    const int words = share.piece_words(j);
#pragma unroll 1
    for (int i = tid; i < words; i += kThreadsHere) {
      const int64_t first = from + i * kPerWord<T>;
      const uint4 d = far_grad_word<T>(a, w[i], c, f, coef, static_cast<int>(q.y - first));
      if (bulk_out) {
        w[i] = d;
      } else {
        const T* const el = reinterpret_cast<const T*>(&d);
        for (int m = 0; m < kPerWord<T>; ++m) dz[first + m] = el[m];
      }
    }
    if (bulk_out) fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.done[slot]);
  }
  const int el = cluster_rank() == 0 && warp == 0 ? ragged_element(share, a.vocab, lane) : -1;
  if (el >= 0) {
    const float d = f * far_power(half_below(q.in[lane], c), a.k, a.k_lo);
    dz[el] = from_f32<T>(el == q.y ? d + coef : d);
  }
  return true;
}

template <typename T, int PASS>
__device__ void grad_rows(const LossArgs& a, RingShared& sh, int warp, bool bulk_out) {
  constexpr int kTeam = team_warps(PASS), kTeams = grad_warps(PASS) / kTeam;
  constexpr int kThreadsHere = kTeam * 32;
  constexpr int kSlots = slots(PASS), kAllThreads = grad_warps(PASS) * 32;
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const uint32_t team = warp / kTeam;
  const int lane = threadIdx.x & 31, tid = (warp % kTeam) * 32 + lane;
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  uint32_t use = 0;
  for (uint32_t n = 0; take_row(sh, n, 128u); ++n) {
    const QueueRow& q = sh.queue[n % kQueue];
    if (q.kind == kRowStop) return;
    const int e = n % kQueue;
    T* const dz = static_cast<T*>(a.dlogits) + q.row * a.dstride;
    if (sums(PASS) && !warp_wait(&sh.ready[e], (n / kQueue) & 1u)) {
      atomicOr(&sh.gave_up, 256u);
      return;
    }
    if (q.kind != kRowLive) {
      if (q.kind == kRowZero) {
        const RowShare<T> share(dz, a.vocab, rank, ranks);
        uint4* const out = reinterpret_cast<uint4*>(const_cast<unsigned char*>(share.base));
        for (int i = warp * 32 + lane; i < share.words; i += kAllThreads)
          out[i] = make_uint4(0, 0, 0, 0);
        const int el = rank == 0 && warp == 0 ? ragged_element(share, a.vocab, lane) : -1;
        if (el >= 0) dz[el] = from_f32<T>(0.0f);
      } else {
        if (!far_pieces<T, PASS>(a, sh, n, warp, use, bulk_out)) return;
      }
      leave_row(sh, n);
      continue;
    }
    const RowShare<T> share(static_cast<const T*>(a.logits) + q.row * a.stride, a.vocab, rank,
                            ranks);
    float c, f, coef;
    if (sums(PASS)) {
      c = sh.result[e].c;
      f = sh.result[e].f;
      coef = sh.result[e].coef;
    } else {
      c = q.in[kInReference];
      coef = q.in[kInSlope] * out_scale;
      f = grad_factor<T>(a, RowSum{c, q.in[kInSum]}, coef);
    }
    // the token's place relative to this thread's first word
    const int64_t from = share.first + tid * kPerWord<T>;
    const int at = static_cast<int>(q.y - from);            // vocab is at most 2^30
    for (int j = 0; j < share.pieces; ++j, ++use) {
      if (use % kTeams != team) continue;
      const uint32_t slot = use % kSlots;
      if (!sums(PASS) && !warp_wait(&sh.full[slot], (use / kSlots) & 1u)) {
        atomicOr(&sh.gave_up, 8u);
        return;
      }
      uint4* const w = reinterpret_cast<uint4*>(sh.slot[slot]) + tid;
      const int words = share.piece_words(j);
      const int at_piece = at - j * (kSlotWords * kPerWord<T>);
      auto one = [&](int i) {
        const uint4 d = grad_word<T>(a, w[i], c, f, coef, at_piece - i * kPerWord<T>);
        if (bulk_out) {
          w[i] = d;
        } else {
          const T* const el = reinterpret_cast<const T*>(&d);
          T* const out = dz + from + (static_cast<int64_t>(j) * kSlotWords + i) * kPerWord<T>;
#pragma unroll
          for (int m = 0; m < kPerWord<T>; ++m) out[m] = el[m];
        }
      };
      if (words == kSlotWords) {
#pragma unroll
        for (int i = 0; i < kSlotWords / kThreadsHere; ++i) one(i * kThreadsHere);
      } else {
        for (int i = 0; tid + i < words; i += kThreadsHere) one(i);
      }
      if (bulk_out) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.done[slot]);
    }
    const int el = rank == 0 && warp == 0 ? ragged_element(share, a.vocab, lane) : -1;
    if (el >= 0) {
      float d = exp2_fast(grad_arg<T>(a, q.in[lane], c)) * f;
      if (el == q.y) d += coef;
      dz[el] = from_f32<T>(d);
    }
    leave_row(sh, n);
  }
}

template <typename T, int PASS>
__global__ void __launch_bounds__(kRingThreads, 1) ring_kernel(const __grid_constant__ LossArgs a, const int bulk_out) {
  extern __shared__ __align__(128) unsigned char raw[];
  RingShared& sh = *reinterpret_cast<RingShared*>(raw);
  const uint32_t ranks = cluster_size();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.done[i], team_warps(PASS));
      mbar_init(&sh.empty[i], writes_gradient(PASS) ? 1 : team_warps(PASS));
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&sh.queue_full[i], 1);
      // the loader, the workers and, where there are any, finisher and storer
      mbar_init(&sh.queue_empty[i],
                1 + kWorkers + (sums(PASS) ? 1 : 0) + (writes_gradient(PASS) ? 1 : 0));
      mbar_init(&sh.summed[i], sums(PASS) ? sum_warps(PASS) : 1);
      mbar_init(&sh.ready[i], 1);
    }
    for (int i = 0; i < kJoins; ++i) mbar_init(&sh.joined[i], ranks);
    sh.gave_up = 0u;
    fence_mbar_init();
  }
  cluster_sync();
  let_next_kernel_start();
  wait_for_previous_kernel();
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const int warp = threadIdx.x >> 5;
  if (warp == 0) {
    if (threadIdx.x == 0) load_rows<T, PASS>(a, sh);
  } else if (warp == 1) {
    schedule<T, PASS>(a, sh);
  } else if (warp == 2) {
    if constexpr (sums(PASS)) finish_rows<T, PASS>(a, sh, acc);
  } else if (warp == 3) {
    if (writes_gradient(PASS) && (threadIdx.x & 31) == 0) store_rows<T, PASS>(a, sh, bulk_out != 0);
  } else if (warp - kFirstWorker < sum_warps(PASS)) {
    if constexpr (sums(PASS)) sum_rows<T, PASS>(a, sh, warp - kFirstWorker);
  } else {
    if constexpr (writes_gradient(PASS))
      grad_rows<T, PASS>(a, sh, warp - kFirstWorker - sum_warps(PASS), bulk_out != 0);
  }
  __syncwarp();
  // no CTA leaves while another may still write to its shared memory
  cluster_sync();
  if (threadIdx.x == 0 && sh.gave_up != 0u) atomicOr(a.fault, sh.gave_up);
  if (policy_pass(PASS) && cluster_rank() == 0) {
    // the sums sit in the finisher
    __shared__ double s_acc[4];
    if (threadIdx.x == 64)
      for (int i = 0; i < 4; ++i) s_acc[i] = acc[i];
    __syncthreads();
    const double mine[4] = {s_acc[0], s_acc[1], s_acc[2], s_acc[3]};
    double out[4];
    if (last_cta_sums(mine, a.partial, a.ticket, blockIdx.x / ranks, gridDim.x / ranks, out))
      write_policy_stats(a, out);
  }
}

// ---- pairs

constexpr int kPairThreads = 1024;      // half of them per sequence

// A float32 sum with its rounding errors beside it (TwoSum, Knuth): 48 bits
// without float64, which GB300 runs at 2 per SM and cycle.
struct PairSum {
  float s = 0.0f, e = 0.0f;
  __device__ __forceinline__ void add(float x, float xe = 0.0f) {
    const float t = s + x, b = t - s;
    if (isfinite(t)) e += (s - (t - b)) + (x - b) + xe;   // an infinite sum has no error
    s = t;
  }
};

// -log sigmoid(d)
__device__ __forceinline__ float minus_log_sigmoid(float d) {
  return log1pf(expf(-fabsf(d))) + fmaxf(-d, 0.0f);
}

// One CTA per pair, one half per sequence: both sequences' rewards
// beta * sum of w (logp - ref) over their rows with a weight and a token, the
// pair's loss, and d loss / d logp of those rows.
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const LossArgs a) {
  constexpr int kHalf = kPairThreads / 2;
  __shared__ float2 s_warp[kPairThreads / 32];
  __shared__ float s_sum[2];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int p = blockIdx.x, side = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = p + side * a.pairs;
  const int64_t lo = min(max(static_cast<int64_t>(a.starts[q]), (int64_t)0), a.rows);
  const int64_t hi = min(max(static_cast<int64_t>(a.starts[q + 1]), lo), a.rows);
  auto weight = [&](int64_t t) {
    const int64_t y = label_of(a, t);
    const float w = a.weights != nullptr ? a.weights[t] : 1.0f;
    return y >= 0 && y < a.vocab ? w : 0.0f;
  };
  PairSum x;
  for (int64_t t = lo + tid; t < hi; t += kHalf) {
    const float lp = a.logps[t], ref = a.ref_logps[t], w = weight(t);
    if (w != 0.0f) x.add(w * (lp - ref));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x.add(__shfl_xor_sync(kFull, x.s, o), __shfl_xor_sync(kFull, x.e, o));
  if (lane == 0) s_warp[warp] = make_float2(x.s, x.e);
  __syncthreads();
  if (tid < 32) {
    x = PairSum{};
    if (lane < kHalf / 32) x = PairSum{s_warp[warp + lane].x, s_warp[warp + lane].y};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      x.add(__shfl_xor_sync(kFull, x.s, o), __shfl_xor_sync(kFull, x.e, o));
    if (lane == 0) s_sum[side] = a.beta * x.s + a.beta * x.e;
  }
  __syncthreads();
  const float chosen = s_sum[0], rejected = s_sum[1], d = chosen - rejected, e = a.smoothing;
  // d loss / d d = e - sigmoid(-d), over the pairs' mean
  const float z = expf(-fabsf(d));
  const float sig = d >= 0.0f ? z / (1.0f + z) : 1.0f / (1.0f + z);
  const float slope = (e - sig) * a.beta / static_cast<float>(a.pairs);
  if (tid == 0) a.rewards[q] = s_sum[side];
  for (int64_t t = lo + tid; t < hi; t += kHalf) {
    const float w = weight(t);
    if (w != 0.0f) a.row_coef[t] = w * (side == 0 ? slope : -slope);
  }
  float loss = (1.0f - e) * minus_log_sigmoid(d);
  if (e > 0.0f) loss += e * minus_log_sigmoid(-d);         // not 0 * inf
  const double mine[4] = {loss, d > 0.0f ? 1.0 : 0.0, chosen, rejected};
  double out[4];
  if (last_cta_sums(mine, a.partial, a.ticket, blockIdx.x, gridDim.x, out))
    for (int i = 0; i < 4; ++i)
      a.stats[i] = static_cast<float>(out[i]) / static_cast<float>(a.pairs);
}

// ---- launches

template <typename T, int PASS>
cudaError_t prepare_pass() {
  return cudaFuncSetAttribute(ring_kernel<T, PASS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(sizeof(RingShared)));
}
template <typename T>
cudaError_t prepare_typed() {
  cudaError_t e = prepare_pass<T, kPassLogps>();
  if (e == cudaSuccess) e = prepare_pass<T, kPassPolicy>();
  if (e == cudaSuccess) e = prepare_pass<T, kPassPolicyGrad>();
  if (e == cudaSuccess) e = prepare_pass<T, kPassPrefer>();
  if (e == cudaSuccess) e = prepare_pass<T, kPassGrad>();
  return e;
}

cudaLaunchConfig_t ring_config(int clusters, int size, cudaStream_t s, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(size);
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(clusters * size));
  c.blockDim = dim3(kRingThreads);
  c.dynamicSmemBytes = sizeof(RingShared);
  c.stream = s;
  c.attrs = attr;
  c.numAttrs = 1;
  return c;
}

// CTAs per row.  Where a share of the row waits in the ring for the row's sum,
// room beside it for the next rows is worth more CTAs per row: at most
// kSharePieces of the kMaxSlots.  With fewer rows than half the clusters, rows are
// cut finer, down to one slot per CTA.
int cluster_for(int pass, int64_t rows, int64_t row_bytes, int sms) {
  int size = 1;
  if (pass == kPassPolicyGrad)
    while (size < kMaxCluster && row_bytes > 1LL * kSharePieces * kSlotBytes * size) size *= 2;
  while (size < kMaxCluster && rows * size * 2 <= sms && row_bytes > kSlotBytes * size) size *= 2;
  return size;
}

template <typename T>
constexpr int dtype_index() {
  return std::is_same<T, float>::value ? ADAMW_F32
                                       : (std::is_same<T, __half>::value ? ADAMW_F16 : ADAMW_BF16);
}

template <typename T, int PASS>
cudaError_t launch_pass(const LossArgs& a, const LossLimits& lim, cudaStream_t s) {
  // the wide stores and bulk copies out need every gradient row at its logits'
  // offset from the 16-byte grid
  const bool same_grid =
      a.dlogits != nullptr &&
      ((reinterpret_cast<uintptr_t>(a.dlogits) - reinterpret_cast<uintptr_t>(a.logits)) % 16 == 0) &&
      (((a.dstride - a.stride) * static_cast<int64_t>(sizeof(T))) % 16 == 0);
  if (a.vocab <= kSmallVocabBytes / static_cast<int>(sizeof(T)))
    return launch_small_vocab<T>(static_cast<Pass>(PASS), a, same_grid,
                                 lim.small_ctas[dtype_index<T>()], s);
  const int size = cluster_for(PASS, a.rows, static_cast<int64_t>(a.vocab) * sizeof(T), lim.sms);
  int most = lim.clusters[size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3];
  const int clusters = static_cast<int>(a.rows < 1 ? 1 : (a.rows < most ? a.rows : most));
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t c = ring_config(clusters, size, s, attr);
  // the second pass may come up while the one before drains
  if (PASS == kPassGrad) c.numAttrs += early_start(&attr[1]);
  return cudaLaunchKernelEx(&c, ring_kernel<T, PASS>, a, same_grid ? 1 : 0);
}

cudaError_t launch_pairs(const LossArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(a.pairs));
  c.blockDim = dim3(kPairThreads);
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = early_start(&attr);
  return cudaLaunchKernelEx(&c, pair_kernel, a);
}

template <typename T>
cudaError_t launch_typed(LossKind kind, LossArgs a, const LossLimits& lim, cudaStream_t s) {
  const int64_t row_bytes = static_cast<int64_t>(a.vocab) * sizeof(T);
  cudaError_t e;
  switch (kind) {
    case kLossLogps: return launch_pass<T, kPassLogps>(a, lim, s);
    case kLossPolicy:
      if (a.dlogits == nullptr) {
        a.row_stat = nullptr;
        a.row_coef = nullptr;
        return launch_pass<T, kPassPolicy>(a, lim, s);
      }
      // a share must fit the ring whole
      if (row_bytes <= static_cast<int64_t>(kMaxSlots - 1) * kSlotBytes * kMaxCluster)
        return launch_pass<T, kPassPolicyGrad>(a, lim, s);
      e = cudaMemsetAsync(a.row_coef, 0, a.rows * sizeof(float), s);
      if (e == cudaSuccess) e = launch_pass<T, kPassPolicy>(a, lim, s);
      if (e == cudaSuccess && a.rows > 0) e = launch_pass<T, kPassGrad>(a, lim, s);
      return e;
    case kLossPrefer:
      e = launch_pass<T, kPassPrefer>(a, lim, s);
      if (e != cudaSuccess) return e;
      if ((e = launch_pairs(a, s)) != cudaSuccess) return e;
      if (a.dlogits != nullptr && a.rows > 0) e = launch_pass<T, kPassGrad>(a, lim, s);
      return e;
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t prepare_token_loss(int sms, LossLimits* lim) {
  cudaError_t e = prepare_typed<float>();
  if (e == cudaSuccess) e = prepare_typed<__half>();
  if (e == cudaSuccess) e = prepare_typed<__nv_bfloat16>();
  if (e == cudaSuccess) e = prepare_small_vocab<float>(sms, lim->small_ctas[ADAMW_F32]);
  if (e == cudaSuccess) e = prepare_small_vocab<__half>(sms, lim->small_ctas[ADAMW_F16]);
  if (e == cudaSuccess) e = prepare_small_vocab<__nv_bfloat16>(sms, lim->small_ctas[ADAMW_BF16]);
  lim->sms = sms;
  for (int i = 0; e == cudaSuccess && i < 4; ++i) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t c = ring_config(1, 1 << i, nullptr, &attr);
    e = cudaOccupancyMaxActiveClusters(&lim->clusters[i], ring_kernel<float, kPassPolicyGrad>, &c);
    if (e == cudaSuccess && lim->clusters[i] < 1) e = cudaErrorInvalidConfiguration;
    if (lim->clusters[i] > kLossMaxCtas) lim->clusters[i] = kLossMaxCtas;
  }
  return e;
}

cudaError_t launch_token_loss(adamw_dtype dt, LossKind kind, const LossArgs& a,
                              const LossLimits& lim, cudaStream_t s) {
  switch (dt) {
    case ADAMW_F32: return launch_typed<float>(kind, a, lim, s);
    case ADAMW_F16: return launch_typed<__half>(kind, a, lim, s);
    case ADAMW_BF16: return launch_typed<__nv_bfloat16>(kind, a, lim, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace adamw
