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
constexpr int kSlots = 13;
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
constexpr int kBatch = 4;                       // rows whose inputs it fetches together
constexpr int kSharePieces = 7;                 // of a row that waits for its sum, at most

// Warps of either kind; a pass with one kind gives it all of them.
__host__ __device__ constexpr int sum_warps(int pass) {
  return !sums(pass) ? 0 : (writes_gradient(pass) ? kWorkers / 2 : kWorkers);
}
__host__ __device__ constexpr int grad_warps(int pass) { return kWorkers - sum_warps(pass); }

enum RowKind { kRowLive, kRowZero, kRowStop };
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
  alignas(128) unsigned char slot[kSlots][kSlotBytes];
  QueueRow queue[kQueue];
  DealtRow dealt[kBatch + 32 * kRowsPerLane];   // this cluster's next rows, scheduler only
  float2 part[kQueue][kWorkers];          // (c, s) of every summing warp
  float2 cross[kJoins][kMaxCluster];      // (c, s) of every CTA of the cluster
  struct {
    float c, f, coef, pad;
  } result[kQueue];                       // what the gradient warps need of a row
  uint64_t full[kSlots];      // a slot's copy has landed
  uint64_t done[kSlots];      // a slot's gradients are in place
  uint64_t empty[kSlots];     // a slot may be filled again
  uint64_t queue_full[kQueue], queue_empty[kQueue];
  uint64_t summed[kQueue];    // a row's `part` is complete
  uint64_t joined[kJoins];    // a row's `cross` is complete
  uint64_t ready[kQueue];     // a row's `result` is there
  uint32_t gave_up;
};

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
  // labels and weights of the next step's rows, on their way while this step's
  // rows are dealt
  int64_t ahead_y[kRowsPerLane];
  float ahead_w[kRowsPerLane];
  auto look = [&](int64_t at) {
    const float* const weights = PASS == kPassGrad ? a.row_coef : a.weights;
#pragma unroll
    for (int u = 0; u < kRowsPerLane; ++u) {
      const int64_t i = at + 32 * u + lane;
      // gradients of known rows run from the last row to the first: the pass
      // before ended there, so the end of the logits is still in L2
      const int64_t t = PASS == kPassGrad ? a.rows - 1 - i : i;
      ahead_y[u] = i < a.rows ? label_of(a, t) : -1;
      ahead_w[u] = i < a.rows && weights != nullptr ? weights[t] : 1.0f;
    }
  };
  look(0);
  for (;;) {
    if (next == held) next = held = 0;
    while (held - next < kBatch && held <= kBatch && base < a.rows) {
      int64_t y[kRowsPerLane];
      float w[kRowsPerLane];
#pragma unroll
      for (int u = 0; u < kRowsPerLane; ++u) {
        y[u] = ahead_y[u];
        w[u] = ahead_w[u];
      }
      look(base + 32 * kRowsPerLane);
#pragma unroll
      for (int u = 0; u < kRowsPerLane; ++u) {
        const int64_t i = base + 32 * u + lane;
        const int64_t t = PASS == kPassGrad ? a.rows - 1 - i : i;
        const bool is_live = w[u] != 0.0f && y[u] >= 0 && y[u] < a.vocab;
        const uint32_t on = __ballot_sync(kFull, is_live);
        const uint32_t off = __ballot_sync(kFull, i < a.rows && !is_live);
        const uint32_t before = (1u << lane) - 1u;
        const uint32_t turn = is_live ? (live_turn + __popc(on & before)) % clusters
                                      : (zero_turn + __popc(off & before)) % clusters;
        const bool mine = i < a.rows && turn == me;
        live_turn = (live_turn + __popc(on)) % clusters;
        zero_turn = (zero_turn + __popc(off)) % clusters;
        if (mine && rank == 0) {
          if (PASS == kPassPrefer) a.row_coef[t] = 0.0f;
          if (PASS != kPassGrad && !is_live) {
            a.logps[t] = 0.0f;
            if (a.lse != nullptr) a.lse[t] = 0.0f;
          }
        }
        const bool send = mine && (is_live || writes_gradient(PASS));
        const uint32_t sends = __ballot_sync(kFull, send);
        if (send)
          sh.dealt[held + __popc(sends & before)] = {t, is_live ? kRowLive : kRowZero,
                                                     static_cast<int32_t>(y[u])};
        held += __popc(sends);
      }
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
      if (sent >= kQueue && !mbar_wait(&sh.queue_empty[q], (sent / kQueue - 1) & 1u)) {
        atomicOr(&sh.gave_up, 1u);
        return;
      }
      if (lane < kInputs) sh.queue[q].in[lane] = in[i];
      if (lane == 0) static_cast<DealtRow&>(sh.queue[q]) = d;
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
__device__ __forceinline__ bool take_row(RingShared& sh, uint32_t n, uint32_t site) {
  if (mbar_wait(&sh.queue_full[n % kQueue], (n / kQueue) & 1u)) return true;
  atomicOr(&sh.gave_up, site);
  return false;
}

template <typename T>
__device__ void load_rows(const LossArgs& a, RingShared& sh) {
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  uint32_t use = 0;
  bool ok = true;
  for (uint32_t n = 0; ok && (ok = take_row(sh, n, 2u)); ++n) {
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
  // after a wait that gave up, the copies in flight land before the CTA may leave
  if (!ok)
    for (uint32_t u = use > kSlots ? use - kSlots : 0; u < use; ++u)
      mbar_wait(&sh.full[u % kSlots], (u / kSlots) & 1u);
}

template <typename T>
__device__ void store_rows(const LossArgs& a, RingShared& sh, bool bulk_out) {
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
  constexpr int kThreadsHere = sum_warps(PASS) * 32;
  constexpr int kEach = kSlotWords / kThreadsHere;       // words per thread and full piece
  constexpr int kRun = kEach < 2 ? kEach : 2;            // words summed together
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int lane = threadIdx.x & 31, tid = warp * 32 + lane;
  uint32_t use = 0;
  for (uint32_t n = 0; take_row(sh, n, 4u); ++n) {
    const QueueRow& q = sh.queue[n % kQueue];
    if (q.kind == kRowStop) return;
    if (q.kind == kRowLive) {
      const RowShare<T> share(static_cast<const T*>(a.logits) + q.row * a.stride, a.vocab, rank,
                              ranks);
      RowSum r{kLowest, 0.0f};
      for (int j = 0; j < share.pieces; ++j, ++use) {
        const uint32_t slot = use % kSlots;
        if (!mbar_wait(&sh.full[slot], (use / kSlots) & 1u)) {
          atomicOr(&sh.gave_up, 8u);
          return;
        }
        const uint4* const w = reinterpret_cast<const uint4*>(sh.slot[slot]) + tid;
        const int words = share.piece_words(j);
        if (words == kSlotWords) {
#pragma unroll
          for (int i = 0; i < kEach; i += kRun) {
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
      if (!mbar_wait(&sh.summed[e], (n / kQueue) & 1u)) {
        atomicOr(&sh.gave_up, 32u);
        return;
      }
      RowSum r{kLowest, 0.0f};
      if (lane < sum_warps(PASS)) r = RowSum{sh.part[e][lane].x, sh.part[e][lane].y};
      r.join_lanes<sum_warps(PASS)>();
      if (ranks > 1) {
        r = RowSum{__shfl_sync(kFull, r.c, 0), __shfl_sync(kFull, r.s, 0)};
        const int b = joins % kJoins;
        if (lane < static_cast<int>(ranks)) {
          cluster_store2(cluster_map(&sh.cross[b][rank], lane), r.c, r.s);
          cluster_arrive(cluster_map(&sh.joined[b], lane));
        }
        if (!mbar_wait_cluster(&sh.joined[b], (joins / kJoins) & 1u)) {
          atomicOr(&sh.gave_up, 64u);
          return;
        }
        ++joins;
        r = RowSum{kLowest, 0.0f};
        if (lane < static_cast<int>(ranks)) r = RowSum{sh.cross[b][lane].x, sh.cross[b][lane].y};
        r.join_lanes<kMaxCluster>();
      }
      const Log2Sum l = log2_sum(r);
      const float logp = logp_of(a, q.in[kInToken], l);
      float slope = 0.0f;
      if (policy_pass(PASS)) {
        const PolicyTerm p = policy_term(a, {q.in[kInWeight], q.in[kInAdvantage], q.in[kInOld], q.in[kInRef]}, logp);
        slope = p.slope;
        acc[1] += p.policy;
        acc[2] += p.kl;
        acc[3] += p.clipped;
      }
      if (lane == 0) {
        if (writes_gradient(PASS)) {
          const float coef = slope * out_scale;
          sh.result[e] = {r.c, -coef / r.s, coef, 0.0f};
        }
        if (rank == 0) {
          a.logps[row] = logp;
          if (a.lse != nullptr) a.lse[row] = lse_of(l);
          if ((PASS == kPassPrefer || PASS == kPassPolicy) && a.row_stat != nullptr) {
            a.row_stat[row] = make_float2(r.c, r.s);
            if (PASS == kPassPolicy) a.row_coef[row] = slope;
          }
        }
      }
    }
    if (writes_gradient(PASS) && lane == 0) mbar_arrive(&sh.ready[e]);
    leave_row(sh, n);
  }
}

template <typename T, int PASS>
__device__ void grad_rows(const LossArgs& a, RingShared& sh, int warp, bool bulk_out) {
  constexpr int kThreadsHere = grad_warps(PASS) * 32;
  constexpr int kEach = kSlotWords / (kThreadsHere > 0 ? kThreadsHere : 1);
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int lane = threadIdx.x & 31, tid = warp * 32 + lane;
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  uint32_t use = 0;
  for (uint32_t n = 0; take_row(sh, n, 128u); ++n) {
    const QueueRow& q = sh.queue[n % kQueue];
    if (q.kind == kRowStop) return;
    const int e = n % kQueue;
    T* const dz = static_cast<T*>(a.dlogits) + q.row * a.dstride;
    if (sums(PASS) && !mbar_wait(&sh.ready[e], (n / kQueue) & 1u)) {
      atomicOr(&sh.gave_up, 256u);
      return;
    }
    if (q.kind == kRowZero) {
      const RowShare<T> share(dz, a.vocab, rank, ranks);
      uint4* const out = reinterpret_cast<uint4*>(const_cast<unsigned char*>(share.base));
      for (int i = tid; i < share.words; i += kThreadsHere) out[i] = make_uint4(0, 0, 0, 0);
      if (rank == 0 && tid < share.head) dz[tid] = from_f32<T>(0.0f);
      if (rank == 0 && tid < share.tail) dz[a.vocab - 1 - tid] = from_f32<T>(0.0f);
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
      f = -coef / q.in[kInSum];
    }
    // the token's place relative to this thread's first word
    const int64_t from = share.first + tid * kPerWord<T>;
    const int at = static_cast<int>(q.y - from);            // vocab is at most 2^30
    for (int j = 0; j < share.pieces; ++j, ++use) {
      const uint32_t slot = use % kSlots;
      if (!sums(PASS) && !mbar_wait(&sh.full[slot], (use / kSlots) & 1u)) {
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
        for (int i = 0; i < kEach; ++i) one(i * kThreadsHere);
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
__global__ void __launch_bounds__(kRingThreads, 1) ring_kernel(const LossArgs a, const int bulk_out) {
  extern __shared__ __align__(128) unsigned char raw[];
  RingShared& sh = *reinterpret_cast<RingShared*>(raw);
  const uint32_t ranks = cluster_size();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.done[i], grad_warps(PASS) > 0 ? grad_warps(PASS) : 1);
      mbar_init(&sh.empty[i], writes_gradient(PASS) ? 1 : sum_warps(PASS));
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
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const int warp = threadIdx.x >> 5;
  if (warp == 0) {
    if (threadIdx.x == 0) load_rows<T>(a, sh);
  } else if (warp == 1) {
    schedule<T, PASS>(a, sh);
  } else if (warp == 2) {
    if constexpr (sums(PASS)) finish_rows<T, PASS>(a, sh, acc);
  } else if (warp == 3) {
    if (writes_gradient(PASS) && (threadIdx.x & 31) == 0) store_rows<T>(a, sh, bulk_out != 0);
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
    if (last_cta_sums(mine, a.partial, a.ticket, blockIdx.x / ranks, gridDim.x / ranks, out)) {
      a.stats[0] = static_cast<float>(out[1] + static_cast<double>(a.kl_coef) * out[2]);
      a.stats[1] = static_cast<float>(out[1]);
      a.stats[2] = static_cast<float>(out[2]);
      a.stats[3] = static_cast<float>(out[3]);
    }
  }
}

// ---- pairs

constexpr int kPairThreads = 256;

__device__ __forceinline__ bool pref_live(const LossArgs& a, int64_t t, float& w) {
  const int64_t y = label_of(a, t);
  w = a.weights != nullptr ? a.weights[t] : 1.0f;
  return w != 0.0f && y >= 0 && y < a.vocab;
}
// Sum over [lo, hi) of w (logp - ref), in every thread; rows without weight or
// token add nothing.
__device__ double sequence_sum(const LossArgs& a, int64_t lo, int64_t hi, double* s_warp) {
  double x = 0.0;
  for (int64_t t = lo + threadIdx.x; t < hi; t += kPairThreads) {
    float w;
    if (pref_live(a, t, w))
      x += static_cast<double>(w) * (static_cast<double>(a.logps[t]) - a.ref_logps[t]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
  for (int i = 0; i < kPairThreads / 32; ++i) x += s_warp[i];
  return x;
}

// -log sigmoid(d)
__device__ __forceinline__ float minus_log_sigmoid(float d) {
  return log1pf(expf(-fabsf(d))) + fmaxf(-d, 0.0f);
}

// One CTA per pair: both sequences' rewards, the pair's loss, and
// d loss / d logp of their rows.
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const LossArgs a) {
  __shared__ double s_warp[kPairThreads / 32];
  const int p = blockIdx.x;
  int64_t lo[2], hi[2];
  double sum[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int s = p + side * a.pairs;
    lo[side] = min(max(static_cast<int64_t>(a.starts[s]), (int64_t)0), a.rows);
    hi[side] = min(max(static_cast<int64_t>(a.starts[s + 1]), lo[side]), a.rows);
    sum[side] = sequence_sum(a, lo[side], hi[side], s_warp);
  }
  const double beta = a.beta, chosen = beta * sum[0], rejected = beta * sum[1];
  const float e = a.smoothing, d = static_cast<float>(chosen - rejected);
  // d loss / d d = e - sigmoid(-d), over the pairs' mean
  const float t = expf(-fabsf(d));
  const float sig = d >= 0.0f ? t / (1.0f + t) : 1.0f / (1.0f + t);
  const float slope = (e - sig) * a.beta / static_cast<float>(a.pairs);
  if (threadIdx.x == 0) {
    a.rewards[p] = static_cast<float>(chosen);
    a.rewards[p + a.pairs] = static_cast<float>(rejected);
  }
#pragma unroll
  for (int side = 0; side < 2; ++side)
    for (int64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kPairThreads) {
      float w;
      if (pref_live(a, t, w)) a.row_coef[t] = w * (side == 0 ? slope : -slope);
    }
  const double mine[4] = {(1.0f - e) * minus_log_sigmoid(d) + e * minus_log_sigmoid(-d),
                          d > 0.0f ? 1.0 : 0.0, chosen, rejected};
  double out[4];
  if (last_cta_sums(mine, a.partial, a.ticket, blockIdx.x, gridDim.x, out))
    for (int i = 0; i < 4; ++i) a.stats[i] = static_cast<float>(out[i] / a.pairs);
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
// kSharePieces of the kSlots.  With fewer rows than half the clusters, rows are
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
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t c = ring_config(clusters, size, s, &attr);
  return cudaLaunchKernelEx(&c, ring_kernel<T, PASS>, a, same_grid ? 1 : 0);
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
      if (row_bytes <= static_cast<int64_t>(kSlots - 1) * kSlotBytes * kMaxCluster)
        return launch_pass<T, kPassPolicyGrad>(a, lim, s);
      e = cudaMemsetAsync(a.row_coef, 0, a.rows * sizeof(float), s);
      if (e == cudaSuccess) e = launch_pass<T, kPassPolicy>(a, lim, s);
      if (e == cudaSuccess && a.rows > 0) e = launch_pass<T, kPassGrad>(a, lim, s);
      return e;
    case kLossPrefer:
      e = launch_pass<T, kPassPrefer>(a, lim, s);
      if (e != cudaSuccess) return e;
      pair_kernel<<<a.pairs, kPairThreads, 0, s>>>(a);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
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
