// token_loss.cu -- the token losses' row kernel, and the pairs of the
// preference loss.
//
// One cluster of C CTAs (C = 1, 2, 4, 8) works through rows of logits; each CTA
// has its share of every row pass through a ring of shared-memory slots:
//   producer (one thread)   bulk copies (TMA engine) of 16 KB pieces into free
//                           slots; for gradients, bulk copies of finished
//                           slots out to dlogits
//   scheduler (one warp)    walks the rows' labels and weights ahead of the
//                           others, deals live rows (and the rows that only
//                           need zeros) out to the clusters in turn, and hands
//                           each of its cluster's rows on with everything the
//                           row's arithmetic reads from memory
//   consumers (16 warps)    sum the exponentials of a row's pieces, join the
//                           sum over the cluster, and turn the same pieces,
//                           still in shared memory, into gradients in place
// A policy-loss row is so read once and its gradient written once.  What bounds
// it is DRAM: 4 bytes per 16-bit logit against about 11 instructions.
#include <cmath>

#include "cluster.cuh"
#include "token_math.cuh"

namespace adamw {
namespace {

constexpr int kSlotBytes = 16384;
constexpr int kSlots = 13;
constexpr int kSlotWords = kSlotBytes / 16;
constexpr int kConsumers = 16;                  // warps
constexpr int kConsumerThreads = kConsumers * 32;
constexpr int kRingThreads = kConsumerThreads + 64;
constexpr int kQueue = 8;                       // rows handed on ahead
constexpr int kPending = 16;                    // rows with slots in flight, at most kSlots
constexpr int kMaxCluster = 8;
constexpr int kRowsPerLane = 4;                 // rows the scheduler looks at per lane and step

// What a launch does with each live row.
enum Pass {
  kPassLogps,        // log-probabilities
  kPassPolicy,       // and the policy term
  kPassPolicyGrad,   // and the gradient
  kPassPrefer,       // log-probabilities, reference and sum kept for kPassGrad
  kPassGrad          // gradients of rows whose reference, sum and slope are known
};
__host__ __device__ constexpr bool writes_gradient(int pass) {
  return pass == kPassPolicyGrad || pass == kPassGrad;
}
__host__ __device__ constexpr bool policy_pass(int pass) {
  return pass == kPassPolicy || pass == kPassPolicyGrad;
}

enum RowKind { kRowLive, kRowZero, kRowStop };
struct QueueRow {
  int64_t row;
  int32_t kind;
  int32_t y;                  // the row's token
  float zy;
  PolicyRow policy;
  float c, s, slope;          // kPassGrad
  float edge[16];             // the row's first and last elements off the 16-byte grid
};

struct RingShared {
  alignas(128) unsigned char slot[kSlots][kSlotBytes];
  QueueRow queue[kQueue];
  float2 part[2][kMaxCluster * kConsumers];     // (c, s) of every consumer warp of the cluster
  struct {
    unsigned char* dst;
    int32_t words, pad;
  } pending[kPending];
  uint64_t full[kSlots];      // a slot's copy has landed
  uint64_t done[kSlots];      // the consumers are through with a slot
  uint64_t queue_full[kQueue], queue_empty[kQueue];
  uint64_t joined[2];         // the cluster's partial sums are in `part`
  uint32_t gave_up;
};

// A row of logits as this CTA sees it: elements off the 16-byte grid at either
// end, and its share of the 16-byte words between.
template <typename T>
struct RowShare {
  const unsigned char* base;  // the CTA's first word
  int64_t first;              // the element that word starts with
  int head, tail;             // ragged elements of the whole row
  int words, pieces;
  __device__ __forceinline__ RowShare(const T* z, int vocab, uint32_t rank, uint32_t ranks) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(z);
    const uintptr_t hi = lo + static_cast<uintptr_t>(vocab) * sizeof(T);
    const uintptr_t lo16 = (lo + 15) & ~static_cast<uintptr_t>(15);
    const uintptr_t hi16 = hi & ~static_cast<uintptr_t>(15);
    if (lo16 >= hi16) {       // no whole word: every element is ragged (at most 14)
      head = hi <= lo16 ? vocab : static_cast<int>((lo16 - lo) / sizeof(T));
      tail = vocab - head;
      words = pieces = 0;
      base = nullptr;
      first = 0;
      return;
    }
    head = static_cast<int>((lo16 - lo) / sizeof(T));
    tail = static_cast<int>((hi - hi16) / sizeof(T));
    const int64_t all = static_cast<int64_t>((hi16 - lo16) / 16);
    const int64_t per = ((all + ranks - 1) / ranks + 7) / 8 * 8;
    const int64_t from = min(per * rank, all);
    words = static_cast<int>(min(per, all - from));
    pieces = (words + kSlotWords - 1) / kSlotWords;
    base = reinterpret_cast<const unsigned char*>(lo16) + from * 16;
    first = head + from * kPerWord<T>;
  }
  __device__ __forceinline__ int piece_words(int j) const {
    return min(kSlotWords, words - j * kSlotWords);
  }
};

// ---- scheduler

template <int PASS>
__device__ __forceinline__ bool row_live(const LossArgs& a, int64_t t) {
  if (PASS == kPassGrad) return a.row_coef[t] != 0.0f;
  const int64_t y = label_of(a, t);
  return y >= 0 && y < a.vocab && (a.weights == nullptr || a.weights[t] != 0.0f);
}

template <typename T, int PASS>
__device__ void schedule(const LossArgs& a, RingShared& sh) {
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const uint32_t me = blockIdx.x / ranks, clusters = gridDim.x / ranks;
  const int lane = threadIdx.x & 31;
  uint32_t sent = 0;
  uint32_t live_turn = 0, zero_turn = 0;       // whose turn the next live / zero row is
  auto send = [&](int64_t row, int kind) -> bool {
    QueueRow& q = sh.queue[sent % kQueue];
    if (sent >= kQueue &&
        !mbar_wait(&sh.queue_empty[sent % kQueue], (sent / kQueue - 1) & 1u)) return false;
    if (kind == kRowLive) {
      const T* const z = static_cast<const T*>(a.logits) + row * a.stride;
      const RowShare<T> share(z, a.vocab, rank, ranks);
      const int64_t y = label_of(a, row);
      if (lane < 8) {
        if (lane < share.head) q.edge[lane] = to_f32(z[lane]);
      } else if (lane < 16) {
        if (lane - 8 < share.tail) q.edge[lane] = to_f32(z[a.vocab - share.tail + lane - 8]);
      } else if (lane == 16) {
        if (PASS != kPassGrad) q.zy = to_f32(z[y]);
      } else if (lane == 17) {
        if (policy_pass(PASS)) {
          q.policy.w = a.weights[row];
          q.policy.adv = a.advantages[row];
          q.policy.old = a.old_logps != nullptr ? a.old_logps[row] : 0.0f;
          q.policy.ref = a.ref_logps != nullptr ? a.ref_logps[row] : 0.0f;
        }
        if (PASS == kPassGrad) {
          const float2 st = a.row_stat[row];
          q.c = st.x;
          q.s = st.y;
          q.slope = a.row_coef[row];
        }
      }
      if (lane == 0) q.y = static_cast<int32_t>(y);
    }
    if (lane == 0) {
      q.row = row;
      q.kind = kind;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.queue_full[sent % kQueue]);
    ++sent;
    return true;
  };
  bool ok = true;
  for (int64_t base = 0; ok && base < a.rows; base += 32 * kRowsPerLane) {
    bool live[kRowsPerLane];
#pragma unroll
    for (int u = 0; u < kRowsPerLane; ++u) {
      const int64_t i = base + 32 * u + lane;
      // gradients of known rows run from the last row to the first: the pass
      // before ended there, so the end of the logits is still in L2
      const int64_t t = PASS == kPassGrad ? a.rows - 1 - i : i;
      live[u] = i < a.rows && row_live<PASS>(a, t);
    }
#pragma unroll
    for (int u = 0; u < kRowsPerLane; ++u) {
      const int64_t i = base + 32 * u + lane;
      const uint32_t in = __ballot_sync(kFull, i < a.rows);
      const uint32_t on = __ballot_sync(kFull, live[u]);
      const uint32_t off = in & ~on;
      const uint32_t before = (1u << lane) - 1u;
      const uint32_t turn = live[u] ? (live_turn + __popc(on & before)) % clusters
                                    : (zero_turn + __popc(off & before)) % clusters;
      uint32_t mine = __ballot_sync(kFull, i < a.rows && turn == me);
      live_turn = (live_turn + __popc(on)) % clusters;
      zero_turn = (zero_turn + __popc(off)) % clusters;
      while (ok && mine != 0u) {
        const int l = __ffs(mine) - 1;
        mine &= mine - 1u;
        const int64_t r = base + 32 * u + l;
        const int64_t t = PASS == kPassGrad ? a.rows - 1 - r : r;
        const bool is_live = (on >> l) & 1u;
        if (rank == 0 && lane == 0) {
          if (PASS == kPassPrefer) a.row_coef[t] = 0.0f;
          if (PASS != kPassGrad && !is_live) {
            a.logps[t] = 0.0f;
            if (a.lse != nullptr) a.lse[t] = 0.0f;
          }
        }
        if (is_live) ok = send(t, kRowLive);
        else if (writes_gradient(PASS)) ok = send(t, kRowZero);
      }
    }
  }
  if (ok) ok = send(0, kRowStop);
  if (!ok && lane == 0) atomicOr(&sh.gave_up, 1u);
}

// ---- producer

template <typename T, int PASS>
__device__ void produce(const LossArgs& a, RingShared& sh, bool bulk_out) {
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  constexpr bool kGrad = writes_gradient(PASS);
  uint32_t loads = 0, freed = 0;           // slot uses issued / whose slot may be refilled
  uint32_t stores = 0;
  uint32_t taken = 0;                      // queue rows taken
  uint32_t rows_in = 0, rows_out = 0;      // pending rows
  int piece = 0, pieces = 0, out_piece = 0;
  const unsigned char* src = nullptr;
  int words = 0;
  bool more = true, ok = true;
  while (ok) {
    // fill every free slot; wait for a row only when nothing is left to drain
    while (more && (!kGrad || loads - freed < kSlots)) {
      if (piece == pieces) {
        uint64_t* const bar = &sh.queue_full[taken % kQueue];
        const uint32_t parity = (taken / kQueue) & 1u;
        if (!mbar_try_wait(bar, parity)) {
          if (kGrad && stores != loads) break;
          if (!mbar_wait(bar, parity)) {
            ok = false;
            break;
          }
        }
        const QueueRow& q = sh.queue[taken % kQueue];
        const int kind = q.kind;
        const int64_t row = q.row;
        mbar_arrive(&sh.queue_empty[taken % kQueue]);
        ++taken;
        if (kind == kRowStop) {
          more = false;
          break;
        }
        if (kind == kRowZero) continue;
        const RowShare<T> share(static_cast<const T*>(a.logits) + row * a.stride, a.vocab, rank,
                                ranks);
        if (share.pieces == 0) continue;
        src = share.base;
        words = share.words;
        pieces = share.pieces;
        piece = 0;
        if (kGrad) {
          auto& p = sh.pending[rows_in % kPending];
          p.dst = reinterpret_cast<unsigned char*>(static_cast<T*>(a.dlogits) + row * a.dstride +
                                                   share.first);
          p.words = words;
          ++rows_in;
        }
      }
      const int s = loads % kSlots;
      if (!kGrad && loads >= kSlots &&
          !mbar_wait(&sh.done[s], (loads / kSlots - 1) & 1u)) {
        ok = false;
        break;
      }
      const uint32_t bytes = 16u * min(kSlotWords, words - piece * kSlotWords);
      mbar_expect_tx(&sh.full[s], bytes);
      bulk_g2s(sh.slot[s], src + static_cast<int64_t>(piece) * kSlotBytes, bytes, &sh.full[s]);
      ++loads;
      ++piece;
    }
    if (!ok) break;
    if (!kGrad) break;                     // every row has been issued
    if (stores == loads) {
      if (!more) break;
      continue;
    }
    if (piece < pieces && rows_in - rows_out == 1 && freed < stores) {
      // the consumers wait for the rest of this row, which may need the slot
      // whose copy out was left running
      bulk_wait_read_all();
      freed = stores;
      continue;
    }
    const int s = stores % kSlots;
    if (!mbar_wait(&sh.done[s], (stores / kSlots) & 1u)) {
      ok = false;
      break;
    }
    const auto& p = sh.pending[rows_out % kPending];
    if (bulk_out) {
      bulk_s2g(p.dst + static_cast<int64_t>(out_piece) * kSlotBytes, sh.slot[s],
               16u * min(kSlotWords, p.words - out_piece * kSlotWords));
      bulk_commit();
    }
    ++stores;
    if ((++out_piece) * kSlotWords >= p.words) {
      out_piece = 0;
      ++rows_out;
    }
    if (bulk_out) {
      bulk_wait_read_all_but_one();
      freed = stores - 1;
    } else {
      freed = stores;
    }
  }
  if (!ok) {
    atomicOr(&sh.gave_up, 2u);
    // copies in flight land before the CTA may leave
    for (uint32_t u = loads > kSlots ? loads - kSlots : 0; u < loads; ++u)
      mbar_wait(&sh.full[u % kSlots], (u / kSlots) & 1u);
  }
  bulk_wait_all();
}

// ---- consumers

template <typename T, int PASS>
__device__ void consume(const LossArgs& a, RingShared& sh, bool bulk_out, double (&acc)[4]) {
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int tid = threadIdx.x - 64, lane = tid & 31, warp = tid >> 5;
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  uint32_t use = 0, sums = 0;
  for (uint32_t n = 0;; ++n) {
    if (!mbar_wait(&sh.queue_full[n % kQueue], (n / kQueue) & 1u)) {
      if (lane == 0) atomicOr(&sh.gave_up, 4u);
      return;
    }
    const QueueRow& q = sh.queue[n % kQueue];
    const int64_t row = q.row;
    if (q.kind == kRowStop) return;
    if (q.kind == kRowZero) {
      T* const dz = static_cast<T*>(a.dlogits) + row * a.dstride;
      const RowShare<T> share(dz, a.vocab, rank, ranks);
      uint4* const out = reinterpret_cast<uint4*>(const_cast<unsigned char*>(share.base));
      for (int i = tid; i < share.words; i += kConsumerThreads) out[i] = make_uint4(0, 0, 0, 0);
      if (rank == 0 && tid < share.head) dz[tid] = from_f32<T>(0.0f);
      if (rank == 0 && tid < share.tail) dz[a.vocab - 1 - tid] = from_f32<T>(0.0f);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.queue_empty[n % kQueue]);
      continue;
    }
    const T* const z = static_cast<const T*>(a.logits) + row * a.stride;
    const RowShare<T> share(z, a.vocab, rank, ranks);
    // the ragged element this thread looks after: rank 0's first warp has them all
    const bool ragged = rank == 0 && warp == 0 &&
                        (lane < 8 ? lane < share.head : (lane < 16 && lane - 8 < share.tail));
    RowSum r{kLowest, 0.0f};
    float slope, logp = 0.0f, lse = 0.0f;
    if (PASS != kPassGrad) {
      for (int j = 0; j < share.pieces; ++j) {
        const uint32_t u = use + j;
        if (!mbar_wait(&sh.full[u % kSlots], (u / kSlots) & 1u)) {
          if (lane == 0) atomicOr(&sh.gave_up, 8u);
          return;
        }
        const uint4* const w = reinterpret_cast<const uint4*>(sh.slot[u % kSlots]);
        const int words = share.piece_words(j);
        if (words == kSlotWords) {
#pragma unroll
          for (int i = 0; i < kSlotWords / kConsumerThreads; ++i)
            add_word<T>(a, w[tid + i * kConsumerThreads], r);
        } else {
          for (int i = tid; i < words; i += kConsumerThreads) add_word<T>(a, w[i], r);
        }
        if (!writes_gradient(PASS)) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.done[u % kSlots]);
        }
      }
      if (ragged) {
        const float x = q.edge[lane];
        r.raise(x * a.k);
        r.s += exp2_fast(arg(a, x, r.c));
      }
      // join over the warp, then over all warps of the cluster: every warp
      // leaves its pair in every CTA
      r.join_warp();
      float2* const part = sh.part[sums & 1u];
      uint64_t* const bar = &sh.joined[sums & 1u];
      if (lane < static_cast<int>(ranks)) {
        cluster_store2(cluster_map(&part[rank * kConsumers + warp], lane), r.c, r.s);
        cluster_arrive(cluster_map(bar, lane));
      }
      if (!mbar_wait_cluster(bar, (sums >> 1) & 1u)) {
        if (lane == 0) atomicOr(&sh.gave_up, 16u);
        return;
      }
      ++sums;
      r = RowSum{kLowest, 0.0f};
      for (int i = lane; i < static_cast<int>(ranks) * kConsumers; i += 32)
        r.join(part[i].x, part[i].y);
      r.join_warp();
      const Log2Sum l = log2_sum(r);
      logp = logp_of(a, q.zy, l);
      lse = lse_of(l);
      if (policy_pass(PASS)) {
        const PolicyTerm p = policy_term(a, q.policy, logp);
        slope = p.slope;
        if (tid == 0) {
          acc[1] += p.policy;
          acc[2] += p.kl;
          acc[3] += p.clipped;
        }
      }
      if (rank == 0 && tid == 0) {
        a.logps[row] = logp;
        if (a.lse != nullptr) a.lse[row] = lse;
        if (PASS == kPassPrefer || PASS == kPassPolicy) {
          if (a.row_stat != nullptr) a.row_stat[row] = make_float2(r.c, r.s);
          if (PASS == kPassPolicy && a.row_coef != nullptr) a.row_coef[row] = slope;
        }
      }
    } else {
      r.c = q.c;
      r.s = q.s;
      slope = q.slope;
    }
    if (writes_gradient(PASS)) {
      const float coef = slope * out_scale;
      const float f = -coef / r.s;
      T* const dz = static_cast<T*>(a.dlogits) + row * a.dstride;
      for (int j = 0; j < share.pieces; ++j) {
        const uint32_t u = use + j;
        if (PASS == kPassGrad && !mbar_wait(&sh.full[u % kSlots], (u / kSlots) & 1u)) {
          if (lane == 0) atomicOr(&sh.gave_up, 8u);
          return;
        }
        uint4* const w = reinterpret_cast<uint4*>(sh.slot[u % kSlots]);
        const int words = share.piece_words(j);
        // the token's place relative to the piece's first element
        const int64_t first = share.first + static_cast<int64_t>(j) * kSlotWords * kPerWord<T>;
        const int at = static_cast<int>(max(min(q.y - first, (int64_t)INT32_MAX), (int64_t)-1));
        auto one = [&](int i) {
          const int rel = at < 0 ? -1 : at - i * kPerWord<T>;
          const uint4 d = grad_word<T>(a, w[i], r.c, f, coef, rel);
          if (bulk_out) {
            w[i] = d;
          } else {
            const T* const e = reinterpret_cast<const T*>(&d);
#pragma unroll
            for (int m = 0; m < kPerWord<T>; ++m) dz[first + i * kPerWord<T> + m] = e[m];
          }
        };
        if (words == kSlotWords) {
#pragma unroll
          for (int i = 0; i < kSlotWords / kConsumerThreads; ++i) one(tid + i * kConsumerThreads);
        } else {
          for (int i = tid; i < words; i += kConsumerThreads) one(i);
        }
        if (bulk_out) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.done[u % kSlots]);
      }
      if (ragged) {
        const int e = lane < 8 ? lane : a.vocab - share.tail + lane - 8;
        float d = exp2_fast(grad_arg<T>(a, q.edge[lane], r.c)) * f;
        if (e == q.y) d += coef;
        dz[e] = from_f32<T>(d);
      }
    }
    use += share.pieces;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.queue_empty[n % kQueue]);
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
      mbar_init(&sh.done[i], kConsumers);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&sh.queue_full[i], 1);
      mbar_init(&sh.queue_empty[i], kConsumers + 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&sh.joined[i], kConsumers * ranks);
    sh.gave_up = 0u;
    fence_mbar_init();
  }
  cluster_sync();
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  if (threadIdx.x < 32) {
    if (threadIdx.x == 0) produce<T, PASS>(a, sh, bulk_out != 0);
  } else if (threadIdx.x < 64) {
    schedule<T, PASS>(a, sh);
  } else {
    consume<T, PASS>(a, sh, bulk_out != 0, acc);
  }
  __syncwarp();
  // no CTA leaves while another may still write to its shared memory
  cluster_sync();
  if (threadIdx.x == 0 && sh.gave_up != 0u) atomicOr(a.fault, sh.gave_up);
  if (policy_pass(PASS) && cluster_rank() == 0) {
    // the sums sit in the first consumer thread
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
__device__ __forceinline__ double minus_log_sigmoid(double d) {
  return log1p(exp(-fabs(d))) + fmax(-d, 0.0);
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
  const double beta = a.beta, e = a.smoothing;
  const double chosen = beta * sum[0], rejected = beta * sum[1], d = chosen - rejected;
  // d loss / d d = e - sigmoid(-d), over the pairs' mean
  const double sig = d >= 0.0 ? exp(-d) / (1.0 + exp(-d)) : 1.0 / (1.0 + exp(d));
  const float slope = static_cast<float>((e - sig) * beta / a.pairs);
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
  const double mine[4] = {(1.0 - e) * minus_log_sigmoid(d) + e * minus_log_sigmoid(-d),
                          d > 0.0 ? 1.0 : 0.0, chosen, rejected};
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

// CTAs per row.  A gradient pass keeps a CTA's share of the row in the ring
// until the row's sum is known and wants room beside it to fetch the next row:
// at most 8 of the 13 slots.  With fewer rows than half the clusters, the rows
// are cut finer, down to one slot per CTA.
int cluster_for(int pass, int64_t rows, int64_t row_bytes, int sms) {
  int size = 1;
  if (pass == kPassPolicyGrad)
    while (size < kMaxCluster && row_bytes > 8LL * kSlotBytes * size) size *= 2;
  while (size < kMaxCluster && rows * size * 2 <= sms && row_bytes > kSlotBytes * size) size *= 2;
  return size;
}

template <typename T, int PASS>
cudaError_t launch_ring(const LossArgs& a, const LossLimits& lim, cudaStream_t s) {
  const int size = cluster_for(PASS, a.rows, static_cast<int64_t>(a.vocab) * sizeof(T), lim.sms);
  int most = lim.clusters[size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3];
  const int clusters = static_cast<int>(a.rows < 1 ? 1 : (a.rows < most ? a.rows : most));
  // the bulk copies out need every gradient row at its logits' offset from the
  // 16-byte grid
  const bool bulk_out =
      a.dlogits != nullptr &&
      ((reinterpret_cast<uintptr_t>(a.dlogits) - reinterpret_cast<uintptr_t>(a.logits)) % 16 == 0) &&
      (((a.dstride - a.stride) * static_cast<int64_t>(sizeof(T))) % 16 == 0);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t c = ring_config(clusters, size, s, &attr);
  return cudaLaunchKernelEx(&c, ring_kernel<T, PASS>, a, bulk_out ? 1 : 0);
}

template <typename T>
cudaError_t launch_typed(LossKind kind, LossArgs a, const LossLimits& lim, cudaStream_t s) {
  const int64_t row_bytes = static_cast<int64_t>(a.vocab) * sizeof(T);
  cudaError_t e;
  switch (kind) {
    case kLossLogps: return launch_ring<T, kPassLogps>(a, lim, s);
    case kLossPolicy:
      if (a.dlogits == nullptr) {
        a.row_stat = nullptr;
        a.row_coef = nullptr;
        return launch_ring<T, kPassPolicy>(a, lim, s);
      }
      // a share must fit the ring whole
      if (row_bytes <= static_cast<int64_t>(kSlots - 1) * kSlotBytes * kMaxCluster)
        return launch_ring<T, kPassPolicyGrad>(a, lim, s);
      e = cudaMemsetAsync(a.row_coef, 0, a.rows * sizeof(float), s);
      if (e == cudaSuccess) e = launch_ring<T, kPassPolicy>(a, lim, s);
      if (e == cudaSuccess && a.rows > 0) e = launch_ring<T, kPassGrad>(a, lim, s);
      return e;
    case kLossPrefer:
      e = launch_ring<T, kPassPrefer>(a, lim, s);
      if (e != cudaSuccess) return e;
      pair_kernel<<<a.pairs, kPairThreads, 0, s>>>(a);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      if (a.dlogits != nullptr && a.rows > 0) e = launch_ring<T, kPassGrad>(a, lim, s);
      return e;
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t prepare_token_loss(int sms, LossLimits* lim) {
  cudaError_t e = prepare_typed<float>();
  if (e == cudaSuccess) e = prepare_typed<__half>();
  if (e == cudaSuccess) e = prepare_typed<__nv_bfloat16>();
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
