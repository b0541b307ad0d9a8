// layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//   mean, rstd = 1 / sqrt(var + eps) per row;  xhat = (x - mean) rstd
//   y  = xhat w + b
//   dx = rstd (w dy - mean_j(w dy) - xhat mean_j(w dy xhat))
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// A group of G threads holds a row in registers, 16 or 32 elements a thread, and a
// resident grid walks the rows, bulk copies (TMA engine) keeping each group's
// next rows on their way into shared memory.  A thread has the same columns of
// every row: the weight stays in registers, and so do the column sums of the
// backward pass, which are added over a CTA's groups, then over the CTAs by a
// second kernel, always in the same order.
// Statistics and sums are float32; the variance is the mean of squared
// differences from the mean (no cancellation).  What bounds both passes is
// DRAM: two (three) accesses per element.  Rows wider than 16384 take the loops at
// the end of this file.
#include "async_copy.cuh"
#include "operators.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kMaxWidth = 16384;       // of a row in registers
template <int G> constexpr int kCta = G < 128 ? 128 : G;
// Resident threads per SM, by the registers a thread with `each` elements needs
// (a CTA of 512 threads is better off with a second one beside it: 8192 columns
// take 96 us with 1024 threads and 117 with 512; at 4096 columns 768 threads,
// which do not spill, take 88 us against 98).
constexpr int forward_threads(int group, int each) {
  return group >= 512 ? 1024 : (each == 16 ? 768 : 512);
}
// A group of 1024 threads has no registers left for the column sums: they are a
// kernel of their own then.
__host__ __device__ constexpr bool sums_columns(int group) { return group <= 512; }
constexpr int backward_threads(int group, int each) {
  return !sums_columns(group) ? 1024 : (each == 16 ? 512 : 256);
}
constexpr int kStages = 4;             // rows on their way per group, at most
constexpr int kSmemPerSm = 184 * 1024;  // for the rows on their way
// Rows of a group whose column sums one launch adds up in registers.  131072 x 8192
// bfloat16 backward: 965 us in one launch, 983 in two of at most 512 rows, 1002 in
// four of at most 256.
constexpr int kRunRows = 512;

template <typename W>
__device__ __forceinline__ float param(const void* p, int j, float none) {
  return p != nullptr ? to_f32(static_cast<const W*>(p)[j]) : none;
}

// How the rows of a call's matrices lie: on the 16-byte grid; off it, a row of
// each matrix by the same shift (dense rows of an odd width); each in its own way.
enum class Lie { grid, shifted, any };

// A thread's EACH elements of a row as loaded: 16-byte words of a row whose
// first one starts after `head` elements, or single elements where the matrices
// lie each in its own way; thread tid has the columns
// head + (i G + tid) E .. + E - 1.  A shifted row's elements before its first and
// after its last whole word, fewer than E each, go one each to the last threads
// as a pair more.  (Masked words at both ends instead cost every warp with one of
// them as much again as the rest of a row.)  Rows `period` apart have the same
// shift and a CTA keeps to such rows, so that a thread keeps its columns.
// 32768 rows of bfloat16, with words against single elements, us: 1601 columns
// forward 55 against 74, backward 78 against 92; 5001 columns 197 against 404 and
// 268 against 370.  float32 gains less (5001: 231 against 390, 335 against 360)
// and nothing at 1601 (80 against 74, 102 against 104).
// The arithmetic takes the columns in pairs (two float32 operations per
// instruction: without, both passes issued 22 to 27 instructions per element and
// were bound by that).
template <typename T, Lie LIE, int G, int EACH>
struct Piece {
  static constexpr bool kWords = LIE != Lie::any;
  static constexpr bool kShifted = LIE == Lie::shifted;
  static constexpr int E = kWords ? 16 / sizeof(T) : 1;
  static constexpr int N = EACH / E;
  static constexpr int kPairs = EACH / 2 + (kShifted ? 1 : 0);
  using Raw = typename std::conditional<kWords, uint4, T>::type;
  Raw raw[N];
  T end[2];              // of a shifted row: of its first and of its last elements

  // A thread's place in the rows.
  struct Place {
    int tid, width;
    int shift;           // elements from the 16-byte grid to the row
    int head, tail;      // columns [0, head) and [tail, width) lie outside whole words
    __device__ __forceinline__ Place(int tid_, int width_, int shift_)
        : tid(tid_), width(width_), shift(kShifted ? shift_ : 0), head(0), tail(width_) {
      if (kShifted) {
        head = min((E - shift) % E, width);
        tail = head + (width - head) / E * E;
      }
    }
    // Column of element m, and whether the thread has it.
    __device__ __forceinline__ int column(int m) const {
      if (m >= EACH) return (m == EACH ? 0 : tail) + G - 1 - tid;
      return head + (m / E * G + tid) * E + m % E;
    }
    __device__ __forceinline__ bool has(int m) const {
      return column(m) < (m < EACH ? tail : m == EACH ? head : width);
    }
    // Whether it has no part in pair k, the one more of a shifted row.
    __device__ __forceinline__ bool idle(int k) const { return k >= EACH / 2 && tid < G - E; }
    // Whether it has word i (a word has all its elements or none).
    __device__ __forceinline__ bool word(int i) const { return has(i * E); }
  };

  static __device__ __forceinline__ Raw zero() {
    if constexpr (kWords) return make_uint4(0u, 0u, 0u, 0u);
    else return from_f32<T>(0.0f);
  }
  // From a row's whole words in shared memory; elements it has not read as 0.
  __device__ __forceinline__ void load(const unsigned char* words, const Place& at) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      raw[i] = at.word(i) ? reinterpret_cast<const Raw*>(words)[i * G + at.tid] : zero();
  }
  __device__ __forceinline__ float2 pair(int k) const {
    if (k >= EACH / 2) return make_float2(to_f32(end[0]), to_f32(end[1]));
    if constexpr (!kWords) {
      return make_float2(to_f32(raw[2 * k]), to_f32(raw[2 * k + 1]));
    } else if constexpr (sizeof(T) == 4) {
      const uint4& r = raw[k / 2];
      return k % 2 ? make_float2(__uint_as_float(r.z), __uint_as_float(r.w))
                   : make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
    } else {
      const uint4& r = raw[k / 4];
      return unpack_pair<T>(k % 4 == 0 ? r.x : k % 4 == 1 ? r.y : k % 4 == 2 ? r.z : r.w);
    }
  }
  // x where the thread has pair k's elements, else 0.
  static __device__ __forceinline__ float2 inside(float2 x, int k, const Place& at) {
    const bool in0 = k < EACH / 2 ? at.word(2 * k / E) : at.has(2 * k);
    const bool in1 = kWords && k < EACH / 2 ? in0 : at.has(2 * k + 1);
    return make_float2(in0 ? x.x : 0.0f, in1 ? x.y : 0.0f);
  }
  // Stores f(pair) at every column the thread has, rounded once.
  template <typename F>
  static __device__ __forceinline__ void store(T* row, const Place& at, F f) {
#pragma unroll
    for (int k = kWords ? EACH / 2 : 0; k < kPairs; ++k) {
      if (at.idle(k)) continue;
      const float2 x = f(k);
      if (at.has(2 * k)) row[at.column(2 * k)] = from_f32<T>(x.x);
      if (at.has(2 * k + 1)) row[at.column(2 * k + 1)] = from_f32<T>(x.y);
    }
    if constexpr (kWords) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!at.word(i)) continue;
        uint4 out;
        if constexpr (sizeof(T) == 4) {
          const float2 x = f(2 * i), y = f(2 * i + 1);
          out = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x),
                           __float_as_uint(y.y));
        } else {
          out = make_uint4(pack_pair<T>(f(4 * i)), pack_pair<T>(f(4 * i + 1)),
                           pack_pair<T>(f(4 * i + 2)), pack_pair<T>(f(4 * i + 3)));
        }
        __stcs(reinterpret_cast<uint4*>(row + at.column(i * E)), out);
      }
    }
  }
};

// A thread's pairs of a parameter; 0 where it has no column.
template <typename W, typename P>
__device__ __forceinline__ void load_params(const void* p, float none, const typename P::Place& at,
                                            float2 (&out)[P::kPairs]) {
#pragma unroll
  for (int k = 0; k < P::kPairs; ++k)
    out[k] = make_float2(at.has(2 * k) ? param<W>(p, at.column(2 * k), none) : 0.0f,
                         at.has(2 * k + 1) ? param<W>(p, at.column(2 * k + 1), none) : 0.0f);
}

__device__ __forceinline__ float plus(float x, float y) { return x + y; }
__device__ __forceinline__ float2 plus(float2 x, float2 y) { return add2(x, y); }
__device__ __forceinline__ float from_lane(float x, int o) { return __shfl_xor_sync(kFull, x, o); }
__device__ __forceinline__ float2 from_lane(float2 x, int o) {
  return make_float2(__shfl_xor_sync(kFull, x.x, o), __shfl_xor_sync(kFull, x.y, o));
}

// Sums over a group, a warp or the whole CTA; every thread of it gets them.  Two
// places in turn, so that one barrier per sum is enough.
template <typename V, int G>
struct GroupSum {
  static constexpr int kWarps = G / 32;
  V* part;               // [2][kWarps], 16-byte aligned
  int turn = 0;
  __device__ __forceinline__ V operator()(V x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = plus(x, from_lane(x, o));
    if (G > 32) {
      V* const p = part + turn * kWarps;
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) p[threadIdx.x / 32] = x;
      __syncthreads();
      constexpr int kWords = kWarps * sizeof(V) / 16 > 0 ? kWarps * sizeof(V) / 16 : 1;
      uint4 w[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
      const V* const v = reinterpret_cast<const V*>(w);
      x = v[0];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) x = plus(x, v[i]);
    }
    return x;
  }
};

// 1 / sqrt(x) for x >= 0: the hardware's approximation and one Newton step,
// about an ulp, in a sixth of the instructions of a root and a division (0 gives
// inf and inf gives 0, as they do).
__device__ __forceinline__ float inverse_root(float x) {
  const float y = rsqrtf(x);
  const float z = fmaf(y * fmaf(-x * y, y, 1.0f), 0.5f, y);
  return x > 0.0f && x <= 3.40282347e38f ? z : y;
}

// Whether a barrier's phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The rows of a group, in turn, of ARRAYS matrices: bulk copies into a ring of
// stages.  `take` leaves the current row in registers, `refill` (after every
// thread of the group has taken its part) sends for the row that comes `stages`
// rows later.
// Shifted rows are copied with what else their first and last words hold, the
// rows beside them; where that would be memory before the first row or after the
// last one, the threads read the elements of that word for themselves.
// Of rows that lie each in its own way whole words are copied, each row to the
// offset it has from the grid; the elements outside whole words come by plain
// loads, a row ahead, and the thread that has one puts it into the stage.
template <typename P, typename T, Lie LIE, int G, int ARRAYS>
struct Rows {
  const T* base[ARRAYS];
  int64_t stride[ARRAYS];
  int64_t rows, step, ahead;     // ahead: the next row to send for
  int64_t row;                   // the current row
  int32_t width, stages;
  unsigned char* ring;           // [stages][ARRAYS][pitch]
  uint64_t* full;                // [stages]
  uint64_t wait_ns;              // limit of a wait
  uint32_t* fault;
  uint32_t n = 0;
  // 1 + the use for which this thread's wait gave up: it waits no more, and thread
  // 0 sends no more.  (Where thread 0's own wait for a use succeeded its stage may be
  // filled again, whoever else gave up on it.)
  uint32_t lost = 0;
  // of the current row off the grid: its offset, whether this thread has one of
  // its first elements, the thread's column among its last ones, and both
  uint32_t off[ARRAYS];
  bool first[ARRAYS];
  int mine[ARRAYS];
  T edge[ARRAYS][2];
  // of shifted rows: their words; the first `low` of them are copied without
  // their first, the last `high` without their last word
  int32_t words, low, high;

  using Place = typename P::Place;
  static __host__ __device__ __forceinline__ uint32_t pitch_of(int32_t width) {
    return LIE == Lie::grid ? width * sizeof(T) : (width * sizeof(T) + 15) / 16 * 16 + 16;
  }
  __device__ __forceinline__ unsigned char* slot(uint32_t stage, int m) const {
    return ring + (stage * ARRAYS + m) * pitch_of(width);
  }
  __device__ __forceinline__ const T* start_of(int64_t r, int m) const { return base[m] + r * stride[m]; }

  // Of shifted rows, those whose first (last) word reaches past a matrix.
  __device__ __forceinline__ void find_edges(const Place& at) {
    words = (at.shift + width + P::E - 1) / P::E;
    low = 0;
    high = 0;
#pragma unroll
    for (int m = 0; m < ARRAYS; ++m) {
      const int over = words * P::E - at.shift - width;
      const int s = static_cast<int>(min(stride[m], static_cast<int64_t>(P::E)));
      low = max(low, (at.shift + s - 1) / s);
      high = max(high, (over + s - 1) / s);
    }
  }
  // A row's elements before its first and from its last 16-byte boundary on.
  struct Edges {
    uint32_t off;        // bytes from the grid to the row
    int head, tail;      // elements [0, head) and [tail, width)
  };
  __device__ __forceinline__ Edges edges(const T* p) const {
    const uint32_t lo = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
    Edges e;
    e.off = lo & 15u;
    e.head = min(static_cast<int>((0u - lo & 15u) / sizeof(T)), width);
    e.tail = max(width - static_cast<int>((lo + width * static_cast<uint32_t>(sizeof(T)) & 15u) / sizeof(T)),
                 e.head);
    return e;
  }
  // This thread's column among the last ones, or one past the width.
  __device__ __forceinline__ int tail_column(const Edges& e, int tid) const {
    return e.tail + (tid - e.tail & G - 1);
  }
  __device__ __forceinline__ void fetch_edges(int tid) {
    if (LIE != Lie::any || row >= rows) return;
#pragma unroll
    for (int m = 0; m < ARRAYS; ++m) {
      const T* const p = start_of(row, m);
      const Edges e = edges(p);
      const int c = tail_column(e, tid);
      off[m] = e.off;
      mine[m] = c;
      first[m] = tid < e.head;
      if (first[m]) edge[m][0] = p[tid];
      if (c < width) edge[m][1] = p[c];
    }
  }
  __device__ __forceinline__ void send(uint32_t stage, const Place& at) {
    // bytes [from, from + bytes) of the row's place in the stage
    uint32_t from[ARRAYS], bytes[ARRAYS], all = 0;
    const T* source[ARRAYS];
#pragma unroll
    for (int m = 0; m < ARRAYS; ++m) {
      const T* const p = start_of(ahead, m);
      if (LIE == Lie::grid) {
        from[m] = 0;
        bytes[m] = width * sizeof(T);
        source[m] = p;
      } else if (LIE == Lie::shifted) {
        const int w0 = ahead < low ? 1 : 0, w1 = ahead + high < rows ? words : words - 1;
        from[m] = 16 * w0;
        bytes[m] = w1 > w0 ? 16 * (w1 - w0) : 0;
        source[m] = p - at.shift + w0 * P::E;
      } else {
        const Edges e = edges(p);
        from[m] = e.off + e.head * sizeof(T);
        bytes[m] = static_cast<uint32_t>(e.tail - e.head) * sizeof(T);
        source[m] = p + e.head;
      }
      all += bytes[m];
    }
    mbar_expect_tx(&full[stage], all);
#pragma unroll
    for (int m = 0; m < ARRAYS; ++m)
      if (bytes[m] != 0u) bulk_g2s(slot(stage, m) + from[m], source[m], bytes[m], &full[stage]);
  }
  // Called by every thread of the CTA.
  __device__ __forceinline__ void start(const Place& at) {
    if (at.tid == 0) {
      for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
      fence_mbar_init();
    }
    __syncthreads();
    if (LIE == Lie::shifted) find_edges(at);
    for (int i = 0; i < stages; ++i, ahead += step)
      if (at.tid == 0 && ahead < rows) send(i, at);
    fetch_edges(at.tid);
  }
  __device__ __forceinline__ void take(P (&p)[ARRAYS], const Place& at) {
    const uint32_t stage = n % stages;
    if (lost == 0u) {
      const uint32_t parity = (n / stages) & 1u;
      if (!(wait_ns != 0 ? mbar_wait(&full[stage], parity, wait_ns) : mbar_test(&full[stage], parity))) {
        lost = n + 1;
        atomicOr(fault, 1u);
      }
    }
#pragma unroll
    for (int m = 0; m < ARRAYS; ++m) {
      unsigned char* s = slot(stage, m);
      if (LIE == Lie::any) {
        s += off[m];
        if (first[m]) reinterpret_cast<T*>(s)[at.tid] = edge[m][0];
        if (mine[m] < width) reinterpret_cast<T*>(s)[mine[m]] = edge[m][1];
      }
      if (LIE == Lie::shifted) {
        p[m].end[0] = p[m].end[1] = from_f32<T>(0.0f);
        if (!at.idle(P::kPairs - 1)) {
          constexpr int m0 = 2 * P::kPairs - 2, m1 = m0 + 1;
          const bool has0 = at.has(m0), has1 = at.has(m1);
          const int c0 = at.column(m0), c1 = at.column(m1);
          const T* const x = reinterpret_cast<const T*>(s) + at.shift;
          if (has0) p[m].end[0] = x[c0];
          if (has1) p[m].end[1] = x[c1];
          if (row < low || row + high >= rows) {
            const T* const g = start_of(row, m);
            if (has0) p[m].end[0] = g[c0];
            if (has1) p[m].end[1] = g[c1];
          }
        }
        if (at.shift != 0) s += 16;
      }
      p[m].load(s, at);
    }
    row += step;
    fetch_edges(at.tid);
  }
  __device__ __forceinline__ void refill(const Place& at) {
    if (G == 32) __syncwarp();
    if (at.tid == 0 && ahead < rows && lost == 0u) {
      if (LIE == Lie::any) fence_proxy_async_smem();
      send(n % stages, at);
    }
    ahead += step;
    ++n;
  }
  // After a wait of the sender's that gave up, the copies that may still be on their
  // way (the newest of each stage) land before the CTA may leave.
  __device__ __forceinline__ void finish(const Place& at) {
    if (at.tid != 0 || lost == 0u) return;
    const uint32_t all = stages, sent = min(lost - 1u + all, n);
    for (uint32_t i = sent > all ? sent - all : 0; i < sent; ++i)
      mbar_wait(&full[i % all], (i / all) & 1u);
  }
};

// A group's first row: a CTA has rows that are its own number modulo `period`.
template <int GROUPS>
__device__ __forceinline__ int64_t first_row(int period, int group) {
  const int64_t b = blockIdx.x;
  return b % period + period * (b / period * GROUPS + group);
}
template <typename T>
__device__ __forceinline__ int shift_of(const T* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

template <typename T, typename W, Lie LIE, int G, int EACH>
__global__ void __launch_bounds__(kCta<G>, forward_threads(G, EACH) / kCta<G>)
ln_forward_kernel(const LayerNormArgs a) {
  using P = Piece<T, LIE, G, EACH>;
  constexpr int kPairs = P::kPairs;
  constexpr int kGroups = kCta<G> / G;
  extern __shared__ __align__(16) unsigned char s_ring[];
  __shared__ __align__(16) float s_part[2 * G / 32];
  __shared__ uint64_t s_full[kGroups][kStages];
  const int group = threadIdx.x / G, tid = threadIdx.x % G;
  GroupSum<float, G> group_sum{s_part};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t t = first_row<kGroups>(a.period, group);
  const typename P::Place at(tid, a.width, shift_of(static_cast<const T*>(a.x) + t * a.x_stride));
  using R = Rows<P, T, LIE, G, 1>;
  R rows{{static_cast<const T*>(a.x)}, {a.x_stride}, a.rows, step, t, t, a.width, a.stages,
         s_ring + group * a.stages * R::pitch_of(a.width), s_full[group], a.wait_ns, a.fault};
  rows.start(at);
  float2 w[kPairs], b[kPairs];
  load_params<W, P>(a.weight, 1.0f, at, w);
  load_params<W, P>(a.bias, 0.0f, at, b);
  const float inv_width = 1.0f / static_cast<float>(a.width);
  for (; t < a.rows; t += step) {
    P p[1];
    rows.take(p, at);
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kPairs; ++k)
      if (!at.idle(k)) sum = add2(sum, p[0].pair(k));
    const float mean = group_sum(sum.x + sum.y) * inv_width;
    rows.refill(at);
    float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      if (at.idle(k)) continue;
      const float2 d = P::inside(add2(p[0].pair(k), both(-mean)), k, at);
      sq = fma2(d, d, sq);
    }
    const float var = group_sum(sq.x + sq.y) * inv_width;
    const float rstd = inverse_root(var + a.eps);
    P::store(static_cast<T*>(a.y) + t * a.y_stride, at, [&](int k) {
      return fma2(mul2(add2(p[0].pair(k), both(-mean)), both(rstd)), w[k], b[k]);
    });
    if (tid == 0) {
      a.mean[t] = mean;
      a.rstd[t] = rstd;
    }
  }
  rows.finish(at);
}

template <typename T, typename W, Lie LIE, int G, int EACH>
__global__ void __launch_bounds__(kCta<G>, backward_threads(G, EACH) / kCta<G>)
ln_backward_kernel(const LayerNormArgs a) {
  using P = Piece<T, LIE, G, EACH>;
  constexpr int kPairs = P::kPairs;
  constexpr int kGroups = kCta<G> / G;
  extern __shared__ __align__(16) unsigned char s_ring[];
  __shared__ __align__(16) float2 s_part[2 * G / 32];
  __shared__ uint64_t s_full[kGroups][kStages];
  __shared__ float2 s_add[kGroups > 1 ? 2 * kPairs * G : 1];
  let_next_kernel_start();
  const int group = threadIdx.x / G, tid = threadIdx.x % G;
  GroupSum<float2, G> group_sum{s_part};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t t = first_row<kGroups>(a.period, group);
  const typename P::Place at(tid, a.width, shift_of(static_cast<const T*>(a.x) + t * a.x_stride));
  using R = Rows<P, T, LIE, G, 2>;
  R rows{{static_cast<const T*>(a.x), static_cast<const T*>(a.dy)}, {a.x_stride, a.dy_stride},
         a.rows, step, t, t, a.width, a.stages,
         s_ring + group * a.stages * 2 * R::pitch_of(a.width), s_full[group], a.wait_ns, a.fault};
  rows.start(at);
  float2 w[kPairs], gw[kPairs], gb[kPairs];
  load_params<W, P>(a.weight, 1.0f, at, w);
#pragma unroll
  for (int k = 0; k < kPairs; ++k) gw[k] = gb[k] = make_float2(0.0f, 0.0f);
  const float inv_width = 1.0f / static_cast<float>(a.width);
  float next_mean = 0.0f, next_rstd = 0.0f;
  if (t < a.rows) {
    next_mean = a.mean[t];
    next_rstd = a.rstd[t];
  }
  for (; t < a.rows; t += step) {
    const float mean = next_mean, rstd = next_rstd;
    if (t + step < a.rows) {
      next_mean = a.mean[t + step];
      next_rstd = a.rstd[t + step];
    }
    P p[2];
    rows.take(p, at);
    // xhat = (x - mean) rstd; outside the row dy is 0, so nothing is added there
    const float2 m = both(-mean), r = both(rstd);
    float2 sum1 = make_float2(0.0f, 0.0f), sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      if (at.idle(k)) continue;
      const float2 g = p[1].pair(k), h = mul2(add2(p[0].pair(k), m), r), wg = mul2(g, w[k]);
      sum1 = add2(sum1, wg);
      sum2 = fma2(wg, h, sum2);
      if (sums_columns(G)) {
        gw[k] = fma2(g, h, gw[k]);
        gb[k] = add2(gb[k], g);
      }
    }
    const float2 s = group_sum(make_float2(sum1.x + sum1.y, sum2.x + sum2.y));
    rows.refill(at);
    // dx = rstd w dy - rstd m1 - (rstd m2) xhat
    const float2 c1 = both(-rstd * (s.x * inv_width)), c2 = both(-rstd * (s.y * inv_width));
    P::store(static_cast<T*>(a.dx) + t * a.dx_stride, at, [&](int k) {
      const float2 h = mul2(add2(p[0].pair(k), m), r);
      return fma2(mul2(p[1].pair(k), w[k]), r, fma2(h, c2, c1));
    });
  }
  rows.finish(at);
  if (!sums_columns(G) || a.partial == nullptr) return;
  // the CTA's groups, in their order
  for (int g = 1; g < kGroups; ++g) {
    __syncthreads();
    if (group == g) {
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        s_add[(2 * k) * G + tid] = gw[k];
        s_add[(2 * k + 1) * G + tid] = gb[k];
      }
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        gw[k] = add2(gw[k], s_add[(2 * k) * G + tid]);
        gb[k] = add2(gb[k], s_add[(2 * k + 1) * G + tid]);
      }
    }
  }
  if (group != 0) return;
  wait_for_previous_kernel();          // which may have left sums to add to
  float* const pw = a.partial + static_cast<int64_t>(blockIdx.x) * a.width;
  float* const pb = pw + static_cast<int64_t>(a.parts) * a.width;
  auto put = [&](float* p, float x) { *p = a.add != 0 ? *p + x : x; };
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    if (at.has(2 * k)) {
      put(pw + at.column(2 * k), gw[k].x);
      put(pb + at.column(2 * k), gb[k].x);
    }
    if (at.has(2 * k + 1)) {
      put(pw + at.column(2 * k + 1), gw[k].y);
      put(pb + at.column(2 * k + 1), gb[k].y);
    }
  }
}

// dw (blockIdx.y 0) and db (1): the CTAs' column sums, 32 columns per CTA, the
// parts split over 32 rows of threads and those joined in order.
constexpr int kTile = 32;
template <typename W>
__global__ void __launch_bounds__(kTile * kTile) ln_reduce_kernel(const LayerNormArgs a) {
  __shared__ float s_sum[kTile][kTile + 1];
  wait_for_previous_kernel();
  const int col = threadIdx.x % kTile, row = threadIdx.x / kTile;
  const int j = blockIdx.x * kTile + col;
  void* const out = blockIdx.y == 0 ? a.dweight : a.dbias;
  if (out == nullptr) return;
  const float* const p = a.partial + static_cast<int64_t>(blockIdx.y) * a.parts * a.width;
  float t = 0.0f;
  if (j < a.width) {
#pragma unroll 4
    for (int i = row; i < a.parts; i += kTile) t += __ldcg(p + static_cast<int64_t>(i) * a.width + j);
  }
  s_sum[row][col] = t;
  __syncthreads();
  // a warp per column: 32 sums in a fixed tree
  t = s_sum[col][row];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
  const int jt = blockIdx.x * kTile + row;
  if (col == 0 && jt < a.width) static_cast<W*>(out)[jt] = from_f32<W>(t);
}

// ---- rows wider than the registers of a group
//
// A CTA takes a row, its first kKeep words per thread in registers and the rest
// read again (from L1 and L2) for each pass over it.  Column sums of rows of more
// than 8192 columns are a kernel of their own, which reads x and dy once more.

constexpr int kWideThreads = 1024;
constexpr int kKeep = 4;

// Words of E elements of a row, E 1 where it is off the 16-byte grid.
template <typename T, bool VEC>
struct WideRow {
  static constexpr int E = VEC ? 16 / sizeof(T) : 1;
  using Raw = typename std::conditional<VEC, uint4, T>::type;
  const Raw* p;
  Raw keep[kKeep];
  __device__ __forceinline__ WideRow(const T* row, int words) : p(reinterpret_cast<const Raw*>(row)) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (static_cast<int>(threadIdx.x) + i * kWideThreads < words)
        keep[i] = p[threadIdx.x + i * kWideThreads];
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&x)[E]) {
    if constexpr (!VEC) {
      x[0] = to_f32(r);
    } else if constexpr (sizeof(T) == 4) {
      x[0] = __uint_as_float(r.x);
      x[1] = __uint_as_float(r.y);
      x[2] = __uint_as_float(r.z);
      x[3] = __uint_as_float(r.w);
    } else {
      const uint32_t v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_pair<T>(v[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  static __device__ __forceinline__ void store(T* row, int word, const float (&x)[E]) {
    alignas(16) T out[E];
#pragma unroll
    for (int i = 0; i < E; ++i) out[i] = from_f32<T>(x[i]);
    reinterpret_cast<Raw*>(row)[word] = *reinterpret_cast<const Raw*>(out);
  }
};

// E consecutive elements of a parameter from column j on (a multiple of E), in
// 16-byte loads where it lies on the grid: loaded singly, each warp's loads
// touch a sector per lane, and 8000 x 12288 bf16 took 294 us forward.
template <typename W, int E>
__device__ __forceinline__ void param_word(const void* p, int j, float none, float (&out)[E]) {
  constexpr int kPer = 16 / sizeof(W);
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = none;
  } else if (E % kPer == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0u) {
#pragma unroll
    for (int i = 0; i < E / kPer; ++i) {
      const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const W*>(p) + j) + i);
      float x[kPer];
      WideRow<W, true>::widen(r, x);
#pragma unroll
      for (int e = 0; e < kPer; ++e) out[i * kPer + e] = x[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = to_f32(static_cast<const W*>(p)[j + e]);
  }
}

// f(word index, i) for every word of this thread; i < kKeep: it is in `keep`.
template <typename F>
__device__ __forceinline__ void wide_words(int words, F f) {
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (static_cast<int>(threadIdx.x) + i * kWideThreads < words)
      f(static_cast<int>(threadIdx.x) + i * kWideThreads, i);
  for (int w = threadIdx.x + kKeep * kWideThreads; w < words; w += kWideThreads) f(w, kKeep);
}

template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kWideThreads) ln_forward_wide_kernel(const LayerNormArgs a) {
  __shared__ float s_warp[kWideThreads / 32];
  using Row = WideRow<T, VEC>;
  constexpr int E = Row::E;
  const int words = a.width / E;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const Row x(static_cast<const T*>(a.x) + t * a.x_stride, words);
    T* const y = static_cast<T*>(a.y) + t * a.y_stride;
    auto get = [&](int w, int i, float (&v)[E]) { Row::widen(i < kKeep ? x.keep[i] : x.p[w], v); };
    float sum = 0.0f;
    wide_words(words, [&](int w, int i) {
      float v[E];
      get(w, i, v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += v[e];
    });
    const float mean = block_sum<kWideThreads>(sum, s_warp) / a.width;
    float sq = 0.0f;
    wide_words(words, [&](int w, int i) {
      float v[E];
      get(w, i, v);
#pragma unroll
      for (int e = 0; e < E; ++e) sq = fmaf(v[e] - mean, v[e] - mean, sq);
    });
    const float rstd = inverse_root(block_sum<kWideThreads>(sq, s_warp) / a.width + a.eps);
    wide_words(words, [&](int w, int i) {
      float v[E], weight[E], bias[E];
      get(w, i, v);
      param_word<W, E>(a.weight, w * E, 1.0f, weight);
      param_word<W, E>(a.bias, w * E, 0.0f, bias);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = fmaf((v[e] - mean) * rstd, weight[e], bias[e]);
      Row::store(y, w, v);
    });
    if (threadIdx.x == 0) {
      a.mean[t] = mean;
      a.rstd[t] = rstd;
    }
  }
}

template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kWideThreads) ln_backward_wide_kernel(const LayerNormArgs a) {
  __shared__ float s_warp[kWideThreads / 32];
  using Row = WideRow<T, VEC>;
  constexpr int E = Row::E;
  const int words = a.width / E;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const Row x(static_cast<const T*>(a.x) + t * a.x_stride, words);
    const Row dy(static_cast<const T*>(a.dy) + t * a.dy_stride, words);
    T* const dx = static_cast<T*>(a.dx) + t * a.dx_stride;
    const float mean = a.mean[t], rstd = a.rstd[t];
    // xhat and w dy of a word
    auto get = [&](int w, int i, float (&h)[E], float (&g)[E]) {
      Row::widen(i < kKeep ? x.keep[i] : x.p[w], h);
      Row::widen(i < kKeep ? dy.keep[i] : dy.p[w], g);
      float weight[E];
      param_word<W, E>(a.weight, w * E, 1.0f, weight);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        h[e] = (h[e] - mean) * rstd;
        g[e] *= weight[e];
      }
    };
    float s1 = 0.0f, s2 = 0.0f;
    wide_words(words, [&](int w, int i) {
      float h[E], g[E];
      get(w, i, h, g);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        s1 += g[e];
        s2 = fmaf(g[e], h[e], s2);
      }
    });
    const float m1 = block_sum<kWideThreads>(s1, s_warp) / a.width;
    const float m2 = block_sum<kWideThreads>(s2, s_warp) / a.width;
    wide_words(words, [&](int w, int i) {
      float h[E], g[E];
      get(w, i, h, g);
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = rstd * (g[e] - m1 - h[e] * m2);
      Row::store(dx, w, g);
    });
  }
}

// Column sums over the rows blockIdx.y, blockIdx.y + parts, ...; a thread has one
// word of columns.  The wider the rows, the fewer the parts of one wave of CTAs, and
// the longer a part's sum (32768 rows of 65537 columns: 16384 terms).  So it goes to
// memory every kRun rows, and an error is at most kRun + terms / kRun units.
constexpr int kColumnThreads = 256;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kColumnThreads) ln_columns_wide_kernel(const LayerNormArgs a) {
  using Row = WideRow<T, VEC>;
  constexpr int E = Row::E;
  constexpr int kRows = 4;               // loads of as many rows under way
  constexpr int kRun = 256;
  const int w = blockIdx.x * kColumnThreads + threadIdx.x;
  if (w * E >= a.width) return;
  float gw[E], gb[E];
#pragma unroll
  for (int e = 0; e < E; ++e) gw[e] = gb[e] = 0.0f;
  float* const pw = a.partial + static_cast<int64_t>(blockIdx.y) * a.width + w * E;
  float* const pb = pw + static_cast<int64_t>(a.parts) * a.width;
  int run = 0;
  bool first = true;
  auto put = [&] {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      pw[e] = first ? gw[e] : pw[e] + gw[e];
      pb[e] = first ? gb[e] : pb[e] + gb[e];
      gw[e] = gb[e] = 0.0f;
    }
    first = false;
  };
  for (int64_t t0 = blockIdx.y; t0 < a.rows; t0 += static_cast<int64_t>(kRows) * a.parts) {
    if (++run > kRun / kRows) {
      put();
      run = 1;
    }
    typename Row::Raw x[kRows], g[kRows];
    float mean[kRows], rstd[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t t = t0 + static_cast<int64_t>(u) * a.parts;
      if (t >= a.rows) break;
      x[u] = reinterpret_cast<const typename Row::Raw*>(static_cast<const T*>(a.x) + t * a.x_stride)[w];
      g[u] = reinterpret_cast<const typename Row::Raw*>(static_cast<const T*>(a.dy) + t * a.dy_stride)[w];
      mean[u] = a.mean[t];
      rstd[u] = a.rstd[t];
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (t0 + static_cast<int64_t>(u) * a.parts >= a.rows) break;
      float h[E], d[E];
      Row::widen(x[u], h);
      Row::widen(g[u], d);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        gw[e] = fmaf(d[e], (h[e] - mean[u]) * rstd[u], gw[e]);
        gb[e] += d[e];
      }
    }
  }
  put();
}

// ---- launches

int64_t at_most(int64_t n, int64_t most) { return n < most ? n : most; }

// Wider rows have their column sums taken by ln_columns_wide_kernel, by CTAs of
// kColumnThreads words of `each` elements (at most 8), in this many parts.
constexpr int kOwnColumns = 512 * 16;
int wide_columns(int32_t width, int each) {
  return (width / each + kColumnThreads - 1) / kColumnThreads;
}
int64_t wide_parts(int columns, int sms) {
  const int64_t most = static_cast<int64_t>(kNormPartsPerSm) * sms;
  return columns < most ? most / columns : 1;
}

// Rows on their way per group, as many as fit beside the other resident CTAs.
template <int G>
int stages_for(int64_t row_bytes, int per_sm) {
  const int64_t fit = kSmemPerSm / per_sm / (kCta<G> / G) / row_bytes;
  return static_cast<int>(fit < 1 ? 1 : (fit < kStages ? fit : kStages));
}

// CTAs of a launch: as many as there are rows for, at most what is resident; a
// multiple of the period.
template <int GROUPS>
int ctas_for(const LayerNormArgs& a, int64_t resident) {
  const int64_t need = (a.rows + GROUPS - 1) / GROUPS + a.period - 1;
  return static_cast<int>(at_most(need, resident) / a.period * a.period);
}

template <typename T, typename W, Lie LIE, int G, int EACH>
int forward_group(LayerNormArgs a, int sms, cudaStream_t s) {
  constexpr int kGroups = kCta<G> / G, kPerSm = forward_threads(G, EACH) / kCta<G>;
  const int ctas = ctas_for<kGroups>(a, static_cast<int64_t>(kPerSm) * sms);
  const int64_t row = Rows<Piece<T, LIE, G, EACH>, T, LIE, G, 1>::pitch_of(a.width);
  a.stages = stages_for<G>(row, kPerSm);
  ln_forward_kernel<T, W, LIE, G, EACH><<<ctas, kCta<G>, kGroups * a.stages * row, s>>>(a);
  return ctas;
}

template <typename T, typename W, Lie LIE, int G, int EACH>
int backward_group(LayerNormArgs a, int sms, cudaStream_t s) {
  constexpr int kGroups = kCta<G> / G, kPerSm = backward_threads(G, EACH) / kCta<G>;
  static_assert(kPerSm <= kNormPartsPerSm, "partial sums of every CTA");
  const int ctas = ctas_for<kGroups>(a, static_cast<int64_t>(kPerSm) * sms);
  a.parts = ctas;
  if (a.dweight == nullptr && a.dbias == nullptr) a.partial = nullptr;
  const int64_t row = 2 * static_cast<int64_t>(
                              Rows<Piece<T, LIE, G, EACH>, T, LIE, G, 2>::pitch_of(a.width));
  a.stages = stages_for<G>(row, kPerSm);
  // a launch for every kRunRows rows of a group, so that no column sum in registers
  // has more terms: an error is then at most kRunRows + launches units
  const int64_t rows = a.rows;
  const int64_t runs = a.partial == nullptr || !sums_columns(G)
                           ? 1
                           : (rows - 1) / (static_cast<int64_t>(kRunRows) * kGroups * ctas) + 1;
  // the same number of rows each, and their shift on the 16-byte grid
  const int64_t each = ((rows - 1) / runs / a.period + 1) * a.period;
  const LayerNormArgs all = a;
  for (int64_t from = 0; from < rows; from += each) {
    a.x = static_cast<const T*>(all.x) + from * a.x_stride;
    a.dy = static_cast<const T*>(all.dy) + from * a.dy_stride;
    a.dx = static_cast<T*>(all.dx) + from * a.dx_stride;
    a.mean = all.mean + from;
    a.rstd = all.rstd + from;
    a.rows = at_most(rows - from, each);
    a.add = from > 0;
    // the CTAs of a launch come up as those of the one before leave (four launches
    // that did not took 1029 us where these take 1002)
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(static_cast<unsigned>(ctas));
    c.blockDim = dim3(kCta<G>);
    c.dynamicSmemBytes = kGroups * a.stages * row;
    c.stream = s;
    c.attrs = &attr;
    c.numAttrs = a.add != 0 ? early_start(&attr) : 0;
    cudaLaunchKernelEx(&c, ln_backward_kernel<T, W, LIE, G, EACH>, a);
  }
  return ctas;
}

// The group of a width.
#define ADAMW_LN_GROUPS(call)           \
  (a.width <= 512    ? call(32, 16)     \
   : a.width <= 1024 ? call(32, 32)     \
   : a.width <= 2048 ? call(128, 16)    \
   : a.width <= 4096 ? call(256, 16)    \
   : a.width <= 8192 ? call(512, 16)    \
                     : call(1024, 16))

// Lets the row kernels of one width use the shared memory of their stages.
template <typename T, typename W, Lie LIE, int G, int EACH>
cudaError_t prepare_group() {
  const cudaError_t e = cudaFuncSetAttribute(ln_forward_kernel<T, W, LIE, G, EACH>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(ln_backward_kernel<T, W, LIE, G, EACH>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
}
template <typename T, typename W, Lie LIE>
cudaError_t prepare_lie(int32_t width) {
  LayerNormArgs a{};
  a.width = width;
#define ADAMW_LN_CALL(G, EACH) prepare_group<T, W, LIE, G, EACH>()
  return ADAMW_LN_GROUPS(ADAMW_LN_CALL);
#undef ADAMW_LN_CALL
}
template <typename T, typename W>
cudaError_t prepare_width(int32_t width) {
  cudaError_t e = prepare_lie<T, W, Lie::grid>(width);
  if (e == cudaSuccess) e = prepare_lie<T, W, Lie::shifted>(width);
  if (e == cudaSuccess) e = prepare_lie<T, W, Lie::any>(width);
  return e;
}

// How a call's matrices lie, of `width` columns and elements of `size` bytes.
struct Layout {
  uintptr_t at;
  int64_t stride;        // bytes
  bool grid, same = true;
  Layout(const void* p, int64_t stride_, int64_t width, int64_t size)
      : at(reinterpret_cast<uintptr_t>(p)), stride(stride_ * size),
        grid(at % 16 == 0 && stride % 16 == 0 && width * size % 16 == 0) {}
  void join(const void* p, int64_t stride_, int64_t size) {
    same = same && (reinterpret_cast<uintptr_t>(p) - at) % 16 == 0 && (stride_ * size - stride) % 16 == 0;
  }
  Lie lie() const { return !same ? Lie::any : (grid ? Lie::grid : Lie::shifted); }
  int period() const {
    int p = 1;
    while (lie() == Lie::shifted && stride * p % 16 != 0) p *= 2;
    return p;
  }
};

#define ADAMW_LN_FORWARD(G, EACH)                                                     \
  (lie == Lie::grid      ? forward_group<T, W, Lie::grid, G, EACH>(a, sms, s)         \
   : lie == Lie::shifted ? forward_group<T, W, Lie::shifted, G, EACH>(a, sms, s)      \
                         : forward_group<T, W, Lie::any, G, EACH>(a, sms, s))
#define ADAMW_LN_BACKWARD(G, EACH)                                                    \
  (lie == Lie::grid      ? backward_group<T, W, Lie::grid, G, EACH>(a, sms, s)        \
   : lie == Lie::shifted ? backward_group<T, W, Lie::shifted, G, EACH>(a, sms, s)     \
                         : backward_group<T, W, Lie::any, G, EACH>(a, sms, s))

template <typename T, typename W>
cudaError_t forward(LayerNormArgs a, int sms, cudaStream_t s) {
  Layout lay(a.x, a.x_stride, a.width, sizeof(T));
  lay.join(a.y, a.y_stride, sizeof(T));
  const Lie lie = lay.lie();
  a.period = lay.period();
  if (a.width > kMaxWidth) {
    const int ctas = static_cast<int>(at_most(a.rows, 2LL * sms));
    if (lie == Lie::grid) ln_forward_wide_kernel<T, W, true><<<ctas, kWideThreads, 0, s>>>(a);
    else ln_forward_wide_kernel<T, W, false><<<ctas, kWideThreads, 0, s>>>(a);
  } else {
    ADAMW_LN_GROUPS(ADAMW_LN_FORWARD);
  }
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t backward(LayerNormArgs a, int sms, cudaStream_t s) {
  Layout lay(a.x, a.x_stride, a.width, sizeof(T));
  lay.join(a.dy, a.dy_stride, sizeof(T));
  lay.join(a.dx, a.dx_stride, sizeof(T));
  const Lie lie = lay.lie();
  a.period = lay.period();
  if (a.rows == 0) {
    a.parts = 0;
  } else {
    const bool own_columns = a.width > kOwnColumns;
    if (own_columns && (a.dweight != nullptr || a.dbias != nullptr)) {
      // before the rows: dx may be dy.  One wave of CTAs.
      const bool vec = lie == Lie::grid;
      const int columns = wide_columns(a.width, vec ? 16 / static_cast<int>(sizeof(T)) : 1);
      a.parts = static_cast<int32_t>(at_most(a.rows, wide_parts(columns, sms)));
      const dim3 grid(columns, a.parts);
      if (vec) ln_columns_wide_kernel<T, true><<<grid, kColumnThreads, 0, s>>>(a);
      else ln_columns_wide_kernel<T, false><<<grid, kColumnThreads, 0, s>>>(a);
    }
    if (a.width > kMaxWidth) {
      const int ctas = static_cast<int>(at_most(a.rows, 2LL * sms));
      if (lie == Lie::grid) ln_backward_wide_kernel<T, W, true><<<ctas, kWideThreads, 0, s>>>(a);
      else ln_backward_wide_kernel<T, W, false><<<ctas, kWideThreads, 0, s>>>(a);
    } else {
      const int ctas = ADAMW_LN_GROUPS(ADAMW_LN_BACKWARD);
      if (!own_columns) a.parts = ctas;
    }
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (a.dweight == nullptr && a.dbias == nullptr)) return e;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>((a.width + kTile - 1) / kTile), 2);
  c.blockDim = dim3(kTile * kTile);
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = early_start(&attr);
  return cudaLaunchKernelEx(&c, ln_reduce_kernel<W>, a);
}

}  // namespace

int64_t norm_parts(int32_t width, int sms) {
  return width > kOwnColumns ? wide_parts(wide_columns(width, 8), sms) : int64_t{kNormPartsPerSm} * sms;
}

cudaError_t prepare_layer_norm(int32_t width) {
  cudaError_t e = prepare_width<float, float>(width);
  if (e == cudaSuccess) e = prepare_width<__half, float>(width);
  if (e == cudaSuccess) e = prepare_width<__half, __half>(width);
  if (e == cudaSuccess) e = prepare_width<__nv_bfloat16, float>(width);
  if (e == cudaSuccess) e = prepare_width<__nv_bfloat16, __nv_bfloat16>(width);
  return e;
}

#define ADAMW_LN_DISPATCH(fn)                                                     \
  if (dt == ADAMW_F32 && wdt == ADAMW_F32) return fn<float, float>(a, sms, s);    \
  if (dt == ADAMW_F16 && wdt == ADAMW_F32) return fn<__half, float>(a, sms, s);   \
  if (dt == ADAMW_F16 && wdt == ADAMW_F16) return fn<__half, __half>(a, sms, s);  \
  if (dt == ADAMW_BF16 && wdt == ADAMW_F32)                                       \
    return fn<__nv_bfloat16, float>(a, sms, s);                                   \
  if (dt == ADAMW_BF16 && wdt == ADAMW_BF16)                                      \
    return fn<__nv_bfloat16, __nv_bfloat16>(a, sms, s);                           \
  return cudaErrorInvalidValue;

cudaError_t launch_layer_norm_forward(adamw_dtype dt, adamw_dtype wdt, const LayerNormArgs& a,
                                      int sms, cudaStream_t s) {
  ADAMW_LN_DISPATCH(forward)
}
cudaError_t launch_layer_norm_backward(adamw_dtype dt, adamw_dtype wdt, const LayerNormArgs& a,
                                       int sms, cudaStream_t s) {
  ADAMW_LN_DISPATCH(backward)
}
#undef ADAMW_LN_DISPATCH
#undef ADAMW_LN_GROUPS
#undef ADAMW_LN_FORWARD
#undef ADAMW_LN_BACKWARD

}  // namespace adamw
