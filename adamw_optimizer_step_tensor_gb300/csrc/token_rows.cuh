// token_rows.cuh -- what the two row kernels of the token losses share: passes,
// and how a row is cut into 16-byte words.
#pragma once

#include "token_math.cuh"

namespace adamw {

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

__host__ __device__ constexpr bool sums(int pass) { return pass != kPassGrad; }
// Vocabularies of up to this many bytes per row are held in registers
// (token_loss_small.cu).
constexpr int kSmallVocabBytes = 65536;
template <typename T>
cudaError_t prepare_small_vocab(int sms, int (&ctas)[kSmallGroups]);
template <typename T>
cudaError_t launch_small_vocab(Pass pass, const LossArgs& a, bool same_grid, const int (&ctas)[kSmallGroups],
                               cudaStream_t s);

namespace {

constexpr int kPieceWords = 1024;

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
    // ranks is a power of two; shares start on 128-byte steps of the words
    const int64_t per = (((all + ranks - 1) >> (__ffs(ranks) - 1)) + 7) & ~static_cast<int64_t>(7);
    const int64_t from = min(per * rank, all);
    words = static_cast<int>(min(per, all - from));
    pieces = (words + kPieceWords - 1) / kPieceWords;
    base = reinterpret_cast<const unsigned char*>(lo16) + from * 16;
    first = head + from * kPerWord<T>;
  }
  __device__ __forceinline__ int piece_words(int j) const {
    return min(kPieceWords, words - j * kPieceWords);
  }
};

// The element off the 16-byte grid that lane `lane` looks after, or -1: the
// row's first elements on lanes 0.., its last on lanes 8...
template <typename T>
__device__ __forceinline__ int ragged_element(const RowShare<T>& share, int vocab, int lane) {
  if (lane < 8) return lane < share.head ? lane : -1;
  return lane < 16 && lane - 8 < share.tail ? vocab - share.tail + lane - 8 : -1;
}

// ---- far rows (see token_math.cuh)

// A word's sum of 2^((z - m) k).
template <typename T>
__device__ __forceinline__ float far_word(const uint4& w, float m, float k, float k_lo) {
  float2 x[kPerWord<T> / 2];
  unpack<T>(w, x);
  float t = 0.0f;
#pragma unroll
  for (int j = 0; j < kPerWord<T> / 2; ++j)
    t += far_power(half_below(x[j].x, m), k, k_lo) + far_power(half_below(x[j].y, m), k, k_lo);
  return t;
}
constexpr int kFarLoads = 4;             // words on their way per thread
template <typename T>
__device__ __forceinline__ void far_load(const uint4* w, int i, int threads, int words,
                                         uint4 (&v)[kFarLoads]) {
#pragma unroll
  for (int u = 0; u < kFarLoads; ++u)
    v[u] = i + u * threads < words ? w[i + u * threads] : lowest_word<T>();
}
// Of the logits that thread `tid` of `threads` looks after, the largest (NaN
// ignored), and the sum of 2^((z - m) k).
template <typename T>
__device__ __forceinline__ float far_max(const T* z, int vocab, uint32_t rank, uint32_t ranks, int tid,
                                         int threads) {
  const RowShare<T> share(z, vocab, rank, ranks);
  const uint4* const w = reinterpret_cast<const uint4*>(share.base);
  float m = -INFINITY;
#pragma unroll 1
  for (int i = tid; i < share.words; i += kFarLoads * threads) {
    uint4 v[kFarLoads];
    far_load<T>(w, i, threads, share.words, v);
    m = fmaxf(m, words_max<T, kFarLoads>(v));
  }
  const int e = rank == 0 && tid < 16 ? ragged_element(share, vocab, tid) : -1;
  return e >= 0 ? fmaxf(m, to_f32(z[e])) : m;
}
template <typename T>
__device__ __forceinline__ float far_sum(const T* z, int vocab, uint32_t rank, uint32_t ranks, int tid,
                                         int threads, float m, float k, float k_lo) {
  const RowShare<T> share(z, vocab, rank, ranks);
  const uint4* const w = reinterpret_cast<const uint4*>(share.base);
  m = fmaxf(m, -3.40282347e38f);        // -inf logits alone add nothing
  float s = 0.0f;
#pragma unroll 1
  for (int i = tid; i < share.words; i += kFarLoads * threads) {
    uint4 v[kFarLoads];
    far_load<T>(w, i, threads, share.words, v);
#pragma unroll
    for (int u = 0; u < kFarLoads; ++u) s += far_word<T>(v[u], m, k, k_lo);
  }
  const int e = rank == 0 && tid < 16 ? ragged_element(share, vocab, tid) : -1;
  return e >= 0 ? s + far_power(half_below(to_f32(z[e]), m), k, k_lo) : s;
}
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

}  // namespace
}  // namespace adamw
