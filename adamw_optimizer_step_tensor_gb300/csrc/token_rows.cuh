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

}  // namespace
}  // namespace adamw
