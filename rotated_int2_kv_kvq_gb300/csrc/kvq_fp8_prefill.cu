// kvq_fp8_prefill.cu — causal attention of each sequence's new tokens over the 8-bit paged cache,
// all of it or a sliding window and the first tokens.
//
// Row r of sequence b sits at position p and attends to the positions t <= p with t > p - window
// or t < sinks (window 0: all).  The kernel is that of kvq_prefill.cu: the producers turn codes
// into bf16 operands, which hold an entry code * 2^e exactly, and everything behind them is the
// BF16 cache's path (query, weights and sums).  Whole key tiles that no row of a row tile sees are
// left out of the line of work, so a window costs its own length.
#include "kvq_internal.cuh"

namespace kvq {
namespace {

// Registers a thread at launch; the parts after the roles part come out of it.
constexpr int kRegLaunch = 128;

}  // namespace
}  // namespace kvq

#include "kvq_prefill.cuh"

namespace kvq {

cudaError_t launch_fp8_prefill(const PrefillArgs& a, int num_sms, cudaStream_t st) {
  return launch<false, true>(a, num_sms, st);
}

}  // namespace kvq
