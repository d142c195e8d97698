// kvq_fp8_prefill.cu — causal attention of each sequence's new tokens over the 8-bit paged cache,
// all of it or a sliding window and the first tokens.
//
// Row r of sequence b sits at position p and attends to the positions t <= p with t > p - window
// or t < sinks (window 0: all).  An entry is code * 2^e with one e for a page's keys and one for its
// values, so that
//   logit_t = scale 2^x 2^ek (q~ . code_t),   out = sum_t w_t (code_t 2^ev) / sum_t w_t,
// with q = q~ 2^x.  The kernel is that of kvq_prefill.cu (its roles, its line of work and its joining
// of cut items), with these differences:
//   keys    : the codes are the tensor core's 8-bit operand as they are; producers only move them
//             from the record's order into rows.  The query is two 8-bit parts of 4 bits of mantissa
//             each, two products of half a 16-bit one's time.  A page's 2^ek goes into its columns'
//             scores: eight columns' factors a tile in place of one.
//   values  : fp16, code 2^ev exactly, by bit moves and one product a pair, because their sum spans
//             pages; weights are fp16 then.  A tile with a page that fp16 does not hold (2^ev outside
//             2^-21 .. 2^1) is bf16, and so are its weights, whose sum is that of the rounded ones.
//   windows : whole key tiles that no row of a row tile sees are left out of the line of work, so a
//             window costs its own length; partly hidden tiles are masked in TMEM first.
//   NaN     : a value that is not finite is stored as zero and noted, and spoils the rows that see it.
//   queries : the next item's rows come into shared memory by bulk copies as soon as the
//             last product has read this one's, and are made operands from there.
//   registers: 176 / 96 / 64 a thread (softmax, producers, issue), with the issuing warp's loop apart
//             from the scheduler's: next to this much shared memory L1 holds nearly nothing, and a
//             spilled register is a round trip to L2.  Nothing is spilled.
//
// Measured (32 query, 8 KV heads): 4096 new tokens at 32K 1535 to 1590 us from one
// GPU to another, at the power limit (1320 TFLOP/s).  The products alone take 1086 at
// the rate of a large library product, 1218 at the rate that one keeps up; the BF16 cache takes 1800,
// the INT2 cache 1450.  A CTA's time for a key tile is 2.3 us: 1.35 of a row tile's softmax and 1.0
// that it waits for scores behind the other row tile's (timed with bf16 weights), so the chain scores ->
// softmax -> weights -> output bounds it, as it does the other caches'.  Spills and instructions count
// most.  With bf16 weights: registers 168 / 112 / 64 with 68 bytes of the softmax's spilled 1585,
// 168 / 120 / 56 with the issuing warp's 1940, 160 / 128 / 64 2270.  With fp16 ones: their sum in two
// chains, 96 bytes of the softmax's spilled, 2068; what bf16 tiles need unrolled beside it 1565 to 1595,
// windows 245, drafts 67.  Where every tile is bf16: 1755, 251 and 66; values above 57344, or not finite,
// a word at a time: 3500, 347 and 119.
// A prompt of 8191 tokens with a window of 1024: 236 to 239 us for products of 68.  Ten key tiles an item where
// eight hold its window, a third of them partly hidden (2.3 us of softmax for 1.4); and 9 us an item,
// seven items a CTA, for its queries (3), the first scores (1.5), results (2.4) and the wait for the
// other row tile's.  Queries by plain loads when the item begins: 273.
// Eight drafts of five tokens at 8K: 64 us, 27 key tiles a CTA, at the pace of the producers' loads: two
// pages a warp, a tile ahead (pages from L2 53; without the values' conversion 57, the keys' copies 59,
// both 51; without the products 62, the softmax 61; without the four of them 48).
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
