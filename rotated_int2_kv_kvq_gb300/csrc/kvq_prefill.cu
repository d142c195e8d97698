// kvq_prefill.cu — causal attention of each sequence's new tokens over its paged
// cache (INT2 or BF16), on the fifth-generation tensor cores.
//
// Row r of sequence b (len = seq_lens[b], n_b new tokens) sits at position
// p = len - n_b + r and attends to positions [0, p]:
//   out = softmax(sm_scale * q . k_t, t <= p) . v_t
// with k_t, v_t the cache's entries; for the INT2 cache the query is first
// rotated by R_K and the output rotated back by R_V^T, as kvq_decode does.
//
// One CTA per SM works through (sequence, KV head, row tile) items.  A row tile
// is 256 rows (token, query head of the KV head's group): two MMA tiles of 128
// that share each key tile of 128 positions (8 pages).  Roles:
//   warps 0-3, 4-7 : softmax of the first and second 128 rows, a thread a row;
//   warps 8-11     : page producers: codes (or bf16 fragments) -> fp16 (bf16)
//                    operands in shared memory, two pages a warp, two stages;
//   warp 12        : its elected thread issues every tcgen05.mma;
//   warp 13        : one thread finds the next item while this one is worked on.
// Scores S = Q K^T and the output O live in TMEM (2 x 128 + 2 x 128 columns);
// the weights P overwrite S's columns and feed the second product from TMEM.
// While one row tile's softmax runs, the tensor core works on the other's.  An item
// of at most 128 rows has one row tile only: there both softmax groups take it, the
// even and the odd key tiles, with an O each, joined at the item's end.
//
// INT2: the two rotations are tensor-core steps of the same pipeline, with the
// rotation matrices (laid out once by kvq_set_rotation) in a stage's place of
// the pages: first S = q R_K, which the softmax threads turn into the fp16
// operand Q, and at an item's end out = o R_V^T from the normalised o.
//
// All key tiles of all items form one line of work, cut into equal ranges, one
// per CTA: ragged batches, a single long chunk and a few decode tokens all fill
// the GPU without a choice of split counts.  An item that a range border cuts
// leaves partial (max, sum, O) states, joined by the combine kernel.
//
// Measured (32 query, 8 KV heads): 4096 new tokens at 32K, INT2: 1490 us in long runs, at the
// power limit (1390 TFLOP/s, 75 % of the bf16 rate of a large library product on the same
// GPU, 1865), 1442 us in short ones; the products alone, with the softmax and the unpacking
// left out, take 1091 us at the power limit.
// What is left is the chain S -> softmax -> P -> O of a row tile, of which two fit TMEM:
// tensor pipe 59 % and issue slots 58 % busy, the exponentials' unit 29 %.  Two prompts
// of 4093, BF16: 288 us.  Sixteen decode tokens beside a 1021-token chunk: 178 us, of which
// the uneven line is a part: a key tile counts one unit, though one of a one-row-tile item
// takes half as long as one of two row tiles, so the CTAs on the chunk end last.
// Eight drafts of five tokens at up to 8K: 51 us, of which the launches, the line's
// setup, the rotations and the join take about half.
// Tried and slower: half tiles of 64 columns (2045 us: such a product runs at half rate),
// producer warps for keys and values apart (1759), eight producer warps (1844), a ring of
// raw records in shared memory (1745), no CTA-wide barrier between items (1524: spills),
// part of the exponentials as polynomials (an eighth of them: 1494).
#include "kvq_internal.cuh"

namespace kvq {
namespace {

// Registers a thread: at launch, and after the roles part (warpgroups: two softmax,
// producers, one for issue and schedule).  The parts come out of the launch's, so
// they must not add up to more, or a role would wait for ever.
constexpr int kRegLaunch = 128;

}  // namespace
}  // namespace kvq

#include "kvq_prefill.cuh"

namespace kvq {
namespace {

// ---- the rotation bank ---------------------------------------------------------------
// What kvq_set_rotation derives from R [2][Hkv][D][D]: R_V^T in fp32 (the decode's combine),
// and the prefill's operands: R_K^T as two bf16 parts (hi + lo: 16 bits of each entry) and R_V
// as fp16, each a 128 x 128 K-major operand in the swizzled layout above, row n, column k of
// head kv.  A CTA takes a 32 x 32 tile through shared memory, so that reads and writes are
// both along rows: one kernel, as many launches as before the operands (a CTA a head that read
// R_V by columns took 58 us).
__global__ void __launch_bounds__(256) rotation_bank_kernel(const float* R, int Hkv, bool identity_q,
                                                            float* RVt, uint16_t* hi, uint16_t* lo,
                                                            uint16_t* rv) {
  __shared__ float tile[32][33];
  const bool value = blockIdx.z >= static_cast<unsigned>(Hkv);
  const size_t mat = static_cast<size_t>(value ? blockIdx.z - Hkv : blockIdx.z) * kDim * kDim;
  const float* src = R + static_cast<size_t>(blockIdx.z) * kDim * kDim;
  const int bx = blockIdx.x * 32, by = blockIdx.y * 32, x = threadIdx.x;
  auto at = [&](int n, int k) {
    return mat + (k >> 6) * (kTileBytes / 4) + n * 64 + ((((k >> 3) & 7) ^ (n & 7)) << 3) + (k & 7);
  };
  for (int y = threadIdx.y; y < 32; y += 8) {
    const float e = src[(by + y) * kDim + bx + x];
    tile[y][x] = e;
    if (value) rv[at(by + y, bx + x)] = __half_as_ushort(__float2half_rn(e));
  }
  __syncthreads();
  for (int y = threadIdx.y; y < 32; y += 8) {
    const int n = bx + y, k = by + x;
    const float e = tile[x][y];                    // R[k][n]
    if (value) {
      RVt[mat + n * kDim + k] = e;
    } else {
      const float q = identity_q ? (n == k ? 1.0f : 0.0f) : e;
      const __nv_bfloat16 h = __float2bfloat16_rn(q);
      hi[at(n, k)] = __bfloat16_as_ushort(h);
      lo[at(n, k)] = __bfloat16_as_ushort(__float2bfloat16_rn(q - __bfloat162float(h)));
    }
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

PrefillWs prefill_ws_layout(int num_sms) {
  PrefillWs w;
  size_t o = 0;
  w.cuts_off = o;
  o += up256(static_cast<size_t>(num_sms) * sizeof(PrefillArgs::Cut));
  w.ml_off = o;
  o += up256(static_cast<size_t>(num_sms) * 2 * kRows * 8);
  w.part_off = o;
  o += up256(static_cast<size_t>(num_sms) * 2 * kRows * kDim * 4);
  w.total = o;
  return w;
}

cudaError_t launch_rotation_bank(const float* R, int Hkv, bool identity_q, float* RVt, uint16_t* hi,
                                 uint16_t* lo, uint16_t* rv, cudaStream_t st) {
  rotation_bank_kernel<<<dim3(kDim / 32, kDim / 32, 2 * Hkv), dim3(32, 8), 0, st>>>(R, Hkv, identity_q,
                                                                                   RVt, hi, lo, rv);
  return cudaGetLastError();
}

cudaError_t launch_prefill(const PrefillArgs& a, bool int2, int num_sms, cudaStream_t st) {
  return int2 ? launch<true>(a, num_sms, st) : launch<false>(a, num_sms, st);
}

}  // namespace kvq
