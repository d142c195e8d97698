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

constexpr int kTileKeys = 128;             // key positions per tile
constexpr int kTilePages = kTileKeys / kPage;
constexpr int kRows = 256;                 // rows per item: two MMA tiles
constexpr int kThreads = 512;
constexpr int kProdWarp0 = 8, kMmaWarp = 12, kSchedWarp = 13;
// Registers a thread: at launch, and after the roles part (warpgroups: two softmax,
// producers, one for issue and schedule).  The parts come out of the launch's, so
// they must not add up to more, or a role would wait for ever.
constexpr int kRegLaunch = 128;
template <bool INT2>
struct Regs {
  static constexpr int kSoftmax = INT2 ? 184 : 176, kProducer = INT2 ? 96 : 112, kIssue = 48;
  static_assert(2 * kSoftmax + kProducer + kIssue <= 4 * kRegLaunch, "register split");
};
constexpr int kStages = 2;
constexpr int kFlags = 4;                  // key tiles whose missing pages are kept
constexpr int kTileBytes = 128 * 128 * 2;  // one 128 x 128 16-bit operand
constexpr float kLazy = 8.0f;              // log2 growth of a row maximum before O is rescaled
// The INT2 path's weights are 2^(s - reference + kBias), up to 2^15 with a reference that lags by kLazy:
// fp16 then keeps its 11 bits down to 2^-21 of the reference (14.5 nats below it) and something down to
// 2^-32, so that a long flat tail behind one dominant key keeps its mass.  O and the sum carry the same
// factor.  Without it a tail at 2^-22.6 came out 13.7 % too large and one at 2^-25 as zero.  A smaller
// kLazy would leave more room but rescales O more often (4096 tokens at 32K: 8: 1441 us, 7: 1459,
// 6: 1487, 4: 1519; without the factor 1442).
constexpr float kBias = 15.0f - kLazy;

struct Smem {
  static constexpr int kQ = 0;                              // [2][32 KB]
  static constexpr int kK = kQ + 2 * kTileBytes;            // [stages][32 KB]
  static constexpr int kV = kK + kStages * kTileBytes;      // [stages][32 KB]
  static constexpr int kBar = kV + kStages * kTileBytes;    // mbarriers
  static constexpr int kAny = kBar + 160;                   // u8 [kFlags][4]: a producer warp has set a bit of
  static constexpr int kBad = kAny + 16;                    // u32 [kFlags][4] tokens without a valid page
  static constexpr int kPoison = kBad + 64;                 // u32 [2] first position with a NaN / Inf value
  static constexpr int kItem = kPoison + 16;                // Item [2]
  static constexpr int kScan = kItem + 128;                 // long long [16]
  static constexpr int kLine = kScan + 128;                 // Line
  static constexpr int kTmem = kLine + 48;
  static constexpr int kPair = kTmem + 16;                  // float2 [128]: a split row's scale, then (max, sum) of its odd tiles
  static constexpr int kBytes = kPair + 1024;
  static constexpr int kAlloc = kBytes + 1024;              // base rounded up to 1024
};

// barrier indices
enum { kKFull = 0, kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages, kVEmpty = kVFull + kStages,
       kSFull = kVEmpty + kStages, kPFull = kSFull + 2, kDrain = kPFull + 2, kNumBars };
static_assert(kNumBars * 8 <= 160, "barriers");

using Cut = PrefillArgs::Cut;

struct Line {               // a CTA's range of the line of work
  long long cur, end;       // its next unit, its end
  long long per;            // units per range
  long long b_first;        // first unit of sequence b
  int b;                    // the sequence of `cur` (or one before it)
};
static_assert(sizeof(Line) <= 48, "Line");

struct Item {
  int b, kv;                // sequence, KV head
  int row0;                 // first token row (in q / out) of the tile
  int tokens;               // tokens in the tile
  int pos0;                 // position of its first token
  int key_end;              // positions the tile sees: last token's position + 1 (0: none)
  int tile_begin, tiles;    // key tiles of this CTA's part
  int part;                 // partial slot, or -1 when this CTA has the whole item
  int done;                 // no item left
};
static_assert(sizeof(Item) <= 64, "two items");

// ---- tcgen05 ---------------------------------------------------------------------

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The issuing warp runs converged with warp-uniform operands (the tensor core takes
// its descriptors from uniform registers); `one` is true in its elected lane.
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(one)
      : "memory");
}
// Operand descriptors differ in their low words only (the address); the high word:
// 8-row groups 1024 bytes apart, descriptor version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                          uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(one), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                          uint32_t acc, uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(one), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void tc_ld32(uint32_t (&v)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}
// Orders the loads' registers: nothing that uses them is scheduled before the wait.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                 "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                 "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]),
                 "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                 "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]),
                 "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t (&v)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 128 columns of this thread's row.
__device__ __forceinline__ void tc_ld_row(uint32_t (&v)[4][32], uint32_t addr) {
#pragma unroll
  for (int c = 0; c < 4; ++c) tc_ld32(v[c], addr + 32 * c);
#pragma unroll
  for (int c = 0; c < 4; ++c) tc_wait_ld(v[c]);
}

// Shared-memory operand of 128 rows x 128 columns of 16 bits, K-major, as two
// 64-column halves of 128-byte rows with the 128-byte swizzle (16-byte chunk c of
// row r at chunk c ^ (r & 7)); 8-row groups 1024 bytes apart.  The low word of its
// descriptor, and what its 16-column step k adds to it.
__device__ __forceinline__ uint32_t tile_desc(uint32_t base) { return (base >> 4) | (1u << 16); }
__device__ __forceinline__ constexpr uint32_t desc_step(int k) {
  return ((k >> 2) * (kTileBytes / 2) + (k & 3) * 32) >> 4;
}
// fp32 accumulate, M = N = 128, both operands fp16 (0) or bf16 (1), K-major
constexpr uint32_t idesc_f16(int bf16) {
  return (1u << 4) | (static_cast<uint32_t>(bf16) << 7) | (static_cast<uint32_t>(bf16) << 10) |
         ((128u >> 3) << 17) | ((128u >> 4) << 24);
}

// One lane's arrival, as a predicated instruction: no branch for the warp to diverge at
// (the tcgen05 loads that follow are warp-wide).
__device__ __forceinline__ void arrive_if(uint32_t bar, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(static_cast<uint32_t>(on))
      : "memory");
}

// ---- element orders ---------------------------------------------------------------
// S = sum_d q_d k_d and O = sum_t p_t v_t do not depend on the order of d and t, so
// both follow the page record's: a producer lane's codes become whole 16-byte
// chunks, and its stores are free of bank conflicts.
//   d = 16w + 8h + 2t + e : half t >> 1, chunk 4 (t & 1) + ((2h + (w >> 2)) ^ (2 (t >> 1))),
//                           element 2 (w & 3) + e of the chunk;
//   position in the tile = 64 g + 32 pp + 16 pi + 8 th + 2t + e : row (column of S,
//                           K index of V) 64 g + 16 t + 8 pp + 4 pi + 2 th + e.
__device__ __forceinline__ constexpr int col_pos(int c) {
  return (c & 64) | ((c >> 3) & 1) << 5 | ((c >> 2) & 1) << 4 | ((c >> 1) & 1) << 3 |
         ((c >> 4) & 3) << 1 | (c & 1);
}

// ---- the line of work ---------------------------------------------------------------
// Row tiles of a sequence with n new tokens behind p0 old ones, TR tokens a tile
// (TR = 256 / G): tile k sees ceil((p0 + min((k + 1) TR, n)) / 128) key tiles, and
// counts for kItemCost units more (its queries, rotations and results: 8 us beside
// 1.4 to 1.9 us a key tile), so that ranges of many short items are not the longest.
constexpr int kItemCost = 4;
struct Seq {
  int row0, n, p0;       // first row, new tokens, position of the first
  bool ok;               // false: invalid lengths; its rows get zeros
  uint32_t bad;          // status bit of an invalid sequence, or 0
  int rts;               // row tiles
  long long units;       // of one KV head (invalid: one per row tile)
};

__device__ __forceinline__ long long half_sum(long long m) {   // sum of ceil(i / 2), i = 1 .. m
  return ((m + 1) * (m + 1)) >> 2;
}
// units of row tiles 0 .. k-1, all of them full
__device__ __forceinline__ long long units_before(const Seq& s, int k, int TR) {
  if (!s.ok) return k;
  const long long cost = static_cast<long long>(k) * kItemCost;
  if (TR == 64) {
    const long long a = (s.p0 + 63) >> 6;
    return half_sum(a + k) - half_sum(a) + cost;
  }
  const long long a = (s.p0 + 127) >> 7, kk = k;
  return a * kk + (TR >> 7) * (kk * (kk + 1) >> 1) + cost;
}
__device__ __noinline__ Seq load_seq(const PrefillArgs& a, int b, int TR) {
  Seq s;
  const int r0 = a.cu_q[b], r1 = a.cu_q[b + 1];
  const int len = a.seq_lens[b];
  s.row0 = r0;
  s.n = r1 - r0;
  s.ok = true;
  s.bad = 0;
  if (r0 < 0 || r1 < r0 || r1 > a.n) {     // not a range of rows: nothing to write
    s.n = 0;
    s.ok = false;
    s.bad = KVQ_STATUS_BAD_SEQ;
  } else if (len < s.n || len > a.max_pages * kPage) {
    s.ok = false;
    s.bad = KVQ_STATUS_BAD_SEQLEN;
  }
  s.p0 = s.ok ? len - s.n : 0;
  s.rts = (s.n + TR - 1) / TR;
  s.units = s.rts == 0 ? 0
            : s.ok     ? units_before(s, s.rts - 1, TR) + kItemCost + (len + kTileKeys - 1) / kTileKeys
                       : s.rts;
  return s;
}

// Exclusive prefix of v over the block's threads; *total = the sum.
__device__ __forceinline__ long long block_prefix(long long v, long long* red, long long* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[w] = x;
  __syncthreads();
  long long before = 0, sum = 0;
#pragma unroll 1
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < w) before += red[i];
    sum += red[i];
  }
  __syncthreads();
  *total = sum;
  return before + x - v;
}

// ---- producers -----------------------------------------------------------------------

// The raw bytes of two pages that one lane turns into operands.
struct RawInt2 {
  uint4 k[2], v[2];
  uint2 km[2];          // {s, z} of key tokens L >> 2 and (L >> 2) + 8
  uint2 vm[2][2];       // {s, z} of value tokens 2t + i and 2t + i + 8
};

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Codes of both 16-bit halves of `w` at bits [2i, 2i + 2), i <= 4, as exact fp16
// values: 1024 + code * 4^i in the mantissa, then * 4^-i - 1024 * 4^-i.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  constexpr uint32_t mask = 0x00030003u << (2 * I);
  const uint32_t x = (w & mask) | 0x64006400u;
  constexpr uint32_t mul = (0x3c00u - (I << 11)) * 0x10001u;             // 2^-2I
  constexpr uint32_t sub = (0x8000u | (0x6400u - (I << 11))) * 0x10001u;  // -2^(10-2I)
  return hfma2(x, mul, sub);
}
template <int W>
__device__ __forceinline__ uint32_t dequant(uint32_t w, uint32_t s2, uint32_t z2) {
  const uint32_t c = W < 5 ? code_pair<W < 5 ? W : 0>(w) : code_pair<W >= 5 ? W - 5 : 0>(w >> 10);
  return hfma2(c, s2, z2);
}
__device__ __forceinline__ uint32_t dup_lo(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t x) { return __byte_perm(x, x, 0x3232); }

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Nonzero bits where a half of x is infinite or NaN (fp16 / bf16).
__device__ __forceinline__ uint32_t nonfinite_f16(uint32_t x) {
  return ((x & 0x7c00u) == 0x7c00u ? 1u : 0u) | ((x & 0x7c000000u) == 0x7c000000u ? 2u : 0u);
}

__device__ __forceinline__ void int2_load(RawInt2& r, int i, const uint8_t* rec, int lane) {
  if (!rec) {
    r.k[i] = r.v[i] = make_uint4(0, 0, 0, 0);
    r.km[i] = r.vm[i][0] = r.vm[i][1] = make_uint2(0, 0);
    return;
  }
  r.k[i] = *reinterpret_cast<const uint4*>(rec + 16 * lane);
  r.v[i] = *reinterpret_cast<const uint4*>(rec + 512 + 16 * lane);
  r.km[i] = *reinterpret_cast<const uint2*>(rec + 1024 + 16 * (lane >> 2));
  r.vm[i][0] = *reinterpret_cast<const uint2*>(rec + 1024 + 32 * (lane & 3) + 8);
  r.vm[i][1] = *reinterpret_cast<const uint2*>(rec + 1024 + 32 * (lane & 3) + 16 + 8);
}

// Values at positions >= key_end (p = the page's first position) become zeros:
// their slots may hold anything.
__device__ __forceinline__ void int2_clip(RawInt2& r, int i, int p, int key_end, int lane) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int tau = 2 * (lane & 3) + e;
    if (p + tau >= key_end) r.vm[i][e].x = 0;
    if (p + tau + 8 >= key_end) r.vm[i][e].y = 0;
  }
}

// Where this lane's part of a key page's tokens goes: chunk j of the token pair (pi, th)
// at key_at(base, j, 4 pi + 2 th).  The swizzle is an exclusive or, so the lane's part
// of it is in the base and the rest is a constant.
__device__ __forceinline__ uint32_t key_base(uint32_t ks, int pair, int lane) {
  const int tau7 = lane >> 2, t = lane & 3;
  const int row = 64 * (pair >> 1) + 16 * (tau7 >> 1) + 8 * (pair & 1) + (tau7 & 1);
  return ks + (t >> 1) * (kTileBytes / 2) + row * 128 +
         (((4 * (t & 1)) ^ (2 * (t >> 1)) ^ (tau7 & 1)) << 4);
}
__device__ __forceinline__ uint32_t key_at(uint32_t base, int j, int r) {
  return (base ^ ((j ^ r) << 4)) + r * 128;
}

// Two pages (pair `pw` of the tile) into a stage's K operand.
__device__ __forceinline__ void int2_store_k(const RawInt2& r, uint32_t ks, int pw, int lane) {
  const uint32_t base = key_base(ks, pw, lane);
#pragma unroll
  for (int pi = 0; pi < 2; ++pi) {
    const uint32_t w[4] = {r.k[pi].x, r.k[pi].y, r.k[pi].z, r.k[pi].w};
    const uint32_t m[2] = {r.km[pi].x, r.km[pi].y};
#pragma unroll
    for (int th = 0; th < 2; ++th) {
      const uint32_t s2 = dup_lo(m[th]), z2 = dup_hi(m[th]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = w[2 * th + h];
        sts128(key_at(base, 2 * h, 4 * pi + 2 * th), dequant<0>(x, s2, z2), dequant<1>(x, s2, z2),
               dequant<2>(x, s2, z2), dequant<3>(x, s2, z2));
        sts128(key_at(base, 2 * h + 1, 4 * pi + 2 * th), dequant<4>(x, s2, z2),
               dequant<5>(x, s2, z2), dequant<6>(x, s2, z2), dequant<7>(x, s2, z2));
      }
    }
  }
}

// The same pages into a stage's V operand.  Returns the lane's bits of tokens
// (16 pi + tau) whose values are not all finite; those tokens' values are stored
// as zeros.
__device__ __forceinline__ uint32_t int2_store_v(const RawInt2& r, uint32_t vs, int pw, int lane) {
  const int g64 = pw >> 1, pp = pw & 1;
  uint32_t poison = 0;
  {
    const int g = lane >> 2, t = lane & 3;
    uint32_t s2[4], z2[4];          // token pairs (pi, th)
#pragma unroll
    for (int pi = 0; pi < 2; ++pi)
#pragma unroll
      for (int th = 0; th < 2; ++th) {
        const uint32_t m0 = th ? r.vm[pi][0].y : r.vm[pi][0].x;
        const uint32_t m1 = th ? r.vm[pi][1].y : r.vm[pi][1].x;
        uint32_t s = __byte_perm(m0, m1, 0x5410), z = __byte_perm(m0, m1, 0x7632);
        // the largest |value| of a token is that of code 0 or 3
        const uint32_t bad = nonfinite_f16(z) | nonfinite_f16(hfma2(s, 0x42004200u, z));
        if (bad) {
          const uint32_t keep = ((bad & 1) ? 0u : 0xffffu) | ((bad & 2) ? 0u : 0xffff0000u);
          s &= keep;
          z &= keep;
          poison |= bad << (16 * pi + 8 * th + 2 * t);
        }
        s2[2 * pi + th] = s;
        z2[2 * pi + th] = z;
      }
    uint32_t row = vs + g64 * (kTileBytes / 2) + g * 128 + (((2 * t + pp) ^ g) << 4);
    uint32_t w0 = r.v[0].x, w1 = r.v[0].z, w2 = r.v[1].x, w3 = r.v[1].z;
#define KVQ_V(M)                                                                        \
  sts128(row + (16 * M) * 128, dequant<M>(w0, s2[0], z2[0]), dequant<M>(w1, s2[1], z2[1]), \
         dequant<M>(w2, s2[2], z2[2]), dequant<M>(w3, s2[3], z2[3]));
#pragma unroll
    for (int dh = 0; dh < 2; ++dh) {
      KVQ_V(0) KVQ_V(1) KVQ_V(2) KVQ_V(3) KVQ_V(4) KVQ_V(5) KVQ_V(6) KVQ_V(7)
      row += 8 * 128;
      w0 = r.v[0].y;
      w1 = r.v[0].w;
      w2 = r.v[1].y;
      w3 = r.v[1].w;
    }
#undef KVQ_V
  }
  return poison;
}

// BF16 pages: the record's 4-byte pairs are moved, not converted.  A lane's eight
// loads of a page's keys (or of half a page pair's values) are in flight while the
// eight before are stored.
__device__ __forceinline__ void bf16_load_key(uint4 (&x)[8], const uint8_t* rec, int lane) {
#pragma unroll
  for (int w = 0; w < 8; ++w)
    x[w] = rec ? *reinterpret_cast<const uint4*>(rec + 512 * w + 16 * lane) : make_uint4(0, 0, 0, 0);
}

// A key page: chunk (th, h, w >> 2) of a token takes one word of each of four loads.
__device__ __forceinline__ void bf16_store_key(const uint4 (&x)[8], uint32_t base, int pi) {
#pragma unroll
  for (int th = 0; th < 2; ++th)
#pragma unroll
    for (int j = 0; j < 4; ++j) {           // j = 2h + (w >> 2)
      auto word = [&](int w) {
        const uint4& q = x[4 * (j & 1) + w];
        return (j >> 1) ? (th ? q.w : q.z) : (th ? q.y : q.x);
      };
      sts128(key_at(base, j, 4 * pi + 2 * th), word(0), word(1), word(2), word(3));
    }
}

// Elements 64 hf .. 64 hf + 63 of two pages' values.
__device__ __forceinline__ void bf16_load_value(uint4 (&x)[8], const uint8_t* const (&rec)[2], int hf,
                                                int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i)             // page i & 1, m = 4 hf + (i >> 1)
    x[i] = rec[i & 1] ? *reinterpret_cast<const uint4*>(rec[i & 1] + 4096 + 512 * (4 * hf + (i >> 1)) +
                                                        16 * lane)
                      : make_uint4(0, 0, 0, 0);
}

// NaN and infinite elements of a word become zeros; bits of the halves that had one.
__device__ __forceinline__ uint32_t bf16_clean(uint32_t& x) {
  const uint32_t bad = ((x & 0x7f80u) == 0x7f80u ? 1u : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 2u : 0u);
  x &= ((bad & 1) ? 0u : 0xffffu) | ((bad & 2) ? 0u : 0xffff0000u);
  return bad;
}

// Returns the lane's bits of tokens (16 pi + tau) that have a NaN or an infinity here.
__device__ __forceinline__ uint32_t bf16_store_value(uint4 (&x)[8], int p0, int key_end, uint32_t vs,
                                                     int pw, int hf, int lane) {
  const int g64 = pw >> 1, pp = pw & 1, g = lane >> 2, t = lane & 3;
  if (p0 + 2 * kPage > key_end) {           // positions >= key_end: zeros
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int th = 0; th < 2; ++th) {
        const int p = p0 + 16 * (i & 1) + 8 * th + 2 * t;
        const uint32_t keep = (p < key_end ? 0xffffu : 0u) | (p + 1 < key_end ? 0xffff0000u : 0u);
        if (th) {
          x[i].z &= keep;
          x[i].w &= keep;
        } else {
          x[i].x &= keep;
          x[i].y &= keep;
        }
      }
  }
  // largest |value| (NaN counts as larger)
  uint32_t big = 0;
  auto maxabs = [&](uint32_t b) {
    b &= 0x7fff7fffu;
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(big) : "r"(b));
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    maxabs(x[i].x);
    maxabs(x[i].y);
    maxabs(x[i].z);
    maxabs(x[i].w);
  }
  uint32_t poison = 0;
  if ((big & 0x7f80u) == 0x7f80u || (big & 0x7f800000u) == 0x7f800000u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      poison |= (bf16_clean(x[i].x) | bf16_clean(x[i].y)) << (16 * (i & 1) + 2 * t);
      poison |= (bf16_clean(x[i].z) | bf16_clean(x[i].w)) << (16 * (i & 1) + 8 + 2 * t);
    }
  }
  const uint32_t row = vs + g64 * (kTileBytes / 2) + (64 * hf + g) * 128 + (((2 * t + pp) ^ g) << 4);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint4 &u = x[2 * m], &v = x[2 * m + 1];
    sts128(row + (16 * m) * 128, u.x, u.z, v.x, v.z);
    sts128(row + (16 * m + 8) * 128, u.y, u.w, v.y, v.w);
  }
  return poison;
}

// A warp's wait for a phase, given up after two seconds of the global timer (its low
// word wraps after 4.3): all lanes have seen the phase complete, or none goes on (the
// tcgen05 loads and stores that follow are warp-wide).  Kept short: some twenty of
// these lie between the roles' loops, which share the instruction cache.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  bool ok = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    uint32_t t0, t1;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
#pragma unroll 1
    do {
      ok = mbar_try_wait_sleep(bar, parity, 100000u);
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t1));
    } while (!__all_sync(0xffffffffu, ok) && t1 - t0 < 2000000000u);
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}

// ---- fp32 pairs ---------------------------------------------------------------------
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// The two bf16 values of a word.
__device__ __forceinline__ uint64_t bf16_pair(uint32_t x) {
  return pair2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The power of two that brings the largest |f x| of this thread's 128 columns x into
// [1, 2), and its inverse: the row's fp16 operand then neither overflows nor loses
// bits, whatever its size.
__device__ __forceinline__ void row_scale(uint32_t addr, float f, float& down, float& up) {
  float mx = 0.0f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t v[32];
    tc_ld32(v, addr + 32 * c);
    tc_wait_ld(v);
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      mx = max3(mx, fabsf(__uint_as_float(v[i])), fabsf(__uint_as_float(v[i + 1])));
  }
  const uint32_t ex = min((__float_as_uint(mx * f) >> 23) & 255u, 253u);
  down = __uint_as_float((254u - ex) << 23);
  up = __uint_as_float(ex << 23);
}

// N registers a thread for the calling warpgroup.
template <int N>
__device__ __forceinline__ void reg_set() {
  if constexpr (N >= kRegLaunch) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// All of the CTA's threads, from whichever role's code.
__device__ __forceinline__ void sync_cta() { asm volatile("barrier.sync 0;" ::: "memory"); }

// ---- the attention kernel ------------------------------------------------------------
//
// Steps of an item: [INT2: R_K] key tiles [INT2, whole item, rotated output: R_V].
// Keys and values have stages and barriers of their own: K of a tile is free after
// the second row tile's scores, two products before V, so that each operand's
// producers have five products' time to refill a stage.  R_K takes a stage of both
// (its two parts), R_V one of K.  Row tile t's S_full completes once per step
// (scores or a rotation's product) and once when O is complete; P_full once per
// operand from the softmax threads (Q, P of each tile, o).

template <bool INT2>
struct Steps {
  int pre, tiles, post;
  __device__ __forceinline__ Steps(const Item& w, const PrefillArgs& a)
      : pre(INT2 && w.tiles > 0 ? 1 : 0),
        tiles(w.tiles),
        post(INT2 && w.tiles > 0 && w.part < 0 && a.rv_tile ? 1 : 0),
        split(w.tokens * a.G <= 128) {}
  bool split;       // one row tile: its even and odd key tiles go to the two softmax groups
  __device__ __forceinline__ int keys() const { return pre + tiles + post; }   // stages of K
  __device__ __forceinline__ int values() const { return pre + tiles; }        // stages of V
};

// The pages of an item's sequence and KV head.
template <bool INT2>
struct Pages {
  const int32_t* table;
  const uint8_t* pool;
  size_t stride;
  int count, ids;
  __device__ __forceinline__ Pages(const PrefillArgs& a, const Item& w)
      : table(a.page_table + static_cast<size_t>(w.b) * a.max_pages),
        pool(a.pool + static_cast<size_t>(w.kv) * (INT2 ? kInt2Rec : kBf16Rec)),
        stride(static_cast<size_t>(a.Hkv) * (INT2 ? kInt2Rec : kBf16Rec)),
        count((w.key_end + kPage - 1) / kPage),
        ids(a.num_pool_pages) {}
  // id of the sequence's page p; -1 behind its last page, or where `wanted` is false
  __device__ __forceinline__ int id(int p, bool wanted) const {
    return wanted && p < count ? table[p] : -1;
  }
  __device__ __forceinline__ const uint8_t* record(int i) const {
    return i >= 0 && i < ids ? pool + static_cast<size_t>(i) * stride : nullptr;
  }
};

// A wait gave up somewhere in the CTA: every role leaves after the same item.
__device__ __forceinline__ bool item_end(bool alive, const PrefillArgs& a, volatile uint32_t* abort) {
  if (!alive) {
    atomicOr(a.status, KVQ_STATUS_TIMEOUT);
    *abort = 1;
  }
  sync_cta();
  return *abort == 0;
}

// The item's query rows into the Q operands, by the first 384 threads.
template <bool INT2>
__device__ __forceinline__ void load_q(const PrefillArgs& a, const Item& w, uint8_t* smem) {
  const int lg = a.G >> 1, rows = w.tokens << lg;         // log2 of 1, 2, 4
  const int pieces = (rows > 128 ? 256 : 128) * 16;
  constexpr int kStep = kMmaWarp * 32, kBatch = 6;        // loads in flight a thread
#pragma unroll 1
  for (int base = threadIdx.x; base < pieces; base += kBatch * kStep) {
    uint4 v[kBatch];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int idx = base + y * kStep, row = idx >> 4;
      v[y] = make_uint4(0, 0, 0, 0);
      if (row < rows)
        v[y] = *reinterpret_cast<const uint4*>(
            a.q + static_cast<size_t>(w.row0 + (row >> lg)) * a.q_stride +
            ((w.kv << lg) + (row & (a.G - 1))) * kDim + 8 * (idx & 15));
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int idx = base + y * kStep, row = idx >> 4, c = idx & 15;
      if (idx >= pieces) break;
      uint8_t* at = smem + Smem::kQ + (row >> 7) * kTileBytes + (row & 127) * 128;
      if constexpr (INT2) {         // d in order: the left operand of q R_K
        *reinterpret_cast<uint4*>(at + (c >> 3) * (kTileBytes / 2) + (((c & 7) ^ (row & 7)) << 4)) = v[y];
      } else {                      // the 16-byte piece holds the pairs t = 0 .. 3 of one (w, h)
        const uint32_t x[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
        const int wq = c >> 1, h = c & 1;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int ch = 4 * (t & 1) + ((2 * h + (wq >> 2)) ^ (2 * (t >> 1)));
          *reinterpret_cast<uint32_t*>(at + (t >> 1) * (kTileBytes / 2) + ((ch ^ (row & 7)) << 4) +
                                       4 * (wq & 3)) = x[t];
        }
      }
    }
  }
  fence_proxy_async();
}

// Word k of the tile's positions that a row sees whose own position is `limit`.
__device__ __forceinline__ uint32_t visible(int limit, int k) {
  const int e = limit - 32 * k;          // last visible bit
  return e >= 31 ? 0xffffffffu : e < 0 ? 0u : (2u << e) - 1u;
}

// One tile's scores (this thread's row, all 128 in registers) into weights: the
// running maximum, the weights as 16-bit pairs into TMEM, their sum.  BF16: the sum is that of
// the rounded weights, so that a weight's rounding (2^-8) moves the output by what sets its
// value apart from the rest only, and a row that sees one token returns it exactly (error
// against 64 bits on two 4093-token prompts 0.0022 against 0.0023; 279 us against 282).
// INT2: the fp16 rounding is an eighth of that and the sum of the unrounded ones (the two
// conversions would cost 5 to 11 % there) as good, 0.0018 either way.
template <bool INT2>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t to, float scale, bool first,
                                             int limit, bool edge, uint32_t any, const volatile uint32_t* bad,
                                             float& mref, float& l) {
  if (edge || any != 0) {
    // Hidden scores become -inf in TMEM first, 32 columns a step: rolled and apart from
    // the tiles' common path, whose code it would double.  Column 32c + i stands for
    // position 64 (c >> 1) + 4 (c & 1) + col_pos(i).
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t hide[2], x[32];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int w = (c & 2) + k;
        hide[k] = (bad[w] | ~visible(limit, w)) >> (4 * (c & 1));
      }
      tc_ld32(x, ts + 32 * c);
      tc_wait_ld(x);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int o = col_pos(i);
        if ((hide[o >> 5] >> (o & 31)) & 1) x[i] = 0xff800000u;
      }
      tc_st32(ts + 32 * c, x);
    }
    tc_wait_st();
  }
  uint32_t v[4][32];
  tc_ld_row(v, ts);
  float m[4];                    // four chains, a quarter of the columns each
#pragma unroll
  for (int c = 0; c < 4; ++c) m[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
  for (int i = 2; i < 32; i += 2)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      m[c] = max3(m[c], __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]));
  const float mnew = fmaxf(mref, fmaxf(max3(m[0], m[1], m[2]), m[3]) * scale);
  // The reference is a whole power of two at or below the maximum, so that two references
  // of a row differ by an exact factor and its weights are rounded alike whichever part of
  // the work, and so whichever batch or chunking, they fall in (a sequence's outputs alone and
  // beside others: 0.3 % of the INT2 path's bf16 results differ against 13 % with references
  // that are plain maxima, 0.05 % against 39 % of the BF16 path's; times alike within 0.5 %).
  if (first) {
    mref = floorf(mnew);
  } else {
    // O is rescaled only when a maximum grew by 2^8 (the weights stay below that times
    // kBias's 2^7, in range of fp16, and the sums are fp32): a step that most tiles skip
    const bool grow = mnew > mref + kLazy;
    if (__any_sync(0xffffffffu, grow)) {
      const float top = floorf(mnew), f = grow ? fast_exp2(mref - top) : 1.0f;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tc_ld16(o, to + 16 * c);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tc_st16(to + 16 * c, o);
      }
      l *= f;
      if (grow) mref = top;
    }
  }
  const float neg = mref == -INFINITY ? 0.0f : (INT2 ? kBias : 0.0f) - mref;
  const uint64_t sc2 = pair2(scale, scale), ng2 = pair2(neg, neg);
  uint64_t s0 = 0, s1 = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t* x = &v[2 * h + (i >> 4)][2 * (i & 15)];
      float x0, x1;
      split2(fma2(pair2(__uint_as_float(x[0]), __uint_as_float(x[1])), sc2, ng2), x0, x1);
      const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
      pk[i] = INT2 ? pack_half2(p0, p1) : pack_bf162(p0, p1);
      const uint64_t w = INT2 ? pair2(p0, p1) : bf16_pair(pk[i]);
      if (i & 1) s1 = add2(s1, w);
      else s0 = add2(s0, w);
    }
    tc_st32(ts + 32 * h, pk);     // all of S is in registers: P may overwrite it
  }
  float a0, a1;
  split2(add2(s0, s1), a0, a1);
  l += a0 + a1;
  tc_wait_st();
}

// The CTA's next item from its range of the line of work (not inlined: it runs once an
// item, and the roles' code shares the instruction cache).
__device__ __noinline__ void next_item(const PrefillArgs& a, Line& line, Item& w) {
  const int TR = kRows / a.G;
  const long long cur = line.cur;
  w.done = 1;
  if (cur >= line.end) return;
  Seq s = load_seq(a, line.b, TR);
  while (cur >= line.b_first + s.units * a.Hkv) {       // ends: cur < total
    line.b_first += s.units * a.Hkv;
    s = load_seq(a, ++line.b, TR);
  }
  const long long local = cur - line.b_first;
  const int kv = static_cast<int>(local / s.units);
  const long long r = local - kv * s.units;
  int lo = 0, hi = s.rts - 1;                     // last row tile that starts at or before r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (units_before(s, mid, TR) <= r) lo = mid;
    else hi = mid - 1;
  }
  // the item's first units are its cost, one per key tile follows: unit `tile0` is tile 0
  const int tok0 = lo * TR, cost = s.ok ? kItemCost : 0;
  const long long tile0 = cur - (r - units_before(s, lo, TR)) + cost;
  w.b = line.b;
  w.kv = kv;
  w.row0 = s.row0 + tok0;
  w.tokens = min(TR, s.n - tok0);
  w.pos0 = s.p0 + tok0;
  w.key_end = s.ok ? w.pos0 + w.tokens : 0;
  const int all = s.ok ? (w.key_end + kTileKeys - 1) / kTileKeys : 1;
  const int t0 = static_cast<int>(max(cur - tile0, 0ll));
  const int t1 = static_cast<int>(min(static_cast<long long>(all), line.end - tile0));
  if (t1 <= t0) return;               // the range ends before the item's first tile
  w.tile_begin = t0;
  w.tiles = s.ok ? t1 - t0 : 0;
  w.part = (t0 == 0 && t1 == all) ? -1 : static_cast<int>(blockIdx.x) * 2 + (t0 == 0 ? 1 : 0);
  w.done = 0;
  if (t0 > 0) {       // an item that ranges before this one began: what joining it takes
    Cut c;
    c.row0 = w.row0;
    c.rows = w.tokens * a.G;
    c.kv = kv;
    c.first = static_cast<int>(tile0 / line.per);
    c.last = static_cast<int>((tile0 + all - 1) / line.per);
    a.cuts[blockIdx.x] = c;
  }
  line.cur = tile0 + t1;
}

// This CTA's range of the line: thread i sums a run of sequences; the thread whose run
// holds the range's first unit knows its sequence.
__device__ __noinline__ void start_line(const PrefillArgs& a, Line* line, long long* red) {
  const int tid = threadIdx.x, TR = kRows / a.G;
  const int per_thread = (a.batch + kThreads - 1) / kThreads;
  const int b_lo = min(tid * per_thread, a.batch), b_hi = min(b_lo + per_thread, a.batch);
  long long mine = 0;
#pragma unroll 1
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq s = load_seq(a, b, TR);
    if (s.bad && blockIdx.x == 0) atomicOr(a.status, s.bad);
    mine += s.units * a.Hkv;
  }
  long long total;
  const long long before = block_prefix(mine, red, &total);
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long u0 = min(per * blockIdx.x, total), u1 = min(u0 + per, total);
  if (tid == 0) {
    line->cur = u0;
    line->end = u1;
    line->per = per;
  }
  if (u0 < u1 && before <= u0 && u0 < before + mine) {
    long long u = before;
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) {
      const long long su = load_seq(a, b, TR).units * a.Hkv;
      if (u0 < u + su) {
        line->b = b;
        line->b_first = u;
        break;
      }
      u += su;
    }
  }
}

template <bool INT2>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar = sb + Smem::kBar;
  Item* items = reinterpret_cast<Item*>(smem + Smem::kItem);
  long long* red = reinterpret_cast<long long*>(smem + Smem::kScan);
  Line* line = reinterpret_cast<Line*>(smem + Smem::kLine);
  volatile uint32_t* badw = reinterpret_cast<volatile uint32_t*>(smem + Smem::kBad);
  uint32_t* first_bad = reinterpret_cast<uint32_t*>(smem + Smem::kPoison);
  volatile uint32_t* poison = first_bad;
  volatile uint32_t* anyw = reinterpret_cast<volatile uint32_t*>(smem + Smem::kAny);
  volatile uint8_t* any8 = reinterpret_cast<volatile uint8_t*>(smem + Smem::kAny);
  volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem + Smem::kTmem + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  auto B = [&](int i) { return bar + 8 * i; };
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(B(kKFull + i), 4);
      mbar_init(B(kKEmpty + i), 1);
      mbar_init(B(kVFull + i), 4);
      mbar_init(B(kVEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(B(kSFull + i), 2);
      mbar_init(B(kPFull + i), 4);
    }
    mbar_init(B(kDrain), 1);
    fence_mbar_init();
    *abort = 0;
    first_bad[0] = 0xffffffffu;
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     sb + Smem::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();

  start_line(a, line, red);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Smem::kTmem);

  bool alive = true;                // false after a wait gave up
  uint32_t itk = 0, itv = 0, itf = 0;   // K and V stages and key tiles so far

  if (warp < kProdWarp0) {
    // ======================= softmax: a thread a row =======================
    reg_set<Regs<INT2>::kSoftmax>();
    const int t = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
    uint8_t* qrow = smem + Smem::kQ + t * kTileBytes + (tid & 127) * 128;
    const int r7 = tid & 7;
    float2* pair = reinterpret_cast<float2*>(smem + Smem::kPair) + (tid & 127);
    uint32_t ns = 0;                // S_full phases
    for (uint32_t i = 0;; ++i) {
      sync_cta();                   // the item is there
      const Item w = items[i & 1];
      if (w.done) break;
      load_q<INT2>(a, w, smem);
      sync_cta();                   // Q is there
      const Steps<INT2> st(w, a);
      const int rows = w.tokens * a.G;
      const int row = st.split ? (tid & 127) : tid;
      const int tok = row / a.G, g = row - tok * a.G;
      const bool valid = row < rows, some = (row & ~31) < rows;
      const int first = st.split ? t : 0, step = st.split ? 2 : 1;    // this group's key tiles
      float mref = -INFINITY, l = 0.0f, scale = a.log2_scale;
      auto wait_s = [&]() {
        alive = warp_wait(B(kSFull + t), ns & 1);
        ++ns;
        tc_fence_after();
        return alive;
      };
      auto give = [&]() {           // an operand of this row tile is ready
        tc_fence_before();
        __syncwarp();
        arrive_if(B(kPFull + t), lane == 0);
      };
      if (first < st.tiles) {
        if (INT2 && (t == 0 || !st.split) && wait_s()) {
          if (some) {
            // q R_K -> fp16 Q, a power of two a row apart, in the pages' order of d
            float down, up;
            row_scale(ts, 1.0f, down, up);
            scale = fmaxf(scale * up, 1.17549435e-38f);  // a row of zeros: 0 * -inf would be NaN
            pair->x = scale;        // for the group of the odd tiles
#pragma unroll 1
            for (int wq = 0; wq < 2; ++wq) {
              uint32_t v[2][32];
#pragma unroll
              for (int c = 0; c < 2; ++c) tc_ld32(v[c], ts + 64 * wq + 32 * c);
#pragma unroll
              for (int c = 0; c < 2; ++c) tc_wait_ld(v[c]);
              auto h2 = [&](int d) {
                return pack_half2(__uint_as_float(v[d >> 5][d & 31]) * down,
                                  __uint_as_float(v[d >> 5][(d & 31) + 1]) * down);
              };
#pragma unroll
              for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int ch = 4 * (tt & 1) + ((2 * h + wq) ^ (2 * (tt >> 1))), d = 8 * h + 2 * tt;
                  *reinterpret_cast<uint4*>(qrow + (tt >> 1) * (kTileBytes / 2) + ((ch ^ r7) << 4)) =
                      make_uint4(h2(d), h2(d + 16), h2(d + 32), h2(d + 48));
                }
            }
            fence_proxy_async();
          }
          give();
        }
        const int pos = w.pos0 + tok;
        for (int j = first; j < st.tiles && alive; j += step) {
          const int limit = valid ? pos - (w.tile_begin + j) * kTileKeys : kTileKeys;
          const bool edge = __any_sync(0xffffffffu, limit < kTileKeys - 1);
          if (!wait_s()) break;
          if (INT2 && st.split && j == 1) scale = pair->x;
          // the tile's missing pages, written before its operands were handed over; the slot
          // is written again four tiles later, which weights of two tiles later precede
          const uint32_t f = (itf + j) % kFlags;
          if (some)
            softmax_tile<INT2>(ts, to, scale, j == first, limit, edge, anyw[f], badw + 4 * f, mref, l);
          give();
        }
        // O is complete.  A row sees all positions up to its own, so it sees a NaN or an
        // infinity if the first one is there (the producers stored zeros in their place).
        if (alive && wait_s() && poison[i & 1] <= static_cast<uint32_t>(pos))
          l = __int_as_float(0x7fffffff);
      }
      if (st.split && st.tiles > 1) {
        // the odd tiles' state to the even tiles' thread of the same row (same TMEM lane)
        if (t == 1) *pair = make_float2(l == 0.0f ? -INFINITY : mref, l);
        tc_fence_before();
        asm volatile("barrier.sync 1, 256;" ::: "memory");
        tc_fence_after();
        if (t == 0 && alive && some) {
          const float2 o = *pair;
          const float mx = fmaxf(mref, o.x), ms = mx == -INFINITY ? 0.0f : mx;
          const float f0 = fast_exp2(mref - ms), f1 = fast_exp2(o.x - ms);
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t x[16], y[16];
            tc_ld16(x, to + 16 * c);
            tc_ld16(y, to + 128 + 16 * c);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[e] = __float_as_uint(__uint_as_float(x[e]) * f0 + __uint_as_float(y[e]) * f1);
            tc_st16(to + 16 * c, x);
          }
          tc_wait_st();
          l = l * f0 + o.y * f1;
          mref = mx;
        }
      }
      const bool active = t == 0 || !st.split;
      // ---- this part's result ----
      const size_t orow = static_cast<size_t>(w.row0 + tok) * a.H + w.kv * a.G + g;
      if (active && alive && w.part >= 0) {
        if (some) {
          float* po = a.part + (static_cast<size_t>(w.part) * kRows + row) * kDim;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tc_ld32(v, to + 32 * c);
            tc_wait_ld(v);
            if (valid) {
              uint4* dst = reinterpret_cast<uint4*>(po + 32 * c);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                dst[x] = make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
            }
            __syncwarp();
          }
          if (valid)
            a.part_ml[static_cast<size_t>(w.part) * kRows + row] =
                make_float2(l == 0.0f ? -INFINITY : mref, l);
        }
      } else if (active && alive) {
        float f = l == 0.0f ? 0.0f : 1.0f / l;
        uint4* dst = reinterpret_cast<uint4*>(a.out + orow * kDim);
        if (st.post) {
          if (some) {
            // o / l -> fp16, a power of two a row apart: the left operand of o R_V^T
            // (normalised first, as the joining kernel does, to be rounded alike)
            float down, up;
            row_scale(to, f, down, up);
            f *= down;            // exact: `down` is a power of two
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              tc_ld32(v, to + 32 * c);
              tc_wait_ld(v);
              auto h2 = [&](int d) {
                return pack_half2(__uint_as_float(v[d]) * f, __uint_as_float(v[d + 1]) * f);
              };
#pragma unroll
              for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4*>(qrow + (c >> 1) * (kTileBytes / 2) +
                                          (((4 * (c & 1) + x) ^ r7) << 4)) =
                    make_uint4(h2(8 * x), h2(8 * x + 2), h2(8 * x + 4), h2(8 * x + 6));
            }
            f = up;
            fence_proxy_async();
          }
          give();
          wait_s();
        }
        if (alive && st.tiles == 0) {
          if (valid)
#pragma unroll
            for (int x = 0; x < 16; ++x) dst[x] = make_uint4(0, 0, 0, 0);
        } else if (alive && some) {
          const uint32_t src = st.post ? ts : to;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tc_ld32(v, src + 32 * c);
            tc_wait_ld(v);
            if (valid) {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  o[e] = pack_bf162(__uint_as_float(v[8 * x + 2 * e]) * f,
                                    __uint_as_float(v[8 * x + 2 * e + 1]) * f);
                dst[4 * c + x] = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
            __syncwarp();
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      itk += st.keys();
      itv += st.values();
      itf += st.tiles;
      if (!item_end(alive, a, abort)) break;
    }
  } else if (warp < kMmaWarp) {
    // ======================= producers =======================
    reg_set<Regs<INT2>::kProducer>();
    const int pw = warp - kProdWarp0;
    uint32_t copy_k = 0, copy_v = 0;       // stages of the last bulk copies
    for (uint32_t i = 0;; ++i) {
      sync_cta();
      const Item w = items[i & 1];
      if (w.done) break;
      const Steps<INT2> st(w, a);
      const Pages<INT2> pages(a, w);
      const int first = w.tile_begin * kTilePages + 2 * pw;       // the pair: first + 8 j, + 1
      auto wait_empty = [&](int empty, uint32_t k) {
        alive = alive && warp_wait(B(empty + k % kStages), ((k / kStages) & 1) ^ 1);
        return alive;
      };
      auto give = [&](int full, uint32_t k) {
        fence_proxy_async();
        __syncwarp();
        arrive_if(B(full + k % kStages), lane == 0);
      };
      auto kbuf = [&](uint32_t k) { return sb + Smem::kK + (k % kStages) * kTileBytes; };
      auto vbuf = [&](uint32_t k) { return sb + Smem::kV + (k % kStages) * kTileBytes; };
      // the pair's records (of the tile that is loaded next) and the ids behind them
      const uint8_t* rec[2];
      RawInt2 raw;
      // a rotation's operand (32 KB, already in the operand's layout) into a stage by one
      // bulk copy, whose bytes complete the stage's phase with the warps' arrivals
      auto give_copy = [&](int full, uint32_t k, uint32_t dst, const uint16_t* src) {
        if (lane == 0) {
          const uint32_t bar = B(full + k % kStages);
          if (pw == 0) {
            mbar_arrive_expect_tx(bar, kTileBytes);
            bulk_g2s(dst, src, kTileBytes, bar);
          } else {
            mbar_arrive(bar);
          }
        }
        __syncwarp();
      };
      const size_t mat = static_cast<size_t>(w.kv) * kDim * kDim;
      if (st.pre && wait_empty(kKEmpty, itk) && wait_empty(kVEmpty, itv)) {
        give_copy(kKFull, itk, kbuf(itk), a.rk_hi + mat);
        give_copy(kVFull, itv, vbuf(itv), a.rk_lo + mat);
        copy_k = itk;
        copy_v = itv;
      }
      int id[2];
      uint4 x[8];
      auto records = [&](int j) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          rec[y] = pages.record(id[y]);
          id[y] = pages.id(first + kTilePages * (j + 1) + y, j + 1 < st.tiles);
        }
      };
#pragma unroll
      for (int y = 0; y < 2; ++y) id[y] = pages.id(first + y, st.tiles > 0);
      records(0);
      if constexpr (INT2) {
#pragma unroll
        for (int y = 0; y < 2; ++y) int2_load(raw, y, rec[y], lane);
      } else {
        bf16_load_key(x, rec[0], lane);
      }
      load_q<INT2>(a, w, smem);
      sync_cta();                   // Q is there
      for (int j = 0; j < st.tiles && alive; ++j) {
        const uint32_t k = itk + st.pre + j, kv = itv + st.pre + j;
        const uint32_t f = itf + j, slot = f % kFlags;
        const int p0 = (first + kTilePages * j) * kPage;
        uint32_t bad = 0, poison;
        auto key_flags = [&]() {
          if (lane == 0) {
            badw[4 * slot + pw] = bad;
            any8[4 * slot + pw] = bad != 0;
            if (bad) atomicOr(a.status, KVQ_STATUS_BAD_PAGE);
          }
        };
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (!rec[y] && p0 + kPage * y < w.key_end) bad |= 0xffffu << (16 * y);
        if (!wait_empty(kKEmpty, k)) break;
        key_flags();
        if constexpr (INT2) {
          int2_store_k(raw, kbuf(k), pw, lane);
          give(kKFull, k);
          if (p0 + 2 * kPage > w.key_end) {
#pragma unroll
            for (int y = 0; y < 2; ++y) int2_clip(raw, y, p0 + kPage * y, w.key_end, lane);
          }
          const RawInt2 now = raw;
          records(j + 1);
#pragma unroll
          for (int y = 0; y < 2; ++y) int2_load(raw, y, rec[y], lane);
          if (!wait_empty(kVEmpty, kv)) break;
          poison = int2_store_v(now, vbuf(kv), pw, lane);
        } else {
          uint4 ahead[8];
          bf16_load_key(ahead, rec[1], lane);
          const uint32_t base = key_base(kbuf(k), pw, lane);
          bf16_store_key(x, base, 0);
          bf16_load_value(x, rec, 0, lane);
          bf16_store_key(ahead, base, 1);
          give(kKFull, k);
          bf16_load_value(ahead, rec, 1, lane);
          if (!wait_empty(kVEmpty, kv)) break;
          poison = bf16_store_value(x, p0, w.key_end, vbuf(kv), pw, 0, lane);
          records(j + 1);
          bf16_load_key(x, rec[0], lane);
          poison |= bf16_store_value(ahead, p0, w.key_end, vbuf(kv), pw, 1, lane);
        }
        if (poison) atomicMin(first_bad + (i & 1), p0 + __ffs(poison) - 1);
        give(kVFull, kv);
      }
      if (st.post && alive && wait_empty(kKEmpty, itk + st.pre + st.tiles)) {
        const uint32_t k = itk + st.pre + st.tiles;
        give_copy(kKFull, k, kbuf(k), a.rv_tile + mat);
        copy_k = k;
      }
      itk += st.keys();
      itv += st.values();
      itf += st.tiles;
      if (!item_end(alive, a, abort)) break;
    }
    // after a wait gave up: a copy may still be under way that nobody waited for
    if (INT2 && *abort) {
      (void)warp_wait(B(kKFull + copy_k % kStages), (copy_k / kStages) & 1);
      (void)warp_wait(B(kVFull + copy_v % kStages), (copy_v / kStages) & 1);
    }
  } else {
    // ======================= tensor-core issue, schedule =======================
    reg_set<Regs<INT2>::kIssue>();
    uint32_t np0 = 0, np1 = 0;      // P_full phases
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), one = elect_one();
    if (warp == kSchedWarp && lane == 0) {
      a.cuts[blockIdx.x].rows = 0;
      next_item(a, *line, items[0]);
    }
    __syncwarp();
    for (uint32_t i = 0;; ++i) {
      sync_cta();
      const Item w = items[i & 1];
      if (w.done) break;
      if (warp == kSchedWarp && lane == 0) {
        first_bad[(i + 1) & 1] = 0xffffffffu;
        next_item(a, *line, items[(i + 1) & 1]);
      }
      __syncwarp();
      const Steps<INT2> st(w, a);
      sync_cta();                   // Q is there
      if (warp == kMmaWarp && st.tiles > 0) {
        constexpr uint32_t idesc = idesc_f16(INT2 ? 0 : 1), idesc_bf = idesc_f16(1);
        const bool both = __shfl_sync(0xffffffffu, st.split ? 0 : 1, 0) != 0;
        const int tiles = __shfl_sync(0xffffffffu, st.tiles, 0);
        auto full = [&](int bar, uint32_t k) {
          alive = alive && warp_wait(B(bar + k % kStages), (k / kStages) & 1);
          tc_fence_after();
          return alive;
        };
        // S_t (or O_t) once the products before are done; the plain arrival passes on what
        // this warp saw of the producers' flags
        auto scored = [&](int t) {
          tc_commit(B(kSFull + t), one);
          arrive_if(B(kSFull + t), one);
        };
        auto empty = [&](int bar, uint32_t k) { tc_commit(B(bar + k % kStages), one); };
        auto operand = [&](int t) {      // Q, P or o of row tile t
          uint32_t& n = t ? np1 : np0;
          alive = alive && warp_wait(B(kPFull + t), n & 1);
          ++n;
          tc_fence_after();
          return alive;
        };
        // S_t = Q_t X^T, X a stage's K (or V) operand
        auto product = [&](int t, uint32_t x, uint32_t id, bool add) {
          const uint32_t q = tile_desc(sb + Smem::kQ + (both ? t : 0) * kTileBytes);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_ss(tm + t * 128, q + desc_step(k), x + desc_step(k), id, add || k != 0, one);
        };
        auto kdesc = [&](uint32_t k) { return tile_desc(sb + Smem::kK + (k % kStages) * kTileBytes); };
        auto vdesc = [&](uint32_t k) { return tile_desc(sb + Smem::kV + (k % kStages) * kTileBytes); };
        auto weighted = [&](int t, uint32_t v, bool add) {     // O_t += P_t V
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_ts(tm + 256 + t * 128, tm + t * 128 + 8 * k, v + desc_step(k), idesc,
                      add || k != 0, one);
        };
        uint32_t k = __shfl_sync(0xffffffffu, itk, 0), v = __shfl_sync(0xffffffffu, itv, 0);
        if (st.pre && full(kKFull, k) && full(kVFull, v)) {
#pragma unroll 1
          for (int t = 0; t < 2; ++t)
            if (t == 0 || both) {
              product(t, kdesc(k), idesc_bf, false);
              product(t, vdesc(v), idesc_bf, true);
              scored(t);
            }
          empty(kKEmpty, k);
          empty(kVEmpty, v);
          ++k;
          ++v;
        }
        if (st.pre) {
          operand(0);
          if (both) operand(1);
        }
        // Step s: O_t += P_t V, then row tile t's next scores, t = s % 2.  Both row tiles:
        // tile s / 2 each; one row tile: tile s, to group t.  Two scores ahead.
        const int total = both ? 2 * tiles : tiles;
        for (int s0 = -2; s0 < total && alive; s0 += 2) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int s = s0 + t;
            if (s >= total) break;
            const bool last = t == 1 || !both;       // of the stages' users
            if (s0 >= 0) {
              if (!full(kVFull, v) || !operand(t)) break;
              weighted(t, vdesc(v), s0 != 0);
              if (last) empty(kVEmpty, v++);
            }
            const bool more = s + 2 < total;
            if (more) {
              if (!full(kKFull, k)) break;
              product(t, kdesc(k), idesc, false);
              if (last) empty(kKEmpty, k++);
            }
            if (s0 >= 0 || more) scored(t);          // the next scores, or O
          }
        }
        if (st.post && alive && full(kKFull, k)) {
#pragma unroll 1
          for (int t = 0; t < 2; ++t)
            if ((t == 0 || both) && operand(t)) {
              product(t, kdesc(k), idesc, false);
              scored(t);
            }
          empty(kKEmpty, k);
        }
      }
      __syncwarp();
      itk += st.keys();
      itv += st.values();
      itf += st.tiles;
      if (!item_end(alive, a, abort)) break;
    }
  }

  // nothing of this CTA may be in flight when it gives its TMEM back
  if (warp == kMmaWarp) {
    tc_commit(B(kDrain), elect_one());
    (void)warp_wait(B(kDrain), 0);
  }
  tc_fence_before();
  sync_cta();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

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

// Joins the partial states of the items that range borders cut, rotates by R_V^T
// (INT2) and writes bf16.  CTA x stands for the border before range x + 1, y for 16 of
// the item's rows; the item's first border does the work.  A warp joins four rows side
// by side (their loads are independent: two round trips to L2 in all), a lane holding
// elements 4 lane .. + 3; then the 16 rows go through mma.sync, 32 output columns a
// warp, as fp16 with a power of two a row apart: a product of 16 x 128 x 128 is too
// small for tcgen05's 128 rows.  Bound by those round trips and the launch.
constexpr int kJoinRows = 16;
constexpr int kJoinPitch = kDim + 8;      // halves: rows 4 banks apart

__global__ void __launch_bounds__(128) prefill_combine_kernel(const __grid_constant__ PrefillArgs a) {
  __shared__ __align__(16) uint16_t os[kJoinRows * kJoinPitch];
  __shared__ float ups[kJoinRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut c = a.cuts[blockIdx.x + 1];
  const int row0 = blockIdx.y * kJoinRows;
  if (c.rows <= row0 || c.first != static_cast<int>(blockIdx.x)) return;
  const int rows = min(c.rows - row0, kJoinRows), parts = c.last - c.first + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.G;
  const int g = lane >> 2, t = lane & 3;
  const bool rotate = a.rv_tile != nullptr;
  // part i of row `row`: CTA first + i left it, the first one in its second slot
  auto slot = [&](int i, int row) {
    return static_cast<size_t>(2 * (c.first + i) + (i == 0 ? 1 : 0)) * kRows + row0 + row;
  };
  auto out_row = [&](int row) {
    const int tk = (row0 + row) / G, gg = (row0 + row) - tk * G;
    return a.out + (static_cast<size_t>(c.row0 + tk) * a.H + c.kv * G + gg) * kDim;
  };
  // R_V's rows n = 32 warp + 8i + g, chunks 4q + t: asked for first, used last
  uint4 b[4][4];
  if (rotate) {
    const uint16_t* rv = a.rv_tile + static_cast<size_t>(c.kv) * kDim * kDim;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int ch = 4 * q + t;
        b[i][q] = *reinterpret_cast<const uint4*>(rv + (ch >> 3) * (kTileBytes / 4) +
                                                  (32 * warp + 8 * i + g) * 64 + (((ch & 7) ^ g) << 3));
      }
  }
  float m[4], l[4];
  float4 o[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.0f;
    o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // rows behind the last read row 0's parts and are not written
  auto row_of = [&](int x) { return 4 * warp + x < rows ? 4 * warp + x : 0; };
  for (int i = lane; i < parts; i += 32)
#pragma unroll
    for (int x = 0; x < 4; ++x) m[x] = fmaxf(m[x], a.part_ml[slot(i, row_of(x))].x);
#pragma unroll
  for (int y = 16; y > 0; y >>= 1)
#pragma unroll
    for (int x = 0; x < 4; ++x) m[x] = fmaxf(m[x], __shfl_xor_sync(0xffffffffu, m[x], y));
  for (int base = 0; base < parts; base += 32) {
    float f[4] = {0.f, 0.f, 0.f, 0.f}, fl[4] = {0.f, 0.f, 0.f, 0.f};
    if (base + lane < parts) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 ml = a.part_ml[slot(base + lane, row_of(x))];
        f[x] = ml.y == 0.0f ? 0.0f : fast_exp2(ml.x - (m[x] == -INFINITY ? 0.0f : m[x]));
        fl[x] = f[x] * ml.y;
      }
    }
#pragma unroll
    for (int y = 16; y > 0; y >>= 1)
#pragma unroll
      for (int x = 0; x < 4; ++x) fl[x] += __shfl_xor_sync(0xffffffffu, fl[x], y);
#pragma unroll
    for (int x = 0; x < 4; ++x) l[x] += fl[x];
    const int count = min(32, parts - base);
#pragma unroll 2
    for (int i = 0; i < count; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float fi = __shfl_sync(0xffffffffu, f[x], i);
        const float4 v = *reinterpret_cast<const float4*>(a.part + slot(base + i, row_of(x)) * kDim + 4 * lane);
        o[x].x = fmaf(fi, v.x, o[x].x);
        o[x].y = fmaf(fi, v.y, o[x].y);
        o[x].z = fmaf(fi, v.z, o[x].z);
        o[x].w = fmaf(fi, v.w, o[x].w);
      }
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int row = 4 * warp + x;
    const float inv = l[x] == 0.0f ? 0.0f : 1.0f / l[x];
    o[x] = make_float4(o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv);
    if (rotate) {
      float mx = fmaxf(fmaxf(fabsf(o[x].x), fabsf(o[x].y)), fmaxf(fabsf(o[x].z), fabsf(o[x].w)));
#pragma unroll
      for (int y = 16; y > 0; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
      const uint32_t ex = min((__float_as_uint(mx) >> 23) & 255u, 253u);
      const float down = __uint_as_float((254u - ex) << 23);
      *reinterpret_cast<uint2*>(os + row * kJoinPitch + 4 * lane) =
          make_uint2(pack_half2(o[x].x * down, o[x].y * down), pack_half2(o[x].z * down, o[x].w * down));
      if (lane == 0) ups[row] = __uint_as_float(ex << 23);
    } else if (row < rows) {
      *reinterpret_cast<uint2*>(out_row(row) + 4 * lane) =
          make_uint2(pack_bf162(o[x].x, o[x].y), pack_bf162(o[x].z, o[x].w));
    }
  }
  if (!rotate) return;
  __syncthreads();
  // out[row][n] = sum_k o[row][k] R_V[n][k], the k of a step in the order of the lanes'
  // 16-byte chunks: 8 (4q + t) + 4i + {0, 1} and {2, 3}
  float acc[4][4] = {};
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint16_t* ar = os + g * kJoinPitch + 8 * (4 * q + t) + 4 * i;
      const uint2 lo = *reinterpret_cast<const uint2*>(ar);
      const uint2 hi = *reinterpret_cast<const uint2*>(ar + 8 * kJoinPitch);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        mma_f16(acc[n], lo.x, hi.x, lo.y, hi.y, i ? b[n][q].z : b[n][q].x, i ? b[n][q].w : b[n][q].y);
    }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = g + 8 * half;
    if (row >= rows) continue;
    const float up = ups[row];
#pragma unroll
    for (int n = 0; n < 4; ++n)
      *reinterpret_cast<uint32_t*>(out_row(row) + 32 * warp + 8 * n + 2 * t) =
          pack_bf162(acc[n][2 * half] * up, acc[n][2 * half + 1] * up);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <bool INT2>
cudaError_t launch(const PrefillArgs& a, int num_sms, cudaStream_t st) {
  static bool attr_set[64] = {};       // per device: the attributes are per context
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel<INT2>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kAlloc);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, prefill_kernel<INT2>);
    if (e != cudaSuccess) return e;
    // see kRegLaunch; the build checks it too (build.py, REGISTERS)
    if (fa.numRegs != kRegLaunch) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  prefill_kernel<INT2><<<num_sms, kThreads, Smem::kAlloc, st>>>(a);
  if (num_sms > 1) {
    // a programmatic dependent: it is launched while the first kernel ends
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms - 1, kRows / kJoinRows);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, prefill_combine_kernel, a);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

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
