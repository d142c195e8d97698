// kvq_rope.cu — rotary positions: the cos / sin table scaled for long contexts,
// the rotation of bf16 rows (and its inverse), and the append of rotated keys
// and plain values into the BF16 paged cache.  (The INT2 append rotates inside
// append_int2_kernel.)
//
// The rotation of a pair (a, b) by the angle of its position is
//   a' = a cos - b sin,  b' = b cos + a sin,
// computed as rope_pair does (fp32, no contraction) and rounded to bf16.  That
// is a linear map with an orthogonal matrix (times the table's amplitude), so
// its inverse with amplitude 1, and its gradient always, is the rotation with
// sin negated.
#include "kvq_internal.cuh"

namespace kvq {
namespace {

// ---------------------------------------------------------------------------
// Table.  Entry (p, i) is amplitude * cos / sin of p * f_i.  The angle is kept
// as a 64-bit fixed-point fraction of a turn, p * F_i mod 2^64 with
// F_i = f_i / (2 pi) * 2^64 (made on the host in fp64): the integer product
// wraps exactly, so the reduction by full turns costs no fp64.  The angle is off by
// F_i's error, some p f_i 2^-53, and by 2^-32 of a turn (1.5e-9 rad) for the product's
// low half, which is dropped.  The top two bits (rounded) are the quadrant; the rest,
// y = at most pi / 4, is rounded to fp32 (pi / 4 * 2^-24); the Taylor series up to y^9
// (sine) and y^10 (cosine) leave less than 2e-9 and their fp32 steps 2^-23.  Below 3e-7
// together up to 2^20 positions (tested).
// Writes are the bound: 4 * table_len * rot_dim bytes; 131072 x 128 takes 16.5 us
// (4.1 TB/s), 8192 x 128 6 us, most of it the launch.
// ---------------------------------------------------------------------------
struct TableArgs {
  float* table;
  int table_len, half;
  float amplitude;
  uint64_t turns[kDim / 2];
};

constexpr int kTableThreads = 256;

__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ TableArgs a) {
  const int rows = kTableThreads / a.half;              // >= 4
  const int r = threadIdx.x / a.half, i = threadIdx.x - r * a.half;
  if (r >= rows) return;
  const uint64_t f = a.turns[i];
  const long long step = static_cast<long long>(gridDim.x) * rows;
  long long p = static_cast<long long>(blockIdx.x) * rows + r;
  for (; p < a.table_len; p += step) {
    const uint32_t hi = static_cast<uint32_t>((static_cast<uint64_t>(p) * f) >> 32);
    const uint32_t quad = (hi + 0x20000000u) >> 30;      // nearest quarter turn (mod 4)
    const int rest = static_cast<int>(hi - (quad << 30));  // in [-2^29, 2^29)
    const float y = static_cast<float>(rest) * 1.46291807926715968e-9f;   // pi / 2^31
    const float z = y * y;
    const float s = fmaf(y * z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), y);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720),
                                         1.0f / 24), -0.5f), 1.0f);
    const float cs = (quad & 1u) ? s : c, sn = (quad & 1u) ? c : s;
    float* t = a.table + static_cast<size_t>(p) * (2 * a.half) + i;
    t[0] = a.amplitude * ((quad == 1u || quad == 2u) ? -cs : cs);
    t[a.half] = a.amplitude * ((quad & 2u) ? -sn : sn);
  }
}

// ---------------------------------------------------------------------------
// Rotation of rows x[n][heads][128] -> y.  One CTA per token, so the token's cos / sin
// row is read from DRAM once and from L1 by its other heads; a thread owns units of
// its heads, one or two at a time (eight CTAs per SM are worth more than more loads a
// thread: 8191 x 32 heads took 27.5 us with 8 CTAs of 32 registers, for which the two
// vector forms spill 16 bytes, 39.2 with 4 of 54):
//   kHalfVec  : 8 elements of the first half and their 8 partners (2 x 16 B);
//   kInterVec : 8 adjacent elements, four pairs (16 B);
//   kScalar   : one pair (any even rot_dim),
// and, behind the rotated part, 16 B (kScalar: two elements) copied unchanged.  The
// units' elements are loaded before the position is looked at, so that its two
// dependent loads (position, table row) overlap them.
// HBM bound at 2 * 2 bytes per element: 8191 x 32 heads in 27.5 us, 73 % of the copy rate.
// ---------------------------------------------------------------------------
enum RopeMode { kHalfVec, kInterVec, kScalar };

struct RopeRowArgs {
  const uint16_t* x;
  uint16_t* y;
  long long x_stride, y_stride;
  int heads, n;
  const int32_t* positions;
  RopeArgs r;
  float sign;            // +1, or -1 for the inverse
  uint32_t* status;
};

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight elements of each half (kHalfVec) of a pair group, rotated.
__device__ __forceinline__ void rotate_halves(uint4& va, uint4& vb, const float* cosp, const float* sinp,
                                              float sign) {
  const float4 c0 = *reinterpret_cast<const float4*>(cosp);
  const float4 c1 = *reinterpret_cast<const float4*>(cosp + 4);
  const float4 s0 = *reinterpret_cast<const float4*>(sinp);
  const float4 s1 = *reinterpret_cast<const float4*>(sinp + 4);
  uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
  const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float p0, q0, p1, q1;
    rope_pair(lo_f(wa[e]), lo_f(wb[e]), c[2 * e], sign * s[2 * e], p0, q0);
    rope_pair(hi_f(wa[e]), hi_f(wb[e]), c[2 * e + 1], sign * s[2 * e + 1], p1, q1);
    wa[e] = pack_bf162(p0, p1);
    wb[e] = pack_bf162(q0, q1);
  }
  va = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  vb = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

// Four adjacent pairs (kInterVec), rotated.
__device__ __forceinline__ void rotate_pairs(uint4& v, const float* cosp, const float* sinp, float sign) {
  const float4 c4 = *reinterpret_cast<const float4*>(cosp);
  const float4 s4 = *reinterpret_cast<const float4*>(sinp);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float p, q;
    rope_pair(lo_f(w[e]), hi_f(w[e]), c[e], sign * s[e], p, q);
    w[e] = pack_bf162(p, q);
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int MODE>
__global__ void __launch_bounds__(256, 8) rope_kernel(RopeRowArgs a) {
  const int rot = a.r.rot_dim, half = rot >> 1;
  // units per head: rotated ones, then copied ones
  const int rot_units = MODE == kHalfVec ? rot / 16 : MODE == kInterVec ? rot / 8 : half;
  const int units = rot_units + (MODE == kScalar ? (kDim - rot) / 2 : (kDim - rot) / 8);
  const int total = a.heads * units;
  const int tok = blockIdx.x;
  const uint16_t* xr = a.x + static_cast<size_t>(tok) * a.x_stride;
  uint16_t* yr = a.y + static_cast<size_t>(tok) * a.y_stride;
  const int pos = a.positions[tok];
  constexpr int kU = MODE == kHalfVec ? 1 : 2;      // units in flight a thread
  for (int base = threadIdx.x; base < total; base += kU * 256) {
    uint4 va[kU], vb[kU];
    int at[kU], u[kU];                               // first element of the unit's head; unit
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int idx = base + i * 256, head = idx / units;
      u[i] = idx - head * units;
      at[i] = head * kDim;
      if (idx >= total) continue;
      const uint16_t* xh = xr + at[i];
      if constexpr (MODE == kScalar) {
        const bool inter = a.r.style == KVQ_ROPE_INTERLEAVED, turn = u[i] < rot_units;
        const int d0 = !turn ? rot + 2 * (u[i] - rot_units) : inter ? 2 * u[i] : u[i];
        va[i].x = xh[d0];
        va[i].y = xh[turn && !inter ? u[i] + half : d0 + 1];
      } else if (u[i] >= rot_units) {
        va[i] = *reinterpret_cast<const uint4*>(xh + rot + 8 * (u[i] - rot_units));
      } else {
        va[i] = *reinterpret_cast<const uint4*>(xh + 8 * u[i]);
        if (MODE == kHalfVec) vb[i] = *reinterpret_cast<const uint4*>(xh + half + 8 * u[i]);
      }
    }
    if (pos < 0 || pos >= a.r.table_len) {
      if (threadIdx.x == 0) atomicOr(a.status, KVQ_STATUS_BAD_POS);
      return;
    }
    const float* cosp = a.r.table + static_cast<size_t>(pos) * rot;
    const float* sinp = cosp + half;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      if (base + i * 256 >= total) break;
      uint16_t* yh = yr + at[i];
      const bool turn = u[i] < rot_units;
      if constexpr (MODE == kScalar) {
        const bool inter = a.r.style == KVQ_ROPE_INTERLEAVED;
        const int d0 = !turn ? rot + 2 * (u[i] - rot_units) : inter ? 2 * u[i] : u[i];
        const int d1 = turn && !inter ? u[i] + half : d0 + 1;
        if (turn) {
          float p, q;
          rope_pair(__uint_as_float(va[i].x << 16), __uint_as_float(va[i].y << 16), cosp[u[i]],
                    a.sign * sinp[u[i]], p, q);
          va[i].x = __bfloat16_as_ushort(__float2bfloat16_rn(p));
          va[i].y = __bfloat16_as_ushort(__float2bfloat16_rn(q));
        }
        yh[d0] = static_cast<uint16_t>(va[i].x);
        yh[d1] = static_cast<uint16_t>(va[i].y);
      } else if (!turn) {
        *reinterpret_cast<uint4*>(yh + rot + 8 * (u[i] - rot_units)) = va[i];
      } else if constexpr (MODE == kHalfVec) {
        rotate_halves(va[i], vb[i], cosp + 8 * u[i], sinp + 8 * u[i], a.sign);
        *reinterpret_cast<uint4*>(yh + 8 * u[i]) = va[i];
        *reinterpret_cast<uint4*>(yh + half + 8 * u[i]) = vb[i];
      } else {
        rotate_pairs(va[i], cosp + 4 * u[i], sinp + 4 * u[i], a.sign);
        *reinterpret_cast<uint4*>(yh + 8 * u[i]) = va[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Append of rotated keys and plain values into the BF16 cache.
//
// A BF16 record (include/kvq.h) interleaves its 16 tokens element by element, so
// a token alone is written in 2-byte pieces (a key's pairs would allow 4), while a
// whole page is 512 16-byte pieces.  A CTA takes about kSpan consecutive tokens
// of one KV head, stages them in shared memory (rotating the keys there), and
// writes every page that its tokens fill completely with 16-byte stores; the
// others element by element.  So that a run of tokens that starts inside a page does
// not cut a page at every CTA border, CTA k starts at the first page border at
// or behind token kSpan * k: at kSpan * k + (-position mod 16), which its
// neighbour computes alike (the ranges partition the tokens whatever the
// positions are; only the speed depends on them).
// HBM bound: 2 * 256 bytes read and 512 written per (token, KV head); 32767 x 8 heads
// in 86 us (49 % of the copy rate: a CTA's loads, transpose and stores follow one
// another, five CTAs an SM; spans of 48 and 32 tokens 95 and 103), a 64-token step 6.2
// on the GPU (the call's host side takes 7.7).
// ---------------------------------------------------------------------------
constexpr int kSpan = 64;      // the widest span; 16 and 4 for fewer tokens (launch below)
constexpr int kMaxTok = kSpan + kPage - 1;
// 68 words a row: rows 4 banks apart, so the 8 rows x 4 words of a key piece and
// the 4 row pairs x 8 elements of a value piece are in different banks
constexpr int kRowB = 2 * kDim + 16;
constexpr int kBfThreads = 256;
constexpr int kLoads = 2;      // 16-byte pieces in flight a thread (4: fewer CTAs per SM, 96 against 86 us)

struct BfSmem {
  static constexpr int kK = 0;
  static constexpr int kV = kK + kMaxTok * kRowB;
  static constexpr int kRec = kV + kMaxTok * kRowB;        // long long [kMaxTok]: record * 16 + slot, or -1
  static constexpr int kAng = kRec + (kMaxTok + 1) / 2 * 16;
  static constexpr int kLead = kAng + kMaxTok * 4;         // u8 [kMaxTok]: 1 page leader, 2 member
  static constexpr int kBytes = (kLead + kMaxTok + 15) / 16 * 16;
};

__device__ __forceinline__ long long span_start(const AppendArgs& a, int k, int span) {
  const long long t = static_cast<long long>(k) * span;
  if (t >= a.n) return a.n;
  if (k == 0 || span < kPage) return t;       // no page fits a narrow span
  const long long s = t + (static_cast<unsigned>(-a.positions[t]) & (kPage - 1));
  return s < a.n ? s : a.n;
}

// MODE: how the keys are rotated: in registers between their load and the staging
// (kHalfVec, kInterVec), or pair by pair in shared memory (kScalar).
template <int MODE>
__global__ void __launch_bounds__(kBfThreads) append_bf16_rope_kernel(AppendArgs a, int span) {
  extern __shared__ __align__(16) uint8_t sm[];
  long long* rec = reinterpret_cast<long long*>(sm + BfSmem::kRec);
  int* ang = reinterpret_cast<int*>(sm + BfSmem::kAng);
  uint8_t* lead = sm + BfSmem::kLead;
  const int kv = blockIdx.y, tid = threadIdx.x;
  const int half = a.rope.rot_dim >> 1, rot = a.rope.rot_dim;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const long long t0 = span_start(a, blockIdx.x, span);
  const int cnt = static_cast<int>(span_start(a, blockIdx.x + 1, span) - t0);   // <= kMaxTok
  if (cnt <= 0) return;

  // The tokens' rows.  Keys: units as in rope_kernel (a piece of each half, or four
  // pairs, or a copied piece); kScalar: plain pieces.  Then values, a piece a unit.
  const int rot_units = MODE == kHalfVec ? rot / 16 : MODE == kInterVec ? rot / 8 : 0;
  const int units = rot_units + (MODE == kScalar ? 16 : (kDim - rot) / 8);
  const int kpieces = cnt * units, pieces = kpieces + cnt * 16;
  const int32_t* ang_pos = a.rope_positions ? a.rope_positions : a.positions;
#pragma unroll 1
  for (int base = tid; base < pieces; base += kLoads * kBfThreads) {
    uint4 va[kLoads], vb[kLoads];
    int w[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = base + i * kBfThreads;
      w[i] = -1;
      if (idx >= pieces) continue;
      if (idx >= kpieces) {
        const int k = (idx - kpieces) >> 4, ch = (idx - kpieces) & 15;
        va[i] = *reinterpret_cast<const uint4*>(a.V + static_cast<size_t>(t0 + k) * a.v_stride +
                                                kv * kDim + 8 * ch);
        continue;
      }
      const int k = idx / units, u = idx - k * units;
      const uint16_t* src = a.K + static_cast<size_t>(t0 + k) * a.k_stride + kv * kDim;
      if (u < rot_units) {
        va[i] = *reinterpret_cast<const uint4*>(src + 8 * u);
        if (MODE == kHalfVec) vb[i] = *reinterpret_cast<const uint4*>(src + half + 8 * u);
        w[i] = ang_pos[t0 + k];
      } else {
        va[i] = *reinterpret_cast<const uint4*>(src + (MODE == kScalar ? 0 : rot) + 8 * (u - rot_units));
      }
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = base + i * kBfThreads;
      if (idx >= pieces) break;
      if (idx >= kpieces) {
        const int k = (idx - kpieces) >> 4, ch = (idx - kpieces) & 15;
        *reinterpret_cast<uint4*>(sm + BfSmem::kV + k * kRowB + 16 * ch) = va[i];
        continue;
      }
      const int k = idx / units, u = idx - k * units;
      uint8_t* dst = sm + BfSmem::kK + k * kRowB;
      if (u >= rot_units) {
        *reinterpret_cast<uint4*>(dst + 2 * ((MODE == kScalar ? 0 : rot) + 8 * (u - rot_units))) = va[i];
        continue;
      }
      if (w[i] >= 0 && w[i] < a.rope.table_len) {     // else the token is skipped below
        const float* t = a.rope.table + static_cast<size_t>(w[i]) * rot;
        if constexpr (MODE == kHalfVec) rotate_halves(va[i], vb[i], t + 8 * u, t + half + 8 * u, 1.0f);
        if constexpr (MODE == kInterVec) rotate_pairs(va[i], t + 4 * u, t + half + 4 * u, 1.0f);
      }
      *reinterpret_cast<uint4*>(dst + 16 * u) = va[i];
      if (MODE == kHalfVec) *reinterpret_cast<uint4*>(dst + 2 * half + 16 * u) = vb[i];
    }
  }
  if (tid < cnt) {
    const long long tok = t0 + tid;
    const int b = a.seq_idx[tok], p = a.positions[tok];
    const int w = a.rope_positions ? a.rope_positions[tok] : p;
    long long r = -1;
    uint32_t bad = 0;
    if (b < 0 || b >= a.batch) {
      bad = KVQ_STATUS_BAD_SEQ;
    } else if (p < 0 || p >= a.max_pages * kPage) {
      bad = KVQ_STATUS_BAD_POS;
    } else {
      const int page = a.page_table[static_cast<size_t>(b) * a.max_pages + p / kPage];
      if (page < 0 || page >= a.num_pool_pages) bad = KVQ_STATUS_BAD_PAGE;
      else r = (static_cast<long long>(page) * a.Hkv + kv) * kPage + (p % kPage);
    }
    const bool in = w >= 0 && w < a.rope.table_len;
    if (!in) bad |= KVQ_STATUS_BAD_POS;
    if (bad) atomicOr(a.status, bad);
    rec[tid] = in ? r : -1;
    ang[tid] = in ? w : -1;
    lead[tid] = 0;
  }
  __syncthreads();

  // page leaders: 16 tokens in slot order of one record (slot 0 first)
  if (tid < cnt && tid + kPage <= cnt && rec[tid] >= 0 && rec[tid] % kPage == 0) {
    bool full = true;
    for (int j = 1; j < kPage; ++j) full = full && rec[tid + j] == rec[tid] + j;
    if (full) lead[tid] = 1;
  }
  // rotate the keys in place: thread -> (token, pair)
  for (int idx = tid; MODE == kScalar && idx < cnt * (kDim / 2); idx += kBfThreads) {
    const int k = idx / (kDim / 2), i = idx % (kDim / 2);
    if (i >= half || ang[k] < 0) continue;
    const float* t = a.rope.table + static_cast<size_t>(ang[k]) * rot + i;
    const bool inter = a.rope.style == KVQ_ROPE_INTERLEAVED;
    uint16_t* row = reinterpret_cast<uint16_t*>(sm + BfSmem::kK + k * kRowB);
    const int d0 = inter ? 2 * i : i, d1 = inter ? 2 * i + 1 : i + half;
    float p, q;
    rope_pair(__uint_as_float(static_cast<uint32_t>(row[d0]) << 16),
              __uint_as_float(static_cast<uint32_t>(row[d1]) << 16), t[0], t[half], p, q);
    row[d0] = __bfloat16_as_ushort(__float2bfloat16_rn(p));
    row[d1] = __bfloat16_as_ushort(__float2bfloat16_rn(q));
  }
  __syncthreads();
  if (tid < cnt && lead[tid] != 1) {      // tokens of a page that a leader before them writes
    for (int j = 1; j < kPage; ++j)
      if (tid - j >= 0 && lead[tid - j] == 1) lead[tid] = 2;
  }
  __syncthreads();

  for (int k = 0; k < cnt; ++k) {
    if (lead[k] != 1) continue;
    uint8_t* base = a.pool + (rec[k] / kPage) * kBf16Rec;
    {                          // keys: tokens L/4 and L/4 + 8, elements 16w + 2t (+8)
      const int L = tid & 31, w = tid >> 5;
      const uint8_t* r0 = sm + BfSmem::kK + (k + (L >> 2)) * kRowB + 2 * (16 * w + 2 * (L & 3));
      const uint8_t* r1 = r0 + 8 * kRowB;
      *reinterpret_cast<uint4*>(base + 512 * w + 16 * L) =
          make_uint4(*reinterpret_cast<const uint32_t*>(r0), *reinterpret_cast<const uint32_t*>(r1),
                     *reinterpret_cast<const uint32_t*>(r0 + 16),
                     *reinterpret_cast<const uint32_t*>(r1 + 16));
    }
    if (tid < 128) {           // values: tokens 2t, 2t + 1 (+8), elements 16w + g, g + 1 (+8), g even
      const int t = tid & 3, g = 2 * ((tid >> 2) & 3), w = tid >> 4;
      const uint8_t* r0 = sm + BfSmem::kV + (k + 2 * t) * kRowB + 2 * (16 * w + g);
      uint32_t lo[4], hi[4];   // th, dh
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* r = r0 + 8 * (i >> 1) * kRowB + 16 * (i & 1);
        const uint32_t e0 = *reinterpret_cast<const uint32_t*>(r);
        const uint32_t e1 = *reinterpret_cast<const uint32_t*>(r + kRowB);
        lo[i] = __byte_perm(e0, e1, 0x5410);
        hi[i] = __byte_perm(e0, e1, 0x7632);
      }
      uint4* dst = reinterpret_cast<uint4*>(base + 4096 + 512 * w + 16 * (4 * g + t));
      dst[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      dst[4] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
  }
  for (int idx = tid; idx < cnt * kDim; idx += kBfThreads) {
    const int k = idx / kDim, d = idx % kDim;
    if (lead[k] != 0 || rec[k] < 0) continue;
    uint8_t* base = a.pool + (rec[k] / kPage) * kBf16Rec;
    const int tau = static_cast<int>(rec[k] % kPage), w = d >> 4, r = d & 15;
    {
      const int L = 4 * (tau & 7) + ((r >> 1) & 3), reg = (tau >> 3) + 2 * (r >> 3);
      *reinterpret_cast<uint16_t*>(base + 512 * w + 16 * L + 4 * reg + 2 * (r & 1)) =
          *reinterpret_cast<const uint16_t*>(sm + BfSmem::kK + k * kRowB + 2 * d);
    }
    {
      const int L = 4 * (r & 7) + ((tau & 7) >> 1), reg = 2 * (tau >> 3) + (r >> 3);
      *reinterpret_cast<uint16_t*>(base + 4096 + 512 * w + 16 * L + 4 * reg + 2 * (tau & 1)) =
          *reinterpret_cast<const uint16_t*>(sm + BfSmem::kV + k * kRowB + 2 * d);
    }
  }
}

}  // namespace

cudaError_t launch_rope_table(float* table, int table_len, int rot_dim, const uint64_t* turns,
                              float amplitude, cudaStream_t st) {
  TableArgs a;
  a.table = table;
  a.table_len = table_len;
  a.half = rot_dim / 2;
  a.amplitude = amplitude;
  for (int i = 0; i < kDim / 2; ++i) a.turns[i] = i < a.half ? turns[i] : 0;
  const int rows = kTableThreads / a.half;
  long long ctas = (static_cast<long long>(table_len) + rows - 1) / rows;
  if (ctas > 152 * 8) ctas = 152 * 8;     // one wave of 8 CTAs per SM; each loops over rows
  rope_table_kernel<<<static_cast<int>(ctas), kTableThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rope(const uint16_t* x, long long x_stride, uint16_t* y, long long y_stride,
                        int heads, const int32_t* positions, int n, const RopeArgs& r, bool inverse,
                        uint32_t* status, cudaStream_t st) {
  RopeRowArgs a;
  a.x = x;
  a.y = y;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.heads = heads;
  a.n = n;
  a.positions = positions;
  a.r = r;
  a.sign = inverse ? -1.0f : 1.0f;
  a.status = status;
  // 16-byte units where the pairs allow them: eight pairs a half, or whole
  // 16-byte groups of adjacent pairs
  const bool inter = r.style == KVQ_ROPE_INTERLEAVED;
  if (!inter && r.rot_dim % 16 == 0) rope_kernel<kHalfVec><<<n, 256, 0, st>>>(a);
  else if (inter && r.rot_dim % 8 == 0) rope_kernel<kInterVec><<<n, 256, 0, st>>>(a);
  else rope_kernel<kScalar><<<n, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_append_bf16_rope(const AppendArgs& a, int num_sms, cudaStream_t st) {
  // the widest span that still gives every SM a CTA: wide spans write whole
  // pages, narrow ones spread a decode step's few tokens over the GPU
  int span = kSpan;
  while (span > 4 && (static_cast<long long>(a.n) + span - 1) / span * a.Hkv < num_sms) span /= 4;
  dim3 grid((static_cast<unsigned>(a.n) + span - 1) / span, a.Hkv);
  const bool inter = a.rope.style == KVQ_ROPE_INTERLEAVED;
  if (!inter && a.rope.rot_dim % 16 == 0)
    append_bf16_rope_kernel<kHalfVec><<<grid, kBfThreads, BfSmem::kBytes, st>>>(a, span);
  else if (inter && a.rope.rot_dim % 8 == 0)
    append_bf16_rope_kernel<kInterVec><<<grid, kBfThreads, BfSmem::kBytes, st>>>(a, span);
  else
    append_bf16_rope_kernel<kScalar><<<grid, kBfThreads, BfSmem::kBytes, st>>>(a, span);
  return cudaGetLastError();
}

}  // namespace kvq
