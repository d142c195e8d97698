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
// wraps exactly, so the reduction by full turns costs no fp64 and the error is
// that of F_i, p * 2^-53 of a turn at most.  The top two bits (rounded) are the
// quadrant; the rest, at most 1/8 turn, goes through sincospif.
// Writes are the bound: 4 * table_len * rot_dim bytes.
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
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    const float cs = (quad & 1u) ? s : c, sn = (quad & 1u) ? c : s;
    float* t = a.table + static_cast<size_t>(p) * (2 * a.half) + i;
    t[0] = a.amplitude * ((quad == 1u || quad == 2u) ? -cs : cs);
    t[a.half] = a.amplitude * ((quad & 2u) ? -sn : sn);
  }
}

// ---------------------------------------------------------------------------
// Rotation of rows x[n][heads][128] -> y.  One CTA per token (looping when the
// grid is capped), so the token's cos / sin row is read from DRAM once and from
// L1 by its other heads; a thread owns one unit of one head:
//   kHalfVec  : 8 elements of the first half and their 8 partners (2 x 16 B);
//   kInterVec : 8 adjacent elements, four pairs (16 B);
//   kScalar   : one pair (any even rot_dim),
// and, behind the rotated part, 16 B (kScalar: two elements) copied unchanged.
// HBM bound at 2 * 2 bytes per element.
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

template <int MODE>
__global__ void __launch_bounds__(256) rope_kernel(RopeRowArgs a) {
  const int rot = a.r.rot_dim, half = rot >> 1;
  // units per head: rotated ones, then copied ones
  const int rot_units = MODE == kHalfVec ? rot / 16 : MODE == kInterVec ? rot / 8 : half;
  const int units = rot_units + (MODE == kScalar ? (kDim - rot) / 2 : (kDim - rot) / 8);
  const int total = a.heads * units;
  for (int tok = blockIdx.x; tok < a.n; tok += gridDim.x) {
    const int pos = a.positions[tok];
    if (pos < 0 || pos >= a.r.table_len) {
      if (threadIdx.x == 0) atomicOr(a.status, KVQ_STATUS_BAD_POS);
      continue;
    }
    const float* cosp = a.r.table + static_cast<size_t>(pos) * rot;
    const float* sinp = cosp + half;
    const uint16_t* xr = a.x + static_cast<size_t>(tok) * a.x_stride;
    uint16_t* yr = a.y + static_cast<size_t>(tok) * a.y_stride;
    for (int idx = threadIdx.x; idx < total; idx += blockDim.x) {
      const int head = idx / units, u = idx - head * units;
      const uint16_t* xh = xr + head * kDim;
      uint16_t* yh = yr + head * kDim;
      if (u >= rot_units) {
        if (MODE == kScalar) {
          const int d = rot + 2 * (u - rot_units);
          *reinterpret_cast<uint32_t*>(yh + d) = *reinterpret_cast<const uint32_t*>(xh + d);
        } else {
          const int d = rot + 8 * (u - rot_units);
          *reinterpret_cast<uint4*>(yh + d) = *reinterpret_cast<const uint4*>(xh + d);
        }
        continue;
      }
      if constexpr (MODE == kHalfVec) {
        const int d = 8 * u;
        const uint4 va = *reinterpret_cast<const uint4*>(xh + d);
        const uint4 vb = *reinterpret_cast<const uint4*>(xh + half + d);
        const float4 c0 = *reinterpret_cast<const float4*>(cosp + d);
        const float4 c1 = *reinterpret_cast<const float4*>(cosp + d + 4);
        const float4 s0 = *reinterpret_cast<const float4*>(sinp + d);
        const float4 s1 = *reinterpret_cast<const float4*>(sinp + d + 4);
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
        const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
        uint32_t oa[4], ob[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p0, q0, p1, q1;
          rope_pair(lo_f(wa[e]), lo_f(wb[e]), c[2 * e], a.sign * s[2 * e], p0, q0);
          rope_pair(hi_f(wa[e]), hi_f(wb[e]), c[2 * e + 1], a.sign * s[2 * e + 1], p1, q1);
          oa[e] = pack_bf162(p0, p1);
          ob[e] = pack_bf162(q0, q1);
        }
        *reinterpret_cast<uint4*>(yh + d) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
        *reinterpret_cast<uint4*>(yh + half + d) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
      } else if constexpr (MODE == kInterVec) {
        const uint4 v = *reinterpret_cast<const uint4*>(xh + 8 * u);
        const float4 c4 = *reinterpret_cast<const float4*>(cosp + 4 * u);
        const float4 s4 = *reinterpret_cast<const float4*>(sinp + 4 * u);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p, q;
          rope_pair(lo_f(w[e]), hi_f(w[e]), c[e], a.sign * s[e], p, q);
          o[e] = pack_bf162(p, q);
        }
        *reinterpret_cast<uint4*>(yh + 8 * u) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        const bool inter = a.r.style == KVQ_ROPE_INTERLEAVED;
        const int d0 = inter ? 2 * u : u, d1 = inter ? 2 * u + 1 : u + half;
        const float x0 = __uint_as_float(static_cast<uint32_t>(xh[d0]) << 16);
        const float x1 = __uint_as_float(static_cast<uint32_t>(xh[d1]) << 16);
        float p, q;
        rope_pair(x0, x1, cosp[u], a.sign * sinp[u], p, q);
        yh[d0] = __bfloat16_as_ushort(__float2bfloat16_rn(p));
        yh[d1] = __bfloat16_as_ushort(__float2bfloat16_rn(q));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Append of rotated keys and plain values into the BF16 cache.
//
// A BF16 record (include/kvq.h) interleaves its 16 tokens element by element, so
// a token alone is written in 4-byte (keys) and 2-byte (values) pieces, while a
// whole page is 512 16-byte pieces.  A CTA takes about kSpan consecutive tokens
// of one KV head, stages them in shared memory (rotating the keys there), and
// writes every page that its tokens fill completely with 16-byte stores; the
// others element by element.  So that a run of tokens that starts inside a page does
// not cut a page at every CTA border, CTA k starts at the first page border at
// or behind token kSpan * k: at kSpan * k + (-position mod 16), which its
// neighbour computes alike (the ranges partition the tokens whatever the
// positions are; only the speed depends on them).
// HBM bound: 2 * 256 bytes read and 512 written per (token, KV head).
// ---------------------------------------------------------------------------
constexpr int kSpan = 64;      // the widest span; 16 and 4 for fewer tokens (launch below)
constexpr int kMaxTok = kSpan + kPage - 1;
// 68 words a row: rows 4 banks apart, so the 8 rows x 4 words of a key piece and
// the 4 row pairs x 8 elements of a value piece are in different banks
constexpr int kRowB = 2 * kDim + 16;
constexpr int kBfThreads = 256;

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

  // the tokens' rows, 16 bytes a thread, keys then values
  for (int idx = tid; idx < 2 * cnt * 16; idx += kBfThreads) {
    const int ch = idx & 15, k = (idx >> 4) % cnt, which = (idx >> 4) / cnt;
    const uint16_t* src = which ? a.V + static_cast<size_t>(t0 + k) * a.v_stride
                                : a.K + static_cast<size_t>(t0 + k) * a.k_stride;
    *reinterpret_cast<uint4*>(sm + (which ? BfSmem::kV : BfSmem::kK) + k * kRowB + 16 * ch) =
        *reinterpret_cast<const uint4*>(src + kv * kDim + 8 * ch);
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
  for (int idx = tid; idx < cnt * (kDim / 2); idx += kBfThreads) {
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
    for (int u = tid; u < 512; u += kBfThreads) {
      const int L = u & 31, w = (u >> 5) & 7;
      uint4 o;
      if (u < 256) {           // keys: tokens L/4 and L/4 + 8, elements 16w + 2t (+8)
        const uint8_t* r0 = sm + BfSmem::kK + (k + (L >> 2)) * kRowB + 2 * (16 * w + 2 * (L & 3));
        const uint8_t* r1 = r0 + 8 * kRowB;
        o = make_uint4(*reinterpret_cast<const uint32_t*>(r0),
                       *reinterpret_cast<const uint32_t*>(r1),
                       *reinterpret_cast<const uint32_t*>(r0 + 16),
                       *reinterpret_cast<const uint32_t*>(r1 + 16));
      } else {                 // values: tokens 2t, 2t + 1 (+8), elements 16w + g (+8)
        const uint8_t* r0 = sm + BfSmem::kV + (k + 2 * (L & 3)) * kRowB + 2 * (16 * w + (L >> 2));
        auto pair = [&](const uint8_t* p) {
          return static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) |
                 (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + kRowB)) << 16);
        };
        o = make_uint4(pair(r0), pair(r0 + 16), pair(r0 + 8 * kRowB), pair(r0 + 8 * kRowB + 16));
      }
      *reinterpret_cast<uint4*>(base + (u < 256 ? 0 : 4096) + 512 * w + 16 * L) = o;
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
  append_bf16_rope_kernel<<<grid, kBfThreads, BfSmem::kBytes, st>>>(a, span);
  return cudaGetLastError();
}

}  // namespace kvq
