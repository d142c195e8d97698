// kvq_norm.cu — root-mean-square norms of query and key heads with the rotation by the
// token's position in the same pass, and the backward pass.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps),   n_d = x_d r w_d,   y = T n
// with T the token's rotation (include/kvq.h, kvq_rope).  T is linear, so with dn = T^t dy,
// xh = x r and g = dn w:
//   dx = r (g - xh mean_d(g_d xh_d)),   dw_d = sum over rows of dn_d xh_d.
// Everything is fp32 between the bf16 loads and the one rounding of y or dx.
//
// A row (token, head) is worked on by 8 lanes, 16 elements each (backward: 16 lanes of 8), so that
// a pair of the rotation is in one lane and the sums over a row are a few shuffles.
//
// Both directions are bound by HBM: each element is read once and written once (backward: two read).
// Measured, 32 query and 8 key heads, rot_dim 128: forward of 8191 tokens 29.3 us (172 MB, 5.9 TB/s, 86 %
// of the copy rate); backward of 4099 tokens 27.8 us (128 MB), of which 24 are the rows (5.3 TB/s: a CTA
// has 23 rows a group, so that its start is an eighth) and 4 the weights' sum behind them.  16 tokens
// 1.4 us, 257 tokens' backward 4.0 (8 and 2 heads, interleaved): launches and dependent loads.
// Rotated parts that are no multiple of 16 elements (interleaved: 8) go by single elements (kScalar): 51 to
// 58 us and 42.
#include "kvq_internal.cuh"

namespace kvq {
namespace {

// How a lane's E elements (16, 8 lanes a row, or 8, 16 lanes a row) lie in the row, U = E / 2:
//   kHalfVec  : U of the first half of the rotated part and their U partners, or E behind it;
//   kInterVec : U elements (U / 2 pairs) in each half of the head;
//   kScalar   : U pairs of the rotated part or behind it (any even rot_dim).
enum NormMode { kHalfVec, kInterVec, kScalar };

template <int MODE, int E>
struct Lane {
  static constexpr int U = E / 2, kLanes = kDim / E;
  int u;             // lane of the row
  int at0, at1;      // first elements of the two units (vector forms)
  __device__ __forceinline__ Lane(int lane, const RopeArgs& r) : u(lane % kLanes), at0(U * u), at1(64 + U * u) {
    if (MODE == kHalfVec) {
      const int turned = r.rot_dim / E;
      at0 = u < turned ? U * u : r.rot_dim + E * (u - turned);
      at1 = u < turned ? (r.rot_dim >> 1) + U * u : at0 + U;
    }
  }
  // first and second element of pair i of the lane's U (kScalar)
  __device__ __forceinline__ void pair(int i, const RopeArgs& r, int& d0, int& d1) const {
    const int j = u + kLanes * i, half = r.rot_dim >> 1;
    const bool inter = r.style == KVQ_ROPE_INTERLEAVED, turned = j < half;
    d0 = !turned ? r.rot_dim + 2 * (j - half) : inter ? 2 * j : j;
    d1 = turned && !inter ? j + half : d0 + 1;
  }
  // element of the head that v[e] stands for
  __device__ __forceinline__ int dim(int e, const RopeArgs& r) const {
    if constexpr (MODE == kScalar) {
      int d0, d1;
      pair(e >> 1, r, d0, d1);
      return (e & 1) ? d1 : d0;
    } else {
      return e < U ? at0 + e : at1 + e - U;
    }
  }
  // cos and sin of the lane's U pairs; 1 and 0 where nothing turns
  __device__ __forceinline__ void angles(float (&c)[U], float (&s)[U], const float* row, float sign,
                                         const RopeArgs& r) const {
    const int half = r.rot_dim >> 1;
    // two pairs at a time: half is even in the vector forms
    auto two = [&](int k, int i, bool on) {
      float2 x = make_float2(1.f, 1.f), y = make_float2(0.f, 0.f);
      if (on) {
        x = *reinterpret_cast<const float2*>(row + i);
        y = *reinterpret_cast<const float2*>(row + half + i);
      }
      c[k] = x.x, c[k + 1] = x.y;
      s[k] = sign * y.x, s[k + 1] = sign * y.y;
    };
    auto four = [&](int k, int i, bool on) {      // half is a multiple of 4
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on) {
        x = *reinterpret_cast<const float4*>(row + i);
        y = *reinterpret_cast<const float4*>(row + half + i);
      }
      c[k] = x.x, c[k + 1] = x.y, c[k + 2] = x.z, c[k + 3] = x.w;
      s[k] = sign * y.x, s[k + 1] = sign * y.y, s[k + 2] = sign * y.z, s[k + 3] = sign * y.w;
    };
    if constexpr (MODE == kHalfVec) {
#pragma unroll
      for (int k = 0; k < U; k += 4) four(k, U * u + k, u < r.rot_dim / E);
    } else if constexpr (MODE == kInterVec && E == 16) {
      four(0, 4 * u, at0 < r.rot_dim);
      four(4, 32 + 4 * u, at1 < r.rot_dim);
    } else if constexpr (MODE == kInterVec) {
      two(0, 2 * u, at0 < r.rot_dim);
      two(2, 32 + 2 * u, at1 < r.rot_dim);
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int j = u + kLanes * i;
        c[i] = j < half ? row[j] : 1.0f;
        s[i] = j < half ? sign * row[half + j] : 0.0f;
      }
    }
  }
};

// The raw bf16 elements of a lane: U words, the first and second half its two units (vector
// forms), word i its pair i (kScalar).
template <int MODE, int E>
__device__ __forceinline__ void load_raw(uint32_t (&w)[E / 2], const uint16_t* row, const Lane<MODE, E>& l,
                                         const RopeArgs& r) {
  if constexpr (MODE == kScalar) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      int d0, d1;
      l.pair(i, r, d0, d1);
      w[i] = row[d0] | static_cast<uint32_t>(row[d1]) << 16;
    }
  } else if constexpr (E == 16) {
    const uint4 a = *reinterpret_cast<const uint4*>(row + l.at0);
    const uint4 b = *reinterpret_cast<const uint4*>(row + l.at1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(row + l.at0);
    const uint2 b = *reinterpret_cast<const uint2*>(row + l.at1);
    w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
  }
}
template <int E>
__device__ __forceinline__ void unpack(float (&v)[E], const uint32_t (&w)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int MODE, int E>
__device__ __forceinline__ void store_row(uint16_t* row, const float (&v)[E], const Lane<MODE, E>& l,
                                          const RopeArgs& r) {
  uint32_t w[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) w[i] = pack_bf162(v[2 * i], v[2 * i + 1]);
  if constexpr (MODE == kScalar) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      int d0, d1;
      l.pair(i, r, d0, d1);
      row[d0] = static_cast<uint16_t>(w[i]);
      row[d1] = static_cast<uint16_t>(w[i] >> 16);
    }
  } else if constexpr (E == 16) {
    *reinterpret_cast<uint4*>(row + l.at0) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + l.at1) = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    *reinterpret_cast<uint2*>(row + l.at0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + l.at1) = make_uint2(w[2], w[3]);
  }
}

// v's pairs turned by (c, s).
template <int MODE, int E>
__device__ __forceinline__ void turn(float (&v)[E], const float (&c)[E / 2], const float (&s)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const int a = MODE == kHalfVec ? i : 2 * i, b = MODE == kHalfVec ? E / 2 + i : 2 * i + 1;
    const float x = v[a], y = v[b];
    v[a] = x * c[i] - y * s[i];
    v[b] = y * c[i] + x * s[i];
  }
}

// The same of neighbouring elements in pairs.
template <int MODE, int U>
__device__ __forceinline__ void turn_pairs(uint64_t (&v)[U], const float (&c)[U], const float (&s)[U]) {
  if constexpr (MODE == kHalfVec) {
#pragma unroll
    for (int i = 0; i < U / 2; ++i) {
      const uint64_t x = v[i], y = v[U / 2 + i], cc = pair2(c[2 * i], c[2 * i + 1]);
      v[i] = fma2(x, cc, mul2(y, pair2(-s[2 * i], -s[2 * i + 1])));
      v[U / 2 + i] = fma2(y, cc, mul2(x, pair2(s[2 * i], s[2 * i + 1])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float x, y;
      split2(v[i], x, y);
      v[i] = pair2(x * c[i] - y * s[i], y * c[i] + x * s[i]);
    }
  }
}

template <int LANES>
__device__ __forceinline__ float sum_row(float x) {      // over the lanes of a row
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int MODE, int E>
__device__ __forceinline__ void load_weight(float (&w)[E], const float* weight, const Lane<MODE, E>& l,
                                            const RopeArgs& r) {
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = weight ? weight[l.dim(e, r)] : 1.0f;
}

// ---- forward ---------------------------------------------------------------------------
// A warp takes 4 ROWS heads of one token, queries or keys: the token's angles and the weight are
// in registers for all of them, and the elements are asked for before the position, so that its two
// dependent loads (position, table row) overlap them (8191 tokens 29.6 us, after it 33.0).
constexpr int kFwdThreads = 128;

template <int MODE, int ROWS>
__global__ void __launch_bounds__(kFwdThreads) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  const int lane = threadIdx.x & 31;
  // tasks of a token: blockIdx.y the runs of 4 ROWS query heads, then of key heads
  const long long task = static_cast<long long>(blockIdx.x) * (kFwdThreads / 32) + (threadIdx.x >> 5);
  if (task >= a.n) return;
  const int tok = static_cast<int>(task);
  constexpr int kPer = 4 * ROWS;
  const int nq = a.q.x ? (a.q.heads + kPer - 1) / kPer : 0, part = blockIdx.y;
  const bool is_q = part < nq;
  const NormRows& x = is_q ? a.q : a.k;
  const int first = (is_q ? part : part - nq) * kPer + (lane >> 3);
  const uint16_t* xr = x.x + static_cast<size_t>(tok) * x.x_stride;
  uint16_t* yr = x.y + static_cast<size_t>(tok) * x.y_stride;
  const Lane<MODE, 16> l(lane, a.rope);
  dependency_wait();
  const int pos = a.positions[tok];
  uint32_t raw[ROWS][8];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int head = first + 4 * i;
    load_raw(raw[i], xr + (head < x.heads ? head : 0) * kDim, l, a.rope);
  }
  if (pos < 0 || pos >= a.rope.table_len) {
    if (lane == 0) atomicOr(a.status, KVQ_STATUS_BAD_POS);
    return;
  }
  float c[8], s[8], w[16];
  l.angles(c, s, a.rope.table + static_cast<size_t>(pos) * a.rope.rot_dim, 1.0f, a.rope);
  load_weight(w, x.weight, l, a.rope);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int head = first + 4 * i;
    float v[16];
    unpack<16>(v, raw[i]);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(v[e], v[e], ss);
    const float r = rsqrtf(sum_row<8>(ss) * (1.0f / kDim) + a.eps);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = v[e] * r * w[e];
    turn<MODE, 16>(v, c, s);
    if (head < x.heads) store_row(yr + head * kDim, v, l, a.rope);
  }
}

__device__ __forceinline__ void copy_async8(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}

// ---- backward --------------------------------------------------------------------------
// The first a.q_ctas CTAs take the queries, the others the keys.  A row group takes a run of rows
// (token, head), so that a token's angles serve several of them; each lane keeps its 8 elements'
// share of dw, summed over the CTA at the end and over the CTAs by a second kernel, always in the
// same order.  The elements of the next rows are under way into shared memory by asynchronous
// copies (a lane reads back its own, so nothing is waited for but them); with the next row in
// registers instead 4099 tokens of 40 heads took 32.2 us where this took 29.0, 28.5 since two
// elements share an instruction.  4 CTAs an SM spill (34.5), 2 CTAs of 16 elements a lane: 29.7.
constexpr int kBwdThreads = 256;
constexpr int kBwdE = 8;              // elements of a row a lane has
constexpr int kAhead = 4;             // rows a lane has under way
constexpr int kBwdCtas = 3;           // CTAs an SM

template <int MODE>
__global__ void __launch_bounds__(kBwdThreads, kBwdCtas) norm_rope_backward_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring_raw[];
  __shared__ float red[kBwdThreads / 32][kDim];
  const bool is_q = static_cast<int>(blockIdx.x) < a.q_ctas;
  const NormRows& x = is_q ? a.q : a.k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane<MODE, kBwdE> l(lane, a.rope);
  constexpr int U = kBwdE / 2, kLanes = kDim / kBwdE, kRowsCta = kBwdThreads / kLanes;
  static_assert(U == 4, "a uint2 of the ring");
  uint2* ring = reinterpret_cast<uint2*>(ring_raw);                // [kAhead][4][kBwdThreads]
  dependency_wait();
  float wf[kBwdE], c[U], s[U];
  load_weight(wf, x.weight, l, a.rope);
  uint64_t w[U], dw[U];                // pairs of neighbouring elements
#pragma unroll
  for (int e = 0; e < U; ++e) {
    w[e] = pair2(wf[2 * e], wf[2 * e + 1]);
    dw[e] = 0;
    c[e] = s[e] = 0.0f;
  }
  const int ctas = is_q ? a.q_ctas : static_cast<int>(gridDim.x) - a.q_ctas;
  const long long rows = static_cast<long long>(a.n) * x.heads;
  const long long groups = static_cast<long long>(ctas) * kRowsCta;
  const long long per = (rows + groups - 1) / groups;          // uniform: the loop's shuffles
  const long long r0 = ((static_cast<long long>(blockIdx.x) - (is_q ? 0 : a.q_ctas)) * kRowsCta +
                        threadIdx.x / kLanes) * per;
  const int mine = static_cast<int>(max(0ll, min(per, rows - r0)));
  int tok = mine > 0 ? static_cast<int>(r0 / x.heads) : 0, head = mine > 0 ? static_cast<int>(r0 % x.heads) : 0;
  bool fresh = true, good = false;
  // of the row that is asked for next, and of the one that is written
  int head_ahead = head;
  const uint16_t* xr = x.x + static_cast<size_t>(tok) * x.x_stride + head * kDim;
  const uint16_t* dr = x.dy + static_cast<size_t>(tok) * x.dy_stride + head * kDim;
  uint16_t* to = x.y + static_cast<size_t>(tok) * x.y_stride + head * kDim;
  const long long gap = static_cast<long long>(x.heads) * kDim;
  auto ask = [&](int i) {
    if (MODE != kScalar && i < mine) {
      const uint32_t at = smem_u32(ring + (i % kAhead) * 4 * kBwdThreads + threadIdx.x);
      constexpr int kStep = static_cast<int>(sizeof(uint2)) * kBwdThreads;
      copy_async8(at, xr + l.at0);
      copy_async8(at + kStep, xr + l.at1);
      copy_async8(at + 2 * kStep, dr + l.at0);
      copy_async8(at + 3 * kStep, dr + l.at1);
      xr += kDim;
      dr += kDim;
      if (++head_ahead == x.heads) {
        head_ahead = 0;
        xr += x.x_stride - gap;
        dr += x.dy_stride - gap;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kAhead - 1; ++i) ask(i);
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const bool in = i < mine;
    ask(i + kAhead - 1);
    if (in && fresh) {
      const int pos = a.positions[tok];
      good = pos >= 0 && pos < a.rope.table_len;
      if (!good && l.u == 0) atomicOr(a.status, KVQ_STATUS_BAD_POS);
      l.angles(c, s, a.rope.table + static_cast<size_t>(good ? pos : 0) * a.rope.rot_dim, -1.0f, a.rope);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    uint32_t rx[U] = {}, rd[U] = {};
    if (in) {
      if constexpr (MODE == kScalar) {
        load_raw(rx, x.x + static_cast<size_t>(tok) * x.x_stride + head * kDim, l, a.rope);
        load_raw(rd, x.dy + static_cast<size_t>(tok) * x.dy_stride + head * kDim, l, a.rope);
      } else {
        const uint2* from = ring + (i % kAhead) * 4 * kBwdThreads + threadIdx.x;
        const uint2 e[4] = {from[0], from[kBwdThreads], from[2 * kBwdThreads], from[3 * kBwdThreads]};
        rx[0] = e[0].x, rx[1] = e[0].y, rx[2] = e[1].x, rx[3] = e[1].y;
        rd[0] = e[2].x, rd[1] = e[2].y, rd[2] = e[3].x, rd[3] = e[3].y;
      }
    }
    uint64_t v[U], d[U];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      v[e] = bf16_pair(rx[e]);
      d[e] = bf16_pair(rd[e]);
    }
    turn_pairs<MODE>(d, c, s);
    uint64_t ss2 = 0, gx2 = 0;
#pragma unroll
    for (int e = 0; e < U; ++e) {
      ss2 = fma2(v[e], v[e], ss2);
      gx2 = fma2(mul2(d[e], w[e]), v[e], gx2);
    }
    float ss, gx, x1;
    split2(ss2, ss, x1);
    ss += x1;
    split2(gx2, gx, x1);
    gx += x1;
    const float r = rsqrtf(sum_row<kLanes>(ss) * (1.0f / kDim) + a.eps);
    const float m = sum_row<kLanes>(gx) * r * (1.0f / kDim);
    if (in && good) {
      const uint64_t r2 = pair2(r, r), m2 = pair2(-m, -m);
      float y[kBwdE];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const uint64_t xh = mul2(v[e], r2);
        dw[e] = fma2(d[e], xh, dw[e]);
        split2(mul2(fma2(xh, m2, mul2(d[e], w[e])), r2), y[2 * e], y[2 * e + 1]);
      }
      store_row(to, y, l, a.rope);
    }
    fresh = head + 1 == x.heads;
    head = fresh ? 0 : head + 1;
    tok += fresh ? 1 : 0;
    to += kDim;
    if (fresh) to += x.y_stride - gap;
  }
  dependents_begin();
  float sums[kBwdE];
#pragma unroll
  for (int e = 0; e < U; ++e) split2(dw[e], sums[2 * e], sums[2 * e + 1]);
#pragma unroll
  for (int e = 0; e < kBwdE; ++e) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) sums[e] += __shfl_xor_sync(0xffffffffu, sums[e], o);
    if (lane < kLanes) red[warp][l.dim(e, a.rope)] = sums[e];
  }
  __syncthreads();
  if (threadIdx.x < kDim) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kBwdThreads / 32; ++i) sum += red[i][threadIdx.x];
    a.part[static_cast<size_t>(blockIdx.x) * kDim + threadIdx.x] = sum;
  }
}

// dw of the queries or the keys: 8 elements a CTA, a warp 4 of the CTAs' parts at a time, always in the
// same order (32 elements a CTA, a part a warp: 0.5 us more).
__global__ void __launch_bounds__(1024) norm_weight_kernel(const __grid_constant__ NormArgs a, int ctas) {
  __shared__ float red[32][8];
  dependency_wait();
  float* dw = blockIdx.y == 0 ? a.q.dw : a.k.dw;
  if (!dw) return;
  const int first = blockIdx.y == 0 ? 0 : a.q_ctas, parts = (blockIdx.y == 0 ? a.q_ctas : ctas) - first;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 8 + (lane & 7);
  const float* p = a.part + static_cast<size_t>(first) * kDim + col;
  float sum = 0.0f;
#pragma unroll 4
  for (int i = 4 * warp + (lane >> 3); i < parts; i += 128) sum += p[static_cast<size_t>(i) * kDim];
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  sum += __shfl_xor_sync(0xffffffffu, sum, 16);
  if (lane < 8) red[warp][lane] = sum;
  __syncthreads();
  if (warp == 0) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += red[8 * (lane >> 3) + i][lane & 7];
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (lane < 8) dw[col] = sum;
  }
}

NormMode mode_of(const RopeArgs& r) {
  const bool inter = r.style == KVQ_ROPE_INTERLEAVED;
  return !inter && r.rot_dim % 16 == 0 ? kHalfVec : inter && r.rot_dim % 8 == 0 ? kInterVec : kScalar;
}

}  // namespace

int norm_backward_ctas(int num_sms) { return kBwdCtas * num_sms; }

template <int MODE>
static cudaError_t forward(const NormArgs& a, int num_sms, cudaStream_t st) {
  // Two rows a group where one each would be a warp a scheduler or more, else one, for more warps
  // (tokens of 32 and 8 heads, two rows against one: 8191 29.6 and 33.2 us, 1024 5.0 and 5.9, 256 2.4
  // and 2.5, 64 the same, 16 1.7 and 1.5; four rows, 8191: 29.2)
  const int quads = (a.q.x ? (a.q.heads + 3) / 4 : 0) + (a.k.x ? (a.k.heads + 3) / 4 : 0);
  const bool wide = static_cast<long long>(a.n) * quads >= 4 * num_sms;
  const int per = wide ? 8 : 4;
  const dim3 grid((static_cast<unsigned>(a.n) + kFwdThreads / 32 - 1) / (kFwdThreads / 32),
                  (a.q.x ? (a.q.heads + per - 1) / per : 0) + (a.k.x ? (a.k.heads + per - 1) / per : 0));
  return launch_dependent(wide ? norm_rope_kernel<MODE, 2> : norm_rope_kernel<MODE, 1>, grid, dim3(kFwdThreads), 0,
                          st, a);
}

cudaError_t launch_norm_rope(const NormArgs& a, int num_sms, cudaStream_t st) {
  switch (mode_of(a.rope)) {
    case kHalfVec: return forward<kHalfVec>(a, num_sms, st);
    case kInterVec: return forward<kInterVec>(a, num_sms, st);
    default: return forward<kScalar>(a, num_sms, st);
  }
}

template <int MODE>
static cudaError_t backward(const NormArgs& a, int ctas, cudaStream_t st) {
  constexpr int kSmem = MODE == kScalar ? 0 : kAhead * 4 * kBwdThreads * kBwdE;
  static bool attr_set[64] = {};       // per device: the attributes are per context
  int dev = 0;
  cudaGetDevice(&dev);
  if (kSmem > 0 && (dev < 0 || dev >= 64 || !attr_set[dev])) {
    const cudaError_t e = cudaFuncSetAttribute(norm_rope_backward_kernel<MODE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  return launch_dependent(norm_rope_backward_kernel<MODE>, dim3(ctas), dim3(kBwdThreads), kSmem, st, a);
}

cudaError_t launch_norm_rope_backward(NormArgs a, int num_sms, cudaStream_t st) {
  // a row a group at least, shared out between queries and keys by their rows
  const long long hq = a.q.x ? a.q.heads : 0, hk = a.k.x ? a.k.heads : 0;
  const long long groups = kBwdThreads / (kDim / kBwdE);
  long long ctas = ((hq + hk) * a.n + groups - 1) / groups + 1;
  if (ctas > norm_backward_ctas(num_sms)) ctas = norm_backward_ctas(num_sms);
  long long q = hq + hk > 0 ? (ctas * hq + (hq + hk) / 2) / (hq + hk) : 0;
  if (hq > 0 && q < 1) q = 1;
  if (hk > 0 && q > ctas - 1) q = ctas - 1;
  a.q_ctas = static_cast<int>(q);
  const int g = static_cast<int>(ctas);
  if (a.n > 0) {
    cudaError_t e;
    switch (mode_of(a.rope)) {
      case kHalfVec: e = backward<kHalfVec>(a, g, st); break;
      case kInterVec: e = backward<kInterVec>(a, g, st); break;
      default: e = backward<kScalar>(a, g, st);
    }
    if (e != cudaSuccess) return e;
  }
  // launched while the first kernel ends
  return launch_dependent(norm_weight_kernel, dim3(kDim / 8, 2), dim3(1024), 0, st, a, a.n > 0 ? g : 0);
}

}  // namespace kvq
