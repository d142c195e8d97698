// kvq_norm.cu — root-mean-square norms of query and key heads with the rotation by the
// token's position in the same pass, and the backward pass.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps),   n_d = x_d r w_d,   y = T n
// with T the token's rotation (include/kvq.h, kvq_rope).  T is linear, so with dn = T^t dy,
// xh = x r and g = dn w:
//   dx = r (g - xh mean_d(g_d xh_d)),   dw_d = sum over rows of dn_d xh_d.
// Everything is fp32 between the bf16 loads and the one rounding of y or dx.
//
// A row (token, head) is worked on by 8 lanes, 16 elements each, so that a pair of the
// rotation is in one lane and the sums over a row are three shuffles.
#include "kvq_internal.cuh"

namespace kvq {
namespace {

// How a lane's 16 elements lie in the row:
//   kHalfVec  : 8 of the first half of the rotated part and their 8 partners, or 16 behind it;
//   kInterVec : 8 elements (four pairs) in each half of the head;
//   kScalar   : eight pairs of the rotated part or behind it (any even rot_dim).
enum NormMode { kHalfVec, kInterVec, kScalar };

template <int MODE>
struct Lane {
  int u;             // lane of the row, 0 .. 7
  int at0, at1;      // first elements of the two 8-element units (vector forms)
  __device__ __forceinline__ Lane(int lane, const RopeArgs& r) : u(lane & 7), at0(8 * u), at1(64 + 8 * u) {
    if (MODE == kHalfVec) {
      const int turned = r.rot_dim >> 4;
      at0 = u < turned ? 8 * u : r.rot_dim + 16 * (u - turned);
      at1 = u < turned ? (r.rot_dim >> 1) + 8 * u : at0 + 8;
    }
  }
  // first and second element of pair i of the lane's eight (kScalar)
  __device__ __forceinline__ void pair(int i, const RopeArgs& r, int& d0, int& d1) const {
    const int j = u + 8 * i, half = r.rot_dim >> 1;
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
      return e < 8 ? at0 + e : at1 + e - 8;
    }
  }
  // cos and sin of the lane's eight pairs; 1 and 0 where nothing turns
  __device__ __forceinline__ void angles(float (&c)[8], float (&s)[8], const float* row, float sign,
                                         const RopeArgs& r) const {
    const int half = r.rot_dim >> 1;
    auto four = [&](int k, int i, bool on) {
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on) {
        // half is a multiple of 4 in the vector forms
        x = *reinterpret_cast<const float4*>(row + i);
        y = *reinterpret_cast<const float4*>(row + half + i);
      }
      c[k] = x.x, c[k + 1] = x.y, c[k + 2] = x.z, c[k + 3] = x.w;
      s[k] = sign * y.x, s[k + 1] = sign * y.y, s[k + 2] = sign * y.z, s[k + 3] = sign * y.w;
    };
    if constexpr (MODE == kHalfVec) {
      const bool on = u < (r.rot_dim >> 4);
      four(0, 8 * u, on);
      four(4, 8 * u + 4, on);
    } else if constexpr (MODE == kInterVec) {
      four(0, 4 * u, at0 < r.rot_dim);
      four(4, 32 + 4 * u, at1 < r.rot_dim);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = u + 8 * i;
        c[i] = j < half ? row[j] : 1.0f;
        s[i] = j < half ? sign * row[half + j] : 0.0f;
      }
    }
  }
};

// The raw bf16 elements of a lane: 8 words, words 0-3 and 4-7 its two units (vector forms),
// word i its pair i (kScalar).
template <int MODE>
__device__ __forceinline__ void load_raw(uint32_t (&w)[8], const uint16_t* row, const Lane<MODE>& l,
                                         const RopeArgs& r) {
  if constexpr (MODE == kScalar) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int d0, d1;
      l.pair(i, r, d0, d1);
      w[i] = row[d0] | static_cast<uint32_t>(row[d1]) << 16;
    }
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(row + l.at0);
    const uint4 b = *reinterpret_cast<const uint4*>(row + l.at1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void unpack(float (&v)[16], const uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int MODE>
__device__ __forceinline__ void store_row(uint16_t* row, const float (&v)[16], const Lane<MODE>& l,
                                          const RopeArgs& r) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf162(v[2 * i], v[2 * i + 1]);
  if constexpr (MODE == kScalar) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int d0, d1;
      l.pair(i, r, d0, d1);
      row[d0] = static_cast<uint16_t>(w[i]);
      row[d1] = static_cast<uint16_t>(w[i] >> 16);
    }
  } else {
    *reinterpret_cast<uint4*>(row + l.at0) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + l.at1) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// v's pairs turned by (c, s).
template <int MODE>
__device__ __forceinline__ void turn(float (&v)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = MODE == kHalfVec ? i : 2 * i, b = MODE == kHalfVec ? 8 + i : 2 * i + 1;
    const float x = v[a], y = v[b];
    v[a] = x * c[i] - y * s[i];
    v[b] = y * c[i] + x * s[i];
  }
}

__device__ __forceinline__ float sum8(float x) {      // over the 8 lanes of a row
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  return x + __shfl_xor_sync(0xffffffffu, x, 4);
}

template <int MODE>
__device__ __forceinline__ void load_weight(float (&w)[16], const float* weight, const Lane<MODE>& l,
                                            const RopeArgs& r) {
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = weight ? weight[l.dim(e, r)] : 1.0f;
}

// ---- forward ---------------------------------------------------------------------------
// A warp takes one token's queries or keys, kHeads at a time a row group: the token's angles
// and the weight are in registers for all of them.
constexpr int kFwdThreads = 128;

template <int MODE>
__global__ void __launch_bounds__(kFwdThreads) norm_rope_kernel(const __grid_constant__ NormArgs a, int rows) {
  const int lane = threadIdx.x & 31;
  const long long task = static_cast<long long>(blockIdx.x) * (kFwdThreads / 32) + (threadIdx.x >> 5);
  // tasks of a token: runs of 4 * rows query heads, then of key heads
  const int per = 4 * rows, nq = a.q.x ? (a.q.heads + per - 1) / per : 0,
            nk = a.k.x ? (a.k.heads + per - 1) / per : 0;
  const int tok = static_cast<int>(task / (nq + nk)), part = static_cast<int>(task % (nq + nk));
  if (tok >= a.n) return;
  const bool is_q = part < nq;
  const NormRows& x = is_q ? a.q : a.k;
  const int first = (is_q ? part : part - nq) * per + (lane >> 3);
  const uint16_t* xr = x.x + static_cast<size_t>(tok) * x.x_stride;
  uint16_t* yr = x.y + static_cast<size_t>(tok) * x.y_stride;
  const Lane<MODE> l(lane, a.rope);
  const int pos = a.positions[tok];
  if (pos < 0 || pos >= a.rope.table_len) {
    if (lane == 0) atomicOr(a.status, KVQ_STATUS_BAD_POS);
    return;
  }
  float c[8], s[8], w[16];
  l.angles(c, s, a.rope.table + static_cast<size_t>(pos) * a.rope.rot_dim, 1.0f, a.rope);
  load_weight(w, x.weight, l, a.rope);
  for (int i = 0; i < rows; ++i) {
    const int head = first + 4 * i;
    const bool on = head < x.heads;
    uint32_t raw[8];
    load_raw(raw, xr + (on ? head : 0) * kDim, l, a.rope);
    float v[16];
    unpack(v, raw);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(v[e], v[e], ss);
    const float r = rsqrtf(sum8(ss) * (1.0f / kDim) + a.eps);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = v[e] * r * w[e];
    turn<MODE>(v, c, s);
    if (on) store_row(yr + head * kDim, v, l, a.rope);
  }
}

// ---- backward --------------------------------------------------------------------------
// blockIdx.y: queries or keys.  Row groups stride over the rows (token, head); each lane keeps
// its 16 elements' share of dw, summed over the CTA at the end and over the CTAs by a second
// kernel, always in the same order.
constexpr int kBwdThreads = 256;

template <int MODE>
__global__ void __launch_bounds__(kBwdThreads) norm_rope_backward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[kBwdThreads / 32][kDim];
  const bool is_q = blockIdx.y == 0;
  const NormRows& x = is_q ? a.q : a.k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane<MODE> l(lane, a.rope);
  float w[16], dw[16];
  load_weight(w, x.weight, l, a.rope);
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.0f;
  const long long rows = x.x ? static_cast<long long>(a.n) * x.heads : 0;
  const long long step = static_cast<long long>(gridDim.x) * (kBwdThreads / 8);
  const long long first = static_cast<long long>(blockIdx.x) * (kBwdThreads / 8) + (threadIdx.x >> 3);
  for (long long base = first - (lane >> 3); base < rows; base += step) {     // uniform in the warp
    const long long row = base + (lane >> 3);
    const bool in = row < rows;
    const int tok = in ? static_cast<int>(row / x.heads) : 0, head = in ? static_cast<int>(row % x.heads) : 0;
    const int pos = a.positions[tok];
    const bool good = pos >= 0 && pos < a.rope.table_len, on = in && good;
    if (in && !good && l.u == 0) atomicOr(a.status, KVQ_STATUS_BAD_POS);
    uint32_t rx[8], rd[8];
    load_raw(rx, x.x + static_cast<size_t>(tok) * x.x_stride + head * kDim, l, a.rope);
    load_raw(rd, x.dy + static_cast<size_t>(tok) * x.dy_stride + head * kDim, l, a.rope);
    float c[8], s[8], v[16], d[16];
    l.angles(c, s, a.rope.table + static_cast<size_t>(good ? pos : 0) * a.rope.rot_dim, -1.0f, a.rope);
    unpack(v, rx);
    unpack(d, rd);
    turn<MODE>(d, c, s);
    float ss = 0.0f, gx = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      ss = fmaf(v[e], v[e], ss);
      gx = fmaf(d[e] * w[e], v[e], gx);
    }
    const float r = rsqrtf(sum8(ss) * (1.0f / kDim) + a.eps);
    const float m = sum8(gx) * r * (1.0f / kDim);
    if (on) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float xh = v[e] * r;
        dw[e] = fmaf(d[e], xh, dw[e]);
        v[e] = r * (d[e] * w[e] - xh * m);
      }
      store_row(x.y + static_cast<size_t>(tok) * x.y_stride + head * kDim, v, l, a.rope);
    }
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], 8);
    dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], 16);
    if (lane < 8) red[warp][l.dim(e, a.rope)] = dw[e];
  }
  __syncthreads();
  if (threadIdx.x < kDim) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kBwdThreads / 32; ++i) sum += red[i][threadIdx.x];
    a.part[(static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kDim + threadIdx.x] = sum;
  }
}

// dw of the queries or the keys: 32 elements a CTA, the CTAs' parts in order.
__global__ void __launch_bounds__(256) norm_weight_kernel(const __grid_constant__ NormArgs a, int parts) {
  __shared__ float red[8][32];
  float* dw = blockIdx.y == 0 ? a.q.dw : a.k.dw;
  if (!dw) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float* p = a.part + static_cast<size_t>(blockIdx.y) * parts * kDim + blockIdx.x * 32 + lane;
  float sum = 0.0f;
  for (int i = warp; i < parts; i += 8) sum += p[static_cast<size_t>(i) * kDim];
  red[warp][lane] = sum;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += red[i][lane];
    dw[blockIdx.x * 32 + lane] = sum;
  }
}

NormMode mode_of(const RopeArgs& r) {
  const bool inter = r.style == KVQ_ROPE_INTERLEAVED;
  return !inter && r.rot_dim % 16 == 0 ? kHalfVec : inter && r.rot_dim % 8 == 0 ? kInterVec : kScalar;
}

}  // namespace

int norm_backward_parts(int n, int num_sms) {
  // at most four CTAs an SM; a row group each for the rows of few tokens
  const long long most = 4LL * num_sms;
  return static_cast<int>(n < most ? (n < 1 ? 1 : n) : most);
}

cudaError_t launch_norm_rope(const NormArgs& a, cudaStream_t st) {
  const int rows = 1;
  const int per = 4 * rows;
  const long long tasks = static_cast<long long>(a.n) * ((a.q.x ? (a.q.heads + per - 1) / per : 0) +
                                                         (a.k.x ? (a.k.heads + per - 1) / per : 0));
  const long long grid = (tasks + kFwdThreads / 32 - 1) / (kFwdThreads / 32);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int g = static_cast<int>(grid);
  switch (mode_of(a.rope)) {
    case kHalfVec: norm_rope_kernel<kHalfVec><<<g, kFwdThreads, 0, st>>>(a, rows); break;
    case kInterVec: norm_rope_kernel<kInterVec><<<g, kFwdThreads, 0, st>>>(a, rows); break;
    default: norm_rope_kernel<kScalar><<<g, kFwdThreads, 0, st>>>(a, rows);
  }
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_backward(const NormArgs& a, int num_sms, cudaStream_t st) {
  const int parts = norm_backward_parts(a.n, num_sms);
  const dim3 grid(parts, 2);
  switch (mode_of(a.rope)) {
    case kHalfVec: norm_rope_backward_kernel<kHalfVec><<<grid, kBwdThreads, 0, st>>>(a); break;
    case kInterVec: norm_rope_backward_kernel<kInterVec><<<grid, kBwdThreads, 0, st>>>(a); break;
    default: norm_rope_backward_kernel<kScalar><<<grid, kBwdThreads, 0, st>>>(a);
  }
  norm_weight_kernel<<<dim3(kDim / 32, 2), 256, 0, st>>>(a, parts);
  return cudaGetLastError();
}

}  // namespace kvq
