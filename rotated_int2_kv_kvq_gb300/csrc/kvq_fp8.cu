// kvq_fp8.cu — the 8-bit paged cache: keys and values quantised as they are appended, and
// positions read back.  Layout and rounding are defined in include/kvq.h.
//
// An entry is code * 2^e: e4m3 codes, one exponent for the 16 x 128 keys and one for the values
// of a page and KV head.  A power of two makes x * 2^-e exact, so a code has one rounding, and
// codes that are rounded again because a later token raised e lose bits only where they become
// subnormal (below 2^-6 * 2^e, 2^-13 of the page's largest): a floating code needs no finer scale.
//
// Work is shared out by pages: a page's tokens of one call are consecutive rows of one
// sequence, and the CTA that holds the first of them (the leader) does all of them, a warp a
// (page, KV head), so that nothing is shared between warps.
//
// Both directions move bytes; what bounds them is the chain of a short CTA's loads (sequence, its
// lengths, page id, rows) and their instructions.  Measured, 3 ragged prompts of 32767 tokens in all,
// 8 KV heads: append 37 us (201 MB, 5.5 TB/s), reading 49152 positions 48 us (302 MB, 6.2 TB/s, 92 % of
// the copy rate).  Append: pages that a call fills whole without the masks of part pages (5 us less), a
// sequence's rows and lengths in one load (1.4 less).  Tried and slower: keys and values one after the
// other with 3 or 4 CTAs an SM in place of 2 (+1 to +2 us), 32 to 128 rows a CTA (+0.3 to +12), one warp
// that finds all of a CTA's units (+4).  At 4, 2 and 1 KV heads append 25, 22 and 15 us (4.0, 2.3 and 1.7
// TB/s), reading 29, 22 and 18: a CTA's page or two of rows leave some of its eight warps without work.
// A step of 64 sequences: append 5.3 us, reading the last pages 5.3, nearly all of it launches and the
// chain, which for the append goes on with the page's scales and its older codes.
#include <type_traits>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 16;            // rows a CTA looks through for leaders

struct Unit {
  int row;                              // first row
  int slot, count;                      // its slot in the page; rows of the page
  int page;                             // id, or -1
};

// The sequence of row i, the last b with cu[b] <= i: by 32 probes a step down to 32 candidates, whose
// rows and lengths are read at once (a load less in a chain of five).
struct Owner {
  int b, r0, r1, len;
};
__device__ __forceinline__ Owner find_owner(const Fp8RowArgs& a, int i, int lane) {
  int lo = 0, hi = a.batch;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, p = lo + (lane + 1) * step;
    const unsigned below = __ballot_sync(0xffffffffu, p < hi && a.cu[p] <= i);
    lo += __popc(below) * step;
    hi = min(lo + step, hi);
  }
  const int p = min(lo + lane, hi - 1);
  const int r0 = a.cu[p], r1 = a.cu[p + 1], len = a.seq_lens[p];
  const int own = max(__popc(__ballot_sync(0xffffffffu, lo + lane < hi && r0 <= i)) - 1, 0);
  return Owner{lo + own, __shfl_sync(0xffffffffu, r0, own), __shfl_sync(0xffffffffu, r1, own),
               __shfl_sync(0xffffffffu, len, own)};
}

// The leaders among rows [row0, row0 + rows) as units in shared memory.  A sequence whose
// lengths do not fit gets units without a page where KEEP_BAD (the reader writes zeros), else
// none.  The status bits of all sequences are set by the first CTA.
template <bool KEEP_BAD>
__device__ __forceinline__ int find_units(const Fp8RowArgs& a, int row0, int rows, Unit* units, int* count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) *count = 0;
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
      const int r0 = a.cu[b], r1 = a.cu[b + 1], len = a.seq_lens[b];
      if (r0 < 0 || r1 < r0 || r1 > a.n) atomicOr(a.status, KVQ_STATUS_BAD_SEQ);
      else if (len < r1 - r0 || len > a.max_pages * kPage) atomicOr(a.status, KVQ_STATUS_BAD_SEQLEN);
    }
  }
  for (int k = warp; k < rows; k += kWarps) {
    const int i = row0 + k;
    if (i >= a.n) break;
    const Owner o = find_owner(a, i, lane);
    const int b = o.b, r0 = o.r0, r1 = o.r1, len = o.len;
    if (r0 < 0 || i < r0 || i >= r1 || r1 > a.n) continue;
    const bool ok = len >= r1 - r0 && len <= a.max_pages * kPage;
    if (!ok && !KEEP_BAD) continue;
    const int pos = ok ? len - r1 + i : i - r0;
    const int slot = pos & (kPage - 1);
    if (i != r0 && slot != 0) continue;
    int page = ok ? a.page_table[static_cast<size_t>(b) * a.max_pages + pos / kPage] : -1;
    if (page < 0 || page >= a.num_pool_pages) {
      if (ok && lane == 0) atomicOr(a.status, KVQ_STATUS_BAD_PAGE);
      if (!KEEP_BAD) continue;
      page = -1;
    }
    if (lane == 0) units[atomicAdd(count, 1)] = Unit{i, slot, min(kPage - slot, r1 - i), page};
  }
  __syncthreads();
  return *count;
}

// ---- append -----------------------------------------------------------------------------
// Staging of half a record (K or V): 512-byte quarters 16 bytes apart in banks, so that the
// 2-byte pieces of the 16 pieces of a row fall into different banks.
constexpr int kQuarter = 512 + 16;
constexpr int kStage = 4 * kQuarter;

__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }

// Largest |x| of the warp's rows as bf16 bits; not finite ones are made NaN, do not count and
// set `nan`.
__device__ __forceinline__ uint32_t largest(uint4 (&x)[8], bool& nan) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max_bits(max_bits(max_bits(max_bits(m, x[j].x), x[j].y), x[j].z), x[j].w);
  uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  nan = top >= 0x7f80u;
  if (nan) {
    m = 0;
    auto fix = [&](uint32_t& w) {
      uint32_t keep = 0xffffffffu;
      if ((w & 0x7f80u) == 0x7f80u) w |= 0x40u, keep &= 0xffff0000u;
      if ((w & 0x7f800000u) == 0x7f800000u) w |= 0x400000u, keep &= 0xffffu;
      m = max_bits(m, w & keep);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) fix(x[j].x), fix(x[j].y), fix(x[j].z), fix(x[j].w);
    top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  }
  return top;
}

// The least exponent e >= kFp8MinExp with x <= 448 * 2^e (448 = 1.75 * 2^8), x as bf16 bits.
__device__ __forceinline__ int exponent_for(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 127 - ((bits & 0x7fu) <= 0x60u ? 8 : 7);
  return max(e, kFp8MinExp);
}
// Whether a stored scale is one of this library's, and its exponent.
__device__ __forceinline__ bool scale_exponent(uint32_t bits, int& e) {
  e = static_cast<int>(bits >> 23) - 127;
  return (bits & 0x807fffffu) == 0 && e >= kFp8MinExp && e <= kFp8MaxExp;
}

// Codes of what the four codes of w stand for on a scale 2^k times larger (f as two fp16
// numbers 2^-k): exact products unless they round to zero codes anyway.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, uint32_t f) {
  uint32_t lo, hi;
  uint16_t a, b;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(fp8_lo(w)), "r"(f));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(fp8_hi(w)), "r"(f));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(lo));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(hi));
  return a | static_cast<uint32_t>(b) << 16;
}

// Half a record from global memory (or zeros) into the stage, on a scale 2^k times larger.
__device__ __forceinline__ void stage_old(uint8_t* stage, const uint8_t* rec, bool held, int k, int lane) {
  const uint32_t f = k <= 24 ? static_cast<uint32_t>(__half_as_ushort(__float2half_rn(pow2(-k)))) * 0x10001u : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (held) {
      w = *reinterpret_cast<const uint4*>(rec + 512 * i + 16 * lane);
      if (k > 0) w = make_uint4(rescale4(w.x, f), rescale4(w.y, f), rescale4(w.z, f), rescale4(w.w, f));
    }
    *reinterpret_cast<uint4*>(stage + kQuarter * i + 16 * lane) = w;
  }
}

__device__ __forceinline__ void unpack8(float (&v)[8], const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16) * inv;
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
  }
}

__global__ void __launch_bounds__(kThreads, 2) fp8_append_kernel(const __grid_constant__ Fp8RowArgs a, int rows) {
  __shared__ Unit units[kMaxRows];
  __shared__ int count;
  __shared__ __align__(16) uint8_t stages[kWarps][2][kStage];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dependency_wait();
  const int n_units = find_units<false>(a, blockIdx.x * rows, rows, units, &count);
  const int kv0 = blockIdx.y * kWarps, heads = min(kWarps, a.Hkv - kv0);
  uint8_t *sk = stages[warp][0], *sv = stages[warp][1];
  // lane: piece c (8 elements) of the 8 tokens of half hf of the page
  const int c = lane & 15, hf = lane >> 4;
  for (int p = warp; p < n_units * heads; p += kWarps) {
    const Unit u = units[p / heads];
    const int kv = kv0 + p % heads;
    uint8_t* rec = a.pool + (static_cast<size_t>(u.page) * a.Hkv + kv) * kFp8Rec;
    uint4 x[8], y[8];
    const bool full = u.count == kPage;
    unsigned in = 0;                      // bit j: token 8 hf + j is one of the call's
    if (full) {
      const uint16_t *fk = a.K + (static_cast<size_t>(u.row) + 8 * hf) * a.k_stride + kv * kDim + 8 * c;
      const uint16_t *fv = a.V + (static_cast<size_t>(u.row) + 8 * hf) * a.v_stride + kv * kDim + 8 * c;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = *reinterpret_cast<const uint4*>(fk + j * a.k_stride);
        y[j] = *reinterpret_cast<const uint4*>(fv + j * a.v_stride);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = 8 * hf + j - u.slot;
        x[j] = y[j] = make_uint4(0, 0, 0, 0);
        if (k >= 0 && k < u.count) {
          in |= 1u << j;
          const size_t row = static_cast<size_t>(u.row) + k;
          x[j] = *reinterpret_cast<const uint4*>(a.K + row * a.k_stride + kv * kDim + 8 * c);
          y[j] = *reinterpret_cast<const uint4*>(a.V + row * a.v_stride + kv * kDim + 8 * c);
        }
      }
    }
    // what the page holds counts unless this call begins it (or it was never written)
    uint4 old = make_uint4(0, 0, 0, 0);
    int ek0 = kFp8MinExp, ev0 = kFp8MinExp;
    bool held = u.slot > 0;
    if (held) {
      old = *reinterpret_cast<const uint4*>(rec + 4096);
      held = scale_exponent(old.x, ek0) && scale_exponent(old.y, ev0);
      if (!held) {
        old.z = 0;
        ek0 = ev0 = kFp8MinExp;
      }
    }
    bool nan_k, nan_v;
    const int ek = max(exponent_for(largest(x, nan_k)), ek0), ev = max(exponent_for(largest(y, nan_v)), ev0);
    if (!full) {
      stage_old(sk, rec, held, ek - ek0, lane);
      stage_old(sv, rec + 2048, held, ev - ev0, lane);
    }
    __syncwarp();
    const float ik = pow2(-ek), iv = pow2(-ev);
    auto encode = [&](auto whole) {
      constexpr bool kWhole = decltype(whole)::value;
      // keys: the pairs t = 0 .. 3 of piece c = 2w + h
      uint8_t* at = sk + kQuarter * (c >> 2) + 4 * (hf + 2 * (c & 1)) + 2 * ((c >> 1) & 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!kWhole && !(in >> j & 1)) continue;
        float v[8];
        unpack8(v, x[j], ik);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          *reinterpret_cast<uint16_t*>(at + 64 * j + 16 * t) = fp8_encode(v[2 * t], v[2 * t + 1]);
      }
      // values: tokens 2t, 2t + 1 of the half are neighbours
      at = sv + kQuarter * (c >> 2) + 4 * (2 * ((c >> 1) & 1) + (c & 1)) + 2 * hf;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const unsigned both = kWhole ? 3 : in >> (2 * t) & 3;
        if (both == 0) continue;
        float v0[8], v1[8];
        unpack8(v0, y[2 * t], iv);
        unpack8(v1, y[2 * t + 1], iv);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const uint16_t code = fp8_encode(v0[g], v1[g]);
          uint8_t* to = at + 64 * g + 16 * t;
          if (both == 3) *reinterpret_cast<uint16_t*>(to) = code;
          else if (both == 1) to[0] = static_cast<uint8_t>(code);
          else to[1] = static_cast<uint8_t>(code >> 8);
        }
      }
    };
    if (full) encode(std::true_type());
    else encode(std::false_type());
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<uint4*>(rec + 512 * i + 16 * lane) =
          *reinterpret_cast<const uint4*>(sk + kQuarter * i + 16 * lane);
      *reinterpret_cast<uint4*>(rec + 2048 + 512 * i + 16 * lane) =
          *reinterpret_cast<const uint4*>(sv + kQuarter * i + 16 * lane);
    }
    if (lane == 0)
      *reinterpret_cast<uint4*>(rec + 4096) =
          make_uint4(__float_as_uint(pow2(ek)), __float_as_uint(pow2(ev)),
                     (old.z & 3u) | (nan_k ? 1u : 0u) | (nan_v ? 2u : 0u), 0u);
    __syncwarp();
  }
}

// ---- read -------------------------------------------------------------------------------
// Two codes as two bf16 numbers on the scale s.
__device__ __forceinline__ uint32_t decode2(uint32_t h2, float s) {
  return pack_bf162(half_lo(h2) * s, half_hi(h2) * s);
}

constexpr int kPitch = 2 * kDim + 16;    // bytes of a staged row: rows 4 banks apart

// A staged page's rows that the call wants, to `out`.
__device__ __forceinline__ void write_rows(const uint8_t* stage, const Unit& u, uint16_t* out, long long stride,
                                           int kv, int lane) {
  __syncwarp();
  const int c = lane & 15, hf = lane >> 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int tau = 8 * hf + j, k = tau - u.slot;
    if (k >= 0 && k < u.count)
      *reinterpret_cast<uint4*>(out + (static_cast<size_t>(u.row) + k) * stride + kv * kDim + 8 * c) =
          *reinterpret_cast<const uint4*>(stage + tau * kPitch + 16 * c);
  }
  __syncwarp();
}

__global__ void __launch_bounds__(kThreads) fp8_read_kernel(const __grid_constant__ Fp8RowArgs a, int rows) {
  __shared__ Unit units[kMaxRows];
  __shared__ int count;
  __shared__ __align__(16) uint8_t stages[kWarps][kPage * kPitch];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dependency_wait();
  const int n_units = find_units<true>(a, blockIdx.x * rows, rows, units, &count);
  const int kv0 = blockIdx.y * kWarps, heads = min(kWarps, a.Hkv - kv0);
  uint8_t* stage = stages[warp];
  const int g = lane >> 2, t = lane & 3;
  for (int p = warp; p < n_units * heads; p += kWarps) {
    const Unit u = units[p / heads];
    const int kv = kv0 + p % heads;
    uint4 x[4], y[4], meta = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = y[i] = make_uint4(0, 0, 0, 0);
    if (u.page >= 0) {
      const uint8_t* rec = a.pool + (static_cast<size_t>(u.page) * a.Hkv + kv) * kFp8Rec;
      meta = *reinterpret_cast<const uint4*>(rec + 4096);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = *reinterpret_cast<const uint4*>(rec + 512 * i + 16 * lane);
        y[i] = *reinterpret_cast<const uint4*>(rec + 2048 + 512 * i + 16 * lane);
      }
    }
    if (a.K) {
      // word r of load i: token g + 8 (r & 1), elements 16 w + 8 (r >> 1) + 2t + {0, 1} of w = 2i, 2i + 1
      const float s = __uint_as_float(meta.x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint8_t* to = stage + (g + 8 * (r & 1)) * kPitch + 2 * (32 * i + 8 * (r >> 1) + 2 * t);
          *reinterpret_cast<uint32_t*>(to) = decode2(fp8_lo(w[r]), s);
          *reinterpret_cast<uint32_t*>(to + 32) = decode2(fp8_hi(w[r]), s);
        }
      }
      write_rows(stage, u, a.K, a.k_stride, kv, lane);
    }
    if (a.V) {
      // word r of load i: element 16 (2i + (r >> 1)) + 8 (r & 1) + g of tokens 2t, 2t + 1, 2t + 8, 2t + 9
      const float s = __uint_as_float(meta.y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint8_t* to = stage + 2 * t * kPitch + 2 * (16 * (2 * i + (r >> 1)) + 8 * (r & 1) + g);
          const uint32_t lo = decode2(fp8_lo(w[r]), s), hi = decode2(fp8_hi(w[r]), s);
          *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(lo);
          *reinterpret_cast<uint16_t*>(to + kPitch) = static_cast<uint16_t>(lo >> 16);
          *reinterpret_cast<uint16_t*>(to + 8 * kPitch) = static_cast<uint16_t>(hi);
          *reinterpret_cast<uint16_t*>(to + 9 * kPitch) = static_cast<uint16_t>(hi >> 16);
        }
      }
      write_rows(stage, u, a.V, a.v_stride, kv, lane);
    }
  }
}

// Rows a CTA looks through: the most (up to a page) that still give every SM a CTA.
int rows_per_cta(const Fp8RowArgs& a, int num_sms) {
  const long long groups = (a.Hkv + kWarps - 1) / kWarps;
  int rows = kMaxRows;
  while (rows > 1 && (a.n + rows - 1) / rows * groups < num_sms) rows /= 2;
  return rows;
}

}  // namespace

cudaError_t launch_fp8_append(const Fp8RowArgs& a, int num_sms, cudaStream_t st) {
  const int rows = rows_per_cta(a, num_sms);
  const dim3 grid((static_cast<unsigned>(a.n) + rows - 1) / rows, (a.Hkv + kWarps - 1) / kWarps);
  return launch_dependent(fp8_append_kernel, grid, dim3(kThreads), 0, st, a, rows);
}

cudaError_t launch_fp8_read(const Fp8RowArgs& a, int num_sms, cudaStream_t st) {
  const int rows = rows_per_cta(a, num_sms);
  const dim3 grid((static_cast<unsigned>(a.n) + rows - 1) / rows, (a.Hkv + kWarps - 1) / kWarps);
  return launch_dependent(fp8_read_kernel, grid, dim3(kThreads), 0, st, a, rows);
}

}  // namespace kvq
