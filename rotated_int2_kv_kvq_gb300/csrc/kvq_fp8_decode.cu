// kvq_fp8_decode.cu — attention of one query token a sequence over the 8-bit paged cache, all
// of it or a sliding window and the first tokens.
//
// Entries are code * 2^e with one e for a page's keys and one for its values (include/kvq.h),
// and a page is the M = 16 tokens of an mma.sync tile, so no entry is ever scaled: codes become
// fp16 operands by one conversion a pair, and the two factors go into the page's scores,
//   logit_t = scale 2^ek (q . code_t),
// and its weights, w_t = 2^(logit_t - m + ev - er), m the running maximum.  er is that of a run of
// pages whose ev lies within er - 6 .. er + 7: where a page's does not, what the run has summed goes
// times 2^er into the fp32 totals and the page begins the next run.  So a weight's range is spent on
// logits alone, whatever the scales of other pages: w fits fp16.  Query and weights enter as an fp16
// part and a residual in a column of its own (times 2^11): products of fp32 accuracy, as kvq_decode's;
// a weight's error is 2^-23 of it, or 2^-30 of the largest weight's.
//
// All visible pages of all (sequence, KV head) items form one line of work, cut into equal
// ranges, one a CTA; an item that a border cuts leaves partial states for the joining kernel.
//
// HBM bounds it: every visible page is read once, by a bulk copy a page into a warp's own ring of
// three; when a CTA's part of an item ends, the next part's ids and first two pages are under way while
// the warps wait for one another and join.  Measured, 32 query and 8 KV heads: 16 x 32K 181 us (1.08
// GB, 6.0 TB/s, 88 % of the copy rate; 187 with the parts one after the other; 4, 2 and 1 KV heads 96, 53
// and 32); the SMs of the GPU's larger clusters get some 15 % less bandwidth each, so equal ranges end
// after 143 to 183 us, and what would even that out costs as much: 2 to 6 times as many CTAs 185 to
// 193, ranges that shrink towards the end 181 to 200 (windows more), pages by tickets 186 to 213.
// 64 windows of 4100 positions 86 us (462 MB, 5.4 TB/s; 89 likewise): 512 items, so two or three
// parts a CTA.  1 x 1K 8.3 us on the GPU, two launches and a chain of loads.
#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
constexpr int kMinUnits = kWarps;       // pages of a CTA's range at least: one a warp
constexpr int kItemCost = 40;           // pages that an item counts for beside its own
constexpr int kFlush = 16;              // pages of a warp between flushes of the accumulators
constexpr int kMaxCtas = 1024;          // of the grid: sizes the joining kernel's arrays
constexpr float kLazy = 8.0f;           // log2 by which the reference may lag behind the maximum
constexpr int kBelow = 6, kAbove = 7;   // of a run's er: 2^(kLazy + kAbove) fits fp16
// Totals are in units of 2^u, u = 0 until an exponent passes kUnitTop: then values of up to 2^128,
// times weights of up to 2^kLazy, summed over any length, fit fp32.
constexpr int kUnitTop = 86;

struct __align__(16) Smem {
  uint8_t ring[kWarps][kStages][kFp8Rec];
  uint64_t bar[kWarps][kStages];
  int ids[kWarps][kStages];
  float m[kWarps][kMaxG], l[kWarps][kMaxG];
  long long red[kWarps];
  int u[kWarps];                        // the unit of a warp's totals
  int state[kWarps];                    // the stage that a warp's state is in
};

// What a sequence's query sees: positions [0, lead) and [first, len), in pages 0 .. sp - 1 and
// sp + skip onwards, `pages` of them.
struct Seen {
  int len, first, lead, sp, skip, pages;
  bool bad;
};
__device__ __forceinline__ Seen seen_of(const Fp8DecodeArgs& a, int b) {
  Seen s;
  s.len = a.seq_lens[b];
  s.bad = s.len < 0 || s.len > a.max_pages * kPage;
  if (s.bad) s.len = 0;
  s.first = a.window > 0 ? max(0, s.len - a.window) : 0;
  s.lead = min(a.sinks, s.first);
  s.sp = (s.lead + kPage - 1) / kPage;
  s.skip = max(0, s.first / kPage - s.sp);
  s.pages = (s.len + kPage - 1) / kPage - s.skip;
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
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) before += red[i];
    sum += red[i];
  }
  __syncthreads();
  *total = sum;
  return before + x - v;
}

struct Start {            // a CTA's range of the line of work
  long long cur, end, per;
  long long b_first;      // first unit of sequence b
  int b;
};

// An item counts its pages, at least one, and kItemCost more for what it costs a CTA whatever its
// length (query, page ids and first records to wait for, the warps' states to join): in the line,
// those units come before its first page.  (64 ragged sequences up to 16K: without 138 us, 8: 119,
// 16: 108, 32: 98; 64 windows of 4100: 97, 93, 90, 88; 16 x 32K the same whatever.  Since parts
// overlap: 32: 96.5 and 87.8, 40: 96.2 and 87.0, 48: 96.4 and 87.4; with 1, 2 and 4 KV heads, where 40
// takes 22.9, 32.4, 53.4 and 21.4, 29.6, 48.5, 32 and 48 are within 2 % of it, 16 is 2 to 9 % slower.)
__device__ __forceinline__ int item_units(const Seen& s) { return max(s.pages, 1) + kItemCost; }
__device__ __forceinline__ void start_line(const Fp8DecodeArgs& a, Start* line, long long* red) {
  const int tid = threadIdx.x;
  const int per_thread = (a.batch + kThreads - 1) / kThreads;
  const int b_lo = min(tid * per_thread, a.batch), b_hi = min(b_lo + per_thread, a.batch);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Seen s = seen_of(a, b);
    if (s.bad && blockIdx.x == 0) atomicOr(a.status, KVQ_STATUS_BAD_SEQLEN);
    mine += static_cast<long long>(item_units(s)) * a.Hkv;
  }
  long long total;
  const long long before = block_prefix(mine, red, &total);
  const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(kMinUnits));
  const long long u0 = min(per * blockIdx.x, total), u1 = min(u0 + per, total);
  if (tid == 0) {
    line->cur = u0;
    line->end = u1;
    line->per = per;
  }
  if (u0 < u1 && before <= u0 && u0 < before + mine) {
    long long u = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long su = static_cast<long long>(item_units(seen_of(a, b))) * a.Hkv;
      if (u0 < u + su) {
        line->b = b;
        line->b_first = u;
        break;
      }
      u += su;
    }
  }
  __syncthreads();
}

// B fragments of the query: column 2h holds q_h * 2^-x (largest element in [1, 2)) as fp16, column
// 2h + 1 the residual times 2^11.  Returns 2^x of head lane & 3.
__device__ __forceinline__ float query_frags(const Fp8DecodeArgs& a, int b, int kv, int lane, uint32_t (&qf)[16]) {
  const int g = lane >> 2, t = lane & 3, head = g >> 1;
  const bool use = head < a.G;
  const uint32_t* row = reinterpret_cast<const uint32_t*>(
      a.q + (static_cast<size_t>(b) * a.H + kv * a.G + (use ? head : 0)) * kDim);
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    qf[i] = use ? row[4 * i + t] : 0u;       // elements 8i + 2t, + 1
    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(qf[i] << 16)), fabsf(__uint_as_float(qf[i] & 0xffff0000u))));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const uint32_t ex = min(max((__float_as_uint(mx) >> 23) & 255u, 1u), 253u);   // 1: subnormal ones too
  const float down = __uint_as_float((254u - ex) << 23), up = __uint_as_float(ex << 23);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float x = __uint_as_float(qf[i] << 16) * down, y = __uint_as_float(qf[i] & 0xffff0000u) * down;
    const uint32_t hi = pack_half2(x, y);
    qf[i] = (g & 1) ? pack_half2((x - half_lo(hi)) * 2048.0f, (y - half_hi(hi)) * 2048.0f) : hi;
  }
  return __shfl_sync(0xffffffffu, up, 8 * t);
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_fp8_kernel(const __grid_constant__ Fp8DecodeArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  __shared__ Start line;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&sm.bar[warp][s]), 1);
    fence_mbar_init();
  }
  dependency_wait();
  start_line(a, &line, sm.red);
  if (tid == 0) a.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
  const size_t page_stride = static_cast<size_t>(a.Hkv) * kFp8Rec;
  uint32_t used = 0;                 // ring stages so far
  bool alive = true;

  // The part of an item that this CTA works on, and the warp's pages of it.
  long long cur = line.cur, b_first = line.b_first;
  int b = line.b, kv = 0, j0 = 0, j1 = 0, count = 0;
  Seen s = {};
  int blk = 0, ids = -1, ids_next = -1;
  auto page_of = [&](int i) {        // the warp's i-th page
    const int j = j0 + warp + kWarps * i;
    return j < s.sp ? j : j + s.skip;
  };
  auto load_ids = [&](int k) {
    const int i = 32 * k + lane;
    return i < count ? a.page_table[static_cast<size_t>(b) * a.max_pages + page_of(i)] : -1;
  };
  auto first_page = [&]() { return b_first + static_cast<long long>(kv) * item_units(s) + kItemCost; };   // in the line
  // the part at `cur`, false where the range ends (before the item's first page)
  auto begin = [&]() {
    if (cur >= line.end) return false;
    s = seen_of(a, b);
    while (cur >= b_first + static_cast<long long>(item_units(s)) * a.Hkv) {     // ends: cur < total
      b_first += static_cast<long long>(item_units(s)) * a.Hkv;
      s = seen_of(a, ++b);
    }
    kv = static_cast<int>((cur - b_first) / item_units(s));
    const long long item = first_page();
    j0 = static_cast<int>(max(cur - item, 0ll));
    j1 = static_cast<int>(min(static_cast<long long>(max(s.pages, 1)), line.end - item));
    if (j1 <= 0) return false;
    const int jp = min(j1, s.pages);                                             // pages j0 .. jp - 1
    count = jp - j0 > warp ? (jp - j0 - warp + kWarps - 1) / kWarps : 0;
    blk = 0;
    ids = load_ids(0);
    ids_next = load_ids(1);
    return true;
  };
  auto issue = [&](int i) {
    if ((i >> 5) != blk) {
      blk = i >> 5;
      ids = ids_next;
      ids_next = load_ids(blk + 1);
    }
    const int id = __shfl_sync(0xffffffffu, ids, i & 31);
    if (lane == 0) {
      const int slot = (used + i) % kStages;
      const uint32_t bar = smem_u32(&sm.bar[warp][slot]);
      const bool ok = id >= 0 && id < a.num_pool_pages;
      sm.ids[warp][slot] = ok ? id : -1;
      if (ok) {
        mbar_arrive_expect_tx(bar, kFp8Rec);
        bulk_g2s(smem_u32(sm.ring[warp][slot]),
                 a.pool + static_cast<size_t>(kv) * kFp8Rec + static_cast<size_t>(id) * page_stride, kFp8Rec, bar);
      } else {
        atomicOr(a.status, KVQ_STATUS_BAD_PAGE);
        mbar_arrive(bar);
      }
    }
  };
  bool have = false, whole = false;  // a part whose states are to be joined; into `to`: all of an item
  float* to = nullptr;
  while (true) {
    // the next part's ids and first copies are under way while the warps wait for one another and join
    const bool more = alive && begin();
    __syncwarp();
    if (have && lane == 0) fence_proxy_async();      // the stages were read
    if (more)
#pragma unroll 1
      for (int k = 0; k < kStages - 1 && k < count; ++k) issue(k);
    if (have) {
      const bool stop = __syncthreads_or(!alive);
      for (int e = tid; e < a.G * kDim; e += kThreads) {
        const int h = e / kDim, d = e % kDim;
        float M = -INFINITY, U = 0.0f, L = 0.0f, o = 0.0f, state[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          state[w] = reinterpret_cast<const float*>(sm.ring[w][sm.state[w]])[e];
          M = fmaxf(M, sm.m[w][h]);
          U = fmaxf(U, static_cast<float>(sm.u[w]));
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          // a warp without a token has l = 0 (one that met a NaN logit has l = NaN and no maximum)
          const float x = sm.m[w][h], lw = sm.l[w][h];
          if (lw == 0.0f) continue;
          const float f = x == M ? 1.0f : fast_exp2(x - M);
          L = fmaf(f, lw, L);
          o = fmaf(f, state[w] * fast_exp2(static_cast<float>(sm.u[w]) - U), o);
        }
        if (whole) {
          to[e] = L == 0.0f ? 0.0f : o / L * fast_exp2(U);
        } else {
          float* p = to + h * kPartStride;
          p[4 + d] = o;
          if (d == 0) {
            p[0] = M;
            p[1] = L;
            p[2] = U;
          }
        }
      }
      __syncthreads();
      if (stop) {                  // a wait ran out: what this warp asked for has to land
        if (more)
          for (int k = 0; k < kStages - 1 && k < count; ++k)
            mbar_drain(smem_u32(&sm.bar[warp][(used + k) % kStages]), ((used + k) / kStages) & 1);
        break;
      }
    }
    if (!more) break;
    if (have && lane == 0) fence_proxy_async();      // a state was written over the last stage
    __syncwarp();
    if (count >= kStages) issue(kStages - 1);
    uint32_t qf[16];
    const float up = query_frags(a, b, kv, lane, qf);
    float acc[8][4], tot[8][2];
#pragma unroll
    for (int mb = 0; mb < 8; ++mb) {
      tot[mb][0] = tot[mb][1] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[mb][k] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;      // of head t
    int er = 0;                         // the run's exponent
    if (lane == 0) sm.u[warp] = 0;
    __syncwarp();
    auto flush = [&]() {
      const float f = pow2(-sm.u[warp]), fe = pow2(er);
#pragma unroll
      for (int mb = 0; mb < 8; ++mb) {
        tot[mb][0] = fmaf(fmaf(acc[mb][1], 0x1p-11f, acc[mb][0]) * f, fe, tot[mb][0]);
        tot[mb][1] = fmaf(fmaf(acc[mb][3], 0x1p-11f, acc[mb][2]) * f, fe, tot[mb][1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[mb][k] = 0.0f;
      }
    };

    int i = 0;
    for (; i < count; ++i) {
      const int slot = (used + i) % kStages;
      if (!mbar_wait_bounded(smem_u32(&sm.bar[warp][slot]), ((used + i) / kStages) & 1)) {
        if (lane == 0) atomicOr(a.status, KVQ_STATUS_TIMEOUT);
        alive = false;
        break;
      }
      const bool page_ok = sm.ids[warp][slot] >= 0;
      const uint8_t* st = sm.ring[warp][slot];
      const uint4 meta = *reinterpret_cast<const uint4*>(st + 4096);
      float sa[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 w = *reinterpret_cast<const uint4*>(st + 512 * k + 16 * lane);
        mma_f16(sa, fp8_lo(w.x), fp8_lo(w.y), fp8_lo(w.z), fp8_lo(w.w), qf[4 * k], qf[4 * k + 1]);
        mma_f16(sb, fp8_hi(w.x), fp8_hi(w.y), fp8_hi(w.z), fp8_hi(w.w), qf[4 * k + 2], qf[4 * k + 3]);
      }
      uint4 vw[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) vw[k] = *reinterpret_cast<const uint4*>(st + 2048 + 512 * k + 16 * lane);
      __syncwarp();
      if (i + kStages < count) {
        if (lane == 0) fence_proxy_async();
        issue(i + kStages);
      }
      if (!page_ok) continue;
      const int pos = page_of(i) * kPage;
      auto visible = [&](int tau) {
        const int p = pos + tau;
        return p < s.len && (p >= s.first || p < s.lead);
      };
      // the powers of two first: a sum of products times 2^ek alone may overflow where the score does not
      const float kf = fminf(__uint_as_float(meta.x) * up * a.log2_scale, 3.4028235e38f);
      const int ev = static_cast<int>(meta.y >> 23) - 127;
      if (ev < er - kBelow || ev > er + kAbove) {      // alike in all lanes
        flush();
        er = ev;
        if (const int u = sm.u[warp]; ev > u + kUnitTop) {
          __syncwarp();
          const float f = pow2(u + kUnitTop - ev);
#pragma unroll
          for (int mb = 0; mb < 8; ++mb) {
            tot[mb][0] *= f;
            tot[mb][1] *= f;
          }
          if (lane == 0) sm.u[warp] = ev - kUnitTop;
          __syncwarp();
        }
      }
      const float l0 = visible(g) ? fmaf(sa[1] + sb[1], 0x1p-11f, sa[0] + sb[0]) * kf : -INFINITY;
      const float l1 = visible(g + 8) ? fmaf(sa[3] + sb[3], 0x1p-11f, sa[2] + sb[2]) * kf : -INFINITY;
      float pm = fmaxf(l0, l1);
      pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 4));
      pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 8));
      pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 16));
      if (__any_sync(0xffffffffu, pm > m + kLazy)) {
        // whole powers of two: their differences are exact, and a weight is rounded alike whichever
        // reference it meets
        const float mn = fmaxf(m, floorf(pm)), f = m == mn ? 1.0f : fast_exp2(m - mn);
        l *= f;
#pragma unroll
        for (int mb = 0; mb < 8; ++mb) {
          tot[mb][0] *= f;
          tot[mb][1] *= f;
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[mb][k] *= f;
        }
        m = mn;
      }
      const float mr = m == -INFINITY ? 0.0f : m, wr = mr - static_cast<float>(ev - er);
      l += fast_exp2(l0 - mr) + fast_exp2(l1 - mr);
      const float w0 = fast_exp2(l0 - wr), w1 = fast_exp2(l1 - wr);
      const uint32_t hi = pack_half2(w0, w1);
      const uint32_t lo = pack_half2((w0 - half_lo(hi)) * 2048.0f, (w1 - half_hi(hi)) * 2048.0f);
      const uint32_t p0 = movmatrix_trans(__byte_perm(hi, lo, 0x5410));
      const uint32_t p1 = movmatrix_trans(__byte_perm(hi, lo, 0x7632));
      if (meta.z & 2u) {       // NaN codes among the values: hidden tokens' must not reach the sum
        const uint32_t keep = (visible(2 * t) ? 0xffu : 0u) | (visible(2 * t + 1) ? 0xff00u : 0u) |
                              (visible(2 * t + 8) ? 0xff0000u : 0u) | (visible(2 * t + 9) ? 0xff000000u : 0u);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          vw[k] = make_uint4(vw[k].x & keep, vw[k].y & keep, vw[k].z & keep, vw[k].w & keep);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mma_f16(acc[2 * k], fp8_lo(vw[k].x), fp8_lo(vw[k].y), fp8_hi(vw[k].x), fp8_hi(vw[k].y), p0, p1);
        mma_f16(acc[2 * k + 1], fp8_lo(vw[k].z), fp8_lo(vw[k].w), fp8_hi(vw[k].z), fp8_hi(vw[k].w), p0, p1);
      }
      if (i % kFlush == kFlush - 1) flush();
    }
    if (i < count) {
      // stage i gave up; it and the stages issued after it may still be in flight
      for (int j = i; j < count && j < i + kStages; ++j)
        mbar_drain(smem_u32(&sm.bar[warp][(used + j) % kStages]), ((used + j) / kStages) & 1);
    }
    used += count;
    flush();
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);

    // the warps' states, each in a stage of its own ring (its copies have landed), then joined
    float* mine = reinterpret_cast<float*>(sm.ring[warp][(used + kStages - 1) % kStages]);
    if (lane == 0) sm.state[warp] = (used + kStages - 1) % kStages;
    if (t < a.G) {
#pragma unroll
      for (int mb = 0; mb < 8; ++mb) {
        mine[t * kDim + 16 * mb + g] = tot[mb][0];
        mine[t * kDim + 16 * mb + 8 + g] = tot[mb][1];
      }
      if (g == 0) {
        sm.m[warp][t] = m;
        sm.l[warp][t] = l;
      }
    }
    // where the joined state goes
    const int units = max(s.pages, 1);
    const long long item = first_page();
    whole = j0 == 0 && j1 == units;
    to = whole ? a.out + (static_cast<size_t>(b) * a.H + kv * a.G) * kDim
               : a.part + static_cast<size_t>(2 * blockIdx.x + (j0 == 0 ? 1 : 0)) * kMaxG * kPartStride;
    if (tid == 0 && j0 > 0)     // an item that CTAs before this one began: what joining it takes
      a.cuts[blockIdx.x] = make_int4(b, kv, static_cast<int>(item / line.per),
                                     static_cast<int>((item + units - 1) / line.per));
    cur = item + j1;
    have = true;
  }
  dependents_begin();
}

// Joins the partial states of the items that range borders cut.  CTA (x, h): border behind range
// x, head h; the item's first border does the work.
__global__ void __launch_bounds__(kDim) join_fp8_kernel(const __grid_constant__ Fp8DecodeArgs a) {
  __shared__ float f[kMaxCtas], red[3][4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y;
  dependency_wait();
  const int4 c = a.cuts[blockIdx.x + 1];
  if (c.x < 0 || c.z != static_cast<int>(blockIdx.x)) return;
  const int parts = c.w - c.z + 1;
  // part i: CTA first + i left it, the first one in its second slot
  auto part = [&](int i) {
    return a.part + (static_cast<size_t>(2 * (c.z + i) + (i == 0 ? 1 : 0)) * kMaxG + h) * kPartStride;
  };
  float M = -INFINITY, U = 0.0f, L = 0.0f;
  for (int i = tid; i < parts; i += kDim) {
    M = fmaxf(M, part(i)[0]);
    U = fmaxf(U, part(i)[2]);
  }
  auto all = [&](float x, int which, bool sum) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      x = sum ? x + y : fmaxf(x, y);
    }
    if (lane == 0) red[which][warp] = x;
    __syncthreads();
    return sum ? (red[which][0] + red[which][1]) + (red[which][2] + red[which][3])
               : fmaxf(fmaxf(red[which][0], red[which][1]), fmaxf(red[which][2], red[which][3]));
  };
  M = all(M, 0, false);
  U = all(U, 1, false);
  for (int i = tid; i < parts; i += kDim) {
    const float x = part(i)[0], lw = part(i)[1], g = x == M ? 1.0f : fast_exp2(x - M);
    L += lw == 0.0f ? 0.0f : g * lw;
    f[i] = lw == 0.0f ? 0.0f : g * fast_exp2(part(i)[2] - U);
  }
  L = all(L, 2, true);        // its barrier is also that of f
  float o = 0.0f;
#pragma unroll 8
  for (int i = 0; i < parts; ++i) o = fmaf(f[i], part(i)[4 + tid], o);
  a.out[(static_cast<size_t>(c.x) * a.H + c.y * a.G + h) * kDim + tid] =
      L == 0.0f ? 0.0f : o / L * fast_exp2(U);
}

int grid_of(int num_sms) {
  const int n = num_sms * kCtasPerSm;
  return n < kMaxCtas ? n : kMaxCtas;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

Fp8DecodeWs fp8_decode_ws_layout(int num_sms) {
  Fp8DecodeWs w;
  const size_t ctas = grid_of(num_sms);
  w.cuts_off = 0;
  w.part_off = up256(ctas * sizeof(int4));
  w.total = w.part_off + up256(ctas * 2 * kMaxG * kPartStride * sizeof(float));
  return w;
}

cudaError_t launch_fp8_decode(const Fp8DecodeArgs& a, int num_sms, cudaStream_t st) {
  static bool attr_set[64] = {};       // per device: the attributes are per context
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(decode_fp8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(Smem)));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(decode_fp8_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               static_cast<int>(cudaSharedmemCarveoutMaxShared));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int grid = grid_of(num_sms);
  e = launch_dependent(decode_fp8_kernel, dim3(grid), dim3(kThreads), sizeof(Smem), st, a);
  if (e == cudaSuccess && grid > 1)
    e = launch_dependent(join_fp8_kernel, dim3(grid - 1, a.G), dim3(kDim), 0, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvq
