// qs_sample.cu -- a token for each row of logits: temperature, top-k, top-p, min-p,
// and a draw from the weights that are left, by a given uniform number.
//
// Source: "QuantSpec Guide: Self-Speculative Decoding & Quantized KV", "The
// Self-Speculative Verification Loop": drafted and emitted tokens are drawn from
// the models' distributions, which the acceptance test takes too.
//
// Mathematics.  In the order of falling logits (equal ones by rising index) every
// filter keeps a front part, so what all of them leave is a front part too: the
// logits above some value t, and those equal to t up to some index.  Top-k and
// top-p ask for the element at which a running sum (of ones, of weights) reaches a
// target; it is found with a histogram over the logits' range whose bin is then sorted
// (or, where it holds too much, spread over a histogram of its own).  The draw is the
// same question in the order of the indices.
//
// Two ways are shorter, and taken where they lead to the end.  A small top-k: of the
// 512 threads of each CTA every one knows the largest of its logits, and the k-th
// largest of those is a lower bound for the k-th largest logit, with little above it
// but what is asked for; that little is sorted and the rest done by one CTA.  Top-p
// over everything: one pass adds the weights, exactly, and makes a histogram of them
// rounded to 2^-30; a second adds exactly what stands in front of the bin that
// it names and collects the bin.  If the bin is the wrong one, or too full, the long
// way is taken.
//
// Which token that is hangs on sums of up to 400 thousand weights compared with a
// border, so the weights are formed to about 2^-36 (twofold fp32, with a table of
// 2^(-i / 16)) and added as 64-bit integers of 2^-44: sums that no order changes.
//
// A row is shared by a cluster of CTAs, each of which holds a slice of it in shared
// memory: the logits come from memory once.
//
// Bound by latency for a row or few (32,000 logits, top-k 50: 14.2 us, eight steps that
// wait for one another), by instructions for many: 60 rows of 128,000 with top-p and
// probabilities 107 to 127 us by the logits' values, some 250 instructions a logit, 90 of
// them the first pass's exact weight; 257 rows of 65,537 with mixed settings 111 to 121.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "qs_common.cuh"

namespace cg = cooperative_groups;

namespace qs {
namespace {

typedef unsigned long long u64;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kThreads = 512, kWarpsS = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kCap = 1024;        // candidates that are sorted at once
constexpr int kQueue = 32 + 32 * 8;  // places that a warp collects
constexpr int kMaxC = 8;          // CTAs to a row at most
constexpr int kSmallK = 512;      // top-k at most for the short way
constexpr int kFew = 128;         // candidates that are put in order by counting
constexpr int kFewInBin = 256;    // ... of a bin
constexpr int kUnit = 44;         // a weight of 1 is 2^44
constexpr int kOutline = 14;      // an outline of the weights is in multiples of 2^14
constexpr float kNone = -INFINITY;

struct SampleArgs {
  const void *logits;
  int V, C;
  long long stride;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t *top_k;
  int32_t *token;
  float *probs;
  int list_off, hist_off, part_off, queue_off;  // in dynamic shared memory, behind the slice
};

// 2^(j / 16) 2^44 for j = 0 .. 15, rounded.
struct Pow2Table {
  u64 v[16];
};
constexpr Pow2Table make_table() {
  Pow2Table t{};
  double r = 1.0;
  for (int j = 0; j < 16; ++j, r *= 1.0442737824274138403)  // 2^(1/16)
    t.v[j] = (u64)(r * 17592186044416.0 + 0.5);
  return t;
}
__constant__ Pow2Table c_pow2 = make_table();
// The table in shared memory: entry i is 2^(-i / 16) 2^44, down to a weight of 2^-46.
constexpr int kPow2 = 16 * 46 + 1;
__device__ __forceinline__ u64 pow2_entry(int i) {
  const int sh = (i + 15) >> 4;  // (rounded: half a unit before the shift)
  return (c_pow2.v[-i & 15] + (sh ? 1ull << (sh - 1) : 0)) >> sh;
}

// A row's weights: w = 2^(c (x - m)), c = log2(e) / T.
struct Weights {
  float half_m, c_hi, c_lo;  // m / 2; 2 c in two parts
  bool flat;                 // every kept logit weighs 1 (the largest is +inf)
  const u64 *pow2;           // the table

  // w = 2^(-i / 16) (1 + q 2^-36); false for less than `least` (a power of 2, as its
  // logarithm)
  __device__ __forceinline__ bool parts(float x, float least, int &i, int &q) const {
    // (x - m) / 2 in two parts: halves, so that no finite logits overflow
    const float a = 0.5f * x, s = __fsub_rn(a, half_m), bb = __fsub_rn(s, a);
    const float e = __fsub_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fadd_rn(half_m, bb));
    const float ph = __fmul_rn(s, c_hi);
    if (!(ph > least)) return false;
    const float pl = __fmaf_rn(s, c_hi, -ph) + __fmaf_rn(s, c_lo, e * c_hi);
    // the exponent to the nearest 1 / 16, and the rest
    const float magic = 786432.f, t = __fadd_rn(ph, magic), r = __fsub_rn(ph, __fsub_rn(t, magic));
    i = __float_as_int(magic) - __float_as_int(t);
    // 2^(r + pl) - 1 = z + z^2 / 2 + ..., z = (r + pl) ln 2, |r| <= 1 / 32
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.9046542121259336e-9f;
    const float z = __fmul_rn(r, kLn2);
    const float zl = __fmaf_rn(r, kLn2, -z) + __fmaf_rn(r, kLn2Lo, pl * kLn2);
    const float h = z * z * (0.5f + z * (0.16666667f + z * (0.041666668f + z * 0.0083333338f)));
    q = __float2int_rn(z * 68719476736.f) + __float2int_rn((zl + (h + z * zl)) * 68719476736.f);  // 2^36
    return true;
  }
  static __device__ __forceinline__ u64 combine(u64 t, int q) {
    return t + (u64)(((long long)(int)(t >> 14) * q + (1ll << 21)) >> 22);
  }
  // in units of 2^-44, rounded; 0 for less than 2^-46
  __device__ __forceinline__ u64 operator()(float x) const {
    if (flat) return 1ull << kUnit;
    int i, q;
    if (!parts(x, -45.9f, i, q)) return 0;
    return combine(pow2[i], q);
  }
  // times scale, as a float; 0 for less than 2^-107 (a share in up to QS_MAX_VOCAB
  // weights is a normal number down to there)
  __device__ __forceinline__ float scaled(float x, float scale) const {
    if (flat) return scale;
    int i, q;
    if (!parts(x, -107.f, i, q)) return 0.f;
    const u64 w = combine(pow2[i & 15], q);
    return (float)w * 5.684341886080802e-14f * scale * __int_as_float((127 - (i >> 4)) << 23);
  }
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Floats as integers of the same order (no NaN; zeros carry no sign here).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// floor(x y) for y in [0, 1)
__device__ __noinline__ u64 part_of(u64 x, float y) {
  if (!(y > 0.f)) return 0;
  int e;
  const u64 m = (u64)(frexpf(y, &e) * 16777216.f);  // y = m 2^(e - 24)
  const int k = 24 - e;                             // >= 24
  const u64 lo = x * m, hi = __umul64hi(x, m);
  if (k >= 128) return 0;
  return k >= 64 ? (k == 64 ? hi : hi >> (k - 64)) : (lo >> k) | (hi << (64 - k));
}

struct Shared {
  float mx, mn, mt;       // of the slice: largest, smallest; the smallest of the threads' largest
  float rmx, rmn;         // of the bin that is spread again
  u64 total[2][2];        // sums of a pass over the slice (one pass, and the next)
  u64 front, in_bin;      // in front of a bin, and in it
  float top_p, min_p, u;  // of the row, read by the first CTA for all
  int top_k;
  u64 scan[kWarpsS], part[kWarpsS];
  float fred[3][kWarpsS];
  u64 pow2[kPow2];
  float c_hi, c_lo, x_min_, floor_, below;
  double min_below;       // below the largest logit: the floor, and what min-p keeps
  // what the first CTA found
  int bin, n_list, index;
  u64 before;
  uint32_t n_in_bin;
  float t, x_min, scale;
  int tie, done;
};

template <typename T>
struct Row {
  cg::cluster_group cl;
  Shared &s;
  static constexpr int E = 16 / sizeof(T);  // elements per vector
  const uint4 *slice;  // in vectors; elements outside the slice are NaN
  uint32_t *hist;   // [4][kBins]: three 15-bit limbs of a weight, a count
  u64 *list;        // candidates, ordered for sorting
  uint16_t *queue;  // [warp][kQueue]: see named()
  int rank, C, x0, n_vec;  // element e of vector v is logit x0 + v E + e
  float m;          // the row's largest logit
  bool inf;         // it is +inf
  int tid, lane, warp;
  int pass = 0;     // of sums()

  // f(x, index) for the valid logits of vector v, in order
  template <typename F>
  __device__ __forceinline__ void vec(int v, F &&f) const {
    const uint4 raw = slice[v];
    const T *p = reinterpret_cast<const T *>(&raw);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = __fadd_rn(as_float(p[e]), 0.f);  // (-0 is 0)
      if (x > kNone && (!inf || x == INFINITY)) f(x, x0 + v * E + e);
    }
  }
  // ... and for all of the slice, in any order
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
#pragma unroll 1
    for (int v = tid; v < n_vec; v += kThreads) vec(v, f);
  }

  __device__ __forceinline__ Shared &of(int r) const { return *cl.map_shared_rank(&s, r); }

  // (largest, smallest) over the cluster, through s.rmx / s.rmn
  __device__ void reduce_range(float hi, float lo, float &out_hi, float &out_lo) {
    for (int o = 16; o; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (lane == 0) {
      s.fred[0][warp] = hi;
      s.fred[1][warp] = lo;
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll 1
      for (int k = 1; k < kWarpsS; ++k) {
        hi = fmaxf(hi, s.fred[0][k]);
        lo = fminf(lo, s.fred[1][k]);
      }
      s.rmx = hi;
      s.rmn = lo;
    }
    cluster_sync();
    out_hi = -INFINITY;
    out_lo = INFINITY;
#pragma unroll 1
    for (int r = 0; r < C; ++r) {
      out_hi = fmaxf(out_hi, of(r).rmx);
      out_lo = fminf(out_lo, of(r).rmn);
    }
  }

  // exclusive sum over the CTA's threads
  __device__ __noinline__ u64 scan(u64 v) {
    u64 x = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s.scan[warp] = x;
    __syncthreads();
    u64 before = 0;
#pragma unroll 1
    for (int w = 0; w < warp; ++w) before += s.scan[w];
    return before + x - v;
  }
  __device__ __forceinline__ u64 warp_sum(u64 w) const {
#pragma unroll
    for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    return w;
  }
  // the CTA's sum, for every thread (what it overwrites may still be read: only after
  // a barrier since the last use)
  __device__ __noinline__ u64 block_sum(u64 w) {
    w = warp_sum(w);
    if (lane == 0) s.scan[warp] = w;
    __syncthreads();
    u64 a = 0;
#pragma unroll 1
    for (int k = 0; k < kWarpsS; ++k) a += s.scan[k];
    return a;
  }
  // The cluster's sum of each CTA's own; what the lower ranks have; and the sum of
  // a second number.
  __device__ __noinline__ u64 exchange(u64 own, u64 &before, u64 own2, u64 &total2) {
    // (a CTA may be a pass ahead of one that still reads this sum, never two)
    const int k = pass++ & 1;
    if (tid == 0) {
      s.total[k][0] = own;
      s.total[k][1] = own2;
    }
    cluster_sync();
    // (the sums of all CTAs at once, a lane each)
    const u64 t = lane < C ? of(lane).total[k][0] : 0, t2 = lane < C ? of(lane).total[k][1] : 0;
    before = warp_sum(lane < rank ? t : 0);
    total2 = warp_sum(t2);
    return warp_sum(t);
  }
  __device__ __forceinline__ u64 exchange(u64 own, u64 &before) {
    u64 none;
    return exchange(own, before, 0, none);
  }

  // Sums of weight(x, index) in the order of the indices: the cluster's total, what
  // stands before this CTA's slice, and the slice's own.  A warp takes a run of it.
  __device__ __forceinline__ void run_of(int &v0, int &v1) const {
    const int per = (n_vec + kWarpsS - 1) / kWarpsS;
    v0 = min(n_vec, warp * per);
    v1 = min(n_vec, v0 + per);
  }
  // body(x, index) for the valid logits that take(x, index) names, in any order and by
  // full warps: each warp collects their places in its run of the slice and takes 32
  // at a time.  (Where one in ten is named, almost every warp would go through the body
  // for every logit.)
  template <typename Take, typename Body>
  __device__ __forceinline__ void named(Take &&take, Body &&body) const {
    uint16_t *q = queue + warp * kQueue;
    int v0, v1, count = 0;
    run_of(v0, v1);
    auto work = [&](int from, bool mine) {
      if (!mine || !chk(from + lane < kQueue, 71)) return;
      const int at = q[from + lane];
      if (!chk(at < n_vec * E, 72)) return;
      body(__fadd_rn(as_float(reinterpret_cast<const T *>(slice)[at]), 0.f), x0 + at);
    };
#pragma unroll 1
    for (int b = v0; b < v1; b += 32) {
      const int v = b + lane;
      unsigned hits = 0;
      if (v < v1) {
        const uint4 raw = slice[v];
        const T *p = reinterpret_cast<const T *>(&raw);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float x = __fadd_rn(as_float(p[e]), 0.f);
          if (x > kNone && (!inf || x == INFINITY) && take(x, x0 + v * E + e)) hits |= 1u << e;
        }
      }
      if (!__any_sync(0xffffffffu, hits != 0)) continue;
      const int n = __popc(hits);
      int before = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      const int all = __shfl_sync(0xffffffffu, before, 31);
      uint16_t *to = q + count + before - n;
      for (; hits; hits &= hits - 1)
        if (chk(smem_in(smem_addr(to), 2) && to < q + kQueue && v * E + E <= 65536, 71))
          *to++ = (uint16_t)(v * E + __ffs(hits) - 1);
      count += all;
      __syncwarp();
      while (count >= 32) {
        count -= 32;
        work(count, true);
      }
      __syncwarp();
    }
    work(0, lane < count);
    __syncwarp();
  }

  // The same sums, where only the logits that `take` names weigh anything.
  template <typename Take, typename F>
  __device__ u64 sums_named(Take &&take, F &&weight, u64 &before, u64 &own) {
    u64 w = 0;
    named(take, [&](float x, int) { w += weight(x); });
    return join(w, before, own);
  }
  template <typename F>
  __device__ u64 sums(F &&weight, u64 &before, u64 &own) {
    int v0, v1;
    run_of(v0, v1);
    u64 w = 0;
#pragma unroll 1
    for (int v = v0 + lane; v < v1; v += 32) vec(v, [&](float x, int i) { w += weight(x, i); });
    return join(w, before, own);
  }
  __device__ __noinline__ u64 join(u64 w, u64 &before, u64 &own) {
    w = warp_sum(w);
    __syncthreads();
    if (lane == 0) s.part[warp] = w;
    __syncthreads();
    own = 0;
#pragma unroll 1
    for (int k = 0; k < kWarpsS; ++k) own += s.part[k];
    return exchange(own, before);
  }

  // After sums(): the first index at which the running sum reaches target
  // (1 .. total), known to one thread of the CTA that holds it (-1 elsewhere).
  template <typename F>
  __device__ int locate(F &&weight, u64 before, u64 target) {
    u64 at_ = before;
#pragma unroll 1
    for (int k = 0; k < warp; ++k) at_ += s.part[k];
    if (target <= at_ || target > at_ + s.part[warp]) return -1;
    int v0, v1;
    run_of(v0, v1);
#pragma unroll 1
    for (int b = v0; b < v1; b += 32) {
      u64 p = 0;
      if (b + lane < v1) vec(b + lane, [&](float x, int i) { p += weight(x, i); });
      if (!__any_sync(0xffffffffu, p != 0)) continue;
      u64 x = p;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, at_ + x >= target);
      if (hit) {
        if (lane != __ffs(hit) - 1) return -1;
        at_ += x - p;
        int index = -1;
        vec(b + lane, [&](float y, int i) {
          at_ += weight(y, i);
          if (index < 0 && at_ >= target) index = i;
        });
        return index;
      }
      at_ += __shfl_sync(0xffffffffu, x, 31);
    }
    return -1;
  }

  // Sort list[0, n) (n <= kCap), ascending, in the first CTA.
  __device__ __noinline__ void sort(int n) {
    int p = 32;
    while (p < n) p <<= 1;
    if (!chk(p <= kCap && smem_in(smem_addr(list), 8 * p), 73)) return;
    for (int i = n + tid; i < p; i += kThreads) list[i] = ~0ull;
#pragma unroll 1
    for (int k = 2; k <= p; k <<= 1)
#pragma unroll 1
      for (int j = k >> 1; j; j >>= 1) {
        // (up to 64 elements: one warp does it)
        if (p > 64) __syncthreads(); else if (k == 2) __syncthreads(); else __syncwarp();
        for (int i = tid; i < p / 2; i += kThreads) {
          const int a = ((i & ~(j - 1)) << 1) | (i & (j - 1)), b = a | j;
          const u64 x = list[a], y = list[b];
          if ((x > y) == ((a & k) == 0)) {
            list[a] = y;
            list[b] = x;
          }
        }
      }
    __syncthreads();
  }

  static __device__ __forceinline__ u64 entry(float x, int i) {
    return ((u64)~ordered(x) << 32) | (uint32_t)i;
  }
  static __device__ __forceinline__ float value(u64 e) { return from_ordered(~(uint32_t)(e >> 32)); }

  // Put a logit into the first CTA's list (which holds kCap; all are counted).
  __device__ __forceinline__ void collect(Shared &s0, u64 *list0, float x, int i) const {
    const int k = atomicAdd(&s0.n_list, 1);
    if (k < kCap && chk(smem_in(smem_addr(list + k), 8) && i >= 0, 73)) list0[k] = entry(x, i);
  }

  // In the first CTA: the position in the sorted list at which a running sum of
  // weight(x), starting from `before`, reaches target; n - 1 at the latest.
  template <typename F>
  __device__ int reach(int n, F &&weight, u64 before, u64 target) {
    u64 w[kCap / kThreads], sum = 0;
#pragma unroll
    for (int k = 0; k < kCap / kThreads; ++k) {
      const int i = tid * (kCap / kThreads) + k;
      w[k] = i < n ? weight(value(list[i])) : 0;
      sum += w[k];
    }
    u64 at_ = before + scan(sum);
    if (tid == 0) s.index = n - 1;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kCap / kThreads; ++k) {
      const int i = tid * (kCap / kThreads) + k;
      if (i < n && at_ < target && at_ + w[k] >= target) s.index = i;
      at_ += w[k];
    }
    __syncthreads();
    return s.index;
  }

  // Falling logits from hi on to bins 0 .. kBins - 1: a map that keeps their order
  // and takes hi and lo apart, however far or near they are.
  struct Binning {
    float mul, hi, scale;
    __device__ Binning(float lo, float hi_) {
      const float d = __fsub_rn(hi_, lo);
      mul = d <= 3e38f ? (d < 8.7e-19f ? 1.2676506e30f : 1.f) : 0.5f;  // (2^100: subnormal steps)
      hi = mul * hi_;
      scale = (float)kBins / __fsub_rn(hi, mul * lo);
    }
    __device__ __forceinline__ float before(float x) const { return __fsub_rn(hi, __fmul_rn(mul, x)) * scale; }
    __device__ __forceinline__ int operator()(float x) const {
      return (int)fminf(before(x), (float)(kBins - 1));
    }
  };

  // In the first CTA: s.bin, the bin at which the running sum of w (two bins a thread)
  // from `before` on reaches target, s.before in front of it, s.n_in_bin; -1 if none.
  static constexpr int P = kBins / kThreads;
  __device__ __noinline__ void find_bin(const u64 (&w)[P], const uint32_t (&cnt)[P], u64 before, u64 target) {
    u64 sum = 0;
#pragma unroll
    for (int k = 0; k < P; ++k) sum += w[k];
    u64 at_ = before + scan(sum);
    if (tid == 0) s.bin = -1;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if (at_ < target && at_ + w[k] >= target) {
        s.bin = tid * P + k;
        s.before = at_;
        s.n_in_bin = cnt[k];
      }
      at_ += w[k];
    }
  }

  // One histogram over [lo, hi] of what weight says (of ones where COUNT), and the
  // bin in which the running sum from `before` reaches target, for every thread.
  struct Found {
    int bin;
    u64 before;         // sum in front of the bin
    uint32_t n_in_bin;  // logits in it
  };
  template <bool COUNT, typename F>
  __device__ Found histogram(float lo, float hi, const Binning &bin_of, F &&weight, u64 before,
                             u64 target) {
    for (int i = tid; i < 4 * kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    each([&](float x, int) {
      if (x < lo || x > hi) return;
      const int b = bin_of(x);
      if (!chk(b >= 0 && b < kBins && smem_in(smem_addr(hist + 3 * kBins + b), 4), 74)) return;
      atomicAdd(&hist[3 * kBins + b], 1u);
      if (!COUNT) {
        const u64 w = weight(x);
        atomicAdd(&hist[b], (uint32_t)(w & 0x7FFF));
        atomicAdd(&hist[kBins + b], (uint32_t)(w >> 15) & 0x7FFF);
        atomicAdd(&hist[2 * kBins + b], (uint32_t)(w >> 30));
      }
    });
    cluster_sync();
    if (rank == 0) {
      u64 w[P];
      uint32_t cnt[P];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int b = tid * P + k;
        w[k] = 0;
        cnt[k] = 0;
#pragma unroll 1
        for (int r = 0; r < C; ++r) {
          const uint32_t *h = cl.map_shared_rank(hist, r);
          cnt[k] += h[3 * kBins + b];
          if (!COUNT) w[k] += (u64)h[b] + ((u64)h[kBins + b] << 15) + ((u64)h[2 * kBins + b] << 30);
        }
        if (COUNT) w[k] = cnt[k];
      }
      find_bin(w, cnt, before, target);
      if (tid == 0) s.n_list = 0;
    }
    cluster_sync();
    const Shared &s0 = of(0);
    return Found{s0.bin, s0.before, s0.n_in_bin};
  }

  // The element, in falling order, at which the running sum of weight over the logits
  // in [lo, hi] reaches target: value t and index; false where it does not.
  template <bool COUNT, typename F>
  __device__ __noinline__ bool element(float lo, float hi, F weight, u64 target, float &t, int &tie) {
    u64 before = 0;
#pragma unroll 1
    for (;;) {
      if (lo == hi) {  // equal logits: the one whose turn it is
        const u64 w = COUNT ? 1 : weight(hi);
        const u64 nth = (target - before + w - 1) / w;
        auto eq = [&](float x, int) -> u64 { return x == hi; };
        u64 front, own;
        if (sums(eq, front, own) < nth) return false;
        const int i = locate(eq, front, nth);
        if (i >= 0) of(0).tie = i;
        cluster_sync();
        t = hi;
        tie = of(0).tie;
        return true;
      }
      const Binning bin_of(lo, hi);
      const Found f = histogram<COUNT>(lo, hi, bin_of, weight, before, target);
      if (f.bin < 0) return false;
      before = f.before;
      const float l = lo, h = hi;
      auto in = [=](float x) { return x >= l && x <= h && bin_of(x) == f.bin; };
      if (f.n_in_bin <= kCap) {
        Shared &s0 = of(0);
        u64 *list0 = cl.map_shared_rank(list, 0);
        each([&](float x, int i) {
          if (in(x)) collect(s0, list0, x, i);
        });
        cluster_sync();
        if (rank == 0) {
          const int n = min(s.n_list, kCap);
          sort(n);
          const int i = COUNT ? (int)(target - before) - 1 : reach(n, weight, before, target);
          if (tid == 0) {
            s.t = value(list[i]);
            s.tie = (int)(uint32_t)list[i];
          }
        }
        cluster_sync();
        t = of(0).t;
        tie = of(0).tie;
        return true;
      }
      float a = -INFINITY, b = INFINITY;
      each([&](float x, int) {
        if (in(x)) {
          a = fmaxf(a, x);
          b = fminf(b, x);
        }
      });
      reduce_range(a, b, hi, lo);
    }
  }
};

// The smallest whole number that is at least x y (y in [0, 1)).
__device__ __noinline__ u64 ceil_part_of(u64 x, float y) {
  if (!(y > 0.f)) return 0;
  int e;
  const u64 m = (u64)(frexpf(y, &e) * 16777216.f);
  const int sh = 24 - e;
  const u64 l = x * m, h = __umul64hi(x, m);
  const bool rest = sh >= 128  ? (l | h) != 0
                    : sh > 64  ? l != 0 || (h << (128 - sh)) != 0
                    : sh == 64 ? l != 0
                               : (l << (64 - sh)) != 0;
  return part_of(x, y) + (rest ? 1 : 0);
}
// The running sum that a draw by u asks for: the first above u times the total.
__device__ __forceinline__ u64 draw_target(u64 total, float u) {
  const u64 t = u >= 1.f ? total : part_of(total, u) + 1;
  return t < total ? t : total;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared s;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, row = blockIdx.x / a.C, rank = blockIdx.x % a.C;
  constexpr int E = 16 / sizeof(T);
  const int lane = tid & 31, warp = tid >> 5;
  uint32_t *hist = reinterpret_cast<uint32_t *>(smem + a.hist_off);
  pdl_trigger();
  for (int i = tid; i < kPow2; i += kThreads) s.pow2[i] = pow2_entry(i);
  for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  if (tid == 0) s.n_list = 0;
  pdl_wait();
  // the slice, by whole vectors of memory where they lie inside it
  const int per = (a.V + a.C - 1) / a.C, lo_i = min(a.V, rank * per), hi_i = min(a.V, lo_i + per);
  const T *src = static_cast<const T *>(a.logits) + row * a.stride + lo_i;
  const int n = hi_i - lo_i, first = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  const int n_vec = n ? (n + first + E - 1) / E : 0;
  Row<T> R{cl, s, reinterpret_cast<const uint4 *>(smem), hist, reinterpret_cast<u64 *>(smem + a.list_off),
           reinterpret_cast<uint16_t *>(smem + a.queue_off), rank, a.C, lo_i - first, n_vec, 0.f, false, tid, lane, warp};
  float hi = -INFINITY, lo = INFINITY;
  if (rank == 0 && tid == kThreads - 1) {
    // the row's settings, read once for the whole cluster
    float T_ = a.temperature ? a.temperature[row] : 1.f, min_p = a.min_p ? a.min_p[row] : 0.f;
    s.top_k = a.top_k ? a.top_k[row] : 0;
    s.top_p = a.top_p ? a.top_p[row] : 1.f;
    s.u = a.u[row];
    const bool greedy = !(T_ >= 8.673617379884035e-19f);
    if (greedy) {
      s.top_k = 1;
      T_ = 1.f;
    }
    if (!(min_p > 0.f)) min_p = 0.f;
    // 2 log2(e) / T in two parts, the second from the first one's remainder
    constexpr float kL = 2.885390043258667f, kLLo = 3.851925e-8f;
    const float c_hi = kL / T_, rest = __fmaf_rn(-c_hi, T_, kL) + kLLo;
    s.c_hi = c_hi;
    s.c_lo = T_ < 1e30f ? rest / T_ : 0.f;
    s.below = T_ * 31.8848f;  // 46 ln 2, and a little
    s.min_p = min_p;
    // (64 bits take one thread longer than the rest of it: only where asked for)
    s.min_below = min_p > 0.f && min_p < 1.f ? (double)T_ * log((double)min_p) : 0.0;
  }
  {
    const uint4 *vsrc = reinterpret_cast<const uint4 *>(src - first);
#pragma unroll 1
    for (int v0 = tid; v0 < n_vec; v0 += 4 * kThreads) {
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int v = v0 + k * kThreads;
        if (v >= n_vec || !chk(16 * (v + 1) <= a.hist_off, 70)) continue;
        if (v * E >= first && (v + 1) * E - first <= n) {
          x[k] = vsrc[v];
        } else {  // an end: element by element, NaN outside
          T *p = reinterpret_cast<T *>(smem) + v * E;
          for (int e = 0; e < E; ++e) {
            const int i = v * E + e - first;
            const uint32_t none = ~0u;
            p[e] = i >= 0 && i < n ? src[i] : *reinterpret_cast<const T *>(&none);
          }
          x[k] = reinterpret_cast<const uint4 *>(smem)[v];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int v = v0 + k * kThreads;
        if (v >= n_vec || !chk(16 * (v + 1) <= a.hist_off, 70)) continue;
        reinterpret_cast<uint4 *>(smem)[v] = x[k];
        const T *p = reinterpret_cast<const T *>(&x[k]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float y = __fadd_rn(as_float(p[e]), 0.f);
          if (y > kNone) {
            hi = fmaxf(hi, y);
            lo = fminf(lo, y);
          }
        }
      }
    }
  }
  float *probs = a.probs ? a.probs + (size_t)row * a.V : nullptr;
  const float mine = hi;  // the largest of this thread's logits
  float mn, mt = hi > kNone ? hi : INFINITY;
  {
    for (int o = 16; o; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      mt = fminf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    }
    if (lane == 0) {
      s.fred[0][warp] = hi;
      s.fred[1][warp] = lo;
      s.fred[2][warp] = mt;
    }
    __syncthreads();
    if (probs) {
      // zeros, while the rest is found out; what is kept is written over them at the
      // end, by other threads, many barriers later (and where probs are the logits
      // themselves, this slice has been read)
      float *z = probs + lo_i;
      const int head = min(n, (int)(-(reinterpret_cast<uintptr_t>(z) >> 2) & 3)), quads = (n - head) >> 2;
      if (tid < head) z[tid] = 0.f;
      float4 *z4 = reinterpret_cast<float4 *>(z + head);
      for (int i = tid; i < quads; i += kThreads)
        if (chk(head + 4 * i + 4 <= n && lo_i + n <= a.V, 78)) z4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int i = head + 4 * quads + tid;
      if (i < n) z[i] = 0.f;
    }
    if (warp == 0) {
      hi = lane < kWarpsS ? s.fred[0][lane] : -INFINITY;
      lo = lane < kWarpsS ? s.fred[1][lane] : INFINITY;
      mt = lane < kWarpsS ? s.fred[2][lane] : INFINITY;
      for (int o = 8; o; o >>= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        mt = fminf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      }
      if (lane == 0) {
        s.mx = hi;
        s.mn = lo;
        s.mt = mt;
      }
    }
    cluster_sync();
    const bool has = lane < a.C;
    hi = has ? R.of(lane).mx : -INFINITY;
    mn = has ? R.of(lane).mn : INFINITY;
    mt = has ? R.of(lane).mt : INFINITY;
    for (int o = kMaxC / 2; o; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mt = fminf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    }
    hi = __shfl_sync(0xffffffffu, hi, 0);
    mn = __shfl_sync(0xffffffffu, mn, 0);
    mt = __shfl_sync(0xffffffffu, mt, 0);
  }
  const float m = R.m = hi;
  if (!(m > kNone)) {  // nothing to keep (the whole cluster alike)
    if (rank == 0 && tid == 0) a.token[row] = -1;
    cluster_sync();  // (the others have read this CTA's maximum)
    return;
  }
  R.inf = m == INFINITY;
  if (R.inf) mn = m;
  Shared &s0 = R.of(0);
  float top_p = s0.top_p;
  const float u = s0.u;
  int k = s0.top_k;
  if (k <= 0 || k > a.V) k = a.V;
  if (!(top_p < 1.f)) top_p = 1.f;
  Weights w;
  w.half_m = 0.5f * m;
  w.c_hi = s0.c_hi;
  w.c_lo = s0.c_lo;
  w.flat = R.inf;
  w.pow2 = s.pow2;
  if (tid == 0) {
    // x >= x_min: what min-p keeps.  Logits of weights below 2^-46, under the floor,
    // count as none: no sum or draw asks for them
    const float min_p = s0.min_p;
    s.x_min_ = min_p >= 1.f || (min_p > 0.f && R.inf) ? m
               : min_p > 0.f                          ? __double2float_ru((double)m + s0.min_below)
                                                      : kNone;
    s.floor_ = R.inf ? m : fmaxf(mn, __fsub_rd(m, s0.below));
  }
  __syncthreads();
  const float x_min = s.x_min_, floor_x = s.floor_;

  // what is kept: x > t, or x == t up to index tie; and x >= x_min
  float t = kNone, scale = 0.f;
  int tie = -1;

  bool done = false;  // t, tie, x_min and scale are final, the token is written
  u64 *list0 = cl.map_shared_rank(R.list, 0);
  if (k <= kSmallK && k < a.V && !R.inf && mt < m) {
    // ---- a small top-k: the k-th largest of the threads' largest logits bounds it
    const typename Row<T>::Binning bin_of(mt, m);
    if (mine > kNone && chk(bin_of(mine) >= 0 && bin_of(mine) < kBins, 74))
      atomicAdd(&cl.map_shared_rank(hist, 0)[bin_of(mine)], 1u);
    cluster_sync();
    if (rank == 0) {
      u64 cw[Row<T>::P];
      uint32_t cc[Row<T>::P];
#pragma unroll
      for (int i = 0; i < Row<T>::P; ++i) cw[i] = cc[i] = hist[tid * Row<T>::P + i];
      R.find_bin(cw, cc, 0, (u64)k);
    }
    cluster_sync();
    const int bin = s0.bin;
    const float bin_end = bin == kBins - 1 ? INFINITY : (float)(bin + 1);
    if (bin >= 0) {
      R.each([&](float x, int i) {
        if (x >= mt && bin_of.before(x) < bin_end) R.collect(s0, list0, x, i);
      });
    }
    cluster_sync();
    if (rank == 0) {
      u64 *weight_of = reinterpret_cast<u64 *>(smem + a.part_off);
      const int found = bin >= 0 ? s.n_list : kCap + 1;
      if (found <= kCap) {
        // The first k of them in falling order, thread i the i-th.  Up to kFew of them
        // are put in order by counting, for each, those in front of it
        const bool few = found <= kFew;
        u64 e = 0;
        int place = tid;
        if (few) {
          if (tid < found) {
            e = R.list[tid];
            place = 0;
#pragma unroll 4
            for (int i = 0; i < found; ++i) place += R.list[i] < e;
          }
        } else {
          R.sort(found);
          if (tid < k) e = R.list[tid];
        }
        const bool mine_k = tid < found && place < k;
        const float x = Row<T>::value(e);
        const int index = (int)(uint32_t)e;
        const u64 wx = mine_k ? w(x) : 0;
        if (few) {
          __syncthreads();
          if (mine_k && chk(place < kCap && a.part_off + 8 * (place + 1) <= a.list_off, 75)) {
            R.list[place] = e;
            weight_of[place] = wx;
          }
          __syncthreads();
        } else if (mine_k && chk(a.part_off + 8 * (tid + 1) <= a.list_off, 75)) {
          weight_of[tid] = wx;
        }
        // what stands in front of each, and all together
        u64 before;
        if (few) {
          before = 0;
          u64 all = 0;
#pragma unroll 4
          for (int i = 0; i < k; ++i) {
            const u64 y = weight_of[i];
            all += y;
            if (i < place) before += y;
          }
          if (tid == 0) s.front = all;
          __syncthreads();
        } else {
          before = R.scan(wx);
          if (tid == k - 1) s.front = before + wx;
          __syncthreads();
        }
        bool keep = mine_k && x >= x_min;
        if (top_p < 1.f && keep && place > 0) keep = before < ceil_part_of(s.front, top_p);
        // (a front part: x_min and the target only fall)
        const int kept = __syncthreads_count(keep);
        if (keep && place == kept - 1) {
          s.t = x;
          s.tie = index;
          s.front = before + wx;
        }
        __syncthreads();
        const u64 total = s.front, target = draw_target(total, u);
        // the draw, in the order of the indices
        if (keep) {
          u64 upto = 0;
#pragma unroll 4
          for (int i = 0; i < kept; ++i)
            if ((int)(uint32_t)R.list[i] <= index) upto += weight_of[i];
          if (upto >= target && upto - wx < target) a.token[row] = index;
        }
        if (tid == 0) s.scale = 17592186044416.f / (float)total;
      }
      if (tid == 0) s.done = found <= kCap;
      __syncthreads();
    }
    cluster_sync();
    done = s0.done;
    if (done) {
      t = s0.t;
      tie = s0.tie;
      scale = s0.scale;
    }
  }
  auto in_front = [&](float x, int i) { return x > t || (x == t && i <= tie); };
  if (!done) {
    if (k < a.V) {
      // With fewer than k logits above the floor top-k takes nothing away that weighs
      // anything.  The rest of the k is looked for only where the probabilities tell what
      // is kept down there (one row of 32,000 fp16 logits, top-k 1000 with 190 of them
      // above the floor: 16 us without probabilities, 30 with them).
      const auto one = [](float) -> u64 { return 1; };
      if (!R.template element<true>(k == 1 ? m : floor_x, m, one, (u64)k, t, tie) && probs && top_p >= 1.f &&
          x_min < floor_x && mn < floor_x)
        R.template element<true>(mn, m, one, (u64)k, t, tie);
    }
    if (tie < 0) t = kNone;
    u64 front, own, total = 0;  // of what is kept (0: not known yet)
    if (top_p < 1.f && k > 1) {
      // ---- top-p: the total and an outline of the weights, then the bin it points to
      const float lo_p = fmaxf(floor_x, t);
      bool found = false;
      u64 target = 0;
      if (lo_p < m) {
        const typename Row<T>::Binning bin_of(lo_p, m);
        for (int i = tid; i < 2 * kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
        u64 sum = 0;
        R.each([&](float x, int i) {
          if (x < lo_p || !in_front(x, i)) return;
          const u64 wx = w(x);
          sum += wx;
          // (in units of 2^-30, in two parts: most weights have but one)
          const uint32_t r = (uint32_t)((wx + (1ull << (kOutline - 1))) >> kOutline);
          const int b = bin_of(x);
          if (!chk(b >= 0 && b < kBins, 74)) return;
          if (r & 0x7FFF) atomicAdd(&hist[b], r & 0x7FFF);
          if (r >> 15) atomicAdd(&hist[kBins + b], r >> 15);
        });
        target = ceil_part_of(R.exchange(R.block_sum(sum), front), top_p);
        if (target < 1) target = 1;
        if (rank == 0) {
          u64 bw[Row<T>::P];
          uint32_t none[Row<T>::P] = {};
#pragma unroll
          for (int i = 0; i < Row<T>::P; ++i) {
            uint32_t h0[kMaxC], h1[kMaxC];
#pragma unroll
            for (int r = 0; r < kMaxC; ++r) {
              const uint32_t *h = cl.map_shared_rank(hist, r < a.C ? r : 0) + tid * Row<T>::P + i;
              h0[r] = r < a.C ? h[0] : 0;
              h1[r] = r < a.C ? h[kBins] : 0;
            }
            bw[i] = 0;
#pragma unroll
            for (int r = 0; r < kMaxC; ++r) bw[i] += h0[r] + ((u64)h1[r] << 15);
          }
          R.find_bin(bw, none, 0, max(1ull, target >> kOutline));
          if (tid == 0) s.n_list = 0;
        }
        cluster_sync();
        const int bin = s0.bin;
        u64 above = 0, inside = 0;
        const float bin_end = bin == kBins - 1 ? INFINITY : (float)(bin + 1);
        if (bin >= 0)
          R.named([&](float x, int i) { return bin_of.before(x) < bin_end && x >= lo_p && in_front(x, i); },
                  [&](float x, int i) {
                    const u64 wx = w(x);
                    if (bin_of(x) < bin) {
                      above += wx;
                    } else {
                      inside += wx;
                      R.collect(s0, list0, x, i);
                    }
                  });
        // (a warp's share is that of its run of the slice, as the draw wants it)
        above = R.warp_sum(above);
        if (lane == 0) s.part[warp] = above;
        u64 sum_i;
        const u64 own_a = R.block_sum(lane == 0 ? above : 0);
        __syncthreads();
        const u64 sum_a = R.exchange(own_a, front, R.block_sum(inside), sum_i);
        const int n_list = s0.n_list;
        found = bin >= 0 && n_list <= kCap && sum_a < target && target <= sum_a + sum_i;
        if (found && rank == 0) {
          if (n_list <= kFewInBin) {
            // a thread each: the one whose turn it is knows it from those in front of it
            u64 *weight_of = reinterpret_cast<u64 *>(smem + a.part_off);
            u64 e = 0, wx = 0, before = sum_a;
            if (tid < n_list && chk(a.part_off + 8 * (tid + 1) <= a.list_off, 75)) {
              e = R.list[tid];
              weight_of[tid] = wx = w(Row<T>::value(e));
            }
            __syncthreads();
            if (tid < n_list) {
#pragma unroll 4
              for (int i = 0; i < n_list; ++i)
                if (R.list[i] < e) before += weight_of[i];
              if (before < target && target <= before + wx) {
                s.t = Row<T>::value(e);
                s.tie = (int)(uint32_t)e;
                s.front = before + wx;
              }
            }
          } else {
            R.sort(n_list);
            const int at = R.reach(n_list, w, sum_a, target);
            if (tid == 0) {
              s.t = Row<T>::value(R.list[at]);
              s.tie = (int)(uint32_t)R.list[at];
              s.front = 0;
            }
          }
        }
        cluster_sync();
        if (found) {
          t = s0.t;
          tie = s0.tie;
          // Where min-p takes nothing more, the draw's sums are known but for the bin's
          // share in them: of the slices in front, and of this one's warps.
          const u64 all = s0.front;
          if (all && !(x_min > t)) {
            const int per_warp = max(1, (n_vec + kWarpsS - 1) / kWarpsS);
            u64 f = 0;
            if (tid < n_list) {
              const u64 e = list0[tid];
              const float x = Row<T>::value(e);
              const int i = (int)(uint32_t)e;
              if (i < hi_i && in_front(x, i)) {
                const u64 wx = w(x);
                if (i < lo_i) f = wx;
                else if (chk((i - R.x0) / E / per_warp < kWarpsS, 77)) atomicAdd(&s.part[(i - R.x0) / E / per_warp], wx);
              }
            }
            front += R.block_sum(f);
            total = all;
          }
        }
      } else {
        // all equal: so many of them
        target = ceil_part_of(
            R.sums([&](float x, int i) -> u64 { return in_front(x, i) ? w(x) : 0; }, front, own), top_p);
        if (target < 1) target = 1;
      }
      if (!found) R.template element<false>(lo_p, m, w, target, t, tie);
    }
    auto kept = [&](float x, int i) -> u64 { return x >= x_min && in_front(x, i) ? w(x) : 0; };
    if (!total)
      total = R.sums_named([&](float x, int i) { return x >= x_min && x >= floor_x && in_front(x, i); }, w, front, own);
    const int index = R.locate(kept, front, draw_target(total, u));
    if (index >= 0) a.token[row] = index;
    scale = 17592186044416.f / (float)total;
  }
  if (probs)
    R.named([&](float x, int i) { return x >= x_min && in_front(x, i); },
            [&](float x, int i) {
              if (chk(i >= 0 && i < a.V, 78)) probs[i] = w.scaled(x, scale);
            });
  cluster_sync();  // the others have read this CTA's sums
}

template <typename T>
qs_status launch_sample(const SampleArgs &a, int rows, int smem, cudaStream_t st) {
  static int mask = 0;
  const qs_status s = set_smem_once((const void *)sample_kernel<T>, 227 * 1024 - (int)sizeof(Shared) - 1024, &mask);
  if (s != QS_OK) return s;
  return launch_pdl_cluster(sample_kernel<T>, dim3((unsigned)rows * a.C), dim3(kThreads), a.C, smem, st, a);
}

}  // namespace
}  // namespace qs

using namespace qs;

extern "C" qs_status qs_sample(const void *logits, qs_dtype dtype, int32_t rows, int32_t V,
                               int64_t row_stride, const float *temperature, const int32_t *top_k,
                               const float *top_p, const float *min_p, const float *u, int32_t *token,
                               float *probs, qs_stream_t stream) {
  if (!logits || !u || !token || rows < 1 || V < 1) return QS_ERR_ARG;
  if (dtype != QS_FP16 && dtype != QS_BF16 && dtype != QS_FP32) return QS_ERR_ARG;
  if (rows > 1 && row_stride < V) return QS_ERR_ARG;
  if (V > QS_MAX_VOCAB || rows > (1 << 24)) return QS_ERR_UNSUPPORTED;
  const int size = dtype == QS_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size) return QS_ERR_ALIGN;
  const void *ptrs[] = {temperature, top_k, top_p, min_p, u, token, probs};
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % 4) return QS_ERR_ALIGN;
  // probabilities are written while other rows' logits may still be read: only row on row
  if (probs && !(probs == logits && dtype == QS_FP32 && (rows == 1 || row_stride == V))) {
    // the first row that ends behind the start of probs
    const intptr_t step = rows > 1 ? row_stride * size : 0, len = (intptr_t)V * size;
    const intptr_t behind = reinterpret_cast<intptr_t>(probs) - reinterpret_cast<intptr_t>(logits) - len;
    const intptr_t r = behind < 0 || step == 0 ? 0 : behind / step + 1;
    if (r < rows && overlap(probs, sizeof(float) * V * rows, static_cast<const char *>(logits) + r * step, len))
      return QS_ERR_ARG;
  }
  SampleArgs a = {logits, V, 1, rows > 1 ? row_stride : 0, temperature, top_p, min_p, u, top_k, token,
                  probs, 0, 0, 0, 0};
  // CTAs to a row: so many that two fit an SM (slices of 64 KB), and more while every
  // CTA has an SM of its own and 4096 logits or more.  Measured, 1 / 2 / 4 / 8 CTAs: one row
  // of 32,000 fp16 17.2 / 15.1 / 13.9 / 14.5 us; 30 of 128,000 bf16 with top-p and
  // probabilities (4 / 8) 116 / 81; 60 of them (4 / 5 / 8) 123 / 142 / 144; 257 of 65,537
  // fp32 (4 / 6 / 8) 117 / 153 / 182.  (Taken before the second pass left the draw's sums.)
  int sms = 0;
  const qs_status st0 = sm_count(&sms);
  if (st0 != QS_OK) return st0;
  while (a.C < kMaxC && (long long)V * size > 66 * 1024 * a.C) a.C *= 2;
  while (a.C < kMaxC && (long long)rows * a.C <= sms && V > 8192 * a.C) a.C *= 2;
  const int per = (V + a.C - 1) / a.C;
  a.hist_off = (per * size + 32 + 127) / 128 * 128;
  // (the candidates' weights take room of a histogram: no step has both)
  static_assert(kSmallK * 8 <= 3 * kBins * 4, "");
  a.part_off = a.hist_off + kBins * 4;
  a.list_off = a.hist_off + 4 * kBins * 4;
  a.queue_off = a.list_off + kCap * 8;
  const int smem = a.queue_off + kWarpsS * kQueue * 2;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == QS_FP32) return launch_sample<float>(a, rows, smem, st);
  if (dtype == QS_FP16) return launch_sample<__half>(a, rows, smem, st);
  return launch_sample<__nv_bfloat16>(a, rows, smem, st);
}

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_sample(unsigned long long *out2, int reset) {
  return read_check_failures(out2, reset);
}
#endif
