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
// target; it is found with histograms over the logits' range, each one's bin then
// sorted (or, where it holds too much, spread over a histogram of its own).  The
// draw is the same question in the order of the indices.
//
// Which token that is hangs on sums of up to 400 thousand weights compared with a
// border, so the weights are formed to about 2^-36 (twofold fp32, with a table of
// 2^(j / 32)) and added as 64-bit integers of 2^-44: sums that no order changes.
//
// A row is shared by a cluster of CTAs, each of which holds a slice of it in shared
// memory: the logits come from memory once.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "qs_common.cuh"

namespace cg = cooperative_groups;

namespace qs {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512, kWarpsS = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kCap = 1024;        // candidates that are sorted at once
constexpr int kMaxC = 8;          // CTAs to a row at most
constexpr int kMaxSlice = QS_MAX_VOCAB / kMaxC;
constexpr int kMaxIter = (kMaxSlice * 4 / 16 + 1 + kThreads - 1) / kThreads + 1;
constexpr int kUnit = 44;         // a weight of 1 is 2^44
constexpr float kNone = -INFINITY;

struct SampleArgs {
  const void *logits;
  int V, C;
  long long stride;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t *top_k;
  int32_t *token;
  float *probs;
  int list_off, hist_off;  // in dynamic shared memory, behind the slice
};

// 2^(j / 32) 2^44 for j = -16 .. 16, rounded.
struct Pow2Table {
  u64 v[33];
};
constexpr double root2_32(int j) {
  double r = 1.0;
  const double s = 1.0218971486541166782;  // 2^(1/32)
  for (int i = 0; i < (j < 0 ? -j : j); ++i) r *= s;
  return j < 0 ? 1.0 / r : r;
}
constexpr Pow2Table make_table() {
  Pow2Table t{};
  for (int j = -16; j <= 16; ++j) t.v[j + 16] = (u64)(root2_32(j) * 17592186044416.0 + 0.5);
  return t;
}
__constant__ Pow2Table c_pow2 = make_table();

// A row's weights: w = 2^(c (x - m)), c = log2(e) / T.
struct Weights {
  float half_m, c_hi, c_lo;  // m / 2; 2 c in two parts
  bool flat;                 // every kept logit weighs 1 (the largest is +inf)
  const u64 *pow2;           // the table, in shared memory

  // w = W 2^n, W of 2^44; W = 0 for less than 2^-64.
  __device__ __forceinline__ u64 mantissa(float x, int &n) const {
    n = 0;
    if (flat) return 1ull << kUnit;
    // (x - m) / 2 in two parts: halves, so that no finite logits overflow
    const float a = 0.5f * x, s = __fsub_rn(a, half_m), bb = __fsub_rn(s, a);
    const float e = __fsub_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fadd_rn(half_m, bb));
    const float ph = __fmul_rn(s, c_hi);
    if (!(ph > -64.f)) return 0;
    const float pl = __fmaf_rn(s, c_hi, -ph) + __fmaf_rn(s, c_lo, e * c_hi);
    const float nf = rintf(ph), f = __fsub_rn(ph, nf), jf = rintf(f * 32.f);
    const float r = __fmaf_rn(jf, -0.03125f, f);  // exact, up to 1/64
    n = (int)nf;
    // 2^(r + pl) - 1 = z + z^2 / 2 + ..., z = (r + pl) ln 2
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.9046542121259336e-9f;
    const float z = __fmul_rn(r, kLn2);
    const float zl = __fmaf_rn(r, kLn2, -z) + __fmaf_rn(r, kLn2Lo, pl * kLn2);
    const float h = z * z * (0.5f + z * (0.16666667f + z * (0.041666668f + z * 0.0083333338f)));
    const float lo = zl + (h + z * zl);
    const int q = __float2int_rn(z * 137438953472.f) + __float2int_rn(lo * 137438953472.f);  // 2^37
    const u64 t = pow2[(int)jf + 16];
    return t + (u64)(((long long)(int)(t >> 14) * q) >> 23);
  }
  __device__ __forceinline__ u64 operator()(float x) const {  // in units of 2^-44, rounded
    int n;
    const u64 w = mantissa(x, n);
    return n >= 0 ? w << n : n > -60 ? (w + (1ull << (-n - 1))) >> -n : 0;
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
__device__ __forceinline__ u64 part_of(u64 x, float y) {
  if (!(y > 0.f)) return 0;
  int e;
  const u64 m = (u64)(frexpf(y, &e) * 16777216.f);  // y = m 2^(e - 24)
  const int k = 24 - e;                             // >= 24
  const u64 lo = x * m, hi = __umul64hi(x, m);
  if (k >= 128) return 0;
  return k >= 64 ? (k == 64 ? hi : hi >> (k - 64)) : (lo >> k) | (hi << (64 - k));
}

struct Shared {
  float mx, mn;           // of the slice
  float rmx, rmn;         // of the bin that is spread again
  u64 total[2];           // sum of a pass over the slice (one pass, and the next)
  float temperature, top_p, min_p, u;  // of the row, read by the first CTA for all
  int top_k;
  u64 part[kMaxIter][kWarpsS];
  u64 scan[kWarpsS];
  float fred[2][kWarpsS];
  u64 pow2[33];
  // what the first CTA found
  int bin, n_list, index;
  u64 before, in_bin;
  uint32_t n_in_bin, n_upto;
  float t;
  int tie;
};

template <typename T>
struct Row {
  static constexpr int E = 16 / sizeof(T);  // elements per vector
  cg::cluster_group cl;
  Shared &s;
  uint8_t *slice;   // 16-byte vectors; elements outside the slice are NaN
  uint32_t *hist;   // [4][kBins]: three 15-bit limbs of a weight, a count
  u64 *list;        // candidates, ordered for sorting
  int rank, C, x0, n_vec, first;  // index of element e of vector v: x0 + v E + e - first
  float m;          // the row's largest logit
  bool inf;         // it is +inf
  int tid, lane, warp;
  int pass = 0;     // of sums()

  // f(x, index) for the valid logits of vector v
  template <typename F>
  __device__ __forceinline__ void vec(int v, F &&f) const {
    const uint4 raw = reinterpret_cast<const uint4 *>(slice)[v];
    const T *p = reinterpret_cast<const T *>(&raw);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = __fadd_rn(as_float(p[e]), 0.f);  // (-0 is 0)
      if (x > kNone && (!inf || x == INFINITY)) f(x, x0 + v * E + e - first);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F &&f) const {
    for (int v = tid; v < n_vec; v += kThreads) vec(v, f);
  }

  __device__ __forceinline__ Shared &of(int r) const { return *cl.map_shared_rank(&s, r); }

  // (largest, smallest) over the cluster, through s.mx / s.mn or s.rmx / s.rmn
  __device__ void reduce_range(float hi, float lo, float Shared::*a, float Shared::*b, float &out_hi,
                               float &out_lo) {
    for (int o = 16; o; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (lane == 0) {
      s.fred[0][warp] = hi;
      s.fred[1][warp] = lo;
    }
    __syncthreads();
    if (warp == 0) {
      hi = lane < kWarpsS ? s.fred[0][lane] : -INFINITY;
      lo = lane < kWarpsS ? s.fred[1][lane] : INFINITY;
      for (int o = 16; o; o >>= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      }
      if (lane == 0) {
        s.*a = hi;
        s.*b = lo;
      }
    }
    cl.sync();
    out_hi = -INFINITY;
    out_lo = INFINITY;
    for (int r = 0; r < C; ++r) {
      out_hi = fmaxf(out_hi, of(r).*a);
      out_lo = fminf(out_lo, of(r).*b);
    }
  }

  // exclusive sum over the CTA's threads
  __device__ u64 scan(u64 v) {
    u64 x = v;
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s.scan[warp] = x;
    __syncthreads();
    u64 before = 0;
    for (int w = 0; w < warp; ++w) before += s.scan[w];
    return before + x - v;
  }

  // Sums of weight(x, index) in the order of the indices: the cluster's total, what
  // stands before this CTA's slice, and the slice's own.
  template <typename F>
  __device__ u64 sums(F &&weight, u64 &before, u64 &all) {
    u64 mine = 0;
    for (int it = 0; it * kThreads < n_vec; ++it) {
      u64 w = 0;
      const int v = it * kThreads + tid;
      if (v < n_vec) vec(v, [&](float x, int i) { w += weight(x, i); });
      for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      if (lane == 0) s.part[it][warp] = w;
      mine += w;
    }
    if (lane == 0) s.scan[warp] = mine;  // (every lane of a warp holds its sum)
    __syncthreads();
    all = 0;
    for (int w = 0; w < kWarpsS; ++w) all += s.scan[w];
    // (a CTA may be a pass ahead of one that still reads this sum, never two)
    const int at = pass++ & 1;
    if (tid == 0) s.total[at] = all;
    cl.sync();
    u64 total = 0;
    before = 0;
    for (int r = 0; r < C; ++r) {
      const u64 t = of(r).total[at];
      if (r < rank) before += t;
      total += t;
    }
    return total;
  }

  // After sums(): the first index at which the running sum reaches target
  // (1 .. total), known to the CTA that holds it (-1 elsewhere, in every thread but one).
  template <typename F>
  __device__ int locate(F &&weight, u64 before, u64 all, u64 target) {
    if (target <= before || target > before + all || warp != 0) return -1;
    u64 at = before;
    int it = 0, w = 0;
    for (;; ++it) {  // (the sums of an iteration's warps, a lane each)
      u64 p = lane < kWarpsS ? s.part[it][lane] : 0, x = p;
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, at + x >= target);
      if (hit) {
        w = __ffs(hit) - 1;
        at += __shfl_sync(0xffffffffu, x - p, w);
        break;
      }
      at += __shfl_sync(0xffffffffu, x, 31);
    }
    const int v = it * kThreads + w * 32 + lane;
    u64 p = 0, x;
    if (v < n_vec) vec(v, [&](float y, int i) { p += weight(y, i); });
    x = p;
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at + x >= target);
    if (lane != __ffs(hit) - 1) return -1;
    at += x - p;
    int index = -1;
    vec(v, [&](float y, int i) {
      at += weight(y, i);
      if (index < 0 && at >= target) index = i;
    });
    return index;
  }

  // Sort list[0, n) (n <= kCap), ascending, in the first CTA.
  __device__ void sort(int n) {
    int p = 32;
    while (p < n) p <<= 1;
    for (int i = n + tid; i < p; i += kThreads) list[i] = ~0ull;
    for (int k = 2; k <= p; k <<= 1)
      for (int j = k >> 1; j; j >>= 1) {
        __syncthreads();
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

  // Put the valid logits for which take(x) holds into the first CTA's list (their
  // number is known to be at most kCap), sorted.  Ends with the first CTA alone
  // knowing it.
  template <typename F>
  __device__ int gather(F &&take) {
    if (rank == 0 && tid == 0) s.n_list = 0;
    cl.sync();
    Shared &s0 = of(0);
    u64 *list0 = cl.map_shared_rank(list, 0);
    each([&](float x, int i) {
      if (take(x)) {
        const int at = atomicAdd(&s0.n_list, 1);
        if (at < kCap) list0[at] = entry(x, i);
      }
    });
    cl.sync();
    if (rank != 0) return 0;
    const int n = min(s.n_list, kCap);
    sort(n);
    return n;
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
    u64 at = before + scan(sum);
    if (tid == 0) s.index = n - 1;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kCap / kThreads; ++k) {
      const int i = tid * (kCap / kThreads) + k;
      if (i < n && at < target && at + w[k] >= target) s.index = i;
      at += w[k];
    }
    __syncthreads();
    return s.index;
  }

  // One histogram over [lo, hi] of what weight says (of ones where COUNT), and the
  // bin in which the running sum from `before` reaches target.  Every thread of the
  // cluster gets the answer.
  struct Found {
    int bin;
    u64 before, in_bin;      // sum in front of the bin, and in it
    uint32_t n_in_bin, n_upto;  // logits in it, and up to its end within the range
  };
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
    __device__ __forceinline__ int operator()(float x) const {
      return (int)fminf(__fsub_rn(hi, __fmul_rn(mul, x)) * scale, (float)(kBins - 1));
    }
  };
  template <bool COUNT, typename F>
  __device__ Found histogram(float lo, float hi, const Binning &bin_of, F &&weight, u64 before,
                             u64 target) {
    for (int i = tid; i < 4 * kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    each([&](float x, int) {
      if (x < lo || x > hi) return;
      const int b = bin_of(x);
      atomicAdd(&hist[3 * kBins + b], 1u);
      if (!COUNT) {
        const u64 w = weight(x);
        atomicAdd(&hist[b], (uint32_t)(w & 0x7FFF));
        atomicAdd(&hist[kBins + b], (uint32_t)(w >> 15) & 0x7FFF);
        atomicAdd(&hist[2 * kBins + b], (uint32_t)(w >> 30));
      }
    });
    cl.sync();
    if (rank == 0) {
      constexpr int P = kBins / kThreads;
      u64 w[P], sum = 0;
      uint32_t cnt[P];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int b = tid * P + k;
        w[k] = 0;
        cnt[k] = 0;
        for (int r = 0; r < C; ++r) {
          const uint32_t *h = cl.map_shared_rank(hist, r);
          cnt[k] += h[3 * kBins + b];
          if (!COUNT)
            w[k] += (u64)h[b] + ((u64)h[kBins + b] << 15) + ((u64)h[2 * kBins + b] << 30);
        }
        if (COUNT) w[k] = cnt[k];
        sum += w[k];
      }
      uint32_t n = 0;
#pragma unroll
      for (int k = 0; k < P; ++k) n += cnt[k];
      u64 at = before + scan(sum);
      const uint32_t n0 = (uint32_t)scan(n);
      if (tid == 0) s.bin = -1;
      __syncthreads();
      uint32_t upto = n0;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        upto += cnt[k];
        if (at < target && at + w[k] >= target) {
          s.bin = tid * P + k;
          s.before = at;
          s.in_bin = w[k];
          s.n_in_bin = cnt[k];
          s.n_upto = upto;
        }
        at += w[k];
      }
    }
    cl.sync();
    const Shared &s0 = of(0);
    return Found{s0.bin, s0.before, s0.in_bin, s0.n_in_bin, s0.n_upto};
  }

  // The element, in falling order, at which the running sum of weight over the logits
  // in [lo, hi] reaches target: value t and index; false where it does not.
  template <bool COUNT, typename F>
  __device__ bool element(float lo, float hi, F &&weight, u64 target, float &t, int &tie) {
    u64 before = 0;
    for (;;) {
      if (lo == hi) {  // equal logits: the one whose turn it is
        const u64 w = COUNT ? 1 : weight(hi);
        const u64 nth = (target - before + w - 1) / w;
        auto eq = [&](float x, int) -> u64 { return x == hi; };
        u64 front, own;
        if (sums(eq, front, own) < nth) return false;
        const int i = locate(eq, front, own, nth);
        if (i >= 0) of(0).tie = i;
        cl.sync();
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
        const int n = gather(in);
        if (rank == 0) {
          const int i = COUNT ? (int)(target - before) - 1 : reach(n, weight, before, target);
          if (tid == 0) {
            s.t = value(list[i]);
            s.tie = (int)(uint32_t)list[i];
          }
        }
        cl.sync();
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
      reduce_range(a, b, &Shared::rmx, &Shared::rmn, hi, lo);
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared s;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, row = blockIdx.x / a.C, rank = blockIdx.x % a.C;
  constexpr int E = 16 / sizeof(T);
  Row<T> R{cl, s, smem, reinterpret_cast<uint32_t *>(smem + a.hist_off),
           reinterpret_cast<u64 *>(smem + a.list_off), rank, a.C, 0, 0, 0, 0.f, false,
           tid, tid & 31, tid >> 5};
  pdl_trigger();
  if (tid < 33) s.pow2[tid] = c_pow2.v[tid];
  pdl_wait();
  // the slice, by whole vectors of memory where they lie inside it
  const int per = (a.V + a.C - 1) / a.C, lo_i = min(a.V, rank * per), hi_i = min(a.V, lo_i + per);
  const T *src = static_cast<const T *>(a.logits) + row * a.stride + lo_i;
  const int n = hi_i - lo_i, first = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  R.x0 = lo_i;
  R.first = first;
  R.n_vec = n ? (n + first + E - 1) / E : 0;
  float hi = -INFINITY, lo = INFINITY;
  {
    const uint4 *vsrc = reinterpret_cast<const uint4 *>(src - first);
    for (int v0 = tid; v0 < R.n_vec; v0 += 4 * kThreads) {
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int v = v0 + k * kThreads;
        if (v >= R.n_vec) continue;
        if (v * E >= first && (v + 1) * E - first <= n) {
          x[k] = vsrc[v];
        } else {  // an end: element by element, NaN outside
          T *p = reinterpret_cast<T *>(&x[k]);
          x[k] = make_uint4(~0u, ~0u, ~0u, ~0u);
          for (int e = 0; e < E; ++e) {
            const int i = v * E + e - first;
            if (i >= 0 && i < n) p[e] = src[i];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int v = v0 + k * kThreads;
        if (v >= R.n_vec) continue;
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
  if (rank == 0 && tid == 0) {
    s.temperature = a.temperature ? a.temperature[row] : 1.f;
    s.top_k = a.top_k ? a.top_k[row] : 0;
    s.top_p = a.top_p ? a.top_p[row] : 1.f;
    s.min_p = a.min_p ? a.min_p[row] : 0.f;
    s.u = a.u[row];
  }
  float mn;
  R.reduce_range(hi, lo, &Shared::mx, &Shared::mn, R.m, mn);
  const float m = R.m;
  float *probs = a.probs ? a.probs + (size_t)row * a.V : nullptr;
  if (!(m > kNone)) {  // nothing to keep (the whole cluster alike)
    if (rank == 0 && tid == 0) a.token[row] = -1;
    if (probs)
      for (int i = lo_i + tid; i < hi_i; i += kThreads) probs[i] = 0.f;
    cl.sync();  // (the others have read this CTA's maximum)
    return;
  }
  R.inf = m == INFINITY;
  if (R.inf) mn = m;
  const Shared &s0 = R.of(0);
  float T_ = s0.temperature, top_p = s0.top_p, min_p = s0.min_p;
  const float u = s0.u;
  int k = s0.top_k;
  const bool greedy = !(T_ >= 8.673617379884035e-19f);
  if (k <= 0 || k > a.V) k = a.V;
  if (greedy) {
    k = 1;
    T_ = 1.f;
  }
  if (!(top_p < 1.f)) top_p = 1.f;
  if (!(min_p > 0.f)) min_p = 0.f;
  const double c = 1.4426950408889634074 / (double)T_;
  Weights w;
  w.half_m = 0.5f * m;
  w.c_hi = (float)(2.0 * c);
  w.c_lo = (float)(2.0 * c - (double)w.c_hi);
  w.flat = R.inf;
  w.pow2 = s.pow2;

  // what is kept: x > t, or x == t up to index tie; and x >= x_min
  float t = kNone, x_min = kNone;
  int tie = -1;
  if (min_p >= 1.f)
    x_min = m;
  else if (min_p > 0.f && !R.inf)
    x_min = __double2float_ru((double)m + (double)T_ * log((double)min_p));
  // Logits of weights below 2^-46 count as none: no sum or draw asks for them (with
  // fewer than k above the floor, top-k takes nothing away that weighs anything)
  float floor_x = mn;
  if (!R.inf) floor_x = fmaxf(mn, __double2float_rd((double)m - 46.0 / c));
  if (k < a.V)
    R.template element<true>(k == 1 ? m : floor_x, m, [](float) -> u64 { return 1; }, (u64)k, t, tie);
  if (tie < 0) t = kNone;
  auto in_front = [&](float x, int i) { return x > t || (x == t && i <= tie); };
  u64 front, own;
  if (top_p < 1.f && k > 1) {
    const u64 total = R.sums([&](float x, int i) -> u64 { return in_front(x, i) ? w(x) : 0; }, front, own);
    // the smallest front part that reaches top_p of the total: what stands in front
    // of its last token is below.  (At the value t the sums also count what top-k
    // cut off, but behind the element that is asked for.)
    const u64 below = part_of(total, top_p);  // floor
    u64 target = below;
    {  // ceil: exact products stay
      int e;
      const u64 mant = (u64)(frexpf(fmaxf(top_p, 0.f), &e) * 16777216.f);
      const int sh = 24 - e;
      const u64 l = total * mant, h = __umul64hi(total, mant);
      const bool rest = sh >= 128 ? (l | h) != 0
                        : sh > 64 ? l != 0 || (h << (128 - sh)) != 0
                                  : sh == 64 ? l != 0 : (l << (64 - sh)) != 0;
      if (top_p > 0.f && rest) ++target;
    }
    if (target < 1) target = 1;
    R.template element<false>(fmaxf(floor_x, t), m, [&](float x) { return w(x); }, target, t, tie);
  }
  auto kept = [&](float x, int i) -> u64 { return x >= x_min && in_front(x, i) ? w(x) : 0; };
  const u64 total = R.sums(kept, front, own);
  u64 target = u >= 1.f ? total : part_of(total, u) + 1;
  if (target > total) target = total;
  const int index = R.locate(kept, front, own, target);
  if (index >= 0) a.token[row] = index;
  if (probs) {
    const double inv = 1.0 / (double)total;
    const float scale = (float)(inv * 17592186044416.0);
    for (int i = lo_i + tid; i < hi_i; i += kThreads) {
      const T *p = reinterpret_cast<const T *>(smem) + first;
      const float x = __fadd_rn(as_float(p[i - lo_i]), 0.f);
      float pr = 0.f;
      if (x > kNone && (!R.inf || x == INFINITY) && x >= x_min && in_front(x, i)) {
        int e;
        const u64 wm = w.mantissa(x, e);
        pr = ldexpf((float)wm * 5.684341886080802e-14f * scale, e);
      }
      probs[i] = pr;
    }
  }
  cl.sync();  // the others have read this CTA's sums
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
  SampleArgs a = {logits, V, 1, rows > 1 ? row_stride : 0, temperature, top_p, min_p, u, top_k, token,
                  probs, 0, 0};
  while (a.C < kMaxC && V > 8192 * a.C) a.C *= 2;
  const int per = (V + a.C - 1) / a.C;
  const int slice = (per * size + 32 + 127) / 128 * 128;
  a.hist_off = slice;
  a.list_off = slice + 4 * kBins * 4;
  const int smem = a.list_off + kCap * 8;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == QS_FP32) return launch_sample<float>(a, rows, smem, st);
  if (dtype == QS_FP16) return launch_sample<__half>(a, rows, smem, st);
  return launch_sample<__nv_bfloat16>(a, rows, smem, st);
}
