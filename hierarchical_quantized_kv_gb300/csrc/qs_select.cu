// qs_select.cu -- which groups of the cache a KV head should attend over: the
// k groups whose keys could score highest against the head's queries.
//
// The cache already holds a box around the keys of every group: channel d of
// its tokens lies in [z_d, z_d + 255 s_d] (zero and scale of the per-channel
// quantization).  The largest score a key in that box can have with a query q,
//   sum_d max(q_d z_d, q_d (z_d + 255 s_d)) = q . z + 255 relu(q) . s,
// bounds the score of every token of the group (the criterion of Quest, 2024, for
// blocks of keys), and is two dot products with the 512 bytes of scales and zeros
// the attention reads anyway.  A head's
// score for a group is the maximum over its query rows.
//
// Which of two close groups is taken must not depend on rounding: scores come
// from the tensor cores in fp32 with a bound E on their error; a group more than
// 2 E above the k-th largest score is in, one more than 2 E below is out, and
// only what lies between (a few groups) is summed again to about 46 bits, where
// sums of fp16 products are as good as exact.
//
// Bound by latency at one sequence (512 B per group and head: 4 MB for a 32k
// context of 32 heads) and by HBM for large batches.  A cluster of CTAs per
// (sequence, KV head) shares the scoring; its first CTA, in whose shared
// memory the scores meet, selects.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include "qs_common.cuh"

namespace cg = cooperative_groups;

namespace qs {
namespace {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kTile = 16;  // groups a warp scores at once (rows of the MMA)
constexpr int kMaxRows = 24;
// Groups per sequence: score (4 bytes), close sum (8), list entry (4) and flag
// (1) of each lie in shared memory.
constexpr int kMaxSelectGroups = 12800;

struct SelectSmem {
  double *exact;   // [n] close sum of list entry i
  float *score;    // [n]
  int *list;       // [n] groups near the border, ascending
  uint8_t *flag;   // [n] 1: selected
  __device__ static SelectSmem at(uint8_t *p, int cap) {
    SelectSmem s;
    s.exact = reinterpret_cast<double *>(p);
    s.score = reinterpret_cast<float *>(p + (size_t)8 * cap);
    s.list = reinterpret_cast<int *>(p + (size_t)12 * cap);
    s.flag = p + (size_t)16 * cap;
    return s;
  }
};
constexpr size_t select_smem(int cap) { return (size_t)17 * cap; }

// Keys whose unsigned order is the numbers' order (-0 and +0 alike, NaN as the
// lowest number).
__device__ __forceinline__ uint32_t key_of(float x) {
  x = x == x ? x + 0.0f : -INFINITY;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ unsigned long long key_of(double x) {
  x = x == x ? x + 0.0 : -INFINITY;
  const unsigned long long u = __double_as_longlong(x);
  return u >> 63 ? ~u : u | (1ull << 63);
}

// A number as the sum of two fp32 ones (this GPU adds fp64 numbers at a
// sixty-fourth of the fp32 rate: the close sums below took 5 us of a 15 us
// call in fp64).  two_sum is exact (Knuth); a sum of pairs is off by less than
// 2^-46 of the two numbers' magnitudes, and the same whichever comes first.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  const float l = __fadd_rn(s.l, __fadd_rn(a.l, b.l)), h = __fadd_rn(s.h, l);
  return Pair{h, __fsub_rn(l, __fsub_rn(h, s.h))};  // (|l| is far below |s.h|, or s.h is zero)
}

struct BlockScratch {
  int hist[256];
  int warp[kSelWarps];
  int digit, above;
};

// Key of the k-th largest of n keys below 2^BITS (1 <= k <= n), and how many are
// larger: radix selection from the top byte down, by the whole CTA (0.5 us a
// byte).
template <typename K, int BITS, typename KeyOf>
__device__ __forceinline__ K kth_largest(int n, int k, int *n_above, BlockScratch &S, KeyOf key_at) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  K prefix = 0;
  int need = k;
#pragma unroll 1
  for (int shift = BITS - 8; shift >= 0; shift -= 8) {
    S.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const K key = key_at(i);
      // (shifted twice: a shift by the key's whole width is undefined)
      if (((key >> shift) >> 8) == prefix) atomicAdd(&S.hist[(int)(key >> shift) & 255], 1);
    }
    __syncthreads();
    // thread t: values in bins above 255 - t (bins in descending order)
    const int bin = 255 - tid, cnt = S.hist[bin];
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) S.warp[w] = incl;
    __syncthreads();
    for (int i = 0; i < w; ++i) incl += S.warp[i];
    if (incl >= need && incl - cnt < need) {
      S.digit = bin;
      S.above = incl - cnt;
    }
    __syncthreads();
    prefix = (prefix << 8) | (K)S.digit;
    need -= S.above;
  }
  *n_above = k - need;
  return prefix;
}

// Positions in order: the number of set predicates before this thread's in
// the CTA, and the total.  Called by the whole CTA.
__device__ __forceinline__ int block_rank(bool pred, int *total, BlockScratch &S) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(0xffffffffu, pred);
  __syncthreads();  // the previous call's counts have been read
  if (lane == 0) S.warp[w] = __popc(m);
  __syncthreads();
  int before = __popc(m & ((1u << lane) - 1)), sum = 0;
  for (int i = 0; i < kSelWarps; ++i) {
    if (i == w) before += sum;
    sum += S.warp[i];
  }
  *total = sum;
  return before;
}

// Channel in position p of a key scale / zero row.
__device__ __forceinline__ int kmeta_channel(int p) {
  return 32 * ((p >> 3) & 3) + 8 * (p >> 5) + 2 * ((p >> 2) & 1) + ((p >> 1) & 1) + 4 * (p & 1);
}

__device__ __forceinline__ uint4 ld16(const uint16_t *p) {
  return *reinterpret_cast<const uint4 *>(p);
}

// Grid (cluster size, H, B).  NCG: column groups of eight query rows.  (Two CTAs an
// SM asked for in the usual variant, or the compiler stops at 108 registers with
// fewer rows in flight: 16 x 32 heads of 512 groups 41.7 us; so 30.3.)
template <int NCG>
__global__ void __launch_bounds__(kSelThreads, NCG == 1 ? 2 : 1)
    select_kernel(qs_cache c, Pages pg, const uint16_t *q, int R, int k_sel, int32_t *sel) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ BlockScratch S;
  // the first CTA's: largest sum of magnitudes, smallest and largest key of a score
  __shared__ int s_mag, s_n;
  __shared__ unsigned s_kmin, s_kmax;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), n_ranks = (int)cluster.num_blocks();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int w = tid >> 5, lane = tid & 31, r = lane >> 2, cq = lane & 3;
  SelectSmem M = SelectSmem::at(smem_raw, c.cap_groups);
  if (tid == 0) {
    s_mag = 0;
    s_kmin = 0xFFFFFFFFu;
    s_kmax = 0;
  }
  pdl_trigger();
  // While the kernel before still runs: counters, queries, and the first
  // tile's rows (or its page numbers) towards L2 (L1 would be stale)
  {
    const size_t bh = (size_t)b * c.H + h;
    if (tid == 0) prefetch_l2(c.state + (size_t)b * QS_STATE_WORDS);
    if (tid < 2 * R) prefetch_l2(q + bh * R * kD + 64 * tid);
    const int g0 = kTile * (rank * kSelWarps + w) + (lane & 15);
    if (pg.table) {
      if (g0 < c.cap_groups && (lane & 15) == lane) prefetch_l2(pg.table + (size_t)b * c.cap_groups + g0);
    } else if (g0 < c.cap_groups) {  // 512 bytes a group: four lines, two a lane
      const uint16_t *m = c.meta + (bh * c.cap_groups + g0) * 512 + 128 * (lane >> 4);
      prefetch_l2(m);
      prefetch_l2(m + 64);
    }
  }
  pdl_wait();
  // Should somebody change the counter meanwhile (against the rule that calls on a
  // cache are ordered), warps and CTAs may differ in it.  The selection is then
  // worth nothing, but a CTA goes one way, all meet the cluster's barriers and the
  // first CTA leaves last, so that no store goes to one that has gone; and that CTA
  // selects by the one number that its first thread read.
  int32_t *st = c.state + (size_t)b * QS_STATE_WORDS;
  const int n_warp = min(max(st[QS_ST_N_GROUPS], 0), c.cap_groups);
  if (tid == 0) s_n = n_warp;
  const size_t bh = (size_t)b * c.H + h;
  int32_t *out = sel + bh * k_sel;
  if (__syncthreads_and(n_warp <= k_sel)) {  // all of them
    if (rank == 0)
      for (int i = tid; i < k_sel; i += kSelThreads) out[i] = i < s_n ? i : -1;
    if (n_ranks > 1) {
      cluster.barrier_arrive();
      cluster.barrier_wait();
      cluster.sync();
    }
    return;
  }
  int n = n_warp;
  // the first CTA's shared memory is written below: it must have started
  cluster.barrier_arrive();

  // ---- scores: a warp takes 16 groups.  A = their zero (or scale) rows, as
  // stored: lane (r, cq) loads 16 bytes of rows r and r + 8, which are two
  // k-blocks' fragments; B = q in the order of those rows.
  const uint16_t *qh = q + bh * R * kD;
  uint32_t q0[NCG][8], q1[NCG][8];
#pragma unroll
  for (int g = 0; g < NCG; ++g) {
    const int row = 8 * g + r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < R && chk(in_range((bh * R + row) * kD, kD, (size_t)c.B * c.H * R * kD), 44))
        x = ld16(qh + (size_t)row * kD + 32 * cq + 8 * i);
      q0[g][2 * i] = prmt(x.x, x.z, 0x5410);
      q1[g][2 * i] = prmt(x.x, x.z, 0x7632);
      q0[g][2 * i + 1] = prmt(x.y, x.w, 0x5410);
      q1[g][2 * i + 1] = prmt(x.y, x.w, 0x7632);
    }
  }
  const int n_tiles = (n + kTile - 1) / kTile;
  float *score0 = cluster.map_shared_rank(M.score, 0);
  bool started = false;
  float mag = 0.f;
  unsigned kmin = 0xFFFFFFFFu, kmax = 0;
#pragma unroll 1
  for (int t = rank * kSelWarps + w; t < n_tiles; t += n_ranks * kSelWarps) {
    uint4 zr[2][4], sr[2][4];  // zero and scale rows of groups r and r + 8
    bool good[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = kTile * t + r + 8 * j;
      const long long place = g < n ? group_slot(c, pg, b, h, g) : -1;
      good[j] = place >= 0 && chk(in_range((size_t)place, 1, group_slots(c, pg)), 43);
      if (g < n && place < 0 && h == 0 && cq == 0) atomicOr(&st[QS_ST_ERR], QS_DEV_PAGE);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        zr[j][i] = sr[j][i] = make_uint4(0, 0, 0, 0);
        if (good[j]) {
          const uint16_t *m = c.meta + (size_t)place * 4 * 128 + 8 * (4 * i + cq);
          sr[j][i] = ld16(m + QS_META_K_SCALE * 128);
          zr[j][i] = ld16(m + QS_META_K_ZERO * 128);
        }
      }
    }
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int g = 0; g < NCG; ++g) {
      // each MMA starts from zero and its result is added in fp32, so the
      // tensor core's own rounding never runs along a chain
      float az[4] = {0, 0, 0, 0}, as[4] = {0, 0, 0, 0}, aa[4] = {0, 0, 0, 0};
#pragma unroll
      for (int kb = 0; kb < 8; ++kb) {
        const int i = kb >> 1;
        const uint32_t z0 = kb & 1 ? zr[0][i].z : zr[0][i].x, z2 = kb & 1 ? zr[0][i].w : zr[0][i].y;
        const uint32_t z1 = kb & 1 ? zr[1][i].z : zr[1][i].x, z3 = kb & 1 ? zr[1][i].w : zr[1][i].y;
        const uint32_t s0 = kb & 1 ? sr[0][i].z : sr[0][i].x, s2 = kb & 1 ? sr[0][i].w : sr[0][i].y;
        const uint32_t s1 = kb & 1 ? sr[1][i].z : sr[1][i].x, s3 = kb & 1 ? sr[1][i].w : sr[1][i].y;
        const uint32_t b0 = q0[g][kb], b1 = q1[g][kb];
        const uint32_t p0 = h2_as_u32(__hmax2(u32_as_h2(b0), u32_as_h2(0u)));
        const uint32_t p1 = h2_as_u32(__hmax2(u32_as_h2(b1), u32_as_h2(0u)));
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        float dz[4] = {0, 0, 0, 0}, ds[4] = {0, 0, 0, 0}, da[4] = {0, 0, 0, 0};
        mma16816(dz, z0, z1, z2, z3, b0, b1);
        mma16816(ds, s0, s1, s2, s3, p0, p1);
        mma16816(da, z0 & kAbs, z1 & kAbs, z2 & kAbs, z3 & kAbs, b0 & kAbs, b1 & kAbs);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          az[x] += dz[x];
          as[x] += ds[x];
          aa[x] += da[x];
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // rows r (x < 2) and r + 8, columns 2 cq + x % 2
        if (8 * g + 2 * cq + (x & 1) < R) {
          best[x >> 1] = fmaxf(best[x >> 1], fmaf(255.f, as[x], az[x]));
          const float a = fmaf(255.f, as[x], aa[x]);
          mag = a < FLT_MAX ? fmaxf(mag, a) : INFINITY;  // (NaN too)
        }
      }
    }
    if (!started) {
      cluster.barrier_wait();
      started = true;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x = best[j];
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      const int g = kTile * t + r + 8 * j;
      if (cq == 0 && g < n) {
        x = good[j] ? x : -INFINITY;
        // (the first CTA's shared memory is laid out as this one's)
        if (chk(smem_in(smem_addr(M.score + g), 4) && M.score + g < (float *)M.list, 40)) score0[g] = x;
        kmin = min(kmin, key_of(x));
        kmax = max(kmax, key_of(x));
      }
    }
  }
  if (!started) cluster.barrier_wait();
  // A product's exponent is taken from the operands' exponent fields, where a
  // subnormal zero or scale counts as 2^-14: as much again for each channel,
  // sum |q| (1 + 255) 2^-14 <= 2 max |q|.
  uint32_t qmax = 0;
#pragma unroll
  for (int g = 0; g < NCG; ++g)
#pragma unroll
    for (int kb = 0; kb < 8; ++kb)
      qmax = h2_as_u32(__hmax2_nan(u32_as_h2(qmax), __hmax2_nan(__habs2(u32_as_h2(q0[g][kb])),
                                                                __habs2(u32_as_h2(q1[g][kb])))));
  const float2 qm = __half22float2(u32_as_h2(qmax));
  mag += 2.f * __int_as_float(__reduce_max_sync(
                   0xffffffffu, max(__float_as_int(qm.x), __float_as_int(qm.y))));
  // (mag >= 0: ordered as integers)
  const int wmag = __reduce_max_sync(0xffffffffu, __float_as_int(mag));
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0 && kmax >= kmin) {
    atomicMax(cluster.map_shared_rank(&s_mag, 0), wmag);
    atomicMin(cluster.map_shared_rank(&s_kmin, 0), kmin);
    atomicMax(cluster.map_shared_rank(&s_kmax, 0), kmax);
  }
  cluster.sync();  // all scores are in the first CTA
  if (rank != 0) return;
  n = s_n;

  // ---- selection.  One MMA adds 17 numbers, aligned to the largest and cut
  // no coarser than 2^-23 of it: off by less than 2^-18.9 of the sum of their
  // magnitudes; the eight fp32 additions and the last multiply-add add
  // 9 x 2^-24.  Together under 2^-18.
  const float E = __int_as_float(s_mag) * 0x1p-18f;
  // The k-th largest score up to the top 16 bits of the keys' range (a few
  // rounding steps of a score, below E as a rule): it lies in [t_lo, t_hi].
  const unsigned k0 = s_kmin, k1 = s_kmax;
  const int shift = max(0, 16 - __clz(k1 - k0));  // (k1 == k0: clz 32, shift 0)
  int above;
  const unsigned t = kth_largest<unsigned, 16>(n, k_sel, &above, S, [&](int i) {
    return (key_of(M.score[i]) - k0) >> shift;
  });
  const float t_lo = float_of(k0 + (t << shift)), t_hi = float_of(k0 + (t << shift) + ((1u << shift) - 1));
  // (infinite or NaN limits, from queries that are not finite, leave every
  // group to the close sums)
  const float hi = __fadd_ru(t_hi, 2.f * E), lo = __fadd_rd(t_lo, -2.f * E);
  int m = 0, n_in = 0;
  for (int base = 0; base < n; base += kSelThreads) {
    const int g = base + tid;
    const float x = g < n ? M.score[g] : 0.f;
    const bool in = g < n && x > hi, near = g < n && !in && !(x < lo);
    int tot;
    const int at = m + block_rank(near, &tot, S);
    if (g < n && chk(smem_in(smem_addr(M.flag + g), 1), 40)) M.flag[g] = in;
    if (near && chk(smem_in(smem_addr(M.list + at), 4) && (uint8_t *)(M.list + at) < M.flag, 41))
      M.list[at] = g;
    m += tot;
    n_in += __syncthreads_count(in);
  }
  const int need = k_sel - n_in;  // of the m groups near the border
  auto take = [&](int i) {        // the i-th of them is selected
    const int g = M.list[i];
    if (chk(i < c.cap_groups && g >= 0 && g < n, 41)) M.flag[g] = 1;
  };
  if (need >= m) {
    for (int i = tid; i < m; i += kSelThreads) take(i);
  } else if (need > 0) {
    // close sums: half a warp per group, lane l of it holds positions 8 l ..
    // 8 l + 7 of the rows, which are eight channels that lie together
    const int l = lane & 15, ch = kmeta_channel(8 * l);
    for (int base = 2 * w; base < m; base += 2 * kSelWarps) {
      const int i = base + (lane >> 4);
      long long place = i < m ? group_slot(c, pg, b, h, M.list[i]) : -1;
      if (place >= 0 && !chk(in_range((size_t)place, 1, group_slots(c, pg)), 43)) place = -1;
      uint4 sw = make_uint4(0, 0, 0, 0), zw = sw;
      if (place >= 0) {
        const uint16_t *mt = c.meta + (size_t)place * 4 * 128 + 8 * l;
        sw = ld16(mt + QS_META_K_SCALE * 128);
        zw = ld16(mt + QS_META_K_ZERO * 128);
      }
      Pair best{-INFINITY, 0.f};
#pragma unroll 2
      for (int row = 0; row < R; ++row) {
        const uint4 qw = ld16(qh + (size_t)row * kD + ch);
        // positions 2 x, 2 x + 1 of the eight: channels c, c + 4 with c = 0, 1, 2, 3
        const uint32_t qp[4] = {prmt(qw.x, qw.z, 0x5410), prmt(qw.x, qw.z, 0x7632),
                                prmt(qw.y, qw.w, 0x5410), prmt(qw.y, qw.w, 0x7632)};
        const uint32_t sp[4] = {sw.x, sw.y, sw.z, sw.w}, zp[4] = {zw.x, zw.y, zw.z, zw.w};
        Pair ds[4], dz[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 qv = __half22float2(u32_as_h2(qp[x])), sv = __half22float2(u32_as_h2(sp[x])),
                       zv = __half22float2(u32_as_h2(zp[x]));
          // (products of two fp16 numbers are exact in fp32)
          dz[x] = two_sum(__fmul_rn(qv.x, zv.x), __fmul_rn(qv.y, zv.y));
          ds[x] = two_sum(__fmul_rn(fmaxf(qv.x, 0.f), sv.x), __fmul_rn(fmaxf(qv.y, 0.f), sv.y));
        }
        const Pair sum_s = (ds[0] + ds[1]) + (ds[2] + ds[3]);
        const float p = __fmul_rn(255.f, sum_s.h), e = __fmaf_rn(255.f, sum_s.h, -p);
        Pair d = ((dz[0] + dz[1]) + (dz[2] + dz[3])) + Pair{p, __fmaf_rn(255.f, sum_s.l, e)};
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
          d = d + Pair{__shfl_xor_sync(0xffffffffu, d.h, o), __shfl_xor_sync(0xffffffffu, d.l, o)};
        if (d.h > best.h || (d.h == best.h && d.l > best.l)) best = d;
      }
      if (l == 0 && i < m && chk((float *)(M.exact + i) < M.score, 41))
        M.exact[i] = place >= 0 ? (double)best.h + (double)best.l : -INFINITY;
    }
    __syncthreads();
    if (m <= kSelThreads) {  // a thread an entry counts those before it
      if (tid < m) {
        const double x = M.exact[tid] + 0.0;
        int before = 0;
        for (int i = 0; i < m; ++i) before += M.exact[i] > x || (M.exact[i] == x && i < tid);
        if (before < need) take(tid);
      }
    } else {
      const unsigned long long k64 = kth_largest<unsigned long long, 64>(
          m, need, &above, S, [&](int i) { return key_of(M.exact[i]); });
      // those above the need-th, then those equal to it from the lowest index on
      int equal = 0;
      for (int base = 0; base < m; base += kSelThreads) {
        const int i = base + tid;
        const unsigned long long x = i < m ? key_of(M.exact[i]) : 0;
        int tot;
        const int at = equal + block_rank(i < m && x == k64, &tot, S);
        if (i < m && (x > k64 || (x == k64 && at < need - above))) take(i);
        equal += tot;
      }
    }
  }
  __syncthreads();
  int done = 0;
  for (int base = 0; base < n; base += kSelThreads) {
    const int g = base + tid;
    const bool in = g < n && M.flag[g];
    int tot;
    const int at = done + block_rank(in, &tot, S);
    if (in && at < k_sel && chk(in_range(bh * k_sel + at, 1, (size_t)c.B * c.H * k_sel), 42)) out[at] = g;
    done += tot;
  }
  for (int i = done + tid; i < k_sel; i += kSelThreads) out[i] = -1;  // (never with finite queries)
}

// CTAs per (sequence, KV head): one per 128 groups (a tile for each warp), at
// most 8, as long as the whole grid stays within two CTAs an SM (four sequences
// of 8 KV heads and 1,022 groups: clusters of 8, 9.9 us; of 4, 11.4).
int cluster_size(const qs_cache &c, int sms) {
  int n = 1;
  while (n < 8 && n * kSelWarps * kTile < c.cap_groups && (long long)c.B * c.H * n * 2 <= 2 * sms) n *= 2;
  return n;
}

int g_sel_ready[3] = {0, 0, 0};  // one bit per device ordinal below 32

template <int NCG>
qs_status launch_select(const qs_cache &c, const Pages &pg, const uint16_t *q, int R, int k_sel,
                        int32_t *sel, cudaStream_t stream) {
  int sms = 0;
  qs_status s = sm_count(&sms);
  if (s != QS_OK) return s;
  s = set_smem_once((const void *)select_kernel<NCG>, (int)select_smem(kMaxSelectGroups),
                    &g_sel_ready[NCG - 1]);
  if (s != QS_OK) return s;
  const int cl = cluster_size(c, sms);
  return launch_pdl_cluster(select_kernel<NCG>, dim3(cl, c.H, c.B), dim3(kSelThreads), cl,
                            select_smem(c.cap_groups), stream, c, pg, q, R, k_sel, sel);
}

}  // namespace
}  // namespace qs

using namespace qs;

extern "C" qs_status qs_select_groups(const qs_cache *c, const qs_pages *pg, const uint16_t *q,
                                      int32_t n_q, int32_t group, int32_t k_sel, int32_t *sel,
                                      qs_stream_t stream) {
  qs_cache cc;
  Pages pages;
  const qs_status s = check_pages(c, pg, false, &cc, &pages);
  if (s != QS_OK) return s;
  if (!q || !sel || n_q < 1 || n_q > kMaxQ || group < 1 || group > kMaxRows ||
      group * n_q > kMaxRows || k_sel < 1)
    return QS_ERR_ARG;
  if (cc.cap_groups > kMaxSelectGroups) return QS_ERR_UNSUPPORTED;
  if (!aligned16(q) || reinterpret_cast<uintptr_t>(sel) % 4) return QS_ERR_ALIGN;
  const int R = group * n_q;
  cudaStream_t st = (cudaStream_t)stream;
  if (R <= 8) return launch_select<1>(cc, pages, q, R, k_sel, sel, st);
  return R <= 16 ? launch_select<2>(cc, pages, q, R, k_sel, sel, st)
                 : launch_select<3>(cc, pages, q, R, k_sel, sel, st);
}

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_select(unsigned long long *out2, int reset) {
  return read_check_failures(out2, reset);
}
#endif
