// qs_quantize.cu -- quantize-on-flush: one G-token fp16 buffer half becomes
// one hierarchical group (C_U / C_L nibble planes plus fp16 scale and zero).
//
// Source: "QuantSpec: Self-Speculative Decoding with Hierarchical Quantized
// KV Cache" (Pith review), "What carries the argument" (C_INT8 = 2^4 C_U +
// C_L, one shared scale and zero-point, a half is quantized once every G
// steps) and Figure 7 / Appendix D (keys per channel over G tokens, values
// per token over G channels, asymmetric).  "QuantSpec Guide", quantizer
// section: min/max, 255 levels, round, clamp, q >> 4 and q & 15.
//
// Convention QS-RN-v1 (every fp32 step IEEE round-to-nearest-even; this file
// is compiled without fast-math so __fsub_rn / __fdiv_rn are exact IEEE):
//   r = max - min, s = r == 0 ? 0 : fp16_round_up(r / 255), z = min (+0 if 0),
//   q = s == 0 ? 0 : clamp(rne((x - z) / s), 0, 255).
#include "qs_common.cuh"

namespace qs {

namespace {

constexpr int kParts = 4;           // CTAs per (head, sequence)
constexpr int kSlice = kD / kParts;  // key channels / value tokens per CTA
// Warps per CTA.  A flush of few heads is one wave of small CTAs, so its time is
// one CTA's chain of phases, and sixteen warps shorten every phase but the
// packing (32 heads: 4.2 us; eight warps 5.2, four 6.2); one of many is bound
// by instruction issue like a prefill, where four are best (8 x 32 heads: 9.4 us;
// eight 10.5, sixteen 12.4).  In a prefill of many waves, what a thread does once
// per quarter (addresses, scales) counts: four warps, twice the elements a
// thread, 147 us for 32 heads of 32k tokens (0.82 of the copy bandwidth's rate;
// eight: 175).  A prompt of one or two quarters per CTA is a chain again (four
// sequences of 1k tokens and 8 heads: eight warps 7.3 us, four 8.5), and a very
// short one takes sixteen (two heads of 1k tokens: 3.6 us; eight 3.8, four 4.1).
constexpr int kFlushWarps = 16, kBatchFlushWarps = 4;
// Group quarters per quantizing CTA of a prefill, loads pipelined one ahead, at
// most.
constexpr int kPrefillQuarters = 8;

// One CTA owns key channels [32p, 32p+32) (one 16-byte column of every key
// row) and value tokens [32p, 32p+32) (value quarter p).
// Value codes in shared memory: blocks of 32 bytes of a row swapped by its
// number, so that the four token pairs a group of lanes reads (and the four
// tokens half a warp writes) fall into different banks.
__device__ __forceinline__ int code_col(int row, int col) { return col ^ (32 * ((row >> 1) & 3)); }
template <int QW>
struct FlushSmem {
  __half k[kG][kSlice];          // keys of the slice   [token][channel - 32p]
  __half v[kSlice][kD];          // values of the slice [token - 32p][channel]
  uint8_t vc[kSlice][kD];        // value codes
  union {
    struct {
      uint32_t kmin[QW][kSlice / 2], kmax[QW][kSlice / 2];  // half2 per channel pair
    };
    struct {  // (written by the warp that has read those)
      float kzf[kSlice], krf[kSlice];  // key zero, reciprocal of the key scale
      uint16_t ks[kSlice], kz[kSlice];
    };
  };
  uint16_t vs[kSlice], vz[kSlice];
  int act, base, g, place;
};

__device__ __forceinline__ void scale_zero(float mn, float mx, uint16_t &s_bits, uint16_t &z_bits,
                                           float &sf, float &zf) {
  const float r = __fsub_rn(mx, mn);
  __half s = __float2half_ru(__fdiv_rn(r, 255.0f));
  if (r == 0.0f) s = __ushort_as_half(0);
  s_bits = __half_as_ushort(s);
  // exact (mn is an fp16 value); a zero minimum is stored as +0
  z_bits = (mn == 0.0f) ? (uint16_t)0 : __half_as_ushort(__float2half_rn(mn));
  sf = __half2float(s);
  zf = mn;
}

// q = clamp(rne(fl((x - z) / s)), 0, 255) with fl the IEEE fp32 quotient, as
// QS-RN-v1 defines it, without a divide per element: a = fl(x - z) is never
// negative (z is the group's minimum), rf = fl(1 / s) is exact to 2^-24, so
// the exact product a rf is within 2^-15 of fl(a / s) (which is at most 255 (1 +
// 2^-23), since s >= r / 255).  Adding 1.5 * 2^23 in one fused multiply-add
// rounds it to the nearest even integer n, which then stands in the low byte of
// the sum; a second one gives the remainder a rf - n.  The two quotients round
// alike unless that lies within 2^-12 of a half; there the exact quotient
// decides (about one element in 2^11).  A zero scale means a zero range: a = 0,
// and rf is taken as 0, which gives code 0.  A quotient that is not a number (an
// element that is not one, or a range that is infinite) has code 0; its remainder
// is not a number either and takes the element the exact quotient's way.
constexpr float kRound = 12582912.f;  // 1.5 * 2^23
constexpr float kNear = 0.5f - 0x1p-12f;

// The larger number, NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float reciprocal(float sf) { return sf == 0.f ? 0.f : __frcp_rn(sf); }

// Low bytes of four words, in order.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return prmt(prmt(a, b, 0x0040), prmt(c, d, 0x0040), 0x5410);
}

// Codes of eight values that lie together at p in shared memory (x: the same,
// loaded), a byte each: codes 0..3 and 4..7, or (EVEN_ODD) 0, 2, 4, 6 and 1, 3,
// 5, 7.  z_at(i), s_at(i): zero and scale of value i, for the rare exact ones,
// which a loop of their own takes one by one from memory (eight divides in line
// at every place made a loop body larger than the instruction cache).
template <bool EVEN_ODD, typename Zero, typename Scale>
__device__ __forceinline__ uint2 codes8(const __half *p, const uint4 &x, const float (&zf)[8],
                                        const float (&rf)[8], Zero z_at, Scale s_at) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float d[8], far = 0.f;
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(u32_as_h2(w[i >> 1]));
    const float a = __fsub_rn(i & 1 ? f.y : f.x, zf[i]);
    const float n = __fmaf_rn(a, rf[i], kRound);
    d[i] = __fmaf_rn(a, rf[i], -__fsub_rn(n, kRound));
    far = max_nan(far, fabsf(d[i]));
    t[i] = __float_as_uint(n);
  }
  uint2 q = EVEN_ODD ? make_uint2(low_bytes(t[0], t[2], t[4], t[6]), low_bytes(t[1], t[3], t[5], t[7]))
                     : make_uint2(low_bytes(t[0], t[1], t[2], t[3]), low_bytes(t[4], t[5], t[6], t[7]));
  if (!(far <= kNear)) {
    unsigned near = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) near |= fabsf(d[i]) <= kNear ? 0u : 1u << i;
#pragma unroll 1
    while (near) {
      const int i = __ffs(near) - 1;
      near &= near - 1;
      const float a = __fsub_rn(__half2float(p[i]), z_at(i));
      const float u = __fdiv_rn(a, s_at(i));
      const uint32_t n = u == u ? __float_as_uint(__fadd_rn(u, kRound)) & 0xFFu : 0u;
      const int sh = EVEN_ODD ? 8 * (i >> 1) : 8 * (i & 3);
      uint32_t &word = (EVEN_ODD ? i & 1 : i >> 2) ? q.y : q.x;
      word = (word & ~(0xFFu << sh)) | (n << sh);
    }
  }
  return q;
}

// Eight codes' nibble words: ev holds codes 0, 2, 4, 6 and od 1, 3, 5, 7, a byte
// each; nibble j of the result belongs to code j.
__device__ __forceinline__ uint32_t upper_nibbles(uint32_t ev, uint32_t od) {
  return bitsel(ev >> 4, od, 0x0F0F0F0Fu);
}
__device__ __forceinline__ uint32_t lower_nibbles(uint32_t ev, uint32_t od) {
  return bitsel(ev, od << 4, 0x0F0F0F0Fu);
}

// Word W of a group's upper plane.  Two-bit draft layout: nibble j of word k of
// the C_U2 plane (first 4 KB of the group's 8 KB) holds the two-bit field (C_U =
// 4 C_U2 + M2) of word 2k's nibble j in its low half and of word 2k+1's in its
// high half, and word k of the M2 plane (second 4 KB) the same of M2; the lanes
// of words 2k and 2k + 1 are neighbours (W and lane have the same parity, the
// whole warp calls), the even one writes the C_U2 word, the odd one the M2 word.
__device__ __forceinline__ void store_upper(uint8_t *base, int W, uint32_t w, bool two_bit) {
  if (!two_bit) {
    *reinterpret_cast<uint32_t *>(base + 4 * W) = w;
    return;
  }
  const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 1);
  const uint32_t v = (W & 1) ? ((other & 0x33333333u) | ((w & 0x33333333u) << 2))
                             : (((w >> 2) & 0x33333333u) | (other & 0xCCCCCCCCu));
  *reinterpret_cast<uint32_t *>(base + (W & 1 ? kG * kD / 4 : 0) + 4 * (W >> 1)) = v;
}

// Transposes the 4 x 4 words of four neighbouring lanes (m = lane % 4): word j of
// lane m goes to word m of lane j.
__device__ __forceinline__ void transpose4(uint32_t (&x)[4], int m) {
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const bool hi = m & o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & o) continue;
      const uint32_t y = __shfl_xor_sync(0xffffffffu, hi ? x[j] : x[j | o], o);
      if (hi)
        x[j] = y;
      else
        x[j | o] = y;
    }
  }
}

// Position of channel c in a key scale / zero row (inverse of the header's
// map p -> 32((p>>3)&3) + 8(p>>5) + 2((p>>2)&1) + ((p>>1)&1) + 4(p&1)).
__device__ __forceinline__ int kmeta_pos(int c) {
  return ((c >> 2) & 1) | ((c & 1) << 1) | (((c >> 1) & 1) << 2) | (((c >> 5) & 3) << 3) |
         (((c >> 3) & 3) << 5);
}

// Position of token t in a value scale / zero row (inverse of
// p -> 32(p>>5) + ((p>>2)&7) + 16((p>>1)&1) + 8(p&1)).
__device__ __forceinline__ int vmeta_pos(int t) {
  return ((t >> 3) & 1) | (((t >> 4) & 1) << 1) | ((t & 7) << 2) | ((t >> 5) << 5);
}

// Asynchronous 16-byte copy global -> shared through the load/store path
// (cached in L2 only; addresses 16-byte aligned), its commit group, and the
// wait until at most N of the thread's groups are still in flight.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A CTA's share of a group is a quarter: key channels [32 part, 32 part +
// 32) and value tokens [32 part, 32 part + 32).
// 1. loads of a group quarter into kt / vt: the key column slice (64 B of
// each of 128 rows) and 32 value rows; ASYNC: as cp.async copies, one commit
// group (the caller waits for it before quantize_loaded).
template <int QW, bool ASYNC>
__device__ __forceinline__ void load_part(__half (*kt)[kSlice], __half (*vt)[kD], const __half *gk,
                                          const __half *gv, int part, int tid) {
  constexpr int kQThreads = 32 * QW;
  for (int e = tid; e < kG * 4; e += kQThreads) {  // 4 x 16 B per key row
    const int t = e >> 2, q = e & 3;
    const uint4 *src = reinterpret_cast<const uint4 *>(gk + (size_t)t * kD + part * kSlice) + q;
    if (ASYNC)
      cp_async16(smem_addr(&kt[t][0]) + 16 * q, src);
    else
      reinterpret_cast<uint4 *>(&kt[t][0])[q] = *src;
  }
  for (int e = tid; e < kSlice * kD / 8; e += kQThreads) {
    const uint4 *src = reinterpret_cast<const uint4 *>(gv + (size_t)part * kSlice * kD) + e;
    if (ASYNC)
      cp_async16(smem_addr(&vt[0][0]) + 16 * e, src);
    else
      reinterpret_cast<uint4 *>(&vt[0][0])[e] = *src;
  }
  if (ASYNC) cp_async_commit();
}

__device__ __forceinline__ uint32_t hmin2_u32(uint32_t a, uint32_t b) {
  return h2_as_u32(__hmin2(u32_as_h2(a), u32_as_h2(b)));
}
__device__ __forceinline__ uint32_t hmax2_u32(uint32_t a, uint32_t b) {
  return h2_as_u32(__hmax2(u32_as_h2(a), u32_as_h2(b)));
}
__device__ __forceinline__ float half_bits_to_float(uint32_t b) {
  return __half2float(__ushort_as_half((uint16_t)b));
}

// Phases 2-7 of a group quarter whose rows are in kt / vt (all loads landed
// and visible to the CTA).  Bound by instruction issue, so every phase works
// on as much as a load brings: minima and maxima on pairs of fp16 values
// (exact), eight codes a thread at a time, planes assembled from words of even
// and of odd codes by one shift and one bit select each.
template <int QW>
__device__ void quantize_loaded(FlushSmem<QW> &S, const __half (*kt)[kSlice],
                                const __half (*vt)[kD], const qs_cache &c, size_t grp, int part,
                                int tid) {
  constexpr int kQWarps = QW, kQThreads = 32 * QW;
  const int warp = tid >> 5, lane = tid & 31;
  const bool two_bit = c.upper_bits == 2;

  // 2. keys: min / max per channel pair.  Thread = pair tid % 16 of every second
  // token of a run (the two halves of a warp read neighbouring rows).
  {
    constexpr int kTs = 16 * kG / kQThreads;  // tokens per thread
    const int slot = tid >> 4, t0 = 2 * kTs * (slot >> 1) + (slot & 1);
    uint32_t mn = 0x7C007C00u, mx = 0xFC00FC00u;  // +inf, -inf
#pragma unroll
    for (int i = 0; i < kTs; ++i) {
      const uint32_t x = *reinterpret_cast<const uint32_t *>(&kt[t0 + 2 * i][2 * (tid & 15)]);
      mn = hmin2_u32(mn, x);
      mx = hmax2_u32(mx, x);
    }
    mn = hmin2_u32(mn, __shfl_xor_sync(0xffffffffu, mn, 16));
    mx = hmax2_u32(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    if (lane < 16) {
      S.kmin[warp][lane] = mn;
      S.kmax[warp][lane] = mx;
    }
  }
  __syncthreads();
  if (tid < kSlice) {
    // 3. keys: scale and zero of the channel slice
    const int sh = 16 * (tid & 1);
    uint32_t mn = S.kmin[0][tid >> 1], mx = S.kmax[0][tid >> 1];
#pragma unroll
    for (int w = 1; w < kQWarps; ++w) {
      mn = hmin2_u32(mn, S.kmin[w][tid >> 1]);
      mx = hmax2_u32(mx, S.kmax[w][tid >> 1]);
    }
    uint16_t sb, zb;
    float sf, zf;
    scale_zero(half_bits_to_float(mn >> sh), half_bits_to_float(mx >> sh), sb, zb, sf, zf);
    static_assert(kSlice == 32, "one warp");
    __syncwarp();
    S.ks[tid] = sb;
    S.kz[tid] = zb;
    S.kzf[tid] = zf;
    S.krf[tid] = reciprocal(sf);
  }
  // 4. values: kLt threads a token, each kCh runs of eight channels; min / max
  // (as the pair min, -max, one shuffle for both), scale, codes
  {
    constexpr int kLt = kQThreads / kSlice, kCh = kD / 8 / kLt;
    static_assert(kLt >= 4 && kLt <= 16 && kCh >= 1, "128 to 512 threads");
    const int t = tid / kLt, lt = tid % kLt;
    // run i of a thread: with four threads a token, odd tokens take the runs from
    // the last one down (two rows of 64 bytes otherwise meet in one half of the
    // banks)
    auto run = [&](int i) { return 8 * (lt + kLt * (kLt == 4 ? i ^ (3 * (t & 1)) : i)); };
    uint4 x[kCh];
    uint32_t mn = 0x7C007C00u, mx = 0xFC00FC00u;
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      x[i] = *reinterpret_cast<const uint4 *>(&vt[t][run(i)]);
      mn = hmin2_u32(hmin2_u32(mn, hmin2_u32(x[i].x, x[i].y)), hmin2_u32(x[i].z, x[i].w));
      mx = hmax2_u32(hmax2_u32(mx, hmax2_u32(x[i].x, x[i].y)), hmax2_u32(x[i].z, x[i].w));
    }
    uint32_t mm = prmt(hmin2_u32(mn, prmt(mn, 0, 0x1032)), hmax2_u32(mx, prmt(mx, 0, 0x1032)) ^ 0x80008000u,
                       0x5410);
#pragma unroll
    for (int o = 1; o < kLt; o <<= 1) mm = hmin2_u32(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    uint16_t sb, zb;
    float sf, zf;
    scale_zero(half_bits_to_float(mm & 0xFFFFu), -half_bits_to_float(mm >> 16), sb, zb, sf, zf);
    if (lt == 0) {
      S.vs[t] = sb;
      S.vz[t] = zb;
    }
    const float rf = reciprocal(sf);
    const float zs[8] = {zf, zf, zf, zf, zf, zf, zf, zf}, rs[8] = {rf, rf, rf, rf, rf, rf, rf, rf};
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      *reinterpret_cast<uint2 *>(&S.vc[t][code_col(t, run(i))]) = codes8<false>(
          &vt[t][run(i)], x[i], zs, rs, [&](int) { return zf; }, [&](int) { return sf; });
    }
  }
  __syncthreads();

  if (tid >= kQThreads - kD) {
    // 5. value planes, by the last four warps: thread = word m (eight tokens of
    // the quarter) of four channels; nibble j of the word belongs to token
    // 2 m + j / 4 + 8 (j & 1) + 16 (j / 2 & 1)
    const int i = tid - (kQThreads - kD), m = i & 3, d0 = 4 * (i >> 2);
    uint32_t x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = 2 * m + (j >> 2) + 8 * (j & 1) + 16 * ((j >> 1) & 1);
      x[j] = *reinterpret_cast<const uint32_t *>(&S.vc[t][code_col(t, d0)]);
    }
    // bytes of four rows (even or odd j) to a word per channel
    uint32_t wrd[2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t a = prmt(x[e], x[2 + e], 0x5140), b = prmt(x[4 + e], x[6 + e], 0x5140);
      const uint32_t f = prmt(x[e], x[2 + e], 0x7362), g = prmt(x[4 + e], x[6 + e], 0x7362);
      wrd[e][0] = prmt(a, b, 0x5410);
      wrd[e][1] = prmt(a, b, 0x7632);
      wrd[e][2] = prmt(f, g, 0x5410);
      wrd[e][3] = prmt(f, g, 0x7632);
    }
    uint32_t up[4], lo[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      up[d] = upper_nibbles(wrd[0][d], wrd[1][d]);
      lo[d] = lower_nibbles(wrd[0][d], wrd[1][d]);
    }
    // word m of four channels to the four words of channel d0 + m, which lie
    // together (a store of 16 bytes a lane; words stored one by one fill half a
    // sector each: 32 heads of 32k tokens 156 us, two-bit layout 172, against 152 and
    // 159)
    transpose4(up, m);
    transpose4(lo, m);
    const int W = 4 * (part * kD + d0 + m);
    uint8_t *vu = c.v_upper + grp * kG * (kD / 2);
    if (two_bit) {
      *reinterpret_cast<uint2 *>(vu + 2 * W) =
          make_uint2(bitsel(up[0] >> 2, up[1], 0x33333333u), bitsel(up[2] >> 2, up[3], 0x33333333u));
      *reinterpret_cast<uint2 *>(vu + kG * kD / 4 + 2 * W) =
          make_uint2(bitsel(up[0], up[1] << 2, 0x33333333u), bitsel(up[2], up[3] << 2, 0x33333333u));
    } else {
      *reinterpret_cast<uint4 *>(vu + 4 * W) = make_uint4(up[0], up[1], up[2], up[3]);
    }
    *reinterpret_cast<uint4 *>(c.v_lower + grp * kG * (kD / 2) + 4 * W) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  // 6. key codes and planes: thread = eight channels of a token (one word of
  // each plane), the same channels in every step
  {
    const int o = tid & 3;
    float zf[8], rf[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 z4 = *reinterpret_cast<const float4 *>(&S.kzf[8 * o + 4 * i]);
      const float4 r4 = *reinterpret_cast<const float4 *>(&S.krf[8 * o + 4 * i]);
      zf[4 * i] = z4.x; zf[4 * i + 1] = z4.y; zf[4 * i + 2] = z4.z; zf[4 * i + 3] = z4.w;
      rf[4 * i] = r4.x; rf[4 * i + 1] = r4.y; rf[4 * i + 2] = r4.z; rf[4 * i + 3] = r4.w;
    }
#pragma unroll 2
    for (int t = tid >> 2; t < kG; t += kQThreads / 4) {
      const uint2 q = codes8<true>(
          &kt[t][8 * o], *reinterpret_cast<const uint4 *>(&kt[t][8 * o]), zf, rf,
          [&](int i) { return S.kzf[8 * o + i]; },
          [&](int i) { return half_bits_to_float(S.ks[8 * o + i]); });
      const uint32_t ev = q.x, od = q.y;
      const int W = 16 * t + 4 * part + o;
      store_upper(c.k_upper + grp * kG * (kD / 2), W, upper_nibbles(ev, od), two_bit);
      *reinterpret_cast<uint32_t *>(c.k_lower + grp * kG * (kD / 2) + 4 * W) = lower_nibbles(ev, od);
    }
  }
  // 7. metadata: key scale / zero of the channel slice, value scale / zero of the quarter
  if (tid < kSlice) {
    uint16_t *m = c.meta + grp * 4 * 128;
    int kp = kmeta_pos(part * kSlice + tid), vp = vmeta_pos(part * kSlice + tid);
    if (!chk(kp >= 0 && kp < 128 && vp >= 0 && vp < 128, 21)) kp = vp = 0;
    m[QS_META_K_SCALE * 128 + kp] = S.ks[tid];
    m[QS_META_K_ZERO * 128 + kp] = S.kz[tid];
    m[QS_META_V_SCALE * 128 + vp] = S.vs[tid];
    m[QS_META_V_ZERO * 128 + vp] = S.vz[tid];
  }
}

// One CTA's share of quantizing a group of G tokens whose fp16 key and value
// rows (D channels each, row stride D) start at gk and gv: key channels
// [32 part, 32 part + 32) and value tokens [32 part, 32 part + 32), written
// as group `grp` (index into the n_grp entries of the group arrays).  32 QW
// threads.
template <int QW>
__device__ void quantize_part(FlushSmem<QW> &S, const __half *gk, const __half *gv,
                              const qs_cache &c, size_t n_grp, size_t grp, int part, int tid) {
  // checked build: a group index out of the arrays writes nothing (the same
  // for every thread of the CTA)
  if (!chk(in_range(grp, 1, n_grp), 20)) return;
  load_part<QW, false>(S.k, S.v, gk, gv, part, tid);
  __syncthreads();
  quantize_loaded(S, S.k, S.v, c, grp, part, tid);
}

// The prefill's shared memory: a second pair of row buffers (first, so the
// asynchronous copies stay 16-byte aligned) and the flush's.
template <int QW>
struct PrefillSmem {
  __half k1[kG][kSlice];
  __half v1[kSlice][kD];
  FlushSmem<QW> f;
  int place[kPrefillQuarters / 4 + 1];  // entries of the CTA's groups
};
// Six CTAs of four warps fit an SM (with five, 152 us where six take 147): 227 KB,
// and a KB of each CTA is the system's.
static_assert(6 * (sizeof(PrefillSmem<4>) + 1024) <= 227 * 1024, "six CTAs an SM");

}  // namespace

// n_next >= 0: flush the sequences whose buffer cannot take n_next more
// tokens (qs_need_flush's rule; mask unused); else the masked ones (all
// without a mask).
template <int QW>
__global__ void __launch_bounds__(32 * QW)
    flush_kernel(qs_cache c, Pages pg, const uint8_t *mask, int n_next) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  FlushSmem<QW> &S = *reinterpret_cast<FlushSmem<QW> *>(smem_raw);
  const int part = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  int32_t *st = c.state + (size_t)b * QS_STATE_WORDS;
  if (tid == 0) {
    const int fill = st[QS_ST_FILL], pending = st[QS_ST_PENDING], ng = st[QS_ST_N_GROUPS];
    int act = n_next >= 0 ? (fill + n_next > kRing) : (mask ? (mask[b] != 0) : 1);
    const bool lead = (h == 0 && part == 0);
    if (act && fill - pending < kG) {
      if (lead) atomicOr(&st[QS_ST_ERR], QS_DEV_FLUSH_UNCOMMITTED);
      act = 0;
    } else if (act && (ng < 0 || ng >= c.cap_groups)) {
      if (lead) atomicOr(&st[QS_ST_ERR], QS_DEV_CAPACITY);
      act = 0;
    }
    // (the page is looked up once: the entry that was found good is the one used)
    const long long place = act ? group_slot(c, pg, b, h, ng) : 0;
    if (place < 0) {
      if (lead) atomicOr(&st[QS_ST_ERR], QS_DEV_PAGE);
      act = 0;
    }
    S.place = (int)place;  // a group takes 33 KB: places stay far below 2^31
    S.act = act;
    S.base = st[QS_ST_HALF_BASE] & 1;
    S.g = ng;
  }
  __syncthreads();
  if (!S.act) return;
  const int base = S.base, g = S.g;
  const size_t bh = (size_t)b * c.H + h;
  const __half *gk = reinterpret_cast<const __half *>(c.buf_k) + (bh * kRing + base * kG) * kD;
  const __half *gv = reinterpret_cast<const __half *>(c.buf_v) + (bh * kRing + base * kG) * kD;

  quantize_part(S, gk, gv, c, group_slots(c, pg), (size_t)S.place, part, tid);
  __syncthreads();
  // every CTA of the sequence has read the old counters once the ticket
  // reaches kParts H - 1 (the planes are published by the kernel's end)
  if (tid == 0 && atom_add_acq_rel_gpu(&st[QS_ST_TICKET], 1) == kParts * c.H - 1) {
    st[QS_ST_N_GROUPS] = g + 1;
    st[QS_ST_HALF_BASE] = base ^ 1;
    st[QS_ST_FILL] -= kG;
    st[QS_ST_TICKET] = 0;
  }
}

// Bulk prefill of empty caches from a prompt (k, v: fp16 [B][H][T][D]).
// Grid (nq + 2, H, B), or, into pages, ((nq + 2) H, 1, B) with the heads of a
// page side by side: block x < nq quantizes group quarters [x Q, x Q + Q) of the
// sequence's head (quarter i: part i % 4 of group i / 4; Q = quarters), the next
// quarter's rows copied into the second buffer while the current one is quantized;
// the last two blocks copy buffer halves 0 and 1.  The CTA that arrives last on
// the sequence's ticket writes the counters, so every CTA reads the old (empty)
// ones first.
template <int QW>
__global__ void __launch_bounds__(32 * QW, 24 / QW)
    prefill_kernel(qs_cache c, Pages pg, const uint16_t *k, const uint16_t *v, int T,
                   const int32_t *len, int nq, int quarters) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  PrefillSmem<QW> &PS = *reinterpret_cast<PrefillSmem<QW> *>(smem_raw);
  FlushSmem<QW> &S = PS.f;
  const int x = pg.table ? blockIdx.x / c.H : blockIdx.x, h = pg.table ? blockIdx.x % c.H : blockIdx.y;
  const int b = blockIdx.z, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  int32_t *st = c.state + (size_t)b * QS_STATE_WORDS;
  if (pg.table)  // (read below, once the prompt's length is known)
    for (int g = 32 * tid; g < c.cap_groups; g += 32 * 32 * QW) prefetch_l1(pg.table + (size_t)b * c.cap_groups + g);
  if (tid == 0) {
    const int L = len[b];
    const bool lead = (h == 0 && x == 0);
    int act = 1, ng = 0;
    if (st[QS_ST_N_GROUPS] != 0 || st[QS_ST_FILL] != 0 || st[QS_ST_PENDING] != 0 || L < 0 ||
        L > T) {
      if (lead) atomicOr(&st[QS_ST_ERR], QS_DEV_PREFILL);
      act = 0;
    } else {
      ng = L > 2 * kG ? (L - 2 * kG + kG - 1) / kG : 0;
      if (ng > c.cap_groups) {
        if (lead) atomicOr(&st[QS_ST_ERR], QS_DEV_CAPACITY);
        act = 0;
      }
    }
    S.act = act;
    S.g = ng;
    S.base = act ? L - ng * kG : 0;  // fill
  }
  __syncthreads();
  if (!S.act) return;
  const int ng = S.g, fill = S.base;
  const size_t bh = (size_t)b * c.H + h;
  const uint16_t *kp = k + bh * T * kD, *vp = v + bh * T * kD;
  // Paged: every page the prompt needs, looked at by every CTA alike (while its
  // first rows are on their way): a bad one leaves the whole sequence unchanged.
  // bad_own: an entry that this thread has read already and will use is a bad one.
  auto pages_good = [&](bool bad_own) {
    if (!pg.table) return true;
    int bad = bad_own;
    for (int g = tid; g < ng; g += 32 * QW) bad |= group_slot(c, pg, b, h, g) < 0;
    if (!__syncthreads_or(bad)) return true;
    if (h == 0 && x == 0 && tid == 0) atomicOr(&st[QS_ST_ERR], QS_DEV_PAGE);
    return false;
  };
  if (x < nq) {
    const int q0 = x * quarters, q1 = min(q0 + quarters, 4 * ng);
    const __half *kh = reinterpret_cast<const __half *>(kp), *vh = reinterpret_cast<const __half *>(vp);
    // the rows of quarter i go to buffer i % 2 (a quarter whose rows fail the
    // checked build's range check is not copied)
    auto load = [&](int i) {
      const int g = i >> 2;
      if (chk(in_range(((size_t)g + 1) * kG, 0, (size_t)T), 22))
        load_part<QW, true>(i & 1 ? PS.k1 : S.k, i & 1 ? PS.v1 : S.v, kh + (size_t)g * kG * kD,
                                       vh + (size_t)g * kG * kD, i & 3, tid);
    };
    if (q0 < q1) load(q0);
    // (looked up once: a table read a quarter, even from L1, cost 9 % of the call)
    const int g0 = q0 >> 2;
    long long own = 0;
    if (tid < kPrefillQuarters / 4 + 1 && g0 + tid < ng) {
      own = group_slot(c, pg, b, h, g0 + tid);
      PS.place[tid] = (int)own;
    }
    if (!pages_good(own < 0)) {
      cp_async_wait<0>();
      return;
    }
    for (int i = q0; i < q1; ++i) {
      cp_async_wait<0>();
      // quarter i's rows, copied by every thread, are visible; the buffer and
      // the scratch of quarter i - 1 are free
      __syncthreads();
      if (i + 1 < q1) load(i + 1);
      const int g = i >> 2;
      const size_t grp = (size_t)PS.place[g - g0];
      // checked build: the group's prompt rows inside the prompt array
      if (chk(in_range(((size_t)g + 1) * kG, 0, (size_t)T), 22) &&
          chk(in_range(grp, 1, group_slots(c, pg)), 20))
        quantize_loaded(S, i & 1 ? PS.k1 : S.k, i & 1 ? PS.v1 : S.v, c, grp, i & 3, tid);
    }
  } else {
    if (!pages_good(false)) return;
    // buffer half x - nq: tokens i in [G half, G half + G) that are < fill
    const int i0 = (x - nq) * kG, i1 = min(i0 + kG, fill);
    const uint4 *ks = reinterpret_cast<const uint4 *>(kp + (size_t)ng * kG * kD);
    const uint4 *vs = reinterpret_cast<const uint4 *>(vp + (size_t)ng * kG * kD);
    uint4 *kd = reinterpret_cast<uint4 *>(c.buf_k + bh * kRing * kD);
    uint4 *vd = reinterpret_cast<uint4 *>(c.buf_v + bh * kRing * kD);
    if (chk(i1 <= kRing && (size_t)ng * kG + i1 <= (size_t)T, 23))
      // four rows' pieces a thread in flight at once
      for (int e0 = i0 * (kD / 8) + tid; e0 < i1 * (kD / 8); e0 += 4 * 32 * QW) {
        uint4 xk[4], xv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = e0 + u * 32 * QW;
          if (e < i1 * (kD / 8)) {
            xk[u] = ks[e];
            xv[u] = vs[e];
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = e0 + u * 32 * QW;
          if (e < i1 * (kD / 8)) {
            kd[e] = xk[u];
            vd[e] = xv[u];
          }
        }
      }
  }
  __syncthreads();
  if (tid == 0 && atom_add_acq_rel_gpu(&st[QS_ST_TICKET], 1) == (int)(gridDim.x * gridDim.y) - 1) {
    st[QS_ST_N_GROUPS] = ng;
    st[QS_ST_FILL] = fill;
    st[QS_ST_PENDING] = 0;
    st[QS_ST_HALF_BASE] = 0;
    st[QS_ST_TICKET] = 0;
  }
}

}  // namespace qs

using namespace qs;

namespace {

// Quarters per CTA, by the prompt's quarters per SM: 8 for a prompt of many waves
// of CTAs (more than 120 an SM; 32 heads of 32k tokens: 147 us, four 150); 4 where
// eight leave the last wave half empty (32 heads of 9k tokens: 48 us; eight 52);
// fewer for a short one, whose time is one CTA's chain of quarters: 2 up to ten an
// SM, 1 up to five (two heads of 1k tokens: 15.6 us with eight quarters of four
// warps a CTA).
int prefill_quarters(long long total, int sms) {
  if (total > 120ll * sms) return kPrefillQuarters;
  return total > 10ll * sms ? 4 : total > 5ll * sms ? 2 : 1;
}

template <int QW>
qs_status launch_prefill(const qs_cache &c, const Pages &pg, const uint16_t *k, const uint16_t *v, int T,
                         const int32_t *d_len, int gmax, int quarters, qs_stream_t stream) {
  static int ready = 0;
  const int smem = (int)sizeof(PrefillSmem<QW>);
  const qs_status s = set_smem_once((const void *)prefill_kernel<QW>, smem, &ready);
  if (s != QS_OK) return s;
  const int nq = (4 * gmax + quarters - 1) / quarters;
  const dim3 grid = pg.table ? dim3((unsigned)(nq + 2) * c.H, 1, c.B) : dim3(nq + 2, c.H, c.B);
  return launch_pdl(prefill_kernel<QW>, grid, dim3(32 * QW), smem, (cudaStream_t)stream, c, pg, k, v, T, d_len, nq, quarters);
}

qs_status prefill(const qs_cache &c, const Pages &pg, const uint16_t *k, const uint16_t *v, int32_t T,
                  const int32_t *d_len, qs_stream_t stream) {
  if (!k || !v || !d_len || T < 0 || T > (1 << 26)) return QS_ERR_ARG;
  if (!aligned16(k) || !aligned16(v)) return QS_ERR_ALIGN;
  const int gmax = T > 2 * kG ? (T - 2 * kG + kG - 1) / kG : 0;
  const long long total = (long long)4 * gmax * c.H * c.B;
  int sms = 0;
  const qs_status s = sm_count(&sms);
  if (s != QS_OK) return s;
  const int quarters = prefill_quarters(total, sms);
  if (quarters > 2) return launch_prefill<4>(c, pg, k, v, T, d_len, gmax, quarters, stream);
  // (one CTA of sixteen warps a quarter, at most two an SM; else eight warps)
  return total <= 2ll * sms
             ? launch_prefill<16>(c, pg, k, v, T, d_len, gmax, quarters, stream)
             : launch_prefill<8>(c, pg, k, v, T, d_len, gmax, quarters, stream);
}

template <int QW>
qs_status launch_flush(const qs_cache &c, const Pages &pg, const uint8_t *d_mask, int n_next,
                       qs_stream_t stream) {
  static int ready = 0;
  const int smem = (int)sizeof(FlushSmem<QW>);
  const qs_status s = set_smem_once((const void *)flush_kernel<QW>, smem, &ready);
  if (s != QS_OK) return s;
  return launch_pdl(flush_kernel<QW>, dim3(kParts, c.H, c.B), dim3(32 * QW), smem,
                    (cudaStream_t)stream, c, pg, d_mask, n_next);
}

// Two CTAs of sixteen warps fit an SM: beyond those the narrow ones win.
qs_status flush(const qs_cache &c, const Pages &pg, const uint8_t *d_mask, int n_next,
                qs_stream_t stream) {
  int sms = 0;
  const qs_status s = sm_count(&sms);
  if (s != QS_OK) return s;
  return (long long)kParts * c.H * c.B <= 2ll * sms
             ? launch_flush<kFlushWarps>(c, pg, d_mask, n_next, stream)
             : launch_flush<kBatchFlushWarps>(c, pg, d_mask, n_next, stream);
}

}  // namespace

extern "C" {

qs_status qs_prefill(const qs_cache *c, const uint16_t *k, const uint16_t *v, int32_t T,
                     const int32_t *d_len, qs_stream_t stream) {
  const qs_status s = check_cache(c);
  return s != QS_OK ? s : prefill(*c, Pages{nullptr, 0}, k, v, T, d_len, stream);
}

qs_status qs_prefill_paged(const qs_cache *c, const qs_pages *pg, const uint16_t *k,
                           const uint16_t *v, int32_t T, const int32_t *d_len, qs_stream_t stream) {
  qs_cache cc;
  Pages pages;
  const qs_status s = check_pages(c, pg, true, &cc, &pages);
  return s != QS_OK ? s : prefill(cc, pages, k, v, T, d_len, stream);
}

qs_status qs_quantize_flush(const qs_cache *c, const uint8_t *d_mask, qs_stream_t stream) {
  const qs_status s = check_cache(c);
  return s != QS_OK ? s : flush(*c, Pages{nullptr, 0}, d_mask, -1, stream);
}

qs_status qs_quantize_flush_paged(const qs_cache *c, const qs_pages *pg, const uint8_t *d_mask,
                                  qs_stream_t stream) {
  qs_cache cc;
  Pages pages;
  const qs_status s = check_pages(c, pg, true, &cc, &pages);
  return s != QS_OK ? s : flush(cc, pages, d_mask, -1, stream);
}

qs_status qs_quantize_flush_due(const qs_cache *c, int32_t n_next, qs_stream_t stream) {
  const qs_status s = check_cache(c);
  if (s != QS_OK) return s;
  if (n_next < 0 || n_next > kRing) return QS_ERR_ARG;
  return flush(*c, Pages{nullptr, 0}, nullptr, n_next, stream);
}

qs_status qs_quantize_flush_due_paged(const qs_cache *c, const qs_pages *pg, int32_t n_next,
                                      qs_stream_t stream) {
  qs_cache cc;
  Pages pages;
  const qs_status s = check_pages(c, pg, true, &cc, &pages);
  if (s != QS_OK) return s;
  if (n_next < 0 || n_next > kRing) return QS_ERR_ARG;
  return flush(cc, pages, nullptr, n_next, stream);
}

}  // extern "C"

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_quantize(unsigned long long *out2, int reset) {
  return read_check_failures(out2, reset);
}
#endif
