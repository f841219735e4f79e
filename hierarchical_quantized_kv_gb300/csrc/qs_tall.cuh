// qs_tall.cuh -- decode attention of many query rows per KV head (the nodes of a tree
// times the query heads that share a KV head): both products on the fifth-generation
// tensor cores, 128 rows at a time.
//
// Mathematics.  S = Q K^T and O = P V over tiles of 128 tokens, a group of the cache
// or half of the buffer, with a running maximum m and sum l per row:
//   P = 2^(S c - m),  O <- O a + P V,  l <- l a + sum P,  a = 2^(m_old - m),
// where m only moves when a row's maximum rises by more than 2^kRaise, so that O,
// which lives in tensor memory, is rescaled a few times in a call and not in every
// tile.  The values enter as their codes less 128, exact in fp16, and their scales go
// with the weights, P' = P s, rounded to fp16 (of a P and an s in fp32); the zeros are
// summed in fp32.  m is a maximum of S c + e, 2^e the least power of two above a unit's
// scales, so that P' uses fp16's range for values of any size and never passes it.  A
// token's mask (what a node of the tree sees) concerns the buffer alone.
//
// Design (GB300).
//  * One CTA per SM takes an equal range of (sequence, KV head, unit)s, as the split
//    kernel does, and writes a partial (O, m, l) for each segment it touches; a second
//    kernel joins them, by the differences of their m, which are scores.
//  * Roles (23 warps): one starts the bulk copies of planes and scales into a ring; one
//    makes scales and zeros ready; eight make the operand tiles of the keys (128 rows of
//    128 fp16, the 128-byte swizzle of K-major operands), four those of the values, in a
//    ring of three or four; one issues the MMAs (an elected lane, from uniform code); eight
//    do the softmax, a row per thread or, up to 64 rows, two threads.
//  * The roles share the instruction caches: the loops are kept short (unrolled over
//    whole tiles, with the segments' bookkeeping inside, an early form had 188 KB of code
//    and took 102 us instead of 62 for 240 rows of 32k).
//  * Two streams alternate on the tensor core, so that one multiplies while the other's
//    softmax runs.  With more than 128 rows they are two row tiles over the same keys
//    and values; else they take every other unit.
//  * S (fp32) and O lie in tensor memory; P replaces S there as fp16 and is the second
//    product's A operand, so scores never touch shared memory.
//  * Keys enter the product in two fp16 tiles that add up to them, K = T1 + T2.  Rounded
//    to fp16 once, a key with a large channel moves its scores by 1e-3 and more, and
//    the output by as much as six of its own roundings.  With s = s_h + s_l, s_h the
//    scale to three bits, and codes centred on 128, T1 = s_h c' + z_h is exact (a multiple
//    of a unit below 2048 of them) and T2 = s_l c' + z_l, a sixteenth of the range at
//    most, is rounded: two fused multiply-adds for a pair instead of one, and a third
//    product.  A warp of its own splits the scales and zeros of a group, once.
//  * The planes' layouts fit: keys are stored by token, channels side by side, and
//    values by channel, tokens side by side, both K-major as they are.  Within
//    eight channels the keys' nibbles come out as 0 4 1 5 2 6 3 7; the queries are
//    stored in that order too.
//
// Measured (replays on the same inputs): 240 rows over 32k tokens of 8 KV heads 66 us (17 by
// the two products' operations, 26 with the third); there the making of a unit's tiles and its products wait for
// one another, in the room that shared memory has. 26 rows over 8 x 32 heads, ragged to 64k
// tokens, 0.96 ms (0.37 by bytes): shared memory's bandwidth, of which the scores' operands
// take 128 KB a unit, and the chain of scores, softmax and weights.  A draft takes the same
// way, with both key tiles: 25 rows over 32k tokens of 32 heads 116 us (21 by bytes), 32
// rows of 8 heads 41 (5).
#pragma once

#include "qs_split.cuh"

namespace qs {
namespace {

constexpr int kTile = 128;                 // rows, tokens and channels of a tile
constexpr int kTileBytes = kTile * kTile * 2;
// Operand tiles in the ring: a unit has three (T1 and T2 of the keys, the values).
template <int MT>
constexpr int op_tiles() { return MT == 2 ? 3 : 4; }
// Warps of the softmax, and those that make operand tiles of keys and of values (whose
// tiles take a third of the work).  Each of the former arrives once on a tile's barrier,
// each of the latter kValArrive times.
constexpr int kSoftWarps = 8, kKeyWarps = 8, kValWarps = 4, kValArrive = kKeyWarps / kValWarps;
constexpr int kMmaWarp = kSoftWarps + kKeyWarps + kValWarps, kLoadWarp = kMmaWarp + 1, kPrepWarp = kMmaWarp + 2;
constexpr int kTallThreads = 32 * (kPrepWarp + 1);
constexpr float kRaise = 8.f;              // log2 by which a maximum may be behind
constexpr float kTallShift = 7.f;          // weights are taken as 2^(y - m + 7): P' up to 2^15
constexpr int kFlags = 8;                  // units whose flags are kept
constexpr int kScales = 3;                 // units whose value scales are kept
constexpr int kMaxTreeRows = 512;
constexpr int kStaticBytes = 3584;         // room for TallShared

// A piece of a unit in the ring of raw copies: keys or values.
template <int MODE>
struct TallCfg {
  static constexpr bool kDraft = MODE == QS_DRAFT_UPPER4;
  static constexpr int kUpOff = 0, kLowOff = 8192, kMetaOff = kDraft ? 8192 : 16384;
  // the keys' scales and zeros as their tiles' makers take them: s_h, s_l, z_h, z_l, in
  // the order of the key codes
  static constexpr int kPrepOff = kMetaOff + 512;
  static constexpr int kRawBytes = kPrepOff + 1024;
};
template <int MODE, int MT>
struct TallLayout {
  static constexpr int kQOff = 0;
  static constexpr int kOpOff = MT * kTileBytes;
  static constexpr int kRawOff = kOpOff + op_tiles<MT>() * kTileBytes;
  static constexpr int kScaleBytes = 1024;  // 128 tokens' s, and z + 128 s, in fp32
  static constexpr int kRest = 227 * 1024 - 1024 - kRawOff - 7 * kMaxB * 4 - kScales * kScaleBytes - kStaticBytes;
  static constexpr int kRawFit = kRest / TallCfg<MODE>::kRawBytes;
  static constexpr int kRaw = kRawFit < 10 ? kRawFit : 10;
  static constexpr int kScaleOff = kRawOff + kRaw * TallCfg<MODE>::kRawBytes;
  static constexpr int kTabOff = kScaleOff + kScales * kScaleBytes;
  static constexpr int kSmem = kTabOff + 7 * kMaxB * 4;  // (+ up to 1 KB of alignment)
  static_assert(kRaw >= 3, "");
};

struct TallParams {
  qs_cache c;
  Pages pg;
  const uint16_t *q;
  uint16_t *out;
  float *lse, *ws;
  const int32_t *parent;
  int n_tree, n_q, R;
  int n_mp;    // pairs of row tiles per KV head
  int rows;    // rows of a partial
  int P;       // CTAs
  float sl2;
  uint64_t wait_ns;
  int no_issue;
  size_t ws_floats;
};

// ------------------------------------------------------------------ tcgen05

// K-major operand tile with the 128-byte swizzle: rows of 128 bytes, eight of them to
// a 1024-byte pattern.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | 1ull << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// fp16 operands, fp32 sums, 128 x 128
constexpr uint32_t kMmaDesc = 1u << 4 | (kTile / 8) << 17 | (kTile / 16) << 24;

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kMmaDesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kMmaDesc), "r"(add)
      : "memory");
}
// True in one lane of a converged warp (the same one every time, as an arrival
// covers the MMAs of its own thread).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// An arrival on bar when every MMA issued so far is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void tc_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define QS_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define QS_S8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// 32 columns of the warp's 32 lanes; the load's wait is part of the statement, so
// that nothing can use the registers before it
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : QS_R8(v, 0), QS_R8(v, 8), QS_R8(v, 16), QS_R8(v, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
          QS_S8(v, 0),
      QS_S8(v, 8), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : QS_R8(v, 0), QS_R8(v, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::QS_S8(v, 0), "r"(addr)
               : "memory");
}

// ------------------------------------------------------- operand conversion

// Eight codes of a word pair as four fp16 pairs (elements j and j + 4), exact: the
// code goes into the mantissa of 1024 (with the draft's midpoint), and 1024 and 128 are
// taken off again.
template <int MODE>
__device__ __forceinline__ void code_pairs(uint32_t wu, uint32_t wl, uint32_t (&e)[4]) {
  if (MODE == QS_VERIFY_INT8) {
    const uint32_t ev = bitsel(wl, wu << 4, 0x0F0F0F0Fu), od = bitsel(wl >> 4, wu, 0x0F0F0F0Fu);
    constexpr uint32_t k64 = 0x64646464u;
    e[0] = prmt(ev, k64, 0x4240);
    e[1] = prmt(od, k64, 0x4240);
    e[2] = prmt(ev, k64, 0x4341);
    e[3] = prmt(od, k64, 0x4341);
  } else {
    constexpr uint32_t m = 0x00F000F0u, k = 0x64086408u;
    e[0] = ((wu << 4) & m) | k;
    e[1] = (wu & m) | k;
    e[2] = ((wu >> 4) & m) | k;
    e[3] = ((wu >> 8) & m) | k;
  }
}
// The two-bit draft: field sh (0 or 2) of each nibble of a C_U2 word.
template <int SH>
__device__ __forceinline__ void code_pairs2(uint32_t x, uint32_t (&e)[4]) {
  constexpr uint32_t m = 0x00C000C0u, k = 0x64206420u;
  e[0] = ((x << (6 - SH)) & m) | k;
  e[1] = (SH <= 2 ? ((x << (2 - SH)) & m) : 0) | k;
  e[2] = ((x >> (2 + SH)) & m) | k;
  e[3] = ((x >> (6 + SH)) & m) | k;
}
// The code less 128.
__device__ __forceinline__ uint32_t centred(uint32_t e) {
  return h2_as_u32(__hsub2(u32_as_h2(e), __half2half2(__ushort_as_half(0x6480))));
}
__device__ __forceinline__ uint32_t fma2(uint32_t e, uint32_t s, uint32_t z) {
  return h2_as_u32(__hfma2(u32_as_h2(e), u32_as_h2(s), u32_as_h2(z)));
}
// Pairs of fp32: one instruction for two.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 d;
  asm("mov.b64 %0, {%1,%2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float lo_of(f32x2 x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_of(f32x2 x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ f32x2 fma_f32x2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 mul_f32x2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add_f32x2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ ulonglong2 lds2x64(uint32_t a) {
  if (!chk(smem_in(a, 16), 1)) return make_ulonglong2(0, 0);
  ulonglong2 v;
  asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  if (!chk(smem_in(a, 16), 60)) return;
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Chunk c (eight elements) of row r of an operand tile.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int r, int c) {
  return tile + (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
// Eight channels in the order of the key codes.
__device__ __forceinline__ void sts_permuted(uint32_t a, uint4 x) {
  sts128(a, prmt(x.x, x.z, 0x5410), prmt(x.x, x.z, 0x7632), prmt(x.y, x.w, 0x5410), prmt(x.y, x.w, 0x7632));
}

// Four words of upper codes, and of lower ones, from word 4 i of a plane on; a two-bit draft gets its C_U2 words doubled.
template <int MODE, int UB>
__device__ __forceinline__ void raw_words4(uint32_t raw, int i, uint32_t (&u)[4], uint32_t (&l)[4]) {
  using C = TallCfg<MODE>;
  if (UB == 4) {
    const uint4 x = lds128(raw + C::kUpOff + 16 * i);
    u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
  } else {
    const uint2 a = lds64(raw + C::kUpOff + 8 * i);
    if (C::kDraft) {
      u[0] = u[1] = a.x;
      u[2] = u[3] = a.y;
    } else {
      const uint2 m = lds64(raw + C::kUpOff + 4096 + 8 * i);
      u[0] = upper_from2(a.x, m.x, 0); u[1] = upper_from2(a.x, m.x, 2);
      u[2] = upper_from2(a.y, m.y, 0); u[3] = upper_from2(a.y, m.y, 2);
    }
  }
  l[0] = l[1] = l[2] = l[3] = 0;
  if (!C::kDraft) {
    const uint4 x = lds128(raw + C::kLowOff + 16 * i);
    l[0] = x.x; l[1] = x.y; l[2] = x.z; l[3] = x.w;
  }
}
template <int MODE, int UB, int W>
__device__ __forceinline__ void word_pairs(uint32_t u, uint32_t l, uint32_t (&e)[4]) {
  if (UB == 2 && MODE == QS_DRAFT_UPPER4) code_pairs2<2 * (W & 1)>(u, e);
  else code_pairs<MODE>(u, l, e);
}

__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  if (!chk(smem_in(a, 8), 60)) return;
  asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// A group's scales and zeros, by one warp, four channels (tokens) a lane.  Keys: s_h
// s to its nearest three bits, 4 g .. 8 g with g a quarter of its power of two, s_l the
// rest; z + 128 s (the zero of centred codes) in z_h, its nearest multiple of g as far as
// 1024 g, and z_l.  |s_h c' + z_h| <= 8 * 128 g + 1024 g = 2048 g: exact.  (And z_h keeps it within
// fp16, -128 s_h + z_h >= -65504 and 127 s_h + z_h <= 65504, so that keys near the type's
// ends leave no infinity in a tile.)  A zero far outside the range, |z + 128 s| above about
// a half of 255 s, stays in T2 in part, which is then rounded at that size: at worst as
// one rounding of the key would.
template <int MODE>
__device__ __forceinline__ void prep_keys(uint32_t raw, int lane) {
  using C = TallCfg<MODE>;
  const uint2 sw = lds64(raw + C::kMetaOff + 8 * lane), zw = lds64(raw + C::kMetaOff + 256 + 8 * lane);
  uint32_t sh[2], sl[2], zh[2], zl[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t s2 = k ? sw.y : sw.x, z2 = k ? zw.y : zw.x;
    sh[k] = (s2 + 0x00800080u) & 0xFF00FF00u;  // (a scale is 514 at most)
    sl[k] = h2_as_u32(__hsub2(u32_as_h2(s2), u32_as_h2(sh[k])));
    const float2 s = __half22float2(u32_as_h2(s2)), z = __half22float2(u32_as_h2(z2));
    float h[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sf = i ? s.y : s.x, zc = fmaf(128.f, sf, i ? z.y : z.x);
      // g and 1 / g from the exponent (a scale of 0: the zero alone)
      const uint32_t ex = __float_as_uint(sf) & 0x7F800000u;
      const float g = __uint_as_float(ex) * 0.25f, inv = __uint_as_float((254u << 23) - ex) * 4.f;
      const float s_h = i ? __high2float(u32_as_h2(sh[k])) : __low2float(u32_as_h2(sh[k]));
      const float least = fmaxf(-1024.f, ceilf(fmaf(128.f, s_h, -65504.f) * inv));
      const float most = fminf(1024.f, floorf(fmaf(-127.f, s_h, 65504.f) * inv));
      h[i] = ex ? fminf(fmaxf(rintf(zc * inv), least), most) * g : __half2float(__float2half_rn(zc));
      l[i] = zc - h[i];
    }
    zh[k] = pack_half2(h[0], h[1]);
    zl[k] = pack_half2(l[0], l[1]);
  }
  const uint32_t at = raw + C::kPrepOff + 8 * lane;
  sts64(at, sh[0], sh[1]);
  sts64(at + 256, sl[0], sl[1]);
  sts64(at + 512, zh[0], zh[1]);
  sts64(at + 768, zl[0], zl[1]);
}
// Values: s, and the zero of centred codes, of each token in order, in fp32 (raw 0: a
// unit of buffer tokens, whose values are no codes; dead: nothing).  The four entries
// from position 4 k of a quarter on are tokens k, k + 8, k + 16, k + 24 of it.
// Returns e with s <= 2^e for all of them (for normal ones the least).
template <int MODE>
__device__ __forceinline__ int prep_values(uint32_t raw, bool dead, uint32_t to, int lane) {
  using C = TallCfg<MODE>;
  const uint32_t at = to + 128 * (lane >> 3) + 4 * (lane & 7);  // (token 32 (lane / 8) + lane % 8)
  float s[4], z[4];
  uint32_t most2 = dead ? 0 : 0x3C00u;
  if (raw && !dead) {
    const uint2 sw = lds64(raw + C::kMetaOff + 8 * lane), zw = lds64(raw + C::kMetaOff + 256 + 8 * lane);
    const float2 s0 = __half22float2(u32_as_h2(sw.x)), s1 = __half22float2(u32_as_h2(sw.y));
    const float2 z0 = __half22float2(u32_as_h2(zw.x)), z1 = __half22float2(u32_as_h2(zw.y));
    s[0] = s0.x; s[1] = s0.y; s[2] = s1.x; s[3] = s1.y;
    most2 = __vmaxu2(sw.x, sw.y);
    z[0] = z0.x; z[1] = z0.y; z[2] = z1.x; z[3] = z1.y;
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = fmaf(128.f, s[j], z[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] = dead ? 0.f : 1.f;
      z[j] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!chk(smem_in(at + 32 * j, 4) && smem_in(at + 512 + 32 * j, 4), 60)) continue;
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 32 * j), "f"(s[j]) : "memory");
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 512 + 32 * j), "f"(z[j]) : "memory");
  }
  // (not negative, so their bits keep the order)
  const uint32_t most = __reduce_max_sync(0xffffffffu, max(most2 & 0xFFFFu, most2 >> 16));
  return (int)((most + 0x3FFu) >> 10) - 15;
}

// A group's keys into the tiles T1 and T2, by the key warps (dw): a lane takes a word
// (eight channels) of a token, a warp two tokens at a time, kAhead of them loaded
// before the first is used; the scales stay in registers.  The lanes of a
// quarter-warp write all eight 16-byte columns of the swizzle.
template <int MODE, int UB>
__device__ __forceinline__ void keys_tile(uint32_t raw, uint32_t t1, uint32_t t2, int dw, int lane) {
  using C = TallCfg<MODE>;
  constexpr int kAhead = 4;
  static_assert(kTile % (2 * kKeyWarps * kAhead) == 0, "");
  const int w = lane & 15, f = 2 * (w & 1);
  // the 16-byte piece of a scale row that belongs to word w
  const uint32_t prep = raw + C::kPrepOff + 16 * ((w >> 2) + 4 * (w & 3));
  const uint4 sh = lds128(prep), sl = lds128(prep + 256), zh = lds128(prep + 512), zl = lds128(prep + 768);
#pragma unroll 1
  for (int t0 = 2 * dw + (lane >> 4); t0 < kTile; t0 += 2 * kKeyWarps * kAhead) {
    uint32_t u[kAhead], l[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int t = t0 + 2 * kKeyWarps * k;
      if (UB == 4) {
        u[k] = lds32(raw + C::kUpOff + 64 * t + 4 * w);
      } else {
        u[k] = lds32(raw + C::kUpOff + 32 * t + 4 * (w >> 1));
        if (C::kDraft) u[k] >>= f;
        else u[k] = upper_from2(u[k], lds32(raw + C::kUpOff + 4096 + 32 * t + 4 * (w >> 1)), f);
      }
      l[k] = C::kDraft ? 0 : lds32(raw + C::kLowOff + 64 * t + 4 * w);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      uint32_t e[4];
      word_pairs<MODE, UB, 0>(u[k], l[k], e);
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = centred(e[j]);
      const uint32_t at = tile_at(0, t0 + 2 * kKeyWarps * k, w);
      sts128(t1 + at, fma2(e[0], sh.x, zh.x), fma2(e[1], sh.y, zh.y), fma2(e[2], sh.z, zh.z), fma2(e[3], sh.w, zh.w));
      sts128(t2 + at, fma2(e[0], sl.x, zl.x), fma2(e[1], sl.y, zl.y), fma2(e[2], sl.z, zl.z), fma2(e[3], sl.w, zl.w));
    }
  }
}

// A group's value codes, less 128, by the value warps (one to a quarter): a lane takes a
// quarter's 32 tokens of a channel.  Word w's pair j is tokens 8 j + 2 w and the next,
// so pair j of the four words is eight tokens in order.
template <int MODE, int UB>
__device__ __forceinline__ void values_tile(uint32_t raw, uint32_t tile, int q, int lane) {
#pragma unroll 2
  for (int d = lane; d < kTile; d += 32) {
    uint32_t u[4], l[4], e[4][4];
    raw_words4<MODE, UB>(raw, kTile * q + d, u, l);
    word_pairs<MODE, UB, 0>(u[0], l[0], e[0]);
    word_pairs<MODE, UB, 1>(u[1], l[1], e[1]);
    word_pairs<MODE, UB, 2>(u[2], l[2], e[2]);
    word_pairs<MODE, UB, 3>(u[3], l[3], e[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sts128(tile_at(tile, d, 4 * q + j), centred(e[0][j]), centred(e[1][j]), centred(e[2][j]), centred(e[3][j]));
  }
}

// ------------------------------------------------------------------- kernel

// The order in which the MMAs take a piece's n units of keys (K, two tiles) and values
// (V): MT = 2: K0 V0 K1 V1 ..; MT = 1: K0 K1 V0 K2 V1 .. V(n-1).  Places with k tiles for
// the keys (k = 1: the raw copies), and the steps from one unit's to the next one's.
template <int MT>
__device__ __forceinline__ int first_values(int n, int k) {
  return MT == 2 || n <= 1 ? k : 2 * k;
}
template <int MT>
__device__ __forceinline__ int keys_step(int g, int k) {
  return MT == 1 && g == 0 ? k : k + 1;
}
template <int MT>
__device__ __forceinline__ int values_step(int g, int n, int k) {
  return MT == 1 && g == n - 2 ? 1 : k + 1;
}
// Item i of the 2 n in that order: its unit, and whether it is the values.
template <int MT>
__device__ __forceinline__ int item_of(int i, int n, bool &values) {
  if (MT == 2) {
    values = i & 1;
    return i >> 1;
  }
  values = i > 0 && (!(i & 1) || i == 2 * n - 1);
  return i == 2 * n - 1 ? n - 1 : values ? (i - 2) >> 1 : (i + 1) >> 1;
}

// A place in a ring of N and the parity of its turn.
template <int N>
struct Ring {
  int slot = 0, par = 0;
  __device__ __forceinline__ void add(int by) {  // up to N
    slot += by;
    if (slot >= N) {
      slot -= N;
      par ^= 1;
    }
  }
  __device__ __forceinline__ void add_any(int by) {
    const int x = slot + by;
    par ^= (x / N) & 1;
    slot = x % N;
  }
};

// A CTA's part of one segment.
struct Piece {
  int b, h, mp, ord;     // sequence, KV head, pair of row tiles, ordinal of the segment
  int u0, n;             // first unit in the segment, units
  int ng, fill, hb;      // of the sequence
};

__device__ __forceinline__ Tables tables_of(const int *tab) {
  int *t = const_cast<int *>(tab);
  return Tables{t, t + kMaxB, t + 2 * kMaxB, t + 3 * kMaxB, t + 4 * kMaxB, t + 5 * kMaxB, t + 6 * kMaxB};
}

struct TallShared {
  uint64_t raw_full[10], raw_empty[10], prep_full[10], op_full[4], op_empty[4];
  uint64_t scale_full[kScales], scale_empty[kScales];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2], q_full, q_empty, drain, pair[4];
  uint64_t bad[8];        // nodes with values that are not finite, per piece
  long long total;
  uint32_t tmem;
  int abort;
  int raw_dead[10], dead[kFlags], scale_exp[kScales];
  Piece piece[kPrepWarp + 1];  // each warp's current one
  float swap[2][kSoftWarps][32];  // between two threads of a row
};
static_assert(sizeof(TallShared) <= kStaticBytes, "");

// (Through shared memory, and not inlined: it runs once a piece in five places, whose
// loops share the instruction caches; and no thread may have a stack.  With nearly all
// of the SM's memory taken as shared memory, 27 warps' stacks of 200 bytes do not stay in
// what is left, and every access of theirs went to L2: 1290 us instead of 725.)
__device__ __noinline__ void piece_at(int B, int n_mp, const int *tab, int x, int x1, Piece *out) {
  const Tables T = tables_of(tab);
  int lo = 0, hi = B - 1;  // the last sequence whose units start at x or before (it has units)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (T.base[mid] <= x) lo = mid; else hi = mid - 1;
  }
  const int len = T.len[lo], off = x - T.base[lo], seg = off / len, u0 = off - seg * len;
  __syncwarp();
  out->b = lo;
  out->h = n_mp == 1 ? seg : seg >> 1;
  out->mp = n_mp == 1 ? 0 : seg & 1;
  out->ord = T.ord0[lo] + seg;
  out->u0 = u0;
  out->n = min(x1 - x, len - u0);
  out->ng = T.ng[lo];
  out->fill = T.fill[lo];
  out->hb = T.hb[lo];
  __syncwarp();
}

// bar's phase with the given parity, or false when the time is up or another role
// gave up.  (The clock is asked late: reading it takes longer than most waits.)
__device__ __forceinline__ bool tall_wait(TallShared &s, const uint64_t &bar, uint32_t parity, uint64_t ns) {
  const uint32_t a = smem_addr(&bar);
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(a, parity)) return true;
    if (i & 63) continue;
    if (*reinterpret_cast<volatile int *>(&s.abort)) return false;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > ns) {
      *reinterpret_cast<volatile int *>(&s.abort) = 1;
      return false;
    }
  }
}
// The same for a whole warp: all lanes agree.
__device__ __forceinline__ bool warp_wait(TallShared &s, const uint64_t &bar, uint32_t parity, uint64_t ns) {
  return __all_sync(0xffffffffu, tall_wait(s, bar, parity, ns));
}

// 128 buffer tokens from i0 on into an operand tile, straight from memory: keys...
__device__ __forceinline__ void buffer_keys_tile(const uint4 *src, int base, int i0, int fill, uint32_t tile, int dt) {
  constexpr int kStep = 2 * kKeyWarps;  // tokens at a time
#pragma unroll 1
  for (int t0 = dt >> 4; t0 < kTile; t0 += 2 * kStep) {
    uint4 x[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = t0 + kStep * k;
      x[k] = t < kTile && i0 + t < fill ? src[((base + t) & (kRing - 1)) * 16 + (dt & 15)] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (t0 + kStep * k < kTile) sts_permuted(tile_at(tile, t0 + kStep * k, dt & 15), x[k]);
  }
}
// ... and values, four tokens of eight channels per thread, turned in registers.
// Values of nodes (from token tree0 on) that are not finite become 0 (they meet the
// zero weights of rows that do not see the node); returns those nodes' bits.
__device__ __forceinline__ uint64_t buffer_values_tile(const uint4 *src, int base, int i0, int fill, int tree0,
                                                    uint32_t tile, int dt) {
  uint64_t bad = 0;
#pragma unroll 1
  for (int i = dt; i < 512; i += 32 * kValWarps) {
    const int tc = (i & 7) | ((i >> 4) & 8), dc = (i >> 3) & 15, t0 = 8 * tc + 4 * (i >> 8);
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = i0 + t0 + k < fill ? src[((base + t0 + k) & (kRing - 1)) * 16 + dc] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = i0 + t0 + k - tree0;
      if (j < 0) continue;
      unsigned f = drop_nonfinite(x[k].x);
      f |= drop_nonfinite(x[k].y);
      f |= drop_nonfinite(x[k].z);
      f |= drop_nonfinite(x[k].w);
      if (f) bad |= 1ull << (j & 63);
    }
    const uint32_t *xs = reinterpret_cast<const uint32_t *>(x);
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const uint32_t sel = d & 1 ? 0x7632 : 0x5410;
      const int k = d >> 1;
      sts64(tile_at(tile, 8 * dc + d, tc) + 8 * (i >> 8), prmt(xs[k], xs[4 + k], sel),
            prmt(xs[8 + k], xs[12 + k], sel));
    }
  }
  return bad;
}

// The row (of up to 128) that tile row t of stream s stands for with one row tile, or
// -1: few rows lie there twice, so that the streams' softmax warps (a quarter of the
// tile's rows each, and with it one of the SM's four schedulers) are not the same.
__device__ __forceinline__ int one_tile_row(int t, int s, int R) {
  if (R <= 32) return (t >> 5) == 1 + s ? t & 31 : -1;
  if (R <= 64) return (t >> 6) == s ? t & 63 : -1;
  return t;
}

// A piece's queries into their operand tiles (rows past the last: zeros).
template <int MT>
__device__ __forceinline__ void query_tiles(const uint4 *src, int row0, int R, uint32_t tiles, int dt) {
#pragma unroll 1
  for (int i0 = dt; i0 < MT * kTile * 16; i0 += 2 * 32 * kKeyWarps) {
    uint4 x[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = i0 + k * 32 * kKeyWarps;
      int row = row0 + (i >> 4);
      if (MT == 1) row = max(one_tile_row(row, 0, R), one_tile_row(row, 1, R));
      x[k] = i < MT * kTile * 16 && row >= 0 && row < R ? src[(size_t)row * 16 + (i & 15)] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = i0 + k * 32 * kKeyWarps, row = i >> 4;
      if (i < MT * kTile * 16)
        sts_permuted(tile_at(tiles + (row / kTile) * kTileBytes, row % kTile, i & 15), x[k]);
    }
  }
}

// Up to this many rows a row has two threads in the softmax, of warps that read the
// same lanes of tensor memory, for 64 tokens each.
constexpr int kPairedRows = 64;

// Column of the first of tokens 16 k .. of P, in the place of S: with each half of the
// tokens inside its half of S, so that two warps do not write what the other reads.
__device__ __forceinline__ constexpr int p_column(int k) { return 8 * k + (k >= 4 ? 32 : 0); }

// The tokens i0 .. i0 + 127 of the buffer that a row sees, a bit each: those in front
// of the tree, and of the tree the bits of sees.  The scores of the others (of tokens
// 16 k0 .. 16 k1 - 1) become -inf.
__device__ __forceinline__ void mask_scores(uint32_t t_s, int k0, int k1, int i0, int fill, int tree0, uint64_t sees,
                                            bool dead) {
#pragma unroll 1
  for (int k = k0 >> 1; k < k1 >> 1; ++k) {
    const int i = i0 + 32 * k, before = tree0 - i;  // tokens of the word in front of the tree
    uint32_t vis = before >= 32 ? ~0u : before <= 0 ? 0u : (1u << before) - 1;
    if (before < 32) {
      const uint64_t node = before >= 0 ? sees << before : -before < 64 ? sees >> -before : 0;
      vis |= (uint32_t)node;
    }
    const int have = fill - i;
    if (have < 32) vis &= have <= 0 ? 0u : (1u << have) - 1;
    if (dead) vis = 0;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t v[16];
      tc_ld16(t_s + 32 * k + 16 * h, v);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (!(vis >> j & 1)) v[j] = 0xFF800000u;
      tc_st16(t_s + 32 * k + 16 * h, v);
      vis >>= 16;
    }
  }
  tc_wait_st();
}

template <int MODE, int UB, int MT>
__global__ void __launch_bounds__(kTallThreads, 1) tall_kernel(const __grid_constant__ TallParams prm) {
  using L = TallLayout<MODE, MT>;
  using C = TallCfg<MODE>;
  constexpr int NR = L::kRaw, NOP = op_tiles<MT>();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ TallShared sh;
  // tiles start at multiples of 1024 bytes
  uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const qs_cache &c = prm.c;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, p = blockIdx.x;
  Tables T = tables_at(smem, L::kTabOff);
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 0; i < NR; ++i) {
      mbar_init(smem_addr(&sh.raw_full[i]), 1);
      mbar_init(smem_addr(&sh.raw_empty[i]), kKeyWarps + 1);
      mbar_init(smem_addr(&sh.prep_full[i]), 1);
    }
#pragma unroll 1
    for (int i = 0; i < NOP; ++i) {
      mbar_init(smem_addr(&sh.op_full[i]), kKeyWarps);
      mbar_init(smem_addr(&sh.op_empty[i]), 1);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.p_full[i]), 4);
      mbar_init(smem_addr(&sh.o_full[i]), 1);
      mbar_init(smem_addr(&sh.o_empty[i]), 4);
    }
    mbar_init(smem_addr(&sh.q_full), kKeyWarps);
    mbar_init(smem_addr(&sh.q_empty), 1);
#pragma unroll 1
    for (int i = 0; i < kScales; ++i) {
      mbar_init(smem_addr(&sh.scale_full[i]), 1);
      mbar_init(smem_addr(&sh.scale_empty[i]), MT == 2 ? 8 : 4);
    }
    mbar_init(smem_addr(&sh.drain), 1);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) mbar_init(smem_addr(&sh.pair[i]), 2);
    fence_mbar_init();
    sh.abort = 0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) sh.bad[i] = 0;
  }
  if (w == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_before_sync();
  }
  pdl_trigger();
  pdl_wait();
  if (w == 0) {
    qs_cache ct = c;  // segments: (sequence, KV head, pair of row tiles)
    ct.H = c.H * prm.n_mp;
    const long long tot = build_tables<kTile, true>(ct, prm.n_tree, 0, INT_MAX, T, lane);
    if (lane == 0) sh.total = tot;
  }
  __syncthreads();
  tc_after_sync();
  const long long U = sh.total;
  const int x0 = (int)range_lo(p, U, prm.P), x1 = (int)range_lo(p + 1, U, prm.P);
  const uint32_t tmem = sh.tmem;  // columns: S (and P) of stream s at 128 s, O at 256 + 128 s
  const uint64_t ns = prm.wait_ns;
  auto bar = [&](const uint64_t &b) { return smem_addr(&b); };
  auto tile = [&](int slot) { return sbase + L::kOpOff + slot * kTileBytes; };
  auto scale_at = [&](int slot) { return sbase + L::kScaleOff + slot * L::kScaleBytes; };
  auto raw_at = [&](int slot) { return sbase + L::kRawOff + slot * C::kRawBytes; };

  if (w == kLoadWarp) {
    // ------------------------------------------------------------- copies
    int r = 0, slot = 0, round = 0;  // raw pieces so far, the next one's place
    const uint64_t pol = l2_evict_first_policy();
    bool ok = true;
#pragma unroll 1
    for (int x = x0; ok && x < x1;) {
      piece_at(c.B, prm.n_mp, T.ng, x, x1, &sh.piece[w]);
      const volatile Piece &pc = sh.piece[w];  // (read where needed)
      const int n = pc.n;
      x += n;
      int at0 = -64, places = 0;  // lane k: the place of unit at0 + k
#pragma unroll 1
      for (int i = 0; i < 2 * n; ++i) {
        bool values;
        const int g = item_of<MT>(i, n, values), u = pc.u0 + g;
        if (u >= pc.ng) continue;  // the buffer is read by the warps that use it
        if (!values && g >= at0 + 32) {
          // (values come one unit behind the keys: keep one)
          at0 = max(0, g - 1);
          places = pc.u0 + at0 + lane < pc.ng
                       ? (int)group_slot(c, prm.pg, pc.b, pc.h, pc.u0 + at0 + lane) : -1;
        }
        const int place = __shfl_sync(0xffffffffu, places, (g - at0) & 31);
        if (round > 0 && !warp_wait(sh, sh.raw_empty[slot], (round - 1) & 1, ns)) {
          ok = false;
          break;
        }
        if (lane == 0 && !prm.no_issue) {
          const uint32_t dst = raw_at(slot), b = bar(sh.raw_full[slot]);
          sh.raw_dead[slot] = place < 0;
          if (place < 0 || !chk(in_range(place, 1, group_slots(c, prm.pg)) && smem_in(dst, C::kRawBytes), 61)) {
            if (!values) atomicOr(&c.state[(size_t)pc.b * QS_STATE_WORDS + QS_ST_ERR], QS_DEV_PAGE);
            mbar_arrive(b);
          } else {
            constexpr int kUp = C::kDraft && UB == 2 ? 4096 : 8192;
            mbar_arrive_expect_tx(b, kUp + (C::kDraft ? 0 : 8192) + 512);
            const size_t off = (size_t)place * 8192;
            // (with two pairs of row tiles the other one reads them again)
            if (prm.n_mp == 1)
              bulk_g2s_hint(dst + C::kUpOff, (values ? c.v_upper : c.k_upper) + off, kUp, b, pol);
            else
              bulk_g2s(dst + C::kUpOff, (values ? c.v_upper : c.k_upper) + off, kUp, b);
            if (!C::kDraft) {
              if (prm.n_mp == 1)
                bulk_g2s_hint(dst + C::kLowOff, (values ? c.v_lower : c.k_lower) + off, 8192, b, pol);
              else
                bulk_g2s(dst + C::kLowOff, (values ? c.v_lower : c.k_lower) + off, 8192, b);
            }
            bulk_g2s(dst + C::kMetaOff, c.meta + (size_t)place * 512 + (values ? 256 : 0), 512, b);
          }
        }
        ++r;
        if (++slot == NR) {
          slot = 0;
          ++round;
        }
      }
    }
    // after a timeout nothing may still land in shared memory when the CTA ends
    // (raw_full completes for every piece that was issued)
    if (*reinterpret_cast<volatile int *>(&sh.abort) && lane == 0 && !prm.no_issue) {
      const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
      for (int k = max(0, r - NR); k < r; ++k)
        while (!mbar_try_wait(bar(sh.raw_full[k % NR]), (k / NR) & 1))
          if (globaltimer_ns() - t0 > ns) break;
    }
  } else if (w == kMmaWarp) {
    // --------------------------------------------------------------- MMAs
    // The whole warp goes along, so that addresses and conditions are uniform; one
    // elected lane issues.
    {
      int n_s = 0, n_e = 0, piece = 0;  // bits 0, 1: parities of the streams' S, and of their sums
      int begun = 0;                    // bits: the stream has handed over sums before
      Ring<NOP> start;             // the piece's first operand tile
      bool ok = true;
      const uint64_t q_desc = operand_desc(sbase + L::kQOff), op_desc = operand_desc(sbase + L::kOpOff);
#pragma unroll 1
      for (int x = x0; ok && x < x1; ++piece) {
        piece_at(c.B, prm.n_mp, T.ng, x, x1, &sh.piece[w]);
        const volatile Piece &pc = sh.piece[w];  // (read where needed)
        const int n = pc.n, steps = MT == 2 ? 2 * n + 2 : n + 2;
        x += n;
        Ring<NOP> rk = start, rv = start;  // the next keys' tile, the next values'
        rv.add(first_values<MT>(n, 2));
#pragma unroll 1
        for (int t = 0; t < steps; ++t) {
          const int s = t & 1, g = MT == 2 ? t >> 1 : t;  // stream; unit whose scores are next
          const int gv = MT == 2 ? g - 1 : g - 2;         // unit whose values are next
          if (gv >= 0) {
            ok = warp_wait(sh, sh.p_full[s], ((n_s >> s) & 1) ^ 1, ns) &&
                 warp_wait(sh, sh.op_full[rv.slot], rv.par, ns);
            const bool first = MT == 2 ? gv == 0 : gv < 2;
            if (ok && first && (begun >> s & 1)) ok = warp_wait(sh, sh.o_empty[s], ((n_e >> s) & 1) ^ 1, ns);
            if (!ok) break;
            tc_after_sync();
            const uint64_t b = op_desc + rv.slot * (kTileBytes >> 4);
            const bool last = MT == 2 ? gv == n - 1 : gv >= n - 2;  // the stream's last unit here
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_ts(tmem + 256 + 128 * s, tmem + 128 * s + p_column(k), b + ((k >> 2) * (kTile * 8) + (k & 3) * 2),
                       !first || k > 0);
              if (MT == 1 || s == 1) mma_commit(bar(sh.op_empty[rv.slot]));
              if (last) mma_commit(bar(sh.o_full[s]));
            }
            __syncwarp();
            if (MT == 1 || s == 1) rv.add(values_step<MT>(gv, n, 2));
            if (last) {
              n_e ^= 1 << s;
              begun |= 1 << s;
            }
          }
          if (g < n) {
            Ring<NOP> r2 = rk;
            r2.add(1);
            // (the first tile's arrivals come before the second one's)
            ok = warp_wait(sh, sh.op_full[r2.slot], r2.par, ns);
            if (ok && g == 0) ok = warp_wait(sh, sh.q_full, piece & 1, ns);
            if (!ok) break;
            tc_after_sync();
            const uint64_t a = q_desc + (MT == 2 ? s * (kTileBytes >> 4) : 0);
            const uint64_t b1 = op_desc + rk.slot * (kTileBytes >> 4), b2 = op_desc + r2.slot * (kTileBytes >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t off = (k >> 2) * (kTile * 8) + (k & 3) * 2;  // (in units of 16 bytes)
                mma_ss(tmem + 128 * s, a + off, b1 + off, k > 0);
              }
              if (MT == 1 || s == 1) mma_commit(bar(sh.op_empty[rk.slot]));
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t off = (k >> 2) * (kTile * 8) + (k & 3) * 2;
                mma_ss(tmem + 128 * s, a + off, b2 + off, 1);
              }
              mma_commit(bar(sh.s_full[s]));
              if (MT == 1 || s == 1) {
                mma_commit(bar(sh.op_empty[r2.slot]));
                if (g == n - 1) mma_commit(bar(sh.q_empty));
              }
            }
            __syncwarp();
            n_s ^= 1 << s;
            if (MT == 1 || s == 1) rk.add(keys_step<MT>(g, 2));
          }
        }
        start.add_any(3 * n);
      }
      // no MMA may be in flight when the CTA gives its tensor memory back
      if (elect_one()) mma_commit(bar(sh.drain));
      __syncwarp();
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar(sh.drain), 0))
        if (globaltimer_ns() - t0 > ns) break;
    }
    __syncwarp();
  } else if (w == kPrepWarp) {
    // --------------------------------------------------- scales and zeros
    Ring<NR> raw;
    Ring<kScales> sc;
    int unit = 0;  // units so far
    bool ok = true;
#pragma unroll 1
    for (int x = x0; ok && x < x1;) {
      piece_at(c.B, prm.n_mp, T.ng, x, x1, &sh.piece[w]);
      const volatile Piece &pc = sh.piece[w];  // (read where needed)
      const int n = pc.n;
      x += n;
#pragma unroll 1
      for (int i = 0; i < 2 * n; ++i) {
        bool values, dead = false;
        const int g = item_of<MT>(i, n, values);
        const bool group = pc.u0 + g < pc.ng;
        if (group) {
          ok = warp_wait(sh, sh.raw_full[raw.slot], raw.par, ns);
          if (!ok) break;
          dead = *reinterpret_cast<volatile int *>(&sh.raw_dead[raw.slot]) != 0;
        }
        if (!values) {
          if (!group) continue;
          if (!dead) prep_keys<MODE>(raw_at(raw.slot), lane);
        } else {
          if (unit >= kScales) ok = warp_wait(sh, sh.scale_empty[sc.slot], sc.par ^ 1, ns);
          if (!ok) break;
          const int e = prep_values<MODE>(group ? raw_at(raw.slot) : 0, dead, scale_at(sc.slot), lane);
          if (lane == 0) *reinterpret_cast<volatile int *>(&sh.scale_exp[sc.slot]) = e;
        }
        __syncwarp();
        if (lane == 0) {
          if (group) {  // (of values too, so that the barrier's turns are the slot's)
            mbar_arrive(bar(sh.prep_full[raw.slot]));
            mbar_arrive(bar(sh.raw_empty[raw.slot]));
          }
          if (values) mbar_arrive(bar(sh.scale_full[sc.slot]));
        }
        if (group) raw.add(1);
        if (values) {
          sc.add(1);
          ++unit;
        }
      }
    }
  } else if (w >= kSoftWarps) {
    // ----------------------------------------------------- operand tiles
    const bool values = w >= kSoftWarps + kKeyWarps;
    const int dw = w - kSoftWarps - (values ? kKeyWarps : 0), dt = dw * 32 + lane;
    const int threads = 32 * (values ? kValWarps : kKeyWarps), arrivals = values ? kValArrive : 1;
    Ring<NOP> start;
    Ring<NR> raw_start;
    int piece = 0, unit0 = 0, o0 = 0;
    bool ok = true;
#pragma unroll 1
    for (int x = x0; ok && x < x1; ++piece) {
      piece_at(c.B, prm.n_mp, T.ng, x, x1, &sh.piece[w]);
      const volatile Piece &pc = sh.piece[w];  // (read where needed)
      const int n = pc.n, n_grp = min(n, max(0, pc.ng - pc.u0));  // units; groups among them
      if (!chk(pc.b >= 0 && pc.b < c.B && pc.h >= 0 && pc.h < c.H, 64)) break;
      const size_t bh = (size_t)pc.b * c.H + pc.h;
      x += n;
      if (!values) {
        // the piece's queries, once no MMA reads the last one's any more
        if (piece > 0 && !warp_wait(sh, sh.q_empty, (piece - 1) & 1, ns)) break;
        query_tiles<MT>(reinterpret_cast<const uint4 *>(prm.q + bh * prm.R * kD), pc.mp * 2 * kTile, prm.R,
                        sbase + L::kQOff, dt);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.q_full));
      } else if (dt == 0) {
        // (an entry that no warp here can have reached again, nor the softmax still
        // reads: each is within three pieces of this one)
        sh.bad[(piece + 4) & 7] = 0;
      }
      Ring<NOP> op = start;
      Ring<NR> raw = raw_start;
      int o = o0;  // operand tiles before this one
      if (values) {
        op.add(first_values<MT>(n, 2));
        raw.add(first_values<MT>(n_grp, 1));
        o += first_values<MT>(n, 2);
      }
#pragma unroll 1
      for (int g = 0; g < n; ++g) {
        Ring<NOP> op2 = op;  // (the keys' second tile)
        op2.add(1);
        // (tiles are consumed in the ring's order: with the second one free the first is)
        const Ring<NOP> &last = values ? op : op2;
        if (o + (values ? 0 : 1) >= NOP && !warp_wait(sh, sh.op_empty[last.slot], last.par ^ 1, ns)) {
          ok = false;
          break;
        }
        const uint32_t dst = tile(op.slot), dst2 = tile(op2.slot);
        if (g < n_grp) {
          // the copy; and, by a warp that has waited for it, what the keys' scales were
          // made into
          if (!warp_wait(sh, values ? sh.raw_full[raw.slot] : sh.prep_full[raw.slot], raw.par, ns)) {
            ok = false;
            break;
          }
          const bool dead = *reinterpret_cast<volatile int *>(&sh.raw_dead[raw.slot]) != 0;
          if (dead) {  // a group that is left out: nothing that could disturb the sums
#pragma unroll 1
            for (int k = dt; k < kTileBytes / 16; k += threads) {
              sts128(dst + 16 * k, 0, 0, 0, 0);
              if (!values) sts128(dst2 + 16 * k, 0, 0, 0, 0);
            }
          } else if (values) {
            values_tile<MODE, UB>(raw_at(raw.slot), dst, dw, lane);
          } else {
            keys_tile<MODE, UB>(raw_at(raw.slot), dst, dst2, dw, lane);
          }
          if (!values && dt == 0) *reinterpret_cast<volatile int *>(&sh.dead[(unit0 + g) % kFlags]) = dead;
          __syncwarp();
          if (lane < arrivals) mbar_arrive(bar(sh.raw_empty[raw.slot]));
          raw.add(values ? values_step<MT>(g, n_grp, 1) : keys_step<MT>(g, 1));
        } else {
          const int i0 = (pc.u0 + g - pc.ng) * kTile, base = pc.hb * kG + i0;
          const size_t row0 = bh * kRing * 16;
          if (!values) {
            // (fp16 already: T2 is zero)
            buffer_keys_tile(reinterpret_cast<const uint4 *>(c.buf_k) + row0, base, i0, pc.fill, dst, dt);
#pragma unroll 1
            for (int k = dt; k < kTileBytes / 16; k += threads) sts128(dst2 + 16 * k, 0, 0, 0, 0);
          } else {
            const uint64_t bad = buffer_values_tile(reinterpret_cast<const uint4 *>(c.buf_v) + row0, base, i0,
                                                    pc.fill, pc.fill - prm.n_tree, dst, dt);
            if (bad) atomicOr(reinterpret_cast<unsigned long long *>(&sh.bad[piece & 7]), bad);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane < arrivals) {
          mbar_arrive(bar(sh.op_full[op.slot]));
          if (!values) mbar_arrive(bar(sh.op_full[op2.slot]));
        }
        const int by = values ? values_step<MT>(g, n, 2) : keys_step<MT>(g, 2);
        op.add(by);
        o += by;
      }
      start.add_any(3 * n);
      raw_start.add_any(2 * n_grp);
      o0 += 3 * n;
      unit0 += n;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const bool paired = MT == 1 && prm.R <= kPairedRows;
    const int s = paired ? (w >> 1) & 1 : w >> 2, lanes = 32 * (w & 3), row_t = lanes + lane;  // stream; row in the tile
    // this warp's share of the tokens, and of the channels of O, in sixteens
    const int k0 = paired ? w & 4 : 0, k1 = paired ? k0 + 4 : 8;
    const uint32_t t_s = tmem + 128 * s + ((uint32_t)lanes << 16);
    const uint32_t t_o = tmem + 256 + 128 * s + ((uint32_t)lanes << 16);
    int n_s = 0, n_e = 0, n_x = 0, unit0 = 0;
    Ring<kScales> scale_start;
    bool ok = true;
    // what the row's other thread has
    auto swap = [&](float mine, float &other) {
      sh.swap[n_x & 1][w][lane] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh.pair[w & 3]));
      if (!warp_wait(sh, sh.pair[w & 3], n_x & 1, ns)) return false;
      other = sh.swap[n_x & 1][w ^ 4][lane];
      ++n_x;
      return true;
    };
#pragma unroll 1
    for (int x = x0, piece = 0; ok && x < x1; ++piece) {
      piece_at(c.B, prm.n_mp, T.ng, x, x1, &sh.piece[w]);
      const volatile Piece &pc = sh.piece[w];  // (read where needed)
      const int n = pc.n;
      x += n;
      // (row: of the KV head; row_p: in the partial)
      const int row_p = MT == 2 ? row_t : one_tile_row(row_t, s, prm.R);
      const int row = MT == 2 ? 2 * kTile * pc.mp + s * kTile + row_t : row_p;
      const bool live_warp = row >= 0 && row - lane < prm.R;
      if (!chk(pc.b >= 0 && pc.b < c.B, 64)) break;
      uint64_t sees = 0;
      if (pc.u0 + n > pc.ng && live_warp) {  // the buffer: the nodes that this row sees
        uint64_t mm[2];
        bool bad = false;
        tree_ancestors(prm.parent + (size_t)pc.b * prm.n_tree, prm.n_tree, lane, mm, bad);
        if (bad) atomicOr(&c.state[(size_t)pc.b * QS_STATE_WORDS + QS_ST_ERR], QS_DEV_TREE);
        sees = ancestors_of(mm, prm.n_tree - prm.n_q + row % prm.n_q);
      }
      // the weights' maximum: 2^(m c + em); bv: what the zeros of the values add
      float m = -INFINITY, em = 0.f, l = 0.f, bv = 0.f;
      int done = 0;
      // the stream's units of the piece
#pragma unroll 1
      for (int g = MT == 2 ? 0 : s; g < n; g += MT == 2 ? 1 : 2) {
        const int u = pc.u0 + g;
        ok = warp_wait(sh, sh.s_full[s], n_s & 1, ns);
        Ring<kScales> sc = scale_start;  // unit g's value scales
        sc.add_any(g);
        ok = ok && warp_wait(sh, sh.scale_full[sc.slot], sc.par, ns);
        if (!ok) break;
        ++n_s;
        tc_after_sync();
        if (live_warp) {
          const bool dead = u < pc.ng && *reinterpret_cast<volatile int *>(&sh.dead[(unit0 + g) % kFlags]);
          if (dead || u >= pc.ng)
            mask_scores(t_s, k0, k1, (u - pc.ng) * kTile, pc.fill, pc.fill - prm.n_tree, sees, dead);
          float mx = -INFINITY;
#pragma unroll 1
          for (int k = k0; k < k1; k += 2) {
            uint32_t v[32];
            tc_ld32(t_s + 16 * k, v);
            float a = __uint_as_float(v[0]), e = __uint_as_float(v[1]);
#pragma unroll
            for (int i = 2; i < 32; i += 2) {
              a = fmaxf(a, __uint_as_float(v[i]));
              e = fmaxf(e, __uint_as_float(v[i + 1]));
            }
            mx = fmaxf(mx, fmaxf(a, e));
          }
          if (paired) {
            float other;
            ok = swap(mx, other);
            if (!ok) break;
            mx = fmaxf(mx, other);
          }
          // (differences of scores, not of products: one may be far beyond what a
          // product keeps to the last bit)
          const float es = (float)*reinterpret_cast<volatile int *>(&sh.scale_exp[sc.slot]);
          const float up = (mx - m) * prm.sl2 + (es - em);
          const bool raise = mx > -INFINITY && (m == -INFINITY || up > kRaise);
          if (__any_sync(0xffffffffu, raise)) {
            const float a = raise ? (m == -INFINITY ? 0.f : fast_exp2(-up)) : 1.f;
            if (done > 0) {
#pragma unroll 1
              for (int k = k0; k < k1; ++k) {
                uint32_t v[16];
                tc_ld16(t_o + 16 * k, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * a);
                tc_st16(t_o + 16 * k, v);
              }
            }
            l *= a;
            bv *= a;
            if (raise) {
              m = mx;
              em = es;
            }
          }
          const float off = kTallShift - em, base = m == -INFINITY ? 0.f : -m;
          // The values are codes: P' = p s, and their zeros go with p alone, in fp32.  (The
          // largest p is a power of two, so P' of the token that counts most is exact.)
          const f32x2 sl2 = pack2(prm.sl2, prm.sl2), off2 = pack2(off, off), base2 = pack2(base, base);
          f32x2 l2 = pack2(0.f, 0.f), bv2 = l2;
          const uint32_t scales = scale_at(sc.slot);
#pragma unroll 1
          for (int k = k0; k < k1; ++k) {
            uint32_t y16[16], ph[8];
            tc_ld16(t_s + 16 * k, y16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const ulonglong2 s4 = lds2x64(scales + 64 * k + 16 * i), z4 = lds2x64(scales + 512 + 64 * k + 16 * i);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const f32x2 x = pack2(__uint_as_float(y16[4 * i + 2 * h]), __uint_as_float(y16[4 * i + 2 * h + 1]));
                const f32x2 y = fma_f32x2(add_f32x2(x, base2), sl2, off2);
                const f32x2 p = pack2(fast_exp2(lo_of(y)), fast_exp2(hi_of(y)));
                l2 = add_f32x2(l2, p);
                bv2 = fma_f32x2(p, h ? z4.y : z4.x, bv2);
                const f32x2 ps = mul_f32x2(p, h ? s4.y : s4.x);
                ph[2 * i + h] = pack_half2(lo_of(ps), hi_of(ps));
              }
            }
            tc_st8(t_s + p_column(k), ph);
          }
          l += lo_of(l2) + hi_of(l2);
          bv += lo_of(bv2) + hi_of(bv2);
          tc_wait_st();
        }
        ++done;
        tc_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(sh.p_full[s]));
          mbar_arrive(bar(sh.scale_empty[sc.slot]));
        }
      }
      if (!ok) break;
      if (paired && live_warp) {
        float l2, bv2;
        ok = swap(l, l2) && swap(bv, bv2);
        if (!ok) break;
        l += l2;
        bv += bv2;
      }
      // the piece's partial: rows side by side, four channels each; its sums without the
      // values' exponent (a power of two, so nothing is rounded), so that m alone stands
      // for their size and partials are compared by differences of scores too
      const float unit = __int_as_float((127 + (int)em) << 23);
      l *= unit;
      float *part = prm.ws + ((size_t)(pc.ord + p) * 2 + s) * prm.rows * (kD + 2);
      const bool mine = live_warp && row < prm.R &&
                        chk(in_range((size_t)(part - prm.ws), (size_t)prm.rows * (kD + 2), prm.ws_floats), 62);
      if (done > 0) {
        ok = warp_wait(sh, sh.o_full[s], n_e & 1, ns);
        if (!ok) break;
        ++n_e;
        tc_after_sync();
        if (live_warp) {
          if (sees & *reinterpret_cast<volatile uint64_t *>(&sh.bad[piece & 7])) l = NAN;
          const float add = l == l ? bv : NAN;
#pragma unroll 1
          for (int k = k0; k < k1; ++k) {
            uint32_t v[16];
            tc_ld16(t_o + 16 * k, v);
            if (mine)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                reinterpret_cast<float4 *>(part)[(4 * k + i) * prm.rows + row_p] =
                    make_float4((__uint_as_float(v[4 * i]) + add) * unit, (__uint_as_float(v[4 * i + 1]) + add) * unit,
                                (__uint_as_float(v[4 * i + 2]) + add) * unit, (__uint_as_float(v[4 * i + 3]) + add) * unit);
          }
        }
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.o_empty[s]));
      }
      if (mine && k0 == 0) {
        part[prm.rows * kD + row_p] = m;
        part[prm.rows * (kD + 1) + row_p] = l;
      }
      unit0 += n;
      scale_start.add_any(n);
    }
  }
  __syncthreads();
  if (sh.abort && threadIdx.x == 0)
    for (int b = 0; b < c.B; ++b) atomicOr(&c.state[(size_t)b * QS_STATE_WORDS + QS_ST_ERR], QS_DEV_TIMEOUT);
  if (w == kMmaWarp) {
    tc_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Joins the partials: a CTA has eight rows of a KV head, so that its threads walk the
// same partials (with eight rows across two heads a call of 25 rows took 4 us more); a
// thread takes four channels of a row and every kJoinParts-th partial, six of them in
// flight, and they meet at the end.  The CTAs that hold a segment, and where their
// partials lie, follow from the counters as in the kernel above.
constexpr int kJoinParts = 4, kJoinLane = 256, kJoinThreads = kJoinParts * kJoinLane, kJoinBatch = 6;

__global__ void __launch_bounds__(kJoinThreads) tall_join_kernel(const __grid_constant__ TallParams prm, int MT) {
  __shared__ int tab[7 * kMaxB];
  __shared__ long long s_total;
  __shared__ float4 s_o[kJoinThreads - kJoinLane];
  __shared__ float2 s_ml[kJoinThreads - kJoinLane];
  const qs_cache &c = prm.c;
  Tables T = tables_at(reinterpret_cast<uint8_t *>(tab), 0);
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x < 32) {
    qs_cache ct = c;
    ct.H = c.H * prm.n_mp;
    const long long tot = build_tables<kTile, true>(ct, prm.n_tree, 0, INT_MAX, T, threadIdx.x);
    if (threadIdx.x == 0) s_total = tot;
  }
  __syncthreads();
  const int part = threadIdx.x / kJoinLane, ti = threadIdx.x % kJoinLane;
  const int eights = (prm.R + 7) / 8, bh = blockIdx.x / eights, c4 = ti >> 3;
  const int row = 8 * (blockIdx.x % eights) + (ti & 7);
  const bool here = row < prm.R;
  const size_t at = (size_t)bh * prm.R + row;
  float M = -INFINITY, Ls = 0.f;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fold = [&](float mn, float m, float l, float4 o) {
    if (l == 0.f) return;  // nothing seen there (its sums were not written)
    const float f = m == -INFINITY ? 1.f : fast_exp2((m - mn) * prm.sl2);  // (no maximum: all NaN)
    A.x = fmaf(f, o.x, A.x); A.y = fmaf(f, o.y, A.y);
    A.z = fmaf(f, o.z, A.z); A.w = fmaf(f, o.w, A.w);
    Ls = fmaf(f, l, Ls);
  };
  auto rescale = [&](float mn) {
    const float a = M == -INFINITY ? 0.f : fast_exp2((M - mn) * prm.sl2);
    A.x *= a; A.y *= a; A.z *= a; A.w *= a;
    Ls *= a;
    M = mn;
  };
  int len = 0, b = 0;
  if (here) {
    const int h = bh % c.H;
    b = bh / c.H;
    len = T.len[b];
    if (len > 0) {
      const int seg = h * prm.n_mp + row / (2 * kTile), s0 = T.base[b] + seg * len, ord = T.ord0[b] + seg;
      const int plo = cta_of(s0, s_total, prm.P), phi = cta_of(s0 + len - 1, s_total, prm.P);
      const int row_t = row % kTile, s_at = MT == 2 ? (row / kTile) & 1 : 0, sh = MT == 2 ? 0 : 1;
      const size_t size = (size_t)prm.rows * (kD + 2);
      const int np = (phi - plo + 1) << sh;
#pragma unroll 1
      for (int k0 = part; k0 < np; k0 += kJoinParts * kJoinBatch) {
        float m[kJoinBatch], l[kJoinBatch];
        float4 o[kJoinBatch];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
          const int k = k0 + kJoinParts * i;
          m[i] = -INFINITY;
          l[i] = 0.f;
          if (k >= np) continue;
          const size_t off = ((size_t)(ord + plo + (k >> sh)) * 2 + s_at + (k & sh)) * size;
          if (!chk(in_range(off, size, prm.ws_floats), 63)) continue;
          const float *from = prm.ws + off;
          m[i] = from[prm.rows * kD + row_t];
          l[i] = from[prm.rows * (kD + 1) + row_t];
          o[i] = reinterpret_cast<const float4 *>(from)[c4 * prm.rows + row_t];
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) mn = fmaxf(mn, m[i]);
        rescale(mn);
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) fold(mn, m[i], l[i], o[i]);
      }
    }
  }
  if (part) {
    s_o[threadIdx.x - kJoinLane] = A;
    s_ml[threadIdx.x - kJoinLane] = make_float2(M, Ls);
  }
  __syncthreads();
  if (part || !here || !chk(in_range(at, 1, (size_t)c.B * c.H * prm.R), 65)) return;
  uint2 *out = reinterpret_cast<uint2 *>(prm.out + at * kD + 4 * c4);
  if (len == 0) {  // n_tree > fill
    *out = make_uint2(0, 0);
    if (c4 == 0) {
      if (prm.lse) prm.lse[at] = -INFINITY;
      atomicOr(&c.state[(size_t)b * QS_STATE_WORDS + QS_ST_ERR], QS_DEV_NQ_GT_FILL);
    }
    return;
  }
  float mn = M;
#pragma unroll
  for (int k = 0; k < kJoinParts - 1; ++k) mn = fmaxf(mn, s_ml[k * kJoinLane + ti].x);
  rescale(mn);
#pragma unroll
  for (int k = 0; k < kJoinParts - 1; ++k)
    fold(mn, s_ml[k * kJoinLane + ti].x, s_ml[k * kJoinLane + ti].y, s_o[k * kJoinLane + ti]);
  const float inv = 1.f / Ls;
  *out = make_uint2(pack_half2(A.x * inv, A.y * inv), pack_half2(A.z * inv, A.w * inv));
  if (prm.lse && c4 == 0) prm.lse[at] = fmaf(M, prm.sl2, log2f(Ls) - kTallShift) * 0.69314718055994531f;
}

// --------------------------------------------------------------- host side

// Rows of a partial: a row tile's, in eights (its four channels lie 16-byte aligned).
inline int tall_rows(int R) { return R < kTile ? (R + 7) / 8 * 8 : kTile; }
inline size_t tall_ws_bytes(int P, int B, int H, int R) {
  const int n_mp = (R + 2 * kTile - 1) / (2 * kTile), rows = tall_rows(R);
  return ((size_t)P + (size_t)B * H * n_mp) * 2 * rows * (kD + 2) * sizeof(float);
}

template <int MODE, int UB, int MT>
qs_status launch_tall(const TallParams &prm, cudaStream_t st) {
  constexpr int smem = TallLayout<MODE, MT>::kSmem + 1024;
  static int mask = 0;
  qs_status s = set_smem_once((const void *)tall_kernel<MODE, UB, MT>, smem, &mask);
  if (s != QS_OK) return s;
  s = launch_pdl(tall_kernel<MODE, UB, MT>, dim3(prm.P), dim3(kTallThreads), smem, st, prm);
  if (s != QS_OK) return s;
  return launch_pdl(tall_join_kernel, dim3((unsigned)(prm.c.B * prm.c.H * ((prm.R + 7) / 8))), dim3(kJoinThreads), 0, st, prm, MT);
}
template <int MODE>
qs_status launch_tall_mode(const TallParams &prm, cudaStream_t st) {
  const bool two = prm.R > kTile;
  if (prm.c.upper_bits == 2) return two ? launch_tall<MODE, 2, 2>(prm, st) : launch_tall<MODE, 2, 1>(prm, st);
  return two ? launch_tall<MODE, 4, 2>(prm, st) : launch_tall<MODE, 4, 1>(prm, st);
}

}  // namespace
}  // namespace qs
