// qs_read.cu -- reading the cache back: a window of each sequence's tokens as
// fp16 rows, the quantized groups as the draft or the verify pass sees them,
// the buffered tokens as they are.
//
//   k[t][d] = s_K[d] code + z_K[d],   v[t][d] = s_V[t] code + z_V[t],
//   code = 16 C_U + C_L (verify), 16 C_U + 8 or 64 C_U2 + 32 (draft),
// rounded once to fp16 (a code is exact in fp16, so one half-precision fused
// multiply-add is the correctly rounded value).
//
// Bound by HBM: per token and head 264 B (verify; draft 136 B, two-bit draft
// 72 B) come in and 512 B go out.
#include "qs_common.cuh"

namespace qs {
namespace {

constexpr int kReadThreads = 256;
// shared-memory row of a value tile: 16 bytes of padding, so that the eight
// rows of a transposed 8x8 store fall into different banks
constexpr int kTileRow = 2 * kD + 16;

// (a plain load but for L1: see pdl_wait)
__device__ __forceinline__ uint32_t ld_stream(const uint8_t *p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// The raw bits behind eight nibbles: word W of a group's 4-bit plane.
struct Raw {
  uint32_t u, m, l;
};

template <int MODE, int UB>
__device__ __forceinline__ Raw load_raw(const uint8_t *up, const uint8_t *lo, int W) {
  Raw r{0, 0, 0};
  if (UB == 4) {
    r.u = ld_stream(up + 4 * W);
  } else {
    r.u = ld_stream(up + 4 * (W >> 1));
    if (MODE == QS_VERIFY_INT8) r.m = ld_stream(up + 4096 + 4 * (W >> 1));
  }
  if (MODE == QS_VERIFY_INT8) r.l = ld_stream(lo + 4 * W);
  return r;
}

// Codes of nibbles 0, 2, 4, 6 (ev) and 1, 3, 5, 7 (od), a byte each.
template <int MODE, int UB>
__device__ __forceinline__ void codes8(const Raw &r, int W, uint32_t &ev, uint32_t &od) {
  const int sh = 2 * (W & 1);  // two-bit layout: which field of its word
  if (MODE == QS_DRAFT_UPPER4 && UB == 2) {
    const uint32_t t = r.u >> sh;
    ev = ((t & 0x03030303u) << 6) | 0x20202020u;
    od = ((t & 0x30303030u) << 2) | 0x20202020u;
    return;
  }
  const uint32_t wu =
      UB == 4 ? r.u : (((r.u << (2 - sh)) & 0xCCCCCCCCu) | ((r.m >> sh) & 0x33333333u));
  if (MODE == QS_DRAFT_UPPER4) {
    ev = ((wu << 4) & 0xF0F0F0F0u) | 0x08080808u;
    od = (wu & 0xF0F0F0F0u) | 0x08080808u;
  } else {
    ev = bitsel(r.l, wu << 4, 0x0F0F0F0Fu);
    od = bitsel(r.l >> 4, wu, 0x0F0F0F0Fu);
  }
}

// Two codes, as the halves 1024 + code, to s * code + z; a sum past the
// largest fp16 value (a group that reaches the type's ends, its scale rounded
// up) is held there.
__device__ __forceinline__ uint32_t dequant2(uint32_t magic, uint32_t s, uint32_t z) {
  const __half2 c = __hsub2(u32_as_h2(magic), u32_as_h2(0x64006400u));
  const __half2 x = __hfma2(u32_as_h2(s), c, u32_as_h2(z));
  return h2_as_u32(__hmin2(x, u32_as_h2(0x7BFF7BFFu)));
}
constexpr uint32_t kMagic = 0x64646464u;  // high byte of 1024 + code

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1,
                                                  uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

// Grid (128-token units the window touches, H, B), or, from pages, (units x H,
// 1, B) with the heads of a page side by side: one CTA reads one unit of one
// head.  Keys are token-major like the output: a thread turns eight
// nibbles of a row into 16 output bytes.  Values are stored channel-major: a
// warp's word holds token pairs of one channel per lane, exactly the 8x8
// fragments that a transposed matrix store turns into token-major rows of a
// shared tile.
template <int MODE, int UB>
__global__ void __launch_bounds__(kReadThreads)
    read_kernel(qs_cache c, Pages pg, int tok0, int T, uint16_t *k_out, uint16_t *v_out) {
  __shared__ __align__(16) uint8_t tile[kG * kTileRow];
  __shared__ __align__(16) uint16_t ks[kD], kz[kD];
  const int h = pg.table ? blockIdx.x % c.H : blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  // unit: tokens [128 u, 128 u + 128)
  const int u = tok0 / kG + (pg.table ? blockIdx.x / c.H : blockIdx.x);
  pdl_trigger();
  pdl_wait();
  const int32_t *st = c.state + (size_t)b * QS_STATE_WORDS;
  const int ng = min(max(st[QS_ST_N_GROUPS], 0), c.cap_groups);
  const size_t bh = (size_t)b * c.H + h;
  // output row r of the unit is token 128 u + r, row 128 u + r - tok0 of out
  const int r_lo = max(0, tok0 - u * kG), r_hi = (int)min((long long)kG, (long long)tok0 + T - (long long)u * kG);
  const long long out0 = ((long long)bh * T + ((long long)u * kG - tok0)) * kD;
  // checked build: the 16 bytes at dst are in the output and in this head's rows
  auto row_ok = [&](long long dst) {
    return dst >= (long long)bh * T * kD && dst + 8 <= (long long)(bh + 1) * T * kD &&
           bh < (size_t)c.B * c.H;
  };
  if (u >= ng) {
    const int fill = min(max(st[QS_ST_FILL], 0), kRing);
    const int i0 = (u - ng) * kG, base = (st[QS_ST_HALF_BASE] & 1) * kG;
    const int hi = min(r_hi, fill - i0);  // rows [r_lo, hi) of the unit
    if (u - ng > 1) return;
    // (four rows' pieces a thread in flight at once)
    for (int e0 = r_lo * (kD / 8) + tid; e0 < hi * (kD / 8); e0 += 4 * kReadThreads) {
      uint4 xk[4], xv[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int e = e0 + n * kReadThreads, r = e / (kD / 8);
        if (e >= hi * (kD / 8)) continue;
        const size_t row = bh * kRing + ((base + i0 + r) & (kRing - 1));
        const size_t src = row * kD + 8 * (e % (kD / 8));
        if (!chk(in_range(row, 1, (size_t)c.B * c.H * kRing), 51)) {
          xk[n] = xv[n] = make_uint4(0, 0, 0, 0);
          continue;
        }
        if (k_out) xk[n] = *reinterpret_cast<const uint4 *>(c.buf_k + src);
        if (v_out) xv[n] = *reinterpret_cast<const uint4 *>(c.buf_v + src);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int e = e0 + n * kReadThreads;
        if (e >= hi * (kD / 8)) continue;
        const long long dst = out0 + (long long)e * 8;
        if (!chk(row_ok(dst), 52)) continue;
        if (k_out) *reinterpret_cast<uint4 *>(k_out + dst) = xk[n];
        if (v_out) *reinterpret_cast<uint4 *>(v_out + dst) = xv[n];
      }
    }
    return;
  }
  const long long grp = group_slot(c, pg, b, h, u);
  if (grp < 0) {
    if (h == 0 && tid == 0) atomicOr(&c.state[(size_t)b * QS_STATE_WORDS + QS_ST_ERR], QS_DEV_PAGE);
    return;
  }
  if (!chk(in_range((size_t)grp, 1, group_slots(c, pg)), 50)) return;
  constexpr int kPlane = kG * kD / 2, kIter = kPlane / 4 / kReadThreads;
  const uint16_t *meta = c.meta + (size_t)grp * 4 * 128;
  const int w = tid >> 5, lane = tid & 31, r = lane >> 2, cq = lane & 3;
  Raw kr[kIter], vr[kIter];
  if (k_out) {
#pragma unroll
    for (int i = 0; i < kIter; ++i)
      kr[i] = load_raw<MODE, UB>(c.k_upper + grp * kPlane, c.k_lower + grp * kPlane, tid + kReadThreads * i);
  }
  // value word of item i: quarter w / 2, channel 8 md + r, tokens around 2 cq
  auto v_word = [&](int i) { return ((w >> 1) * kD + 8 * ((w & 1) * kIter + i) + r) * 4 + cq; };
  if (v_out) {
#pragma unroll
    for (int i = 0; i < kIter; ++i)
      vr[i] = load_raw<MODE, UB>(c.v_upper + grp * kPlane, c.v_lower + grp * kPlane, v_word(i));
  }
  if (tid < kD) {  // key scales and zeros to channel order
    const int p = tid;
    const int ch = 32 * ((p >> 3) & 3) + 8 * (p >> 5) + 2 * ((p >> 2) & 1) + ((p >> 1) & 1) + 4 * (p & 1);
    ks[ch] = meta[QS_META_K_SCALE * 128 + p];
    kz[ch] = meta[QS_META_K_ZERO * 128 + p];
  }
  if (v_out) {
    // scales of the token pairs (2 cq, 2 cq + 1) + 0, 8, 16, 24: the lane's
    // eight values lie together
    const int p0 = 32 * (w >> 1) + 8 * cq;
    const uint4 sw = *reinterpret_cast<const uint4 *>(meta + QS_META_V_SCALE * 128 + p0);
    const uint4 zw = *reinterpret_cast<const uint4 *>(meta + QS_META_V_ZERO * 128 + p0);
    const uint32_t s[4] = {prmt(sw.x, sw.z, 0x5410), prmt(sw.x, sw.z, 0x7632),
                           prmt(sw.y, sw.w, 0x5410), prmt(sw.y, sw.w, 0x7632)};
    const uint32_t z[4] = {prmt(zw.x, zw.z, 0x5410), prmt(zw.x, zw.z, 0x7632),
                           prmt(zw.y, zw.w, 0x5410), prmt(zw.y, zw.w, 0x7632)};
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      uint32_t ev, od;
      codes8<MODE, UB>(vr[i], v_word(i), ev, od);
      const int md = (w & 1) * kIter + i;
      // matrix m: tokens 8 m .. 8 m + 7 of the quarter; this lane names row
      // lane % 8 of matrix lane / 8
      uint32_t addr = smem_addr(tile) + (32 * (w >> 1) + lane) * kTileRow + 16 * md;
      if (!chk(addr + 16 <= smem_addr(tile) + (uint32_t)sizeof(tile), 53)) addr = smem_addr(tile);
      stmatrix_x4_trans(addr, dequant2(prmt(ev, kMagic, 0x4240), s[0], z[0]),
                        dequant2(prmt(od, kMagic, 0x4240), s[1], z[1]),
                        dequant2(prmt(ev, kMagic, 0x4341), s[2], z[2]),
                        dequant2(prmt(od, kMagic, 0x4341), s[3], z[3]));
    }
  }
  __syncthreads();
  if (k_out) {
    const int col = 8 * (tid & 15);  // the thread's channels, the same in every row
    const uint4 s4 = *reinterpret_cast<const uint4 *>(ks + col), z4 = *reinterpret_cast<const uint4 *>(kz + col);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int W = tid + kReadThreads * i, row = W >> 4;
      uint32_t ev, od;
      codes8<MODE, UB>(kr[i], W, ev, od);
      const uint32_t a = prmt(ev, od, 0x5140), d = prmt(ev, od, 0x7362);  // channels 0..3, 4..7
      uint4 x;
      x.x = dequant2(prmt(a, kMagic, 0x4140), s4.x, z4.x);
      x.y = dequant2(prmt(a, kMagic, 0x4342), s4.y, z4.y);
      x.z = dequant2(prmt(d, kMagic, 0x4140), s4.z, z4.z);
      x.w = dequant2(prmt(d, kMagic, 0x4342), s4.w, z4.w);
      if (row >= r_lo && row < r_hi && chk(row_ok(out0 + row * kD + col), 52))
        *reinterpret_cast<uint4 *>(k_out + out0 + row * kD + col) = x;
    }
  }
  if (v_out) {
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int e = tid + kReadThreads * i, row = e >> 4, col = 8 * (e & 15);
      const uint4 x = *reinterpret_cast<const uint4 *>(tile + row * kTileRow + 2 * col);
      if (row >= r_lo && row < r_hi && chk(row_ok(out0 + row * kD + col), 52))
        *reinterpret_cast<uint4 *>(v_out + out0 + row * kD + col) = x;
    }
  }
}

template <int MODE>
qs_status launch_read(const qs_cache &c, const Pages &pg, int tok0, int T, uint16_t *k, uint16_t *v,
                      cudaStream_t s) {
  const unsigned n = (tok0 + T - 1) / kG - tok0 / kG + 1;
  const dim3 grid = pg.table ? dim3(n * c.H, 1, c.B) : dim3(n, c.H, c.B), block(kReadThreads);
  return c.upper_bits == 2 ? launch_pdl(read_kernel<MODE, 2>, grid, block, 0, s, c, pg, tok0, T, k, v)
                           : launch_pdl(read_kernel<MODE, 4>, grid, block, 0, s, c, pg, tok0, T, k, v);
}

}  // namespace
}  // namespace qs

using namespace qs;

extern "C" qs_status qs_cache_read(const qs_cache *c, const qs_pages *pg, qs_mode mode, int32_t tok0,
                                   int32_t T, uint16_t *k, uint16_t *v, qs_stream_t stream) {
  qs_cache cc;
  Pages pages;
  const qs_status s = check_pages(c, pg, false, &cc, &pages);
  if (s != QS_OK) return s;
  if (mode != QS_DRAFT_UPPER4 && mode != QS_VERIFY_INT8) return QS_ERR_ARG;
  if ((!k && !v) || tok0 < 0 || tok0 > (1 << 30) || T < 1 || T > (1 << 26)) return QS_ERR_ARG;
  if ((k && !aligned16(k)) || (v && !aligned16(v))) return QS_ERR_ALIGN;
  return mode == QS_DRAFT_UPPER4
             ? launch_read<QS_DRAFT_UPPER4>(cc, pages, tok0, T, k, v, (cudaStream_t)stream)
             : launch_read<QS_VERIFY_INT8>(cc, pages, tok0, T, k, v, (cudaStream_t)stream);
}

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_read(unsigned long long *out2, int reset) {
  return read_check_failures(out2, reset);
}
#endif
