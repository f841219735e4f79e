// qs_attn_tree.cu -- decode attention of the nodes of a tree of drafted tokens.
// Few rows run through the split kernel (qs_split.cuh) in its tree variants.
#include "qs_split.cuh"

using namespace qs;

namespace qs {
namespace {

// Position of channel ch in a key scale / zero row, of token t of a group in a value
// row, and of token t of a quarter among the nibbles of a value row (include/qs.h).
__device__ __forceinline__ int k_row_pos(int ch) {
  const int r = ch & 7;
  return 32 * ((ch >> 3) & 3) + 8 * (ch >> 5) + 4 * ((r >> 1) & 1) + 2 * (r & 1) + (r >> 2);
}
__device__ __forceinline__ int v_row_pos(int t) {
  return 32 * (t >> 5) + 4 * (t & 7) + 2 * ((t >> 4) & 1) + ((t >> 3) & 1);
}
__device__ __forceinline__ int v_nibble(int t) {
  return 8 * ((t >> 1) & 3) + 4 * (t & 1) + 2 * ((t >> 4) & 1) + ((t >> 3) & 1);
}

// Nibble i of a group's upper plane, in either layout, or (two-bit drafts) its top half.
__device__ __forceinline__ int upper_nibble(const uint8_t *plane, int i, int bits, bool top_only) {
  if (bits == 4) return (plane[i >> 1] >> (4 * (i & 1))) & 15;
  const int w = i >> 3, src = 8 * (w >> 1) + (i & 7), sh = 2 * (w & 1);
  const int two = (((plane[src >> 1] >> (4 * (src & 1))) & 15) >> sh) & 3;
  if (top_only) return 4 * two;
  return 4 * two + (((((plane + 4096)[src >> 1] >> (4 * (src & 1))) & 15) >> sh) & 3);
}

__device__ __forceinline__ float half_at(const uint16_t *p) {
  return __half2float(*reinterpret_cast<const __half *>(p));
}

// One CTA of 128 threads per query row, one pass over its tokens 128 at a time:
// thread t forms the score of token t, then thread d the sum of channel d.
__global__ void __launch_bounds__(kD) tree_row_kernel(const Params prm, int mode) {
  __shared__ float s_q[kD], s_p[kG], s_zv[kG], s_red[4];
  const qs_cache &c = prm.c;
  const int row = blockIdx.x % prm.R, h = blockIdx.x / prm.R % c.H, b = blockIdx.x / prm.R / c.H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  int32_t *st = c.state + (size_t)b * QS_STATE_WORDS;
  const int ng = min(max(st[QS_ST_N_GROUPS], 0), c.cap_groups);
  const int fill = min(max(st[QS_ST_FILL], 0), kRing), hb = st[QS_ST_HALF_BASE] & 1;
  const size_t at = ((size_t)b * c.H + h) * prm.R + row;
  uint16_t *out = prm.out + at * kD;
  if (prm.n_tree > fill) {
    out[tid] = 0;
    if (tid == 0) {
      if (prm.lse) prm.lse[at] = -INFINITY;
      atomicOr(&st[QS_ST_ERR], QS_DEV_NQ_GT_FILL);
    }
    return;
  }
  uint64_t m[2];
  bool bad = false;
  tree_ancestors(prm.parent + (size_t)b * prm.n_tree, prm.n_tree, lane, m, bad);
  if (bad) atomicOr(&st[QS_ST_ERR], QS_DEV_TREE);
  const uint64_t sees = ancestors_of(m, prm.n_tree - prm.n_q + row % prm.n_q);
  const int tree0 = fill - prm.n_tree;
  const float q = half_at(prm.q + at * kD + tid);
  auto reduce = [&](float v, bool mx) {
    for (int o = 16; o; o >>= 1) {
      const float w = __shfl_xor_sync(0xffffffffu, v, o);
      v = mx ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if (lane == 0) s_red[warp] = v;
    __syncthreads();
    return mx ? fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]))
              : s_red[0] + s_red[1] + s_red[2] + s_red[3];
  };
  float M = -INFINITY, L = 0.f, O = 0.f;
  const int units = ng + (fill + kG - 1) / kG;
  const bool draft = mode == QS_DRAFT_UPPER4, two = c.upper_bits == 2;
  for (int u = 0; u < units; ++u) {
    float s = -INFINITY, zq = 0.f;
    long long grp = -1;
    if (u < ng) {
      grp = group_slot(c, prm.pg, b, h, u);
      if (grp < 0) {
        if (tid == 0) atomicOr(&st[QS_ST_ERR], QS_DEV_PAGE);
        continue;
      }
      const uint16_t *meta = c.meta + grp * 512;
      s_q[tid] = q * half_at(meta + k_row_pos(tid));
      zq = reduce(q * half_at(meta + 128 + k_row_pos(tid)), false);
      const uint8_t *ku = c.k_upper + grp * 8192, *kl = c.k_lower + grp * 8192;
      float dot = 0.f;
      for (int d = 0; d < kD; ++d) {
        const int i = tid * kD + d, up = upper_nibble(ku, i, c.upper_bits, draft);
        const int code = draft ? 16 * up + (two ? 32 : 8) : 16 * up + ((kl[i >> 1] >> (4 * (i & 1))) & 15);
        dot = fmaf(s_q[d], (float)code, dot);
      }
      s = (dot + zq) * prm.sl2;
    } else {
      const int i = (u - ng) * kG + tid;
      s_q[tid] = q;
      __syncthreads();
      if (i < fill && (i < tree0 || ((sees >> ((i - tree0) & 63)) & 1))) {
        const uint16_t *k = c.buf_k + (((size_t)b * c.H + h) * kRing + ((hb * kG + i) & (kRing - 1))) * kD;
        float dot = 0.f;
        for (int d = 0; d < kD; ++d) dot = fmaf(s_q[d], half_at(k + d), dot);
        s = dot * prm.sl2;
      }
    }
    const float mn = fmaxf(M, reduce(s, true));
    const float a = M == -INFINITY ? 0.f : exp2f(M - mn), p = s == -INFINITY ? 0.f : exp2f(s - mn);
    if (u < ng) {
      const uint16_t *meta = c.meta + grp * 512;
      s_p[tid] = p * half_at(meta + 256 + v_row_pos(tid));
      s_zv[tid] = p * half_at(meta + 384 + v_row_pos(tid));
    } else {
      s_p[tid] = p;
    }
    M = mn;
    L = L * a + reduce(p, false);
    O *= a;
    if (u < ng) {
      const uint8_t *vu = c.v_upper + grp * 8192, *vl = c.v_lower + grp * 8192;
      for (int t = 0; t < kG; ++t) {
        const int i = 32 * (128 * (t >> 5) + tid) + v_nibble(t & 31);
        const int up = upper_nibble(vu, i, c.upper_bits, draft);
        const int code = draft ? 16 * up + (two ? 32 : 8) : 16 * up + ((vl[i >> 1] >> (4 * (i & 1))) & 15);
        O = fmaf(s_p[t], (float)code, O + s_zv[t]);
      }
    } else {
      for (int t = 0; t < kG; ++t) {
        const int i = (u - ng) * kG + t;
        if (i >= fill || (i >= tree0 && !((sees >> ((i - tree0) & 63)) & 1))) continue;
        O = fmaf(s_p[t], half_at(c.buf_v + (((size_t)b * c.H + h) * kRing + ((hb * kG + i) & (kRing - 1))) * kD + tid), O);
      }
    }
    __syncthreads();
  }
  *reinterpret_cast<__half *>(out + tid) = __float2half_rn(O / L);
  if (prm.lse && tid == 0) prm.lse[at] = (M + log2f(L)) * 0.69314718055994531f;
}

constexpr int kMaxTreeRows = 512;

bool tree_sizes_ok(int32_t n_q, int32_t group) {
  return n_q >= 1 && n_q <= QS_MAX_TREE && group >= 1 && group <= kMaxTreeRows && group * n_q <= kMaxTreeRows;
}

}  // namespace
}  // namespace qs

extern "C" {

qs_status qs_attn_tree_workspace_size(const qs_cache *c, int32_t n_q, int32_t group, size_t *bytes) {
  qs_status s = check_cache_any(c);
  if (s != QS_OK) return s;
  if (!bytes || !tree_sizes_ok(n_q, group)) return QS_ERR_ARG;
  const int bits = c->upper_bits & ~QS_PAGED, R = group * n_q;
  if (R > kMaxR) {
    *bytes = 16;
    return QS_OK;
  }
  int P = 0;
  for (const qs_mode mode : {QS_DRAFT_UPPER4, QS_VERIFY_INT8}) {
    int p = 0;
    if ((s = grid_size<kListed | kTree>(mode, packed_rows(mode, R), bits, (R + 7) / 8, p)) != QS_OK) return s;
    if (p > P) P = p;
  }
  *bytes = ws_bytes(P, c->B, c->H, R);
  return QS_OK;
}

qs_status qs_attn_decode_tree(const qs_cache *c, const qs_pages *pg, qs_mode mode,
                              const int32_t *parent, int32_t n_tree, const uint16_t *q, int32_t n_q,
                              int32_t group, float softmax_scale, uint16_t *out, float *lse,
                              void *workspace, size_t workspace_bytes, qs_stream_t stream) {
  Params prm = {};
  qs_status s = check_pages(c, pg, false, &prm.c, &prm.pg);
  if (s != QS_OK) return s;
  if (!parent || !tree_sizes_ok(n_q, group) || n_tree < n_q || n_tree > QS_MAX_TREE) return QS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(parent) % 4) return QS_ERR_ALIGN;
  prm.parent = parent;
  prm.n_tree = n_tree;
  prm.wait_ns = kWaitLimitNs;
  cudaStream_t st = (cudaStream_t)stream;
  const int R = group * n_q;
  if (R > kMaxR) {
    s = check_queries(mode, q, softmax_scale, out, lse);
    if (s != QS_OK) return s;
    set_queries(prm, q, n_q, group, softmax_scale, out, lse);
    return launch_pdl(tree_row_kernel, dim3((unsigned)prm.c.B * prm.c.H * R), dim3(kD), 0, st, prm, (int)mode);
  }
  s = fill_params<kListed | kTree>(prm, mode, q, n_q, group, softmax_scale, out, lse, workspace,
                                   workspace_bytes);
  if (s != QS_OK) return s;
  if ((s = choose_clusters<kTree>(prm, mode)) != QS_OK) return s;
  const bool packed = packed_rows(mode, R);
  if (prm.C < 2) return launch_kind<kListed | kTree>(mode, packed, prm, st);
  prm.P = prm.c.B * prm.c.H * prm.K * prm.C;
  return launch_kind<kClustered | kTree>(mode, packed, prm, st);
}

}  // extern "C"

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_tree(unsigned long long *out2, int reset) {
  return read_check_failures(out2, reset);
}
#endif
