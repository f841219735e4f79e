// qs_attn_list.cu -- entry points of the decode attention over listed groups:
// the groups of a paged cache, and the groups selected for each head (of a
// contiguous or a paged cache).  The kernel is the contiguous one's
// (qs_split.cuh) in its listed variants: a segment's units are entries of a
// list, looked up at kernel start beside the first copies, so the stream of
// bulk copies and everything after it stay the same.
#include "qs_split.cuh"

using namespace qs;

namespace {

// CTAs that share a segment in the clustered kernel; 1: the split kernel.
// The clustered kernel starts and ends about 7 us sooner (verify: 11 us), but
// gives every segment as many CTAs as every other and leaves some of the SMs
// idle (sizes are powers of two).  So it is for segments of equal length, one
// sequence or selections, where the longer share of a CTA costs less than
// that: measured, 0.36 us a unit for a draft and 0.6 us for a verify pass, for
// every eight query rows.  Split against clustered, in us:
//   one sequence, 32 heads, 32 selected groups, draft      18.0   12.7
//   one sequence, 32 heads, 32k tokens, draft / verify     37.9 / 56.0   33.9 / 51.9
//   one sequence, 8 KV heads of 4, 32k tokens, draft       21.5   20.9
//   one sequence, 8 KV heads of 4, 128k tokens, draft      37.6   54.8 (not taken)
int cluster_size(const Params &prm, qs_mode mode) {
  const long long segs = (long long)prm.c.B * prm.c.H;
  if (prm.c.B > 1 && !prm.sel) return 1;
  int n = 1;
  while (n < kMaxCluster && segs * n * 2 <= prm.P) n *= 2;
  if (n == 1) return 1;
  const long long groups = prm.sel && prm.k_sel < prm.c.cap_groups ? prm.k_sel : prm.c.cap_groups;
  const double units = groups + (mode == QS_DRAFT_UPPER4 ? 8 : 4);  // (and a full buffer)
  const double extra = units / n - units * segs / prm.P;
  const double unit_us = (mode == QS_DRAFT_UPPER4 ? 0.36 : 0.6) * prm.ncg;
  return extra * unit_us < (mode == QS_DRAFT_UPPER4 ? 7.0 : 11.0) ? n : 1;
}

qs_status decode_listed(Params &prm, qs_mode mode, const uint16_t *k_new, const uint16_t *v_new,
                        int32_t n_new, const uint16_t *q, int32_t n_q, int32_t group,
                        float softmax_scale, uint16_t *out, float *lse, void *workspace,
                        size_t workspace_bytes, qs_stream_t stream) {
  if ((k_new != nullptr) != (v_new != nullptr) || n_new < 0 || n_new > kRing ||
      (n_new > 0) != (k_new != nullptr))
    return QS_ERR_ARG;
  if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return QS_ERR_ALIGN;
  prm.wait_ns = kWaitLimitNs;
  prm.k_new = k_new;
  prm.v_new = v_new;
  prm.n_new = n_new;
  const qs_status s = fill_params<kListed>(prm, mode, q, n_q, group, softmax_scale, out, lse,
                                           workspace, workspace_bytes);
  if (s != QS_OK) return s;
  const bool packed = packed_rows(mode, prm.R);
  cudaStream_t st = (cudaStream_t)stream;
  prm.C = cluster_size(prm, mode);
  if (prm.C < 2) return launch_kind<kListed>(mode, packed, prm, st);
  const int grid = prm.c.B * prm.c.H * prm.C;
  const qs_status g = grid_size<kClustered>(mode, packed, prm.c.upper_bits, prm.ncg, prm.P);
  if (g != QS_OK) return g;
  prm.P = grid;
  return launch_kind<kClustered>(mode, packed, prm, st);
}

}  // namespace

extern "C" {

qs_status qs_attn_decode_paged(const qs_cache *c, const qs_pages *pg, qs_mode mode,
                               const uint16_t *k_new, const uint16_t *v_new, int32_t n_new,
                               const uint16_t *q, int32_t n_q, int32_t group, float softmax_scale,
                               uint16_t *out, float *lse, void *workspace, size_t workspace_bytes,
                               qs_stream_t stream) {
  Params prm = {};
  const qs_status s = check_pages(c, pg, true, &prm.c, &prm.pg);
  if (s != QS_OK) return s;
  return decode_listed(prm, mode, k_new, v_new, n_new, q, n_q, group, softmax_scale, out, lse,
                       workspace, workspace_bytes, stream);
}

qs_status qs_attn_decode_sparse(const qs_cache *c, const qs_pages *pg, qs_mode mode,
                                const int32_t *sel, int32_t k_sel, const uint16_t *k_new,
                                const uint16_t *v_new, int32_t n_new, const uint16_t *q, int32_t n_q,
                                int32_t group, float softmax_scale, uint16_t *out, float *lse,
                                void *workspace, size_t workspace_bytes, qs_stream_t stream) {
  Params prm = {};
  const qs_status s = check_pages(c, pg, false, &prm.c, &prm.pg);
  if (s != QS_OK) return s;
  if (!sel || k_sel < 1) return QS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(sel) % 4) return QS_ERR_ALIGN;
  prm.sel = sel;
  prm.k_sel = k_sel;
  return decode_listed(prm, mode, k_new, v_new, n_new, q, n_q, group, softmax_scale, out, lse,
                       workspace, workspace_bytes, stream);
}

}  // extern "C"

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_listed(unsigned long long *out2, int reset) {
  if (cudaMemcpyFromSymbol(out2, g_check_fail, sizeof(g_check_fail)) != cudaSuccess) return 1;
  if (reset) {
    const unsigned long long z[2] = {0, 0};
    if (cudaMemcpyToSymbol(g_check_fail, z, sizeof(z)) != cudaSuccess) return 1;
  }
  return 0;
}
#endif
