// qs_attn_list.cu -- entry points of the decode attention over listed groups:
// the groups of a paged cache, and the groups selected for each head (of a
// contiguous or a paged cache).  The kernel is the contiguous one's
// (qs_split.cuh) in its listed variants: a segment's units are entries of a
// list, looked up at kernel start beside the first copies, so the stream of
// bulk copies and everything after it stay the same.
#include "qs_split.cuh"

using namespace qs;

namespace {

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
  return decode<true>(prm, mode, q, n_q, group, softmax_scale, out, lse, workspace, workspace_bytes,
                      stream);
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
