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
                        size_t workspace_bytes, uint64_t wait_ns, int no_issue,
                        qs_stream_t stream) {
  if ((k_new != nullptr) != (v_new != nullptr) || n_new < 0 || n_new > kRing ||
      (n_new > 0) != (k_new != nullptr))
    return QS_ERR_ARG;
  if (k_new && (!aligned16(k_new) || !aligned16(v_new))) return QS_ERR_ALIGN;
  prm.wait_ns = wait_ns;
  prm.no_issue = no_issue;
  prm.k_new = k_new;
  prm.v_new = v_new;
  prm.n_new = n_new;
  qs_status s = fill_params<kListed>(prm, mode, q, n_q, group, softmax_scale, out, lse,
                                           workspace, workspace_bytes);
  if (s != QS_OK) return s;
  const bool packed = packed_rows(mode, prm.R);
  cudaStream_t st = (cudaStream_t)stream;
  if ((s = choose_clusters<0>(prm, mode)) != QS_OK) return s;
  if (prm.C < 2) return launch_kind<kListed>(mode, packed, prm, st);
  prm.P = prm.c.B * prm.c.H * prm.K * prm.C;
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
                       workspace, workspace_bytes, kWaitLimitNs, 0, stream);
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
                       workspace, workspace_bytes, kWaitLimitNs, 0, stream);
}

// Test entry, not declared in include/qs.h: qs_attn_decode_paged with every
// pipeline wait limited to wait_ns (1 us .. 100 ms) and no copy ever issued, so
// the first wait of every warp runs out (as qs_test_attn_decode_timeout does for
// the contiguous kernel).
qs_status qs_test_attn_paged_timeout(const qs_cache *c, const qs_pages *pg, qs_mode mode,
                                     const uint16_t *q, int32_t n_q, int32_t group,
                                     float softmax_scale, uint16_t *out, float *lse, void *workspace,
                                     size_t workspace_bytes, uint64_t wait_ns, qs_stream_t stream) {
  if (wait_ns < 1000ull || wait_ns > 100000000ull) return QS_ERR_ARG;
  Params prm = {};
  const qs_status s = check_pages(c, pg, true, &prm.c, &prm.pg);
  if (s != QS_OK) return s;
  return decode_listed(prm, mode, nullptr, nullptr, 0, q, n_q, group, softmax_scale, out, lse,
                       workspace, workspace_bytes, wait_ns, 1, stream);
}

}  // extern "C"

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_listed(unsigned long long *out2, int reset) {
  return read_check_failures(out2, reset);
}
#endif
