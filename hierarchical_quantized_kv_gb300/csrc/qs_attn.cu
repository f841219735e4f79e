// qs_attn.cu -- entry points of the decode attention over a contiguous cache
// (the kernel: qs_split.cuh).
#include "qs_split.cuh"

using namespace qs;

extern "C" {

qs_status qs_attn_workspace_size_gqa(const qs_cache *c, int32_t n_q, int32_t group,
                                     size_t *bytes) {
  qs_status s = check_cache_any(c);
  if (s != QS_OK) return s;
  const int bits = c->upper_bits & ~QS_PAGED;
  if (!bytes || n_q < 1 || n_q > kMaxQ || group < 1 || group * n_q > kMaxR) return QS_ERR_ARG;
  int P0 = 0, P1 = 0, P2 = 0;
  if ((s = grid_size<kContiguous>(QS_DRAFT_UPPER4, false, bits, 1, P0)) != QS_OK) return s;
  if ((s = grid_size<kContiguous>(QS_DRAFT_UPPER4, true, bits, 1, P1)) != QS_OK) return s;
  if ((s = grid_size<kContiguous>(QS_VERIFY_INT8, false, bits, (group * n_q + 7) / 8, P2)) != QS_OK) return s;
  const int P = P0 > P1 ? (P0 > P2 ? P0 : P2) : (P1 > P2 ? P1 : P2);
  *bytes = ws_bytes(P, c->B, c->H, group * n_q);
  return QS_OK;
}

qs_status qs_attn_workspace_size(const qs_cache *c, int32_t n_q, size_t *bytes) {
  return qs_attn_workspace_size_gqa(c, n_q, 1, bytes);
}

}  // extern "C"

namespace {

qs_status decode_contiguous(const qs_cache *c, qs_mode mode, const uint16_t *q, int32_t n_q,
                            int32_t group, float softmax_scale, uint16_t *out, float *lse,
                            void *workspace, size_t workspace_bytes, uint64_t wait_ns, int no_issue,
                            const uint16_t *k_new, const uint16_t *v_new, int32_t n_new,
                            qs_stream_t stream) {
  const qs_status s = check_cache(c);
  if (s != QS_OK) return s;
  Params prm = {};
  prm.c = *c;
  prm.wait_ns = wait_ns;
  prm.no_issue = no_issue;
  prm.k_new = k_new;
  prm.v_new = v_new;
  prm.n_new = n_new;
  const qs_status f = fill_params<kContiguous>(prm, mode, q, n_q, group, softmax_scale, out, lse,
                                               workspace, workspace_bytes);
  if (f != QS_OK) return f;
  return launch_kind<kContiguous>(mode, packed_rows(mode, prm.R), prm, (cudaStream_t)stream);
}

}  // namespace

extern "C" {

qs_status qs_attn_decode_gqa(const qs_cache *c, qs_mode mode, const uint16_t *q, int32_t n_q,
                             int32_t group, float softmax_scale, uint16_t *out, float *lse,
                             void *workspace, size_t workspace_bytes, qs_stream_t stream) {
  return decode_contiguous(c, mode, q, n_q, group, softmax_scale, out, lse, workspace, workspace_bytes,
                kWaitLimitNs, 0, nullptr, nullptr, 0, stream);
}

qs_status qs_attn_decode_append(const qs_cache *c, qs_mode mode, const uint16_t *k_new,
                                const uint16_t *v_new, int32_t n_new, const uint16_t *q,
                                int32_t n_q, int32_t group, float softmax_scale, uint16_t *out,
                                float *lse, void *workspace, size_t workspace_bytes,
                                qs_stream_t stream) {
  if (!k_new || !v_new || n_new < 1 || n_new > kRing) return QS_ERR_ARG;
  if (!aligned16(k_new) || !aligned16(v_new)) return QS_ERR_ALIGN;
  return decode_contiguous(c, mode, q, n_q, group, softmax_scale, out, lse, workspace, workspace_bytes,
                kWaitLimitNs, 0, k_new, v_new, n_new, stream);
}

qs_status qs_attn_decode(const qs_cache *c, qs_mode mode, const uint16_t *q, int32_t n_q,
                         float softmax_scale, uint16_t *out, float *lse, void *workspace,
                         size_t workspace_bytes, qs_stream_t stream) {
  return qs_attn_decode_gqa(c, mode, q, n_q, 1, softmax_scale, out, lse, workspace,
                            workspace_bytes, stream);
}

// Test entry, not declared in include/qs.h: qs_attn_decode_gqa with every
// pipeline wait limited to wait_ns (1 us .. 100 ms) and no copy ever issued,
// so the first wait of every warp runs out.  It exercises the failure path
// of the kernel without a fault: the sequences get QS_DEV_TIMEOUT, the
// kernel returns within a few multiples of wait_ns, no output is written, and
// the arrival counters end at zero, so the next ordinary call on the cache is
// valid.
qs_status qs_test_attn_decode_timeout(const qs_cache *c, qs_mode mode, const uint16_t *q,
                                      int32_t n_q, int32_t group, float softmax_scale,
                                      uint16_t *out, float *lse, void *workspace,
                                      size_t workspace_bytes, uint64_t wait_ns,
                                      qs_stream_t stream) {
  if (wait_ns < 1000ull || wait_ns > 100000000ull) return QS_ERR_ARG;
  return decode_contiguous(c, mode, q, n_q, group, softmax_scale, out, lse, workspace, workspace_bytes,
                wait_ns, 1, nullptr, nullptr, 0, stream);
}

}  // extern "C"

#if QS_CHECKED
extern "C" int qs_checked_failures_quantize(unsigned long long *out2, int reset);
extern "C" int qs_checked_failures_listed(unsigned long long *out2, int reset);
extern "C" int qs_checked_failures_select(unsigned long long *out2, int reset);
extern "C" int qs_checked_failures_read(unsigned long long *out2, int reset);

// Checked build only (-DQS_CHECKED=1): the number of failed bounds checks of
// the kernels since the last reset, and the tag of the first (attention: 1
// shared-memory load, 2 copy destination, 3 group index, 4 buffer row, 6 ldmatrix
// row, 7 partial slot, 8 merge source, 9 query row, 10 output head, 11 tail
// partials; quantizer: 20 flush group, 21 metadata position, 22 prefill group
// rows, 23 prefill buffer rows; listed attention: 30 page table entry, 31 entry of
// the selection, 32 place of a unit, 33 a cluster's sums in shared memory, 34 its
// sums in the workspace; selection: 40 score, 41 list of close groups, 42 output,
// 43 scales and zeros, 44 query row; read back: 50 group, 51 buffer row, 52 output
// row, 53 tile row).  reset != 0 zeroes the counts.  Returns 0, or 1 if a CUDA call
// failed.
extern "C" int qs_checked_failures(unsigned long long *count, unsigned int *first_tag, int reset) {
  unsigned long long f[5][2];
  if (read_check_failures(f[0], reset) || qs_checked_failures_quantize(f[1], reset) ||
      qs_checked_failures_listed(f[2], reset) || qs_checked_failures_select(f[3], reset) ||
      qs_checked_failures_read(f[4], reset))
    return 1;
  *count = 0;
  *first_tag = 0;
  for (const auto &x : f) {
    if (*count == 0 && x[0]) *first_tag = (unsigned int)x[1];
    *count += x[0];
  }
  return 0;
}
#endif
