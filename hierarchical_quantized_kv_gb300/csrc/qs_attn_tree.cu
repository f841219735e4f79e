// qs_attn_tree.cu -- decode attention of the nodes of a tree of drafted tokens.
// Few rows per KV head run through the split kernel (qs_split.cuh) in its tree
// variants, more of them through the tensor cores 128 at a time (qs_tall.cuh).
#include "qs_tall.cuh"

using namespace qs;

namespace qs {
namespace {

bool tree_sizes_ok(int32_t n_q, int32_t group) {
  return n_q >= 1 && n_q <= QS_MAX_TREE && group >= 1 && group <= kMaxTreeRows && group * n_q <= kMaxTreeRows;
}

// Rows that the split kernel takes: its work grows with each eight of them, the other
// kernel's does not, and a draft's halves it there only.  Split / tall, us, for 32 heads
// of 32k tokens, 8 heads of 32k, 8 heads of 4k, 4 x 32 heads of 32k:
//   verify, 16 rows   87 / 114   34 / 41   15 / 19   280 / 409
//   verify, 17 rows  131 / 115   45 / 42   20 / 20   454 / 411
//   draft,  24 rows  100 / 115   35 / 42   18 / 20   334 / 408
// (24 is also the most that the split kernel's layout holds.)
constexpr int split_rows(qs_mode mode) { return mode == QS_VERIFY_INT8 ? 16 : kMaxR; }
static_assert(split_rows(QS_VERIFY_INT8) <= 16, "wide_verify leaves out the variants for more");

qs_status decode_tall(const Params &a, qs_mode mode, void *workspace, size_t workspace_bytes,
                      cudaStream_t st) {
  TallParams prm = {};
  prm.c = a.c;
  prm.pg = a.pg;
  prm.q = a.q;
  prm.out = a.out;
  prm.lse = a.lse;
  prm.ws = static_cast<float *>(workspace);
  prm.parent = a.parent;
  prm.n_tree = a.n_tree;
  prm.n_q = a.n_q;
  prm.R = a.R;
  prm.n_mp = (a.R + 2 * kTile - 1) / (2 * kTile);
  prm.rows = tall_rows(a.R);
  prm.sl2 = a.sl2;
  prm.wait_ns = a.wait_ns;
  prm.no_issue = a.no_issue;
  prm.ws_floats = workspace_bytes / sizeof(float);
  const qs_status s = sm_count(&prm.P);
  if (s != QS_OK) return s;
  if (!workspace || !aligned16(workspace) || workspace_bytes < tall_ws_bytes(prm.P, a.c.B, a.c.H, a.R))
    return QS_ERR_WORKSPACE;
  return mode == QS_VERIFY_INT8 ? launch_tall_mode<QS_VERIFY_INT8>(prm, st)
                                : launch_tall_mode<QS_DRAFT_UPPER4>(prm, st);
}

qs_status decode_tree(const qs_cache *c, const qs_pages *pg, qs_mode mode, const int32_t *parent,
                      int32_t n_tree, const uint16_t *q, int32_t n_q, int32_t group,
                      float softmax_scale, uint16_t *out, float *lse, void *workspace,
                      size_t workspace_bytes, uint64_t wait_ns, int no_issue, qs_stream_t stream) {
  Params prm = {};
  qs_status s = check_pages(c, pg, false, &prm.c, &prm.pg);
  if (s != QS_OK) return s;
  if (!parent || !tree_sizes_ok(n_q, group) || n_tree < n_q || n_tree > QS_MAX_TREE) return QS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(parent) % 4) return QS_ERR_ALIGN;
  prm.parent = parent;
  prm.n_tree = n_tree;
  prm.wait_ns = wait_ns;
  prm.no_issue = no_issue;
  cudaStream_t st = (cudaStream_t)stream;
  if (group * n_q > split_rows(mode)) {
    s = check_queries(mode, q, softmax_scale, out, lse);
    if (s != QS_OK) return s;
    set_queries(prm, q, n_q, group, softmax_scale, out, lse);
    return decode_tall(prm, mode, workspace, workspace_bytes, st);
  }
  s = fill_params<kListed | kTree>(prm, mode, q, n_q, group, softmax_scale, out, lse, workspace,
                                   workspace_bytes);
  if (s != QS_OK) return s;
  if ((s = choose_clusters<kTree>(prm, mode)) != QS_OK) return s;
  const bool packed = packed_rows(mode, prm.R);
  if (prm.C < 2) return launch_kind<kListed | kTree>(mode, packed, prm, st);
  prm.P = prm.c.B * prm.c.H * prm.K * prm.C;
  return launch_kind<kClustered | kTree>(mode, packed, prm, st);
}

}  // namespace
}  // namespace qs

extern "C" {

qs_status qs_attn_tree_workspace_size(const qs_cache *c, int32_t n_q, int32_t group, size_t *bytes) {
  qs_status s = check_cache_any(c);
  if (s != QS_OK) return s;
  if (!bytes || !tree_sizes_ok(n_q, group)) return QS_ERR_ARG;
  const int bits = c->upper_bits & ~QS_PAGED, R = group * n_q;
  // for either mode, and for every call of fewer rows (a level of the tree, say): few rows
  // may take the split kernel, whose CTAs leave more partials than the other one's
  *bytes = 0;
  if (R > split_rows(QS_VERIFY_INT8)) {
    int sms = 0;
    if ((s = sm_count(&sms)) != QS_OK) return s;
    *bytes = tall_ws_bytes(sms, c->B, c->H, R);
  }
  for (const qs_mode mode : {QS_DRAFT_UPPER4, QS_VERIFY_INT8})
    for (int r = 1; r <= R && r <= split_rows(mode); ++r) {
      int P = 0;
      if ((s = grid_size<kListed | kTree>(mode, packed_rows(mode, r), bits, (r + 7) / 8, P)) != QS_OK) return s;
      const size_t split = ws_bytes(P, c->B, c->H, r);
      if (split > *bytes) *bytes = split;
    }
  return QS_OK;
}

qs_status qs_attn_decode_tree(const qs_cache *c, const qs_pages *pg, qs_mode mode,
                              const int32_t *parent, int32_t n_tree, const uint16_t *q, int32_t n_q,
                              int32_t group, float softmax_scale, uint16_t *out, float *lse,
                              void *workspace, size_t workspace_bytes, qs_stream_t stream) {
  return decode_tree(c, pg, mode, parent, n_tree, q, n_q, group, softmax_scale, out, lse, workspace,
                     workspace_bytes, kWaitLimitNs, 0, stream);
}

// Test entry, not declared in include/qs.h: qs_attn_decode_tree with every pipeline
// wait limited to wait_ns (1 us .. 100 ms) and no copy ever issued, so that the waits
// for the first group run out (as qs_test_attn_decode_timeout does).
qs_status qs_test_attn_tree_timeout(const qs_cache *c, const qs_pages *pg, qs_mode mode,
                                    const int32_t *parent, int32_t n_tree, const uint16_t *q, int32_t n_q,
                                    int32_t group, float softmax_scale, uint16_t *out, float *lse,
                                    void *workspace, size_t workspace_bytes, uint64_t wait_ns,
                                    qs_stream_t stream) {
  if (wait_ns < 1000ull || wait_ns > 100000000ull) return QS_ERR_ARG;
  return decode_tree(c, pg, mode, parent, n_tree, q, n_q, group, softmax_scale, out, lse, workspace,
                     workspace_bytes, wait_ns, 1, stream);
}

}  // extern "C"

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_tree(unsigned long long *out2, int reset) {
  return read_check_failures(out2, reset);
}
#endif
