// qs_tree.cu -- what a round over a tree of drafted tokens does to the buffer:
// the append with position rotation, and the acceptance of a path.  (The attention
// of the nodes: qs_attn_tree.cu.)
//
// Source: "QuantSpec: Self-Speculative Decoding with Hierarchical Quantized KV
// Cache" (Pith review), "What carries the argument": new tokens enter the double
// full-precision buffer, rejected speculative ones are dropped before
// quantization -- here the ones off the accepted path.
#include "qs_common.cuh"

namespace qs {
namespace {

constexpr int kVec = kD / 8;  // uint4 of eight fp16 per row

// ------------------------------------------------------------------ rotation

constexpr int kRotThreads = 256;
constexpr int kRotTokens = 4;     // tokens per CTA at most
constexpr int kMaxHalf = kD / 2;  // pairs per row at most

struct RotArgs {
  qs_cache c;
  qs_rows k, v, q;
  uint16_t *q_out;
  const int32_t *offset;
  const float *inv_freq;
  int hq, n_new, rot, inter;
  int log_tokens, splits;  // tokens per CTA, as a power of 2; CTAs that share a tile's rows
};

// p * inv_freq in turns without loss: a turn is 2^64, so the product by the
// (signed) position wraps by itself.  inv_freq / 2 pi carries the 53 bits of a
// double: 2^-23 turns at the last position of 32 bits, 2^-38 at 65k.
__device__ __forceinline__ unsigned long long turns(float inv_freq) {
  const double t = (double)inv_freq * 0.15915494309189533577;
  return (unsigned long long)((t - floor(t)) * 18446744073709551616.0);
}

// Four neighbouring pairs (x, y) of a vector, a pair a word: x cos - y sin, y cos + x sin.
__device__ __forceinline__ void turn_neighbours(uint4 &a, const float2 *cs) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(u32_as_h2(x[i])), t = cs[i];
    x[i] = pack_half2(v.x * t.x - v.y * t.y, v.y * t.x + v.x * t.y);
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
}
// Eight pairs whose halves lie in two vectors.
__device__ __forceinline__ void turn_halves(uint4 &a, uint4 &b, const float2 *cs) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = __half22float2(u32_as_h2(x[i])), v = __half22float2(u32_as_h2(y[i]));
    const float2 t0 = cs[2 * i], t1 = cs[2 * i + 1];
    x[i] = pack_half2(u.x * t0.x - v.x * t0.y, u.y * t1.x - v.y * t1.y);
    y[i] = pack_half2(v.x * t0.x + u.x * t0.y, v.y * t1.x + u.y * t1.y);
  }
  a = make_uint4(x[0], x[1], x[2], x[3]);
  b = make_uint4(y[0], y[1], y[2], y[3]);
}

// CTA (tile, split, sequence): 1 << a.log_tokens tokens of the sequence, and every
// splits-th part of their H + H + hq rows (keys, values, queries).  An item is two
// 16-byte vectors of a row, eight items a row, whose lanes' vectors lie side by side:
// a pair of vectors that turn together, or two on their own.  The CTA's angles go
// through shared memory, so their sines are formed once for all heads.
// Bound by memory, for few tokens by a launch and its chain of reads.  Two items a
// thread in flight and five CTAs an SM, against four items and three: eight trees of 64
// tokens 7.0 us (9.0), sixteen sequences of 256 35.6 (36.6; 201 MB, 0.83 of the copy
// bandwidth).  Rows split over two or three CTAs more: 39 and 42.
template <bool INTER>
__global__ void __launch_bounds__(kRotThreads, 5) append_rotary_kernel(const RotArgs a) {
  __shared__ float2 s_cs[kRotTokens * kMaxHalf];
  __shared__ unsigned long long s_turns[kMaxHalf];
  const qs_cache &c = a.c;
  const int b = blockIdx.z, j0 = blockIdx.x << a.log_tokens, nt = min(1 << a.log_tokens, a.n_new - j0);
  const int half = a.rot / 2;
  pdl_trigger();
  pdl_wait();
  int32_t *st = c.state + (size_t)b * QS_STATE_WORDS;
  const int ng = st[QS_ST_N_GROUPS], fill = st[QS_ST_FILL], pending = st[QS_ST_PENDING];
  const int base = st[QS_ST_HALF_BASE] & 1;
  if (threadIdx.x < half) s_turns[threadIdx.x] = turns(a.inv_freq[threadIdx.x]);
  const bool room = fill >= 0 && fill + a.n_new <= kRing;
  __syncthreads();
  for (int i = threadIdx.x; i < nt * kMaxHalf; i += kRotThreads) {
    const int j = i / kMaxHalf, f = i % kMaxHalf;
    if (f >= half) continue;
    const int pos = ng * kG + fill + (a.offset ? a.offset[(size_t)b * a.n_new + j0 + j] - pending : j0 + j);
    // the signed fraction of a turn, in half turns
    const long long p = (long long)((unsigned long long)(long long)pos * s_turns[f]);
    float2 cs;
    sincospif((float)(int)(p >> 32) * 4.656612873077393e-10f, &cs.y, &cs.x);
    if (chk(i < kRotTokens * kMaxHalf && f < kMaxHalf, 80)) s_cs[i] = cs;
  }
  __syncthreads();
  const int rows = 2 * c.H + a.hq, per = (rows + a.splits - 1) / a.splits;
  const int r0 = blockIdx.y * per, r1 = min(rows, r0 + per);
  const int n_items = (r1 - r0) << (a.log_tokens + 3);
  const int turning = INTER ? 0 : a.rot / 16;  // items of a row whose vectors turn together
  constexpr int U = 2;  // items in flight per thread
#pragma unroll 1
  for (int e0 = threadIdx.x; e0 < n_items; e0 += U * kRotThreads) {
    uint4 x[U], y[U];
    uint4 *dst[U];
    const int i = e0 & 7;  // (the same for all U)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * kRotThreads;
      const int j = (e >> 3) & ((1 << a.log_tokens) - 1), row = r0 + (e >> (a.log_tokens + 3));
      dst[u] = nullptr;
      if (e >= n_items || j >= nt) continue;
      const bool is_q = row >= 2 * c.H, is_v = !is_q && row >= c.H;
      const int h = is_q ? row - 2 * c.H : is_v ? row - c.H : row;
      const qs_rows &s = is_q ? a.q : is_v ? a.v : a.k;
      const bool together = !is_v && i < turning;
      const int vx = is_v || together ? i : i + turning, vy = together ? i + turning : i + 8;
      const uint4 *src = reinterpret_cast<const uint4 *>(s.data + b * s.stride_b + h * s.stride_h +
                                                         (j0 + j) * s.stride_t);
      x[u] = src[vx];
      y[u] = src[vy];
      if (!chk(b < c.B && h >= 0 && h < (is_q ? a.hq : c.H) && j0 + j < a.n_new && vx < kVec && vy < kVec, 81)) continue;
      if (is_q) {
        const size_t at = ((size_t)b * a.hq + h) * a.n_new + j0 + j;
        if (chk(in_range(at, 1, (size_t)c.B * a.hq * a.n_new), 82)) dst[u] = reinterpret_cast<uint4 *>(a.q_out) + at * kVec;
      } else if (room) {
        const int slot = (base * kG + fill + j0 + j) & (kRing - 1);
        const size_t at = ((size_t)b * c.H + h) * kRing + slot;
        if (chk(in_range(at, 1, (size_t)c.B * c.H * kRing), 83))
          dst[u] = reinterpret_cast<uint4 *>(is_v ? c.buf_v : c.buf_k) + at * kVec;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!dst[u]) continue;
      const int e = e0 + u * kRotThreads;
      const int j = (e >> 3) & ((1 << a.log_tokens) - 1), row = r0 + (e >> (a.log_tokens + 3));
      const bool is_v = row >= c.H && row < 2 * c.H, together = !is_v && i < turning;
      const float2 *cs = s_cs + j * kMaxHalf;
      if (INTER) {
        if (!is_v && 8 * i < a.rot) turn_neighbours(x[u], cs + 4 * i);
        if (!is_v && 8 * i + 64 < a.rot) turn_neighbours(y[u], cs + 4 * i + 32);
      } else if (together) {
        turn_halves(x[u], y[u], cs + 8 * i);
      }
      dst[u][is_v || together ? i : i + turning] = x[u];
      dst[u][together ? i + turning : i + 8] = y[u];
    }
  }
  if (!room) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(&st[QS_ST_ERR], QS_DEV_OVERFLOW);
    return;
  }
  __syncthreads();
  // every CTA of the sequence has read the old counters once the last one arrives
  if (threadIdx.x == 0 &&
      atom_add_acq_rel_gpu(&st[QS_ST_TICKET], 1) == (int)(gridDim.x * gridDim.y) - 1) {
    st[QS_ST_FILL] = fill + a.n_new;
    st[QS_ST_PENDING] = pending + a.n_new;
    st[QS_ST_TICKET] = 0;
  }
}

// ---------------------------------------------------------------- acceptance

constexpr int kAccThreads = 256;

// One CTA per (head, sequence).  Its first warp walks the tree, two nodes a lane:
// a step is a shuffle (the target's token of the current node) and two votes (the
// nodes that hang from it with that token).  Then the CTA reads the rows of the
// path that have to move, all before the first is written: they only move
// forward, so one may lie where an earlier one goes.  Bound by its chain of reads
// (counters, tree, rows): with a copy of the counters and an append in front 5.9 us for
// a tree of 16 nodes of 8 heads, 10 for sixteen of 64 of 32 heads.
__global__ void __launch_bounds__(kAccThreads)
    tree_accept_kernel(qs_cache c, const int32_t *parent, const int32_t *draft, const int32_t *target,
                       int n, int32_t *n_keep, int32_t *path, int32_t *emitted) {
  __shared__ int s_path[QS_MAX_TREE], s_keep, s_fill, s_base;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  int32_t *st = c.state + (size_t)b * QS_STATE_WORDS;
  if (tid < 32) {
    const int fill = st[QS_ST_FILL], pending = st[QS_ST_PENDING], base = st[QS_ST_HALF_BASE] & 1;
    int up[2], tok[2], tgt[2];
    bool bad = fill > kRing || pending > fill || n > pending;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int j = tid + 32 * k;
      const size_t at = (size_t)b * n + j;
      up[k] = tok[k] = tgt[k] = -1;
      if (j < n && chk(in_range(at, 1, (size_t)c.B * n), 84)) {
        up[k] = parent[at];
        tok[k] = draft[at];
        tgt[k] = target[at];
        bad |= up[k] < -1 || up[k] >= j;
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    int keep = 0;
    int mine[2] = {-1, -1}, out[2] = {-1, -1};  // entries tid and tid + 32 of path and emitted
    if (!bad) {
      int at = 0;
      for (; keep < n;) {
        const int a0 = __shfl_sync(0xffffffffu, tgt[0], at & 31), a1 = __shfl_sync(0xffffffffu, tgt[1], at & 31);
        const int t = at < 32 ? a0 : a1;
        if (tid == (keep & 31)) {
          mine[keep >> 5] = at;
          out[keep >> 5] = t;
        }
        ++keep;
        const unsigned m0 = __ballot_sync(0xffffffffu, up[0] == at && tok[0] == t && tok[0] >= 0);
        const unsigned m1 = __ballot_sync(0xffffffffu, up[1] == at && tok[1] == t && tok[1] >= 0);
        if (!(m0 | m1)) break;
        at = m0 ? __ffs(m0) - 1 : 31 + __ffs(m1);
      }
    }
    s_path[tid] = mine[0];
    s_path[tid + 32] = mine[1];
    if (tid == 0) {
      s_keep = keep;
      s_fill = fill;
      s_base = base;
    }
    if (h == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (tid + 32 * k < n && chk(in_range((size_t)b * n + tid + 32 * k, 1, (size_t)c.B * n), 84)) {
          path[(size_t)b * n + tid + 32 * k] = mine[k];
          emitted[(size_t)b * n + tid + 32 * k] = out[k];
        }
      if (tid == 0) {
        n_keep[b] = keep;
        if (bad) atomicOr(&st[QS_ST_ERR], QS_DEV_TREE);
      }
    }
  }
  __syncthreads();
  const int keep = s_keep;
  if (keep == 0) return;
  const int first = s_base * kG + s_fill - n;
  const size_t row0 = ((size_t)b * c.H + h) * kRing;
  uint4 *bk = reinterpret_cast<uint4 *>(c.buf_k) + row0 * kVec, *bv = reinterpret_cast<uint4 *>(c.buf_v) + row0 * kVec;
  constexpr int U = QS_MAX_TREE * kVec / kAccThreads;
  uint4 xk[U], xv[U];
  const int col = tid % kVec;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = tid / kVec + u * (kAccThreads / kVec);
    if (i < keep && s_path[i] != i) {
      if (!chk(i < QS_MAX_TREE && s_path[i] >= 0 && s_path[i] < n && in_range(row0, kRing, (size_t)c.B * c.H * kRing), 85))
        continue;
      const int src = (first + s_path[i]) & (kRing - 1);
      xk[u] = bk[src * kVec + col];
      xv[u] = bv[src * kVec + col];
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = tid / kVec + u * (kAccThreads / kVec);
    if (i < keep && s_path[i] != i) {
      const int dst = (first + i) & (kRing - 1);
      bk[dst * kVec + col] = xk[u];
      bv[dst * kVec + col] = xv[u];
    }
  }
  // every head has read the old counters once the ticket reaches H - 1
  if (tid == 0 && atom_add_acq_rel_gpu(&st[QS_ST_TICKET], 1) == c.H - 1) {
    st[QS_ST_FILL] = s_fill - n + keep;
    st[QS_ST_PENDING] = 0;
    st[QS_ST_TICKET] = 0;
  }
}

qs_status check_rows(const qs_rows *r) {
  if (!r->data) return QS_ERR_ARG;
  if (r->stride_b % 8 || r->stride_h % 8 || r->stride_t % 8) return QS_ERR_SHAPE;
  return aligned16(r->data) ? QS_OK : QS_ERR_ALIGN;
}

// [p, p + bytes) shares memory with what lies between the first and the last of B x heads
// x n rows.
bool over_rows(const void *p, size_t bytes, const qs_rows &r, int B, int heads, int n) {
  const int64_t ends[] = {(B - 1) * r.stride_b, (heads - 1) * r.stride_h, (n - 1) * r.stride_t};
  int64_t lo = 0, hi = kD;
  for (const int64_t e : ends) (e < 0 ? lo : hi) += e;
  return overlap(p, bytes, r.data + lo, (size_t)(hi - lo) * sizeof(uint16_t));
}

// The rows lie as a contiguous [B][heads][n][D] does.
bool contiguous_rows(const qs_rows &r, int B, int heads, int n) {
  return (n == 1 || r.stride_t == kD) && (heads == 1 || r.stride_h == (int64_t)n * kD) &&
         (B == 1 || r.stride_b == (int64_t)heads * n * kD);
}

}  // namespace
}  // namespace qs

using namespace qs;

extern "C" {

qs_status qs_buffer_append_rotary(const qs_cache *c, const qs_rows *k, const qs_rows *v,
                                  const qs_rows *q, uint16_t *q_out, int32_t group, int32_t n_new,
                                  const int32_t *offset, const float *inv_freq, int32_t rot,
                                  int32_t interleaved, qs_stream_t stream) {
  qs_status s = check_cache_any(c);
  if (s != QS_OK) return s;
  if (!k || !v || !inv_freq || (q != nullptr) != (q_out != nullptr)) return QS_ERR_ARG;
  if (n_new < 1 || n_new > kRing || (q && (group < 1 || group > 1024))) return QS_ERR_ARG;
  if (rot < 16 || rot > kD || rot % 16) return QS_ERR_ARG;
  const qs_rows none = {nullptr, 0, 0, 0};
  const qs_rows *rows[] = {k, v, q};
  for (const qs_rows *r : rows)
    if (r && (s = check_rows(r)) != QS_OK) return s;
  if (!aligned16(q_out) || reinterpret_cast<uintptr_t>(inv_freq) % 4 ||
      reinterpret_cast<uintptr_t>(offset) % 4)
    return QS_ERR_ALIGN;
  RotArgs a = {*c, *k, *v, q ? *q : none, q_out, offset, inv_freq, q ? c->H * group : 0, n_new, rot,
               interleaved != 0, 0, 1};
  if (q) {  // (a row is written when others may still be read)
    const size_t bytes = sizeof(uint16_t) * kD * c->B * a.hq * n_new;
    const bool in_place = q_out == q->data && contiguous_rows(*q, c->B, a.hq, n_new);
    if ((!in_place && over_rows(q_out, bytes, *q, c->B, a.hq, n_new)) ||
        over_rows(q_out, bytes, *k, c->B, c->H, n_new) || over_rows(q_out, bytes, *v, c->B, c->H, n_new))
      return QS_ERR_ARG;
  }
  const long long n_rows = 2ll * c->H + a.hq;
  int sms = 0;
  if ((s = sm_count(&sms)) != QS_OK) return s;
  // four tokens to a CTA, fewer where that leaves SMs without one; then their rows over
  // several CTAs, 32 items (of 8 lanes) each at least
  a.log_tokens = 2;
  const auto tiles = [&] { return (long long)((n_new + (1 << a.log_tokens) - 1) >> a.log_tokens) * c->B; };
  while (a.log_tokens > 0 && tiles() < sms) --a.log_tokens;
  long long split = (2ll * sms + tiles() - 1) / tiles(), most = ((n_rows << a.log_tokens) + 31) / 32;
  if (split > most) split = most;
  a.splits = (int)(split < 1 ? 1 : split > 65535 ? 65535 : split);
  const dim3 grid((n_new + (1 << a.log_tokens) - 1) >> a.log_tokens, a.splits, c->B);
  return launch_pdl(a.inter ? append_rotary_kernel<true> : append_rotary_kernel<false>, grid,
                    dim3(kRotThreads), 0, (cudaStream_t)stream, a);
}

qs_status qs_tree_accept(const qs_cache *c, const int32_t *parent, const int32_t *draft,
                         const int32_t *target, int32_t n_tree, int32_t *n_keep, int32_t *path,
                         int32_t *emitted, qs_stream_t stream) {
  const qs_status s = check_cache_any(c);
  if (s != QS_OK) return s;
  if (!parent || !draft || !target || !n_keep || !path || !emitted) return QS_ERR_ARG;
  if (n_tree < 1 || n_tree > QS_MAX_TREE) return QS_ERR_ARG;
  const void *ptrs[] = {parent, draft, target, n_keep, path, emitted};
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % 4) return QS_ERR_ALIGN;
  // every head's CTA walks the tree, while one of them already writes the outputs
  const size_t nodes = sizeof(int32_t) * c->B * n_tree, sizes[] = {nodes, nodes, nodes, sizeof(int32_t) * c->B, nodes, nodes};
  for (int out = 3; out < 6; ++out)
    for (int i = 0; i < out; ++i)
      if (overlap(ptrs[out], sizes[out], ptrs[i], sizes[i])) return QS_ERR_ARG;
  return launch_pdl(tree_accept_kernel, dim3(c->H, c->B), dim3(kAccThreads), 0, (cudaStream_t)stream,
                    *c, parent, draft, target, (int)n_tree, n_keep, path, emitted);
}

}  // extern "C"

#if QS_CHECKED
// Checked build only: this file's failure count and first failing tag.
extern "C" int qs_checked_failures_buffer_tree(unsigned long long *out2, int reset) {
  return read_check_failures(out2, reset);
}
#endif
