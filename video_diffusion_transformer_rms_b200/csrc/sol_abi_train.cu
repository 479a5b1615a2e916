// C ABI of the training operators (declared in include/sol.h): host-side
// argument checks, then the launches on the caller's stream.  Nothing is
// allocated on the device and nothing is synchronised.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <utility>

#include "sol.h"
#include "sol_check.h"
#include "sol_launch.h"
#include "sol_train.h"

namespace sol {
namespace {

constexpr int64_t kMaxSamples = int64_t(1) << 30;  // 2 * sample + modality is 32-bit

// No exception crosses the C boundary.
template <typename F>
sol_status guarded(F &&body) {
  try {
    return body();
  } catch (...) {
    return SOL_ERR_CUDA;  // the host ran out of memory
  }
}

int dtype_index(sol_dtype dt) { return dt == SOL_F32 ? 0 : 1; }

// An array of a call.
struct Arr {
  const char *name;
  const void *p;
  int64_t bytes;
};
// An output and an input that it may equal exactly.
struct Alias {
  const void *out;
  const void *in;
};
// Every output overlaps no other argument, except those in `equal`.
sol_status check_overlaps(const char *fn, std::initializer_list<Arr> ins,
                          std::initializer_list<Arr> outs, std::initializer_list<Alias> equal) {
  auto may = [&](const void *o, const void *i) {
    for (const Alias &e : equal)
      if (e.out == o && e.in == i && o == i) return true;
    return false;
  };
  for (const Arr &o : outs) {
    if (!o.p || o.bytes == 0) continue;
    const Span so = span_of(o.p, 1, 0, o.bytes);
    for (const Arr &i : ins) {
      if (!i.p || i.bytes == 0 || (i.bytes == o.bytes && may(o.p, i.p))) continue;
      if (spans_overlap(so, span_of(i.p, 1, 0, i.bytes)))
        return fail(SOL_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, o.name, i.name);
    }
    for (const Arr &q : outs) {
      if (&q == &o || !q.p || q.bytes == 0) continue;
      if (spans_overlap(so, span_of(q.p, 1, 0, q.bytes)))
        return fail(SOL_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, o.name, q.name);
    }
  }
  return SOL_OK;
}

// dtype, B, L, n_video and D of the row operators.
sol_status check_rows(const char *fn, int64_t B, int64_t L, int64_t n_video, int64_t D,
                      sol_dtype dtype) {
  if (dtype != SOL_F32 && dtype != SOL_BF16)
    return fail(SOL_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
  if (B < 0 || L < 0 || D <= 0 || n_video < 0 || n_video > L)
    return fail(SOL_ERR_INVALID_ARG, "%s: need B, L >= 0, D > 0 and 0 <= n_video <= L", fn);
  if (B > kMaxRows || L > kMaxRows || B * L > kMaxRows)
    return fail(SOL_ERR_UNSUPPORTED, "%s: B*L must be below 2^31 rows", fn);
  if (B >= kMaxSamples)
    return fail(SOL_ERR_UNSUPPORTED, "%s: B must be below 2^30 samples", fn);
  const int es = esize_of(dtype);
  if (D > kMaxRowBytesRms / es)
    return fail(SOL_ERR_UNSUPPORTED, "%s: D=%lld exceeds %lld elements", fn, (long long)D,
                (long long)(kMaxRowBytesRms / es));
  if (D * es % 16 != 0)
    return fail(SOL_ERR_MISALIGNED, "%s: D*%d bytes must be a multiple of 16 (D=%lld)", fn, es,
                (long long)D);
  return SOL_OK;
}

sol_status check_aligned(const char *fn, std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (!aligned16(p))
      return fail(SOL_ERR_MISALIGNED, "%s: pointers must be 16-byte aligned", fn);
  return SOL_OK;
}

sol_status check_workspace(const char *fn, const void *ws, size_t bytes, size_t need) {
  if (!ws) return fail(SOL_ERR_INVALID_ARG, "%s: workspace must be non-null", fn);
  if (bytes < need)
    return fail(SOL_ERR_INVALID_ARG, "%s: workspace has %zu bytes, needs %zu", fn, bytes, need);
  return check_aligned(fn, {ws});
}

bool sizes_ok(int64_t B, int64_t L, int64_t D) {
  return B >= 0 && L >= 0 && D > 0 && B <= kMaxRows && L <= kMaxRows && B * L <= kMaxRows &&
         D <= kMaxRowBytesRms / 2;
}

Segments segments(int64_t B, int64_t L, int64_t n_video, bool keyed) {
  Segments s{};
  s.rows = B * L;
  s.keys = keyed ? static_cast<int>(2 * B) : 1;
  s.L = static_cast<int>(keyed ? L : s.rows);
  s.n_video = static_cast<int>(keyed ? n_video : s.rows);
  return s;
}

sol_status norm_backward(const char *fn, bool rms, const void *dy, const void *x,
                         const float *mean, const float *rstd, const void *gamma,
                         const void *beta, const void *scale, const void *dres, void *dx,
                         float *dgamma, float *dbeta, float *dscale, float *dshift, int64_t B,
                         int64_t L, int64_t n_video, int64_t D, float eps, void *workspace,
                         size_t workspace_bytes, sol_dtype dtype, sol_stream_t stream) {
  sol_status st = check_rows(fn, B, L, n_video, D, dtype);
  if (st != SOL_OK) return st;
  if (rms && !(eps >= 0.f)) return fail(SOL_ERR_INVALID_ARG, "%s: need eps >= 0", fn);
  if (!scale && (dscale || dshift))
    return fail(SOL_ERR_INVALID_ARG, "%s: dscale and dshift need scale", fn);
  const int64_t rows = B * L;
  const bool sums = dgamma || dbeta || dscale || dshift;
  if (rows > 0 && (!dy || !x || !dx || (rms ? !scale : (!mean || !rstd))))
    return fail(SOL_ERR_INVALID_ARG, "%s: dy, x, dx%s must be non-null", fn,
                rms ? " and scale" : ", mean and rstd");
  st = check_aligned(fn, {dy, x, gamma, beta, scale, dres, dx, dgamma, dbeta, dscale, dshift});
  if (st != SOL_OK) return st;
  if ((reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd)) & 3u)
    return fail(SOL_ERR_MISALIGNED, "%s: mean and rstd must be 4-byte aligned", fn);
  const size_t need = sol_norm_backward_workspace_bytes(B, L, D);
  if (rows > 0 && sums) {
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != SOL_OK) return st;
  }
  const int64_t act = rows * D * esize_of(dtype), vec = D * esize_of(dtype);
  st = check_overlaps(
      fn,
      {{"dy", dy, act}, {"x", x, act}, {"dres", dres, act}, {"mean", mean, rows * 4},
       {"rstd", rstd, rows * 4}, {"gamma", gamma, vec}, {"beta", beta, vec},
       {"scale", scale, 2 * B * vec}},
      {{"dx", dx, act}, {"dgamma", dgamma, D * 4}, {"dbeta", dbeta, D * 4},
       {"dscale", dscale, 2 * B * D * 4}, {"dshift", dshift, 2 * B * D * 4},
       {"workspace", sums && rows > 0 ? workspace : nullptr, static_cast<int64_t>(need)}},
      {{dx, dy}, {dx, x}, {dx, dres}});
  if (st != SOL_OK) return st;

  SumArgs s{};
  s.seg = segments(B, L, n_video, scale != nullptr);
  if (rows > 0) {
    NormBwdArgs a{};
    a.dy = dy;
    a.x = x;
    a.mean = mean;
    a.rstd = rstd;
    a.gamma = gamma;
    a.scale = scale;
    a.dres = dres;
    a.dx = dx;
    a.partial = sums ? static_cast<float *>(workspace) : nullptr;
    a.seg = s.seg;
    a.nvec = static_cast<int>(vec / 16);
    a.D = static_cast<int>(D);
    a.eps = eps;
    a.rms = rms;
    const cudaError_t e = launch_norm_backward(a, dtype_index(dtype), stream);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    s.seg = a.seg;
  }
  s.partial = static_cast<const float *>(workspace);
  s.sums = 2;
  s.D = static_cast<int>(D);
  s.scale = scale;
  s.gamma = gamma;
  s.beta = beta;
  s.dscale = dscale;
  s.dshift = dshift;
  s.dgamma = dgamma;
  s.dbeta = dbeta;
  s.mult = 1.f;
  const cudaError_t e = launch_segment_sums(s, dtype_index(dtype), stream);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

// p, rng and site of a dropout into `a`.
sol_status check_dropout(const char *fn, const uint64_t *rng, uint64_t site, float p,
                         bool rows, DropArgs &a) {
  if (!(p >= 0.f && p <= 1.f)) return fail(SOL_ERR_INVALID_ARG, "%s: need 0 <= p <= 1", fn);
  const double thr = std::nearbyint(static_cast<double>(p) * 4294967296.0);
  a.drop = thr > 0.0;
  if (rows && a.drop && !rng)
    return fail(SOL_ERR_INVALID_ARG, "%s: rng must be non-null with p > 0", fn);
  if (reinterpret_cast<uintptr_t>(rng) & 7u)
    return fail(SOL_ERR_MISALIGNED, "%s: rng must be 8-byte aligned", fn);
  a.rng = rng;
  a.site = site;
  a.drop_max = a.drop ? static_cast<uint32_t>(thr - 1.0) : 0;
  a.keep_scale = p < 1.f ? static_cast<float>(1.0 / (1.0 - static_cast<double>(p))) : 0.f;
  return SOL_OK;
}

// ---- rotary positions ---------------------------------------------------------

sol_status check_plan(const char *fn, const sol_rope_plan *plan, sol_dtype dtype) {
  if (dtype != SOL_F32 && dtype != SOL_BF16)
    return fail(SOL_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
  if (!plan) return fail(SOL_ERR_INVALID_ARG, "%s: plan must be non-null", fn);
  if (plan->head_dim < 2 || plan->head_dim > 256 || plan->rot_dim <= 0 ||
      plan->rot_dim > plan->head_dim || plan->rot_dim % 2 != 0 || plan->n_axes < 1 ||
      plan->n_axes > 8 || (plan->half_split != 0 && plan->half_split != 1))
    return fail(SOL_ERR_INVALID_ARG, "%s: bad plan (head_dim %d, rot_dim %d, n_axes %d)", fn,
                plan->head_dim, plan->rot_dim, plan->n_axes);
  for (int i = 0; i < plan->rot_dim / 2; ++i)
    if (plan->axis[i] >= plan->n_axes || !std::isfinite(plan->freq[i]))
      return fail(SOL_ERR_INVALID_ARG, "%s: plan pair %d has axis %d, frequency %g", fn, i,
                  plan->axis[i], plan->freq[i]);
  const int E = 16 / esize_of(dtype);
  if (plan->head_dim % E != 0 || plan->head_dim / E > 32 ||
      (plan->half_split && plan->rot_dim / 2 % E != 0))
    return fail(SOL_ERR_UNSUPPORTED,
                "%s: head_dim (half-split: rot_dim / 2) must be a multiple of %d, head_dim at "
                "most %d",
                fn, E, 32 * E);
  return SOL_OK;
}

// Bytes from the first to past the last element of a heads array; < 0 if a
// stride is negative or the extent does not fit.
int64_t heads_extent(const sol_heads &h, int64_t B, int64_t L, int head_dim, int es) {
  if (h.stride_b < 0 || h.stride_row < 0 || h.stride_head < 0) return -1;
  const __int128 n = static_cast<__int128>(B - 1) * h.stride_b +
                     static_cast<__int128>(L - 1) * h.stride_row +
                     static_cast<__int128>(h.n_heads - 1) * h.stride_head + head_dim;
  if (n > (static_cast<__int128>(1) << 56)) return -1;
  return static_cast<int64_t>(n) * es;
}

sol_status check_heads(const char *fn, const char *name, const sol_heads *h, int64_t n_heads,
                       int64_t B, int64_t L, int head_dim, int es) {
  if (!h || !h->data) return fail(SOL_ERR_INVALID_ARG, "%s: %s must be non-null", fn, name);
  if (h->n_heads != n_heads)
    return fail(SOL_ERR_INVALID_ARG, "%s: %s has %lld heads, expected %lld", fn, name,
                (long long)h->n_heads, (long long)n_heads);
  if (heads_extent(*h, B, L, head_dim, es) < 0)
    return fail(SOL_ERR_INVALID_ARG, "%s: %s has a stride out of range", fn, name);
  if (!aligned16(h->data) || h->stride_b * es % 16 || h->stride_row * es % 16 ||
      h->stride_head * es % 16)
    return fail(SOL_ERR_MISALIGNED, "%s: %s and its strides must be 16-byte aligned", fn, name);
  return SOL_OK;
}

bool same_heads(const sol_heads &a, const sol_heads &b) {
  return a.data == b.data && a.stride_b == b.stride_b && a.stride_row == b.stride_row &&
         a.stride_head == b.stride_head && a.n_heads == b.n_heads;
}

// True if no two elements of the array share an address: with the axes in order of
// their strides, each steps over all that lies below it.
bool heads_separate(const sol_heads &h, int64_t B, int64_t L, int head_dim) {
  std::pair<int64_t, int64_t> ax[3] = {
      {h.stride_b, B}, {h.stride_row, L}, {h.stride_head, h.n_heads}};
  std::sort(ax, ax + 3);
  __int128 extent = head_dim;
  for (const auto &[stride, n] : ax) {
    if (n < 2) continue;
    if (stride < extent) return false;
    extent += static_cast<__int128>(n - 1) * stride;
  }
  return true;
}

// The bytes of a strided array: runs of `width` bytes at p plus any sum of t * step
// with 0 <= t < count, one t per axis.
struct Runs {
  const void *p;
  int64_t width;
  int64_t extent;                     // from the first byte past the last
  std::pair<int64_t, int64_t> ax[3];  // (step, count)
};
Runs runs_of(const sol_heads &h, int64_t B, int64_t L, int head_dim, int es) {
  // (the step of an axis of one element says nothing)
  auto axis = [&](int64_t stride, int64_t n) {
    return std::pair<int64_t, int64_t>(n > 1 ? stride * es : 0, n);
  };
  return {h.data, int64_t(head_dim) * es, heads_extent(h, B, L, head_dim, es),
          {axis(h.stride_b, B), axis(h.stride_row, L), axis(h.stride_head, h.n_heads)}};
}

// True if no byte of `a` is one of `b`.  They meet where the distance between two
// runs, b.p - a.p + sum t * step (t >= 0 for b's axes, <= 0 for a's), lies in
// (-b.width, a.width).  Axes of one step count as one; from the largest step down,
// only the t from which the smaller steps still reach that interval are followed: two
// or three per axis where the steps nest, as in any layout of a tensor or of slices of
// one.  Layouts that take more than kMeetSteps to tell apart count as meeting.
constexpr int kMeetSteps = 1 << 14;
class Distance {
 public:
  Distance(const Runs &a, const Runs &b) : wa_(a.width), wb_(b.width) {
    off_ = static_cast<__int128>(reinterpret_cast<intptr_t>(b.p)) -
           reinterpret_cast<intptr_t>(a.p);
    for (const auto &[step, count] : b.ax) add(step, 0, count - 1);
    for (const auto &[step, count] : a.ax) add(step, 1 - count, 0);
    for (int i = n_ - 1; i >= 0; --i) {
      term_[i].least = term_[i].lo * term_[i].step + (i + 1 < n_ ? term_[i + 1].least : 0);
      term_[i].most = term_[i].hi * term_[i].step + (i + 1 < n_ ? term_[i + 1].most : 0);
    }
  }
  bool meets() { return meets_from(0, off_); }

 private:
  struct Term {
    __int128 step, lo, hi;
    __int128 least, most;  // of this term and all smaller ones
  };
  void add(int64_t step, int64_t lo, int64_t hi) {
    if (step == 0 || lo == hi) return;
    int i = 0;  // the terms stand in falling order of their steps
    while (i < n_ && term_[i].step > step) ++i;
    if (i < n_ && term_[i].step == step) {
      term_[i].lo += lo;
      term_[i].hi += hi;
      return;
    }
    for (int j = n_++; j > i; --j) term_[j] = term_[j - 1];
    term_[i] = Term{step, lo, hi, 0, 0};
  }
  static __int128 floor_div(__int128 x, __int128 y) {  // y > 0
    return x / y - (x % y < 0 ? 1 : 0);
  }
  bool meets_from(int i, __int128 off) {
    const __int128 least = i < n_ ? term_[i].least : 0, most = i < n_ ? term_[i].most : 0;
    if (off + least >= wa_ || off + most <= -wb_) return false;
    if (i == n_ || --left_ < 0) return true;
    const Term &t = term_[i];
    const __int128 rest_least = t.least - t.lo * t.step, rest_most = t.most - t.hi * t.step;
    // t * step < wa - off - rest_least and t * step > -wb - off - rest_most
    const __int128 first = std::max(t.lo, floor_div(-wb_ - off - rest_most, t.step) + 1);
    const __int128 last = std::min(t.hi, floor_div(wa_ - off - rest_least - 1, t.step));
    for (__int128 k = first; k <= last; ++k)
      if (meets_from(i + 1, off + k * t.step)) return true;
    return false;
  }
  __int128 wa_, wb_, off_;
  Term term_[6];
  int n_ = 0, left_ = kMeetSteps;
};
__attribute__((noinline)) bool runs_meet(const Runs &a, const Runs &b) {
  return Distance(a, b).meets();
}

// True if a heads array and a contiguous one, or two heads arrays, share no byte.  Most
// lie apart altogether.
bool disjoint(const Runs &a, const Arr &b) {
  return !spans_overlap(span_of(a.p, 1, 0, a.extent), span_of(b.p, 1, 0, b.bytes)) ||
         !runs_meet(a, Runs{b.p, b.bytes, b.bytes, {{0, 1}, {0, 1}, {0, 1}}});
}

// True if a and b, heads arrays, lie in column blocks of rows of one pitch (q, k and v
// of a merged projection), whatever their samples' steps: said without following those.
bool column_blocks(const Runs &a, const Runs &b) {
  const int64_t ld = a.ax[1].first;
  if (ld <= 0 || ld != b.ax[1].first || a.ax[0].first % ld != 0 || b.ax[0].first % ld != 0)
    return false;
  const int64_t wa = (a.ax[2].second - 1) * a.ax[2].first + a.width;
  const int64_t wb = (b.ax[2].second - 1) * b.ax[2].first + b.width;
  int64_t c = (static_cast<int64_t>(reinterpret_cast<intptr_t>(b.p) -
                                    reinterpret_cast<intptr_t>(a.p))) %
              ld;
  if (c < 0) c += ld;
  return wa <= c && c + wb <= ld;
}

bool disjoint(const Runs &a, const Runs &b) {
  return !spans_overlap(span_of(a.p, 1, 0, a.extent), span_of(b.p, 1, 0, b.extent)) ||
         column_blocks(a, b) || !runs_meet(a, b);
}

HeadsArg heads_arg(const sol_heads *h, int es) {
  if (!h) return HeadsArg{nullptr, 0, 0, 0};
  return HeadsArg{h->data, h->stride_b * es, h->stride_row * es, h->stride_head * es};
}

// The checks and arguments that the forward and the backward call share.  x:
// the forward inputs (backward: null without the norm), g: the gradients of
// the outputs (backward only), out: what the call writes.
sol_status rope_args(const char *fn, const sol_rope_plan *plan, const sol_positions *pos,
                     const sol_heads *const (&x)[2], const sol_heads *const (&g)[2],
                     const sol_heads *const (&out)[2], const void *gamma_q, const void *gamma_k,
                     int qk_norm, bool back, int64_t B, int64_t L, float eps, sol_dtype dtype,
                     std::initializer_list<Arr> other_outs, RopeArgs &a, bool &empty) {
  empty = false;
  sol_status st = check_plan(fn, plan, dtype);
  if (st != SOL_OK) return st;
  if (qk_norm != 0 && qk_norm != 1)
    return fail(SOL_ERR_INVALID_ARG, "%s: qk_norm must be 0 or 1", fn);
  if (!qk_norm && (gamma_q || gamma_k))
    return fail(SOL_ERR_INVALID_ARG, "%s: gamma_q and gamma_k need qk_norm", fn);
  if (qk_norm && !(eps >= 0.f)) return fail(SOL_ERR_INVALID_ARG, "%s: need eps >= 0", fn);
  if (B < 0 || L < 0) return fail(SOL_ERR_INVALID_ARG, "%s: need B, L >= 0", fn);
  if (B > kMaxRows || L > kMaxRows || B * L > kMaxRows)
    return fail(SOL_ERR_UNSUPPORTED, "%s: B*L must be below 2^31 rows", fn);
  const bool need_x = !back || qk_norm;
  if (!need_x && (x[0] || x[1]))
    return fail(SOL_ERR_INVALID_ARG, "%s: q and k must be null without qk_norm", fn);
  const int hd = plan->head_dim, es = esize_of(dtype);
  a = RopeArgs{};
  for (int t = 0; t < 2; ++t) {
    const bool have = out[t] != nullptr;
    if (t == 0 && !have) return fail(SOL_ERR_INVALID_ARG, "%s: the q arguments are required", fn);
    if (((x[t] != nullptr) != (have && need_x)) || ((g[t] != nullptr) != (have && back)))
      return fail(SOL_ERR_INVALID_ARG, "%s: the %s arguments must be given together", fn,
                  t ? "k" : "q");
    if (!have) continue;
    if (out[t]->n_heads < 1 || out[t]->n_heads > kMaxRopeHeads)
      return fail(SOL_ERR_UNSUPPORTED, "%s: 1 to %lld heads (got %lld)", fn,
                  (long long)kMaxRopeHeads, (long long)out[t]->n_heads);
    a.heads[t] = static_cast<int>(out[t]->n_heads);
  }
  if (!out[1] && gamma_k)
    return fail(SOL_ERR_INVALID_ARG, "%s: gamma_k without k", fn);
  if (!pos || pos->type < SOL_POS_I32 || pos->type > SOL_POS_F32 || pos->reserved != 0 ||
      pos->stride_axis < 0 || pos->stride_b < 0)
    return fail(SOL_ERR_INVALID_ARG, "%s: bad positions", fn);
  if (B * L == 0) {
    empty = true;
    return SOL_OK;
  }
  if (!pos->data) return fail(SOL_ERR_INVALID_ARG, "%s: positions must be non-null", fn);
  const int pes = pos->type == SOL_POS_I64 ? 8 : 4;
  if (reinterpret_cast<uintptr_t>(pos->data) % pes)
    return fail(SOL_ERR_MISALIGNED, "%s: positions must be aligned to their element", fn);
  st = check_aligned(fn, {gamma_q, gamma_k});
  if (st != SOL_OK) return st;
  for (int t = 0; t < 2; ++t) {
    if (!out[t]) continue;
    for (const sol_heads *h : {x[t], g[t], out[t]}) {
      if (!h) continue;
      const char *name = h == out[t] ? (t ? "the k output" : "the q output")
                                     : (t ? "a k input" : "a q input");
      st = check_heads(fn, name, h, a.heads[t], B, L, hd, es);
      if (st != SOL_OK) return st;
    }
    if (!heads_separate(*out[t], B, L, hd))
      return fail(SOL_ERR_INVALID_ARG, "%s: the strides of an output make its heads overlap", fn);
  }
  const __int128 n_pos = static_cast<__int128>(plan->n_axes - 1) * pos->stride_axis +
                         static_cast<__int128>(B - 1) * pos->stride_b + L;
  if (n_pos > (static_cast<__int128>(1) << 56))
    return fail(SOL_ERR_INVALID_ARG, "%s: positions have a stride out of range", fn);
  const int64_t pos_bytes = static_cast<int64_t>(n_pos) * pes;
  const Arr small[] = {{"positions", pos->data, pos_bytes},
                       {"gamma_q", gamma_q, static_cast<int64_t>(hd) * es},
                       {"gamma_k", gamma_k, static_cast<int64_t>(hd) * es}};
  Runs rx[2], rg[2], ro[2];
  for (int t = 0; t < 2; ++t) {
    if (x[t]) rx[t] = runs_of(*x[t], B, L, hd, es);
    if (g[t]) rg[t] = runs_of(*g[t], B, L, hd, es);
    if (out[t]) ro[t] = runs_of(*out[t], B, L, hd, es);
  }
  for (int t = 0; t < 2; ++t) {
    if (!out[t]) continue;
    for (const Arr &s : small)
      if (s.p && !disjoint(ro[t], s))
        return fail(SOL_ERR_INVALID_ARG, "%s: an output overlaps %s", fn, s.name);
    for (const Arr &o : other_outs)
      if (o.p && o.bytes && !disjoint(ro[t], o))
        return fail(SOL_ERR_INVALID_ARG, "%s: an output overlaps %s", fn, o.name);
    for (int u = 0; u < 2; ++u)
      for (int in = 0; in < 2; ++in) {
        const sol_heads *h = in ? g[u] : x[u];
        if (!h || (u == t && same_heads(*h, *out[t]))) continue;
        if (!disjoint(ro[t], in ? rg[u] : rx[u]))
          return fail(SOL_ERR_INVALID_ARG,
                      "%s: an output must equal its own input exactly or overlap no argument", fn);
      }
  }
  if (out[1] && !disjoint(ro[0], ro[1]))
    return fail(SOL_ERR_INVALID_ARG, "%s: the two outputs overlap", fn);
  for (const Arr &o : other_outs) {
    if (!o.p || !o.bytes) continue;
    const Span so = span_of(o.p, 1, 0, o.bytes);
    for (const Arr &s : small)
      if (s.p && spans_overlap(so, span_of(s.p, 1, 0, s.bytes)))
        return fail(SOL_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, o.name, s.name);
    for (const Arr &q : other_outs)
      if (&q != &o && q.p && q.bytes && spans_overlap(so, span_of(q.p, 1, 0, q.bytes)))
        return fail(SOL_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, o.name, q.name);
    for (int u = 0; u < 2; ++u)
      if ((x[u] && !disjoint(rx[u], o)) || (g[u] && !disjoint(rg[u], o)))
        return fail(SOL_ERR_INVALID_ARG, "%s: %s overlaps an input", fn, o.name);
  }

  for (int t = 0; t < 2; ++t) {
    a.x[t] = heads_arg(x[t], es);
    a.g[t] = heads_arg(g[t], es);
    a.out[t] = heads_arg(out[t], es);
  }
  a.gamma[0] = gamma_q;
  a.gamma[1] = gamma_k;
  a.pos = pos->data;
  a.pos_stride_axis = pos->stride_axis;
  a.pos_stride_b = pos->stride_b;
  a.pos_type = pos->type;
  a.L = static_cast<int>(L);
  a.rows = B * L;
  a.head_dim = hd;
  a.rot_dim = plan->rot_dim;
  a.eps = eps;
  a.inv_hd = static_cast<float>(1.0 / hd);
  for (int i = 0; i < plan->rot_dim / 2; ++i) {
    a.axis[i] = plan->axis[i];
    a.freq[i] = plan->freq[i];
  }
  return SOL_OK;
}

cudaError_t launch_rope(RopeArgs &a, RopeMode mode, bool half, sol_dtype dtype,
                        cudaStream_t stream, int *ctas) {
  return dtype == SOL_F32 ? launch_rope_axes_f32(a, mode, half, stream, ctas)
                          : launch_rope_axes_bf16(a, mode, half, stream, ctas);
}

}  // namespace
}  // namespace sol

using namespace sol;

extern "C" {

sol_status sol_layer_norm(const void *x, void *y, float *mean, float *rstd, const void *gamma,
                          const void *beta, const void *scale, const void *shift, int64_t B,
                          int64_t L, int64_t n_video, int64_t D, float eps, sol_dtype dtype,
                          sol_stream_t stream) {
  return guarded([&]() -> sol_status {
    const char *fn = "sol_layer_norm";
    sol_status st = check_rows(fn, B, L, n_video, D, dtype);
    if (st != SOL_OK) return st;
    if (!(eps >= 0.f)) return fail(SOL_ERR_INVALID_ARG, "%s: need eps >= 0", fn);
    if ((mean == nullptr) != (rstd == nullptr))
      return fail(SOL_ERR_INVALID_ARG, "%s: give both mean and rstd, or neither", fn);
    if ((scale == nullptr) != (shift == nullptr))
      return fail(SOL_ERR_INVALID_ARG, "%s: give both scale and shift, or neither", fn);
    const int64_t rows = B * L;
    if (rows == 0) return ok();
    if (!x || !y) return fail(SOL_ERR_INVALID_ARG, "%s: x and y must be non-null", fn);
    st = check_aligned(fn, {x, y, gamma, beta, scale, shift});
    if (st != SOL_OK) return st;
    if ((reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd)) & 3u)
      return fail(SOL_ERR_MISALIGNED, "%s: mean and rstd must be 4-byte aligned", fn);
    const int64_t vec = D * esize_of(dtype), act = rows * vec;
    st = check_overlaps(fn,
                        {{"x", x, act}, {"gamma", gamma, vec}, {"beta", beta, vec},
                         {"scale", scale, 2 * B * vec}, {"shift", shift, 2 * B * vec}},
                        {{"y", y, act}, {"mean", mean, rows * 4}, {"rstd", rstd, rows * 4}},
                        {{y, x}});
    if (st != SOL_OK) return st;
    LnArgs a{};
    a.x = x;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.gamma = gamma;
    a.beta = beta;
    a.scale = scale;
    a.shift = shift;
    a.rows = rows;
    a.L = static_cast<int>(scale ? L : rows);
    a.n_video = static_cast<int>(scale ? n_video : rows);
    a.nvec = static_cast<int>(vec / 16);
    a.D = static_cast<int>(D);
    a.eps = eps;
    const cudaError_t e = launch_layer_norm(a, dtype_index(dtype), stream);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return ok();
  });
}

size_t sol_norm_backward_workspace_bytes(int64_t B, int64_t L, int64_t D) {
  if (!sizes_ok(B, L, D)) return 0;
  return static_cast<size_t>(sum_slots(B * L, 2 * B)) * 2 * static_cast<size_t>(D) * 4;
}

size_t sol_dropout_backward_workspace_bytes(int64_t B, int64_t L, int64_t D) {
  if (!sizes_ok(B, L, D)) return 0;
  return static_cast<size_t>(sum_slots(B * L, 2 * B)) * static_cast<size_t>(D) * 4;
}

sol_status sol_layer_norm_backward(const void *dy, const void *x, const float *mean,
                                   const float *rstd, const void *gamma, const void *beta,
                                   const void *scale, const void *dres, void *dx, float *dgamma,
                                   float *dbeta, float *dscale, float *dshift, int64_t B,
                                   int64_t L, int64_t n_video, int64_t D, void *workspace,
                                   size_t workspace_bytes, sol_dtype dtype,
                                   sol_stream_t stream) {
  return guarded([&]() -> sol_status {
    return norm_backward("sol_layer_norm_backward", false, dy, x, mean, rstd, gamma, beta, scale,
                         dres, dx, dgamma, dbeta, dscale, dshift, B, L, n_video, D, 0.f,
                         workspace, workspace_bytes, dtype, stream);
  });
}

sol_status sol_rms_adaln_backward(const void *dy, const void *x, const void *scale,
                                  const void *gamma, const void *dres, void *dx, float *dscale,
                                  float *dshift, float *dgamma, int64_t B, int64_t L,
                                  int64_t n_video, int64_t D, float eps, void *workspace,
                                  size_t workspace_bytes, sol_dtype dtype, sol_stream_t stream) {
  return guarded([&]() -> sol_status {
    return norm_backward("sol_rms_adaln_backward", true, dy, x, nullptr, nullptr, gamma, nullptr,
                         scale, dres, dx, dgamma, nullptr, dscale, dshift, B, L, n_video, D, eps,
                         workspace, workspace_bytes, dtype, stream);
  });
}

sol_status sol_dropout_residual(const void *h, const void *branch, const void *gate, void *out,
                                const uint64_t *rng, uint64_t site, float p, int64_t B, int64_t L,
                                int64_t n_video, int64_t D, sol_dtype dtype,
                                sol_stream_t stream) {
  return guarded([&]() -> sol_status {
    const char *fn = "sol_dropout_residual";
    sol_status st = check_rows(fn, B, L, n_video, D, dtype);
    if (st != SOL_OK) return st;
    const int64_t rows = B * L;
    DropArgs a{};
    st = check_dropout(fn, rng, site, p, rows > 0, a);
    if (st != SOL_OK) return st;
    if (rows == 0) return ok();
    if (!branch || !out)
      return fail(SOL_ERR_INVALID_ARG, "%s: branch and out must be non-null", fn);
    st = check_aligned(fn, {h, branch, gate, out});
    if (st != SOL_OK) return st;
    const int64_t vec = D * esize_of(dtype), act = rows * vec;
    st = check_overlaps(fn,
                        {{"h", h, act}, {"branch", branch, act}, {"gate", gate, 2 * B * vec},
                         {"rng", rng, 16}},
                        {{"out", out, act}}, {{out, h}, {out, branch}});
    if (st != SOL_OK) return st;
    a.h = h;
    a.branch = branch;
    a.gate = gate;
    a.out = out;
    a.seg = segments(B, L, n_video, gate != nullptr);
    a.nvec = static_cast<int>(vec / 16);
    a.D = static_cast<int>(D);
    const cudaError_t e = launch_dropout_residual(a, dtype_index(dtype), stream);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return ok();
  });
}

sol_status sol_dropout_residual_backward(const void *dout, const void *branch, const void *gate,
                                         void *dbranch, float *dgate, const uint64_t *rng,
                                         uint64_t site, float p, int64_t B, int64_t L,
                                         int64_t n_video, int64_t D, void *workspace,
                                         size_t workspace_bytes, sol_dtype dtype,
                                         sol_stream_t stream) {
  return guarded([&]() -> sol_status {
    const char *fn = "sol_dropout_residual_backward";
    sol_status st = check_rows(fn, B, L, n_video, D, dtype);
    if (st != SOL_OK) return st;
    const int64_t rows = B * L;
    DropArgs a{};
    st = check_dropout(fn, rng, site, p, rows > 0, a);
    if (st != SOL_OK) return st;
    if (dgate && !gate) return fail(SOL_ERR_INVALID_ARG, "%s: dgate needs gate", fn);
    if (rows > 0 && (!dout || !dbranch || (dgate && !branch)))
      return fail(SOL_ERR_INVALID_ARG, "%s: dout, dbranch (and branch, with dgate) must be "
                  "non-null", fn);
    st = check_aligned(fn, {dout, branch, gate, dbranch, dgate});
    if (st != SOL_OK) return st;
    const size_t need = sol_dropout_backward_workspace_bytes(B, L, D);
    const bool sums = dgate && rows > 0;
    if (sums) {
      st = check_workspace(fn, workspace, workspace_bytes, need);
      if (st != SOL_OK) return st;
    }
    const int64_t vec = D * esize_of(dtype), act = rows * vec;
    st = check_overlaps(fn,
                        {{"dout", dout, act}, {"branch", branch, act},
                         {"gate", gate, 2 * B * vec}, {"rng", rng, 16}},
                        {{"dbranch", dbranch, act}, {"dgate", dgate, 2 * B * D * 4},
                         {"workspace", sums ? workspace : nullptr, static_cast<int64_t>(need)}},
                        {{dbranch, dout}, {dbranch, branch}});
    if (st != SOL_OK) return st;
    a.gate = gate;
    a.out = dbranch;
    a.seg = segments(B, L, n_video, gate != nullptr);
    a.nvec = static_cast<int>(vec / 16);
    a.D = static_cast<int>(D);
    if (rows > 0 && !dgate) {  // the forward kernel on dout, without h
      a.branch = dout;
      const cudaError_t e = launch_dropout_residual(a, dtype_index(dtype), stream);
      if (e != cudaSuccess) return cuda_fail(e, fn);
      return ok();
    }
    if (rows > 0) {
      a.dout = dout;
      a.branch = branch;
      a.partial = static_cast<float *>(workspace);
      const cudaError_t e = launch_dropout_backward(a, dtype_index(dtype), stream);
      if (e != cudaSuccess) return cuda_fail(e, fn);
    }
    SumArgs s{};
    s.seg = a.seg;
    s.partial = a.partial;
    s.sums = 1;
    s.D = a.D;
    s.dscale = dgate;
    s.mult = a.keep_scale;
    const cudaError_t e = launch_segment_sums(s, dtype_index(dtype), stream);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return ok();
  });
}

sol_status sol_rope_plan_init(sol_rope_plan *plan, int64_t head_dim, int64_t rot_dim,
                              int64_t n_axes, const int64_t *sections, double theta,
                              int per_axis_freq, int interleaved, int half_split) {
  return guarded([&]() -> sol_status {
    const char *fn = "sol_rope_plan_init";
    if (!plan || !sections)
      return fail(SOL_ERR_INVALID_ARG, "%s: plan and sections must be non-null", fn);
    if (head_dim < 2 || head_dim > 256 || rot_dim <= 0 || rot_dim > head_dim || rot_dim % 2 != 0)
      return fail(SOL_ERR_INVALID_ARG,
                  "%s: need head_dim in [2, 256] and an even rot_dim in [2, head_dim]", fn);
    if (n_axes < 1 || n_axes > 8)
      return fail(SOL_ERR_INVALID_ARG, "%s: need 1 to 8 axes", fn);
    if (!(theta > 0.0) || !std::isfinite(theta))
      return fail(SOL_ERR_INVALID_ARG, "%s: theta must be > 0 and finite", fn);
    for (int f : {per_axis_freq, interleaved, half_split})
      if (f != 0 && f != 1)
        return fail(SOL_ERR_INVALID_ARG,
                    "%s: per_axis_freq, interleaved and half_split must be 0 or 1", fn);
    int64_t sum = 0;
    for (int64_t a = 0; a < n_axes; ++a) {
      if (sections[a] < 0 || sections[a] > 128)
        return fail(SOL_ERR_INVALID_ARG, "%s: sections[%lld] is out of range", fn, (long long)a);
      sum += sections[a];
    }
    if (sum != rot_dim / 2)
      return fail(SOL_ERR_INVALID_ARG, "%s: sections sum to %lld, not rot_dim/2 = %lld", fn,
                  (long long)sum, (long long)(rot_dim / 2));
    sol_rope_plan p{};
    p.head_dim = static_cast<int32_t>(head_dim);
    p.rot_dim = static_cast<int32_t>(rot_dim);
    p.n_axes = static_cast<int32_t>(n_axes);
    p.half_split = half_split;
    int64_t taken[8] = {0};
    int a = 0;
    for (int i = 0; i < rot_dim / 2; ++i) {
      while (taken[a] == sections[a]) a = (a + 1) % static_cast<int>(n_axes);
      const double e = per_axis_freq
                           ? static_cast<double>(taken[a]) / static_cast<double>(sections[a])
                           : 2.0 * i / static_cast<double>(rot_dim);
      p.axis[i] = static_cast<uint8_t>(a);
      p.freq[i] = std::pow(theta, -e);
      ++taken[a];
      if (interleaved) a = (a + 1) % static_cast<int>(n_axes);
    }
    *plan = p;
    return ok();
  });
}

size_t sol_rope_backward_workspace_bytes(int64_t head_dim) {
  if (head_dim < 2 || head_dim > 256) return 0;
  return static_cast<size_t>(kMaxRopeCtas) * 2 * static_cast<size_t>(head_dim) * 4;
}

sol_status sol_rope_axes(const sol_rope_plan *plan, const sol_positions *pos, const sol_heads *q,
                         const sol_heads *k, const sol_heads *q_out, const sol_heads *k_out,
                         const void *gamma_q, const void *gamma_k, int qk_norm, int64_t B,
                         int64_t L, float eps, sol_dtype dtype, sol_stream_t stream) {
  return guarded([&]() -> sol_status {
    const char *fn = "sol_rope_axes";
    RopeArgs a{};
    bool empty = false;
    const sol_heads *const x[2] = {q, k}, *const g[2] = {nullptr, nullptr},
                           *const out[2] = {q_out, k_out};
    const sol_status st = rope_args(fn, plan, pos, x, g, out, gamma_q, gamma_k, qk_norm, false,
                                    B, L, eps, dtype, {}, a, empty);
    if (st != SOL_OK) return st;
    if (empty) return ok();
    int ctas = 0;
    const cudaError_t e = launch_rope(a, qk_norm ? kNormRotate : kRotate,
                                      plan->half_split != 0, dtype, stream, &ctas);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return ok();
  });
}

sol_status sol_rope_axes_backward(const sol_rope_plan *plan, const sol_positions *pos,
                                  const sol_heads *dq_out, const sol_heads *dk_out,
                                  const sol_heads *q, const sol_heads *k, const sol_heads *dq,
                                  const sol_heads *dk, const void *gamma_q, const void *gamma_k,
                                  float *dgamma_q, float *dgamma_k, int qk_norm, int64_t B,
                                  int64_t L, float eps, void *workspace, size_t workspace_bytes,
                                  sol_dtype dtype, sol_stream_t stream) {
  return guarded([&]() -> sol_status {
    const char *fn = "sol_rope_axes_backward";
    RopeArgs a{};
    bool empty = false;
    const bool sums = dgamma_q || dgamma_k;
    if (sums && qk_norm == 0)
      return fail(SOL_ERR_INVALID_ARG, "%s: dgamma needs qk_norm", fn);
    if (dgamma_k && !dk) return fail(SOL_ERR_INVALID_ARG, "%s: dgamma_k without k", fn);
    const int64_t hd = plan ? plan->head_dim : 0;
    const size_t need = sums ? sol_rope_backward_workspace_bytes(hd) : 0;
    sol_status st = check_aligned(fn, {dgamma_q, dgamma_k});
    if (st == SOL_OK && sums && B > 0 && L > 0)
      st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != SOL_OK) return st;
    const sol_heads *const x[2] = {q, k}, *const g[2] = {dq_out, dk_out},
                           *const out[2] = {dq, dk};
    st = rope_args(fn, plan, pos, x, g, out, gamma_q, gamma_k, qk_norm, true, B, L, eps, dtype,
                   {{"dgamma_q", dgamma_q, hd * 4},
                    {"dgamma_k", dgamma_k, hd * 4},
                    {"workspace", sums ? workspace : nullptr, static_cast<int64_t>(need)}},
                   a, empty);
    if (st != SOL_OK) return st;
    int ctas = 0;
    if (!empty) {
      if (sums) a.partial = static_cast<float *>(workspace);
      const cudaError_t e = launch_rope(a, qk_norm ? kNormRotateBack : kRotateBack,
                                        plan->half_split != 0, dtype, stream, &ctas);
      if (e != cudaSuccess) return cuda_fail(e, fn);
    }
    const cudaError_t e = launch_rope_dgamma(static_cast<const float *>(workspace), ctas,
                                             static_cast<int>(hd), dgamma_q, dgamma_k, stream);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return ok();
  });
}

}  // extern "C"
