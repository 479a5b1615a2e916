// Layer norm with optional weight, bias and adaptive modulation:
//   n = (x - mean) * rstd * gamma + beta,  rstd = 1 / sqrt(var + eps),
//   y = n * (1 + scale[b][m]) + shift[b][m]
// per token row, m = video/audio modality of the row.  Per channel this is
// y = (x - mean) * rstd * fac + off with fac = gamma * (1 + scale) and
// off = beta * (1 + scale) + shift, both kept in fp32 registers and rebuilt
// only when a CTA crosses a modality or sample boundary.
//
// The same persistent cp.async ring as RMS-AdaLN: chunks of rows dealt
// round-robin over the CTAs, R rows per iteration, compile-time CTA size and
// vectors per thread.
//
// Statistics in one barrier: each warp takes the mean of its own slice of the
// row and the sum of squares about it, both from registers, and the warps'
// (sum, M2) pairs are combined exactly,
//   mean = sum sum_w / D,  M2 = sum M2_w + n_w (mean_w - mean)^2,
// so a row whose mean is large against its spread loses no digits, as
// mean(x^2) - mean^2 would.
//
// Bound by HBM: x read, y written, 2*D*esize bytes per row.
#include "sol_device.cuh"
#include "sol_train.h"

namespace sol {
namespace {

// A staged vector, read again at each use: holding a row's unpacked channels
// across the reductions took 252 registers at 128 x 5 and left 8 warps on an
// SM (0.469 ms at the 5 s clip).
__device__ __forceinline__ uint4 ld_staged(const uint4 *p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p))
               : "memory");
  return v;
}

// Threads per SM that the registers are to leave room for (128 registers a
// thread): 0.424 ms at the 5 s clip, against 0.449 ms without the bound (150
// registers) and 0.78 ms at 96 registers, which spill.
constexpr int kLnThreadsPerSm = 512;

template <typename T, int NT, int VPT, int R, int S, int K, bool FULL>
__global__ void __launch_bounds__(NT, kLnThreadsPerSm / NT < 16 ? kLnThreadsPerSm / NT : 16)
    layer_norm_kernel(const LnArgs a) {
  static_assert(K % R == 0, "an iteration's rows must lie in one chunk");
  using IO = Io<T>;
  constexpr int P = IO::E / 2;
  constexpr int NW = NT / 32;
  extern __shared__ __align__(16) unsigned char smem[];
  float4 *red = reinterpret_cast<float4 *>(smem);  // [2][R][NW]: sum_w, M2_w, mean_w, n_w
  uint4 *ring = reinterpret_cast<uint4 *>(smem + 2 * R * NW * 16);  // [S][R][VPT][NT]

  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int warp = tid >> 5;
  const int64_t row_bytes = static_cast<int64_t>(a.nvec) * 16;
  const float inv_D = 1.f / static_cast<float>(a.D);

  bool ok[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) ok[k] = FULL || k * NT + tid < a.nvec;
  // elements of a row that this warp holds
  float n_w = 0.f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int m = a.nvec - k * NT - warp * 32;
    n_w += static_cast<float>((m < 0 ? 0 : (m > 32 ? 32 : m)) * IO::E);
  }
  const float inv_nw = n_w > 0.f ? 1.f / n_w : 0.f;

  RowOrder<K, R> ro;
  ro.init(a.rows);
  const int count = ro.count;
  const int iters = (count + R - 1) / R;
  const unsigned char *xc = static_cast<const unsigned char *>(a.x);
  unsigned char *yc = static_cast<unsigned char *>(a.y);

  auto slot = [&](int s, int q, int k) -> uint4 * {
    return &ring[((s * R + q) * VPT + k) * NT + tid];
  };
  auto issue = [&](int it, int s) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int j = it * R + q;
      if (j < count) {
        const uint4 *src = reinterpret_cast<const uint4 *>(xc + ro.row(j) * row_bytes) + tid;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
          if (ok[k]) cp_async16(slot(s, q, k), src + k * NT);
      }
    }
    cp_async_commit();
  };

#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(s, s);

  float2 fac[VPT][P], off[VPT][P];
  int key = -1;
  int cons = 0;
  int buf = 0;
  TokenCursor cur;

  auto load_vectors = [&]() {
    const int64_t koff = static_cast<int64_t>(key) * a.nvec + tid;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (ok[k]) {
#pragma unroll
        for (int m = 0; m < P; ++m) {
          fac[k][m] = splat2(1.f);
          off[k][m] = splat2(0.f);
        }
        if (a.gamma)
          IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.gamma) + k * NT + tid), fac[k]);
        if (a.beta)
          IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.beta) + k * NT + tid), off[k]);
        if (a.scale) {
          float2 sc[P], sh[P];
          IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.scale) + koff + k * NT), sc);
          IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.shift) + koff + k * NT), sh);
#pragma unroll
          for (int m = 0; m < P; ++m) {
            sc[m] = add2(sc[m], splat2(1.f));
            fac[k][m] = mul2(fac[k][m], sc[m]);
            off[k][m] = fma2(off[k][m], sc[m], sh[m]);
          }
        }
      }
    }
  };
  auto row_sum = [&](int q) -> float {
    float2 acc = splat2(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (ok[k]) {
        float2 x[P];
        IO::unpack(ld_staged(slot(cons, q, k)), x);
#pragma unroll
        for (int m = 0; m < P; ++m) acc = add2(x[m], acc);
      }
    }
    return acc.x + acc.y;
  };
  auto spread = [&](int q, float mu) -> float {
    float2 acc = splat2(0.f);
    const float2 neg = splat2(-mu);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (ok[k]) {
        float2 x[P];
        IO::unpack(ld_staged(slot(cons, q, k)), x);
#pragma unroll
        for (int m = 0; m < P; ++m) {
          const float2 d = add2(x[m], neg);
          acc = fma2(d, d, acc);
        }
      }
    }
    return acc.x + acc.y;
  };
  // (mean, rstd) of the row whose warp sums are parked in red[buf][q]
  auto combine = [&](int q) -> float2 {
    const float4 *r = red + (buf * R + q) * NW;
    float4 v[NW];
    float sum = 0.f, m2 = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      v[w] = r[w];
      sum += v[w].x;
    }
    const float mean = sum * inv_D;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float d = v[w].z - mean;
      m2 += fmaf(v[w].w * d, d, v[w].y);
    }
    return make_float2(mean, rsqrtf(fmaf(m2, inv_D, a.eps)));
  };
  auto store_row = [&](int q, int j, float2 st) {
    const int64_t row = ro.row(j);
    const float2 inv2 = splat2(st.y), neg = splat2(-st.x);
    uint4 *yrow = reinterpret_cast<uint4 *>(yc + row * row_bytes) + tid;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (ok[k]) {
        float2 x[P], o[P];
        IO::unpack(ld_staged(slot(cons, q, k)), x);
#pragma unroll
        for (int m = 0; m < P; ++m)
          o[m] = fma2(add2(x[m], neg), mul2(fac[k][m], inv2), off[k][m]);
        st_stream16(yrow + k * NT, IO::pack(o));
      }
    }
    if (a.mean && tid == 0) {
      a.mean[row] = st.x;
      a.rstd[row] = st.y;
    }
  };

  for (int it = 0; it < iters; ++it) {
    issue(it + S - 1, cons == 0 ? S - 1 : cons - 1);
    if (ro.run_start(it * R)) cur.init(ro.row(it * R), a.L);
    const int nrows = count - it * R < R ? count - it * R : R;
    bool same = true;  // every row of this iteration uses the cached vectors
    {
      TokenCursor c = cur;
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (q < nrows) same &= (2 * c.b + (c.r >= a.n_video ? 1 : 0)) == key;
        c.next(a.L);
      }
    }
    cp_async_wait<S - 1>();

    if (same) {
      float sum[R], mu[R], m2[R];
#pragma unroll
      for (int q = 0; q < R; ++q) sum[q] = q < nrows ? row_sum(q) : 0.f;
#pragma unroll
      for (int q = 0; q < R; ++q) {
        sum[q] = warp_sum(sum[q]);
        mu[q] = sum[q] * inv_nw;
      }
#pragma unroll
      for (int q = 0; q < R; ++q) m2[q] = q < nrows ? spread(q, mu[q]) : 0.f;
#pragma unroll
      for (int q = 0; q < R; ++q) m2[q] = warp_sum(m2[q]);
      if (NW > 1) {
        if (lane == 0) {
#pragma unroll
          for (int q = 0; q < R; ++q)
            red[(buf * R + q) * NW + warp] = make_float4(sum[q], m2[q], mu[q], n_w);
        }
        __syncthreads();
      }
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (q < nrows) {
          const float2 st = NW > 1 ? combine(q)
                                   : make_float2(mu[q], rsqrtf(fmaf(m2[q], inv_D, a.eps)));
          store_row(q, it * R + q, st);
        }
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (q < nrows) cur.next(a.L);
    } else {
      // a modality or sample boundary: rebuild the vectors row by row
#pragma unroll 1
      for (int q = 0; q < nrows; ++q) {
        const int nkey = 2 * cur.b + (cur.r >= a.n_video ? 1 : 0);
        if (nkey != key) {
          key = nkey;
          load_vectors();
        }
        const float sum = warp_sum(row_sum(q));
        const float mu = sum * inv_nw;
        const float m2 = warp_sum(spread(q, mu));
        float2 st;
        if (NW > 1) {
          if (lane == 0) red[(buf * R + q) * NW + warp] = make_float4(sum, m2, mu, n_w);
          __syncthreads();
          st = combine(q);
        } else {
          st = make_float2(mu, rsqrtf(fmaf(m2, inv_D, a.eps)));
        }
        store_row(q, it * R + q, st);
        cur.next(a.L);
      }
    }
    buf ^= 1;
    cons = (cons + 1 == S) ? 0 : cons + 1;
  }
  cp_async_wait<0>();
}

template <int VPT>
constexpr int kLnRows = VPT <= 5 ? 2 : 1;

// chunk of consecutive rows per CTA turn, as RMS-AdaLN's
constexpr int kLnChunk = 8;

template <typename T, int NT, int VPT, bool FULL>
cudaError_t launch_t(const LnArgs &a, cudaStream_t stream) {
  constexpr int R = kLnRows<VPT>, S = 2;
  auto *kern = &layer_norm_kernel<T, NT, VPT, R, S, kLnChunk, FULL>;
  const void *fn = reinterpret_cast<const void *>(kern);
  const size_t smem = 2 * R * (NT / 32) * 16 + static_cast<size_t>(S) * R * VPT * NT * 16;
  const int per_sm = resident_blocks(fn, NT, smem);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t grid = static_cast<int64_t>(per_sm) * device_sms();
  if (grid > a.rows) grid = a.rows;
  kern<<<static_cast<unsigned>(grid), NT, smem, stream>>>(a);
  return cudaGetLastError();
}

// A short launch whose split covers the row exactly takes the unguarded
// instantiation (FULL), as in RMS-AdaLN: 36.7 against 41.0 us at 8,264 rows of
// 5120 bf16; at 126,552 rows it was 3% slower.
constexpr int64_t kFullMaxRows = 16384;

template <typename T>
cudaError_t dispatch(const LnArgs &a, int threads, int vpt, cudaStream_t stream) {
#define SOL_CASE(NT, V)                                       \
  if (threads == NT && vpt == V)                              \
    return a.nvec == NT * V && a.rows <= kFullMaxRows        \
               ? launch_t<T, NT, V, true>(a, stream)          \
               : launch_t<T, NT, V, false>(a, stream);
  SOL_SPLITS(SOL_CASE)
#undef SOL_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_layer_norm(const LnArgs &a, int dtype, cudaStream_t stream) {
  int threads = 0, vpt = 0;
  if (!pick_split(a.nvec, &threads, &vpt)) return cudaErrorInvalidValue;
  return dtype == 0 ? dispatch<float>(a, threads, vpt, stream)
                    : dispatch<__nv_bfloat16>(a, threads, vpt, stream);
}

}  // namespace sol
