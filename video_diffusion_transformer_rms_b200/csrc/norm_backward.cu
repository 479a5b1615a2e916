// Backward pass of the layer norm and of RMS-AdaLN.
//
// With W = gamma * (1 + scale[b][m]), g = dy * W and x^ = (x - mean) * rstd
// (RMS: mean = 0), per token row
//   dx = rstd * (g - mean(g) - x^ * mean(g * x^)) [+ dres]     (RMS: no mean(g))
// and per (sample, modality) the sums over its rows
//   S1 = sum dy * x^,   S0 = sum dy,
// from which segment_sums.cu forms every vector gradient.
//
// One pass over dy and x.  A CTA owns a contiguous share of rows, cut into
// runs of one (sample, modality).  Thread (tx, ty) owns vectors tx, tx + NT,
// ... of the rows of group ty: NT threads span a row, RG groups share the
// CTA.  Rows are staged by cp.async; a row's two sums are taken in one
// reduction (layer norm: g and g * (x - mean), from the saved statistics; RMS:
// x^2 and g * x, so nothing has to be saved), with one barrier per iteration
// of R rows per group, none if a warp spans the row.  After it the row is read
// from shared memory again rather than kept in registers, which hold W, S1 and
// S0 of the thread's channels for the whole run: fp32, added to in row order.
// At the end of a run the groups' sums are joined through shared memory and
// written to the CTA's workspace slot; no atomics, so results repeat.
//
// Bound by HBM: dy and x read, dx written, 3*D*esize bytes per row (4 with
// dres).  The partial sums are 8*D bytes per CTA and run.
#include "segment_sums.cuh"
#include "sol_device.cuh"

namespace sol {
namespace {

// Registers are capped so that two CTAs share an SM while a row takes at most
// two vectors per thread (up to 320 threads).
template <int VPT>
constexpr int kNormThreads = VPT <= 2 ? 320 : 512;
template <int VPT>
constexpr int kNormCtas = VPT <= 2 ? 2 : 1;

// S ring stages of R rows per group.
template <typename T, int VPT, bool RMS, bool DRES, int R, int S>
__global__ void __launch_bounds__(kNormThreads<VPT>, kNormCtas<VPT>)
    norm_backward_kernel(const NormBwdArgs a) {
  using IO = Io<T>;
  constexpr int P = IO::E / 2;
  constexpr int NIN = DRES ? 3 : 2;  // staged per row: x, dy, [dres]
  extern __shared__ __align__(16) unsigned char smem[];

  const int NT = blockDim.x, RG = blockDim.y;
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int tid = ty * NT + tx;
  const int NW = NT >> 5;
  const int lane = tx & 31, warp = tx >> 5;
  const int threads = NT * RG;
  float2 *red = reinterpret_cast<float2 *>(smem);  // [2][RG][NW][R]
  uint4 *ring = reinterpret_cast<uint4 *>(smem + ((2 * RG * NW * R * 8 + 15) & ~15));
  // ring: [S][R][NIN][VPT][threads]

  const int64_t row_bytes = static_cast<int64_t>(a.nvec) * 16;
  const unsigned char *src[3] = {static_cast<const unsigned char *>(a.x),
                                 static_cast<const unsigned char *>(a.dy),
                                 static_cast<const unsigned char *>(a.dres)};
  unsigned char *dxc = static_cast<unsigned char *>(a.dx);
  const float inv_D = 1.f / static_cast<float>(a.D);

  bool ok[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) ok[k] = k * NT + tx < a.nvec;
  auto slot = [&](int s, int q, int in, int k) -> uint4 * {
    return &ring[(((s * R + q) * NIN + in) * VPT + k) * threads + tid];
  };

  int buf = 0;  // which half of `red`
  int64_t row = share_begin(a.seg, blockIdx.x);
  const int64_t share_end = share_begin(a.seg, blockIdx.x + 1);
  while (row < share_end) {
    const int key = key_of(a.seg, row);
    int64_t run_end, unused;
    key_rows(a.seg, key, &unused, &run_end);
    if (run_end > share_end) run_end = share_end;
    const int count = static_cast<int>(run_end - row);
    const int step = RG * R;  // rows of one iteration: group ty takes R of them
    const int iters = (count + step - 1) / step;

    float2 W[VPT][P], s1[VPT][P], s0[VPT][P];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
#pragma unroll
      for (int m = 0; m < P; ++m) {
        W[k][m] = splat2(1.f);
        s1[k][m] = splat2(0.f);
        s0[k][m] = splat2(0.f);
      }
      if (ok[k]) {
        if (a.gamma)
          IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.gamma) + k * NT + tx), W[k]);
        if (a.scale) {
          float2 sc[P];
          IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.scale) +
                                   static_cast<int64_t>(key) * a.nvec + k * NT + tx),
                     sc);
#pragma unroll
          for (int m = 0; m < P; ++m) W[k][m] = mul2(W[k][m], add2(sc[m], splat2(1.f)));
        }
      }
    }

    auto issue = [&](int it, int s) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int j = it * step + ty * R + q;
        if (j < count) {
          const int64_t off = (row + j) * row_bytes + tx * 16;
#pragma unroll
          for (int in = 0; in < NIN; ++in)
#pragma unroll
            for (int k = 0; k < VPT; ++k)
              if (ok[k]) cp_async16(slot(s, q, in, k), src[in] + off + k * NT * 16);
        }
      }
      cp_async_commit();
    };
    // saved statistics of this group's rows of iteration `it`
    auto load_stats = [&](int it, float2 (&st)[R]) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int j = it * step + ty * R + q;
        st[q] = make_float2(0.f, 0.f);
        if (!RMS && j < count) st[q] = make_float2(__ldg(a.mean + row + j), __ldg(a.rstd + row + j));
      }
    };

#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s, s);
    float2 st[R], st_next[R];
    load_stats(0, st);

    int cons = 0;
    for (int it = 0; it < iters; ++it) {
      issue(it + S - 1, cons == 0 ? S - 1 : cons - 1);
      load_stats(it + 1, st_next);
      cp_async_wait<S - 1>();

      // the row's two sums: layer norm (g, g * (x - mean)), RMS (x^2, g * x)
      float2 sum[R];
#pragma unroll
      for (int q = 0; q < R; ++q) {
        float2 u = splat2(0.f), v = splat2(0.f);
        if (it * step + ty * R + q < count) {
          const float2 neg = splat2(-st[q].x);
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            if (ok[k]) {
              float2 x[P], d[P];
              IO::unpack(*slot(cons, q, 0, k), x);
              IO::unpack(*slot(cons, q, 1, k), d);
#pragma unroll
              for (int m = 0; m < P; ++m) {
                const float2 g = mul2(d[m], W[k][m]);
                if constexpr (RMS) {
                  u = fma2(x[m], x[m], u);
                  v = fma2(g, x[m], v);
                } else {
                  u = add2(g, u);
                  v = fma2(g, add2(x[m], neg), v);
                }
              }
            }
          }
        }
        sum[q] = make_float2(u.x + u.y, v.x + v.y);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          sum[q].x += __shfl_xor_sync(0xffffffffu, sum[q].x, o);
          sum[q].y += __shfl_xor_sync(0xffffffffu, sum[q].y, o);
        }
      }
      if (NW > 1) {
        float2 *r = red + (buf * RG + ty) * NW * R;
        if (lane == 0) {
#pragma unroll
          for (int q = 0; q < R; ++q) r[warp * R + q] = sum[q];
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < R; ++q) sum[q] = splat2(0.f);
        for (int w = 0; w < NW; ++w)
#pragma unroll
          for (int q = 0; q < R; ++q) sum[q] = add2(sum[q], r[w * R + q]);
        buf ^= 1;
      }

#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int j = it * step + ty * R + q;
        if (j < count) {
          // dx = rstd * g + a1 * (x - mean) + a0
          const float rstd = RMS ? rsqrtf(fmaf(sum[q].x, inv_D, a.eps)) : st[q].y;
          const float a1 = -rstd * rstd * rstd * sum[q].y * inv_D;
          const float a0 = RMS ? 0.f : -rstd * sum[q].x * inv_D;
          const float2 neg = splat2(-st[q].x), r2 = splat2(rstd), a12 = splat2(a1),
                       a02 = splat2(a0);
          uint4 *out = reinterpret_cast<uint4 *>(dxc + (row + j) * row_bytes) + tx;
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            if (ok[k]) {
              float2 x[P], d[P], o[P];
              IO::unpack(*slot(cons, q, 0, k), x);
              IO::unpack(*slot(cons, q, 1, k), d);
              if constexpr (DRES) IO::unpack(*slot(cons, q, 2, k), o);
#pragma unroll
              for (int m = 0; m < P; ++m) {
                if constexpr (!RMS) x[m] = add2(x[m], neg);
                s1[k][m] = fma2(mul2(x[m], r2), d[m], s1[k][m]);
                s0[k][m] = add2(s0[k][m], d[m]);
                const float2 base = DRES ? add2(o[m], a02) : a02;
                o[m] = fma2(mul2(d[m], W[k][m]), r2, fma2(x[m], a12, base));
              }
              st_stream16(out + k * NT, IO::pack(o));
            }
          }
        }
        st[q] = st_next[q];
      }
      cons = (cons + 1 == S) ? 0 : cons + 1;
    }
    cp_async_wait<0>();

    if (a.partial) {
      float *dst = a.partial + (blockIdx.x + static_cast<int64_t>(key)) * 2 * a.D;
      if (RG > 1) {
        // groups 1.. park their sums in the ring, group 0 adds them in order
        float2 *park = reinterpret_cast<float2 *>(ring);  // [2 * VPT * P][threads]
        __syncthreads();
        if (ty > 0) {
#pragma unroll
          for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int m = 0; m < P; ++m) {
              park[(k * P + m) * threads + tid] = s1[k][m];
              park[((VPT + k) * P + m) * threads + tid] = s0[k][m];
            }
        }
        __syncthreads();
        if (ty == 0) {
          for (int y = 1; y < RG; ++y)
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
              for (int m = 0; m < P; ++m) {
                s1[k][m] = add2(s1[k][m], park[(k * P + m) * threads + y * NT + tx]);
                s0[k][m] = add2(s0[k][m], park[((VPT + k) * P + m) * threads + y * NT + tx]);
              }
        }
        __syncthreads();  // the ring is free again
      }
      if (ty == 0) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          if (ok[k]) {
            float2 *p1 = reinterpret_cast<float2 *>(dst) + (k * NT + tx) * P;
            float2 *p0 = reinterpret_cast<float2 *>(dst + a.D) + (k * NT + tx) * P;
#pragma unroll
            for (int m = 0; m < P; ++m) {
              p1[m] = s1[k][m];
              p0[m] = s0[k][m];
            }
          }
        }
      }
    }
    row = run_end;
  }
}

template <typename T, int VPT, bool RMS, bool DRES>
cudaError_t launch_t(NormBwdArgs &a, cudaStream_t stream) {
  constexpr int R = VPT <= 2 ? 2 : 1, S = 2;  // wider rows: what shared memory holds
  const int NT = ((a.nvec + VPT - 1) / VPT + 31) / 32 * 32;
  const int RG = NT >= 256 ? 1 : 256 / NT;
  auto *kern = &norm_backward_kernel<T, VPT, RMS, DRES, R, S>;
  const size_t smem = ((2 * RG * (NT / 32) * R * 8 + 15) & ~15) +
                      static_cast<size_t>(S) * R * (DRES ? 3 : 2) * VPT * NT * RG * 16;
  const int per_sm =
      resident_blocks(reinterpret_cast<const void *>(kern), NT * RG, smem);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t ctas = static_cast<int64_t>(per_sm) * device_sms();
  if (ctas > kMaxSumCtas) ctas = kMaxSumCtas;
  const int64_t most = (a.seg.rows + RG - 1) / RG;  // a row per group at least
  if (ctas > most) ctas = most;
  a.seg.ctas = static_cast<int>(ctas);
  kern<<<static_cast<unsigned>(ctas), dim3(NT, RG), smem, stream>>>(a);
  return cudaGetLastError();
}

// One vector per thread up to 32 (a warp spans the row), two up to 640 (320
// threads), then as few as 512 threads can hold.
template <typename T, bool RMS, bool DRES>
cudaError_t dispatch(NormBwdArgs &a, cudaStream_t stream) {
  if (a.nvec <= 32) return launch_t<T, 1, RMS, DRES>(a, stream);
  if (a.nvec <= 640) return launch_t<T, 2, RMS, DRES>(a, stream);
  if (a.nvec <= 1536) return launch_t<T, 3, RMS, DRES>(a, stream);
  return launch_t<T, 4, RMS, DRES>(a, stream);
}

template <typename T>
cudaError_t dispatch_kind(NormBwdArgs &a, cudaStream_t stream) {
  if (a.rms)
    return a.dres ? dispatch<T, true, true>(a, stream) : dispatch<T, true, false>(a, stream);
  return a.dres ? dispatch<T, false, true>(a, stream) : dispatch<T, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_norm_backward(NormBwdArgs &a, int dtype, cudaStream_t stream) {
  return dtype == 0 ? dispatch_kind<float>(a, stream)
                    : dispatch_kind<__nv_bfloat16>(a, stream);
}

}  // namespace sol
