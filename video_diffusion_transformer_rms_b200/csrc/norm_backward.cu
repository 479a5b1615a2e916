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

// Sums of up to four values over the warp with six shuffles: after it lane 8i
// holds the sum of value i.  Each step sends the values that the partner keeps.
__device__ __forceinline__ float warp_sum4(float a, float b, float c, float d, int lane) {
  const bool hi = lane & 16, mid = lane & 8;
  float u = hi ? c : a, v = hi ? d : b;
  u += __shfl_xor_sync(0xffffffffu, hi ? a : c, 16);
  v += __shfl_xor_sync(0xffffffffu, hi ? b : d, 16);
  float w = mid ? v : u;
  w += __shfl_xor_sync(0xffffffffu, mid ? u : v, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}

// S ring stages of R (1 or 2) rows per group.  Each warp has a block of the
// ring to itself, its slots 512 bytes (a vector per lane) apart: every slot is
// a constant offset whatever the CTA's shape.
template <typename T, int VPT, bool RMS, bool DRES, bool FULL, int R, int S>
__global__ void __launch_bounds__(kNormThreads<VPT>, kNormCtas<VPT>)
    norm_backward_kernel(const NormBwdArgs a) {
  using IO = Io<T>;
  constexpr int P = IO::E / 2;
  constexpr int NIN = DRES ? 3 : 2;  // staged per row: x, dy, [dres]
  constexpr int STAGE = R * NIN * VPT;
  extern __shared__ __align__(16) unsigned char smem[];

  const int NT = blockDim.x, RG = blockDim.y;
  const int tx = threadIdx.x, ty = threadIdx.y;
  const int tid = ty * NT + tx;
  const int NW = NT >> 5;
  const int lane = tx & 31, warp = tx >> 5;
  const int threads = NT * RG;
  float4 *red = reinterpret_cast<float4 *>(smem);  // [2][RG][NW]: two sums of two rows
  uint4 *ring = reinterpret_cast<uint4 *>(red + 2 * RG * NW);  // [warp][S * STAGE][32]
  uint4 *mine = ring + (tid >> 5) * (S * STAGE * 32) + lane;

  const int64_t row_bytes = static_cast<int64_t>(a.nvec) * 16;
  const unsigned char *src[3] = {static_cast<const unsigned char *>(a.x),
                                 static_cast<const unsigned char *>(a.dy),
                                 static_cast<const unsigned char *>(a.dres)};
  unsigned char *dxc = static_cast<unsigned char *>(a.dx);
  const float inv_D = 1.f / static_cast<float>(a.D);

  // Only the last vector of a thread can lie past the row: the launcher's NT
  // has (VPT - 1) * NT <= nvec.
  const bool last = FULL || (VPT - 1) * NT + tx < a.nvec;
  auto ok = [&](int k) { return k < VPT - 1 || last; };
  auto slot = [&](int s, int q, int in, int k) -> uint4 * {
    return mine + (s * STAGE + (q * NIN + in) * VPT + k) * 32;
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
              if (ok(k)) cp_async16(slot(s, q, in, k), src[in] + off + k * NT * 16);
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

    float2 W[VPT][P], s1[VPT][P], s0[VPT][P];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
#pragma unroll
      for (int m = 0; m < P; ++m) {
        W[k][m] = splat2(1.f);
        s1[k][m] = splat2(0.f);
        s0[k][m] = splat2(0.f);
      }
      if (ok(k)) {
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

    int cons = 0;
    for (int it = 0; it < iters; ++it) {
      issue(it + S - 1, cons == 0 ? S - 1 : cons - 1);
      load_stats(it + 1, st_next);
      cp_async_wait<S - 1>();

      // the row's two sums: layer norm (g, g * (x - mean)), RMS (x^2, g * x); x -
      // mean is formed first, which loses nothing when they are close
      float2 sum[R];
#pragma unroll
      for (int q = 0; q < R; ++q) {
        float2 u = splat2(0.f), v = splat2(0.f);
        if (it * step + ty * R + q < count) {
          const float2 neg = splat2(-st[q].x);
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            if (ok(k)) {
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
      const float part = warp_sum4(sum[0].x, sum[0].y, sum[R - 1].x, sum[R - 1].y, lane);
      if (NW > 1) {
        float4 *r = red + (buf * RG + ty) * NW;
        if ((lane & 7) == 0) reinterpret_cast<float *>(r + warp)[lane >> 3] = part;
        __syncthreads();
        float2 t0 = splat2(0.f), t1 = splat2(0.f);
#pragma unroll 4
        for (int w = 0; w < NW; ++w) {
          const float4 v = r[w];
          t0 = add2(t0, make_float2(v.x, v.y));
          t1 = add2(t1, make_float2(v.z, v.w));
        }
        sum[0] = t0;
        if constexpr (R == 2) sum[1] = t1;
        buf ^= 1;
      } else {
        sum[0].x = __shfl_sync(0xffffffffu, part, 0);
        sum[0].y = __shfl_sync(0xffffffffu, part, 8);
        if constexpr (R == 2) {
          sum[1].x = __shfl_sync(0xffffffffu, part, 16);
          sum[1].y = __shfl_sync(0xffffffffu, part, 24);
        }
      }

#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int j = it * step + ty * R + q;
        if (j < count) {
          // dx = W * (rstd * dy) + a1 * (x - mean) + a0
          const float rstd = RMS ? rsqrtf(fmaf(sum[q].x, inv_D, a.eps)) : st[q].y;
          const float m2 = rstd * sum[q].y * inv_D;  // mean(g * x^)
          const float2 a1 = splat2(-rstd * m2 * rstd), a0 = splat2(-rstd * sum[q].x * inv_D);
          const float2 r2 = splat2(rstd), neg = splat2(-st[q].x);
          uint4 *out = reinterpret_cast<uint4 *>(dxc + (row + j) * row_bytes) + tx;
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            if (ok(k)) {
              float2 x[P], d[P], o[P];
              IO::unpack(*slot(cons, q, 0, k), x);
              IO::unpack(*slot(cons, q, 1, k), d);
              if constexpr (DRES) IO::unpack(*slot(cons, q, 2, k), o);
#pragma unroll
              for (int m = 0; m < P; ++m) {
                if constexpr (!RMS) x[m] = add2(x[m], neg);
                const float2 rd = mul2(d[m], r2);
                s1[k][m] = fma2(x[m], rd, s1[k][m]);
                s0[k][m] = add2(s0[k][m], d[m]);
                if constexpr (DRES) {
                  o[m] = fma2(x[m], a1, o[m]);
                  if constexpr (!RMS) o[m] = add2(o[m], a0);
                } else {
                  o[m] = RMS ? mul2(x[m], a1) : fma2(x[m], a1, a0);
                }
                o[m] = fma2(rd, W[k][m], o[m]);
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
          if (ok(k)) {
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

// Rows per group that a CTA takes at least: fewer would write more partial sums
// than the rows they come from.
constexpr int kNormMinRows = 4;

template <typename T, int VPT, bool RMS, bool DRES, bool FULL>
cudaError_t launch_full(NormBwdArgs &a, cudaStream_t stream) {
  // Rows per group and stages.  One row where a third input is staged (two
  // would leave shared memory for one CTA per SM) and in RMS (0.654 against
  // 0.678 ms for two at the 5 s clip; the layer norm 0.743 against 0.649 ms).
  // Three stages of one row, two where the rows come in pairs or with a third
  // input (RMS at the 5 s clip: 3 stages 0.625 ms, 4 0.629, 2 0.624 and slower at
  // 8,264 rows; layer norm of 60,000 rows of 4,096 fp32: 3 stages 0.483 ms, 2
  // 0.518).
  constexpr int R = VPT > 2 || DRES || RMS ? 1 : 2;
  constexpr int S = R == 2 || DRES ? 2 : 3;
  const int NT = ((a.nvec + VPT - 1) / VPT + 31) / 32 * 32;
  const int RG = NT >= 256 ? 1 : 256 / NT;
  auto *kern = &norm_backward_kernel<T, VPT, RMS, DRES, FULL, R, S>;
  const size_t smem = 2 * RG * (NT / 32) * 16 +
                      static_cast<size_t>(S) * R * (DRES ? 3 : 2) * VPT * NT * RG * 16;
  const int per_sm =
      resident_blocks(reinterpret_cast<const void *>(kern), NT * RG, smem);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t ctas = static_cast<int64_t>(per_sm) * device_sms();
  if (ctas > kMaxSumCtas) ctas = kMaxSumCtas;
  const int64_t most = (a.seg.rows + kNormMinRows * RG - 1) / (kNormMinRows * RG);
  if (ctas > most) ctas = most;
  cut_shares(&a.seg, ctas);
  kern<<<static_cast<unsigned>(ctas), dim3(NT, RG), smem, stream>>>(a);
  return cudaGetLastError();
}

// RMS rows that fill every thread's vectors take the unguarded instantiation
// (0.716 -> 0.672 ms at the 5 s clip); the layer norm was 2% slower with it.
template <typename T, int VPT, bool RMS, bool DRES>
cudaError_t launch_t(NormBwdArgs &a, cudaStream_t stream) {
  return RMS && a.nvec % (32 * VPT) == 0 ? launch_full<T, VPT, RMS, DRES, RMS>(a, stream)
                                         : launch_full<T, VPT, RMS, DRES, false>(a, stream);
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
