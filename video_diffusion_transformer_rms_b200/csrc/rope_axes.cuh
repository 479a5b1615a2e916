// Rotary positions with several axes at explicit position ids, optionally
// behind the per-head RMS norm of q and k, forward and backward:
//   forward   y = R(pos) n,  n = x * rstd * gamma (or n = x),
//             rstd = 1 / sqrt(mean(x^2) + eps) over the head's channels
//   backward  g = R(pos)^T dy;  without the norm dx = g; with it
//             dx = rstd * (gamma g - x^ mean(x^ gamma g)),  x^ = x * rstd,
//             dgamma = sum over rows and heads of g * x^
// where R(pos) turns pair i of the first rot_dim channels by the angle
// pos[axis_i] * freq_i and leaves the rest as they are.
//
// A CTA takes tiles of `tile_rows` token rows.  Its threads first compute the
// tile's angles, once for all q and k heads: the product in fp64, reduced to
// [-pi, pi] by a two-part 2 pi, then sin and cos of the fp32 rest, corrected
// to first order by what that rounding dropped.  cos and sin go to shared
// memory (two buffers, so one barrier per tile).  Then G consecutive lanes own
// one head vector at a time (16 bytes per lane; G is the next power of two,
// lanes past head_dim idle), U of them per pass in flight from global memory.
// A head's sums are G-lane shuffles.  Half-split pairs fetch their partner
// elements from the lane that holds them by shuffle.
//
// dgamma: each thread keeps fp32 sums of its channels over all its heads and
// rows; the CTA joins them in a fixed order and writes one partial row.
//
// Bound by HBM: forward and backward without the norm read and write every
// head once; the backward with the norm reads dy and x and writes dx.
#pragma once

#include <math.h>

#include "sol_device.cuh"
#include "sol_train.h"

namespace sol {
namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ uint4 ld_head16(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// cos and sin of pos * freq.
__device__ __forceinline__ float2 cos_sin(double pos, double freq) {
  const double ang = pos * freq;
  const double turns = rint(ang * 0.15915494309189533577);      // 1 / (2 pi)
  double r = fma(turns, -6.2831853071795862320, ang);           // 2 pi, upper part
  r = fma(turns, -2.4492935982947064e-16, r);                   // and the rest of it
  const float hi = static_cast<float>(r);
  const float lo = static_cast<float>(r - static_cast<double>(hi));
  float s, c;
  sincosf(hi, &s, &c);
  return make_float2(fmaf(-lo, s, c), fmaf(lo, c, s));
}

// N consecutive floats of a table row (N = 2 or a multiple of 4, aligned to
// 4 * min(N, 4) bytes).
template <int N>
__device__ __forceinline__ void ld_table(const float *p, float (&v)[N]) {
  if constexpr (N == 2) {
    const float2 t = *reinterpret_cast<const float2 *>(p);
    v[0] = t.x;
    v[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 t = *reinterpret_cast<const float4 *>(p + i);
      v[i] = t.x;
      v[i + 1] = t.y;
      v[i + 2] = t.z;
      v[i + 3] = t.w;
    }
  }
}

// MODE as RopeMode.  HALF: pair i = elements (i, i + rot_dim / 2), else
// (2i, 2i + 1).
template <typename T, int G, bool HALF, int MODE, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_axes_kernel(
    const __grid_constant__ RopeArgs a) {
  using IO = Io<T>;
  constexpr int E = IO::E, P = E / 2;
  constexpr bool NORM = MODE == kNormRotate || MODE == kNormRotateBack;
  constexpr bool BACK = MODE == kRotateBack || MODE == kNormRotateBack;
  constexpr bool DGAMMA = MODE == kNormRotateBack;
  constexpr int GROUPS = kRopeThreads / G;  // head vectors per pass
  extern __shared__ __align__(16) unsigned char smem[];

  const int tid = threadIdx.x;
  const int group = tid / G, gl = tid % G;
  const bool active = gl * E < a.head_dim;
  const int TR = a.tile_rows;
  // pairs of a table row: HALF one entry per rotary pair, else per element pair
  const int npairs = HALF ? a.rot_dim / 2 : a.head_dim / 2;
  const int pitch = (npairs + 3) & ~3;
  float *cosb = reinterpret_cast<float *>(smem);           // [2][TR][pitch]
  float *sinb = cosb + 2 * TR * pitch;                     // [2][TR][pitch]
  int64_t *offs = reinterpret_cast<int64_t *>(sinb + 2 * TR * pitch);  // [2][TR][6]

  // this lane's table column, and in a half-split head its partner lane and
  // which half it holds; lanes past rot_dim keep their elements, lanes past
  // head_dim read column 0 and store nothing
  int col = active ? gl * P : 0, partner = 0;
  bool second = false, turns = true;
  if constexpr (HALF) {
    const int half = a.rot_dim / 2, e0 = gl * E;
    turns = e0 < a.rot_dim;
    second = e0 >= half;
    col = turns ? (second ? e0 - half : e0) : 0;
    partner = turns ? (second ? gl - half / E : gl + half / E) : gl;
    partner += (tid & 31) - gl;
  }

  float2 gam[2][P];
  float2 dgam[2][P];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int m = 0; m < P; ++m) {
      gam[t][m] = splat2(1.f);
      dgam[t][m] = splat2(0.f);
    }
  if constexpr (NORM) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (a.gamma[t] && active)
        IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.gamma[t]) + gl), gam[t]);
  }

  // rotate v (elements gl*E .. of a head) by the angles of tile row `cs`;
  // BACK turns the other way
  auto rotate = [&](float2 (&v)[P], const float *cs, const float *sn) {
    if constexpr (HALF) {
      float2 w[P];
#pragma unroll
      for (int m = 0; m < P; ++m) {
        w[m].x = __shfl_sync(0xffffffffu, v[m].x, partner);
        w[m].y = __shfl_sync(0xffffffffu, v[m].y, partner);
      }
      // first: v cos - w sin; second: v cos + w sin
      const float2 sg = splat2((second != BACK) ? 1.f : -1.f);
      float c[E], s[E];
      ld_table(cs + col, c);
      ld_table(sn + col, s);
      if (turns) {
#pragma unroll
        for (int m = 0; m < P; ++m)
          v[m] = fma2(v[m], make_float2(c[2 * m], c[2 * m + 1]),
                      mul2(w[m], mul2(make_float2(s[2 * m], s[2 * m + 1]), sg)));
      }
    } else {
      float c[P], s[P];
      ld_table(cs + col, c);
      ld_table(sn + col, s);
#pragma unroll
      for (int m = 0; m < P; ++m) {
        const float x = v[m].x, y = v[m].y, t = BACK ? -s[m] : s[m];
        v[m].x = fmaf(x, c[m], -(y * t));
        v[m].y = fmaf(x, t, y * c[m]);
      }
    }
  };

  const int64_t tiles = (a.rows + TR - 1) / TR;
  int buf = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int64_t row0 = tile * TR;
    const int nrows = a.rows - row0 < TR ? static_cast<int>(a.rows - row0) : TR;
    float *cosr = cosb + buf * TR * pitch, *sinr = sinb + buf * TR * pitch;
    int64_t *off = offs + buf * TR * 6;

    for (int i = tid; i < nrows * npairs; i += kRopeThreads) {
      const int r = i / npairs, p = i - r * npairs;
      float2 cs = make_float2(1.f, 0.f);
      if (2 * p < a.rot_dim) {
        const unsigned row = static_cast<unsigned>(row0) + r, b = row / static_cast<unsigned>(a.L);
        const int64_t at = a.axis[p] * a.pos_stride_axis + b * a.pos_stride_b +
                           (row - b * static_cast<unsigned>(a.L));
        double pos;
        if (a.pos_type == SOL_POS_I32)
          pos = static_cast<double>(__ldg(static_cast<const int *>(a.pos) + at));
        else if (a.pos_type == SOL_POS_I64)
          pos = static_cast<double>(__ldg(static_cast<const long long *>(a.pos) + at));
        else
          pos = static_cast<double>(__ldg(static_cast<const float *>(a.pos) + at));
        cs = cos_sin(pos, a.freq[p]);
      }
      cosr[r * pitch + p] = cs.x;
      sinr[r * pitch + p] = cs.y;
    }
    for (int i = tid; i < nrows * 6; i += kRopeThreads) {
      const int r = i / 6, w = i - r * 6;
      const HeadsArg &h = w < 2 ? a.x[w] : (w < 4 ? a.g[w - 2] : a.out[w - 4]);
      const unsigned row = static_cast<unsigned>(row0) + r, b = row / static_cast<unsigned>(a.L);
      off[r * 6 + w] = b * h.sb + (row - b * static_cast<unsigned>(a.L)) * h.sr;
    }
    __syncthreads();

#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int heads = a.heads[t];
      const int items = nrows * heads;
      const unsigned char *xin = static_cast<const unsigned char *>(a.x[t].data) + gl * 16;
      const unsigned char *gin = static_cast<const unsigned char *>(a.g[t].data) + gl * 16;
      unsigned char *out = static_cast<unsigned char *>(a.out[t].data) + gl * 16;
      for (int base = group; base - group < items; base += GROUPS * U) {
        uint4 vx[U], vg[U];
        int row[U], head[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = base + u * GROUPS;
          row[u] = heads == 1 ? i
                              : static_cast<int>(__umulhi(static_cast<unsigned>(i), a.magic[t]));
          head[u] = i - row[u] * heads;
          vx[u] = make_uint4(0, 0, 0, 0);
          vg[u] = make_uint4(0, 0, 0, 0);
          if (i < items && active) {
            if constexpr (MODE != kRotateBack)
              vx[u] = ld_head16(xin + off[row[u] * 6 + t] + head[u] * a.x[t].sh);
            if constexpr (BACK)
              vg[u] = ld_head16(gin + off[row[u] * 6 + 2 + t] + head[u] * a.g[t].sh);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = base + u * GROUPS;
          const bool live = i < items;
          const int r = live ? row[u] : 0;
          const float *cs = cosr + r * pitch, *sn = sinr + r * pitch;
          float2 x[P], g[P];
          if constexpr (MODE != kRotateBack) IO::unpack(vx[u], x);
          if constexpr (BACK) {
            IO::unpack(vg[u], g);
            rotate(g, cs, sn);
          }
          if constexpr (NORM) {
            float2 sq = splat2(0.f), dot = splat2(0.f);
#pragma unroll
            for (int m = 0; m < P; ++m) {
              sq = fma2(x[m], x[m], sq);
              if constexpr (BACK) dot = fma2(mul2(x[m], gam[t][m]), g[m], dot);
            }
            float s = sq.x + sq.y, d = dot.x + dot.y;
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) {
              s += __shfl_xor_sync(0xffffffffu, s, o);
              if constexpr (BACK) d += __shfl_xor_sync(0xffffffffu, d, o);
            }
            const float rstd = rsqrtf(fmaf(s, a.inv_hd, a.eps));
            const float2 r2 = splat2(rstd);
            if constexpr (BACK) {
              // dx = rstd * (gamma g) - x * rstd^3 * mean(x gamma g)
              const float2 k2 = splat2(-rstd * rstd * rstd * d * a.inv_hd);
#pragma unroll
              for (int m = 0; m < P; ++m) {
                if (live) dgam[t][m] = fma2(g[m], mul2(x[m], r2), dgam[t][m]);
                g[m] = fma2(x[m], k2, mul2(mul2(gam[t][m], g[m]), r2));
              }
            } else {
#pragma unroll
              for (int m = 0; m < P; ++m) x[m] = mul2(mul2(x[m], r2), gam[t][m]);
            }
          }
          if constexpr (!BACK) rotate(x, cs, sn);
          if (live && active) {
            unsigned char *dst = out + off[r * 6 + 4 + t] + head[u] * a.out[t].sh;
            if constexpr (BACK)
              st_stream16(dst, IO::pack(g));
            else
              st_stream16(dst, IO::pack(x));
          }
        }
      }
    }
  }

  if constexpr (DGAMMA) {
    if (a.partial) {
      // [group][channel]: the groups' sums, added in order by one thread per
      // channel of q and k
      __syncthreads();
      float *park = reinterpret_cast<float *>(smem);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (active) {
#pragma unroll
          for (int m = 0; m < P; ++m)
            reinterpret_cast<float2 *>(park + group * a.head_dim + gl * E)[m] = dgam[t][m];
        }
        __syncthreads();
        for (int c = tid; c < a.head_dim; c += kRopeThreads) {
          float s = 0.f;
          for (int y = 0; y < GROUPS; ++y) s += park[y * a.head_dim + c];
          a.partial[(static_cast<int64_t>(blockIdx.x) * 2 + t) * a.head_dim + c] = s;
        }
        __syncthreads();
      }
    }
  }
}

template <typename T, int G, bool HALF, int MODE>
cudaError_t launch_t(RopeArgs &a, cudaStream_t stream, int *ctas) {
  constexpr int U = 4;
  constexpr int GROUPS = kRopeThreads / G;
  auto *kern = &rope_axes_kernel<T, G, HALF, MODE, U>;
  const int npairs = HALF ? a.rot_dim / 2 : a.head_dim / 2;
  const int pitch = (npairs + 3) & ~3;
  const int heads = a.heads[0] + a.heads[1];
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidConfiguration;
  // Rows per tile: one angle per thread at least, and enough heads for a full
  // pass of U vectors per thread; fewer while the rows would leave SMs idle.
  int tr = kRopeThreads / npairs;
  if (tr < 1) tr = 1;
  while (tr < 32 && tr * heads < GROUPS * U) tr *= 2;
  if (tr > 32) tr = 32;
  while (tr > 1 && (a.rows + tr - 1) / tr < 2 * sms) tr /= 2;
  a.tile_rows = tr;
  size_t smem = static_cast<size_t>(tr) * (4 * pitch * 4 + 2 * 6 * 8);
  const size_t park = static_cast<size_t>(GROUPS) * a.head_dim * 4;
  if (MODE == kNormRotateBack && a.partial && smem < park) smem = park;
  const int per_sm = resident_blocks(reinterpret_cast<const void *>(kern), kRopeThreads, smem);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t grid = static_cast<int64_t>(per_sm) * sms;
  const int64_t tiles = (a.rows + tr - 1) / tr;
  if (grid > tiles) grid = tiles;
  if (grid > kMaxRopeCtas) grid = kMaxRopeCtas;
  *ctas = static_cast<int>(grid);
  kern<<<static_cast<unsigned>(grid), kRopeThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, bool HALF, int MODE>
cudaError_t dispatch_lanes(RopeArgs &a, cudaStream_t stream, int *ctas) {
  const int lanes = a.head_dim / Io<T>::E;
  if (lanes <= 2) return launch_t<T, 2, HALF, MODE>(a, stream, ctas);
  if (lanes <= 4) return launch_t<T, 4, HALF, MODE>(a, stream, ctas);
  if (lanes <= 8) return launch_t<T, 8, HALF, MODE>(a, stream, ctas);
  if (lanes <= 16) return launch_t<T, 16, HALF, MODE>(a, stream, ctas);
  if (lanes <= 32) return launch_t<T, 32, HALF, MODE>(a, stream, ctas);
  return cudaErrorInvalidValue;
}

template <typename T, bool HALF>
cudaError_t dispatch_mode(RopeArgs &a, RopeMode mode, cudaStream_t stream, int *ctas) {
  switch (mode) {
    case kRotate: return dispatch_lanes<T, HALF, kRotate>(a, stream, ctas);
    case kNormRotate: return dispatch_lanes<T, HALF, kNormRotate>(a, stream, ctas);
    case kRotateBack: return dispatch_lanes<T, HALF, kRotateBack>(a, stream, ctas);
    case kNormRotateBack: return dispatch_lanes<T, HALF, kNormRotateBack>(a, stream, ctas);
  }
  return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace sol
