// Rotary positions with several axes at explicit position ids, optionally
// behind the per-head RMS norm of q and k, forward and backward:
//   forward   y = R(pos) n,  n = x * rstd * gamma (or n = x),
//             rstd = 1 / sqrt(mean(x^2) + eps) over the head's channels
//   backward  g = R(pos)^T dy;  without the norm dx = g; with it
//             dx = rstd * (gamma g - x^ mean(x^ gamma g)),  x^ = x * rstd,
//             dgamma = sum over rows and heads of g * x^
// where R(pos) turns pair i of the first rot_dim channels by the angle
// pos[axis_i] * freq_i and leaves the rest as they are: copied bit for bit without
// the norm, multiplied by nothing but rstd * gamma with it.  (A turn by 0 is not
// that: Inf * 0 is NaN, and would reach the channel's neighbour too.)
//
// A warp owns a token row, as long as there is one for every warp of the grid;
// the rows left after the last whole round are shared by WR warps each, so the
// round they make is shorter.  A warp's lanes first compute the row's angles, a
// few rotary pairs each, once for all q and k heads: the product in fp64, reduced
// to [-pi, pi] by a two-part 2 pi, then sin and cos of the fp32 rest, corrected
// to first order by what that rounding dropped.  They meet in the warp's own
// shared memory, so nothing waits for another warp.  Then G consecutive lanes
// own one head vector at a time (16 bytes per lane; G is the next power of two,
// lanes past head_dim idle).  A lane sees the same channels in every head: its cos and sin, with
// gamma folded in, stay in registers for the row.  Several vectors per lane are
// in flight: as a batch of loads into registers, or, in the norm's backward
// pass, which needs the registers for its sums and two vectors per head, through
// a ring in shared memory that cp.async fills across the ends of q, of k and of
// rows.  A head's sums are G-lane shuffles, and 1/rms one factor at the end.
// Half-split pairs fetch their partner channels as raw 32-bit words from the
// lane that holds them.
//
// dgamma: each lane keeps fp32 sums of its channels over all its heads and
// rows (a row's in registers, added to shared memory once a row); the CTA joins
// them in a fixed order and writes one partial row.
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

__device__ __forceinline__ float2 and2(float2 v, uint32_t x, uint32_t y) {
  return make_float2(__uint_as_float(__float_as_uint(v.x) & x),
                     __uint_as_float(__float_as_uint(v.y) & y));
}

// cos and sin of pos * freq.  (Reduced to a part of a turn and sincospif: 3 to
// 11% slower in calls of few rows, which wait for the angles.)
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

// CTAs per SM that the registers are to leave room for: 80 registers a thread,
// 128 in the norm's backward pass.  5 s clip, 40 + 40 heads of 128 in bf16:
// forward with the norm 0.83 ms (64 registers: 0.87), backward 1.23 ms (80
// registers spill: 2.38 with a ring of single heads, 1.29 without).
template <int MODE>
constexpr int kRopeMinCtas = MODE == kNormRotateBack ? 2 : 3;
// Depth of the loads in flight: vectors per lane, or in the norm's backward pass
// ring entries of kRopeEntry heads each, which spread the ring's bookkeeping.
// Under the power cap (5 s clip, half-split / interleaved): 2 entries of 4 heads
// 1.365 / 1.314 ms, of 5 1.367 / 1.312, 3 of 3 1.393 / 1.332, 4 of 2 1.395 / -.
template <int MODE>
constexpr int kRopeDepth = MODE == kNormRotateBack ? 2 : 4;
constexpr int kRopeEntry = 4;

// MODE as RopeMode.  HALF: pair i = channels (i, i + rot_dim / 2), else
// (2i, 2i + 1).  PART: rot_dim < head_dim; a form of its own, as full rotations
// need no masks (5 s clip, 96 of 128 channels turned, with masks / turned by 0
// instead: forward with the norm 0.878 / 0.837 ms, half-split 0.902 / 0.874; its
// gradient and the forms without the norm take the same time).  The rows from whole_rows on are shared by 2^tail_log2 warps.
template <typename T, int G, bool HALF, int MODE, bool PART, int D>
__global__ void __launch_bounds__(kRopeThreads, kRopeMinCtas<MODE>)
    rope_axes_kernel(const __grid_constant__ RopeArgs a, int whole_rows, int tail_log2) {
  using IO = Io<T>;
  constexpr int E = IO::E, P = E / 2;
  constexpr bool NORM = MODE == kNormRotate || MODE == kNormRotateBack;
  constexpr bool BACK = MODE == kRotateBack || MODE == kNormRotateBack;
  constexpr bool DGAMMA = MODE == kNormRotateBack;
  constexpr int RV = kRopeEntry;
  constexpr int GW = 32 / G;                          // heads a warp holds at a time
  constexpr int NPL = G * E / 64 > 0 ? G * E / 64 : 1;  // rotary pairs per lane, at most
  constexpr int GROUPS = kRopeThreads / G;
  extern __shared__ __align__(16) unsigned char smem[];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gl = tid % G;
  const bool active = gl * E < a.head_dim;
  const int half = a.rot_dim / 2;
  // norm's backward pass: the ring (x and dy) and the lanes' dgamma sums; then
  // each warp's cos and sin, one entry per pair (interleaved: identity pairs past
  // rot_dim)
  constexpr int PITCH = G * P;
  uint4 *ring = reinterpret_cast<uint4 *>(smem) + tid;                   // [D][2 RV][threads]
  float2 *sums = reinterpret_cast<float2 *>(smem + (DGAMMA ? D * 2 * RV * kRopeThreads * 16 : 0));
  float *cosw = reinterpret_cast<float *>(sums + (DGAMMA ? 2 * P * kRopeThreads : 0)) +
                warp * 2 * PITCH;
  float *sinw = cosw + PITCH;
  if constexpr (DGAMMA) {
#pragma unroll
    for (int m = 0; m < 2 * P; ++m) sums[m * kRopeThreads + tid] = splat2(0.f);  // [t][m][thread]
  }

  // this lane's first table column; half-split: the lane that holds the partner
  // channels, and whether the lane's channels are the second of their pairs
  int col = active ? gl * P : 0, partner = lane;
  bool second = false, turns = true;
  if constexpr (HALF) {
    const int e0 = gl * E;
    turns = e0 < a.rot_dim;
    second = turns && e0 >= half;
    col = turns ? (second ? e0 - half : e0) : 0;
    if (turns) partner = second ? lane - half / E : lane + half / E;
  }
  // PART: all ones for the pairs that are turned (half-split: for the vector), 0 for
  // the others, whose cross terms are masked away
  uint32_t keep[P];
#pragma unroll
  for (int i = 0; i < P; ++i) keep[i] = (HALF ? turns : gl * P + i < half) ? 0xffffffffu : 0u;

  // frequency and position array of the pairs this lane computes
  double freq[NPL];
  int64_t axis_off[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int p = lane + 32 * i;
    freq[i] = p < half ? a.freq[p] : 0.0;
    axis_off[i] = p < half ? a.axis[p] * a.pos_stride_axis : 0;
  }
  auto load_pos = [&](int64_t row, double (&pos)[NPL]) {
    const unsigned b = static_cast<unsigned>(row) / static_cast<unsigned>(a.L);
    const int64_t at =
        b * a.pos_stride_b + (static_cast<unsigned>(row) - b * static_cast<unsigned>(a.L));
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      if (a.pos_type == SOL_POS_I32)
        pos[i] = static_cast<double>(__ldg(static_cast<const int *>(a.pos) + at + axis_off[i]));
      else if (a.pos_type == SOL_POS_I64)
        pos[i] =
            static_cast<double>(__ldg(static_cast<const long long *>(a.pos) + at + axis_off[i]));
      else
        pos[i] = static_cast<double>(__ldg(static_cast<const float *>(a.pos) + at + axis_off[i]));
    }
  };
  // identity entries past rot_dim are written once
  if constexpr (!HALF && PART) {
    for (int p = half + lane; p < PITCH; p += 32) {
      cosw[p] = 1.f;
      sinw[p] = 0.f;
    }
  }

  for (int phase = 0; phase < 2; ++phase) {
    const int wr_log2 = phase == 0 ? 0 : tail_log2, WR = 1 << wr_log2;
    const int rpb = (kRopeThreads / 32) >> wr_log2;            // rows of a CTA at a time
    const int slot0 = (warp & (WR - 1)) * GW, step = WR * GW;  // heads slot0 + lane / G + i * step
    const int slot = slot0 + lane / G;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * rpb;
    const int64_t end = phase == 0 ? whole_rows : a.rows;
    int64_t row = (phase == 0 ? 0 : whole_rows) + static_cast<int64_t>(blockIdx.x) * rpb +
                  (warp >> wr_log2);
    // passes over the heads of q and of k
    const int passes_q = a.heads[0] > slot0 ? (a.heads[0] - slot0 + step - 1) / step : 0;
    const int passes_k = a.heads[1] > slot0 ? (a.heads[1] - slot0 + step - 1) / step : 0;
    if (passes_q + passes_k == 0) row = end;  // more warps than heads: none for this one

    // The ring's producer: it walks the same rows, tensors and passes as the loop
    // below, D - 1 entries of up to RV heads ahead.
    int64_t prow = row;
    int pt = passes_q > 0 ? 0 : 1, phead = slot, pleft = 0, pslot = 0, cons = 0;
    const unsigned char *px = nullptr, *pg = nullptr;
    auto seek = [&]() {
      const unsigned b = static_cast<unsigned>(prow) / static_cast<unsigned>(a.L);
      const unsigned r = static_cast<unsigned>(prow) - b * static_cast<unsigned>(a.L);
      phead = slot;
      pleft = pt == 0 ? passes_q : passes_k;
      px = static_cast<const unsigned char *>(a.x[pt].data) +
           (b * a.x[pt].sb + r * a.x[pt].sr + slot * a.x[pt].sh) + gl * 16;
      pg = static_cast<const unsigned char *>(a.g[pt].data) +
           (b * a.g[pt].sb + r * a.g[pt].sr + slot * a.g[pt].sh) + gl * 16;
    };
    auto produce = [&]() {
      if (prow < end) {
        const int64_t xstep = a.x[pt].sh * step, gstep = a.g[pt].sh * step;
        uint4 *dst = ring + pslot * (2 * RV * kRopeThreads);
#pragma unroll
        for (int u = 0; u < RV; ++u) {
          if (active && phead + u * step < a.heads[pt]) {
            cp_async16(dst + 2 * u * kRopeThreads, px + u * xstep);
            cp_async16(dst + (2 * u + 1) * kRopeThreads, pg + u * gstep);
          }
        }
        phead += RV * step;
        px += RV * xstep;
        pg += RV * gstep;
        pleft -= RV;
        if (pleft <= 0) {
          if (pt == 0 && passes_k > 0) {
            pt = 1;
          } else {
            pt = passes_q > 0 ? 0 : 1;
            prow += stride;
          }
          if (prow < end) seek();
        }
      }
      cp_async_commit();
      pslot = pslot + 1 == D ? 0 : pslot + 1;
    };
    if constexpr (DGAMMA) {
      if (prow < end) seek();
#pragma unroll
      for (int i = 0; i < D - 1; ++i) produce();
    }

    double pos[NPL];
    if (row < end) load_pos(row, pos);
    for (; row < end; row += stride) {
      const unsigned b = static_cast<unsigned>(row) / static_cast<unsigned>(a.L);
      const unsigned r = static_cast<unsigned>(row) - b * static_cast<unsigned>(a.L);
      __syncwarp();  // every lane has read the previous row's table
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int p = lane + 32 * i;
        if (p < half) {
          const float2 cs = cos_sin(pos[i], freq[i]);
          cosw[p] = cs.x;
          sinw[p] = cs.y;
        }
      }
      __syncwarp();
      if (row + stride < end) load_pos(row + stride, pos);

#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int passes = t == 0 ? passes_q : passes_k;
        if (passes == 0) continue;
        float2 dg[P];  // this row's part of dgam[t]
#pragma unroll
        for (int m = 0; m < P; ++m) dg[m] = splat2(0.f);
        // cos, sin and gamma of the lane's channels (gp: its partner channels)
        float2 c[P], s[P], gam[P], gp[P];
#pragma unroll
        for (int m = 0; m < P; ++m) gam[m] = gp[m] = splat2(1.f);
        if constexpr (NORM) {
          if (a.gamma[t]) {
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (active) raw = ld_shared_vec(static_cast<const uint4 *>(a.gamma[t]) + gl);
            uint4 rp = raw;
            if constexpr (HALF && !BACK) {
              rp.x = __shfl_sync(0xffffffffu, raw.x, partner);
              rp.y = __shfl_sync(0xffffffffu, raw.y, partner);
              rp.z = __shfl_sync(0xffffffffu, raw.z, partner);
              rp.w = __shfl_sync(0xffffffffu, raw.w, partner);
            }
            IO::unpack(raw, gam);
            IO::unpack(rp, gp);
          }
        }
        // the turn of one component pair (u, v) held as A, B:
        //   interleaved forward   even = e A - o B,  odd = e C + o D
        //   interleaved backward  even = e c + o s,  odd = o c - e s
        //   half-split            out = own A + partner B
        float2 A[P], B[P];
        if constexpr (HALF) {
#pragma unroll
          for (int m = 0; m < P; ++m) {
            c[m] = turns ? *reinterpret_cast<const float2 *>(cosw + col + 2 * m) : splat2(1.f);
            s[m] = turns ? *reinterpret_cast<const float2 *>(sinw + col + 2 * m) : splat2(0.f);
            const float sg = (second != BACK) ? 1.f : -1.f;
            A[m] = BACK ? c[m] : mul2(c[m], gam[m]);
            B[m] = mul2(s[m], splat2(sg));
            if constexpr (!BACK) B[m] = mul2(B[m], gp[m]);
            if constexpr (PART) B[m] = and2(B[m], keep[0], keep[0]);  // gp may be Inf
          }
        } else {
          // entry m: pairs 2m and 2m + 1 of the lane; first P/2 entries of A, B for
          // the even outputs, the others for the odd ones
#pragma unroll
          for (int m = 0; m < P / 2; ++m) {
            c[m] = *reinterpret_cast<const float2 *>(cosw + col + 2 * m);
            s[m] = *reinterpret_cast<const float2 *>(sinw + col + 2 * m);
            const float2 ge = make_float2(gam[2 * m].x, gam[2 * m + 1].x);
            const float2 go = make_float2(gam[2 * m].y, gam[2 * m + 1].y);
            if constexpr (BACK) {
              A[m] = c[m];
              B[m] = s[m];
            } else {
              A[m] = mul2(c[m], ge);                              // even from even
              B[m] = mul2(mul2(s[m], go), splat2(-1.f));          // even from odd
              A[m + P / 2] = mul2(c[m], go);                      // odd from odd
              B[m + P / 2] = mul2(s[m], ge);                      // odd from even
              if constexpr (PART) {  // ge and go may be Inf
                B[m] = and2(B[m], keep[2 * m], keep[2 * m + 1]);
                B[m + P / 2] = and2(B[m + P / 2], keep[2 * m], keep[2 * m + 1]);
              }
            }
            gam[2 * m] = ge;  // kept in the same split as the channels
            gam[2 * m + 1] = go;
          }
        }

        // one head vector (dy with it in the norm's backward pass) to dst
        auto turn = [&](uint4 vx, uint4 vg, bool live, unsigned char *dst) {
          // v: the vector that is turned; o: the turned one
          const uint4 v = BACK ? vg : vx;
          float2 o[P];
          if constexpr (HALF) {
            uint4 vp;
            vp.x = __shfl_sync(0xffffffffu, v.x, partner);
            vp.y = __shfl_sync(0xffffffffu, v.y, partner);
            vp.z = __shfl_sync(0xffffffffu, v.z, partner);
            vp.w = __shfl_sync(0xffffffffu, v.w, partner);
            if constexpr (PART && NORM)
              vp = make_uint4(vp.x & keep[0], vp.y & keep[0], vp.z & keep[0], vp.w & keep[0]);
            float2 own[P], oth[P];
            IO::unpack(v, own);
            IO::unpack(vp, oth);
#pragma unroll
            for (int m = 0; m < P; ++m) o[m] = fma2(own[m], A[m], mul2(oth[m], B[m]));
          } else {
            float2 ev[P / 2], od[P / 2];
            IO::unpack_eo(v, ev, od);
#pragma unroll
            for (int m = 0; m < P / 2; ++m) {
              float2 ex = ev[m], ox = od[m];  // what crosses over to the other component
              if constexpr (PART && NORM) {
                ex = and2(ex, keep[2 * m], keep[2 * m + 1]);
                ox = and2(ox, keep[2 * m], keep[2 * m + 1]);
              }
              if constexpr (BACK) {
                const float2 neg = mul2(B[m], splat2(-1.f));
                o[2 * m] = fma2(ev[m], A[m], mul2(ox, B[m]));
                o[2 * m + 1] = fma2(od[m], A[m], mul2(ex, neg));
              } else {
                o[2 * m] = fma2(ev[m], A[m], mul2(ox, B[m]));
                o[2 * m + 1] = fma2(od[m], A[m + P / 2], mul2(ex, B[m + P / 2]));
              }
            }
          }
          if constexpr (NORM) {
            float2 x[P];
            if constexpr (HALF) {
              IO::unpack(vx, x);
            } else {
              float2 ev[P / 2], od[P / 2];
              IO::unpack_eo(vx, ev, od);
#pragma unroll
              for (int m = 0; m < P / 2; ++m) {
                x[2 * m] = ev[m];
                x[2 * m + 1] = od[m];
              }
            }
            float2 sq = splat2(0.f), dot = splat2(0.f), h[P];
#pragma unroll
            for (int m = 0; m < P; ++m) {
              sq = fma2(x[m], x[m], sq);
              if constexpr (BACK) {
                h[m] = mul2(o[m], gam[m]);
                dot = fma2(h[m], x[m], dot);
              }
            }
            float ss = sq.x + sq.y, d = dot.x + dot.y;
#pragma unroll
            for (int w = G / 2; w > 0; w >>= 1) {
              ss += __shfl_xor_sync(0xffffffffu, ss, w);
              if constexpr (BACK) d += __shfl_xor_sync(0xffffffffu, d, w);
            }
            const float rstd = rsqrtf(fmaf(ss, a.inv_hd, a.eps));
            const float2 r2 = splat2(rstd);
            if constexpr (BACK) {
              // x^ = x rstd;  dx = rstd (h - x^ mean(x^ h))
              const float2 k2 = splat2(-rstd * rstd * d * a.inv_hd);
#pragma unroll
              for (int m = 0; m < P; ++m) {
                x[m] = mul2(x[m], r2);
                if (live) dg[m] = fma2(o[m], x[m], dg[m]);
                o[m] = fma2(x[m], k2, mul2(h[m], r2));
              }
            } else {
#pragma unroll
              for (int m = 0; m < P; ++m) o[m] = mul2(o[m], r2);
            }
          }
          if (live) {
            uint4 res;
            if constexpr (HALF) {
              res = IO::pack(o);
            } else {
              float2 ev[P / 2], od[P / 2];
#pragma unroll
              for (int m = 0; m < P / 2; ++m) {
                ev[m] = o[2 * m];
                od[m] = o[2 * m + 1];
              }
              res = IO::pack_eo(ev, od);
            }
            if constexpr (PART && !NORM) {
              // the words of unturned channels as they were read; a pair is one
              // 32-bit word in bf16, two in fp32
              constexpr int W = sizeof(T) / 2;  // words of a pair
              res.x = keep[0] ? res.x : v.x;
              res.y = keep[1 / W] ? res.y : v.y;
              res.z = keep[2 / W] ? res.z : v.z;
              res.w = keep[3 / W] ? res.w : v.w;
            }
            st_stream16(dst, res);
          }
        };
        unsigned char *out = static_cast<unsigned char *>(a.out[t].data) +
                             (b * a.out[t].sb + r * a.out[t].sr + slot * a.out[t].sh) + gl * 16;
        const int64_t ostep = a.out[t].sh * step;
        int head = slot;
        if constexpr (DGAMMA) {
#pragma unroll 1
          for (int i = 0; i < passes; i += RV, head += RV * step, out += RV * ostep) {
            produce();
            cp_async_wait<D - 1>();
            const uint4 *entry = ring + cons * (2 * RV * kRopeThreads);
            cons = cons + 1 == D ? 0 : cons + 1;
#pragma unroll
            for (int u = 0; u < RV; ++u) {
              if (i + u < passes) {  // the same for the whole warp
                const bool live = active && head + u * step < a.heads[t];
                uint4 vx = make_uint4(0, 0, 0, 0), vg = make_uint4(0, 0, 0, 0);
                if (live) {
                  vx = entry[2 * u * kRopeThreads];
                  vg = entry[(2 * u + 1) * kRopeThreads];
                }
                turn(vx, vg, live, out + u * ostep);
              }
            }
          }
        } else {
          const HeadsArg &in = BACK ? a.g[t] : a.x[t];
          const unsigned char *src = static_cast<const unsigned char *>(in.data) +
                                     (b * in.sb + r * in.sr + slot * in.sh) + gl * 16;
          const int64_t istep = in.sh * step;
          for (int i = 0; i < passes; i += D, head += D * step) {
            uint4 v[D];
#pragma unroll
            for (int u = 0; u < D; ++u) {
              v[u] = make_uint4(0, 0, 0, 0);
              if (active && head + u * step < a.heads[t]) v[u] = ld_head16(src + u * istep);
            }
            src += D * istep;
#pragma unroll
            for (int u = 0; u < D; ++u)
              if (i + u < passes)  // the same for the whole warp
                turn(v[u], v[u], active && head + u * step < a.heads[t], out + u * ostep);
            out += D * ostep;
          }
        }
        if constexpr (DGAMMA) {
#pragma unroll
          for (int m = 0; m < P; ++m) {
            float2 *sum = sums + (t * P + m) * kRopeThreads + tid;
            *sum = add2(*sum, dg[m]);
          }
        }
      }
    }
    if constexpr (DGAMMA) cp_async_wait<0>();
  }

  if constexpr (DGAMMA) {
    if (a.partial) {
      // channel c of q and k: the groups' sums, added in order by one thread
      __syncthreads();
      for (int i = tid; i < 2 * a.head_dim; i += kRopeThreads) {
        const int t = i >= a.head_dim ? 1 : 0, c = i - t * a.head_dim;
        // where the lane of channel c keeps it: float2 entry and component
        const int e = c % E;
        const int m = HALF ? e / 2 : 2 * (e / 4) + (e & 1);
        const int comp = HALF ? e & 1 : (e / 2) & 1;
        const float2 *p = sums + (t * P + m) * kRopeThreads + c / E;
        float s = 0.f;
        for (int y = 0; y < GROUPS; ++y) s += comp ? p[y * G].y : p[y * G].x;
        a.partial[(static_cast<int64_t>(blockIdx.x) * 2 + t) * a.head_dim + c] = s;
      }
    }
  }
}

template <typename T, int G, bool HALF, int MODE, bool PART>
cudaError_t launch_t(RopeArgs &a, cudaStream_t stream, int *ctas) {
  constexpr bool DGAMMA = MODE == kNormRotateBack;
  constexpr int D = kRopeDepth<MODE>;
  constexpr int GW = 32 / G, WARPS = kRopeThreads / 32;
  auto *kern = &rope_axes_kernel<T, G, HALF, MODE, PART, D>;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidConfiguration;
  constexpr int PITCH = G * Io<T>::E / 2;
  const size_t ring = static_cast<size_t>(kRopeThreads) * (D * kRopeEntry * 32 + Io<T>::E * 8);
  const size_t smem = (DGAMMA ? ring : 0) +
                      static_cast<size_t>(WARPS) * 2 * PITCH * 4;
  const int per_sm = resident_blocks(reinterpret_cast<const void *>(kern), kRopeThreads, smem);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t grid = static_cast<int64_t>(per_sm) * sms;
  if (grid > kMaxRopeCtas) grid = kMaxRopeCtas;
  const int64_t warps = grid * WARPS, whole = a.rows / warps * warps, tail = a.rows - whole;
  const int heads = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
  int wr = 0;
  while ((1 << wr) < WARPS && (GW << wr) < heads && (tail << (wr + 1)) <= warps) ++wr;
  if (whole == 0) grid = ((tail << wr) + WARPS - 1) / WARPS;
  *ctas = static_cast<int>(grid);
  kern<<<static_cast<unsigned>(grid), kRopeThreads, smem, stream>>>(a, static_cast<int>(whole),
                                                                   wr);
  return cudaGetLastError();
}

template <typename T, int G, bool HALF, int MODE>
cudaError_t dispatch_part(RopeArgs &a, cudaStream_t stream, int *ctas) {
  return a.rot_dim < a.head_dim ? launch_t<T, G, HALF, MODE, true>(a, stream, ctas)
                                : launch_t<T, G, HALF, MODE, false>(a, stream, ctas);
}

template <typename T, bool HALF, int MODE>
cudaError_t dispatch_lanes(RopeArgs &a, cudaStream_t stream, int *ctas) {
  const int lanes = a.head_dim / Io<T>::E;
  if (lanes <= 2) return dispatch_part<T, 2, HALF, MODE>(a, stream, ctas);
  if (lanes <= 4) return dispatch_part<T, 4, HALF, MODE>(a, stream, ctas);
  if (lanes <= 8) return dispatch_part<T, 8, HALF, MODE>(a, stream, ctas);
  if (lanes <= 16) return dispatch_part<T, 16, HALF, MODE>(a, stream, ctas);
  if (lanes <= 32) return dispatch_part<T, 32, HALF, MODE>(a, stream, ctas);
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
