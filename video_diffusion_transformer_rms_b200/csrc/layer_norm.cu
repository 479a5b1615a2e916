// Layer norm with optional weight, bias and adaptive modulation:
//   n = (x - mean) * rstd * gamma + beta,  rstd = 1 / sqrt(var + eps),
//   y = n * (1 + scale[b][m]) + shift[b][m]
// per token row, m = video/audio modality of the row.  Per channel this is
// y = (x - mean) * rstd * fac + off with fac = gamma * (1 + scale) and
// off = beta * (1 + scale) + shift, both kept in fp32 registers and rebuilt
// only when a CTA crosses a modality or sample boundary.
//
// The same persistent cp.async ring as RMS-AdaLN: chunks of rows dealt
// round-robin over the CTAs, a row per iteration, compile-time CTA size and
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

// A staged vector, read from shared memory at every use.
__device__ __forceinline__ uint4 ld_staged(const uint4 *p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p))
               : "memory");
  return v;
}

// Threads per SM that the registers are to leave room for: 128 registers a
// thread while its vectors fit them (102: 0.75 ms at the 5 s clip, spilled).
template <int VPT>
constexpr int kLnThreadsPerSm = VPT <= 5 ? 512 : 256;

// A row of up to four vectors per thread stays in registers across the two
// reductions; a wider one is read from shared memory again for each.  5 s clip in
// short runs / in long ones under the power cap, 8,264 rows: 160 x 4 held 0.405 /
// 0.426 ms, 32.5 us; 128 x 5 read again 0.422 / 0.421 ms, 34.6 us.  (Held, 128 x 5
// takes 252 registers: 0.469 ms.)
constexpr int kLnHeld = 4;

// FULL: the split covers the row exactly, no access needs a guard.
template <typename T, int NT, int VPT, int S, int K, bool FULL>
__global__ void __launch_bounds__(NT, kLnThreadsPerSm<VPT> / NT < 16 ? kLnThreadsPerSm<VPT> / NT : 16)
    layer_norm_kernel(const LnArgs a) {
  using IO = Io<T>;
  constexpr int P = IO::E / 2;
  constexpr int NW = NT / 32;
  constexpr bool HOLD = VPT <= kLnHeld;
  extern __shared__ __align__(16) unsigned char smem[];
  float4 *red = reinterpret_cast<float4 *>(smem);               // [2][NW]: sum, M2, mean, n
  uint4 *ring = reinterpret_cast<uint4 *>(smem + 2 * NW * 16);  // [S][VPT][NT]

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

  RowOrder<K> ro;
  ro.init(a.rows);
  const int count = ro.count;
  const unsigned char *xc = static_cast<const unsigned char *>(a.x);
  unsigned char *yc = static_cast<unsigned char *>(a.y);

  auto slot = [&](int s, int k) -> uint4 * { return &ring[(s * VPT + k) * NT + tid]; };
  auto issue = [&](int j, int s) {
    if (j < count) {
      const uint4 *src = reinterpret_cast<const uint4 *>(xc + ro.row(j) * row_bytes) + tid;
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (ok[k]) cp_async16(slot(s, k), src + k * NT);
    }
    cp_async_commit();
  };

#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(s, s);

  float2 fac[VPT][P], off[VPT][P];
  int key = -1;
  int cons = 0;
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

  for (int j = 0; j < count; ++j) {
    issue(j + S - 1, cons == 0 ? S - 1 : cons - 1);
    const int64_t row = ro.row(j);
    if (ro.run_start(j)) cur.init(row, a.L);
    const int nkey = 2 * cur.b + (cur.r >= a.n_video ? 1 : 0);
    if (nkey != key) {  // a modality or sample boundary: rebuild the vectors
      key = nkey;
      load_vectors();
    }
    cp_async_wait<S - 1>();

    float2 held[HOLD ? VPT : 1][P];
    auto channels = [&](int k, float2 (&x)[P]) {
      if constexpr (HOLD) {
#pragma unroll
        for (int m = 0; m < P; ++m) x[m] = held[k][m];
      } else {
        IO::unpack(ld_staged(slot(cons, k)), x);
      }
    };
    float2 acc = splat2(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (ok[k]) {
        if constexpr (HOLD) IO::unpack(ld_staged(slot(cons, k)), held[k]);
        float2 x[P];
        channels(k, x);
#pragma unroll
        for (int m = 0; m < P; ++m) acc = add2(x[m], acc);
      }
    }
    const float sum = warp_sum(acc.x + acc.y);
    float mean = sum * inv_nw;  // of the warp's slice
    acc = splat2(0.f);
    float2 neg = splat2(-mean);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (ok[k]) {
        float2 x[P];
        channels(k, x);
#pragma unroll
        for (int m = 0; m < P; ++m) {
          const float2 d = add2(x[m], neg);
          acc = fma2(d, d, acc);
        }
      }
    }
    float m2 = warp_sum(acc.x + acc.y);
    if (NW > 1) {
      float4 *r = red + (j & 1) * NW;
      if (lane == 0) r[warp] = make_float4(sum, m2, mean, n_w);
      __syncthreads();
      float4 v[NW];
      mean = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        v[w] = r[w];
        mean += v[w].x;
      }
      mean *= inv_D;
      m2 = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float d = v[w].z - mean;
        m2 += fmaf(v[w].w * d, d, v[w].y);
      }
    }
    const float rstd = rsqrtf(fmaf(m2, inv_D, a.eps));

    neg = splat2(-mean);
    const float2 inv2 = splat2(rstd);
    uint4 *yrow = reinterpret_cast<uint4 *>(yc + row * row_bytes) + tid;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (ok[k]) {
        float2 x[P], o[P];
        channels(k, x);
#pragma unroll
        for (int m = 0; m < P; ++m)
          o[m] = fma2(add2(x[m], neg), mul2(fac[k][m], inv2), off[k][m]);
        st_stream16(yrow + k * NT, IO::pack(o));
      }
    }
    if (a.mean && tid == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    cur.next(a.L);
    cons = (cons + 1 == S) ? 0 : cons + 1;
  }
  cp_async_wait<0>();
}

// Chunk of consecutive rows per CTA turn, as RMS-AdaLN's.
constexpr int kLnChunk = 8;
// Rows of the ring: one ahead.  More in flight is slower where the tensors are far
// larger than L2 (160 x 4, short / long runs at the 5 s clip: 2 rows 0.405 /
// 0.426 ms, 3 rows 0.459 / 0.422, 4 rows 0.472 / 0.462; 250,000 rows of 2,048
// bf16: 0.330, 0.373 and 0.376), and none ahead waits (0.558).
constexpr int kLnStages = 2;

template <typename T, int NT, int VPT, bool FULL>
cudaError_t launch_t(const LnArgs &a, cudaStream_t stream) {
  auto *kern = &layer_norm_kernel<T, NT, VPT, kLnStages, kLnChunk, FULL>;
  const void *fn = reinterpret_cast<const void *>(kern);
  const size_t smem = 2 * (NT / 32) * 16 + static_cast<size_t>(kLnStages) * VPT * NT * 16;
  const int per_sm = resident_blocks(fn, NT, smem);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t grid = static_cast<int64_t>(per_sm) * device_sms();
  if (grid > a.rows) grid = a.rows;
  kern<<<static_cast<unsigned>(grid), NT, smem, stream>>>(a);
  return cudaGetLastError();
}

// Four vectors per thread up to 256 threads, then more.  A split that covers the
// row exactly takes the unguarded instantiation: at the 5 s clip (160 x 4) 0.405
// against 0.417 ms, 0.429 / 0.444 in long runs; 8,264 rows 5% faster; 250,000 rows of
// 2,048 bf16 0.319 / 0.408 ms.
template <typename T>
cudaError_t dispatch(const LnArgs &a, int threads, int vpt, cudaStream_t stream) {
#define SOL_CASE(NT, V)                                                \
  if (threads == NT && vpt == V)                                       \
    return a.nvec == NT * V ? launch_t<T, NT, V, true>(a, stream)      \
                            : launch_t<T, NT, V, false>(a, stream);
  SOL_QK_OTF_SPLITS(SOL_CASE)
#undef SOL_CASE
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_layer_norm(const LnArgs &a, int dtype, cudaStream_t stream) {
  int threads = 0, vpt = 0;
  if (!pick_split_otf(a.nvec, &threads, &vpt)) return cudaErrorInvalidValue;
  return dtype == 0 ? dispatch<float>(a, threads, vpt, stream)
                    : dispatch<__nv_bfloat16>(a, threads, vpt, stream);
}

}  // namespace sol
