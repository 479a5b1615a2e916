// Dropout in front of the AdaLN-gated residual, forward and backward:
//   out     = h + gate[b][m] * keep * branch / (1 - p)
//   dbranch = gate[b][m] * keep * dout / (1 - p)
//   dgate[b][m] = sum over its rows of keep * dout * branch / (1 - p)
//
// The mask is never stored.  keep of element e of [B, L, D] is a function of
// (seed, offset + site, e) alone: word e mod 4 of Philox4x32-10 (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011)
// at counter (e / 4, offset + site) under key seed; the element is dropped
// where the word is below p * 2^32.  So the backward pass, any launch shape
// and any split of the rows give the same mask.  seed and offset are read
// from device memory: a captured graph that advances them draws a new mask on
// every replay.
//
// A thread owns one 16-byte vector of channels (NT threads span a tile of the
// row's vectors, RG groups of them take different rows) and U rows at a time:
// it issues the U rows' loads, computes the U vectors' words while they are
// in flight and then writes.  The gate of the current (sample, modality)
// stays in registers.
//
// Bound by HBM (3*D*esize bytes per row, forward and backward) with the
// generator close behind: a Philox call is 20 wide multiplies and 20
// three-input xors for four elements.
#include "segment_sums.cuh"
#include "sol_device.cuh"

namespace sol {
namespace {

constexpr int kDropThreads = 256;  // bound on NT * RG

// The ten round keys of a seed.
struct PhiloxKey {
  uint32_t a[10], b[10];
  __device__ __forceinline__ void init(uint64_t seed) {
    uint32_t x = static_cast<uint32_t>(seed), y = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      a[r] = x;
      b[r] = y;
      x += 0x9E3779B9u;
      y += 0xBB67AE85u;
    }
  }
  __device__ __forceinline__ uint4 words(uint64_t lo, uint64_t hi) const {
    uint32_t c0 = static_cast<uint32_t>(lo), c1 = static_cast<uint32_t>(lo >> 32);
    uint32_t c2 = static_cast<uint32_t>(hi), c3 = static_cast<uint32_t>(hi >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
      const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
      c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ a[r];
      c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ b[r];
      c1 = static_cast<uint32_t>(p1);
      c3 = static_cast<uint32_t>(p0);
    }
    return make_uint4(c0, c1, c2, c3);
  }
};

// 16-byte load not kept in L1: the tensors are read once.
__device__ __forceinline__ uint4 ld_stream16(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Bit i: element i of the vector at counter `ctr` is kept.
template <int E>
__device__ __forceinline__ uint32_t keep_bits(const PhiloxKey &key, uint64_t ctr, uint64_t hi,
                                              uint32_t drop_max) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    const uint4 w = key.words(ctr + i, hi);
    bits |= (w.x > drop_max ? 1u : 0u) << (4 * i);
    bits |= (w.y > drop_max ? 2u : 0u) << (4 * i);
    bits |= (w.z > drop_max ? 4u : 0u) << (4 * i);
    bits |= (w.w > drop_max ? 8u : 0u) << (4 * i);
  }
  return bits;
}
template <int P>
__device__ __forceinline__ void drop_pairs(float2 (&v)[P], uint32_t bits) {
#pragma unroll
  for (int m = 0; m < P; ++m) {
    v[m].x = (bits >> (2 * m)) & 1u ? v[m].x : 0.f;
    v[m].y = (bits >> (2 * m + 1)) & 1u ? v[m].y : 0.f;
  }
}

template <typename T, bool DROP, bool RES, bool GATE, int U>
__global__ void __launch_bounds__(kDropThreads) dropout_residual_kernel(const DropArgs a,
                                                                        int tiles) {
  using IO = Io<T>;
  constexpr int P = IO::E / 2;
  const int NT = blockDim.x, RG = blockDim.y, ty = threadIdx.y;
  const int col = static_cast<int>(blockIdx.x % tiles) * NT + threadIdx.x;
  if (col >= a.nvec) return;
  const uint4 *branch = static_cast<const uint4 *>(a.branch) + col;
  const uint4 *h = static_cast<const uint4 *>(a.h) + col;
  uint4 *out = static_cast<uint4 *>(a.out) + col;

  PhiloxKey pk;
  uint64_t hi = 0;
  if constexpr (DROP) {
    pk.init(__ldg(reinterpret_cast<const unsigned long long *>(a.rng)));
    hi = __ldg(reinterpret_cast<const unsigned long long *>(a.rng) + 1) + a.site;
  }
  float2 gt[P];  // gate * 1 / (1 - p) of `key`
#pragma unroll
  for (int m = 0; m < P; ++m) gt[m] = splat2(a.keep_scale);
  int key = -1;

  const int rows = static_cast<int>(a.seg.rows), L = a.seg.L;
  const int step = RG * U;
  // rows in blocks of `step` consecutive ones dealt round-robin over the CTAs
  // of a tile, so the grid works through one window of the tensors
  const int64_t stride = static_cast<int64_t>(gridDim.x / tiles) * step;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x / tiles) * step; r0 < rows; r0 += stride) {
    const int first = static_cast<int>(r0) + ty;
    uint4 vb[U], vh[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = static_cast<int64_t>(first) + u * RG;
      if (row < rows) {
        vb[u] = ld_stream16(branch + row * a.nvec);
        if constexpr (RES) vh[u] = ld_stream16(h + row * a.nvec);
      }
    }
    int b = 0, r = 0;
    if constexpr (GATE) {
      b = first / L;
      r = first - b * L;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = static_cast<int64_t>(first) + u * RG;
      if (row < rows) {
        if constexpr (GATE) {
          const int nkey = 2 * b + (r >= a.seg.n_video ? 1 : 0);
          if (nkey != key) {
            key = nkey;
            IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.gate) +
                                     static_cast<int64_t>(key) * a.nvec + col),
                       gt);
#pragma unroll
            for (int m = 0; m < P; ++m) gt[m] = mul2(gt[m], splat2(a.keep_scale));
          }
        }
        float2 x[P], o[P];
        IO::unpack(vb[u], x);
        if constexpr (DROP) {
          const uint64_t ctr = (static_cast<uint64_t>(row) * a.nvec + col) * (IO::E / 4);
          drop_pairs(x, keep_bits<IO::E>(pk, ctr, hi, a.drop_max));
        }
        if constexpr (RES) {
          IO::unpack(vh[u], o);
#pragma unroll
          for (int m = 0; m < P; ++m) o[m] = fma2(gt[m], x[m], o[m]);
        } else {
#pragma unroll
          for (int m = 0; m < P; ++m) o[m] = mul2(gt[m], x[m]);
        }
        st_stream16(out + row * a.nvec, IO::pack(o));
      }
      if constexpr (GATE) {
        r += RG;
        while (r >= L) {
          r -= L;
          ++b;
        }
      }
    }
  }
}

// blockIdx.x = tile + tiles * share; the rows of a share are cut into runs of
// one (sample, modality), whose sums go to slot share + key.
template <typename T, bool DROP, int U>
__global__ void __launch_bounds__(kDropThreads) dropout_backward_kernel(const DropArgs a,
                                                                        int tiles) {
  using IO = Io<T>;
  constexpr int P = IO::E / 2;
  __shared__ float2 park[P * kDropThreads];
  const int NT = blockDim.x, RG = blockDim.y, ty = threadIdx.y;
  const int tid = ty * NT + threadIdx.x;
  const int share = static_cast<int>(blockIdx.x / tiles);
  const int col = static_cast<int>(blockIdx.x % tiles) * NT + threadIdx.x;
  const bool ok = col < a.nvec;
  const uint4 *branch = static_cast<const uint4 *>(a.branch) + col;
  const uint4 *dout = static_cast<const uint4 *>(a.dout) + col;
  uint4 *out = static_cast<uint4 *>(a.out) + col;

  PhiloxKey pk;
  uint64_t hi = 0;
  if constexpr (DROP) {
    pk.init(__ldg(reinterpret_cast<const unsigned long long *>(a.rng)));
    hi = __ldg(reinterpret_cast<const unsigned long long *>(a.rng) + 1) + a.site;
  }

  int64_t row = share_begin(a.seg, share);
  const int64_t share_end = share_begin(a.seg, share + 1);
  while (row < share_end) {
    const int key = key_of(a.seg, row);
    int64_t run_end, unused;
    key_rows(a.seg, key, &unused, &run_end);
    if (run_end > share_end) run_end = share_end;

    float2 gt[P], sum[P];
#pragma unroll
    for (int m = 0; m < P; ++m) sum[m] = splat2(0.f);
    if (ok) {
      IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.gate) +
                               static_cast<int64_t>(key) * a.nvec + col),
                 gt);
#pragma unroll
      for (int m = 0; m < P; ++m) gt[m] = mul2(gt[m], splat2(a.keep_scale));
      for (int64_t r0 = row + ty; r0 < run_end; r0 += RG * U) {
        uint4 vd[U], vb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t r = r0 + u * RG;
          if (r < run_end) {
            vd[u] = ld_stream16(dout + r * a.nvec);
            vb[u] = ld_stream16(branch + r * a.nvec);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t r = r0 + u * RG;
          if (r < run_end) {
            float2 d[P], x[P];
            IO::unpack(vd[u], d);
            IO::unpack(vb[u], x);
            if constexpr (DROP) {
              const uint64_t ctr = (static_cast<uint64_t>(r) * a.nvec + col) * (IO::E / 4);
              const uint32_t bits = keep_bits<IO::E>(pk, ctr, hi, a.drop_max);
              drop_pairs(d, bits);
              drop_pairs(x, bits);  // an infinite branch value adds nothing where dropped
            }
#pragma unroll
            for (int m = 0; m < P; ++m) {
              sum[m] = fma2(d[m], x[m], sum[m]);
              d[m] = mul2(gt[m], d[m]);
            }
            st_stream16(out + r * a.nvec, IO::pack(d));
          }
        }
      }
    }
    if (RG > 1) {
      if (ty > 0) {
#pragma unroll
        for (int m = 0; m < P; ++m) park[m * kDropThreads + tid] = sum[m];
      }
      __syncthreads();
      if (ty == 0) {
        for (int y = 1; y < RG; ++y)
#pragma unroll
          for (int m = 0; m < P; ++m)
            sum[m] = add2(sum[m], park[m * kDropThreads + y * NT + tid]);
      }
      __syncthreads();
    }
    if (ok && ty == 0) {
      float2 *dst = reinterpret_cast<float2 *>(
                        a.partial + (share + static_cast<int64_t>(key)) * a.D) +
                    static_cast<int64_t>(col) * P;
#pragma unroll
      for (int m = 0; m < P; ++m) dst[m] = sum[m];
    }
    row = run_end;
  }
}

// Vectors of a row over `tiles` tiles of NT threads: the tile count of at
// most 256 threads each that leaves the fewest threads idle, the wider tile
// where they tie (640 vectors: 4 x 160).
void pick_tiles(int nvec, int *tiles, int *nt) {
  const int t0 = (nvec + kDropThreads - 1) / kDropThreads;
  int best = -1;
  for (int t = t0; t < t0 + 4; ++t) {
    const int n = ((nvec + t - 1) / t + 31) / 32 * 32;
    if (best < 0 || t * n < best) {
      best = t * n;
      *tiles = t;
      *nt = n;
    }
  }
}

template <typename T, bool DROP, bool RES, bool GATE>
cudaError_t launch_fwd(const DropArgs &a, cudaStream_t stream) {
  constexpr int U = 4;
  int tiles = 1, nt = 32;
  pick_tiles(a.nvec, &tiles, &nt);
  const int rg = kDropThreads / nt;
  auto *kern = &dropout_residual_kernel<T, DROP, RES, GATE, U>;
  const int per_sm = resident_blocks(reinterpret_cast<const void *>(kern), nt * rg, 0);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t shares = static_cast<int64_t>(per_sm) * device_sms() / tiles;
  const int64_t most = (a.seg.rows + rg * U - 1) / (rg * U);
  if (shares > most) shares = most;
  if (shares < 1) shares = 1;
  kern<<<static_cast<unsigned>(shares * tiles), dim3(nt, rg), 0, stream>>>(a, tiles);
  return cudaGetLastError();
}

template <typename T, bool DROP>
cudaError_t launch_bwd(DropArgs &a, cudaStream_t stream) {
  constexpr int U = 4;
  int tiles = 1, nt = 32;
  pick_tiles(a.nvec, &tiles, &nt);
  const int rg = kDropThreads / nt;
  auto *kern = &dropout_backward_kernel<T, DROP, U>;
  const int per_sm = resident_blocks(reinterpret_cast<const void *>(kern), nt * rg, 0);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t shares = static_cast<int64_t>(per_sm) * device_sms() / tiles;
  const int64_t most = (a.seg.rows + rg * U - 1) / (rg * U);
  if (shares > most) shares = most;
  if (shares > kMaxSumCtas) shares = kMaxSumCtas;
  if (shares < 1) shares = 1;
  a.seg.ctas = static_cast<int>(shares);
  kern<<<static_cast<unsigned>(shares * tiles), dim3(nt, rg), 0, stream>>>(a, tiles);
  return cudaGetLastError();
}

template <typename T, bool DROP>
cudaError_t fwd_kind(const DropArgs &a, cudaStream_t stream) {
  if (a.h)
    return a.gate ? launch_fwd<T, DROP, true, true>(a, stream)
                  : launch_fwd<T, DROP, true, false>(a, stream);
  return a.gate ? launch_fwd<T, DROP, false, true>(a, stream)
                : launch_fwd<T, DROP, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_dropout_residual(const DropArgs &a, int dtype, cudaStream_t stream) {
  if (dtype == 0)
    return a.drop ? fwd_kind<float, true>(a, stream) : fwd_kind<float, false>(a, stream);
  return a.drop ? fwd_kind<__nv_bfloat16, true>(a, stream)
                : fwd_kind<__nv_bfloat16, false>(a, stream);
}

cudaError_t launch_dropout_backward(DropArgs &a, int dtype, cudaStream_t stream) {
  if (dtype == 0)
    return a.drop ? launch_bwd<float, true>(a, stream) : launch_bwd<float, false>(a, stream);
  return a.drop ? launch_bwd<__nv_bfloat16, true>(a, stream)
                : launch_bwd<__nv_bfloat16, false>(a, stream);
}

}  // namespace sol
