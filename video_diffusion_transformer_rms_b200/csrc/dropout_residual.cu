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
// it issues the U rows' loads and computes the U vectors' words while they
// arrive.  The gate of the current (sample, modality) stays in registers.
//
// HBM traffic is 3*D*esize bytes per row, forward and backward, but the issue
// slots are as scarce: a Philox call is 20 wide multiplies and 20 three-input
// xors for four elements.  So the rest is kept small: a dropped element is a
// predicated multiply-add that does not happen, the two calls of a bf16 vector
// share the upper counter word and what depends on it alone, rows are 32-bit
// indexes.
//
// dbranch is rounded in the formula's order, gate * (dout * 1 / (1 - p)): where the
// exact product is a tie of bf16 (p = 1/4 makes many), another order rounds it the other
// way.  It costs a multiplication that a gate scaled once would not: 0.650 against
// 0.643 ms at the 5 s clip.  Forward, where the sum with h hides it, the gate is scaled.
#include "segment_sums.cuh"
#include "sol_device.cuh"

namespace sol {
namespace {

// 128 threads with up to 128 registers, 4 rows each: 0.623 ms for the forward
// pass at the 5 s clip, 0.650 ms for the backward.  (Against 0.627 and 0.653 of an
// earlier form, 256 threads x 128 registers took 0.655 and 0.683, x 80 0.677 and
// 0.733.)
constexpr int kDropThreads = 128;  // bound on NT * RG
constexpr int kDropCtas = 4;       // CTAs per SM the registers are to leave room for
// rows per thread and pass (fp32, 60,000 x 5120: three 0.564, four 0.588 ms; its
// gradient the same; bf16 at the 5 s clip: three 0.645, four 0.621 ms)
template <typename T>
constexpr int kDropRows = sizeof(T) == 4 ? 3 : 4;

// The ten round keys of a seed.
struct PhiloxKey {
  uint32_t a[10], b[10];
  __device__ __forceinline__ void init(uint64_t seed) {
    uint32_t x = static_cast<uint32_t>(seed), y = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      a[r] = x;
      b[r] = y;
      // opaque: otherwise the keys are added up again in every call, 20 of its
      // 60 instructions
      asm volatile("" : "+r"(a[r]), "+r"(b[r]));
      x += 0x9E3779B9u;
      y += 0xBB67AE85u;
    }
  }
  __device__ __forceinline__ uint4 words(uint32_t c0, uint32_t c1, uint32_t c2,
                                         uint32_t c3) const {
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
__device__ __forceinline__ uint4 ld_stream16(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// acc += a * b where the word keeps the element.
__device__ __forceinline__ void fma_kept(uint32_t word, uint32_t drop_max, float a, float b,
                                         float &acc) {
  asm("{\n\t.reg .pred p;\n\tsetp.gt.u32 p, %1, %2;\n\t@p fma.rn.f32 %0, %3, %4, %0;\n\t}"
      : "+f"(acc)
      : "r"(word), "r"(drop_max), "f"(a), "f"(b));
}
// acc += a * b where the word keeps the element; prod becomes 0 where not.
__device__ __forceinline__ void fma_select_kept(uint32_t word, uint32_t drop_max, float a, float b,
                                                float &acc, float &prod) {
  asm("{\n\t.reg .pred p;\n\tsetp.gt.u32 p, %2, %3;\n\t@p fma.rn.f32 %0, %4, %5, %0;\n\t"
      "selp.f32 %1, %1, 0f00000000, p;\n\t}"
      : "+f"(acc), "+f"(prod)
      : "r"(word), "r"(drop_max), "f"(a), "f"(b));
}

// The words of a vector of E elements; `ctr` is the counter of its first
// element, a multiple of E / 4, so adding 1 for the second call carries nowhere.
template <int E>
__device__ __forceinline__ void vector_words(const PhiloxKey &key, uint64_t ctr, uint64_t hi,
                                             uint4 (&w)[E / 4]) {
  const uint32_t c0 = static_cast<uint32_t>(ctr), c1 = static_cast<uint32_t>(ctr >> 32);
#pragma unroll
  for (int i = 0; i < E / 4; ++i)
    w[i] = key.words(c0 + i, c1, static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32));
}

template <typename T, bool DROP, bool RES, bool GATE>
__global__ void __launch_bounds__(kDropThreads, kDropCtas)
    dropout_residual_kernel(const DropArgs a, int tiles) {
  using IO = Io<T>;
  constexpr int E = IO::E, P = E / 2, U = kDropRows<T>;
  const int NT = blockDim.x, RG = blockDim.y;
  const int col = static_cast<int>(blockIdx.x % tiles) * NT + threadIdx.x;
  const int64_t row_bytes = static_cast<int64_t>(a.nvec) * 16, step = RG * row_bytes;
  const unsigned char *branch = static_cast<const unsigned char *>(a.branch) + col * 16;
  const unsigned char *h = static_cast<const unsigned char *>(a.h) + col * 16;
  unsigned char *out = static_cast<unsigned char *>(a.out) + col * 16;

  PhiloxKey pk;
  uint64_t hi = 0;
  if constexpr (DROP) {
    pk.init(__ldg(reinterpret_cast<const unsigned long long *>(a.rng)));
    hi = __ldg(reinterpret_cast<const unsigned long long *>(a.rng) + 1) + a.site;
  }
  if (col >= a.nvec) return;
  // Without h the call is also the gradient, which keeps the formula's order
  constexpr bool LATE = DROP && GATE && !RES;
  const float2 ks = splat2(a.keep_scale);
  float2 gt[P];  // gate (* 1 / (1 - p)) of the current (sample, modality)
#pragma unroll
  for (int m = 0; m < P; ++m) gt[m] = splat2(a.keep_scale);
  int key_end = 0;  // first row past the ones `gt` is for

  // rows in blocks of RG * U consecutive ones dealt round-robin over the CTAs of
  // a tile, so the grid works through one window of the tensors
  const int rows = static_cast<int>(a.seg.rows), block = RG * U;
  const int64_t stride = static_cast<int64_t>(gridDim.x / tiles) * block;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x / tiles) * block; r0 < rows; r0 += stride) {
    // rows of this thread in the block: `first`, RG apart
    const int64_t first64 = r0 + threadIdx.y;
    const int first = static_cast<int>(first64);
    const int n = first64 < rows ? (rows - 1 - first) / RG + 1 : 0;
    const int64_t off = first64 * row_bytes;
    const uint64_t ctr = (static_cast<uint64_t>(first64) * a.nvec + col) * (E / 4);
    const uint32_t ctr_step = static_cast<uint32_t>(RG) * a.nvec * (E / 4);
    uint4 vb[U], vh[U];
    auto load = [&](int u) {
      vb[u] = ld_stream16(branch + off + u * step);
      if constexpr (RES) vh[u] = ld_stream16(h + off + u * step);
    };
    auto finish = [&](int u) {
      float2 x[P], o[P];
      IO::unpack(vb[u], x);
      if constexpr (RES) IO::unpack(vh[u], o);
      if constexpr (DROP) {
        uint4 w[E / 4];
        vector_words<E>(pk, ctr + u * ctr_step, hi, w);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          float2 &x0 = x[2 * i], &x1 = x[2 * i + 1];
          if constexpr (RES) {
            float2 &o0 = o[2 * i], &o1 = o[2 * i + 1];
            fma_kept(w[i].x, a.drop_max, gt[2 * i].x, x0.x, o0.x);
            fma_kept(w[i].y, a.drop_max, gt[2 * i].y, x0.y, o0.y);
            fma_kept(w[i].z, a.drop_max, gt[2 * i + 1].x, x1.x, o1.x);
            fma_kept(w[i].w, a.drop_max, gt[2 * i + 1].y, x1.y, o1.y);
          } else {
            if constexpr (LATE) {
              x0 = mul2(x0, ks);
              x1 = mul2(x1, ks);
            }
            x0 = mul2(gt[2 * i], x0);
            x1 = mul2(gt[2 * i + 1], x1);
            o[2 * i].x = w[i].x > a.drop_max ? x0.x : 0.f;
            o[2 * i].y = w[i].y > a.drop_max ? x0.y : 0.f;
            o[2 * i + 1].x = w[i].z > a.drop_max ? x1.x : 0.f;
            o[2 * i + 1].y = w[i].w > a.drop_max ? x1.y : 0.f;
          }
        }
      } else {
#pragma unroll
        for (int m = 0; m < P; ++m) o[m] = RES ? fma2(gt[m], x[m], o[m]) : mul2(gt[m], x[m]);
      }
      st_stream16(out + off + u * step, IO::pack(o));
    };
    if (n >= U && (!GATE || first + (U - 1) * RG < key_end)) {
      // a whole block under the present gate
#pragma unroll
      for (int u = 0; u < U; ++u) load(u);
#pragma unroll
      for (int u = 0; u < U; ++u) finish(u);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < n) load(u);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u < n) {
          if constexpr (GATE) {
            if (first + u * RG >= key_end) {
              const int key = key_of(a.seg, first + u * RG);
              int64_t begin, end;
              key_rows(a.seg, key, &begin, &end);
              key_end = static_cast<int>(end);
              IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.gate) +
                                       static_cast<int64_t>(key) * a.nvec + col),
                         gt);
              if constexpr (!LATE) {
#pragma unroll
                for (int m = 0; m < P; ++m) gt[m] = mul2(gt[m], ks);
              }
            }
          }
          finish(u);
        }
      }
    }
  }
}

// blockIdx.x = tile + tiles * share; the rows of a share are cut into runs of
// one (sample, modality), whose sums go to slot share + key.
template <typename T, bool DROP>
__global__ void __launch_bounds__(kDropThreads, kDropCtas)
    dropout_backward_kernel(const DropArgs a, int tiles) {
  using IO = Io<T>;
  constexpr int E = IO::E, P = E / 2, U = kDropRows<T>;
  __shared__ float2 park[P * kDropThreads];
  const int NT = blockDim.x, RG = blockDim.y, ty = threadIdx.y;
  const int tid = ty * NT + threadIdx.x;
  const int share = static_cast<int>(blockIdx.x / tiles);
  const int col = static_cast<int>(blockIdx.x % tiles) * NT + threadIdx.x;
  const bool ok = col < a.nvec;
  const int64_t row_bytes = static_cast<int64_t>(a.nvec) * 16, step = RG * row_bytes;
  const unsigned char *branch = static_cast<const unsigned char *>(a.branch) + col * 16;
  const unsigned char *dout = static_cast<const unsigned char *>(a.dout) + col * 16;
  unsigned char *out = static_cast<unsigned char *>(a.out) + col * 16;

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

    const float2 ks = splat2(a.keep_scale);
    float2 gt[P], sum[P];
#pragma unroll
    for (int m = 0; m < P; ++m) sum[m] = splat2(0.f);
    if (ok) {
      IO::unpack(ld_shared_vec(static_cast<const uint4 *>(a.gate) +
                               static_cast<int64_t>(key) * a.nvec + col),
                 gt);
      // rows of this thread in the run
      const int64_t first = row + ty;
      int n = first < run_end ? static_cast<int>((run_end - 1 - first) / RG) + 1 : 0;
      int64_t off = first * row_bytes;
      uint64_t ctr = (static_cast<uint64_t>(first) * a.nvec + col) * (E / 4);
      const uint32_t ctr_step = static_cast<uint32_t>(RG) * a.nvec * (E / 4);
      uint4 vd[U], vb[U];
      auto load = [&](int u) {
        vd[u] = ld_stream16(dout + off + u * step);
        vb[u] = ld_stream16(branch + off + u * step);
      };
      auto finish = [&](int u) {
        float2 d[P], x[P], o[P];
        IO::unpack(vd[u], d);
        IO::unpack(vb[u], x);
#pragma unroll
        for (int m = 0; m < P; ++m) o[m] = mul2(gt[m], DROP ? mul2(d[m], ks) : d[m]);
        if constexpr (DROP) {
          uint4 w[E / 4];
          vector_words<E>(pk, ctr + u * ctr_step, hi, w);
#pragma unroll
          for (int i = 0; i < E / 4; ++i) {
            const int m = 2 * i;
            fma_select_kept(w[i].x, a.drop_max, d[m].x, x[m].x, sum[m].x, o[m].x);
            fma_select_kept(w[i].y, a.drop_max, d[m].y, x[m].y, sum[m].y, o[m].y);
            fma_select_kept(w[i].z, a.drop_max, d[m + 1].x, x[m + 1].x, sum[m + 1].x, o[m + 1].x);
            fma_select_kept(w[i].w, a.drop_max, d[m + 1].y, x[m + 1].y, sum[m + 1].y, o[m + 1].y);
          }
        } else {
#pragma unroll
          for (int m = 0; m < P; ++m) sum[m] = fma2(d[m], x[m], sum[m]);
        }
        st_stream16(out + off + u * step, IO::pack(o));
      };
      for (; n >= U; n -= U, off += U * step, ctr += U * ctr_step) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(u);
#pragma unroll
        for (int u = 0; u < U; ++u) finish(u);
      }
#pragma unroll
      for (int u = 0; u < U - 1; ++u)
        if (u < n) load(u);
#pragma unroll
      for (int u = 0; u < U - 1; ++u)
        if (u < n) finish(u);
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

// Vectors of a row over `tiles` tiles of NT threads, at most kDropThreads: of the
// four smallest tile counts the one that leaves the fewest threads idle, the wider
// tile where they tie (640 vectors: 5 x 128).
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
  int tiles = 1, nt = 32;
  pick_tiles(a.nvec, &tiles, &nt);
  const int rg = kDropThreads / nt;
  auto *kern = &dropout_residual_kernel<T, DROP, RES, GATE>;
  const int per_sm = resident_blocks(reinterpret_cast<const void *>(kern), nt * rg, 0);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t shares = static_cast<int64_t>(per_sm) * device_sms() / tiles;
  const int64_t most = (a.seg.rows + rg * kDropRows<T> - 1) / (rg * kDropRows<T>);
  if (shares > most) shares = most;
  if (shares < 1) shares = 1;
  kern<<<static_cast<unsigned>(shares * tiles), dim3(nt, rg), 0, stream>>>(a, tiles);
  return cudaGetLastError();
}

template <typename T, bool DROP>
cudaError_t launch_bwd(DropArgs &a, cudaStream_t stream) {
  int tiles = 1, nt = 32;
  pick_tiles(a.nvec, &tiles, &nt);
  const int rg = kDropThreads / nt;
  auto *kern = &dropout_backward_kernel<T, DROP>;
  const int per_sm = resident_blocks(reinterpret_cast<const void *>(kern), nt * rg, 0);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  int64_t shares = static_cast<int64_t>(per_sm) * device_sms() / tiles;
  const int64_t most = (a.seg.rows + rg * kDropRows<T> - 1) / (rg * kDropRows<T>);
  if (shares > most) shares = most;
  if (shares > kMaxSumCtas) shares = kMaxSumCtas;
  if (shares < 1) shares = 1;  // never more than rows
  cut_shares(&a.seg, shares);
  kern<<<static_cast<unsigned>(a.seg.ctas * tiles), dim3(nt, rg), 0, stream>>>(a, tiles);
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
