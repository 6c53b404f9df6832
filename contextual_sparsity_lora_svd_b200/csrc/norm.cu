// RMS normalisation with a frozen per-channel gain, fused with the residual
// add before it (forward) and with the sum of the branch gradients and the
// residual gradient (backward).  Rows of up to 16384 channels: one 128-thread
// block per row, each thread holding its 16-byte chunks in registers, so every
// input is read once and every output written once (a block-wide sum in
// between).  Longer rows: one warp per row in two passes.  Every value is
// rounded to bf16 where it is stored, and the normalisation reads the rounded
// residual sum, the value the backward sees.
//
// The variants with 8-bit checkpoints (act8.cuh) write the codes of H and N in
// the same pass (a 32-channel block is four neighbouring lanes' chunks, its
// maximum two shuffles), and read H as codes in the backward: 1.03 bytes a
// value in place of 2, and no separate pass over H and N to pack them.  At
// 4096 x 4096: forward 26 us (169 MB), backward 25 us (118 MB; every value of a
// row is on its way before the first use, 24 warps an SM).
#include "act8.cuh"
#include "act8_dev.cuh"
#include "attention.cuh"

namespace slora {
namespace {

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __low2float(h[i]);
    f[2 * i + 1] = __high2float(h[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return u;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// h = X + A (rounded), N = h rstd g
__global__ void rmsnorm_fwd_kernel(const uint4* __restrict__ X, const uint4* __restrict__ A,
                                   const uint4* __restrict__ g, int64_t T, int nch, float eps,
                                   uint4* __restrict__ Hout, uint4* __restrict__ N,
                                   float* __restrict__ rstd) {
  const int64_t row = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= T) return;
  const int64_t o = row * nch;
  auto load_h = [&](int c, float (&h)[8]) {
    unpack8(X[o + c], h);
    if (A) {
      float a[8];
      unpack8(A[o + c], a);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = __bfloat162float(__float2bfloat16_rn(h[i] + a[i]));
    }
  };
  float ss = 0.f;
  for (int c = lane; c < nch; c += 32) {
    float h[8];
    load_h(c, h);
    if (A && Hout) Hout[o + c] = pack8(h);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += h[i] * h[i];
  }
  ss = warp_sum(ss);
  const float r = rsqrtf(ss / float(nch * 8) + eps);
  if (lane == 0 && rstd) rstd[row] = r;
  if (!N) return;
  for (int c = lane; c < nch; c += 32) {
    float h[8], gg[8];
    load_h(c, h);
    unpack8(g[c], gg);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] *= r * gg[i];
    N[o + c] = pack8(h);
  }
}

// dX = dRes + r g dN - h r^3 mean(h g dN), dN = dN0 + dN1 + dN2
__global__ void rmsnorm_bwd_kernel(const uint4* __restrict__ Hin, const float* __restrict__ rstd,
                                   const uint4* __restrict__ g, const uint4* __restrict__ dN0,
                                   const uint4* __restrict__ dN1, const uint4* __restrict__ dN2,
                                   const uint4* __restrict__ dRes, int64_t T, int nch,
                                   uint4* __restrict__ dX) {
  const int64_t row = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= T) return;
  const int64_t o = row * nch;
  auto load_dn = [&](int c, float (&dn)[8]) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dn[i] = 0.f;
    const uint4* srcs[3] = {dN0, dN1, dN2};
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      if (!srcs[s]) continue;
      unpack8(srcs[s][o + c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) dn[i] += t[i];
    }
  };
  float dot = 0.f;
  for (int c = lane; c < nch; c += 32) {
    float h[8], gg[8], dn[8];
    unpack8(Hin[o + c], h);
    unpack8(g[c], gg);
    load_dn(c, dn);
#pragma unroll
    for (int i = 0; i < 8; ++i) dot += h[i] * gg[i] * dn[i];
  }
  dot = warp_sum(dot);
  const float r = rstd[row];
  const float coef = r * r * r * dot / float(nch * 8);
  for (int c = lane; c < nch; c += 32) {
    float h[8], gg[8], dn[8], res[8];
    unpack8(Hin[o + c], h);
    unpack8(g[c], gg);
    load_dn(c, dn);
    if (dRes) unpack8(dRes[o + c], res);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = r * gg[i] * dn[i] - h[i] * coef;
      h[i] = dRes ? res[i] + v : v;
    }
    dX[o + c] = pack8(h);
  }
}

constexpr int kRowThreads = 128;

__device__ __forceinline__ float block_sum128(float v, float* red) {
  v = warp_sum(v);
  const int w = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[w] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];  // fixed order
}

// One block per row; thread t holds chunks t, t + 128, ... (CPT of them).
template <int CPT>
__global__ void __launch_bounds__(kRowThreads)
    rmsnorm_fwd_row_kernel(const uint4* __restrict__ X, const uint4* __restrict__ A,
                           const uint4* __restrict__ g, int nch, float eps,
                           uint4* __restrict__ Hout, uint4* __restrict__ N,
                           float* __restrict__ rstd) {
  __shared__ float red[4];
  const int64_t o = int64_t(blockIdx.x) * nch;
  float h[CPT][8];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = threadIdx.x + k * kRowThreads;
    if (c < nch) {
      unpack8(X[o + c], h[k]);
      if (A) {
        float a[8];
        unpack8(A[o + c], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = __bfloat162float(__float2bfloat16_rn(h[k][i] + a[i]));
        if (Hout) Hout[o + c] = pack8(h[k]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += h[k][i] * h[k][i];
    }
  }
  const float r = rsqrtf(block_sum128(ss, red) / float(nch * 8) + eps);
  if (threadIdx.x == 0 && rstd) rstd[blockIdx.x] = r;
  if (!N) return;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = threadIdx.x + k * kRowThreads;
    if (c < nch) {
      float gg[8];
      unpack8(g[c], gg);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] *= r * gg[i];
      N[o + c] = pack8(h[k]);
    }
  }
}

template <int CPT>
__global__ void __launch_bounds__(kRowThreads)
    rmsnorm_bwd_row_kernel(const uint4* __restrict__ Hin, const float* __restrict__ rstd,
                           const uint4* __restrict__ g, const uint4* __restrict__ dN0,
                           const uint4* __restrict__ dN1, const uint4* __restrict__ dN2,
                           const uint4* __restrict__ dRes, int nch, uint4* __restrict__ dX) {
  __shared__ float red[4];
  const int64_t o = int64_t(blockIdx.x) * nch;
  float h[CPT][8], gd[CPT][8];
  float dot = 0.f;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = threadIdx.x + k * kRowThreads;
    if (c < nch) {
      float t[8], gg[8];
      unpack8(Hin[o + c], h[k]);
      unpack8(g[c], gg);
      unpack8(dN0[o + c], gd[k]);
      if (dN1) {
        unpack8(dN1[o + c], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) gd[k][i] += t[i];
      }
      if (dN2) {
        unpack8(dN2[o + c], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) gd[k][i] += t[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        gd[k][i] *= gg[i];  // g dN
        dot += h[k][i] * gd[k][i];
      }
    }
  }
  const float r = rstd[blockIdx.x];
  const float coef = r * r * r * block_sum128(dot, red) / float(nch * 8);
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = threadIdx.x + k * kRowThreads;
    if (c < nch) {
      float res[8];
      if (dRes) unpack8(dRes[o + c], res);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = r * gd[k][i] - h[k][i] * coef;
        h[k][i] = dRes ? res[i] + v : v;
      }
      dX[o + c] = pack8(h[k]);
    }
  }
}

// A row's chunks stay packed between the two passes over them (4 registers a
// chunk); the arithmetic and its order are those of the kernels above.  Rows above
// 4096 channels lie in up to four parts of 128 threads, four chunks a thread:
// thread t of part p holds chunks t + 128 (p CPT + k), and its sum goes on where
// thread t of part p - 1 left it, so the bits are those of one part with all the
// chunks.  That part's registers leave 8 to 12 warps an SM; with residual,
// 2048 x 11008: forward 60 -> 40 us, backward 59 -> 39; 4096 x 8192: 57 -> 55 and
// 55 -> 49.  (Parts of two chunks a thread: backward 52 both.)
template <int PARTS, typename F>
__device__ __forceinline__ float row_sum(float* chain, float* red, F add) {
  const int part = threadIdx.x / kRowThreads, t = threadIdx.x % kRowThreads;
  float v = 0.0f;
  if constexpr (PARTS == 1) {
    return block_sum128(add(v), red);
  } else {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      if (part == p) {
        v = add(p ? chain[t] : 0.0f);
        chain[t] = v;
      }
      if (p + 1 < PARTS) __syncthreads();
    }
    if (part == PARTS - 1) {
      v = warp_sum(v);
      if ((t & 31) == 0) red[t >> 5] = v;
    }
    __syncthreads();
    return red[0] + red[1] + red[2] + red[3];  // (block_sum128's order)
  }
}
template <int CPT, int PARTS>
__global__ void __launch_bounds__(kRowThreads * PARTS)
    rmsnorm_fwd_act8_kernel(const uint4* __restrict__ X, const uint4* __restrict__ A,
                            const uint4* __restrict__ g, int nch, float eps,
                            uint4* __restrict__ Hout, uint4* __restrict__ N,
                            float* __restrict__ rstd, uint2* __restrict__ h8,
                            uint8_t* __restrict__ h8s, uint2* __restrict__ n8,
                            uint8_t* __restrict__ n8s) {
  __shared__ float red[4], chain[PARTS > 1 ? kRowThreads : 1];
  const int first = threadIdx.x % kRowThreads + threadIdx.x / kRowThreads * (CPT * kRowThreads);
  grid_wait();
  grid_ahead();
  const int64_t o = int64_t(blockIdx.x) * nch;
  const int nchp = (nch + 3) & ~3;  // chunks of a checkpoint's row
  const int64_t o8 = int64_t(blockIdx.x) * nchp;
  uint4 u[CPT], a[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = first + k * kRowThreads;
    u[k] = c < nch ? X[o + c] : make_uint4(0, 0, 0, 0);
    if (A && c < nch) a[k] = A[o + c];
  }
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = first + k * kRowThreads;
    if (c < nch && A) {
      float h[8], b[8];
      unpack8(u[k], h);
      unpack8(a[k], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] += b[i];
      u[k] = pack8(h);
      if (Hout) Hout[o + c] = u[k];
    }
    if (h8) {
      const uint32_t byte = act8_byte_bf16(u[k]);
      if (c < nchp) {
        h8[o8 + c] = act8_codes8_bf16(u[k], byte);
        if ((c & 3) == 0) h8s[(o8 + c) >> 2] = uint8_t(byte);
      }
    }
  }
  const float ss = row_sum<PARTS>(chain, red, [&](float v) {
#pragma unroll
    for (int k = 0; k < CPT; ++k)
      if (first + k * kRowThreads < nch) {
        float h[8];
        unpack8(u[k], h);
#pragma unroll
        for (int i = 0; i < 8; ++i) v += h[i] * h[i];
      }
    return v;
  });
  const float r = rsqrtf(ss / float(nch * 8) + eps);
  if (threadIdx.x == 0 && rstd) rstd[blockIdx.x] = r;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = first + k * kRowThreads;
    if (c < nch) {
      float h[8], gg[8];
      unpack8(u[k], h);
      unpack8(g[c], gg);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] *= r * gg[i];
      u[k] = pack8(h);  // the checkpoint holds the stored, rounded values
      N[o + c] = u[k];
    }
    if (n8) {
      const uint32_t byte = act8_byte_bf16(u[k]);
      if (c < nchp) {
        n8[o8 + c] = act8_codes8_bf16(u[k], byte);
        if ((c & 3) == 0) n8s[(o8 + c) >> 2] = uint8_t(byte);
      }
    }
  }
}

// Blocks an SM: 80 registers a thread at four chunks, 64 at three.
constexpr int row_blocks(int cpt, int parts) {
  return cpt == 4 ? 6 / parts : cpt == 3 ? 8 / parts : 1;
}
template <int CPT, int PARTS>
__global__ void __launch_bounds__(kRowThreads * PARTS, row_blocks(CPT, PARTS))
    rmsnorm_bwd_act8_kernel(const uint2* __restrict__ h8, const uint8_t* __restrict__ h8s,
                            const float* __restrict__ rstd, const uint4* __restrict__ g,
                            const uint4* __restrict__ dN0, const uint4* __restrict__ dN1,
                            const uint4* __restrict__ dN2, const uint4* __restrict__ dRes,
                            int nch, uint4* __restrict__ dX) {
  __shared__ float red[4], chain[PARTS > 1 ? kRowThreads : 1];
  const int first = threadIdx.x % kRowThreads + threadIdx.x / kRowThreads * (CPT * kRowThreads);
  grid_wait();
  grid_ahead();
  const int64_t o = int64_t(blockIdx.x) * nch, o8 = int64_t(blockIdx.x) * ((nch + 3) & ~3);
  // every input of the row is on its way before the first use
  uint2 hc[CPT];
  uint32_t hb[CPT];
  uint4 d0[CPT], res[CPT];
  const float r = rstd[blockIdx.x];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = first + k * kRowThreads;
    hc[k] = make_uint2(0, 0);
    hb[k] = 7u;
    d0[k] = res[k] = make_uint4(0, 0, 0, 0);
    if (c < nch) {
      hc[k] = h8[o8 + c];
      hb[k] = h8s[(o8 + c) >> 2];
      d0[k] = dN0[o + c];
      if (dRes) res[k] = dRes[o + c];
    }
  }
  float gd[CPT][8];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = first + k * kRowThreads;
    if (c < nch) {
      float t[8];
      unpack8(d0[k], gd[k]);
      if (dN1) {
        unpack8(dN1[o + c], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) gd[k][i] += t[i];
      }
      if (dN2) {
        unpack8(dN2[o + c], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) gd[k][i] += t[i];
      }
      unpack8(g[c], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) gd[k][i] *= t[i];  // g dN
    }
  }
  const float dot = row_sum<PARTS>(chain, red, [&](float v) {
#pragma unroll
    for (int k = 0; k < CPT; ++k)
      if (first + k * kRowThreads < nch) {
        float h[8];
        act8_values8(hc[k], hb[k], h);
#pragma unroll
        for (int i = 0; i < 8; ++i) v += h[i] * gd[k][i];
      }
    return v;
  });
  const float coef = r * r * r * dot / float(nch * 8);
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = first + k * kRowThreads;
    if (c < nch) {
      float h[8], b[8];
      act8_values8(hc[k], hb[k], h);
      unpack8(res[k], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = r * gd[k][i] - h[i] * coef;
        h[i] = dRes ? b[i] + v : v;
      }
      dX[o + c] = pack8(h);
    }
  }
}

}  // namespace

slora_status rmsnorm_fwd_run(const void* X, const void* A, const void* g, int64_t T, int64_t d,
                             float eps, void* Hout, void* N, float* rstd, cudaStream_t st) {
  if (T == 0) return SLORA_OK;
  const int nch = int(d / 8);
  LaunchScope ls(kNorm, double(T) * d * 2 * (2 + (A ? 1 : 0) + (A && Hout ? 1 : 0)), st);
  const auto* x = static_cast<const uint4*>(X);
  const auto* a = static_cast<const uint4*>(A);
  const auto* gg = static_cast<const uint4*>(g);
  auto* h = static_cast<uint4*>(Hout);
  auto* n = static_cast<uint4*>(N);
  const unsigned rows = unsigned(T);
  if (nch <= kRowThreads) {
    rmsnorm_fwd_row_kernel<1><<<rows, kRowThreads, 0, st>>>(x, a, gg, nch, eps, h, n, rstd);
  } else if (nch <= 2 * kRowThreads) {
    rmsnorm_fwd_row_kernel<2><<<rows, kRowThreads, 0, st>>>(x, a, gg, nch, eps, h, n, rstd);
  } else if (nch <= 4 * kRowThreads) {
    rmsnorm_fwd_row_kernel<4><<<rows, kRowThreads, 0, st>>>(x, a, gg, nch, eps, h, n, rstd);
  } else if (nch <= 8 * kRowThreads) {
    rmsnorm_fwd_row_kernel<8><<<rows, kRowThreads, 0, st>>>(x, a, gg, nch, eps, h, n, rstd);
  } else if (nch <= 16 * kRowThreads) {
    rmsnorm_fwd_row_kernel<16><<<rows, kRowThreads, 0, st>>>(x, a, gg, nch, eps, h, n, rstd);
  } else {
    rmsnorm_fwd_kernel<<<unsigned((T + 7) / 8), 256, 0, st>>>(x, a, gg, T, nch, eps, h, n, rstd);
  }
  SLORA_CHECK_LAUNCH();
  return SLORA_OK;
}

slora_status rmsnorm_bwd_run(const void* Hin, const float* rstd, const void* g, const void* dN0,
                             const void* dN1, const void* dN2, const void* dRes, int64_t T,
                             int64_t d, void* dX, cudaStream_t st) {
  if (T == 0) return SLORA_OK;
  const int nch = int(d / 8);
  const int nin = 2 + (dN0 ? 1 : 0) + (dN1 ? 1 : 0) + (dN2 ? 1 : 0) + (dRes ? 1 : 0);
  LaunchScope ls(kNorm, double(T) * d * 2 * nin, st);
  const auto* hin = static_cast<const uint4*>(Hin);
  const auto* gg = static_cast<const uint4*>(g);
  const auto* n0 = static_cast<const uint4*>(dN0);
  const auto* n1 = static_cast<const uint4*>(dN1);
  const auto* n2 = static_cast<const uint4*>(dN2);
  const auto* res = static_cast<const uint4*>(dRes);
  auto* dx = static_cast<uint4*>(dX);
  const unsigned rows = unsigned(T);
  if (nch <= kRowThreads) {
    rmsnorm_bwd_row_kernel<1><<<rows, kRowThreads, 0, st>>>(hin, rstd, gg, n0, n1, n2, res, nch, dx);
  } else if (nch <= 2 * kRowThreads) {
    rmsnorm_bwd_row_kernel<2><<<rows, kRowThreads, 0, st>>>(hin, rstd, gg, n0, n1, n2, res, nch, dx);
  } else if (nch <= 4 * kRowThreads) {
    rmsnorm_bwd_row_kernel<4><<<rows, kRowThreads, 0, st>>>(hin, rstd, gg, n0, n1, n2, res, nch, dx);
  } else if (nch <= 8 * kRowThreads) {
    rmsnorm_bwd_row_kernel<8><<<rows, kRowThreads, 0, st>>>(hin, rstd, gg, n0, n1, n2, res, nch, dx);
  } else if (nch <= 16 * kRowThreads) {
    rmsnorm_bwd_row_kernel<16><<<rows, kRowThreads, 0, st>>>(hin, rstd, gg, n0, n1, n2, res, nch,
                                                             dx);
  } else {
    rmsnorm_bwd_kernel<<<unsigned((T + 7) / 8), 256, 0, st>>>(hin, rstd, gg, n0, n1, n2, res, T,
                                                             nch, dx);
  }
  SLORA_CHECK_LAUNCH();
  return SLORA_OK;
}

// Levels of 128 chunks in as few parts of at most four as hold them, evenly.
#define SLORA_ROW(KERNEL, CPT, PARTS, ...)                                                    \
  SLORA_CUDA(launch_early(KERNEL<CPT, PARTS>, dim3(rows), kRowThreads * PARTS, 0, st, __VA_ARGS__))
#define SLORA_ROW_SWITCH(KERNEL, ...)                                \
  switch ((nch + kRowThreads - 1) / kRowThreads) {                   \
    case 1: SLORA_ROW(KERNEL, 1, 1, __VA_ARGS__); break;             \
    case 2: SLORA_ROW(KERNEL, 2, 1, __VA_ARGS__); break;             \
    case 3: SLORA_ROW(KERNEL, 3, 1, __VA_ARGS__); break;             \
    case 4: SLORA_ROW(KERNEL, 4, 1, __VA_ARGS__); break;             \
    case 5: case 6: SLORA_ROW(KERNEL, 3, 2, __VA_ARGS__); break;     \
    case 7: case 8: SLORA_ROW(KERNEL, 4, 2, __VA_ARGS__); break;     \
    case 9: SLORA_ROW(KERNEL, 3, 3, __VA_ARGS__); break;             \
    case 10: case 11: case 12:                                       \
      SLORA_ROW(KERNEL, 4, 3, __VA_ARGS__);                          \
      break;                                                         \
    default: SLORA_ROW(KERNEL, 4, 4, __VA_ARGS__);                   \
  }

slora_status rmsnorm_fwd_act8_run(const void* X, const void* A, const void* g, int64_t T,
                                  int64_t d, float eps, void* Hout, void* N, float* rstd,
                                  const slora_act8* H8, const slora_act8* N8, cudaStream_t st) {
  if (T == 0) return SLORA_OK;
  const int nch = int(d / 8);
  LaunchScope ls(kNorm, double(T) * d * (2.0 * (2 + (A ? 1 : 0) + (A && Hout ? 1 : 0)) +
                                         1.03125 * ((H8 ? 1 : 0) + (N8 ? 1 : 0))), st);
  const auto* x = static_cast<const uint4*>(X);
  const auto* a = static_cast<const uint4*>(A);
  const auto* gg = static_cast<const uint4*>(g);
  auto* h = static_cast<uint4*>(Hout);
  auto* n = static_cast<uint4*>(N);
  uint2* h8 = H8 ? reinterpret_cast<uint2*>(H8->codes) : nullptr;
  uint8_t* h8s = H8 ? H8->scales : nullptr;
  uint2* n8 = N8 ? reinterpret_cast<uint2*>(N8->codes) : nullptr;
  uint8_t* n8s = N8 ? N8->scales : nullptr;
  const unsigned rows = unsigned(T);
  SLORA_ROW_SWITCH(rmsnorm_fwd_act8_kernel, x, a, gg, nch, eps, h, n, rstd, h8, h8s, n8, n8s)
  return SLORA_OK;
}

slora_status rmsnorm_bwd_act8_run(const slora_act8& H8, const float* rstd, const void* g,
                                  const void* dN0, const void* dN1, const void* dN2,
                                  const void* dRes, int64_t T, int64_t d, void* dX,
                                  cudaStream_t st) {
  if (T == 0) return SLORA_OK;
  const int nch = int(d / 8);
  const int nin = 2 + (dN1 ? 1 : 0) + (dN2 ? 1 : 0) + (dRes ? 1 : 0);
  LaunchScope ls(kNorm, double(T) * d * (2.0 * nin + 1.03125), st);
  const auto* h8 = reinterpret_cast<const uint2*>(H8.codes);
  const auto* gg = static_cast<const uint4*>(g);
  const auto* n0 = static_cast<const uint4*>(dN0);
  const auto* n1 = static_cast<const uint4*>(dN1);
  const auto* n2 = static_cast<const uint4*>(dN2);
  const auto* res = static_cast<const uint4*>(dRes);
  auto* dx = static_cast<uint4*>(dX);
  const unsigned rows = unsigned(T);
  SLORA_ROW_SWITCH(rmsnorm_bwd_act8_kernel, h8, H8.scales, rstd, gg, n0, n1, n2, res, nch, dx)
  return SLORA_OK;
}

}  // namespace slora
