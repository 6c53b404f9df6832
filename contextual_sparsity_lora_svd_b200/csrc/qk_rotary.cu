// Rotation of the q and k rows by their positions, with an optional RMS norm
// of every head before it, forward and backward.
//
// Mathematics, per head x of hd channels (SparseLoRA article, section 1: q/k
// channels are kept per head; sections 3 and 6: a context row's skipped
// channels are not computed, so they are zero here and their gradient is
// dropped):
//   forward   y = R(n),  n = x r g,  r = 1 / sqrt(mean(x^2) + eps)
//   backward  dn = R^T dy;  u = g dn;  dx = r u - x r^3 mean(x u);
//             dg = sum over rows and heads of dn x r
// R turns pair p of the leading `dims` channels by pos * f_p; the remaining
// channels are pairs of angle 0.  r is recomputed in the backward: the head is
// in registers anyway, so no statistic is stored between the two.
//
// Angles: f_p / 2 pi is held in units of 2^-64 turn, so pos * f_p modulo one
// turn is one wrapping 64-bit product, exact at every position, and
// sin and cos take an argument in [-1, 1) half turns.  A product in fp32 is off
// by 4e-3 rad at position 100000.
//
// Bound: memory.  Forward 2 + 2 bytes a channel, backward 2 + 4 + 2 (fp32 dy).
// A team of lanes owns one head (V pairs a lane: two 16-byte loads at V = 8),
// so the norm is a few shuffles and every value is read and written once.  A
// block takes R rows of one tensor at a time, computes their R * hd / 2
// sines and cosines once into shared memory (sincospi costs about as much as
// four heads' rotation) and its teams walk the rows' heads, loading one head
// ahead.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "qk_rotary.cuh"

namespace slora {

__device__ int g_qk_bad_index = 0;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;  // rows of a chunk

struct QkPart {
  const void* X;
  long long ldx;
  const void *Xc, *Xo;
  const int32_t* inv;
  int n_idx;
  const void* g;
  void* out;  // Y, or dX
  long long ldo;
  void *outc, *outo;
  const void* dY;
  long long ldy;
  float* dgp;  // [blocks of this part][hd] partial sums of dg, or null
  int heads, blocks;
};
struct QkParams {
  QkPart part[2];
  unsigned long long turns[kMaxHeadDim / 2];
  const int32_t* pos;
  const int32_t* ctx_off;  // sliced: context rows before sequence b, [batch + 1]
  long long T;
  int seq, hd, dims, R, units, tl;
  float eps, mscale;
};

template <typename T, int V>
struct alignas(V * sizeof(T) >= 16 ? 16 : V * sizeof(T)) Raw {
  T v[V];
};
// V consecutive elements in as few loads as their size allows (16 bytes each).
template <typename T, int V>
__device__ __forceinline__ void ld_vec(const T* p, Raw<T, V>& r) {
  constexpr int B = V * int(sizeof(T));
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i)
      reinterpret_cast<uint4*>(r.v)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (B == 8) {
    *reinterpret_cast<uint2*>(r.v) = *reinterpret_cast<const uint2*>(p);
  } else if constexpr (B == 4) {
    *reinterpret_cast<uint32_t*>(r.v) = *reinterpret_cast<const uint32_t*>(p);
  } else {
    r.v[0] = p[0];
  }
}
template <typename T, int V>
__device__ __forceinline__ void st_vec(T* p, const Raw<T, V>& r) {
  constexpr int B = V * int(sizeof(T));
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(r.v)[i];
  } else if constexpr (B == 8) {
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(r.v);
  } else if constexpr (B == 4) {
    *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(r.v);
  } else {
    p[0] = r.v[0];
  }
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else return __float2bfloat16_rn(x);
}

// A lane's two groups of V channels of one unit: pair i of the unit is
// (lo[i], hi[i]).  Half layout: group A holds the first members, group B the
// second.  Interleaved: A then B hold 2V consecutive channels.
template <int V, bool kInter>
struct Pairs {
  static __device__ __forceinline__ void split(const float (&a)[V], const float (&b)[V],
                                               float (&lo)[V], float (&hi)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (kInter && V > 1) {
        lo[i] = 2 * i < V ? a[(2 * i) % V] : b[(2 * i) % V];
        hi[i] = 2 * i < V ? a[(2 * i + 1) % V] : b[(2 * i + 1) % V];
      } else {
        lo[i] = a[i];
        hi[i] = b[i];
      }
    }
  }
  static __device__ __forceinline__ void join(const float (&lo)[V], const float (&hi)[V],
                                              float (&a)[V], float (&b)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (kInter && V > 1) {
        a[e] = e % 2 ? hi[e / 2] : lo[e / 2];
        b[e] = e % 2 ? hi[(V + e) / 2] : lo[(V + e) / 2];
      } else {
        a[e] = lo[e];
        b[e] = hi[e];
      }
    }
  }
};

// Units a lane owns: V = 8 covers 256 channels with 16 lanes; narrower
// vectors need two or four units on 32 lanes.
template <int V>
constexpr int units_per_lane() {
  return V == 8 ? 1 : (V == 2 ? 2 : 4);
}

// One head's raw rows in flight.
template <typename T, typename G, int V, bool kBwd>
struct Item {
  Raw<T, V> xa[units_per_lane<V>()], xb[units_per_lane<V>()];
  Raw<G, V> ya[kBwd ? units_per_lane<V>() : 1], yb[kBwd ? units_per_lane<V>() : 1];
};

template <typename T, typename G, int V, bool kInter, bool kBwd, bool kSliced>
__global__ void __launch_bounds__(kThreads) qk_rotary_kernel(const __grid_constant__ QkParams P) {
  constexpr int NU = units_per_lane<V>();
  extern __shared__ __align__(16) float2 tab[];  // [R][V / 2][units][2] (V = 1: [R][units])
  __shared__ unsigned long long s_turns[kMaxHeadDim / 2];
  __shared__ int s_kind[kMaxRows];  // sliced: context row, or -1 - output row
  __shared__ float s_red[kBwd ? kThreads / 32 : 1][kBwd ? kMaxHeadDim : 1];
  const int tid = threadIdx.x;
  const bool second = int(blockIdx.x) >= P.part[0].blocks;
  const QkPart& q = P.part[second ? 1 : 0];
  const int blk = int(blockIdx.x) - (second ? P.part[0].blocks : 0);
  const int hd = P.hd, dims = P.dims, np = hd / 2, U = P.units, tl = P.tl;
  for (int p = tid; p < dims / 2; p += kThreads) s_turns[p] = P.turns[p];

  // this lane's place: team `team` of the block, units lt, lt + tl, ...
  const int lt = tid % tl, nteams = kThreads / tl;
  const int team = tid / tl, team0 = (tid & ~31) / tl;  // first team of this warp
  int offa[NU], offb[NU];
  bool act[NU];
  float glo[NU][V], ghi[NU][V];
  const bool norm = q.g != nullptr;
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    const int u = lt + j * tl, p0 = u * V;
    act[j] = u < U;
    if (kInter) {
      offa[j] = 2 * p0;
      offb[j] = 2 * p0 + V;
    } else if (p0 < dims / 2) {
      offa[j] = p0;
      offb[j] = p0 + dims / 2;
    } else {
      offa[j] = p0 + dims / 2;          // dims + (p0 - dims / 2)
      offb[j] = offa[j] + np - dims / 2;  // + half of the unrotated channels
    }
    float a[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = b[i] = 1.0f;
    if (norm && act[j]) {
      const T* g = static_cast<const T*>(q.g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[i] = to_f(g[offa[j] + i]);
        b[i] = to_f(g[offb[j] + i]);
      }
    }
    Pairs<V, kInter>::split(a, b, glo[j], ghi[j]);
  }
  float dglo[kBwd ? NU : 1][V], dghi[kBwd ? NU : 1][V];
  if constexpr (kBwd) {
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) dglo[j][i] = dghi[j][i] = 0.0f;
  }

  const long long nchunks = (P.T + P.R - 1) / P.R;
  const int dr = nteams / q.heads, dh = nteams % q.heads;
  for (long long ch = blk; ch < nchunks; ch += q.blocks) {
    const long long t0 = ch * P.R;
    const int nrow = int(min((long long)P.R, P.T - t0));
    const int place = P.pos ? 0 : int(t0 % P.seq);  // of the chunk's first row in its sequence
    __syncthreads();  // the previous chunk's table has been read (and s_turns is written)
    for (int e = tid; e < nrow * np; e += kThreads) {
      const int r = e / np, p = e - r * np;
      float s = 0.0f, c = 1.0f;
      if (p < dims / 2) {
        const long long pos = P.pos ? P.pos[t0 + r] : int(unsigned(place + r) % unsigned(P.seq));
        const unsigned long long turn = (unsigned long long)pos * s_turns[p];
        // the top 32 bits as a signed fraction: half turns in [-1, 1)
        sincospif(float(int(turn >> 32)) * 4.656612873077393e-10f, &s, &c);
        s *= P.mscale;
        c *= P.mscale;
      }
      const int at = V == 1 ? r * U + p
                            : ((r * (V / 2) + (p % V) / 2) * U + p / V) * 2 + (p & 1);
      tab[at] = make_float2(c, s);
    }
    if constexpr (kSliced) {
      if (tid < nrow) {
        const long long t = t0 + tid;
        const int b = int(t / P.seq), i = int(t % P.seq);
        const int o0 = P.ctx_off[b], o1 = P.ctx_off[b + 1];
        s_kind[tid] = i < o1 - o0 ? o0 + i : int(-1 - (t - o1));
      }
    }
    __syncthreads();

    const int items = nrow * q.heads;
    auto load = [&](int r, int h, bool valid, Item<T, G, V, kBwd>& it) {
      if (!valid) return;
      const long long t = t0 + r;
      const T* x = nullptr;
      int kind = -1;
      if constexpr (kSliced) {
        kind = s_kind[r];
        if (kind < 0)
          x = static_cast<const T*>(q.Xo) + (long long)(-1 - kind) * q.heads * hd + h * hd;
        else
          x = static_cast<const T*>(q.Xc) + (long long)kind * q.n_idx;
      } else {
        x = static_cast<const T*>(q.X) + t * q.ldx + h * hd;
      }
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        if (!act[j]) continue;
        if (!kBwd || norm) {
          if (kSliced && kind >= 0) {
            const int32_t* inv = q.inv + h * hd;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const int ia = inv[offa[j] + i], ib = inv[offb[j] + i];
              it.xa[j].v[i] = ia >= 0 ? x[ia] : from_f<T>(0.0f);
              it.xb[j].v[i] = ib >= 0 ? x[ib] : from_f<T>(0.0f);
            }
          } else {
            ld_vec(x + offa[j], it.xa[j]);
            ld_vec(x + offb[j], it.xb[j]);
          }
        }
        if constexpr (kBwd) {
          const G* y = static_cast<const G*>(q.dY) + t * q.ldy + h * hd;
          ld_vec(y + offa[j], it.ya[j]);
          ld_vec(y + offb[j], it.yb[j]);
        }
      }
    };
    auto table = [&](int r, int j, float2 (&cs)[V]) {
      const int u = lt + j * tl;
      if constexpr (V == 1) {
        cs[0] = tab[r * U + u];
      } else {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
          const float4 f = reinterpret_cast<const float4*>(tab)[(r * (V / 2) + k) * U + u];
          cs[2 * k] = make_float2(f.x, f.y);
          cs[2 * k + 1] = make_float2(f.z, f.w);
        }
      }
    };
    auto team_sum = [&](float v) {
      for (int s = tl >> 1; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
      return v;
    };
    auto store = [&](int r, int h, int j, const float (&lo)[V], const float (&hi)[V]) {
      float a[V], b[V];
      Pairs<V, kInter>::join(lo, hi, a, b);
      Raw<T, V> ra, rb;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ra.v[i] = from_f<T>(a[i]);
        rb.v[i] = from_f<T>(b[i]);
      }
      T* o;
      if constexpr (kSliced && kBwd) {
        const int kind = s_kind[r];
        if (kind >= 0) {
          T* oc = static_cast<T*>(q.outc) + (long long)kind * q.n_idx;
          const int32_t* inv = q.inv + h * hd;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int ia = inv[offa[j] + i], ib = inv[offb[j] + i];
            if (ia >= 0) oc[ia] = ra.v[i];
            if (ib >= 0) oc[ib] = rb.v[i];
          }
          return;
        }
        o = static_cast<T*>(q.outo) + (long long)(-1 - kind) * q.heads * hd + h * hd;
      } else {
        o = static_cast<T*>(q.out) + (t0 + r) * q.ldo + h * hd;
      }
      st_vec(o + offa[j], ra);
      st_vec(o + offb[j], rb);
    };
    auto compute = [&](int r, int h, bool valid, const Item<T, G, V, kBwd>& it) {
      float xlo[NU][V], xhi[NU][V];
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        float a[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const bool on = valid && act[j] && (!kBwd || norm);
          a[i] = on ? to_f(it.xa[j].v[i]) : 0.0f;
          b[i] = on ? to_f(it.xb[j].v[i]) : 0.0f;
          ss += a[i] * a[i] + b[i] * b[i];
        }
        Pairs<V, kInter>::split(a, b, xlo[j], xhi[j]);
      }
      float rs = 1.0f;
      if (norm) rs = rsqrtf(team_sum(ss) / float(hd) + P.eps);
      if constexpr (!kBwd) {
        if (!valid) return;
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          if (!act[j]) continue;
          float2 cs[V];
          table(r, j, cs);
          float lo[V], hi[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float l = norm ? xlo[j][i] * rs * glo[j][i] : xlo[j][i];
            const float m = norm ? xhi[j][i] * rs * ghi[j][i] : xhi[j][i];
            lo[i] = l * cs[i].x - m * cs[i].y;
            hi[i] = m * cs[i].x + l * cs[i].y;
          }
          store(r, h, j, lo, hi);
        }
      } else {
        float dlo[NU][V], dhi[NU][V];  // dn = R^T dy
        float dot = 0.0f;              // sum of x g dn
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          const bool on = valid && act[j];
          float a[V], b[V], lo[V], hi[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            a[i] = on ? to_f(it.ya[j].v[i]) : 0.0f;
            b[i] = on ? to_f(it.yb[j].v[i]) : 0.0f;
          }
          Pairs<V, kInter>::split(a, b, lo, hi);
          float2 cs[V];
          if (on) table(r, j, cs);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float c = on ? cs[i].x : 1.0f, s = on ? cs[i].y : 0.0f;
            dlo[j][i] = lo[i] * c + hi[i] * s;
            dhi[j][i] = hi[i] * c - lo[i] * s;
            dot += xlo[j][i] * glo[j][i] * dlo[j][i] + xhi[j][i] * ghi[j][i] * dhi[j][i];
          }
        }
        if (norm) {
          const float coef = rs * rs * rs * (team_sum(dot) / float(hd));
#pragma unroll
          for (int j = 0; j < NU; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              dglo[j][i] += dlo[j][i] * (xlo[j][i] * rs);
              dghi[j][i] += dhi[j][i] * (xhi[j][i] * rs);
              dlo[j][i] = rs * (glo[j][i] * dlo[j][i]) - xlo[j][i] * coef;
              dhi[j][i] = rs * (ghi[j][i] * dhi[j][i]) - xhi[j][i] * coef;
            }
        }
        if (!valid) return;
#pragma unroll
        for (int j = 0; j < NU; ++j)
          if (act[j]) store(r, h, j, dlo[j], dhi[j]);
      }
    };

    // the next head's rows load while this one is computed; every lane of a
    // warp runs the same number of rounds (the team sums are warp-wide)
    int r = team / q.heads, h = team % q.heads;
    Item<T, G, V, kBwd> cur, nxt;
    load(r, h, team < items, cur);
    for (int base = team0; base < items; base += nteams) {
      const int it = base + (team - team0);
      int r2 = r + dr, h2 = h + dh;
      if (h2 >= q.heads) {
        h2 -= q.heads;
        ++r2;
      }
      load(r2, h2, it + nteams < items, nxt);
      compute(r, h, it < items, cur);
      cur = nxt;
      r = r2;
      h = h2;
    }
  }

  if constexpr (kBwd) {
    if (!q.dgp) return;
    // this block's dg: lanes of a warp that own the same channels, then the
    // warps in order
#pragma unroll
    for (int j = 0; j < NU; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        for (int s = tl; s < 32; s <<= 1) {
          dglo[j][i] += __shfl_xor_sync(0xffffffffu, dglo[j][i], s);
          dghi[j][i] += __shfl_xor_sync(0xffffffffu, dghi[j][i], s);
        }
      float a[V], b[V];
      Pairs<V, kInter>::join(dglo[j], dghi[j], a, b);
      if (act[j] && (tid & 31) < tl) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s_red[tid >> 5][offa[j] + i] = a[i];
          s_red[tid >> 5][offb[j] + i] = b[i];
        }
      }
    }
    __syncthreads();
    for (int c = tid; c < hd; c += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) v += s_red[w][c];
      q.dgp[(long long)blk * hd + c] = v;
    }
  }
}

// dg of each part: the blocks' partial sums, 32 channels a block, 32 groups of
// partials a channel added in a fixed order.
struct DgParams {
  const float* part[2];
  float* dg[2];
  int blocks[2];
  int hd;
};
__global__ void __launch_bounds__(1024) qk_dg_kernel(const __grid_constant__ DgParams p) {
  __shared__ float red[32][33];
  const int which = blockIdx.y, cl = threadIdx.x & 31, gr = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cl;
  if (!p.dg[which]) return;
  float v = 0.0f;
  if (c < p.hd)
    for (int b = gr; b < p.blocks[which]; b += 32)
      v += p.part[which][(long long)b * p.hd + c];
  red[gr][cl] = v;
  __syncthreads();
  if (gr == 0 && c < p.hd) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][cl];
    p.dg[which][c] = s;
  }
}

// Sliced rows: block 0 and 1 invert the channel lists (inv[channel] = column,
// or -1), block 2 writes the context rows before every sequence.
template <int CAP>
struct SliceParams {
  const int32_t* idx[2];
  int32_t* inv[2];
  int n_idx[2], n[2];
  int32_t* ctx_off;
  int batch;
  int ctx_len[CAP];
};
template <int CAP>
__global__ void __launch_bounds__(1024) qk_slice_kernel(const __grid_constant__ SliceParams<CAP> p) {
  if (blockIdx.x < 2) {
    const int w = blockIdx.x;
    if (!p.inv[w]) return;
    for (int i = threadIdx.x; i < p.n[w]; i += blockDim.x) p.inv[w][i] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n_idx[w]; i += blockDim.x) {
      const int c = p.idx[w][i];
      if (c < 0 || c >= p.n[w] || atomicCAS(&p.inv[w][c], -1, i) != -1)
        atomicExch(&g_qk_bad_index, 1);
    }
    return;
  }
  // exclusive scan of ctx_len, 1024 sequences at a time (batch is at most kMaxBatch)
  __shared__ int part[1024];
  int carry = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    const int own = b < p.batch ? p.ctx_len[b] : 0;
    part[threadIdx.x] = own;
    __syncthreads();
    for (int s = 1; s < 1024; s <<= 1) {
      const int add = threadIdx.x >= s ? part[threadIdx.x - s] : 0;
      __syncthreads();
      part[threadIdx.x] += add;
      __syncthreads();
    }
    if (b < p.batch) p.ctx_off[b + 1] = carry + part[threadIdx.x];
    if (b == 0) p.ctx_off[0] = 0;
    carry += part[1023];
    __syncthreads();
  }
}

template <int CAP>
void launch_slices(const QkDesc& D, const slora_tokens* tok, int32_t* const* inv, int32_t* ctx_off,
                   cudaStream_t st) {
  SliceParams<CAP> p{};
  for (int i = 0; i < D.nparts; ++i) {
    if (!D.part[i].idx) continue;
    p.idx[i] = D.part[i].idx;
    p.inv[i] = inv[i];
    p.n_idx[i] = D.part[i].n_idx;
    p.n[i] = D.part[i].heads * D.head_dim;
  }
  p.ctx_off = ctx_off;
  p.batch = D.ti.batch;
  for (int b = 0; b < D.ti.batch; ++b) p.ctx_len[b] = tok->ctx_len[b];
  qk_slice_kernel<CAP><<<3, 1024, 0, st>>>(p);
}

template <typename T, typename G, int V, bool kInter, bool kBwd, bool kSliced>
slora_status launch(const QkParams& P, int grid, cudaStream_t st) {
  const int smem = P.R * (P.hd / 2) * int(sizeof(float2));  // at most 8 KB
  qk_rotary_kernel<T, G, V, kInter, kBwd, kSliced><<<grid, kThreads, smem, st>>>(P);
  SLORA_CHECK_LAUNCH();
  return SLORA_OK;
}
template <typename T, typename G, int V, bool kInter, bool kBwd>
slora_status launch_s(bool sliced, const QkParams& P, int grid, cudaStream_t st) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    if (sliced) return launch<T, G, V, kInter, kBwd, true>(P, grid, st);
  }
  return launch<T, G, V, kInter, kBwd, false>(P, grid, st);
}
template <typename T, typename G, bool kBwd>
slora_status launch_v(int V, bool inter, bool sliced, const QkParams& P, int grid,
                      cudaStream_t st) {
  if (V == 8)
    return inter ? launch_s<T, G, 8, true, kBwd>(sliced, P, grid, st)
                 : launch_s<T, G, 8, false, kBwd>(sliced, P, grid, st);
  if (V == 2)
    return inter ? launch_s<T, G, 2, true, kBwd>(sliced, P, grid, st)
                 : launch_s<T, G, 2, false, kBwd>(sliced, P, grid, st);
  return inter ? launch_s<T, G, 1, true, kBwd>(sliced, P, grid, st)
               : launch_s<T, G, 1, false, kBwd>(sliced, P, grid, st);
}

// The widest vector (in channels of one group) that every row of the call
// takes: 16-byte accesses at 8, pairs at 2.  A unit may not straddle the
// members of a pair, so in the half layout the width divides both halves.
int vector_width(const QkDesc& D, bool backward) {
  for (int V : {8, 2}) {
    bool ok = D.rot.inter ? D.head_dim % (2 * V) == 0
                          : (D.rot.dims / 2) % V == 0 && (D.head_dim / 2 - D.rot.dims / 2) % V == 0;
    for (int i = 0; i < D.nparts && ok; ++i) {
      const slora_qk_rows& q = D.part[i];
      if (!q.idx && (!backward || q.g)) ok = ok && q.ldx % V == 0;
      if (!backward) ok = ok && q.ldy % V == 0;
      else ok = ok && q.lddy % V == 0 && (q.idx || q.lddx % V == 0);
    }
    if (ok) return V;
  }
  return 1;
}

constexpr int kBlocksPerSm = 4;

int grid_blocks() { return num_sms() * kBlocksPerSm; }

}  // namespace

slora_status rotary_plan(const char* fn, const slora_rotary* rot, int head_dim, RotaryPlan* out) {
  if (!rot) SLORA_FAIL(SLORA_ERR_INVALID_ARG, "%s: rot is NULL", fn);
  if (head_dim < 2 || head_dim > kMaxHeadDim || head_dim % 2)
    SLORA_FAIL(SLORA_ERR_SHAPE, "%s: head_dim %d must be even, 2 .. %d", fn, head_dim, kMaxHeadDim);
  const int dims = rot->dims == 0 ? head_dim : rot->dims;
  if (dims < 2 || dims > head_dim || dims % 2)
    SLORA_FAIL(SLORA_ERR_SHAPE, "%s: rotated dims %d must be even, 2 .. head_dim", fn, rot->dims);
  if (rot->layout != SLORA_ROTARY_HALF && rot->layout != SLORA_ROTARY_INTERLEAVED)
    SLORA_FAIL(SLORA_ERR_INVALID_ARG, "%s: unknown rotary layout %d", fn, rot->layout);
  if (rot->scaling < SLORA_ROTARY_PLAIN || rot->scaling > SLORA_ROTARY_YARN)
    SLORA_FAIL(SLORA_ERR_INVALID_ARG, "%s: unknown rotary scaling %d", fn, rot->scaling);
  if (!(rot->base > 1.0) || !std::isfinite(rot->base))
    SLORA_FAIL(SLORA_ERR_INVALID_ARG, "%s: rotary base %g must be a finite value > 1", fn, rot->base);
  const bool scaled = rot->scaling != SLORA_ROTARY_PLAIN;
  const double s = scaled ? rot->factor : 1.0;
  if (!(s >= 1.0) || !std::isfinite(s))
    SLORA_FAIL(SLORA_ERR_INVALID_ARG, "%s: rotary factor %g must be a finite value >= 1", fn, s);
  if (!(rot->mscale >= 0.0) || !std::isfinite(rot->mscale))
    SLORA_FAIL(SLORA_ERR_INVALID_ARG, "%s: rotary mscale %g must be finite and >= 0", fn, rot->mscale);
  const bool bands = rot->scaling == SLORA_ROTARY_BANDS, yarn = rot->scaling == SLORA_ROTARY_YARN;
  double low = rot->low, high = rot->high;
  if (low == 0.0 && high == 0.0) {
    low = 1.0;
    high = bands ? 4.0 : 32.0;
  }
  if (bands || yarn) {
    if (rot->orig_len < 1)
      SLORA_FAIL(SLORA_ERR_SHAPE, "%s: orig_len %d must be positive", fn, rot->orig_len);
    if (!(low > 0.0 && low < high) || !std::isfinite(high))
      SLORA_FAIL(SLORA_ERR_INVALID_ARG, "%s: rotary turns low %g, high %g: 0 < low < high", fn, low,
                 high);
  }
  double base = rot->base;
  if (rot->scaling == SLORA_ROTARY_NTK) {
    if (dims < 4)
      SLORA_FAIL(SLORA_ERR_SHAPE, "%s: NTK scaling needs 4 rotated channels or more", fn);
    base *= std::pow(s, double(dims) / double(dims - 2));
    if (!std::isfinite(base))
      SLORA_FAIL(SLORA_ERR_INVALID_ARG, "%s: rotary base overflows at factor %g", fn, s);
  }
  const double two_pi = 6.283185307179586476925286766559;
  // YARN: the pairs (as a fraction) that make `high` and `low` turns, rounded outwards
  double ylo = 0.0, yhi = 0.0;
  if (yarn) {
    auto pair_of = [&](double turns) {
      return dims * std::log(double(rot->orig_len) / (two_pi * turns)) / (2.0 * std::log(base));
    };
    ylo = std::max(std::floor(pair_of(high)), 0.0);
    yhi = std::min(std::ceil(pair_of(low)), double(dims - 1));
  }
  auto clamp01 = [](double v) { return std::min(1.0, std::max(0.0, v)); };
  for (int p = 0; p < dims / 2; ++p) {
    const double f = std::pow(base, -2.0 * p / dims);
    double g = f;
    if (rot->scaling == SLORA_ROTARY_LINEAR) g = f / s;
    if (bands) {
      const double m = clamp01((rot->orig_len * f / two_pi - low) / (high - low));
      g = m * f + (1.0 - m) * f / s;
    }
    if (yarn) {
      const double m = clamp01((p - ylo) / std::max(yhi - ylo, 0.001));
      g = m * f / s + (1.0 - m) * f;
    }
    // g <= 1, so the turns stay below 2^64 / 2 pi
    out->turns[p] = (unsigned long long)std::llround(g / two_pi * 18446744073709551616.0);
  }
  out->inter = rot->layout == SLORA_ROTARY_INTERLEAVED;
  out->dims = dims;
  out->mscale = float(rot->mscale != 0.0 ? rot->mscale : (yarn ? 0.1 * std::log(s) + 1.0 : 1.0));
  return SLORA_OK;
}

slora_status qk_rotary_run(const QkDesc& D, bool backward, const slora_tokens* tok, Arena& ar,
                           bool plan, cudaStream_t st) {
  const int hd = D.head_dim;
  bool sliced = false, any_dg = false;
  for (int i = 0; i < D.nparts; ++i) {
    sliced = sliced || D.part[i].idx;
    any_dg = any_dg || (backward && D.part[i].g && D.part[i].dg);
  }
  const int max_blocks = grid_blocks();
  int32_t* inv[2] = {nullptr, nullptr};
  int32_t* ctx_off = nullptr;
  float* dgp = nullptr;
  if (sliced) {
    ctx_off = ar.take<int32_t>(size_t(D.ti.batch) + 1);
    for (int i = 0; i < D.nparts; ++i)
      if (D.part[i].idx) inv[i] = ar.take<int32_t>(size_t(D.part[i].heads) * hd);
  }
  // one partial of each block; the parts' blocks together are at most max_blocks + 1
  if (any_dg) dgp = ar.take<float>(size_t(max_blocks + 1) * hd);
  if (plan) return SLORA_OK;
  SLORA_TRY(arena_fits(ar, "qk_rotary"));

  if (sliced) {
    LaunchScope ls(kAux, double(D.ti.batch) * 4, st);
    if (D.ti.batch <= 64) launch_slices<64>(D, tok, inv, ctx_off, st);
    else launch_slices<kMaxBatch>(D, tok, inv, ctx_off, st);
    SLORA_CHECK_LAUNCH();
  }

  const int V = vector_width(D, backward);
  QkParams P{};
  P.pos = D.pos;
  P.ctx_off = ctx_off;
  P.T = D.ti.T;
  P.seq = D.ti.seq;
  P.hd = hd;
  P.dims = D.rot.dims;
  P.eps = D.eps;
  P.mscale = D.rot.mscale;
  std::copy(D.rot.turns, D.rot.turns + kMaxHeadDim / 2, P.turns);
  P.units = hd / 2 / V;
  const int nu = V == 8 ? 1 : (V == 2 ? 2 : 4);
  P.tl = 1;
  while (P.tl < 32 && P.tl * nu < P.units) P.tl *= 2;
  // rows of a chunk: eight share a table, fewer where the rows would not give
  // every block one
  P.R = int(std::min<int64_t>(kMaxRows, std::max<int64_t>(1, D.ti.T / max_blocks)));
  const int64_t nchunks = (D.ti.T + P.R - 1) / P.R;
  int heads = 0;
  for (int i = 0; i < D.nparts; ++i) heads += D.part[i].heads;
  int grid = 0;
  double bytes = 0.0;
  const double es = D.dt == kF32 ? 4 : 2, gs = D.gdt == kF32 ? 4 : 2;
  for (int i = 0; i < D.nparts; ++i) {
    const slora_qk_rows& s = D.part[i];
    QkPart& q = P.part[i];
    q.X = s.X; q.ldx = s.ldx; q.Xc = s.X_ctx; q.Xo = s.X_out;
    q.inv = inv[i]; q.n_idx = s.n_idx; q.g = s.g; q.heads = s.heads;
    if (backward) {
      q.out = s.dX; q.ldo = s.lddx; q.outc = s.dX_ctx; q.outo = s.dX_out;
      q.dY = s.dY; q.ldy = s.lddy;
    } else {
      q.out = s.Y; q.ldo = s.ldy;
    }
    // blocks in proportion to the heads
    const int64_t share = i == 0 ? std::max<int64_t>(1, int64_t(max_blocks) * s.heads / heads)
                                 : std::max<int64_t>(1, max_blocks - P.part[0].blocks);
    q.blocks = int(std::min<int64_t>(share, nchunks));
    if (any_dg && s.g && s.dg) q.dgp = dgp + int64_t(grid) * hd;
    grid += q.blocks;
    const double n = double(D.ti.T) * s.heads * hd;
    bytes += n * (backward ? (s.g ? es : 0) + gs + es : 2 * es);
  }
  {
    LaunchScope ls(kElementwise, bytes, st);
    const bool in = D.rot.inter != 0;
    if (!backward) {
      if (D.dt == kF32)
        SLORA_TRY((launch_v<float, float, false>(V, in, sliced, P, grid, st)));
      else
        SLORA_TRY((launch_v<__nv_bfloat16, float, false>(V, in, sliced, P, grid, st)));
    } else if (D.dt == kF32) {
      SLORA_TRY((launch_v<float, float, true>(V, in, sliced, P, grid, st)));
    } else if (D.gdt == kF32) {
      SLORA_TRY((launch_v<__nv_bfloat16, float, true>(V, in, sliced, P, grid, st)));
    } else {
      SLORA_TRY((launch_v<__nv_bfloat16, __nv_bfloat16, true>(V, in, sliced, P, grid, st)));
    }
  }
  if (any_dg) {
    DgParams d{};
    d.hd = hd;
    for (int i = 0; i < D.nparts; ++i) {
      d.part[i] = P.part[i].dgp;
      d.dg[i] = P.part[i].dgp ? D.part[i].dg : nullptr;
      d.blocks[i] = P.part[i].blocks;
    }
    LaunchScope ls(kAux, double(grid) * hd * 4, st);
    qk_dg_kernel<<<dim3(unsigned((hd + 31) / 32), unsigned(D.nparts)), 1024, 0, st>>>(d);
    SLORA_CHECK_LAUNCH();
  }
  return SLORA_OK;
}

slora_status qk_check_error(bool clear) {
  int v = 0;
  SLORA_CUDA(cudaDeviceSynchronize());
  SLORA_CUDA(cudaMemcpyFromSymbol(&v, g_qk_bad_index, sizeof(int)));
  if (clear && v) {
    const int z = 0;
    SLORA_CUDA(cudaMemcpyToSymbol(g_qk_bad_index, &z, sizeof(int)));
  }
  if (v)
    SLORA_FAIL(SLORA_ERR_INVALID_ARG,
               "a channel list of a sliced q or k held an entry outside its channels or one twice");
  return SLORA_OK;
}

}  // namespace slora
