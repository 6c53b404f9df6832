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
// Bound: memory.  Forward 2 + 2 bytes a channel, backward 2 + 4 + 2 (fp32 dy);
// the arithmetic is close behind, so it runs on packed pairs of fp32 values
// (fma.rn.f32x2).  A team of lanes owns one head (V pairs a lane: two 16-byte
// loads at V = 8), so the norm is a few shuffles and every value is read and
// written once.  A warp owns one row at a time, or a share of its heads where
// rows are few: it computes the row's hd / 2 sines and cosines once, spread
// over its lanes, keeps each lane's in registers and walks the heads, loading
// one head ahead.  Nothing in the loop waits for another warp.
//
// Sliced rows: the inverse channel list lies in shared memory, and a context
// row's compact channels are staged there with wide loads, gathered from (and
// in the backward scattered back to) by channel, and stored with wide stores.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "qk_rotary.cuh"

namespace slora {

__device__ int g_qk_bad_index = 0;

namespace {

constexpr int kWarps = 8;  // of a block, fewer where sliced rows need the shared memory

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
  int chunks, per_chunk;  // a row's heads in `chunks` shares of per_chunk
};
struct QkParams {
  QkPart part[2];
  unsigned long long turns[kMaxHeadDim / 2];
  const int32_t* pos;
  const int32_t* ctx_off;  // sliced: context rows before sequence b, [batch + 1]
  int T, seq, hd, dims, units, tl;
  int stage;  // sliced: elements of a warp's staged row (a multiple of 8)
  float eps, mscale;
};

// Two fp32 values as one operand of the packed instructions.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

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
// Packed pairs of a unit (V = 1: the second value of the one is zero).
template <int V>
constexpr int packs() {
  return V == 1 ? 1 : V / 2;
}
template <int V>
__device__ __forceinline__ void pack_all(const float (&v)[V], f2 (&p)[packs<V>()]) {
  if constexpr (V == 1) {
    p[0] = pack2(v[0], 0.0f);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = pack2(v[2 * i], v[2 * i + 1]);
  }
}
template <int V>
__device__ __forceinline__ void unpack_all(const f2 (&p)[packs<V>()], float (&v)[V]) {
  if constexpr (V == 1) {
    float z;
    unpack2(p[0], v[0], z);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) unpack2(p[i], v[2 * i], v[2 * i + 1]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void zero(Raw<T, V>& r) {
#pragma unroll
  for (int i = 0; i < V; ++i) r.v[i] = from_f<T>(0.0f);
}
// Raw groups of a unit to its packed first and second members.
template <typename T, int V, bool kInter>
__device__ __forceinline__ void members(const Raw<T, V>& ra, const Raw<T, V>& rb,
                                        f2 (&lo)[packs<V>()], f2 (&hi)[packs<V>()]) {
  float a[V], b[V], l[V], h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    a[i] = to_f(ra.v[i]);
    b[i] = to_f(rb.v[i]);
  }
  Pairs<V, kInter>::split(a, b, l, h);
  pack_all<V>(l, lo);
  pack_all<V>(h, hi);
}

// One head's rows in flight (zeros where this lane has none).
template <typename T, typename G, int V, bool kBwd>
struct Item {
  static constexpr int NU = units_per_lane<V>();
  Raw<T, V> xa[NU], xb[NU];
  Raw<G, V> ya[kBwd ? NU : 1], yb[kBwd ? NU : 1];
};

template <typename T, typename G, int V, bool kInter, bool kBwd, bool kSliced>
__global__ void __launch_bounds__(kWarps * 32, kBwd ? 2 : 3)
    qk_rotary_kernel(const __grid_constant__ QkParams P) {
  constexpr int NU = units_per_lane<V>(), NP = packs<V>();
  // [warps][hd / 2] cosines and sines (the backward's dg at the end), then for
  // sliced rows the inverse channel list and the warps' staged rows
  extern __shared__ __align__(16) float2 smem[];
  __shared__ unsigned long long s_turns[kMaxHeadDim / 2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nwarps = blockDim.x >> 5;
  const bool second = int(blockIdx.x) >= P.part[0].blocks;
  const QkPart& q = P.part[second ? 1 : 0];
  const int blk = int(blockIdx.x) - (second ? P.part[0].blocks : 0);
  const int hd = P.hd, dims = P.dims, np = hd / 2, U = P.units, tl = P.tl;
  const int heads = q.heads;
  float2* tab = smem + warp * np;
  uint16_t* s_inv = nullptr;
  T* stage = nullptr;
  if constexpr (kSliced) {
    s_inv = reinterpret_cast<uint16_t*>(smem + (nwarps * np + 1) / 2 * 2);  // 16-byte aligned
    stage = reinterpret_cast<T*>(s_inv + (heads * hd + 7) / 8 * 8) + warp * P.stage;
    for (int i = tid; i < heads * hd; i += blockDim.x) s_inv[i] = uint16_t(q.inv[i]);  // -1: 65535
  }
  for (int p = tid; p < dims / 2; p += blockDim.x) s_turns[p] = P.turns[p];
  __syncthreads();

  // this lane's place: team `team` of the warp, units lt, lt + tl, ...
  const int lt = lane % tl, team = lane / tl, tpw = 32 / tl;
  int offa[NU], offb[NU];
  bool act[NU];
  f2 glo[NU][NP], ghi[NU][NP];
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
      offa[j] = p0 + dims / 2;            // dims + (p0 - dims / 2)
      offb[j] = offa[j] + np - dims / 2;  // + half of the unrotated channels
    }
    float a[V], b[V], l[V], h[V];
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
    Pairs<V, kInter>::split(a, b, l, h);
    pack_all<V>(l, glo[j]);
    pack_all<V>(h, ghi[j]);
  }
  f2 dglo[kBwd ? NU : 1][NP], dghi[kBwd ? NU : 1][NP];
  if constexpr (kBwd) {
#pragma unroll
    for (int j = 0; j < NU; ++j)
#pragma unroll
      for (int i = 0; i < NP; ++i) dglo[j][i] = dghi[j][i] = 0ull;
  }
  f2 cs[NU][NP], sn[NU][NP];
  const f2 minus1 = pack2(-1.0f, -1.0f);

  // compact context row of row t, or -1 - its output row
  auto kind_of = [&](int t) {
    const int b = t / P.seq, i = t - b * P.seq;
    const int o0 = P.ctx_off[b], o1 = P.ctx_off[b + 1];
    return i < o1 - o0 ? o0 + i : -1 - (t - o1);
  };
  // the rows of one head that global memory holds at full width
  auto load = [&](int t, int h, bool valid, int kind, Item<T, G, V, kBwd>& it) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const bool on = valid && act[j];
      zero(it.xa[j]);
      zero(it.xb[j]);
      if (on && (!kBwd || norm) && (!kSliced || kind < 0)) {
        const T* x = kSliced ? static_cast<const T*>(q.Xo) +
                                   ((long long)(-1 - kind) * heads + h) * hd
                             : static_cast<const T*>(q.X) + t * q.ldx + h * hd;
        ld_vec(x + offa[j], it.xa[j]);
        ld_vec(x + offb[j], it.xb[j]);
      }
      if constexpr (kBwd) {
        zero(it.ya[j]);
        zero(it.yb[j]);
        if (on) {
          const G* y = static_cast<const G*>(q.dY) + t * q.ldy + h * hd;
          ld_vec(y + offa[j], it.ya[j]);
          ld_vec(y + offb[j], it.yb[j]);
        }
      }
    }
  };
  // cosines and sines of a row, from the warp's lanes to each lane's pairs
  auto angles = [&](int pos) {
    __syncwarp();
    for (int p = lane; p < np; p += 32) {
      float s = 0.0f, c = 1.0f;
      if (p < dims / 2) {
        const unsigned long long turn = (unsigned long long)(long long)pos * s_turns[p];
        // the top 32 bits as a signed fraction: half turns in [-1, 1)
        sincospif(float(int(turn >> 32)) * 4.656612873077393e-10f, &s, &c);
        s *= P.mscale;
        c *= P.mscale;
      }
      tab[p] = make_float2(c, s);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int p0 = (lt + j * tl) * V;
      float c[V], s[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 w = act[j] ? tab[p0 + i] : make_float2(1.0f, 0.0f);
        c[i] = w.x;
        s[i] = w.y;
      }
      pack_all<V>(c, cs[j]);
      pack_all<V>(s, sn[j]);
    }
  };
  auto team_sum = [&](float v) {
    for (int s = tl >> 1; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
  };
  auto store = [&](int t, int h, int kind, int j, const f2 (&lo)[NP], const f2 (&hi)[NP]) {
    float l[V], m[V], a[V], b[V];
    unpack_all<V>(lo, l);
    unpack_all<V>(hi, m);
    Pairs<V, kInter>::join(l, m, a, b);
    Raw<T, V> ra, rb;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ra.v[i] = from_f<T>(a[i]);
      rb.v[i] = from_f<T>(b[i]);
    }
    if constexpr (kSliced && kBwd) {
      if (kind >= 0) {  // into the staged row, over this lane's own x
        const uint16_t* inv = s_inv + h * hd;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int ia = inv[offa[j] + i], ib = inv[offb[j] + i];
          if (ia != 65535) stage[ia] = ra.v[i];
          if (ib != 65535) stage[ib] = rb.v[i];
        }
        return;
      }
    }
    T* o = kSliced && kBwd
               ? static_cast<T*>(q.outo) + ((long long)(-1 - kind) * heads + h) * hd
               : static_cast<T*>(q.out) + t * q.ldo + h * hd;
    st_vec(o + offa[j], ra);
    st_vec(o + offb[j], rb);
  };
  auto compute = [&](int t, int h, bool valid, int kind, Item<T, G, V, kBwd>& it) {
    f2 xlo[NU][NP], xhi[NU][NP];
    f2 ss = 0ull;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if constexpr (kSliced) {
        if (kind >= 0 && valid && act[j] && (!kBwd || norm)) {
          const uint16_t* inv = s_inv + h * hd;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int ia = inv[offa[j] + i], ib = inv[offb[j] + i];
            if (ia != 65535) it.xa[j].v[i] = stage[ia];
            if (ib != 65535) it.xb[j].v[i] = stage[ib];
          }
        }
      }
      members<T, V, kInter>(it.xa[j], it.xb[j], xlo[j], xhi[j]);
      if (norm) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          ss = fma2(xlo[j][i], xlo[j][i], ss);
          ss = fma2(xhi[j][i], xhi[j][i], ss);
        }
      }
    }
    float rs = 1.0f;
    if (norm) {
      float a, b;
      unpack2(ss, a, b);
      rs = rsqrtf(team_sum(a + b) / float(hd) + P.eps);
    }
    const f2 rs2 = pack2(rs, rs);
    if constexpr (!kBwd) {
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        f2 lo[NP], hi[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          f2 l = xlo[j][i], m = xhi[j][i];
          if (norm) {
            l = mul2(mul2(l, rs2), glo[j][i]);
            m = mul2(mul2(m, rs2), ghi[j][i]);
          }
          lo[i] = fma2(mul2(m, sn[j][i]), minus1, mul2(l, cs[j][i]));
          hi[i] = fma2(m, cs[j][i], mul2(l, sn[j][i]));
        }
        if (valid && act[j]) store(t, h, kind, j, lo, hi);
      }
    } else {
      f2 dlo[NU][NP], dhi[NU][NP];  // dn = R^T dy, then g dn
      f2 dot = 0ull;                // sum of x g dn
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        f2 ylo[NP], yhi[NP];
        members<G, V, kInter>(it.ya[j], it.yb[j], ylo, yhi);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          f2 l = fma2(yhi[i], sn[j][i], mul2(ylo[i], cs[j][i]));
          f2 m = fma2(mul2(ylo[i], sn[j][i]), minus1, mul2(yhi[i], cs[j][i]));
          if (norm) {
            dglo[j][i] = fma2(l, mul2(xlo[j][i], rs2), dglo[j][i]);
            dghi[j][i] = fma2(m, mul2(xhi[j][i], rs2), dghi[j][i]);
            l = mul2(l, glo[j][i]);
            m = mul2(m, ghi[j][i]);
            dot = fma2(xlo[j][i], l, dot);
            dot = fma2(xhi[j][i], m, dot);
          }
          dlo[j][i] = l;
          dhi[j][i] = m;
        }
      }
      if (norm) {
        float a, b;
        unpack2(dot, a, b);
        const float coef = -(rs * rs * rs) * (team_sum(a + b) / float(hd));
        const f2 coef2 = pack2(coef, coef);
#pragma unroll
        for (int j = 0; j < NU; ++j)
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            dlo[j][i] = fma2(dlo[j][i], rs2, mul2(xlo[j][i], coef2));
            dhi[j][i] = fma2(dhi[j][i], rs2, mul2(xhi[j][i], coef2));
          }
      }
#pragma unroll
      for (int j = 0; j < NU; ++j)
        if (valid && act[j]) store(t, h, kind, j, dlo[j], dhi[j]);
    }
  };
  // a context row's compact channels to the stage, and back from it
  auto stage_in = [&](int kind) {
    const T* x = static_cast<const T*>(q.Xc) + (long long)kind * q.n_idx;
    __syncwarp();
    if (q.n_idx % 8 == 0) {
      for (int i = lane * 8; i < q.n_idx; i += 256)
        *reinterpret_cast<uint4*>(stage + i) = *reinterpret_cast<const uint4*>(x + i);
    } else {
      for (int i = lane; i < q.n_idx; i += 32) stage[i] = x[i];
    }
    __syncwarp();
  };
  auto stage_out = [&](int kind) {
    T* x = static_cast<T*>(q.outc) + (long long)kind * q.n_idx;
    __syncwarp();
    if (q.n_idx % 8 == 0) {
      for (int i = lane * 8; i < q.n_idx; i += 256)
        *reinterpret_cast<uint4*>(x + i) = *reinterpret_cast<const uint4*>(stage + i);
    } else {
      for (int i = lane; i < q.n_idx; i += 32) x[i] = stage[i];
    }
    __syncwarp();
  };
  auto position = [&](int t) { return P.pos ? P.pos[t] : t % P.seq; };

  // unit u: share u % chunks of row u / chunks
  const int units = P.T * q.chunks, stride = q.blocks * nwarps;
  int u = blk * nwarps + warp;
  Item<T, G, V, kBwd> cur, nxt;
  int t = 0, h0 = 0, h1 = 0, pos = 0, kind = -1;
  if (u < units) {
    t = u / q.chunks;
    h0 = (u - t * q.chunks) * q.per_chunk;
    h1 = min(heads, h0 + q.per_chunk);
    pos = position(t);
    if constexpr (kSliced) kind = kind_of(t);
    load(t, h0 + team, h0 + team < h1, kind, cur);
  }
  while (u < units) {  // the same rounds for every lane of a warp
    const int u2 = u + stride;
    int t2 = 0, h02 = 0, h12 = 0, pos2 = 0, kind2 = -1;
    if (u2 < units) {
      t2 = u2 / q.chunks;
      h02 = (u2 - t2 * q.chunks) * q.per_chunk;
      h12 = min(heads, h02 + q.per_chunk);
      pos2 = position(t2);
      if constexpr (kSliced) kind2 = kind_of(t2);
    }
    if constexpr (kSliced) {
      if (kind >= 0 && (!kBwd || norm)) stage_in(kind);
    }
    angles(pos);
    for (int hb = h0; hb < h1; hb += tpw) {
      const int h = hb + team;
      const bool more = hb + tpw < h1;
      const int hn = more ? h + tpw : h02 + team;
      load(more ? t : t2, hn, hn < (more ? h1 : h12), more ? kind : kind2, nxt);
      compute(t, h, h < h1, kind, cur);
      cur = nxt;
    }
    if constexpr (kSliced && kBwd) {
      if (kind >= 0) stage_out(kind);
    }
    u = u2;
    t = t2;
    h0 = h02;
    h1 = h12;
    pos = pos2;
    kind = kind2;
  }

  if constexpr (kBwd) {
    if (!q.dgp) return;
    // this block's dg: the warp's teams by shuffles, then the warps in order
    float* red = reinterpret_cast<float*>(smem) + warp * hd;  // over this warp's table
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      float l[V], m[V], a[V], b[V];
      unpack_all<V>(dglo[j], l);
      unpack_all<V>(dghi[j], m);
#pragma unroll
      for (int i = 0; i < V; ++i)
        for (int s = tl; s < 32; s <<= 1) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], s);
          m[i] += __shfl_xor_sync(0xffffffffu, m[i], s);
        }
      Pairs<V, kInter>::join(l, m, a, b);
      if (act[j] && lane < tl) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          red[offa[j] + i] = a[i];
          red[offb[j] + i] = b[i];
        }
      }
    }
    __syncthreads();
    for (int c = tid; c < hd; c += blockDim.x) {
      float v = 0.0f;
      for (int w = 0; w < nwarps; ++w) v += reinterpret_cast<const float*>(smem)[w * hd + c];
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

struct Geometry {
  int warps, smem, grid;
};

template <typename T, typename G, int V, bool kInter, bool kBwd, bool kSliced>
slora_status launch(const QkParams& P, const Geometry& g, cudaStream_t st) {
  auto kernel = qk_rotary_kernel<T, G, V, kInter, kBwd, kSliced>;
  if (g.smem > 48 * 1024)
    SLORA_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, g.smem));
  kernel<<<g.grid, g.warps * 32, g.smem, st>>>(P);
  SLORA_CHECK_LAUNCH();
  return SLORA_OK;
}
template <typename T, typename G, int V, bool kInter, bool kBwd>
slora_status launch_s(bool sliced, const QkParams& P, const Geometry& g, cudaStream_t st) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    if (sliced) return launch<T, G, V, kInter, kBwd, true>(P, g, st);
  }
  return launch<T, G, V, kInter, kBwd, false>(P, g, st);
}
template <typename T, typename G, bool kBwd>
slora_status launch_v(int V, bool inter, bool sliced, const QkParams& P,
                      const Geometry& g, cudaStream_t st) {
  if (V == 8)
    return inter ? launch_s<T, G, 8, true, kBwd>(sliced, P, g, st)
                 : launch_s<T, G, 8, false, kBwd>(sliced, P, g, st);
  if (V == 2)
    return inter ? launch_s<T, G, 2, true, kBwd>(sliced, P, g, st)
                 : launch_s<T, G, 2, false, kBwd>(sliced, P, g, st);
  return inter ? launch_s<T, G, 1, true, kBwd>(sliced, P, g, st)
               : launch_s<T, G, 1, false, kBwd>(sliced, P, g, st);
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

// Blocks an SM holds at once (registers: launch bounds of the kernel).
int blocks_per_sm(bool backward) { return backward ? 2 : 3; }
// Warps of a block and its shared memory: tables, and for sliced rows the
// inverse channel list and a staged row a warp, within half an SM's memory as
// long as that leaves a warp.
void block_shape(const QkDesc& D, bool sliced, Geometry* g, int* stage) {
  int n = 0, ni = 0;
  for (int i = 0; i < D.nparts; ++i) {
    n = std::max(n, D.part[i].heads * D.head_dim);
    ni = std::max(ni, D.part[i].idx ? D.part[i].n_idx : 0);
  }
  *stage = (ni + 7) / 8 * 8;
  g->warps = kWarps;
  for (;; g->warps /= 2) {
    g->smem = (g->warps * D.head_dim * 4 + 15) / 16 * 16;
    if (sliced) g->smem += (n + 7) / 8 * 16 + g->warps * *stage * 2;
    if (!sliced || g->warps == 1 || g->smem <= 100 * 1024) return;
  }
}

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
  // f_p = base^(-2p / dims) by products in long double (2^-64 each)
  const long double ratio = std::pow((long double)base, -2.0L / dims);
  long double power = 1.0L;
  for (int p = 0; p < dims / 2; ++p, power *= ratio) {
    const double f = double(power);
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
  const int max_blocks = num_sms() * blocks_per_sm(backward);
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
  P.T = int(D.ti.T);
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
  Geometry g;
  block_shape(D, sliced, &g, &P.stage);
  int heads = 0;
  for (int i = 0; i < D.nparts; ++i) heads += D.part[i].heads;
  g.grid = 0;
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
    // blocks in proportion to the heads; a row's heads in as many shares as
    // give every warp about eight units, down to one round of a warp's teams
    // (sliced rows stay whole: their stage is a row)
    const int share = i == 0 ? std::max(1, int(int64_t(max_blocks) * s.heads / heads))
                             : std::max(1, max_blocks - P.part[0].blocks);
    const int rounds = (s.heads + 32 / P.tl - 1) / (32 / P.tl);
    const int64_t want = int64_t(share) * g.warps * 8;
    q.chunks = s.idx ? 1 : int(std::min<int64_t>(rounds, (want + D.ti.T - 1) / D.ti.T));
    q.per_chunk = (rounds + q.chunks - 1) / q.chunks * (32 / P.tl);
    q.chunks = (s.heads + q.per_chunk - 1) / q.per_chunk;
    q.blocks = int(std::min<int64_t>(share, (D.ti.T * q.chunks + g.warps - 1) / g.warps));
    if (any_dg && s.g && s.dg) q.dgp = dgp + int64_t(g.grid) * hd;
    g.grid += q.blocks;
    const double n = double(D.ti.T) * s.heads * hd;
    bytes += n * (backward ? (s.g ? es : 0) + gs + es : 2 * es);
  }
  {
    LaunchScope ls(kElementwise, bytes, st);
    const bool in = D.rot.inter != 0;
    if (!backward) {
      if (D.dt == kF32)
        SLORA_TRY((launch_v<float, float, false>(V, in, sliced, P, g, st)));
      else
        SLORA_TRY((launch_v<__nv_bfloat16, float, false>(V, in, sliced, P, g, st)));
    } else if (D.dt == kF32) {
      SLORA_TRY((launch_v<float, float, true>(V, in, sliced, P, g, st)));
    } else if (D.gdt == kF32) {
      SLORA_TRY((launch_v<__nv_bfloat16, float, true>(V, in, sliced, P, g, st)));
    } else {
      SLORA_TRY((launch_v<__nv_bfloat16, __nv_bfloat16, true>(V, in, sliced, P, g, st)));
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
    LaunchScope ls(kAux, double(g.grid) * hd * 4, st);
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
