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
// channels are grouped into pairs too, but not turned by angle 0: an infinite or NaN
// partner times sin 0 is no zero.  r is recomputed in the backward: the head is
// in registers anyway, so no statistic is stored between the two.
//
// Angles: f_p / 2 pi is held in units of 2^-64 turn, so pos * f_p modulo one
// turn is one wrapping 64-bit product, exact at every position (a product in
// fp32 is off by 4e-3 rad at position 100000).  Its top bits give the quadrant,
// the rest an angle within pi / 4, whose Taylor sums to the 9th and 8th power
// leave 2e-9 and 3e-8.
//
// Bound: memory.  Forward 2 + 2 bytes a channel, backward 2 + 4 + 2 (fp32 dy);
// the arithmetic is close behind, so it runs on packed pairs of fp32 values
// (fma.rn.f32x2).  A team of lanes owns one head (V pairs a lane: two 16-byte
// loads at V = 8), so the norm is a few shuffles and every value is read and
// written once.  A warp owns one row at a time, or a share of its heads where
// rows are few: it computes the row's hd / 2 sines and cosines once, spread
// over its lanes, keeps each lane's in registers and walks the heads, the next
// ones on their way to shared memory.  Nothing in the loop waits for another
// warp.  32 + 8 heads of 128 channels, 8192 rows: 32 us, as long as a plain copy
// of the same 168 MB takes (33 us); with norms, fp32 dy and dg backward 60 us for
// 336 MB.
//
// Sliced rows: the inverse channel list lies in shared memory; a context row's
// compact channels are staged there, gathered from (and in the backward
// scattered back to) by channel, and stored with wide stores.  An output row's
// heads pass through the same stage, two ahead.  The next row is asked into L2
// meanwhile: a second stage a warp would cost more resident warps than it
// hides.  A forward and backward of 64 heads x 4096 rows at half the channels
// take 112 us, bound by issue and latency at 16 (backward) and 24 warps an SM.
// Other ways, at an earlier state of the rest: two stages a warp 131 us against
// 129, a full-width row a warp 147; the staged row swizzled against bank conflicts
// (a quarter fewer) 120 against 116.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "qk_rotary.cuh"

namespace slora {

__device__ int g_qk_bad_index = 0;

namespace {

constexpr int kWarps = 8;  // of a block, fewer where sliced rows need the shared memory
constexpr int kSmallBatch = 64;  // sequences whose offsets travel in the parameters

struct QkPart {
  const void* X;
  long long ldx;
  const void *Xc, *Xo;
  const int32_t* idx;
  int n_idx;
  const void* g;
  void* out;  // Y, or dX
  long long ldo;
  void *outc, *outo;
  const void* dY;
  long long ldy;
  float* dgp;  // [blocks of this part][hd] partial sums of dg, or null
  int heads, blocks;
  int lg_chunks, per_chunk;  // a row's heads in 2^lg_chunks shares of per_chunk
};
struct QkParams {
  QkPart part[2];
  unsigned long long turns[kMaxHeadDim / 2];
  const int32_t* pos;
  // sliced: context rows before sequence b, [batch + 1]; up to kSmallBatch in `off`
  const int32_t* ctx_off;
  int off[kSmallBatch + 1];
  int T, seq, hd, dims, units, tl;
  int TC, batch, batch_pow;  // sliced: context rows, sequences, a power of two not above them
  int stage;  // sliced: elements of a warp's stage, a multiple of 8; the last 8 stay zero
  float eps, mscale, inv_hd;
  unsigned seq_mul, seq_shift;  // t / seq = umulhi(t, seq_mul) >> seq_shift for t < 2^31, seq > 1
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

// Units a lane owns: V = 8 covers 256 channels with 16 lanes, V = 4 with 32;
// narrower vectors need two or four units a lane.
template <int V>
constexpr int units_per_lane() {
  return V >= 4 ? 1 : (V == 2 ? 2 : 4);
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
// Raw groups of a unit to its packed first and second members, and back.  bf16
// goes by words: a word of a group is two neighbours of it (half layout) or one
// pair (interleaved).
template <typename T, int V, bool kInter>
__device__ __forceinline__ void members(const Raw<T, V>& ra, const Raw<T, V>& rb,
                                        f2 (&lo)[packs<V>()], f2 (&hi)[packs<V>()]) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value && V > 1) {
    const uint32_t* wa = reinterpret_cast<const uint32_t*>(ra.v);
    const uint32_t* wb = reinterpret_cast<const uint32_t*>(rb.v);
    auto first = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto last = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if constexpr (kInter) {
        const uint32_t w0 = 2 * i < V / 2 ? wa[(2 * i) % (V / 2)] : wb[(2 * i) % (V / 2)];
        const uint32_t w1 = 2 * i + 1 < V / 2 ? wa[(2 * i + 1) % (V / 2)] : wb[(2 * i + 1) % (V / 2)];
        lo[i] = pack2(first(w0), first(w1));
        hi[i] = pack2(last(w0), last(w1));
      } else {
        lo[i] = pack2(first(wa[i]), last(wa[i]));
        hi[i] = pack2(first(wb[i]), last(wb[i]));
      }
    }
  } else {
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
}
template <typename T, int V, bool kInter>
__device__ __forceinline__ void groups(const f2 (&lo)[packs<V>()], const f2 (&hi)[packs<V>()],
                                       Raw<T, V>& ra, Raw<T, V>& rb) {
  float l[V], m[V];
  unpack_all<V>(lo, l);
  unpack_all<V>(hi, m);
  if constexpr (std::is_same<T, __nv_bfloat16>::value && V > 1) {
    __nv_bfloat162* wa = reinterpret_cast<__nv_bfloat162*>(ra.v);
    __nv_bfloat162* wb = reinterpret_cast<__nv_bfloat162*>(rb.v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if constexpr (kInter) {
        wa[i] = __floats2bfloat162_rn(l[i], m[i]);
        wb[i] = __floats2bfloat162_rn(l[V / 2 + i], m[V / 2 + i]);
      } else {
        wa[i] = __floats2bfloat162_rn(l[2 * i], l[2 * i + 1]);
        wb[i] = __floats2bfloat162_rn(m[2 * i], m[2 * i + 1]);
      }
    }
  } else {
    float a[V], b[V];
    Pairs<V, kInter>::join(l, m, a, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ra.v[i] = from_f<T>(a[i]);
      rb.v[i] = from_f<T>(b[i]);
    }
  }
}

// Cosine and sine of pos * turns (2^-64 turn each), times m.
__device__ __forceinline__ void cos_sin(int pos, unsigned long long turns, float m, float& c,
                                        float& s) {
  const int top = int(((unsigned long long)(long long)pos * turns) >> 32);  // 2^-32 turn
  const unsigned quad = (unsigned(top) + 0x20000000u) >> 30;                // nearest quarter turn
  const int rest = int(unsigned(top) - (quad << 30));                       // within an eighth
  const float a = float(rest) * 1.4629180792671596e-9f;                     // 2 pi / 2^32
  const float z = a * a;
  float sp = fmaf(z, 2.7557319223985893e-6f, -1.9841269841269841e-4f);  // 1/9!, -1/7!
  sp = fmaf(z, sp, 8.3333333333333333e-3f);                             // 1/5!
  sp = fmaf(z, sp, -1.6666666666666667e-1f);                            // -1/3!
  sp = fmaf(a * z, sp, a);
  float cp = fmaf(z, 2.4801587301587302e-5f, -1.3888888888888889e-3f);  // 1/8!, -1/6!
  cp = fmaf(z, cp, 4.1666666666666667e-2f);                             // 1/4!
  cp = fmaf(z, cp, -0.5f);
  cp = fmaf(z, cp, 1.0f);
  c = (quad & 1u) ? sp : cp;
  s = (quad & 1u) ? cp : sp;
  c *= ((quad + 1u) & 2u) ? -m : m;
  s *= (quad & 2u) ? -m : m;
}

// Rows on their way to shared memory: kAhead items of a warp beside the one
// that is computed, each lane's own pieces of up to 16 bytes (an asynchronous
// copy has at least 4: V > 1; single channels load when their turn comes).
// Sliced rows: dy alone.
template <bool kBwd, bool kSliced>
constexpr int ahead() {
  return kBwd ? (kSliced ? 1 : 2) : 3;
}
template <typename T, int V>
constexpr int piece_bytes() {
  return V * int(sizeof(T)) < 16 ? V * int(sizeof(T)) : 16;
}
template <typename T, int V>
constexpr int group_pieces() {
  return V * int(sizeof(T)) / piece_bytes<T, V>();
}
// Bytes of x (or dy) of one lane and item, and of a warp's ring.
template <typename T, int V>
constexpr int item_bytes() {
  return 2 * units_per_lane<V>() * V * int(sizeof(T));
}
template <typename T, typename G, int V, bool kBwd, bool kSliced>
constexpr int ring_bytes() {
  return V == 1 ? 0
                : (ahead<kBwd, kSliced>() + 1) * 32 *
                      ((kSliced ? 0 : item_bytes<T, V>()) + (kBwd ? item_bytes<G, V>() : 0));
}
// kThrough: part of a 32-byte sector whose other part the lane copies next;
// through L1, so that the sector is fetched once (as pieces below 16 bytes are).
template <int BYTES, bool kThrough>
__device__ __forceinline__ void copy_piece(uint32_t dst, const void* src, bool on) {
  if constexpr (BYTES == 16 && !kThrough)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src),
                 "n"(BYTES), "r"(on ? BYTES : 0)
                 : "memory");
}
template <int BYTES>
__device__ __forceinline__ void read_piece(void* to, uint32_t src) {
  uint32_t* w = static_cast<uint32_t*>(to);
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(src));
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(src));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(src));
}
template <int N>
__device__ __forceinline__ void copies_but(void) {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where a warp is: row t of unit u, `left` rounds of the unit from this one on;
// this team's head starts at channel e.  x, y, o: the row's elements.
template <typename T, typename G>
struct Place {
  int u, t, e, left;
  int kind;  // sliced: compact context row of row t, or -1 - output row
  bool first;
  const T* x;
  const G* y;
  T* o;
};

// Blocks of kWarps warps an SM by registers: 80 a thread, 128 for the backward with
// eight pairs a lane (80 would spill: sliced 57 -> 79 us) or one (likewise).  16 + 4
// heads of 80 channels, 20 of them rotated, 8192 rows, sliced: backward 69 us at
// two blocks, 59 at three; forward with eight pairs 32 at three, 35 at two or four.
constexpr int blocks_of(bool backward, int V) {
  return backward && (V == 8 || V == 1) ? 2 : 3;
}

// kPart: heads of which only the leading channels are rotated.  (With the whole heads'
// kernels looking at each unit too, 32 + 8 heads of 128, 8192 rows, forward with norms
// took 33 us for 32.)
template <typename T, typename G, int V, bool kInter, bool kBwd, bool kSliced, bool kPart>
__global__ void __launch_bounds__(kWarps * 32, blocks_of(kBwd, V))
    qk_rotary_kernel(const __grid_constant__ QkParams P) {
  constexpr int NU = units_per_lane<V>(), NP = packs<V>();
  constexpr int kAhead = ahead<kBwd, kSliced>();
  constexpr bool kRingX = V > 1 && !kSliced, kRingY = V > 1 && kBwd, kRing = kRingX || kRingY;
  constexpr bool kThroughStage = V > 1 && kSliced;  // output rows' x
  // [warps][hd / 2 cosines, hd / 2 sines] (the backward's dg at the end), the
  // warps' rings, then for sliced rows the inverse channel list (a channel that
  // is not computed: the stage's zero) and a stage a warp
  extern __shared__ __align__(16) float smem[];
  __shared__ unsigned long long s_turns[kMaxHeadDim / 2];
  grid_wait();
  grid_ahead();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nwarps = blockDim.x >> 5;
  const bool second = int(blockIdx.x) >= P.part[0].blocks;
  const QkPart q = second ? P.part[1] : P.part[0];  // (in registers: read in every round)
  const int blk = int(blockIdx.x) - (second ? P.part[0].blocks : 0);
  const int hd = P.hd, dims = P.dims, np = hd / 2, U = P.units, tl = P.tl;
  const int heads = q.heads, n = heads * hd;
  float* tab = smem + warp * hd;
  char* rings = reinterpret_cast<char*>(smem + (nwarps * hd + 3) / 4 * 4);  // 16-byte aligned
  const uint32_t ring = uint32_t(__cvta_generic_to_shared(rings)) +
                        warp * ring_bytes<T, G, V, kBwd, kSliced>();
  // of a warp's item: x, then dy
  constexpr int kXBytes = 32 * item_bytes<T, V>(), kYBytes = kBwd ? 32 * item_bytes<G, V>() : 0;
  constexpr int kYAt = kRingX ? kXBytes : 0, kItemBytes = kYAt + kYBytes;
  __shared__ int s_off[kSliced ? kSmallBatch + 1 : 1];
  const int32_t* ctx_off = kSliced && P.batch <= kSmallBatch ? s_off : P.ctx_off;
  uint16_t* s_inv = nullptr;
  T* stage = nullptr;
  const unsigned skipped = P.stage - 8;
  if constexpr (kSliced) {
    s_inv = reinterpret_cast<uint16_t*>(rings + nwarps * ring_bytes<T, G, V, kBwd, kSliced>());
    stage = reinterpret_cast<T*>(s_inv + (n + 7) / 8 * 8) + warp * P.stage;
    // every block inverts the list for itself (8 KB of indices from L2): a launch
    // that did it once before cost 4 to 5 us
    for (int i = tid; i < n; i += blockDim.x) s_inv[i] = uint16_t(skipped);
    if (P.batch <= kSmallBatch)
      for (int i = tid; i <= P.batch; i += blockDim.x) s_off[i] = P.off[i];
    __syncthreads();
    auto listed = [&](int i) {  // entry i's channel, or -1
      const int c = q.idx[i];
      return c >= 0 && c < n ? c : -1;
    };
#pragma unroll 4
    for (int i = tid; i < q.n_idx; i += blockDim.x) {
      const int c = listed(i);
      if (c >= 0) s_inv[c] = uint16_t(i);
    }
    __syncthreads();
    if (blk == 0)  // outside its channels, or a later or earlier entry took the place
      for (int i = tid; i < q.n_idx; i += blockDim.x) {
        const int c = listed(i);
        if (c < 0 || s_inv[c] != i) atomicExch(&g_qk_bad_index, 1);
      }
    if (lane < 8) stage[skipped + lane] = from_f<T>(0.0f);
  }
  for (int p = tid; p < dims / 2; p += blockDim.x) s_turns[p] = P.turns[p];
  __syncthreads();

  // this lane's place: team `team` of the warp, units lt, lt + tl, ...; group B
  // lies `apart` channels behind group A
  const int lt = lane % tl, team = lane / tl, tpw = 32 / tl;
  int offa[NU], apart[NU], turned[NU];  // turned: the unit's leading pairs that are rotated
  bool act[NU];
  f2 glo[NU][NP], ghi[NU][NP];
  const bool norm = q.g != nullptr;
  const bool reads_x = !kBwd || norm;
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    const int u = lt + j * tl, p0 = u * V;
    act[j] = u < U;
    turned[j] = dims / 2 - p0;
    if (!act[j]) {
      offa[j] = apart[j] = 0;
    } else if (kInter) {
      offa[j] = 2 * p0;
      apart[j] = V;
    } else if (p0 < dims / 2) {
      offa[j] = p0;
      apart[j] = dims / 2;
    } else {
      offa[j] = p0 + dims / 2;   // dims + (p0 - dims / 2)
      apart[j] = np - dims / 2;  // half of the unrotated channels
    }
    float a[V], b[V], l[V], h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = b[i] = 1.0f;
    if (norm && act[j]) {
      const T* g = static_cast<const T*>(q.g) + offa[j];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a[i] = to_f(g[i]);
        b[i] = to_f(g[apart[j] + i]);
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
  // Pack i of unit j by its angles, forwards or back.
  auto turn = [&](int j, int i, f2& lo, f2& hi) {
    const f2 l = lo, m = hi;
    if constexpr (kBwd) {
      lo = fma2(m, sn[j][i], mul2(l, cs[j][i]));
      hi = fma2(mul2(l, sn[j][i]), minus1, mul2(m, cs[j][i]));
    } else {
      lo = fma2(mul2(m, sn[j][i]), minus1, mul2(l, cs[j][i]));
      hi = fma2(m, cs[j][i], mul2(l, sn[j][i]));
    }
  };
  // Unit j: of a head that is rotated in part only the pairs that are (in the half layout
  // all of a unit's or none, else the leading ones).
  auto turn_unit = [&](int j, f2 (&lo)[NP], f2 (&hi)[NP]) {
    if (!kPart || turned[j] >= V) {
#pragma unroll
      for (int i = 0; i < NP; ++i) turn(j, i, lo[i], hi[i]);
    } else if (kInter && turned[j] > 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        f2 a = lo[i], b = hi[i];
        turn(j, i, a, b);
        float a0, a1, b0, b1, l0, l1, m0, m1;
        unpack2(a, a0, a1);
        unpack2(b, b0, b1);
        unpack2(lo[i], l0, l1);
        unpack2(hi[i], m0, m1);
        const bool first = 2 * i < turned[j], second = 2 * i + 1 < turned[j];
        lo[i] = pack2(first ? a0 : l0, second ? a1 : l1);
        hi[i] = pack2(first ? b0 : m0, second ? b1 : m1);
      }
    }
  };

  using At = Place<T, G>;
  const int units = P.T << q.lg_chunks, stride = q.blocks * nwarps, step = tpw * hd;
  // this lane's pieces of one tensor's row from channel e, zeros where it has
  // none: [unit][group][piece][lane]
  auto fetch_rows = [&](auto* row, int e, bool valid, uint32_t dst) {
    using R = typename std::remove_cv<typename std::remove_pointer<decltype(row)>::type>::type;
    constexpr int PB = piece_bytes<R, V>(), PG = group_pieces<R, V>();
    constexpr bool kThrough = PG > 1 || kInter;
    dst += lane * PB;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const bool on = valid && act[j];
      const auto* a = row + (e + offa[j]);
      const auto* b = a + apart[j];
#pragma unroll
      for (int i = 0; i < PG; ++i) {
        copy_piece<PB, kThrough>(dst + ((2 * j) * PG + i) * 32 * PB, a + i * (PB / sizeof(R)), on);
        copy_piece<PB, kThrough>(dst + ((2 * j + 1) * PG + i) * 32 * PB, b + i * (PB / sizeof(R)),
                                 on);
      }
    }
  };
  auto from_ring = [&](auto& ra, auto& rb, int j, uint32_t src) {
    using R = typename std::remove_reference<decltype(ra.v[0])>::type;
    constexpr int PB = piece_bytes<R, V>(), PG = group_pieces<R, V>();
    src += lane * PB;
#pragma unroll
    for (int i = 0; i < PG; ++i) {
      read_piece<PB>(reinterpret_cast<char*>(ra.v) + i * PB, src + ((2 * j) * PG + i) * 32 * PB);
      read_piece<PB>(reinterpret_cast<char*>(rb.v) + i * PB,
                     src + ((2 * j + 1) * PG + i) * 32 * PB);
    }
  };
  // an item's rows to ring place k
  auto fetch = [&](const At& w, int k) {
    if constexpr (kRing) {
      if (w.u < units) {
        const bool valid = w.e < n;
        const int e = min(w.e, n - hd);  // inside the row either way
        const uint32_t dst = ring + k * kItemBytes;
        if (kRingX && reads_x) fetch_rows(w.x, e, valid, dst);
        if constexpr (kRingY) fetch_rows(w.y, e, valid, dst + kYAt);
      }
    }
    if constexpr (kRing) asm volatile("cp.async.commit_group;" ::: "memory");  // one an item
  };
  // cosines and sines of a row, from the warp's lanes to each lane's pairs
  auto angles = [&](int pos) {
    __syncwarp();
    for (int p = lane; p < np; p += 32) {
      float c = 1.0f, s = 0.0f;
      if (p < dims / 2) cos_sin(pos, s_turns[p], P.mscale, c, s);
      tab[p] = c;
      tab[np + p] = s;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int p0 = act[j] ? (lt + j * tl) * V : 0;  // (a lane without a unit: any values)
      Raw<float, V> c, s;
      if constexpr (V >= 4) {
        ld_vec(tab + p0, c);
        ld_vec(tab + np + p0, s);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          c.v[i] = tab[p0 + i];
          s.v[i] = tab[np + p0 + i];
        }
      }
      pack_all<V>(c.v, cs[j]);
      pack_all<V>(s.v, sn[j]);
    }
  };
  // sums over a team, two at once (v2's and w2's halves added first)
  auto team_sums = [&](f2 v2, f2 w2, float& v, float& w) {
    float a, b;
    unpack2(v2, a, b);
    v = a + b;
    if constexpr (kBwd) {
      unpack2(w2, a, b);
      w = a + b;
    }
    auto add = [&](int s) {
      const float x = __shfl_xor_sync(0xffffffffu, v, s);
      if constexpr (kBwd) w += __shfl_xor_sync(0xffffffffu, w, s);
      v += x;
    };
    if (tl == 8) {  // heads of 128 channels
      add(1);
      add(2);
      add(4);
    } else {
      for (int s = 1; s < tl; s <<= 1) add(s);
    }
  };
  // a context row's channels of one head: their places in the staged row
  auto offsets = [&](int e, int j, Raw<uint16_t, V>& ia, Raw<uint16_t, V>& ib) {
    const uint16_t* inv = s_inv + e + offa[j];
    ld_vec(inv, ia);
    ld_vec(inv + apart[j], ib);
  };
  auto store = [&](const At& w, int j, const f2 (&lo)[NP], const f2 (&hi)[NP]) {
    Raw<T, V> ra, rb;
    groups<T, V, kInter>(lo, hi, ra, rb);
    if constexpr (kSliced && kBwd) {
      if (w.kind >= 0) {  // into the staged row, over this lane's own x
        Raw<uint16_t, V> ia, ib;
        offsets(w.e, j, ia, ib);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (ia.v[i] != skipped) stage[ia.v[i]] = ra.v[i];
          if (ib.v[i] != skipped) stage[ib.v[i]] = rb.v[i];
        }
        return;
      }
    }
    T* o = w.o + (w.e + offa[j]);
    st_vec(o, ra);
    st_vec(o + apart[j], rb);
  };
  auto compute = [&](const At& w, int k, int sx) {  // sx: the stage's place of an output row's x
    const bool valid = w.e < n;
    const uint32_t src = ring + k * kItemBytes;
    f2 xlo[NU][NP], xhi[NU][NP];
    f2 ss = 0ull;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if (kSliced && w.kind >= 0) {
        // gathered from the staged row, its zero where a channel is not computed
        float a[V], b[V], l[V], h[V];
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = b[i] = 0.0f;
        if (reads_x) {
          Raw<uint16_t, V> ia, ib;
          offsets(min(w.e, n - hd), j, ia, ib);  // (a team without a head: the last one's)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            a[i] = to_f(stage[ia.v[i]]);
            b[i] = to_f(stage[ib.v[i]]);
          }
          if (!valid || !act[j]) {
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] = b[i] = 0.0f;
          }
        }
        Pairs<V, kInter>::split(a, b, l, h);
        pack_all<V>(l, xlo[j]);
        pack_all<V>(h, xhi[j]);
      } else {
        Raw<T, V> xa, xb;
        if (kRingX && reads_x) {
          from_ring(xa, xb, j, src);
        } else if (kThroughStage && reads_x) {
          from_ring(xa, xb, j, uint32_t(__cvta_generic_to_shared(stage)) + sx * kXBytes);
        } else {
          zero(xa);
          zero(xb);
          if (valid && act[j] && reads_x) {
            const T* x = w.x + (w.e + offa[j]);
            ld_vec(x, xa);
            ld_vec(x + apart[j], xb);
          }
        }
        members<T, V, kInter>(xa, xb, xlo[j], xhi[j]);
      }
      if (norm) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          ss = fma2(xlo[j][i], xlo[j][i], ss);
          ss = fma2(xhi[j][i], xhi[j][i], ss);
        }
      }
    }
    if constexpr (!kBwd) {
      f2 rs2 = 0ull;
      if (norm) {
        float sum, none;
        team_sums(ss, 0ull, sum, none);
        const float rs = rsqrtf(fmaf(sum, P.inv_hd, P.eps));
        rs2 = pack2(rs, rs);
      }
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
          lo[i] = l;
          hi[i] = m;
        }
        turn_unit(j, lo, hi);
        if (valid && act[j]) store(w, j, lo, hi);
      }
    } else {
      f2 dlo[NU][NP], dhi[NU][NP];  // dn = R^T dy
      f2 dot = 0ull;                // sum of x g dn
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        Raw<G, V> ya, yb;
        if constexpr (kRingY) {
          from_ring(ya, yb, j, src + kYAt);
        } else {
          zero(ya);
          zero(yb);
          if (valid && act[j]) {
            const G* y = w.y + (w.e + offa[j]);
            ld_vec(y, ya);
            ld_vec(y + apart[j], yb);
          }
        }
        members<G, V, kInter>(ya, yb, dlo[j], dhi[j]);
        turn_unit(j, dlo[j], dhi[j]);
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (norm) {
            dot = fma2(mul2(xlo[j][i], glo[j][i]), dlo[j][i], dot);
            dot = fma2(mul2(xhi[j][i], ghi[j][i]), dhi[j][i], dot);
          }
      }
      if (norm) {
        float sum, proj;
        team_sums(ss, dot, sum, proj);
        const float rs = rsqrtf(fmaf(sum, P.inv_hd, P.eps));
        const float coef = -(rs * rs) * (proj * P.inv_hd);  // of x r
        const f2 rs2 = pack2(rs, rs), coef2 = pack2(coef, coef);
#pragma unroll
        for (int j = 0; j < NU; ++j)
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const f2 xl = mul2(xlo[j][i], rs2), xh = mul2(xhi[j][i], rs2);
            dglo[j][i] = fma2(dlo[j][i], xl, dglo[j][i]);
            dghi[j][i] = fma2(dhi[j][i], xh, dghi[j][i]);
            dlo[j][i] = fma2(mul2(dlo[j][i], glo[j][i]), rs2, mul2(xl, coef2));
            dhi[j][i] = fma2(mul2(dhi[j][i], ghi[j][i]), rs2, mul2(xh, coef2));
          }
      }
#pragma unroll
      for (int j = 0; j < NU; ++j)
        if (valid && act[j]) store(w, j, dlo[j], dhi[j]);
    }
  };

  auto sequence_of = [&](int t) {
    return P.seq == 1 ? t : int(__umulhi(unsigned(t), P.seq_mul) >> P.seq_shift);
  };
  // unit u: share u % chunks of row u / chunks (a power of two of them)
  auto enter = [&](At& w, bool in, bool out) {  // the first round of unit w.u
    if (w.u >= units) return;
    w.t = w.u >> q.lg_chunks;
    const int h0 = (w.u & ((1 << q.lg_chunks) - 1)) * q.per_chunk;
    w.e = (h0 + team) * hd;
    w.left = (min(heads - h0, q.per_chunk) + tpw - 1) / tpw;
    w.first = true;
    if constexpr (kSliced) {
      // the context rows first, the output rows, which cost less, behind them:
      // a warp's last unit is a light one
      const bool ctx = w.u < P.TC;
      const int at = ctx ? w.u : w.u - P.TC;
      // its sequence: the last one with at most `at` such rows before it
      int b = 0;
      for (int s = P.batch_pow; s; s >>= 1)
        if (b + s < P.batch) {
          const int before = ctx_off[b + s];
          if ((ctx ? before : (b + s) * P.seq - before) <= at) b += s;
        }
      const int o0 = ctx_off[b], o1 = ctx_off[b + 1];
      w.kind = ctx ? at : -1 - at;
      w.t = ctx ? b * P.seq + (at - o0) : at + o1;
      const long long full = w.kind < 0 ? (long long)(-1 - w.kind) * n : 0;
      w.x = static_cast<const T*>(q.Xo) + full;
      w.o = kBwd ? static_cast<T*>(q.outo) + full : static_cast<T*>(q.out) + w.t * q.ldo;
    } else {
      if (in) w.x = static_cast<const T*>(q.X) + w.t * q.ldx;
      if (out) w.o = static_cast<T*>(q.out) + w.t * q.ldo;
    }
    if (kBwd && in) w.y = static_cast<const G*>(q.dY) + w.t * q.ldy;
  };
  auto next = [&](At& w, bool in, bool out) {
    w.first = false;
    w.e += step;
    if (--w.left > 0) return;
    w.u += stride;
    enter(w, in, out);
  };
  // Sliced: a context row's compact channels to the stage, and back from it
  auto copy_row = [&](T* to, const T* from) {
    __syncwarp();
    if (q.n_idx % 8 == 0) {
#pragma unroll 4
      for (int i = lane * 8; i < q.n_idx; i += 256)
        *reinterpret_cast<uint4*>(to + i) = *reinterpret_cast<const uint4*>(from + i);
    } else {
      for (int i = lane; i < q.n_idx; i += 32) to[i] = from[i];
    }
    __syncwarp();
  };
  // ... the x of round `ahead` of an output row to the stage's place sx
  auto ask_ahead = [&](const At& w, int ahead, int sx) {
    if constexpr (kThroughStage) {
      if (w.left > ahead) {
        const int e = w.e + ahead * step;
        fetch_rows(w.x, min(e, n - hd), e < n,
                   uint32_t(__cvta_generic_to_shared(stage)) + sx * kXBytes);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  // ... and the x of this warp's next unit on its way to L2
  auto ask_for_next = [&](const At& w) {
    At then = w;
    then.u += stride;
    if (!reads_x || then.u >= units) return;
    enter(then, true, false);
    const bool ctx = then.kind >= 0;
    const char* from = ctx ? static_cast<const char*>(q.Xc) +
                                 (long long)then.kind * q.n_idx * int(sizeof(T))
                           : reinterpret_cast<const char*>(then.x);
    const int bytes = (ctx ? q.n_idx : n) * int(sizeof(T));
    for (int i = lane * 128; i < bytes; i += 32 * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
  };

  // w: the item that is computed; f: the one whose rows are asked for (rows that
  // are not copied ahead are w's own)
  constexpr bool kIn = !kRingX || (kBwd && !kRingY);
  At w, f;
  w.u = f.u = blk * nwarps + warp;
  w.kind = f.kind = -1;
  w.left = f.left = 0;
  enter(w, kIn, true);
  enter(f, true, false);
  if constexpr (kRing) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      fetch(f, k);
      if (f.u < units) next(f, true, false);
    }
  }
  int sx = 0;              // the stage's place of this round
  while (w.u < units) {    // the same rounds for every lane of a warp
#pragma unroll
    for (int k = 0; k <= kAhead; ++k) {  // ring places
      if (w.u >= units) break;
      if constexpr (kRing) {
        fetch(f, (k + kAhead) % (kAhead + 1));
        if (f.u < units) next(f, true, false);
      }
      if constexpr (kSliced) {
        if (w.first) {
          ask_for_next(w);
          if (w.kind >= 0 && reads_x)
            copy_row(stage, static_cast<const T*>(q.Xc) + (long long)w.kind * q.n_idx);
        }
        if (w.kind < 0 && reads_x) {
          if (w.first) {
            __syncwarp();  // the last row's channels have been read
            sx = 0;
            ask_ahead(w, 0, 0);
            ask_ahead(w, 1, 1);
          }
          ask_ahead(w, 2, sx == 0 ? 2 : sx - 1);
        }
      }
      // this item's copies, those of its x behind two rounds of the stage's
      if constexpr (kThroughStage) {
        if (w.kind < 0 && reads_x) copies_but<2>();
        else copies_but<kRing ? kAhead : 0>();
      } else if constexpr (kRing) {
        copies_but<kAhead>();
      }
      if (w.first) {
        int pos;
        if (P.pos) pos = P.pos[w.t];
        else pos = w.t - sequence_of(w.t) * P.seq;
        angles(pos);
      }
      compute(w, k, sx);
      sx = sx == 2 ? 0 : sx + 1;
      if constexpr (kSliced && kBwd) {
        if (w.kind >= 0 && w.left == 1)
          copy_row(static_cast<T*>(q.outc) + (long long)w.kind * q.n_idx, stage);
      }
      next(w, kIn, true);
    }
  }
  copies_but<0>();

  if constexpr (kBwd) {
    if (!q.dgp) return;
    // this block's dg: the warp's teams by shuffles, then the warps in order
    float* red = smem + warp * hd;  // over this warp's table
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
          red[offa[j] + apart[j] + i] = b[i];
        }
      }
    }
    __syncthreads();
    for (int c = tid; c < hd; c += blockDim.x) {
      float v = 0.0f;
      for (int k2 = 0; k2 < nwarps; ++k2) v += smem[k2 * hd + c];
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
  grid_wait();
  grid_ahead();
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

// The context rows before every sequence of a large batch.
struct OffsetParams {
  int32_t* ctx_off;
  int batch;
  int ctx_len[kMaxBatch];
};
__global__ void __launch_bounds__(1024) qk_offsets_kernel(const __grid_constant__ OffsetParams p) {
  // exclusive scan of ctx_len, 1024 sequences at a time (batch is at most kMaxBatch)
  __shared__ int part[1024];
  grid_wait();
  grid_ahead();
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

struct Geometry {
  int warps, smem, grid;
};
constexpr int kSmShared = 226 * 1024;            // that blocks share, 2 KB of each its own
constexpr int kMostShared = kSmShared - 2 * 1024;  // a block's dynamic part

template <typename T, typename G, int V, bool kInter, bool kBwd, bool kSliced, bool kPart>
slora_status launch(const QkParams& P, const Geometry& g, cudaStream_t st) {
  auto kernel = qk_rotary_kernel<T, G, V, kInter, kBwd, kSliced, kPart>;
  // the limit belongs to the kernel, not to this call: always the same one, or a smaller
  // call on another host thread would lower it under this call's launch
  if (g.smem > 48 * 1024)
    SLORA_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kMostShared));
  SLORA_CUDA(launch_early(kernel, dim3(unsigned(g.grid)), g.warps * 32, size_t(g.smem), st, P));
  return SLORA_OK;
}
template <typename T, typename G, int V, bool kInter, bool kBwd>
slora_status launch_s(bool sliced, const QkParams& P, const Geometry& g, cudaStream_t st) {
  const bool part = P.dims < P.hd;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    if (sliced)
      return part ? launch<T, G, V, kInter, kBwd, true, true>(P, g, st)
                  : launch<T, G, V, kInter, kBwd, true, false>(P, g, st);
  }
  return part ? launch<T, G, V, kInter, kBwd, false, true>(P, g, st)
              : launch<T, G, V, kInter, kBwd, false, false>(P, g, st);
}
template <typename T, typename G, bool kBwd>
slora_status launch_v(int V, bool inter, bool sliced, const QkParams& P,
                      const Geometry& g, cudaStream_t st) {
  if (V == 8)
    return inter ? launch_s<T, G, 8, true, kBwd>(sliced, P, g, st)
                 : launch_s<T, G, 8, false, kBwd>(sliced, P, g, st);
  if (V == 4)
    return inter ? launch_s<T, G, 4, true, kBwd>(sliced, P, g, st)
                 : launch_s<T, G, 4, false, kBwd>(sliced, P, g, st);
  if (V == 2)
    return inter ? launch_s<T, G, 2, true, kBwd>(sliced, P, g, st)
                 : launch_s<T, G, 2, false, kBwd>(sliced, P, g, st);
  return inter ? launch_s<T, G, 1, true, kBwd>(sliced, P, g, st)
               : launch_s<T, G, 1, false, kBwd>(sliced, P, g, st);
}

// The widest vector (in channels of one group) that every row of the call
// takes.  A unit may not straddle the members of a pair, so in the half layout
// the width divides both halves.  (16 + 4 heads of 96 channels, 24 of them
// rotated, 8192 rows: forward 38 us with single loads of 2, 28 us at 4, by now 26.)
int vector_width(const QkDesc& D, bool backward) {
  for (int V : {8, 4, 2}) {
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

constexpr double kAngles = 0.6;  // a unit's angles, in rounds (about 150 of 245 instructions)

// Warps of a block, its shared memory (tables and rings, and for sliced rows the
// inverse channel list and a stage a warp) and the blocks that an SM
// holds of them: by registers (blocks_of), and by shared memory, 226 KB with 2 KB
// of a block's own.  Eight warps, or the smaller block that keeps more warps resident.
struct Shape {
  int warps = 1, smem = 0, per_sm = 1, stage = 0;
};
Shape block_shape(const QkDesc& D, bool backward, bool sliced, int V) {
  int n = 0, ni = 0;
  for (int i = 0; i < D.nparts; ++i) {
    n = std::max(n, D.part[i].heads * D.head_dim);
    ni = std::max(ni, D.part[i].idx ? D.part[i].n_idx : 0);
  }
  // a staged row, or three items of an output row's x
  const int stage = std::max((ni + 7) / 8 * 8, V == 1 ? 0 : 3 * 32 * 2 * std::max(V, 4)) + 8;
  // a warp's ring (ring_bytes): one item more than is on its way
  const int pair = 2 * ((sliced ? 0 : dt_size(D.dt)) + (backward ? dt_size(D.gdt) : 0));
  const int items = backward ? (sliced ? 2 : 3) : 4;
  const int ring = V == 1 ? 0 : items * 32 * std::max(V, 4) * pair;
  Shape best;
  for (int w = kWarps; w >= 1; w /= 2) {
    Shape s;
    s.warps = w;
    s.stage = stage;
    s.smem = (w * D.head_dim * 4 + 15) / 16 * 16 + w * ring;
    if (sliced) s.smem += (n + 7) / 8 * 16 + w * stage * 2;
    s.per_sm = std::min(kWarps * blocks_of(backward, V) / w, kSmShared / (s.smem + 2048));
    if (w == kWarps || s.warps * s.per_sm > best.warps * best.per_sm) best = s;
  }
  return best;
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
  const int V = vector_width(D, backward);
  const Shape shape = block_shape(D, backward, sliced, V);
  const int max_blocks = num_sms() * std::max(shape.per_sm, 1);
  int32_t* ctx_off = nullptr;
  float* dgp = nullptr;
  if (sliced && D.ti.batch > kSmallBatch) ctx_off = ar.take<int32_t>(size_t(D.ti.batch) + 1);
  // one partial of each block; the parts' blocks together are at most max_blocks + 1
  if (any_dg) dgp = ar.take<float>(size_t(max_blocks + 1) * hd);
  if (plan) return SLORA_OK;
  SLORA_TRY(arena_fits(ar, "qk_rotary"));

  QkParams P{};
  if (sliced && D.ti.batch <= kSmallBatch) {
    for (int b = 0; b < D.ti.batch; ++b) P.off[b + 1] = P.off[b] + tok->ctx_len[b];
  } else if (sliced) {
    OffsetParams o{};
    o.ctx_off = ctx_off;
    o.batch = D.ti.batch;
    std::copy(tok->ctx_len, tok->ctx_len + D.ti.batch, o.ctx_len);
    LaunchScope ls(kAux, double(D.ti.batch) * 4, st);
    SLORA_CUDA(launch_early(qk_offsets_kernel, dim3(1), 1024, 0, st, o));
  }
  P.pos = D.pos;
  P.ctx_off = ctx_off;
  P.T = int(D.ti.T);
  P.seq = D.ti.seq;
  P.TC = int(D.ti.T_C);
  P.batch = D.ti.batch;
  P.batch_pow = 1;
  while (2 * P.batch_pow <= P.batch) P.batch_pow *= 2;
  P.hd = hd;
  P.dims = D.rot.dims;
  P.eps = D.eps;
  P.mscale = D.rot.mscale;
  P.inv_hd = 1.0f / float(hd);
  if (P.seq > 1) {
    unsigned l = 1;
    while ((uint64_t(1) << l) < uint64_t(P.seq)) ++l;
    P.seq_shift = l - 1;
    P.seq_mul = unsigned(((uint64_t(1) << (31 + l)) + uint64_t(P.seq) - 1) / uint64_t(P.seq));
  }
  std::copy(D.rot.turns, D.rot.turns + kMaxHeadDim / 2, P.turns);
  P.units = hd / 2 / V;
  const int nu = V >= 4 ? 1 : (V == 2 ? 2 : 4);
  P.tl = 1;
  while (P.tl < 32 && P.tl * nu < P.units) P.tl *= 2;
  Geometry g;
  g.warps = shape.warps;
  g.smem = shape.smem;
  P.stage = shape.stage;
  auto rounds_of = [&](int i, int lg) {  // of a share of part i's heads in 2^lg shares
    const int all = (D.part[i].heads + 32 / P.tl - 1) / (32 / P.tl);
    return (all + (1 << lg) - 1) >> lg;
  };
  auto work = [&](int i) { return rounds_of(i, 0) + kAngles; };
  double total = 0.0;
  for (int i = 0; i < D.nparts; ++i) total += work(i);
  g.grid = 0;
  double bytes = 0.0;
  const double es = D.dt == kF32 ? 4 : 2, gs = D.gdt == kF32 ? 4 : 2;
  for (int i = 0; i < D.nparts; ++i) {
    const slora_qk_rows& s = D.part[i];
    QkPart& q = P.part[i];
    q.X = s.X; q.ldx = s.ldx; q.Xc = s.X_ctx; q.Xo = s.X_out;
    q.idx = s.idx; q.n_idx = s.n_idx; q.g = s.g; q.heads = s.heads;
    if (backward) {
      q.out = s.dX; q.ldo = s.lddx; q.outc = s.dX_ctx; q.outo = s.dX_out;
      q.dY = s.dY; q.ldy = s.lddy;
    } else {
      q.out = s.Y; q.ldo = s.ldy;
    }
    // blocks in proportion to the parts' work on a row
    const int share = i == 0 ? std::max(1, int(max_blocks * work(i) / total))
                             : std::max(1, max_blocks - P.part[0].blocks);
    // a row's heads in the number of shares (a power of two, none empty) whose
    // slowest warp has the least to do: units a warp, times rounds a unit and
    // the unit's angles (sliced rows stay whole: their stage is a row)
    const int rounds = rounds_of(i, 0), warps = share * g.warps;
    auto cost = [&](int lg) {
      const int64_t units = D.ti.T << lg;
      return double((units + warps - 1) / warps) * (rounds_of(i, lg) + kAngles);
    };
    q.lg_chunks = 0;
    for (int lg = 1; !s.idx && lg <= 6 && ((1 << lg) - 1) * rounds_of(i, lg) < rounds; ++lg)
      if (cost(lg) < cost(q.lg_chunks)) q.lg_chunks = lg;
    q.per_chunk = rounds_of(i, q.lg_chunks) * (32 / P.tl);
    q.blocks = int(std::min<int64_t>(share, ((D.ti.T << q.lg_chunks) + g.warps - 1) / g.warps));
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
    SLORA_CUDA(launch_early(qk_dg_kernel, dim3(unsigned((hd + 31) / 32), unsigned(D.nparts)), 1024,
                            0, st, d));
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
