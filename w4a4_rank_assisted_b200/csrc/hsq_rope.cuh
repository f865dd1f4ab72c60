// hsq_rope.cuh -- rotary positions at the output of a fused QKV linear, and the
// paged cache append that rotates on the way.
//
// Pair i of a head (elements 2i, 2i+1, or i and P+i) at a token whose position
// along the pair's axis is p turns by t = p f_i:
//     (x, y) -> scale (x cos t - y sin t, x sin t + y cos t);
// with t -> -t the map is the transpose, which is its gradient.  Both kernels move
// bytes: every element is read and written once, and the angle is shared by all
// heads of a token, so a thread keeps the angles of V pairs (two pieces of V
// elements) in registers and walks over heads with them.
//
// The angle: p f_i is formed in fp64 (a product of 24-bit factors is exact there;
// in fp32, position 10^5 leaves an angle an error of 4e-3), divided by 2 pi, its
// nearest whole number of turns taken away, and only the rest, in [-1/2, 1/2]
// turns, is rounded to fp32 for sincospi.
#pragma once

#include "hsq_device.cuh"

namespace hsq {

constexpr int kRopeMaxPairs = 256;
constexpr int kRopeThreads = 256;
// heads whose pieces a thread requests before it uses the first
constexpr int kRopeBatch = 4;

enum PosType { kPosI32 = 0, kPosI64 = 1, kPosF32 = 2 };
enum HeadType { kHeadBf16 = 0, kHeadF32 = 1, kHeadE4m3 = 2 };

// A rotation and the positions it reads.
struct RopeTable {
  const float* freqs;  // [pairs]
  const void* pos;     // [pos_rows][pos_ld], or nullptr: the caller's own position on every axis
  long long pos_ld;
  int pairs, pos_type, pos_rows;
  float scale, sign;               // sign: -1 for the transpose
  uint32_t axis2[kRopeMaxPairs / 16];  // two bits a pair: its axis
};

struct HeadsView {
  void* data;
  long long ts, hs;  // elements between tokens, and between heads
};

__device__ __forceinline__ double rope_position(const RopeTable& t, size_t row, int axis) {
  const size_t at = row * static_cast<size_t>(t.pos_ld) + axis;
  if (t.pos_type == kPosI32) return static_cast<double>(__ldg(static_cast<const int*>(t.pos) + at));
  if (t.pos_type == kPosI64) return static_cast<double>(__ldg(static_cast<const long long*>(t.pos) + at));
  return static_cast<double>(__ldg(static_cast<const float*>(t.pos) + at));
}

// cos and sin (times scale) of pair i at a token: its row of the positions, or
// position `own`.
__device__ __forceinline__ void rope_angle(const RopeTable& t, int i, size_t row, double own, float& c, float& s) {
  const int axis = (t.axis2[i >> 4] >> (2 * (i & 15))) & 3;
  const double p = t.pos ? rope_position(t, row, axis) : own;
  const double turns = p * static_cast<double>(__ldg(t.freqs + i)) * 0.15915494309189534;
  const double rest = turns - rint(turns);
  sincospif(2.f * static_cast<float>(rest), &s, &c);
  c *= t.scale;
  s *= t.scale * t.sign;
}

// V consecutive elements of a head as fp32, and back.
template <typename T, int V>
__device__ __forceinline__ void load_piece(const T* p, float (&f)[V]) {
  if constexpr (sizeof(T) == 2 && V == 8) {
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), f);
  } else if constexpr (sizeof(T) == 2 && V == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.y));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  } else if constexpr (sizeof(T) == 4 && V == 4) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    f[0] = w.x; f[1] = w.y; f[2] = w.z; f[3] = w.w;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = static_cast<float>(p[j]);
  }
}

// Two values -> two E4M3 bytes (the first in the low byte): nearest, ties to
// even, saturating at 448; NaN stays NaN.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int V>
__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const float (&f)[V]) {
  if constexpr (V % 4 == 0) {
    uint32_t w[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = __float2bfloat16_rn(f[j]);
  }
}
template <int V>
__device__ __forceinline__ void store_piece(float* p, const float (&f)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<float4*>(p + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = f[j];
  }
}
template <int V>
__device__ __forceinline__ void store_piece(uint8_t* p, const float (&f)[V]) {
  if constexpr (V % 4 == 0) {
    uint32_t w[V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j)
      w[j] = static_cast<uint32_t>(e4m3x2(f[4 * j], f[4 * j + 1])) |
             (static_cast<uint32_t>(e4m3x2(f[4 * j + 2], f[4 * j + 3])) << 16);
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = static_cast<uint8_t>(e4m3x2(f[j], 0.f) & 0xffu);
  }
}

// The unit of work along a head: for u < P / V two pieces of V elements that
// hold V whole pairs, and behind them the pieces that no pair covers.
//   halves, and V = 1: the pairs join element j of one piece and of the other;
//   adjacent pairs: each piece holds V / 2 pairs.
template <int V, bool ADJ>
struct RopeUnit {
  int a, b;     // element offsets of the pieces; b < 0: one piece, not rotated
  int pa, pb;   // first pair of each piece (ADJ with V > 1), or of the pairing (pa)
  __device__ __forceinline__ RopeUnit(int u, int P) {
    const int ru = P / V;
    if (u >= ru) {
      a = 2 * P + (u - ru) * V;
      b = -1;
      pa = pb = 0;
    } else if (ADJ && V == 1) {
      a = 2 * u;
      b = 2 * u + 1;
      pa = pb = u;
    } else {
      a = u * V;
      b = P + u * V;
      pa = ADJ ? a / 2 : a;
      pb = ADJ ? b / 2 : a;
    }
  }
  // the pair whose angle is kept at place j (of V)
  __device__ __forceinline__ int pair(int j) const {
    return (ADJ && V > 1) ? (j < V / 2 ? pa + j : pb + j - V / 2) : pa + j;
  }
  static __device__ __forceinline__ void rotate(float (&x)[V], float (&y)[V], const float (&c)[V], const float (&s)[V]) {
    auto turn = [](float& p, float& q, float cc, float ss) {
      const float p0 = p;
      p = fmaf(p0, cc, -q * ss);
      q = fmaf(p0, ss, q * cc);
    };
    if constexpr (ADJ && V > 1) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        turn(x[2 * j], x[2 * j + 1], c[j], s[j]);
        turn(y[2 * j], y[2 * j + 1], c[V / 2 + j], s[V / 2 + j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) turn(x[j], y[j], c[j], s[j]);
    }
  }
};

struct RopeArgs {
  HeadsView x, y;
  RopeTable rot;
  int tokens, heads, dim;
  int units;      // of a head: P / V, and the unrotated pieces unless x is y
  int splits;     // threads that share a (token, unit)'s heads
  int per_split;  // heads of each
};

// Thread (token, split, unit), units fastest: neighbours read neighbouring
// pieces of one head.
template <typename T, int V, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  grid_dep_wait();  // x comes from the preceding kernel
  if (threadIdx.x == 0) grid_dep_launch();
  const long long idx = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long row = idx / a.units;
  const int u = static_cast<int>(idx - row * a.units);
  const long long tok = row / a.splits;
  if (tok >= a.tokens) return;
  const int h0 = static_cast<int>(row - tok * a.splits) * a.per_split, h1 = min(a.heads, h0 + a.per_split);
  const RopeUnit<V, ADJ> un(u, a.rot.pairs);
  const T* x = static_cast<const T*>(a.x.data) + tok * a.x.ts;
  T* y = static_cast<T*>(a.y.data) + tok * a.y.ts;
  float c[V], s[V];
  if (un.b >= 0) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      rope_angle(a.rot, un.pair(j), static_cast<size_t>(tok % a.rot.pos_rows), 0.0, c[j], s[j]);
  }
  for (int h = h0; h < h1; h += kRopeBatch) {
    float p[kRopeBatch][V], q[kRopeBatch][V];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i)
      if (h + i < h1) {
        load_piece<T, V>(x + (h + i) * a.x.hs + un.a, p[i]);
        if (un.b >= 0) load_piece<T, V>(x + (h + i) * a.x.hs + un.b, q[i]);
      }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i)
      if (h + i < h1) {
        if (un.b >= 0) {
          RopeUnit<V, ADJ>::rotate(p[i], q[i], c, s);
          store_piece<V>(y + (h + i) * a.y.hs + un.b, q[i]);
        }
        store_piece<V>(y + (h + i) * a.y.hs + un.a, p[i]);
      }
  }
}

struct CacheView {
  void* data;
  long long ps, ss, hs;  // elements between pages, between slots, between heads
  const float* scale;    // E4M3: [kv_heads], or nullptr for 1
};

struct AppendArgs {
  HeadsView k, v, q, q_out;
  CacheView kc, vc;
  RopeTable rot;       // pairs = 0: no rotation
  const int* table;    // [seqs][table_ld] page of each page_size tokens
  const int* lens;     // [seqs] tokens already cached; negative: the sequence takes no part
  const int* cu;       // [seqs + 1], or nullptr: token t is sequence t's
  long long table_ld;
  int tokens, seqs, q_heads, kv_heads, dim;
  int pages, page_size, max_pages;
  int units, splits, per_split;
  int q_in_place;
};

// Token t's sequence (the last b with cu[b] <= t, by halving) and its place; false
// for rows in front of the first sequence or behind the last.
__device__ __forceinline__ bool append_place(const AppendArgs& a, int t, int& seq, long long& pos) {
  int b = t;
  int first = t;
  if (a.cu) {
    int lo = 0, hi = a.seqs;  // cu[lo] <= t < cu[hi] once both ends have been checked
    if (t < __ldg(a.cu) || t >= __ldg(a.cu + a.seqs)) return false;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    first = __ldg(a.cu + lo);
  }
  const int len = __ldg(a.lens + b);
  if (len < 0) return false;
  seq = b;
  pos = static_cast<long long>(len) + (t - first);
  return true;
}

// Thread (token, split, unit) as in rope_kernel; its heads are the q heads, then
// the k heads, then the v heads.  C: the cache's element type.
template <typename T, typename C, int V, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  grid_dep_wait();
  if (threadIdx.x == 0) grid_dep_launch();
  const long long idx = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long row = idx / a.units;
  const int u = static_cast<int>(idx - row * a.units);
  const long long tok = row / a.splits;
  if (tok >= a.tokens) return;
  const int nh = a.q_heads + 2 * a.kv_heads;
  const int h0 = static_cast<int>(row - tok * a.splits) * a.per_split, h1 = min(nh, h0 + a.per_split);
  const RopeUnit<V, ADJ> un(u, a.rot.pairs);
  int seq = 0;
  long long pos = 0;
  if (!append_place(a, static_cast<int>(tok), seq, pos)) return;
  // the page: a table entry outside the cache, or a place outside the table, is
  // reported and nothing is written for the token's k and v
  const long long pi = pos / a.page_size;
  int page = -1;
  if (h1 > a.q_heads) {
    if (pi < a.max_pages) page = __ldg(a.table + static_cast<long long>(seq) * a.table_ld + pi);
    if (page < 0 || page >= a.pages) {
      page = -1;
      atomicOr(&g_status, kStatusBadPage);
    }
  }
  const long long slot = pos - pi * a.page_size;
  float c[V], s[V];
  if (un.b >= 0 && h0 < a.q_heads + a.kv_heads) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      rope_angle(a.rot, un.pair(j), static_cast<size_t>(tok), static_cast<double>(pos), c[j], s[j]);
  }
  const T* xq = static_cast<const T*>(a.q.data) + tok * a.q.ts;
  const T* xk = static_cast<const T*>(a.k.data) + tok * a.k.ts;
  const T* xv = static_cast<const T*>(a.v.data) + tok * a.v.ts;
  for (int h = h0; h < h1; h += kRopeBatch) {
    float p[kRopeBatch][V], q[kRopeBatch][V];
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i)
      if (h + i < h1) {
        const int e = h + i;
        const T* x = e < a.q_heads ? xq + e * a.q.hs
                     : e < a.q_heads + a.kv_heads ? xk + (e - a.q_heads) * a.k.hs
                                                  : xv + (e - a.q_heads - a.kv_heads) * a.v.hs;
        load_piece<T, V>(x + un.a, p[i]);
        if (un.b >= 0) load_piece<T, V>(x + un.b, q[i]);
      }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i)
      if (h + i < h1) {
        const int e = h + i;
        if (un.b >= 0 && e < a.q_heads + a.kv_heads) RopeUnit<V, ADJ>::rotate(p[i], q[i], c, s);
        if (e < a.q_heads) {
          T* y = static_cast<T*>(a.q_out.data) + tok * a.q_out.ts + e * a.q_out.hs;
          if (un.b >= 0) store_piece<V>(y + un.b, q[i]);
          if (un.b >= 0 || !a.q_in_place) store_piece<V>(y + un.a, p[i]);
        } else if (page >= 0) {
          const bool is_k = e < a.q_heads + a.kv_heads;
          const CacheView& cv = is_k ? a.kc : a.vc;
          const int hd = e - a.q_heads - (is_k ? 0 : a.kv_heads);
          C* y = static_cast<C*>(cv.data) + page * cv.ps + slot * cv.ss + hd * cv.hs;
          if constexpr (sizeof(C) == 1) {
            if (cv.scale) {
              const float sc = __ldg(cv.scale + hd);
#pragma unroll
              for (int j = 0; j < V; ++j) {
                p[i][j] = __fdiv_rn(p[i][j], sc);
                if (un.b >= 0) q[i][j] = __fdiv_rn(q[i][j], sc);
              }
            }
          }
          store_piece<V>(y + un.a, p[i]);
          if (un.b >= 0) store_piece<V>(y + un.b, q[i]);
        }
      }
  }
}

}  // namespace hsq
