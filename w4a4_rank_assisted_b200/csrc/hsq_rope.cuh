// hsq_rope.cuh -- rotary positions at the output of a fused QKV linear, and the
// paged cache append that rotates on the way.
//
// Pair i of a head (elements 2i, 2i+1, or i and P+i) at a token whose position
// along the pair's axis is p turns by t = p f_i:
//     (x, y) -> scale (x cos t - y sin t, x sin t + y cos t);
// with t -> -t the map is the transpose, which is its gradient.  Both kernels move
// bytes: every element is read and written once, and the angles are shared by all
// heads of a token.  A block takes a few tokens with all their heads (as many as fit):
// it forms each token's angles once, into shared memory, while the first pieces that
// its threads have requested are on their way; then every thread rotates its pieces of
// two heads, pass by pass, the next pass's pieces requested first.  (A thread that
// formed its own angles and walked over the heads took twice as long.)
//
// Bound by memory once there are enough tokens: 20.1 us at 4608 tokens x 48 heads x 128
// in bf16 (113 MB: 5.6 TB/s, 0.86 of the copy rate), 26.3 us at 15606 x 16 x 80 in fp32
// (160 MB: 0.93), 42.5 us for the append of 9203 tokens of 32 + 8 + 8 heads x 128 (226 MB:
// 0.81); by launch and latency below: 2.2 us for one token's rotation, 3.2 us for its
// append (a page lookup is loads that depend on one another).
//
// The angle: p f_i is formed in fp64 (a product of 24-bit factors is exact there;
// in fp32, position 10^5 leaves an angle an error of 4e-3), divided by 2 pi, its
// nearest whole number of turns taken away, and only the rest, in [-1/2, 1/2]
// turns, is rounded to fp32 for sincospi.
#pragma once

#include <type_traits>

#include "hsq_device.cuh"

namespace hsq {

constexpr int kRopeMaxPairs = 256;
constexpr int kRopeThreads = 256;  // most threads of a block
// Heads of a thread and a pass.  Four leave room for two blocks per SM instead of three:
// 21.8 against 20.1 us (4608 tokens x 48 heads x 128, bf16), 54 against 26.3 (15606 x 16 x
// 80, fp32).
constexpr int kRopeHeads = 2;
constexpr int kRopeShared = 32768;  // shared memory of a block's tokens: their angles and cache rows

enum PosType { kPosI32 = 0, kPosI64 = 1, kPosF32 = 2 };

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

// V consecutive elements of a head as loaded (one access), and as fp32.  What is only
// moved is stored as loaded: through fp32 a bf16 NaN would lose its sign and payload.
template <typename T, int V>
struct Piece {
  uint32_t w[V * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(w) == 16) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (sizeof(w) == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    else return __uint_as_float((j & 1) ? (w[j / 2] & 0xffff0000u) : (w[j / 2] << 16));
  }
};
template <typename T>
struct Piece<T, 1> {
  T x;
  __device__ __forceinline__ void load(const T* p) { x = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = x; }
  __device__ __forceinline__ float at(int) const { return static_cast<float>(x); }
};

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
  __device__ __forceinline__ int second() const { return b < 0 ? a : b; }  // (always readable)
  // the pair whose angle is kept at place j (of V)
  __device__ __forceinline__ int pair(int j) const {
    return (ADJ && V > 1) ? (j < V / 2 ? pa + j : pb + j - V / 2) : pa + j;
  }
  // cos and sin of the unit's places at one token (ang: its pairs; 16-byte aligned for V > 1)
  __device__ __forceinline__ void angles(const float2* ang, float (&c)[V], float (&s)[V]) const {
    if constexpr (V == 1) {
      const float2 cs = ang[pa];
      c[0] = cs.x;
      s[0] = cs.y;
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float4 cs = *reinterpret_cast<const float4*>(ang + pair(j));
        c[j] = cs.x; s[j] = cs.y;
        c[j + 1] = cs.z; s[j + 1] = cs.w;
      }
    }
  }
  // the pieces (p, q) turned by the angles (c, s): x and y of pair j are gathered, two
  // pairs a packed instruction
  static __device__ __forceinline__ void rotate(float (&p)[V], float (&q)[V], const float (&c)[V], const float (&s)[V]) {
    auto x = [&](int j) -> float& { return (ADJ && V > 1) ? (j < V / 2 ? p[2 * j] : q[2 * j - V]) : p[j]; };
    auto y = [&](int j) -> float& { return (ADJ && V > 1) ? (j < V / 2 ? p[2 * j + 1] : q[2 * j + 1 - V]) : q[j]; };
    if constexpr (V == 1) {
      const float x0 = p[0];
      p[0] = fmaf(x0, c[0], q[0] * -s[0]);
      q[0] = fmaf(x0, s[0], q[0] * c[0]);
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const float2 xx = make_float2(x(j), x(j + 1)), yy = make_float2(y(j), y(j + 1));
        const float2 cc = make_float2(c[j], c[j + 1]), ss = make_float2(s[j], s[j + 1]);
        const float2 u = __ffma2_rn(xx, cc, __fmul2_rn(yy, make_float2(-ss.x, -ss.y)));
        const float2 v = __ffma2_rn(xx, ss, __fmul2_rn(yy, cc));
        x(j) = u.x; x(j + 1) = u.y;
        y(j) = v.x; y(j + 1) = v.y;
      }
    }
  }
};

// How a call is cut into blocks: a block takes `passes` times `tokens` tokens and
// `splits` x kRopeHeads heads, its threads (token, split, unit) with the units fastest
// (neighbours read neighbouring pieces of a head); grid (token blocks, head blocks).
// A head of more than kRopeThreads units is walked over.
struct RopeGrid {
  int units, lanes;  // pieces to walk, threads on them
  int splits, tokens, passes;
};

struct RopeArgs {
  HeadsView x, y;
  RopeTable rot;
  RopeGrid g;
  int tokens, heads;
};

template <typename T, int V, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 4 ? 4 : 3) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) float2 rope_angles[];  // [tokens of the block][pairs]
  grid_dep_wait();  // x comes from the preceding kernel
  if (threadIdx.x == 0) grid_dep_launch();
  const int t = threadIdx.x, P = a.rot.pairs;
  const int u0 = t % a.g.lanes, slot = t / a.g.lanes, sp = slot % a.g.splits, tk = slot / a.g.splits;
  const int t0 = static_cast<int>(blockIdx.x) * a.g.tokens * a.g.passes;  // (below tokens)
  const int n = min(a.g.tokens * a.g.passes, a.tokens - t0);              // tokens of the block
  const int h0 = (static_cast<int>(blockIdx.y) * a.g.splits + sp) * kRopeHeads;
  // the thread's pieces of its first token; out of range: the block's last token and
  // the last head are read, and nothing is written
  RopeUnit<V, ADJ> un(u0, P);
  Piece<T, V> p[kRopeHeads], q[kRopeHeads];
  const T* x[kRopeHeads];
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    x[i] = static_cast<const T*>(a.x.data) + (t0 + min(tk, n - 1)) * a.x.ts + min(h0 + i, a.heads - 1) * a.x.hs;
    p[i].load(x[i] + un.a);
    q[i].load(x[i] + un.second());
  }
  for (int i = t; i < n * P; i += blockDim.x) {
    const int k = i / P, j = i - k * P;
    float c, s;
    rope_angle(a.rot, j, static_cast<size_t>((t0 + k) % a.rot.pos_rows), 0.0, c, s);
    rope_angles[i] = make_float2(c, s);
  }
  __syncthreads();
  if (tk >= a.g.tokens || h0 >= a.heads) return;
  T* y = static_cast<T*>(a.y.data) + (t0 + tk) * a.y.ts + h0 * a.y.hs;
  const long long x_step = a.g.tokens * a.x.ts, y_step = a.g.tokens * a.y.ts;
  int u = u0;
  for (int k = tk; k < n;) {
    const RopeUnit<V, ADJ> now = un;
    T* yk = y;
    float c[V], s[V];
    if (now.b >= 0) now.angles(rope_angles + k * P, c, s);
    Piece<T, V> pc[kRopeHeads], qc[kRopeHeads];
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i) {
      pc[i] = p[i];
      qc[i] = q[i];
    }
    // the next pass's pieces (with V > 1 a thread has one unit of every token)
    if (V == 1 && (u += a.g.lanes) < a.g.units) {
      un = RopeUnit<V, ADJ>(u, P);
    } else {
      k += a.g.tokens;
      y += y_step;
      if constexpr (V == 1) un = RopeUnit<V, ADJ>(u = u0, P);
#pragma unroll
      for (int i = 0; i < kRopeHeads; ++i) x[i] += x_step;
    }
    if (k < n) {
#pragma unroll
      for (int i = 0; i < kRopeHeads; ++i) {
        p[i].load(x[i] + un.a);
        q[i].load(x[i] + un.second());
      }
    }
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i) {
      if (h0 + i >= a.heads) break;
      if (now.b >= 0) {
        float f[V], g[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          f[j] = pc[i].at(j);
          g[j] = qc[i].at(j);
        }
        RopeUnit<V, ADJ>::rotate(f, g, c, s);
        store_piece<V>(yk + now.b, g);
        store_piece<V>(yk + now.a, f);
      } else {
        pc[i].store(yk + now.a);
      }
      yk += a.y.hs;
    }
  }
}

struct CacheView {
  void* data;
  long long ps, ss, hs;  // elements between pages, between slots, between heads (k's and v's alike)
  const float* scale;    // E4M3: [kv_heads], or nullptr for 1
};

struct AppendArgs {
  HeadsView k, v, q, q_out;
  CacheView kc, vc;
  RopeTable rot;       // pairs = 0: no rotation
  RopeGrid g;          // over the q heads, then the k heads, then the v heads
  const int* table;    // [seqs][table_ld] page of each page_size tokens
  const int* lens;     // [seqs] tokens already cached; negative: the sequence takes no part
  const int* cu;       // [seqs + 1], or nullptr: token t is sequence t's
  long long table_ld;
  int tokens, seqs, q_heads, kv_heads;
  int pages, page_size, max_pages;
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

// What a block knows of one of its tokens: its place in its sequence (negative: it
// takes no part), and the cache row it goes to (page < 0: none).
struct AppendToken {
  long long pos;
  int page, slot;
};

// C: the cache's element type.
template <typename T, typename C, int V, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, 3) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  extern __shared__ __align__(16) float2 rope_angles[];  // [tokens of the block][pairs], then the tokens
  AppendToken* toks = reinterpret_cast<AppendToken*>(rope_angles + a.g.tokens * a.g.passes * a.rot.pairs);
  grid_dep_wait();
  if (threadIdx.x == 0) grid_dep_launch();
  const int t = threadIdx.x, P = a.rot.pairs;
  const int u0 = t % a.g.lanes, slot = t / a.g.lanes, sp = slot % a.g.splits, tk = slot / a.g.splits;
  const int t0 = static_cast<int>(blockIdx.x) * a.g.tokens * a.g.passes;  // (below tokens)
  const int n = min(a.g.tokens * a.g.passes, a.tokens - t0);              // tokens of the block
  const int nh = a.q_heads + 2 * a.kv_heads, nr = a.q_heads + a.kv_heads;
  const int h0 = (static_cast<int>(blockIdx.y) * a.g.splits + sp) * kRopeHeads;
  Piece<T, V> p[kRopeHeads], q[kRopeHeads];
  auto load = [&](int k, const RopeUnit<V, ADJ>& un) {
    const long long tok = t0 + min(k, n - 1);
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i) {
      const int e = min(h0 + i, nh - 1);
      const HeadsView& src = e < a.q_heads ? a.q : e < nr ? a.k : a.v;
      const int hd = e - (e < a.q_heads ? 0 : e < nr ? a.q_heads : nr);
      const T* x = static_cast<const T*>(src.data) + tok * src.ts + hd * src.hs;
      p[i].load(x + un.a);
      q[i].load(x + (un.b < 0 ? un.a : un.b));
    }
  };
  load(tk, RopeUnit<V, ADJ>(u0, P));
  for (int k = t; k < n; k += blockDim.x) {
    AppendToken o{-1, -1, 0};
    int seq = 0;
    if (append_place(a, t0 + k, seq, o.pos)) {
      // the page: a table entry outside the cache, or a place outside the table, is
      // reported and nothing is written for the token's k and v
      const long long pi = o.pos >> 32 ? o.pos / a.page_size
                                       : static_cast<long long>(static_cast<uint32_t>(o.pos) / static_cast<uint32_t>(a.page_size));
      if (pi < a.max_pages) o.page = __ldg(a.table + static_cast<long long>(seq) * a.table_ld + pi);
      if (o.page < 0 || o.page >= a.pages) {
        o.page = -1;
        atomicOr(&g_status, kStatusBadPage);
      }
      o.slot = static_cast<int>(o.pos - pi * a.page_size);
    }
    toks[k] = o;
  }
  __syncthreads();
  for (int i = t; i < n * P; i += blockDim.x) {
    const int k = i / P, j = i - k * P;
    float c, s;
    rope_angle(a.rot, j, static_cast<size_t>(t0 + k), static_cast<double>(toks[k].pos), c, s);
    rope_angles[i] = make_float2(c, s);
  }
  __syncthreads();
  if (tk >= a.g.tokens || h0 >= nh) return;
  const int walk = (a.g.units - u0 + a.g.lanes - 1) / a.g.lanes;  // units of this thread
  for (int k = tk, w = 0; k < n;) {
    const AppendToken me = toks[k];
    const long long tok = t0 + k;
    const float2* ang = rope_angles + k * P;
    const RopeUnit<V, ADJ> un(u0 + w * a.g.lanes, P);
    Piece<T, V> pc[kRopeHeads], qc[kRopeHeads];
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i) {
      pc[i] = p[i];
      qc[i] = q[i];
    }
    if (++w == walk) {
      w = 0;
      k += a.g.tokens;
    }
    if (k < n) load(k, RopeUnit<V, ADJ>(u0 + w * a.g.lanes, P));  // the next pass's pieces
    if (me.pos < 0) continue;
    float c[V], s[V];
    if (un.b >= 0) un.angles(ang, c, s);
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i) {
      const int e = h0 + i;
      if (e >= nh) break;
      const bool turned = un.b >= 0 && e < nr, is_q = e < a.q_heads, is_k = !is_q && e < nr;
      const int hd = e - (is_q ? 0 : is_k ? a.q_heads : nr);
      auto q_row = [&] { return static_cast<T*>(a.q_out.data) + tok * a.q_out.ts + hd * a.q_out.hs; };
      auto cache_row = [&](const CacheView& cv) {
        return static_cast<C*>(cv.data) + me.page * cv.ps + me.slot * cv.ss + hd * cv.hs;
      };
      auto values = [&](float (&f)[V], float (&g)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          f[j] = pc[i].at(j);
          g[j] = qc[i].at(j);
        }
        if (turned) RopeUnit<V, ADJ>::rotate(f, g, c, s);
      };
      if constexpr (std::is_same_v<T, C>) {
        if (!is_q && me.page < 0) continue;
        T* y = is_q ? q_row() : cache_row(is_k ? a.kc : a.vc);
        if (turned) {
          float f[V], g[V];
          values(f, g);
          store_piece<V>(y + un.a, f);
          store_piece<V>(y + un.b, g);
        } else {
          if (!is_q || !a.q_in_place) pc[i].store(y + un.a);
          if (un.b >= 0) qc[i].store(y + un.b);
        }
      } else {
        float f[V], g[V];
        values(f, g);
        if (is_q) {
          T* y = q_row();
          if (turned) {
            store_piece<V>(y + un.b, g);
            store_piece<V>(y + un.a, f);
          } else if (!a.q_in_place) {
            pc[i].store(y + un.a);
          }
        } else if (me.page >= 0) {
          const CacheView& cv = is_k ? a.kc : a.vc;
          C* y = cache_row(cv);
          if constexpr (sizeof(C) == 1) {
            if (cv.scale) {
              const float sc = __ldg(cv.scale + hd);
#pragma unroll
              for (int j = 0; j < V; ++j) {
                f[j] = __fdiv_rn(f[j], sc);
                g[j] = __fdiv_rn(g[j], sc);
              }
            }
          }
          store_piece<V>(y + un.a, f);
          if (un.b >= 0) store_piece<V>(y + un.b, g);
        }
      }
    }
  }
}

}  // namespace hsq
