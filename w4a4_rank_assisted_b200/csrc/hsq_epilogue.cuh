// hsq_epilogue.cuh -- the linear's epilogue beyond U L2 + b:
//
//     Y[m,n] = act(z[m,n]) * mul[m / mul_rows, n] + residual[m,n],
//     z = sum_g sx sw P_g + U L2 + b,
//
// applied to the fp32 accumulators before the one rounding to the output type,
// so that a block's activation, gate and residual cost no pass over Y of their
// own (a separate pass reads and writes M N elements once more, and rounds z to
// 16 bits first).  act: identity, relu, gelu in its tanh and erf forms, silu.
// mul is the other half of a gated MLP (mul_rows = 1) or a modulation vector per
// sample (mul_rows = the sample's tokens); either operand is bf16 or fp32.
//
// silu(z) = z / (1 + e^-z), and the tanh gelu 0.5 z (1 + tanh u) = z / (1 + e^-2u)
// with u = sqrt(2/pi) (z + 0.044715 z^3): one exponential and one quotient each,
// to a few 2^-23 relative.  The erf gelu is
//     max(z, 0) - |z|/2 erfc(|z| / sqrt 2),   erfc(w) = e^(-w^2) t Q(t), t = 1 / (1 + 0.45 w),
// Q of degree 9 fitted to erfc(w) e^(w^2) / t over all w >= 0 for the least largest
// relative error (3.3e-8): the complement keeps its relative accuracy for negative
// z, where 1 + erf cancels, at two special-function instructions like the others.
#pragma once

#include "hsq_device.cuh"

namespace hsq {

// The same numbers as hsq_act in include/hsq.h.
enum EpiAct { kActNone = 0, kActRelu = 1, kActGeluTanh = 2, kActGeluErf = 3, kActSilu = 4 };

struct EpiArgs {
  const void* mul;  // [ceil(M / mul_rows)] rows of N, mul_ld apart, or nullptr
  const void* res;  // [M] rows of N, res_ld apart, or nullptr (may be Y itself)
  long long mul_ld, res_ld;
  int act, mul_rows, mul_f32, res_f32;
};

// z / (1 + 2^t) of two values: two special-function instructions each.  2^t overflows
// to infinity, whose reciprocal is 0, where the quotient is below 2^-126 |z|.
__device__ __forceinline__ float epi_ex2(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
__device__ __forceinline__ float epi_rcp(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}
__device__ __forceinline__ float2 epi_sigmoid_form(const float2& z, const float2& t) {
  const float2 d = __fadd2_rn(make_float2(epi_ex2(t.x), epi_ex2(t.y)), make_float2(1.f, 1.f));
  return __fmul2_rn(z, make_float2(epi_rcp(d.x), epi_rcp(d.y)));
}

__device__ __forceinline__ float2 epi_gelu_erf(const float2& z) {
  // beyond 64 the product below is 0 (of an infinity it would be NaN)
  const float2 a = make_float2(fminf(fabsf(z.x), 64.f), fminf(fabsf(z.y), 64.f));
  constexpr float kT = 0.45f * 0.70710678118654752f, kE = -0.5f * 1.4426950408889634f;
  const float2 d = __ffma2_rn(a, make_float2(kT, kT), make_float2(1.f, 1.f));
  const float2 t = make_float2(epi_rcp(d.x), epi_rcp(d.y));
  const float2 w = __fmul2_rn(__fmul2_rn(a, make_float2(kE, kE)), a);
  constexpr float c[10] = {0.25388532876968384f, 0.25388315320014954f,  0.22827163338661194f,   0.17525216937065125f,
                           0.11995021998882294f, -0.022357264533638954f, 0.14239974319934845f,  -0.3005811870098114f,
                           0.1906871646642685f,  -0.04139094427227974f};
  float2 q = make_float2(c[9], c[9]);
#pragma unroll
  for (int i = 8; i >= 0; --i) q = __ffma2_rn(q, t, make_float2(c[i], c[i]));
  q = __fmul2_rn(__fmul2_rn(q, t), make_float2(epi_ex2(w.x), epi_ex2(w.y)));
  return __ffma2_rn(__fmul2_rn(a, make_float2(-0.5f, -0.5f)), q,
                    make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y));
}

template <int ACT>
__device__ __forceinline__ float2 epi_act(const float2& z) {
  constexpr float kLog2e = 1.4426950408889634f, kTanh = -2.f * 0.79788456080286536f * kLog2e;
  if constexpr (ACT == kActRelu) return make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);
  if constexpr (ACT == kActGeluTanh) {
    const float2 p = __ffma2_rn(__fmul2_rn(z, make_float2(0.044715f, 0.044715f)), z, make_float2(1.f, 1.f));
    return epi_sigmoid_form(z, __fmul2_rn(__fmul2_rn(z, make_float2(kTanh, kTanh)), p));
  }
  if constexpr (ACT == kActGeluErf) return epi_gelu_erf(z);
  if constexpr (ACT == kActSilu) return epi_sigmoid_form(z, __fmul2_rn(z, make_float2(-kLog2e, -kLog2e)));
  return z;
}

// act of the pairs that each(f) hands to f, in place.  The switch stands outside: it
// is uniform over the launch, and a launch then runs through one activation's code
// only.
template <class Each>
__device__ __forceinline__ void epi_act_each(int act, Each&& each) {
  switch (act) {
    case kActRelu: each([](float2& z) { z = epi_act<kActRelu>(z); }); break;
    case kActGeluTanh: each([](float2& z) { z = epi_act<kActGeluTanh>(z); }); break;
    case kActGeluErf: each([](float2& z) { z = epi_act<kActGeluErf>(z); }); break;
    case kActSilu: each([](float2& z) { z = epi_act<kActSilu>(z); }); break;
    default: break;
  }
}

// Element n of mul's row for token m, and of residual's row m (1 and 0 where
// there is none).  Plain loads: residual may be Y itself, each of whose elements
// the thread that writes it reads first.
__device__ __forceinline__ float epi_scalar(const void* p, int f32, size_t at) {
  return f32 ? static_cast<const float*>(p)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ float epi_mul_at(const EpiArgs& e, int m, int n) {
  if (!e.mul) return 1.f;
  const int row = e.mul_rows == 1 ? m : m / e.mul_rows;
  return epi_scalar(e.mul, e.mul_f32, static_cast<size_t>(row) * e.mul_ld + n);
}
__device__ __forceinline__ float epi_res_at(const EpiArgs& e, int m, int n) {
  return e.res ? epi_scalar(e.res, e.res_f32, static_cast<size_t>(m) * e.res_ld + n) : 0.f;
}

// act(z) * mul + residual of N elements in place.
template <int N>
__device__ __forceinline__ void epi_values(const EpiArgs& e, float (&z)[N], const float (&mul)[N], const float (&res)[N]) {
  epi_act_each(e.act, [&](auto&& f) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float2 p = make_float2(z[i], i + 1 < N ? z[i + 1] : 0.f);
      f(p);
      z[i] = p.x;
      if (i + 1 < N) z[i + 1] = p.y;
    }
  });
  if (e.mul) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] *= mul[i];
  }
  if (e.res) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] += res[i];
  }
}

// Requests the lines of mul and residual under rows m0 .. m0 + 31, columns n0 ..
// n0 + CW - 1 of Y into L2 (a lane per row and 128 bytes), for the loads that follow
// the tile's sums.
template <int CW>
__device__ __forceinline__ void epi_prefetch(const EpiArgs& e, int m0, int n0, int M, int N) {
  const int m = m0 + lane_id();
  if (m >= M) return;
  auto rows = [&](const void* p, int f32, long long ld, int row) {
    const char* at = static_cast<const char*>(p) + (static_cast<size_t>(row) * ld + n0) * (f32 ? 4 : 2);
    const int bytes = min(CW, N - n0) * (f32 ? 4 : 2);
    for (int o = 0; o < bytes; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + o));
  };
  if (n0 >= N) return;
  if (e.mul && e.mul_rows == 1) rows(e.mul, e.mul_f32, e.mul_ld, m);
  if (e.res) rows(e.res, e.res_f32, e.res_ld, m);
}

// One operand's box under the warp's part of Y: 32 rows of 128 bytes (64 bf16 or 32
// fp32 columns), eight lanes to a row, so that each access covers whole lines.
// fetch requests HOLD of its 8 accesses into registers, land lays the box in the warp's
// staging buffer (16-byte chunk c of row r at chunk c ^ (r % 8): the writes, and the
// readers' pairs, touch 32 different banks).  Rows behind M read row M - 1 and columns
// behind N the row's first ones: nothing outside the operand is read, and those
// outputs are clipped by the TMA unit.
struct EpiOperand {
  const void* p;
  long long ld;
  int rows;  // tokens to a row
  bool f32;
};
template <int HOLD>
struct EpiBox {
  uint4 w[HOLD];
  __device__ __forceinline__ void fetch(const EpiOperand& o, int y0, int n0, int M, int N, int part = 0) {
    const int lane = lane_id();
    int n = n0 + (lane & 7) * (o.f32 ? 4 : 8);
    if (n >= N) n = 0;
    const char* base = static_cast<const char*>(o.p) + static_cast<size_t>(n) * (o.f32 ? 4 : 2);
    const size_t pitch = static_cast<size_t>(o.ld) * (o.f32 ? 4 : 2);
    const int m0 = y0 + 4 * HOLD * part + (lane >> 3);
    if (o.rows == 1) {
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        w[i] = *reinterpret_cast<const uint4*>(base + static_cast<size_t>(min(m0 + 4 * i, M - 1)) * pitch);
    } else {
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        w[i] = *reinterpret_cast<const uint4*>(base + static_cast<size_t>(min(m0 + 4 * i, M - 1) / o.rows) * pitch);
    }
  }
  // Defines the registers where nothing is fetched.  A conditional load alone leaves
  // them live from the loop over tiles on, and the accumulators spill.
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int i = 0; i < HOLD; ++i)
      asm volatile("" : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w));
  }
  __device__ __forceinline__ void put(uint8_t* stg, int part) const {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int r = 4 * (HOLD * part + i) + (lane >> 3);
      *reinterpret_cast<uint4*>(stg + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) = w[i];
    }
  }
  // the box whose first part has been fetched, into stg
  __device__ __forceinline__ void land(const EpiOperand& o, uint8_t* stg, int y0, int n0, int M, int N) {
    __syncwarp();  // the box before has been read
    put(stg, 0);
#pragma unroll
    for (int part = 1; part < 8 / HOLD; ++part) {
      fetch(o, y0, n0, M, N, part);
      put(stg, part);
    }
    __syncwarp();
  }
};

// act(z) * mul + residual in place on the warp's accumulators of 32 rows y0 .. and 128
// columns n0 ..: each(lo, hi, f) calls f(z, row, column) on the pairs of neighbouring
// columns that the thread holds in lo .. hi - 1, as straight code on registers.  (A
// rolled loop that reads the accumulators back from Tensor Memory or shared memory
// took longer for every activation and operand: a warp shares its scheduler with one
// other, so passes are bound by latency.)  A box is requested before the arithmetic on
// the one before it, the first before the activation.
template <int HOLD, class Each>
__device__ __forceinline__ void epi_apply_rows(const EpiArgs& e, uint8_t* stg, int y0, int n0, int M, int N, Each&& each) {
  const EpiOperand mul{e.mul, e.mul_ld, e.mul_rows, e.mul_f32 != 0}, res{e.res, e.res_ld, 1, e.res_f32 != 0};
  EpiBox<HOLD> box;
  if (mul.p) box.fetch(mul, y0, n0, M, N);
  else if (res.p) box.fetch(res, y0, n0, M, N);
  else box.none();
  epi_act_each(e.act, [&](auto&& f) { each(0, 128, [&](float2& z, int, int) { f(z); }); });
  auto boxes = [&](const EpiOperand& o, const EpiOperand& after, auto&& f) {
    if (!o.f32) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        box.land(o, stg, y0, n0 + 64 * k, M, N);
        if (k == 0) box.fetch(o, y0, n0 + 64, M, N);
        else if (after.p) box.fetch(after, y0, n0, M, N);
        else box.none();
        each(64 * k, 64 * k + 64, [&](float2& z, int r, int c) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(stg + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) +
                                                               (c & 7) * 2);
          f(z, make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
        });
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        box.land(o, stg, y0, n0 + 32 * k, M, N);
        if (k < 3) box.fetch(o, y0, n0 + 32 * (k + 1), M, N);
        else if (after.p) box.fetch(after, y0, n0, M, N);
        else box.none();
        each(32 * k, 32 * k + 32, [&](float2& z, int r, int c) {
          f(z, *reinterpret_cast<const float2*>(stg + r * 128 + ((((c >> 2) & 7) ^ (r & 7)) << 4) + (c & 3) * 4));
        });
      }
    }
  };
  const EpiOperand nothing{nullptr, 0, 1, false};
  if (mul.p) boxes(mul, res, [](float2& a, const float2& m) { a = __fmul2_rn(a, m); });
  if (res.p) boxes(res, nothing, [](float2& a, const float2& r) { a = __fadd2_rn(a, r); });
  __syncwarp();  // the buffer has been read
}

// f(z, operand) on R x B pairs of accumulators z(i, b), whose operands lie at(i, b)
// elements into p: `ahead` pairs are requested at a time, then used.
template <int R, int B, int AHEAD, class Z, class At, class F>
__device__ __forceinline__ void epi_quads_operand(const void* p, bool f32, Z&& z, At&& at, F&& f) {
  static_assert((R * B) % AHEAD == 0, "whole batches");
  if (!f32) {
#pragma unroll
    for (int j0 = 0; j0 < R * B; j0 += AHEAD) {
      uint32_t w[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        w[j] = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p) + at((j0 + j) % R, (j0 + j) / R));
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        f(z((j0 + j) % R, (j0 + j) / R),
          make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)));
    }
  } else {
#pragma unroll
    for (int j0 = 0; j0 < R * B; j0 += AHEAD / 2) {
      float2 w[AHEAD / 2];
#pragma unroll
      for (int j = 0; j < AHEAD / 2; ++j)
        w[j] = *reinterpret_cast<const float2*>(static_cast<const float*>(p) + at((j0 + j) % R, (j0 + j) / R));
#pragma unroll
      for (int j = 0; j < AHEAD / 2; ++j) f(z((j0 + j) % R, (j0 + j) / R), w[j]);
    }
  }
}

// act(z) * mul + residual in place on the thread's R x B pairs of accumulators z(i, b):
// R rows, B pairs of neighbouring columns in each.  Straight code on registers: a
// rolled loop that reads the accumulators back from Tensor Memory or shared memory
// took longer for every activation and operand (a warp shares its scheduler with one
// other, so its passes are bound by latency).  No conditional load: one that may
// leave its register undefined keeps it live from the loop over tiles on, and the
// accumulators spill.
template <int R, int B, int AHEAD, class Z, class MulAt, class ResAt>
__device__ __forceinline__ void epi_apply_quads(const EpiArgs& e, Z&& z, MulAt&& mul_at, ResAt&& res_at) {
  epi_act_each(e.act, [&](auto&& f) {
#pragma unroll
    for (int j = 0; j < R * B; ++j) f(z(j % R, j / R));
  });
  if (e.mul)
    epi_quads_operand<R, B, AHEAD>(e.mul, e.mul_f32 != 0, z, mul_at, [](float2& a, const float2& m) { a = __fmul2_rn(a, m); });
  if (e.res)
    epi_quads_operand<R, B, AHEAD>(e.res, e.res_f32 != 0, z, res_at, [](float2& a, const float2& r) { a = __fadd2_rn(a, r); });
}

// The same on accumulators of R output features feature(i) by 2 B tokens token(t),
// the pair z(i, b) holding tokens 2b and 2b + 1 of the thread: operands by elements, a
// batch requested at a time.
template <int R, int B, class T, class Z, class Feature, class Token, class F>
__device__ __forceinline__ void epi_columns_operand(const T* p, long long ld, int rows, Z&& z, Feature&& feature,
                                                    Token&& token, F&& f) {
  constexpr int BB = R * B > 16 ? 16 / R : B;  // pairs of columns to a batch
  static_assert(B % BB == 0, "whole batches");
#pragma unroll
  for (int b0 = 0; b0 < B; b0 += BB) {
    T w[2 * R * BB];
#pragma unroll
    for (int t = 0; t < 2 * BB; ++t) {
      int row = token(2 * b0 + t);
      if (rows != 1) row /= rows;
#pragma unroll
      for (int i = 0; i < R; ++i) w[t * R + i] = p[static_cast<size_t>(row) * ld + feature(i)];
    }
#pragma unroll
    for (int b = 0; b < BB; ++b)
#pragma unroll
      for (int i = 0; i < R; ++i)
        f(z(i, b0 + b), make_float2(static_cast<float>(w[2 * b * R + i]), static_cast<float>(w[(2 * b + 1) * R + i])));
  }
}
template <int R, int B, class Z, class Feature, class Token>
__device__ __forceinline__ void epi_apply_columns(const EpiArgs& e, Z&& z, Feature&& feature, Token&& token) {
  epi_act_each(e.act, [&](auto&& f) {
#pragma unroll
    for (int j = 0; j < R * B; ++j) f(z(j % R, j / R));
  });
  auto operand = [&](const void* p, int f32, long long ld, int rows, auto&& f) {
    if (f32) epi_columns_operand<R, B>(static_cast<const float*>(p), ld, rows, z, feature, token, f);
    else epi_columns_operand<R, B>(static_cast<const __nv_bfloat16*>(p), ld, rows, z, feature, token, f);
  };
  if (e.mul) operand(e.mul, e.mul_f32, e.mul_ld, e.mul_rows, [](float2& a, const float2& m) { a = __fmul2_rn(a, m); });
  if (e.res) operand(e.res, e.res_f32, e.res_ld, 1, [](float2& a, const float2& r) { a = __fadd2_rn(a, r); });
}

}  // namespace hsq
