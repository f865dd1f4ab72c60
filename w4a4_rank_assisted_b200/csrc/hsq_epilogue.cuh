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
// with u = sqrt(2/pi) (z + 0.044715 z^3): one exponential and one quotient each.  The
// relative error grows with the exponent's argument t (-z or -2u), whose fp32 rounding
// the exponential passes on: at most (9 + 6.4 |t|) 2^-24 where t > 0, a few 2^-23
// elsewhere (silu: 16 x 2^-23 at z = -40, 32 x 2^-23 at -80).  The erf gelu is
//     max(z, 0) - |z|/2 erfc(|z| / sqrt 2),   erfc(w) = e^(-w^2) t Q(t), t = 1 / (1 + 0.45 w),
// Q of degree 9 fitted to erfc(w) e^(w^2) / t over all w >= 0 for the least largest
// relative error (with its coefficients in fp32: 4.7e-8 up to w = 9, where e^(-w^2)
// leaves fp32's range, 6.4e-8 beyond); e^(-w^2) adds 2 (w^2 + 1) 2^-23 or so.  The
// complement keeps its relative accuracy for negative z, where 1 + erf cancels, at
// two special-function instructions like the others.
#pragma once

#include <type_traits>

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

// A kernel's arguments: those of its plain form, and an epilogue's behind them in the
// instantiations that apply one.  (With one structure for both, the plain NVFP4 GEMM
// was compiled differently and took 1.1 % longer at each of FLUX.1's layers.)
template <class Args>
struct WithEpilogue : Args {
  EpiArgs epi;
};
template <class Args, bool EPI>
using KernelArgs = std::conditional_t<EPI, WithEpilogue<Args>, Args>;

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

// One operand's box under the warp's part of Y: 32 rows of 64 bytes (32 bf16 or 16
// fp32 columns), copied asynchronously into 2 KB of the warp's staging buffer: 16-byte
// chunk c of row r at chunk c ^ (r / 2 % 4) of its 64 bytes, so that eight rows' chunk
// c fall into 32 different banks.  Rows behind M read row M - 1 and columns behind N
// the row's first ones: nothing outside the operand is read, and those outputs are
// clipped by the TMA unit.
struct EpiOperand {
  const void* p;
  long long ld;
  int rows;  // tokens to a row
  bool f32;
};
__device__ __forceinline__ void epi_fetch(const EpiOperand& o, uint8_t* box, int y0, int n0, int M, int N) {
  const int lane = lane_id(), c = lane & 3;
  int n = n0 + c * (o.f32 ? 4 : 8);
  if (n >= N) n = 0;
  const char* base = static_cast<const char*>(o.p) + static_cast<size_t>(n) * (o.f32 ? 4 : 2);
  const size_t pitch = static_cast<size_t>(o.ld) * (o.f32 ? 4 : 2);
  auto rows = [&](auto&& row) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       smem_u32(box + r * 64 + ((c ^ ((r >> 1) & 3)) << 4))),
                   "l"(base + static_cast<size_t>(row(min(y0 + r, M - 1))) * pitch)
                   : "memory");
    }
  };
  if (o.rows == 1) rows([](int m) { return m; });
  else rows([&](int m) { return m / o.rows; });
}
// Four 8 x 8 blocks of 16-bit elements, a row's address from each lane: lane l gets
// elements 2 (l % 4), + 1 of row l / 4 of each.
__device__ __forceinline__ void ldmatrix_x4(uint32_t saddr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ float2 epi_pair16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// How the threads hold the warp's accumulators of 32 rows, and read a box for them: use16 / use32 apply f(z, operand) to the pairs of neighbouring
// columns in a box of 32 bf16 / 16 fp32 columns, the k-th of the warp's.
//   Quads: tcgen05.ld 16x256b: lane l has rows l / 4 + 8i and columns 8b + 2 (l % 4), + 1
template <int NBLK>
struct EpiQuads {
  float2 (&acc)[4 * NBLK];
  template <class F>
  __device__ __forceinline__ void all(F&& f) {
#pragma unroll
    for (int j = 0; j < 4 * NBLK; ++j) f(acc[j]);
  }
  template <class F>
  __device__ __forceinline__ void use16(const uint8_t* box, int k, F&& f) {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // block b of row group i: its rows' addresses from lanes 8b .. 8b + 7
      const int r = 8 * i + (lane & 7);
      uint32_t w[4];
      ldmatrix_x4(smem_u32(box + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4)), w);
#pragma unroll
      for (int b = 0; b < 4; ++b) f(acc[i * NBLK + 4 * k + b], epi_pair16(w[b]));
    }
  }
  template <class F>
  __device__ __forceinline__ void use32(const uint8_t* box, int k, F&& f) {
    const int lane = lane_id(), qc = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
#pragma unroll
      for (int b = 0; b < 2; ++b)
        f(acc[i * NBLK + 2 * k + b],
          *reinterpret_cast<const float2*>(box + r * 64 + (((2 * b + (qc >> 1)) ^ ((r >> 1) & 3)) << 4) + (qc & 1) * 8));
    }
  }
};
//   Rows: tcgen05.ld 32x32b: lane l has row l, v[c] its columns 16 c ..
struct EpiRows {
  uint32_t (&v)[8][16];
  __device__ __forceinline__ float2& pair(int j) { return reinterpret_cast<float2*>(v[j >> 3])[j & 7]; }
  template <class F>
  __device__ __forceinline__ void all(F&& f) {
#pragma unroll
    for (int j = 0; j < 64; ++j) f(pair(j));
  }
  template <class F>
  __device__ __forceinline__ void use16(const uint8_t* box, int k, F&& f) {
    const int lane = lane_id();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 q = *reinterpret_cast<const uint4*>(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) f(pair(16 * k + 4 * c + e), epi_pair16(w[e]));
    }
  }
  template <class F>
  __device__ __forceinline__ void use32(const uint8_t* box, int k, F&& f) {
    const int lane = lane_id();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 q = *reinterpret_cast<const float4*>(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
      f(pair(8 * k + 2 * c), make_float2(q.x, q.y));
      f(pair(8 * k + 2 * c + 1), make_float2(q.z, q.w));
    }
  }
};

// act(z) * mul + residual in place on the warp's accumulators of 32 rows y0 .. and CW
// columns n0 .. (n0 < N).  stg: the warp's 4 KB staging buffer, through which the
// operands come in two boxes of 2 KB in turn, each requested while the one before it is
// used, the first two ahead of the activation.
//
// The accumulators stay where they are, in straight code.  A warp shares its
// scheduler with one other here, so a pass over them is bound by latency: rolled loops
// that read them back from Tensor Memory or shared memory took longer for every
// activation and operand.  No operand waits in registers: those loaded under a
// condition stay live from the loop over tiles on, and the accumulators spill.
// (The NVFP4 kernel, whose registers are not split between its warps, does spill: 716
// bytes of stores and 1744 of loads in its instantiation with an epilogue.)
// Bound by the activation's special-function instructions (two an element: 2 us per
// 128 x 256 tile) and by instruction latency.  Measured with the activation step, us
// (none / silu / mul / silu * mul / silu * mul + residual): 606 / 656 / 675 / 704 / 769 at
// M = 8192, K = 4096, N = 12288, groups of 128 (2 % either way with the clock); 82 / 93 /
// 95 / 104 / 115 at M = 4096, K = 1152, N = 4608, groups of 64; NVFP4 at M = 4096, K =
// 4608, N = 1152: 95.1 / 98.5 / 99.9 / 100.8 / 104.7.  An elementwise pass over Y and mul
// (600 MB) takes 86 us at the first size, 17 at the second, 4 at the third: on these
// tiles the epilogue saves a rounding and a launch, and hardly any time.
template <int CW, class Acc>
__device__ __forceinline__ void epi_apply(const EpiArgs& e, uint8_t* stg, int y0, int n0, int M, int N, Acc&& acc) {
  const EpiOperand mul{e.mul, e.mul_ld, e.mul_rows, e.mul_f32 != 0}, res{e.res, e.res_ld, 1, e.res_f32 != 0};
  static_assert(CW % 64 == 0, "an even number of boxes, so that an operand starts at buffer 0");
  // box k of an operand into buffer k % 2; one group each, empty where there is no operand
  auto request = [&](const EpiOperand& o, int k) {
    if (o.p) epi_fetch(o, stg + (k & 1) * 2048, y0, n0 + (o.f32 ? 16 : 32) * k, M, N);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (mul.p || res.p) {
    if (lane_id() == 0) bulk_wait_read_all();  // the last tile's stores have left the buffer
    __syncwarp();
    if (mul.p) {
      request(mul, 0);
      request(mul, 1);
    } else {
      request(res, 0);
      request(res, 1);
    }
  }
  epi_act_each(e.act, [&](auto&& f) { acc.all(f); });
  auto boxes = [&](const EpiOperand& o, const EpiOperand& after, auto&& f) {
    auto step = [&](int k, int n, auto&& use) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();  // the box is whole
      use(stg + (k & 1) * 2048);
      __syncwarp();  // ... and has been read
      if (k + 2 < n) request(o, k + 2);
      else request(after, k + 2 - n);
    };
    if (!o.f32) {
#pragma unroll
      for (int k = 0; k < CW / 32; ++k) step(k, CW / 32, [&](const uint8_t* box) { acc.use16(box, k, f); });
    } else {
#pragma unroll
      for (int k = 0; k < CW / 16; ++k) step(k, CW / 16, [&](const uint8_t* box) { acc.use32(box, k, f); });
    }
  };
  const EpiOperand nothing{nullptr, 0, 1, false};
  if (mul.p) boxes(mul, res, [](float2& z, const float2& m) { z = __fmul2_rn(z, m); });
  if (res.p) boxes(res, nothing, [](float2& z, const float2& r) { z = __fadd2_rn(z, r); });
}

// act(z) * mul + residual in place on accumulators of R output features feature(i) by
// 2 B tokens token(t) (the decode tiles), the pair z(i, b) holding tokens 2b and 2b + 1
// of the thread: operands by elements, a batch of up to 32 requested at a time (one
// feature at a time, with the activation chosen inside, 30.2 instead of 26.2 us at M =
// 16, K = 12288, N = 4096; 25.6 without an epilogue).
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
