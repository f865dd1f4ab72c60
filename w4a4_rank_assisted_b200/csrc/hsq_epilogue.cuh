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
// to a few 2^-23 relative.  The erf gelu is 0.5 z erfc(-z / sqrt 2): the
// complement keeps its relative accuracy for negative z, where 1 + erf cancels.
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

__device__ __forceinline__ float epi_sigmoid_form(float z, float t) {  // z / (1 + e^t)
  return __fdividef(z, 1.f + __expf(t));
}

__device__ __forceinline__ float epi_act(float z, int act) {
  switch (act) {  // uniform over the launch
    case kActRelu: return z < 0.f ? 0.f : z;
    case kActGeluTanh: return epi_sigmoid_form(z, -1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.f));
    case kActGeluErf: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case kActSilu: return epi_sigmoid_form(z, -z);
    default: return z;
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

// act(z) * mul + residual of one element.
__device__ __forceinline__ float epi_value(const EpiArgs& e, float z, float mul, float res) {
  float v = epi_act(z, e.act);
  if (e.mul) v *= mul;
  if (e.res) v += res;
  return v;
}

// Eight consecutive elements of a row, as loaded (bf16: lo alone).
struct EpiOct {
  uint4 lo, hi;
};
__device__ __forceinline__ void epi_load8(const void* p, int f32, size_t at, EpiOct& o) {
  if (f32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    o.lo = q[0];
    o.hi = q[1];
  } else {
    o.lo = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
  }
}
__device__ __forceinline__ void epi_float8(const EpiOct& o, int f32, float (&f)[8]) {
  if (f32) {
    const uint32_t w[8] = {o.lo.x, o.lo.y, o.lo.z, o.lo.w, o.hi.x, o.hi.y, o.hi.z, o.hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  } else {
    bf16x8_to_f32(o.lo, f);
  }
}

// The operands of one 32 x 32 box of Y for the lane layout of epi_store_box.
struct EpiBox {
  EpiOct mul[4], res[4];
};
__device__ __forceinline__ void epi_load_box(const EpiArgs& e, int m0, int n0, int M, int N, EpiBox& b) {
  const int lane = lane_id(), n = n0 + 8 * (lane & 3);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int m = m0 + 8 * p + (lane >> 2);
    if (m < M && n < N) {  // N % 8 == 0: eight columns are all in or all out
      if (e.mul) {
        const int row = e.mul_rows == 1 ? m : m / e.mul_rows;
        epi_load8(e.mul, e.mul_f32, static_cast<size_t>(row) * e.mul_ld + n, b.mul[p]);
      }
      if (e.res) epi_load8(e.res, e.res_f32, static_cast<size_t>(m) * e.res_ld + n, b.res[p]);
    }
  }
}

// Writes one 32 x 32 box of Y from the warp's staged fp32 accumulators: stg holds
// 32 rows of 128 bytes, 16-byte chunk c of row r at chunk c ^ (r % 8).  A lane
// takes eight consecutive columns of rows lane / 4 + 8p, so every global access is
// 16 bytes (32 for fp32) and four lanes cover a row's 64 (128) bytes; the lanes'
// shared reads of one chunk fall into eight distinct 16-byte banks.
__device__ __forceinline__ void epi_store_box(const EpiArgs& e, const uint8_t* stg, const EpiBox& b, int m0, int n0,
                                              int M, int N, void* Y, int out_f32) {
  const int lane = lane_id(), n = n0 + 8 * (lane & 3);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int rl = 8 * p + (lane >> 2), m = m0 + rl;
    if (m >= M || n >= N) continue;
    float z[8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float4*>(z + 4 * h) =
          *reinterpret_cast<const float4*>(stg + rl * 128 + (((2 * (lane & 3) + h) ^ (rl & 7)) << 4));
    switch (e.act) {
      case kActRelu:
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = epi_act(z[i], kActRelu);
        break;
      case kActGeluTanh:
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = epi_act(z[i], kActGeluTanh);
        break;
      case kActGeluErf:
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = epi_act(z[i], kActGeluErf);
        break;
      case kActSilu:
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = epi_act(z[i], kActSilu);
        break;
      default: break;
    }
    if (e.mul) {
      float f[8];
      epi_float8(b.mul[p], e.mul_f32, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] *= f[i];
    }
    if (e.res) {
      float f[8];
      epi_float8(b.res[p], e.res_f32, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] += f[i];
    }
    const size_t off = static_cast<size_t>(m) * N + n;
    if (out_f32) {
      float4* y = reinterpret_cast<float4*>(static_cast<float*>(Y) + off);
      y[0] = make_float4(z[0], z[1], z[2], z[3]);
      y[1] = make_float4(z[4], z[5], z[6], z[7]);
    } else {
      uint4 w;
      __nv_bfloat162* wb = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
      for (int i = 0; i < 4; ++i) wb[i] = __floats2bfloat162_rn(z[2 * i], z[2 * i + 1]);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(Y) + off) = w;
    }
  }
}

}  // namespace hsq
