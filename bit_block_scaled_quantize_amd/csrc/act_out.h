// The output of nvfp4_gemm_act, shared by its kernels: z = product + bias (FP32); the pre-activation
// BF16(z) where asked for; d = BF16(act(z) + residual). act takes the unrounded z.
#pragma once

#include "activation.h"
#include "launch.h"

namespace nvfp4 {

__device__ __forceinline__ float bias_at(const ActOut& o, int64_t col) {
  if (o.bias == nullptr) return 0.0f;
  return o.bias_f32 ? static_cast<const float*>(o.bias)[col] : bf16_lo(static_cast<const uint16_t*>(o.bias)[col]);
}

// Element (row, col); returns |stored d|.
template <int ACT>
__device__ __forceinline__ float put_act(const ActOut& o, uint16_t* d, int64_t ldd, int64_t row, int64_t col, float v) {
  const float z = v + bias_at(o, col);
  if (o.preact != nullptr) o.preact[row * o.ldp + col] = (uint16_t)bf16_rn_bits(z);
  float y = act<ACT>(z);
  if (o.residual != nullptr) y += bf16_lo(o.residual[row * o.ldr + col]);
  const uint32_t b = bf16_rn_bits(y);
  d[row * ldd + col] = (uint16_t)b;
  return fabsf(__uint_as_float(b << 16));
}

// The same with the kind known at run time (uniform).
__device__ __forceinline__ float put_act_of(int act, const ActOut& o, uint16_t* d, int64_t ldd, int64_t row,
                                            int64_t col, float v) {
  switch (act) {
    case kActRelu2: return put_act<kActRelu2>(o, d, ldd, row, col, v);
    case kActGelu: return put_act<kActGelu>(o, d, ldd, row, col, v);
    case kActSilu: return put_act<kActSilu>(o, d, ldd, row, col, v);
    default: return put_act<kActNone>(o, d, ldd, row, col, v);
  }
}

// Four consecutive elements of a row with their bias and residual (two BF16 a word) at hand.
template <int ACT, class V>
__device__ __forceinline__ float put_act4(const ActOut& o, uint16_t* d, int64_t ldd, int64_t row, int64_t col,
                                          const V& v, const float (&bias)[4], v2u32 res) {
  float z[4], y[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    z[q] = v[q] + bias[q];
    y[q] = act<ACT>(z[q]);
    if (o.residual != nullptr) y[q] += (q & 1) ? bf16_hi(res[q >> 1]) : bf16_lo(res[q >> 1]);
  }
  if (o.preact != nullptr)
    *reinterpret_cast<v2u32_any*>(o.preact + row * o.ldp + col) = v2u32{bf16_rn_pair(z[0], z[1]), bf16_rn_pair(z[2], z[3])};
  const v2u32 w = {bf16_rn_pair(y[0], y[1]), bf16_rn_pair(y[2], y[3])};
  *reinterpret_cast<v2u32_any*>(d + row * ldd + col) = w;
  return fmaxf(fmaxf(fabsf(bf16_lo(w.x)), fabsf(bf16_hi(w.x))), fmaxf(fabsf(bf16_lo(w.y)), fabsf(bf16_hi(w.y))));
}

template <class V>
__device__ __forceinline__ float put_act4_of(int act, const ActOut& o, uint16_t* d, int64_t ldd, int64_t row, int64_t col,
                                             const V& v, const float (&bias)[4], v2u32 res) {
  switch (act) {
    case kActRelu2: return put_act4<kActRelu2>(o, d, ldd, row, col, v, bias, res);
    case kActGelu: return put_act4<kActGelu>(o, d, ldd, row, col, v, bias, res);
    case kActSilu: return put_act4<kActSilu>(o, d, ldd, row, col, v, bias, res);
    default: return put_act4<kActNone>(o, d, ldd, row, col, v, bias, res);
  }
}

// Eight consecutive elements of a row with their bias and residual at hand, every array moved as one 16-byte
// vector from wherever it starts. Non-temporal: the outputs go out to HBM and leave the caches to the operands.
template <int ACT>
__device__ __forceinline__ float put_act8(const ActOut& o, uint16_t* d, int64_t ldd, int64_t row, int64_t col,
                                          const float (&v)[8], const float (&bias)[8], v4u32 res) {
  float z[8], y[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    z[q] = v[q] + bias[q];
    y[q] = act<ACT>(z[q]);
  }
  if (o.preact != nullptr)
    __builtin_nontemporal_store(
        v4u32{bf16_rn_pair(z[0], z[1]), bf16_rn_pair(z[2], z[3]), bf16_rn_pair(z[4], z[5]), bf16_rn_pair(z[6], z[7])},
        reinterpret_cast<v4u32_any*>(o.preact + row * o.ldp + col));
  v4u32 w;
  float mx = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (o.residual != nullptr) {
      y[2 * q] += bf16_lo(res[q]);
      y[2 * q + 1] += bf16_hi(res[q]);
    }
    w[q] = bf16_rn_pair(y[2 * q], y[2 * q + 1]);
    mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[q])), fabsf(bf16_hi(w[q]))));
  }
  __builtin_nontemporal_store(w, reinterpret_cast<v4u32_any*>(d + row * ldd + col));
  return mx;
}

}  // namespace nvfp4
