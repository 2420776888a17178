// NVFP4 weight rows times a few token columns: the product inside the GEMM for few rows and the
// expert layer for few tokens. Such a product is bound by reading the weights once (4.5 bits per
// element); the matrix cores have two orders of work to spare, so a 16-column instruction is fed
// with however few tokens there are, and decoding is shared by nothing but the lanes.
//
// v_mfma_f32_16x16x32_f16 with the weights as A (rows) and the tokens as B (columns): lane l holds
// row / column l % 16 and 8 K-values picked by g = l / 16. Over a K step of 128 a lane owns the 32
// consecutive elements [128 s + 32 g, + 32) of its row (16 bytes of codes, two scale bytes) and feeds
// their four octets to four instructions; K order is free as long as rows and columns agree. The
// result holds column l % 16, rows 4 g .. 4 g + 3. Codes decode to FP16 exactly (e2m1 * e4m3 has at
// most 6 significant bits in [2^-10, 2688]), products are exact, sums FP32.
//
// A workgroup takes 16 R rows; its waves share them and split K, every wave the next step in
// turn (together they read whole 256-byte runs of each row), and add up through LDS in a fixed
// order. Everything goes straight from memory to registers, the next step's loads ahead of this
// step's arithmetic: no element is used twice in a workgroup.
#pragma once

#include "device_common.h"

namespace nvfp4 {
namespace skinny {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;

// FP16 pair (S * 2^-8 twice) of an E4M3 scale code, and 8 codes as e2m1 * S (the conversion's own
// scale operand returns the 2^8).
__device__ __forceinline__ half2v scale_pair(uint32_t s) { return __builtin_bit_cast(half2v, s * 0x00800080u); }

__device__ __forceinline__ half8 decode8(uint32_t codes, half2v s2) {
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, 0) * s2;
  const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, 1) * s2;
  const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, 2) * s2;
  const half2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, 3) * s2;
  return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The 32 codes of one row at element k (a multiple of 32) and their two scale bytes, with zero
// scales at and past K, which zero whatever the codes are. k past K reads the row's start instead.
struct Run { v4u32 codes; uint32_t scales; };

// K32: K is a multiple of 32 (rows of codes start on 16 bytes, of scales on 2).
template <bool K32>
__device__ __forceinline__ Run load_run(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                        int64_t K, int64_t k) {
  Run r;
  if constexpr (K32) {
    const int64_t at = k < K ? k : 0;
    r.codes = ld_u32x4(codes + (at >> 1));
    const uint32_t s = *reinterpret_cast<const uint16_t*>(scales + (at >> 4));
    r.scales = k < K ? s : 0u;
  } else {
    const int64_t a = k < K ? k : 0, b = k + 16 < K ? k + 16 : 0;
    const v2u32 lo = *reinterpret_cast<const v2u32*>(codes + (a >> 1));
    const v2u32 hi = *reinterpret_cast<const v2u32*>(codes + (b >> 1));
    r.codes = v4u32{lo.x, lo.y, hi.x, hi.y};
    const uint32_t s0 = scales[a >> 4], s1 = scales[b >> 4];
    r.scales = (k < K ? s0 : 0u) | (k + 16 < K ? s1 << 8 : 0u);
  }
  return r;
}

__device__ __forceinline__ half8 octet(const Run& r, int t) {
  return decode8(r.codes[t], scale_pair((r.scales >> (8 * (t >> 1))) & 0xFFu));
}

// acc[i][c] += rows 16 i .. + 15 of the tile times token columns 16 c .. + 15, over the steps
// first, first + stride, ... below K. row_codes / row_scales: this lane's row of each fragment.
// Tok: load(c, k) -> Raw (the lane's 32 elements of column 16 c + l % 16 at element k, 0 past K or
// without a token), octet(c, raw, t) -> half8.
template <int R, int C, bool K32, class Tok>
__device__ __forceinline__ void accumulate(const uint8_t* const (&row_codes)[R], const uint8_t* const (&row_scales)[R],
                                           int64_t K, int first, int stride, const Tok& tok, float4v (&acc)[R][C]) {
  const int g = (threadIdx.x & 63) >> 4;
  const int steps = (int)((K + kStep - 1) / kStep);
  Run w[R];
  typename Tok::Raw x[C];
  int64_t k = (int64_t)first * kStep + g * 32;
#pragma unroll
  for (int i = 0; i < R; ++i) w[i] = load_run<K32>(row_codes[i], row_scales[i], K, k);
#pragma unroll
  for (int c = 0; c < C; ++c) x[c] = tok.load(c, k);
#pragma unroll 1
  for (int s = first; s < steps; s += stride) {
    k += (int64_t)stride * kStep;                             // past K: the loads below give zeros
    Run wn[R];
    typename Tok::Raw xn[C];
#pragma unroll
    for (int i = 0; i < R; ++i) wn[i] = load_run<K32>(row_codes[i], row_scales[i], K, k);
#pragma unroll
    for (int c = 0; c < C; ++c) xn[c] = tok.load(c, k);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      half8 b[C];
#pragma unroll
      for (int c = 0; c < C; ++c) b[c] = tok.octet(c, x[c], t);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const half8 a = octet(w[i], t);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[i][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[c], acc[i][c], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) w[i] = wn[i];
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = xn[c];
  }
}

// Each wave's sums into LDS (W waves x R C fragments of 64 x 4 floats), then fragment f summed over
// the waves in order. All threads call put, then a barrier, then take.
template <int R, int C>
__device__ __forceinline__ void put(float* red, int wave, const float4v (&acc)[R][C]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int c = 0; c < C; ++c)
      *reinterpret_cast<float4v*>(red + (((wave * R + i) * C + c) * 64 + lane) * 4) = acc[i][c];
}

template <int W, int R, int C>
__device__ __forceinline__ float4v take(const float* red, int i, int c) {
  const int lane = threadIdx.x & 63;
  float4v s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < W; ++w) s += *reinterpret_cast<const float4v*>(red + (((w * R + i) * C + c) * 64 + lane) * 4);
  return s;
}

}  // namespace skinny
}  // namespace nvfp4
