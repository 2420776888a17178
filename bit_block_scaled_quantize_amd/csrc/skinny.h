// NVFP4 weight rows times a few token columns: the product inside the GEMM for few rows and the
// expert layer for few tokens. Such a product is bound by reading the weights once (4.5 bits per
// element); the matrix cores have two orders of work to spare, so a 16-column instruction is fed
// with however few tokens there are, and decoding is shared by nothing but the lanes.
//
// v_mfma_f32_16x16x32_f16 with the weights as A (rows) and the tokens as B (columns): lane l holds
// row / column l % 16 and 8 K-values picked by g = l / 16. Over a K step a lane owns one run of
// consecutive elements of its row and feeds its octets to as many instructions; K order is free as long
// as rows and columns agree. With runs of 64, steps of 256, the four lanes of a row read whole 128-byte
// lines between them (two loads apart) and 16 scale bytes. The result holds column l % 16, rows
// 4 g .. 4 g + 3. Codes decode to FP16 exactly (e2m1 * e4m3 has at most 6 significant bits in
// [2^-10, 2688]), products are exact, sums FP32.
//
// A workgroup takes 16 R rows; its W waves share them and split K, every wave the next step in
// turn (together they read whole runs of each row), and add up through LDS in a fixed order.
// Everything goes straight from memory to registers, a few steps of the weights in flight per
// wave: no element is used twice in a workgroup, and what such a product waits for is HBM's
// latency (about 2 us under load, so 5 TB/s want 40 KB in flight on every CU).
#pragma once

#include "device_common.h"

namespace nvfp4 {
namespace skinny {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// How a lane reads its runs. kAligned: 64 elements, K a multiple of 64. The others take any K (a multiple
// of 16): rows start on 8 bytes and scales on any. kHalf: 32 elements, the scales byte by byte. kWord: 64
// elements, K at least 64: half runs that are whole are loaded as such, the 16 elements of a K that ends inside
// one apart, the scales as one unaligned word, moved back where it would leave the matrix.
// Measured, us (kHalf / kWord), few-row GEMM: 1003 x 1857 x 2704 31 / 25, 256 x 5120 x 5136 56 / 38, 1 x 5120 x
// 5136 10.4 / 9.3, 1 x 5120 x 32 3.9 / 4.8. Expert layer, where a wave has only a few steps and the last is mostly
// empty: 64 tokens, 528 x 2064 72 / 81, 2000 x 1360 80 / 82; 7 tokens, 1040 x 720 29 / 31.
enum Shape { kAligned, kWord, kHalf };
template <Shape S> constexpr int kRun = S == kHalf ? 32 : 64;
template <Shape S> constexpr int kOctets = kRun<S> / 8;
template <Shape S> constexpr int kStep = 4 * kRun<S>;

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

// Loads go through a buffer resource over a matrix (below 2 GiB) with one 32-bit offset a lane: a lane
// without an element gives an offset past any buffer and gets zeros, so there are no branches
// around the loads and nothing to clear afterwards.
constexpr uint32_t kBeyond = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
  // base and size made scalar: they are uniform, which the compiler cannot always see
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo), (short)0,
                                           (int)__builtin_amdgcn_readfirstlane((uint32_t)bytes), 0x00020000);
}

__device__ __forceinline__ v4u32 load16(__amdgpu_buffer_rsrc_t b, uint32_t at) {
  return __builtin_bit_cast(v4u32, __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0));
}

// An NVFP4 matrix [rows, K].
struct Matrix {
  __amdgpu_buffer_rsrc_t codes, scales;
  const uint8_t* scale_bytes;
  uint32_t K, last_scale;                                     // last_scale: offset of the last four scale bytes (kWord)
  __device__ __forceinline__ Matrix(const uint8_t* c, const uint8_t* s, int64_t rows, int64_t k)
      : codes(buffer(c, rows * (k >> 1))), scales(buffer(s, rows * (k >> 4))), scale_bytes(s), K((uint32_t)k),
        last_scale((uint32_t)(rows * (k >> 4)) - 4u) {}
};

// The codes of one row's run at element k (a multiple of the run) and its scale bytes, zeros at and
// past K and without a row; and the same as it is loaded, since arithmetic on a value, even a
// widening, would wait for it where it is loaded.
template <Shape S>
struct Run {
  v4u32 lo, hi;
  uint32_t scales;
};
template <>
struct Run<kHalf> {
  v2u32 lo, hi;
  uint8_t s0, s1;
};
template <Shape S>
struct Loaded {
  Run<S> run;
};
template <>
struct Loaded<kWord> {
  Run<kWord> run;
  v2u32 tail;
};

template <Shape S>
__device__ __forceinline__ Loaded<S> load_run(const Matrix& m, uint32_t row, bool live, uint32_t k) {
  Loaded<S> r;
  const uint32_t c = row * (m.K >> 1) + (k >> 1), s = row * (m.K >> 4) + (k >> 4);
  const bool a = live && k < m.K;
  if constexpr (S == kAligned) {
    const uint32_t at = a ? c : kBeyond;
    r.run.lo = load16(m.codes, at);
    r.run.hi = load16(m.codes, at + 16);
    r.run.scales = __builtin_amdgcn_raw_buffer_load_b32(m.scales, a ? s : kBeyond, 0, 0);
  } else if constexpr (S == kHalf) {
    const bool b = live && k + 16 < m.K;
    r.run.lo = __builtin_bit_cast(v2u32, __builtin_amdgcn_raw_buffer_load_b64(m.codes, a ? c : kBeyond, 0, 0));
    r.run.hi = __builtin_bit_cast(v2u32, __builtin_amdgcn_raw_buffer_load_b64(m.codes, b ? c + 8 : kBeyond, 0, 0));
    r.run.s0 = __builtin_amdgcn_raw_buffer_load_b8(m.scales, a ? s : kBeyond, 0, 0);
    r.run.s1 = __builtin_amdgcn_raw_buffer_load_b8(m.scales, b ? s + 1 : kBeyond, 0, 0);
  } else {
    r.run.lo = load16(m.codes, live && k + 32 <= m.K ? c : kBeyond);
    r.run.hi = load16(m.codes, live && k + 64 <= m.K ? c + 16 : kBeyond);
    const uint32_t t = m.K - 16;
    r.tail = __builtin_bit_cast(v2u32, __builtin_amdgcn_raw_buffer_load_b64(
        m.codes, a && t - k < 64u && (t & 16u) == 0 ? c + ((t - k) >> 1) : kBeyond, 0, 0));
    const uint32_t at = a ? s : 0u;
    r.run.scales = *reinterpret_cast<const u32_any*>(m.scale_bytes + (at < m.last_scale ? at : m.last_scale));
  }
  return r;
}

template <Shape S>
__device__ __forceinline__ const Run<S>& run_of(const Loaded<S>& r, const Matrix&, uint32_t, bool, uint32_t) {
  return r.run;
}

__device__ __forceinline__ Run<kWord> run_of(const Loaded<kWord>& r, const Matrix& m, uint32_t row, bool live, uint32_t k) {
  Run<kWord> o = r.run;
  const uint32_t from_k = m.K - 16 - k;                       // the tail's place in the run: 0 or 32 if in it
  if (from_k == 0u) {
    o.lo.x = r.tail.x;
    o.lo.y = r.tail.y;
  }
  if (from_k == 32u) {
    o.hi.x = r.tail.x;
    o.hi.y = r.tail.y;
  }
  const uint32_t s = row * (m.K >> 4) + (k >> 4);
  const uint32_t back = s > m.last_scale ? s - m.last_scale : 0u;
  const uint32_t left = live && k < m.K ? (m.K - k) >> 4 : 0u;          // scales of the run that are the row's
  o.scales = left == 0u ? 0u : (r.run.scales >> (8u * back)) & (left >= 4u ? 0xFFFFFFFFu : (1u << (8u * left)) - 1u);
  return o;
}

template <Shape S>
__device__ __forceinline__ half8 octet_of(const Run<S>& r, int t) {
  if constexpr (S == kHalf) return decode8(t < 2 ? r.lo[t & 1] : r.hi[t & 1], scale_pair(t < 2 ? r.s0 : r.s1));
  else
    return decode8(t < 4 ? r.lo[t & 3] : r.hi[t & 3], scale_pair((r.scales >> (8 * (t >> 1))) & 0xFFu));
}

// acc[i][c] += rows 16 i .. + 15 of the tile times token columns 16 c .. + 15, over the steps
// first, first + stride, ... below `steps` (from element 0 on). row: this lane's row of each
// fragment. Tok: load(c, k) -> Raw, what the lane needs of column 16 c + l % 16 for its run at k;
// cook(c, raw, k) -> Cur; octet(cur, k, t) -> half8, zeros past K or without a token.
// Loads return in the order of issue and the wait counts the younger ones, so a step's loads stay
// together and in step order (the scheduling barriers), the tokens as far ahead as the weights.
// A: steps in flight (they cost 9, 11 or 5 registers for each fragment of rows or NVFP4 columns).
template <int R, int C, int A, Shape S, class Tok>
struct Pipe {
  Loaded<S> w[A][R];
  typename Tok::Raw x[A][C];

  static __device__ __forceinline__ uint32_t element(int s) {
    return (uint32_t)s * kStep<S> + ((threadIdx.x & 63) >> 4) * kRun<S>;
  }

  __device__ __forceinline__ void load(const Matrix& m, const uint32_t (&row)[R], const Tok& tok, int d, int s) {
    const uint32_t k = element(s);
#pragma unroll
    for (int c = 0; c < C; ++c) x[d][c] = tok.load(c, k);
#pragma unroll
    for (int i = 0; i < R; ++i) w[d][i] = load_run<S>(m, row[i], true, k);
    __builtin_amdgcn_sched_barrier(0);
  }

  __device__ __forceinline__ void start(const Matrix& m, const uint32_t (&row)[R], const Tok& tok, int first, int stride) {
#pragma unroll
    for (int d = 0; d < A; ++d) load(m, row, tok, d, first + d * stride);
  }

  __device__ __forceinline__ void run(const Matrix& m, const uint32_t (&row)[R], const Tok& tok, int first, int stride,
                                      int steps, float4v (&acc)[R][C]) {
#pragma unroll 1
    for (int s0 = first; s0 < steps; s0 += A * stride) {
#pragma unroll
      for (int d = 0; d < A; ++d) {
        const int s = s0 + d * stride;
        if (s >= steps) return;                               // uniform (a break would look like another turn)
        const uint32_t k = element(s);
        Run<S> a[R];
        typename Tok::Cur b[C];
        if constexpr (S == kWord) {                           // (the others: where they are used; here up to 5 % more)
#pragma unroll
          for (int i = 0; i < R; ++i) a[i] = run_of(w[d][i], m, row[i], true, k);
#pragma unroll
          for (int c = 0; c < C; ++c) b[c] = tok.cook(c, x[d][c], k);
        }
#pragma unroll
        for (int t = 0; t < kOctets<S>; ++t) {
          half8 v[C];
#pragma unroll
          for (int c = 0; c < C; ++c) {
            if constexpr (S == kWord) v[c] = tok.octet(b[c], k, t);
            else v[c] = tok.octet(tok.cook(c, x[d][c], k), k, t);
          }
#pragma unroll
          for (int i = 0; i < R; ++i) {
            half8 u;
            if constexpr (S == kWord) u = octet_of(a[i], t);
            else u = octet_of(w[d][i].run, t);
#pragma unroll
            for (int c = 0; c < C; ++c) acc[i][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(u, v[c], acc[i][c], 0, 0, 0);
          }
        }
        load(m, row, tok, d, s + A * stride);
      }
    }
  }
};

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
