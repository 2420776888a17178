// One AdamW step over many tensors in one launch, states in FP32 or in 8 bits.
//
// For every element (FP32, each operation rounded once, no contraction):
//   g  = c * grad                         c = min(1, max_norm / (norm + 1e-6)), 1 without clipping
//   m' = b1 m + (1 - b1) g                v' = b2 v + (1 - b2) g^2
//   p' = p (1 - lr wd) - lr / (1 - b1^t) * m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
//   w' = BF16(p')                         the weights the layer's quantizer reads
// 8-bit states hold m and r = sqrt(v) as E4M3 elements with one power-of-two (E8M0) scale per 32
// elements: 2^e with the smallest e that keeps the block's maximum at or below 448 (no
// saturation), e >= -117 so that every element is a normal FP32 number. r instead of v halves
// the exponent range: one block spans a factor 2^17.8 = 2.3e5 in r, 5e10 in v. Rounding is
// stochastic: with b2 = 0.95..0.999 a step moves v by less than half an E4M3 step, so rounding
// to nearest would leave r where it is for ever, while up where fraction + h/65536 >= 1 (h: 16
// random bits) keeps the running mean's expectation. 16 bits because the rule truncates: on
// average it rounds down by 2^-17 of a gap, and at b2 = 0.999 the 2^-9 of 8 bits would be a third
// of what a step takes from r. m and r of an element share their h: only the two errors' product
// knows. Rounding never makes a nonzero r 0 (m / eps would follow); below 2^-75, where r^2 leaves
// FP32, r falls to 0, and m, no larger than gradients of that size make it, is nothing against eps.
//
// Memory bound: 4 + 8 + 2 bytes (grad, p in and out, w) plus 16 (FP32 m, v in and out) or 4.125
// (8 bits) per element against about 40 and 110 vector operations. Each thread takes 8
// consecutive elements (one Philox call gives their 8 times 16 bits, 4 neighbouring lanes a
// block of 32). A workgroup takes one chunk of 2048 elements of one tensor (the table holds the chunk's
// tensor, so finding it is one load and not a search).
// Measured: 209.7 M elements, FP32 states 1150 us (5.5 TB/s), their gradient's norm 154 (5.4 TB/s); 80.2 M
// elements, 8 bits 257 us (5.6 TB/s); a dozen tensors of 1 to 20480 elements 4.2 us, which is a launch.
#include "device_common.h"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                                       // elements per thread and pass
constexpr int64_t kPass = (int64_t)kThreads * kPer;
static_assert(kAdamWChunk % kPass == 0, "a workgroup takes a chunk in whole passes");

struct Elems { float v[kPer]; };

// Elements [i, i + 8) of a tensor of n, as whole vectors from any element boundary; 0 past its end.
__device__ __forceinline__ Elems load_f32(const float* p, int64_t i, int64_t n) {
  Elems e;
  if (i + kPer <= n) {
    const v4f32 a = *reinterpret_cast<const v4f32_any*>(p + i), b = *reinterpret_cast<const v4f32_any*>(p + i + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      e.v[q] = a[q];
      e.v[q + 4] = b[q];
    }
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q) e.v[q] = i + q < n ? p[i + q] : 0.0f;
  }
  return e;
}

__device__ __forceinline__ void store_f32(float* p, int64_t i, int64_t n, const Elems& e) {
  if (i + kPer <= n) {
    *reinterpret_cast<v4f32_any*>(p + i) = v4f32{e.v[0], e.v[1], e.v[2], e.v[3]};
    *reinterpret_cast<v4f32_any*>(p + i + 4) = v4f32{e.v[4], e.v[5], e.v[6], e.v[7]};
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (i + q < n) p[i + q] = e.v[q];
  }
}

__device__ __forceinline__ Elems load_grad(const void* p, bool bf16, int64_t i, int64_t n) {
  if (!bf16) return load_f32(static_cast<const float*>(p), i, n);
  Elems e;
  const uint16_t* h = static_cast<const uint16_t*>(p);
  if (i + kPer <= n) {
    const v4u32 w = *reinterpret_cast<const v4u32_any*>(h + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      e.v[2 * q] = bf16_lo(w[q]);
      e.v[2 * q + 1] = bf16_hi(w[q]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q) e.v[q] = i + q < n ? bf16_lo(h[i + q]) : 0.0f;
  }
  return e;
}

// Stores e rounded to BF16; returns the largest stored magnitude.
__device__ __forceinline__ float store_bf16(uint16_t* p, int64_t i, int64_t n, const Elems& e) {
  v4u32 w;
  float mx = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    w[q] = bf16_rn_pair(e.v[2 * q], e.v[2 * q + 1]);
    mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[q])), fabsf(bf16_hi(w[q]))));
  }
  if (i + kPer <= n) {
    *reinterpret_cast<v4u32_any*>(p + i) = w;
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (i + q < n) p[i + q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
  }
  return mx;                                                  // elements past n are 0
}

// ---- 8-bit states ----------------------------------------------------------------------------
struct Codes { uint32_t lo, hi; };                            // 8 codes, element 0 in the low byte

__device__ __forceinline__ Codes load_codes(const uint8_t* p, int64_t i, int64_t n) {
  if (i + kPer <= n) {
    const v2u32 w = *reinterpret_cast<const v2u32_any*>(p + i);
    return Codes{w.x, w.y};
  }
  Codes c{0, 0};
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const uint32_t b = i + q < n ? p[i + q] : 0u;
    if (q < 4) c.lo |= b << (8 * q); else c.hi |= b << (8 * (q - 4));
  }
  return c;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, Codes c) {
  if (i + kPer <= n) {
    *reinterpret_cast<v2u32_any*>(p + i) = v2u32{c.lo, c.hi};
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (i + q < n) p[i + q] = (uint8_t)((q < 4 ? c.lo : c.hi) >> (8 * (q & 3)));
  }
}

// 2^(s - 127) of an E8M0 code; 0 for code 0, the scale of an all-zero block.
__device__ __forceinline__ float e8m0_value(uint32_t s) { return __uint_as_float(s << 23); }

__device__ __forceinline__ Elems decode_codes(Codes c, float scale) {
  Elems e;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = (int)(h ? c.hi : c.lo);
    const v2f32 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    e.v[4 * h] = a[0] * scale;
    e.v[4 * h + 1] = a[1] * scale;
    e.v[4 * h + 2] = b[0] * scale;
    e.v[4 * h + 3] = b[1] * scale;
  }
  return e;
}

// E8M0 code of a block's scale from its maximum: the smallest e with amax <= 448 * 2^e
// (448 = 1.75 * 2^8), at least -117; 0 for an all-zero block.
__device__ __forceinline__ uint32_t scale_code(float amax) {
  if (amax == 0.0f) return 0u;
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)((e < -117 ? -117 : e) + 127);
}

// E4M3 code of y = |x| 2^-e (at most 448), rounded up iff fraction + r / 65536 >= 1.
__device__ __forceinline__ uint32_t e4m3_sr(float y, uint32_t r) {
  const uint32_t fine = ((__float_as_uint(y) + (r << 4)) >> 20) - (120u << 3);
  const uint32_t low = (uint32_t)(y * 512.0f + (float)r * 0x1p-16f);   // steps of 2^-9
  return y < 0.015625f ? low : (fine & 0x7Fu);
}

// The 8 elements of one lane in a block of 32 (lanes 4k .. 4k + 3) -> codes and the scale code.
template <bool KEEP_NONZERO>
__device__ __forceinline__ Codes encode_codes(const Elems& e, const u32x4& rnd, uint32_t& scale) {
  float mx = 0.0f;
#pragma unroll
  for (int q = 0; q < kPer; ++q) mx = fmaxf(mx, fabsf(e.v[q]));
  mx = fmaxf(mx, __shfl_xor(mx, 1, 64));
  mx = fmaxf(mx, __shfl_xor(mx, 2, 64));
  scale = scale_code(mx);
  const float inv = __uint_as_float((254u - scale) << 23);    // 2^-e; every y is 0 for scale 0
  Codes c{0, 0};
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const uint32_t w = q < 2 ? rnd.x : q < 4 ? rnd.y : q < 6 ? rnd.z : rnd.w;
    const uint32_t r = (q & 1) ? w >> 16 : w & 0xFFFFu;
    const float a = fabsf(e.v[q]);
    uint32_t k = e4m3_sr(a * inv, r);
    if (KEEP_NONZERO) k = (a > 0.0f && k == 0u) ? 1u : k;
    else k |= (__float_as_uint(e.v[q]) >> 31) << 7;
    if (q < 4) c.lo |= k << (8 * q); else c.hi |= k << (8 * (q - 4));
  }
  return c;
}

// Sum over the workgroup in a fixed order, the same for every thread (all threads must call).
__device__ __forceinline__ double group_sum(double v) {
  __shared__ double red[kThreads / 64];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) s += red[w];
  return s;
}

// partial[b] = sum of g^2 over the chunks b, b + gridDim.x, ...: FP32 over the 8 elements that a
// thread squares per chunk, binary64 beyond, a fixed order throughout. (A |g| above 1.8e19 makes it infinite.)
__global__ __launch_bounds__(kThreads) void k_grad_norm(const AdamWEntry* __restrict__ table,
                                                        const int32_t* __restrict__ chunk_of, int64_t chunks,
                                                        double* __restrict__ partial) {
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const AdamWEntry& t = table[chunk_of[c]];
    const int64_t n = t.n, c0 = (c - t.first_chunk) * kAdamWChunk;
    const bool bf16 = t.flags & kAdamWGradBf16;
    float s = 0.0f;
#pragma unroll
    for (int64_t o = 0; o < kAdamWChunk; o += kPass) {
      const int64_t i = c0 + o + (int64_t)threadIdx.x * kPer;
      if (i < n) {
        const Elems g = load_grad(t.grad, bf16, i, n);
#pragma unroll
        for (int q = 0; q < kPer; ++q) s += g.v[q] * g.v[q];
      }
    }
    sum += (double)s;
  }
  sum = group_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <bool EIGHT>
__global__ __launch_bounds__(kThreads) void k_adamw(const AdamWEntry* __restrict__ table,
                                                    const int32_t* __restrict__ chunk_of, AdamWHyper hp,
                                                    const double* __restrict__ partial, int parts,
                                                    float* __restrict__ norm_out, float* __restrict__ amax_out) {
  const int32_t ti = chunk_of[blockIdx.x];
  const AdamWEntry& t = table[ti];
  const int64_t n = t.n, c0 = ((int64_t)blockIdx.x - t.first_chunk) * kAdamWChunk;
  const bool bf16 = t.flags & kAdamWGradBf16;
  float clip = 1.0f;
  bool skip = false;                                          // uniform
  if (parts > 0) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
    const float norm = (float)sqrt(group_sum(s));
    clip = fminf(hp.max_norm / (norm + 1e-6f), 1.0f);
    skip = !(norm <= kFltMax);                                // infinite or NaN: the step changes nothing
    if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  }
  const float shrink = 1.0f - hp.lr * t.weight_decay;
  float mx = 0.0f;
  // one pass, and a loop all the same: ahead of it the compiler asks for the entry's pointers together, without
  // it one after the other (a dozen tensors of 1 to 20480 elements 4.2 us, 4.9 without the loop)
#pragma unroll 1
  for (int64_t o = 0; o < kAdamWChunk && c0 + o < n; o += kPass) {
    const int64_t i = c0 + o + (int64_t)threadIdx.x * kPer;   // lanes past n carry zeros to the shuffles
    Elems p = load_f32(t.p, i, n);
    const Elems grad = load_grad(t.grad, bf16, i, n);
    Elems m, v;
    Codes mc{0, 0}, rc{0, 0};
    uint32_t ms = 0, rs = 0;
    if constexpr (EIGHT) {
      mc = load_codes(static_cast<const uint8_t*>(t.m), i, n);
      rc = load_codes(static_cast<const uint8_t*>(t.v), i, n);
      if (i < n) {
        ms = t.m_scale[i >> 5];
        rs = t.v_scale[i >> 5];
      }
      m = decode_codes(mc, e8m0_value(ms));
      v = decode_codes(rc, e8m0_value(rs));
    } else {
      m = load_f32(static_cast<const float*>(t.m), i, n);
      v = load_f32(static_cast<const float*>(t.v), i, n);
    }
    if (!skip) {
      Elems r;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const float g = parts > 0 ? grad.v[q] * clip : grad.v[q];
        const float v0 = EIGHT ? v.v[q] * v.v[q] : v.v[q];
        m.v[q] = hp.beta1 * m.v[q] + hp.one_beta1 * g;
        v.v[q] = hp.beta2 * v0 + hp.one_beta2 * (g * g);
        r.v[q] = sqrtf(v.v[q]);
        const float denom = r.v[q] * hp.inv_sqrt_bc2 + hp.eps;
        p.v[q] = p.v[q] * shrink - hp.step_size * (m.v[q] / denom);
      }
      if constexpr (EIGHT) {
        const uint64_t grp = (uint64_t)i >> 3;
        const u32x4 rnd = philox4x32_10(u32x4{(uint32_t)grp, (uint32_t)(grp >> 32), hp.step, (uint32_t)ti},
                                        (uint32_t)hp.seed, (uint32_t)(hp.seed >> 32));
        // (elements past n are 0 in m and r: they do not count towards their block's maximum)
        mc = encode_codes<false>(m, rnd, ms);
        rc = encode_codes<true>(r, rnd, rs);
      }
    }
    if (i < n) {
      store_f32(t.p_out, i, n, p);
      float big = 0.0f;
      if (t.w_out != nullptr) {
        big = store_bf16(t.w_out, i, n, p);
      } else {
#pragma unroll
        for (int q = 0; q < kPer; ++q) big = fmaxf(big, fabsf(p.v[q]));
      }
      mx = fmaxf(mx, big);
      if constexpr (EIGHT) {
        store_codes(static_cast<uint8_t*>(t.m_out), i, n, mc);
        store_codes(static_cast<uint8_t*>(t.v_out), i, n, rc);
        if ((i & 31) == 0) {
          t.m_scale_out[i >> 5] = (uint8_t)ms;
          t.v_scale_out[i >> 5] = (uint8_t)rs;
        }
      } else {
        store_f32(static_cast<float*>(t.m_out), i, n, m);
        store_f32(static_cast<float*>(t.v_out), i, n, v);
      }
    }
  }
  if (amax_out != nullptr) {                                  // uniform
    mx = wave_max(mx);
    if ((threadIdx.x & 63) == 0) atomic_raise_nonneg(&amax_out[ti], mx);
  }
}

}  // namespace

int adamw_norm_parts(int64_t chunks) { return (int)(chunks < kAdamWMaxParts ? chunks : kAdamWMaxParts); }

hipError_t launch_adamw(const void* table, int64_t count, int64_t chunks, bool eight, const AdamWHyper& hp,
                        bool clip, double* ws, float* norm_out, float* amax_out, hipStream_t stream) {
  const AdamWEntry* entries = static_cast<const AdamWEntry*>(table);
  const int32_t* chunk_of = reinterpret_cast<const int32_t*>(entries + count);
  if (amax_out) {
    const hipError_t e = launch_fill(amax_out, count, 0.0f, stream);
    if (e != hipSuccess) return e;
  }
  if (chunks == 0) {                                          // nothing but empty tensors
    if (clip && norm_out) return launch_fill(norm_out, 1, 0.0f, stream);
    return hipGetLastError();
  }
  const int parts = clip ? adamw_norm_parts(chunks) : 0;
  if (clip) hipLaunchKernelGGL(k_grad_norm, dim3(parts), dim3(kThreads), 0, stream, entries, chunk_of, chunks, ws);
  if (eight)
    hipLaunchKernelGGL(k_adamw<true>, dim3((unsigned)chunks), dim3(kThreads), 0, stream, entries, chunk_of, hp, ws,
                       parts, norm_out, amax_out);
  else
    hipLaunchKernelGGL(k_adamw<false>, dim3((unsigned)chunks), dim3(kThreads), 0, stream, entries, chunk_of, hp, ws,
                       parts, norm_out, amax_out);
  return hipGetLastError();
}

}  // namespace nvfp4
