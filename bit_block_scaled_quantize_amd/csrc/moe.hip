// A whole mixture-of-experts layer for a few tokens (at most 64), experts in NVFP4:
//   l = x R^T;  the k largest l of a token pick its experts (ties: the lowest index)
//   score = softmax(l) or sigmoid(l);  w_j = score_j * routed_scale, or score_j / (sum over the picked
//   + 1e-20) * routed_scale
//   y = sum_j w_j W2_j h_j,  h_j = act(W1_j x), or act(G_j x) * (U_j x) with W1_j = [G_j; U_j]
//
// Bound by reading each chosen expert's weights once (9/16 byte per element): 1 token with 6 of
// 128 experts of 2688 x 1856 reads 34 MB, 64 tokens read most of the 718 MB. Three launches, each
// the next one's dependence on all of the one before:
//  1. k_route: logits (a wave per expert, 8 tokens at a time), x in FP16; the last workgroup of a
//     token group to finish picks its tokens' experts, the last group to finish sorts the
//     (token, expert) pairs by expert.
//  2. k_expert<UP>: 16 R rows of one used expert times its tokens (skinny.h), the activation, h.
//  3. k_expert<DOWN>: the same over W2, the routing weight, one partial result per pair; the last
//     workgroup of a row tile to finish adds the k partials of each token in order.
// "The last to finish" is found with a counter that the last one resets: nothing waits for
// anything, and no sum depends on an order of arrival.
//
// The matrix instruction takes FP16 columns: x and h are scaled by a power of two per token (per
// pair) that brings their largest magnitude into [2^14, 2^15). A BF16 x is then exact down to
// 2^-28 of that maximum, and what is lost below is under 2^-40 of it; an FP32 h keeps 11 bits,
// three more than the BF16 result. Non-finite tokens take scale 1 and come out non-finite; other
// tokens' columns do not see them.
#include "activation.h"
#include "launch.h"
#include "skinny.h"

namespace nvfp4 {
namespace {

using namespace skinny;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kGroupTokens = 8;                               // tokens per workgroup of k_route

// 2^e with max |v| 2^e in [2^14, 2^15); 1 for a zero or non-finite maximum. Exponents are kept
// where the scale and its inverse are normal numbers.
__device__ __forceinline__ float half_scale(float top) {
  const uint32_t b = __float_as_uint(top) >> 23;              // biased exponent
  if (top == 0.0f || b == 255u) return 1.0f;
  const int e = 14 - ((int)b - 127);
  return __uint_as_float((uint32_t)((e > 120 ? 120 : e) + 127) << 23);
}

__device__ __forceinline__ half2v half_pair(float a, float b) { return half2v{(_Float16)a, (_Float16)b}; }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// True in the workgroup that is the last of `total` to call this with `counter`, which it resets.
// What the others wrote before is visible to it afterwards. All threads call.
__device__ __forceinline__ bool last_to_finish(int* counter, int total) {
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int before = atomicAdd(counter, 1);
    last = before == total - 1;
    if (last) atomicExch(counter, 0);
  }
  __syncthreads();
  const bool is_last = last != 0;
  __syncthreads();
  if (is_last) __threadfence();
  return is_last;
}

// Eight elements of a BF16 or FP32 row from element i (0 past n).
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int64_t i, int64_t n, bool vec, float (&v)[8]) {
  if (vec && i + 8 <= n) {
    if constexpr (F32) {
      const v4f32 a = ld_f32x4(static_cast<const float*>(row) + i), b = ld_f32x4(static_cast<const float*>(row) + i + 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] = a[q];
        v[q + 4] = b[q];
      }
    } else {
      const v4u32 w = ld_u32x4(static_cast<const uint16_t*>(row) + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = bf16_lo(w[q]);
        v[2 * q + 1] = bf16_hi(w[q]);
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (F32) v[q] = i + q < n ? static_cast<const float*>(row)[i + q] : 0.0f;
      else v[q] = i + q < n ? bf16_lo(static_cast<const uint16_t*>(row)[i + q]) : 0.0f;
    }
  }
}

// The k largest logits of one token (one wave), ties to the lowest expert, NaN last; ids and weights.
// At most kMoeMaxExperts experts: lane l holds experts l, l + 64, ...
__device__ __forceinline__ void pick_experts(const MoeArgs& a, const MoeWork& w, int t) {
  constexpr int kPer = (int)(kMoeMaxExperts / 64);
  const int lane = threadIdx.x & 63;
  const float* logits = w.logits + (int64_t)t * a.experts;
  float key[kPer];
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane + 64 * j;
    const float l = e < a.experts ? logits[e] : -INFINITY;
    key[j] = l == l ? l : -INFINITY;
    top = fmaxf(top, l);
  }
  float denom = 0.0f;                                         // of the softmax over all experts
  if (!a.sigmoid) {
    top = wave_max(top);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = lane + 64 * j;
      if (e < a.experts) denom += expf(logits[e] - top);
    }
    denom = wave_sum(denom);
  }
  uint32_t taken = 0;                                         // bit j: this lane's expert j
  float mine = 0.0f, total = 0.0f;                            // lane j keeps pick j's score
  int id = 0;
  for (int j = 0; j < a.top_k; ++j) {
    float best = -INFINITY;
    int at = -1;
#pragma unroll
    for (int q = kPer - 1; q >= 0; --q)                       // the lowest of equals last
      if (lane + 64 * q < a.experts && !((taken >> q) & 1u) && (at < 0 || key[q] >= best)) {
        best = key[q];
        at = q;
      }
    const float m = wave_max(at < 0 ? -INFINITY : best);
    // among the lanes that hold it, the lowest expert: lowest q, then lowest lane
    int e = at >= 0 && best == m ? lane + 64 * at : 0x7FFFFFFF;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const int other = __shfl_xor(e, o, 64);
      e = other < e ? other : e;
    }
    if ((e & 63) == lane) taken |= 1u << (e >> 6);
    const float l = logits[e];
    const float s = a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top) / denom;
    total += s;
    if (lane == j) {
      mine = s;
      id = e;
    }
  }
  if (lane < a.top_k) {
    const float wt = (a.renormalize ? mine / (total + 1e-20f) : mine) * a.routed_scale;
    const int64_t p = (int64_t)t * a.top_k + lane;
    w.ids[p] = id;
    w.weights[p] = wt;
    if (a.ids_out) a.ids_out[p] = id;
    if (a.weights_out) a.weights_out[p] = wt;
  }
}

// The pairs (token t, pick j), numbered t * top_k + j, sorted by expert: w.order[w.begin[u] ..
// w.begin[u + 1]) are those of the u-th used expert w.expert[u]. The order within an expert is that
// of arrival; a pair's place decides which column it takes and nothing of its result.
__device__ __forceinline__ void sort_pairs(const MoeArgs& a, const MoeWork& w) {
  __shared__ int count[kMoeMaxExperts], start[kMoeMaxExperts], used_before[kMoeMaxExperts];
  const int pairs = a.tokens * a.top_k;
  for (int e = threadIdx.x; e < a.experts; e += kThreads) count[e] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += kThreads) atomicAdd(&count[w.ids[p]], 1);
  __syncthreads();
  if (threadIdx.x < 64) {                                     // one wave: exclusive sums over the experts
    int pos = 0, used = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
      const int e = e0 + threadIdx.x;
      const int c = e < a.experts ? count[e] : 0;
      int sum = c;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(sum, d);
        if ((int)threadIdx.x >= d) sum += y;
      }
      const uint64_t have = __ballot(c > 0);
      if (e < a.experts) {
        start[e] = pos + sum - c;
        used_before[e] = used + __popcll(have & ((1ull << threadIdx.x) - 1));
      }
      pos += __shfl(sum, 63);
      used += __popcll(have);
    }
    if (threadIdx.x == 0) {
      *w.used = used;
      w.begin[used] = pairs;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kThreads) {
    if (count[e] > 0) {
      w.expert[used_before[e]] = e;
      w.begin[used_before[e]] = start[e];
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += kThreads) w.order[atomicAdd(&start[w.ids[p]], 1)] = p;
}

// Grid: x = blocks of 4 experts, then one more block that brings the group's tokens to FP16; y =
// groups of 8 tokens.
template <bool F32>
__global__ __launch_bounds__(kThreads) void k_route(MoeArgs a, MoeWork w, bool vec_x, bool vec_r) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.y * kGroupTokens;
  const int nt = a.tokens - t0 < kGroupTokens ? a.tokens - t0 : kGroupTokens;
  const int blocks = (int)gridDim.x - 1;
  const int64_t H = a.hidden;
  if ((int)blockIdx.x == blocks) {
    for (int q = wave; q < nt; q += kWaves) {
      const int t = t0 + q;
      const uint16_t* row = a.x + (int64_t)t * a.ldx;
      float top = 0.0f;
      for (int64_t i = lane * 8; i < H; i += 512) {
        float v[8];
        load8<false>(row, i, H, vec_x, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
      }
      const float s = half_scale(wave_max(top));
      for (int64_t i = lane * 8; i < H; i += 512) {            // H is a multiple of 16
        float v[8];
        load8<false>(row, i, H, vec_x, v);
        half8 o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = (_Float16)(v[j] * s);
        *reinterpret_cast<half8*>(w.x16 + (int64_t)t * H + i) = o;
      }
      if (lane == 0) w.x_inv[t] = 1.0f / s;                   // a power of two: exact
      if (lane < a.top_k) w.h_top[(int64_t)t * a.top_k + lane] = 0u;
    }
    return;
  }
  const int e = blockIdx.x * kWaves + wave;
  if (e < a.experts) {
    const void* row = static_cast<const uint8_t*>(a.router) + (int64_t)e * H * (F32 ? 4 : 2);
    float acc[kGroupTokens] = {};
    for (int64_t i = lane * 8; i < H; i += 512) {
      float r[8];
      load8<F32>(row, i, H, vec_r, r);
#pragma unroll
      for (int q = 0; q < kGroupTokens; ++q) {
        if (q < nt) {                                         // uniform
          float v[8];
          load8<false>(a.x + (int64_t)(t0 + q) * a.ldx, i, H, vec_x, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[q] = __builtin_fmaf(r[j], v[j], acc[q]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kGroupTokens; ++q) {
      if (q < nt) {
        const float l = wave_sum(acc[q]);
        if (lane == 0) w.logits[(int64_t)(t0 + q) * a.experts + e] = l;
      }
    }
  }
  if (!last_to_finish(&w.counters[1 + blockIdx.y], blocks)) return;
  for (int q = wave; q < nt; q += kWaves) pick_experts(a, w, t0 + q);
  if (!last_to_finish(&w.counters[0], (int)gridDim.y)) return;
  sort_pairs(a, w);
}

// Columns of the up product: FP16 rows of x.
template <int C>
struct TokensHalf {
  struct Raw { half8 v[4]; };
  const _Float16* row[C];
  bool live[C];
  int64_t K;
  __device__ __forceinline__ Raw load(int c, int64_t k) const {
    Raw r;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      r.v[t] = half8{};
      if (live[c] && k + 8 * t < K) r.v[t] = *reinterpret_cast<const half8*>(row[c] + k + 8 * t);
    }
    return r;
  }
  __device__ __forceinline__ half8 octet(int, const Raw& r, int t) const { return r.v[t]; }
};

// Columns of the down product: FP32 rows of h, scaled into FP16.
template <int C>
struct TokensFloat {
  struct Raw { v4f32 v[8]; };
  const float* row[C];
  float scale[C];                                             // a power of two per column
  bool live[C];
  int64_t K;
  __device__ __forceinline__ Raw load(int c, int64_t k) const {
    Raw r;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      r.v[2 * t] = r.v[2 * t + 1] = v4f32{};
      if (live[c] && k + 8 * t < K) {
        r.v[2 * t] = ld_f32x4(row[c] + k + 8 * t);
        r.v[2 * t + 1] = ld_f32x4(row[c] + k + 8 * t + 4);
      }
    }
    return r;
  }
  __device__ __forceinline__ half8 octet(int c, const Raw& r, int t) const {
    const v4f32 a = r.v[2 * t] * scale[c], b = r.v[2 * t + 1] * scale[c];
    return half8{(_Float16)a[0], (_Float16)a[1], (_Float16)a[2], (_Float16)a[3],
                 (_Float16)b[0], (_Float16)b[1], (_Float16)b[2], (_Float16)b[3]};
  }
};

// 16 R weight rows of one used expert times its tokens, 16 C at a time (the weights' second and
// later readings come from the cache). Grid: used experts (as many as there can be; the surplus
// leaves at once) x row tiles, tiles of one expert next to each other.
// UP: rows of W1, K = hidden -> h[pair][f]. GATED: fragments 0 .. R/2 - 1 hold the gate's rows, the
// others the same rows of U. DOWN: rows of W2, K = ffn -> part[pair][n], then y.
template <bool UP, bool GATED, int R, int C, bool K32>
__global__ __launch_bounds__(kThreads) void k_expert(MoeArgs a, MoeWork w, int tiles) {
  constexpr int RO = GATED ? R / 2 : R;                       // fragments of output rows
  __shared__ __attribute__((aligned(16))) float red[kWaves * R * C * 64 * 4];
  const int u = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int used = *w.used;
  if (u >= used) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int e = w.expert[u];
  const int p0 = w.begin[u], p1 = w.begin[u + 1];
  const int64_t K = UP ? a.hidden : a.ffn, N = UP ? a.ffn : a.hidden;
  const int64_t n0 = (int64_t)tile * (16 * RO);
  const GemmOperand& m = UP ? a.w1 : a.w2;
  const uint8_t *rc[R], *rs[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    int64_t n = n0 + 16 * (i % RO) + r;
    n = n < N ? n : n0;                                       // rows past N: not stored
    const int64_t row = (int64_t)e * (GATED ? 2 * N : N) + (i >= RO ? N : 0) + n;
    rc[i] = m.codes + row * (K >> 1);
    rs[i] = m.scales + row * (K >> 4);
  }
  const float gs = m.global_scale[e];
  for (int q0 = p0; q0 < p1; q0 += 16 * C) {
    int pair[C];
    bool live[C];
    float4v acc[R][C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int q = q0 + 16 * c + r;
      live[c] = q < p1;
      pair[c] = w.order[live[c] ? q : q0];
#pragma unroll
      for (int i = 0; i < R; ++i) acc[i][c] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    }
    float inv[C];                                             // undoes the column's power of two
    if constexpr (UP) {
      TokensHalf<C> tok;
      tok.K = K;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int t = pair[c] / a.top_k;
        tok.row[c] = w.x16 + (int64_t)t * K;
        tok.live[c] = live[c];
        inv[c] = w.x_inv[t];
      }
      accumulate<R, C, K32>(rc, rs, K, wave, kWaves, tok, acc);
    } else {
      TokensFloat<C> tok;
      tok.K = K;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float s = half_scale(__uint_as_float(w.h_top[pair[c]]));
        tok.row[c] = w.h + (int64_t)pair[c] * K;
        tok.scale[c] = s;
        tok.live[c] = live[c];
        inv[c] = w.weights[pair[c]] / s;                      // s a power of two: exact
      }
      accumulate<R, C, K32>(rc, rs, K, wave, kWaves, tok, acc);
    }
    if (q0 != p0) __syncthreads();                            // the last round's sums have been read
    put<R, C>(red, wave, acc);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float top = 0.0f;
#pragma unroll 1
      for (int i = wave; i < RO; i += kWaves) {
        const int64_t n = n0 + 16 * i + 4 * g;                // N % 16 == 0: all four rows or none
        float4v v = take<kWaves, R, C>(red, i, c);
        const float f = gs * inv[c];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] *= f;
        if constexpr (UP) {
          float4v z = v;
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = act_of(a.act, z[q]);
          if constexpr (GATED) {
            const float4v up = take<kWaves, R, C>(red, i + RO, c);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] *= up[q] * f;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) top = fmaxf(top, n < N ? fabsf(v[q]) : 0.0f);
        }
        float* out = (UP ? w.h : w.part) + (int64_t)pair[c] * N + n;
        if (live[c] && n < N) *reinterpret_cast<float4v*>(out) = v;
      }
      if constexpr (UP) {
        // NaN is dropped by the maximum and stays in h; an infinite maximum gives scale 1
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        if (live[c] && g == 0 && top > 0.0f) atomicMax(&w.h_top[pair[c]], __float_as_uint(top));
      }
    }
  }
  if constexpr (!UP) {
    if (!last_to_finish(&w.counters[1 + kMoeMaxTokens / kGroupTokens + tile], used)) return;
    const int rows = (int)(N - n0 < 16 * R ? N - n0 : 16 * R);
    for (int i = threadIdx.x; i < a.tokens * 16 * R; i += kThreads) {
      const int t = i / (16 * R), n = i % (16 * R);
      if (n >= rows) continue;
      const float* part = w.part + (int64_t)t * a.top_k * N + n0 + n;
      float s = 0.0f;
      for (int j = 0; j < a.top_k; ++j) s += part[(int64_t)j * N];
      a.y[(int64_t)t * a.ldy + n0 + n] = (uint16_t)bf16_rn_bits(s);
    }
  }
}

constexpr int kRows = 4;                                      // fragments of 16 rows per workgroup

int64_t tiles_of(int64_t rows, int frags) { return (rows + 16 * frags - 1) / (16 * frags); }

template <bool UP, bool GATED>
void launch_expert(const MoeArgs& a, const MoeWork& w, hipStream_t stream) {
  const int64_t K = UP ? a.hidden : a.ffn, N = UP ? a.ffn : a.hidden;
  const int64_t pairs = (int64_t)a.tokens * a.top_k;
  const int64_t most = pairs < a.experts ? pairs : a.experts;
  const int tiles = (int)tiles_of(N, GATED ? kRows / 2 : kRows);
  const dim3 grid((unsigned)(most * tiles));
#define NVFP4_EX(C, K32) \
  hipLaunchKernelGGL((k_expert<UP, GATED, kRows, C, K32>), grid, dim3(kThreads), 0, stream, a, w, tiles)
  if (a.tokens <= 16) {
    if (K % 32 == 0) NVFP4_EX(1, true); else NVFP4_EX(1, false);
  } else {
    if (K % 32 == 0) NVFP4_EX(2, true); else NVFP4_EX(2, false);
  }
#undef NVFP4_EX
}

}  // namespace

// Workspace layout, every part on 256 bytes. The counters come first: they are zero before and
// after every call.
size_t moe_layout(const MoeArgs& a, uint8_t* base, MoeWork* w) {
  size_t at = 0;
  auto part = [&](size_t bytes) {
    uint8_t* p = base ? base + at : nullptr;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t T = (size_t)a.tokens, P = T * (size_t)a.top_k, E = (size_t)a.experts;
  MoeWork x;
  x.counters = reinterpret_cast<int*>(part(moe_counter_bytes(a.hidden)));
  x.used = reinterpret_cast<int*>(part(4));
  x.expert = reinterpret_cast<int*>(part(4 * E));
  x.begin = reinterpret_cast<int*>(part(4 * (E + 1)));
  x.order = reinterpret_cast<int*>(part(4 * P));
  x.ids = reinterpret_cast<int*>(part(4 * P));
  x.weights = reinterpret_cast<float*>(part(4 * P));
  x.logits = reinterpret_cast<float*>(part(4 * T * E));
  x.x_inv = reinterpret_cast<float*>(part(4 * T));
  x.h_top = reinterpret_cast<uint32_t*>(part(4 * P));
  x.x16 = reinterpret_cast<_Float16*>(part(2 * T * (size_t)a.hidden));
  x.h = reinterpret_cast<float*>(part(4 * P * (size_t)a.ffn));
  x.part = reinterpret_cast<float*>(part(4 * P * (size_t)a.hidden));
  if (w) *w = x;
  return at;
}

// One counter per row tile of the down product (the smallest tile has 16 rows), after those of k_route.
size_t moe_counter_bytes(int64_t hidden) {
  return 4 * (size_t)(1 + kMoeMaxTokens / kGroupTokens + (hidden + 15) / 16);
}

hipError_t launch_moe(const MoeArgs& a, uint8_t* ws, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  MoeWork w;
  moe_layout(a, ws, &w);
  const bool vec_x = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % 8 == 0;
  const bool vec_r = reinterpret_cast<uintptr_t>(a.router) % 16 == 0;      // hidden % 16 == 0
  const dim3 grid((unsigned)((a.experts + kWaves - 1) / kWaves + 1),
                  (unsigned)((a.tokens + kGroupTokens - 1) / kGroupTokens));
  if (a.router_f32) hipLaunchKernelGGL(k_route<true>, grid, dim3(kThreads), 0, stream, a, w, vec_x, vec_r);
  else hipLaunchKernelGGL(k_route<false>, grid, dim3(kThreads), 0, stream, a, w, vec_x, vec_r);
  if (a.gated) launch_expert<true, true>(a, w, stream);
  else launch_expert<true, false>(a, w, stream);
  launch_expert<false, false>(a, w, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
