// A whole mixture-of-experts layer for a few tokens (at most 64), experts in NVFP4:
//   l = x R^T;  the k largest l of a token pick its experts (ties: the lowest index)
//   score = softmax(l) or sigmoid(l);  w_j = score_j * routed_scale, or score_j / (sum over the picked
//   + 1e-20) * routed_scale
//   y = sum_j w_j W2_j h_j,  h_j = act(W1_j x), or act(G_j x) * (U_j x) with W1_j = [G_j; U_j]
//
// Bound by reading each chosen expert's weights once (9/16 byte per element): 1 token with 6 of
// 128 experts of 2688 x 1856 reads 34 MB, 64 tokens read most of the 718 MB. Three launches, or four, each
// depending on all of the one before:
//  1. k_route: logits (4 experts and 8 tokens a workgroup), x in FP16; the last workgroup of a
//     token group to finish picks its tokens' experts, the last group to finish sorts the
//     (token, expert) pairs by expert.
//  2. k_expert<UP>: 32 rows (gated: 16 of each half; for one token 16) of one used expert times its tokens
//     (skinny.h), the activation, h.
//  3. k_expert<DOWN>: 16, 32 or 64 rows of W2 likewise, the routing weight, one partial result per pair.
//  4. y, the k partials of each token added in order: up to 4 tokens by the last workgroup of a row tile
//     to finish, beyond by k_join (there is so much to add that those workgroups would be the launch's tail).
// Measured (that layer, us): 1 token 8.0 + 8.0 + 8.6 (the weights at 2 TB/s in the products: 17 MB each is
// 4 us of reading behind a launch's 3 us and the round trips to the routing, x and the weights); 64 tokens 17 +
// 95 + 96 + 5 (3.6 TB/s). Routing one token is latency: the logits, the counter, the picks one after the other.
// "The last to finish" is found with a counter that the last one resets: nothing waits for
// anything, and no sum depends on an order of arrival.
//
// The matrix instruction takes FP16 columns: x and h are scaled by a power of two per token (per
// pair) that brings their largest magnitude into [2^14, 2^15). A BF16 x is then exact down to
// 2^-28 of that maximum, and what is lost below is under 2^-40 of it; an FP32 h keeps 11 bits,
// three more than the BF16 result. A pair's maximum is known only when all of its h is, so h is
// stored with a scale for each 16 rows (its maximum beside it) and brought to the pair's in
// k_expert<DOWN>. Non-finite tokens take scale 1 and come out non-finite; other tokens' columns do not
// see them.
#include "activation.h"
#include "launch.h"
#include "skinny.h"

namespace nvfp4 {
namespace {

using namespace skinny;

constexpr int kRouteThreads = 512, kRouteWaves = 8;
constexpr int kRouteExperts = 4;                              // per workgroup of k_route
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

// What one workgroup writes and another of the same launch reads goes past the caches that are not
// shared (each XCD has its own L2) by device-scope accesses of single words; a release fence
// instead would write back the whole L2, once per workgroup (5400 of them took 0.4 ms).
template <class T>
__device__ __forceinline__ void put_shared(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T get_shared(const T* p) {
  return __hip_atomic_load(const_cast<T*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// True in the workgroup that is the last of `total` to call this with `counter`, which it resets.
// What the others had put_shared before is there for its get_shared: every wave waits until its
// stores have been acknowledged, then the workgroup meets, then it is counted. All threads call.
__device__ __forceinline__ bool last_to_finish(int* counter, int total) {
  __shared__ int last;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (total == 1) return true;                                // uniform: nobody else
  if (threadIdx.x == 0) {
    const int before = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = before == total - 1;
    if (last) put_shared(counter, 0);
  }
  __syncthreads();
  const bool is_last = last != 0;
  __syncthreads();
  return is_last;
}

// Eight elements of a BF16 or FP32 row from element i, 0 past n. VEC: as whole vectors through a buffer
// resource (the row starts on 16 bytes, n is a multiple of 8), which needs no branch past n, so the
// loads of several rows and places are in flight together.
struct Row {
  const void* p;
  __amdgpu_buffer_rsrc_t b;
};
template <bool F32, bool VEC>
__device__ __forceinline__ Row row_of(const void* p, int64_t n) {
  Row r;
  r.p = p;
  if constexpr (VEC) r.b = buffer(p, n * (F32 ? 4 : 2));
  return r;
}
template <bool F32, bool VEC>
struct Eight {
  v4u32 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const Row& row, int i, int n) {
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < (F32 ? 2 : 1); ++q) w[q] = load16(row.b, (uint32_t)i * (F32 ? 4 : 2) + 16 * q);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v[q] = 0u;
        if (i + q < n) v[q] = F32 ? static_cast<const uint32_t*>(row.p)[i + q] : static_cast<const uint16_t*>(row.p)[i + q];
      }
      if constexpr (F32) {
        w[0] = v4u32{v[0], v[1], v[2], v[3]};
        w[1] = v4u32{v[4], v[5], v[6], v[7]};
      } else {
        w[0] = v4u32{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
      }
    }
  }
  __device__ __forceinline__ float operator[](int q) const {
    if constexpr (F32) return __uint_as_float(w[q >> 2][q & 3]);
    else return (q & 1) ? bf16_hi(w[0][q >> 1]) : bf16_lo(w[0][q >> 1]);
  }
};

// The k largest logits of one token (one wave), ties to the lowest expert; its experts and weights.
// At most kMoeMaxExperts experts: lane l holds experts l, l + 64, ... A NaN logit ranks last, and one
// anywhere makes every weight of the token NaN.
__device__ __forceinline__ void pick_experts(const MoeArgs& a, const MoeWork& w, int t, int* own_ids) {
  constexpr int kPer = (int)(kMoeMaxExperts / 64);
  const int lane = threadIdx.x & 63;
  const float* logits = w.logits + (int64_t)t * a.experts;
  float key[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {                            // all in flight together
    if (64 * j >= a.experts) break;                           // uniform
    const int e = lane + 64 * j;
    key[j] = get_shared(&logits[e < a.experts ? e : a.experts - 1]);
  }
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (64 * j >= a.experts) break;
    bad |= key[j] != key[j];
    key[j] = lane + 64 * j < a.experts && key[j] == key[j] ? key[j] : -INFINITY;
    top = fmaxf(top, key[j]);
  }
  bad = __any(bad);
  top = wave_fold_max(top);
  float denom = 0.0f;                                         // of the softmax over all experts
  if (!a.sigmoid) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (64 * j < a.experts) denom += lane + 64 * j < a.experts ? expf(key[j] - top) : 0.0f;
    denom = wave_fold_sum(denom);
  }
  uint32_t taken = 0;                                         // bit j: this lane's expert j
  float mine = 0.0f, total = 0.0f;                            // lane j keeps pick j's score
  int id = 0;
  for (int j = 0; j < a.top_k; ++j) {
    float best = -INFINITY;
    int at = -1;
#pragma unroll
    for (int q = kPer - 1; q >= 0; --q) {                     // the lowest of equals last
      if (64 * q >= a.experts) continue;                      // uniform
      if (lane + 64 * q < a.experts && !((taken >> q) & 1u) && (at < 0 || key[q] >= best)) {
        best = key[q];
        at = q;
      }
    }
    const float l = wave_fold_max(best);                      // the pick's logit
    // among the lanes that hold it the lowest expert; top_k <= experts: one is left
    int e = 0;
#pragma unroll
    for (int q = kPer - 1; q >= 0; --q) {
      if (64 * q >= a.experts) continue;
      const uint64_t have = __ballot(at == q && best == l);
      e = have != 0 ? 64 * q + __builtin_ctzll(have) : e;
    }
    if ((e & 63) == lane) taken |= 1u << (e >> 6);
    const float s = a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top) / denom;
    total += s;
    if (lane == j) {
      mine = s;
      id = e;
    }
  }
  if (lane < a.top_k) {
    float wt = (a.renormalize ? mine / (total + 1e-20f) : mine) * a.routed_scale;
    if (bad) wt = __uint_as_float(0x7FC00000u);
    const int64_t p = (int64_t)t * a.top_k + lane;
    own_ids[lane] = id;
    put_shared(&w.ids[p], id);
    w.weights[p] = wt;
    if (a.ids_out) a.ids_out[p] = id;
    if (a.weights_out) a.weights_out[p] = wt;
  }
}

// The pairs (token t, pick j), numbered t * top_k + j, by expert: those of the u-th used expert
// w.expert[u] are w.order[u * 64 .. + w.count[u]) (a token has an expert at most once). Which slot a
// pair gets decides the column it takes and nothing of its result.
// own_ids: all the pairs' experts where one group has every token, else null (they are in w.ids).
__device__ __forceinline__ void sort_pairs(const MoeArgs& a, const MoeWork& w, const int* own_ids) {
  const int pairs = a.tokens * a.top_k;
  if (a.tokens == 1) {
    if ((int)threadIdx.x < pairs) {
      w.expert[threadIdx.x] = own_ids[threadIdx.x];
      w.count[threadIdx.x] = 1;
      w.order[threadIdx.x * kMoeMaxTokens] = threadIdx.x;
    }
    if (threadIdx.x == 0) *w.used = pairs;
    return;
  }
  __shared__ int count[kMoeMaxExperts], place[kMoeMaxExperts];
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) count[e] = 0;
  constexpr int kMine = (int)(kMoeMaxTokens * kMoeMaxTopK / kRouteThreads);
  int id[kMine], slot[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int p = threadIdx.x + i * kRouteThreads;
    id[i] = p < pairs ? (own_ids ? own_ids[p] : get_shared(&w.ids[p])) : -1;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (id[i] >= 0) slot[i] = atomicAdd(&count[id[i]], 1);
  __syncthreads();
  if (threadIdx.x < 64) {                                     // one wave numbers the used experts
    int used = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
      const int e = e0 + threadIdx.x;
      const int c = e < a.experts ? count[e] : 0;
      const uint64_t have = __ballot(c > 0);
      const int u = used + __popcll(have & ((1ull << threadIdx.x) - 1));
      if (c > 0) {
        place[e] = u;
        w.expert[u] = e;
        w.count[u] = c;
      }
      used += __popcll(have);
    }
    if (threadIdx.x == 0) *w.used = used;
    for (int u = used + (int)threadIdx.x; u < a.experts; u += 64) w.count[u] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (id[i] >= 0) w.order[place[id[i]] * kMoeMaxTokens + slot[i]] = threadIdx.x + i * kRouteThreads;
}

// Grid: x = blocks of 4 experts, then 8 blocks that bring one token each to FP16; y = groups of 8
// tokens. A logit block's waves split the hidden dimension, so that a row's loads are in flight
// together. NT: tokens of a group computed (1, or 8 with the surplus repeating the first).
// VEC: x's rows and the router's start on 16 bytes.
template <bool F32, int NT, bool VEC>
__global__ __launch_bounds__(kRouteThreads) void k_route(MoeArgs a, MoeWork w) {
  __shared__ float red[kRouteWaves][kRouteExperts * NT];
  __shared__ int own_ids[kGroupTokens * kMoeMaxTopK];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.y * kGroupTokens;
  const int nt = a.tokens - t0 < kGroupTokens ? a.tokens - t0 : kGroupTokens;
  const int blocks = (int)gridDim.x - kGroupTokens;
  const int H = (int)a.hidden;
  constexpr int kTurn = kRouteThreads * 8;
  if ((int)blockIdx.x >= blocks) {
    const int q = (int)blockIdx.x - blocks;
    if (q >= nt) return;
    const int t = t0 + q;
    const Row row = row_of<false, VEC>(a.x + (int64_t)t * a.ldx, H);
    float top = 0.0f;
    for (int i = threadIdx.x * 8; i < H; i += kTurn) {
      Eight<false, VEC> v;
      v.load(row, i, H);
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[k]));
    }
    top = wave_fold_max(top);
    if (lane == 0) red[wave][0] = top;
    __syncthreads();
    top = red[0][0];
#pragma unroll
    for (int v = 1; v < kRouteWaves; ++v) top = fmaxf(top, red[v][0]);
    const float s = half_scale(top);
    for (int i = threadIdx.x * 8; i < H; i += kTurn) {         // H is a multiple of 16
      Eight<false, VEC> v;
      v.load(row, i, H);
      half8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = (_Float16)(v[j] * s);
      *reinterpret_cast<half8*>(w.x16 + (int64_t)t * H + i) = o;
    }
    if (threadIdx.x == 0) w.x_inv[t] = 1.0f / s;              // a power of two: exact
    return;
  }
  const int e0 = blockIdx.x * kRouteExperts;
  float acc[kRouteExperts][NT] = {};
  for (int i = threadIdx.x * 8; i < H; i += kTurn) {
    Eight<F32, VEC> r[kRouteExperts];
    Eight<false, VEC> v[NT];
#pragma unroll
    for (int e = 0; e < kRouteExperts; ++e)
      r[e].load(row_of<F32, VEC>(static_cast<const uint8_t*>(a.router) +
                                     (int64_t)(e0 + e < a.experts ? e0 + e : e0) * H * (F32 ? 4 : 2), H), i, H);
#pragma unroll
    for (int q = 0; q < NT; ++q)
      v[q].load(row_of<false, VEC>(a.x + (int64_t)(t0 + (q < nt ? q : 0)) * a.ldx, H), i, H);
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int e = 0; e < kRouteExperts; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[e][q] = __builtin_fmaf(r[e][k], v[q][k], acc[e][q]);
  }
#pragma unroll
  for (int e = 0; e < kRouteExperts; ++e)
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const float s = wave_fold_sum(acc[e][q]);
      if (lane == 0) red[wave][e * NT + q] = s;
    }
  __syncthreads();
  if (threadIdx.x < kRouteExperts * NT) {
    const int e = threadIdx.x / NT, q = threadIdx.x % NT;
    float l = 0.0f;
#pragma unroll
    for (int v = 0; v < kRouteWaves; ++v) l += red[v][threadIdx.x];
    if (e0 + e < a.experts && q < nt) put_shared(&w.logits[(int64_t)(t0 + q) * a.experts + e0 + e], l);
  }
  if (!last_to_finish(&w.counters[1 + blockIdx.y], blocks)) return;
  for (int q = wave; q < nt; q += kRouteWaves) pick_experts(a, w, t0 + q, own_ids + q * a.top_k);
  if (gridDim.y == 1) {
    __syncthreads();
    sort_pairs(a, w, own_ids);
  } else if (last_to_finish(&w.counters[0], (int)gridDim.y)) {
    sort_pairs(a, w, nullptr);
  }
}

// Columns staged in LDS as FP16: rows of `pitch` bytes and one run of zeros for the lanes
// without a token. Nothing of them is loaded in the loop over K, whose only loads are the weights'.
constexpr int kZeroBytes = 2 * kRun<kAligned>;
constexpr int kChunk = 4096;                                  // elements of K staged at a time
struct TokensLds {
  struct Raw {};
  typedef Raw Cur;
  const uint8_t* at;                                          // of the lane's row
  uint32_t k0, K, mask;                                       // first element staged; 0 for the zeros
  __device__ __forceinline__ Raw load(int, uint32_t) const { return Raw{}; }
  __device__ __forceinline__ Cur cook(int, const Raw& r, uint32_t) const { return r; }
  __device__ __forceinline__ half8 octet(const Cur&, uint32_t k, int t) const {
    // past K the weights' scales are zero, and what LDS holds there is finite
    return *reinterpret_cast<const half8*>(at + ((2 * (k - k0)) & mask) + 16 * t);
  }
};

// y[t][n], y[t][n + 1] of the tokens t = first, first + step, ...: the routed experts' parts added in order,
// the loads of two tokens' eight experts in flight together.
__device__ __forceinline__ void join_pairs(const MoeArgs& a, const MoeWork& w, int64_t n, int first, int step) {
  const int64_t N = a.hidden;
  if (n >= N) return;
  for (int t0 = first; t0 < a.tokens; t0 += 2 * step) {
    const int t1 = t0 + step < a.tokens ? t0 + step : t0;
    float lo[2] = {}, hi[2] = {};
    for (int j0 = 0; j0 < a.top_k; j0 += 8) {
      uint64_t v[2][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int jj = j0 + j < a.top_k ? j0 + j : j0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[i][j] = get_shared(reinterpret_cast<const uint64_t*>(w.part + ((int64_t)(i ? t1 : t0) * a.top_k + jj) * N + n));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j < a.top_k) {                               // uniform
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            lo[i] += __uint_as_float((uint32_t)v[i][j]);
            hi[i] += __uint_as_float((uint32_t)(v[i][j] >> 32));
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + i * step;
      if (t < a.tokens) {
        uint16_t* y = a.y + (int64_t)t * a.ldy + n;
        const uint32_t b = bf16_rn_pair(lo[i], hi[i]);
        y[0] = (uint16_t)b;
        y[1] = (uint16_t)(b >> 16);
      }
    }
  }
}

// 16 R weight rows of one used expert times its tokens, kCols at a time (the weights' second and
// later readings come from the cache). Grid: used experts (as many as there can be; the surplus
// leaves at once) x row tiles, tiles of one expert next to each other.
// UP: rows of W1, K = hidden -> h[pair][f]. GATED: fragments 0 .. R/2 - 1 hold the gate's rows, the
// others the same rows of U. DOWN: rows of W2, K = ffn -> part[pair][n], then y.
// kCols: columns staged at a time (8, or 1 for one token). A: steps in flight.
// JOIN: the last workgroup of a row tile writes y.
// The waves split K, the same number of them whatever the batch: the order of a token's sums, and so its
// result, does not depend on how many tokens there are.
constexpr int kWaves = 4, kThreads = 64 * kWaves;
template <bool UP, bool GATED, int R, int A, int kCols, bool JOIN, Shape S>
__global__ __launch_bounds__(kThreads) void k_expert(MoeArgs a, MoeWork w, int tiles, uint32_t pitch) {
  static_assert(!GATED || R % 2 == 0, "a gated tile holds as many gate as up fragments");
  static_assert(R <= kWaves, "a wave per fragment of output rows");
  constexpr int RO = GATED ? R / 2 : R;                       // fragments of output rows
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  float* red = reinterpret_cast<float*>(lds);                 // kWaves R fragments
  uint8_t* const zeros = lds + kWaves * R * 64 * 16;          // a run's worth
  uint8_t* const tokens = zeros + kZeroBytes;                 // kCols rows of pitch bytes
  const int u = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  // one round trip for all of the routing that does not depend on more of it (slots past the
  // count hold anything and are not followed; the count is 0 past the used experts)
  int mine = w.order[u * (int)kMoeMaxTokens + (r & (kCols - 1))];
  const int e = w.expert[u], count = w.count[u];
  if (count == 0) return;
  const int64_t K = UP ? a.hidden : a.ffn, N = UP ? a.ffn : a.hidden;
  const int64_t n0 = (int64_t)tile * (16 * RO);
  const GemmOperand& m = UP ? a.w1 : a.w2;
  const int64_t rows = GATED ? 2 * N : N;                     // of one expert
  const Matrix weights(m.codes + e * rows * (K >> 1), m.scales + e * rows * (K >> 4), rows, K);
  uint32_t row[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t n = n0 + 16 * (i % RO) + r;
    row[i] = (uint32_t)((i >= RO ? N : 0) + (n < N ? n : n0));      // rows past N: not stored
  }
  if (threadIdx.x < kZeroBytes / 4) reinterpret_cast<uint32_t*>(zeros)[threadIdx.x] = 0u;
  const float gs = m.global_scale[e];
  for (int q0 = 0; q0 < count; q0 += kCols) {
    const int nc = count - q0 < kCols ? count - q0 : kCols;   // columns of this round
    if (q0 > 0) mine = w.order[u * (int)kMoeMaxTokens + q0 + (r < nc ? r : 0)];
    const bool live = r < nc;
    const int pair = __shfl(mine, live ? r : 0);              // dead lanes: column 0's
    float4v acc[R][1];
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i][0] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    float inv = 1.0f;                                         // undoes the column's power of two (exact)
    float weight = 1.0f;                                      // DOWN: the pair's
    float scale = 1.0f;                                       // DOWN: the column's, in the lanes of row c
    Pipe<R, 1, A, S, TokensLds> pipe;
    for (int64_t k0 = 0; k0 < K; k0 += kChunk) {
      const int64_t len = K - k0 < kChunk ? K - k0 : kChunk;
      const int first = (int)(k0 / kStep<S>) + wave;
      TokensLds tok{live ? tokens + r * pitch : zeros, (uint32_t)k0, (uint32_t)K, live ? 0xFFFFFFFFu : 0u};
      // The columns' elements, 8 at a time, zeros up to a whole step; column c's pair is in lane c of
      // every wave. The first turn's loads (all of them, as a rule) are issued ahead of the weights', so
      // that waiting for them does not wait for those.
      const int octets = (int)((len + kStep<S> - 1) / kStep<S>) * (kStep<S> / 8);
      half8 v[kCols];
      float vs[kCols];                                        // DOWN: maxima of the elements' fragments
      auto fetch = [&](int o) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          v[c] = half8{};
          vs[c] = 0.0f;
          if (c < nc && 8 * o < len) {
            const int p = __builtin_amdgcn_readlane(pair, c);
            if constexpr (UP) {
              v[c] = *reinterpret_cast<const half8*>(w.x16 + (int64_t)(p / a.top_k) * K + k0 + 8 * o);
            } else {
              v[c] = *reinterpret_cast<const half8*>(w.h + (int64_t)p * K + k0 + 8 * o);
              vs[c] = w.h_top[(int64_t)p * (K / 16) + (k0 + 8 * o) / 16];
            }
          }
        }
      };
      float top[kCols];
      if (k0 == 0) {
        if constexpr (UP) {
          inv = w.x_inv[pair / a.top_k];
        } else {
          weight = w.weights[pair];
          const int frags = (int)(K / 16);
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            top[c] = 0.0f;
            if (c < nc) {
              const float* t = w.h_top + (int64_t)__builtin_amdgcn_readlane(pair, c) * frags;
              const float t0 = t[lane < frags ? lane : 0], t1 = t[lane + 64 < frags ? lane + 64 : 0];
              top[c] = fmaxf(t0, t1);
              for (int i = lane + 128; i < frags; i += 64) top[c] = fmaxf(top[c], t[i]);
            }
          }
        }
      }
      fetch(threadIdx.x);
      pipe.start(weights, row, tok, first, kWaves);
      if constexpr (!UP) {
        if (k0 == 0) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            if (c < nc) {
              const float s = half_scale(wave_fold_max(top[c]));
              scale = r == c ? s : scale;
            }
          }
          inv = 1.0f / scale;
        }
      }
      if (k0 > 0 || q0 > 0) __syncthreads();                  // the columns staged before have been read
      for (int o = threadIdx.x; o < octets; o += kThreads) {
        if (o >= kThreads) fetch(o);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          if (c < nc) {
            if constexpr (!UP) {                              // from the fragment's scale to the column's
              const float f = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(scale), c)) /
                              half_scale(vs[c]);              // both powers of two: exact
#pragma unroll
              for (int q = 0; q < 8; ++q) v[c][q] = (_Float16)((float)v[c][q] * f);
            }
            *reinterpret_cast<half8*>(tokens + c * pitch + 16 * o) = v[c];
          }
        }
      }
      __syncthreads();
      pipe.run(weights, row, tok, first, kWaves, (int)((k0 + len + kStep<S> - 1) / kStep<S>), acc);
    }
    put<R, 1>(red, wave, acc);
    __syncthreads();
    if (wave < RO) {                                          // a wave per fragment of output rows
      const int64_t n = n0 + 16 * wave + 4 * g;               // N % 16 == 0: all four rows or none
      const float f = gs * weight;                            // (times inv it can be too small for FP32 where v f inv is not)
      float4v v = take<kWaves, R, 1>(red, wave, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = v[q] * f * inv;
      if constexpr (UP) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = act_of(a.act, v[q]);
        if constexpr (GATED) {
          const float4v up = take<kWaves, R, 1>(red, wave + RO, 0);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] *= up[q] * f * inv;
        }
        // this fragment's maximum; NaN is dropped by it and stays in h, an infinite one gives scale 1
        float top = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) top = fmaxf(top, fabsf(v[q]));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float s = half_scale(top);
        if (live && n < N) {
          typedef _Float16 half4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<half4*>(w.h + (int64_t)pair * N + n) =
              half4{(_Float16)(v[0] * s), (_Float16)(v[1] * s), (_Float16)(v[2] * s), (_Float16)(v[3] * s)};
          if (g == 0) w.h_top[(int64_t)pair * (N / 16) + n / 16] = top;
        }
      } else if (live && n < N) {
        uint64_t* out = reinterpret_cast<uint64_t*>(w.part + (int64_t)pair * N + n);
        if constexpr (!JOIN) *reinterpret_cast<float4v*>(out) = v;
        else put_shared(out, (uint64_t)__float_as_uint(v[0]) | (uint64_t)__float_as_uint(v[1]) << 32);
        if constexpr (JOIN) put_shared(out + 1, (uint64_t)__float_as_uint(v[2]) | (uint64_t)__float_as_uint(v[3]) << 32);
      }
    }
    // (the next round's first barrier, after its pipe.start, keeps put from overtaking take)
  }
  if constexpr (JOIN) {
    if (!last_to_finish(&w.counters[1 + kMoeMaxTokens / kGroupTokens + tile], *w.used)) return;
    constexpr int kPairs = 8 * R;
    join_pairs(a, w, n0 + threadIdx.x % kPairs * 2, threadIdx.x / kPairs, kThreads / kPairs);
  }
}

// y after a k_expert<DOWN> that left the joining to a launch of its own: 64 rows x 8 tokens a workgroup.
__global__ __launch_bounds__(256) void k_join(MoeArgs a, MoeWork w) {
  join_pairs(a, w, (int64_t)blockIdx.x * 64 + threadIdx.x % 32 * 2, (int)blockIdx.y * 8 + (int)threadIdx.x / 32, 64);
}

constexpr int kJoinTokens = 4;                                // up to here k_expert<DOWN> writes y itself
constexpr int kMostCols = 8;                                  // tokens of an expert at a time
constexpr int kMostLds = kWaves * 4 * 64 * 16 + kZeroBytes + kMostCols * (2 * kChunk + 16);

int64_t tiles_of(int64_t rows, int frags) { return (rows + 16 * frags - 1) / (16 * frags); }

template <bool UP, bool GATED, int R, int A, int COLS, bool JOIN, Shape S>
hipError_t launch_expert_as(const MoeArgs& a, const MoeWork& w, hipStream_t stream) {
  // the staged columns can take more LDS than a launch may by default
  static const hipError_t ready = hipFuncSetAttribute((const void*)k_expert<UP, GATED, R, A, COLS, JOIN, S>,
                                                      hipFuncAttributeMaxDynamicSharedMemorySize, kMostLds);
  if (ready != hipSuccess) return ready;
  const int64_t K = UP ? a.hidden : a.ffn, N = UP ? a.ffn : a.hidden;
  const int64_t pairs = (int64_t)a.tokens * a.top_k;
  const int64_t most = pairs < a.experts ? pairs : a.experts;
  const int tiles = (int)tiles_of(N, GATED ? R / 2 : R);
  const int64_t staged = K < kChunk ? (K + kStep<S> - 1) / kStep<S> * kStep<S> : kChunk;
  const uint32_t pitch = (uint32_t)(2 * staged + 16);         // rows start 4 banks apart
  const size_t bytes = (size_t)kWaves * R * 64 * 16 + kZeroBytes + (size_t)COLS * pitch;
  hipLaunchKernelGGL((k_expert<UP, GATED, R, A, COLS, JOIN, S>), dim3((unsigned)(most * tiles)), dim3(kThreads), bytes,
                     stream, a, w, tiles, pitch);
  return hipSuccess;
}

template <bool UP, bool GATED, Shape S>
hipError_t launch_expert_k(const MoeArgs& a, const MoeWork& w, hipStream_t stream) {
  // (us on 122 experts of 2688 x 1856, 64 tokens: up R = 2 with A = 1, 2, 3: 95, 95, 93, R = 4: 98; down
  // R = 2: 108 with A = 1, 110 with 2; R = 4: 96 with A = 1, 115 with 2. Few tokens, the whole layer of 128
  // experts, weights from HBM: R = 2 with A = 2, 3, 4: 1 token 27.7, 28.1, 28.5, 4 tokens 59, 65, 70; R = 1:
  // 25.6, 25.6, 25.8 and 68, 69, 69. 8 waves, R = 2, A = 2: 27.1 and 77, but at 64 tokens down 129 to 140)
  constexpr int R = UP ? 2 : 4, A = UP ? 3 : 1;
  if (a.tokens == 1) return launch_expert_as<UP, GATED, GATED ? 2 : 1, 2, 1, !UP, S>(a, w, stream);
  if (a.tokens <= kJoinTokens) return launch_expert_as<UP, GATED, 2, 2, kMostCols, !UP, S>(a, w, stream);
  return launch_expert_as<UP, GATED, R, A, kMostCols, false, S>(a, w, stream);
}

template <bool UP, bool GATED>
hipError_t launch_expert(const MoeArgs& a, const MoeWork& w, hipStream_t stream) {
  return (UP ? a.hidden : a.ffn) % 64 == 0 ? launch_expert_k<UP, GATED, kAligned>(a, w, stream)
                                           : launch_expert_k<UP, GATED, kHalf>(a, w, stream);
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
  x.count = reinterpret_cast<int*>(part(4 * E));
  x.order = reinterpret_cast<int*>(part(4 * (P < E ? P : E) * (size_t)kMoeMaxTokens));
  x.ids = reinterpret_cast<int*>(part(4 * P));
  x.weights = reinterpret_cast<float*>(part(4 * P));
  x.logits = reinterpret_cast<float*>(part(4 * T * E));
  x.x_inv = reinterpret_cast<float*>(part(4 * T));
  x.h_top = reinterpret_cast<float*>(part(4 * P * (size_t)a.ffn / 16));
  x.x16 = reinterpret_cast<_Float16*>(part(2 * T * (size_t)a.hidden));
  x.h = reinterpret_cast<_Float16*>(part(2 * P * (size_t)a.ffn));
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
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % 8 == 0 &&
                   reinterpret_cast<uintptr_t>(a.router) % 16 == 0;        // hidden % 16 == 0
  const dim3 grid((unsigned)((a.experts + kRouteExperts - 1) / kRouteExperts + kGroupTokens),
                  (unsigned)((a.tokens + kGroupTokens - 1) / kGroupTokens));
#define NVFP4_RT(F32, NT, VEC) \
  hipLaunchKernelGGL((k_route<F32, NT, VEC>), grid, dim3(kRouteThreads), 0, stream, a, w)
#define NVFP4_RN(F32, VEC) do { if (a.tokens == 1) NVFP4_RT(F32, 1, VEC); else NVFP4_RT(F32, 8, VEC); } while (0)
  if (vec && a.router_f32) NVFP4_RN(true, true);
  else if (vec) NVFP4_RN(false, true);
  else if (a.router_f32) NVFP4_RN(true, false);
  else NVFP4_RN(false, false);
#undef NVFP4_RN
#undef NVFP4_RT
  hipError_t e = a.gated ? launch_expert<true, true>(a, w, stream) : launch_expert<true, false>(a, w, stream);
  if (e != hipSuccess || (e = launch_expert<false, false>(a, w, stream)) != hipSuccess) return e;
  if (a.tokens > kJoinTokens)
    hipLaunchKernelGGL(k_join, dim3((unsigned)((a.hidden + 63) / 64), (unsigned)((a.tokens + 7) / 8)), dim3(256), 0,
                       stream, a, w);
  return hipGetLastError();
}

}  // namespace nvfp4
