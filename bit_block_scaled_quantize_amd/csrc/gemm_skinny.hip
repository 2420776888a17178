// nvfp4_gemm_act for few rows of A (the tokens of a generation step, a short prompt): D = act(A B^T + bias) +
// residual with B's rows as the matrix instruction's rows and A's rows as its columns (skinny.h).
// Bound by reading B, N K * 9/16 bytes, up to 64 rows; beyond, workgroups on the same rows of B take 64
// rows of A each and find B in the cache.
// Measured: 1 x 20480 x 5120 18.3 us (59 MB, 3.2 TB/s), 1 x 5120 x 5120 7.9; 64 x 5120 x 5120 15.7, where decoding
// is what it does; 1003 x 1857 x 2704 with residual, bias and Z 28 (0.36 PFLOP/s): the decoding again, every
// workgroup's own.
#include "act_out.h"
#include "launch.h"
#include "skinny.h"

namespace nvfp4 {
namespace {

using namespace skinny;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// Columns from NVFP4 rows: decoded like the weights.
template <Shape S>
struct TokensNvfp4 {
  typedef Loaded<S> Raw;
  typedef Run<S> Cur;
  Matrix a;
  uint32_t rows, first;                                       // first: the lane's row of A in the first fragment
  __device__ __forceinline__ Raw load(int c, uint32_t k) const {
    const uint32_t m = 16u * (uint32_t)c + first;
    return load_run<S>(a, m, m < rows, k);
  }
  __device__ __forceinline__ Cur cook(int c, const Raw& x, uint32_t k) const {
    const uint32_t m = 16u * (uint32_t)c + first;
    return run_of(x, a, m, m < rows, k);
  }
  __device__ __forceinline__ half8 octet(const Cur& x, uint32_t, int t) const { return octet_of(x, t); }
};

template <int R, int C, Shape S>
__global__ __launch_bounds__(kThreads) void k_gemm_skinny(GemmOperand A, GemmOperand B, int64_t M, int64_t N,
                                                          int64_t K, int act, ActOut out, uint16_t* __restrict__ D,
                                                          int64_t ldd, float* __restrict__ amax) {
  __shared__ __attribute__((aligned(16))) float red[kWaves * R * C * 64 * 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R), m0 = (int64_t)blockIdx.y * (16 * C);
  const Matrix weights(B.codes, B.scales, N, K);
  uint32_t row[R];
#pragma unroll
  for (int i = 0; i < R; ++i) row[i] = (uint32_t)(n0 + 16 * i + r < N ? n0 + 16 * i + r : n0);   // rows past N: not stored
  const TokensNvfp4<S> tok{Matrix(A.codes, A.scales, M, K), (uint32_t)M, (uint32_t)(m0 + r)};
  float4v acc[R][C];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[i][c] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
  // (one step ahead is enough, and better, where four column fragments' arithmetic covers it)
  Pipe<R, C, C == 4 ? 1 : 2, S, TokensNvfp4<S>> pipe;
  pipe.start(weights, row, tok, wave, kWaves);
  pipe.run(weights, row, tok, wave, kWaves, (int)((K + kStep<S> - 1) / kStep<S>), acc);
  put<R, C>(red, wave, acc);
  // Fragment f = kPer wave + j of the R C, rows first, so that a wave's fragments are neighbours in a
  // row of D: a lane has four consecutive columns of one row of each, moved as one vector wherever the
  // row starts. Bias and residual are asked for ahead of the barrier.
  constexpr int kPer = (R * C + kWaves - 1) / kWaves;
  float bias[kPer][4];
  v2u32 res[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int f = wave * kPer + j;
    const int64_t m = m0 + 16 * (f / R) + r, n = n0 + 16 * (f % R) + 4 * g;
    const bool in = f < R * C && m < M && n + 4 <= N;
    res[j] = v2u32{0, 0};
    if (in && out.residual != nullptr) res[j] = *reinterpret_cast<const v2u32_any*>(out.residual + m * out.ldr + n);
#pragma unroll
    for (int q = 0; q < 4; ++q) bias[j][q] = in ? bias_at(out, n + q) : 0.0f;
  }
  __syncthreads();
  const float alpha = A.global_scale[0] * B.global_scale[0];
  float mx = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int f = wave * kPer + j;
    if (f < R * C) {                                          // uniform
      float4v v = take<kWaves, R, C>(red, f % R, f / R);
      const int64_t m = m0 + 16 * (f / R) + r, n = n0 + 16 * (f % R) + 4 * g;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] *= alpha;
      if (m < M && n + 4 <= N) {
        mx = fmaxf(mx, put_act4_of(act, out, D, ldd, m, n, v, bias[j], res[j]));
      } else if (m < M) {                                     // the last columns of an N that is not a multiple of 4
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < N) mx = fmaxf(mx, put_act_of(act, out, D, ldd, m, n + q, v[q]));
      }
    }
  }
  if (amax != nullptr && wave * kPer < R * C) {                      // uniform
    mx = wave_fold_max(mx);
    if (lane == 0) atomic_raise_nonneg(amax, mx);
  }
}

template <int R, int C, Shape S>
void launch_as(const GemmOperand& a, const GemmOperand& b, int64_t M, int64_t N, int64_t K, int act, const ActOut& out,
               uint16_t* D, int64_t ldd, float* amax, hipStream_t stream) {
  const dim3 grid((unsigned)((N + 16 * R - 1) / (16 * R)), (unsigned)((M + 16 * C - 1) / (16 * C)));
  hipLaunchKernelGGL((k_gemm_skinny<R, C, S>), grid, dim3(kThreads), 0, stream, a, b, M, N, K, act, out, D, ldd, amax);
}

}  // namespace

// Workgroups of 32 columns and 64 rows that the product makes.
int64_t few_row_blocks(int64_t M, int64_t N) { return (M + 63) / 64 * ((N + 31) / 32); }

// Up to 64 rows always; beyond by the number of workgroups, to which this kernel's time is
// proportional. The tile kernel takes 256 x 256 tiles one to a CU: its time hardly depends on their
// number up to a round; up to a quarter of the CUs it cuts them into column quarters, beyond it splits K, whose
// joining costs some 25 us. Measured, us (this kernel / tiles), 64 tiles or fewer: 512 x 5120 (1280
// workgroups): K 1088 20 / 20, 5120 52 / 54; 1500 x 1857 x 2688 (1416) 29 / 32; 1536 x 2048 (1536): K 1088 20 / 20, 5120
// 54 / 57; 768 x 5120 (1920): K 1088 24 / 21, 5120 68 / 60. More tiles: 1024 x 5120 (2560): K 320 23 / 40, 2688
// 42 / 60, 5120 83 / 82, 20480 281 / 229; 1536 x 5120 (3840): K 1088 42 / 54, 5120 124 / 96. For a K that is not a
// multiple of 64 that kernel has its operands copied first: 1003 x 5120, K 5136 84 / 98, 8208 118 / 128 (6144
// 107 / 101, 8192 127 / 116).
bool gemm_act_few_rows(int64_t M, int64_t N, int64_t K) {
  if (K == 0) return false;
  if (M <= 64) return true;
  const int64_t tiles = (M + 255) / 256 * ((N + 255) / 256);
  return few_row_blocks(M, N) <= (tiles <= 64 ? 1536 : K <= (K % 64 == 0 ? 5120 : 10240) ? 2560 : 1280);
}

hipError_t launch_gemm_skinny(GemmOperand a, GemmOperand b, int64_t M, int64_t N, int64_t K, int act, const ActOut& out,
                              uint16_t* D, int64_t ldd, float* amax, hipStream_t stream) {
#define NVFP4_SK(R, C)                                                                   \
  (K % 64 == 0 ? launch_as<R, C, kAligned>(a, b, M, N, K, act, out, D, ldd, amax, stream) \
   : K > 64    ? launch_as<R, C, kWord>(a, b, M, N, K, act, out, D, ldd, amax, stream)    \
               : launch_as<R, C, kHalf>(a, b, M, N, K, act, out, D, ldd, amax, stream))
  if (M <= 16) NVFP4_SK(2, 1);
  else if (M <= 32) NVFP4_SK(2, 2);
  else if (few_row_blocks(M, N) <= 640) NVFP4_SK(2, 4);       // 64 columns halve the decoding of A, and the workgroups:
  else NVFP4_SK(4, 4);                                        // 5120 x 5120, 256 rows 40 / 40 us, 512 63 / 56
#undef NVFP4_SK
  return hipGetLastError();
}

}  // namespace nvfp4
