// nvfp4_gemm_act for few rows of A (the tokens of a generation step, a short prompt): D = act(A B^T + bias) +
// residual with B's rows as the matrix instruction's rows and A's rows as its columns (skinny.h).
// Bound by reading B, N K * 9/16 bytes, up to 64 rows; beyond, workgroups on the same rows of B take 64
// rows of A each and find B in the cache.
#include "act_out.h"
#include "launch.h"
#include "skinny.h"

namespace nvfp4 {
namespace {

using namespace skinny;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// Columns from NVFP4 rows: decoded like the weights.
template <int C, bool K64>
struct TokensNvfp4 {
  typedef Run<K64> Raw;
  Matrix a;
  uint32_t rows, first;                                       // first: the lane's row of A in the first fragment
  __device__ __forceinline__ Raw load(int c, uint32_t k) const {
    const uint32_t m = 16u * (uint32_t)c + first;
    return load_run<K64>(a, m, m < rows, k);
  }
  __device__ __forceinline__ half8 octet(const Raw& x, uint32_t, int t) const { return octet_of(x, t); }
};

template <int R, int C, bool K64>
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
  const TokensNvfp4<C, K64> tok{Matrix(A.codes, A.scales, M, K), (uint32_t)M, (uint32_t)(m0 + r)};
  float4v acc[R][C];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[i][c] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
  // (one step ahead is enough, and better, where four column fragments' arithmetic covers it)
  Pipe<R, C, C == 4 ? 1 : 2, K64, TokensNvfp4<C, K64>> pipe;
  pipe.start(weights, row, tok, wave, kWaves);
  pipe.run(weights, row, tok, wave, kWaves, (int)((K + kStep<K64> - 1) / kStep<K64>), acc);
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

template <int R, int C>
void launch_rc(const GemmOperand& a, const GemmOperand& b, int64_t M, int64_t N, int64_t K, int act, const ActOut& out,
               uint16_t* D, int64_t ldd, float* amax, hipStream_t stream) {
  const dim3 grid((unsigned)((N + 16 * R - 1) / (16 * R)), (unsigned)((M + 16 * C - 1) / (16 * C)));
  if (K % 64 == 0)
    hipLaunchKernelGGL((k_gemm_skinny<R, C, true>), grid, dim3(kThreads), 0, stream, a, b, M, N, K, act, out, D, ldd, amax);
  else
    hipLaunchKernelGGL((k_gemm_skinny<R, C, false>), grid, dim3(kThreads), 0, stream, a, b, M, N, K, act, out, D, ldd, amax);
}

}  // namespace

// Workgroups of 32 columns and 64 rows that the product makes.
int64_t few_row_blocks(int64_t M, int64_t N) { return (M + 63) / 64 * ((N + 31) / 32); }

// Up to 64 rows always; beyond by the number of workgroups: the tile kernel takes whole rounds of
// 256 x 256 tiles (or quarters of them), so its time hardly depends on them below a round, and this
// kernel's is proportional to them. Measured, us (this kernel / tiles): 5120 x 5120: 256 rows (640
// workgroups) 40 / 51, 512 (1280) 56 / 54, 1024 (2560) 88 / 83; 20480 x 5120: 128 (1280) 56 / 78, 256
// (2560) 89 / 82; 1856 x 2688: 1024 (928) 23 / 32. A K that is not a multiple of 64 (runs of 32 here,
// copied operands there): 1857 x 2704: 1003 (944) 33 / 42; 5120 x 5136: 512 (1280) 85 / 71.
bool gemm_act_few_rows(int64_t M, int64_t N, int64_t K) {
  if (K == 0) return false;
  return M <= 64 || few_row_blocks(M, N) <= (K % 64 == 0 ? 1280 : 960);
}

hipError_t launch_gemm_skinny(GemmOperand a, GemmOperand b, int64_t M, int64_t N, int64_t K, int act, const ActOut& out,
                              uint16_t* D, int64_t ldd, float* amax, hipStream_t stream) {
#define NVFP4_SK(R, C) launch_rc<R, C>(a, b, M, N, K, act, out, D, ldd, amax, stream)
  if (M <= 16) NVFP4_SK(2, 1);
  else if (M <= 32) NVFP4_SK(2, 2);
  else if (few_row_blocks(M, N) <= 640) NVFP4_SK(2, 4);       // 64 columns halve the decoding of A, and the workgroups:
  else NVFP4_SK(4, 4);                                        // 5120 x 5120, 256 rows 40 / 40 us, 512 63 / 56
#undef NVFP4_SK
  return hipGetLastError();
}

}  // namespace nvfp4
