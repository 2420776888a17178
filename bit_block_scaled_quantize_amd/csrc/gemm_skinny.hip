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
  Pipe<R, C, 2, K64, TokensNvfp4<C, K64>> pipe;
  pipe.start(weights, row, tok, wave, kWaves);
  pipe.run(weights, row, tok, wave, kWaves, (int)((K + kStep<K64> - 1) / kStep<K64>), acc);
  put<R, C>(red, wave, acc);
  __syncthreads();
  const float alpha = A.global_scale[0] * B.global_scale[0];
  float mx = 0.0f;
#pragma unroll 1
  for (int f = wave; f < R * C; f += kWaves) {
    const int i = f / C, c = f % C;
    const float4v v = take<kWaves, R, C>(red, i, c);
    const int64_t m = m0 + 16 * c + r, n = n0 + 16 * i + 4 * g;
    if (m < M) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < N) mx = fmaxf(mx, put_act_of(act, out, D, ldd, m, n + q, v[q] * alpha));
    }
  }
  if (amax != nullptr && wave < R * C) {                      // uniform
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

// Up to 64 rows always; beyond by the number of workgroups, each worth 64 rows x 32 columns: the tile
// kernel takes whole rounds of 256 x 256 tiles (or quarters of them), so its time hardly depends on
// them below a round, and this kernel's is proportional to them. Measured, us (this kernel / tiles):
// 5120 x 5120: 384 rows (960 workgroups) 52 / 54, 512 (1280) 66 / 54; 5120 x 20480: 384 (960) 170 / 190,
// 512 (1280) 212 / 188; 2688 x 1856: 768 (1008) 23 / 26, 1024 (1344) 32 / 27. With a K that is not a
// multiple of 64 (runs of 32 here, copied operands there), 5120 x 5136: 256 (640) 59 / 71, 512 (1280)
// 96 / 71; 1857 x 2704: 512 (472) 25 / 40, 1003 (944) 42 / 42.
bool gemm_act_few_rows(int64_t M, int64_t N, int64_t K) {
  if (K == 0) return false;
  return M <= 64 || (M + 63) / 64 * ((N + 31) / 32) <= (K % 64 == 0 ? 1024 : 768);
}

hipError_t launch_gemm_skinny(GemmOperand a, GemmOperand b, int64_t M, int64_t N, int64_t K, int act, const ActOut& out,
                              uint16_t* D, int64_t ldd, float* amax, hipStream_t stream) {
#define NVFP4_SK(R, C) launch_rc<R, C>(a, b, M, N, K, act, out, D, ldd, amax, stream)
  if (M <= 16) NVFP4_SK(2, 1);
  else if (M <= 32) NVFP4_SK(2, 2);
  else NVFP4_SK(2, 4);
#undef NVFP4_SK
  return hipGetLastError();
}

}  // namespace nvfp4
