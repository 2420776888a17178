// The backward of a linear layer's activation and bias from one read of the output gradient:
//   dZ = dY * act'(Z) (stored in BF16),  dbias[n] = sum over m of dZ[m, n] (FP32, before the rounding)
// and with act none dbias alone (dZ is dY).
//
// Memory bound: 2 or 4 bytes (dY) + 2 (Z) + 2 (dZ) per element against some 15 vector operations.
// A workgroup takes 512 columns and a run of rows, its four waves every fourth row; a thread
// keeps 8 columns' sums in registers. The waves' sums meet in LDS, the row runs' sums in the
// workspace (or go straight to dbias where one run covers all rows), both added in a fixed
// order, so the sums do not change from run to run.
#include <type_traits>

#include "activation.h"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 512;                                    // 64 lanes x 8
constexpr int kWaves = kThreads / 64;

// Eight consecutive columns of a row, WHOLE: as whole vectors from wherever the row starts; else the
// last `left` < 8 columns of a row one by one, 0 past them.
template <bool F32, bool WHOLE>
__device__ __forceinline__ void load_row(const void* p, int64_t at, int left, float (&v)[8]) {
  if constexpr (WHOLE && F32) {
    const float* f = static_cast<const float*>(p) + at;
    const v4f32 a = *reinterpret_cast<const v4f32_any*>(f), b = *reinterpret_cast<const v4f32_any*>(f + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = a[q];
      v[q + 4] = b[q];
    }
  } else if constexpr (WHOLE) {
    const v4u32 w = *reinterpret_cast<const v4u32_any*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = bf16_lo(w[q]);
      v[2 * q + 1] = bf16_hi(w[q]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] = 0.0f;
      if (q < left) v[q] = F32 ? static_cast<const float*>(p)[at + q] : bf16_lo(static_cast<const uint16_t*>(p)[at + q]);
    }
  }
}

template <int ACT, bool F32>
__global__ __launch_bounds__(kThreads) void k_act_grad(const void* __restrict__ dy, int64_t ldy,
                                                       const uint16_t* __restrict__ z, int64_t ldz,
                                                       uint16_t* __restrict__ dz, int64_t lddz, int64_t M, int64_t N,
                                                       int64_t rows, float* __restrict__ sums, int accumulate) {
  __shared__ float red[kWaves][kCols];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c0 = (int64_t)blockIdx.x * kCols;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = r0 + rows < M ? r0 + rows : M;
  float sum[8] = {};
  const int64_t c = c0 + lane * 8;
  auto walk = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    const int left = (int)(N - c < 8 ? N - c : 8);
#pragma unroll 4
    for (int64_t r = r0 + wave; r < r1; r += kWaves) {
      float g[8];
      load_row<F32, WHOLE>(dy, r * ldy + c, left, g);
      if constexpr (ACT != kActNone) {
        float x[8];
        load_row<false, WHOLE>(z, r * ldz + c, left, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) g[q] *= act_slope<ACT>(x[q]);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] += g[q];
      if (dz != nullptr) {
        const v4u32 w = {bf16_rn_pair(g[0], g[1]), bf16_rn_pair(g[2], g[3]), bf16_rn_pair(g[4], g[5]),
                         bf16_rn_pair(g[6], g[7])};
        uint16_t* out = dz + r * lddz + c;
        if constexpr (WHOLE) {
          *reinterpret_cast<v4u32_any*>(out) = w;
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < left) out[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
        }
      }
    }
  };
  if (c + 8 <= N) walk(std::true_type{});
  else if (c < N) walk(std::false_type{});
  if (sums == nullptr) return;                                // uniform
#pragma unroll
  for (int q = 0; q < 8; ++q) red[wave][lane * 8 + q] = sum[q];
  __syncthreads();
  for (int i = threadIdx.x; i < kCols; i += kThreads) {
    if (c0 + i < N) {
      const float s = (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
      float* out = sums + (int64_t)blockIdx.y * N + c0 + i;   // with one run of rows: dbias itself
      *out = accumulate ? *out + s : s;
    }
  }
}

// dbias[n] (+)= sum of parts[i][n]: 64 columns a workgroup, wave w the runs w, w + 4, ...
__global__ __launch_bounds__(kThreads) void k_column_sums(const float* __restrict__ parts, int64_t count, int64_t N,
                                                          float* __restrict__ dbias, int accumulate) {
  __shared__ float red[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int64_t i = wave; i < count; i += kWaves) s += parts[i * N + n];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && n < N) {
    const float t = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
    dbias[n] = accumulate ? dbias[n] + t : t;
  }
}

// Runs of rows: about 8 workgroups per CU, at least 8 rows each (two per wave), at most 256 runs.
int64_t row_runs(int64_t M, int64_t N) {
  const int64_t blocks = (N + kCols - 1) / kCols;
  int64_t runs = 2048 / blocks;
  runs = runs < (M + 7) / 8 ? runs : (M + 7) / 8;
  runs = runs < 256 ? runs : 256;
  return runs < 1 ? 1 : runs;
}

int64_t rows_per_run(int64_t M, int64_t N) {
  const int64_t runs = row_runs(M, N);
  return ((M + runs - 1) / runs + kWaves - 1) / kWaves * kWaves;
}

}  // namespace

size_t act_grad_workspace_bytes(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0) return 0;
  const int64_t rows = rows_per_run(M, N), runs = (M + rows - 1) / rows;
  return runs > 1 ? (size_t)runs * (size_t)N * sizeof(float) : 0;
}

hipError_t launch_act_grad(const void* dy, bool fp32, int64_t ldy, const uint16_t* z, int64_t ldz, int act,
                           uint16_t* dz, int64_t lddz, float* dbias, bool accumulate, int64_t M, int64_t N,
                           float* ws, hipStream_t stream) {
  if (N == 0) return hipSuccess;
  if (M == 0) return dbias && !accumulate ? launch_fill(dbias, N, 0.0f, stream) : hipSuccess;
  const int64_t rows = rows_per_run(M, N), runs = (M + rows - 1) / rows;
  float* sums = dbias ? (runs > 1 ? ws : dbias) : nullptr;
  const int add = accumulate && runs == 1;
  const dim3 grid((unsigned)((N + kCols - 1) / kCols), (unsigned)runs);
#define NVFP4_AG2(A, F) \
  hipLaunchKernelGGL((k_act_grad<A, F>), grid, dim3(kThreads), 0, stream, dy, ldy, z, ldz, dz, lddz, M, N, rows, sums, add)
#define NVFP4_AG(A) do { if (fp32) NVFP4_AG2(A, true); else NVFP4_AG2(A, false); } while (0)
  switch (act) {
    case kActRelu2: NVFP4_AG(kActRelu2); break;
    case kActGelu: NVFP4_AG(kActGelu); break;
    case kActSilu: NVFP4_AG(kActSilu); break;
    default: NVFP4_AG(kActNone); break;
  }
#undef NVFP4_AG
#undef NVFP4_AG2
  if (dbias && runs > 1)
    hipLaunchKernelGGL(k_column_sums, dim3((unsigned)((N + 63) / 64)), dim3(kThreads), 0, stream, ws, runs, N, dbias,
                       accumulate ? 1 : 0);
  return hipGetLastError();
}

}  // namespace nvfp4
