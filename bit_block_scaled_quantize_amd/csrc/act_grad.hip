// The backward of a linear layer's activation and bias from one read of the output gradient:
//   dZ = dY * act'(Z) (stored in BF16),  dbias[n] = sum over m of dZ[m, n] (FP32, before the rounding)
// and with act none dbias alone (dZ is dY).
//
// Memory bound: 2 or 4 bytes (dY) + 2 (Z) + 2 (dZ) per element against some 15 vector operations.
// 8192 x 20480, BF16 dY: relu2 204 us (4.9 TB/s), gelu 209, none 144; rows of 19858, which start anywhere:
// 8021 of them 225 (4.3 TB/s).
// A workgroup takes COLS columns and a run of rows, COLS / 8 threads to a row: four rows at a time with 512
// columns, 32 with 64. A thread keeps 8 columns' sums in registers. The rows' sums meet in LDS, the row
// runs' sums in the workspace (or go straight to dbias where one run covers all rows), both added in a
// fixed order, so the sums do not change from run to run.
#include <type_traits>

#include "activation.h"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWide = 512, kNarrow = 64;                      // columns of a workgroup
constexpr int kWaves = kThreads / 64;

// Eight columns of a row as they are loaded, whole vectors from wherever the row starts.
template <bool F32>
struct Eight {
  v4u32 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Eight<F32> load_eight(const void* p, int64_t at) {
  Eight<F32> e;
  const uint8_t* b = static_cast<const uint8_t*>(p) + at * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) e.w[i] = *reinterpret_cast<const v4u32_any*>(b + 16 * i);
  return e;
}
// The same one by one, zeros past the first `left`: rows shorter than eight.
template <bool F32>
__device__ __forceinline__ Eight<F32> load_few(const void* p, int64_t at, int left) {
  Eight<F32> e = {};
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (q < left) {
      if constexpr (F32) e.w[q >> 2][q & 3] = static_cast<const uint32_t*>(p)[at + q];
      else e.w[0][q >> 1] |= (uint32_t)static_cast<const uint16_t*>(p)[at + q] << (16 * (q & 1));
    }
  }
  return e;
}
template <bool F32>
__device__ __forceinline__ float element(const Eight<F32>& e, int q) {
  if constexpr (F32) return __uint_as_float(e.w[q >> 2][q & 3]);
  else return q & 1 ? bf16_hi(e.w[0][q >> 1]) : bf16_lo(e.w[0][q >> 1]);
}

template <int ACT, bool F32, int COLS>
__global__ __launch_bounds__(kThreads) void k_act_grad(const void* __restrict__ dy, int64_t ldy,
                                                       const uint16_t* __restrict__ z, int64_t ldz,
                                                       uint16_t* __restrict__ dz, int64_t lddz, int64_t M, int64_t N,
                                                       int64_t rows, float* __restrict__ sums, int accumulate) {
  constexpr int kLanes = COLS / 8, kRows = kThreads / kLanes; // threads of a row, rows at a time
  constexpr int kBatch = 4;                                   // rows of a thread loaded together
  __shared__ float red[kRows][COLS];
  const int lane = threadIdx.x % kLanes;
  const int slot = kLanes == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes) : threadIdx.x / kLanes;
  const int64_t c0 = (int64_t)blockIdx.x * COLS;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = r0 + rows < M ? r0 + rows : M;
  float sum[8] = {};
  const int64_t c = c0 + lane * 8;
  // The last columns of an N that is not a multiple of 8 are read as the eight that end there, and the
  // `skip` first of those, a neighbour's, left alone: one walk for all lanes of a wave, which otherwise
  // takes the rows twice.
  const int64_t at = c + 8 <= N || N < 8 ? c : N - 8;
  const int skip = (int)(c - at);
  auto walk = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;            // N >= 8
    const int left = (int)(N - c);
    for (int64_t r = r0 + slot; r < r1; r += kBatch * kRows) {
      Eight<F32> gv[kBatch];
      Eight<false> xv[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int64_t rb = r + b * kRows < r1 ? r + b * kRows : r;       // past the run: not used
        if constexpr (WHOLE) gv[b] = load_eight<F32>(dy, rb * ldy + at);
        else gv[b] = load_few<F32>(dy, rb * ldy + at, left);
        if constexpr (ACT != kActNone) {
          if constexpr (WHOLE) xv[b] = load_eight<false>(z, rb * ldz + at);
          else xv[b] = load_few<false>(z, rb * ldz + at, left);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (r + b * kRows >= r1) break;
        float g[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          g[q] = element(gv[b], q);
          if constexpr (ACT != kActNone) g[q] *= act_slope<ACT>(element(xv[b], q));
          sum[q] += g[q];
        }
        if (dz != nullptr) {
          const v4u32 w = {bf16_rn_pair(g[0], g[1]), bf16_rn_pair(g[2], g[3]), bf16_rn_pair(g[4], g[5]),
                           bf16_rn_pair(g[6], g[7])};
          uint16_t* out = dz + (r + b * kRows) * lddz + at;
          if (WHOLE && skip == 0) {
            *reinterpret_cast<v4u32_any*>(out) = w;
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q >= skip && (WHOLE || q < left)) out[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
          }
        }
      }
    }
  };
  if (c < N) {
    if (N >= 8) walk(std::true_type{});                       // uniform
    else walk(std::false_type{});
  }
  if (sums == nullptr) return;                                // uniform
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (c < N && q >= skip) red[slot][(int)(at - c0) + q] = sum[q];
  __syncthreads();
  for (int i = threadIdx.x; i < COLS; i += kThreads) {
    if (c0 + i < N) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < kRows; j += 2) s += red[j][i] + red[j + 1][i];
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
  const int64_t blocks = (N + kWide - 1) / kWide;
  int64_t runs = 2048 / blocks;
  runs = runs < (M + 7) / 8 ? runs : (M + 7) / 8;
  runs = runs < 256 ? runs : 256;
  return runs < 1 ? 1 : runs;
}

// Few rows: narrow workgroups, each over all of them, and one launch instead of two (us, narrow / wide, gelu,
// BF16 of 5120 columns: 8 rows 3.3 / 4.0, 32 3.4 / 6.0, 123 5.2 / 7.1, 256 7.9 / 6.8, 512 13 / 8.5; of 1857: 123
// 7.0 / 7.1, 256 11 / 6.5).
constexpr int64_t kNarrowRows = 128;

int64_t rows_per_run(int64_t M, int64_t N) {
  if (M <= kNarrowRows) return M;
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
  const int64_t cols = M <= kNarrowRows ? kNarrow : kWide;
  const dim3 grid((unsigned)((N + cols - 1) / cols), (unsigned)runs);
#define NVFP4_AG3(A, F, C) \
  hipLaunchKernelGGL((k_act_grad<A, F, C>), grid, dim3(kThreads), 0, stream, dy, ldy, z, ldz, dz, lddz, M, N, rows, sums, add)
#define NVFP4_AG2(A, F) do { if (cols == kNarrow) NVFP4_AG3(A, F, kNarrow); else NVFP4_AG3(A, F, kWide); } while (0)
#define NVFP4_AG(A) do { if (fp32) NVFP4_AG2(A, true); else NVFP4_AG2(A, false); } while (0)
  switch (act) {
    case kActRelu2: NVFP4_AG(kActRelu2); break;
    case kActGelu: NVFP4_AG(kActGelu); break;
    case kActSilu: NVFP4_AG(kActSilu); break;
    default: NVFP4_AG(kActNone); break;
  }
#undef NVFP4_AG
#undef NVFP4_AG2
#undef NVFP4_AG3
  if (dbias && runs > 1)
    hipLaunchKernelGGL(k_column_sums, dim3((unsigned)((N + 63) / 64)), dim3(kThreads), 0, stream, ws, runs, N, dbias,
                       accumulate ? 1 : 0);
  return hipGetLastError();
}

}  // namespace nvfp4
