// The tokens' way to the experts of the grouped GEMMs and back, for batches of any size:
//   sort      pairs p = t k + j (token t's j-th expert) ordered by expert, by p within one; each expert's run of
//             rows starts at a multiple of `align` and ends with rows that hold no pair
//   gather    xs[row] = x[t] (times a weight), zeros in the rows without a pair
//   combine   out[t] = sum over j of w[t, j] y[row of (t, j)], in the order of j
//   gradient  dy[row] = w dout[t];  dw[t, j] = <dout[t], y[row]>
// The gradient of gather is combine without weights, that of combine with respect to y is gather with them (here
// from the same read as dw). Pairs whose expert is out of range have no row and add nothing.
//
// Sort: a counting sort, so stable without a sort of its own: the pairs are cut into chunks of 4096, (1) every chunk
// counts its experts, (2) every chunk adds up the counts, which gives it its first row of every expert, and places its
// pairs; the rows without a pair are marked on the side. Latency, not bytes: 98304 pairs are 0.4 MB. A batch of one chunk takes
// one launch; where all counts are too many for every workgroup to add up, one workgroup does it in a launch between
// the two.
// Gather, combine, gradient: memory bound. 16384 tokens, 6 of 128 experts, hidden 2688: sorted in 12 us, gathered in 152 (629 MB,
// 4.1 TB/s), combined in 225 us (FP32, 1.15 GB, 5.1 TB/s), the gradient in 333 (1.69 GB, 5.1 TB/s).
#include "eight.h"
#include "launch.h"
#include "moe_layout.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;         // of the kernels over rows
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kPer = 4;                                       // pairs of a thread
constexpr int kChunk = kPer * kSortThreads;                   // wave w takes 256 after each other, 64 at a time
// Up to this many chunks every workgroup adds the counts up by itself (24 chunks of 128 experts: 12 us, with a scan between
// 16; 512 of 1024: 98 and 103), from there a launch between does it (1024 of 128: 53 us, without 69): all workgroups of
// the former run at once.
constexpr int64_t kChunksEach = 512;

__device__ __forceinline__ bool valid(int id, int experts) { return (uint32_t)id < (uint32_t)experts; }
__device__ __forceinline__ int64_t pair_at(int64_t p0, int i) {
  return p0 + (threadIdx.x >> 6) * (kPer * 64) + i * 64 + (threadIdx.x & 63);
}

// The expert of each of this thread's pairs, -1 past the last pair.
__device__ __forceinline__ void load_ids(const int* __restrict__ ids, int64_t p0, int64_t pairs, int (&id)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) id[i] = pair_at(p0, i) < pairs ? ids[pair_at(p0, i)] : -1;
}

// The rank of each pair among the chunk's of its expert, in the order of the pairs, and the chunk's number of every expert's
// in total[] (LDS). A wave finds among its 64 pairs those with the same expert (a ballot for every bit of the number), the
// first of them adds their number to the wave's own count; the waves' counts are then added up.
__device__ __forceinline__ void rank_chunk(const int (&id)[kPer], int experts, int (&rank)[kPer], int (*count)[kMoeSortMaxExperts], int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = lane; e < experts; e += 64) count[wave][e] = 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    uint64_t same = __ballot(valid(id[i], experts));
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const uint64_t set = __ballot((id[i] >> b) & 1);
      same &= (id[i] >> b) & 1 ? set : ~set;
    }
    const uint64_t below = same & ((1ull << lane) - 1);
    if (valid(id[i], experts)) {
      rank[i] = count[wave][id[i]] + __popcll(below);
      // every lane has read before the first one adds: a wave's LDS operations are done in order
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (below == 0) count[wave][id[i]] += __popcll(same);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kSortThreads) {   // counts of the waves before
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = count[w][e];
      count[w][e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (valid(id[i], experts)) rank[i] += count[wave][id[i]];
}
static_assert(kMoeSortMaxExperts == 1 << 10, "the bits of an expert's number");

// From every expert's number of pairs (total[e], LDS) its first row start[e] (LDS), and the end start[experts]. All
// threads of the workgroup, an expert each.
__device__ __forceinline__ void lay_out(const int* total, int* start, int experts, int align) {
  static_assert(kMoeSortMaxExperts <= kSortThreads, "an expert each");
  __shared__ int sums[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = threadIdx.x;
  const int mine = e < experts ? padded_run(total[e], align) : 0;
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int at = upto - mine;
  for (int w = 0; w < wave; ++w) at += sums[w];
  if (e < experts) {
    start[e] = at;
    if (e == experts - 1) start[experts] = at + mine;
  }
  __syncthreads();
}

// The offsets, and -1 for the rows without a pair, shared out over `parts` workgroups: a wave an expert's, everybody
// those behind the last expert's.
__device__ __forceinline__ void mark(const int* total, const int* start, int experts, int64_t rows, int part, int parts,
                                     int64_t* __restrict__ offsets, int* __restrict__ pair_of) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (part == 0)
    for (int e = threadIdx.x; e <= experts; e += kSortThreads) offsets[e] = start[e];
  for (int e = part * kSortWaves + wave; e < experts; e += parts * kSortWaves)
    each_64th(start[e] + total[e], start[e + 1], lane, [&](int64_t r) { pair_of[r] = -1; });
  for (int64_t r = start[experts] + (int64_t)part * kSortThreads + threadIdx.x; r < rows; r += (int64_t)parts * kSortThreads) pair_of[r] = -1;
}

// counts[chunk][e]
__global__ __launch_bounds__(kSortThreads) void k_moe_count(const int* __restrict__ ids, int64_t pairs, int experts,
                                                            int* __restrict__ counts) {
  __shared__ int count[kMoeSortMaxExperts];
  for (int e = threadIdx.x; e < experts; e += kSortThreads) count[e] = 0;
  int id[kPer];
  load_ids(ids, (int64_t)blockIdx.x * kChunk, pairs, id);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (valid(id[i], experts)) atomicAdd(&count[id[i]], 1);   // a number: the order of the additions does not show
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kSortThreads) counts[(int64_t)blockIdx.x * experts + e] = count[e];
}

// total[e] = the counts of all chunks, before[e] = those of the chunks before `chunk` (LDS). Few experts: a thread adds up
// a share of the chunks.
__device__ __forceinline__ void add_up(const int* __restrict__ counts, int64_t chunks, int64_t chunk, int experts, int* part, int* total, int* before) {
  const int shares = kSortThreads / experts, share = threadIdx.x / experts, e = threadIdx.x % experts;
  int all = 0, until = 0;
  if (share < shares) {
#pragma unroll 4
    for (int64_t c = share; c < chunks; c += shares) {
      const int n = counts[c * experts + e];
      all += n;
      until += c < chunk ? n : 0;
    }
  }
  part[threadIdx.x] = all;
  part[kSortThreads + threadIdx.x] = until;
  __syncthreads();
  if (threadIdx.x < experts) {
    all = until = 0;
    for (int s = 0; s < shares; ++s) {
      all += part[s * experts + threadIdx.x];
      until += part[kSortThreads + s * experts + threadIdx.x];
    }
    total[threadIdx.x] = all;
    before[threadIdx.x] = until;
  }
  __syncthreads();
}

// One workgroup: counts[chunk][e] becomes the row of the chunk's first pair of expert e.
__global__ __launch_bounds__(kSortThreads) void k_moe_scan(int* __restrict__ counts, int64_t chunks, int experts, int align,
                                                           int64_t rows, int64_t* __restrict__ offsets,
                                                           int* __restrict__ pair_of) {
  __shared__ int total[kMoeSortMaxExperts], start[kMoeSortMaxExperts + 1], part[kSortThreads];
  const int shares = kSortThreads / experts;                  // at least one
  const int share = threadIdx.x / experts, e = threadIdx.x % experts;
  const int64_t per = (chunks + shares - 1) / shares;
  const int64_t c0 = share * per, c1 = c0 + per < chunks ? c0 + per : chunks;
  int sum = 0;
  if (share < shares) {
#pragma unroll 8
    for (int64_t c = c0; c < c1; ++c) sum += counts[c * experts + e];
  }
  part[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x < experts) {
    int t = 0;
    for (int s = 0; s < shares; ++s) t += part[s * experts + threadIdx.x];
    total[threadIdx.x] = t;
  }
  __syncthreads();
  lay_out(total, start, experts, align);
  mark(total, start, experts, rows, 0, 1, offsets, pair_of);
  if (share < shares) {
    int at = start[e];
    for (int s = 0; s < share; ++s) at += part[s * experts + e];
    for (int64_t c = c0; c < c1; c += 8) {
      int n[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = c + i < c1 ? counts[(c + i) * experts + e] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i < c1) counts[(c + i) * experts + e] = at;
        at += n[i];
      }
    }
  }
}

// Places a chunk's pairs. FIRST: where its first rows come from: its own counts (the only chunk), all chunks' counts, or
// k_moe_scan.
enum First { kAlone, kCounts, kScanned };
template <int FIRST>
__global__ __launch_bounds__(kSortThreads) void k_moe_place(const int* __restrict__ ids, int64_t pairs, int experts, int align, int64_t rows,
                                                            const int* __restrict__ counts, int64_t* __restrict__ offsets,
                                                            int* __restrict__ row_of, int* __restrict__ pair_of) {
  __shared__ int count[kSortWaves][kMoeSortMaxExperts];
  __shared__ int own[kMoeSortMaxExperts], total[kMoeSortMaxExperts], before[kMoeSortMaxExperts], start[kMoeSortMaxExperts + 1];
  const int64_t p0 = (int64_t)blockIdx.x * kChunk;
  int id[kPer], rank[kPer];
  load_ids(ids, p0, pairs, id);
  if constexpr (FIRST == kCounts) {
    add_up(counts, gridDim.x, blockIdx.x, experts, &count[0][0], total, before);
    lay_out(total, start, experts, align);
    mark(total, start, experts, rows, blockIdx.x, gridDim.x, offsets, pair_of);
  }
  rank_chunk(id, experts, rank, count, own);
  if constexpr (FIRST == kAlone) {
    lay_out(own, start, experts, align);
    mark(own, start, experts, rows, 0, 1, offsets, pair_of);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = pair_at(p0, i);
    if (p >= pairs) continue;
    int row = -1;
    if (valid(id[i], experts)) {
      if constexpr (FIRST == kScanned) row = counts[(int64_t)blockIdx.x * experts + id[i]] + rank[i];
      else row = start[id[i]] + rank[i] + (FIRST == kCounts ? before[id[i]] : 0);
      pair_of[row] = (int)p;
    }
    row_of[p] = row;
  }
}

// ---- rows ------------------------------------------------------------------------------------
template <bool F32>
__device__ __forceinline__ void put(void* p, int64_t row, int64_t ld, int64_t i, int64_t n, const Elems& e) {
  if constexpr (F32) store_f32(static_cast<float*>(p) + row * ld, i, n, e);
  else store_bf16(static_cast<uint16_t*>(p) + row * ld, i, n, e);
}
__device__ __forceinline__ Elems nothing() {
  Elems e;
#pragma unroll
  for (int q = 0; q < 8; ++q) e.v[q] = 0.0f;
  return e;
}

// A wave a row, a few vectors of it in flight together; without weights it is a copy. NT: stores past the caches, of outputs
// larger than the last-level cache (256 MB), of which the next kernel would find nothing there: gathered and
// quantized from there, 572 MB: 473 us against 511, 308 MB: 257 against 279; 175 MB: 145 against 142.
constexpr int kRowBatch = 6;
constexpr int64_t kCached = (int64_t)256 << 20;
template <bool F32, bool NT>
__global__ __launch_bounds__(kThreads) void k_moe_gather(const void* __restrict__ x, int64_t ldx, int64_t pairs, int top_k,
                                                         const int* __restrict__ pair_of, const float* __restrict__ weights,
                                                         void* __restrict__ out, int64_t ldo, int64_t rows, int64_t n) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (row >= rows) return;
  const int pair = pair_of[row];
  const bool has = (uint64_t)(int64_t)pair < (uint64_t)pairs;
  const float w = has && weights ? weights[pair] : 1.0f;
  const void* src = has ? row_at<F32>(x, (uint32_t)pair / (uint32_t)top_k, ldx) : nullptr;
  void* dst = row_at<F32>(out, row, ldo);
  for (int64_t i0 = lane * 8; i0 < n; i0 += kRowBatch * 64 * 8) {
    Raw<F32> v[kRowBatch];
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b) {
      v[b] = Raw<F32>{};
      if (has && i0 + b * 512 < n) v[b] = load_raw<F32>(src, i0 + b * 512, n);
    }
    if (weights) {                                            // uniform
#pragma unroll
      for (int b = 0; b < kRowBatch; ++b) {
        float e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = raw_at(v[b], q) * w;
        v[b] = pack<F32>(e);
      }
    }
#pragma unroll
    for (int b = 0; b < kRowBatch; ++b)
      if (i0 + b * 512 < n) store_raw<F32, NT>(dst, i0 + b * 512, n, v[b]);
  }
}

// Eight columns of a token a thread.
template <bool F32, bool OUT32>
__global__ __launch_bounds__(kThreads) void k_moe_combine(const void* __restrict__ y, int64_t ldy, int64_t rows,
                                                          const int* __restrict__ row_of, const float* __restrict__ weights,
                                                          int64_t tokens, int top_k, void* __restrict__ out, int64_t ldo, int64_t n) {
  const int64_t vecs = (n + 7) / 8;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= tokens * vecs) return;
  const int64_t t = (uint64_t)id >> 32 ? id / vecs : (int64_t)((uint32_t)id / (uint32_t)vecs);
  const int64_t i = (id - t * vecs) * 8;
  Elems sum = nothing();
  constexpr int kBatch = 4;                                   // rows of a token in flight together
  for (int j = 0; j < top_k && rows > 0; j += kBatch) {
    Elems e[kBatch];
    float w[kBatch];
    bool has[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      has[b] = false;
      if (j + b < top_k) {                                    // uniform
        const int64_t row = row_of[t * top_k + j + b];
        has[b] = (uint64_t)row < (uint64_t)rows;
        w[b] = weights ? weights[t * top_k + j + b] : 1.0f;
        e[b] = load_any(row_at<F32>(y, has[b] ? row : 0, ldy), !F32, i, n);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int q = 0; q < 8; ++q) sum.v[q] = has[b] ? sum.v[q] + w[b] * e[b].v[q] : sum.v[q];
  }
  put<OUT32>(out, t, ldo, i, n, sum);
}

// The first blocks a wave a pair (token after token, so that a token's dout is read once from HBM), the
// others zeros into the rows without one.
template <bool F32, bool OUT32>
__global__ __launch_bounds__(kThreads) void k_moe_combine_grad(const void* __restrict__ dout, int64_t lddo,
                                                               const void* __restrict__ y, int64_t ldy, int64_t rows,
                                                               const int* __restrict__ row_of, const int* __restrict__ pair_of,
                                                               const float* __restrict__ weights, int64_t pairs, int top_k,
                                                               void* __restrict__ dy, int64_t lddy, float* __restrict__ dw,
                                                               int64_t n, int64_t pair_blocks) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if ((int64_t)blockIdx.x >= pair_blocks) {                   // uniform
    if (dy == nullptr) return;
    const int64_t r0 = ((int64_t)blockIdx.x - pair_blocks) * 64;
    const int64_t mine = r0 + lane;
    const bool empty = mine < rows && (uint64_t)(int64_t)pair_of[mine] >= (uint64_t)pairs;
    uint64_t todo = __ballot(empty);
    for (int k = 0; todo != 0; ++k, todo &= todo - 1) {
      if (k % kWaves != wave) continue;
      const int64_t row = r0 + __builtin_ctzll(todo);
      for (int64_t i = lane * 8; i < n; i += 64 * 8) put<OUT32>(dy, row, lddy, i, n, nothing());
    }
    return;
  }
  const int64_t p = (int64_t)blockIdx.x * kWaves + wave;
  if (p >= pairs) return;
  const int64_t row = row_of[p];
  if ((uint64_t)row >= (uint64_t)rows) {
    if (dw && lane == 0) dw[p] = 0.0f;
    return;
  }
  const float w = weights[p];
  const void* g_row = row_at<OUT32>(dout, (uint32_t)p / (uint32_t)top_k, lddo);
  const void* y_row = row_at<F32>(y, row, ldy);
  float dot = 0.0f;
#pragma unroll 4
  for (int64_t i = lane * 8; i < n; i += 64 * 8) {
    Elems g = load_any(g_row, !OUT32, i, n);
    if (dw) {
      const Elems e = load_any(y_row, !F32, i, n);
#pragma unroll
      for (int q = 0; q < 8; ++q) dot += g.v[q] * e.v[q];
    }
    if (dy) {
#pragma unroll
      for (int q = 0; q < 8; ++q) g.v[q] *= w;
      put<OUT32>(dy, row, lddy, i, n, g);
    }
  }
  if (dw) {
    dot = wave_fold_sum(dot);
    if (lane == 0) dw[p] = dot;
  }
}

}  // namespace

int64_t moe_sort_chunks(int64_t pairs) { return (pairs + kChunk - 1) / kChunk; }

size_t moe_sort_workspace_bytes(int64_t pairs, int64_t experts) {
  const int64_t c = moe_sort_chunks(pairs);
  return c > 1 ? (size_t)c * (size_t)experts * sizeof(int) : 0;
}

hipError_t launch_moe_sort(const int* ids, int64_t pairs, int experts, int align, int64_t rows, int64_t* offsets, int* row_of,
                           int* pair_of, int* ws, hipStream_t stream) {
  const int64_t chunks = moe_sort_chunks(pairs);
  const dim3 grid((unsigned)(chunks < 1 ? 1 : chunks)), block(kSortThreads);
#define NVFP4_PLACE(F) hipLaunchKernelGGL(k_moe_place<F>, grid, block, 0, stream, ids, pairs, experts, align, rows, ws, offsets, row_of, pair_of)
  if (chunks <= 1) {
    NVFP4_PLACE(kAlone);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_moe_count, grid, block, 0, stream, ids, pairs, experts, ws);
  if (chunks <= kChunksEach) {
    NVFP4_PLACE(kCounts);
  } else {
    hipLaunchKernelGGL(k_moe_scan, dim3(1), block, 0, stream, ws, chunks, experts, align, rows, offsets, pair_of);
    NVFP4_PLACE(kScanned);
  }
#undef NVFP4_PLACE
  return hipGetLastError();
}

hipError_t launch_moe_gather(const void* x, bool fp32, int64_t ldx, int64_t pairs, int top_k, const int* pair_of,
                             const float* weights, void* out, int64_t ldo, int64_t rows, int64_t n, hipStream_t stream) {
  const dim3 grid((unsigned)((rows + kWaves - 1) / kWaves)), block(kThreads);
  const bool nt = rows * n * (fp32 ? 4 : 2) > kCached;
#define NVFP4_MG(A, B) hipLaunchKernelGGL((k_moe_gather<A, B>), grid, block, 0, stream, x, ldx, pairs, top_k, pair_of, weights, out, ldo, rows, n)
  if (fp32) { if (nt) NVFP4_MG(true, true); else NVFP4_MG(true, false); }
  else      { if (nt) NVFP4_MG(false, true); else NVFP4_MG(false, false); }
#undef NVFP4_MG
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* y, bool fp32, int64_t ldy, int64_t rows, const int* row_of, const float* weights,
                              int64_t tokens, int top_k, void* out, bool out32, int64_t ldo, int64_t n, hipStream_t stream) {
  const int64_t total = tokens * ((n + 7) / 8);
  const dim3 grid((unsigned)((total + kThreads - 1) / kThreads)), block(kThreads);
#define NVFP4_MC(A, B) hipLaunchKernelGGL((k_moe_combine<A, B>), grid, block, 0, stream, y, ldy, rows, row_of, weights, tokens, top_k, out, ldo, n)
  if (fp32) { if (out32) NVFP4_MC(true, true); else NVFP4_MC(true, false); }
  else      { if (out32) NVFP4_MC(false, true); else NVFP4_MC(false, false); }
#undef NVFP4_MC
  return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const void* dout, bool out32, int64_t lddo, const void* y, bool fp32, int64_t ldy, int64_t rows,
                                   const int* row_of, const int* pair_of, const float* weights, int64_t pairs, int top_k,
                                   void* dy, int64_t lddy, float* dw, int64_t n, hipStream_t stream) {
  const int64_t pair_blocks = (pairs + kWaves - 1) / kWaves, row_blocks = dy ? (rows + 63) / 64 : 0;
  const dim3 grid((unsigned)(pair_blocks + row_blocks)), block(kThreads);
  if (pair_blocks + row_blocks == 0) return hipSuccess;
#define NVFP4_MG(A, B) hipLaunchKernelGGL((k_moe_combine_grad<A, B>), grid, block, 0, stream, dout, lddo, y, ldy, rows, row_of, pair_of, weights, pairs, top_k, dy, lddy, dw, n, pair_blocks)
  if (fp32) { if (out32) NVFP4_MG(true, true); else NVFP4_MG(true, false); }
  else      { if (out32) NVFP4_MG(false, true); else NVFP4_MG(false, false); }
#undef NVFP4_MG
  return hipGetLastError();
}

}  // namespace nvfp4
