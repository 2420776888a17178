// Softmax cross entropy of a language model's output head, logits l = x W^T never kept:
//   lse[t] = log sum over v of exp(l[t, v]);   loss[t] = lse[t] - l[t, target[t]]
//   backward, with the gradient g[t] of each loss:  G[t, v] = g[t] exp(l[t, v] - lse[t]),  the target's g[t] (exp(-loss[t]) - 1)
//   dx = G W,  dW = G^T x
// x [T, H] and W [V, H] in BF16, products and sums in FP32; a target outside 0 .. V - 1 does not count: loss 0, G 0.
//
// Forward: one product in tiles of W's rows times tokens. A lane of a finished tile holds one token's logits for its
// rows, so the tile leaves the maximum and the sum of exp(l - maximum) of each of its tokens without their targets, and the logit of a
// token whose target lies in it. k_merge joins the tiles' pairs: with d = log(sum over the other words of exp(l - l[target])) the loss is
// log(1 + exp(d)), which keeps the digits of a small loss (as lse - l[target], two numbers rounded at their size, a loss of 1e-6 at
// logits of 25 was all rounding). Backward: the logits are computed again, a piece of
// the vocabulary at a time, and leave the product as G in BF16: 8 bits of each entry's own size, what a BF16 dx or dW keeps of its sums, and
// what x and W, its partners in both products, keep of the numbers that they stand for. An FP32 dW is the FP32 sum of these
// (1024 tokens, 8000 words, hidden 512: off by 5.7e-5 of its norm, in the words that are no token's target by 1.4e-3; a BF16 dW by
// 1.7e-3); the other half of each G would be a fifth product, a third of the backward's time. The target's G comes from the loss, since 1 - exp(l - lse)
// of a confident token is made of lse's rounding (logits of 25: three times its value off). Mostly a token's largest by far, it keeps
// what BF16 leaves of it in FP32: dx gets it when its shares are joined, dW, in BF16 once more (2^-17 of G), from the tile that holds the
// word. dW's rows of the piece are G^T x, and dx grows by G W in FP32, rounded once after the last piece. Four products in all, 2 T H V
// operations each: bound by the matrix cores.
//
// One kernel does all of them: D[n, m] = sum over k of A[m, k] B[n, k]. A workgroup of 4 waves owns a tile, a wave TM x TN
// tiles of v_mfma_f32_16x16x32_bf16 (of the two shapes the one that moves fewer accumulators per operation: the chip is at
// its power limit in these products, and 8192 x 32768 x 5120 took 2220 us with 32 x 32 x 16, 1975 with it). The operands
// go from global memory into LDS by DMA, two stages of 64 elements of k, a KB an operation.
//  - An operand whose rows are contiguous in k lies there by rows of 128 bytes, the 16-byte piece c of row r at c ^ (r / 2
//    % 8), so that any 16 of the rows which a fragment's lanes read fall on all 64 banks.
//  - One that is contiguous in its rows (W and x in the gradients' products, G in dW's) lies there by lines of k, and the
//    LDS reads transpose it (ds_read_b64_tr_b16); its 32-byte pieces are swapped likewise. No operand is ever
//    transposed in memory (with W^T, G^T and x^T written and read again the backward took 7360 us, now 6330).
// The operations are issued one by one between the products (all together after the barrier: 2420 us for the above with the
// larger shape, one every four products 2220): several fill the address unit's queue, and the wave waits.
// FP32 gradients that are added to are on their way two columns before their addition (50021 words, hidden 1040, 333 tokens:
// dW 212 us without, 143 with).
// Measured: 8192 tokens, 131072 words, hidden 5120: forward 7.8 ms (1.42 PFLOP/s), backward 25 (1.30). 1003 tokens, 32003 words,
// hidden 2704: forward 175 to 180 us (0.97). 333 tokens, 50021 words, hidden 1040: forward 76, G 69, dx 73, dW 72 us; rows of 2080
// bytes begin inside a line of 128, so each piece of a stage is parts of two (hidden 1024: 66 and 59 us), and a round of tiles has
// 17 steps of a us, or 6 for dW, between its first loads and its last stores.
#include <type_traits>
#include <utility>

#include "device_common.h"
#include "launch.h"

namespace nvfp4 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(3))) bf16x4* lds_4_t;

constexpr int kThreads = 256;
constexpr int kStepK = 64, kStepBytes = 128, kStages = 2;
constexpr float kLog2e = 1.44269504088896341f;
constexpr int kBucket = 128;                                  // words: no tile of dW holds a part of one

// A workgroup's tile: 4 waves, WM x WN of them, each TM x TN matrix instructions of 16 x 16.
template <int TM, int TN, int WM, int WN>
struct Tile {
  static_assert(WM * WN == 4, "four waves");
  static constexpr int kTilesM = TM, kTilesN = TN, kWavesM = WM, kWavesN = WN, kWaveM = 16 * TM, kWaveN = 16 * TN;
  static constexpr int kM = kWaveM * WM, kN = kWaveN * WN;
  static constexpr int kAtOnce = TM * TN <= 16 ? 2 : 1;       // workgroups of a compute unit: by LDS and registers
  static constexpr int kOpsA = kM / 8, kOps = (kM + kN) / 8;  // DMA operations of a stage, 1 KB each
  static constexpr int kOpsOfWave = kOps / 4;
  static_assert(kOpsA % 4 == 0, "a wave's i-th operation is of A, or of B, for every wave");
  static constexpr int kStageBytes = (kM + kN) * kStepBytes;
  static constexpr int kLds = kStages * kStageBytes;
};
using Full = Tile<8, 8, 2, 2>;                                // 256 x 256
using Half = Tile<4, 4, 2, 2>;                                // 128 x 128, two workgroups on a compute unit
using Few = Tile<4, 2, 4, 1>;                                 // 256 rows of A, 32 of B

// s_waitcnt immediate (gfx9 encoding): vmcnt(vm) lgkmcnt(lgkm), expcnt not waited on.
constexpr int waitcnt_imm(int vm, int lgkm) { return (vm & 0xF) | ((vm >> 4) << 14) | (0x7 << 4) | ((lgkm & 0xF) << 8); }

// An operand of `rows` rows: element (row, k) at p[row * ld + k], or where the kernel takes it transposed (TA, TB) at
// p[k * ld + row].
struct Rows {
  const uint16_t* p;
  int64_t rows, ld;
};

enum Epilogue : int { kLse = 0, kGrad = 1, kStoreBf16 = 2, kStoreF32 = 3, kAddF32 = 4 };

struct Out {
  // kLse: A is W (m a word), B is x (n a token)
  const int64_t* targets;
  float* part;                  // [tiles of m * waves of m][2][tokens]: maximum, sum, of the words that are not the token's target
  float* picked;                // [tokens]: the target's logit
  // kGrad: likewise; d [tokens, ld] BF16
  const float *lse, *grad;
  const float* loss;            // or null: the target's G from its logit and lse
  // of the target's G what BF16 leaves of it [tokens]: kGrad writes it, dW's products add it with x
  float* rest;
  const int *by_word, *start;   // the tokens in the order of their targets; where those of words 128 b begin
  int64_t first, vocab;         // the word that row 0 of A is; all words
  // kGrad, kStore..: d[n * ld + m]; m up to m_store (beyond A's rows zeros)
  void* d;
  int64_t ld, m_store;
  int64_t slice;                // elements between the results of two shares of k
  int64_t buckets;              // of all words
};

// Tile (tm, tn) for workgroup `bid`: consecutive workgroups go to the 8 XCDs in turn, so each XCD gets a run of
// ids of its own; ids walk bands of 8 tile rows, column by column, so that the tiles in flight on one
// XCD share their panels in its L2.
__device__ __forceinline__ void tile_of(int64_t bid, int64_t tiles_m, int64_t tiles_n, int64_t& tm, int64_t& tn) {
  const int64_t n = tiles_m * tiles_n, per = (n + 7) / 8, xcd = bid % 8, local = bid / 8;
  const int64_t tall = n % 8 == 0 ? 8 : n % 8;
  const int64_t id = xcd < tall ? xcd * per + local : tall * per + (xcd - tall) * (per - 1) + local;
  const int64_t band = 8 * tiles_n, first = id / band * 8;
  const int64_t height = tiles_m - first < 8 ? tiles_m - first : 8;
  tm = first + id % band % height;
  tn = id % band / height;
}

// f(0) .. f(N - 1), the index a constant.
template <int N, class F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  each_of<N>(f, std::make_integer_sequence<int, N>{});
}

// acc = the tile's products over the steps [s0, s1) of K.
template <class C, bool TA, bool TB>
__device__ __forceinline__ void multiply(Rows A, Rows B, int64_t m0, int64_t n0, int64_t K, int s0, int s1, uint8_t* lds,
                                         f32x4 (&acc)[C::kTilesM][C::kTilesN]) {
  constexpr int TM = C::kTilesM, TN = C::kTilesN, kOpsOfWave = C::kOpsOfWave;
  static_assert(!TA || C::kM == 256 || C::kM == 128, "lines of 512 or 256 bytes");
  static_assert(!TB || C::kN == 256 || C::kN == 128, "lines of 512 or 256 bytes");
  constexpr int kLineA = 2 * C::kM, kLineB = 2 * C::kN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::kWavesN, wn = wave % C::kWavesN;
  constexpr uint32_t kBeyond = 0x80000000u;                   // past the part of an operand that any resource spans
  // What step s needs of an operand as a buffer descriptor: the tile's rows, or (transposed) the step's 64 lines from the
  // tile's first column on; what lies past it reads as zero, and everything of a step that there is not. (Columns past a
  // transposed operand's last are the next line's: they end in results that are not stored. Sizes up to a
  // multiple of 8: an operand without that many has zeros there, and a dword of two elements is in or out.)
  auto descriptor = [&](const Rows& o, int64_t r0, int64_t tall, bool transposed, int s) {
    const int64_t k0 = transposed ? (int64_t)s * kStepK : 0, left = o.rows - r0;
    const int64_t lines = transposed ? (K - k0 < kStepK ? K - k0 : kStepK) : (left < tall ? left : tall);
    const int64_t last = ((transposed ? left : K) + 7) & ~int64_t(7);
    const int64_t bytes = lines > 0 && left > 0 && s < s1 ? ((lines - 1) * o.ld + last) * 2 : 0;
    const uint64_t base = reinterpret_cast<uint64_t>(o.p + (bytes ? (transposed ? k0 * o.ld + r0 : r0 * o.ld) : 0));
    auto uniform = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); };
    return v4u32{uniform((uint32_t)base), uniform((uint32_t)(base >> 32) & 0xFFFF), uniform((uint32_t)bytes), 0x00020000u};
  };
  const uint32_t pitch_a = (uint32_t)(A.ld * 2), pitch_b = (uint32_t)(B.ld * 2);
  // A wave's i-th operation is number op = 4 i + wave of a stage.
  //  rows: 8 rows of 128 bytes, lane's row 8 op + lane / 8; the place of piece c of a row is c ^ (row / 2 % 8)
  //  transposed: 2 lines (k) of 512 bytes, lane's line k = 2 op + lane / 32; the place of the 32 bytes c of a line is
  //  c ^ (k % 4 + 4 (k / 8 % 2)), where k / 8 % 2 is i % 2; or 4 lines of 256, k = 4 op + lane / 16 and k / 8 % 2 wave / 2
  const uint32_t piece = (uint32_t)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
  const uint32_t column_512 = ((uint32_t)(((lane & 31) >> 1) ^ ((2 * wave + (lane >> 5)) & 3)) * 32) + (lane & 1) * 16;
  const uint32_t column_256 = ((uint32_t)(((lane & 15) >> 1) ^ (lane >> 4 | (wave & 2) << 1)) * 32) + (lane & 1) * 16;
  const uint32_t row_bytes = (uint32_t)(K * 2);
  uint32_t offset[kOpsOfWave];                                // of this lane in its operations, from the descriptor's base
  each<kOpsOfWave>([&](auto index) {
    constexpr int i = decltype(index)::value;
    constexpr bool is_a = 4 * i < C::kOpsA, T = is_a ? TA : TB;
    constexpr int in = is_a ? i : i - C::kOpsA / 4;           // among the operand's operations of this wave
    const uint32_t pitch = is_a ? pitch_a : pitch_b;
    if constexpr (!T) offset[i] = (uint32_t)(32 * in + 8 * wave + (lane >> 3)) * pitch + piece;
    else if constexpr ((is_a ? kLineA : kLineB) == 512) offset[i] = (uint32_t)(8 * in + 2 * wave + (lane >> 5)) * pitch + (column_512 ^ (in % 2 ? 128u : 0u));
    else offset[i] = (uint32_t)(16 * in + 4 * wave + (lane >> 4)) * pitch + column_256;
  });
  struct Stage {
    v4u32 a, b;
    uint32_t k;                                               // this lane's place in a row; past everything where the row has none
  };
  auto stage_of = [&](int s) {
    const uint32_t k = (uint32_t)s * kStepBytes;
    return Stage{descriptor(A, m0, C::kM, TA, s), descriptor(B, n0, C::kN, TB, s), k + piece < row_bytes ? k : 0x80000000u};
  };
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_ptr_t)lds;
  auto dma = [&](const Stage& st, uint32_t base, auto index) { // base: of the stage, at this wave's first operation
    constexpr int i = decltype(index)::value, place = 4 * i * 1024;
    constexpr bool is_a = 4 * i < C::kOpsA;
    const uint32_t at = (is_a ? TA : TB) ? offset[i] : offset[i] + st.k;
    const v4u32 d = is_a ? st.a : st.b;
    // By hand, since the compiler waits for every DMA in flight before a transposing read of LDS. It writes no register;
    // the waits for what it writes to LDS are the explicit ones below.
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
                 :: "s"(base), "i"(place), "v"(at), "s"(d) : "m0", "scc", "memory");
  };
  // Fragments of half a step (32 elements of k): lane l holds elements 8 (l / 16) .. + 7 of row l % 16.
  //  rows: one piece. transposed: twice four elements of k from lines in which the 16 rows lie side by side; sixteen lanes
  //  ask for 4 lines of 32 bytes, eight bytes each, and get them transposed.
  const uint32_t row_at = (uint32_t)(lane & 15) * kStepBytes + (uint32_t)((lane >> 4) ^ (lane >> 1 & 7)) * 16;
  auto line_at = [&](int line) {
    return (uint32_t)((8 * (lane >> 4) + (lane >> 2 & 3)) * line) + (uint32_t)((lane >> 2 & 3) | (lane >> 4 & 1) << 2) * 32 + (lane & 3) * 8;
  };
  // where in the stage that is read: rows by half, transposed by the place of a row block in its line
  constexpr int kPlacesA = TA ? TM : 2, kPlacesB = TB ? TN : 2;
  uint32_t at_a[kPlacesA], at_b[kPlacesB];
  {
    const uint32_t pa = lds_base, pb = pa + C::kM * kStepBytes;
    const int ra = wm * C::kWaveM, rb = wn * C::kWaveN;       // the wave's first row
#pragma unroll
    for (int i = 0; i < kPlacesA; ++i) {
      if constexpr (TA) at_a[i] = pa + (ra + 16 * i) / 128 * 256 + (line_at(kLineA) ^ (uint32_t)((ra / 16 + i) % 8 * 32));
      else at_a[i] = pa + ra * kStepBytes + (row_at ^ (uint32_t)(64 * i));
    }
#pragma unroll
    for (int i = 0; i < kPlacesB; ++i) {
      if constexpr (TB) at_b[i] = pb + (rb + 16 * i) / 128 * 256 + (line_at(kLineB) ^ (uint32_t)((rb / 16 + i) % 8 * 32));
      else at_b[i] = pb + rb * kStepBytes + (row_at ^ (uint32_t)(64 * i));
    }
  }
  auto frag_rows = [](uint32_t at, int i) { return *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(at + i * 16 * kStepBytes); };
  auto frag_lines = [](uint32_t at, int half, int line) {
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_4_t)(uintptr_t)(at + half * 32 * line));
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_4_t)(uintptr_t)(at + half * 32 * line + 4 * line));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto barrier = [] {
    // plain s_barrier: a fence would also wait for the DMA in flight; the empty asm statements keep the compiler
    // from moving LDS accesses across it
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{};
  const uint32_t lds_wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_base + (uint32_t)wave * 1024));
  each<2>([&](auto b) {
    const Stage st = stage_of(s0 + b);
    each<kOpsOfWave>([&](auto i) { dma(st, lds_wave + b * C::kStageBytes, i); });
  });
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(kOpsOfWave, 15));    // the first stage landed
  barrier();
  constexpr int kReads = TM + TN, kSlots = TM * TN, kTail = kSlots >= 16 ? 8 : 0;
  bf16x8 a[2][TM], b[2][TN];
  // reads in the order of their use
  auto read = [&](auto set, auto index) {
    constexpr int r = decltype(index)::value, h = decltype(set)::value;
    if constexpr (r < TN) {
      if constexpr (TB) b[h][r] = frag_lines(at_b[r], h, kLineB);
      else b[h][r] = frag_rows(at_b[h], r);
    } else {
      if constexpr (TA) a[h][r - TN] = frag_lines(at_a[r - TN], h, kLineA);
      else a[h][r - TN] = frag_rows(at_a[h], r - TN);
    }
  };
  each<kReads>([&](auto r) { read(std::integral_constant<int, 0>{}, r); });

  // Two halves of a step; the next half's fragments are read while one's products run. When the second half begins, the
  // wave has read all of its stage: once its own DMA of the other stage has landed it meets the others, reads on there,
  // and the DMA of the step after next refills this one, an operation every few products: several together fill the
  // address unit's queue, and a wave whose next operation finds no room there issues no products either.
  int s = s0, other = C::kStageBytes;                         // other: from the stage that is read to the other one
  do {                                                        // a share without a step multiplies zeros once
    const Stage next = stage_of(s + 2);
    each<2>([&](auto half) {
      constexpr int t = decltype(half)::value;
      if constexpr (t == 1) {
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
        barrier();
#pragma unroll
        for (int i = 0; i < kPlacesA; ++i) at_a[i] += other;
#pragma unroll
        for (int i = 0; i < kPlacesB; ++i) at_b[i] += other;
      }
      const uint32_t refill = lds_wave + (uint32_t)(C::kStageBytes - other) / 2;
      each<kSlots>([&](auto slot) {
        constexpr int p = decltype(slot)::value;
        // what goes before product p: a read (done some products before the half ends), an operation of the DMA
        each<kReads>([&](auto r) {
          if constexpr (1 + r * (kSlots - 1 - kTail) / kReads == p) read(std::integral_constant<int, t ^ 1>{}, r);
        });
        if constexpr (t == 1)
          each<kOpsOfWave>([&](auto i) {
            if constexpr ((2 * i + 1) * kSlots / (2 * kOpsOfWave) == p) dma(next, refill, i);
          });
        constexpr int i = p / TN, j = p % TN;
        asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(a[t][i]), "v"(b[t][j]));
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    other = -other;
  } while (++s < s1);
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));              // no DMA outlives the tile
  asm volatile("s_nop 15\n\ts_nop 15");                       // the last products are in their accumulators
}

// acc += rest[t] x[t] over the tokens whose target is one of the tile's words (dW's products: B's rows are words), [from, to) in the order
// of words: 32 at a time one more half step, whose B holds rest (in BF16: 2^-17 of G) at each token's word and zeros.
// Words that many tokens end in make their tiles longer. G and dW of 8192 tokens, 131072 words, hidden 5120: 17.0 ms with targets drawn
// uniformly, 17.1 with the v-th word's share proportional to 1 / v, 17.0 with one word for all; 8192, 32768 and 1024: 1.12 ms, 1.24, 1.52.
template <class C>
__device__ __forceinline__ void add_rest(const Rows& A, int64_t m0, int64_t n0, int from, int to, const Out& o,
                                         f32x4 (&acc)[C::kTilesM][C::kTilesN]) {
  constexpr int TM = C::kTilesM, TN = C::kTilesN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t word_of_lane = o.first + n0 + wave % C::kWavesN * C::kWaveN + (lane & 15);
  const int64_t m_of_wave = m0 + wave / C::kWavesN * C::kWaveM;
  for (int e0 = from; e0 < to; e0 += 32) {                    // lane l: tokens 8 (l / 16) .. + 7, row or word l % 16
    // loads without a branch, all on their way together: past the end the last token's, of which zeros are made
    const int first = e0 + 8 * (lane >> 4);
    int token[8], at[8];
    uint32_t rest[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) token[q] = o.by_word[first + q < to ? first + q : to - 1];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      at[q] = (int)(o.targets[token[q]] - word_of_lane);
      rest[q] = bf16_rn_bits(o.rest[token[q]]);
    }
    bf16x8 a[TM], b[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t row = m_of_wave + 16 * i, m = (row < A.rows ? row : 0) + (lane & 15);   // A.rows is a multiple of 16
      uint32_t x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = A.p[(int64_t)token[q] * A.ld + m];
      v4u32 w;
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = (first + 2 * q < to ? x[2 * q] : 0u) | (first + 2 * q + 1 < to ? x[2 * q + 1] << 16 : 0u);
      a[i] = __builtin_bit_cast(bf16x8, w);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (first + q >= to) rest[q] = 0u;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      v4u32 w;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = (at[2 * q] == 16 * j ? rest[2 * q] : 0u) | (at[2 * q + 1] == 16 * j ? rest[2 * q + 1] << 16 : 0u);
      b[j] = __builtin_bit_cast(bf16x8, w);
    }
    __builtin_amdgcn_sched_barrier(0);
    each<TM * TN>([&](auto slot) {
      constexpr int i = decltype(slot)::value / TN, j = decltype(slot)::value % TN;
      f32x4& sum = acc[i][j];
      const bf16x8 &fa = a[i], &fb = b[j];
      asm("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(sum) : "v"(fa), "v"(fb));
    });
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15");                     // the products are in their accumulators
  }
}

template <class C, int EPI, bool TA, bool TB>
__global__ __launch_bounds__(kThreads, C::kAtOnce) void k_product(Rows A, Rows B, int64_t K, int64_t tiles_m, int64_t tiles_n, int shares, Out o) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
  constexpr int TM = C::kTilesM, TN = C::kTilesN;
  const int64_t tiles = tiles_m * tiles_n;
  const int share = (int)(blockIdx.x / tiles);
  int64_t tm, tn;
  tile_of(blockIdx.x - share * tiles, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = tm * C::kM, n0 = tn * C::kN;
  const int steps = (int)((K + kStepK - 1) / kStepK);
  const int s0 = (int)((int64_t)steps * share / shares), s1 = (int)((int64_t)steps * (share + 1) / shares);
  f32x4 acc[TM][TN];
  int from = 0, to = 0;
  if constexpr (TB) {
    const int64_t b = (o.first + n0) / kBucket;               // pieces and tiles begin with a bucket; its words are of this piece
    from = o.start[b];
    to = o.start[b + C::kN / kBucket < o.buckets ? b + C::kN / kBucket : o.buckets];
  }
  multiply<C, TA, TB>(A, B, m0, n0, K, s0, s1, lds, acc);
  if constexpr (TB) add_rest<C>(A, m0, n0, from, to, o, acc);

  // lane l holds of each 16 x 16 tile column n = l % 16, rows m = 4 (l / 16) + 0 .. 3
  const int lane = threadIdx.x & 63, lane_n = lane & 15, lane_m = 4 * (lane >> 4);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mw = m0 + wave / C::kWavesN * C::kWaveM, nw = n0 + wave % C::kWavesN * C::kWaveN;
  // of this wave's rows: how many are A's
  const int rows = (int)(A.rows - mw < C::kWaveM ? A.rows - mw : C::kWaveM);
  constexpr bool kPacked = EPI == kGrad || EPI == kStoreBf16;
  // BF16 results go through LDS, so that a store covers whole rows of the wave's tile and not 32 bytes of each of 16: row n
  // of kWaveM elements, 16 bytes c of it at c ^ (n % kPieces). The stages are free once every wave has read them.
  constexpr int kPieces = C::kWaveM / 8;
  static_assert(!kPacked || 4 * C::kWaveN * C::kWaveM * 2 <= C::kLds, "LDS of the output pass");
  uint8_t* own = lds + wave * C::kWaveN * C::kWaveM * 2;
  if constexpr (kPacked) __syncthreads();
  // kAddF32: the sums so far of a column are on their way two columns ahead
  const int stored = (int)(o.m_store - mw < C::kWaveM ? o.m_store - mw : C::kWaveM);
  constexpr int kAhead = 2;
  v4f32 old[EPI == kAddF32 ? TN : 1][TM];
  auto place = [&](int j) { return static_cast<float*>(o.d) + share * o.slice + (nw + 16 * j + lane_n) * o.ld + mw + lane_m; };
  auto request = [&](int j) {
    if (j < TN && nw + 16 * j + lane_n < B.rows) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
        if (16 * i < stored) old[j][i] = *reinterpret_cast<const v4f32_any*>(place(j) + 16 * i);
    }
  };
  if constexpr (EPI == kAddF32) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) request(j);
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    // one column's values at a time out of the accumulators: read together they take every vector register
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TM; ++i) asm volatile("" : "+a"(acc[i][j]));
    const int64_t n = nw + 16 * j + lane_n;
    if constexpr (EPI == kLse) {
      const int64_t word = n < B.rows ? o.targets[n] - mw : -1;
      const int at = word >= 0 && word < rows ? (int)word : -1;
      if (__ballot(at >= 0)) {                                // few tiles hold a target of their tokens
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (at >= 0 && at - lane_m == 16 * i + r) {
              o.picked[n] = acc[i][j][r];
              acc[i][j][r] = -INFINITY;
            }
      }
      float top = -INFINITY, sum = 0.0f;
      auto pass = [&](auto whole) {
        auto value = [&](int i, int r) { return decltype(whole)::value || 16 * i + lane_m + r < rows ? acc[i][j][r] : -INFINITY; };
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) top = fmaxf(top, value(i, r));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) sum += __builtin_amdgcn_exp2f((value(i, r) - base) * kLog2e);
      };
      if (rows == C::kWaveM) pass(std::true_type{});
      else pass(std::false_type{});
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (n < B.rows && lane < 16) {
        float* part = o.part + (tm * C::kWavesM + wave / C::kWavesN) * 2 * B.rows + n;
        part[0] = top;
        part[B.rows] = sum;
      }
    } else if constexpr (kPacked) {
      float lse = 0.0f, gr = 0.0f;
      int target = -1;                                        // among this lane's rows, if it is one of them
      float own_g = 0.0f;                                     // the target's G
      if constexpr (EPI == kGrad) {
        if (n < B.rows) {
          lse = o.lse[n];
          const int64_t id = o.targets[n], word = id - o.first - mw;
          target = word >= lane_m && word < C::kWaveM ? (int)word - lane_m : -1;
          gr = (uint64_t)id < (uint64_t)o.vocab ? o.grad[n] : 0.0f;   // a token whose target does not count
        }
      }
      float less = 0.0f;                                      // the target's probability - 1
      if constexpr (EPI == kGrad) {
        if (__ballot(target >= 0)) {                          // few tiles hold a target of their tokens
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) less = target == 16 * i + r ? acc[i][j][r] - lse : less;
          if (target >= 0 && o.loss != nullptr) less = -o.loss[n];
          less = expm1f(less);
        }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = acc[i][j][r];
          if constexpr (EPI == kGrad) {
            const float p = __builtin_amdgcn_exp2f((v[r] - lse) * kLog2e);
            v[r] = gr * (target == 16 * i + r ? less : p);
            if (16 * i + r >= rows - lane_m || gr == 0.0f) v[r] = 0.0f;
            if (target == 16 * i + r) own_g = v[r];
          }
        }
        const int row = 16 * j + lane_n, c = 2 * i + (lane >> 5);
        *reinterpret_cast<v2u32*>(own + row * (C::kWaveM * 2) + (c ^ (row & (kPieces - 1))) * 16 + (lane >> 4 & 1) * 8) =
            v2u32{bf16_rn_pair(v[0], v[1]), bf16_rn_pair(v[2], v[3])};
      }
      if constexpr (EPI == kGrad) {
        if (target >= 0 && (target & 15) < 4) o.rest[n] = own_g - bf16_lo(bf16_rn_bits(own_g));
      }
    } else {
      if constexpr (EPI == kAddF32) request(j + kAhead);
      if (n < B.rows) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          if (16 * i >= stored) continue;                     // m_store is a multiple of 16
          v4f32 w = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
          if constexpr (EPI == kAddF32) w += old[j][i];
          *reinterpret_cast<v4f32_any*>(place(j) + 16 * i) = w;
        }
      }
    }
  }
  if constexpr (kPacked) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");    // the wave's LDS writes before its reads
    constexpr int kRowsAt = 64 / kPieces;                     // rows of an instruction
    const int c = lane % kPieces;
#pragma unroll 4
    for (int row = lane / kPieces; row < C::kWaveN; row += kRowsAt) {
      const int64_t n = nw + row, m = mw + (c ^ (row & (kPieces - 1))) * 8;
      const v4u32 w = *reinterpret_cast<const v4u32*>(own + row * (C::kWaveM * 2) + c * 16);
      if (n < B.rows && m < o.m_store) *reinterpret_cast<v4u32_any*>(static_cast<uint16_t*>(o.d) + n * o.ld + m) = w;
    }
  }
}

// lse and loss from the tiles' pairs: 16 tokens a workgroup, a token's pairs dealt out to 64 lanes.
constexpr int kMergeWaves = 16, kMergeTokens = 16;
__global__ __launch_bounds__(kMergeWaves * 64) void k_merge(const float* __restrict__ part, int64_t parts, int64_t tokens, int64_t vocab,
                                                            const int64_t* __restrict__ targets, const float* __restrict__ picked,
                                                            float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float tops[kMergeWaves][kMergeTokens], sums[kMergeWaves][kMergeTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, column = lane & (kMergeTokens - 1);
  const int64_t t = (int64_t)blockIdx.x * kMergeTokens + column;
  float top = -INFINITY, sum = 0.0f;
  // sum exp(top) with another pair: a pair of no words (past the vocabulary, the target alone) is (-inf, 0)
  auto join = [](float& top, float& sum, float m, float s) {
    const float to = fmaxf(top, m), base = to == -INFINITY ? 0.0f : to;
    sum = sum * __builtin_amdgcn_exp2f((top - base) * kLog2e) + s * __builtin_amdgcn_exp2f((m - base) * kLog2e);
    top = to;
  };
  if (t < tokens) {
#pragma unroll 4
    for (int64_t p = threadIdx.x / kMergeTokens; p < parts; p += kMergeWaves * 64 / kMergeTokens)
      join(top, sum, part[2 * p * tokens + t], part[(2 * p + 1) * tokens + t]);
  }
#pragma unroll
  for (int d = kMergeTokens; d < 64; d <<= 1) join(top, sum, __shfl_xor(top, d, 64), __shfl_xor(sum, d, 64));
  if (lane < kMergeTokens) {
    tops[wave][column] = top;
    sums[wave][column] = sum;
  }
  __syncthreads();
  if (threadIdx.x < kMergeTokens && t < tokens) {
#pragma unroll
    for (int w = 1; w < kMergeWaves; ++w) join(top, sum, tops[w][column], sums[w][column]);
    const float others = top + logf(sum);                     // a token that does not count: of all words
    float l = others, mine = 0.0f;
    if ((uint64_t)targets[t] < (uint64_t)vocab) {
      const float p = picked[t], d = (top - p) + logf(sum), more = log1pf(expf(-fabsf(d)));
      mine = d > 0.0f ? d + more : p == INFINITY ? NAN : more;
      l = d > 0.0f ? others + more : p + mine;
    }
    if (lse) lse[t] = l;
    if (loss) loss[t] = mine;
  }
}

// dx = BF16(sum of the shares, one after the other, + rest[t] W[target[t]])
__global__ __launch_bounds__(kThreads) void k_join_shares(const float* __restrict__ sums, int64_t slice, int shares, int64_t tokens,
                                                          int64_t hidden, const float* __restrict__ rest, const int64_t* __restrict__ targets,
                                                          const uint16_t* __restrict__ words, int64_t ldw, int64_t vocab,
                                                          uint16_t* __restrict__ dx, int64_t ld) {
  const int64_t vecs = hidden / 4, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= tokens * vecs) return;
  const int64_t t = id / vecs, c = (id - t * vecs) * 4, target = targets[t];
  const float* from = sums + t * hidden + c;
  v4f32 s = *reinterpret_cast<const v4f32*>(from);
  constexpr int kBatch = 8;                                   // shares on their way together
  for (int k = 1; k < shares; k += kBatch) {
    v4f32 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) v[b] = k + b < shares ? *reinterpret_cast<const v4f32*>(from + (k + b) * slice) : v4f32{};
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (k + b < shares) s += v[b];
  }
  if ((uint64_t)target < (uint64_t)vocab) {
    const float f = rest[t];
    const v2u32 w = *reinterpret_cast<const v2u32_any*>(words + target * ldw + c);
    if (f != 0.0f) s += v4f32{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)} * f;
  }
  *reinterpret_cast<v2u32_any*>(dx + t * ld + c) = v2u32{bf16_rn_pair(s.x, s.y), bf16_rn_pair(s.z, s.w)};
}

// by_word = the counted tokens in the order of (target, token), behind them the others; start[b] = the number of counted tokens with a
// target below 128 b, b = 0 .. buckets. A lane a token (a bound), its place the number of those before it; the workgroup's waves look
// through a share of the tokens each. Every token looks at every other: with 32768 words 6 us for 333 tokens, 30 for 8192, 0.33 ms
// for 32768, 3.9 ms for 131072 (with hidden 1024 one in seven of what the products take there), some 1 s at the limit of 2^21.
constexpr int kOrderWaves = 16;
__global__ __launch_bounds__(kOrderWaves * 64) void k_order(const int64_t* __restrict__ targets, int64_t tokens, int64_t vocab, int64_t buckets,
                                                            int* __restrict__ by_word, int* __restrict__ start) {
  __shared__ int64_t keys[kOrderWaves * 64];
  __shared__ int places[kOrderWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t groups = (tokens + 63) / 64, id = (blockIdx.x < groups ? blockIdx.x : blockIdx.x - groups) * 64 + lane;
  const bool bound = blockIdx.x >= groups;
  auto key_of = [&](int64_t t) { return (uint64_t)t < (uint64_t)vocab ? t : vocab; };
  const int64_t key = bound ? (id * kBucket < vocab ? id * kBucket : vocab) : id < tokens ? key_of(targets[id]) : 0;
  int before = 0;
  // a wave looks through 64 of each 1024 tokens; past the last one a key that is before no other
  int64_t next = (int64_t)threadIdx.x < tokens ? key_of(targets[threadIdx.x]) : INT64_MAX;
  for (int64_t t0 = 0; t0 < tokens; t0 += kOrderWaves * 64) {
    const int64_t t = t0 + kOrderWaves * 64 + threadIdx.x;
    keys[threadIdx.x] = next;                                 // the wave's own: read by no other
    next = t < tokens ? key_of(targets[t]) : INT64_MAX;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // equal keys: a bound counts none of them, a token those of the tokens before it
    const int64_t mine = bound ? 0 : id - (t0 + wave * 64);
#pragma unroll 16
    for (int k = 0; k < 64; ++k) {
      const int64_t other = keys[wave * 64 + k];
      before += (int)(other < key) | ((int)(other == key) & (int)(k < mine));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  places[wave][lane] = before;
  __syncthreads();
  if (wave != 0) return;
  int place = 0;
#pragma unroll
  for (int w = 0; w < kOrderWaves; ++w) place += places[w][lane];
  if (bound) {
    if (id <= buckets) start[id] = place;
  } else if (id < tokens) {
    by_word[place] = (int)id;
  }
}

// dw = 0 (no tokens)
__global__ __launch_bounds__(kThreads) void k_zero_rows(uint8_t* __restrict__ d, int64_t row_bytes, int64_t pitch, int64_t rows) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t i = (int64_t)threadIdx.x * 4; i < row_bytes; i += kThreads * 4) *reinterpret_cast<uint16_t*>(d + r * pitch + i) = 0, *reinterpret_cast<uint16_t*>(d + r * pitch + i + 2) = 0;
}

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
// The tile of a product of `rows_a` x `rows_b` results. Few: B's rows fit; bound by A's bytes. Full moves the least through LDS
// for an operation, and Half (two thirds of its rate at best, LDS bound) is taken where it leaves out a quarter of the
// products, those with rows that there are not: 50021 words, hidden 1040, 333 tokens (384 or 512 rows): 70 us against 83,
// 64 tokens: 26 against 38; 1003 tokens, no rows less: 242 against 203.
// Also where all of Full leave half the chip idle and the contraction is not cut (`cut`: dx's is): 2048 tokens, 4000 words, hidden
// 4096 (128 tiles): forward 66 us against 90; 700, 1500 and 512 (18 tiles): 19 against 31.
enum Tiling { kFull, kHalf, kFew };
Tiling tiling(int64_t rows_a, int64_t rows_b, bool few, bool cut) {
  if (few && rows_b <= Few::kN) return kFew;
  if (!cut && up(rows_a, 256) * up(rows_b, 256) <= 128 * 65536) return kHalf;
  return up(rows_a, 256) * up(rows_b, 256) * 3 >= up(rows_a, 128) * up(rows_b, 128) * 4 ? kHalf : kFull;
}

template <int EPI, bool TA, bool TB>
void product(const Rows& a, const Rows& b, int64_t K, int shares, const Out& o, hipStream_t stream) {
  auto go = [&](auto tile) {
    using C = decltype(tile);
    const int64_t tm = (a.rows + C::kM - 1) / C::kM, tn = (b.rows + C::kN - 1) / C::kN;
    hipLaunchKernelGGL((k_product<C, EPI, TA, TB>), dim3((unsigned)(tm * tn * shares)), dim3(kThreads), 0, stream, a, b, K, tm, tn, shares, o);
  };
  const Tiling t = tiling(a.rows, b.rows, !TB, TA && !TB);
  if constexpr (!TB) {
    if (t == kFew) return go(Few{});
  }
  if (t == kHalf) go(Half{});
  else go(Full{});
}

constexpr int64_t kPad = 64;
// Elements of a row of G: whole lines of 128 bytes, an odd number of them, so that rows under each other do not all fall on
// one channel of the memory.
int64_t odd_lines(int64_t v) { return ((v + kPad - 1) / kPad | 1) * kPad; }

// Rows that begin inside a line of 128 bytes cost the DMA two lines for a piece. Where hidden makes x's rows so, large products read a
// copy of x in whole lines (W would be too much to copy; where only x's stride makes them so, it stays): from 2^36 products on (8192 x 32768 x 5136: forward 2116 us
// against 2341, backward 6841 against 7114; 1003 x 32003 x 2704, at the limit: 185 and 191; 333 x 50021 x 1040, a quarter of
// it: 4 us less in whole lines, and the copy takes 5).
__global__ __launch_bounds__(kThreads) void k_realign(const uint16_t* __restrict__ x, int64_t ldx, int64_t tokens, int64_t hidden,
                                                      uint16_t* __restrict__ out, int64_t ld) {
  const int64_t vecs = hidden / 8, id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= tokens * vecs) return;
  const int64_t t = id / vecs, c = (id - t * vecs) * 8;
  *reinterpret_cast<v4u32*>(out + t * ld + c) = *reinterpret_cast<const v4u32*>(x + t * ldx + c);
}
bool realigned(int64_t T, int64_t V, int64_t H) { return H % kPad != 0 && (double)T * (double)V * (double)H >= 68719476736.0; }
size_t realigned_bytes(int64_t T, int64_t V, int64_t H) { return realigned(T, V, H) ? (size_t)up(T * odd_lines(H) * 2, 256) : 0; }
// x, or its copy at `place`.
Rows tokens_of(const uint16_t* x, int64_t ldx, int64_t T, int64_t V, int64_t H, void* place, hipStream_t stream) {
  if (!realigned(T, V, H) || ldx % kPad == 0) return Rows{x, T, ldx};
  const int64_t ld = odd_lines(H);
  uint16_t* copy = static_cast<uint16_t*>(place);
  hipLaunchKernelGGL(k_realign, dim3((unsigned)((T * (H / 8) + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, x, ldx, T, H, copy, ld);
  return Rows{copy, T, ld};
}

// Pairs (maximum, sum) that the forward's product leaves of each token.
int64_t pairs_of(int64_t T, int64_t V) {
  const Tiling t = tiling(V, T, true, false);
  return t == kFew ? up(V, Few::kM) / Few::kWaveM : t == kHalf ? up(V, Half::kM) / Half::kWaveM : up(V, Full::kM) / Full::kWaveM;
}

constexpr int64_t kPieceElements = int64_t(1) << 28;          // of G at a time: 512 MB in BF16
constexpr int64_t kMaxPiece = int64_t(1) << 20;               // row strides stay below 2^22 elements
constexpr int kMaxShares = 64;

struct BackwardPlan {
  int64_t piece, ld;            // words of a piece; row stride of G
  int shares;                   // of the contraction of dx
  size_t x, g, rest, by_word, start, sums, bytes;   // places in the workspace
  int64_t buckets;
};
BackwardPlan plan_backward(int64_t T, int64_t V, int64_t H) {
  BackwardPlan p;
  p.piece = kPieceElements / T / 256 * 256;
  if (p.piece > kMaxPiece) p.piece = kMaxPiece;
  if (p.piece < 256) p.piece = 256;
  if (p.piece > V) p.piece = V;
  p.ld = odd_lines(p.piece);
  // dx, whose tiles are few, is cut along its contraction: the rounds of tiles over the chip, each so many steps (1.5 us
  // of Full, 1 of two Halves, 0.5 of two Fews) and some 4 us around them, against writing and reading the shares' sums.
  const Tiling t = tiling(H, T, true, true);
  const int64_t side_n = t == kFew ? Few::kN : t == kHalf ? Half::kN : Full::kN, side_m = t == kHalf ? Half::kM : Full::kM;
  const int64_t tiles = up(H, side_m) / side_m * (up(T, side_n) / side_n), steps = up(p.piece, kStepK) / kStepK;
  const int64_t slots = t == kFull ? 256 : 512;
  const double step = t == kFull ? 1.5 : t == kHalf ? 1.0 : 0.5;
  auto cost = [&](int64_t k) {
    return (double)up(tiles * k, slots) / slots * (step * (double)(up(steps, k) / k) + 4.0) + (double)k * (double)T * (double)H * 8e-6 / 4.0;
  };
  p.shares = 1;
  for (int s = 2; s <= kMaxShares && s <= steps; ++s)
    if (cost(s) < cost(p.shares)) p.shares = s;
  size_t at = 0;
  auto take = [&](int64_t elements, int64_t size) {
    const size_t here = at;
    at += (size_t)up(elements * size, 256);
    return here;
  };
  p.x = take((int64_t)realigned_bytes(T, V, H), 1);
  p.g = take(T * p.ld, 2);
  p.rest = take(T, 4);
  p.buckets = up(V, kBucket) / kBucket;
  p.by_word = take(T, 4);
  p.start = take(p.buckets + 1, 4);
  p.sums = take(p.shares * T * H, 4);
  p.bytes = at;
  return p;
}

}  // namespace

size_t head_workspace_bytes(int64_t T, int64_t V, int64_t H) {
  if (T <= 0 || V <= 0) return 0;
  return realigned_bytes(T, V, H) + (size_t)(pairs_of(T, V) * 2 + 1) * (size_t)T * sizeof(float);
}

hipError_t launch_head_loss(const uint16_t* x, int64_t T, int64_t ldx, const uint16_t* w, int64_t V, int64_t ldw, int64_t H,
                            const int64_t* targets, float* loss, float* lse, void* ws, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  float* picked = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + realigned_bytes(T, V, H));
  Out o{};
  o.targets = targets;
  o.picked = picked;
  o.part = picked + T;
  product<kLse, false, false>(Rows{w, V, ldw}, tokens_of(x, ldx, T, V, H, ws, stream), H, 1, o, stream);
  hipLaunchKernelGGL(k_merge, dim3((unsigned)((T + kMergeTokens - 1) / kMergeTokens)), dim3(kMergeWaves * 64), 0, stream, o.part, pairs_of(T, V),
                     T, V, targets, picked, loss, lse);
  return hipGetLastError();
}

size_t head_grad_workspace_bytes(int64_t T, int64_t V, int64_t H) {
  return T <= 0 || V <= 0 ? 0 : plan_backward(T, V, H).bytes;
}

hipError_t launch_head_grad(const uint16_t* x, int64_t T, int64_t ldx, const uint16_t* w, int64_t V, int64_t ldw, int64_t H,
                            const int64_t* targets, const float* lse, const float* loss, const float* grad, uint16_t* dx, int64_t lddx, void* dw,
                            int dw_kind, int64_t lddw, void* ws, hipStream_t stream) {
  if (T == 0) {
    const int64_t size = dw_kind == kHeadBf16 ? 2 : 4;        // H is a multiple of 16
    if (dw && dw_kind != kHeadF32Add)
      hipLaunchKernelGGL(k_zero_rows, dim3((unsigned)(V < 2048 ? V : 2048)), dim3(kThreads), 0, stream, static_cast<uint8_t*>(dw), H * size,
                         lddw * size, V);
    return hipGetLastError();
  }
  const BackwardPlan p = plan_backward(T, V, H);
  uint8_t* base = static_cast<uint8_t*>(ws);
  uint16_t* g = reinterpret_cast<uint16_t*>(base + p.g);
  float *rest = reinterpret_cast<float*>(base + p.rest), *sums = reinterpret_cast<float*>(base + p.sums);
  int *by_word = reinterpret_cast<int*>(base + p.by_word), *start = reinterpret_cast<int*>(base + p.start);
  if (dw) hipLaunchKernelGGL(k_order, dim3((unsigned)((T + 63) / 64 + p.buckets / 64 + 1)), dim3(kOrderWaves * 64), 0, stream, targets, T, V,
                             p.buckets, by_word, start);
  const Rows tokens = tokens_of(x, ldx, T, V, H, base + p.x, stream);
  for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
    const int64_t n = V - v0 < p.piece ? V - v0 : p.piece;
    const Rows words{w + v0 * ldw, n, ldw};
    Out o{};
    o.targets = targets;
    o.lse = lse;
    o.grad = grad;
    o.loss = loss;
    o.rest = rest;
    o.first = v0;
    o.vocab = V;
    o.d = g;
    o.ld = p.ld;
    o.m_store = up(n, kPad);
    product<kGrad, false, false>(words, tokens, H, 1, o, stream);
    if (dx) {
      Out d{};
      d.d = sums;
      d.ld = H;
      d.m_store = H;
      d.slice = T * H;
      const Rows a{words.p, H, ldw}, b{g, T, p.ld};
      if (v0 == 0) product<kStoreF32, true, false>(a, b, n, p.shares, d, stream);
      else product<kAddF32, true, false>(a, b, n, p.shares, d, stream);
    }
    if (dw) {
      Out d{};
      d.targets = targets;
      d.first = v0;
      d.rest = rest;
      d.by_word = by_word;
      d.start = start;
      d.buckets = p.buckets;
      d.ld = lddw;
      d.m_store = H;
      const Rows a{tokens.p, H, tokens.ld}, b{g, n, p.ld};
      if (dw_kind == kHeadBf16) {
        d.d = static_cast<uint16_t*>(dw) + v0 * lddw;
        product<kStoreBf16, true, true>(a, b, T, 1, d, stream);
      } else {
        d.d = static_cast<float*>(dw) + v0 * lddw;
        if (dw_kind == kHeadF32Add) product<kAddF32, true, true>(a, b, T, 1, d, stream);
        else product<kStoreF32, true, true>(a, b, T, 1, d, stream);
      }
    }
  }
  if (dx) hipLaunchKernelGGL(k_join_shares, dim3((unsigned)((T * (H / 4) + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, sums, T * H,
                             p.shares, T, H, rest, targets, w, ldw, V, dx, lddx);
  return hipGetLastError();
}

}  // namespace nvfp4
