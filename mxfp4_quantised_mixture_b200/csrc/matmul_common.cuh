// What the MXFP4 product kernels share: arguments, tile order, the scale bytes'
// way from global to shared memory, and the output stores.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"
#include "groups.cuh"
#include "mlp_plan.cuh"
#include "tc_sm100.cuh"

namespace moe {
namespace mm {

constexpr int BKB = 128;            // code bytes per row and stage: 256 k
constexpr int kStepsPerStage = 4;   // MMAs of 64 k per stage
constexpr int kStagesPerChunk = 4;  // scale chunk: 1024 k, 8 words of 4 scales
constexpr int kWords = 2 * kStagesPerChunk;
constexpr int kWordBytes = 512;     // one scale word of 128 rows, in tcgen05.cp's order
constexpr int kChunkSlots = 2;
constexpr int kMaxStages = 8;
constexpr int kTableBytes = 4 * (kMaxGroups + 2) * 4;  // group table
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kTestWaitNs = 200000ull;  // the injected wait of test_timeout_cta
constexpr int64_t kMaxTiles = (int64_t(1) << 31) - (1 << 16);  // tile numbers, and a grid past them

enum Mode : int { kDense = 0, kGrouped = 1, kWgrad = 2 };

// How the output is stored, a template argument of the kernels: with all three
// ways in one kernel the epilogue's instruction fetches took a fifth of the
// weight gradient's time (32 experts of 2880 x 2880, 32768
// rows: 328 against 273 us in fp32, 297 against 231 in bf16).
enum Out : int { kFp32 = 0, kBf16Pairs = 1, kBf16 = 2 };  // pairs: rows of even length

struct Args {
  int mode, E;
  FastDiv xt, yt;          // tiles along B's rows, and along A's
  int split;               // CTAs of a cluster that share a tile's k range, 1 for none
  const int32_t* offsets;  // grouped, wgrad
  const uint8_t* xs;       // scales of B, [rows][ks]
  const uint8_t* ys;       // scales of A, [rows][ks]
  int64_t x_rows;          // n of the output (per group where B has groups)
  int64_t y_rows;          // rows of A
  int64_t x_total;         // rows of B over all groups
  int64_t K;               // contraction length (wgrad: its padded capacity)
  int64_t S;               // bound of the offsets' values
  float alpha;
  void* out;
  int32_t* status;
  int fail_cta = -1;  // testing: this CTA's first wait gives up
};

// One output tile: B rows [x0, ..) (of matrix e where B has groups), A rows
// [y0, y0 + ny), k in [k0, k0 + 64 steps), first output row out_row.
struct Work {
  int64_t out_row;
  int x0, y0, k0;
  int e, ny, steps;
};

// Every group's first unit (tile of A rows, or 128 positions), first row and
// rows, in shared memory.
struct Groups {
  int *pfx, *lo, *n, *width;  // width: rows of a tile
};

__device__ __forceinline__ Groups group_table(void* at) {
  Groups g;
  g.pfx = static_cast<int*>(at);
  g.lo = g.pfx + kMaxGroups + 2;
  g.n = g.lo + kMaxGroups + 2;
  g.width = g.n + kMaxGroups + 2;
  return g;
}

__device__ __forceinline__ void abort_cta(volatile int* abort, int32_t* status) {
  *abort = 1;
  record_status(status, MOE_ERR_TIMEOUT);
}

// Every lane of a converged warp waits for a phase; the answer is the same in
// all of them.  CLUSTER: the other CTA arrives at the barrier too.
template <bool CLUSTER = false>
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         int32_t* status) {
  if (__all_sync(0xFFFFFFFFu, tc::mbar_wait<CLUSTER>(bar, parity, abort, kWaitLimitNs))) return true;
  abort_cta(abort, status);
  return false;
}

// Testing only: in CTA a.fail_cta the warp waits, briefly, on a barrier that
// nothing completes, and gives up as a timeout would.  False once it has.
__device__ __forceinline__ bool injected_timeout(const Args& a, uint64_t* never, volatile int* abort) {
  if (static_cast<int>(blockIdx.x) != a.fail_cta) return true;
  if (__all_sync(0xFFFFFFFFu, tc::mbar_wait(never, 0, abort, kTestWaitNs))) return true;
  abort_cta(abort, a.status);
  return false;
}

// A whole warp waits: lane 0 polls (sleeping sleep_ns between polls: a spinning
// warp takes issue slots and shared-memory turns from the one thread that
// issues the MMAs), then every lane takes the completed phase with a poll of
// its own for the acquire ordering.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int32_t* status, uint32_t sleep_ns) {
  bool r = true;
  if ((threadIdx.x & 31) == 0) r = tc::mbar_wait_sleep(bar, parity, abort, kWaitLimitNs, sleep_ns);
  r = __shfl_sync(0xFFFFFFFFu, r, 0);
  if (r) {
    bool mine = tc::mbar_try_wait(bar, parity);
    for (int k = 0; k < 1024 && !mine; ++k) mine = tc::mbar_try_wait(bar, parity);
    r = __all_sync(0xFFFFFFFFu, mine);
  }
  if (!r) abort_cta(abort, status);
  return r;
}

// Even split of n rows into tiles of at most NT: the width of each, a multiple
// of STEP (as NT is).
template <int NT, int STEP>
__device__ __forceinline__ int tile_width(int n) {
  const int t = (n + NT - 1) / NT;
  return t == 0 ? STEP : ((n + t - 1) / t + STEP - 1) / STEP * STEP;
}

// Tiles are numbered with the B side fastest, so the CTAs running at one time
// share a few tiles of A rows.  `e` is the caller's cursor over the groups:
// its tiles' numbers only rise.
template <int NT, int STEP, int BX>
__device__ __forceinline__ Work work_of(const Args& a, const Groups& g, uint32_t i, int& e) {
  Work w;
  uint32_t u = i / a.xt;
  w.x0 = static_cast<int>(i - u * a.xt.d) * BX;
  w.k0 = 0;
  w.steps = static_cast<int>((a.K + 63) / 64);
  int lo = 0, n = static_cast<int>(a.y_rows), width = g.width[kMaxGroups];
  if (a.mode == kGrouped) {
    while (static_cast<int>(u) >= g.pfx[e + 1]) ++e;
    u -= g.pfx[e];
    lo = g.lo[e];
    n = g.n[e];
    width = g.width[e];
  } else if (a.mode == kWgrad) {
    e = static_cast<int>(u / a.yt);
    u -= e * a.yt.d;
    // never past the capacity, whatever the offsets hold
    const int64_t k0 = static_cast<int64_t>(g.pfx[e]) * kGroupAlign;
    const int64_t room = a.K - k0;
    const int64_t len = room < 0 ? 0 : (g.n[e] < room ? g.n[e] : room);
    w.k0 = len > 0 ? static_cast<int>(k0) : 0;
    w.steps = static_cast<int>((len + 63) / 64);
  }
  w.e = e;
  w.y0 = lo + static_cast<int>(u) * width;
  w.ny = min(width, lo + n - w.y0);
  w.out_row = w.y0 + (a.mode == kWgrad ? static_cast<int64_t>(e) * a.y_rows : 0);
  return w;
}

// 32 scale bytes (a chunk of a row) from address p of an array that ends at
// `end`, as eight words; bytes from `n` on read as 0 (their codes are zero).
// Rows start at any byte, so the chunk is read as the three aligned 16-byte
// pieces that cover it and shifted into place.
struct Pieces {
  uint4 v[3];
};

__device__ __forceinline__ bool past_end(const uint8_t* p, int n, const uint8_t* end) {
  const uint8_t* last = p + n - 1;  // the piece of the last byte ends behind the array
  return n > 0 && last - (reinterpret_cast<uintptr_t>(last) & 15u) + 16 > end;
}

__device__ __forceinline__ Pieces load_pieces(const uint8_t* p, int n, const uint8_t* end) {
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint4* a0 = reinterpret_cast<const uint4*>(p - mis);
  const bool all = !past_end(p, n, end);
  Pieces r;
#pragma unroll
  for (int j = 0; j < 3; ++j)
    r.v[j] = all && n > 0 && 16 * j < mis + n ? __ldg(a0 + j) : make_uint4(0u, 0u, 0u, 0u);
  return r;
}

static __device__ __noinline__ void load_bytes(const uint8_t* p, int n, uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = 0u;
    for (int j = 4 * i; j < n && j < 4 * i + 4; ++j)
      w[i] |= static_cast<uint32_t>(__ldg(p + j)) << (8 * (j & 3));
  }
}

__device__ __forceinline__ void align_words(const Pieces& r, const uint8_t* p, int n, uint32_t (&w)[8]) {
  uint32_t x[12];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    x[4 * j] = r.v[j].x;
    x[4 * j + 1] = r.v[j].y;
    x[4 * j + 2] = r.v[j].z;
    x[4 * j + 3] = r.v[j].w;
  }
  const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
#pragma unroll
  for (int i = 0; i < 11; ++i) x[i] = mis & 4u ? x[i + 1] : x[i];
#pragma unroll
  for (int i = 0; i < 9; ++i) x[i] = mis & 8u ? x[i + 2] : x[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], (mis & 3u) * 8);
  if (n < 32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int left = n - 4 * i;
      if (left < 4) w[i] = left > 0 ? w[i] & ((1u << (8 * left)) - 1u) : 0u;
    }
  }
}

// 16 accumulator columns of this lane's output column, times alpha, to p, p +
// ld, ... (elements).  ALL: every row exists (else the first ny do).
template <bool F32, bool ALL>
__device__ __forceinline__ void store16(const uint32_t (&r)[16], float alpha, void* p, uint32_t ld, int ny) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float v = alpha * __uint_as_float(r[k]);
    if (ALL || k < ny) {
      const uint64_t at = static_cast<uint64_t>(k) * ld;
      if (F32)
        static_cast<float*>(p)[at] = v;
      else
        static_cast<uint16_t*>(p)[at] = static_cast<uint16_t>(cvt_bf16x2(v, 0.f));
    }
  }
}

// The same in bf16 for an even ld: two rows are packed, then neighbouring lanes
// swap halves, so each lane stores two output columns of every second row: half
// the stores.  p is the lane's own row and column (odd lanes: the next row, the
// column before).
template <bool ALL>
__device__ __forceinline__ void store16_pairs(const uint32_t (&r)[16], float alpha, char* p, uint32_t ld2,
                                              int ny) {
  const int odd = threadIdx.x & 1;
  const uint32_t pick = odd ? 0x3276u : 0x5410u;  // the other's high half and mine, or my low half and its
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t own = cvt_bf16x2(alpha * __uint_as_float(r[2 * k]), alpha * __uint_as_float(r[2 * k + 1]));
    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
    if (ALL || 2 * k + odd < ny)
      *reinterpret_cast<uint32_t*>(p + static_cast<uint64_t>(k) * 2 * ld2) = __byte_perm(own, got, pick);
  }
}

// Columns [c0, c1) of a tile's accumulator (a multiple of 16 of them, the last
// ones possibly past its ny rows), to output column n.
template <int OUT>
__device__ __forceinline__ void store_columns(uint32_t acc, const Args& a, const Work& w, int64_t n,
                                              int c0, int c1) {
  constexpr int kSize = OUT == kFp32 ? 4 : 2;
  const bool live = n < a.x_rows;
  const uint32_t ld = static_cast<uint32_t>(a.x_rows);
  char* p = static_cast<char*>(a.out) + ((w.out_row + c0) * a.x_rows + n) * kSize;
  if (OUT == kBf16Pairs && (threadIdx.x & 1)) p += static_cast<int64_t>(ld) * 2 - 2;
  const int64_t step = static_cast<int64_t>(16) * ld * kSize;
  uint32_t r[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) r[k] = 0u;  // an empty sum, if nothing is loaded
#pragma unroll 1
  for (int c = c0; c < c1; c += 16) {
    if (w.steps > 0) {
      tc::tmem_ld16(acc + c, r);
      tc::tmem_ld_wait();
    }
    const int ny = live ? w.ny - c : 0;
    if (__all_sync(0xFFFFFFFFu, ny >= 16)) {
      if (OUT == kBf16Pairs)  // lanes 2j, 2j + 1 exist together
        store16_pairs<true>(r, a.alpha, p, 2 * ld, ny);
      else
        store16<OUT == kFp32, true>(r, a.alpha, p, ld, ny);
    } else {
      if (OUT == kBf16Pairs)
        store16_pairs<false>(r, a.alpha, p, 2 * ld, ny);
      else
        store16<OUT == kFp32, false>(r, a.alpha, p, ld, ny);
    }
    p += step;
  }
}

// The group table, by one whole warp (NT rows of A to a tile).
template <int NT, int STEP>
__device__ __forceinline__ void fill_groups(const Args& a, const Groups& g) {
  if ((threadIdx.x & 31) == 0) g.width[kMaxGroups] = tile_width<NT, STEP>(static_cast<int>(a.y_rows));
  if (a.mode == kDense) return;
  group_prefix(a.E, g.pfx, [&](int e) {
    int64_t lo, hi;
    group_rows(a.offsets, e, a.S, lo, hi);
    const int n = static_cast<int>(hi - lo);
    g.lo[e] = static_cast<int>(lo);
    g.n[e] = n;
    g.width[e] = tile_width<NT, STEP>(n);
    return a.mode == kGrouped ? (n + NT - 1) / NT : (n + kGroupAlign - 1) / kGroupAlign;
  });
}

// Number of tiles of BX rows of B by up to NT rows of A.
__device__ __forceinline__ uint32_t tiles(const Args& a, const Groups& g) {
  return a.xt.d * (a.mode == kDense ? a.yt.d : (a.mode == kGrouped ? g.pfx[a.E] : a.yt.d * a.E));
}

// Host side of the same: the two tile counts into the arguments, and an upper
// bound of the number of tiles.
inline int64_t plan_tiles(Args* a, int bx, int nt) {
  const int64_t xt = (a->x_rows + bx - 1) / bx, yt = (a->y_rows + nt - 1) / nt;
  a->xt = fast_div(static_cast<uint32_t>(xt));
  a->yt = fast_div(static_cast<uint32_t>(yt));
  return xt * (a->mode == kDense ? yt : (a->mode == kGrouped ? yt + a->E : yt * a->E));
}

// Stages and scale chunks of a tile.
__device__ __forceinline__ int stages_of(const Work& w) {
  return (w.steps + kStepsPerStage - 1) / kStepsPerStage;
}
__device__ __forceinline__ int chunks_of(const Work& w) {
  return (stages_of(w) + kStagesPerChunk - 1) / kStagesPerChunk;
}

// One tile's scale rows of a 128-row block: from its first row (of this lane,
// at the tile's first k) to the end of the array.
struct ScaleBlock {
  const uint8_t *base, *end;
  int rows, left;  // rows that exist; bytes of a row from the tile's first k
};

// blk 0: the B rows from x0; blk 1, 2: the A rows in steps of 128.
__device__ __forceinline__ ScaleBlock scale_block(const Args& a, const Work& w, int blk, int x0, int ks) {
  ScaleBlock b;
  const uint8_t* all = blk == 0 ? a.xs : a.ys;
  const int64_t row0 = blk == 0 ? x0 + (a.mode == kGrouped ? w.e * a.x_rows : 0)
                                : static_cast<int64_t>(w.y0) + (blk - 1) * 128;
  b.base = all + (row0 + (threadIdx.x & 31)) * ks + w.k0 / 32;
  b.end = all + (blk == 0 ? a.x_total : a.y_rows) * ks;
  b.rows = blk == 0 ? static_cast<int>(min(a.x_rows - x0, static_cast<int64_t>(128)))
                    : w.ny - (blk - 1) * 128;
  b.left = ks - w.k0 / 32;
  return b;
}

// Chunk q of a block, by one warp: lane l carries the 32 bytes of rows l, l +
// 32, l + 64 and l + 96, which are the 16 bytes of row l of tcgen05.cp's order
// for each of the 8 words.  `ready` is asked once, before the first store.
template <int ROWS, typename Ready>
__device__ __forceinline__ bool move_chunk(const ScaleBlock& b, int q, int ks, uint8_t* dst, Ready ready) {
  const int lane = threadIdx.x & 31;
  const int byte = q * kWords * 4;
  const int n = min(32, b.left - byte);
#pragma unroll
  for (int c0 = 0; c0 < 4; c0 += ROWS) {
    const uint8_t* p = b.base + byte + c0 * 32 * ks;
    Pieces raw[ROWS];
#pragma unroll
    for (int c = 0; c < ROWS; ++c)
      raw[c] = load_pieces(p + c * 32 * ks, lane + 32 * (c0 + c) < b.rows ? n : 0, b.end);
    uint32_t v[ROWS][8];
#pragma unroll
    for (int c = 0; c < ROWS; ++c) {
      const int nr = lane + 32 * (c0 + c) < b.rows ? n : 0;
      align_words(raw[c], p + c * 32 * ks, nr, v[c]);
      if (past_end(p + c * 32 * ks, nr, b.end)) load_bytes(p + c * 32 * ks, nr, v[c]);
    }
    if (c0 == 0 && !ready()) return false;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      uint8_t* at = dst + k * kWordBytes + lane * 16 + c0 * 4;
      if constexpr (ROWS == 4)
        *reinterpret_cast<uint4*>(at) = make_uint4(v[0][k], v[1][k], v[2][k], v[3][k]);
      else
        *reinterpret_cast<uint2*>(at) = make_uint2(v[0][k], v[1][k]);
    }
  }
  return true;
}

// Tensor map of packed codes: rows of `row` bytes, boxes of 128 bytes x box_rows.
inline bool encode_codes(CUtensorMap* map, const void* base, int64_t row, int64_t rows, int64_t mats,
                         int box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(mats)};
  const cuuint64_t strides[2] = {dims[0], dims[0] * dims[1]};
  const cuuint32_t box[3] = {BKB, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The way to store rows of x_rows elements of a type.
inline Out out_of(int out_type, int64_t x_rows) {
  return out_type == MOE_OUT_FP32 ? kFp32 : (x_rows % 2 == 0 ? kBf16Pairs : kBf16);
}

// The two-CTA kernel (csrc/matmul_pair.cu).
moe_status launch_pair(const Args& a, int out_type, const uint8_t* xq, const uint8_t* yq,
                       cudaStream_t stream);

}  // namespace mm
}  // namespace moe
