// Products of two MXFP4 matrices on the tensor core, whole or in groups of rows.
//
// "MXFP4-based MoE technical review", section 2 (MXFP4 training: every product
// on block-scaled operands); "Tricks from OpenAI gpt-oss ..." (summary),
// section 8 (GEMMs that read the E2M1 blocks and their scales directly).
//   dense    out[m][n]    = alpha sum_k A[m][k] B[n][k]
//   grouped  out[r][n]    = alpha sum_k A[r][k] B[e][n][k], r a row of group e
//   wgrad    out[e][m][n] = alpha sum_p A[m][p] B[n][p], p a position of group e
//
// Both operands stay packed (two codes to a byte) from HBM to the tensor core:
// kind::mxf4 MMAs multiply E2M1 codes and apply the two E8M0 scales of every
// 32-wide block themselves, accumulating in fp32.
//
// Orientation: the B side (the output's contiguous axis n) takes the MMA's M =
// 128 lanes and the A side its N columns, up to NT of them and only as many as
// the tile has rows.  An accumulator lane then is one output column, so a
// warp's stores are contiguous with no staging, and a decode batch of a few
// rows costs the tensor core only those rows.
//
// Persistent, one CTA per SM (two for the narrow tiles).  Warp roles:
//   warp 0      producer: per stage of 256 k, 128 x 128 bytes of B codes and
//               NT x 128 bytes of A codes by TMA (zeros past the ends)
//   warp 1      tensor-memory owner and MMA issuer; it also copies each stage's
//               scale words from shared to tensor memory (tcgen05.cp)
//   scale loaders (4 or 6 warps): E8M0 bytes from global memory, in chunks of
//               1024 k (32 bytes of a row), laid down in shared memory in the
//               order tcgen05.cp takes them
//   epilogue (4 or 8 warps), one or two per lane quarter, from a
//               double-buffered accumulator, so it overlaps the next tile's MMAs
// Every wait is bounded (2 s); on expiry the kernel records MOE_ERR_TIMEOUT,
// waits for its own copies and MMAs to finish and returns.
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "groups.cuh"
#include "mlp_plan.cuh"
#include "tc_sm100.cuh"

namespace moe {
namespace {

constexpr int BX = 128;                  // B rows per tile (MMA M)
constexpr int BKB = 128;                 // code bytes per row and stage: 256 k
constexpr int kStepsPerStage = 4;        // MMAs of 64 k per stage
constexpr int kStagesPerChunk = 4;       // scale chunk: 1024 k, 8 words of 4 scales
constexpr int kWords = 2 * kStagesPerChunk;
constexpr int X_BYTES = BX * BKB;
constexpr int kWordBytes = 512;  // one scale word of 128 rows, in tcgen05.cp's order
constexpr int kTableBytes = 3 * (kMaxGroups + 2) * 4;  // group table
constexpr int kMaxStages = 8;
constexpr int kChunkSlots = 2;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Warps: producer, MMA issuer, scale loaders, epilogue.  The wide tiles, one
// CTA per SM, take two warps of the epilogue per lane quarter.
__host__ __device__ constexpr int y_blocks(int NT) { return (NT + 127) / 128; }
__host__ __device__ constexpr int ctas_per_sm(int NT) { return NT <= 64 ? 2 : 1; }
__host__ __device__ constexpr int scale_warps(int NT) { return 2 * (1 + y_blocks(NT)); }
__host__ __device__ constexpr int epi_warps(int NT) { return NT > 64 ? 8 : 4; }
__host__ __device__ constexpr int threads(int NT) {
  return 32 * (2 + scale_warps(NT) + epi_warps(NT));
}

enum Mode : int { kDense = 0, kGrouped = 1, kWgrad = 2 };

__host__ __device__ constexpr int acc_cols(int NT) { return NT < 32 ? 32 : NT; }
__host__ __device__ constexpr int sf_cols(int NT) { return 2 * 4 * (1 + y_blocks(NT)); }
__host__ __device__ constexpr int tmem_cols(int NT) {
  const int need = 2 * acc_cols(NT) + 2 * sf_cols(NT);
  return need <= 128 ? 128 : (need <= 256 ? 256 : 512);
}
__host__ __device__ constexpr int stage_bytes(int NT) { return X_BYTES + NT * BKB; }
__host__ __device__ constexpr int chunk_bytes(int NT) { return kWords * (1 + y_blocks(NT)) * kWordBytes; }
__host__ __device__ constexpr int stages(int NT) {
  const int room = (ctas_per_sm(NT) == 2 ? 112 : 226) * 1024 - 1024 - 512 - kTableBytes -
                   kChunkSlots * chunk_bytes(NT);
  const int n = room / stage_bytes(NT);
  return n < kMaxStages ? n : kMaxStages;
}
__host__ __device__ constexpr int smem_bytes(int NT) {
  return 1024 + stages(NT) * stage_bytes(NT) + kChunkSlots * chunk_bytes(NT) + kTableBytes + 512;
}

struct Args {
  int mode, E;
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
  int out_f32;
  int32_t* status;
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
  int *pfx, *lo, *n;
};

// two fp32 -> bf16x2, round to nearest even (lo in the low half)
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void abort_cta(volatile int* abort, int32_t* status) {
  *abort = 1;
  record_status(status, MOE_ERR_TIMEOUT);
}

__device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity, volatile int* abort,
                                      int32_t* status) {
  if (tc::mbar_wait(bar, parity, abort, kWaitLimitNs)) return true;
  abort_cta(abort, status);
  return false;
}

// A whole warp waits: lane 0 polls, then every lane takes the completed phase
// with a poll of its own for the acquire ordering.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int32_t* status) {
  bool r = true;
  if ((threadIdx.x & 31) == 0) r = tc::mbar_wait(bar, parity, abort, kWaitLimitNs);
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
// of 16 (the MMA's N step).
template <int NT>
__device__ __forceinline__ int tile_width(int n) {
  const int t = (n + NT - 1) / NT;
  return t == 0 ? 16 : ((n + t - 1) / t + 15) / 16 * 16;
}

// Tiles are numbered with the B side fastest, so the CTAs running at one time
// share a few tiles of A rows.  `e` is the caller's cursor over the groups:
// its tiles' numbers only rise.
template <int NT>
__device__ __forceinline__ Work work_of(const Args& a, const Groups& g, uint32_t xt, uint32_t yt,
                                        uint32_t i, int& e) {
  Work w;
  uint32_t u = i / xt;
  w.x0 = static_cast<int>(i - u * xt) * BX;
  w.k0 = 0;
  w.steps = static_cast<int>((a.K + 63) / 64);
  int lo = 0, n = static_cast<int>(a.y_rows);
  if (a.mode == kGrouped) {
    while (static_cast<int>(u) >= g.pfx[e + 1]) ++e;
    u -= g.pfx[e];
    lo = g.lo[e];
    n = g.n[e];
  } else if (a.mode == kWgrad) {
    e = static_cast<int>(u / yt);
    u -= e * yt;
    // never past the capacity, whatever the offsets hold
    const int64_t k0 = static_cast<int64_t>(g.pfx[e]) * kGroupAlign;
    const int64_t room = a.K - k0;
    const int64_t len = room < 0 ? 0 : (g.n[e] < room ? g.n[e] : room);
    w.k0 = len > 0 ? static_cast<int>(k0) : 0;
    w.steps = static_cast<int>((len + 63) / 64);
  }
  const int width = tile_width<NT>(n);
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

__device__ __noinline__ void load_bytes(const uint8_t* p, int n, uint32_t (&w)[8]) {
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

// 16 accumulator columns (output rows row0 + c, c < ny - c0) of this lane's
// output column n, times alpha, into out.
template <bool F32>
__device__ __forceinline__ void store16(const uint32_t (&r)[16], float alpha, void* out, int64_t row,
                                        int64_t ld, int64_t n, bool live, int ny) {
  if (F32) {
    float* p = static_cast<float*>(out) + row * ld + n;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (live && k < ny) *p = alpha * __uint_as_float(r[k]);
      p += ld;
    }
  } else if ((ld & 1) == 0) {
    // neighbouring lanes swap halves of a column pair, so each stores two
    // output columns of one row: half the stores
    const int odd = threadIdx.x & 1;
    uint16_t* p = static_cast<uint16_t*>(out) + (row + odd) * ld + (n - odd);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const float v0 = alpha * __uint_as_float(r[k]), v1 = alpha * __uint_as_float(r[k + 1]);
      const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 1);
      const uint32_t packed = odd ? cvt_bf16x2(got, v1) : cvt_bf16x2(v0, got);
      if (live && k + odd < ny) *reinterpret_cast<uint32_t*>(p) = packed;
      p += 2 * ld;
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(out) + row * ld + n;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float v = alpha * __uint_as_float(r[k]);
      if (live && k < ny) *p = static_cast<uint16_t>(cvt_bf16x2(v, v));
      p += ld;
    }
  }
}

// Columns [c0, c1) of a tile's accumulator (a multiple of 16 of them, the last
// ones possibly past its ny rows).
template <bool F32>
__device__ __forceinline__ void store_columns(uint32_t acc, const Args& a, const Work& w, int64_t n,
                                              int c0, int c1) {
  const bool live = n < a.x_rows;
  for (int c = c0; c < c1; c += 32) {
    uint32_t r[2][16];
    const bool two = c + 16 < c1;
    if (w.steps > 0) {
      tc::tmem_ld16(acc + c, r[0]);
      if (two) tc::tmem_ld16(acc + c + 16, r[1]);
      tc::tmem_ld_wait();
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) r[0][k] = r[1][k] = 0u;  // an empty sum
    }
    store16<F32>(r[0], a.alpha, a.out, w.out_row + c, a.x_rows, n, live, w.ny - c);
    if (two) store16<F32>(r[1], a.alpha, a.out, w.out_row + c + 16, a.x_rows, n, live, w.ny - c - 16);
  }
}

template <int NT>
__global__ void __launch_bounds__(threads(NT), ctas_per_sm(NT))
    mxfp4_matmul_kernel(const __grid_constant__ CUtensorMap map_x,
                        const __grid_constant__ CUtensorMap map_y, const Args a) {
  constexpr int NS = stages(NT), STAGE = stage_bytes(NT), YB = y_blocks(NT);
  constexpr int ACC = acc_cols(NT), SF = sf_cols(NT), TMEM = tmem_cols(NT);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* chunks = smem + NS * STAGE;
  constexpr int kEpi = epi_warps(NT), kEpi0 = 2 + scale_warps(NT);
  Groups grp;
  grp.pfx = reinterpret_cast<int*>(chunks + kChunkSlots * chunk_bytes(NT));
  grp.lo = grp.pfx + kMaxGroups + 2;
  grp.n = grp.lo + kMaxGroups + 2;
  uint64_t* full = reinterpret_cast<uint64_t*>(grp.n + kMaxGroups + 2);  // [NS] stage copies landed
  uint64_t* empty = full + kMaxStages;     // [NS] stage MMAs complete
  uint64_t* sfull = empty + kMaxStages;    // [2] scale chunk written
  uint64_t* sempty = sfull + kChunkSlots;  // [2] scale chunk read
  uint64_t* dfull = sempty + kChunkSlots;  // [2] accumulator complete
  uint64_t* dempty = dfull + 2;            // [2] accumulator read
  uint64_t* drain = dempty + 2;            // every MMA issued has completed
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kChunkSlots; ++s) {
      tc::mbar_init(&sfull[s], 1 + YB);
      tc::mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&dfull[b], 1);
      tc::mbar_init(&dempty[b], kEpi);
    }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_y);
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_holder, TMEM);
    tc::tmem_relinquish();
  }
  if (warp == 2 && a.mode != kDense)
    group_prefix(a.E, grp.pfx, [&](int e) {
      int64_t lo, hi;
      group_rows(a.offsets, e, a.S, lo, hi);
      const int n = static_cast<int>(hi - lo);
      grp.lo[e] = static_cast<int>(lo);
      grp.n[e] = n;
      return a.mode == kGrouped ? (n + NT - 1) / NT : (n + kGroupAlign - 1) / kGroupAlign;
    });
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t xt = static_cast<uint32_t>((a.x_rows + BX - 1) / BX);
  const uint32_t yt = static_cast<uint32_t>((a.y_rows + NT - 1) / NT);
  const uint32_t n_work =
      xt * (a.mode == kDense ? yt : (a.mode == kGrouped ? grp.pfx[a.E] : yt * a.E));
  const int ks = static_cast<int>(a.K / 32);
  int ge = 0;  // this role's cursor over the groups

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t g = 0;
      bool ok = true;
      for (uint32_t i = blockIdx.x; ok && i < n_work; i += gridDim.x) {
        const Work w = work_of<NT>(a, grp, xt, yt, i, ge);
        const int nst = (w.steps + kStepsPerStage - 1) / kStepsPerStage;
        for (int st = 0; st < nst; ++st, ++g) {
          const uint32_t s = g % NS, n = g / NS;
          if (n > 0 && !wait1(&empty[s], (n - 1) & 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + s * STAGE;
          const int kb = w.k0 / 2 + st * BKB;
          tc::mbar_arrive_expect_tx(&full[s], STAGE);
          tc::tma_load_3d(dst, &map_x, &full[s], kb, w.x0,
                          a.mode == kGrouped ? w.e : 0);
          tc::tma_load_2d(dst + X_BYTES, &map_y, &full[s], kb, w.y0);
        }
      }
      // every copy this thread issued has landed before the CTA exits
      for (uint32_t i = g > NS ? g - NS : 0; i < g; ++i)
        tc::mbar_drain(&full[i % NS], (i / NS) & 1, kWaitLimitNs / 8);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      uint32_t g = 0, ch = 0, it = 0;
      bool ok = true;
      for (uint32_t i = blockIdx.x; ok && i < n_work; i += gridDim.x, ++it) {
        const Work w = work_of<NT>(a, grp, xt, yt, i, ge);
        const uint32_t idesc = tc::idesc_mxf4(BX, (w.ny + 15) & ~15);
        const uint32_t d = tmem + (it & 1) * ACC;
        // accumulator it & 1 was last used by tile it - 2
        if (it >= 2 && !wait1(&dempty[it & 1], ((it >> 1) - 1) & 1, abort_flag, a.status)) break;
        const int nst = (w.steps + kStepsPerStage - 1) / kStepsPerStage;
        for (int st = 0; st < nst; ++st, ++g) {
          const int cw = st % kStagesPerChunk;
          const uint32_t cs = ch % kChunkSlots;
          if (cw == 0 && !wait1(&sfull[cs], (ch / kChunkSlots) & 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          // the tensor-memory scale columns of stage g were last read by stage g - 2
          if (g >= 2) {
            const uint32_t p = g - 2;
            if (!wait1(&empty[p % NS], (p / NS) & 1, abort_flag, a.status)) {
              ok = false;
              break;
            }
          }
          const uint32_t s = g % NS;
          if (!wait1(&full[s], (g / NS) & 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t sf = tmem + 2 * ACC + (g & 1) * SF;
          const uint32_t chunk = tc::smem_u32(chunks + cs * chunk_bytes(NT));
          // columns: [word 0: X, Y blocks][word 1: X, Y blocks], 4 columns a block
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < 1 + YB; ++b)
              tc::tmem_cp_32x128b(sf + (h * (1 + YB) + b) * 4,
                                  tc::smem_desc_rows16(chunk + (b * kWords + cw * 2 + h) * kWordBytes));
          const uint64_t xd = tc::smem_desc_sw128(tc::smem_u32(smem + s * STAGE));
          const uint64_t yd = tc::smem_desc_sw128(tc::smem_u32(smem + s * STAGE + X_BYTES));
          const int left = w.steps - st * kStepsPerStage;
#pragma unroll
          for (int k = 0; k < kStepsPerStage; ++k) {
            if (k >= left) break;
            const uint32_t sx = sf + (k >> 1) * (1 + YB) * 4, id = (k & 1) * 2;
            // a descriptor addresses shared memory in 16-byte units: +2 per 64 codes
            tc::mma_mxf4_ss(d, xd + 2 * k, yd + 2 * k, idesc | tc::idesc_sf_ids(id, id),
                            (st | k) != 0 ? 1u : 0u, sx, sx + 4);
          }
          tc::mma_commit(&empty[s]);
          if (cw == kStagesPerChunk - 1 || st == nst - 1) {
            tc::mma_commit(&sempty[cs]);
            ++ch;
          }
        }
        if (ok) tc::mma_commit(&dfull[it & 1]);
      }
      // completes once every operation this thread issued has finished
      if (g > 0)
        tc::mma_commit(drain);
      else
        tc::mbar_arrive(drain);
    }
  } else if (warp < kEpi0) {
    // -------------------------------------------------------- scale loaders
    // One warp per block of 128 rows (B's, then A's): lane l carries the 32
    // bytes of the chunk of rows l, l + 32, l + 64 and l + 96, which are the 16
    // bytes of row l of tcgen05.cp's order for each of the 8 words.  Two groups
    // of warps take every second chunk each, so one's loads are in flight while
    // the other's chunk is used.
    const uint32_t mine = static_cast<uint32_t>(warp - 2) / (1 + YB);
    const int blk = (warp - 2) % (1 + YB);
    const uint8_t* all = blk == 0 ? a.xs : a.ys;
    const uint8_t* end = all + (blk == 0 ? a.x_total : a.y_rows) * ks;
    uint32_t ch = 0;
    bool ok = true;
    for (uint32_t i = blockIdx.x; ok && i < n_work; i += gridDim.x) {
      const Work w = work_of<NT>(a, grp, xt, yt, i, ge);
      const int nst = (w.steps + kStepsPerStage - 1) / kStepsPerStage;
      const int nch = (nst + kStagesPerChunk - 1) / kStagesPerChunk;
      const int64_t row0 = blk == 0 ? w.x0 + (a.mode == kGrouped ? w.e * a.x_rows : 0)
                                    : static_cast<int64_t>(w.y0) + (blk - 1) * 128;
      const int rows = blk == 0 ? static_cast<int>(min(a.x_rows - w.x0, static_cast<int64_t>(BX)))
                                : w.ny - (blk - 1) * 128;
      const uint8_t* base = all + (row0 + lane) * ks + w.k0 / 32;
      const int left = ks - w.k0 / 32;
      for (int q = 0; q < nch; ++q, ++ch) {
        if ((ch & 1) != mine) continue;
        const int byte = q * kWords * 4;
        const uint8_t* p = base + byte;
        const int n = min(32, left - byte);
        Pieces raw[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          raw[c] = load_pieces(p + c * 32 * ks, lane + 32 * c < rows ? n : 0, end);
        uint32_t v[4][8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int nr = lane + 32 * c < rows ? n : 0;
          align_words(raw[c], p + c * 32 * ks, nr, v[c]);
          if (past_end(p + c * 32 * ks, nr, end)) load_bytes(p + c * 32 * ks, nr, v[c]);
        }
        const uint32_t cs = ch % kChunkSlots, use = ch / kChunkSlots;
        if (use > 0 && !warp_wait(&sempty[cs], (use - 1) & 1, abort_flag, a.status)) {
          ok = false;
          break;
        }
        uint8_t* dst = chunks + cs * chunk_bytes(NT) + blk * kWords * kWordBytes + lane * 16;
#pragma unroll
        for (int k = 0; k < kWords; ++k)
          *reinterpret_cast<uint4*>(dst + k * kWordBytes) = make_uint4(v[0][k], v[1][k], v[2][k], v[3][k]);
        // the tensor core's copy reads shared memory through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sfull[cs]);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;  // the lane quarter this warp may read
    const int part = (warp - kEpi0) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    uint32_t it = 0;
    for (uint32_t i = blockIdx.x; i < n_work; i += gridDim.x, ++it) {
      const Work w = work_of<NT>(a, grp, xt, yt, i, ge);
      const uint32_t b = it & 1;
      if (!warp_wait(&dfull[b], (it >> 1) & 1, abort_flag, a.status)) break;
      tc::tc_fence_after();
      const int64_t n = static_cast<int64_t>(w.x0) + q * 32 + lane;
      const uint32_t acc = tmem + b * ACC + lane_base;
      // the tile's columns, split over this quarter's warps in steps of 32
      const int all = (w.ny + 15) & ~15;
      const int half = kEpi == 8 ? (all / 2 + 31) & ~31 : all;
      const int c0 = part ? min(half, all) : 0, c1 = part ? all : min(half, all);
      if (a.out_f32)
        store_columns<true>(acc, a, w, n, c0, c1);
      else
        store_columns<false>(acc, a, w, n, c0, c1);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&dempty[b]);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) tc::mbar_drain(drain, 0, kWaitLimitNs / 8);
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, TMEM);
  }
}

// ------------------------------------------------------------ host helpers

bool encode(CUtensorMap* map, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank),
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
moe_status launch_nt(const Args& a, const uint8_t* xq, const uint8_t* yq, int64_t max_work,
                     cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (!bit || !(done.load() & bit)) {
    if (cudaFuncSetAttribute(mxfp4_matmul_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_bytes(NT)) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    done.fetch_or(bit);
  }
  const cuuint64_t row = static_cast<cuuint64_t>(a.K) / 2;
  const cuuint64_t xm = static_cast<cuuint64_t>(a.mode == kGrouped ? a.E : 1);
  CUtensorMap mx, my;
  const cuuint64_t xd[3] = {row, static_cast<cuuint64_t>(a.x_rows), xm};
  const cuuint64_t xs[2] = {row, row * static_cast<cuuint64_t>(a.x_rows)};
  const cuuint32_t xb[3] = {BKB, BX, 1};
  const cuuint64_t yd[2] = {row, static_cast<cuuint64_t>(a.y_rows)};
  const cuuint64_t ys[1] = {row};
  const cuuint32_t yb[2] = {BKB, NT};
  if (!encode(&mx, 3, xq, xd, xs, xb) || !encode(&my, 2, yq, yd, ys, yb)) return MOE_ERR_CUDA;
  const int64_t cap = static_cast<int64_t>(sm_count()) * ctas_per_sm(NT);
  const dim3 grid(static_cast<unsigned>(max_work < cap ? max_work : cap));
  return launch(mxfp4_matmul_kernel<NT>, grid, dim3(threads(NT)), smem_bytes(NT), stream, mx, my, a);
}

// Rows of A per tile: `rows` is what one tile may meet, twice the mean of a
// group where there are groups.
moe_status run(Args a, const uint8_t* xq, const uint8_t* yq, int64_t rows, cudaStream_t stream) {
  const int NT = rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : (rows <= 128 ? 128 : 224)));
  const int64_t xt = (a.x_rows + BX - 1) / BX, yt = (a.y_rows + NT - 1) / NT;
  const int64_t max_work = xt * (a.mode == kDense ? yt : (a.mode == kGrouped ? yt + a.E : yt * a.E));
  switch (NT) {
    case 16: return launch_nt<16>(a, xq, yq, max_work, stream);
    case 32: return launch_nt<32>(a, xq, yq, max_work, stream);
    case 64: return launch_nt<64>(a, xq, yq, max_work, stream);
    case 128: return launch_nt<128>(a, xq, yq, max_work, stream);
    default: return launch_nt<224>(a, xq, yq, max_work, stream);
  }
}

constexpr int64_t kMaxRows = int64_t(1) << 27, kMaxK = int64_t(1) << 24;

moe_status check(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q, const uint8_t* b_s,
                 const void* out, int32_t out_type, const int32_t* d_status) {
  if (out_type != MOE_OUT_BF16 && out_type != MOE_OUT_FP32) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {a_q, a_s, b_q, b_s, out};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(d_status) & 3u) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status mxfp4_matmul(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q,
                        const uint8_t* b_s, int64_t M, int64_t N, int64_t K, float alpha,
                        void* out, int32_t out_type, int32_t* d_status, moe_stream stream) {
  using namespace moe;
  if (M < 0 || N < 0 || M > kMaxRows || N > kMaxRows || K < 32 || K > kMaxK || K % 32)
    return MOE_ERR_SHAPE;
  if (M == 0 || N == 0) return MOE_OK;
  moe_status st = check(a_q, a_s, b_q, b_s, out, out_type, d_status);
  if (st != MOE_OK) return st;
  if ((st = check_device()) != MOE_OK) return st;
  Args a{};
  a.mode = kDense;
  a.E = 1;
  a.xs = b_s;
  a.ys = a_s;
  a.x_rows = a.x_total = N;
  a.y_rows = M;
  a.K = K;
  a.alpha = alpha;
  a.out = out;
  a.out_f32 = out_type == MOE_OUT_FP32;
  a.status = d_status;
  return run(a, b_q, a_q, M, static_cast<cudaStream_t>(stream));
}

moe_status mxfp4_matmul_grouped(const uint8_t* a_q, const uint8_t* a_s, const int32_t* offsets,
                                int32_t E, const uint8_t* b_q, const uint8_t* b_s, int64_t S,
                                int64_t N, int64_t K, float alpha, void* out, int32_t out_type,
                                int32_t* d_status, moe_stream stream) {
  using namespace moe;
  if (E < 1 || E > kMaxGroups || S < 0 || N < 0 || S > kMaxRows || N > kMaxRows / E || K < 32 ||
      K > kMaxK || K % 32)
    return MOE_ERR_SHAPE;
  if (S == 0 || N == 0) return MOE_OK;
  moe_status st = check(a_q, a_s, b_q, b_s, out, out_type, d_status);
  if (st != MOE_OK) return st;
  if (!offsets || !aligned16(offsets)) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  Args a{};
  a.mode = kGrouped;
  a.E = E;
  a.offsets = offsets;
  a.xs = b_s;
  a.ys = a_s;
  a.x_rows = N;
  a.x_total = N * E;
  a.y_rows = S;
  a.K = K;
  a.S = S;
  a.alpha = alpha;
  a.out = out;
  a.out_f32 = out_type == MOE_OUT_FP32;
  a.status = d_status;
  return run(a, b_q, a_q, 2 * ((S + E - 1) / E), static_cast<cudaStream_t>(stream));
}

moe_status mxfp4_matmul_grouped_wgrad(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q,
                                      const uint8_t* b_s, const int32_t* offsets, int32_t E,
                                      int64_t M, int64_t N, int64_t P, float alpha, void* out,
                                      int32_t out_type, int32_t* d_status, moe_stream stream) {
  using namespace moe;
  if (E < 1 || E > kMaxGroups || M < 0 || N < 0 || M > kMaxRows / E || N > kMaxRows || P < 0 ||
      P > kMaxK || P % kGroupAlign)
    return MOE_ERR_SHAPE;
  if (M == 0 || N == 0) return MOE_OK;
  // without a position (P = 0) there is nothing to read, only zeros to write
  const void* some = out;
  moe_status st = P > 0 ? check(a_q, a_s, b_q, b_s, out, out_type, d_status)
                        : check(static_cast<const uint8_t*>(some), static_cast<const uint8_t*>(some),
                                static_cast<const uint8_t*>(some), static_cast<const uint8_t*>(some),
                                out, out_type, d_status);
  if (st != MOE_OK) return st;
  if (!offsets || !aligned16(offsets)) return MOE_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_OK) return st;
  if (P == 0) {
    const size_t bytes = static_cast<size_t>(E) * M * N * (out_type == MOE_OUT_FP32 ? 4 : 2);
    if (cudaMemsetAsync(out, 0, bytes, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    return MOE_OK;
  }
  Args a{};
  a.mode = kWgrad;
  a.E = E;
  a.offsets = offsets;
  a.xs = b_s;
  a.ys = a_s;
  a.x_rows = a.x_total = N;
  a.y_rows = M;
  a.K = P;
  a.S = P;  // a group never has more rows than positions
  a.alpha = alpha;
  a.out = out;
  a.out_f32 = out_type == MOE_OUT_FP32;
  a.status = d_status;
  return run(a, b_q, a_q, M, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
