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
//   warps 2-5   scale loaders: E8M0 bytes from global memory, in chunks of 1024
//               k (32 bytes of a row, one sector), laid down in shared memory in
//               the order tcgen05.cp takes them
//   warps 6-9   epilogue, one per lane quarter, from a double-buffered
//               accumulator, so it overlaps the next tile's MMAs
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
// one scale word of 128 rows: 512 bytes in tcgen05.cp's order, 16 apart so that
// the loaders' stores of 8 words meet no bank conflict
constexpr int kWordBytes = 512 + 16;
constexpr int kThreads = 320;
constexpr int kScaleWarps = 4, kEpiWarps = 4;
constexpr int kMaxStages = 8;
constexpr int kChunkSlots = 2;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

enum Mode : int { kDense = 0, kGrouped = 1, kWgrad = 2 };

__host__ __device__ constexpr int y_blocks(int NT) { return (NT + 127) / 128; }
__host__ __device__ constexpr int acc_cols(int NT) { return NT < 32 ? 32 : NT; }
__host__ __device__ constexpr int sf_cols(int NT) { return 2 * 4 * (1 + y_blocks(NT)); }
__host__ __device__ constexpr int tmem_cols(int NT) {
  const int need = 2 * acc_cols(NT) + 2 * sf_cols(NT);
  return need <= 128 ? 128 : (need <= 256 ? 256 : 512);
}
__host__ __device__ constexpr int ctas_per_sm(int NT) { return NT <= 64 ? 2 : 1; }
__host__ __device__ constexpr int stage_bytes(int NT) { return X_BYTES + NT * BKB; }
__host__ __device__ constexpr int chunk_bytes(int NT) { return kWords * (1 + y_blocks(NT)) * kWordBytes; }
__host__ __device__ constexpr int stages(int NT) {
  const int room = (ctas_per_sm(NT) == 2 ? 112 : 226) * 1024 - 1024 - 512 -
                   (kMaxGroups + 1) * 8 - kChunkSlots * chunk_bytes(NT);
  const int n = room / stage_bytes(NT);
  return n < kMaxStages ? n : kMaxStages;
}
__host__ __device__ constexpr int smem_bytes(int NT) {
  return 1024 + stages(NT) * stage_bytes(NT) + kChunkSlots * chunk_bytes(NT) +
         (kMaxGroups + 1) * 8 + 512;
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
  int64_t S;               // wgrad: the capacity's last position / grouped: rows of A
  float alpha;
  void* out;
  int out_f32;
  int32_t* status;
};

// One output tile: B rows [x0, ..) of matrix xm, A rows [y0, y0 + ny), k in
// [k0, k0 + 64 steps), out row y0 + i + yo.
struct Work {
  int64_t x0, y0, k0, out_row;
  int e, ny, steps;
  bool live;
};

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
__device__ __forceinline__ int tile_width(int64_t n) {
  const int64_t t = (n + NT - 1) / NT;
  return t == 0 ? 16 : static_cast<int>(((n + t - 1) / t + 15) / 16 * 16);
}

// Tiles are numbered with the B side fastest, so the CTAs running at one time
// share a few tiles of A rows.
template <int NT>
__device__ __forceinline__ Work work_of(const Args& a, const int64_t* pfx, int64_t xt, int64_t i) {
  Work w;
  w.x0 = i % xt * BX;
  int64_t u = i / xt;
  w.e = 0;
  w.k0 = 0;
  w.live = true;
  int64_t lo = 0, n = a.y_rows;
  w.steps = static_cast<int>((a.K + 63) / 64);
  if (a.mode == kGrouped) {
    w.e = group_of(pfx, a.E, u);
    u -= pfx[w.e];
    int64_t hi;
    group_rows(a.offsets, w.e, a.y_rows, lo, hi);
    n = hi - lo;
  } else if (a.mode == kWgrad) {
    const int64_t yt = (a.y_rows + NT - 1) / NT;
    w.e = static_cast<int>(u / yt);
    u %= yt;
    int64_t glo, ghi;
    group_rows(a.offsets, w.e, a.S, glo, ghi);
    w.k0 = pfx[w.e] * kGroupAlign;
    // never past the capacity, whatever the offsets hold
    const int64_t room = a.K - w.k0;
    const int64_t len = room < 0 ? 0 : (ghi - glo < room ? ghi - glo : room);
    w.steps = static_cast<int>((len + 63) / 64);
  }
  const int width = tile_width<NT>(n);
  w.y0 = lo + u * width;
  const int64_t left = lo + n - w.y0;
  w.ny = static_cast<int>(left < width ? (left < 0 ? 0 : left) : width);
  w.out_row = w.y0 + (a.mode == kWgrad ? static_cast<int64_t>(w.e) * a.y_rows : 0);
  return w;
}

// Four scale bytes of a row from byte b of its ks; bytes past the row's end
// read as 0 (their codes are zero).  `total` bounds the whole array.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* __restrict__ s, int64_t row_off,
                                               int64_t b, int64_t ks, int64_t total) {
  if (b >= ks) return 0u;
  const int64_t at = row_off + b;
  uint32_t v;
  if ((ks & 3) == 0) {
    v = __ldg(reinterpret_cast<const uint32_t*>(s + at));
  } else if (at + 8 <= total) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(s + (at & ~int64_t(3)));
    v = __funnelshift_r(__ldg(p), __ldg(p + 1), static_cast<uint32_t>(at & 3) * 8);
  } else {
    v = 0;
    for (int i = 0; i < 4 && at + i < total; ++i) v |= static_cast<uint32_t>(__ldg(s + at + i)) << (8 * i);
  }
  const int64_t left = ks - b;
  return left < 4 ? v & ((1u << (8 * left)) - 1u) : v;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT))
    mxfp4_matmul_kernel(const __grid_constant__ CUtensorMap map_x,
                        const __grid_constant__ CUtensorMap map_y, const Args a) {
  constexpr int NS = stages(NT), STAGE = stage_bytes(NT), YB = y_blocks(NT);
  constexpr int ACC = acc_cols(NT), SF = sf_cols(NT), TMEM = tmem_cols(NT);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* chunks = smem + NS * STAGE;
  int64_t* pfx = reinterpret_cast<int64_t*>(chunks + kChunkSlots * chunk_bytes(NT));
  uint64_t* full = reinterpret_cast<uint64_t*>(pfx + kMaxGroups + 1);  // [NS] stage copies landed
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
      tc::mbar_init(&sfull[s], kScaleWarps);
      tc::mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&dfull[b], 1);
      tc::mbar_init(&dempty[b], kEpiWarps);
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
    group_prefix(a.E, pfx, [&](int e) {
      int64_t lo, hi;
      group_rows(a.offsets, e, a.mode == kGrouped ? a.y_rows : a.S, lo, hi);
      return a.mode == kGrouped ? (hi - lo + NT - 1) / NT
                                : (hi - lo + kGroupAlign - 1) / kGroupAlign;
    });
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int64_t xt = (a.x_rows + BX - 1) / BX;
  const int64_t yt = (a.y_rows + NT - 1) / NT;
  const int64_t n_work =
      xt * (a.mode == kDense ? yt : (a.mode == kGrouped ? pfx[a.E] : yt * a.E));
  const int64_t ks = a.K / 32;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int64_t g = 0;
      bool ok = true;
      for (int64_t i = blockIdx.x; ok && i < n_work; i += gridDim.x) {
        const Work w = work_of<NT>(a, pfx, xt, i);
        const int nst = (w.steps + kStepsPerStage - 1) / kStepsPerStage;
        for (int st = 0; st < nst; ++st, ++g) {
          const int s = static_cast<int>(g % NS);
          const int64_t n = g / NS;
          if (n > 0 && !wait1(&empty[s], (n - 1) & 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + s * STAGE;
          const int kb = static_cast<int>(w.k0 / 2) + st * BKB;
          tc::mbar_arrive_expect_tx(&full[s], STAGE);
          tc::tma_load_3d(dst, &map_x, &full[s], kb, static_cast<int>(w.x0),
                          a.mode == kGrouped ? w.e : 0);
          tc::tma_load_2d(dst + X_BYTES, &map_y, &full[s], kb, static_cast<int>(w.y0));
        }
      }
      // every copy this thread issued has landed before the CTA exits
      for (int64_t i = g > NS ? g - NS : 0; i < g; ++i)
        tc::mbar_drain(&full[i % NS], (i / NS) & 1, kWaitLimitNs / 8);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      int64_t g = 0, ch = 0, it = 0;
      bool ok = true;
      for (int64_t i = blockIdx.x; ok && i < n_work; i += gridDim.x, ++it) {
        const Work w = work_of<NT>(a, pfx, xt, i);
        const uint32_t idesc = tc::idesc_mxf4(BX, (w.ny + 15) & ~15);
        const uint32_t d = tmem + static_cast<uint32_t>(it & 1) * ACC;
        // accumulator it & 1 was last used by tile it - 2
        if (it >= 2 && !wait1(&dempty[it & 1], ((it >> 1) - 1) & 1, abort_flag, a.status)) break;
        const int nst = (w.steps + kStepsPerStage - 1) / kStepsPerStage;
        for (int st = 0; st < nst; ++st, ++g) {
          const int cw = st % kStagesPerChunk;
          const int cs = static_cast<int>(ch % kChunkSlots);
          if (cw == 0 && !wait1(&sfull[cs], (ch / kChunkSlots) & 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          // the tensor-memory scale columns of stage g were last read by stage g - 2
          if (g >= 2) {
            const int64_t p = g - 2;
            if (!wait1(&empty[p % NS], (p / NS) & 1, abort_flag, a.status)) {
              ok = false;
              break;
            }
          }
          const int s = static_cast<int>(g % NS);
          if (!wait1(&full[s], (g / NS) & 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t sf = tmem + 2 * ACC + static_cast<uint32_t>(g & 1) * SF;
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
  } else if (warp < 2 + kScaleWarps) {
    // -------------------------------------------------------- scale loaders
    // Lane (word w = lane % 8, quarter c = lane / 8) carries word w of rows
    // 32 c + rr: 8 neighbouring lanes read 32 contiguous bytes of a row.
    const int wi = warp - 2, kw = lane & 7, c = lane >> 3;
    const int64_t x_bytes = a.x_total * ks, y_bytes = a.y_rows * ks;
    int64_t ch = 0;
    bool ok = true;
    for (int64_t i = blockIdx.x; ok && i < n_work; i += gridDim.x) {
      const Work w = work_of<NT>(a, pfx, xt, i);
      const int nst = (w.steps + kStepsPerStage - 1) / kStepsPerStage;
      const int nch = (nst + kStagesPerChunk - 1) / kStagesPerChunk;
      const int64_t xrow = w.x0 + (a.mode == kGrouped ? static_cast<int64_t>(w.e) * a.x_rows : 0);
      for (int q = 0; q < nch; ++q, ++ch) {
        const int64_t byte = w.k0 / 32 + (static_cast<int64_t>(q) * kWords + kw) * 4;
        uint32_t v[8 * (1 + YB)];
#pragma unroll
        for (int b = 0; b < 1 + YB; ++b)
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int row = (b > 0 ? b - 1 : 0) * 128 + c * 32 + wi + 4 * r;
            const bool in = b == 0 ? w.x0 + row < a.x_rows : row < w.ny;
            v[b * 8 + r] = !in ? 0u
                           : b == 0
                               ? scale_word(a.xs, (xrow + row) * ks, byte, ks, x_bytes)
                               : scale_word(a.ys, (w.y0 + row) * ks, byte, ks, y_bytes);
          }
        const int cs = static_cast<int>(ch % kChunkSlots);
        const int64_t n = ch / kChunkSlots;
        if (n > 0 && !warp_wait(&sempty[cs], (n - 1) & 1, abort_flag, a.status)) {
          ok = false;
          break;
        }
        uint8_t* chunk = chunks + cs * chunk_bytes(NT);
#pragma unroll
        for (int b = 0; b < 1 + YB; ++b)
#pragma unroll
          for (int r = 0; r < 8; ++r)
            *reinterpret_cast<uint32_t*>(chunk + (b * kWords + kw) * kWordBytes +
                                         (wi + 4 * r) * 16 + c * 4) = v[b * 8 + r];
        // the tensor core's copy reads shared memory through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sfull[cs]);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;  // the lane quarter this warp may read
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    int64_t it = 0;
    for (int64_t i = blockIdx.x; i < n_work; i += gridDim.x, ++it) {
      const Work w = work_of<NT>(a, pfx, xt, i);
      const int b = static_cast<int>(it & 1);
      if (!warp_wait(&dfull[b], (it >> 1) & 1, abort_flag, a.status)) break;
      tc::tc_fence_after();
      const int64_t n = w.x0 + q * 32 + lane;
      const bool live = n < a.x_rows;
      const uint32_t acc = tmem + static_cast<uint32_t>(b) * ACC + lane_base;
      for (int c = 0; c < w.ny; c += 16) {
        uint32_t r[16];
        if (w.steps > 0) {
          tc::tmem_ld16(acc + c, r);
          tc::tmem_ld_wait();
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) r[k] = 0u;  // an empty sum
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float v = a.alpha * __uint_as_float(r[k]);
          if (live && c + k < w.ny) {
            const int64_t at = (w.out_row + c + k) * a.x_rows + n;
            if (a.out_f32)
              static_cast<float*>(a.out)[at] = v;
            else
              static_cast<uint16_t*>(a.out)[at] = f32_to_bf16_rne(v);
          }
        }
      }
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
  return launch(mxfp4_matmul_kernel<NT>, grid, dim3(kThreads), smem_bytes(NT), stream, mx, my, a);
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
  a.S = int64_t(1) << 31;
  a.alpha = alpha;
  a.out = out;
  a.out_f32 = out_type == MOE_OUT_FP32;
  a.status = d_status;
  return run(a, b_q, a_q, M, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
