// The MXFP4 products on CTA pairs: tiles of 256 rows of B by up to 192 rows of A.
//
// "MXFP4-based MoE technical review", section 2 (MXFP4 training).  The same
// products as csrc/matmul.cu, for more than 128 rows of A.
//
// What bounds a 4-bit product is not the tensor core but the shared memory that
// feeds it: 64 k of a 128 x 192 tile take the tensor core 96 cycles and move 10
// KB into and out of shared memory, 213 bytes a cycle where an SM has 128.  A
// pair of SMs (cta_group::2, M = 256) holds 128 rows of B and half of the A rows
// in each, so the same 96 cycles per SM move 7 KB, 146 bytes a cycle; the block
// scales' way adds a third of that.  Wider tiles would move less per product, but
// two accumulators of 192 columns and two stages of scales fill tensor memory.
//   8192 x 5760 x 2880: 85 us alone, 3.2 PFLOP/s (96 us, 2.8 PFLOP/s, in a loop
//   that draws the power limit); without the scales' loads and the epilogue 63,
//   without the MMAs too 45, which is 13 TB/s out of L2.  The one-CTA form with
//   224-row tiles took 139 us.
//
// The tensor core takes the block scales from tensor memory; here warps write
// them with tcgen05.st beside the MMAs, two stages deep.  (tcgen05.cp from words
// laid down in shared memory costs the MMAs nothing, and was measured too: 92-96
// us, because the words' buffers leave the raw scales too little depth against
// the copy ring's own queue.)  Waits and issue stay with whole warps and an
// elected lane: under `lane == 0` four MMAs and one wait took 480 cycles instead
// of 245.  Arrivals on the other CTA's barriers release this CTA's shared memory
// at cluster scope by a fence for it alone, which costs nothing measurable.  With
// mbarrier.arrive.release.cluster the same product took 93 us in a loop for the
// second CTA's copies alone and 114 for the scale writers' arrivals too, against 81.
//
// Warp roles, in each CTA of the pair:
//   warp 0       producer: per stage of 512 k its own 128 rows of B and its half
//                of the A rows, by TMA into its own shared memory
//   warp 1       tensor-memory owner; in the first CTA the MMA issuer, in the
//                second it tells the issuer that a stage's codes have landed
//   warps 2, 3   scale loaders: cp.async of chunks of 1024 k (32 bytes of a
//                row, as the three aligned 16-byte pieces that cover them: rows
//                start at any byte), three chunks deep; they queue behind the
//                copy ring's 172 KB
//   warps 4-11   scale writers, two groups of one per lane quarter: a stage's
//                bytes shifted into words and put into tensor memory, and the
//                issuer told
//   warps 12-19  epilogue, two per lane quarter, from a double-buffered
//                accumulator
// The issuer's commits reach both CTAs' barriers.  Every wait is bounded (2 s);
// on expiry the kernel records MOE_ERR_TIMEOUT, waits for its own copies and
// MMAs to finish and returns.  Copies are always local to a CTA and awaited by
// it; the CTAs of a pair leave together.
#include <cuda.h>

#include <atomic>

#include "matmul_common.cuh"

namespace moe {
namespace {

using namespace mm;

constexpr int NT = 192;    // rows of A per tile
constexpr int STEP = 32;   // in steps of the pair's N
constexpr int BX = 256;    // rows of B per tile
constexpr int X_BYTES = 128 * BKB, Y_BYTES = NT / 2 * BKB, WINDOW = X_BYTES + Y_BYTES;
constexpr int WPS = 2;                     // windows of 256 k per stage
constexpr int STAGE = WPS * WINDOW;
constexpr int STEPS = WPS * kStepsPerStage;  // MMAs of 64 k per stage
constexpr int SPC = kStagesPerChunk / WPS;   // stages per scale chunk
constexpr int kWriters = 4, kEpi = 8;  // warps (writers: per group)
constexpr int kWriter0 = 4, kEpi0 = 12;
constexpr int kThreads = 32 * (kEpi0 + kEpi);
constexpr int kRowsAtOnce = 16;  // rows of scales the two loader warps take at once
// a scale chunk in shared memory: of every row the three aligned 16-byte pieces
// that cover its 32 bytes
constexpr int kRowBytes = 48, kRows = 128 + NT;
constexpr int kChunkBytes = kRows * kRowBytes;
constexpr int kSlots = 3;
constexpr int SFW = 4 + 8;             // scale columns of one word (128 k): B's rows, A's rows
constexpr int SF = 2 * WPS * SFW;      // of a stage
constexpr int TMEM = 512;
constexpr int SLOTS = 2;               // stages of scales in tensor memory
static_assert(2 * NT + SLOTS * SF <= TMEM, "two accumulators and the scale slots");
constexpr int NS = 3;  // copy ring
static_assert(SLOTS == 2 && SLOTS <= NS, "a slot's last stage is found by its ring barrier");
constexpr int kSmem = 1024 + NS * STAGE + kSlots * kChunkBytes + kTableBytes + 512;
static_assert(NS <= kMaxStages && kSmem <= 227 * 1024, "shared memory");

__device__ __forceinline__ int pair_stages(const Work& w) { return (w.steps + STEPS - 1) / STEPS; }

// Lane 0 waits for a phase (its own sleep short), the warp follows.
__device__ __forceinline__ bool lead_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int32_t* status) {
  bool r = true;
  if ((threadIdx.x & 31) == 0) r = tc::mbar_wait_sleep(bar, parity, abort, kWaitLimitNs, 20);
  r = __shfl_sync(0xFFFFFFFFu, r, 0);
  if (!r) abort_cta(abort, status);
  return r;
}

template <int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mxfp4_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_x,
                             const __grid_constant__ CUtensorMap map_y, const Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* chunks = smem + NS * STAGE;
  const Groups grp = group_table(chunks + kSlots * kChunkBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(grp.width + kMaxGroups + 2);  // [NS] own copies landed
  uint64_t* ready = full + kMaxStages;     // [NS] both CTAs' codes and scales (first CTA)
  uint64_t* empty = ready + kMaxStages;    // [NS] stage MMAs complete
  uint64_t* sfull = empty + kMaxStages;    // [3] scale chunk in shared memory
  uint64_t* sempty = sfull + kSlots;       // [3] scale chunk read
  uint64_t* dfull = sempty + kSlots;  // [2] accumulator complete
  uint64_t* dempty = dfull + 2;            // [2] accumulator read by both CTAs (first CTA)
  uint64_t* drain = dempty + 2;            // every MMA issued has completed
  uint64_t* never = drain + 1;             // nothing completes it (testing)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(tc::cluster_rank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&ready[s], 2 * kWriters + 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      tc::mbar_init(&sfull[s], 64);
      tc::mbar_init(&sempty[s], 2 * kWriters);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&dfull[b], 1);
      tc::mbar_init(&dempty[b], 2 * kEpi);
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init(never, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_y);
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tmem_holder, TMEM);
    tc::tmem_relinquish_pair();
  }
  if (warp == 2) fill_groups<NT, STEP>(a, grp);
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers exist before either is told anything
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t n_work = tiles(a, grp);
  const uint32_t first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  const int ks = static_cast<int>(a.K / 32);
  int ge = 0;  // this role's cursor over the groups

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t s = 0, phase = 0, issued = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < n_work; i += stride) {
      const Work w = work_of<NT, STEP, BX>(a, grp, i, ge);
      const int nst = pair_stages(w), half = ((w.ny + STEP - 1) & ~(STEP - 1)) / 2;
      for (int st = 0; st < nst; ++st) {
        if (issued >= NS && !all_wait(&empty[s], phase ^ 1u, abort_flag, a.status)) {
          ok = false;
          break;
        }
        if (tc::elect_one()) {
          const int nw = min(WPS, stages_of(w) - st * WPS);
          tc::mbar_arrive_expect_tx(&full[s], nw * WINDOW);
#pragma unroll
          for (int v = 0; v < WPS; ++v) {
            if (v >= nw) break;
            uint8_t* dst = smem + s * STAGE + v * WINDOW;
            const int kb = w.k0 / 2 + (st * WPS + v) * BKB;
            tc::tma_load_3d(dst, &map_x, &full[s], kb, w.x0 + rank * 128, a.mode == kGrouped ? w.e : 0);
            tc::tma_load_3d(dst + X_BYTES, &map_y, &full[s], kb, w.y0 + rank * half, 0);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == NS) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    // every copy this warp issued has landed before the CTA exits
    for (uint32_t i = issued > NS ? issued - NS : 0; i < issued; ++i)
      tc::mbar_drain(&full[i % NS], (i / NS) & 1, kWaitLimitNs / 8);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    bool ok = injected_timeout(a, never, abort_flag);
    if (rank == 0) {
      const uint64_t desc0 = tc::smem_desc_sw128(tc::smem_u32(smem));
      uint32_t it = 0, s = 0, phase = 0, slot = 0;
      bool any = false;
      for (uint32_t i = first; ok && i < n_work; i += stride, ++it) {
        const Work w = work_of<NT, STEP, BX>(a, grp, i, ge);
        const uint32_t idesc = tc::idesc_mxf4(BX, (w.ny + STEP - 1) & ~(STEP - 1));
        const uint32_t d = tmem + (it & 1) * NT;
        // accumulator it & 1 was last used by tile it - 2
        if (it >= 2 && !all_wait<true>(&dempty[it & 1], ((it >> 1) - 1) & 1, abort_flag, a.status)) break;
        const int nst = pair_stages(w);
        for (int st = 0; st < nst; ++st) {
          // its own codes, then the other CTA's and both CTAs' scales
          if (!all_wait(&full[s], phase, abort_flag, a.status) ||
              !all_wait<true>(&ready[s], phase, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t sf = tmem + 2 * NT + slot * SF;
          // a descriptor addresses shared memory in 16-byte units
          const uint64_t xd = desc0 + s * (STAGE / 16);
          const int left = w.steps - st * STEPS;
          if (tc::elect_one()) {
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
              if (k >= left) break;
              const uint32_t sx = sf + (k >> 1) * SFW, id = (k & 1) * 2;
              const uint64_t xk = xd + (k / kStepsPerStage) * (WINDOW / 16) + 2 * (k % kStepsPerStage);
              tc::mma_mxf4_pair(d, xk, xk + X_BYTES / 16, idesc | tc::idesc_sf_ids(id, id),
                                (st | k) != 0 ? 1u : 0u, sx, sx + 4);
            }
            tc::mma_commit_pair(&empty[s]);
            if (st == nst - 1) tc::mma_commit_pair(&dfull[it & 1]);
          }
          __syncwarp();
          any = true;
          if (++s == NS) {
            s = 0;
            phase ^= 1u;
          }
          if (++slot == SLOTS) slot = 0;
        }
        // an empty sum: its zeros wait for nothing
        if (nst == 0 && tc::elect_one()) tc::mma_commit_pair(&dfull[it & 1]);
        any |= nst == 0;
        __syncwarp();
      }
      // completes, in both CTAs, once every operation this warp issued has finished
      if (tc::elect_one()) {
        if (any) {
          tc::mma_commit_pair(drain);
        } else {
          tc::mbar_arrive(drain);
          tc::mbar_arrive_cluster(tc::cluster_addr(drain, 1));
        }
      }
    } else {
      // the second CTA: its codes' arrival, passed on to the issuer, whose MMAs
      // read them (the tcgen05 fences order tensor memory only)
      const uint32_t to = tc::cluster_addr(ready, 0);
      uint32_t s = 0, phase = 0;
      for (uint32_t i = first; ok && i < n_work; i += stride) {
        const int nst = pair_stages(work_of<NT, STEP, BX>(a, grp, i, ge));
        for (int st = 0; ok && st < nst; ++st) {
          ok = all_wait(&full[s], phase, abort_flag, a.status);
          if (ok && lane == 0) tc::mbar_arrive_cluster(to + s * 8);
          if (++s == NS) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp < kWriter0) {
    // -------------------------------------------------------- scale loaders
    // Three threads to a row, one per piece; a piece's bytes past its row's end
    // (or the array's) are not read and become 0, as their codes are.
    // A thread's rows are 16 apart, so one misalignment holds for all of them and
    // a copy takes five instructions.  (At any other distance it took 25, and the
    // loaders' own instructions held the products back.)
    const int lt = (warp - 2) * 32 + lane;
    const int r0 = lt / 3, piece = lt % 3;  // 48 of the 64 threads have one
    const int64_t pitch = static_cast<int64_t>(kRowsAtOnce) * ks;
    uint32_t slot = 0, phase = 0, ch = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < n_work; i += stride) {
      const Work w = work_of<NT, STEP, BX>(a, grp, i, ge);
      const int nch = chunks_of(w), left = ks - w.k0 / 32;
      const int64_t x0 = static_cast<int64_t>(w.x0) + rank * 128;
      const int xr = static_cast<int>(min(a.x_rows - x0, static_cast<int64_t>(128)));
      const uint8_t* px = a.xs + (x0 + (a.mode == kGrouped ? w.e * a.x_rows : 0) + r0) * ks + w.k0 / 32;
      const uint8_t* py = a.ys + (static_cast<int64_t>(w.y0) + r0) * ks + w.k0 / 32;
      const int mx = static_cast<int>(reinterpret_cast<uintptr_t>(px) & 15u);
      const int my = static_cast<int>(reinterpret_cast<uintptr_t>(py) & 15u);
      px += 16 * piece - mx;
      py += 16 * piece - my;
      for (int q = 0; q < nch; ++q, ++ch) {
        if (ch >= kSlots && !warp_wait(&sempty[slot], phase ^ 1u, abort_flag, a.status, 50)) {
          ok = false;
          break;
        }
        const int byte = q * kWords * 4, n = min(32, left - byte);
        const int bx = max(0, min(16, mx + n - 16 * piece)), by = max(0, min(16, my + n - 16 * piece));
        const uint32_t dst = tc::smem_u32(chunks + slot * kChunkBytes) + r0 * kRowBytes + piece * 16;
        if (r0 < kRowsAtOnce) {
          // of an absent row or piece nothing is read: its size is 0
          const uint8_t* p = px + byte;
#pragma unroll
          for (int j = 0; j < 128; j += kRowsAtOnce) {
            const bool in = r0 + j < xr && bx > 0;
            tc::cp_async16(dst + j * kRowBytes, in ? p : a.xs, in ? bx : 0);
            p += pitch;
          }
          p = py + byte;
#pragma unroll
          for (int j = 0; j < NT; j += kRowsAtOnce) {
            const bool in = r0 + j < w.ny && by > 0;
            tc::cp_async16(dst + (128 + j) * kRowBytes, in ? p : a.ys, in ? by : 0);
            p += pitch;
          }
        }
        tc::cp_async_arrive(&sfull[slot]);
        if (++slot == kSlots) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    tc::cp_async_wait_all();
  } else if (warp < kEpi0) {
    // -------------------------------------------------------- scale writers
    // Lane l holds rows l + 32 c of both sides, which are column c of lane l in
    // every quarter of tensor memory.  The two groups of four warps take every
    // second stage each, and with it one of the two slots of scale columns.
    const int q = warp & 3;
    const uint32_t mine = static_cast<uint32_t>(warp - kWriter0) >> 2;
    const uint32_t cols = tmem + (static_cast<uint32_t>(q * 32) << 16) + 2 * NT + mine * SF;
    const uint32_t to = tc::cluster_addr(ready, 0);
    uint32_t g = 0, s = 0, cs = 0, cphase = 0;
    // the slot of stage g was last read by the MMAs of stage g - 2
    uint32_t old = mine, old_phase = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < n_work; i += stride) {
      const Work w = work_of<NT, STEP, BX>(a, grp, i, ge);
      const int nst = pair_stages(w);
      const int64_t x0 = static_cast<int64_t>(w.x0) + rank * 128;
      // a row's misalignment: chunks are 32 bytes apart and a lane's rows 32 rows,
      // so every chunk and every row of this lane has the same
      const uint32_t mx = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
          a.xs + (x0 + (a.mode == kGrouped ? w.e * a.x_rows : 0) + lane) * ks + w.k0 / 32)) & 15u;
      const uint32_t my = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
          a.ys + (static_cast<int64_t>(w.y0) + lane) * ks + w.k0 / 32)) & 15u;
      for (int st = 0; st < nst; ++st, ++g) {
        const int cw = st % SPC;
        if ((g & 1) == mine) {
          if (!warp_wait(&sfull[cs], cphase, abort_flag, a.status, 20)) {
            ok = false;
            break;
          }
          const uint8_t* src = chunks + cs * kChunkBytes + lane * kRowBytes + cw * 16;
          uint32_t r[SF];  // columns: [word 0: B 4, A 6, none 2][word 1: ...]...
#pragma unroll
          for (int j = 0; j < kRows / 32; ++j) {
            const uint32_t mis = j < 4 ? mx : my;
            const uint4 lo = *reinterpret_cast<const uint4*>(src + 32 * j * kRowBytes);
            const uint4 hi = *reinterpret_cast<const uint4*>(src + 32 * j * kRowBytes + 16);
            uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int k = 0; k < 7; ++k) x[k] = mis & 4u ? x[k + 1] : x[k];
#pragma unroll
            for (int k = 0; k < 5; ++k) x[k] = mis & 8u ? x[k + 2] : x[k];
#pragma unroll
            for (int k = 0; k < 2 * WPS; ++k) r[k * SFW + j] = __funnelshift_r(x[k], x[k + 1], (mis & 3u) * 8);
          }
#pragma unroll
          for (int k = 0; k < 2 * WPS; ++k)
#pragma unroll
            for (int j = kRows / 32; j < SFW; ++j) r[k * SFW + j] = 0u;
          if (g >= 2) {
            if (!lead_wait(&empty[old], old_phase, abort_flag, a.status)) {
              ok = false;
              break;
            }
            if ((old += 2) >= NS) {
              old -= NS;
              old_phase ^= 1u;
            }
          }
          tc::tc_fence_after();
#pragma unroll
          for (int j = 0; j < SF / 16; ++j)
            tc::tmem_st16(cols + 16 * j, *reinterpret_cast<const uint32_t(*)[16]>(r + 16 * j));
          tc::tmem_st_wait();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_cluster(to + s * 8);
        }
        if (++s == NS) s = 0;
        // both groups let a chunk go, whichever of its stages were theirs
        if (cw == SPC - 1 || st == nst - 1) {
          if (lane == 0) tc::mbar_arrive(&sempty[cs]);
          if (++cs == kSlots) {
            cs = 0;
            cphase ^= 1u;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;  // the lane quarter this warp may read
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    uint32_t it = 0;
    for (uint32_t i = first; i < n_work; i += stride, ++it) {
      const Work w = work_of<NT, STEP, BX>(a, grp, i, ge);
      const uint32_t b = it & 1;
      if (!warp_wait(&dfull[b], (it >> 1) & 1, abort_flag, a.status, 100)) break;
      tc::tc_fence_after();
      const int64_t n = static_cast<int64_t>(w.x0) + rank * 128 + q * 32 + lane;
      const uint32_t acc = tmem + b * NT + lane_base;
      // the tile's columns, split over this quarter's two warps in steps of 32
      const int all = (w.ny + 15) & ~15, half = (all / 2 + 31) & ~31;
      const int part = (warp - kEpi0) >> 2;
      const int c0 = part ? min(half, all) : 0, c1 = part ? all : min(half, all);
      store_columns<OUT>(acc, a, w, n, c0, c1);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::cluster_addr(&dempty[b], 0));
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) tc::mbar_drain(drain, 0, kWaitLimitNs / 8);
    __syncwarp();
  }
  tc::cluster_sync();  // neither CTA touches the other's memory from here on
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, TMEM);
  }
}

template <int OUT>
moe_status launch_one(Args a, const uint8_t* xq, const uint8_t* yq, cudaStream_t stream) {
  const int64_t most = plan_tiles(&a, BX, NT);
  if (most > kMaxTiles) return MOE_ERR_SHAPE;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (!bit || !(done.load() & bit)) {
    if (cudaFuncSetAttribute(mxfp4_matmul_pair_kernel<OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    done.fetch_or(bit);
  }
  CUtensorMap mx, my;
  if (!encode_codes(&mx, xq, a.K / 2, a.x_rows, a.mode == kGrouped ? a.E : 1, 128) ||
      !encode_codes(&my, yq, a.K / 2, a.y_rows, 1, NT / 2))
    return MOE_ERR_CUDA;
  const int64_t pairs = sm_count() / 2;
  const dim3 grid(static_cast<unsigned>(2 * (most < pairs ? most : pairs)));
  return launch(mxfp4_matmul_pair_kernel<OUT>, grid, dim3(kThreads), kSmem, stream, mx, my, a);
}

}  // namespace

namespace mm {

moe_status launch_pair(const Args& a, int out_type, const uint8_t* xq, const uint8_t* yq,
                       cudaStream_t stream) {
  switch (out_of(out_type, a.x_rows)) {
    case kFp32: return launch_one<kFp32>(a, xq, yq, stream);
    case kBf16Pairs: return launch_one<kBf16Pairs>(a, xq, yq, stream);
    default: return launch_one<kBf16>(a, xq, yq, stream);
  }
}

}  // namespace mm
}  // namespace moe
