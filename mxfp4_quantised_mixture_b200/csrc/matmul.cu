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
// With few tiles a cluster of CTAs shares each one's k range, if it is long; the
// partial sums meet in shared memory and are added in rank order.
//
// What bounds it: with few rows to an expert the weights' way from HBM.  The 20B
// decode batch's gate/up products (256 rows, 32 experts, 5760 x 2880: 285 MB)
// take 52-57 us, 5.0-5.4 TB/s, which is what copies of 128-byte rows by TMA reach
// on this part.  A single small product (4 x 2880 x 2880) takes 10 us, most of it
// fixed: first instruction fetches, first loads, the scales' way to tensor
// memory, the cluster's two meetings.
//
// Persistent, one CTA per SM (two for tiles of up to 64 rows).  Warp roles:
//   warp 0      producer: per stage of 256 k, 128 x 128 bytes of B codes and
//               NT x 128 bytes of A codes by TMA (zeros past the ends)
//   warp 1      tensor-memory owner and MMA issuer; it also copies each stage's
//               scale words from shared to tensor memory (tcgen05.cp)
//   warps 2-5   scale loaders: E8M0 bytes from global memory, in chunks of 1024
//               k (32 bytes of a row), laid down in shared memory in the order
//               tcgen05.cp takes them
//   the rest    epilogue, one or two warps per lane quarter, from a
//               double-buffered accumulator, so it overlaps the next tile's MMAs
// Every wait is bounded (2 s); on expiry the kernel records MOE_ERR_TIMEOUT,
// waits for its own copies and MMAs to finish and returns.
#include <cuda.h>

#include <atomic>

#include "matmul_common.cuh"

namespace moe {
namespace {

using namespace mm;

constexpr int BX = 128;  // B rows per tile (MMA M)
constexpr int STEP = 16; // rows of A come in steps of the MMA's N
constexpr int X_BYTES = BX * BKB;

// Warps: producer, MMA issuer, scale loaders, epilogue.  The widest tiles, one
// CTA per SM, take two warps of the epilogue per lane quarter.
__host__ __device__ constexpr int ctas_per_sm(int NT) { return NT <= 64 ? 2 : 1; }
constexpr int kScaleWarps = 4;  // two groups of one warp per side
__host__ __device__ constexpr int epi_warps(int NT) { return NT > 64 ? 8 : 4; }
__host__ __device__ constexpr int threads(int NT) { return 32 * (2 + kScaleWarps + epi_warps(NT)); }

constexpr int SF = 2 * 4 * 2;  // scale columns of a stage: two words of both sides' 128-row blocks
__host__ __device__ constexpr int tmem_cols(int NT) {
  const int need = 2 * NT + 2 * SF;
  return need <= 128 ? 128 : (need <= 256 ? 256 : 512);
}
__host__ __device__ constexpr int stage_bytes(int NT) { return X_BYTES + NT * BKB; }
constexpr int kChunkBytes = 2 * kWords * kWordBytes;
__host__ __device__ constexpr int stages(int NT) {
  const int room = (ctas_per_sm(NT) == 2 ? 112 : 226) * 1024 - 1024 - 512 - kTableBytes -
                   kChunkSlots * kChunkBytes;
  const int n = room / stage_bytes(NT);
  return n < kMaxStages ? n : kMaxStages;
}
__host__ __device__ constexpr int smem_bytes(int NT) {
  return 1024 + stages(NT) * stage_bytes(NT) + kChunkSlots * kChunkBytes + kTableBytes + 512;
}

// Whether a tile of nst stages is worth sharing between `split` CTAs.  Their two
// meetings and the sum cost 1 us with 32 rows of A to a tile, 2 with 64 and 2.5
// with 128, a stage takes 0.42 us, so sharing has to take 6 (9) stages off a CTA:
// 64 x 1024 takes at K = 1024 (4 stages) 7.4 us alone and 8.2 shared, at 2048 9.0
// and 8.6, at 8192 19.5 and 9.6; 128 x 1024 7.8 and 9.4, 9.8 and 10.3, 20.5 and
// 11.7; eight groups of 1024 positions, 256 x 256 each, 9.4 and 11.4.
template <int NT>
__host__ __device__ constexpr bool sharing_pays(int nst, int split) {
  return nst - (nst + split - 1) / split >= (NT > 64 ? 9 : 6);
}

// Columns [c0, c1) of the accumulator as fp32 into shared memory, [column][lane].
__device__ __forceinline__ void stage_columns(uint32_t acc, const Work& w, float* to, int x, int c0, int c1) {
  for (int c = c0; c < c1; c += 16) {
    uint32_t r[16];
    if (w.steps > 0) {
      tc::tmem_ld16(acc + c, r);
      tc::tmem_ld_wait();
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) r[k] = 0u;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) to[(c + k) * BX + x] = __uint_as_float(r[k]);
  }
}

template <int NT, int OUT>
__global__ void __launch_bounds__(threads(NT), ctas_per_sm(NT))
    mxfp4_matmul_kernel(const __grid_constant__ CUtensorMap map_x,
                        const __grid_constant__ CUtensorMap map_y, const Args a) {
  constexpr int NS = stages(NT), STAGE = stage_bytes(NT);
  constexpr int ACC = NT, TMEM = tmem_cols(NT);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* chunks = smem + NS * STAGE;
  constexpr int kEpi = epi_warps(NT), kEpi0 = 2 + kScaleWarps;
  const Groups grp = group_table(chunks + kChunkSlots * kChunkBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(grp.width + kMaxGroups + 2);  // [NS] stage copies landed
  uint64_t* empty = full + kMaxStages;     // [NS] stage MMAs complete
  uint64_t* sfull = empty + kMaxStages;    // [2] scale chunk written
  uint64_t* sempty = sfull + kChunkSlots;  // [2] scale chunk read
  uint64_t* dfull = sempty + kChunkSlots;  // [2] accumulator complete
  uint64_t* dempty = dfull + 2;            // [2] accumulator read
  uint64_t* drain = dempty + 2;            // every MMA issued has completed
  uint64_t* never = drain + 1;             // nothing completes it (testing)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kChunkSlots; ++s) {
      tc::mbar_init(&sfull[s], 2);
      tc::mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&dfull[b], 1);
      tc::mbar_init(&dempty[b], kEpi);
    }
    tc::mbar_init(drain, 1);
    tc::mbar_init(never, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_y);
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_holder, TMEM);
    tc::tmem_relinquish();
  }
  if (warp == 2) fill_groups<NT, STEP>(a, grp);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  uint32_t n_work = tiles(a, grp);
  // with a split, the CTAs of a cluster take one tile, each its share of k, or the
  // first of them the whole of a short one
  const uint32_t split = static_cast<uint32_t>(a.split);
  const uint32_t rank = split > 1 ? tc::cluster_rank() : 0u;
  const uint32_t first = blockIdx.x / split, stride = gridDim.x / split;
  bool shared = false;
  if (split > 1 && first < n_work) {
    int e = 0;  // the host knows every length but those of a weight gradient's groups
    shared = a.mode != kWgrad ||
             sharing_pays<NT>(stages_of(work_of<NT, STEP, BX>(a, grp, first, e)), a.split);
    if (!shared && rank > 0) n_work = 0;
  }
  const auto next_work = [&](uint32_t i, int& e) {
    Work w = work_of<NT, STEP, BX>(a, grp, i, e);
    if (shared) {
      const int nst = stages_of(w);
      const int s0 = static_cast<int>(rank) * nst / a.split, s1 = static_cast<int>(rank + 1) * nst / a.split;
      w.k0 += s0 * kStepsPerStage * 64;
      w.steps = min(w.steps - s0 * kStepsPerStage, (s1 - s0) * kStepsPerStage);
    }
    return w;
  };
  const int ks = static_cast<int>(a.K / 32);
  int ge = 0;  // this role's cursor over the groups

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t s = 0, phase = 0, issued = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < n_work; i += stride) {
      const Work w = next_work(i, ge);
      const int nst = stages_of(w);
      for (int st = 0; st < nst; ++st) {
        if (issued >= NS && !all_wait(&empty[s], phase ^ 1u, abort_flag, a.status)) {
          ok = false;
          break;
        }
        if (tc::elect_one()) {
          uint8_t* dst = smem + s * STAGE;
          const int kb = w.k0 / 2 + st * BKB;
          tc::mbar_arrive_expect_tx(&full[s], STAGE);
          tc::tma_load_3d(dst, &map_x, &full[s], kb, w.x0, a.mode == kGrouped ? w.e : 0);
          tc::tma_load_3d(dst + X_BYTES, &map_y, &full[s], kb, w.y0, 0);
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
    const uint64_t desc0 = tc::smem_desc_sw128(tc::smem_u32(smem));
    const uint64_t sdesc0 = tc::smem_desc_rows16(tc::smem_u32(chunks));
    uint32_t ch = 0, it = 0, s = 0, phase = 0, g = 0;
    uint32_t old = 0, old_phase = 0;  // ring slot of stage g - 2
    bool ok = injected_timeout(a, never, abort_flag);
    for (uint32_t i = first; ok && i < n_work; i += stride, ++it) {
      const Work w = next_work(i, ge);
      const uint32_t idesc = tc::idesc_mxf4(BX, (w.ny + STEP - 1) & ~(STEP - 1));
      const uint32_t d = tmem + (it & 1) * ACC;
      // accumulator it & 1 was last used by tile it - 2
      if (it >= 2 && !all_wait(&dempty[it & 1], ((it >> 1) - 1) & 1, abort_flag, a.status)) break;
      const int nst = stages_of(w);
      for (int st = 0; st < nst; ++st, ++g) {
        const int cw = st % kStagesPerChunk;
        const uint32_t cs = ch % kChunkSlots;
        if (cw == 0 && !all_wait(&sfull[cs], (ch / kChunkSlots) & 1, abort_flag, a.status)) {
          ok = false;
          break;
        }
        // the tensor-memory scale columns of stage g were last read by stage g - 2
        if (g >= 2) {
          if (!all_wait(&empty[old], old_phase, abort_flag, a.status)) {
            ok = false;
            break;
          }
          if (++old == NS) {
            old = 0;
            old_phase ^= 1u;
          }
        }
        if (!all_wait(&full[s], phase, abort_flag, a.status)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t sf = tmem + 2 * ACC + (g & 1) * SF;
        // a descriptor addresses shared memory in 16-byte units
        const uint64_t sd = sdesc0 + (cs * kChunkBytes + cw * 2 * kWordBytes) / 16;
        const uint64_t xd = desc0 + s * (STAGE / 16), yd = xd + X_BYTES / 16;
        const int left = w.steps - st * kStepsPerStage;
        if (tc::elect_one()) {
          // columns: [word 0: B, A][word 1: B, A], 4 columns each
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              tc::tmem_cp_32x128b(sf + (h * 2 + b) * 4, sd + (b * kWords + h) * (kWordBytes / 16));
#pragma unroll
          for (int k = 0; k < kStepsPerStage; ++k) {
            if (k >= left) break;
            const uint32_t sx = sf + (k >> 1) * 8, id = (k & 1) * 2;
            tc::mma_mxf4_ss(d, xd + 2 * k, yd + 2 * k, idesc | tc::idesc_sf_ids(id, id),
                            (st | k) != 0 ? 1u : 0u, sx, sx + 4);
          }
          tc::mma_commit(&empty[s]);
          if (cw == kStagesPerChunk - 1 || st == nst - 1) tc::mma_commit(&sempty[cs]);
          if (st == nst - 1) tc::mma_commit(&dfull[it & 1]);
        }
        __syncwarp();
        if (cw == kStagesPerChunk - 1 || st == nst - 1) ++ch;
        if (++s == NS) {
          s = 0;
          phase ^= 1u;
        }
      }
      // an empty sum: its zeros wait for nothing
      if (nst == 0 && tc::elect_one()) tc::mma_commit(&dfull[it & 1]);
      __syncwarp();
    }
    // completes once every operation this warp issued has finished
    if (tc::elect_one()) {
      if (it > 0 || g > 0)
        tc::mma_commit(drain);
      else
        tc::mbar_arrive(drain);
    }
  } else if (warp < kEpi0) {
    // -------------------------------------------------------- scale loaders
    // One warp per 128-row block (B's, then A's), and two groups of them that
    // take every second chunk, so one's loads are in flight while the other's
    // chunk is used.
    const uint32_t mine = static_cast<uint32_t>(warp - 2) >> 1;
    const int blk = (warp - 2) & 1;
    uint32_t ch = 0;
    bool ok = true;
    for (uint32_t i = first; ok && i < n_work; i += stride) {
      const Work w = next_work(i, ge);
      const ScaleBlock b = scale_block(a, w, blk, w.x0, ks);
      const int nch = chunks_of(w);
      for (int q = 0; q < nch; ++q, ++ch) {
        if ((ch & 1) != mine) continue;
        const uint32_t cs = ch % kChunkSlots, use = ch / kChunkSlots;
        ok = move_chunk<4>(b, q, ks, chunks + cs * kChunkBytes + blk * kWords * kWordBytes, [&] {
          return use == 0 || warp_wait(&sempty[cs], (use - 1) & 1, abort_flag, a.status, 50);
        });
        if (!ok) break;
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
    for (uint32_t i = first; i < n_work; i += stride, ++it) {
      const Work w = next_work(i, ge);
      const uint32_t b = it & 1;
      if (!warp_wait(&dfull[b], (it >> 1) & 1, abort_flag, a.status, 100)) break;
      tc::tc_fence_after();
      const int64_t n = static_cast<int64_t>(w.x0) + q * 32 + lane;
      const uint32_t acc = tmem + b * ACC + lane_base;
      // the tile's columns, split over this quarter's warps in steps of 32
      const int all = (w.ny + 15) & ~15;
      const int half = kEpi == 8 ? (all / 2 + 31) & ~31 : all;
      const int c0 = part ? min(half, all) : 0, c1 = part ? all : min(half, all);
      if (!shared)
        store_columns<OUT>(acc, a, w, n, c0, c1);
      else
        stage_columns(acc, w, reinterpret_cast<float*>(smem), q * 32 + lane, c0, c1);
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&dempty[b]);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (shared) {
    // every CTA's share of the sum lies in its ring's memory (its MMAs are done
    // with it); the columns are shared out and each is added up in rank order
    tc::cluster_sync();
    if (*abort_flag == 0) {
      int e = 0;
      const Work w = work_of<NT, STEP, BX>(a, grp, first, e);
      // 32 threads to a column of 128, four neighbours each
      constexpr int kCols = threads(NT) / 32;
      const int x = lane * 4;
      const int64_t n = static_cast<int64_t>(w.x0) + x;
      for (int c = static_cast<int>(rank) * kCols + warp; c < w.ny; c += kCols * a.split) {
        float4 part[8];
        const uint32_t off = static_cast<uint32_t>(c * BX + x) * 4;
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r)
          part[r] = r < split ? tc::ld_cluster_f32x4(tc::cluster_addr(smem, r) + off)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          v[0] += part[r].x;
          v[1] += part[r].y;
          v[2] += part[r].z;
          v[3] += part[r].w;
        }
        const int64_t at = (w.out_row + c) * a.x_rows + n;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (n + k >= a.x_rows) break;
          if (OUT == kFp32)
            static_cast<float*>(a.out)[at + k] = a.alpha * v[k];
          else
            static_cast<uint16_t*>(a.out)[at + k] = static_cast<uint16_t>(cvt_bf16x2(a.alpha * v[k], 0.f));
        }
      }
    }
    tc::cluster_sync();  // no CTA leaves while another reads its share
  }
  if (warp == 1) {
    if (lane == 0) tc::mbar_drain(drain, 0, kWaitLimitNs / 8);
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, TMEM);
  }
}

// ------------------------------------------------------------ host helpers

struct ClusterLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {};
  ClusterLaunch(unsigned grid, int block, int smem, int cluster, cudaStream_t stream) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
  }
};

// How many clusters of `size` CTAs the device runs at a time (asked once).
template <int NT, int OUT>
int clusters_at_once(int dev, int size) {
  static std::atomic<int> known[64][9];
  const bool keep = dev >= 0 && dev < 64;
  int n = keep ? known[dev][size].load() - 1 : -1;
  if (n >= 0) return n;
  ClusterLaunch l(static_cast<unsigned>(size), threads(NT), smem_bytes(NT), size, nullptr);
  if (cudaOccupancyMaxActiveClusters(&n, mxfp4_matmul_kernel<NT, OUT>, &l.cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (keep) known[dev][size].store(n + 1);
  return n;
}

template <int NT, int OUT>
moe_status launch_one(Args a, const uint8_t* xq, const uint8_t* yq, cudaStream_t stream) {
  const int64_t max_work = plan_tiles(&a, BX, NT);
  if (max_work > kMaxTiles) return MOE_ERR_SHAPE;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (!bit || !(done.load() & bit)) {
    if (cudaFuncSetAttribute(mxfp4_matmul_kernel<NT, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_bytes(NT)) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    done.fetch_or(bit);
  }
  CUtensorMap mx, my;
  if (!encode_codes(&mx, xq, a.K / 2, a.x_rows, a.mode == kGrouped ? a.E : 1, BX) ||
      !encode_codes(&my, yq, a.K / 2, a.y_rows, 1, NT))
    return MOE_ERR_CUDA;
  // Few tiles leave most SMs without one: a cluster of up to 8 CTAs shares each
  // tile's k range, as long as a CTA keeps two stages of it and all the clusters
  // run at once (23 clusters of 6 do not: 22 fit, and the last would wait).  Of a
  // weight gradient only the positions of all groups are known here: a cluster
  // whose group is short leaves it to one CTA.
  const int64_t sms = sm_count(), nst = (a.K + kStepsPerStage * 64 - 1) / (kStepsPerStage * 64);
  int64_t split = sms / max_work;
  if (split > nst / 2) split = nst / 2;
  if (split > 8) split = 8;
  while (split > 1 && clusters_at_once<NT, OUT>(dev, static_cast<int>(split)) < max_work) --split;
  a.split = split > 1 && sharing_pays<NT>(static_cast<int>(nst), static_cast<int>(split))
                ? static_cast<int>(split) : 1;
  const int64_t cap = sms * ctas_per_sm(NT);
  const int64_t ctas = a.split > 1 ? max_work * a.split : (max_work < cap ? max_work : cap);
  ClusterLaunch l(static_cast<unsigned>(ctas), threads(NT), smem_bytes(NT), a.split, stream);
  const cudaLaunchConfig_t& cfg = l.cfg;
  if (cudaLaunchKernelEx(&cfg, mxfp4_matmul_kernel<NT, OUT>, mx, my, a) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

template <int NT>
moe_status launch_nt(const Args& a, int out_type, const uint8_t* xq, const uint8_t* yq, cudaStream_t stream) {
  switch (out_of(out_type, a.x_rows)) {
    case kFp32: return launch_one<NT, kFp32>(a, xq, yq, stream);
    case kBf16Pairs: return launch_one<NT, kBf16Pairs>(a, xq, yq, stream);
    default: return launch_one<NT, kBf16>(a, xq, yq, stream);
  }
}

// Rows of A per tile: `rows` is what one tile may meet, twice the mean of a
// group where there are groups (few of which then need a second tile, which reads
// its weights again).  Groups of up to 128 take 64 even so: two CTAs of an SM hide
// each other's waits, which one of 128 rows does not.  us by tile width, bf16 out:
//   32 experts of 5760 x 2880           32 rows   64   128   pairs
//     8 rows each                          54     54    72    57
//     8 on average, one expert has 132     57     59    78    58
//     20 each                              55     57    80    63
//     20, falling from 173                 66     62    83    61
//     40 each                              86     59    78    64
//     40, falling from 329                 81     70    86    69
//     60 each                              87     61    80    67
//   128 such experts, 60 each             344    212   306   240
// (16-row tiles: 54 us and more throughout.)
// More than 128 rows take the CTA pairs, unless they are so few 128 x 128 tiles
// that two thirds of the SMs would have none: 300 x 300 takes 8.2 instead of 8.9
// us at K = 1024 and 13 instead of 26 at 16384, 800 x 700 8.6 instead of 9.2 at
// 1024 and 12.8 instead of 12.7 at 4096, 1000 x 600 x 8192 15 instead of 18; 512 x
// 2880 x 8192, at 92 tiles, takes 21 instead of 18.5.
moe_status run(const Args& a, int out_type, const uint8_t* xq, const uint8_t* yq, int64_t rows,
               cudaStream_t stream) {
  if (rows > 128 && a.x_rows > 128) {
    Args few = a;
    if (3 * plan_tiles(&few, BX, 128) > sm_count()) return launch_pair(a, out_type, xq, yq, stream);
  }
  const int NT = rows <= 32 ? 32 : (rows <= (a.mode == kGrouped ? 128 : 64) ? 64 : 128);
  switch (NT) {
    case 32: return launch_nt<32>(a, out_type, xq, yq, stream);
    case 64: return launch_nt<64>(a, out_type, xq, yq, stream);
    default: return launch_nt<128>(a, out_type, xq, yq, stream);
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
  return mxfp4_matmul_ex(a_q, a_s, b_q, b_s, M, N, K, alpha, out, out_type, d_status, -1, stream);
}

moe_status mxfp4_matmul_ex(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q,
                           const uint8_t* b_s, int64_t M, int64_t N, int64_t K, float alpha,
                           void* out, int32_t out_type, int32_t* d_status,
                           int32_t test_timeout_cta, moe_stream stream) {
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
  a.status = d_status;
  a.fail_cta = test_timeout_cta;
  return run(a, out_type, b_q, a_q, M, static_cast<cudaStream_t>(stream));
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
  a.status = d_status;
  return run(a, out_type, b_q, a_q, 2 * ((S + E - 1) / E), static_cast<cudaStream_t>(stream));
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
  a.status = d_status;
  return run(a, out_type, b_q, a_q, M, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
