// bf16 -> MXFP4 along the other axis: the transpose of the input, quantised in
// blocks of 32 along what were its rows.
//
// "MXFP4-based MoE technical review", section 2 (MXFP4 training): a block-scaled
// product needs its blocks along the axis it sums over, and a linear map's two
// backward products sum over the other axes than its forward product, so their
// operands are quantised again, transposed.  Format and rounding are those of
// mxfp4_quantize (csrc/quantize.cu).
//
// One CTA takes 128 rows x 128 columns.  A lane owns two neighbouring columns
// (one 32-bit word) of one 32-row block: 32 loads, each of them 128 contiguous
// bytes per warp, all in flight at once; the block maximum is then a maximum
// over the lane's own registers, with no shuffle.  The codes (16 bytes per
// column and block) go through shared memory so that the four blocks of a
// column leave as one 64-byte run.  HBM-bound: 2 bytes read and 17/32 byte
// written per element.  32 matrices of 5760 x 2880: 242 us, 5.6 TB/s, 0.87 of the
// copy rate.  (256 rows to a CTA were 10% slower; 64-bit divisions in the tile
// arithmetic cost 30%.)  Grouped, 32768 x 2880 rows in 32 groups: 49 us, 5.0 TB/s,
// 0.77 of it: each tile's group, offsets and loads follow one another, and a tile's
// stores keep the next one's loads waiting (issue slots 62% used).
//
// Grouped rows (a ragged batch sorted by expert): the output positions of a
// group start at a multiple of 128 and are zero behind its last row, so a
// product over one group's positions never meets another's, and a 128-row tile
// belongs to one group.
#include "common.cuh"
#include "e2m1.cuh"
#include "groups.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128, kCols = 128;

template <bool GROUPED>
__global__ void __launch_bounds__(kThreads)
    quantize_transposed_kernel(const uint32_t* __restrict__ w, int64_t rows, int64_t cols,
                               uint32_t batch, const int32_t* __restrict__ offsets, int E, int64_t P,
                               FastDiv col_tiles, FastDiv row_tiles,
                               uint8_t* __restrict__ q, uint8_t* __restrict__ s,
                               int32_t* __restrict__ status) {
  __shared__ uint4 codes[kCols * 4];
  __shared__ uint32_t scales[kCols];
  __shared__ int64_t pfx[kMaxGroups + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rb = warp & 3;                       // 32-row block of the tile
  const int lc = (warp >> 2) * 64 + lane * 2;    // first of this lane's two columns
  uint32_t n_tiles = batch * row_tiles.d * col_tiles.d;
  if (GROUPED) {
    if (warp == 0)
      group_prefix(E, pfx, [&](int e) {
        int64_t lo, hi;
        group_rows(offsets, e, rows, lo, hi);
        return (hi - lo + kGroupAlign - 1) / kGroupAlign;
      });
    __syncthreads();
    // no tile behind the last group's, nor past the output whatever the offsets hold
    n_tiles = min(static_cast<int64_t>(row_tiles.d), pfx[E]) * col_tiles.d;
  }
  const uint32_t pitch = static_cast<uint32_t>(cols / 2);  // words of a row
  for (uint32_t i = blockIdx.x; i < n_tiles; i += gridDim.x) {
    const uint32_t it = i / col_tiles, ct = i - it * col_tiles.d;
    const uint32_t b = GROUPED ? 0u : it / row_tiles, rt = it - b * row_tiles.d;
    int64_t r0 = static_cast<int64_t>(rt) * kRows, r_end = rows;  // source rows of the tile: [r0, r_end)
    if (GROUPED) {
      const int e = group_of(pfx, E, rt);
      int64_t lo;
      group_rows(offsets, e, rows, lo, r_end);
      r0 = lo + (rt - pfx[e]) * kRows;
    }
    const int64_t c0 = static_cast<int64_t>(ct) * kCols;
    const bool col_ok = c0 + lc < cols;  // cols is even
    const int64_t rs = r0 + rb * 32;
    const int n = col_ok ? static_cast<int>(min(max(r_end - rs, int64_t(0)), int64_t(32))) : 0;
    const uint32_t* src = w + (b * rows + rs) * static_cast<int64_t>(pitch) + (c0 + lc) / 2;
    uint32_t v[32];
    if (n == 32) {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = __ldg(src + static_cast<uint64_t>(k) * pitch);
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = k < n ? __ldg(src + static_cast<uint64_t>(k) * pitch) : 0u;
    }
    uint32_t m2 = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) m2 = __vmaxu2(m2, v[k] & 0x7FFF7FFFu);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t m = h ? m2 >> 16 : m2 & 0xFFFFu;
      const int sb = scale_byte(m);
      const float inv = inverse_scale(sb);
      uint32_t c[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t x = v[8 * g + k];
          f[k] = __uint_as_float(h ? x & 0xFFFF0000u : x << 16) * inv;
        }
        c[g] = cvt_e2m1x8(f);
      }
      // 128-byte lines of two columns, their 16-byte slots permuted by the
      // line so that neither side meets a bank conflict
      const int line = (lc + h) >> 1;
      codes[line * 8 + ((h * 4 + rb) ^ (line & 7))] = make_uint4(c[0], c[1], c[2], c[3]);
      reinterpret_cast<uint8_t*>(scales)[(lc + h) * 4 + rb] = static_cast<uint8_t>(sb);
      if (m >= 0x7F80u) record_status(status, MOE_ERR_NONFINITE);
    }
    __syncthreads();
    const int64_t p0 = static_cast<int64_t>(rt) * kRows;  // first output position
#pragma unroll
    for (int k = 0; k < kCols * 4 / kThreads; ++k) {
      const int j = threadIdx.x + k * kThreads, col = j >> 2, blk = j & 3, line = col >> 1;
      if (c0 + col < cols && p0 + blk * 32 < P)
        *reinterpret_cast<uint4*>(q + (b * cols + c0 + col) * (P / 2) + p0 / 2 + blk * 16) =
            codes[line * 8 + (((col & 1) * 4 + blk) ^ (line & 7))];
    }
    for (int j = threadIdx.x; j < kCols; j += kThreads) {
      if (c0 + j >= cols) continue;
      uint8_t* dst = s + (b * cols + c0 + j) * (P / 32) + p0 / 32;
      if (P % 128 == 0) {
        *reinterpret_cast<uint32_t*>(dst) = scales[j];
      } else {
        for (int blk = 0; blk < 4; ++blk)
          if (p0 + blk * 32 < P) dst[blk] = static_cast<uint8_t>(scales[j] >> (8 * blk));
      }
    }
    __syncthreads();
  }
}

// Checks of the pointers shared by both entries; n: rows of the input.
moe_status check(const uint16_t* w, int64_t n, const uint8_t* q, const uint8_t* s,
                 const int32_t* d_status) {
  if (n > 0 && (!w || !q || !s)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(q) || !aligned16(s)) return MOE_ERR_INVALID_ARG;
  if (d_status && (reinterpret_cast<uintptr_t>(d_status) & 3u)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

template <bool GROUPED>
moe_status launch_tiles(const uint16_t* w, int64_t batch, int64_t rows, int64_t cols, const int32_t* offsets,
                        int32_t E, int64_t P, uint8_t* q, uint8_t* s, int32_t* d_status, moe_stream stream) {
  const int64_t ct = (cols + kCols - 1) / kCols, rt = (P + kRows - 1) / kRows;
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  const int64_t tiles = batch * rt * ct;
  return launch(quantize_transposed_kernel<GROUPED>, dim3(static_cast<unsigned>(tiles < cap ? tiles : cap)),
                dim3(kThreads), 0, static_cast<cudaStream_t>(stream), reinterpret_cast<const uint32_t*>(w),
                rows, cols, static_cast<uint32_t>(batch), offsets, E, P, fast_div(static_cast<uint32_t>(ct)),
                fast_div(static_cast<uint32_t>(rt)), q, s, d_status);
}

bool sizes_ok(int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 0 || rows < 0 || cols < 8 || cols % 8) return false;
  const int64_t lim = int64_t(1) << 40;
  if (rows > (int64_t(1) << 31) || cols > (int64_t(1) << 31) || batch > lim) return false;
  if (rows > 0 && (cols > lim / rows || (batch > 0 && batch > lim / (rows * cols)))) return false;
  return true;
}

// A tile's number fits the division by multiplication (below 2^31).  A tile writes
// 8 columns of 16 bytes and more, so a refused output would not fit in 256 GB.
bool tiles_ok(int64_t batch, int64_t cols, int64_t P) {
  const int64_t ct = (cols + kCols - 1) / kCols, rt = (P + kRows - 1) / kRows;
  return batch * rt <= (int64_t(1) << 31) / ct;
}

}  // namespace
}  // namespace moe

extern "C" {

int64_t mxfp4_transposed_width(int64_t rows, int32_t E) {
  if (rows < 0 || rows > (int64_t(1) << 31) || E < 0 || E > moe::kMaxGroups) return 0;
  if (E == 0) return (rows + 31) / 32 * 32;
  const int64_t a = moe::kGroupAlign;
  return (rows + (a - 1) * E) / a * a;
}

moe_status mxfp4_quantize_transposed(const uint16_t* w_bf16, int64_t batch, int64_t rows,
                                     int64_t cols, uint8_t* q_packed, uint8_t* scales,
                                     int32_t* d_status, moe_stream stream) {
  using namespace moe;
  if (!sizes_ok(batch, rows, cols)) return MOE_ERR_SHAPE;
  if (batch == 0 || rows == 0) return MOE_OK;
  const int64_t P = mxfp4_transposed_width(rows, 0);
  if (!tiles_ok(batch, cols, P)) return MOE_ERR_SHAPE;
  moe_status st = check(w_bf16, batch * rows, q_packed, scales, d_status);
  if (st != MOE_OK) return st;
  if ((st = check_device()) != MOE_OK) return st;
  return launch_tiles<false>(w_bf16, batch, rows, cols, nullptr, 0, P, q_packed, scales, d_status, stream);
}

moe_status mxfp4_quantize_transposed_grouped(const uint16_t* w_bf16, int64_t rows, int64_t cols,
                                             const int32_t* offsets, int32_t E, uint8_t* q_packed,
                                             uint8_t* scales, int32_t* d_status,
                                             moe_stream stream) {
  using namespace moe;
  if (!sizes_ok(1, rows, cols) || E < 1 || E > kMaxGroups) return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  const int64_t P = mxfp4_transposed_width(rows, E);
  if (!tiles_ok(1, cols, P)) return MOE_ERR_SHAPE;
  if (!offsets || !aligned16(offsets)) return MOE_ERR_INVALID_ARG;
  moe_status st = check(w_bf16, rows, q_packed, scales, d_status);
  if (st != MOE_OK) return st;
  if ((st = check_device()) != MOE_OK) return st;
  return launch_tiles<true>(w_bf16, 1, rows, cols, offsets, E, P, q_packed, scales, d_status, stream);
}

}  // extern "C"
