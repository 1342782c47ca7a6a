// Gradient of the weighted combine and of the softmax over the chosen experts.
//
// "Welcome GPT OSS, the new open-source model family from OpenAI" (summary),
// section 4: the chosen experts' outputs are mixed with the softmax weights
// taken over the chosen experts.  With p = slot_pos[t k + j]:
//   out[t]     = sum_j w[t][j] y[p]                       (the combine)
//   dy[p]      = w[t][j] dout[t]
//   dw[t][j]   = sum_d dout[t][d] y[p][d]
//   dscore[t][j] = w[t][j] (dw[t][j] - sum_i w[t][i] dw[t][i])
// the last being the softmax's gradient with respect to the k chosen logits
// (every other logit's gradient is zero).
//
// HBM-bound: dout and the k expert rows are read once, the k gradient rows
// written once (16384 tokens, k = 4, D = 2880: 850 MB in 141 us, 6.0 TB/s, 0.93
// of the copy rate).  One CTA per token: a thread keeps 8 consecutive d of dout in
// registers for all k rows, so dout is read once, and the k partial dot
// products stay in registers until one block reduction (shuffles, then one
// fixed-order sum over the warps: the result does not depend on scheduling).
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <int K>
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                            const int32_t* __restrict__ slot_pos, const float* __restrict__ w,
                            int64_t T, int64_t S, int vec_per_row, uint4* __restrict__ dy,
                            float* __restrict__ dw, float* __restrict__ dscore) {
  __shared__ float part[kWarps][K];
  const bool dots = dw != nullptr || dscore != nullptr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    int64_t row[K];
    float wt[K], acc[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int32_t p = __ldg(slot_pos + t * K + j);
      row[j] = p >= 0 && p < S ? static_cast<int64_t>(p) * vec_per_row : -1;
      wt[j] = __ldg(w + t * K + j);
      acc[j] = 0.f;
    }
    for (int v = threadIdx.x; v < vec_per_row; v += kThreads) {
      const uint4 g = __ldg(dout + t * vec_per_row + v);
      uint4 yr[K];
#pragma unroll
      for (int j = 0; j < K; ++j)
        yr[j] = dots && row[j] >= 0 ? __ldg(y + row[j] + v) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
      float gf[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        gf[2 * q] = __uint_as_float(gw[q] << 16);
        gf[2 * q + 1] = __uint_as_float(gw[q] & 0xFFFF0000u);
      }
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (row[j] < 0) continue;
        const uint32_t yw[4] = {yr[j].x, yr[j].y, yr[j].z, yr[j].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[j] = fmaf(gf[2 * q], __uint_as_float(yw[q] << 16), acc[j]);
          acc[j] = fmaf(gf[2 * q + 1], __uint_as_float(yw[q] & 0xFFFF0000u), acc[j]);
        }
        uint4 o;
        o.x = cvt_bf16x2(wt[j] * gf[0], wt[j] * gf[1]);
        o.y = cvt_bf16x2(wt[j] * gf[2], wt[j] * gf[3]);
        o.z = cvt_bf16x2(wt[j] * gf[4], wt[j] * gf[5]);
        o.w = cvt_bf16x2(wt[j] * gf[6], wt[j] * gf[7]);
        dy[row[j] + v] = o;
      }
    }
    if (!dots) continue;
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
      if (lane == 0) part[warp][j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      float d[K], mean = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        d[j] = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) d[j] += part[i][j];
        mean = fmaf(wt[j], d[j], mean);
      }
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (dw) dw[t * K + j] = d[j];
        if (dscore) dscore[t * K + j] = wt[j] * (d[j] - mean);
      }
    }
    __syncthreads();
  }
}

template <int K>
moe_status launch_k(int grid, cudaStream_t stream, const uint16_t* dout, const uint16_t* y,
                    const int32_t* slot_pos, const float* w, const moe_shape& sh, uint16_t* dy,
                    float* dw, float* dscore) {
  return launch(combine_backward_kernel<K>, dim3(grid), dim3(kThreads), 0, stream,
                reinterpret_cast<const uint4*>(dout), reinterpret_cast<const uint4*>(y), slot_pos,
                w, static_cast<int64_t>(sh.T), static_cast<int64_t>(sh.T) * sh.k, sh.d_model / 8,
                reinterpret_cast<uint4*>(dy), dw, dscore);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_combine_backward(const uint16_t* dout, const uint16_t* y_perm,
                                           const int32_t* slot_pos, const float* topk_w,
                                           moe_shape shape, uint16_t* dy_perm, float* dtopk_w,
                                           float* dscore, moe_stream stream) {
  using namespace moe;
  if (!shape_ok(shape)) return MOE_ERR_SHAPE;
  if (shape.T == 0) return MOE_OK;
  if (!dout || !slot_pos || !topk_w || !dy_perm) return MOE_ERR_INVALID_ARG;
  if ((dtopk_w || dscore) && !y_perm) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {dout, y_perm, slot_pos, topk_w, dy_perm, dtopk_w, dscore};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  const int64_t cap = static_cast<int64_t>(sm_count()) * (2048 / kThreads);
  const int grid = static_cast<int>(shape.T < cap ? shape.T : cap);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (shape.k) {
    case 1: return launch_k<1>(grid, s, dout, y_perm, slot_pos, topk_w, shape, dy_perm, dtopk_w, dscore);
    case 2: return launch_k<2>(grid, s, dout, y_perm, slot_pos, topk_w, shape, dy_perm, dtopk_w, dscore);
    case 3: return launch_k<3>(grid, s, dout, y_perm, slot_pos, topk_w, shape, dy_perm, dtopk_w, dscore);
    case 4: return launch_k<4>(grid, s, dout, y_perm, slot_pos, topk_w, shape, dy_perm, dtopk_w, dscore);
    case 5: return launch_k<5>(grid, s, dout, y_perm, slot_pos, topk_w, shape, dy_perm, dtopk_w, dscore);
    case 6: return launch_k<6>(grid, s, dout, y_perm, slot_pos, topk_w, shape, dy_perm, dtopk_w, dscore);
    case 7: return launch_k<7>(grid, s, dout, y_perm, slot_pos, topk_w, shape, dy_perm, dtopk_w, dscore);
    default: return launch_k<8>(grid, s, dout, y_perm, slot_pos, topk_w, shape, dy_perm, dtopk_w, dscore);
  }
}
