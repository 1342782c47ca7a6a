// Gradient of the sort by expert, with the router's share of it.
//
// "MXFP4-based MoE technical review", section 4 (routing over sparse
// experts); "Welcome GPT OSS ..." (summary), section 4 (softmax over the
// chosen experts' scores only).  A token's row is copied to k places of the
// permuted order, so its gradient is the sum of theirs; the router's scores
// x . Wr_e depend on it too, and only the k chosen ones have a gradient:
//   dx[t][d] = sum_j dx_perm[slot_pos[t k + j]][d]
//            + sum_j dscore[t][j] * Wr[topk_idx[t][j]][d]
// summed in fp32, j ascending, rounded once to bf16.
//
// HBM-bound: (k + 1) * 2 bytes per output element (the router matrix stays in
// L2).  16384 tokens, k = 4, D = 2880 with the router's share: 473 MB in 80 us,
// 5.9 TB/s, 0.91 of the copy rate (bf16 by one conversion per pair: 85 us with
// the bitwise rounding).  Each thread owns 8 consecutive d of one token, with all of its 16-byte
// loads in flight before the first sum.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void add8(float (&acc)[8], uint4 r, float f) {
  const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    acc[2 * q] = fmaf(f, __uint_as_float(rr[q] << 16), acc[2 * q]);
    acc[2 * q + 1] = fmaf(f, __uint_as_float(rr[q] & 0xFFFF0000u), acc[2 * q + 1]);
  }
}

template <int K, bool ROUTER>
__global__ void __launch_bounds__(kThreads)
    permute_backward_kernel(const uint4* __restrict__ dx_perm, const int32_t* __restrict__ slot_pos,
                            const int32_t* __restrict__ idx, const float* __restrict__ dscore,
                            const uint4* __restrict__ w_router, int E, uint32_t n, int S,
                            FastDiv vec_per_row, uint4* __restrict__ dx) {
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) {
    const uint32_t t = i / vec_per_row;
    const int v = static_cast<int>(i - t * vec_per_row.d);
    uint4 r[K], wr[K];
    float ds[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int32_t p = __ldg(slot_pos + t * K + j);
      r[j] = p >= 0 && p < S ? __ldg(dx_perm + static_cast<int64_t>(p) * vec_per_row.d + v)
                             : make_uint4(0u, 0u, 0u, 0u);
      if (ROUTER) {
        const int e = __ldg(idx + t * K + j);
        const bool in = static_cast<unsigned>(e) < static_cast<unsigned>(E);
        wr[j] = in ? __ldg(w_router + static_cast<int64_t>(e) * vec_per_row.d + v)
                   : make_uint4(0u, 0u, 0u, 0u);
        ds[j] = in ? __ldg(dscore + t * K + j) : 0.f;
      }
    }
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) add8(acc, r[j], 1.f);
    if (ROUTER) {
#pragma unroll
      for (int j = 0; j < K; ++j) add8(acc, wr[j], ds[j]);
    }
    uint4 o;
    o.x = cvt_bf16x2(acc[0], acc[1]);
    o.y = cvt_bf16x2(acc[2], acc[3]);
    o.z = cvt_bf16x2(acc[4], acc[5]);
    o.w = cvt_bf16x2(acc[6], acc[7]);
    dx[i] = o;
  }
}

template <int K>
moe_status launch_k(cudaStream_t stream, const uint16_t* dx_perm, const int32_t* slot_pos,
                    const int32_t* idx, const float* dscore, const uint16_t* w_router,
                    const moe_shape& sh, uint16_t* dx) {
  const int vec = sh.d_model / 8;
  const int64_t want = (static_cast<int64_t>(sh.T) * vec + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(sm_count()) * 16;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
  // T D / 8 <= 2^31: every index fits the division by multiplication
  const uint32_t n = static_cast<uint32_t>(static_cast<int64_t>(sh.T) * vec);
  const int S = sh.T * sh.k;
  const FastDiv fd = fast_div(static_cast<uint32_t>(vec));
  const uint4* in = reinterpret_cast<const uint4*>(dx_perm);
  const uint4* wr = reinterpret_cast<const uint4*>(w_router);
  uint4* out = reinterpret_cast<uint4*>(dx);
  return w_router ? launch(permute_backward_kernel<K, true>, grid, dim3(kThreads), 0, stream, in,
                           slot_pos, idx, dscore, wr, sh.E, n, S, fd, out)
                  : launch(permute_backward_kernel<K, false>, grid, dim3(kThreads), 0, stream, in,
                           slot_pos, idx, dscore, wr, sh.E, n, S, fd, out);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_permute_backward(const uint16_t* dx_perm, const int32_t* slot_pos,
                                           moe_shape shape, uint16_t* dx, const int32_t* topk_idx,
                                           const float* dscore, const uint16_t* w_router,
                                           moe_stream stream) {
  using namespace moe;
  if (!shape_ok(shape)) return MOE_ERR_SHAPE;
  if (shape.T == 0) return MOE_OK;
  if (!dx_perm || !slot_pos || !dx) return MOE_ERR_INVALID_ARG;
  // the router's share needs all three of its arguments, or none
  const bool router = w_router != nullptr;
  if ((topk_idx != nullptr) != router || (dscore != nullptr) != router) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {dx_perm, slot_pos, dx, topk_idx, dscore, w_router};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
  moe_status st = check_device();
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (shape.k) {
    case 1: return launch_k<1>(s, dx_perm, slot_pos, topk_idx, dscore, w_router, shape, dx);
    case 2: return launch_k<2>(s, dx_perm, slot_pos, topk_idx, dscore, w_router, shape, dx);
    case 3: return launch_k<3>(s, dx_perm, slot_pos, topk_idx, dscore, w_router, shape, dx);
    case 4: return launch_k<4>(s, dx_perm, slot_pos, topk_idx, dscore, w_router, shape, dx);
    case 5: return launch_k<5>(s, dx_perm, slot_pos, topk_idx, dscore, w_router, shape, dx);
    case 6: return launch_k<6>(s, dx_perm, slot_pos, topk_idx, dscore, w_router, shape, dx);
    case 7: return launch_k<7>(s, dx_perm, slot_pos, topk_idx, dscore, w_router, shape, dx);
    default: return launch_k<8>(s, dx_perm, slot_pos, topk_idx, dscore, w_router, shape, dx);
  }
}
