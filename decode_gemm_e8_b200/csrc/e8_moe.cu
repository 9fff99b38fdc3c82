// Mixture-of-experts layer for a few tokens, experts in the microscaled 4-bit
// form: router, the chosen experts' gate and up products, the activation, the
// down products and their weighted sum.
//
// Bound by the bytes of the chosen experts' weights (17/32 a value).
#include "e8_internal.h"
#include "e8_mx4.cuh"

namespace e8 {
namespace moe {

constexpr int kMaxExperts = 512;

// One CTA a token.  Products of two bf16 are exact in fp32; the sums are fp64,
// so that another order of adding cannot change which experts are chosen.
__global__ void __launch_bounds__(256)
    k_moe_route(const uint16_t* __restrict__ X, int H, const uint16_t* __restrict__ R, int E,
                int topk, int renorm, int32_t* __restrict__ experts, float* __restrict__ probs,
                int32_t* __restrict__ experts_out, float* __restrict__ probs_out) {
  __shared__ double logit[kMaxExperts];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint16_t* x = X + (size_t)t * H;
  for (int e = warp; e < E; e += 8) {
    double s = 0.0;
    for (int k = lane; k < H; k += 32)
      s += (double)(__uint_as_float((uint32_t)x[k] << 16) *
                    __uint_as_float((uint32_t)R[(size_t)e * H + k] << 16));
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) logit[e] = s;
  }
  __syncthreads();
  if (warp) return;
  uint32_t taken = 0;   // bit j: expert lane + 32 j
  double top = 0.0;
  float chosen_sum = 0.0f, mine = 0.0f;
  int mine_e = 0;
  for (int i = 0; i < topk; ++i) {
    // key order: larger logit, then lower expert; NaN below everything
    int be = INT32_MAX;
    double bv = 0.0;
    bool bnan = true;
    for (int e = lane, j = 0; e < E; e += 32, ++j) {
      if (taken >> j & 1u) continue;
      const double v = logit[e];
      const bool nan = v != v;
      if (be == INT32_MAX || (bnan && !nan) || (!bnan && !nan && v > bv)) {
        be = e;
        bv = v;
        bnan = nan;
      }
    }
    for (int o = 16; o; o >>= 1) {
      const int oe = __shfl_xor_sync(0xFFFFFFFFu, be, o);
      const double ov = __shfl_xor_sync(0xFFFFFFFFu, bv, o);
      const bool on = __shfl_xor_sync(0xFFFFFFFFu, (int)bnan, o) != 0;
      bool take;
      if (oe == INT32_MAX) take = false;
      else if (be == INT32_MAX) take = true;
      else if (on != bnan) take = bnan;
      else if (!on && ov != bv) take = ov > bv;
      else take = oe < be;
      if (take) {
        be = oe;
        bv = ov;
        bnan = on;
      }
    }
    if (i == 0) top = bv;
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
    const float p = expf((float)(bv - top));
    chosen_sum += p;
    if (lane == i) {
      mine = p;
      mine_e = be;
    }
  }
  float sum = chosen_sum;
  if (!renorm) {
    sum = 0.0f;
    for (int e = lane; e < E; e += 32) sum += expf((float)(logit[e] - top));
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  }
  if (lane < topk) {
    experts[t * topk + lane] = mine_e;
    probs[t * topk + lane] = mine / sum;
    if (experts_out) experts_out[t * topk + lane] = mine_e;
    if (probs_out) probs_out[t * topk + lane] = mine / sum;
  }
}

// One lane's share of a row's dot product with x: blocks of 32 in turn.
__device__ __forceinline__ float row_dot(const uint8_t* __restrict__ codes,
                                         const uint8_t* __restrict__ scales, int64_t row, int K,
                                         const float* __restrict__ x, int lane) {
  const int64_t cs = mx4::code_stride(K), kqs = mx4::scale_tiles(K);
  float acc = 0.0f;
  for (int c = lane * 8; c < K; c += 256) {
    const uint32_t code = *reinterpret_cast<const uint32_t*>(codes + row * cs + c / 2);
    const float s =
        mx4::scale_value(scales[mx4::scale_at(row, c >> 7, kqs) + ((c >> 5) & 3)]);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) d = fmaf(mx4::code_value(code >> (4 * i)), x[c + i], d);
    acc = fmaf(d, s, acc);
  }
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  return acc;
}

// Grid (I / 32, T * topk): 32 values of h for one chosen expert of one token.
__global__ void __launch_bounds__(256)
    k_moe_up(const uint16_t* __restrict__ X, int H, const int32_t* __restrict__ experts, int topk,
             const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int I,
             float* __restrict__ h) {
  extern __shared__ float xs[];
  const int slot = blockIdx.y, t = slot / topk, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = experts[slot];
  for (int k = threadIdx.x; k < H; k += 256)
    xs[k] = __uint_as_float((uint32_t)X[(size_t)t * H + k] << 16);
  __syncthreads();
  codes += (int64_t)e * 2 * I * mx4::code_stride(H);
  scales += (int64_t)e * mx4::scale_bytes(2 * I, H);
  for (int j = 0; j < 4; ++j) {
    const int i = blockIdx.x * 32 + warp * 4 + j;
    const float g = row_dot(codes, scales, 2 * i, H, xs, lane);
    const float u = row_dot(codes, scales, 2 * i + 1, H, xs, lane);
    if (lane == 0) h[(size_t)slot * I + i] = g / (1.0f + expf(-g)) * u;
  }
}

// Grid (H / 32, T): 32 outputs of one token, its experts in turn.
__global__ void __launch_bounds__(256)
    k_moe_down(const float* __restrict__ h, int I, const int32_t* __restrict__ experts,
               const float* __restrict__ probs, int topk, const uint8_t* __restrict__ codes,
               const uint8_t* __restrict__ scales, int H, uint16_t* __restrict__ Y) {
  const int t = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = 0; j < 4; ++j) {
    const int row = blockIdx.x * 32 + warp * 4 + j;
    float y = 0.0f;
    for (int s = t * topk; s < (t + 1) * topk; ++s) {
      const int64_t e = experts[s];
      y = fmaf(probs[s], row_dot(codes + e * H * mx4::code_stride(I),
                                 scales + e * mx4::scale_bytes(H, I), row, I, h + (size_t)s * I,
                                 lane), y);
    }
    if (lane == 0) Y[(size_t)t * H + row] = (uint16_t)(pack_bf16x2(y, 0.0f) & 0xFFFFu);
  }
}

}  // namespace moe

// Workspace: experts [T topk], probs [T topk], h fp32 [T topk][I].
size_t moe_workspace(int64_t T, int64_t H, int64_t E, int topk, int64_t I) {
  (void)H; (void)E;
  const size_t slots = (size_t)T * topk, part = (slots * 4 + 255) & ~size_t(255);
  return 2 * part + ((slots * I * 4 + 255) & ~size_t(255));
}

cudaError_t launch_moe(const MoeArgs& a, int sm_count, cudaStream_t st) {
  (void)sm_count;
  const int slots = a.T * a.topk;
  const size_t part = ((size_t)slots * 4 + 255) & ~size_t(255);
  uint8_t* w = static_cast<uint8_t*>(a.workspace);
  int32_t* experts = reinterpret_cast<int32_t*>(w);
  float* probs = reinterpret_cast<float*>(w + part);
  float* h = reinterpret_cast<float*>(w + 2 * part);
  moe::k_moe_route<<<a.T, 256, 0, st>>>(a.X, a.H, a.router, a.E, a.topk, a.renorm, experts, probs,
                                        a.experts, a.probs);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = ensure_smem_limit(moe::k_moe_up, kMaxDynSmem);
  if (e != cudaSuccess) return e;
  moe::k_moe_up<<<dim3(a.I / 32, slots), 256, (size_t)a.H * 4, st>>>(a.X, a.H, experts, a.topk,
                                                                    a.w13_codes, a.w13_scales, a.I,
                                                                    h);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  moe::k_moe_down<<<dim3(a.H / 32, a.T), 256, 0, st>>>(h, a.I, experts, probs, a.topk, a.w2_codes,
                                                       a.w2_scales, a.H, a.Y);
  return cudaGetLastError();
}

}  // namespace e8
