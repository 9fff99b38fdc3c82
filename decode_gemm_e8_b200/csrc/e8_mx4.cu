// Microscaled 4-bit form: encoder and decoder.
//
// Both are one pass over the data and bound by HBM: the encoder reads 2 or 4
// bytes a value and writes 17/32, the decoder the other way round (2 written).
// Four lanes hold one block of 32 (8 values each), so a warp reads 256
// consecutive values of a row in 16-byte loads, the block's maximum takes two
// shuffles, each lane converts its 8 values with the hardware e2m1 conversion
// (round to nearest even, saturating: the form's own rule) and the warp writes
// 128 consecutive bytes of codes.  The scale exponent is the exponent field of
// the maximum, and the division by it is an exact multiplication.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "e8_internal.h"
#include "e8_mx4.cuh"

namespace e8 {
namespace mx4 {

constexpr int kThreads = 256;
constexpr int kRows = 4;   // rows a warp has in flight at once

template <int DT> struct Elem;
template <> struct Elem<0> { using T = uint16_t; };
template <> struct Elem<1> { using T = uint16_t; };
template <> struct Elem<2> { using T = float; };

template <int DT>
__device__ __forceinline__ float to_float(typename Elem<DT>::T v) {
  if constexpr (DT == 0) return __uint_as_float((uint32_t)v << 16);
  else if constexpr (DT == 1) return __half2float(__ushort_as_half(v));
  else return v;
}

// Eight values of a row from column c on (zeros past K).
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const typename Elem<DT>::T* __restrict__ row, int64_t c,
                                      int64_t K, float (&v)[8]) {
  if (VEC && c + 8 <= K) {
    if constexpr (DT == 2) {
      const float4 a = *reinterpret_cast<const float4*>(row + c);
      const float4 b = *reinterpret_cast<const float4*>(row + c + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(row + c);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = to_float<DT>((uint16_t)(w[i] & 0xFFFFu));
        v[2 * i + 1] = to_float<DT>((uint16_t)(w[i] >> 16));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < K ? to_float<DT>(row[c + i]) : 0.0f;
  }
}

// One warp job: kRows rows of one 256-column chunk.  Rows run to the next
// multiple of 128 so that the padding rows' scales are written as zero.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
    k_mx4_encode(const typename Elem<DT>::T* __restrict__ X, int64_t rows, int64_t K, int64_t ldx,
                 uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t jobs,
                 int64_t chunks, int64_t row_groups, int release) {
  if (release) grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t cs = code_stride(K), kqs = scale_tiles(K), sb = scale_bytes(rows, K);
  const int64_t job = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (job >= jobs) return;
  const int64_t chunk = job % chunks, rest = job / chunks;
  const int64_t row0 = rest % row_groups * kRows, b = rest / row_groups;
  const int64_t c = chunk * 256 + lane * 8;
  X += b * rows * ldx;
  codes += b * rows * cs;
  scales += b * sb;
  float v[kRows][8];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (row0 + r < rows) {
      load8<DT, VEC>(X + (row0 + r) * ldx, c, K, v[r]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][i] = 0.0f;
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    // the maximum of the magnitudes' bits: a NaN or an infinity wins
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[r][i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t byte = scale_byte(__uint_as_float(m));
    uint32_t code = 0;
    if (byte != 255u) {
      const float inv = inv_scale(byte);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][i] *= inv;
      code = pack8(v[r]);
    }
    const int64_t row = row0 + r;
    if (row < rows && c / 2 < cs) *reinterpret_cast<uint32_t*>(codes + row * cs + c / 2) = code;
    // lanes 0 and 16 collect the four bytes of their 128-column tile (blocks
    // past the matrix hold zeros, whose byte is 0)
    const int base = lane & 16;
    uint32_t q = __shfl_sync(0xFFFFFFFFu, byte, base);
    q |= __shfl_sync(0xFFFFFFFFu, byte, base + 4) << 8;
    q |= __shfl_sync(0xFFFFFFFFu, byte, base + 8) << 16;
    q |= __shfl_sync(0xFFFFFFFFu, byte, base + 12) << 24;
    const int64_t kq = chunk * 2 + (lane >> 4);
    if ((lane & 15) == 0 && kq < kqs)
      *reinterpret_cast<uint32_t*>(scales + scale_at(row, kq, kqs)) = q;
  }
}

// One warp job: kRows rows of one 256-column chunk, 8 values a lane.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
    k_mx4_decode(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                 int64_t rows, int64_t K, uint16_t* __restrict__ out, int64_t jobs, int64_t chunks,
                 int64_t row_groups) {
  const int lane = threadIdx.x & 31;
  const int64_t cs = code_stride(K), kqs = scale_tiles(K), sb = scale_bytes(rows, K);
  const int64_t job = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (job >= jobs) return;
  const int64_t chunk = job % chunks, rest = job / chunks;
  const int64_t row0 = rest % row_groups * kRows, b = rest / row_groups;
  const int64_t c = chunk * 256 + lane * 8;
  if (c >= K) return;
  codes += b * rows * cs;
  scales += b * sb;
  out += b * rows * K;
  const int64_t kq = c >> 7;
  uint32_t code[kRows], byte[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t row = row0 + r;
    code[r] = byte[r] = 0;
    if (row < rows) {
      code[r] = *reinterpret_cast<const uint32_t*>(codes + row * cs + c / 2);
      byte[r] = scales[scale_at(row, kq, kqs) + ((c >> 5) & 3)];
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t row = row0 + r;
    if (row >= rows) return;
    const float s = scale_value(byte[r]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = code_value(code[r] >> (4 * i)) * s;
    uint16_t* o = out + row * K + c;
    if (VEC && c + 8 <= K) {
      *reinterpret_cast<uint4*>(o) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < K) o[i] = (uint16_t)(pack_bf16x2(v[i], 0.0f) & 0xFFFFu);
    }
  }
}

struct Jobs {
  int64_t jobs, chunks, row_groups;
  unsigned grid;
};
static bool plan(int64_t batch, int64_t rows, int64_t K, bool pad_rows, Jobs* j) {
  j->chunks = (K + 255) / 256;
  j->row_groups = pad_rows ? (rows + 127) / 128 * (128 / kRows) : (rows + kRows - 1) / kRows;
  j->jobs = batch * j->row_groups * j->chunks;
  const int64_t grid = (j->jobs + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > INT32_MAX) return false;
  j->grid = (unsigned)grid;
  return true;
}

template <int DT>
static cudaError_t encode_as(const void* X, int64_t batch, int64_t rows, int64_t K, int64_t ldx,
                             uint8_t* codes, uint8_t* scales, int release, cudaStream_t st) {
  using T = typename Elem<DT>::T;
  Jobs j;
  if (!plan(batch, rows, K, true, &j)) return cudaErrorInvalidValue;
  const T* x = static_cast<const T*>(X);
  // 16-byte loads need every row to start on 16 bytes
  const bool vec = aligned16(X) && (ldx * (int64_t)sizeof(T)) % 16 == 0;
  if (vec)
    k_mx4_encode<DT, true><<<j.grid, kThreads, 0, st>>>(x, rows, K, ldx, codes, scales, j.jobs,
                                                        j.chunks, j.row_groups, release);
  else
    k_mx4_encode<DT, false><<<j.grid, kThreads, 0, st>>>(x, rows, K, ldx, codes, scales, j.jobs,
                                                         j.chunks, j.row_groups, release);
  return cudaGetLastError();
}

}  // namespace mx4

cudaError_t launch_mx4_encode(const void* X, int dtype, int64_t batch, int64_t rows, int64_t K,
                              int64_t ldx, uint8_t* codes, uint8_t* scales, int release,
                              cudaStream_t st) {
  if (dtype == 0) return mx4::encode_as<0>(X, batch, rows, K, ldx, codes, scales, release, st);
  if (dtype == 1) return mx4::encode_as<1>(X, batch, rows, K, ldx, codes, scales, release, st);
  return mx4::encode_as<2>(X, batch, rows, K, ldx, codes, scales, release, st);
}

cudaError_t launch_mx4_decode(const uint8_t* codes, const uint8_t* scales, int64_t batch,
                              int64_t rows, int64_t K, uint16_t* out, cudaStream_t st) {
  mx4::Jobs j;
  if (!mx4::plan(batch, rows, K, false, &j)) return cudaErrorInvalidValue;
  if (K % 8 == 0)
    mx4::k_mx4_decode<true><<<j.grid, mx4::kThreads, 0, st>>>(codes, scales, rows, K, out, j.jobs,
                                                              j.chunks, j.row_groups);
  else
    mx4::k_mx4_decode<false><<<j.grid, mx4::kThreads, 0, st>>>(codes, scales, rows, K, out, j.jobs,
                                                               j.chunks, j.row_groups);
  return cudaGetLastError();
}

}  // namespace e8
