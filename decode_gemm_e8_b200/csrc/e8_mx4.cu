// Microscaled 4-bit form: encoder and decoder.
//
// Both are one pass over the data and bound by HBM: the encoder reads 2 or 4
// bytes a value and writes 17/32, the decoder the other way round (2 written).
// What they must not do is compute more than HBM allows, about 5 instructions a
// value: four lanes hold one block of 32 (8 values each), so a warp reads 256
// consecutive values of a row in 16-byte loads; for 16-bit types the block's
// maximum is taken on packed pairs of bit patterns; each lane converts its 8 values
// with the hardware e2m1 conversion (round to nearest even, saturating: the form's
// own rule) and the warp writes 128 consecutive bytes of codes.  The scale exponent
// is the exponent field of the maximum, and the division by it is an exact
// multiplication.  The decoder looks codes up as bf16 bytes (byte permutation) and
// scales pairs.  Rows that do not start on 16 bytes go one value a lane, so that every
// load or store of a warp is still of neighbouring values: a block is then a whole
// warp's, and nibbles or codes travel by shuffles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "e8_internal.h"
#include "e8_mx4.cuh"

namespace e8 {
namespace mx4 {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
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
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight values of a row from column c on (zeros past K), as they lie in memory.
template <int DT>
struct Eight {
  uint32_t w[DT == 2 ? 8 : 4];
  __device__ __forceinline__ void load(const typename Elem<DT>::T* __restrict__ row, int64_t c,
                                       int64_t K) {
    if (c + 8 <= K) {
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(row + c));
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      if constexpr (DT == 2) {
        const uint4 b = __ldcs(reinterpret_cast<const uint4*>(row + c + 4));
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
      }
    } else {
      zero();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < K) {
          if constexpr (DT == 2) w[i] = __float_as_uint(row[c + i]);
          else w[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
        }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& v : w) v = 0;
  }
  // bits of the largest magnitude over the lanes of a block, as fp32: magnitudes
  // compare as integers, and a NaN or an infinity wins
  __device__ __forceinline__ float block_max() const {
    uint32_t m = 0;
    if constexpr (DT == 2) {
#pragma unroll
      for (uint32_t v : w) m = max(m, v & 0x7FFFFFFFu);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      return __uint_as_float(m);
    } else {
#pragma unroll
      for (uint32_t v : w) m = max_u16x2(m, v & 0x7FFF7FFFu);
      m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      return to_float<DT>((uint16_t)max(m & 0xFFFFu, m >> 16));
    }
  }
  __device__ __forceinline__ uint32_t codes(float inv) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (DT == 2) v[i] = __uint_as_float(w[i]) * inv;
      else if constexpr (DT == 0)
        v[i] = ((i & 1) ? bf16_hi_to_f32(w[i / 2]) : bf16_lo_to_f32(w[i / 2])) * inv;
      else v[i] = to_float<1>((uint16_t)(w[i / 2] >> (16 * (i & 1)))) * inv;
    }
    return pack8(v);
  }
};

// Grid: x 256-column chunks, y blocks of 8 x kRows rows, z matrices.  Rows run to the
// next multiple of 128 so that the padding rows' scales are written as zero.
template <int DT>
__global__ void __launch_bounds__(kThreads, 4)
    k_mx4_encode(const typename Elem<DT>::T* __restrict__ X, int64_t batch, int64_t rows,
                 int64_t rows_padded, int64_t K, int64_t ldx, uint8_t* __restrict__ codes,
                 uint8_t* __restrict__ scales, int release) {
  if (release) grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cs = code_stride(K), kqs = scale_tiles(K);
  const int64_t c = (int64_t)blockIdx.x * 256 + lane * 8;
  const int64_t kq = (int64_t)blockIdx.x * 2 + (lane >> 4);
  const bool code_lane = c / 2 < cs, scale_lane = (lane & 15) == 0 && kq < kqs;
  for (int64_t b = blockIdx.z; b < batch; b += gridDim.z) {
    const typename Elem<DT>::T* x = X + b * rows * ldx;
    uint8_t* to = codes + b * rows * cs + c / 2;
    uint8_t* sc = scales + b * rows_padded / 128 * kqs * 512;
    for (int64_t row0 = ((int64_t)blockIdx.y * kWarps + warp) * kRows; row0 < rows_padded;
         row0 += (int64_t)gridDim.y * kWarps * kRows) {
      Eight<DT> v[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (row0 + r < rows) v[r].load(x + (row0 + r) * ldx, c, K);
        else v[r].zero();
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t row = row0 + r;
        const uint32_t byte = scale_byte(v[r].block_max());
        const uint32_t code = byte == 255u ? 0u : v[r].codes(inv_scale(byte));
        if (row < rows && code_lane) *reinterpret_cast<uint32_t*>(to + row * cs) = code;
        // the four bytes of a 128-column tile meet in lanes 0 and 16 (blocks past the
        // matrix hold zeros, whose byte is 0)
        uint32_t q = byte | __shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8;
        q |= __shfl_down_sync(0xFFFFFFFFu, q, 8) << 16;
        if (scale_lane) *reinterpret_cast<uint32_t*>(sc + scale_at(row, kq, kqs)) = q;
      }
    }
  }
}

// The same for rows that do not start on 16 bytes: load i of a warp is its block i.
template <int DT>
__global__ void __launch_bounds__(kThreads, 4)
    k_mx4_encode_any(const typename Elem<DT>::T* __restrict__ X, int64_t batch, int64_t rows,
                     int64_t rows_padded, int64_t K, int64_t ldx, uint8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales, int release) {
  if (release) grid_dep_launch();
  constexpr int kR = 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cs = code_stride(K), kqs = scale_tiles(K);
  const int64_t c0 = (int64_t)blockIdx.x * 256;
  for (int64_t b = blockIdx.z; b < batch; b += gridDim.z) {
    const typename Elem<DT>::T* x = X + b * rows * ldx + c0 + lane;
    uint8_t* to = codes + b * rows * cs + c0 / 2;
    uint8_t* sc = scales + b * rows_padded / 128 * kqs * 512;
    for (int64_t row0 = ((int64_t)blockIdx.y * kWarps + warp) * kR; row0 < rows_padded;
         row0 += (int64_t)gridDim.y * kWarps * kR) {
      float v[kR][8];
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[r][i] = row0 + r < rows && c0 + 32 * i + lane < K
                        ? to_float<DT>(__ldcs(x + (row0 + r) * ldx + 32 * i)) : 0.0f;
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int64_t row = row0 + r;
        uint32_t word = 0, q[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t m =
              __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[r][i]) & 0x7FFFFFFFu);
          const uint32_t byte = scale_byte(__uint_as_float(m));
          q[i / 4] |= byte << (8 * (i & 3));
          float e[8] = {byte == 255u ? 0.0f : v[r][i] * inv_scale(byte)};
          // the code is the low nibble of lane % 8; eight lanes make a word
          uint32_t n = (pack8(e) & 15u) << (4 * (lane & 7));
          n |= __shfl_xor_sync(0xFFFFFFFFu, n, 1);
          n |= __shfl_xor_sync(0xFFFFFFFFu, n, 2);
          n |= __shfl_xor_sync(0xFFFFFFFFu, n, 4);
          // lane 4 i + j keeps word j of block i
          const uint32_t mine = __shfl_sync(0xFFFFFFFFu, n, (lane & 3) * 8);
          if (lane >> 2 == i) word = mine;
        }
        if (row < rows && c0 / 2 + lane * 4 < cs)
          *reinterpret_cast<uint32_t*>(to + row * cs + lane * 4) = word;
        if (lane < 2 && (int64_t)blockIdx.x * 2 + lane < kqs)
          *reinterpret_cast<uint32_t*>(sc + scale_at(row, (int64_t)blockIdx.x * 2 + lane, kqs)) =
              lane ? q[1] : q[0];
      }
    }
  }
}

// Codes 0..3 (low 16 bits of w) -> two bf16 pairs, unscaled: magnitudes 0, .5, 1, 1.5,
// 2, 3, 4, 6 are 0000 3F00 3F80 3FC0 4000 4040 4080 40C0 in bf16.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& a, uint32_t& b) {
  const uint32_t sel = w & 0x7777u;
  const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel);
  const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
  a = __byte_perm(lo, hi, 0x5140) | ((w << 12) & 0x8000u) | ((w << 24) & 0x80000000u);
  b = __byte_perm(lo, hi, 0x7362) | ((w << 4) & 0x8000u) | ((w << 16) & 0x80000000u);
}
// 2^(byte - 127) in both halves: subnormal for byte 0, NaN for byte 255.
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t byte) {
  const uint32_t s = byte == 0u ? 0x0040u : (byte == 255u ? 0x7FC0u : byte << 7);
  return s | s << 16;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Grid as the encoder's.  VEC: every row of `out` starts on 16 bytes.
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 4)
    k_mx4_decode(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                 int64_t batch, int64_t rows, int64_t K, uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cs = code_stride(K), kqs = scale_tiles(K), sb = scale_bytes(rows, K);
  const int64_t c0 = (int64_t)blockIdx.x * 256, c = c0 + lane * 8, kq = c >> 7;
  const bool in = c / 2 < cs;
  for (int64_t b = blockIdx.z; b < batch; b += gridDim.z) {
    const uint8_t* from = codes + b * rows * cs + c / 2;
    const uint8_t* sc = scales + b * sb + ((c >> 5) & 3);
    uint16_t* to = out + b * rows * K;
    for (int64_t row0 = ((int64_t)blockIdx.y * kWarps + warp) * kRows; row0 < rows;
         row0 += (int64_t)gridDim.y * kWarps * kRows) {
      uint32_t code[kRows], byte[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const bool ok = in && row0 + r < rows;
        code[r] = ok ? __ldcs(reinterpret_cast<const uint32_t*>(from + (row0 + r) * cs)) : 0u;
        byte[r] = ok ? sc[scale_at(row0 + r, kq, kqs)] : 0u;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t row = row0 + r;
        if (row >= rows) break;
        uint32_t v[4];
        codes_to_bf16(code[r], v[0], v[1]);
        codes_to_bf16(code[r] >> 16, v[2], v[3]);
        const uint32_t s = scale_bf16x2(byte[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul_bf16x2(v[i], s);
        if (VEC) {
          // K is a multiple of 8 here
          if (c < K)
            __stcs(reinterpret_cast<uint4*>(to + row * K + c), make_uint4(v[0], v[1], v[2], v[3]));
        } else {
          // store i: 32 neighbouring values, value `lane` of which is element lane % 8
          // of lane 4 i + lane / 8
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int src = 4 * i + (lane >> 3);
            const uint32_t p0 = __shfl_sync(0xFFFFFFFFu, v[0], src),
                           p1 = __shfl_sync(0xFFFFFFFFu, v[1], src),
                           p2 = __shfl_sync(0xFFFFFFFFu, v[2], src),
                           p3 = __shfl_sync(0xFFFFFFFFu, v[3], src);
            const uint32_t p = lane & 4 ? (lane & 2 ? p3 : p2) : (lane & 2 ? p1 : p0);
            if (c0 + 32 * i + lane < K)
              to[row * K + c0 + 32 * i + lane] = (uint16_t)(lane & 1 ? p >> 16 : p);
          }
        }
      }
    }
  }
}

// Row blocks and matrices beyond the grid's limits are walked in the kernels' loops.
static dim3 grid_of(int64_t batch, int64_t rows, int64_t K, int rows_a_block) {
  const int64_t y = (rows + rows_a_block - 1) / rows_a_block;
  return dim3((unsigned)((K + 255) / 256), (unsigned)(y < 65535 ? y : 65535),
              (unsigned)(batch < 65535 ? batch : 65535));
}

template <int DT>
static cudaError_t encode_as(const void* X, int64_t batch, int64_t rows, int64_t K, int64_t ldx,
                             uint8_t* codes, uint8_t* scales, int release, cudaStream_t st) {
  using T = typename Elem<DT>::T;
  const T* x = static_cast<const T*>(X);
  const int64_t padded = (rows + 127) / 128 * 128;
  // 16-byte loads need every row to start on 16 bytes
  if (aligned16(X) && (ldx * (int64_t)sizeof(T)) % 16 == 0)
    k_mx4_encode<DT><<<grid_of(batch, padded, K, kWarps * kRows), kThreads, 0, st>>>(
        x, batch, rows, padded, K, ldx, codes, scales, release);
  else
    k_mx4_encode_any<DT><<<grid_of(batch, padded, K, kWarps * 2), kThreads, 0, st>>>(
        x, batch, rows, padded, K, ldx, codes, scales, release);
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
  using namespace mx4;
  const dim3 grid = grid_of(batch, rows, K, kWarps * kRows);
  if (K % 8 == 0)
    k_mx4_decode<true><<<grid, kThreads, 0, st>>>(codes, scales, batch, rows, K, out);
  else
    k_mx4_decode<false><<<grid, kThreads, 0, st>>>(codes, scales, batch, rows, K, out);
  return cudaGetLastError();
}

}  // namespace e8
