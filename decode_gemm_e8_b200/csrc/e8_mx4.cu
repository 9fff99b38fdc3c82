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
// scales pairs.  Rows that do not start on 16 bytes still move in aligned 16-byte words,
// which neighbouring lanes share by shuffles and a funnel shift.
#include <type_traits>

#include "e8_internal.h"
#include "e8_mx4.cuh"

namespace e8 {
namespace mx4 {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 4;   // rows a warp has in flight at once

// Rows that start anywhere.  Lane l reads the 16-byte words (2 of them in fp32) that
// hold its first value; what is missing at their end it gets from lane l + 1, lane 31
// from memory.  A word that is not wholly inside the row is read value by value.
template <int DT>
struct Shifted {
  static constexpr int kPer = DT == 2 ? 4 : 8;     // values a word
  static constexpr int kWords = DT == 2 ? 2 : 1;
  uint32_t w[4 * kWords], next[4];
  int shift;   // values between the word's start and the lane's first value: one for a row

  static __device__ __forceinline__ void word(const typename Elem<DT>::T* __restrict__ row,
                                              int64_t c, int64_t K, uint32_t* to) {
    if (c >= 0 && c + kPer <= K) {
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(row + c));
      to[0] = a.x; to[1] = a.y; to[2] = a.z; to[3] = a.w;
    } else {
      to[0] = to[1] = to[2] = to[3] = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (c + i >= 0 && c + i < K) {
          if constexpr (DT == 2) to[i] = __float_as_uint(row[c + i]);
          else to[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
        }
    }
  }
  __device__ __forceinline__ void load(const typename Elem<DT>::T* __restrict__ row, int64_t c,
                                       int64_t K) {
    shift = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(*row));
#pragma unroll
    for (int i = 0; i < kWords; ++i) word(row, c - shift + i * kPer, K, w + 4 * i);
    next[0] = next[1] = next[2] = next[3] = 0;
    if ((threadIdx.x & 31) == 31) word(row, c - shift + kWords * kPer, K, next);
  }
  __device__ __forceinline__ void zero() {
    shift = 0;
#pragma unroll
    for (uint32_t& v : w) v = 0;
    next[0] = next[1] = next[2] = next[3] = 0;
  }
  __device__ __forceinline__ Eight<DT> get() const {
    constexpr int n = 4 * kWords;
    uint32_t t[n + 4];
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = __shfl_down_sync(0xFFFFFFFFu, w[i], 1);
      t[n + i] = (threadIdx.x & 31) == 31 ? next[i] : v;
    }
    // by 4-byte words first, then by half a word
    const int words = DT == 2 ? shift : shift >> 1;
    if (words & 2) {
#pragma unroll
      for (int i = 0; i < n + 2; ++i) t[i] = t[i + 2];
    }
    if (words & 1) {
#pragma unroll
      for (int i = 0; i < n + 1; ++i) t[i] = t[i + 1];
    }
    Eight<DT> e;
#pragma unroll
    for (int i = 0; i < n; ++i)
      e.w[i] = DT == 2 ? t[i] : __funnelshift_r(t[i], t[i + 1], 16 * (shift & 1));
    return e;
  }
};

// Grid: x 256-column chunks, y blocks of 8 x R rows, z matrices.  Rows run to the
// next multiple of 128 so that the padding rows' scales are written as zero.
// WIDE: every row starts on 16 bytes.
template <int DT, bool WIDE, int R>
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
    for (int64_t row0 = ((int64_t)blockIdx.y * kWarps + warp) * R; row0 < rows_padded;
         row0 += (int64_t)gridDim.y * kWarps * R) {
      std::conditional_t<WIDE, Eight<DT>, Shifted<DT>> in[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (row0 + r < rows) in[r].load(x + (row0 + r) * ldx, c, K);
        else in[r].zero();
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t row = row0 + r;
        Eight<DT> v;
        if constexpr (WIDE) v = in[r];
        else v = in[r].get();
        const uint32_t byte = scale_byte(v.block_max());
        const uint32_t code = byte == 255u ? 0u : v.codes(inv_scale(byte));
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
          // The aligned 16-byte word that holds the lane's first value: its start comes
          // from the lane before.  Words that are not wholly this warp's are stored
          // value by value, and lane 31 stores the values after its word.
          uint16_t* first = to + row * K + c;
          const int shift = (int)((reinterpret_cast<uintptr_t>(first) & 15) / 2);
          uint32_t t[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            t[i] = __shfl_up_sync(0xFFFFFFFFu, v[i], 1);
            t[4 + i] = v[i];
          }
          // values 8 - shift .. of the eight pairs-of-values words, shift may be 0
          const int skip = 8 - shift;
          uint32_t o[4];
          {
            uint32_t u[9];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = t[i];
            u[8] = 0;
            if (skip & 8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) u[i] = u[i + 4];
            } else {
              if (skip & 4) {
#pragma unroll
                for (int i = 0; i < 6; ++i) u[i] = u[i + 2];
              }
              if (skip & 2) {
#pragma unroll
                for (int i = 0; i < 5; ++i) u[i] = u[i + 1];
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(u[i], u[i + 1], 16 * (skip & 1));
          }
          if (lane > 0 && c - shift + 8 <= K) {
            __stcs(reinterpret_cast<uint4*>(first - shift), make_uint4(o[0], o[1], o[2], o[3]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t at = c - shift + i;
              if (at >= (lane > 0 ? 0 : c) && at < K)
                first[i - shift] = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
            }
          }
          if (lane == 31) {
#pragma unroll
            for (int i = 1; i < 8; ++i)
              if (i >= skip && c + i < K) first[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
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

template <int DT, bool WIDE, int R>
static cudaError_t encode_as(const void* X, int64_t batch, int64_t rows, int64_t K, int64_t ldx,
                             uint8_t* codes, uint8_t* scales, int release, cudaStream_t st) {
  const int64_t padded = (rows + 127) / 128 * 128;
  k_mx4_encode<DT, WIDE, R><<<grid_of(batch, padded, K, kWarps * R), kThreads, 0, st>>>(
      static_cast<const typename Elem<DT>::T*>(X), batch, rows, padded, K, ldx, codes, scales,
      release);
  return cudaGetLastError();
}

}  // namespace mx4

cudaError_t launch_mx4_encode(const void* X, int dtype, int64_t batch, int64_t rows, int64_t K,
                              int64_t ldx, uint8_t* codes, uint8_t* scales, int release,
                              cudaStream_t st) {
  using namespace mx4;
  const auto go = [&](auto f) { return f(X, batch, rows, K, ldx, codes, scales, release, st); };
  const bool wide = aligned16(X) && (batch * rows == 1 || ldx * (dtype == 2 ? 4 : 2) % 16 == 0);
  if (dtype == 0) return wide ? go(encode_as<0, true, kRows>) : go(encode_as<0, false, kRows>);
  if (dtype == 1) return wide ? go(encode_as<1, true, kRows>) : go(encode_as<1, false, kRows>);
  return wide ? go(encode_as<2, true, kRows>) : go(encode_as<2, false, 2>);
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
