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
// which neighbouring lanes share by shuffles and a funnel shift.  14336 x 4096: encoded
// in 42 us from fp32 (6.4 TB/s) and 27 us from bf16 (5.5), decoded in 28 us (5.3); 1021 x
// 4099 fp16 6.2 and 5.8 us, 1021 x 4096 3.8 and 3.6: there instructions bound it, 180
// of a warp for 256 values instead of 80 to 95.
#include <type_traits>

#include "e8_internal.h"
#include "e8_mx4.cuh"

namespace e8 {
namespace mx4 {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// What a warp's R rows of 256 columns touch: kFull, the matrix alone, and with rows that
// start anywhere a word more on either side, of other rows; kTail, its right end too, past
// which nothing is kept; kEnds, rows so near to an end of the matrix that words around them
// may lie outside of it.
enum : int { kFull = 0, kTail = 1, kEnds = 2 };

// Rows that start anywhere.  Lane l reads the 16-byte words (2 of them in fp32) that
// hold its first value; what is missing at their end it gets from lane l + 1, lane 31
// from memory.  What lies before the row is shifted out, what lies behind it cleared (get).
template <int DT>
struct Shifted {
  using T = typename Elem<DT>::T;
  static constexpr int kPer = DT == 2 ? 4 : 8;     // values a word
  static constexpr int kWords = DT == 2 ? 2 : 1;
  uint32_t w[4 * kWords], next[4];
  int shift;   // values between the word's start and the lane's first value: one for a row

  // (loads under a predicate: in a branch each would be waited for before the next)
  template <int MODE>
  static __device__ __forceinline__ void word(const T* __restrict__ row, int64_t c, int64_t K,
                                              bool on, uint32_t* to) {
    if constexpr (MODE != kEnds) {
      const uint32_t in = on && (MODE == kFull || c < K);
      asm volatile(
          "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
          "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
          "@p ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}\n"
          : "=&r"(to[0]), "=&r"(to[1]), "=&r"(to[2]), "=&r"(to[3])
          : "l"(row + c), "r"(in));
    } else {
      to[0] = to[1] = to[2] = to[3] = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (on && c + i >= 0 && c + i < K) {
          if constexpr (DT == 2) to[i] = __float_as_uint(row[c + i]);
          else to[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
        }
    }
  }
  template <int MODE>
  __device__ __forceinline__ void load(const T* __restrict__ row, int64_t c, int64_t K) {
    shift = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
#pragma unroll
    for (int i = 0; i < kWords; ++i) word<MODE>(row, c - shift + i * kPer, K, true, w + 4 * i);
    word<MODE>(row, c - shift + kWords * kPer, K, (threadIdx.x & 31) == 31, next);
  }
  __device__ __forceinline__ void zero() {
    shift = 0;
#pragma unroll
    for (uint32_t& v : w) v = 0;
    next[0] = next[1] = next[2] = next[3] = 0;
  }
  // `left`: values of the row from the lane's first on, if fewer than 8
  template <int MODE>
  __device__ __forceinline__ Eight<DT> get(int left) const {
    constexpr int n = 4 * kWords;
    uint32_t t[n + 4];
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = __shfl_down_sync(0xFFFFFFFFu, w[i], 1);
      t[n + i] = (threadIdx.x & 31) == 31 ? next[i] : v;
    }
    // (one shift for a row: a branch costs less than choosing word by word)
    Eight<DT> e;
    const auto from = [&](auto words) {
#pragma unroll
      for (int i = 0; i < n; ++i)
        e.w[i] = DT == 2 ? t[i + words]
                         : __funnelshift_r(t[i + words], t[i + words + 1], 16 * (shift & 1));
    };
    switch (DT == 2 ? shift : shift >> 1) {
      case 0: from(std::integral_constant<int, 0>()); break;
      case 1: from(std::integral_constant<int, 1>()); break;
      case 2: from(std::integral_constant<int, 2>()); break;
      default: from(std::integral_constant<int, 3>());
    }
    if constexpr (MODE != kFull) {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        if constexpr (DT == 2) e.w[i] = i < left ? e.w[i] : 0u;
        else e.w[i] = 2 * i + 1 < left ? e.w[i] : 2 * i < left ? e.w[i] & 0xFFFFu : 0u;
      }
    }
    return e;
  }
};

// R rows of 256 columns, c the lane's first; x, to and sc point at the first row, `to` and
// `sc` at the lane's column; `rows` are left in the matrix.
template <int DT, bool WIDE, int R, int MODE>
__device__ __forceinline__ void encode_rows(const typename Elem<DT>::T* __restrict__ x,
                                            int64_t ldx, int64_t c, int64_t K, int64_t rows,
                                            uint8_t* __restrict__ to, int64_t cs,
                                            uint8_t* __restrict__ sc, int64_t kqs) {
  std::conditional_t<WIDE, Eight<DT>, Shifted<DT>> in[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (MODE == kFull || r < rows) {
      if constexpr (!WIDE) in[r].template load<MODE>(x, c, K);
      else if constexpr (MODE == kFull) in[r].load(x + c);
      else in[r].load(x, c, K);
    } else {
      in[r].zero();
    }
    x += ldx;
  }
  const int left = K - c < 8 ? (int)(K - c) : 8;
  const bool code_lane = MODE == kFull || c / 2 < cs;
  const bool scale_lane = (threadIdx.x & 3) == 0 && (MODE == kFull || c / 128 < kqs);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    Eight<DT> v;
    if constexpr (WIDE) v = in[r];
    else v = in[r].template get<MODE>(left);
    const uint32_t byte = v.block_byte(), code = v.codes(byte);
    if (code_lane && (MODE == kFull || r < rows)) *reinterpret_cast<uint32_t*>(to) = code;
    to += cs;
    // (blocks past the matrix hold zeros, whose byte is 0)
    if (scale_lane) sc[16 * r] = (uint8_t)byte;
  }
}

// Grid: x 256-column chunks, y blocks of 8 x R rows, z matrices.  Rows run to the
// next multiple of 128 so that the padding rows' scales are written as zero.
// WIDE: every row starts on 16 bytes.  With checks that are made once for R rows and
// pointers that step from row to row a 256-column row of bf16 takes 81 of a warp's
// instructions; with a check and 64-bit products for each it took 158, and the kernel
// was bound by issuing them (14336 x 4096 bf16: 45 us, now 27).
template <int DT, bool WIDE, int R>
__global__ void __launch_bounds__(kThreads, 4)
    k_mx4_encode(const typename Elem<DT>::T* __restrict__ X, int64_t batch, int64_t rows,
                 int64_t rows_padded, int64_t K, int64_t ldx, uint8_t* __restrict__ codes,
                 uint8_t* __restrict__ scales) {
  static_assert(32 % R == 0, "R rows are in one group of 32");
  grid_dep_wait();   // before anything is read or written: launch_after
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cs = code_stride(K), kqs = scale_tiles(K);
  const int64_t c0 = (int64_t)blockIdx.x * 256, c = c0 + lane * 8;
  const bool full = c0 + (WIDE ? 256 : 264) <= K;
  for (int64_t b = blockIdx.z; b < batch; b += gridDim.z) {
    for (int64_t row0 = ((int64_t)blockIdx.y * kWarps + warp) * R; row0 < rows_padded;
         row0 += (int64_t)gridDim.y * kWarps * R) {
      const typename Elem<DT>::T* x = X + (b * rows + row0) * ldx;
      uint8_t* to = codes + (b * rows + row0) * cs + c / 2;
      uint8_t* sc = scales + b * rows_padded / 128 * kqs * 512 + scale_at(row0, c >> 7, kqs) +
                    ((lane >> 2) & 3);
      // eight rows on are eight values on, at least: a word
      const int64_t before = b * rows + row0, behind = (batch - b) * rows - row0 - R;
      if (!WIDE && ((c0 == 0 && before < 8) || behind < 8))
        encode_rows<DT, WIDE, R, WIDE ? kTail : kEnds>(x, ldx, c, K, rows - row0, to, cs, sc, kqs);
      else if (full && row0 + R <= rows)
        encode_rows<DT, WIDE, R, kFull>(x, ldx, c, K, rows - row0, to, cs, sc, kqs);
      else
        encode_rows<DT, WIDE, R, kTail>(x, ldx, c, K, rows - row0, to, cs, sc, kqs);
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

// A lane's eight values (one word of codes) as four bf16 pairs.
__device__ __forceinline__ void decode8(uint32_t code, uint32_t byte, uint32_t (&v)[4]) {
  codes_to_bf16(code, v[0], v[1]);
  codes_to_bf16(code >> 16, v[2], v[3]);
  const uint32_t s = scale_bf16x2(byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul_bf16x2(v[i], s);
}

// Grid as the encoder's, rows to the last one only.  VEC: every row of `out` starts on
// 16 bytes.  Else lane l stores the aligned word that holds the first of its own values,
// whose start it gets from lane l - 1; lane 0 has no other task, so a chunk is 248
// columns.  Words that are not wholly inside the row are stored value by value.
template <bool VEC>
constexpr int kDecodeColumns = VEC ? 256 : 248;
template <bool VEC>
constexpr int kDecodeRows = VEC ? 8 : 4;   // a warp has in flight at once
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 4)
    k_mx4_decode(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                 int64_t batch, int64_t rows, int64_t K, uint16_t* __restrict__ out) {
  constexpr int kRows = kDecodeRows<VEC>;
  static_assert(32 % kRows == 0, "the rows are in one group of 32");
  grid_dep_wait();   // (values are tokens to other calls: launch_after)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cs = code_stride(K), kqs = scale_tiles(K), sb = scale_bytes(rows, K);
  const int64_t c = (int64_t)blockIdx.x * kDecodeColumns<VEC> + (VEC ? lane : lane - 1) * 8;
  const bool in = c >= 0 && c / 2 < cs;
  const int left = K - c < 16 ? (int)(K - c) : 16;   // values from the lane's first on
  for (int64_t b = blockIdx.z; b < batch; b += gridDim.z) {
    for (int64_t row0 = ((int64_t)blockIdx.y * kWarps + warp) * kRows; row0 < rows;
         row0 += (int64_t)gridDim.y * kWarps * kRows) {
      const uint8_t* from = codes + (b * rows + row0) * cs + c / 2;
      const uint8_t* sc = scales + b * sb + scale_at(row0, c >> 7, kqs) + ((c >> 5) & 3);
      uint16_t* to = out + (b * rows + row0) * K + c;
      const int n = rows - row0 < kRows ? (int)(rows - row0) : kRows;
      uint32_t code[kRows], byte[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const bool ok = in && r < n;
        code[r] = ok ? __ldcs(reinterpret_cast<const uint32_t*>(from)) : 0u;
        byte[r] = ok ? sc[16 * r] : 0u;
        from += cs;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r == n) break;
        uint32_t v[4];
        decode8(code[r], byte[r], v);
        if constexpr (VEC) {
          // K is a multiple of 8 here
          if (c < K) __stcs(reinterpret_cast<uint4*>(to), make_uint4(v[0], v[1], v[2], v[3]));
        } else {
          // values `skip` .. `skip` + 7 of the lane before and this one
          const int shift = (int)((reinterpret_cast<uintptr_t>(to) & 15) / 2), skip = 8 - shift;
          uint32_t t[9];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            t[i] = __shfl_up_sync(0xFFFFFFFFu, v[i], 1);
            t[4 + i] = v[i];
          }
          t[8] = 0;
          uint32_t o[4];
          const auto from = [&](auto words) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = __funnelshift_r(t[i + words], t[i + words + 1], 16 * (skip & 1));
          };
          switch (skip >> 1) {
            case 0: from(std::integral_constant<int, 0>()); break;
            case 1: from(std::integral_constant<int, 1>()); break;
            case 2: from(std::integral_constant<int, 2>()); break;
            case 3: from(std::integral_constant<int, 3>()); break;
            default: from(std::integral_constant<int, 4>());
          }
          // the word's values lo .. hi - 1 are the row's
          const int lo = c == 0 ? shift : 0, hi = left + shift < 8 ? left + shift : 8;
          if (lane > 0) {
            if (lo == 0 && hi == 8) {
              __stcs(reinterpret_cast<uint4*>(to - shift), make_uint4(o[0], o[1], o[2], o[3]));
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i >= lo && i < hi) to[i - shift] = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
            }
          }
        }
        to += K;
      }
    }
  }
}

// Row blocks and matrices beyond the grid's limits are walked in the kernels' loops.
static dim3 grid_of(int64_t batch, int64_t rows, int64_t chunks, int rows_a_block) {
  const int64_t y = (rows + rows_a_block - 1) / rows_a_block;
  return dim3((unsigned)chunks, (unsigned)(y < 65535 ? y : 65535),
              (unsigned)(batch < 65535 ? batch : 65535));
}

template <int DT, bool WIDE, int R>
static cudaError_t encode_as(const void* X, int64_t batch, int64_t rows, int64_t K, int64_t ldx,
                             uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const int64_t padded = (rows + 127) / 128 * 128;
  return launch_after(k_mx4_encode<DT, WIDE, R>,
                      grid_of(batch, padded, (K + 255) / 256, kWarps * R), dim3(kThreads), 0, st,
                      static_cast<const typename Elem<DT>::T*>(X), batch, rows, padded, K, ldx,
                      codes, scales);
}

}  // namespace mx4

cudaError_t launch_mx4_encode(const void* X, int dtype, int64_t batch, int64_t rows, int64_t K,
                              int64_t ldx, uint8_t* codes, uint8_t* scales, int sm_count,
                              cudaStream_t st) {
  using namespace mx4;
  const auto go = [&](auto f) { return f(X, batch, rows, K, ldx, codes, scales, st); };
  const bool wide = aligned16(X) && (batch * rows == 1 || ldx * (dtype == 2 ? 4 : 2) % 16 == 0);
  // Rows in flight, 16-bit types: 8 where that still fills the SMs (14336 x 4096 bf16: 27.9
  // us, with 4 rows 32.1; 1021 x 4096 5.0 and 4.4); with words of a neighbour to hold half
  // as many (14336 x 4099 bf16 44 us, with 2 rows 54).  In fp32 4 and 2, all that fit the
  // registers.
  const bool many = (K + 255) / 256 * ((rows + 63) / 64) * batch >= 4 * sm_count;
  if (dtype == 0)
    return many ? (wide ? go(encode_as<0, true, 8>) : go(encode_as<0, false, 4>))
                : (wide ? go(encode_as<0, true, 4>) : go(encode_as<0, false, 2>));
  if (dtype == 1)
    return many ? (wide ? go(encode_as<1, true, 8>) : go(encode_as<1, false, 4>))
                : (wide ? go(encode_as<1, true, 4>) : go(encode_as<1, false, 2>));
  return wide ? go(encode_as<2, true, 4>) : go(encode_as<2, false, 2>);
}

cudaError_t launch_mx4_decode(const uint8_t* codes, const uint8_t* scales, int64_t batch,
                              int64_t rows, int64_t K, uint16_t* out, cudaStream_t st) {
  using namespace mx4;
  if (K % 8 == 0)
    return launch_after(k_mx4_decode<true>,
                        grid_of(batch, rows, (K + 255) / 256, kWarps * kDecodeRows<true>),
                        dim3(kThreads), 0, st, codes, scales, batch, rows, K, out);
  // up to 7 columns of the words before a row's first value
  return launch_after(k_mx4_decode<false>,
                      grid_of(batch, rows, (K + 7 + 247) / 248, kWarps * kDecodeRows<false>),
                      dim3(kThreads), 0, st, codes, scales, batch, rows, K, out);
}

}  // namespace e8
