// Microscaled 4-bit form (blocks of 32 e2m1 values, one power-of-two scale):
// layout rules and number helpers shared by its kernels.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "e8_common.cuh"

namespace e8 {
namespace mx4 {

// Launches a kernel that may start while the one before it in the stream ends, if that one
// lets it (grid_dep_launch); it waits for it (grid_dep_wait) before it reads or writes.
// The rule of the library on who may let the next kernel start:
//   - only a kernel that writes nothing a call takes as X, idx1 or idx2: the int8
//     transform of e8_gemm (k_act_q8) and the product behind it read those before their
//     own waits, so the kernel that wrote them must be over when they start;
//   - and only behind its own wait, if the next one reads weights ahead of its wait: what
//     came before this kernel is then over (the encoder in front of a product).
// Of the microscaled kernels the encoder does (it writes codes and scales, which nothing
// reads ahead); products and the decoder write bf16, which is X to e8_gemm, and do not.
// (Products of 1 x 4096 x 4096 in a row take 6.9 us each, and 5.7 if they did; one behind
// an encoder still starts while that one ends.)
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Tiles of `size` in n >= 1 (n may be 2^31 - 1: no sum of the two).
__host__ __device__ __forceinline__ constexpr int tiles_of(int n, int size) {
  return (n - 1) / size + 1;
}
// Bytes of one row of codes: 16 for each block of 32.
__host__ __device__ __forceinline__ int64_t code_stride(int64_t K) { return (K + 31) / 32 * 16; }
// Tiles of 128 columns in a row of scale tiles.
__host__ __device__ __forceinline__ int64_t scale_tiles(int64_t K) { return (K + 127) / 128; }
__host__ __device__ __forceinline__ int64_t scale_bytes(int64_t rows, int64_t K) {
  return (rows + 127) / 128 * scale_tiles(K) * 512;
}
// Byte offset of the four scales of row `row` in column tile `kq`.
__host__ __device__ __forceinline__ int64_t scale_at(int64_t row, int64_t kq, int64_t kqs) {
  return ((row >> 7) * kqs + kq) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Scale byte of a block whose largest magnitude is `amax` (>= 0, maybe inf or
// NaN): the exponent field less 2, clamped at 0; 255 when amax is not finite.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t e = __float_as_uint(amax) >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^-(byte - 127), a normal number for every byte the encoder computes (<= 252).
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127): subnormal for byte 0, NaN for byte 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u)
                    : (byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23));
}

// Eight floats -> eight e2m1 codes (element 0 in the low nibble), nearest even,
// saturating.
__device__ __forceinline__ uint32_t pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// ------------------------------------------------------------ encoding ---
// DT: E8_DT_* (0 bf16, 1 fp16, 2 fp32).
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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight values of a row from column c on (zeros past K), as they lie in memory; one
// lane's share of a block, four lanes a block.
template <int DT>
struct Eight {
  using T = typename Elem<DT>::T;
  uint32_t w[DT == 2 ? 8 : 4];
  // all eight there, on 16 bytes
  __device__ __forceinline__ void load(const T* __restrict__ at) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(at));
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    if constexpr (DT == 2) {
      const uint4 b = __ldcs(reinterpret_cast<const uint4*>(at + 4));
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
  }
  // wide: the row starts on 16 bytes
  __device__ __forceinline__ void load(const T* __restrict__ row, int64_t c, int64_t K,
                                       bool wide = true) {
    if (wide && c + 8 <= K) {
      load(row + c);
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
  // The block's scale byte, over its four lanes: magnitudes compare as integers, and a
  // NaN or an infinity wins.
  __device__ __forceinline__ uint32_t block_byte() const {
    uint32_t m = 0;
    if constexpr (DT == 2) {
#pragma unroll
      for (uint32_t v : w) m = max(m, v & 0x7FFFFFFFu);
    } else {
#pragma unroll
      for (uint32_t v : w) m = max_u16x2(m, v & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
    }
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return scale_byte(DT == 2 ? __uint_as_float(m) : to_float<DT == 2 ? 0 : DT>((uint16_t)m));
  }
  // The codes under a scale byte (zeros under 255).  bf16 values are scaled as pairs in
  // bf16: exactly, but for results below 2^-126, which are code 0 either way.
  __device__ __forceinline__ uint32_t codes(uint32_t byte) const {
    float v[8];
    if constexpr (DT == 0) {
      const uint32_t inv = (254u - byte) * 0x00800080u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t p = mul_bf16x2(w[i], inv);
        v[2 * i] = bf16_lo_to_f32(p);
        v[2 * i + 1] = bf16_hi_to_f32(p);
      }
    } else {
      const float inv = inv_scale(byte);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = (DT == 2 ? __uint_as_float(w[i % (DT == 2 ? 8 : 4)])
                        : to_float<1>((uint16_t)(w[i / 2] >> (16 * (i & 1))))) * inv;
    }
    const uint32_t c = pack8(v);
    return byte == 255u ? 0u : c;
  }
};

// ------------------------------------------------------- tensor cores ---
// Their callers run in a branch that elect.sync chose the thread of: under any other
// condition the compiler has to serve several threads, at some 40 cycles an
// instruction (measured; 9 a scale copy and the tensor cores' own time an MMA here).
// Instruction descriptor of tcgen05.mma.kind::mxf4: e2m1 A and B (both K-major),
// ue8m0 scales, fp32 accumulator, K = 64.  sf: which pair of the four scale
// bytes of a 32-bit tensor-memory column this step takes (0 or 2), for A and B.
__host__ __device__ constexpr uint32_t idesc_mxf4(uint32_t M, uint32_t N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 7) << 27) |
         (sf << 29);
}

// D[tmem] (+)= (A[smem] scaled) * (B[smem] scaled)^T, scales in tensor memory.
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;"
      "\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// The same for kind::mxf8f6f4 with e2m1 A (each 16 values in 16 bytes of shared
// memory, packed in the first 8) and e4m3 B, K = 32; sf: the byte of the scale
// columns this step takes (0..3).
__host__ __device__ constexpr uint32_t idesc_mxf4_f8(uint32_t M, uint32_t N, uint32_t sf) {
  return (sf << 4) | (5u << 7) | (0u << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 7) << 27) |
         (sf << 29);
}
__device__ __forceinline__ void mma_mxf8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Matrix descriptors from their low word, so that the issuing thread's loop adds
// to one register.  Codes: K-major rows of 128 bytes with the 128-byte swizzle;
// scales: 8 rows of 16 bytes after one another.
__device__ __forceinline__ uint32_t code_desc_lo(uint32_t smem) { return (smem >> 4) | (1u << 16); }
__device__ __forceinline__ uint64_t code_desc(uint32_t lo) {
  return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lo;
}
__device__ __forceinline__ uint32_t scale_desc_lo(uint32_t smem) {
  return (smem >> 4) | ((128u >> 4) << 16);
}
// One 512-byte scale tile (32 lanes of 16 bytes) into four columns of tensor
// memory, repeated in all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t desc_lo) {
  asm volatile(
      "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"((uint64_t)((128u >> 4) | (1u << 14)) << 32 | desc_lo)
               : "memory");
}

// The same two for a pair of CTAs (cta_group::2): M = 256, each CTA holds 128 rows of
// A, half the rows of B and all scales its tensor memory needs.
__device__ __forceinline__ void mma_mxf4_2sm(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;"
      "\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void copy_scales_2sm(uint32_t taddr, uint32_t desc_lo) {
  asm volatile(
      "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"((uint64_t)((128u >> 4) | (1u << 14)) << 32 | desc_lo)
               : "memory");
}

}  // namespace mx4
}  // namespace e8
