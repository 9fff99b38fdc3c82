// Product of two matrices in the microscaled 4-bit form, on the tensor cores'
// own block-scaled 4-bit path (tcgen05.mma.kind::mxf4): codes and scales go from
// HBM to the tensor cores as they are stored, nothing is decoded.
//
// Y[m][n] = bf16(sum_k A[m][k] W[n][k]).  A product of two e2m1 values and two
// powers of two is exact in fp32; the accumulator is fp32; the one rounding to
// fewer bits is that of Y.
#include "e8_internal.h"
#include "e8_mx4.cuh"
#include "e8_tmap.h"

namespace e8 {
namespace mx4 {

// ------------------------------------------------------------ few tokens ---
// Swapped operands: 128 rows of W are the MMA's M side, bn tokens its N side, so
// that a single token costs one narrow MMA and the weights are read once.  The
// K range is split over a cluster of `splits` CTAs when there are fewer row tiles
// than SMs; every CTA leaves its partial tile in its own shared memory and each
// then adds up, in rank order, the columns it was given (distributed shared
// memory), so results do not depend on timing.
//   warps 0, 6 TMA producers of W (128 x 256 K, 16 KB) and of the tokens: codes
//              with the 128-byte swizzle, scale tiles by plain bulk copies.  One
//              thread each: at 16 KB a stage the SM's share of HBM leaves an issuing
//              thread some 350 cycles a stage
//   warp 1     tensor-memory allocation; one thread copies the stage's scales to
//              tensor memory (a slot of its own for each stage, so that no copy
//              meets an MMA that still reads) and issues the MMAs
//   warps 2-5  epilogue
//   warps 2-9  with up to 8 tokens that are not encoded yet (DT >= 0), instead of warp
//              6: each encodes the tokens of one of the 8 ring slots, every CTA for
//              itself.  With / without the encoder's launch, in us a call in a row of
//              them at N x K = 4096 x 4096 and 14336 x 4096: 1 token 7.2 / 6.4 and 11.0 /
//              10.0, 8 tokens 7.4 / 7.2 and 11.1 / 10.3; 16 tokens 7.6 / 8.9 and 11.2 / 13.1
// Bound by HBM on W once it runs (16 x 14336 x 4096 11.1 us, 4.9 of them its bytes), the
// rest is its start (5 us: launch, barriers, tensor memory, first tile) and its end.
constexpr int kStreamThreads = 224, kStreamThreadsX = 320;
constexpr int kStreamRows = 128;
constexpr int kBK = 256;               // K of a stage: 128 bytes of codes
constexpr int kCodeTile = 128 * 128;   // bytes of 128 rows
constexpr int kMaxStages = 8;
constexpr int kSfCol = 256;            // first tensor-memory column of the scales
constexpr int kStreamSmem = 225 * 1024;

struct StreamArgs {
  const uint8_t *w_scales, *a_scales;
  uint16_t* Y;
  int M, N, K;
  int bn, stages, splits;
  int early;   // the weights may be read before the preceding kernel has ended
  const void* X;   // tokens to encode, row stride ldx; wide: its rows start on 16 bytes
  int64_t ldx;
  int wide;
  uint32_t* status;
};

__host__ __device__ __forceinline__ int stream_stage_bytes(int bn) {
  return kCodeTile + bn * 128 + 1024 + 1024 * ((bn + 127) / 128);
}

template <int DT>
__global__ void __launch_bounds__(DT < 0 ? kStreamThreads : kStreamThreadsX, 1)
    k_mx4_stream(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                 const __grid_constant__ StreamArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.splits, rank = (int)blockIdx.x % S;
  const int n0 = (int)blockIdx.x / S * kStreamRows, m0 = (int)blockIdx.y * a.bn;
  const int nbt = (a.bn + 127) / 128;
  const int stage_bytes = stream_stage_bytes(a.bn);
  const int kblocks = tiles_of(a.K, kBK), kqs = (int)scale_tiles(a.K);
  const int kb0 = (int)((int64_t)kblocks * rank / S);
  const int nkb = (int)((int64_t)kblocks * (rank + 1) / S) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 2);   // W's producer and the tokens'
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    if (DT < 0) tma_prefetch_desc(&tmA);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (!a.early) grid_dep_wait();

  const uint32_t ring = smem_u32(smem);
  if (warp == 0) {
    if (elect_one()) {
      // codes and scales of W
      const uint8_t* sf = a.w_scales + ((int64_t)(n0 >> 7) * kqs + 2 * kb0) * 512;
      uint32_t st = ring, ph = 1;
      int s = 0;
      for (int i = 0; i < nkb; ++i) {
        if (!mbar_wait_lazy(&empty[s], ph, &abort_flag, a.status, kDevTimeoutEmpty)) break;
        // both 128-column scale tiles of the stage, or the last one alone
        const uint32_t sb = 2 * (kb0 + i) + 1 < kqs ? 1024u : 512u;
        mbar_arrive_expect_tx(&full[s], (uint32_t)kCodeTile + sb);
        load_2d(st, &tmW, &full[s], (kb0 + i) * 128, n0);
        load_bulk(st + kCodeTile + (uint32_t)a.bn * 128u, sf, sb, &full[s]);
        sf += 1024;
        st += (uint32_t)stage_bytes;
        if (++s == a.stages) {
          s = 0;
          ph ^= 1u;
          st = ring;
        }
      }
    }
  } else if (DT >= 0 && warp >= 2) {
    if constexpr (DT >= 0) {
      // the tokens of slot warp - 2, all rows' loads in flight before the first is encoded
      const typename Elem<DT>::T* x = static_cast<const typename Elem<DT>::T*>(a.X);
      const int e = warp - 2;
      const uint32_t st = ring + (uint32_t)(e * stage_bytes) + kCodeTile;
      uint32_t ph = 1;
      for (int i = e; i < nkb; i += kMaxStages) {
        const int64_t c = (int64_t)(kb0 + i) * kBK + lane * 8;
        Eight<DT> v[kMx4Small];
#pragma unroll
        for (int r = 0; r < kMx4Small; ++r) {
          if (r < a.M) v[r].load(x + r * a.ldx, c, a.K, a.wide != 0);
          else v[r].zero();
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_lazy(&empty[e], ph, &abort_flag, a.status,
                                                    kDevTimeoutEmpty)))
          break;
        ph ^= 1u;
#pragma unroll
        for (int g = 0; g < kMx4Small; g += 4) {
          if (g < a.M) {
#pragma unroll
            for (int r = g; r < g + 4; ++r) {
              const uint32_t byte = v[r].block_byte(), code = v[r].codes(byte);
              uint32_t f = byte | __shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8;
              f |= __shfl_down_sync(0xFFFFFFFFu, f, 8) << 16;
              const uint32_t at = st + (uint32_t)(r * 128 + (((lane >> 2) ^ (r & 7)) << 4)) +
                                  (uint32_t)(lane & 3) * 4u;
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(code) : "memory");
              // the four scales of 128 columns, in lanes 0 and 16
              if ((lane & 15) == 0)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(
                                 st + (uint32_t)a.bn * 128u + 1024u + (uint32_t)(lane >> 4) * 512u +
                                 (uint32_t)r * 16u),
                             "r"(f)
                             : "memory");
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[e]);
      }
    }
  } else if (DT < 0 && warp == 6) {
    if (a.early) grid_dep_wait();
    if (elect_one()) {
      // codes and scales of the tokens
      const int tiles = min(nbt, (a.M - m0 + 127) / 128);
      const uint8_t* sf = a.a_scales + ((int64_t)(m0 >> 7) * kqs + 2 * kb0) * 512;
      uint32_t st = ring + kCodeTile, ph = 1;
      int s = 0;
      for (int i = 0; i < nkb; ++i) {
        if (!mbar_wait_lazy(&empty[s], ph, &abort_flag, a.status, kDevTimeoutEmpty)) break;
        const uint32_t sb = 2 * (kb0 + i) + 1 < kqs ? 1024u : 512u;
        mbar_arrive_expect_tx(&full[s], (uint32_t)a.bn * 128u + sb * (uint32_t)tiles);
        load_2d(st, &tmA, &full[s], (kb0 + i) * 128, m0);
        const uint32_t to = st + (uint32_t)a.bn * 128u + 1024u;
        load_bulk(to, sf, sb, &full[s]);
        if (tiles > 1) load_bulk(to + 1024u, sf + (size_t)kqs * 512, sb, &full[s]);
        sf += 1024;
        st += (uint32_t)stage_bytes;
        if (++s == a.stages) {
          s = 0;
          ph ^= 1u;
          st = ring + kCodeTile;
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc0 = idesc_mxf4(128, (uint32_t)a.bn, 0),
                     idesc1 = idesc_mxf4(128, (uint32_t)a.bn, 2);
      const uint32_t t_off = kCodeTile >> 4, f_off = t_off + (uint32_t)a.bn * 8u;
      const uint32_t sf_cols = 8u + 8u * (uint32_t)nbt, half = 4u * (uint32_t)nbt;
      uint32_t st = ring >> 4, ph = 0, cols = tmem + kSfCol;
      int s = 0, left = a.K - kb0 * kBK;   // columns from here on
      for (int i = 0; i < nkb; ++i) {
        if (!mbar_wait_lazy(&full[s], ph, &abort_flag, a.status, kDevTimeoutFull)) break;
        tc_fence_after();
        const uint32_t w = code_desc_lo(st << 4), t = w + t_off;
        const uint32_t f = scale_desc_lo((st + f_off) << 4), sfb = cols + 8u;
        // 64 columns an MMA; a scale tile serves two
        copy_scales(cols, f);
        copy_scales(sfb, f + 64u);
        if (nbt > 1) copy_scales(sfb + 4u, f + 128u);
        if (left > 128) {
          copy_scales(cols + 4u, f + 32u);
          copy_scales(sfb + half, f + 96u);
          if (nbt > 1) copy_scales(sfb + half + 4u, f + 160u);
        }
        mma_mxf4(tmem, code_desc(w), code_desc(t), idesc0, cols, sfb, i > 0);
        if (left > 64) mma_mxf4(tmem, code_desc(w + 2u), code_desc(t + 2u), idesc1, cols, sfb, 1);
        if (left > 128)
          mma_mxf4(tmem, code_desc(w + 4u), code_desc(t + 4u), idesc0, cols + 4u, sfb + half, 1);
        if (left > 192)
          mma_mxf4(tmem, code_desc(w + 6u), code_desc(t + 6u), idesc1, cols + 4u, sfb + half, 1);
        mma_commit(&empty[s]);
        left -= kBK;
        st += (uint32_t)stage_bytes >> 4;
        cols += sf_cols;
        if (++s == a.stages) {
          s = 0;
          ph ^= 1u;
          st = ring >> 4;
          cols = tmem + kSfCol;
        }
      }
      mma_commit(&done);   // also after a wait that gave up: nothing may be in flight at the end
    }
  }
  __syncwarp();
  // every warp: all MMAs of this CTA have finished
  const bool ok = mbar_wait_lazy(&done, 0, &abort_flag, a.status, kDevTimeoutMma);
  __syncwarp();
  tc_fence_after();
  const int cols = min(a.bn, a.M - m0);
  if (abort_flag) {
    // copies in flight may still land: give them time before the CTA exits
    const uint64_t t0 = global_timer_ns();
    while (ns_since(t0) < 1000000ull) {
    }
  }
  if (S == 1) {
    if (warp >= 2 && warp < 6 && ok) {
      const int quarter = warp & 3, n = n0 + quarter * 32 + lane;
      for (int c = 0; c < cols; c += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + (uint32_t)c + ((uint32_t)(quarter * 32) << 16), r);
        tmem_ld_wait();
        if (n < a.N) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < cols)
              a.Y[(size_t)(m0 + c + j) * a.N + n] =
                  (uint16_t)(pack_bf16x2(__uint_as_float(r[j]), 0.0f) & 0xFFFFu);
        }
      }
    }
  } else {
    float* part = reinterpret_cast<float*>(smem);   // [column][128], the ring is free
    if (warp >= 2 && warp < 6) {
      const int quarter = warp & 3;
      for (int c = 0; c < cols; c += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + (uint32_t)c + ((uint32_t)(quarter * 32) << 16), r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < cols) part[(c + j) * 128 + quarter * 32 + lane] = __uint_as_float(r[j]);
      }
    }
    cluster_arrive();
    cluster_wait();
    // a warp a column, four rows a lane; the loads of two columns in flight
    const int n = n0 + lane * 4, warps = (int)(blockDim.x >> 5);
    const bool four = (a.N & 3) == 0;   // (Y starts on 16 bytes)
#pragma unroll 2
    for (int c = rank + warp * S; c < cols; c += warps * S) {
      const uint32_t at = smem_u32(part + c * 128 + lane * 4);
      float4 v[8];
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p < S) v[p] = ld_shared_cluster_v4(mapa_shared(at, (uint32_t)p));
      float4 y = v[0];
#pragma unroll
      for (int p = 1; p < 8; ++p)
        if (p < S) {
          y.x += v[p].x;
          y.y += v[p].y;
          y.z += v[p].z;
          y.w += v[p].w;
        }
      const uint32_t lo = pack_bf16x2(y.x, y.y), hi = pack_bf16x2(y.z, y.w);
      uint16_t* to = a.Y + (size_t)(m0 + c) * a.N + n;
      if (four) {
        if (n < a.N) *reinterpret_cast<uint2*>(to) = make_uint2(lo, hi);
      } else {
        if (n < a.N) to[0] = (uint16_t)lo;
        if (n + 1 < a.N) to[1] = (uint16_t)(lo >> 16);
        if (n + 2 < a.N) to[2] = (uint16_t)hi;
        if (n + 3 < a.N) to[3] = (uint16_t)(hi >> 16);
      }
    }
    __syncwarp();
    cluster_arrive();   // no CTA leaves while another reads its shared memory
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// DT < 0: encoded tokens a_codes / a_scales; else X.
template <int DT>
static cudaError_t launch_stream(const void* X, int64_t ldx, const uint8_t* a_codes,
                                 const uint8_t* a_scales, int64_t M, const uint8_t* w_codes,
                                 const uint8_t* w_scales, int64_t N, int64_t K, uint16_t* Y,
                                 uint32_t* status, int sm_count, int early, cudaStream_t st) {
  StreamArgs a;
  a.w_scales = w_scales;
  a.a_scales = a_scales;
  a.Y = Y;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  // one token tile up to 256 tokens; more of them start on 256, where scale tiles do
  a.bn = M >= 256 ? 256 : (int)((M + 15) / 16 * 16);
  a.stages = kStreamSmem / stream_stage_bytes(a.bn);
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  // (slot e's tokens are warp 2 + e's)
  static_assert(kMx4Small <= 16 && kStreamSmem / (kCodeTile + 16 * 128 + 2048) >= kMaxStages, "");
  a.early = early;
  a.X = X;
  a.ldx = ldx;
  a.wide = aligned16(X) && (M == 1 || (ldx * (DT == 2 ? 4 : 2)) % 16 == 0);
  a.status = status;
  const int64_t tiles_n = (N + kStreamRows - 1) / kStreamRows, tiles_m = (M + a.bn - 1) / a.bn;
  const int kblocks = (int)((K + kBK - 1) / kBK);
  int S = 1;
  while (S < 8 && 2 * S <= kblocks && tiles_n * tiles_m * 2 * S <= sm_count) S *= 2;
  a.splits = S;
  if (tiles_m > 65535 || tiles_n * S > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t cs = code_stride(K);
  CUtensorMap tw, ta = {};
  if (!encode_tmap_2d(&tw, w_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)N, (uint64_t)cs, 128,
                    128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (DT < 0 && !encode_tmap_2d(&ta, a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)M,
                               (uint64_t)cs, (uint32_t)a.bn, 128, CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_limit(k_mx4_stream<DT>, kMaxDynSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles_n * S), (unsigned)tiles_m);
  cfg.blockDim = dim3(DT < 0 ? kStreamThreads : kStreamThreadsX);
  cfg.dynamicSmemBytes = 1024 + (size_t)a.stages * stream_stage_bytes(a.bn);
  // room for the partial tile of a split product
  const size_t part = 1024 + (size_t)a.bn * 512;
  if (S > 1 && cfg.dynamicSmemBytes < part) cfg.dynamicSmemBytes = part;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, k_mx4_stream<DT>, tw, ta, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ----------------------------------------------------------- many tokens ---
// Two CTAs compute a 256 x 192 tile (cta_group::2), each holding 128 rows of A and 96
// of W.
//   Why 192 columns: reading an fp32 accumulator of 128 x 256 out of tensor memory
//   takes an SM about 2000 cycles, a fifth of the 16 stages of K = 4096, so it has to
//   overlap the next tile's MMAs; two accumulators of 192 columns (384) and the scales
//   of five stages (120) fit the 512 columns, two of 256 do not.
//   Every copy reads global memory into its own CTA: no TMA multicast, as in the
//   library's other kernels, which also serve runs on several GPUs.
//   An SM's 31 KB a stage come from L2 (about 43 bytes a cycle, measured over all SMs)
//   while the stage's MMAs take some 480 cycles, so L2 bounds it before the tensor cores
//   do.  Clusters of two pairs that shared A by multicast read 22 KB, but only 33 of them,
//   132 SMs, fit: 105 us for 4096 x 14336 x 4096 with the encoder's launch, 103 this way.
// Persistent, one pair of SMs a cluster.  4096 x 14336 x 4096: 95.6 us, 5.0 PFLOP/s, the
// tensor pipe active 70 % of the cycles on all 148 SMs.
//   warp 0      TMA producer of each CTA; a pair's bytes are counted by its leader
//   warp 1      tensor memory; in the leader scale copies, MMAs, commits
//   warps 2-9   epilogue: 64 columns at a time to bf16, shared memory and TMA stores
namespace pair {
constexpr int kThreads = 320;
constexpr int kN = 192;                            // columns of a pair's tile
constexpr int kStages = 5;
constexpr uint32_t kWTile = kN / 2 * 128;
constexpr uint32_t kScaleOff = kCodeTile + kWTile;
constexpr uint32_t kStageBytes = kScaleOff + 1024 + 2048;
constexpr int kSfCol0 = 2 * kN, kSfCols = 24;
constexpr int kPitch = 66;                         // elements of a staged row
constexpr int kStaged = 8 * 4352;                  // bytes, a piece of each epilogue warp
static_assert(kSfCol0 + kStages * kSfCols <= 512, "tensor memory");
static_assert(32 * kPitch * 2 <= 4352, "staging");
}  // namespace pair

struct PairArgs {
  uint16_t* Y;
  int M, N, K;
  uint32_t* status;
};

__global__ void __launch_bounds__(pair::kThreads, 1)
    k_mx4_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmAs, const __grid_constant__ CUtensorMap tmWs,
               const __grid_constant__ CUtensorMap tmY, const __grid_constant__ PairArgs a) {
  using namespace pair;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int first = (int)blockIdx.x / 2, step = (int)gridDim.x / 2;
  const int tiles_m = tiles_of(a.M, 256), tiles = tiles_m * tiles_of(a.N, kN);
  const int kblocks = tiles_of(a.K, kBK), kqs = (int)scale_tiles(a.K);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);    // the leader's producer; the copies add bytes
      mbar_init(&empty[s], 1);   // the leader's commit, to both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 16);   // eight epilogue warps of each CTA (the leader's is used)
    }
    mbar_init(&drain, 1);
    abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmAs);
    tma_prefetch_desc(&tmWs);
  }
  if (warp == 1) {
    tmem_alloc_2sm(&tmem_slot, 512);
    tmem_relinquish_2sm();
  }
  // both CTAs' barriers are initialised before any copy or commit reaches them
  __syncwarp();
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  grid_dep_wait();
  const uint32_t tmem = tmem_slot;
  const uint32_t ring = smem_u32(smem);

  if (warp == 0) {
    if (elect_one()) {
      uint32_t st = ring, ph = 1;
      int s = 0;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int tn = tile / tiles_m, tm = tile - tn * tiles_m;
        const int n0 = tn * kN, tr = tm * 2 + rank;   // this CTA's 128 rows of A
        const int fa = tr * kqs, fw = (n0 >> 7) * kqs;
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = mbar_wait_lazy(&empty[s], ph, &abort_flag, a.status, kDevTimeoutEmpty);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * kStageBytes);
          const uint32_t bar = smem_u32(&full[s]) & kPeerBitMask;
          load_2d_2sm(st, &tmA, bar, kb * 128, tr * 128);
          load_2d_2sm(st + kCodeTile, &tmW, bar, kb * 128, n0 + rank * (kN / 2));
          // scale tiles of 128 rows: two 512-byte rows of the map, the stage's columns; W's
          // two tiles go to both CTAs
          load_2d_2sm(st + kScaleOff, &tmAs, bar, 0, fa + 2 * kb);
          load_2d_2sm(st + kScaleOff + 1024u, &tmWs, bar, 0, fw + 2 * kb);
          load_2d_2sm(st + kScaleOff + 2048u, &tmWs, bar, 0, fw + kqs + 2 * kb);
          st += kStageBytes;
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
            st = ring;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc0 = idesc_mxf4(256, kN, 0), idesc1 = idesc_mxf4(256, kN, 2);
      uint32_t st = ring >> 4, ph = 0, cols = tmem + kSfCol0;
      int s = 0, local = 0;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step, ++local) {
        const int buf = local & 1;
        if (!mbar_wait_lazy(&acc_empty[buf], ((uint32_t)(local >> 1) & 1u) ^ 1u, &abort_flag,
                            a.status, kDevTimeoutMma))
          break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * kN);
        // a tile of 192 rows of W starts at row 0 or 64 of a scale tile; a tensor-memory
        // column holds the scales of 32 rows
        const uint32_t skip = (uint32_t)((tile / tiles_m) & 1) * 2u;
        int left = a.K;   // columns from here on
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = mbar_wait_lazy(&full[s], ph, &abort_flag, a.status, kDevTimeoutFull);
          if (!ok) break;
          tc_fence_after();
          const uint32_t x = code_desc_lo(st << 4), w = x + (kCodeTile >> 4);
          const uint32_t f = scale_desc_lo((st << 4) + kScaleOff);
          const uint32_t sfb = cols + 8u, sfb_at = sfb + skip;
          // 64 columns an MMA; a scale tile serves two
          copy_scales_2sm(cols, f);
          copy_scales_2sm(sfb, f + 64u);
          copy_scales_2sm(sfb + 4u, f + 128u);
          if (left > 128) {
            copy_scales_2sm(cols + 4u, f + 32u);
            copy_scales_2sm(sfb + 8u, f + 96u);
            copy_scales_2sm(sfb + 12u, f + 160u);
          }
          mma_mxf4_2sm(d, code_desc(x), code_desc(w), idesc0, cols, sfb_at, kb > 0);
          if (left > 64)
            mma_mxf4_2sm(d, code_desc(x + 2u), code_desc(w + 2u), idesc1, cols, sfb_at, 1);
          if (left > 128)
            mma_mxf4_2sm(d, code_desc(x + 4u), code_desc(w + 4u), idesc0, cols + 4u, sfb_at + 8u, 1);
          if (left > 192)
            mma_mxf4_2sm(d, code_desc(x + 6u), code_desc(w + 6u), idesc1, cols + 4u, sfb_at + 8u, 1);
          mma_commit_2sm_mc(&empty[s], 0x3);
          left -= kBK;
          st += kStageBytes >> 4;
          cols += kSfCols;
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
            st = ring >> 4;
            cols = tmem + kSfCol0;
          }
        }
        if (ok) mma_commit_2sm_mc(&acc_full[buf], 0x3);
      }
      // every MMA of this thread has finished once `drain` flips
      mma_commit_2sm(&drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&drain, 0) && ns_since(t0) < 200000000ull) {
      }
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t release = mapa_shared(smem_u32(&acc_empty[0]), 0u);
    const bool vec = (a.N & 7) == 0;
    uint8_t* piece = smem + kStages * kStageBytes + (warp - 2) * 4096;
    uint16_t* staged =
        reinterpret_cast<uint16_t*>(smem + kStages * kStageBytes + (warp - 2) * 4352);
    int local = 0;
    for (int tile = first; tile < tiles; tile += step, ++local) {
      const int buf = local & 1;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_lazy(&acc_full[buf], (uint32_t)(local >> 1) & 1u,
                                                  &abort_flag, a.status, kDevTimeoutMma)))
        break;
      tc_fence_after();
      const int tn = tile / tiles_m, tm = tile - tn * tiles_m;
      const int row0 = (tm * 2 + rank) * 128 + quarter * 32;
      // pieces of 64 columns: the first and the last, or the middle one
#pragma unroll 1
      for (int c = half * 64; c < kN; c += 128) {
        uint32_t r[64], v[32];
        const uint32_t at = tmem + (uint32_t)(buf * kN + c) + ((uint32_t)(quarter * 32) << 16);
        tmem_ld32(at, r);
        tmem_ld32(at + 32u, r + 32);
        tmem_ld_wait();
        if (c + 128 >= kN) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(release + (uint32_t)buf * 8u);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
          v[j] = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        const int col = tn * kN + c;
        if (vec) {
          // 128-byte swizzle and a TMA store: stores of each lane's own row would fill
          // the queue that the barriers and the MMAs' issue go through
          if (lane == 0) bulk_wait_read_all();   // the copy before has left the buffer
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(piece + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row0 < a.M && col < a.N)
            tma_store_2d(&tmY, smem_u32(piece), col, row0);
        } else {
          // rows of Y start anywhere: a warp stores 32 neighbouring values of a row
#pragma unroll
          for (int j = 0; j < 32; ++j)
            reinterpret_cast<uint32_t*>(staged)[lane * (kPitch / 2) + j] = v[j];
          __syncwarp();
          const int rows = min(32, a.M - row0);
          for (int i = 0; i < rows; ++i) {
            uint16_t* y = a.Y + (size_t)(row0 + i) * a.N + col;
#pragma unroll
            for (int j = 0; j < 64; j += 32)
              if (col + j + lane < a.N) y[j + lane] = staged[i * kPitch + j + lane];
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_all();   // stores read this CTA's shared memory
  }
  __syncwarp();
  if (abort_flag) {
    // copies in flight may still land: give them time before the CTA exits
    const uint64_t t0 = global_timer_ns();
    while (ns_since(t0) < 1000000ull) {
    }
  }
  // no CTA frees its tensor memory or leaves while the pair's MMAs, another CTA's
  // epilogue or a copy into it may still be under way
  __syncwarp();
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_2sm(tmem, 512);
  }
}

// A map of [rows][row_bytes] bytes as 32-bit words: the scale tiles, 512 bytes each.
static bool scale_map(CUtensorMap* map, const uint8_t* scales, int64_t rows, int64_t K) {
  return encode_tmap_2d(map, scales, CU_TENSOR_MAP_DATA_TYPE_INT32, 4,
                      (uint64_t)((rows + 127) / 128 * scale_tiles(K)), 128, 2, 128,
                      CU_TENSOR_MAP_SWIZZLE_NONE);
}

static cudaError_t launch_pair(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                               const uint8_t* w_codes, const uint8_t* w_scales, int64_t N,
                               int64_t K, uint16_t* Y, uint32_t* status, int sm_count, int early,
                               cudaStream_t st) {
  using namespace pair;
  PairArgs a;
  a.Y = Y;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.status = status;
  const uint64_t cs = (uint64_t)code_stride(K);
  CUtensorMap ta, tw, tas, tws, ty = {};
  if (!encode_tmap_2d(&ta, a_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)M, cs, 128, 128,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_2d(&tw, w_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)N, cs, kN / 2, 128,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !scale_map(&tas, a_scales, M, K) || !scale_map(&tws, w_scales, N, K) ||
      ((N & 7) == 0 && !encode_tmap_2d(&ty, Y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (uint64_t)M,
                                     (uint64_t)N, 32, 64, CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_limit(k_mx4_pair, kMaxDynSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((M + 255) / 256) * ((N + kN - 1) / kN);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 1024 + (size_t)kStages * kStageBytes + kStaged;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  const int64_t pairs = tiles < sm_count / 2 ? tiles : sm_count / 2;
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.numAttrs = early ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, k_mx4_pair, ta, tw, tas, tws, ty, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mx4

// Tokens above which the pair kernel takes over: the stream kernel then reads W for a
// second tile of tokens.  In us a product of encoded matrices, stream / pair, by N x K:
//                  128 tokens     256     |     257          512         1000
//    4096 x 4096   9.4 / 11.2  12.5 / 11.3 | 14.6 / 11.3  15.0 / 11.5  17.7 / 16.1
//   14336 x 4096  13.8 / 16.7  19.1 / 17.1 | 26.2 / 20.7  34.0 / 21.4  63.3 / 30.5
//    4096 x 1024   7.1 /  6.6   9.9 /  6.8 | 11.2 /  6.8  12.0 /  7.5  12.9 /  9.9
//     512 x 4096   7.1 /  9.7   9.9 /  9.6 |  9.9 /  9.7  10.2 /  9.6  19.3 /  9.8
//   4096 x 14336  13.1 / 22.5  17.2 / 22.8 | 22.3 / 22.5  22.8 / 22.9  32.3 / 37.8
//    512 x 14336   8.9 / 19.8  12.2 / 20.0 | 12.4 / 20.0  13.0 / 21.2  23.8 / 21.4
// What tokens alone do not say: short sums would be faster in pairs from fewer tokens on,
// and with few columns and a long K, which the pair kernel does not split, the stream
// kernel would be up to some 800.
constexpr int kPairFrom = 256;

cudaError_t launch_mx4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                            const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, int64_t K,
                            uint16_t* Y, uint32_t* status, int sm_count, int early,
                            cudaStream_t st) {
  const int64_t scale_rows = ((M > N ? M : N) + 127) / 128 * mx4::scale_tiles(K);
  if (M > kPairFrom && scale_rows <= INT32_MAX / 2)
    return mx4::launch_pair(a_codes, a_scales, M, w_codes, w_scales, N, K, Y, status, sm_count,
                            early, st);
  return mx4::launch_stream<-1>(nullptr, 0, a_codes, a_scales, M, w_codes, w_scales, N, K, Y,
                                status, sm_count, early, st);
}

cudaError_t launch_mx4_gemm_small(const void* X, int dtype, int64_t M, int64_t ldx,
                                  const uint8_t* w_codes, const uint8_t* w_scales, int64_t N,
                                  int64_t K, uint16_t* Y, uint32_t* status, int sm_count,
                                  cudaStream_t st) {
  if (dtype == 0)
    return mx4::launch_stream<0>(X, ldx, nullptr, nullptr, M, w_codes, w_scales, N, K, Y, status,
                                 sm_count, 0, st);
  if (dtype == 1)
    return mx4::launch_stream<1>(X, ldx, nullptr, nullptr, M, w_codes, w_scales, N, K, Y, status,
                                 sm_count, 0, st);
  return mx4::launch_stream<2>(X, ldx, nullptr, nullptr, M, w_codes, w_scales, N, K, Y, status,
                               sm_count, 0, st);
}

}  // namespace e8
