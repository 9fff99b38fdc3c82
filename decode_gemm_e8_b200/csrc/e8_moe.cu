// Mixture-of-experts layer for a few tokens, experts in the microscaled 4-bit
// form.  Bound by the bytes of the chosen experts' weights (17/32 a value); all
// launches after the first are programmatic, so that a kernel's prologue overlaps
// its predecessor's end.
//
//   k_moe_logits  router logits (products exact in fp32, sums in fp64) and the
//                 activations as two e4m3 rows a token
//   k_moe_route   top-k, probabilities, and the slots (token, choice) sorted by
//                 expert
//   k_moe_gemm    twice.  The tensor cores take the 4-bit weights as they are
//                 (tcgen05.mma.kind::mxf8f6f4, e2m1 x e4m3): 128 rows of an expert's
//                 matrix on the M side, its tokens on the N side.  The activations
//                 enter as hi + lo, hi = e4m3(x / s), lo = e4m3(16 (x / s - hi)):
//                 four significant bits each, so a bf16 value is held exactly
//                 unless it is 2^14 times smaller than the largest of its row, and
//                 then within 2^-21 of that.  A dequantised operand would cost
//                 about one instruction a weight, which alone exceeds the time HBM
//                 needs to deliver it.
//     up          gate and up rows alternate, so a tile holds both factors of 64
//                 values of h = silu(g) u; the epilogue writes h as two e4m3 rows
//                 again, with a power-of-two scale for the tile's 64 values
//     down        every slot's product times its probability goes to a buffer; the
//                 unit that brings a token's last contribution adds them in the
//                 order of the choices, so the sums do not depend on timing
// With few units the K range is split; partial sums are added in order by the unit
// that arrives last.
#include "e8_internal.h"
#include "e8_mx4.cuh"
#include "e8_tmap.h"

namespace e8 {
namespace moe {

constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTopk = 16;
constexpr int kMaxSlots = kMaxTokens * kMaxTopk;

// Scale byte of an e4m3 pair for values of magnitude up to amax: amax / s lies in
// [128, 256), well inside e4m3's 448; lo's scale is 2^-4 of it, hence the least byte 4.
__device__ __forceinline__ uint32_t pair_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 11u ? e - 7u : 4u);
}
// hi in the low byte, lo in the next.
__device__ __forceinline__ uint32_t to_pair(float v) {
  uint32_t r;
  asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 hh;\n\t.reg .f32 f, d;\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, 0f00000000, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 hh, h;\n\t"
      "mov.b32 {a, b}, hh;\n\t"
      "cvt.f32.f16 f, a;\n\t"
      "sub.f32 d, %1, f;\n\t"
      "mul.f32 d, d, 0f41800000;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, d, 0f00000000;\n\t"
      "or.b16 h, h, l;\n\t"
      "cvt.u32.u16 %0, h;\n\t}\n"
      : "=r"(r)
      : "f"(v));
  return r;
}

// ------------------------------------------------------------------ router ---
constexpr int kLogitTokens = 4;   // tokens a warp takes with one expert's row

// Blocks [0, T): one token's e4m3 rows.  Then 8 experts x kLogitTokens tokens a
// block, one expert a warp.  All blocks clear the counters of the later kernels.
__global__ void __launch_bounds__(256)
    k_moe_logits(const uint16_t* __restrict__ X, int T, int H, const uint16_t* __restrict__ R,
                 int E, double* __restrict__ logits, uint8_t* __restrict__ Xq,
                 float* __restrict__ xs, int* __restrict__ counters, int n_counters) {
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n_counters; i += gridDim.x * 256)
    counters[i] = 0;
  if ((int)blockIdx.x < T) {
    __shared__ uint32_t wmax[8];
    const int t = blockIdx.x;
    const uint4* x = reinterpret_cast<const uint4*>(X + (size_t)t * H);
    uint32_t m = 0;
    for (int k = threadIdx.x; k < H / 8; k += 256) {
      const uint4 v = x[k];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m = max(m, max((w[i] << 16) & 0x7FFF0000u, w[i] & 0x7FFF0000u));
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) wmax[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, wmax[i]);
    const uint32_t byte = pair_byte(m);
    const float inv = byte == 255u ? 0.0f : mx4::inv_scale(byte);
    uint2* hi = reinterpret_cast<uint2*>(Xq + (size_t)(2 * t) * H);
    uint2* lo = reinterpret_cast<uint2*>(Xq + (size_t)(2 * t + 1) * H);
    for (int k = threadIdx.x; k < H / 8; k += 256) {
      const uint4 v = x[k];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t h2[2] = {0, 0}, l2[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = (i & 1) ? bf16_hi_to_f32(w[i >> 1]) : bf16_lo_to_f32(w[i >> 1]);
        const uint32_t p = to_pair(f * inv);
        h2[i >> 2] |= (p & 0xFFu) << (8 * (i & 3));
        l2[i >> 2] |= (p >> 8) << (8 * (i & 3));
      }
      hi[k] = make_uint2(h2[0], h2[1]);
      lo[k] = make_uint2(l2[0], l2[1]);
    }
    if (threadIdx.x == 0) xs[t] = mx4::scale_value(byte);
    return;
  }
  const int b = blockIdx.x - T, eb = (E + 7) / 8;
  const int e = b % eb * 8 + warp, t0 = b / eb * kLogitTokens;
  if (e >= E) return;
  double s[kLogitTokens] = {};
  const uint4* r = reinterpret_cast<const uint4*>(R + (size_t)e * H);
  for (int k = lane; k < H / 8; k += 32) {
    const uint4 rv = r[k];
    const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
    for (int j = 0; j < kLogitTokens; ++j) {
      if (t0 + j >= T) break;
      const uint4 v = reinterpret_cast<const uint4*>(X + (size_t)(t0 + j) * H)[k];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[j] += (double)(bf16_lo_to_f32(rw[i]) * bf16_lo_to_f32(w[i]));
        s[j] += (double)(bf16_hi_to_f32(rw[i]) * bf16_hi_to_f32(w[i]));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kLogitTokens; ++j) {
    for (int o = 16; o; o >>= 1) s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], o);
    if (lane == 0 && t0 + j < T) logits[(size_t)(t0 + j) * E + e] = s[j];
  }
}

// Sorted slots: active expert a has the slots slot_of[off[a]] .. slot_of[off[a + 1] - 1].
struct Lists {
  int* nact;
  int* expert;    // [nact]
  int* off;       // [nact + 1]
  int* slot_of;   // [T topk], slot = token * topk + choice
  float* probs;   // [T topk] by slot
};

// One block.  Warp w chooses for tokens w, w + 32, ..: the largest key (fp64 bits
// in an order-preserving form, NaN lowest) by two 32-bit warp reductions, then the
// lowest expert that has it.
__global__ void __launch_bounds__(1024)
    k_moe_route(const double* __restrict__ logits, int T, int E, int topk, int renorm, Lists l,
                int32_t* __restrict__ experts_out, float* __restrict__ probs_out) {
  __shared__ int16_t chosen[kMaxSlots];
  __shared__ uint16_t count[32][kMaxExperts];   // slots of an expert in a group of 32 slots
  __shared__ int first[kMaxExperts];
  __shared__ uint32_t wsum[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slots = T * topk, groups = (slots + 31) / 32;
  grid_dep_launch();
  for (int i = tid; i < groups * kMaxExperts; i += 1024) (&count[0][0])[i] = 0;
  grid_dep_wait();
  for (int t = warp; t < T; t += 32) {
    uint64_t key[kMaxExperts / 32];
#pragma unroll
    for (int j = 0; j < kMaxExperts / 32; ++j) {
      const int e = lane + 32 * j;
      key[j] = 0;
      if (e < E) {
        const double v = logits[(size_t)t * E + e] + 0.0;   // -0 becomes 0
        const uint64_t u = (uint64_t)__double_as_longlong(v);
        key[j] = v != v ? 1ull : (u >> 63 ? ~u : u | (1ull << 63));
      }
    }
    double top = 0.0;
    float sum = 0.0f, mine = 0.0f;
    int mine_e = 0;
    for (int i = 0; i < topk; ++i) {
      uint64_t best = 0;
      int be = E;
#pragma unroll
      for (int j = 0; j < kMaxExperts / 32; ++j)
        if (key[j] > best) {
          best = key[j];
          be = lane + 32 * j;
        }
      const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(best >> 32));
      const bool in_hi = (uint32_t)(best >> 32) == hi && best != 0;
      const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, in_hi ? (uint32_t)best : 0u);
      const bool in = in_hi && (uint32_t)best == lo;
      const int e = (int)__reduce_min_sync(0xFFFFFFFFu, in ? (uint32_t)be : 0xFFFFFFFFu);
#pragma unroll
      for (int j = 0; j < kMaxExperts / 32; ++j)
        if (lane + 32 * j == e) key[j] = 0;
      const double v = logits[(size_t)t * E + e];
      if (i == 0) top = v;
      const float p = expf((float)(v - top));
      sum += p;
      if (lane == i) {
        mine = p;
        mine_e = e;
      }
    }
    if (!renorm) {
      sum = 0.0f;
      for (int e = lane; e < E; e += 32) sum += expf((float)(logits[(size_t)t * E + e] - top));
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    if (lane < topk) {
      const int s = t * topk + lane;
      chosen[s] = (int16_t)mine_e;
      l.probs[s] = mine / sum;
      if (experts_out) experts_out[s] = mine_e;
      if (probs_out) probs_out[s] = mine / sum;
    }
  }
  __syncthreads();
  // this thread's slot: its place among the slots of its expert in its group
  const int e = tid < slots ? chosen[tid] : -1;
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
  const int place = __popc(same & ((1u << lane) - 1u));
  if (e >= 0 && place == 0) count[warp][e] = (uint16_t)__popc(same);
  __syncthreads();
  // per expert: running count over the groups; then a scan over experts of
  // (is active, slots) packed in one word
  uint32_t v = 0;
  if (tid < E) {
    uint32_t run = 0;
    for (int g = 0; g < groups; ++g) {
      const uint32_t c = count[g][tid];
      count[g][tid] = (uint16_t)run;
      run += c;
    }
    v = run ? (1u << 16) | run : 0u;
  }
  uint32_t scan = v;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) wsum[warp] = scan;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; ++w) before += wsum[w];
  const uint32_t ex = before + scan - v;   // of the experts before this one
  if (tid < E) {
    first[tid] = (int)(ex & 0xFFFFu);
    if (v) {
      l.expert[ex >> 16] = tid;
      l.off[ex >> 16] = (int)(ex & 0xFFFFu);
    }
    if (tid == E - 1) {
      const int n = (int)((ex + v) >> 16);
      *l.nact = n;
      l.off[n] = slots;
    }
  }
  __syncthreads();
  if (e >= 0) l.slot_of[first[e] + count[warp][e] + place] = tid;
}

// ---------------------------------------------------------------- products ---
constexpr int kThreads = 224;
constexpr int kRows = 128;                 // rows of a unit
constexpr int kBK = 128;                   // K of a stage
constexpr int kWBytes = kRows * kBK;       // 16 values in 16 bytes, 8 of them used
constexpr int kMaxStages = 5;                // of 2 kBK columns: one barrier round for 16 KB of weights
constexpr int kConstCol = 256, kSfCol = 264;   // tensor-memory columns of the scales
constexpr int kRingBytes = 212 * 1024;

struct GemmArgs {
  Lists l;
  const uint8_t* w_scales;
  int K, tiles, splits;    // tiles of 128 rows of one expert; K split in `splits`
  int T, topk, stages, b_rows;
  const float* xs;         // up: scale of each token's pair
  uint8_t* hq;             // up: writes, down: reads through the tensor map
  uint8_t* h_scales;       // [active expert][I / 128][512]
  int I;
  float* part;             // partial sums / slot products, fp32
  int* counters;
  uint16_t* Y;
  uint32_t* status;
};

__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// The lists in shared memory.
struct SharedLists {
  int16_t expert[kMaxExperts], off[kMaxExperts + 1], slot[kMaxSlots];
};
// The units of one block in turn: all row tiles and K parts of an expert, then the next.
struct Unit {
  int a, tile, part, expert, off, n, k0, nk;
};
__device__ __forceinline__ Unit unit_at(const GemmArgs& g, const SharedLists& l, int u) {
  Unit r;
  const int per = g.tiles * g.splits;
  r.a = u / per;
  const int rest = u % per;
  r.tile = rest / g.splits;
  r.part = rest % g.splits;
  r.expert = l.expert[r.a];
  r.off = l.off[r.a];
  r.n = l.off[r.a + 1] - r.off;
  const int kq = g.K / kBK;
  r.k0 = kq * r.part / g.splits;
  r.nk = kq * (r.part + 1) / g.splits - r.k0;
  return r;
}

template <bool UP>
__global__ void __launch_bounds__(kThreads, 1)
    k_moe_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ GemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ __align__(16) uint8_t const_sf[512];
  __shared__ __align__(16) uint8_t stage_h[8][2][64];
  __shared__ uint32_t h_max[4][8];
  __shared__ int ready[kMaxTokens];
  __shared__ SharedLists lists;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = 2 * (kWBytes + g.b_rows * kBK + 1024);

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&full[s], 2);   // both producers
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(&drain, 1);
    abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  if (UP && threadIdx.x >= 64 && threadIdx.x < 192) {
    // scales of the activations: 1 for hi rows (even), 2^-4 for lo rows
    reinterpret_cast<uint32_t*>(const_sf)[threadIdx.x - 64] =
        ((threadIdx.x - 64) / 4) & 1 ? 0x7B7B7B7Bu : 0x7F7F7F7Fu;
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (UP) {
    grid_dep_wait();
    grid_dep_launch();
  }
  // (down: the lists were complete before the up kernel let this one start)
  const int nact = *g.l.nact;
  for (int i = threadIdx.x; i <= nact; i += kThreads) {
    lists.off[i] = (int16_t)g.l.off[i];
    if (i < nact) lists.expert[i] = (int16_t)g.l.expert[i];
  }
  for (int i = threadIdx.x; i < g.T * g.topk; i += kThreads)
    lists.slot[i] = (int16_t)g.l.slot_of[i];
  __syncthreads();
  const int units = nact * g.tiles * g.splits;

  const uint32_t ring = smem_u32(smem), b_bytes = (uint32_t)(g.b_rows * 128);
  const int kqs = g.K / 128;
  if (warp == 0) {
    if (lane == 0) {
      // codes and scales of the weights; they do not depend on the preceding kernel
      tma_prefetch_desc(&tmW);
      uint32_t st = ring, ph = 1;
      int s = 0;
      bool ok = true;
      for (int i = blockIdx.x; i < units && ok; i += gridDim.x) {
        const Unit u = unit_at(g, lists, i);
        const int row = (u.expert * g.tiles + u.tile) * kRows;
        const uint8_t* sf = g.w_scales + ((int64_t)(row >> 7) * kqs + u.k0) * 512;
        int x = u.k0 * 128;
        for (int k = u.nk; k > 0; k -= 2) {
          if (!mbar_wait_lazy(&empty[s], ph, &abort_flag, g.status, kDevTimeoutEmpty)) {
            ok = false;
            break;
          }
          // the tensor map unpacks: its bytes are counted as they lie in memory
          const uint32_t half = k > 1 ? 2u : 1u;
          mbar_arrive_expect_tx(&full[s], half * (kWBytes / 2 + 512u));
          load_2d(st, &tmW, &full[s], x, row);
          if (k > 1) load_2d(st + kWBytes, &tmW, &full[s], x + 128, row);
          load_bulk(st + 2u * (kWBytes + b_bytes), sf, half * 512u, &full[s]);
          x += 256;
          sf += 1024;
          st += (uint32_t)stage_bytes;
          if (++s == g.stages) {
            s = 0;
            ph ^= 1u;
            st = ring;
          }
        }
      }
    }
  } else if (warp == 6) {
    // the tokens' rows: two (hi and lo) a copy in the up product, where tokens lie in
    // order of the batch; sixteen a copy in the down product, sorted by expert
    if (lane == 0) tma_prefetch_desc(&tmB);
    if (!UP) grid_dep_wait();
    uint32_t st = ring + 2u * kWBytes, ph = 1;
    int s = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < units && ok; i += gridDim.x) {
      const Unit u = unit_at(g, lists, i);
      const int copies = UP ? u.n : (u.n + 7) / 8;
      int row0 = 0, row1 = 0;
      if (UP) {
        if (lane < u.n) row0 = lists.slot[u.off + lane] / g.topk * 2;
        if (lane + 32 < u.n) row1 = lists.slot[u.off + lane + 32] / g.topk * 2;
      } else {
        row0 = 2 * u.off + lane * 16;
      }
      const uint32_t bytes = UP ? (uint32_t)copies * 256u : (uint32_t)copies * 2048u + 512u;
      const uint32_t to = (uint32_t)lane * (UP ? 256u : 2048u);
      const uint8_t* sf = g.h_scales + ((int64_t)u.a * kqs + u.k0) * 512;
      int x = u.k0 * 128;
      for (int k = u.nk; k > 0; k -= 2) {
        ok = __all_sync(0xFFFFFFFFu,
                        mbar_wait_lazy(&empty[s], ph, &abort_flag, g.status, kDevTimeoutEmpty));
        if (!ok) break;
        const uint32_t half = k > 1 ? 2u : 1u;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], half * bytes);
        __syncwarp();
        for (uint32_t h = 0; h < half; ++h) {
          if (lane < copies) load_2d(st + h * b_bytes + to, &tmB, &full[s], x + 128 * (int)h, row0);
          if (UP && lane + 32 < copies)
            load_2d(st + h * b_bytes + to + 32u * 256u, &tmB, &full[s], x + 128 * (int)h, row1);
        }
        if (!UP && lane == 0) load_bulk(st + 2u * b_bytes + 1024u, sf, half * 512u, &full[s]);
        x += 256;
        sf += 1024;
        st += (uint32_t)stage_bytes;
        if (++s == g.stages) {
          s = 0;
          ph ^= 1u;
          st = ring + 2u * kWBytes;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      if (UP) mx4::copy_scales(tmem + kConstCol, mx4::scale_desc_lo(smem_u32(const_sf)));
      const uint32_t b_off = 2u * kWBytes >> 4, f_off = 2u * (kWBytes + b_bytes) >> 4;
      uint32_t st = ring >> 4, ph = 0, cols = tmem + kSfCol;
      int s = 0, local = 0;
      bool ok = true;
      for (int i = blockIdx.x; i < units && ok; i += gridDim.x, ++local) {
        const Unit u = unit_at(g, lists, i);
        const int buf = local & 1;
        if (!mbar_wait_lazy(&acc_empty[buf], ((uint32_t)(local >> 1) & 1u) ^ 1u, &abort_flag,
                            g.status, kDevTimeoutMma))
          break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)buf * 128u;
        const uint32_t idesc = mx4::idesc_mxf4_f8(128, (uint32_t)(u.n + 7) / 8 * 16, 0);
        uint32_t acc = 0;
        for (int k = u.nk; k > 0; k -= 2) {
          if (!mbar_wait_lazy(&full[s], ph, &abort_flag, g.status, kDevTimeoutFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w = mx4::code_desc_lo(st << 4), b = w + b_off;
          const uint32_t f = mx4::scale_desc_lo((st + f_off) << 4);
          const uint32_t sfb = UP ? tmem + kConstCol : cols + 8u;
          mx4::copy_scales(cols, f);
          if (!UP) mx4::copy_scales(sfb, f + 64u);
          if (k > 1) {
            mx4::copy_scales(cols + 4u, f + 32u);
            if (!UP) mx4::copy_scales(sfb + 4u, f + 96u);
          }
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            mx4::mma_mxf8f6f4(d, mx4::code_desc(w + 2u * j), mx4::code_desc(b + 2u * j),
                              idesc | (j << 4) | (j << 29), cols, sfb, acc);
            acc = 1;
          }
          if (k > 1) {
            const uint32_t w1 = w + (kWBytes >> 4), b1 = b + (b_bytes >> 4);
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              mx4::mma_mxf8f6f4(d, mx4::code_desc(w1 + 2u * j), mx4::code_desc(b1 + 2u * j),
                                idesc | (j << 4) | (j << 29), cols + 4u, UP ? sfb : sfb + 4u, 1);
          }
          mma_commit(&empty[s]);
          st += (uint32_t)stage_bytes >> 4;
          cols += 16u;
          if (++s == g.stages) {
            s = 0;
            ph ^= 1u;
            st = ring >> 4;
            cols = tmem + kSfCol;
          }
        }
        if (ok) mma_commit(&acc_full[buf]);
      }
      // every MMA of this thread has finished once `drain` flips
      mma_commit(&drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&drain, 0) && global_timer_ns() - t0 < 200000000ull) {
      }
    }
  } else {
    const int quarter = warp & 3, row = quarter * 32 + lane, et = (int)threadIdx.x - 64;
    const int slots = g.T * g.topk, width = g.tiles * kRows;
    int local = 0;
    for (int i = blockIdx.x; i < units; i += gridDim.x, ++local) {
      const Unit u = unit_at(g, lists, i);
      const int buf = local & 1;
      const bool ok = mbar_wait_lazy(&acc_full[buf], (uint32_t)(local >> 1) & 1u, &abort_flag,
                                     g.status, kDevTimeoutMma);
      __syncwarp();
      if (bar_red_or(1, 128, !ok)) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)buf * 128u + ((uint32_t)(quarter * 32) << 16);
      // eight tokens' values of this row (hi + lo)
      auto read8 = [&](int j0, float (&v)[8]) {
        uint32_t r[16];
        tmem_ld16(d + (uint32_t)j0 * 2u, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = __uint_as_float(r[2 * j]) + __uint_as_float(r[2 * j + 1]);
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
      };
      if (UP) {
        bool last = true;
        if (g.splits > 1) {
          for (int j0 = 0; j0 < u.n; j0 += 8) {
            float v[8];
            read8(j0, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j0 + j < u.n)
                g.part[((size_t)u.part * slots + u.off + j0 + j) * width + u.tile * kRows + row] =
                    v[j];
          }
          release();
          __threadfence();
          bar_sync(1, 128);
          if (et == 0)
            ready[0] = atomicAdd(&g.counters[u.a * g.tiles + u.tile], 1) == g.splits - 1;
          bar_sync(1, 128);
          last = ready[0] != 0;
          bar_sync(1, 128);   // ready is free again
          __threadfence();
        }
        if (last) {
          for (int j0 = 0; j0 < u.n; j0 += 8) {
            float v[8];
            if (g.splits == 1) {
              read8(j0, v);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                v[j] = 0.0f;
                if (j0 + j < u.n)
                  for (int p = 0; p < g.splits; ++p)
                    v[j] += __ldcg(&g.part[((size_t)p * slots + u.off + j0 + j) * width +
                                           u.tile * kRows + row]);
              }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float x = j0 + j < u.n ? g.xs[lists.slot[u.off + j0 + j] / g.topk] : 0.0f;
              const float mine = v[j] * x, other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
              const float gate = lane & 1 ? other : mine, up = lane & 1 ? mine : other;
              v[j] = j0 + j < u.n ? gate / (1.0f + __expf(-gate)) * up : 0.0f;
              const uint32_t m =
                  __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[j]) & 0x7FFFFFFFu);
              if (lane == 0) h_max[quarter][j] = m;
            }
            bar_sync(1, 128);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t byte = pair_byte(
                  max(max(h_max[0][j], h_max[1][j]), max(h_max[2][j], h_max[3][j])));
              const uint32_t p = byte == 255u ? 0u : to_pair(v[j] * mx4::inv_scale(byte));
              stage_h[j][lane & 1][quarter * 16 + lane / 2] = (uint8_t)(lane & 1 ? p >> 8 : p);
            }
            if (et < 16 && j0 + et / 2 < u.n) {
              // scale bytes of hi and lo rows, both blocks of 32 of this tile
              const int j = et / 2, r = 2 * (j0 + j) + (et & 1), at = u.tile * 64;
              uint32_t byte = pair_byte(
                  max(max(h_max[0][j], h_max[1][j]), max(h_max[2][j], h_max[3][j])));
              if ((et & 1) && byte != 255u) byte -= 4u;
              *reinterpret_cast<uint16_t*>(
                  g.h_scales + ((int64_t)u.a * (g.I / 128) + at / 128) * 512 + (r & 31) * 16 +
                  (r >> 5) * 4 + (at & 127) / 32) = (uint16_t)(byte | byte << 8);
            }
            bar_sync(1, 128);
            if (et < 64 && j0 + et / 8 < u.n) {
              const int j = et / 8, r = (et >> 2) & 1, q = et & 3;
              *reinterpret_cast<uint4*>(g.hq + (size_t)(2 * (u.off + j0 + j) + r) * g.I +
                                        u.tile * 64 + q * 16) =
                  *reinterpret_cast<const uint4*>(&stage_h[j][r][q * 16]);
            }
          }
        }
        if (g.splits == 1) release();
      } else {
        for (int j0 = 0; j0 < u.n; j0 += 8) {
          float v[8];
          read8(j0, v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j0 + j < u.n) {
              const int slot = lists.slot[u.off + j0 + j];
              g.part[((size_t)u.part * slots + slot) * width + u.tile * kRows + row] =
                  v[j] * g.l.probs[slot];
            }
        }
        release();
        __threadfence();
        bar_sync(1, 128);
        if (et < u.n) {
          const int t = lists.slot[u.off + et] / g.topk;
          ready[et] =
              atomicAdd(&g.counters[u.tile * g.T + t], 1) == g.topk * g.splits - 1 ? t : -1;
        }
        bar_sync(1, 128);
        __threadfence();
        for (int j = 0; j < u.n; ++j) {
          const int t = ready[j];
          if (t < 0) continue;
          float y = 0.0f;
#pragma unroll 8
          for (int c = 0; c < g.topk * g.splits; ++c)
            y += __ldcg(&g.part[((size_t)(c % g.splits) * slots + t * g.topk + c / g.splits) *
                                    width + u.tile * kRows + row]);
          g.Y[(size_t)t * width + u.tile * kRows + row] =
              (uint16_t)(pack_bf16x2(y, 0.0f) & 0xFFFFu);
        }
        bar_sync(1, 128);   // ready is free again
      }
    }
  }
  __syncwarp();
  if (abort_flag) {
    // copies in flight may still land: give them time before the CTA exits
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- host ---
// K parts of a product of `tiles` row tiles of an expected number of experts: the
// rounds of units over the SMs, each as long as its share of K and about four
// stages of fixed cost.
static int choose_splits(int64_t T, int64_t E, int topk, int64_t tiles, int64_t K) {
  double miss = 1.0;
  for (int64_t t = 0; t < T; ++t) miss *= 1.0 - (double)topk / (double)E;
  const double n = (double)E * (1.0 - miss);
  const int64_t units = (int64_t)(n + 0.5 < 1.0 ? 1.0 : n + 0.5) * tiles;
  const int kq = (int)(K / kBK);
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= 8 && s <= kq; ++s) {
    const double rounds = (double)((units * s + 147) / 148);
    const double c = rounds * ((double)kq / s + 4.0) + (s > 1 ? 2.0 : 0.0);
    if (c < cost - 1e-9) {
      cost = c;
      best = s;
    }
  }
  return best;
}

struct Layout {
  size_t logits, xq, xs, lists, hq, h_scales, part_up, part_down, counters, total;
  int splits_up, splits_down, max_act, n_up, n_down;
};
static Layout layout(int64_t T, int64_t H, int64_t E, int topk, int64_t I) {
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~size_t(255);
    return here;
  };
  const size_t slots = (size_t)T * topk;
  l.max_act = (int)(slots < (size_t)E ? slots : (size_t)E);
  l.splits_up = choose_splits(T, E, topk, 2 * I / kRows, H);
  l.splits_down = choose_splits(T, E, topk, H / kRows, I);
  l.n_up = (int)(l.max_act * (2 * I / kRows));
  l.n_down = (int)(T * (H / kRows));
  l.logits = take((size_t)T * E * 8);
  l.xq = take((size_t)T * 2 * H);
  l.xs = take((size_t)T * 4);
  l.lists = take((1 + (size_t)E + (size_t)E + 1 + 2 * slots) * 4);
  l.hq = take(slots * 2 * I);
  l.h_scales = take((size_t)l.max_act * (I / 128) * 512);
  l.part_up = take(l.splits_up > 1 ? (size_t)l.splits_up * slots * 2 * I * 4 : 0);
  l.part_down = take((size_t)l.splits_down * slots * H * 4);
  l.counters = take((size_t)(l.n_up + l.n_down) * 4);
  l.total = at;
  return l;
}

// 4-bit rows unpacked to 16 bytes for each 16 values on the way to shared memory
// (row length and start a multiple of 128 values).
static bool weights_map(CUtensorMap* map, const uint8_t* base, uint64_t rows, uint64_t K) {
  // one matrix's map depends on these arguments alone; the last few are kept
  struct Entry {
    const void* base;
    uint64_t rows, K;
    CUtensorMap map;
  };
  constexpr int kEntries = 64;
  thread_local Entry cache[kEntries];
  thread_local int used = 0, next = 0;
  for (int i = 0; i < used; ++i)
    if (cache[i].base == base && cache[i].rows == rows && cache[i].K == K) {
      *map = cache[i].map;
      return true;
    }
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  cuuint32_t box[2] = {128, (cuuint32_t)kRows};
  cuuint32_t estr[2] = {1, 1};
  if (fn(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<uint8_t*>(base), dims, strides,
         box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  cache[next].base = base;
  cache[next].rows = rows;
  cache[next].K = K;
  cache[next].map = *map;
  next = (next + 1) % kEntries;
  if (used < kEntries) ++used;
  return true;
}

}  // namespace moe

size_t moe_workspace(int64_t T, int64_t H, int64_t E, int topk, int64_t I) {
  return moe::layout(T, H, E, topk, I).total;
}

cudaError_t launch_moe(const MoeArgs& a, int sm_count, cudaStream_t st) {
  using namespace moe;
  const Layout l = layout(a.T, a.H, a.E, a.topk, a.I);
  uint8_t* w = static_cast<uint8_t*>(a.workspace);
  const int slots = a.T * a.topk;
  double* logits = reinterpret_cast<double*>(w + l.logits);
  float* xs = reinterpret_cast<float*>(w + l.xs);
  int* counters = reinterpret_cast<int*>(w + l.counters);
  Lists ls;
  ls.nact = reinterpret_cast<int*>(w + l.lists);
  ls.expert = ls.nact + 1;
  ls.off = ls.expert + a.E;
  ls.slot_of = ls.off + a.E + 1;
  ls.probs = reinterpret_cast<float*>(ls.slot_of + slots);

  CUtensorMap tw13, tw2, tx, th;
  if (!weights_map(&tw13, a.w13_codes, (uint64_t)a.E * 2 * a.I, (uint64_t)a.H) ||
      !weights_map(&tw2, a.w2_codes, (uint64_t)a.E * a.H, (uint64_t)a.I) ||
      !make_tmap_2d(&tx, w + l.xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.T * 2,
                    (uint64_t)a.H, 2, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&th, w + l.hq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)slots * 2,
                    (uint64_t)a.I, 16, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_limit(k_moe_gemm<true>, kMaxDynSmem);
  if (e == cudaSuccess) e = ensure_smem_limit(k_moe_gemm<false>, kMaxDynSmem);
  if (e != cudaSuccess) return e;

  const int logit_blocks =
      a.T + (a.E + 7) / 8 * ((a.T + kLogitTokens - 1) / kLogitTokens);
  k_moe_logits<<<logit_blocks, 256, 0, st>>>(a.X, a.T, a.H, a.router, a.E, logits, w + l.xq, xs,
                                             counters, l.n_up + l.n_down);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  e = cudaLaunchKernelEx(&cfg, k_moe_route, (const double*)logits, a.T, a.E, a.topk, a.renorm, ls,
                         a.experts, a.probs);
  if (e != cudaSuccess) return e;

  GemmArgs g;
  g.l = ls;
  g.T = a.T;
  g.topk = a.topk;
  g.b_rows = (2 * a.T + 15) / 16 * 16;
  const int stage_bytes = 2 * (kWBytes + g.b_rows * kBK + 1024);
  g.stages = kRingBytes / stage_bytes < kMaxStages ? kRingBytes / stage_bytes : kMaxStages;
  g.xs = xs;
  g.hq = w + l.hq;
  g.h_scales = w + l.h_scales;
  g.I = a.I;
  g.Y = a.Y;
  g.status = a.status;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 1024 + (size_t)g.stages * stage_bytes;

  g.w_scales = a.w13_scales;
  g.K = a.H;
  g.tiles = 2 * a.I / kRows;
  g.splits = l.splits_up;
  g.part = reinterpret_cast<float*>(w + l.part_up);
  g.counters = counters;
  int64_t units = (int64_t)l.max_act * g.tiles * g.splits;
  cfg.gridDim = dim3((unsigned)(units < sm_count ? units : sm_count));
  e = cudaLaunchKernelEx(&cfg, k_moe_gemm<true>, tw13, tx, g);
  if (e != cudaSuccess) return e;

  g.w_scales = a.w2_scales;
  g.K = a.I;
  g.tiles = a.H / kRows;
  g.splits = l.splits_down;
  g.part = reinterpret_cast<float*>(w + l.part_down);
  g.counters = counters + l.n_up;
  units = (int64_t)l.max_act * g.tiles * g.splits;
  cfg.gridDim = dim3((unsigned)(units < sm_count ? units : sm_count));
  e = cudaLaunchKernelEx(&cfg, k_moe_gemm<false>, tw2, th, g);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace e8
