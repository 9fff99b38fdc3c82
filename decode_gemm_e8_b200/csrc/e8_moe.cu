// Mixture-of-experts layer for a few tokens, experts in the microscaled 4-bit
// form.  Bound by the bytes of the chosen experts' weights (17/32 a value); all
// launches after the first are programmatic, so that a kernel's prologue overlaps
// its predecessor's end.
//
//   k_moe_route   router logits (products exact in fp32 and summed in fp64), top-k and
//                 probabilities, and the activations as two e4m3 rows a token
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
//     down        every slot's product times its probability goes to a buffer
//   k_moe_combine adds a token's slots in the order of its choices: no sum depends on
//                 timing (a count of arrivals at the end of each down unit cost three
//                 times the unit's own work at 64 tokens)
// With few units the K range is split; the up product's partial sums are added in order
// by the unit that arrives last, the down product's by k_moe_combine.
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
constexpr int kRouteCtas = 8, kRouteTokens = 4;   // a cluster takes 4 tokens

// Sums 16 values over the warp's lanes; lane l returns the sum of v[l >> 1].
__device__ __forceinline__ double warp_sum16(double (&v)[16], int lane) {
#pragma unroll
  for (int w = 8; w; w >>= 1) {
    const bool up = (lane & (2 * w)) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const double send = up ? v[i] : v[i + w];
      v[i] = (up ? v[i + w] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, send, 2 * w);
    }
  }
  return v[0] + __shfl_xor_sync(0xFFFFFFFFu, v[0], 1);
}

// One cluster of 8 CTAs for 4 tokens: each CTA takes an eighth of the experts, its
// warps 4 experts x 4 tokens of a part of H each (16 fp64 sums a lane; converting
// bf16 to fp64 costs four times an fp64 product, so every converted value is used
// four times).  The logits of token j go to CTA j, which chooses; CTAs 4..7 write
// the tokens' e4m3 rows meanwhile.  One launch and no counters: the logits cross
// CTAs in distributed shared memory.
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(256)
    k_moe_route(const uint16_t* __restrict__ X, int T, int H, const uint16_t* __restrict__ R,
                int E, int topk, int renorm, int32_t* __restrict__ experts,
                float* __restrict__ probs, int32_t* __restrict__ experts_out,
                float* __restrict__ probs_out, uint8_t* __restrict__ Xq, float* __restrict__ xs,
                int* __restrict__ counters, int n_counters) {
  __shared__ double part[16][16];   // [experts of four x part of H][expert, token]
  __shared__ double logit[kMaxExperts];
  __shared__ uint64_t key[kMaxExperts];
  __shared__ int chosen[kMaxTopk];
  __shared__ uint32_t wmax[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank(), t0 = (int)blockIdx.x / kRouteCtas * kRouteTokens;
  const int nt = min(kRouteTokens, T - t0);
  grid_dep_launch();
  cluster_arrive();   // (the wait below: every CTA of the cluster has started)
  for (int i = blockIdx.x * 256 + tid; i < n_counters; i += gridDim.x * 256) counters[i] = 0;

  const int per = (E + kRouteCtas - 1) / kRouteCtas, e0 = rank * per;
  const int ne = min(per, E - e0), groups = ne > 0 ? (ne + 3) / 4 : 0;
  const int parts = groups > 0 && groups < 8 ? 8 / groups : 1, chunks = (H + 255) / 256;
  for (int item = warp; item < groups * parts; item += 8) {
    const int e = e0 + item / parts * 4, p = item % parts;
    double acc[16] = {};
    for (int c = chunks * p / parts; c < chunks * (p + 1) / parts; ++c) {
      const int k = c * 256 + lane * 8;
      uint4 r[4], x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[j] = x[j] = make_uint4(0, 0, 0, 0);
        if (k < H && e + j < e0 + ne)
          r[j] = *reinterpret_cast<const uint4*>(R + (size_t)(e + j) * H + k);
        if (k < H && j < nt)
          x[j] = *reinterpret_cast<const uint4*>(X + (size_t)(t0 + j) * H + k);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        double rd[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = i < 2 ? r[j].x : i < 4 ? r[j].y : i < 6 ? r[j].z : r[j].w;
          rd[j] = (double)((i & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= nt) break;
          const uint32_t w = i < 2 ? x[j].x : i < 4 ? x[j].y : i < 6 ? x[j].z : x[j].w;
          const double xd = (double)((i & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w));
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q * 4 + j] = fma(rd[q], xd, acc[q * 4 + j]);
        }
      }
    }
    const double s = warp_sum16(acc, lane);
    if (!(lane & 1)) part[item][lane >> 1] = s;
  }
  __syncthreads();
  cluster_wait();
  if (tid < ne * kRouteTokens) {
    const int el = tid / kRouteTokens, j = tid % kRouteTokens;
    double s = 0.0;
    for (int p = 0; p < parts; ++p) s += part[el / 4 * parts + p][(el & 3) * 4 + j];
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(
                     mapa_shared(smem_u32(&logit[e0 + el]), (uint32_t)j)),
                 "d"(s)
                 : "memory");
  }
  __syncwarp();
  cluster_arrive();
  if (rank >= kRouteTokens && rank - kRouteTokens < nt) {
    // hi and lo rows of one token
    const int t = t0 + rank - kRouteTokens;
    const uint4* x = reinterpret_cast<const uint4*>(X + (size_t)t * H);
    uint32_t m = 0;
    for (int k = tid; k < H / 8; k += 256) {
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
    for (int k = tid; k < H / 8; k += 256) {
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
    if (tid == 0) xs[t] = mx4::scale_value(byte);
  }
  __syncwarp();
  cluster_wait();
  if (rank >= nt) return;
  // this CTA chooses for token t0 + rank: an expert's place is the number of experts
  // before it (larger logit, or the same and a lower number; NaN comes last)
  const int t = t0 + rank;
  for (int e = tid; e < E; e += 256) {
    const double v = logit[e] + 0.0;   // -0 becomes 0
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    key[e] = v != v ? 0ull : (u >> 63 ? ~u : u | (1ull << 63));
  }
  __syncthreads();
  for (int e = tid; e < E; e += 256) {
    const uint64_t mine = key[e];
    int place = 0;
#pragma unroll 4
    for (int j = 0; j < E; ++j) place += key[j] > mine || (key[j] == mine && j < e);
    if (place < topk) chosen[place] = e;
  }
  __syncthreads();
  if (warp) return;
  const double top = logit[chosen[0]];
  float p = 0.0f, sum = 0.0f;
  if (lane < topk) p = expf((float)(logit[chosen[lane]] - top));
  if (renorm) {
    sum = p;
  } else {
    for (int e = lane; e < E; e += 32) sum += expf((float)(logit[e] - top));
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane < topk) {
    const int s = t * topk + lane;
    experts[s] = chosen[lane];
    probs[s] = p / sum;
    if (experts_out) experts_out[s] = chosen[lane];
    if (probs_out) probs_out[s] = p / sum;
  }
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
  const int32_t* experts;  // by slot = token * topk + choice
  const float* probs;
  const uint8_t *w_codes, *w_scales;
  int K, tiles, splits;    // tiles of 128 rows of one expert; K split in `splits`
  // Divisions without a divide: `per` = tiles * splits units an expert, the block's first
  // expert and rest, the grid's step in the same terms, and ceil(2^16 / d) for the
  // divisors splits and topk (exact: dividend < 8192, divisor <= 16, product < 2^16 off)
  int per, step_a, step_rest, by_splits, by_topk, by_per;
  int T, E, topk, stages, b_rows;
  const uint8_t* xq;       // up: the tokens' hi and lo rows
  const float* xs;         // up: scale of each token's pair
  uint8_t* hq;             // up: writes, down: reads through the tensor map
  uint8_t* h_scales;       // [active expert][I / 128][512]
  int I;
  float* part;             // partial sums / slot products, fp32
  int* counters;
  uint32_t* status;
};

__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// Counts this block's arrival after its other threads' writes (a barrier came before).
__device__ __forceinline__ int arrive_gpu(int* counter) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier once this thread's copies so far have landed.
__device__ __forceinline__ void copy_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// Slots sorted by expert: active expert a (in order of number) has the slots
// slot[off[a]] .. slot[off[a + 1] - 1], by rising slot.
struct SharedLists {
  int16_t expert[kMaxExperts], off[kMaxExperts + 1], slot[kMaxSlots];
  uint8_t token[kMaxSlots];
  int16_t k_at[9];   // first 128-column step of each K part
  int nact;
  uint32_t wsum[8];
};

// Up to 32 slots: one warp, a lane a slot.
__device__ __forceinline__ void build_small(SharedLists& l, const int32_t* __restrict__ experts,
                                            int slots, int by_topk) {
  const int lane = threadIdx.x & 31;
  const int e = lane < slots ? experts[lane] : INT32_MAX;
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
  const bool head = (same & ((1u << lane) - 1u)) == 0 && lane < slots;
  // slots and active experts before this one's
  int pos = __popc(same & ((1u << lane) - 1u)), act = 0;
#pragma unroll 4
  for (int j = 0; j < slots; ++j) {
    const int other = __shfl_sync(0xFFFFFFFFu, e, j);
    const bool other_head = __shfl_sync(0xFFFFFFFFu, (int)head, j) != 0;
    pos += other < e;
    act += other < e && other_head;
  }
  if (lane < slots) {
    l.slot[pos] = (int16_t)lane;
    l.token[pos] = (uint8_t)(lane * by_topk >> 16);
    if (head) {
      l.expert[act] = (int16_t)e;
      l.off[act] = (int16_t)pos;
    }
  }
  const int nact = __popc(__ballot_sync(0xFFFFFFFFu, head));
  if (lane == 0) {
    l.off[nact] = (int16_t)slots;
    l.nact = nact;
  }
}

// Any number (all threads; `scratch`: 32 E + 4 kMaxSlots + 2 E bytes).
__device__ __forceinline__ void build_lists(SharedLists& l, uint8_t* scratch,
                                            const int32_t* __restrict__ experts, int slots, int E,
                                            int by_topk) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = (slots + 31) / 32;
  uint8_t* count = scratch;   // [groups][E]: slots of an expert in a group of 32 slots
  int16_t* se = reinterpret_cast<int16_t*>(scratch + 32 * kMaxExperts);
  int16_t* sp = se + kMaxSlots;
  int16_t* first = sp + kMaxSlots;
  for (int i = tid; i < (groups * E + 3) / 4; i += kThreads)
    reinterpret_cast<uint32_t*>(count)[i] = 0;
  __syncthreads();
  for (int g = warp; g < groups; g += kThreads / 32) {
    const int s = g * 32 + lane, e = s < slots ? experts[s] : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const int place = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && place == 0) count[g * E + e] = (uint8_t)__popc(same);
    se[s] = (int16_t)e;
    sp[s] = (int16_t)place;
  }
  __syncthreads();
  // running counts over the groups, then a scan over experts of (is active, slots)
  const int per = (E + kThreads - 1) / kThreads;
  uint32_t mine = 0;
  for (int e = tid * per; e < min(E, (tid + 1) * per); ++e) {
    uint32_t run = 0;
#pragma unroll 4
    for (int g = 0; g < groups; ++g) {
      const uint32_t c = count[g * E + e];
      count[g * E + e] = (uint8_t)run;
      run += c;
    }
    first[e] = (int16_t)run;
    mine += run ? (1u << 16) | run : 0u;
  }
  uint32_t scan = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) l.wsum[warp] = scan;
  __syncthreads();
  uint32_t at = scan - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) at += l.wsum[w];
    total += l.wsum[w];
  }
  for (int e = tid * per; e < min(E, (tid + 1) * per); ++e) {
    const uint32_t n = (uint32_t)first[e];
    first[e] = (int16_t)(at & 0xFFFFu);
    if (n) {
      l.expert[at >> 16] = (int16_t)e;
      l.off[at >> 16] = (int16_t)(at & 0xFFFFu);
      at += (1u << 16) | n;
    }
  }
  if (tid == 0) {
    l.nact = (int)(total >> 16);
    l.off[total >> 16] = (int16_t)slots;
  }
  __syncthreads();
  for (int s = tid; s < slots; s += kThreads) {
    const int pos = first[se[s]] + count[(s >> 5) * E + se[s]] + sp[s];
    l.slot[pos] = (int16_t)s;
    l.token[pos] = (uint8_t)(s * by_topk >> 16);
  }
  fence_proxy_async_smem();   // the scratch space becomes the copies' ring
}

// The units of one block in turn: all row tiles and K parts of an expert, then the next.
struct Unit {
  int a, rest;                                    // active expert; tile * splits + part
  int tile, part, expert, off, n, k0, nk;
  __device__ __forceinline__ void begin(const GemmArgs& g) {
    a = g.per > (int)blockIdx.x ? 0 : (int)blockIdx.x * g.by_per >> 16;
    rest = (int)blockIdx.x - a * g.per;
  }
  __device__ __forceinline__ void next(const GemmArgs& g) {
    a += g.step_a;
    rest += g.step_rest;
    if (rest >= g.per) {
      rest -= g.per;
      ++a;
    }
  }
  // false after the last unit
  __device__ __forceinline__ bool load(const GemmArgs& g, const SharedLists& l) {
    if (a >= l.nact) return false;
    tile = rest * g.by_splits >> 16;
    part = rest - tile * g.splits;
    expert = l.expert[a];
    off = l.off[a];
    n = l.off[a + 1] - off;
    k0 = l.k_at[part];
    nk = l.k_at[part + 1] - k0;
    return true;
  }
};

// Warps: 0 weights producer, 6 tokens producer, 1 MMAs, 2..5 epilogue.  At 16 KB of
// weights a stage the SM's share of HBM leaves each role some 700 cycles a stage: one
// elected thread runs a role's whole loop with its addresses in registers.
template <bool UP>
__global__ void __launch_bounds__(kThreads, 1)
    k_moe_gemm(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ GemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ __align__(16) uint8_t const_sf[512];
  __shared__ __align__(16) float stage_v[8][128 + 4];
  __shared__ int ready;
  __shared__ float token_scale[kMaxTokens];
  __shared__ SharedLists lists;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b_bytes = (uint32_t)(g.b_rows * 128);
  const uint32_t stage_bytes = 2u * (kWBytes + b_bytes + 1024u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&full[s], UP ? 33 : 2);   // the weights' producer, and the tokens'
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(&drain, 1);
    abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    if (!UP) tma_prefetch_desc(&tmB);
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
  if (UP) {
    grid_dep_wait();
    grid_dep_launch();
  }
  // (down: the choice was complete before the up kernel let this one start)
  if (!UP) grid_dep_launch();
  tc_fence_before();
  const int slots = g.T * g.topk;
  if (UP && threadIdx.x < g.T) token_scale[threadIdx.x] = g.xs[threadIdx.x];
  if (threadIdx.x >= 128 && threadIdx.x <= 128 + g.splits)
    lists.k_at[threadIdx.x - 128] =
        (int16_t)((g.K / kBK) * ((int)threadIdx.x - 128) * g.by_splits >> 16);
  if (slots > 32) build_lists(lists, smem, g.experts, slots, g.E, g.by_topk);
  else if (warp == 2) build_small(lists, g.experts, slots, g.by_topk);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t ring = smem_u32(smem);
  const int kqs = g.K / kBK;

  if (warp == 0) {
    if (elect_one()) {
      // codes and scales of the weights; they do not depend on the preceding kernel
      uint32_t st = ring, ph = 1;
      int s = 0;
      bool ok = true;
      Unit u;
      for (u.begin(g); ok && u.load(g, lists); u.next(g)) {
        const int row = (u.expert * g.tiles + u.tile) * kRows;
        const uint8_t* sf = g.w_scales + ((int64_t)(row >> 7) * kqs + u.k0) * 512;
        int x = u.k0 * kBK;
        bool ahead = true;
        for (int k = u.nk; k > 0; k -= 2) {
          ok = mbar_wait_lazy(&empty[s], ph, &abort_flag, g.status, kDevTimeoutEmpty);
          if (!ok) break;
          // the tensor map unpacks: its bytes are counted as they lie in memory
          const uint32_t half = k > 1 ? 2u : 1u;
          mbar_arrive_expect_tx(&full[s], half * (kWBytes / 2 + 512u));
          load_2d(st, &tmW, &full[s], x, row);
          if (k > 1) load_2d(st + kWBytes, &tmW, &full[s], x + kBK, row);
          load_bulk(st + 2u * (kWBytes + b_bytes), sf, half * 512u, &full[s]);
          if (ahead) {
            // the next unit lies in other pages: a first access there costs microseconds
            // (address translation) and the ring holds less than two
            Unit v = u;
            v.next(g);
            if (v.load(g, lists)) {
              const int64_t next = (int64_t)(v.expert * g.tiles + v.tile);
              prefetch_l2(g.w_codes + next * kRows * (g.K / 2) + v.k0 * 64);
              prefetch_l2(g.w_scales + (next * kqs + v.k0) * 512);
            }
            ahead = false;
          }
          x += 2 * kBK;
          sf += 1024;
          st += stage_bytes;
          if (++s == g.stages) {
            s = 0;
            ph ^= 1u;
            st = ring;
          }
        }
      }
    }
  } else if (warp == 6) {
    if (!UP) {
      // until the up product has ended HBM would idle: the first unit's weights beyond
      // the ring go to L2
      Unit u;
      u.begin(g);
      if (u.load(g, lists)) {
        const uint8_t* at = g.w_codes + (int64_t)(u.expert * g.tiles + u.tile) * kRows * (g.K / 2) +
                            u.k0 * 64;
        for (int r = lane; r < kRows; r += 32)
          bulk_prefetch_l2(at + (int64_t)r * (g.K / 2), (uint32_t)u.nk * 64u);
      }
      // sorted by expert: sixteen rows a copy
      grid_dep_wait();
      if (elect_one()) {
        uint32_t st = ring + 2u * kWBytes, ph = 1;
        int s = 0;
        bool ok = true;
        for (; ok && u.load(g, lists); u.next(g)) {
          const uint8_t* sf = g.h_scales + ((int64_t)u.a * kqs + u.k0) * 512;
          const uint32_t copies = (uint32_t)(u.n + 7) / 8;
          int x = u.k0 * kBK;
          for (int k = u.nk; k > 0; k -= 2) {
            ok = mbar_wait_lazy(&empty[s], ph, &abort_flag, g.status, kDevTimeoutEmpty);
            if (!ok) break;
            const uint32_t half = k > 1 ? 2u : 1u;
            mbar_arrive_expect_tx(&full[s], half * (copies * 2048u + 512u));
            for (uint32_t q = 0; q < copies; ++q) {
              load_2d(st + q * 2048u, &tmB, &full[s], x, 2 * u.off + (int)q * 16);
              if (k > 1)
                load_2d(st + b_bytes + q * 2048u, &tmB, &full[s], x + kBK, 2 * u.off + (int)q * 16);
            }
            load_bulk(st + 2u * b_bytes + 1024u, sf, half * 512u, &full[s]);
            x += 2 * kBK;
            sf += 1024;
            st += stage_bytes;
            if (++s == g.stages) {
              s = 0;
              ph ^= 1u;
              st = ring + 2u * kWBytes;
            }
          }
        }
      }
    } else {
      // tokens lie in order of the batch; 16 lanes copy the 256 bytes of each of a
      // token's two rows, 16 bytes a lane, to where the 128-byte swizzle has them
      const int r = lane >> 4, c = lane & 15;
      const uint8_t* src = g.xq + (size_t)r * g.K + c * 16;
      const uint32_t to = (c >> 3) * b_bytes + (uint32_t)r * 128u;
      uint32_t st = ring + 2u * kWBytes, ph = 1;
      int s = 0;
      bool ok = true;
      Unit u;
      for (u.begin(g); ok && u.load(g, lists); u.next(g)) {
        const int row0 = lane < u.n ? lists.token[u.off + lane] * 2 * g.K : 0;
        const int row1 = lane + 32 < u.n ? lists.token[u.off + lane + 32] * 2 * g.K : 0;
        int x = u.k0 * kBK;
        for (int k = u.nk; k > 0; k -= 2) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_lazy(&empty[s], ph, &abort_flag, g.status,
                                                      kDevTimeoutEmpty));
          if (!ok) break;
          uint32_t dst = st + to;
#pragma unroll 4
          for (int j = 0; j < u.n; ++j) {
            const int row = __shfl_sync(0xFFFFFFFFu, j < 32 ? row0 : row1, j & 31);
            if (k > 1 || c < 8)
              copy_async16(dst + (uint32_t)(((c & 7) ^ ((2 * j + r) & 7)) << 4), src + row + x);
            dst += 256u;
          }
          copy_async_arrive(&full[s]);
          x += 2 * kBK;
          st += stage_bytes;
          if (++s == g.stages) {
            s = 0;
            ph ^= 1u;
            st = ring + 2u * kWBytes;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t b_off = 2u * kWBytes >> 4, f_off = 2u * (kWBytes + b_bytes) >> 4;
      uint32_t st = ring >> 4, ph = 0, cols = tmem + kSfCol;
      int s = 0, local = 0;
      bool ok = true;
      if (UP) mx4::copy_scales(tmem + kConstCol, mx4::scale_desc_lo(smem_u32(const_sf)));
      Unit u;
      for (u.begin(g); ok && u.load(g, lists); u.next(g), ++local) {
        const int buf = local & 1;
        if (!mbar_wait_lazy(&acc_empty[buf], ((uint32_t)(local >> 1) & 1u) ^ 1u, &abort_flag,
                            g.status, kDevTimeoutMma))
          break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)buf * 128u;
        const uint32_t idesc = mx4::idesc_mxf4_f8(128, (uint32_t)(u.n + 7) / 8 * 16, 0);
        for (int k = u.nk; k > 0; k -= 2) {
          ok = mbar_wait_lazy(&full[s], ph, &abort_flag, g.status, kDevTimeoutFull);
          if (!ok) break;
          tc_fence_after();
          if (UP) fence_proxy_async_smem();   // the tokens' rows came by ordinary copies
          const uint32_t w = mx4::code_desc_lo(st << 4), b = w + b_off;
          const uint32_t w1 = w + (kWBytes >> 4), b1 = b + (b_bytes >> 4);
          const uint32_t f = mx4::scale_desc_lo((st + f_off) << 4);
          const uint32_t sfb = UP ? tmem + kConstCol : cols + 8u, sfb1 = UP ? sfb : sfb + 4u;
          mx4::copy_scales(cols, f);
          if (!UP) mx4::copy_scales(sfb, f + 64u);
          if (k > 1) {
            mx4::copy_scales(cols + 4u, f + 32u);
            if (!UP) mx4::copy_scales(sfb1, f + 96u);
          }
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j)
            mx4::mma_mxf8f6f4(d, mx4::code_desc(w + 2u * j), mx4::code_desc(b + 2u * j),
                              idesc | (j << 4) | (j << 29), cols, sfb,
                              (k < u.nk || j > 0) ? 1u : 0u);
          if (k > 1) {
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              mx4::mma_mxf8f6f4(d, mx4::code_desc(w1 + 2u * j), mx4::code_desc(b1 + 2u * j),
                                idesc | (j << 4) | (j << 29), cols + 4u, sfb1, 1);
          }
          mma_commit(&empty[s]);
          st += stage_bytes >> 4;
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
    const int width = g.tiles * kRows;
    int local = 0;
    Unit u;
    for (u.begin(g); u.load(g, lists); u.next(g), ++local) {
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
#pragma unroll 1
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
          bar_sync(1, 128);
          if (et == 0)
            ready = arrive_gpu(&g.counters[u.a * g.tiles + u.tile]) == g.splits - 1;
          bar_sync(1, 128);
          last = ready != 0;
        }
        if (last) {
#pragma unroll 1
          for (int j0 = 0; j0 < u.n; j0 += 8) {
            if (g.splits == 1) {
              float v[8];
              read8(j0, v);
#pragma unroll
              for (int j = 0; j < 8; ++j) stage_v[j][row] = v[j];
              bar_sync(1, 128);
            }
            // 16 lanes a token, four values of h (eight rows) a lane
            const int j = j0 + et / 16, q = et & 15;
            const bool mine = j < u.n;
            float4 p0 = make_float4(0, 0, 0, 0), p1 = p0;
            if (mine) {
              if (g.splits == 1) {
                p0 = *reinterpret_cast<const float4*>(&stage_v[et / 16][q * 8]);
                p1 = *reinterpret_cast<const float4*>(&stage_v[et / 16][q * 8 + 4]);
              } else {
                const float* at = g.part + (size_t)(u.off + j) * width + u.tile * kRows + q * 8;
                for (int p = 0; p < g.splits; ++p) {
                  const float4 a = __ldcg(reinterpret_cast<const float4*>(at));
                  const float4 b = __ldcg(reinterpret_cast<const float4*>(at + 4));
                  p0.x += a.x; p0.y += a.y; p0.z += a.z; p0.w += a.w;
                  p1.x += b.x; p1.y += b.y; p1.z += b.z; p1.w += b.w;
                  at += (size_t)slots * width;
                }
              }
            }
            const float x = mine ? token_scale[lists.token[u.off + j]] : 0.0f;
            const float gate[4] = {p0.x * x, p0.z * x, p1.x * x, p1.z * x};
            const float up[4] = {p0.y * x, p0.w * x, p1.y * x, p1.w * x};
            float h[4];
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              h[e] = gate[e] / (1.0f + __expf(-gate[e])) * up[e];
              m = max(m, __float_as_uint(h[e]) & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const uint32_t byte = pair_byte(m);
            const float inv = byte == 255u ? 0.0f : mx4::inv_scale(byte);
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t p = byte == 255u ? 0u : to_pair(h[e] * inv);
              hi |= (p & 0xFFu) << (8 * e);
              lo |= (p >> 8) << (8 * e);
            }
            if (mine) {
              uint8_t* out = g.hq + (size_t)(2 * (u.off + j)) * g.I + u.tile * 64 + q * 4;
              *reinterpret_cast<uint32_t*>(out) = hi;
              *reinterpret_cast<uint32_t*>(out + g.I) = lo;
              if (q < 2) {
                // scale bytes of the hi and the lo row, both blocks of 32 of this tile
                const int r = 2 * j + q, at = u.tile * 64;
                const uint32_t by = q && byte != 255u ? byte - 4u : byte;
                *reinterpret_cast<uint16_t*>(
                    g.h_scales + ((int64_t)u.a * (g.I / 128) + at / 128) * 512 + (r & 31) * 16 +
                    (r >> 5) * 4 + (at & 127) / 32) = (uint16_t)(by | by << 8);
              }
            }
            if (g.splits == 1) bar_sync(1, 128);   // stage_v is free again
          }
        }
        if (g.splits == 1) release();
      } else {
#pragma unroll 1
        for (int j0 = 0; j0 < u.n; j0 += 8) {
          float v[8];
          read8(j0, v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j0 + j < u.n) {
              const int slot = lists.slot[u.off + j0 + j];
              g.part[((size_t)u.part * slots + slot) * width + u.tile * kRows + row] =
                  v[j] * __ldg(&g.probs[slot]);
            }
        }
        release();
      }
      if (UP && g.splits > 1) bar_sync(1, 128);   // `ready` is free again
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
// Y[t] = sum of the slots' shares, by K part and then by choice; four columns a thread.
__global__ void __launch_bounds__(128)
    k_moe_combine(const float* __restrict__ part, int topk, int splits, int slots, int H,
                  uint16_t* __restrict__ Y) {
  const int col = ((int)blockIdx.x * 128 + (int)threadIdx.x) * 4, t = blockIdx.y;
  grid_dep_wait();
  if (col >= H) return;
  float4 y = make_float4(0, 0, 0, 0);
  const float* at = part + (size_t)t * topk * H + col;
  for (int p = 0; p < splits; ++p) {
#pragma unroll 8
    for (int c = 0; c < topk; ++c) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(at + (size_t)c * H));
      y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
    }
    at += (size_t)slots * H;
  }
  *reinterpret_cast<uint2*>(Y + (size_t)t * H + col) =
      make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
}

// ------------------------------------------------------------------- host ---
// K parts of a product of `tiles` row tiles of an expected number of experts: the
// rounds of units over the SMs, each as long as its share of K plus about six of the
// 128-column steps; `join` is the further cost of a split in such steps.
static int choose_splits(int64_t T, int64_t E, int topk, int64_t tiles, int64_t K, double join) {
  double miss = 1.0;
  for (int64_t t = 0; t < T; ++t) miss *= 1.0 - (double)topk / (double)E;
  const double n = (double)E * (1.0 - miss);
  const int64_t units = (int64_t)(n + 0.5 < 1.0 ? 1.0 : n + 0.5) * tiles;
  const int kq = (int)(K / kBK);
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= 8 && s <= kq; ++s) {
    const double rounds = (double)((units * s + 147) / 148);
    const double c = rounds * ((double)kq / s + 6.0) + (s > 1 ? join : 0.0);
    if (c < cost - 1e-9) {
      cost = c;
      best = s;
    }
  }
  return best;
}

struct Layout {
  size_t xq, xs, experts, probs, hq, h_scales, part_up, part_down, counters, total;
  int splits_up, splits_down, max_act, n_up;
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
  // joining the up product's parts takes five round trips to memory at the end of a unit;
  // the down product's parts are added where the choices are
  l.splits_up = choose_splits(T, E, topk, 2 * I / kRows, H, 20.0);
  l.splits_down = choose_splits(T, E, topk, H / kRows, I, 1.0);
  l.n_up = l.splits_up > 1 ? (int)(l.max_act * (2 * I / kRows)) : 0;
  l.xq = take((size_t)T * 2 * H);
  l.xs = take((size_t)T * 4);
  l.experts = take(slots * 4);
  l.probs = take(slots * 4);
  l.hq = take(slots * 2 * I);
  l.h_scales = take((size_t)l.max_act * (I / 128) * 512);
  l.part_up = take(l.splits_up > 1 ? (size_t)l.splits_up * slots * 2 * I * 4 : 0);
  l.part_down = take((size_t)l.splits_down * slots * H * 4);
  l.counters = take((size_t)l.n_up * 4);
  l.total = at;
  return l;
}

// The unit walk's constants for a grid of `grid` blocks.
static void set_units(GemmArgs* g, int grid) {
  g->per = g->tiles * g->splits;
  g->step_a = grid / g->per;
  g->step_rest = grid % g->per;
  g->by_splits = (65536 + g->splits - 1) / g->splits;
  g->by_topk = (65536 + g->topk - 1) / g->topk;
  g->by_per = (65536 + g->per - 1) / g->per;
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
  float* xs = reinterpret_cast<float*>(w + l.xs);
  int* counters = reinterpret_cast<int*>(w + l.counters);
  int32_t* experts = reinterpret_cast<int32_t*>(w + l.experts);
  float* probs = reinterpret_cast<float*>(w + l.probs);

  CUtensorMap tw13, tw2, th;
  if (!weights_map(&tw13, a.w13_codes, (uint64_t)a.E * 2 * a.I, (uint64_t)a.H) ||
      !weights_map(&tw2, a.w2_codes, (uint64_t)a.E * a.H, (uint64_t)a.I) ||
      !make_tmap_2d(&th, w + l.hq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)slots * 2,
                    (uint64_t)a.I, 16, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_limit(k_moe_gemm<true>, kMaxDynSmem);
  if (e == cudaSuccess) e = ensure_smem_limit(k_moe_gemm<false>, kMaxDynSmem);
  if (e != cudaSuccess) return e;

  k_moe_route<<<(a.T + kRouteTokens - 1) / kRouteTokens * kRouteCtas, 256, 0, st>>>(
      a.X, a.T, a.H, a.router, a.E, a.topk, a.renorm, experts, probs, a.experts, a.probs, w + l.xq,
      xs, counters, l.n_up);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  GemmArgs g;
  g.experts = experts;
  g.probs = probs;
  g.E = a.E;
  g.xq = w + l.xq;
  g.T = a.T;
  g.topk = a.topk;
  g.b_rows = (2 * a.T + 15) / 16 * 16;
  const int stage_bytes = 2 * (kWBytes + g.b_rows * kBK + 1024);
  g.stages = kRingBytes / stage_bytes < kMaxStages ? kRingBytes / stage_bytes : kMaxStages;
  g.xs = xs;
  g.hq = w + l.hq;
  g.h_scales = w + l.h_scales;
  g.I = a.I;
  g.status = a.status;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 1024 + (size_t)g.stages * stage_bytes;

  g.w_codes = a.w13_codes;
  g.w_scales = a.w13_scales;
  g.K = a.H;
  g.tiles = 2 * a.I / kRows;
  g.splits = l.splits_up;
  g.part = reinterpret_cast<float*>(w + l.part_up);
  g.counters = counters;
  int64_t units = (int64_t)l.max_act * g.tiles * g.splits;
  cfg.gridDim = dim3((unsigned)(units < sm_count ? units : sm_count));
  set_units(&g, (int)cfg.gridDim.x);
  e = cudaLaunchKernelEx(&cfg, k_moe_gemm<true>, tw13, th, g);
  if (e != cudaSuccess) return e;

  g.w_codes = a.w2_codes;
  g.w_scales = a.w2_scales;
  g.K = a.I;
  g.tiles = a.H / kRows;
  g.splits = l.splits_down;
  g.part = reinterpret_cast<float*>(w + l.part_down);
  units = (int64_t)l.max_act * g.tiles * g.splits;
  cfg.gridDim = dim3((unsigned)(units < sm_count ? units : sm_count));
  set_units(&g, (int)cfg.gridDim.x);
  e = cudaLaunchKernelEx(&cfg, k_moe_gemm<false>, tw2, th, g);
  if (e != cudaSuccess) return e;

  cfg.gridDim = dim3((unsigned)((a.H + 511) / 512), (unsigned)a.T);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, k_moe_combine, (const float*)g.part, a.topk, g.splits, slots, a.H,
                         a.Y);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace e8
