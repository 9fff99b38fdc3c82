// Mixture-of-experts layer for a few tokens, experts in the microscaled 4-bit
// form.  Bound by the bytes of the chosen experts' weights (17/32 a value), and with
// one token by the latency of the steps between them; two launches.
//
//   k_moe_route   router logits (products exact in fp32 and summed in fp64), top-k and
//                 probabilities, and the activations as two e4m3 rows a token
//   k_moe_experts everything else, one block an SM: the up products' units, the down
//                 products', the weighted sums, claimed in this order from one counter
//                 by the blocks as they go.  A block waits only for units with lower
//                 numbers, which running blocks have claimed, so the launch needs no
//                 co-residence and no end of a phase leaves blocks idle; the ring of
//                 weight tiles runs through all of it, so HBM is busy while a block
//                 waits for the activations of its next product (as three kernels, the
//                 starts and ends of each cost 15 us together).
//     The tensor cores take the 4-bit weights as they are (tcgen05.mma.kind::mxf8f6f4,
//     e2m1 x e4m3): 128 rows of an expert's matrix on the M side, its tokens on the N
//     side.  The activations enter as hi + lo, hi = e4m3(x / s), lo = e4m3(16 (x / s -
//     hi)): four significant bits each.  amax / s lies in [2^7, 2^8) and lo's least step
//     is 2^-13 s, the last place of a bf16 value of 2^-6 s: values down to 2^-13 of the
//     row's largest are held exactly, smaller ones within 2^-14 s, 2^-21 of the largest.
//     A dequantised operand would cost about one instruction a weight, which alone
//     exceeds the time HBM needs to deliver it.
//     up          gate and up rows alternate, so a tile holds both factors of 64 values
//                 of h = silu(g) u; the epilogue writes h as two e4m3 rows again, with
//                 a power-of-two scale for the tile's 64 values: within 2^-9 of each (a
//                 bf16 h: 2^-8) down to 2^-12 of the largest.  (Three rows would hold 2^-13,
//                 for half as many bytes of activations again; an output's error against
//                 64 bits is 0.0018 of it in the norm, 0.0017 the rounding of Y alone.)
//     down        every slot's product times its probability goes to a buffer
//     sums        a token's slots are added in the order of its choices
// Few up units are split over K, their partial sums added in order by the unit that
// arrives last; the down units' parts are added with the slots.  No result depends on
// timing or on which block claimed what.
// 64 tokens, 8 of 128 experts (2048, 768): 80 us for 317 MB, 6.2 TB/s in the up products and
// 4.8 in the down products; 1 token, 8 of 64 (2048, 1024): 24 us, of which the router 5,
// the way to the first products 4, h to the other blocks 4, the sums 5.
#include "e8_internal.h"
#include "e8_mx4.cuh"
#include "e8_tmap.h"

namespace e8 {
namespace moe {

constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTopk = 16;
constexpr int kMaxSlots = kMaxTokens * kMaxTopk;

// Scale byte of an e4m3 pair for values of magnitude up to amax: amax / s lies in
// [128, 256), well inside e4m3's 448; lo's scale is 2^-4 of it, hence the least byte 4, for
// amax below 2^-116 (a bf16 value is then a multiple of 2^-133 = 2^-10 s and still exact).
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
constexpr int kRouteCtas = 8;

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

// One cluster of 8 CTAs for NT tokens (4; 1 for small batches, whose time is latency):
// each CTA takes an eighth of the experts, its warps 4 experts x NT tokens of a part of H
// each (4 NT fp64 sums a lane; converting bf16 to fp64 costs four times an fp64 product,
// so converted values are used several times).  A step's loads are under way while the
// step before is computed.  The logits of token j go to CTA j, which chooses; CTAs 4..7
// write the tokens' e4m3 rows meanwhile.  One launch and no counters: the logits cross
// CTAs in distributed shared memory.
template <int NT>
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
  const int rank = (int)cluster_ctarank(), t0 = (int)blockIdx.x / kRouteCtas * NT;
  const int nt = min(NT, T - t0);
  grid_dep_launch();
  cluster_arrive();   // (the wait below: every CTA of the cluster has started)
  const int per = (E + kRouteCtas - 1) / kRouteCtas, e0 = rank * per;
  const int ne = min(per, E - e0), groups = ne > 0 ? (ne + 3) / 4 : 0;
  const int parts = groups > 0 && groups < 8 ? 8 / groups : 1, chunks = (H + 255) / 256;
  for (int item = warp; item < groups * parts; item += 8) {
    const int e = e0 + item / parts * 4, p = item % parts;
    const int end = chunks * (p + 1) / parts;
    double acc[4 * NT] = {};
    uint4 r[4], x[NT];
    auto load = [&](int c) {
      const int k = c * 256 + lane * 8;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        r[j] = k < H && e + j < e0 + ne
                   ? *reinterpret_cast<const uint4*>(R + (size_t)(e + j) * H + k)
                   : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        x[j] = k < H && j < nt ? *reinterpret_cast<const uint4*>(X + (size_t)(t0 + j) * H + k)
                               : make_uint4(0, 0, 0, 0);
    };
    int c = chunks * p / parts;
    if (c < end) load(c);
#pragma unroll 2
    for (; c < end; ++c) {
      uint4 rn[4], xn[NT];
#pragma unroll
      for (int j = 0; j < 4; ++j) rn[j] = r[j];
#pragma unroll
      for (int j = 0; j < NT; ++j) xn[j] = x[j];
      if (c + 1 < end) load(c + 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        double rd[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = i < 2 ? rn[j].x : i < 4 ? rn[j].y : i < 6 ? rn[j].z : rn[j].w;
          rd[j] = (double)((i & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w));
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t w = i < 2 ? xn[j].x : i < 4 ? xn[j].y : i < 6 ? xn[j].z : xn[j].w;
          const double xd = (double)((i & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w));
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q * NT + j] = fma(rd[q], xd, acc[q * NT + j]);
        }
      }
    }
    if constexpr (NT == 4) {
      const double s = warp_sum16(acc, lane);
      if (!(lane & 1)) part[item][lane >> 1] = s;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        for (int o = 16; o; o >>= 1) acc[q] += __shfl_xor_sync(0xFFFFFFFFu, acc[q], o);
        if (lane == 0) part[item][q] = acc[q];
      }
    }
  }
  for (int i = blockIdx.x * 256 + tid; i < n_counters; i += gridDim.x * 256) counters[i] = 0;
  __syncthreads();
  cluster_wait();
  if (tid < ne * NT) {
    const int el = tid / NT, j = tid % NT;
    double s = 0.0;
    for (int p = 0; p < parts; ++p) s += part[el / 4 * parts + p][(el & 3) * NT + j];
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(
                     mapa_shared(smem_u32(&logit[e0 + el]), (uint32_t)j)),
                 "d"(s)
                 : "memory");
  }
  __syncwarp();
  cluster_arrive();
  if (rank >= 4 && rank - 4 < nt) {
    // hi and lo rows of one token
    const int t = t0 + rank - 4;
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
  // before it (larger logit, or the same and a lower number; NaN comes last); `ways`
  // neighbouring threads share an expert's comparisons
  const int t = t0 + rank;
  for (int e = tid; e < E; e += 256) {
    const double v = logit[e] + 0.0;   // -0 becomes 0
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    key[e] = v != v ? 0ull : (u >> 63 ? ~u : u | (1ull << 63));
  }
  __syncthreads();
  const int ways = E <= 32 ? 8 : E <= 64 ? 4 : E <= 128 ? 2 : 1;
  for (int i = tid; i < (E * ways + 31) / 32 * 32; i += 256) {
    const int e = i / ways, w = i & (ways - 1);
    const uint64_t mine = e < E ? key[e] : 0ull;
    int place = 0;
#pragma unroll 8
    for (int j = w; j < E; j += ways) place += key[j] > mine || (key[j] == mine && j < e);
    for (int o = 1; o < ways; o <<= 1) place += __shfl_xor_sync(0xFFFFFFFFu, place, o);
    if (w == 0 && e < E && place < topk) chosen[place] = e;
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

// ----------------------------------------------------------------- experts ---
constexpr int kThreads = 320;
constexpr int kSlots = 4;                  // claimed units a block has in hand
constexpr int kRows = 128;                 // rows of a unit
constexpr int kBK = 128;                   // columns of a step: a tile of scales
constexpr int kWBytes = kRows * kBK;       // 16 values in 16 bytes, 8 of them used
constexpr int kMaxStages = 5;              // of two steps: one barrier round for 16 KB of weights
constexpr int kConstCol = 256, kSfCol = 264;   // tensor-memory columns of the scales
constexpr int kRingBytes = 212 * 1024;     // at least three stages, and one block an SM
constexpr int kMaxGrid = 160;              // blocks
constexpr int kMaxUpParts = 8, kMaxDownParts = 16;   // K parts of a unit

struct ExpertArgs {
  const int32_t* experts;  // by slot = token * topk + choice
  const float* probs;
  const uint8_t *w13_codes, *w13_scales, *w2_codes, *w2_scales;
  int T, E, topk, by_topk, H, I;   // by_topk = ceil(2^16 / topk): a slot's token without a divide
  int down_parts;
  const uint8_t* xq;       // the tokens' hi and lo rows
  const float* xs;         // scale of each token's pair
  uint8_t* hq;             // the slots' hi and lo rows of h, sorted by expert
  uint8_t* h_scales;       // [active expert][I / 128][512]
  float* part_up;          // [split up unit * parts + part][T][128]
  float* part_down;        // [part][slot][H]
  int* claimed;            // units so far
  int* up_done;            // [active expert]: finished up units
  int* up_total;           // finished up units of all
  int* up_joined;          // [split up unit]: arrived parts
  int* down_done;          // [tile]: finished units
  uint16_t* Y;
  uint32_t* status;
};

__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// One thread tells (or counts) for its block after a barrier that the others' writes
// came before.
__device__ __forceinline__ void fence_gpu() {
  asm volatile("fence.acq_rel.gpu;" ::: "memory");
}
__device__ __forceinline__ void add_gpu(int* counter) {
  asm volatile("red.relaxed.gpu.global.add.s32 [%0], 1;" ::"l"(counter) : "memory");
}
__device__ __forceinline__ int arrive_gpu(int* counter) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}
__device__ __forceinline__ int ld_acquire_gpu(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Waits until *counter has reached `want`; bounded as mbar_wait_lazy is.
__device__ __forceinline__ bool wait_gpu(const int* counter, int want,
                                         volatile uint32_t* abort_flag, uint32_t* status) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire_gpu(counter) >= want) return true;
    if ((it & 31u) == 0) {
      if (ld_shared_volatile(abort_flag)) return false;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (ns_between(t0, t) > kWaitLimitNs) {
        st_shared_volatile(abort_flag, 1u);
        if (status) atomicOr(status, kDevTimeoutCluster);
        return false;
      }
    }
  }
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
  int nact;
  uint32_t most;   // tokens of the fullest expert
  uint32_t wsum[kThreads / 32];
};
static_assert(kMaxTokens == 64, "a token is a bit of an expert's mask");

// Builds the lists of up to 32 slots (one warp, a lane a slot).
__device__ __forceinline__ void build_small(SharedLists& l, const int32_t* __restrict__ experts,
                                            int slots, int by_topk) {
  const int lane = threadIdx.x & 31;
  const int e = lane < slots ? experts[lane] : INT32_MAX;
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, e), lower = (1u << lane) - 1u;
  const bool head = (same & lower) == 0 && lane < slots;
  // slots and active experts before this one's
  int pos = __popc(same & lower), act = 0;
#pragma unroll 1
  for (int j = 0; j < slots; ++j) {
    const int other = __shfl_sync(0xFFFFFFFFu, head ? e : e | (1 << 30), j);
    pos += (other & ~(1 << 30)) < e;
    act += other < e;
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
  const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, lane < slots ? __popc(same) : 0);
  if (lane == 0) {
    l.off[nact] = (int16_t)slots;
    l.nact = nact;
    l.most = most;
  }
}

// Builds the lists (all threads; l.most 0 on entry).  mask[e]: the tokens that chose expert e, zero on
// entry; a token chooses an expert once, so its place is the number of lower bits.
// chosen: the expert of each slot; first: slots before an expert's.
__device__ __forceinline__ void build_lists(SharedLists& l, unsigned long long* mask,
                                            int16_t* chosen, int16_t* first,
                                            const int32_t* __restrict__ experts, int slots, int E,
                                            int by_topk) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll
  for (int i = 0; i < (kMaxSlots + kThreads - 1) / kThreads; ++i) {
    const int s = tid + i * kThreads;
    if (s < slots) {
      const int e = experts[s], t = s * by_topk >> 16;
      chosen[s] = (int16_t)e;
      atomicOr(reinterpret_cast<uint32_t*>(mask + e) + (t >> 5), 1u << (t & 31));
    }
  }
  __syncthreads();
  // a scan over experts of (is active, slots) in one word
  constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
  uint32_t mine = 0, n[kPer], most = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    n[i] = e < E ? (uint32_t)__popcll(mask[e]) : 0u;
    mine += n[i] ? (1u << 16) | n[i] : 0u;
    most = max(most, n[i]);
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) atomicMax(&l.most, most);
  uint32_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) l.wsum[warp] = scan;
  __syncthreads();
  uint32_t at = scan - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) at += l.wsum[w];
    total += l.wsum[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (n[i]) {
      first[e] = (int16_t)(at & 0xFFFFu);
      l.expert[at >> 16] = (int16_t)e;
      l.off[at >> 16] = (int16_t)(at & 0xFFFFu);
      at += (1u << 16) | n[i];
    }
  }
  if (tid == 0) {
    l.nact = (int)(total >> 16);
    l.off[total >> 16] = (int16_t)slots;
  }
  __syncthreads();
  for (int s = tid; s < slots; s += kThreads) {
    const int t = s * by_topk >> 16, e = chosen[s];
    const int pos = first[e] + __popcll(mask[e] & ((1ull << t) - 1ull));
    l.slot[pos] = (int16_t)s;
    l.token[pos] = (uint8_t)t;
  }
  fence_proxy_async_smem();   // the scratch space becomes the copies' ring
  __syncthreads();
}

// A unit as the scheduler warp writes it down for the others.  The numbers run over the
// up products (row tiles of an expert, then the next expert's), the down products (each
// tile in parts of K), and the sums (128 columns of four tokens).  The up units that
// fill no whole round of the blocks are split over K between them and come first, so
// that the joining of their parts is over long before the down products ask for it.
enum : int { kUp = 0, kDown = 1, kSum = 2, kEnd = 3 };
struct Unit {
  int kind;
  int active, tile, part, parts;   // active expert; row tile; part of K
  int expert, off, n;              // n tokens from slot[off] on
  int k0, nk;                      // 128-column steps of K
  int joined;                      // number of a split up unit
  int want, want_all;              // up units, parts counted, of this expert and of all
};

// Warps: 0 weights producer, 6 and 7 activations producers, 1 MMAs, 2..5 epilogue, 8
// scheduler, 9 tells other blocks of finished units (a release to the whole GPU takes a
// microsecond or two under load, which the epilogue does not wait for).  At 16 KB of
// weights a stage the SM's share of HBM leaves each role some 700 cycles a stage: one
// elected thread runs a role's whole loop with its addresses in registers, and what a whole
// warp waits for all its lanes poll (64 tokens 80 us; with branches on lane 0 instead of
// elected threads 81.6, with polls by lane 0 87.8).
__global__ void __launch_bounds__(kThreads, 1)
    k_moe_experts(const __grid_constant__ CUtensorMap tm13, const __grid_constant__ CUtensorMap tm2,
                  const __grid_constant__ ExpertArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ __align__(16) uint8_t const_sf[512];
  __shared__ __align__(16) float stage_v[8][128 + 4];
  __shared__ int ready;
  __shared__ float token_scale[kMaxTokens];
  __shared__ SharedLists lists;
  __shared__ Unit units[kSlots];
  __shared__ uint64_t unit_full[kSlots], unit_empty[kSlots], told_full[2], told_empty[2];
  __shared__ uint64_t weights_took[2];   // units by parity: two may be taken between looks
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    lists.most = 0;
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 33);   // the weights' producer, and the lanes of the other
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_empty[i], 9);   // three threads and six warps read it
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&told_full[i], 4);
      mbar_init(&told_empty[i], 1);
    }
    mbar_init(&weights_took[0], 1);
    mbar_init(&weights_took[1], 1);
    mbar_init(&drain, 1);
    abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tm13);
    tma_prefetch_desc(&tm2);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  if (threadIdx.x >= 64 && threadIdx.x < 192) {
    // scales of the tokens' rows: 1 for hi rows (even), 2^-4 for lo rows
    reinterpret_cast<uint32_t*>(const_sf)[threadIdx.x - 64] =
        ((threadIdx.x - 64) / 4) & 1 ? 0x7B7B7B7Bu : 0x7F7F7F7Fu;
    fence_proxy_async_smem();
  }
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(smem);
  int16_t* chosen = reinterpret_cast<int16_t*>(mask + kMaxExperts);
  // in the ring's bytes, hence only for build_lists, which fences its writes from the
  // copies that follow them there
  const int slots = g.T * g.topk;
  if (slots > 32)
    for (int i = threadIdx.x; i < g.E; i += kThreads) mask[i] = 0ull;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  grid_dep_wait();
  int claim = 0;
  if (threadIdx.x == 256) claim = atomicAdd(g.claimed, 1);
  if (threadIdx.x < g.T) token_scale[threadIdx.x] = g.xs[threadIdx.x];
  if (slots > 32)
    build_lists(lists, mask, chosen, chosen + kMaxSlots, g.experts, slots, g.E, g.by_topk);
  else if (warp == 0)
    build_small(lists, g.experts, slots, g.by_topk);
  __syncthreads();
  // a stage holds two steps: weights, the rows of the fullest expert's tokens, scales
  const uint32_t b_bytes = (2u * lists.most + 15u) / 16u * 16u * 128u;
  const uint32_t stage_bytes = 2u * (kWBytes + b_bytes + 1024u);
  const int stages = min(kMaxStages, (int)((uint32_t)kRingBytes / stage_bytes));
  const uint32_t ring = smem_u32(smem);
  const int up_tiles = 2 * g.I / kRows, down_tiles = g.H / kRows;

  // The next unit of a role that is one thread, and of one that is a warp; false when the
  // block gives up.  Every role takes all units.
  int slot_at = 0;
  uint32_t slot_ph = 0;
  auto look = [&](Unit& u) {
    const bool ok = mbar_wait_lazy(&unit_full[slot_at], slot_ph, &abort_flag, g.status,
                                   kDevTimeoutFull);
    u = units[slot_at];
    return ok;
  };
  auto taken = [&]() {
    mbar_arrive(&unit_empty[slot_at]);
  };
  auto advance = [&]() {
    if (++slot_at == kSlots) {
      slot_at = 0;
      slot_ph ^= 1u;
    }
  };
  auto take = [&](Unit& u) {
    const bool ok = look(u);
    if (ok) taken();
    advance();
    return ok && u.kind != kEnd;
  };
  auto take_warp = [&](Unit& u) {
    const bool ok = __all_sync(0xFFFFFFFFu, look(u));
    __syncwarp();
    if (ok && lane == 0) taken();
    advance();
    return ok && u.kind != kEnd;
  };

  if (warp == 9) {
    if (elect_one()) {
      Unit u;
      int i = 0;
      while (take(u)) {
        if (u.kind == kSum) continue;
        if (!mbar_wait_lazy(&told_full[i & 1], (uint32_t)(i >> 1) & 1u, &abort_flag, g.status,
                            kDevTimeoutMma))
          break;
        // the four epilogue warps' writes came before; a part of a unit counts as one of it
        fence_gpu();
        if (u.kind == kDown) {
          add_gpu(&g.down_done[u.tile]);
        } else {
          add_gpu(&g.up_done[u.active]);
          add_gpu(g.up_total);
        }
        mbar_arrive(&told_empty[i & 1]);
        ++i;
      }
    }
  } else if (warp == 8) {
    claim = __shfl_sync(0xFFFFFFFFu, claim, 0);
    if (elect_one()) {
      const int nact = lists.nact, ups = nact * up_tiles, grid = (int)gridDim.x;
      const int whole = ups / grid * grid, rest = ups - whole;
      const int up_parts = rest ? min(min(kMaxUpParts, grid / rest), g.H / kBK) : 1;
      const int n_split = rest * up_parts, n_up = n_split + whole;
      const int per_down = down_tiles * g.down_parts, n_down = n_up + nact * per_down;
      const int n_all = n_down + down_tiles * ((g.T + 3) / 4);
      int s = 0, ahead = 0;
      uint32_t ph = 1, took = 0;   // units waited for: barrier in bit 0, phase in bit 1
      for (;;) {
        Unit u = {};
        u.kind = claim < n_up ? kUp : claim < n_down ? kDown : claim < n_all ? kSum : kEnd;
        if (u.kind < kSum) {
          const bool down = u.kind == kDown;
          const int kq = (down ? g.I : g.H) / kBK;
          u.parts = 1;
          u.part = 0;
          if (down) {
            const int i = claim - n_up;
            u.active = i / per_down;
            const int at = i - u.active * per_down;
            u.parts = g.down_parts;
            u.tile = at / u.parts;
            u.part = at - u.tile * u.parts;
            // of this expert's up tiles, those that were split
            const int split = min(up_tiles, max(0, (u.active + 1) * up_tiles - whole));
            u.want = up_tiles + split * (up_parts - 1);
            u.want_all = n_up;
          } else {
            int i = claim - n_split;
            if (i < 0) {
              const int unit = claim / up_parts;
              u.parts = up_parts;
              u.part = claim - unit * up_parts;
              u.joined = unit;
              i = whole + unit;
            }
            u.active = i / up_tiles;
            u.tile = i - u.active * up_tiles;
          }
          u.expert = lists.expert[u.active];
          u.off = lists.off[u.active];
          u.n = lists.off[u.active + 1] - u.off;
          u.k0 = kq * u.part / u.parts;
          u.nk = kq * (u.part + 1) / u.parts - u.k0;
          // a first access to other pages costs microseconds (address translation), and
          // the ring holds less than two
          const int64_t tile = (int64_t)u.expert * (down ? down_tiles : up_tiles) + u.tile;
          prefetch_l2((down ? g.w2_codes : g.w13_codes) + tile * kRows * (kq * 64) + u.k0 * 64);
          prefetch_l2((down ? g.w2_scales : g.w13_scales) + (tile * kq + u.k0) * 512);
        } else if (u.kind == kSum) {
          u.active = (claim - n_down) / down_tiles;   // four tokens
          u.tile = claim - n_down - u.active * down_tiles;
        }
        if (!mbar_wait_lazy(&unit_empty[s], ph, &abort_flag, g.status, kDevTimeoutEmpty)) break;
        units[s] = u;
        mbar_arrive(&unit_full[s]);
        if (u.kind == kEnd) break;
        if (++s == kSlots) {
          s = 0;
          ph ^= 1u;
        }
        // The next one when the weights' producer begins this unit, or the one before if
        // it is short: claimed in time, and not kept from blocks that would be sooner.
        if (u.kind < kSum && u.nk <= 8 && ahead == 0) {
          ahead = 1;
        } else {
          if (!mbar_wait_lazy(&weights_took[took & 1u], took >> 1 & 1u, &abort_flag, g.status,
                              kDevTimeoutEmpty))
            break;
          ++took;
        }
        claim = atomicAdd(g.claimed, 1);
      }
    }
  } else if (warp == 0) {
    if (elect_one()) {
      uint32_t st = ring, ph = 1;
      int s = 0;
      bool ok = true;
      Unit u;
      for (uint32_t i = 0; ok && take(u); ++i) {
        mbar_arrive(&weights_took[i & 1u]);
        if (u.kind == kSum) continue;
        const bool down = u.kind == kDown;
        const int kqs = (down ? g.I : g.H) / kBK;
        const int row = (u.expert * (down ? down_tiles : up_tiles) + u.tile) * kRows;
        const uint8_t* sf =
            (down ? g.w2_scales : g.w13_scales) + ((int64_t)(row >> 7) * kqs + u.k0) * 512;
        const CUtensorMap* map = down ? &tm2 : &tm13;
        int x = u.k0 * kBK;
        for (int k = u.nk; k > 0; k -= 2) {
          ok = mbar_wait_lazy(&empty[s], ph, &abort_flag, g.status, kDevTimeoutEmpty);
          if (!ok) break;
          // the tensor map unpacks: its bytes are counted as they lie in memory
          const uint32_t half = k > 1 ? 2u : 1u;
          mbar_arrive_expect_tx(&full[s], half * (kWBytes / 2 + 512u));
          load_2d(st, map, &full[s], x, row);
          if (k > 1) load_2d(st + kWBytes, map, &full[s], x + kBK, row);
          load_bulk(st + 2u * (kWBytes + b_bytes), sf, half * 512u, &full[s]);
          x += 2 * kBK;
          sf += 1024;
          st += stage_bytes;
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
            st = ring;
          }
        }
      }
    }
  } else if (warp >= 6) {
    // The two warps take turns, a stage each.  16 lanes copy the 256 bytes of each of a
    // token's two rows, 16 bytes a lane, to where the 128-byte swizzle has them
    const int r = lane >> 4, c = lane & 15;
    const uint32_t to = (c >> 3) * b_bytes + (uint32_t)r * 128u;
    uint32_t st = ring + 2u * kWBytes, ph = 1;
    int s = 0, turn = warp & 1;
    bool ok = true, all_up = false;
    Unit u;
    while (ok && take_warp(u)) {
      if (u.kind == kSum) continue;
      const bool down = u.kind == kDown;
      const int cols = down ? g.I : g.H;
      const uint8_t* src = (down ? g.hq + (size_t)u.off * 2 * g.I : g.xq) + (size_t)r * cols + c * 16;
      const int row0 = (down ? lane : lane < u.n ? lists.token[u.off + lane] : 0) * 2 * cols;
      const int row1 =
          (down ? lane + 32 : lane + 32 < u.n ? lists.token[u.off + lane + 32] : 0) * 2 * cols;
      const uint8_t* sf = g.h_scales + ((int64_t)u.active * (g.I / kBK) + u.k0) * 512 + lane * 16;
      if (down) {
        // every tile of the expert's h; once all experts' are there nothing is asked again
        if (!all_up) {
          all_up = ld_acquire_gpu(g.up_total) == u.want_all;
          ok = all_up || wait_gpu(&g.up_done[u.active], u.want, &abort_flag, g.status);
          all_up = __all_sync(0xFFFFFFFFu, all_up);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
        }
      }
      int x = u.k0 * kBK;
      for (int k = u.nk; k > 0; k -= 2, turn ^= 1) {
        if (turn == 0) {
          ok = __all_sync(0xFFFFFFFFu,
                          mbar_wait_lazy(&empty[s], ph, &abort_flag, g.status, kDevTimeoutEmpty));
          if (!ok) break;
          uint32_t dst = st + to;
#pragma unroll 4
          for (int j = 0; j < u.n; ++j) {
            const int row = __shfl_sync(0xFFFFFFFFu, j < 32 ? row0 : row1, j & 31);
            if (k > 1 || c < 8)
              copy_async16(dst + (uint32_t)(((c & 7) ^ ((2 * j + r) & 7)) << 4), src + row + x);
            dst += 256u;
          }
          if (down) {
            const uint32_t f = st + 2u * b_bytes + 1024u + (uint32_t)lane * 16u;
            copy_async16(f, sf);
            if (k > 1) copy_async16(f + 512u, sf + 512);
          }
          copy_async_arrive(&full[s]);
        }
        x += 2 * kBK;
        sf += 1024;
        st += stage_bytes;
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
          st = ring + 2u * kWBytes;
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t b_off = 2u * kWBytes >> 4, f_off = 2u * (kWBytes + b_bytes) >> 4;
      uint32_t st = ring >> 4, ph = 0, cols = tmem + kSfCol;
      int s = 0, local = 0;
      bool ok = true;
      mx4::copy_scales(tmem + kConstCol, mx4::scale_desc_lo(smem_u32(const_sf)));
      Unit u;
      while (ok && take(u)) {
        if (u.kind == kSum) continue;
        const bool down = u.kind == kDown;
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
          fence_proxy_async_smem();   // the activations came by ordinary copies
          const uint32_t w = mx4::code_desc_lo(st << 4), b = w + b_off;
          const uint32_t w1 = w + (kWBytes >> 4), b1 = b + (b_bytes >> 4);
          const uint32_t f = mx4::scale_desc_lo((st + f_off) << 4);
          const uint32_t sfb = down ? cols + 8u : tmem + kConstCol, sfb1 = down ? sfb + 4u : sfb;
          mx4::copy_scales(cols, f);
          if (down) mx4::copy_scales(sfb, f + 64u);
          if (k > 1) {
            mx4::copy_scales(cols + 4u, f + 32u);
            if (down) mx4::copy_scales(sfb1, f + 96u);
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
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
            st = ring >> 4;
            cols = tmem + kSfCol;
          }
        }
        if (ok) mma_commit(&acc_full[buf]);
        ++local;
      }
      // every MMA of this thread has finished once `drain` flips
      mma_commit(&drain);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&drain, 0) && ns_since(t0) < 200000000ull) {
      }
    }
  } else {
    const int quarter = warp & 3, row = quarter * 32 + lane, et = (int)threadIdx.x - 64;
    int local = 0;
    Unit u = {};
    u.parts = 1;
    // The first two passes are rehearsals without tokens, of an up and of a down unit:
    // their instructions come from memory while the first products are under way, and not
    // when their sums are waited for.
    for (int pass = 0;; ++pass) {
      const bool live = pass > 1;
      uint32_t d = tmem + ((uint32_t)(quarter * 32) << 16);
      u.kind = pass == 1 ? kDown : kUp;
      if (live) {
        const bool got = take_warp(u);
        if (bar_red_or(1, 128, !got)) break;
        if (u.kind == kSum) {
          // Y: 128 columns of four tokens, a warp a token, four columns a lane
          const bool ok = wait_gpu(&g.down_done[u.tile], lists.nact * g.down_parts,
                                              &abort_flag, g.status);
          __syncwarp();
          if (bar_red_or(1, 128, !ok)) break;
          const int t = u.active * 4 + quarter;
          if (t < g.T) {
            const int col = u.tile * kRows + lane * 4;
            const float* at = g.part_down + (size_t)t * g.topk * g.H + col;
            float4 y = make_float4(0, 0, 0, 0);
            // (eight loads under way at a time, added in the order of parts and choices)
            const int terms = g.down_parts * g.topk;
            int c = 0;
            for (int i = 0; i < terms; i += 8) {
              float4 v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                v[k] = i + k < terms ? __ldcg(reinterpret_cast<const float4*>(at))
                                     : make_float4(0, 0, 0, 0);
                const bool wrap = ++c == g.topk;
                at += (size_t)(wrap ? slots - g.topk + 1 : 1) * g.H;
                if (wrap) c = 0;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                y.x += v[k].x; y.y += v[k].y; y.z += v[k].z; y.w += v[k].w;
              }
            }
            *reinterpret_cast<uint2*>(g.Y + (size_t)t * g.H + col) =
                make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
          }
          continue;
        }
        const int buf = local & 1;
        const bool ok = mbar_wait_lazy(&acc_full[buf], (uint32_t)(local >> 1) & 1u, &abort_flag,
                                       g.status, kDevTimeoutMma);
        __syncwarp();
        if (bar_red_or(1, 128, !ok)) break;
        tc_fence_after();
        d += (uint32_t)buf * 128u;
      }
      const int parts = u.parts, n = u.n;
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
        if (live && lane == 0) mbar_arrive(&acc_empty[local & 1]);
      };
      if (u.kind == kUp) {
        float* part = g.part_up + (size_t)u.joined * parts * g.T * kRows;
        bool last = true;
        if (parts > 1) {
#pragma unroll 1
          for (int j0 = 0; j0 < n; j0 += 8) {
            float v[8];
            read8(j0, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j0 + j < n) part[((size_t)u.part * g.T + j0 + j) * kRows + row] = v[j];
          }
          bar_sync(1, 128);
          if (et == 0) ready = arrive_gpu(&g.up_joined[u.joined]) == parts - 1;
          bar_sync(1, 128);
          last = ready != 0;
        }
        if (last) {
          int j0 = 0;
#pragma unroll 1
          do {
            if (parts == 1) {
              float v[8];
              read8(j0, v);
#pragma unroll
              for (int j = 0; j < 8; ++j) stage_v[j][row] = v[j];
              bar_sync(1, 128);
            }
            // 16 lanes a token, four values of h (eight rows) a lane
            const int j = j0 + et / 16, q = et & 15;
            const bool mine = j < n;
            float4 p0 = make_float4(0, 0, 0, 0), p1 = p0;
            if (parts == 1) {
              p0 = *reinterpret_cast<const float4*>(&stage_v[et / 16][q * 8]);
              p1 = *reinterpret_cast<const float4*>(&stage_v[et / 16][q * 8 + 4]);
            } else if (mine) {
              const float* at = part + (size_t)j * kRows + q * 8;
              float4 a[kMaxUpParts], b[kMaxUpParts];
#pragma unroll
              for (int p = 0; p < kMaxUpParts; ++p) {
                const bool in = p < parts;
                a[p] = in ? __ldcg(reinterpret_cast<const float4*>(at)) : make_float4(0, 0, 0, 0);
                b[p] = in ? __ldcg(reinterpret_cast<const float4*>(at + 4))
                          : make_float4(0, 0, 0, 0);
                at += (size_t)g.T * kRows;
              }
#pragma unroll
              for (int p = 0; p < kMaxUpParts; ++p) {
                p0.x += a[p].x; p0.y += a[p].y; p0.z += a[p].z; p0.w += a[p].w;
                p1.x += b[p].x; p1.y += b[p].y; p1.z += b[p].z; p1.w += b[p].w;
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
                    g.h_scales + ((int64_t)u.active * (g.I / 128) + at / 128) * 512 + (r & 31) * 16 +
                    (r >> 5) * 4 + (at & 127) / 32) = (uint16_t)(by | by << 8);
              }
            }
            bar_sync(1, 128);   // stage_v is free again
            j0 += 8;
          } while (j0 < n);
        }
        release();
      } else {
        int j0 = 0;
#pragma unroll 1
        do {
          float v[8];
          read8(j0, v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j0 + j < n) {
              const int slot = lists.slot[u.off + j0 + j];
              g.part_down[((size_t)u.part * slots + slot) * g.H + u.tile * kRows + row] =
                  v[j] * __ldg(&g.probs[slot]);
            }
          j0 += 8;
        } while (j0 < n);
        release();
      }
      if (live) {
        // (two units back the other warp has told)
        const bool ok = mbar_wait_lazy(&told_empty[local & 1], ((uint32_t)(local >> 1) & 1u) ^ 1u,
                                       &abort_flag, g.status, kDevTimeoutMma);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&told_full[local & 1]);
        ++local;
      }
    }
  }
  __syncwarp();
  if (abort_flag) {
    // copies in flight may still land: give them time before the CTA exits
    const uint64_t t0 = global_timer_ns();
    while (ns_since(t0) < 1000000ull) {
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
// K parts of the down product's units: at most eight stages a unit, so that the end is
// even and a block that waits for one expert's h has other units to do; more when even so
// there are not two units for three SMs, down to two stages each.  The SMs are a B200's:
// the workspace's size depends on the split and is asked for without a device.
constexpr int kSms = 148;
static int choose_splits(int64_t T, int64_t E, int topk, int64_t tiles, int64_t K) {
  const int kq = (int)(K / kBK);
  const int64_t slots = T * topk, units = (slots < E ? slots : E) * tiles;
  int64_t s = (kq + 15) / 16, few = kSms * 2 / 3 / units;
  if (few > kq / 4) few = kq / 4;
  if (s < few) s = few;
  return s > kMaxDownParts ? kMaxDownParts : (int)s;
}

struct Layout {
  size_t xq, xs, experts, probs, hq, h_scales, part_up, part_down, counters, total;
  int splits_down, max_act, n_counters;
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
  l.splits_down = choose_splits(T, E, topk, H / kRows, I);
  l.xq = take((size_t)T * 2 * H);
  l.xs = take((size_t)T * 4);
  l.experts = take(slots * 4);
  l.probs = take(slots * 4);
  l.hq = take(slots * 2 * I);
  l.h_scales = take((size_t)l.max_act * (I / 128) * 512);
  l.part_up = take((size_t)kMaxGrid * T * kRows * 4);   // units x parts <= blocks
  l.part_down = take((size_t)l.splits_down * slots * H * 4);
  l.n_counters = 2 + l.max_act + kMaxGrid + (int)(H / kRows);
  l.counters = take((size_t)l.n_counters * 4);
  l.total = at;
  return l;
}

// 4-bit rows unpacked to 16 bytes for each 16 values on the way to shared memory
// (row length and start a multiple of 128 values).
static bool weights_map(CUtensorMap* map, const uint8_t* base, uint64_t rows, uint64_t K) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  cuuint32_t box[2] = {128, (cuuint32_t)kRows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<uint8_t*>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe

size_t moe_workspace(int64_t T, int64_t H, int64_t E, int topk, int64_t I) {
  return moe::layout(T, H, E, topk, I).total;
}

cudaError_t launch_moe(const MoeArgs& a, int sm_count, cudaStream_t st) {
  using namespace moe;
  const Layout l = layout(a.T, a.H, a.E, a.topk, a.I);
  uint8_t* w = static_cast<uint8_t*>(a.workspace);
  ExpertArgs g;
  int32_t* experts = reinterpret_cast<int32_t*>(w + l.experts);
  float* probs = reinterpret_cast<float*>(w + l.probs);
  float* xs = reinterpret_cast<float*>(w + l.xs);
  int* counters = reinterpret_cast<int*>(w + l.counters);
  CUtensorMap tm13, tm2;
  if (!weights_map(&tm13, a.w13_codes, (uint64_t)a.E * 2 * a.I, (uint64_t)a.H) ||
      !weights_map(&tm2, a.w2_codes, (uint64_t)a.E * a.H, (uint64_t)a.I))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_limit(k_moe_experts, kMaxDynSmem);
  if (e != cudaSuccess) return e;

  // one token a cluster while all clusters are resident at once (8 CTAs each)
  if (a.T * kRouteCtas <= sm_count)
    k_moe_route<1><<<a.T * kRouteCtas, 256, 0, st>>>(
        a.X, a.T, a.H, a.router, a.E, a.topk, a.renorm, experts, probs, a.experts, a.probs,
        w + l.xq, xs, counters, l.n_counters);
  else
    k_moe_route<4><<<(a.T + 3) / 4 * kRouteCtas, 256, 0, st>>>(
        a.X, a.T, a.H, a.router, a.E, a.topk, a.renorm, experts, probs, a.experts, a.probs,
        w + l.xq, xs, counters, l.n_counters);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  g.experts = experts;
  g.probs = probs;
  g.w13_codes = a.w13_codes;
  g.w13_scales = a.w13_scales;
  g.w2_codes = a.w2_codes;
  g.w2_scales = a.w2_scales;
  g.T = a.T;
  g.E = a.E;
  g.topk = a.topk;
  g.by_topk = (65535 + a.topk) / a.topk;
  g.H = a.H;
  g.I = a.I;
  g.down_parts = l.splits_down;
  g.xq = w + l.xq;
  g.xs = xs;
  g.hq = w + l.hq;
  g.h_scales = w + l.h_scales;
  g.part_up = reinterpret_cast<float*>(w + l.part_up);
  g.part_down = reinterpret_cast<float*>(w + l.part_down);
  g.claimed = counters;
  g.up_total = counters + 1;
  g.up_done = counters + 2;
  g.up_joined = g.up_done + l.max_act;
  g.down_done = g.up_joined + kMaxGrid;
  g.Y = a.Y;
  g.status = a.status;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count < kMaxGrid ? sm_count : kMaxGrid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 1024 + kRingBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_moe_experts, tm13, tm2, g);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace e8
