// w4_moe.cuh -- the whole routed layer with 4-bit expert weights for T <= 16 tokens, in two
// launches:
//
//   1. w4_front_kernel: fp64 partial logits over 64-row slices of W_router (every slice read
//      once, for all tokens), squared norms for the rounding bound, and the counters' zeros;
//   2. w4_moe_kernel: each token's selection (the sum of its partial logits, the verified top-k
//      and the weights, as in router.cuh) by whichever CTAs take one; then every CTA lists the
//      active experts and their (token, slot) pairs for itself -- at most 128 pairs -- and takes
//      units from a counter: 16 gate | up features of one expert (GEGLU, h), then the W_down
//      strips of one expert, then its share of the weighted sum.
//
// The second kernel is the weight stream of w4_stream.cuh.  A unit waits only for units (and
// selections) that were taken before it, by CTAs that are running, so it ends under any schedule;
// its weights are already on their way while it waits.  What bounds it: the active experts' bytes
// at the memory's rate; at one token the chain of the two launches, the selection and the three
// hand-overs through L2.
#pragma once
#include "router.cuh"
#include "w4_stream.cuh"

namespace moe {

constexpr int W4M_SLICE = 64;      // rows of W_router per CTA of the front kernel
constexpr int W4M_FRONT_THREADS = 256;
constexpr int W4M_MAX_PAIRS = 128;

// ----------------------------------------------------------------------------- partial logits
// part_logit [S][T][E], part_xn2 [S][T] and part_wn2 [S][warps] over slice blockIdx.x, for the
// tokens of group blockIdx.y.  Thread = two experts x every n-th row of the slice, W4M_TT tokens;
// its rows' weights are loaded before any is used.  Every product is exact in fp64.  part_wn2:
// per warp a bound of its columns' parts of |w_e|^2, so that the sum over slices and warps bounds
// every column's squared norm (the rounding bound needs no more, and 8 numbers a slice are read
// instead of E).
constexpr int W4M_TT = 4;
__global__ void __launch_bounds__(W4M_FRONT_THREADS) w4_front_kernel(
    const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ wr, int T, int H, int E,
    double* __restrict__ part_logit, double* __restrict__ part_xn2, double* __restrict__ part_wn2,
    int* __restrict__ counters, int n_counters, unsigned* __restrict__ stats, int32_t* __restrict__ ids,
    int k, __nv_bfloat16* __restrict__ xfrag) {
  constexpr int TT = W4M_TT;
  pdl_wait();
  pdl_trigger();
  __shared__ double xs[W4M_SLICE][TT];
  __shared__ double red[2 * TT][W4M_FRONT_THREADS];
  const int tid = threadIdx.x, s = blockIdx.x, h0 = s * W4M_SLICE, t0 = blockIdx.y * TT;
  const int nt = min(TT, T - t0);
  if (blockIdx.y == 0) {
    for (int i = s * W4M_FRONT_THREADS + tid; i < n_counters; i += gridDim.x * W4M_FRONT_THREADS)
      counters[i] = 0;
    if (s == 0 && tid < 5) stats[tid] = 0;
    if (s == 0 && tid < T * k) ids[tid] = -1;   // not selected yet
  }
  const int pairs = E / 2, groups = W4M_FRONT_THREADS / pairs;   // E % 4 == 0, E <= 256
  const int ep = tid % pairs, grp = tid / pairs;
  const bool active = grp < groups;
  const __nv_bfloat16* wp = wr + (size_t)h0 * E + 2 * ep;
  constexpr int BATCH = 16;   // rows of a thread loaded at once
  uint32_t w[BATCH];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int h = grp + (i0 + i) * groups;
      w[i] = active && h < W4M_SLICE ? __ldg(reinterpret_cast<const unsigned*>(wp + (size_t)h * E)) : 0u;
    }
  };
  load(0);
  {
    const int t = tid / W4M_SLICE, h = tid % W4M_SLICE;   // 4 tokens x 64 rows = one element a thread
    const __nv_bfloat16 v = t < nt ? x[(size_t)(t0 + t) * H + h0 + h] : __float2bfloat16_rn(0.f);
    xs[h][t] = (double)__bfloat162float(v);
    if (t < nt) xfrag[w4_frag_index(T > 8 ? 2 : 1, t0 + t, h0 + h)] = v;
  }
  __syncthreads();
  double acc[TT][2], wn[2] = {0.0, 0.0};
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t][0] = acc[t][1] = 0.0;
  for (int i0 = 0;;) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int h = min(grp + (i0 + i) * groups, W4M_SLICE - 1);   // rows past the end hold zeros
      const double w0 = (double)__uint_as_float(w[i] << 16);
      const double w1 = (double)__uint_as_float(w[i] & 0xffff0000u);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const double xv = xs[h][t];
        acc[t][0] = fma(xv, w0, acc[t][0]);
        acc[t][1] = fma(xv, w1, acc[t][1]);
      }
      wn[0] = fma(w0, w0, wn[0]);
      wn[1] = fma(w1, w1, wn[1]);
    }
    i0 += BATCH;
    if (i0 * groups >= W4M_SLICE) break;
    load(i0);
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    red[2 * t][tid] = acc[t][0];
    red[2 * t + 1][tid] = acc[t][1];
  }
  if (blockIdx.y == 0) {
    double m = fmax(wn[0], wn[1]);
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, off));
    // with fewer than 32 pairs several parts of a column lie in one warp
    if ((tid & 31) == 0)
      part_wn2[s * (W4M_FRONT_THREADS / 32) + tid / 32] = pairs < 32 ? m * (32 / pairs + 1) : m;
  }
  __syncthreads();
  // join the row groups, in group order
  for (int i = tid; i < nt * E; i += W4M_FRONT_THREADS) {
    const int t = i / E, e = i - t * E;
    double v = 0.0;
    for (int g = 0; g < groups; ++g) v += red[2 * t + (e & 1)][g * pairs + e / 2];
    part_logit[((size_t)s * T + t0 + t) * E + e] = v;
  }
  if (tid / 32 < nt) {
    const int t = tid / 32, lane = tid & 31;
    double v = xs[lane][t] * xs[lane][t];
    v = fma(xs[lane + 32][t], xs[lane + 32][t], v);
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0) part_xn2[(size_t)s * T + t0 + t] = v;
  }
}
static_assert(W4S_EPI_WARPS == 2, "one joining warp per accumulator tile");
static_assert(W4M_TT * W4M_SLICE == W4M_FRONT_THREADS, "one activation per thread");

// ----------------------------------------------------------------------------- the layer
struct W4Moe {
  const __nv_bfloat16 *x, *wr;
  const float* bias;
  const uint8_t *wg, *wu, *wd;      // packed experts
  const double *part_logit, *part_xn2, *part_wn2;
  int slices;                       // of the front kernel
  int T, H, E, I, k, renorm;
  double beta_scale;
  int32_t* ids;
  float* wts;
  unsigned* stats;
  int32_t *counts, *offsets, *perm; // optional outputs
  // counters, zeroed by the front kernel: {-, -, next unit, tokens with weights, GEMM-1 units
  // joined, ...}, claimed [16] per token,
  // h_ready [128] per active expert, o_ready [row blocks of W_down]
  int* ctr;
  __nv_bfloat16* h;                 // [T k][I]
  // activations of experts with many rows: x of all tokens, h per active expert, as fragments with
  // a column per token
  __nv_bfloat16 *xfrag, *hfrag;
  float* o;                         // [T k][H]: expert outputs
  __nv_bfloat16* y;
};
constexpr int W4M_CTR_CLAIM = 8, W4M_CTR_H = W4M_CTR_CLAIM + W4_MAX_T, W4M_CTR_O = W4M_CTR_H + W4M_MAX_PAIRS;

// Wait until *p >= target (another CTA's release), polling without a pause: these hand-overs are
// on the layer's critical path.
__device__ __forceinline__ bool w4m_wait(const int* p, int target) {
  if (ld_acquire_gpu(p) >= target) return true;
  const uint64_t t0 = global_timer_ns();
  while (ld_acquire_gpu(p) < target)
    if (global_timer_ns() - t0 > *reinterpret_cast<volatile unsigned long long*>(&g_wait_limit_ns)) {
      raise_error(MOE_DEVERR_TIMEOUT);
      return false;
    }
  return true;
}

// The exact recomputation of a token whose decisions the bounds cannot settle (rare; kept out of
// line so that it does not cost the kernel registers).
__device__ __noinline__ void w4_exact_token(const double* sL, const double* sB, int t, const W4Moe& a,
                                            double* scratch) {
  const int lane = threadIdx.x & 31;
  double L[8], B[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    L[i] = e < a.E ? sL[e] : -DBL_MAX;
    B[i] = e < a.E ? sB[e] : 0.0;
  }
  router_finish_token<8>(L, B, t, a.x, a.wr, a.bias, a.H, a.E, a.k, a.renorm, a.ids, a.wts, a.stats, scratch);
}

// Select token t with the whole CTA.  scratch: at least 16 KB, 16-byte aligned.  Each launch runs
// this code cold (T CTAs, once), so it is kept short: integer keys for the ranking instead of
// fp64 comparisons, few unrolled loops.
__device__ __forceinline__ void w4_select(const W4Moe& a, int t, uint8_t* scratch) {
  constexpr int WARPS = W4S_THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, E = a.E;
  double* sL = reinterpret_cast<double*>(scratch);   // [256] logits (-inf past E)
  double* sB = sL + 256;                             // [256] rounding bounds
  double* sSelV = sB + 256;                          // [8]
  double* sSelB = sSelV + 8;                         // [8]
  int* sSelE = reinterpret_cast<int*>(sSelB + 8);    // [8]
  double* sNorm = sSelB + 16;                        // [1] rounding bound without the bias
  double* sPart = sSelB + 24;                        // [W4S_THREADS]
  unsigned long long* sKey = reinterpret_cast<unsigned long long*>(sPart + W4S_THREADS);   // [256]
  int* sRank = reinterpret_cast<int*>(sKey + 256);            // [256]
  const int groups = W4S_THREADS / E, e = tid % E, grp = tid / E;
  // the slices' partial sums: each group of threads adds every groups-th slice
  if (grp < groups) {
    double v = 0.0;
    const double* p = a.part_logit + ((size_t)grp * a.T + t) * E + e;
    const size_t step = (size_t)groups * a.T * E;
    const int n = (a.slices - grp + groups - 1) / groups;
    for (int s = 0; s < n; s += 24) {
      double q[24];
#pragma unroll
      for (int i = 0; i < 24; ++i) q[i] = s + i < n ? __ldcg(p + (s + i) * step) : 0.0;
#pragma unroll
      for (int i = 0; i < 24; ++i) v += q[i];
    }
    sPart[tid] = v;
  }
  if (warp == WARPS - 1) {
    // the last warp also adds the norms: |x_t|^2 and the bound of every |w_e|^2
    double v = 0.0, w2 = 0.0;
    for (int s = lane; s < a.slices; s += 32) v += __ldcg(a.part_xn2 + (size_t)s * a.T + t);
#pragma unroll 4
    for (int s = lane; s < a.slices * (W4M_FRONT_THREADS / 32); s += 32) w2 += __ldcg(a.part_wn2 + s);
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      v += __shfl_xor_sync(0xffffffffu, v, off);
      w2 += __shfl_xor_sync(0xffffffffu, w2, off);
    }
    if (lane == 0) *sNorm = a.beta_scale * sqrt(v * w2) * (1.0 + 1e-6);
  }
  __syncthreads();
  if (tid < E) {
    double v = 0.0;
    for (int g = 0; g < groups; ++g) v += sPart[g * E + tid];
    const double b = a.bias ? (double)a.bias[tid] : 0.0;
    if (a.bias) v += b;
    sL[tid] = v;
    sB[tid] = *sNorm + a.beta_scale * fabs(b);
    // an unsigned key in the logits' order (-0 as 0, NaN below every number)
    const long long bits = __double_as_longlong(v + 0.0);
    sKey[tid] = isnan(v) ? 1ull : (unsigned long long)(bits ^ ((bits >> 63) | (1ll << 63)));
    sRank[tid] = 0;
  }
  __syncthreads();
  // rank of expert e by (logit desc, id asc): each group of threads counts over a part of the ids
  if (grp < groups) {
    const unsigned long long mine = sKey[e];
    const int lo = (grp * (E / 2) / groups) * 2, hi = ((grp + 1) * (E / 2) / groups) * 2;   // E is even
    int r = 0;
#pragma unroll 4
    for (int x = lo; x < hi; x += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(sKey + x);
      r += two.x > mine - (x < e ? 1 : 0);
      r += two.y > mine - (x + 1 < e ? 1 : 0);
    }
    if (r) atomicAdd(&sRank[e], r);
  }
  __syncthreads();
  if (tid < E && sRank[tid] < a.k) {
    const int r = sRank[tid];
    sSelE[r] = tid;
    sSelV[r] = sL[tid];
    sSelB[r] = sB[tid];
  }
  __syncthreads();
  // every decision must hold under the rounding bounds (as in router_finish_token)
  bool ok = true;
  if (tid < E && sRank[tid] >= a.k) ok = sSelV[a.k - 1] - sL[tid] > sSelB[a.k - 1] + sB[tid];
  if (tid + 1 < a.k) ok = ok && (sSelV[tid] - sSelV[tid + 1] > sSelB[tid] + sSelB[tid + 1]);
  ok = __syncthreads_and(ok);
  if (tid < 32) {
    if (!ok) {
      w4_exact_token(sL, sB, t, a, sPart);
    } else {
      // the ids at once: other CTAs poll them to start their streams; the weights are needed last
      if (lane < a.k) *reinterpret_cast<volatile int32_t*>(a.ids + (size_t)t * a.k + lane) = sSelE[lane];
      // The differences are taken in fp64; their exponentials and the sum in fp32 (the weights are
      // fp32: off by at most 0.37 * 2^-24 for the differences' rounding plus a few 2^-24; a token that
      // goes through w4_exact_token gets them in fp64, within the same 1e-6).  The fp64 exp's code
      // alone, fetched cold once a launch, took 3 us.
      const double m = sSelV[0];
      const float ex = lane < a.k ? expf((float)(sSelV[lane] - m)) : 0.f;
      float sum = ex;
      if (!a.renorm) {
        sum = 0.f;
#pragma unroll 1
        for (int i = lane; i < E; i += 32) sum += expf((float)(sL[i] - m));
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane < a.k) a.wts[(size_t)t * a.k + lane] = ex / sum;
    }
    __syncwarp();
    if (lane == 0) red_release_add_gpu(a.ctr + 3, 1);
  }
  __syncthreads();
}

// The CTA's lists of active experts and their pairs, expert by expert in ascending id, pairs
// ascending (the stable permutation of the dispatch).
struct W4List {
  int* pair;    // [128] pairs in expert order
  int* step;    // [128] blocks per chunk of each active expert's units: gate | up, down (16 bits each)
  int* off;     // [129] first position of each active expert, and the end
  int* expert;  // [128] ids of the active experts
  int* info;    // {active experts}
};
// An expert of more rows than this takes its activations as fragments of all tokens (one copy a
// chunk, columns of other tokens unused); fewer rows are copied one by one.
constexpr int W4M_NARROW = 3;

// sKeys: 128 id + pair of all pairs (past T k: larger than any), then 4 ints of scratch; 16-byte
// aligned.
__device__ __forceinline__ void w4_build_lists(const W4Moe& a, const W4List& L, int* sKeys, int stage,
                                                int record, int frag_block, int& lg1, int& lg2) {
  const int tid = threadIdx.x, P = a.T * a.k;
  unsigned* sFirst = reinterpret_cast<unsigned*>(sKeys + W4M_MAX_PAIRS);   // an expert's first places
  if (tid < P) {
    const int mine = sKeys[tid];
    int before = 0;
#pragma unroll 4
    for (int q = 0; q < P; q += 4) {
      const int4 o = *reinterpret_cast<const int4*>(sKeys + q);
      before += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
    }
    L.pair[before] = tid;
  }
  __syncthreads();
  // thread = place in expert order from here
  const int id = tid < P ? sKeys[L.pair[tid]] >> 7 : -1;
  const bool first = tid < P && (tid == 0 || sKeys[L.pair[tid - 1]] >> 7 != id);
  const unsigned firsts = __ballot_sync(0xffffffffu, first);
  if ((tid & 31) == 0 && tid < W4M_MAX_PAIRS) sFirst[tid >> 5] = firsts;
  __syncthreads();
  int n = 0, at = __popc(firsts & ((1u << (tid & 31)) - 1));   // active experts, and those before this one
#pragma unroll
  for (int i = 0; i < W4M_MAX_PAIRS / 32; ++i) {
    const int m = __popc(sFirst[i]);
    n += m;
    at += i < tid >> 5 ? m : 0;
  }
  if (first) {
    L.expert[at] = id;
    L.off[at] = tid;
  }
  if (tid == 0) {
    L.off[n] = P;
    *L.info = n;
  }
  __syncthreads();
  // Strips of a unit: 2 << lg1 (gate and up of 16 << lg1 features) and 2 << lg2.  A taller unit reads
  // the activations less often and is published once, but the last round of units is longer: it is
  // taken with four rounds or more (two where experts hold many rows).  H = 2816, I = 704: 12 tokens
  // on 68 experts 98 us with low units, 95 with tall ones; 16 tokens on 19 experts (1.4 rounds of tall
  // ones) 55 and 66.
  const int rounds = (P > W4M_NARROW * n ? 2 : 4) * gridDim.x;
  lg1 = n * (a.I / W4_ROWS) / 2 >= rounds ? 1 : 0;
  lg2 = n * (a.H / W4_ROWS) / 8 >= rounds ? 2 : 1;
  if (tid < n) {
    // blocks per chunk: as many as fit a stage, evened out over the unit
    const int rows = L.off[tid + 1] - L.off[tid];
    auto even = [&](int kb, int strips) {
      const int most = rows > W4M_NARROW ? stage / (strips * record + frag_block)
                                         : (stage - 64 * rows) / (strips * record + 128 * rows);
      const int chunks = (kb + most - 1) / most;
      return (kb + chunks - 1) / chunks;
    };
    L.step[tid] = even(a.H / W4_KB, 2 << lg1) | even(a.I / W4_KB, 2 << lg2) << 16;
  }
  __syncthreads();
}

// Counts, offsets and permutation for the caller (one CTA writes them).
__device__ __forceinline__ void w4_write_aux(const W4Moe& a, const W4List& L, const int* sKeys) {
  const int P = a.T * a.k;
  for (int e = threadIdx.x; e <= a.E; e += W4S_THREADS) {
    int less = 0, equal = 0;
    for (int q = 0; q < P; ++q) {
      less += sKeys[q] >> 7 < e;
      equal += sKeys[q] >> 7 == e;
    }
    if (a.offsets) a.offsets[e] = less;
    if (a.counts && e < a.E) a.counts[e] = equal;
  }
  if (a.perm)
    for (int q = threadIdx.x; q < P; q += W4S_THREADS) a.perm[q] = L.pair[q];
}

// A unit, from the producer to the other roles; rewritten only after every multiply warp has
// released a later unit's chunk (the ring holds at most W4S_STAGES chunks).
struct __align__(16) W4Desc {
  int unit;     // -1: no more work
  int strips, rows, lg;
  int blocks;   // along K
  int step;     // blocks per chunk
  int wide;     // 1: activations are fragments
  int pad;
};
constexpr int W4M_DESCS = W4S_STAGES + 1;
constexpr int W4M_LISTS = 4 * (4 + 4 * W4M_MAX_PAIRS + 4);
template <int NB> __host__ __device__ constexpr int w4m_stage() {
  return (W4S_SMEM - 2 * w4s_acc_bytes<NB>() - W4Sync::BYTES - (int)sizeof(W4Desc) * W4M_DESCS - 32 - W4M_LISTS) /
         W4S_STAGES / 128 * 128;
}

template <int NB, bool G32, bool ZP>
__global__ void __launch_bounds__(W4S_THREADS, 2) w4_moe_kernel(const __grid_constant__ W4Moe a) {
  constexpr int R = 512 + (G32 ? 2 : 1) * (ZP ? 48 : 32);
  constexpr int STAGE = w4m_stage<NB>(), FB = w4_frag_block<NB>();
  uint8_t* at = w4sm + W4S_STAGES * STAGE;
  float* acc_tiles = reinterpret_cast<float*>(at);
  at += 2 * w4s_acc_bytes<NB>();
  W4Desc* descs = reinterpret_cast<W4Desc*>(at);
  at += sizeof(W4Desc) * W4M_DESCS;
  int4* acc_unit = reinterpret_cast<int4*>(at);   // [2] {unit, strips, rows, lg}
  at += 32;
  W4Sync sy;
  sy.init(at);
  at += W4Sync::BYTES;
  W4List list;
  list.info = reinterpret_cast<int*>(at);
  int* s_token = list.info + 1;
  list.pair = list.info + 4;
  list.step = list.pair + W4M_MAX_PAIRS;
  list.expert = list.pair + 2 * W4M_MAX_PAIRS;
  list.off = list.pair + 3 * W4M_MAX_PAIRS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sy.reset(1);
  pdl_wait();
  pdl_trigger();
  // ---- selection: CTA t selects token t.  Every CTA then polls the ids themselves (-1 until they
  // are there).  The CTAs wait for CTAs that may not have started, if other work holds the SMs: one
  // that has waited long takes any token that nobody has claimed, so the wait ends.
  int* sKeys = reinterpret_cast<int*>(acc_tiles);   // scratch until the first unit is joined
  const int P = a.T * a.k;
  if (tid == 0) {
    const bool dead = *reinterpret_cast<volatile unsigned*>(&g_error_word) & MOE_DEVERR_TIMEOUT;
    *s_token = dead ? -1 : (int)blockIdx.x < a.T && !atomicExch(a.ctr + W4M_CTR_CLAIM + blockIdx.x, 1) ? (int)blockIdx.x
                                                                                                   : a.T;
  }
  __syncthreads();
  const uint64_t since = global_timer_ns();
  while (true) {
    const int t = *s_token;
    if (t < 0) return;   // an earlier launch's wait ran out, or this one's: nothing is in flight
    if (t < a.T) w4_select(a, t, w4sm);
    // wait a while for the ids
    int id = tid < P ? -1 : 0xffffff;
    const uint64_t t0 = global_timer_ns();
    while (id < 0 && global_timer_ns() - t0 < 20000)
      id = *reinterpret_cast<const volatile int32_t*>(a.ids + tid);
    if (tid < W4M_MAX_PAIRS) sKeys[tid] = max(id, 0) << 7 | tid;
    if (__syncthreads_and(id >= 0)) break;
    if (tid == 0) {
      int next = a.T;
      for (int i = 0; i < a.T && next == a.T; ++i)
        if (!atomicExch(a.ctr + W4M_CTR_CLAIM + i, 1)) next = i;
      if (next == a.T && global_timer_ns() - since > *reinterpret_cast<volatile unsigned long long*>(&g_wait_limit_ns)) {
        raise_error(MOE_DEVERR_TIMEOUT);
        next = -1;
      }
      *s_token = next;
    }
    __syncthreads();
  }
  int lg1, lg2;
  w4_build_lists(a, list, sKeys, STAGE, R, FB, lg1, lg2);
  if (blockIdx.x == 0 && (a.counts || a.offsets || a.perm)) {
    w4_write_aux(a, list, sKeys);
    __syncthreads();
  }
  const int n_act = *list.info;
  const int kb1 = a.H / W4_KB, kb2 = a.I / W4_KB, strips1 = a.I / W4_ROWS, strips2 = a.H / W4_ROWS;
  const int nb1 = strips1 >> lg1;                            // gate | up units of an expert (I % 64 == 0)
  const int nb2 = (strips2 + (2 << lg2) - 1) >> (lg2 + 1);   // W_down row blocks
  const int U1 = n_act * nb1, units = U1 + n_act * nb2;
  // v / per = umulhi(v, magic), exact as v * per < 2^32 (at most 128 * 512 units of 512 an expert)
  const unsigned magic1 = 0xffffffffu / nb1 + 1, magic2 = 0xffffffffu / nb2 + 1;
  auto split = [&](int c, bool& down, int& ai, int& blk) {
    down = c >= U1;
    const int v = down ? c - U1 : c, per = down ? nb2 : nb1;
    ai = per == 1 ? v : (int)__umulhi((unsigned)v, down ? magic2 : magic1);
    blk = v - ai * per;
  };
  int* h_ready = a.ctr + W4M_CTR_H;
  int* o_ready = a.ctr + W4M_CTR_O;

  if (warp == W4S_MMA_WARPS + W4S_EPI_WARPS) {
    if (lane == 0) {
      fence_proxy_async_smem();   // the ring held generic writes (the selection's scratch)
      fence_proxy_async_global();
      const uint32_t ring = smem_u32(w4sm);
      W4Pos pos;
      int q = 0, n_unit = 0;
      bool ok = true, all_h = false;
      // Wait for the next stage; false when the CTA gives up.
      auto acquire = [&] {
        if (sy.aborted() || (q >= W4S_STAGES && !sy.wait(sy.empty(pos.s), pos.phase ^ 1))) return false;
        sy.flags[1] = q + 1;
        return true;
      };
      int c = atomicAdd(a.ctr + 2, 1);
      while (ok && c < units) {
        const int next = atomicAdd(a.ctr + 2, 1);   // one unit ahead
        bool down;
        int ai, blk;
        split(c, down, ai, blk);
        const int off = list.off[ai], rows = list.off[ai + 1] - off, e = list.expert[ai];
        const bool wide = rows > W4M_NARROW;
        const int lg = down ? lg2 : lg1, s0 = down ? blk << (lg + 1) : blk << lg, kb = down ? kb2 : kb1;
        const int strips = down ? min(2 << lg, strips2 - s0) : 2 << lg;
        const size_t pitch = (size_t)kb * R;
        const size_t w_at = ((size_t)e * (down ? strips2 : strips1) + s0) * pitch;
        const int step = down ? list.step[ai] >> 16 : list.step[ai] & 0xffff;
        int4* d = reinterpret_cast<int4*>(descs + n_unit % W4M_DESCS);
        const int width = down ? a.I : a.H;
        const __nv_bfloat16* act = wide ? (down ? a.hfrag + (size_t)ai * kb2 * (FB / 2) : a.xfrag) : down ? a.h : a.x;
        const int row_bytes = wide ? FB : 128 * rows;   // activations of a block
        // weights and activation rows of the chunk at block b, into stage s
        auto weights = [&](int b, int s) {
          const uint32_t bytes = min(step, kb - b) * R;
          uint32_t dst = ring + s * STAGE;
          mbar_arrive_expect_tx(sy.full(s), strips * bytes + row_bytes * min(step, kb - b));
          if (down) {
            // strips whose whole depth is one chunk are one run of bytes
            const uint8_t* src = a.wd + w_at + (size_t)b * R;
            if (step >= kb) bulk_load(dst, src, strips * bytes, sy.full(s));
            for (int i = 0; step < kb && i < strips; ++i, src += pitch, dst += bytes)
              bulk_load(dst, src, bytes, sy.full(s));
          } else {
            size_t from = w_at + (size_t)b * R;
            for (int i = 0; i < strips; i += 2, from += pitch, dst += 2 * bytes) {
              bulk_load(dst, a.wg + from, bytes, sy.full(s));
              bulk_load(dst + bytes, a.wu + from, bytes, sy.full(s));
            }
          }
        };
        auto activations = [&](int b, int s) {
          const int n = min(step, kb - b);
          uint32_t dst = ring + s * STAGE + strips * n * R;
          if (wide) bulk_load(dst, act + (size_t)b * (FB / 2), n * FB, sy.full(s));
          for (int i = 0; !wide && i < rows; ++i, dst += 128 * n + 64) {
            const int pair = list.pair[off + i];
            bulk_load(dst, act + (size_t)(down ? pair : pair / a.k) * width + 64 * b, 128 * n, sy.full(s));
          }
        };
        int b = 0;
        if (down) {
          // the first stages' weights, then wait for the expert's h, then its rows
          const W4Pos from = pos;
          int n = 0;
          for (; n < W4S_STAGES && n * step < kb && ok; ++n) {
            ok = acquire();
            if (!ok) break;
            if (n == 0) {
              d[0] = make_int4(c, strips, rows, lg);
              d[1] = make_int4(kb, step, wide, 0);
            }
            weights(n * step, pos.s);
            ++q;
            pos.next();
          }
          if (ok && !all_h) {
            ok = w4m_wait(h_ready + ai, nb1);
            all_h = ld_acquire_gpu(a.ctr + 4) == U1;
          }
          fence_proxy_async_global();
          W4Pos p = from;
          // also when giving up: the chunks were announced with their activations
          for (int i = 0; i < n; ++i, p.next()) activations(i * step, p.s);
          b = n * step;
        }
        for (; b < kb && ok; b += step) {
          ok = acquire();
          if (!ok) break;
          if (b == 0) {
            d[0] = make_int4(c, strips, rows, lg);
            d[1] = make_int4(kb, step, wide, 0);
          }
          weights(b, pos.s);
          activations(b, pos.s);
          ++q;
          pos.next();
        }
        ++n_unit;
        c = next;
      }
      if (ok) {
        ok = acquire();
        descs[n_unit % W4M_DESCS].unit = -1;
        if (ok) mbar_arrive(sy.full(pos.s));
      }
      if (!ok) sy.abort();
    }
  } else if (warp < W4S_MMA_WARPS) {
    const int g = lane >> 2, t = lane & 3;
    float acc[2][NB][4];
#pragma unroll
    for (int i = 0; i < 2 * NB * 4; ++i) acc[i / (4 * NB)][i / 4 % NB][i % 4] = 0.f;
    W4Pos pos;
    bool ok = true;
    for (int n_unit = 0;; ++n_unit) {
      if (!sy.wait(sy.full(pos.s), pos.phase)) {
        ok = false;
        break;
      }
      const uint32_t head = (uint32_t)(reinterpret_cast<const uint8_t*>(descs + n_unit % W4M_DESCS) - w4sm);
      const uint4 d0 = lds<uint4>(head), d1 = lds<uint4>(head + 16);
      const int unit = (int)d0.x, strips = d0.y, rows = d0.z, lg = d0.w, kb = d1.x, step = d1.y;
      const bool wide = d1.z;
      const uint32_t x_block = wide ? FB : 128, x_half = wide ? NB * 512 : 64;
      const int slices = W4S_MMA_WARPS >> lg, group = warp & ((1 << lg) - 1), slice = warp >> lg;
      for (int b = 0; unit >= 0 && b < kb; b += step) {
        if (b && !sy.wait(sy.full(pos.s), pos.phase)) {
          ok = false;
          break;
        }
        if (2 * group < strips) {
          const int n = min(step, kb - b);
          // this warp's blocks: those whose place along K is `slice` modulo the slices
          const int f = (slice - b) & (slices - 1);
          const uint32_t st = pos.s * STAGE;
          // a unit's odd last strip is multiplied twice; the second sum is not read
          const uint32_t to1 = 2 * group + 1 < strips ? n * R : 0;
          uint32_t xr[NB];
#pragma unroll
          for (int j = 0; j < NB; ++j)
            xr[j] = st + strips * n * R + f * x_block +
                    (wide ? 512 * j + 16 * lane : min(g + 8 * j, rows - 1) * (128 * n + 64) + 16 * t);
          w4s_blocks<NB, G32, ZP>(acc, (n - f + slices - 1) >> (3 - lg),
                                  st + (2 * group * n + f) * R + 16 * lane, to1, slices * R, xr,
                                  x_block * slices, x_half, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.empty(pos.s));
        pos.next();
      }
      if (!ok) break;
      // hand the unit's partial sums (or the end) to the joining warps
      const int buf = n_unit & 1;
      if (n_unit >= 2 && !sy.wait(sy.acc_empty(buf), ((n_unit >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      if (warp == 0 && lane == 0) acc_unit[buf] = make_int4(unit, strips, rows, lg);
      if (unit >= 0)
        w4s_put<NB>(acc, smem_u32(acc_tiles) + buf * w4s_acc_bytes<NB>(), ((slice << lg) + group) * 2, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.acc_full(buf));
      if (unit < 0) {
        // the end, to the other joining warp too
        const int last = buf ^ 1, m = n_unit + 1;
        ok = m < 2 || sy.wait(sy.acc_empty(last), ((m >> 1) - 1) & 1);
        if (!ok) break;
        if (warp == 0 && lane == 0) acc_unit[last] = make_int4(-1, 0, 0, 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.acc_full(last));
        break;
      }
    }
    if (!ok) sy.abort();
  } else {
    // the joining warps take the units in turn, one accumulator tile each: publishing a unit's
    // outputs takes a fence of almost a microsecond, which must not hold up the next unit
    const int buf = warp - W4S_MMA_WARPS;
    const float* acc = acc_tiles + buf * (w4s_acc_bytes<NB>() / 4);
    for (int n = 0;; ++n) {
      if (sy.aborted() || !sy.wait(sy.acc_full(buf), n & 1)) {
        sy.abort();
        break;
      }
      const int4 u = acc_unit[buf];
      if (u.x < 0) break;
      bool down;
      int ai, blk;
      split(u.x, down, ai, blk);
      const int off = list.off[ai], rows = u.z;
      const bool wide = rows > W4M_NARROW;
      if (!down) {
        const int feats = 16 << lg1;
        for (int i = lane; i < feats * rows; i += 32) {
          const int r = i & (feats - 1), c = i >> (lg1 + 4), n = feats * blk + r;
          const int pair = list.pair[off + c], col = wide ? pair / a.k : c;
          const float gt = w4s_join<NB>(acc, u.w, 2 * (r >> 4), col, r & 15);
          const float up = w4s_join<NB>(acc, u.w, 2 * (r >> 4) + 1, col, r & 15);
          const __nv_bfloat16 h = __float2bfloat16_rn(w4_geglu(gt, up));
          if (wide) a.hfrag[(size_t)ai * kb2 * (FB / 2) + w4_frag_index(NB, col, n)] = h;
          else a.h[(size_t)pair * a.I + n] = h;
        }
      } else {
        const int n0 = (blk << (lg2 + 1)) * W4_ROWS;
        for (int c = 0; c < rows; ++c) {
          const int pair = list.pair[off + c], col = wide ? pair / a.k : c;
          float* o = a.o + (size_t)pair * a.H + n0;
#pragma unroll 2
          for (int i = lane; i < 16 * u.y; i += 32) o[i] = w4s_join<NB>(acc, u.w, i >> 4, col, i & 15);
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sy.acc_empty(buf));
        __threadfence();   // the warp's stores before either count
        atomicAdd(down ? o_ready + blk : h_ready + ai, 1);
        if (!down) atomicAdd(a.ctr + 4, 1);
      }
    }
  }
  __syncthreads();
  if (sy.aborted()) {
    if (tid == 0) sy.drain();
    return;
  }
  // ---- the weighted sum of each token's slots, in slot order: this CTA's share of four outputs
  // a thread, once every expert's rows of that block are there
  const int quads = a.H / 4, items = a.T * quads;
  const int share = (items + gridDim.x - 1) / gridDim.x;
  for (int i = blockIdx.x * share + tid; i < min(items, (int)(blockIdx.x + 1) * share); i += W4S_THREADS) {
    const int t = i / quads, n = 4 * (i - t * quads);
    if (!w4m_wait(o_ready + (n / W4_ROWS >> (lg2 + 1)), n_act) || !w4m_wait(a.ctr + 3, a.T))
      return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < a.k; ++j) {
      const float4 p = __ldcg(reinterpret_cast<const float4*>(a.o + ((size_t)t * a.k + j) * a.H + n));
      const float w = __ldcg(a.wts + (size_t)t * a.k + j);
      v.x = fmaf(w, p.x, v.x);
      v.y = fmaf(w, p.y, v.y);
      v.z = fmaf(w, p.z, v.z);
      v.w = fmaf(w, p.w, v.w);
    }
    uint2 r;
    r.x = pack_bf16x2(v.x, v.y);
    r.y = pack_bf16x2(v.z, v.w);
    *reinterpret_cast<uint2*>(a.y + (size_t)t * a.H + n) = r;
  }
}

}  // namespace moe
