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
// part_logit [S][T][E], part_xn2 [S][T], part_wn2 [S][E] over slice blockIdx.x.  Thread = two
// experts x every n-th row of the slice, all tokens (TT >= T of them); its rows' weights are
// loaded before any is used.  Every product is exact in fp64.
template <int TT>
__global__ void __launch_bounds__(W4M_FRONT_THREADS) w4_front_kernel(
    const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ wr, int T, int H, int E,
    double* __restrict__ part_logit, double* __restrict__ part_xn2, double* __restrict__ part_wn2,
    int* __restrict__ counters, int n_counters, unsigned* __restrict__ stats) {
  pdl_wait();
  pdl_trigger();
  __shared__ double xs[W4M_SLICE][TT];
  __shared__ double red[W4M_FRONT_THREADS][6];
  const int tid = threadIdx.x, s = blockIdx.x, h0 = s * W4M_SLICE;
  for (int i = s * W4M_FRONT_THREADS + tid; i < n_counters; i += gridDim.x * W4M_FRONT_THREADS)
    counters[i] = 0;
  if (s == 0 && tid < 5) stats[tid] = 0;
  const int pairs = E / 2, groups = W4M_FRONT_THREADS / pairs;   // E % 4 == 0, E <= 256
  const int ep = tid % pairs, grp = tid / pairs;
  const bool active = grp < groups;
  constexpr int MAXR = 32;   // rows of a thread loaded at once
  uint32_t w[MAXR];
  const __nv_bfloat16* wp = wr + (size_t)h0 * E + 2 * ep;
#pragma unroll
  for (int i = 0; i < MAXR; ++i) {
    const int h = grp + i * groups;
    w[i] = active && h < W4M_SLICE ? __ldg(reinterpret_cast<const unsigned*>(wp + (size_t)h * E)) : 0u;
  }
  for (int i = tid; i < W4M_SLICE * TT; i += W4M_FRONT_THREADS) {
    const int t = i / W4M_SLICE, h = i % W4M_SLICE;
    xs[h][t] = t < T ? (double)__bfloat162float(x[(size_t)t * H + h0 + h]) : 0.0;
  }
  __syncthreads();
  double acc[TT][2], wn[2] = {0.0, 0.0};
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t][0] = acc[t][1] = 0.0;
  if (active) {
#pragma unroll
    for (int i = 0; i < MAXR; ++i) {
      const int h = grp + i * groups;
      if (h < W4M_SLICE) {
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
    }
  }
  // join the row groups, two tokens (or one, and the norms) at a time, in group order
#pragma unroll
  for (int t = 0; t <= TT; t += 2) {
    __syncthreads();
    if (t < TT) {
      red[tid][0] = acc[t < TT ? t : 0][0];
      red[tid][1] = acc[t < TT ? t : 0][1];
      red[tid][2] = acc[t + 1 < TT ? t + 1 : 0][0];
      red[tid][3] = acc[t + 1 < TT ? t + 1 : 0][1];
    } else {
      red[tid][0] = wn[0];
      red[tid][1] = wn[1];
    }
    __syncthreads();
    for (int i = tid; i < 2 * E; i += W4M_FRONT_THREADS) {
      const int u = i / E, e = i - u * E;
      double v = 0.0;
      for (int g = 0; g < groups; ++g) v += red[g * pairs + e / 2][2 * u + (e & 1)];
      if (t < TT) {
        if (t + u < T) part_logit[((size_t)s * T + t + u) * E + e] = v;
      } else if (u == 0) {
        part_wn2[(size_t)s * E + e] = v;
      }
    }
  }
  if (tid < T) {
    double v = 0.0;
    for (int h = 0; h < W4M_SLICE; ++h) v = fma(xs[h][tid], xs[h][tid], v);
    part_xn2[(size_t)s * T + tid] = v;
  }
}

// ----------------------------------------------------------------------------- the layer
struct W4Moe {
  const __nv_bfloat16 *x, *wr;
  const float* bias;
  const uint8_t *wg, *wu, *wd;      // packed experts
  const double *part_logit, *part_xn2, *part_wn2;
  int slices;                       // of the front kernel
  int T, H, E, I, k, renorm, lg2;   // lg2: log2 of the row groups of a W_down unit
  double beta_scale;
  int32_t* ids;
  float* wts;
  unsigned* stats;
  int32_t *counts, *offsets, *perm; // optional outputs
  // counters, zeroed by the front kernel: {next token to select, tokens selected, next unit, -},
  // h_ready [128] per active expert, o_ready [row blocks of W_down]
  int* ctr;
  __nv_bfloat16* h;                 // [T k][I]
  float* o;                         // [T k][H]: weighted expert outputs
  __nv_bfloat16* y;
};
constexpr int W4M_CTR_H = 4, W4M_CTR_O = W4M_CTR_H + W4M_MAX_PAIRS;

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

// Select token t with the whole CTA.  scratch: at least 16 KB, 16-byte aligned.
__device__ __forceinline__ void w4_select(const W4Moe& a, int t, uint8_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, E = a.E;
  double* sL = reinterpret_cast<double*>(scratch);   // [256] logits
  double* sB = sL + 256;                             // [256] rounding bounds
  double* sSelV = sB + 256;                          // [8]
  double* sSelB = sSelV + 8;                         // [8]
  int* sSelE = reinterpret_cast<int*>(sSelB + 8);    // [8]
  double* sXn = sSelB + 16;                          // [1]
  double* sPart = sSelB + 24;                        // [W4S_THREADS][2]
  int* sRank = reinterpret_cast<int*>(sPart + 2 * W4S_THREADS);   // [256]
  const int groups = W4S_THREADS / E, e = tid % E, grp = tid / E;
  // the slices' partial sums: each group of threads adds every groups-th slice
  if (grp < groups) {
    double v = 0.0, w2 = 0.0;
    const double* p = a.part_logit + (size_t)t * E + e;
    const size_t step = (size_t)a.T * E;
#pragma unroll 8
    for (int s = grp; s < a.slices; s += groups) {
      v += __ldcg(p + s * step);
      w2 += __ldcg(a.part_wn2 + (size_t)s * E + e);
    }
    sPart[2 * tid] = v;
    sPart[2 * tid + 1] = w2;
  }
  if (tid >= W4S_THREADS - 32) {
    double v = 0.0;
    for (int s = lane; s < a.slices; s += 32) v += __ldcg(a.part_xn2 + (size_t)s * a.T + t);
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0) *sXn = v;
  }
  if (tid < 256) sRank[tid] = 0;
  __syncthreads();
  if (tid < E) {
    double v = 0.0, w2 = 0.0;
    for (int g = 0; g < groups; ++g) {
      v += sPart[2 * (g * E + tid)];
      w2 += sPart[2 * (g * E + tid) + 1];
    }
    const double b = a.bias ? (double)a.bias[tid] : 0.0;
    if (a.bias) v += b;
    sL[tid] = v;
    sB[tid] = a.beta_scale * (sqrt(*sXn * w2) * (1.0 + 1e-6) + fabs(b));
  }
  __syncthreads();
  // rank of expert e by (logit desc, id asc); NaN ranks below every number
  if (grp < groups) {
    const double ve = isnan(sL[e]) ? -INFINITY : sL[e];
    int r = 0;
#pragma unroll 4
    for (int e2 = grp; e2 < E; e2 += groups) {
      const double v2 = sL[e2];
      r += rank_before(isnan(v2) ? -INFINITY : v2, e2, ve, e) ? 1 : 0;
    }
    if (r) atomicAdd(&sRank[e], r);
  }
  __syncthreads();
  if (tid < E && sRank[tid] < a.k) {
    sSelE[sRank[tid]] = tid;
    sSelV[sRank[tid]] = sL[tid];
    sSelB[sRank[tid]] = sB[tid];
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
      const double m = sSelV[0];
      const double ex = lane < a.k ? exp(sSelV[lane] - m) : 0.0;
      double denom = 0.0;
      if (a.renorm) {
        for (int r = 0; r < a.k; ++r) denom += __shfl_sync(0xffffffffu, ex, r);
      } else {
        double sum = 0.0;
        for (int i = lane; i < E; i += 32) sum += exp(sL[i] - m);
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        denom = sum;
      }
      if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = sSelE[lane];
        a.wts[(size_t)t * a.k + lane] = (float)(ex / denom);
      }
    }
    __syncwarp();
    if (lane == 0) red_release_add_gpu(a.ctr + 1, 1);
  }
  __syncthreads();
}

// The CTA's lists of active experts and their pairs, expert by expert in ascending id, pairs
// ascending (the stable permutation of the dispatch).
struct W4List {
  int* pair;    // [128] pairs in expert order
  float* w;     // [128] their weights
  int* off;     // [129] first position of each active expert, and the end
  int* expert;  // [128] ids of the active experts
  int* info;    // {active experts}
};

__device__ __forceinline__ void w4_build_lists(const W4Moe& a, const W4List& L, int* sIds) {
  const int tid = threadIdx.x, P = a.T * a.k;
  int* sFirst = sIds + W4M_MAX_PAIRS;   // 1: the first pair of its expert
  const int id = tid < P ? __ldcg(a.ids + tid) : 0x7fffffff;
  if (tid < W4M_MAX_PAIRS) sIds[tid] = id;
  if (tid == 0) *L.info = 0;
  __syncthreads();
  int before = 0, same = 0;
  if (tid < P) {
    for (int q = 0; q < P; ++q) {
      const int o = sIds[q];
      before += o < id || (o == id && q < tid);
      same += o == id && q < tid;
    }
    sFirst[tid] = same == 0;
    if (same == 0) atomicAdd(L.info, 1);
    L.pair[before] = tid;
    L.w[before] = __ldcg(a.wts + tid);
  }
  __syncthreads();
  if (tid < P && same == 0) {
    int at = 0;
    for (int q = 0; q < P; ++q) at += sFirst[q] && sIds[q] < id;
    L.expert[at] = id;
    L.off[at] = before;
  }
  if (tid == 0) L.off[*L.info] = P;
  __syncthreads();
}

// Counts, offsets and permutation for the caller (one CTA writes them).
__device__ __forceinline__ void w4_write_aux(const W4Moe& a, const W4List& L, const int* sIds) {
  const int P = a.T * a.k;
  for (int e = threadIdx.x; e <= a.E; e += W4S_THREADS) {
    int less = 0, equal = 0;
    for (int q = 0; q < P; ++q) {
      less += sIds[q] < e;
      equal += sIds[q] == e;
    }
    if (a.offsets) a.offsets[e] = less;
    if (a.counts && e < a.E) a.counts[e] = equal;
  }
  if (a.perm)
    for (int q = threadIdx.x; q < P; q += W4S_THREADS) a.perm[q] = L.pair[q];
}

template <int NB, bool G32, bool ZP>
__global__ void __launch_bounds__(W4S_THREADS, 2) w4_moe_kernel(const __grid_constant__ W4Moe a) {
  constexpr int R = 512 + (G32 ? 2 : 1) * (ZP ? 48 : 32);
  constexpr int S = W4Ring<NB>::STAGES;
  extern __shared__ __align__(128) uint8_t w4sm[];
  const W4Smem L = w4s_layout<NB>(w4sm);
  const W4Bars<NB> bar{L.bars};
  W4List list;
  list.info = L.list;
  list.pair = L.list + 4;
  list.w = reinterpret_cast<float*>(list.pair + W4M_MAX_PAIRS);
  list.expert = list.pair + 2 * W4M_MAX_PAIRS;
  list.off = list.pair + 3 * W4M_MAX_PAIRS;
  int* s_token = L.list + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) w4s_init<NB>(L);
  pdl_wait();
  pdl_trigger();
  // ---- selection: tokens are taken from a counter until none is left (at once, when an earlier
  // launch's wait has run out)
  bool dead = false;
  while (true) {
    if (tid == 0) {
      dead = *reinterpret_cast<volatile unsigned*>(&g_error_word) & MOE_DEVERR_TIMEOUT;
      *s_token = dead ? a.T : atomicAdd(a.ctr, 1);
    }
    __syncthreads();
    const int t = *s_token;
    __syncthreads();
    if (t >= a.T) break;
    w4_select(a, t, w4sm);
  }
  if (tid == 0) *s_token = !dead && wait_counter_geq(a.ctr + 1, a.T);
  __syncthreads();
  if (!*s_token) return;   // nothing is in flight
  __threadfence();
  int* sIds = reinterpret_cast<int*>(L.acc);   // scratch until the first unit is joined
  w4_build_lists(a, list, sIds);
  if (blockIdx.x == 0 && (a.counts || a.offsets || a.perm)) {
    w4_write_aux(a, list, sIds);
    __syncthreads();
  }
  const int n_act = *list.info;
  const int kb1 = a.H / W4_KB, kb2 = a.I / W4_KB, strips1 = a.I / W4_ROWS, strips2 = a.H / W4_ROWS;
  const int nb2 = (strips2 + (2 << a.lg2) - 1) >> (a.lg2 + 1);   // W_down row blocks
  const int U1 = n_act * strips1, units = U1 + n_act * nb2;
  int* h_ready = a.ctr + W4M_CTR_H;
  int* o_ready = a.ctr + W4M_CTR_O;

  if (warp == W4S_MMA_WARPS + W4S_EPI_WARPS) {
    fence_proxy_async_smem();   // the ring held generic writes (the selection's scratch)
    fence_proxy_async_global();
    W4Producer<NB, R> p{L, w4sm, lane};
    bool ok = true;
    int c = 0;
    if (lane == 0) c = atomicAdd(a.ctr + 2, 1);
    c = __shfl_sync(0xffffffffu, c, 0);
    while (ok && c < units) {
      int next = 0;
      if (lane == 0) next = atomicAdd(a.ctr + 2, 1);   // one unit ahead
      W4Unit un;
      un.id = c;
      const bool down = c >= U1;
      const int v = down ? c - U1 : c, per = down ? nb2 : strips1, ai = v / per, b = v - ai * per;
      const int off = list.off[ai], e = list.expert[ai];
      un.rows = list.off[ai + 1] - off;
      const int pair = list.pair[off + min(lane, un.rows - 1)];
      const __nv_bfloat16* row;
      if (!down) {
        un.kb = kb1;
        un.strips = 2;
        un.lg = 0;
        un.pitch = 0;
        const size_t at = ((size_t)e * strips1 + b) * kb1 * R;
        un.s0 = a.wg + at;
        un.s1 = a.wu + at;
        row = a.x + (size_t)(pair / a.k) * a.H;
      } else {
        un.kb = kb2;
        const int s0 = b << (a.lg2 + 1);
        un.strips = min(2 << a.lg2, strips2 - s0);
        un.lg = a.lg2;
        un.pitch = (size_t)kb2 * R;
        un.s0 = a.wd + ((size_t)e * strips2 + s0) * un.pitch;
        un.s1 = un.s0 + un.pitch;
        row = a.h + (size_t)pair * a.I;
      }
      const int step = w4s_chunk_blocks<NB, R>(un.kb, un.strips, un.rows);
      int first = 0;
      if (down) {
        // the first stages' weights, then wait for the expert's h, then its rows
        const int pre = min((un.kb + step - 1) / step, S);
        for (int i = 0; i < pre && ok; ++i)
          ok = p.weights(un, i * step, min(step, un.kb - i * step), p.q + i);
        int ready = 1;
        if (ok && lane == 0) ready = wait_counter_geq(h_ready + ai, W4S_EPI_WARPS * strips1);
        ok = __shfl_sync(0xffffffffu, ready, 0) && ok;
        fence_proxy_async_global();
        for (int i = 0; i < pre && ok; ++i) p.rows(un, i * step, min(step, un.kb - i * step), p.q + i, row);
        p.q += pre;
        first = pre * step;
      }
      for (; first < un.kb && ok; first += step) {
        const int n = min(step, un.kb - first);
        ok = p.weights(un, first, n, p.q);
        if (ok) p.rows(un, first, n, p.q, row);
        ++p.q;
      }
      c = __shfl_sync(0xffffffffu, next, 0);
    }
    if (ok) ok = p.stop();
    if (!ok) *reinterpret_cast<volatile int*>(L.abort_flag) = 1;
  } else if (warp < W4S_MMA_WARPS) {
    w4s_multiply<NB, G32, ZP>(L, warp, lane);
  } else {
    const int et = tid - 32 * W4S_MMA_WARPS;
    for (int n = 0;; ++n) {
      const int b = n & 1;
      if (!w4s_wait(bar.acc_full(b), (n >> 1) & 1)) {
        *reinterpret_cast<volatile int*>(L.abort_flag) = 1;
        break;
      }
      const int4 u = L.acc_unit[b];
      if (u.x < 0) break;
      const float* acc = L.acc + b * (w4s_acc_bytes<NB>() / 4);
      const bool down = u.x >= U1;
      const int v = down ? u.x - U1 : u.x, per = down ? nb2 : strips1, ai = v / per, blk = v - ai * per;
      const int off = list.off[ai];
      if (!down) {
        for (int i = et; i < 16 * u.z; i += 32 * W4S_EPI_WARPS) {
          const int r = i & 15, c = i >> 4;
          const float gt = w4s_join<NB>(acc, 0, 0, c, r), up = w4s_join<NB>(acc, 0, 1, c, r);
          a.h[(size_t)list.pair[off + c] * a.I + 16 * blk + r] = __float2bfloat16_rn(w4_geglu(gt, up));
        }
      } else {
        const int n0 = (blk << (a.lg2 + 1)) * W4_ROWS;
        for (int c = 0; c < u.z; ++c) {
          float* o = a.o + (size_t)list.pair[off + c] * a.H + n0;
          const float w = list.w[off + c];
          for (int i = et; i < 16 * u.y; i += 32 * W4S_EPI_WARPS)
            o[i] = w * w4s_join<NB>(acc, u.w, i >> 4, c, i & 15);
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar.acc_empty(b));
        red_release_add_gpu(down ? o_ready + blk : h_ready + ai, 1);
      }
    }
  }
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(L.abort_flag)) {
    if (tid == 0) w4s_drain<NB>(L);
    return;
  }
  // ---- the weighted sum of each token's slots, in slot order: this CTA's share of four outputs
  // a thread, once every expert's rows of that block are there
  const int quads = a.H / 4, items = a.T * quads;
  const int share = (items + gridDim.x - 1) / gridDim.x;
  for (int i = blockIdx.x * share + tid; i < min(items, (int)(blockIdx.x + 1) * share); i += W4S_THREADS) {
    const int t = i / quads, n = 4 * (i - t * quads);
    if (!wait_counter_geq(o_ready + (n / W4_ROWS >> (a.lg2 + 1)), W4S_EPI_WARPS * n_act)) return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < a.k; ++j) {
      const float4 p = __ldcg(reinterpret_cast<const float4*>(a.o + ((size_t)t * a.k + j) * a.H + n));
      v.x += p.x;
      v.y += p.y;
      v.z += p.z;
      v.w += p.w;
    }
    uint2 r;
    r.x = pack_bf16x2(v.x, v.y);
    r.y = pack_bf16x2(v.z, v.w);
    *reinterpret_cast<uint2*>(a.y + (size_t)t * a.H + n) = r;
  }
}

}  // namespace moe
