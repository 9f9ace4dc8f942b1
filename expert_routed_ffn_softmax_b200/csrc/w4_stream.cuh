// w4_stream.cuh -- products of a few activation rows (at most 16) with packed 4-bit weights, as
// one stream of weight bytes: the linear layer and the two halves of the dense GEGLU MLP here, the
// routed experts of a whole MoE layer in w4_moe.cuh.
//
// What bounds it.  At T <= 16 a weight byte meets at most 64 flops, so the work is reading the
// weights once at the memory's rate, decoding two weights per byte on the way: per SM about 23
// bytes (46 weights) a clock.  The decode and the products of a block (1024 weights) take 24 clocks
// of an SM, 35 with two row tiles (measured by repeating them), its bytes 22: both must run at once,
// and do to two thirds (2816 x 131072 in 46 us for one row, 68 for 16; the bytes alone 30).
//
// Roles of a CTA (two CTAs per SM, so that one multiplies while the other joins or waits):
//   producer     one thread copies each unit in chunks of consecutive blocks, one bulk copy per
//                strip (a strip's run of blocks is contiguous), into a ring of stages.  Its code
//                per chunk is kept to the copies: beside warps that issue all the time every
//                instruction of it costs some ten clocks (with a header and a table per chunk and
//                the activations copied along it took 2000 to 3600 clocks a chunk and the stream
//                ran at 0.3 to 0.6 of the memory's rate);
//   multiply     8 warps = row groups of two strips x slices of the blocks along K; a block is one
//                16-byte shared read per lane, decoded in registers into operands of the matrix
//                instruction (w4_block);
//   join         2 warps add the K slices' fp32 sums through an accumulator tile in shared memory,
//                in a fixed order, and write the outputs, while the multiply warps are at the next
//                unit.
// Every wait is bounded; a wait that runs out sets the device error word and ends the CTA after
// its copies in flight have landed.
#pragma once
#include "gemm_persistent.cuh"
#include "w4.cuh"

namespace moe {

constexpr int W4S_MMA_WARPS = 8, W4S_EPI_WARPS = 2;
constexpr int W4S_THREADS = 32 * (W4S_MMA_WARPS + W4S_EPI_WARPS + 1);
constexpr int W4S_EPI_THREADS = 32 * W4S_EPI_WARPS;
// Two large stages: what the roles do once a chunk costs more than the finer overlap of three or four
// smaller ones gives (T = 16, 2816 x 131072: 67 us with two, 70 with three, 78 with four; the routed
// layer at 16 tokens 102 and 112).
constexpr int W4S_STAGES = 2;
constexpr int W4S_COL = 20;             // floats per accumulator column (16 rows, padded)
constexpr int W4S_SMEM = 115712;        // two CTAs per SM
// accumulator tile: 16 (K slice, strip) pairs x 8 NB columns
template <int NB> __host__ __device__ constexpr int w4s_acc_bytes() { return 16 * 8 * NB * W4S_COL * 4; }

enum W4Mode { W4_LINEAR = 0, W4_LINEAR_F32 = 1, W4_GEGLU = 2 };

// Bounded wait for warps that wait long and often beside warps that compute: the hint lets the
// hardware park the warp until the phase completes.  False also when the CTA gives up (*abort); that
// is looked at only when a wait is long, so the usual one costs a few instructions.
__device__ __forceinline__ bool w4s_wait(uint32_t bar, uint32_t parity, const volatile int* abort) {
  constexpr uint32_t kParkNs = 20000;
  uint64_t t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kParkNs)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > *reinterpret_cast<volatile unsigned long long*>(&g_wait_limit_ns)) {
      raise_error(MOE_DEVERR_TIMEOUT);
      return false;
    }
  }
}

// Barriers and flags of a CTA.
struct W4Sync {
  uint32_t base;
  volatile int* flags;   // {abort, phases issued (chunks, the end), activations issued, takeovers asked for}
  __device__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ uint32_t empty(int s) const { return base + 8u * (W4S_STAGES + s); }
  __device__ uint32_t acc_full(int b) const { return base + 8u * (2 * W4S_STAGES + b); }
  __device__ uint32_t acc_empty(int b) const { return base + 8u * (2 * W4S_STAGES + 2 + b); }
  __device__ uint32_t act_full() const { return base + 8u * (2 * W4S_STAGES + 4); }
  __device__ uint32_t steal_full() const { return base + 8u * (2 * W4S_STAGES + 5); }
  static constexpr int BYTES = 8 * (2 * W4S_STAGES + 6) + 16;
  __device__ void init(uint8_t* at) {
    base = smem_u32(at);
    flags = reinterpret_cast<volatile int*>(at + 8 * (2 * W4S_STAGES + 6));
  }
  // joiners: joining warps that release an accumulator tile
  __device__ void reset(int joiners) const {
    for (int s = 0; s < W4S_STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), W4S_MMA_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), W4S_MMA_WARPS);
      mbar_init(acc_empty(b), joiners);
    }
    mbar_init(act_full(), 1);
    mbar_init(steal_full(), 1);
    flags[0] = flags[1] = flags[2] = flags[3] = 0;
    fence_barrier_init();
  }
  __device__ void abort() const { flags[0] = 1; }
  __device__ bool aborted() const { return flags[0] != 0; }
  __device__ bool wait(uint32_t bar, uint32_t parity) const { return w4s_wait(bar, parity, flags); }
  // After the roles have ended with an abort: wait for everything that still writes this CTA's shared
  // memory, whatever the limit of the other waits: the copies of the last chunks (a stage is issued
  // again only when its chunk has been consumed), the activations, the answer to the last request to
  // take over a unit (the next request is made only when the answer before it has been read).
  __device__ void drain() const {
    for (int q = max(0, flags[1] - W4S_STAGES); q < flags[1]; ++q)
      mbar_wait_ns(full(q % W4S_STAGES), (q / W4S_STAGES) & 1, kDrainLimitNs);
    if (flags[2]) mbar_wait_ns(act_full(), 0, kDrainLimitNs);
    if (flags[3]) mbar_wait_ns(steal_full(), (flags[3] - 1) & 1, kDrainLimitNs);
  }
};

// Position in the ring: stage and the parity of its current phase.
struct W4Pos {
  int s = 0;
  uint32_t phase = 0;
  __device__ void next() {
    if (++s == W4S_STAGES) {
      s = 0;
      phase ^= 1;
    }
  }
};

// acc += this warp's blocks of one chunk: n blocks from record address w (+ 16 lane, strip 0; strip
// 1 at + to1) every w_step bytes, activations at xr every x_step bytes (a block's second half at
// + x_half).
template <int NB, bool G32, bool ZP>
__device__ __forceinline__ void w4s_blocks(float (&acc)[2][NB][4], int n, uint32_t w, uint32_t to1,
                                           uint32_t w_step, uint32_t (&xr)[NB], uint32_t x_step,
                                           uint32_t x_half, int lane) {
#pragma unroll 1
  for (; n > 0; --n) {
    const uint32_t rec[2] = {w, w + to1};
    w4_block<2, NB, G32, ZP>(acc, rec, lane, xr, x_half);
    w += w_step;
#pragma unroll
    for (int j = 0; j < NB; ++j) xr[j] += x_step;
  }
}

// Store this warp's partial sums into the accumulator tile at `tile` (entry = K slice x strips +
// strip) and clear them.
template <int NB>
__device__ __forceinline__ void w4s_put(float (&acc)[2][NB][4], uint32_t tile, int entry, int lane) {
  const uint32_t dst = tile + 4 * ((entry * 8 * NB + 2 * (lane & 3)) * W4S_COL + (lane >> 2));
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(
                         dst + 4 * (((i * NB + j) * 8 + (v & 1)) * W4S_COL + 8 * (v >> 1))),
                     "f"(acc[i][j][v])
                     : "memory");
        acc[i][j][v] = 0.f;
      }
}
// Sum over the K slices, in slice order, of one accumulator element.
template <int NB>
__device__ __forceinline__ float w4s_join(const float* acc, int lg, int strip, int col, int row) {
  const float* p = acc + (strip * 8 * NB + col) * W4S_COL + row;
  float v = 0.f;
  for (int s = 0; s < W4S_MMA_WARPS >> lg; ++s) v += p[(s * 2 * 8 * NB * W4S_COL) << lg];
  return 4.f * v;   // the decoded weights are quarters
}

// gelu_tanh(a) * u, with a (1 + tanh z) / 2 = a / (1 + exp(-2 z)): no sum that cancels, so negative
// gates keep their leading digits too (an approximate tanh good to 2^-11 leaves gelu(-3) off by a fifth).
// Relative error under 2^-14 for |a| <= 9; where the denominator passes 2^126 (a < -10) the quotient is
// 0 instead of less than 2^-122.  The call's one rounding between its products follows: h goes to bf16, the operand type of
// the second product (fp32 h would be two operands and twice the products); with the output's own
// rounding a call is 0.0024 from float64 in relative norm, 0.0017 if h kept fp32.
__device__ __forceinline__ float w4_geglu(float a, float u) {
  const float e = __expf(-1.5957691216057308f * (a + 0.044715f * a * a * a));
  return __fdividef(a, 1.f + e) * u;
}

// ----------------------------------------------------------------------------- work stealing
// Take over a CTA of this grid that has not started (cluster launch control): the answer, 16 bytes
// at `answer`, completes on `bar`.  SMs stream at different rates, so units dealt out in advance
// end at the pace of the slowest SM; this hands them out as CTAs become free, without a counter
// that something would have to zero before each launch.
__device__ __forceinline__ void steal_request(uint32_t answer, uint32_t bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          answer),
      "r"(bar)
      : "memory");
}
// The taken CTA's blockIdx.x, or -1 when none was left (no further request may follow then).
__device__ __forceinline__ int steal_answer(uint32_t answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(answer)
      : "memory");
  fence_proxy_async_smem();   // this read before the next answer is written
  return got ? (int)x : -1;
}

// ----------------------------------------------------------------------------- activations
// Activations in the multiply warps' order ("fragments"): per block along K 2 halves x NB row tiles
// x 32 lanes x 16 bytes, lane 4 g + t of (h, j) holding elements 64 b + 32 h + 8 t .. + 7 of row
// g + 8 j.  Rows past T hold anything: they only reach outputs that are not stored.
template <int NB>
__host__ __device__ constexpr int w4_frag_block() { return 2 * NB * 512; }
__host__ __device__ inline size_t w4_frag_index(int nb, int row, int k) {   // in elements
  return ((((size_t)(k >> 6) * 2 + ((k >> 5) & 1)) * nb + (row >> 3)) * 32 + 4 * (row & 7) + ((k >> 3) & 3)) * 8 +
         (k & 7);
}
// x [T][K] -> fragments, one 16-byte vector a thread.
__global__ void __launch_bounds__(256) w4_fragment_kernel(const __nv_bfloat16* __restrict__ x, int T, int K,
                                                          int nb, __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int per = K / 8;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < T * per; i += gridDim.x * 256) {
    const int row = i / per, k = 8 * (i - row * per);
    *reinterpret_cast<uint4*>(out + w4_frag_index(nb, row, k)) =
        __ldg(reinterpret_cast<const uint4*>(x + (size_t)row * K + k));
  }
}

// ----------------------------------------------------------------------------- linear, GEGLU
struct W4Linear {
  const uint8_t *w0, *w1;       // packed matrix; gate and up for GEGLU
  const __nv_bfloat16* act;     // [T][K], or fragments
  void* out;                    // [T][N]
  int T, K, N;
  int lg;                       // log2 of the row groups: 2 << lg strips per unit
  int step;                     // blocks per chunk
  int stage;                    // bytes of a stage
  int frag;                     // 1: act holds fragments and a chunk brings its blocks' along;
                                // 0: a CTA keeps all of act in shared memory
  int out_frag;                 // GEGLU: h is written as fragments of this many row tiles (or 0)
  int cluster;                  // CTAs that share a unit's K (1, 2, 4 or 8)
  int steal;                    // 1: more units than CTAs run at once (cluster 1)
  int early;                    // 1: the previous kernel does not write the weights and started
                                // after every kernel before it had ended: the first weight
                                // copies may start before it has ended
};

// Shared memory: ring, activations of the CTA's slice of K (rows 64 bytes apart, so that the two
// rows a quarter warp reads fall in different halves of the banks), accumulator tiles, the
// cluster's partial sums, ids, barriers.
struct W4LinearSmem {
  int act, acc, part, answer, unit, sync, total;
};
constexpr int W4S_UNITS = W4S_STAGES + 1;   // unit ids in flight from the producer to the others
template <int NB>
__host__ __device__ inline W4LinearSmem w4_linear_smem(int T, int K, int frag, int stage, int cluster, int lg) {
  W4LinearSmem L;
  const int most = (K / W4_KB + cluster - 1) / cluster;   // blocks of a CTA's slice of K
  L.act = W4S_STAGES * stage;
  L.acc = L.act + (frag ? 0 : T * (128 * most + 64));
  L.part = L.acc + (cluster > 1 ? 1 : 2) * w4s_acc_bytes<NB>();
  L.answer = (L.part + (cluster > 1 ? (32 << lg) * T * 4 : 0) + 15) / 16 * 16;
  L.unit = L.answer + 16;
  L.sync = L.unit + (W4S_UNITS + 2 + 3) / 4 * 16;   // barriers: 8-byte aligned
  L.total = L.sync + W4Sync::BYTES;
  return L;
}

// Units: 2 << lg strips (GEGLU: the gate and up strips of 16 << lg features, in turn).  A CTA
// starts with the unit of its block index and takes over units of CTAs that have not started.  A
// cluster takes one unit, each CTA a slice of K, and CTA r adds the r-th part of the unit's outputs
// over the CTAs, in rank order: taller units read the activations less often, and the slices keep
// every SM busy.
template <int NB, bool G32, bool ZP, int MODE>
__global__ void __launch_bounds__(W4S_THREADS, 2) w4_linear_kernel(const __grid_constant__ W4Linear a) {
  constexpr int R = 512 + (G32 ? 2 : 1) * (ZP ? 48 : 32);
  constexpr int FB = w4_frag_block<NB>();
  const W4LinearSmem SL = w4_linear_smem<NB>(a.T, a.K, a.frag, a.stage, a.cluster, a.lg);
  W4Sync sy;
  sy.init(w4sm + SL.sync);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sy.reset(W4S_EPI_WARPS);
  if (a.cluster > 1) cluster_sync();   // every CTA of the cluster runs before any stores to it
  if (!a.early) {
    pdl_wait();
    pdl_trigger();
  }
  // nothing is done when an earlier launch's wait has run out
  if (tid == 0 && (*reinterpret_cast<volatile unsigned*>(&g_error_word) & MOE_DEVERR_TIMEOUT)) sy.abort();
  __syncthreads();
  // unit ids: from the producer to the multiply warps (rewritten only after every multiply warp
  // has released a later unit's chunk), and on to the joining warps
  int* unit_ring = reinterpret_cast<int*>(w4sm + SL.unit);
  int* acc_unit = unit_ring + W4S_UNITS;
  const int rank = blockIdx.x % a.cluster, first_unit = blockIdx.x / a.cluster;
  const int kb = a.K / W4_KB, strips_all = a.N / W4_ROWS;
  const int k0 = rank * kb / a.cluster, blocks = (rank + 1) * kb / a.cluster - k0;   // slice of K
  const int act_pitch = 128 * blocks + 64;
  // strips of unit u (its matrix, or of each of gate and up)
  auto strips_of = [&](int u) {
    return MODE == W4_GEGLU ? min(1 << a.lg, strips_all - (u << a.lg))
                            : min(2 << a.lg, strips_all - (u << (a.lg + 1)));
  };
  if (warp == W4S_MMA_WARPS + W4S_EPI_WARPS) {
    if (lane == 0) {
      const uint32_t ring = smem_u32(w4sm), answer = smem_u32(w4sm + SL.answer);
      const size_t pitch = (size_t)kb * R;
      bool ok = !sy.aborted(), waited = !a.early;
      int q = 0, n_unit = 0, n_steal = 0;
      W4Pos pos;
      // act, once the previous kernel has ended: all of it, or the fragments of the chunks whose
      // weights are on their way already
      auto activations = [&](int chunks) {
        fence_proxy_async_global();
        if (!a.frag) {
          sy.flags[2] = 1;
          mbar_arrive_expect_tx(sy.act_full(), a.T * 128 * blocks);
          for (int t = 0; t < a.T; ++t)
            bulk_load(smem_u32(w4sm + SL.act) + t * act_pitch, a.act + (size_t)t * a.K + 64 * k0, 128 * blocks,
                      sy.act_full());
        }
        for (int i = 0; a.frag && i < chunks; ++i) {
          const int n = min(a.step, blocks - i * a.step), ns = (MODE == W4_GEGLU ? 2 : 1) * strips_of(first_unit);
          bulk_load(ring + i * a.stage + ns * a.step * R, a.act + (size_t)(k0 + i * a.step) * (FB / 2), n * FB, sy.full(i));
        }
        waited = true;
      };
      auto wait_previous = [&](int chunks) {
        pdl_wait();
        pdl_trigger();
        activations(chunks);
      };
      if (ok && waited) activations(0);
      for (int u = first_unit; u >= 0 && ok; ++n_unit) {
        unit_ring[n_unit % W4S_UNITS] = u;
        if (a.steal) {
          sy.flags[3] = ++n_steal;
          steal_request(answer, sy.steal_full());
        }
        const int ns = strips_of(u), all = MODE == W4_GEGLU ? 2 * ns : ns;
        const size_t at = ((size_t)u << (MODE == W4_GEGLU ? a.lg : a.lg + 1)) * pitch + (size_t)k0 * R;
        for (int b = 0; b < blocks; b += a.step, ++q, pos.next()) {
          // in the first unit weights go ahead until the ring is full
          if (!waited && q == W4S_STAGES) wait_previous(q);
          if (sy.aborted() || (q >= W4S_STAGES && !sy.wait(sy.empty(pos.s), pos.phase ^ 1))) {
            ok = false;
            break;
          }
          const int n = min(a.step, blocks - b);
          const uint32_t bytes = n * R, bar = sy.full(pos.s);
          uint32_t dst = ring + pos.s * a.stage;
          const uint8_t* src = a.w0 + at + (size_t)b * R;
          sy.flags[1] = q + 1;
          mbar_arrive_expect_tx(bar, all * bytes + (a.frag ? n * FB : 0));
          if (MODE == W4_GEGLU) {
            const uint8_t* up = a.w1 + at + (size_t)b * R;
            for (int i = 0; i < ns; ++i, src += pitch, up += pitch, dst += 2 * a.step * R) {
              bulk_load(dst, src, bytes, bar);
              bulk_load(dst + a.step * R, up, bytes, bar);
            }
          } else {
            for (int i = 0; i < ns; ++i, src += pitch, dst += a.step * R) bulk_load(dst, src, bytes, bar);
          }
          if (a.frag && waited) bulk_load(dst, a.act + (size_t)(k0 + b) * (FB / 2), n * FB, bar);
        }
        if (!waited) wait_previous(q);
        u = -1;
        if (a.steal) {
          if (!sy.wait(sy.steal_full(), (n_steal - 1) & 1)) ok = false;
          else u = steal_answer(answer);
        }
      }
      if (!waited) pdl_wait();
      if (ok && a.cluster == 1) {
        // the end, through a stage of its own
        if (q >= W4S_STAGES && !sy.wait(sy.empty(pos.s), pos.phase ^ 1)) ok = false;
        unit_ring[n_unit % W4S_UNITS] = -1;
        if (ok) {
          sy.flags[1] = q + 1;
          mbar_arrive(sy.full(pos.s));
        }
      }
      if (!ok) sy.abort();
    }
  } else if (warp < W4S_MMA_WARPS) {
    const int slices = W4S_MMA_WARPS >> a.lg, group = warp & ((1 << a.lg) - 1), slice = warp >> a.lg;
    float acc[2][NB][4];
#pragma unroll
    for (int i = 0; i < 2 * NB * 4; ++i) acc[i / (4 * NB)][i / 4 % NB][i % 4] = 0.f;
    W4Pos pos;
    int n_acc = 0;
    bool ok = true;
    // This lane's activations (of its rows in shared memory, from block 0; or of a stage's fragments)
    // and weights (of a stage); a chunk's strips are a.step blocks apart whatever it holds
    const uint32_t x_half = a.frag ? NB * 512 : 64, x_block = a.frag ? FB : 128;
    const uint32_t strip = a.step * R, w0 = 2 * group * strip + 16 * lane;
    uint32_t x0[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
      x0[j] = a.frag ? 512 * j + 16 * lane
                     : SL.act + min((lane >> 2) + 8 * j, a.T - 1) * act_pitch + 16 * (lane & 3);
    for (; ok; ++n_acc) {
      int u = -1;
      uint32_t to1 = 0, x_at = 0;
      bool mine = false;
      for (int b = 0; b < blocks; b += a.step) {
        if (!sy.wait(sy.full(pos.s), pos.phase)) {
          ok = false;
          break;
        }
        if (b == 0) {
          u = unit_ring[n_acc % W4S_UNITS];
          if (u < 0) break;
          const int ns = (MODE == W4_GEGLU ? 2 : 1) * strips_of(u);
          mine = 2 * group < ns;
          // a unit's odd last strip is multiplied twice; the second sum is not read
          to1 = 2 * group + 1 < ns ? strip : 0;
          x_at = a.frag ? ns * strip : 0;
          if (n_acc == 0 && !a.frag && !sy.wait(sy.act_full(), 0)) {
            ok = false;
            break;
          }
        }
        if (mine) {
          // this warp's blocks: those whose place along K is `slice` modulo the slices
          const int f = (slice - b) & (slices - 1);
          const uint32_t st = pos.s * a.stage, x_st = (a.frag ? st + x_at : b * 128) + f * x_block;
          uint32_t xr[NB];
#pragma unroll
          for (int j = 0; j < NB; ++j) xr[j] = x0[j] + x_st;
          w4s_blocks<NB, G32, ZP>(acc, (min(a.step, blocks - b) - f + slices - 1) >> (3 - a.lg), st + w0 + f * R,
                                  to1,
                                  slices * R, xr, x_block * slices, x_half, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sy.empty(pos.s));
        pos.next();
      }
      if (!ok) break;
      if (a.cluster > 1) {
        // one unit: the whole CTA joins it below
        w4s_put<NB>(acc, smem_u32(w4sm + SL.acc), ((slice << a.lg) + group) * 2, lane);
        break;
      }
      const int buf = n_acc & 1;
      if (n_acc >= 2 && !sy.wait(sy.acc_empty(buf), ((n_acc >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      if (warp == 0 && lane == 0) acc_unit[buf] = u;
      if (u >= 0)
        w4s_put<NB>(acc, smem_u32(w4sm + SL.acc) + buf * w4s_acc_bytes<NB>(), ((slice << a.lg) + group) * 2,
                    lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.acc_full(buf));
      if (u < 0) break;
    }
    if (!ok) sy.abort();
  } else {
    const int et = tid - 32 * W4S_MMA_WARPS;
    if (a.early) pdl_wait();   // the outputs may be what the previous kernel still reads
    for (int n = 0; a.cluster == 1; ++n) {
      const int buf = n & 1;
      if (sy.aborted() || !sy.wait(sy.acc_full(buf), (n >> 1) & 1)) {
        sy.abort();
        break;
      }
      const int u = acc_unit[buf];
      if (u < 0) break;
      const float* acc = reinterpret_cast<const float*>(w4sm + SL.acc) + buf * (w4s_acc_bytes<NB>() / 4);
      const int wide = 16 * strips_of(u);
      for (int c = 0; c < a.T; ++c)
        for (int i = et; i < wide; i += W4S_EPI_THREADS) {
          if (MODE == W4_GEGLU) {
            const float gt = w4s_join<NB>(acc, a.lg, 2 * (i >> 4), c, i & 15);
            const float up = w4s_join<NB>(acc, a.lg, 2 * (i >> 4) + 1, c, i & 15);
            const int f = (16 << a.lg) * u + i;
            const size_t o = a.out_frag ? w4_frag_index(a.out_frag, c, f) : (size_t)c * a.N + f;
            static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(w4_geglu(gt, up));
          } else {
            const float v = w4s_join<NB>(acc, a.lg, i >> 4, c, i & 15);
            const size_t o = (size_t)c * a.N + (32 << a.lg) * (size_t)u + i;
            if (MODE == W4_LINEAR_F32) static_cast<float*>(a.out)[o] = v;
            else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(sy.acc_empty(buf));
    }
  }
  __syncthreads();
  if (sy.aborted() && tid == 0) sy.drain();
  if (a.cluster == 1) return;
  // ---- a cluster's unit: this CTA's sums over its slice of K go to the CTAs that add them.  Rows of
  // a GEGLU unit are counted in pairs (gate, up) of the same feature.
  const int rows = 32 << a.lg, share = rows / a.cluster;
  float* part = reinterpret_cast<float*>(w4sm + SL.part);
  if (!sy.aborted()) {
    const float* acc = reinterpret_cast<const float*>(w4sm + SL.acc);
    for (int i = tid; i < rows * a.T; i += W4S_THREADS) {
      const int r = i & (rows - 1), c = i >> (a.lg + 5), owner = r / share;
      const int strip = MODE == W4_GEGLU ? 2 * (r >> 5) + (r & 1) : r >> 4;
      const int row = MODE == W4_GEGLU ? (r >> 1) & 15 : r & 15;
      const uint32_t dst = smem_u32(part + (rank * a.T + c) * share + r - owner * share);
      st_cluster_u32(mapa_shared(dst, owner), __float_as_uint(w4s_join<NB>(acc, a.lg, strip, c, row)));
    }
  }
  cluster_sync();
  if (sy.aborted()) return;
  if (a.early) pdl_wait();   // the outputs may be what the previous kernel still reads
  const int outs = MODE == W4_GEGLU ? share / 2 : share, wide = 16 * strips_of(first_unit);
  const int n0 = (MODE == W4_GEGLU ? 16 << a.lg : 32 << a.lg) * first_unit;
  for (int i = tid; i < outs * a.T; i += W4S_THREADS) {
    const int r = i % outs, c = i / outs, n = rank * outs + r;
    if (n >= wide) continue;
    float v = 0.f, up = 0.f;
    for (int s = 0; s < a.cluster; ++s) {
      const float* p = part + (s * a.T + c) * share;
      v += p[MODE == W4_GEGLU ? 2 * r : r];
      if (MODE == W4_GEGLU) up += p[2 * r + 1];
    }
    const size_t o = (size_t)c * a.N + n0 + n;
    if (MODE == W4_GEGLU)
      static_cast<__nv_bfloat16*>(a.out)[a.out_frag ? w4_frag_index(a.out_frag, c, n0 + n) : o] =
          __float2bfloat16_rn(w4_geglu(v, up));
    else if (MODE == W4_LINEAR_F32) static_cast<float*>(a.out)[o] = v;
    else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
  }
}

}  // namespace moe
