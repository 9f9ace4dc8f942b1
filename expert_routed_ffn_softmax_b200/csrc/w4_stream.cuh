// w4_stream.cuh -- products of a few activation rows (at most 16) with packed 4-bit weights, as
// one stream of weight bytes: the linear layer, the two halves of the dense GEGLU MLP, and the
// routed experts of a whole MoE layer (w4_moe.cuh) are the same pipeline over different units.
//
// What bounds it.  At T <= 16 a weight byte meets at most 64 flops, so the work is reading the
// weights once at the memory's rate, decoding two weights per byte on the way.  Per SM that is
// about 23 bytes (46 weights) a clock, 45 % of the issue slots for the decode at T <= 8.
//
// Roles of a CTA (13 warps, two CTAs per SM so that one decodes while the other joins or waits):
//   warp 12      producer: copies each unit in chunks of consecutive blocks with bulk copies --
//                one per strip (codes and scales of a strip's run of blocks are contiguous) and
//                one per activation row -- into a ring of stages, up to 90 KB ahead;
//   warps 0-7    multiply: warp = (row group of two strips) x (slice of the blocks along K); a
//                block is one 16-byte shared read per lane, decoded in registers into operands
//                of the matrix instruction (w4_block);
//   warps 8-11   join the K slices' fp32 sums through a double-buffered accumulator tile in
//                shared memory, in a fixed order, and write the outputs, while the multiply
//                warps are at the next unit.
// Every wait is bounded; a wait that runs out sets the device error word and ends the CTA after
// its copies in flight have landed.
#pragma once
#include "gemm_persistent.cuh"
#include "w4.cuh"

namespace moe {

constexpr int W4S_MMA_WARPS = 8, W4S_EPI_WARPS = 4;
constexpr int W4S_THREADS = 32 * (W4S_MMA_WARPS + W4S_EPI_WARPS + 1);
constexpr int W4S_COL = 20;    // floats per accumulator column (16 rows, padded against conflicts)
// Ring stages and their bytes: two CTAs per SM, activation tiles of 8 (NB = 1) or 16 rows.
template <int NB> struct W4Ring;
template <> struct W4Ring<1> { static constexpr int STAGES = 3, BYTES = 30720; };
template <> struct W4Ring<2> { static constexpr int STAGES = 3, BYTES = 23552; };
template <int NB> __host__ __device__ constexpr int w4s_acc_bytes() { return 16 * 8 * NB * W4S_COL * 4; }
constexpr int W4S_MISC = 3072;
template <int NB> __host__ __device__ constexpr int w4s_smem() {
  return W4Ring<NB>::STAGES * W4Ring<NB>::BYTES + 2 * w4s_acc_bytes<NB>() + W4S_MISC;
}

enum W4Mode { W4_LINEAR = 0, W4_LINEAR_F32 = 1, W4_GEGLU = 2, W4_MOE = 3 };

// What a stage holds, written by the producer before the stage's barrier completes: the common
// part, and where each multiply warp finds its share (so that it computes next to nothing).
struct __align__(16) W4Chunk {
  int unit;       // -1: no more work
  int last;       // 1: the unit's last chunk
  int strips;     // strips of the unit
  int lg;         // log2 of the row groups (of two strips) that the multiply warps are split over
  int rows;       // activation rows
  int x_pitch;    // bytes between them
  int slices;     // slices along K: a warp takes every slices-th block
  int pad;
  struct __align__(16) Share {
    uint32_t w;   // first block's record of the first strip
    uint32_t to1; // bytes to the same record of the second strip
    uint32_t x;   // row 0's activations of the first block
    int n;        // blocks
  } share[W4S_MMA_WARPS];
};

struct W4Smem {
  uint32_t bars;          // full[S], empty[S], acc_full[2], acc_empty[2]
  W4Chunk* chunk;         // [S]
  int4* acc_unit;         // [2] {unit, strips, rows, log2 row groups}
  int* abort_flag;
  int* issued;            // chunks issued / consumed, for the drain after a failure
  int* consumed;
  float* acc;             // [2][16][8 NB][W4S_COL]
  int* list;              // the rest of the miscellaneous bytes (routed layer)
};
template <int NB>
__device__ __forceinline__ W4Smem w4s_layout(uint8_t* sm) {
  constexpr int S = W4Ring<NB>::STAGES;
  uint8_t* p = sm + S * W4Ring<NB>::BYTES;
  W4Smem L;
  L.acc = reinterpret_cast<float*>(p);
  p += 2 * w4s_acc_bytes<NB>();
  L.bars = smem_u32(p);
  p += (8 * (2 * S + 4) + 15) / 16 * 16;
  L.chunk = reinterpret_cast<W4Chunk*>(p);
  p += sizeof(W4Chunk) * S;
  L.acc_unit = reinterpret_cast<int4*>(p);
  p += 32;
  L.abort_flag = reinterpret_cast<int*>(p);
  L.issued = L.abort_flag + 1;
  L.consumed = L.abort_flag + 2;
  L.list = L.abort_flag + 4;
  return L;
}
template <int NB>
struct W4Bars {
  static constexpr int S = W4Ring<NB>::STAGES;
  uint32_t base;
  __device__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ uint32_t empty(int s) const { return base + 8u * (S + s); }
  __device__ uint32_t acc_full(int b) const { return base + 8u * (2 * S + b); }
  __device__ uint32_t acc_empty(int b) const { return base + 8u * (2 * S + 2 + b); }
};

template <int NB>
__device__ __forceinline__ void w4s_init(const W4Smem& L) {
  const W4Bars<NB> bar{L.bars};
  for (int s = 0; s < W4Ring<NB>::STAGES; ++s) {
    mbar_init(bar.full(s), 1);
    mbar_init(bar.empty(s), W4S_MMA_WARPS);
  }
  for (int b = 0; b < 2; ++b) {
    mbar_init(bar.acc_full(b), W4S_MMA_WARPS);
    mbar_init(bar.acc_empty(b), W4S_EPI_WARPS);
  }
  *L.abort_flag = 0;
  *L.issued = 0;
  *L.consumed = 0;
  fence_barrier_init();
}

// Bounded wait for warps that wait long and often beside warps that compute: the hint lets the
// hardware park the warp until the phase completes.  Without it a try_wait returns after some 150
// clocks and the waiting warps' loops took 37 % of the SM's instructions (ncu, T = 1).
__device__ __forceinline__ bool w4s_wait(uint32_t bar, uint32_t parity) {
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
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > *reinterpret_cast<volatile unsigned long long*>(&g_wait_limit_ns)) {
      raise_error(MOE_DEVERR_TIMEOUT);
      return false;
    }
  }
}

// Blocks per chunk: as many as fit a stage, evened out over the unit.  Activation rows keep 64
// bytes between them, so that two rows' 64-byte fragments fall in different halves of the banks.
template <int NB, int R>
__device__ __forceinline__ int w4s_chunk_blocks(int kb, int strips, int rows) {
  const int most = (W4Ring<NB>::BYTES - 64 * rows) / (strips * R + 128 * rows);
  const int chunks = (kb + most - 1) / most;
  return (kb + chunks - 1) / chunks;
}

// A unit for the producer: strips' bytes, activation rows.
struct W4Unit {
  const uint8_t *s0, *s1;     // strips 0 and 1 (further strips follow s0 at `pitch`)
  size_t pitch;
  int id, strips, rows, lg, kb;
};

// The producer's side of the ring.
template <int NB, int R>
struct W4Producer {
  const W4Smem& L;
  uint8_t* ring;
  int lane, q = 0;

  // Wait for the next stage, announce the chunk and start its weight copies.  All lanes call.
  __device__ bool weights(const W4Unit& u, int first, int blocks, int qq) {
    constexpr int S = W4Ring<NB>::STAGES;
    const W4Bars<NB> bar{L.bars};
    const int s = qq % S;
    if (*reinterpret_cast<volatile int*>(L.abort_flag) ||
        (qq >= S && !w4s_wait(bar.empty(s), ((qq / S) - 1) & 1)))
      return false;
    const uint32_t at = smem_u32(ring + s * W4Ring<NB>::BYTES);
    if (lane < W4S_MMA_WARPS) {
      // share of multiply warp `lane`: blocks whose index along K is its slice modulo the slices
      const int slices = W4S_MMA_WARPS >> u.lg, group = lane & ((1 << u.lg) - 1), slice = lane >> u.lg;
      const int b = (slice - first) & (slices - 1);
      W4Chunk::Share sh;
      sh.w = at + (2 * group * blocks + b) * R;
      // a unit's odd last strip is multiplied twice; the second sum is not read
      sh.to1 = 2 * group + 1 < u.strips ? blocks * R : 0;
      sh.x = at + u.strips * blocks * R + 128 * b;
      sh.n = 2 * group < u.strips ? (blocks - b + slices - 1) >> (3 - u.lg) : 0;
      L.chunk[s].share[lane] = sh;
      if (lane == 0) {
        int4* c = reinterpret_cast<int4*>(&L.chunk[s]);
        c[0] = make_int4(u.id, first + blocks >= u.kb, u.strips, u.lg);
        c[1] = make_int4(u.rows, 128 * blocks + 64, slices, 0);
        *reinterpret_cast<volatile int*>(L.issued) = qq + 1;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(bar.full(s), (uint32_t)(blocks * (u.strips * R + 128 * u.rows)));
    __syncwarp();
    if (lane < u.strips) {
      const uint8_t* src = (lane == 1 ? u.s1 : u.s0 + lane * u.pitch) + (size_t)first * R;
      bulk_load(at + lane * blocks * R, src, blocks * R, bar.full(s));
    }
    return true;
  }
  // Start the chunk's activation copies (row: this lane's row, for lanes < u.rows).
  __device__ void rows(const W4Unit& u, int first, int blocks, int qq, const __nv_bfloat16* row) {
    constexpr int S = W4Ring<NB>::STAGES;
    const W4Bars<NB> bar{L.bars};
    const int s = qq % S;
    if (lane < u.rows)
      bulk_load(smem_u32(ring + s * W4Ring<NB>::BYTES) + u.strips * blocks * R +
                    lane * (128 * blocks + 64),
                row + 64 * first, 128 * blocks, bar.full(s));
  }
  __device__ bool stop() {
    constexpr int S = W4Ring<NB>::STAGES;
    const W4Bars<NB> bar{L.bars};
    const int s = q % S;
    if (q >= S && !w4s_wait(bar.empty(s), ((q / S) - 1) & 1)) return false;
    if (lane == 0) {
      L.chunk[s].unit = -1;
      mbar_arrive(bar.full(s));
    }
    return true;
  }
};

// Multiply warps.
template <int NB, bool G32, bool ZP>
__device__ __forceinline__ void w4s_multiply(const W4Smem& L, int warp, int lane) {
  constexpr int S = W4Ring<NB>::STAGES;
  constexpr int R = 512 + (G32 ? 2 : 1) * (ZP ? 48 : 32);
  const W4Bars<NB> bar{L.bars};
  const int g = lane >> 2, t = lane & 3;
  const uint32_t chunk_at = smem_u32(L.chunk), acc_at = smem_u32(L.acc);
  float acc[2][NB][4];
#pragma unroll
  for (int i = 0; i < 2 * NB * 4; ++i) acc[i / (4 * NB)][i / 4 % NB][i % 4] = 0.f;
  int n_acc = 0, s = 0;
  uint32_t phase = 0;
  for (int q = 0;; ++q) {
    if (!w4s_wait(bar.full(s), phase)) {
      *reinterpret_cast<volatile int*>(L.abort_flag) = 1;
      return;
    }
    const uint32_t head = chunk_at + s * (uint32_t)sizeof(W4Chunk);
    const uint4 h0 = lds_v4<0>(head), h1 = lds_v4<16>(head);
    const int unit = (int)h0.x, last = h0.y, strips = h0.z, lg = h0.w, rows = h1.x;
    if (warp == 0 && lane == 0) *reinterpret_cast<volatile int*>(L.consumed) = q + 1;
    if (unit >= 0) {
      const uint4 share = lds_v4<32>(head + 16 * warp);
      uint32_t w = share.x + 16 * lane, xr[NB];
      const uint32_t w_step = h1.z * R, x_step = h1.z * 128;
#pragma unroll
      for (int j = 0; j < NB; ++j) xr[j] = share.z + min(g + 8 * j, rows - 1) * h1.y + 16 * t;
#pragma unroll 1
      for (int n = share.w; n > 0; --n) {
        const uint32_t rec[2] = {w, w + share.y};
        w4_block<2, NB, G32, ZP>(acc, rec, lane, xr);
        w += w_step;
#pragma unroll
        for (int j = 0; j < NB; ++j) xr[j] += x_step;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.empty(s));
    }
    if (++s == S) {
      s = 0;
      phase ^= 1;
    }
    if (unit >= 0 && !last) continue;
    // hand the unit's partial sums (or the end) to the joining warps
    const int b = n_acc & 1;
    if (n_acc >= 2 && !w4s_wait(bar.acc_empty(b), ((n_acc >> 1) - 1) & 1)) {
      *reinterpret_cast<volatile int*>(L.abort_flag) = 1;
      return;
    }
    if (warp == 0 && lane == 0) L.acc_unit[b] = make_int4(unit, strips, rows, lg);
    if (unit >= 0) {
      const int group = warp & ((1 << lg) - 1), slice = warp >> lg;
      const uint32_t dst = acc_at + b * w4s_acc_bytes<NB>() +
                           4 * ((((slice << lg) + group) * 16 * NB + 2 * t) * W4S_COL + g);
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
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.acc_full(b));
    if (unit < 0) return;
    ++n_acc;
  }
}

// Sum over the K slices, in slice order, of one accumulator element.
template <int NB>
__device__ __forceinline__ float w4s_join(const float* acc, int lg, int strip, int col, int row) {
  const float* p = acc + (strip * 8 * NB + col) * W4S_COL + row;
  float v = 0.f;
  for (int s = 0; s < W4S_MMA_WARPS >> lg; ++s) v += p[(s * 2 * 8 * NB * W4S_COL) << lg];
  return v;
}

// gelu_tanh(a) * u.  tanh.approx.f32 (documented: relative error 2^-11) is far below the
// rounding of the product to bf16.
__device__ __forceinline__ float w4_geglu(float a, float u) {
  const float th = tanh_approx(0.7978845608028654f * (a + 0.044715f * a * a * a));
  return 0.5f * a * (1.f + th) * u;
}

// After the roles have ended: wait for copies that were issued and not consumed.
template <int NB>
__device__ __forceinline__ void w4s_drain(const W4Smem& L) {
  const W4Bars<NB> bar{L.bars};
  const int to = *reinterpret_cast<volatile int*>(L.issued);
  for (int q = *reinterpret_cast<volatile int*>(L.consumed); q < to; ++q)
    mbar_wait_ns(bar.full(q % W4Ring<NB>::STAGES), (q / W4Ring<NB>::STAGES) & 1, kDrainLimitNs);
}

// ----------------------------------------------------------------------------- linear, GEGLU
struct W4Linear {
  const uint8_t *w0, *w1;       // packed matrix; gate and up for GEGLU
  const __nv_bfloat16* act;     // [T][K]
  void* out;                    // [T][N]
  int T, K, N, lg, units;
  int early;                    // 1: the previous kernel does not write the weights and started
                                // after every kernel before it had ended (dense MLP): the first
                                // weight copies may start before it has ended
};

// Units: 2 << lg strips (GEGLU: the gate and up strips of 16 features), dealt round robin.
template <int NB, bool G32, bool ZP, int MODE>
__global__ void __launch_bounds__(W4S_THREADS, 2) w4_linear_kernel(W4Linear a) {
  constexpr int R = 512 + (G32 ? 2 : 1) * (ZP ? 48 : 32);
  extern __shared__ __align__(128) uint8_t w4sm[];
  const W4Smem L = w4s_layout<NB>(w4sm);
  const W4Bars<NB> bar{L.bars};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) w4s_init<NB>(L);
  __syncthreads();
  if (!a.early) {
    pdl_wait();
    pdl_trigger();
  }
  const int kb = a.K / W4_KB;
  if (warp == W4S_MMA_WARPS + W4S_EPI_WARPS) {
    W4Producer<NB, R> p{L, w4sm, lane};
    // no units when an earlier launch's wait has run out
    int units = 0;
    if (lane == 0 && !(*reinterpret_cast<volatile unsigned*>(&g_error_word) & MOE_DEVERR_TIMEOUT))
      units = a.units;
    units = __shfl_sync(0xffffffffu, units, 0);
    const __nv_bfloat16* row = a.act + (size_t)min(lane, a.T - 1) * a.K;
    bool ok = true, waited = !a.early;
    fence_proxy_async_global();
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      W4Unit un;
      const int s0 = MODE == W4_GEGLU ? u : u << (a.lg + 1);
      un.pitch = (size_t)kb * R;
      un.s0 = a.w0 + s0 * un.pitch;
      un.s1 = MODE == W4_GEGLU ? a.w1 + s0 * un.pitch : un.s0 + un.pitch;
      un.id = u;
      un.strips = MODE == W4_GEGLU ? 2 : min(2 << a.lg, a.N / W4_ROWS - s0);
      un.rows = a.T;
      un.lg = a.lg;
      un.kb = kb;
      const int step = w4s_chunk_blocks<NB, R>(kb, un.strips, un.rows);
      int first = 0;
      if (!waited) {
        // the first stages' weights before the previous kernel has ended, then its rows
        const int pre = min((kb + step - 1) / step, W4Ring<NB>::STAGES);
        for (int i = 0; i < pre && ok; ++i)
          ok = p.weights(un, i * step, min(step, kb - i * step), p.q + i);
        pdl_wait();
        pdl_trigger();
        fence_proxy_async_global();
        waited = true;
        for (int i = 0; i < pre && ok; ++i)
          p.rows(un, i * step, min(step, kb - i * step), p.q + i, row);
        p.q += pre;
        first = pre * step;
      }
      for (; first < kb && ok; first += step) {
        const int n = min(step, kb - first);
        ok = p.weights(un, first, n, p.q);
        if (ok) p.rows(un, first, n, p.q, row);
        ++p.q;
      }
    }
    if (!waited) pdl_wait();
    if (ok) ok = p.stop();
    if (!ok) *reinterpret_cast<volatile int*>(L.abort_flag) = 1;
  } else if (warp < W4S_MMA_WARPS) {
    w4s_multiply<NB, G32, ZP>(L, warp, lane);
  } else {
    const int et = tid - 32 * W4S_MMA_WARPS;
    if (a.early) pdl_wait();   // outputs may be what the previous kernel still reads
    for (int n = 0;; ++n) {
      const int b = n & 1;
      if (!w4s_wait(bar.acc_full(b), (n >> 1) & 1)) {
        *reinterpret_cast<volatile int*>(L.abort_flag) = 1;
        break;
      }
      const int4 u = L.acc_unit[b];
      if (u.x < 0) break;
      const float* acc = L.acc + b * (w4s_acc_bytes<NB>() / 4);
      if (MODE == W4_GEGLU) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
        for (int i = et; i < 16 * a.T; i += 32 * W4S_EPI_WARPS) {
          const int r = i & 15, c = i >> 4;
          const float gt = w4s_join<NB>(acc, u.w, 0, c, r), up = w4s_join<NB>(acc, u.w, 1, c, r);
          out[(size_t)c * a.N + 16 * u.x + r] = __float2bfloat16_rn(w4_geglu(gt, up));
        }
      } else {
        const int wide = 16 * u.y, n0 = (u.x << (a.lg + 1)) * W4_ROWS;
        for (int c = 0; c < a.T; ++c)
          for (int i = et; i < wide; i += 32 * W4S_EPI_WARPS) {
            const float v = w4s_join<NB>(acc, u.w, i >> 4, c, i & 15);
            const size_t o = (size_t)c * a.N + n0 + i;
            if (MODE == W4_LINEAR_F32) static_cast<float*>(a.out)[o] = v;
            else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.acc_empty(b));
    }
  }
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(L.abort_flag) && tid == 0) w4s_drain<NB>(L);
}

}  // namespace moe
