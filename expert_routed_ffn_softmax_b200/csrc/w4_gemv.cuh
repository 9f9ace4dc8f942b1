// w4_gemv.cuh -- products of a few activation rows (at most 16) with packed 4-bit weights.
//
// One CTA of 8 warps computes 32 outputs (two strips of 16; gate and up strips of the same 16
// features for GEGLU) for the rows of one tile: the warps split the blocks along K, each lane
// loads its 16 bytes of codes straight into registers, and the partial sums are added in warp
// order through shared memory.
#pragma once
#include "w4.cuh"

namespace moe {

struct W4Gemv {
  const uint8_t *w0, *w1;          // packed matrices [E]; w1 (up) for GEGLU only
  const __nv_bfloat16* act;        // activation rows of K elements
  void* out;                       // bf16 / fp32 rows of N elements
  const int32_t *tile_num, *tile_expert, *tile_row0, *tile_rows, *perm;   // null: one tile, rows 0..T-1
  const float* weight;             // per pair: the factor of the output row (or null)
  int T, K, N, group, zeros;
  int act_div;                     // activation row of pair q: q / act_div
};

enum W4Out { W4_BF16 = 0, W4_F32 = 1, W4_GEGLU = 2 };

template <int NB, bool G32, bool ZP, int MODE>
__global__ void __launch_bounds__(256) w4_gemv_kernel(W4Gemv a) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[8][2][16][8 * NB + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  int expert = 0, row0 = 0, rows = a.T;
  if (a.tile_num) {
    if ((int)blockIdx.y >= *a.tile_num) return;
    expert = a.tile_expert[blockIdx.y];
    row0 = a.tile_row0[blockIdx.y];
    rows = a.tile_rows[blockIdx.y];
  }
  auto pair_of = [&](int i) { return a.perm ? a.perm[row0 + i] : i; };
  const int kb = a.K / W4_KB, strips = a.N / W4_ROWS;
  constexpr int R = 512 + (G32 ? 2 : 1) * (ZP ? 48 : 32);
  const int s0 = MODE == W4_GEGLU ? blockIdx.x : 2 * blockIdx.x;
  const uint8_t* strip[2];
  strip[0] = a.w0 + ((size_t)expert * strips + s0) * kb * R;
  strip[1] = MODE == W4_GEGLU ? a.w1 + ((size_t)expert * strips + s0) * kb * R : strip[0] + (size_t)kb * R;
  const int ns = MODE == W4_GEGLU ? 2 : min(2, strips - s0);
  const __nv_bfloat16* xr[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
    xr[j] = a.act + (size_t)(pair_of(min(g + 8 * j, rows - 1)) / a.act_div) * a.K + 8 * t;
  float acc[2][NB][4] = {};
  for (int b = warp; b < kb; b += 8) {
    uint4 xf[2][NB];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        xf[h][j] = *reinterpret_cast<const uint4*>(xr[j] + 64 * b + 32 * h);
    for (int s = 0; s < 2; ++s)
      if (s < ns) w4_block<NB, G32, ZP>(acc[s], strip[s] + (size_t)b * R, lane, xf);
  }
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][s][g + 8 * (i >> 1)][8 * j + 2 * t + (i & 1)] = acc[s][j][i];
  __syncthreads();
  const int outs = MODE == W4_GEGLU ? 16 : 16 * ns;
  for (int i = tid; i < outs * rows; i += 256) {
    const int r = i % outs, c = i / outs;
    float v[2] = {0.f, 0.f};
    for (int s = 0; s < (MODE == W4_GEGLU ? 2 : 1); ++s)
      for (int w = 0; w < 8; ++w) v[s] += red[w][MODE == W4_GEGLU ? s : r >> 4][r & 15][c];
    const int q = pair_of(c);
    const size_t o = (size_t)q * a.N + 16 * s0 + r;
    if (MODE == W4_GEGLU) {
      const float u = v[0];
      const float th = tanhf(0.7978845608028654f * (u + 0.044715f * u * u * u));
      static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(0.5f * u * (1.f + th) * v[1]);
    } else if (MODE == W4_F32) {
      static_cast<float*>(a.out)[o] = a.weight ? a.weight[q] * v[0] : v[0];
    } else {
      static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v[0]);
    }
  }
}

// y[t] = sum over the k slots, in slot order, of the weighted fp32 rows o[t k + j].
__global__ void __launch_bounds__(256) w4_combine_kernel(const float* __restrict__ o, int T, int k, int H,
                                                         __nv_bfloat16* __restrict__ y) {
  pdl_trigger();
  pdl_wait();
  for (int i = blockIdx.x * 256 + threadIdx.x; i < T * H; i += gridDim.x * 256) {
    const int t = i / H, n = i - t * H;
    float v = 0.f;
    for (int j = 0; j < k; ++j) v += o[((size_t)t * k + j) * H + n];
    y[i] = __float2bfloat16_rn(v);
  }
}

}  // namespace moe
