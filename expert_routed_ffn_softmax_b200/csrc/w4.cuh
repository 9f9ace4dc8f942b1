// w4.cuh -- 4-bit weights with one bf16 scale (and optionally one zero point) per group of
// 32, 64 or 128 consecutive elements along the reduction axis, activations left in bf16:
//
//     value(n, k) = (code(n, k) - zero(n, k / group)) * scale(n, k / group)
//
// with code and zero in 0..15 (zero = 8 everywhere in the symmetric form).
//
// This file holds the packed layout, the way into it (from bf16 weights or from a checkpoint's
// codes and scales), the way back to bf16, and the 16-row x 64-deep product of one packed block
// with up to 16 activation rows that the few-token kernels are built from.
//
// Packed layout.  A matrix of N outputs and reduction depth K is cut into strips of 16 rows
// (outputs) and blocks of 64 elements along K; record (strip, block) holds everything the
// block's product needs, so that a strip is one contiguous byte range and any run of its
// blocks is one bulk copy:
//   512 bytes of codes: 16 bytes per lane of the warp that multiplies the block.  Lane
//       l = 4 g + t holds rows g and g + 8, elements 8 t .. 8 t + 7 of each 32-element half:
//       words (row g, half 0), (row g + 8, half 0), (row g, half 1), (row g + 8, half 1).  In a
//       word, nibble i < 4 is element 2 i and nibble 4 + i is element 2 i + 1, so that one mask
//       leaves a pair of neighbours in the halves of a register, as the operands of the matrix
//       instruction want them.
//   then 32 bytes per group of the block (two groups of 32, else one): bf16 scales, rows
//       interleaved 0, 8, 1, 9, .. 7, 15 (one 4-byte read gives a lane both of its rows);
//       a 128-element group repeats its scales in both of its blocks (3 % of the bytes, in
//       return for blocks that stand alone);
//   then, asymmetric form only, 16 bytes per group of the block: zero points, same row order.
#pragma once
#include "ptx.cuh"

namespace moe {

constexpr int W4_ROWS = 16;      // rows of a strip
constexpr int W4_KB = 64;        // elements of a block along K
constexpr int W4_MAX_T = 16;     // activation rows of the few-token kernels

// Groups of one block, and the bytes of one record.
__host__ __device__ constexpr int w4_groups(int group) { return group == 32 ? 2 : 1; }
__host__ __device__ constexpr int w4_record(int group, bool zeros) {
  return 512 + w4_groups(group) * (zeros ? 48 : 32);
}
__host__ __device__ inline size_t w4_matrix_bytes(int K, int N, int group, bool zeros) {
  return (size_t)(N / W4_ROWS) * (K / W4_KB) * w4_record(group, zeros);
}

// Eight codes in element order (element j in nibble j) -> the word order above.
__device__ __forceinline__ uint32_t w4_interleave(uint32_t w) {
  auto squeeze = [](uint32_t v) {   // nibbles 0, 2, 4, 6 of v -> nibbles 0..3
    v &= 0x0F0F0F0Fu;
    v = (v | (v >> 4)) & 0x00FF00FFu;
    return (v | (v >> 8)) & 0xFFFFu;
  };
  return squeeze(w) | (squeeze(w >> 4) << 16);
}
// Position of row r (0..15) in a group's scales and zero points.
__device__ __forceinline__ int w4_row_slot(int r) { return 2 * (r & 7) + (r >> 3); }

// ----------------------------------------------------------------------------- into the layout
// A tile of the packing kernels: 64 rows x 128 elements (4 strips x 2 blocks; ragged at the
// matrix's ends), assembled in shared memory and written as runs of two records per strip.
constexpr int W4_TILE_N = 64, W4_TILE_K = 128;
// Bytes between a tile's records: an odd number of 16s, so that strips fall in different banks (a
// warp's stores of codes met 16 deep at 576 bytes: the quantiser took 193 us instead of 169 for 128
// matrices of 2816 x 704).
__host__ __device__ constexpr int w4_tile_pitch(int record) { return record | 16; }
constexpr int W4_TILE_BYTES = 4 * 2 * w4_tile_pitch(608);

// A record of tile (n0, k0) of matrix `e` for each of 8 warps: strip warp / 2, block warp % 2 (false
// past the matrix's ends); `at` is its offset in the packed matrices, `in_tile` its offset in the tile.
__device__ __forceinline__ bool w4_tile_record(int e, int n0, int k0, int K, int N, int R, size_t& at,
                                               int& in_tile) {
  const int warp = threadIdx.x >> 5, strip = n0 / W4_ROWS + (warp >> 1), block = k0 / W4_KB + (warp & 1);
  at = (((size_t)e * (N / W4_ROWS) + strip) * (K / W4_KB) + block) * R;
  in_tile = warp * w4_tile_pitch(R);
  return strip < N / W4_ROWS && block < K / W4_KB;
}
// Write the assembled records [strip][block][R].
__device__ __forceinline__ void w4_store_tile(const uint8_t* rec, uint8_t* packed, int e, int n0,
                                              int k0, int K, int N, int R) {
  size_t at;
  int in_tile;
  if (w4_tile_record(e, n0, k0, K, N, R, at, in_tile))
    for (int v = 16 * (threadIdx.x & 31); v < R; v += 512)
      *reinterpret_cast<uint4*>(packed + at + v) = *reinterpret_cast<const uint4*>(rec + in_tile + v);
}

// codes uint8 [E][N][K/2] (element 2b in the low nibble of byte b), scales bf16 [E][N][G],
// zeros uint8 [E][N][G] or null (G = ceil(K / group)) -> packed.  Only the low nibble of a zero
// point is kept.  Each thread moves 16 bytes (32 codes of one row), so a row gives a tile 64 bytes, half
// a line.  128 matrices of 2816 x 704: 79 us with groups of 32 or 64, 81 with zero points (3.4 to 3.7 of
// the memory's 6.55 TB/s); one of 2816 x 2112 3.6 us.  Run once a checkpoint, so it is left at that.
__global__ void __launch_bounds__(256) w4_pack_kernel(const uint8_t* __restrict__ codes,
                                                      const __nv_bfloat16* __restrict__ scales,
                                                      const uint8_t* __restrict__ zeros, int K,
                                                      int N, int group, uint8_t* __restrict__ packed) {
  __shared__ __align__(16) uint8_t rec[W4_TILE_BYTES];
  const bool zp = zeros != nullptr;
  const int R = w4_record(group, zp), gpb = w4_groups(group), G = (K + group - 1) / group;
  const int n0 = blockIdx.x * W4_TILE_N, k0 = blockIdx.y * W4_TILE_K, e = blockIdx.z;
  const int row = threadIdx.x >> 2, part = threadIdx.x & 3;   // 32 elements of one row
  const int n = n0 + row, k = k0 + 32 * part;
  if (n < N && k < K) {
    const size_t at = (size_t)e * N + n;
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(codes + at * (K / 2) + k / 2));
    const int strip = row >> 4, r = row & 15, block = part >> 1, half = part & 1;
    uint8_t* b = rec + (strip * 2 + block) * w4_tile_pitch(R);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int t = 0; t < 4; ++t)
      *reinterpret_cast<uint32_t*>(b + 16 * (4 * (r & 7) + t) + 8 * half + 4 * (r >> 3)) =
          w4_interleave(w[t]);
    if (half == 0 || gpb == 2) {
      const int gi = half * (gpb - 1);
      const size_t ga = at * G + k / group;
      reinterpret_cast<__nv_bfloat16*>(b + 512)[gi * 16 + w4_row_slot(r)] = scales[ga];
      if (zp) b[512 + gpb * 32 + gi * 16 + w4_row_slot(r)] = zeros[ga] & 15;
    }
  }
  __syncthreads();
  w4_store_tile(rec, packed, e, n0, k0, K, N, R);
}

// Decoding.  A pair of codes becomes a pair of exact bf16 values (code - zero) / 4 in one logical
// operation and one fused multiply-add; the 4 is put back where the sums are joined.  The logical pipe is
// the scarce one (half the issue rate), so the shifts are kept to one per eight codes:
//   nibbles 0 and 4 of a word: OR with 0x4300 makes 128 + code (whose unit in the last place is
//       1), times 1/4, minus (128 + zero) / 4;
//   nibbles 1 and 5 stay where they are: a bf16 with nothing above bit 7 is its low byte times
//       2^-133, also when that is subnormal, so the masked pair is code * 2^-129; times 2^127,
//       minus zero / 4;
//   nibbles 2, 6 and 3, 7: the same after a shift by 8.
struct W4Zero {
  uint32_t a, b;   // -(128 + zero) / 4 and -zero / 4, in both halves
};
constexpr uint32_t W4_QUARTER = 0x3E803E80u, W4_2P127 = 0x7F007F00u;
__device__ __forceinline__ uint32_t w4_fma(uint32_t v, uint32_t m, uint32_t a) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(m), "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t w4_low(uint32_t word, const W4Zero& z) {
  return w4_fma((word & 0x000F000Fu) | 0x43004300u, W4_QUARTER, z.a);
}
__device__ __forceinline__ uint32_t w4_high(uint32_t word, const W4Zero& z) {
  return w4_fma(word & 0x00F000F0u, W4_2P127, z.b);
}
// The subtrahends for a zero point in the low byte of `zero` (8 when symmetric).
__device__ __forceinline__ W4Zero w4_zero(uint32_t zero) {
  W4Zero z;
  z.a = zero * 0x00010001u + 0xC200C200u;                     // -(32 + zero / 4)
  z.b = w4_fma(z.a, 0x3F803F80u /* 1 */, 0x42004200u /* 32 */);
  return z;
}

// A tile of bf16 weights in shared memory, [128 along K][64 rows], 8 elements of padding.  In the
// two kernels below a thread has 16 elements along K of two neighbouring rows.
__device__ __forceinline__ uint32_t* w4_word(uint8_t* rec, int R, int row, int part, int i) {
  const int r = row & 15;
  return reinterpret_cast<uint32_t*>(rec + ((row >> 4) * 2 + (part >> 2)) * R +
                                     16 * (4 * (r & 7) + 2 * (part & 1) + i) + 8 * ((part >> 1) & 1) +
                                     4 * (r >> 3));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 w4_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 w4_add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// rint(x / s) with the correctly rounded quotient; 0 unless s is positive and finite.  Out of line:
// rarely needed.
__device__ __noinline__ float w4_rounded_quotient(float x, float s) {
  return s > 0.f && s < INFINITY ? rintf(__fdiv_rn(x, s)) : 0.f;
}

// bf16 weights w [E][K][N] (N contiguous) -> packed.  Per group, in fp32, every step one
// rounding to nearest even: symmetric scale = bf16(max |w| / 7), code = clamp(rint(w / scale)
// + 8, 0, 15); asymmetric lo = min(w, 0), hi = max(w, 0), scale = bf16((hi - lo) / 15), zero =
// clamp(rint(-lo / scale), 0, 15), code = clamp(rint(w / scale) + zero, 0, 15).  A scale that is
// zero, infinite or NaN gives codes and zero points of 8.  The extremes propagate NaN, so a group
// with a NaN or an infinity has such a scale, whose product with 8 - 8 is NaN for all of the group.
//
// Bound by its instructions (11 a weight), then its bytes (2.5 to 2.6 a weight): a warp reads two
// rows a lane, whole lines along N, straight into registers (through shared memory it took 169 us for
// 128 matrices of 2816 x 704, so 143: 4.5 TB/s); 48 registers keep 40 warps on an SM (63 did with
// zero points: 172 us, so 160); the division is a multiplication by the reciprocal, within 2^-19 of the
// quotient (at most 16); adding 1.5 * 2^23 rounds to an integer in the low bits, and eight of those
// add up to a packed word when the constant parts are taken off at the end.  The product rounds
// like the quotient once it has been rounded to a multiple of 2^-11 (fused with the product, by an
// addend of 1.5 * 2^12, which the second addition takes off again): a weight a 2^i and a scale b 2^j
// have 8-bit a and b, so a quotient either is a half-integer h or differs from it by at least
// 2^(j-2) / (b 2^j) > 2^-10.
template <bool ZP>
__global__ void __launch_bounds__(256, 5) w4_quantize_kernel(const __nv_bfloat16* __restrict__ w, int K,
                                                          int N, int group,
                                                          uint8_t* __restrict__ packed) {
  __shared__ __align__(16) uint8_t rec[W4_TILE_BYTES];
  __shared__ __nv_bfloat162 s_lo[8][32], s_hi[8][32];
  const int R = w4_record(group, ZP), pitch = w4_tile_pitch(R), gpb = w4_groups(group);
  const int n0 = blockIdx.x * W4_TILE_N, k0 = blockIdx.y * W4_TILE_K, e = blockIdx.z;
  const int pair = threadIdx.x & 31, part = threadIdx.x >> 5;   // rows 2 pair, + 1; k 16 part .. + 15
  const bool in = n0 + 2 * pair < N && k0 + 16 * part < K;
  const __nv_bfloat16* src = w + ((size_t)e * K + k0 + 16 * part) * N + n0 + 2 * pair;
  __nv_bfloat162 v[16];
  __nv_bfloat162 lo = __float2bfloat162_rn(0.f), hi = lo;
  if (in) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t two = __ldg(reinterpret_cast<const uint32_t*>(src + (size_t)i * N));
      v[i] = *reinterpret_cast<const __nv_bfloat162*>(&two);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      lo = __hmin2_nan(lo, v[i]);
      hi = __hmax2_nan(hi, v[i]);
    }
  }
  s_lo[part][pair] = lo;
  s_hi[part][pair] = hi;
  __syncthreads();
  if (in) {
    const int span = group / 16, p0 = part / span * span;   // the 16-element parts of the group
    for (int i = p0; i < p0 + span; ++i) {
      lo = __hmin2_nan(lo, s_lo[i][pair]);
      hi = __hmax2_nan(hi, s_hi[i][pair]);
    }
    constexpr float SNAP = 6144.f;                        // 1.5 * 2^12
    constexpr float ROUND = 12582912.f;                   // 1.5 * 2^23
    constexpr uint32_t BITS = 0x4B400000u;                // its bits
    __nv_bfloat16 sb[2];
    float s[2], inv[2];
    int z[2];
    uint32_t word[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float l = c ? __high2float(lo) : __low2float(lo), h = c ? __high2float(hi) : __low2float(hi);
      sb[c] = __float2bfloat16_rn(ZP ? __fdiv_rn(__fsub_rn(h, l), 15.f) : __fdiv_rn(fmaxf(-l, h), 7.f));
      s[c] = __bfloat162float(sb[c]);
      inv[c] = __fdiv_rn(1.f, s[c]);
      z[c] = ZP && s[c] > 0.f && s[c] < INFINITY ? (int)fminf(fmaxf(rintf(__fdiv_rn(-l, s[c])), 0.f), 15.f) : 8;
      word[c][0] = word[c][1] = ((uint32_t)z[c] - BITS) * 0x11111111u;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t x2 = *reinterpret_cast<const uint32_t*>(&v[i]);
      float2 q = w4_fma2(make_float2(__uint_as_float(x2 << 16), __uint_as_float(x2 & 0xffff0000u)),
                         make_float2(inv[0], inv[1]), make_float2(SNAP, SNAP));
      q = w4_add2(q, make_float2(ROUND - SNAP, ROUND - SNAP));
      uint32_t bits[2] = {__float_as_uint(q.x), __float_as_uint(q.y)};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // the rounding of the scale can leave the largest quotient at 16 - zero
        if (ZP) bits[c] = min(bits[c], BITS + 15u - (uint32_t)z[c]);
        word[c][i >> 3] += bits[c] << (4 * (((i & 7) >> 1) + 4 * (i & 1)));
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 2 * pair + c;
      if (!(s[c] > 1e-30f && s[c] < 1e30f)) {   // 0, subnormal, infinite or NaN, now or as a reciprocal: by division
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          uint32_t exact = 0;
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const float x = __bfloat162float(src[(size_t)(8 * u + i) * N + c]);
            const float q = w4_rounded_quotient(x, s[c]) + (float)z[c];
            exact |= (uint32_t)(int)fminf(fmaxf(q, 0.f), 15.f) << (4 * ((i >> 1) + 4 * (i & 1)));
          }
          if (u) word[c][1] = exact;
          else word[c][0] = exact;
        }
      }
      *w4_word(rec, pitch, row, part, 0) = word[c][0];
      *w4_word(rec, pitch, row, part, 1) = word[c][1];
      if ((part & (gpb == 2 ? 1 : 3)) == 0) {
        uint8_t* b = rec + ((row >> 4) * 2 + (part >> 2)) * pitch;
        const int at = ((part >> 1) & (gpb - 1)) * 16 + w4_row_slot(row & 15);
        reinterpret_cast<__nv_bfloat16*>(b + 512)[at] = sb[c];
        if (ZP) b[512 + gpb * 32 + at] = (uint8_t)z[c];
      }
    }
  }
  __syncthreads();
  w4_store_tile(rec, packed, e, n0, k0, K, N, R);
}

// packed -> bf16 w [E][K][N]: each value rounded once.  Bound by its bytes (110 us, 5.9 TB/s, for
// 128 matrices of 2816 x 704 with groups of 32): codes are decoded in pairs as the products do (a
// quarter of the difference, exact), times 4, times the scale, and a warp writes whole lines from
// registers.
__global__ void __launch_bounds__(256) w4_dequantize_kernel(const uint8_t* __restrict__ packed, int K,
                                                            int N, int group, int zeros,
                                                            __nv_bfloat16* __restrict__ w) {
  __shared__ __align__(16) uint8_t rec[W4_TILE_BYTES];
  const int R = w4_record(group, zeros), pitch = w4_tile_pitch(R), gpb = w4_groups(group);
  const int n0 = blockIdx.x * W4_TILE_N, k0 = blockIdx.y * W4_TILE_K, e = blockIdx.z;
  const int strips = min(4, (N - n0) / W4_ROWS), blocks = min(2, (K - k0) / W4_KB);
  size_t from;
  int in_tile;
  if (w4_tile_record(e, n0, k0, K, N, R, from, in_tile))
    for (int v = 16 * (threadIdx.x & 31); v < R; v += 512)
      *reinterpret_cast<uint4*>(rec + in_tile + v) = __ldg(reinterpret_cast<const uint4*>(packed + from + v));
  __syncthreads();
  const int pair = threadIdx.x & 31, part = threadIdx.x >> 5;
  if (2 * pair < 16 * strips && part < 4 * blocks) {
    uint32_t val[2][8];   // per row, pairs along K
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 2 * pair + c;
      const uint8_t* b = rec + ((row >> 4) * 2 + (part >> 2)) * pitch;
      const int at = ((part >> 1) & (gpb - 1)) * 16 + w4_row_slot(row & 15);
      const uint32_t s2 = reinterpret_cast<const uint16_t*>(b + 512)[at] * 0x00010001u;
      const W4Zero z = w4_zero(zeros ? b[512 + gpb * 32 + at] : 8u);
      const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&s2), four = __float2bfloat162_rn(4.f);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t word = *w4_word(rec, pitch, row, part, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t d = i & 1 ? w4_high(word >> (4 * (i - 1)), z) : w4_low(word >> (4 * i), z);
          const __nv_bfloat162 q = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&d), four), s);
          val[c][4 * u + i] = *reinterpret_cast<const uint32_t*>(&q);
        }
      }
    }
    __nv_bfloat16* dst = w + ((size_t)e * K + k0 + 16 * part) * N + n0 + 2 * pair;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      *reinterpret_cast<uint32_t*>(dst + (size_t)(2 * i) * N) = __byte_perm(val[0][i], val[1][i], 0x5410);
      *reinterpret_cast<uint32_t*>(dst + (size_t)(2 * i + 1) * N) = __byte_perm(val[0][i], val[1][i], 0x7632);
    }
  }
}

// ----------------------------------------------------------------------------- the block product
// D = A B (+ D unless `clear`, a constant) for 16 x 16 A (row-major), 16 x 8 B, bf16 in, fp32 accumulation.  tcgen05.mma would
// need the decoded weights in shared or tensor memory: a write and a read of four times the
// bytes that arrive.  Here a lane decodes its 16 bytes in registers, which are already the
// instruction's operand, and at 16 activation rows the products are far from either rate.
// (Not volatile: the compiler may interleave independent chains.)
__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1, bool clear) {
  const float c0 = clear ? 0.f : d[0], c1 = clear ? 0.f : d[1];
  const float c2 = clear ? 0.f : d[2], c3 = clear ? 0.f : d[3];
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Reads at a byte offset into the kernel's dynamic shared memory (named, so that the compiler knows
// the address space and folds constant offsets into the load).
extern __shared__ __align__(128) uint8_t w4sm[];
template <typename V>
__device__ __forceinline__ V lds(uint32_t off) {
  return *reinterpret_cast<const V*>(w4sm + off);
}

// acc[i][j] += block i * activation fragments, for the records of NS strips at the same place
// along K, in shared memory: rec[i] = the record's offset + 16 lane.  x[j]: the offset of the
// lane's 8 activations of the first half (elements 8 t .. + 7 of row g + 8 j, for lane 4 g + t);
// those of the second half are x_half bytes on.
// acc[i][j]: (row g, activation rows 8 j + 2 t and + 1), (row g + 8, the same).  The products of
// a group are exact integers (over 4) times bf16, summed in fp32 by the matrix instruction; the
// scale is applied once per group, in fp32, so nothing is rounded to bf16 on the way.
template <int NS, int NB, bool G32, bool ZP>
__device__ __forceinline__ void w4_block(float (&acc)[NS][NB][4], const uint32_t (&rec)[NS], int lane,
                                         const uint32_t (&x)[NB], uint32_t x_half) {
  constexpr int GPB = G32 ? 2 : 1;
  uint4 q[NS];
  uint32_t sc[NS], zp[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    q[i] = lds<uint4>(rec[i]);
    sc[i] = rec[i] - 16 * lane + 4 * (lane >> 2);         // this lane's two rows' scales,
    if (ZP) zp[i] = rec[i] - 16 * lane + 2 * (lane >> 2);   // and zero points
  }
  float p[NS][NB][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 xf[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) xf[j] = lds<uint4>(h ? x[j] + x_half : x[j]);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const uint32_t lo = h ? q[i].z : q[i].x, hi = h ? q[i].w : q[i].y;
      W4Zero z_lo = {0xC208C208u, 0xC000C000u}, z_hi = z_lo;   // zero points of 8
      if (ZP) {
        const uint32_t two = lds<uint16_t>(zp[i] + 512 + GPB * 32 + (G32 ? 16 * h : 0));
        z_lo = w4_zero(two & 0xffu);
        z_hi = w4_zero(two >> 8);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t wl = s ? lo >> 8 : lo, wh = s ? hi >> 8 : hi;
        const uint32_t a0 = w4_low(wl, z_lo), a1 = w4_low(wh, z_hi);
        const uint32_t a2 = w4_high(wl, z_lo), a3 = w4_high(wh, z_hi);
#pragma unroll
        for (int j = 0; j < NB; ++j)
          w4_mma(p[i][j], a0, a1, a2, a3, s ? xf[j].z : xf[j].x, s ? xf[j].w : xf[j].y,
                 s == 0 && (G32 || h == 0));
      }
      if (G32 || h == 1) {
        const uint32_t s2 = lds<uint32_t>(sc[i] + 512 + (G32 ? 32 * h : 0));
        const float s_lo = __uint_as_float(s2 << 16), s_hi = __uint_as_float(s2 & 0xffff0000u);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          acc[i][j][0] = fmaf(s_lo, p[i][j][0], acc[i][j][0]);
          acc[i][j][1] = fmaf(s_lo, p[i][j][1], acc[i][j][1]);
          acc[i][j][2] = fmaf(s_hi, p[i][j][2], acc[i][j][2]);
          acc[i][j][3] = fmaf(s_hi, p[i][j][3], acc[i][j][3]);
        }
      }
    }
  }
}

}  // namespace moe
