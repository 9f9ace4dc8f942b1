// w4_abi.cuh -- the C ABI of the 4-bit weight-only calls (part of moe.cu's translation unit, so
// that these kernels share the device error word with the others).
#pragma once
#include "w4.cuh"
#include "w4_gemv.cuh"

namespace moe {
namespace {

bool w4_group_ok(int group) { return group == 32 || group == 64 || group == 128; }
bool w4_matrix_ok(int K, int N) {
  return K >= 64 && K <= 16384 && K % 64 == 0 && N >= 16 && N <= 1048576 && N % 16 == 0;
}

// Launch a kernel of the (activation tiles, group, zero point) family.
template <int MODE>
void w4_gemv(const Launch& launch, dim3 grid, const W4Gemv& a) {
  auto go = [&](auto kernel) { launch(true, kernel, grid, dim3(256), 0, a); };
  auto by_zero = [&](auto nb, auto g32) {
    if (a.zeros) go(w4_gemv_kernel<decltype(nb)::value, decltype(g32)::value, true, MODE>);
    else go(w4_gemv_kernel<decltype(nb)::value, decltype(g32)::value, false, MODE>);
  };
  auto by_group = [&](auto nb) {
    if (a.group == 32) by_zero(nb, std::true_type{});
    else by_zero(nb, std::false_type{});
  };
  if (a.T <= 8) by_group(std::integral_constant<int, 1>{});
  else by_group(std::integral_constant<int, 2>{});
}

struct W4Layout {
  size_t h = 0, o = 0, total = 0;
};
W4Layout w4_layout(size_t at, size_t pairs, int H, int I, bool routed) {
  W4Layout L;
  L.h = at;
  at = align256(at + 2 * pairs * I);
  L.o = at;
  if (routed) at = align256(at + sizeof(float) * pairs * H);
  L.total = at;
  return L;
}
constexpr unsigned kW4LayerFlags = MOE_FLAG_NO_RENORM | MOE_FLAG_W4_ZEROS;
unsigned w4_router_flags(unsigned flags) { return (flags & MOE_FLAG_NO_RENORM) | MOE_FLAG_ROUTER_FP64; }

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_w4_packed_bytes(int E, int K, int N, int group, unsigned flags) {
  if (E < 1 || E > 4096 || !w4_matrix_ok(K, N) || !w4_group_ok(group) || (flags & ~MOE_FLAG_W4_ZEROS))
    return 0;
  return E * w4_matrix_bytes(K, N, group, flags & MOE_FLAG_W4_ZEROS);
}

moe_status_t moe_w4_pack(const uint8_t* codes, const void* scales, const uint8_t* zeros, int E, int K,
                         int N, int group, void* packed, void* stream) {
  if (E < 0 || K <= 0 || N <= 0 || !w4_group_ok(group)) return MOE_ERR_INVALID_ARG;
  if (E == 0) return MOE_OK;
  if (!codes || !scales || !packed || !aligned16(codes) || !aligned16(packed) ||
      (reinterpret_cast<uintptr_t>(scales) & 1))
    return MOE_ERR_INVALID_ARG;
  if (moe_w4_packed_bytes(E, K, N, group, 0) == 0) return MOE_ERR_UNSUPPORTED;
  int dev = 0;
  if (!device_state(&dev)) return MOE_ERR_CUDA;
  t_kernels = 0;
  const Launch launch{static_cast<cudaStream_t>(stream), false};
  launch(false, w4_pack_kernel, dim3((N + W4_TILE_N - 1) / W4_TILE_N, (K + W4_TILE_K - 1) / W4_TILE_K, E),
         dim3(256), 0, codes, static_cast<const __nv_bfloat16*>(scales), zeros, K, N, group,
         static_cast<uint8_t*>(packed));
  return launched();
}

moe_status_t moe_w4_quantize_weights(const void* w, int E, int K, int N, int group, unsigned flags,
                                     void* packed, void* stream) {
  if (E < 0 || K <= 0 || N <= 0 || !w4_group_ok(group) || (flags & ~MOE_FLAG_W4_ZEROS))
    return MOE_ERR_INVALID_ARG;
  if (E == 0) return MOE_OK;
  if (!w || !packed || !aligned16(w) || !aligned16(packed)) return MOE_ERR_INVALID_ARG;
  if (moe_w4_packed_bytes(E, K, N, group, flags) == 0) return MOE_ERR_UNSUPPORTED;
  int dev = 0;
  if (!device_state(&dev)) return MOE_ERR_CUDA;
  t_kernels = 0;
  const Launch launch{static_cast<cudaStream_t>(stream), false};
  launch(false, (flags & MOE_FLAG_W4_ZEROS) ? w4_quantize_kernel<true> : w4_quantize_kernel<false>,
         dim3((N + W4_TILE_N - 1) / W4_TILE_N, (K + W4_TILE_K - 1) / W4_TILE_K, E), dim3(256), 0,
         static_cast<const __nv_bfloat16*>(w), K, N, group, static_cast<uint8_t*>(packed));
  return launched();
}

moe_status_t moe_w4_dequantize_weights(const void* packed, int E, int K, int N, int group,
                                       unsigned flags, void* w, void* stream) {
  if (E < 0 || K <= 0 || N <= 0 || !w4_group_ok(group) || (flags & ~MOE_FLAG_W4_ZEROS))
    return MOE_ERR_INVALID_ARG;
  if (E == 0) return MOE_OK;
  if (!w || !packed || !aligned16(w) || !aligned16(packed)) return MOE_ERR_INVALID_ARG;
  if (moe_w4_packed_bytes(E, K, N, group, flags) == 0) return MOE_ERR_UNSUPPORTED;
  int dev = 0;
  if (!device_state(&dev)) return MOE_ERR_CUDA;
  t_kernels = 0;
  const Launch launch{static_cast<cudaStream_t>(stream), false};
  launch(false, w4_dequantize_kernel,
         dim3((N + W4_TILE_N - 1) / W4_TILE_N, (K + W4_TILE_K - 1) / W4_TILE_K, E), dim3(256), 0,
         static_cast<const uint8_t*>(packed), K, N, group, (flags & MOE_FLAG_W4_ZEROS) ? 1 : 0,
         static_cast<__nv_bfloat16*>(w));
  return launched();
}

moe_status_t moe_linear_w4(const void* x, const void* w, int T, int K, int N, int group,
                           unsigned flags, void* y, void* stream) {
  if (T < 0 || K <= 0 || N <= 0 || !w4_group_ok(group) ||
      (flags & ~(MOE_FLAG_W4_ZEROS | MOE_FLAG_F32_OUT)))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w || !y || !aligned16(x) || !aligned16(w) || !aligned16(y) || x == y)
    return MOE_ERR_INVALID_ARG;
  if (T > W4_MAX_T || !w4_matrix_ok(K, N)) return MOE_ERR_UNSUPPORTED;
  int dev = 0;
  if (!device_state(&dev)) return MOE_ERR_CUDA;
  t_kernels = 0;
  W4Gemv a = {};
  a.w0 = static_cast<const uint8_t*>(w);
  a.act = static_cast<const __nv_bfloat16*>(x);
  a.out = y;
  a.T = T;
  a.K = K;
  a.N = N;
  a.group = group;
  a.zeros = (flags & MOE_FLAG_W4_ZEROS) ? 1 : 0;
  a.act_div = 1;
  const Launch launch{static_cast<cudaStream_t>(stream), true};
  const dim3 grid((N + 31) / 32);
  if (flags & MOE_FLAG_F32_OUT) w4_gemv<W4_F32>(launch, grid, a);
  else w4_gemv<W4_BF16>(launch, grid, a);
  return launched();
}

size_t moe_dense_w4_workspace_size(int T, int H, int I) {
  if (T < 1 || T > W4_MAX_T || H < 64 || H > 16384 || H % 64 || I < 64 || I > 8192 || I % 64) return 0;
  return w4_layout(0, T, H, I, false).total;
}

moe_status_t moe_dense_ffn_w4(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                              int T, int H, int I, int group, unsigned flags, void* y,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || H <= 0 || I <= 0 || !w4_group_ok(group) || (flags & ~MOE_FLAG_W4_ZEROS))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w_gate || !w_up || !w_down || !y || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down) ||
      !aligned16(y) || !aligned16(workspace) || x == y)
    return MOE_ERR_INVALID_ARG;
  if (moe_dense_w4_workspace_size(T, H, I) == 0) return MOE_ERR_UNSUPPORTED;
  const W4Layout L = w4_layout(0, T, H, I, false);
  if (workspace_bytes < L.total) return MOE_ERR_NO_WORKSPACE;
  int dev = 0;
  if (!device_state(&dev)) return MOE_ERR_CUDA;
  t_kernels = 0;
  const Launch launch{static_cast<cudaStream_t>(stream), true};
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(workspace) + L.h);
  W4Gemv a = {};
  a.w0 = static_cast<const uint8_t*>(w_gate);
  a.w1 = static_cast<const uint8_t*>(w_up);
  a.act = static_cast<const __nv_bfloat16*>(x);
  a.out = h;
  a.T = T;
  a.K = H;
  a.N = I;
  a.group = group;
  a.zeros = (flags & MOE_FLAG_W4_ZEROS) ? 1 : 0;
  a.act_div = 1;
  w4_gemv<W4_GEGLU>(launch, dim3(I / 16), a);
  if (const moe_status_t s = launched(); s != MOE_OK) return s;
  a.w0 = static_cast<const uint8_t*>(w_down);
  a.w1 = nullptr;
  a.act = h;
  a.out = y;
  a.K = I;
  a.N = H;
  w4_gemv<W4_BF16>(launch, dim3((H + 31) / 32), a);
  return launched();
}

size_t moe_w4_workspace_size(int T, int H, int E, int I, int k, unsigned flags) {
  if ((flags & ~kW4LayerFlags) || T > W4_MAX_T || !shape_supported(T, H, E, I, k, true)) return 0;
  return w4_layout(make_layout(T, H, E, I, k, w4_router_flags(flags), true).total, (size_t)T * k, H, I,
                   true)
      .total;
}

moe_status_t moe_forward_w4(const void* x, const void* w_router, const float* router_bias,
                            const void* w_gate, const void* w_up, const void* w_down, int T, int H,
                            int E, int I, int k, int group, unsigned flags, void* y,
                            const moe_aux_t* aux, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (T < 0 || H <= 0 || E <= 0 || I <= 0 || k < 1 || k > E || !w4_group_ok(group) ||
      (flags & ~kW4LayerFlags))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !w_gate || !w_up || !w_down || !y || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(w_gate) || !aligned16(w_up) ||
      !aligned16(w_down) || !aligned16(y) || !aligned16(workspace) || x == y)
    return MOE_ERR_INVALID_ARG;
  if (moe_w4_workspace_size(T, H, E, I, k, flags) == 0) return MOE_ERR_UNSUPPORTED;
  const unsigned rflags = w4_router_flags(flags);
  const Layout L = make_layout(T, H, E, I, k, rflags, true);
  const W4Layout W = w4_layout(L.total, (size_t)T * k, H, I, true);
  if (workspace_bytes < W.total) return MOE_ERR_NO_WORKSPACE;
  int dev = 0;
  DeviceState* d = device_state(&dev);
  if (!d) return MOE_ERR_CUDA;
  t_kernels = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* ids = (aux && aux->topk_ids) ? aux->topk_ids : reinterpret_cast<int32_t*>(ws + L.ids);
  float* wts = (aux && aux->topk_weights) ? aux->topk_weights : reinterpret_cast<float*>(ws + L.wts);
  int32_t* counts =
      (aux && aux->expert_counts) ? aux->expert_counts : reinterpret_cast<int32_t*>(ws + L.counts);
  int32_t* offsets = (aux && aux->expert_offsets) ? aux->expert_offsets
                                                  : reinterpret_cast<int32_t*>(ws + L.offsets);
  int32_t* perm = (aux && aux->perm) ? aux->perm : reinterpret_cast<int32_t*>(ws + L.perm);
  unsigned* stats = (aux && aux->router_stats) ? aux->router_stats
                                               : reinterpret_cast<unsigned*>(ws + L.stats);
  int32_t* inv = reinterpret_cast<int32_t*>(ws + L.inv);
  Profiler prof{d, st, false};
  const RouteBufs rb{ids, wts, stats, counts, offsets, perm, inv};
  if (const moe_status_t rs = route_and_dispatch(x, w_router, router_bias, T, H, E, k, rflags, rb, ws,
                                                 L, *d, st, prof, false);
      rs != MOE_OK)
    return rs;
  const Launch launch{st, true};
  W4Gemv a = {};
  a.w0 = static_cast<const uint8_t*>(w_gate);
  a.w1 = static_cast<const uint8_t*>(w_up);
  a.act = static_cast<const __nv_bfloat16*>(x);
  a.out = ws + W.h;
  a.tile_num = reinterpret_cast<int32_t*>(ws + L.tile_num);
  a.tile_expert = reinterpret_cast<int32_t*>(ws + L.tile_expert);
  a.tile_row0 = reinterpret_cast<int32_t*>(ws + L.tile_row0);
  a.tile_rows = reinterpret_cast<int32_t*>(ws + L.tile_rows);
  a.perm = perm;
  a.T = T;
  a.K = H;
  a.N = I;
  a.group = group;
  a.zeros = (flags & MOE_FLAG_W4_ZEROS) ? 1 : 0;
  a.act_div = k;
  const int tiles = std::min(E, T * k);
  w4_gemv<W4_GEGLU>(launch, dim3(I / 16, tiles), a);
  if (const moe_status_t s = launched(); s != MOE_OK) return s;
  a.w0 = static_cast<const uint8_t*>(w_down);
  a.w1 = nullptr;
  a.act = reinterpret_cast<const __nv_bfloat16*>(ws + W.h);
  a.out = ws + W.o;
  a.weight = wts;
  a.K = I;
  a.N = H;
  a.act_div = 1;
  w4_gemv<W4_F32>(launch, dim3((H + 31) / 32, tiles), a);
  if (const moe_status_t s = launched(); s != MOE_OK) return s;
  launch(true, w4_combine_kernel, dim3((T * H + 255) / 256), dim3(256), 0,
         reinterpret_cast<const float*>(ws + W.o), T, k, H, static_cast<__nv_bfloat16*>(y));
  return launched();
}

}  // extern "C"
