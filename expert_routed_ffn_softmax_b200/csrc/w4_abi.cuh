// w4_abi.cuh -- the C ABI of the 4-bit weight-only calls (part of moe.cu's translation unit, so
// that these kernels share the device error word with the others).
#pragma once
#include "w4.cuh"
#include "w4_stream.cuh"
#include "w4_moe.cuh"

namespace moe {
namespace {

bool w4_group_ok(int group) { return group == 32 || group == 64 || group == 128; }
bool w4_matrix_ok(int K, int N) {
  return K >= 64 && K <= 16384 && K % 64 == 0 && N >= 16 && N <= 1048576 && N % 16 == 0;
}

// Call fn(activation tiles, 32-element groups, zero points) with the three as types.
template <typename F>
auto w4_by_form(int T, int group, bool zeros, F&& fn) {
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  auto by_zero = [&](auto nb, auto g32) {
    return zeros ? fn(nb, g32, std::true_type{}) : fn(nb, g32, std::false_type{});
  };
  auto by_group = [&](auto nb) {
    return group == 32 ? by_zero(nb, std::true_type{}) : by_zero(nb, std::false_type{});
  };
  return T <= 8 ? by_group(One{}) : by_group(Two{});
}

// CTAs of the streaming kernels that run at once.
int w4_slots(const DeviceState& d) { return 2 * std::max(1, d.num_sms); }

// log2 of the row groups (of two strips) per unit of a linear layer.  A taller unit reads the
// activations less often and joins fewer partial sums; a lower one deals out more evenly.  The
// cost of a choice is its rounds of units over the CTAs, each the unit's weight and activation
// bytes plus what a unit costs apart from them, in bytes.
int w4_row_groups(int T, int K, int N, int record, int slots) {
  int best = 0;
  double least = 0;
  for (int lg = 0; lg < 4; ++lg) {
    const int tall = 2 << lg, units = (N / W4_ROWS + tall - 1) / tall;
    const double cost =
        (units + slots - 1) / slots * ((double)tall * (K / W4_KB) * record + 2.0 * T * K + 6144.0);
    if (lg == 0 || cost < least) {
      least = cost;
      best = lg;
    }
  }
  return best;
}

// One linear layer (or the gate | up half of a GEGLU MLP) on the streaming kernel.
template <int MODE>
moe_status_t w4_stream(const Launch& launch, const DeviceState& d, W4Linear a, int group, bool zeros) {
  const int slots = w4_slots(d);
  a.lg = MODE == W4_GEGLU ? 0 : w4_row_groups(a.T, a.K, a.N, w4_record(group, zeros), slots);
  a.units = MODE == W4_GEGLU ? a.N / W4_ROWS : (a.N / W4_ROWS + (2 << a.lg) - 1) >> (a.lg + 1);
  w4_by_form(a.T, group, zeros, [&](auto nb, auto g32, auto zp) {
    constexpr int NB = decltype(nb)::value;
    launch(true, w4_linear_kernel<NB, decltype(g32)::value, decltype(zp)::value, MODE>,
           dim3(std::min(a.units, slots)), dim3(W4S_THREADS), w4s_smem<NB>(), a);
  });
  return launched();
}

// Shared memory limits of the streaming kernels, once per device.
template <int MODE>
bool w4_linear_attrs() {
  bool ok = true;
  for (int f = 0; f < 8; ++f)
    w4_by_form(f & 1 ? 16 : 8, f & 2 ? 32 : 64, f & 4, [&](auto nb, auto g32, auto zp) {
      constexpr int NB = decltype(nb)::value;
      ok = ok && cudaFuncSetAttribute(w4_linear_kernel<NB, decltype(g32)::value, decltype(zp)::value, MODE>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      w4s_smem<NB>()) == cudaSuccess;
    });
  return ok;
}
bool w4_moe_attrs() {
  bool ok = true;
  for (int f = 0; f < 8; ++f)
    w4_by_form(f & 1 ? 16 : 8, f & 2 ? 32 : 64, f & 4, [&](auto nb, auto g32, auto zp) {
      constexpr int NB = decltype(nb)::value;
      ok = ok && cudaFuncSetAttribute(w4_moe_kernel<NB, decltype(g32)::value, decltype(zp)::value>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      w4s_smem<NB>()) == cudaSuccess;
    });
  return ok;
}
DeviceState* w4_device_state(int* dev) {
  static bool done[kMaxDevices] = {};
  static std::mutex mu;
  DeviceState* d = device_state(dev);
  if (!d) return nullptr;
  std::lock_guard<std::mutex> lk(mu);
  if (!done[*dev]) {
    if (!w4_linear_attrs<W4_LINEAR>() || !w4_linear_attrs<W4_LINEAR_F32>() ||
        !w4_linear_attrs<W4_GEGLU>() || !w4_moe_attrs()) {
      cuda_failed(cudaGetLastError());
      return nullptr;
    }
    done[*dev] = true;
  }
  return d;
}

// Workspace of the routed layer: the front kernel's partial sums, ids and weights, counters, h and
// the weighted expert outputs.
struct W4Layout {
  size_t logit = 0, xn2 = 0, wn2 = 0, stats = 0, ids = 0, wts = 0, ctr = 0, h = 0, o = 0, total = 0;
  int slices = 0, lg2 = 0, n_ctr = 0;
};
W4Layout w4_layout(int T, int H, int E, int I, int k) {
  W4Layout L;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  const size_t P = (size_t)T * k;
  L.slices = H / W4M_SLICE;
  // W_down units of 128 rows
  L.lg2 = 2;
  L.n_ctr = W4M_CTR_O + H / W4_ROWS;
  L.logit = take(sizeof(double) * L.slices * T * E);
  L.xn2 = take(sizeof(double) * L.slices * T);
  L.wn2 = take(sizeof(double) * L.slices * E);
  L.stats = take(5 * sizeof(unsigned));
  L.ids = take(sizeof(int32_t) * P);
  L.wts = take(sizeof(float) * P);
  L.ctr = take(sizeof(int) * L.n_ctr);
  L.h = take(2 * P * I);
  L.o = take(sizeof(float) * P * H);
  L.total = at;
  return L;
}
constexpr unsigned kW4LayerFlags = MOE_FLAG_NO_RENORM | MOE_FLAG_W4_ZEROS;

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
  DeviceState* d = w4_device_state(&dev);
  if (!d) return MOE_ERR_CUDA;
  t_kernels = 0;
  W4Linear a = {};
  a.w0 = static_cast<const uint8_t*>(w);
  a.act = static_cast<const __nv_bfloat16*>(x);
  a.out = y;
  a.T = T;
  a.K = K;
  a.N = N;
  const bool zeros = flags & MOE_FLAG_W4_ZEROS;
  const Launch launch{static_cast<cudaStream_t>(stream), true};
  return (flags & MOE_FLAG_F32_OUT) ? w4_stream<W4_LINEAR_F32>(launch, *d, a, group, zeros)
                                    : w4_stream<W4_LINEAR>(launch, *d, a, group, zeros);
}

size_t moe_dense_w4_workspace_size(int T, int H, int I) {
  if (T < 1 || T > W4_MAX_T || H < 64 || H > 16384 || H % 64 || I < 64 || I > 8192 || I % 64) return 0;
  return align256(2 * (size_t)T * I);   // h
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
  if (workspace_bytes < moe_dense_w4_workspace_size(T, H, I)) return MOE_ERR_NO_WORKSPACE;
  int dev = 0;
  DeviceState* d = w4_device_state(&dev);
  if (!d) return MOE_ERR_CUDA;
  t_kernels = 0;
  const Launch launch{static_cast<cudaStream_t>(stream), true};
  __nv_bfloat16* h = static_cast<__nv_bfloat16*>(workspace);
  const bool zeros = flags & MOE_FLAG_W4_ZEROS;
  W4Linear a = {};
  a.w0 = static_cast<const uint8_t*>(w_gate);
  a.w1 = static_cast<const uint8_t*>(w_up);
  a.act = static_cast<const __nv_bfloat16*>(x);
  a.out = h;
  a.T = T;
  a.K = H;
  a.N = I;
  if (const moe_status_t s = w4_stream<W4_GEGLU>(launch, *d, a, group, zeros); s != MOE_OK) return s;
  a.w0 = static_cast<const uint8_t*>(w_down);
  a.w1 = nullptr;
  a.act = h;
  a.out = y;
  a.K = I;
  a.N = H;
  a.early = 1;
  return w4_stream<W4_LINEAR>(launch, *d, a, group, zeros);
}

size_t moe_w4_workspace_size(int T, int H, int E, int I, int k, unsigned flags) {
  if ((flags & ~kW4LayerFlags) || T > W4_MAX_T || !shape_supported(T, H, E, I, k, true)) return 0;
  return w4_layout(T, H, E, I, k).total;
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
  const W4Layout W = w4_layout(T, H, E, I, k);
  if (workspace_bytes < W.total) return MOE_ERR_NO_WORKSPACE;
  int dev = 0;
  DeviceState* d = w4_device_state(&dev);
  if (!d) return MOE_ERR_CUDA;
  t_kernels = 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  W4Moe a = {};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.wr = static_cast<const __nv_bfloat16*>(w_router);
  a.bias = router_bias;
  a.wg = static_cast<const uint8_t*>(w_gate);
  a.wu = static_cast<const uint8_t*>(w_up);
  a.wd = static_cast<const uint8_t*>(w_down);
  double* logit = reinterpret_cast<double*>(ws + W.logit);
  double* xn2 = reinterpret_cast<double*>(ws + W.xn2);
  double* wn2 = reinterpret_cast<double*>(ws + W.wn2);
  a.part_logit = logit;
  a.part_xn2 = xn2;
  a.part_wn2 = wn2;
  a.slices = W.slices;
  a.T = T;
  a.H = H;
  a.E = E;
  a.I = I;
  a.k = k;
  a.renorm = (flags & MOE_FLAG_NO_RENORM) ? 0 : 1;
  a.lg2 = W.lg2;
  const double u = std::ldexp(1.0, -53), n = (double)H + 8.0;
  a.beta_scale = 2.0 * (n * u / (1.0 - n * u)) * 1.01;
  a.ids = (aux && aux->topk_ids) ? aux->topk_ids : reinterpret_cast<int32_t*>(ws + W.ids);
  a.wts = (aux && aux->topk_weights) ? aux->topk_weights : reinterpret_cast<float*>(ws + W.wts);
  a.stats = (aux && aux->router_stats) ? aux->router_stats : reinterpret_cast<unsigned*>(ws + W.stats);
  a.counts = aux ? aux->expert_counts : nullptr;
  a.offsets = aux ? aux->expert_offsets : nullptr;
  a.perm = aux ? aux->perm : nullptr;
  a.ctr = reinterpret_cast<int*>(ws + W.ctr);
  a.h = reinterpret_cast<__nv_bfloat16*>(ws + W.h);
  a.o = reinterpret_cast<float*>(ws + W.o);
  a.y = static_cast<__nv_bfloat16*>(y);
  const Launch launch{static_cast<cudaStream_t>(stream), true};
  auto front = [&](auto kernel) {
    launch(true, kernel, dim3(W.slices), dim3(W4M_FRONT_THREADS), 0, a.x, a.wr, T, H, E, logit, xn2, wn2,
           a.ctr, W.n_ctr, a.stats);
  };
  if (T <= 2) front(w4_front_kernel<2>);
  else if (T <= 8) front(w4_front_kernel<8>);
  else front(w4_front_kernel<16>);
  if (const moe_status_t s = launched(); s != MOE_OK) return s;
  w4_by_form(T, group, flags & MOE_FLAG_W4_ZEROS, [&](auto nb, auto g32, auto zp) {
    constexpr int NB = decltype(nb)::value;
    launch(true, w4_moe_kernel<NB, decltype(g32)::value, decltype(zp)::value>, dim3(w4_slots(*d)),
           dim3(W4S_THREADS), w4s_smem<NB>(), a);
  });
  return launched();
}

}  // extern "C"
