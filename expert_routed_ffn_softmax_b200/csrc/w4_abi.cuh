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

// How a linear layer (or the gate | up half of a GEGLU MLP) is cut: units of 2 << lg strips,
// `cluster` CTAs sharing a unit's K.  A CTA keeps its slice of the activations in shared memory
// where all of K would fit beside a ring of two 16 KB stages (T <= 8, rows up to T K = 30 K elements);
// longer ones come as fragments with each chunk of weights.  A taller unit reads the activations less
// often, a lower one and slices of K spread a small matrix over the SMs (two CTAs each).  More units
// than run at once are only stolen without clusters: a cluster's start and meeting would be paid for
// every unit.
//
// The choice is the one with the least time by a model of what was measured on B200 (ns).  Per
// block and strip, the largest of: decoding and products, 26 with two CTAs on an SM and 18 + 1.1 T
// with one (45 for two row tiles); its bytes at 22 a ns (32 for a CTA alone on its SM, without
// fragments); its copies at 100 each.  Per cluster 400 a CTA (200 with fragments, whose own launch
// hides its start) and 0.3 for every sum exchanged.  The model ranks cuts; what every cut pays alike
// (launches, the first copy, the last join: 3 to 6 us) is not in it.  Over 17 shapes (T 1 to 16, K 704
// to 16384, N 704 to 131072) and all 16 cuts of each, timed one by one, the choice was within 7 % of
// the best (10 % at T = 12, 16384 x 2048) and the best itself in 9 of them.
struct W4Plan {
  int lg = 0, cluster = 1, units = 0, step = 0, stage = 0, smem = 0, frag = 0, steal = 0;
};
// Whether activations [T][K] come as fragments.
template <int NB> bool w4_frag(int T, int K) {
  return NB == 2 || w4_linear_smem<NB>(T, K, 0, 16384, 1, 0).total > W4S_SMEM;
}
template <int NB>
W4Plan w4_plan(int mode, int T, int K, int N, int record, int sms) {
  W4Plan best;
  best.frag = w4_frag<NB>(T, K);
  const int kb = K / W4_KB;
  double least = 0;
  for (int cluster = 1; cluster <= 8 && cluster <= kb; cluster *= 2)
    for (int lg = 0; lg < 4; ++lg) {
      const int strips = 2 << lg, per = mode == W4_GEGLU ? 1 << lg : strips, most = (kb + cluster - 1) / cluster;
      const int rest = w4_linear_smem<NB>(T, K, best.frag, 0, cluster, lg).total;
      const int room = std::min((W4S_SMEM - rest) / W4S_STAGES / 128 * 128, 46080);
      const int block = strips * record + (best.frag ? w4_frag_block<NB>() : 0);
      if (room < block) continue;
      W4Plan p = best;
      p.lg = lg;
      p.cluster = cluster;
      p.units = (N / W4_ROWS + per - 1) / per;
      // a CTA's only unit, where it is long, comes in two chunks at least, so that it is multiplied
      // while it arrives (T = 1, 2112 x 2816: 36 KB in one chunk take 1.4 us longer; but T = 7 in two
      // slices of K, 19 KB in two chunks, 0.2, and T = 16 in four, 9 blocks and their fragments, 0.5)
      const bool halve = p.units * cluster <= 2 * sms && most >= 2 * W4S_MMA_WARPS && most * block >= 24576;
      const int chunks = std::max((most + room / block - 1) / (room / block), halve ? 2 : 1);
      p.step = (most + chunks - 1) / chunks;
      p.stage = (p.step * block + 127) / 128 * 128;
      p.smem = w4_linear_smem<NB>(T, K, p.frag, p.stage, cluster, lg).total;
      const int ctas = p.units * cluster;
      if (cluster > 1 && ctas > 2 * sms) continue;
      const double products = NB == 2 ? 45.0 : ctas > sms ? 26.0 : 18.0 + 1.1 * T;
      const double unit = (double)strips * most *
                          std::max({products, (double)block / strips / (ctas > sms || p.frag ? 22.0 : 32.0),
                                    100.0 * (strips + p.frag) / (strips * p.step)});
      const double act = p.frag ? 0.0 : 128.0 * T * most / 22.0;
      const double cost = ctas <= 2 * sms
                              ? unit + act + (cluster > 1 ? (p.frag ? 200.0 : 400.0) * cluster + 0.3 * (32 << lg) * T : 0.0)
                              : (p.units / (2.0 * sms) + 1.0) * (unit + 250.0) + act;
      if (least == 0 || cost < least) {
        least = cost;
        best = p;
      }
    }
  best.steal = best.cluster == 1 && best.units > 2 * sms;
  return best;
}

template <int MODE>
moe_status_t w4_stream(cudaStream_t st, const DeviceState& d, W4Linear a, int group, bool zeros) {
  w4_by_form(a.T, group, zeros, [&](auto nb, auto g32, auto zp) {
    constexpr int NB = decltype(nb)::value;
    const int sms = std::max(1, d.num_sms);
    const W4Plan p = w4_plan<NB>(MODE, a.T, a.K, a.N, w4_record(group, zeros), sms);
    a.lg = p.lg;
    a.cluster = p.cluster;
    a.step = p.step;
    a.stage = p.stage;
    a.frag = p.frag;
    a.steal = p.steal;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.units * p.cluster);
    cfg.blockDim = dim3(W4S_THREADS);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, w4_linear_kernel<NB, decltype(g32)::value, decltype(zp)::value, MODE>, a);
    ++t_kernels;
  });
  return launched();
}

// Activations x [T][K] for w4_stream: x itself, or its fragments in `scratch` (one launch more,
// after which the stream may start its weights early).
bool w4_needs_fragments(int T, int K) { return T > 8 ? w4_frag<2>(T, K) : w4_frag<1>(T, K); }
size_t w4_fragment_bytes(int T, int K) {
  return w4_needs_fragments(T, K) ? align256((size_t)(K / W4_KB) * (T > 8 ? w4_frag_block<2>() : w4_frag_block<1>()))
                                  : 0;
}
void w4_activations(cudaStream_t st, const void* x, void* scratch, W4Linear& a) {
  a.act = static_cast<const __nv_bfloat16*>(x);
  if (!w4_needs_fragments(a.T, a.K)) return;
  const Launch launch{st, true};
  launch(true, w4_fragment_kernel, dim3((a.T * a.K / 8 + 255) / 256), dim3(256), 0, a.act, a.T, a.K,
         a.T > 8 ? 2 : 1, static_cast<__nv_bfloat16*>(scratch));
  a.act = static_cast<const __nv_bfloat16*>(scratch);
  a.early = 1;
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
                                      W4S_SMEM) == cudaSuccess;
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
                                      W4S_SMEM) == cudaSuccess;
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
  size_t xfrag = 0, hfrag = 0;
  int slices = 0, n_ctr = 0;
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
  L.n_ctr = W4M_CTR_O + H / W4_ROWS;
  L.logit = take(sizeof(double) * L.slices * T * E);
  L.xn2 = take(sizeof(double) * L.slices * T);
  L.wn2 = take(sizeof(double) * L.slices * (W4M_FRONT_THREADS / 32));
  L.stats = take(5 * sizeof(unsigned));
  L.ids = take(sizeof(int32_t) * P);
  L.wts = take(sizeof(float) * P);
  L.ctr = take(sizeof(int) * L.n_ctr);
  L.h = take(2 * P * I);
  L.o = take(sizeof(float) * P * H);
  // fragments of x, and of h per expert with many rows (fewer than P / 3 of them)
  const size_t block = T > 8 ? w4_frag_block<2>() : w4_frag_block<1>();
  L.xfrag = take(block * (H / W4_KB));
  L.hfrag = take(block * (I / W4_KB) * std::min<size_t>(E, P));
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

size_t moe_linear_w4_workspace_size(int T, int K) {
  if (T < 1 || T > W4_MAX_T || !w4_matrix_ok(K, 16)) return 0;
  return w4_fragment_bytes(T, K);
}

moe_status_t moe_linear_w4(const void* x, const void* w, int T, int K, int N, int group,
                           unsigned flags, void* y, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (T < 0 || K <= 0 || N <= 0 || !w4_group_ok(group) ||
      (flags & ~(MOE_FLAG_W4_ZEROS | MOE_FLAG_F32_OUT)))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w || !y || !aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(workspace) || x == y)
    return MOE_ERR_INVALID_ARG;
  if (T > W4_MAX_T || !w4_matrix_ok(K, N)) return MOE_ERR_UNSUPPORTED;
  const size_t need = w4_fragment_bytes(T, K);
  if (need && !workspace) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_NO_WORKSPACE;
  int dev = 0;
  DeviceState* d = w4_device_state(&dev);
  if (!d) return MOE_ERR_CUDA;
  t_kernels = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  W4Linear a = {};
  a.w0 = static_cast<const uint8_t*>(w);
  a.out = y;
  a.T = T;
  a.K = K;
  a.N = N;
  w4_activations(st, x, workspace, a);
  const bool zeros = flags & MOE_FLAG_W4_ZEROS;
  return (flags & MOE_FLAG_F32_OUT) ? w4_stream<W4_LINEAR_F32>(st, *d, a, group, zeros)
                                    : w4_stream<W4_LINEAR>(st, *d, a, group, zeros);
}

// Workspace of the dense MLP: h (rows, or fragments), then the fragments of x.
size_t moe_dense_w4_workspace_size(int T, int H, int I) {
  if (T < 1 || T > W4_MAX_T || H < 64 || H > 16384 || H % 64 || I < 64 || I > 8192 || I % 64) return 0;
  return std::max(align256(2 * (size_t)T * I), w4_fragment_bytes(T, I)) + w4_fragment_bytes(T, H);
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
  const size_t need = moe_dense_w4_workspace_size(T, H, I);
  if (need == 0) return MOE_ERR_UNSUPPORTED;
  if (workspace_bytes < need) return MOE_ERR_NO_WORKSPACE;
  int dev = 0;
  DeviceState* d = w4_device_state(&dev);
  if (!d) return MOE_ERR_CUDA;
  t_kernels = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool zeros = flags & MOE_FLAG_W4_ZEROS;
  W4Linear a = {};
  a.w0 = static_cast<const uint8_t*>(w_gate);
  a.w1 = static_cast<const uint8_t*>(w_up);
  a.out = workspace;
  a.T = T;
  a.K = H;
  a.N = I;
  a.out_frag = w4_needs_fragments(T, I) ? (T > 8 ? 2 : 1) : 0;
  w4_activations(st, x, static_cast<uint8_t*>(workspace) + need - w4_fragment_bytes(T, H), a);
  if (const moe_status_t s = w4_stream<W4_GEGLU>(st, *d, a, group, zeros); s != MOE_OK) return s;
  a.w0 = static_cast<const uint8_t*>(w_down);
  a.w1 = nullptr;
  a.act = static_cast<const __nv_bfloat16*>(workspace);
  a.out = y;
  a.K = I;
  a.N = H;
  a.early = 1;
  return w4_stream<W4_LINEAR>(st, *d, a, group, zeros);
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
  a.xfrag = reinterpret_cast<__nv_bfloat16*>(ws + W.xfrag);
  a.hfrag = reinterpret_cast<__nv_bfloat16*>(ws + W.hfrag);
  a.y = static_cast<__nv_bfloat16*>(y);
  const Launch launch{static_cast<cudaStream_t>(stream), true};
  launch(true, w4_front_kernel, dim3(W.slices, (T + W4M_TT - 1) / W4M_TT), dim3(W4M_FRONT_THREADS), 0, a.x,
         a.wr, T, H, E, logit, xn2, wn2, a.ctr, W.n_ctr, a.stats, a.ids, k, a.xfrag);
  if (const moe_status_t s = launched(); s != MOE_OK) return s;
  w4_by_form(T, group, flags & MOE_FLAG_W4_ZEROS, [&](auto nb, auto g32, auto zp) {
    constexpr int NB = decltype(nb)::value;
    launch(true, w4_moe_kernel<NB, decltype(g32)::value, decltype(zp)::value>, dim3(w4_slots(*d)),
           dim3(W4S_THREADS), W4S_SMEM, a);
  });
  return launched();
}

moe_status_t moe_debug_w4_cut(int T, int K, int N, int group, unsigned flags, int geglu, int sms, int* out) {
  if (!out || !w4_group_ok(group) || (flags & ~MOE_FLAG_W4_ZEROS) || sms < 1) return MOE_ERR_INVALID_ARG;
  if (T < 1 || T > W4_MAX_T || !w4_matrix_ok(K, N)) return MOE_ERR_UNSUPPORTED;
  const int mode = geglu ? W4_GEGLU : W4_LINEAR, record = w4_record(group, flags & MOE_FLAG_W4_ZEROS);
  const W4Plan p = T > 8 ? w4_plan<2>(mode, T, K, N, record, sms) : w4_plan<1>(mode, T, K, N, record, sms);
  const int cut[6] = {p.cluster, 2 << p.lg, p.units, p.step, p.frag, p.steal};
  std::copy(cut, cut + 6, out);
  return MOE_OK;
}

}  // extern "C"
