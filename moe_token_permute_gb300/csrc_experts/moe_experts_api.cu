// moe_experts_api.cu -- host side of the C ABI declared in include/moe_experts.h.
//
// Argument checks happen before any device is touched; nothing allocates or
// synchronises.  Each entry point is one launch, or for the backward passes
// one launch per gradient.
#include "moe_experts.h"
#ifdef MOE_DEBUG_HOOKS
#include "debug_hooks.h"
#endif

#include <algorithm>
#include <type_traits>

#include "../csrc/common.cuh"
#include "expert_decode.cuh"
#include "expert_grad.cuh"
#include "expert_math.cuh"
#include "expert_product.cuh"
#include "host_util.cuh"
#include "product_host.cuh"
#include "unpermute_grad.cuh"

namespace moe {
namespace experts {
namespace {

bool is_type(moe_dtype_t dt) { return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_FP16; }
bool is_act(moe_activation_t a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_RELU; }

// The kernels count rows in 32 bits, in steps of up to 512 that may pass the last row.
constexpr int64_t kMostRows = INT32_MAX - 1023;

// Sizes of a [E, N, K] weight and its rows.
bool sizes_ok(int64_t num_rows, int64_t K, int64_t N, int32_t E) {
  return num_rows >= 0 && num_rows <= kMostRows && K >= 8 && N >= 8 && K % 8 == 0 && N % 8 == 0 &&
         K <= INT32_MAX / 2 && N <= INT32_MAX / 2 && E >= 1 && E <= MOE_MAX_LOCAL_EXPERTS;
}

bool base_ok(const void* p) { return p != nullptr && aligned(p, 16); }
bool base_or_null(const void* p) { return p == nullptr || aligned(p, 16); }

unsigned* status_of(void* workspace) {
  return workspace == nullptr ? nullptr : &static_cast<WsHeader*>(workspace)->status;
}

// lhs: the weight, or dz for d_weight; rhs: the rows, or dz for d_rows.
template <typename T, int kUse>
cudaError_t launch_product(const ProductArgs& a, const void* lhs, const void* rhs, int sms,
                           cudaStream_t s) {
  CUtensorMap map_a, map_b;
  bool ok;
  if (kUse == kWeightGrad) {
    // Without rows the products are empty and the maps are never used.
    const int64_t rows = std::max<int64_t>(1, a.num_rows);
    const void* any = a.out;
    ok = make_map<T>(&map_a, lhs != nullptr ? lhs : any, 0, rows, a.N, kSlice) &&
         make_map<T>(&map_b, rhs != nullptr ? rhs : any, 0, rows, a.K, kSlice);
  } else {
    const int64_t depth = kUse == kRowsGrad ? a.N : a.K;
    ok = (kUse == kGated ? make_gated_map<T>(&map_a, lhs, a.E, a.N / 2, a.K)
                         : make_map<T>(&map_a, lhs, a.E, a.N, a.K,
                                       kUse == kRowsGrad ? kSlice : 128)) &&
         make_map<T>(&map_b, rhs, 0, a.num_rows, depth, 64);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int64_t pairs = sms / 2;
  const int splits = kUse == kWeightGrad
                         ? 1
                         : tile_splits(most_tiles<kUse>(a, kMaxN),
                                       ceil_div(kUse == kRowsGrad ? a.N : a.K, kSlice), pairs);
  const int64_t tiles = most_tiles<kUse>(a, splits > 1 ? kMaxN : kLeastCap);
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  const unsigned blocks = 2 * splits * static_cast<unsigned>(std::min<int64_t>(tiles, pairs));
  return launch_clusters(k_expert_product<T, kUse>, dim3(blocks), dim3(2 * splits),
                         kProductThreads, product_smem(a.E), s, map_a, map_b, a);
}

template <typename T, int kUse>
cudaError_t launch_forward(const ProductArgs& a, const void* weight, const void* rows, int sms,
                           cudaStream_t s) {
  constexpr bool kGatedForm = kUse == kGated;
  if (!decode_pays(kGatedForm, a.num_rows, a.E, a.K))
    return launch_product<T, kUse>(a, weight, rows, sms, s);
  // Tasks at most: every expert with rows has one group, and each further
  // kDecodeGroup rows one more.
  const int64_t groups = std::min<int64_t>(a.E, a.num_rows) + a.num_rows / kDecodeGroup;
  const int64_t tasks = groups * ((kGatedForm ? a.N / 2 : a.N) / kDecodeFeatures);
  if (tasks > INT32_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap map;
  if (!make_decode_map<T>(&map, weight, a.E, a.N, a.K))
    return cudaErrorInvalidValue;
  return launch(k_expert_decode<T, kGatedForm>,
                dim3(static_cast<unsigned>(std::min<int64_t>(tasks, sms))), kDecodeThreads,
                DecodeShape<kGatedForm>::kSmem, s, map, static_cast<const T*>(rows), a);
}

template <typename T, bool kGatedForm>
cudaError_t launch_act_grad(const void* d_out, const void* z, void* dz, const int64_t* offset,
                            int E, int64_t num_rows, int64_t W, moe_activation_t act,
                            unsigned* status, int sms, cudaStream_t s) {
  auto kern = k_act_grad<T, kGatedForm, MOE_ACT_NONE>;
  if (act == MOE_ACT_SILU) kern = k_act_grad<T, kGatedForm, MOE_ACT_SILU>;
  if (act == MOE_ACT_GELU) kern = k_act_grad<T, kGatedForm, MOE_ACT_GELU>;
  if (act == MOE_ACT_RELU) kern = k_act_grad<T, kGatedForm, MOE_ACT_RELU>;
  const int64_t columns = ceil_div(W / 8, 32);
  if (columns > 65535) return cudaErrorInvalidConfiguration;
  // About 8 blocks per SM, and never fewer than one.
  const int64_t grid = std::min(ceil_div(num_rows, kGradWarps),
                                std::max<int64_t>(1, 8 * static_cast<int64_t>(sms) / columns));
  return launch(kern, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(columns)),
                kGradThreads, 0, s,
                static_cast<const T*>(d_out), static_cast<const T*>(z), static_cast<T*>(dz),
                offset, E, num_rows, W, status);
}

template <typename T>
cudaError_t launch_bias_grad(const void* dz, const int64_t* offset, int E, int64_t num_rows,
                             int64_t N, void* d_bias, unsigned* status, int sms,
                             cudaStream_t s) {
  // Few rows per expert: wide blocks; few blocks: clusters that share the rows.
  const bool wide = num_rows <= 16 * static_cast<int64_t>(E);
  const int64_t blocks = ceil_div(N, wide ? 8 * kBiasWide : 8 * kBiasNarrow);
  const unsigned splits = !wide && blocks * E <= sms ? kBiasSplit : 1;
  return launch_clusters(wide ? k_bias_grad<T, kBiasWide> : k_bias_grad<T, kBiasNarrow>,
                         dim3(static_cast<unsigned>(blocks), E, splits), dim3(1, 1, splits),
                         kGradThreads, 0, s, static_cast<const T*>(dz), offset, num_rows, N,
                         static_cast<T*>(d_bias), status);
}

// d_rows and d_weight of z = x W^T from dz.  beside_previous: the launch before is
// one of this call that only reads dz too.  The two products run beside one another
// where the first leaves SMs free (at its end, or all along when it is small).
template <typename T>
cudaError_t product_gradients(const void* dz, const void* rows, const void* weight,
                              const int64_t* offset, int64_t num_rows, int64_t K, int64_t N,
                              int E, void* d_rows, void* d_weight, bool beside_previous,
                              unsigned* status, int sms, cudaStream_t s) {
  ProductArgs a = {};
  a.beside_previous = beside_previous;
  a.offset = offset;
  a.num_rows = num_rows;
  a.K = K;
  a.N = N;
  a.E = E;
  a.status = status;
  if (d_rows != nullptr && num_rows > 0) {
    a.out = d_rows;
    const cudaError_t err = launch_product<T, kRowsGrad>(a, weight, dz, sms, s);
    if (err != cudaSuccess) return err;
    a.beside_previous = true;
  }
  if (d_weight != nullptr) {
    a.out = d_weight;
    return launch_product<T, kWeightGrad>(a, dz, rows, sms, s);
  }
  return cudaSuccess;
}

template <typename VecT>
cudaError_t launch_unpermute_backward(const void* d_out, const void* rows, int64_t num_rows,
                                      int64_t H, const float* w, const int32_t* inv, int64_t T,
                                      int K, void* d_rows, float* d_w, unsigned* status, int sms,
                                      cudaStream_t s) {
  const int64_t vecs = H * 2 / static_cast<int64_t>(sizeof(VecT));
  // (t, k) per warp: one while there are few, then so many that the warps are 150
  // per SM (64: DeepSeek-V3 shape T = 4096 162 us instead of 150; 220 and more:
  // DeepSeek-V2-Lite with its map 36 us instead of 30).
  const int64_t items = T * K;
  const int64_t per_warp =
      std::max<int64_t>(1, std::min<int64_t>(32, items / (150 * static_cast<int64_t>(sms))));
  const int64_t blocks = ceil_div(ceil_div(items, per_warp), kCombineWarps);
  return launch(k_unpermute_backward<VecT>, dim3(static_cast<unsigned>(blocks)),
                kCombineWarps * 32, 0, s, static_cast<const VecT*>(d_out),
                static_cast<const VecT*>(rows), num_rows, vecs, w, inv, items, K,
                static_cast<int>(per_warp), static_cast<VecT*>(d_rows), d_w, status);
}

int finish(cudaError_t err) {
  if (err == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

}  // namespace
}  // namespace experts
}  // namespace moe

using namespace moe;
using namespace moe::experts;

extern "C" {

int moe_expert_gated(const void* permuted_rows, const void* weight, moe_dtype_t dtype,
                     const int64_t* expert_first_token_offset, int64_t num_rows,
                     int64_t hidden_size, int64_t ffn_size, int32_t num_local_experts,
                     moe_activation_t activation, void* out, void* preact, void* workspace,
                     moe_stream_t stream) {
  if (!is_type(dtype) || !is_act(activation) || ffn_size < 8 || ffn_size > INT32_MAX / 4 ||
      ffn_size % 8 != 0 || !sizes_ok(num_rows, hidden_size, 2 * ffn_size, num_local_experts))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (num_rows == 0) return MOE_OK;
  if (expert_first_token_offset == nullptr || !aligned(expert_first_token_offset, 8) ||
      !base_ok(permuted_rows) || !base_ok(weight) || !base_ok(out) || !base_or_null(preact))
    return MOE_ERR_INVALID_ARG;
  const int sms = supported_sm_count();
  if (sms == 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  ProductArgs a = {};
  a.offset = expert_first_token_offset;
  a.num_rows = num_rows;
  a.K = hidden_size;
  a.N = 2 * ffn_size;
  a.E = num_local_experts;
  a.act = activation;
  a.out = out;
  a.preact = preact;
  a.status = status_of(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return finish(dtype == MOE_DTYPE_BF16 ? launch_forward<__nv_bfloat16, kGated>(a, weight, permuted_rows, sms, s)
                                        : launch_forward<__half, kGated>(a, weight, permuted_rows, sms, s));
}

int moe_expert_gated_backward(const void* d_out, const void* permuted_rows, const void* weight,
                              moe_dtype_t dtype, const int64_t* expert_first_token_offset,
                              int64_t num_rows, int64_t hidden_size, int64_t ffn_size,
                              int32_t num_local_experts, moe_activation_t activation,
                              const void* preact, void* d_preact, void* d_rows, void* d_weight,
                              void* workspace, moe_stream_t stream) {
  if (!is_type(dtype) || !is_act(activation) || ffn_size < 8 || ffn_size > INT32_MAX / 4 ||
      ffn_size % 8 != 0 || !sizes_ok(num_rows, hidden_size, 2 * ffn_size, num_local_experts))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (expert_first_token_offset == nullptr || !aligned(expert_first_token_offset, 8))
    return MOE_ERR_INVALID_ARG;
  if (!base_or_null(d_rows) || !base_or_null(d_weight)) return MOE_ERR_INVALID_ARG;
  if (num_rows > 0) {
    if (!base_ok(d_out) || !base_ok(preact) || !base_ok(d_preact)) return MOE_ERR_INVALID_ARG;
    if (d_rows != nullptr && !base_ok(weight)) return MOE_ERR_INVALID_ARG;
    if (d_weight != nullptr && !base_ok(permuted_rows)) return MOE_ERR_INVALID_ARG;
  }
  const int sms = supported_sm_count();
  if (sms == 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = dtype == MOE_DTYPE_BF16;
  unsigned* status = status_of(workspace);
  if (num_rows > 0) {
    const cudaError_t err =
        bf ? launch_act_grad<__nv_bfloat16, true>(d_out, preact, d_preact,
                                                  expert_first_token_offset, num_local_experts,
                                                  num_rows, ffn_size, activation, status, sms, s)
           : launch_act_grad<__half, true>(d_out, preact, d_preact, expert_first_token_offset,
                                           num_local_experts, num_rows, ffn_size, activation,
                                           status, sms, s);
    if (err != cudaSuccess) return finish(err);
  }
  auto gradients = bf ? product_gradients<__nv_bfloat16> : product_gradients<__half>;
  return finish(gradients(d_preact, permuted_rows, weight, expert_first_token_offset, num_rows,
                          hidden_size, 2 * ffn_size, num_local_experts, d_rows, d_weight, false,
                          status, sms, s));
}

int moe_expert_linear(const void* rows, const void* weight, moe_dtype_t dtype,
                      const int64_t* expert_first_token_offset, int64_t num_rows, int64_t in_size,
                      int64_t out_size, int32_t num_local_experts, const void* bias,
                      moe_activation_t activation, const void* residual, void* out, void* preact,
                      void* workspace, moe_stream_t stream) {
  if (!is_type(dtype) || !is_act(activation) ||
      !sizes_ok(num_rows, in_size, out_size, num_local_experts))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (num_rows == 0) return MOE_OK;
  if (expert_first_token_offset == nullptr || !aligned(expert_first_token_offset, 8) ||
      !base_ok(rows) || !base_ok(weight) || !base_ok(out) || !base_or_null(bias) ||
      !base_or_null(residual) || !base_or_null(preact))
    return MOE_ERR_INVALID_ARG;
  const int sms = supported_sm_count();
  if (sms == 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  ProductArgs a = {};
  a.offset = expert_first_token_offset;
  a.num_rows = num_rows;
  a.K = in_size;
  a.N = out_size;
  a.E = num_local_experts;
  a.act = activation;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.preact = preact;
  a.status = status_of(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return finish(dtype == MOE_DTYPE_BF16 ? launch_forward<__nv_bfloat16, kForward>(a, weight, rows, sms, s)
                                        : launch_forward<__half, kForward>(a, weight, rows, sms, s));
}

int moe_expert_linear_backward(const void* d_out, const void* rows, const void* weight,
                               moe_dtype_t dtype, const int64_t* expert_first_token_offset,
                               int64_t num_rows, int64_t in_size, int64_t out_size,
                               int32_t num_local_experts, moe_activation_t activation,
                               const void* preact, void* d_preact, void* d_rows, void* d_weight,
                               void* d_bias, void* workspace, moe_stream_t stream) {
  if (!is_type(dtype) || !is_act(activation) ||
      !sizes_ok(num_rows, in_size, out_size, num_local_experts))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (expert_first_token_offset == nullptr || !aligned(expert_first_token_offset, 8))
    return MOE_ERR_INVALID_ARG;
  if (!base_or_null(d_rows) || !base_or_null(d_weight) || !base_or_null(d_bias))
    return MOE_ERR_INVALID_ARG;
  const bool with_act = activation != MOE_ACT_NONE;
  if (!with_act && (preact != nullptr || d_preact != nullptr)) return MOE_ERR_INVALID_ARG;
  if (num_rows > 0) {
    if (!base_ok(d_out)) return MOE_ERR_INVALID_ARG;
    if (with_act && (!base_ok(preact) || !base_ok(d_preact))) return MOE_ERR_INVALID_ARG;
    if (d_rows != nullptr && !base_ok(weight)) return MOE_ERR_INVALID_ARG;
    if (d_weight != nullptr && !base_ok(rows)) return MOE_ERR_INVALID_ARG;
  }
  const int sms = supported_sm_count();
  if (sms == 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = dtype == MOE_DTYPE_BF16;
  unsigned* status = status_of(workspace);
  const void* dz = d_out;
  cudaError_t err = cudaSuccess;
  if (with_act && num_rows > 0) {
    auto grad = bf ? launch_act_grad<__nv_bfloat16, false> : launch_act_grad<__half, false>;
    err = grad(d_out, preact, d_preact, expert_first_token_offset, num_local_experts, num_rows,
               out_size, activation, status, sms, s);
    dz = d_preact;
  }
  if (err == cudaSuccess && d_bias != nullptr) {
    auto grad = bf ? launch_bias_grad<__nv_bfloat16> : launch_bias_grad<__half>;
    err = grad(dz, expert_first_token_offset, num_local_experts, num_rows, out_size, d_bias,
               status, sms, s);
  }
  if (err != cudaSuccess) return finish(err);
  auto gradients = bf ? product_gradients<__nv_bfloat16> : product_gradients<__half>;
  return finish(gradients(dz, rows, weight, expert_first_token_offset, num_rows, in_size, out_size,
                          num_local_experts, d_rows, d_weight, d_bias != nullptr, status, sms, s));
}

int moe_unpermute_backward(const void* d_out, const void* permuted_rows, int64_t num_rows,
                           const float* topk_weights, const int32_t* inv_permuted_idx,
                           int64_t num_tokens, int64_t hidden_size, int32_t topk, void* d_rows,
                           float* d_topk_weights, void* workspace, moe_stream_t stream) {
  const int64_t T = num_tokens, H = hidden_size;
  if (T < 0 || H < 1 || topk < 1 || topk > MOE_MAX_TOPK || num_rows < 0) return MOE_ERR_INVALID_ARG;
  if (T > INT32_MAX / topk || num_rows > INT32_MAX || H > INT64_MAX / 32)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (d_out == nullptr || topk_weights == nullptr || inv_permuted_idx == nullptr ||
      !aligned(d_out, 2) || !aligned(permuted_rows, 2) || !aligned(topk_weights, 4) ||
      !aligned(inv_permuted_idx, 4) || !aligned(d_rows, 2) || !aligned(d_topk_weights, 4))
    return MOE_ERR_INVALID_ARG;
  if (num_rows > 0 && (permuted_rows == nullptr) != (d_topk_weights == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (d_rows == nullptr && d_topk_weights == nullptr) return MOE_ERR_INVALID_ARG;
  const int sms = supported_sm_count();
  if (sms == 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned* status = status_of(workspace);
  size_t vb = 16;
  while (vb > 2 && (H * 2 % static_cast<int64_t>(vb) != 0 || !aligned(d_out, vb) ||
                    !aligned(permuted_rows, vb) || !aligned(d_rows, vb)))
    vb /= 2;
  auto run = vb == 16  ? launch_unpermute_backward<uint4>
             : vb == 8 ? launch_unpermute_backward<uint2>
             : vb == 4 ? launch_unpermute_backward<uint32_t>
                       : launch_unpermute_backward<uint16_t>;
  return finish(run(d_out, permuted_rows, num_rows, H, topk_weights, inv_permuted_idx, T, topk,
                    d_rows, d_topk_weights, status, sms, s));
}

#ifdef MOE_DEBUG_HOOKS
int moe_debug_set_expert_wait(int slices, unsigned long long wait_ns) {
  if (slices < 0 || wait_ns == 0) return MOE_ERR_INVALID_ARG;
  if (cudaMemcpyToSymbol(g_debug_slices, &slices, sizeof(slices)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_debug_wait_ns, &wait_ns, sizeof(wait_ns)) != cudaSuccess ||
      !set_quant_wait(slices, wait_ns)) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
#endif

}  // extern "C"
