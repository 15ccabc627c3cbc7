// moe_quant_api.cu -- host side of the C ABI declared in include/moe_quant.h.
//
// Argument checks happen before any device is touched; nothing allocates or
// synchronises.  Each entry point is one launch.
#include "moe_quant.h"
#ifdef MOE_DEBUG_HOOKS
#include "debug_hooks.h"
#endif

#include <algorithm>
#include <type_traits>

#include "expert_math.cuh"
#include "host_util.cuh"
#include "int8_product.cuh"
#include "product_host.cuh"
#include "quant_decode.cuh"
#include "quant_product.cuh"
#include "quant_rows.cuh"

namespace moe {
namespace experts {
namespace {

bool is_type(moe_dtype_t dt) { return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_FP16; }
bool is_code(moe_dtype_t dt) { return dt == MOE_DTYPE_FP8_E4M3 || dt == MOE_DTYPE_INT8; }
bool is_act(moe_activation_t a) { return a >= MOE_ACT_NONE && a <= MOE_ACT_RELU; }

// The kernels count rows in 32 bits, in steps of up to 512 that may pass the last row.
constexpr int64_t kMostRows = INT32_MAX - 1023;

bool base_ok(const void* p) { return p != nullptr && aligned(p, 16); }
bool base_or_null(const void* p) { return p == nullptr || aligned(p, 16); }
bool scales_ok(const void* p) { return p != nullptr && aligned(p, 4); }

bool row_size_ok(int64_t K) { return K >= 16 && K % 16 == 0 && K <= INT32_MAX / 2; }

unsigned* status_of(void* workspace) {
  return workspace == nullptr ? nullptr : &static_cast<WsHeader*>(workspace)->status;
}

int finish(cudaError_t err) {
  if (err == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

template <typename T, bool kWide>
cudaError_t launch_quant_fp8(const QuantRowsArgs& a, int sms, cudaStream_t s) {
  const int64_t slots = a.num_rows * ceil_div(a.H, kQuantGroup) * 8;
  const int64_t grid = std::min<int64_t>(ceil_div(slots, kQuantThreads), kFp8Blocks * static_cast<int64_t>(sms));
  return launch(k_quant_rows_fp8<T, kWide>, dim3(static_cast<unsigned>(grid)), kQuantThreads, 0, s,
                a);
}

template <typename T, bool kWide>
cudaError_t launch_quant_int8(const QuantRowsArgs& a, int sms, cudaStream_t s) {
  // A warp a row up to 2048 columns, unless there are too few rows for that to fill the
  // SMs; a block beyond 4096.
  const int64_t pieces = a.H / 16;
  const bool few = a.num_rows < 16 * static_cast<int64_t>(sms);
  const int threads = pieces <= (few ? 32 : 128) ? 32 : pieces <= (few ? 128 : 256) ? 64 : 256;
  auto kern = pieces <= 64 && threads == 32 ? k_quant_rows_int8<T, kWide, 32, 2>
              : threads == 32               ? k_quant_rows_int8<T, kWide, 32, 4>
              : threads == 64               ? k_quant_rows_int8<T, kWide, 64, 4>
                                            : k_quant_rows_int8<T, kWide, 256, 4>;
  const int64_t grid = std::min<int64_t>(ceil_div(a.num_rows, kQuantThreads / threads),
                                         kInt8Blocks * static_cast<int64_t>(sms));
  return launch(kern, dim3(static_cast<unsigned>(grid)), kQuantThreads, 0, s, a);
}

template <typename T, int kUse, int kHalves>
cudaError_t launch_int8_tiles(const CUtensorMap& map_a, const CUtensorMap& map_b,
                              const QuantArgs& a, int sms, cudaStream_t s) {
  constexpr int kStep = m_step<kUse>() / 2 * kHalves;
  const int splits = kHalves == 1 ? tile_splits(most_tiles<kUse>(a, kInt8Columns, kStep),
                                                ceil_div(a.K, kRawSlice), sms)
                                  : 1;
  const int64_t tiles = most_tiles<kUse>(a, splits > 1 ? kInt8Columns : kLeastCap, kStep);
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  const unsigned blocks = splits * static_cast<unsigned>(std::min<int64_t>(tiles, sms / splits));
  return launch_clusters(k_int8_product<T, kUse, kHalves>, dim3(blocks), dim3(splits),
                         kInt8Threads, int8_product_smem(a.E), s, map_a, map_b, a);
}

template <typename T, bool kGatedForm>
cudaError_t launch_int8(const QuantArgs& a, int sms, cudaStream_t s) {
  constexpr int kUse = kGatedForm ? kGated : kForward;
  CUtensorMap map_a, map_b;
  if (!(kGatedForm ? make_gated_map<uint8_t>(&map_a, a.weight, a.E, a.N / 2, a.K)
                   : make_map<uint8_t>(&map_a, a.weight, a.E, a.N, a.K, 128)) ||
      !make_map<uint8_t>(&map_b, a.codes, 0, a.num_rows, a.K, 64))
    return cudaErrorInvalidValue;
  return int8_two_halves(most_tiles<kUse>(a, kInt8Columns), sms)
             ? launch_int8_tiles<T, kUse, 2>(map_a, map_b, a, sms, s)
             : launch_int8_tiles<T, kUse, 1>(map_a, map_b, a, sms, s);
}

template <typename T, bool kGatedForm>
cudaError_t launch_fp8(const QuantArgs& a, int sms, cudaStream_t s) {
  constexpr int kUse = kGatedForm ? kGated : kForward;
  CUtensorMap map_rows, map_weight;
  if (!make_map<uint8_t>(&map_rows, a.codes, 0, a.num_rows, a.K, 64) ||
      !make_map<uint8_t>(&map_weight, a.weight, a.E, a.N, a.K, 128))
    return cudaErrorInvalidValue;
  const int64_t tiles = most_tiles<kUse>(a, kTileRows);
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  const int splits = tile_splits(tiles, ceil_div(a.K, kGroupSlice), sms);
  const unsigned blocks = splits * static_cast<unsigned>(std::min<int64_t>(tiles, sms / splits));
  return launch_clusters(k_quant_product<T, kUse>, dim3(blocks), dim3(splits),
                         kQuantProductThreads, quant_product_smem(a.E), s, map_rows, map_weight,
                         a);
}

template <typename T, bool kFp8, bool kGatedForm>
cudaError_t launch_quant_product(const QuantArgs& a, int sms, cudaStream_t s) {
  if (!quant_decode_pays(kFp8, kGatedForm, a.num_rows, a.E, a.K, kGatedForm ? a.N / 2 : a.N))
    return kFp8 ? launch_fp8<T, kGatedForm>(a, sms, s) : launch_int8<T, kGatedForm>(a, sms, s);
  // Tasks at most: every expert with rows has one group, and each further
  // kDecodeGroup rows one more.
  const int64_t groups = std::min<int64_t>(a.E, a.num_rows) + a.num_rows / kDecodeGroup;
  const int64_t tasks = groups * ((kGatedForm ? a.N / 2 : a.N) / kDecodeFeatures);
  if (tasks > INT32_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap map;
  if (!make_decode_map<uint8_t>(&map, a.weight, a.E, a.N, a.K)) return cudaErrorInvalidValue;
  return launch(k_quant_decode<T, kFp8, kGatedForm>,
                dim3(static_cast<unsigned>(std::min<int64_t>(tasks, sms))), kDecodeThreads,
                DecodeShape<true>::kSmem, s, map, a);
}

template <bool kGatedForm>
int product(const QuantArgs& a, moe_dtype_t code_dtype, moe_dtype_t out_dtype,
            moe_activation_t activation, int64_t width, void* workspace, moe_stream_t stream) {
  if (!is_code(code_dtype) || !is_type(out_dtype) || !is_act(activation) || a.num_rows < 0 ||
      a.num_rows > kMostRows || !row_size_ok(a.K) || width < 8 || width % 8 != 0 ||
      width > INT32_MAX / 4 || a.E < 1 || a.E > MOE_MAX_LOCAL_EXPERTS)
    return MOE_ERR_INVALID_ARG;
  if (code_dtype == MOE_DTYPE_INT8 && a.K > MOE_INT8_MAX_IN) return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (a.num_rows == 0) return MOE_OK;
  if (a.offset == nullptr || !aligned(a.offset, 8) || !base_ok(a.codes) || !scales_ok(a.scales) ||
      !base_ok(a.weight) || !scales_ok(a.weight_scales) || !base_ok(a.out) ||
      !base_or_null(a.bias) || !base_or_null(a.residual))
    return MOE_ERR_INVALID_ARG;
  const int sms = supported_sm_count();
  if (sms == 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = code_dtype == MOE_DTYPE_FP8_E4M3, bf = out_dtype == MOE_DTYPE_BF16;
  auto run = fp8 ? (bf ? launch_quant_product<__nv_bfloat16, true, kGatedForm>
                       : launch_quant_product<__half, true, kGatedForm>)
                 : (bf ? launch_quant_product<__nv_bfloat16, false, kGatedForm>
                       : launch_quant_product<__half, false, kGatedForm>);
  return finish(run(a, sms, s));
}

}  // namespace

#ifdef MOE_DEBUG_HOOKS
bool set_quant_wait(int slices, unsigned long long wait_ns) {
  return cudaMemcpyToSymbol(g_debug_slices, &slices, sizeof(slices)) == cudaSuccess &&
         cudaMemcpyToSymbol(g_debug_wait_ns, &wait_ns, sizeof(wait_ns)) == cudaSuccess;
}
#endif

}  // namespace experts
}  // namespace moe

using namespace moe;
using namespace moe::experts;

extern "C" {

int moe_quant_rows(const void* rows, moe_dtype_t dtype, const int64_t* expert_first_token_offset,
                   int64_t num_rows, int64_t hidden_size, int32_t num_local_experts,
                   moe_dtype_t code_dtype, void* codes, float* scales, void* workspace,
                   moe_stream_t stream) {
  if (!is_type(dtype) || !is_code(code_dtype) || num_rows < 0 || num_rows > kMostRows ||
      !row_size_ok(hidden_size))
    return MOE_ERR_INVALID_ARG;
  if (expert_first_token_offset != nullptr &&
      (!aligned(expert_first_token_offset, 8) || num_local_experts < 1 ||
       num_local_experts > MOE_MAX_LOCAL_EXPERTS))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (num_rows == 0) return MOE_OK;
  if (!base_ok(rows) || !base_ok(codes) || !scales_ok(scales)) return MOE_ERR_INVALID_ARG;
  const int sms = supported_sm_count();
  if (sms == 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  const QuantRowsArgs a = {rows, expert_first_token_offset, num_rows, hidden_size,
                           num_local_experts, codes, scales, status_of(workspace)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto pick = [&](auto type, auto wide) {
    using T = decltype(type);
    return code_dtype == MOE_DTYPE_FP8_E4M3 ? launch_quant_fp8<T, decltype(wide)::value>
                                            : launch_quant_int8<T, decltype(wide)::value>;
  };
  const bool wide = aligned(rows, 32);
  auto run = dtype == MOE_DTYPE_BF16
                 ? (wide ? pick(__nv_bfloat16(), std::true_type()) : pick(__nv_bfloat16(), std::false_type()))
                 : (wide ? pick(__half(), std::true_type()) : pick(__half(), std::false_type()));
  return finish(run(a, sms, s));
}

int moe_expert_gated_quant(const void* permuted_codes, const float* permuted_scales,
                           const void* weight, const float* weight_scales, moe_dtype_t code_dtype,
                           moe_dtype_t out_dtype, const int64_t* expert_first_token_offset,
                           int64_t num_rows, int64_t hidden_size, int64_t ffn_size,
                           int32_t num_local_experts, moe_activation_t activation, void* out,
                           void* workspace, moe_stream_t stream) {
  if (ffn_size < 0 || ffn_size > INT32_MAX / 4) return MOE_ERR_INVALID_ARG;
  const QuantArgs a = {expert_first_token_offset, num_rows, hidden_size, 2 * ffn_size,
                       num_local_experts, activation, permuted_codes, permuted_scales, weight,
                       weight_scales, nullptr, nullptr, out, status_of(workspace)};
  return product<true>(a, code_dtype, out_dtype, activation, ffn_size, workspace, stream);
}

int moe_expert_linear_quant(const void* codes, const float* scales, const void* weight,
                            const float* weight_scales, moe_dtype_t code_dtype,
                            moe_dtype_t out_dtype, const int64_t* expert_first_token_offset,
                            int64_t num_rows, int64_t in_size, int64_t out_size,
                            int32_t num_local_experts, const void* bias,
                            moe_activation_t activation, const void* residual, void* out,
                            void* workspace, moe_stream_t stream) {
  const QuantArgs a = {expert_first_token_offset, num_rows, in_size, out_size, num_local_experts,
                       activation, codes, scales, weight, weight_scales, bias, residual, out,
                       status_of(workspace)};
  return product<false>(a, code_dtype, out_dtype, activation, out_size, workspace, stream);
}

}  // extern "C"
