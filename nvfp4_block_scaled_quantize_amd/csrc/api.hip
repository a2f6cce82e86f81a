// api.hip -- the C ABI of include/nvfp4_mi355x.h: host-side validation, the
// per-device gfx950 check, workspace checks, stream-ordered launches and the
// external-weight registry.  Nothing here allocates device memory or
// synchronizes; only the registry keeps (caller-owned) pointers.
#include <mutex>
#include <string.h>
#include <unordered_map>

#include "../../include/nvfp4_mi355x.h"
#include "attention.h"
#include "fp8.h"
#include "internal.h"
#include "moe_decode.h"

namespace {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  int ok;        // 1 if gfx950, 0 if not
  int num_cus;   // compute units
};

// Properties of the current device, queried once per device; nullptr if HIP
// reports an error.
const DeviceInfo* current_device() {
  static std::once_flag once[kMaxDevices];
  static DeviceInfo info[kMaxDevices];
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::call_once(once[dev], [dev]() {
    hipDeviceProp_t p;
    const bool got = hipGetDeviceProperties(&p, dev) == hipSuccess;
    info[dev].ok = (got && strncmp(p.gcnArchName, "gfx950", 6) == 0) ? 1 : 0;
    info[dev].num_cus = got ? p.multiProcessorCount : 0;
  });
  return &info[dev];
}

int32_t device_status() {
  const DeviceInfo* d = current_device();
  if (!d) return NVFP4_EHIP;
  return d->ok ? NVFP4_OK : NVFP4_EUNSUPPORTED;
}

int32_t hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_EHIP; }

bool aligned4(const void* p) { return ((uintptr_t)p % 4) == 0; }

struct Bytes {
  const void* p;
  size_t n;
};
bool overlap(const Bytes& a, const Bytes& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}
// Whether one of the first `written` buffers overlaps another of the n.
bool any_overlap(const Bytes* b, int written, int n) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(b[i], b[j])) return true;
  return false;
}
bool aligned256(const void* p) { return ((uintptr_t)p % 256) == 0; }

// External weights of "Fused Nvfp4 GEMM All Reduce Plugin" (external-weight
// mode): (device, resource id) -> the caller's weight and scale pointers.
struct ExternalWeight {
  const uint8_t* weight;
  const uint8_t* scale;
  int32_t out_features, in_features;
};

struct Registry {
  std::mutex mu;
  std::unordered_map<uint64_t, ExternalWeight> map;
};

Registry& registry() {
  static Registry r;
  return r;
}

uint64_t registry_key(int32_t device, int32_t resource_id) {
  return ((uint64_t)(uint32_t)device << 32) | (uint32_t)resource_id;
}

}  // namespace

extern "C" {

const char* nvfp4_status_string(int32_t status) {
  switch (status) {
    case NVFP4_OK: return "ok";
    case NVFP4_EINVAL: return "invalid argument";
    case NVFP4_EUNSUPPORTED: return "unsupported device or size";
    case NVFP4_EWORKSPACE: return "workspace missing or too small";
    case NVFP4_EHIP: return "HIP runtime error";
    case NVFP4_ESCRATCH: return "problem larger than the fixed scratch of the no-allocation entry point";
    default: return "unknown status";
  }
}

size_t nvfp4_quantize_workspace_size(int64_t rows, int64_t k, int64_t group_rows) {
  if (rows <= 0 || k <= 0 || group_rows <= 1 || rows % group_rows != 0) return 0;
  const int np = nvfp4::quant_num_parts(group_rows * k);
  return (size_t)(rows / group_rows) * (size_t)(np + 1) * sizeof(float);
}

static int32_t quantize_common(const void* x, int32_t dtype, int64_t rows, int64_t k_out,
                               int32_t act, int64_t group_rows, uint8_t* codes, uint8_t* sf,
                               float* g_dec, float* scale_out, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP16) return NVFP4_EINVAL;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_SWIGLU && act != NVFP4_ACT_RELU2) return NVFP4_EINVAL;
  if (rows < 0 || k_out <= 0 || (k_out % 16) != 0 || group_rows < 1) return NVFP4_EINVAL;
  if (rows > 0 && (rows % group_rows) != 0) return NVFP4_EINVAL;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !sf || !g_dec) return NVFP4_EINVAL;
  if (!aligned4(g_dec) || (scale_out && !aligned4(scale_out))) return NVFP4_EINVAL;
  if (((uintptr_t)x % 2) != 0) return NVFP4_EINVAL;
  if (rows > 0x7FFFFFFFLL) return NVFP4_EUNSUPPORTED;                // grid.x limit
  const int64_t k_in = (act == NVFP4_ACT_SWIGLU) ? 2 * k_out : k_out;
  if (k_in > (int64_t)1 << 40) return NVFP4_EUNSUPPORTED;
  nvfp4::QuantArgs a{};
  a.x = x; a.dtype = dtype; a.act = act; a.rows = rows; a.k_out = k_out; a.group_rows = group_rows;
  a.codes = codes; a.sf = sf; a.g_dec = g_dec; a.scale_out = scale_out; a.parts = nullptr;
  a.nparts = 0;
  if (group_rows > 1) {
    if ((rows / group_rows) > 65535) return NVFP4_EUNSUPPORTED;   // grid.y limit of the partial pass
    const size_t need = nvfp4_quantize_workspace_size(rows, k_out, group_rows);
    if (!workspace || workspace_bytes < need || !aligned4(workspace)) return NVFP4_EWORKSPACE;
    a.parts = (float*)workspace;
    a.nparts = nvfp4::quant_num_parts(group_rows * k_out);
  }
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  a.num_cus = current_device()->num_cus;
  return hip_status(nvfp4::launch_quantize(a, (hipStream_t)stream));
}

int32_t nvfp4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, int64_t group_rows,
                       uint8_t* codes, uint8_t* sf, float* g_dec, float* scale_out,
                       void* workspace, size_t workspace_bytes, void* stream) {
  return quantize_common(x, dtype, rows, k, NVFP4_ACT_NONE, group_rows, codes, sf, g_dec,
                         scale_out, workspace, workspace_bytes, stream);
}

int32_t nvfp4_mx_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k_out, int32_t act,
                          int64_t group_rows, int32_t layout, uint8_t* codes, uint8_t* sf,
                          float* g_dec, void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP16) return NVFP4_EINVAL;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_SWIGLU && act != NVFP4_ACT_RELU2) return NVFP4_EINVAL;
  if (layout != NVFP4_MX_ROWS && layout != NVFP4_MX_TILED) return NVFP4_EINVAL;
  if (rows < 0 || k_out <= 0 || group_rows < 1) return NVFP4_EINVAL;
  if ((k_out % (layout == NVFP4_MX_TILED ? 128 : 32)) != 0) return NVFP4_EINVAL;
  if (act != NVFP4_ACT_NONE && group_rows != 1) return NVFP4_EINVAL;
  if (rows > 0 && (rows % group_rows) != 0) return NVFP4_EINVAL;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !sf || !g_dec) return NVFP4_EINVAL;
  if (((uintptr_t)x % 16) != 0 || !aligned4(codes) || !aligned4(g_dec)) return NVFP4_EINVAL;
  if (k_out > 32768 || rows > 0x7FFFFF00LL) return NVFP4_EUNSUPPORTED;   // grid of whole 256-row sets
  nvfp4::QuantArgs a{};
  a.x = x; a.dtype = dtype; a.act = act; a.rows = rows; a.k_out = k_out; a.group_rows = group_rows;
  a.codes = codes; a.sf = sf; a.g_dec = g_dec; a.scale_out = nullptr; a.parts = nullptr;
  a.nparts = 0; a.mx = 1; a.tiled = (layout == NVFP4_MX_TILED) ? 1 : 0;
  if (group_rows > 1) {
    if ((rows / group_rows) > 65535) return NVFP4_EUNSUPPORTED;   // grid.y limit of the partial pass
    const size_t need = nvfp4_quantize_workspace_size(rows, k_out, group_rows);
    if (!workspace || workspace_bytes < need || !aligned4(workspace)) return NVFP4_EWORKSPACE;
    a.parts = (float*)workspace;
    a.nparts = nvfp4::quant_num_parts(group_rows * k_out);
  }
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  a.num_cus = current_device()->num_cus;
  return hip_status(nvfp4::launch_quantize(a, (hipStream_t)stream));
}

int32_t nvfp4_mx_tile(const uint8_t* codes, const uint8_t* sf, int64_t rows, int64_t k,
                      uint8_t* codes_tiled, uint8_t* sf_tiled, void* stream) {
  if (rows < 0 || k <= 0 || (k % 128) != 0) return NVFP4_EINVAL;
  if (rows == 0) return NVFP4_OK;
  if (!codes || !sf || !codes_tiled || !sf_tiled) return NVFP4_EINVAL;
  if (((uintptr_t)codes % 16) != 0 || ((uintptr_t)codes_tiled % 16) != 0 ||
      ((uintptr_t)sf_tiled % 2) != 0)
    return NVFP4_EINVAL;
  // four 1 KiB tiles per workgroup of the permutation: grid.x < 2^31
  if (k > (1LL << 24) || (rows + 31) / 32 * (k / 64) > (1LL << 32)) return NVFP4_EUNSUPPORTED;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  return hip_status(nvfp4::launch_mx_tile(codes, sf, rows, k, codes_tiled, sf_tiled,
                                          (hipStream_t)stream));
}

int32_t nvfp4_mx_gemm(const uint8_t* a_tiled, const uint8_t* a_sf_tiled, const float* a_g,
                      int64_t a_group_rows, const uint8_t* w_tiled, const uint8_t* w_sf_tiled,
                      const float* w_gscale, void* y, int64_t B, int64_t N, int64_t K, void* stream) {
  if (B < 0 || N <= 0 || K <= 0 || (N % 32) != 0 || (K % 128) != 0 || a_group_rows < 1)
    return NVFP4_EINVAL;
  if (B > 0 && (B % a_group_rows) != 0) return NVFP4_EINVAL;
  if (B == 0) return NVFP4_OK;
  if (!a_tiled || !a_sf_tiled || !a_g || !w_tiled || !w_sf_tiled || !w_gscale || !y) return NVFP4_EINVAL;
  if (((uintptr_t)a_tiled % 16) != 0 || ((uintptr_t)w_tiled % 16) != 0 || !aligned4(a_sf_tiled) ||
      !aligned4(w_sf_tiled) || !aligned4(a_g) || !aligned4(w_gscale) || ((uintptr_t)y % 16) != 0)
    return NVFP4_EINVAL;
  if (B > 0x7FFFFFE0LL || N > 0x7FFFFFE0LL || K > (1LL << 24)) return NVFP4_EUNSUPPORTED;
  if (((B + 255) / 256) * ((N + 255) / 256) > 0x7FFFFFFFLL) return NVFP4_EUNSUPPORTED;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::MxGemmArgs g{a_tiled, a_sf_tiled, a_g, a_group_rows, w_tiled, w_sf_tiled, w_gscale, y, B, N, K};
  return hip_status(nvfp4::launch_mx_gemm(g, (hipStream_t)stream));
}

int32_t nvfp4_act_quant(const void* x, int32_t dtype, int64_t rows, int64_t k_out, int32_t act,
                        uint8_t* codes, uint8_t* sf, float* g_dec, float* scale_out, void* stream) {
  return quantize_common(x, dtype, rows, k_out, act, 1, codes, sf, g_dec, scale_out, nullptr, 0,
                         stream);
}

size_t nvfp4_gemm_workspace_size(int64_t B, int64_t N, int64_t K) {
  if (B <= 0 || N <= 0 || K <= 0) return 0;
  return nvfp4::gemm_workspace_bytes(B, N, K);
}

int32_t nvfp4_gemm(const uint8_t* a, const float* a_scale, const uint8_t* w, const uint8_t* w_sf,
                   const float* w_gscale, void* y, int64_t B, int64_t N, int64_t K,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || N <= 0 || K <= 0 || (K % 16) != 0) return NVFP4_EINVAL;
  if (B == 0) return NVFP4_OK;
  if (!a || !a_scale || !w || !w_sf || !w_gscale || !y) return NVFP4_EINVAL;
  if (!aligned4(a_scale) || !aligned4(w_gscale) || ((uintptr_t)y % 2) != 0) return NVFP4_EINVAL;
  if (B > 0x7FFFFFFFLL || N > 0x7FFFFFFFLL || K > 0x7FFFFFFFLL) return NVFP4_EUNSUPPORTED;
  const size_t need = nvfp4::gemm_workspace_bytes(B, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned256(workspace)))
    return NVFP4_EWORKSPACE;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::GemmArgs g{a, a_scale, w, w_sf, w_gscale, y, B, N, K, workspace, workspace_bytes, 0};
  return hip_status(nvfp4::launch_gemm(g, (hipStream_t)stream));
}

int32_t nvfp4_pretile_weight(const uint8_t* w, const uint8_t* w_sf, int64_t N, int64_t K,
                             uint8_t* w_tiled, uint8_t* sf_tiled, void* stream) {
  if (N <= 0 || K <= 0 || (N % 16) != 0 || (K % 128) != 0) return NVFP4_EINVAL;
  if (!w || !w_sf || !w_tiled || !sf_tiled) return NVFP4_EINVAL;
  if (((uintptr_t)w % 16) != 0 || ((uintptr_t)w_tiled % 16) != 0 || ((uintptr_t)w_sf % 2) != 0 ||
      ((uintptr_t)sf_tiled % 4) != 0)
    return NVFP4_EINVAL;
  if (N > 0x7FFFFFFFLL || K > (1LL << 24)) return NVFP4_EUNSUPPORTED;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  return hip_status(nvfp4::launch_pretile(w, w_sf, N, K, w_tiled, sf_tiled, (hipStream_t)stream));
}

int32_t nvfp4_gemm_pretiled(const uint8_t* a, const float* a_scale, const uint8_t* w_tiled,
                            const uint8_t* sf_tiled, const float* w_gscale, void* y, int64_t B,
                            int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (B < 0 || N <= 0 || K <= 0 || (N % 16) != 0 || (K % 128) != 0) return NVFP4_EINVAL;
  if (B == 0) return NVFP4_OK;
  if (!a || !a_scale || !w_tiled || !sf_tiled || !w_gscale || !y) return NVFP4_EINVAL;
  if (!aligned4(a_scale) || !aligned4(w_gscale) || ((uintptr_t)y % 2) != 0) return NVFP4_EINVAL;
  if (((uintptr_t)w_tiled % 16) != 0 || ((uintptr_t)sf_tiled % 4) != 0) return NVFP4_EINVAL;
  if (B > 0x7FFFFFFFLL || N > 0x7FFFFFFFLL || K > (1LL << 24)) return NVFP4_EUNSUPPORTED;
  const size_t need = nvfp4::gemm_workspace_bytes(B, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned256(workspace)))
    return NVFP4_EWORKSPACE;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::GemmArgs g{a, a_scale, w_tiled, sf_tiled, w_gscale, y, B, N, K, workspace, workspace_bytes, 1};
  return hip_status(nvfp4::launch_gemm(g, (hipStream_t)stream));
}

int32_t nvfp4_register_weight(int32_t device, int32_t resource_id, const uint8_t* weight,
                              const uint8_t* scale, int32_t out_features, int32_t in_features,
                              int32_t scale_cols) {
  if (device < 0 || resource_id < 0 || !weight || !scale) return NVFP4_EINVAL;
  if (out_features <= 0 || in_features <= 0 || (in_features % 16) != 0 ||
      scale_cols != in_features / 16)
    return NVFP4_EINVAL;
  Registry& r = registry();
  std::lock_guard<std::mutex> lock(r.mu);
  const bool inserted =
      r.map.emplace(registry_key(device, resource_id),
                    ExternalWeight{weight, scale, out_features, in_features}).second;
  return inserted ? NVFP4_OK : NVFP4_EINVAL;
}

int32_t nvfp4_unregister_weight(int32_t device, int32_t resource_id) {
  if (device < 0 || resource_id < 0) return NVFP4_EINVAL;
  Registry& r = registry();
  std::lock_guard<std::mutex> lock(r.mu);
  return r.map.erase(registry_key(device, resource_id)) == 1 ? NVFP4_OK : NVFP4_EINVAL;
}

int32_t nvfp4_gemm_external(const uint8_t* a, const float* a_scale, int32_t resource_id,
                            const float* w_gscale, void* y, int64_t B, int64_t N, int64_t K,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (resource_id < 0) return NVFP4_EINVAL;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return NVFP4_EHIP;
  ExternalWeight ew;
  {
    Registry& r = registry();
    std::lock_guard<std::mutex> lock(r.mu);
    const auto it = r.map.find(registry_key(dev, resource_id));
    if (it == r.map.end()) return NVFP4_EINVAL;
    ew = it->second;
  }
  if (N != ew.out_features || K != ew.in_features) return NVFP4_EINVAL;
  return nvfp4_gemm(a, a_scale, ew.weight, ew.scale, w_gscale, y, B, N, K, workspace,
                    workspace_bytes, stream);
}

size_t nvfp4_moe_w4a16_workspace_size(int32_t tokens, int32_t experts, int32_t top_k,
                                      int32_t hidden, int32_t inter) {
  if (tokens <= 0 || experts <= 0 || top_k <= 0 || hidden <= 0 || inter <= 0) return 0;
  return nvfp4::moe_workspace_bytes(tokens, experts, top_k, hidden, inter);
}

// Argument checks shared by both MoE entry points (everything but the
// workspace); NVFP4_OK for tokens == 0 too (the caller returns early).
static int32_t moe_check(const float* router_logits, const float* correction_bias, const void* x,
                         const uint8_t* w1, const uint8_t* w1_sf, const float* w1_g,
                         const uint8_t* w2, const uint8_t* w2_sf, const float* w2_g, void* out,
                         int32_t tokens, int32_t experts, int32_t top_k, int32_t hidden,
                         int32_t inter, int32_t n_group, int32_t topk_group) {
  if (tokens < 0 || tokens > (1 << 24) || experts <= 0 || experts > 256 || n_group <= 0 ||
      experts % n_group != 0)
    return NVFP4_EINVAL;
  const int gsize = experts / n_group;
  if (topk_group < 1 || topk_group > n_group || top_k < 1 || top_k > 16 ||
      top_k > topk_group * gsize)
    return NVFP4_EINVAL;
  if (hidden <= 0 || inter <= 0 || hidden % 64 != 0 || inter % 64 != 0 || inter > 8192 ||
      (int64_t)hidden * inter > (int64_t(1) << 31))
    return NVFP4_EINVAL;
  if (tokens == 0) return NVFP4_OK;
  if (!router_logits || !correction_bias || !x || !w1 || !w1_sf || !w1_g || !w2 || !w2_sf ||
      !w2_g || !out)
    return NVFP4_EINVAL;
  if (((uintptr_t)x % 16) != 0 || ((uintptr_t)out % 8) != 0 || ((uintptr_t)w1 % 16) != 0 ||
      ((uintptr_t)w2 % 16) != 0 || !aligned4(w1_sf) || !aligned4(w2_sf) ||
      !aligned4(router_logits) || !aligned4(correction_bias) || !aligned4(w1_g) || !aligned4(w2_g))
    return NVFP4_EINVAL;
  return NVFP4_OK;
}

int32_t nvfp4_moe_w4a16(const float* router_logits, const float* correction_bias, const void* x,
                        const uint8_t* w1, const uint8_t* w1_sf, const float* w1_g,
                        const uint8_t* w2, const uint8_t* w2_sf, const float* w2_g, void* out,
                        int32_t* topk_ids_out, float* topk_w_out, int32_t tokens, int32_t experts,
                        int32_t top_k, int32_t hidden, int32_t inter, int32_t n_group,
                        int32_t topk_group, int32_t norm_topk_prob, float routed_scaling,
                        void* workspace, size_t workspace_bytes, void* stream) {
  const int32_t st = moe_check(router_logits, correction_bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g,
                               out, tokens, experts, top_k, hidden, inter, n_group, topk_group);
  if (st != NVFP4_OK || tokens == 0) return st;
  const size_t need = nvfp4::moe_workspace_bytes(tokens, experts, top_k, hidden, inter);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return NVFP4_EWORKSPACE;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::MoeArgs m{router_logits, correction_bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, out,
                   topk_ids_out, topk_w_out, tokens, experts, top_k, hidden, inter, n_group,
                   topk_group, norm_topk_prob ? 1 : 0, routed_scaling, workspace, workspace_bytes,
                   current_device()->num_cus, 0};
  return hip_status(nvfp4::launch_moe(m, (hipStream_t)stream));
}

int32_t nvfp4_moe_w4a16_pretiled(const float* router_logits, const float* correction_bias,
                                 const void* x, const uint8_t* w1, const uint8_t* w1_sf,
                                 const float* w1_g, const uint8_t* w2, const uint8_t* w2_sf,
                                 const float* w2_g, void* out, int32_t* topk_ids_out,
                                 float* topk_w_out, int32_t tokens, int32_t experts, int32_t top_k,
                                 int32_t hidden, int32_t inter, int32_t n_group,
                                 int32_t topk_group, int32_t norm_topk_prob, float routed_scaling,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  const int32_t st = moe_check(router_logits, correction_bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g,
                               out, tokens, experts, top_k, hidden, inter, n_group, topk_group);
  if (st != NVFP4_OK) return st;
  if (hidden % 128 != 0 || inter % 128 != 0) return NVFP4_EINVAL;   // whole 128-k chunks
  if (tokens == 0) return NVFP4_OK;
  const size_t need = nvfp4::moe_workspace_bytes(tokens, experts, top_k, hidden, inter);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return NVFP4_EWORKSPACE;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::MoeArgs m{router_logits, correction_bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, out,
                   topk_ids_out, topk_w_out, tokens, experts, top_k, hidden, inter, n_group,
                   topk_group, norm_topk_prob ? 1 : 0, routed_scaling, workspace, workspace_bytes,
                   current_device()->num_cus, 1};
  return hip_status(nvfp4::launch_moe(m, (hipStream_t)stream));
}

int32_t nvfp4_moe_w4a16_noalloc(const float* router_logits, const float* correction_bias,
                                const void* x, const uint8_t* w1, const uint8_t* w1_sf,
                                const float* w1_g, const uint8_t* w2, const uint8_t* w2_sf,
                                const float* w2_g, void* out, int32_t* topk_ids_out,
                                float* topk_w_out, int32_t tokens, int32_t experts, int32_t top_k,
                                int32_t hidden, int32_t inter, int32_t n_group, int32_t topk_group,
                                int32_t norm_topk_prob, float routed_scaling, void* stream) {
  const int32_t st = moe_check(router_logits, correction_bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g,
                               out, tokens, experts, top_k, hidden, inter, n_group, topk_group);
  if (st != NVFP4_OK || tokens == 0) return st;
  const size_t need = nvfp4::moe_workspace_bytes(tokens, experts, top_k, hidden, inter);
  if (need > (size_t)NVFP4_NOALLOC_SCRATCH_BYTES) return NVFP4_ESCRATCH;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  void* scratch = nullptr;
  size_t scratch_bytes = 0;
  if (nvfp4::moe_noalloc_scratch(&scratch, &scratch_bytes) != hipSuccess || scratch_bytes < need)
    return NVFP4_EHIP;
  nvfp4::MoeArgs m{router_logits, correction_bias, x, w1, w1_sf, w1_g, w2, w2_sf, w2_g, out,
                   topk_ids_out, topk_w_out, tokens, experts, top_k, hidden, inter, n_group,
                   topk_group, norm_topk_prob ? 1 : 0, routed_scaling, scratch, scratch_bytes,
                   current_device()->num_cus, 0};
  return hip_status(nvfp4::launch_moe(m, (hipStream_t)stream));
}

static bool moe_decode_sizes(int32_t tokens, int32_t experts, int32_t top_k, int32_t hidden, int32_t inter) {
  return tokens >= 0 && experts >= 1 && experts <= 256 && top_k >= 1 && top_k <= 16 && top_k <= experts && hidden >= 64 &&
         hidden % 64 == 0 && inter >= 64 && inter % 64 == 0;
}

size_t nvfp4_moe_decode_workspace_size(int32_t tokens, int32_t experts, int32_t top_k, int32_t hidden, int32_t inter) {
  if (!moe_decode_sizes(tokens, experts, top_k, hidden, inter) || tokens < 1 || tokens > nvfp4::kMoeDecodeMaxTokens ||
      hidden > 65536 || inter > 65536)
    return 0;
  return nvfp4::moe_decode_workspace_bytes(tokens, experts, top_k, hidden, inter);
}

int32_t nvfp4_moe_decode(const void* x, int32_t dtype, const void* router, const float* correction_bias,
                         const uint8_t* w1, const uint8_t* w1_sf, const float* w1_g, const uint8_t* w2,
                         const uint8_t* w2_sf, const float* w2_g, int32_t tiled, void* out, int32_t* topk_ids_out,
                         float* topk_w_out, int32_t tokens, int32_t experts, int32_t top_k, int32_t hidden,
                         int32_t inter, int32_t act, int32_t n_group, int32_t topk_group, int32_t norm_topk_prob,
                         float routed_scaling, void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP16) return NVFP4_EINVAL;
  if (act != NVFP4_ACT_SWIGLU && act != NVFP4_ACT_RELU2) return NVFP4_EINVAL;
  if (!moe_decode_sizes(tokens, experts, top_k, hidden, inter)) return NVFP4_EINVAL;
  if (n_group < 1 || experts % n_group != 0 || topk_group < 1 || topk_group > n_group ||
      top_k > topk_group * (experts / n_group))
    return NVFP4_EINVAL;
  if (tiled && (hidden % 128 != 0 || inter % 128 != 0)) return NVFP4_EINVAL;   // whole 128-k chunks
  if (tokens > nvfp4::kMoeDecodeMaxTokens || hidden > 65536 || inter > 65536) return NVFP4_EUNSUPPORTED;
  if (tokens == 0) return NVFP4_OK;
  if (!x || !router || !correction_bias || !w1 || !w1_sf || !w1_g || !w2 || !w2_sf || !w2_g || !out) return NVFP4_EINVAL;
  if ((((uintptr_t)x | (uintptr_t)router | (uintptr_t)w1 | (uintptr_t)w2) % 16) != 0 || ((uintptr_t)out % 8) != 0 ||
      !aligned4(w1_sf) || !aligned4(w2_sf) || !aligned4(correction_bias) || !aligned4(w1_g) ||
      !aligned4(w2_g) || !aligned4(topk_ids_out) || !aligned4(topk_w_out))
    return NVFP4_EINVAL;
  const size_t need = nvfp4::moe_decode_workspace_bytes(tokens, experts, top_k, hidden, inter);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return NVFP4_EWORKSPACE;
  // what is written overlaps nothing else, but out may be x
  const size_t t = (size_t)tokens, e = (size_t)experts, values = (size_t)hidden * inter;
  const size_t n1 = e * values * (act == NVFP4_ACT_SWIGLU ? 2 : 1), n2 = e * values, pairs = t * top_k * 4, io = t * hidden * 2;
  const Bytes all[] = {{out, io}, {topk_ids_out, topk_ids_out ? pairs : 0}, {topk_w_out, topk_w_out ? pairs : 0},
                       {workspace, need}, {router, e * hidden * 2}, {correction_bias, e * 4}, {w1, n1 / 2}, {w1_sf, n1 / 16},
                       {w1_g, e * 4}, {w2, n2 / 2}, {w2_sf, n2 / 16}, {w2_g, e * 4}, {x, out == x ? 0 : io}};
  if (any_overlap(all, 4, 13)) return NVFP4_EINVAL;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::MoeDecodeArgs m{x, dtype, router, correction_bias, w1, w1_sf, w1_g, w2, w2_sf, w2_g, out, topk_ids_out,
                         topk_w_out, tokens, experts, top_k, hidden, inter, act, n_group, topk_group,
                         norm_topk_prob ? 1 : 0, routed_scaling, tiled ? 1 : 0, workspace};
  return hip_status(nvfp4::launch_moe_decode(m, (hipStream_t)stream));
}

int32_t nvfp4_page_maps(const int32_t* ctx_lens, const int32_t* new_lens, int32_t seqs,
                        int32_t* block_table, int32_t max_pages, const int32_t* free_pages,
                        int32_t num_free, int32_t page_size, int64_t tokens, int32_t* cu_new,
                        int32_t* kv_lens, int64_t* slot_map, int32_t* positions, int32_t* taken,
                        void* stream) {
  if (seqs < 0 || max_pages < 0 || num_free < 0 || page_size < 1 || tokens < 0) return NVFP4_EINVAL;
  if (!cu_new || !taken || !aligned4(cu_new) || !aligned4(taken)) return NVFP4_EINVAL;
  if (seqs > 0 && (!ctx_lens || !new_lens || !kv_lens)) return NVFP4_EINVAL;
  if (seqs > 0 && max_pages > 0 && !block_table) return NVFP4_EINVAL;
  if (num_free > 0 && !free_pages) return NVFP4_EINVAL;
  if (tokens > 0 && (!slot_map || !positions)) return NVFP4_EINVAL;
  if (!aligned4(ctx_lens) || !aligned4(new_lens) || !aligned4(block_table) || !aligned4(free_pages) ||
      !aligned4(kv_lens) || ((uintptr_t)slot_map % 8) != 0 || !aligned4(positions))
    return NVFP4_EINVAL;
  if (seqs > (1 << 20) || tokens > 0x7FFF0000LL) return NVFP4_EUNSUPPORTED;
  // every workgroup reads the inputs while others already write: what is written overlaps nothing else,
  // but for lengths updated in place (see launch_page_maps)
  const size_t n = (size_t)seqs, t = (size_t)tokens;
  const Bytes all[] = {{block_table, n * max_pages * 4}, {cu_new, (n + 1) * 4}, {kv_lens, n * 4}, {slot_map, t * 8},
                       {positions, t * 4}, {taken, 4}, {ctx_lens, n * 4}, {new_lens, n * 4},
                       {free_pages, (size_t)num_free * 4}};
  constexpr int kWritten = 6, kAll = 9, kKvLens = 2, kCtxLens = 6;
  for (int i = 0; i < kWritten; ++i)
    for (int j = i + 1; j < kAll; ++j) {
      const bool in_place = i == kKvLens && j == kCtxLens && kv_lens == ctx_lens;
      if (overlap(all[i], all[j]) && !in_place) return NVFP4_EINVAL;
    }
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::PageMapsArgs a{ctx_lens, new_lens, block_table, free_pages, seqs, max_pages, num_free, page_size,
                        tokens, cu_new, kv_lens, slot_map, positions, taken};
  return hip_status(nvfp4::launch_page_maps(a, (hipStream_t)stream));
}

int32_t nvfp4_kv_write(const void* k, const void* v, int64_t tokens, int32_t kv_heads, int32_t head_dim,
                       int64_t k_stride, int64_t k_head_stride, int64_t v_stride, int64_t v_head_stride,
                       const int64_t* slot_map, void* k_cache, void* v_cache, int32_t page_size,
                       int64_t num_pages, void* stream) {
  if (tokens < 0 || kv_heads < 1 || head_dim < 1 || page_size < 1 || num_pages < 0) return NVFP4_EINVAL;
  if (k_stride < 0 || k_head_stride < 0 || v_stride < 0 || v_head_stride < 0) return NVFP4_EINVAL;
  if (tokens == 0 || num_pages == 0) return NVFP4_OK;
  if (!k || !v || !slot_map || !k_cache || !v_cache) return NVFP4_EINVAL;
  if ((((uintptr_t)k | (uintptr_t)v | (uintptr_t)k_cache | (uintptr_t)v_cache) % 2) != 0 ||
      ((uintptr_t)slot_map % 8) != 0)
    return NVFP4_EINVAL;
  // the kernel divides element and slot numbers below 2^51
  if (kv_heads > 65536 || head_dim > 65536 || tokens > (1LL << 50) / ((int64_t)kv_heads * head_dim) ||
      num_pages > (1LL << 50) / page_size)
    return NVFP4_EUNSUPPORTED;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::KvWriteArgs a{k, v, tokens, kv_heads, head_dim, k_stride, k_head_stride, v_stride, v_head_stride,
                       slot_map, k_cache, v_cache, page_size, num_pages};
  return hip_status(nvfp4::launch_kv_write(a, (hipStream_t)stream));
}

// Whether the rows [tokens, heads] of dim elements lie apart: heads within tokens, or tokens within heads.
static bool rows_apart(int64_t tokens, int64_t heads, int64_t dim, int64_t stride, int64_t head_stride) {
  if (tokens <= 1 && heads <= 1) return true;
  if (tokens <= 1) return head_stride >= dim;
  if (heads <= 1) return stride >= dim;
  auto inside = [dim](int64_t n, int64_t small, int64_t large) {   // n rows `small` apart, again after `large`
    return small >= dim && large >= dim && small <= (large - dim) / (n - 1);
  };
  return inside(heads, head_stride, stride) || inside(tokens, stride, head_stride);
}

int32_t nvfp4_rope_kv_write(const void* q, const void* k, const void* v, int32_t dtype, int64_t tokens,
                            int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t q_stride,
                            int64_t q_head_stride, int64_t k_stride, int64_t k_head_stride, int64_t v_stride,
                            int64_t v_head_stride, const int32_t* positions, const float* inv_freq,
                            int32_t rotary_dim, int32_t interleaved, float mscale, const int64_t* slot_map,
                            void* q_out, int64_t q_out_stride, int64_t q_out_head_stride, void* k_out,
                            int64_t k_out_stride, int64_t k_out_head_stride, void* k_cache, void* v_cache,
                            int32_t page_size, int64_t num_pages, void* stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP16) return NVFP4_EINVAL;
  if (tokens < 0 || q_heads < 0 || kv_heads < 1 || head_dim < 2 || page_size < 1 || num_pages < 0) return NVFP4_EINVAL;
  if (rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2 != 0) return NVFP4_EINVAL;
  if (!(mscale >= -0x1p96f && mscale <= 0x1p96f)) return NVFP4_EINVAL;
  if (q_stride < 0 || q_head_stride < 0 || k_stride < 0 || k_head_stride < 0 || v_stride < 0 || v_head_stride < 0 ||
      q_out_stride < 0 || q_out_head_stride < 0 || k_out_stride < 0 || k_out_head_stride < 0)
    return NVFP4_EINVAL;
  if (rotary_dim > 512 || q_heads > 65536 || kv_heads > 65536 ||
      ((int64_t)q_heads + 2 * (int64_t)kv_heads) * head_dim > (1 << 24) || tokens >= (1 << 24) ||
      num_pages > (1LL << 50) / page_size)
    return NVFP4_EUNSUPPORTED;
  if (tokens == 0) return NVFP4_OK;
  if (!k || !v || !positions || !inv_freq || !slot_map || (q_heads > 0 && (!q || !q_out)) ||
      (num_pages > 0 && (!k_cache || !v_cache)))
    return NVFP4_EINVAL;
  if ((((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)k_out | (uintptr_t)k_cache |
        (uintptr_t)v_cache) % 2) != 0 || !aligned4(positions) || !aligned4(inv_freq) || ((uintptr_t)slot_map % 8) != 0)
    return NVFP4_EINVAL;
  if ((q_heads > 0 && !rows_apart(tokens, q_heads, head_dim, q_out_stride, q_out_head_stride)) ||
      (k_out && !rows_apart(tokens, kv_heads, head_dim, k_out_stride, k_out_head_stride)))
    return NVFP4_EINVAL;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::RopeKvArgs a{};
  a.q = q; a.k = k; a.v = v; a.dtype = dtype; a.tokens = tokens; a.q_heads = q_heads; a.kv_heads = kv_heads;
  a.head_dim = head_dim; a.q_stride = q_stride; a.q_head_stride = q_head_stride; a.k_stride = k_stride;
  a.k_head_stride = k_head_stride; a.v_stride = v_stride; a.v_head_stride = v_head_stride; a.positions = positions;
  a.inv_freq = inv_freq; a.rotary_dim = rotary_dim; a.interleaved = interleaved ? 1 : 0; a.mscale = mscale;
  a.slot_map = slot_map; a.q_out = q_out; a.qo_stride = q_out_stride; a.qo_head_stride = q_out_head_stride;
  a.k_out = k_out; a.ko_stride = k_out_stride; a.ko_head_stride = k_out_head_stride; a.k_cache = k_cache;
  a.v_cache = v_cache; a.page_size = page_size; a.num_pages = num_pages;
  return hip_status(nvfp4::launch_rope_kv(a, (hipStream_t)stream));
}

int32_t nvfp4_fp8_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, int32_t act, int32_t block_rows,
                           uint8_t* codes, float* scale, void* stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP16) return NVFP4_EINVAL;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_SWIGLU && act != NVFP4_ACT_RELU2) return NVFP4_EINVAL;
  if (rows < 0 || k <= 0 || k % 16 != 0 || (block_rows != 1 && block_rows != 128)) return NVFP4_EINVAL;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !scale || ((uintptr_t)x % 2) != 0 || !aligned4(scale)) return NVFP4_EINVAL;
  // one launch: fewer than 2^32 threads
  const int64_t nkb = (k + 127) / 128;
  if (k > (1LL << 30) || rows > (1LL << 37)) return NVFP4_EUNSUPPORTED;
  if (block_rows == 1 ? rows > ((1LL << 30) - (1 << 16)) / nkb : (rows + 127) / 128 > ((1LL << 24) - 1) / nkb)
    return NVFP4_EUNSUPPORTED;
  // workgroups write while others still read
  const size_t r = (size_t)rows, row = (size_t)k * (act == NVFP4_ACT_SWIGLU ? 4 : 2);
  const Bytes all[] = {{codes, r * k}, {scale, (r + block_rows - 1) / block_rows * nkb * 4}, {x, r * row}};
  if (any_overlap(all, 2, 3)) return NVFP4_EINVAL;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::Fp8QuantArgs a{x, dtype, act, rows, (int)k, block_rows, codes, scale};
  return hip_status(nvfp4::launch_fp8_quantize(a, (hipStream_t)stream));
}

int32_t nvfp4_fp8_gemm(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale, void* y,
                       int32_t out_dtype, int64_t B, int64_t N, int64_t K, void* stream) {
  if (out_dtype != NVFP4_BF16 && out_dtype != NVFP4_FP16) return NVFP4_EINVAL;
  if (B < 0 || N <= 0 || K <= 0 || K % 16 != 0) return NVFP4_EINVAL;
  if (B == 0) return NVFP4_OK;
  if (!a || !a_scale || !w || !w_scale || !y) return NVFP4_EINVAL;
  if ((((uintptr_t)a | (uintptr_t)w) % 16) != 0 || !aligned4(a_scale) || !aligned4(w_scale) || ((uintptr_t)y % 2) != 0)
    return NVFP4_EINVAL;
  // offsets inside a tile of 256 rows are 32 bits; tiles are counted in 24 bits
  if (K >= (1 << 24) || B > (1 << 30) || N > (1 << 30) ||
      ((B + 127) / 128) * ((N + 127) / 128) > (1 << 22))
    return NVFP4_EUNSUPPORTED;
  const size_t nkb = ((size_t)K + 127) / 128;
  const Bytes all[] = {{y, (size_t)B * N * 2}, {a, (size_t)B * K}, {a_scale, B * nkb * 4}, {w, (size_t)N * K},
                       {w_scale, ((size_t)N + 127) / 128 * nkb * 4}};
  if (any_overlap(all, 1, 5)) return NVFP4_EINVAL;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::Fp8GemmArgs g{a, a_scale, w, w_scale, y, out_dtype, (int)B, (int)N, (int)K};
  return hip_status(nvfp4::launch_fp8_gemm(g, (hipStream_t)stream));
}

// Checks shared by both attention entry points.
static int32_t attn_check(const void* q, int32_t dtype, int32_t seqs, int64_t tokens, int32_t q_heads,
                          int32_t kv_heads, int32_t head_dim, int64_t q_stride, int64_t q_head_stride,
                          float scale, int32_t window, const void* out, const float* lse) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_FP16) return NVFP4_EINVAL;
  if (seqs < 0 || tokens < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return NVFP4_EINVAL;
  if (head_dim < 8 || head_dim > 128 || head_dim % 8 != 0 || window < 0) return NVFP4_EINVAL;
  // scale log2 e and its inverse are normal numbers
  if (!(scale >= 0x1p-96f && scale <= 0x1p96f)) return NVFP4_EINVAL;
  if (q_stride < 0 || q_head_stride < 0 || q_stride % 8 != 0 || q_head_stride % 8 != 0) return NVFP4_EINVAL;
  if (tokens == 0) return NVFP4_OK;
  if (!q || !out || ((uintptr_t)q % 16) != 0 || ((uintptr_t)out % 16) != 0 || !aligned4(lse)) return NVFP4_EINVAL;
  if (q_heads > 65536 || seqs > (1 << 20) || tokens > (1LL << 30) ||
      tokens * (q_heads / kv_heads) > (1LL << 30))
    return NVFP4_EUNSUPPORTED;
  return NVFP4_OK;
}

int32_t nvfp4_prompt_attn(const void* q, const void* k, const void* v, int32_t dtype, const int32_t* cu_seqlens,
                          int32_t seqs, int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                          int64_t q_stride, int64_t q_head_stride, int64_t k_stride, int64_t k_head_stride,
                          int64_t v_stride, int64_t v_head_stride, float scale, int32_t window, void* out,
                          float* lse, void* stream) {
  const int32_t st = attn_check(q, dtype, seqs, tokens, q_heads, kv_heads, head_dim, q_stride, q_head_stride,
                                scale, window, out, lse);
  if (st != NVFP4_OK) return st;
  if (k_stride < 0 || k_head_stride < 0 || v_stride < 0 || v_head_stride < 0 ||
      ((k_stride | k_head_stride | v_stride | v_head_stride) % 8) != 0)
    return NVFP4_EINVAL;
  if (tokens == 0) return NVFP4_OK;
  if (!k || !v || !cu_seqlens || !aligned4(cu_seqlens) || (((uintptr_t)k | (uintptr_t)v) % 16) != 0)
    return NVFP4_EINVAL;
  nvfp4::AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.dtype = dtype; a.cu = cu_seqlens; a.seqs = seqs; a.tokens = (int)tokens;
  a.q_heads = q_heads; a.kv_heads = kv_heads; a.head_dim = head_dim;
  a.q_stride = q_stride; a.q_head_stride = q_head_stride; a.k_stride = k_stride;
  a.k_head_stride = k_head_stride; a.v_stride = v_stride; a.v_head_stride = v_head_stride;
  a.scale = scale; a.window = window; a.out = out; a.lse = lse;
  if (!nvfp4::prompt_attn_fits(a)) return NVFP4_EUNSUPPORTED;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  return hip_status(nvfp4::launch_prompt_attn(a, (hipStream_t)stream));
}

size_t nvfp4_paged_attn_workspace_size(int32_t seqs, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                                       int32_t head_dim) {
  if (seqs < 0 || tokens <= 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 8 ||
      head_dim > 128)
    return 0;
  return nvfp4::paged_attn_workspace_bytes(seqs, tokens, q_heads, kv_heads, head_dim);
}

int32_t nvfp4_paged_attn(const void* q, int32_t dtype, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, const int32_t* cu_new, const int32_t* kv_lens, int32_t seqs,
                         int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t page_size,
                         int64_t num_pages, int32_t max_pages, int64_t q_stride, int64_t q_head_stride,
                         float scale, int32_t window, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const int32_t st = attn_check(q, dtype, seqs, tokens, q_heads, kv_heads, head_dim, q_stride, q_head_stride,
                                scale, window, out, lse);
  if (st != NVFP4_OK) return st;
  if (page_size < 1 || num_pages < 0 || max_pages < 0) return NVFP4_EINVAL;
  if ((int64_t)max_pages * page_size > (1LL << 30) || num_pages > (1LL << 31)) return NVFP4_EUNSUPPORTED;
  if (tokens == 0) return NVFP4_OK;
  if (!cu_new || !aligned4(cu_new)) return NVFP4_EINVAL;
  if (seqs > 0 && (!kv_lens || !aligned4(kv_lens))) return NVFP4_EINVAL;
  if (seqs > 0 && max_pages > 0 && (!block_table || !aligned4(block_table))) return NVFP4_EINVAL;
  if (num_pages > 0 && (!k_cache || !v_cache)) return NVFP4_EINVAL;
  if ((((uintptr_t)k_cache | (uintptr_t)v_cache) % 16) != 0) return NVFP4_EINVAL;
  const size_t need = nvfp4::paged_attn_workspace_bytes(seqs, tokens, q_heads, kv_heads, head_dim);
  if (!workspace || workspace_bytes < need || !aligned256(workspace)) return NVFP4_EWORKSPACE;
  const int32_t ds = device_status();
  if (ds != NVFP4_OK) return ds;
  nvfp4::AttnArgs a{};
  a.q = q; a.k = k_cache; a.v = v_cache; a.dtype = dtype; a.cu = cu_new; a.kv_lens = kv_lens;
  a.block_table = block_table; a.seqs = seqs; a.tokens = (int)tokens; a.q_heads = q_heads;
  a.kv_heads = kv_heads; a.head_dim = head_dim; a.page_size = page_size; a.max_pages = max_pages;
  a.num_pages = num_pages; a.q_stride = q_stride; a.q_head_stride = q_head_stride; a.scale = scale;
  a.window = window; a.out = out; a.lse = lse; a.workspace = workspace;
  return hip_status(nvfp4::launch_paged_attn(a, (hipStream_t)stream));
}

}  // extern "C"
