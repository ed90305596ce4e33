// expert_api.cu -- the C ABI of the expert operators: argument checks,
// workspace carving and kernel launches. See include/moe_ep.h for the
// contract of every entry point.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include "expert_internal.cuh"
#include "moe_ep.h"

namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int validate(const moe_expert_config_t* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->num_experts < 1 || c->hidden < 1 || c->inter < 1 || c->rows_max < 1)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_BF16 && c->dtype != MOE_FP8_E4M3) return MOE_ERR_INVALID_ARG;
  if (c->train != 0 && c->train != 1) return MOE_ERR_INVALID_ARG;
  const bool fp8 = c->dtype == MOE_FP8_E4M3;
  const int unit = fp8 ? 128 : 8;
  if (c->num_experts > MOE_MAX_EXPERTS || c->hidden % unit != 0 || c->inter % unit != 0 ||
      (fp8 && c->train))
    return MOE_ERR_UNSUPPORTED;
  // int32 row indices with room for a tile past the end, and int32 columns of
  // the joint gate and up projection
  if (c->rows_max >= (1ll << 31) - 256 || c->inter > (1 << 29) || c->hidden > (1 << 29))
    return MOE_ERR_UNSUPPORTED;
  // int32 tile numbers: 128 rows x 128 columns at least, per expert and widest
  // side of a product
  const long long wide = (c->hidden > 2ll * c->inter ? c->hidden : 2ll * c->inter) / 128 + 1;
  constexpr long long kMost = (1ll << 31) - 4096;  // a step past the last tile fits too
  if ((c->rows_max / 128 + c->num_experts) * wide >= kMost ||
      wide * wide * c->num_experts >= kMost)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t workspace_bytes(const moe_expert_config_t* c) {
  return kAlign + (c->train ? (size_t)c->rows_max * 2 * c->inter * 2 : 0);
}

moe::ExpertArgs expert_args(moe_expert_t x, const int32_t* offset) {
  moe::ExpertArgs a{};
  a.offset = offset;
  a.E = x->cfg.num_experts;
  a.rows_max = x->cfg.rows_max;
  a.F = x->cfg.inter;
  a.status = x->status;
  a.wait_limit = x->wait_limit;
  return a;
}

// Whether the few-rows kernels run: they stream each expert's weights once for
// every eight rows it has. By the rows a call can have and their average per
// expert. Measured (us, tiles / few rows; top-8 of E = 256, H = 7168, F = 2048):
// gated bf16 110 / 86 at 8 rows, 545 / 529 at 64, 1414 / 1381 at 256, 2169 /
// 2546 at 1536; gated e4m3 307 / 289 at 64; down bf16 71 / 50 at 8, 277 / 261
// at 64; down e4m3, with little to read per row of weights, 47 / 37 at 8,
// 113 / 92 at 32, 154 / 166 at 64. E = 8, H = 4096, F = 1408, gated bf16:
// 48 / 42 at 32, 49 / 61 at 128. Above 64 rows the gain is a few per cent and
// one expert with all of them would cost many passes.
bool use_rows(moe_expert_t x, moe::ExpertOp op) {
  const long long E3 = 3ll * x->cfg.num_experts, rows = x->cfg.rows_max;
  const bool fp8_down = op == moe::kDown && x->cfg.dtype == MOE_FP8_E4M3;
  return rows <= (E3 > 8 ? E3 : 8) && rows <= (fp8_down ? 48 : 64);
}

cudaError_t forward(moe_expert_t x, moe::ExpertOp op, const moe::ExpertArgs& a, const void* in,
                    const void* w, void* stream) {
  const bool fp8 = x->cfg.dtype == MOE_FP8_E4M3;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return use_rows(x, op) ? moe::launch_expert_rows(op, fp8, a, in, w, x->num_sms, st)
                     : moe::launch_expert_gemm(op, fp8, a, in, w, x->num_sms, st);
}

}  // namespace

extern "C" {

size_t moe_expert_workspace_bytes(const moe_expert_config_t* cfg) {
  return validate(cfg) == MOE_OK ? workspace_bytes(cfg) : 0;
}

int moe_expert_create(const moe_expert_config_t* cfg, void* d_workspace, size_t bytes,
                      moe_expert_t* out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  const int rc = validate(cfg);
  if (rc != MOE_OK) return rc;
  if (!d_workspace) return MOE_ERR_INVALID_ARG;
  if (bytes < workspace_bytes(cfg) || !aligned(d_workspace, kAlign)) return MOE_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      moe::expert_gemm_prepare() != cudaSuccess ||
      cudaMemset(d_workspace, 0, kAlign) != cudaSuccess ||
      cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess)  // before work on any stream
    return MOE_ERR_CUDA;
  moe_expert* x = static_cast<moe_expert*>(calloc(1, sizeof(moe_expert)));
  if (!x) return MOE_ERR_INVALID_ARG;
  x->cfg = *cfg;
  x->device = dev;
  x->num_sms = sms;
  x->status = static_cast<uint32_t*>(d_workspace);
  x->dgu = cfg->train ? reinterpret_cast<uint16_t*>(static_cast<char*>(d_workspace) + kAlign)
                      : nullptr;
  x->wait_limit = 1ll << 32;
  *out = x;
  return MOE_OK;
}

int moe_expert_destroy(moe_expert_t x) {
  free(x);
  return MOE_OK;
}

int moe_expert_gated(moe_expert_t x, const int32_t* expert_offset, const void* in,
                     const float* in_scale, const void* w13, const float* w13_scale, void* hid,
                     float* hid_scale, void* gate_up, void* stream) {
  if (!x || !expert_offset || !in || !w13 || !hid) return MOE_ERR_INVALID_ARG;
  const bool fp8 = x->cfg.dtype == MOE_FP8_E4M3;
  if (fp8 ? (!in_scale || !w13_scale || !hid_scale || gate_up)
          : (in_scale || w13_scale || hid_scale))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(in, 16) || !aligned(w13, 16) || !aligned(hid, 16) || !aligned(gate_up, 16) ||
      !aligned(expert_offset, 4) || !aligned(in_scale, 4) || !aligned(w13_scale, 4) ||
      !aligned(hid_scale, 4))
    return MOE_ERR_INVALID_ARG;
  moe::ExpertArgs a = expert_args(x, expert_offset);
  a.N = x->cfg.inter;
  a.K = x->cfg.hidden;
  a.sa = in_scale;
  a.sb = w13_scale;
  a.out = hid;
  a.out_scale = hid_scale;
  a.gu_out = static_cast<uint16_t*>(gate_up);
  return cuda_rc(forward(x, moe::kGated, a, in, w13, stream));
}

int moe_expert_down(moe_expert_t x, const int32_t* expert_offset, const void* hid,
                    const float* hid_scale, const void* w2, const float* w2_scale, void* y,
                    void* stream) {
  if (!x || !expert_offset || !hid || !w2 || !y) return MOE_ERR_INVALID_ARG;
  const bool fp8 = x->cfg.dtype == MOE_FP8_E4M3;
  if (fp8 ? (!hid_scale || !w2_scale) : (hid_scale || w2_scale)) return MOE_ERR_INVALID_ARG;
  if (!aligned(hid, 16) || !aligned(w2, 16) || !aligned(y, 16) || !aligned(expert_offset, 4) ||
      !aligned(hid_scale, 4) || !aligned(w2_scale, 4))
    return MOE_ERR_INVALID_ARG;
  moe::ExpertArgs a = expert_args(x, expert_offset);
  a.N = x->cfg.hidden;
  a.K = x->cfg.inter;
  a.sa = hid_scale;
  a.sb = w2_scale;
  a.out = y;
  return cuda_rc(forward(x, moe::kDown, a, hid, w2, stream));
}

int moe_expert_backward(moe_expert_t x, const int32_t* expert_offset, const void* in,
                        const void* gate_up, const void* hid, const void* dy, const void* w13,
                        const void* w2, void* dx, void* dw13, void* dw2, void* stream) {
  if (!x || !expert_offset || !in || !gate_up || !hid || !dy || !w13 || !w2)
    return MOE_ERR_INVALID_ARG;
  if ((!dw13) != (!dw2) || (!dx && !dw13)) return MOE_ERR_INVALID_ARG;
  if (!aligned(in, 16) || !aligned(gate_up, 16) || !aligned(hid, 16) || !aligned(dy, 16) ||
      !aligned(w13, 16) || !aligned(w2, 16) || !aligned(dx, 16) || !aligned(dw13, 16) ||
      !aligned(dw2, 16) || !aligned(expert_offset, 4))
    return MOE_ERR_INVALID_ARG;
  if (!x->cfg.train) return MOE_ERR_STATE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int H = x->cfg.hidden, F = x->cfg.inter;
  moe::ExpertArgs a = expert_args(x, expert_offset);
  a.N = F;
  a.K = H;
  a.gu = static_cast<const uint16_t*>(gate_up);
  a.out = x->dgu;
  cudaError_t e = moe::launch_expert_gemm(moe::kDgate, false, a, dy, w2, x->num_sms, st);
  a.gu = nullptr;
  if (e == cudaSuccess && dx) {
    a.N = H;
    a.K = 2 * F;
    a.out = dx;
    e = moe::launch_expert_gemm(moe::kDx, false, a, x->dgu, w13, x->num_sms, st);
  }
  if (e == cudaSuccess && dw13) {
    a.M = 2 * F;
    a.N = H;
    a.out = dw13;
    e = moe::launch_expert_gemm(moe::kDw, false, a, x->dgu, in, x->num_sms, st);
    if (e == cudaSuccess) {
      a.M = H;
      a.N = F;
      a.out = dw2;
      e = moe::launch_expert_gemm(moe::kDw, false, a, dy, hid, x->num_sms, st);
    }
  }
  return cuda_rc(e);
}

int moe_expert_set_wait_limit(moe_expert_t x, int64_t cycles) {
  if (!x || cycles < 0) return MOE_ERR_INVALID_ARG;
  x->wait_limit = cycles;
  return MOE_OK;
}

int moe_expert_read_status(moe_expert_t x, uint32_t* flags, void* stream) {
  if (!x || !flags) return MOE_ERR_INVALID_ARG;
  // all on the caller's stream: a later call on it finds the word cleared
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(flags, x->status, sizeof(uint32_t), cudaMemcpyDeviceToHost, st) !=
          cudaSuccess ||
      cudaMemsetAsync(x->status, 0, sizeof(uint32_t), st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // extern "C"
