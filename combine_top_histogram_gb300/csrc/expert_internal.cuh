// expert_internal.cuh -- shared declarations of the expert operators: kernel
// argument blocks, the host-side handle and launcher prototypes.
// Not installed; the public interface is include/moe_ep.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ep.h"

namespace moe {

// What a product over the segments computes and writes.
enum ExpertOp : int {
  kGated = 0,  // h = silu(x Wg^T) * (x Wu^T), gate and up columns in one tile
  kDown = 1,   // y = h W2^T
  kDgate = 2,  // dh = dy W2, then d(gate), d(up) from dh and the kept pre-activations
  kDx = 3,     // dx = [d(gate), d(up)] W13
  kDw = 4,     // W gradient: a^T b over the rows of a segment
};

struct ExpertArgs {
  const int32_t* offset;   // [E+1] first row of each segment
  int E;
  long long rows_max;      // rows every row buffer holds
  int M;                   // kDw: rows of the gradient; otherwise unused
  int N;                   // output columns (kGated, kDgate: F)
  int K;                   // reduction length (kDw: unused, the segment's rows)
  int nt;                  // tiles along N
  int F;                   // kGated, kDgate: up columns start F after gate columns
  int a_box;               // rows of one row-operand copy
  const float* sa;         // FP8: scales of the row operand [rows, K/128]
  const float* sb;         // FP8: scales of the weights
  void* out;
  float* out_scale;        // kGated, FP8: scales of h [rows, F/128]
  uint16_t* gu_out;        // kGated, bf16: kept pre-activations [rows, 2F], or null
  const uint16_t* gu;      // kDgate: kept pre-activations
  uint32_t* status;
  long long wait_limit;    // clock cycles a device wait may last
};

// One product over the segments: `a` rows [rows_max, K] (kDw: [rows_max, M]),
// `b` weights (kDw: rows [rows_max, N]).
cudaError_t launch_expert_gemm(ExpertOp op, bool fp8, const ExpertArgs& args, const void* a,
                               const void* b, int num_sms, cudaStream_t st);
// kGated or kDown for a few rows (expert_rows.cu).
cudaError_t launch_expert_rows(ExpertOp op, bool fp8, const ExpertArgs& args, const void* a,
                               const void* b, int num_sms, cudaStream_t st);
// Opts the kernels in to their shared memory and checks their register split.
cudaError_t expert_gemm_prepare();

}  // namespace moe

// Host-side handle of an expert block: configuration plus pointers into the
// caller's workspace.
struct moe_expert {
  moe_expert_config_t cfg;
  int device;
  int num_sms;
  uint32_t* status;
  uint16_t* dgu;           // [rows_max, 2F] (training only)
  long long wait_limit;
};
