// expert_internal.cuh -- shared declarations of the expert operators: kernel
// argument blocks, the host-side handle and launcher prototypes.
// Not installed; the public interface is include/moe_ep.h.
#pragma once

#include <cuda.h>
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
  kGatedCodes = 5,  // kGated and kDown of int8 codes widened to fp16, with their scales in the
  kDownCodes = 6,   // epilogue; h is fp32
};

// Types of the operands, by the C ABI's numbers.
enum ExpertType : int { kBf16 = MOE_BF16, kE4m3 = MOE_FP8_E4M3, kInt8 = MOE_INT8 };

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
  const float* sa;         // scales of the row operand: FP8 [rows, K/128], INT8 [rows]
  const float* sb;         // scales of the weights: FP8 per 128 x 128, INT8 per channel
  void* out;               // INT8: h in fp32 [rows, F]
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
cudaError_t launch_expert_rows(ExpertOp op, ExpertType type, const ExpertArgs& args, const void* a,
                               const void* b, int num_sms, cudaStream_t st);
// INT8: codes as fp16, of the segments' rows [rows, K], and of the weights [E, weight_rows, K] of
// the experts that have rows (expert_codes.cu).
cudaError_t launch_widen_rows(const ExpertArgs& args, const void* a, uint16_t* x16, int num_sms,
                              cudaStream_t st);
cudaError_t launch_widen_weights(const ExpertArgs& args, long long weight_rows, const void* b,
                                 uint16_t* w16, int num_sms, cudaStream_t st);
// INT8: codes [rows, F] and scales [rows] of the segments' rows of h (expert_codes.cu).
cudaError_t launch_expert_quantise(const ExpertArgs& args, const float* h, int8_t* codes,
                                   float* scale, int num_sms, cudaStream_t st);
// INT8: tokens of a tile and CTAs that share one, of kGated (p.N = F) or kDown.
struct Int8Plan {
  int tokens, split;
};
Int8Plan expert_int8_plan(ExpertOp op, const ExpertArgs& p, int num_sms);
// INT8: kGated (to fp32 h) or kDown on the tensor cores (expert_int8.cu).
cudaError_t launch_expert_int8(ExpertOp op, const ExpertArgs& args, const void* a, const void* b,
                               int num_sms, cudaStream_t st);
// Opt the kernels that a type's handles launch (the first: with those of backward, or
// without) in to their shared memory and check their register split.
cudaError_t expert_gemm_prepare(ExpertType type, bool train);
cudaError_t expert_int8_prepare();

// TMA map of a row-major tensor [planes][rows][cols] of 16-bit values, or of bytes; copies of
// box_rows rows x 128 (or 64) bytes, swizzled over as many, zeros outside. planes = 0: two-dimensional.
cudaError_t make_map(CUtensorMap* m, const void* base, bool bytes, long long cols, long long rows,
                     long long planes, int box_rows, int row_bytes = 128);

}  // namespace moe

// Host-side handle of an expert block: configuration plus pointers into the
// caller's workspace.
struct moe_expert {
  moe_expert_config_t cfg;
  int device;
  int num_sms;
  uint32_t* status;
  uint16_t* dgu;           // [rows_max, 2F] (training only)
  float* h32;              // [rows_max, F] (INT8 only)
  uint16_t *x16, *w16;     // fp16 codes of rows and weights (INT8 with many rows only)
  long long wait_limit;
};
