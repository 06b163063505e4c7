// layer_kernels.h -- launches of the kernels between a layer's projections: inputs of the gated delta rule, norms.
#pragma once

#include "kernels.h"

namespace rssm {

struct GdnInputsArgs {
  int rows, H, Hk, out_heads;       // heads of v; of q and k; of the outputs q and k (Hk or H)
  const void *q, *k, *a, *b;        // rows of [Hk][128] and [H]
  long long stride_q, stride_k, stride_a, stride_b;  // elements from one row to the next
  const float *A_log, *bias;        // [H]
  float eps;
  void *q_out, *k_out;              // [rows][out_heads][128]
  float *alpha, *beta;              // [rows][H]
  int vector_rows, gate_rows;       // rows of a block (the launch's to fill in)
};
cudaError_t launch_gdn_inputs(const GdnInputsArgs &a, int esz, int num_sms, cudaStream_t stream);

struct NormArgs {
  int rows, columns, group;         // group divides columns
  int x_dtype, gate_dtype, weight_dtype, out_dtype;
  int scale;                        // rssm_scale: of an 8-bit output
  int norm_first;                   // gated: the norm before the gate
  int weight_columns;               // columns, or group: one weight for all groups
  float eps, offset;
  const void *x, *gate, *weight;
  void *residual;                   // or null
  long long stride_x, stride_gate, stride_residual;
  void *out;                        // [rows][columns]
  float *scales;                    // [rows] or [rows][ceil(columns / 128)]
};
cudaError_t launch_norm(const NormArgs &a, bool gated, cudaStream_t stream);

}  // namespace rssm
