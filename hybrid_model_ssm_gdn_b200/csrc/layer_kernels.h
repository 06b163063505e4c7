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
// How the launch is cut: blocks of `vectors` rows of q or of k, then blocks of `gates` rows.  A row a block while that leaves the
// SMs with few of them (64 rows of 16 heads: 6.1 us, with several rows a block 8.2), otherwise as many as give every 16 lanes
// kInputItems vectors.
constexpr int kInputItems = 4;  // heads' vectors that 16 lanes have on their way at a time
struct InputsCut {
  int vectors, gates;
  long long blocks;
};
inline InputsCut cut_inputs(int rows, int H, int Hk, bool few) {
  auto most = [&](int n) { return few || n < 1 ? 1 : n; };
  InputsCut c{most(16 * kInputItems / Hk), most(1024 / H), 0};
  c.blocks = 2 * (((long long)rows + c.vectors - 1) / c.vectors) + ((long long)rows + c.gates - 1) / c.gates;
  return c;
}
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
