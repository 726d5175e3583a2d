// Internal declarations of the linear attention calls and of the head norms:
// launch parameter blocks and the launchers that kda_linear_api.cu calls after
// validating the public arguments.
#pragma once

#include "kda_ssm.cuh"

namespace kda {

struct LinearParams {
  SegParams seg;
  const void *q, *k, *v;
  void *o;
  int qs, ks, vs, os;  // row strides in bytes
  const float *g;
  int gs;     // row stride in bytes, 0: one row
  int H, rep;  // heads, heads that share a q and k
  int DK, DV;
  float scale;
  float *pool;
  int vec;  // q, k, v rows start on 16 bytes
};

struct QkParams {
  const void *x[2];  // queries, keys
  void *y[2];
  const void *w[2];
  int xs[2], ys[2];  // row strides in bytes
  int heads[2];
  const float *table;
  const int32_t *pos;
  unsigned int *err;
  int N, d, rot, max_pos, interleaved, norm;
  float eps, q_scale;
  int per_token, tokens;  // groups of lanes on a token, tokens of a block
};

struct GateParams {
  const void *x, *gate, *w;
  void *y;
  int xs, gs, ys;  // row strides in bytes
  int N, H, d, silu;
  float eps;
};

cudaError_t launch_linear_walk(const LinearParams &p, kda_dtype dt, bool step, cudaStream_t s);
cudaError_t launch_qk_norm(const QkParams &p, kda_dtype dt, cudaStream_t s);
cudaError_t launch_gated_norm(const GateParams &p, kda_dtype x_dt, kda_dtype dt, cudaStream_t s);

}  // namespace kda
