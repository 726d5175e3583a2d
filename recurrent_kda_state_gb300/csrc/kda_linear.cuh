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
  int o_vec;  // rows of o do
  // Prompts that are split: tokens of a chunk (their log2) and chunks of a part
  // (0: segments are whole), parts that the grid and the workspace hold, each part's decay and
  // its state, first what it adds and then the one before it.
  int chunk_log2, part_chunks, max_parts;
  int max_cut;         // the most parts that are not their segment's last
  float2 *part_decay;  // [max_parts][H]
  float *part_state;   // [max_parts][H][d_v * d_k]
  int spin_limit;      // polls of a bounded wait before it gives up
};

// e^g = hi + lo.  Near 0 from e^g - 1, whose error is relative to itself: a
// state lives through thousands of tokens when g is small, and the 2^-25 by
// which one fp32 e^g is off is the same every time.
__device__ __forceinline__ float2 decay_pair(float g) {
  if (fabsf(g) < 0.5f) {
    const float b = expm1f(g), hi = 1.0f + b;
    return make_float2(hi, b - (hi - 1.0f));
  }
  return make_float2(expf(g), 0.0f);
}
__device__ __forceinline__ float decayed(float s, float2 a, float add) {
  return fmaf(s, a.x, fmaf(s, a.y, add));
}

// Log decays are summed in fixed point, in units of 2^-44 log 2: exact, and
// without fp64, which this GPU has little of.  A token's is held within
// e^{+-210}, beyond fp32 in both directions, so that 64 of them fit.
constexpr float kFixed = 17592186044416.0f, kUnit = 1.0f / kFixed;
__device__ __forceinline__ long long fixed_log2(float g) {
  g = fminf(fmaxf(g, -210.0f), 210.0f);
  const float hi = g * kLog2e, lo = fmaf(g, kLog2e, -hi) + g * 1.92596299e-8f;  // log2(e) - kLog2e
  return __float2ll_rn(hi * kFixed) + __float2ll_rn(lo * kFixed);
}
__device__ __forceinline__ float unfixed(long long x) { return __ll2float_rn(x) * kUnit; }
constexpr long long kMostFixed = 1LL << 60;  // of a part's sum, which is held within it

// Parts of segment i, 0 for one without tokens or with a bad table entry.  What a cut
// saves has to pay for going over its first part twice: a segment of up to 3/2 of a
// part stays whole (lengths 3000, 500, 300 and 296, 64 heads of 128 x 64, parts of 41
// chunks, the state of Q S as one bf16: 209 us when it was cut, 168 so).
__device__ __forceinline__ int segment_parts(const LinearParams &p, int i) {
  const int b = p.seg.cu[i], e = p.seg.cu[i + 1], p0 = p.seg.start_pos ? p.seg.start_pos[i] : 0;
  if (b < 0 || e <= b || e > p.seg.N || p0 < 0) return 0;
  const int size = 1 << p.chunk_log2;
  const int chunks = (int)(((p0 & (size - 1)) + (long long)(e - b) + size - 1) >> p.chunk_log2);
  return 2LL * chunks <= 3LL * p.part_chunks ? 1 : (chunks + p.part_chunks - 1) / p.part_chunks;
}
// Table entries of segments that no part stands for, reported by one block: as a
// block of its own would, where segments are whole.
__device__ __forceinline__ void report_segments(const LinearParams &p) {
  for (int i = threadIdx.x; i < p.seg.B; i += blockDim.x) {
    SegLoc s;
    if (locate_segment(p.seg, i, &s) && s.len > 0 && p.seg.start_pos && p.seg.start_pos[i] < 0)
      set_error(p.seg.err, KDA_DERR_SEGMENT);
  }
}
struct PartLoc {
  int seg, part, parts;  // seg < 0: no such part
  int index;             // among the parts of all segments
};
// The segment and place of part `target` of all segments' parts in their order, or
// of those that are not their segment's last; for a whole warp.
template <bool LAST = true>
__device__ __forceinline__ PartLoc find_part(const LinearParams &p, int target) {
  const int lane = threadIdx.x & 31;
  int before = 0, index = 0;  // counted parts of the segments before, and all their parts
  for (int base = 0; base < p.seg.B; base += 32) {
    const int parts = base + lane < p.seg.B ? segment_parts(p, base + lane) : 0;
    const int n = LAST ? parts : max(parts - 1, 0);
    int upto = n, all = parts;
#pragma unroll
    for (int w = 1; w < 32; w *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, upto, w), r = __shfl_up_sync(0xffffffffu, all, w);
      if (lane >= w) upto += o, all += r;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > target);
    if (past) {
      const int l = __ffs(past) - 1, its = __shfl_sync(0xffffffffu, parts, l);
      const int part = target - (before + __shfl_sync(0xffffffffu, upto - n, l));
      return {base + l, part, its, index + __shfl_sync(0xffffffffu, all, l) - its + part};
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
    index += __shfl_sync(0xffffffffu, all, 31);
  }
  return {-1, 0, 0, 0};
}

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
  float share;  // of the sum of squares: 1 / d for its mean, else 1
  int per_token, tokens;  // groups of lanes on a token, tokens of a block
};

struct GateParams {
  const void *x, *gate, *w;
  void *y;
  int xs, gs, ys;  // row strides in bytes
  int N, H, d, silu;
  float eps;
  float share;  // 1 / d
};

// The states before the parts of every cut segment, in the place of what the parts
// add: a thread follows four states of one head, F::plain of them in the pool, for
// every gridDim.y-th of the cut segments.  Bound by the latency of kAhead parts' loads
// in turn; four of them and 64 registers, so that an SM holds four blocks and the 512 of
// one cut segment run at once, three rows of them in two to three turns (eight and 102
// registers: four prompts of 4096 tokens, 64 heads of 128 x 64, 136 us in all, 128 so; one
// of 8192, 32 heads of 128 x 128, 127 and 125, with the state of Q S as one bf16).
template <typename F>
__global__ void __launch_bounds__(256, 4) linear_join_kernel(const LinearParams p) {
  constexpr int kAhead = 4;
  begin_after_stream();
  const int state4 = p.DK * p.DV / 4, idx = blockIdx.x * 256 + threadIdx.x, h = idx / state4, e = idx % state4;
  const int lane = threadIdx.x & 31;
  const long long step = (long long)p.H * state4;
  int index = 0, turn = 0;  // parts of the segments before, cut segments so far
  for (int base = 0; base < p.seg.B; base += 32) {
    const int n = base + lane < p.seg.B ? segment_parts(p, base + lane) : 0;
    int upto = n;
#pragma unroll
    for (int w = 1; w < 32; w *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, upto, w);
      if (lane >= w) upto += o;
    }
    for (unsigned cut = __ballot_sync(0xffffffffu, n > 1); cut; cut &= cut - 1) {
      const int l = __ffs(cut) - 1, parts = __shfl_sync(0xffffffffu, n, l);
      const int first = index + __shfl_sync(0xffffffffu, upto, l) - parts;
      if (turn++ % gridDim.y != blockIdx.y) continue;
      SegLoc s;
      if (first + parts > p.max_parts || h >= p.H || !locate_segment(p.seg, base + l, &s)) continue;
      float4 S =
          *reinterpret_cast<const float4 *>(p.pool + ((long long)s.slot * p.H + h) * p.DK * p.DV + F::plain(e));
      float4 *at = reinterpret_cast<float4 *>(p.part_state) + ((long long)first * p.H + h) * state4 + e;
      const float2 *decay = p.part_decay + (long long)first * p.H + h;
      for (int q = 0; q < parts; q += kAhead) {
        float4 add[kAhead];
        float2 a[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int r = min(q + u, parts - 2);
          add[u] = at[r * step];
          a[u] = decay[(long long)r * p.H];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (q + u < parts) at[(q + u) * step] = S;
          S = make_float4(decayed(S.x, a[u], add[u].x), decayed(S.y, a[u], add[u].y), decayed(S.z, a[u], add[u].z),
                          decayed(S.w, a[u], add[u].w));
        }
      }
      __syncwarp();
    }
    index += __shfl_sync(0xffffffffu, upto, 31);
  }
}
template <typename F>
cudaError_t launch_linear_join(const LinearParams &p, cudaStream_t s) {
  const long long blocks = ((long long)p.H * p.DK * p.DV / 4 + 255) / 256;
  // more rows than are resident at once: several cut segments' loads beside one another
  const long long rows = 152 * 8 / blocks + 1;
  return launch_after(linear_join_kernel<F>, dim3((unsigned)blocks, p.seg.B < rows ? p.seg.B : (int)rows), dim3(256),
                      0, s, p);
}

// Where the chunks of a batch run, for the choice of its parts.
struct LinearCut {
  int blocks, of_part;  // that the GPU holds; that a part takes, with all heads
  int chunk, least;     // tokens of a chunk, chunks of a part at least
  int room() const { return of_part < blocks ? blocks / of_part : 1; }
};
LinearCut linear_cut(int dtype, int H, int d_k, int d_v);

cudaError_t launch_linear_walk(const LinearParams &p, kda_dtype dt, bool step, cudaStream_t s);
// Prompts in bf16 with d_k and d_v of 64 or 128, on the tensor cores.
cudaError_t launch_linear_tc(const LinearParams &p, cudaStream_t s);
inline bool linear_uses_tc(int dtype, int d_k, int d_v) {
  return dtype == KDA_BF16 && d_k >= 64 && d_v >= 64;
}
// Chunks of a part of a batch (0: it is not split) and the most parts it can
// have; the most of any batch of at most N tokens and B segments (0: none is split).
int linear_part_chunks(int N, int B, const LinearCut &c);
int linear_max_parts(int N, int B, int part, const LinearCut &c);
int linear_max_cut(int N, int B, int part, const LinearCut &c);
size_t linear_workspace_parts(int N, int B, const LinearCut &c);
// Bytes of the parts' decays at the start of the workspace.
inline size_t linear_decay_bytes(size_t parts, int H) {
  return (parts * H * sizeof(float2) + 255) & ~(size_t)255;
}
inline size_t linear_workspace_bytes(size_t parts, int H, int d_k, int d_v) {
  return parts ? linear_decay_bytes(parts, H) + parts * H * d_k * d_v * sizeof(float) : 0;
}
cudaError_t launch_qk_norm(const QkParams &p, kda_dtype dt, cudaStream_t s);
cudaError_t launch_gated_norm(const GateParams &p, kda_dtype x_dt, kda_dtype dt, cudaStream_t s);

}  // namespace kda
