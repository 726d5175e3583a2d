// Short causal depthwise convolution over packed segments, with the last
// W - 1 inputs of each sequence kept in its slot:
//     y[t] = act(bias + sum_j w[j] u[t + j]),  u = [slot's W - 1 rows; x rows]
//
// Memory bound: x is read and y written once, 2 W + 4 flops a value.  A
// thread owns one 16-byte vector of channels and walks down a run of tokens
// with the W - 1 previous rows in registers, eight rows of loads in flight.
// A prompt's segments are cut into tiles of p.tile tokens, each with its own
// W - 1 rows before it.  Tile 0 alone reads the slot and alone writes it (it
// fetches the segment's last rows itself), so no other block can see a state
// that is already replaced.
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kRows = 8;  // rows of loads in flight

// Tokens [t0, t1) of the segment (local indices; t0 = 0 or t0 >= W - 1).
template <typename T, int V, int W>
__device__ __forceinline__ void conv_run(const ConvParams &p, const SegLoc &s, int i, int c,
                                         int t0, int t1) {
  const long long D = p.D;
  const T *x = static_cast<const T *>(p.x) + (long long)s.begin * p.xs + c;
  T *y = static_cast<T *>(p.y) + (long long)s.begin * p.ys + c;
  T *state = static_cast<T *>(p.pool) + (long long)s.slot * (W - 1) * D + c;
  const T *wp = static_cast<const T *>(p.weight) + (long long)c * W;
  const T *bp = static_cast<const T *>(p.bias);

  float w[W][V], bias[V], win[W - 1][V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    bias[e] = bp ? in_scalar<T>(bp + c + e) : 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = in_scalar<T>(wp + e * W + j);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    if (t0 == 0) load_elems<T, V>(state + j * D, win[j]);
    else load_elems<T, V>(x + (long long)(t0 - (W - 1) + j) * p.xs, win[j]);
  }
  if (t0 == 0 && s.keep > 0) {  // the state after `keep` tokens: u[keep .. keep + W - 2]
    float row[W - 1][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int at = s.keep + j - (W - 1);
      if (at >= 0) {
        load_elems<T, V>(x + (long long)at * p.xs, row[j]);
      } else {
#pragma unroll
        for (int q = 0; q < W - 1; ++q)
          if (q == s.keep + j) {
#pragma unroll
            for (int e = 0; e < V; ++e) row[j][e] = win[q][e];
          }
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_elems<T, V>(state + j * D, row[j]);
  }

  const bool ckpt = p.seg.ckpt_slots != nullptr;
  const long long p0 = ckpt && p.seg.start_pos ? p.seg.start_pos[i] : 0;
  const long long every = p.seg.ckpt_every;
  long long next = ckpt ? ((p0 + t0) / every + 1) * every - p0 : 0;  // tokens to the next checkpoint
  for (int t = t0; t < t1; t += kRows) {
    float in[kRows][V];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (t + r < t1) load_elems<T, V>(x + (long long)(t + r) * p.xs, in[r]);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (t + r >= t1) break;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float acc = bias[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) acc = fmaf(w[j][e], win[j][e], acc);
        acc = fmaf(w[W - 1][e], in[r][e], acc);
        o[e] = p.silu ? silu_f(acc) : acc;
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
        win[W - 2][e] = in[r][e];
      }
      store_elems<T, V>(y + (long long)(t + r) * p.ys, o);
      if (ckpt && t + r + 1 == next) {
        next += every;
        const int slot = checkpoint_slot(p.seg, i, p0, t + r + 1);
        if (slot >= 0) {
          T *to = static_cast<T *>(p.pool) + (long long)slot * (W - 1) * D + c;
#pragma unroll
          for (int j = 0; j < W - 1; ++j) store_elems<T, V>(to + j * D, win[j]);
        }
      }
    }
  }
}

// One row of threads (threadIdx.y) per tile; blockIdx.x: channels.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvParams p) {
  const int i = blockIdx.y * blockDim.y + threadIdx.y;
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (i >= p.seg.B || c >= p.D) return;
  SegLoc s;
  if (!locate_segment(p.seg, i, &s) || s.len == 0) return;
  conv_run<T, V, W>(p, s, i, c, 0, s.len);
}

// Tile g of the batch belongs to the last segment i with
// cu[i] / tile + i <= g: that leaves every segment at least the tiles it
// needs.  Found by a 32-way search of one warp (B <= 65535: four rounds).
__device__ __forceinline__ int find_segment(const SegParams &p, int g, int tile) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned m = __ballot_sync(~0u, i < hi && p.cu[i] / tile + i <= g);
    lo += m ? (31 - __clz(m)) * step : 0;
    hi = min(lo + step, hi);
  }
  return lo;
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(128) conv_prefill_kernel(const ConvParams p) {
  const int g = blockIdx.y * blockDim.y + threadIdx.y;
  const int i = find_segment(p.seg, g, p.tile);
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (c >= p.D) return;
  SegLoc s;
  if (!locate_segment(p.seg, i, &s)) return;
  const long long t0 = (long long)(g - (s.begin / p.tile + i)) * p.tile;
  if (t0 < 0 || t0 >= s.len) return;
  conv_run<T, V, W>(p, s, i, c, (int)t0, (int)min((long long)s.len, t0 + p.tile));
}

template <typename T, int V, int W>
cudaError_t launch_w(const ConvParams &p, bool step, cudaStream_t st) {
  const int nvec = (p.D + V - 1) / V;
  const int bx = nvec >= 128 ? 128 : (nvec + 31) / 32 * 32;
  const dim3 block(bx, 128 / bx);
  const int gx = (nvec + bx - 1) / bx;
  if (step) {
    const dim3 grid(gx, (p.seg.B + block.y - 1) / block.y);
    conv_step_kernel<T, V, W><<<grid, block, 0, st>>>(p);
    return cudaGetLastError();
  }
  // Tiles as long as they leave every SM its four blocks of 128 threads.
  ConvParams q = p;
  const long long want = 152LL * 4 * 128;
  long long tile = (long long)p.seg.N * nvec / want / kRows * kRows;
  q.tile = (int)(tile < kRows ? kRows : tile > 64 ? 64 : tile);
  long long tiles = (long long)p.seg.N / q.tile + p.seg.B;
  while ((tiles + block.y - 1) / block.y > 65535) {  // the grid's y limit
    q.tile *= 2;
    tiles = (long long)p.seg.N / q.tile + p.seg.B;
  }
  const dim3 grid(gx, (unsigned)((tiles + block.y - 1) / block.y));
  conv_prefill_kernel<T, V, W><<<grid, block, 0, st>>>(q);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_v(const ConvParams &p, bool step, cudaStream_t st) {
  switch (p.W) {
    case 2: return launch_w<T, V, 2>(p, step, st);
    case 3: return launch_w<T, V, 3>(p, step, st);
    default: return launch_w<T, V, 4>(p, step, st);
  }
}

template <typename T>
cudaError_t launch_t(const ConvParams &p, bool step, cudaStream_t st) {
  constexpr int V = InVec<T>::kElems;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y) |
                         (uintptr_t)(p.xs * (long long)sizeof(T)) |
                         (uintptr_t)(p.ys * (long long)sizeof(T));
  const bool vec = (bits & 15) == 0 && p.D % V == 0;
  return vec ? launch_v<T, V>(p, step, st) : launch_v<T, 1>(p, step, st);
}

}  // namespace

cudaError_t launch_conv(const ConvParams &p, kda_dtype dt, bool step, cudaStream_t s) {
  return dt == KDA_F32 ? launch_t<float>(p, step, s) : launch_t<__nv_bfloat16>(p, step, s);
}

}  // namespace kda
