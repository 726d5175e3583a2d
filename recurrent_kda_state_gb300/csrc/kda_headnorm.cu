// Norms of each head's channels: of queries and keys, with the position
// rotation and a scale, and of a layer's outputs, with their gate.
//
// Memory bound: every row is read and written once.  A head's row is held by a
// group of lanes, each with vectors of 16 bytes where rows and channels allow
// it, else with single elements; sums of squares go through shuffles, in fp32.
// Nothing is written before the whole group has read its row, lane by lane at
// the same places, so outputs may be the inputs.
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// V elements in fp32 (V = 1, or as many as 16 bytes of T2 hold, aligned).
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = in_scalar<T>(p);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += InVec<T>::kElems) InVec<T>::load(p + i, v + i);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = out_scalar<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    static_assert(V == 1 || V == 8, "16 bytes");
    uint4 r;
    uint32_t *w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = r;
  }
}

__device__ __forceinline__ float group_total(float v, int lanes) {
  for (int w = lanes / 2; w > 0; w /= 2) v += __shfl_xor_sync(0xffffffffu, v, w);
  return v;
}

// A lane's unit is two runs of V channels, A and B.  Channels that turn with
// one another are in one unit: as pairs (A[i], B[i]) in halves, as neighbours
// inside a run (for V = 1 a unit is the pair itself).
template <typename T, int V, int U>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const QkParams p, int lanes) {
  begin_after_stream();
  const int group = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int tok = blockIdx.x * p.tokens + group / p.per_token;
  const int total = p.heads[0] + p.heads[1];
  const bool here = group < p.tokens * p.per_token && tok < p.N;
  int pos = 0;
  bool turn = p.rot > 0 && here;
  if (turn) {
    pos = p.pos[tok];
    if (pos < 0 || pos >= p.max_pos) {
      if (l == 0) set_error(p.err, KDA_DERR_POSITION);
      pos = -1;
    }
  }
  const float *cs = p.table + (long long)pos * p.rot;
  const int half = p.rot / 2, units = p.d / (2 * V);
  // every lane of a warp takes part in the shuffles, with or without a head
  for (int first = 0; first < total; first += p.per_token) {
    const int head = first + group % p.per_token;
    const bool live = here && head < total && pos >= 0;
    const int which = head < p.heads[0] ? 0 : 1;
    const int hh = which ? head - p.heads[0] : head;
    float a[U][V], b[U][V], sum = 0.0f;
    int ca[U], cb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = l + u * lanes;
      if (p.interleaved || j * V >= half) {
        ca[u] = 2 * j * V;
        cb[u] = ca[u] + V;
      } else {
        ca[u] = j * V;
        cb[u] = half + j * V;
      }
      if (live && j < units) {
        const T *x = row_at(static_cast<const T *>(p.x[which]), tok, p.xs[which]) + hh * p.d;
        load_vec<T, V>(x + ca[u], a[u]);
        load_vec<T, V>(x + cb[u], b[u]);
#pragma unroll
        for (int e = 0; e < V; ++e) sum = fmaf(a[u][e], a[u][e], fmaf(b[u][e], b[u][e], sum));
      }
    }
    sum = group_total(sum, lanes);
    if (!live) continue;
    const float r = p.norm == KDA_NORM_NONE ? 1.0f
                    : __frsqrt_rn((p.norm == KDA_NORM_RMS ? sum / (float)p.d : sum) + p.eps);
    const float scale = which ? 1.0f : p.q_scale;
    T *y = row_at(static_cast<T *>(p.y[which]), tok, p.ys[which]) + hh * p.d;
    const T *w = static_cast<const T *>(p.w[which]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (l + u * lanes >= units) continue;
      float wa[V], wb[V];
      if (w) {
        load_vec<T, V>(w + ca[u], wa);
        load_vec<T, V>(w + cb[u], wb);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        a[u][e] *= r;
        b[u][e] *= r;
        if (w) {
          a[u][e] *= wa[e];
          b[u][e] *= wb[e];
        }
      }
      if (turn && ca[u] < p.rot) {
        if (!p.interleaved || V == 1) {
          const int i = p.interleaved ? ca[u] / 2 : ca[u];
          float c[V], s[V];
          load_vec<float, V>(cs + i, c);
          load_vec<float, V>(cs + half + i, s);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float t = a[u][e];
            a[u][e] = t * c[e] - b[u][e] * s[e];
            b[u][e] = b[u][e] * c[e] + t * s[e];
          }
        } else {
          auto inside = [&](float (&x)[V], int at) {
            if (at >= p.rot) return;
#pragma unroll
            for (int e = 0; e + 1 < V; e += 2) {
              const float c = cs[at / 2 + e / 2], s = cs[half + at / 2 + e / 2], t = x[e];
              x[e] = t * c - x[e + 1] * s;
              x[e + 1] = x[e + 1] * c + t * s;
            }
          };
          inside(a[u], ca[u]);
          inside(b[u], cb[u]);
        }
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        a[u][e] *= scale;
        b[u][e] *= scale;
      }
      store_vec<T, V>(y + ca[u], a[u]);
      store_vec<T, V>(y + cb[u], b[u]);
    }
  }
}

template <typename TX, typename T, int V, int U>
__global__ void __launch_bounds__(kThreads) gated_norm_kernel(const GateParams p, int lanes) {
  begin_after_stream();
  const int groups = kThreads / lanes, l = threadIdx.x % lanes;
  const long long item = (long long)blockIdx.x * groups + threadIdx.x / lanes;
  const bool live = item < (long long)p.N * p.H;
  const int tok = (int)(item / p.H), head = (int)(item % p.H), units = p.d / V;
  float x[U][V], g[U][V], sum = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (l + u * lanes) * V;
    if (live && l + u * lanes < units) {
      load_vec<TX, V>(row_at(static_cast<const TX *>(p.x), tok, p.xs) + head * p.d + c, x[u]);
      if (p.gate) load_vec<T, V>(row_at(static_cast<const T *>(p.gate), tok, p.gs) + head * p.d + c, g[u]);
#pragma unroll
      for (int e = 0; e < V; ++e) sum = fmaf(x[u][e], x[u][e], sum);
    }
  }
  sum = group_total(sum, lanes);
  if (!live) return;
  const float r = __frsqrt_rn(sum / (float)p.d + p.eps);
  const T *w = static_cast<const T *>(p.w);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (l + u * lanes) * V;
    if (l + u * lanes >= units) continue;
    float wv[V];
    if (w) load_vec<T, V>(w + c, wv);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float y = x[u][e] * r;
      if (w) y *= wv[e];
      if (p.gate) {
        const float act = 1.0f / (1.0f + expf(-g[u][e]));
        y *= p.silu ? g[u][e] * act : act;
      }
      x[u][e] = y;
    }
    store_vec<T, V>(row_at(static_cast<T *>(p.y), tok, p.ys) + head * p.d + c, x[u]);
  }
}

int pow2_up(int n) {
  int r = 1;
  while (r < n) r *= 2;
  return r;
}

// Whether V-element vectors serve all rows of a view.
bool fits(const void *p, long long stride_bytes) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

template <typename T>
cudaError_t qk_norm(QkParams p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  // runs of V channels: no run is cut by the rotation's borders, rows start on 16 bytes
  bool vec = p.d % (2 * V) == 0 && (p.interleaved ? p.rot % V == 0 : p.rot % (2 * V) == 0);
  for (int i = 0; i < 2; ++i)
    if (p.heads[i]) vec = vec && fits(p.x[i], p.xs[i]) && fits(p.y[i], p.ys[i]);
  const int units = p.d / (vec ? 2 * V : 2), lanes = pow2_up(units < 32 ? units : 32);
  const int total = p.heads[0] + p.heads[1], most = kThreads / lanes;
  const int passes = (total + most - 1) / most;
  p.per_token = (total + passes - 1) / passes;
  p.tokens = most / p.per_token;
  const int threads = (p.tokens * p.per_token * lanes + 31) / 32 * 32;
  const dim3 grid((p.N + p.tokens - 1) / p.tokens);
  if (vec) return launch_after(qk_norm_kernel<T, V, 1>, grid, dim3(threads), 0, s, p, lanes);
  return launch_after(qk_norm_kernel<T, 1, 4>, grid, dim3(threads), 0, s, p, lanes);
}

template <typename TX, typename T>
cudaError_t gated_norm(const GateParams &p, cudaStream_t s) {
  constexpr int V = 16 / (sizeof(T) < sizeof(TX) ? sizeof(T) : sizeof(TX));
  const bool vec = p.d % V == 0 && fits(p.x, p.xs) && fits(p.y, p.ys) && (!p.gate || fits(p.gate, p.gs));
  const int units = p.d / (vec ? V : 1), lanes = pow2_up(units < 32 ? units : 32);
  const int groups = kThreads / lanes;
  const long long blocks = ((long long)p.N * p.H + groups - 1) / groups;
  if (vec) return launch_after(gated_norm_kernel<TX, T, V, 2>, dim3(blocks), dim3(kThreads), 0, s, p, lanes);
  return launch_after(gated_norm_kernel<TX, T, 1, 8>, dim3(blocks), dim3(kThreads), 0, s, p, lanes);
}

}  // namespace

cudaError_t launch_qk_norm(const QkParams &p, kda_dtype dt, cudaStream_t s) {
  return dt == KDA_F32 ? qk_norm<float>(p, s) : qk_norm<__nv_bfloat16>(p, s);
}

cudaError_t launch_gated_norm(const GateParams &p, kda_dtype x_dt, kda_dtype dt, cudaStream_t s) {
  if (x_dt == KDA_F32)
    return dt == KDA_F32 ? gated_norm<float, float>(p, s) : gated_norm<float, __nv_bfloat16>(p, s);
  return dt == KDA_F32 ? gated_norm<__nv_bfloat16, float>(p, s)
                       : gated_norm<__nv_bfloat16, __nv_bfloat16>(p, s);
}

}  // namespace kda
