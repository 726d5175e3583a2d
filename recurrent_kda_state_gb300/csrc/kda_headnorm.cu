// Norms of each head's channels: of queries and keys, with the position
// rotation and a scale, and of a layer's outputs, with their gate.
//
// Memory bound: every row is read and written once.  A head's row is held by a
// group of lanes, each with vectors of 16 bytes where rows and channels allow
// it, else with single elements; sums of squares go through shuffles, in fp32.
// A lane writes where it has read before, so outputs may be the inputs.
//
// Blocks that fill the machine once walk down the rows with the next ones under
// way, and arithmetic is in packed pairs: with a block for every few rows these
// kernels were bound by issue slots (70 % busy) and starts, not by memory.  8192
// tokens of 64 heads of 128 in bf16, rotated: 78 us so, 56 with four heads a group
// and pairs, 45.4 walking, 90 % of the copy bandwidth.  Gated, 8192 x 32 heads of
// 128 from fp32 to bf16: 71, 54, 46, with pairs 42.6 (94 %).
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // of a group of lanes that walks down the tokens
constexpr int kSms = 152;

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
    __stcs(reinterpret_cast<uint4 *>(p), r);
  }
}

__device__ __forceinline__ float group_total(float v, int lanes) {
#pragma unroll
  for (int w = 16; w > 0; w /= 2) {
    const float o = __shfl_xor_sync(0xffffffffu, v, w);
    if (w < lanes) v += o;
  }
  return v;
}

// V elements as they are in memory.
template <typename T, int V>
struct Raw {
  static constexpr int kWords = V == 1 ? 1 : V * (int)sizeof(T) / 16;
  using Word = typename std::conditional<V == 1, T, uint4>::type;
  Word w[kWords];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const Word *>(p)[i];
  }
  // Rows pass through once: marked to leave L2 first.
  __device__ __forceinline__ void load_once(const T *p) {
    if constexpr (V == 1) load(p);
    else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const Word *>(p) + i);
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (V == 1) {
      return in_scalar<T>(&w[0]);
    } else {
      const uint4 q = w[e * (int)sizeof(T) / 16];
      const int word = e * (int)sizeof(T) / 4 % 4;
      const uint32_t u = word == 0 ? q.x : word == 1 ? q.y : word == 2 ? q.z : q.w;
      if constexpr (sizeof(T) == 4) return __uint_as_float(u);
      else return __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
    }
  }
  __device__ __forceinline__ f2 pair(int e) const { return pack2(get(2 * e), get(2 * e + 1)); }
};

enum Turn { kNoTurn, kHalves, kNeighbours };

// A lane's unit is two runs of V channels, A and B.  Channels that turn with
// one another are in one unit: as pairs (A[i], B[i]) in halves, as neighbours
// inside a run (for V = 1 a unit is the pair itself).
template <typename T, int V, Turn TURN>
struct Unit {
  int ca, cb;  // first channels
  bool mine;   // whether the head has this unit
  __device__ __forceinline__ Unit(const QkParams &p, int j) {
    const int half = p.rot / 2;
    const bool paired = TURN == kHalves && j * V < half;
    ca = paired ? j * V : 2 * j * V;
    cb = paired ? half + j * V : ca + V;
    mine = j < p.d / (2 * V);
  }
  // The table's row at `cs`: a value for each of A's channels, or for the
  // neighbours of A and then of B; what is not rotated turns by nothing.
  __device__ __forceinline__ void angles(const QkParams &p, const float *cs, float (&c)[V], float (&s)[V]) const {
    const int half = p.rot / 2;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      c[e] = 1.0f;
      s[e] = 0.0f;
    }
    if (TURN == kNoTurn || !mine || ca >= p.rot) return;
    if constexpr (TURN == kHalves || V == 1) {
      const int i = TURN == kNeighbours ? ca / 2 : ca;
      load_vec<float, V>(cs + i, c);
      load_vec<float, V>(cs + half + i, s);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (ca + 2 * e < p.rot) {  // B may lie behind the rotation
          c[e] = cs[ca / 2 + e];
          s[e] = cs[half + ca / 2 + e];
        }
    }
  }
};
template <typename T, int V>
__device__ __forceinline__ float squares(const Raw<T, V> &a, const Raw<T, V> &b) {
  if constexpr (V == 1) {
    return fmaf(a.get(0), a.get(0), b.get(0) * b.get(0));
  } else {
    f2 sum = mul2(a.pair(0), a.pair(0));
#pragma unroll
    for (int e = 1; e < V / 2; ++e) sum = fma2(a.pair(e), a.pair(e), sum);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) sum = fma2(b.pair(e), b.pair(e), sum);
    const float2 v = unpack2(sum);
    return v.x + v.y;
  }
}
// Weights of a unit's channels; 1 where there are none.
template <typename T, int V>
struct Weights {
  static constexpr int N = V == 1 ? 1 : V / 2;
  using P = typename std::conditional<V == 1, float, f2>::type;
  P a[N], b[N];
  __device__ __forceinline__ void load(const T *w, int ca, int cb) {
    Raw<T, V> ra, rb;
    if (w) {
      ra.load(w + ca);
      rb.load(w + cb);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if constexpr (V == 1) {
        a[e] = w ? ra.get(0) : 1.0f;
        b[e] = w ? rb.get(0) : 1.0f;
      } else {
        a[e] = w ? ra.pair(e) : both(1.0f);
        b[e] = w ? rb.pair(e) : both(1.0f);
      }
    }
  }
};
// x times r (the norm and the scale) and the weights, turned.
template <Turn TURN, typename T, int V>
__device__ __forceinline__ void finish(float r, const Raw<T, V> &xa, const Raw<T, V> &xb, const Weights<T, V> &w,
                                       const float (&c)[V], const float (&s)[V], T *ya, T *yb) {
  if constexpr (V == 1) {
    const float a = xa.get(0) * r * w.a[0], b = xb.get(0) * r * w.b[0];
    *ya = out_scalar<T>(TURN == kNoTurn ? a : a * c[0] - b * s[0]);
    *yb = out_scalar<T>(TURN == kNoTurn ? b : b * c[0] + a * s[0]);
  } else {
    float oa[V], ob[V];
    auto put = [](float (&o)[V], int e, f2 x) {
      const float2 v = unpack2(x);
      o[2 * e] = v.x;
      o[2 * e + 1] = v.y;
    };
    auto inside = [](f2 x, float ct, float st) {  // (x, z) c + (-z, x) s
      const float2 v = unpack2(x);
      return fma2(x, both(ct), mul2(pack2(v.y, v.x), pack2(-st, st)));
    };
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      const f2 a = mul2(mul2(xa.pair(e), both(r)), w.a[e]), b = mul2(mul2(xb.pair(e), both(r)), w.b[e]);
      if constexpr (TURN == kHalves) {
        const f2 ct = pack2(c[2 * e], c[2 * e + 1]), st = pack2(s[2 * e], s[2 * e + 1]);
        put(oa, e, fma2(a, ct, mul2(b, pack2(-s[2 * e], -s[2 * e + 1]))));
        put(ob, e, fma2(b, ct, mul2(a, st)));
      } else if constexpr (TURN == kNeighbours) {
        put(oa, e, inside(a, c[e], s[e]));
        put(ob, e, inside(b, c[V / 2 + e], s[V / 2 + e]));
      } else {
        put(oa, e, a);
        put(ob, e, b);
      }
    }
    store_vec<T, V>(ya, oa);
    store_vec<T, V>(yb, ob);
  }
}
// What the norm multiplies by.
__device__ __forceinline__ float norm_factor(const QkParams &p, float sum) {
  return p.norm == KDA_NORM_NONE ? 1.0f : rsqrtf(fmaf(sum, p.share, p.eps));
}
// The row of the table of a position, NULL (and the error bit) if it has none.
__device__ __forceinline__ const float *table_row(const QkParams &p, int pos, bool report) {
  if (pos >= 0 && pos < p.max_pos) return p.table + (long long)pos * p.rot;
  if (report) set_error(p.err, KDA_DERR_POSITION);
  return nullptr;
}

// 1 / (1 + e^-v).  log2(e) and its product with v are rounded before ex2: up to 0.62 |v| ulp.
__device__ __forceinline__ float sigmoid(float v) { return rcpf(1.0f + ex2f(-kLog2e * v)); }
__device__ __forceinline__ f2 sigmoid(f2 v) {
  const float2 d = unpack2(add2(exp2_2(mul2(v, both(-kLog2e))), both(1.0f)));
  return pack2(rcpf(d.x), rcpf(d.y));
}

// Few tokens, or rows that take single elements: a group of lanes for each head
// of a block's tokens.
template <typename T, int V, int U, Turn TURN>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(QkParams p, int lanes) {
  begin_after_stream();
  const int group = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int tok = blockIdx.x * p.tokens + group / p.per_token;
  const int total = p.heads[0] + p.heads[1];
  const bool here = group < p.tokens * p.per_token && tok < p.N;
  const int pos = TURN != kNoTurn && here ? p.pos[tok] : 0;
  // every lane of a warp takes part in the shuffles, with or without a head
  for (int first = 0; first < total; first += p.per_token) {
    const int head = first + group % p.per_token, which = head < p.heads[0] ? 0 : 1;
    const int at = (which ? head - p.heads[0] : head) * p.d;
    Raw<T, V> a[U], b[U];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Unit<T, V, TURN> unit(p, l + u * lanes);
      if (here && head < total && unit.mine) {
        const T *x = row_at(static_cast<const T *>(p.x[which]), tok, p.xs[which]) + at;
        a[u].load(x + unit.ca);
        b[u].load(x + unit.cb);
        sum += squares(a[u], b[u]);
      }
    }
    const float *cs = TURN != kNoTurn && here ? table_row(p, pos, first == 0 && l == 0) : nullptr;
    sum = group_total(sum, lanes);
    if (!here || head >= total || (TURN != kNoTurn && !cs)) continue;
    const float r = norm_factor(p, sum) * (which ? 1.0f : p.q_scale);
    T *y = row_at(static_cast<T *>(p.y[which]), tok, p.ys[which]) + at;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Unit<T, V, TURN> unit(p, l + u * lanes);
      if (!unit.mine) continue;
      float c[V], s[V];
      unit.angles(p, cs, c, s);
      Weights<T, V> w;
      w.load(static_cast<const T *>(p.w[which]), unit.ca, unit.cb);
      finish<TURN>(r, a[u], b[u], w, c, s, y + unit.ca, y + unit.cb);
    }
  }
}

// Many tokens: a group of lanes keeps kHeads heads, all of queries or all of keys,
// and walks down the tokens; a head's row of the next token is under way as soon as
// this token's is done with.  blockIdx.y: a tile of the heads.
template <typename T, Turn TURN>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_rows_kernel(QkParams p, int lanes) {
  constexpr int V = 16 / sizeof(T);
  begin_after_stream();
  const int group = threadIdx.x / lanes, l = threadIdx.x % lanes;
  // groups of queries' heads come first, then those of the keys'
  const int sets = (p.heads[0] + kHeads - 1) / kHeads;
  int set = blockIdx.y * p.per_token + group % p.per_token;
  const int which = set < sets ? 0 : 1;
  const bool report = set == 0 && l == 0;
  set -= which ? sets : 0;
  const Unit<T, V, TURN> unit(p, l);
  int heads = (which ? p.heads[1] : p.heads[0]) - set * kHeads;  // of the group, if it has any
  if (group >= p.tokens * p.per_token) heads = 0;
  const int stride = which ? p.xs[1] : p.xs[0], out = which ? p.ys[1] : p.ys[0];
  const T *x = static_cast<const T *>(which ? p.x[1] : p.x[0]) + set * kHeads * p.d;
  T *y = static_cast<T *>(which ? p.y[1] : p.y[0]) + set * kHeads * p.d;
  const float scale = which ? 1.0f : p.q_scale;
  const long long step = (long long)gridDim.x * p.tokens;
  long long tok = (long long)blockIdx.x * p.tokens + group / p.per_token;
  Raw<T, V> a[kHeads], b[kHeads];
  auto ask = [&](long long t, int n) {
    if (t < p.N && n < heads && unit.mine) {
      const T *from = row_at(x, (int)t, stride) + n * p.d;
      a[n].load_once(from + unit.ca);
      b[n].load_once(from + unit.cb);
    }
  };
#pragma unroll
  for (int n = 0; n < kHeads; ++n) ask(tok, n);
  auto position = [&](long long t) { return TURN != kNoTurn && t < p.N && heads > 0 ? p.pos[t] : 0; };
  int pos = position(tok);
  Weights<T, V> w;
  if (heads > 0 && unit.mine) w.load(static_cast<const T *>(which ? p.w[1] : p.w[0]), unit.ca, unit.cb);
  // the block's tokens: every lane of a warp takes part in the shuffles
  for (long long base = (long long)blockIdx.x * p.tokens; base < p.N; base += step, tok += step) {
    const bool here = tok < p.N && heads > 0;
    const float *cs = TURN != kNoTurn && here ? table_row(p, pos, report) : nullptr;
    const bool sound = here && unit.mine && (TURN == kNoTurn || cs);
    float c[V], s[V];
    if (sound) unit.angles(p, cs, c, s);
    pos = position(tok + step);
    T *to = row_at(y, here ? (int)tok : 0, out);
#pragma unroll
    for (int n = 0; n < kHeads; ++n) {
      const bool live = n < heads && sound;
      const float sum = group_total(live ? squares(a[n], b[n]) : 0.0f, lanes);
      if (live)
        finish<TURN>(norm_factor(p, sum) * scale, a[n], b[n], w, c, s, to + n * p.d + unit.ca,
                     to + n * p.d + unit.cb);
      ask(tok + step, n);
    }
  }
}

// A group of lanes takes the rows of one head each in turn, the next one's loads
// under way while it works on a row.
template <typename TX, typename T, int V, int U>
__global__ void __launch_bounds__(kThreads, V == 1 ? 1 : 5) gated_norm_kernel(GateParams p, int lanes) {
  constexpr int N = V == 1 ? 1 : V / 2;
  begin_after_stream();
  const unsigned groups = kThreads / lanes, l = threadIdx.x % lanes, items = (unsigned)p.N * p.H;
  const unsigned units = p.d / V, step = gridDim.x * groups;
  unsigned item = blockIdx.x * groups + threadIdx.x / lanes;
  // the item's token and head, and how far they are from one item to the next
  int tok = item / p.H, head = item % p.H;
  const int tok_step = step / p.H, head_step = step % p.H;
  Raw<TX, V> x[U];
  Raw<T, V> g[U], w[U];
  auto load = [&](unsigned i) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i < items && l + u * lanes < units) {
        const int c = head * p.d + (l + u * lanes) * V;
        x[u].load_once(row_at(static_cast<const TX *>(p.x), tok, p.xs) + c);
        if (p.gate) g[u].load_once(row_at(static_cast<const T *>(p.gate), tok, p.gs) + c);
      }
  };
  load(item);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (p.w && l + u * lanes < units) w[u].load(static_cast<const T *>(p.w) + (l + u * lanes) * V);
  // every lane of a warp takes part in the shuffles, with or without a row
  for (unsigned base = blockIdx.x * groups; base < items; base += step) {
    using P = typename std::conditional<V == 1, float, f2>::type;
    P y[U][N], act[U][N];
    float sum = 0.0f;
    T *to = row_at(static_cast<T *>(p.y), tok, p.ys) + head * p.d + l * V;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (item >= items || l + u * lanes >= units) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if constexpr (V == 1) {
          y[u][e] = x[u].get(0);
          sum = fmaf(y[u][e], y[u][e], sum);
          if (p.gate) act[u][e] = sigmoid(g[u].get(0));
        } else {
          y[u][e] = x[u].pair(e);
          const float2 q = unpack2(mul2(y[u][e], y[u][e]));
          sum += q.x + q.y;
          if (p.gate) act[u][e] = sigmoid(g[u].pair(e));
        }
      }
      if (p.silu) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if constexpr (V == 1) act[u][e] *= g[u].get(0);
          else act[u][e] = mul2(act[u][e], g[u].pair(e));
        }
      }
    }
    tok += tok_step;
    head += head_step;
    if (head >= p.H) head -= p.H, ++tok;
    load(item + step);
    sum = group_total(sum, lanes);
    const float r = rsqrtf(fmaf(sum, p.share, p.eps));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (item >= items || l + u * lanes >= units) continue;
      float o[V];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if constexpr (V == 1) {
          float v = y[u][e] * r;
          if (p.w) v *= w[u].get(0);
          o[0] = p.gate ? v * act[u][e] : v;
        } else {
          f2 v = mul2(y[u][e], both(r));
          if (p.w) v = mul2(v, w[u].pair(e));
          if (p.gate) v = mul2(v, act[u][e]);
          const float2 q = unpack2(v);
          o[2 * e] = q.x;
          o[2 * e + 1] = q.y;
        }
      }
      store_vec<T, V>(to + u * lanes * V, o);
    }
    item += step;
  }
}

int up(int a, int b) { return (a + b - 1) / b; }
int pow2_up(int n) {
  int r = 1;
  while (r < n) r *= 2;
  return r;
}

// Whether V-element vectors serve all rows of a view.
bool fits(const void *p, long long stride_bytes) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

template <typename T, Turn TURN>
cudaError_t qk_norm(QkParams p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  // runs of V channels: no run is cut by the rotation's borders, rows start on 16 bytes
  bool vec = p.d % (2 * V) == 0 && (TURN == kNeighbours ? p.rot % V == 0 : p.rot % (2 * V) == 0);
  for (int i = 0; i < 2; ++i)
    if (p.heads[i]) vec = vec && fits(p.x[i], p.xs[i]) && fits(p.y[i], p.ys[i]);
  const int units = p.d / (vec ? 2 * V : 2), lanes = pow2_up(units < 32 ? units : 32), most = kThreads / lanes;
  const int total = p.heads[0] + p.heads[1];
  const bool rows = vec && (long long)p.N * total >= (long long)kHeads * kSms * 2 * most;
  const int sets = rows ? up(p.heads[0], kHeads) + up(p.heads[1], kHeads) : total;
  const int passes = up(sets, most);
  p.per_token = up(sets, passes);
  p.tokens = most / p.per_token;
  const int threads = up(p.tokens * p.per_token * lanes, 32) * 32;
  const int blocks = (int)(((long long)p.N + p.tokens - 1) / p.tokens);
  if (rows) {
    const int fill = up(2 * kSms, passes);
    return launch_after(qk_norm_rows_kernel<T, TURN>, dim3(blocks < fill ? blocks : fill, passes), dim3(threads), 0,
                        s, p, lanes);
  }
  if (vec) return launch_after(qk_norm_kernel<T, V, 1, TURN>, dim3(blocks), dim3(threads), 0, s, p, lanes);
  return launch_after(qk_norm_kernel<T, 1, 4, TURN>, dim3(blocks), dim3(threads), 0, s, p, lanes);
}

template <typename T>
cudaError_t qk_norm(const QkParams &p, cudaStream_t s) {
  if (p.rot == 0) return qk_norm<T, kNoTurn>(p, s);
  return p.interleaved ? qk_norm<T, kNeighbours>(p, s) : qk_norm<T, kHalves>(p, s);
}

template <typename TX, typename T>
cudaError_t gated_norm(const GateParams &p, cudaStream_t s) {
  constexpr int V = 16 / (sizeof(T) < sizeof(TX) ? sizeof(T) : sizeof(TX)), U = V == 8 ? 1 : 2;
  const bool vec = p.d % V == 0 && fits(p.x, p.xs) && fits(p.y, p.ys) && (!p.gate || fits(p.gate, p.gs));
  const int units = p.d / (vec ? V : 1), lanes = pow2_up(units < 32 ? units : 32);
  const long long groups = kThreads / lanes, blocks = ((long long)p.N * p.H + groups - 1) / groups;
  const dim3 grid(blocks < kSms * 5 ? blocks : kSms * 5);
  if (vec) return launch_after(gated_norm_kernel<TX, T, V, U>, grid, dim3(kThreads), 0, s, p, lanes);
  return launch_after(gated_norm_kernel<TX, T, 1, 8>, grid, dim3(kThreads), 0, s, p, lanes);
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
