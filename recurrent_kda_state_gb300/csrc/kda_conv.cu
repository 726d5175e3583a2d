// Short causal depthwise convolution over packed segments, with the last
// W - 1 inputs of each sequence kept in its slot:
//     y[t] = act(bias + sum_j w[j] u[t + j]),  u = [slot's W - 1 rows; x rows]
//
// Memory bound: x is read and y written once, 2 W + 4 flops a value.  A
// thread owns four neighbouring channels and walks down a run of tokens with
// the W - 1 previous rows in registers and eight rows (six in fp32) under way,
// as raw elements: the place of a row that was used takes a new one.  Four
// channels, not the eight of a 16-byte bf16 vector: those took 190 registers,
// which left eight warps an SM and 165 us where this takes 65, 91 % of the copy
// bandwidth (8192 x 12288, W = 4).
// A prompt's segments are cut into tiles of p.tile tokens, each with its own
// W - 1 rows before it.  Tile 0 alone reads the slot and alone writes it (it
// fetches the segment's last rows itself), so no other block can see a state
// that is already replaced.
// Odd channels, or rows that are not on a multiple of four elements, take one
// element a thread: 8192 x 12287 101 us, in fp32 147 (12288: 124).
#include "kda_ssm.cuh"

namespace kda {
namespace {

// Blocks of 128 threads on an SM, and rows of loads in flight of a thread: what
// registers leave (bf16 68 us with six blocks, 84 with eight; fp32 8.2 us with
// five blocks and six rows, 8.6 with six and four, 5003 x 1000).
template <typename T>
__host__ __device__ constexpr int blocks_of() {
  return sizeof(T) == 2 ? 7 : 5;
}
template <typename T>
__host__ __device__ constexpr int rows_ahead() {
  return sizeof(T) == 2 ? 8 : 6;
}
constexpr int kTileUnit = 8;  // tiles are multiples of this many tokens,
constexpr int kMaxTile = 48;  // and this long where there are enough of them

// V values in fp32, as packed pairs where there are four: one instruction for
// two channels.
template <int V>
struct Vals {
  using P = typename std::conditional<V == 1, float, f2>::type;
  static constexpr int N = V == 1 ? 1 : V / 2;
  P v[N];
};
__device__ __forceinline__ float madd(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ f2 madd(f2 a, f2 b, f2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float silu_of(float v) { return silu_f(v); }
__device__ __forceinline__ f2 silu_of(f2 v) { return silu2(v); }

// V elements as they are in memory (V = 1, or 4 of them aligned as a whole).
template <typename T, int V>
struct Elems {
  using Raw = typename std::conditional<V == 1, T,
              typename std::conditional<sizeof(T) == 4, uint4, uint2>::type>::type;
  Raw r;
  __device__ __forceinline__ void load(const T *p) { r = *reinterpret_cast<const Raw *>(p); }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Raw *>(p) = r; }
  // Rows pass through once: marked to leave L2 first (5003 x 1000 fp32 among
  // other data of 400 MB: 10.4 us without the marks, 9.9 with them; called again
  // and again on 80 MB, which L2 holds, 6.9 and 8.4; 8192 x 12288: no difference).
  __device__ __forceinline__ void load_once(const T *p) {
    if constexpr (V == 1) load(p);
    else r = __ldcs(reinterpret_cast<const Raw *>(p));
  }
  __device__ __forceinline__ void store_once(T *p) const {
    if constexpr (V == 1) store(p);
    else __stcs(reinterpret_cast<Raw *>(p), r);
  }
  __device__ __forceinline__ Vals<V> get() const {
    Vals<V> o;
    if constexpr (V == 1) {
      o.v[0] = in_scalar<T>(&r);
    } else if constexpr (sizeof(T) == 4) {
      o.v[0] = pack2(__uint_as_float(r.x), __uint_as_float(r.y));
      o.v[1] = pack2(__uint_as_float(r.z), __uint_as_float(r.w));
    } else {
      o.v[0] = pack2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
      o.v[1] = pack2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
    }
    return o;
  }
  __device__ __forceinline__ void set(const Vals<V> &o) {
    if constexpr (V == 1) {
      r = out_scalar<T>(o.v[0]);
    } else {
      const float2 a = unpack2(o.v[0]), b = unpack2(o.v[1]);
      if constexpr (sizeof(T) == 4) {
        r = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                       __float_as_uint(b.y));
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(a.x, a.y);
        const __nv_bfloat162 q = __floats2bfloat162_rn(b.x, b.y);
        r = make_uint2(*reinterpret_cast<const uint32_t *>(&p),
                       *reinterpret_cast<const uint32_t *>(&q));
      }
    }
  }
};

// The taps and biases of a thread's channels; asked for before the segment is
// looked up, which they do not depend on.
template <typename T, int V, int W>
struct Taps {
  Vals<V> w[W], bias;
  __device__ __forceinline__ Taps(const ConvParams &p, int c) {
    const T *wp = static_cast<const T *>(p.weight) + (long long)c * W;
    const T *bp = static_cast<const T *>(p.bias);
    float flat[W][V], b[V];
    alignas(16) T e[V * W];  // [channel][tap]
#pragma unroll
    for (int j = 0; j < W; ++j) {
      Elems<T, V> q;
      q.load(wp + j * V);
      *reinterpret_cast<typename Elems<T, V>::Raw *>(e + j * V) = q.r;
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
      b[u] = bp ? in_scalar<T>(bp + c + u) : 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) flat[j][u] = in_scalar<T>(&e[u * W + j]);
    }
#pragma unroll
    for (int n = 0; n < Vals<V>::N; ++n) {
      if constexpr (V == 1) bias.v[n] = b[n];
      else bias.v[n] = pack2(b[2 * n], b[2 * n + 1]);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if constexpr (V == 1) w[j].v[n] = flat[j][n];
        else w[j].v[n] = pack2(flat[j][2 * n], flat[j][2 * n + 1]);
      }
    }
  }
};

// Tokens [t0, t1) of the segment (local indices; t0 = 0 or t0 >= W - 1).
template <typename T, int V, int W>
__device__ __forceinline__ void conv_run(const ConvParams &p, const Taps<T, V, W> &f,
                                         const SegLoc &s, int i, int c, int t0, int t1) {
  using E = Elems<T, V>;
  constexpr int kRows = rows_ahead<T>();
  const long long D = p.D;
  const T *x = row_at(static_cast<const T *>(p.x), s.begin, p.xs) + c;
  T *y = row_at(static_cast<T *>(p.y), s.begin, p.ys) + c;
  T *state = static_cast<T *>(p.pool) + (long long)s.slot * (W - 1) * D + c;

  E in[kRows], win[W - 1];
  const T *ahead = row_at(x, t0, p.xs);  // the next row to ask for
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (t0 + r < t1) in[r].load_once(ahead);
    ahead = row_at(ahead, 1, p.xs);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    if (t0 == 0) win[j].load(state + j * D);
    else win[j].load(row_at(x, t0 - (W - 1) + j, p.xs));
  }
  // the state after k tokens, u[k .. k + W - 2], into a slot
  auto write_state = [&](int k, int slot) {
    E row[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int at = k + j - (W - 1);
      if (at >= 0) {
        row[j].load(row_at(x, at, p.xs));
      } else {  // only where t0 = 0: win is the slot's
#pragma unroll
        for (int q = 0; q < W - 1; ++q)
          if (q == k + j) row[j] = win[q];
      }
    }
    T *to = static_cast<T *>(p.pool) + (long long)slot * (W - 1) * D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[j].store(to + j * D);
  };
  if (t0 == 0 && s.keep > 0) write_state(s.keep, s.slot);
  if (p.seg.ckpt_slots) {
    const long long p0 = p.seg.start_pos ? p.seg.start_pos[i] : 0, every = p.seg.ckpt_every;
    for (long long k = ((p0 + t0) / every + 1) * every - p0; k <= t1; k += every) {
      const int slot = checkpoint_slot(p.seg, i, p0, k);
      if (slot >= 0) write_state((int)k, slot);
    }
  }

  T *out = row_at(y, t0, p.ys);
  Vals<V> last[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) last[j] = win[j].get();
  auto token = [&](const E &cur) {
    const Vals<V> x = cur.get();
    Vals<V> acc = f.bias;
#pragma unroll
    for (int n = 0; n < Vals<V>::N; ++n) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) acc.v[n] = madd(f.w[j].v[n], last[j].v[n], acc.v[n]);
      acc.v[n] = madd(f.w[W - 1].v[n], x.v[n], acc.v[n]);
      if (p.silu) acc.v[n] = silu_of(acc.v[n]);
    }
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) last[j] = last[j + 1];
    last[W - 2] = x;
    E o;
    o.set(acc);
    o.store_once(out);
    out = row_at(out, 1, p.ys);
  };
  int t = t0;
  for (; t + 2 * kRows <= t1; t += kRows) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      token(in[r]);
      in[r].load_once(ahead);
      ahead = row_at(ahead, 1, p.xs);
    }
  }
  for (; t < t1; t += kRows) {  // the last rows, fewer than twice kRows
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (t + r < t1) token(in[r]);
      if (t + r + kRows < t1) in[r].load_once(ahead);
      ahead = row_at(ahead, 1, p.xs);
    }
  }
}

// One row of threads (threadIdx.y) per tile; blockIdx.x: channels.
template <typename T, int V, int W>
__global__ void __launch_bounds__(128, blocks_of<T>()) conv_step_kernel(const ConvParams p) {
  begin_after_stream();
  const int i = blockIdx.y * blockDim.y + threadIdx.y;
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (i >= p.seg.B || c >= p.D) return;
  const Taps<T, V, W> f(p, c);
  SegLoc s;
  if (!locate_segment(p.seg, i, &s) || s.len == 0) return;
  conv_run<T, V, W>(p, f, s, i, c, 0, s.len);
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
__global__ void __launch_bounds__(128, blocks_of<T>()) conv_prefill_kernel(const ConvParams p) {
  begin_after_stream();
  const int g = blockIdx.y * blockDim.y + threadIdx.y;
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * V;
  const Taps<T, V, W> f(p, c < p.D ? c : 0);
  const int i = find_segment(p.seg, g, p.tile);
  if (c >= p.D) return;
  SegLoc s;
  if (!locate_segment(p.seg, i, &s)) return;
  const long long t0 = (long long)(g - (s.begin / p.tile + i)) * p.tile;
  if (t0 < 0 || t0 >= s.len) return;
  conv_run<T, V, W>(p, f, s, i, c, (int)t0, (int)min((long long)s.len, t0 + p.tile));
}

template <typename T, int V, int W>
cudaError_t launch_w(const ConvParams &p, bool step, cudaStream_t st) {
  const int nvec = (p.D + V - 1) / V;
  const int bx = nvec >= 128 ? 128 : (nvec + 31) / 32 * 32;
  const dim3 block(bx, 128 / bx);
  const int gx = (nvec + bx - 1) / bx;
  if (step) {
    const dim3 grid(gx, (p.seg.B + block.y - 1) / block.y);
    return launch_after(conv_step_kernel<T, V, W>, grid, block, 0, st, p);
  }
  // Tiles as long as leaves every SM its blocks of 128 threads once.
  ConvParams q = p;
  const long long want = 152LL * blocks_of<T>() * 128;
  long long tile = (long long)p.seg.N * nvec / want / kTileUnit * kTileUnit + kTileUnit;
  q.tile = (int)(tile < kTileUnit ? kTileUnit : tile > kMaxTile ? kMaxTile : tile);
  long long tiles = (long long)p.seg.N / q.tile + p.seg.B;
  while ((tiles + block.y - 1) / block.y > 65535) {  // the grid's y limit
    q.tile *= 2;
    tiles = (long long)p.seg.N / q.tile + p.seg.B;
  }
  const dim3 grid(gx, (unsigned)((tiles + block.y - 1) / block.y));
  return launch_after(conv_prefill_kernel<T, V, W>, grid, block, 0, st, q);
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
  constexpr int V = 4;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y) |
                         (uintptr_t)(p.xs | p.ys);
  const bool vec = bits % (V * sizeof(T)) == 0 && p.D % V == 0;
  return vec ? launch_v<T, V>(p, step, st) : launch_v<T, 1>(p, step, st);
}

}  // namespace

cudaError_t launch_conv(const ConvParams &p, kda_dtype dt, bool step, cudaStream_t s) {
  return dt == KDA_F32 ? launch_t<float>(p, step, s) : launch_t<__nv_bfloat16>(p, step, s);
}

}  // namespace kda
