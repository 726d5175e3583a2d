// Selective scan steps: rows of one or a few tokens, the state h [D][S] of
// each sequence in its slot:
//     h[n] = exp(delta A[n]) h[n] + delta x B[n],   y = C . h + D x  (gated)
//
// Memory bound: the states are read and written once, which is nearly all
// the bytes there are.  A thread owns eight states of one channel (S / 8 lanes
// a channel) and keeps their A in registers while it walks over the rows of
// its group, so A is read once per block and not once per row.  The states of
// the next rows are under way by asynchronous copies into a ring in shared
// memory, where each thread reads back only what it copied itself: no
// barriers, and enough bytes in flight for HBM with few registers.
// Rows of one token (no segment table) ask for the next row's token one row
// ahead; rows that may have several load kChunk tokens at a time, since a
// token's latency, not its work, is what a draft of eight costs.  The sum over
// states is a butterfly over the channel's lanes.
#include <type_traits>

#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kStates = 8;     // of a thread
constexpr int kQuads = kStates / 4;
constexpr int kRing = 4;       // rows of states in flight, the current one among them
constexpr int kMaxRows = 128;  // of a block

// Four neighbouring elements as they are in memory.
template <typename T>
struct Four {
  using Raw = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
  Raw r;
  template <bool VEC>
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (VEC) {
      r = *reinterpret_cast<const Raw *>(p);
    } else {
      alignas(16) T e[4] = {p[0], p[1], p[2], p[3]};
      r = *reinterpret_cast<const Raw *>(e);
    }
  }
  __device__ __forceinline__ void get(f2 *v) const {  // two pairs
    if constexpr (sizeof(T) == 4) {
      v[0] = pack2(__uint_as_float(r.x), __uint_as_float(r.y));
      v[1] = pack2(__uint_as_float(r.z), __uint_as_float(r.w));
    } else {
      v[0] = pack2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
      v[1] = pack2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
    }
  }
};

// One token's inputs of a thread.
template <typename T>
struct Token {
  T x, d, z;
  Four<T> b[kQuads], c[kQuads];
};

// Blocks on an SM (registers).
template <typename T>
__host__ __device__ constexpr int step_blocks(bool one) {
  return one && sizeof(T) == 2 ? 4 : 3;
}

// ONE: every row is one token, row i token i.  VEC: B and C by fours.
template <typename T, int S, bool VEC, bool ONE>
__global__ void __launch_bounds__(kThreads, step_blocks<T>(ONE)) scan_step_kernel(const ScanParams p) {
  constexpr int L = S / kStates;  // lanes of a channel
  constexpr int kChunk = ONE ? 1 : sizeof(T) == 2 ? 4 : 2;
  __shared__ SegLoc rec[kMaxRows];
  __shared__ ulonglong2 ring[kRing][kQuads][kThreads];

  const int tid = threadIdx.x, l = tid % L;
  const int ch = blockIdx.x * (kThreads / L) + tid / L;
  const bool on = ch < p.C_;
  const int c = on ? ch : p.C_ - 1;
  const int g = c / (p.C_ / p.G);
  const int i0 = blockIdx.y, di = gridDim.y;  // the block's rows
  const int rows = (p.seg.B - i0 + di - 1) / di;
  for (int r = tid; r < rows; r += kThreads) {
    SegLoc s;
    if (!locate_segment(p.seg, i0 + r * di, &s)) s.len = 0;
    rec[r] = s;
  }

  // states 4 (l + L j) + {0 .. 3}, as pairs
  f2 a[2 * kQuads];
#pragma unroll
  for (int j = 0; j < kQuads; ++j) {
    const ulonglong2 v =
        *reinterpret_cast<const ulonglong2 *>(p.A + (long long)c * S + 4 * (l + L * j));
    a[2 * j] = mul2(v.x, both(kLog2e));
    a[2 * j + 1] = mul2(v.y, both(kLog2e));
  }
  const float skip = p.D ? p.D[c] : 0.0f, bias = p.dtb ? p.dtb[c] : 0.0f;
  const long long row = (long long)p.C_ * S;
  float *pool = p.pool + (long long)c * S + 4 * l;
  const T *xb = static_cast<const T *>(p.x) + c, *db = static_cast<const T *>(p.dt) + c;
  const T *zb = p.z ? static_cast<const T *>(p.z) + c : nullptr;
  const T *Bb = static_cast<const T *>(p.B) + g * S + 4 * l;
  const T *Cb = static_cast<const T *>(p.C) + g * S + 4 * l;
  T *yb = static_cast<T *>(p.y) + c;

  auto fetch = [&](Token<T> &k, int t) {
    k.x = xb[t * p.xs];
    k.d = db[t * p.dts];
    if (zb) k.z = zb[t * p.zs];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      k.b[j].template load<VEC>(Bb + t * p.bs + 4 * L * j);
      k.c[j].template load<VEC>(Cb + t * p.cs + 4 * L * j);
    }
  };
  Token<T> in[kChunk];
  if (ONE) fetch(in[0], i0);
  __syncthreads();

  auto ask = [&](int r) {  // row r's states into the ring
    if (r < rows && rec[r].len > 0) {
      const float *from = pool + rec[r].slot * row;
#pragma unroll
      for (int j = 0; j < kQuads; ++j)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(&ring[r % kRing][j][tid])),
                     "l"(from + 4 * L * j)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int r = 0; r < kRing - 1; ++r) ask(r);

  for (int r = 0; r < rows; ++r) {
    ask(r + kRing - 1);
    const SegLoc s = rec[r];
    f2 h[2 * kQuads];
    // Token t of the row: h steps on, and its y goes out.
    auto token = [&](const Token<T> &k, int t) {
      const float x = in_scalar<T>(&k.x);
      float d = in_scalar<T>(&k.d) + bias;
      if (p.softplus) d = softplus_f(d);
      const f2 dd = both(d), dx = both(d * x);
      f2 o = 0;
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        f2 b[2], cc[2];
        k.b[j].get(b);
        k.c[j].get(cc);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f2 &v = h[2 * j + e];
          v = fma2(exp2_2(mul2(dd, a[2 * j + e])), v, mul2(dx, b[e]));
          o = fma2(cc[e], v, o);
        }
      }
      if (t + 1 == s.keep && on) {
#pragma unroll
        for (int j = 0; j < kQuads; ++j)
          *reinterpret_cast<ulonglong2 *>(pool + s.slot * row + 4 * L * j) =
              make_ulonglong2(h[2 * j], h[2 * j + 1]);
      }
      const float2 u = unpack2(o);
      float sum = u.x + u.y;
#pragma unroll
      for (int m = 1; m < L; m *= 2) sum += __shfl_xor_sync(~0u, sum, m);
      if (on && l == 0) {
        sum = fmaf(skip, x, sum);
        if (zb) sum *= silu_f(in_scalar<T>(&k.z));
        yb[(s.begin + t) * p.ys] = out_scalar<T>(sum);
      }
    };
    auto take = [&]() {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        const ulonglong2 v = ring[r % kRing][j][tid];
        h[2 * j] = v.x;
        h[2 * j + 1] = v.y;
      }
    };
    if constexpr (ONE) {
      const Token<T> now = in[0];
      if (r + 1 < rows) fetch(in[0], i0 + (r + 1) * di);
      take();
      if (s.len > 0) token(now, 0);
    } else {
      for (int t = 0; t < s.len; t += kChunk) {
#pragma unroll
        for (int u = 0; u < kChunk; ++u)
          if (t + u < s.len) fetch(in[u], s.begin + t + u);
        if (t == 0) take();
#pragma unroll
        for (int u = 0; u < kChunk; ++u)
          if (t + u < s.len) token(in[u], t + u);
      }
    }
  }
}

// Groups that the rows of a batch are dealt to, for gx blocks a group and
// `room` blocks on the machine: the number that ends first, if a block takes
// the time of its rows and of two more (its start).  Groups that overflow one
// wave by a few blocks cost a second one: 256 rows of 4096 channels with 64
// states took 115 us in 640 blocks where 608 fit, and TODO us by this rule.
int row_groups(int gx, int B, int room) {
  long long best = 0;
  int groups = 0;
  for (int gy = (B + kMaxRows - 1) / kMaxRows; gy <= B; ++gy) {
    const long long waves = ((long long)gx * gy + room - 1) / room;
    const long long cost = waves * ((B + gy - 1) / gy + 2);
    if (!groups || cost < best) {
      best = cost;
      groups = gy;
    }
    if ((long long)gx * gy >= 4LL * room) break;
  }
  return groups;
}

template <typename T, int S>
cudaError_t launch_step(const ScanParams &p, cudaStream_t st) {
  constexpr int cpb = kThreads / (S / kStates);
  const bool one = p.seg.cu == nullptr;
  const int gx = (p.C_ + cpb - 1) / cpb, B = p.seg.B;
  const int gy = row_groups(gx, B, 152 * step_blocks<T>(one));
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p.B) | reinterpret_cast<uintptr_t>(p.C) |
                         (uintptr_t)((p.bs | p.cs) * (long long)sizeof(T));
  const bool vec = (bits & (4 * sizeof(T) - 1)) == 0;
  const dim3 grid(gx, gy);
  if (one && vec) scan_step_kernel<T, S, true, true><<<grid, kThreads, 0, st>>>(p);
  else if (one) scan_step_kernel<T, S, false, true><<<grid, kThreads, 0, st>>>(p);
  else if (vec) scan_step_kernel<T, S, true, false><<<grid, kThreads, 0, st>>>(p);
  else scan_step_kernel<T, S, false, false><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_t(const ScanParams &p, cudaStream_t st) {
  switch (p.S) {
    case 16: return launch_step<T, 16>(p, st);
    case 32: return launch_step<T, 32>(p, st);
    case 64: return launch_step<T, 64>(p, st);
    default: return launch_step<T, 128>(p, st);
  }
}

}  // namespace

cudaError_t launch_scan_step(const ScanParams &p, kda_dtype dt, cudaStream_t s) {
  return dt == KDA_F32 ? launch_step_t<float>(p, s) : launch_step_t<__nv_bfloat16>(p, s);
}

}  // namespace kda
