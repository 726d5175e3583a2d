// Selective scan steps: rows of one or a few tokens, the state h [D][S] of
// each sequence in its slot:
//     h[n] = exp(delta A[n]) h[n] + delta x B[n],   y = C . h + D x  (gated)
//
// Memory bound: the states are read and written once, which is nearly all
// the bytes there are (256 rows of 4096 channels with 64 states: 87 us, 93 % of
// the copy bandwidth; 94 us in fp32).  A thread owns eight states of one channel (S / 8 lanes
// a channel) and keeps their A in registers while it walks over the rows of
// its group, so A is read once per block and not once per row.  The states of
// the next rows are under way by asynchronous copies into a ring in shared
// memory, where each thread reads back only what it copied itself: no
// barriers, and enough bytes in flight for HBM with few registers.
// Rows of one token (no segment table) ask for the next row's token one row
// ahead.  Rows that may have several take them from shared memory, up to kTake
// at a time and two such items ahead: a draft of eight costs its work, not
// eight latencies (64 rows, eight of them of eight tokens, 4096 channels: 11 us,
// 13 to 17 with the tokens loaded to registers in chunks; 64 us with 128 states,
// 64 % of the copy bandwidth, where 16 lanes of a channel prepare the same time
// step).  The sum over
// states is a butterfly over the channel's lanes.
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kPerSm = 4;      // blocks on an SM; fp32 inputs, one token a row: 3
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

// The recurrence of a thread's states over one token; returns its share of
// C . h.
template <typename T>
__device__ __forceinline__ float scan_token(f2 (&h)[2 * kQuads], const f2 (&a)[2 * kQuads],
                                            float d, float dx, const Four<T> *b,
                                            const Four<T> *c) {
  const f2 dd = both(d), dx2 = both(dx);
  f2 o = 0;
#pragma unroll
  for (int j = 0; j < kQuads; ++j) {
    f2 bb[2], cc[2];
    b[j].get(bb);
    c[j].get(cc);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f2 &v = h[2 * j + e];
      v = fma2(exp2_2(mul2(dd, a[2 * j + e])), v, mul2(dx2, bb[e]));
      o = fma2(cc[e], v, o);
    }
  }
  const float2 u = unpack2(o);
  return u.x + u.y;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = 1; m < L; m *= 2) v += __shfl_xor_sync(~0u, v, m);
  return v;
}

template <int S>
__device__ __forceinline__ void load_decay(const float *A, int c, int l, f2 (&a)[2 * kQuads]) {
  constexpr int L = S / kStates;
#pragma unroll
  for (int j = 0; j < kQuads; ++j) {  // states 4 (l + L j) + {0 .. 3}, as pairs
    const ulonglong2 v =
        *reinterpret_cast<const ulonglong2 *>(A + (long long)c * S + 4 * (l + L * j));
    const float2 x = unpack2(v.x), y = unpack2(v.y);
    a[2 * j] = pack2(exponent_scale(x.x), exponent_scale(x.y));
    a[2 * j + 1] = pack2(exponent_scale(y.x), exponent_scale(y.y));
  }
}

__device__ __forceinline__ void async16(void *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}
__device__ __forceinline__ void async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The rows of a block: blockIdx.y, + gridDim.y, ..; checked, once.
__device__ __forceinline__ int take_rows(const SegParams &p, SegLoc *rec) {
  const int di = gridDim.y, rows = (p.B - (int)blockIdx.y + di - 1) / di;
  for (int r = threadIdx.x; r < rows; r += kThreads) {
    SegLoc s;
    if (!locate_segment(p, blockIdx.y + r * di, &s)) s.len = 0;
    rec[r] = s;
  }
  return rows;
}

// One token's inputs of a thread.
template <typename T>
struct Token {
  T x, d, z;
  Four<T> b[kQuads], c[kQuads];
};

// Rows of one token, row i token i.  VEC: B and C are read by fours.
template <typename T, int S, bool VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? kPerSm : 3)
    scan_one_kernel(const ScanParams p) {
  constexpr int L = S / kStates;  // lanes of a channel
  __shared__ SegLoc rec[kMaxRows];
  __shared__ ulonglong2 ring[kRing][kQuads][kThreads];
  begin_after_stream();

  const int tid = threadIdx.x, l = tid % L;
  const int ch = blockIdx.x * (kThreads / L) + tid / L;
  const bool on = ch < p.C_;
  const int c = on ? ch : p.C_ - 1;
  const int g = c / (p.C_ / p.G);
  const int i0 = blockIdx.y, di = gridDim.y;
  const int rows = take_rows(p.seg, rec);

  f2 a[2 * kQuads];
  load_decay<S>(p.A, c, l, a);
  const float skip = p.D ? p.D[c] : 0.0f, bias = p.dtb ? p.dtb[c] : 0.0f;
  const long long row = (long long)p.C_ * S;
  float *pool = p.pool + (long long)c * S + 4 * l;
  const T *xb = static_cast<const T *>(p.x) + c, *db = static_cast<const T *>(p.dt) + c;
  const T *zb = p.z ? static_cast<const T *>(p.z) + c : nullptr;
  const T *Bb = static_cast<const T *>(p.B) + g * S + 4 * l;
  const T *Cb = static_cast<const T *>(p.C) + g * S + 4 * l;
  T *yb = static_cast<T *>(p.y) + c;

  auto fetch = [&](Token<T> &k, int t) {
    k.x = *row_at(xb, t, p.xs);
    k.d = *row_at(db, t, p.dts);
    if (zb) k.z = *row_at(zb, t, p.zs);
    const T *b = row_at(Bb, t, p.bs), *c4 = row_at(Cb, t, p.cs);
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      k.b[j].template load<VEC>(b + 4 * L * j);
      k.c[j].template load<VEC>(c4 + 4 * L * j);
    }
  };
  Token<T> ahead;  // the next row's
  fetch(ahead, i0);
  __syncthreads();

  auto ask = [&](int r) {  // row r's states into the ring
    if (r < rows && rec[r].len > 0) {
      const float *from = pool + rec[r].slot * row;
#pragma unroll
      for (int j = 0; j < kQuads; ++j) async16(&ring[r % kRing][j][tid], from + 4 * L * j);
    }
    async_commit();
  };
#pragma unroll
  for (int r = 0; r < kRing - 1; ++r) ask(r);

  for (int r = 0; r < rows; ++r) {
    ask(r + kRing - 1);
    const SegLoc s = rec[r];
    const Token<T> now = ahead;
    if (r + 1 < rows) fetch(ahead, i0 + (r + 1) * di);
    async_wait<kRing - 1>();
    if (s.len == 0) continue;
    f2 h[2 * kQuads];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const ulonglong2 v = ring[r % kRing][j][tid];
      h[2 * j] = v.x;
      h[2 * j + 1] = v.y;
    }
    const float x = in_scalar<T>(&now.x);
    float d = in_scalar<T>(&now.d) + bias;
    if (p.softplus) d = softplus_f(d);
    float o = scan_token<T>(h, a, d, d * x, now.b, now.c);
    if (s.keep > 0 && on) {
#pragma unroll
      for (int j = 0; j < kQuads; ++j)
        *reinterpret_cast<ulonglong2 *>(pool + s.slot * row + 4 * L * j) =
            make_ulonglong2(h[2 * j], h[2 * j + 1]);
    }
    o = lanes_sum<L>(o);
    if (on && l == 0) {
      o = fmaf(skip, x, o);
      if (zb) o *= silu_f(in_scalar<T>(&now.z));
      *row_at(yb, s.begin, p.ys) = out_scalar<T>(o);
    }
  }
}

// Rows of any number of tokens.  VEC: every row of a token tensor starts on 16
// bytes and a group's channels are a multiple of 16 bytes.
template <typename T, int S, bool VEC>
__global__ void __launch_bounds__(kThreads, kPerSm) scan_rows_kernel(const ScanParams p, int bpg) {
  constexpr int L = S / kStates, V = InVec<T>::kElems;
  constexpr int kTake = 16 / sizeof(T);             // tokens of an item
  constexpr int kStages = 3;                        // items in shared memory
  constexpr int kChans = kThreads / L;              // of a block, all of one group
  constexpr int NC = kChans / V, NS = S / V;        // 16-byte pieces of a token's rows
  constexpr int kPieces = 3 * NC + 2 * NS;
  __shared__ SegLoc rec[kMaxRows];
  __shared__ ulonglong2 ring[kStages][kQuads][kThreads];
  __shared__ uint4 toks[kStages][kTake][kPieces];   // x, dt, z, B, C of a token
  begin_after_stream();

  const int tid = threadIdx.x, l = tid % L, cl = tid / L;
  const int per = p.C_ / p.G, g = blockIdx.x / bpg;
  const int c0 = g * per + (blockIdx.x % bpg) * kChans;
  const int nch = min(kChans, (g + 1) * per - c0);
  const bool on = cl < nch;
  const int c = c0 + (on ? cl : nch - 1);
  const int rows = take_rows(p.seg, rec);

  f2 a[2 * kQuads];
  load_decay<S>(p.A, c, l, a);
  const float skip = p.D ? p.D[c] : 0.0f, bias = p.dtb ? p.dtb[c] : 0.0f;
  const long long row = (long long)p.C_ * S;
  float *pool = p.pool + (long long)c * S + 4 * l;
  T *yb = static_cast<T *>(p.y) + c;
  __syncthreads();

  // Items: kTake tokens of a row, from token t of row r on.
  auto skip_empty = [&](int r) {
    while (r < rows && rec[r].len == 0) ++r;
    return r;
  };
  auto advance = [&](int &r, int &t) {
    t += kTake;
    if (t >= rec[r].len) {
      r = skip_empty(r + 1);
      t = 0;
    }
  };
  auto ask = [&](int stage, int r, int t) {
    if (r < rows) {
      const SegLoc s = rec[r];
      if (t == 0) {
        const float *from = pool + s.slot * row;
#pragma unroll
        for (int j = 0; j < kQuads; ++j) async16(&ring[stage][j][tid], from + 4 * L * j);
      }
      const int n = min(kTake, s.len - t) * kPieces;
      for (int k = tid; k < n; k += kThreads) {
        const int u = k / kPieces, at = k % kPieces, tok = s.begin + t + u;
        const T *from;
        int first, left;  // element of the row, elements there are from it on
        if (at < 3 * NC) {
          const int w = at / NC;
          if (w == 2 && !p.z) continue;
          first = at % NC * V;
          left = nch - first;
          const T *base = static_cast<const T *>(w == 0 ? p.x : w == 1 ? p.dt : p.z) + c0;
          from = row_at(base, tok, w == 0 ? p.xs : w == 1 ? p.dts : p.zs) + first;
        } else {
          const bool is_b = at < 3 * NC + NS;
          first = (at - 3 * NC - (is_b ? 0 : NS)) * V;
          left = S;
          const T *base = static_cast<const T *>(is_b ? p.B : p.C) + g * S;
          from = row_at(base, tok, is_b ? p.bs : p.cs) + first;
        }
        if (left <= 0) continue;
        if (VEC) {
          async16(&toks[stage][u][at], from);
        } else {
          alignas(16) T e[V];
#pragma unroll
          for (int q = 0; q < V; ++q) e[q] = q < left ? from[q] : out_scalar<T>(0.0f);
          toks[stage][u][at] = *reinterpret_cast<const uint4 *>(e);
        }
      }
    }
    async_commit();
  };

  int r = skip_empty(0), t = 0;
  int ra = r, ta = 0;  // the item to ask for next
  int sa = 0, st = 0;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) {
    ask(sa, ra, ta);
    sa = sa + 1 == kStages ? 0 : sa + 1;
    if (ra < rows) advance(ra, ta);
  }
  f2 h[2 * kQuads];
  while (r < rows) {
    async_wait<kStages - 2>();
    // The item is there for all, and all are done with the one before it,
    // whose place the next one takes.
    __syncthreads();
    ask(sa, ra, ta);
    sa = sa + 1 == kStages ? 0 : sa + 1;
    if (ra < rows) advance(ra, ta);

    const SegLoc s = rec[r];
    if (t == 0) {
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        const ulonglong2 v = ring[st][j][tid];
        h[2 * j] = v.x;
        h[2 * j + 1] = v.y;
      }
    }
    const int n = min(kTake, s.len - t);
    for (int u = 0; u < n; ++u) {
      const T *in = reinterpret_cast<const T *>(toks[st][u]);
      const T *bc = in + 3 * kChans + 4 * l;
      Four<T> b[kQuads], cc[kQuads];
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        b[j].template load<true>(bc + 4 * L * j);
        cc[j].template load<true>(bc + S + 4 * L * j);
      }
      const float x = in_scalar<T>(in + cl);
      float d = in_scalar<T>(in + kChans + cl) + bias;
      if (p.softplus) d = softplus_f(d);
      float o = scan_token<T>(h, a, d, d * x, b, cc);
      if (t + u + 1 == s.keep && on) {
#pragma unroll
        for (int j = 0; j < kQuads; ++j)
          *reinterpret_cast<ulonglong2 *>(pool + s.slot * row + 4 * L * j) =
              make_ulonglong2(h[2 * j], h[2 * j + 1]);
      }
      o = lanes_sum<L>(o);
      if (on && l == 0) {
        o = fmaf(skip, x, o);
        if (p.z) o *= silu_f(in_scalar<T>(in + 2 * kChans + cl));
        *row_at(yb, s.begin + t + u, p.ys) = out_scalar<T>(o);
      }
    }
    advance(r, t);
    st = st + 1 == kStages ? 0 : st + 1;
  }
}

// Groups that the rows of a batch are dealt to, for gx blocks a group and
// `room` blocks on the machine: as many as fill one to four waves, whichever
// ends first if a block takes the time of its rows and of two more (its
// start).  Rows count alike, since their lengths are on the device: with drafts
// the group that has most of them lasts longest.  Groups that overflow a wave by a few blocks cost another one: 256
// rows of 4096 channels with 64 states took 115 us in 640 blocks where 608 fit,
// and 89 us by this rule.
int row_groups(int gx, int B, int room) {
  const int least = (B + kMaxRows - 1) / kMaxRows;
  long long best = 0;
  int groups = 0;
  for (int w = 1; w <= 4; ++w) {
    int gy = w * room / gx;
    gy = gy < least ? least : gy > B ? B : gy;
    const long long waves = ((long long)gx * gy + room - 1) / room;
    const long long cost = waves * ((B + gy - 1) / gy + 2);
    if (!groups || cost < best) {
      best = cost;
      groups = gy;
    }
  }
  return groups;
}

template <typename T, int S>
cudaError_t launch_step(const ScanParams &p, cudaStream_t st) {
  constexpr int kChans = kThreads / (S / kStates);
  const uintptr_t bc = reinterpret_cast<uintptr_t>(p.B) | reinterpret_cast<uintptr_t>(p.C) |
                       (uintptr_t)(p.bs | p.cs);
  if (!p.seg.cu) {
    const int gx = (p.C_ + kChans - 1) / kChans;
    const dim3 grid(gx, row_groups(gx, p.seg.B, 152 * (sizeof(T) == 2 ? kPerSm : 3)));
    return launch_after(bc % (4 * sizeof(T)) == 0 ? scan_one_kernel<T, S, true>
                                                  : scan_one_kernel<T, S, false>,
                        grid, dim3(kThreads), 0, st, p);
  }
  const uintptr_t all = bc | reinterpret_cast<uintptr_t>(p.x) |
                        reinterpret_cast<uintptr_t>(p.dt) | reinterpret_cast<uintptr_t>(p.z) |
                        (uintptr_t)(p.xs | p.dts | p.zs);
  const int per = p.C_ / p.G, bpg = (per + kChans - 1) / kChans, gx = p.G * bpg;
  const dim3 grid(gx, row_groups(gx, p.seg.B, 152 * kPerSm));
  return launch_after(all % 16 == 0 && per % InVec<T>::kElems == 0 ? scan_rows_kernel<T, S, true>
                                                                    : scan_rows_kernel<T, S, false>,
                      grid, dim3(kThreads), 0, st, p, bpg);
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
