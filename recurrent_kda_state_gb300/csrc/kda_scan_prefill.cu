// Selective scan of packed prompts:
//     h[n] = exp(delta A[n]) h[n] + delta x B[n],   y = C . h + D x  (gated)
//
// Per (token, channel, state) one ex2 and four fp32 operations, against 8
// bytes per (token, channel): at S = 16 the arithmetic pipes bound it, not
// HBM.  The bare loop over tokens (ex2, the products and sums, the loads of B
// and C from shared memory) takes 105 cycles per SM quarter for 512 states,
// whichever way states and channels are packed; MUFU alone would take 64,
// the fp32 pipe 72.
//   - A thread owns eight states of two neighbouring channels in registers
//     (S / 8 lanes a channel pair).  The pair's values travel as packed fp32
//     pairs, one instruction for both.
//   - A block takes tiles of 16 tokens: x, dt and z rows by asynchronous
//     copies, B and C through registers, the next tile's while this one's
//     are used; one barrier a tile.
//   - Of each group of S / 8 tokens, lane l prepares token l for its pair
//     (softplus, delta x), hands it to the pair's lanes through shared memory,
//     and ends with that token's y, since the sums over lanes are exchanged
//     token against token.  So skip, gate and the store need no second pass
//     through shared memory and every lane has its share of them.
//
// Few long segments leave most of the machine idle, so with a workspace a
// segment is cut into parts: a first launch computes each part's end state
// from a zero start and its sum of delta; the second starts part k from
// h = exp(A sum_j delta) h + end_j over the parts before it, and does the rest.
// The first launch repeats the exponentials (two fifths of the time of a
// prompt that is cut everywhere).  Around the two:
//   - in large ragged batches a launch before them lists the parts, the long
//     ones first (scan_plan_kernel);
//   - where segments have many parts, one between them joins the ends once
//     instead of every part for itself (scan_join_kernel; 8192 tokens of 4096
//     channels in 48 parts: 281 us without it, 266 with it).
// 265 us for 8192 x 4096 channels x 16 states in bf16 (268 MB: 40 us at the
// copy bandwidth; the two bare loops alone 163 us), 304 us in fp32; 16384 tokens
// in 37 prompts 421 to 486 us over ten draws of their lengths (428 us in the
// figures below, 0 to 2414 tokens), 474 us in fp32.  Channels that are no
// multiple of a vector: 8192 x 4095 337 us, 455 us in fp32.
#include <algorithm>
#include <cmath>

#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kStates = 8;  // of a thread, for each of two channels
constexpr int kTile = 16;   // tokens of a tile; parts and tiles start on multiples of it
constexpr int kCarry = 2 * kStates + 2;  // floats a thread carries between parts

// Blocks on an SM, set by registers.  The first launch is faster with four of
// more registers (266 us the pair, 269 with five and 270 with six, 8192 tokens
// of 4096 channels), the second with five (274 with four).
__host__ __device__ constexpr int blocks_of(int elem, int S, bool local) {
  return elem == 4 ? 3 : S <= 32 && !local ? 5 : 4;
}

template <typename T, int S>
struct Shape {
  static constexpr int kLanes = S / kStates;        // of a channel pair
  static constexpr int kPairs = kThreads / kLanes;  // of a block
  static constexpr int kChans = 2 * kPairs;
  // bytes of a staged row: the padding lets kLanes tokens of a warp's pairs be
  // read without bank conflicts
  static constexpr int kPad = 64 * (int)sizeof(T) / kLanes;
  static constexpr int kPitch = kChans * (int)sizeof(T) + (kPad < 16 ? 16 : kPad);
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void copy16(void *to, const void *from, bool on) {
  const int n = on ? 16 : 0;  // 0: the 16 bytes become zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from),
               "r"(n) : "memory");
}

// The part of a segment that a block works on.
struct Part {
  int i;           // segment
  int k, count;    // part of it, number of its parts
  int v0;          // its first carry slot in the workspace
  int at;          // local token of the part's first tile (may be below 0)
  int lo, hi;      // local tokens [lo, hi)
  long long p0;    // absolute position of the segment's first token
};

__device__ __forceinline__ long long first_position(const SegParams &g, int i) {
  return g.ckpt_slots && g.start_pos ? g.start_pos[i] : 0;
}
__device__ __forceinline__ int part_count(int len, int r, int part) {
  return (int)(((long long)len + r + part - 1) / part);
}

template <bool LOCAL>
__device__ __forceinline__ bool find_part(const ScanParams &p, int v, Part *q, SegLoc *s) {
  const SegParams &g = p.seg;
  int i = v, k = -1;
  if (p.table) {
    const int2 total = p.table[0];
    if (v >= (LOCAL ? total.y : total.x)) return false;
    const int2 at = p.table[1 + v];
    i = at.x;
    k = at.y;
  } else if (p.part) {  // the last segment with cu[i] / part + spare i <= v: room for its parts
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = g.B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int j = lo + lane * step;
      const unsigned m = __ballot_sync(~0u, j < hi && g.cu[j] / p.part + p.spare * j <= v);
      lo += m ? (31 - __clz(m)) * step : 0;
      hi = min(lo + step, hi);
    }
    i = lo;
  }
  if (!locate_segment(g, i, s) || s->len == 0) return false;
  q->i = i;
  q->p0 = first_position(g, i);
  const int r = (int)(q->p0 & (kTile - 1));  // tiles end on absolute multiples
  if (!p.part) {
    q->k = 0;
    q->count = 1;
    q->v0 = 0;
    q->at = -r;
    q->hi = s->len;
  } else {
    q->v0 = s->begin / p.part + p.spare * i;
    q->k = k >= 0 ? k : v - q->v0;
    q->count = part_count(s->len, r, p.part);
    if (q->k < 0 || q->k >= q->count) return false;
    const long long at = (long long)q->k * p.part - r;
    q->at = (int)at;
    q->hi = (int)min((long long)s->len, at + p.part);
  }
  q->lo = max(0, q->at);
  return true;
}

// The parts of all segments in the order they are worked on, as {segment,
// part}: first all but each segment's last part, which are the longest, then
// the last ones by falling length.  Long blocks that start last would keep the
// machine waiting, and blocks with nothing to do, scattered among the others,
// would leave the work unevenly spread over the SMs.  One block.
constexpr int kPlanThreads = 1024, kBuckets = 64;
__global__ void __launch_bounds__(kPlanThreads)
    scan_plan_kernel(const ScanParams p, int room, int room_local) {
  __shared__ unsigned long long first[kBuckets];  // parts of a length, then where they go
  __shared__ bool sound;
  begin_after_stream();
  const int tid = threadIdx.x;
  if (tid < kBuckets) first[tid] = 0;
  __syncthreads();
  auto segment = [&](int i, int *count, int *bucket) {
    SegLoc s;
    if (!locate_segment(p.seg, i, &s) || s.len == 0) return false;
    const int r = (int)(first_position(p.seg, i) & (kTile - 1));
    *count = part_count(s.len, r, p.part);
    const long long last = s.len + r - (*count - 1LL) * p.part;  // tokens, 1 .. part
    *bucket = 1 + (int)((p.part - last) * (kBuckets - 2) / p.part);
    return true;
  };
  int n, b;
  for (int i = tid; i < p.seg.B; i += kPlanThreads) {
    if (!segment(i, &n, &b)) continue;
    if (n > 1) atomicAdd(&first[0], (unsigned long long)(n - 1));
    atomicAdd(&first[b], 1ull);
  }
  __syncthreads();
  if (tid == 0) {
    const unsigned long long local = first[0];
    unsigned long long sum = 0;
    for (int k = 0; k < kBuckets; ++k) {
      const unsigned long long c = first[k];
      first[k] = sum;
      sum += c;
    }
    // Segments that overlap can have more parts than the table has room for:
    // nothing is done then.
    sound = sum <= (unsigned)room && local <= (unsigned)room_local;
    p.table[0] = sound ? make_int2((int)sum, (int)local) : make_int2(0, 0);
    if (!sound) set_error(p.seg.err, KDA_DERR_SEGMENT);
  }
  __syncthreads();
  if (!sound) return;
  for (int i = tid; i < p.seg.B; i += kPlanThreads) {
    if (!segment(i, &n, &b)) continue;
    if (n > 1) {
      const int at = (int)atomicAdd(&first[0], (unsigned long long)(n - 1));
      for (int k = 0; k < n - 1; ++k) p.table[1 + at + k] = make_int2(i, k);
    }
    p.table[1 + (int)atomicAdd(&first[b], 1ull)] = make_int2(i, n - 1);
  }
}

// LOCAL: the first launch (end states of the parts, no outputs).
template <typename T, int S, bool VEC, bool LOCAL>
__global__ void __launch_bounds__(kThreads, blocks_of(sizeof(T), S, LOCAL))
    scan_prefill_kernel(const ScanParams p, int nblk) {
  using Sh = Shape<T, S>;
  constexpr int V = InVec<T>::kElems, NC = Sh::kChans / V, L = Sh::kLanes;
  constexpr int ITEMS = kTile * NC, NI = (ITEMS + kThreads - 1) / kThreads;
  constexpr int NB = kTile * S / kThreads;
  constexpr int TENSORS = LOCAL ? 2 : 3;
  constexpr int kRaw = kTile * Sh::kPitch;  // bytes of a tensor's tile
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char *raw = smem;                                     // [2][x, dt, z][kRaw]
  float *sbc = reinterpret_cast<float *>(raw + 2 * TENSORS * kRaw);  // [2][B, C][kTile][S]
  constexpr int kBC = (LOCAL ? 1 : 2) * kTile * S;
  float4 *swarp = reinterpret_cast<float4 *>(sbc + 2 * kBC);     // [2][kThreads]

  // The first launch of a call waits for the stream before it lets the next
  // begin, so that one may read the call's inputs at once and waits only for
  // the carried states.  A large batch waits for the launch to end: blocks that
  // start into the gaps it leaves are unevenly spread.
  const bool first = LOCAL || !p.part;
  if (first) begin_after_stream();
  if (LOCAL && !p.table) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int tid = threadIdx.x;
  const int v = blockIdx.x / nblk, blk = blockIdx.x % nblk;
  Part q;
  SegLoc s;
  if (!find_part<LOCAL>(p, v, &q, &s)) return;
  if (LOCAL && q.k + 1 >= q.count) return;

  // the block's channels: kChans of one group
  const int per = p.C_ / p.G, bpg = nblk / p.G, g = blk / bpg;
  const int c0 = g * per + (blk % bpg) * Sh::kChans;
  const int nch = min(Sh::kChans, (g + 1) * per - c0);

  // this thread's pair of channels and states 4 (l + kLanes j) + {0 .. 3}
  const int l = tid % Sh::kLanes, pr = tid / Sh::kLanes;
  const int ca = c0 + min(2 * pr, nch - 1), cb = c0 + min(2 * pr + 1, nch - 1);
  f2 a[kStates], h[kStates];
#pragma unroll
  for (int j = 0; j < kStates / 4; ++j) {
    const int n = 4 * (l + Sh::kLanes * j);
    const float4 x = *reinterpret_cast<const float4 *>(p.A + (long long)ca * S + n);
    const float4 y = *reinterpret_cast<const float4 *>(p.A + (long long)cb * S + n);
    a[4 * j] = pack2(exponent_scale(x.x), exponent_scale(y.x));
    a[4 * j + 1] = pack2(exponent_scale(x.y), exponent_scale(y.y));
    a[4 * j + 2] = pack2(exponent_scale(x.z), exponent_scale(y.z));
    a[4 * j + 3] = pack2(exponent_scale(x.w), exponent_scale(y.w));
  }

  const long long row = (long long)p.C_ * S;
  auto load_state = [&](const float *from) {
#pragma unroll
    for (int j = 0; j < kStates / 4; ++j) {
      const int n = 4 * (l + Sh::kLanes * j);
      const float4 x = *reinterpret_cast<const float4 *>(from + (long long)ca * S + n);
      const float4 y = *reinterpret_cast<const float4 *>(from + (long long)cb * S + n);
      h[4 * j] = pack2(x.x, y.x);
      h[4 * j + 1] = pack2(x.y, y.y);
      h[4 * j + 2] = pack2(x.z, y.z);
      h[4 * j + 3] = pack2(x.w, y.w);
    }
  };
  auto store_state = [&](float *to) {
#pragma unroll
    for (int j = 0; j < kStates / 4; ++j) {
      const int n = 4 * (l + Sh::kLanes * j);
      const float2 x = unpack2(h[4 * j]), y = unpack2(h[4 * j + 1]), z = unpack2(h[4 * j + 2]),
                   w = unpack2(h[4 * j + 3]);
      if (2 * pr < nch)
        *reinterpret_cast<float4 *>(to + (long long)ca * S + n) = make_float4(x.x, y.x, z.x, w.x);
      if (2 * pr + 1 < nch)
        *reinterpret_cast<float4 *>(to + (long long)cb * S + n) = make_float4(x.y, y.y, z.y, w.y);
    }
  };
  // carry slot of a part: [value][thread], so that warps move whole lines
  auto carry = [&](int slot) {
    return p.ws + ((long long)slot * nblk + blk) * (kCarry * kThreads) + tid;
  };
  auto store_carry = [&](int slot, f2 sum) {
    float *w = carry(slot);
#pragma unroll
    for (int n = 0; n < kStates; ++n) {
      const float2 x = unpack2(h[n]);
      w[(2 * n) * kThreads] = x.x;
      w[(2 * n + 1) * kThreads] = x.y;
    }
    const float2 x = unpack2(sum);
    w[2 * kStates * kThreads] = x.x;
    w[(2 * kStates + 1) * kThreads] = x.y;
  };

  f2 bias = 0, skip = 0;
  if (p.dtb) bias = pack2(p.dtb[ca], p.dtb[cb]);
  if (!LOCAL && p.D) skip = pack2(p.D[ca], p.D[cb]);

  const T *rows[3] = {row_at(static_cast<const T *>(p.x), s.begin, p.xs) + c0,
                      row_at(static_cast<const T *>(p.dt), s.begin, p.dts) + c0,
                      row_at(static_cast<const T *>(p.z), s.begin, p.zs) + c0};
  const int strides[3] = {p.xs, p.dts, p.zs};
  const T *B = row_at(static_cast<const T *>(p.B), s.begin, p.bs) + g * S;
  const T *C = row_at(static_cast<const T *>(p.C), s.begin, p.cs) + g * S;
  T *y = row_at(static_cast<T *>(p.y), s.begin, p.ys) + c0 + 2 * pr;
  const bool gate = !LOCAL && p.z != nullptr;

  // 16 bytes (V channels of one token) at a time; what lies outside the part
  // or the block's channels becomes zero
  auto fetch_rows = [&](int at, int stage) {
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      const int it = tid + k * kThreads;
      if (ITEMS % kThreads != 0 && it >= ITEMS) break;
      const int t = at + it / NC, c = (it % NC) * V;
      const bool on = t >= q.lo && t < q.hi && c < nch;
#pragma unroll
      for (int w = 0; w < TENSORS; ++w) {
        if (w == 2 && !gate) break;
        unsigned char *to =
            raw + (stage * TENSORS + w) * kRaw + it / NC * Sh::kPitch + it % NC * 16;
        const T *from = on ? row_at(rows[w], t, strides[w]) + c : rows[w];
        if (VEC) {
          copy16(to, on ? static_cast<const void *>(from) : p.A, on);
        } else {
          alignas(16) T e[V];
#pragma unroll
          for (int u = 0; u < V; ++u) e[u] = on && c + u < nch ? from[u] : out_scalar<T>(0.0f);
          *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(e);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  T rb[NB], rc[NB];  // converted when they are staged, not when they are asked for
  auto fetch_bc = [&](int at) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int e = tid + k * kThreads, t = at + e / S;
      const bool on = t >= q.lo && t < q.hi;
      rb[k] = on ? row_at(B, t, p.bs)[e % S] : out_scalar<T>(0.0f);
      if (!LOCAL) rc[k] = on ? row_at(C, t, p.cs)[e % S] : out_scalar<T>(0.0f);
    }
  };

  f2 sum = 0;
  const int tiles = (q.hi - q.at + kTile - 1) / kTile;
  fetch_rows(q.at, 0);
  fetch_bc(q.at);

  // What the launch before this one wrote is read from here on.
  if (!first) begin_after_stream();

  // The state at the part's start.  The carry slot of part 0 holds the slot's
  // own state, since the last part replaces that; slot k holds part k - 1's
  // end (for k = 1 the whole state, beyond from a zero start) and its sum of
  // delta.
  float *mine = p.pool + s.slot * row;
  if (LOCAL) {
    if (q.k == 0) {
      load_state(mine);
      store_carry(q.v0, 0);
    } else {
#pragma unroll
      for (int n = 0; n < kStates; ++n) h[n] = 0;
    }
  } else if (q.count == 1) {
    load_state(mine);
  } else {
    const int from = q.k == 0 ? 0 : p.joined ? q.k : 1;
#pragma unroll
    for (int n = 0; n < kStates; ++n) {
      const float *w = carry(q.v0 + from);
      h[n] = pack2(w[(2 * n) * kThreads], w[(2 * n + 1) * kThreads]);
    }
#pragma unroll 4
    for (int k = 2; k <= (p.joined ? 0 : q.k); ++k) {
      const float *w = carry(q.v0 + k);
      const f2 d = pack2(w[2 * kStates * kThreads], w[(2 * kStates + 1) * kThreads]);
#pragma unroll
      for (int n = 0; n < kStates; ++n)
        h[n] = fma2(exp2_2(mul2(d, a[n])), h[n],
                    pack2(w[(2 * n) * kThreads], w[(2 * n + 1) * kThreads]));
    }
  }

  for (int j = 0; j < tiles; ++j) {
    const int at = q.at + j * kTile, stage = j & 1;
    const bool whole = at >= q.lo && at + kTile <= q.hi;
    const int nt = min(kTile, q.hi - at);
    float *sb = sbc + stage * kBC, *sc = sb + kTile * S;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      sb[tid + k * kThreads] = in_scalar<T>(&rb[k]);
      if (!LOCAL) sc[tid + k * kThreads] = in_scalar<T>(&rc[k]);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // The tile is there for all, and all are done with the one before it,
    // whose place the next one takes.
    __syncthreads();
    if (j + 1 < tiles) {
      fetch_rows(at + kTile, stage ^ 1);
      fetch_bc(at + kTile);
    }

    // Lane l prepares token t + l of a group of L for its pair of channels,
    // hands it to the pair's lanes, and ends with that token's y.
    const unsigned char *mine_raw =
        raw + stage * TENSORS * kRaw + l * Sh::kPitch + 2 * pr * (int)sizeof(T);
    auto pair_of = [&](int w, int t) {
      const unsigned char *from = mine_raw + w * kRaw + t * Sh::kPitch;
      if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const f2 *>(from);
      } else {
        const uint32_t e = *reinterpret_cast<const uint32_t *>(from);
        return pack2(__uint_as_float(e << 16), __uint_as_float(e & 0xffff0000u));
      }
    };
    auto prepare = [&](int t) {  // the group's {delta, delta x}; returns x
      const f2 x = pair_of(0, t);
      f2 d = add2(pair_of(1, t), bias);
      if (p.softplus) d = softplus2(d);
      // outside the part (x is zero there): the state stays as it is
      if (!whole && !(at + t + l >= q.lo && at + t + l < q.hi)) d = 0;
      ulonglong2 w;
      w.x = d;
      w.y = mul2(d, x);
      reinterpret_cast<ulonglong2 *>(swarp)[(t / L & 1) * kThreads + tid] = w;
      return x;
    };
    f2 xnext = prepare(0);
    for (int t = 0; t < nt; t += L) {
      __syncwarp();
      const f2 x = xnext;
      const ulonglong2 *grp = reinterpret_cast<const ulonglong2 *>(swarp) +
                              (t / L & 1) * kThreads + (tid - l);
      if (t + L < nt) xnext = prepare(t + L);
      f2 part[5];  // sums over 1, 2, 4, .. lanes that wait for their neighbours
      f2 out = 0;
#pragma unroll
      for (int u = 0; u < L; ++u) {
        const ulonglong2 w = grp[u];
        const float4 *bp = reinterpret_cast<const float4 *>(sb + (t + u) * S) + l;
        const float4 *cp = reinterpret_cast<const float4 *>(sc + (t + u) * S) + l;
        if (LOCAL) sum = add2(sum, w.x);
        f2 o[2] = {0, 0};
#pragma unroll
        for (int n = 0; n < kStates; n += 4) {
          const float4 b4 = bp[L * n / 4];
          float4 c4;
          if (!LOCAL) c4 = cp[L * n / 4];
          const float b[4] = {b4.x, b4.y, b4.z, b4.w}, c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[n + i] = fma2(exp2_2(mul2(w.x, a[n + i])), h[n + i], mul2(w.y, both(b[i])));
            if (!LOCAL) o[i & 1] = fma2(both(c[i]), h[n + i], o[i & 1]);
          }
        }
        if (!LOCAL) {
          // neighbours exchange: of two tokens (pairs, fours, ..) the lane
          // whose bit is set keeps the second, the other the first
          f2 s2 = add2(o[0], o[1]);
          int m = 1, lev = 0;
#pragma unroll
          for (int bits = u; bits & 1; bits >>= 1, m *= 2, ++lev) {
            const bool up = l & m;
            const float2 give = unpack2(up ? part[lev] : s2);
            s2 = add2(up ? s2 : part[lev], pack2(__shfl_xor_sync(~0u, give.x, m),
                                                 __shfl_xor_sync(~0u, give.y, m)));
          }
          part[lev] = s2;
          out = s2;
        }
      }
      if (!LOCAL) {
        out = fma2(skip, x, out);
        if (gate) out = mul2(out, silu2(pair_of(2, t)));
        const float2 r = unpack2(out);
        const int tt = at + t + l;
        if (tt >= q.lo && tt < q.hi) {
          T *to = row_at(y, tt, p.ys);
          if (VEC) {
            if (2 * pr < nch) store_pair<T>(to, r);
          } else {
            if (2 * pr < nch) to[0] = out_scalar<T>(r.x);
            if (2 * pr + 1 < nch) to[1] = out_scalar<T>(r.y);
          }
        }
      }
    }
    if (!LOCAL && p.seg.ckpt_slots) {
      const int end = at + kTile;
      const int ck = end <= q.hi ? checkpoint_slot(p.seg, q.i, q.p0, end) : -1;
      if (ck >= 0) store_state(p.pool + ck * row);
    }
  }
  if (LOCAL) store_carry(q.v0 + q.k + 1, sum);
  else if (q.hi == s.len) store_state(mine);
}

// Joins the parts of each segment: carry slot k, which holds the end of part
// k - 1 from a zero start, becomes the state that part k starts from.  One
// thread per two states (blockIdx.y: which of a thread's); the loads of 16
// parts are under way at a time.
template <int S>
__global__ void __launch_bounds__(kThreads) scan_join_kernel(const ScanParams p, int nblk) {
  constexpr int L = S / kStates, kChans = 2 * kThreads / L, kAhead = 16;
  begin_after_stream();
  const int i = blockIdx.x / nblk, blk = blockIdx.x % nblk, n = blockIdx.y, tid = threadIdx.x;
  SegLoc s;
  if (!locate_segment(p.seg, i, &s) || s.len == 0) return;
  const int count = part_count(s.len, (int)(first_position(p.seg, i) & (kTile - 1)), p.part);
  if (count <= 2) return;
  const int per = p.C_ / p.G, bpg = nblk / p.G, g = blk / bpg;
  const int c0 = g * per + (blk % bpg) * kChans;
  const int nch = min(kChans, (g + 1) * per - c0);
  const int l = tid % L, pr = tid / L, st = 4 * (l + L * (n / 4)) + n % 4;
  const long long ca = c0 + min(2 * pr, nch - 1), cb = c0 + min(2 * pr + 1, nch - 1);
  const f2 a = pack2(exponent_scale(p.A[ca * S + st]), exponent_scale(p.A[cb * S + st]));

  const long long step = (long long)nblk * kCarry * kThreads;
  float *w = p.ws + (s.begin / p.part + p.spare * i + 1LL) * step +
             (long long)blk * kCarry * kThreads + tid;  // carry slot 1
  f2 h = pack2(w[(2 * n) * kThreads], w[(2 * n + 1) * kThreads]);
  for (int k = 2; k < count; k += kAhead) {
    f2 v[kAhead], d[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (k + u < count) {
        const float *from = w + (u + 1) * step;
        v[u] = pack2(from[(2 * n) * kThreads], from[(2 * n + 1) * kThreads]);
        d[u] = pack2(from[2 * kStates * kThreads], from[(2 * kStates + 1) * kThreads]);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      w += step;
      if (k + u < count) {
        h = fma2(exp2_2(mul2(d[u], a)), h, v[u]);
        const float2 o = unpack2(h);
        w[(2 * n) * kThreads] = o.x;
        w[(2 * n + 1) * kThreads] = o.y;
      }
    }
  }
}

template <typename T, int S, bool LOCAL>
constexpr size_t smem_bytes() {
  return 2 * (LOCAL ? 2 : 3) * (size_t)(kTile * Shape<T, S>::kPitch) +
         2 * (LOCAL ? 1 : 2) * kTile * S * sizeof(float) + 2 * kThreads * sizeof(float4);
}

int blocks_of_row(int C, int S, int G) {
  const int chans = 2 * kThreads / (S / kStates);
  return G * ((C / G + chans - 1) / chans);
}

// Tokens of a part, 0 to walk segments whole.  The same for both types, and for
// lengths that only the device knows.  (Figures: 4096 channels with 16 states,
// bf16, whose five blocks an SM of the second launch the shares are made for;
// fp32 has three.)
int part_tokens(int N, int B, int C, int S, int G) {
  const long long nblk = blocks_of_row(C, S, G), room = 152LL * blocks_of(2, S, false);
  if (2LL * B * nblk > 0x7fffffffLL) return 0;
  // An equal share of the work for two waves of blocks: a batch that fills the
  // machine by itself is not cut, a long segment beside short ones is (8192
  // tokens in one prompt: 266 us; 274 in one wave or in three).
  long long part = ((long long)N * nblk + 2 * room - 1) / (2 * room);
  // With three blocks an SM before any cut, not below twice the mean length: a
  // cut costs the first launch, and gains only what blocks longer than others
  // waste at the end (32 prompts of 512 tokens: 336 us whole, 452 at the share; 40
  // of 1 to 900: 435 and 566; 37 of 0 to 2414, 16384 tokens in all: 428 and 422,
  // and 604 whole).  With fewer blocks the longest prompt would last longer
  // than the rest (12 of 1 to 3000: 521 us at the share, 709 with this rule).
  const long long twice = (2LL * N + B - 1) / B;
  if (B * nblk >= 3 * 152 && part < twice) part = twice;
  part = (part + kTile - 1) / kTile * kTile;
  // A part walks its tokens and then the parts before it, at about the same
  // time each, so parts below sqrt(N) tokens gain nothing; and 32 tokens are
  // what a part's start costs (333 tokens of 500 channels with 64 states: 37 us
  // in parts of 128 tokens, 19 in parts of 32).
  while (part < 32 || part * part < N) part += kTile;
  if (part >= N) return 0;
  while (((long long)N / part + 2LL * B) * nblk > 0x7fffffffLL) part *= 2;
  return (int)part;
}

// Floats of the table of at most `parts` parts at the start of the workspace.
size_t table_floats(size_t parts) { return (2 * (1 + parts) + 63) / 64 * 64; }

template <typename T, int S, bool VEC, bool LOCAL>
cudaError_t launch_pass(const ScanParams &p, int nblk, int parts, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<T, S, LOCAL>();
  auto *kernel = scan_prefill_kernel<T, S, VEC, LOCAL>;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)((long long)nblk * parts));
  return launch_after(kernel, grid, dim3(kThreads), smem, st, p, nblk);
}

template <typename T, int S, bool VEC>
cudaError_t launch_prefill_v(ScanParams p, cudaStream_t st) {
  const int nblk = blocks_of_row(p.C_, S, p.G);
  p.part = p.ws ? part_tokens(p.seg.N, p.seg.B, p.C_, S, p.G) : 0;
  if (!p.part) return launch_pass<T, S, VEC, false>(p, nblk, p.seg.B, st);
  p.spare = p.seg.ckpt_slots && p.seg.start_pos ? 2 : 1;
  const int parts = p.seg.N / p.part + p.spare * p.seg.B;
  p.joined = p.seg.N / p.part > 16 * p.seg.B;
  int local = parts;
  cudaError_t e = cudaSuccess;
  p.table = nullptr;
  // The order of the parts is worth its launch where the blocks' tokens come to
  // some 50 us (16384 tokens in 37 prompts: 428 us with it, 505 without).
  if (p.seg.B > 1 && (long long)p.seg.N * nblk >= 100000) {
    p.table = reinterpret_cast<int2 *>(p.ws);
    local = parts - p.seg.B;
    e = launch_after(scan_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p, parts, local);
  }
  p.ws += table_floats(parts);
  if (e == cudaSuccess && local > 0) e = launch_pass<T, S, VEC, true>(p, nblk, local, st);
  if (e == cudaSuccess && p.joined)
    e = launch_after(scan_join_kernel<S>, dim3((unsigned)((long long)nblk * p.seg.B), kStates),
                     dim3(kThreads), 0, st, p, nblk);
  return e != cudaSuccess ? e : launch_pass<T, S, VEC, false>(p, nblk, parts, st);
}

template <typename T, int S>
cudaError_t launch_prefill_s(const ScanParams &p, cudaStream_t st) {
  constexpr int V = InVec<T>::kElems;
  uintptr_t bits = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.dt) |
                   reinterpret_cast<uintptr_t>(p.z) | reinterpret_cast<uintptr_t>(p.y);
  bits |= (uintptr_t)(p.xs | p.dts | p.ys | p.zs);
  const bool vec = (bits & 15) == 0 && (p.C_ / p.G) % V == 0;
  return vec ? launch_prefill_v<T, S, true>(p, st) : launch_prefill_v<T, S, false>(p, st);
}

template <typename T>
cudaError_t launch_prefill_t(const ScanParams &p, cudaStream_t st) {
  switch (p.S) {
    case 16: return launch_prefill_s<T, 16>(p, st);
    case 32: return launch_prefill_s<T, 32>(p, st);
    case 64: return launch_prefill_s<T, 64>(p, st);
    default: return launch_prefill_s<T, 128>(p, st);
  }
}

}  // namespace

cudaError_t launch_scan_prefill(const ScanParams &p, kda_dtype dt, cudaStream_t s) {
  return dt == KDA_F32 ? launch_prefill_t<float>(p, s) : launch_prefill_t<__nv_bfloat16>(p, s);
}

long long scan_prefill_blocks(int B, int C, int S, int G) {
  return (long long)B * blocks_of_row(C, S, G);
}

bool scan_splits(int N, int B, int C, int S, int G) { return part_tokens(N, B, C, S, G) > 0; }

// A smaller batch may need more than a larger one (5000 tokens of 25 blocks
// across: 47 carry slots in 19 prompts, 80 in 18), and a server has one
// workspace for all of them.  So this bounds the need of every batch up to
// these sizes: part_tokens' least parts, 32 tokens, an equal share for two
// waves and sqrt(N), allow at most the three counts below, which grow with N.
size_t scan_workspace_floats(int N, int B, int C, int S, int G) {
  const long long nblk = blocks_of_row(C, S, G), room = 152LL * blocks_of(2, S, false);
  if (B * nblk > 0x7fffffffLL) return 0;  // refused by the call
  // one or two segments that give every SM three blocks stay whole
  if (N <= 32 || (B <= 2 && nblk >= 3 * 152)) return 0;
  long long parts = std::min<long long>(N / 32, 2 * room / nblk);
  parts = std::min(parts, (long long)std::sqrt((double)N));
  const long long slots = std::min(parts + 2LL * B, 0x7fffffffLL / nblk);
  return table_floats(slots) + (size_t)(slots * nblk) * kCarry * kThreads;
}

}  // namespace kda
