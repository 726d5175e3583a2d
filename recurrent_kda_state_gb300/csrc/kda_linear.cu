// Linear attention with a decay for each head, token by token:
//     S = e^g S + k v^T,   o = scale S^T q
// for steps, and for prompts that the tensor cores do not take (fp32, or dims
// below 64).
//
// A warp owns 16 value channels of one (segment, head): rows of 16 states of
// S^T with d_k contiguous keys, of which a lane holds d_k / KL.  One pass over
// the state: loaded to registers before the tokens, written after the last
// kept one.  Steps are bound by those bytes (8 d_k d_v a row and head); tokens
// go through shared memory, converted to fp32 once a block.  Blocks of four
// warps, states marked to leave L2 first: 256 rows of 32 heads of 128 x 128 in
// 161 us, the copy bandwidth (without the marks 186; eight warps 178, two 199).
//
// Prompts are bound by the chain from token to token (0.1 to 0.2 us each), so long
// ones are cut into parts of 16 tokens and more: 8192 tokens of 32 heads of 128 x 128
// in fp32 1280 us, whole 2280; then by fp32 arithmetic, three packed operations a pair
// of states and token, two without q.
//
// e^g is kept as hi + lo.  A state lives through thousands of tokens when g is
// small, and the 2^-25 by which one fp32 e^g is off is the same every time:
// after n tokens the state would be n 2^-25 off.
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kTile = 16;  // tokens in shared memory

template <int DK>
struct Walk {
  static constexpr int kKL = DK >= 32 ? 8 : 4;     // lanes along the keys
  static constexpr int kRL = 32 / kKL;             // lanes along the values
  static constexpr int kR = 16 / kRL;              // values of a lane
  static constexpr int kK4 = DK / kKL / 4;         // float4s of keys of a lane
};

// Sums of acc[r] over the KL lanes of a group; the lane's sum is that of row
// (lane in group) / 2, for R = KL / 2 rows.
template <int KL, int R>
__device__ __forceinline__ float group_sum(float (&acc)[R], int kl) {
  static_assert(R == KL / 2, "rows halve with the lanes");
#pragma unroll
  for (int w = KL / 2, n = R; n > 1; w /= 2, n /= 2) {
    const bool up = kl & w;
#pragma unroll
    for (int j = 0; j < n / 2; ++j) {
      const float send = up ? acc[j] : acc[j + n / 2];
      const float keep = up ? acc[j + n / 2] : acc[j];
      acc[j] = keep + __shfl_xor_sync(0xffffffffu, send, w);
    }
  }
  return acc[0] + __shfl_xor_sync(0xffffffffu, acc[0], 1);
}

// Four consecutive values in fp32.
__device__ __forceinline__ void four(const float *p, f2 &a, f2 &b) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  a = pack2(v.x, v.y);
  b = pack2(v.z, v.w);
}
__device__ __forceinline__ void four(const __nv_bfloat16 *p, f2 &a, f2 &b) {
  const uint2 r = *reinterpret_cast<const uint2 *>(p);
  a = pack2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
  b = pack2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}

// 16 bytes of a token's row into shared memory.
template <typename T>
__device__ __forceinline__ void stage16(const T *src, T *dst, bool vec) {
  if (vec) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 16 / (int)sizeof(T); ++i) dst[i] = src[i];
  }
}

// What a block does: steps; prompts, whole segments or parts with their outputs; or
// what a part that is not its segment's last adds to the state.
enum Kind { kStep, kPrompt, kSum };

template <typename T, int DK, Kind KIND>
__global__ void __launch_bounds__(128) linear_walk_kernel(const LinearParams p) {
  using W = Walk<DK>;
  constexpr int KL = W::kKL, RL = W::kRL, R = W::kR, K4 = W::kK4, V = 16 / sizeof(T);
  constexpr int kStages = KIND == kStep ? 1 : 2;                        // the next tile is under way
  constexpr int kRun = KIND == kStep ? 1 : KIND == kPrompt && DK == 128 ? 2 : 4;  // tokens at a time
  __shared__ __align__(16) T qs[KIND == kSum ? 1 : kStages][KIND == kSum ? 1 : kTile][DK];
  __shared__ __align__(16) T ks[kStages][kTile][DK], vs[kStages][kTile][64];
  __shared__ float2 as[kStages][kTile];
  begin_after_stream();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.H, target = blockIdx.x / p.H;
  PartLoc loc = {target, 0, 1, 0};
  if (KIND != kStep && p.part_chunks) {
    if (KIND == kPrompt && blockIdx.x == 0 && blockIdx.y == 0) report_segments(p);
    loc = find_part<KIND == kPrompt>(p, target);
    if (loc.seg < 0 || loc.index >= p.max_parts) return;
  }
  const int i = loc.seg;
  SegLoc s;
  if (!locate_segment(p.seg, i, &s) || s.len == 0) return;
  const int p0 = KIND != kStep && p.seg.start_pos ? p.seg.start_pos[i] : 0;
  if (p0 < 0) {
    set_error(p.seg.err, KDA_DERR_SEGMENT);
    return;
  }
  int first = 0, end = s.len;  // the block's tokens
  if (KIND != kStep && loc.parts > 1) {
    const long long part = (long long)p.part_chunks << p.chunk_log2, skew = p0 & ((1 << p.chunk_log2) - 1);
    first = (int)max(0LL, loc.part * part - skew);
    end = (int)min((long long)s.len, (loc.part + 1) * part - skew);
  }
  const int cols = blockDim.x / 2, col0 = blockIdx.y * cols;  // values of the block
  const int kl = lane % KL, row0 = warp * 16 + lane / KL;
  const int at = (col0 + row0) * DK + 4 * kl;
  const long long head_size = (long long)p.DV * DK;

  auto stage = [&](int t0, int buf) {
    const int n = min(kTile, end - t0);
    for (int e = tid; e < n * (DK / V); e += blockDim.x) {
      const int t = e / (DK / V), c = e % (DK / V) * V, tok = s.begin + t0 + t;
      if constexpr (KIND != kSum)
        stage16(row_at(static_cast<const T *>(p.q), tok, p.qs) + h / p.rep * DK + c, &qs[buf][t][c], p.vec);
      stage16(row_at(static_cast<const T *>(p.k), tok, p.ks) + h / p.rep * DK + c, &ks[buf][t][c], p.vec);
    }
    for (int e = tid; e < n * (cols / V); e += blockDim.x) {
      const int t = e / (cols / V), c = e % (cols / V) * V;
      stage16(row_at(static_cast<const T *>(p.v), s.begin + t0 + t, p.vs) + h * p.DV + col0 + c, &vs[buf][t][c],
              p.vec);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto log_decay = [&](int t0) {
    return tid < kTile && t0 + tid < end ? row_at(p.g, s.begin + t0 + tid, p.gs)[h] : 0.0f;
  };

  f2 S[R][2 * K4];
  {
    const bool ws = KIND != kStep && loc.parts > 1;
    const float *src = (ws ? p.part_state + ((long long)loc.index * p.H + h) * head_size
                           : p.pool + ((long long)s.slot * p.H + h) * head_size) + at;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < K4; ++c) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (KIND != kSum) v = __ldcs(reinterpret_cast<const float4 *>(src + r * RL * DK + 4 * KL * c));
        S[r][2 * c] = pack2(v.x, v.y);
        S[r][2 * c + 1] = pack2(v.z, v.w);
      }
  }
  stage(first, 0);
  float g = log_decay(first);
  auto store = [&](float *base) {
    float *dst = base + at;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < K4; ++c) {
        const float2 a = unpack2(S[r][2 * c]), b = unpack2(S[r][2 * c + 1]);
        __stcs(reinterpret_cast<float4 *>(dst + r * RL * DK + 4 * KL * c), make_float4(a.x, a.y, b.x, b.y));
      }
  };
  auto store_slot = [&](int slot) { store(p.pool + ((long long)slot * p.H + h) * head_size); };
  // tokens of the segment after which the next checkpoint is due
  long long due = 0x7fffffffffffLL;
  if (KIND == kPrompt && p.seg.ckpt_slots)
    due = ((long long)p0 + first) / p.seg.ckpt_every * p.seg.ckpt_every + p.seg.ckpt_every - p0;
  long long sum_g = 0;  // of a part, by the first warp
  float nan = 0.0f;

  // One token of the tile: the state, and the products with q of the lane's keys.
  auto token = [&](int buf, int t, float (&acc)[R]) {
    const float2 a = as[buf][t];
    const f2 hi = both(a.x), lo = both(a.y);
    f2 sum[R], v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = both(in_scalar<T>(&vs[buf][t][row0 + r * RL]));
#pragma unroll
    for (int c = 0; c < K4; ++c) {
      f2 k0, k1, q0, q1;
      four(&ks[buf][t][4 * kl + 4 * KL * c], k0, k1);
      if constexpr (KIND != kSum) four(&qs[buf][t][4 * kl + 4 * KL * c], q0, q1);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        S[r][2 * c] = fma2(S[r][2 * c], hi, fma2(S[r][2 * c], lo, mul2(k0, v[r])));
        S[r][2 * c + 1] = fma2(S[r][2 * c + 1], hi, fma2(S[r][2 * c + 1], lo, mul2(k1, v[r])));
        if constexpr (KIND != kSum) {
          sum[r] = c == 0 ? mul2(S[r][0], q0) : fma2(S[r][2 * c], q0, sum[r]);
          sum[r] = fma2(S[r][2 * c + 1], q1, sum[r]);
        }
      }
    }
    if constexpr (KIND != kSum) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 u = unpack2(sum[r]);
        acc[r] = u.x + u.y;
      }
    }
  };
  auto output = [&](int tok, float (&acc)[R]) {
    const float y = group_sum<KL, R>(acc, kl);
    if ((kl & 1) == 0)
      row_at(static_cast<T *>(p.o), s.begin + tok, p.os)[h * p.DV + col0 + row0 + kl / 2 * RL] =
          out_scalar<T>(y * p.scale);
  };

  for (int t0 = first, buf = 0; t0 < end; t0 += kTile) {
    const int n = min(kTile, end - t0);
    if (tid < kTile) as[buf][tid] = decay_pair(g);
    if (KIND == kSum && warp == 0) {
      long long x = fixed_log2(g);
      if (__any_sync(0xffffffffu, g != g)) nan = __int_as_float(0x7fffffff);
#pragma unroll
      for (int m = 16; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
      sum_g = min(max(sum_g + x, -kMostFixed), kMostFixed);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (kStages > 1 && t0 + kTile < end) {
      stage(t0 + kTile, buf ^ 1);
      g = log_decay(t0 + kTile);
    }
    // runs of tokens without a state to store, kRun at a time: only the state goes
    // from one to the next, so that their sums overlap
    for (int t = 0; t < n;) {
      int stop = n;
      if (KIND == kPrompt) stop = (int)min((long long)n, due - t0);
      if (KIND != kSum && s.keep > t0 + t) stop = min(stop, s.keep - t0);
      for (; kRun > 1 && t + kRun <= stop; t += kRun) {
        float acc[kRun][R];
#pragma unroll
        for (int u = 0; u < kRun; ++u) token(buf, t + u, acc[u]);
        if constexpr (KIND != kSum) {
#pragma unroll
          for (int u = 0; u < kRun; ++u) output(t0 + t + u, acc[u]);
        }
      }
      for (; t < stop; ++t) {
        float acc[R];
        token(buf, t, acc);
        if constexpr (KIND != kSum) output(t0 + t, acc);
      }
      const int done = t0 + t;
      if (KIND == kPrompt && done == due) {
        const int c = checkpoint_slot(p.seg, i, p0, done);
        if (c >= 0) store_slot(c);
        due += p.seg.ckpt_every;
      }
      if (KIND != kSum && done == s.keep) store_slot(s.slot);
    }
    if (kStages > 1) {
      buf ^= 1;
    } else if (t0 + kTile < end) {
      __syncthreads();
      stage(t0 + kTile, 0);
      g = log_decay(t0 + kTile);
    }
  }
  if constexpr (KIND == kSum) {
    const long long place = (long long)loc.index * p.H + h;
    store(p.part_state + place * head_size);
    if (tid == 0 && blockIdx.y == 0) {
      const float2 a = decay_pair(unfixed(sum_g) * kLn2);
      p.part_decay[place] = make_float2(a.x + nan, a.y);
    }
  }
}

struct Plain {
  __device__ __forceinline__ static int plain(int e) { return 4 * e; }
};

template <typename T, int DK>
cudaError_t walk(const LinearParams &p, bool step, cudaStream_t s) {
  const int warps = p.DV < 64 ? p.DV / 16 : 4, slices = p.DV / 16 / warps;
  const dim3 block(32 * warps);
  if (step) return launch_after(linear_walk_kernel<T, DK, kStep>, dim3(p.seg.B * p.H, slices), block, 0, s, p);
  const dim3 grid((p.part_chunks ? p.max_parts : p.seg.B) * p.H, slices);
  if (p.part_chunks) {
    cudaError_t e = launch_after(linear_walk_kernel<T, DK, kSum>, dim3(p.max_cut * p.H, slices), block, 0, s, p);
    if (e == cudaSuccess) e = launch_linear_join<Plain>(p, s);
    if (e != cudaSuccess) return e;
  }
  return launch_after(linear_walk_kernel<T, DK, kPrompt>, grid, block, 0, s, p);
}
template <typename T>
cudaError_t walk(const LinearParams &p, bool step, cudaStream_t s) {
  switch (p.DK) {
    case 16: return walk<T, 16>(p, step, s);
    case 32: return walk<T, 32>(p, step, s);
    case 64: return walk<T, 64>(p, step, s);
    default: return walk<T, 128>(p, step, s);
  }
}

}  // namespace

cudaError_t launch_linear_walk(const LinearParams &p, kda_dtype dt, bool step, cudaStream_t s) {
  return dt == KDA_F32 ? walk<float>(p, step, s) : walk<__nv_bfloat16>(p, step, s);
}

}  // namespace kda
