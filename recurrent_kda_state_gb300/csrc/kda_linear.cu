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
// 166 us, 97 % of the copy bandwidth (without the marks 186; eight warps 178,
// two 199).
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

// `count` values of a token's row from global memory into fp32.
template <typename T>
__device__ __forceinline__ void stage4(const T *src, float *dst, bool vec) {
  float4 v;
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      v = *reinterpret_cast<const float4 *>(src);
    } else {
      const uint2 r = *reinterpret_cast<const uint2 *>(src);
      v = make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                      __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
    }
  } else {
    v = make_float4(in_scalar<T>(src), in_scalar<T>(src + 1), in_scalar<T>(src + 2),
                    in_scalar<T>(src + 3));
  }
  *reinterpret_cast<float4 *>(dst) = v;
}

template <typename T, int DK>
__global__ void __launch_bounds__(128) linear_walk_kernel(const LinearParams p) {
  using W = Walk<DK>;
  constexpr int KL = W::kKL, RL = W::kRL, R = W::kR, K4 = W::kK4;
  __shared__ __align__(16) float qs[kTile][DK], ks[kTile][DK], vs[kTile][64];
  __shared__ float2 as[kTile];
  begin_after_stream();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.H, i = blockIdx.x / p.H;
  SegLoc s;
  if (!locate_segment(p.seg, i, &s) || s.len == 0) return;
  const int cols = blockDim.x / 2, col0 = blockIdx.y * cols;  // values of the block
  const int kl = lane % KL, row0 = warp * 16 + lane / KL;
  const long long head_state = (long long)h * p.DV * DK, slot_state = (long long)p.H * p.DV * DK;
  const long long at = head_state + (long long)(col0 + row0) * DK + 4 * kl;

  f2 S[R][2 * K4];
  {
    const float *src = p.pool + s.slot * slot_state + at;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < K4; ++c) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(src + (long long)r * RL * DK + 4 * KL * c));
        S[r][2 * c] = pack2(v.x, v.y);
        S[r][2 * c + 1] = pack2(v.z, v.w);
      }
  }
  auto store = [&](int slot) {
    float *dst = p.pool + slot * slot_state + at;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < K4; ++c) {
        const float2 a = unpack2(S[r][2 * c]), b = unpack2(S[r][2 * c + 1]);
        __stcs(reinterpret_cast<float4 *>(dst + (long long)r * RL * DK + 4 * KL * c),
               make_float4(a.x, a.y, b.x, b.y));
      }
  };
  const long long p0 = p.seg.start_pos ? p.seg.start_pos[i] : 0;
  if (p0 < 0) {
    set_error(p.seg.err, KDA_DERR_SEGMENT);
    return;
  }
  // tokens after which the next checkpoint is due
  long long due = p.seg.ckpt_slots ? p.seg.ckpt_every - p0 % p.seg.ckpt_every : 0x7fffffffffffLL;
  const int hq = h / p.rep;
  for (int t0 = 0; t0 < s.len; t0 += kTile) {
    const int n = min(kTile, s.len - t0);
    __syncthreads();
    for (int e = tid; e < n * (DK / 4); e += blockDim.x) {
      const int t = e / (DK / 4), c = e % (DK / 4) * 4;
      stage4(row_at(static_cast<const T *>(p.q), s.begin + t0 + t, p.qs) + hq * DK + c, &qs[t][c], p.vec);
      stage4(row_at(static_cast<const T *>(p.k), s.begin + t0 + t, p.ks) + hq * DK + c, &ks[t][c], p.vec);
    }
    for (int e = tid; e < n * (cols / 4); e += blockDim.x) {
      const int t = e / (cols / 4), c = e % (cols / 4) * 4;
      stage4(row_at(static_cast<const T *>(p.v), s.begin + t0 + t, p.vs) + h * p.DV + col0 + c, &vs[t][c],
             p.vec);
    }
    if (tid < n) as[tid] = decay_pair(row_at(p.g, s.begin + t0 + tid, p.gs)[h]);
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float2 a = as[t];
      const f2 hi = both(a.x), lo = both(a.y);
      float acc[R];
      f2 sum[R];
#pragma unroll
      for (int c = 0; c < K4; ++c) {
        const float4 kv = *reinterpret_cast<const float4 *>(&ks[t][4 * kl + 4 * KL * c]);
        const float4 qv = *reinterpret_cast<const float4 *>(&qs[t][4 * kl + 4 * KL * c]);
        const f2 k0 = pack2(kv.x, kv.y), k1 = pack2(kv.z, kv.w);
        const f2 q0 = pack2(qv.x, qv.y), q1 = pack2(qv.z, qv.w);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const f2 v = both(vs[t][row0 + r * RL]);
          S[r][2 * c] = fma2(S[r][2 * c], hi, fma2(S[r][2 * c], lo, mul2(k0, v)));
          S[r][2 * c + 1] = fma2(S[r][2 * c + 1], hi, fma2(S[r][2 * c + 1], lo, mul2(k1, v)));
          sum[r] = c == 0 ? mul2(S[r][0], q0) : fma2(S[r][2 * c], q0, sum[r]);
          sum[r] = fma2(S[r][2 * c + 1], q1, sum[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 u = unpack2(sum[r]);
        acc[r] = u.x + u.y;
      }
      const float y = group_sum<KL, R>(acc, kl);
      if ((kl & 1) == 0)
        row_at(static_cast<T *>(p.o), s.begin + t0 + t, p.os)[h * p.DV + col0 + row0 + kl / 2 * RL] =
            out_scalar<T>(y * p.scale);
      const int done = t0 + t + 1;
      if (done == due) {
        const int c = checkpoint_slot(p.seg, i, p0, done);
        if (c >= 0) store(c);
        due += p.seg.ckpt_every;
      }
      if (done == s.keep) store(s.slot);
    }
  }
}

template <typename T, int DK>
cudaError_t walk(const LinearParams &p, int blocks, int warps, cudaStream_t s) {
  return launch_after(linear_walk_kernel<T, DK>, dim3(blocks, p.DV / 16 / warps), dim3(32 * warps), 0, s,
                      p);
}
template <typename T>
cudaError_t walk(const LinearParams &p, int blocks, int warps, cudaStream_t s) {
  switch (p.DK) {
    case 16: return walk<T, 16>(p, blocks, warps, s);
    case 32: return walk<T, 32>(p, blocks, warps, s);
    case 64: return walk<T, 64>(p, blocks, warps, s);
    default: return walk<T, 128>(p, blocks, warps, s);
  }
}

}  // namespace

cudaError_t launch_linear_walk(const LinearParams &p, kda_dtype dt, bool step, cudaStream_t s) {
  const int blocks = p.seg.B * p.H;
  const int warps = p.DV < 64 ? p.DV / 16 : 4;
  return dt == KDA_F32 ? walk<float>(p, blocks, warps, s) : walk<__nv_bfloat16>(p, blocks, warps, s);
}

}  // namespace kda
