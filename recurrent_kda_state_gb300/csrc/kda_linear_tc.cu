// Prompts of linear attention on the tensor cores (tcgen05, accumulators in
// TMEM): bf16, d_k and d_v of 64 or 128, chunks of 64 tokens.  With the log
// decays g of a chunk, G_i = g_1 + .. + g_i, and the state S [d_k][d_v] before it:
//     O  = diag(e^G) Q S + (tril(Q K^T) * e^{G_i - G_j}) V
//     S' = e^{G_C} S + K~^T V,   K~_j = e^{G_C - G_j} k_j
//
// Long segments are cut into parts that run at the same time, in three launches:
// what each part adds to the state (sum_kernel), the states before the parts
// (linear_join_kernel), the outputs (out_kernel, which alone runs for whole segments).
//
// Precision.  Decays are summed in fixed point and kept as hi + lo, so that a token
// that forgets everything costs the later ones nothing.  K~ (or V, where it is
// narrower, with the same weights) is split into three bf16, which hold 24 bits, and
// the other is exact.  The tensor cores cut what they add in a step of 16 products, always
// downwards, a little behind the last bit of the largest, so the small parts come first,
// and sums are no longer than a chunk (12 steps; a part in one accumulator left states
// 2.6e-6 off); chunks are added in registers.  Keys and values of one sign, 2000 tokens:
// states 1.6e-6 off with the large parts first.
// The masked Q K^T and the state of Q S are split into two each: 8 bits of 24 cut off,
// the next 16 rounded to 8, so that their products are off by 2^-16 at most.
//
// One block of 256 threads walks the chunks of a part, two blocks an SM, so that
// one's products run beside the other's conversions.  An MMA of 128 x 128 x 16
// takes 64 cycles, and as long with 64 rows; reading both operands from shared
// memory is the limit for 128 x 64 x 16 (48 cycles, 32 with one of them in TMEM).
//
// A value of v that is not finite would make NaN of the earlier tokens' outputs too, by
// the zeros of the mask: it is dropped from the tile (each value is looked at once, which
// takes 3 us of 8192 tokens) and its channel's outputs and state are made NaN afterwards.
//
// 8192 tokens, 32 heads of 128 x 128, in 9 parts, 138 us (125 with the state of Q S as
// one bf16, 2^-8 of its products off, and v unchecked): 42 for what they add, 95 for the
// outputs and the rest to join them, where the bytes of both passes take 63 at the copy
// bandwidth.  No unit is busy (tensor pipe 28 %, DRAM 35 %): a chunk is a chain of
// products, conversions and barriers, and two blocks do not fill its gaps.
#include "kda_linear.cuh"
#include "kda_tma.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
// TMEM columns: outputs [d_v][token], the state in bf16 [d_v][d_k / 2], its first 8
// bits and then its next 8, and U [d_v][d_k], before which Q K^T [token][token] has its
// place, and with d_k = 128 the state's second bits.
constexpr uint32_t kAccO = 0, kState = 64, kAccU = 128;
template <int DK>
constexpr uint32_t kState2 = DK == 64 ? kState + 32 : kAccU + 64;

__device__ __forceinline__ uint64_t dadd(uint64_t d, uint32_t off) { return d + (off >> 4); }

// A warp waits for the tensor cores (bounded); its threads agree on the outcome,
// and the block's at its next barrier.
__device__ __forceinline__ bool warp_wait(uint64_t *mbar, uint32_t parity, int limit) {
  const bool ok = __all_sync(0xffffffffu, umma::mbar_wait(mbar, parity, limit)) != 0;
  umma::fence_after_sync();
  return ok;
}
// Publish this thread's tiles to the tensor cores and meet the issuing thread;
// whether every thread is `ok`.
__device__ __forceinline__ bool tiles_ready(bool ok) {
  umma::fence_smem_to_async();
  umma::fence_before_sync();
  const bool all = __syncthreads_and(ok) != 0;
  umma::fence_after_sync();
  return all;
}

// q, k and v as rows of channels, where they start on 16 bytes.
struct Maps {
  CUtensorMap q, k, v;
};
// The 64 rows of D channels from `channel` on, in swizzled blocks of 64 channels
// `block` bytes apart; what lies behind the chunk's tokens comes with them.
template <int D>
__device__ __forceinline__ void load_box(uint32_t to, uint32_t block, const CUtensorMap *map, int channel, int row,
                                         uint64_t *mbar) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    tma_load2(to + i * block, map, channel + 64 * i, row, umma::smem_u32(mbar));
}

// The tokens of chunk q of a segment (chunks end at absolute multiples of 64).
struct Chunk {
  int begin, n;
  __device__ __forceinline__ Chunk(const SegLoc &s, int skew, int q) {
    const long long b = (long long)q * 64 - skew, e = b + 64;
    const int lo = b > 0 ? (int)b : 0, hi = e < s.len ? (int)e : s.len;
    begin = s.begin + lo;
    n = hi - lo;
  }
};

// A thread's share of 64 rows of D channels in such blocks: 16 bytes of every
// kStep-th row.
template <int D, int THREADS>
struct Rows {
  static constexpr int kChunks = D / 8, kStep = THREADS / kChunks, kLoads = 64 / kStep;
  static_assert(kStep % 8 == 0, "rows of one place in the swizzle");
  int row, chunk;
  __device__ __forceinline__ explicit Rows(int t) : row(t / kChunks), chunk(t % kChunks) {}
  // Byte offset of the thread's e-th 16 bytes, and its row.
  __device__ __forceinline__ uint32_t place(int e, uint32_t block) const {
    return (chunk >> 3) * block + (row >> 3) * 1024 + (row & 7) * 128 + (((chunk & 7) ^ (row & 7)) << 4) +
           e * (kStep / 8) * 1024;
  }
  __device__ __forceinline__ int row_of(int e) const { return row + e * kStep; }
  // Rows that the tensor maps do not take, by plain loads; zeros behind the tokens.
  __device__ __forceinline__ void load(unsigned char *sm, uint32_t block, const void *base, int stride,
                                       int channel, const Chunk &c) const {
#pragma unroll 1
    for (int e = 0; e < kLoads; ++e) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (row_of(e) < c.n) {
        const unsigned short *x =
            row_at(static_cast<const unsigned short *>(base), c.begin + row_of(e), stride) + channel + chunk * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)x[2 * i] | (uint32_t)x[2 * i + 1] << 16;
      }
      *reinterpret_cast<uint4 *>(sm + place(e, block)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // Zeros in the rows from n on, of the thread's first `loads`.
  __device__ __forceinline__ void clear(unsigned char *sm, uint32_t block, int n, int loads = kLoads) const {
#pragma unroll 1
    for (int e = 0; e < loads; ++e)
      if (row_of(e) >= n) *reinterpret_cast<uint4 *>(sm + place(e, block)) = make_uint4(0, 0, 0, 0);
  }
};

__device__ __forceinline__ uint32_t round2(f2 x) {
  const float2 v = unpack2(x);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ f2 widen2(uint32_t b) {
  return pack2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}
// The first 8 bits of two values as bf16; x keeps the others.
__device__ __forceinline__ uint32_t peel(f2 &x) {
  const float2 v = unpack2(x);
  const uint32_t a = __float_as_uint(v.x), b = __float_as_uint(v.y);
  x = fma2(pack2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u)), both(-1.0f), x);
  return __byte_perm(a, b, 0x7632);
}

// Eight keys or values times w, in three bf16 parts, which hold its 24 bits.
__device__ __forceinline__ void split3(const uint4 &k, unsigned char *hi, unsigned char *mid, unsigned char *lo,
                                       float w) {
  const uint32_t in[4] = {k.x, k.y, k.z, k.w};
  uint32_t h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f2 x = mul2(widen2(in[i]), both(w));
    h[i] = peel(x);
    m[i] = peel(x);
    const float2 v = unpack2(x);
    l[i] = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
  }
  *reinterpret_cast<uint4 *>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4 *>(mid) = make_uint4(m[0], m[1], m[2], m[3]);
  *reinterpret_cast<uint4 *>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}

// Whether any of the bf16 values taken in is a NaN or an infinity, whose product with 0
// is a NaN: one instruction for two of them.
struct AllFinite {
  __nv_bfloat162 sum = __bfloat162bfloat162(__ushort_as_bfloat16(0));
  __device__ __forceinline__ void take(const uint4 &x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const __nv_bfloat162 zero = __bfloat162bfloat162(__ushort_as_bfloat16(0));
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), zero, sum);
  }
  __device__ __forceinline__ bool failed() const {
    return (*reinterpret_cast<const uint32_t *>(&sum) & 0x7fff7fffu) != 0;
  }
};
__device__ __forceinline__ bool finite(unsigned short bf16) { return (bf16 & 0x7f80) != 0x7f80; }

// Which takes the decays e^{G_C - G_j} and is split, keys or values: the narrower
// (64 heads of 128 x 64, 4096 tokens, the state of Q S as one bf16: 117 us with the keys,
// 112 with the values).
template <int DK, int DV>
constexpr bool kOfValues = DV < DK;

// What a thread holds of the state: a row (value channel: its lane of TMEM) and
// half of the columns (key channels).  With d_v = 64 the warps of lanes 64 on hold
// none.
template <int DK, int DV>
struct Frag {
  static constexpr int NS = DK / 2;  // columns
  __device__ __forceinline__ static bool any(int warp) { return DV == 128 || (warp & 3) < 2; }
  __device__ __forceinline__ static int row(int warp, int lane) { return 32 * (warp & 3) + lane; }
  __device__ __forceinline__ static int col(int warp) { return NS * (warp >> 2); }
  // The warp's place among those that hold any.
  __device__ __forceinline__ static int place(int warp) {
    return DV == 128 ? warp : (warp & 1) + 2 * (warp >> 2);
  }
  // Float4 f of a thread in a part's state: a warp's are contiguous.
  __device__ __forceinline__ static int at(int warp, int lane, int f) {
    return (place(warp) * (NS / 4) + f) * 32 + lane;
  }
  // The place of a part's e-th float4 in a state of the pool.
  __device__ __forceinline__ static int plain(int e) {
    const int w = e / 32 / (NS / 4), warp = DV == 128 ? w : (w & 1) + 4 * (w >> 1);
    return row(warp, e % 32) * DK + col(warp) + 4 * (e / 32 % (NS / 4));
  }
};

// Decays of a chunk, for a warp that has the log decays of tokens 2 lane and 2
// lane + 1 (0 behind the last token): the sums from the first token on.
struct ChunkDecay {
  long long g0, g1, total;
  float nan0, nan1, nan;  // 0, or NaN from a token on whose decay is NaN
  __device__ __forceinline__ ChunkDecay(float a, float b) {
    const int lane = threadIdx.x & 31;
    const long long x0 = fixed_log2(a), x1 = x0 + fixed_log2(b);
    long long upto = x1;
#pragma unroll
    for (int w = 1; w < 32; w *= 2) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, w);
      if (lane >= w) upto += o;
    }
    g0 = upto - x1 + x0;
    g1 = upto;
    total = __shfl_sync(0xffffffffu, upto, 31);
    nan0 = nan1 = nan = 0.0f;
    const unsigned bad = __ballot_sync(0xffffffffu, a != a || b != b);
    if (bad) {
      nan = __int_as_float(0x7fffffff);
      const int first = __ffs(bad) - 1;
      if (lane > first || (lane == first && a != a)) nan0 = nan;
      if (lane >= first) nan1 = nan;
    }
  }
};

// The log decay of the e-th of a lane's two tokens.
__device__ __forceinline__ float log_decay(const LinearParams &p, const Chunk &c, int h, int e) {
  const int t = 2 * (threadIdx.x & 31) + e;
  return t < c.n ? row_at(p.g, c.begin + t, p.gs)[h] : 0.0f;
}

// ------------------------------------------------------- what a part adds
template <int DK, int DV>
struct SumLay {
  static constexpr uint32_t kK = DK * 128, kV = DV * 128, kPart = kOfValues<DK, DV> ? kV : kK;
  static constexpr uint32_t K = 0, V = 2 * kK, MID = V + 2 * kV, LO = MID + kPart, W = LO + kPart, MBAR = W + 512,
                            TSLOT = MBAR + 24, END = TSLOT + 8;
};

// U = sum_j e^{G_end - G_j} k_j v_j^T over a part that is not its segment's last,
// chunk by chunk from the end, so that a chunk's weights need only the decay of
// those already done.  Two accumulators: one is read while the next chunk's
// products run.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2) sum_kernel(const LinearParams p, const __grid_constant__ Maps maps) {
  using Lay = SumLay<DK, DV>;
  using F = Frag<DK, DV>;
  constexpr int NS = F::NS;
  constexpr bool kOfV = kOfValues<DK, DV>;
  extern __shared__ __align__(1024) unsigned char sm[];
  begin_after_stream();
  const int h = blockIdx.x % p.H;
  const PartLoc loc = find_part<false>(p, blockIdx.x / p.H);
  if (loc.seg < 0 || loc.index >= p.max_parts) return;
  SegLoc s;
  if (!locate_segment(p.seg, loc.seg, &s)) return;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int skew = p.seg.start_pos ? p.seg.start_pos[loc.seg] & 63 : 0;
  const int nq = p.part_chunks, q1 = loc.part * nq + nq - 1;
  const uint32_t sb = umma::smem_u32(sm);
  float *w = reinterpret_cast<float *>(sm + Lay::W);
  uint64_t *mbar = reinterpret_cast<uint64_t *>(sm + Lay::MBAR);  // products, rows of the two stages
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Lay::TSLOT);
  const Rows<DK, kThreads> kr(tid);
  const Rows<DV, kThreads> vr(tid);

  constexpr int kLoadWarp = 7;
  int asked = -1;  // by the load warp
  auto load = [&](int it) {
    if (it >= nq) return;
    const Chunk c(s, skew, q1 - it);
    const uint32_t kt = Lay::K + (it & 1) * Lay::kK, vt = Lay::V + (it & 1) * Lay::kV;
    if (!p.vec) {
      kr.load(sm + kt, 8192, p.k, p.ks, h / p.rep * DK, c);
      vr.load(sm + vt, 8192, p.v, p.vs, h * DV, c);
    } else if (warp == kLoadWarp) {
      if (umma::elect_one()) {
        uint64_t *full = mbar + 1 + (it & 1);
        mbar_expect_tx(umma::smem_u32(full), Lay::kK + Lay::kV);
        load_box<DK>(sb + kt, 8192, &maps.k, h / p.rep * DK, c.begin, full);
        load_box<DV>(sb + vt, 8192, &maps.v, h * DV, c.begin, full);
      }
      asked = it;
    }
  };
  long long later = 0;
  float nan = 0.0f, g[2] = {0.0f, 0.0f};
  auto ask = [&](int it) {  // warp 0
    if (it >= nq) return;
    const Chunk c(s, skew, q1 - it);
    g[0] = log_decay(p, c, h, 0);
    g[1] = log_decay(p, c, h, 1);
  };
  auto weigh = [&](int it) {
    const ChunkDecay d(g[0], g[1]);
    float *to = w + (it & 1) * 64 + 2 * lane;
    nan += d.nan;
    to[0] = ex2f(unfixed(later + (d.total - d.g0))) + nan;
    to[1] = ex2f(unfixed(later + (d.total - d.g1))) + nan;
    later = min(max(later + d.total, -kMostFixed), kMostFixed);
  };
  if (warp == 0) ask(0);
  if (warp == kLoadWarp) {
    if (umma::elect_one()) {
      for (int i = 0; i < 3; ++i) umma::mbar_init(mbar + i, 1);
      umma::fence_smem_to_async();
    }
    __syncwarp();
  }
  load(0);
  load(1);
  if (warp == 1) umma::tmem_alloc(tslot, 256);
  if (warp == 0) {
    weigh(0);
    if (nq > 1) {
      ask(1);
      weigh(1);
      ask(2);
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *tslot, tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  bool ok = true;
  float U[NS];
#pragma unroll
  for (int e = 0; e < NS; ++e) U[e] = 0.0f;
  auto take = [&](int it) {  // the products of chunk it, which are done
    if (!F::any(warp)) return;
#pragma unroll
    for (int e = 0; e < NS; e += 32) {
      float v[32];
      umma::tmem_ld32(tl + (it & 1) * 128 + F::col(warp) + e, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) U[e + i] += v[i];
    }
  };
  int it = 0;
  for (; it < nq; ++it) {
    // the chunk's rows are there, and those of the chunk before are done with
    if (it > 0) {
      ok = warp_wait(mbar, (it - 1) & 1, p.spin_limit);
      if (ok) load(it + 1);
    }
    if (p.vec) ok = warp_wait(mbar + 1 + (it & 1), (it >> 1) & 1, p.spin_limit) && ok;
    const int n = Chunk(s, skew, q1 - it).n;
    const uint32_t kt = Lay::K + (it & 1) * Lay::kK, vt = Lay::V + (it & 1) * Lay::kV;
    if (ok) {
      if (n < 64) {
        kr.clear(sm + kt, 8192, n);
        vr.clear(sm + vt, 8192, n);
      }
      auto split = [&](const auto &r, uint32_t tile) {
#pragma unroll
        for (int e = 0; e < r.kLoads; ++e) {
          const uint32_t off = r.place(e, 8192);
          unsigned char *x = sm + tile + off;
          split3(*reinterpret_cast<const uint4 *>(x), x, sm + Lay::MID + off, sm + Lay::LO + off,
                 w[(it & 1) * 64 + r.row_of(e)]);
        }
      };
      if constexpr (kOfV) split(vr, vt);
      else split(kr, kt);
    }
    if (!(ok = tiles_ready(ok))) break;
    if (warp == 3 && umma::elect_one()) {
      const uint32_t id = umma::idesc_bf16_abmn(128, DK);
#pragma unroll
      for (int part = 2; part >= 0; --part) {
        const uint32_t its = part == 1 ? Lay::MID : Lay::LO;
        const uint64_t dk = umma::sdesc_sw128_mn(sb + (part == 0 || kOfV ? kt : its), 8192);
        const uint64_t dv = umma::sdesc_sw128_mn(sb + (part == 0 || !kOfV ? vt : its), DV == 128 ? 8192 : 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma::mma_bf16(tmem + (it & 1) * 128, dadd(dv, kk * 2048), dadd(dk, kk * 2048), id,
                         (uint32_t)(part < 2 || kk > 0));
      }
      umma::commit(mbar);
    }
    // while the products run, the weights in the place of this chunk's, which the
    // next barrier publishes
    if (warp == 0 && it + 2 < nq) {
      weigh(it + 2);
      ask(it + 3);
    }
    if (it > 0) take(it - 1);
  }
  if (ok) {
    ok = warp_wait(mbar, (nq - 1) & 1, p.spin_limit);
    if (ok) take(nq - 1);
    ok = __syncthreads_and(ok) != 0;
  }
  if (ok) {
    const long long at = (long long)loc.index * p.H + h;
    float4 *dst = reinterpret_cast<float4 *>(p.part_state + at * DK * DV);
    if (F::any(warp)) {
#pragma unroll
      for (int f = 0; f < NS / 4; ++f)
        dst[F::at(warp, lane, f)] = make_float4(U[4 * f], U[4 * f + 1], U[4 * f + 2], U[4 * f + 3]);
    }
    if (warp == 0 && lane == 0) {
      const float2 a = decay_pair(unfixed(later) * kLn2);
      p.part_decay[at] = make_float2(a.x + nan, a.y);
    }
  } else if (warp == 0 && lane == 0) {
    set_error(p.seg.err, KDA_DERR_TIMEOUT);
    // one more bounded chance for the tensor cores before TMEM is freed
    const int last = min(it, nq) - 1;
    if (last >= 0 && !umma::mbar_wait(mbar, last & 1, kDrainWaitPolls)) set_error(p.seg.err, KDA_DERR_UNSAFE);
  }
  if (!ok && warp == kLoadWarp)  // and for the loads, before shared memory is
    for (int i = max(asked - 1, 0); i <= asked; ++i)
      if (!umma::mbar_wait(mbar + 1 + (i & 1), (i >> 1) & 1, kDrainWaitPolls)) set_error(p.seg.err, KDA_DERR_UNSAFE);
  umma::fence_before_sync();
  __syncthreads();
  if (warp == 1) umma::tmem_dealloc(tmem, 256);
}

// ----------------------------------------------------------------- outputs
template <int DK, int DV>
struct OutLay {
  static constexpr bool kOfV = kOfValues<DK, DV>;
  static constexpr uint32_t kQK = DK * 256, kV = DV * 128, kPart = kOfV ? kV : DK * 128;  // kPart: of K~ or V~
  // The masked Q K^T: hi in Q's first block, lo in its second or in a place of its
  // own; the outputs come after it, half of the tokens in each.
  // K~ has its hi in the place of the keys; V, which P V needs too, stays beside V~.
  static constexpr uint32_t QK = 0, V = 2 * kQK, HI = V + kV, MID = HI + (kOfV ? kPart : 0), LO = MID + kPart,
                            P2 = LO + kPart;
  // States on their way between rows in registers and lines in memory: 4 KB a warp,
  // in the place of K~ or V~ where that is large enough.
  static constexpr uint32_t TURN = DK == 64 ? P2 + 8192 : HI, MISC = DK == 64 ? TURN + 32768 : P2;
  static constexpr uint32_t G = MISC, EG = G + 512, A = EG + 256, MBAR = A + 8, ISSUED = MBAR + 56,
                            TSLOT = ISSUED + 16, END = TSLOT + 8;
};
static_assert(2 * (OutLay<128, 128>::END + 1024) <= 228 * 1024, "two blocks an SM");

// Outputs are made as [d_v][token], so that the state, which has a value channel a
// lane, is an operand from TMEM as soon as it is rounded.  Per chunk: Q K^T and Q S;
// then the warps of lanes 0 to 63, where Q K^T has the tokens' rows, mask it, the
// others split K~ and load, all scale Q S; then P V and U, and while U runs the
// outputs leave; then the state takes U.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2) out_kernel(const LinearParams p, const __grid_constant__ Maps maps) {
  using Lay = OutLay<DK, DV>;
  using F = Frag<DK, DV>;
  constexpr int NS = F::NS;
  constexpr bool kOfV = Lay::kOfV;
  extern __shared__ __align__(1024) unsigned char sm[];
  begin_after_stream();
  const int h = blockIdx.x % p.H, target = blockIdx.x / p.H;
  PartLoc loc = {target, 0, 1, 0};
  if (p.part_chunks) {
    if (blockIdx.x == 0) report_segments(p);
    loc = find_part(p, target);
    if (loc.seg < 0) return;
  }
  SegLoc s;
  if (!locate_segment(p.seg, loc.seg, &s) || s.len == 0) return;
  const int p0 = p.seg.start_pos ? p.seg.start_pos[loc.seg] : 0;
  if (p0 < 0) {
    set_error(p.seg.err, KDA_DERR_SEGMENT);
    return;
  }
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int quad = warp & 3, half = warp >> 2, skew = p0 & 63;
  const int chunks = (int)((skew + (long long)s.len + 63) >> 6);
  const int q0 = loc.part * p.part_chunks, q1 = loc.part + 1 == loc.parts ? chunks : q0 + p.part_chunks;
  const uint32_t sb = umma::smem_u32(sm);
  float *G = reinterpret_cast<float *>(sm + Lay::G);  // -G_j: 64 hi, 64 lo
  float *eg = reinterpret_cast<float *>(sm + Lay::EG);
  float2 *whole = reinterpret_cast<float2 *>(sm + Lay::A);
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + Lay::MBAR);  // Q K^T, Q S, P V, U
  uint64_t *full = bar + 4;                                      // q and k (two stages), v
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Lay::TSLOT);
  int *bad_v = reinterpret_cast<int *>(sm + Lay::TSLOT + 4);  // the last chunk with such a value in v
  const bool tokens = quad < 2;                        // the warps of the tokens' rows
  const int t2 = ((quad & 1) + 2 * half) * 32 + lane;  // thread among the others
  const Rows<DK, 128> kr(t2);
  const Rows<DV, 128> vr(t2);

  constexpr int kLoadWarp = 7;
  // chunks whose products of q, U and P V, loads of q and k, loads of v were issued last
  int *issued = reinterpret_cast<int *>(sm + Lay::ISSUED);
  auto load_qk = [&](int q) {
    if (q >= q1) return;
    const Chunk c(s, skew, q);
    const int at = q - q0;
    const uint32_t to = Lay::QK + (at & 1) * Lay::kQK;
    if (!p.vec) {
      if (tokens) return;
      kr.load(sm + to, 16384, p.q, p.qs, h / p.rep * DK, c);
      kr.load(sm + to + 8192, 16384, p.k, p.ks, h / p.rep * DK, c);
    } else if (warp == kLoadWarp) {
      if (umma::elect_one()) {
        mbar_expect_tx(umma::smem_u32(full + (at & 1)), Lay::kQK);
        load_box<DK>(sb + to, 16384, &maps.q, h / p.rep * DK, c.begin, full + (at & 1));
        load_box<DK>(sb + to + 8192, 16384, &maps.k, h / p.rep * DK, c.begin, full + (at & 1));
        issued[2] = at;
      }
    }
  };
  auto load_v = [&](int q) {
    if (q >= q1) return;
    const Chunk c(s, skew, q);
    if (!p.vec) {
      if (!tokens) vr.load(sm + Lay::V, 8192, p.v, p.vs, h * DV, c);
    } else if (warp == kLoadWarp) {
      if (umma::elect_one()) {
        mbar_expect_tx(umma::smem_u32(full + 2), Lay::kV);
        load_box<DV>(sb + Lay::V, 8192, &maps.v, h * DV, c.begin, full + 2);
        issued[3] = q - q0;
      }
    }
  };
  // The decays of the next chunk: one warp asks for them at the start of a chunk,
  // sums and publishes them when the chunk's own are done with.
  constexpr int kDecayWarp = 4;
  float g[2] = {0.0f, 0.0f};
  auto ask = [&](int q) {
    if (q >= q1) return;
    const Chunk c(s, skew, q);
    g[0] = log_decay(p, c, h, 0);
    g[1] = log_decay(p, c, h, 1);
  };
  auto weigh = [&]() {
    const ChunkDecay d(g[0], g[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long x = e ? d.g1 : d.g0;
      const float hi = __ll2float_rn(-x), nan = e ? d.nan1 : d.nan0;
      G[2 * lane + e] = hi * kUnit + nan;
      G[64 + 2 * lane + e] = unfixed(-x - __float2ll_rn(hi));
      eg[2 * lane + e] = ex2f(unfixed(x)) + nan;
    }
    if (lane == 0) {
      const float2 a = decay_pair(unfixed(d.total) * kLn2);
      *whole = make_float2(a.x + d.nan, a.y);
    }
  };
  if (warp == kDecayWarp) ask(q0);
  if (warp == kLoadWarp) {
    if (umma::elect_one()) {
      for (int i = 0; i < 7; ++i) umma::mbar_init(bar + i, 1);
      for (int i = 0; i < 4; ++i) issued[i] = -1;
      *bad_v = -1;
      umma::fence_smem_to_async();
    }
    __syncwarp();
  }
  load_qk(q0);
  load_v(q0);
  if (warp == 1) umma::tmem_alloc(tslot, 256);
  const int col = F::col(warp);
  f2 S[NS / 2];
  // A state's rows of 32 floats between memory (lines of 128 bytes, four an
  // instruction) and registers (a row a lane).
  unsigned char *turn = sm + Lay::TURN + F::place(warp) * 4096;
  auto line = [&](int r, int c) { return reinterpret_cast<float4 *>(turn + r * 128 + ((c ^ (r & 7)) << 4)); };
  auto head_at = [&](int slot) {
    return p.pool + ((long long)slot * p.H + h) * DK * DV + (32 * quad + lane / 8) * DK + col + lane % 8 * 4;
  };
  auto store = [&](int slot) {
    if (!F::any(warp)) return;
    float *to = head_at(slot);
#pragma unroll
    for (int e = 0; e < NS; e += 32) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float2 x = unpack2(S[e / 2 + 2 * c]), y = unpack2(S[e / 2 + 2 * c + 1]);
        *line(lane, c) = make_float4(x.x, x.y, y.x, y.y);
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4 *>(to + 4 * j * DK + e) = *line(4 * j + lane / 8, lane % 8);
      __syncwarp();
    }
  };
  if (F::any(warp) && loc.parts > 1) {
    const float4 *src = reinterpret_cast<const float4 *>(p.part_state + ((long long)target * p.H + h) * DK * DV);
#pragma unroll
    for (int f = 0; f < NS / 4; ++f) {
      const float4 v = src[F::at(warp, lane, f)];
      S[2 * f] = pack2(v.x, v.y);
      S[2 * f + 1] = pack2(v.z, v.w);
    }
  } else if (F::any(warp)) {
    const float *from = head_at(s.slot);
#pragma unroll
    for (int e = 0; e < NS; e += 32) {
      float4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const float4 *>(from + 4 * j * DK + e);
#pragma unroll
      for (int j = 0; j < 8; ++j) *line(4 * j + lane / 8, lane % 8) = v[j];
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float4 x = *line(lane, c);
        S[e / 2 + 2 * c] = pack2(x.x, x.y);
        S[e / 2 + 2 * c + 1] = pack2(x.z, x.w);
      }
      __syncwarp();
    }
  }
  if (warp == kDecayWarp) weigh();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *tslot, tl = tmem + ((uint32_t)(quad * 32) << 16);
  auto tile = [&]() {  // the state in bf16, in two
    if (!F::any(warp)) return;
#pragma unroll
    for (int e = 0; e < NS / 2; e += 16) {
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        f2 x = S[e + i];
        hi[i] = peel(x);
        lo[i] = round2(x);
      }
      umma::tmem_st(tl + kState + col / 2 + e, hi);
      umma::tmem_st(tl + kState2<DK> + col / 2 + e, lo);
    }
  };
  // The two warps of a quarter of the lanes meet.
  auto meet = [&]() {
    umma::fence_before_sync();
    asm volatile("bar.sync %0, 64;" ::"r"(3 + quad) : "memory");
    umma::fence_after_sync();
  };
  auto bad_at = [&](int token, int channel) {
    return !finite(row_at(static_cast<const unsigned short *>(p.v), token, p.vs)[h * DV + channel]);
  };
  tile();
  bool ok = true;
  for (int q = q0; q < q1; ++q) {
    const Chunk c(s, skew, q);
    const uint32_t par = (q - q0) & 1, qk = Lay::QK + par * Lay::kQK, pl = DK == 64 ? Lay::P2 : qk + 16384;
    // q and k of this chunk, for those who use them
    if (p.vec && (!tokens || warp == kDecayWarp))
      ok = warp_wait(full + par, ((q - q0) >> 1) & 1, p.spin_limit) && ok;
    if (!(ok = tiles_ready(ok))) break;
    if (warp == kDecayWarp) ask(q + 1);
    if (warp == kDecayWarp && umma::elect_one()) {
      const uint64_t dq = umma::sdesc_sw128(sb + qk);
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
        umma::mma_bf16(tmem + kAccU, dadd(dq, off), dadd(dq, off + 8192), umma::idesc_bf16(128, 64),
                       (uint32_t)kk);
      }
      umma::commit(bar);
#pragma unroll
      for (int part = 1; part >= 0; --part) {
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk)
          umma::mma_bf16_ts(tmem + kAccO, tmem + (part ? kState2<DK> : kState) + kk * 8,
                            dadd(dq, (kk >> 2) * 16384 + (kk & 3) * 32), umma::idesc_bf16(128, 64),
                            (uint32_t)(part < 1 || kk > 0));
      }
      umma::commit(bar + 1);
      issued[0] = q - q0;
    }
    load_qk(q + 1);
    const float2 a = *whole;
    ok = warp_wait(bar, par, p.spin_limit);
    if (p.vec && kOfV && (!tokens || warp == kDecayWarp)) ok = warp_wait(full + 2, par, p.spin_limit) && ok;
    // The last kLoads-th of them by kDecayWarp.
    using Split = Rows<kOfV ? DV : DK, 128>;
    constexpr uint32_t kBlock = kOfV ? 8192 : 16384;
    unsigned char *x = sm + (kOfV ? Lay::V : qk + 8192);
    auto split = [&](const Split &r, int e, AllFinite &check) {
      const int j = r.row_of(e);
      const uint32_t at = r.place(e, 8192);
      unsigned char *in = x + r.place(e, kBlock), *m = sm + Lay::MID + at;
      const uint4 v = *reinterpret_cast<const uint4 *>(in);
      if (kOfV) check.take(v);
      split3(v, kOfV ? sm + Lay::HI + at : in, m, m + Lay::kPart,
             ex2f((G[j] - G[63]) + (G[64 + j] - G[127])));
    };
    // P V would multiply a NaN or an infinity of v with the zeros of earlier tokens too:
    // such a value leaves the tile, and NaN is put where it belongs afterwards.
    auto drop = [&](const Rows<DV, 128> &r, int from, int to) {
#pragma unroll 1
      for (int e = from; e < to; ++e) {
        unsigned short *v = reinterpret_cast<unsigned short *>(sm + Lay::V + r.place(e, 8192));
#pragma unroll 1
        for (int u = 0; u < 8; ++u)
          if (!finite(v[u])) v[u] = 0;
      }
      *bad_v = q - q0;
    };
    if (!tokens && ok) {
      const Split r(t2);
      if (c.n < 64) {
        r.clear(x, kBlock, c.n, r.kLoads - 1);
        if (kOfV) kr.clear(sm + qk + 8192, 16384, c.n);
      }
      AllFinite check;
#pragma unroll 2
      for (int e = 0; e < r.kLoads - 1; ++e) split(r, e, check);
      if (kOfV && check.failed()) drop(vr, 0, vr.kLoads - 1);
    }
    if (warp == kDecayWarp && ok) {
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const Split r(32 * e + lane);
        const int last = r.kLoads - 1;
        if (r.row_of(last) >= c.n) *reinterpret_cast<uint4 *>(x + r.place(last, kBlock)) = make_uint4(0, 0, 0, 0);
        AllFinite check;
        split(r, last, check);
        if (kOfV && check.failed()) drop(Rows<DV, 128>(32 * e + lane), last, last + 1);
      }
    }
    ok = warp_wait(bar + 1, par, p.spin_limit) && ok;
    if (tokens && ok) {
      const int i = 32 * quad + lane;
      if (warp != kDecayWarp) {  // whose part is zero, and skipped
        const float ih = -G[i], il = -G[64 + i];
#pragma unroll 1
        for (int e = 0; e < 32; e += 16) {
          float x[16];
          umma::tmem_ld16(tl + kAccU + 32 * half + e, x);
#pragma unroll
          for (int v = 0; v < 16; v += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int u = 0; u < 8; u += 2) {
              const int j = 32 * half + e + v + u;
              const float2 jh = *reinterpret_cast<const float2 *>(G + j);
              const float2 jl = *reinterpret_cast<const float2 *>(G + 64 + j);
              const f2 d = add2(add2(both(ih), pack2(jh.x, jh.y)), add2(both(il), pack2(jl.x, jl.y)));
              float2 y = unpack2(mul2(exp2_2(d), pack2(x[v + u], x[v + u + 1])));
              y.x = j <= i ? y.x : 0.0f;
              y.y = j + 1 <= i ? y.y : 0.0f;
              f2 z = pack2(y.x, y.y);
              hi[u / 2] = peel(z);
              lo[u / 2] = round2(z);
            }
            const uint32_t off = umma::sw128_off16(i, 32 * half + e + v, 64);
            *reinterpret_cast<uint4 *>(sm + qk + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(sm + pl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      }
    }
    if (ok && F::any(warp)) {  // Q S of 32 tokens, each with its decay
#pragma unroll 1
      for (int e = 32 * half; e < 32 * half + 32; e += 16) {
        float x[16];
        umma::tmem_ld16(tl + kAccO + e, x);
        uint32_t b[16];
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
          const float2 d = *reinterpret_cast<const float2 *>(eg + e + u);
          const float2 v = unpack2(mul2(pack2(x[u], x[u + 1]), pack2(d.x, d.y)));
          b[u] = __float_as_uint(v.x);
          b[u + 1] = __float_as_uint(v.y);
        }
        umma::tmem_st(tl + kAccO + e, b);
      }
    }
    if (!kOfV && !tokens) {  // v of this chunk
      if (p.vec) ok = warp_wait(full + 2, par, p.spin_limit) && ok;
      if (ok) {
        if (c.n < 64) vr.clear(sm + Lay::V, 8192, c.n);
        AllFinite check;
#pragma unroll
        for (int e = 0; e < vr.kLoads; ++e)
          check.take(*reinterpret_cast<const uint4 *>(sm + Lay::V + vr.place(e, 8192)));
        if (check.failed()) drop(vr, 0, vr.kLoads);
      }
    }
    if (!(ok = tiles_ready(ok))) break;
    if (warp == 3 && umma::elect_one()) {
      const uint64_t dv = umma::sdesc_sw128_mn(sb + Lay::V, DV == 128 ? 8192 : 0);
#pragma unroll
      for (int part = 1; part >= 0; --part) {
        const uint64_t dp = umma::sdesc_sw128(sb + (part ? pl : qk));
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
          umma::mma_bf16(tmem + kAccO, dadd(dv, kk * 2048), dadd(dp, kk * 32), umma::idesc_bf16_amn(128, 64), 1u);
#pragma unroll
        for (int kk = 2; kk < 4; ++kk)  // the later half of the tokens, for its own alone
          umma::mma_bf16(tmem + kAccO + 32, dadd(dv, kk * 2048), dadd(dp, 4096 + kk * 32),
                         umma::idesc_bf16_amn(128, 32), 1u);
      }
      umma::commit(bar + 2);
#pragma unroll
      for (int part = 2; part >= 0; --part) {
        const uint32_t its = part == 0 ? Lay::HI : part == 1 ? Lay::MID : Lay::LO;
        const uint64_t dk = kOfV || part == 0 ? umma::sdesc_sw128_mn(sb + qk + 8192, 16384)
                                              : umma::sdesc_sw128_mn(sb + its, 8192);
        const uint64_t dw = kOfV ? umma::sdesc_sw128_mn(sb + its, DV == 128 ? 8192 : 0) : dv;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma::mma_bf16(tmem + kAccU, dadd(dw, kk * 2048), dadd(dk, kk * 2048),
                         umma::idesc_bf16_abmn(128, DK), (uint32_t)(part < 2 || kk > 0));
      }
      umma::commit(bar + 3);
      issued[1] = q - q0;
    }
    if (warp == kDecayWarp) weigh();
    ok = warp_wait(bar + 2, par, p.spin_limit);
    // the outputs of 32 tokens, gathered by the four warps that have their channels
    // (16 bytes at a time in places swizzled by the token)
    unsigned char *stage = sm + (half ? pl : qk);
    if (ok && F::any(warp)) {
#pragma unroll
      for (int e = 0; e < 32; e += 16) {
        float x[16];
        umma::tmem_ld_rows16(tl + (e << 16) + kAccO + 32 * half, x);
        uint32_t b[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) b[u] = round2(mul2(pack2(x[2 * u], x[2 * u + 1]), both(p.scale)));
        const int tok = 8 * (lane >> 4) + (lane & 7), chunk = 4 * quad + e / 8 + ((lane >> 3) & 1);
        const uint32_t to = umma::smem_u32(stage) + tok * (DV * 2) + ((chunk ^ (tok & 7)) << 4);
        umma::stmatrix4_trans(to, b[0], b[1], b[2], b[3]);
        umma::stmatrix4_trans(to + 16 * (DV * 2), b[4], b[5], b[6], b[7]);
      }
    }
    asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
    if (ok) {
      constexpr int kLanes = DV / 8, kStep = 128 / kLanes;  // threads of a row, rows at a time
      const int t = quad * 32 + lane, at = t % kLanes * 8;
      int i = t / kLanes;
      auto row = [&](int r) {
        return row_at(static_cast<__nv_bfloat16 *>(p.o), c.begin + 32 * half + r, p.os) + h * DV + at;
      };
      auto staged = [&](int r) {
        return reinterpret_cast<const __nv_bfloat16 *>(stage + r * (DV * 2) + ((t % kLanes ^ (r & 7)) << 4));
      };
      if (*bad_v == q - q0) {  // NaN from the first such value of a channel on
        unsigned hit = 0;
        int j = 0;
#pragma unroll 1
        for (; i < 32 && 32 * half + i < c.n; i += kStep) {
#pragma unroll 1
          for (; j <= 32 * half + i; ++j)
#pragma unroll 1
            for (int u = 0; u < 8; ++u)
              if (bad_at(c.begin + j, at + u)) hit |= 1u << u;
#pragma unroll 1
          for (int u = 0; u < 8; ++u) row(i)[u] = hit >> u & 1 ? __ushort_as_bfloat16(0x7fff) : staged(i)[u];
        }
      } else {
        __nv_bfloat16 *o = row(i);
#pragma unroll
        for (int e = 0; e < 32 / kStep; ++e) {
          if (32 * half + i < c.n) {
            const __nv_bfloat16 *from = staged(i);
            if (p.o_vec) {
              *reinterpret_cast<uint4 *>(o) = *reinterpret_cast<const uint4 *>(from);
            } else {
#pragma unroll 1
              for (int u = 0; u < 8; ++u) o[u] = from[u];
            }
          }
          i += kStep;
          o = row_at(o, kStep, p.os);
        }
      }
    }
    ok = warp_wait(bar + 3, par, p.spin_limit) && ok;
    if (ok) {
      load_v(q + 1);
      if (F::any(warp)) {
        const f2 ah = both(a.x), al = both(a.y);
#pragma unroll
        for (int e = 0; e < NS; e += 16) {
          float u[16];
          umma::tmem_ld16(tl + kAccU + col + e, u);
#pragma unroll
          for (int x = 0; x < 16; x += 2)
            S[(e + x) / 2] = fma2(S[(e + x) / 2], ah, fma2(S[(e + x) / 2], al, pack2(u[x], u[x + 1])));
        }
        if (!kOfV && *bad_v == q - q0) {  // V~ keeps such values, V has lost them
          bool hit = false;
#pragma unroll 1
          for (int j = 0; j < c.n; ++j) hit = hit || bad_at(c.begin + j, F::row(warp, lane));
          if (hit) {
#pragma unroll
            for (int e = 0; e < NS / 2; ++e) S[e] = both(__int_as_float(0x7fffffff));
          }
        }
      }
    }
    // the state's second bits go where the other warp of these lanes reads U
    if (DK == 128) meet();
    if (ok) {
      tile();
      if (p.seg.ckpt_slots) {  // positions fit 32 bits without a sign
        const unsigned every = p.seg.ckpt_every, pos = p0 + (c.begin - s.begin) + c.n;
        const unsigned m = pos / every - p0 / every - 1;
        if (pos % every == 0 && m < (unsigned)p.seg.max_ckpt) {
          const int slot = p.seg.ckpt_slots[(long long)loc.seg * p.seg.max_ckpt + m];
          if (slot >= p.seg.P) set_error(p.seg.err, KDA_DERR_SLOT);
          else if (slot >= 0) store(slot);
        }
      }
    }
  }
  ok = __syncthreads_and(ok) != 0;
  if (!ok) {
    if (tid == 0) {
      set_error(p.seg.err, KDA_DERR_TIMEOUT);
      // one more bounded chance for the tensor cores before TMEM is freed
      for (int i = 0; i < 4; ++i) {
        const int last = issued[i / 2];
        if (last >= 0 && !umma::mbar_wait(bar + i, last & 1, kDrainWaitPolls))
          set_error(p.seg.err, KDA_DERR_UNSAFE);
      }
      // and for the loads, before shared memory is
      for (int i = max(issued[2] - 1, 0); i <= issued[2]; ++i)
        if (!umma::mbar_wait(full + (i & 1), (i >> 1) & 1, kDrainWaitPolls)) set_error(p.seg.err, KDA_DERR_UNSAFE);
      if (issued[3] >= 0 && !umma::mbar_wait(full + 2, issued[3] & 1, kDrainWaitPolls))
        set_error(p.seg.err, KDA_DERR_UNSAFE);
    }
  } else if (q1 == chunks) {
    store(s.slot);
  }
  umma::fence_before_sync();
  __syncthreads();
  if (warp == 1) umma::tmem_dealloc(tmem, 256);
}

template <typename K>
cudaError_t allow(K *kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK, int DV>
cudaError_t linear_tc(const LinearParams &p, cudaStream_t s) {
  constexpr size_t sum_bytes = SumLay<DK, DV>::END, out_bytes = OutLay<DK, DV>::END;
  Maps maps = {};
  cudaError_t e = cudaSuccess;
  if (p.vec) {
    const int qk = p.H / p.rep * DK;
    e = rows_map(&maps.q, p.q, p.seg.N, qk, p.qs);
    if (e == cudaSuccess) e = rows_map(&maps.k, p.k, p.seg.N, qk, p.ks);
    if (e == cudaSuccess) e = rows_map(&maps.v, p.v, p.seg.N, p.H * DV, p.vs);
  }
  // per device, and cheap beside a launch
  if (e == cudaSuccess) e = allow(out_kernel<DK, DV>, out_bytes);
  if (e != cudaSuccess) return e;
  if (!p.part_chunks)
    return launch_after(out_kernel<DK, DV>, dim3(p.seg.B * p.H), dim3(kThreads), out_bytes, s, p, maps);
  if ((e = allow(sum_kernel<DK, DV>, sum_bytes)) != cudaSuccess) return e;
  e = launch_after(sum_kernel<DK, DV>, dim3(p.max_cut * p.H), dim3(kThreads), sum_bytes, s, p, maps);
  if (e == cudaSuccess) e = launch_linear_join<Frag<DK, DV>>(p, s);
  if (e != cudaSuccess) return e;
  return launch_after(out_kernel<DK, DV>, dim3(p.max_parts * p.H), dim3(kThreads), out_bytes, s, p, maps);
}

}  // namespace

cudaError_t launch_linear_tc(const LinearParams &p, cudaStream_t s) {
  if (p.DK == 128) return p.DV == 128 ? linear_tc<128, 128>(p, s) : linear_tc<128, 64>(p, s);
  return p.DV == 128 ? linear_tc<64, 128>(p, s) : linear_tc<64, 64>(p, s);
}

}  // namespace kda
