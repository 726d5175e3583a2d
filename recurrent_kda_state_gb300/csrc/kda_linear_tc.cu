// Prompts of linear attention on the tensor cores (tcgen05, accumulators in
// TMEM): bf16, d_k and d_v of 64 or 128, chunks of 64 tokens.  With the log
// decays g of a chunk, G_i = g_1 + .. + g_i, and the state S [d_k][d_v] before it:
//     O  = diag(e^G) Q S + (tril(Q K^T) * e^{G_i - G_j}) V
//     S' = e^{G_C} S + K~^T V,   K~_j = e^{G_C - G_j} k_j
//
// Long segments are cut into parts that run at the same time, in three launches:
// what each part adds to the state (sum_kernel), the states before the parts
// (join_kernel), the outputs (out_kernel, which alone runs for whole segments).
//
// Precision.  Decays are summed in fp64 and kept as hi + lo, so that a token
// that forgets everything costs the later ones nothing.  K~ is split into three
// bf16, which hold 24 bits, and V is exact: states are as good as fp32 products
// and sums make them.  The masked Q K^T is split into two (2^-17).  The state
// enters Q S as bf16: an error of 2^-9 of its products, as the rounding of the
// outputs has.
//
// One block of 256 threads walks the chunks of a part, two blocks an SM, so that
// one's products run beside the other's conversions.  The [Q; K] rows are one
// operand of 128 rows: with Q alone (64 rows) an MMA takes as long.
#include "kda_linear.cuh"
#include "kda_umma.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr double kLog2eD = 1.4426950408889634;
constexpr uint32_t kAccO = 0, kAccU = 128;  // TMEM columns; Q K^T comes before U, in its place

__device__ __forceinline__ uint64_t dadd(uint64_t d, uint32_t off) { return d + (off >> 4); }

// Every thread waits for the tensor cores (bounded); they agree on the outcome.
__device__ __forceinline__ bool tc_wait(uint64_t *mbar, uint32_t &phase, int limit) {
  const bool all = __syncthreads_and(umma::mbar_wait(mbar, phase, limit)) != 0;
  if (all) phase ^= 1u;
  umma::fence_after_sync();
  return all;
}
// Publish this thread's tiles to the tensor cores and meet the issuing thread.
__device__ __forceinline__ void tiles_ready() {
  umma::fence_smem_to_async();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
}

__device__ __forceinline__ void copy_wait_but_one() {
  asm volatile("cp.async.wait_group 1;" ::: "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// ROWS = 64 rows of D channels into K/64 swizzled blocks of `block` bytes; rows
// from n on are zeros.
template <int D>
__device__ __forceinline__ void load_rows(unsigned char *sm, uint32_t block, const void *base, int tok,
                                          int stride, int channel, int n, bool vec) {
  constexpr int kChunks = D / 8;
#pragma unroll
  for (int e = 0; e < 64 * kChunks / kThreads; ++e) {
    const int idx = e * kThreads + threadIdx.x, row = idx / kChunks, c = idx % kChunks;
    unsigned char *dst = sm + (c >> 3) * block + (row >> 3) * 1024 + (row & 7) * 128 +
                         (((c & 7) ^ (row & 7)) << 4);
    const __nv_bfloat16 *src =
        row_at(static_cast<const __nv_bfloat16 *>(base), tok + (row < n ? row : 0), stride) + channel + c * 8;
    if (vec) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                   :: "r"(umma::smem_u32(dst)), "l"(src), "r"(row < n ? 16 : 0) : "memory");
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = __bfloat16_as_ushort(src[2 * i]), b = __bfloat16_as_ushort(src[2 * i + 1]);
        w[i] = row < n ? a | b << 16 : 0;
      }
      *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Eight keys times w, in three bf16 parts.
__device__ __forceinline__ void split3(uint4 k, float w, uint4 *hi, uint4 *mid, uint4 *lo) {
  const uint32_t in[4] = {k.x, k.y, k.z, k.w};
  uint32_t h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(in[i] << 16) * w, b = __uint_as_float(in[i] & 0xffff0000u) * w;
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    const float2 f = __bfloat1622float2(p);
    h[i] = *reinterpret_cast<const uint32_t *>(&p);
    umma::split_bf16x2(a - f.x, b - f.y, m[i], l[i]);
  }
  *hi = make_uint4(h[0], h[1], h[2], h[3]);
  *mid = make_uint4(m[0], m[1], m[2], m[3]);
  *lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// What a thread holds of the state: a row (value channel) and NS of its columns
// (key channels).  d_v = 64: the lanes above 63 repeat the rows and take other
// columns.
template <int DK, int DV>
struct Frag {
  static constexpr int NS = DK * DV / kThreads;
  __device__ __forceinline__ static int row(int warp, int lane) {
    return DV == 128 ? 32 * (warp & 3) + lane : 32 * (warp & 1) + lane;
  }
  __device__ __forceinline__ static int col(int warp) {
    return NS * (DV == 128 ? warp >> 2 : (warp >> 1 & 1) + 2 * (warp >> 2));
  }
};
// Float4 f of a thread in a part's state: a warp's are contiguous.
template <int NS>
__device__ __forceinline__ int frag_at(int warp, int lane, int f) {
  return (warp * (NS / 4) + f) * 32 + lane;
}

// A token's log decay in units of log 2; what is below e^-15000 forgets.
__device__ __forceinline__ double log2_decay(float g) {
  return (double)(g < -15000.0f ? -15000.0f : g) * kLog2eD;
}

// The chunk's decays g of tokens 2 lane and 2 lane + 1, summed from the first.
struct ChunkDecay {
  double g0, g1, total;
  __device__ __forceinline__ ChunkDecay(float a, float b) {
    const int lane = threadIdx.x & 31;
    const double x0 = log2_decay(a), x1 = x0 + log2_decay(b);
    double upto = x1;
#pragma unroll
    for (int w = 1; w < 32; w *= 2) {
      const double o = __shfl_up_sync(0xffffffffu, upto, w);
      if (lane >= w) upto += o;
    }
    g0 = upto - x1 + x0;
    g1 = upto;
    total = __shfl_sync(0xffffffffu, upto, 31);
  }
};
__device__ __forceinline__ float2 halves(double g) {
  const float hi = (float)g;
  return make_float2(hi, (float)(g - (double)hi));
}
__device__ __forceinline__ float2 total_decay(double log2) { return decay_pair((float)(log2 / kLog2eD)); }

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

// ------------------------------------------------------- what a part adds
template <int DK, int DV>
struct SumLay {
  static constexpr uint32_t kK = DK * 128, kV = DV * 128;
  static constexpr uint32_t K = 0, V = 2 * kK, MID = V + 2 * kV, LO = MID + kK, MISC = LO + kK;
  static constexpr uint32_t W = MISC, MBAR = W + 256, TSLOT = MBAR + 8, END = TSLOT + 8;
};

// U = sum_j e^{G_end - G_j} k_j v_j^T over a part that is not its segment's last,
// chunk by chunk from the end, so that a chunk's weights need only the decay of
// those already done; one accumulator, read once.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2) sum_kernel(const LinearParams p) {
  using Lay = SumLay<DK, DV>;
  using F = Frag<DK, DV>;
  extern __shared__ __align__(1024) unsigned char sm[];
  begin_after_stream();
  const int h = blockIdx.x % p.H, target = blockIdx.x / p.H;
  const PartLoc loc = find_part(p, target);
  if (loc.seg < 0 || loc.part + 1 >= loc.parts) return;
  SegLoc s;
  if (!locate_segment(p.seg, loc.seg, &s)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int skew = p.seg.start_pos ? p.seg.start_pos[loc.seg] & 63 : 0;
  const int q0 = loc.part * p.part_chunks, nq = p.part_chunks, hq = h / p.rep;
  const uint32_t sb = umma::smem_u32(sm);
  float *w = reinterpret_cast<float *>(sm + Lay::W);
  uint64_t *mbar = reinterpret_cast<uint64_t *>(sm + Lay::MBAR);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Lay::TSLOT);

  auto load = [&](int it) {
    if (it < nq) {
      const Chunk c(s, skew, q0 + nq - 1 - it);
      load_rows<DK>(sm + Lay::K + (it & 1) * Lay::kK, 8192, p.k, c.begin, p.ks, hq * DK, c.n, p.vec);
      load_rows<DV>(sm + Lay::V + (it & 1) * Lay::kV, 8192, p.v, c.begin, p.vs, h * DV, c.n, p.vec);
    }
    copy_commit();
  };
  double later = 0.0;
  auto weigh = [&](int it) {  // warp 0
    const Chunk c(s, skew, q0 + nq - 1 - it);
    float g[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) g[e] = 2 * lane + e < c.n ? row_at(p.g, c.begin + 2 * lane + e, p.gs)[h] : 0.0f;
    const ChunkDecay d(g[0], g[1]);
    w[2 * lane] = ex2f((float)(later + (d.total - d.g0)));
    w[2 * lane + 1] = ex2f((float)(later + (d.total - d.g1)));
    later += d.total;
  };
  load(0);
  load(1);
  if (warp == 1) umma::tmem_alloc(tslot, 128);
  if (tid == 0) umma::mbar_init(mbar, 1);
  if (warp == 0) weigh(0);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *tslot, tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  uint32_t phase = 0;
  bool ok = true;
  int it = 0;
  for (; it < nq; ++it) {
    // the chunk's rows are there, and those of the chunk before are done with
    if (it > 0) {
      copy_wait();
      if (!(ok = tc_wait(mbar, phase, p.spin_limit))) break;
      load(it + 1);
    } else {
      copy_wait_but_one();
      __syncthreads();
    }
    const uint32_t kt = Lay::K + (it & 1) * Lay::kK, vt = Lay::V + (it & 1) * Lay::kV;
    {
      constexpr int kC = DK / 32;  // 16-byte chunks of a thread
      const int j = tid >> 2, c0 = (tid & 3) * kC;
      const float wj = w[j];
#pragma unroll
      for (int e = 0; e < kC; ++e) {
        const int c = c0 + e;
        const uint32_t off = (c >> 3) * 8192 + (j >> 3) * 1024 + (j & 7) * 128 + (((c & 7) ^ (j & 7)) << 4);
        uint4 *k = reinterpret_cast<uint4 *>(sm + kt + off);
        split3(*k, wj, k, reinterpret_cast<uint4 *>(sm + Lay::MID + off),
               reinterpret_cast<uint4 *>(sm + Lay::LO + off));
      }
    }
    tiles_ready();
    if (tid == 0) {
      const uint64_t dv = umma::sdesc_sw128_mn(sb + vt, DV == 128 ? 8192 : 0);
      const uint32_t id = umma::idesc_bf16_abmn(128, DK);
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        const uint64_t dk = umma::sdesc_sw128_mn(sb + (part == 0 ? kt : part == 1 ? Lay::MID : Lay::LO), 8192);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma::mma_bf16(tmem, dadd(dv, kk * 2048), dadd(dk, kk * 2048), id, (uint32_t)(it | part | kk));
      }
      umma::commit(mbar);
    }
    if (warp == 0 && it + 1 < nq) weigh(it + 1);
  }
  if (ok) ok = tc_wait(mbar, phase, p.spin_limit);
  if (ok) {
    const long long at = (long long)target * p.H + h;
    float4 *dst = reinterpret_cast<float4 *>(p.part_state + at * DK * DV);
#pragma unroll
    for (int c = 0; c < F::NS; c += 16) {
      float v[16];
      umma::tmem_ld16(tl + F::col(warp) + c, v);
#pragma unroll
      for (int f = 0; f < 4; ++f)
        dst[frag_at<F::NS>(warp, lane, c / 4 + f)] =
            make_float4(v[4 * f], v[4 * f + 1], v[4 * f + 2], v[4 * f + 3]);
    }
    if (tid == 0) p.part_decay[at] = total_decay(later);
  } else if (tid == 0) {
    set_error(p.seg.err, KDA_DERR_TIMEOUT);
    if (!umma::mbar_wait(mbar, phase, kDrainWaitPolls)) set_error(p.seg.err, KDA_DERR_UNSAFE);
  }
  copy_wait();
  umma::fence_before_sync();
  __syncthreads();
  if (warp == 1) umma::tmem_dealloc(tmem, 128);
}

// ------------------------------------------------ states before the parts
// A thread follows four states of one (segment, head) through the parts.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) join_kernel(const LinearParams p) {
  using F = Frag<DK, DV>;
  constexpr int kState4 = DK * DV / 4, kAhead = 8;
  begin_after_stream();
  const int i = blockIdx.y, parts = segment_parts(p, i);
  if (parts < 2) return;
  const int first = parts_before(p, i);
  SegLoc s;
  if (first + parts > p.max_parts || !locate_segment(p.seg, i, &s)) return;
  const int h = blockIdx.x / (kState4 / kThreads), e = blockIdx.x % (kState4 / kThreads) * kThreads + threadIdx.x;
  const int lane = e % 32, f = e / 32 % (F::NS / 4), warp = e / 32 / (F::NS / 4);
  float4 S = *reinterpret_cast<const float4 *>(p.pool + ((long long)s.slot * p.H + h) * DK * DV +
                                               F::row(warp, lane) * DK + F::col(warp) + 4 * f);
  float4 *at = reinterpret_cast<float4 *>(p.part_state) + ((long long)first * p.H + h) * kState4 + e;
  const float2 *decay = p.part_decay + (long long)first * p.H + h;
  const long long step = (long long)p.H * kState4;
  for (int q = 0; q < parts; q += kAhead) {
    float4 add[kAhead];
    float2 a[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (q + u + 1 < parts) {
        add[u] = at[(q + u) * step];
        a[u] = decay[(long long)(q + u) * p.H];
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (q + u >= parts) break;
      at[(q + u) * step] = S;
      if (q + u + 1 < parts)
        S = make_float4(decayed(S.x, a[u], add[u].x), decayed(S.y, a[u], add[u].y),
                        decayed(S.z, a[u], add[u].z), decayed(S.w, a[u], add[u].w));
    }
  }
}

// ----------------------------------------------------------------- outputs
template <int DK, int DV>
struct OutLay {
  static constexpr uint32_t kQK = DK * 256, kV = DV * 128;
  static constexpr uint32_t kKt = DK * 128;  // a part of K~
  static constexpr uint32_t kS = DK * DV * 2 > 2 * kKt ? DK * DV * 2 : 2 * kKt;
  // The masked Q K^T: hi in Q's first block, lo in its second or behind the state.
  static constexpr uint32_t QK = 0, V = 2 * kQK, S = V + kV, P2 = S + kS;
  static constexpr uint32_t MISC = P2 + (DK == 64 ? 16384 : 0);
  static constexpr uint32_t G = MISC, W = G + 512, A = W + 256, MBAR = A + 8, TSLOT = MBAR + 8,
                            END = TSLOT + 8;
};
static_assert(2 * (OutLay<128, 128>::END + 1024) <= 228 * 1024, "two blocks an SM");

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 2) out_kernel(const LinearParams p) {
  using Lay = OutLay<DK, DV>;
  using F = Frag<DK, DV>;
  constexpr int NS = F::NS;
  extern __shared__ __align__(1024) unsigned char sm[];
  begin_after_stream();
  const int h = blockIdx.x % p.H, target = blockIdx.x / p.H;
  PartLoc loc = {target, 0, 1};
  if (p.part_chunks) {
    if (blockIdx.x == 0)  // segments that no part stands for
      for (int i = threadIdx.x; i < p.seg.B; i += kThreads) {
        const int b = p.seg.cu[i], e = p.seg.cu[i + 1];
        if (b < 0 || e < b || e > p.seg.N || (p.seg.start_pos && p.seg.start_pos[i] < 0))
          set_error(p.seg.err, KDA_DERR_SEGMENT);
      }
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
  const int skew = p0 & 63, hq = h / p.rep;
  const int chunks = (int)((skew + (long long)s.len + 63) >> 6);
  int q0 = 0, q1 = chunks;
  if (p.part_chunks) {
    q0 = loc.part * p.part_chunks;
    q1 = min(chunks, q0 + p.part_chunks);
  }
  const uint32_t sb = umma::smem_u32(sm);
  float2 *G = reinterpret_cast<float2 *>(sm + Lay::G);
  float *w = reinterpret_cast<float *>(sm + Lay::W);
  float2 *whole = reinterpret_cast<float2 *>(sm + Lay::A);
  uint64_t *mbar = reinterpret_cast<uint64_t *>(sm + Lay::MBAR);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Lay::TSLOT);

  auto load_qk = [&](int q) {
    if (q < q1) {
      const Chunk c(s, skew, q);
      unsigned char *dst = sm + Lay::QK + ((q - q0) & 1) * Lay::kQK;
      load_rows<DK>(dst, 16384, p.q, c.begin, p.qs, hq * DK, c.n, p.vec);
      load_rows<DK>(dst + 8192, 16384, p.k, c.begin, p.ks, hq * DK, c.n, p.vec);
    }
    copy_commit();
  };
  auto load_v = [&](int q) {
    if (q < q1) {
      const Chunk c(s, skew, q);
      load_rows<DV>(sm + Lay::V, 8192, p.v, c.begin, p.vs, h * DV, c.n, p.vec);
    }
    copy_commit();
  };
  auto log_decays = [&](int q, float (&g)[2]) {  // of the lane's tokens
    const Chunk c(s, skew, q);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      g[e] = q < q1 && 2 * lane + e < c.n ? row_at(p.g, c.begin + 2 * lane + e, p.gs)[h] : 0.0f;
  };
  auto weigh = [&](const float (&g)[2]) {  // one warp
    const ChunkDecay d(g[0], g[1]);
    G[2 * lane] = halves(d.g0);
    G[2 * lane + 1] = halves(d.g1);
    w[2 * lane] = ex2f((float)(d.total - d.g0));
    w[2 * lane + 1] = ex2f((float)(d.total - d.g1));
    if (lane == 0) *whole = total_decay(d.total);
  };
  load_qk(q0);
  load_v(q0);
  if (warp == 1) umma::tmem_alloc(tslot, 256);
  if (tid == 0) umma::mbar_init(mbar, 1);
  constexpr int kDecayWarp = 2;
  float g[2];
  if (warp == kDecayWarp) {
    log_decays(q0, g);
    weigh(g);
  }
  const int row = F::row(warp, lane), col = F::col(warp);
  const long long head_at = (long long)h * DK * DV + row * DK + col, slot_size = (long long)p.H * DK * DV;
  float S[NS];
  {
    const float4 *src = loc.parts > 1 ? reinterpret_cast<const float4 *>(
                                            p.part_state + ((long long)target * p.H + h) * DK * DV)
                                      : reinterpret_cast<const float4 *>(p.pool + s.slot * slot_size + head_at);
#pragma unroll
    for (int f = 0; f < NS / 4; ++f) {
      const float4 v = src[loc.parts > 1 ? frag_at<NS>(warp, lane, f) : f];
      S[4 * f] = v.x;
      S[4 * f + 1] = v.y;
      S[4 * f + 2] = v.z;
      S[4 * f + 3] = v.w;
    }
  }
  auto store = [&](int slot) {
    float4 *dst = reinterpret_cast<float4 *>(p.pool + slot * slot_size + head_at);
#pragma unroll
    for (int f = 0; f < NS / 4; ++f) dst[f] = make_float4(S[4 * f], S[4 * f + 1], S[4 * f + 2], S[4 * f + 3]);
  };
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = *tslot, tl = tmem + ((uint32_t)(quad * 32) << 16);
  uint32_t phase = 0;
  bool ok = true, owed = false;
  for (int q = q0; q < q1; ++q) {
    const Chunk c(s, skew, q);
    const uint32_t qk = Lay::QK + ((q - q0) & 1) * Lay::kQK, pl = DK == 64 ? Lay::P2 : qk + 16384;
    if (warp == kDecayWarp) log_decays(q + 1, g);
#pragma unroll
    for (int e = 0; e < NS; e += 8) {  // the state as [d_v][d_k]
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(S[e + 2 * i], S[e + 2 * i + 1]);
        b[i] = *reinterpret_cast<const uint32_t *>(&x);
      }
      *reinterpret_cast<uint4 *>(sm + Lay::S + umma::sw128_off16(row, col + e, DV)) =
          make_uint4(b[0], b[1], b[2], b[3]);
    }
    copy_wait_but_one();  // q and k of this chunk
    tiles_ready();
    if (tid == 0) {
      const uint64_t dq = umma::sdesc_sw128(sb + qk), ds = umma::sdesc_sw128(sb + Lay::S);
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
        umma::mma_bf16(tmem + kAccU, dadd(dq, off), dadd(dq, off + 8192), umma::idesc_bf16(128, 64),
                       (uint32_t)kk);
      }
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk)
        umma::mma_bf16(tmem + kAccO, dadd(dq, (kk >> 2) * 16384 + (kk & 3) * 32),
                       dadd(ds, (kk >> 2) * (DV * 128) + (kk & 3) * 32), umma::idesc_bf16(128, DV),
                       (uint32_t)kk);
      umma::commit(mbar);
    }
    owed = true;
    load_qk(q + 1);
    if (!(ok = tc_wait(mbar, phase, p.spin_limit))) break;
    owed = false;
    const float2 a = *whole;
    if (quad < 2) {  // rows of the chunk's tokens
      const int i = 32 * quad + lane;
      const float2 gi = G[i];
      float x[32];
      umma::tmem_ld32(tl + kAccU + 32 * half, x);
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int j = 32 * half + e + u;
          const float2 gj = G[j];
          x[e + u] = j <= i ? x[e + u] * ex2f((gi.x - gj.x) + (gi.y - gj.y)) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) umma::split_bf16x2(x[e + 2 * u], x[e + 2 * u + 1], hi[u], lo[u]);
        const uint32_t off = umma::sw128_off16(i, 32 * half + e, 64);
        *reinterpret_cast<uint4 *>(sm + qk + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(sm + pl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      const float eg = ex2f(gi.x + gi.y);
#pragma unroll
      for (int e = 0; e < DV / 2; e += 32) {
        const uint32_t at = tl + kAccO + half * (DV / 2) + e;
        umma::tmem_ld32(at, x);
#pragma unroll
        for (int u = 0; u < 32; ++u) x[u] *= eg;
        umma::tmem_st32(at, x);
      }
    } else {  // keys: hi in place, mid and lo where the state was
      const int t = ((quad - 2) + 2 * half) * 32 + lane, j = t >> 1;
      const float wj = w[j];
#pragma unroll
      for (int e = 0; e < DK / 16; ++e) {
        const int ch = (t & 1) * (DK / 16) + e;
        const uint32_t off = (j >> 3) * 1024 + (j & 7) * 128 + (((ch & 7) ^ (j & 7)) << 4);
        uint4 *k = reinterpret_cast<uint4 *>(sm + qk + 8192 + (ch >> 3) * 16384 + off);
        unsigned char *m = sm + Lay::S + (ch >> 3) * 8192 + off;
        split3(*k, wj, k, reinterpret_cast<uint4 *>(m), reinterpret_cast<uint4 *>(m + Lay::kKt));
      }
    }
    copy_wait_but_one();  // v of this chunk
    tiles_ready();
    if (tid == 0) {
      const uint64_t dva = umma::sdesc_sw128_mn(sb + Lay::V, DV == 128 ? 8192 : 0);
      const uint64_t dvb = umma::sdesc_sw128_mn(sb + Lay::V, 8192);
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        const uint64_t dk = part == 0 ? umma::sdesc_sw128_mn(sb + qk + 8192, 16384)
                                      : umma::sdesc_sw128_mn(sb + Lay::S + (part - 1) * Lay::kKt, 8192);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma::mma_bf16(tmem + kAccU, dadd(dva, kk * 2048), dadd(dk, kk * 2048),
                         umma::idesc_bf16_abmn(128, DK), (uint32_t)(part | kk));
      }
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint64_t dp = umma::sdesc_sw128(sb + (part ? pl : qk));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma::mma_bf16(tmem + kAccO, dadd(dp, kk * 32), dadd(dvb, kk * 2048),
                         umma::idesc_bf16_bmn(128, DV), 1u);
      }
      umma::commit(mbar);
    }
    owed = true;
    if (!(ok = tc_wait(mbar, phase, p.spin_limit))) break;
    owed = false;
    load_v(q + 1);
    if (warp == kDecayWarp) weigh(g);
#pragma unroll
    for (int e = 0; e < NS; e += 16) {
      float u[16];
      umma::tmem_ld16(tl + kAccU + col + e, u);
#pragma unroll
      for (int x = 0; x < 16; ++x) S[e + x] = decayed(S[e + x], a, u[x]);
    }
    if (p.seg.ckpt_slots) {
      const int slot = checkpoint_slot(p.seg, loc.seg, p0, c.begin - s.begin + c.n);
      if (slot >= 0) store(slot);
    }
    if (quad < 2) {
      const int i = 32 * quad + lane;
      __nv_bfloat16 *o = row_at(static_cast<__nv_bfloat16 *>(p.o), c.begin + i, p.os) + h * DV + half * (DV / 2);
#pragma unroll
      for (int e = 0; e < DV / 2; e += 16) {
        float x[16];
        umma::tmem_ld16(tl + kAccO + half * (DV / 2) + e, x);
        if (i >= c.n) continue;
        uint32_t b[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * u] * p.scale, x[2 * u + 1] * p.scale);
          b[u] = *reinterpret_cast<const uint32_t *>(&y);
        }
        if (p.o_vec) {
          *reinterpret_cast<uint4 *>(o + e) = make_uint4(b[0], b[1], b[2], b[3]);
          *reinterpret_cast<uint4 *>(o + e + 8) = make_uint4(b[4], b[5], b[6], b[7]);
        } else {
#pragma unroll
          for (int u = 0; u < 16; ++u)
            o[e + u] = __ushort_as_bfloat16((unsigned short)(b[u / 2] >> (u & 1) * 16));
        }
      }
    }
  }
  if (!ok) {
    if (tid == 0) {
      set_error(p.seg.err, KDA_DERR_TIMEOUT);
      // one more bounded chance for the tensor cores before TMEM is freed
      if (owed && !umma::mbar_wait(mbar, phase, kDrainWaitPolls)) set_error(p.seg.err, KDA_DERR_UNSAFE);
    }
  } else if (loc.part + 1 == loc.parts) {
    store(s.slot);
  }
  copy_wait();
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
  // per device, and cheap beside a launch
  cudaError_t e = allow(out_kernel<DK, DV>, out_bytes);
  if (e != cudaSuccess) return e;
  if (!p.part_chunks)
    return launch_after(out_kernel<DK, DV>, dim3(p.seg.B * p.H), dim3(kThreads), out_bytes, s, p);
  if ((e = allow(sum_kernel<DK, DV>, sum_bytes)) != cudaSuccess) return e;
  const dim3 grid(p.max_parts * p.H);
  if ((e = launch_after(sum_kernel<DK, DV>, grid, dim3(kThreads), sum_bytes, s, p)) != cudaSuccess) return e;
  if ((e = launch_after(join_kernel<DK, DV>, dim3(p.H * (DK * DV / 4 / kThreads), p.seg.B), dim3(kThreads), 0, s,
                        p)) != cudaSuccess)
    return e;
  return launch_after(out_kernel<DK, DV>, grid, dim3(kThreads), out_bytes, s, p);
}

constexpr int kBlocks = 2 * 152;  // that the GPU holds
constexpr int kMinPart = 2;       // chunks of a part
constexpr int kMaxSplitSeqs = 1024;

}  // namespace

// Parts that fill the machine once where there are few long segments; more
// segments fill it alone, and searching them costs more.
int linear_part_chunks(int N, int B, int H) {
  if (B > kMaxSplitSeqs) return 0;
  const long long pc = ((long long)N * H + 64 * kBlocks - 1) / (64 * kBlocks);
  const int part = pc < kMinPart ? kMinPart : (int)pc;
  return (long long)part * 64 < N ? part : 0;
}
int linear_max_parts(int N, int B, int H) { return N / (64 * linear_part_chunks(N, B, H)) + 2 * B; }

size_t linear_workspace_parts(int N, int B, int H) {
  if (!linear_part_chunks(N, 1, H)) return 0;
  const int b = B < kMaxSplitSeqs ? B : kMaxSplitSeqs;
  const int most = N / (64 * kMinPart), fill = kBlocks / H + 1;
  return (most < fill ? most : fill) + 2 * b;
}

cudaError_t launch_linear_tc(const LinearParams &p, cudaStream_t s) {
  if (p.DK == 128) return p.DV == 128 ? linear_tc<128, 128>(p, s) : linear_tc<128, 64>(p, s);
  return p.DV == 128 ? linear_tc<64, 128>(p, s) : linear_tc<64, 64>(p, s);
}

}  // namespace kda
