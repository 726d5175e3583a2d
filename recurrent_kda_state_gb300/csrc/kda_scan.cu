// Selective scan over packed segments, the state h [D][S] of each sequence in
// its slot:
//     h[n] = exp(delta A[n]) h[n] + delta x B[n],   y = C . h + D x  (gated)
//
// A thread owns four states of one channel, S / 4 neighbouring lanes a
// channel, and walks down the segment's tokens; the sum over states is a
// butterfly over the channel's lanes.
#include "kda_ssm.cuh"

namespace kda {
namespace {

template <typename T>
__device__ __forceinline__ float4 load4(const T *p, bool vec) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      return *reinterpret_cast<const float4 *>(p);
    } else {
      const uint2 a = *reinterpret_cast<const uint2 *>(p);
      return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u),
                         __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u));
    }
  }
  return make_float4(in_scalar<T>(p), in_scalar<T>(p + 1), in_scalar<T>(p + 2),
                     in_scalar<T>(p + 3));
}

constexpr int kStepThreads = 256;

template <typename T, int S>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(const ScanParams p, bool vec) {
  constexpr int L = S / 4;  // lanes of a channel
  const int i = blockIdx.y + blockIdx.z * gridDim.y;
  if (i >= p.seg.B) return;
  SegLoc s;
  if (!locate_segment(p.seg, i, &s) || s.len == 0) return;
  const int l = threadIdx.x % L;
  const int ch = blockIdx.x * (kStepThreads / L) + threadIdx.x / L;
  const bool on = ch < p.C_;
  const int c = on ? ch : p.C_ - 1;
  const int g = c / (p.C_ / p.G);

  float4 a = *reinterpret_cast<const float4 *>(p.A + (long long)c * S + 4 * l);
  a.x *= kLog2e; a.y *= kLog2e; a.z *= kLog2e; a.w *= kLog2e;
  const float skip = p.D ? p.D[c] : 0.0f, bias = p.dtb ? p.dtb[c] : 0.0f;
  const long long row = (long long)p.C_ * S;
  float *state = p.pool + s.slot * row + (long long)c * S + 4 * l;
  float4 h = *reinterpret_cast<const float4 *>(state);
  const T *x = static_cast<const T *>(p.x) + s.begin * p.xs + c;
  const T *dt = static_cast<const T *>(p.dt) + s.begin * p.dts + c;
  const T *z = p.z ? static_cast<const T *>(p.z) + s.begin * p.zs + c : nullptr;
  const T *B = static_cast<const T *>(p.B) + s.begin * p.bs + g * S + 4 * l;
  const T *C = static_cast<const T *>(p.C) + s.begin * p.cs + g * S + 4 * l;
  T *y = static_cast<T *>(p.y) + s.begin * p.ys + c;
  const long long p0 = p.seg.start_pos ? p.seg.start_pos[i] : 0;

  for (int t = 0; t < s.len; ++t) {
    const float xt = in_scalar<T>(x + t * p.xs);
    float d = in_scalar<T>(dt + t * p.dts) + bias;
    if (p.softplus) d = softplus_f(d);
    const float4 b = load4<T>(B + t * p.bs, vec), cc = load4<T>(C + t * p.cs, vec);
    const float dx = d * xt;
    h.x = fmaf(ex2f(d * a.x), h.x, dx * b.x);
    h.y = fmaf(ex2f(d * a.y), h.y, dx * b.y);
    h.z = fmaf(ex2f(d * a.z), h.z, dx * b.z);
    h.w = fmaf(ex2f(d * a.w), h.w, dx * b.w);
    float o = fmaf(cc.x, h.x, cc.y * h.y) + fmaf(cc.z, h.z, cc.w * h.w);
#pragma unroll
    for (int m = 1; m < L; m *= 2) o += __shfl_xor_sync(~0u, o, m);
    if (on && l == 0) {
      o = fmaf(skip, xt, o);
      if (z) o *= silu_f(in_scalar<T>(z + t * p.zs));
      y[t * p.ys] = out_scalar<T>(o);
    }
    if (t + 1 == s.keep && on) *reinterpret_cast<float4 *>(state) = h;
    if (p.seg.ckpt_slots) {
      const int ck = checkpoint_slot(p.seg, i, p0, t + 1);
      if (ck >= 0 && on)
        *reinterpret_cast<float4 *>(p.pool + ck * row + (long long)c * S + 4 * l) = h;
    }
  }
}

template <typename T, int S>
cudaError_t launch_step(const ScanParams &p, cudaStream_t st) {
  const int cpb = kStepThreads / (S / 4);
  const int gz = (p.seg.B + 65534) / 65535;
  const dim3 grid((p.C_ + cpb - 1) / cpb, gz > 1 ? 65535 : p.seg.B, gz);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p.B) | reinterpret_cast<uintptr_t>(p.C) |
                         (uintptr_t)(p.bs * (long long)sizeof(T)) |
                         (uintptr_t)(p.cs * (long long)sizeof(T));
  const bool vec = (bits & (4 * sizeof(T) - 1)) == 0;
  scan_step_kernel<T, S><<<grid, kStepThreads, 0, st>>>(p, vec);
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
