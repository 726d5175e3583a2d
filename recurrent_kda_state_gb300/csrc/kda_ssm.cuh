// Internal declarations of the state space layers' translation units: launch
// parameter blocks, device helpers and the launchers that kda_ssm_api.cu calls
// after validating the public arguments.
#pragma once

#include <type_traits>

#include "kda_internal.cuh"

namespace kda {

// Device address of the library's error word (nullptr: lookup failed), and
// whether launches on the current device are refused (kda_api.cu).
unsigned int *error_word();
bool device_refused();

// Segments of the packed batch and what becomes of their states.
struct SegParams {
  const int32_t *cu;          // [B + 1]; NULL: row i is token i
  const int32_t *slots;       // [B]
  const int32_t *commit;      // [B] or NULL (steps)
  const int32_t *ckpt_slots;  // [B][max_ckpt] or NULL (prompts)
  const int32_t *start_pos;   // [B] or NULL (prompts)
  unsigned int *err;
  int B, N, P, max_ckpt, ckpt_every;
};

struct ConvParams {
  SegParams seg;
  const void *x, *weight, *bias;
  void *y, *pool;
  int xs, ys;  // row strides in bytes
  int D, W, silu;
  int tile;  // prompts: tokens of a tile
};

struct ScanParams {
  SegParams seg;
  const void *x, *dt, *z, *B, *C;
  void *y;
  int xs, dts, zs, bs, cs, ys;  // row strides in bytes
  const float *A, *D, *dtb;
  float *pool;
  float *ws;  // prompts: carried states of split segments, or NULL
  int C_, S, G, softplus;
  int part;  // prompts: tokens of a part, 0 = segments are not split
  int spare;   // prompts: part numbers kept for a segment beyond len / part
  int joined;  // prompts: a launch of its own has joined the parts' states
  int2 *table;  // prompts: {parts, parts but the last ones}, then {segment, part}; or NULL
};

constexpr int kMaxSlotArrays = 64;
struct MoveParams {
  unsigned char *base[kMaxSlotArrays];
  long long bytes[kMaxSlotArrays];   // of a slot
  long long ws_off[kMaxSlotArrays];  // of the array in a move's staging area
  int first[kMaxSlotArrays + 1];     // first chunk of the array
  const int32_t *src, *dst;
  unsigned char *ws;
  long long ws_bytes;  // staging area of one move
  unsigned int *err;
  int L, n, P;
};

__host__ __device__ inline long long pad16(long long b) { return (b + 15) & ~15LL; }

// A segment's rows and slot, checked against the batch and the pool; false
// (and the error bit) if they are not sound.  keep: tokens that the stored
// state takes in.
struct SegLoc {
  int begin, len, slot, keep;
};
__device__ __forceinline__ bool locate_segment(const SegParams &p, int i, SegLoc *s) {
  int b = i, e = i + 1;
  if (p.cu) {
    b = p.cu[i];
    e = p.cu[i + 1];
  }
  s->slot = p.slots[i];
  if (b < 0 || e < b || e > p.N) {
    set_error(p.err, KDA_DERR_SEGMENT);
    return false;
  }
  if (s->slot < 0 || s->slot >= p.P) {
    set_error(p.err, KDA_DERR_SLOT);
    return false;
  }
  s->begin = b;
  s->len = e - b;
  s->keep = p.commit ? p.commit[i] : s->len;
  if (s->keep < 0 || s->keep > s->len) {
    set_error(p.err, KDA_DERR_ACCEPT);
    return false;
  }
  return true;
}

// Checkpoint slot for the state after `local` tokens of segment i (absolute
// position start_pos + local), or -1 if none is wanted there.
__device__ __forceinline__ int checkpoint_slot(const SegParams &p, int i, long long p0,
                                               long long local) {
  const long long pos = p0 + local;
  if (!p.ckpt_slots || local <= 0 || pos % p.ckpt_every != 0) return -1;
  const long long m = pos / p.ckpt_every - p0 / p.ckpt_every - 1;
  if (m < 0 || m >= p.max_ckpt) return -1;
  const int slot = p.ckpt_slots[(long long)i * p.max_ckpt + m];
  if (slot >= p.P) {
    set_error(p.err, KDA_DERR_SLOT);
    return -1;
  }
  return slot;
}

// Every kernel of these calls is launched as a dependent of the work before it
// on the stream: its blocks may start while that work ends, and wait here
// before they touch memory.  None lets the next launch start early by itself:
// blocks that wait beside running ones cost more than they save (16 rows of 8
// tokens of the convolution: 4.4 us a call in a graph, 3.4 without).
__device__ __forceinline__ void begin_after_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... Args>
cudaError_t launch_after(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t st, const Args &...args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// 2^x and 1/x of the special function unit (2 ulp and 1 ulp).
__device__ __forceinline__ float ex2f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcpf(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// A log2(e), -inf held at the lowest finite value: a time step of 0, such as
// that of a token which pads a tile, leaves the state, and 0 * -inf would be NaN.
__device__ __forceinline__ float exponent_scale(float a) {
  const float r = a * kLog2e;
  return r < -3.4028234e38f ? -3.4028234e38f : r;
}

// v * sigmoid(v).  Below about -87.3 the reciprocal of 1 + e^-v is flushed to
// 0, and with it values of less than 1.1e-36 in magnitude; -inf gives NaN, as
// -inf / (1 + inf) does.  log2(e) v is rounded before ex2, which costs up to
// |v| / 2 ulp.
__device__ __forceinline__ float silu_f(float v) { return v * rcpf(1.0f + ex2f(-kLog2e * v)); }

// log(1 + e^v) = max(v, 0) + log1p(u), u = e^-|v| in (0, 1], with log1p(u) / u
// a polynomial of degree 8, fitted numerically on [0, 1].  Its coefficients as
// written are within 6.4e-8 of the function (6.0e-8 low at u = 0), log1p(u) as
// evaluated in fp32 within 1.8e-7; ex2 adds its 2 ulp of u.  Relative, not only
// absolute, accuracy matters: time steps of 1e-3 and less are ordinary.  No
// division: the special function unit is what the scan needs most.
__host__ __device__ constexpr float log1p_coef(int i) {
  return i == 0   ? 0.99999994f
         : i == 1 ? -0.49999437f
         : i == 2 ? 0.33317935f
         : i == 3 ? -0.24833946f
         : i == 4 ? 0.19071309f
         : i == 5 ? -0.13590600f
         : i == 6 ? 0.077380739f
         : i == 7 ? -0.028991956f
                  : 0.0051058256f;
}
__device__ __forceinline__ float softplus_f(float v) {
  const float u = ex2f(-kLog2e * fabsf(v));
  float r = log1p_coef(8);
#pragma unroll
  for (int i = 7; i >= 0; --i) r = fmaf(r, u, log1p_coef(i));
  return fmaf(u, r, fmaxf(v, 0.0f));
}

// Packed fp32 pairs: one instruction for two values.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 exp2_2(f2 v) {
  const float2 e = unpack2(v);
  return pack2(ex2f(e.x), ex2f(e.y));
}
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }

// softplus_f and silu_f of two values.
__device__ __forceinline__ f2 softplus2(f2 v) {
  const float2 w = unpack2(v);
  const f2 u = exp2_2(mul2(pack2(fabsf(w.x), fabsf(w.y)), both(-kLog2e)));
  f2 r = both(log1p_coef(8));
#pragma unroll
  for (int i = 7; i >= 0; --i) r = fma2(r, u, both(log1p_coef(i)));
  return fma2(u, r, pack2(fmaxf(w.x, 0.0f), fmaxf(w.y, 0.0f)));
}
__device__ __forceinline__ f2 silu2(f2 v) {
  const float2 d = unpack2(add2(exp2_2(mul2(v, both(-kLog2e))), both(1.0f)));
  return mul2(v, pack2(rcpf(d.x), rcpf(d.y)));
}

template <typename T>
__device__ __forceinline__ T out_scalar(float v);
template <>
__device__ __forceinline__ float out_scalar<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 out_scalar<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Row t of a token tensor: one multiply-add, since strides are 32-bit bytes.
template <typename T>
__device__ __forceinline__ T *row_at(T *base, int t, int stride) {
  using B = typename std::conditional<std::is_const<T>::value, const char, char>::type;
  return reinterpret_cast<T *>(reinterpret_cast<B *>(base) + (long long)t * stride);
}

template <typename T>
__device__ __forceinline__ void store_pair(T *p, float2 v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float2 *>(p) = v;
  else *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}

cudaError_t launch_conv(const ConvParams &p, kda_dtype dt, bool step, cudaStream_t s);
cudaError_t launch_scan_prefill(const ScanParams &p, kda_dtype dt, cudaStream_t s);
cudaError_t launch_scan_step(const ScanParams &p, kda_dtype dt, cudaStream_t s);
cudaError_t launch_moves(const MoveParams &p, cudaStream_t s);

// Chunks of kMoveChunk bytes that a slot of `bytes` is copied in.
constexpr int kMoveChunk = 16384;
inline long long move_chunks(long long bytes) { return (bytes + kMoveChunk - 1) / kMoveChunk; }

// Blocks of the scan of B whole segments.
long long scan_prefill_blocks(int B, int C, int S, int G);
// Whether a batch is split when it has a workspace.
bool scan_splits(int N, int B, int C, int S, int G);
// Workspace floats of any split batch of at most N tokens and B segments (0:
// none is split).
size_t scan_workspace_floats(int N, int B, int C, int S, int G);

}  // namespace kda
