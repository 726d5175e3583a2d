// Public calls of the state space layers: argument validation on the host,
// then launches on the caller's stream.  Nothing is allocated here.
#include "kda_ssm.cuh"

namespace {

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ECUDA; }
bool dtype_ok(int dt) { return dt == KDA_F32 || dt == KDA_BF16; }
size_t elem(int dt) { return dt == KDA_F32 ? 4 : 2; }
constexpr int kMaxSeqs = 65535;
constexpr int kMaxTokens = 0x7fff0000;  // tiles may pass the last token
constexpr int kMaxChannels = 1 << 20;
constexpr int64_t kMaxStride = 0x7fffffff;  // bytes

// A token view: pointer, element alignment, row stride.
int check_view(const void *p, int64_t stride, int row, int dt) {
  if (!p) return KDA_EINVAL;
  if (!aligned(p, elem(dt))) return KDA_EALIGN;
  if (stride < row || stride > kMaxStride / (int64_t)elem(dt)) return KDA_ESHAPE;
  return KDA_OK;
}
int check_param(const void *p, bool needed) {
  if (!p) return needed ? KDA_EINVAL : KDA_OK;
  return aligned(p, 16) ? KDA_OK : KDA_EALIGN;
}

int check_batch(int dt, int32_t B, int32_t N, int32_t D) {
  if (!dtype_ok(dt)) return KDA_EDTYPE;
  if (B < 0 || N < 0) return KDA_EINVAL;
  if (B > kMaxSeqs || D < 1 || D > kMaxChannels || N > kMaxTokens) return KDA_ESHAPE;
  return KDA_OK;
}

// The slot tables: KDA_OK also for a batch without segments.
int check_tables(const int32_t *cu, bool step, int32_t B, int32_t N, const int32_t *slots,
                 const int32_t *ckpt, int32_t max_ckpt, int32_t every, int grain) {
  if (every < 0 || max_ckpt < 0 || every % grain != 0) return KDA_EINVAL;
  if (every > 0 && max_ckpt > 0 && !ckpt) return KDA_EINVAL;
  if (B == 0) return KDA_OK;
  if (!slots || (!cu && !step)) return KDA_EINVAL;
  if (!cu && N != B) return KDA_EINVAL;  // one token a row
  if (!aligned(cu, 4) || !aligned(slots, 4) || !aligned(ckpt, 4)) return KDA_EALIGN;
  return KDA_OK;
}

int conv_impl(const kda_conv_tokens *t, kda_conv_pool *pool, const int32_t *slots,
              const int32_t *ckpt, int32_t max_ckpt, int32_t every, const int32_t *start,
              const int32_t *commit, bool step, kda_stream_t stream) {
  if (!pool || !pool->base || !t) return KDA_EINVAL;
  if (!aligned(pool->base, 16)) return KDA_EALIGN;
  int st = check_batch(t->dtype, t->num_seqs, t->num_tokens, t->channels);
  if (st) return st;
  if (pool->dtype != t->dtype) return KDA_EDTYPE;
  if (t->width < 2 || t->width > 4 || pool->num_slots < 1) return KDA_ESHAPE;
  if (pool->channels != t->channels || pool->width != t->width) return KDA_ESHAPE;
  if ((st = check_tables(t->cu_seqlens, step, t->num_seqs, t->num_tokens, slots, ckpt, max_ckpt,
                         every, 1)))
    return st;
  if (!aligned(start, 4) || !aligned(commit, 4)) return KDA_EALIGN;
  if (t->num_seqs == 0 || t->num_tokens == 0) return KDA_OK;
  if ((st = check_view(t->x, t->x_stride, t->channels, t->dtype))) return st;
  if ((st = check_view(t->y, t->y_stride, t->channels, t->dtype))) return st;
  if (t->x == t->y) return KDA_EINVAL;
  if ((st = check_param(t->weight, true))) return st;
  if ((st = check_param(t->bias, false))) return st;
  if (kda::device_refused()) return KDA_EDEVICE;
  kda::ConvParams p = {};
  p.seg.err = kda::error_word();
  if (!p.seg.err) return KDA_ECUDA;
  p.seg.cu = t->cu_seqlens;
  p.seg.slots = slots;
  p.seg.commit = commit;
  p.seg.ckpt_slots = every > 0 && max_ckpt > 0 ? ckpt : nullptr;
  p.seg.start_pos = start;
  p.seg.B = t->num_seqs;
  p.seg.N = t->num_tokens;
  p.seg.P = pool->num_slots;
  p.seg.max_ckpt = max_ckpt;
  p.seg.ckpt_every = every;
  const int64_t es = (int64_t)elem(t->dtype);
  p.x = t->x;
  p.weight = t->weight;
  p.bias = t->bias;
  p.y = t->y;
  p.pool = pool->base;
  p.xs = (int)(t->x_stride * es);
  p.ys = (int)(t->y_stride * es);
  p.D = t->channels;
  p.W = t->width;
  p.silu = t->silu != 0;
  return cuda_status(kda::launch_conv(p, t->dtype, step, reinterpret_cast<cudaStream_t>(stream)));
}

bool state_ok(int s) { return s == 16 || s == 32 || s == 64 || s == 128; }

int scan_impl(const kda_scan_tokens *t, kda_scan_pool *pool, const int32_t *slots,
              const int32_t *ckpt, int32_t max_ckpt, int32_t every, const int32_t *start,
              const int32_t *commit, void *ws, size_t ws_bytes, bool step, kda_stream_t stream) {
  if (!pool || !pool->base || !t) return KDA_EINVAL;
  if (!aligned(pool->base, 16)) return KDA_EALIGN;
  int st = check_batch(t->dtype, t->num_seqs, t->num_tokens, t->channels);
  if (st) return st;
  if (!state_ok(t->state) || pool->num_slots < 1) return KDA_ESHAPE;
  if (t->groups < 1 || t->channels % t->groups != 0) return KDA_ESHAPE;
  if (pool->channels != t->channels || pool->state != t->state) return KDA_ESHAPE;
  if ((st = check_tables(t->cu_seqlens, step, t->num_seqs, t->num_tokens, slots, ckpt, max_ckpt,
                         every, 16)))
    return st;
  if (!aligned(start, 4) || !aligned(commit, 4)) return KDA_EALIGN;
  if (t->num_seqs == 0 || t->num_tokens == 0) return KDA_OK;
  const int bc = t->groups * t->state;
  if ((st = check_view(t->x, t->x_stride, t->channels, t->dtype))) return st;
  if ((st = check_view(t->dt, t->dt_stride, t->channels, t->dtype))) return st;
  if (t->z && (st = check_view(t->z, t->z_stride, t->channels, t->dtype))) return st;
  if ((st = check_view(t->B, t->b_stride, bc, t->dtype))) return st;
  if ((st = check_view(t->C, t->c_stride, bc, t->dtype))) return st;
  if ((st = check_view(t->y, t->y_stride, t->channels, t->dtype))) return st;
  if (t->y == t->x || t->y == t->dt || t->y == t->z) return KDA_EINVAL;
  if ((st = check_param(t->A, true))) return st;
  if ((st = check_param(t->D, false))) return st;
  if ((st = check_param(t->dt_bias, false))) return st;
  if (!step && kda::scan_prefill_blocks(t->num_seqs, t->channels, t->state, t->groups) > 0x7fffffffLL)
    return KDA_ESHAPE;
  if (!aligned(ws, 256)) return KDA_EALIGN;
  const bool split = ws && kda::scan_splits(t->num_tokens, t->num_seqs, t->channels, t->state,
                                            t->groups);
  if (split && ws_bytes < kda::scan_workspace_floats(t->num_tokens, t->num_seqs, t->channels,
                                                     t->state, t->groups) * sizeof(float))
    return KDA_ENOSPC;
  if (kda::device_refused()) return KDA_EDEVICE;
  kda::ScanParams p = {};
  p.seg.err = kda::error_word();
  if (!p.seg.err) return KDA_ECUDA;
  p.seg.cu = t->cu_seqlens;
  p.seg.slots = slots;
  p.seg.commit = commit;
  p.seg.ckpt_slots = every > 0 && max_ckpt > 0 ? ckpt : nullptr;
  p.seg.start_pos = start;
  p.seg.B = t->num_seqs;
  p.seg.N = t->num_tokens;
  p.seg.P = pool->num_slots;
  p.seg.max_ckpt = max_ckpt;
  p.seg.ckpt_every = every;
  const int64_t es = (int64_t)elem(t->dtype);
  p.x = t->x;
  p.dt = t->dt;
  p.z = t->z;
  p.B = t->B;
  p.C = t->C;
  p.y = t->y;
  p.xs = (int)(t->x_stride * es);
  p.dts = (int)(t->dt_stride * es);
  p.zs = t->z ? (int)(t->z_stride * es) : 0;
  p.bs = (int)(t->b_stride * es);
  p.cs = (int)(t->c_stride * es);
  p.ys = (int)(t->y_stride * es);
  p.A = t->A;
  p.D = t->D;
  p.dtb = t->dt_bias;
  p.pool = pool->base;
  p.ws = split ? static_cast<float *>(ws) : nullptr;
  p.C_ = t->channels;
  p.S = t->state;
  p.G = t->groups;
  p.softplus = t->dt_softplus != 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(step ? kda::launch_scan_step(p, t->dtype, s)
                          : kda::launch_scan_prefill(p, t->dtype, s));
}

// The arrays and the layout of a move's staging area; the chunks of all
// arrays must fit the grid.
int check_arrays(const kda_slot_array *a, int32_t n, kda::MoveParams *p) {
  if (n < 0 || n > kda::kMaxSlotArrays || (n > 0 && !a)) return KDA_EINVAL;
  long long off = 0, chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (!a[i].base) return KDA_EINVAL;
    if (!aligned(a[i].base, 16)) return KDA_EALIGN;
    if (a[i].slot_bytes < 4 || a[i].slot_bytes % 4 != 0 || a[i].slot_bytes >> 40)
      return KDA_ESHAPE;
    p->base[i] = static_cast<unsigned char *>(a[i].base);
    p->bytes[i] = (long long)a[i].slot_bytes;
    p->ws_off[i] = off;
    p->first[i] = (int)chunks;
    off += kda::pad16(p->bytes[i]);
    chunks += kda::move_chunks(p->bytes[i]);
    if (chunks > 0x7fffffffLL) return KDA_ESHAPE;
  }
  p->L = n;
  p->first[n] = (int)chunks;
  p->ws_bytes = off;
  return KDA_OK;
}

// Whether the bytes of n moves' staging areas can be counted.
bool staging_fits(const kda::MoveParams &p, int32_t n) {
  return n == 0 || (size_t)p.ws_bytes <= SIZE_MAX / (size_t)n;
}

}  // namespace

extern "C" {

int kda_conv_prefill(const kda_conv_tokens *tok, kda_conv_pool *pool,
                     const int32_t *state_slots, const int32_t *ckpt_slots, int32_t max_ckpt,
                     int32_t ckpt_every, const int32_t *start_pos, kda_stream_t stream) {
  return conv_impl(tok, pool, state_slots, ckpt_slots, max_ckpt, ckpt_every, start_pos, nullptr,
                   false, stream);
}

int kda_conv_step(const kda_conv_tokens *tok, kda_conv_pool *pool, const int32_t *state_slots,
                  const int32_t *commit_len, kda_stream_t stream) {
  return conv_impl(tok, pool, state_slots, nullptr, 0, 0, nullptr, commit_len, true, stream);
}

int kda_scan_prefill(const kda_scan_tokens *tok, kda_scan_pool *pool,
                     const int32_t *state_slots, const int32_t *ckpt_slots, int32_t max_ckpt,
                     int32_t ckpt_every, const int32_t *start_pos, void *workspace,
                     size_t workspace_bytes, kda_stream_t stream) {
  return scan_impl(tok, pool, state_slots, ckpt_slots, max_ckpt, ckpt_every, start_pos, nullptr,
                   workspace, workspace_bytes, false, stream);
}

size_t kda_scan_workspace_size(int32_t num_tokens, int32_t num_seqs, int32_t channels,
                               int32_t state, int32_t groups) {
  if (num_tokens < 0 || num_tokens > kMaxTokens || num_seqs < 1 || num_seqs > kMaxSeqs || channels < 1 ||
      channels > kMaxChannels || !state_ok(state) || groups < 1 || channels % groups != 0)
    return 0;
  return kda::scan_workspace_floats(num_tokens, num_seqs, channels, state, groups) *
         sizeof(float);
}

int kda_scan_step(const kda_scan_tokens *tok, kda_scan_pool *pool, const int32_t *state_slots,
                  const int32_t *commit_len, kda_stream_t stream) {
  return scan_impl(tok, pool, state_slots, nullptr, 0, 0, nullptr, commit_len, nullptr, 0, true,
                   stream);
}

size_t kda_move_workspace_size(const kda_slot_array *arrays, int32_t num_arrays, int32_t n) {
  kda::MoveParams p = {};
  if (n < 0 || check_arrays(arrays, num_arrays, &p) != KDA_OK) return 0;
  return staging_fits(p, n) ? (size_t)p.ws_bytes * (size_t)n : 0;
}

int kda_move_slots(const kda_slot_array *arrays, int32_t num_arrays, int32_t num_slots,
                   const int32_t *src, const int32_t *dst, int32_t n, void *workspace,
                   size_t workspace_bytes, kda_stream_t stream) {
  kda::MoveParams p = {};
  const int st = check_arrays(arrays, num_arrays, &p);
  if (st) return st;
  if (n < 0) return KDA_EINVAL;
  if (num_slots < 1) return KDA_ESHAPE;
  if (n == 0 || num_arrays == 0) return KDA_OK;
  if (!src || !dst) return KDA_EINVAL;
  if (!aligned(src, 4) || !aligned(dst, 4)) return KDA_EALIGN;
  if (workspace) {
    if (!aligned(workspace, 256)) return KDA_EALIGN;
    if (!staging_fits(p, n) || workspace_bytes < (size_t)p.ws_bytes * (size_t)n)
      return KDA_ENOSPC;
  }
  if (kda::device_refused()) return KDA_EDEVICE;
  p.err = kda::error_word();
  if (!p.err) return KDA_ECUDA;
  p.src = src;
  p.dst = dst;
  p.ws = static_cast<unsigned char *>(workspace);
  p.n = n;
  p.P = num_slots;
  return cuda_status(kda::launch_moves(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
