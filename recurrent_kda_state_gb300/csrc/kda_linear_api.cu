// Public calls of linear attention and of the head norms: argument validation
// on the host, then launches on the caller's stream.  Nothing is allocated here.
#include "kda_checks.cuh"
#include "kda_linear.cuh"
#include <cmath>

namespace {

using namespace kda;

bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Heads of a row: as many channels as other rows may have.
bool heads_ok(int heads, int d) { return heads >= 1 && heads <= kMaxChannels / d; }

int linear_impl(const kda_linear_tokens *t, kda_state_pool *pool, const int32_t *slots,
                const int32_t *ckpt, int32_t max_ckpt, int32_t every, const int32_t *start,
                const int32_t *commit, void *ws, size_t ws_bytes, bool step, kda_stream_t stream) {
  if (!pool || !pool->base || !t) return KDA_EINVAL;
  if (!aligned(pool->base, 16)) return KDA_EALIGN;
  if (!dtype_ok(t->dtype)) return KDA_EDTYPE;
  if (t->num_seqs < 0 || t->num_tokens < 0) return KDA_EINVAL;
  if (t->num_seqs > kMaxSeqs || t->num_tokens > kMaxTokens) return KDA_ESHAPE;
  if (!dim_ok(t->d_k) || !dim_ok(t->d_v) || pool->num_slots < 1) return KDA_ESHAPE;
  if (!heads_ok(t->num_heads, t->d_k > t->d_v ? t->d_k : t->d_v)) return KDA_ESHAPE;
  if (t->num_qk_heads < 1 || t->num_heads % t->num_qk_heads != 0) return KDA_ESHAPE;
  if (pool->num_heads != t->num_heads || pool->d_k != t->d_k || pool->d_v != t->d_v)
    return KDA_ESHAPE;
  int st = check_tables(t->cu_seqlens, step, t->num_seqs, t->num_tokens, slots, ckpt, max_ckpt,
                        every, 64);
  if (st) return st;
  if (!aligned(start, 4) || !aligned(commit, 4)) return KDA_EALIGN;
  if (t->num_seqs == 0 || t->num_tokens == 0) return KDA_OK;
  const int qk = t->num_qk_heads * t->d_k, vo = t->num_heads * t->d_v;
  if ((st = check_view(t->q, t->q_stride, qk, t->dtype))) return st;
  if ((st = check_view(t->k, t->k_stride, qk, t->dtype))) return st;
  if ((st = check_view(t->v, t->v_stride, vo, t->dtype))) return st;
  if ((st = check_view(t->o, t->o_stride, vo, t->dtype))) return st;
  if ((st = check_view(t->g, t->g_stride ? t->g_stride : t->num_heads, t->num_heads, KDA_F32)))
    return st;
  if (t->o == t->q || t->o == t->k || t->o == t->v || t->o == (const void *)t->g) return KDA_EINVAL;
  if ((long long)t->num_seqs * t->num_heads > 0x7fffffffLL) return KDA_ESHAPE;
  if (!aligned(ws, 256)) return KDA_EALIGN;
  const bool tc = !step && linear_uses_tc(t->dtype, t->d_k, t->d_v);
  const LinearCut cut = linear_cut(t->dtype, t->num_heads, t->d_k, t->d_v);
  const int part = !step && ws ? linear_part_chunks(t->num_tokens, t->num_seqs, cut) : 0;
  const int parts = part ? linear_max_parts(t->num_tokens, t->num_seqs, part, cut) : 0;
  if (ws_bytes < linear_workspace_bytes(parts, t->num_heads, t->d_k, t->d_v)) return KDA_ENOSPC;
  if ((long long)parts * t->num_heads > 0x7fffffffLL) return KDA_ESHAPE;
  if (device_refused()) return KDA_EDEVICE;
  LinearParams p = {};
  p.seg.err = error_word();
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
  p.q = t->q;
  p.k = t->k;
  p.v = t->v;
  p.o = t->o;
  p.qs = (int)(t->q_stride * es);
  p.ks = (int)(t->k_stride * es);
  p.vs = (int)(t->v_stride * es);
  p.os = (int)(t->o_stride * es);
  p.g = t->g;
  p.gs = (int)(t->g_stride * 4);
  p.H = t->num_heads;
  p.rep = t->num_heads / t->num_qk_heads;
  p.DK = t->d_k;
  p.DV = t->d_v;
  p.scale = t->scale;
  p.pool = pool->base;
  p.vec = aligned(t->q, 16) && aligned(t->k, 16) && aligned(t->v, 16) && p.qs % 16 == 0 &&
          p.ks % 16 == 0 && p.vs % 16 == 0;
  p.o_vec = aligned(t->o, 16) && p.os % 16 == 0;
  p.chunk_log2 = cut.chunk == 64 ? 6 : 4;
  p.part_chunks = part;
  p.max_parts = parts;
  p.max_cut = part ? linear_max_cut(t->num_tokens, t->num_seqs, part, cut) : 0;
  p.part_decay = part ? static_cast<float2 *>(ws) : nullptr;
  p.part_state = part ? reinterpret_cast<float *>(static_cast<unsigned char *>(ws) +
                                                  linear_decay_bytes(parts, p.H))
                      : nullptr;
  p.spin_limit = wait_limit_polls();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(tc ? launch_linear_tc(p, s) : launch_linear_walk(p, t->dtype, step, s));
}

// Outputs of a view: the input itself, or rows that start elsewhere.
int check_out(const void *x, int64_t x_stride, const void *y, int64_t y_stride) {
  return x == y && x_stride != y_stride ? KDA_EINVAL : KDA_OK;
}

}  // namespace

namespace kda {

// Two blocks of the tensor cores' kernel on an SM; of the walking one's four to
// eight, with half of 128 value channels each, whose parts may be short: a token waits
// for the one before (333 tokens x 6 heads of 64 x 32 in fp32: 28 us in parts of 64
// tokens, 15 in parts of 16, 14 of 8; 1001 tokens x 2 x 16 x 16 20, 18 and 24).
LinearCut linear_cut(int dtype, int H, int d_k, int d_v) {
  if (linear_uses_tc(dtype, d_k, d_v)) return {2 * 152, H, 64, 2};
  return {152 * (d_k == 128 ? 4 : d_k == 64 ? 6 : 8), H * (d_v > 64 ? 2 : 1), 16, 1};
}

constexpr int kMaxSplitSeqs = 1024;

// Parts of a batch of B segments, by what it would take in units of a chunk's time,
// `of_64` of the time of 64 tokens.  A segment's last part is half a part on average;
// a part costs kPart beside its chunks; parts that do not fill the machine take as long
// as one; those that are not a segment's last are gone over before, at kSum a chunk, and
// joined.  Whole, the longest segment counts, whose length is on the device alone: for
// lengths cut at random it is 1 + 1/2 + .. + 1/B times the mean (four prompts of 4096
// tokens in all, 64 heads of 128 x 64, the longest 1469, 1505, 2172, 3031: whole 100, 106,
// 143, 190 us, in parts 143, 126, 127, 115; one of 4096 alone, 32 heads of 128 x 128, 273
// and 86).  More than kMaxSplitSeqs segments fill the machine alone, and searching them
// costs more.
int linear_part_chunks(int N, int B, const LinearCut &c) {
  if (B > kMaxSplitSeqs || B < 1 || N <= c.chunk * c.least) return 0;
  const double of_64 = 64.0 / c.chunk, chunks = (double)N / c.chunk + 0.5 * B, share = (double)c.of_part / c.blocks;
  auto time = [&](double parts, double of_part) {
    const double waves = parts * share;
    return (waves <= 1.0 ? 1.0 : waves + 0.5) * of_part;
  };
  const double kPart = 1.5 * of_64, kSum = 0.5, kLaunch = of_64, kLarge = 12.0 * of_64;
  const double longest = std::fmin(chunks, (1.0 + 0.55 * std::log2(B)) * chunks / B);
  const double even = B * share * (chunks / B + kPart);
  double least = longest + kPart > even ? longest + kPart : even;
  int best = 0;
  const int most = 2 * c.room() + B;  // which the workspace is sized for
  for (int k = 2; k <= most; k += k / 16 + 1) {
    int part = (int)(chunks / k) + 1;
    if (part < c.least) part = c.least;
    const double cut = chunks / part - 0.5 * B;
    if (cut > 0.0) {
      const double t = time(cut + B, part + kPart) + time(cut, kSum * part + of_64) + kLaunch;
      if (t < least) best = part, least = t;
    }
    if (part == c.least) break;
  }
  // Better whole: but in a large batch a segment that is far longer than expected is
  // cut, which costs 6 to 10 us for two nearly empty launches where there is none (37
  // prompts of 16384 tokens, the longest 985 to 1519: 229 to 260 us whole, 238 to 270
  // so; with one of 5000: 364 and 303, of 8000: 551 and 302).
  if (!best && B > 1 && even >= kLarge) best = (int)(1.2 * std::fmax(longest, even) + 4 * of_64);
  return (long long)best * c.chunk < N ? best : 0;
}
// A segment of n tokens that begins inside a chunk touches at most n / chunk + 2 of
// them, and one more than its first part's are needed for a cut.
int linear_max_parts(int N, int B, int part, const LinearCut &c) { return N / (c.chunk * part) + 2 * B; }
int linear_max_cut(int N, int B, int part, const LinearCut &c) { return (N / c.chunk + B) / part + 1; }
// linear_part_chunks makes at most 2 room + B parts of a batch's chunks.
size_t linear_workspace_parts(int N, int B, const LinearCut &c) {
  if (N <= c.chunk * c.least) return 0;
  const int b = B < kMaxSplitSeqs ? B : kMaxSplitSeqs, most = N / (c.chunk * c.least);
  const int fill = 2 * c.room() + b;
  return (most < fill ? most : fill) + 2 * b;
}

}  // namespace kda

extern "C" {

int kda_linear_prefill(const kda_linear_tokens *tok, kda_state_pool *pool,
                       const int32_t *state_slots, const int32_t *ckpt_slots, int32_t max_ckpt,
                       int32_t ckpt_every, const int32_t *start_pos, void *workspace,
                       size_t workspace_bytes, kda_stream_t stream) {
  return linear_impl(tok, pool, state_slots, ckpt_slots, max_ckpt, ckpt_every, start_pos, nullptr,
                     workspace, workspace_bytes, false, stream);
}

size_t kda_linear_workspace_size(int32_t num_tokens, int32_t num_seqs, int32_t num_heads,
                                 int32_t d_k, int32_t d_v, kda_dtype dtype) {
  if (num_tokens < 0 || num_tokens > kMaxTokens || num_seqs < 1 || num_seqs > kMaxSeqs ||
      !dim_ok(d_k) || !dim_ok(d_v) || !heads_ok(num_heads, d_k > d_v ? d_k : d_v) ||
      !dtype_ok(dtype))
    return 0;
  return linear_workspace_bytes(
      linear_workspace_parts(num_tokens, num_seqs, linear_cut(dtype, num_heads, d_k, d_v)), num_heads,
      d_k, d_v);
}

int kda_linear_step(const kda_linear_tokens *tok, kda_state_pool *pool, const int32_t *state_slots,
                    const int32_t *commit_len, kda_stream_t stream) {
  return linear_impl(tok, pool, state_slots, nullptr, 0, 0, nullptr, commit_len, nullptr, 0, true,
                     stream);
}

int kda_qk_norm(const kda_qk_tokens *t, kda_stream_t stream) {
  if (!t) return KDA_EINVAL;
  if (!dtype_ok(t->dtype)) return KDA_EDTYPE;
  if (t->num_tokens < 0 || t->norm < KDA_NORM_NONE || t->norm > KDA_NORM_L2) return KDA_EINVAL;
  if (t->head_dim < 2 || t->head_dim > 256 || t->head_dim % 2 != 0) return KDA_ESHAPE;
  if (t->rot_dim < 0 || t->rot_dim > t->head_dim || t->rot_dim % 2 != 0) return KDA_ESHAPE;
  const int heads[2] = {t->num_q_heads, t->num_k_heads};
  if (heads[0] < 0 || heads[1] < 0) return KDA_EINVAL;
  if (t->num_tokens > kMaxTokens) return KDA_ESHAPE;
  if (heads[0] > kMaxChannels / t->head_dim || heads[1] > kMaxChannels / t->head_dim)
    return KDA_ESHAPE;
  if (t->rot_dim > 0 && t->max_pos < 1) return KDA_ESHAPE;
  if (t->num_tokens == 0 || heads[0] + heads[1] == 0) return KDA_OK;
  int st;
  QkParams p = {};
  const void *x[2] = {t->q, t->k};
  void *y[2] = {t->q_out, t->k_out};
  const void *w[2] = {t->q_weight, t->k_weight};
  const int64_t xs[2] = {t->q_stride, t->k_stride}, ys[2] = {t->q_out_stride, t->k_out_stride};
  const int64_t es = (int64_t)elem(t->dtype);
  for (int i = 0; i < 2; ++i) {
    if (!heads[i]) continue;
    const int row = heads[i] * t->head_dim;
    if ((st = check_view(x[i], xs[i], row, t->dtype))) return st;
    if ((st = check_view(y[i], ys[i], row, t->dtype))) return st;
    if ((st = check_out(x[i], xs[i], y[i], ys[i]))) return st;
    if ((st = check_param(w[i], false))) return st;
    p.x[i] = x[i];
    p.y[i] = y[i];
    p.w[i] = w[i];
    p.xs[i] = (int)(xs[i] * es);
    p.ys[i] = (int)(ys[i] * es);
    p.heads[i] = heads[i];
  }
  if (heads[0] && heads[1] && (y[0] == y[1] || y[0] == x[1] || y[1] == x[0])) return KDA_EINVAL;
  if (t->rot_dim > 0) {
    if ((st = check_param(t->cos_sin, true))) return st;
    if (!t->positions) return KDA_EINVAL;
    if (!aligned(t->positions, 4)) return KDA_EALIGN;
  }
  if (device_refused()) return KDA_EDEVICE;
  p.err = error_word();
  if (!p.err) return KDA_ECUDA;
  p.table = t->cos_sin;
  p.pos = t->positions;
  p.N = t->num_tokens;
  p.d = t->head_dim;
  p.rot = t->rot_dim;
  p.max_pos = t->max_pos;
  p.interleaved = t->interleaved != 0;
  p.norm = t->norm;
  p.eps = t->eps;
  p.q_scale = t->q_scale;
  p.share = t->norm == KDA_NORM_RMS ? 1.0f / (float)t->head_dim : 1.0f;
  return cuda_status(launch_qk_norm(p, t->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_gated_norm(const kda_gate_tokens *t, kda_stream_t stream) {
  if (!t) return KDA_EINVAL;
  if (!dtype_ok(t->dtype) || !dtype_ok(t->x_dtype)) return KDA_EDTYPE;
  if (t->num_tokens < 0) return KDA_EINVAL;
  if (t->head_dim < 1 || t->head_dim > 256 || !heads_ok(t->num_heads, t->head_dim))
    return KDA_ESHAPE;
  // a block takes one head's row at least
  if (t->num_tokens > kMaxTokens || (long long)t->num_tokens * t->num_heads > 0x7fffffffLL)
    return KDA_ESHAPE;
  if (t->num_tokens == 0) return KDA_OK;
  const int row = t->num_heads * t->head_dim;
  int st;
  if ((st = check_view(t->x, t->x_stride, row, t->x_dtype))) return st;
  if (t->gate && (st = check_view(t->gate, t->gate_stride, row, t->dtype))) return st;
  if ((st = check_view(t->y, t->y_stride, row, t->dtype))) return st;
  if ((st = check_param(t->weight, false))) return st;
  if (t->x == t->y && t->x_dtype != t->dtype) return KDA_EINVAL;
  if ((st = check_out(t->x, t->x_stride, t->y, t->y_stride))) return st;
  if (t->gate && (st = check_out(t->gate, t->gate_stride, t->y, t->y_stride))) return st;
  if (device_refused()) return KDA_EDEVICE;
  GateParams p = {};
  const int64_t es = (int64_t)elem(t->dtype);
  p.x = t->x;
  p.gate = t->gate;
  p.w = t->weight;
  p.y = t->y;
  p.xs = (int)(t->x_stride * (int64_t)elem(t->x_dtype));
  p.gs = t->gate ? (int)(t->gate_stride * es) : 0;
  p.ys = (int)(t->y_stride * es);
  p.N = t->num_tokens;
  p.H = t->num_heads;
  p.d = t->head_dim;
  p.silu = t->gate && t->silu;
  p.share = 1.0f / (float)t->head_dim;
  p.eps = t->eps;
  return cuda_status(launch_gated_norm(p, t->x_dtype, t->dtype,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
