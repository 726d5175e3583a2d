// Host checks of arguments that the calls on strided token rows share.
#pragma once

#include "kda_internal.cuh"

namespace kda {

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ECUDA; }
inline bool dtype_ok(int dt) { return dt == KDA_F32 || dt == KDA_BF16; }
inline size_t elem(int dt) { return dt == KDA_F32 ? 4 : 2; }
constexpr int kMaxSeqs = 65535;
constexpr int kMaxTokens = 0x7fff0000;  // tiles may pass the last token
constexpr int kMaxChannels = 1 << 20;
constexpr int64_t kMaxStride = 0x7fffffff;  // bytes

// A token view: pointer, element alignment, row stride.
inline int check_view(const void *p, int64_t stride, int row, int dt) {
  if (!p) return KDA_EINVAL;
  if (!aligned(p, elem(dt))) return KDA_EALIGN;
  if (stride < row || stride > kMaxStride / (int64_t)elem(dt)) return KDA_ESHAPE;
  return KDA_OK;
}
inline int check_param(const void *p, bool needed) {
  if (!p) return needed ? KDA_EINVAL : KDA_OK;
  return aligned(p, 16) ? KDA_OK : KDA_EALIGN;
}

// The slot tables: KDA_OK also for a batch without segments.
inline int check_tables(const int32_t *cu, bool step, int32_t B, int32_t N, const int32_t *slots,
                        const int32_t *ckpt, int32_t max_ckpt, int32_t every, int grain) {
  if (every < 0 || max_ckpt < 0 || every % grain != 0) return KDA_EINVAL;
  if (every > 0 && max_ckpt > 0 && !ckpt) return KDA_EINVAL;
  if (B == 0) return KDA_OK;
  if (!slots || (!cu && !step)) return KDA_EINVAL;
  if (!cu && N != B) return KDA_EINVAL;  // one token a row
  if (!aligned(cu, 4) || !aligned(slots, 4) || !aligned(ckpt, 4)) return KDA_EALIGN;
  return KDA_OK;
}

}  // namespace kda
