// Copies, forks, compaction and freeing of slots over all arrays of a model
// in one call.  Memory bound: each moved byte is read once and written once.
//
// A block copies one chunk of one move; blockIdx.x runs over the chunks of
// all arrays, blockIdx.y over the moves.  Moves act as if all at once: a move
// whose src is the dst of another would read what that one wrote, so a first
// launch stages such sources in the workspace, and the second takes them from
// there.  Whether a source is one is found by a look through dst, which costs
// a block n / 256 loads and no table.
#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Whether another move writes slot s.
__device__ __forceinline__ bool written_by_other(const MoveParams &p, int s, int i) {
  bool hit = false;
  for (int j = threadIdx.x; j < p.n; j += kThreads) hit |= p.dst[j] == s && j != i;
  return __syncthreads_or(hit);
}

template <typename V>
__device__ __forceinline__ void copy_chunk(V *to, const V *from, long long n) {
  constexpr int U = kMoveChunk / (kThreads * 16);  // loads in flight
  for (long long b = 0; b < n; b += U * kThreads) {
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long at = b + u * kThreads + threadIdx.x;
      if (at < n) v[u] = from ? from[at] : V{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long at = b + u * kThreads + threadIdx.x;
      if (at < n) to[at] = v[u];
    }
  }
}

template <bool STAGE>
__global__ void __launch_bounds__(kThreads) move_kernel(const MoveParams p) {
  for (int i = blockIdx.y; i < p.n; i += gridDim.y) {
    const int src = p.src[i], dst = p.dst[i];
    if (dst < 0 || src == dst) continue;
    if (dst >= p.P || src >= p.P) {
      if (!STAGE && blockIdx.x == 0 && threadIdx.x == 0) set_error(p.err, KDA_DERR_SLOT);
      continue;
    }
    const bool staged = p.ws && src >= 0 && written_by_other(p, src, i);
    if (STAGE && !staged) continue;
    int a = 0;
    while (a + 1 < p.L && p.first[a + 1] <= (int)blockIdx.x) ++a;
    const long long off = (long long)((int)blockIdx.x - p.first[a]) * kMoveChunk;
    const long long left = p.bytes[a] - off, bytes = left < kMoveChunk ? left : kMoveChunk;
    unsigned char *area = p.ws + i * p.ws_bytes + p.ws_off[a] + off;
    const unsigned char *from = src < 0 ? nullptr : p.base[a] + src * p.bytes[a] + off;
    unsigned char *to = p.base[a] + dst * p.bytes[a] + off;
    if (STAGE) to = area;
    else if (staged) from = area;
    if (p.bytes[a] % 16 == 0)
      copy_chunk(reinterpret_cast<uint4 *>(to), reinterpret_cast<const uint4 *>(from), bytes / 16);
    else
      copy_chunk(reinterpret_cast<uint32_t *>(to), reinterpret_cast<const uint32_t *>(from),
                 bytes / 4);
  }
}

}  // namespace

cudaError_t launch_moves(const MoveParams &p, cudaStream_t s) {
  const dim3 grid(p.first[p.L], p.n < 65535 ? p.n : 65535);
  if (p.ws) {
    move_kernel<true><<<grid, kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  move_kernel<false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace kda
