// Copies, forks, compaction and freeing of slots over all arrays of a model
// in one call.  Memory bound: each moved byte is read once and written once.
//
// Moves act as if all at once: a move whose src is the dst of another has to
// read before that one writes.  Two ways:
//   - A thread owns 16 bytes at one place of every slot of an array and does
//     all moves there, readers of a slot before its writer.  Nothing but its
//     own program order is needed, and no byte is moved twice.  Where the
//     moves form a cycle, one of its sources is put aside in the workspace.
//   - A block copies one chunk of one move.  A first launch stages the sources
//     that another move writes in the workspace, and the second takes them
//     from there.  For many moves of little data, where a thread that does
//     them all would leave most of the machine idle.
// 64 moves, half of them into places that others leave, and 16 frees: 280 KB
// slots in 8 layers 63 us the first way (330 MB, 5.2 TB/s) and 76 the second,
// in 2 layers 22.4 and 20.7 us, 70 KB slots in one layer 15.6 and 7.6; 8 moves
// and 2 frees of 280 KB in one layer 5.7 and 7.5.  So the first way serves up to
// 16 moves, and more of them where it has two blocks a move.
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
  begin_after_stream();
  for (int i = blockIdx.y; i < p.n; i += gridDim.y) {
    const int src = p.src[i], dst = p.dst[i];
    if (dst < 0) continue;
    if (dst >= p.P || src >= p.P) {
      if (!STAGE && blockIdx.x == 0 && threadIdx.x == 0) set_error(p.err, KDA_DERR_SLOT);
      continue;
    }
    if (src == dst) continue;
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

constexpr int kMaxPlan = 1024;           // moves of the first way
constexpr int kColumns = kThreads * 16;  // bytes of a slot that a block owns

// The moves in an order in which every reader of a slot comes before its
// writer: by falling distance from the end of their chain, move i being
// followed by the writer of its source.  A cycle is cut at its lowest move,
// which comes last, its source put aside before.
struct Plan {
  int src[kMaxPlan], dst[kMaxPlan];    // as given; dst -1: nothing to do
  int next[kMaxPlan], rank[kMaxPlan];  // the writer of src; distance from the end
  int2 todo[kMaxPlan];                 // {src, dst} in order; src -1: zero, -2 - i: put aside
  int put[kMaxPlan];                   // the moves whose source is put aside
  int count, puts;
};

__device__ __forceinline__ void make_plan(const MoveParams &p, Plan &s) {
  const int n = p.n;
  if (threadIdx.x == 0) s.count = s.puts = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    int src = p.src[i], dst = p.dst[i];
    if (dst >= 0 && (dst >= p.P || src >= p.P)) {
      if (blockIdx.x == 0) set_error(p.err, KDA_DERR_SLOT);
      dst = -1;
    }
    s.src[i] = src < 0 ? -1 : src;
    s.dst[i] = dst < 0 || src == dst ? -1 : dst;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    int w = -1;
    if (s.dst[i] >= 0 && s.src[i] >= 0)
      for (int j = 0; j < n; ++j)
        if (s.dst[j] == s.src[i]) w = j;
    s.next[i] = w;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    int d = 0, at = i;
    while (s.next[at] >= 0 && d < n) at = s.next[at], ++d;
    if (d == n) {  // `at` is on a cycle: find its lowest move, and the way there
      int low = at;
      for (int j = s.next[at]; j != at; j = s.next[j]) low = min(low, j);
      for (d = 0, at = i; at != low; at = s.next[at]) ++d;
      if (i == low) s.put[atomicAdd(&s.puts, 1)] = i;
    }
    s.rank[i] = d;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    if (s.dst[i] < 0) continue;
    int before = 0;
    for (int j = 0; j < n; ++j)
      before += s.dst[j] >= 0 && (s.rank[j] > s.rank[i] || (s.rank[j] == s.rank[i] && j < i));
    const bool aside = s.rank[i] == 0 && s.next[i] >= 0;
    s.todo[before] = make_int2(aside ? -2 - i : s.src[i], s.dst[i]);
    atomicAdd(&s.count, 1);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads, 4) move_columns_kernel(const MoveParams p) {
  __shared__ Plan s;
  begin_after_stream();
  make_plan(p, s);
  int a = 0;
  while (a + 1 < p.L && p.first[a + 1] <= (int)blockIdx.x) ++a;
  const long long bytes = p.bytes[a];
  const long long off = (long long)((int)blockIdx.x - p.first[a]) * kColumns + threadIdx.x * 16;
  if (off >= bytes) return;
  unsigned char *base = p.base[a] + off, *aside = p.ws + p.ws_off[a] + off;
  for (int k = 0; k < s.puts; ++k) {
    const int i = s.put[k];
    *reinterpret_cast<uint4 *>(aside + i * p.ws_bytes) =
        *reinterpret_cast<const uint4 *>(base + s.src[i] * bytes);
  }
  constexpr int U = 8;  // loads in flight
  for (int k = 0; k < s.count; k += U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u < s.count) {
        const int from = s.todo[k + u].x;
        const unsigned char *at =
            from >= 0 ? base + from * bytes : aside + (-2 - from) * p.ws_bytes;
        v[u] = make_uint4(0, 0, 0, 0);
        if (from != -1) v[u] = *reinterpret_cast<const uint4 *>(at);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u < s.count) *reinterpret_cast<uint4 *>(base + s.todo[k + u].y * bytes) = v[u];
  }
}

}  // namespace

cudaError_t launch_moves(const MoveParams &p, cudaStream_t s) {
  if (p.ws && p.n <= kMaxPlan) {
    MoveParams q = p;
    long long blocks = 0;
    bool whole = true;  // every slot starts on 16 bytes
    for (int i = 0; i < p.L; ++i) {
      q.first[i] = (int)blocks;
      blocks += (p.bytes[i] + kColumns - 1) / kColumns;
      whole &= p.bytes[i] % 16 == 0;
      if (blocks > 0x7fffffffLL) whole = false;
      if (!whole) break;
    }
    q.first[p.L] = (int)blocks;
    if (whole && (p.n <= 16 || blocks >= 2 * p.n)) {
      return launch_after(move_columns_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, q);
    }
  }
  const dim3 grid(p.first[p.L], p.n < 65535 ? p.n : 65535);
  if (p.ws) {
    const cudaError_t e = launch_after(move_kernel<true>, grid, dim3(kThreads), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  return launch_after(move_kernel<false>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace kda
