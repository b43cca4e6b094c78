// pages.cu — forking sequences and compacting the pool, over all planes of a
// cache (the K and V caches of every layer, or their codes and scales) in one
// launch.
//
// fork: child i of parent p gets p's table row; whole blocks are shared, and
// the last block, when it is not full, is copied into a fresh block of the
// child in every plane ("大模型推理KV Cache内存管理与PagedAttention分页显存实战":
// several samples of one prompt share its blocks under reference counts).
// compact: block src moves to block dst in every plane for a list of moves,
// and table entries follow.
//
// Both are copies of contiguous blocks within a plane, bound by memory (2 x
// the bytes moved) or, for a few small blocks, by the launch; a layer's blocks
// are small in a 4-bit cache (8 KB of codes and 512 B of scales for 16 tokens
// of 8 heads), so a launch per layer would cost more than the copies. The
// work is cut into items of at most 4 KB of one block of one plane, one warp
// each, all its loads in flight before the first store; the planes' pointers
// travel in the launch's arguments. On a B200: 700 blocks of 4 layers of 32
// heads in 16 bits (1.47 GB) 244 us, 6.0 TB/s; 128 partial blocks of 32 layers
// in 4 bits (94 MB) 18 us; a few blocks 4 us, the launch.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "decode_args.h"
#include "device_common.cuh"
#include "pages.h"

namespace paged {
namespace {

constexpr int kWarps = 8;               // warps per CTA
constexpr int kVec = 8;                 // 16-byte vectors per lane of an item
constexpr int kItem = 32 * kVec * 16;   // bytes of an item

struct Planes {
  uint8_t* base[kMaxPlanes];
  int32_t first[kMaxPlanes + 1];  // items of the planes before this one, per copied block
  int32_t bytes16[kMaxPlanes];    // 16-byte vectors of a block
  int32_t num;
};

// Item `item` (of the items of one copied block): copy src -> dst.
__device__ __forceinline__ void copy_item(const Planes& pl, int item, int64_t src, int64_t dst,
                                          int lane) {
  int lo = 0, hi = pl.num;  // the plane with first[lo] <= item < first[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pl.first[mid] <= item) lo = mid;
    else hi = mid;
  }
  const int64_t n = pl.bytes16[lo];
  const int at = (item - pl.first[lo]) * (kItem / 16);
  const uint4* s = reinterpret_cast<const uint4*>(pl.base[lo]) + src * n;
  uint4* d = reinterpret_cast<uint4*>(pl.base[lo]) + dst * n;
  uint4 v[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const int j = at + lane + 32 * k;
    if (j < n) v[k] = __ldcs(s + j);
  }
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const int j = at + lane + 32 * k;
    if (j < n) __stcs(d + j, v[k]);
  }
}

// Context length of parent p, clipped to its table row.
__device__ __forceinline__ int parent_context(const ForkArgs& a, int p) {
  const int64_t most = static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
  const int ctx = a.context_lens[p];
  return ctx < 0 ? 0 : ctx > most ? static_cast<int>(most) : ctx;
}

__global__ void __launch_bounds__(kWarps * 32)
    fork_kernel(const ForkArgs a, const __grid_constant__ Planes pl) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_child = pl.first[pl.num] + (a.write_tables ? 1 : 0);
  const int64_t total = static_cast<int64_t>(a.num_children) * per_child;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp; i < total; i += stride) {
    const int child = static_cast<int>(i / per_child), item = static_cast<int>(i % per_child);
    const int p = a.parents[child];
    const bool known = p >= 0 && p < a.num_seqs;
    const int ctx = known ? parent_context(a, p) : 0;
    const int nblk = (ctx + a.block_size - 1) / a.block_size;
    const int32_t* row = a.block_tables + static_cast<int64_t>(known ? p : 0) * a.max_blocks_per_seq;
    const int fresh = a.fresh_blocks[child];
    const bool own = ctx % a.block_size != 0 && fresh >= 0;  // the last block is the child's own
    if (item < pl.first[pl.num]) {
      if (!own || fresh >= a.num_blocks) continue;
      const int src = row[nblk - 1];
      if (src < 0 || src >= a.num_blocks) continue;
      copy_item(pl, item, src, fresh, lane);
      continue;
    }
    // the child's row and length, and what is wrong with its request
    int32_t* out = a.new_block_tables + static_cast<int64_t>(child) * a.max_blocks_per_seq;
    for (int j = lane; j < a.max_blocks_per_seq; j += 32) {
      int32_t id = j < nblk ? row[j] : -1;
      if (j < nblk && (id < 0 || id >= a.num_blocks)) report(a.err, kErrBadBlockId);
      if (own && j == nblk - 1) id = fresh < a.num_blocks ? fresh : -1;
      out[j] = id;
    }
    if (lane == 0) {
      a.new_context_lens[child] = ctx;
      if (!known) report(a.err, kErrBadParent);
      else if (a.context_lens[p] != ctx) report(a.err, kErrContextClipped);
      if (own && fresh >= a.num_blocks) report(a.err, kErrBadBlockId);
    }
  }
}

// The move whose source is `id`, or -1 (the sources ascend).
__device__ __forceinline__ int find_move(const int2* moves, int n, int id) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (moves[mid].x < id) lo = mid + 1;
    else hi = mid;
  }
  return lo < n && moves[lo].x == id ? lo : -1;
}

__device__ __forceinline__ bool move_ok(int2 m, int64_t num_blocks) {
  return m.x >= 0 && m.x < num_blocks && m.y >= 0 && m.y < num_blocks;
}

__global__ void __launch_bounds__(kWarps * 32)
    compact_kernel(const CompactArgs a, const __grid_constant__ Planes pl) {
  const int lane = threadIdx.x & 31;
  const int2* moves = reinterpret_cast<const int2*>(a.moves);
  // the first CTAs: table entries that name a moved block, and the checks
  if (blockIdx.x < static_cast<unsigned>(a.table_ctas)) {
    const int64_t stride = static_cast<int64_t>(a.table_ctas) * blockDim.x;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    for (int64_t i = t; i < a.num_entries; i += stride) {
      const int m = find_move(moves, a.num_moves, a.block_tables[i]);
      if (m >= 0 && move_ok(moves[m], a.num_blocks)) a.block_tables[i] = moves[m].y;
    }
    for (int64_t i = t; i < a.num_moves; i += stride) {
      if (!move_ok(moves[i], a.num_blocks)) report(a.err, kErrBadBlockId);
      if ((i > 0 && moves[i - 1].x >= moves[i].x) ||
          find_move(moves, a.num_moves, moves[i].y) >= 0)
        report(a.err, kErrBadMoves);
    }
    return;
  }
  const int per_move = pl.first[pl.num];
  const int64_t total = static_cast<int64_t>(a.num_moves) * per_move;
  const int64_t stride = static_cast<int64_t>(gridDim.x - a.table_ctas) * kWarps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x - a.table_ctas) * kWarps + (threadIdx.x >> 5);
       i < total; i += stride) {
    const int2 m = moves[i / per_move];
    if (move_ok(m, a.num_blocks)) copy_item(pl, static_cast<int>(i % per_move), m.x, m.y, lane);
  }
}

// Planes [at, at + kMaxPlanes) of the caller's as launch arguments.
Planes pack(const PlaneRef* planes, int num, int at) {
  Planes p{};
  p.num = std::min(num - at, kMaxPlanes);
  for (int i = 0; i < p.num; ++i) {
    p.base[i] = static_cast<uint8_t*>(planes[at + i].base);
    p.bytes16[i] = static_cast<int32_t>(planes[at + i].block_bytes / 16);
    p.first[i + 1] =
        p.first[i] + static_cast<int32_t>((planes[at + i].block_bytes + kItem - 1) / kItem);
  }
  return p;
}

unsigned grid_for(int64_t items, int sm_count) {
  // up to eight CTAs of eight warps per SM, striding beyond that
  const int64_t ctas = (items + kWarps - 1) / kWarps;
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ctas, sm_count * 8LL)));
}

}  // namespace

cudaError_t launch_fork(ForkArgs a, const PlaneRef* planes, int num_planes, int sm_count,
                        cudaStream_t stream) {
  for (int at = 0; at == 0 || at < num_planes; at += kMaxPlanes) {
    const Planes p = pack(planes, num_planes, at);
    a.write_tables = at == 0;
    const int64_t items =
        static_cast<int64_t>(a.num_children) * (p.first[p.num] + (a.write_tables ? 1 : 0));
    fork_kernel<<<grid_for(items, sm_count), kWarps * 32, 0, stream>>>(a, p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_compact(CompactArgs a, const PlaneRef* planes, int num_planes, int sm_count,
                           cudaStream_t stream) {
  for (int at = 0; at == 0 || at < num_planes; at += kMaxPlanes) {
    const Planes p = pack(planes, num_planes, at);
    const int64_t entries = std::max<int64_t>(a.num_entries, a.num_moves);
    a.table_ctas = at == 0 ? static_cast<int>(std::min<int64_t>((entries + 255) / 256, sm_count))
                           : 0;
    const int64_t items = static_cast<int64_t>(a.num_moves) * p.first[p.num];
    if (a.table_ctas == 0 && items == 0) continue;
    compact_kernel<<<a.table_ctas + grid_for(items, sm_count), kWarps * 32, 0, stream>>>(a, p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace paged
