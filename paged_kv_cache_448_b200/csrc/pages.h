// pages.h — host/device arguments of the page operators (pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace paged {

constexpr int kMaxPlanes = 128;  // planes per launch (their pointers are launch arguments)

// A plane: num_blocks blocks of block_bytes contiguous bytes.
struct PlaneRef {
  void* base;
  int64_t block_bytes;
};

struct ForkArgs {
  const int32_t* block_tables;  // [num_seqs, max_blocks_per_seq]
  const int32_t* context_lens;  // [num_seqs]
  const int32_t* parents;       // [num_children]
  const int32_t* fresh_blocks;  // [num_children]; negative: share the last block
  int32_t* new_block_tables;    // [num_children, max_blocks_per_seq]
  int32_t* new_context_lens;    // [num_children]
  int32_t* err;                 // optional error word
  int64_t num_blocks;
  int32_t num_seqs, max_blocks_per_seq, num_children, block_size;
  int32_t write_tables;         // this launch writes rows and lengths (set by launch_fork)
};

struct CompactArgs {
  const int32_t* moves;   // [num_moves][2]: source, destination; sources ascending
  int32_t* block_tables;  // num_entries entries, rewritten in place
  int32_t* err;           // optional error word
  int64_t num_blocks, num_entries;
  int32_t num_moves;
  int32_t table_ctas;     // CTAs that rewrite entries (set by launch_compact)
};

cudaError_t launch_fork(ForkArgs a, const PlaneRef* planes, int num_planes, int sm_count,
                        cudaStream_t stream);
cudaError_t launch_compact(CompactArgs a, const PlaneRef* planes, int num_planes, int sm_count,
                           cudaStream_t stream);

}  // namespace paged
