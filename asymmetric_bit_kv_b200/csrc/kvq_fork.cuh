// Parameters and launcher of the sequence copy (kvq_fork_sequence).
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr int kForkLayers = 32, kForkDsts = 64;  // layers and destinations of one launch

// What one layer copies. Rings and sinks are contiguous per sequence; block
// records are head_bytes per KV head, heads head_stride apart, from the
// source's own area (contiguous cache) or from its last, partly filled page.
struct ForkLayer {
  uint8_t* blocks;
  void *ring_k, *ring_v, *sink_k, *sink_v;
  int32_t* lens;        // [max_batch][kLensStride]
  int32_t* page_table;  // paged: [max_batch][max_pages]
  int64_t ring_k_bytes, ring_v_bytes, sink_bytes;  // of one sequence
  int64_t head_bytes, head_stride;
  int32_t full_pages;   // paged: filled pages, shared by reference
  int32_t tail_src;     // paged: the source's last page (head_bytes > 0)
};

struct ForkParams {
  int32_t src, num_dsts, layers, num_kv_heads, page_blocks, max_pages;
  int32_t dst[kForkDsts];
  ForkLayer layer[kForkLayers];
  int32_t tail_dst[kForkLayers][kForkDsts];  // paged: each destination's last page
};

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream);

}  // namespace kvq
