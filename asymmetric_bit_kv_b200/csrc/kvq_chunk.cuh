// Parameters and launchers of chunk attention (kvq_chunk_attention): a chunk
// of new tokens of every sequence attends to the sequence's cached tokens and
// causally to the chunk itself.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// A sequence with new tokens, in launch order (the host puts the longest work
// first). Positions: cached token c of a sequence is sink c (c < s), then
// position c - s after the sinks: a quantized token below q (keys) / qv
// (values), else a ring token. New token t is the sequence's token len + t,
// len = s + q + n. Query token t sees token c when c <= len + t and, with a
// window, when also c > len + t - window or c < sink_tokens. The fields of an
// entry lie together: a CTA reads them once, from a cold constant cache.
struct ChunkEntry {
  int32_t item0;  // first work item
  int32_t seq;
  int32_t s, q, qv, n;  // host mirror of the lengths
  int32_t t;      // new tokens
  int32_t off;    // first row of the sequence in k, v, q and out
  // Tensor-core kernel: how the sequence's units (KV head, tile of query rows)
  // are cut. splits > 0: so many ranges of the tokens, both slots of a CTA on
  // every tile (256 rows); splits < 0: -splits ranges, the slots on alternate
  // tiles (at most 128 rows). A row of several parts leaves part j at record
  // part0 + (h * rows + r) * parts + j of ws_o / ws_ml, and the merge kernel
  // joins the rows merge0 .. of all entries (entries of one part take none).
  int32_t splits, part0, merge0;
  int32_t pad;
};

// One launch.
struct ChunkParams {
  LayerView L;
  const void* k;        // [tokens][Hkv][D] kv dtype, the chunk's keys
  const void* v;
  const void* q;        // [tokens][Hq][D] kv dtype
  void* out;            // [tokens][Hq][D] out dtype
  float* ws_o;          // [records][D]
  float2* ws_ml;        // [records]: (maximum in log2 units, sum)
  int32_t* err;
  float scale_log2;     // softmax scale * log2(e)
  int32_t out_dtype;
  int32_t num_q_heads;
  int32_t window;       // 0: none
  int32_t sink_tokens;  // S of the cache: tokens that stay visible outside the window
  int32_t tokens;       // rows of k and v
  int32_t nseq;         // entries
  int32_t items;        // work items of all entries
  int32_t merge_rows;
  // Shared pages (decode of forked sequences; 0: chunk attention). An entry is
  // then a run of sequences off .. off + t - 1 with one query token each, whose
  // first q positions lie in pages that all of them hold: its rows see those
  // positions and nothing else, and part j of a row of q goes to record
  // row * slots + part0 + j, beside the decode kernel's partials of the row.
  int32_t slots;
  ChunkEntry e[KVQ_MAX_BATCH];

  // The entry that work item (merge row) x belongs to.
  __device__ __forceinline__ int entry_of_item(int x) const {
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (e[mid].item0 <= x) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
  __device__ __forceinline__ int entry_of_merge(int x) const {
    int lo = 0, hi = nseq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (e[mid].merge0 <= x) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};
// Parts of each row of an entry with these splits.
__host__ __device__ inline int chunk_parts(int splits) { return splits < 0 ? -2 * splits : splits; }

constexpr int kChunkRows = 16;  // query rows (token, head) of one CTA of the CUDA-core kernel

// The CUDA-core kernel: every cache format.
cudaError_t launch_chunk_simple(const ChunkParams& p, cudaStream_t stream);

// The tensor-core kernel and the merge of its parts: layers whose keys and
// values share one residual length.
constexpr int kChunkSlotRows = 128;  // query rows of one slot; a CTA has two
constexpr int kChunkTile = 128;      // tokens of a tile
bool chunk_tc_supported(const LayerView& L);
cudaError_t launch_chunk_tc(const ChunkParams& p, cudaStream_t stream);

}  // namespace kvq
