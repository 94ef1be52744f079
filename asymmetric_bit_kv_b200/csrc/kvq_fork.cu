// Copies of a sequence: rings, sinks, the block records that cannot be
// shared, the length table and the page table of every layer, for every
// destination, in one launch.
//
// Bound by HBM writes: a destination's bytes are written once, the source's
// read once, since a CTA keeps its piece in registers and stores it to every
// destination. A piece is kPiece bytes of one layer's areas laid end to end
// (key ring, value ring, key sinks, value sinks, then the records head by
// head); all areas are multiples of 16 bytes, so a 16-byte unit lies in one.
// Measured (8 KV heads): K2 V4, ring of 128 tokens and 14 blocks of 64 in the last
// page, 15 copies and 8 layers (159 MB written) 48 us, 3.3 TB/s, 63 copies and 32
// layers (2.67 GB) 516 us, 5.2 TB/s; K4 V2, ring of 64 and no partly filled page, 15
// copies and 8 layers (31 MB) 14 us; 3 copies, 2 layers 10 us.
#include <algorithm>

#include "kvq_fork.cuh"

namespace kvq {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                          // 16-byte units in flight per thread
constexpr int64_t kPiece = kThreads * kUnits * 16;  // bytes per CTA

__host__ __device__ inline int64_t layer_bytes(const ForkLayer& f, int hkv) {
  return f.ring_k_bytes + f.ring_v_bytes + 2 * f.sink_bytes + f.head_bytes * hkv;
}

// Address of byte `at` of a layer's areas in sequence b (`page`: its last
// page); at is a multiple of 16.
__device__ __forceinline__ uint8_t* area(const ForkParams& p, const ForkLayer& f, int64_t at, int b, int page) {
  if (at < f.ring_k_bytes) return static_cast<uint8_t*>(f.ring_k) + b * f.ring_k_bytes + at;
  at -= f.ring_k_bytes;
  if (at < f.ring_v_bytes) return static_cast<uint8_t*>(f.ring_v) + b * f.ring_v_bytes + at;
  at -= f.ring_v_bytes;
  if (at < f.sink_bytes) return static_cast<uint8_t*>(f.sink_k) + b * f.sink_bytes + at;
  at -= f.sink_bytes;
  if (at < f.sink_bytes) return static_cast<uint8_t*>(f.sink_v) + b * f.sink_bytes + at;
  at -= f.sink_bytes;
  const int64_t h = at / f.head_bytes, own = p.page_blocks > 0 ? page : b;
  return f.blocks + (own * p.num_kv_heads + h) * f.head_stride + (at - h * f.head_bytes);
}

__global__ void __launch_bounds__(kThreads) fork_kernel(ForkParams p) {
  const ForkLayer& f = p.layer[blockIdx.y];
  const int64_t total = layer_bytes(f, p.num_kv_heads), base = blockIdx.x * kPiece + threadIdx.x * 16;
  uint4 x[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t at = base + u * kThreads * 16;
    if (at < total) x[u] = *reinterpret_cast<const uint4*>(area(p, f, at, p.src, f.tail_src));
  }
  for (int i = 0; i < p.num_dsts; ++i) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t at = base + u * kThreads * 16;
      if (at < total) *reinterpret_cast<uint4*>(area(p, f, at, p.dst[i], p.tail_dst[blockIdx.y][i])) = x[u];
    }
  }
  if (blockIdx.x != 0) return;
  const int32_t* len = f.lens + (int64_t)p.src * kLensStride;
  for (int e = threadIdx.x; e < p.num_dsts * kLensStride; e += kThreads)
    f.lens[(int64_t)p.dst[e / kLensStride] * kLensStride + e % kLensStride] = len[e % kLensStride];
  if (p.page_blocks > 0) {
    const int32_t* row = f.page_table + (int64_t)p.src * p.max_pages;
    const int pages = f.full_pages + (f.head_bytes > 0 ? 1 : 0);
    for (int i = 0; i < p.num_dsts; ++i) {
      int32_t* to = f.page_table + (int64_t)p.dst[i] * p.max_pages;
      for (int k = threadIdx.x; k < pages; k += kThreads)
        to[k] = k < f.full_pages ? row[k] : p.tail_dst[blockIdx.y][i];
    }
  }
}

}  // namespace

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  int64_t most = 0;
  for (int l = 0; l < p.layers; ++l) most = std::max(most, layer_bytes(p.layer[l], p.num_kv_heads));
  fork_kernel<<<dim3((unsigned)((most + kPiece - 1) / kPiece), p.layers), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kvq
