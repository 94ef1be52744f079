// Chunk attention on the CUDA cores: any cache format.
//
// Method: attention of a chunk of a prompt over the quantized cache and the
// chunk's own exact keys and values ("KIVI" README, Overview: prefill attends
// in full precision, the cache holds per-channel keys, per-token values and
// the exact recent window), x_hat = q*d + m ("KV1-1.2B" card, BQ2_0).
//
//   out[t] = sum_j 2^(z_tj - m_t) v_j / sum_j 2^(z_tj - m_t),
//   z_tj = scale * log2(e) * q_t . k_j over the tokens j that t sees,
// in one pass over j with the running maximum m_t and sum.
//
// A CTA takes kChunkRows query rows (token, query head of one KV head) of one
// (sequence, KV head) and walks the tokens they see 32 at a time: the tile's
// keys and values are dequantized once into shared memory as fp32 (rotated
// back for a Hadamard cache), then each warp scores its rows with one lane
// per token and accumulates the values with four channels per lane. Everything
// is fp32. Bound by shared-memory loads and FMAs, as a plain fp32 kernel is:
// 4096 new tokens over 32768 (32 query and 8 KV heads) take 1.55 s, 1.5 TFLOP/s.
#include "kvq_chunk.cuh"

namespace kvq {

namespace {

constexpr int kTile = 32;     // tokens per tile: one per lane
constexpr int kWarps = 4;
constexpr int kRowsPerWarp = kChunkRows / kWarps;

// Key (KEY) or value of cached position p (after the sinks) at channels
// 4*lane .. 4*lane + 3, in the original basis.
template <bool KEY>
__device__ __forceinline__ void cached_token(const LayerView& L, int b, int h, int p, int q_len, int lane,
                                             float (&x)[4]) {
  const int64_t unit = (int64_t)b * L.num_kv_heads + h;
  if (p >= q_len) {
    const int R = KEY ? L.residual : L.residual_v;
    const void* ring = KEY ? L.ring_k : L.ring_v;
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = load_kv(ring, (unit * R + p % R) * kHeadDim + 4 * lane + c, L.kv_dtype);
    return;
  }
  const int G = L.group_k, t = p % G;
  const uint8_t* rec = record_ptr(L, b, h, p / G);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int d = 4 * lane + c;
    uint32_t code;
    __half sc, z;
    if constexpr (KEY) {
      const int per = 32 / L.k_bits;
      code = (*reinterpret_cast<const uint32_t*>(rec + kc_word_byte(L, d, t / per)) >> ((t % per) * L.k_bits)) &
             ((1u << L.k_bits) - 1);
      const __half2 sz = *reinterpret_cast<const __half2*>(rec + ksz_pair_byte(L, t, d));
      sc = __low2half(sz);
      z = __high2half(sz);
    } else {
      const int per = 32 / L.v_bits;
      code = (*reinterpret_cast<const uint32_t*>(rec + vc_word_byte(L, t, d / per)) >> ((d % per) * L.v_bits)) &
             ((1u << L.v_bits) - 1);
      sc = *reinterpret_cast<const __half*>(rec + vsz_half_byte(L, t, d / L.group_v, false));
      z = *reinterpret_cast<const __half*>(rec + vsz_half_byte(L, t, d / L.group_v, true));
    }
    x[c] = dequant_value(code, sc, z);
  }
  if (L.hadamard) rotate_lane(x, lane);  // H . H = 1
}

__global__ void __launch_bounds__(32 * kWarps) chunk_simple_kernel(ChunkParams p) {
  __shared__ float sq[kChunkRows][kHeadDim];
  __shared__ float sk[kTile][kHeadDim + 1];  // the pad keeps one lane per token free of bank conflicts
  __shared__ float sv[kTile][kHeadDim];
  const LayerView& L = p.L;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x;
  const int i = p.entry_of_item(item), b = p.e[i].seq;
  const int h = (item - p.e[i].item0) % L.num_kv_heads, rt = (item - p.e[i].item0) / L.num_kv_heads;
  const int ngr = p.num_q_heads / L.num_kv_heads;
  const int rows = p.e[i].t * ngr, r0 = rt * kChunkRows;  // row r: token r / ngr, head h * ngr + r % ngr
  const int s = p.e[i].s, len = s + p.e[i].q + p.e[i].n;
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q);
  for (int e = threadIdx.x; e < kChunkRows * kHeadDim; e += blockDim.x) {
    const int r = r0 + e / kHeadDim;
    float x = 0.f;
    if (r < rows) {
      const int64_t row = (int64_t)(p.e[i].off + r / ngr) * p.num_q_heads + h * ngr + r % ngr;
      x = load_kv(q, row * kHeadDim + e % kHeadDim, L.kv_dtype) * p.scale_log2;
    }
    sq[e / kHeadDim][e % kHeadDim] = x;
  }
  float m[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][4];
  int pos[kRowsPerWarp];  // the row's token index in its sequence
#pragma unroll
  for (int e = 0; e < kRowsPerWarp; ++e) {
    m[e] = -INFINITY;
    l[e] = 0.f;
    o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
    pos[e] = len + (r0 + warp * kRowsPerWarp + e) / ngr;
  }
  // tokens that some row of the CTA sees: the sinks, then [first, end)
  const int end = len + (min(r0 + kChunkRows, rows) - 1) / ngr + 1;
  const int first = p.window > 0 ? max(0, len + r0 / ngr - p.window + 1) : 0;
  for (int c0 = 0; c0 < end; c0 += kTile) {
    if (c0 + kTile <= first && c0 >= p.sink_tokens) {  // nothing of this tile is visible: on to the window
      c0 = (first / kTile - 1) * kTile;
      continue;
    }
    __syncthreads();
    for (int t = warp; t < kTile; t += kWarps) {
      const int c = c0 + t;
      float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
      if (c < s) {
        const int64_t row = (((int64_t)b * L.num_kv_heads + h) * KVQ_MAX_SINKS + c) * kHeadDim + 4 * lane;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = load_kv(L.sink_k, row + e, L.kv_dtype);
          y[e] = load_kv(L.sink_v, row + e, L.kv_dtype);
        }
      } else if (c < len) {
        cached_token<true>(L, b, h, c - s, p.e[i].q, lane, x);
        cached_token<false>(L, b, h, c - s, p.e[i].qv, lane, y);
      } else if (c < end) {
        const int64_t row = ((int64_t)(p.e[i].off + c - len) * L.num_kv_heads + h) * kHeadDim + 4 * lane;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = load_kv(p.k, row + e, L.kv_dtype);
          y[e] = load_kv(p.v, row + e, L.kv_dtype);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sk[t][4 * lane + e] = x[e];
        sv[t][4 * lane + e] = y[e];
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kRowsPerWarp; ++e) {
      const int c = c0 + lane;  // this lane's token
      const bool seen = c <= pos[e] && (p.window == 0 || c > pos[e] - p.window || c < p.sink_tokens) && c < end;
      const unsigned any = __ballot_sync(0xffffffffu, seen);
      if (any == 0) continue;
      float z = 0.f;
      const float* qr = sq[warp * kRowsPerWarp + e];
#pragma unroll 16
      for (int d = 0; d < kHeadDim; ++d) z = fmaf(qr[d], sk[lane][d], z);
      if (!seen) z = -INFINITY;
      float mx = z;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[e], mx);
      const float a = exp2f(m[e] - mn), w = exp2f(z - mn);  // mn is finite: some token is seen
      float ws = w;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
      m[e] = mn;
      l[e] = l[e] * a + ws;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[e][d] *= a;
      for (int t = 0; t < kTile; ++t) {
        if (!((any >> t) & 1)) continue;  // a token that is not seen may hold anything
        const float wt = __shfl_sync(0xffffffffu, w, t);
        const float4 v4 = *reinterpret_cast<const float4*>(&sv[t][4 * lane]);
        o[e][0] = fmaf(wt, v4.x, o[e][0]);
        o[e][1] = fmaf(wt, v4.y, o[e][1]);
        o[e][2] = fmaf(wt, v4.z, o[e][2]);
        o[e][3] = fmaf(wt, v4.w, o[e][3]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kRowsPerWarp; ++e) {
    const int r = r0 + warp * kRowsPerWarp + e;
    if (r >= rows) break;
    const int64_t at = ((int64_t)(p.e[i].off + r / ngr) * p.num_q_heads + h * ngr + r % ngr) * kHeadDim + 4 * lane;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const float x = __fdiv_rn(o[e][d], l[e]);  // every row sees its own token
      if (p.out_dtype == KVQ_F32) reinterpret_cast<float*>(p.out)[at + d] = x;
      else if (p.out_dtype == KVQ_BF16) reinterpret_cast<__nv_bfloat16*>(p.out)[at + d] = __float2bfloat16_rn(x);
      else reinterpret_cast<__half*>(p.out)[at + d] = __float2half_rn(x);
    }
  }
}

}  // namespace

cudaError_t launch_chunk_simple(const ChunkParams& p, cudaStream_t stream) {
  if (p.items <= 0) return cudaSuccess;
  chunk_simple_kernel<<<p.items, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kvq
