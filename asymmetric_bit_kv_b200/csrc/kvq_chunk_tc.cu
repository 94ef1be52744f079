// Chunk attention on the tensor cores (tcgen05, tensor memory): layers whose
// keys and values share one residual length.
//
// Method: the formula of kvq_chunk.cu. A work item is one (sequence, KV head,
// tile of query rows); a row is (new token, query head of the KV head), so all
// query heads of a KV head share every dequantized key and value. The item
// walks the tokens its rows see in tiles of 128: first the quantized positions
// (phase A, tiles of positions 128a ..), then the exact tokens (phase B: the
// list sinks, ring, new tokens, in order). Per tile: S = Q K^T (128x128x128
// per slot), online softmax, O += P V.
//
// Why this shape. Two slots of 128 rows use all 512 columns of tensor memory
// (S0 | S1 | O0 | O1, fp32; P overwrites S as 16-bit pairs) and alternate: one
// slot's softmax runs while the tensor cores work on the other's products.
//  * More than 128 rows: both slots walk the same tiles (256 rows share each
//    dequantized tile).
//  * At most 128 rows: the slots take alternate tiles, each a part of its own.
// An item may also cover only a range of the tiles (few rows, long caches);
// parts are merged by chunk_combine_kernel.
//
// Warps: 0-3 and 4-7 the softmax of slots 0 and 1 (a thread owns a row, so
// maxima, sums and the rotation of a row need no exchange), 8, 9, 12, 13 key
// tiles, 10, 11, 14, 15 value tiles (each kind on two of the four schedulers),
// 16 issues the MMAs, 17 copies packed parts, 18 and 19 look through the values
// of tiles that some rows see in part (registers move between whole warpgroups,
// setmaxnreg 144 + 144 + 72 + 72 + 48 = 5 x 96). The hot
// loops are kept short (half a row of scores, one row of codes at a time) and
// what runs once per item is kept rolled: four roles share an SM's instruction
// caches, and unrolled whole tiles spent most of their time waiting for
// instructions.
//
// Operands. Phase A: codes become fp16 in three instructions per pair (mask
// into the mantissa of 1024, subtract, one fma q*d + m: the only rounding).
// Keys are packed along tokens and values along channels, so expanding a row
// of codes gives both operands with tokens (channels) contiguous: MN-major B
// tiles with 128-byte swizzle. A word's codes come out in extraction order
// (i, i + n/2), which permutes the tokens of a key tile: value rows are stored
// in the same order (their channels are put back by one permute per pair).
// Queries are scaled by a power of two per row (exact but for subnormals), so
// that any bf16 query fits fp16. Phase B: keys, values, queries and
// probabilities in the kv dtype, keys K-major.
//
// Softmax: probabilities are 2^(z - m + 6) with m a whole number that is raised
// only when the sum of 64 of a row's probabilities reaches 2^14: one pass over
// the scores without their maximum; rescaling O and what the tile has written
// is rare and exact (powers of two); fp16 probabilities stay below 2^14 and
// keep 14 + 6 binary orders below m before they turn subnormal.
//
// Measured (one B200; 32 query and 8 KV heads, K2 V4): 4096 new tokens over
// 32768 in 2630 us, 890 TFLOP/s, 0.54 of the measured rate of large products; a
// slot's chain (scores, exp2, probabilities, product) bounds it, with no pipe
// above half (tensor and exp2 first). 16 x 5 tokens over 8192: 125 us, 1.5 us a
// tile by the same chain and 31 us of launch, start, end and merge (at 120 us
// without expanding codes 103, with half the softmax 112). 2 x 300 tokens over
// 8190, rotated per-token keys: 126 us, of which an item's start and end take a
// third. Slower, when the first of these took 2555 to 2618: tiles of 64 tokens
// (2774), sixteen softmax warps (2705), an issuing warp per slot (2720), the
// softmax skipped by warps without rows (2893). What the compiler makes of the hot
// loops moves these figures by 5%, also when code elsewhere in the kernel changes.
//
// Every wait is bounded (~2 s): a thread that gives up sets the device error
// word and an abort flag that ends the others' waits.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "kvq_chunk.cuh"

namespace kvq {

namespace {

constexpr int kRows = kChunkSlotRows, kTile = kChunkTile, kD = kHeadDim;
constexpr int kThreads = 640;
constexpr int kLaunchRegisters = 96;  // of a thread: what setmaxnreg deals out, 5 x 96 = 144 + 144 + 72 + 72 + 48
constexpr int kProducers = 128;  // threads of the key warps, and of the value warps
constexpr int kKStages = 2, kVStages = 2;
constexpr int kRawStages = 4;           // raw stages at most
constexpr int kTileBytes = kTile * kD * 2;
constexpr int kHalf = kTileBytes / 2;  // one 64-wide block of a tile: 128 rows of 128 bytes
constexpr int kQOff = 0, kKOff = 2 * kTileBytes, kVOff = kKOff + kKStages * kTileBytes;
constexpr int kBarOff = kVOff + kVStages * kTileBytes;
constexpr int kBarBytes = 8 * (2 * kKStages + 3 * kVStages + 4 * 2 + 3 * kRawStages + 1);
constexpr int kRawOff = kBarOff + 256, kRawBytes = 34304;  // packed parts: at most 18,432 bytes each
constexpr int kSmemBytes = kRawOff + kRawBytes + 1024;     // + alignment of the base to 1024
static_assert(kBarBytes <= 8 * 32 && kBarBytes <= kRawOff - kBarOff, "a barrier per lane of a warp");
constexpr int kMixed = 10;  // tiles of an item that some of its rows see in part (Lost)
constexpr int kTmemS = 0, kTmemO = 256;           // columns of slot 0; slot 1 is 128 further
constexpr float kOffset = 6.f, kMost = 16384.f;  // of the probabilities: see above
constexpr long long kWaitCycles = 4000000000LL;

// ------------------------------------------------------------- PTX helpers
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {  // and arrive
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase with the given parity; false when the item was aborted
// (by this thread after ~2 s, or by another one).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (*abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// After an abort: waits for copies or products in flight (or ~2 s).
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity) && clock64() - t0 < kWaitCycles) {
  }
}
// mbar_wait by a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}
// One lane of the (converged) warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// 32 columns of this warp's 32 lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15])::"memory");
}
// Orders the loaded registers after the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool present) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(present ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t bits2(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return bits2(__floats2half2_rn(lo, hi));
  }
}

// Instruction descriptor: fp32 accumulator, A and B f16 or bf16, B MN-major or
// K-major, N = M = 128.
__device__ __forceinline__ uint32_t inst_desc(bool bf16, bool b_mn) {
  const uint32_t t = bf16 ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(kTile >> 3) << 17) |
         ((uint32_t)(kRows >> 4) << 24);
}

// The chunk's keys and values as matrices [tokens][Hkv * D], boxes of 128
// tokens x 64 channels with the 128-byte swizzle.
struct alignas(64) ChunkMaps {
  CUtensorMap k, v;
};

// ------------------------------------------------------------------ the item
struct Item {
  int i, b, h;          // table entry, sequence, KV head
  int ngr, lg;          // query heads per KV head (1, 2, 4 or 8) and the logarithm
  int rows, r0;         // rows of the unit, first row of the item
  int off;              // the sequence's first row in k, v, q and out
  bool both;            // both slots walk every tile (else alternate tiles)
  int t0, t1;           // first and last new token of the item's rows
  int s, q, n;          // sinks, quantized positions, ring tokens
  int nA, a0;           // phase A: tiles a0 .. a0 + nA - 1 of positions
  int nB, b0, b_sink;   // phase B: tile 0 first if b_sink, then tiles b0 ..
  int k0, k1;           // the item's range of the nA + nB tiles
  int part, parts;      // first part of the item, parts of the unit's rows
  int first_e;          // phase B entries below this stay visible outside the window

  // row of q and out of row r of the unit
  __device__ __forceinline__ int64_t row_of(const ChunkParams& p, int r) const {
    return (int64_t)(off + (r >> lg)) * p.num_q_heads + (h << lg) + (r & (ngr - 1));
  }
  __device__ __forceinline__ int tile_b(int k) const {  // phase B tile of k >= nA
    const int j = k - nA;
    return b_sink ? (j == 0 ? 0 : b0 + j - 1) : b0 + j;
  }
  __device__ __forceinline__ int steps() const { return both ? 2 * (k1 - k0) : k1 - k0; }
  // tiles of slot w
  __device__ __forceinline__ int slot_tiles(int w) const { return both ? k1 - k0 : (k1 - k0 + 1 - w) / 2; }
};

__device__ __forceinline__ Item find_item(const ChunkParams& p, int idx) {
  Item it;
  const int lo = p.entry_of_item(idx);
  const int hkv = p.L.num_kv_heads;
  it.i = lo;
  it.b = p.e[lo].seq;
  it.ngr = p.num_q_heads / hkv;
  it.lg = __ffs(it.ngr) - 1;
  it.off = p.e[lo].off;
  it.rows = p.e[lo].t * it.ngr;
  it.both = p.e[lo].splits > 0;
  const int ns = abs(p.e[lo].splits), tiles = (it.rows + 2 * kRows - 1) / (2 * kRows);
  int x = idx - p.e[lo].item0;
  const int sp = x % ns;
  x /= ns;
  it.h = x % hkv;
  it.r0 = (tiles - 1 - x / hkv) * 2 * kRows;  // the rows that see most first
  it.t0 = it.r0 >> it.lg;
  it.t1 = (min(it.r0 + 2 * kRows, it.rows) - 1) >> it.lg;
  it.s = p.e[lo].s;
  it.q = p.e[lo].q;
  it.n = p.e[lo].n;
  const int after = it.n + it.t0 - p.window + 1;  // first visible entry past the quantized positions, if >= 0
  const int low_a = p.window > 0 ? max(0, it.q + after) : 0;
  it.a0 = low_a / kTile;
  it.nA = low_a >= it.q ? 0 : (it.q + kTile - 1) / kTile - it.a0;
  it.first_e = it.q > 0 ? it.s : p.sink_tokens;
  const int low_b = p.window > 0 ? max(0, it.s + after) : 0;
  it.b0 = low_b / kTile;
  it.b_sink = it.first_e > 0 && it.b0 > 0 ? 1 : 0;
  it.nB = p.slots > 0 ? 0 : (it.s + it.n + it.t1 + kTile) / kTile - it.b0 + it.b_sink;
  const int64_t total = it.nA + it.nB;
  it.k0 = (int)(total * sp / ns);
  it.k1 = (int)(total * (sp + 1) / ns);
  it.parts = chunk_parts(p.e[lo].splits);
  it.part = it.both ? sp : 2 * sp;
  return it;
}

// ----------------------------------------------------------------- producers
// Four fp16 pairs of a 4-bit word's codes (i, i + 4), eight of a 2-bit word's
// (i, i + 8), two of an 8-bit word's (2i, 2i + 1), as exact integers.
template <int B>
__device__ __forceinline__ __half2 code_pair(uint32_t w, uint32_t w8, int i) {
  if constexpr (B == 8) {
    return __hsub2(half2_of(__byte_perm(w, 0x64646464u, i == 0 ? 0x4140 : 0x4342)), half2_of(0x64006400u));
  } else {
    constexpr int per = 8 / B;  // code positions in a byte
    const int k = i % per;
    const uint32_t m = ((1u << B) - 1u) << (B * k);
    const uint32_t x = ((i < per ? w : w8) & (m | (m << 16))) | 0x64006400u;  // 1024 + code * 2^(B k)
    if (k == 0) return __hsub2(half2_of(x), half2_of(0x64006400u));
    const __half f = __float2half_rn(1.f / (float)(1 << (B * k))), o = __float2half_rn(-1024.f / (float)(1 << (B * k)));
    return __hfma2(half2_of(x), __half2half2(f), __half2half2(o));
  }
}
template <int B>
constexpr int codes_per_word() { return 32 / B; }
// Place of code j of a word in extraction order, and the code at place c.
__host__ __device__ inline int place_of(int j, int per) {
  return per == 4 ? j : (j < per / 2 ? 2 * j : 2 * (j - per / 2) + 1);
}
__host__ __device__ inline int code_at(int c, int per) { return per == 4 ? c : ((c & 1) ? per / 2 : 0) + (c >> 1); }

// The largest code of a group whose scale was rounded up may stand for more
// than the largest fp16 number, 65504: it is taken as that. NaN stays.
__device__ __forceinline__ __half2 limit2(__half2 y) { return __hmin2_nan(y, half2_of(0x7bff7bffu)); }
// Whether some of a row's codes may: its groups' scales and zero points, each
// twice in a word. Hardly ever, so that the row is then mended, by a function
// that stays out of the hot loops: 16 x 5 tokens over 8192 took 119 us with it
// (without any of this 120; the function in line 132, the limit at every pair
// 138).
template <int B>
__device__ __forceinline__ bool past_fp16(const uint32_t (&s)[2], const uint32_t (&z)[2]) {
  const __half2 top = __float2half2_rn((float)((1 << B) - 1));
  return bits2(__hmax2(__hfma2(top, half2_of(s[0]), half2_of(z[0])), __hfma2(top, half2_of(s[1]), half2_of(z[1])))) ==
         0x7c007c00u;
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __noinline__ void limit_row(uint32_t row) {
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    const uint4 v = lds16(row + (c << 4));
    sts16(row + (c << 4), bits2(limit2(half2_of(v.x))), bits2(limit2(half2_of(v.y))), bits2(limit2(half2_of(v.z))),
          bits2(limit2(half2_of(v.w))));
  }
}

// Expands 64 codes (2 * B words) into a 128-byte row of fp16 at `row`, chunk
// c at c ^ x. sz(word, pair, s2, z2) gives the (scale, scale) and (zero, zero)
// halves of the two codes of a pair.
// NATURAL: the codes' own order instead, one more permute per pair. LIMIT: see
// limit2; else the caller looks at the row's scales (past_fp16).
template <int B, bool NATURAL, bool LIMIT, class SZ>
__device__ __forceinline__ void expand_row(const uint32_t (&w)[2 * B], uint32_t row, int x, SZ sz) {
  constexpr int per = 32 / B, pairs = per / 2;
#pragma unroll
  for (int j = 0; j < 2 * B; ++j) {
    const uint32_t w8 = w[j] >> 8;
    uint32_t h[pairs];
#pragma unroll
    for (int i = 0; i < pairs; ++i) {
      uint32_t s2, z2;
      sz(j, j * pairs + i, s2, z2);
      const __half2 y = __hfma2(code_pair<B>(w[j], w8, i), half2_of(s2), half2_of(z2));
      h[i] = bits2(LIMIT ? limit2(y) : y);
    }
    if constexpr (NATURAL && B != 8) {
      uint32_t o[pairs];
#pragma unroll
      for (int i = 0; i < pairs / 2; ++i) {
        o[i] = __byte_perm(h[2 * i], h[2 * i + 1], 0x5410);
        o[pairs / 2 + i] = __byte_perm(h[2 * i], h[2 * i + 1], 0x7632);
      }
#pragma unroll
      for (int i = 0; i < pairs; ++i) h[i] = o[i];
    }
    if constexpr (B == 8) {  // two words fill a chunk
      const uint32_t at = row + (((j >> 1) ^ x) << 4) + 8 * (j & 1);
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(h[0]), "r"(h[1]) : "memory");
    } else {
#pragma unroll
      for (int c = 0; c < pairs / 4; ++c)
        sts16(row + (((j * (pairs / 4) + c) ^ x) << 4), h[4 * c], h[4 * c + 1], h[4 * c + 2], h[4 * c + 3]);
    }
  }
}
__device__ __forceinline__ void zero_row(uint32_t row) {
#pragma unroll
  for (int c = 0; c < 8; ++c) sts16(row + (c << 4), 0u, 0u, 0u, 0u);
}

struct Bars {  // shared-memory addresses of arrays of barriers
  uint32_t k_full, k_empty, v_full, v_empty, s_full, p_ready, o_done, q_ready, raw_full, raw_empty, drain;
  uint32_t v_look, raw_look;  // in the place of v_full, raw_full for a mixed tile (Lost)
};

// What a row does not see must not matter, but 0 times an infinite or NaN value
// is NaN. In a mixed tile, which some of the item's rows see in part only, such
// values are therefore taken as zeros, and their tokens noted, a bit each: the
// rows that see one become NaN in the end (lose_row). Mixed tiles are a window's
// first ones of phase A (its low edge moves over at most 255 tokens, 3 tiles), the
// sinks' and a window's first ones of phase B, and the last ones, where each row
// sees up to its own token. A tile that all rows see needs none of this. Warps 18
// and 19 look through mixed tiles between their arrival and their use, so that
// the others' loops stay as they are: 4096 new tokens over 32768 take 2630 us (2570
// without all of this), 16 x 5 over 8192 125 (119), 4 x 2048 over nothing 217 (208).
// In the value warps' loop, by calls that hardly ever ran, the first two took 2630
// to 2800 and 130 to 143.
struct Lost {
  uint32_t bits[4 * kMixed];
  int any;
  int a_end, b_low, b_high, end;  // mixed: tiles k < a_end of phase A, k < b_low and k >= b_high of phase B, k < end

  __device__ __forceinline__ void set(const ChunkParams& p, const Item& it) {
    const int low_a = p.window > 0 ? it.q + it.n + it.t1 - p.window : -1;  // hidden from some row: up to here
    const int low_b = p.window > 0 ? it.s + it.n + it.t1 - p.window : -1;
    a_end = low_a < 0 ? 0 : min(it.nA, low_a / kTile - it.a0 + 1);
    b_low = it.nA + (low_b < 0 ? 0 : it.b_sink + max(0, low_b / kTile - it.b0 + 1));
    b_high = it.nA + max(0, (it.s + it.n + it.t0 + 1) / kTile - it.b0 + it.b_sink);
    end = it.nA + it.nB;
    any = 0;
  }
  // Number of tile k among the mixed ones, or -1.
  __device__ __forceinline__ int tile_a(int k) const { return k < a_end ? k : -1; }
  __device__ __forceinline__ int tile_b(int k, int nA) const {
    return k < b_low ? 3 + k - nA : k >= b_high ? 6 + end - k : -1;
  }
  __device__ __forceinline__ void note(int tile, int token) {
    atomicOr(&bits[4 * tile + (token >> 5)], 1u << (token & 31));
    *reinterpret_cast<volatile int*>(&any) = 1;
  }
};
static_assert(kSmemBytes + sizeof(Lost) + 16 <= 227 * 1024, "shared memory of one CTA");

// Packed parts. Warp 17 copies every 64-token part of the item's quantized
// tiles (one block, a tile of a 128-token block with the block's key scales, or
// two 32-token blocks) into a ring of raw stages; the key and value warps
// expand from there. What a producer thread reads of a part sits at offsets
// that it works out once.
struct RawLayout {
  int bytes, stages;  // of a stage
  int tile;           // offset of the (first) tile in a stage: 512 with shared key scales, else 0
  __device__ __forceinline__ explicit RawLayout(const LayerView& L) {
    tile = L.rec_ksz_off >= 0 ? kD * 4 : 0;
    bytes = L.group_k == 32 ? 2 * (int)L.record_bytes : tile + L.tile_bytes;
    bytes = (bytes + 127) & ~127;
    stages = min(kRawStages, kRawBytes / bytes);
  }
};
// A walk over the ring: stage and the parity of its next phase.
struct RawRing {
  int stage = 0, stages;
  uint32_t parity = 0;
  __device__ __forceinline__ explicit RawRing(int n) : stages(n) {}
  __device__ __forceinline__ void next() {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
};
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// One thread.
__device__ bool copy_parts(const ChunkParams& p, const Item& it, uint32_t smem, const Bars& bar, const Lost& lost,
                           volatile int* abort) {
  const LayerView& L = p.L;
  const int tiles = min(it.k1, it.nA) - it.k0;
  const RawLayout raw(L);
  RawRing ring(raw.stages);
  const int G = L.group_k, mixed = 2 * (lost.a_end - it.k0);  // parts of mixed tiles, which come first
  auto arrived = [&](int u) { return (u < mixed ? bar.raw_look : bar.raw_full) + 8 * (u % raw.stages); };
  for (int u = 0; u < 2 * tiles; ++u, ring.next()) {
    const int pos = (it.a0 + it.k0) * kTile + 64 * u;
    if (u >= raw.stages && !mbar_wait(bar.raw_empty + 8 * ring.stage, ring.parity ^ 1u, abort)) {
      for (int v = u - raw.stages; v < u; ++v) mbar_drain(arrived(v), (v / raw.stages) & 1);
      return false;
    }
    const uint32_t full = arrived(u), dst = smem + kRawOff + ring.stage * raw.bytes;
    if (pos >= it.q) {
      mbar_arrive(full);
      continue;
    }
    const uint8_t* rec = record_ptr(L, it.b, it.h, pos / G);
    const uint32_t rb = (uint32_t)L.record_bytes;
    if (G == 32) {
      const bool two = pos + 32 < it.q;
      mbar_expect_tx(full, two ? 2 * rb : rb);
      bulk_g2s(dst, rec, rb, full);
      if (two) bulk_g2s(dst + rb, record_ptr(L, it.b, it.h, pos / G + 1), rb, full);
    } else {
      mbar_expect_tx(full, raw.tile + L.tile_bytes);
      if (raw.tile) bulk_g2s(dst, rec + L.rec_ksz_off, kD * 4, full);
      const int64_t tile = G == 128 ? ((pos >> 6) & 1) * L.tile_bytes : 0;
      bulk_g2s(dst + raw.tile, rec + L.tile0_off + tile, L.tile_bytes, full);
    }
  }
  // (as in produce_exact: after an abort nobody else may wait for the last ones)
  for (int v = max(0, 2 * tiles - raw.stages); v < 2 * tiles; ++v)
    mbar_drain(arrived(v), (v / raw.stages) & 1);
  return true;
}

__device__ __forceinline__ uint32_t lds4(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t addr) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

// The warp has read what it needs of the stage.
__device__ __forceinline__ void release_raw(const Bars& bar, const RawRing& ring) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar.raw_empty + 8 * ring.stage);
}

// Key tiles of phase A: thread kt expands channel kt of a part.
template <int KB>
__device__ bool produce_keys(const ChunkParams& p, const Item& it, uint32_t smem, const Bars& bar, int kt,
                             volatile int* abort) {
  const int parts = 2 * (min(it.k1, it.nA) - it.k0);
  if (parts <= 0) return true;
  const LayerView& L = p.L;
  const bool axis0 = L.k_axis == 0, wide = L.group_k >= 64;
  const RawLayout raw(L);
  RawRing ring(raw.stages);
  // the channel's codes (64-token tiles: a row of KB / 2 chunks; 32-token
  // blocks: the same words in two blocks), its scales or its group's
  const int x = wide ? chunk_swizzle(kt, KB / 2) : KB == 8 ? chunk_swizzle(kt, 2) : 0;
  const int codes = raw.tile + L.kc_off + 4 * (wide ? kt * 2 * KB : KB == 2 ? kc_word_index(kt, 0, 2) : kt * KB);
  const int sz = raw.tile ? 4 * kt : L.ksz_off + 4 * kt;
  const int block = wide ? 0 : (int)L.record_bytes;
  const int tok = raw.tile + L.ksz_off + 4 * (kt / L.group_v), ng = kD / L.group_v;
  const int tok2 = wide ? tok + 32 * 4 * ng : tok + block;
  int valid = it.q - (it.a0 + it.k0) * kTile;  // positions of the part that exist, and of those after it
  const uint32_t dst = smem + kKOff + kt * 128;
  int st = 0;
  uint32_t phase = 1;  // of the stage's empty barrier: the first pass does not wait
#pragma unroll 1
  for (int u = 0; u < parts; ++u, valid -= 64, ring.next()) {
    if (!mbar_wait_warp(bar.raw_full + 8 * ring.stage, ring.parity, abort)) return false;
    const uint32_t src = smem + kRawOff + ring.stage * raw.bytes;
    uint32_t w[2 * KB], s[2], z[2];
    if (wide) {
#pragma unroll
      for (int e = 0; e < KB / 2; ++e) {
        const uint4 v = lds16(src + codes + ((e ^ x) << 4));
        w[4 * e] = v.x, w[4 * e + 1] = v.y, w[4 * e + 2] = v.z, w[4 * e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if constexpr (KB == 2) {
          w[2 * b] = lds4(src + codes + b * block);
          w[2 * b + 1] = lds4(src + codes + b * block + 4);
        } else {
#pragma unroll
          for (int e = 0; e < KB / 4; ++e) {
            const uint4 v = lds16(src + codes + b * block + ((e ^ x) << 4));
            w[KB * b + 4 * e] = v.x, w[KB * b + 4 * e + 1] = v.y, w[KB * b + 4 * e + 2] = v.z,
                           w[KB * b + 4 * e + 3] = v.w;
          }
        }
      }
    }
    if (axis0) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t v = lds4(src + sz + b * block);
        s[b] = __byte_perm(v, v, 0x1010);
        z[b] = __byte_perm(v, v, 0x3232);
      }
    }
    if (axis0) release_raw(bar, ring);
    if (!(u & 1) && !mbar_wait_warp(bar.k_empty + 8 * st, phase, abort)) return false;
    const uint32_t row = dst + st * kTileBytes + (u & 1) * kHalf;
    if (valid <= 0) {
      zero_row(row);
    } else if (axis0) {
      expand_row<KB, false, false>(w, row, kt & 7, [&](int, int pair, uint32_t& s2, uint32_t& z2) {
        s2 = s[pair >> 4];
        z2 = z[pair >> 4];
      });
      if (past_fp16<KB>(s, z)) limit_row(row);
    } else {
      // per-token keys: the (scale, zero) of each token, the same for a group's
      // channels (a second block that is not there leaves what the stage held:
      // its tokens are hidden)
      constexpr int per = 32 / KB;
      uint32_t t[per];
      expand_row<KB, false, true>(w, row, kt & 7, [&](int word, int pair, uint32_t& s2, uint32_t& z2) {
        const int i = pair % (per / 2);
        if (i == 0) {
          const uint32_t at = src + (word < KB ? tok + word * per * 4 * ng : tok2 + (word - KB) * per * 4 * ng);
          if (ng == 1) {
#pragma unroll
            for (int e = 0; e < per; e += 4) {
              const uint4 v = lds16(at + 4 * e);
              t[e] = v.x, t[e + 1] = v.y, t[e + 2] = v.z, t[e + 3] = v.w;
            }
          } else {
#pragma unroll
            for (int e = 0; e < per; ++e) t[e] = lds4(at + 4 * e * ng);
          }
        }
        const uint32_t a = t[code_at(2 * i, per)], c = t[code_at(2 * i + 1, per)];
        s2 = __byte_perm(a, c, 0x5410);
        z2 = __byte_perm(a, c, 0x7632);
      });
    }
    if (!axis0) release_raw(bar, ring);
    if (u & 1) {
      fence_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(bar.k_full + 8 * st);
      if (++st == kKStages) {
        st = 0;
        phase ^= 1u;
      }
    }
  }
  return true;
}

// Token of a 64-token part that value thread i of 64 expands. Eight lanes in a
// row read stored rows that differ in their last three bits and write places
// that do, so that neither the loads nor the stores conflict:
//  * key words of per codes: stored row (t % c) (T / c) + t / c, c = per / 2,
//    place 2 (t % c) + (t / c) % 2 (c = 2: t itself) in its group of per;
//  * 32-token blocks with 2-bit keys: their own order (vc_row).
__device__ __forceinline__ int value_token(int i, int kb, bool pair32) {
  const int l = i & 7, j = i >> 3;
  if (pair32) return 32 * (j >> 2) + 8 * (l >> 1) + (l & 1) + 2 * ((j + (l >> 2)) & 3);
  const int c = 16 / kb;
  return c * (l + 8 * (j / c)) + ((j + (kb == 8 ? l >> 2 : l >> 1)) & (c - 1));
}
// Value tiles of phase A: thread vt expands half vt / 64 (64 channels) of a
// token of a part, into the keys' token order.
template <int VB>
__device__ bool produce_values(const ChunkParams& p, const Item& it, uint32_t smem, const Bars& bar, int vt,
                               volatile int* abort) {
  const int parts = 2 * (min(it.k1, it.nA) - it.k0);
  if (parts <= 0) return true;
  const LayerView& L = p.L;
  const RawLayout raw(L);
  RawRing ring(raw.stages);
  const int per = 32 / L.k_bits, half = vt >> 6;
  const int tok = value_token(vt & 63, L.k_bits, pair_layout(L.group_k, L.k_bits));
  const int place = (tok & ~(per - 1)) + place_of(tok & (per - 1), per);
  // where its codes and scales sit in a stage
  const int TT = L.tile_tokens, t = tok & (TT - 1), ng = kD / L.group_v;
  const int tile = raw.tile + (TT == 32 && tok >= 32 ? (int)L.record_bytes : 0);
  const int crow = vc_row(t, TT, L.k_bits), x = chunk_swizzle(crow, VB);
  const int codes = tile + L.vc_off + crow * VB * 16;
  int sz[2], zo[2];  // scale and zero point of the half's 32-channel groups
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int g = (64 * half + 32 * e) / L.group_v;
    sz[e] = tile + L.vsz_off + 2 * vsz_half_index(t, g, TT, L.k_bits, ng, false);
    zo[e] = tile + L.vsz_off + 2 * vsz_half_index(t, g, TT, L.k_bits, ng, true);
  }
  int valid = it.q - (it.a0 + it.k0) * kTile - tok;  // > 0: the thread's token exists
  const uint32_t dst = smem + kVOff + half * kHalf + place * 128;
  int st = 0;
  uint32_t phase = 1;
#pragma unroll 1
  for (int u = 0; u < parts; ++u, valid -= 64, ring.next()) {
    if (!mbar_wait_warp(bar.raw_full + 8 * ring.stage, ring.parity, abort)) return false;
    const uint32_t src = smem + kRawOff + ring.stage * raw.bytes;
    uint32_t w[2 * VB], s[2], z[2];
#pragma unroll
    for (int e = 0; e < VB / 2; ++e) {
      const uint4 v = lds16(src + codes + (((half * (VB / 2) + e) ^ x) << 4));
      w[4 * e] = v.x, w[4 * e + 1] = v.y, w[4 * e + 2] = v.z, w[4 * e + 3] = v.w;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t a = lds2(src + sz[e]), b = lds2(src + zo[e]);
      s[e] = __byte_perm(a, a, 0x1010);
      z[e] = __byte_perm(b, b, 0x1010);
    }
    // (before the wait: with a single raw stage the keys of this tile may still
    // have to pass through it, and the product that frees a value stage is
    // issued after the next scores)
    release_raw(bar, ring);
    if (!(u & 1) && !mbar_wait_warp(bar.v_empty + 8 * st, phase, abort)) return false;
    const uint32_t row = dst + st * kTileBytes + (u & 1) * (64 * 128);
    if (valid <= 0) {
      zero_row(row);
    } else {
      expand_row<VB, true, false>(w, row, place & 7, [&](int, int pair, uint32_t& s2, uint32_t& z2) {
        s2 = s[pair >> 4];
        z2 = z[pair >> 4];
      });
      if (past_fp16<VB>(s, z)) limit_row(row);
    }
    if (u & 1) {
      fence_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(bar.v_full + 8 * st);
      if (++st == kVStages) {
        st = 0;
        phase ^= 1u;
      }
    }
  }
  return true;
}

// Key or value tiles of phase B: rows of exact tokens as they are (both
// operands take [64-channel half][token][128 bytes]). A tile of new tokens
// only is one TMA load per half; the others (sinks, ring, the chunk's end) are
// copied row by row, with zeros past the last token that a row sees.
// lost: of values, whose mixed tiles arrive at `look`; else null.
template <int STAGES>
__device__ bool produce_exact(const ChunkParams& p, const Item& it, uint32_t tiles, uint32_t full, uint32_t empty,
                              const Lost* lost, uint32_t look,
                              const void* sink, const void* ring, const void* fresh, const CUtensorMap* map, int kt,
                              volatile int* abort) {
  const LayerView& L = p.L;
  const int64_t unit = (int64_t)it.b * L.num_kv_heads + it.h;
  const int ch = kt & 15;
  const uint4* sink_p = reinterpret_cast<const uint4*>(sink) + unit * KVQ_MAX_SINKS * 16 + ch;
  const uint4* ring_p = reinterpret_cast<const uint4*>(ring) + unit * L.residual * 16 + ch;
  const uint4* new_p = reinterpret_cast<const uint4*>(fresh) + ((int64_t)it.off * L.num_kv_heads + it.h) * 16 + ch;
  const int64_t stride = (int64_t)L.num_kv_heads * 16;
  const int held = it.s + it.n, last = held + it.t1;
  const int slot0 = it.q % L.residual;  // ring slot of the first ring token
  uint32_t looks = 0;                   // bit st: parity of the mixed tiles so far in stage st
  auto tile_mbar_drain = [&](int n) {   // of the item's tile n, the last one in its stage
    const int k = it.k0 + n, st = n % STAGES;
    if (lost && k >= it.nA && lost->tile_b(k, it.nA) >= 0) mbar_drain(look + 8 * st, ((looks >> st) & 1u) ^ 1u);
    else mbar_drain(full + 8 * st, (n / STAGES) & 1);
  };
  for (int k = max(it.k0, it.nA); k < it.k1; ++k) {
    const int c = k - it.k0, st = c % STAGES, e0 = it.tile_b(k) * kTile;
    if (c >= STAGES && !mbar_wait_warp(empty + 8 * st, ((c / STAGES) - 1) & 1, abort)) {
      for (int n = c - STAGES; n < c; ++n) tile_mbar_drain(n);
      return false;
    }
    const bool mixed = lost && lost->tile_b(k, it.nA) >= 0;
    if (mixed) looks ^= 1u << st;
    const uint32_t dst = tiles + st * kTileBytes, bar = (mixed ? look : full) + 8 * st;
    if (e0 >= held && e0 - held + kTile <= p.e[it.i].t) {
      if ((kt & 31) == 0) {
        if (kt == 0) {
          mbar_expect_tx(bar, kTileBytes);
#pragma unroll
          for (int half = 0; half < 2; ++half)
            asm volatile(
                "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                ::"r"(dst + half * kHalf), "l"(map), "r"(it.h * kD + 64 * half), "r"(it.off + e0 - held), "r"(bar)
                : "memory");
        } else {
          mbar_arrive(bar);
        }
      }
      __syncwarp();
      continue;
    }
#pragma unroll 4
    for (int i = 0; i < kTile * 16 / kProducers; ++i) {
      const int row = (kt >> 4) + kProducers / 16 * i, e = e0 + row;
      const uint4* src;
      if (e >= held) {
        src = new_p + min(e - held, it.t1) * stride;
      } else if (e < it.s) {
        src = sink_p + e * 16;
      } else {
        int slot = slot0 + e - it.s;
        if (slot >= L.residual) slot -= L.residual;
        src = ring_p + slot * 16;
      }
      cp_async16(dst + (ch >> 3) * kHalf + row * 128 + (((ch & 7) ^ (row & 7)) << 4), src, e <= last);
    }
    asm volatile("cp.async.commit_group;\n cp.async.wait_group 0;" ::: "memory");
    fence_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  }
  // the last copies, in case of an abort: the block must not end under them
  // (else they have been waited for by the time that the others end)
  if (kt == 0)
    for (int n = max(max(it.k0, it.nA), it.k1 - STAGES) - it.k0; n < it.k1 - it.k0; ++n) tile_mbar_drain(n);
  return true;
}

// Warps 18 and 19 (x: thread of 64): the values of mixed tiles. Of a part of phase
// A (warp 18: whoever waits for a stage's phases must wait for each) the scales
// and zero points of tokens that are not finite become 0, before the value warps
// expand them; in a tile of phase B 16-byte pieces with values that are not finite
// do.
__device__ bool look_through(const ChunkParams& p, const Item& it, uint32_t smem, const Bars& bar, int x, Lost& lost,
                             volatile int* abort) {
  const LayerView& L = p.L;
  const int parts = 2 * (min(min(it.k1, it.nA), lost.a_end) - it.k0);
  if (x < 32 && parts > 0) {
    const RawLayout raw(L);
    RawRing ring(raw.stages);
    const int TT = L.tile_tokens, ng = kD / L.group_v;
    const bool order = vsz_operand_order(TT, L.k_bits);
    const int zero = order ? 8 : 2, next = order ? 16 : 4;  // bytes from a scale to its zero point, to the next group's
    uint32_t at[2];  // the first scale of tokens x and x + 32
#pragma unroll
    for (int e = 0; e < 2; ++e)
      at[e] = smem + kRawOff + raw.tile + L.vsz_off + (TT == 32 ? e * (int)L.record_bytes : 0) +
              2 * vsz_half_index(TT == 32 ? x : x + 32 * e, 0, TT, L.k_bits, ng, false);
#pragma unroll 1
    for (int u = 0; u < parts; ++u, ring.next()) {
      if (!mbar_wait_warp(bar.raw_look + 8 * ring.stage, ring.parity, abort)) return false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if ((it.a0 + it.k0) * kTile + 64 * u + x + 32 * e >= it.q) break;
        const uint32_t first = at[e] + ring.stage * raw.bytes;
        bool finite = true;
#pragma unroll 1
        for (uint32_t sz = first; sz < first + ng * next; sz += next) {
          if ((lds2(sz) & 0x7c00u) != 0x7c00u && (lds2(sz + zero) & 0x7c00u) != 0x7c00u) continue;
          asm volatile("st.shared.u16 [%0], %2;\n st.shared.u16 [%1], %2;" ::"r"(sz), "r"(sz + zero),
                       "h"((unsigned short)0)
                       : "memory");
          finite = false;
        }
        if (!finite) lost.note(lost.tile_a(it.k0 + (u >> 1)), 64 * (u & 1) + x + 32 * e);
      }
      fence_async_smem();  // (the stage is copied into again)
      __syncwarp();
      if (x == 0) mbar_arrive(bar.raw_full + 8 * ring.stage);
    }
  }
  // exponents of ones only carry into the sign bits
  const uint32_t one = L.kv_dtype == KVQ_BF16 ? 0x00800080u : 0x04000400u, exponents = 0x80008000u - one;
  uint32_t looks = 0;
#pragma unroll 1
  for (int k = max(it.k0, it.nA); k < it.k1; ++k) {
    const int tile = lost.tile_b(k, it.nA), st = (k - it.k0) % kVStages;
    if (tile < 0) continue;
    if (!mbar_wait_warp(bar.v_look + 8 * st, (looks >> st) & 1u, abort)) return false;
    looks ^= 1u << st;
    // (tokens past the item's last row too: a tile copied as a whole has them)
    const int rows = min(kTile, it.s + it.n + p.e[it.i].t - it.tile_b(k) * kTile);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const uint32_t first = smem + kVOff + st * kTileBytes + half * kHalf + (x & 7) * 16;
#pragma unroll 4
      for (int row = x >> 3; row < rows; row += 8) {
        const uint4 v = lds16(first + row * 128);
        const uint32_t a = ((v.x & exponents) + one) | ((v.y & exponents) + one);
        const uint32_t b = ((v.z & exponents) + one) | ((v.w & exponents) + one);
        if (((a | b) & 0x80008000u) == 0u) continue;
        sts16(first + row * 128, 0u, 0u, 0u, 0u);
        lost.note(tile, row);
      }
    }
    fence_async_smem();
    __syncwarp();
    if ((x & 31) < kProducers / 64) mbar_arrive(bar.v_full + 8 * st);  // for the four value warps
  }
  return true;
}

// ------------------------------------------------------------------- softmax
constexpr float kRsqrtD = (float)(1.0 / 11.313708498984761);  // 1 / sqrt(128)
// Radix-2 butterflies of one row held by one thread, then 1/sqrt(128): x . H.
__device__ __forceinline__ void rotate_row(float (&x)[kD]) {
#pragma unroll
  for (int w = 1; w < kD; w *= 2)
#pragma unroll
    for (int c = 0; c < kD; ++c)
      if ((c & w) == 0) {
        const float a = x[c], b = x[c + w];
        x[c] = a + b;
        x[c + w] = a - b;
      }
#pragma unroll
  for (int c = 0; c < kD; ++c) x[c] *= kRsqrtD;
}

// The warp's 32 query rows into its slot's A tile, two rows at a time (16 lanes
// with 8 channels each, so that loads are whole rows): phase A (fp16, times a
// power of two per row, rotated for a Hadamard cache) or phase B (as they are),
// with the sign of the softmax scale. Returns log2-units per score of the row
// of this lane.
__device__ __forceinline__ float load_queries(const ChunkParams& p, const Item& it, int first, uint32_t tile,
                                              int tile_row, bool phase_a) {
  const int lane = threadIdx.x & 31, ch = lane & 15, up = lane >> 4;
  const bool bf16 = p.L.kv_dtype == KVQ_BF16;
  const float scale = fabsf(p.scale_log2);
  const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
  float cs = fmaxf(scale, 1e-37f);  // never 0: a masked score is -inf times this
  const uint32_t dst = tile + (ch >> 3) * kHalf;
  auto chunk = [&](int i) {  // of row 2i + up
    const int row = tile_row + 2 * i + up;
    return dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
  };
  uint4 v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {  // all loads before any use
    const int r = first + 2 * i + up;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < it.rows) v[i] = __ldg(reinterpret_cast<const uint4*>(p.q) + it.row_of(p, r) * 16 + ch);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) sts16(chunk(i), v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
  if (phase_a) {
    // in place (a lane reads what it wrote); kept rolled: this runs once per
    // item, from a cold instruction cache
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const uint4 q = lds16(chunk(i));
      uint32_t w[4] = {q.x, q.y, q.z, q.w};
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 f;
        if (bf16) f = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
        else f = __half22float2(half2_of(w[e]));
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      if (p.L.hadamard) {
        // butterflies of half-width 1, 2, 4 in the lane, 8 .. 64 across the 16 lanes
#pragma unroll
        for (int d = 1; d < 8; d *= 2)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((e & d) == 0) {
              const float a = x[e], b = x[e + d];
              x[e] = a + b;
              x[e + d] = a - b;
            }
#pragma unroll
        for (int d = 1; d < 16; d *= 2)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y = __shfl_xor_sync(0xffffffffu, x[e], d);
            x[e] = (ch & d) ? y - x[e] : x[e] + y;
          }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= kRsqrtD;
      }
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
      for (int d = 1; d < 16; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      // the row's largest value to [8, 16)
      const int ex = mx > 0.f ? min(100, 3 - ((int)(__float_as_uint(mx) >> 23) - 127)) : 0;
      const float f = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack2<false>(x[2 * e] * f, x[2 * e + 1] * f);
      const float c = fmaxf(scale * __uint_as_float((uint32_t)(127 - ex) << 23), 1e-37f);
      const float c0 = __shfl_sync(0xffffffffu, c, 0), c1 = __shfl_sync(0xffffffffu, c, 16);
      if ((lane >> 1) == i) cs = (lane & 1) ? c1 : c0;
      sts16(chunk(i), w[0], w[1], w[2], w[3]);
    }
  }
  return cs;
}

// Bits [a, b) of a word (bounds outside 0 .. 32 are cut off).
__device__ __forceinline__ uint32_t bit_range(int a, int b) {
  const uint32_t below_b = b <= 0 ? 0u : b >= 32 ? 0xffffffffu : (1u << b) - 1u;
  const uint32_t below_a = a <= 0 ? 0u : a >= 32 ? 0xffffffffu : (1u << a) - 1u;
  return below_b & ~below_a;
}
// Bits in token order to the places of code_at: a perfect shuffle of each
// group of `per` bits (per = 4: none).
__device__ __forceinline__ uint32_t shuffle_bits(uint32_t x, int per) {
  auto swap = [&](uint32_t m, int d) {  // swaps the bits of m with those d above
    const uint32_t t = (x ^ (x >> d)) & m;
    x ^= t ^ (t << d);
  };
  if (per == 16) swap(0x00f000f0u, 4);
  if (per >= 8) {
    swap(0x0c0c0c0cu, 2);
    swap(0x22222222u, 1);
  }
  return x;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The state of one row's softmax.
struct RowState {
  float m = -INFINITY;  // a whole number, or -inf
  float l = 0.f;
};
// Packed probabilities 2^(s cs + bias) of 32 columns, added to sum.
template <bool BF16>
__device__ __forceinline__ void probabilities(const uint32_t* s, float cs, float bias, uint32_t* w,
                                              uint64_t (&sum)[4]) {
  const uint64_t cs2 = pair_of(cs, cs), b2 = pair_of(bias, bias);
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float a, b;
    unpair(fma2(pair_of(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), cs2, b2), a, b);
    a = ex2(a);
    b = ex2(b);
    sum[c & 3] = add2(sum[c & 3], pair_of(a, b));
    w[c] = pack2<BF16>(a, b);
  }
}
// Half a tile (64 columns, scores in s). The probabilities go by the m so far.
// Their sum tells whether that was good enough: below kMost none of them passes
// fp16's range. Else (always on a row's first tile, hardly ever later) m
// is raised to the maximum, what was written is rescaled and the half is
// computed again. Packed pairs go over the columns 32h .. of the scores already
// read.
template <bool BF16>
__device__ __forceinline__ void softmax_half(const uint32_t (&s)[64], int h, float cs, RowState& st, uint32_t tm_s,
                                             uint32_t tm_o, bool have_o) {
  uint32_t w[32];
  uint64_t sum[4] = {0, 0, 0, 0};
  float a, b;
  probabilities<BF16>(s, cs, kOffset - st.m, w, sum);
  probabilities<BF16>(s + 32, cs, kOffset - st.m, w + 16, sum);
  unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
  float l = a + b;
  // (a row that has seen nothing yet computed 2^(-inf + inf): again, as zeros)
  if (__any_sync(0xffffffffu, !(l < kMost) || st.m == -INFINITY)) {
    float top = __uint_as_float(s[0]);
#pragma unroll
    for (int c = 1; c < 63; c += 2) top = max3(top, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    top = fmaxf(top, __uint_as_float(s[63])) * cs;
    const float m = top > st.m ? ceilf(top) : st.m;
    const float f = m > st.m ? ex2(st.m - m) : 1.f;  // a power of two; 0 while m = -inf
    st.m = m;
    st.l *= f;
    const float bias = m == -INFINITY ? 0.f : kOffset - m;
    sum[0] = sum[1] = sum[2] = sum[3] = 0;
    probabilities<BF16>(s, cs, bias, w, sum);
    probabilities<BF16>(s + 32, cs, bias, w + 16, sum);
    unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
    l = a + b;
    // the slot's previous product is complete (its scores' barrier completed
    // after it), and so O is at rest; the tile's own probabilities so far too
    tmem_wait_st();
    if (have_o) {
#pragma unroll 1
      for (int c = 0; c < kD; c += 16) {
        uint32_t o[16];
        tmem_ld16(tm_o + c, o);
        tmem_wait_ld16(o);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st16(tm_o + c, o);
      }
    }
#pragma unroll 1
    for (int c = 0; c < 2 * h; ++c) {
      uint32_t o[16];
      tmem_ld16(tm_s + 16 * c, o);
      tmem_wait_ld16(o);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float2 x;
        if constexpr (BF16) x = make_float2(__uint_as_float(o[e] << 16), __uint_as_float(o[e] & 0xffff0000u));
        else x = __half22float2(half2_of(o[e]));
        o[e] = pack2<BF16>(x.x * f, x.y * f);
      }
      tmem_st16(tm_s + 16 * c, o);
    }
  }
  tmem_st32(tm_s + 32 * h, w);
  st.l += l;
}
// Scores whose bit is clear become -inf.
__device__ __forceinline__ void mask_chunk(uint32_t* s, uint32_t bits) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!((bits >> e) & 1u)) s[e] = 0xff800000u;
}
__device__ bool softmax_slot(const ChunkParams& p, const Item& it, int w, uint32_t smem, uint32_t tmem,
                             const Bars& bar, volatile int* abort) {
  const LayerView& L = p.L;
  const int row = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const int r = it.r0 + (it.both ? w * kRows : 0) + row;
  const int t = min(r, it.rows - 1) >> it.lg;  // the row's new token
  const bool bf16 = L.kv_dtype == KVQ_BF16;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t tm_s = tmem + lanes + kTmemS + w * kTile, tm_o = tmem + lanes + kTmemO + w * kD;
  const uint32_t qtile = smem + kQOff + w * kTileBytes;
  const int n = it.slot_tiles(w);
  RowState st;
  const int per = 32 / L.k_bits;  // key codes per word
  const int hi_b = it.s + it.n + t;                        // phase B: the row's own entry
  const int lo_b = p.window > 0 ? hi_b - p.window : -1;     // entries up to this are hidden
  const int lo_a = p.window > 0 ? it.q + it.n + t - p.window : -1;
  // tile-uniform: does any row of the item hide something of a tile?
  const int first_hi = it.s + it.n + it.t0, last_lo_b = p.window > 0 ? it.s + it.n + it.t1 - p.window : -1;
  const int last_lo_a = p.window > 0 ? it.q + it.n + it.t1 - p.window : -1;
  const uint32_t s_full = bar.s_full + 8 * w, p_ready = bar.p_ready + 8 * w;
  const int step = it.both ? 1 : 2, k_first = it.k0 + (it.both ? 0 : w);  // the slot's tiles: k_first, + step, ...
  const int tiles_a = min(n, max(0, (it.nA - k_first + step - 1) / step));
  bool have_o = false;
  uint32_t parity = 0;
#pragma unroll 1
  for (int ph = 0; ph < 2; ++ph) {
    const bool in_a = ph == 0;
    int left = in_a ? tiles_a : n - tiles_a;
    if (left == 0) continue;
    const float cs = load_queries(p, it, r & ~31, qtile, row & ~31, in_a);
    fence_async_smem();
    tc_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar.q_ready + 8 * w);
    // the tile's first position (phase A) or entry, and the next one's. A row
    // sees positions or entries in (lo, hi), and entries below `sinks`; all of
    // the item's rows see all of a tile that lies in (most_lo, least_hi).
    int k = k_first + (in_a ? 0 : tiles_a * step);
    int at = in_a ? (it.a0 + k) * kTile : it.tile_b(k) * kTile;
    const int lo = in_a ? lo_a : lo_b, hi = in_a ? it.q : hi_b + 1;
    const int most_lo = in_a ? last_lo_a : last_lo_b, least_hi = in_a ? it.q : first_hi + 1;
    const int sinks = in_a ? 0 : min(it.first_e, hi_b + 1);
    const bool half_type = in_a || !bf16;
#pragma unroll 1
    for (; left > 0; --left) {
      const bool masked = at + kTile > least_hi || at <= most_lo;
      if (!mbar_wait_warp(s_full, parity, abort)) return false;
      tc_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t s[64];
        tmem_ld32(tm_s + 64 * h, s);
        tmem_ld32(tm_s + 64 * h + 32, s + 32);
        tmem_wait_ld(s);
        tmem_wait_ld(s + 32);
        if (masked) {
#pragma unroll
          for (int e = 0; e < 64; e += 32) {
            const int c = at + 64 * h + e;
            const uint32_t bits = bit_range(lo + 1 - c, hi - c) | bit_range(0 - c, sinks - c);
            mask_chunk(s + e, in_a ? shuffle_bits(bits, per) : bits);
          }
        }
        if (half_type) softmax_half<false>(s, h, cs, st, tm_s, tm_o, have_o);
        else softmax_half<true>(s, h, cs, st, tm_s, tm_o, have_o);
      }
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(p_ready);
      have_o = true;
      parity ^= 1u;
      k += step;
      at = in_a ? at + step * kTile : it.tile_b(k) * kTile;
    }
    // every product of the phase in O (and done with the queries)
    if (!mbar_wait_warp(bar.o_done + 8 * w, in_a || tiles_a == 0 ? 0 : 1, abort)) return false;
    tc_after();
    if (in_a && L.hadamard) {  // O out of the rotated basis
      float x[kD];
#pragma unroll
      for (int c = 0; c < kD; c += 32) tmem_ld32(tm_o + c, reinterpret_cast<uint32_t*>(x) + c);
#pragma unroll
      for (int c = 0; c < kD; c += 32) tmem_wait_ld(reinterpret_cast<uint32_t*>(x) + c);
      rotate_row(x);
#pragma unroll
      for (int c = 0; c < kD; c += 32) tmem_st32(tm_o + c, reinterpret_cast<const uint32_t*>(x) + c);
      tmem_wait_st();
    }
  }
  // ---- the row's output or part: through the warp's share of the query tile
  // (8 KB, free now), so that stores are whole rows; 16-bit rows at once, fp32
  // ones in two halves of 64 channels
  const int lane = threadIdx.x & 31, first = r & ~31;
  const uint32_t mine = qtile + (row & ~31) * 256, to = mine + lane * 256;
  const bool parts = it.parts > 1 || p.slots > 0;
  const bool wide = parts || p.out_dtype == KVQ_F32, ob = p.out_dtype == KVQ_BF16;
  const int64_t rec0 = p.e[it.i].part0 + it.part + (it.both ? 0 : w);
  auto record = [&](int rr) {
    return rec0 + (p.slots > 0 ? it.row_of(p, rr) * p.slots : ((int64_t)it.h * it.rows + rr) * it.parts);
  };
  // (sum and output are 2^kOffset times those of the maximum m)
  if (parts && r < it.rows) p.ws_ml[record(r)] = make_float2(st.m - kOffset, st.l);
  const float f = parts ? 1.f : 1.f / st.l;  // every row sees its own token
  for (int half = 0; half < (wide ? 2 : 1); ++half) {
    __syncwarp();
#pragma unroll 1
    for (int c = 0; c < (wide ? 4 : 8); ++c) {  // 16 channels: a 16-byte chunk e at e ^ (lane % 16)
      uint32_t y[16];
      if (n > 0) {
        tmem_ld16(tm_o + 64 * half + 16 * c, y);
        tmem_wait_ld16(y);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
      if (wide) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sts16(to + (((4 * c + e) ^ (lane & 15)) << 4), y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
      } else {
        uint32_t z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = __uint_as_float(y[2 * e]), b = __uint_as_float(y[2 * e + 1]);
          z[e] = ob ? pack2<true>(a, b) : pack2<false>(a, b);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          sts16(to + (((2 * c + e) ^ (lane & 15)) << 4), z[4 * e], z[4 * e + 1], z[4 * e + 2], z[4 * e + 3]);
      }
    }
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int l = 2 * i + (lane >> 4), rr = first + l, c = lane & 15;
      const uint4 v = lds16(mine + l * 256 + ((c ^ (l & 15)) << 4));
      if (rr >= it.rows) continue;
      if (parts) reinterpret_cast<uint4*>(p.ws_o + record(rr) * kD + 64 * half)[c] = v;
      else if (wide)
        reinterpret_cast<uint4*>(static_cast<float*>(p.out) + it.row_of(p, rr) * kD + 64 * half)[c] = v;
      else reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + it.row_of(p, rr) * kD)[c] = v;
    }
  }
  return true;
}

// Shared-memory descriptors: start >> 4, leading and stride byte offsets >> 4,
// version 1 (bit 46), 128-byte swizzle (2 at bit 61). K-major tiles: rows of
// 64 k-elements (128 bytes), 8-row groups 1024 bytes apart. MN-major tiles:
// rows of 64 mn-elements, one k each, 8-k groups 1024 bytes apart and the
// second 64 mn-elements kHalf further. They differ in the low word only.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride, version, swizzle
constexpr uint32_t kDescK = 1u << 16, kDescMn = (uint32_t)(kHalf >> 4) << 16;  // leading offset
// The eight k-steps of one slot's scores (MN: expanded keys, else exact ones)
// and of its product with the values.
template <bool MN>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t q_lo, uint32_t k_lo, uint32_t id) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    constexpr int kStep = 2048 >> 4;
    const int step = ((e >> 2) * kHalf + (e & 3) * 32) >> 4;
    mma_ss(d, desc_of(q_lo + step, kDescHi), desc_of(k_lo + (MN ? e * kStep : step), kDescHi), id, e > 0);
  }
}
__device__ __forceinline__ void issue_values(uint32_t d, uint32_t p, uint32_t v_lo, uint32_t id, bool acc) {
#pragma unroll
  for (int e = 0; e < 8; ++e) mma_ts(d, p + 8 * e, desc_of(v_lo + e * (2048 >> 4), kDescHi), id, acc || e > 0);
}

// One warp issues every product of the item (by one elected lane; the warp
// walks the loop together, so that descriptors are warp-uniform values), in the
// order S(0), S(1), then
// P V of step v and S of step v + 2: a slot's next scores are queued behind
// its own product (which reads the P they overwrite) while the other slot's
// softmax runs. The tensor cores idle while this thread does anything else, so
// a step is kept short: what it needs is counted, not worked out. (One warp per
// slot lets the slots fall into step with each other: 12% slower.)
__device__ bool issue_products(const ChunkParams& p, const Item& it, uint32_t smem, uint32_t tmem, const Bars& bar,
                               volatile int* abort) {
  const int steps = it.steps();
  const bool leader = elect_one();
  const bool bf16 = p.L.kv_dtype == KVQ_BF16, both = it.both;
  const uint32_t q_lo = ((smem + kQOff) >> 4) | kDescK;
  const uint32_t k_base = (smem + kKOff) >> 4, v_lo = ((smem + kVOff) >> 4) | kDescMn;
  const uint32_t id_a = inst_desc(false, true), id_bk = inst_desc(bf16, false), id_bv = inst_desc(bf16, true);
  constexpr uint32_t kTileLo = kTileBytes >> 4;
  static_assert(kKStages == 2 && kVStages == 2, "stages are counted in one bit");
  const int first_b = it.nA - it.k0;  // tiles of the item before phase B
  // tile n of the item (counted from k0) sits in stage n % 2, in phase n / 2
  auto scores = [&](int w, int n) {
    const uint32_t lo = k_base + (n & 1) * kTileLo, d = tmem + kTmemS + w * kTile, q = q_lo + w * kTileLo;
    if (n < first_b) {
      if (leader) issue_scores<true>(d, q, lo | kDescMn, id_a);
    } else {
      if (leader) issue_scores<false>(d, q, lo | kDescK, id_bk);
    }
    if (leader) tc_commit(bar.s_full + 8 * w);
    if (leader && (!both || w == 1)) tc_commit(bar.k_empty + 8 * (n & 1));
    __syncwarp();
  };
  for (int v = 0; v < 2 && v < steps; ++v) {
    const int n = both ? 0 : v;
    if (!mbar_wait_warp(bar.q_ready + 8 * v, 0, abort)) return false;
    if (!mbar_wait_warp(bar.k_full + 8 * (n & 1), 0, abort)) return false;
    tc_after();
    scores(v, n);
  }
  int n = 0;  // tile of step v; the slot's next tile is n + ahead
  const int ahead = both ? 1 : 2;
#pragma unroll 1
  for (int v = 0; v < steps; ++v) {
    const int w = v & 1, next = n + ahead;
    const bool more = v + 2 < steps;
    // a slot that enters phase B rewrites its query only after this product
    const bool enter_b = more && next >= first_b && n < first_b;
    if (!both || w == 0) {
      if (!mbar_wait_warp(bar.v_full + 8 * (n & 1), (n >> 1) & 1, abort)) return false;
      if (more && !mbar_wait_warp(bar.k_full + 8 * (next & 1), (next >> 1) & 1, abort)) return false;
    }
    if (!mbar_wait_warp(bar.p_ready + 8 * w, (v >> 1) & 1, abort)) return false;
    tc_after();
    const uint32_t od = tmem + kTmemO + w * kD, op = tmem + kTmemS + w * kTile, ov = v_lo + (n & 1) * kTileLo;
    const uint32_t id = n < first_b ? id_a : id_bv;
    if (leader) {
      issue_values(od, op, ov, id, v > 1);
      if (!more || enter_b) tc_commit(bar.o_done + 8 * w);  // the slot's last product of the phase
    }
    if (leader && (!both || w == 1)) tc_commit(bar.v_empty + 8 * (n & 1));
    __syncwarp();
    if (more) {
      if (enter_b) {
        if (!mbar_wait_warp(bar.q_ready + 8 * w, 1, abort)) return false;
        tc_after();
      }
      scores(w, next);
    }
    n += both ? w : 1;
  }
  return true;
}

// After all else, where values were left out: thread x of 256 makes its row NaN
// (its output, or the sum of its part) if it sees one of them.
// (The softmax has all that this works out again, and no registers to keep it:
// there it cost 16 x 5 tokens over 8192 15 us.)
__device__ __forceinline__ void lose_row(const ChunkParams& p, const Lost& lost, int x) {
  const Item it = find_item(p, blockIdx.x);
  const int w = x >> 7, r = it.r0 + (it.both ? x : x & 127);
  if (r >= it.rows) return;
  const int t = r >> it.lg, hi_b = it.s + it.n + t, sinks = min(it.first_e, hi_b + 1);
  const int lo_a = p.window > 0 ? it.q + it.n + t - p.window : -1, lo_b = p.window > 0 ? hi_b - p.window : -1;
  bool sees = false;
  for (int k = it.k0; k < it.k1 && !sees; ++k) {
    const bool in_a = k < it.nA;
    const int tile = in_a ? lost.tile_a(k) : lost.tile_b(k, it.nA);
    for (int e = 0; e < 4 && tile >= 0; ++e) {
      const int c = (in_a ? it.a0 + k : it.tile_b(k)) * kTile + 32 * e;
      const uint32_t seen = in_a ? bit_range(lo_a + 1 - c, it.q - c)
                                 : bit_range(lo_b + 1 - c, hi_b + 1 - c) | bit_range(0 - c, sinks - c);
      sees = sees || (lost.bits[4 * tile + e] & seen) != 0u;
    }
  }
  if (!sees) return;
  const float nan = __int_as_float(0x7fffffff);
  if (it.parts > 1) {
    p.ws_ml[p.e[it.i].part0 + it.part + (it.both ? 0 : w) + ((int64_t)it.h * it.rows + r) * it.parts].y = nan;
    return;
  }
  const int64_t at = it.row_of(p, r) * kD;
  for (int c = 0; c < kD; ++c) {
    if (p.out_dtype == KVQ_F32) static_cast<float*>(p.out)[at + c] = nan;
    else static_cast<uint16_t*>(p.out)[at + c] = 0x7fffu;  // NaN in both types
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    chunk_tc_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ ChunkMaps maps) {
  extern __shared__ uint8_t raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ Lost s_lost;
  const uint32_t smem = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  volatile int* abort = &s_abort;
  Bars bar;
  {
    uint32_t at = smem + kBarOff;
    bar.k_full = at, at += 8 * kKStages;
    bar.k_empty = at, at += 8 * kKStages;
    bar.v_full = at, at += 8 * kVStages;
    bar.v_empty = at, at += 8 * kVStages;
    bar.s_full = at, at += 16;
    bar.p_ready = at, at += 16;
    bar.o_done = at, at += 16;
    bar.q_ready = at, at += 16;
    bar.raw_full = at, at += 8 * kRawStages;
    bar.raw_empty = at, at += 8 * kRawStages;
    bar.raw_look = at, at += 8 * kRawStages;
    bar.v_look = at, at += 8 * kVStages;
    bar.drain = at;
  }
  // the merge of the parts may be scheduled (it waits for this grid before it
  // reads): 2 us of 123 for 300 new tokens
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Item it = find_item(p, blockIdx.x);
  if (warp == 17) {  // a barrier per lane
    const int lane = threadIdx.x & 31;
    const uint32_t at = smem + kBarOff + 8 * lane;
    auto in = [&](uint32_t first, int n) { return at >= first && at < first + 8 * n; };
    // arrivals: of the key or value warps, of a slot's warps, of one thread or a commit
    const bool produced = in(bar.k_full, kKStages) || in(bar.v_full, kVStages) || in(bar.v_look, kVStages);
    const bool slot = in(bar.p_ready, 2) || in(bar.q_ready, 2), raw_empty = in(bar.raw_empty, kRawStages);
    if (8 * lane < kBarBytes) mbar_init(at, produced ? kProducers / 32 : slot ? 4 : raw_empty ? kProducers / 16 : 1);
    if (lane == 0) {
      s_abort = 0;
      s_lost.set(p, it);
    }
    for (int e = lane; e < 4 * kMixed; e += 32) s_lost.bits[e] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = s_tmem;
  const LayerView& L = p.L;
  const int kt = ((warp >> 2) & 1) * 64 + (threadIdx.x & 63);  // of 128 key or value threads
  // (all warps of a warpgroup must execute the same setmaxnreg: it comes before
  // the key and value warps of a group part)
  const int group = warp >> 2;
  if (group < 2) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    (void)softmax_slot(p, it, group, smem, tmem, bar, abort);
  } else if (group < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (!(warp & 2)) {
      const bool ok = L.k_bits == 2   ? produce_keys<2>(p, it, smem, bar, kt, abort)
                      : L.k_bits == 4 ? produce_keys<4>(p, it, smem, bar, kt, abort)
                                      : produce_keys<8>(p, it, smem, bar, kt, abort);
      if (ok)
        (void)produce_exact<kKStages>(p, it, smem + kKOff, bar.k_full, bar.k_empty, nullptr, 0u, L.sink_k, L.ring_k, p.k,
                                      &maps.k, kt, abort);
    } else {
      const bool ok = L.v_bits == 2   ? produce_values<2>(p, it, smem, bar, kt, abort)
                      : L.v_bits == 4 ? produce_values<4>(p, it, smem, bar, kt, abort)
                                      : produce_values<8>(p, it, smem, bar, kt, abort);
      if (ok)
        (void)produce_exact<kVStages>(p, it, smem + kVOff, bar.v_full, bar.v_empty, &s_lost, bar.v_look, L.sink_v, L.ring_v,
                                      p.v, &maps.v, kt, abort);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 16) {
      (void)issue_products(p, it, smem, tmem, bar, abort);
      // let the products in flight finish before the tensor memory goes,
      // whoever gave up and when
      if (elect_one()) tc_commit(bar.drain);
      __syncwarp();
      mbar_drain(bar.drain, 0);
      __syncwarp();
    }
    if (warp == 17 && (threadIdx.x & 31) == 0) (void)copy_parts(p, it, smem, bar, s_lost, abort);
    if (warp >= 18) (void)look_through(p, it, smem, bar, threadIdx.x & 63, s_lost, abort);
    __syncwarp();
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 16)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  if (threadIdx.x == 0 && s_abort) atomicOr(p.err, 1);
  if (s_lost.any && threadIdx.x < 2 * kRows) lose_row(p, s_lost, threadIdx.x);
}

// Merges the parts of a row (parts > 1): a warp per row, four channels a lane.
constexpr int kCombineWarps = 8;
__global__ void __launch_bounds__(32 * kCombineWarps) chunk_combine_kernel(const __grid_constant__ ChunkParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t g = (int64_t)blockIdx.x * kCombineWarps + (threadIdx.x >> 5);
  if (g >= p.merge_rows) return;
  const int i = p.entry_of_merge((int)g), ngr = p.num_q_heads / p.L.num_kv_heads, rows = p.e[i].t * ngr;
  const int parts = chunk_parts(p.e[i].splits);
  const int64_t x = g - p.e[i].merge0;  // h * rows + r
  const int64_t rec = p.e[i].part0 + x * parts;
  float M = -INFINITY;
  for (int e = lane; e < parts; e += 32) M = fmaxf(M, p.ws_ml[rec + e].x);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int e = 0; e < parts; ++e) {
    const float2 ml = p.ws_ml[rec + e];
    const float4 v = reinterpret_cast<const float4*>(p.ws_o + (rec + e) * kD)[lane];
    const float f = ex2(ml.x - M);  // 0 for a part that saw nothing
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
    l = fmaf(f, ml.y, l);
  }
  const float f = 1.f / l;
  const int h = (int)(x / rows), r = (int)(x % rows);
  const int64_t at = ((int64_t)(p.e[i].off + r / ngr) * p.num_q_heads + h * ngr + r % ngr) * kD + 4 * lane;
  if (p.out_dtype == KVQ_F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) =
        make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
  } else {
    const bool ob = p.out_dtype == KVQ_BF16;
    const uint32_t a = ob ? pack2<true>(acc.x * f, acc.y * f) : pack2<false>(acc.x * f, acc.y * f);
    const uint32_t c = ob ? pack2<true>(acc.z * f, acc.w * f) : pack2<false>(acc.z * f, acc.w * f);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at) = make_uint2(a, c);
  }
}

}  // namespace

namespace {

// cuTensorMapEncodeTiled, looked up once (the runtime is the only library
// linked).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

cudaError_t make_map(CUtensorMap& m, const ChunkParams& p, const void* data) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)p.L.num_kv_heads * kD, (cuuint64_t)p.tokens};
  const cuuint64_t strides[1] = {(cuuint64_t)p.L.num_kv_heads * kD * 2};
  const cuuint32_t box[2] = {64, kTile}, one[2] = {1, 1};
  const CUtensorMapDataType t =
      p.L.kv_dtype == KVQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUresult r = encode(&m, t, 2, const_cast<void*>(data), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

bool chunk_tc_supported(const LayerView& L) { return L.residual_v == L.residual; }

cudaError_t launch_chunk_tc(const ChunkParams& p, cudaStream_t stream) {
  if (p.items <= 0) return cudaSuccess;
  // a build whose launch brings fewer registers would wait for them forever
  static std::atomic<bool> checked{false};
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, chunk_tc_kernel);
    if (e != cudaSuccess) return e;
    if (a.numRegs < kLaunchRegisters) return cudaErrorLaunchOutOfResources;
    checked.store(true, std::memory_order_relaxed);
  }
  ChunkMaps maps;
  cudaError_t e = make_map(maps.k, p, p.k);
  if (e == cudaSuccess) e = make_map(maps.v, p, p.v);
  if (e != cudaSuccess) return e;
  // (set on every launch: it is per device, and a few hundred nanoseconds)
  e = cudaFuncSetAttribute(chunk_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  chunk_tc_kernel<<<p.items, kThreads, kSmemBytes, stream>>>(p, maps);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.merge_rows == 0) return e;
  const unsigned merges = (unsigned)((p.merge_rows + kCombineWarps - 1) / kCombineWarps);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(merges);
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_combine_kernel, p);
}

}  // namespace kvq
