// attn_core.cuh — the attention pipeline shared by the prompt kernel and the paged tree
// kernel: o = softmax(scale q k^T) v over tiles of 128 keys, on 5th-generation tensor cores.
//
// A work item is (sequence, key/value head, block of query rows); a query row is
// (token, query head of the group), row = token * G + g, so that all G = H_q / H_kv heads
// that read a key/value head share its tiles.  A block holds up to two row tiles of 128
// rows, and every key and value tile is read once for both.  384 threads, one CTA per SM
// (TMEM):
//   warps 0-3, 4-7  softmax of pipeline 0 and 1: one thread per row (= TMEM lane)
//   product warps   issue the tensor-core products: one, with heads up to 64 one per pipeline
//   copy warp       work list, tensor copies (TMA)
//   fix warps       the other two (one): value rows of partly visible tiles (below), masks of
//                   trees, outputs of sequences without work
// The roles run over the work list as one stream of key tiles: the next item's copies and
// first score products go out while the current one finishes.
//
//   S_t = Q_t K^T   (tcgen05.mma, both operands in shared memory; 128 fp32 TMEM columns)
//   P_t = 2^(c S_t - c m), c = scale log2(e)   (16-bit pairs over S_t's own columns)
//   O_t += P_t V    (A from TMEM, V as the MN-major operand)
// with a running row maximum m that moves (and rescales O_t and the sum) only when a tile
// exceeds it by more than e^8: P stays below e^8, far inside fp16's range, and O and the
// row sum stay in fp32.  P is rounded to the io type because that is what the second
// product takes; the sum adds the values before that rounding.  While one pipeline's
// softmax runs, the tensor core works for the other.
//
// What bounds it.  d = 128: the tensor core.  A 128-key step of both pipelines is 32
// instructions of 64 cycles (2048) and measures 2724: P lies over S, so S_t waits until
// P_t V is done, twice a step, and the product warp's own instructions fill the rest (a
// 32768-token prompt, 16 heads over 4: 2.6-2.8 ms call after call, where the power cap sets the
// clock, 1570-1690 TFLOP/s, 80-86% of the measured library burst and 90-97% of its sustained
// rate; 2.40 ms for the first few calls at full clock).  Heads up to 64: the softmax; 32,768 exponentials are 1024 cycles a step and the
// whole of it ~2400, against 1280 of products.  There P has columns of its own, the next
// S_t goes out as soon as the threads hold the last one, and two product warps keep up with
// the shorter products (8192 tokens, 16 heads: 174 -> 147 us).  Tried and slower: two
// threads per row, 64-key half steps, narrower tensor-memory loads with 16 warps, two
// product warps at d = 128, uneven register shares.
//
// A lone row tile leaves pipeline 1 idle; with ALT its key tiles go to both pipelines in
// turn (two partial softmaxes of the same rows), which the epilogue joins: pipeline 1 hands
// its maximum and sum over, gets both weights back, and each writes half of the columns.
//
// Value rows that no row of the item may see.  A product cannot skip them: 0 x NaN is NaN.
// The fix warps therefore zero the rows past the visible keys of a tile (the end of a
// sequence, stale positions of a page) before the product reads it, and in tiles where the
// mask differs from row to row they replace non-finite values by zero and raise the item's
// `dirty` flag; the epilogue then adds those values to just the rows that see them.  Such
// tiles land on barriers of the fix warps' own: a warp that only sees some of the tiles
// could not tell a ring slot's phase from the one after next.
//
// Every wait is bounded.  On expiry the CTA stops and marks the sequences of all its items from
// the first one that its softmax warps have not all put out, those known ahead and those still
// to come among them, TGDN_SEQ_TIMEOUT.
#pragma once

#include <cuda_fp16.h>

#include "launch_after.cuh"
#include "tgdn_device.cuh"
#include "tgdn_kernels.h"

namespace tgdn {
namespace attn {

constexpr int kKeys = 128;   // keys per tile
constexpr int kRows = 128;   // query rows per row tile
constexpr int kBlock = 384;
constexpr int kMmaWarp = 8;  // (the first after the softmax warps)
constexpr int kRing = 4;     // work items known ahead
constexpr int kFixRing = 4;  // value tiles being made safe (at most 4 value tiles are in flight)
constexpr float kGap = 8.f;  // lazy rescaling threshold (natural log units)
constexpr uint32_t kTmemCols = 512;  // S_0, S_1 (128 each), O_0, O_1 (128 each)
constexpr int kMaxNodes = TGDN_MAX_NODES;

// Shared-memory layout for heads padded to DP = 64, 96 or 128 elements (96: 8192 tokens with
// d = 96 155 us after 186 as 128; tiles are laid out as for 128).
template <int DP, bool PAGED>
struct Lay {
  static constexpr int kHalves = (DP + 63) / 64;               // 128-byte swizzled halves of a row
  static constexpr int kHalf = kKeys * 128;             // one half of a tile
  static constexpr int kTile = kHalf * kHalves;         // a key, value or query tile
  // key and value tiles in flight: what shared memory holds (paged: beside the masks)
  static constexpr int kStages = DP == 64 ? 8 : PAGED ? 4 : 5;
  static constexpr int kOffKV = 2 * kTile;              // (the two query tiles come first)
  static constexpr int kOffMisc = kOffKV + kStages * kTile;
  // tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (DP each), and P over its own S, or
  // apart where it fits
  static constexpr bool kApart = DP == 64;
  static constexpr uint32_t kColO = 256, kColP = kApart ? 256 + 2 * DP : 0;
  static constexpr uint32_t kStepP = kApart ? 64 : 128;  // columns between P_0 and P_1
  // warps: with P apart a product warp for each row tile (short products: one warp's own
  // instructions would set the pace), else one for both, which keeps them half a step apart
  static constexpr int kMmaWarps = kApart ? 2 : 1;
  static constexpr int kCopyWarp = kMmaWarp + kMmaWarps, kFixWarp = kCopyWarp + 1;
  static constexpr int kFixWarps = kBlock / 32 - kFixWarp;
};

constexpr int kAltTiles = 2;  // key tiles from which pipelines alternate (4: 1 prompt of 300 tokens 9.5 us after 9.0)

// One piece of work: key tiles [u0, u1) of an item.
struct Seg {
  int b, lo, N;      // sequence, its first row, its rows (tokens or nodes); b < 0: no more work
  int tok0, hk;      // first token of row tile 0; key/value head
  int e0, e1;        // row tile t takes tiles [u0, e_t); e_t <= u0: it has none
  int u0, u1;
  int P, npre;       // cached positions and their tiles (paged)
  int part;          // -1: the whole item; else this CTA's partial-result slot
  int zero;          // the sequence came with an error: its outputs are zeros
  int alt;           // one row tile: its key tiles go to the two pipelines in turn
  __device__ void set_alt() { alt = e1 <= u0 && u1 - u0 >= kAltTiles; }
};

struct Args {
  int B, T, H_q, H_kv, G, d, tpt;  // tpt: tokens per row tile = 128 / G
  int gbox;                        // bytes of one half of a query box: 128 * G * tpt
  float scale;
  const int32_t* cu;
  int32_t* status;
  void* o;
  int64_t o_stride;                // elements between tokens
  int o_wide;                      // every row and head of o on a 32-byte boundary
  const void* v;                   // new rows' values (prompt or tree), for the rare exact path
  int64_t v_stride;
  // paged
  int n_max, ps, n_pages, max_pages;
  const int32_t *parent, *table, *len, *held;
  int tiles;                       // row tiles per item: 2, or 1 when items are few
  // partial results (null: items are never split): [slot][DP / 4][part_rows] float4 of O
  // unnormalised, [slot][part_rows] of (reference maximum in log2 units, sum)
  float* part;
  float2* part_ml;
  int4* desc;                      // [grid][2]: the split item that begins in a CTA's range
  int part_rows;                   // rows per partial slot
  int min_share;                   // least key tiles per CTA
  int runs, joins;                 // CTAs of the attention kernel; of a narrow join per row group
  int hold_b, hold_h;              // sequence and head whose queries never come (test hook), or -1
  uint64_t wait_ns;                // limit of the copy warp's waits
};
// (hold_* and wait_ns of Args; a limit for every wait, read from memory, took registers from all
// the roles: 16 uneven prompts 152 -> 161 us, mixed trees 222 -> 236)
static void set_hooks(Args& a) {
  const WaitHooks h = wait_hooks();
  a.hold_b = h.hold_item < 0 ? -1 : h.hold_item / a.H_kv;
  a.hold_h = h.hold_item < 0 ? -1 : h.hold_item % a.H_kv;
  a.wait_ns = h.wait_ns ? h.wait_ns : kWaitLimitNs;
}
__device__ __forceinline__ void timed_out(const Args& a, int b) {
  atomicCAS(&a.status[b], TGDN_SEQ_OK, TGDN_SEQ_TIMEOUT);
}

// (o_wide of Args)
static int wide_rows(const void* o, int64_t stride, int d) {
  return reinterpret_cast<uintptr_t>(o) % 32 == 0 && stride % 16 == 0 && d % 16 == 0;
}

template <typename E> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kFmt = 1, kExp = 0x7f807f80u, kStep = 0x00800080u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
};
template <> struct Elem<__half> {
  static constexpr uint32_t kFmt = 0, kExp = 0x7c007c00u, kStep = 0x04000400u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
};

// Instruction descriptor, fp32 accumulation; bf16 or fp16 operands of one type.
__host__ __device__ constexpr uint32_t idesc(uint32_t fmt, int M, int N, int b_mn) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 columns of this thread's lane and their maximum (NaN values are passed over).
__device__ __forceinline__ void ld_max32(uint32_t at, float* r, float& top) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
        "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
        "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31]), "=f"(top)
      : "r"(at)
      : "memory");
}
// Until this thread's tensor-memory loads are complete; the operands keep every use of the
// loaded registers behind the wait.
__device__ __forceinline__ void ld_wait32(float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]),
                 "+r"(u[6]), "+r"(u[7]), "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]),
                 "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15]), "+r"(u[16]), "+r"(u[17]),
                 "+r"(u[18]), "+r"(u[19]), "+r"(u[20]), "+r"(u[21]), "+r"(u[22]), "+r"(u[23]),
                 "+r"(u[24]), "+r"(u[25]), "+r"(u[26]), "+r"(u[27]), "+r"(u[28]), "+r"(u[29]),
                 "+r"(u[30]), "+r"(u[31])
               :
               : "memory");
}

// Bounded wait.  What is not there at once is awaited out of line: the roles' loops compete
// for the instruction cache.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_wait_suspend(bar, parity, abort);
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try(bar, parity) || wait_slow(bar, parity, abort);
}

// The copy warp's, whose limit a test can shorten.
static __device__ __noinline__ bool wait_copies_slow(uint64_t* bar, uint32_t parity,
                                                     volatile int* abort, uint64_t limit_ns) {
  return mbar_wait_suspend(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool wait_copies(uint64_t* bar, uint32_t parity, volatile int* abort,
                                            uint64_t limit_ns) {
  return mbar_try(bar, parity) || wait_copies_slow(bar, parity, abort, limit_ns);
}

// The product warp's waits and arrivals take shared-memory addresses (its own instructions
// set the pace of short steps).
__device__ __forceinline__ bool try_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
static __device__ __noinline__ bool wait_slow_at(uint32_t bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = global_ns();
  while (!try_at(bar, parity)) {
    if (*abort) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// Two-wide fp32 arithmetic and the three-input maximum (NaN operands are passed over).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A value that all lanes of the warp hold, so that code depending on it is compiled as
// warp-uniform (addresses and descriptors in uniform registers).
__device__ __forceinline__ int uniform(int x, int from = 0) {
  return __shfl_sync(0xffffffffu, x, from);
}

// Tensor-core instructions of a convergent warp, issued by its elected lane (the same lane
// every time).  Elected in place, four to an asm block with the descriptors' low words added
// up inside, an instruction costs its 64 cycles also beside busy warps; under a branch or a
// predicate computed from the lane number the same instructions took ~92.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 1024-byte stride, 128B swizzle
// D = A B over four k-steps of 16 elements (64 elements: one 128-byte half of both tiles), or
// D += A B with add.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint32_t a, uint32_t b, uint32_t id,
                                        uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 u, v;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t"
      "add.u32 u, %1, 2;\n\tadd.u32 v, %2, 2;\n\tmov.b64 x, {u, %5};\n\tmov.b64 y, {v, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u32 u, %1, 4;\n\tadd.u32 v, %2, 4;\n\tmov.b64 x, {u, %5};\n\tmov.b64 y, {v, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u32 u, %1, 6;\n\tadd.u32 v, %2, 6;\n\tmov.b64 x, {u, %5};\n\tmov.b64 y, {v, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(add), "r"(kDescHi)
      : "memory");
}
// Two k-steps of them, D += A B.
__device__ __forceinline__ void mma_ss2(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
  asm volatile(
      "{\n\t.reg .pred t, e;\n\t.reg .b32 u, v;\n\t.reg .b64 x, y;\n\t"
      "setp.eq.b32 t, %3, %3;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.u32 u, %1, 2;\n\tadd.u32 v, %2, 2;\n\tmov.b64 x, {u, %4};\n\tmov.b64 y, {v, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(kDescHi)
      : "memory");
}
// Four over 64 keys with A (16-bit pairs, 8 columns per k-step) in tensor memory and B
// MN-major (2048 bytes per k-step).
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint32_t b, uint32_t id,
                                        uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 u, v;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t"
      "add.u32 u, %1, 8;\n\tadd.u32 v, %2, 128;\n\tmov.b64 y, {v, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t"
      "add.u32 u, %1, 16;\n\tadd.u32 v, %2, 256;\n\tmov.b64 y, {v, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t"
      "add.u32 u, %1, 24;\n\tadd.u32 v, %2, 384;\n\tmov.b64 y, {v, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, t;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(add), "r"(kDescHi)
      : "memory");
}
// Arrives on the barrier once every tensor-core instruction of that lane so far is complete.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// A tensor copy by the elected lane of a convergent warp (26 cycles each; from a branch over
// lanes 51, and then 16 boxes of 16 positions took longer than the products on them).
__device__ __forceinline__ void copy_box(uint32_t to, const CUtensorMap* map, uint32_t bar, int x,
                                         int y, int z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(to),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void st_global32(void* to, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
struct alignas(16) Bars {
  uint64_t kvfull[8], kvempty[8];
  uint64_t qfull, qempty, drain[2];
  uint64_t sfull[2], sread[2], pready[2][2], pvdone[2];
  uint64_t partfull[kFixRing], fixed[kFixRing];
  uint64_t maskfull[2], maskempty[2];
  uint64_t alt_in, alt_back, alt_done;
  uint64_t stolen;
  uint64_t segfull[kRing], segempty[kRing];
  uint4 steal;  // the answer to a request for another CTA's work
  float2 alt_ml[kRows];  // row maximum and sum of pipeline 1; then the weights of both
  Seg seg[kRing];
  int dirty[kRing], bad[kRing];
  uint32_t tmem;
  int abort;
  int taken, put_out[8];  // at the end: items taken on; items each softmax warp is done with
};

// Paged: ancestor-or-self sets of an item's nodes (node-index space), two items' worth, and a
// copy of the parents for each warp that builds them.
constexpr int kMaskWords = kMaxNodes / 32;
constexpr int kMaskBytes = 2 * 2 * kRows * kMaskWords * 4;
static_assert(sizeof(Bars) % 16 == 0, "the masks behind it are read 16 bytes at a time");

template <int DP, bool PAGED>
constexpr int smem_bytes() {
  return Lay<DP, PAGED>::kOffMisc + (int)sizeof(Bars) + (PAGED ? kMaskBytes + 4 * kMaxNodes : 0) + 1024;
}
static_assert(smem_bytes<128, true>() <= 227 * 1024 && smem_bytes<128, false>() <= 227 * 1024,
              "fits one CTA per SM");

// ------------------------------------------------------------------ masks and the rare path
// Whether tile u needs the value check, its visible rows, and whether the mask differs by row.
template <bool PAGED>
__device__ __forceinline__ bool tile_part(const Seg& s, int u, int& lim, bool& by_row) {
  if (PAGED) {
    if (u < s.npre) {
      lim = min(kKeys, s.P - u * kKeys);
      by_row = false;
      return lim < kKeys;
    }
    lim = min(kKeys, s.N - (u - s.npre) * kKeys);
    by_row = s.N > 1;
    return true;
  }
  lim = min(kKeys, s.N - u * kKeys);
  by_row = u * kKeys + kKeys - 1 > s.tok0;
  return by_row;
}

// Sum of the non-finite values of column `col` over the keys of partly visible tiles that
// this row sees (mask words of the tree, or keys up to its own token).
template <typename E, bool PAGED>
__device__ __noinline__ float nonfinite_sum(const Args* a, const Seg* s, int tok,
                                            const uint32_t* mask, int col) {
  const E* v = static_cast<const E*>(a->v);
  float sum = 0.f;
  for (int u = s->u0; u < s->u1; ++u) {
    int lim;
    bool by_row;
    if (!tile_part<PAGED>(*s, u, lim, by_row) || !by_row) continue;
    const int k0 = (u - (PAGED ? s->npre : 0)) * kKeys;
    for (int k = k0; k < k0 + lim; ++k) {
      const bool seen = PAGED ? (mask[k >> 5] >> (k & 31)) & 1u : k <= tok;
      if (!seen) continue;
      const float x = Elem<E>::up(v[(int64_t)(s->lo + k) * a->v_stride + (int64_t)s->hk * a->d + col]);
      if (!isfinite(x)) sum += x;
    }
  }
  return sum;
}

// ------------------------------------------------------------------ the pipeline
// W: the work list of this CTA; `bool next(Seg&)` is called by every lane of the copy warp.
// ALT: items of one row tile may give their key tiles to the two pipelines in turn (prompts).
// P16: pages of 16 positions.
template <int DP, typename E, bool PAGED, bool ALT, bool P16, typename W>
__device__ __forceinline__ void pipeline(uint8_t* smem, const Args& a, const CUtensorMap* qmap,
                                         const CUtensorMap* kmap, const CUtensorMap* vmap,
                                         const CUtensorMap* kpmap, const CUtensorMap* vpmap) {
  using L = Lay<DP, PAGED>;
  constexpr int NS = L::kStages;
  Bars* br = reinterpret_cast<Bars*>(smem + L::kOffMisc);
  uint32_t* smask = reinterpret_cast<uint32_t*>(smem + L::kOffMisc + sizeof(Bars));  // [2][256][8]
  uint16_t* spar = reinterpret_cast<uint16_t*>(smem + L::kOffMisc + sizeof(Bars) + kMaskBytes);  // [2][256]
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = uniform(tid >> 5);
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&br->kvfull[i], 1);
      mbar_init(&br->kvempty[i], L::kMmaWarps);
    }
    mbar_init(&br->qfull, 1);
    mbar_init(&br->qempty, L::kMmaWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&br->drain[i], 1);
    mbar_init(&br->alt_in, 4);
    mbar_init(&br->alt_back, 4);
    mbar_init(&br->alt_done, 8);
    mbar_init(&br->stolen, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&br->sfull[i], 1);
      mbar_init(&br->sread[i], 4);
      mbar_init(&br->pready[i][0], 4);
      mbar_init(&br->pready[i][1], 4);
      mbar_init(&br->pvdone[i], 1);
    }
    for (int i = 0; i < kFixRing; ++i) {
      mbar_init(&br->partfull[i], 1);
      mbar_init(&br->fixed[i], L::kFixWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&br->maskfull[i], L::kFixWarps);
      mbar_init(&br->maskempty[i], 8);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&br->segfull[i], 1);
      mbar_init(&br->segempty[i], L::kMmaWarps + 8 + L::kFixWarps);
    }
    fence_mbar_init();
    br->abort = 0;
  }
  if (warp == kMmaWarp) tmem_alloc(&br->tmem, kTmemCols);
  if (tid >= L::kCopyWarp * 32 && tid < L::kCopyWarp * 32 + (PAGED ? 5 : 3)) {
    const CUtensorMap* maps[5] = {qmap, kmap, vmap, kpmap, vpmap};
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[lane])) : "memory");
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  grid_dependency_wait();
  const uint32_t tmem = br->tmem;
  volatile int* abort = &br->abort;
  bool ok = true;

  if (warp == L::kCopyWarp) {
    // ---------------- work list and copies
    W work(a, &br->steal, &br->stolen);
    uint32_t cnt = 0, fix = 0;  // key and value tiles requested; values to be made safe
    int n_q = 0;       // items whose queries were requested
    auto slot_free = [&](uint32_t c) -> bool {
      return c < NS || wait_copies(&br->kvempty[c % NS], ((c / NS) - 1) & 1, abort, a.wait_ns);
    };
    int n = 0;
    Seg s;
    for (; ok; ++n) {
      const int r = n % kRing;
      if (n >= kRing) ok = wait_copies(&br->segempty[r], ((n / kRing) - 1) & 1, abort, a.wait_ns);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const bool more = work.next(s);
      if (!more) s.b = -1;
      if (lane == 0) {
        br->seg[r] = s;
        br->dirty[r] = 0;
        br->bad[r] = 0;
        mbar_arrive(&br->segfull[r]);
      }
      __syncwarp();
      if (!more) break;
      // page of this lane in tile u (lanes past the tile's pages, or a bad entry: -1)
      const int ppt = PAGED ? max(1, kKeys / a.ps) : 1;
      const int prow = PAGED ? min(a.ps, kKeys) : kKeys;
      auto page_of = [&](int u) -> int {
        if (!PAGED || u >= s.npre || lane >= ppt) return -1;
        const int64_t at = (int64_t)u * kKeys + (int64_t)lane * a.ps;
        if (at >= s.P) return -1;
        return a.table[(int64_t)s.b * a.max_pages + at / a.ps];
      };
      int page = page_of(s.u0);
      auto load = [&](int u, bool val, int pg) {
        uint64_t* bar = &br->kvfull[cnt % NS];
        int lim;
        bool by_row;
        if (val && tile_part<PAGED>(s, u, lim, by_row)) {
          // lands on a barrier of the warps that make it safe (they see only such tiles, in
          // turn, and the ring cannot pass one by); the products wait for those warps
          if (lane == 0) mbar_arrive(bar);
          bar = &br->partfull[fix++ % kFixRing];
        }
        uint8_t* dst = smem + L::kOffKV + (cnt % NS) * L::kTile;
        if (PAGED && u < s.npre) {
          const CUtensorMap* m = val ? vpmap : kpmap;
          const int left = s.P - u * kKeys;
          const int np = min(ppt, (left + a.ps - 1) / a.ps);
          if (lane == 0) mbar_arrive_expect_tx(bar, np * prow * 128 * L::kHalves);
          __syncwarp();
          const int z = pg * a.H_kv + s.hk;
          if (P16 && np == kKeys / 16) {
            // (17- and 129-node trees over up to 8100 positions 221 us after 239; in the kernel
            // for all page sizes the larger ones lost 1-2%)
            const uint32_t to = uniform(smem_addr(dst)), b = uniform(smem_addr(bar));
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i) {
              const int zi = uniform(z, i);
#pragma unroll
              for (int h = 0; h < L::kHalves; ++h)
                copy_box(to + h * L::kHalf + i * 16 * 128, m, b, h * 64, 0, zi);
            }
          } else if (lane < np) {
            const int in = a.ps > kKeys ? (u * kKeys) % a.ps : 0;
#pragma unroll
            for (int h = 0; h < L::kHalves; ++h)
              tma_load_3d(dst + h * L::kHalf + lane * prow * 128, m, bar, h * 64, in, z);
          }
        } else if (lane == 0) {
          const CUtensorMap* m = val ? vmap : kmap;
          const int row = s.lo + (u - (PAGED ? s.npre : 0)) * kKeys;
          mbar_arrive_expect_tx(bar, L::kTile);
#pragma unroll
          for (int h = 0; h < L::kHalves; ++h)
            tma_load_3d(dst + h * L::kHalf, m, bar, h * 64, s.hk, row);
        }
        __syncwarp();
        ++cnt;
      };
      for (int u = s.u0; ok && u < s.u1; ++u) {
        if (PAGED) {
          const bool mine = u < s.npre && lane < ppt && (int64_t)u * kKeys + (int64_t)lane * a.ps < s.P;
          const bool wrong = mine && (page < 0 || page >= a.n_pages);
          if (__any_sync(0xffffffffu, wrong)) {
            // a page outside the pool: nothing of it is read; the sequence gets zeros
            if (wrong) page = 0;
            if (lane == 0) {
              br->bad[r] = 1;
              atomicCAS(&a.status[s.b], TGDN_SEQ_OK, TGDN_SEQ_BAD_PAGE);
            }
            __syncwarp();
          }
        }
        const int next_page = u + 1 < s.u1 ? page_of(u + 1) : -1;
        if (!(ALT && s.alt) || u == s.u0) {
          ok = slot_free(cnt);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          load(u, false, page);
        }
        if (u == s.u0) {  // the queries, once the previous item's score products are done
          if (n > 0) ok = wait_copies(&br->qempty, (n - 1) & 1, abort, a.wait_ns);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          const bool come = s.b != a.hold_b || s.hk != a.hold_h;
          n_q += come;
          if (come && lane == 0) {
            const int tiles = s.e1 > s.u0 ? 2 : 1;
            mbar_arrive_expect_tx(&br->qfull, tiles * a.gbox * L::kHalves);
            for (int t = 0; t < tiles; ++t)
#pragma unroll
              for (int h = 0; h < L::kHalves; ++h)
                tma_load_3d(smem + t * L::kTile + h * L::kHalf, qmap, &br->qfull, h * 64,
                            s.hk * a.G, s.lo + s.tok0 + t * a.tpt);
          }
          __syncwarp();
        }
        // (alternating: the other pipeline's scores are due before this one's product)
        if (ALT && !PAGED && s.alt && u + 1 < s.u1) {
          ok = slot_free(cnt);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          load(u + 1, false, -1);
        }
        ok = slot_free(cnt);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        load(u, true, page);
        page = next_page;
      }
    }
    if (lane == 0) br->taken = n;
    if (!ok) {
      work.drop();
      // let the copies in flight land before the shared memory goes (bounded)
      for (uint32_t c = cnt > NS ? cnt - NS : 0; c < cnt; ++c)
        (void)mbar_wait(&br->kvfull[c % NS], (c / NS) & 1);
      for (uint32_t c = fix > kFixRing ? fix - kFixRing : 0; c < fix; ++c)
        (void)mbar_wait(&br->partfull[c % kFixRing], (c / kFixRing) & 1);
      if (n_q > 0) (void)mbar_wait(&br->qfull, (n_q - 1) & 1);
    }
  } else if (warp >= kMmaWarp && warp < kMmaWarp + L::kMmaWarps) {
    // ---------------- products.  The whole warp runs this role with equal values.
    constexpr bool kOwn = L::kMmaWarps == 2;  // this warp serves one row tile
    const int mine = warp - kMmaWarp;
    // Waits that fail are noted (`ok`) and looked at once per step: what is issued meanwhile
    // stays within the operands' buffers and counts for nothing.
    const uint32_t sb = smem_addr(br);
    auto at = [&](const void* member) {
      return sb + (uint32_t)(static_cast<const char*>(member) - reinterpret_cast<const char*>(br));
    };
    const uint32_t b_full = at(br->kvfull), b_empty = at(br->kvempty), b_fixed = at(br->fixed);
    const uint32_t b_s = at(br->sfull), b_read = at(br->sread), b_p = at(br->pready),
                   b_pv = at(br->pvdone), b_qempty = at(&br->qempty);
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (!try_at(bar, parity)) ok = wait_slow_at(bar, parity, abort) && ok;
      __syncwarp();
    };
    // Place in the ring of key and value tiles.
    struct Place {
      uint32_t slot, parity;
      __device__ void step() {
        if (++slot == NS) slot = 0, parity ^= 1;
      }
    };
    Place kp{0, 0}, vp{1, 0};   // the next key tile, the value tile of the step
    uint32_t fix = 0;           // value tiles made safe
    uint32_t done[2] = {0, 0};  // steps of each row tile
    constexpr uint32_t id_s = idesc(Elem<E>::kFmt, 128, kKeys, 0);
    constexpr uint32_t id_o = idesc(Elem<E>::kFmt, 128, DP, 1);
    const uint32_t utm = uniform(tmem);
    // descriptors' low words: address and leading byte offset in 16-byte units (value tiles:
    // the distance of their two 64-column halves)
    const uint32_t dQ = (smem_addr(smem) >> 4) | (1u << 16);
    const uint32_t dK = (smem_addr(smem + L::kOffKV) >> 4) | (1u << 16);
    const uint32_t dV = (smem_addr(smem + L::kOffKV) >> 4) | ((uint32_t)(L::kHalf >> 4) << 16);
    // An operand buffer is free once this warp's products that read it are done, or at once.
    auto release = [&](uint32_t bar, bool used) {
      if (!kOwn || used) commit(bar);
      else if (lane == 0) arrive_at(bar);
    };
    auto score = [&](int t, uint32_t slot, int rows) {  // S_t = Q_rows K^T of the tile in the slot
      // the previous O_t += P_t V has read P_t where that lies in S_t's columns
      if (!L::kApart && done[t] > 0) wait(b_pv + t * 8, (done[t] - 1) & 1);
      tc_fence_after_sync();
      const uint32_t q = dQ + rows * (L::kTile >> 4), k = dK + slot * (L::kTile >> 4);
#pragma unroll
      for (int h = 0; h < L::kHalves; ++h) {
        const uint32_t qh = q + h * (L::kHalf >> 4), kh = k + h * (L::kHalf >> 4);
        if (DP - h * 64 == 32) mma_ss2(utm + t * 128, qh, kh, id_s);
        else mma_ss4(utm + t * 128, qh, kh, id_s, h);
      }
      commit(b_s + t * 8);
    };
    // O_t (+)= P_t V of the step, 64 keys at a time as their P comes.  With P apart the next
    // S_t goes out as soon as this one has been read, beside the softmax on it.
    auto pv = [&](int t, bool first, bool more, const Place& vp, const Place& kp, int rows) {
      const uint32_t v = dV + vp.slot * (L::kTile >> 4);
      const uint32_t add = first ? 0u : 1u;
      if (L::kApart) {  // S_t is in the softmax threads' registers
        wait(b_read + t * 8, done[t] & 1);
        if (more) {
          wait(b_full + kp.slot * 8, kp.parity);
          score(t, kp.slot, rows);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wait(b_p + t * 16 + h * 8, done[t] & 1);
        tc_fence_after_sync();
        mma_ts4(utm + L::kColO + t * DP, utm + L::kColP + t * L::kStepP + h * 32, v + h * 512, id_o,
                h | add);
      }
      commit(b_pv + t * 8);
      ++done[t];
    };
    for (int n = 0; ok; ++n) {
      const int r = n % kRing;
      wait(at(&br->segfull[r]), (n / kRing) & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      Seg s = br->seg[r];
      if (uniform(s.b) < 0) break;
      s.u0 = uniform(s.u0), s.u1 = uniform(s.u1), s.e0 = uniform(s.e0), s.e1 = uniform(s.e1);
      s.N = uniform(s.N), s.P = uniform(s.P), s.npre = uniform(s.npre), s.tok0 = uniform(s.tok0);
      // steps of the row tiles that this warp serves
      const int e0 = kOwn && mine != 0 ? s.u0 : s.e0, e1 = kOwn && mine != 1 ? s.u0 : s.e1;
      const int e = max(e0, e1);
      wait(at(&br->qfull), n & 1);
      wait(b_full + kp.slot * 8, kp.parity);
      if (ALT && uniform(s.alt)) {
        // Key tiles in turn to the two pipelines, both on row tile 0; K_0 K_1 V_0 K_2 V_1 ...
        const int steps = s.u1 - s.u0;
        Place c = kp;  // the next place
        for (int t = 0; t < 2; ++t) {
          const bool used = !kOwn || mine == t;
          if (t == 1) wait(b_full + c.slot * 8, c.parity);
          if (used) score(t, c.slot, 0);
          release(b_empty + c.slot * 8, used);
          c.step();
        }
        if (steps == 2) release(b_qempty, true);
        for (int i = 0; i < steps; ++i) {
          const int t = i & 1;
          const bool used = !kOwn || mine == t, more = i + 2 < steps;
          wait(b_full + c.slot * 8, c.parity);
          int lim;
          bool by_row;
          if (tile_part<PAGED>(s, s.u0 + i, lim, by_row)) {
            wait(b_fixed + (fix % kFixRing) * 8, (fix / kFixRing) & 1);
            ++fix;
          }
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          Place k = c;
          k.step();
          if (used) pv(t, i < 2, more, c, k, 0);
          release(b_empty + c.slot * 8, used);
          c = k;
          if (more) {
            if (!L::kApart || !used) wait(b_full + k.slot * 8, k.parity);
            if (!L::kApart) score(t, k.slot, 0);
            release(b_empty + k.slot * 8, used);
            if (i + 3 == steps) release(b_qempty, true);
            c.step();
          }
        }
        kp = vp = c;
        vp.step();
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&br->segempty[r]);
        continue;
      }
      if (e0 > s.u0) score(0, kp.slot, 0);
      if (e1 > s.u0) score(1, kp.slot, 1);
      release(b_empty + kp.slot * 8, e > s.u0);
      if (s.u1 - s.u0 == 1) release(b_qempty, e > s.u0);
      kp.step(), kp.step();
      for (int u = s.u0; u < s.u1; ++u) {
        const bool x0 = u < e0, x1 = u < e1;          // this warp's steps
        const bool y0 = u + 1 < e0, y1 = u + 1 < e1;  // and next scores
        wait(b_full + vp.slot * 8, vp.parity);
        int lim;
        bool by_row;
        if (tile_part<PAGED>(s, u, lim, by_row)) {
          wait(b_fixed + (fix % kFixRing) * 8, (fix / kFixRing) & 1);
          ++fix;
        }
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (x0) pv(0, u == s.u0, y0, vp, kp, 0);
        if (!L::kApart && y0) {
          wait(b_full + kp.slot * 8, kp.parity);
          score(0, kp.slot, 0);
        }
        if (x1) pv(1, u == s.u0, y1, vp, kp, 1);
        release(b_empty + vp.slot * 8, u < e);
        if (u + 1 < s.u1) {
          // (a tile this warp has no step for is awaited too, or its phases could be lapped)
          if ((!L::kApart && !y0) || (kOwn && u + 1 >= e)) wait(b_full + kp.slot * 8, kp.parity);
          if (!L::kApart && y1) score(1, kp.slot, 1);
          release(b_empty + kp.slot * 8, u + 1 < e);
          if (u + 2 == s.u1) release(b_qempty, u + 1 < e);
          kp.step(), kp.step();
        }
        vp.step(), vp.step();
      }
      ok = __all_sync(0xffffffffu, ok) != 0;
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&br->segempty[r]);
    }
    // every product and every arrival it owes is done before the shared memory goes
    commit(at(&br->drain[mine]));
    (void)mbar_wait(&br->drain[mine], 0);
    __syncwarp();
  } else if (warp >= L::kFixWarp) {
    // ---------------- value rows that must not reach the product
    constexpr int kFix = L::kFixWarps * 32;
    const int ft = tid - L::kFixWarp * 32;  // 0 .. kFix - 1
    W::first(a, ft, kFix);  // status words
    uint32_t cnt = 0, fix = 0;
    int built = 0;
    for (int n = 0; ok; ++n) {
      const int r = n % kRing;
      ok = wait_bar(&br->segfull[r], (n / kRing) & 1, abort);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const Seg s = br->seg[r];
      if (s.b < 0) break;
      if (PAGED && s.u1 > s.npre) {
        // The ancestor-or-self sets of the item's nodes, ahead of the softmax warps (they come
        // to the tree's tiles last): each lane walks up from a node, in a copy of the parents.
        const int k = built++;
        if (k >= 2) ok = wait_bar(&br->maskempty[k & 1], ((k >> 1) - 1) & 1, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        uint16_t* par = spar + (warp - L::kFixWarp) * kMaxNodes;
        __syncwarp();
        for (int i = lane; i < s.N; i += 32) par[i] = (uint16_t)a.parent[s.lo + i];
        __syncwarp();
        for (int i = ft; i < 2 * a.tpt && s.tok0 + i < s.N; i += kFix) {
          uint64_t m[kMaxNodes / 64];
#pragma unroll
          for (int w = 0; w < kMaxNodes / 64; ++w) m[w] = 0;
          int x = s.tok0 + i;
          for (int up = 0; up <= TGDN_MAX_DEPTH && x < s.N; ++up) {  // (the root's parent: 0xffff)
#pragma unroll
            for (int w = 0; w < kMaxNodes / 64; ++w)
              if ((x >> 6) == w) m[w] |= 1ull << (x & 63);
            x = par[x];
          }
          uint64_t* out = reinterpret_cast<uint64_t*>(smask + ((k & 1) * 2 * kRows + i) * kMaskWords);
#pragma unroll
          for (int w = 0; w < kMaxNodes / 64; ++w) out[w] = m[w];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&br->maskfull[k & 1]);
      }
      const int steps = s.u1 - s.u0;
      const uint32_t base = cnt;
      cnt += 2 * steps;
      for (int u = s.u0; ok && u < s.u1; ++u) {
        int lim;
        bool by_row;
        if (!tile_part<PAGED>(s, u, lim, by_row)) continue;
        const int i = u - s.u0;  // (the copies' order)
        const uint32_t cv = base + (ALT && s.alt ? min(2 * i + 2, steps + i) : 2 * i + 1);
        ok = wait_bar(&br->partfull[fix % kFixRing], (fix / kFixRing) & 1, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        uint4* tile = reinterpret_cast<uint4*>(smem + L::kOffKV + (cv % NS) * L::kTile);
        uint32_t acc = 0;
        for (int i = ft; i < L::kTile / 16; i += kFix) {
          const int row = (i >> 3) & (kKeys - 1);
          if (row >= lim) {
            tile[i] = make_uint4(0, 0, 0, 0);
          } else if (by_row) {
            const uint4 w = tile[i];
            acc |= ((w.x & Elem<E>::kExp) + Elem<E>::kStep) | ((w.y & Elem<E>::kExp) + Elem<E>::kStep) |
                   ((w.z & Elem<E>::kExp) + Elem<E>::kStep) | ((w.w & Elem<E>::kExp) + Elem<E>::kStep);
          }
        }
        if (acc & 0x80008000u) {  // a non-finite value among this thread's
          br->dirty[r] = 1;
          uint32_t* w32 = reinterpret_cast<uint32_t*>(tile);
          for (int i = ft; i < L::kTile / 16; i += kFix)
            for (int j = 0; j < 4; ++j) {
              uint32_t w = w32[i * 4 + j];
              const uint32_t top = ((w & Elem<E>::kExp) + Elem<E>::kStep) & 0x80008000u;
              if (top & 0x8000u) w &= 0xffff0000u;
              if (top & 0x80000000u) w &= 0x0000ffffu;
              w32[i * 4 + j] = w;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&br->fixed[fix % kFixRing]);
        ++fix;
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&br->segempty[r]);
    }
    W::last(a, ft, kFix);  // outputs of sequences that have no work
  } else {
    // ---------------- softmax: row tile t, one row per thread
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lanes, tO = tmem + L::kColO + t * DP + lanes;
    const uint32_t tO0 = tmem + L::kColO + lanes;
    const uint32_t tP = tmem + L::kColP + t * L::kStepP + lanes;
    const float c2 = a.scale * 1.4426950408889634f;
    const float gap = kGap / a.scale;
    const int tok_in = row / a.G, g = row - tok_in * a.G;
    uint32_t done = 0;
    int built = 0, alts = 0;  // items with masks; items with alternating pipelines
    bool read_by_other = false;
    int n = 0;
    for (; ok; ++n) {
      const int r = n % kRing;
      ok = wait_bar(&br->segfull[r], (n / kRing) & 1, abort);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const Seg s = br->seg[r];
      if (s.b < 0) break;
      const int rt = ALT ? 0 : t;  // row tile
      const int e = t == 0 || (ALT && s.alt) ? s.e0 : s.e1;
      const int first = s.u0 + (ALT && s.alt ? t : 0), stride = ALT && s.alt ? 2 : 1;
      if (e > first) {
        const int tok = s.tok0 + rt * a.tpt + tok_in;
        const bool live = tok_in < a.tpt && tok < s.N;
        const uint32_t* mask = smask + ((built & 1) * 2 * kRows + rt * a.tpt + tok_in) * kMaskWords;
        if (ALT && read_by_other) {  // the last item's O_t has been read by the other pipeline's warps
          ok = wait_bar(&br->alt_done, (alts - 1) & 1, abort);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          read_by_other = false;
        }
        float m = -INFINITY;
        float2 la = make_float2(0.f, 0.f), lb = la;  // the row's sum, in four parts
        for (int u = first; u < e; u += stride) {
          ok = wait_bar(&br->sfull[t], done & 1, abort);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after_sync();
          float x[kKeys], mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) ld_max32(tS + q * 32, x + q * 32, mx[q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) ld_wait32(x + q * 32);
          asm volatile("" : "+f"(mx[0]), "+f"(mx[1]), "+f"(mx[2]), "+f"(mx[3]));  // (after the wait)
          if (L::kApart) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&br->sread[t]);
            __syncwarp();  // (tensor-memory accesses take the whole warp together)
          }
          // masks; the maxima again where they apply
          bool masked = false;
          if constexpr (PAGED) {
            if (u >= s.npre) {
              if (u == first || u - stride < s.npre) ok = wait_bar(&br->maskfull[built & 1], (built >> 1) & 1, abort);
              if (!(ok = __all_sync(0xffffffffu, ok))) break;
              const uint4 w4 = reinterpret_cast<const uint4*>(mask)[u - s.npre];
              const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
              masked = true;
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!((w[q] >> c) & 1u)) x[q * 32 + c] = -INFINITY;
            } else if (s.P - u * kKeys < kKeys) {
              const int lim = s.P - u * kKeys;
              masked = true;
#pragma unroll
              for (int c = 0; c < kKeys; ++c)
                if (c >= lim) x[c] = -INFINITY;
            }
          } else if (u * kKeys + kKeys - 1 > s.tok0) {
            const int lim = live ? tok - u * kKeys : -1;
            masked = true;
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
              if (c > lim) x[c] = -INFINITY;
          }
          if (masked) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mx[j] = fmaxf(x[j * 32], x[j * 32 + 1]);
#pragma unroll
              for (int c = 2; c < 32; c += 2) mx[j] = max3(mx[j], x[j * 32 + c], x[j * 32 + c + 1]);
            }
          }
          mx[0] = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          if (L::kApart && done > 0) {  // the last product has read P and is in O
            ok = wait_bar(&br->pvdone[t], (done - 1) & 1, abort);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after_sync();
          }
          const bool need = live && mx[0] > m + gap;  // also the first finite maximum
          if (__any_sync(0xffffffffu, need)) {
            const float alpha =
                need ? (m == -INFINITY ? 0.f : fast_exp2((m - mx[0]) * c2)) : 1.f;
            if (need) m = mx[0];
            la.x *= alpha, la.y *= alpha, lb.x *= alpha, lb.y *= alpha;
            if (u > first) {  // (the last product on O_t is done)
              __syncwarp();
#pragma unroll 1
              for (int q = 0; q < DP / 16; ++q) {
                float o[16];
                uint32_t w[16];
                tmem_ld16(tO + q * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 16; ++c) w[c] = __float_as_uint(o[c] * alpha);
                tmem_st16(tO + q * 16, w);
              }
            }
          }
          const float mc = m == -INFINITY ? 0.f : -m * c2;
          const float2 cc = make_float2(c2, c2), mm = make_float2(mc, mc);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float2 y = fma2(make_float2(x[q * 32 + 2 * c], x[q * 32 + 2 * c + 1]), cc, mm);
              y.x = fast_exp2(y.x);
              y.y = fast_exp2(y.y);
              if (c & 1) lb = add2(lb, y);
              else la = add2(la, y);
              w[c] = Elem<E>::pack(y.x, y.y);
            }
            tmem_st16(tP + q * 16, w);
            if (q & 1) {  // 64 keys are ready
              tmem_st_wait();
              tc_fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(&br->pready[t][q >> 1]);
              __syncwarp();
            }
          }
          ++done;
        }
        // the item's last product on O_t
        if (ok) ok = wait_bar(&br->pvdone[t], (done - 1) & 1, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) {
          if (lane == 0) timed_out(a, s.b);  // (with the rest of the items at the teardown)
          break;
        }
        tc_fence_after_sync();
        E* orow = static_cast<E*>(a.o) + (int64_t)(s.lo + tok) * a.o_stride +
                  (int64_t)(s.hk * a.G + g) * a.d;
        // 32 columns of this row's output: what `dirty` asks for added, scaled, rounded.
        auto put = [&](float (&o)[32], int q, bool dirty, bool bad, float inv) {
          if (dirty) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (q * 32 + c < a.d)
                o[c] += nonfinite_sum<E, PAGED>(&a, &br->seg[r], tok, mask, q * 32 + c);
          }
          if (PAGED && s.part >= 0) {  // a part: column groups of four, rows side by side
            float4* part = reinterpret_cast<float4*>(a.part) +
                           ((int64_t)(blockIdx.x * 2 + s.part) * (DP / 4) + q * 8) * a.part_rows +
                           t * kRows + row;
#pragma unroll
            for (int c = 0; c < 8; ++c)
              part[(int64_t)c * a.part_rows] =
                  make_float4(o[c * 4], o[c * 4 + 1], o[c * 4 + 2], o[c * 4 + 3]);
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                w[i] = bad ? 0u : Elem<E>::pack(o[c * 16 + 2 * i] * inv, o[c * 16 + 2 * i + 1] * inv);
              E* to = orow + q * 32 + c * 16;
              const int left = a.d - (q * 32 + c * 16);
              if (a.o_wide && left >= 16) {
                st_global32(to, w);
              } else {
                if (left > 0) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                if (left > 8) *reinterpret_cast<uint4*>(to + 8) = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        };
        if (ALT && s.alt) {
          // Pipeline 1 hands over its maximum and sum and gets both weights back; each writes
          // half of the columns.
          const float l = (la.x + la.y) + (lb.x + lb.y);
          const uint32_t turn = alts++ & 1;
          if (t == 1) {
            br->alt_ml[row] = make_float2(m, l);
          } else {
            ok = wait_bar(&br->alt_in, turn, abort);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const float2 other = br->alt_ml[row];
            const float top = fmaxf(m, other.x);
            const float w0 = m == -INFINITY ? 0.f : fast_exp2((m - top) * c2);
            const float w1 = other.x == -INFINITY ? 0.f : fast_exp2((other.x - top) * c2);
            const float both = l * w0 + other.y * w1, inv = both == 0.f ? 0.f : 1.f / both;
            br->alt_ml[row] = make_float2(w0 * inv, w1 * inv);
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(t == 1 ? &br->alt_in : &br->alt_back);
          if (t == 1) ok = wait_bar(&br->alt_back, turn, abort);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after_sync();
          const float2 w = br->alt_ml[row];
          const bool dirty = *reinterpret_cast<volatile int*>(&br->dirty[r]) != 0;
          constexpr int kFirst = (DP / 32 + 1) / 2;  // pipeline 0's share, 32 columns apiece
#pragma unroll 1
          for (int q = t == 0 ? 0 : kFirst; q < (t == 0 ? kFirst : DP / 32); ++q) {
            __syncwarp();
            float o[32], x[32];
            tmem_ld32(tO0 + q * 32, o);
            tmem_ld32(tO0 + DP + q * 32, x);
            ld_wait32(o);
            ld_wait32(x);
            if (!live) continue;
            // (without weight O adds nothing, finite or not)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              o[c] = (w.x == 0.f ? 0.f : o[c] * w.x) + (w.y == 0.f ? 0.f : x[c] * w.y);
            put(o, q, dirty, false, 1.f);
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&br->alt_done);
          read_by_other = true;
        } else {
          const bool dirty = *reinterpret_cast<volatile int*>(&br->dirty[r]) != 0;
          const bool bad = PAGED && (s.zero || *reinterpret_cast<volatile int*>(&br->bad[r]) != 0);
          const float l = (la.x + la.y) + (lb.x + lb.y);
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
          for (int q = 0; q < DP / 32; ++q) {
            __syncwarp();  // (`put` parts the warp, and the load takes all of it together)
            float o[32];
            tmem_ld32(tO + q * 32, o);
            ld_wait32(o);
            if (live) put(o, q, dirty, bad, inv);
          }
          if (PAGED && s.part >= 0 && live)
            a.part_ml[(int64_t)(blockIdx.x * 2 + s.part) * a.part_rows + t * kRows + row] =
                make_float2(m == -INFINITY ? 0.f : m * c2, l);
          tc_fence_before_sync();
        }
      }
      if (PAGED && s.u1 > s.npre) {  // done with the item's masks
        ok = wait_bar(&br->maskfull[built & 1], (built >> 1) & 1, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (lane == 0) mbar_arrive(&br->maskempty[built & 1]);
        ++built;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&br->segempty[r]);
    }
    if (lane == 0) br->put_out[warp] = n;
  }
  // ---------------- teardown
  tc_fence_before_sync();
  const bool all_ok = __syncthreads_and(ok) != 0;
  if (!all_ok && tid == 0) {  // the items taken on and not put out (the ring still has them all)
    int n = br->taken;
    for (int w = 0; w < 8; ++w) n = min(n, br->put_out[w]);
    for (; n < br->taken; ++n) timed_out(a, br->seg[n % kRing].b);
  }
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace attn
}  // namespace tgdn
