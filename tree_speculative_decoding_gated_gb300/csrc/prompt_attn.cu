// prompt_attn.cu — causal attention over whole prompts (packed rows, grouped heads).
//
//   o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   within each sequence.
//
// The pipeline of attn_core.cuh over items (sequence, block of 2 x 128 query rows,
// key/value head).  One CTA per item is launched, each sequence's last (longest) blocks
// first; the CTAs that run take over the places of those that have not started (cluster
// launch control), so that a CTA's copies and first products of the next item go out while
// it finishes the last and uneven lengths even out.  Against items dealt out in turns,
// 16 prompts of up to 4001 tokens (d = 128): 168 us after 192; items of one length lose a
// little by the requests (6 prompts of up to 2500 tokens, d = 64: 49.5 us after 46.5).
//
// Bound by the tensor core (d = 128) or the softmax (d = 64), as attn_core.cuh says: a
// 32768-token prompt 2.6-2.8 ms (1570-1690 TFLOP/s of the visible half), 16 uneven prompts
// 151 us (1170), where the diagonal tiles, half masked, and the items' ends take the rest; 6
// prompts at d = 64 39-40 us (430).  One prompt of 97 tokens takes 6.7 us: a launch, the
// first copies, one tile, the output.
#include "attn_core.cuh"

namespace tgdn {
namespace attn {

struct PromptWork {
  const Args& a;
  uint4* answer;
  uint64_t* bar;
  int lane, chunk = 0;       // sequences from `chunk` on ...
  int before = 0;            // ... begin at this item
  int high = 0;              // ... and may use rows from this one on
  int asked = 0;             // requests made; the last one is open while open is set
  bool open = false;
  int64_t x;                 // the next item, or -1

  __device__ PromptWork(const Args& args, uint4* ans, uint64_t* b)
      : a(args), answer(ans), bar(b), lane(threadIdx.x & 31), x(blockIdx.x) {
    ask();
  }

  // The rows of this lane's sequence c + lane (whole warp): false when its range leaves [0, T)
  // or begins below an earlier one's end (`high`: the end of those before c), so that no row
  // has two sequences and the rows bound the items.
  static __device__ bool range_of(const Args& a, int c, int high, int lane, int& lo, int& N,
                                  int& next_high) {
    lo = N = 0;
    int hi = 0;
    bool good = c + lane < a.B;
    if (good) {
      lo = a.cu[c + lane];
      hi = a.cu[c + lane + 1];
      good = lo >= 0 && hi >= lo && hi <= a.T;
    }
    int top = good ? hi : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, top, o);
      if (lane >= o) top = max(top, y);
    }
    int under = __shfl_up_sync(0xffffffffu, top, 1);
    under = lane == 0 ? high : max(under, high);
    next_high = max(high, __shfl_sync(0xffffffffu, top, 31));
    good = good && lo >= under;
    N = good ? hi - lo : 0;
    return good;
  }
  // The status words (whole warp), once per launch: by CTA 0 or, should that be taken over before
  // it starts (nothing promises that it starts first), by the CTA that takes it over.
  static __device__ __noinline__ void write_status(const Args& a, int lane) {
    int high = 0;
    for (int c = 0; c < a.B; c += 32) {
      int lo, N;
      const bool good = range_of(a, c, high, lane, lo, N, high);
      if (c + lane < a.B) a.status[c + lane] = good ? TGDN_SEQ_OK : TGDN_SEQ_BAD_RANGE;
    }
  }
  static __device__ void first(const Args& a, int ft, int) {
    if (blockIdx.x == 0 && ft < 32) write_status(a, ft);
  }
  static __device__ void last(const Args&, int, int) {}

  // Requests the place of a CTA of this grid that has not started.
  __device__ void ask() {
    if (lane == 0) {
      fence_proxy_async_smem();  // the last answer was read
      mbar_arrive_expect_tx(bar, 16);
      asm volatile(
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
          "[%1];" ::"r"(smem_addr(answer)),
          "r"(smem_addr(bar))
          : "memory");
    }
    __syncwarp();
    ++asked;
    open = true;
  }
  // The number of the CTA whose place was given, or -1 (none is left, or the answer did not
  // come in time).
  __device__ int64_t answered() {
    const bool came = __all_sync(0xffffffffu, mbar_wait(bar, (asked - 1) & 1)) != 0;
    open = false;
    if (!came) {  // (whatever was taken over is lost)
      for (int b = lane; b < a.B; b += 32) timed_out(a, b);
      return -1;
    }
    uint32_t got, cta;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "=r"(cta)
        : "r"(smem_addr(answer))
        : "memory");
    __syncwarp();
    if (got && cta == 0) write_status(a, lane);
    return got ? (int64_t)cta : -1;
  }
  // Item x, if there is one (numbers mostly ascend: the search goes on where the last ended).
  __device__ bool find(Seg& s) {
    if (x < before) chunk = before = high = 0;
    const int blk = a.tpt * a.tiles;  // tokens per item
    for (; chunk < a.B; chunk += 32) {
      int lo, N, next_high;
      (void)range_of(a, chunk, high, lane, lo, N, next_high);
      const int items = (N + blk - 1) / blk * a.H_kv;
      int upto = items;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int total = __shfl_sync(0xffffffffu, upto, 31);
      if (x < before + total) {
        const int at = (int)(x - before);
        const int f = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
        s.b = chunk + f;
        s.lo = __shfl_sync(0xffffffffu, lo, f);
        s.N = __shfl_sync(0xffffffffu, N, f);
        const int in = at - __shfl_sync(0xffffffffu, upto - items, f);
        const int blocks = (s.N + blk - 1) / blk;
        s.hk = in % a.H_kv;
        s.tok0 = (blocks - 1 - in / a.H_kv) * blk;
        s.u0 = 0;
        s.e0 = (min(s.tok0 + a.tpt, s.N) - 1) / kKeys + 1;
        s.e1 = a.tiles > 1 && s.tok0 + a.tpt < s.N
                   ? (min(s.tok0 + 2 * a.tpt, s.N) - 1) / kKeys + 1 : 0;
        s.u1 = max(s.e0, s.e1);
        s.set_alt();
        s.P = s.npre = 0;
        s.part = -1;
        s.zero = 0;
        return true;
      }
      before += total;
      high = next_high;
    }
    return false;
  }
  // The answer to the request made an item ago is there; the next one goes out at once.
  __device__ bool next(Seg& s) {
    while (x >= 0) {
      const bool found = find(s);  // (numbers past the last item have no work)
      x = answered();
      if (x >= 0) ask();
      if (found) return true;
    }
    return false;
  }
  // After an early end: the items taken over and not done.  No request stays open when the
  // shared memory goes.
  __device__ void drop() {
    while (x >= 0 || open) {
      if (x < 0) x = answered();
      Seg s;
      if (x >= 0 && find(s) && lane == 0) timed_out(a, s.b);
      x = -1;
    }
  }
};

template <int DP, typename E, bool ALT>
__global__ void __launch_bounds__(kBlock, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
  extern __shared__ uint8_t pa_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(pa_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  pipeline<DP, E, false, ALT, false, PromptWork>(smem, a, &qmap, &kmap, &vmap, nullptr, nullptr);
}

// Single row tiles whose key tiles alternate between the pipelines, from this mean length on:
// one prompt of 2000 tokens 29.2 us after 32.0 (d = 64: 20.9 after 26.5); 16 of up to 300
// tokens, whose few key tiles do not pay for joining, 13.1 after 11.9.
constexpr int kAltTokens = 768;

template <int DP, typename E>
static cudaError_t launch(const Args& a, const CUtensorMap& q, const CUtensorMap& k,
                          const CUtensorMap& v, int grid, cudaStream_t s) {
  const auto kern = a.tiles == 1 && a.T / a.B >= kAltTokens ?
                        prompt_attn_kernel<DP, E, true> : prompt_attn_kernel<DP, E, false>;
  constexpr int smem = smem_bytes<DP, false>();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(grid), dim3(kBlock), smem, s, q, k, v, a);
}

}  // namespace attn

cudaError_t launch_prompt_attn(int B, int T, int H_q, int H_kv, int d, int io, float scale,
                               const int32_t* cu, const CUtensorMap& q, const CUtensorMap& k,
                               const CUtensorMap& v, const void* v_rows, int64_t v_stride,
                               void* o, int64_t o_stride, int32_t* status, cudaStream_t s) {
  using namespace attn;
  Args a{};
  a.B = B;
  a.T = T;
  a.H_q = H_q;
  a.H_kv = H_kv;
  a.G = H_q / H_kv;
  a.d = d;
  a.tpt = kRows / a.G;
  a.gbox = 128 * a.G * a.tpt;
  a.scale = scale;
  a.cu = cu;
  a.status = status;
  a.o = o;
  a.o_stride = o_stride;
  a.o_wide = wide_rows(o, o_stride, d);
  a.v = v_rows;
  a.v_stride = v_stride;
  set_hooks(a);
  // At most T / blk + B blocks per head.  One row tile per item when two would leave SMs idle,
  // and with small heads, whose alternating pipelines lose least, while items are few: 5000
  // tokens, 16 heads of 64 elements 67 us after 76, 16000 tokens, 4 heads 148 after 186; at
  // d = 128 the same rule loses (9000 tokens 265 us after 219), and so do short prompts (20 of
  // up to 1200 tokens, d = 64, 32.6 after 29.7).
  const int sms = device_sm_count();
  auto items = [&](int tiles) { return ((long)T / (a.tpt * tiles) + B) * H_kv; };
  a.tiles = items(2) >= (d <= 64 && T / B >= kAltTokens ? 4 : 1) * sms ? 2 : 1;
  const long n = items(a.tiles);
  if (n > 0x3fffffffL) return cudaErrorInvalidConfiguration;
  const int grid = (int)n;
  auto go = [&](auto e) {
    using E = decltype(e);
    return d > 96 ? launch<128, E>(a, q, k, v, grid, s)
         : d > 64 ? launch<96, E>(a, q, k, v, grid, s) : launch<64, E>(a, q, k, v, grid, s);
  };
  return io == TGDN_BF16 ? go(__nv_bfloat16()) : go(__half());
}

}  // namespace tgdn
