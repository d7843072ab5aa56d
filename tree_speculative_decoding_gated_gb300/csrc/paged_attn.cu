// paged_attn.cu — ancestor-masked tree attention over a paged key/value cache.
//
// Node n of sequence b attends to the cached positions 0 .. len[b] - 1, which lie in the
// pages of its table row, and to the tree nodes on its own root path, itself included;
// a one-node tree is plain single-token decoding.  The pipeline of attn_core.cuh, a key
// tile being 128 / page_size page boxes of cached positions, then the tree's own rows.
//
// Decoding reads each cached key and value once for a handful of query rows, so memory
// bounds it, and what costs is uneven lengths.  All key tiles of all items are therefore
// numbered through and every CTA takes an equal run of them, wherever it begins and ends
// (kMinShare at least: a cut costs a join).  A run covers whole items and at most two
// cut ones; the parts of a cut item (O unnormalised, reference maximum, sum) go to the
// workspace and paged_merge_kernel joins them in order of their keys, so results do not
// depend on timing.  Without a workspace items stay whole.
//
// Measured: single tokens over up to 131072 positions (8 sequences, 2 heads of 128, fp16)
// 104 us for 622 MB, 89% of the copy bandwidth.  64-node trees over up to 4096 positions
// (16 sequences) 32 us for 65 MB: a CTA has at most 7 steps of two row tiles, under 10 us;
// the start takes ~5, and the parts of cut items (128 KB each in fp32) are 23 MB written
// and read again by a join of ~9 us when it runs alone.  A batch of 17- and 129-node trees
// over up to 8100 positions 222 us: 129 nodes of four heads are five row tiles in three
// blocks, which read the same keys at times of their own (1052 MB from DRAM for 491, 27% L2
// hits): a step takes 1.96 us where one whose keys are there takes 1.4.
#include <algorithm>

#include "attn_core.cuh"

namespace tgdn {
namespace attn {

// Key tiles per CTA below which a cut costs more than it saves: two where the parts are joined
// eight rows at a time (7-node trees over 1500 positions 14.8 and 12.7 us, 4 trees of 64 nodes
// over 4000 23.0 and 20.9), four else.  Caches that can hold no more key tiles than kSplitTiles
// are never cut: 6, or 4 for up to kFewRows rows (one token over 600 positions 13.3 us whole,
// 12.3 cut, over 300 11.1 and 11.8; 16 trees of 7 nodes over 500 12.5 and 16.4).
constexpr int kFewRows = 8;
constexpr int kMinShare[2] = {4, 2};    // [narrow join]
constexpr int kSplitTiles[2] = {6, 4};  // [few rows]
// An item's start and output, in key tiles (0: 64-node trees over 4096 positions 35.2 us, 1: 33.5,
// 2: 31.5).
constexpr int kItemCost = 2;

// Cached and tree key tiles of sequence b; 0: no work (empty, or an error).
struct Plan {
  int lo, N, P, npre, nt, st;
};
__device__ __forceinline__ Plan plan_of(const Args& a, int b) {
  Plan p{};
  p.lo = a.cu[b];
  const int hi = a.cu[b + 1];
  p.st = a.status[b];
  p.P = a.len[b];
  const int held = a.held[b];
  p.N = hi > p.lo ? hi - p.lo : 0;  // (far apart the wrong way round the difference would wrap)
  // (words this kernel itself may write count as planned: every CTA plans the same work)
  const bool run = p.st == TGDN_SEQ_OK || p.st == TGDN_SEQ_TIMEOUT || p.st == TGDN_SEQ_BAD_PAGE;
  if (!run || p.lo < 0 || p.N <= 0 || hi > a.T || p.N > a.n_max || p.P < 0 || held < 0 ||
      held > a.max_pages || p.P > (int64_t)held * a.ps || (p.P > 0 && a.n_pages == 0))
    return p;  // nt = 0
  p.npre = (p.P + kKeys - 1) / kKeys;
  p.nt = p.npre + (p.N + kKeys - 1) / kKeys;
  return p;
}
__device__ __forceinline__ int64_t items_of(const Args& a, const Plan& p) {
  const int blk = a.tpt * 2;
  return p.nt ? (int64_t)((p.N + blk - 1) / blk) * a.H_kv : 0;
}

// Quotient of non-negative numbers (nearly always small ones, which divide faster).
__device__ __forceinline__ int64_t divide(int64_t n, int64_t by) {
  if ((n | by) >> 32 == 0) return (uint32_t)n / (uint32_t)by;
  return n / by;
}

__device__ __forceinline__ int64_t warp_sum_upto(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

struct PagedWork {
  const Args& a;
  int lane, n = 0;
  int64_t x, x1, share;
  int4 d0, d1;
  // the 32 sequences from `chunk` on (a lane each): their tiles before them and in them
  int chunk = 0;
  Plan p;
  int64_t before = 0, tiles, upto, total;

  __device__ void load(int c) {
    chunk = c;
    p = Plan{};
    if (c + lane < a.B) p = plan_of(a, c + lane);
    tiles = items_of(a, p) * (p.nt + kItemCost);
    upto = warp_sum_upto(tiles, lane);
    total = __shfl_sync(0xffffffffu, upto, 31);
  }
  __device__ PagedWork(const Args& args, uint4*, uint64_t*) : a(args), lane(threadIdx.x & 31) {
    // (a call that ends early must leave nothing for the merge to read)
    if (a.part != nullptr && lane == 0) a.desc[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    load(0);
    int64_t sum = total;
    if (a.B > 32) {
      int64_t more = 0;
      for (int b = 32 + lane; b < a.B; b += 32) {
        const Plan q = plan_of(a, b);
        more += items_of(a, q) * (q.nt + kItemCost);
      }
      sum += __shfl_sync(0xffffffffu, warp_sum_upto(more, lane), 31);
    }
    share = divide(sum + gridDim.x - 1, gridDim.x);
    if (share < a.min_share) share = a.min_share;
    x = min(sum, share * blockIdx.x);
    x1 = min(sum, x + share);
    d0 = make_int4(-1, 0, 0, 0);
    d1 = make_int4(0, 0, 0, 0);
  }

  // Sequences without work but with rows: zeros, and the word for a bad length.
  static __device__ void first(const Args&, int, int) {}
  static __device__ void last(const Args& a, int ft, int n) {
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      const Plan p = plan_of(a, b);
      if (p.nt || p.N <= 0 || p.st == TGDN_SEQ_BAD_RANGE || p.lo < 0 || p.lo + p.N > a.T) continue;
      const int v8 = a.H_q * a.d / 8;  // 16-byte pieces of a row
      for (int64_t i = ft; i < (int64_t)p.N * v8; i += n)
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + (p.lo + i / v8) * a.o_stride)[i % v8] =
            make_uint4(0, 0, 0, 0);
      if (ft == 0) atomicCAS(&a.status[b], TGDN_SEQ_OK, TGDN_SEQ_BAD_PAGE);
    }
  }

  // After an early end: the sequences with work in the rest of the run, and that of the cut item,
  // which is not named to the join.
  __device__ void drop() {
    if (d0.x >= 0 && lane == 0) timed_out(a, d0.x);
    while (x < x1) {
      const int64_t begin = before + upto - tiles;
      if (tiles > 0 && begin < x1 && begin + tiles > x) timed_out(a, chunk + lane);
      before += total;
      if (before >= x1 || chunk + 32 >= a.B) return;
      load(chunk + 32);
    }
  }
  __device__ bool next(Seg& s) {
    while (x < x1) {
      for (;;) {
        if (x >= before + total) {
          if (chunk + 32 >= a.B) {  // (lengths that shrank since the sum was taken)
            x = x1;
            break;
          }
          before += total;
          load(chunk + 32);
          continue;
        }
        const int64_t at = x - before;
        const int f = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
        const int64_t in = at - __shfl_sync(0xffffffffu, upto - tiles, f);
        s.b = chunk + f;
        s.lo = __shfl_sync(0xffffffffu, p.lo, f);
        s.N = __shfl_sync(0xffffffffu, p.N, f);
        s.P = __shfl_sync(0xffffffffu, p.P, f);
        s.npre = __shfl_sync(0xffffffffu, p.npre, f);
        const int nt = __shfl_sync(0xffffffffu, p.nt, f);
        s.zero = __shfl_sync(0xffffffffu, p.st, f) != TGDN_SEQ_OK;
        const int item = (int)divide(in, nt + kItemCost);
        s.hk = item % a.H_kv;
        s.tok0 = item / a.H_kv * a.tpt * 2;
        s.u0 = (int)(in - (int64_t)item * (nt + kItemCost));
        const int64_t x_item = x - s.u0, x_next = x_item + nt + kItemCost;
        if (a.part == nullptr || s.u0 >= nt) {
          x = x_next;
          if (s.u0 > 0) break;  // another CTA's item
          s.u1 = nt;
        } else {
          s.u1 = (int)min((int64_t)nt, s.u0 + (x1 - x));
          x = min(x_next, x1);
        }
        s.part = s.u0 == 0 && s.u1 == nt ? -1 : (n == 0 ? 0 : 1);
        s.e0 = s.u1;
        s.e1 = s.tok0 + a.tpt < s.N ? s.u1 : 0;
        s.alt = 0;
        if (s.u0 == 0 && s.u1 < nt) {
          d0 = make_int4(s.b, s.lo, s.N, s.tok0);
          d1 = make_int4(s.hk, (int)divide(x_item + nt - 1, share), s.part, 0);
        }
        ++n;
        return true;
      }
    }
    if (a.part != nullptr && lane == 0) {
      a.desc[2 * blockIdx.x] = d0;
      a.desc[2 * blockIdx.x + 1] = d1;
    }
    return false;
  }
};

template <int DP, typename E, bool P16>
__global__ void __launch_bounds__(kBlock, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap kpmap,
                  const __grid_constant__ CUtensorMap vpmap, const __grid_constant__ Args a) {
  extern __shared__ uint8_t pg_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(pg_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  pipeline<DP, E, true, false, P16, PagedWork>(smem, a, &qmap, &kmap, &vmap, &kpmap, &vpmap);
}

// Joins the parts of an item that begins in one run and goes on into later ones, a row group
// (32 query rows, or 8) per CTA:
//   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s
// First the weights, several lanes per row, so that all statistics are under way at once;
// then the sums, a thread per row and four columns, whose loads wait for nothing.
//   32 rows: one CTA per row group and run; those of runs that name no item leave at once.
//   8 rows (NARROW): rows that are no more, or few items, whose CTAs seek out their runs; what
//   few rows leave of a CTA takes parts in turn.  More parts are under way and more CTAs
//   share an item: 33-node trees over 34400 positions (7 items of ~25 parts) 107 -> 29 us a
//   call, 7-node ones over 9696 30.8 -> 16.1; where items are many the CTAs cost more than
//   they save (8 trees of 64 nodes over 1000 positions, 32 items, 19.7 -> 25.6).
constexpr int kMergeRows = 32, kNarrowRows = 8;
constexpr int kMaxParts = 160;
template <int DP, typename E, bool NARROW>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ Args a) {
  constexpr int kGroup = NARROW ? kNarrowRows : kMergeRows;
  __shared__ float s_w[kMaxParts][kGroup];
  __shared__ float s_inv[kGroup];
  __shared__ float4 s_sum[256];
  __shared__ __align__(16) uint8_t s_out[kGroup][DP * 2 + 16];
  grid_dependency_wait();
  const int tid = threadIdx.x;
  int c = blockIdx.y;  // (an item's row groups go to different SMs)
  int4 d0, d1;
  if (!NARROW || gridDim.y == a.runs) {
    d0 = a.desc[2 * c], d1 = a.desc[2 * c + 1];
    if (d0.x < 0) return;
  } else {  // the blockIdx.y-th run that names a cut item
    __shared__ int s_run;
    if (tid < 32) {
      int x[kMaxParts / 32], left = c, run = -1;
#pragma unroll
      for (int j = 0; j < kMaxParts / 32; ++j)
        x[j] = j * 32 + tid < a.runs ? a.desc[2 * (j * 32 + tid)].x : -1;
#pragma unroll
      for (int j = 0; j < kMaxParts / 32; ++j) {
        const uint32_t cut = __ballot_sync(0xffffffffu, x[j] >= 0);
        if (x[j] >= 0 && __popc(cut & ((1u << tid) - 1)) == left) run = j * 32 + tid;
        left -= __popc(cut);
      }
      run = __reduce_max_sync(0xffffffffu, run);
      if (tid == 0) s_run = run;
    }
    __syncthreads();
    c = s_run;
    if (c < 0) return;
    d0 = a.desc[2 * c], d1 = a.desc[2 * c + 1];
  }
  const int r0 = blockIdx.x * kGroup, R = min(kGroup, a.part_rows - r0);
  if ((r0 / kRows) * a.tpt + d0.w >= d0.z) return;  // no row of this row tile exists
  // part i lies in CTA c + i's first slot, the first part in the slot its CTA named
  // (no CTA after the last has any: lengths that grow under way could name one)
  const int parts = min(min(d1.y, a.runs - 1) - c + 1, kMaxParts);
  auto slot = [&](int i) -> int64_t { return 2 * (c + i) + (i == 0 ? d1.z : 0); };
  int rp = 1;  // threads side by side over rows: the power of two from R up
  while (rp < R) rp *= 2;
  constexpr int C = DP / 4;                    // column groups
  constexpr int kPer = NARROW ? 1 : C / 8;     // of them, the most of one thread
  constexpr int kNext = NARROW ? 16 : 4;       // parts under way
  const int r = tid & (rp - 1), over = tid / rp;
  const int step = min(256 / rp, C);           // threads over the columns
  const int turns = 256 / rp / step;           // and over the parts
  const int cg0 = over % step, turn = over / step;
  const float4* part = reinterpret_cast<const float4*>(a.part) + r0 + min(r, R - 1);
  float4 acc[kPer], o[kNext][kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kNext; ++j)
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (i0 + j * turns < parts && cg0 + k * step < C)
          o[j][k] = part[(slot(i0 + j * turns) * C + cg0 + k * step) * a.part_rows];
  };
  load(turn);  // (needs no weights)
  {
    const int sub = min(32, 256 / rp), rw = tid / sub, i0 = tid % sub;  // sub lanes per row
    const float2* ml = a.part_ml + r0 + min(rw, R - 1);
    constexpr int kStat = 4;
    float2 v[kStat];  // (all there are, but for many parts of many rows)
    float M = -INFINITY, sum = 0.f;
    for (int b = i0; b < parts; b += kStat * sub) {
#pragma unroll
      for (int j = 0; j < kStat; ++j) {
        const int i = b + j * sub;
        v[j] = i < parts ? ml[slot(i) * a.part_rows] : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < kStat; ++j)
        if (v[j].y != 0.f) M = fmaxf(M, v[j].x);
    }
    for (int o = sub / 2; o > 0; o /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int b = i0; b < parts; b += kStat * sub) {
#pragma unroll
      for (int j = 0; j < kStat; ++j) {
        const int i = b + j * sub;
        if (i >= parts) continue;
        if (parts > kStat * sub) v[j] = ml[slot(i) * a.part_rows];
        const float w = v[j].y == 0.f ? 0.f : fast_exp2(v[j].x - M);
        sum = fmaf(w, v[j].y, sum);
        if (rw < R) s_w[i][rw] = w;
      }
    }
    for (int o = sub / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (rw < R && i0 == 0) s_inv[rw] = sum == 0.f ? 0.f : 1.f / sum;
  }
  __syncthreads();
  for (int i0 = turn; i0 < parts; i0 += kNext * turns) {
    if (i0 != turn) load(i0);
#pragma unroll
    for (int j = 0; j < kNext; ++j) {
      const int i = i0 + j * turns;
      const float w = i < parts && r < R ? s_w[i][r] : 0.f;
      if (w == 0.f) continue;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (cg0 + k * step >= C) continue;
        acc[k].x = fmaf(w, o[j][k].x, acc[k].x);
        acc[k].y = fmaf(w, o[j][k].y, acc[k].y);
        acc[k].z = fmaf(w, o[j][k].z, acc[k].z);
        acc[k].w = fmaf(w, o[j][k].w, acc[k].w);
      }
    }
  }
  if (turns > 1) {  // (step = C: a thread has one column group)
    s_sum[tid] = acc[0];
    __syncthreads();
    for (int k = 1; turn == 0 && k < turns; ++k) {
      const float4 o = s_sum[tid + k * step * rp];
      acc[0].x += o.x, acc[0].y += o.y, acc[0].z += o.z, acc[0].w += o.w;
    }
  }
  if (r < R && turn == 0) {
    const float inv = s_inv[r];
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (cg0 + k * step < C)
        *reinterpret_cast<uint2*>(&s_out[r][(cg0 + k * step) * 8]) =
            make_uint2(Elem<E>::pack(acc[k].x * inv, acc[k].y * inv),
                       Elem<E>::pack(acc[k].z * inv, acc[k].w * inv));
  }
  __syncthreads();
  const bool ok = a.status[d0.x] == TGDN_SEQ_OK;
  const int pieces = a.d / 8;  // 16-byte pieces of a row
  for (int e = tid; e < R * pieces; e += 256) {
    const int i = e / pieces, x = e - i * pieces;
    const int rr = r0 + i, t = rr / kRows, row = rr % kRows, tok_in = row / a.G;
    const int tok = d0.w + t * a.tpt + tok_in;
    if (tok_in >= a.tpt || tok >= d0.z) continue;
    E* to = static_cast<E*>(a.o) + (int64_t)(d0.y + tok) * a.o_stride +
            (int64_t)(d1.x * a.G + row - tok_in * a.G) * a.d + x * 8;
    *reinterpret_cast<uint4*>(to) =
        ok ? *reinterpret_cast<const uint4*>(&s_out[i][x * 16]) : make_uint4(0, 0, 0, 0);
  }
}

struct Split {
  int grid, rows;
  size_t part_off, ml_off, bytes;
};
static Split split_of(int n_max, int G, int d) {
  Split p;
  const int dp = d > 96 ? 128 : d > 64 ? 96 : 64, tpt = kRows / G;
  p.grid = std::min(device_sm_count(), kMaxParts);
  p.rows = n_max <= tpt ? std::max(n_max, 1) * G : 2 * kRows;
  p.part_off = ((size_t)p.grid * 2 * sizeof(int4) + 255) / 256 * 256;
  p.ml_off = p.part_off + (size_t)p.grid * 2 * p.rows * dp * sizeof(float);
  p.bytes = p.ml_off + (size_t)p.grid * 2 * p.rows * sizeof(float2);
  return p;
}

template <int DP, typename E>
static cudaError_t launch(const Args& a, int grid, const CUtensorMap& q, const CUtensorMap& k,
                          const CUtensorMap& v, const CUtensorMap& kp, const CUtensorMap& vp,
                          cudaStream_t s) {
  const auto kern = a.ps == 16 ? paged_attn_kernel<DP, E, true> : paged_attn_kernel<DP, E, false>;
  constexpr int smem = smem_bytes<DP, true>();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_after(kern, dim3(grid), dim3(kBlock), smem, s, q, k, v, kp, vp, a);
  if (e != cudaSuccess || a.part == nullptr) return e;
  if (a.joins > 0)  // (few rows in all, or few items)
    return launch_after(paged_merge_kernel<DP, E, true>,
                        dim3((a.part_rows + kNarrowRows - 1) / kNarrowRows, a.joins), dim3(256), 0, s, a);
  return launch_after(paged_merge_kernel<DP, E, false>,
                      dim3((a.part_rows + kMergeRows - 1) / kMergeRows, grid), dim3(256), 0, s, a);
}

}  // namespace attn

size_t paged_attn_workspace_bytes(const tgdn_tree& t, int H_q, int H_kv, int d) {
  return attn::split_of(t.n_max, H_q / H_kv, d).bytes;
}

cudaError_t launch_paged_attn(const tgdn_tree& t, const tgdn_pages& pg, int H_q, int H_kv, int d,
                              int io, float scale, const CUtensorMap& q, const CUtensorMap& k,
                              const CUtensorMap& v, const CUtensorMap& kp, const CUtensorMap& vp,
                              const void* v_rows, int64_t v_stride, void* o, int64_t o_stride,
                              void* ws, size_t ws_bytes, cudaStream_t s) {
  using namespace attn;
  Args a{};
  a.B = t.B;
  a.T = t.T;
  a.H_q = H_q;
  a.H_kv = H_kv;
  a.G = H_q / H_kv;
  a.d = d;
  a.tpt = kRows / a.G;
  a.gbox = 128 * a.G * a.tpt;
  a.tiles = 2;
  a.scale = scale;
  a.cu = t.cu_nodes;
  a.status = t.status;
  a.o = o;
  a.o_stride = o_stride;
  a.o_wide = wide_rows(o, o_stride, d);
  a.v = v_rows;
  a.v_stride = v_stride;
  set_hooks(a);
  a.n_max = t.n_max;
  a.ps = pg.page_size;
  a.n_pages = pg.n_pages;
  a.max_pages = pg.max_pages;
  a.parent = t.parent;
  a.table = pg.table;
  a.len = pg.len;
  a.held = pg.held;
  const Split p = split_of(t.n_max, a.G, d);
  a.part_rows = p.rows;
  a.runs = p.grid;
  // (few items: no more than four joining CTAs per SM)
  const int64_t items = (int64_t)t.B * H_kv * ((t.n_max + 2 * a.tpt - 1) / (2 * a.tpt));
  if (p.rows <= kNarrowRows) a.joins = p.grid;
  else if (items * ((p.rows + kNarrowRows - 1) / kNarrowRows) <= 4 * p.grid) a.joins = std::max((int)items, 1);
  // a short cache is not split: the merge would take longer than the tiles it spares
  const int64_t most = ((int64_t)pg.max_pages * pg.page_size + kKeys - 1) / kKeys + (t.n_max + kKeys - 1) / kKeys;
  a.min_share = kMinShare[a.joins > 0];
  if (ws != nullptr && ws_bytes >= p.bytes && most > kSplitTiles[p.rows <= kFewRows]) {
    a.desc = static_cast<int4*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part_off);
    a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + p.ml_off);
  }
  auto go = [&](auto e) {
    using E = decltype(e);
    return d > 96 ? launch<128, E>(a, p.grid, q, k, v, kp, vp, s)
         : d > 64 ? launch<96, E>(a, p.grid, q, k, v, kp, vp, s)
                  : launch<64, E>(a, p.grid, q, k, v, kp, vp, s);
  };
  return io == TGDN_BF16 ? go(__nv_bfloat16()) : go(__half());
}

}  // namespace tgdn
