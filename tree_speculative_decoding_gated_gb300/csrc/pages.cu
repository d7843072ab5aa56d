// pages.cu — the paged key/value cache: bookkeeping on the device and copies in every layer.
//
// Whole numbers throughout, and the same for the same calls: free pages are listed in
// ascending order by block-wide prefix sums (no atomic decides an order), sequences and
// forks are served in the order given.  A planning kernel of one CTA validates, counts and
// writes a plan to the workspace; the kernel after it, which moves the data, spreads over
// the device.  Copies are bound by memory: 16-byte pieces, read and written once.
//
// Measured: compaction of a pool of 9 layers (455 MB read and written) 72 us of kernels, 65 of
// them the copies at 7.0 TB/s (a plain copy runs at 6.7; some of what is written stays in L2);
// a branch's life (24 forks, reserve, append of paths in 9
// layers, free) 22 us of kernels for 35 MB: six small launches, 3-4 us each, which are
// chained so that each is set up while the one before drains.
#include "launch_after.cuh"
#include "tgdn_device.cuh"
#include "tgdn_kernels.h"

namespace tgdn {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPerThread = 8;  // reference counts per thread and round of a scan

// Workspace: head (16 ints), then four arrays of max(n_pages, B, TGDN_PAGES_MAX_LIST) ints.
struct PagesWs {
  int32_t *head, *a, *b, *c, *d;
};
static size_t ws_len(const tgdn_pages& p) {
  size_t n = TGDN_PAGES_MAX_LIST;
  if ((size_t)p.n_pages > n) n = p.n_pages;
  if ((size_t)p.B > n) n = p.B;
  return (n + 63) / 64 * 64;
}
size_t pages_workspace_bytes(const tgdn_pages& p) { return (64 + 4 * ws_len(p)) * sizeof(int32_t); }
static PagesWs ws_of(const tgdn_pages& p, void* ws) {
  int32_t* w = static_cast<int32_t*>(ws);
  const size_t n = ws_len(p);
  return PagesWs{w, w + 64, w + 64 + n, w + 64 + 2 * n, w + 64 + 3 * n};
}

// ----------------------------------------------------------------- one-CTA primitives
// Exclusive prefix sum over the CTA's threads; *total: the sum.  Two barriers.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* total) {
  __shared__ int64_t s_warp[kPlanWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  const int64_t before = (warp ? s_warp[warp - 1] : 0) + x - v;
  *total = s_warp[kPlanWarps - 1];
  __syncthreads();  // s_warp is free again
  return before;
}

// The pages of [lo, hi) whose reference count is zero (FREE) or not, in ascending order:
// f(rank, page) for ranks below `want`; returns the number found, which is exact up to
// `want` (the scan stops there).
template <bool FREE, typename F>
__device__ __forceinline__ int64_t list_pages(const int32_t* refs, int lo, int hi, int64_t want,
                                              F&& f) {
  int64_t found = 0;
  for (int64_t base = lo; base < hi && found < want; base += kPlanThreads * kPerThread) {
    const int64_t i0 = base + (int64_t)threadIdx.x * kPerThread;
    uint32_t hit = 0;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      if (i0 + j < hi && (refs[i0 + j] == 0) == FREE) hit |= 1u << j;
    int64_t total;
    int64_t rank = found + block_scan(__popc(hit), &total);
    while (hit) {
      const int j = __ffs(hit) - 1;
      hit &= hit - 1;
      if (rank < want) f(rank, (int)(i0 + j));
      ++rank;
    }
    found += total;
  }
  return found < want ? found : want;
}

__device__ __forceinline__ bool sound(const tgdn_pages& p, int len, int held) {
  return len >= 0 && held >= 0 && held <= p.max_pages && len <= (int64_t)held * p.page_size;
}

// ----------------------------------------------------------------- reserve
__global__ void __launch_bounds__(kPlanThreads) pages_reserve_kernel(tgdn_pages p, PagesWs w,
                                                                     const int32_t* add) {
  grid_launch_dependents();
  grid_dependency_wait();
  // pages each sequence lacks and where they begin in the list of free pages
  int32_t *need = w.a, *off = w.b, *list = w.c;
  int64_t sum = 0;
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + threadIdx.x;
    int n = 0;
    if (b < p.B) {
      const int len = p.len[b], held = p.held[b], more = add[b];
      int st = TGDN_SEQ_OK;
      if (!sound(p, len, held) || more < 0) {
        st = TGDN_SEQ_BAD_PAGE;
      } else {
        const int64_t want = ((int64_t)len + more + p.page_size - 1) / p.page_size;
        if (want > p.max_pages) st = TGDN_SEQ_NO_PAGES;
        else if (want > held) n = (int)(want - held);
      }
      p.status[b] = st;
    }
    int64_t total;
    const int64_t before = sum + block_scan(n, &total);
    if (b < p.B) {
      // (past 2^31 pages nothing is served: any value above the pool's size does)
      need[b] = n;
      off[b] = (int)(before > 0x3fffffff ? 0x3fffffff : before);
    }
    sum += total;
  }
  const int64_t found = list_pages<true>(p.refs, 0, p.n_pages, sum,
                                         [&](int64_t k, int page) { list[k] = page; });
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < p.B; b += kPlanWarps) {
    const int n = need[b], o = off[b];
    if (n == 0) continue;
    if ((int64_t)o + n > found) {
      if (lane == 0) p.status[b] = TGDN_SEQ_NO_PAGES;
      continue;
    }
    const int held = p.held[b];
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
      const int page = list[o + i];
      p.table[(int64_t)b * p.max_pages + held + i] = page;
      p.refs[page] = 1;
    }
    if (lane == 0) p.held[b] = held + n;
  }
}

cudaError_t launch_pages_reserve(const tgdn_pages& p, const int32_t* add, void* ws, cudaStream_t s) {
  return launch_after(pages_reserve_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, ws_of(p, ws), add);
}

// ----------------------------------------------------------------- append
constexpr int kAppendRows = 8;  // rows per CTA and turn: 8 x 64 pieces (4 heads of 128) feed 128 threads

// Rows that sequence b appends, or -1 (its range leaves the arrays).
__device__ __forceinline__ int rows_to_append(const AppendArgs& a, int b) {
  const int lo = a.cu[b], hi = a.cu[b + 1];
  if (lo < 0 || hi < lo || hi > a.T) return -1;
  if (a.path == nullptr) return hi - lo;
  const int n = a.n_path[b];
  return n < 0 || n > a.path_len ? -1 : n;
}

// Groups of kAppendRows rows, numbered through the sequences in order (each by its own range:
// ranges need not be sound or apart), a group per CTA and turn; blockIdx.y: the layer.
__global__ void __launch_bounds__(128) pages_append_kernel(const AppendArgs a) {
  grid_launch_dependents();
  grid_dependency_wait();
  const tgdn_pages& p = a.p;
  __shared__ int64_t s_to[kAppendRows];  // page * page_size + position in the page, or -1
  __shared__ int s_row[kAppendRows];
  __shared__ int s_seq, s_first;         // sequence and first row of this group; -1: no more
  const int layer = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int d8 = a.pool.d / 8, pieces = a.pool.H_kv * d8;
  const int64_t page8 = (int64_t)pieces * p.page_size;  // 16-byte pieces of a page
  uint4* kp = static_cast<uint4*>(a.pool.data) + (int64_t)layer * 2 * p.n_pages * page8;
  uint4* vp = kp + (int64_t)p.n_pages * page8;
  const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k) + layer * a.k_layer);
  const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v) + layer * a.v_layer);
  int chunk = 0;       // (warp 0) sequences from here on ...
  int64_t before = 0;  // ... begin at this group
  for (int64_t x = blockIdx.x;; x += gridDim.x) {
    if (tid < 32) {
      int seq = -1, first = 0;
      while (chunk < p.B) {
        const int n = chunk + lane < p.B ? rows_to_append(a, chunk + lane) : 0;
        const int groups = n > 0 ? (n + kAppendRows - 1) / kAppendRows : 0;
        int64_t upto = groups;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        const int64_t total = __shfl_sync(0xffffffffu, upto, 31);
        if (x < before + total) {
          const int f = __ffs(__ballot_sync(0xffffffffu, upto > x - before)) - 1;
          seq = chunk + f;
          first = (int)(x - before - __shfl_sync(0xffffffffu, upto - groups, f)) * kAppendRows;
          break;
        }
        before += total;
        chunk += 32;
      }
      if (lane == 0) {
        s_seq = seq;
        s_first = first;
      }
    }
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    if (tid < kAppendRows) {
      const int i = s_first + tid, lo = a.cu[b];
      int row = -1;
      if (i < rows_to_append(a, b)) {
        if (a.path == nullptr) {
          row = lo + i;
        } else {
          const int node = a.path[(int64_t)b * a.path_len + i];
          if (node >= 0 && node < a.cu[b + 1] - lo) row = lo + node;
        }
      }
      int64_t to = -1;
      if (row >= 0) {
        const int len = p.len[b], held = p.held[b];
        const int64_t at = (int64_t)len + i;
        if (sound(p, len, held) && at < (int64_t)held * p.page_size) {
          const int page = p.table[(int64_t)b * p.max_pages + at / p.page_size];
          if (page >= 0 && page < p.n_pages) to = (int64_t)page * p.page_size + at % p.page_size;
        }
      }
      s_to[tid] = to;
      s_row[tid] = row;
    }
    __syncthreads();
    for (int e = tid; e < kAppendRows * pieces; e += 128) {
      const int r = e / pieces, c = e - r * pieces;
      const int64_t to = s_to[r];
      if (to < 0) continue;
      const int h = c / d8, y = c - h * d8;
      const int64_t page = to / p.page_size, in = to % p.page_size;
      const int64_t dst = page * page8 + ((int64_t)h * p.page_size + in) * d8 + y;
      const int64_t src = (int64_t)s_row[r];
      const uint4 kv = ks[src * (a.k_row / 8) + c], vv = vs[src * (a.v_row / 8) + c];
      kp[dst] = kv;
      vp[dst] = vv;
    }
    __syncthreads();
  }
}

// Status of every sequence's append and, if asked for, its new length: a warp per sequence.
__global__ void __launch_bounds__(128) pages_advance_kernel(const AppendArgs a, int advance) {
  grid_launch_dependents();
  grid_dependency_wait();
  const tgdn_pages& p = a.p;
  const int b = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= p.B) return;
  const int n = rows_to_append(a, b), len = p.len[b], held = p.held[b];
  int st = TGDN_SEQ_OK;
  if (n < 0) {
    st = TGDN_SEQ_BAD_RANGE;
  } else if (!sound(p, len, held)) {
    st = TGDN_SEQ_BAD_PAGE;
  } else if ((int64_t)len + n > (int64_t)held * p.page_size) {
    st = TGDN_SEQ_NO_PAGES;
  } else if (n > 0) {
    bool range = true, page_ok = true;
    if (a.path != nullptr) {
      const int N = a.cu[b + 1] - a.cu[b];
      for (int i = lane; i < n; i += 32) {
        const int node = a.path[(int64_t)b * a.path_len + i];
        range &= node >= 0 && node < N;
      }
    }
    for (int64_t i = len / p.page_size + lane; i <= ((int64_t)len + n - 1) / p.page_size; i += 32) {
      const int page = p.table[(int64_t)b * p.max_pages + i];
      page_ok &= page >= 0 && page < p.n_pages;
    }
    if (!__all_sync(0xffffffffu, range)) st = TGDN_SEQ_BAD_RANGE;
    else if (!__all_sync(0xffffffffu, page_ok)) st = TGDN_SEQ_BAD_PAGE;
  }
  if (lane == 0) {
    p.status[b] = st;
    if (advance && st == TGDN_SEQ_OK && n > 0) p.len[b] = len + n;
  }
}

cudaError_t launch_pages_append(const AppendArgs& a, bool advance, cudaStream_t s) {
  // groups there can be when the ranges are sound (each CTA goes on to further ones)
  const int64_t groups = a.path != nullptr
                             ? (int64_t)a.p.B * ((a.path_len + kAppendRows - 1) / kAppendRows)
                             : (int64_t)a.T / kAppendRows + a.p.B;
  if (a.T > 0 && groups > 0) {
    const int64_t most = 16 * device_sm_count();  // CTAs per layer that can be resident
    const unsigned grid = (unsigned)(groups < most ? groups : most);
    const cudaError_t e = launch_after(pages_append_kernel, dim3(grid, a.pool.layers), dim3(128), 0, s, a);
    if (e != cudaSuccess) return e;
  }
  return launch_after(pages_advance_kernel, dim3((a.p.B + 3) / 4), dim3(128), 0, s, a,
                      advance ? 1 : 0);
}

// ----------------------------------------------------------------- fork
// Plan per fork i: a = full pages or -1, b = filled positions of the last page, c = its
// page, d = its copy.
__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan_kernel(tgdn_pages p, PagesWs w,
                                                                       int n, const int32_t* src,
                                                                       const int32_t* dst,
                                                                       int32_t* status) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += kPlanWarps) {
    const int x = src[i], y = dst[i];
    int len = 0, held = 0;
    bool good = x >= 0 && x < p.B && y >= 0 && y < p.B;
    if (good) {
      len = p.len[x];
      held = p.held[x];
      good = sound(p, len, held) && p.held[y] == 0;
    }
    bool mine = true;
    if (good) {
      for (int j = lane; j < i; j += 32) mine &= dst[j] != y;
      for (int j = lane; j < (len + p.page_size - 1) / p.page_size; j += 32) {
        const int page = p.table[(int64_t)x * p.max_pages + j];
        mine &= page >= 0 && page < p.n_pages;
      }
    }
    good = __all_sync(0xffffffffu, good && mine);
    if (lane == 0) {
      w.a[i] = good ? len / p.page_size : -1;
      w.b[i] = good ? len % p.page_size : 0;
      w.c[i] = good && len % p.page_size
                   ? p.table[(int64_t)x * p.max_pages + len / p.page_size] : -1;
    }
  }
  __syncthreads();
  int64_t sum = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int need = i < n && w.b[i] > 0;
    int64_t total;
    const int64_t before = sum + block_scan(need, &total);
    if (i < n) w.d[i] = need ? (int)before : -1;  // its rank among the free pages
    sum += total;
  }
  __shared__ int s_list[TGDN_PAGES_MAX_LIST];  // (ranks are below n)
  const int64_t found = list_pages<true>(p.refs, 0, p.n_pages, sum,
                                         [&](int64_t k, int page) { s_list[k] = page; });
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    int st = w.a[i] < 0 ? TGDN_SEQ_BAD_PAGE : TGDN_SEQ_OK;
    const int rank = w.d[i];
    if (rank >= 0) {
      if (rank < found) {
        w.d[i] = s_list[rank];
      } else {
        w.a[i] = -1;
        st = TGDN_SEQ_NO_PAGES;
      }
    }
    status[i] = st;
  }
}

// blockIdx.x: fork; blockIdx.y 0: its table row, counts and lengths; else one head of one
// layer's keys or values of the last page.
__global__ void __launch_bounds__(128) pages_fork_kernel(tgdn_pages p, tgdn_pool pool, PagesWs w,
                                                         const int32_t* src, const int32_t* dst) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int full = w.a[i], tail = w.b[i];
  if (full < 0) return;
  const int from = w.c[i], to = w.d[i];
  if (blockIdx.y == 0) {
    const int x = src[i], y = dst[i];
    const int32_t* row = p.table + (int64_t)x * p.max_pages;
    int32_t* out = p.table + (int64_t)y * p.max_pages;
    for (int j = tid; j < full; j += 128) {
      out[j] = row[j];
      atomicAdd(&p.refs[row[j]], 1);
    }
    if (tid == 0) {
      if (tail > 0) {
        out[full] = to;
        p.refs[to] = 1;
      }
      p.len[y] = full * p.page_size + tail;
      p.held[y] = full + (tail > 0);
      p.status[y] = TGDN_SEQ_OK;
    }
    return;
  }
  if (tail == 0) return;
  const int slab = blockIdx.y - 1;  // (layer, keys or values, head)
  const int h = slab % pool.H_kv, buf = slab / pool.H_kv;
  const int64_t head8 = (int64_t)p.page_size * pool.d / 8;  // 16-byte pieces of a head's slab
  uint4* base = static_cast<uint4*>(pool.data) + ((int64_t)buf * p.n_pages * pool.H_kv + h) * head8;
  const uint4* s4 = base + (int64_t)from * pool.H_kv * head8;
  uint4* d4 = base + (int64_t)to * pool.H_kv * head8;
#pragma unroll 4
  for (int e = tid; e < tail * (pool.d / 8); e += 128) d4[e] = s4[e];
}

cudaError_t launch_pages_fork(const tgdn_pages& p, const tgdn_pool& pool, int n,
                              const int32_t* src, const int32_t* dst, int32_t* status, void* ws,
                              cudaStream_t s) {
  const PagesWs w = ws_of(p, ws);
  const cudaError_t e = launch_after(pages_fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, w,
                                     n, src, dst, status);
  if (e != cudaSuccess) return e;
  return launch_after(pages_fork_kernel, dim3(n, 1 + pool.layers * 2 * pool.H_kv), dim3(128), 0, s,
                      p, pool, w, src, dst);
}

// ----------------------------------------------------------------- free
__global__ void __launch_bounds__(128) pages_free_kernel(tgdn_pages p, const int32_t* seq) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = seq[blockIdx.x], tid = threadIdx.x;
  if (b < 0 || b >= p.B) return;
  // a sequence listed again is released by its first place in the list
  bool again = false;
  for (int j = tid; j < (int)blockIdx.x; j += 128) again |= seq[j] == b;
  const int held = p.held[b];
  if (__syncthreads_or(again)) return;
  if (held < 0 || held > p.max_pages) {
    // left as it is: past its own pages a row keeps old numbers, which others may hold now
    if (tid == 0) p.status[b] = TGDN_SEQ_BAD_PAGE;
    return;
  }
  bool bad = false;
  for (int j = tid; j < held; j += 128) {
    const int page = p.table[(int64_t)b * p.max_pages + j];
    if (page < 0 || page >= p.n_pages) {
      bad = true;
    } else if (atomicSub(&p.refs[page], 1) <= 0) {
      atomicAdd(&p.refs[page], 1);
      bad = true;
    }
  }
  bad = __syncthreads_or(bad) != 0;
  if (tid == 0) {
    p.held[b] = 0;
    p.len[b] = 0;
    p.status[b] = bad ? TGDN_SEQ_BAD_PAGE : TGDN_SEQ_OK;
  }
}

cudaError_t launch_pages_free(const tgdn_pages& p, int n, const int32_t* seq, cudaStream_t s) {
  return launch_after(pages_free_kernel, dim3(n), dim3(128), 0, s, p, seq);
}

// ----------------------------------------------------------------- compact
// head[0] = pages in use, head[1] = moves; a = holes, b = movers, c[page] = where a page
// from n_live on goes (-1: it is free).
__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(tgdn_pages p, PagesWs w,
                                                                          int32_t* n_live) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t all = 0x7fffffff;
  const int live = (int)list_pages<false>(p.refs, 0, p.n_pages, all, [](int64_t, int) {});
  (void)list_pages<true>(p.refs, 0, live, all, [&](int64_t k, int page) { w.a[k] = page; });
  for (int i = live + threadIdx.x; i < p.n_pages; i += kPlanThreads) w.c[i] = -1;
  __syncthreads();
  const int64_t moves = list_pages<false>(p.refs, live, p.n_pages, all, [&](int64_t k, int page) {
    w.b[k] = page;
    w.c[page] = w.a[k];
  });
  if (threadIdx.x == 0) {
    w.head[0] = live;
    w.head[1] = (int)moves;
    *n_live = live;
  }
}

constexpr int kMoveBytes = 16384;  // bytes per step of a CTA's copies: four 16-byte loads a thread

__global__ void __launch_bounds__(256) pages_compact_kernel(tgdn_pages p, tgdn_pool pool, PagesWs w) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int live = w.head[0], moves = w.head[1], tid = threadIdx.x;
  // tables: a warp per sequence; reference counts: a thread per move
  for (int b = blockIdx.x * 8 + (tid >> 5); b < p.B; b += gridDim.x * 8) {
    const int held = p.held[b];
    bool good = sound(p, p.len[b], held);
    // (every entry that names a moved page follows it, whatever else is wrong with the sequence)
    for (int j = tid & 31; j < min(held, p.max_pages); j += 32) {
      int32_t* e = p.table + (int64_t)b * p.max_pages + j;
      const int page = *e;
      if (page < 0 || page >= p.n_pages || (page >= live && w.c[page] < 0)) good = false;
      else if (page >= live) *e = w.c[page];
    }
    good = __all_sync(0xffffffffu, good);
    if ((tid & 31) == 0) p.status[b] = good ? TGDN_SEQ_OK : TGDN_SEQ_BAD_PAGE;
  }
  for (int k = blockIdx.x * 256 + tid; k < moves; k += gridDim.x * 256) {
    p.refs[w.a[k]] = p.refs[w.b[k]];
    p.refs[w.b[k]] = 0;
  }
  const int64_t page16 = (int64_t)pool.H_kv * p.page_size * pool.d / 8;  // 16-byte pieces
  const int64_t steps = (page16 * 16 + kMoveBytes - 1) / kMoveBytes;
  const int64_t jobs = (int64_t)moves * pool.layers * 2 * steps;
  for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int64_t step = job % steps, kb = job / steps;
    const int k = (int)(kb % moves);
    const int64_t buf = kb / moves;
    uint4* base = static_cast<uint4*>(pool.data) + buf * p.n_pages * page16;
    const uint4* from = base + w.b[k] * page16;
    uint4* to = base + w.a[k] * page16;
    const int64_t e0 = step * (kMoveBytes / 16);
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e0 + j * 256 + tid < page16) x[j] = from[e0 + j * 256 + tid];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e0 + j * 256 + tid < page16) to[e0 + j * 256 + tid] = x[j];
  }
}

cudaError_t launch_pages_compact(const tgdn_pages& p, const tgdn_pool& pool, int32_t* n_live,
                                 void* ws, cudaStream_t s) {
  const PagesWs w = ws_of(p, ws);
  const cudaError_t e = launch_after(pages_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p,
                                     w, n_live);
  if (e != cudaSuccess) return e;
  return launch_after(pages_compact_kernel, dim3(device_sm_count() * 8), dim3(256), 0, s, p, pool, w);
}

}  // namespace tgdn
