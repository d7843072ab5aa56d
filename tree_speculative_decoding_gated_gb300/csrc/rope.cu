// rope.cu — rotary positions of q and k.
//
// Pair i of a head is turned by p f_i (p: the row's position).  The turn p f_i / (2 pi) is
// formed as p times a 64-bit binary fraction, which wraps at whole turns exactly (2^-64 of a
// turn per position), so a position of a million keeps the phase that fp32 angles lose.
//
// Bound by memory: every element is read and written once.  A CTA takes a few rows; their
// rot/2 cosines and sines go to shared memory once per row and serve all its heads, then
// each thread turns 16-byte pieces (in the half layout the two pieces of its pairs).
// Measured: 16384 rows of 20 heads of 128 (bf16, half of each head turned, 168 MB) 33 us,
// 5.1 TB/s, 76% of the copy bandwidth (43.6 us before the loads went ahead of the angles);
// 33 rows 2.9 us, a launch and two rounds of loads.
#include <cuda_fp16.h>

#include "launch_after.cuh"
#include "tgdn_device.cuh"
#include "tgdn_kernels.h"

namespace tgdn {

constexpr int kRopeThreads = 256;
constexpr int kAhead = 4;      // loads in flight per thread (two pieces each in the half layout)
constexpr int kRopeRows = 16;  // rows per CTA at most

template <typename E> struct RopeIo;
template <> struct RopeIo<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void up(const uint4& w, float* x) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 down(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <> struct RopeIo<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void up(const uint4& w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 down(const float* x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <> struct RopeIo<__half> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void up(const uint4& w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 down(const float* x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 p = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// The sequence of row t, or -1.  Called by a whole warp, which tests 32 offsets at a time:
// the last b with cu[b] <= t, where its range is sound and holds t; offsets that decrease
// somewhere can hide t's sequence from that, so otherwise the first sound range around t.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int T, int t) {
  const int lane = threadIdx.x & 31;
  auto holds = [&](int b) {
    const int c0 = cu[b], c1 = cu[b + 1];
    return c0 >= 0 && c0 <= t && t < c1 && c1 <= T;
  };
  int b = -1;
  for (int c = 0; c < B; c += 32) {
    const uint32_t below = __ballot_sync(0xffffffffu, c + lane < B && cu[c + lane] <= t);
    if (below) b = c + 31 - __clz(below);
    if (below != 0xffffffffu) break;
  }
  if (b >= 0 && holds(b)) return b;
  for (int c = 0; c < B; c += 32) {
    const uint32_t in = __ballot_sync(0xffffffffu, c + lane < B && holds(min(c + lane, B - 1)));
    if (in) return c + __ffs(in) - 1;
  }
  return -1;
}

// The rows' positions (a warp per row) and their cosines and sines, to shared memory.
__device__ __forceinline__ void rope_table(const RopeArgs& a, int t0, int rows, float2* turn,
                                           int64_t* s_pos, int* s_ok) {
  const int tid = threadIdx.x, half = a.rot / 2;
  for (int r = tid >> 5; r < rows; r += kRopeThreads / 32) {
    const int t = t0 + r;
    const int b = t < a.T ? sequence_of(a.cu, a.B, a.T, t) : -1;
    if ((tid & 31) == 0) {
      s_ok[r] = b >= 0;
      if (b >= 0)
        s_pos[r] = (int64_t)(a.base ? a.base[b] : 0) + (a.off ? a.off[t] : t - a.cu[b]);
    }
  }
  __syncthreads();
  for (int e = tid; e < rows * half; e += kRopeThreads) {
    const int r = e / half, i = e - r * half;
    if (!s_ok[r]) continue;
    uint64_t f = (uint64_t)s_pos[r] * a.freq[i];
    if (a.transpose) f = 0 - f;
    // 2^-63 of a signed 64-bit turn fraction: the angle in half turns, in [-1, 1)
    const float h = (float)(int64_t)f * 1.0842021724855044e-19f;
    float s, c;
    sincospif(h, &s, &c);
    turn[e] = make_float2(c * a.mscale, s * a.mscale);
  }
  __syncthreads();
}

template <typename E>
__device__ __forceinline__ const E* rope_in(const RopeArgs& a, int64_t t, int h) {
  return h < a.H_q ? static_cast<const E*>(a.q) + t * a.q_stride + (int64_t)h * a.d
                   : static_cast<const E*>(a.k) + t * a.k_stride + (int64_t)(h - a.H_q) * a.d;
}
template <typename E>
__device__ __forceinline__ E* rope_out(const RopeArgs& a, int64_t t, int h) {
  return h < a.H_q ? static_cast<E*>(a.q_out) + t * a.q_out_stride + (int64_t)h * a.d
                   : static_cast<E*>(a.k_out) + t * a.k_out_stride + (int64_t)(h - a.H_q) * a.d;
}

// 16-byte pieces: a unit is one piece (interleaved pairs), or the two pieces of eight pairs
// (halves), or one piece past rot that is copied.  A thread loads kAhead units at once, the
// first ones before the rows' angles are known, so that the loads do not wait for them; the
// unit, head and row advance by fixed steps instead of divisions.
template <typename E, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int rows) {
  extern __shared__ __align__(16) float2 turn[];  // [rows][rot / 2]: mscale (cos, sin)
  constexpr int V = RopeIo<E>::V;
  __shared__ int64_t s_pos[kRopeRows];
  __shared__ int s_ok[kRopeRows];
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x, t0 = blockIdx.x * rows;
  const int heads = a.H_q + a.H_kv, half = a.rot / 2;
  const int turned = PAIRS ? a.rot / V : half / V, copied = a.rot / V;  // units; first copied piece
  const int units = turned + a.d / V - copied;
  const int all = min(rows, a.T - t0) * heads * units;
  int u = tid % units, h = tid / units, r = h / heads;
  h -= r * heads;
  const int du = kRopeThreads % units, dh0 = kRopeThreads / units, dr = dh0 / heads,
            dh = dh0 - dr * heads;
  uint4 x4[kAhead], y4[kAhead];
  uint4* out[kAhead];
  int uu[kAhead], rr[kAhead];
  auto load = [&](int e) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      uu[k] = -1;
      if (e + k * kRopeThreads < all) {
        const uint4* in = reinterpret_cast<const uint4*>(rope_in<E>(a, t0 + r, h));
        out[k] = reinterpret_cast<uint4*>(rope_out<E>(a, t0 + r, h));
        uu[k] = u;
        rr[k] = r;
        x4[k] = in[u < turned ? u : copied + (u - turned)];
        if (!PAIRS && u < turned) y4[k] = in[u + turned];
      }
      u += du;
      h += dh;
      r += dr;
      if (u >= units) u -= units, ++h;
      if (h >= heads) h -= heads, ++r;
    }
  };
  load(tid);
  rope_table(a, t0, rows, turn, s_pos, s_ok);
  for (int e = tid;;) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (uu[k] < 0 || !s_ok[rr[k]]) continue;
      if (uu[k] >= turned) {
        out[k][copied + (uu[k] - turned)] = x4[k];
        continue;
      }
      float x[V], y[V];
      const float2* cs = turn + rr[k] * half;
      RopeIo<E>::up(x4[k], x);
      if (PAIRS) {
#pragma unroll
        for (int i = 0; i < V / 2; i += 2) {
          const float4 w = *reinterpret_cast<const float4*>(cs + uu[k] * (V / 2) + i);
          y[2 * i] = x[2 * i] * w.x - x[2 * i + 1] * w.y;
          y[2 * i + 1] = x[2 * i] * w.y + x[2 * i + 1] * w.x;
          y[2 * i + 2] = x[2 * i + 2] * w.z - x[2 * i + 3] * w.w;
          y[2 * i + 3] = x[2 * i + 2] * w.w + x[2 * i + 3] * w.z;
        }
        out[k][uu[k]] = RopeIo<E>::down(y);
      } else {
        float z[V];
        RopeIo<E>::up(y4[k], y);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float4 w = *reinterpret_cast<const float4*>(cs + uu[k] * V + i);
          z[i] = x[i] * w.x - y[i] * w.y;
          y[i] = x[i] * w.y + y[i] * w.x;
          z[i + 1] = x[i + 1] * w.z - y[i + 1] * w.w;
          y[i + 1] = x[i + 1] * w.w + y[i + 1] * w.z;
        }
        out[k][uu[k]] = RopeIo<E>::down(z);
        out[k][uu[k] + turned] = RopeIo<E>::down(y);
      }
    }
    e += kAhead * kRopeThreads;
    if (e >= all) break;
    load(e);
  }
}

// Any other width (rot not a whole number of pieces): one pair, or one copied element, per
// thread and turn.
template <typename E>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const RopeArgs a, int rows) {
  extern __shared__ __align__(16) float2 turn[];
  __shared__ int64_t s_pos[kRopeRows];
  __shared__ int s_ok[kRopeRows];
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x, t0 = blockIdx.x * rows;
  rope_table(a, t0, rows, turn, s_pos, s_ok);
  const int heads = a.H_q + a.H_kv, half = a.rot / 2;
  const int units = half + (a.d - a.rot);
  for (int e = tid; e < rows * heads * units; e += kRopeThreads) {
    const int u = e % units, rh = e / units, h = rh % heads, r = rh / heads;
    if (!s_ok[r]) continue;
    const E* in = rope_in<E>(a, t0 + r, h);
    E* out = rope_out<E>(a, t0 + r, h);
    if (u >= half) {
      out[a.rot + u - half] = in[a.rot + u - half];
      continue;
    }
    const int i0 = a.interleaved ? 2 * u : u, i1 = a.interleaved ? 2 * u + 1 : u + half;
    const float2 w = turn[r * half + u];
    const float x = static_cast<float>(in[i0]), y = static_cast<float>(in[i1]);
    out[i0] = static_cast<E>(x * w.x - y * w.y);
    out[i1] = static_cast<E>(x * w.y + y * w.x);
  }
}

template <typename E>
static cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t s) {
  constexpr int V = RopeIo<E>::V;
  const bool pairs = a.interleaved != 0;
  const bool pieces = (pairs ? a.rot : a.rot / 2) % V == 0;
  // about two rounds of loads per thread where there are rows enough to keep every SM busy
  const int units = pieces ? (pairs ? a.rot / V : a.rot / 2 / V) + (a.d - a.rot) / V : a.d;
  const int full = 2 * kAhead * kRopeThreads / ((a.H_q + a.H_kv) * units);
  const int spread = a.T / (2 * device_sm_count());
  const int most = full < spread ? full : spread;
  const int rows = most < 1 ? 1 : most > kRopeRows ? kRopeRows : most;
  const unsigned grid = (unsigned)((a.T + rows - 1) / rows);
  const size_t smem = (size_t)rows * (a.rot / 2) * sizeof(float2);
  const auto kern = !pieces ? rope_any_kernel<E> : pairs ? rope_kernel<E, true> : rope_kernel<E, false>;
  return launch_after(kern, dim3(grid), dim3(kRopeThreads), smem, s, a, rows);
}

cudaError_t launch_rope(const RopeArgs& a, int io, cudaStream_t s) {
  if (io == TGDN_F32) return launch_rope_t<float>(a, s);
  if (io == TGDN_BF16) return launch_rope_t<__nv_bfloat16>(a, s);
  return launch_rope_t<__half>(a, s);
}

}  // namespace tgdn
