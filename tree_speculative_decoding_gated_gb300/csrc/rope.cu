// rope.cu — rotary positions of q and k.
//
// Pair i of a head is turned by p f_i (p: the row's position).  The turn p f_i / (2 pi) is
// formed as p times a 64-bit binary fraction, which wraps at whole turns exactly (2^-64 of a
// turn per position), so a position of a million keeps the phase that fp32 angles lose.
//
// Bound by memory: every element is read and written once.  A CTA takes a few rows; their
// rot/2 cosines and sines go to shared memory once per row and serve all its heads, then
// each thread turns 16-byte pieces (in the half layout the two pieces of its pairs).
#include <cuda_fp16.h>

#include "tgdn_device.cuh"
#include "tgdn_kernels.h"

namespace tgdn {

constexpr int kRopeThreads = 256;

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

// The sequence of row t, or -1: the last b with cu[b] <= t, if its range is sound.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int T, int t) {
  int lo = 0, hi = B;  // cu[lo] <= t is kept where it holds at all
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int c0 = cu[lo], c1 = cu[lo + 1];
  return c0 >= 0 && c0 <= t && t < c1 && c1 <= T ? lo : -1;
}

// rows: rows per CTA.  PAIRED: the half layout with rot / 2 a multiple of the 16-byte piece,
// so that a thread holds both pieces of its pairs; otherwise element by element.
template <typename E>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int rows) {
  extern __shared__ float2 turn[];  // [rows][rot / 2]: mscale (cos, sin)
  constexpr int V = RopeIo<E>::V;
  __shared__ int64_t s_pos[32];
  __shared__ int s_ok[32];
  const int tid = threadIdx.x, t0 = blockIdx.x * rows;
  const int half = a.rot / 2;
  if (tid < rows) {
    const int t = t0 + tid;
    const int b = t < a.T ? sequence_of(a.cu, a.B, a.T, t) : -1;
    s_ok[tid] = b >= 0;
    if (b >= 0)
      s_pos[tid] = (int64_t)(a.base ? a.base[b] : 0) + (a.off ? a.off[t] : t - a.cu[b]);
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
  const int pieces = a.d / V, heads = a.H_q + a.H_kv;
  auto row_in = [&](int r, int h) -> const E* {
    const int64_t t = t0 + r;
    return h < a.H_q ? static_cast<const E*>(a.q) + t * a.q_stride + (int64_t)h * a.d
                     : static_cast<const E*>(a.k) + t * a.k_stride + (int64_t)(h - a.H_q) * a.d;
  };
  auto row_out = [&](int r, int h) -> E* {
    const int64_t t = t0 + r;
    return h < a.H_q
               ? static_cast<E*>(a.q_out) + t * a.q_out_stride + (int64_t)h * a.d
               : static_cast<E*>(a.k_out) + t * a.k_out_stride + (int64_t)(h - a.H_q) * a.d;
  };
  if (a.interleaved ? a.rot % V == 0 : half % V == 0) {
    // units: in the half layout a pair of pieces (p, p + half / V), else one piece; the
    // pieces past rot are copied
    const int turned = a.interleaved ? a.rot / V : half / V;
    const int units = turned + (pieces - a.rot / V);
    for (int e = tid; e < rows * heads * units; e += kRopeThreads) {
      const int u = e % units, rh = e / units, h = rh % heads, r = rh / heads;
      if (!s_ok[r]) continue;
      const uint4* in = reinterpret_cast<const uint4*>(row_in(r, h));
      uint4* out = reinterpret_cast<uint4*>(row_out(r, h));
      if (u >= turned) {
        const int p = a.rot / V + (u - turned);
        if (in != out) out[p] = in[p];
        continue;
      }
      float x[V], y[V];
      const float2* cs = turn + r * half;
      if (a.interleaved) {
        RopeIo<E>::up(in[u], x);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const float2 w = cs[u * (V / 2) + i];
          y[2 * i] = x[2 * i] * w.x - x[2 * i + 1] * w.y;
          y[2 * i + 1] = x[2 * i] * w.y + x[2 * i + 1] * w.x;
        }
        out[u] = RopeIo<E>::down(y);
      } else {
        float z[V];
        RopeIo<E>::up(in[u], x);
        RopeIo<E>::up(in[u + turned], y);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 w = cs[u * V + i];
          z[i] = x[i] * w.x - y[i] * w.y;
          y[i] = x[i] * w.y + y[i] * w.x;
        }
        out[u] = RopeIo<E>::down(z);
        out[u + turned] = RopeIo<E>::down(y);
      }
    }
    return;
  }
  // any other width: one pair, or one copied element, per thread
  const int units = half + (a.d - a.rot);
  for (int e = tid; e < rows * heads * units; e += kRopeThreads) {
    const int u = e % units, rh = e / units, h = rh % heads, r = rh / heads;
    if (!s_ok[r]) continue;
    const E* in = row_in(r, h);
    E* out = row_out(r, h);
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
  const int rows = a.T >= 8 * device_sm_count() * 4 ? 8 : a.T >= 2 * device_sm_count() ? 2 : 1;
  const unsigned grid = (unsigned)((a.T + rows - 1) / rows);
  rope_kernel<E><<<grid, kRopeThreads, (size_t)rows * (a.rot / 2) * sizeof(float2), s>>>(a, rows);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs& a, int io, cudaStream_t s) {
  if (io == TGDN_F32) return launch_rope_t<float>(a, s);
  if (io == TGDN_BF16) return launch_rope_t<__nv_bfloat16>(a, s);
  return launch_rope_t<__half>(a, s);
}

}  // namespace tgdn
