// rope.cu -- rotary positions with several axes, for q and k in one launch.
//
// Pair p of a head (channels p and p + d/2, or 2p and 2p + 1) is rotated by
//     theta = positions[b, n, axis(p)] * freq(p)
//     (x, y) -> (x cos theta - y sin theta, x sin theta + y cos theta);
// pairs behind the table stay as they are.  The backward is the rotation by
// -theta.
//
// Angles: theta / 2 pi modulo 1 as a 64-bit fixed-point fraction.  The host
// turns freq into F = freq / 2 pi * 2^64 (modulo 2^64); position * F in 64-bit
// integers is then reduced exactly, with an error below |position| * 2^-64
// turns, however far the position; its upper 32 bits, as a signed fraction of
// a half turn, go to sincospif.  In fp32 the product alone would be off by
// 2^-24 of its size: 0.06 rad at a position of a million.
//
// Memory bound: q and k are read and written once.  A block takes a run of
// tokens; it computes the cosines and sines of its (token, pair)s once into
// shared memory, then its threads stream over (token, head, eight pairs) with
// 16-byte loads and stores.
#include <cuda_bf16.h>

#include "kernels.h"

namespace eio {
namespace {

constexpr int kRopeThreads = 256;

struct Pairs8 {
  float a[8], b[8];
};

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return u;
}

// The 16 channels of eight pairs as two runs of eight: lo and hi halves of a
// head, or (interleaved) one run of 16.
template <typename T>
__device__ __forceinline__ void load_runs(const T* lo, const T* hi, float* a, float* b) {
  if constexpr (sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(lo), v = *reinterpret_cast<const uint4*>(hi);
    unpack8(u, a);
    unpack8(v, b);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(lo + 4 * i), v = *reinterpret_cast<const float4*>(hi + 4 * i);
      a[4 * i] = u.x, a[4 * i + 1] = u.y, a[4 * i + 2] = u.z, a[4 * i + 3] = u.w;
      b[4 * i] = v.x, b[4 * i + 1] = v.y, b[4 * i + 2] = v.z, b[4 * i + 3] = v.w;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store_runs(T* lo, T* hi, const float* a, const float* b) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(lo) = pack8(a);
    *reinterpret_cast<uint4*>(hi) = pack8(b);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<float4*>(lo + 4 * i) = make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
      *reinterpret_cast<float4*>(hi + 4 * i) = make_float4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
    }
  }
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 cs[];  // [tokens of the block][pairs, rounded up to 8]
  const int chunks = a.d / 16, half = a.d / 2;
  const int padded = chunks * 8;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long first = static_cast<long long>(blockIdx.x) * a.tokens_per_block;
  const int nt = static_cast<int>(min(static_cast<long long>(a.tokens_per_block), tokens - first));

  for (int i = threadIdx.x; i < nt * padded; i += kRopeThreads) {
    const int t = i / padded, p = i % padded;
    float s = 0.f, c = 1.f;
    if (p < a.n_pairs) {
      const long long tok = first + t;
      const long long pos = a.positions[tok / a.N * a.p_sb + tok % a.N * a.p_sn + a.axis[p]];
      const unsigned long long turns = static_cast<unsigned long long>(pos) * a.freq[p];
      sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
      if (a.inverse) s = -s;
    }
    cs[i] = make_float2(c, s);
  }
  __syncthreads();

  const int heads = a.Hq + a.Hk;
  const int items = nt * heads * chunks;
  for (int i = threadIdx.x; i < items; i += kRopeThreads) {
    const int chunk = i % chunks, row = i / chunks;
    const int t = row / heads, h = row % heads;
    const long long tok = first + t;
    const long long b = tok / a.N, n = tok % a.N;
    const bool isq = h < a.Hq;
    const long long in_at = isq ? b * a.q_sb + n * a.q_sn + h * a.d : b * a.k_sb + n * a.k_sn + (h - a.Hq) * a.d;
    const long long out_at = isq ? b * a.qo_sb + n * a.qo_sn + h * a.d : b * a.ko_sb + n * a.ko_sn + (h - a.Hq) * a.d;
    const T* in = static_cast<const T*>(isq ? a.q : a.k) + in_at;
    T* out = static_cast<T*>(isq ? a.q_out : a.k_out) + out_at;
    const int lo = INTERLEAVED ? 16 * chunk : 8 * chunk, hi = INTERLEAVED ? 16 * chunk + 8 : half + 8 * chunk;
    float x[8], y[8];
    load_runs(in + lo, in + hi, x, y);
    const float2* w = cs + t * padded + 8 * chunk;
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float* r = j < 4 ? x + 2 * j : y + 2 * j - 8;
        const float u = r[0], v = r[1];
        r[0] = u * w[j].x - v * w[j].y;
        r[1] = u * w[j].y + v * w[j].x;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = x[j], v = y[j];
        x[j] = u * w[j].x - v * w[j].y;
        y[j] = u * w[j].y + v * w[j].x;
      }
    }
    store_runs(out + lo, out + hi, x, y);
  }
}

template <typename T, bool INTERLEAVED>
cudaError_t launch_t(const RopeArgs& a, cudaStream_t s) {
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long blocks = (tokens + a.tokens_per_block - 1) / a.tokens_per_block;
  const size_t smem = static_cast<size_t>(a.tokens_per_block) * (a.d / 2) * sizeof(float2);
  rope_kernel<T, INTERLEAVED><<<static_cast<unsigned>(blocks), kRopeThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(bool bf16, bool interleaved, RopeArgs a, cudaStream_t s) {
  a.tokens_per_block = 4;
  if (bf16) return interleaved ? launch_t<__nv_bfloat16, true>(a, s) : launch_t<__nv_bfloat16, false>(a, s);
  return interleaved ? launch_t<float, true>(a, s) : launch_t<float, false>(a, s);
}

}  // namespace eio
