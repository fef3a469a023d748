// kv4_rows.cu -- rows of K and V into the pages of the 4-bit cache, and back.
//
// kv4_append: the group of 32 channels x of one token and head is stored as
//     m = max |x|,  s = bf16(m / 7),  c = 8 + floor(x / s + 1/2)
// kv4_read: (c - 8) * s, rounded once to bf16.
//
// Both are memory bound: per token and head 4 d bytes of bf16 rows and
// d + d / 8 bytes of cache, with about ten instructions a channel pair.
#include <cuda_bf16.h>

#include "kernels.h"
#include "kv4.cuh"

namespace eio {
namespace {

constexpr int kRowThreads = 256;

// The tokens that sequence b appends: rows 0 .. n - 1 of the call's k and v, at
// positions len - n .. len - 1; none (and the error latched) for counts that
// do not fit the rows, the sequence or the table.
__device__ __forceinline__ int append_count(const Kv4AppendArgs& a, int b, int* first) {
  const int len = a.pages.seqlens[b];
  const int n = a.n_new ? a.n_new[b] : a.N;
  const long long room = static_cast<long long>(a.pages.max_pages) << a.pages.page_shift;
  if (n < 0 || n > a.N || len < n || len > room) {
    atomicCAS(a.pages.err, 0, kErrDeviceArg);
    return 0;
  }
  *first = len - n;
  return n;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  constexpr int G = D / 32;
  const long long total = static_cast<long long>(a.pages.B) * a.N * a.pages.Hkv * G;
  const long long i = static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i >= total) return;
  const int grp = static_cast<int>(i % G);
  const long long row = i / G;
  const int h = static_cast<int>(row % a.pages.Hkv);
  const int n = static_cast<int>(row / a.pages.Hkv % a.N), b = static_cast<int>(row / a.pages.Hkv / a.N);
  int first = 0;
  if (n >= append_count(a, b, &first)) return;
  const int pos = first + n, tok = pos & 15;
  const long long at = kv4_tile_at<D>(a.pages, b, h, pos, kErrDeviceArg);
  if (at < 0) return;
  uint8_t* tile = a.pages.pool + at;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(which ? a.v : a.k) +
                               (which ? b * a.v_sb + n * a.v_sn : b * a.k_sb + n * a.k_sn) + h * D + grp * 32;
    uint32_t w[16];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 u = reinterpret_cast<const uint4*>(src)[j];
      w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
    const uint32_t s = kv4_scale_bits(m);
    const float inv = kv4_inverse(s);
    uint32_t out[4];  // eight channels each, low nibble first
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = w[4 * j + k];
        // a group that holds infinities or NaNs has code 8 everywhere
        const float lo = inv == 0.f ? 0.f : __uint_as_float(x << 16), hi = inv == 0.f ? 0.f : __uint_as_float(x & 0xffff0000u);
        o |= kv4_code(lo, inv) << (8 * k) | kv4_code(hi, inv) << (8 * k + 4);
      }
      out[j] = o;
    }
    if (which == 0) {
#pragma unroll
      for (int t = 0; t < 4; ++t) *reinterpret_cast<uint32_t*>(tile + tok * (D / 2) + t * (4 * G) + grp * 4) = out[t];
    } else {
      uint8_t* v = tile + kv4_off_v(D) + (tok >> 3) * (4 * D) + ((tok & 7) >> 1) * (4 * G) + grp * 4 + (tok & 1) * 2;
#pragma unroll
      for (int g = 0; g < 8; ++g) *reinterpret_cast<uint16_t*>(v + g * (16 * G)) = static_cast<uint16_t>(out[g >> 1] >> (16 * (g & 1)));
    }
    *reinterpret_cast<uint16_t*>(tile + (which ? kv4_off_vs(D) : kv4_off_ks(D)) + tok * (2 * G) + grp * 2) = static_cast<uint16_t>(s);
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const Kv4ReadArgs a) {
  constexpr int G = D / 32;
  const long long total = static_cast<long long>(a.pages.B) * a.N * a.pages.Hkv * G;
  const long long i = static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i >= total) return;
  const int grp = static_cast<int>(i % G);
  const long long row = i / G;
  const int h = static_cast<int>(row % a.pages.Hkv);
  const int n = static_cast<int>(row / a.pages.Hkv % a.N), b = static_cast<int>(row / a.pages.Hkv / a.N);
  const long long room = static_cast<long long>(a.pages.max_pages) << a.pages.page_shift;
  int len = a.pages.seqlens[b], start = a.start ? a.start[b] : 0;
  if (len < 0 || len > room || start < 0) {
    atomicCAS(a.pages.err, 0, kErrDeviceArg);
    len = 0;
    start = 0;
  }
  const long long pos = static_cast<long long>(start) + n;
  const long long at = pos < len ? kv4_tile_at<D>(a.pages, b, h, static_cast<int>(pos), kErrDeviceArg) : -1;
  const int tok = static_cast<int>(pos & 15);
  const uint8_t* tile = a.pages.pool + (at < 0 ? 0 : at);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(which ? a.v : a.k) + row * D + grp * 32);
    uint32_t w[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
    float s = 0.f;
    if (at >= 0) {
      const uint16_t sb = *reinterpret_cast<const uint16_t*>(tile + (which ? kv4_off_vs(D) : kv4_off_ks(D)) + tok * (2 * G) + grp * 2);
      s = __uint_as_float(static_cast<uint32_t>(sb) << 16);
      if (which == 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const uint32_t*>(tile + tok * (D / 2) + t * (4 * G) + grp * 4);
      } else {
        const uint8_t* v = tile + kv4_off_v(D) + (tok >> 3) * (4 * D) + ((tok & 7) >> 1) * (4 * G) + grp * 4 + (tok & 1) * 2;
#pragma unroll
        for (int g = 0; g < 8; g += 2)
          w[g >> 1] = *reinterpret_cast<const uint16_t*>(v + g * (16 * G)) |
                      static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(v + (g + 1) * (16 * G))) << 16;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 u;
      __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float lo = static_cast<float>(static_cast<int>((w[j] >> (8 * k)) & 15u) - 8);
        const float hi = static_cast<float>(static_cast<int>((w[j] >> (8 * k + 4)) & 15u) - 8);
        o[k] = __floats2bfloat162_rn(lo * s, hi * s);
      }
      dst[j] = u;
    }
  }
}

template <typename A>
unsigned row_blocks(const A& a, int d) {
  const long long total = static_cast<long long>(a.pages.B) * a.N * a.pages.Hkv * (d / 32);
  return static_cast<unsigned>((total + kRowThreads - 1) / kRowThreads);
}

}  // namespace

cudaError_t launch_kv4_append(int d, const Kv4AppendArgs& a, cudaStream_t s) {
  if (d == 64) kv4_append_kernel<64><<<row_blocks(a, d), kRowThreads, 0, s>>>(a);
  else kv4_append_kernel<128><<<row_blocks(a, d), kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(int d, const Kv4ReadArgs& a, cudaStream_t s) {
  if (d == 64) kv4_read_kernel<64><<<row_blocks(a, d), kRowThreads, 0, s>>>(a);
  else kv4_read_kernel<128><<<row_blocks(a, d), kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace eio
