// decode_kv4.cu -- attention of the Sq newest tokens of each sequence over the
// 4-bit paged cache.
//
//     O = softmax(q K^T scale) V,   K = (ck - 8) sk,  V = (cv - 8) sv
//
// One block per (sequence, token, query head), four warps over the keys, each
// lane d / 32 channels of every key (one group's share), an online softmax per
// warp and one merge at the end.
#include <cuda_bf16.h>

#include "kernels.h"
#include "kv4.cuh"

namespace eio {
namespace {

constexpr int kDecWarps = 4;

template <int D>
__device__ __forceinline__ void k_channels(const uint8_t* tile, int tok, int lane, float* x) {
  constexpr int G = D / 32;
  // lane: channels 32 grp + lane of every group
#pragma unroll
  for (int grp = 0; grp < G; ++grp) {
    const uint8_t byte = tile[tok * (D / 2) + (lane >> 3) * (4 * G) + grp * 4 + ((lane & 7) >> 1)];
    const uint16_t s = *reinterpret_cast<const uint16_t*>(tile + kv4_off_ks(D) + tok * (2 * G) + grp * 2);
    x[grp] = static_cast<float>(static_cast<int>((byte >> (4 * (lane & 1))) & 15) - 8) * __uint_as_float(static_cast<uint32_t>(s) << 16);
  }
}

template <int D>
__device__ __forceinline__ void v_channels(const uint8_t* tile, int tok, int lane, float* x) {
  constexpr int G = D / 32;
#pragma unroll
  for (int grp = 0; grp < G; ++grp) {
    const uint8_t byte = tile[kv4_off_v(D) + (tok >> 3) * (4 * D) + (lane >> 2) * (16 * G) + ((tok & 7) >> 1) * (4 * G) +
                              grp * 4 + (tok & 1) * 2 + ((lane & 3) >> 1)];
    const uint16_t s = *reinterpret_cast<const uint16_t*>(tile + kv4_off_vs(D) + tok * (2 * G) + grp * 2);
    x[grp] = static_cast<float>(static_cast<int>((byte >> (4 * (lane & 1))) & 15) - 8) * __uint_as_float(static_cast<uint32_t>(s) << 16);
  }
}

template <int D>
__global__ void __launch_bounds__(kDecWarps * 32) decode_kv4_kernel(const DecodeKv4Args a) {
  constexpr int G = D / 32;
  const int row = blockIdx.x;  // [B, Sq, Hq]
  const int hq = row % a.Hq, sq = row / a.Hq % a.Sq, b = row / a.Hq / a.Sq;
  const int h = hq / (a.Hq / a.pages.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long room = static_cast<long long>(a.pages.max_pages) << a.pages.page_shift;
  int len = a.pages.seqlens[b];
  if (len < 0 || len > room) {
    atomicCAS(a.pages.err, 0, kErrDeviceArg);
    len = 0;
  }
  const int keys = len - a.Sq + sq + 1;
  float q[G], acc[G], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    q[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[static_cast<size_t>(row) * D + 32 * i + lane]);
    acc[i] = 0.f;
  }
  for (int j = warp; j < keys; j += kDecWarps) {
    const long long at = kv4_tile_at<D>(a.pages, b, h, j, kErrDeviceArg);
    if (at < 0) continue;
    float x[G];
    k_channels<D>(a.pages.pool + at, j & 15, lane, x);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), alpha = exp2f(m - (mn == -INFINITY ? 0.f : mn)), p = exp2f(s - (mn == -INFINITY ? 0.f : mn));
    v_channels<D>(a.pages.pool + at, j & 15, lane, x);
    l = fmaf(l, alpha, p);
#pragma unroll
    for (int i = 0; i < G; ++i) acc[i] = fmaf(acc[i], alpha, p * x[i]);
    m = mn;
  }
  __shared__ float sm[kDecWarps], sl[kDecWarps], so[kDecWarps][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < G; ++i) so[warp][32 * i + lane] = acc[i];
  __syncthreads();
  float M = -INFINITY, W = 0.f;
  for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kDecWarps; ++w) W += sl[w] * exp2f(sm[w] - (M == -INFINITY ? 0.f : M));
  for (int c = threadIdx.x; c < D; c += kDecWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kDecWarps; ++w) o += so[w][c] * exp2f(sm[w] - (M == -INFINITY ? 0.f : M));
    static_cast<__nv_bfloat16*>(a.o)[static_cast<size_t>(row) * D + c] = __float2bfloat16_rn(W == 0.f ? 0.f : o / W);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[(static_cast<size_t>(b) * a.Hq + hq) * a.Sq + sq] = W == 0.f ? -INFINITY : (M + log2f(W)) * 0.69314718055994530942f;
}

}  // namespace

size_t decode_kv4_workspace_bytes(int, int, int, int, long long, int) { return 0; }

cudaError_t launch_decode_kv4(int d, const DecodeKv4Args& a, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(a.pages.B) * a.Sq * a.Hq;
  if (d == 64) decode_kv4_kernel<64><<<blocks, kDecWarps * 32, 0, s>>>(a);
  else decode_kv4_kernel<128><<<blocks, kDecWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace eio
