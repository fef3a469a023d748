// copy_pages.cu -- pages of a pool copied to other pages of it, for forked
// sequences (their last, partly filled page) and for pools made dense.
//
// The page numbers come from the host and travel as kernel parameters: no
// device list, no copy before the launch, and a captured graph holds its own.
// No destination is also a source or named twice (the caller of the launcher
// has checked), so the copies are independent.  Memory bound: every byte is
// read once and written once.  4000 pages of 73,728 bytes: 91 us, 6.5 TB/s, in one launch
// (eight launches of 500 took 132).
#include "kernels_kv4.h"

namespace eio {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 4;                            // 16-byte pieces of a thread, all in flight at once
constexpr int kCopyChunk = kCopyThreads * kCopyEach;  // of a block: 16 KB

template <int N>
struct Moves {
  int src[N], dst[N];
};

template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(uint8_t* pool, long long page_bytes, const __grid_constant__ Moves<N> m) {
  const long long n = page_bytes / 16, at = static_cast<long long>(blockIdx.x) * kCopyChunk + threadIdx.x;
  const uint4* from = reinterpret_cast<const uint4*>(pool + m.src[blockIdx.y] * page_bytes) + at;
  uint4* to = reinterpret_cast<uint4*>(pool + m.dst[blockIdx.y] * page_bytes) + at;
  uint4 x[kCopyEach];
#pragma unroll
  for (int i = 0; i < kCopyEach; ++i)
    if (at + i * kCopyThreads < n) x[i] = __ldcs(from + i * kCopyThreads);
#pragma unroll
  for (int i = 0; i < kCopyEach; ++i)
    if (at + i * kCopyThreads < n) __stcs(to + i * kCopyThreads, x[i]);
}

template <int N>
cudaError_t launch_n(void* pool, long long page_bytes, const int* src, const int* dst, int n, cudaStream_t s) {
  Moves<N> m;
  for (int i = 0; i < n; ++i) m.src[i] = src[i], m.dst[i] = dst[i];
  const long long chunks = (page_bytes / 16 + kCopyChunk - 1) / kCopyChunk;
  if (chunks > 0x7fffffffll) return cudaErrorInvalidValue;
  copy_pages_kernel<N><<<dim3(static_cast<unsigned>(chunks), n), kCopyThreads, 0, s>>>(static_cast<uint8_t*>(pool), page_bytes, m);
  return cudaGetLastError();
}

}  // namespace

// One launch takes up to 4000 moves (32 KB of parameters are the most); few moves take little ones.
cudaError_t launch_copy_pages(void* pool, long long page_bytes, const int* src, const int* dst, int n, cudaStream_t s) {
  constexpr int kFew = 32, kMost = 4000;
  if (n <= kFew) return launch_n<kFew>(pool, page_bytes, src, dst, n, s);
  for (int i = 0; i < n; i += kMost) {
    const cudaError_t e = launch_n<kMost>(pool, page_bytes, src + i, dst + i, n - i < kMost ? n - i : kMost, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace eio
