// copy_pages.cu -- pages of a pool copied to other pages of it, for forked
// sequences (their last, partly filled page) and for pools made dense.
//
// The page numbers come from the host and travel as kernel parameters: no
// device list, no copy before the launch, and a captured graph holds its own.
// No destination is also a source or named twice (the caller of the launcher
// has checked), so the copies are independent.  Memory bound: every byte is
// read once and written once.
#include "kernels.h"

namespace eio {
namespace {

constexpr int kCopyThreads = 256;

template <int N>
struct Moves {
  int src[N], dst[N];
};

template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(uint8_t* pool, long long page_bytes, const __grid_constant__ Moves<N> m) {
  const uint4* from = reinterpret_cast<const uint4*>(pool + m.src[blockIdx.y] * page_bytes);
  uint4* to = reinterpret_cast<uint4*>(pool + m.dst[blockIdx.y] * page_bytes);
  const long long n = page_bytes / 16;
  for (long long i = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; i < n; i += static_cast<long long>(gridDim.x) * kCopyThreads)
    to[i] = from[i];
}

template <int N>
cudaError_t launch_n(void* pool, long long page_bytes, const int* src, const int* dst, int n, cudaStream_t s) {
  Moves<N> m;
  for (int i = 0; i < n; ++i) m.src[i] = src[i], m.dst[i] = dst[i];
  const long long chunks = (page_bytes / 16 + 4 * kCopyThreads - 1) / (4 * kCopyThreads);
  const dim3 grid(static_cast<unsigned>(chunks < 64 ? chunks : 64), n);
  copy_pages_kernel<N><<<grid, kCopyThreads, 0, s>>>(static_cast<uint8_t*>(pool), page_bytes, m);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_copy_pages(void* pool, long long page_bytes, const int* src, const int* dst, int n, cudaStream_t s) {
  constexpr int kMost = 500;  // 4000 bytes of parameters
  for (int i = 0; i < n; i += kMost) {
    const cudaError_t e = launch_n<kMost>(pool, page_bytes, src + i, dst + i, n - i < kMost ? n - i : kMost, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace eio
