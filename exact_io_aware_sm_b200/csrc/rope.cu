// rope.cu -- rotary positions with several axes, for q and k in one launch.
//
// Pair p of a head (channels p and p + d/2, or 2p and 2p + 1) is rotated by
//     theta = positions[b, n, axis(p)] * freq(p)
//     (x, y) -> (x cos theta - y sin theta, x sin theta + y cos theta);
// pairs behind the table are copied bit by bit (a rotation by 0 would carry a partner's
// infinity or NaN over and lose the sign of a zero, and a bf16 NaN its bits when it is
// rounded again).  The backward is the rotation by -theta.
//
// Angles: theta / 2 pi modulo 1 as a 64-bit fixed-point fraction.  The host
// turns freq into F = freq / 2 pi * 2^64 (modulo 2^64); position * F in 64-bit
// integers is then reduced exactly, with an error below |position| * 2^-64
// turns, however far the position; its upper 32 bits, as a signed fraction of
// a half turn rounded to fp32 (pi 2^-25 = 2^-23.3 rad), go to sincospif.  In fp32 the product
// alone would be off by 2^-24 of its size: 0.06 rad at a position of a million.
//
// Memory bound: q and k are read and written once.  A block takes a run of
// tokens; it computes the cosines and sines of its (token, pair)s once into
// shared memory (for every head) while the first pieces of work (token, head, eight
// pairs) are on their way, then its threads stream over them with 16-byte loads and
// stores, four pieces in flight.  24960 tokens of 48 heads of 128 (613 MB): 98 us alone,
// 6.2 TB/s of the 6.46 that a copy reaches (112 when the interleaved form read
// 32 bytes a thread in two halves); the GPT-2 training step's q and k (25 MB), cold: 13.
#include <cuda_bf16.h>

#include "kernels_kv4.h"

namespace eio {
namespace {

constexpr int kRopeThreads = 256;

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

// The 16 channels of a piece of work: eight pairs, in 16-byte words that the threads
// of a head's kChunks pieces read and write side by side.  Word i of piece c is channels
// V (c + kChunks i) .. + V - 1 with V = 16 / sizeof(T): i < kWords / 2 are in the head's
// lower half and word i + kWords / 2 holds their partners, or (interleaved) every word its own pairs.
template <typename T>
struct Piece {
  static constexpr int V = 16 / sizeof(T), kWords = 16 / V;
  uint4 word[kWords];
};

// Which of a piece's eight pairs pair p of a head is, and of which piece.
template <typename T, int CHUNKS, bool INTERLEAVED>
__device__ __forceinline__ int place_of_pair(int p, int* chunk) {
  constexpr int kPairs = INTERLEAVED ? Piece<T>::V / 2 : Piece<T>::V;  // of a word
  const int w = p / kPairs;
  *chunk = w % CHUNKS;
  return w / CHUNKS * kPairs + p % kPairs;
}

template <typename T>
__device__ __forceinline__ void open_word(const uint4& u, float* f) {
  if constexpr (sizeof(T) == 2) {
    unpack8(u, f);
  } else {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
}

template <typename T>
__device__ __forceinline__ uint4 close_word(const float* f) {
  if constexpr (sizeof(T) == 2) return pack8(f);
  else return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// The first `live` of a word's eight bf16 values from x, the others from `old`, bit by bit.
__device__ __forceinline__ uint4 first_of(const uint4& x, const uint4& old, int live) {
  auto two = [&](uint32_t a, uint32_t b, int i) { return live > i + 1 ? a : live == i + 1 ? __byte_perm(a, b, 0x7610) : b; };
  return make_uint4(two(x.x, old.x, 0), two(x.y, old.y, 2), two(x.z, old.z, 4), two(x.w, old.w, 6));
}

template <typename T>
constexpr int kRopeEach = sizeof(T) == 2 ? 4 : 2;  // pieces of work that a thread has in flight: 128 bytes

// PARTIAL: the table has fewer than D / 2 pairs.  A kernel of its own, since the words as they were read and
// what tells the pairs apart cost registers: in one kernel for both, whole tables in fp32 took 95 -> 97 to 101 us
// (613 MB).  Partial ones take 95 in fp32 and 101 to 103 in bf16 (95 and 99 when the rest was rotated by 0).
template <typename T, int D, bool INTERLEAVED, bool PARTIAL>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kEach = kRopeEach<T>;
  constexpr int kChunks = D / 16, kHalf = D / 2;  // pieces of eight pairs, pairs of a head
  // Cosine and sine: two pairs of piece c at [token][2 of its pairs][c], so that the pieces' reads are consecutive.
  extern __shared__ float4 cs[];
  const int first = static_cast<int>(blockIdx.x) * a.tokens_per_block;
  const int nt = min(a.tokens_per_block, a.B * a.N - first);
  const int b0 = first / a.N, n0 = first - b0 * a.N;

  const int heads = a.Hq + a.Hk, items = nt * heads * kChunks;
  const int chunk = threadIdx.x % kChunks;  // kRopeThreads is a multiple of kChunks: the same for all of a thread's items
  constexpr int V = Piece<T>::V, kWords = Piece<T>::kWords;
  constexpr int kPairs = INTERLEAVED ? V / 2 : V;  // of a word
  Piece<T> piece[kEach];
  T* out[kEach];
  int tok[kEach];
  auto load = [&](int i0) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = i0 + e * kRopeThreads;
      if (i >= items) break;
      const int row = i / kChunks, t = row / heads, h = row - t * heads;
      tok[e] = t;
      int b = b0, n = n0 + t;
      while (n >= a.N) n -= a.N, ++b;
      const T* in;
      if (h < a.Hq) {
        in = static_cast<const T*>(a.q) + b * a.q_sb + n * a.q_sn + h * D;
        out[e] = static_cast<T*>(a.q_out) + b * a.qo_sb + n * a.qo_sn + h * D;
      } else {
        in = static_cast<const T*>(a.k) + b * a.k_sb + n * a.k_sn + (h - a.Hq) * D;
        out[e] = static_cast<T*>(a.k_out) + b * a.ko_sb + n * a.ko_sn + (h - a.Hq) * D;
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w) piece[e].word[w] = __ldcs(reinterpret_cast<const uint4*>(in + V * (chunk + kChunks * w)));
    }
  };
  load(threadIdx.x);  // on its way while the angles are computed

  for (int i = threadIdx.x; i < nt * kHalf; i += kRopeThreads) {
    const int t = i / kHalf, p = i % kHalf;
    float s = 0.f, c = __uint_as_float(0x7fffffffu);  // NaN: no rotation
    if (!PARTIAL || p < a.n_pairs) {
      int b = b0, n = n0 + t;
      while (n >= a.N) n -= a.N, ++b;
      const long long pos = a.positions[b * a.p_sb + n * a.p_sn + a.axis[p]];
      const unsigned long long turns = static_cast<unsigned long long>(pos) * a.freq[p];
      sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
      if (a.inverse) s = -s;
    }
    int of;
    const int at = place_of_pair<T, kChunks, INTERLEAVED>(p, &of);
    reinterpret_cast<float2*>(cs)[2 * (t * (kHalf / 2) + at / 2 * kChunks + of) + at % 2] = make_float2(c, s);
  }
  __syncthreads();

  for (int i0 = threadIdx.x; i0 < items; i0 += kEach * kRopeThreads) {
    if (i0 != threadIdx.x) load(i0);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (i0 + e * kRopeThreads >= items) break;
      float x[16];
#pragma unroll
      for (int w = 0; w < kWords; ++w) open_word<T>(piece[e].word[w], x + V * w);
      const float4* turn = cs + tok[e] * (kHalf / 2) + chunk;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 r = turn[j * kChunks];  // pairs 2 j and 2 j + 1
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float c = k ? r.z : r.x, s = k ? r.w : r.y;
          const int p = 2 * j + k, i = INTERLEAVED ? 2 * p : p, partner = INTERLEAVED ? i + 1 : i + 8;
          const float u = x[i], v = x[partner];
          if (PARTIAL && sizeof(T) == 4 && c != c) continue;  // behind the table
          x[i] = u * c - v * s;
          x[partner] = u * s + v * c;
        }
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        uint4 y = close_word<T>(x + V * w);
        if constexpr (PARTIAL && sizeof(T) == 2) {
          const int pair = kPairs * (chunk + kChunks * (INTERLEAVED ? w : w % (kWords / 2)));  // the word's first
          y = first_of(y, piece[e].word[w], (a.n_pairs - pair) * (V / kPairs));
        }
        *reinterpret_cast<uint4*>(out[e] + V * (chunk + kChunks * w)) = y;
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(bool interleaved, const RopeArgs& a, cudaStream_t s) {
  const int tokens = a.B * a.N;
  const int blocks = (tokens - 1) / a.tokens_per_block + 1;
  const size_t smem = static_cast<size_t>(a.tokens_per_block) * D / 2 * sizeof(float2);
  auto launch = [&](auto kernel) { kernel<<<blocks, kRopeThreads, smem, s>>>(a); };
  if (a.n_pairs < D / 2) launch(interleaved ? rope_kernel<T, D, true, true> : rope_kernel<T, D, false, true>);
  else launch(interleaved ? rope_kernel<T, D, true, false> : rope_kernel<T, D, false, false>);
  return cudaGetLastError();
}

}  // namespace

// Tokens of a block: one round of its threads' pieces where there are blocks enough for every SM to hold
// four, fewer tokens where there are not.
cudaError_t launch_rope(bool bf16, bool interleaved, RopeArgs a, cudaStream_t s) {
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long per_token = static_cast<long long>(a.Hq + a.Hk) * (a.d / 16);
  long long each = kRopeThreads * (bf16 ? kRopeEach<__nv_bfloat16> : kRopeEach<float>) / per_token;
  if (each > tokens / (4 * 148)) each = tokens / (4 * 148);
  a.tokens_per_block = each < 1 ? 1 : each > 16 ? 16 : static_cast<int>(each);
  switch (a.d) {
    case 32: return bf16 ? launch_t<__nv_bfloat16, 32>(interleaved, a, s) : launch_t<float, 32>(interleaved, a, s);
    case 64: return bf16 ? launch_t<__nv_bfloat16, 64>(interleaved, a, s) : launch_t<float, 64>(interleaved, a, s);
    default: return bf16 ? launch_t<__nv_bfloat16, 128>(interleaved, a, s) : launch_t<float, 128>(interleaved, a, s);
  }
}

}  // namespace eio
