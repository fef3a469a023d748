// kv4_rows.cu -- rows of K and V into the pages of the 4-bit cache, and back.
//
// kv4_append: the group of 32 channels x of one token and head is stored as
//     m = max |x|,  s = bf16(m / 7),  c = 8 + floor(x / s + 1/2)
// kv4_read: (c - 8) * s, rounded once to bf16.
//
// One warp a tile of the cache (16 tokens of one head), whatever part of it the
// call covers: lane (g, t) takes channels 8 t .. 8 t + 7 of every group of tokens
// g and g + 8, so that rows move in 16-byte pieces (64 contiguous bytes a group and
// token), codes in 16-byte pieces too, and the maximum of a group needs two shuffles.
// K's codes are then in place; V's pairs of tokens exchange halves with the lane of
// the other token.  A token's bytes are its own: a tile that is covered in part
// is written in part, never read.
//
// Both move, per token and head, 4 d bytes of bf16 rows and d + d / 8 bytes of cache.
// 16384 tokens of 8 heads of 128 (86 MB each way, 13.3 us at the rate of a copy): append
// 18.5 us, read 15.4; a thread a group of 32 channels, with its scattered stores, took 58
// for both.  The append fills no pipe (9 instructions a value; the integer pipe is busy for
// 53 % of the cycles, issue slots 55 %): its blocks make 2.3 rounds of 6 an SM, each of
// which loads, narrows and stores once, so that the rounds' loads and arithmetic hardly overlap.
#include <cuda_bf16.h>

#include "kernels_kv4.h"
#include "kv4.cuh"

namespace eio {
namespace {

constexpr int kRowWarps = 4;

// Tiles that n consecutive tokens may touch.
__host__ __device__ constexpr int tiles_of(int n) { return (n + 14) / 16 + 1; }

struct TileAt {
  int b, tile, h;  // the tile'th of those that sequence b's tokens touch
  bool ok;
};

// Blocks of a sequence: a warp each (tile, head).
__host__ __device__ constexpr unsigned blocks_of(int N, int Hkv) {
  return (static_cast<unsigned>(tiles_of(N)) * static_cast<unsigned>(Hkv) + kRowWarps - 1) / kRowWarps;
}

__device__ __forceinline__ TileAt my_tile(int Hkv, int N) {
  const unsigned blocks = blocks_of(N, Hkv), b = blockIdx.x / blocks;
  const unsigned i = (blockIdx.x - b * blocks) * kRowWarps + (threadIdx.x >> 5), tile = i / static_cast<unsigned>(Hkv);
  return {static_cast<int>(b), static_cast<int>(tile), static_cast<int>(i - tile * Hkv), tile < static_cast<unsigned>(tiles_of(N))};
}

// A lane's group words [G] to or from 4 G consecutive bytes.
template <int G>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t* w) {
  if constexpr (G == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int G>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (G == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  }
}

// The largest magnitudes of a lane's eight channels of a group, two at a time in the halves of a word.
__device__ __forceinline__ uint32_t largest8(const uint4& x) {
  return __vimax3_u16x2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}

// A row of G groups, eight channels of each here and the others in three more lanes: the codes of the eight (low
// nibbles first) and the scales, two groups to a word.
template <int G>
__device__ __forceinline__ void narrow(const uint4* x, uint32_t* codes, uint32_t* scales) {
#pragma unroll
  for (int i = 0; i < G / 2; ++i) {
    const uint32_t a = largest8(x[2 * i]), b = largest8(x[2 * i + 1]);
    uint32_t m = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));  // of the first group, of the second
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    uint32_t s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t mk = k ? m >> 16 : m & 0xffffu;
      const bool has = kv4_has_codes(mk);
      s[k] = kv4_scale_bits(mk, has);
      const uint4& u = x[2 * i + k];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      codes[2 * i + k] = has ? kv4_codes(w, kv4_inverse(s[k])) : 0x88888888u;
    }
    scales[i] = __byte_perm(s[0], s[1], 0x5410);
  }
}

// (c - 8) s of eight codes as bf16, rounded once.
__device__ __forceinline__ uint4 widen(uint32_t w, uint32_t scale) {
  const uint32_t s2 = scale | scale << 16;
  uint32_t y[4];  // codes i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = (w >> (4 * i) & 0x000f000fu) | 0x43004300u;  // 128 + c
    const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c), __floats2bfloat162_rn(136.f, 136.f)),
                                     *reinterpret_cast<const __nv_bfloat162*>(&s2));
    y[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410), __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632));
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_append_kernel(const Kv4AppendArgs a) {
  constexpr int G = D / 32;
  const TileAt x = my_tile(a.pages.Hkv, a.N);
  if (!x.ok) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // The tokens that sequence b appends: rows 0 .. n - 1 of k and v, positions len - n .. len - 1.
  const int len = a.pages.seqlens[x.b];
  const int n = a.n_new ? a.n_new[x.b] : a.N;
  if (n < 0 || n > a.N || len < n || len > static_cast<long long>(a.pages.max_pages) << a.pages.page_shift) {
    if (lane == 0) atomicCAS(a.pages.err, 0, kErrDeviceArg);
    return;
  }
  const int first = len - n, pos0 = (first & ~15) + 16 * x.tile;
  if (n == 0 || pos0 >= len) return;
  const long long at = kv4_tile_at<D>(a.pages, x.b, x.h, pos0, kErrDeviceArg);
  if (at < 0) return;
  uint8_t* tile = a.pages.pool + at;
  uint4 in[2][2][G];  // of K and V, tokens g and g + 8, every group
  bool live[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int pos = pos0 + g + 8 * r, i = pos - first;
    live[r] = i >= 0 && pos < len;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(which ? a.v : a.k) +
                                 (which ? x.b * a.v_sb + i * a.v_sn : x.b * a.k_sb + i * a.k_sn) + x.h * D + 8 * t;
#pragma unroll
      for (int grp = 0; grp < G; ++grp) in[which][r][grp] = live[r] ? *reinterpret_cast<const uint4*>(row + 32 * grp) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int tok = g + 8 * r;
    uint32_t w[G], s[G / 2];
    narrow<G>(in[0][r], w, s);
    if (live[r]) {
      store_words<G>(tile + (tok * 4 + t) * (4 * G), w);
      if (t == 0) {
#pragma unroll
        for (int i = 0; i < G / 2; ++i) *reinterpret_cast<uint32_t*>(tile + kv4_off_ks(D) + tok * (2 * G) + 4 * i) = s[i];
      }
    }
    narrow<G>(in[1][r], w, s);
    if (live[r] && t == 1) {
#pragma unroll
      for (int i = 0; i < G / 2; ++i) *reinterpret_cast<uint32_t*>(tile + kv4_off_vs(D) + tok * (2 * G) + 4 * i) = s[i];
    }
    // The lane of an even token takes channels 8 t .. 8 t + 3 of both tokens of the pair, that of the odd one the rest.
    const int odd = g & 1;
    const bool other = __shfl_xor_sync(0xffffffffu, live[r], 4);
#pragma unroll
    for (int grp = 0; grp < G; ++grp) {
      const uint32_t y = __shfl_xor_sync(0xffffffffu, w[grp], 4);
      w[grp] = odd ? __byte_perm(y, w[grp], 0x7632) : __byte_perm(w[grp], y, 0x5410);
    }
    uint8_t* v = tile + kv4_off_v(D) + r * (4 * D) + ((2 * t + odd) * 4 + (g >> 1)) * (4 * G);
    if (live[r] && other) {
      store_words<G>(v, w);
    } else if (live[r] || other) {
      const int hi = odd ? live[r] : other;  // the odd token is the one that is appended
#pragma unroll
      for (int grp = 0; grp < G; ++grp) *reinterpret_cast<uint16_t*>(v + 4 * grp + 2 * hi) = static_cast<uint16_t>(w[grp] >> (16 * hi));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) kv4_read_kernel(const Kv4ReadArgs a) {
  constexpr int G = D / 32;
  const TileAt x = my_tile(a.pages.Hkv, a.N);
  if (!x.ok) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  int len = a.pages.seqlens[x.b], start = a.start ? a.start[x.b] : 0;
  if (len < 0 || len > static_cast<long long>(a.pages.max_pages) << a.pages.page_shift || start < 0) {
    if (lane == 0) atomicCAS(a.pages.err, 0, kErrDeviceArg);
    len = 0;
    start = 0;
  }
  const long long pos0 = (static_cast<long long>(start) & ~15ll) + 16 * x.tile;
  const long long at = pos0 < len ? kv4_tile_at<D>(a.pages, x.b, x.h, static_cast<int>(pos0), kErrDeviceArg) : -1;
  const uint8_t* tile = a.pages.pool + (at < 0 ? 0 : at);
  const int odd = g & 1;
  uint32_t w[2][2][G], s[2][2][G / 2];  // of K and V, tokens g and g + 8
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int tok = g + 8 * r;
    const bool live = at >= 0 && pos0 + tok < len;
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
      s[0][r][i] = live ? *reinterpret_cast<const uint32_t*>(tile + kv4_off_ks(D) + tok * (2 * G) + 4 * i) : 0u;
      s[1][r][i] = live ? *reinterpret_cast<const uint32_t*>(tile + kv4_off_vs(D) + tok * (2 * G) + 4 * i) : 0u;
    }
#pragma unroll
    for (int i = 0; i < G; ++i) w[0][r][i] = w[1][r][i] = 0x88888888u;
    if (at >= 0) {
      load_words<G>(tile + (tok * 4 + t) * (4 * G), w[0][r]);
      load_words<G>(tile + kv4_off_v(D) + r * (4 * D) + ((2 * t + odd) * 4 + (g >> 1)) * (4 * G), w[1][r]);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int grp = 0; grp < G; ++grp) {  // V: back from half the channels of two tokens to all of one
      uint32_t& v = w[1][r][grp];
      const uint32_t y = __shfl_xor_sync(0xffffffffu, v, 4);
      v = odd ? __byte_perm(y, v, 0x7632) : __byte_perm(v, y, 0x5410);
    }
    const long long i = pos0 + g + 8 * r - start;  // row of the output
    if (i < 0 || i >= a.N) continue;
    const long long row = ((static_cast<long long>(x.b) * a.N + i) * a.pages.Hkv + x.h) * D + 8 * t;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(which ? a.v : a.k) + row);
#pragma unroll
      for (int grp = 0; grp < G; ++grp) {
        const uint32_t pair = s[which][r][grp >> 1];
        out[4 * grp] = widen(w[which][r][grp], grp & 1 ? pair >> 16 : pair & 0xffffu);
      }
    }
  }
}

template <typename A>
unsigned row_blocks(const A& a) { return static_cast<unsigned>(a.pages.B) * blocks_of(a.N, a.pages.Hkv); }

}  // namespace

cudaError_t launch_kv4_append(int d, const Kv4AppendArgs& a, cudaStream_t s) {
  if (d == 64) kv4_append_kernel<64><<<row_blocks(a), kRowWarps * 32, 0, s>>>(a);
  else kv4_append_kernel<128><<<row_blocks(a), kRowWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(int d, const Kv4ReadArgs& a, cudaStream_t s) {
  if (d == 64) kv4_read_kernel<64><<<row_blocks(a), kRowWarps * 32, 0, s>>>(a);
  else kv4_read_kernel<128><<<row_blocks(a), kRowWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace eio
