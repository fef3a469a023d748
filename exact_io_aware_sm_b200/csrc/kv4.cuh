// kv4.cuh -- the pages of the 4-bit KV cache: their layout, and the quantiser.
//
// A page holds T tokens (16, 32, 64, 128 or 256) of every KV head: [Hkv][T / 16
// tiles].  A tile is 16 tokens of one head, 18 d bytes, everything that the
// attention over those 16 keys needs in one contiguous run (a multiple of 128
// bytes, so that one bulk copy brings any number of consecutive tiles of a page):
//
//   K codes   [tok][t 0..3][group][4 bytes]                  8 d bytes
//   V codes   [tok / 8][g 0..7][t 0..3][group][tok % 2][2 bytes], t = tok % 8 / 2
//   K scales  [tok][group] bf16                              32 (d / 32) bytes
//   V scales  [tok][group] bf16
//
// A group is 32 channels of one token and head; a code c in 0..15 (4 bits, low
// nibble first) stands for (c - 8) * s with the group's scale s.  K's channel
// 32 group + 8 t + n is nibble n of its four bytes; V's channel 32 group + 4 g
// + i is nibble i of its two.  The orders inside K and V are those of the
// m16n8k16 fragments that the decode kernel builds from them: lane (g, t) of a
// warp finds the codes that its A fragments take (K: token g, every group's
// t-th eight channels; V: tokens 2t, 2t + 1, every group's g-th four channels)
// in 16 (d = 64: 8) consecutive bytes, and the 32 lanes' runs are consecutive.
// Every byte belongs to one token, so that a token is written without reading
// its neighbours.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "kernels_kv4.h"

namespace eio {

constexpr int kKv4Tile = 16;    // tokens
constexpr int kKv4Group = 32;   // channels that share a scale

__host__ __device__ constexpr int kv4_tile_bytes(int d) { return 18 * d; }
__host__ __device__ constexpr int kv4_off_v(int d) { return 8 * d; }
__host__ __device__ constexpr int kv4_off_ks(int d) { return 16 * d; }
__host__ __device__ constexpr int kv4_off_vs(int d) { return 17 * d; }

// The byte offset of the tile that holds token `tok` of sequence b, head h;
// -1 (and the error latched) where the table names no page of the pool.
template <int D>
__device__ __forceinline__ long long kv4_tile_at(const Kv4Pages& p, int b, int h, int tok, int err_code) {
  const int id = p.table[static_cast<size_t>(b) * p.max_pages + (tok >> p.page_shift)];
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.n_pages)) {
    atomicCAS(p.err, 0, err_code);
    return -1;
  }
  const int tiles = 1 << (p.page_shift - 4);
  return ((static_cast<long long>(id) * p.Hkv + h) * tiles + ((tok >> 4) & (tiles - 1))) * kv4_tile_bytes(D);
}

// The scale of a group from the largest magnitude of its bf16 values, given
// as bits (sign cleared; integers order like the magnitudes, infinities and
// NaNs above all): bf16(m / 7); 0 below 2^-100, so that every scale and its
// reciprocal are normal fp32 numbers; NaN where the group holds an infinity
// or a NaN.  m * (1/7) in fp32 rounds to the bf16 of the exact quotient: m
// has 8 significant bits, so m / 7 is a bf16 value or at least 2^-12 of its
// size away from every border between two.
__device__ __forceinline__ bool kv4_has_codes(uint32_t m) { return m - 0x0d80u < 0x7f80u - 0x0d80u; }  // finite, at least 2^-100
__device__ __forceinline__ uint32_t kv4_scale_bits(uint32_t m, bool has_codes) {
  const float s = __uint_as_float(m << 16) * (1.f / 7.f);
  return has_codes ? __bfloat16_as_ushort(__float2bfloat16_rn(s)) : m < 0x7f80u ? 0u : 0x7fffu;
}

// Codes are 8 + floor(x / s + 1/2): x / s has a distance of 0 or at least 2^-9
// from every half-integer (quotients of two 8-bit significands of magnitude at
// most 7: |2 X 2^c - (2 k + 1) S| / 2 S with integers where c >= -1, and below
// that x / s < 1/2 by at least 2^-9).  So x * (1 / s) + 8.5 + M, rounded to a
// multiple of 2^-10 or finer by the size of M, has that integer before the point
// whatever the last bits of the product, ties upwards among them: with M = 1.5 *
// 2^(23 - i) it is bits i .. i + 3 of the sum.  Codes stay in 1..15: |x| is at most m
// and s at least (m / 7) (1 - 2^-8).
__device__ __forceinline__ float kv4_inverse(uint32_t scale_bits) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__uint_as_float(scale_bits << 16)));
  return y;
}

// The codes of eight bf16 values (pairs, low half first), low nibbles first; inv is kv4_inverse of their group's scale.
__device__ __forceinline__ uint32_t kv4_codes(const uint32_t* w, float inv) {
  auto sum = [&](int j, float m) {
    const uint32_t x = j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16;
    return __float_as_uint(fmaf(__uint_as_float(x), inv, m));
  };
  // three codes at a time at bits 10, 14 and 18
  auto three = [&](int j) { return (sum(j, 12296.5f) & 0x3c00u) | (sum(j + 1, 776.5f) & 0x3c000u) | (sum(j + 2, 56.5f) & 0x3c0000u); };
  const uint32_t two = (sum(6, 12296.5f) & 0x3c00u) | (sum(7, 776.5f) & 0x3c000u);
  return three(0) >> 10 | three(3) << 2 | two << 14;
}

}  // namespace eio
