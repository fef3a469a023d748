// decode_kv4.cu -- attention of the Sq newest tokens of each sequence over the
// 4-bit paged cache.
//
//     O = softmax(q K^T scale) V,   K = (ck - 8) sk,  V = (cv - 8) sv
//
// The cache is read once: 18 d / 16 bytes a key and KV head, against 1.3
// instructions a value to widen the codes, so both the memory and the issue
// slots matter.
//
//   decode_kv4_kernel  persistent, one CTA per SM.  A stage is 32 keys (two
//     tiles of the cache) of a unit (sequence, KV head, block of at most 8 NCG
//     columns, a column being a (query head, token) pair of the head's group).
//     The stages of all units in a row are cut into equal runs, one for each
//     warp: no counters, and the work of any two warps differs by one stage
//     whatever the lengths.  Each warp is its own pipeline: a ring of stages
//     filled by bulk copies (a tile is one contiguous run), an online softmax,
//     warp-level MMAs on the codes:
//       S^T (16 keys x 8 columns): per group of 32 channels two MMAs of the
//         codes c themselves: the bits of a nibble, masked out of the word, are
//         the fp16 number c 2^-24 or c 2^-20, so widening costs an AND for two
//         codes.  The -8 is the accumulator's first value (-8 sum q), the group's
//         scale multiplies the group's sum.  q goes in as fp16, scaled by a power
//         of two so that its largest magnitude is in [2^14, 2^15): exact down to
//         2^-28 of that largest.
//       O^T (d x 8 columns): codes as bf16 (128 + c, less 136), times P sv: the
//         scale belongs to the key, so it multiplies P before the rounding to bf16
//         (one rounding for each term, 2^-9, as in attn_decode).
//     A unit that lies in one warp's run is finished there; the others leave
//     their numerator, maximum and sum in the workspace.
//   decode_kv4_combine_kernel  one CTA per query row: joins those.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.h"
#include "kv4.cuh"
#include "pdl.cuh"
#include "ptx_sm100.cuh"
#include "warp_mma.cuh"

namespace eio {
namespace {

constexpr int kStageKeys = 32;
constexpr int kMaxCtas = 148;
constexpr int kRingBudget = 222 * 1024;
constexpr int kCombineThreads = 256;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRebase = 8.f;  // move the exponent base only when the maximum grows by more

template <int D, int NCG>
struct Cfg {
  static constexpr int W = NCG == 1 ? 12 : 8;  // warps
  static constexpr int G = D / 32;
  static constexpr int kTile = kv4_tile_bytes(D);
  static constexpr int kStage = 2 * kTile;
  static constexpr int R = kRingBudget / (W * (kStage + 24)) < 8 ? kRingBudget / (W * (kStage + 24)) : 8;
  static constexpr int kOffMeta = W * R * kStage;
  static constexpr int kOffBars = kOffMeta + W * R * 16;
  static constexpr int kSmem = kOffBars + W * R * 8 + 128;
  static constexpr int kCols = 8 * NCG;
  static constexpr int kSlotFloats = kCols * (D + 2);  // numerators [col][D], then (maximum, sum) [col]
};

// How a call's stages are laid out and cut, the same for both kernels.
struct Split {
  long long total;  // stages
  long long parts;  // runs: part i is stages [i total / parts, (i + 1) total / parts)
  __device__ long long first(long long i) const { return i * total / parts; }
  __device__ long long part_of(long long x) const { return ((x + 1) * parts - 1) / total; }
};

__device__ __forceinline__ int checked_len(const Kv4Pages& p, int b) {
  const int len = p.seqlens[b];
  if (len < 0 || len > static_cast<long long>(p.max_pages) << p.page_shift) {
    atomicCAS(p.err, 0, kErrDeviceArg);
    return 0;
  }
  return len;
}

// D (16x8 f32) = A (16x16 f16, row) * B (16x8 f16, col) + C.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Nibble 4 i of both halves of w as bf16 numbers c - 8.
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t x = (w & 0x000f000fu) | 0x43004300u;  // 128 + c
  __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x), __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<uint32_t*>(&v);
}

template <int G>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t* w) {
  if constexpr (G == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  }
}

// G bf16 scales as fp32.
template <int G>
__device__ __forceinline__ void lds_scales(const uint8_t* p, float* s) {
  uint32_t w[G / 2];
  if constexpr (G == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < G / 2; ++i) {
    s[2 * i] = __uint_as_float(w[i] << 16);
    s[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

struct Columns {
  int blocks, per;  // column blocks of a KV head's group, columns of each (the last may have fewer)
};

template <int D, int NCG>
__global__ void __launch_bounds__(Cfg<D, NCG>::W * 32, 1)
    decode_kv4_kernel(const DecodeKv4Args a, const Columns cols, long long* start, float* slots) {
  using C = Cfg<D, NCG>;
  constexpr int R = C::R, G = C::G;
  extern __shared__ __align__(128) uint8_t smem[];
  const Kv4Pages& pg = a.pages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * R * C::kStage;
  int4* meta = reinterpret_cast<int4*>(smem + C::kOffMeta) + warp * R;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBars) + warp * R;
  const int units = pg.Hkv * cols.blocks;
  const int heads = a.Hq / pg.Hkv, live_cols = heads * a.Sq;

  if (lane == 0) {
    for (int r = 0; r < R; ++r) mbar_init(&bars[r], 1);
    fence_mbar_init();
  }
  pdl_launch_dependents();
  __syncwarp();

  // All stages of the call; the first CTA's first warp leaves where each sequence starts for the second kernel.
  Split sp;
  {
    long long sum = 0;
    for (int b = lane; b < pg.B; b += 32) sum += (checked_len(pg, b) + kStageKeys - 1) / kStageKeys;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    sp.total = sum * units;
    const long long warps = static_cast<long long>(gridDim.x) * C::W;
    sp.parts = sp.total < warps ? sp.total : warps;
  }
  const bool scribe = blockIdx.x == 0 && warp == 0;
  // Parts go round the CTAs, so that few of them still use every SM.
  const long long part = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  const bool idle = part >= sp.parts;
  if (idle && !scribe) return;
  const long long x0 = idle ? 0 : sp.first(part), x1 = idle ? 0 : sp.first(part + 1);

  // The producer's place: stage st (of nst) of unit u of sequence b.
  int b = 0, u = 0, st = 0, nst = 0, len = 0;
  {
    long long base = 0;  // stages of a KV head before this group of 32 sequences
    bool found = idle;
    for (int c = 0; c < pg.B && (scribe || !found); c += 32) {
      const int l = c + lane < pg.B ? checked_len(pg, c + lane) : 0;
      const int n = (l + kStageKeys - 1) / kStageKeys;
      long long pre = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, pre, off);
        if (lane >= off) pre += v;
      }
      pre += base;
      if (scribe && c + lane < pg.B) start[1 + c + lane] = pre;
      const unsigned past = __ballot_sync(0xffffffffu, pre * units > x0);
      if (!found && past) {
        const int src = __ffs(past) - 1;
        b = c + src;
        len = __shfl_sync(0xffffffffu, l, src);
        nst = __shfl_sync(0xffffffffu, n, src);
        const long long before = __shfl_sync(0xffffffffu, pre, src) - nst;
        const long long in = x0 - before * units;
        u = static_cast<int>(in / nst);
        st = static_cast<int>(in % nst);
        found = true;
      }
      base = __shfl_sync(0xffffffffu, pre, 31);
    }
    if (scribe && lane == 0) start[0] = 0;
  }
  if (idle) return;

  int left = static_cast<int>(x1 - x0);  // stages still to be produced
  bool fresh = true;                     // the next one is its run's first of a unit
  int win = 0, ids = 0;                  // lane i holds the page id of page win + i of sequence b
  bool no_win = true;
  const int tiles_shift = pg.page_shift - 4;
  auto page_of = [&](int p) -> int {
    if (no_win || p - win >= 32 || p < win) {
      win = p;
      no_win = false;
      ids = 0;
      if ((static_cast<long long>(p + lane) << pg.page_shift) < len) {
        ids = pg.table[static_cast<size_t>(b) * pg.max_pages + p + lane];
        if (static_cast<unsigned>(ids) >= static_cast<unsigned>(pg.n_pages)) {
          atomicCAS(pg.err, 0, kErrDeviceArg);
          ids = -1;
        }
      }
    }
    return __shfl_sync(0xffffffffu, ids, p - win);
  };
  auto produce = [&](int slot) {
    if (st == nst) {  // the next unit, in the next sequence that has one
      st = 0;
      fresh = true;
      no_win = true;
      if (++u == units) {
        u = 0;
        do {
          ++b;
          len = checked_len(pg, b);
        } while (len == 0 && b + 1 < pg.B);
        nst = (len + kStageKeys - 1) / kStageKeys;
      }
    }
    const int k0 = st * kStageKeys;
    const int ntiles = len - k0 > 16 ? 2 : 1;
    const int p0 = page_of(k0 >> pg.page_shift);
    const int h = u / cols.blocks;
    const uint8_t* src = pg.pool + (((static_cast<long long>(p0) * pg.Hkv + h) << tiles_shift) + ((k0 >> 4) & ((1 << tiles_shift) - 1))) * C::kTile;
    uint8_t* dst = ring + slot * C::kStage;
    int bad = p0 < 0 ? 3 : 0;
    uint32_t bytes = p0 < 0 ? 0 : ntiles * C::kTile;
    const uint8_t* src1 = nullptr;
    if (tiles_shift == 0) {  // pages of one tile: the second tile is elsewhere
      if (bytes) bytes = C::kTile;
      bad &= 1;
      if (ntiles == 2) {
        const int p1 = page_of((k0 >> 4) + 1);
        if (p1 < 0) bad |= 2;
        else src1 = pg.pool + (static_cast<long long>(p1) * pg.Hkv + h) * C::kTile;
      }
    }
    --left;
    const int flags = (fresh ? 1 : 0) | (st + 1 == nst || left == 0 ? 2 : 0) | bad << 2;
    fresh = false;
    if (lane == 0) meta[slot] = make_int4(b, u, k0 | flags, len);
    fence_proxy_async_smem();  // earlier generic accesses to this slot come first
    mbar_arrive_expect_tx_elect(&bars[slot], bytes + (src1 ? C::kTile : 0));
    if (bytes) bulk_load_elect(dst, src, bytes, &bars[slot]);
    if (src1) bulk_load_elect(dst + C::kTile, src1, C::kTile, &bars[slot]);
    ++st;
  };

  uint32_t produced = 0, consumed = 0;
  for (int r = 0; r < R && left > 0; ++r, ++produced) produce(r);
  __syncwarp();

  uint32_t qf[NCG][G][4];       // B fragments of q: two MMAs a group
  float bias[NCG][G][2];        // -8 sum of q over a group, columns 2t and 2t + 1
  float fac[NCG][2];            // a raw score times this is the score in log2 units
  int vis[NCG][2];              // keys that the column sees
  float acc[NCG][G][2][4];      // O^T: channels 32 group + 4 g + 2 j (and + 1), columns 2t, 2t + 1
  float m[NCG][2], l[NCG][2];
  int seg_k0 = 0, which = 0;
  bool ok = true;

  auto begin_unit = [&](int ub, int uu, int ulen) {
    const int h = uu / cols.blocks, c0 = uu % cols.blocks * cols.per;
#pragma unroll
    for (int cg = 0; cg < NCG; ++cg) {
      const int c = cg * 8 + g, col = c0 + c;
      const bool live = c < cols.per && col < live_cols;
      const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.q) +
                                 ((static_cast<size_t>(ub) * a.Sq + (live ? col % a.Sq : 0)) * a.Hq + h * heads + (live ? col / a.Sq : 0)) * D + 8 * t;
      uint4 raw[G];
#pragma unroll
      for (int grp = 0; grp < G; ++grp) raw[grp] = live ? *reinterpret_cast<const uint4*>(row + 32 * grp) : make_uint4(0u, 0u, 0u, 0u);
      uint32_t mx = 0;
#pragma unroll
      for (int grp = 0; grp < G; ++grp) {
        const uint32_t w[4] = {raw[grp].x, raw[grp].y, raw[grp].z, raw[grp].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = max(mx, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = min(max(141 - static_cast<int>(mx >> 7), -100), 100);  // q 2^e
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      float fc = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 24 - e) << 23);
#pragma unroll
      for (int grp = 0; grp < G; ++grp) {
        const uint32_t w[4] = {raw[grp].x, raw[grp].y, raw[grp].z, raw[grp].w};
        float x[8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16) * up;
          x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * up;
        }
        // codes (n, n + 4) of a word sit 16 bits apart; odd n are masked 4 bits higher, 16 times as large
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float f = n & 1 ? 1.f / 16.f : 1.f;
          const __half2 v = __floats2half2_rn(x[n] * f, x[n + 4] * f);
          qf[cg][grp][n] = *reinterpret_cast<const uint32_t*>(&v);
          const float2 back = __half22float2(v);
          sum += (back.x + back.y) * (n & 1 ? 16.f : 1.f);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -8.f * 5.9604644775390625e-08f;  // 2^-24
#pragma unroll
        for (int j = 0; j < 2; ++j) bias[cg][grp][j] = __shfl_sync(0xffffffffu, sum, (2 * t + j) * 4);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[cg][grp][j][i] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        fac[cg][j] = __shfl_sync(0xffffffffu, fc, (2 * t + j) * 4);
        vis[cg][j] = ulen - a.Sq + 1 + (c0 + cg * 8 + 2 * t + j) % a.Sq;
        m[cg][j] = -INFINITY;
        l[cg][j] = 0.f;
      }
    }
  };

  // One stage: keys k0 .. k0 + 31.  EDGE: some key is past a column's last one, or its page is missing.
  auto stage = [&](auto edge_c, const uint8_t* base, int k0, int bad, int ntiles) {
    constexpr bool EDGE = decltype(edge_c)::value;
    float s[2][NCG][4];
    auto masked = [&](int tile, int cg, int i) {
      return (bad >> tile & 1) || k0 + tile * 16 + g + (i >> 1) * 8 >= vis[cg][i & 1];
    };
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      if (EDGE && tile >= ntiles) {
#pragma unroll
        for (int cg = 0; cg < NCG; ++cg)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[tile][cg][i] = -INFINITY;
        continue;
      }
      const uint8_t* p = base + tile * C::kTile;
      uint32_t w[2][G];
      float ks[2][G];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lds_words<G>(p + ((g + 8 * r) * 4 + t) * (4 * G), w[r]);
        lds_scales<G>(p + kv4_off_ks(D) + (g + 8 * r) * (2 * G), ks[r]);
      }
#pragma unroll
      for (int grp = 0; grp < G; ++grp) {
        const uint32_t f0[4] = {w[0][grp] & 0x000f000fu, w[1][grp] & 0x000f000fu, w[0][grp] & 0x00f000f0u, w[1][grp] & 0x00f000f0u};
        const uint32_t v0 = w[0][grp] >> 8, v1 = w[1][grp] >> 8;
        const uint32_t f1[4] = {v0 & 0x000f000fu, v1 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x00f000f0u};
#pragma unroll
        for (int cg = 0; cg < NCG; ++cg) {
          float raw[4];
          mma_f16(raw, f0, qf[cg][grp][0], qf[cg][grp][1], bias[cg][grp][0], bias[cg][grp][1], bias[cg][grp][0], bias[cg][grp][1]);
          mma_f16(raw, f1, qf[cg][grp][2], qf[cg][grp][3], raw[0], raw[1], raw[2], raw[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[tile][cg][i] = grp == 0 ? raw[i] * ks[i >> 1][0] : fmaf(raw[i], ks[i >> 1][grp], s[tile][cg][i]);
        }
      }
      if constexpr (EDGE) {
#pragma unroll
        for (int cg = 0; cg < NCG; ++cg)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (masked(tile, cg, i)) s[tile][cg][i] = -INFINITY;
      }
    }
#pragma unroll
    for (int cg = 0; cg < NCG; ++cg)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = fmaxf(fmaxf(s[0][cg][j], s[0][cg][j + 2]), fmaxf(s[1][cg][j], s[1][cg][j + 2]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        v *= fac[cg][j];
        if (v > m[cg][j] + kRebase) {
          const float alpha = wm_ex2(m[cg][j] - v);
          l[cg][j] *= alpha;
#pragma unroll
          for (int grp = 0; grp < G; ++grp)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              acc[cg][grp][i][j] *= alpha;
              acc[cg][grp][i][j + 2] *= alpha;
            }
          m[cg][j] = v;
        }
      }
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      if (EDGE && tile >= ntiles) continue;
      const uint8_t* p = base + tile * C::kTile;
#pragma unroll
      for (int cg = 0; cg < NCG; ++cg)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mb = m[cg][i & 1];  // -inf in a column that has seen no key yet: its p are 0
          float& x = s[tile][cg][i];
          x = wm_ex2(fmaf(x, fac[cg][i & 1], EDGE && mb == -INFINITY ? 0.f : -mb));
          l[cg][i & 1] += x;
        }
      uint32_t w[2][G];
      float vs[2][G];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lds_words<G>(p + kv4_off_v(D) + ((r * 8 + g) * 4 + t) * (4 * G), w[r]);
        lds_scales<G>(p + kv4_off_vs(D) + (g + 8 * r) * (2 * G), vs[r]);
      }
#pragma unroll
      for (int grp = 0; grp < G; ++grp) {
        uint32_t pb[NCG][2];
#pragma unroll
        for (int cg = 0; cg < NCG; ++cg) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = s[tile][cg][i] * vs[i >> 1][grp];
            if (EDGE && masked(tile, cg, i)) x[i] = 0.f;  // whatever the scale of a masked key holds
          }
          pb[cg][0] = movmatrix_trans(wm_pack_bf16x2(x[0], x[1]));
          pb[cg][1] = movmatrix_trans(wm_pack_bf16x2(x[2], x[3]));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t af[4] = {code_pair(w[0][grp] >> (8 * j)), code_pair(w[0][grp] >> (8 * j + 4)),
                                  code_pair(w[1][grp] >> (8 * j)), code_pair(w[1][grp] >> (8 * j + 4))};
#pragma unroll
          for (int cg = 0; cg < NCG; ++cg) mma_16816(acc[cg][grp][j], af, pb[cg][0], pb[cg][1]);
        }
      }
    }
  };

  auto end_unit = [&](int ub, int uu, bool whole) {
    const int h = uu / cols.blocks, c0 = uu % cols.blocks * cols.per;
    float* slot = slots + (2 * part + which) * C::kSlotFloats;
#pragma unroll
    for (int cg = 0; cg < NCG; ++cg)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[cg][j];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int c = cg * 8 + 2 * t + j, col = c0 + c;
        if (c < cols.per && col < live_cols) {
          if (whole) {
            const int hq = h * heads + col / a.Sq, sq = col % a.Sq;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + ((static_cast<size_t>(ub) * a.Sq + sq) * a.Hq + hq) * D + 4 * g;
#pragma unroll
            for (int grp = 0; grp < G; ++grp) {
              const float* x = acc[cg][grp][0];
              const float* y = acc[cg][grp][1];
              *reinterpret_cast<uint2*>(o + 32 * grp) =
                  make_uint2(wm_pack_bf16x2(x[j] * inv, x[j + 2] * inv), wm_pack_bf16x2(y[j] * inv, y[j + 2] * inv));
            }
            if (g == 0 && a.lse) a.lse[(static_cast<size_t>(ub) * a.Hq + hq) * a.Sq + sq] = sum == 0.f ? -INFINITY : (m[cg][j] + log2f(sum)) * kLn2;
          } else {
            float* o = slot + c * D + 4 * g;
#pragma unroll
            for (int grp = 0; grp < G; ++grp) {
              const float* x = acc[cg][grp][0];
              const float* y = acc[cg][grp][1];
              *reinterpret_cast<float4*>(o + 32 * grp) = make_float4(x[j], x[j + 2], y[j], y[j + 2]);
            }
            if (g == 0) *reinterpret_cast<float2*>(slot + C::kCols * D + 2 * c) = make_float2(m[cg][j], sum);
          }
        }
      }
    which = 1;
  };

  while (consumed < produced) {
    const int slot = static_cast<int>(consumed % R);
    const bool mine = mbar_wait(&bars[slot], (consumed / R) & 1);
    if (!__all_sync(0xffffffffu, mine)) {
      ok = false;
      break;
    }
    const int4 md = meta[slot];
    const int k0 = md.z & ~31, flags = md.z & 31, ulen = md.w;
    if (flags & 1) {
      begin_unit(md.x, md.y, ulen);
      seg_k0 = k0;
    }
    const uint8_t* base = ring + slot * C::kStage;
    const int bad = flags >> 2 & 3;
    if (bad || k0 + kStageKeys > ulen - a.Sq + 1) stage(std::true_type{}, base, k0, bad, ulen - k0 > 16 ? 2 : 1);
    else stage(std::false_type{}, base, k0, 0, 2);
    __syncwarp();
    ++consumed;
    if (left > 0) {
      produce(slot);
      ++produced;
    }
    if (flags & 2) end_unit(md.x, md.y, seg_k0 == 0 && k0 + kStageKeys >= ulen);
  }
  if (!ok) {
    if (lane == 0) atomicCAS(pg.err, 0, kErrDeviceTimeout);
    // every copy that this warp started lands before the CTA retires
    for (uint32_t c = consumed; c < produced; ++c) mbar_wait(&bars[c % R], (c / R) & 1);
  }
}

template <int D, int NCG>
__global__ void __launch_bounds__(kCombineThreads) decode_kv4_combine_kernel(const DecodeKv4Args a, const Columns cols, long long warps,
                                                                            const long long* start, const float* slots) {
  using C = Cfg<D, NCG>;
  constexpr int kLanes = D / 4, kRows = kCombineThreads / kLanes;  // threads of a slot's row, rows at once
  __shared__ float red[kCombineThreads / 32], sums[kRows];
  __shared__ float4 part_o[kRows][kLanes];
  const int row = blockIdx.x;  // [B, Sq, Hq]
  const int hq = row % a.Hq, sq = row / a.Hq % a.Sq, b = row / a.Hq / a.Sq;
  const int heads = a.Hq / a.pages.Hkv, units = a.pages.Hkv * cols.blocks;
  const int col = hq % heads * a.Sq + sq, c = col % cols.per;
  const int u = hq / heads * cols.blocks + col / cols.per;
  const int tid = threadIdx.x;
  pdl_wait();  // the first kernel has finished and its slots are visible
  Split sp;
  sp.total = start[a.pages.B] * units;
  sp.parts = sp.total < warps ? sp.total : warps;
  const long long s0 = start[b];
  const int nst = static_cast<int>(start[b + 1] - s0);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + static_cast<size_t>(row) * D;
  float* lse = a.lse ? a.lse + (static_cast<size_t>(b) * a.Hq + hq) * a.Sq + sq : nullptr;
  if (nst == 0) {
    if (tid < D) o[tid] = __float2bfloat16_rn(0.f);
    if (tid == 0 && lse) *lse = -INFINITY;
    return;
  }
  const long long first = s0 * units + static_cast<long long>(u) * nst;
  const long long i0 = sp.part_of(first);
  const int n = static_cast<int>(sp.part_of(first + nst - 1) - i0) + 1;
  if (n == 1) return;  // one warp had the whole unit and has written it
  // The unit's first part may have begun in an earlier unit; it is then that warp's second slot.
  const int late = sp.first(i0) < first ? 1 : 0;
  auto slot = [&](int i) { return slots + (2 * (i0 + i) + (i == 0 ? late : 0)) * C::kSlotFloats; };
  float M = -INFINITY;
  for (int i = tid; i < n; i += kCombineThreads) M = fmaxf(M, slot(i)[C::kCols * D + 2 * c]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if ((tid & 31) == 0) red[tid >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCombineThreads / 32; ++i) M = fmaxf(M, red[i]);
  if (M == -INFINITY) M = 0.f;  // nothing seen, or NaN: weights 0
  const int r = tid / kLanes, ch = tid % kLanes;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  float W = 0.f;
#pragma unroll 4
  for (int i = r; i < n; i += kRows) {
    const float* s = slot(i);
    const float2 ml = *reinterpret_cast<const float2*>(s + C::kCols * D + 2 * c);
    const float4 x = *reinterpret_cast<const float4*>(s + c * D + 4 * ch);
    const float w = wm_ex2(ml.x - M);
    W = fmaf(w, ml.y, W);
    O.x = fmaf(w, x.x, O.x), O.y = fmaf(w, x.y, O.y), O.z = fmaf(w, x.z, O.z), O.w = fmaf(w, x.w, O.w);
  }
  part_o[r][ch] = O;
  if (ch == 0) sums[r] = W;
  __syncthreads();
  if (tid < D) {
    float num = 0.f;
    W = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      num += reinterpret_cast<const float*>(part_o[i])[tid];
      W += sums[i];
    }
    o[tid] = __float2bfloat16_rn(W == 0.f ? 0.f : num / W);
    if (tid == 0 && lse) *lse = W == 0.f ? -INFINITY : (M + log2f(W)) * kLn2;
  }
}

Columns columns_of(int G, int Sq) {
  const int n = G * Sq, blocks = (n + 15) / 16;
  return {blocks, (n + blocks - 1) / blocks};
}

size_t header_bytes(int B) { return (static_cast<size_t>(B + 1) * sizeof(long long) + 255) / 256 * 256; }

long long most_parts(int B, int units, long long max_tokens, int warps) {
  const double most = static_cast<double>(B) * units * static_cast<double>((max_tokens + kStageKeys - 1) / kStageKeys);
  const long long parts = static_cast<long long>(kMaxCtas) * warps;
  return most < static_cast<double>(parts) ? static_cast<long long>(most) : parts;
}

template <int D, int NCG>
size_t workspace_of(int B, int units, long long max_tokens) {
  using C = Cfg<D, NCG>;
  return header_bytes(B) + 2 * static_cast<size_t>(most_parts(B, units, max_tokens, C::W)) * C::kSlotFloats * sizeof(float);
}

template <int D, int NCG>
cudaError_t launch_dn(const Columns cols, const DecodeKv4Args& a, cudaStream_t s) {
  using C = Cfg<D, NCG>;
  static_assert(C::kSmem <= 227 * 1024 && C::R >= 3, "the rings of all warps fit one SM");
  static DeviceOnce attr_set;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!attr_set.test(dev)) {
    e = cudaFuncSetAttribute(decode_kv4_kernel<D, NCG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set.set(dev);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const Kv4Pages& p = a.pages;
  const int units = p.Hkv * cols.blocks;
  const long long parts = most_parts(p.B, units, static_cast<long long>(p.max_pages) << p.page_shift, C::W);
  int grid = sms < kMaxCtas ? sms : kMaxCtas;
  if (parts < grid) grid = static_cast<int>(parts);
  long long* start = static_cast<long long*>(a.work);
  float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(a.work) + header_bytes(p.B));
  decode_kv4_kernel<D, NCG><<<grid, C::W * 32, C::kSmem, s>>>(a, cols, start, slots);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after_pdl(decode_kv4_combine_kernel<D, NCG>, dim3(static_cast<unsigned>(p.B) * a.Sq * a.Hq), dim3(kCombineThreads), 0, s, a,
                          cols, static_cast<long long>(grid) * C::W, static_cast<const long long*>(start), static_cast<const float*>(slots));
}

}  // namespace

// One group of 8 MMA columns where the (query head, token) pairs of a KV head fit it, two otherwise.
size_t decode_kv4_workspace_bytes(int B, int Sq, int Hq, int Hkv, long long max_tokens, int d) {
  const Columns c = columns_of(Hq / Hkv, Sq);
  const int units = Hkv * c.blocks;
  if (d == 64) return c.per <= 8 ? workspace_of<64, 1>(B, units, max_tokens) : workspace_of<64, 2>(B, units, max_tokens);
  return c.per <= 8 ? workspace_of<128, 1>(B, units, max_tokens) : workspace_of<128, 2>(B, units, max_tokens);
}

cudaError_t launch_decode_kv4(int d, const DecodeKv4Args& a, cudaStream_t s) {
  const Columns c = columns_of(a.Hq / a.pages.Hkv, a.Sq);
  if (d == 64) return c.per <= 8 ? launch_dn<64, 1>(c, a, s) : launch_dn<64, 2>(c, a, s);
  return c.per <= 8 ? launch_dn<128, 1>(c, a, s) : launch_dn<128, 2>(c, a, s);
}

}  // namespace eio
