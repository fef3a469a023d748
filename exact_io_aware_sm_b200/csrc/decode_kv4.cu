// decode_kv4.cu -- attention of the Sq newest tokens of each sequence over the
// 4-bit paged cache.
//
//     O = softmax(q K^T scale) V,   K = (ck - 8) sk,  V = (cv - 8) sv
//
// The cache is read once: 18 d / 8 bits of codes and scales a key and KV head.
// 524287 keys x 8 KV heads (604 MB) take 111 us while the clock holds and 124 when the load
// has brought it down, 5.4 to 4.9 TB/s of the 6.46 that a copy reaches.  At 1.78 GHz that is 202
// thousand cycles, of which HBM's rate accounts for 166 and the start and the joining for about 20.  The
// 264 instructions of 16 keys (45 % of them integer ones, which take two cycles each) need about 340
// cycles of a scheduler, HBM's rate gives it 376 at 1.78 GHz and 342 at 1.62: the lower the clock, the more
// the instructions bind.  64 sequences of 1024 to 8192 keys (333 MB): 72 us.
//
//   decode_kv4_kernel  persistent, one CTA per SM.  A stage is 32 keys (two
//     tiles of the cache) of a unit (sequence, KV head, block of at most 8
//     columns, a column being a (query head, token) pair of the head's group).
//     The units in a row, each counted as its stages and three more for its start and
//     end, are cut into equal runs, one for each CTA, and those into equal runs for
//     its warps: no counters, whatever the lengths.  One warp brings the stages of
//     all the others (lane i those of warp i) into a ring for each by bulk copies: a
//     tile is one contiguous run.  The others never wait for one another: online
//     softmax and warp-level MMAs on the codes.  The bits of a nibble masked out of a
//     word are the fp16 number c 2^-24, or c 2^-20 four bits higher, so that widening
//     two codes costs one AND; fp16's subnormal numbers are exact in the MMA.
//       S^T (16 keys x 8 columns): two MMAs for each group of 32 channels, whose
//         scale multiplies their sum.  The -8 of c - 8 is one more MMA, of the
//         scales with -8 sum q over each group in four bf16 parts (32 bits).  q goes
//         in as fp16, scaled by a power of two so that its largest magnitude is in
//         [2^14, 2^15): exact down to 2^-28 of that.
//       O^T (d x 8 columns): the scale belongs to the key, so P sv is rounded to
//         fp16, as P is relative to a base that is at most 2^8 below the column's running
//         maximum, and as a product relative to a power of two (a reference, of a column and a
//         group): when a reference moves, the largest product becomes 2^6 to 2^7.  2^-11 of each
//         term, down to 2^-30 of the column's largest.  Relative to the largest scale so far,
//         whoever sees it, a key of no weight with a V some 2^24 times larger than the others'
//         took all their digits; this costs 1 to 5 % (64 sequences of 1024 to 8192 keys 70.7 ->
//         71.9 us on the device, 64 query heads 79.4 -> 80.3).
//         The codes go in as c - 8, a subtraction of subnormal numbers for two of
//         them: taking 8 sum P sv off at the end cost a third less, but over the
//         524287 keys the sums of c lost the digits that the difference is made of
//         (O off by 0.0041 of its norm instead of 0.0016).
//     The base and the references of a column move only when its weights or products have
//     outgrown them (a test of sums, and of sums of the fp16 products), so that a stage needs
//     no maximum and no shuffles (93 -> 82 us for 64 sequences of 1024 to 8192 keys when that
//     came in, with what it made possible).
//     Up to 4 columns (grouped heads, one token) fill half an MMA; the other half
//     then holds the odd groups of channels (F = 2): scaling, P sv and the sums cost
//     half (157 -> 138 us for the 524287 keys).
//     A unit that lies in one warp's run is finished there, one in a CTA's run by
//     the CTA once its warps are done; the others leave numerators, maxima and sums.
//   decode_kv4_combine_kernel  one CTA for each boundary between two runs: joins the
//     unit that lies across it, in the order of its parts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels_kv4.h"
#include "kv4.cuh"
#include "pdl.cuh"
#include "ptx_sm100.cuh"
#include "warp_mma.cuh"

namespace eio {
namespace {

constexpr int kMaxCtas = 148;
constexpr int kUnitCost = 3;  // of a unit's start and end, in stages (measured: 1 to 4)
constexpr int kRingBudget = 222 * 1024;
constexpr int kMostIdle = 1 << 24;  // rounds (of 100 ns or so) in which no stage was taken
constexpr int kCombineThreads = 512;
constexpr float kSpare = 12.f;  // a join's weights are 2^-12 at most, so that numerators up to fp32's largest add up within it
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kMostWeight = 256.f;  // of a lane's four keys of a column, relative to the base: more moves the base
constexpr float kMostProduct = 32768.f;  // P sv in fp16, summed over the lane's: more moves the references
constexpr int kMostUp = 120;             // log2 of what small products are raised by (scales end at 2^-103)

template <int D, int F>
struct Cfg {
  static constexpr int W = F == 2 || D == 64 ? 15 : 11;  // warps that compute (128 or 168 registers); one more brings the stages
  static constexpr int kKeys = 32;                      // of a stage: two tiles
  static constexpr int kThreads = (W + 1) * 32;
  static constexpr int G = D / 32;
  static constexpr int N = G / F;  // groups, or pairs of groups (F = 2), that share a set of MMA columns
  static constexpr int kTile = kv4_tile_bytes(D);
  static constexpr int kStage = 2 * kTile;
  static constexpr int kFit = kRingBudget / (W * (kStage + 32));
  static constexpr int R = kFit < 8 ? kFit : 8;  // stages of a warp's ring
  static constexpr int kOffMeta = W * R * kStage;
  static constexpr int kOffBars = kOffMeta + W * R * 16;
  static constexpr int kOffSegs = kOffBars + 2 * W * R * 8;  // full and free barriers
  static constexpr int kSmem = kOffSegs + 2 * W * 16 + 16;
  static constexpr int kCols = 8 / F;
  static constexpr int kSlotFloats = kCols * (D + 2);  // numerators [col][D], then (maximum, sum) [col]
  static constexpr int kSlots = W + 2;                 // of a CTA: one a warp, two for what leaves the CTA
};

// What a unit of len keys is counted for when the runs are cut: its stages and kUnitCost for its start and end (the
// queries' fragments, the results); nothing where there are no keys.
template <int KEYS>
__device__ __forceinline__ int cost_of(int len) {
  return len > 0 ? (len + KEYS - 1) / KEYS + kUnitCost : 0;
}

// Where the run of a CTA starts: at cost x of all, stage st (of nst) of unit u of sequence b.
struct Run {
  long long x;
  int b, u, st, nst;
  long long pad;
};

// A segment (the part of a unit in a warp's run) that is not a whole unit.
struct Segment {
  int b, u;  // b < 0: none
  int ends;  // bit 0: with the unit's first stage, bit 1: with its last
  int near;  // its results are in the warp's ring, else in its slot
};

__device__ __forceinline__ int checked_len(const Kv4Pages& p, int b) {
  const int len = p.seqlens[b];
  if (len < 0 || len > static_cast<long long>(p.max_pages) << p.page_shift) {
    atomicCAS(p.err, 0, kErrDeviceArg);
    return 0;
  }
  return len;
}

// D (16x8 f32) += A (16x16, row) * B (16x8, col), f16 and bf16; free to be scheduled.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_first(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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

// Contiguous global -> shared copy of `bytes`, completing on `bar`, issued by this thread.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Whether the phase of the given parity has completed; does not wait.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// G bf16 scales, packed.
template <int G>
__device__ __forceinline__ void lds_scales(const uint8_t* p, uint32_t* w) {
  if constexpr (G == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// An 8 x 8 tile of 16-bit values transposed (free to be scheduled, unlike movmatrix_trans).
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Bytes 1 and 3 of a word as 16-bit numbers.
__device__ __forceinline__ uint32_t high_bytes(uint32_t w) { return __byte_perm(w, 0u, 0x4341); }

// Differences of two fp16 pairs (of subnormal numbers: exact).
__device__ __forceinline__ uint32_t less_f16x2(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}

// Products of two bf16 pairs.
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) {
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two fp32 products in one instruction.
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

struct Columns {
  int blocks, per;  // column blocks of a KV head's group, columns of each (the last may have fewer)
};

// The warp that brings the stages: lane i those of warp i's run, into that warp's ring.
template <int D, int F>
__device__ __forceinline__ void bring_stages(const DecodeKv4Args& a, const Columns& cols, Run* runs, uint8_t* ring, int4* meta, uint64_t* full,
                                             uint64_t* free_, int2* first_unit) {
  using C = Cfg<D, F>;
  constexpr int R = C::R, W = C::W;
  const Kv4Pages& pg = a.pages;
  const int lane = threadIdx.x & 31;
  const int units = pg.Hkv * cols.blocks;
  const int tiles_shift = pg.page_shift - 4;
  const long long page_bytes = (static_cast<long long>(pg.Hkv) << tiles_shift) * C::kTile;

  // All units' costs, cut for the CTAs and then for the warps of each.
  const int len0 = lane < pg.B ? checked_len(pg, lane) : 0;  // of the first 32 sequences
  long long total = cost_of<C::kKeys>(len0);
  for (int b = lane + 32; b < pg.B; b += 32) total += cost_of<C::kKeys>(checked_len(pg, b));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  total *= units;
  const unsigned ctas = gridDim.x, cta = blockIdx.x;
  const long long each = total >> 32 ? total / ctas : static_cast<unsigned>(total) / ctas;
  const unsigned more = static_cast<unsigned>(total - each * ctas);
  const long long cta_x = each * cta + min(cta, more);
  const long long n_cta = each + (cta < more);
  const long long each_w = n_cta >> 32 ? n_cta / W : static_cast<unsigned>(n_cta) / W;
  const unsigned more_w = static_cast<unsigned>(n_cta - each_w * W);
  const long long x0 = cta_x + each_w * lane + min(static_cast<unsigned>(lane), more_w);
  int left = lane < W ? static_cast<int>(each_w + (lane < more_w)) : 0;  // stages still to be brought

  // The place: stage st (of nst) of column block cb of KV head h of sequence b.
  int b = 0, h = 0, cb = 0, st = 0, nst = 0, len = 0;
  bool placed = left == 0;
  long long base = 0;  // costs of a KV head's units before this group of 32 sequences
  for (int c = 0; c < pg.B && !__all_sync(0xffffffffu, placed); c += 32) {
    const int l = c == 0 ? len0 : c + lane < pg.B ? checked_len(pg, c + lane) : 0;
    long long pre = cost_of<C::kKeys>(l);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, pre, off);
      if (lane >= off) pre += v;
    }
    pre += base;
    int lo = 0;  // sequences of the group that end at or before x0
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
      const long long v = __shfl_sync(0xffffffffu, pre, lo + step - 1);
      if (v * units <= x0) lo += step;
    }
    base = __shfl_sync(0xffffffffu, pre, 31);
    const int ll = __shfl_sync(0xffffffffu, l, lo);
    const long long end = __shfl_sync(0xffffffffu, pre, lo);
    if (!placed && end * units > x0) {
      placed = true;
      b = c + lo;
      len = ll;
      const int cost = cost_of<C::kKeys>(ll);
      const long long in = x0 - (end - cost) * units;
      const int u = static_cast<int>(in >> 32 ? in / cost : static_cast<unsigned>(in) / static_cast<unsigned>(cost));
      nst = cost - kUnitCost;
      st = static_cast<int>(in - static_cast<long long>(u) * cost) - kUnitCost;
      if (st < 0) {  // the unit's start, which is no stage
        left = max(left + st, 0);
        st = 0;
      }
      h = u / cols.blocks;
      cb = u - h * cols.blocks;
    }
  }
  if (lane == 0) {
    runs[cta] = Run{cta_x, b, h * cols.blocks + cb, st, nst, 0};
    if (cta + 1 == ctas) runs[ctas].x = total;
    *first_unit = make_int2(b, h * cols.blocks + cb);
  }
  if (lane < W && left == 0) {  // an empty run
    meta[0] = make_int4(-1, 0, 0, 0);
    mbar_arrive(&full[0]);
  }

  // The page id of page p of sequence b; -1 where there is no such page of the pool, 0 (of no use) past the sequence's end.
  auto page_id = [&](int p) -> int {
    if (static_cast<long long>(p) << pg.page_shift >= len) return 0;
    const int id = pg.table[static_cast<size_t>(b) * pg.max_pages + p];
    return static_cast<unsigned>(id) < static_cast<unsigned>(pg.n_pages) ? id : -1;
  };
  // Where the next stage is: id its page, src its tiles there, in_page the stages that the page still has; pages of
  // one tile have half a stage each, id and id_next.  Ids are read a page (a stage) ahead.
  int id = 0, id_next = 0, id_first = 0, in_page = 0;
  const uint8_t* src = nullptr;
  const long long head_bytes = static_cast<long long>(C::kTile) << tiles_shift;
  auto enter_page = [&](int tile) {
    src = pg.pool + max(id, 0) * page_bytes + h * head_bytes + tile * C::kTile;
    in_page = ((1 << tiles_shift) - tile) >> 1;
  };
  auto look = [&]() {
    const int p = (st * C::kKeys) >> pg.page_shift;
    id = page_id(p);
    id_next = page_id(p + 1);
  };
  if (left > 0) {
    look();
    id_first = st == 0 ? id : page_id(0);
    enter_page((st * 2) & ((1 << tiles_shift) - 1));
  }
  const bool small_pages = tiles_shift == 0;
  int unit = h * cols.blocks + cb;
  int fresh = 1;  // the next stage is its run's first of a unit
  int issued = 0, slot = 0, idle = 0;
  uint32_t phase = 1;  // parity of the slot's last release; the first round finds every slot free
  while (__any_sync(0xffffffffu, left > 0)) {
    const bool go = left > 0 && mbar_test(&free_[slot], phase);
    if (go) {
      const int k0 = st * C::kKeys, this_unit = unit, this_b = b, this_len = len;
      const bool two = len - k0 > 16;
      uint8_t* dst = ring + slot * C::kStage;
      uint64_t* bar = &full[slot];
      int bad = id < 0 ? 3 : 0;
      if (small_pages) bad = (id < 0 ? 1 : 0) | (two && id_next < 0 ? 2 : 0);
      --left;
      ++st;
      if (st == nst) left = max(left - kUnitCost, 0);  // the next unit's start
      const int flags = fresh | (st == nst || left == 0 ? 2 : 0) | bad << 2;
      fresh = 0;
      meta[slot] = make_int4(this_b, this_unit, k0 | flags, left == 0 ? this_len | static_cast<int>(0x80000000u) : this_len);
      if (!small_pages) {
        const uint32_t bytes = bad ? 0u : two ? C::kStage : C::kTile;
        mbar_arrive_expect_tx(bar, bytes);
        if (bytes) bulk_load(dst, src, bytes, bar);
      } else {
        const bool one = id >= 0, other = two && id_next >= 0;
        mbar_arrive_expect_tx(bar, (one + other) * C::kTile);
        if (one) bulk_load(dst, src, C::kTile, bar);
        if (other) bulk_load(dst + C::kTile, pg.pool + id_next * page_bytes + h * head_bytes, C::kTile, bar);
      }
      if (bad) atomicCAS(pg.err, 0, kErrDeviceArg);
      src += C::kStage;
      ++issued;
      if (++slot == R) {
        slot = 0;
        phase ^= 1;
      }
      if (left > 0) {
        if (st == nst) {  // the next unit, in the next sequence that has one
          st = 0;
          fresh = 1;
          ++unit;
          if (++cb == cols.blocks) {
            cb = 0;
            if (++h == pg.Hkv) {
              h = unit = 0;
              do {
                ++b;
                len = b < pg.B ? checked_len(pg, b) : 1;  // past the end only where lengths changed under the call
              } while (len == 0);
              b = min(b, pg.B - 1);
              nst = (len + C::kKeys - 1) / C::kKeys;
              id_first = page_id(0);
            }
          }
          id = id_first;
          id_next = page_id(1);
          enter_page(0);
        } else if (small_pages) {
          look();
          enter_page(0);
        } else if (--in_page == 0) {
          id = id_next;
          id_next = page_id(((st * C::kKeys) >> pg.page_shift) + 1);
          enter_page(0);
        }
      }
    }
    if (__any_sync(0xffffffffu, go)) {
      idle = 0;
    } else {
      if (++idle > kMostIdle) {
        if (lane == 0) atomicCAS(pg.err, 0, kErrDeviceTimeout);
        break;
      }
      __nanosleep(20);
    }
  }
  // Every copy lands before the CTA retires.
  for (int i = max(issued - R, 0); i < issued; ++i) mbar_wait(&full[i % R], (i / R) & 1);
  __syncwarp();
}

template <int D, int F>
__global__ void __launch_bounds__(Cfg<D, F>::kThreads, 1)
    decode_kv4_kernel(const DecodeKv4Args a, const Columns cols, Run* runs, float* slots) {
  using C = Cfg<D, F>;
  constexpr int R = C::R, G = C::G, W = C::W;
  extern __shared__ __align__(128) uint8_t smem[];
  const Kv4Pages& pg = a.pages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  Segment* segs = reinterpret_cast<Segment*>(smem + C::kOffSegs);
  int2* first_unit = reinterpret_cast<int2*>(segs + 2 * W);  // the unit that the CTA's run starts in
  const int heads = a.Hq / pg.Hkv, live_cols = heads * a.Sq;
  float* const my_slots = slots + static_cast<size_t>(blockIdx.x) * C::kSlots * C::kSlotFloats;
  // Warp w's ring: stages, what they are (sequence, unit, first key | flags, length | last of the run), barriers.
  const int stream = warp < W ? warp : min(lane, W - 1);
  uint8_t* ring = smem + stream * R * C::kStage;
  int4* meta = reinterpret_cast<int4*>(smem + C::kOffMeta) + stream * R;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBars) + stream * R;
  uint64_t* free_ = full + W * R;

  if (warp == W && lane < W) {
    for (int r = 0; r < R; ++r) mbar_init(&full[r], 1), mbar_init(&free_[r], 1);
    fence_mbar_init();
    segs[2 * lane].b = segs[2 * lane + 1].b = -1;
  }
  pdl_launch_dependents();
  __syncthreads();

  if (warp == W) {
    bring_stages<D, F>(a, cols, runs, ring, meta, full, free_, first_unit);
  } else {
    if (warp == W - 1) {  // sequences without a token are shared out among the CTAs
      const int ctas = gridDim.x;
      for (int b0 = blockIdx.x; b0 < pg.B; b0 += 32 * ctas) {
        const int bl = b0 + lane * ctas;
        unsigned none = __ballot_sync(0xffffffffu, bl < pg.B && checked_len(pg, bl) == 0);
        for (; none; none &= none - 1) {
          const size_t be = b0 + (__ffs(none) - 1) * ctas;
          uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + be * a.Sq * a.Hq * D);
          for (long long i = lane; i < static_cast<long long>(a.Sq) * a.Hq * (D / 8); i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
          if (a.lse)
            for (int i = lane; i < a.Sq * a.Hq; i += 32) a.lse[be * a.Sq * a.Hq + i] = -INFINITY;
        }
      }
    }

  // Columns.  An MMA has 8; with F = 2 the upper four repeat the lower four for the odd groups (of a pair
  // of groups), so that one accumulator holds both groups' sums and a lane scales only its own group's.  This lane:
  // column g as a row of q (and of the B operands), columns 2 t and 2 t + 1 of the accumulators.
  constexpr int NS = C::N;
  const int half_q = F == 2 ? g >> 2 : 0, half = F == 2 ? t >> 1 : 0;
  const uint32_t pick = half ? 0x3244u : 0x1044u;  // F = 2: this lane's scale of a packed pair, as fp32
  uint32_t qf[G][4];         // B fragments of q: two MMAs a group
  uint32_t less[2];          // B fragment of -8 sum of q over each group, in four bf16 parts
  float fac[2];              // a raw score times this is the score in log2 units
  int vis[2];                // keys that the column sees
  float acc[G][2][4];        // O^T: channels 32 group + 4 g + 2 j (and 16 times the next one), columns 2 t, 2 t + 1
  float l[2];                // sum
  float mneg[2];             // less the base (the maximum in log2 units when it last moved); inf: no key was seen yet
  float rinv[NS][2];         // P sv of the lane's group goes in times this, a power of two for each column
  int seg_k0 = 0, which = 0;

  // The token and the query head (of the KV head's group) of a column; false where there is none.
  auto column = [&](int pc, int c0, int* hd, int* tk) {
    const int c = pc & (C::kCols - 1), col = c0 + c;
    *hd = a.Sq == 1 ? col : col / a.Sq;
    *tk = col - *hd * a.Sq;
    return c < cols.per && col < live_cols;
  };
  auto begin_unit = [&](int ub, int uu, int ulen) {
    const int uh = cols.blocks == 1 ? uu : uu / cols.blocks, c0 = (uu - uh * cols.blocks) * cols.per;
    const size_t row0 = static_cast<size_t>(ub) * a.Sq * a.Hq + uh * heads;
    uint4 raw[G];
    int hd, tk;
    const bool live = column(g, c0, &hd, &tk);
    const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.q) + (row0 + (live ? tk * a.Hq + hd : 0)) * D + 8 * t;
#pragma unroll
    for (int grp = 0; grp < G; ++grp) raw[grp] = live ? *reinterpret_cast<const uint4*>(row + 32 * grp) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t mx = 0;
#pragma unroll
    for (int grp = 0; grp < G; ++grp) {
      const uint4 w = raw[grp];
      mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
    }
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = min(max(141 - static_cast<int>(mx >> 7), -100), 100);  // q 2^e
    // A row that is not finite, or would not be as fp16, gives NaN by its sum; its scores would be NaN at every stage.
    const uint32_t none = mx >> 7 > 242 ? 0x7fffffffu : 0u;
    if (none) {
#pragma unroll
      for (int grp = 0; grp < G; ++grp) raw[grp] = make_uint4(0u, 0u, 0u, 0u);
    }
    // Positive and finite, so that masked scores (-inf) and scores of 0 stay what they are whatever the scale.
    const float fc = fminf(fmaxf(a.scale_log2 * pow2(24 - e), pow2(-126)), 3.0e38f);
    // Codes n and n + 4 of a word sit 16 bits apart; odd n are masked 4 bits higher, 16 times as large.
    const uint32_t up = static_cast<uint32_t>(127 + e) << 7 | static_cast<uint32_t>(123 + e) << 23;  // bf16 2^e, 2^(e - 4)
    float x0 = 0.f, x1 = 0.f;
#pragma unroll
    for (int grp = 0; grp < G; ++grp) {
      const uint32_t y[4] = {times(raw[grp].x, up), times(raw[grp].y, up), times(raw[grp].z, up), times(raw[grp].w, up)};
      const bool mine = F == 1 || half_q == (grp & 1);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t v = __byte_perm(y[n >> 1], y[2 + (n >> 1)], n & 1 ? 0x7632 : 0x5410);
        qf[grp][n] = mine ? pack_f16x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)) : 0u;
      }
      // 8 sum q of the columns, by an MMA; -8 sum q of this lane's column g in the two groups of its k
      const uint32_t eights[4] = {0x00080008u, 0x00080008u, 0x00800080u, 0x00800080u};
      float d[4];
      mma_f16_first(d, eights, qf[grp][0], qf[grp][1]);
      mma_f16(d, eights, qf[grp][2], qf[grp][3]);
      const int pc = F == 2 ? (g & 3) + 4 * (grp & 1) : g;
      const float d0 = __shfl_sync(0xffffffffu, d[0], pc >> 1), d1 = __shfl_sync(0xffffffffu, d[1], pc >> 1);
      const float sum = pc & 1 ? -d1 : -d0;
      if (G == 2 || (grp >> 1) == (t & 1)) {
        if (grp & 1) x1 = sum;
        else x0 = sum;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[grp][0][i] = acc[grp][1][i] = 0.f;
    }
    // Row k of this operand is part k / G of group k % G (d = 128: parts 0 and 1 in b0, 2 and 3 in b1;
    // d = 64: 0 to 3 in b0), so that a row of K's scales, repeated, is the other operand.
    uint32_t parts[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      parts[i] = half_q ? 0u : wm_pack_bf16x2(x0, x1);
      x0 -= __uint_as_float(parts[i] << 16);
      x1 -= __uint_as_float(parts[i] & 0xffff0000u);
    }
    if constexpr (G == 4) {
      less[0] = t < 2 ? parts[0] : parts[1];
      less[1] = t < 2 ? parts[2] : parts[3];
    } else {
      less[0] = t == 0 ? parts[0] : t == 1 ? parts[1] : t == 2 ? parts[2] : parts[3];
      less[1] = 0;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      fac[j] = __shfl_sync(0xffffffffu, fc, (2 * t + j) * 4);
      int hd, tk;
      column(2 * t + j, c0, &hd, &tk);
      vis[j] = ulen - a.Sq + 1 + tk;
      mneg[j] = INFINITY;
      const uint32_t sum = __shfl_sync(0xffffffffu, none, (2 * t + j) * 4);
      l[j] = vis[j] > 0 ? __uint_as_float(sum) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) rinv[i][0] = rinv[i][1] = pow2(kMostUp);
  };

  // This lane's scale of set n (its group, or the lane's one of its pair) among packed scales.
  auto scale_at = [&](const uint32_t* w, int n) -> float {
    if constexpr (F == 2) return __uint_as_float(__byte_perm(w[n], 0u, pick));
    else return __uint_as_float(n & 1 ? w[n >> 1] & 0xffff0000u : w[n >> 1] << 16);
  };

  // Two tiles of a stage: keys k0 .. k0 + 31; bit i of bad: the page of tile i is missing.
  auto two_tiles = [&](const uint8_t* base, int k0, int bad, int ulen) {
    float s[2][4];
    uint32_t vs[2][2][G / 2];
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const uint8_t* p = base + tile * C::kTile;
      uint32_t w[2][G], ks[2][G / 2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lds_words<G>(p + ((g + 8 * r) * 4 + t) * (4 * G), w[r]);
        lds_scales<G>(p + kv4_off_ks(D) + (g + 8 * r) * (2 * G), ks[r]);
        lds_scales<G>(p + kv4_off_vs(D) + (g + 8 * r) * (2 * G), vs[tile][r]);
      }
      const uint32_t lo = *reinterpret_cast<const uint32_t*>(p + kv4_off_ks(D) + g * (2 * G) + (t % (G / 2)) * 4);
      const uint32_t hi = *reinterpret_cast<const uint32_t*>(p + kv4_off_ks(D) + (g + 8) * (2 * G) + (t % (G / 2)) * 4);
      const uint32_t sc[4] = {lo, hi, lo, hi};
      mma_bf16_first(s[tile], sc, less[0], less[1]);
      float raw[4];
#pragma unroll
      for (int grp = 0; grp < G; ++grp) {
        const uint32_t f0[4] = {w[0][grp] & 0x000f000fu, w[1][grp] & 0x000f000fu, w[0][grp] & 0x00f000f0u, w[1][grp] & 0x00f000f0u};
        const uint32_t v0 = high_bytes(w[0][grp]), v1 = high_bytes(w[1][grp]), l0 = v0 & 0x000f000fu, l1 = v1 & 0x000f000fu;
        const uint32_t f1[4] = {l0, l1, less_f16x2(v0, l0), less_f16x2(v1, l1)};
        const float k_lo = scale_at(ks[0], grp / F), k_hi = scale_at(ks[1], grp / F);
        if (grp % F == 0) mma_f16_first(raw, f0, qf[grp][0], qf[grp][1]);
        else mma_f16(raw, f0, qf[grp][0], qf[grp][1]);
        mma_f16(raw, f1, qf[grp][2], qf[grp][3]);
        if (grp % F == F - 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s[tile][i] = fmaf(raw[i], i < 2 ? k_lo : k_hi, s[tile][i]);
        }
      }
      if constexpr (F == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[tile][i] += __shfl_xor_sync(0xffffffffu, s[tile][i], 2);
      }
    }
    if (bad || k0 + 32 > ulen - a.Sq + 1) {  // some key is past a column's last one, or its page is missing
#pragma unroll
      for (int tile = 0; tile < 2; ++tile)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int key = k0 + tile * 16 + 8 * r + g;
          const bool gone = (bad >> tile & 1) || key >= ulen;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (gone || key >= vis[j]) s[tile][2 * r + j] = -INFINITY;
          if (gone) {
#pragma unroll
            for (int i = 0; i < G / 2; ++i) vs[tile][r][i] = 0;
          }
        }
    }
    // P relative to the base, and P sv in fp16.  A column's base and references move seldom, where its own weights or
    // products have grown too large for them (or are NaN: no base yet, a scale that is not finite): only then are its
    // maximum and its largest products looked for.
    float p[2][4], some[2];
    uint32_t pv[NS][2][2];  // [][tile][r]: the B fragments before they are transposed
    bool moves[2];
    auto weights = [&](float n0, float n1) {
#pragma unroll
      for (int tile = 0; tile < 2; ++tile)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[tile][i] = wm_ex2(fmaf(s[tile][i], fac[i & 1], i & 1 ? n1 : n0));
#pragma unroll
      for (int j = 0; j < 2; ++j) some[j] = (p[0][j] + p[0][j + 2]) + (p[1][j] + p[1][j + 2]);
    };
    auto products = [&]() {
      __half2 sums[2][2];  // short chains: the vote waits for them
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int tile = 0; tile < 2; ++tile)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float v = scale_at(vs[tile][r], n);
            const float2 w = mul2(make_float2(p[tile][2 * r], p[tile][2 * r + 1]), make_float2(rinv[n][0], rinv[n][1]));
            const float2 y = mul2(w, make_float2(v, v));  // the scale last: a weight of 0 stays 0 whatever the scale
            pv[n][tile][r] = pack_f16x2(y.x, y.y);
            const __half2 x = *reinterpret_cast<const __half2*>(&pv[n][tile][r]);
            sums[tile][r] = n == 0 ? x : __hadd2(sums[tile][r], x);
          }
      const __half2 sum = __habs2(__hadd2(__hadd2(sums[0][0], sums[0][1]), __hadd2(sums[1][0], sums[1][1])));
      moves[0] = !(__low2float(sum) < kMostProduct) || some[0] > kMostWeight;
      moves[1] = !(__high2float(sum) < kMostProduct) || some[1] > kMostWeight;
    };
    weights(mneg[0], mneg[1]);
    products();
    if (__any_sync(0xffffffffu, moves[0] || moves[1])) {
      bool mine[2];  // this lane's columns are among those that move: what one column needs changes no other
#pragma unroll
      for (int j = 0; j < 2; ++j) mine[j] = __ballot_sync(0xffffffffu, moves[j]) & (F == 2 ? 0x55555555u << (t & 1) : 0x11111111u << t);
      // V scales that are not finite leave the products (0 NaN = NaN would reach other groups' sums, and columns
      // that do not see the key) and go straight to the groups of the columns that see them.
      uint32_t odd = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int i = 0; i < G / 2; ++i) {
          uint32_t& v = vs[x >> 1][x & 1][i];
          if ((v & 0x7f80u) == 0x7f80u) odd |= 1u << (x * 8 + 2 * i), v &= 0xffff0000u;
          if ((v & 0x7f800000u) == 0x7f800000u) odd |= 2u << (x * 8 + 2 * i), v &= 0xffffu;
        }
      if (__any_sync(0xffffffffu, odd != 0)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t sees = 0;
          for (int x = 0; x < 4; ++x)
            if (k0 + x * 8 + g < vis[j]) sees |= odd >> (x * 8);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) sees |= __shfl_xor_sync(0xffffffffu, sees, off);
#pragma unroll
          for (int grp = 0; grp < G; ++grp)
            if (sees >> grp & 1) {
#pragma unroll
              for (int i = 0; i < 2; ++i) acc[grp][i][j] = acc[grp][i][j + 2] = __uint_as_float(0x7fffffffu);
            }
        }
      }
      float alpha[2];  // what a new base leaves of the column's sums
      int up[2];       // the octaves of it; differences of whole numbers, so that many moves lose one at most
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = fmaxf(fmaxf(s[0][j], s[0][j + 2]), fmaxf(s[1][j], s[1][j + 2]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        v *= fac[j];
        alpha[j] = 1.f;
        up[j] = 0;
        if (mine[j] && v > -mneg[j]) {
          if (mneg[j] != INFINITY) {
            alpha[j] = wm_ex2(-mneg[j] - v);
            up[j] = static_cast<int>(fminf(floorf(v) - floorf(-mneg[j]), 126.f));
            l[j] *= alpha[j];
          }
          mneg[j] = -v;
        }
      }
      // a column that still sees no key has weights 0
      weights(mneg[0] == INFINITY ? 0.f : mneg[0], mneg[1] == INFINITY ? 0.f : mneg[1]);
      // The largest product of the stage becomes 2^6 to 2^7, or less where an earlier one is larger.
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = 0.f;
#pragma unroll
          for (int tile = 0; tile < 2; ++tile)
#pragma unroll
            for (int r = 0; r < 2; ++r) x = fmaxf(x, fabsf(p[tile][2 * r + j] * scale_at(vs[tile][r], n)));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
          if (mine[j]) {
            const int old = static_cast<int>(__float_as_uint(rinv[n][j]) >> 23) - 127;
            const int now = min(min(old + up[j], 6 + 127 - static_cast<int>(__float_as_uint(x) >> 23)), kMostUp);
            const float f = alpha[j] * pow2(max(now - old, -126));
            rinv[n][j] = pow2(now);
#pragma unroll
            for (int grp = n * F; grp < n * F + F; ++grp)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                acc[grp][i][j] *= f;
                acc[grp][i][j + 2] *= f;
              }
          }
        }
      products();
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) l[j] += some[j];
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const uint8_t* at = base + tile * C::kTile;
      uint32_t w[2][G];
#pragma unroll
      for (int r = 0; r < 2; ++r) lds_words<G>(at + kv4_off_v(D) + ((r * 8 + g) * 4 + t) * (4 * G), w[r]);
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const uint32_t b0 = transposed(pv[n][tile][0]), b1 = transposed(pv[n][tile][1]);
#pragma unroll
        for (int grp = n * F; grp < n * F + F; ++grp) {
          // c - 8 in rows g and 16 (c - 8) in rows g + 8, from c, 16 c, and c + 16 c' with 128 + c: all exact
          const uint32_t v0 = high_bytes(w[0][grp]), v1 = high_bytes(w[1][grp]);
          const uint32_t x0 = (v0 & 0x000f000fu) | 0x00800080u, x1 = (v1 & 0x000f000fu) | 0x00800080u;
          const uint32_t f0[4] = {less_f16x2(w[0][grp] & 0x000f000fu, 0x00080008u), less_f16x2(w[0][grp] & 0x00f000f0u, 0x00800080u),
                                  less_f16x2(w[1][grp] & 0x000f000fu, 0x00080008u), less_f16x2(w[1][grp] & 0x00f000f0u, 0x00800080u)};
          const uint32_t f1[4] = {less_f16x2(x0, 0x00880088u), less_f16x2(v0, x0), less_f16x2(x1, 0x00880088u), less_f16x2(v1, x1)};
          mma_f16(acc[grp][0], f0, b0, b1);
          mma_f16(acc[grp][1], f1, b0, b1);
        }
      }
    }
  };

  // The run's last segment goes to the ring, which is free by then.
  auto end_unit = [&](int ub, int uu, bool starts, bool ends, bool near) {
    const int uh = cols.blocks == 1 ? uu : uu / cols.blocks, c0 = (uu - uh * cols.blocks) * cols.per;
    const size_t row0 = static_cast<size_t>(ub) * a.Sq * a.Hq + uh * heads;
    const bool whole = starts && ends;
    float* slot = near ? reinterpret_cast<float*>(ring) : my_slots + warp * C::kSlotFloats;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float sum = l[j];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      int hd, tk;
      if (column(2 * t + j, c0, &hd, &tk)) {
        const int c = (2 * t + j) & (C::kCols - 1);
        // A part of a unit leaves its sums times the power of two that makes the sum of P 1/2 to 1: its numerators
        // are then no larger than V.
        const int e = min(max(static_cast<int>(__float_as_uint(sum) >> 23) - 126, -126), 126);
        const float inv = sum == 0.f ? 0.f : whole ? 1.f / sum : pow2(-e);
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + (row0 + static_cast<size_t>(tk) * a.Hq + hd) * D + 4 * g + 32 * half;
        float* part = slot + c * D + 4 * g + 32 * half;
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          // raw numerators are in units of 2^-24 (odd channels: of 2^-20); 1 / rinv is exact, and goes in last
          const float f = __uint_as_float((254u << 23) - __float_as_uint(rinv[n][j]));
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = j + 2 * (i & 1);
            y[i] = (half ? acc[F * n + F - 1][i >> 1][at] : acc[F * n][i >> 1][at]) * inv * (i & 1 ? pow2(20) : pow2(24)) * f;
          }
          if (whole) *reinterpret_cast<uint2*>(o + 32 * F * n) = make_uint2(wm_pack_bf16x2(y[0], y[1]), wm_pack_bf16x2(y[2], y[3]));
          else *reinterpret_cast<float4*>(part + 32 * F * n) = make_float4(y[0], y[1], y[2], y[3]);
        }
        if (g == 0 && half == 0) {
          if (!whole) *reinterpret_cast<float2*>(slot + C::kCols * D + 2 * c) = make_float2(e - mneg[j], sum * inv);
          else if (a.lse) a.lse[(static_cast<size_t>(ub) * a.Hq + uh * heads + hd) * a.Sq + tk] = sum == 0.f ? -INFINITY : (log2f(sum) - mneg[j]) * kLn2;
        }
      }
    }
    __syncwarp();
    if (!whole && lane == 0) segs[2 * warp + which] = Segment{ub, uu, starts | ends << 1, near};
    which = 1;
  };

  int slot = 0;
  uint32_t phase = 0;
  while (true) {
    if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], phase))) {
      if (lane == 0) atomicCAS(pg.err, 0, kErrDeviceTimeout);
      break;
    }
    const int4 md = meta[slot];
    if (md.x < 0) break;  // an empty run
    const int k0 = md.z & ~31, flags = md.z & 31, ulen = md.w & 0x7fffffff;
    if (flags & 1) {
      begin_unit(md.x, md.y, ulen);
      seg_k0 = k0;
    }
    two_tiles(ring + slot * C::kStage, k0, flags >> 2, ulen);
    __syncwarp();
    if (lane == 0) mbar_arrive(&free_[slot]);
    if (++slot == R) {
      slot = 0;
      phase ^= 1;
    }
    if (flags & 2) {
      end_unit(md.x, md.y, seg_k0 == 0, k0 + C::kKeys >= ulen, md.w < 0);
      if (md.w < 0) break;
    }
  }
  }
  __syncthreads();

  // Segments of one unit follow one another in the warps' slots: join them, all units' columns at once.
  Segment sg;
  sg.b = -1;
  if (lane < 2 * W) sg = segs[lane];
  const unsigned valid = __ballot_sync(0xffffffffu, sg.b >= 0);
  const unsigned firsts = __ballot_sync(0xffffffffu, sg.b >= 0 && (sg.ends & 1)) | (valid & (0u - valid));
  const unsigned near = __ballot_sync(0xffffffffu, sg.b >= 0 && sg.near);
  const unsigned endings = __ballot_sync(0xffffffffu, sg.b >= 0 && (sg.ends & 2));
  const int items = cols.per * (D / 4);
  int i0 = __ffs(firsts) - 1, passed = 0;  // the first segment of the unit at hand; units before it, times items
  for (int at = threadIdx.x; firsts; at += C::kThreads) {
    while (i0 >= 0 && at >= passed + items) {
      passed += items;
      i0 = __ffs(firsts & ~((2u << i0) - 1u)) - 1;
    }
    if (i0 < 0) break;
    const unsigned later = firsts & ~((2u << i0) - 1u);
    unsigned members = valid & ~((1u << i0) - 1u) & ((later & (0u - later)) - 1u);
    const Segment first = segs[i0];
    const bool ends = endings >> (31 - __clz(members)) & 1;
    const int uh = first.u / cols.blocks, c0 = (first.u - uh * cols.blocks) * cols.per;
    const int item = at - passed, c = item / (D / 4), ch = item % (D / 4) * 4, col = c0 + c;
    if (col >= live_cols) continue;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, sum = 0.f;
    while (members) {
      constexpr int kBatch = 6;  // loads in flight
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (members) {
          const int x = __ffs(members) - 1;
          const float* from = near >> x & 1 ? reinterpret_cast<const float*>(smem + (x >> 1) * R * C::kStage) : my_slots + (x >> 1) * C::kSlotFloats;
          ml[i] = *reinterpret_cast<const float2*>(from + C::kCols * D + 2 * c);
          v[i] = *reinterpret_cast<const float4*>(from + c * D + ch);
          members &= members - 1;
        }
      }
      float top = M;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x + kSpare);
      const float zero = top == -INFINITY ? 0.f : top, old = wm_ex2(M - zero);
      M = top;
      sum *= old;
      O.x *= old, O.y *= old, O.z *= old, O.w *= old;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float wt = wm_ex2(ml[i].x - zero);
        sum = fmaf(wt, ml[i].y, sum);
        O.x = fmaf(wt, v[i].x, O.x), O.y = fmaf(wt, v[i].y, O.y), O.z = fmaf(wt, v[i].z, O.z), O.w = fmaf(wt, v[i].w, O.w);
      }
    }
    if ((first.ends & 1) && ends) {
      const int hd = col / a.Sq, sq = col - hd * a.Sq, hq = uh * heads + hd;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + ((static_cast<size_t>(first.b) * a.Sq + sq) * a.Hq + hq) * D + ch) =
          make_uint2(wm_pack_bf16x2(O.x * inv, O.y * inv), wm_pack_bf16x2(O.z * inv, O.w * inv));
      if (ch == 0 && a.lse)
        a.lse[(static_cast<size_t>(first.b) * a.Hq + hq) * a.Sq + sq] = sum == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(sum)) * kLn2;
    } else {
      // what leaves the CTA: slot 0 for the unit that its run starts in, slot 1 for one that starts later
      float* out = my_slots + (W + (first.b == first_unit->x && first.u == first_unit->y ? 0 : 1)) * C::kSlotFloats;
      *reinterpret_cast<float4*>(out + c * D + ch) = O;
      if (ch == 0) *reinterpret_cast<float2*>(out + C::kCols * D + 2 * c) = make_float2(M, sum);
    }
  }
}

template <int D, int F>
__global__ void __launch_bounds__(kCombineThreads) decode_kv4_combine_kernel(const DecodeKv4Args a, const Columns cols, int ctas,
                                                                            const Run* runs, const float* slots) {
  using C = Cfg<D, F>;
  __shared__ float4 part_o[kCombineThreads];
  __shared__ float2 part_ml[kCombineThreads];
  const int i = blockIdx.x + 1;  // the boundary before the run of CTA i
  const int tid = threadIdx.x;
  pdl_wait();  // the first kernel has finished and its slots are visible
  const Run run = runs[i];
  const long long total = runs[ctas].x, before = runs[i - 1].x, later = runs[min(tid + i, ctas)].x;
  // The first stage of the unit at the boundary; the boundary is the unit's first one, or another CTA's.
  const long long first = run.x - run.st;
  if (run.x >= total || run.st == 0 || first < before) return;
  // It has parts in CTA i - 1 and in every later one that starts inside it.
  const int n = 1 + __syncthreads_count(tid + i < ctas && later < first + run.nst);
  const int late = before + kUnitCost < first ? 1 : 0;  // the unit starts after CTA i - 1's run does
  const int heads = a.Hq / a.pages.Hkv, live_cols = heads * a.Sq;
  const int uh = run.u / cols.blocks, c0 = (run.u - uh * cols.blocks) * cols.per;
  const int items = cols.per * (D / 4), rows = kCombineThreads / items;
  const int item = tid % items, r = tid / items;
  const int c = item / (D / 4), ch = item % (D / 4) * 4;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, sum = 0.f;
  if (r < rows && c0 + c < live_cols) {
#pragma unroll 4
    for (int k = r; k < n; k += rows) {
      const float* from = slots + (static_cast<size_t>(i - 1 + k) * C::kSlots + C::W + (k == 0 ? late : 0)) * C::kSlotFloats;
      const float2 ml = *reinterpret_cast<const float2*>(from + C::kCols * D + 2 * c);
      const float4 v = *reinterpret_cast<const float4*>(from + c * D + ch);
      const float top = fmaxf(M, ml.x + kSpare), zero = top == -INFINITY ? 0.f : top;
      const float old = wm_ex2(M - zero), wt = wm_ex2(ml.x - zero);
      M = top;
      sum = fmaf(wt, ml.y, sum * old);
      O.x = fmaf(wt, v.x, O.x * old), O.y = fmaf(wt, v.y, O.y * old), O.z = fmaf(wt, v.z, O.z * old), O.w = fmaf(wt, v.w, O.w * old);
    }
  }
  part_o[tid] = O;
  part_ml[tid] = make_float2(M, sum);
  __syncthreads();
  if (r > 0 || c0 + c >= live_cols) return;
  float top = M;
  for (int k = 1; k < rows; ++k) top = fmaxf(top, part_ml[k * items + item].x);
  const float zero = top == -INFINITY ? 0.f : top;
  O = make_float4(0.f, 0.f, 0.f, 0.f);
  sum = 0.f;
  for (int k = 0; k < rows; ++k) {
    const float2 ml = part_ml[k * items + item];
    const float4 v = part_o[k * items + item];
    const float wt = wm_ex2(ml.x - zero);
    sum = fmaf(wt, ml.y, sum);
    O.x = fmaf(wt, v.x, O.x), O.y = fmaf(wt, v.y, O.y), O.z = fmaf(wt, v.z, O.z), O.w = fmaf(wt, v.w, O.w);
  }
  const int col = c0 + c, hq = uh * heads + col / a.Sq, sq = col % a.Sq;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + ((static_cast<size_t>(run.b) * a.Sq + sq) * a.Hq + hq) * D + ch) =
      make_uint2(wm_pack_bf16x2(O.x * inv, O.y * inv), wm_pack_bf16x2(O.z * inv, O.w * inv));
  if (ch == 0 && a.lse) a.lse[(static_cast<size_t>(run.b) * a.Hq + hq) * a.Sq + sq] = sum == 0.f ? -INFINITY : (zero + log2f(sum)) * kLn2;
}

// More columns than an MMA has go in equal blocks, which share the cache's bytes through L2: 16 columns in two
// blocks took 47 us where two MMAs a code fragment took 51 (19 sequences x 4 tokens: the wider state left
// too few warps).
Columns columns_of(int G, int Sq) {
  const int n = G * Sq, blocks = (n + 7) / 8;
  return {blocks, (n + blocks - 1) / blocks};
}

constexpr size_t kRunsBytes = (kMaxCtas + 1) * sizeof(Run);
static_assert(kRunsBytes % 16 == 0 && sizeof(Run) == 32, "slots start 16-byte aligned");

// CTAs of a call: one per SM, fewer where even the longest sequences have fewer stages.
int ctas_of(int B, int units, long long max_tokens, int keys) {
  const double most = static_cast<double>(B) * units * static_cast<double>((max_tokens + keys - 1) / keys);
  return most < kMaxCtas ? static_cast<int>(most) : kMaxCtas;
}

template <int D, int F>
size_t workspace_of(int B, int units, long long max_tokens) {
  using C = Cfg<D, F>;
  return kRunsBytes + static_cast<size_t>(ctas_of(B, units, max_tokens, C::kKeys)) * C::kSlots * C::kSlotFloats * sizeof(float);
}

template <int D, int F>
cudaError_t launch_df(const Columns cols, const DecodeKv4Args& a, cudaStream_t s) {
  using C = Cfg<D, F>;
  static_assert(C::kSmem <= 227 * 1024 && C::R >= 2 && 2 * C::W <= 32 && C::R * C::kStage >= C::kSlotFloats * 4, "the rings of all warps fit one SM");
  static DeviceOnce attr_set;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!attr_set.test(dev)) {
    e = cudaFuncSetAttribute(decode_kv4_kernel<D, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set.set(dev);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const Kv4Pages& p = a.pages;
  const int most = ctas_of(p.B, p.Hkv * cols.blocks, static_cast<long long>(p.max_pages) << p.page_shift, C::kKeys);
  const int grid = most < sms ? most : sms;
  Run* runs = static_cast<Run*>(a.work);
  float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(a.work) + kRunsBytes);
  decode_kv4_kernel<D, F><<<grid, C::kThreads, C::kSmem, s>>>(a, cols, runs, slots);
  e = cudaGetLastError();
  if (e != cudaSuccess || grid == 1) return e;
  return launch_after_pdl(decode_kv4_combine_kernel<D, F>, dim3(grid - 1), dim3(kCombineThreads), 0, s, a, cols, grid,
                          static_cast<const Run*>(runs), static_cast<const float*>(slots));
}

// Up to 4 columns fill half an MMA and share it between two groups of channels (F = 2), up to 8 fill one (F = 1).
template <typename Fn>
auto with_form(int d, int per, Fn fn) {
  using std::integral_constant;
  if (d == 64) return per <= 4 ? fn(integral_constant<int, 64>{}, integral_constant<int, 2>{}) : fn(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  return per <= 4 ? fn(integral_constant<int, 128>{}, integral_constant<int, 2>{}) : fn(integral_constant<int, 128>{}, integral_constant<int, 1>{});
}

}  // namespace

size_t decode_kv4_workspace_bytes(int B, int Sq, int Hq, int Hkv, long long max_tokens, int d) {
  const Columns c = columns_of(Hq / Hkv, Sq);
  return with_form(d, c.per, [&](auto D, auto F) { return workspace_of<D(), F()>(B, Hkv * c.blocks, max_tokens); });
}

cudaError_t launch_decode_kv4(int d, const DecodeKv4Args& a, cudaStream_t s) {
  const Columns c = columns_of(a.Hq / a.pages.Hkv, a.Sq);
  return with_form(d, c.per, [&](auto D, auto F) { return launch_df<D(), F()>(c, a, s); });
}

}  // namespace eio
