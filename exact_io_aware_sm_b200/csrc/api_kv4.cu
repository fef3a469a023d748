// api_kv4.cu -- the C ABI of the operators around the 4-bit paged KV cache
// (declared in include/attn.h): argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <vector>

#include "../../include/attn.h"
#include "kernels_kv4.h"
#include "kv4.cuh"

namespace {

using namespace eio;

int fail(int code, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  set_error_detail(msg);
  return code;
}

int launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? ATTN_OK : fail(ATTN_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The sizes of the cache a call works on, into p (all but its pointers).
int check_pages(int B, int Hkv, int d, int n_pages, int page, int max_pages, Kv4Pages* p) {
  if (B < 1 || Hkv < 1 || n_pages < 1 || max_pages < 1)
    return fail(ATTN_ERR_SHAPE, "B, Hkv, n_pages and max_pages must be >= 1");
  if (B > (1 << 24) || Hkv > 65535) return fail(ATTN_ERR_SHAPE, "B must be at most 2^24 and Hkv 65535");
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "the 4-bit cache needs d in {64, 128}");
  int shift = 4;
  while (shift <= 8 && page != 1 << shift) ++shift;
  if (shift > 8) return fail(ATTN_ERR_UNSUPPORTED, "page (%d) must be 16, 32, 64, 128 or 256 tokens", page);
  if (static_cast<long long>(max_pages) << shift > kKv4MaxTokens)
    return fail(ATTN_ERR_SHAPE, "max_pages * page must be at most 2^30 tokens");
  p->B = B;
  p->Hkv = Hkv;
  p->n_pages = n_pages;
  p->max_pages = max_pages;
  p->page_shift = shift;
  return ATTN_OK;
}

// Rows that an append or a read covers: a warp each 16 of a head, numbered in 32 bits; positions of rows stay in them too.
int check_rows(int B, int N, int Hkv) {
  if (N < 1 || N > kKv4MaxTokens || static_cast<long long>(B) * N >= (1ll << 31))
    return fail(ATTN_ERR_SHAPE, "N must be 1 to 2^30 and B * N below 2^31");
  if (B * ((N / 16 + 2.0) * Hkv + 4) >= 2147483648.0)
    return fail(ATTN_ERR_SHAPE, "too many rows: B * (N / 16 + 2) * Hkv must be below 2^31");
  return ATTN_OK;
}

int ready(void* stream, int** err) { return device_error_word(static_cast<cudaStream_t>(stream), err); }

}  // namespace

extern "C" {

int attn_rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions, const uint8_t* axes,
              const double* freq, const int64_t* strides, int B, int N, int Hq, int Hk, int d, int n_axes, int n_pairs,
              int interleaved, int inverse, int dtype, void* stream) {
  if (!q || !q_out || !positions || !axes || !freq || !strides || (Hk > 0 && (!k || !k_out)))
    return fail(ATTN_ERR_NULL, "q, q_out, positions, axes, freq, strides (and k, k_out with Hk > 0) must be non-NULL");
  if (B < 1 || N < 1 || Hq < 1 || Hk < 0) return fail(ATTN_ERR_SHAPE, "B, N and Hq must be >= 1, Hk >= 0");
  if (Hq > 65535 || Hk > 65535 || static_cast<long long>(B) * N >= (1ll << 31))
    return fail(ATTN_ERR_SHAPE, "Hq and Hk must be <= 65535 and B * N below 2^31");
  if (d != 32 && d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "attn_rope needs d in {32, 64, 128}");
  if (dtype != ATTN_BF16 && dtype != ATTN_F32)
    return fail(ATTN_ERR_UNSUPPORTED, "dtype %d is not ATTN_BF16 or ATTN_F32", dtype);
  if (n_axes < 1 || n_axes > 4) return fail(ATTN_ERR_SHAPE, "n_axes (%d) must be 1 to 4", n_axes);
  if (n_pairs < 1 || n_pairs > d / 2)
    return fail(ATTN_ERR_SHAPE, "n_pairs (%d) must be 1 to d / 2 (%d)", n_pairs, d / 2);
  const int esize = dtype == ATTN_BF16 ? 2 : 4;
  for (int i = 0; i < 8; ++i)
    if ((i % 4 < 2 || Hk > 0) && (strides[i] < 0 || strides[i] * esize % 16 != 0))
      return fail(ATTN_ERR_ALIGN, "strides of q, k and the outputs must be multiples of 16 bytes");
  if (strides[8] < 0 || strides[9] < 0) return fail(ATTN_ERR_SHAPE, "strides of positions must not be negative");
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(positions, 4) ||
      (Hk > 0 && (!aligned(k, 16) || !aligned(k_out, 16))))
    return fail(ATTN_ERR_ALIGN, "device pointers must be 16-byte aligned (positions: 4-byte)");
  RopeArgs a{};
  for (int p = 0; p < n_pairs; ++p) {
    if (axes[p] >= n_axes) return fail(ATTN_ERR_SHAPE, "axes[%d] is %d; positions have %d axes", p, axes[p], n_axes);
    if (!(std::fabs(freq[p]) <= kRopeMaxFreq))
      return fail(ATTN_ERR_SHAPE, "freq[%d] must be finite and at most %g in magnitude", p, kRopeMaxFreq);
    // turns per position, modulo 1, as a 64-bit fraction
    long double turns = static_cast<long double>(freq[p]) * 0.159154943091895335768883763372514362L;  // 1 / 2 pi
    turns -= static_cast<long double>(static_cast<long long>(turns));
    if (turns < 0) turns += 1;
    const long double high = turns * 4294967296.0L;
    const unsigned long long hi = static_cast<unsigned long long>(static_cast<long long>(high));
    a.freq[p] = (hi << 32) + static_cast<unsigned long long>(static_cast<long long>((high - static_cast<long double>(hi)) * 4294967296.0L));
    a.axis[p] = axes[p];
  }
  if (int rc = require_sm100()) return rc;
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.positions = positions;
  a.q_sb = strides[0], a.q_sn = strides[1], a.k_sb = strides[2], a.k_sn = strides[3];
  a.qo_sb = strides[4], a.qo_sn = strides[5], a.ko_sb = strides[6], a.ko_sn = strides[7];
  a.p_sb = strides[8], a.p_sn = strides[9];
  a.B = B;
  a.N = N;
  a.Hq = Hq;
  a.Hk = Hk;
  a.d = d;
  a.n_axes = n_axes;
  a.n_pairs = n_pairs;
  a.inverse = inverse != 0;
  return launched(launch_rope(dtype == ATTN_BF16, interleaved != 0, a, static_cast<cudaStream_t>(stream)), "rope");
}

int attn_kv4_append(const void* k, const void* v, void* pool, const int32_t* table, const int32_t* seqlens,
                    const int32_t* n_new, const int64_t* strides, int B, int N, int Hkv, int d, int n_pages, int page,
                    int max_pages, void* stream) {
  if (!k || !v || !pool || !table || !seqlens || !strides)
    return fail(ATTN_ERR_NULL, "k, v, pool, table, seqlens and strides must be non-NULL");
  Kv4AppendArgs a{};
  if (int rc = check_pages(B, Hkv, d, n_pages, page, max_pages, &a.pages)) return rc;
  if (int rc = check_rows(B, N, Hkv)) return rc;
  for (int i = 0; i < 4; ++i)
    if (strides[i] < 0 || strides[i] % 8 != 0)
      return fail(ATTN_ERR_ALIGN, "strides of k and v must be multiples of 16 bytes");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pool, 128) || !aligned(table, 4) || !aligned(seqlens, 4) ||
      !aligned(n_new, 4))
    return fail(ATTN_ERR_ALIGN, "k and v must be 16-byte aligned, pool 128-byte, table, seqlens and n_new 4-byte");
  if (int rc = ready(stream, &a.pages.err)) return rc;
  a.pages.pool = static_cast<uint8_t*>(pool);
  a.pages.table = table;
  a.pages.seqlens = seqlens;
  a.k = k;
  a.v = v;
  a.n_new = n_new;
  a.k_sb = strides[0], a.k_sn = strides[1], a.v_sb = strides[2], a.v_sn = strides[3];
  a.N = N;
  return launched(launch_kv4_append(d, a, static_cast<cudaStream_t>(stream)), "4-bit cache append");
}

int attn_kv4_read(void* k, void* v, const void* pool, const int32_t* table, const int32_t* seqlens,
                  const int32_t* start, int B, int N, int Hkv, int d, int n_pages, int page, int max_pages,
                  void* stream) {
  if (!k || !v || !pool || !table || !seqlens)
    return fail(ATTN_ERR_NULL, "k, v, pool, table and seqlens must be non-NULL");
  Kv4ReadArgs a{};
  if (int rc = check_pages(B, Hkv, d, n_pages, page, max_pages, &a.pages)) return rc;
  if (int rc = check_rows(B, N, Hkv)) return rc;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pool, 128) || !aligned(table, 4) || !aligned(seqlens, 4) ||
      !aligned(start, 4))
    return fail(ATTN_ERR_ALIGN, "k and v must be 16-byte aligned, pool 128-byte, table, seqlens and start 4-byte");
  if (int rc = ready(stream, &a.pages.err)) return rc;
  a.pages.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
  a.pages.table = table;
  a.pages.seqlens = seqlens;
  a.k = k;
  a.v = v;
  a.start = start;
  a.N = N;
  return launched(launch_kv4_read(d, a, static_cast<cudaStream_t>(stream)), "4-bit cache read");
}

static int check_decode(int B, int Sq, int Hq, int Hkv, int d, int n_pages, int page, int max_pages, Kv4Pages* p) {
  if (int rc = check_pages(B, Hkv, d, n_pages, page, max_pages, p)) return rc;
  if (Sq < 1 || Hq < 1) return fail(ATTN_ERR_SHAPE, "Sq and Hq must be >= 1");
  if (Hq % Hkv != 0) return fail(ATTN_ERR_SHAPE, "Hq (%d) is not a multiple of Hkv (%d)", Hq, Hkv);
  if (Sq > (1 << 20) || Hq > (1 << 20) || static_cast<double>(B) * Sq * Hq > (1 << 30))
    return fail(ATTN_ERR_SHAPE, "too many query rows");
  // A warp counts its stages (32 keys of 8 columns; up to 4 more for a unit's rounding, start and end) in 32 bits:
  // 2^41 are 1.4e9 for each of 148 x 11.
  const long long blocks = (static_cast<long long>(Hq / Hkv) * Sq + 7) / 8;
  if (static_cast<double>(B) * Hkv * blocks * ((static_cast<long long>(max_pages) << p->page_shift) / 32 + 4) >= 2199023255552.0)
    return fail(ATTN_ERR_SHAPE, "too much work: B * Hkv * ceil(Hq / Hkv * Sq / 8) * (max_pages * page / 32 + 4) must be below 2^41");
  return ATTN_OK;
}

int64_t attn_decode_kv4_workspace(int B, int Sq, int Hq, int Hkv, int d, int page, int max_pages) {
  Kv4Pages p{};
  if (check_decode(B, Sq, Hq, Hkv, d, 1, page, max_pages, &p)) return -1;
  return static_cast<int64_t>(
      decode_kv4_workspace_bytes(B, Sq, Hq, Hkv, static_cast<long long>(max_pages) << p.page_shift, d));
}

int attn_decode_kv4(const void* q, const void* pool, const int32_t* table, const int32_t* seqlens, void* o, float* lse,
                    void* workspace, int64_t workspace_bytes, int B, int Sq, int Hq, int Hkv, int d, int n_pages,
                    int page, int max_pages, float scale, void* stream) {
  if (!q || !pool || !table || !seqlens || !o)
    return fail(ATTN_ERR_NULL, "q, pool, table, seqlens and o must be non-NULL");
  DecodeKv4Args a{};
  if (int rc = check_decode(B, Sq, Hq, Hkv, d, n_pages, page, max_pages, &a.pages)) return rc;
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(ATTN_ERR_SHAPE, "scale must be positive and finite");
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(pool, 128) || !aligned(table, 4) || !aligned(seqlens, 4) ||
      !aligned(lse, 4) || !aligned(workspace, 16))
    return fail(ATTN_ERR_ALIGN, "q, o and workspace must be 16-byte aligned, pool 128-byte, table, seqlens and lse 4-byte");
  const int64_t need = static_cast<int64_t>(
      decode_kv4_workspace_bytes(B, Sq, Hq, Hkv, static_cast<long long>(max_pages) << a.pages.page_shift, d));
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(ATTN_ERR_WORKSPACE, "attn_decode_kv4 needs a workspace of %lld bytes, got %lld", static_cast<long long>(need),
                workspace ? static_cast<long long>(workspace_bytes) : 0ll);
  if (int rc = ready(stream, &a.pages.err)) return rc;
  a.pages.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
  a.pages.table = table;
  a.pages.seqlens = seqlens;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.work = workspace;
  a.Sq = Sq;
  a.Hq = Hq;
  a.scale_log2 = scale * 1.4426950408889634f;
  return launched(launch_decode_kv4(d, a, static_cast<cudaStream_t>(stream)), "4-bit cache decode");
}

int attn_copy_pages(void* pool, int64_t page_bytes, int n_pages, const int32_t* src, const int32_t* dst, int n,
                    void* stream) {
  if (n < 0) return fail(ATTN_ERR_SHAPE, "n must be >= 0");
  if (!pool || (n > 0 && (!src || !dst))) return fail(ATTN_ERR_NULL, "pool, src and dst must be non-NULL");
  if (n_pages < 1 || page_bytes < 16 || page_bytes % 16 != 0)
    return fail(ATTN_ERR_SHAPE, "n_pages must be >= 1 and page_bytes a positive multiple of 16");
  if (!aligned(pool, 16)) return fail(ATTN_ERR_ALIGN, "pool must be 16-byte aligned");
  try {
    std::vector<bool> taken(n_pages, false);
    for (int i = 0; i < n; ++i) {
      if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages)
        return fail(ATTN_ERR_SHAPE, "move %d (page %d to %d) leaves the pool of %d pages", i, src[i], dst[i], n_pages);
      if (taken[dst[i]]) return fail(ATTN_ERR_SHAPE, "page %d is a destination twice", dst[i]);
      taken[dst[i]] = true;
    }
    for (int i = 0; i < n; ++i)
      if (taken[src[i]]) return fail(ATTN_ERR_SHAPE, "page %d is both a source and a destination", src[i]);
  } catch (const std::exception& e) {
    return fail(ATTN_ERR_WORKSPACE, "checking the moves: %s", e.what());
  }
  if (int rc = require_sm100()) return rc;
  if (n == 0) return ATTN_OK;
  return launched(launch_copy_pages(pool, page_bytes, src, dst, n, static_cast<cudaStream_t>(stream)), "page copy");
}

}  // extern "C"
