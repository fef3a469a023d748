// kernels_kv4.h -- launchers of rotary positions and of the 4-bit paged KV cache,
// shared between the C ABI (api_kv4.cu) and the kernel files.
#pragma once

#include "kernels.h"

namespace eio {

// Rotary positions (rope.cu).  Strides in elements; heads and channels are
// contiguous.  freq: turns per position as a 64-bit fraction of a turn.
constexpr int kRopeMaxPairs = 64;
constexpr double kRopeMaxFreq = 65536.;
struct RopeArgs {
  const void* q;             // [B, N, Hq, d]
  const void* k;             // [B, N, Hk, d], Hk may be 0
  void* q_out;
  void* k_out;
  const int* positions;      // [B, N, n_axes]
  long long q_sb, q_sn, k_sb, k_sn, qo_sb, qo_sn, ko_sb, ko_sn, p_sb, p_sn;
  unsigned long long freq[kRopeMaxPairs];
  unsigned char axis[kRopeMaxPairs];
  int B, N, Hq, Hk, d, n_axes, n_pairs, inverse;
  int tokens_per_block;
};
cudaError_t launch_rope(bool bf16, bool interleaved, RopeArgs a, cudaStream_t s);

// The pages of a 4-bit KV cache (layout in kv4.cuh).
constexpr long long kKv4MaxTokens = 1ll << 30;  // of one sequence: positions and their rounding stay in 32 bits
struct Kv4Pages {
  uint8_t* pool;         // [n_pages][Hkv][T / 16][tile]
  const int* table;      // [B][max_pages] page ids
  const int* seqlens;    // [B] tokens, the appended or queried ones included
  int* err;
  int n_pages, max_pages, page_shift, B, Hkv;  // T = 1 << page_shift
};
struct Kv4AppendArgs {
  Kv4Pages pages;
  const void* k;       // [B, N, Hkv, d] bf16, strides in elements
  const void* v;
  const int* n_new;    // [B], or null: N each
  long long k_sb, k_sn, v_sb, v_sn;
  int N;
};
struct Kv4ReadArgs {
  Kv4Pages pages;
  void* k;             // [B, N, Hkv, d] bf16 (written)
  void* v;
  const int* start;    // [B] first position, or null: 0
  int N;
};
cudaError_t launch_kv4_append(int d, const Kv4AppendArgs& a, cudaStream_t s);
cudaError_t launch_kv4_read(int d, const Kv4ReadArgs& a, cudaStream_t s);

struct DecodeKv4Args {
  Kv4Pages pages;
  const void* q;       // [B, Sq, Hq, d] bf16
  void* o;             // [B, Sq, Hq, d] bf16
  float* lse;          // [B, Hq, Sq] or null
  void* work;
  int Sq, Hq;
  float scale_log2;
};
cudaError_t launch_decode_kv4(int d, const DecodeKv4Args& a, cudaStream_t s);
size_t decode_kv4_workspace_bytes(int B, int Sq, int Hq, int Hkv, long long max_tokens, int d);

// Pages src[i] of a pool copied to pages dst[i]; no destination named twice or also a source.
cudaError_t launch_copy_pages(void* pool, long long page_bytes, const int* src, const int* dst, int n, cudaStream_t s);

// The current device's error word (the one attn_sync_status reads), for calls
// on stream s; an attn_status (ATTN_ERR_UNSUPPORTED on a device that is not sm_100).
// Allocated at a device's first call, which is refused while s is captured.
int device_error_word(cudaStream_t s, int** out);

}  // namespace eio
