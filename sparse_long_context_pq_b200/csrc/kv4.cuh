// Device helpers and launch interfaces of the 4-bit KV cache (number format and tile layout:
// include/pqhsa.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace pqhsa {

constexpr int kTileTok = HSA_KV4_TILE_TOKENS;      // tokens per tile
constexpr int kTileBytes = HSA_KV4_TILE_BYTES;
constexpr int kOffV = 1024;                        // value codes within a tile
constexpr int kOffScale = 2048;                    // scale words within a tile
constexpr int kKv4MaxSms = 160;                    // blocks that the workspace has slots for, by SMs
// Places on the lines of steps are 32-bit. The host refuses longer lines; a kernel that finds one, by device lengths that
// have grown since, does no work and flags it.
constexpr long long kKv4MaxSteps = 1ll << 30;      // kv4_attend.cu
constexpr long long kKv4MaxWideSteps = 1ll << 31;  // kv4_prefill.cu

// What every kv4 kernel knows of the cache.
struct Kv4View {
  uint8_t* cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t* err;
  int B, Hq, Hkv, max_pages, num_pages;
  int page_tiles_log2;       // log2(page_size / 16)
};

// Tokens of sequence b, never more than its block table covers.
__device__ __forceinline__ int kv4_len(const Kv4View& c, int b) {
  const long long cap = static_cast<long long>(c.max_pages) << (c.page_tiles_log2 + 4);
  return static_cast<int>(max(0ll, min(static_cast<long long>(c.seq_lens[b]), cap)));
}

// Page of 16-token tile t of sequence b, -1 (flagged) if the block table has none.
__device__ __forceinline__ int kv4_page(const Kv4View& c, int b, int t) {
  const int page = c.block_table[static_cast<size_t>(b) * c.max_pages + (t >> c.page_tiles_log2)];
  if (page < 0 || page >= c.num_pages) {
    record_error(c.err, HSA_DEVERR_PAGE);
    return -1;
  }
  return page;
}

// Number in the cache (below 2^31, as the host checks) of head h's tile t (a sequence's tile number) in its page.
__device__ __forceinline__ uint32_t kv4_tile_index(const Kv4View& c, int page, int h, int t) {
  const uint32_t in_page = t & ((1 << c.page_tiles_log2) - 1);
  return ((static_cast<uint32_t>(page) * c.Hkv + h) << c.page_tiles_log2) + in_page;
}
__device__ __forceinline__ size_t kv4_tile_offset(const Kv4View& c, int page, int h, int t) {
  return static_cast<size_t>(kv4_tile_index(c, page, h, t)) * kTileBytes;
}

// A row of q passes through fp16 over a power of two, 2^q_exponent, which takes its largest element (magnitude `top`) to
// [2^13, 2^14): fp16 has all its 11 bits down to 2^-27 of that element. A row with an infinity has no weights, whatever
// its keys, and becomes NaN.
__device__ __forceinline__ int q_exponent(float top) {
  const int e = static_cast<int>(__float_as_uint(top) >> 23) - 140;
  return e > 114 ? 0 : max(e, -126);
}
// Where a row's ref begins: below every logit, and finite, so that a masked one, -inf, less it is -inf.
constexpr float kLowest = -3.4028235e38f;
// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// What a row of q is multiplied by.
__device__ __forceinline__ float q_factor(float top, int e) { return top < INFINITY ? pow2i(-e) : __int_as_float(0x7fffffff); }

// The four bytes of w, each a pair of codes (low nibble first), as fp16 pairs.
__device__ __forceinline__ void e2m1_to_f16x2(uint32_t w, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
      : "r"(w));
}
// Product of two fp16 pairs (exact for a code and a scale: at most six significant bits).
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Scale byte `i` of w in both halves of an fp16 pair: byte << 7 is the scale in fp16.
__device__ __forceinline__ uint32_t scale_both(uint32_t w, int i) { return ((w >> (8 * i)) & 0xffu) * 0x00800080u; }
// Scale bytes `i` and `i + 1` of w as an fp16 pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, int i) {
  const uint32_t v = w >> (8 * i);
  return ((v & 0xffu) << 7) | ((v & 0xff00u) << 15);
}

// ---- launch interfaces -------------------------------------------------------
struct Kv4RowsParams {
  Kv4View c;
  uint8_t* k;                 // rows of T, first element
  uint8_t* v;
  long long k_tok, k_head, v_tok, v_head;   // strides in bytes
  const int32_t* cu;          // [B + 1]
  const int32_t* start;       // read: first position; write: null (the last tokens)
  int n_rows;                 // rows behind k and v (cu_host[B])
};
// max_tiles: the most 16-token tiles that one sequence's rows touch
cudaError_t launch_kv4_write(int dtype, const Kv4RowsParams& p, int max_tiles, cudaStream_t stream, bool pdl);
cudaError_t launch_kv4_read(int dtype, const Kv4RowsParams& p, int max_tiles, cudaStream_t stream, bool pdl);

struct Kv4AttendParams {
  Kv4View c;
  const uint8_t* q;           // rows of [Hq][128] of the call's type
  long long q_tok;            // bytes between query tokens
  uint8_t* out;               // [rows][Hq][128]
  float* lse;                 // [rows][Hq] or null
  const int32_t* cu;          // [B + 1], or null: one query token a sequence
  float* parts;               // partial results of the blocks (see kv4_attend.cu)
  int n_rows;                 // query tokens behind q
  int causal, window, G;
  uint32_t inv_G;             // ceil(2^32 / G)
  float scale;
  int solo;                   // set by the launcher: no unit crosses blocks
};
// Rows (query tokens x heads of a group) of one unit of work; max_rows: the most that a sequence has for one KV head.
int kv4_attend_rows(int dtype, int max_rows);
size_t kv4_attend_part_bytes();
int kv4_attend_step_tokens();
// The work of a call: steps of kv4_attend_step_tokens tokens, and units, of all sequences together, the steps of the
// longest unit, and the most query rows that a sequence has for one KV head.
struct Kv4Load {
  long long steps, units, longest;
  int max_rows;
};
cudaError_t launch_kv4_attend(int dtype, int rows, const Kv4AttendParams& p, const Kv4Load& load, int sms,
                              cudaStream_t stream, bool pdl);

// Many query rows a KV head, 16-bit types (kv4_prefill.cu); p.cu is not null.
double kv4_prefill_steps(long long T, long long n, int G, bool causal, long long window, bool exact);   // of one head
size_t kv4_prefill_part_bytes();
cudaError_t launch_kv4_prefill(int dtype, const Kv4AttendParams& p, int sms, cudaStream_t stream, bool pdl);

// api.cu
int device_sms();      // multiprocessors of the current device, 0 on an error
bool pdl_enabled();

}  // namespace pqhsa
