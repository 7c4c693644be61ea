// Host side of the 4-bit KV cache calls of include/pqhsa.h: argument validation, planning and
// launches. No allocation and no state.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "../../include/pqhsa.h"
#include "kv4.cuh"

using namespace pqhsa;

namespace {

constexpr int kMaxGroup = 128;      // query heads a KV head
constexpr int kMaxBatch = 65535;    // grid rows
// Query rows a KV head up to which the streaming kernel is used. Measured (us), streaming and 256-row kernel: 64 rows on
// 8 heads of 131072 tokens 149 and 160, of 16384 46 and 57, on 64 x 8 heads of 2000 167 and 214, but on 16 x 8 of 5000 113
// and 104; 72 rows on those 145 and 105, on 8 heads of 131072 206 and 161: past 64 rows a third unit of 32 reads the
// cache's bytes a third time.
constexpr int kFewRows = 64;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t elem_bytes(int32_t dtype) { return dtype == HSA_F32 ? 4 : 2; }
bool known_type(int32_t dtype) { return dtype == HSA_F32 || dtype == HSA_BF16 || dtype == HSA_F16; }

hsa_status check_kv4(const hsa_kv4_cache* kv) {
  if (!kv || !kv->cache || !kv->block_table || !kv->seq_lens || !kv->seq_lens_host) return HSA_ERR_INVALID_ARG;
  if (kv->B < 1 || kv->Hkv < 1 || kv->Hq < 1 || kv->max_pages < 1 || kv->num_pages < 1) return HSA_ERR_INVALID_ARG;
  if (kv->Hq % kv->Hkv) return HSA_ERR_INVALID_ARG;
  if (kv->Hq / kv->Hkv > kMaxGroup || kv->B > kMaxBatch) return HSA_ERR_UNSUPPORTED;
  if (kv->D != kD) return HSA_ERR_UNSUPPORTED;
  if (kv->page_size != 16 && kv->page_size != 32 && kv->page_size != 64 && kv->page_size != 128)
    return HSA_ERR_UNSUPPORTED;
  if (!aligned(kv->cache, 256) || !aligned(kv->block_table, 4) || !aligned(kv->seq_lens, 4)) return HSA_ERR_ALIGNMENT;
  const long long tmax = static_cast<long long>(kv->max_pages) * kv->page_size;
  if (tmax >= (1LL << 30)) return HSA_ERR_UNSUPPORTED;   // differences of positions, rows and windows are 32-bit
  if (static_cast<long long>(kv->num_pages) * kv->Hkv * (kv->page_size / kTileTok) >= (1LL << 31))
    return HSA_ERR_UNSUPPORTED;                          // tile numbers are 32-bit
  for (int b = 0; b < kv->B; ++b)
    if (kv->seq_lens_host[b] < 0 || kv->seq_lens_host[b] > tmax) return HSA_ERR_CAPACITY;
  return HSA_OK;
}

size_t workspace_bytes() {
  return sizeof(WsHeader) + align_up(std::max(kv4_attend_part_bytes(), kv4_prefill_part_bytes()), 256);
}

hsa_status check_workspace(const void* ws, size_t bytes) {
  return !ws || !aligned(ws, 256) || bytes < workspace_bytes() ? HSA_ERR_WORKSPACE : HSA_OK;
}

hsa_status check_rows(const hsa_kv4_rows* r, int32_t dtype) {
  if (!r || !r->data) return HSA_ERR_INVALID_ARG;
  const long long e = elem_bytes(dtype);
  if (!aligned(r->data, 16) || r->token_stride * e % 16 || r->head_stride * e % 16) return HSA_ERR_ALIGNMENT;
  return HSA_OK;
}

// Whether no two of n x heads rows share an element.
bool rows_apart(const hsa_kv4_rows* r, long long n, long long heads) {
  long long near = std::llabs(r->token_stride), far = std::llabs(r->head_stride), count = n;   // the closer rows, and how many
  if (n == 1 || (heads > 1 && far < near)) {
    std::swap(near, far);
    count = heads;
  }
  if (count == 1) return true;
  return near >= kD && (n == 1 || heads == 1 || far >= near * (count - 1) + kD);
}

// cu[0] = 0, not falling; *most: the largest step.
hsa_status check_cu(const int32_t* cu, const int32_t* cu_host, int B, int* most) {
  if (!cu || !cu_host) return HSA_ERR_INVALID_ARG;
  if (!aligned(cu, 4)) return HSA_ERR_ALIGNMENT;
  if (cu_host[0] != 0) return HSA_ERR_INVALID_ARG;
  *most = 0;
  for (int b = 0; b < B; ++b) {
    if (cu_host[b + 1] < cu_host[b]) return HSA_ERR_INVALID_ARG;
    *most = std::max(*most, cu_host[b + 1] - cu_host[b]);
  }
  return HSA_OK;
}

Kv4View view(const hsa_kv4_cache* kv, void* ws) {
  Kv4View c = {};
  c.cache = static_cast<uint8_t*>(kv->cache);
  c.block_table = kv->block_table;
  c.seq_lens = kv->seq_lens;
  c.err = static_cast<int32_t*>(ws);
  c.B = kv->B;
  c.Hq = kv->Hq;
  c.Hkv = kv->Hkv;
  c.max_pages = kv->max_pages;
  c.num_pages = kv->num_pages;
  for (int s = kv->page_size / kTileTok; s > 1; s >>= 1) ++c.page_tiles_log2;
  return c;
}

Kv4RowsParams rows_params(const hsa_kv4_cache* kv, const hsa_kv4_rows* k, const hsa_kv4_rows* v, int32_t dtype,
                          const int32_t* cu, int n_rows, void* ws) {
  const long long e = elem_bytes(dtype);
  Kv4RowsParams p = {};
  p.c = view(kv, ws);
  p.k = static_cast<uint8_t*>(k->data);
  p.v = static_cast<uint8_t*>(v->data);
  p.k_tok = k->token_stride * e;
  p.k_head = k->head_stride * e;
  p.v_tok = v->token_stride * e;
  p.v_head = v->head_stride * e;
  p.cu = cu;
  p.n_rows = n_rows;
  return p;
}

// Checks shared by the two attention calls, and their launch. cu_host: null with one query token a sequence.
hsa_status attend(const hsa_kv4_cache* kv, const void* q, int64_t q_stride, void* out, float* lse, int32_t dtype,
                  const int32_t* cu, const int32_t* cu_host, float scale, int32_t causal, int32_t window, void* ws,
                  size_t ws_bytes, cudaStream_t stream) {
  hsa_status st = check_kv4(kv);
  if (st != HSA_OK) return st;
  if (!q || !out || !known_type(dtype) || !std::isfinite(scale) || window < 0 || (causal != 0 && causal != 1))
    return HSA_ERR_INVALID_ARG;
  if (window > 0 && !causal) return HSA_ERR_INVALID_ARG;
  int most = 1, n_rows = kv->B;
  if (cu_host || cu) {
    st = check_cu(cu, cu_host, kv->B, &most);
    if (st != HSA_OK) return st;
    n_rows = cu_host[kv->B];
    if (static_cast<long long>(most) * (kv->Hq / kv->Hkv) >= (1LL << 25)) return HSA_ERR_UNSUPPORTED;   // token_of
  }
  const long long e = elem_bytes(dtype);
  if (!aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4)) || q_stride * e % 16) return HSA_ERR_ALIGNMENT;
  st = check_workspace(ws, ws_bytes);
  if (st != HSA_OK) return st;
  if (n_rows == 0) return HSA_OK;
  if (q == out) return HSA_ERR_INVALID_ARG;   // blocks read q while others write
  Kv4AttendParams p = {};
  p.c = view(kv, ws);
  p.q = static_cast<const uint8_t*>(q);
  p.q_tok = q_stride * e;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.cu = cu;
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sizeof(WsHeader));
  p.n_rows = n_rows;
  p.causal = causal;
  p.window = window < static_cast<long long>(kv->max_pages) * kv->page_size ? window : 0;   // else it leaves nothing out
  p.G = kv->Hq / kv->Hkv;
  p.inv_G = static_cast<uint32_t>(((1ull << 32) + p.G - 1) / p.G);   // not used for G = 1
  p.scale = scale;
  if (cu && dtype != HSA_F32 && most * p.G > kFewRows) {
    double steps = 0;
    for (int exact = 0; exact < 2; ++exact) {   // counted out only where rows times tokens are too many
      steps = 0;
      for (int b = 0; b < kv->B; ++b)
        steps += kv->Hkv * kv4_prefill_steps(kv->seq_lens_host[b], cu_host[b + 1] - cu_host[b], p.G, causal, p.window, exact);
      if (steps < kKv4MaxWideSteps) break;
    }
    if (steps >= kKv4MaxWideSteps) return HSA_ERR_UNSUPPORTED;
    const int sms = device_sms();
    if (!sms) return HSA_ERR_CUDA;
    return launch_kv4_prefill(dtype, p, sms, stream, pdl_enabled()) == cudaSuccess ? HSA_OK : HSA_ERR_CUDA;
  }
  const int rows = kv4_attend_rows(dtype, most * p.G);
  Kv4Load load = {0, 0, 0, most * p.G};
  const int step = kv4_attend_step_tokens();
  for (int b = 0; b < kv->B; ++b) {
    const long long T = kv->seq_lens_host[b], n = cu_host ? cu_host[b + 1] - cu_host[b] : 1;
    if (n == 0 || T == 0) continue;
    const long long lo = window > 0 ? std::max(0ll, T - n - window + 1) / step : 0;
    const long long of_unit = (T + step - 1) / step - lo, units = (n * p.G + rows - 1) / rows * kv->Hkv;
    if (units >= kKv4MaxSteps) return HSA_ERR_UNSUPPORTED;
    load.steps += of_unit * units;
    if (load.steps >= kKv4MaxSteps) return HSA_ERR_UNSUPPORTED;
    load.units += units;
    load.longest = std::max(load.longest, of_unit);
  }
  const int sms = device_sms();
  if (!sms) return HSA_ERR_CUDA;
  const cudaError_t err = launch_kv4_attend(dtype, rows, p, load, sms, stream, pdl_enabled());
  return err == cudaSuccess ? HSA_OK : HSA_ERR_CUDA;
}

}  // namespace

extern "C" {

void hsa_kv4_abi_sizes(int64_t* cache, int64_t* rows) {
  if (cache) *cache = sizeof(hsa_kv4_cache);
  if (rows) *rows = sizeof(hsa_kv4_rows);
}

size_t hsa_kv4_workspace_bytes(const hsa_kv4_cache* kv) { return check_kv4(kv) == HSA_OK ? workspace_bytes() : 0; }

hsa_status hsa_kv4_write(const hsa_kv4_cache* kv, const hsa_kv4_rows* k, const hsa_kv4_rows* v, int32_t dtype,
                         const int32_t* cu_new, const int32_t* cu_new_host, void* ws, size_t ws_bytes,
                         cudaStream_t stream) {
  hsa_status st = check_kv4(kv);
  if (st != HSA_OK) return st;
  if (!known_type(dtype)) return HSA_ERR_INVALID_ARG;
  if ((st = check_rows(k, dtype)) != HSA_OK || (st = check_rows(v, dtype)) != HSA_OK) return st;
  int most = 0;
  if ((st = check_cu(cu_new, cu_new_host, kv->B, &most)) != HSA_OK) return st;
  for (int b = 0; b < kv->B; ++b)
    if (cu_new_host[b + 1] - cu_new_host[b] > kv->seq_lens_host[b]) return HSA_ERR_CAPACITY;
  if ((st = check_workspace(ws, ws_bytes)) != HSA_OK) return st;
  if (most == 0) return HSA_OK;
  const Kv4RowsParams p = rows_params(kv, k, v, dtype, cu_new, cu_new_host[kv->B], ws);
  return launch_kv4_write(dtype, p, most / kTileTok + 2, stream, pdl_enabled()) == cudaSuccess ? HSA_OK : HSA_ERR_CUDA;
}

hsa_status hsa_kv4_read(const hsa_kv4_cache* kv, const hsa_kv4_rows* k, const hsa_kv4_rows* v, int32_t dtype,
                        const int32_t* start, const int32_t* start_host, const int32_t* cu, const int32_t* cu_host,
                        void* ws, size_t ws_bytes, cudaStream_t stream) {
  hsa_status st = check_kv4(kv);
  if (st != HSA_OK) return st;
  if (!known_type(dtype) || !start || !start_host) return HSA_ERR_INVALID_ARG;
  if ((st = check_rows(k, dtype)) != HSA_OK || (st = check_rows(v, dtype)) != HSA_OK) return st;
  int most = 0;
  if ((st = check_cu(cu, cu_host, kv->B, &most)) != HSA_OK) return st;
  if (!aligned(start, 4)) return HSA_ERR_ALIGNMENT;
  for (int b = 0; b < kv->B; ++b) {
    if (start_host[b] < 0) return HSA_ERR_INVALID_ARG;
    if (static_cast<long long>(start_host[b]) + cu_host[b + 1] - cu_host[b] > kv->seq_lens_host[b])
      return HSA_ERR_CAPACITY;
  }
  if ((st = check_workspace(ws, ws_bytes)) != HSA_OK) return st;
  if (most == 0) return HSA_OK;
  const int n = cu_host[kv->B];
  if (k->data == v->data || !rows_apart(k, n, kv->Hkv) || !rows_apart(v, n, kv->Hkv)) return HSA_ERR_INVALID_ARG;
  Kv4RowsParams p = rows_params(kv, k, v, dtype, cu, cu_host[kv->B], ws);
  p.start = start;
  return launch_kv4_read(dtype, p, most / kTileTok + 2, stream, pdl_enabled()) == cudaSuccess ? HSA_OK : HSA_ERR_CUDA;
}

hsa_status dense_decode_kv4(const hsa_kv4_cache* kv, const void* q, void* out, float* lse, int32_t dtype, float scale,
                            int32_t window, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return attend(kv, q, kv ? static_cast<int64_t>(kv->Hq) * kD : 0, out, lse, dtype, nullptr, nullptr, scale, 1, window,
                ws, ws_bytes, stream);
}

hsa_status dense_prefill_kv4(const hsa_kv4_cache* kv, const void* q, int64_t q_stride, void* out, float* lse,
                             int32_t dtype, const int32_t* cu_q, const int32_t* cu_q_host, float scale, int32_t causal,
                             int32_t window, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!cu_q || !cu_q_host) return HSA_ERR_INVALID_ARG;
  return attend(kv, q, q_stride, out, lse, dtype, cu_q, cu_q_host, scale, causal, window, ws, ws_bytes, stream);
}

}  // extern "C"
