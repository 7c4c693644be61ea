// Attention over the 4-bit KV cache for many query rows a KV head (chunks of prompts): matrix
// products on the 5th-generation tensor cores.
//
// Work. A unit is (sequence, KV head, 256 query rows), its tokens are steps of 128 (only those
// that some row of the unit sees). As in kv4_attend.cu all units' steps lie on one line and
// every block, one an SM, takes an equal share of it; units that cross blocks leave a partial a
// block, which the merge kernel joins.
//
// A block has 14 warps, each walking through the block's segments for itself:
//   warps 0-3, 4-7  softmax of rows 0-127 and 128-255, one row a thread: S from TMEM, weights
//                   2^(S f - ref) as fp16 back into TMEM over S, now and then O scaled down;
//   warps 8-11      keys and values: codes x scales to fp16 (exact) in 128-byte-swizzled shared
//                   memory, two stages of 128 tokens each, the next tokens' codes in registers;
//   warps 12, 13    one lane each issues a half's MMAs: S = Q K^T (both operands in shared memory,
//                   K-major) and O += P V (P in TMEM, V with dims contiguous), M = N = 128, so that one
//                   half's products run under the other's softmax.
// A unit of at most 128 rows gives both halves the same rows, one the even steps and one the odd
// ones; their sums are joined at the end.
// TMEM: S of both halves (128 columns each; P takes the first 64), O of both (128 each).
// The MMAs of a half are issued by one thread and run in that order: P V of a step before the next
// S overwrites P, and S full means that every earlier P V has been added to O.
//
// What bounds it: the tensor cores need 2048 clocks for a step (4 x 128 x 128 x 128 products),
// ex2 as many (256 x 128 at 16 a clock), shared memory about 2000 (operands and dequantised tiles).
// Measured, a step takes about 5400 (2048 tokens over 32768, 32 heads on 8: 1.39 ms, 765 TFLOP/s): a
// half's chain is S full, maximum, weights, P, P V, the next S, with its softmax (about 2400 for 128 rows
// x 128 tokens) beside the other half's on the same schedulers, and TMEM has no room for a second S.
// Between two segments there are about 12000 clocks of output and q (4 sequences of 2048: 0.34 ms).
//
// q, weights and their accuracy are those of kv4_attend.cu for 16-bit calls: q over a power of two
// in fp16, P in fp16 up to 2^(kHead + kGrow), sums and statistics in fp32. ref moves by whole
// numbers, so that weights and sums made before are scaled exactly. S f - ref is one fused operation: below 2^23
// that is at most a quarter off the rounded S f less ref. Where a larger logit shows up, the warp's S is multiplied
// in TMEM from then on, and rounded, so that the largest logit meets a ref made of it (the same in registers
// cost 4% of 2048 tokens over 32768, this costs 2.5%).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4.cuh"

namespace pqhsa {
namespace {

constexpr int kRows = 256;                      // query rows of a unit
constexpr int kStepTok = 128;
constexpr int kStepTiles = kStepTok / kTileTok;
constexpr int kThreads = 14 * 32;
constexpr float kHead = 11.f, kGrow = 4.f;
constexpr float kWhole = 8388608.f;             // 2^23: larger logits are whole numbers, up to far more than kHead apart
constexpr int kRun = 128;                       // steps of a half that the tensor cores sum without rounding
constexpr int kPiece = 64;                      // tokens of a step that a softmax thread holds at a time
constexpr uint32_t kOperand = 128 * kD * 2;     // 32 KB: 128 rows of 128 fp16
constexpr uint32_t kHalfOp = kOperand / 2;      // one 64-element half (128 bytes a row)
constexpr int kSlot = kRows * (kD + 2);         // floats of a partial: m, l, acc

struct Smem {
  static constexpr uint32_t q = 0;              // two halves of rows
  static constexpr uint32_t k = 2 * kOperand;   // two stages
  static constexpr uint32_t v = k + 2 * kOperand;
  static constexpr uint32_t poison = v + 2 * kOperand;          // u32 [4 steps][8 dim groups][4 x 32 tokens]
  static constexpr uint32_t flags = poison + 4 * 8 * 4 * 4;     // u32 [4 steps][4 warps]
  static constexpr uint32_t bars = flags + 4 * 4 * 4;
  static constexpr uint32_t total = bars + 32 * 8;
};
constexpr size_t kSmemBytes = Smem::total + 1024;   // + alignment of the swizzle atoms

// D fp32, A and B fp16, M = N = 128; B's dims contiguous ("transposed") for P V.
constexpr uint32_t kIdescQK = (1u << 4) | (128u >> 3 << 17) | (128u >> 4 << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

// Operand in 128-byte swizzle atoms (8 rows x 128 bytes, 1024 bytes apart). K-major: rows are M or N,
// a 64-element half of K per 128 bytes. Dims-contiguous: rows are K (tokens), the 64-dim halves kHalfOp apart.
__device__ __forceinline__ uint64_t desc_k_major(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(kHalfOp >> 4) << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kIdescQK), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kIdescPV), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// As mbar_wait, with fewer instructions a poll (the waiting warps share issue slots with the working ones): the
// clock is read every 1024 polls.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, int32_t* err) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 0;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 1023u) == 1023u) {
      const uint64_t t = global_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) break;
    }
  }
  record_error(err, HSA_DEVERR_TIMEOUT);
  return false;
}
// The same with pauses, for waits whose end may be noticed late.
__device__ __forceinline__ bool wait_idle(uint64_t* bar, uint32_t parity, int32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  while (true) {
    __nanosleep(64);
    if (mbar_try_wait(bar, parity)) return true;
    if (global_ns() - t0 > kWaitLimitNs) break;
  }
  record_error(err, HSA_DEVERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool wait_long_warp(uint64_t* bar, uint32_t parity, int32_t* err) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_long(bar, parity, err);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}
// Barrier of the four softmax warps of a half and its MMA warp.
__device__ __forceinline__ void half_barrier(int half) {
  if (half == 0)
    asm volatile("bar.sync 2, 160;" ::: "memory");
  else
    asm volatile("bar.sync 3, 160;" ::: "memory");
}
// n columns of S times f, a row a lane. Not inlined: it is almost never called, and the loop around it is long enough.
__device__ __noinline__ void scale_tmem(uint32_t at, int n, float f) {
#pragma unroll 1
  for (int c = 0; c < n; c += 16) {
    uint32_t y[16];
    tmem_ld16(at + c, y);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__fmul_rn(__uint_as_float(y[i]), f));
    tmem_st16(at + c, y);
  }
  tmem_wait_st();
}
// The tensor cores cut off what does not fit a sum, a bias that grows with its tokens (a million of them came out 6e-3
// too small). So O holds kRun steps at most (16384 tokens, -6e-5): then each thread adds its row, with rounding, to its
// sums in a slot of the workspace, which holds their ref too, and in the end those to O (2048 tokens over 32768
// 1367 -> 1392 us).
enum Fold { kFoldFirst, kFoldMore, kFoldBack };
__device__ __noinline__ void fold(uint32_t o, float* slot, float ref, Fold how) {
  const float w = how == kFoldFirst ? 0.f : fast_exp2(slot[threadIdx.x] - ref);
  if (how != kFoldBack) slot[threadIdx.x] = ref;
  float4* sums = reinterpret_cast<float4*>(slot + 2 * kRows) + threadIdx.x;
#pragma unroll 1
  for (int c = 0; c < kD; c += 32) {
    float4 s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = how == kFoldFirst ? make_float4(0.f, 0.f, 0.f, 0.f) : sums[(c / 4 + i) * kRows];
    uint32_t y[32];
    tmem_ld32(o + c, y);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = make_float4(
          fmaf(s[i].x, w, __uint_as_float(y[4 * i])), fmaf(s[i].y, w, __uint_as_float(y[4 * i + 1])),
          fmaf(s[i].z, w, __uint_as_float(y[4 * i + 2])), fmaf(s[i].w, w, __uint_as_float(y[4 * i + 3])));
      if (how != kFoldBack) sums[(c / 4 + i) * kRows] = v;
      y[4 * i] = __float_as_uint(v.x);
      y[4 * i + 1] = __float_as_uint(v.y);
      y[4 * i + 2] = __float_as_uint(v.z);
      y[4 * i + 3] = __float_as_uint(v.w);
    }
    if (how == kFoldBack) {
      tmem_st16(o + c, y);
      tmem_st16(o + c + 16, y + 16);
    }
  }
  tmem_wait_st();
}
// Largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two floats as the register pair that the f32x2 instructions take, and back (moves that the allocator removes).
__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 unpair(unsigned long long v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
// Two products; one with an addition behind it may come out as a fused multiply-add.
__device__ __forceinline__ unsigned long long fmul2_rn(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Loads that leave L1 alone: the cache's bytes pass once.
__device__ __forceinline__ uint4 load_once16(const uint8_t* at) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(at));
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void* at, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}
__device__ __forceinline__ void store16(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint2 load_once8(const uint8_t* at) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(at));
  return v;
}

template <typename T>
__device__ __forceinline__ float4 q4_of(uint2 v) {
  if (sizeof(T) == 2 && __is_same(T, __nv_bfloat16)) return make_float4(bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (__is_same(T, __nv_bfloat16)) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  return pack_f16x2(lo, hi);
}

// ---- the line of steps ---------------------------------------------------------

struct Seq {
  int T, n, r0, nrt;     // tokens, query tokens, first query token's row, units a head
};
__device__ __forceinline__ Seq sequence(const Kv4AttendParams& p, int b) {
  Seq s;
  s.T = kv4_len(p.c, b);
  s.r0 = p.cu[b];
  s.n = p.cu[b + 1] - s.r0;
  s.n = max(0, min(s.n, p.n_rows - s.r0));
  if (s.r0 < 0) s.n = 0;
  s.nrt = (s.n * p.G + kRows - 1) / kRows;
  return s;
}
__device__ __forceinline__ int token_of(const Kv4AttendParams& p, int row) {
  return p.G == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.inv_G));
}
// Steps [x, y) of a sequence that some row of row tile rt sees.
__device__ __forceinline__ int2 unit_steps(const Kv4AttendParams& p, const Seq& s, int rt) {
  const int first = s.T - s.n + token_of(p, rt * kRows);
  const int last = s.T - s.n + token_of(p, min(rt * kRows + kRows, s.n * p.G) - 1);
  const int lo = p.window > 0 ? max(0, first - p.window + 1) / kStepTok : 0;
  const int hi = p.causal ? (last < 0 ? 0 : last / kStepTok + 1) : (s.T + kStepTok - 1) / kStepTok;
  return make_int2(lo, max(lo, hi));
}
// Steps of one head of a sequence, by a whole warp.
__device__ __forceinline__ long long head_steps(const Kv4AttendParams& p, const Seq& s) {
  long long sum = 0;
#pragma unroll 1
  for (int rt = threadIdx.x & 31; rt - static_cast<int>(threadIdx.x & 31) < s.nrt; rt += 32) {
    const int2 u = rt < s.nrt ? unit_steps(p, s, rt) : make_int2(0, 0);
    sum += __reduce_add_sync(0xffffffffu, u.y - u.x);
  }
  return sum;
}

// A piece of a unit: what a block works on at a time.
struct Segment {
  int b, h;
  int T, n, r0, row0, rows;
  int k0, k1;            // steps of the sequence
  int open;              // bits: begins at its unit's first step, ends at its last
  int slot;              // of the workspace, where it is not the whole unit
};

// A block's share of the line, walked through segment by segment by a whole warp.
struct Walk {
  int g, end, b, h, rt, in_unit, count;
  Seq s;
  __device__ __forceinline__ void start(const Kv4AttendParams& p) {
    Walk w = {};
    w.find(p);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) *this = w;
    __syncwarp();
  }
  __device__ __forceinline__ void find(const Kv4AttendParams& p) {
    long long all = 0;
#pragma unroll 1
    for (int i = 0; i < p.c.B; ++i) all += head_steps(p, sequence(p, i)) * p.c.Hkv;
    const bool past = all >= kKv4MaxWideSteps;   // by lengths that the host did not see
    if (past && blockIdx.x == 0 && threadIdx.x == 0) record_error(p.c.err, HSA_DEVERR_LIMIT);
    const int W = past ? 0 : static_cast<int>(all);
    const int N = min(static_cast<int>(gridDim.x), W), c = blockIdx.x;
    if (c >= N) {
      g = end = 0;
      return;
    }
    const int each = W / N, rest = W - each * N;
    g = each * c + min(c, rest);
    end = g + each + (c < rest ? 1 : 0);
    int left = g;
#pragma unroll 1
    for (;; ++b) {
      s = sequence(p, b);
      const int of_head = static_cast<int>(head_steps(p, s));
      if (left < of_head * p.c.Hkv) {
        h = left / of_head;
        left -= h * of_head;
        break;
      }
      left -= of_head * p.c.Hkv;
    }
#pragma unroll 1
    for (;; ++rt) {
      const int2 u = unit_steps(p, s, rt);
      if (left < u.y - u.x) break;
      left -= u.y - u.x;
    }
    in_unit = left;
  }
  // The next segment into n (shared memory), by a whole warp; false at the end.
  __device__ __forceinline__ bool next(const Kv4AttendParams& p, Segment& n) {
    Walk w = *this;
    Segment x;
    const bool more = w.step(p, x);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      *this = w;
      n = x;
    }
    __syncwarp();
    return more;
  }
  __device__ __forceinline__ bool step(const Kv4AttendParams& p, Segment& n) {
    if (g >= end) return false;
    int2 u = unit_steps(p, s, rt);
#pragma unroll 1
    while (in_unit >= u.y - u.x) {   // next unit with steps
      in_unit = 0;
      if (++rt >= s.nrt) {
        rt = 0;
        if (++h >= p.c.Hkv) {
          h = 0;
          if (++b >= p.c.B) return false;
          s = sequence(p, b);
        }
      }
      u = s.nrt ? unit_steps(p, s, rt) : make_int2(0, 0);
    }
    n.b = b;
    n.h = h;
    n.T = s.T;
    n.n = s.n;
    n.r0 = s.r0;
    n.row0 = rt * kRows;
    n.rows = min(kRows, s.n * p.G - n.row0);
    n.k0 = u.x + in_unit;
    n.k1 = min(u.y, n.k0 + end - g);
    n.open = (in_unit == 0 ? 1 : 0) | (n.k1 == u.y ? 2 : 0);
    n.slot = 2 * static_cast<int>(blockIdx.x) + (n.open == 1 && count > 0 ? 1 : 0);
    ++count;
    g += n.k1 - n.k0;
    in_unit += n.k1 - n.k0;
    return true;
  }
};

// What the merge kernel knows of a slot.
struct SlotInfo {
  int h, r0, row0, rows;
  int begins, ends, used, pad;
};

template <typename T>
__device__ __forceinline__ void write_row(const Kv4AttendParams& p, int r0, int h, int qrow, int c0, const float* x);

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const __grid_constant__ Kv4AttendParams p) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint32_t tmem_slot;
  __shared__ Walk walks[kThreads / 32];
  __shared__ Segment segments_s[kThreads / 32 + 8];   // the softmax warps have two
  __shared__ float factor[kRows];     // logits from S, in log2 units
  __shared__ float2 other[128];       // ref and l of the odd steps' half
  __shared__ unsigned other_poison[128];
  uint32_t* poison_s = reinterpret_cast<uint32_t*>(sm + Smem::poison);
  uint32_t* flags_s = reinterpret_cast<uint32_t*>(sm + Smem::flags);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Smem::bars);
  uint64_t* k_full = bars;            // [2] four warps
  uint64_t* k_empty = bars + 2;       // [2] commits of the halves that read the stage
  uint64_t* v_full = bars + 4;        // [2] four warps
  uint64_t* v_empty = bars + 6;       // [2] as k_empty
  uint64_t* s_full = bars + 8;        // [2 halves] commit
  uint64_t* o_full = bars + 10;       // [2 halves] commit, once a run
  uint64_t* drained = bars + 12;      // [2 halves] commit, at the end

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4);
      mbar_init(k_empty + i, 2);
      mbar_init(v_full + i, 4);
      mbar_init(v_empty + i, 2);
      mbar_init(s_full + i, 1);
      mbar_init(o_full + i, 1);
      mbar_init(drained + i, 1);
    }
    fence_mbar_init();
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  SlotInfo* info =
      reinterpret_cast<SlotInfo*>(p.parts + static_cast<size_t>(2 * kKv4MaxSms) * kSlot) + 2 * blockIdx.x;
  if (tid < 2) info[tid].used = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // ---- rows that see nothing: the first n - T query tokens, or all of an empty sequence ----
#pragma unroll 1
  for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
    const Seq s = sequence(p, b);
    const int blind = s.T == 0 ? s.n : p.causal ? max(0, s.n - s.T) : 0;
#pragma unroll 1
    for (long long i = tid; i < static_cast<long long>(blind) * p.c.Hq * (kD / 8); i += kThreads) {
      const size_t at = static_cast<size_t>(s.r0) * p.c.Hq * (kD / 8) + i;
      reinterpret_cast<uint4*>(p.out)[at] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse && at % (kD / 8) == 0) p.lse[at / (kD / 8)] = -INFINITY;
    }
  }

  // in shared memory, a copy a warp: the registers are wanted elsewhere
  Walk& walk = walks[warp];
  walk.start(p);
  if (warp < 8) {
    // ================= q, and softmax: one row a thread =================
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + half * 128, to = tmem + lanes + 256 + half * 128;
    bool more = walk.next(p, segments_s[warp]);
    int done = 0;         // this half's steps so far: phase of its barriers
    int runs = 0;         // and runs: phase of o_full
    int it = 0;           // the block's steps so far: place of their flags
    bool ok = true;       // a wait gave up: from there on only the barriers, which all eight warps pass
#pragma unroll 1
    for (int segments = 0; more; ++segments) {
      const Segment& cur = segments_s[warp + (segments & 1 ? kThreads / 32 : 0)];
      const int first_step = cur.k0, steps = cur.k1 - first_step;
      const bool split = cur.rows <= 128;
      // ---- q: rows over a power of two (with the scale's sign), fp16, K-major swizzled ----
      // two rows an instruction, eight values a lane, all of a warp's rows in flight
      const int mine = split ? 16 : 32;       // rows of this warp
      {
        uint4 x8[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int row = min(warp * mine + min(2 * k, mine - 2) + (lane >> 4), cur.rows - 1);
          const int i = token_of(p, cur.row0 + row);
          x8[k] = __ldg(reinterpret_cast<const uint4*>(
              p.q + (static_cast<long long>(cur.r0) + i) * p.q_tok +
              (static_cast<size_t>(cur.h) * p.G + (cur.row0 + row - i * p.G)) * kD * sizeof(T)) + (lane & 15));
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          if (2 * k >= mine) break;
          const int row = warp * mine + 2 * k + (lane >> 4);
          const float4 a = q4_of<T>(make_uint2(x8[k].x, x8[k].y)), b = q4_of<T>(make_uint2(x8[k].z, x8[k].w));
          float top = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                            fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int e = q_exponent(top);
          const float down = copysignf(q_factor(top, e), p.scale);
          const int r = row & 127;
          store16(smem_addr(sm) + Smem::q + (row >> 7) * kOperand + ((lane >> 3) & 1) * kHalfOp + r * 128 +
                      (((lane & 7) ^ (r & 7)) << 4),
                  pack_f16x2(a.x * down, a.y * down), pack_f16x2(a.z * down, a.w * down),
                  pack_f16x2(b.x * down, b.y * down), pack_f16x2(b.z * down, b.w * down));
          // never so small that a masked logit, -inf times f, is NaN
          if ((lane & 15) == 0) factor[row] = fmaxf(fabsf(p.scale * kLog2e * pow2i(e)), 1e-36f);
        }
      }
      fence_proxy_async_smem();
      asm volatile("bar.sync 4, 320;" ::: "memory");   // q and its factors; the MMA warps wait for them too

      const int row = split ? tid & 127 : tid;
      float f = factor[row];
      const bool real = row < cur.rows;
      const int pos = cur.T - cur.n + token_of(p, cur.row0 + (real ? row : 0));
      const int hi = !real ? -1 : p.causal ? pos : cur.T - 1;
      const int lo = p.window > 0 ? pos - p.window + 1 : 0;
      float ref = kLowest;
      bool scaled = false;          // S has been multiplied by f, which is 1 from then on
      unsigned long long l2[2] = {0, 0};
      unsigned poison = 0;          // bits 0-7: dim groups with a value that is not finite, bit 8: the whole row
      const int first = split ? half : 0, by = split ? 2 : 1;
      // slot of the sums of earlier runs: that of the partial; of a whole unit the second, which the last segment gets
      auto sums = [&]() { return p.parts + static_cast<size_t>(cur.open == 3 ? 2 * blockIdx.x + 1 : cur.slot) * kSlot; };
#pragma unroll 1
      for (int run = first; run < steps; run += kRun * by) {
        if (run > first) {
          ok = ok && wait_long_warp(o_full + half, runs++ & 1, p.c.err);
          tc_fence_after();
          if (ok) fold(to, sums(), ref, run == first + kRun * by ? kFoldFirst : kFoldMore);
          tc_fence_before();
        }
        const int run_end = min(steps, run + kRun * by);
#pragma unroll 1
        for (int j = run; j < run_end; j += by, ++done) {
          // After a wait that gave up there is no more work, but the barriers that others share are still passed.
          if (ok) ok = wait_long_warp(s_full + half, done & 1, p.c.err);
          if (!ok) {
            half_barrier(half);
            continue;
          }
          tc_fence_after();
          const int k0 = (first_step + j) * kStepTok;
          const uint4 fl = *reinterpret_cast<const uint4*>(flags_s + ((it + j) & 3) * 4);
          const unsigned flags = fl.x | fl.y | fl.z | fl.w;     // bits 0-7: tiles without a page, bit 8: poison
          const int from = max(0, lo - k0), upto = min(kStepTok - 1, hi - k0);   // tokens of the step that the row sees
          const bool masked = __any_sync(0xffffffffu, from > 0 || upto < kStepTok - 1 || (flags & 0xffu));
          auto seen32 = [&](int c0) -> uint32_t {   // those among [c0, c0 + 32)
            const int a = max(from - c0, 0), z = min(upto - c0, 31);
            uint32_t m = a <= z ? (0xffffffffu >> (31 - z)) & (0xffffffffu << a) : 0u;
            const unsigned gone = (flags >> (c0 / kTileTok)) & 3u;
            if (gone & 1u) m &= 0xffff0000u;
            if (gone & 2u) m &= 0x0000ffffu;
            return m;
          };
          if (flags & 0x100u) {   // values that are not finite, in blocks of 16 dims
            const uint32_t* words = poison_s + ((it + j) & 3) * 32;
#pragma unroll 1
            for (int gr = 0; gr < 8; ++gr) {
              uint32_t seen = 0;
#pragma unroll 1
              for (int q = 0; q < 4; ++q) seen |= words[gr * 4 + q] & seen32(q * 32);
              if (seen) poison |= 1u << gr;
            }
          }
          if (scaled) scale_tmem(ts, kStepTok, factor[row]);
          // in pieces of kPiece tokens: more at a time spill, and local memory is slow beside 200 KB of shared memory
#pragma unroll 1
          for (int q = 0; q < kStepTok / kPiece; ++q) {
            uint32_t x[kPiece];
#pragma unroll
            for (int k = 0; k < kPiece; k += 32) tmem_ld32(ts + q * kPiece + k, x + k);
            tmem_wait_ld();
            if (masked) {
#pragma unroll
              for (int k = 0; k < kPiece; k += 32) {
                const uint32_t m = seen32(q * kPiece + k);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[k + i] = (m >> i) & 1u ? x[k + i] : 0xff800000u;
              }
            }
            float tops[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tops[k] = max3_nan(__uint_as_float(x[k]), __uint_as_float(x[k + 4]), __uint_as_float(x[k + 8]));
#pragma unroll
            for (int i = 12; i + 8 <= kPiece; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tops[k] = max3_nan(tops[k], __uint_as_float(x[i + k]), __uint_as_float(x[i + 4 + k]));
#pragma unroll
            for (int k = 0; k < 4; ++k) tops[k] = max3_nan(tops[k], __uint_as_float(x[kPiece - 4 + k]), tops[k]);
            const float top = __fmul_rn(max3_nan(max3_nan(tops[0], tops[1], tops[2]), tops[3], tops[3]), f);
            if (__any_sync(0xffffffffu, !(__fsub_rn(top, ref) <= kHead + kGrow))) {
              // a logit of 2^23 or more: S of this piece and the rest times f, and the piece once more
              if (!scaled && __any_sync(0xffffffffu, fabsf(top) >= kWhole && top != -INFINITY)) {
                scaled = true;
                scale_tmem(ts + q * kPiece, kStepTok - q * kPiece, f);
                f = 1.f;
                --q;
                continue;
              }
              if (isnan(top)) poison |= 0x100u;
              const bool grow = __fsub_rn(top, ref) > kHead + kGrow;
              const float next = !grow ? ref : fabsf(top) < kWhole ? ceilf(top) - kHead : top;
              const float down = fmaxf(ref - next, -127.f);              // a whole number
              const float shrink = __int_as_float((static_cast<int>(down) + 127) << 23);   // 0 for 2^-127 and less
              ref = next;
              l2[0] = fmul2_rn(l2[0], pair(shrink, shrink));
              l2[1] = fmul2_rn(l2[1], pair(shrink, shrink));
              uint32_t y[16];
              tmem_wait_st();   // weights and O of this step that are stored already are read back below
              if (j > run) {
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                  tmem_ld16(to + k * 16, y);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * shrink);
                  tmem_st16(to + k * 16, y);
                }
              }
              const uint32_t s2 = pack_f16x2(shrink, shrink);
#pragma unroll 1
              for (int k = 0; k < q * (kPiece / 32); ++k) {     // weights of this step that are written already
                tmem_ld16(ts + k * 16, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = hmul2(y[i], s2);
                tmem_st16(ts + k * 16, y);
              }
            }
            const unsigned long long ref2 = pair(-ref, -ref);
            const unsigned long long f2 = pair(f, f);
#pragma unroll
            for (int i = 0; i < kPiece / 2; ++i) {
              const float2 y = unpair(ffma2_rn(pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), f2, ref2));
              const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
              l2[i & 1] = fadd2_rn(l2[i & 1], pair(e.x, e.y));
              x[i] = pack_f16x2(e.x, e.y);
            }
#pragma unroll
            for (int k = 0; k < kPiece / 32; ++k) tmem_st16(ts + (q * kPiece / 32 + k) * 16, x + 16 * k);
          }
          tmem_wait_st();
          tc_fence_before();
          half_barrier(half);   // this half's weights are there, for its MMA warp
        }
      }
      it += steps;
      more = walk.next(p, segments_s[warp + (segments & 1 ? 0 : kThreads / 32)]);   // while the last products run
      ok = ok && wait_long_warp(o_full + half, runs++ & 1, p.c.err);
      tc_fence_after();
      if (ok && steps > first + kRun * by) fold(to, sums(), ref, kFoldBack);
      // ---- the result, or a partial ----
      const float2 l01 = unpair(fadd2_rn(l2[0], l2[1]));
      float l = l01.x + l01.y;
      float mine_w = 1.f, other_w = 0.f;
      float4* staged = reinterpret_cast<float4*>(sm + Smem::q);   // [32 pieces][128 rows]; the products with q are done
      const bool none = half >= steps && split;                   // no step: O holds nothing of this segment
      if (split) {
        asm volatile("bar.sync 1, 256;" ::: "memory");   // both halves are done with q
        if (half == 1 && ok) {
          other[row] = make_float2(none ? kLowest : ref, none ? 0.f : l);
          other_poison[row] = poison;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t x[32];
            tmem_ld32(to + q * 32, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              staged[(q * 8 + i) * 128 + row] =
                  none ? make_float4(0.f, 0.f, 0.f, 0.f)
                       : make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]),
                                     __uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3]));
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (half == 0 && ok) {
          const float2 o = other[row];
          poison |= other_poison[row];
          const float m = fmaxf(ref, o.x);
          mine_w = fast_exp2(ref - m);
          other_w = fast_exp2(o.x - m);
          ref = m;
          l = l * mine_w + o.y * other_w;
        }
      }
      if (ok && (!split || half == 0)) {
        const bool whole = cur.open == 3, empty = l < 1.f;   // the largest weight is 2^(kHead - 1) or more
        if (empty) l = 0.f;
        if (poison & 0x100u) l = __int_as_float(0x7fffffff);
        const float inv = !whole ? 1.f : empty ? 0.f : __frcp_rn(l);
        mine_w *= inv;
        other_w *= inv;
        float* slot = p.parts + static_cast<size_t>(cur.slot) * kSlot;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t x[32];
          tmem_ld32(to + q * 32, x);
          tmem_wait_ld();
          const float a0 = (poison >> (2 * q)) & 0x101u ? __int_as_float(0x7fffffff) : 0.f;
          const float a1 = (poison >> (2 * q + 1)) & 0x81u ? __int_as_float(0x7fffffff) : 0.f;
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(x[i]) * mine_w + (i < 16 ? a0 : a1);
          if (split) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 v = staged[(q * 8 + i) * 128 + row];
              y[4 * i] = fmaf(v.x, other_w, y[4 * i]);
              y[4 * i + 1] = fmaf(v.y, other_w, y[4 * i + 1]);
              y[4 * i + 2] = fmaf(v.z, other_w, y[4 * i + 2]);
              y[4 * i + 3] = fmaf(v.w, other_w, y[4 * i + 3]);
            }
          }
          if (!whole) {        // [4 dims][row] of the slot
            if (real)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<float4*>(slot + 2 * kRows)[(q * 8 + i) * kRows + row] =
                    make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          } else if (split) {
            if (real) write_row<T>(p, cur.r0, cur.h, cur.row0 + row, q * 32, y);
          } else {             // through the place of q, a row's 16-byte pieces swizzled
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(sm + Smem::q + row * 256 + (((4 * q + i) ^ (row & 15)) << 4)) =
                  make_uint4(pack2<T>(y[8 * i], y[8 * i + 1]), pack2<T>(y[8 * i + 2], y[8 * i + 3]),
                             pack2<T>(y[8 * i + 4], y[8 * i + 5]), pack2<T>(y[8 * i + 6], y[8 * i + 7]));
          }
        }
        if (whole && !split) {
          __syncwarp();
#pragma unroll 4
          for (int k = 0; k < 16; ++k) {     // two rows an instruction
            const int o = warp * 32 + 2 * k + (lane >> 4);
            const uint4 v = *reinterpret_cast<const uint4*>(sm + Smem::q + o * 256 + (((lane & 15) ^ (o & 15)) << 4));
            if (o < cur.rows) {
              const int i = token_of(p, cur.row0 + o);
              reinterpret_cast<uint4*>(p.out)[((static_cast<size_t>(cur.r0) + i) * p.c.Hq + cur.h * p.G +
                                               (cur.row0 + o - i * p.G)) * (kD / 8) + (lane & 15)] = v;
            }
          }
        }
        if (real) {
          if (whole) {
            const int i = token_of(p, cur.row0 + row);
            if (p.lse)
              p.lse[(static_cast<size_t>(cur.r0) + i) * p.c.Hq + cur.h * p.G + (cur.row0 + row - i * p.G)] =
                  l == 0.f ? -INFINITY : (ref + __log2f(l)) * 0.6931471805599453f;
          } else {
            slot[row] = ref;
            slot[kRows + row] = l;
          }
        }
        if (!whole && tid == 0)
          info[cur.slot & 1] = SlotInfo{cur.h, cur.r0, cur.row0, cur.rows, cur.open & 1, cur.open >> 1, 1, 0};
      }
      tc_fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");   // O, factors and staged sums have been read
    }
  } else if (warp < 12) {
    // ================= keys and values =================
    const int w = warp & 3;                    // tiles 2w, 2w + 1 of a step
    const int r = lane >> 2, t = lane & 3;
    // Where this lane stores its four 16-byte pieces of a tile half (stage, tile and half are added):
    // keys: word i of a row's 16 bytes is dims 32 t + 8 i ..; lanes with t >= 2 take words 2, 3, 0, 1, so that the
    // eight lanes that store together meet eight different pieces of the banks;
    // values: [token][piece]; the two tokens of a byte part ways, and lanes of odd r store the odd token first.
    uint32_t to_k[4], to_v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v_row = 2 * t + ((i >> 1) ^ (r & 1));
      const int k_piece = (t & 1) * 4 + (i ^ (t & 2)), v_piece = (r & 3) * 2 + (i & 1);
      to_k[i] = smem_addr(sm) + Smem::k + (t >> 1) * kHalfOp + 2 * w * 2048 + r * 128 + ((k_piece ^ r) << 4);
      to_v[i] = smem_addr(sm) + Smem::v + (r >> 2) * kHalfOp + 2 * w * 2048 + v_row * 128 + ((v_piece ^ v_row) << 4);
    }
    const uint8_t* code_base = p.c.cache + lane * 16;
    const uint8_t* scale_base = p.c.cache + kOffScale + lane * 8;
    const uint32_t first_group = t & 2 ? 0x2301u : 0x3210u;   // bytes of a scale word, keys: the first word's group first
    const uint32_t sel0 = r & 1 ? 0x7632u : 0x5410u, sel1 = r & 1 ? 0x5410u : 0x7632u;
    int it = 0;
    bool ok = true;
    Segment& cur = segments_s[warp];
#pragma unroll 1
    while (ok && walk.next(p, cur)) {
      const int steps = cur.k1 - cur.k0, tokens = cur.T, k0 = cur.k0;
      int where = -1;                            // lane: cache tile of tile 32 * batch + lane of the segment
      unsigned gone = 0;                         // bits: of the loaded tiles, those without a page
      size_t tile[2];                            // byte offsets of the tiles of the step that is loaded next
      uint4 kc[2][2], vc[2][2];
      uint2 sc[2];
      // page numbers of 32 tiles (four steps) ahead; one warp also has their bytes brought into L2
      auto look_up = [&](int j) -> int {
        const int tl = (k0 + j) * kStepTiles + lane;
        if (tl > (tokens - 1) / kTileTok || tl >= (k0 + steps) * kStepTiles) return -1;
        const int page = kv4_page(p.c, cur.b, tl);
        if (page < 0) return -1;
        const uint32_t at = kv4_tile_index(p.c, page, cur.h, tl);
        if (w == 0) prefetch_l2(p.c.cache + static_cast<size_t>(at) * kTileBytes, kTileBytes);
        return static_cast<int>(at);
      };
      int ahead = look_up(0);
      auto find = [&](int j) {
        if ((j & 3) == 0) {
          where = ahead;
          ahead = look_up(j + 4);
        }
        gone = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int at = __shfl_sync(0xffffffffu, where, (j & 3) * kStepTiles + 2 * w + u);
          if (at < 0) gone |= 1u << u;
          tile[u] = static_cast<size_t>(static_cast<uint32_t>(max(at, 0))) * kTileBytes;
        }
      };
      auto fetch = [&](uint4 (&c)[2][2], int off) {   // a tile without a page: zeros
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          c[u][0] = load_once16(code_base + tile[u] + off);
          c[u][1] = load_once16(code_base + tile[u] + off + 512);
          if (off == 0) sc[u] = load_once8(scale_base + tile[u]);
          if (gone >> u & 1u) {
            c[u][0] = c[u][1] = make_uint4(0u, 0u, 0u, 0u);
            if (off == 0) sc[u] = make_uint2(0u, 0u);
          }
        }
      };
      find(0);
      fetch(kc, 0);
      fetch(vc, kOffV);
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        const int i_step = it + j, stage = i_step & 1;
        const uint32_t at = stage * kOperand, parity = ((i_step >> 1) & 1) ^ 1;
        const uint32_t vs[2] = {sc[0].y, sc[1].y};
        // values' scales that are not finite: bytes 248 and up (a zero byte of ~(y | 7))
        unsigned bad = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t z = ~(vs[u] | 0x07070707u);
          bad |= (z - 0x01010101u) & ~z & 0x80808080u;
        }
        const bool any_bad = __any_sync(0xffffffffu, bad != 0u);
        if (lane == 0) ok = wait_idle(k_empty + stage, parity, p.c.err);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t sw = __byte_perm(sc[u].x, 0u, first_group);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 c = kc[u][half];
            const uint32_t cw[4] = {t & 2 ? c.z : c.x, t & 2 ? c.w : c.y, t & 2 ? c.x : c.z, t & 2 ? c.y : c.w};
            const uint32_t sa = scale_both(sw, 2 * half), sb = scale_both(sw, 2 * half + 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t x[4];
              e2m1_to_f16x2(cw[i], x[0], x[1], x[2], x[3]);
              const uint32_t s1 = i < 2 ? sa : sb;
              store16(to_k[i] + at + u * 2048 + half * 1024, hmul2(x[0], s1), hmul2(x[1], s1), hmul2(x[2], s1),
                      hmul2(x[3], s1));
            }
          }
        }
        // what the softmax has to know of the step
        uint32_t word = 0;
        if (any_bad) {                       // group r: bit = token of this warp's 32
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (((vs[u] >> (8 * i)) & 0xffu) >= 248u) word |= 1u << (16 * u + 8 * (i >> 1) + 2 * t + (i & 1));
          word |= __shfl_xor_sync(0xffffffffu, word, 1);
          word |= __shfl_xor_sync(0xffffffffu, word, 2);
        }
        if (t == 0) poison_s[(i_step & 3) * 32 + r * 4 + w] = word;
        if (lane == 0) flags_s[(i_step & 3) * 4 + w] = (gone << (2 * w)) | (any_bad ? 0x100u : 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + stage);
        if (j + 1 < steps) {                 // there before the stage after next is free
          find(j + 1);
          fetch(kc, 0);
        }
        if (lane == 0) ok = wait_idle(v_empty + stage, parity, p.c.err);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        const int left = tokens - (k0 + j) * kStepTok;   // tokens from the step's first on
        const bool edge = left < kStepTok || any_bad;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t s2 = scale_pair(vs[u], 2 * half);
            if (edge) {                      // tokens that are not finite, or past the end, become zeros
              const int tok = (2 * w + u) * kTileTok + half * 8 + 2 * t;
              if ((s2 & 0x7c00u) == 0x7c00u || tok >= left) s2 &= 0xffff0000u;
              if ((s2 & 0x7c000000u) == 0x7c000000u || tok + 1 >= left) s2 &= 0x0000ffffu;
            }
            const uint32_t cw[4] = {vc[u][half].x, vc[u][half].y, vc[u][half].z, vc[u][half].w};
#pragma unroll
            for (int q = 0; q < 2; ++q) {    // eight dims of both tokens
              uint32_t x[8];
              e2m1_to_f16x2(cw[2 * q], x[0], x[1], x[2], x[3]);
              e2m1_to_f16x2(cw[2 * q + 1], x[4], x[5], x[6], x[7]);
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = hmul2(x[k], s2);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t sel = e ? sel1 : sel0;
                store16(to_v[2 * e + q] + at + u * 2048 + half * 1024, __byte_perm(x[0], x[1], sel),
                        __byte_perm(x[2], x[3], sel), __byte_perm(x[4], x[5], sel), __byte_perm(x[6], x[7], sel));
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + stage);
        if (j + 1 < steps) fetch(vc, kOffV);
      }
      it += steps;
    }
  } else {
    // ================= a half's MMAs: one lane =================
    const int half = warp - 12;
    int it = 0;
    bool ok = true;
    Segment& cur = segments_s[warp];
#pragma unroll 1
    while (walk.next(p, cur)) {
      const int steps = cur.k1 - cur.k0;
      const bool split = cur.rows <= 128;
      const int first = split ? half : 0, by = split ? 2 : 1;
      const uint64_t q_desc = desc_k_major(smem_addr(sm + Smem::q) + (split ? 0 : half) * kOperand);
      const uint64_t k_desc = desc_k_major(smem_addr(sm + Smem::k)), v_desc = desc_mn_major(smem_addr(sm + Smem::v));
      const uint32_t d_s = tmem + half * 128, d_o = tmem + 256 + half * 128;
      auto qk = [&](int i) {        // S of the block's step i; its keys are then free, for this half
        const uint64_t b = k_desc + (i & 1) * (kOperand >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalfOp + (kk & 3) * 32) >> 4;
          mma_ss(d_s, q_desc + off, b + off, kk > 0 ? 1u : 0u);
        }
        tc_commit(s_full + half);
        tc_commit(k_empty + (i & 1));
        if (split) mbar_arrive(k_empty + (i & 1));   // the other half does not read it
      };
      auto pv = [&](int i, bool fresh) {   // weights of step i times its values
        const uint64_t b = v_desc + (i & 1) * (kOperand >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_ts(d_o, d_s + kk * 8, b + kk * (2048 >> 4), fresh && kk == 0 ? 0u : 1u);
        tc_commit(v_empty + (i & 1));
        if (split) mbar_arrive(v_empty + (i & 1));
      };
      asm volatile("bar.sync 4, 320;" ::: "memory");   // q is there
      if (lane == 0) {
        tc_fence_after();
        if (ok && first < steps) ok = wait_long(k_full + ((it + first) & 1), ((it + first) >> 1) & 1, p.c.err);
        tc_fence_after();
        if (ok && first < steps) qk(it + first);
      }
      __syncwarp();
      int nth = 0;                  // of the run
#pragma unroll 1
      for (int j = first; j < steps; j += by) {
        // ahead of the weights: the values and the next keys. With split steps these keys are two steps on, and are
        // made after the values between, whose stage is not free before this step's products.
        if (lane == 0 && ok) {
          ok = wait_long(v_full + ((it + j) & 1), ((it + j) >> 1) & 1, p.c.err);
          if (ok && !split && j + by < steps) ok = wait_long(k_full + ((it + j + by) & 1), ((it + j + by) >> 1) & 1, p.c.err);
        }
        __syncwarp();
        half_barrier(half);
        if (lane == 0 && ok) {
          tc_fence_after();
          pv(it + j, nth == 0);
          nth = (nth + 1) % kRun;
          if (nth == 0 && j + by < steps) tc_commit(o_full + half);
          if (j + by < steps) {
            if (split) ok = wait_long(k_full + ((it + j + by) & 1), ((it + j + by) >> 1) & 1, p.c.err);
            tc_fence_after();
            if (ok) qk(it + j + by);
          }
        }
        __syncwarp();
      }
      if (lane == 0 && ok) tc_commit(o_full + half);
      __syncwarp();
      it += steps;
    }
    if (lane == 0) {
      tc_commit(drained + half);
      wait_long(drained + half, 0, p.c.err);   // nothing of ours still writes TMEM
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// 32 values of a row from dim c0 on.
template <typename T>
__device__ __forceinline__ void write_row(const Kv4AttendParams& p, int r0, int h, int qrow, int c0, const float* x) {
  const int i = token_of(p, qrow);
  const size_t at = ((static_cast<size_t>(r0) + i) * p.c.Hq + static_cast<size_t>(h) * p.G + (qrow - i * p.G)) * kD + c0;
  uint4* out = reinterpret_cast<uint4*>(p.out + at * sizeof(T));
#pragma unroll
  for (int k = 0; k < 4; ++k)
    out[k] = make_uint4(pack2<T>(x[8 * k], x[8 * k + 1]), pack2<T>(x[8 * k + 2], x[8 * k + 3]),
                        pack2<T>(x[8 * k + 4], x[8 * k + 5]), pack2<T>(x[8 * k + 6], x[8 * k + 7]));
}

// Joins the partials of the unit that begins in block blockIdx.x and goes on in the next ones: 32 rows x 8 dims a warp.
constexpr int kMergeWarps = 8;
template <typename T>
__global__ void __launch_bounds__(kMergeWarps * 32)
    kv4_prefill_merge_kernel(const __grid_constant__ Kv4AttendParams p, int blocks) {
  pdl_launch_dependents();
  pdl_wait();
  const SlotInfo* info = reinterpret_cast<const SlotInfo*>(p.parts + static_cast<size_t>(2 * kKv4MaxSms) * kSlot);
  const int c = blockIdx.x;
  int s0 = -1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const SlotInfo i = info[2 * c + k];
    if (i.used && i.begins && !i.ends) s0 = 2 * c + k;
  }
  if (s0 < 0) return;
  const SlotInfo u = info[s0];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * 32 + lane;
  if (blockIdx.y * 32 >= u.rows) return;
  int parts = 1;
  while (c + parts < blocks && !info[2 * (c + parts)].ends) ++parts;
  parts = min(parts + 1, blocks - c);   // with the one that ends it
#pragma unroll 1
  for (int d8 = warp; d8 < kD / 8; d8 += kMergeWarps) {
    float m = kLowest, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 2
    for (int i = 0; i < parts; ++i) {
      const float* slot = p.parts + static_cast<size_t>(i == 0 ? s0 : 2 * (c + i)) * kSlot;
      const float mi = slot[row], li = slot[kRows + row];
      const float4* acc = reinterpret_cast<const float4*>(slot + 2 * kRows) + 2 * d8 * kRows + row;
      const float4 v = acc[0], w = acc[kRows];
      const float next = fmaxf(m, mi);
      const float x = fast_exp2(m - next), y = fast_exp2(mi - next);
      m = next;
      l = fmaf(l, x, li * y);
      a = make_float4(fmaf(a.x, x, v.x * y), fmaf(a.y, x, v.y * y), fmaf(a.z, x, v.z * y), fmaf(a.w, x, v.w * y));
      b = make_float4(fmaf(b.x, x, w.x * y), fmaf(b.y, x, w.y * y), fmaf(b.z, x, w.z * y), fmaf(b.w, x, w.w * y));
    }
    if (row >= u.rows) continue;
    const float inv = l == 0.f ? 0.f : __frcp_rn(l);
    const int i = token_of(p, u.row0 + row);
    const size_t at = (static_cast<size_t>(u.r0) + i) * p.c.Hq + static_cast<size_t>(u.h) * p.G + (u.row0 + row - i * p.G);
    reinterpret_cast<uint4*>(p.out)[at * (kD / 8) + d8] =
        make_uint4(pack2<T>(a.x * inv, a.y * inv), pack2<T>(a.z * inv, a.w * inv), pack2<T>(b.x * inv, b.y * inv),
                   pack2<T>(b.z * inv, b.w * inv));
    if (p.lse && d8 == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
  }
}

template <typename T>
cudaError_t launch_prefill_t(const Kv4AttendParams& p, int sms, cudaStream_t stream, bool pdl) {
  cudaError_t e = ensure_dyn_smem<kv4_prefill_kernel<T>>(kSmemBytes);
  if (e != cudaSuccess) return e;
  const int blocks = std::min(sms, kKv4MaxSms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_prefill_kernel<T>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(blocks, kRows / 32);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv4_prefill_merge_kernel<T>, p, blocks);
}

}  // namespace

// As unit_steps, on the host and over all row tiles; not exact: those of a mask that leaves everything.
double kv4_prefill_steps(long long T, long long n, int G, bool causal, long long window, bool exact) {
  const long long every = (T + kStepTok - 1) / kStepTok, tiles = (n * G + kRows - 1) / kRows;
  if (!causal || !exact) return static_cast<double>(every) * static_cast<double>(tiles);
  double sum = 0;
  for (long long t = 0; t < tiles; ++t) {
    const long long first = T - n + t * kRows / G, last = T - n + (std::min((t + 1) * kRows, n * G) - 1) / G;
    const long long lo = window > 0 ? std::max(0ll, first - window + 1) / kStepTok : 0;
    sum += static_cast<double>(std::max(0ll, (last < 0 ? 0 : last / kStepTok + 1) - lo));
  }
  return sum;
}

size_t kv4_prefill_part_bytes() {
  return static_cast<size_t>(2 * kKv4MaxSms) * (kSlot * sizeof(float) + sizeof(SlotInfo));
}

cudaError_t launch_kv4_prefill(int dtype, const Kv4AttendParams& p, int sms, cudaStream_t stream, bool pdl) {
  if (dtype == HSA_BF16) return launch_prefill_t<__nv_bfloat16>(p, sms, stream, pdl);
  if (dtype == HSA_F16) return launch_prefill_t<__half>(p, sms, stream, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace pqhsa
