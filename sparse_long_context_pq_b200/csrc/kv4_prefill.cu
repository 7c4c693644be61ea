// Attention over the 4-bit KV cache for many query rows a KV head (chunks of prompts): matrix
// products on the 5th-generation tensor cores.
//
// Work. A unit is (sequence, KV head, 256 query rows), its tokens are steps of 128 (only those
// that some row of the unit sees). As in kv4_attend.cu all units' steps lie on one line and
// every block, one an SM, takes an equal share of it; units that cross blocks leave a partial a
// block, which the merge kernel joins.
//
// A block has 17 warps:
//   warps 0-3, 4-7    softmax of rows 0-127 and 128-255, one row a thread: S from TMEM, weights
//                     2^(S f - ref) as fp16 back into TMEM over S, now and then O scaled down;
//   warps 8-11, 12-15 keys and values: codes x scales to fp16 (exact) in 128-byte-swizzled shared
//                     memory, two stages of 128 tokens each, the next tokens' codes in registers;
//   warp 16           one lane issues the MMAs: S = Q K^T (both operands in shared memory, K-major)
//                     and O += P V (P in TMEM, V with dims contiguous), M = N = 128, the two row
//                     halves in turn, so that one's products run under the other's softmax.
// TMEM: S of both halves (128 columns each; P takes the first 64), O of both (128 each).
// The MMAs of a block run in the order of their issue: P V of a half is issued before the next
// S of that half overwrites P, and S full means that every earlier P V has been added to O.
//
// What bounds it: the tensor cores need 2048 clocks for a step (4 x 128 x 128 x 128 products),
// ex2 as many (256 x 128 at 16 a clock), shared memory about 2000 (operands and dequantised tiles).
//
// q, weights and their accuracy are those of kv4_attend.cu for 16-bit calls: q over a power of two
// in fp16, P in fp16 up to 2^(kHead + kGrow), sums and statistics in fp32.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4.cuh"

namespace pqhsa {
namespace {

constexpr int kRows = 256;                      // query rows of a unit
constexpr int kStepTok = 128;
constexpr int kStepTiles = kStepTok / kTileTok;
constexpr int kThreads = 17 * 32;
constexpr float kHead = 11.f, kGrow = 4.f;
constexpr uint32_t kOperand = 128 * kD * 2;     // 32 KB: 128 rows of 128 fp16
constexpr uint32_t kHalfOp = kOperand / 2;      // one 64-element half (128 bytes a row)
constexpr int kSlot = kRows * (kD + 2);         // floats of a partial: m, l, acc

struct Smem {
  static constexpr uint32_t q = 0;              // two halves of rows
  static constexpr uint32_t k = 2 * kOperand;   // two stages
  static constexpr uint32_t v = k + 2 * kOperand;
  static constexpr uint32_t factor = v + 2 * kOperand;          // float [256]: logits from S, in log2 units
  static constexpr uint32_t poison = factor + kRows * 4;        // u32 [4 steps][8 dim groups][4 x 32 tokens]
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
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <typename T>
__device__ __forceinline__ float4 load_q4(const uint8_t* at) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
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
__device__ __forceinline__ int head_steps(const Kv4AttendParams& p, const Seq& s) {
  int sum = 0;
#pragma unroll 1
  for (int rt = threadIdx.x & 31; rt - static_cast<int>(threadIdx.x & 31) < s.nrt; rt += 32) {
    const int2 u = rt < s.nrt ? unit_steps(p, s, rt) : make_int2(0, 0);
    sum += __reduce_add_sync(0xffffffffu, u.y - u.x);
  }
  return sum;
}

// A piece of a unit: what a block works on at a time.
struct Segment {
  int b, h, rt;
  int T, n, r0, row0, rows;
  int k0, k1;            // steps of the sequence
  int open;              // bits: begins at its unit's first step, ends at its last
  int slot;              // of the workspace, where it is not the whole unit
  int valid;
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
  __shared__ Segment seg;
  __shared__ uint32_t tmem_slot;
  __shared__ int failed;
  float* factor = reinterpret_cast<float*>(sm + Smem::factor);
  uint32_t* poison_s = reinterpret_cast<uint32_t*>(sm + Smem::poison);
  uint32_t* flags_s = reinterpret_cast<uint32_t*>(sm + Smem::flags);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Smem::bars);
  uint64_t* k_full = bars;            // [2] four warps
  uint64_t* k_empty = bars + 2;       // [2] commit
  uint64_t* v_full = bars + 4;        // [2] four warps
  uint64_t* v_empty = bars + 6;       // [2] commit
  uint64_t* s_full = bars + 8;        // [2 halves] commit
  uint64_t* p_full = bars + 10;       // [2 halves] four warps
  uint64_t* o_full = bars + 12;       // commit, once a segment
  uint64_t* drained = bars + 13;      // commit, at the end

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 4);
      mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
    }
    mbar_init(o_full, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
    failed = 0;
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

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

  // ---- this block's share of the line (every warp for itself; few sequences, few row tiles) ----
  int W = 0;
#pragma unroll 1
  for (int b = 0; b < p.c.B; ++b) W += head_steps(p, sequence(p, b)) * p.c.Hkv;
  const int N = min(static_cast<int>(gridDim.x), W);
  const int each = N > 0 ? W / N : 0, rest = W - each * N;
  const int c = blockIdx.x;
  int g = c < N ? each * c + min(c, rest) : 0;
  const int g_end = c < N ? g + each + (c < rest ? 1 : 0) : 0;
  SlotInfo* info = reinterpret_cast<SlotInfo*>(p.parts + static_cast<size_t>(2 * kKv4MaxSms) * kSlot) + 2 * c;
  if (tid < 2) info[tid].used = 0;

  // Warp 0 walks the line; the others read the segment it leaves.
  int b = 0, before = 0, of_head = 0, h = 0, rt = 0, in_unit = 0;   // unit and step within it
  Seq s = {};
  if (warp == 0 && g < g_end) {
    for (;; ++b) {
      s = sequence(p, b);
      of_head = head_steps(p, s);
      if (g - before < of_head * p.c.Hkv) break;
      before += of_head * p.c.Hkv;
    }
    h = (g - before) / of_head;
    in_unit = g - before - h * of_head;
    for (;; ++rt) {
      const int2 u = unit_steps(p, s, rt);
      if (in_unit < u.y - u.x) break;
      in_unit -= u.y - u.x;
    }
  }

  int it = 0;           // steps done by the block: stages and phases
  int segments = 0;
#pragma unroll 1
  for (;; ++segments) {
    if (warp == 0) {
      Segment n = {};
      if (g < g_end) {
        int2 u = unit_steps(p, s, rt);
        while (in_unit >= u.y - u.x) {   // next unit with steps
          in_unit = 0;
          if (++rt == s.nrt) {
            rt = 0;
            if (++h == p.c.Hkv) {
              h = 0;
              do {
                s = sequence(p, ++b);
              } while (b + 1 < p.c.B && s.nrt == 0);
            }
          }
          u = s.nrt ? unit_steps(p, s, rt) : make_int2(0, 0);
        }
        n.b = b;
        n.h = h;
        n.rt = rt;
        n.T = s.T;
        n.n = s.n;
        n.r0 = s.r0;
        n.row0 = rt * kRows;
        n.rows = min(kRows, s.n * p.G - n.row0);
        n.k0 = u.x + in_unit;
        n.k1 = min(u.y, n.k0 + g_end - g);
        n.open = (in_unit == 0 ? 1 : 0) | (n.k1 == u.y ? 2 : 0);
        n.slot = 2 * c + (n.open == 1 && segments > 0 ? 1 : 0);
        n.valid = 1;
        g += n.k1 - n.k0;
        in_unit += n.k1 - n.k0;
      }
      if (lane == 0) seg = n;
    }
    __syncthreads();
    if (!seg.valid || failed) break;
    const Segment cur = seg;
    const int steps = cur.k1 - cur.k0;

    // ---- q: rows over a power of two, fp16, K-major swizzled ----
#pragma unroll 2
    for (int row = warp; row < kRows; row += 17) {
      uint2 w = make_uint2(0u, 0u);
      float f = 0.f;
      if (row < cur.rows) {
        const int i = token_of(p, cur.row0 + row);
        const float4 x = load_q4<T>(p.q + (static_cast<long long>(cur.r0) + i) * p.q_tok +
                                    (static_cast<size_t>(cur.h) * p.G + (cur.row0 + row - i * p.G)) * kD * sizeof(T) +
                                    lane * 4 * sizeof(T));
        const float top = warp_max_f32(fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 126;
        e = e > 126 ? 0 : max(e, -126);
        const float down = __int_as_float((127 - e) << 23);
        w = make_uint2(pack_f16x2(x.x * down, x.y * down), pack_f16x2(x.z * down, x.w * down));
        f = p.scale * kLog2e * __int_as_float((e + 127) << 23);
      }
      const int r = row & 127, chunk = (lane & 15) >> 1;
      *reinterpret_cast<uint2*>(sm + Smem::q + (row >> 7) * kOperand + (lane >> 4) * kHalfOp + r * 128 +
                                ((chunk ^ (r & 7)) << 4) + (lane & 1) * 8) = w;
      if (lane == 0) factor[row] = f;
    }
    fence_proxy_async_smem();
    __syncthreads();

    if (warp < 8) {
      // ================= softmax: one row a thread =================
      const int half = warp >> 2;
      const int row = tid;                                    // 0 .. 255
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = tmem + lanes + half * 128, to = tmem + lanes + 256 + half * 128;
      const float f = factor[row];
      const bool real = row < cur.rows;
      const int pos = cur.T - cur.n + token_of(p, cur.row0 + (real ? row : 0));
      const int hi = !real ? -1 : p.causal ? pos : cur.T - 1;
      const int lo = p.window > 0 ? pos - p.window + 1 : 0;
      float ref = -1e30f, l = 0.f;
      unsigned poison = 0;
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        if (!mbar_wait_warp(s_full + half, (it + j) & 1, p.c.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int k0 = (cur.k0 + j) * kStepTok;
        const uint4 fl = *reinterpret_cast<const uint4*>(flags_s + ((it + j) & 3) * 4);
        const unsigned flags = fl.x | fl.y | fl.z | fl.w;     // bits 0-7: tiles without a page, bit 8: poison
        // weight of token j of the step, in the row's reach or not
        const int from = max(0, lo - k0), to_ = min(kStepTok - 1, hi - k0);   // tokens of the step that the row sees
        const bool part = from > 0 || to_ < kStepTok - 1 || (flags & 0xffu);
        const bool masked = __any_sync(0xffffffffu, part);
        uint32_t x[32];
        float top = -INFINITY;
        auto mask32 = [&](int c0) -> uint32_t {   // visible tokens among [c0, c0 + 32)
          const int a = max(from - c0, 0), z = min(to_ - c0, 31);
          uint32_t m = a <= z ? (0xffffffffu >> (31 - z)) & (0xffffffffu << a) : 0u;
          const unsigned gone = (flags >> (c0 / kTileTok)) & 3u;
          if (gone & 1u) m &= 0xffff0000u;
          if (gone & 2u) m &= 0x0000ffffu;
          return m;
        };
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_ld32(ts + q * 32, x);
          tmem_wait_ld();
          if (masked) {
            const uint32_t m = mask32(q * 32);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float y = __fmul_rn(__uint_as_float(x[i]), f);
              top = fmaxf(top, (m >> i) & 1u ? y : -INFINITY);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) top = fmaxf(top, __fmul_rn(__uint_as_float(x[i]), f));
          }
        }
        const bool grow = top > ref + (kHead + kGrow);
        if (__any_sync(0xffffffffu, grow)) {
          const float next = grow ? top - kHead : ref;
          const float shrink = grow ? fast_exp2(ref - next) : 1.f;
          ref = next;
          l *= shrink;
          if (j > 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tmem_ld32(to + q * 32, x);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * shrink);
              tmem_st32(to + q * 32, x);
            }
            tmem_wait_st();
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_ld32(ts + q * 32, x);
          tmem_wait_ld();
          const uint32_t m = masked ? mask32(q * 32) : 0xffffffffu;
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float y0 = fast_exp2(__fsub_rn(__fmul_rn(__uint_as_float(x[2 * i]), f), ref));
            float y1 = fast_exp2(__fsub_rn(__fmul_rn(__uint_as_float(x[2 * i + 1]), f), ref));
            if (masked) {
              y0 = (m >> (2 * i)) & 1u ? y0 : 0.f;
              y1 = (m >> (2 * i + 1)) & 1u ? y1 : 0.f;
            }
            l += y0 + y1;
            w[i] = pack_f16x2(y0, y1);
          }
          tmem_st16(ts + q * 16, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + half);
        if (flags & 0x100u) {   // values that are not finite, in blocks of 16 dims that the row sees
          const uint32_t* words = poison_s + ((it + j) & 3) * 32;
#pragma unroll 1
          for (int gr = 0; gr < 8; ++gr) {
            uint32_t seen = 0;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) seen |= words[gr * 4 + q] & mask32(q * 32);
            if (seen) poison |= 1u << gr;
          }
        }
      }
      if (ok && !mbar_wait_warp(o_full, segments & 1, p.c.err)) ok = false;
      if (ok) {
        tc_fence_after();
        const bool whole = cur.open == 3;
        const float inv = l == 0.f ? 0.f : __frcp_rn(l);
        float* slot = p.parts + static_cast<size_t>(cur.slot) * kSlot;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t x[32];
          tmem_ld32(to + q * 32, x);
          tmem_wait_ld();
          const float a0 = (poison >> (2 * q)) & 1u ? __int_as_float(0x7fffffff) : 0.f;
          const float a1 = (poison >> (2 * q + 1)) & 1u ? __int_as_float(0x7fffffff) : 0.f;
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(x[i]) * (whole ? inv : 1.f) + (i < 16 ? a0 : a1);
          if (!real) continue;
          if (whole) {
            write_row<T>(p, cur.r0, cur.h, cur.row0 + row, q * 32, y);
          } else {
            float4* at = reinterpret_cast<float4*>(slot + 2 * kRows + row * kD + q * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) at[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
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
        tc_fence_before();   // O has been read: the next segment's MMAs may overwrite it
      } else if (lane == 0) {
        failed = 1;
      }
    } else if (warp < 16) {
      // ================= keys (warps 8-11) and values (12-15) =================
      const bool keys = warp < 12;
      const int w = warp & 3;                    // tiles 2w, 2w + 1 of a step
      const int r = lane >> 2, t = lane & 3;
      uint64_t* full = keys ? k_full : v_full;
      uint64_t* empty = keys ? k_empty : v_empty;
      const int last_tile = (cur.T - 1) / kTileTok;
      int where = -1;                            // lane: cache tile of tile 32 * batch + lane of the segment
      uint4 code[2][2];
      uint2 sc[2];
      unsigned gone = 0;                         // bits: tiles 2w, 2w + 1 of the loaded step without a page
      auto load = [&](int j) {
        if ((j & 3) == 0) {
          const int tl = (cur.k0 + j) * kStepTiles + lane;
          where = -1;
          if (tl <= last_tile && tl < cur.k1 * kStepTiles) {
            const int page = kv4_page(p.c, cur.b, tl);
            if (page >= 0) where = static_cast<int>(kv4_tile_index(p.c, page, cur.h, tl));
          }
        }
        gone = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int at = __shfl_sync(0xffffffffu, where, (j & 3) * kStepTiles + 2 * w + u);
          if (at >= 0) {
            const uint8_t* tile = p.c.cache + static_cast<size_t>(static_cast<uint32_t>(at)) * kTileBytes;
            const uint4* src = reinterpret_cast<const uint4*>(tile + (keys ? 0 : kOffV)) + lane;
            code[u][0] = __ldg(src);
            code[u][1] = __ldg(src + 32);
            sc[u] = __ldg(reinterpret_cast<const uint2*>(tile + kOffScale) + lane);
          } else {
            gone |= 1u << u;
            code[u][0] = code[u][1] = make_uint4(0u, 0u, 0u, 0u);
            sc[u] = make_uint2(0u, 0u);
          }
        }
      };
      bool ok = true;
      load(0);
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        const int stage = (it + j) & 1;
        uint4 now[2][2] = {{code[0][0], code[0][1]}, {code[1][0], code[1][1]}};
        const uint2 scale[2] = {sc[0], sc[1]};
        const unsigned lost = gone;
        if (j + 1 < steps) load(j + 1);
        if (!mbar_wait_warp(empty + stage, (((it + j) >> 1) & 1) ^ 1, p.c.err)) {
          ok = false;
          break;
        }
        uint8_t* dst = sm + (keys ? Smem::k : Smem::v) + stage * kOperand;
        const int left = cur.T - (cur.k0 + j) * kStepTok;   // tokens from the step's first on
        if (keys) {
          // word i of a row's 16 bytes is dims 32 t + 8 i ..: one 16-byte piece. Lanes with t >= 2 start at word 2:
          // the eight lanes that store together then meet eight different pieces of the banks.
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int row = (2 * w + u) * kTileTok + half * 8 + r;
              const uint32_t cw[4] = {now[u][half].x, now[u][half].y, now[u][half].z, now[u][half].w};
              const uint32_t sa = scale_both(scale[u].x, 2 * half), sb = scale_both(scale[u].x, 2 * half + 1);
              uint8_t* base = dst + (t >> 1) * kHalfOp + row * 128;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t word = t & 2 ? cw[i ^ 2] : cw[i];
                const uint32_t s1 = ((i & 2) != 0) != ((t & 2) != 0) ? sb : sa;
                const int piece = (t & 1) * 4 + (i ^ (t & 2));
                uint32_t x[4];
                e2m1_to_f16x2(word, x[0], x[1], x[2], x[3]);
                *reinterpret_cast<uint4*>(base + ((piece ^ (row & 7)) << 4)) =
                    make_uint4(hmul2(x[0], s1), hmul2(x[1], s1), hmul2(x[2], s1), hmul2(x[3], s1));
              }
            }
          }
          // what the softmax has to know of the step
          unsigned info_bits = lost << (2 * w);
          unsigned bad = 0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t y = scale[u].y;   // values' scales: bytes 248 and up are not finite
            bad |= y & (y << 1) & (y << 2) & (y << 3) & (y << 4) & 0x80808080u;
          }
          if (__any_sync(0xffffffffu, bad != 0u)) {
            uint32_t word = 0;               // group r: bit = token of this warp's 32
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (((scale[u].y >> (8 * i)) & 0xffu) >= 248u) word |= 1u << (16 * u + 8 * (i >> 1) + 2 * t + (i & 1));
            word |= __shfl_xor_sync(0xffffffffu, word, 1);
            word |= __shfl_xor_sync(0xffffffffu, word, 2);
            if (t == 0) poison_s[((it + j) & 3) * 32 + r * 4 + w] = word;
            info_bits |= 0x100u;
          } else if (t == 0) {
            poison_s[((it + j) & 3) * 32 + r * 4 + w] = 0u;
          }
          if (lane == 0) flags_s[((it + j) & 3) * 4 + w] = info_bits;
        } else {
          // the two tokens of a byte part ways; lanes of odd r store the odd token first, against bank conflicts
          const uint32_t sel0 = r & 1 ? 0x7632u : 0x5410u, sel1 = r & 1 ? 0x5410u : 0x7632u;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int tok = (2 * w + u) * kTileTok + half * 8 + 2 * t;
              uint32_t s2 = scale_pair(scale[u].y, 2 * half);
              if ((s2 & 0x7c00u) == 0x7c00u || tok >= left) s2 &= 0xffff0000u;         // not finite, or past the end
              if ((s2 & 0x7c000000u) == 0x7c000000u || tok + 1 >= left) s2 &= 0x0000ffffu;
              const uint32_t cw[4] = {now[u][half].x, now[u][half].y, now[u][half].z, now[u][half].w};
              uint32_t x[16];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                e2m1_to_f16x2(cw[i], x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
#pragma unroll
                for (int q = 0; q < 4; ++q) x[4 * i + q] = hmul2(x[4 * i + q], s2);
              }
              uint8_t* base = dst + (r >> 2) * kHalfOp;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int row = tok + (e ^ (r & 1));
                const uint32_t sel = e ? sel1 : sel0;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const int piece = (r & 3) * 2 + q;
                  *reinterpret_cast<uint4*>(base + row * 128 + ((piece ^ (row & 7)) << 4)) =
                      make_uint4(__byte_perm(x[8 * q], x[8 * q + 1], sel), __byte_perm(x[8 * q + 2], x[8 * q + 3], sel),
                                 __byte_perm(x[8 * q + 4], x[8 * q + 5], sel), __byte_perm(x[8 * q + 6], x[8 * q + 7], sel));
                }
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + stage);
      }
      if (!ok && lane == 0) failed = 1;
    } else if (lane == 0) {
      // ================= MMAs =================
      const uint32_t q_addr = smem_addr(sm + Smem::q);
      bool ok = true;
      auto qk = [&](int half, int stage) {
        const uint32_t a = q_addr + half * kOperand, bk = smem_addr(sm + Smem::k) + stage * kOperand;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kHalfOp + (kk & 3) * 32;
          mma_ss(tmem + half * 128, desc_k_major(a + off), desc_k_major(bk + off), kk > 0 ? 1u : 0u);
        }
      };
      auto pv = [&](int half, int stage, bool first) {
        const uint32_t bv = smem_addr(sm + Smem::v) + stage * kOperand;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + half * 128, tmem + half * 128 + kk * 8, desc_mn_major(bv + kk * 2048),
                 first && kk == 0 ? 0u : 1u);
      };
#pragma unroll 1
      for (int j = 0; ok && j <= steps; ++j) {
        const int i = it + j;                      // step j's scores, step j - 1's products with the values
        const int sk = i & 1, sv = (i - 1) & 1;
        if (j < steps) {
          ok = mbar_wait(k_full + sk, (i >> 1) & 1, p.c.err);
        }
        if (ok && j > 0) ok = mbar_wait(v_full + sv, ((i - 1) >> 1) & 1, p.c.err);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (ok && j > 0) {
            ok = mbar_wait(p_full + half, (i - 1) & 1, p.c.err);
            tc_fence_after();
            if (ok) pv(half, sv, j == 1);
          }
          if (!ok) break;
          if (half == 1 && j > 0) tc_commit(v_empty + sv);
          if (j < steps) {
            tc_fence_after();
            qk(half, sk);
            tc_commit(s_full + half);
          }
        }
        if (ok && j < steps) tc_commit(k_empty + sk);
      }
      if (ok) tc_commit(o_full);
      else failed = 1;
    }
    it += steps;
    __syncwarp();
    __syncthreads();
    tc_fence_after();
  }

  if (warp == 16 && lane == 0) {
    tc_commit(drained);
    mbar_wait(drained, 0, p.c.err);   // nothing of ours still writes TMEM
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
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

// Joins the partials of the unit that begins in block blockIdx.x and goes on in the next ones; a warp a row.
template <typename T>
__global__ void __launch_bounds__(256) kv4_prefill_merge_kernel(const __grid_constant__ Kv4AttendParams p, int blocks) {
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
  const int row = blockIdx.y * 8 + warp;
  if (row >= u.rows) return;
  int parts = 1;
  while (c + parts < blocks && !info[2 * (c + parts)].ends) ++parts;
  ++parts;   // the one that ends it
  float m = -1e30f, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = 0; i < parts; ++i) {
    const float* slot = p.parts + static_cast<size_t>(i == 0 ? s0 : 2 * (c + i)) * kSlot;
    const float mi = slot[row], li = slot[kRows + row];
    const float4 v = *reinterpret_cast<const float4*>(slot + 2 * kRows + row * kD + lane * 4);
    const float next = fmaxf(m, mi);
    const float x = fast_exp2(m - next), y = fast_exp2(mi - next);
    m = next;
    l = fmaf(l, x, li * y);
    acc.x = fmaf(acc.x, x, v.x * y);
    acc.y = fmaf(acc.y, x, v.y * y);
    acc.z = fmaf(acc.z, x, v.z * y);
    acc.w = fmaf(acc.w, x, v.w * y);
  }
  const float inv = l == 0.f ? 0.f : __frcp_rn(l);
  const int i = token_of(p, u.row0 + row);
  const size_t at = (static_cast<size_t>(u.r0) + i) * p.c.Hq + static_cast<size_t>(u.h) * p.G + (u.row0 + row - i * p.G);
  reinterpret_cast<uint2*>(p.out)[at * (kD / 4) + lane] =
      make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
  if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
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
  cfg.gridDim = dim3(blocks, kRows / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv4_prefill_merge_kernel<T>, p, blocks);
}

}  // namespace

size_t kv4_prefill_part_bytes() {
  return static_cast<size_t>(2 * kKv4MaxSms) * (kSlot * sizeof(float) + sizeof(SlotInfo));
}

cudaError_t launch_kv4_prefill(int dtype, const Kv4AttendParams& p, int sms, cudaStream_t stream, bool pdl) {
  if (dtype == HSA_BF16) return launch_prefill_t<__nv_bfloat16>(p, sms, stream, pdl);
  if (dtype == HSA_F16) return launch_prefill_t<__half>(p, sms, stream, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace pqhsa
