// Attention over the 4-bit KV cache for few query rows a KV head (decode, verification of
// drafted tokens): every warp streams tiles through registers and keeps its rows' online
// softmax state to the end of its share.
//
// Work. A unit is (sequence, KV head, tile of query rows); its tokens are steps of two
// 16-token tiles. All units' steps lie on one line, in the order of (sequence, head, row
// tile). Every block takes an equal share of that line and every warp of it an equal share
// of that, so long and short sequences load all warps alike and no barrier stands between
// two units. A warp works through its share unit by unit (a segment each). Units that lie
// within one warp's share are finished there. Of the others a warp has at most two, its
// first and its last: the first goes to a slot in the workspace, the last to shared memory,
// and after the block's only barrier its warps join them. Units that cross blocks leave one
// partial (m, l, acc) a block, and the merge kernel joins those. Shares follow from the
// device lengths alone.
//
// Mathematics of a tile, on mma.sync m16n8k16 (fp16 in, fp32 sums): S^T = K q^T with the 16
// tokens as rows and 8 query rows as columns, P = 2^(S f - ref), O^T += V^T P with dims as
// rows. Keys and values are code x scale, exact in fp16, made in registers straight from the
// tile's bytes: its layout is the fragments' own. q is scaled to at most 1 by a power of
// two (f carries it back); 16-bit q is then one fp16 number, 32-bit q two (hi + lo, 22 bits),
// and P likewise, so that 32-bit calls keep 32-bit accuracy. With at most four 32-bit rows hi
// and lo share one fragment (columns 0-3 and 4-7).
//
// ref is the row's largest logit so far less kHead; it moves when a logit exceeds it by
// kHead + kGrow, so P <= 2^(kHead + kGrow) < 65504, and a weight below 2^(-24 - kHead) of the
// largest is lost.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4.cuh"

namespace pqhsa {
namespace {

constexpr int kStep = 2;            // tiles a step
constexpr int kStepTok = kStep * kTileTok;
constexpr int kStepBytes = kStep * kTileBytes;
constexpr float kHead = 11.f, kGrow = 4.f;
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kPitch = kD + 4;      // floats a row of a warp's partial in shared memory

enum Mode { kHi, kHiLo, kPack };

template <int NR, Mode M>
struct Shape {
  static constexpr int RT = M == kPack ? 4 : 8 * NR;             // query rows of a unit
  static constexpr int QF = NR * (M == kHiLo ? 2 : 1);           // q fragments
  static constexpr bool q_smem = NR > 1;                         // in shared memory, a set a warp
  static constexpr int warps = NR == 1 ? 16 : 8;                 // one block an SM: 128 or 255 registers a thread
  static constexpr int stages = NR == 1 ? 3 : 4;
  static constexpr size_t ring = static_cast<size_t>(stages) * kStepBytes;      // a warp's
  static constexpr size_t part = static_cast<size_t>(RT) * (kPitch + 2) * sizeof(float);
  static_assert(part <= ring, "a warp's last partial lies over its ring");
  static constexpr size_t qbytes = q_smem ? static_cast<size_t>(QF) * 8 * 32 * 8 : 0;
  static constexpr size_t total = warps * (ring + qbytes);
  static_assert(total + 2048 <= 227 * 1024, "shared memory of a block");
  static_assert(2 * warps <= 32, "a lane for each segment that is joined");
};

__device__ __forceinline__ void mma_f16_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }

// ---- shares of the line of steps ---------------------------------------------

struct Seq {
  int T, n, r0;          // tokens, query tokens, first query token's row
  int lo, nt, nrt;       // first step, steps, row tiles
  long long count;       // steps on the line
};

__device__ __forceinline__ Seq sequence(const Kv4AttendParams& p, int b, int RT) {
  Seq s;
  s.T = kv4_len(p.c, b);
  s.r0 = p.cu ? p.cu[b] : b;
  s.n = p.cu ? p.cu[b + 1] - s.r0 : 1;
  s.n = max(0, min(s.n, p.n_rows - s.r0));
  if (s.r0 < 0) s.n = 0;
  const long long first = static_cast<long long>(s.T) - s.n - p.window + 1;   // leftmost position of a window
  s.lo = p.window > 0 && first > 0 ? static_cast<int>(first / kStepTok) : 0;
  const int hi = (s.T + kStepTok - 1) / kStepTok;
  s.nt = s.n > 0 ? hi - s.lo : 0;
  s.nrt = (s.n * p.G + RT - 1) / RT;
  s.count = static_cast<long long>(s.nt) * s.nrt * p.c.Hkv;
  return s;
}

// Query token and head of the group of a query row; p.inv_G = ceil(2^32 / G), exact for rows below 2^25.
__device__ __forceinline__ int token_of(const Kv4AttendParams& p, int row) {
  return p.G == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.inv_G));
}
__device__ __forceinline__ size_t head_row(const Kv4AttendParams& p, int r0, int h, int qrow) {
  const int i = token_of(p, qrow);
  return (static_cast<size_t>(r0) + i) * p.c.Hq + static_cast<size_t>(h) * p.G + (qrow - i * p.G);
}

// Quotient of numbers that hardly ever need 64 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The line of all steps and its equal shares: the first `rest` blocks take one step more.
struct Line {
  long long W, each, rest;
  int N;
  __device__ __forceinline__ Line(long long w, int blocks) : W(w) {
    N = static_cast<int>(min(static_cast<long long>(blocks), w));
    each = N > 0 ? quotient(w, N) : 0;
    rest = w - each * N;
  }
  __device__ __forceinline__ long long begin(int c) const { return each * c + min(static_cast<long long>(c), rest); }
  __device__ __forceinline__ int block_of(long long g) const {
    const long long big = rest * (each + 1);
    return static_cast<int>(g < big ? quotient(g, each + 1) : rest + quotient(g - big, each));
  }
};

// Inclusive sum over the lanes of a warp.
__device__ __forceinline__ long long lane_sums(long long n) {
  const int lane = threadIdx.x & 31;
  if (__all_sync(0xffffffffu, n < (1 << 26))) {
    int x = static_cast<int>(n);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) n += y;
  }
  return n;
}

// Steps of all sequences, and of those before sequence b, by a whole warp.
__device__ __forceinline__ long long line_length(const Kv4AttendParams& p, int RT, int b, long long* before) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  *before = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    const long long n = b0 + lane < p.c.B ? sequence(p, b0 + lane, RT).count : 0;
    const long long x = lane_sums(n);
    if (b >= b0 && b < b0 + 32) *before = base + __shfl_sync(0xffffffffu, x - n, b - b0);
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  return base;
}

// Sequence that holds step g of the line and the steps before it, by a whole warp.
__device__ __forceinline__ int locate(const Kv4AttendParams& p, int RT, long long g, long long* before) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    const long long n = b0 + lane < p.c.B ? sequence(p, b0 + lane, RT).count : 0;
    const long long x = lane_sums(n);
    const unsigned past = __ballot_sync(0xffffffffu, base + x > g);
    if (past) {
      const int l = __ffs(past) - 1;
      *before = base + __shfl_sync(0xffffffffu, x - n, l);
      return b0 + l;
    }
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  *before = base;
  return p.c.B;
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

template <typename T>
__device__ __forceinline__ void store_out(uint8_t* out, size_t at, float4 v);
template <>
__device__ __forceinline__ void store_out<float>(uint8_t* out, size_t at, float4 v) {
  reinterpret_cast<float4*>(out)[at / 4] = v;
}
template <>
__device__ __forceinline__ void store_out<__nv_bfloat16>(uint8_t* out, size_t at, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  reinterpret_cast<uint2*>(out)[at / 4] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
template <>
__device__ __forceinline__ void store_out<__half>(uint8_t* out, size_t at, float4 v) {
  reinterpret_cast<uint2*>(out)[at / 4] = make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
}

// Result of one row's four dims: acc / l, zeros for a row whose mask left nothing.
template <typename T>
__device__ __forceinline__ void finish(const Kv4AttendParams& p, size_t head_row, int d4, float m, float l, float4 a) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  a.x *= inv;
  a.y *= inv;
  a.z *= inv;
  a.w *= inv;
  store_out<T>(p.out, head_row * kD + d4 * 4, a);
  if (p.lse && d4 == 0) p.lse[head_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// 32 consecutive values of q (one row, 32 dims) as fp32.
template <typename T>
__device__ __forceinline__ void load_q32(const uint8_t* row, float* x);
template <>
__device__ __forceinline__ void load_q32<float>(const uint8_t* row, float* x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 v = reinterpret_cast<const float4*>(row)[i];
    x[4 * i] = v.x;
    x[4 * i + 1] = v.y;
    x[4 * i + 2] = v.z;
    x[4 * i + 3] = v.w;
  }
}
template <>
__device__ __forceinline__ void load_q32<__nv_bfloat16>(const uint8_t* row, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(row)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = bf16lo(w[j]);
      x[8 * i + 2 * j + 1] = bf16hi(w[j]);
    }
  }
}
template <>
__device__ __forceinline__ void load_q32<__half>(const uint8_t* row, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(row)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_f16x2(w[j]);
      x[8 * i + 2 * j] = f.x;
      x[8 * i + 2 * j + 1] = f.y;
    }
  }
}

// A segment that is joined with others of its unit.
struct Segment {
  int unit, b;           // unit: row tile and head, -1: none
  int h, r0, row0, rows; // head, first query token's row, first and number of query rows
  int open;              // bits: begins at its unit's first step, ends at its last, begins the block
};

template <typename T, int NR, Mode M>
__global__ void __launch_bounds__(Shape<NR, M>::warps * 32, 1) kv4_attend_kernel(Kv4AttendParams p) {
  using S = Shape<NR, M>;
  constexpr int RT = S::RT;
  constexpr int kWarps = S::warps;
  constexpr int kSlot = RT * (kD + 2);             // floats of a slot in the workspace
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Segment segs[2 * kWarps];             // a warp's first and last
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * S::ring;
  uint2* qs = reinterpret_cast<uint2*>(smem + kWarps * S::ring + warp * S::qbytes);   // [fragment][8][lane]
  if (lane < 2) segs[2 * warp + lane].unit = -1;
  __syncwarp();

  pdl_wait();
  pdl_launch_dependents();

  // ---- this block's and this warp's share of the line ----
  Seq s = {};
  long long before = 0, W, sums = 0;
  const bool few = p.c.B <= 32;                    // one sequence a lane, read once
  if (few) {
    if (lane < p.c.B) s = sequence(p, lane, RT);
    sums = lane_sums(s.count);
    W = __shfl_sync(0xffffffffu, sums, 31);
  } else {
    W = line_length(p, RT, 0, &before);
  }
  const Line line(W, gridDim.x);
  if (static_cast<int>(blockIdx.x) >= line.N) return;
  const long long block_g = line.begin(blockIdx.x);
  const int block_len = static_cast<int>(line.begin(blockIdx.x + 1) - block_g);
  long long g = block_g + static_cast<long long>(block_len) * warp / kWarps;
  const long long g_end = block_g + static_cast<long long>(block_len) * (warp + 1) / kWarps;
  float* first_slot = p.parts + static_cast<size_t>(2 * gridDim.x + blockIdx.x * kWarps + warp) * kSlot;

  if (g < g_end) {
    int b;
    if (few) {
      b = __ffs(__ballot_sync(0xffffffffu, sums > g)) - 1;
      before = __shfl_sync(0xffffffffu, sums - s.count, b);
      s.T = __shfl_sync(0xffffffffu, s.T, b);
      s.n = __shfl_sync(0xffffffffu, s.n, b);
      s.r0 = __shfl_sync(0xffffffffu, s.r0, b);
      s.lo = __shfl_sync(0xffffffffu, s.lo, b);
      s.nt = __shfl_sync(0xffffffffu, s.nt, b);
      s.nrt = __shfl_sync(0xffffffffu, s.nrt, b);
      s.count = __shfl_sync(0xffffffffu, s.count, b);
    } else {
      b = locate(p, RT, g, &before);
      s = sequence(p, b, RT);
    }
    while (g < g_end && b < p.c.B) {
      if (g - before >= s.count) {   // next sequence with work
        before += s.count;
        if (++b < p.c.B) s = sequence(p, b, RT);
        continue;
      }
      const long long in_seq = g - before;
      const int unit = static_cast<int>(quotient(in_seq, s.nt));                    // h * nrt + row tile
      const int a = static_cast<int>(in_seq - static_cast<long long>(unit) * s.nt); // first step of the segment
      const int len = static_cast<int>(min(static_cast<long long>(s.nt - a), g_end - g));
      const int h = s.nrt == 1 ? unit : unit / s.nrt, rt = unit - h * s.nrt;
      const int row0 = rt * RT;
      const int rows = min(RT, s.n * p.G - row0);                // valid query rows

      // ---- copies: stages - 1 steps ahead, tile numbers 16 steps ahead ----
      const int tile0 = (s.lo + a) * kStep;
      const int last_tile = (s.T - 1) / kTileTok;
      int where = -1;               // lane: tile of the cache that holds tile0 + 32 * batch + lane
      unsigned missing = 0;         // two bits a stage: its tiles that have no page, or lie past the end
      auto issue = [&](int i) {
        if (i < len) {
          if ((i & 15) == 0) {
            const int tl = tile0 + i * kStep + lane;
            where = -1;
            if (tl < tile0 + len * kStep && tl <= last_tile) {
              const int page = kv4_page(p.c, b, tl);
              if (page >= 0) where = static_cast<int>(kv4_tile_index(p.c, page, h, tl));
            }
          }
          const int st = i % S::stages;
          missing &= ~(3u << (2 * st));
#pragma unroll
          for (int u = 0; u < kStep; ++u) {
            const int w = __shfl_sync(0xffffffffu, where, (i * kStep + u) & 31);
            if (w >= 0) {
              const uint8_t* src = p.c.cache + static_cast<size_t>(static_cast<uint32_t>(w)) * kTileBytes + lane * 16;
              uint8_t* dst = ring + st * kStepBytes + u * kTileBytes + lane * 16;
#pragma unroll
              for (int j = 0; j < 4; ++j) cp_async_16(dst + j * 512, src + j * 512);
              if (lane < 16) cp_async_16(dst + kOffScale, src + kOffScale);
            } else {
              missing |= 1u << (2 * st + u);
            }
          }
        }
        cp_async_commit();
      };
      __syncwarp();
#pragma unroll
      for (int i = 0; i < S::stages - 1; ++i) issue(i);

      // ---- query fragments and the bounds of each of this lane's columns ----
      uint32_t qf[S::q_smem ? 1 : S::QF][16];
      float f[2 * NR];
      int hi[2 * NR], lo[2 * NR];
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
        const int col = M == kPack ? (r & 3) : nt * 8 + r;
        float x[32];
        float top = 0.f;
        if (col < rows) {
          const int i = token_of(p, row0 + col);
          load_q32<T>(p.q + (static_cast<long long>(s.r0) + i) * p.q_tok +
                          (static_cast<size_t>(h) * p.G + (row0 + col - i * p.G)) * kD * sizeof(T) + t * 32 * sizeof(T),
                      x);
#pragma unroll
          for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[i]));
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e > top >= 2^(e - 1) for normal numbers; out of range or not finite: as it is
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 126;
        e = e > 126 ? 0 : max(e, -126);
        const float down = pow2i(-e);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x0 = x[2 * i] * down, x1 = x[2 * i + 1] * down;
          const uint32_t hi2 = pack_f16x2(x0, x1);
          uint32_t lo2 = 0u;
          if (M != kHi) {
            const float2 back = unpack_f16x2(hi2);
            lo2 = pack_f16x2(x0 - back.x, x1 - back.y);
          }
          const uint32_t v = M == kPack && r >= 4 ? lo2 : hi2;
          if (S::q_smem) {
            reinterpret_cast<uint32_t*>(qs + ((M == kHiLo ? 2 * nt : nt) * 8 + i / 2) * 32 + lane)[i & 1] = v;
            if (M == kHiLo) reinterpret_cast<uint32_t*>(qs + ((2 * nt + 1) * 8 + i / 2) * 32 + lane)[i & 1] = lo2;
          } else {
            qf[0][i] = v;
            if (M == kHiLo) qf[S::QF - 1][i] = lo2;
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int mine = M == kPack ? ((2 * t + j) & 3) : 2 * t + j;
          const int ec = __shfl_sync(0xffffffffu, e, 4 * mine);
          const int c = nt * 8 + mine;
          // never so small that a masked logit, -inf times f, is NaN; logits under 2^-80 are as good as 0
          const float fc = p.scale * kLog2e * pow2i(ec);
          f[2 * nt + j] = fabsf(fc) < 1e-36f ? copysignf(1e-36f, fc) : fc;
          const int pos = s.T - s.n + token_of(p, row0 + c);
          hi[2 * nt + j] = c >= rows ? -1 : p.causal ? pos : s.T - 1;
          lo[2 * nt + j] = p.window > 0 ? pos - p.window + 1 : 0;
        }
      }
      // positions that every row of the unit sees
      const int all_hi = p.causal ? s.T - s.n + token_of(p, row0) : s.T - 1;
      const int all_lo = p.window > 0 ? s.T - s.n + token_of(p, row0 + rows - 1) - p.window + 1 : 0;

      float o[NR][8][4];
      float ref[2 * NR], l[2 * NR];
#pragma unroll
      for (int j = 0; j < 2 * NR; ++j) {
        ref[j] = -1e30f;
        l[j] = 0.f;
      }
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;

#pragma unroll 1
      for (int i = 0; i < len; ++i) {
        cp_async_wait<S::stages - 2>();
        __syncwarp();
        const int st = i % S::stages;
        const unsigned absent = (missing >> (2 * st)) & 3u;
        issue(i + S::stages - 1);
        const uint8_t* stage = ring + st * kStepBytes;
        const int pos = (tile0 + i * kStep) * kTileTok;
        // ---- S^T = K q^T ----
        float sacc[kStep][NR][4];
        uint2 sc[kStep];
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const uint8_t* tile = stage + u * kTileBytes;
          const uint4 k0 = reinterpret_cast<const uint4*>(tile)[lane];
          const uint4 k1 = reinterpret_cast<const uint4*>(tile + 512)[lane];
          sc[u] = reinterpret_cast<const uint2*>(tile + kOffScale)[lane];
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) sacc[u][nt][j] = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t x[4], y[4];
            e2m1_to_f16x2(w0[w], x[0], x[1], x[2], x[3]);
            e2m1_to_f16x2(w1[w], y[0], y[1], y[2], y[3]);
            const uint32_t s0 = scale_both(sc[u].x, w >> 1), s1 = scale_both(sc[u].x, 2 + (w >> 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[j] = hmul2(x[j], s0);
              y[j] = hmul2(y[j], s1);
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              const int i8 = 2 * w + kk;
#pragma unroll
              for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
                for (int part_q = 0; part_q < (M == kHiLo ? 2 : 1); ++part_q) {
                  const int fr = M == kHiLo ? 2 * nt + part_q : nt;
                  uint2 bq;
                  if (S::q_smem) bq = qs[(fr * 8 + i8) * 32 + lane];
                  else bq = make_uint2(qf[S::q_smem ? 0 : fr][2 * i8], qf[S::q_smem ? 0 : fr][2 * i8 + 1]);
                  mma_f16_16816(sacc[u][nt], x[2 * kk], y[2 * kk], x[2 * kk + 1], y[2 * kk + 1], bq.x, bq.y);
                }
              }
            }
          }
          if (M == kPack) {
#pragma unroll
            for (int j = 0; j < 4; ++j) sacc[u][0][j] += __shfl_xor_sync(0xffffffffu, sacc[u][0][j], 2);
          }
        }
        // ---- masks ----
        uint32_t vs[kStep][2];
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          vs[u][0] = scale_pair(sc[u].y, 0);
          vs[u][1] = scale_pair(sc[u].y, 2);
        }
        const bool whole = absent == 0u && pos + kStepTok - 1 <= all_hi && pos >= all_lo;
        if (!whole) {
#pragma unroll
          for (int u = 0; u < kStep; ++u) {
            const int pu = pos + u * kTileTok;
            const bool present = !((absent >> u) & 1u);
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int tp = pu + r + 8 * (j >> 1), c = 2 * nt + (j & 1);
                // times f it is -inf, whatever f's sign
                if (tp > hi[c] || tp < lo[c] || !present) sacc[u][nt][j] = f[c] < 0.f ? INFINITY : -INFINITY;
              }
            // A zero weight must not meet a NaN or an infinity: tokens past the end hold anything.
            const int left = present ? s.T - (pu + 2 * t) : 0;   // tokens from this lane's first on
            vs[u][0] &= (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
            vs[u][1] &= (left > 8 ? 0xffffu : 0u) | (left > 9 ? 0xffff0000u : 0u);
            // Values that are not finite count for the rows that see their token, and for no other:
            // taken out of the product, and added as NaN to those rows' sums of the block's dims.
            const unsigned bad = ((vs[u][0] & 0x7c00u) == 0x7c00u ? 1u : 0u) |
                                 ((vs[u][0] & 0x7c000000u) == 0x7c000000u ? 2u : 0u) |
                                 ((vs[u][1] & 0x7c00u) == 0x7c00u ? 256u : 0u) |
                                 ((vs[u][1] & 0x7c000000u) == 0x7c000000u ? 512u : 0u);
            if (__any_sync(0xffffffffu, bad != 0u)) {
              vs[u][0] &= (bad & 1u ? 0u : 0xffffu) | (bad & 2u ? 0u : 0xffff0000u);
              vs[u][1] &= (bad & 256u ? 0u : 0xffffu) | (bad & 512u ? 0u : 0xffff0000u);
              unsigned all = bad << (2 * t);                       // bit: token of the tile
              all |= __shfl_xor_sync(0xffffffffu, all, 1);
              all |= __shfl_xor_sync(0xffffffffu, all, 2);
#pragma unroll
              for (int c = 0; c < 2 * NR; ++c) {
                const int from = max(0, lo[c] - pu), to = min(kTileTok - 1, hi[c] - pu);
                const bool seen = from <= to && (all & ((2u << to) - (1u << from))) != 0u;
#pragma unroll
                for (int i8 = 0; i8 < 8; ++i8) {
                  if (seen) o[c >> 1][i8][c & 1] = o[c >> 1][i8][(c & 1) + 2] = __int_as_float(0x7fffffff);
                }
              }
            }
          }
        }
        // ---- online softmax: weights 2^(s f - ref) ----
        float y[kStep][NR][4], top = -INFINITY;
#pragma unroll
        for (int u = 0; u < kStep; ++u)
#pragma unroll
          for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // rounded before ref is taken off: ref is made of rounded logits, and large ones must meet it
              sacc[u][nt][j] = __fmul_rn(sacc[u][nt][j], f[2 * nt + (j & 1)]);
              y[u][nt][j] = __fsub_rn(sacc[u][nt][j], ref[2 * nt + (j & 1)]);
              top = fmaxf(top, y[u][nt][j]);
            }
        if (__any_sync(0xffffffffu, top > kHead + kGrow)) {
#pragma unroll
          for (int c = 0; c < 2 * NR; ++c) {
            float mx = -INFINITY;
#pragma unroll
            for (int u = 0; u < kStep; ++u)
#pragma unroll
              for (int j = 0; j < 2; ++j) mx = fmaxf(mx, sacc[u][c >> 1][(c & 1) + 2 * j]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float next = fmaxf(ref[c], mx - kHead);
            const float shrink = fast_exp2(ref[c] - next);
            ref[c] = next;
            l[c] *= shrink;
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) {
              o[c >> 1][i8][c & 1] *= shrink;
              o[c >> 1][i8][(c & 1) + 2] *= shrink;
            }
#pragma unroll
            for (int u = 0; u < kStep; ++u)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                y[u][c >> 1][(c & 1) + 2 * j] = __fsub_rn(sacc[u][c >> 1][(c & 1) + 2 * j], next);
          }
        }
        // ---- O^T += V^T P ----
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          uint32_t ph[NR][2], pl[NR][2];
#pragma unroll
          for (int nt = 0; nt < NR; ++nt) {
            float pr[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int c = 2 * nt + (j & 1);
              pr[j] = fast_exp2(y[u][nt][j]);
              l[c] += pr[j];
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t hi2 = pack_f16x2(pr[2 * half], pr[2 * half + 1]);
              if (M != kHi) {
                const float2 back = unpack_f16x2(hi2);
                const uint32_t lo2 = pack_f16x2(pr[2 * half] - back.x, pr[2 * half + 1] - back.y);
                if (M == kPack) hi2 = t >= 2 ? lo2 : hi2;
                else pl[nt][half] = transpose8x8(lo2);
              }
              ph[nt][half] = transpose8x8(hi2);
            }
          }
          const uint8_t* tile = stage + u * kTileBytes + kOffV;
          const uint4 v0 = reinterpret_cast<const uint4*>(tile)[lane];
          const uint4 v1 = reinterpret_cast<const uint4*>(tile + 512)[lane];
          const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t x[4], y[4];
            e2m1_to_f16x2(w0[w], x[0], x[1], x[2], x[3]);
            e2m1_to_f16x2(w1[w], y[0], y[1], y[2], y[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[j] = hmul2(x[j], vs[u][0]);
              y[j] = hmul2(y[j], vs[u][1]);
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
              for (int nt = 0; nt < NR; ++nt) {
                mma_f16_16816(o[nt][2 * w + kk], x[2 * kk], x[2 * kk + 1], y[2 * kk], y[2 * kk + 1], ph[nt][0],
                              ph[nt][1]);
                if (M == kHiLo)
                  mma_f16_16816(o[nt][2 * w + kk], x[2 * kk], x[2 * kk + 1], y[2 * kk], y[2 * kk + 1], pl[nt][0],
                                pl[nt][1]);
              }
            }
          }
        }
      }
      cp_async_wait<0>();

      // ---- end of a segment: the result, or a partial to be joined ----
      const bool done = a == 0 && len == s.nt;
      const bool last = g + len >= g_end;
      float* slot = last ? reinterpret_cast<float*>(ring) : first_slot;
      const int pitch = last ? kPitch : kD;
      if (!done) __syncwarp();   // the ring has been read
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = 2 * nt + j;
          l[c] += __shfl_xor_sync(0xffffffffu, l[c], 4);
          l[c] += __shfl_xor_sync(0xffffffffu, l[c], 8);
          l[c] += __shfl_xor_sync(0xffffffffu, l[c], 16);
          float v[16];
#pragma unroll
          for (int i8 = 0; i8 < 8; ++i8) {
            v[2 * i8] = o[nt][i8][j];
            v[2 * i8 + 1] = o[nt][i8][j + 2];
          }
          if (M == kPack) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 2);
          }
          const int col = nt * 8 + 2 * t + j;
          if (col >= rows) continue;
          if (done) {
            const size_t at = head_row(p, s.r0, h, row0 + col);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              finish<T>(p, at, 4 * r + i, ref[c], l[c], make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
          } else {
            float* row = slot + 2 * RT + col * pitch + 16 * r;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<float4*>(row)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            if (r == 0) {
              slot[col] = ref[c];
              slot[RT + col] = l[c];
            }
          }
        }
      }
      if (!done && lane == 0) {
        segs[2 * warp + (last ? 1 : 0)] =
            Segment{unit, b, h, s.r0, row0, rows,
                    (a == 0 ? 1 : 0) | (a + len == s.nt ? 2 : 0) | (g == block_g ? 4 : 0)};
      }
      g += len;
    }
  }
  __syncthreads();

  // ---- join the warps' partials, unit by unit; a warp takes rows warp, warp + kWarps, ... ----
  for (int e = 0; e < 2 * kWarps;) {
    const Segment head = segs[e];
    if (head.unit < 0) {
      ++e;
      continue;
    }
    // lane i: whether segment i is one of this unit's (they stand together, but for gaps)
    const bool mine = lane < 2 * kWarps && lane >= e && segs[lane].unit == head.unit && segs[lane].b == head.b;
    const unsigned set = __ballot_sync(0xffffffffu, mine);
    const int final = 31 - __clz(set);
    const bool done = (head.open & 1) && (segs[final].open & 2);
    const float* slot = lane & 1 ? reinterpret_cast<const float*>(smem + (lane >> 1) * S::ring)
                                 : p.parts + static_cast<size_t>(2 * gridDim.x + blockIdx.x * kWarps + (lane >> 1)) * kSlot;
    float* out_slot = p.parts + static_cast<size_t>(2 * blockIdx.x + ((head.open & 5) == 1 ? 1 : 0)) * kSlot;
    for (int row = warp; row < head.rows; row += kWarps) {
      const float m1 = mine ? slot[row] : -INFINITY;
      const float l1 = mine ? slot[RT + row] : 0.f;
      const float m = warp_max(m1);
      const float w = mine ? fast_exp2(m1 - m) : 0.f;   // NaN where a row is NaN
      const float l = warp_sum(w * l1);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (unsigned left = set; left; left &= left - 1) {
        const int i = __ffs(left) - 1;
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float* si = i & 1 ? reinterpret_cast<const float*>(smem + (i >> 1) * S::ring) + row * kPitch
                                : p.parts + static_cast<size_t>(2 * gridDim.x + blockIdx.x * kWarps + (i >> 1)) * kSlot + row * kD;
        const float4 v = *reinterpret_cast<const float4*>(si + 2 * RT + lane * 4);
        acc.x = fmaf(wi, v.x, acc.x);
        acc.y = fmaf(wi, v.y, acc.y);
        acc.z = fmaf(wi, v.z, acc.z);
        acc.w = fmaf(wi, v.w, acc.w);
      }
      if (done) {
        finish<T>(p, head_row(p, head.r0, head.h, head.row0 + row), lane, m, l, acc);
      } else {
        if (lane == 0) {
          out_slot[row] = m;
          out_slot[RT + row] = l;
        }
        *reinterpret_cast<float4*>(out_slot + 2 * RT + row * kD + lane * 4) = acc;
      }
    }
    e = final + 1;
  }
}

// One block a query row of a unit: joins the partials of a unit that several blocks shared, and
// writes the rows of sequences without tokens.
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(Kv4AttendParams p, int RT, int blocks) {
  __shared__ float4 acc_s[kMergeWarps][32];
  __shared__ float max_s[kMergeWarps], sum_s[kMergeWarps];
  __shared__ float weight[kKv4MaxSms];
  static_assert(kKv4MaxSms <= kMergeThreads, "a thread for each part");
  // Lengths and row offsets may be read at once: the attention kernel lets this one start only after it has
  // itself waited for all that came before it.
  pdl_launch_dependents();
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Seq s = sequence(p, b, RT);
  const int rows_all = s.n * p.G;                       // query rows of a head
  const int h = blockIdx.x % p.c.Hkv;
  long long before = 0;
  const Line line(line_length(p, RT, b, &before), blocks);
  pdl_wait();
  for (int qrow = blockIdx.x / p.c.Hkv; qrow < rows_all; qrow += gridDim.x / p.c.Hkv) {
    const size_t at = head_row(p, s.r0, h, qrow);
    if (s.nt == 0) {
      if (warp == 0) finish<T>(p, at, lane, 0.f, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
      continue;
    }
    const int rt = qrow / RT, row = qrow % RT;
    const long long u0 = before + (static_cast<long long>(h) * s.nrt + rt) * s.nt;
    const int c0 = line.block_of(u0), c1 = line.block_of(u0 + s.nt - 1);
    if (c0 == c1) continue;
    const int late = line.begin(c0) == u0 ? 0 : 1;   // the unit is its first block's last segment
    const float* slots = p.parts + static_cast<size_t>(2 * c0) * RT * (kD + 2);
    const int parts = c1 - c0 + 1;                   // at most kKv4MaxSms
    auto slot_of = [&](int i) { return slots + static_cast<size_t>(2 * i + (i == 0 ? late : 0)) * RT * (kD + 2); };
    float mi = -INFINITY, li = 0.f;
    if (tid < parts) {
      mi = slot_of(tid)[row];
      li = slot_of(tid)[RT + row];
    }
    const float wm = warp_max(mi);
    if (lane == 0) max_s[warp] = wm;
    __syncthreads();
    float m = max_s[0];
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) m = fmaxf(m, max_s[w]);
    const float x = tid < parts ? fast_exp2(mi - m) : 0.f;
    if (tid < parts) weight[tid] = x;
    const float ls = warp_sum(x * li);
    if (lane == 0) sum_s[warp] = ls;
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 5
    for (int i = warp; i < parts; i += kMergeWarps) {
      const float4 v = *reinterpret_cast<const float4*>(slot_of(i) + 2 * RT + row * kD + lane * 4);
      const float y = weight[i];
      acc.x = fmaf(v.x, y, acc.x);
      acc.y = fmaf(v.y, y, acc.y);
      acc.z = fmaf(v.z, y, acc.z);
      acc.w = fmaf(v.w, y, acc.w);
    }
    acc_s[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
      float l = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float4 v = acc_s[w][lane];
        l += sum_s[w];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      finish<T>(p, at, lane, m, l, acc);
    }
    __syncthreads();
  }
}

cudaLaunchConfig_t launch_config(dim3 grid, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute* attr,
                                 bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T, int NR, Mode M>
cudaError_t launch_attend_t(const Kv4AttendParams& p, int sms, long long steps, long long units, int max_rows, cudaStream_t stream,
                            bool pdl) {
  using S = Shape<NR, M>;
  cudaError_t e = ensure_dyn_smem<kv4_attend_kernel<T, NR, M>>(S::total);
  if (e != cudaSuccess) return e;
  const long long most = std::min(sms, kKv4MaxSms);
  // a share of at least one step a warp, but of no more units than there are SMs for
  const int blocks = static_cast<int>(std::max(1ll, std::min(most, std::max(units, (steps + S::warps - 1) / S::warps))));
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = launch_config(dim3(blocks), S::warps * 32, S::total, stream, attr, pdl);
  e = cudaLaunchKernelEx(&cfg, kv4_attend_kernel<T, NR, M>, p);
  if (e != cudaSuccess) return e;
  cfg = launch_config(dim3(p.c.Hkv * std::max(1, max_rows), p.c.B), kMergeThreads, 0, stream, attr, pdl);
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel<T>, p, static_cast<int>(S::RT), blocks);
}

template <typename T>
cudaError_t launch_16(int rows, const Kv4AttendParams& p, int sms, long long steps, long long units, int max_rows, cudaStream_t stream,
                      bool pdl) {
  switch (rows) {
    case 8: return launch_attend_t<T, 1, kHi>(p, sms, steps, units, max_rows, stream, pdl);
    case 16: return launch_attend_t<T, 2, kHi>(p, sms, steps, units, max_rows, stream, pdl);
    case 32: return launch_attend_t<T, 4, kHi>(p, sms, steps, units, max_rows, stream, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int kv4_attend_step_tokens() { return kStepTok; }

int kv4_attend_rows(int dtype, int max_rows) {
  if (dtype == HSA_F32) return max_rows <= 4 ? 4 : max_rows <= 8 ? 8 : 16;
  return max_rows <= 8 ? 8 : max_rows <= 16 ? 16 : 32;
}

// Two slots a block and one a warp: of 8 rows with 16 warps, of up to 32 with 8.
size_t kv4_attend_part_bytes() {
  return static_cast<size_t>(2 + 8) * kKv4MaxSms * 32 * (kD + 2) * sizeof(float);
}

cudaError_t launch_kv4_attend(int dtype, int rows, const Kv4AttendParams& p, int sms, long long steps, long long units, int max_rows,
                              cudaStream_t stream, bool pdl) {
  switch (dtype) {
    case HSA_BF16: return launch_16<__nv_bfloat16>(rows, p, sms, steps, units, max_rows, stream, pdl);
    case HSA_F16: return launch_16<__half>(rows, p, sms, steps, units, max_rows, stream, pdl);
    case HSA_F32:
      switch (rows) {
        case 4: return launch_attend_t<float, 1, kPack>(p, sms, steps, units, max_rows, stream, pdl);
        case 8: return launch_attend_t<float, 1, kHiLo>(p, sms, steps, units, max_rows, stream, pdl);
        case 16: return launch_attend_t<float, 2, kHiLo>(p, sms, steps, units, max_rows, stream, pdl);
      }
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pqhsa
