// Attention over the 4-bit KV cache for few query rows a KV head (decode, verification of
// drafted tokens): every warp streams 16-token tiles through registers and joins its rows'
// online softmax states at the end.
//
// Work. A unit is (sequence, KV head, tile of query rows); its tokens are 16-token tiles. All
// units' tiles lie on one line, in the order of (sequence, head, row tile), and every block
// takes an equal share of that line, so long and short sequences load the blocks alike. A
// block works through its share unit by unit (a segment each), its warps taking the
// segment's tiles in turn. A unit that lies within one block's share is finished there; of
// one that does not, each block leaves a partial (m, l, acc) in the workspace, two slots a
// block, and the merge kernel joins them. Shares follow from the device lengths alone.
//
// Mathematics of a tile, on mma.sync m16n8k16 (fp16 in, fp32 sums): S^T = K q^T with the 16
// tokens as rows and 8 query rows as columns, P = 2^(S f - ref), O^T += V^T P with dims as
// rows. Keys and values are code x scale, exact in fp16, made in registers straight from the
// tile's bytes: its layout is the fragments' own. q is scaled to at most 1 by a power of
// two (f carries it back); 16-bit q is then one fp16 number, 32-bit q two (hi + lo, 22 bits),
// and P likewise, so that 32-bit calls keep 32-bit accuracy. With at most four 32-bit rows hi
// and lo share one fragment (columns 0-3 and 4-7).
//
// ref is the row's largest logit so far, up to a growth of 2^kGrow that does not yet move it:
// P <= 2^(kHead + kGrow) < 65504 and below 2^(kHead - 24) of the largest it is lost.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4.cuh"

namespace pqhsa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;          // tiles in flight a warp
constexpr float kHead = 11.f, kGrow = 4.f;
constexpr int kMergeThreads = 128;
constexpr int kPitch = kD + 4;      // floats a row of a warp's partial in shared memory

enum Mode { kHi, kHiLo, kPack };

template <int NR, Mode M>
struct Shape {
  static constexpr int RT = M == kPack ? 4 : 8 * NR;             // query rows of a unit
  static constexpr int QF = NR * (M == kHiLo ? 2 : 1);           // q fragments
  static constexpr bool q_smem = NR > 1;
  static constexpr size_t ring = static_cast<size_t>(kWarps) * kStages * kTileBytes;
  static constexpr size_t part = static_cast<size_t>(kWarps) * RT * (kPitch + 2) * sizeof(float);
  static constexpr size_t qbytes = q_smem ? static_cast<size_t>(QF) * 8 * 32 * 8 : 0;
  static constexpr size_t total = ring + part + qbytes;
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

// ---- shares of the line of tiles ---------------------------------------------

struct Seq {
  int T, n, r0;          // tokens, query tokens, first query token's row
  int lo, nt, nrt;       // first tile, tiles, row tiles
  long long count;       // tiles on the line
};

__device__ __forceinline__ Seq sequence(const Kv4AttendParams& p, int b, int RT) {
  Seq s;
  s.T = kv4_len(p.c, b);
  s.r0 = p.cu ? p.cu[b] : b;
  s.n = p.cu ? p.cu[b + 1] - s.r0 : 1;
  s.n = max(0, min(s.n, p.n_rows - s.r0));
  if (s.r0 < 0) s.n = 0;
  const long long first = static_cast<long long>(s.T) - s.n - p.window + 1;   // leftmost position of a window
  s.lo = p.window > 0 && first > 0 ? static_cast<int>(first / kTileTok) : 0;
  const int hi = (s.T + kTileTok - 1) / kTileTok;
  s.nt = s.n > 0 ? hi - s.lo : 0;
  s.nrt = (s.n * p.G + RT - 1) / RT;
  s.count = static_cast<long long>(s.nt) * s.nrt * p.c.Hkv;
  return s;
}

// Tiles of all sequences, by a whole warp; before: tiles of the sequences before `b`.
__device__ __forceinline__ long long line_length(const Kv4AttendParams& p, int RT, int b, long long* before) {
  const int lane = threadIdx.x & 31;
  long long all = 0, head = 0;
  for (int i = lane; i < p.c.B; i += 32) {
    const long long n = sequence(p, i, RT).count;
    all += n;
    if (i < b) head += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    head += __shfl_xor_sync(0xffffffffu, head, o);
  }
  *before = head;
  return all;
}

// Sequence that holds tile g of the line and the tiles before it, by a whole warp.
__device__ __forceinline__ int locate(const Kv4AttendParams& p, int RT, long long g, long long* before) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    const long long n = b0 + lane < p.c.B ? sequence(p, b0 + lane, RT).count : 0;
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
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

__device__ __forceinline__ long long share_begin(long long W, int N, int c) { return W * c / N; }
__device__ __forceinline__ int share_of(long long W, int N, long long g) {
  return static_cast<int>(((g + 1) * N - 1) / W);
}

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

template <typename T, int NR, Mode M>
__global__ void __launch_bounds__(kThreads, NR == 1 ? 2 : 1) kv4_attend_kernel(Kv4AttendParams p) {
  using S = Shape<NR, M>;
  constexpr int RT = S::RT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + static_cast<size_t>(warp) * kStages * kTileBytes;
  float* part = reinterpret_cast<float*>(smem + S::ring);
  float* part_m = part + kWarps * RT * kPitch;        // [warp][RT]
  float* part_l = part_m + kWarps * RT;
  uint2* qs = reinterpret_cast<uint2*>(smem + S::ring + S::part);   // [fragment][8][lane]

  pdl_wait();
  pdl_launch_dependents();

  long long before = 0;
  const long long W = line_length(p, RT, 0, &before);
  const int N = static_cast<int>(min(static_cast<long long>(gridDim.x), W));
  if (static_cast<int>(blockIdx.x) >= N) return;
  long long g = share_begin(W, N, blockIdx.x);
  const long long g_end = share_begin(W, N, blockIdx.x + 1);
  int b = locate(p, RT, g, &before);
  Seq s = sequence(p, b, RT);
  bool first_segment = true;

  while (g < g_end) {
    while (g - before >= s.count) {   // next sequence with work
      before += s.count;
      s = sequence(p, ++b, RT);
    }
    const long long in_seq = g - before;
    const int unit = static_cast<int>(in_seq / s.nt);          // h * nrt + row tile
    const int a = static_cast<int>(in_seq % s.nt);             // first tile of the segment
    const int len = static_cast<int>(min(static_cast<long long>(s.nt - a), g_end - g));
    const int h = unit / s.nrt, rt = unit % s.nrt;
    const int rows = min(RT, s.n * p.G - rt * RT);             // valid query rows

    // ---- query fragments and the bounds of each of this lane's columns ----
    uint32_t qf[S::q_smem ? 1 : S::QF][16];
    float f[2 * NR];
    int hi[2 * NR], lo[2 * NR];
    if (S::q_smem) __syncthreads();   // the last segment's fragments have been read
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      const int col = M == kPack ? (r & 3) : nt * 8 + r;
      float x[32];
      float top = 0.f;
      if (col < rows) {
        const int row = rt * RT + col;
        load_q32<T>(p.q + (static_cast<long long>(s.r0) + row / p.G) * p.q_tok +
                        (static_cast<size_t>(h) * p.G + row % p.G) * kD * sizeof(T) + t * 32 * sizeof(T),
                    x);
#pragma unroll
        for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[i]));
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.f;
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = top > 0.f && top < INFINITY ? ilogbf(top) + 1 : 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x0 = scalbnf(x[2 * i], -e), x1 = scalbnf(x[2 * i + 1], -e);
        const uint32_t hi2 = pack_f16x2(x0, x1);
        uint32_t lo2 = 0u;
        if (M != kHi) {
          const float2 back = unpack_f16x2(hi2);
          lo2 = pack_f16x2(x0 - back.x, x1 - back.y);
        }
        const uint32_t v = M == kPack && r >= 4 ? lo2 : hi2;
        if (S::q_smem) {
          if (warp == 0) {
            reinterpret_cast<uint32_t*>(qs + ((M == kHiLo ? 2 * nt : nt) * 8 + i / 2) * 32 + lane)[i & 1] = v;
            if (M == kHiLo) reinterpret_cast<uint32_t*>(qs + ((2 * nt + 1) * 8 + i / 2) * 32 + lane)[i & 1] = lo2;
          }
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
        f[2 * nt + j] = scalbnf(p.scale * kLog2e, ec);
        const int pos = s.T - s.n + (rt * RT + c) / p.G;
        hi[2 * nt + j] = c >= rows ? -1 : p.causal ? pos : s.T - 1;
        lo[2 * nt + j] = p.window > 0 ? pos - p.window + 1 : 0;
      }
    }
    if (S::q_smem) __syncthreads();
    // positions that every row of the unit sees
    const int all_hi = p.causal ? s.T - s.n + (rt * RT) / p.G : s.T - 1;
    const int all_lo = p.window > 0 ? s.T - s.n + (rt * RT + rows - 1) / p.G - p.window + 1 : 0;

    // ---- tiles: copies run kStages ahead, page numbers 32 tiles ahead ----
    const int mine = len > warp ? (len - warp + kWarps - 1) / kWarps : 0;   // this warp's tiles
    const int tile0 = s.lo + a + warp;
    int pages = -1;
    unsigned missing = 0;                                          // stages whose tile has no page
    auto issue = [&](int i) {
      if (i < mine) {
        if ((i & 31) == 0 && i + lane < mine) pages = kv4_page(p.c, b, tile0 + (i + lane) * kWarps);
        const int page = __shfl_sync(0xffffffffu, pages, i & 31);
        missing = (missing & ~(1u << (i % kStages))) | (page < 0 ? 1u << (i % kStages) : 0u);
        if (page >= 0) {
          const uint8_t* src = p.c.cache + kv4_tile_offset(p.c, page, h, tile0 + i * kWarps);
          uint8_t* dst = ring + (i % kStages) * kTileBytes;
#pragma unroll
          for (int j = 0; j < 4; ++j) cp_async_16(dst + j * 512 + lane * 16, src + j * 512 + lane * 16);
          if (lane < 16) cp_async_16(dst + kOffScale + lane * 16, src + kOffScale + lane * 16);
        }
      }
      cp_async_commit();
    };
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

    for (int i = 0; i < kStages - 1; ++i) issue(i);
    for (int i = 0; i < mine; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const bool present = !((missing >> (i % kStages)) & 1u);
      issue(i + kStages - 1);
      const uint8_t* tile = ring + (i % kStages) * kTileBytes;
      const int pos = (tile0 + i * kWarps) * kTileTok;
      const uint4 k0 = reinterpret_cast<const uint4*>(tile)[lane];
      const uint4 k1 = reinterpret_cast<const uint4*>(tile + 512)[lane];
      const uint4 v0 = reinterpret_cast<const uint4*>(tile + kOffV)[lane];
      const uint4 v1 = reinterpret_cast<const uint4*>(tile + kOffV + 512)[lane];
      const uint2 sc = reinterpret_cast<const uint2*>(tile + kOffScale)[lane];
      // ---- S^T = K q^T ----
      float sacc[NR][4];
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) sacc[nt][j] = 0.f;
      {
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t x[4], y[4];
          e2m1_to_f16x2(w0[w], x[0], x[1], x[2], x[3]);
          e2m1_to_f16x2(w1[w], y[0], y[1], y[2], y[3]);
          const uint32_t s0 = scale_both(sc.x, w >> 1), s1 = scale_both(sc.x, 2 + (w >> 1));
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
                mma_f16_16816(sacc[nt], x[2 * kk], y[2 * kk], x[2 * kk + 1], y[2 * kk + 1], bq.x, bq.y);
              }
            }
          }
        }
      }
      if (M == kPack) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sacc[0][j] += __shfl_xor_sync(0xffffffffu, sacc[0][j], 2);
      }
      // ---- logits in log2 units, masks ----
      const bool whole = present && pos + kTileTok - 1 <= all_hi && pos >= all_lo;
      uint32_t vs0 = scale_pair(sc.y, 0), vs1 = scale_pair(sc.y, 2);
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) sacc[nt][j] *= f[2 * nt + (j & 1)];
      if (!whole) {
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int tp = pos + r + 8 * (j >> 1), c = 2 * nt + (j & 1);
            if (tp > hi[c] || tp < lo[c] || !present) sacc[nt][j] = -INFINITY;
          }
        // A zero weight must not meet a NaN or an infinity: tokens past the end hold anything.
        const int left = present ? s.T - (pos + 2 * t) : 0;   // tokens from this lane's first on
        vs0 &= (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
        vs1 &= (left > 8 ? 0xffffu : 0u) | (left > 9 ? 0xffff0000u : 0u);
        // Values that are not finite count for the rows that see their token, and for no other:
        // taken out of the product, and added as NaN to those rows' sums of the block's dims.
        const unsigned bad = ((vs0 & 0x7c00u) == 0x7c00u ? 1u : 0u) | ((vs0 & 0x7c000000u) == 0x7c000000u ? 2u : 0u) |
                             ((vs1 & 0x7c00u) == 0x7c00u ? 256u : 0u) | ((vs1 & 0x7c000000u) == 0x7c000000u ? 512u : 0u);
        if (__any_sync(0xffffffffu, bad != 0u)) {
          vs0 &= (bad & 1u ? 0u : 0xffffu) | (bad & 2u ? 0u : 0xffff0000u);
          vs1 &= (bad & 256u ? 0u : 0xffffu) | (bad & 512u ? 0u : 0xffff0000u);
          unsigned all = bad << (2 * t);                       // bit: token of the tile
          all |= __shfl_xor_sync(0xffffffffu, all, 1);
          all |= __shfl_xor_sync(0xffffffffu, all, 2);
#pragma unroll
          for (int c = 0; c < 2 * NR; ++c) {
            const int first = max(0, lo[c] - pos), last = min(kTileTok - 1, hi[c] - pos);
            const bool seen = first <= last && (all & ((2u << last) - (1u << first))) != 0u;
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) {
              if (seen) o[c >> 1][i8][c & 1] = o[c >> 1][i8][(c & 1) + 2] = __int_as_float(0x7fffffff);
            }
          }
        }
      }
      // ---- online softmax ----
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          grow |= fmaxf(sacc[nt][j], sacc[nt][j + 2]) > ref[2 * nt + j] + (kHead + kGrow);
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = 2 * nt + j;
            float mx = fmaxf(sacc[nt][j], sacc[nt][j + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float next = fmaxf(ref[c], mx - kHead);
            const float shrink = fast_exp2(ref[c] - next);
            ref[c] = next;
            l[c] *= shrink;
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) {
              o[nt][i8][j] *= shrink;
              o[nt][i8][j + 2] *= shrink;
            }
          }
      }
      uint32_t ph[NR][2], pl[NR][2];
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
        float pr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          pr[j] = fast_exp2(sacc[nt][j] - ref[2 * nt + (j & 1)]);
          l[2 * nt + (j & 1)] += pr[j];
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
      // ---- O^T += V^T P ----
      {
        const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t x[4], y[4];
          e2m1_to_f16x2(w0[w], x[0], x[1], x[2], x[3]);
          e2m1_to_f16x2(w1[w], y[0], y[1], y[2], y[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = hmul2(x[j], vs0);
            y[j] = hmul2(y[j], vs1);
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

    // ---- join the warps ----
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
        if (M != kPack || t < 2) {
          float* row = part + (warp * RT + col) * kPitch + 16 * r;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(row)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          if (r == 0) {
            part_m[warp * RT + col] = ref[c];
            part_l[warp * RT + col] = l[c];
          }
        }
      }
    }
    __syncthreads();
    const bool done = a == 0 && len == s.nt;
    float* slot = p.parts + static_cast<size_t>(2 * blockIdx.x + (first_segment ? 0 : 1)) * RT * (kD + 2);
    for (int i = tid; i < rows * 32; i += kThreads) {
      const int row = i >> 5, d4 = i & 31;
      float m = -1e30f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, part_m[w * RT + row]);
      float lt = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float x = fast_exp2(part_m[w * RT + row] - m);
        const float4 v = *reinterpret_cast<const float4*>(part + (w * RT + row) * kPitch + d4 * 4);
        lt = fmaf(x, part_l[w * RT + row], lt);
        acc.x = fmaf(x, v.x, acc.x);
        acc.y = fmaf(x, v.y, acc.y);
        acc.z = fmaf(x, v.z, acc.z);
        acc.w = fmaf(x, v.w, acc.w);
      }
      if (done) {
        const int qrow = rt * RT + row;
        const size_t at = (static_cast<size_t>(s.r0) + qrow / p.G) * p.c.Hq + static_cast<size_t>(h) * p.G + qrow % p.G;
        finish<T>(p, at, d4, m, lt, acc);
      } else {
        if (d4 == 0) {
          slot[row] = m;
          slot[RT + row] = lt;
        }
        *reinterpret_cast<float4*>(slot + 2 * RT + row * kD + d4 * 4) = acc;
      }
    }
    __syncthreads();
    g += len;
    first_segment = false;
  }
}

// One block a query row of a unit: joins the partials of a unit that several blocks shared, and
// writes the rows of sequences without tokens.
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(Kv4AttendParams p, int RT, int blocks) {
  __shared__ float4 acc_s[kMergeThreads / 32][32];
  __shared__ float ml_s[2][kMergeThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Seq s = sequence(p, b, RT);
  const int rows_all = s.n * p.G;                       // query rows of a head
  const int h = blockIdx.x % p.c.Hkv;
  long long before = 0;
  long long W = -1;
  int N = 1;
  for (int qrow = blockIdx.x / p.c.Hkv; qrow < rows_all; qrow += gridDim.x / p.c.Hkv) {
    const size_t at = (static_cast<size_t>(s.r0) + qrow / p.G) * p.c.Hq + static_cast<size_t>(h) * p.G + qrow % p.G;
    if (s.nt == 0) {
      if (warp == 0) finish<T>(p, at, lane, 0.f, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
      continue;
    }
    if (W < 0) {
      W = line_length(p, RT, b, &before);
      N = static_cast<int>(min(static_cast<long long>(blocks), W));
    }
    const int rt = qrow / RT, row = qrow % RT;
    const long long u0 = before + (static_cast<long long>(h) * s.nrt + rt) * s.nt;
    const int c0 = share_of(W, N, u0), c1 = share_of(W, N, u0 + s.nt - 1);
    if (c0 == c1) continue;
    const int late = share_begin(W, N, c0) == u0 ? 0 : 1;   // the unit is its first block's last segment
    float m = -1e30f, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0 + warp; c <= c1; c += kMergeThreads / 32) {
      const float* slot = p.parts + static_cast<size_t>(2 * c + (c == c0 ? late : 0)) * RT * (kD + 2);
      const float mc = slot[row], lc = slot[RT + row];
      const float4 v = *reinterpret_cast<const float4*>(slot + 2 * RT + row * kD + lane * 4);
      const float next = fmaxf(m, mc);
      const float x = fast_exp2(m - next), y = fast_exp2(mc - next);
      m = next;
      l = fmaf(l, x, lc * y);
      acc.x = fmaf(acc.x, x, v.x * y);
      acc.y = fmaf(acc.y, x, v.y * y);
      acc.z = fmaf(acc.z, x, v.z * y);
      acc.w = fmaf(acc.w, x, v.w * y);
    }
    acc_s[warp][lane] = acc;
    if (lane == 0) {
      ml_s[0][warp] = m;
      ml_s[1][warp] = l;
    }
    __syncthreads();
    if (warp == 0) {
      m = ml_s[0][0];
#pragma unroll
      for (int w = 1; w < kMergeThreads / 32; ++w) m = fmaxf(m, ml_s[0][w]);
      l = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kMergeThreads / 32; ++w) {
        const float x = fast_exp2(ml_s[0][w] - m);
        const float4 v = acc_s[w][lane];
        l = fmaf(x, ml_s[1][w], l);
        acc.x = fmaf(x, v.x, acc.x);
        acc.y = fmaf(x, v.y, acc.y);
        acc.z = fmaf(x, v.z, acc.z);
        acc.w = fmaf(x, v.w, acc.w);
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
cudaError_t launch_attend_t(const Kv4AttendParams& p, int sms, long long tiles, int max_rows, cudaStream_t stream,
                            bool pdl) {
  using S = Shape<NR, M>;
  cudaError_t e = ensure_dyn_smem<kv4_attend_kernel<T, NR, M>>(S::total);
  if (e != cudaSuccess) return e;
  const long long most = static_cast<long long>(std::min(sms, kKv4MaxSms)) * (NR == 1 ? 2 : 1);
  // a share of at least one tile a warp
  const int blocks = static_cast<int>(std::max(1ll, std::min(most, (tiles + kWarps - 1) / kWarps)));
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = launch_config(dim3(blocks), kThreads, S::total, stream, attr, pdl);
  e = cudaLaunchKernelEx(&cfg, kv4_attend_kernel<T, NR, M>, p);
  if (e != cudaSuccess) return e;
  cfg = launch_config(dim3(p.c.Hkv * std::max(1, max_rows), p.c.B), kMergeThreads, 0, stream, attr, pdl);
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel<T>, p, static_cast<int>(S::RT), blocks);
}

template <typename T>
cudaError_t launch_16(int rows, const Kv4AttendParams& p, int sms, long long tiles, int max_rows, cudaStream_t stream,
                      bool pdl) {
  switch (rows) {
    case 8: return launch_attend_t<T, 1, kHi>(p, sms, tiles, max_rows, stream, pdl);
    case 16: return launch_attend_t<T, 2, kHi>(p, sms, tiles, max_rows, stream, pdl);
    case 32: return launch_attend_t<T, 4, kHi>(p, sms, tiles, max_rows, stream, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int kv4_attend_rows(int dtype, int max_rows) {
  if (dtype == HSA_F32 && max_rows <= 4) return 4;
  return max_rows <= 8 ? 8 : max_rows <= 16 ? 16 : 32;
}

size_t kv4_attend_part_bytes() {   // two slots a block: of 8 rows with two blocks an SM, of up to 32 with one
  return static_cast<size_t>(2) * kKv4MaxSms * 32 * (kD + 2) * sizeof(float);
}

cudaError_t launch_kv4_attend(int dtype, int rows, const Kv4AttendParams& p, int sms, long long tiles, int max_rows,
                              cudaStream_t stream, bool pdl) {
  switch (dtype) {
    case HSA_BF16: return launch_16<__nv_bfloat16>(rows, p, sms, tiles, max_rows, stream, pdl);
    case HSA_F16: return launch_16<__half>(rows, p, sms, tiles, max_rows, stream, pdl);
    case HSA_F32:
      switch (rows) {
        case 4: return launch_attend_t<float, 1, kPack>(p, sms, tiles, max_rows, stream, pdl);
        case 8: return launch_attend_t<float, 1, kHiLo>(p, sms, tiles, max_rows, stream, pdl);
        case 16: return launch_attend_t<float, 2, kHiLo>(p, sms, tiles, max_rows, stream, pdl);
        case 32: return launch_attend_t<float, 4, kHiLo>(p, sms, tiles, max_rows, stream, pdl);
      }
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pqhsa
