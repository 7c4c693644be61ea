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
// and after a barrier the block's warps join them. Units that cross blocks leave one
// partial (m, l, acc) a block, and the merge kernel joins those. Where whole units load the
// blocks evenly enough, shares end with units and there is nothing to merge ("solo"). Shares
// follow from the device lengths alone.
//
// Mathematics of a tile, on mma.sync m16n8k16 (fp16 in, fp32 sums): S^T = K q^T with the 16
// tokens as rows and 8 query rows as columns, P = 2^(S f - ref), O^T += V^T P with dims as
// rows. Keys and values are code x scale, exact in fp16, made in registers straight from the
// tile's bytes: its layout is the fragments' own. q is scaled by a power of two (q_exponent; f
// carries it back); 16-bit q is then one fp16 number, 32-bit q two (hi + lo, 22 bits of elements
// down to 2^-16 of the row's largest, the others to 2^-38 of it), and P likewise, so that 32-bit
// calls keep 32-bit accuracy. A 16-bit call's weights are one fp16 number each, off by 2^-12 of
// themselves at most: against 64 bits its fp16 results are off by 2.9e-4 instead of 2.1e-4 under
// a window of 1024, its bf16 results by 1% more, and half of the P V products are spared. With at most four 32-bit rows hi
// and lo share one fragment (columns 0-3 and 4-7).
//
// ref is the row's largest logit so far less kHead; it moves when a logit exceeds it by
// kHead + kGrow, so P <= 2^(kHead + kGrow) < 65504, and a weight below 2^(-24 - kHead) of the
// largest is lost.
//
// What bounds it. Long batches: the cache's bytes (32 sequences x 8 heads of 32768 tokens with
// bf16 q 204 us, 5.9 TB/s; with fp32 q 221 us). One long sequence: about 14 us beside the bytes
// for the chain lengths -> block table -> tiles, the join and the merge kernel (8 heads of 131072
// tokens 40.9 us with fp32 q, 37.7 us with bf16 q; 1000 tokens 9.4 us). Many rows a tile: the
// tensor instructions of the older kind and the work of making fragments (20 rows on 16 x 8
// heads of 5000 tokens each 48 us).
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
constexpr float kWhole = 8388608.f;   // 2^23: larger logits are whole numbers, up to far more than kHead apart
constexpr int kSoloSteps = 16;
constexpr int kRun = 256;
constexpr int kMergeThreads = 256;
constexpr int kTeamParts = 4;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kPitch = kD + 4;      // floats a row of a warp's partial in shared memory
constexpr int kQPitch = 2 * kD + 16; // bytes a row of q in shared memory

enum Mode { kHi, kHiLo, kPack };

template <int NR, Mode M>
struct Shape {
  static constexpr int RT = M == kPack ? 4 : 8 * NR;             // query rows of a unit
  static constexpr int QF = NR * (M == kHiLo ? 2 : 1);           // q fragments
  static constexpr bool q_smem = NR > 1;                         // in shared memory, a set a warp
  // One block an SM. Its warps: what registers (128 to 255 a thread) and shared memory allow.
  static constexpr int max_warps = NR == 1 ? 16 : 8;
  static constexpr int stages = NR == 2 ? 2 : NR == 4 ? 4 : 3;
  static constexpr int U = 2;                                    // tiles worked on at once
  // The tensor cores cut off what does not fit a sum, a bias that grows with the tiles of a segment (values of
  // one sign: -9e-7 of the result after 64 tiles, -6e-6 after 256). In 32-bit calls the products of U tiles are summed by
  // themselves and added with rounding (-4e-8 at any length; 32 x 8 heads of 32768 tokens 214 -> 221 us).
  static constexpr int sum_tiles = M == kHi ? 1 : U;
  // 16-bit calls sum up to kRun steps in the tensor cores (-3e-5, a sixteenth of fp16's rounding) and then add to sums in
  // the workspace, a lane's own beside their ref: 65536 tokens a warp came out 7e-4 too small, 131072 came out 1.6e-3.
  // It costs 1 to 2% (32 x 8 heads of 32768 tokens 202 -> 204 us), rounded additions as above 4 to 8%.
  static constexpr int run_floats = 32 * (32 * NR + 2 * NR);   // a warp's
  static constexpr size_t ring = static_cast<size_t>(stages) * kStepBytes;      // a warp's
  static constexpr size_t part = static_cast<size_t>(RT) * (kPitch + 2) * sizeof(float);
  static_assert(part <= ring, "a warp's last partial lies over its ring");
  // q in fp16 [hi, lo][row], 272 bytes a row; with NR = 1 it passes through the ring's last stage into registers
  static constexpr int q_rows = 8 * QF;
  static constexpr size_t qspace = static_cast<size_t>(q_rows) * kQPitch;
  static constexpr size_t qbytes = q_smem ? qspace : 0;
  static_assert(q_smem || qspace <= kStepBytes, "a stage holds the rows of q");
  static constexpr size_t of_warp = ring + qbytes;
  static_assert(max_warps * of_warp + 2048 <= 227 * 1024, "shared memory of a block");
  static_assert(2 * max_warps <= 32, "a lane for each segment that is joined");
};

__device__ __forceinline__ void mma_f16_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16-byte asynchronous copy of data that is read once: the first to leave L2, so that a long
// cache does not push out what the next kernels need.
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async_16_hint(void* dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "l"(policy)
               : "memory");
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
  int count;             // steps on the line
};

__device__ __forceinline__ Seq sequence(const Kv4AttendParams& p, int b, int RT) {
  Seq s;
  s.T = kv4_len(p.c, b);
  s.r0 = p.cu ? p.cu[b] : b;
  s.n = p.cu ? p.cu[b + 1] - s.r0 : 1;
  s.n = max(0, min(s.n, p.n_rows - s.r0));
  if (s.r0 < 0) s.n = 0;
  const int first = s.T - s.n - p.window + 1;   // leftmost position of a window (T and the window are below 2^30)
  s.lo = p.window > 0 && first > 0 ? first / kStepTok : 0;
  const int hi = (s.T + kStepTok - 1) / kStepTok;
  s.nt = s.n > 0 ? hi - s.lo : 0;
  s.nrt = (s.n * p.G + RT - 1) / RT;
  s.count = static_cast<int>(static_cast<unsigned>(s.nt) * static_cast<unsigned>(s.nrt) * static_cast<unsigned>(p.c.Hkv));
  return s;
}

// Query token of a query row of a head; p.inv_G = ceil(2^32 / G), exact for rows below 2^25.
__device__ __forceinline__ int token_of(const Kv4AttendParams& p, int row) {
  return p.G == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.inv_G));
}
__device__ __forceinline__ size_t head_row(const Kv4AttendParams& p, int r0, int h, int qrow) {
  const int i = token_of(p, qrow);
  return (static_cast<size_t>(r0) + i) * p.c.Hq + static_cast<size_t>(h) * p.G + (qrow - i * p.G);
}

// The line of all steps (fewer than kKv4MaxSteps) and its equal shares: the first `rest`
// blocks take one step more.
struct Line {
  int W, N, each, rest;
  __device__ __forceinline__ Line(int w, int blocks) : W(w) {
    N = min(blocks, w);
    each = N > 0 ? static_cast<int>(static_cast<unsigned>(w) / static_cast<unsigned>(N)) : 0;
    rest = w - each * N;
  }
  __device__ __forceinline__ int begin(int c) const { return each * c + min(c, rest); }
  __device__ __forceinline__ int block_of(int g) const {
    const int big = rest * (each + 1);
    return g < big ? g / (each + 1) : rest + (g - big) / each;
  }
};

// Inclusive sum over the lanes of a warp.
__device__ __forceinline__ int lane_sums(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Whether the line is too long: its steps counted in 256s beside the exact count, at most 2^24 too few (of 65535
// sequences), and no further than 2^28.
struct Length {
  unsigned of256 = 0;
  // The next 32 sequences, one a lane.
  __device__ __forceinline__ void add(const Kv4AttendParams& p, const Seq& s) {
    const long long count = static_cast<long long>(s.nt) * s.nrt * p.c.Hkv;
    of256 = min(of256 + __reduce_add_sync(0xffffffffu, static_cast<unsigned>(min(count >> 8, 1ll << 22))), 1u << 28);
  }
  __device__ __forceinline__ bool too_long() const { return of256 >= kKv4MaxSteps >> 8; }
};

// A place on the line, by a whole warp: a sequence with the steps and units before it.
struct Spot {
  int b, steps, units;
};
// Totals of all sequences (b = B); none of a line that is too long.
__device__ __forceinline__ Spot line_totals(const Kv4AttendParams& p, int RT) {
  Spot t = {p.c.B, 0, 0};
  Length length;
#pragma unroll 1
  for (int b = threadIdx.x & 31; b - (threadIdx.x & 31) < p.c.B; b += 32) {
    Seq s = {};
    if (b < p.c.B) s = sequence(p, b, RT);
    length.add(p, s);
    t.steps += __reduce_add_sync(0xffffffffu, s.count);
    t.units += __reduce_add_sync(0xffffffffu, s.count ? s.nrt * p.c.Hkv : 0);
  }
  if (length.too_long()) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(p.c.err, HSA_DEVERR_LIMIT);
    t.steps = t.units = 0;
  }
  return t;
}
// The sequence that holds the key-th step (or unit).
__device__ __forceinline__ Spot locate(const Kv4AttendParams& p, int RT, int key, bool by_unit) {
  const int lane = threadIdx.x & 31;
  Spot at = {0, 0, 0};
#pragma unroll 1
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    Seq s = {};
    if (b0 + lane < p.c.B) s = sequence(p, b0 + lane, RT);
    const int u = s.count ? s.nrt * p.c.Hkv : 0;
    const int xs = lane_sums(s.count), xu = lane_sums(u);
    const unsigned past = __ballot_sync(0xffffffffu, (by_unit ? at.units + xu : at.steps + xs) > key);
    if (past) {
      const int l = __ffs(past) - 1;
      at.b = b0 + l;
      at.steps += __shfl_sync(0xffffffffu, xs - s.count, l);
      at.units += __shfl_sync(0xffffffffu, xu - u, l);
      return at;
    }
    at.steps += __shfl_sync(0xffffffffu, xs, 31);
    at.units += __shfl_sync(0xffffffffu, xu, 31);
  }
  at.b = p.c.B;
  return at;
}
// First step of a unit, by a whole warp; the end of the line for a number past the last unit.
__device__ __forceinline__ int unit_step(const Kv4AttendParams& p, int RT, int unit) {
  const Spot at = locate(p, RT, unit, true);
  return at.b < p.c.B ? at.steps + (unit - at.units) * sequence(p, at.b, RT).nt : at.steps;
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
  const float inv = l == 0.f ? 0.f : __frcp_rn(l);
  a.x *= inv;
  a.y *= inv;
  a.z *= inv;
  a.w *= inv;
  store_out<T>(p.out, head_row * kD + d4 * 4, a);
  if (p.lse && d4 == 0) p.lse[head_row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
}

// Four consecutive values of q as fp32.
template <typename T>
__device__ __forceinline__ float4 load_q4(const uint8_t* at);
template <>
__device__ __forceinline__ float4 load_q4<float>(const uint8_t* at) {
  return __ldg(reinterpret_cast<const float4*>(at));
}
template <>
__device__ __forceinline__ float4 load_q4<__nv_bfloat16>(const uint8_t* at) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
  return make_float4(bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y));
}
template <>
__device__ __forceinline__ float4 load_q4<__half>(const uint8_t* at) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
  const float2 a = unpack_f16x2(v.x), b = unpack_f16x2(v.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

// A segment that is joined with others of its unit.
struct Segment {
  int unit, b;           // unit: row tile and head, -1: none
  int h, r0, row0, rows; // head, first query token's row, first and number of query rows
  int open;              // bits: begins at its unit's first step, ends at its last, begins the block
};

template <typename T, int NR, Mode M>
__global__ void __launch_bounds__(Shape<NR, M>::max_warps * 32, 1) kv4_attend_kernel(const __grid_constant__ Kv4AttendParams p) {
  using S = Shape<NR, M>;
  constexpr int RT = S::RT;
  const int warps = blockDim.x >> 5;
  constexpr int kSlot = RT * (kD + 2);             // floats of a slot in the workspace
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Segment segs[2 * S::max_warps];             // a warp's first and last
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * S::ring;
  uint8_t* qs = S::q_smem ? smem + warps * S::ring + warp * S::qbytes : ring + (S::stages - 1) * kStepBytes;
  if (lane < 2) segs[2 * warp + lane].unit = -1;
  __syncwarp();

  pdl_wait();
  pdl_launch_dependents();

  const uint64_t policy = read_once_policy();
  // ---- rows of sequences without tokens: sequence b by block b, b + blocks, ... ----
#pragma unroll 1
  for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
    const Seq e = sequence(p, b, RT);
    if (e.n == 0 || e.nt > 0) continue;
    for (long long i = warp; i < static_cast<long long>(e.n) * p.c.Hq; i += warps)
      finish<T>(p, static_cast<size_t>(e.r0) * p.c.Hq + i, lane, 0.f, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
  }

  // ---- this block's and this warp's share of the line ----
  const Spot all = line_totals(p, RT);
  const Line line(p.solo ? all.units : all.steps, gridDim.x);
  if (static_cast<int>(blockIdx.x) >= line.N) return;
  int block_g = line.begin(blockIdx.x), block_end = line.begin(blockIdx.x + 1);
  if (p.solo) {
    block_g = unit_step(p, RT, block_g);
    block_end = unit_step(p, RT, block_end);
  }
  const int block_len = block_end - block_g;
  // warps: as the blocks, the first ones a step more
  int g = block_g + block_len / warps * warp + min(warp, block_len % warps);
  const int g_end = g + block_len / warps + (warp < block_len % warps ? 1 : 0);
  float* first_slot = p.parts + static_cast<size_t>(2 * gridDim.x + blockIdx.x * warps + warp) * kSlot;

  if (g < g_end) {
    const Spot at = locate(p, RT, g, false);
    int b = at.b, before = at.steps;
    Seq s = sequence(p, b, RT);
    while (g < g_end && b < p.c.B) {
      if (g - before >= s.count) {   // next sequence with work
        before += s.count;
        if (++b < p.c.B) s = sequence(p, b, RT);
        continue;
      }
      const int unit = static_cast<int>(static_cast<unsigned>(g - before) / static_cast<unsigned>(s.nt));   // h * nrt + row tile
      const int a = g - before - unit * s.nt;                    // first step of the segment
      const int len = min(s.nt - a, g_end - g);
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
              for (int j = 0; j < 4; ++j) cp_async_16_hint(dst + j * 512, src + j * 512, policy);
              if (lane < 16) cp_async_16_hint(dst + kOffScale, src + kOffScale, policy);
            } else {
              missing |= 1u << (2 * st + u);
            }
          }
        }
        cp_async_commit();
      };
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < S::stages - 1; ++i) issue(i);

      // ---- query fragments and the bounds of each of this lane's columns ----
      // Row by row, four values a lane.
      int e_mine[NR];               // lane r: exponent of rows r, 8 + r, ... (of four and four: row r & 3)
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
        e_mine[nt] = 0;
#pragma unroll
        for (int c0 = 0; c0 < (M == kPack ? 4 : 8); c0 += 4) {
          if (nt * 8 + c0 >= rows) {   // no rows: zeros
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int at = (M == kHiLo ? 2 * nt : nt) * 8 + c0 + k;
              *reinterpret_cast<uint2*>(qs + at * kQPitch + lane * 8) = make_uint2(0u, 0u);
              if (M == kHiLo) *reinterpret_cast<uint2*>(qs + (at + 8) * kQPitch + lane * 8) = make_uint2(0u, 0u);
              if (M == kPack) *reinterpret_cast<uint2*>(qs + (at + 4) * kQPitch + lane * 8) = make_uint2(0u, 0u);
            }
            continue;
          }
          float4 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = min(nt * 8 + c0 + k, rows - 1);
            const int i = token_of(p, row0 + row);
            x[k] = load_q4<T>(p.q + (static_cast<long long>(s.r0) + i) * p.q_tok +
                              (static_cast<size_t>(h) * p.G + (row0 + row - i * p.G)) * kD * sizeof(T) + lane * 4 * sizeof(T));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float top =
                warp_max_f32(fmaxf(fmaxf(fabsf(x[k].x), fabsf(x[k].y)), fmaxf(fabsf(x[k].z), fabsf(x[k].w))));
            const int e = q_exponent(top);
            const float down = q_factor(top, e);
            const int at = (M == kHiLo ? 2 * nt : nt) * 8 + c0 + k;
            const uint32_t h0 = pack_f16x2(x[k].x * down, x[k].y * down), h1 = pack_f16x2(x[k].z * down, x[k].w * down);
            *reinterpret_cast<uint2*>(qs + at * kQPitch + lane * 8) = make_uint2(h0, h1);
            if (M != kHi) {
              const float2 b0 = unpack_f16x2(h0), b1 = unpack_f16x2(h1);
              *reinterpret_cast<uint2*>(qs + (at + (M == kPack ? 4 : 8)) * kQPitch + lane * 8) =
                  make_uint2(pack_f16x2(x[k].x * down - b0.x, x[k].y * down - b0.y),
                             pack_f16x2(x[k].z * down - b1.x, x[k].w * down - b1.y));
            }
            if ((M == kPack ? (lane & 3) : (lane & 7)) == c0 + k) e_mine[nt] = e;
          }
        }
      }
      __syncwarp();
      uint4 qf[S::q_smem ? 1 : S::QF][4];   // lane: dims [32 t, +32) of row r
      if (!S::q_smem) {
#pragma unroll
        for (int k = 0; k < S::QF; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qf[S::q_smem ? 0 : k][j] = *reinterpret_cast<const uint4*>(qs + (k * 8 + r) * kQPitch + t * 64 + j * 16);
        __syncwarp();                       // before the stage is filled
      }
      float f[2 * NR];
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int own = M == kPack ? ((2 * t + j) & 3) : 2 * t + j;
          // never so small that a masked logit, -inf times f, is NaN; logits under 2^-81 are as good as 0
          const float fc = p.scale * kLog2e * pow2i(__shfl_sync(0xffffffffu, e_mine[nt], own));
          f[2 * nt + j] = fabsf(fc) < 1e-36f ? copysignf(1e-36f, fc) : fc;
        }
      }
      // last and first position that this lane's column c sees
      auto column = [&](int c) { return M == kPack ? ((2 * t + c) & 3) : (c >> 1) * 8 + 2 * t + (c & 1); };
      auto last_seen = [&](int c) {
        const int col = column(c);
        return col >= rows ? -1 : p.causal ? s.T - s.n + token_of(p, row0 + col) : s.T - 1;
      };
      auto first_seen = [&](int c) {
        return p.window > 0 ? s.T - s.n + token_of(p, row0 + column(c)) - p.window + 1 : 0;
      };
      // positions that every row of the unit sees
      const int all_hi = p.causal ? s.T - s.n + token_of(p, row0) : s.T - 1;
      const int all_lo = p.window > 0 ? s.T - s.n + token_of(p, row0 + rows - 1) - p.window + 1 : 0;

      float o[NR][8][4];
      float ref[2 * NR], l[2 * NR];
      unsigned poison = 0;          // bit c: column c saw a value of this lane's dims that is not finite
      // Sums so far, into the workspace (store) or, with what is there, into o.
      auto run_sums = [&](bool store, bool add) {
        float4* sums = reinterpret_cast<float4*>(p.parts + static_cast<size_t>(2 + warps) * gridDim.x * kSlot +
                                                 static_cast<size_t>(blockIdx.x * warps + warp) * S::run_floats) + lane;
        float* refs = reinterpret_cast<float*>(sums - lane + 8 * NR * 32) + lane;
        float shrink[2 * NR];
#pragma unroll
        for (int c = 0; c < 2 * NR; ++c) {
          shrink[c] = add ? fast_exp2(refs[32 * c] - ref[c]) : 0.f;
          if (store) refs[32 * c] = ref[c];
        }
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int i8 = 0; i8 < 8; ++i8) {
            float* v = o[nt][i8];
            if (add) {
              const float4 w = sums[32 * (8 * nt + i8)];
              v[0] = fmaf(w.x, shrink[2 * nt], v[0]);
              v[1] = fmaf(w.y, shrink[2 * nt + 1], v[1]);
              v[2] = fmaf(w.z, shrink[2 * nt], v[2]);
              v[3] = fmaf(w.w, shrink[2 * nt + 1], v[3]);
            }
            if (store) {
              sums[32 * (8 * nt + i8)] = make_float4(v[0], v[1], v[2], v[3]);
              v[0] = v[1] = v[2] = v[3] = 0.f;
            }
          }
      };
#pragma unroll
      for (int j = 0; j < 2 * NR; ++j) {
        ref[j] = kLowest;
        l[j] = 0.f;
      }
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;

#pragma unroll 1
      for (int run = 0; run < len; run += M == kHi ? kRun : len) {
        if (run > 0) run_sums(true, run > kRun);
        const int run_end = M == kHi ? min(len, run + kRun) : len;
#pragma unroll 1
        for (int i = run; i < run_end; ++i) {
          cp_async_wait<S::stages - 2>();
          __syncwarp();
          const int st = i % S::stages;
          const unsigned missing_now = (missing >> (2 * st)) & 3u;
          issue(i + S::stages - 1);
#pragma unroll 1
          for (int u0 = 0; u0 < kStep; u0 += S::U) {
            const uint8_t* stage = ring + st * kStepBytes + u0 * kTileBytes;
            const int pos = (tile0 + i * kStep + u0) * kTileTok;
            const unsigned absent = (missing_now >> u0) & ((1u << S::U) - 1u);
            // ---- S^T = K q^T ----
            float sacc[S::U][NR][4];
            uint2 sc[S::U];
#pragma unroll
            for (int u = 0; u < S::U; ++u) {
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
#pragma unroll
                  for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
                    for (int part_q = 0; part_q < (M == kHiLo ? 2 : 1); ++part_q) {
                      const int fr = M == kHiLo ? 2 * nt + part_q : nt;
                      const uint4 bq = S::q_smem ? *reinterpret_cast<const uint4*>(qs + (fr * 8 + r) * kQPitch + t * 64 + w * 16)
                                                 : qf[S::q_smem ? 0 : fr][w];
                      mma_f16_16816(sacc[u][nt], x[2 * kk], y[2 * kk], x[2 * kk + 1], y[2 * kk + 1], kk ? bq.z : bq.x,
                                    kk ? bq.w : bq.y);
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
            uint32_t vs[S::U][2];
#pragma unroll
            for (int u = 0; u < S::U; ++u) {
              vs[u][0] = scale_pair(sc[u].y, 0);
              vs[u][1] = scale_pair(sc[u].y, 2);
            }
            const bool whole = absent == 0u && pos + S::U * kTileTok - 1 <= all_hi && pos >= all_lo;
            if (!whole) {
              int hi[2 * NR], lo[2 * NR];
#pragma unroll
              for (int c = 0; c < 2 * NR; ++c) {
                hi[c] = last_seen(c);
                lo[c] = first_seen(c);
              }
#pragma unroll
              for (int u = 0; u < S::U; ++u) {
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
                // taken out of the product, and the block's dims of those rows become NaN in the end.
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
                    if (from <= to && (all & ((2u << to) - (1u << from))) != 0u) poison |= 1u << c;
                  }
                }
              }
            }
            // ---- online softmax: weights 2^(s f - ref) ----
            float y[S::U][NR][4], top = -INFINITY;
#pragma unroll
            for (int u = 0; u < S::U; ++u)
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
                for (int u = 0; u < S::U; ++u)
#pragma unroll
                  for (int j = 0; j < 2; ++j) mx = fmaxf(mx, sacc[u][c >> 1][(c & 1) + 2 * j]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float next = fmaxf(ref[c], fabsf(mx) < kWhole ? mx - kHead : mx);   // mx - 11 may round to mx - 16
                const float shrink = fast_exp2(ref[c] - next);
                ref[c] = next;
                l[c] *= shrink;
#pragma unroll
                for (int i8 = 0; i8 < 8; ++i8) {
                  o[c >> 1][i8][c & 1] *= shrink;
                  o[c >> 1][i8][(c & 1) + 2] *= shrink;
                }
#pragma unroll
                for (int u = 0; u < S::U; ++u)
#pragma unroll
                  for (int j = 0; j < 2; ++j)
                    y[u][c >> 1][(c & 1) + 2 * j] = __fsub_rn(sacc[u][c >> 1][(c & 1) + 2 * j], next);
              }
            }
            // ---- O^T += V^T P ----
#pragma unroll
            for (int ub = 0; ub < S::U; ub += S::sum_tiles) {
              uint32_t ph[S::sum_tiles][NR][2], pl[S::sum_tiles][NR][2];
              uint4 v0[S::sum_tiles], v1[S::sum_tiles];
#pragma unroll
              for (int u = 0; u < S::sum_tiles; ++u) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt) {
                  float pr[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const int c = 2 * nt + (j & 1);
                    pr[j] = fast_exp2(y[ub + u][nt][j]);
                    l[c] += pr[j];
                  }
#pragma unroll
                  for (int half = 0; half < 2; ++half) {
                    uint32_t hi2 = pack_f16x2(pr[2 * half], pr[2 * half + 1]);
                    if (M != kHi) {
                      const float2 back = unpack_f16x2(hi2);
                      const uint32_t lo2 = pack_f16x2(pr[2 * half] - back.x, pr[2 * half + 1] - back.y);
                      if (M == kPack) hi2 = t >= 2 ? lo2 : hi2;
                      else pl[u][nt][half] = transpose8x8(lo2);
                    }
                    ph[u][nt][half] = transpose8x8(hi2);
                  }
                }
                const uint8_t* tile = stage + (ub + u) * kTileBytes + kOffV;
                v0[u] = reinterpret_cast<const uint4*>(tile)[lane];
                v1[u] = reinterpret_cast<const uint4*>(tile + 512)[lane];
              }
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                uint32_t x[S::sum_tiles][4], z[S::sum_tiles][4];
#pragma unroll
                for (int u = 0; u < S::sum_tiles; ++u) {
                  const uint32_t w0[4] = {v0[u].x, v0[u].y, v0[u].z, v0[u].w}, w1[4] = {v1[u].x, v1[u].y, v1[u].z, v1[u].w};
                  e2m1_to_f16x2(w0[w], x[u][0], x[u][1], x[u][2], x[u][3]);
                  e2m1_to_f16x2(w1[w], z[u][0], z[u][1], z[u][2], z[u][3]);
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    x[u][j] = hmul2(x[u][j], vs[ub + u][0]);
                    z[u][j] = hmul2(z[u][j], vs[ub + u][1]);
                  }
                }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                  for (int nt = 0; nt < NR; ++nt) {
                    float* to = o[nt][2 * w + kk];
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    float* d = M == kHi ? to : sum;
                    if (M == kHiLo) {      // the small ones first
#pragma unroll
                      for (int u = 0; u < S::sum_tiles; ++u)
                        mma_f16_16816(d, x[u][2 * kk], x[u][2 * kk + 1], z[u][2 * kk], z[u][2 * kk + 1], pl[u][nt][0], pl[u][nt][1]);
                    }
#pragma unroll
                    for (int u = 0; u < S::sum_tiles; ++u)
                      mma_f16_16816(d, x[u][2 * kk], x[u][2 * kk + 1], z[u][2 * kk], z[u][2 * kk + 1], ph[u][nt][0], ph[u][nt][1]);
                    if (M != kHi) {
#pragma unroll
                      for (int j = 0; j < 4; ++j) to[j] += sum[j];
                    }
                  }
                }
              }
            }
          }
        }
      }
      cp_async_wait<0>();
      if (M == kHi && len > kRun) run_sums(false, true);

      // ---- end of a segment: through shared memory, into the result or a partial to be joined ----
      __syncwarp();   // the ring has been read
      float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = 2 * nt + j;
          l[c] += __shfl_xor_sync(0xffffffffu, l[c], 4);
          l[c] += __shfl_xor_sync(0xffffffffu, l[c], 8);
          l[c] += __shfl_xor_sync(0xffffffffu, l[c], 16);
          if (M == kPack) {
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) {
              o[nt][i8][j] += __shfl_xor_sync(0xffffffffu, o[nt][i8][j], 2);
              o[nt][i8][j + 2] += __shfl_xor_sync(0xffffffffu, o[nt][i8][j + 2], 2);
            }
          }
          const int col = nt * 8 + 2 * t + j;
          if (M == kPack && t >= 2) continue;
          float* row = mine + 2 * RT + col * kPitch + 16 * r;
          const float add = (poison >> c) & 1u ? __int_as_float(0x7fffffff) : 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(row)[i] = make_float4(o[nt][2 * i][j] + add, o[nt][2 * i][j + 2] + add,
                                                            o[nt][2 * i + 1][j] + add, o[nt][2 * i + 1][j + 2] + add);
          if (r == 0) {
            mine[col] = ref[c];
            mine[RT + col] = l[c];
          }
        }
      }
      __syncwarp();
      const bool done = a == 0 && len == s.nt;
      if (done || g + len < g_end) {
#pragma unroll 1
        for (int row = 0; row < rows; ++row) {
          const float4 v = *reinterpret_cast<const float4*>(mine + 2 * RT + row * kPitch + lane * 4);
          const float m = mine[row], sum = mine[RT + row];
          if (done) {
            finish<T>(p, head_row(p, s.r0, h, row0 + row), lane, m, sum, v);
          } else {
            if (lane == 0) {
              first_slot[row] = m;
              first_slot[RT + row] = sum;
            }
            *reinterpret_cast<float4*>(first_slot + 2 * RT + row * kD + lane * 4) = v;
          }
        }
      }
      if (!done && lane == 0) {
        segs[2 * warp + (g + len < g_end ? 0 : 1)] =
            Segment{unit, b, h, s.r0, row0, rows,
                    (a == 0 ? 1 : 0) | (a + len == s.nt ? 2 : 0) | (g == block_g ? 4 : 0)};
      }
      g += len;
    }
  }
  __syncthreads();

  // ---- join the warps' partials; a warp takes every warps-th row of all the units together ----
  const int unit = lane < 2 * warps ? segs[lane].unit : -1, unit_b = lane < 2 * warps ? segs[lane].b : 0;
  const unsigned valid = __ballot_sync(0xffffffffu, unit >= 0);
  const unsigned earlier = valid & ((1u << lane) - 1u);
  const int prev = earlier ? 31 - __clz(earlier) : lane;
  const int prev_unit = __shfl_sync(0xffffffffu, unit, prev), prev_b = __shfl_sync(0xffffffffu, unit_b, prev);
  unsigned starts = __ballot_sync(0xffffffffu, unit >= 0 && (!earlier || prev_unit != unit || prev_b != unit_b));
  int item = warp;   // rows still to skip before this warp's next
#pragma unroll 1
  for (; starts; starts &= starts - 1) {
    const int e = __ffs(starts) - 1;
    const unsigned next = starts & (starts - 1);
    const unsigned set = valid & ~((1u << e) - 1u) & (next ? (next & -next) - 1u : 0xffffffffu);
    const Segment head = segs[e];
    const bool mine = (set >> lane) & 1u;
    const bool done = (head.open & 1) && (segs[31 - __clz(set)].open & 2);
    float* out_slot = p.parts + static_cast<size_t>(2 * blockIdx.x + ((head.open & 5) == 1 ? 1 : 0)) * kSlot;
    auto slot_of = [&](int i) -> const float* {
      return i & 1 ? reinterpret_cast<const float*>(smem + (i >> 1) * S::ring)
                   : p.parts + static_cast<size_t>(2 * gridDim.x + blockIdx.x * warps + (i >> 1)) * kSlot;
    };
#pragma unroll 1
    for (; item < head.rows; item += warps) {
      const float m1 = mine ? slot_of(lane)[item] : -INFINITY;
      const float l1 = mine ? slot_of(lane)[RT + item] : 0.f;
      const float m = warp_max_f32(m1);
      const float w = mine ? fast_exp2(m1 - m) : 0.f;
      const float l = warp_sum(w * l1);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (unsigned left = set; left;) {
        float4 v[4];
        float wi[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = left ? __ffs(left) - 1 : e;
          wi[k] = left ? __shfl_sync(0xffffffffu, w, i) : 0.f;
          v[k] = left ? *reinterpret_cast<const float4*>(slot_of(i) + 2 * RT + item * (i & 1 ? kPitch : kD) + lane * 4)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
          left &= left - 1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc.x = fmaf(wi[k], v[k].x, acc.x);
          acc.y = fmaf(wi[k], v[k].y, acc.y);
          acc.z = fmaf(wi[k], v[k].z, acc.z);
          acc.w = fmaf(wi[k], v[k].w, acc.w);
        }
      }
      if (done) {
        finish<T>(p, head_row(p, head.r0, head.h, head.row0 + item), lane, m, l, acc);
      } else {
        if (lane == 0) {
          out_slot[item] = m;
          out_slot[RT + item] = l;
        }
        *reinterpret_cast<float4*>(out_slot + 2 * RT + item * kD + lane * 4) = acc;
      }
    }
    item -= head.rows;
  }
}

// Joins the partials of units that several blocks shared, kTeam warps a query row.
template <typename T, int kTeam>
__global__ void __launch_bounds__(kMergeThreads)
    kv4_merge_kernel(const __grid_constant__ Kv4AttendParams p, int RT, int blocks) {
  __shared__ float4 acc_s[kMergeWarps][32];
  __shared__ float max_s[kMergeWarps], sum_s[kMergeWarps];
  // Lengths and row offsets may be read at once: the attention kernel lets this one start only after it has
  // itself waited for all that came before it.
  pdl_launch_dependents();
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Seq s = sequence(p, b, RT);
  const int rows_all = s.n * p.G;                       // query rows of a head
  const int team = warp / kTeam, member = warp % kTeam;
  int before = 0, W = 0;
  Length length;
#pragma unroll 1
  for (int i = lane; i - lane < p.c.B; i += 32) {
    Seq e = {};
    if (i < p.c.B) e = sequence(p, i, RT);
    length.add(p, e);
    W += __reduce_add_sync(0xffffffffu, e.count);
    before += __reduce_add_sync(0xffffffffu, i < b ? e.count : 0);
  }
  const Line line(W, blocks);
  pdl_wait();
  if (length.too_long()) return;
#pragma unroll 1
  for (unsigned item = blockIdx.x * (kMergeWarps / kTeam) + team; s.nt > 0; item += gridDim.x * (kMergeWarps / kTeam)) {
    const int qrow = item / p.c.Hkv, h = item % p.c.Hkv;
    if (qrow >= rows_all) break;
    const int rt = qrow / RT, row = qrow % RT;
    const int u0 = before + (h * s.nrt + rt) * s.nt;
    const int c0 = line.block_of(u0), c1 = line.block_of(u0 + s.nt - 1);
    if (c0 == c1) continue;
    const int late = line.begin(c0) == u0 ? 0 : 1;   // the unit is its first block's last segment
    const float* slots = p.parts + static_cast<size_t>(2 * c0) * RT * (kD + 2);
    const int parts = c1 - c0 + 1;
    auto slot_of = [&](int i) { return slots + static_cast<size_t>(2 * i + (i == 0 ? late : 0)) * RT * (kD + 2); };
    // a warp takes every kTeam-th part, four in flight
    float m = kLowest, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = member; i0 < parts; i0 += 4 * kTeam) {
      float mi[4], li[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kTeam;
        const float* slot = slot_of(min(i, parts - 1));
        mi[k] = slot[row];
        li[k] = slot[RT + row];
        v[k] = *reinterpret_cast<const float4*>(slot + 2 * RT + row * kD + lane * 4);
        if (i >= parts) mi[k] = -INFINITY;
      }
      const float next = fmaxf(fmaxf(fmaxf(mi[0], mi[1]), fmaxf(mi[2], mi[3])), m);
      const float old = fast_exp2(m - next);
      m = next;
      l *= old;
      acc.x *= old;
      acc.y *= old;
      acc.z *= old;
      acc.w *= old;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i0 + k * kTeam >= parts) break;
        const float y = fast_exp2(mi[k] - m);
        l = fmaf(li[k], y, l);
        acc.x = fmaf(v[k].x, y, acc.x);
        acc.y = fmaf(v[k].y, y, acc.y);
        acc.z = fmaf(v[k].z, y, acc.z);
        acc.w = fmaf(v[k].w, y, acc.w);
      }
    }
    if constexpr (kTeam == 1) {
      finish<T>(p, head_row(p, s.r0, h, qrow), lane, m, l, acc);
      continue;
    }
    acc_s[warp][lane] = acc;
    if (lane == 0) {
      max_s[warp] = m;
      sum_s[warp] = l;
    }
    __syncthreads();
    if (warp == 0) {
      m = max_s[0];
#pragma unroll
      for (int w = 1; w < kMergeWarps; ++w) m = fmaxf(m, max_s[w]);
      l = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float y = fast_exp2(max_s[w] - m);
        const float4 v = acc_s[w][lane];
        l = fmaf(sum_s[w], y, l);
        acc.x = fmaf(v.x, y, acc.x);
        acc.y = fmaf(v.y, y, acc.y);
        acc.z = fmaf(v.z, y, acc.z);
        acc.w = fmaf(v.w, y, acc.w);
      }
      finish<T>(p, head_row(p, s.r0, h, qrow), lane, m, l, acc);
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
cudaError_t launch_attend_t(Kv4AttendParams p, const Kv4Load& load, int sms, cudaStream_t stream, bool pdl) {
  using S = Shape<NR, M>;
  cudaError_t e = ensure_dyn_smem<kv4_attend_kernel<T, NR, M>>(S::max_warps * S::of_warp);
  if (e != cudaSuccess) return e;
  const long long most = std::min(sms, kKv4MaxSms);
  // Solo: blocks take whole units. Their longest share is then longer than the mean by what is compared here,
  // and the joint work is spared, which takes as long as kSoloSteps steps of a block for eight rows and half of that
  // for each eight more. Measured, solo and shared (us): 32 sequences x 8 heads of 500 tokens 12.0 and 15.5, 64 x 8 of
  // 200 13.7 and 15.6, 13 x 8 of 1500 14.2 and 17.3, 20 rows on 16 x 8 of 5000 47 and 50; but 8 units of 1000 11.8 and
  // 9.0, two times 32 rows on 10 x 8 of 2000 62 and 52.
  const long long rounds = (load.units + most - 1) / most;
  p.solo = rounds * load.longest - load.steps / most <= kSoloSteps * (NR + 1) / 2 ? 1 : 0;
  // Steps are spread over the SMs before they are over the warps of one (a block's warps share its issue slots),
  // and there are no more warps than steps.
  const long long per_block = p.solo ? rounds * load.longest : (load.steps + most - 1) / most;
  const int warps = static_cast<int>(std::max(1ll, std::min<long long>(S::max_warps, per_block)));
  const int blocks =
      static_cast<int>(std::max(1ll, std::min(most, p.solo ? load.units : (load.steps + warps - 1) / warps)));
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = launch_config(dim3(blocks), warps * 32, warps * S::of_warp, stream, attr, pdl);
  e = cudaLaunchKernelEx(&cfg, kv4_attend_kernel<T, NR, M>, p);
  if (e != cudaSuccess || p.solo) return e;
  // A unit's partials, about: a few are joined by a warp a row, many by a block a row (us, warp and block: 20 rows on
  // 16 x 8 heads of about 5000 tokens 50.6 and 57.8; 8 heads of 131072 tokens, one row, 42.9 and 39.4).
  const long long parts = load.longest * blocks / std::max(1ll, load.steps) + 2;
  const long long rows = static_cast<long long>(p.c.Hkv) * load.max_rows;
  const bool few = parts <= kTeamParts;
  cfg = launch_config(dim3(static_cast<unsigned>(few ? (rows + kMergeWarps - 1) / kMergeWarps : rows), p.c.B),
                      kMergeThreads, 0, stream, attr, pdl);
  return few ? cudaLaunchKernelEx(&cfg, kv4_merge_kernel<T, 1>, p, static_cast<int>(S::RT), blocks)
             : cudaLaunchKernelEx(&cfg, kv4_merge_kernel<T, kMergeWarps>, p, static_cast<int>(S::RT), blocks);
}

template <typename T>
cudaError_t launch_16(int rows, const Kv4AttendParams& p, const Kv4Load& load, int sms, cudaStream_t stream,
                      bool pdl) {
  switch (rows) {
    case 8: return launch_attend_t<T, 1, kHi>(p, load, sms, stream, pdl);
    case 16: return launch_attend_t<T, 2, kHi>(p, load, sms, stream, pdl);
    case 24: return launch_attend_t<T, 3, kHi>(p, load, sms, stream, pdl);
    case 32: return launch_attend_t<T, 4, kHi>(p, load, sms, stream, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int kv4_attend_step_tokens() { return kStepTok; }

int kv4_attend_rows(int dtype, int max_rows) {
  if (dtype == HSA_F32) return max_rows <= 4 ? 4 : max_rows <= 8 ? 8 : 16;
  return max_rows <= 8 ? 8 : max_rows <= 16 ? 16 : max_rows <= 24 ? 24 : 32;
}

// Two slots a block and one a warp, and a warp's sums of earlier runs: 18 of 8 rows or 10 of 16, 24 or 32, and 16 or 8.
size_t kv4_attend_part_bytes() {
  return static_cast<size_t>(kKv4MaxSms) * (10 * 32 * (kD + 2) + 8 * Shape<4, kHi>::run_floats) * sizeof(float);
}

cudaError_t launch_kv4_attend(int dtype, int rows, const Kv4AttendParams& p, const Kv4Load& load, int sms,
                              cudaStream_t stream, bool pdl) {
  switch (dtype) {
    case HSA_BF16: return launch_16<__nv_bfloat16>(rows, p, load, sms, stream, pdl);
    case HSA_F16: return launch_16<__half>(rows, p, load, sms, stream, pdl);
    case HSA_F32:
      switch (rows) {
        case 4: return launch_attend_t<float, 1, kPack>(p, load, sms, stream, pdl);
        case 8: return launch_attend_t<float, 1, kHiLo>(p, load, sms, stream, pdl);
        case 16: return launch_attend_t<float, 2, kHiLo>(p, load, sms, stream, pdl);
      }
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pqhsa
