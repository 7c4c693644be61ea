// Rows into and out of the 4-bit KV cache: quantise as written, and read back.
//
// One warp works on one tile (16 tokens of one sequence and KV head). A lane holds whole
// scale blocks: of the keys, dims [32 (lane % 4), +32) of tokens lane / 4 and 8 + lane / 4
// (two blocks each); of the values, dims [16 (lane / 4), +16) of the token pairs 2 (lane % 4)
// and 8 + 2 (lane % 4) (one block a token). So no value crosses lanes, and each lane's codes
// and scales are four 16-byte pieces and one 8-byte word of the tile at 16 (8) x lane.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv4.cuh"

namespace pqhsa {
namespace {

constexpr int kRowsThreads = 256;

// 16 values of T as they lie in memory.
template <typename T>
struct Raw {
  uint4 v[sizeof(T)];
  // zeros where not `in`: no branch, so that many loads are in flight
  __device__ __forceinline__ void load(const uint8_t* p, bool in) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
      v[i] = in ? __ldg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0u, 0u, 0u, 0u);
  }
};

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ void widen(const Raw<float>& r, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = __uint_as_float(r.v[i].x);
      x[4 * i + 1] = __uint_as_float(r.v[i].y);
      x[4 * i + 2] = __uint_as_float(r.v[i].z);
      x[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = bf16lo(w[j]);
        x[8 * i + 2 * j + 1] = bf16hi(w[j]);
      }
    }
  }
  static __device__ __forceinline__ uint32_t of(uint32_t h) {   // an fp16 pair, exactly
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(a.x, a.y);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ void widen(const Raw<__half>& r, float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        x[8 * i + 2 * j] = a.x;
        x[8 * i + 2 * j + 1] = a.y;
      }
    }
  }
  static __device__ __forceinline__ uint32_t of(uint32_t h) { return h; }
};

// Largest of |a|, |b| and m, NaN if one is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}

// One block: scale byte and 16 values over scale, not yet rounded to codes.
// a / 6 and x / scale are correctly rounded quotients: one at a rounding border of the few-bit
// result is then exact, so ties are ties, and none beside a border reaches it. x / scale by the
// reciprocal r = 1 / scale, correctly rounded, and one correction: y = x r, y + r (x - y scale)
// (Markstein, IBM J. Res. Dev. 34, 1990), three instructions for two values (32768 tokens x 8 heads
// from bf16 took 73 us with divisions, 47 with this).
__device__ __forceinline__ uint32_t quantise16(float* x) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) top = max_abs(top, x[i], x[i + 1]);
  if (!(top < INFINITY)) {   // a NaN or an infinity
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    return 255u;
  }
  const float y = fminf(__fdiv_rn(top, 6.f), 10240.f);
  uint32_t byte;
  float scale;
  if (y >= 6.103515625e-05f) {   // 2^-14, the smallest normal scale: three mantissa bits, nearest even
    const uint32_t u = __float_as_uint(y);
    const uint32_t r = (u + 0x7ffffu + ((u >> 20) & 1u)) >> 20;
    byte = r - ((127u - 15u) << 3);
    scale = __uint_as_float(r << 20);
  } else {                       // multiples of 2^-17
    const float n = rintf(y * 131072.f);
    byte = static_cast<uint32_t>(n);
    scale = n * 7.62939453125e-06f;
  }
  // a zero scale: top is below half of the smallest, and all codes are zero
  const float r = byte ? __frcp_rn(scale) : 0.f;
  const unsigned long long r2 = pack_f2(r, r), s2 = pack_f2(-scale, -scale);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const unsigned long long v = pack_f2(x[i], x[i + 1]);
    const unsigned long long q = ffma2_rn(v, r2, 0ull);
    const unsigned long long z = ffma2_rn(ffma2_rn(q, s2, v), r2, q);
    x[i] = lo_f(z);
    x[i + 1] = hi_f(z);
  }
  return byte;
}

// Four pairs of values as four bytes of codes (a pair's first value in the low nibble), nearest even, at most 6.
__device__ __forceinline__ uint32_t codes8(float a0, float a1, float b0, float b1, float c0, float c1, float d0, float d1) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1), "f"(d0), "f"(d1));
  return w;
}

// Bound by memory (256 values in and 144 bytes out a token and head): the loads of a tile are all in flight before the
// first is used (32768 tokens x 8 heads from bf16 47 -> 40 us, 4.3 TB/s; 131072 tokens 144 us, 4.8 TB/s).
template <typename T>
__global__ void __launch_bounds__(kRowsThreads) kv4_write_kernel(const __grid_constant__ Kv4RowsParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const Kv4View& c = p.c;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int r0 = p.cu[b];
  const int p1 = kv4_len(c, b);
  const int n = min(p.cu[b + 1] - r0, p.n_rows - r0);
  const int p0 = max(0, p1 - n);
  const int first = r0 + n - p1;   // row of position 0 (may be negative)
  if (n <= 0 || r0 < 0 || p1 <= 0) return;
  const int t0 = p0 / kTileTok, t1 = (p1 + kTileTok - 1) / kTileTok;
  const long long items = static_cast<long long>(t1 - t0) * c.Hkv;
  const long long stride = static_cast<long long>(gridDim.x) * (kRowsThreads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kRowsThreads / 32) + (threadIdx.x >> 5); it < items;
       it += stride) {
    const int t = t0 + static_cast<int>(it / c.Hkv), h = static_cast<int>(it % c.Hkv);
    const int page = kv4_page(c, b, t);
    if (page < 0) continue;
    uint8_t* tile = c.cache + kv4_tile_offset(c, page, h, t);
    const int pos = t * kTileTok;
    uint2* sw = reinterpret_cast<uint2*>(tile + kOffScale) + lane;
    const bool whole = pos >= p0 && pos + kTileTok <= p1;
    const int r = lane >> 2, q = lane & 3;
    Raw<T> kr[2][2], vr[2][2];
    auto load_k = [&]() {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int pk = pos + half * 8 + r;
        const bool in = pk >= p0 && pk < p1;
        const uint8_t* row = p.k + (static_cast<long long>(first) + pk) * p.k_tok + h * p.k_head + q * 32 * sizeof(T);
        kr[half][0].load(row, in);
        kr[half][1].load(row + 16 * sizeof(T), in);
      }
    };
    auto load_v = [&]() {
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pv = pos + half * 8 + 2 * q + e;
          vr[half][e].load(p.v + (static_cast<long long>(first) + pv) * p.v_tok + h * p.v_head + r * 16 * sizeof(T),
                           pv >= p0 && pv < p1);
        }
    };
    load_k();
    if (sizeof(T) == 2) load_v();                      // 64 registers in flight for either width
    uint2 scales = whole ? make_uint2(0u, 0u) : *sw;   // tokens that stay keep their bytes
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int pk = pos + half * 8 + r;
      float x[16], y[16];
      Elem<T>::widen(kr[half][0], x);
      Elem<T>::widen(kr[half][1], y);
      const uint32_t s = quantise16(x) | (quantise16(y) << 8);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float *a = x + 8 * i, *e = y + 8 * i;
        w[i] = codes8(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7]);
        w[2 + i] = codes8(e[0], e[1], e[2], e[3], e[4], e[5], e[6], e[7]);
      }
      if (pk >= p0 && pk < p1) {
        reinterpret_cast<uint4*>(tile + half * 512)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
        scales.x = (scales.x & ~(0xffffu << (16 * half))) | (s << (16 * half));
      }
    }
    if (sizeof(T) == 4) load_v();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int pv = pos + half * 8 + 2 * q;
      const bool in0 = pv >= p0 && pv < p1, in1 = pv + 1 >= p0 && pv + 1 < p1;
      float x[16], y[16];
      Elem<T>::widen(vr[half][0], x);
      Elem<T>::widen(vr[half][1], y);
      const uint32_t s0 = quantise16(x), s1 = quantise16(y);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = codes8(x[4 * i], y[4 * i], x[4 * i + 1], y[4 * i + 1], x[4 * i + 2], y[4 * i + 2], x[4 * i + 3], y[4 * i + 3]);
      if (in0 || in1) {
        uint4* at = reinterpret_cast<uint4*>(tile + kOffV + half * 512) + lane;
        const uint32_t keep = (in0 ? 0u : 0x0f0f0f0fu) | (in1 ? 0u : 0xf0f0f0f0u);
        if (keep) {
          const uint4 old = *at;
          w[0] = (w[0] & ~keep) | (old.x & keep);
          w[1] = (w[1] & ~keep) | (old.y & keep);
          w[2] = (w[2] & ~keep) | (old.z & keep);
          w[3] = (w[3] & ~keep) | (old.w & keep);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
        const uint32_t m = (in0 ? 0xffu : 0u) | (in1 ? 0xff00u : 0u);
        scales.y = (scales.y & ~(m << (16 * half))) | (((s0 | (s1 << 8)) & m) << (16 * half));
      }
    }
    *sw = scales;
  }
}

// Byte offset of 16-byte piece c (eight fp16 values) of row `row` in a warp's 16 x 256 byte stage. The swizzle lets the
// eight lanes that store together, of both layouts, meet eight different pieces of the banks.
__device__ __forceinline__ uint32_t stage_at(int row, int c) {
  const int swizzle = ((c >> 3) & 1) ^ (((row >> 1) & 1) | ((row & 1) << 1) | (((row >> 2) & 1) << 2));
  return row * 256 + ((c ^ swizzle) << 4);
}

// The stage's rows [from, to) to rows of T, coalesced; `out`: row 0.
template <typename T>
__device__ __forceinline__ void store_rows(const uint8_t* stage, uint8_t* out, long long stride, int from, int to) {
  const int lane = threadIdx.x & 31;
  if constexpr (sizeof(T) == 4) { // a row an instruction
#pragma unroll 4
    for (int row = 0; row < kTileTok; ++row) {
      const uint2 h = *reinterpret_cast<const uint2*>(stage + stage_at(row, lane >> 1) + (lane & 1) * 8);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
      if (row >= from && row < to)
        reinterpret_cast<float4*>(out + row * stride)[lane] = make_float4(a.x, a.y, b.x, b.y);
    }
  } else {                        // two
#pragma unroll 4
    for (int k = 0; k < kTileTok / 2; ++k) {
      const int row = 2 * k + (lane >> 4);
      const uint4 h = *reinterpret_cast<const uint4*>(stage + stage_at(row, lane & 15));
      if (row >= from && row < to)
        reinterpret_cast<uint4*>(out + row * stride)[lane & 15] =
            make_uint4(Elem<T>::of(h.x), Elem<T>::of(h.y), Elem<T>::of(h.z), Elem<T>::of(h.w));
    }
  }
}

// Bound by memory: 144 bytes in and 256 values out a token and head. Values pass through shared memory as fp16
// (exact), so that rows leave in whole lines (131072 tokens x 8 heads to bf16 148 -> 108 us, 6.35 TB/s).
template <typename T>
__global__ void __launch_bounds__(kRowsThreads) kv4_read_kernel(const __grid_constant__ Kv4RowsParams p) {
  __shared__ __align__(16) uint8_t stages[kRowsThreads / 32][kTileTok * 256];
  pdl_wait();
  pdl_launch_dependents();
  const Kv4View& c = p.c;
  const int lane = threadIdx.x & 31;
  uint8_t* stage = stages[threadIdx.x >> 5];
  const int b = blockIdx.y;
  const int r0 = p.cu[b];
  const int p0 = p.start[b];
  const int n = min(p.cu[b + 1] - r0, p.n_rows - r0);
  if (n <= 0 || r0 < 0 || p0 < 0) return;
  const long long cap = static_cast<long long>(c.max_pages) << (c.page_tiles_log2 + 4);
  const int p1 = static_cast<int>(min(static_cast<long long>(p0) + n, cap));
  const int t0 = p0 / kTileTok, t1 = (p1 + kTileTok - 1) / kTileTok;
  const long long items = static_cast<long long>(t1 - t0) * c.Hkv;
  const long long stride = static_cast<long long>(gridDim.x) * (kRowsThreads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kRowsThreads / 32) + (threadIdx.x >> 5); it < items;
       it += stride) {
    const int t = t0 + static_cast<int>(it / c.Hkv), h = static_cast<int>(it % c.Hkv);
    const int page = kv4_page(c, b, t);
    uint4 code[4] = {};
    uint2 sc = make_uint2(0u, 0u);
    if (page >= 0) {
      const uint8_t* tile = c.cache + kv4_tile_offset(c, page, h, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) code[i] = __ldg(reinterpret_cast<const uint4*>(tile + i * 512) + lane);
      sc = __ldg(reinterpret_cast<const uint2*>(tile + kOffScale) + lane);
    }
    const int pos = t * kTileTok;
    const int from = max(0, p0 - pos), to = min(kTileTok, p1 - pos);
    const long long row0 = static_cast<long long>(r0) + (pos - p0);
    const int r = lane >> 2, q = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t w[4] = {code[half].x, code[half].y, code[half].z, code[half].w};
      const uint32_t sa = scale_both(sc.x, 2 * half), sb = scale_both(sc.x, 2 * half + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t f[4];
        e2m1_to_f16x2(w[i], f[0], f[1], f[2], f[3]);
        const uint32_t s = i < 2 ? sa : sb;
        *reinterpret_cast<uint4*>(stage + stage_at(half * 8 + r, q * 4 + i)) =
            make_uint4(hmul2(f[0], s), hmul2(f[1], s), hmul2(f[2], s), hmul2(f[3], s));
      }
    }
    __syncwarp();
    store_rows<T>(stage, p.k + row0 * p.k_tok + h * p.k_head, p.k_tok, from, to);
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t w[4] = {code[2 + half].x, code[2 + half].y, code[2 + half].z, code[2 + half].w};
      const uint32_t s = scale_pair(sc.y, 2 * half);
#pragma unroll
      for (int i = 0; i < 2; ++i) {      // (token, token + 1) pairs to (dim, dim + 1) pairs, eight dims at a time
        uint32_t f[8];
        e2m1_to_f16x2(w[2 * i], f[0], f[1], f[2], f[3]);
        e2m1_to_f16x2(w[2 * i + 1], f[4], f[5], f[6], f[7]);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = hmul2(f[k], s);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t sel = e ? 0x7632u : 0x5410u;
          *reinterpret_cast<uint4*>(stage + stage_at(half * 8 + 2 * q + e, 2 * r + i)) =
              make_uint4(__byte_perm(f[0], f[1], sel), __byte_perm(f[2], f[3], sel), __byte_perm(f[4], f[5], sel),
                         __byte_perm(f[6], f[7], sel));
        }
      }
    }
    __syncwarp();
    store_rows<T>(stage, p.v + row0 * p.v_tok + h * p.v_head, p.v_tok, from, to);
    __syncwarp();
  }
}

template <typename T, bool kWrite>
cudaError_t launch_rows(const Kv4RowsParams& p, int max_tiles, cudaStream_t stream, bool pdl) {
  const long long warps = static_cast<long long>(max_tiles) * p.c.Hkv;
  const long long blocks = (warps + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < 1 ? 1 : blocks > 65536 ? 65536 : blocks), p.c.B);
  cfg.blockDim = dim3(kRowsThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (kWrite) return cudaLaunchKernelEx(&cfg, kv4_write_kernel<T>, p);
  return cudaLaunchKernelEx(&cfg, kv4_read_kernel<T>, p);
}

template <bool kWrite>
cudaError_t launch_rows_of(int dtype, const Kv4RowsParams& p, int max_tiles, cudaStream_t stream, bool pdl) {
  switch (dtype) {
    case HSA_F32: return launch_rows<float, kWrite>(p, max_tiles, stream, pdl);
    case HSA_BF16: return launch_rows<__nv_bfloat16, kWrite>(p, max_tiles, stream, pdl);
    case HSA_F16: return launch_rows<__half, kWrite>(p, max_tiles, stream, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_kv4_write(int dtype, const Kv4RowsParams& p, int max_tiles, cudaStream_t stream, bool pdl) {
  return launch_rows_of<true>(dtype, p, max_tiles, stream, pdl);
}
cudaError_t launch_kv4_read(int dtype, const Kv4RowsParams& p, int max_tiles, cudaStream_t stream, bool pdl) {
  return launch_rows_of<false>(dtype, p, max_tiles, stream, pdl);
}

}  // namespace pqhsa
