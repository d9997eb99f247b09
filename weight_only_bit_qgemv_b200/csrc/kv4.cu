// kv4_append and kv4_gather: rows into the 4-bit paged cache and back out (layout in kv4.cuh).
//
// Both are bound by memory: append reads 2 * dim values a token and key head and writes
// 2 * (dim / 2 + dim / 16) bytes. A warp's piece is one token and two key heads, a lane's four
// consecutive values of a row, so that a row is read in whole 128-byte lines, a block's maximum
// is three shuffles among eight lanes, and a lane's four codes are one 16-bit store into the row's
// 64 bytes. The loads of both heads' keys and values are issued before any is used.
//
// Measured (8 key heads, dim 128, float32, a cold L2, a launch's time included): 39,151 tokens are appended in 93 us
// (3.9 TB/s: the quantiser's instructions, 60 % of the cycles on the integer pipe) and gathered in 77 us (4.8 TB/s);
// 64 tokens in 3 us each. A fourth block of 256 threads an SM, 64 registers: appending 10 % slower; 4 or 16 pieces
// a warp instead of 8: 3 to 15 %.
#include <algorithm>

#include "kv4.cuh"
#include "ptx.cuh"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kThreads = 128;
constexpr int kHeadsPerWarp = 2;

// Where a lane's four values of a row are kept: the 16-bit halfword of the row.
// Halfword h = 8 b + 2 t + e of a key row (block b, word t, half e of it), 8 b + g of a value row.
template <int D>
__device__ __forceinline__ int key_halfword(int h) {
  constexpr int NB = D / 32;
  return ((h >> 1 & 3) * NB + (h >> 3)) * 2 + (h & 1);
}
template <int D>
__device__ __forceinline__ int value_halfword(int h) {
  constexpr int NB = D / 32;
  return (h & 7) * NB + (h >> 3);
}

// One block's scale and this lane's four codes of it (eight neighbouring lanes hold the block).
// The arithmetic is qpack's, bit for bit: a = max |x|, s = binary16(a / 7), code = clamp(round(x / s), -8, 7).
// Done as written it takes 200 instructions a row and the kernel runs at a third of the memory's rate. So both
// quotients are approximated, and computed as written only where the approximation could round otherwise:
//   - a * (1 / 7) is off by less than 2 ulp: written out where its 13 bits below binary16's are within 4 of a half,
//     or where binary16 is subnormal (then the code may need the clamp, too);
//   - x * (1 / s) + 192.5, whose last bit is 2^-16, is off by less than 2^-16: written out where its 16 fraction bits
//     are within 1 of a whole number, which is 0 to 2 after adding that 1. Above them, from the third byte on, is
//     round(x / s) in two's complement.
// Written out, x / s is a correctly rounded 32-bit quotient. That is enough: s has 11 significant bits, so
// (k + 1/2) s is exact in 24, and an x next to it differs from it by at least an ulp of x, more than 2^-24 of it,
// while half an ulp of the quotient is at most 2^-24 of it: a quotient that is not a tie cannot become one.
// A block with a NaN or with a scale beyond binary16 becomes NaN as a whole: scale NaN, codes 0.
__device__ __forceinline__ uint32_t quantise(float4 x, uint16_t *scale) {
  float a;  // NaN if one of them is
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(x.x), "f"(x.y), "f"(x.z));
  asm("max.NaN.abs.f32 %0, %0, %1, %1;" : "+f"(a) : "f"(x.w));
#pragma unroll
  for (int i = 1; i < 8; i <<= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, a, i);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(other));
  }
  const float q = a * 0.142857142857f;
  __half h = __float2half_rn(q);
  bool exactly = q < 6.2e-5f;
  if (exactly || ((__float_as_uint(q) + 4u - 0x1000u) & 0x1fffu) <= 8u)
    h = __double2half(__ddiv_rn(static_cast<double>(a), 7.0));
  const float s = __half2float(h);
  if (!(s < INFINITY)) {
    *scale = 0x7fffu;
    return 0;
  }
  *scale = __half_as_ushort(h);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const float v[4] = {x.x, x.y, x.z, x.w};
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = __float_as_uint(fmaf(v[i], inv, 192.5f + 0x1p-16f));
  const uint32_t least = min(__vimin3_u32(t[0] << 16, t[1] << 16, t[2] << 16), t[3] << 16) >> 16;
  uint32_t code = (__byte_perm(t[0], t[2], 0x0062) & 0x0f0fu) | (__byte_perm(t[1], t[3], 0x0062) << 4 & 0xf0f0u);
  if (exactly || least <= 2u) {
    code = 0;
    if (s != 0.0f) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        code |= (static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(v[i], s)), -8.0f), 7.0f))) & 15u)
                << 4 * i;
    }
  }
  return code;
}

struct Place {
  bool in;        // the row belongs to a sequence
  int64_t page;   // its page, -1 if the table has none for it
  int slot;
};

__device__ __forceinline__ Place place_of(int64_t t, const int32_t *cu, const int32_t *start, int batch,
                                          const int32_t *table, int64_t width, int shift, int64_t pages) {
  Place p{false, -1, 0};
  const int b = sequence_of(cu, batch, t);
  if (b < 0) return p;
  p.in = true;
  const int64_t first = start ? start[b] : 0;
  const int64_t at = first + (t - cu[b]);
  const int64_t e = at >> shift;
  if (first < 0 || e >= width) return p;
  const int32_t page = table[b * width + e];
  if (page < 0 || page >= pages) return p;
  p.page = page;
  p.slot = static_cast<int>(at & ((int64_t(1) << shift) - 1));
  return p;
}

struct Args {
  woq_rows k, v;
  uint8_t *codes;
  uint16_t *scales;
  int64_t pages, tokens, width;
  const int32_t *cu, *start, *table;
  int batch, shift, heads, chunks;  // chunks: pairs of key heads of a token
  int64_t per;                      // pieces of a warp
};

// Lanes of a warp that work on one row: D / 4. At D = 64 the lower half has the key row, the upper
// the value row; at D = 128 the whole warp has the key row, then the value row.
//
// A warp takes `per` consecutive pieces (a token's pair of heads), so that it looks a token's page up once, and
// appending, it has the next piece's rows under way while it quantises this one's.
template <int D, bool APPEND, bool F32>
__global__ void __launch_bounds__(kThreads) kv4_rows_kernel(const Args a) {
  constexpr int NB = D / 32, LANES = D / 4, ROWS = 2 * D / 128;  // ROWS: rows a lane has of each head
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t items = a.tokens * a.chunks;
  const int part = lane / LANES;  // D = 64: 0 the key row, 1 the value row
  const int h = lane % LANES;     // halfword of the row, four values
  const int64_t page = int64_t(1) << a.shift;
  const int64_t first = (blockIdx.x * int64_t(kThreads / 32) + (threadIdx.x >> 5)) * a.per;
  const int64_t last = first + a.per < items ? first + a.per : items;
  if (first >= last) return;
  int64_t t = first / a.chunks;
  int chunk = static_cast<int>(first % a.chunks);
  // This lane's rows: keys and values, or one of them. `at`: its values of the first head of the piece at hand, in
  // elements, which goes on by additions.
  woq_rows rows[ROWS];
  int64_t at[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    rows[r] = (ROWS == 2 ? r : part) ? a.v : a.k;
    if (F32) rows[r].dtype = WOQ_F32;
    at[r] = t * rows[r].row_stride + chunk * kHeadsPerWarp * rows[r].head_stride + 4 * h;
  }
  auto load = [&](int h0, float4 (&x)[kHeadsPerWarp][ROWS]) {
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp; ++i)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        x[i][r] = make_float4(0, 0, 0, 0);
        if (h0 + i < a.heads) x[i][r] = load4(rows[r].data, at[r] + i * rows[r].head_stride, rows[r].dtype);
      }
  };
  float4 next[kHeadsPerWarp][ROWS];
  if constexpr (APPEND) load(chunk * kHeadsPerWarp, next);
  Place p = place_of(t, a.cu, a.start, a.batch, a.table, a.width, a.shift, a.pages);
  for (int64_t item = first; item < last; ++item) {
    const int h0 = chunk * kHeadsPerWarp;
    const int64_t token = t;
    const Place at_page = p;
    int64_t here[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      here[r] = at[r];
      at[r] += kHeadsPerWarp * rows[r].head_stride;
    }
    if (++chunk == a.chunks) {
      chunk = 0;
      ++t;
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        at[r] += rows[r].row_stride - int64_t(a.chunks) * kHeadsPerWarp * rows[r].head_stride;
    }
    float4 x[kHeadsPerWarp][ROWS];
    if constexpr (APPEND) {
#pragma unroll
      for (int i = 0; i < kHeadsPerWarp; ++i)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) x[i][r] = next[i][r];
      if (item + 1 < last) load(chunk * kHeadsPerWarp, next);
    }
    if (t != token && item + 1 < last)
      p = place_of(t, a.cu, a.start, a.batch, a.table, a.width, a.shift, a.pages);
    if (!at_page.in || (APPEND && at_page.page < 0)) continue;  // warp-uniform
    // This lane's halfword and scale of the first head's rows; the others are whole pages of rows on.
    const int64_t head0 = at_page.page < 0 ? 0 : at_page.page * a.heads + h0;
    const int64_t row_step = page * (D / 4), scale_step = page * 2 * NB;
    uint16_t *codes[ROWS], *scales[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int kv = ROWS == 2 ? r : part;
      codes[r] = reinterpret_cast<uint16_t *>(a.codes) + head0 * 2 * row_step + at_page.slot * (D / 4) +
                 (kv ? row_step + value_halfword<D>(h) : key_halfword<D>(h));
      scales[r] = a.scales + head0 * scale_step + at_page.slot * 2 * NB + kv * NB + h / 8;
    }
    uint16_t sc[kHeadsPerWarp][ROWS], w[kHeadsPerWarp][ROWS];
    if constexpr (!APPEND) {
#pragma unroll
      for (int i = 0; i < kHeadsPerWarp; ++i)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          sc[i][r] = w[i][r] = 0;
          if (h0 + i >= a.heads || at_page.page < 0) continue;
          w[i][r] = codes[r][2 * i * row_step];
          sc[i][r] = scales[r][i * scale_step];
        }
    }
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp; ++i) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (h0 + i >= a.heads) continue;  // warp-uniform
        if constexpr (APPEND) {
          uint16_t s;
          const uint32_t c = quantise(x[i][r], &s);
          codes[r][2 * i * row_step] = static_cast<uint16_t>(c);
          if ((h & 7) == 0) scales[r][i * scale_step] = s;
        } else {
          const float s = __half2float(__ushort_as_half(sc[i][r]));
          const int c = static_cast<int>(w[i][r]) << 16;  // sign-extend each nibble from the top
          store4(rows[r].data, here[r] + i * rows[r].head_stride, rows[r].dtype,
                 make_float4(s * static_cast<float>(c << 12 >> 28), s * static_cast<float>(c << 8 >> 28),
                             s * static_cast<float>(c << 4 >> 28), s * static_cast<float>(c >> 28)));
        }
      }
    }
  }
}

template <int D, bool APPEND, bool F32>
int launch(const Args &a, cudaStream_t s, const DevInfo &dev) {
  // One piece a warp while they fit the device at once, then as many waves as keep a warp at 8 at most.
  const int64_t items = a.tokens * a.chunks, in_block = kThreads / 32;
  Args b = a;
  b.per = std::min<int64_t>(8, std::max<int64_t>(1, items / (int64_t(dev.sm_count) * in_block * 8)));
  const int64_t warps = (items + b.per - 1) / b.per;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + in_block - 1) / in_block), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv4_rows_kernel<D, APPEND, F32>, b) != cudaSuccess) return WOQ_ECUDA;
  count_launches(1);
  return WOQ_OK;
}

}  // namespace

int launch_kv4_rows(const woq_kv4 &c, const woq_rows &k, const woq_rows &v, int64_t tokens, const int32_t *cu,
                    const int32_t *start, int32_t batch, const int32_t *table, int64_t width, bool append,
                    cudaStream_t s, const DevInfo &dev) {
  Args a;
  a.k = k;
  a.v = v;
  a.codes = c.codes;
  a.scales = c.scales;
  a.pages = c.pages;
  a.tokens = tokens;
  a.width = width;
  a.cu = cu;
  a.start = start;
  a.table = table;
  a.batch = batch;
  a.shift = __builtin_ctz(static_cast<unsigned>(c.page));
  a.heads = c.kv_heads;
  a.chunks = (c.kv_heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
  // float32 rows have kernels of their own: looking at the type takes as long as the address of a load.
  const bool f32 = k.dtype == WOQ_F32 && v.dtype == WOQ_F32;
  if (c.dim == 128)
    return append ? f32 ? launch<128, true, true>(a, s, dev) : launch<128, true, false>(a, s, dev)
           : f32  ? launch<128, false, true>(a, s, dev)
                  : launch<128, false, false>(a, s, dev);
  return append ? f32 ? launch<64, true, true>(a, s, dev) : launch<64, true, false>(a, s, dev)
         : f32  ? launch<64, false, true>(a, s, dev)
                : launch<64, false, false>(a, s, dev);
}

}  // namespace woq
