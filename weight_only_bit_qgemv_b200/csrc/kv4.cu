// kv4_append and kv4_gather: rows into the 4-bit paged cache and back out (layout in kv4.cuh).
//
// Both are bound by memory: append reads 2 * dim values a token and key head and writes
// 2 * (dim / 2 + dim / 16) bytes. A warp takes one token and two key heads, a lane four
// consecutive values of a row, so that a row is read in whole 128-byte lines, a block's maximum
// is three shuffles among eight lanes, and a lane's four codes are one 16-bit store into the row's
// 64 bytes. The loads of both heads' keys and values are issued before any is used.
#include <algorithm>

#include "kv4.cuh"
#include "ptx.cuh"
#include "woq_internal.h"

namespace woq {
namespace {

constexpr int kThreads = 256;
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
// The arithmetic is qpack's: a = max |x|, s = binary16(a / 7), code = clamp(round(x / s)).
// a / 7 is rounded once, from 64 bits. x / s needs only a correctly rounded 32-bit quotient: s has
// 11 significant bits, so (k + 1/2) s is exact in 24, and an x next to it differs from it by at
// least an ulp of x, more than 2^-24 of it, while half an ulp of the quotient is at most 2^-24 of
// it: a quotient that is not a tie cannot become one. A block with a NaN or with a scale beyond
// binary16 becomes NaN as a whole: scale NaN, codes 0.
__device__ __forceinline__ uint32_t quantise(float4 x, uint16_t *scale) {
  float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
  bool bad = isnan(x.x) || isnan(x.y) || isnan(x.z) || isnan(x.w);
#pragma unroll
  for (int i = 1; i < 8; i <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, i));
  const uint32_t mine = 0xffu << (threadIdx.x & 24);
  bad = (__ballot_sync(0xffffffffu, bad) & mine) != 0;
  const __half h = __double2half(__ddiv_rn(static_cast<double>(a), 7.0));
  bad = bad || __hisinf(h);
  *scale = bad ? 0x7fffu : __half_as_ushort(h);
  const float s = __half2float(h);
  if (bad || s == 0.0f) return 0;
  auto code = [s](float v) {
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(v, s)), -8.0f), 7.0f))) & 15u;
  };
  return code(x.x) | code(x.y) << 4 | code(x.z) << 8 | code(x.w) << 12;
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
};

// Lanes of a warp that work on one row: D / 4. At D = 64 the lower half has the key row, the upper
// the value row; at D = 128 the whole warp has the key row, then the value row.
template <int D, bool APPEND>
__global__ void __launch_bounds__(kThreads) kv4_rows_kernel(const Args a) {
  constexpr int NB = D / 32, LANES = D / 4, ROWS = 2 * D / 128;  // ROWS: rows a lane has of each head
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t items = a.tokens * a.chunks;
  const int part = lane / LANES;  // D = 64: 0 the key row, 1 the value row
  const int h = lane % LANES;     // halfword of the row, four values
  for (int64_t item = blockIdx.x * int64_t(kThreads / 32) + (threadIdx.x >> 5); item < items;
       item += int64_t(gridDim.x) * (kThreads / 32)) {
    const int64_t t = item / a.chunks;
    const int h0 = static_cast<int>(item % a.chunks) * kHeadsPerWarp;
    const Place p = place_of(t, a.cu, a.start, a.batch, a.table, a.width, a.shift, a.pages);
    if (!p.in || (APPEND && p.page < 0)) continue;  // warp-uniform
    const int64_t page = int64_t(1) << a.shift;
    float4 x[kHeadsPerWarp][ROWS];
    uint16_t sc[kHeadsPerWarp][ROWS], w[kHeadsPerWarp][ROWS];
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp; ++i) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        x[i][r] = make_float4(0, 0, 0, 0);
        sc[i][r] = w[i][r] = 0;
        const int hd = h0 + i, kv = ROWS == 2 ? r : part;
        if (hd >= a.heads) continue;
        if constexpr (APPEND) {
          const woq_rows &src = kv ? a.v : a.k;
          x[i][r] = load4(src.data, t * src.row_stride + hd * src.head_stride + 4 * h, src.dtype);
        } else if (p.page >= 0) {
          const int64_t base = (p.page * a.heads + hd) * 2;
          const int at = kv ? value_halfword<D>(h) : key_halfword<D>(h);
          w[i][r] = reinterpret_cast<const uint16_t *>(a.codes)[((base + kv) * page + p.slot) * (D / 4) + at];
          sc[i][r] = a.scales[(base / 2 * page + p.slot) * 2 * NB + kv * NB + h / 8];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp; ++i) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int hd = h0 + i, kv = ROWS == 2 ? r : part;
        if (hd >= a.heads) continue;  // warp-uniform
        const int64_t base = (p.page * a.heads + hd) * 2;
        if constexpr (APPEND) {
          uint16_t s;
          const uint32_t c = quantise(x[i][r], &s);
          const int at = kv ? value_halfword<D>(h) : key_halfword<D>(h);
          reinterpret_cast<uint16_t *>(a.codes)[((base + kv) * page + p.slot) * (D / 4) + at] =
              static_cast<uint16_t>(c);
          if ((h & 7) == 0) a.scales[(base / 2 * page + p.slot) * 2 * NB + kv * NB + h / 8] = s;
        } else {
          const woq_rows &dst = kv ? a.v : a.k;
          const float s = __half2float(__ushort_as_half(sc[i][r]));
          const int c = static_cast<int>(w[i][r]) << 16;  // sign-extend each nibble from the top
          store4(dst.data, t * dst.row_stride + hd * dst.head_stride + 4 * h, dst.dtype,
                 make_float4(s * static_cast<float>(c << 12 >> 28), s * static_cast<float>(c << 8 >> 28),
                             s * static_cast<float>(c << 4 >> 28), s * static_cast<float>(c >> 28)));
        }
      }
    }
  }
}

template <int D, bool APPEND>
int launch(const Args &a, cudaStream_t s, const DevInfo &dev) {
  const int64_t warps = a.tokens * a.chunks, per = kThreads / 32;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((warps + per - 1) / per, int64_t(dev.sm_count) * 8)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv4_rows_kernel<D, APPEND>, a) != cudaSuccess) return WOQ_ECUDA;
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
  if (c.dim == 128) return append ? launch<128, true>(a, s, dev) : launch<128, false>(a, s, dev);
  return append ? launch<64, true>(a, s, dev) : launch<64, false>(a, s, dev);
}

}  // namespace woq
