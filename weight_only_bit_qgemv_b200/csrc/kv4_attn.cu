// kv4_attn: one query token a sequence against its cached keys and values, held in 4 bits.
//   s_j = scale q . k_j,   p = softmax(s over the sequence's tokens),   o = sum_j p_j v_j
// with k_j[d] = ks[j, d / 32] * kc[j, d] and v_j likewise (binary16 scales, int4 codes).
//
// Bound: memory. A token and key head is dim + dim / 8 bytes for 4 * dim * (query heads a key head)
// flop; 144 bytes at dim 128. On the CUDA cores the unpacking and one multiply a query head would
// already exceed what the bytes' time leaves, so both products run as warp matrix instructions
// (mma.sync m16n8k16, binary16 in, FP32 out): two codes become two binary16 numbers with one logic
// instruction and one exact subtraction. tcgen05 would want the codes widened fourfold in shared
// memory first, and its 128 rows would be 94 % empty at 8 query heads.
//
// FP32 accuracy: the 16 rows of the left operand are 8 query heads' high binary16 parts and the
// same heads' low parts, so that 22 bits of q, and then of p_j * vs[j, block], take part. The
// query is scaled by a power of two into binary16's range, the value scales likewise (see `room`) where
// those of 32 tokens lie within 2^13 of one another. Where they do not, or some are 0, the products p_j * vs[j, block]
// are made in FP32, and each head and block gets a power of two of its own. Per
// block of 32 the key scale multiplies an FP32 block sum. Sums inside the matrix instructions, which cut
// off what lies below their last bit, run over 32 tokens; from there on they are FP32 additions,
// rounded to nearest. (A masked nibble is a binary16 as it stands, the subnormal u * 2^-24, and the offset
// could be taken off the sums: measured, the matrix instructions then keep 18 bits instead of 26, as they
// align subnormals as if they were 2^-14, and u >= 0 makes what they cut off a drift: 1.7e-4 of
// the result at 115,000 tokens.)
//
// The left operand of the second product is the result of the first without leaving its registers.
//
// Split: all sequences' tokens, in units of 32 per (sequence, key head), are one line that is cut into
// equal parts, a block's each, whatever the lengths are: the lengths are read on the device. A part that
// covers only some of a (sequence, key head) leaves its sum, maximum and total in the workspace;
// the last of the blocks concerned adds them in the order of the tokens (the same bits on every call).
//
// Each warp takes every fourth unit through its own ring of shared memory, filled by bulk copies
// (three per 16 tokens: keys, values, scales are each contiguous within a page). Three blocks of four warps with
// two units each under way keep 110 KB an SM in flight; more blocks or stages gained nothing.
//
// Measured (8 key heads, dim 128): 1 x 1000 tokens 9.9 us, 64 sequences of 1 to 8191 130 us
// (2.3 TB/s), 4 of 100,000 to 131,072 175 us (3.0 TB/s), 16 of 2049 to 16,001 with 8 query heads a key head 70 us; FP32
// products in every unit are 23 % slower.
// What holds it back is not the bytes but 27 instructions a token and key head, issued in 54 % of the
// cycles: three warps a scheduler, whose registers are full, do not cover one another's latencies better.
#include <algorithm>
#include <mutex>

#include "kv4.cuh"
#include "ptx.cuh"
#include "woq_internal.h"

namespace woq {

__device__ unsigned int g_kv4_timeout_flag = 0;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlocksPerSm = 3;
constexpr int kUnit = 32;      // tokens of a unit
constexpr int kStages = 2;     // units in a warp's ring
constexpr int kHeads = 8;      // query heads of a pass: half the rows of a matrix instruction
constexpr int kTop = 14;       // weights reach 2^14, which binary16 holds
constexpr int kFall = 40;      // how far a unit's reference may be below the largest one so far, as a power of two
constexpr int kMoreUnits = 8;  // units that a part may have more so that parts begin and end with their sequences
constexpr long long kWaitLimit = 1LL << 32;  // cycles (~2 s)

template <int D>
struct Shape {
  static constexpr int NB = D / 32;                   // blocks of a row
  static constexpr int RowBytes = D / 2;
  static constexpr int ScaleBytes = 4 * NB;           // of a token: key and value
  static constexpr int Values = kUnit * RowBytes;     // a stage: keys, values, scales of 32 tokens
  static constexpr int Scales = 2 * kUnit * RowBytes;
  static constexpr int Stage = kUnit * (2 * RowBytes + ScaleBytes);
  // A partial result, floats: the heads' sums (rows four apart, so that eight heads' are in different banks),
  // their maxima and their totals.
  static constexpr int HeadStep = D + 4;
  static constexpr int Maxima = kHeads * HeadStep, Totals = Maxima + kHeads;
  static constexpr int Slot = Totals + kHeads;
};

struct Args {
  woq_rows q, o;
  const uint8_t *codes;
  const uint8_t *scales;
  const int32_t *lens, *table;
  int64_t pages, width;
  int batch, shift, kv_heads, group, chunks;
  float scale;
  unsigned *counters;
  float *partials;
  long long wait_limit, stuck_wait;
};

__device__ __forceinline__ void mma(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ __half2 h2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
__device__ __forceinline__ uint32_t u32(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }

// Two codes of a word as binary16: code, and 16 * code. The masked nibble with its sign bit turned
// over (u = code + 8) and an exponent is 1024 + u (1024 + 16 u); the subtraction is exact.
// (w & mask) ^ magic is one instruction if only the mask is an immediate: the magic numbers are kept in registers
// that the compiler does not know the contents of (it made two instructions of two immediates: 128 more a unit).
// Likewise a sum's start at zero: four registers for all instead of four moves for each.
struct Magic {
  uint32_t low, high;
  float zero[4];
  __device__ __forceinline__ Magic() {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("mov.b32 %0, 0;" : "=f"(zero[i]));
    asm volatile("mov.b32 %0, 0x64086408;" : "=r"(low));
    asm volatile("mov.b32 %0, 0x64806480;" : "=r"(high));
  }
};
__device__ __forceinline__ uint32_t low(uint32_t w, const Magic &m) {
  uint32_t u;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0x6a;" : "=r"(u) : "r"(w), "r"(m.low));
  return u32(__hsub2(h2(u), h2(m.low)));
}
__device__ __forceinline__ uint32_t high(uint32_t w, const Magic &m) {
  uint32_t u;
  asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0x6a;" : "=r"(u) : "r"(w), "r"(m.high));
  return u32(__hsub2(h2(u), h2(m.high)));
}

// 2^e as binary16, as its bits, where it has it: from its smallest number on to infinity.
__device__ __forceinline__ int half_bits(int e) { return e < -24 ? 1 : e < -14 ? 1 << (e + 24) : min(e + 15, 31) << 10; }
// The exponent of the binary16 number with these bits (neither 0 nor negative).
__device__ __forceinline__ int half_exponent(int bits) { return bits < 0x400 ? 7 - __clz(bits) : (bits >> 10) - 15; }

// a and b as binary16 high parts and binary16 remainders: 22 bits of each.
__device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}

// The token of a 16-token half that column 2 t + j of its matrix i (of two, 8 tokens each) holds: a quad
// lane's two tokens lie four apart, which spreads the value rows that a half-warp reads over all banks.
__device__ __forceinline__ int token_of(int i, int t, int j) { return 8 * i + t + 4 * j; }

template <int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) kv4_attn_kernel(const Args a) {
  using S = Shape<D>;
  constexpr int NB = S::NB;
  extern __shared__ __align__(128) uint8_t smem[];
  // [ring: kWarps * kStages * Stage][q operands: 2 NB * 32 * 16][results: kWarps * Slot][bars][fac, flags][prefix]
  uint8_t *ring = smem;
  uint4 *qop = reinterpret_cast<uint4 *>(smem + kWarps * kStages * S::Stage);
  float *results = reinterpret_cast<float *>(qop + 2 * NB * 32);
  uint64_t *bars = reinterpret_cast<uint64_t *>(results + kWarps * S::Slot);
  uint64_t *never = bars + kWarps * kStages;                         // nothing arrives on it
  float *fac = reinterpret_cast<float *>(never + 1);                 // [kHeads]
  int *flags = reinterpret_cast<int *>(fac + kHeads);                // abort, last, parts, sequences that have tokens
  int64_t *pre = reinterpret_cast<int64_t *>(flags + 4);             // [batch + 1]: units before a sequence

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  volatile int *abort = flags;
  const Magic magic;

  if (tid == 0) {
    for (int i = 0; i < kWarps * kStages + 1; ++i) ptx::mbar_init(&bars[i], 1);
    ptx::fence_mbar_init();
    flags[0] = 0;
    pre[0] = 0;
  }
  ptx::pdl_wait();

  // Units of each sequence, summed up.
  const int64_t longest = a.width << a.shift;
  auto units_of = [&](int b) -> int64_t {
    int64_t n = a.lens[b];
    n = n < 0 ? 0 : n > longest ? longest : n;
    return (n + kUnit - 1) / kUnit;
  };
  if (warp == 0) {
    int64_t carry = 0;
    int parts = 0, used = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      int64_t n = b0 + lane < a.batch ? units_of(b0 + lane) : 0;
      const int u = static_cast<int>(n);  // less than 2^26
      const int per = max(2, (31 - __clz(u | 1)) >> 1);  // log2 of a part's units: about half of u's
      parts += (u + (1 << per) - 1) >> per;
      used += n > 0;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int64_t m = __shfl_up_sync(0xffffffffu, n, i);
        if (lane >= i) n += m;
      }
      if (b0 + lane < a.batch) pre[b0 + lane + 1] = carry + n;
      carry += __shfl_sync(0xffffffffu, n, 31);
    }
    parts = __reduce_add_sync(0xffffffffu, parts);
    used = __reduce_add_sync(0xffffffffu, used);
    if (lane == 0) {
      flags[2] = parts;
      flags[3] = used;
    }
  }
  __syncthreads();

  const int heads = a.kv_heads * a.chunks;  // passes of a sequence: key heads times chunks of 8 query heads
  const int64_t total = pre[a.batch] * heads;
  // Parts. A unit more for each warp and four parts more to join take about as long, so a sequence of n units goes into
  // about sqrt(n) parts, of a power of two of units and one for each warp at least. Are these more than blocks, then
  // as many parts as blocks, or, if that costs a part few units, as many as give each key head of a sequence the
  // same number. Sequences of one length then have parts of their own, and a block enters one of them only: another
  // one costs it 4 us. Against equal parts of 4 units or more: 1 x 4000 tokens 27 -> 14 us, 8 x 300 17 -> 11,
  // 32 x 500 21 -> 16.
  const int64_t passes = static_cast<int64_t>(flags[3]) * heads;
  int64_t parts = static_cast<int64_t>(flags[2]) * heads;
  if (parts > gridDim.x) {
    parts = gridDim.x;
    const int64_t even = passes > 0 && passes <= parts ? parts / passes * passes : parts;
    if (total / even - total / parts <= kMoreUnits) parts = even;
  }

  // Sequences without tokens: zeros.
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if (pre[b + 1] != pre[b]) continue;
    const int n4 = a.kv_heads * a.group * (D / 4);
    for (int i = tid; i < n4; i += kThreads)
      store4(a.o.data, b * a.o.row_stride + (i / (D / 4)) * a.o.head_stride + 4 * (i % (D / 4)), a.o.dtype,
             make_float4(0, 0, 0, 0));
  }

  const int64_t begin = blockIdx.x < parts ? blockIdx.x * total / parts : 0;
  const int64_t end = blockIdx.x < parts ? (blockIdx.x + 1) * total / parts : 0;
  uint32_t phases = 0;  // parity of each stage of this warp's ring
  uint8_t *mine = ring + warp * kStages * S::Stage;
  uint64_t *bar = bars + warp * kStages;

  // A unit's copies: lane 2 i + h of the first six has the 16 tokens of half h, i = 0 their keys,
  // 1 values, 2 scales, and keeps the table's entry of its half for the unit that is next to copy.
  const int half = lane & 1, what = lane >> 1, page = 1 << a.shift;
  const int unit_bytes = what == 2 ? S::ScaleBytes : S::RowBytes;
  const int64_t page_bytes = int64_t(a.kv_heads) * page * (what == 2 ? S::ScaleBytes : 2 * S::RowBytes);
  uint8_t *into = mine + what * S::Values + 16 * half * unit_bytes;
  const uint32_t pages = static_cast<uint32_t>(a.pages);  // an entry outside, or negative, is no page
  int b = 0, units = 0, pass = 0, u_begin = 0, u_end = 0, len = 0, kvh = 0;
  const int32_t *row = a.table;
  const uint8_t *pool = a.codes;
  float query[kHeads / kWarps][NB];
  int32_t next = -1;     // the entry
  uint32_t there = 0;    // halves that have a page, of the units in the ring: 2 bits each, oldest first
  auto entry = [&](int u) -> int32_t {
    const uint32_t key = static_cast<uint32_t>(u) * kUnit + 16 * half;
    return u < u_end && key < static_cast<uint32_t>(len) ? row[key >> a.shift] : -1;
  };
  auto issue = [&](int u, int st, int32_t e) {
    const bool good = static_cast<uint32_t>(e) < pages;
    const uint32_t halves = __ballot_sync(0xffffffffu, good) & 3u;
    there = there >> 2 | halves << 2 * (kStages - 1);
    if (u >= u_end) return;
    if (lane == 0) ptx::mbar_arrive_expect_tx(&bar[st], __popc(halves) * (S::Stage / 2));
    if (lane < 6 && good) {
      const uint32_t slot = (static_cast<uint32_t>(u) * kUnit + 16 * half) & (page - 1);
      ptx::bulk_load(into + st * S::Stage, pool + e * page_bytes + slot * unit_bytes, 16 * unit_bytes, &bar[st]);
    }
  };
  // The sequence, key head and chunk of unit `cur`, and the copies of this warp's first units there. A sequence has
  // less than 2^31 tokens, so its units and their tokens fit 32 bits.
  auto enter = [&](int64_t cur) {
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] * heads <= cur) lo = mid;
      else hi = mid;
    }
    b = lo;
    units = static_cast<int>(pre[b + 1] - pre[b]);
    const int64_t at = cur - pre[b] * heads;
    pass = static_cast<int>(at / units);
    u_begin = static_cast<int>(at % units);
    u_end = u_begin + static_cast<int>(end - cur < units - u_begin ? end - cur : units - u_begin);
    kvh = pass / a.chunks;
    len = static_cast<int>(a.lens[b] > longest ? longest : a.lens[b]);
    row = a.table + b * a.width;
    pool = what == 2 ? a.scales + int64_t(kvh) * page * S::ScaleBytes
                     : a.codes + (int64_t(kvh) * 2 + what) * page * S::RowBytes;
    // the query's rows h0 .. h0 + nh - 1, under way with the table's entries
    const int h0 = (pass % a.chunks) * kHeads;
#pragma unroll
    for (int i = 0; i < kHeads / kWarps; ++i) {
      const int r = warp + i * kWarps;
      const int64_t base = b * a.q.row_stride + (static_cast<int64_t>(kvh) * a.group + h0 + r) * a.q.head_stride;
#pragma unroll
      for (int k = 0; k < NB; ++k) {  // lane = element of block k
        query[i][k] = 0;
        if (h0 + r < a.group) {
          const int64_t at = base + 32 * k + lane;
          query[i][k] = a.q.dtype == WOQ_F32   ? static_cast<const float *>(a.q.data)[at]
                        : a.q.dtype == WOQ_F16 ? __half2float(static_cast<const __half *>(a.q.data)[at])
                                               : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q.data)[at]);
        }
      }
    }
    int32_t e[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) e[i] = entry(u_begin + warp + i * kWarps);
    next = entry(u_begin + warp + kStages * kWarps);
#pragma unroll
    for (int i = 0; i < kStages; ++i) issue(u_begin + warp + i * kWarps, i, e[i]);
  };
  if (begin < end) enter(begin);
  if (a.stuck_wait > 0 && begin < end) {  // test hook
    if (!ptx::mbar_wait_bounded(never, 0, a.stuck_wait, abort)) {
      *abort = 1;
      atomicOr(&g_kv4_timeout_flag, 1u);
    }
  }

  for (int64_t cur = begin; cur < end;) {
    const int h0 = (pass % a.chunks) * kHeads;
    const int nh = a.group - h0 < kHeads ? a.group - h0 : kHeads;

    // The query times scale * log2(e), times the power of two that brings the row's largest into [2^13, 2^14).
#pragma unroll
    for (int n = 0; n < kHeads / kWarps; ++n) {
      const int r = warp + n * kWarps;
      float (&v)[NB] = query[n];
      float big = 0;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        v[i] *= a.scale;
        big = fmaxf(big, fabsf(v[i]));
      }
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, i));
      int ex = 0;
      if (big > 0 && big < INFINITY) ex = max(ilogbf(big) - 13, -100);
      const float up = ldexpf(1.0f, -ex);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        v[i] *= up;
        // Element `lane` = 8 tt + e of the block: matrix step 2 i + (e / 2 % 2), a or second pair by e % 2,
        // first or second of the pair by e / 4; odd e meet codes 16 times too large.
        const int e = lane & 7, tt = lane >> 3;
        const float x = e & 1 ? v[i] * 0.0625f : v[i];
        const __half h = __float2half_rn(x);
        const __half l = __float2half_rn(x - __half2float(h));
        __half *dst = reinterpret_cast<__half *>(qop + (2 * i + (e >> 1 & 1)) * 32 + (r * 4 + tt)) +
                      4 * (e & 1) + (e >> 2);
        dst[0] = h;  // .x / .z: high parts (rows 0..7)
        dst[2] = l;  // .y / .w: low parts (rows 8..15)
      }
      if (lane == 0) fac[r] = ldexpf(1.0f, ex);
    }
    __syncthreads();

    const float f = fac[g];

    // Weights are p = 2^(score - m) times 2^kTop. m is the unit's own largest score, rounded up, so that a unit's weights
    // keep their bits after a token that had far more weight; it changes by whole powers of two, which are exact.
    float m = -INFINITY;
    float highest = -INFINITY;  // the largest m so far: m is at most 2^kFall below it, which keeps sums finite
    float l = 0;                // this lane's sum of p
    // Value scales are taken times 2^room, so that they are in [2^-12, 2) as a rule: a block's p * vs then reaches 2 at
    // least, and of each token binary16 cuts off at most 2^-25 (p) and 2^-26 (p * vs) of that.
    int room = 0;
    uint32_t lowest = 0xf400f400u;  // twice the bits of 2^(-12 - room), negative
    int width = 0x33ff;             // from there on, the bits that are below those of 2^(1 - room)
    float2 acc[NB][4];  // value block, n-tile: columns of tokens' head g, dims 32 b + 8 t + i and + 4
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0, 0);

    int st = 0;
    bool ok = true;
    for (int u = u_begin + warp; u < u_end; u += kWarps) {
      if (!__all_sync(0xffffffffu, ptx::mbar_wait_bounded(&bar[st], phases >> st & 1, a.wait_limit, abort))) {
        *abort = 1;
        atomicOr(&g_kv4_timeout_flag, 1u);
        ok = false;
        break;
      }
      phases ^= 1u << st;
      const uint8_t *base = mine + st * S::Stage;

      // Tokens of each half that are there: all 32, as a rule.
      const uint32_t pages_ok = there & 3u;
      const int rest = len - u * kUnit;
      const bool full = pages_ok == 3u && rest >= kUnit;

      // ---- scores: two matrices of 8 tokens for each half of the unit ----
      float2 s[2][2];
      uint32_t vs[2][2][2][NB / 2];  // value scales: half, matrix, token, pairs of blocks
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // column g of the matrix is token 8 i + (g / 2) + 4 (g % 2)
          const uint8_t *kr = base + (16 * h + token_of(i, g >> 1, g & 1)) * S::RowBytes + t * (4 * NB);
          uint32_t w[NB];
          if constexpr (NB == 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(kr);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(kr);
            w[0] = x.x; w[1] = x.y;
          }
          uint32_t ks[2][NB / 2];  // scales of this lane's two tokens
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint8_t *sr = base + S::Scales + (16 * h + token_of(i, t, j)) * S::ScaleBytes;
            if constexpr (NB == 4) {
              const uint4 x = *reinterpret_cast<const uint4 *>(sr);
              ks[j][0] = x.x; ks[j][1] = x.y;
              vs[h][i][j][0] = x.z; vs[h][i][j][1] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2 *>(sr);
              ks[j][0] = x.x;
              vs[h][i][j][0] = x.y;
            }
          }
          float2 sum = make_float2(0, 0);
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            float c[4];
            mma(c, qop[(2 * k) * 32 + lane], low(w[k], magic), high(w[k], magic), magic.zero);
            const uint32_t w8 = w[k] >> 8;
            mma(c, qop[(2 * k + 1) * 32 + lane], low(w8, magic), high(w8, magic), c);
            const __half2 s0 = *reinterpret_cast<const __half2 *>(&ks[0][k / 2]);
            const __half2 s1 = *reinterpret_cast<const __half2 *>(&ks[1][k / 2]);
            const float2 sc = make_float2(k & 1 ? __high2float(s0) : __low2float(s0),
                                          k & 1 ? __high2float(s1) : __low2float(s1));
            sum = __ffma2_rn(__fadd2_rn(make_float2(c[0], c[1]), make_float2(c[2], c[3])), sc, sum);
          }
          s[h][i] = sum;  // times f below
        }
      }
      if (!full) {  // warp-uniform: tokens that are not there weigh nothing, whatever the stage holds
        const uint32_t from = ((0u - lowest) & 0xffffu) * 0x00010001u;  // scales that need no look
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (!(pages_ok >> h & 1) || 16 * h + token_of(i, t, j) >= rest) {
                (j ? s[h][i].y : s[h][i].x) = -INFINITY;
#pragma unroll
                for (int k = 0; k < NB / 2; ++k) vs[h][i][j][k] = from;
              }
      }

      // ---- softmax over the unit: weights in the scores' place, `al` for what was summed before ----
      float shift = 0;  // change of room
      float2 al;
      auto softmax = [&] {
        float mx = fmaxf(fmaxf(fmaxf(s[0][0].x, s[0][0].y), fmaxf(s[0][1].x, s[0][1].y)),
                         fmaxf(fmaxf(s[1][0].x, s[1][0].y), fmaxf(s[1][1].x, s[1][1].y)));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // Any token makes the maximum finite, so that -infinity means that there was none: a row of
        // scores that are all NaN or -infinity gives NaN, as the formula does.
        mx *= f;  // a power of two: exact
        if (pages_ok) mx = fmaxf(mx, -3.402823466e38f);
        const float own = ceilf(mx);
        highest = fmaxf(highest, own);
        const float m2 = fmaxf(own, highest - static_cast<float>(kFall));
        const float ref = m2 == -INFINITY ? 0.0f : -m2;
        const float beta = m == -INFINITY ? -INFINITY : m - m2;
        const float alpha = ex2(beta + shift);
        al = make_float2(alpha, alpha);
        l *= ex2(beta);
        m = m2;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 y = __ffma2_rn(s[h][i], make_float2(f, f), make_float2(ref, ref));
            // times 2^kTop only here: an exponent of up to 14 would round at 2^-21
            s[h][i] = __fmul2_rn(make_float2(ex2(y.x), ex2(y.y)), make_float2(1 << kTop, 1 << kTop));
          }
        const float2 sum = __fadd2_rn(__fadd2_rn(s[0][0], s[0][1]), __fadd2_rn(s[1][0], s[1][1]));
        l += sum.x + sum.y;
      };

      // ---- values ----
      // operand(kp, kb, p): the weights times block k's scales, as sums of two binary16 numbers, and what the
      // products with them are to be multiplied with
      auto values = [&](auto operand) {
#pragma unroll
        for (int kp = 0; kp < NB / 2; ++kp) {  // pairs of blocks: one word of a lane's codes
          uint32_t v[2][2][2];  // half, matrix, block of the pair: two tokens' four codes
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint8_t *vr = base + S::Values + 16 * h * S::RowBytes + g * (2 * NB) + kp * 4;
              const uint32_t w0 = *reinterpret_cast<const uint32_t *>(vr + token_of(i, t, 0) * S::RowBytes);
              const uint32_t w1 = *reinterpret_cast<const uint32_t *>(vr + token_of(i, t, 1) * S::RowBytes);
              v[h][i][0] = __byte_perm(w0, w1, 0x5410);
              v[h][i][1] = __byte_perm(w0, w1, 0x7632);
            }
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) {
            const int k = 2 * kp + kb;
            uint4 p[2];
            const auto back = operand(kp, kb, p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float c[4];
              const int sh = 8 * (i >> 1);
              auto pick = [&](uint32_t w) { return i & 1 ? high(w >> sh, magic) : low(w >> sh, magic); };
              mma(c, p[0], pick(v[0][0][kb]), pick(v[0][1][kb]), magic.zero);
              mma(c, p[1], pick(v[1][0][kb]), pick(v[1][1][kb]), c);
              acc[k][i] =
                  __ffma2_rn(acc[k][i], al, back(__fadd2_rn(make_float2(c[0], c[1]), make_float2(c[2], c[3]))));
            }
          }
        }
      };

      // ---- value scales: keep p * vs inside binary16 ----
      // Their bits order them as 16-bit numbers. A scale of 0 or below counts as outside, and only takes a look.
      uint32_t big = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < NB / 2; ++k) big = __viaddmax_u16x2(vs[h][i][j][k], lowest, big);
      if (__any_sync(0xffffffffu, static_cast<int>(max(big & 0xffffu, big >> 16)) > width)) {
        uint32_t most = 0, least = 0xffffffffu, zero = 0;  // sizes; less one, least and most: 0 is the most then
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < NB / 2; ++k) {
                const uint32_t size = vs[h][i][j][k] & 0x7fff7fffu;
                most = __vmaxu2(most, size);
                least = __vminu2(least, __vsub2(size, 0x00010001u));
                zero = __vmaxu2(zero, __vsub2(size, 0x00010001u));
              }
        const int hi = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
        const int lo = __reduce_min_sync(0xffffffffu, min(least & 0xffffu, least >> 16)) + 1;
        if (hi > 0) {
          // What room has to be for the largest and for the least.
          const int r_max = -half_exponent(hi), r_min = -12 - half_exponent(lo);
          const bool zeros = __any_sync(0xffffffffu, max(zero & 0xffffu, zero >> 16) == 0xffffu);
          const bool wide = hi >= 0x7c00 || r_min > r_max || zeros;  // further apart than that, or some are 0
          if (wide || room < r_min || room > r_max) {
            const int next = wide || (r_min <= 0 && r_max >= 0) ? 0 : (r_min + r_max) >> 1;
            shift = static_cast<float>(next - room);
            room = next;
            const int from = half_bits(-12 - room);
            lowest = static_cast<uint32_t>(0x10000 - from) * 0x00010001u;
            width = half_bits(1 - room) - 1 - from;
          }
          if (wide) {  // all of it here, so that the other way stays one piece
            softmax();
            // The products in FP32, times the power of two that brings a head's largest into [2^13, 2^14).
            values([&](int kp, int kb, uint4 (&p)[2]) {
              float2 x[2][2];
              float top = 0;
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const __half2 s0 = h2(vs[h][i][0][kp]), s1 = h2(vs[h][i][1][kp]);
                  x[h][i] = make_float2(s[h][i].x * (kb ? __high2float(s0) : __low2float(s0)),
                                        s[h][i].y * (kb ? __high2float(s1) : __low2float(s1)));
                  top = fmaxf(top, fmaxf(fabsf(x[h][i].x), fabsf(x[h][i].y)));
                }
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
              const int up = min(max(140 - static_cast<int>(__float_as_uint(top) >> 23), -100), 100);
              const float u = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
              const float down = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                split(x[h][0].x * u, x[h][0].y * u, p[h].x, p[h].y);
                split(x[h][1].x * u, x[h][1].y * u, p[h].z, p[h].w);
              }
              return [down](float2 c) { return __fmul2_rn(c, make_float2(down, down)); };
            });
            goto summed;
          }
        }
      }
      if (room != 0) {  // warp-uniform
        // in two steps, as 2^24 is no binary16; each product is exact or, far below the largest, rounded
        const __half2 a1 = __float2half2_rn(ldexpf(1.0f, room / 2));
        const __half2 a2 = __float2half2_rn(ldexpf(1.0f, room - room / 2));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < NB / 2; ++k)
                vs[h][i][j][k] = u32(__hmul2(__hmul2(h2(vs[h][i][j][k]), a1), a2));
      }

      {
        softmax();
        uint32_t ph[2][2], pl[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) split(s[h][i].x, s[h][i].y, ph[h][i], pl[h][i]);
        values([&](int kp, int kb, uint4 (&p)[2]) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // (ph + pl) * vs as a sum of two binary16 again: the product's rounding error is itself a
            // binary16, which the fused multiply-add gives exactly
            uint32_t x[2], y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const __half2 sc = h2(__byte_perm(vs[h][i][0][kp], vs[h][i][1][kp], kb ? 0x7632 : 0x5410));
              const __half2 hi = __hmul2(h2(ph[h][i]), sc);
              x[i] = u32(hi);
              y[i] = u32(__hfma2(h2(pl[h][i]), sc, __hfma2(h2(ph[h][i]), sc, __hneg2(hi))));
            }
            p[h] = make_uint4(x[0], y[0], x[1], y[1]);
          }
          return [](float2 c) { return c; };
        });
      }

    summed:
      __syncwarp();  // every lane has read the stage
      issue(u + kStages * kWarps, st, next);
      next = entry(u + (kStages + 1) * kWarps);
      st = st + 1 == kStages ? 0 : st + 1;
    }
    // This segment, and into the next one's: its copies are under way while this one's results are put together.
    const int this_b = b, this_kvh = kvh, this_pass = pass, this_units = units;
    const int64_t after = cur + (u_end - u_begin);
    __syncwarp();
    if (ok && after < end) enter(after);

    // ---- the four warps' results, then the block's ----
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    float *res = results + warp * S::Slot;
    if (t == 0) {
      res[S::Maxima + g] = m;
      res[S::Totals + g] = l;
    }
    const float even = ldexpf(1.0f, -room), odd = 0.0625f * even;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      float4 *to = reinterpret_cast<float4 *>(res + g * S::HeadStep + 32 * k + 8 * t);
      to[0] = make_float4(acc[k][0].x * even, acc[k][1].x * odd, acc[k][2].x * even, acc[k][3].x * odd);
      to[1] = make_float4(acc[k][0].y * even, acc[k][1].y * odd, acc[k][2].y * even, acc[k][3].y * odd);
    }
    __syncthreads();

    // Thread: head tid / 16, D / 16 dims from (tid % 16) * 4 on, 64 apart.
    const int hd = tid >> 4, d0 = (tid & 15) * 4;
    constexpr int ND = D / 64;
    // Adds up `n` results (the warps' or parts') in their order; `at(k)`: the k-th. Four results' loads are
    // under way at once: one after the other took longer than all else of a short context.
    float M, L;
    float4 o[ND];
    auto join = [&](int64_t n, auto at, auto ld, auto ld4) {
      M = -INFINITY;
      L = 0;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[i] = make_float4(0, 0, 0, 0);
      for (int64_t k0 = 0; k0 < n; k0 += 4) {
        float mk[4], lk[4];
        float4 v[4][ND];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float *r = at(k0 + k < n ? k0 + k : n - 1);
          mk[k] = k0 + k < n ? ld(r + S::Maxima + hd) : -INFINITY;
          lk[k] = ld(r + S::Totals + hd);
#pragma unroll
          for (int i = 0; i < ND; ++i) v[k][i] = ld4(r + hd * S::HeadStep + d0 + 64 * i);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (mk[k] == -INFINITY) continue;  // no token seen
          const float M2 = fmaxf(M, mk[k]);
          const float x = M == -INFINITY ? 0.0f : ex2(M - M2), y = ex2(mk[k] - M2);
          L = L * x + lk[k] * y;
#pragma unroll
          for (int i = 0; i < ND; ++i) {
            o[i].x = o[i].x * x + v[k][i].x * y;
            o[i].y = o[i].y * x + v[k][i].y * y;
            o[i].z = o[i].z * x + v[k][i].z * y;
            o[i].w = o[i].w * x + v[k][i].w * y;
          }
          M = M2;
        }
      }
    };
    auto finish = [&] {
      if (hd >= nh) return;
      const float r = M == -INFINITY ? 0.0f : 1.0f / L;  // no token behind any page: zeros
#pragma unroll
      for (int i = 0; i < ND; ++i)
        store4(a.o.data,
               this_b * a.o.row_stride + (static_cast<int64_t>(this_kvh) * a.group + h0 + hd) * a.o.head_stride + d0 +
                   64 * i,
               a.o.dtype, make_float4(o[i].x * r, o[i].y * r, o[i].z * r, o[i].w * r));
    };
    join(kWarps, [&](int64_t k) { return results + k * S::Slot; }, [](const float *p) { return *p; },
         [](const float *p) { return *reinterpret_cast<const float4 *>(p); });
    const int64_t first = pre[this_b] * heads + int64_t(this_pass) * this_units;
    const int64_t last = first + this_units - 1;  // units of this pass
    if (first >= begin && last < end) {
      finish();
    } else {
      // Part x starts at unit x * total / parts; the part that has unit v is ((v + 1) * parts - 1) / total.
      const int64_t x0 = ((first + 1) * parts - 1) / total, x1 = ((last + 1) * parts - 1) / total;
      float *slot = a.partials + (blockIdx.x * 2 + (cur == begin ? 0 : 1)) * int64_t(S::Slot);
#pragma unroll
      for (int i = 0; i < ND; ++i) *reinterpret_cast<float4 *>(slot + hd * S::HeadStep + d0 + 64 * i) = o[i];
      if ((tid & 15) == 0) {
        slot[S::Maxima + hd] = M;
        slot[S::Totals + hd] = L;
      }
      __threadfence();
      __syncthreads();
      unsigned *counter = a.counters + static_cast<int64_t>(this_b) * heads + this_pass;
      if (tid == 0) flags[1] = atomicAdd(counter, 1u) == static_cast<unsigned>(x1 - x0);
      __syncthreads();
      if (flags[1]) {
        __threadfence();
        if (tid == 0) *counter = 0;
        // Part x0 has this pass as its last segment (slot 1) unless it begins with it; the others
        // begin with it. Parts follow one another in the workspace two slots apart.
        const int64_t begin0 = x0 * total / parts;
        join(x1 - x0 + 1,
             [&](int64_t k) {
               return a.partials + ((x0 + k) * 2 + (k == 0 && begin0 < first ? 1 : 0)) * int64_t(S::Slot);
             },
             [](const float *p) { return __ldcg(p); },
             [](const float *p) { return __ldcg(reinterpret_cast<const float4 *>(p)); });
        finish();
      }
    }
    __syncthreads();  // the results and the query's operands are read
    cur = after;
    if (*abort) {  // uniform: read behind a barrier, written before it
      // The copies that this warp still has in flight end before the block does (or the wait for none gives up).
      int no_abort = 0;
      for (int i = 0; i < kStages; ++i) ptx::mbar_wait_bounded(&bar[i], phases >> i & 1, 1LL << 28, &no_abort);
      break;
    }
  }
  ptx::pdl_launch_dependents();
}

template <int D>
size_t smem_bytes(int batch) {
  using S = Shape<D>;
  return static_cast<size_t>(kWarps) * (kStages * S::Stage + S::Slot * 4) + 2 * S::NB * 32 * 16 + (kWarps * kStages + 1) * 8 +
         (kHeads + 4) * 4 + 8 * (static_cast<size_t>(batch) + 1);
}

template <int D>
int launch(const Args &a, cudaStream_t s, const DevInfo &dev) {
  auto kern = kv4_attn_kernel<D>;
  static std::once_flag once[64];
  static cudaError_t err[64];
  std::call_once(once[dev.device], [&] {
    err[dev.device] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem_bytes<D>(kKv4MaxBatch)));
  });
  if (err[dev.device] != cudaSuccess) return WOQ_ECUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count * kBlocksPerSm), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<D>(a.batch);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return WOQ_ECUDA;
  count_launches(1);
  return WOQ_OK;
}

// The workspace: partial results, of the larger dim's size whatever the call's, and then the counters. So no call's
// partial results lie where another's counters are, and one workspace serves calls of all shapes that it has room for.
size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

size_t partials_bytes(int sm_count) {
  return up256(static_cast<size_t>(sm_count) * kBlocksPerSm * 2 * Shape<128>::Slot * sizeof(float));
}

}  // namespace

size_t kv4_attn_workspace(int32_t batch, int32_t kv_heads, int32_t group, int sm_count) {
  return partials_bytes(sm_count) + up256(static_cast<size_t>(batch) * kv_heads * ((group + kHeads - 1) / kHeads) * 4);
}

int launch_kv4_attn(const woq_rows &q, const woq_kv4 &c, const int32_t *lens, int32_t batch, const int32_t *table,
                    int64_t width, float scale, const woq_rows &o, void *workspace, cudaStream_t s,
                    const DevInfo &dev) {
  Args a;
  a.q = q;
  a.o = o;
  a.codes = c.codes;
  a.scales = reinterpret_cast<const uint8_t *>(c.scales);
  a.lens = lens;
  a.table = table;
  a.pages = c.pages;
  a.width = width;
  a.batch = batch;
  a.shift = __builtin_ctz(static_cast<unsigned>(c.page));
  a.kv_heads = c.kv_heads;
  a.group = q.heads / c.kv_heads;
  a.chunks = (a.group + kHeads - 1) / kHeads;
  a.scale = scale * 1.44269504088896340736f;
  a.partials = static_cast<float *>(workspace);
  a.counters = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(workspace) + partials_bytes(dev.sm_count));
  const long long lim = wait_limit_cycles();
  a.wait_limit = lim > 0 ? lim : kWaitLimit;
  a.stuck_wait = lim < 0 ? -lim : 0;
  return c.dim == 128 ? launch<128>(a, s, dev) : launch<64>(a, s, dev);
}

int read_kv4_timeout_flag(int clear, unsigned *value) {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv4_timeout_flag, sizeof(v)) != cudaSuccess) return WOQ_ECUDA;
  if (clear && v) {
    const unsigned z = 0;
    if (cudaMemcpyToSymbol(g_kv4_timeout_flag, &z, sizeof(z)) != cudaSuccess) return WOQ_ECUDA;
  }
  *value = v;
  return WOQ_OK;
}

}  // namespace woq
