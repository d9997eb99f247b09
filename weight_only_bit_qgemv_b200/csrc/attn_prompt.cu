// attn_prompt: causal attention over whole prompts, packed one after another.
//   s_ij = scale q_i . k_j,  o_i = sum_{j <= i} softmax_j(s_ij) v_j
//
// Bound: the tensor cores; with 16-bit rows the exponentials are as near. A pair of 128 x 128 tiles of scores and
// of weights times values is 1024 cycles of an SM's tensor cores at dim 128 (512 at dim 64), and so are its 16,384
// exponentials at 16 a cycle: each has to run under the other. float32 rows take three products for one.
//
// One block an SM takes 256 query rows of one head as two tiles of 128 and walks the keys in tiles of
// BK up to the diagonal. Two warpgroups have a query tile each, a row a thread: they read the scores
// from tensor memory, keep the row's running maximum and sum, and write the weights back to
// tensor memory as an operand. While one has its exponentials, the tensor cores work for the other. Of four more
// warps 8 has the copies (TMA), 9 issues the scores' matrix instructions, 10 the values', and 11 looks at the
// values on the diagonal. Longest rows come first in a sequence, so that a launch ends with its shortest blocks.
//
// A block that has asked for the last of its copies takes over a block that has not started (cluster launch control):
// that one's place is looked up and its keys, values and, 16-bit rows, queries are under way while the last tiles
// of this one and its output are worked on. Barriers count on from item to item. Against a launch for each block:
// 16 bfloat16 prompts of 301 to 4003 tokens 969 -> 896 us, 3 binary16 ones of 1 to 5003 at dim 64 99 -> 88, 32,768
// bfloat16 tokens 4.01 -> 3.85 ms, 4096 float32 ones 243 -> 238 us; 137 float32 ones, one item a block, 20.2 -> 20.5.
//
// 16-bit rows: the output is summed in tensor memory, against a maximum that may lag behind (at the loop). float32
// rows: each tile's product starts from zero and is added to the output in registers, so that sums
// inside the tensor cores, which cut off instead of rounding, run over BK keys at most; scores are one tile ahead.
//
// float32 rows: a kernel before writes each tile of 64 rows as two binary16 planes, high part and rest, times the
// power of two that brings its largest finite value into [2^13, 2^14) (query rows each by itself). Where the rows' sizes
// are not within 2^10 of one another, each row of keys or values has a power of its own, so that a row's precision
// does not go by a larger one beside or behind it: 22 bits of every value within 2^17 of its row's largest, less what
// the row is below the tile's largest, 2^10 at most. Scores are three products (high x high and the two mixed
// ones, small ones first), the weights are split the same way, times 2^13. Queries turned into planes by the
// block itself were slower (137 tokens 26 instead of 20 us, 24 prompts of 11 to 2011 715 instead of 706): one
// block has the SM, and nothing runs under it.
//
// Masked weights are exact zeros, but zero times a value that is not finite is NaN. The tiles on the diagonal hold
// every masked pair of the block, so their values are looked at, what is not finite is replaced by 0 in shared memory,
// and added after the last tile to the rows that do see it.
//
// Measured (16 query heads on 8 key heads, dim 128): 137 float32 tokens 20 us, 4096 235 us (26 of them the
// planes; 1 PFLOP/s of products in the rest), 24 prompts of 11 to 2011 710 us (130 the planes); 32,768
// bfloat16 tokens 3.9 ms, 1.12 PFLOP/s. The power cap holds the clock of the long ones at 1537 to 1747 MHz.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "kv4.cuh"
#include "ptx.cuh"
#include "woq_internal.h"

namespace woq {

__device__ unsigned int g_prompt_timeout_flag = 0;

namespace {

constexpr int kRows = 128;               // query rows of a warpgroup: the lanes of tensor memory
constexpr int kBlockRows = 2 * kRows;
constexpr int kSplitRows = 64;           // rows of a float32 tile of keys or values
constexpr float kLag = 8;                // what 16-bit rows' weights may exceed 1 by, as a power of two
constexpr int kWeightBits = 13;          // float32 rows' weights reach 2^kWeightBits
constexpr int kSpread = 10;              // one power of two for them, if their sizes lie within 2^kSpread of one another
// A score's factor from which on float32 rows' scores may reach 2^24: they are sums of 128 products below 2^28. Above
// that, `largest less itself` in one fused step would be what its product was rounded by, and from 2^26 on a weight of
// that leaves binary16.
constexpr float kFar = 0x1p-11f;
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;
constexpr uint32_t kTmemCols = 512;
constexpr long long kWaitLimit = 1LL << 32;   // cycles (~2 s)
constexpr long long kDrainLimit = 1LL << 31;

enum { kBf16 = 0, kF16 = 1, kSplit = 2 };

template <int D, int MODE>
struct Cfg {
  static constexpr int Parts = MODE == kSplit ? 2 : 1;       // planes of an operand
  // Keys of a tile. Tensor memory's 512 columns hold two outputs of D columns; the rest is for two query tiles'
  // scores (BK columns) and, 16-bit rows, their weights (BK / 2) or, float32 rows, two tiles' scores (2 BK).
  static constexpr int BK = MODE == kSplit ? 64 : D == 128 ? 80 : 128;
  static constexpr int Subs = D / 64;                        // 128-byte columns of a tile
  static constexpr int QBytes = Parts * kRows * D * 2;
  static constexpr int KvBytes = Parts * BK * D * 2;
  // A 16-bit block has its next queries on the way while it still needs these; float32 queries fill the room.
  static constexpr int QBufs = MODE == kSplit ? 1 : 2;
  static constexpr int Room = 227 * 1024 - 2048 - QBufs * 2 * QBytes;
  static constexpr int Stages = Room / KvBytes > 6 ? 6 : Room / KvBytes;
  static_assert(MODE != kSplit || BK == kSplitRows, "tiles' powers of two");
  static_assert(Stages >= 3, "keys and values of two tiles are in flight at once");
  // Registers of a thread of the two query groups and of the helpers, out of what the block is launched with. float32
  // rows of dim 128 hold an output of 128 numbers and 64 scores: 216 and 72 took 4096 tokens 250 us, 224 and 56 238,
  // 232 and 40 233.
  static constexpr bool Wide = MODE == kSplit && D == 128;
  static constexpr int QueryRegs = Wide ? 232 : MODE == kSplit ? 216 : 200;
  static constexpr int HelperRegs = Wide ? 40 : MODE == kSplit ? 72 : 104;
  static_assert(256 * QueryRegs + 128 * HelperRegs <= kThreads * kLaunchRegs, "register split");
  static constexpr int Smem = QBufs * 2 * QBytes + Stages * KvBytes + 2048;
};

struct Maps {
  CUtensorMap q[2], k[2], v[2];  // [plane]
};

struct Args {
  const int32_t *cu;
  int64_t tokens;
  int batch, q_heads, group;
  float scale;  // times log2(e)
  woq_rows o, v;
  // float32 rows: powers of two by row (queries) and by tile of kSplitRows (keys, values); where that is negative, by row
  const float *q_pow, *k_pow, *v_pow, *k_row, *v_row;
  int64_t tiles;  // entries of a head in k_pow and v_pow
  long long wait_limit, stuck_wait;
};

constexpr int kLooks = kBlockRows / 64 + 1;  // at least the tiles on a block's diagonal

// The tile of query rows that a block has in hand; the next one's record is written beside it.
struct Item {
  int head, start, len, r0, tile0;  // len 0: there are no more
};

struct Shared {
  uint4 claim;        // the answer to a claim of another block's tile
  uint64_t claimed;
  uint64_t item_full[2];
  uint64_t done[2];   // [item & 1] the query warps have written the item's rows
  uint64_t q_full[2][2];  // [buffer][query tile]
  uint64_t kv_full[8], kv_empty[8];
  // [query tile][its scores' buffer]: 16-bit rows have one, float32 rows two. s_free, 16-bit rows: read by
  // the query tile's warps; float32 rows: the weights in their place have been multiplied.
  uint64_t s_full[2][2], s_free[2][2];
  // Weights written; with float32 rows also the product before it read out, which has the place of the next. A
  // warp may be a tile ahead of the others in its query tile, as its scores are: float32 rows have one for each buffer.
  uint64_t p_full[2][2];
  uint64_t t_full[2];
  uint64_t look[kLooks];    // the copy of a diagonal tile's values is under way
  uint64_t looked[kLooks];  // they are there, and finite
  uint64_t looked_all;
  uint64_t drain, never;
  Item item[2];
  uint32_t tmem;
  int abort;
  int nonfinite[2];  // [item & 1]
};

__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}

// 2^e, e within +-126.
__device__ __forceinline__ float power(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ void record_timeout(volatile int *abort) {
  *abort = 1;
  atomicOr(&g_prompt_timeout_flag, 1u);
}

// Tile `target` of all sequences' tiles of `rows` rows: its sequence's rows, its place there, and how
// many tiles of kSplitRows the sequences before have. One warp. False if there are fewer tiles. The search goes on
// where the warp's last one ended, if the target is not before that.
struct Place {
  int start, len, tile, tiles, split0;
};
struct Cursor {
  int b0;          // the first of 32 sequences
  int64_t before;  // tiles of those before it
  int split;       // and theirs of kSplitRows
};
__device__ bool find_tile(const int32_t *cu, int batch, int64_t tokens, int64_t target, int rows, Place &p,
                          Cursor &at) {
  const int lane = threadIdx.x & 31;
  if (target < at.before) at = Cursor{};
  int64_t before = at.before;
  int split = at.split;
  for (int b0 = at.b0; b0 < batch; b0 += 32) {
    const int b = b0 + lane;
    int64_t s = 0, e = 0;
    if (b < batch) {
      s = cu[b];
      e = cu[b + 1];
      s = s < 0 ? 0 : s > tokens ? tokens : s;
      e = e < s ? s : e > tokens ? tokens : e;
    }
    const int len = static_cast<int>(e - s);
    const int n = (len + rows - 1) / rows, ns = (len + kSplitRows - 1) / kSplitRows;
    int sum = n, sums = ns;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, i), y = __shfl_up_sync(0xffffffffu, sums, i);
      if (lane >= i) {
        sum += x;
        sums += y;
      }
    }
    const unsigned has = __ballot_sync(0xffffffffu, before + sum > target);
    if (has) {
      at = Cursor{b0, before, split};
      const int l = __ffs(has) - 1;
      p.start = __shfl_sync(0xffffffffu, static_cast<int>(s), l);
      p.len = __shfl_sync(0xffffffffu, len, l);
      p.tiles = __shfl_sync(0xffffffffu, n, l);
      p.tile = static_cast<int>(target - before - (__shfl_sync(0xffffffffu, sum, l) - p.tiles));
      p.split0 = split + __shfl_sync(0xffffffffu, sums - ns, l);
      return true;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
    split += __shfl_sync(0xffffffffu, sums, 31);
  }
  at = Cursor{batch, before, split};
  return false;
}

// Shared-memory matrix descriptors, 128-byte swizzle: 8-row groups 1024 bytes apart, in the upper word that all
// share. The lower word has the address and, where rows are the summed dimension (values), the distance of
// the 64-element columns; queries and keys, whose rows are the other dimension, do not use it.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t sub_bytes) {
  return ((saddr >> 4) & 0x3FFF) | (sub_bytes >> 4) << 16;
}
__device__ __forceinline__ uint64_t desc(uint32_t low) {
  return static_cast<uint64_t>(64u | 1u << 14 | 2u << 29) << 32 | low;
}
// Instruction descriptor: FP32 result, M = 128, N = n; `cols`: B's rows are the summed dimension.
__host__ __device__ constexpr uint32_t idesc_for(int n, bool bf16, bool cols) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (cols ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

// A warp's wait.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, long long limit, volatile int *abort) {
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, limit, abort));
}

// The same number in all lanes, for the compiler to keep in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

template <int MODE>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  return pack2(a, b, MODE == kBf16 ? WOQ_BF16 : WOQ_F16);
}

// Values of `keys` rows at v that are not finite, added to the output row at o: their products were left out.
// Rolled up and in line: a call, or a pointer to the kernel's arguments, costs the whole kernel registers.
template <int D>
__device__ __forceinline__ void add_nonfinite(void *o, const void *v, int64_t stride, int keys, int dtype) {
#pragma unroll 1
  for (int j = 0; j < keys; ++j) {
#pragma unroll 1
    for (int i = 0; i < D; i += 4) {
      const float4 x = load4(v, j * stride + i, dtype);
      if (isfinite(x.x) && isfinite(x.y) && isfinite(x.z) && isfinite(x.w)) continue;
      float4 y = load4(o, i, dtype);
      if (!isfinite(x.x)) y.x += x.x;
      if (!isfinite(x.y)) y.y += x.y;
      if (!isfinite(x.z)) y.z += x.z;
      if (!isfinite(x.w)) y.w += x.w;
      store4(o, i, dtype, y);
    }
  }
}

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ Maps maps, const Args a) {
  using C = Cfg<D, MODE>;
  constexpr int BK = C::BK, ST = C::Stages;
  // Tensor memory columns of query tile t: scores and weights, and products with the values. float32 rows:
  // tile j's scores are in half j & 1, and its weights in their place; 16-bit rows: the weights are behind the
  // scores. Either way the next scores do not wait for this tile's weights.
  constexpr uint32_t kScores = MODE == kSplit ? 2 * BK : (BK + BK / 2 + 31) / 32 * 32;
  constexpr uint32_t kTile = 2 * kScores;
  static_assert(kTile + 2 * D <= kTmemCols, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *smem_kv = smem + C::QBufs * 2 * C::QBytes;
  Shared &sh = *reinterpret_cast<Shared *>(smem_kv + ST * C::KvBytes);
  volatile int *abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 8 && lane == 0) {
    for (int p = 0; p < C::Parts; ++p) {
      ptx::prefetch_tmap(&maps.q[p]);
      ptx::prefetch_tmap(&maps.k[p]);
      ptx::prefetch_tmap(&maps.v[p]);
    }
  }
  if (warp == 9) {
    ptx::tmem_alloc(&sh.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == 1 && lane == 0) {
    ptx::mbar_init(&sh.claimed, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sh.item_full[i], 1);
      ptx::mbar_init(&sh.done[i], 8);
      for (int b = 0; b < 2; ++b) ptx::mbar_init(&sh.q_full[i][b], 1);
      for (int b = 0; b < 2; ++b) {
        ptx::mbar_init(&sh.s_full[i][b], 1);
        ptx::mbar_init(&sh.s_free[i][b], MODE == kSplit ? 1 : 4);
        ptx::mbar_init(&sh.p_full[i][b], MODE == kSplit ? 8 : 4);
      }
      ptx::mbar_init(&sh.t_full[i], 1);
    }
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(&sh.kv_full[i], 1);
      ptx::mbar_init(&sh.kv_empty[i], 1);
    }
    for (int i = 0; i < kLooks; ++i) {
      ptx::mbar_init(&sh.look[i], 1);
      ptx::mbar_init(&sh.looked[i], 1);
    }
    ptx::mbar_init(&sh.looked_all, 1);
    ptx::mbar_init(&sh.drain, 2);
    ptx::mbar_init(&sh.never, 1);
    ptx::fence_mbar_init();
    sh.abort = 0;
  }
  ptx::pdl_wait();
  Place place{};
  Cursor cursor{};
  bool found = false;  // warp 8's: the item that it is about to hand out
  if (warp == 8) found = find_tile(a.cu, a.batch, a.tokens, blockIdx.x / a.q_heads, kBlockRows, place, cursor);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh.tmem;

  // An item's key tiles: up to the diagonal, and not behind the last row.
  struct Work {
    int head, start, len, r0;
    int n0, n1, nt, diag;  // tiles of the two query tiles, of both, and the first with masked pairs
  };
  auto read_item = [&](int it) {
    const Item &i = sh.item[it & 1];
    Work w{i.head, i.start, i.len, i.r0, 0, 0, 0, 0};
    w.n0 = (min(w.len, w.r0 + kRows) + BK - 1) / BK;
    w.n1 = w.r0 + kRows < w.len ? (min(w.len, w.r0 + 2 * kRows) + BK - 1) / BK : 0;
    w.nt = max(w.n0, w.n1);
    w.diag = w.r0 / BK;
    return w;
  };
  // Barriers count on from item to item. The ring's slots in order: k 0, k 1, v 0, k 2, v 1, ... of an item; `ring`
  // is its first one's place, modulo two rounds, and `looks` likewise its first diagonal tile's.
  int ring = 0, looks = 0;
  auto k_slot = [&](int j) { return ring + (j > 0 ? 2 * j - 1 : 0); };
  auto v_slot = [&](int j, int nt) { return ring + (j + 1 < nt ? 2 * j + 2 : 2 * j + 1); };
  auto advance = [&](const Work &w) {
    ring = (ring + 2 * w.nt) % (2 * ST);
    looks = (looks + w.nt - w.diag) % (2 * kLooks);
  };

  if (warp >= 8) {
    ptx::regs_dec<C::HelperRegs>();
    if (warp == 8) {
      // ---- items, and their copies in the order in which the matrix instructions take them ----
      int64_t target = blockIdx.x;
      long long issued = 0;  // slots filled so far
      bool ok = true;
      auto wait_lane = [&](uint64_t *bar, uint32_t parity) {
        if (ok && !ptx::mbar_wait_bounded(bar, parity, a.wait_limit, abort)) {
          record_timeout(abort);
          ok = false;
        }
        return ok;
      };
      int it = 0, claims = 0, loaded = 0;  // items, claims, items whose queries were copied
      for (;;) {
        if (found || target < 0) {
          ok = it < 2 || warp_wait(&sh.done[it & 1], (it - 2) >> 1 & 1, a.wait_limit, abort);
          if (!ok) {
            record_timeout(abort);
            break;
          }
          if (lane == 0) {
            // a sequence's longest rows first
            sh.item[it & 1] = Item{static_cast<int>(target % a.q_heads), place.start, found ? place.len : 0,
                                   (place.tiles - 1 - place.tile) * kBlockRows, place.split0};
            ptx::mbar_arrive(&sh.item_full[it & 1]);
          }
          __syncwarp();
        }
        if (target < 0) break;
        if (found && lane == 0) {
          const Work w = read_item(it);
          const int kv_head = w.head / a.group;
          const int buf = it % C::QBufs;
          auto queries = [&] {
            for (int t = 0; t < 2; ++t) {
              if (t == 1 && w.n1 == 0) {
                ptx::mbar_arrive(&sh.q_full[buf][1]);  // so that its phases are the items'
                break;
              }
              ptx::mbar_arrive_expect_tx(&sh.q_full[buf][t], C::QBytes);
              for (int p = 0; p < C::Parts; ++p)
                for (int c = 0; c < C::Subs; ++c)
                  ptx::tma_load_3d(smem + (2 * buf + t) * C::QBytes + (p * C::Subs + c) * kRows * 128, &maps.q[p],
                                   &sh.q_full[buf][t], 64 * c, w.head, w.start + w.r0 + t * kRows);
            }
            loaded = it + 1;
          };
          auto kv = [&](const CUtensorMap *m, int at, int tile) {
            const int slot = at % ST;
            if (!wait_lane(&sh.kv_empty[slot], ((at / ST) & 1) ^ 1)) return false;
            ptx::mbar_arrive_expect_tx(&sh.kv_full[slot], C::KvBytes);
            for (int p = 0; p < C::Parts; ++p)
              for (int c = 0; c < C::Subs; ++c)
                ptx::tma_load_3d(smem_kv + slot * C::KvBytes + (p * C::Subs + c) * BK * 128, &m[p],
                                 &sh.kv_full[slot], 64 * c, kv_head, w.start + tile * BK);
            ++issued;
            return true;
          };
          const bool queries_first = C::QBufs == 2 || it == 0;
          if (queries_first) queries();
          kv(maps.k, k_slot(0), 0);
#pragma unroll 1
          for (int j = 0; j < w.nt && ok; ++j) {
            if (j + 1 < w.nt) kv(maps.k, k_slot(j + 1), j + 1);
            if (ok) kv(maps.v, v_slot(j, w.nt), j);
            if (ok && j >= w.diag) ptx::mbar_arrive(&sh.look[(looks + j - w.diag) % kLooks]);
            // their place is the last item's output's until that is written
            if (ok && j == 0 && !queries_first && wait_lane(&sh.done[(it - 1) & 1], (it - 1) >> 1 & 1)) queries();
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (found) {
          advance(read_item(it));
          ++it;
        }
        if (!ok) break;
        // The tile of a block that has not started yet: asked for only now, so that who is done first takes it.
        if (lane == 0) {
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive_expect_tx(&sh.claimed, 16);
          ptx::claim_block(&sh.claim, &sh.claimed);
        }
        int no_abort = 0;
        if (!__all_sync(0xffffffffu, ptx::mbar_wait_bounded(&sh.claimed, claims++ & 1, kDrainLimit, &no_abort))) {
          record_timeout(abort);
          break;
        }
        uint32_t next;
        target = ptx::claimed_block(&sh.claim, &next) ? static_cast<int64_t>(next) : -1;
        found = target >= 0 && find_tile(a.cu, a.batch, a.tokens, target / a.q_heads, kBlockRows, place, cursor);
        __syncwarp();
      }
      if (*abort && lane == 0) {
        // What is in flight ends before the block does.
        int no_abort = 0;
        for (int i = max(0, loaded - C::QBufs); i < loaded; ++i)
          for (int t = 0; t < 2; ++t)
            ptx::mbar_wait_bounded(&sh.q_full[i % C::QBufs][t], i / C::QBufs & 1, kDrainLimit, &no_abort);
        for (long long i = max(0LL, issued - ST); i < issued; ++i)
          ptx::mbar_wait_bounded(&sh.kv_full[i % ST], (i / ST) & 1, kDrainLimit, &no_abort);
      }
    } else if (warp == 9 || warp == 10) {
      // ---- matrix instructions: the warp stays together, one lane issues. Warp 9 has the scores, warp 10 the
      // values, so that the tensor cores have the other's instructions while one waits ----
      {
        constexpr uint32_t kIdescS = idesc_for(BK, MODE == kBf16, false), kIdescT = idesc_for(D, MODE == kBf16, true);
        constexpr int kPlaneQ = kRows * D * 2, kPlaneK = BK * D * 2;
        bool ok = true;
        auto wait_for = [&](uint64_t *bar, uint32_t parity, long long limit) {
          if (ok && !warp_wait(bar, parity, limit, abort)) {
            record_timeout(abort);
            ok = false;
          }
          return ok;
        };
        auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_for(bar, parity, a.wait_limit); };
        if (a.stuck_wait > 0) wait_for(&sh.never, 0, a.stuck_wait);  // test hook
        const uint32_t q_addr = ptx::smem_u32(smem), kv_addr = ptx::smem_u32(smem_kv);
        // Scores of tile j for the query tiles that it concerns, in one elected block: between two instructions
        // the tensor cores wait for whatever the issuing thread does.
        // c0, c1: the query tiles' tiles before this one, of all items.
        auto scores = [&](int j, int buf, int c0, int c1, bool first, bool second) {
          const int b0 = MODE == kSplit ? c0 & 1 : 0, b1 = MODE == kSplit ? c1 & 1 : 0;
          const uint32_t d0 = uniform(tmem + b0 * BK), d1 = uniform(tmem + kScores + b1 * BK);
          const uint32_t q = uniform(desc_low(q_addr + buf * 2 * C::QBytes, 16));
          const uint32_t k = uniform(desc_low(kv_addr + k_slot(j) % ST * C::KvBytes, 16));
          if (ptx::elect_one()) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!(t ? second : first)) continue;
              auto product = [&](int pq, int pk, uint32_t acc) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)  // 16 elements are 2 units of 16 bytes
                  ptx::tc_mma_f16(
                      t ? d1 : d0,
                      desc(q + (t * C::QBytes + pq * kPlaneQ + (kk >> 2) * kRows * 128) / 16 + (kk & 3) * 2),
                      desc(k + (pk * kPlaneK + (kk >> 2) * BK * 128) / 16 + (kk & 3) * 2), kIdescS, kk == 0 ? acc : 1);
              };
              if constexpr (MODE == kSplit) {
                product(1, 0, 0);
                product(0, 1, 1);
              }
              product(0, 0, MODE == kSplit);
              ptx::tc_commit(&sh.s_full[t][t ? b1 : b0]);
            }
            ptx::tc_commit(&sh.kv_empty[k_slot(j) % ST]);  // its keys are needed no more
          }
        };
        // Weights times values. 16-bit rows: added to what is there, from the second tile on; float32 rows: from
        // zero. `last`: the tile's values are needed no more.
        auto values = [&](int t, int j, int c, int slot, bool last) {
          const uint32_t d = uniform(tmem + kTile + t * D);
          const uint32_t p = uniform(tmem + t * kScores + (MODE == kSplit ? (c & 1) * BK : BK));
          const uint32_t v = uniform(desc_low(kv_addr + slot * C::KvBytes, BK * 128));
          if (ptx::elect_one()) {
            auto product = [&](int pp, int pv, uint32_t acc) {
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)  // 16 keys are 2048 bytes of values
                ptx::tc_mma_f16_ts(d, p + pp * (BK / 2) + kk * 8, desc(v + (pv * kPlaneK + kk * 2048) / 16), kIdescT,
                                   kk == 0 ? acc : 1);
            };
            if constexpr (MODE == kSplit) {
              product(1, 0, 0);
              product(0, 1, 1);
            }
            product(0, 0, MODE == kSplit ? 1 : j > 0);
            ptx::tc_commit(&sh.t_full[t]);
            if (MODE == kSplit) ptx::tc_commit(&sh.s_free[t][c & 1]);
            if (last) ptx::tc_commit(&sh.kv_empty[slot]);
          }
        };
        auto full = [&](int i) { return wait(&sh.kv_full[i % ST], (i / ST) & 1); };
        int c0 = 0, c1 = 0;
#pragma unroll 1
        for (int it = 0; wait(&sh.item_full[it & 1], it >> 1 & 1); ++it) {
          const Work w = read_item(it);
          if (w.len == 0) break;
          if (warp == 9) {
            const int buf = it % C::QBufs;
#pragma unroll 1
            for (int j = 0; j < w.nt && ok; ++j) {
              const bool first = j < w.n0, second = j < w.n1;
              // The place for the scores is free: a tile is the c-th (16-bit) or c / 2-th one there.
              const int b0 = MODE == kSplit ? c0 & 1 : 0, b1 = MODE == kSplit ? c1 & 1 : 0;
              const int p0 = (MODE == kSplit ? c0 >> 1 : c0) & 1, p1 = (MODE == kSplit ? c1 >> 1 : c1) & 1;
              if (!full(k_slot(j)) || (first && !wait(&sh.s_free[0][b0], p0 ^ 1)) ||
                  (second && !wait(&sh.s_free[1][b1], p1 ^ 1)))
                break;
              if (j == 0 && !(wait(&sh.q_full[buf][0], it / C::QBufs & 1) &&
                              (!second || wait(&sh.q_full[buf][1], it / C::QBufs & 1))))
                break;
              ptx::tc_fence_after();
              scores(j, buf, c0, c1, first, second);
              c0 += first;
              c1 += second;
            }
          } else {
#pragma unroll 1
            for (int j = 0; j < w.nt && ok; ++j) {
              const int look = looks + j - w.diag, slot = v_slot(j, w.nt);
              if (!full(slot) || (j >= w.diag && !wait(&sh.looked[look % kLooks], look / kLooks & 1))) break;
#pragma unroll 1
              for (int t = 0; t < 2; ++t) {
                if (j >= (t ? w.n1 : w.n0)) continue;
                const int c = t ? c1 : c0;
                if (!wait(&sh.p_full[t][MODE == kSplit ? c & 1 : 0], (MODE == kSplit ? c >> 1 : c) & 1)) break;
                ptx::tc_fence_after();
                values(t, j, c, slot % ST, t == 1 || j >= w.n1);
                if (t) ++c1;
                else ++c0;
              }
            }
          }
          if (!ok) break;
          advance(w);
        }
        if (ptx::elect_one()) ptx::tc_commit(&sh.drain);
      }
    } else if (warp == 11) {
      // ---- values on the diagonal: what is not finite becomes 0 ----
      constexpr uint32_t kExp = MODE == kBf16 ? 0x7f807f80u : 0x7c007c00u;
      constexpr uint32_t kOne = MODE == kBf16 ? 0x00800080u : 0x04000400u;
      bool ok = true;
#pragma unroll 1
      for (int it = 0; ok; ++it) {
        ok = warp_wait(&sh.item_full[it & 1], it >> 1 & 1, a.wait_limit, abort);
        if (!ok) {
          record_timeout(abort);
          break;
        }
        const Work w = read_item(it);
        if (w.len == 0) break;
        const int len = w.len;
        if (lane == 0) sh.nonfinite[it & 1] = 0;
        __syncwarp();
        for (int j = w.diag; j < w.nt && ok; ++j) {
          const int i = v_slot(j, w.nt), look = looks + j - w.diag;
          // The slot's phase is this tile's from the copy's start until the tile has been looked at: only
          // then does its parity mean this tile.
          ok = warp_wait(&sh.look[look % kLooks], look / kLooks & 1, a.wait_limit, abort) &&
               warp_wait(&sh.kv_full[i % ST], (i / ST) & 1, a.wait_limit, abort);
          if (!ok) {
            record_timeout(abort);
            break;
          }
          // The high plane; the other is finite in the sequence's rows, and unknown behind them.
          uint4 *tile = reinterpret_cast<uint4 *>(smem_kv + (i % ST) * C::KvBytes);
          const int planes = (j + 1) * BK > w.len ? C::Parts : 1;
          // Exponents of ones only, in two halves of a word at once: adding one to such an exponent sets the sign.
          auto check = [](const uint4 &x) {
            return (((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne)) &
                   0x80008000u;
          };
          const int pieces = planes * BK * D / 8;
          uint32_t bad = 0;
#pragma unroll 8
          for (int c = lane; c < pieces; c += 32) bad |= check(tile[c]);
          if (__any_sync(0xffffffffu, bad != 0)) {
            bool mine = false;
            for (int c = lane; c < pieces; c += 32) {
              uint4 x = tile[c];
              if (!check(x)) continue;
              uint32_t *w = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t b = ((w[k] & kExp) + kOne) & 0x80008000u;
                if (b & 0x8000u) w[k] &= 0xffff0000u;
                if (b & 0x80000000u) w[k] &= 0xffffu;
              }
              tile[c] = x;
              mine |= j * BK + c / 8 % BK < len;  // not of the rows behind the sequence
            }
            if (mine) sh.nonfinite[it & 1] = 1;
            ptx::fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.looked[look % kLooks]);
        }
        if (!ok) break;
        // One phase an item: the query warps have to be behind the last one.
        ok = it == 0 || warp_wait(&sh.done[(it - 1) & 1], (it - 1) >> 1 & 1, a.wait_limit, abort);
        if (!ok) {
          record_timeout(abort);
          break;
        }
        if (lane == 0) ptx::mbar_arrive(&sh.looked_all);
        advance(w);
      }
    }
  } else {
    // ---- a query tile: one row a thread ----
    ptx::regs_inc<C::QueryRegs>();
    const int t = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + t * kScores, t_addr = tmem + lanes + kTile + t * D;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (!warp_wait(bar, parity, a.wait_limit, abort)) {
        record_timeout(abort);
        ok = false;
      }
      return ok;
    };
    int count = 0;  // tiles before this item's
#pragma unroll 1
    for (int it = 0; wait(&sh.item_full[it & 1], it >> 1 & 1); ++it) {
      const Work w = read_item(it);
      if (w.len == 0) break;
      const int head = w.head, start = w.start, len = w.len, r0 = w.r0, diag = w.diag, kv_head = w.head / a.group;
      const int row = r0 + t * kRows + (threadIdx.x & 127);
      const int n = t ? w.n1 : w.n0;
      // The output goes by way of the query tile's place in shared memory, idle after its last scores, so that a
      // warp's stores are whole rows: written a row a lane, they took as long as three tiles.
      constexpr int kChunks = D * (MODE == kSplit ? 4 : 2) / 16;  // 16-byte pieces of a row
      auto stage = [&](int r, int chunk) {
        return reinterpret_cast<uint4 *>(smem + (it % C::QBufs * 2 + t) * C::QBytes) + r * kChunks + (chunk ^ (r & 7));
      };
      auto write_rows = [&] {
        __syncwarp();
        uint8_t *out = static_cast<uint8_t *>(a.o.data);
        constexpr int kSize = MODE == kSplit ? 4 : 2;
#pragma unroll 4
        for (int i = lane; i < 32 * kChunks; i += 32) {
          const int r = (warp & 3) * 32 + i / kChunks, chunk = i % kChunks, to = r0 + t * kRows + r;
          if (to < len)
            *reinterpret_cast<uint4 *>(out + ((start + to) * a.o.row_stride + head * a.o.head_stride) * kSize +
                                       16 * chunk) = *stage(r, chunk);
        }
        __syncwarp();
        if (sh.nonfinite[it & 1] && row < len)
          add_nonfinite<D>(out + ((start + row) * a.o.row_stride + head * a.o.head_stride) * kSize,
                           static_cast<const uint8_t *>(a.v.data) +
                               ((start + diag * BK) * a.v.row_stride + kv_head * a.v.head_stride) * kSize,
                           a.v.row_stride, row - diag * BK + 1, a.v.dtype);
      };
      if constexpr (MODE != kSplit) {
        // 16-bit rows: a tile's scores in registers, the output summed in tensor memory. The weights
        // are taken against `ref`, a maximum that may lag behind: only when a row's maximum has grown by more
        // than 2^kLag is the row's output scaled down (by its own thread), which a few tiles at a row's
        // start need. The largest weight is then 2^kLag; bfloat16 ones, which have the range below, are taken times
        // 2^-kLag, so that values next to the type's end do not leave 32 bits on the way. The maximum is taken off the scores before
        // they are scaled, so that it less itself is 0 whatever its size: in one fused step it would be what its product
        // was rounded by, which is beyond binary16 for scores of 2^27 (one instruction a pair of scores less, 1.3 %).
        float ref = 0, l = 0;
        const float c = a.scale;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          if (!wait(&sh.s_full[t][0], (count + j) & 1)) break;
          ptx::tc_fence_after();
          uint32_t x[BK / 16][16];
#pragma unroll
          for (int ch = 0; ch < BK / 16; ++ch) ptx::tmem_ld_32x32b_x16(s_addr + 16 * ch, x[ch]);
#pragma unroll
          for (int ch = 0; ch < BK / 16; ++ch) ptx::tmem_ld_wait(x[ch]);
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.s_free[t][0]);
          const int lim = row - j * BK;  // the last column that this row sees
          const bool masked = __any_sync(0xffffffffu, lim < BK - 1);
          if (masked) {
#pragma unroll
            for (int i = 0; i < BK; ++i)
              if (i > lim) x[i >> 4][i & 15] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(x[0][i]);
#pragma unroll
          for (int i = 4; i < BK; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // pairs i + 2 k, i + 2 k + 1 (the last group has one pair for two maxima)
              const int e = i + 2 * k;
              if (e + 1 < BK)
                mx[k] = max3(mx[k], __uint_as_float(x[e >> 4][e & 15]), __uint_as_float(x[(e + 1) >> 4][(e + 1) & 15]));
            }
          // A finite maximum, also where all scores are -infinity or NaN: those rows end as 0 / 0.
          const float m = fmaxf(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), -3.402823466e38f);
          // The last product is complete, its weights and its sum are free to be written.
          if (j > 0) {
            if (!wait(&sh.t_full[t], (count + j - 1) & 1)) break;
            ptx::tc_fence_after();
          }
          if (j == 0) {
            ref = m;
          } else if (__any_sync(0xffffffffu, (m - ref) * c > kLag)) {
            const float next = fmaxf(ref, m), alpha = ex2((ref - next) * c);
            const float2 al = make_float2(alpha, alpha);
            ref = next;
            l *= alpha;
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch) {
              uint32_t y[16];
              ptx::tmem_ld_32x32b_x16(t_addr + 16 * ch, y);
              ptx::tmem_ld_wait(y);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float2 z = __fmul2_rn(make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), al);
                y[i] = __float_as_uint(z.x);
                y[i + 1] = __float_as_uint(z.y);
              }
              ptx::tmem_st_32x32b_x16(t_addr + 16 * ch, y);
            }
          }
          const float2 cc = make_float2(c, c), rr = make_float2(-ref, -ref);
          float2 sum[2] = {make_float2(0, 0), make_float2(0, 0)};
          // The weights are rounded to the rows' type, half a step of each, as the matrix instructions take them beside
          // values of that type. Their sum is of the unrounded ones. Against 64 bits, 16 prompts of 301 to 4003: 2.1e-3
          // of the result's norm (bfloat16; 1.6e-3 is the result's own rounding), binary16 at dim 64 2.6e-4 (2.0e-4).
#pragma unroll
          for (int ch = 0; ch < BK / 16; ++ch) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 y =
                  __fadd2_rn(make_float2(__uint_as_float(x[ch][2 * i]), __uint_as_float(x[ch][2 * i + 1])), rr);
              if constexpr (MODE == kBf16) y = __ffma2_rn(y, cc, make_float2(-kLag, -kLag));
              else y = __fmul2_rn(y, cc);
              y = make_float2(ex2(y.x), ex2(y.y));
              sum[i & 1] = __fadd2_rn(sum[i & 1], y);
              w[i] = pack<MODE>(y.x, y.y);
            }
            ptx::tmem_st_32x32b_x8(s_addr + BK + 8 * ch, w);
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.p_full[t][0]);
        }
        if (ok && n > 0) wait(&sh.t_full[t], (count + n - 1) & 1);
        if (ok && n > 0) wait(&sh.looked_all, it & 1);
        if (ok && n > 0) {
          ptx::tc_fence_after();
          const float inv = 1.0f / l;
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t y[32];
            __syncwarp();
            ptx::tmem_ld_32x32b_x32(t_addr + 32 * ch, y);
            ptx::tmem_ld_wait(y);
            float o[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(y[i]) * inv;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *stage(threadIdx.x & 127, 4 * ch + i) =
                  make_uint4(pack<MODE>(o[8 * i], o[8 * i + 1]), pack<MODE>(o[8 * i + 2], o[8 * i + 3]),
                             pack<MODE>(o[8 * i + 4], o[8 * i + 5]), pack<MODE>(o[8 * i + 6], o[8 * i + 7]));
          }
          write_rows();
        }
      } else {
        float2 o[D / 2];
#pragma unroll
        for (int i = 0; i < D / 2; ++i) o[i] = make_float2(0, 0);
        float m = -INFINITY, l = 0, alpha = 0, v_pow = 1;
        float scale = a.scale;
        const int64_t pow0 = static_cast<int64_t>(kv_head) * a.tiles;
        const int tile0 = sh.item[it & 1].tile0;
        // rows behind the sequence are another's, or none: no scores of theirs make a tile rare
        scale = row < len ? scale * a.q_pow[static_cast<int64_t>(head) * a.tokens + start + row] : 0.0f;
        // o = o alpha + a tile's product
        auto accumulate = [&](int j, float alpha, float v_pow) {
          if (!wait(&sh.t_full[t], (count + j) & 1)) return;
          ptx::tc_fence_after();
          const float2 al = make_float2(alpha, alpha), vp = make_float2(v_pow, v_pow);
          uint32_t x[2][32];
          ptx::tmem_ld_32x32b_x32(t_addr, x[0]);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            ptx::tmem_ld_wait(x[c & 1]);
            if (c + 1 < D / 32) ptx::tmem_ld_32x32b_x32(t_addr + 32 * (c + 1), x[(c + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = make_float2(__uint_as_float(x[c & 1][2 * i]), __uint_as_float(x[c & 1][2 * i + 1]));
              float2 &z = o[16 * c + i];
              z = __ffma2_rn(z, al, __fmul2_rn(y, vp));
            }
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.p_full[t][(count + j + 1) & 1]);
        };
        // A tile whose rows have powers of two of their own, or whose scores may be far from zero (it is rare): its scores
        // become, in their place, the logarithms of the weights times their values' powers, less the largest, so that
        // the tile's own code finds weights of at most 2^13. What they are to be multiplied with, the maximum and the
        // sum are made here.
        struct Own {
          float m, l, alpha, v_pow;
        };
        auto spread_tile = [&](int j, uint32_t s_addr, float k_pow, float v_pow) {
          const int lim = row - j * BK;
          const int64_t first = start + static_cast<int64_t>(j) * BK;
          const int last = static_cast<int>(min(a.tokens - 1 - first, static_cast<int64_t>(BK - 1)));
          const float *kr = a.k_row + kv_head * a.tokens + first, *vr = a.v_row + kv_head * a.tokens + first;
          // f(score, its column) for all columns
          auto each = [&](auto f) {
#pragma unroll 1
            for (int ch = 0; ch < BK; ch += 16) {
              uint32_t x[16];
              ptx::tmem_ld_32x32b_x16(s_addr + ch, x);
              ptx::tmem_ld_wait(x);
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(f(__uint_as_float(x[i]), ch + i));
              __syncwarp();
              ptx::tmem_st_32x32b_x16(s_addr + ch, x);
            }
            ptx::tmem_st_wait();
          };
          float top = -3.402823466e38f;  // finite, also where all scores are -infinity or NaN
          float high = -120;             // what they are multiplied with is a normal number
          each([&](float x, int i) {
            x = i > lim ? -INFINITY : x * (scale * (k_pow < 0 ? __ldg(kr + min(i, last)) : k_pow));
            top = fmaxf(top, x);
            return x;
          });
          Own own;
          own.m = fmaxf(m, top);
          own.alpha = ex2(m - own.m);
          own.l = l * own.alpha;
          each([&](float x, int i) {
            x -= own.m;
            own.l += ex2(x + kWeightBits);
            const float v = i > lim ? 1.0f : v_pow < 0 ? __ldg(vr + min(i, last)) : v_pow;  // a power of two
            x += static_cast<int>(__float_as_uint(v) >> 23) - 127;
            high = fmaxf(high, x);
            return x;
          });
          each([&](float x, int) { return x - high; });
          own.v_pow = ex2(high);
          return own;
        };
        // A tile's weights come before the tile before it is added, whose factors are kept until then.
        auto tiles = [&](auto may_spread) {
#pragma unroll 1
          for (int j = 0; j < n && ok; ++j) {
            const int64_t at = pow0 + min(static_cast<int64_t>(tile0) + j, a.tiles - 1);
            const float k_pow = __ldg(a.k_pow + at);
            float v_next = __ldg(a.v_pow + at);
            const int b = (count + j) & 1;
            if (!wait(&sh.s_full[t][b], (count + j) >> 1 & 1)) break;
            ptx::tc_fence_after();
            const uint32_t s_addr = tmem + lanes + t * kScores + b * BK;
            const float alpha_last = alpha;
            const int lim = row - j * BK;  // the last column that this row sees
            float c = scale * k_pow;
            Own own;
            bool spread = false;
            if constexpr (decltype(may_spread)::value) {
              spread = __any_sync(0xffffffffu, k_pow < 0 || v_next < 0 || c > kFar);
              if (spread) {
                own = spread_tile(j, s_addr, k_pow, v_next);
                m = 0;
                c = 1;
              }
            }
            const bool masked = __any_sync(0xffffffffu, lim < BK - 1);
            // Four maxima and four pairs of sums, so that no addition waits for the one before.
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            float2 sum[4];
            float2 ref;
            const float2 cc = make_float2(c, c);
            auto start_load = [&](int ch, uint32_t (&x)[32]) { ptx::tmem_ld_32x32b_x32(s_addr + 32 * ch, x); };
            auto mask = [&](int ch, uint32_t (&x)[32]) {
              if (masked) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (32 * ch + i > lim) x[i] = 0xff800000u;
              }
            };
            auto top = [&](const uint32_t (&x)[32]) {
#pragma unroll
              for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(x[i]));
            };
            auto settle = [&] {
              const float all = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
              // A finite maximum, also where all scores are -infinity or NaN: those rows end as 0 / 0.
              const float m2 = fmaxf(m, fmaxf(all * c, -3.402823466e38f));
              const float r = kWeightBits - m2;
              ref = make_float2(r, r);
              alpha = ex2(m - m2);
              l *= alpha;
              m = m2;
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[i] = make_float2(0, 0);
            };
            // weights 2^(s c - ref), their sum, and 16 columns of pairs (two of them when split) to write back
            auto weights = [&](int ch, const uint32_t (&x)[32]) {
              uint32_t hi[16], lo[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float2 y = __ffma2_rn(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cc, ref);
                y = make_float2(ex2(y.x), ex2(y.y));
                sum[i & 3] = __fadd2_rn(sum[i & 3], y);
                hi[i] = pack<MODE>(y.x, y.y);
                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi[i]));
                const float2 rest = __fadd2_rn(y, make_float2(-h.x, -h.y));
                lo[i] = pack<MODE>(rest.x, rest.y);
              }
              ptx::tmem_st_32x32b_x16(s_addr + 16 * ch, hi);
              ptx::tmem_st_32x32b_x16(s_addr + BK / 2 + 16 * ch, lo);
            };
            uint32_t x0[32], x1[32];
            start_load(0, x0);
            ptx::tmem_ld_wait(x0);
            start_load(1, x1);
            mask(0, x0);
            top(x0);
            ptx::tmem_ld_wait(x1);
            mask(1, x1);  // both are read before the weights overwrite them
            top(x1);
            settle();
            weights(0, x0);
            weights(1, x1);
#pragma unroll
            for (int i = 0; i < 4; ++i) l += sum[i].x + sum[i].y;
            if (spread) {
              m = own.m;
              l = own.l;
              alpha = own.alpha;
              v_next = own.v_pow;
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.p_full[t][b]);
            if (j > 0) accumulate(j - 1, alpha_last, v_pow);
            else if (count == 0 && lane == 0) ptx::mbar_arrive(&sh.p_full[t][0]);  // nothing to read out yet
            v_pow = v_next;
          }
        };
        // Items with such a tile have a loop of their own: a branch in the other costs it 6 %, as its registers are full.
        float largest = 0, least = 1;
        for (int j = lane; j < n; j += 32) {
          const int64_t at = pow0 + min(static_cast<int64_t>(tile0) + j, a.tiles - 1);
          const float k_pow = __ldg(a.k_pow + at);
          largest = fmaxf(largest, k_pow);
          least = fminf(least, fminf(k_pow, __ldg(a.v_pow + at)));
        }
        largest = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(largest)));
        if (__any_sync(0xffffffffu, least < 0 || scale * largest > kFar)) tiles(std::true_type());
        else tiles(std::false_type());
        if (ok && n > 0) accumulate(n - 1, alpha, v_pow);
        if (ok && n > 0) wait(&sh.looked_all, it & 1);
        if (ok && row < len) {
          const float inv = static_cast<float>(1 << kWeightBits) / l;
#pragma unroll
          for (int i = 0; i < D / 2; ++i) o[i] = make_float2(o[i].x * inv, o[i].y * inv);
#pragma unroll
          for (int i = 0; i < D / 4; ++i)
            *stage(threadIdx.x & 127, i) = make_uint4(__float_as_uint(o[2 * i].x), __float_as_uint(o[2 * i].y),
                                                      __float_as_uint(o[2 * i + 1].x), __float_as_uint(o[2 * i + 1].y));
        }
        __syncwarp();
        if (ok && n > 0) write_rows();
      }
      if (!ok) break;
      count += n;
      // the copies of other queries into these rows' place come after what is read from it here
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.done[it & 1]);
    }
  }

  // ---- teardown: what this block has in flight ends, then its tensor memory is freed ----
  if (warp == 9 && lane == 0) {
    int no_abort = 0;
    ptx::mbar_wait_bounded(&sh.drain, 0, kDrainLimit, &no_abort);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::pdl_launch_dependents();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- float32 rows -> two binary16 planes [heads][tokens][dim] and their powers of two -------------------

struct SplitArgs {
  woq_rows q, k, v;
  const int32_t *cu;
  int64_t tokens, tiles;
  int batch;
  __half *planes[3][2];
  float *q_pow, *k_pow, *v_pow, *k_row, *v_row;
};

constexpr int kSplitThreads = 256;

// x = hi + lo with 22 bits; what is not finite (`finite`: nothing) stays as it is, with nothing beside it.
__device__ __forceinline__ void split4(float4 x, float up, bool finite, uint2 &hi, uint2 &lo) {
  auto two = [&](float a, float b, uint32_t &h, uint32_t &l) {
    const float2 y = __fmul2_rn(make_float2(a, b), make_float2(up, up));
    h = pack<kF16>(y.x, y.y);
    const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    float2 rest = __fadd2_rn(y, make_float2(-back.x, -back.y));
    if (!finite) {
      if (!isfinite(a)) rest.x = 0;
      if (!isfinite(b)) rest.y = 0;
    }
    l = pack<kF16>(rest.x, rest.y);
  };
  two(x.x, x.y, hi.x, lo.x);
  two(x.z, x.w, hi.y, lo.y);
}
// The larger of a and the largest |x|, NaN if there is one among them.
__device__ __forceinline__ float larger(float a, float4 x) {
  asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(x.x), "f"(x.y));
  asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(x.z), "f"(x.w));
  return a;
}
__device__ __forceinline__ float larger(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}
__device__ __forceinline__ float largest_finite(float4 x) {
  auto f = [](float y) { return isfinite(y) ? fabsf(y) : 0.0f; };
  return fmaxf(fmaxf(f(x.x), f(x.y)), fmaxf(f(x.z), f(x.w)));
}
// The power of two that a largest value in [2^13, 2^14) takes, within 2^+-113.
__device__ __forceinline__ int exponent(float big) {
  return big > 0 ? max(min(static_cast<int>(__float_as_uint(big) >> 23) - 140, 113), -113) : 0;
}

// Block (tile of 64 rows of a sequence, a head, or MANY of q, k and v): eight warps of eight rows, a lane four values of a
// row.
template <int D, bool MANY>
__global__ void __launch_bounds__(kSplitThreads, 4) attn_split_kernel(const SplitArgs a) {
  constexpr int LANES = D / 4, ROWS = 8 * LANES / 32;  // rows that a lane has
  __shared__ Place place;
  __shared__ int found;
  __shared__ uint2 warp_big[8];  // the largest of a warp's rows, and the least that is not 0, less one
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    Place p{};
    Cursor start{};
    const bool f = find_tile(a.cu, a.batch, a.tokens, blockIdx.x, kSplitRows, p, start);
    if (lane == 0) {
      place = p;
      found = f;
    }
  }
  __syncthreads();
  if (!found) return;
  const int hq = a.q.heads, hk = a.k.heads;
  for (int y = blockIdx.y; MANY ? y < hq + 2 * hk : y == static_cast<int>(blockIdx.y); y += gridDim.y) {
    const int which = y < hq ? 0 : y < hq + hk ? 1 : 2;
    const int head = which == 0 ? y : which == 1 ? y - hq : y - hq - hk;
    const woq_rows &src = which == 0 ? a.q : which == 1 ? a.k : a.v;
    const float *data = static_cast<const float *>(src.data);
    const int col = 4 * (lane % LANES);
    float4 x[ROWS];
    int row[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      row[i] = place.tile * kSplitRows + warp * 8 + i * (32 / LANES) + lane / LANES;
      x[i] = make_float4(0, 0, 0, 0);
      if (row[i] < place.len)
        x[i] = *reinterpret_cast<const float4 *>(data + (place.start + row[i]) * src.row_stride +
                                                 head * src.head_stride + col);
    }
    int ex = 0;
    bool finite = true, spread = false;
    const int less = which == 2 ? kWeightBits : 0;  // the weights' power is taken off the values'
    float size = 0;  // keys, values: the largest of the row that this lane has in row_sizes()
    if (which != 0) {
      // The block's rows: the bits of the largest value of all, and of the row with the least, if not 0, less one. Bits
      // order what is not negative, NaN above all. The lanes of a row share the work: each step halves its rows.
      auto row_sizes = [&](auto largest) {
        float b[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) b[i] = largest(x[i]);
#pragma unroll
        for (int n = ROWS / 2, k = LANES / 2; k > 0; n /= 2, k /= 2) {
          const bool upper = lane & k;
          if (n > 0) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
              const float other = __shfl_xor_sync(0xffffffffu, upper ? b[i] : b[i + n], k);
              b[i] = larger(upper ? b[i + n] : b[i], other);
            }
          } else {
            b[0] = larger(b[0], __shfl_xor_sync(0xffffffffu, b[0], k));
          }
        }
        size = b[0];
        const uint32_t bits = __float_as_uint(size);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, bits), lo = __reduce_min_sync(0xffffffffu, bits - 1);
        if (lane == 0) warp_big[warp] = make_uint2(hi, lo);
        __syncthreads();
        uint2 all = warp_big[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          const uint2 w = warp_big[i];
          all = make_uint2(max(all.x, w.x), min(all.y, w.y));
        }
        return all;
      };
      uint2 all = row_sizes([](float4 y) { return larger(0.0f, y); });
      finite = all.x < 0x7f800000u;
      if (!finite) {
        __syncthreads();
        all = row_sizes([](float4 y) { return largest_finite(y); });
      }
      ex = exponent(__uint_as_float(all.x));
      spread = all.x > 0 && (all.x >> 23) - (all.y + 1 >> 23) > kSpread;
      if (threadIdx.x == 0)
        (which == 1 ? a.k_pow : a.v_pow)[head * a.tiles + blockIdx.x] = spread ? -1.0f : power(ex - less);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (which == 0) {
        float b = larger(0.0f, x[i]);
#pragma unroll
        for (int k = 1; k < LANES; k <<= 1) b = larger(b, __shfl_xor_sync(0xffffffffu, b, k));
        finite = __all_sync(0xffffffffu, b < INFINITY);
        if (!finite) {
          b = largest_finite(x[i]);
#pragma unroll
          for (int k = 1; k < LANES; k <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, k));
        }
        ex = exponent(b);
      } else if (spread) {
        // row i of a lane's ROWS is with the lanes whose bits below the row's are i's, the highest first
        constexpr int kLow = LANES / ROWS;
        const float b = __shfl_sync(0xffffffffu, size, (lane / LANES) * LANES + i * kLow);
        ex = b > 0 ? exponent(b) : -113;  // a row of zeros has no part in what the others are taken times
      }
      if (row[i] >= place.len) continue;
      const int64_t t = static_cast<int64_t>(head) * a.tokens + place.start + row[i];
      if (which == 0 && col == 0) a.q_pow[t] = power(ex);
      if (spread && col == 0) (which == 1 ? a.k_row : a.v_row)[t] = power(ex - less);
      if (!finite && which != 2) {
        // An infinity in a query or key becomes NaN: beside the low plane's zeros and signs its products would be infinite
        // or NaN by chance.
        auto nan = [](float &y) { y = isfinite(y) ? y : __int_as_float(0x7fffffff); };
        nan(x[i].x);
        nan(x[i].y);
        nan(x[i].z);
        nan(x[i].w);
      }
      uint2 hi, lo;
      split4(x[i], power(-ex), finite, hi, lo);
      *reinterpret_cast<uint2 *>(a.planes[which][0] + t * D + col) = hi;
      *reinterpret_cast<uint2 *>(a.planes[which][1] + t * D + col) = lo;
    }
    if (MANY) __syncthreads();  // warp_big
  }
}

// ---- host side -------------------------------------------------------------------------------------------

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

int64_t split_tiles(int64_t tokens, int32_t batch) { return tokens / kSplitRows + batch; }

template <int D, int MODE>
int launch(const Maps &maps, const Args &a, cudaStream_t s, const DevInfo &dev) {
  using C = Cfg<D, MODE>;
  auto kern = attn_prompt_kernel<D, MODE>;
  static_assert(sizeof(Shared) <= 1024, "barriers");
  static std::once_flag once[64];
  static cudaError_t err[64];
  std::call_once(once[dev.device], [&] {
    err[dev.device] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::Smem);
    cudaFuncAttributes fa;
    // The helpers' registers go to the others out of what a block is launched with: it has to be all of it (the build
    // checks that as well).
    if (err[dev.device] == cudaSuccess) err[dev.device] = cudaFuncGetAttributes(&fa, kern);
    if (err[dev.device] == cudaSuccess && fa.numRegs != kLaunchRegs) err[dev.device] = cudaErrorInvalidValue;
  });
  if (err[dev.device] != cudaSuccess) return WOQ_ECUDA;
  const int64_t blocks = (a.tokens / kBlockRows + a.batch) * a.q_heads;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::Smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, maps, a) != cudaSuccess) return WOQ_ECUDA;
  count_launches(1);
  return WOQ_OK;
}

template <int D>
int launch_split(const SplitArgs &a, cudaStream_t s, const DevInfo &dev) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // A head a block, so that a tile's loads are under way at once in all of them. With more sequences than the lookup
  // of a tile takes in a few steps, a block looks it up for several heads, in eight rounds of blocks.
  // 4096 sequences of a row, 16 and 8 heads: the whole call 3.6 instead of 6.8 ms; 300 of them 0.30 and 0.32.
  const bool many = a.batch > 256;
  const int64_t heads = a.q.heads + 2 * a.k.heads, rounds = (int64_t(dev.sm_count) * 4 * 8 + a.tiles - 1) / a.tiles;
  cfg.gridDim =
      dim3(static_cast<unsigned>(a.tiles), static_cast<unsigned>(many ? std::min(heads, rounds) : heads), 1);
  cfg.blockDim = dim3(kSplitThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kern = many ? attn_split_kernel<D, true> : attn_split_kernel<D, false>;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return WOQ_ECUDA;
  count_launches(1);
  return WOQ_OK;
}

// The workspace of float32 rows: six planes, then the powers of two, and those of single keys and values.
struct Layout {
  size_t plane[3], pow[3], row[3], total;
};
Layout layout(int64_t tokens, int32_t batch, int32_t hq, int32_t hk, int32_t dim) {
  Layout L;
  const size_t t = static_cast<size_t>(tokens);
  const size_t heads[3] = {static_cast<size_t>(hq), static_cast<size_t>(hk), static_cast<size_t>(hk)};
  size_t at = 0;
  for (int i = 0; i < 3; ++i) {
    L.plane[i] = at;
    at += 2 * up256(heads[i] * t * dim * 2);
  }
  const size_t tiles = static_cast<size_t>(split_tiles(tokens, batch));
  for (int i = 0; i < 3; ++i) {
    L.pow[i] = at;
    at += up256(heads[i] * (i == 0 ? t : tiles) * 4);
    L.row[i] = at;
    if (i > 0) at += up256(heads[i] * t * 4);
  }
  L.total = at;
  return L;
}

}  // namespace

size_t attn_prompt_workspace(int64_t tokens, int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t dim,
                             int32_t dtype) {
  return dtype == WOQ_F32 ? layout(tokens, batch, q_heads, kv_heads, dim).total : 0;
}

int launch_attn_prompt(const woq_rows &q, const woq_rows &k, const woq_rows &v, int64_t tokens, const int32_t *cu,
                       int32_t batch, int32_t dim, float scale, const woq_rows &o, void *workspace, cudaStream_t s,
                       const DevInfo &dev) {
  Args a = {};
  a.cu = cu;
  a.tokens = tokens;
  a.batch = batch;
  a.q_heads = q.heads;
  a.group = q.heads / k.heads;
  a.scale = scale * 1.44269504088896340736f;
  a.o = o;
  a.v = v;
  a.tiles = split_tiles(tokens, batch);
  const long long lim = wait_limit_cycles();
  a.wait_limit = lim > 0 ? lim : kWaitLimit;
  a.stuck_wait = lim < 0 ? -lim : 0;
  const int mode = q.dtype == WOQ_F32 ? kSplit : q.dtype == WOQ_F16 ? kF16 : kBf16;
  const CUtensorMapDataType type =
      mode == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  Maps maps = {};
  SplitArgs sp = {};
  const woq_rows *rows[3] = {&q, &k, &v};
  CUtensorMap *dst[3] = {maps.q, maps.k, maps.v};
  const Layout L = mode == kSplit ? layout(tokens, batch, q.heads, k.heads, dim) : Layout{};
  for (int i = 0; i < 3; ++i) {
    const uint32_t box = i == 0 ? kRows
                         : mode == kSplit ? Cfg<128, kSplit>::BK  // the same for both dims
                         : dim == 128     ? Cfg<128, kBf16>::BK
                                          : Cfg<64, kBf16>::BK;
    for (int p = 0; p < (mode == kSplit ? 2 : 1); ++p) {
      const void *base = rows[i]->data;
      int64_t head_stride = rows[i]->head_stride, row_stride = rows[i]->row_stride;
      if (mode == kSplit) {
        head_stride = tokens * dim;
        row_stride = dim;
        sp.planes[i][p] = reinterpret_cast<__half *>(
            static_cast<uint8_t *>(workspace) + L.plane[i] +
            p * up256(static_cast<size_t>(rows[i]->heads) * static_cast<size_t>(tokens) * dim * 2));
        base = sp.planes[i][p];
      }
      if (!make_tensor_map_3d(&dst[i][p], type, 2, base, dim, rows[i]->heads, tokens, head_stride, row_stride, 64, box,
                              CU_TENSOR_MAP_SWIZZLE_128B))
        return WOQ_ECUDA;
    }
  }
  if (mode == kSplit) {
    float *pow[3], *row[3];
    for (int i = 0; i < 3; ++i) {
      pow[i] = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + L.pow[i]);
      row[i] = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + L.row[i]);
    }
    a.q_pow = sp.q_pow = pow[0];
    a.k_pow = sp.k_pow = pow[1];
    a.v_pow = sp.v_pow = pow[2];
    a.k_row = sp.k_row = row[1];
    a.v_row = sp.v_row = row[2];
    sp.q = q;
    sp.k = k;
    sp.v = v;
    sp.cu = cu;
    sp.tokens = tokens;
    sp.tiles = a.tiles;
    sp.batch = batch;
    const int rc = dim == 128 ? launch_split<128>(sp, s, dev) : launch_split<64>(sp, s, dev);
    if (rc != WOQ_OK) return rc;
  }
  if (dim == 128)
    return mode == kSplit ? launch<128, kSplit>(maps, a, s, dev)
           : mode == kF16 ? launch<128, kF16>(maps, a, s, dev)
                          : launch<128, kBf16>(maps, a, s, dev);
  return mode == kSplit ? launch<64, kSplit>(maps, a, s, dev)
         : mode == kF16 ? launch<64, kF16>(maps, a, s, dev)
                        : launch<64, kBf16>(maps, a, s, dev);
}

int read_prompt_timeout_flag(int clear, unsigned *value) {
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_prompt_timeout_flag, sizeof(v)) != cudaSuccess) return WOQ_ECUDA;
  if (clear && v) {
    const unsigned z = 0;
    if (cudaMemcpyToSymbol(g_prompt_timeout_flag, &z, sizeof(z)) != cudaSuccess) return WOQ_ECUDA;
  }
  *value = v;
  return WOQ_OK;
}

}  // namespace woq
