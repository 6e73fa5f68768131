// Attention of a tree of drafted tokens per sequence over its rows' paged cache and window ring.
// The m drafted tokens of a sequence are the last m paged tokens of its rows; token i sees all
// keys before them, the ring's, and of the drafted ones itself and those above it in the tree:
//   o_i = sum_k a_ik v_k,  a_ik = exp(q_i . k / sqrt(d) - lse_i) over what it sees.
//
// The g query heads of a KV head and the m tokens make m g query rows that read the same keys:
// 4 d bytes and 4 d m g flops a key.  Up to 128 rows, one M = 128 tile of tcgen05, HBM bounds it
// (64 rows: 64 flop/B where the chip has 286); more rows take more tiles, which read the keys
// again from L2.
//
// Rows differ in length by the pruning, so the work is cut by tiles of 128 keys, not by rows: the
// tiles of all (row, query tile) pairs form one stream, every block of a persistent grid takes an
// equal contiguous share, and a pair that crosses a share's border is joined from partial sums
// (running maximum, sum and weighted values) by a second kernel.  Shares depend on the lengths
// alone, so results do too.  In a block:
//   warps 0-3   copy 32 keys each of every K and V tile into two 3-stage rings, in the 128-byte
//               swizzled layout that the tensor core reads: whole runs of keys in pages that 32 keys
//               divide or are divided by come as TMA boxes, all others by 16-byte cp.async (pages may
//               be of any size and end anywhere in a tile, and so may the ring begin)
//   warps 4-11  softmax, two threads per query row: S from TMEM, p = 2^(x - m), P as bf16 to TMEM
//   warps 12, 14  issue S = Q K^T (Q in TMEM) and O += P V (P in TMEM), M = 128 each; one warp for
//               both spent its time issuing (1.2 us a tile)
//   warp 13     finds the share's units and brings the page ids of the tiles to come, six tiles ahead
//               (under a saturated HBM a load takes longer than a tile)
// The registers of a block go to the softmax (setmaxnreg: 184 a thread, 96 for the copies, 48 for
// the rest: with fewer the copies or the rest spill, which costs up to 10 us in 52).  S is
// double-buffered in TMEM, so that the products of one tile run beside the softmax of the one
// before.  O is rescaled only when a row's maximum grows by more than 2^8.
//
// Measured, a call in a graph: 8 drafts of one short sequence 12.2 us, 64 sequences of up to 2048
// tokens 52 (floor 30), 33 with rings and pages of 13 20.7 (5), a document of 131072 tokens with 64
// drafts 59 (22), wide trees at d = 64 246 (63), 96 sequences of 16384 tokens 372 (362: 6.6 TB/s).
// A tile with all 128 rows takes 2100 cycles: the softmax of two warps an SM quarter 1400, a wait
// that is over 180, P to TMEM 220, on to the next tile 330; the tensor pipe is 22 % and the issue
// slots are 53 % busy.  P in two buffers (at d = 128 in the place of S) changed that little, 262
// for 246 and 50 for 52; scores read a tile ahead cost 275 for 249, K and V copied by two warps
// each 259 and 62 for 246 and 52.
//
// Which drafted tokens a token sees is a row of 256 bits, closed over the parents in log2(depth)
// rounds at the start of a (row, query tile) whose share reaches the drafted keys.  A masked key
// must not reach a row through 0 x inf: the V rows of drafted tokens are searched for infinities
// and NaN, these multiply as zeros, and rows that do see them get them added at the end.
#include <algorithm>

#include <math_constants.h>

#include "attn_tree.cuh"
#include "launch.cuh"
#include "tc.cuh"

namespace kvs {

__device__ int g_attn_tree_error = 0;

namespace {

constexpr int kErrWaitTimeout = 1;
constexpr int kErrAttnTree = 10;  // a token start, parent, length or page id out of range

constexpr int BM = 128;        // query rows of a tile = TMEM lanes
constexpr int BN = 128;        // keys of a tile
constexpr int kStages = 3;     // of the K ring and of the V ring
constexpr int kCopyWarps = 4;  // 32 keys of a tile each
constexpr int kSoftWarp = 4, kScoreWarp = 12, kFindWarp = 13, kValueWarp = 14;
constexpr int kSoftThreads = 256;
constexpr int kThreads = 16 * 32;  // the last warp only makes up the four
constexpr int kWarps = kThreads / 32;
constexpr int KC = BN / 2;     // keys of a softmax thread and tile
constexpr int kAhead = 8;      // tiles whose page ids are on their way or not yet used
constexpr uint32_t kBox = 128 * 128;  // 128 rows x 64 bf16 (one 128-byte swizzle span)
constexpr uint32_t kTmemCols = 512;
constexpr int kCopyRegs = 96, kSoftRegs = 184, kMmaRegs = 48;
static_assert(kCopyRegs + 2 * kSoftRegs + kMmaRegs <= 65536 / 128, "what the launch has");
constexpr float kRescale = 8.f;  // log2 growth of the row max that forces a rescale of O
constexpr int kMaxBlocks = 160;  // of the persistent grid; sizes the workspace
constexpr int kWords = kMaxDraft / 32;
constexpr long long kL2Bytes = 129ll << 20;
constexpr int kJoinThreads = 256;
constexpr int kUnits = 8;        // units that are known ahead
constexpr int kDirty = 2 * kUnits;  // units whose mark for non-finite drafts is kept
// Tiles whose bits of keys that are there are kept: a copy of tile i + 6 waits for the S product
// of i + 3, and that for the softmax of i + 1.
constexpr int kLive = 8;
constexpr uint32_t kMaxSmem = 232448;

template <int D>
struct Cfg {
  static constexpr uint32_t TILE = D / 64 * kBox;  // one K or V tile
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = OFF_K + kStages * TILE;
  static constexpr uint32_t OFF_XM = OFF_V + kStages * TILE;     // row max exchange [2][2][BM]
  static constexpr uint32_t OFF_XL = OFF_XM + 4 * BM * 4;        // row sum exchange [2][BM]
  static constexpr uint32_t OFF_SEES = OFF_XL + 2 * BM * 4;      // [kMaxDraft][kWords]
  static constexpr uint32_t OFF_UP = OFF_SEES + kMaxDraft * kWords * 4;  // [kMaxDraft]
  static constexpr uint32_t OFF_BAR = OFF_UP + kMaxDraft * 4;
  // q, k_full[3], k_empty[3], v_full[3], v_empty[3], s_full[2], s_empty[2], p[2], o[2], done,
  // ids_full[8], ids_empty[8], unit_full[8], unit_empty[8]
  static constexpr uint32_t NBAR = 22 + 2 * kAhead + 2 * kUnits;
  static constexpr uint32_t USED = OFF_BAR + NBAR * 8;
  static constexpr uint32_t SMEM = USED + 1024;
  // TMEM columns: S buffers, then P (bf16 pairs of one tile), Q (bf16 pairs), O
  static constexpr uint32_t COL_P = 2 * BN, COL_Q = COL_P + BN / 2, COL_O = COL_Q + D / 2;
  static_assert(COL_O + D <= kTmemCols, "TMEM plan");
  static_assert(SMEM + 6144 <= kMaxSmem, "shared-memory plan");
};

// A partial result: O transposed in chunks of four columns [D / 4][BM], then the reference and
// the sum of each row.
__host__ __device__ constexpr int part_floats(int d) { return BM * d + 2 * BM; }

// Workspace: per block the (row, query tile) that ends there having begun in another block (row
// -1: none) and that other block; per block the parts of the pairs that cross its borders (0:
// began before, 1: goes on after).
struct Ends { int row, mt, first, pad; };
__host__ __device__ constexpr size_t ends_bytes() { return kMaxBlocks * sizeof(Ends); }
__device__ __forceinline__ float* block_part(void* ws, int block, int side, int pf) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + ends_bytes()) +
         (size_t)(2 * block + side) * pf;
}

__device__ __forceinline__ void fault() { atomicCAS(&g_attn_tree_error, 0, kErrAttnTree); }

// What a row holds: paged keys, all keys with the ring's, its sequence's first token and their
// number (negative where the token starts are bad).
struct Row {
  int paged, all, t0, m;
  __device__ __forceinline__ int tiles() const { return (all + BN - 1) / BN; }
  __device__ __forceinline__ int first() const { return paged - m; }  // slot of drafted token 0
};

__device__ __forceinline__ Row row_of(const AttnTreeArgs& a, int r) {
  const int b = r - a.by_batch.of(r) * a.B, t0 = a.tok_start[b], t1 = a.tok_start[b + 1];
  const int paged = max(0, min(a.seq_lens[r], a.max_pages * a.page_size));
  const bool good = t0 >= 0 && t1 >= t0 && t1 <= a.N && t1 - t0 <= a.max_draft;
  return {paged, paged + (a.w > 0 ? max(0, min(a.pos[b], a.w)) : 0), t0, good ? t1 - t0 : -1};
}

__device__ __forceinline__ int query_tiles(int m, int g) { return (max(m, 0) * g + BM - 1) / BM; }

// Segment of a (row, query tile) in a block's share; none behind the last.
struct Unit {
  int row, mt, ta, tb;  // key tiles ta .. tb - 1
  Row is;
  __device__ __forceinline__ bool none() const { return ta == tb; }
  __device__ __forceinline__ bool whole() const { return ta == 0 && tb == is.tiles(); }
};

// Walks through the units of a share: the lanes of one warp hold 32 rows.
struct Walk {
  int base, left;
  Row mine;
  Unit u;

  __device__ __forceinline__ void cut() {
    u.tb = min(u.is.tiles(), u.ta + left);
    left -= u.tb - u.ta;
  }
  // the next unit; from a row that is not there (base = row | 31) the first one behind it
  __device__ __forceinline__ bool next(const AttnTreeArgs& a, int rows, int g, int lane) {
    if (left <= 0) return false;
    if (u.mt + 1 < query_tiles(u.is.m, g)) {
      ++u.mt;
    } else {
      u.mt = 0;
      int from = u.row - base + 1;
#pragma unroll 1
      for (;;) {
        if (from >= 32) {
          base += from;
          from = 0;
          if (base >= rows) return false;  // only if lengths change under the call
          mine = {0, 0, 0, 0};
          if (base + lane < rows) mine = row_of(a, base + lane);
        }
        const uint32_t some = __ballot_sync(0xffffffffu, mine.all > 0 && mine.m > 0) & 0xffffffffu << from;
        if (some) {
          const int r = __ffs(some) - 1;
          u.row = base + r;
          u.is.paged = __shfl_sync(0xffffffffu, mine.paged, r);
          u.is.all = __shfl_sync(0xffffffffu, mine.all, r);
          u.is.t0 = __shfl_sync(0xffffffffu, mine.t0, r);
          u.is.m = __shfl_sync(0xffffffffu, mine.m, r);
          break;
        }
        from = 32;
      }
    }
    u.ta = 0;
    cut();
    return true;
  }
};

// Equal contiguous shares of `blocks` blocks of a stream of fewer than 2^31 tiles; the first
// `more` have one more than `each`.
struct Shares {
  int each = 1, more = 0;
  __device__ __forceinline__ Shares(int total, int blocks) {
    if (total > blocks) {
      each = total / blocks;
      more = total - each * blocks;
    }
  }
  __device__ __forceinline__ int first(int block) const { return block * each + min(block, more); }
  __device__ __forceinline__ int of(int tile) const {  // block of a tile
    const int wide = more * (each + 1);
    return tile < wide ? tile / (each + 1) : more + (tile - wide) / each;
  }
};

// 64 of the bits of a token's row from bit `off` on (which may be negative); bits outside are 0.
__device__ __forceinline__ uint64_t bits_from(const uint32_t* row, int off) {
  uint32_t w[3];
  const int w0 = off >> 5, s = off & 31;  // rounds down
#pragma unroll
  for (int i = 0; i < 3; ++i) w[i] = (uint32_t)(w0 + i) < (uint32_t)kWords ? row[w0 + i] : 0u;
  return (uint64_t)__funnelshift_r(w[1], w[2], s) << 32 | __funnelshift_r(w[0], w[1], s);
}
// The same of a row of one word.
__device__ __forceinline__ uint64_t bits_of(uint32_t row, int off) {
  return off >= 32 || off <= -64 ? 0ull : off >= 0 ? (uint64_t)(row >> off) : (uint64_t)row << -off;
}
// The lowest n of 64 bits.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7f80u) == 0x7f80u; }
// Bits 15 and 31: whether either half is not finite (its exponent plus one carries).
__device__ __forceinline__ uint32_t not_finite2(uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; }

// A value that the compiler does not see through: loops stay loops (it peels those whose first or
// last turns differ, which made 20 KB of the search for page ids).
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

__device__ __forceinline__ void named_sync(int id, int nthreads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// Registers a thread from here on; all warps of four call it.  (As the other .aligned instructions
// here it wants its warp together, which a branch before it does not promise.)
template <int N>
__device__ __forceinline__ void give_registers() {
  __syncwarp();
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
  __syncwarp();
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 16-byte async copy global -> shared; keys and values that the call reads once are the first to
// leave L2, so that what is read again stays.
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
template <bool kOnce>
__device__ __forceinline__ void cp_async16_whole(uint32_t dst, const void* src, uint64_t policy) {
  if constexpr (kOnce)
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(dst),
                 "l"(src), "l"(policy));
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src));
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src));
}

// The phase of `bar` that is going on also waits for all copies that this thread has started.
__device__ __forceinline__ void wait_for_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}
template <bool kOnce>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                         int c1, int c2, uint64_t policy) {
  if constexpr (kOnce)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
  else
    tc::tma_load_3d(dst, map, bar, c0, c1, c2);
}

__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float lse_of(float ref, float sum) {
  return sum == 0.f ? -INFINITY : kLn2 * (ref + log2f(sum));
}

// What the copies of a tile need to know of it.
struct TileAt {
  int row, key0, paged, all, first, m, unit, pad;
};

// A warp's copies of its 32 keys of a tile: D / 8 lanes a row, each group of lanes a run of rows,
// so that a lane finds the places of its rows by itself.
template <int D, bool kOnce>
struct Copies {
  static constexpr int kLanes = D / 8, kRows = kLanes;  // lanes of a row; rows of a group of lanes
  const AttnTreeArgs& a;
  const int warp, lane;
  const uint64_t policy;

  // Of the tile: the lane's key's row in the pool or in the rings (rows of a pool that fits the GPU
  // stay within 32 bits), and which of the 32 keys are there and which are in the ring.
  uint32_t at_row = 0, there = 0, ringed = 0;
  __device__ __forceinline__ void resolve(const TileAt& at, const int* ids) {
    const int key = at.key0 + warp * 32 + lane;
    const bool paged = key < at.paged;
    bool ok = key < at.all;
    if (paged) {
      const int page = ids[warp * 32 + lane], idx = a.by_page.of(key);
      ok = (uint32_t)page < (uint32_t)a.capacity;
      at_row = (uint32_t)page * (uint32_t)a.page_size + (uint32_t)(key - idx * a.page_size);
      if (!ok) fault();
    } else {
      at_row = (uint32_t)at.row * (uint32_t)a.w + (uint32_t)(key - at.paged);
    }
    there = __ballot_sync(0xffffffffu, ok);
    ringed = __ballot_sync(0xffffffffu, !paged);
  }
  // row of the tile of this lane's i-th copy, and where the copy goes
  __device__ __forceinline__ int row(int i) const { return warp * 32 + lane / kLanes * kRows + i; }
  __device__ __forceinline__ uint32_t place(int i) const {
    const int c = lane % kLanes;
    return (uint32_t)(c >> 3) * kBox + row(i) * 128 + (((c & 7) ^ (row(i) & 7)) << 4);
  }
  // The keys that are there; what is not becomes zeros if asked for (of V: a weight of 0 times what
  // lies there must be 0; scores of keys that are not there are masked).  A lone warp issues an
  // instruction every few cycles, so a row is few of them: in a loop that chooses between page and
  // ring row by row, 32 keys took 2400 cycles (33 rings and pages of 13: 24.4 us for 20.7).
  __device__ __forceinline__ void copy_rows(bool zeros, const bf16_t* pages, const bf16_t* ring,
                                            uint32_t tile) const {
    const int c = lane % kLanes * 8;
    const uint32_t in_ring = there & ringed;
    // the first keys, all in pages or all in the ring: nothing to choose in a row
    if (!(there & (there + 1)) && (!in_ring || in_ring == there)) {
      const int r0 = row(0) - warp * 32;
      const bf16_t* from = (in_ring ? ring : pages) + c;
      const int mine = __popc(there >> r0 & ((1u << kRows) - 1));
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const uint32_t r = __shfl_sync(0xffffffffu, at_row, r0 + i);
        if (i < mine) cp_async16_whole<kOnce>(tile + place(i), from + (size_t)r * D, policy);
      }
      if (zeros && ~there) {
#pragma unroll 1
        for (int i = 0; i < kRows; ++i)
          if (i >= mine)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + place(i)), "r"(0) : "memory");
      }
      return;
    }
#pragma unroll 1
    for (int i0 = 0; i0 < kRows; i0 += 2) {
      const int r0 = row(i0) - warp * 32;
      uint32_t r[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) r[j] = __shfl_sync(0xffffffffu, at_row, r0 + j);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bf16_t* base = ringed >> (r0 + j) & 1 ? ring : pages;
        const uint32_t to = tile + place(i0 + j);
        if (there >> (r0 + j) & 1)
          cp_async16_whole<kOnce>(to, base + (size_t)r[j] * D + c, policy);
        else if (zeros)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
      }
    }
  }
  // The same 32 keys by TMA, where pages divide them or they pages: a lane a box of up to 32 rows of
  // 64 elements.
  __device__ __forceinline__ void copy_boxes(const TileAt& at, const int* ids, const CUtensorMap* map,
                                             uint32_t tile, uint32_t bar) const {
    constexpr int KH = D / 64;
    const int r = lane / KH * a.box_rows;
    if (r < 32) {
      const int key = at.key0 + warp * 32 + r, inside = key - a.by_page.of(key) * a.page_size;
      tma_load<kOnce>(tile + lane % KH * kBox + (warp * 32 + r) * 128, map, bar, lane % KH * 64, inside,
                      ids[warp * 32 + r], policy);
    }
    __syncwarp();
  }
  // Drafted rows lo .. hi - 1 of this warp's 32 of a V tile that has landed: what is not finite
  // becomes 0; true if there was any.  A lane looks at the chunks that it copied.
  __device__ __forceinline__ bool clean(uint8_t* tile, int lo, int hi) const {
    bool any = false;
#pragma unroll 4
    for (int i = 0; i < kRows; ++i) {
      const int r = row(i) - warp * 32;
      if (r < lo || r >= hi) continue;
      const uint4 x = *reinterpret_cast<const uint4*>(tile + place(i));
      any |= ((not_finite2(x.x) | not_finite2(x.y) | not_finite2(x.z) | not_finite2(x.w)) & 0x80008000u) != 0;
    }
    if (!any) return false;
#pragma unroll 1
    for (int i = 0; i < 4 * kRows; ++i) {
      const int r = row(i >> 2) - warp * 32;
      if (r < lo || r >= hi) continue;
      uint32_t* x = reinterpret_cast<uint32_t*>(tile + place(i >> 2)) + (i & 3);
      uint32_t y = *x;
      if (not_finite(y)) y &= 0xffff0000u;
      if (not_finite(y >> 16)) y &= 0xffffu;
      *x = y;
    }
    return true;
  }
};

// The rest of a wait that does not end at once; false if it runs out, or another's in the block.
// Threads that wait leave the others their issue slots: those that work ahead sleep, the others turn
// in a loop of four instructions.
template <int kSleepNs>
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  const uint64_t t0 = tc::globaltimer();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
      if (tc::mbar_try_wait(bar, parity)) return true;
      if constexpr (kSleepNs > 0) __nanosleep(kSleepNs);
    }
    if (*abort_flag) return false;
    if (tc::globaltimer() - t0 > tc::kWaitLimitNs) {
      *abort_flag = 1u;
      return false;
    }
  }
}

// The code is kept small: at 120 KB (a walk through the rows in every warp, a copy loop per case)
// the warps waited for instructions a third of the time, 1.4 us a tile; now, at 80 to 89 KB, a
// sixteenth at d = 64 and a twelfth at 128.
template <int D, bool kOnce>
__global__ void __launch_bounds__(kThreads, 1) attn_tree_kernel(
    const __grid_constant__ AttnTreeArgs a, const __grid_constant__ CUtensorMap map_k,
    const __grid_constant__ CUtensorMap map_v, int rows) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int warp_tiles[kWarps];
  __shared__ int start_s[1];                 // tiles of all rows
  __shared__ uint32_t misc[2];               // TMEM address, abort flag
  __shared__ __align__(16) TileAt at_s[kAhead];
  __shared__ __align__(16) Unit unit_s[kUnits];
  __shared__ __align__(16) int ids_s[kAhead][BN];          // page ids of a tile's keys
  __shared__ volatile uint32_t live_s[kLive][kCopyWarps];  // keys of a tile that are there
  __shared__ volatile int dirty_s[kDirty];   // n + 1: unit n has drafted values that are not finite
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  const uint32_t sK = sb + C::OFF_K, sV = sb + C::OFF_V;
  float* xm = reinterpret_cast<float*>(smem + C::OFF_XM);
  float* xl = reinterpret_cast<float*>(smem + C::OFF_XL);
  uint32_t* sees = reinterpret_cast<uint32_t*>(smem + C::OFF_SEES);
  int* up = reinterpret_cast<int*>(smem + C::OFF_UP);
  const uint32_t bar0 = sb + C::OFF_BAR;
  const uint32_t bar_q = bar0;  // the query rows are in TMEM (softmax threads arrive)
  auto bar_kfull = [&](int s) { return bar0 + 8u * (1 + s); };
  auto bar_kempty = [&](int s) { return bar0 + 8u * (4 + s); };
  auto bar_vfull = [&](int s) { return bar0 + 8u * (7 + s); };
  auto bar_vempty = [&](int s) { return bar0 + 8u * (10 + s); };
  auto bar_sfull = [&](int s) { return bar0 + 8u * (13 + s); };   // S buffer s = tile & 1
  auto bar_sempty = [&](int s) { return bar0 + 8u * (15 + s); };  // the softmax read it
  // P(i) is ready on p[i & 1] and O += P(i) V(i) completes on o[i & 1]: the softmax waits for
  // P V(i - 1) before it writes P(i), so neither barrier runs two phases ahead of a waiter
  auto bar_p = [&](int i) { return bar0 + 8u * (17 + (i & 1)); };
  auto bar_o = [&](int i) { return bar0 + 8u * (19 + (i & 1)); };
  const uint32_t bar_done = bar0 + 8u * 21;
  auto bar_ids = [&](int s) { return bar0 + 8u * (22 + s); };
  auto bar_idsfree = [&](int s) { return bar0 + 8u * (22 + kAhead + s); };
  auto bar_unit = [&](int n) { return bar0 + 8u * (22 + 2 * kAhead + n % kUnits); };
  auto bar_unitfree = [&](int n) { return bar0 + 8u * (22 + 2 * kAhead + kUnits + n % kUnits); };
  volatile uint32_t* abort_flag = misc + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.Hq / a.Hkv;

  if (tid == 0) {
    tc::mbar_init(bar_q, kSoftThreads);
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(bar_kfull(s), kCopyWarps);
      tc::mbar_init(bar_kempty(s), 1);
      tc::mbar_init(bar_vfull(s), kCopyWarps);
      tc::mbar_init(bar_vempty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(bar_sfull(s), 1);
      tc::mbar_init(bar_sempty(s), kSoftThreads);
      tc::mbar_init(bar_p(s), kSoftThreads);
      tc::mbar_init(bar_o(s), 1);
    }
    tc::mbar_init(bar_done, 2);
    for (int s = 0; s < kAhead; ++s) {
      tc::mbar_init(bar_ids(s), 1);
      tc::mbar_init(bar_idsfree(s), kCopyWarps);
    }
    for (int s = 0; s < kUnits; ++s) {
      tc::mbar_init(bar_unit(s), 1);
      tc::mbar_init(bar_unitfree(s), kSoftThreads / 32 + 2);
    }
    misc[1] = 0u;
    tc::fence_mbar_init();
  }
  if (tid < kDirty) dirty_s[tid] = 0;
  // started beside the end of the kernel before; the join must not start beside that one too
  wait_for_previous();
  let_next_start();

  // --- tiles of all rows, every thread a contiguous range of them; in a second pass the row, query
  // tile and key tile where the share begins
  const int per = (rows + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, rows), r1 = min(r0 + per, rows);
  Ends* ends = static_cast<Ends*>(a.ws);
  int mine = 0, before = 0, s0 = -1, tiles = 0;
#pragma unroll 1
  for (int pass = opaque(0); pass < 2; ++pass) {
    if (pass == 0 || (before <= s0 && s0 < before + mine)) {
      int at = s0 - before;
#pragma unroll 1
      for (int r = r0; r < r1; ++r) {
        const Row x = row_of(a, r);
        const int nt = x.tiles(), n = nt * query_tiles(x.m, g);  // 0 without drafted tokens
        if (pass == 0) {
          mine += n;
          if (blockIdx.x == 0 && (a.seq_lens[r] != x.paged || x.paged < x.m || x.m < 0)) fault();
        } else if (at < n) {
          const int mt = at / nt, ta = at - mt * nt;
          Unit u = {r, mt, ta, min(nt, ta + tiles), x};
          unit_s[0] = u;
          Ends e = {-1, 0, 0, 0};
          if (ta > 0 && u.tb == nt) e = {r, mt, Shares(start_s[0], gridDim.x).of(s0 - ta), 0};
          ends[blockIdx.x] = e;
          break;
        } else {
          at -= n;
        }
      }
    }
    if (pass) break;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_tiles[warp] = incl;
    if (tid == 0) unit_s[0] = {0, 0, 0, 0, {0, 0, 0, 0}};  // stays only if lengths change under the call
    __syncthreads();
    const int theirs = lane < kWarps ? warp_tiles[lane] : 0;  // every warp for itself
    const int total = __reduce_add_sync(0xffffffffu, theirs);
    before = incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0);
    if ((int)blockIdx.x >= total) {
      if (tid == 0) ends[blockIdx.x] = {-1, 0, 0, 0};
      return;
    }
    const Shares shares(total, gridDim.x);
    s0 = shares.first(blockIdx.x);
    tiles = min(shares.first(blockIdx.x + 1), total) - s0;
    start_s[0] = total;  // the same by all
  }
  __syncwarp();
  if (warp == kScoreWarp) {
    tc::tmem_alloc(smem_u32(misc), kTmemCols);
    tc::tmem_relinquish();
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = misc[0];
  const uint32_t t_p = tmem + C::COL_P, t_q = tmem + C::COL_Q, t_o = tmem + C::COL_O;
  // One thread's wait; false if it has run out, or another's in the block.
  auto wait_alone = [&](uint32_t bar, uint32_t parity) -> bool {
    return tc::mbar_try_wait(bar, parity) || wait_on<0>(bar, parity, abort_flag);
  };
  // A warp's.  Once one has run out, a warp only goes through the motions without waiting (tests of
  // that around the work on TMEM cost 200 moves a tile), so that none is left waiting for it; what
  // comes of it does not count.  The same in all lanes.
  bool dead = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xffffffffu, wait_alone(bar, parity));
  };
  auto wait_ahead = [&](uint32_t bar, uint32_t parity) {
    if (!dead)
      dead = !__all_sync(0xffffffffu, tc::mbar_try_wait(bar, parity) || wait_on<100>(bar, parity, abort_flag));
  };

  if (warp < kCopyWarps) {
    // ============================================================ copies of K and V
    give_registers<kCopyRegs>();
    Copies<D, kOnce> copies{a, warp, lane, read_once_policy()};
    // A stage is announced by its copies as they land; the issuer of the products makes them visible
    // to the tensor core.  V of a tile with drafted rows is searched first, when the next tile's
    // copies are on their way.
    int held = -1, held_unit = 0, held_lo = 0, held_hi = 0;  // such a tile
    auto release = [&] {
      const int s = held % kStages;
      if (copies.clean(smem + C::OFF_V + s * C::TILE, held_lo, held_hi))
        dirty_s[held_unit % kDirty] = held_unit + 1;
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar_vfull(s));
      held = -1;
    };
#pragma unroll 1
    for (int i = 0; i < tiles && !dead; ++i) {
      wait(bar_ids(i % kAhead), (uint32_t)(i / kAhead) & 1u);
      if (dead) break;
      const TileAt at = at_s[i % kAhead];
      const int* ids = ids_s[i % kAhead];
      copies.resolve(at, ids);
      const uint32_t there = copies.there;
      const int k0 = at.key0 + warp * 32;
      const int lo = max(0, min(32, at.first - k0)), hi = at.m > 1 ? max(0, min(32, at.paged - k0)) : 0;
      const bool boxes = a.box_rows && !~(there & ~copies.ringed);
      const int s = i % kStages;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t full = kv ? bar_vfull(s) : bar_kfull(s), to = (kv ? sV : sK) + s * C::TILE;
        wait_ahead(kv ? bar_vempty(s) : bar_kempty(s), (uint32_t)(i / kStages & 1) ^ 1u);
        if (dead) break;
        const bool search = kv && lo < hi;
        if (!kv && lane == 0) live_s[i % kLive][warp] = there;
        if (boxes && !search) {
          if (lane == 0) tc::mbar_expect_tx(full, 32 * D * 2);
          __syncwarp();
          copies.copy_boxes(at, ids, kv ? &map_v : &map_k, to, full);
        } else {
          copies.copy_rows(kv, kv ? a.v_pages : a.k_pages, kv ? a.ring_v : a.ring_k, to);
          __syncwarp();
          if (!search) {
            if (kv) tc::fence_proxy_async_smem();  // of the zeros
            wait_for_copies(full);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(full);
          }
        }
        cp_async_commit();
        if (held >= 0) {  // the copies that came after it may still be on their way
          cp_async_wait<1>();
          release();
        }
        if (search) {
          held = i;
          held_unit = at.unit;
          held_lo = lo;
          held_hi = hi;
        }
      }
      if (lane == 0 && !dead) tc::mbar_arrive(bar_idsfree(i % kAhead));
    }
    cp_async_wait<0>();
    if (held >= 0 && !dead) release();
    if (dead) {  // boxes on their way land within microseconds, before the block may leave
      const uint64_t t0 = tc::globaltimer();
      while (tc::globaltimer() - t0 < 1000000) {}
    }
  } else if (warp >= kScoreWarp) {
    // ============================================================ products, page ids
    give_registers<kMmaRegs>();
    if (warp == kScoreWarp) {
      // S = Q K^T of a tile into S buffer tile & 1; one lane issues and waits
      constexpr uint32_t idesc = tc::idesc_bf16(BM, BN);
      int i = 0;
      bool ok = lane == 0;
      for (int n = 0; ok && (ok = wait_alone(bar_unit(n), (uint32_t)(n / kUnits) & 1u)); ++n) {
        const int end = i + unit_s[n % kUnits].tb - unit_s[n % kUnits].ta;
        tc::mbar_arrive(bar_unitfree(n));
        if (end == i || !wait_alone(bar_q, (uint32_t)n & 1u)) break;  // the query rows are in TMEM
#pragma unroll 1
        for (; i < end; ++i) {
          const int s = i % kStages, buf = i & 1;
          ok = wait_alone(bar_kfull(s), (uint32_t)(i / kStages) & 1u) &&
               wait_alone(bar_sempty(buf), ((uint32_t)(i >> 1) & 1u) ^ 1u);
          if (!ok) break;
          tc::fence_after_sync();
          tc::fence_proxy_async_smem();
          const uint64_t k_s = tc::sdesc_sw128(sK + s * C::TILE);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_bf16_ts(tmem + (uint32_t)(buf * BN), t_q + 8u * k,
                            k_s + (((uint32_t)(k >> 2) * kBox + (uint32_t)(k & 3) * 32u) >> 4),
                            idesc, k > 0 ? 1u : 0u);
          tc::commit(bar_sfull(buf));
          tc::commit(bar_kempty(s));
        }
      }
      __syncwarp();
    } else if (warp == kValueWarp) {
      // O += P V of a tile
      constexpr uint32_t idesc = tc::idesc_bf16_bmn(BM, D);
      int i = 0;
      bool ok = lane == 0;
      for (int n = 0; ok && (ok = wait_alone(bar_unit(n), (uint32_t)(n / kUnits) & 1u)); ++n) {
        const int first = i, end = i + unit_s[n % kUnits].tb - unit_s[n % kUnits].ta;
        tc::mbar_arrive(bar_unitfree(n));
        if (end == i) break;
#pragma unroll 1
        for (; i < end; ++i) {
          // the first P of a unit comes after the previous unit's O was read
          const int s = i % kStages;
          ok = wait_alone(bar_vfull(s), (uint32_t)(i / kStages) & 1u) &&
               wait_alone(bar_p(i), (uint32_t)(i >> 1) & 1u);
          if (!ok) break;
          tc::fence_after_sync();
          tc::fence_proxy_async_smem();
          const uint64_t v_s = tc::sdesc_sw128_mn(sV + s * C::TILE, kBox);
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            tc::mma_bf16_ts(t_o, t_p + 8u * k, v_s + (uint32_t)(2048 * k >> 4), idesc,
                            (i > first || k > 0) ? 1u : 0u);
          tc::commit(bar_vempty(s));
          tc::commit(bar_o(i));
        }
      }
      __syncwarp();
    } else if (warp == kFindWarp) {
      // the units, and the page ids of their tiles' keys: these are asked for tile by tile and
      // announced when they have come
      Walk walk;
      walk.u = unit_s[0];
      walk.base = walk.u.row | 31;  // its row is not among the lanes'
      walk.base -= 31;
      walk.left = tiles - (walk.u.tb - walk.u.ta);
      walk.mine = {0, 0, 0, 0};
      if (walk.base + lane < rows) walk.mine = row_of(a, walk.base + lane);
      __syncwarp();
      auto announce = [&](int c) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar_ids(c % kAhead));
      };
      // units are published one ahead of their tiles' page ids: the softmax asks for the next one when
      // it begins one
      auto publish = [&](int n, bool some) {
        wait_ahead(bar_unitfree(n), ((uint32_t)(n / kUnits) & 1u) ^ 1u);
        if (lane == 0 && !dead) {
          unit_s[n % kUnits] = walk.u;
          if (!some) unit_s[n % kUnits].ta = unit_s[n % kUnits].tb;
          tc::mbar_arrive(bar_unit(n));
        }
        __syncwarp();
      };
      int i = 0, n = 0;
      publish(0, true);
#pragma unroll 1
      for (bool more = true; more && !dead; ++n) {
        const Unit u = walk.u;
        more = walk.next(a, rows, g, lane);
        publish(n + 1, more);
        const int* table = a.block_table + (size_t)u.row * a.max_pages;
#pragma unroll 1
        for (int t = u.ta; t < u.tb; ++t, ++i) {
          const int s = i % kAhead;
          wait_ahead(bar_idsfree(s), ((uint32_t)(i / kAhead) & 1u) ^ 1u);
          if (dead) break;
#pragma unroll
          for (int c = lane; c < BN; c += 32) {
            const int key = t * BN + c;
            if (key < u.is.paged) cp_async4(smem_u32(&ids_s[s][c]), table + a.by_page.of(key));
          }
          cp_async_commit();
          if (lane == 0) at_s[s] = {u.row, t * BN, u.is.paged, u.is.all, u.is.first(), u.is.m, n, 0};
          cp_async_wait<kAhead - 2>();
          if (opaque(i) >= kAhead - 2) announce(i - (kAhead - 2));
        }
      }
      cp_async_wait<0>();
      if (!dead)
        for (int c = max(0, i - (kAhead - 2)); c < i; ++c) announce(c);
      __syncwarp();
    }
  } else {
    // ============================================================ softmax + epilogue
    take_registers<kSoftRegs>();
    constexpr int OC = D / 2;   // O columns of this thread in the rescale / epilogue
    constexpr int QW = D / 4;   // 32-bit words (bf16 pairs) of the query row per thread
    const int st = tid - kSoftWarp * 32;     // softmax thread
    const int h = (warp - kSoftWarp) >> 2;   // key half of each tile (and of O's columns)
    const int eq = warp & 3;                 // TMEM lane quarter
    const int row = eq * 32 + lane;          // query row within the tile
    const uint32_t lane_off = (uint32_t)(eq * 32) << 16;
    const float sc2 = rsqrtf((float)D) * kLog2e;
    uint32_t qv[QW];
    int my_up = -1;       // parent of drafted token st (or lane)
    // this thread's part of a unit's query row (zeros past the last), and its token's parent
    auto load_q = [&](const Unit& u) {
      const int x = u.mt * BM + row;
      if (x < u.is.m * g) {
        const int i = a.by_group.of(x), hd = x - i * g, l_hk = a.by_batch.of(u.row);
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (((size_t)l_hk * g + hd) * a.N + u.is.t0 + i) * D + h * OC);
#pragma unroll
        for (int c = 0; c < QW / 4; ++c) {
          const uint4 y = src[c];
          qv[4 * c] = y.x;
          qv[4 * c + 1] = y.y;
          qv[4 * c + 2] = y.z;
          qv[4 * c + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int c = 0; c < QW; ++c) qv[c] = 0u;
      }
      // with up to 32 tokens every warp has them all
      const int token = u.is.m <= 32 ? lane : st;
      if (a.parent && token < u.is.m) my_up = a.parent[u.is.t0 + token];
    };
    auto store_q = [&] {
      __syncwarp();
      if (dead) return;
      if constexpr (QW == 32) tc::tmem_st32(t_q + lane_off + (uint32_t)(h * QW), qv);
      else tc::tmem_st16(t_q + lane_off + (uint32_t)(h * QW), qv);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      tc::mbar_arrive(bar_q);
    };
    // Unit n; where a wait has run out in any warp all of them stop here, none in the same way.
    auto fetch = [&](int n) -> Unit {
      wait(bar_unit(n), (uint32_t)(n / kUnits) & 1u);
      Unit u = unit_s[n % kUnits];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar_unitfree(n));
      __syncwarp();
      if (tc::bar_or(2, kSoftThreads, dead)) u.ta = u.tb;
      return u;
    };
    Unit u = fetch(0);
    if (!u.none()) {
      load_q(u);
      store_q();
    }
    int gs = 0;  // tiles processed (all units): S buffer, exchange buffer, P and O barriers
    int sees_of = -1;  // sequence whose tree is in `sees`
    for (int n = 0; !u.none(); ++n) {
      const int x = u.mt * BM + row, live = u.is.m * g - u.mt * BM;  // query rows of the unit
      const int i = a.by_group.of(x), hd = x - i * g, first = u.is.first();
      const bool mine_live = row < live, warp_live = eq * 32 < live;
      // --- which drafted tokens each one sees, if the segment has drafted keys
      const int b = u.row - a.by_batch.of(u.row) * a.B;
      // the next unit's query rows are asked for early: under a saturated HBM they take longer than a
      // tile
      const int up_now = my_up;
      const Unit next = fetch(n + 1);
      if (!next.none()) load_q(next);
      uint32_t mine_sees = 0;  // of up to 32 tokens
      if (a.parent && u.is.m > 1 && u.tb * BN > first) {
        if (u.is.m <= 32) {  // every warp for itself, a lane a token
          int p = lane < u.is.m ? up_now : -1;
          if (p < -1 || p >= lane) {
            fault();
            p = -1;
          }
          uint32_t bits = 1u << lane;
          // each round doubles the way up that a token has; p is the token above that
          while (__any_sync(0xffffffffu, p >= 0)) {
            const uint32_t theirs = __shfl_sync(0xffffffffu, bits, p & 31);
            const int above = __shfl_sync(0xffffffffu, p, p & 31);
            if (p >= 0) {
              bits |= theirs;
              p = above;
            }
          }
          mine_sees = __shfl_sync(0xffffffffu, bits, i & 31);
        } else if (sees_of != b) {
          sees_of = b;
          uint32_t bits[kWords];
          int p = -1;
          if (st < u.is.m) {
            p = up_now;
            if (p < -1 || p >= st) {
              fault();
              p = -1;
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w) bits[w] = w == st >> 5 ? 1u << (st & 31) : 0u;
          }
          bool more = true;
#pragma unroll 1
          for (int round = 0; more && round < 9; ++round) {
            named_sync(1, kSoftThreads);  // all have read the row of the round (or unit) before
            if (st < u.is.m) {
#pragma unroll
              for (int w = 0; w < kWords; ++w) sees[st * kWords + w] = bits[w];
              up[st] = p;
            }
            __syncwarp();
            more = tc::bar_or(2, kSoftThreads, p >= 0);
            if (p >= 0) {
#pragma unroll
              for (int w = 0; w < kWords; ++w) bits[w] |= sees[p * kWords + w];
              p = up[p];
            }
          }
        }
      }
      float m_used = -CUDART_INF_F, lsum = 0.f;
#pragma unroll 1
      for (int j = u.ta; j < u.tb; ++j, ++gs) {
        const int s = gs & 1;  // max-exchange buffer and S buffer
        wait(bar_sfull(s), (uint32_t)(gs >> 1) & 1u);
        tc::fence_after_sync();
        if (!warp_live) {
          tc::mbar_arrive(bar_sempty(s));
          if (j > u.ta) wait(bar_o(gs - 1), (uint32_t)((gs - 1) >> 1) & 1u);
          tc::mbar_arrive(bar_p(gs));
          continue;
        }
        uint32_t v[KC];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < KC; c += 32)
          tc::tmem_ld32(tmem + lane_off + (uint32_t)(s * BN + h * KC + c), v + c);
        // while they come: of the thread's 64 keys those there are, without drafted ones not seen
        uint64_t vis = (uint64_t)live_s[gs % kLive][2 * h + 1] << 32 | live_s[gs % kLive][2 * h];
        const int kb = j * BN + h * KC;
        if (kb + KC > first && kb < u.is.paged) {
          const uint64_t drafts = low_bits(u.is.paged - kb) & ~low_bits(first - kb);
          const uint64_t seen = !a.parent || u.is.m == 1 ? low_bits(first + i + 1 - kb)
                                : u.is.m <= 32 ? bits_of(mine_sees, kb - first)
                                : mine_live ? bits_from(sees + i * kWords, kb - first) : 0ull;
          vis &= ~drafts | seen;
        }
        const bool masked = __any_sync(0xffffffffu, ~vis != 0);
        tc::tmem_ld_wait();
        tc::fence_before_sync();
        tc::mbar_arrive(bar_sempty(s));  // the next S into this buffer may start now
        if (masked) {
          asm volatile("");  // a branch: most tiles have nothing to mask
          const uint32_t lo = (uint32_t)vis, hi = (uint32_t)(vis >> 32);
#pragma unroll
          for (int c = 0; c < KC; ++c)
            if (!((c < 32 ? lo : hi) >> (c & 31) & 1u)) v[c] = __float_as_uint(-CUDART_INF_F);
        }
        float mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F, mx2 = -CUDART_INF_F, mx3 = -CUDART_INF_F;
#pragma unroll
        for (int c = 0; c < KC; c += 8) {
          mx0 = tc::max3(mx0, __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
          mx1 = tc::max3(mx1, __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
          mx2 = tc::max3(mx2, __uint_as_float(v[c + 4]), __uint_as_float(v[c + 5]));
          mx3 = tc::max3(mx3, __uint_as_float(v[c + 6]), __uint_as_float(v[c + 7]));
        }
        float top = tc::max3(mx0, mx1, fmaxf(mx2, mx3)) * sc2;
        // the two threads of a row are warps eq + 4 and eq + 8: a named barrier per lane quarter
        float* xmj = xm + s * 2 * BM;
        xmj[h * BM + row] = top;
        named_sync(3 + eq, 64);
        top = fmaxf(top, xmj[(h ^ 1) * BM + row]);
        const bool need = top > m_used + kRescale;
        float factor = 1.f;
        if (need) {
          factor = fast_exp2(m_used - top);  // 0 for the first keys
          m_used = top;
          lsum *= factor;
        }
        // p = 2^(x sc2 - m) with packed fp32 pairs; each weight is rounded to bf16 once for P V, as
        // the output is, and enters the sum as it was.  Beside o's own rounding (1.7e-3 in the
        // 2-norm) that shows over long rows, 1.9e-3 to 2.2e-3 together.  A second bf16 part of what
        // the first leaves, as in the attention of one new token, brings 1.7e-3 back; measured
        // with P in the place of S: wide trees 302 for 247 us, 64 sequences 64 for 52, 96 of 16384
        // tokens 412 for 372, the document 67 for 59.  In wide trees nearly all of it is the second
        // part's arithmetic, which falls into the chain of a tile, at d = 128 half its product.
        uint32_t pk[KC / 2];
        const float2 k2 = make_float2(sc2, sc2), nm = make_float2(-finite_ref(m_used), -finite_ref(m_used));
        float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
        for (int c = 0; c < KC; c += 4) {
          const float2 y0 = __ffma2_rn(tc::f2(v[c], v[c + 1]), k2, nm);
          const float2 y1 = __ffma2_rn(tc::f2(v[c + 2], v[c + 3]), k2, nm);
          const float p0 = fast_exp2(y0.x), p1 = fast_exp2(y0.y);
          const float p2 = fast_exp2(y1.x), p3 = fast_exp2(y1.y);
          a0 = __fadd2_rn(a0, make_float2(p0, p1));
          a1 = __fadd2_rn(a1, make_float2(p2, p3));
          pk[c / 2] = pack2(p0, p1);
          pk[c / 2 + 1] = pack2(p2, p3);
        }
        a0 = __fadd2_rn(a0, a1);
        lsum += a0.x + a0.y;

        // P V of the previous tile has read its P (and finished O) before P is written; O is
        // rescaled only when a row's max grew past the threshold.  The unit's first tile needs
        // no wait: the previous unit's last P V was waited for below.
        const bool any_need = __any_sync(0xffffffffu, need);
        if (j > u.ta) {
          wait(bar_o(gs - 1), (uint32_t)((gs - 1) >> 1) & 1u);
          tc::fence_after_sync();
          __syncwarp();
          if (any_need) {
            const uint32_t to = t_o + lane_off + (uint32_t)(h * OC);
#pragma unroll 1
            for (int cb = 0; cb < OC; cb += 32) {
              tc::tmem_ld32(to + cb, v);
              tc::tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * factor);
              tc::tmem_st32(to + cb, v);
            }
            tc::tmem_st_wait();
          }
        }
        __syncwarp();
        tc::tmem_st32(t_p + lane_off + (uint32_t)(h * (KC / 2)), pk);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        tc::mbar_arrive(bar_p(gs));
      }
      // the next unit's query rows take the place of this unit's, whose S products are complete, so
      // that its first ones run while this unit's O is finished and written
      if (!next.none()) store_q();
      // the last two P V products of the unit (on o[0] and o[1]) complete O
      if (u.tb - u.ta > 1) wait(bar_o(gs - 2), (uint32_t)((gs - 2) >> 1) & 1u);
      wait(bar_o(gs - 1), (uint32_t)((gs - 1) >> 1) & 1u);
      tc::fence_after_sync();
      if (warp_live) {
        xl[h * BM + row] = lsum;
        named_sync(3 + eq, 64);
        lsum += xl[(h ^ 1) * BM + row];
        const bool dirty = dirty_s[n % kDirty] == n + 1;
        const float inv = inverse(lsum);
        const size_t out = ((size_t)a.by_batch.of(u.row) * g + hd) * a.N + u.is.t0 + i;
        float* part = block_part(a.ws, blockIdx.x, u.ta > 0 ? 0 : 1, part_floats(D));
#pragma unroll 1
        for (int cb = 0; cb < OC; cb += 32) {
          uint32_t v[32];
          __syncwarp();
          tc::tmem_ld32(t_o + lane_off + (uint32_t)(h * OC + cb), v);
          tc::tmem_ld_wait();
          if (dirty && mine_live) {
            // drafted values that are not finite were zeros above: rows that see them get them
            const int k0 = max(0, u.ta * BN - first), k1 = min(u.is.m, u.tb * BN - first);
#pragma unroll 1
            for (int k = k0; k < k1; ++k) {
              const int slot = first + k;
              const bool seen = !a.parent ? k <= i : u.is.m <= 32 ? mine_sees >> k & 1
                                                    : sees[i * kWords + (k >> 5)] >> (k & 31) & 1;
              if (!seen || slot < 0) continue;
              const int idx = a.by_page.of(slot);
              const int page = a.block_table[(size_t)u.row * a.max_pages + idx];
              if ((uint32_t)page >= (uint32_t)a.capacity) continue;
              const bf16_t* src =
                  a.v_pages + ((size_t)page * a.page_size + slot - idx * a.page_size) * D + h * OC + cb;
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const uint32_t y = *reinterpret_cast<const uint32_t*>(src + c);
                if (not_finite(y)) v[c] = __float_as_uint(__uint_as_float(v[c]) + bf16_lo(y));
                if (not_finite(y >> 16))
                  v[c + 1] = __float_as_uint(__uint_as_float(v[c + 1]) + bf16_hi(y));
              }
            }
          }
          if (!mine_live) continue;
          if (u.whole()) {
            uint4* dst = reinterpret_cast<uint4*>(a.o + out * D + h * OC + cb);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = pack2(__uint_as_float(v[8 * c + 2 * e]) * inv,
                             __uint_as_float(v[8 * c + 2 * e + 1]) * inv);
              dst[c] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(part) + (h * OC + cb) / 4 * BM + row;
#pragma unroll
            for (int c = 0; c < 8; ++c)
              dst[c * BM] = make_float4(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]),
                                        __uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3]));
          }
        }
        if (mine_live && h == 0 && !dead) {
          if (!u.whole()) {
            part[BM * D + row] = m_used;
            part[BM * D + BM + row] = lsum;
          } else if (a.lse) {
            a.lse[out] = lse_of(m_used, lsum);
          }
        }
      }
      u = next;
    }
  }

  // every product issued so far has completed once these commits land
  if ((warp == kScoreWarp || warp == kValueWarp) && lane == 0) {
    tc::commit(bar_done);
    tc::mbar_wait(bar_done, 0);
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) atomicCAS(&g_attn_tree_error, 0, kErrWaitTimeout);
  if (warp == kScoreWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Pairs that cross blocks: block x joins the pair that ends in block x of the first kernel, from
// the part of its first block and those after.  A thread takes eight columns of a query row.
// While the first kernel runs: zeros for tokens that no key is there for.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_tree_join_kernel(
    const __grid_constant__ AttnTreeArgs a, int rows) {
  const int g = a.Hq / a.Hkv;
  const int every = gridDim.x * gridDim.y * (kJoinThreads / 32), lane = threadIdx.x & 31;
  for (int r = (blockIdx.y * gridDim.x + blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
       r < rows; r += every) {
    const Row x = row_of(a, r);
    if (x.all > 0) continue;
    for (int i = lane; i < x.m * g; i += 32) {
      const int tok = a.by_group.of(i);
      const size_t out = ((size_t)a.by_batch.of(r) * g + i - tok * g) * a.N + x.t0 + tok;
      for (int e = 0; e < D / 8; ++e)
        reinterpret_cast<uint4*>(a.o + out * D)[e] = make_uint4(0, 0, 0, 0);
      if (a.lse) a.lse[out] = -INFINITY;
    }
  }
  wait_for_previous();
  const Ends end = static_cast<const Ends*>(a.ws)[blockIdx.x];
  // the bounds hold even if another stream writes the workspace meanwhile
  if ((uint32_t)end.row >= (uint32_t)rows || (uint32_t)end.first >= blockIdx.x || end.mt < 0) return;
  const Row is = row_of(a, end.row);
  const int item = blockIdx.y * kJoinThreads + threadIdx.x, row = item % BM, c8 = item / BM;
  const long long x = (long long)end.mt * BM + row;
  if (x >= (long long)is.m * g) return;
  const int n = blockIdx.x - end.first + 1;
  constexpr int kAhead = 4;
  float top = -INFINITY, sum = 0.f, acc[8] = {};
  for (int p0 = 0; p0 < n; p0 += kAhead) {
    float ref[kAhead], l[kAhead];
    float4 y[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int p = min(p0 + i, n - 1);
      const float* part = block_part(a.ws, end.first + p, p == 0 ? 1 : 0, part_floats(D));
      y[i][0] = reinterpret_cast<const float4*>(part)[2 * c8 * BM + row];
      y[i][1] = reinterpret_cast<const float4*>(part)[(2 * c8 + 1) * BM + row];
      ref[i] = part[BM * D + row];
      l[i] = part[BM * D + BM + row];
    }
    float high = top;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) high = fmaxf(high, ref[i]);
    const float base = finite_ref(high), w = fast_exp2(top - base);
    sum *= w;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= w;
    top = high;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (p0 + i >= n) break;
      const float v = fast_exp2(ref[i] - base);
      sum += l[i] * v;
      acc[0] += y[i][0].x * v;
      acc[1] += y[i][0].y * v;
      acc[2] += y[i][0].z * v;
      acc[3] += y[i][0].w * v;
      acc[4] += y[i][1].x * v;
      acc[5] += y[i][1].y * v;
      acc[6] += y[i][1].z * v;
      acc[7] += y[i][1].w * v;
    }
  }
  const int i = a.by_group.of((int)x), hd = (int)x - i * g;
  const size_t out = ((size_t)a.by_batch.of(end.row) * g + hd) * a.N + is.t0 + i;
  const float inv = inverse(sum);
  reinterpret_cast<uint4*>(a.o + out * D)[c8] =
      make_uint4(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv),
                 pack2(acc[4] * inv, acc[5] * inv), pack2(acc[6] * inv, acc[7] * inv));
  if (a.lse && c8 == 0) a.lse[out] = lse_of(top, sum);
}

template <int D>
cudaError_t launch(AttnTreeArgs a, int rows, cudaStream_t s) {
  using C = Cfg<D>;
  static int nsm[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!nsm[dev]) {
    e = cudaDeviceGetAttribute(&nsm[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
  }
  a.by_batch = Divisor(a.B);
  a.by_page = Divisor(a.page_size);
  a.by_group = Divisor(a.Hq / a.Hkv);
  // pages of 8, 16 or 32 rows, or of several times 32, come by TMA
  a.box_rows = a.page_size % 32 == 0 ? 32 : a.page_size == 8 || a.page_size == 16 ? a.page_size : 0;
  if (a.capacity == 0) a.box_rows = 0;
  const long long row_tiles = ((long long)a.max_pages * a.page_size + a.w + BN - 1) / BN;
  const long long query = ((long long)a.max_draft * (a.Hq / a.Hkv) + BM - 1) / BM;
  const bool read_once = query == 1 && (long long)rows * row_tiles * 2 * C::TILE > kL2Bytes / 2;
  const int sms = std::min(nsm[dev], kMaxBlocks);
  // no more blocks than tiles could need
  const int blocks = (int)std::min<long long>(sms, (long long)rows * query * row_tiles);
  const auto kernel = read_once ? attn_tree_kernel<D, true> : attn_tree_kernel<D, false>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap map_k, map_v;
  e = tma_map_bf16_3d(&map_k, a.box_rows ? a.k_pages : a.q, D, a.box_rows ? a.page_size : 1,
                      a.box_rows ? a.capacity : 1, a.box_rows ? a.box_rows : 8);
  if (e == cudaSuccess)
    e = tma_map_bf16_3d(&map_v, a.box_rows ? a.v_pages : a.q, D, a.box_rows ? a.page_size : 1,
                        a.box_rows ? a.capacity : 1, a.box_rows ? a.box_rows : 8);
  if (e != cudaSuccess) return e;
  count_launches(2);
  Launch first(dim3(blocks), kThreads, s);
  first.cfg.dynamicSmemBytes = C::SMEM;
  e = cudaLaunchKernelEx(&first.cfg, kernel, a, map_k, map_v, rows);
  if (e != cudaSuccess) return e;
  Launch join(dim3(blocks, BM * (D / 8) / kJoinThreads), kJoinThreads, s);
  return cudaLaunchKernelEx(&join.cfg, attn_tree_join_kernel<D>, a, rows);
}

}  // namespace

size_t attn_tree_workspace_bytes(int d) {
  return ends_bytes() + (size_t)kMaxBlocks * 2 * part_floats(d) * sizeof(float);
}

cudaError_t launch_attn_tree(const AttnTreeArgs& a, cudaStream_t s) {
  const int rows = a.L * a.Hkv * a.B;
  if (rows == 0 || a.N == 0) return cudaSuccess;
  return a.d == 128 ? launch<128>(a, rows, s) : launch<64>(a, rows, s);
}

cudaError_t attn_tree_device_error(int* code, bool clear, cudaStream_t s) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(code, g_attn_tree_error, sizeof(int), 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && clear && *code) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_attn_tree_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

}  // namespace kvs
