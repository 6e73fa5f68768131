// Attention of one new token per sequence over its row's paged cache and window ring:
//   o = sum_i a_i v_i,  a_i = exp(q . k_i / sqrt(d) - lse),  lse = ln sum_i exp(q . k_i / sqrt(d))
// over the row's seq_lens[r] paged keys and the min(pos, w) keys of its ring, for the g
// query heads of the row's KV head.  Every key is read once for up to 16 heads (above that,
// once from HBM and from L2 for each further 16): 4 d bytes and 4 d g flops, so HBM bounds it
// (g flop/B; the tensor cores take over 200).
//
// Rows differ in length by the pruning, so the work is cut by tiles, not by rows: all rows'
// tiles of 16 keys (32 at d = 64) form one stream, every warp of a persistent grid takes an equal
// contiguous share, and a row that crosses a share's border is joined from partial sums
// (running maximum, sum and weighted values): within a block through shared memory, between
// blocks by a second kernel.  Shares depend on the lengths alone, so results do too.  Rows
// that cannot be long take a block or cluster each instead (see row_shape).
//
// A warp streams its tiles through a private ring of two cp.async stages (128-byte
// swizzle, no block barrier), across row borders: the loads of the next rows are in
// flight while a row is finished.  Ten warps with two stages reach 6.8 TB/s (96 sequences of
// 16384 tokens, heads kept at 25 to 75 %: 361 us for 2.47 GB, 152 blocks); eight warps with
// three stages take 377 us: more bytes in flight only lengthen every other load.  Short of
// that, about 8 us of a call is latency (scan of the lengths, table, first tile, joins).
// Per tile (mma.m16n8k16, keys in M, heads in N, bf16 -> fp32):
//   S^T = K Q^T       A = K rows by ldmatrix, B = Q in registers
//   P^T = exp2(S^T)   in registers, in two bf16 parts, turned into B operands by movmatrix
//   O^T += V^T P^T    A = V by ldmatrix.trans
// With keys in M a group of 8 query heads fills N exactly; tcgen05 (M = 128) would spend
// its rows on 4 to 8 heads and a TMEM round trip per tile, on a contraction that needs a
// fiftieth of its rate.  The softmax reference is raised only when a tile exceeds it by 2^8
// (one vote per tile instead of a cross-lane maximum); weights stay below 2^8, are summed in
// fp32 and multiply V as two bf16 parts, 2^-15 of a weight together.  One part alone (2^-8)
// shows in o beside its own rounding: 2.0e-3 against 1.7e-3 in the 2-norm.  The second takes
// 33.2 against 32.9 us (64 rings), 361.6 against 360.3 (96 x 16384 tokens), 9.7 against 9.4
// (33 sequences of pages of 13).
#include "attn_decode.cuh"
#include "common.cuh"

namespace kvs {

__device__ int g_attn_decode_error = 0;

namespace {

constexpr int kErrAttnDecode = 9;  // a length or page id out of range

// Keys of a tile: 8 KB of K and V.  Half of that at d = 64 left the arithmetic's latency in
// the way (96 x 16384 tokens: 72 % of the DRAM's rate).
__host__ __device__ constexpr int tile_keys(int d) { return d == 128 ? 16 : 32; }
constexpr int kMaxBlocks = 160;  // of the persistent grid; sizes the workspace
constexpr int kMaxWarps = 16;    // of a block
constexpr long long kL2Bytes = 129ll << 20;
constexpr int kMaxCluster = 8;   // blocks that share a row
constexpr int kJoinThreads = 256;
constexpr int kMaxChunks = 256;  // of rows, in the scan of their tiles
constexpr int kCachedRows = 512; // whose lengths a block keeps in shared memory
constexpr float kSlack = 8.f;    // log2 of how far a weight may exceed the reference

constexpr int kStages = 2;
constexpr int kStageBytes = 2 * tile_keys(128) * 128 * 2;  // either d
constexpr int kRingBytes = kStages * kStageBytes;          // per warp

// A partial result of a row segment: O^T fragments [d / 16 * 4 * NG][32 lanes], then (in
// the workspace) the reference and the sum of each of the 8 NG heads.
__host__ __device__ constexpr int frags(int d, int ng) { return d / 16 * 4 * ng; }
__host__ __device__ constexpr int part_floats(int d, int ng) { return frags(d, ng) * 32 + 16 * ng; }

// Warps of a block: as many as the rings and a partial result each fit beside, or the
// registers allow (d = 128, NG = 2).
__host__ __device__ constexpr int warps_of(int d, int ng) {
  return d == 64 ? (ng == 1 ? 12 : 10) : ng == 1 ? 10 : 8;
}
__host__ __device__ constexpr int warp_bytes(int d, int ng) {
  return kRingBytes + frags(d, ng) * 32 * 4;
}

// Workspace: per block the row that ends there having begun in another block (or -1) and
// that other block; per block the parts of the rows that cross its borders (0: began
// before, 1: goes on after).
struct Ends { int vrow, first; };
__host__ __device__ constexpr size_t ends_bytes() { return kMaxBlocks * sizeof(Ends); }
__device__ __forceinline__ float* block_part(void* ws, int block, int side, int pf) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + ends_bytes()) +
         (size_t)(2 * block + side) * pf;
}

// 16-byte async copy global -> shared under an L2 policy (src_bytes = 0 writes zeros without
// reading).  A call that may read more than half of L2 marks keys and values as the first to
// leave it: they are not read again before the next step, and what is (lengths, tables,
// queries, a part of the keys of a loop over layers) stays.  131072-token document 33.8 ->
// 31.3 us, 64 rings 35.5 -> 33.2; 27 MB that stay in L2 from call to call would take 11.2
// instead of 10.3.
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async16_once(uint32_t dst, const void* src, int src_bytes,
                                                uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n" ::"r"(dst),
               "l"(src), "r"(src_bytes), "l"(policy));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A weight in two bf16 parts: its first eight bits, and what they leave.  The second part is
// taken of p (1 + 2^-20), so that it is not 0 beside a weight (above 2^-112): an infinite value
// then gives infinity with both parts, and not NaN with one.
__device__ __forceinline__ uint32_t high2(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float low(float p) {
  return fmaf(p, 1.f + 0x1p-20f, -__uint_as_float(__float_as_uint(p) & 0xffff0000u));
}

__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }

// The keys of a row: paged tokens, and with the ring's.
struct Keys { int paged, all; };

__device__ __forceinline__ Keys keys_of(const AttnDecodeArgs& a, int len, int pos) {
  const int n = max(0, min(len, a.max_pages * a.page_size));
  return {n, n + max(0, min(pos, a.w))};
}

__device__ __forceinline__ int ring_pos(const AttnDecodeArgs& a, int row) {
  return a.w > 0 ? a.pos[row % a.B] : 0;
}

// A place in the stream of tiles.  The lanes hold the lengths of the 32 rows from `base` on.
template <int kTile>
struct Cursor {
  int row, group, tile;   // group: which 8 NG of the row's query heads
  Keys keys;              // of the row
  int base;
  Keys mine;              // lane i: of row base + i

  __device__ __forceinline__ void fetch(const AttnDecodeArgs& a, int rows, const Keys* cached,
                                        int lane) {
    mine = {0, 0};
    if (base + lane < rows)
      mine = base + lane < kCachedRows ? cached[base + lane]
                                   : keys_of(a, a.seq_lens[base + lane], ring_pos(a, base + lane));
  }
  __device__ __forceinline__ void enter(int r) {
    row = r;
    keys.paged = __shfl_sync(0xffffffffu, mine.paged, r - base);
    keys.all = __shfl_sync(0xffffffffu, mine.all, r - base);
  }
  __device__ __forceinline__ bool at_row_end() const { return (tile + 1) * kTile >= keys.all; }
  // the next tile (there is one); true if it is another row's
  __device__ __forceinline__ bool advance(const AttnDecodeArgs& a, int rows, int groups,
                                          const Keys* cached, int lane) {
    if (!at_row_end()) { ++tile; return false; }
    tile = 0;
    if (++group < groups) return true;
    group = 0;
    int from = row - base + 1;
    for (;;) {
      const uint32_t some = __ballot_sync(0xffffffffu, mine.all > 0) &
                            (from < 32 ? 0xffffffffu << from : 0u);
      if (some) { enter(base + __ffs(some) - 1); return true; }
      base += 32;
      from = 0;
      if (base >= rows) return true;  // not reached while tiles remain
      fetch(a, rows, cached, lane);
    }
  }
};

// The equal contiguous shares of `warps` warps of a stream of tiles; the first `more` have one
// more than `each`.
struct Shares {
  long long each = 1, more = 0;
  __device__ __forceinline__ Shares(long long total, int warps) {
    if (total > warps) {
      each = total <= UINT32_MAX ? (uint32_t)total / (uint32_t)warps : total / warps;
      more = total - each * warps;
    }
  }
  __device__ __forceinline__ long long first(int warp) const {  // tile of a warp
    return warp * each + min((long long)warp, more);
  }
  __device__ __forceinline__ long long of(long long tile) const {  // warp of a tile
    const long long wide = more * (each + 1);
    return tile < wide ? tile / (each + 1) : more + (tile - wide) / each;
  }
};

// Output rows of the 8 NG heads of a group: element offset of head h's row.
__device__ __forceinline__ size_t out_row(const AttnDecodeArgs& a, int row, int g, int head) {
  return ((size_t)(row / a.B) * g + head) * a.B + row % a.B;
}

// Two fragments rows (dims dim .. dim + 15 of eight heads, in the layout of an accumulator)
// to the outputs: a lane gets pairs of dimensions of head lane / 4.
__device__ __forceinline__ void store_frag(bf16_t* out, const float* o, const float* inv,
                                           bool mine) {
  const uint32_t y0 = transpose8x8(pack2(o[0] * inv[0], o[1] * inv[1]));
  const uint32_t y1 = transpose8x8(pack2(o[2] * inv[0], o[3] * inv[1]));
  if (mine) {
    *reinterpret_cast<uint32_t*>(out) = y0;
    *reinterpret_cast<uint32_t*>(out + 8) = y1;
  }
}

__device__ __forceinline__ float inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float lse_of(float ref, float sum) {
  return sum == 0.f ? -INFINITY : kLn2 * (ref + log2f(sum));
}

template <int D>
__device__ __forceinline__ void store_out(const AttnDecodeArgs& a, size_t r, int dim, float acc,
                                          float top, float sum) {
  a.o[r * D + dim] = (bf16_t)(pack2(acc * inverse(sum), 0.f) & 0xffffu);
  if (a.lse && dim == 0) a.lse[r] = lse_of(top, sum);
}

// Eight fragments (32 dimensions of eight heads) from f0 on, summed up: to the outputs.
template <int D, int NG>
__device__ __forceinline__ void store_unit(const AttnDecodeArgs& a, int row, int group, int g,
                                           int f0, const float* acc, const float* top,
                                           const float* sum, int lane) {
  constexpr int KS = D / 16;
  const float inv[2] = {inverse(sum[0]), inverse(sum[1])};
  const int h0 = (group * NG + f0 / (KS * 4)) * 8;
  if (a.lse && lane < 4 && f0 % (KS * 4) == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (h0 + lane * 2 + i < g) a.lse[out_row(a, row, g, h0 + lane * 2 + i)] = lse_of(top[i], sum[i]);
  }
  const int head = h0 + (lane >> 2);
  bf16_t* out = a.o + out_row(a, row, g, head) * D + f0 / 4 % KS * 16 + (lane & 3) * 2;
  store_frag(out, acc, inv, head < g);
  store_frag(out + 16, acc + 4, inv, head < g);
}

// The copies of a warp: finds where the keys of a tile lie, and brings their rows of K and V
// into a stage of its ring.  Lane i has key i (mod the tile) of the tile.  The lanes keep 32
// entries of the row's block table from page tbase on; a load of more of them is used an
// iteration later.
template <int D>
struct Copies {
  static constexpr int kTile = tile_keys(D);
  const AttnDecodeArgs& a;
  const int ps_shift, lane;  // log2 of the page size, or -1
  const uint32_t ring_u;
  uint32_t* live;            // per stage: which of its keys are there
  int tbase = 0, entry = -1;
  int idx = 0, inside = 0;   // the key's page in the row, and its row in the page

  __device__ __forceinline__ void look_up(int row, int tile, const Keys& keys, bool new_row) {
    const int first = tile * kTile, key = first + lane % kTile;
    idx = ps_shift >= 0 ? key >> ps_shift : key / a.page_size;
    inside = key - idx * a.page_size;
    const int paged = min(kTile, keys.paged - first);  // keys of the tile in pages
    if (paged <= 0) return;
    const int p0 = __shfl_sync(0xffffffffu, idx, 0);
    const int p1 = __shfl_sync(0xffffffffu, idx, paged - 1);
    if (new_row || p1 > tbase + 31) {
      tbase = p0;
      const int ahead = keys.paged - 1 - p0 * a.page_size;
      const int have = ps_shift >= 0 ? ahead >> ps_shift : ahead / a.page_size;
      entry = lane <= have ? a.block_table[(size_t)row * a.max_pages + p0 + lane] : -1;
    }
  }

  __device__ __forceinline__ void copy(int row, int tile, const Keys& keys, int stage) {
    const int key0 = tile * kTile + lane % kTile;
    const int page = __shfl_sync(0xffffffffu, entry, (idx - tbase) & 31);
    long long at_row = -1;  // row in the pool, or in the ring
    const bool in_ring = key0 >= keys.paged;
    if (key0 < keys.all) {
      if (in_ring)
        at_row = (long long)row * a.w + (key0 - keys.paged);
      else if ((uint32_t)page < (uint32_t)a.capacity)
        at_row = (long long)page * a.page_size + inside;
      else
        atomicCAS(&g_attn_decode_error, 0, kErrAttnDecode);
    }
    const uint32_t here = __ballot_sync(0xffffffffu, at_row >= 0);
    const uint32_t ringed = __ballot_sync(0xffffffffu, in_ring);
    if (lane == 0) live[stage] = here;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes a row, rows a step
    const int c = lane % kLanes;
    const uint32_t dst = ring_u + stage * kStageBytes;
    const uint64_t policy = read_once_policy();
#pragma unroll
    for (int i = 0; i < kTile / kRows; ++i) {
      const int key = i * kRows + lane / kLanes;
      const long long r = __shfl_sync(0xffffffffu, at_row, key);
      const bool ok = (here >> key) & 1, rg = (ringed >> key) & 1;
      const size_t e = ok ? (size_t)r * D + c * 8 : 0;
      const bf16_t* k = rg ? a.ring_k : a.k_pages;
      const bf16_t* v = rg ? a.ring_v : a.v_pages;
      const uint32_t to = dst + key * (D * 2) + ((c ^ (key & 7)) << 4);
      if (a.read_once) {
        cp_async16_once(to, k + e, ok ? 16 : 0, policy);
        cp_async16_once(to + kTile * D * 2, v + e, ok ? 16 : 0, policy);
      } else {
        cp_async16(to, k + e, ok ? 16 : 0);
        cp_async16(to + kTile * D * 2, v + e, ok ? 16 : 0);
      }
    }
  }
};

// The softmax state of a warp for the 8 NG query heads of a group, in the layout of the
// accumulators: keys or dimensions lane / 4 (+ 8), heads 2 (lane % 4) + {0, 1} of each 8.
template <int D, int NG>
struct Heads {
  static constexpr int KS = D / 16;
  uint32_t q[NG][KS][2];
  float o[NG][KS][4], m[NG][2], l[NG][2];

  __device__ __forceinline__ void start(const AttnDecodeArgs& a, int row, int group, int g,
                                        int lane) {
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int head = (group * NG + j) * 8 + (lane >> 2);
      const bf16_t* src = a.q + out_row(a, row, g, head) * D + (lane & 3) * 2;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        q[j][s][0] = head < g ? *reinterpret_cast<const uint32_t*>(src + s * 16) : 0u;
        q[j][s][1] = head < g ? *reinterpret_cast<const uint32_t*>(src + s * 16 + 8) : 0u;
        o[j][s][0] = o[j][s][1] = o[j][s][2] = o[j][s][3] = 0.f;
      }
      m[j][0] = m[j][1] = -INFINITY;
      l[j][0] = l[j][1] = 0.f;
    }
  }

  // One tile in shared memory (K at kb, V behind it) whose keys `here` are there.
  __device__ __forceinline__ void tile(uint32_t kb, uint32_t here, int lane) {
    constexpr int kTile = tile_keys(D), M = kTile / 16;  // M rows of MMAs
    const float scale = rsqrtf((float)D) * kLog2e;
    float x[M][NG][4] = {};
    {
      const int key = ((lane >> 3) & 1) * 8 + (lane & 7);
      const uint32_t row_u = kb + key * (D * 2);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int n = 0; n < M; ++n) {
          uint32_t k[4];
          ldmatrix_x4(row_u + n * (16 * D * 2) + (((s * 2 + (lane >> 4)) ^ (key & 7)) << 4), k[0],
                      k[1], k[2], k[3]);
#pragma unroll
          for (int j = 0; j < NG; ++j) mma_bf16_16816(x[n][j], k, q[j][s][0], q[j][s][1]);
        }
      }
    }
    bool raise = false;
#pragma unroll
    for (int n = 0; n < M; ++n) {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = n * 16 + (lane >> 2) + (i >> 1) * 8;
          x[n][j][i] = (here >> key) & 1 ? x[n][j][i] * scale : -INFINITY;
          raise |= x[n][j][i] > m[j][i & 1] + kSlack;
        }
      }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = m[j][i];
#pragma unroll
          for (int n = 0; n < M; ++n) top = fmaxf(top, fmaxf(x[n][j][i], x[n][j][i + 2]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float c = fast_exp2(m[j][i] - finite_ref(top));
          m[j][i] = top;
          l[j][i] *= c;
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            o[j][s][i] *= c;
            o[j][s][i + 2] *= c;
          }
        }
      }
    }
    uint32_t hi[M][NG][2], lo[M][NG][2];
#pragma unroll
    for (int n = 0; n < M; ++n) {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = fast_exp2(x[n][j][i] - finite_ref(m[j][i & 1]));
        l[j][0] += p[0] + p[2];
        l[j][1] += p[1] + p[3];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          hi[n][j][i] = transpose8x8(high2(p[2 * i], p[2 * i + 1]));
          lo[n][j][i] = transpose8x8(pack2(low(p[2 * i]), low(p[2 * i + 1])));
        }
      }
    }
    const int key = (lane >> 4) * 8 + (lane & 7);
    const uint32_t row_u = kb + (kTile + key) * (D * 2);
#pragma unroll
    for (int n = 0; n < M; ++n) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint32_t v[4];
        ldmatrix_x4_trans(row_u + n * (16 * D * 2) +
                              (((s * 2 + ((lane >> 3) & 1)) ^ (key & 7)) << 4), v);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          mma_bf16_16816(o[j][s], v, hi[n][j][0], hi[n][j][1]);
          mma_bf16_16816(o[j][s], v, lo[n][j][0], lo[n][j][1]);
        }
      }
    }
  }

  // the sums over the lanes of a column
  __device__ __forceinline__ void fold() {
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 4);
        l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 8);
        l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 16);
      }
  }

  __device__ __forceinline__ void store(const AttnDecodeArgs& a, int row, int group, int g,
                                        int lane) const {
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      float inv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        inv[i] = inverse(l[j][i]);
        const int head = (group * NG + j) * 8 + (lane & 3) * 2 + i;
        if (a.lse && lane < 4 && head < g) a.lse[out_row(a, row, g, head)] = lse_of(m[j][i], l[j][i]);
      }
      const int head = (group * NG + j) * 8 + (lane >> 2);
      bf16_t* out = a.o + out_row(a, row, g, head) * D + (lane & 3) * 2;
#pragma unroll
      for (int s = 0; s < KS; ++s) store_frag(out + s * 16, o[j][s], inv, head < g);
    }
  }

  // a part: fragments to `to`, references and sums of the 8 NG heads
  __device__ __forceinline__ void leave(float* to, float* ref, float* sum, int lane) const {
#pragma unroll
    for (int j = 0; j < NG; ++j) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[((j * KS + s) * 4 + i) * 32 + lane] = o[j][s][i];
      if (lane < 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ref[j * 8 + lane * 2 + i] = m[j][i];
          sum[j * 8 + lane * 2 + i] = l[j][i];
        }
      }
    }
  }
};

template <int D, int NG>
__global__ void __launch_bounds__(warps_of(D, NG) * 32, 1) attn_decode_kernel(
    const __grid_constant__ AttnDecodeArgs a, int rows, int groups, int ps_shift) {
  constexpr int S = kStages, KS = D / 16, PF = part_floats(D, NG), NF = frags(D, NG);
  constexpr int kTile = tile_keys(D);
  constexpr int kWarps = warps_of(D, NG);
  static_assert(NF * 32 * 4 <= kRingBytes && kWarps <= kMaxWarps, "a partial result fits the ring");
  extern __shared__ __align__(1024) uint8_t smem[];
  Keys* cached = reinterpret_cast<Keys*>(smem + kWarps * warp_bytes(D, NG));
  __shared__ long long chunk_tiles[kMaxChunks];
  __shared__ uint32_t live[kWarps][S];
  // what each warp leaves behind: a row that began before its share (head, index w, behind
  // the ring) and one that goes on after it (tail, index kWarps + w, in the ring); the bit
  // masks say where there is one
  __shared__ int vrow_of[2 * kWarps];
  __shared__ float ref_s[2 * kWarps][NG * 8], sum_s[2 * kWarps][NG * 8];
  __shared__ uint32_t heads_m, ends_m, tails_m;
  __shared__ long long head_first;  // the first tile of warp 0's first row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.Hq / a.Hkv;
  // started beside the end of the kernel before; the join must not start beside that one too
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  if (tid == 0) heads_m = ends_m = tails_m = 0;
  const int per = 32 * ((rows + 32 * kMaxChunks - 1) / (32 * kMaxChunks));  // rows of a chunk
  const int chunks = (rows + per - 1) / per;
  const int each = (chunks + 31) / 32;  // chunks of a lane
  const bool few = rows <= 32;          // then every warp has all lengths in its lanes
  Keys lane_keys = {0, 0};
  long long lane_tiles = 0;             // of the lane's row, or its chunks
  if (few) {
    if (lane < rows) lane_keys = keys_of(a, a.seq_lens[lane], ring_pos(a, lane));
    lane_tiles = (lane_keys.all + kTile - 1) / kTile;
    __syncthreads();
  } else {
    // --- tiles of all rows, by chunks of rows; kScan chunks' loads at a time, from rows that
    // are there, before the first use
    constexpr int kScan = 4;
    const int b_step = a.w > 0 ? kWarps * per % a.B : 0;
    for (int c0 = warp; c0 < chunks; c0 += kScan * kWarps) {
      long long sum[kScan] = {};
      for (int i = lane; i < per; i += 32) {
        int len[kScan], pos[kScan];
        int b = a.w > 0 ? (c0 * per + i) % a.B : 0;  // sequence of the row
#pragma unroll
        for (int u = 0; u < kScan; ++u) {
          len[u] = a.seq_lens[min((c0 + u * kWarps) * per + i, rows - 1)];
          pos[u] = a.w > 0 ? a.pos[b] : 0;
          b += b_step;
          if (b >= a.B) b -= a.B;
        }
#pragma unroll
        for (int u = 0; u < kScan; ++u) {
          const int r = (c0 + u * kWarps) * per + i;
          const Keys k = keys_of(a, len[u], pos[u]);
          if (r < min(rows, kCachedRows)) cached[r] = k;
          // a row has fewer than 2^27 tiles: 32 of them add up in 32 bits
          sum[u] += __reduce_add_sync(0xffffffffu, r < rows ? (k.all + kTile - 1u) / kTile : 0u);
        }
      }
#pragma unroll
      for (int u = 0; u < kScan; ++u)
        if (lane == 0 && c0 + u * kWarps < chunks) chunk_tiles[c0 + u * kWarps] = sum[u];
    }
    __syncthreads();
    for (int i = 0; i < each; ++i)
      if (lane * each + i < chunks) lane_tiles += chunk_tiles[lane * each + i];
  }
  // --- every warp for itself (a second barrier would cost more): the sum over the lanes,
  // its share of the stream, and the row where that begins
  long long lanes_incl = lane_tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, lanes_incl, o);
    if (lane >= o) lanes_incl += y;
  }
  const long long total = __shfl_sync(0xffffffffu, lanes_incl, 31) * groups;
  const Shares shares(total, gridDim.x * kWarps);
  const long long warps = min((long long)gridDim.x * kWarps, total);
  const int gw = blockIdx.x * kWarps + warp;
  Ends* ends = static_cast<Ends*>(a.ws);
  if (blockIdx.x * kWarps >= warps) {
    if (tid == 0) ends[blockIdx.x] = {-1, 0};
    return;
  }

  if (gw < warps) {
    const long long t0 = shares.first(gw);
    long long t1 = shares.first(gw + 1);
    const long long u0 = groups == 1 ? t0 : t0 / groups;  // in tiles of one group
    const int l0 = __ffs(__ballot_sync(0xffffffffu, lanes_incl > u0)) - 1;
    long long rel = u0 - __shfl_sync(0xffffffffu, lanes_incl - lane_tiles, l0);
    Cursor<kTile> ld;
    ld.group = 0;
    if (few) {
      ld.base = 0;
      ld.mine = lane_keys;
      ld.enter(l0);
    } else {
      int chunk = l0 * each;
      while (rel >= chunk_tiles[chunk]) rel -= chunk_tiles[chunk++];
      for (ld.base = chunk * per;; ld.base += 32) {
        ld.fetch(a, rows, cached, lane);
        const uint32_t mine = (ld.mine.all + kTile - 1) / kTile;
        uint32_t incl = mine;  // 32 rows of fewer than 2^27 tiles
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, incl > rel);
        if (past) {
          const int l = __ffs(past) - 1;
          ld.enter(ld.base + l);
          rel -= __shfl_sync(0xffffffffu, incl - mine, l);
          break;
        }
        rel -= __shfl_sync(0xffffffffu, incl, 31);
        if (ld.base + 32 >= rows) {  // only if the lengths changed since the scan: no work
          t1 = t0;
          rel = 0;
          ld.enter(ld.base);
          break;
        }
      }
    }
    ld.tile = (int)rel;
    if (groups > 1) {  // the row's tiles come once for each group
      const int nt = max(1, (ld.keys.all + kTile - 1) / kTile);
      const long long off = t0 - (u0 - ld.tile) * groups;
      ld.group = (int)(off / nt);
      ld.tile = (int)(off - (long long)ld.group * nt);
    }
    Cursor<kTile> cur = ld;
    if (tid == 0) head_first = t0 - ld.tile;

    uint8_t* ring = smem + warp * warp_bytes(D, NG);
    const uint32_t ring_u = smem_u32(ring);
    long long to_find = t1 - t0;

    Copies<D> copies{a, ps_shift, lane, ring_u, live[warp]};
    bool found = false, started = false;
    auto issue = [&](int stage) {  // copies the tile that was looked up, looks up the next
      if (found) copies.copy(ld.row, ld.tile, ld.keys, stage);
      cp_async_commit();
      found = to_find > 0;
      if (found) {
        --to_find;
        const bool new_row = started ? ld.advance(a, rows, groups, cached, lane) : true;
        copies.look_up(ld.row, ld.tile, ld.keys, new_row);
        started = true;
      }
    };
    Heads<D, NG> heads;
    heads.start(a, cur.row, cur.group, g, lane);
    bool began_here = cur.tile == 0;
    // the look-up leads the copy by one tile, the copy the arithmetic by S - 1
    int stage = 0;
    for (long long t = t0 - S; t < t1; ++t) {
      if (t >= t0) {
        cp_async_wait<S - 2>();
        __syncwarp();
      }
      issue(stage == 0 ? S - 1 : stage - 1);
      if (t < t0) {
        stage = stage == S - 1 ? 0 : stage + 1;
        continue;
      }
      heads.tile(ring_u + stage * kStageBytes, live[warp][stage], lane);
      stage = stage == S - 1 ? 0 : stage + 1;

      const bool row_end = cur.at_row_end(), last = t + 1 == t1;
      if (!row_end && !last) {
        ++cur.tile;
        continue;
      }
      heads.fold();
      if (row_end && began_here) {
        heads.store(a, cur.row, cur.group, g, lane);
      } else {
        // a part: a tail into the ring, where nothing is in flight any more
        const int id = began_here ? kWarps + warp : warp;
        if (began_here) {
          cp_async_wait<0>();
          __syncwarp();
        }
        heads.leave(reinterpret_cast<float*>(ring + (began_here ? 0 : kRingBytes)), ref_s[id],
                    sum_s[id], lane);
        if (lane == 0) {
          vrow_of[id] = cur.row * groups + cur.group;
          atomicOr(began_here ? &tails_m : &heads_m, 1u << warp);
          if (!began_here && row_end) atomicOr(&ends_m, 1u << warp);
        }
      }
      if (!last) {
        cur.advance(a, rows, groups, cached, lane);
        heads.start(a, cur.row, cur.group, g, lane);
        began_here = true;
      }
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  // --- join the rows that cross shares inside the block: a chain of parts comes from the
  // block before, or begins with a warp's tail, and goes on through the next warps' heads
  // until one ends the row.  Bit 0 of `starts` is the chain from before, bit w + 1 the one
  // that begins with warp w's tail
  const uint32_t heads = heads_m, stop = ends_m | ~heads;
  const uint32_t starts = (heads & 1) | (tails_m << 1);
  if (tid == 0) {
    Ends e = {-1, 0};
    if ((heads & 1) && (ends_m & (stop & -stop)))
      e = {vrow_of[0], (int)(shares.of(head_first) / kWarps)};
    ends[blockIdx.x] = e;
  }
  // a warp takes a chain, or with few chains a slice of one, eight fragments at a time with
  // all their loads in flight
  constexpr int kUnits = NF / 8;
  int slices = kUnits;
  while (slices > NG && __popc(starts) * slices > kWarps) slices >>= 1;
  const int work = __popc(starts) * slices;
  for (int v = warp; v < work; v += kWarps) {
    uint32_t left = starts;
    for (int c = v / slices; c > 0; --c) left &= left - 1;
    const int from = __ffs(left) - 1;  // first head of the chain
    const int len = __ffs(stop >> from) - 1;  // heads that go on (a stop is found: 16 bits of 32)
    const bool ended = (ends_m >> (from + len)) & 1, before = from == 0;
    const int n = len + (ended ? 1 : 0), tail = kWarps + from - 1;  // heads from .. from + n - 1
    const int u0 = v % slices * (kUnits / slices);
    // heads of the lane's columns: even and odd fragments; a slice has one j
    const int h0 = u0 * 8 / (KS * 4) * 8 + (lane & 3) * 2;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!before) top[i] = ref_s[tail][h0 + i];
      for (int p = from; p < from + n; ++p) top[i] = fmaxf(top[i], ref_s[p][h0 + i]);
    }
    for (int u = u0; u < u0 + kUnits / slices; ++u) {
      const int f0 = u * 8;
      float acc[8] = {};
      sum[0] = sum[1] = 0.f;
      auto add = [&](int id) {
        float w[2];
        const float* x = reinterpret_cast<const float*>(
            smem + (id < kWarps ? id * warp_bytes(D, NG) + kRingBytes
                                : (id - kWarps) * warp_bytes(D, NG))) + f0 * 32 + lane;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i] = fast_exp2(ref_s[id][h0 + i] - finite_ref(top[i]));
          sum[i] += sum_s[id][h0 + i] * w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += x[i * 32] * w[i & 1];
      };
      if (!before) add(tail);
#pragma unroll 2
      for (int p = from; p < from + n; ++p) add(p);
      if (ended && !before) {
        const int vrow = vrow_of[tail], row = vrow / groups;
        store_unit<D, NG>(a, row, vrow - row * groups, g, f0, acc, top, sum, lane);
      } else {  // a part for the second kernel
        float* out = block_part(a.ws, blockIdx.x, before ? 0 : 1, PF);
#pragma unroll
        for (int i = 0; i < 8; ++i) out[(f0 + i) * 32 + lane] = acc[i];
        if (lane < 4 && f0 % (KS * 4) == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            out[NF * 32 + h0 + i] = top[i];
            out[NF * 32 + NG * 8 + h0 + i] = sum[i];
          }
        }
      }
    }
  }
}

// While the first kernel runs: the outputs of rows without keys, which no block of it meets,
// and lengths out of range.
template <int D>
__device__ __forceinline__ void rows_without_keys(const AttnDecodeArgs& a, int rows, int g) {
  const int every = gridDim.x * gridDim.y * kJoinThreads;
  for (int r = (blockIdx.y * gridDim.x + blockIdx.x) * kJoinThreads + threadIdx.x; r < rows;
       r += every) {
    const int len = a.seq_lens[r];
    if (len < 0 || len > a.max_pages * a.page_size)
      atomicCAS(&g_attn_decode_error, 0, kErrAttnDecode);
    if (keys_of(a, len, ring_pos(a, r)).all == 0) {
      for (int h = 0; h < g; ++h) {
        uint4* out = reinterpret_cast<uint4*>(a.o + out_row(a, r, g, h) * D);
        for (int e = 0; e < D / 8; ++e) out[e] = make_uint4(0, 0, 0, 0);
        if (a.lse) a.lse[out_row(a, r, g, h)] = -INFINITY;
      }
    }
  }
}

// Rows that cross blocks: block x joins the row that ends in block x of the first kernel,
// from the tail of its first block and the heads of those after.  Registers for six blocks an
// SM let one come up beside each block of the first kernel; six parts with their loads early
// instead of 24, which spilled at d = 64: 36.2 -> 35.1 us for 384 rows of 131 tiles.
template <int D, int NG>
__global__ void __launch_bounds__(kJoinThreads, 6) attn_decode_join_kernel(
    const __grid_constant__ AttnDecodeArgs a, int rows, int groups) {
  constexpr int KS = D / 16, PF = part_floats(D, NG), NF = frags(D, NG);
  constexpr int kFirst = 6;  // parts whose loads start before the weights are known
  __shared__ float ref_s[kMaxBlocks][NG * 8], sum_s[kMaxBlocks][NG * 8];
  const int g = a.Hq / a.Hkv;
  rows_without_keys<D>(a, rows, g);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int f = blockIdx.y * kJoinThreads + threadIdx.x;
  const int j = f / (32 * KS * 4), s = f / 128 % KS, c = f / 32 % 4, ln = f & 31;
  const int h = j * 8 + (ln & 3) * 2 + (c & 1), dim = s * 16 + (ln >> 2) + (c >> 1) * 8;
  // most rows cross one border: these two parts come beside the word on it (384 rows at d = 64
  // 35.2 -> 34.5 us)
  float x2[2], ref2[2], sum2[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const float* from = block_part(a.ws, max((int)blockIdx.x - 1 + p, 0), 1 - p, PF);
    x2[p] = from[f];
    ref2[p] = from[NF * 32 + h];
    sum2[p] = from[NF * 32 + NG * 8 + h];
  }
  const Ends end = static_cast<const Ends*>(a.ws)[blockIdx.x];
  // the bounds hold even if another stream writes the workspace meanwhile
  if ((uint32_t)end.vrow >= (uint32_t)(rows * groups) || (uint32_t)end.first >= blockIdx.x) return;
  const int n = blockIdx.x - end.first + 1;
  const int row = end.vrow / groups;
  const int head = (end.vrow - row * groups) * NG * 8 + h;
  if (n == 2) {
    const float top = fmaxf(ref2[0], ref2[1]), base = finite_ref(top);
    const float w0 = fast_exp2(ref2[0] - base), w1 = fast_exp2(ref2[1] - base);
    if (head < g)
      store_out<D>(a, out_row(a, row, g, head), dim, x2[0] * w0 + x2[1] * w1, top,
                   sum2[0] * w0 + sum2[1] * w1);
    return;
  }
  auto part = [&](int p) { return block_part(a.ws, end.first + p, p == 0 ? 1 : 0, PF); };
  float x[kFirst];
#pragma unroll
  for (int p = 0; p < kFirst; ++p) x[p] = p < n ? part(p)[f] : 0.f;
  for (int i = threadIdx.x; i < n * NG * 8; i += kJoinThreads) {
    const float* q = part(i / (NG * 8)) + NF * 32 + i % (NG * 8);
    ref_s[i / (NG * 8)][i % (NG * 8)] = q[0];
    sum_s[i / (NG * 8)][i % (NG * 8)] = q[NG * 8];
  }
  __syncthreads();
  float top = -INFINITY;
  for (int p = 0; p < n; ++p) top = fmaxf(top, ref_s[p][h]);
  const float base = finite_ref(top);
  float acc = 0.f, sum = 0.f;
#pragma unroll
  for (int p = 0; p < kFirst; ++p) {
    if (p < n) {
      const float w = fast_exp2(ref_s[p][h] - base);
      acc += x[p] * w;
      sum += sum_s[p][h] * w;
    }
  }
#pragma unroll 8
  for (int p = kFirst; p < n; ++p) {
    const float w = fast_exp2(ref_s[p][h] - base);
    acc += part(p)[f] * w;
    sum += sum_s[p][h] * w;
  }
  if (head < g) store_out<D>(a, out_row(a, row, g, head), dim, acc, top, sum);
}

// The same for few rows, each over many blocks: a block per row and fragment, whose warps
// take every eighth part and meet in shared memory, so that the parts' loads come in one or a
// few rounds; which parts they are it works out while the first kernel runs.  Against the
// kernel above (us): one row of 16384 tokens over 103 blocks 9.1 / 14.6, of 262144 over 152
// 30.7 / 34.5; 4 rows over 38 11.9 / 13.6; 8 rows of a 131072-token document over 19 29.6 /
// 30.9; 16 rows over 9 19.1 / 19.6; with the parts read from the first kernel's word on each
// border instead 9.5, 32.4, 12.4, 29.9 and 18.8.  32 rows over 5 take 66.5 / 66.1.
template <int D, int NG>
__global__ void __launch_bounds__(kJoinThreads) attn_decode_join_few_kernel(
    const __grid_constant__ AttnDecodeArgs a, int rows, int groups, int blocks) {
  constexpr int KS = D / 16, PF = part_floats(D, NG), NF = frags(D, NG);
  constexpr int kWarps = kJoinThreads / 32, kAhead = 4;
  __shared__ float acc_s[kWarps][32], top_s[kWarps][32], sum_s[kWarps][32];
  static_assert(kMaxBlocks / 8 <= 32, "a lane per row");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = a.Hq / a.Hkv;
  rows_without_keys<D>(a, rows, g);
  // while the first kernel runs: its blocks that share this row, by the same arithmetic
  const int vrow = blockIdx.x, row = vrow / groups;
  const int tiles = lane < rows ? (keys_of(a, a.seq_lens[lane], ring_pos(a, lane)).all +
                                   tile_keys(D) - 1) / tile_keys(D) : 0;
  long long all = tiles, before = lane < row ? tiles : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  const int mine = __shfl_sync(0xffffffffu, tiles, row);
  const Shares shares(all * groups, blocks * warps_of(D, NG));
  const long long tile0 = before * groups + (long long)(vrow - row * groups) * mine;
  const int first = mine ? (int)(shares.of(tile0) / warps_of(D, NG)) : 0;
  const int n = mine ? (int)(shares.of(tile0 + mine - 1) / warps_of(D, NG)) - first + 1 : 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n == 1) return;  // the first kernel has written it
  const int f = blockIdx.y, j = f / (KS * 4), s = f / 4 % KS, c = f % 4;
  const int h = j * 8 + (lane & 3) * 2 + (c & 1), dim = s * 16 + (lane >> 2) + (c >> 1) * 8;
  float top = -INFINITY, acc = 0.f, sum = 0.f;
  for (int p0 = warp; p0 < n; p0 += kAhead * kWarps) {
    float x[kAhead], ref[kAhead], part_sum[kAhead], high = top;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int p = p0 + i * kWarps;
      const float* from = block_part(a.ws, first + min(p, n - 1), p == 0 ? 1 : 0, PF);
      x[i] = from[f * 32 + lane];
      ref[i] = p < n ? from[NF * 32 + h] : -INFINITY;
      part_sum[i] = from[NF * 32 + NG * 8 + h];
      if (p >= n) x[i] = part_sum[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) high = fmaxf(high, ref[i]);
    const float base = finite_ref(high), w = fast_exp2(top - base);
    acc *= w;
    sum *= w;
    top = high;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float v = fast_exp2(ref[i] - base);
      acc += x[i] * v;
      sum += part_sum[i] * v;
    }
  }
  acc_s[warp][lane] = acc;
  top_s[warp][lane] = top;
  sum_s[warp][lane] = sum;
  __syncthreads();
  if (warp) return;
  top = -INFINITY;
#pragma unroll
  for (int v = 0; v < kWarps; ++v) top = fmaxf(top, top_s[v][lane]);
  acc = sum = 0.f;
#pragma unroll
  for (int v = 0; v < kWarps; ++v) {
    const float w = fast_exp2(top_s[v][lane] - finite_ref(top));
    acc += acc_s[v][lane] * w;
    sum += sum_s[v][lane] * w;
  }
  const int head = (vrow - row * groups) * NG * 8 + h;
  if (head < g) store_out<D>(a, out_row(a, row, g, head), dim, acc, top, sum);
}

// The same for rows that cannot be long: a block, or a cluster of blocks, per row and group
// of heads, with equal contiguous shares of the row's tiles per warp.  No scan over other
// rows, no workspace and no second kernel: a block's warps meet in its shared memory, and a
// cluster's blocks send their parts to the one that sums them up.
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// to the same place in the shared memory of another block of the cluster
__device__ __forceinline__ void st_cluster(const float* to, uint32_t rank, float x) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(to)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}

// What a block of a cluster is sent: eight fragments and eight heads' references and sums,
// from each block for each unit that it owns (units u with u % blocks == rank).  Units and
// blocks are powers of two up to 8, so max(units, blocks) parts arrive at most.
struct Sent { float x[8 * 32], ref[8], sum[8]; };

template <int D, int NG, int W>
__global__ void __launch_bounds__(W * 32, (NG == 1 ? 12 : 8) / W) attn_decode_row_kernel(
    const __grid_constant__ AttnDecodeArgs a, int groups, int ps_shift) {
  constexpr int S = kStages, KS = D / 16, NF = frags(D, NG), H = NG * 8, kTile = tile_keys(D);
  static_assert(NF / 8 <= kMaxCluster && (NF & (NF - 1)) == 0, "units fit what is sent");
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint32_t live[W][S];
  __shared__ float ref_s[W][H], sum_s[W][H];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.Hq / a.Hkv;
  const int blocks = cluster_size(), rank = blockIdx.x % blocks;
  const int vrow = blockIdx.x / blocks, row = vrow / groups, group = vrow - row * groups;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // started beside the kernel before
  const int len = a.seq_lens[row];
  const Keys keys = keys_of(a, len, ring_pos(a, row));
  if (tid == 0 && rank == 0 && keys.paged != len) atomicCAS(&g_attn_decode_error, 0, kErrAttnDecode);
  Sent* sent = reinterpret_cast<Sent*>(smem + W * kRingBytes);
  if (blocks > 1) cluster_arrive();  // this block has started: its shared memory may be written
  uint8_t* ring = smem + warp * kRingBytes;
  const uint32_t ring_u = smem_u32(ring);
  Heads<D, NG> heads;
  heads.start(a, row, group, g, lane);
  {
    const uint32_t tiles = (keys.all + kTile - 1u) / kTile;  // below 2^27, of up to 32 warps
    const uint32_t me = rank * W + warp, all = blocks * W;
    const int t0 = me * tiles / all, t1 = (me + 1) * tiles / all;
    Copies<D> copies{a, ps_shift, lane, ring_u, live[warp]};
    int stage = 0;
    for (int t = t0 - S; t < t1; ++t) {
      if (t >= t0) {
        cp_async_wait<S - 2>();
        __syncwarp();
      }
      const int next = t + S;  // the look-up leads the copy by one tile, as in the stream
      if (next > t0 && next - 1 < t1)
        copies.copy(row, next - 1, keys, stage == 0 ? S - 1 : stage - 1);
      cp_async_commit();
      if (next < t1) copies.look_up(row, next, keys, next == t0);
      if (t >= t0) heads.tile(ring_u + stage * kStageBytes, live[warp][stage], lane);
      stage = stage == S - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncwarp();
  }
  heads.fold();
  heads.leave(reinterpret_cast<float*>(ring), ref_s[warp], sum_s[warp], lane);
  __syncthreads();
  if (blocks > 1) cluster_wait();
  // --- the block's warps, eight fragments a warp at a time
  constexpr int kUnits = NF / 8;
  for (int u = warp; u < kUnits; u += W) {
    const int f0 = u * 8, h0 = f0 / (KS * 4) * 8 + (lane & 3) * 2;
    float top[2], sum[2] = {}, acc[8] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = ref_s[0][h0 + i];
      for (int p = 1; p < W; ++p) top[i] = fmaxf(top[i], ref_s[p][h0 + i]);
    }
#pragma unroll
    for (int p = 0; p < W; ++p) {
      const float* x = reinterpret_cast<const float*>(smem + p * kRingBytes) + f0 * 32 + lane;
      float w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = fast_exp2(ref_s[p][h0 + i] - finite_ref(top[i]));
        sum[i] += sum_s[p][h0 + i] * w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += x[i * 32] * w[i & 1];
    }
    if (blocks == 1) {
      store_unit<D, NG>(a, row, group, g, f0, acc, top, sum, lane);
    } else {
      Sent& to = sent[u / blocks * blocks + rank];
#pragma unroll
      for (int i = 0; i < 8; ++i) st_cluster(&to.x[i * 32 + lane], u % blocks, acc[i]);
      if (lane < 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          st_cluster(&to.ref[lane * 2 + i], u % blocks, top[i]);
          st_cluster(&to.sum[lane * 2 + i], u % blocks, sum[i]);
        }
      }
    }
  }
  if (blocks == 1) return;
  // --- the cluster's blocks, each unit by the block that owns it
  cluster_arrive();
  cluster_wait();
  for (int u = rank + blocks * warp; u < kUnits; u += blocks * W) {
    const Sent* from = sent + u / blocks * blocks;
    const int h = (lane & 3) * 2;
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {}, acc[8] = {};
    for (int p = 0; p < blocks; ++p)
#pragma unroll
      for (int i = 0; i < 2; ++i) top[i] = fmaxf(top[i], from[p].ref[h + i]);
#pragma unroll 4
    for (int p = 0; p < blocks; ++p) {
      float w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = fast_exp2(from[p].ref[h + i] - finite_ref(top[i]));
        sum[i] += from[p].sum[h + i] * w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += from[p].x[i * 32 + lane] * w[i & 1];
    }
    store_unit<D, NG>(a, row, group, g, u * 8, acc, top, sum, lane);
  }
}

// Warps of a block and blocks of a cluster per row where the row kernel takes a call, else
// no warps (the stream).  The actual lengths are on the device, so the rule goes by what a
// row may hold: at most 16 tiles a warp, or 6 where even clusters of 8 leave SMs idle.  Rows
// 30 to 100 % full, row kernel against stream (us): 8 rows of 58 tiles 7.0 / 9.4, of 241
// tiles 11.4 / 10.1; 32 rows of 126 tiles 9.1 / 11.9; 128 rows of 15 tiles 7.0 / 11.5, of 61
// tiles 13.3 / 16.3, of 246 tiles 37.4 / 33.0; 512 rows of 16 tiles 12.9 / 17.2, of 63 tiles
// 32.0 / 32.3, of 249 tiles 101 / 87.  More short rows than three blocks an SM take blocks of
// two warps, six on an SM, which overlap one another's starts and joins better than three of
// four warps: 512 rows of 14 tiles 12.5 / 13.4, 2048 rows of 15 tiles 35.4 / 37.9, 16384 rows
// 203 / 239, 2048 rows of 4 tiles 16.7 / 23.2; of 38 tiles 55.1 / 53.5.
struct RowShape { int warps, cluster; };
RowShape row_shape(long long vrows, long long row_tiles) {
  if (vrows > 152 * 3 && row_tiles <= 2 * 16) return {2, 1};
  int c = 1;
  while (c < kMaxCluster && vrows * c * 2 <= 152 * 3) c *= 2;
  const int most = vrows * c >= 152 ? 16 : 6;
  return {row_tiles <= c * 4 * most ? 4 : 0, c};
}

template <int D, int NG, int W>
cudaError_t launch_rows(const AttnDecodeArgs& a, long long vrows, int cluster, int groups, int shift,
                        cudaStream_t s) {
  constexpr int sent = kMaxCluster * (int)sizeof(Sent);
  const int smem = W * kRingBytes + (cluster > 1 ? sent : 0);
  // the same limit whatever this call needs: another thread may launch the other form
  cudaError_t e = cudaFuncSetAttribute(attn_decode_row_kernel<D, NG, W>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       W * kRingBytes + sent);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(vrows * cluster));
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, attn_decode_row_kernel<D, NG, W>, a, groups, shift);
}

template <int D, int NG>
cudaError_t launch(AttnDecodeArgs a, int rows, int groups, cudaStream_t s) {
  constexpr int kWarps = warps_of(D, NG), kTile = tile_keys(D);
  constexpr int smem = kWarps * warp_bytes(D, NG) + kCachedRows * (int)sizeof(Keys);
  static int nsm[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!nsm[dev]) {
    e = cudaDeviceGetAttribute(&nsm[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
  }
  int shift = -1;
  if ((a.page_size & (a.page_size - 1)) == 0)
    for (shift = 0; (1 << shift) < a.page_size; ++shift) {}
  const long long vrows = (long long)rows * groups;
  const long long row_tiles = ((long long)a.max_pages * a.page_size + a.w + kTile - 1) / kTile;
  a.read_once = groups == 1 && (long long)rows * row_tiles * kStageBytes > kL2Bytes / 2;
  const RowShape shape = row_shape(vrows, row_tiles);
  if (shape.warps == 4) return launch_rows<D, NG, 4>(a, vrows, shape.cluster, groups, shift, s);
  if (shape.warps == 2) return launch_rows<D, NG, 2>(a, vrows, shape.cluster, groups, shift, s);
  // no more blocks than tiles could need
  const long long want = (vrows * row_tiles + kWarps - 1) / kWarps;
  const int sms = nsm[dev] < kMaxBlocks ? nsm[dev] : kMaxBlocks;
  const int blocks = (int)(want < sms ? want : sms);
  e = cudaFuncSetAttribute(attn_decode_kernel<D, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem);
  if (e != cudaSuccess) return e;
  count_launches(2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, NG>, a, rows, groups, shift);
  if (e != cudaSuccess) return e;
  // the join's blocks come up while the first kernel runs and wait for its results
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  if (vrows * 8 <= blocks) {
    cfg.gridDim = dim3((unsigned)vrows, frags(D, NG));
    return cudaLaunchKernelEx(&cfg, attn_decode_join_few_kernel<D, NG>, a, rows, groups, blocks);
  }
  cfg.gridDim = dim3(blocks, frags(D, NG) * 32 / kJoinThreads);
  return cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D, NG>, a, rows, groups);
}

}  // namespace

size_t attn_decode_workspace_bytes(int group, int d) {
  const int ng = group <= 8 ? 1 : 2;
  return ends_bytes() + (size_t)kMaxBlocks * 2 * part_floats(d, ng) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& args, cudaStream_t s) {
  AttnDecodeArgs a = args;
  const int rows = a.L * a.Hkv * a.B, g = a.Hq / a.Hkv;
  if (rows == 0) return cudaSuccess;
  // a copy of no bytes still names an address: one that is there and aligned, whatever came
  // for a pool of no pages or a ring of no slots (those are not checked)
  if (a.capacity == 0) a.k_pages = a.v_pages = a.q;
  if (a.w == 0) a.ring_k = a.ring_v = a.q;
  // groups of 8 heads fill an MMA's N; above 8 a pass takes 16, so that K and V are read
  // once for up to 16 heads
  if (g <= 8)
    return a.d == 128 ? launch<128, 1>(a, rows, 1, s) : launch<64, 1>(a, rows, 1, s);
  const int groups = (g + 15) / 16;
  return a.d == 128 ? launch<128, 2>(a, rows, groups, s) : launch<64, 2>(a, rows, groups, s);
}

cudaError_t attn_decode_device_error(int* code, bool clear, cudaStream_t s) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(code, g_attn_decode_error, sizeof(int), 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && clear && *code) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_attn_decode_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice,
                                s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

}  // namespace kvs
