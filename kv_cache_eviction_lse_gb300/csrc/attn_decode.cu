// Attention of one new token per sequence over its row's paged cache and window ring:
//   o = sum_i a_i v_i,  a_i = exp(q . k_i / sqrt(d) - lse),  lse = ln sum_i exp(q . k_i / sqrt(d))
// over the row's seq_lens[r] paged keys and the min(pos, w) keys of its ring, for the g
// query heads of the row's KV head.  Every key is read once for all g heads: 4 d bytes and
// 4 d g flops, so HBM bounds it (g flop/B; the tensor cores take over 200).
//
// Rows differ in length by the pruning, so the work is cut by tiles, not by rows: all rows'
// tiles of 16 keys form one stream, every warp of a persistent grid takes an equal
// contiguous share, and a row that crosses a share's border is joined from partial sums
// (running maximum, sum and weighted values): within a block through shared memory, between
// blocks by a second kernel.  Shares depend on the lengths alone, so results do too.
//
// A warp streams its tiles through a private ring of cp.async stages (128-byte swizzle, no
// block barrier), across row borders: the loads of the next rows are in flight while a row
// is finished.  Per tile (mma.m16n8k16, keys in M, heads in N, bf16 -> fp32):
//   S^T = K Q^T       A = K rows by ldmatrix, B = Q in registers
//   P^T = exp2(S^T)   in registers, turned into a B operand by movmatrix
//   O^T += V^T P^T    A = V by ldmatrix.trans
// With keys in M a group of 8 query heads fills N exactly; tcgen05 (M = 128) would spend
// its rows on 4 to 8 heads and a TMEM round trip per tile, on a contraction that needs a
// fiftieth of its rate.  The softmax reference is raised only when a tile exceeds it by 2^8
// (one vote per tile instead of a cross-lane maximum); weights stay below 2^8, are rounded
// to bf16 (at most 2^-8 relative, of either sign over the keys) and summed in fp32.
#include "attn_decode.cuh"
#include "common.cuh"

namespace kvs {

__device__ int g_attn_decode_error = 0;

namespace {

constexpr int kErrAttnDecode = 9;  // a length or page id out of range

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;        // keys
constexpr int kMaxBlocks = 160;  // of the persistent grid; sizes the workspace
constexpr int kMaxChunks = 256;  // of rows, in the scan of their tiles
constexpr float kSlack = 8.f;    // log2 of how far a weight may exceed the reference

__host__ __device__ constexpr int stages(int d) { return d == 128 ? 3 : 6; }
__host__ __device__ constexpr int stage_bytes(int d) { return 2 * kTile * d * 2; }
constexpr int kRingBytes = stages(128) * stage_bytes(128);  // per warp, either d

// A partial result of a row segment: O^T fragments [d / 16 * 4 * NG][32 lanes], then the
// reference and the sum of each of the 8 NG heads.
__host__ __device__ constexpr int frags(int d, int ng) { return d / 16 * 4 * ng; }
__host__ __device__ constexpr int part_floats(int d, int ng) { return frags(d, ng) * 32 + 16 * ng; }

// Workspace: per block the row that ends there having begun in another block (or -1) and
// that other block; per warp the part of a row that ends inside its share; per block the
// parts of the rows that cross its borders (0: began before, 1: goes on after).
struct Ends { int vrow, first; };
__host__ __device__ constexpr size_t ends_bytes() { return kMaxBlocks * sizeof(Ends); }
__device__ float* warp_part(void* ws, int warp, int pf) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + ends_bytes()) + (size_t)warp * pf;
}
__device__ float* block_part(void* ws, int block, int side, int pf) {
  return warp_part(ws, kMaxBlocks * kWarps + 2 * block + side, pf);
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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }

// The keys of a row: paged tokens, and with the ring's.
struct Keys { int paged, all; };

__device__ __forceinline__ Keys row_keys(const AttnDecodeArgs& a, int row, bool report) {
  const int room = a.max_pages * a.page_size;
  int n = a.seq_lens[row];
  if (n < 0 || n > room) {
    if (report) atomicCAS(&g_attn_decode_error, 0, kErrAttnDecode);
    n = n < 0 ? 0 : room;
  }
  const int held = a.w > 0 ? max(0, min(a.pos[row % a.B], a.w)) : 0;
  return {n, n + held};
}

// A place in the stream of tiles.  The lanes hold the lengths of the 32 rows from `base` on.
struct Cursor {
  int row, group, tile;   // group: which 8 NG of the row's query heads
  Keys keys;              // of the row
  int base, paged, all;   // lane i: the lengths of row base + i

  __device__ __forceinline__ void fetch(const AttnDecodeArgs& a, int rows, int lane) {
    Keys k = {0, 0};
    if (base + lane < rows) k = row_keys(a, base + lane, false);
    paged = k.paged;
    all = k.all;
  }
  __device__ __forceinline__ void enter(int r) {
    row = r;
    keys.paged = __shfl_sync(0xffffffffu, paged, r - base);
    keys.all = __shfl_sync(0xffffffffu, all, r - base);
  }
  __device__ __forceinline__ bool at_row_end() const { return (tile + 1) * kTile >= keys.all; }
  // the next tile; there is one
  __device__ __forceinline__ void advance(const AttnDecodeArgs& a, int rows, int groups, int lane) {
    if (!at_row_end()) { ++tile; return; }
    tile = 0;
    if (++group < groups) return;
    group = 0;
    int from = row - base + 1;
    for (;;) {
      const uint32_t some = __ballot_sync(0xffffffffu, all > 0) &
                            (from < 32 ? 0xffffffffu << from : 0u);
      if (some) { enter(base + __ffs(some) - 1); return; }
      base += 32;
      from = 0;
      if (base >= rows) return;  // not reached while tiles remain
      fetch(a, rows, lane);
    }
  }
};

// Output rows of the 8 NG heads of a group: element offset of head h's row.
__device__ __forceinline__ size_t out_row(const AttnDecodeArgs& a, int row, int g, int head) {
  return ((size_t)(row / a.B) * g + head) * a.B + row % a.B;
}

template <int D>
__device__ __forceinline__ void store_out(const AttnDecodeArgs& a, size_t r, int dim, float acc,
                                          float top, float sum) {
  a.o[r * D + dim] = (bf16_t)(pack2(sum == 0.f ? 0.f : acc / sum, 0.f) & 0xffffu);
  if (a.lse && dim == 0) a.lse[r] = sum == 0.f ? -INFINITY : kLn2 * (top + log2f(sum));
}

template <int D, int NG>
__global__ void __launch_bounds__(kThreads, 1) attn_decode_kernel(
    const __grid_constant__ AttnDecodeArgs a, int rows, int groups, int ps_shift) {
  constexpr int S = stages(D), KS = D / 16, PF = part_floats(D, NG), NF = frags(D, NG);
  static_assert(PF * 4 <= kRingBytes, "a partial fits the ring");
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long prefix[kMaxChunks + 1];
  __shared__ uint32_t live[kWarps][S];
  // what each warp leaves behind: a row that began before its share (head) and one that
  // goes on after it (tail); nullptr where there is none
  __shared__ float *head_part[kWarps], *tail_part[kWarps];
  __shared__ int head_vrow[kWarps], tail_vrow[kWarps], head_ends[kWarps];
  __shared__ long long head_first;  // the first tile of warp 0's first row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.Hq / a.Hkv;
  asm volatile("griddepcontrol.launch_dependents;");

  // --- tiles of all rows, by chunks of rows
  const int per = 32 * ((rows + 32 * kMaxChunks - 1) / (32 * kMaxChunks));
  const int chunks = (rows + per - 1) / per;
  for (int c = warp; c < chunks; c += kWarps) {
    const bool mine = c % gridDim.x == blockIdx.x;  // reports, and fills empty rows
    long long sum = 0;
    for (int i = lane; i < per; i += 32) {
      const int r = c * per + i;
      const int n = r < rows ? row_keys(a, r, mine).all : -1;
      sum += (max(n, 0) + kTile - 1) / kTile;
      uint32_t empty = mine ? __ballot_sync(0xffffffffu, n == 0) : 0u;
      for (; empty; empty &= empty - 1) {
        const int er = c * per + (i - lane) + __ffs(empty) - 1;
        for (int e = lane; e < g * (D / 8); e += 32)
          reinterpret_cast<uint4*>(a.o + out_row(a, er, g, e / (D / 8)) * D)[e % (D / 8)] =
              make_uint4(0, 0, 0, 0);
        if (a.lse)
          for (int h = lane; h < g; h += 32) a.lse[out_row(a, er, g, h)] = -INFINITY;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) prefix[c + 1] = sum * groups;
  }
  if (lane == 0) {
    head_part[warp] = tail_part[warp] = nullptr;
    head_ends[warp] = 0;
  }
  __syncthreads();
  if (warp == 0) {
    constexpr int kEach = kMaxChunks / 32;
    long long v[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = lane * kEach + i;
      sum += c < chunks ? prefix[c + 1] : 0;
      v[i] = sum;
    }
    long long before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    before -= sum;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = lane * kEach + i;
      if (c < chunks) prefix[c + 1] = before + v[i];
    }
    if (lane == 0) prefix[0] = 0;
  }
  __syncthreads();
  const long long total = prefix[chunks];
  const long long warps = min((long long)gridDim.x * kWarps, total);
  const int gw = blockIdx.x * kWarps + warp;
  Ends* ends = static_cast<Ends*>(a.ws);
  if (blockIdx.x * kWarps >= warps) {
    if (tid == 0) ends[blockIdx.x] = {-1, 0};
    return;
  }

  if (gw < warps) {
    const long long t0 = gw * total / warps, t1 = (gw + 1) * total / warps;
    // --- the row of the share's first tile
    int lo = 0, hi = chunks;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= t0) lo = mid; else hi = mid;
    }
    Cursor ld;
    ld.base = lo * per;
    long long at = prefix[lo];
    int off;  // tiles from the row's first (of all its groups) to t0
    long long row_first;
    for (;;) {
      ld.fetch(a, rows, lane);
      const long long mine = (long long)((ld.all + kTile - 1) / kTile) * groups;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, at + incl > t0);
      if (past) {
        const int l = __ffs(past) - 1;
        ld.enter(ld.base + l);
        row_first = at + __shfl_sync(0xffffffffu, incl - mine, l);
        off = (int)(t0 - row_first);
        break;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
      ld.base += 32;
    }
    const int nt = (ld.keys.all + kTile - 1) / kTile;
    ld.group = off / nt;
    ld.tile = off - ld.group * nt;
    Cursor cur = ld;
    const long long first_vrow_tile = row_first + (long long)ld.group * nt;

    uint8_t* ring = smem + warp * kRingBytes;
    const uint32_t ring_u = smem_u32(ring);
    long long to_load = t1 - t0;

    // --- producer: lane i < 16 finds where key i of the tile lies
    int page = -1, inside = 0;   // paged key: its page id and row in the page
    int slot = -1;               // ring key: its slot
    auto look_up = [&]() {
      page = slot = -1;
      const int key = ld.tile * kTile + lane;
      if (lane < kTile && key < ld.keys.all) {
        if (key < ld.keys.paged) {
          const int idx = ps_shift >= 0 ? key >> ps_shift : key / a.page_size;
          inside = key - idx * a.page_size;
          page = a.block_table[(size_t)ld.row * a.max_pages + idx];
          if (page < 0 || page >= a.capacity) {
            atomicCAS(&g_attn_decode_error, 0, kErrAttnDecode);
            page = -1;
          }
        } else {
          slot = key - ld.keys.paged;
        }
      }
    };
    auto issue = [&](int stage) {
      if (to_load > 0) {
        // row index in the pool, or (negative) in the ring
        long long at_row = -1;
        bool in_ring = false;
        if (page >= 0) {
          at_row = (long long)page * a.page_size + inside;
        } else if (slot >= 0) {
          at_row = (long long)ld.row * a.w + slot;
          in_ring = true;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, at_row >= 0);
        const uint32_t ringed = __ballot_sync(0xffffffffu, in_ring);
        if (lane == 0) live[warp][stage] = here;
        constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes a row, rows a step
        const int c = lane % kLanes;
        const uint32_t dst = ring_u + stage * stage_bytes(D);
#pragma unroll
        for (int i = 0; i < kTile / kRows; ++i) {
          const int key = i * kRows + lane / kLanes;
          const long long r = __shfl_sync(0xffffffffu, at_row, key);
          const bool ok = (here >> key) & 1, rg = (ringed >> key) & 1;
          const size_t e = ok ? (size_t)r * D + c * 8 : 0;
          const bf16_t* k = rg ? a.ring_k : a.k_pages;
          const bf16_t* v = rg ? a.ring_v : a.v_pages;
          const uint32_t to = dst + key * (D * 2) + ((c ^ (key & 7)) << 4);
          cp_async16(to, k + e, ok ? 16 : 0);
          cp_async16(to + kTile * D * 2, v + e, ok ? 16 : 0);
        }
        --to_load;
        if (to_load > 0) {
          ld.advance(a, rows, groups, lane);
          look_up();
        }
      }
      cp_async_commit();
    };
    look_up();
    for (int s = 0; s < S - 1; ++s) issue(s);

    // --- consumer
    const float scale = rsqrtf((float)D) * kLog2e;
    uint32_t qf[NG][KS][2];
    float o[NG][KS][4], m[NG][2], l[NG][2];
    auto start = [&]() {
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const int head = (cur.group * NG + j) * 8 + (lane >> 2);
        const bf16_t* q = a.q + out_row(a, cur.row, g, head) * D + (lane & 3) * 2;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          qf[j][s][0] = head < g ? *reinterpret_cast<const uint32_t*>(q + s * 16) : 0u;
          qf[j][s][1] = head < g ? *reinterpret_cast<const uint32_t*>(q + s * 16 + 8) : 0u;
          o[j][s][0] = o[j][s][1] = o[j][s][2] = o[j][s][3] = 0.f;
        }
        m[j][0] = m[j][1] = -INFINITY;
        l[j][0] = l[j][1] = 0.f;
      }
    };
    start();
    bool began_here = cur.tile == 0;
    if (tid == 0) head_first = first_vrow_tile;
    int stage = 0;
    for (long long t = t0; t < t1; ++t) {
      cp_async_wait<S - 2>();
      __syncwarp();
      issue(stage == 0 ? S - 1 : stage - 1);
      const uint32_t kb = ring_u + stage * stage_bytes(D), vb = kb + kTile * D * 2;
      const uint32_t here = live[warp][stage];
      float x[NG][4] = {};
      {
        const int key = ((lane >> 3) & 1) * 8 + (lane & 7);
        const uint32_t row_u = kb + key * (D * 2);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t k[4];
          ldmatrix_x4(row_u + (((s * 2 + (lane >> 4)) ^ (key & 7)) << 4), k[0], k[1], k[2], k[3]);
#pragma unroll
          for (int j = 0; j < NG; ++j) mma_bf16_16816(x[j], k, qf[j][s][0], qf[j][s][1]);
        }
      }
      bool raise = false;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = (lane >> 2) + (i >> 1) * 8;
          x[j][i] = (here >> key) & 1 ? x[j][i] * scale : -INFINITY;
          raise |= x[j][i] > m[j][i & 1] + kSlack;
        }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(x[j][i], x[j][i + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = fmaxf(m[j][i], top);
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
      uint32_t pf[NG][2];
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = fast_exp2(x[j][i] - finite_ref(m[j][i & 1]));
        l[j][0] += p[0] + p[2];
        l[j][1] += p[1] + p[3];
        pf[j][0] = transpose8x8(pack2(p[0], p[1]));
        pf[j][1] = transpose8x8(pack2(p[2], p[3]));
      }
      {
        const int key = (lane >> 4) * 8 + (lane & 7);
        const uint32_t row_u = vb + key * (D * 2);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t v[4];
          ldmatrix_x4_trans(row_u + (((s * 2 + ((lane >> 3) & 1)) ^ (key & 7)) << 4), v);
#pragma unroll
          for (int j = 0; j < NG; ++j) mma_bf16_16816(o[j][s], v, pf[j][0], pf[j][1]);
        }
      }
      stage = stage == S - 1 ? 0 : stage + 1;

      const bool row_end = cur.at_row_end(), last = t + 1 == t1;
      if (row_end || last) {
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 4);
            l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 8);
            l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 16);
          }
        if (row_end && began_here) {
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            float inv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              inv[i] = l[j][i] == 0.f ? 0.f : 1.f / l[j][i];
              const int head = (cur.group * NG + j) * 8 + (lane & 3) * 2 + i;
              if (a.lse && lane < 4 && head < g)
                a.lse[out_row(a, cur.row, g, head)] =
                    l[j][i] == 0.f ? -INFINITY : kLn2 * (m[j][i] + log2f(l[j][i]));
            }
            const int head = (cur.group * NG + j) * 8 + (lane >> 2);
            bf16_t* out = a.o + out_row(a, cur.row, g, head) * D + (lane & 3) * 2;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              const uint32_t y0 = transpose8x8(pack2(o[j][s][0] * inv[0], o[j][s][1] * inv[1]));
              const uint32_t y1 = transpose8x8(pack2(o[j][s][2] * inv[0], o[j][s][3] * inv[1]));
              if (head < g) {
                *reinterpret_cast<uint32_t*>(out + s * 16) = y0;
                *reinterpret_cast<uint32_t*>(out + s * 16 + 8) = y1;
              }
            }
          }
        } else {
          // a part: into the warp's own ring once nothing is in flight there any more, or
          // (the share goes on) into the workspace
          float* part = warp_part(a.ws, gw, PF);
          if (last) {
            cp_async_wait<0>();
            __syncwarp();
            part = reinterpret_cast<float*>(ring);
          }
#pragma unroll
          for (int j = 0; j < NG; ++j) {
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[((j * KS + s) * 4 + i) * 32 + lane] = o[j][s][i];
            if (lane < 4) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                part[NF * 32 + j * 8 + lane * 2 + i] = m[j][i];
                part[NF * 32 + (NG + j) * 8 + lane * 2 + i] = l[j][i];
              }
            }
          }
          if (lane == 0) {
            const int vrow = cur.row * groups + cur.group;
            if (began_here) {
              tail_part[warp] = part;
              tail_vrow[warp] = vrow;
            } else {
              head_part[warp] = part;
              head_vrow[warp] = vrow;
              head_ends[warp] = row_end;
            }
          }
        }
        if (!last) {
          cur.advance(a, rows, groups, lane);
          start();
          began_here = true;
        }
      } else {
        ++cur.tile;
      }
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  // --- join the rows that cross shares inside the block: a chain of parts comes from the
  // block before (from = -1) or begins with a warp's tail, and goes on through the next
  // warps' heads until one ends the row
  if (tid == 0) ends[blockIdx.x] = {-1, 0};
  for (int from = -1; from < kWarps; ++from) {
    const bool before = from < 0;
    if (before ? head_part[0] == nullptr : tail_part[from] == nullptr) continue;
    const float* part[kWarps + 1];
    int n = 0;
    int ended = 0;
    if (!before) part[n++] = tail_part[from];
    for (int e = from + 1; e < kWarps && head_part[e] != nullptr && !ended; ++e) {
      part[n++] = head_part[e];
      ended = head_ends[e];
    }
    const int vrow = before ? head_vrow[0] : tail_vrow[from];
    const int row = vrow / groups, group = vrow - row * groups;
    // complete here, or a part for the second kernel
    float* out = ended && !before ? nullptr : block_part(a.ws, blockIdx.x, before ? 0 : 1, PF);
    for (int i = tid; i < NF * 32; i += kThreads) {
      const int reg = i >> 5, ln = i & 31;
      const int j = reg / (KS * 4), s = reg / 4 % KS, c = reg & 3;
      const int h = j * 8 + (ln & 3) * 2 + (c & 1);
      const int dim = s * 16 + (ln >> 2) + (c >> 1) * 8;
      float top = -INFINITY, sum = 0.f, acc = 0.f;
      for (int p = 0; p < n; ++p) top = fmaxf(top, part[p][NF * 32 + h]);
      for (int p = 0; p < n; ++p) {
        const float f = fast_exp2(part[p][NF * 32 + h] - finite_ref(top));
        acc += part[p][i] * f;
        sum += part[p][NF * 32 + NG * 8 + h] * f;
      }
      if (out) {
        out[i] = acc;
        if (dim == 0) {
          out[NF * 32 + h] = top;
          out[NF * 32 + NG * 8 + h] = sum;
        }
      } else if (group * NG * 8 + h < g) {
        store_out<D>(a, out_row(a, row, g, group * NG * 8 + h), dim, acc, top, sum);
      }
    }
    if (before && ended && tid == 0) {
      const long long fw = ((head_first + 1) * warps - 1) / total;  // warp of the row's first tile
      ends[blockIdx.x] = {vrow, (int)(fw / kWarps)};
    }
  }
}

// Rows that cross blocks: block x joins the row that ends in block x of the first kernel,
// from the tail of its first block and the heads of those after.
template <int D, int NG>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(
    const __grid_constant__ AttnDecodeArgs a, int groups) {
  constexpr int KS = D / 16, PF = part_floats(D, NG), NF = frags(D, NG);
  __shared__ float weight[kMaxBlocks][NG * 8];
  __shared__ float top_s[NG * 8], sum_s[NG * 8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Ends end = static_cast<const Ends*>(a.ws)[blockIdx.x];
  if (end.vrow < 0) return;
  const int g = a.Hq / a.Hkv, n = blockIdx.x - end.first + 1;
  const int row = end.vrow / groups, group = end.vrow - row * groups;
  auto part = [&](int p) { return block_part(a.ws, end.first + p, p == 0 ? 1 : 0, PF); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int h = warp; h < NG * 8; h += 8) {
    float top = -INFINITY, sum = 0.f;
    for (int p = lane; p < n; p += 32) top = fmaxf(top, part(p)[NF * 32 + h]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int p = lane; p < n; p += 32) {
      const float f = fast_exp2(part(p)[NF * 32 + h] - finite_ref(top));
      weight[p][h] = f;
      sum += part(p)[NF * 32 + NG * 8 + h] * f;
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      top_s[h] = top;
      sum_s[h] = sum;
    }
  }
  __syncthreads();
  for (int i = blockIdx.y * 256 + threadIdx.x; i < NF * 32; i += gridDim.y * 256) {
    const int reg = i >> 5, ln = i & 31;
    const int j = reg / (KS * 4), s = reg / 4 % KS, c = reg & 3;
    const int h = j * 8 + (ln & 3) * 2 + (c & 1);
    float acc = 0.f;
#pragma unroll 4
    for (int p = 0; p < n; ++p) acc += part(p)[i] * weight[p][h];
    const float sum = sum_s[h];
    if (group * NG * 8 + h < g) {
      const int dim = s * 16 + (ln >> 2) + (c >> 1) * 8;
      store_out<D>(a, out_row(a, row, g, group * NG * 8 + h), dim, acc, top_s[h], sum);
    }
  }
}

template <int D, int NG>
cudaError_t launch(const AttnDecodeArgs& a, int rows, int groups, cudaStream_t s) {
  constexpr int smem = kWarps * kRingBytes;
  static int nsm[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!nsm[dev & 63]) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(attn_decode_kernel<D, NG>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    nsm[dev & 63] = n < kMaxBlocks ? n : kMaxBlocks;
  }
  // no more blocks than tiles could need
  const long long keys = (long long)a.max_pages * a.page_size + a.w;
  const long long most = (long long)rows * groups * ((keys + kTile - 1) / kTile);
  const long long want = (most + kWarps - 1) / kWarps;
  const int blocks = (int)(want < nsm[dev & 63] ? want : nsm[dev & 63]);
  int shift = -1;
  if ((a.page_size & (a.page_size - 1)) == 0)
    for (shift = 0; (1 << shift) < a.page_size; ++shift) {}
  count_launches(2);
  attn_decode_kernel<D, NG><<<blocks, kThreads, smem, s>>>(a, rows, groups, shift);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the join's blocks come up while the first kernel runs and wait for its results
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 2 * NG);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D, NG>, a, groups);
}

}  // namespace

size_t attn_decode_workspace_bytes(int rows, int group, int d) {
  (void)rows;
  const int ng = group <= 8 ? 1 : 2;
  return ends_bytes() + (size_t)kMaxBlocks * (kWarps + 2) * part_floats(d, ng) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t s) {
  const int rows = a.L * a.Hkv * a.B, g = a.Hq / a.Hkv;
  if (rows == 0) return cudaSuccess;
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
