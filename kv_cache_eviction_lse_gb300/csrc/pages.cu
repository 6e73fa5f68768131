// What happens to the pages of a cache besides being filled and read: the accepted path of a
// draft moves together, a sequence goes on as several, and pages that no row names any more
// come free.  All three are copies of 16-byte chunks planned from lengths and tables on the
// device; no value is computed, so results are exact.
//
// Bound by latency (a chain of dependent loads: lengths -> table -> rows) until thousands of
// rows move at once, then by HBM.
#include "common.cuh"
#include "launch.cuh"
#include "pages.cuh"

namespace kvs {

__device__ int g_pages_error = 0;

namespace {

constexpr int kErrPoolFull = 4;  // as kvs_decode_step and kvs_append_paged
constexpr int kErrPages = 11;    // a token start, path, fork, length or page id out of range

__device__ __forceinline__ void fault(int code) { atomicCAS(&g_pages_error, 0, code); }

// Slots of a row: what its table has room for, within 32 bits.
__device__ __forceinline__ long long room_of(const PagedArgs& p) {
  return min((long long)p.max_pages * p.page_size, (long long)INT32_MAX - 8192);
}

// Row in the pool of a slot of a row, or -1 where the page id is bad.
__device__ __forceinline__ long long pool_row(const PagedArgs& p, int row, int slot) {
  const int idx = slot / p.page_size;
  const int page = p.block_table[(size_t)row * p.max_pages + idx];
  if ((uint32_t)page >= (uint32_t)p.capacity) return -1;
  return (long long)page * p.page_size + (slot - idx * p.page_size);
}

// ----------------------------------------------------------------------------- accept

constexpr int kAcceptThreads = 128;
constexpr int kAcceptAhead = 8;  // tokens whose chunks are loaded before the first is stored

// A group of D / 4 lanes takes a row; a lane owns one 16-byte column of K or V and walks
// through the accepted tokens in order.  Token j moves from slot base + accept[j] to base + j,
// and accept[j] >= j grows with j, so that a store never meets a later load of its column: no
// lane waits for another.
template <int D>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ AcceptArgs a, int rows) {
  constexpr int G = D / 4;  // lanes of a row: D / 8 columns each of K and V
  const int lane = threadIdx.x % G;
  const int row = blockIdx.x * (kAcceptThreads / G) + threadIdx.x / G;
  wait_for_previous();
  const bool real = row < rows;
  const int b = real ? row % p.B : 0;
  const int t0 = a.tok_start[b], t1 = a.tok_start[b + 1];
  const int n = real ? p.seq_lens[row] : 0;
  int count = real ? a.n_accept[b] : 0;
  const int m = t1 - t0;
  bool bad = t0 < 0 || t1 < t0 || t1 > a.N || count < 0 || count > m || n < m || n > room_of(p);
  if (!real) bad = false;
  if (bad) count = 0;
  const int base = n - m;
  // the whole path, before anything moves
  int most = count;
  if (G < 32) most = max(most, __shfl_xor_sync(0xffffffffu, most, G));
  for (int j0 = 0; j0 < most; j0 += G) {
    const int j = j0 + lane;
    if (j >= count) continue;
    const int at = a.accept[t0 + j], before = j ? a.accept[t0 + j - 1] : -1;
    if (at <= before || at >= m || before < -1) bad = true;
    else if (pool_row(p, row, base + at) < 0 || pool_row(p, row, base + j) < 0) bad = true;
  }
  const uint32_t any = __ballot_sync(0xffffffffu, bad);
  const uint32_t mine = G == 32 ? any : any >> (threadIdx.x & 31 & ~(G - 1)) & ((1u << (G % 32)) - 1);
  if (real && lane == 0) {
    a.seq_lens_out[row] = mine ? n : base + count;
    if (mine) fault(kErrPages);
  }
  if (!real || mine) return;
  uint4* pool = reinterpret_cast<uint4*>(lane < G / 2 ? p.k_pages : p.v_pages) + lane % (G / 2);
  for (int j0 = 0; j0 < count; j0 += kAcceptAhead) {
    uint4 x[kAcceptAhead];
    long long to[kAcceptAhead];
#pragma unroll
    for (int i = 0; i < kAcceptAhead; ++i) {
      to[i] = -1;
      if (j0 + i >= count) continue;
      const int at = a.accept[t0 + j0 + i];
      if (at == j0 + i) continue;  // in its place already
      // checked above; this holds also if another stream changes tables meanwhile
      const long long from = pool_row(p, row, min(base + max(at, 0), n - 1));
      to[i] = pool_row(p, row, base + j0 + i);
      if (from < 0) to[i] = -1;
      if (to[i] >= 0) x[i] = pool[from * (D / 8)];
    }
#pragma unroll
    for (int i = 0; i < kAcceptAhead; ++i)
      if (to[i] >= 0) pool[to[i] * (D / 8)] = x[i];
  }
}

// ----------------------------------------------------------------------------- fork

constexpr int kForkPlanThreads = 1024;
constexpr int kForkThreads = 128;
constexpr int kForkPlanBlocks = kForkThreads;
constexpr int kRingStep = 4;  // 16-byte chunks of K, and of V, that a thread of a ring copies

// The plan of the forks in the workspace: the page counter before them, what each block of rows
// found, and per forked row how many new pages the rows before it in its block take.  Forked
// row r = (l * Hkv + hk) * forks + i.
struct ForkBlock { int pages, code; };
struct ForkPlan {
  int* next;
  ForkBlock* blocks;
  int* before;
  __device__ explicit ForkPlan(void* ws)
      : next(static_cast<int*>(ws)), blocks(reinterpret_cast<ForkBlock*>(next + 4)),
        before(reinterpret_cast<int*>(blocks + kForkPlanBlocks)) {}
};

__device__ __forceinline__ int source_of(const PagedArgs& p, const ForkArgs& a, int r) {
  const int b = a.src[r % a.forks];
  return (uint32_t)b < (uint32_t)p.B ? r / a.forks * p.B + b : -1;
}

__global__ void __launch_bounds__(kForkPlanThreads) fork_plan_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ ForkArgs a, int rows, int per) {
  extern __shared__ uint32_t seen[];  // block 0: a bit per sequence that is a target
  __shared__ int sums[32];
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_previous();
  let_next_start();
  if (tid == 0) err = 0;
  if (blockIdx.x == 0)
    for (int i = tid; i < (p.B + 31) / 32; i += kForkPlanThreads) seen[i] = 0;
  __syncthreads();
  const ForkPlan plan(a.plan);
  if (blockIdx.x == 0) {
    if (tid == 0) {
      plan.next[0] = a.next_page[0];
      if (plan.next[0] < 0) err = kErrPages;
    }
    for (int i = tid; i < a.forks; i += kForkPlanThreads) {
      const int t = a.dst[i];
      if ((uint32_t)t >= (uint32_t)p.B || (atomicOr(&seen[t >> 5], 1u << (t & 31)) >> (t & 31) & 1))
        err = kErrPages;  // out of range, or the target of two forks
    }
    __syncthreads();
    for (int i = tid; i < a.forks; i += kForkPlanThreads) {
      const int t = a.src[i];
      if ((uint32_t)t >= (uint32_t)p.B || (seen[t >> 5] >> (t & 31) & 1)) err = kErrPages;
    }
  }
  const long long lo = ((long long)blockIdx.x * kForkPlanThreads + tid) * per;
  const int r0 = (int)min(lo, (long long)rows), r1 = (int)min(lo + per, (long long)rows);
  int mine = 0;
  for (int r = r0; r < r1; ++r) {
    plan.before[r] = mine;
    const int from = source_of(p, a, r);
    const int n = from < 0 ? 0 : p.seq_lens[from];
    if (n < 0 || n > room_of(p)) err = kErrPages;
    else if (n % p.page_size) ++mine;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int earlier = incl - mine;
  for (int w = 0; w < warp; ++w) earlier += sums[w];
  for (int r = r0; r < r1; ++r) plan.before[r] += earlier;
  if (tid == kForkPlanThreads - 1) plan.blocks[blockIdx.x] = {earlier + mine, err};
}

// Blocks 0 .. row_blocks - 1 take a forked row a warp: its table, length and last page.  The
// blocks behind them take a piece of a forked row's ring each.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ ForkArgs a, int rows,
    int plan_blocks, int plan_shift, int row_blocks, int pieces) {
  __shared__ int base[kForkPlanBlocks];
  __shared__ int warp_sum[kForkThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_previous();
  const ForkPlan plan(a.plan);
  const int next = plan.next[0];
  ForkBlock mine = {0, 0};
  if (tid < plan_blocks) mine = plan.blocks[tid];
  int incl = mine.pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  int code = __syncthreads_or(mine.code) ? kErrPages : 0;
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kForkThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  base[tid] = next + before + incl - mine.pages;
  __syncthreads();
  if (!code && total > 0 && (long long)next + total > p.capacity) code = kErrPoolFull;
  if (blockIdx.x == 0 && tid == 0) {
    a.next_page_out[0] = next + (code ? 0 : total);
    if (code) fault(code);
  }
  if (code) return;
  if ((int)blockIdx.x >= row_blocks) {  // a piece of a ring
    const int r = (blockIdx.x - row_blocks) / pieces, piece = (blockIdx.x - row_blocks) % pieces;
    const int from = source_of(p, a, r), target = a.dst[r % a.forks];
    if (from < 0 || (uint32_t)target >= (uint32_t)p.B) return;
    const int to = r / a.forks * p.B + target;
    const int chunks = a.w * (p.d / 8);
    const size_t src_at = (size_t)from * chunks, dst_at = (size_t)to * chunks;
    uint4* k = reinterpret_cast<uint4*>(a.ring_k);
    uint4* v = reinterpret_cast<uint4*>(a.ring_v);
    const int c0 = piece * (kForkThreads * kRingStep) + tid;
    uint4 x[kRingStep], y[kRingStep];
#pragma unroll
    for (int i = 0; i < kRingStep; ++i) {
      const int c = c0 + i * kForkThreads;
      if (c < chunks) {
        x[i] = k[src_at + c];
        y[i] = v[src_at + c];
      }
    }
#pragma unroll
    for (int i = 0; i < kRingStep; ++i) {
      const int c = c0 + i * kForkThreads;
      if (c < chunks) {
        k[dst_at + c] = x[i];
        v[dst_at + c] = y[i];
      }
    }
    if (piece == 0) {
      for (int i = tid; i < a.w; i += kForkThreads)
        a.ring_score[(size_t)to * a.w + i] = a.ring_score[(size_t)from * a.w + i];
      if (r < a.forks && tid == 0) a.pos[target] = a.pos[from];  // (l, hk) = (0, 0): the sequence
    }
    return;
  }
  const int r = blockIdx.x * (kForkThreads / 32) + warp;
  if (r >= rows) return;
  const int from = source_of(p, a, r), target = a.dst[r % a.forks];
  if (from < 0 || (uint32_t)target >= (uint32_t)p.B) return;
  const int to = r / a.forks * p.B + target;
  const int n = p.seq_lens[from], full = n / p.page_size, rest = n - full * p.page_size;
  if (n < 0 || n > room_of(p)) return;
  const int page = base[r >> plan_shift] + plan.before[r];
  const int* in = p.block_table + (size_t)from * p.max_pages;
  int* out = a.block_table + (size_t)to * p.max_pages;
  if (lane == 0) a.seq_lens[to] = n;
  if (rest) {  // its own copy of the page that it goes on in
    const int old = in[full];
    const bool there = (uint32_t)old < (uint32_t)p.capacity;
    if (!there && lane == 0) fault(kErrPages);
    const int chunks = p.page_size * (p.d / 8), used = there ? rest * (p.d / 8) : 0;
    if ((uint32_t)page < (uint32_t)p.capacity) {
      const size_t src_at = there ? (size_t)old * chunks : 0, dst_at = (size_t)page * chunks;
      uint4* k = reinterpret_cast<uint4*>(p.k_pages);
      uint4* v = reinterpret_cast<uint4*>(p.v_pages);
      for (int c0 = 0; c0 < chunks; c0 += 32 * 8) {
        uint4 x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = c0 + i * 32 + lane;
          x[i] = y[i] = make_uint4(0, 0, 0, 0);
          if (c < used) {
            x[i] = k[src_at + c];
            y[i] = v[src_at + c];
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = c0 + i * 32 + lane;
          if (c < chunks) {
            k[dst_at + c] = x[i];
            v[dst_at + c] = y[i];
          }
        }
      }
    }
  }
  for (int i = lane; i < p.max_pages; i += 32)
    out[i] = i < full ? in[i] : i == full && rest ? page : -1;
}

// ----------------------------------------------------------------------------- reclaim

constexpr int kReclaimThreads = 256;
constexpr int kMaxChunks = 2048;  // of the bits of a pool, counted in every block

// A bit per page that some row names, in chunks of 2^bits pages (at most kMaxChunks of them),
// behind the head.
struct ReclaimHead { int code, pad[3]; };
__host__ __device__ inline int chunk_bits(int capacity) {
  int b = 10;
  while (((capacity - 1) >> b) >= kMaxChunks) ++b;
  return b;
}
__device__ __forceinline__ uint32_t* live_words(void* ws) {
  return reinterpret_cast<uint32_t*>(static_cast<ReclaimHead*>(ws) + 1);
}
// Pages handed out so far: those that can be in use.
__device__ __forceinline__ int handed_out(const PagedArgs& p, const ReclaimArgs& a) {
  return max(0, min(a.next_page[0], p.capacity));
}
__device__ __forceinline__ int chunks_of(int pages, int bits) {
  return (int)(((long long)pages + (1 << bits) - 1) >> bits);
}

__global__ void __launch_bounds__(kReclaimThreads) reclaim_clear_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ ReclaimArgs a, int bits) {
  wait_for_previous();
  let_next_start();
  const long long words = (long long)chunks_of(handed_out(p, a), bits) << (bits - 5);
  uint4* w = reinterpret_cast<uint4*>(live_words(a.ws));
  for (long long i = (long long)blockIdx.x * kReclaimThreads + threadIdx.x; i < words / 4;
       i += (long long)gridDim.x * kReclaimThreads)
    w[i] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x == 0 && threadIdx.x == 0)
    static_cast<ReclaimHead*>(a.ws)->code = (uint32_t)a.next_page[0] > (uint32_t)p.capacity ? kErrPages : 0;
}

__global__ void __launch_bounds__(kReclaimThreads) reclaim_mark_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ ReclaimArgs a, int rows) {
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kReclaimThreads / 32);
  wait_for_previous();
  let_next_start();
  const int pages = handed_out(p, a);
  uint32_t* live = live_words(a.ws);
  bool bad = false;
  for (int row = blockIdx.x * (kReclaimThreads / 32) + (threadIdx.x >> 5); row < rows; row += warps) {
    const int n = p.seq_lens[row];
    if (n < 0 || n > room_of(p)) { bad = true; continue; }
    const int need = n / p.page_size + (n % p.page_size != 0);
    for (int i = lane; i < need; i += 32) {
      const int id = p.block_table[(size_t)row * p.max_pages + i];
      if ((uint32_t)id >= (uint32_t)pages) bad = true;
      else atomicOr(&live[id >> 5], 1u << (id & 31));
    }
  }
  if (bad) atomicMax(&static_cast<ReclaimHead*>(a.ws)->code, kErrPages);
}

// The bits of the live pages with the live pages before every chunk.
struct Live {
  const uint32_t* words;
  const int* before;  // [chunks + 1]
  int bits, chunks;

  __device__ __forceinline__ int rank(int id) const {  // live pages below id
    const int c = id >> bits, w0 = c << (bits - 5), w1 = id >> 5;
    int n = before[c];
    for (int w = w0; w < w1; ++w) n += __popc(words[w]);
    if (id & 31) n += __popc(words[w1] & ((1u << (id & 31)) - 1));
    return n;
  }
  // the s-th live page (or hole), of those below what the chunks cover
  template <bool kHoles>
  __device__ __forceinline__ int select(int s) const {
    int lo = 0, hi = chunks;  // the last chunk with at most s before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((kHoles ? (mid << bits) - before[mid] : before[mid]) <= s) lo = mid; else hi = mid;
    }
    int left = s - (kHoles ? (lo << bits) - before[lo] : before[lo]);
    const int w0 = lo << (bits - 5), w1 = (lo + 1) << (bits - 5);
    for (int w = w0; w < w1; ++w) {
      uint32_t x = kHoles ? ~words[w] : words[w];
      const int n = __popc(x);
      if (left >= n) { left -= n; continue; }
      for (; left > 0; --left) x &= x - 1;
      return w * 32 + __ffs(x) - 1;
    }
    return -1;  // not reached while the bits hold still
  }
};

// Live pages from n_live on go to the holes below it, in order of their ids: as few pages move
// as can, sources and targets are apart, and a page's new id is a matter of two ranks.  Every
// block counts the bits for itself (64 thousand pages: 8 KB).
__global__ void __launch_bounds__(kReclaimThreads) reclaim_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ ReclaimArgs a, int rows, int bits) {
  __shared__ int before[kMaxChunks + 1];
  __shared__ int warp_sum[kReclaimThreads / 32];
  constexpr int kWarps = kReclaimThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gw = blockIdx.x * kWarps + warp, warps = gridDim.x * kWarps;
  wait_for_previous();
  const int pages = handed_out(p, a), chunks = chunks_of(pages, bits);
  const uint32_t* words = live_words(a.ws);
  const int code = static_cast<const ReclaimHead*>(a.ws)->code;
  if (code) {  // everything as it was
    if (blockIdx.x == 0 && tid == 0) {
      a.next_page_out[0] = a.next_page[0];
      fault(code);
    }
    if (a.block_table_out != p.block_table) {
      const long long all = (long long)rows * p.max_pages;
      for (long long i = (long long)blockIdx.x * kReclaimThreads + tid; i < all;
           i += (long long)gridDim.x * kReclaimThreads)
        a.block_table_out[i] = p.block_table[i];
    }
    return;
  }
  // live pages of each chunk, then of those before it
  for (int c = warp; c < chunks; c += kWarps) {
    int n = 0;
    for (int w = lane; w < 1 << (bits - 5); w += 32) n += __popc(words[(c << (bits - 5)) + w]);
    n = warp_sum_int(n);
    if (lane == 0) before[c + 1] = n;
  }
  if (tid == 0) before[0] = 0;
  __syncthreads();
  int carry = 0;
  for (int c0 = 0; c0 < chunks; c0 += kReclaimThreads) {
    const int c = c0 + tid;
    int incl = c < chunks ? before[c + 1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += warp_sum[w];
      all += warp_sum[w];
    }
    if (c < chunks) before[c + 1] = carry + incl;
    carry += all;
    __syncthreads();
  }
  const Live live{words, before, bits, chunks};
  const int n_live = carry;
  const int below = n_live < pages ? live.rank(n_live) : n_live;  // live pages that stay
  const int moving = n_live - below;
  if (blockIdx.x == 0 && tid == 0) a.next_page_out[0] = n_live;

  const int chunks16 = p.page_size * (p.d / 8);  // 16-byte chunks of a page of K
  const int pieces = (chunks16 + 255) / 256;
  uint4* k = reinterpret_cast<uint4*>(p.k_pages);
  uint4* v = reinterpret_cast<uint4*>(p.v_pages);
  for (long long i = gw; i < (long long)moving * pieces; i += warps) {
    const int s = (int)(i / pieces), c0 = (int)(i - (long long)s * pieces) * 256 + lane;
    const int from = live.select<false>(below + s), to = live.select<true>(s);
    if (from < n_live || from >= pages || (uint32_t)to >= (uint32_t)n_live) continue;
    const size_t src_at = (size_t)from * chunks16, dst_at = (size_t)to * chunks16;
    uint4 x[8], y[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = c0 + u * 32;
      if (c < chunks16) {
        x[u] = k[src_at + c];
        y[u] = v[src_at + c];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = c0 + u * 32;
      if (c < chunks16) {
        k[dst_at + c] = x[u];
        v[dst_at + c] = y[u];
      }
    }
  }
  for (int row = gw; row < rows; row += warps) {
    const int n = p.seq_lens[row], need = n / p.page_size + (n % p.page_size != 0);
    const size_t at = (size_t)row * p.max_pages;
    for (int i = lane; i < p.max_pages; i += 32) {
      int id = -1;
      if (i < need) {
        id = p.block_table[at + i];
        if (id >= n_live && id < pages) id = live.select<true>(live.rank(id) - below);
      }
      a.block_table_out[at + i] = id;
    }
  }
}

}  // namespace

size_t fork_workspace_bytes(int rows) {
  return 16 + kForkPlanBlocks * sizeof(ForkBlock) + ((size_t)rows * 4 + 15) / 16 * 16;
}

size_t reclaim_workspace_bytes(int capacity) {
  const int b = chunk_bits(capacity > 0 ? capacity : 1);
  const size_t chunks = ((size_t)capacity + ((size_t)1 << b) - 1) >> b;
  return sizeof(ReclaimHead) + (chunks << (b - 3));
}

cudaError_t launch_accept(const PagedArgs& p, const AcceptArgs& a, cudaStream_t s) {
  const int rows = p.L * p.Hkv * p.B, per_block = kAcceptThreads / (p.d / 4);
  Launch l(dim3((rows + per_block - 1) / per_block), kAcceptThreads, s);
  count_launches(1);
  return p.d == 128 ? cudaLaunchKernelEx(&l.cfg, accept_kernel<128>, p, a, rows)
                    : cudaLaunchKernelEx(&l.cfg, accept_kernel<64>, p, a, rows);
}

cudaError_t launch_fork(const PagedArgs& p, const ForkArgs& a, cudaStream_t s) {
  const int rows = p.L * p.Hkv * a.forks;
  int plan_shift = 10;  // rows of a plan block: its threads times a power of two
  static_assert(kForkPlanThreads == 1 << 10, "a row a thread at least");
  while (((rows - 1) >> plan_shift) >= kForkPlanBlocks) ++plan_shift;
  const int plan_blocks = ((rows - 1) >> plan_shift) + 1, per = 1 << (plan_shift - 10);
  Launch plan(dim3(plan_blocks), kForkPlanThreads, s);
  plan.cfg.dynamicSmemBytes = (p.B + 31) / 32 * 4;
  count_launches(2);
  cudaError_t e = cudaLaunchKernelEx(&plan.cfg, fork_plan_kernel, p, a, rows, per);
  if (e != cudaSuccess) return e;
  const int row_blocks = (rows + kForkThreads / 32 - 1) / (kForkThreads / 32);
  const int pieces = (a.w * (p.d / 8) + kForkThreads * kRingStep - 1) / (kForkThreads * kRingStep);
  Launch copy(dim3((unsigned)(row_blocks + (long long)rows * pieces)), kForkThreads, s);
  return cudaLaunchKernelEx(&copy.cfg, fork_kernel, p, a, rows, plan_blocks, plan_shift, row_blocks,
                            pieces);
}

cudaError_t launch_reclaim(const PagedArgs& p, const ReclaimArgs& a, cudaStream_t s) {
  const int rows = p.L * p.Hkv * p.B, bits = chunk_bits(p.capacity);
  const size_t quads = reclaim_workspace_bytes(p.capacity) / 16;
  const int clear = (int)((quads + kReclaimThreads - 1) / kReclaimThreads);
  count_launches(3);
  Launch c(dim3(clear < 152 ? clear : 152), kReclaimThreads, s);
  cudaError_t e = cudaLaunchKernelEx(&c.cfg, reclaim_clear_kernel, p, a, bits);
  if (e != cudaSuccess) return e;
  const int mark = (rows + kReclaimThreads / 32 - 1) / (kReclaimThreads / 32);
  Launch m(dim3(mark < 152 * 8 ? mark : 152 * 8), kReclaimThreads, s);
  e = cudaLaunchKernelEx(&m.cfg, reclaim_mark_kernel, p, a, rows);
  if (e != cudaSuccess) return e;
  Launch r(dim3(152 * 3), kReclaimThreads, s);
  return cudaLaunchKernelEx(&r.cfg, reclaim_kernel, p, a, rows, bits);
}

cudaError_t pages_device_error(int* code, bool clear, cudaStream_t s) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(code, g_pages_error, sizeof(int), 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && clear && *code) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_pages_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

}  // namespace kvs
