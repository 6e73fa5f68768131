// What happens to the pages of a cache besides being filled and read: the accepted path of a
// draft moves together, a sequence goes on as several, and pages that no row names any more
// come free.  All three are copies of 16-byte chunks planned from lengths and tables on the
// device; no value is computed, so results are exact.
//
// Bound by latency (a chain of dependent loads: lengths -> table -> rows) until thousands of
// rows move at once, then by HBM.  Measured, a call in a graph (floor): paths of four users' drafts
// over 36 layers 2.6 to 2.9 us (0.4), of 64 users 15 (6.9); 3 forks of one sequence 7.1 (0.2), 31
// forks with rings 42 (42); pages given back with few to move 10 (0.6), with a third gone 29 (15.8).
// The pool of a whole model, 3.5 million pages of 16 tokens at d = 64, 36 layers x 8 heads x 24
// sequences: 830 us with 160 thousand pages to move (200), 1740 with a third gone (1007); every
// block counts all bits and a rank walks words one by one there.
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

// Tokens whose chunks are loaded before the first is stored: 16 in blocks of two warps, 64 users'
// drafts 14.8 us; 8 in blocks of four 15.5 (16 in blocks of four 15.6).
constexpr int kAcceptThreads = 64;
constexpr int kAcceptAhead = 16;

// A group of D / 4 lanes takes a row; a lane owns one 16-byte column of K or V and walks
// through the accepted tokens in order.  Token j moves from slot base + accept[j] to base + j,
// and accept[j] >= j grows with j, so that a store never meets a later load of its column: no
// lane waits for another.
template <int D>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ AcceptArgs a, int rows) {
  constexpr int G = D / 4;  // lanes of a row: D / 8 columns each of K and V
  static_assert(G % kAcceptAhead == 0, "lanes hold the tokens of a round");
  const int lane = threadIdx.x % G;
  const int row = blockIdx.x * (kAcceptThreads / G) + threadIdx.x / G;
  wait_for_previous();
  const bool real = row < rows;
  const int b = real ? row % p.B : 0;
  const int t0 = a.tok_start[b], t1 = a.tok_start[b + 1];
  const int n = real ? p.seq_lens[row] : 0;
  int count = real ? a.n_accept[b] : 0;
  const int m = real ? t1 - t0 : 0;  // a row that is not there has no slots to look up
  bool bad = t0 < 0 || t1 < t0 || t1 > a.N || count < 0 || count > m || n < m || n > room_of(p);
  if (!real) bad = false;
  if (bad) count = 0;
  const int base = n - m;
  // Tokens j0 .. j0 + G - 1 of the path, a lane a token: where one comes from and goes to (rows of a
  // pool that fits the GPU stay within 32 bits), -1 where it is in its place already.
  uint32_t from = 0, to = 0;
  bool moves = false;
  int longest = m;
  if (G < 32) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, G));
  const bool few = longest <= G;
  auto path = [&](int j0) {
    const int j = j0 + lane;
    moves = false;
    if (few) {  // the rows of all drafted tokens are asked for beside the path
      const int at = j < count ? a.accept[t0 + j] : -1, before = __shfl_up_sync(0xffffffffu, at, 1, G);
      const long long mine = j < m && !bad ? pool_row(p, row, base + j) : -1;
      to = (uint32_t)mine;
      from = __shfl_sync(0xffffffffu, to, at & (G - 1), G);
      const bool there = __shfl_sync(0xffffffffu, (int)(mine >= 0), at & (G - 1), G);
      if (j < count && (at >= m || at <= (j ? before : -1) || !there || mine < 0)) bad = true;
      moves = j < count && at != j;
      return;
    }
    if (j >= count) return;
    const int at = a.accept[t0 + j], before = j ? a.accept[t0 + j - 1] : -1;
    const bool good = at > before && at < m && before >= -1;
    const long long r = good ? pool_row(p, row, base + at) : -1, q = pool_row(p, row, base + j);
    if (r < 0 || q < 0) bad = true;
    from = (uint32_t)r;
    to = (uint32_t)q;
    moves = at != j;
  };
  // the whole path, before anything moves
  int most = count;
  if (G < 32) most = max(most, __shfl_xor_sync(0xffffffffu, most, G));
  for (int j0 = 0; j0 < most; j0 += G) path(j0);
  const uint32_t any = __ballot_sync(0xffffffffu, bad);
  const uint32_t mine = G == 32 ? any : any >> (threadIdx.x & 31 & ~(G - 1)) & ((1u << (G % 32)) - 1);
  if (real && lane == 0) {
    a.seq_lens_out[row] = mine ? n : base + count;
    if (mine) fault(kErrPages);
  }
  if (mine) count = 0;
  uint4* pool = reinterpret_cast<uint4*>(lane < G / 2 ? p.k_pages : p.v_pages) + lane % (G / 2);
  for (int j0 = 0; j0 < most; j0 += G) {
    if (most > G) {  // again: a longer path does not stay in the lanes
      bad = false;
      path(j0);
      moves &= !bad;  // checked above; this holds also if another stream changes tables meanwhile
    }
    if (mine) moves = false;
    for (int i0 = 0; i0 < G && j0 + i0 < most; i0 += kAcceptAhead) {
      uint4 x[kAcceptAhead];
      uint32_t at[kAcceptAhead];
      bool go[kAcceptAhead];
#pragma unroll
      for (int i = 0; i < kAcceptAhead; ++i) {
        const uint32_t r = __shfl_sync(0xffffffffu, from, i0 + i, G);
        at[i] = __shfl_sync(0xffffffffu, to, i0 + i, G);
        go[i] = __shfl_sync(0xffffffffu, (int)moves, i0 + i, G);
        if (go[i]) x[i] = pool[(size_t)r * (D / 8)];
      }
#pragma unroll
      for (int i = 0; i < kAcceptAhead; ++i)
        if (go[i]) pool[(size_t)at[i] * (D / 8)] = x[i];
    }
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
  if (!code && (long long)next + total > p.capacity) code = total > 0 ? kErrPoolFull : kErrPages;
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
constexpr int kMaxChunks = 8192;  // of the bits of a pool, counted in every block
constexpr int kReclaimSmem = (2 * kMaxChunks + 1) * sizeof(int);  // their counts and bits at most

// A bit per page that some row names, in chunks of 2^bits pages (at most kMaxChunks of them),
// behind the head.
// The head has the pages handed out so far (those that can be in use): the counter may be written
// in place while blocks still come up.
struct ReclaimHead { int code, next, pages, pad; };
__host__ __device__ inline int chunk_bits(int capacity) {
  int b = 5;
  while (((capacity - 1) >> b) >= kMaxChunks) ++b;
  return b;
}
__device__ __forceinline__ uint32_t* live_words(void* ws) {
  return reinterpret_cast<uint32_t*>(static_cast<ReclaimHead*>(ws) + 1);
}
// The pages that can be in use; the bound holds even if another stream writes the workspace
// meanwhile.
__device__ __forceinline__ int pages_of(const ReclaimHead& head, int capacity) {
  return max(0, min(head.pages, capacity));
}
__device__ __forceinline__ int chunks_of(int pages, int bits) {
  return (int)(((long long)pages + (1 << bits) - 1) >> bits);
}

__global__ void __launch_bounds__(kReclaimThreads) reclaim_clear_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ ReclaimArgs a, int bits) {
  wait_for_previous();
  let_next_start();
  const int next = a.next_page[0], pages = max(0, min(next, p.capacity));
  const long long words = (long long)chunks_of(pages, bits) << (bits - 5);
  uint4* w = reinterpret_cast<uint4*>(live_words(a.ws));
  for (long long i = (long long)blockIdx.x * kReclaimThreads + threadIdx.x; i < (words + 3) / 4;
       i += (long long)gridDim.x * kReclaimThreads)
    w[i] = make_uint4(0, 0, 0, 0);
  if (blockIdx.x == 0 && threadIdx.x == 0)
    *static_cast<ReclaimHead*>(a.ws) = {(uint32_t)next > (uint32_t)p.capacity ? kErrPages : 0, next, pages, 0};
}

__global__ void __launch_bounds__(kReclaimThreads) reclaim_mark_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ ReclaimArgs a, int rows) {
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kReclaimThreads / 32);
  wait_for_previous();
  let_next_start();
  const int pages = pages_of(*static_cast<const ReclaimHead*>(a.ws), p.capacity);
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

// The bits of the live pages with the live pages before every chunk.  A chunk is a word, kept in
// shared memory, until there are more than 262144 pages.
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
      const uint32_t x = kHoles ? ~words[w] : words[w];
      const int n = __popc(x);
      if (left >= n) { left -= n; continue; }
      int at = 0;  // the last bit with at most `left` below it that is set
#pragma unroll
      for (int o = 16; o; o >>= 1)
        if (__popc(x & ((1u << (at + o)) - 1)) <= left) at += o;
      return w * 32 + at;
    }
    return -1;  // not reached while the bits hold still
  }
};

// Live pages from n_live on go to the holes below it, in order of their ids: as few pages move
// as can, sources and targets are apart, and a page's new id is a matter of two ranks.  Every
// block counts the bits for itself (64 thousand pages: 8 KB).  A warp takes up to 32 moves, whose
// pages its lanes look up at once.
__global__ void __launch_bounds__(kReclaimThreads) reclaim_kernel(
    const __grid_constant__ PagedArgs p, const __grid_constant__ ReclaimArgs a, int rows, int bits) {
  extern __shared__ int before[];  // [chunks + 1], and the words of one-word chunks
  __shared__ int warp_sum[kReclaimThreads / 32];
  constexpr int kWarps = kReclaimThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gw = blockIdx.x * kWarps + warp, warps = gridDim.x * kWarps;
  wait_for_previous();
  const ReclaimHead head = *static_cast<const ReclaimHead*>(a.ws);
  const int pages = pages_of(head, p.capacity), chunks = chunks_of(pages, bits), code = head.code;
  const uint32_t* words = live_words(a.ws);
  if (code) {  // everything as it was
    if (blockIdx.x == 0 && tid == 0) {
      a.next_page_out[0] = head.next;
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
  // live pages of each chunk, then of those before it, for a run of chunks a thread
  uint32_t* copy = reinterpret_cast<uint32_t*>(before) + chunks + 1;
  if (bits == 5) {
    for (int c = tid; c < chunks; c += kReclaimThreads) {
      const uint32_t x = words[c];
      copy[c] = x;
      before[c] = __popc(x);
    }
    words = copy;
  } else {
    for (int c = warp; c < chunks; c += kWarps) {
      int n = 0;
      for (int w = lane; w < 1 << (bits - 5); w += 32) n += __popc(words[(c << (bits - 5)) + w]);
      n = warp_sum_int(n);
      if (lane == 0) before[c] = n;
    }
  }
  __syncthreads();
  const int run = (chunks + kReclaimThreads - 1) / kReclaimThreads;
  const int c0 = min(tid * run, chunks), c1 = min(c0 + run, chunks);
  int mine = 0;
  for (int c = c0; c < c1; ++c) mine += before[c];
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int n_live = 0, earlier = incl - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) earlier += warp_sum[w];
    n_live += warp_sum[w];
  }
  for (int c = c0; c < c1; ++c) {
    const int n = before[c];
    before[c] = earlier;
    earlier += n;
  }
  if (tid == 0) before[chunks] = n_live;
  __syncthreads();
  const Live live{words, before, bits, chunks};
  const int below = n_live < pages ? live.rank(n_live) : n_live;  // live pages that stay
  const int moving = n_live - below;
  if (blockIdx.x == 0 && tid == 0) a.next_page_out[0] = n_live;

  const int chunks16 = p.page_size * (p.d / 8);  // 16-byte chunks of a page of K
  const int pieces = (chunks16 + 255) / 256;
  uint4* k = reinterpret_cast<uint4*>(p.k_pages);
  uint4* v = reinterpret_cast<uint4*>(p.v_pages);
  const long long moves = (long long)moving * pieces;
  const int per = (int)max(1ll, min(32ll, (moves + warps - 1) / warps));
  for (long long i0 = (long long)gw * per; i0 < moves; i0 += (long long)warps * per) {
    const int count = (int)min((long long)per, moves - i0);
    int from_of = -1, to_of = -1, part_of = 0;
    if (lane < count) {
      const int s = (int)((i0 + lane) / pieces);
      part_of = (int)(i0 + lane - (long long)s * pieces);
      from_of = live.select<false>(below + s);
      to_of = live.select<true>(s);
    }
    for (int i = 0; i < count; ++i) {
      const int from = __shfl_sync(0xffffffffu, from_of, i), to = __shfl_sync(0xffffffffu, to_of, i);
      const int first = __shfl_sync(0xffffffffu, part_of, i) * 256 + lane;
      if (from < n_live || from >= pages || (uint32_t)to >= (uint32_t)min(n_live, pages)) continue;
      const size_t src_at = (size_t)from * chunks16, dst_at = (size_t)to * chunks16;
      uint4 x[8], y[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int c = first + u * 32;
        if (c < chunks16) {
          x[u] = k[src_at + c];
          y[u] = v[src_at + c];
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int c = first + u * 32;
        if (c < chunks16) {
          k[dst_at + c] = x[u];
          v[dst_at + c] = y[u];
        }
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
  return sizeof(ReclaimHead) + ((chunks << (b - 3)) + 15) / 16 * 16;
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
  // the same limit whatever this call needs, since another thread may launch for another pool, and
  // before anything is enqueued
  cudaError_t e = cudaFuncSetAttribute(reclaim_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kReclaimSmem);
  if (e != cudaSuccess) return e;
  count_launches(3);
  Launch c(dim3(clear < 152 ? clear : 152), kReclaimThreads, s);
  e = cudaLaunchKernelEx(&c.cfg, reclaim_clear_kernel, p, a, bits);
  if (e != cudaSuccess) return e;
  const int mark = (rows + kReclaimThreads / 32 - 1) / (kReclaimThreads / 32);
  Launch m(dim3(mark < 152 * 8 ? mark : 152 * 8), kReclaimThreads, s);
  e = cudaLaunchKernelEx(&m.cfg, reclaim_mark_kernel, p, a, rows);
  if (e != cudaSuccess) return e;
  Launch r(dim3(152 * 2), kReclaimThreads, s);
  const int chunks = ((p.capacity - 1) >> bits) + 1;
  r.cfg.dynamicSmemBytes = (chunks + 1 + (bits == 5 ? chunks : 0)) * sizeof(int);
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
