// Position rotation of queries and keys, and the append of new tokens to the paged cache
// with the rotation on the way.
//
// A pair (a, b) of dimensions of a token at position p turns by the angle p f:
//   (a cos - b sin, b cos + a sin).
// f is kept as turns per position in a 64-bit binary fraction, so p f mod 1 is one integer
// product that wraps where the angle does and needs no range reduction (a 32-bit product would
// be off by 0.01 rad at position 131072).  The fraction comes from one product of doubles, with
// 1 / (2 pi) rounded to one: the turns are off by 2^-52 of themselves at most, the angle of a frequency
// up to 1 by p 2^-55 turns.  In [-pi, pi] the hardware's sine and cosine are good to 2^-21, far
// below the bf16 rounding of the result (2^-8 relative); sincospif took a tenth longer where
// a thread has one head (2079 tokens of 14 heads 6.5 against 5.9 us).  The products are
// fp32, and each result is rounded to bf16 once.
//
// Bound by HBM (or, for a few tokens, by latency): every row is read and written once, and
// a thread that has the cosines and sines of its token's 8 pairs reuses them for the heads
// and layers it walks through.  A 16384-token prompt of 2 layers takes 98 us (671 MB, 6.8
// TB/s, the rate of a copy).
#include "common.cuh"
#include "launch.cuh"
#include "rope.cuh"

namespace kvs {

__device__ int g_append_error = 0;

namespace {

constexpr int kErrPoolFull = 4;   // as kvs_decode_step
constexpr int kErrTableFull = 5;
constexpr int kErrAppend = 8;     // token starts, lengths or page ids out of range

constexpr int kThreads = 128;
constexpr int kPlanThreads = 1024;

// The plan of an append in the workspace: the page counter before it, what each block of
// rows found (pages to take, error code), and per row its length and the pages that the rows
// before it in its block take.
constexpr int kPlanBlocks = 128;
struct PlanHead { int next, pad[3]; };
struct PlanBlock { long long pages; int code; };
struct PlanView {
  PlanHead* head;
  PlanBlock* blocks;
  int2* rows;
  __device__ explicit PlanView(void* ws)
      : head(static_cast<PlanHead*>(ws)), blocks(reinterpret_cast<PlanBlock*>(head + 1)),
        rows(reinterpret_cast<int2*>(blocks + kPlanBlocks)) {}
};

__device__ __forceinline__ int tokens_of(const AppendArgs& a, int b) {
  return a.tok_start ? a.tok_start[b + 1] - a.tok_start[b] : 1;
}

__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x);
  x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z);
  x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// One row (head of a token) takes D / 16 threads of two 16-byte chunks each.  Thread u of a
// row rotates pairs 8u .. 8u+7: chunks u and u + rot/16 when the halves pair up, chunks 2u
// and 2u + 1 when neighbours do.  Past the rotated part it copies chunks 2u and 2u + 1.
struct Lane {
  int c0, c1;
  bool rotate;
};

__device__ __forceinline__ Lane lane_of(int u, int rot_dim, int interleaved) {
  Lane l;
  l.rotate = u < rot_dim / 16;
  const bool halves = l.rotate && !interleaved;
  l.c0 = halves ? u : 2 * u;
  l.c1 = halves ? u + rot_dim / 16 : 2 * u + 1;
  return l;
}

__device__ __forceinline__ void angles(const RopeArgs& r, int u, int pos, float* c, float* s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t phase = (uint64_t)(int64_t)pos * r.freq[8 * u + i];
    const float x = (float)(int32_t)(phase >> 32) * (3.14159265358979324f * 0x1p-31f);
    c[i] = __cosf(x);
    s[i] = __sinf(x);
  }
}

__device__ __forceinline__ void rotate(uint4& x0, uint4& x1, const float* c, const float* s,
                                       int interleaved) {
  float a[8], b[8], y0[8], y1[8];
  unpack8(x0, a);
  unpack8(x1, b);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y0[2 * i] = a[2 * i] * c[i] - a[2 * i + 1] * s[i];
      y0[2 * i + 1] = a[2 * i + 1] * c[i] + a[2 * i] * s[i];
      y1[2 * i] = b[2 * i] * c[4 + i] - b[2 * i + 1] * s[4 + i];
      y1[2 * i + 1] = b[2 * i + 1] * c[4 + i] + b[2 * i] * s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y0[i] = a[i] * c[i] - b[i] * s[i];
      y1[i] = b[i] * c[i] + a[i] * s[i];
    }
  }
  x0 = pack8(y0);
  x1 = pack8(y1);
}

template <int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs r) {
  constexpr int kPer = D / 16;
  const int u = threadIdx.x % kPer;
  const int t = blockIdx.x * (kThreads / kPer) + threadIdx.x / kPer;
  if (t >= r.N) return;
  const Lane ln = lane_of(u, r.rot_dim, r.interleaved);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // started beside the kernel before
  float c[8], s[8];
  if (ln.rotate) angles(r, u, r.pos[t], c, s);
  const int n_q = r.q ? r.L * r.Hq : 0, n_all = n_q + (r.k ? r.L * r.Hkv : 0);
  auto row_at = [&](int slab) {
    return ((size_t)(slab < n_q ? slab : slab - n_q) * r.N + t) * D;
  };
  uint4 x0, x1;
  auto load = [&](int slab) {
    const uint4* in = reinterpret_cast<const uint4*>((slab < n_q ? r.q : r.k) + row_at(slab));
    x0 = in[ln.c0];
    x1 = in[ln.c1];
  };
  int slab = blockIdx.y;
  if (slab < n_all) load(slab);
  while (slab < n_all) {
    const int at = slab;
    uint4 y0 = x0, y1 = x1;
    slab += gridDim.y;
    if (slab < n_all) load(slab);
    if (ln.rotate) rotate(y0, y1, c, s, r.interleaved);
    uint4* out = reinterpret_cast<uint4*>((at < n_q ? r.q_out : r.k_out) + row_at(at));
    out[ln.c0] = y0;
    out[ln.c1] = y1;
  }
}

// The plan, by up to kPlanBlocks blocks of rows: what every row has and how many new pages the
// rows before it in its block take.  Whether the whole append fits is known when all blocks
// are done; the append's blocks put that together from their records (see decide).
__global__ void __launch_bounds__(kPlanThreads, 1) append_plan_kernel(const AppendArgs a, int rows,
                                                                      int N, int per) {
  __shared__ long long sums[32];
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // started beside the end of the kernel before; the append must not start beside that too
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) err = 0;
  __syncthreads();
  auto fault = [&](int code) { atomicMax(&err, code); };
  const PlanView plan(a.plan);
  if (blockIdx.x == 0 && tid == 0) {
    const int next = a.next_page[0];
    plan.head->next = next;
    if (next < 0) fault(kErrAppend);
    if (a.tok_start && (a.tok_start[0] != 0 || a.tok_start[a.B] > N)) fault(kErrAppend);
  }
  const int ps = a.page_size;
  // slots and page counts stay within 32 bits
  const long long room = min((long long)a.max_pages * ps, (long long)INT32_MAX - 8192);
  const long long lo = ((long long)blockIdx.x * kPlanThreads + tid) * per;
  const int r0 = (int)min(lo, (long long)rows), r1 = (int)min(lo + per, (long long)rows);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = a.seq_lens[r], b = r % a.B;
    const int from = a.tok_start ? a.tok_start[b] : 0, to = a.tok_start ? a.tok_start[b + 1] : 1;
    plan.rows[r] = {n, (int)mine};
    if (n < 0 || n > room || from < 0 || to < from) { fault(kErrAppend); continue; }
    const int m = to - from;
    if (m == 0) continue;
    if (n + (long long)m > room) { fault(kErrTableFull); continue; }
    if (n % ps) {
      const int pg = a.block_table[(size_t)r * a.max_pages + n / ps];
      if (pg < 0 || pg >= a.capacity) fault(kErrAppend);
    }
    mine += (n + (long long)m + ps - 1) / ps - (n + ps - 1) / ps;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  long long others = sums[lane];  // of the warps; every warp for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, others, o);
    if (lane >= o) others += y;
  }
  const long long warps_before = __shfl_sync(0xffffffffu, others, warp ? warp - 1 : 0);
  const int before = (int)(incl - mine + (warp ? warps_before : 0));
  for (int r = r0; r < r1; ++r) plan.rows[r].y += before;
  if (tid == 31) plan.blocks[blockIdx.x] = {others, err};
}

// What an append's block knows of the whole plan: a code (0 = append), the pages that it takes
// and, per plan block, the first new page of its rows.
struct Decision {
  int code;
  long long total;
};

// Called by all threads of a block, after the plan; base [kPlanBlocks] in shared memory.
__device__ __forceinline__ Decision decide(const AppendArgs& a, const PlanView& plan, int blocks,
                                           int* base) {
  const int next = plan.head->next;
  if (blocks == 1) {
    const PlanBlock b = plan.blocks[0];
    base[0] = next;  // the same by every thread, so that none waits for another
    const bool fits = b.pages == 0 || next + b.pages <= a.capacity;
    return {b.code ? b.code : fits ? 0 : kErrPoolFull, b.pages};
  }
  __shared__ long long sums[kThreads / 32];
  __shared__ int code_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  PlanBlock mine = {0, 0};
  if (tid < blocks) mine = plan.blocks[tid];
  long long incl = mine.pages;
  int code = mine.code;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  code = __reduce_max_sync(0xffffffffu, code);
  if (tid == 0) code_s = 0;
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (lane == 0 && code) atomicMax(&code_s, code);
  long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  static_assert(kPlanBlocks == kThreads, "a thread per plan block");
  base[tid] = (int)(next + before + incl - mine.pages);
  __syncthreads();
  const bool fits = total == 0 || next + total <= a.capacity;
  return {code_s ? code_s : fits ? 0 : kErrPoolFull, total};
}

// The plan has checked every page and table index; this holds also if another stream changes
// tables, token starts or the workspace while the call runs, which nothing can make right.
__device__ __forceinline__ bool inside(const AppendArgs& a, int slot, int idx, int page) {
  if (slot >= 0 && (uint32_t)idx < (uint32_t)a.max_pages && (uint32_t)page < (uint32_t)a.capacity)
    return true;
  atomicCAS(&g_append_error, 0, kErrAppend);
  return false;
}

// The page of a slot of a row: one that the row had, or one of its new ones.
__device__ __forceinline__ int page_of(const AppendArgs& a, int r, int n, int first, int idx) {
  const int have = (n + a.page_size - 1) / a.page_size;
  return idx < have ? a.block_table[(size_t)r * a.max_pages + idx] : first + idx - have;
}

// Blocks 0 .. token_blocks * groups - 1 take tokens (block / groups) and every groups-th
// slab: a head of the queries, or one of keys and values together.  The blocks behind them
// take a row a warp: its new length and the end of its last page.  Nothing is written before
// the plan is known; the first slab's rows, the angles and the token's sequence are ready by
// then.
template <int D>
__global__ void __launch_bounds__(kThreads, 7) append_kernel(const __grid_constant__ RopeArgs r,
                                                             const __grid_constant__ AppendArgs a,
                                                             int token_blocks, int groups,
                                                             int plan_blocks, int plan_shift) {
  constexpr int kPer = D / 16;
  __shared__ int base[kPlanBlocks];
  const PlanView plan(a.plan);
  const int rows = r.L * r.Hkv * a.B;
  if ((int)blockIdx.x >= token_blocks * groups) {
    const int block = blockIdx.x - token_blocks * groups, lane = threadIdx.x & 31;
    const int row = block * (kThreads / 32) + (threadIdx.x >> 5);
    const int m = row < rows ? tokens_of(a, row % a.B) : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Decision d = decide(a, plan, plan_blocks, base);
    if (block == 0 && threadIdx.x == 0) {
      a.next_page_out[0] = plan.head->next + (d.code ? 0 : (int)d.total);
      if (d.code) atomicCAS(&g_append_error, 0, d.code);
    }
    if (row >= rows) return;
    const int2 p = plan.rows[row];
    if (lane == 0) a.seq_lens_out[row] = d.code ? p.x : p.x + m;
    if (d.code) return;
    const int have = (p.x + a.page_size - 1) / a.page_size;
    const int used = (p.x + m) % a.page_size, last = (p.x + m) / a.page_size;
    if (used == 0 || last < have) return;
    const int pg = base[row >> plan_shift] + p.y + last - have;  // the unused rows of a new page
    if (!inside(a, min(p.x, p.x + m), last, pg)) return;
    const size_t at = ((size_t)pg * a.page_size + used) * D;
    const int chunks = (a.page_size - used) * (D / 8);
    for (int c = lane; c < chunks; c += 32) {
      reinterpret_cast<uint4*>(a.k_pages + at)[c] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(a.v_pages + at)[c] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int u = threadIdx.x % kPer;
  const int t = blockIdx.x / groups * (kThreads / kPer) + threadIdx.x / kPer;
  // the token's sequence: the last b with tok_start[b] <= t; none for padding behind the last
  bool live = t < r.N;
  int b = t, j = 0;
  if (a.tok_start) {
    live = live && t < a.tok_start[a.B];
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.tok_start[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    j = t - a.tok_start[b];
  }
  const Lane ln = lane_of(u, r.rot_dim, r.interleaved);
  float c[8], s[8];
  if (live && ln.rotate) angles(r, u, r.pos[t], c, s);
  const int n_q = r.q ? r.L * r.Hq : 0, n_all = live ? n_q + r.L * r.Hkv : 0;
  auto row_at = [&](int head) { return ((size_t)head * r.N + t) * D; };
  uint4 x0, x1, v0 = {}, v1 = {};
  auto load = [&](int slab) {
    const bool is_q = slab < n_q;
    const size_t row = row_at(is_q ? slab : slab - n_q);
    const uint4* in = reinterpret_cast<const uint4*>((is_q ? r.q : r.k) + row);
    x0 = in[ln.c0];
    x1 = in[ln.c1];
    if (!is_q) {
      v0 = reinterpret_cast<const uint4*>(a.v + row)[ln.c0];
      v1 = reinterpret_cast<const uint4*>(a.v + row)[ln.c1];
    }
  };
  int slab = blockIdx.x % groups;
  if (slab < n_all) load(slab);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (decide(a, plan, plan_blocks, base).code) return;
  while (slab < n_all) {
    const int at = slab;
    uint4 y0 = x0, y1 = x1;
    const uint4 w0 = v0, w1 = v1;
    slab += groups;
    if (slab < n_all) load(slab);  // the next rows come while these are turned and stored
    if (ln.rotate) rotate(y0, y1, c, s, r.interleaved);
    if (at < n_q) {
      uint4* out = reinterpret_cast<uint4*>(r.q_out + row_at(at));
      out[ln.c0] = y0;
      out[ln.c1] = y1;
      continue;
    }
    const int cr = (at - n_q) * a.B + b;
    const int2 p = plan.rows[cr];
    const int slot = p.x + j, idx = slot / a.page_size, off = slot - idx * a.page_size;
    if (!inside(a, slot, idx, 0)) continue;
    const int pg = page_of(a, cr, p.x, base[cr >> plan_shift] + p.y, idx);
    if (!inside(a, slot, idx, pg)) continue;
    // a new page enters the table with the first of its rows that this call writes
    if (u == 0 && off == 0) a.block_table[(size_t)cr * a.max_pages + idx] = pg;
    const size_t to = ((size_t)pg * a.page_size + off) * D;
    uint4* out = reinterpret_cast<uint4*>(a.k_pages + to);
    out[ln.c0] = y0;
    out[ln.c1] = y1;
    out = reinterpret_cast<uint4*>(a.v_pages + to);
    out[ln.c0] = w0;
    out[ln.c1] = w1;
  }
}

// Blocks per group of tokens: a thread walks at least four heads with one set of angles (one
// would spend more time on those than on the rows) while that leaves a quarter of the SMs'
// 16 blocks each, and otherwise in about `waves` times those 16.  One layer of 4096 tokens, 32
// and 8 heads, takes 25.8 us with a head a thread and 16.8 with four; 2079 tokens of 14 heads
// 6.2 and 4.9; a 16384-token prompt of 2 layers 102.2, 100.4, 99.2 and 171 us in 2, 4, 8 and
// 32 waves, a chunk of 8192 tokens in 4 layers 126.7, 128.2 and 131.6 us in 2, 3 and 6.
int slab_groups(int token_blocks, int slabs, int waves) {
  const int fill = (152 * 4 + token_blocks - 1) / token_blocks;
  int groups = (152 * 16 * waves + token_blocks - 1) / token_blocks;
  groups = groups < slabs / 4 ? groups : slabs / 4;
  if (groups < fill) groups = fill;
  return groups < 1 ? 1 : groups > slabs ? slabs : groups > 65535 ? 65535 : groups;
}

}  // namespace

size_t append_workspace_bytes(int rows) {
  return sizeof(PlanHead) + kPlanBlocks * sizeof(PlanBlock) + (size_t)rows * sizeof(int2);
}

cudaError_t launch_rope(const RopeArgs& r, cudaStream_t s) {
  const int slabs = (r.q ? r.L * r.Hq : 0) + (r.k ? r.L * r.Hkv : 0);
  if (r.N == 0 || slabs == 0) return cudaSuccess;
  const int per_block = kThreads / (r.d / 16);
  const int blocks = (r.N + per_block - 1) / per_block;
  Launch l(dim3(blocks, slab_groups(blocks, slabs, 8)), kThreads, s);
  count_launches(1);
  return r.d == 128 ? cudaLaunchKernelEx(&l.cfg, rope_kernel<128>, r)
                    : cudaLaunchKernelEx(&l.cfg, rope_kernel<64>, r);
}

cudaError_t launch_append(const RopeArgs& r, const AppendArgs& a, cudaStream_t s) {
  const int rows = r.L * r.Hkv * a.B;
  int plan_shift = 10;  // rows of a plan block: kPlanThreads times a power of two
  static_assert(kPlanThreads == 1 << 10, "a row a thread at least");
  while (((rows - 1) >> plan_shift) >= kPlanBlocks) ++plan_shift;
  const int plan_blocks = ((rows - 1) >> plan_shift) + 1, per = 1 << (plan_shift - 10);
  count_launches(2);
  Launch p(dim3(plan_blocks), kPlanThreads, s);
  cudaError_t e = cudaLaunchKernelEx(&p.cfg, append_plan_kernel, a, rows, r.N, per);
  if (e != cudaSuccess) return e;
  const int slabs = (r.q ? r.L * r.Hq : 0) + r.L * r.Hkv;
  const int per_block = kThreads / (r.d / 16);
  const int blocks = (r.N + per_block - 1) / per_block;
  const int groups = blocks ? slab_groups(blocks, slabs, 2) : 1;
  const int row_blocks = (rows + kThreads / 32 - 1) / (kThreads / 32);
  // its blocks come up beside the plan's and wait for it
  Launch l(dim3(blocks * groups + row_blocks), kThreads, s);
  return r.d == 128 ? cudaLaunchKernelEx(&l.cfg, append_kernel<128>, r, a, blocks, groups,
                                         plan_blocks, plan_shift)
                    : cudaLaunchKernelEx(&l.cfg, append_kernel<64>, r, a, blocks, groups,
                                         plan_blocks, plan_shift);
}

cudaError_t rope_device_error(int* code, bool clear, cudaStream_t s) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(code, g_append_error, sizeof(int), 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && clear && *code) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_append_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

}  // namespace kvs
