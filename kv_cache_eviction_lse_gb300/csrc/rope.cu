// Position rotation of queries and keys, and the append of new tokens to the paged cache
// with the rotation on the way.
//
// A pair (a, b) of dimensions of a token at position p turns by the angle p f:
//   (a cos - b sin, b cos + a sin).
// f is kept as turns per position in a 64-bit binary fraction, so p f mod 1 is one integer
// product that wraps where the angle does: the angle of any 32-bit position is exact to
// p 2^-65 turns and needs no range reduction (a 32-bit product would be off by 0.01 rad at
// position 131072).  In [-pi, pi] the hardware's sine and cosine are good to 2^-21, far
// below the bf16 rounding of the result (2^-8 relative), and shorten small batches (2079
// tokens of 14 heads 6.5 -> 5.9 us against sincospif).  The products are fp32, and each
// result is rounded to bf16 once.
//
// Bound by HBM (or, for a few tokens, by latency): every row is read and written once, and
// a thread that has the cosines and sines of its token's 8 pairs reuses them for the heads
// and layers it walks through.  A 16384-token prompt of 2 layers takes 99 us (671 MB, 6.8
// TB/s, the rate of a copy).
#include "common.cuh"
#include "rope.cuh"

namespace kvs {

__device__ int g_append_error = 0;

namespace {

constexpr int kErrPoolFull = 4;   // as kvs_decode_step
constexpr int kErrTableFull = 5;
constexpr int kErrAppend = 8;     // token starts, lengths or page ids out of range

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;

// The plan of an append in the workspace: a status word (0 = append), then the length
// and the first new page of every row.
constexpr int kPlanHeader = 4;

__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x);
  x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z);
  x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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
  float c[8], s[8];
  if (ln.rotate) angles(r, u, r.pos[t], c, s);
  const int n_q = r.q ? r.L * r.Hq : 0, n_all = n_q + (r.k ? r.L * r.Hkv : 0);
  for (int slab = blockIdx.y; slab < n_all; slab += gridDim.y) {
    const bool is_q = slab < n_q;
    const size_t row = ((size_t)(is_q ? slab : slab - n_q) * r.N + t) * D;
    const uint4* in = reinterpret_cast<const uint4*>((is_q ? r.q : r.k) + row);
    uint4* out = reinterpret_cast<uint4*>((is_q ? r.q_out : r.k_out) + row);
    uint4 x0 = in[ln.c0], x1 = in[ln.c1];
    if (ln.rotate) rotate(x0, x1, c, s, r.interleaved);
    out[ln.c0] = x0;
    out[ln.c1] = x1;
  }
}

// One block decides the whole append: every row's new tokens, its first new page by an
// exclusive sum over the rows, and whether all of it fits.
__global__ void __launch_bounds__(kPlanThreads, 1) append_plan_kernel(const AppendArgs a, int rows,
                                                                   int N) {
  __shared__ long long sums[32];
  __shared__ int err;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) err = 0;
  __syncthreads();
  auto fault = [&](int code) { atomicMax(&err, code); };
  auto tokens = [&](int b) { return a.tok_start ? a.tok_start[b + 1] - a.tok_start[b] : 1; };
  if (a.tok_start) {
    for (int b = tid; b < a.B; b += kPlanThreads)
      if (a.tok_start[b] < 0 || a.tok_start[b + 1] < a.tok_start[b]) fault(kErrAppend);
    if (tid == 0 && (a.tok_start[0] != 0 || a.tok_start[a.B] > N)) fault(kErrAppend);
  }
  const int next = a.next_page[0];
  if (tid == 0 && next < 0) fault(kErrAppend);
  __syncthreads();
  const int ps = a.page_size;
  // slots and page counts stay within 32 bits
  const long long room = min((long long)a.max_pages * ps, (long long)INT32_MAX - 8192);
  const int per = (rows + kPlanThreads - 1) / kPlanThreads;
  const long long lo = (long long)tid * per;
  const int r0 = (int)(lo < rows ? lo : rows), r1 = (int)(lo + per < rows ? lo + per : rows);
  long long mine = 0;
  if (err == 0) {
    for (int r = r0; r < r1; ++r) {
      const int n = a.seq_lens[r], m = tokens(r % a.B);
      a.plan[kPlanHeader + 2 * r] = n;
      if (n < 0 || n > room) { fault(kErrAppend); continue; }
      if (m == 0) continue;
      if (n + (long long)m > room) { fault(kErrTableFull); continue; }
      if (n % ps) {
        const int pg = a.block_table[(size_t)r * a.max_pages + n / ps];
        if (pg < 0 || pg >= a.capacity) fault(kErrAppend);
      }
      mine += (n + (long long)m + ps - 1) / ps - (n + ps - 1) / ps;
    }
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < kPlanThreads / 32 ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sums[lane] = w;
  }
  __syncthreads();
  const long long total = sums[31];
  if (tid == 0 && total > 0 && next + total > a.capacity) fault(kErrPoolFull);
  __syncthreads();
  const int code = err;
  long long first = next + (warp ? sums[warp - 1] : 0) + incl - mine;
  for (int r = r0; r < r1; ++r) {
    if (code) {
      a.seq_lens_out[r] = a.seq_lens[r];
      continue;
    }
    const int n = a.plan[kPlanHeader + 2 * r], m = tokens(r % a.B);
    a.plan[kPlanHeader + 2 * r + 1] = (int)first;
    first += (n + (long long)m + ps - 1) / ps - (n + ps - 1) / ps;
    a.seq_lens_out[r] = n + m;
  }
  if (tid == 0) {
    a.plan[0] = code;
    a.next_page_out[0] = code ? next : (int)(next + total);
    if (code) atomicCAS(&g_append_error, 0, code);
  }
}

// The plan has checked every page and table index; this holds also if another stream changes
// the tables or token starts while the call runs, which nothing can make right.
__device__ __forceinline__ bool inside(const AppendArgs& a, int idx, int page) {
  if ((uint32_t)idx < (uint32_t)a.max_pages && (uint32_t)page < (uint32_t)a.capacity) return true;
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
// clear page ends.  Nothing is written before the plan is known; the first slab's rows, the
// angles and the token's sequence are ready by then.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ RopeArgs r,
                                                          const __grid_constant__ AppendArgs a,
                                                          int token_blocks, int groups) {
  constexpr int kPer = D / 16;
  const int rows = r.L * r.Hkv * a.B;
  if ((int)blockIdx.x >= token_blocks * groups) {
    // one warp per row: the unused rows of the row's last page, where that page is new
    const int row = (blockIdx.x - token_blocks * groups) * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int b = row % a.B;
    const int m = a.tok_start ? a.tok_start[b + 1] - a.tok_start[b] : 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.plan[0] != 0) return;
    const int n = a.plan[kPlanHeader + 2 * row];
    const int have = (n + a.page_size - 1) / a.page_size;
    const int used = (n + m) % a.page_size, last = (n + m) / a.page_size;
    if (used == 0 || last < have) return;
    const int pg = a.plan[kPlanHeader + 2 * row + 1] + last - have;
    if (!inside(a, last, pg)) return;
    const size_t at = ((size_t)pg * a.page_size + used) * D;
    const int chunks = (a.page_size - used) * (D / 8);
    for (int c = threadIdx.x & 31; c < chunks; c += 32) {
      reinterpret_cast<uint4*>(a.k_pages + at)[c] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(a.v_pages + at)[c] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int u = threadIdx.x % kPer;
  const int t = blockIdx.x / groups * (kThreads / kPer) + threadIdx.x / kPer;
  if (t >= r.N) return;
  // the token's sequence: the last b with tok_start[b] <= t
  int b = t, j = 0;
  if (a.tok_start) {
    if (t >= a.tok_start[a.B]) return;  // behind the last sequence
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
  if (ln.rotate) angles(r, u, r.pos[t], c, s);
  const int n_q = r.q ? r.L * r.Hq : 0, n_all = n_q + r.L * r.Hkv;
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
  if (a.plan[0] != 0) return;
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
    const int2 plan = reinterpret_cast<const int2*>(a.plan + kPlanHeader)[cr];
    const int slot = plan.x + j, idx = slot / a.page_size, off = slot - idx * a.page_size;
    if (!inside(a, idx, 0)) continue;
    const int pg = page_of(a, cr, plan.x, plan.y, idx);
    if (!inside(a, idx, pg)) continue;
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

// Blocks per group of tokens: a thread walks several heads with one set of angles, in about
// `waves` times the 8 blocks of an SM.  A 16384-token prompt of 2 layers turns in 102.2,
// 100.4, 99.2 and 171 us with 2, 4, 8 and 32; a chunk of 8192 tokens in 4 layers is
// appended in 130.6, 127.7, 132.7 and 206 us.
int slab_groups(int token_blocks, int slabs, int waves) {
  int groups = (152 * 8 * waves + token_blocks - 1) / token_blocks;
  return groups < 1 ? 1 : groups > slabs ? slabs : groups > 65535 ? 65535 : groups;
}

}  // namespace

size_t append_workspace_bytes(int rows) {
  return ((size_t)kPlanHeader + 2 * (size_t)rows) * sizeof(int);
}

cudaError_t launch_rope(const RopeArgs& r, cudaStream_t s) {
  const int slabs = (r.q ? r.L * r.Hq : 0) + (r.k ? r.L * r.Hkv : 0);
  if (r.N == 0 || slabs == 0) return cudaSuccess;
  const int per_block = kThreads / (r.d / 16);
  const int blocks = (r.N + per_block - 1) / per_block;
  const dim3 grid(blocks, slab_groups(blocks, slabs, 8));
  count_launches(1);
  if (r.d == 128)
    rope_kernel<128><<<grid, kThreads, 0, s>>>(r);
  else
    rope_kernel<64><<<grid, kThreads, 0, s>>>(r);
  return cudaGetLastError();
}

cudaError_t launch_append(const RopeArgs& r, const AppendArgs& a, cudaStream_t s) {
  const int rows = r.L * r.Hkv * a.B;
  count_launches(1);
  append_plan_kernel<<<1, kPlanThreads, 0, s>>>(a, rows, r.N);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || r.N == 0) return e;
  const int slabs = (r.q ? r.L * r.Hq : 0) + r.L * r.Hkv;
  const int per_block = kThreads / (r.d / 16);
  const int blocks = (r.N + per_block - 1) / per_block, groups = slab_groups(blocks, slabs, 4);
  const int clear = a.page_size > 1 ? (rows + kThreads / 32 - 1) / (kThreads / 32) : 0;
  // its blocks come up beside the plan's and wait for it
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks * groups + clear);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return r.d == 128 ? cudaLaunchKernelEx(&cfg, append_kernel<128>, r, a, blocks, groups)
                    : cudaLaunchKernelEx(&cfg, append_kernel<64>, r, a, blocks, groups);
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
