// Attention of one new token per sequence over its row's paged cache and window ring:
//   o = sum_i a_i v_i,  a_i = exp(q . k_i / sqrt(d) - lse),  lse = ln sum_i exp(q . k_i / sqrt(d))
// over the row's seq_lens[r] paged keys and the min(pos, w) keys of its ring, for the g
// query heads of the row's KV head.
//
// One block per row and group of 8 query heads; each warp walks every fourth key with a
// running maximum and sum per head, and the warps meet in shared memory.
#include "attn_decode.cuh"
#include "common.cuh"

namespace kvs {

__device__ int g_attn_decode_error = 0;

namespace {

constexpr int kErrAttnDecode = 9;  // a length or page id out of range
constexpr int kHeads = 8;
constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_decode_kernel(const AttnDecodeArgs a) {
  constexpr int E = D / 32;  // dimensions of a lane
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads], sm_o[kWarps][kHeads][D];
  const int g = a.Hq / a.Hkv;
  const int groups = (g + kHeads - 1) / kHeads;
  const int row = blockIdx.x / groups, h0 = blockIdx.x % groups * kHeads;
  const int heads = min(kHeads, g - h0);
  const int b = row % a.B, hl = row / a.B;  // hl = l * H_kv + hk
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long n = a.seq_lens[row];
  const long long room = (long long)a.max_pages * a.page_size;
  if (n < 0 || n > room) {
    if (threadIdx.x == 0) atomicCAS(&g_attn_decode_error, 0, kErrAttnDecode);
    n = n < 0 ? 0 : room;
  }
  const int held = a.w > 0 ? max(0, min(a.pos[b], a.w)) : 0;
  const float scale = rsqrtf((float)D) * kLog2e;
  float q[kHeads][E], o[kHeads][E], m[kHeads], l[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const size_t at = (((size_t)hl * g + h0 + h) * a.B + b) * D + e * 32 + lane;
      q[h][e] = h < heads ? bf16_lo(a.q[at]) * scale : 0.f;
      o[h][e] = 0.f;
    }
  }
  for (long long i = warp; i < n + held; i += kWarps) {
    const bf16_t *k, *v;
    if (i < n) {
      const int pg = a.block_table[(size_t)row * a.max_pages + i / a.page_size];
      if (pg < 0 || pg >= a.capacity) {
        if (lane == 0) atomicCAS(&g_attn_decode_error, 0, kErrAttnDecode);
        continue;
      }
      const size_t at = ((size_t)pg * a.page_size + i % a.page_size) * D;
      k = a.k_pages + at;
      v = a.v_pages + at;
    } else {
      const size_t at = ((size_t)row * a.w + (i - n)) * D;
      k = a.ring_k + at;
      v = a.ring_v + at;
    }
    float x[kHeads] = {};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float ke = bf16_lo(k[e * 32 + lane]);
#pragma unroll
      for (int h = 0; h < kHeads; ++h) x[h] += q[h][e] * ke;
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      const float s = warp_sum(x[h]);
      const float top = fmaxf(m[h], s);
      const float base = top == -INFINITY ? 0.f : top;
      const float c = fast_exp2(m[h] - base), p = fast_exp2(s - base);
      l[h] = l[h] * c + p;
      m[h] = top;
#pragma unroll
      for (int e = 0; e < E; ++e) o[h][e] = o[h][e] * c + p * bf16_lo(v[e * 32 + lane]);
    }
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (lane == 0) {
      sm_m[warp][h] = m[h];
      sm_l[warp][h] = l[h];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][h][e * 32 + lane] = o[h][e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < heads * D; i += kWarps * 32) {
    const int h = i / D, e = i % D;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w][h]);
    const float base = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kWarps; ++w) {
      const float c = fast_exp2(sm_m[w][h] - base);
      sum += sm_l[w][h] * c;
      acc += sm_o[w][h][e] * c;
    }
    const size_t at = ((size_t)hl * g + h0 + h) * a.B + b;
    const float y = sum == 0.f ? 0.f : acc / sum;
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(0.f), "f"(y));
    a.o[at * D + e] = (bf16_t)(u & 0xffffu);
    if (a.lse && e == 0) a.lse[at] = sum == 0.f ? -INFINITY : kLn2 * (top + log2f(sum));
  }
}

}  // namespace

size_t attn_decode_workspace_bytes(int rows, int group, int d) {
  (void)rows; (void)group; (void)d;
  return 16;
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t s) {
  const int rows = a.L * a.Hkv * a.B, g = a.Hq / a.Hkv;
  if (rows == 0) return cudaSuccess;
  const int blocks = rows * ((g + kHeads - 1) / kHeads);
  count_launches(1);
  if (a.d == 128)
    attn_decode_kernel<128><<<blocks, kWarps * 32, 0, s>>>(a);
  else
    attn_decode_kernel<64><<<blocks, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
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
