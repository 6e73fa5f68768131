// Launcher of the attention of drafted tokens over the paged cache and the window ring.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace kvs {

constexpr int kMaxDraft = 256;  // drafted tokens of a sequence: a thread and 256 bits each

// Division of 0 <= n < 2^31 by a divisor that a call has for all: the compiler's takes 20 times the
// code.  With s = ceil(log2 d) and m = ceil(2^(31 + s) / d), n m / 2^(31 + s) exceeds n / d by less
// than n / 2^(31 + s) < 1 / d.
struct Divisor {
  uint32_t m = 1u << 31;
  int s = 0, d = 1;
  Divisor() = default;
  explicit Divisor(int divisor) : d(divisor) {
    while ((1ll << s) < d) ++s;
    m = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  }
  __host__ __device__ int of(int n) const { return (int)((uint64_t)(uint32_t)n * m >> (31 + s)); }
};

struct AttnTreeArgs {
  const bf16_t* q = nullptr;        // [L][Hq][N][d]
  int L = 0, Hq = 0, Hkv = 0, B = 0, N = 0, d = 0, max_draft = 0;
  int page_size = 0, capacity = 0, max_pages = 0, w = 0;
  const int* tok_start = nullptr;   // [B + 1]
  const int* parent = nullptr;      // [N], or null: chains
  const bf16_t* k_pages = nullptr;  // [capacity][page_size][d]
  const bf16_t* v_pages = nullptr;
  const int* block_table = nullptr; // [rows][max_pages]
  const int* seq_lens = nullptr;    // [rows]
  const int* pos = nullptr;         // [B], with w > 0
  const bf16_t* ring_k = nullptr;   // [rows][w][d]
  const bf16_t* ring_v = nullptr;
  bf16_t* o = nullptr;              // [L][Hq][N][d]
  float* lse = nullptr;             // [L][Hq][N] or null
  void* ws = nullptr;
  int box_rows = 0;                 // set at launch: rows of a TMA box, or 0
  Divisor by_batch, by_page, by_group;  // set at launch: by B, page_size, Hq / Hkv
};

size_t attn_tree_workspace_bytes(int d);
cudaError_t launch_attn_tree(const AttnTreeArgs& a, cudaStream_t s);
cudaError_t attn_tree_device_error(int* code, bool clear, cudaStream_t s);

}  // namespace kvs
