// Launchers of the calls that move, share and free pages of the paged cache.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace kvs {

// The pages of a cache and the rows that use them: row (l * Hkv + hk) * B + b.
struct PagedArgs {
  int L = 0, Hkv = 0, B = 0, d = 0, page_size = 0, capacity = 0, max_pages = 0;
  bf16_t* k_pages = nullptr;        // [capacity][page_size][d]
  bf16_t* v_pages = nullptr;
  const int* block_table = nullptr; // [rows][max_pages]
  const int* seq_lens = nullptr;    // [rows]
};

struct AcceptArgs {
  int N = 0;
  const int* tok_start = nullptr;   // [B + 1]
  const int* n_accept = nullptr;    // [B]
  const int* accept = nullptr;      // [N]
  int* seq_lens_out = nullptr;      // [rows]
};

struct ForkArgs {
  int forks = 0, w = 0;
  const int* src = nullptr;         // [forks]
  const int* dst = nullptr;
  const int* next_page = nullptr;   // [1]
  int* next_page_out = nullptr;
  int* block_table = nullptr;       // the table and the lengths again, to be written
  int* seq_lens = nullptr;
  int* pos = nullptr;               // [B], and the rings [rows][w][...], with w > 0
  float* ring_score = nullptr;
  bf16_t* ring_k = nullptr;
  bf16_t* ring_v = nullptr;
  void* plan = nullptr;             // workspace of fork_workspace_bytes()
};

struct ReclaimArgs {
  const int* next_page = nullptr;   // [1]
  int* next_page_out = nullptr;
  int* block_table_out = nullptr;   // [rows][max_pages]
  void* ws = nullptr;               // workspace of reclaim_workspace_bytes()
};

constexpr int kMaxForkBatch = 131072;  // sequences of a batch with forks (a bit each in a block)

size_t fork_workspace_bytes(int rows);  // rows = L * Hkv * forks
size_t reclaim_workspace_bytes(int capacity);
cudaError_t launch_accept(const PagedArgs& p, const AcceptArgs& a, cudaStream_t s);
cudaError_t launch_fork(const PagedArgs& p, const ForkArgs& a, cudaStream_t s);
cudaError_t launch_reclaim(const PagedArgs& p, const ReclaimArgs& a, cudaStream_t s);
cudaError_t pages_device_error(int* code, bool clear, cudaStream_t s);

}  // namespace kvs
