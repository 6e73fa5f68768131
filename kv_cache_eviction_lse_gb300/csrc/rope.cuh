// Launchers of the position rotation and of the paged append that rotates on the way.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace kvs {

constexpr int kMaxFreqs = 64;  // rotated pairs per head: d / 2 at d = 128

struct RopeArgs {
  const bf16_t* q = nullptr;  // [L][Hq][N][d] or null
  const bf16_t* k = nullptr;  // [L][Hkv][N][d] or null
  bf16_t* q_out = nullptr;
  bf16_t* k_out = nullptr;    // kvs_rope only
  int L = 0, Hq = 0, Hkv = 0, d = 0, N = 0;
  const int* pos = nullptr;   // [N]
  int rot_dim = 0, interleaved = 0;
  // turns per position of each pair as a 64-bit binary fraction (wraps like the angle)
  uint64_t freq[kMaxFreqs] = {};
};

// The paged side of an append: where the tokens' rotated keys and values go.
struct AppendArgs {
  const bf16_t* v = nullptr;        // [L][Hkv][N][d]
  int B = 0, page_size = 0, max_pages = 0, capacity = 0;
  const int* tok_start = nullptr;   // [B + 1], or null: sequence b owns token b
  bf16_t* k_pages = nullptr;        // [capacity][page_size][d]
  bf16_t* v_pages = nullptr;
  const int* next_page = nullptr;   // [1]
  int* next_page_out = nullptr;
  int* block_table = nullptr;       // [rows][max_pages]
  const int* seq_lens = nullptr;    // [rows]
  int* seq_lens_out = nullptr;
  void* plan = nullptr;             // workspace of append_workspace_bytes()
};

size_t append_workspace_bytes(int rows);
cudaError_t launch_rope(const RopeArgs& r, cudaStream_t s);
cudaError_t launch_append(const RopeArgs& r, const AppendArgs& a, cudaStream_t s);
cudaError_t rope_device_error(int* code, bool clear, cudaStream_t s);

}  // namespace kvs
