// Launcher of the single-token attention over the paged cache and the window ring.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace kvs {

struct AttnDecodeArgs {
  const bf16_t* q = nullptr;        // [L][Hq][B][d]
  int L = 0, Hq = 0, Hkv = 0, B = 0, d = 0;
  int page_size = 0, capacity = 0, max_pages = 0, w = 0;
  const bf16_t* k_pages = nullptr;  // [capacity][page_size][d]
  const bf16_t* v_pages = nullptr;
  const int* block_table = nullptr; // [rows][max_pages]
  const int* seq_lens = nullptr;    // [rows]
  const int* pos = nullptr;         // [B], with w > 0
  const bf16_t* ring_k = nullptr;   // [rows][w][d]
  const bf16_t* ring_v = nullptr;
  bf16_t* o = nullptr;              // [L][Hq][B][d]
  float* lse = nullptr;             // [L][Hq][B] or null
  void* ws = nullptr;
  bool read_once = false;           // set at launch: keys and values leave L2 first
};

size_t attn_decode_workspace_bytes(int group, int d);
cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t s);
cudaError_t attn_decode_device_error(int* code, bool clear, cudaStream_t s);

}  // namespace kvs
