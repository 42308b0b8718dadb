// Host-side interfaces of the serving operators (logit rules, token history,
// paged-cache tables) between the C-ABI layer (serve_api.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "specv.h"

namespace specv {

// Device status flags (mirror SPEC_DEV_* of the public header).
constexpr int kFlagIndex = 16;
constexpr int kFlagParam = 32;
constexpr int kFlagPages = 64;
constexpr int kFlagLengths = 128;

struct RulesArgs {
  const char* x;            // logits
  char* out;                // == x: in place
  const int32_t* row_off;   // nullable: dense rows
  int64_t n_rows;           // rows of the buffer
  int B, K, rows, L;        // rows of a block: L (draft) or L + 1 (target)
  int64_t V;
  const int32_t* tokens;    // nullable
  const int32_t* vlen;      // nullable
  const int32_t* seats;     // nullable
  spec_history h;           // h.counts == NULL: no history
  const uint32_t* mask;     // nullable
  const int32_t* mask_rows; // nullable
  int n_masks, mask_len;
  int per;                  // rows of a request that one block takes
  int special;              // room for drafted and biased tokens
  int* status;
};

cudaError_t launch_logit_rules(const RulesArgs& a, int dtype, cudaStream_t st);

cudaError_t launch_history_add(const spec_history& h, const int32_t* seats, int B, const int32_t* tokens, int64_t n,
                               const int32_t* offsets, int width, int output, int* status, cudaStream_t st);
cudaError_t launch_history_clear(const spec_history& h, const int32_t* seats, int B, int* status, cudaStream_t st);

struct KvArgs {
  spec_kv_pages p;
  const int32_t* seats;     // nullable
  int B;
  const int32_t* ctx_len;   // map: tokens in the cache; release: tokens to keep (nullable: none)
  const int32_t* offsets;   // map: [B + 1]
  int64_t N;                // map: entries of kv_slots and positions
  int64_t* kv_slots;
  int32_t* positions;       // nullable
  int32_t* seq_len;
  int32_t* block_table;     // nullable, [B, max_pages]
  int* status;
  int* ticket;
};

cudaError_t launch_kv_map(const KvArgs& a, cudaStream_t st);
cudaError_t launch_kv_release(const KvArgs& a, cudaStream_t st);

}  // namespace specv
