// C ABI of the serving operators (declared in include/specv.h): host-side
// argument checks and launches. No call allocates, frees or synchronises.
#include "specv.h"
#include "serve.h"

using namespace specv;

namespace {

constexpr size_t kStatusBytes = 256;  // header: status word + padding
// The kv calls' ticket lies in the header, where no call has scratch: it stays 0 between calls whatever else used the
// workspace. (The 256 bytes that spec_kv_workspace_size asks for behind the header are not used.)
constexpr size_t kTicketAt = 128, kKvBytes = kStatusBytes + 256;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }  // NULL is aligned
int map_cuda(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

int check_batch(int B, const int32_t* seats, int table) {
  if (B < 1 || !aligned(seats, 4)) return SPEC_ERR_ARG;
  if (B > SPEC_MAX_B) return SPEC_ERR_UNSUPPORTED;
  if (!seats && B > table) return SPEC_ERR_ARG;  // request b sits in seat b
  return SPEC_OK;
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
  return ws && bytes >= need && aligned(ws, 16) ? SPEC_OK : SPEC_ERR_WORKSPACE;
}

int check_history(const spec_history* h) {
  if (!h || !h->counts || !h->seen || h->seats < 1 || h->V < 1 || h->n_bias < 0) return SPEC_ERR_ARG;
  if (h->seats > SPEC_MAX_SEATS || h->V > SPEC_MAX_V || h->n_bias > SPEC_MAX_BIAS) return SPEC_ERR_UNSUPPORTED;
  if (h->n_bias && (!h->bias_tokens || !h->bias_values)) return SPEC_ERR_ARG;
  if (!aligned(h->counts, 4) || !aligned(h->seen, 4) || !aligned(h->repetition, 4) || !aligned(h->frequency, 4) ||
      !aligned(h->presence, 4) || !aligned(h->bias_tokens, 4) || !aligned(h->bias_values, 4))
    return SPEC_ERR_ARG;
  return SPEC_OK;
}

int check_pages(const spec_kv_pages* p, int B) {
  if (!p || !p->page_table || !p->owned || !p->free_pages || !p->free_count) return SPEC_ERR_ARG;
  if (p->seats < 1 || p->max_pages < 1 || p->n_pages < 1 || p->page_size < 1) return SPEC_ERR_ARG;
  if (p->seats > SPEC_MAX_SEATS || p->max_pages > (1 << 30) || static_cast<int64_t>(B) * p->max_pages > 0x7fffffff)
    return SPEC_ERR_UNSUPPORTED;
  if (!aligned(p->page_table, 4) || !aligned(p->owned, 4) || !aligned(p->free_pages, 4) || !aligned(p->free_count, 4))
    return SPEC_ERR_ARG;
  return SPEC_OK;
}

}  // namespace

extern "C" {

size_t spec_rules_workspace_size(int B) { return B < 1 || B > SPEC_MAX_B ? 0 : kStatusBytes; }

size_t spec_kv_workspace_size(int B) { return B < 1 || B > SPEC_MAX_B ? 0 : kKvBytes; }

int spec_logit_rules(const void* logits, void* out, int dtype, const int32_t* row_off, int64_t n_rows, int B, int K,
                     int rows, int L, int64_t V, const int32_t* draft_tokens, const int32_t* verify_len,
                     const spec_history* history, const int32_t* seats, const uint32_t* mask, int n_masks,
                     int mask_len, const int32_t* mask_rows, void* workspace, size_t ws_bytes, spec_stream_t stream) {
  if ((dtype != SPEC_F32 && dtype != SPEC_BF16) || V < 1) return SPEC_ERR_ARG;
  if (n_rows != 0 && (!logits || !out)) return SPEC_ERR_ARG;  // the draft rows of an empty block may be NULL
  if (B < 1 || K < 1 || L < 0 || n_rows < 0 || (rows != L && rows != L + 1)) return SPEC_ERR_ARG;
  if (B > SPEC_MAX_B || K > SPEC_MAX_K || L > SPEC_MAX_L || V > SPEC_MAX_V) return SPEC_ERR_UNSUPPORTED;
  if (n_rows > (int64_t{1} << 40)) return SPEC_ERR_UNSUPPORTED;
  if (row_off ? K != 1 || rows != L + 1 : n_rows != static_cast<int64_t>(B) * K * rows) return SPEC_ERR_ARG;
  const int es = dtype == SPEC_F32 ? 4 : 2;
  if (!aligned(logits, es) || !aligned(out, es) || !aligned(row_off, 4) || !aligned(draft_tokens, 4) ||
      !aligned(verify_len, 4) || !aligned(mask, 4) || !aligned(mask_rows, 4))
    return SPEC_ERR_ARG;
  int e = check_batch(B, seats, history ? history->seats : B);
  if (e) return e;
  if (history) {
    e = check_history(history);
    if (e) return e;
    if (history->V != V || (L > 0 && !draft_tokens)) return SPEC_ERR_ARG;
  }
  if (mask && (n_masks < 1 || mask_len < rows || (!mask_rows && n_masks < B))) return SPEC_ERR_ARG;
  const int64_t bytes = n_rows * V * es;
  const char* x = static_cast<const char*>(logits);
  char* y = static_cast<char*>(out);
  if (x != y && x < y + bytes && y < x + bytes) return SPEC_ERR_ARG;  // neither in place nor apart
  e = check_workspace(workspace, ws_bytes, spec_rules_workspace_size(B));
  if (e) return e;
  if (n_rows == 0 || (x == y && !history && !mask)) return SPEC_OK;
  RulesArgs a = {};
  a.x = x;
  a.out = y;
  a.row_off = row_off;
  a.n_rows = n_rows;
  a.B = B;
  a.K = K;
  a.rows = rows;
  a.L = L;
  a.V = V;
  a.tokens = draft_tokens;
  a.vlen = verify_len;
  a.seats = seats;
  if (history) a.h = *history;
  a.mask = mask;
  a.mask_rows = mask_rows;
  a.n_masks = n_masks;
  a.mask_len = mask_len;
  a.status = static_cast<int*>(workspace);
  return map_cuda(launch_logit_rules(a, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int spec_history_add(const spec_history* history, const int32_t* seats, int B, const int32_t* tokens,
                     int64_t n_tokens, const int32_t* offsets, int output, void* workspace, size_t ws_bytes,
                     spec_stream_t stream) {
  int e = check_history(history);
  if (e) return e;
  e = check_batch(B, seats, history->seats);
  if (e) return e;
  if (n_tokens < 0 || n_tokens > 0x7fffffff || (n_tokens > 0 && !tokens) || (output != 0 && output != 1))
    return SPEC_ERR_ARG;
  if (!offsets && n_tokens % B != 0) return SPEC_ERR_ARG;
  if (!aligned(tokens, 4) || !aligned(offsets, 4)) return SPEC_ERR_ARG;
  e = check_workspace(workspace, ws_bytes, spec_rules_workspace_size(B));
  if (e || n_tokens == 0) return e;
  return map_cuda(launch_history_add(*history, seats, B, tokens, n_tokens, offsets,
                                     static_cast<int>(offsets ? 0 : n_tokens / B), output,
                                     static_cast<int*>(workspace), reinterpret_cast<cudaStream_t>(stream)));
}

int spec_history_clear(const spec_history* history, const int32_t* seats, int B, void* workspace, size_t ws_bytes,
                       spec_stream_t stream) {
  int e = check_history(history);
  if (e) return e;
  e = check_batch(B, seats, history->seats);
  if (e) return e;
  e = check_workspace(workspace, ws_bytes, spec_rules_workspace_size(B));
  if (e) return e;
  return map_cuda(launch_history_clear(*history, seats, B, static_cast<int*>(workspace),
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int spec_kv_map(const spec_kv_pages* pages, const int32_t* seats, int B, const int32_t* ctx_len,
                const int32_t* offsets, int64_t n_tokens, int64_t* kv_slots, int32_t* positions, int32_t* seq_len,
                int32_t* block_table, void* workspace, size_t ws_bytes, spec_stream_t stream) {
  int e = check_pages(pages, B);
  if (e) return e;
  e = check_batch(B, seats, pages->seats);
  if (e) return e;
  if (!ctx_len || !offsets || !seq_len || n_tokens < 0 || n_tokens > 0x7fffffff || (n_tokens > 0 && !kv_slots))
    return SPEC_ERR_ARG;
  if (!aligned(ctx_len, 4) || !aligned(offsets, 4) || !aligned(kv_slots, 8) || !aligned(positions, 4) ||
      !aligned(seq_len, 4) || !aligned(block_table, 4))
    return SPEC_ERR_ARG;
  e = check_workspace(workspace, ws_bytes, spec_kv_workspace_size(B));
  if (e) return e;
  KvArgs a = {};
  a.p = *pages;
  a.seats = seats;
  a.B = B;
  a.ctx_len = ctx_len;
  a.offsets = offsets;
  a.N = n_tokens;
  a.kv_slots = kv_slots;
  a.positions = positions;
  a.seq_len = seq_len;
  a.block_table = block_table;
  a.status = static_cast<int*>(workspace);
  a.ticket = reinterpret_cast<int*>(static_cast<char*>(workspace) + kTicketAt);
  return map_cuda(launch_kv_map(a, reinterpret_cast<cudaStream_t>(stream)));
}

int spec_kv_release(const spec_kv_pages* pages, const int32_t* seats, int B, const int32_t* keep_len,
                    void* workspace, size_t ws_bytes, spec_stream_t stream) {
  int e = check_pages(pages, B);
  if (e) return e;
  e = check_batch(B, seats, pages->seats);
  if (e) return e;
  if (!aligned(keep_len, 4)) return SPEC_ERR_ARG;
  e = check_workspace(workspace, ws_bytes, spec_kv_workspace_size(B));
  if (e) return e;
  KvArgs a = {};
  a.p = *pages;
  a.seats = seats;
  a.B = B;
  a.ctx_len = keep_len;
  a.status = static_cast<int*>(workspace);
  a.ticket = reinterpret_cast<int*>(static_cast<char*>(workspace) + kTicketAt);
  return map_cuda(launch_kv_release(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
