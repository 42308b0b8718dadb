// Paged-cache tables for the ragged lengths of a verify step.
//
// Request b in seat s holds owned[s] pages, listed in page_table[s, :]; the
// free pages are a stack free_pages[0 .. free_count). For a step that appends
// n_b = offsets[b + 1] - offsets[b] tokens behind ctx_b:
//   pages_b = ceil((ctx_b + n_b) / page_size),  need_b = max(0, pages_b - owned)
//   the k-th new page of request b is free_pages[free_count - 1 - (scan_b + k)],
//   scan = exclusive scan of need in request order,
//   kv slot of its token i = page((ctx_b + i) / page_size) * page_size + (ctx_b + i) % page_size.
// Releasing pushes the pages behind ceil(keep_b / page_size) in (request, page)
// order. Both are functions of their inputs alone: no atomic decides an order.
//
// Every block repeats the checks and the scan over the B requests in shared
// memory (a few loads per thread, B <= 4096) and then takes its share of the
// tokens and of the table entries; the last block to finish writes the new
// counts, which until then all blocks read. One launch, no grid barrier.
//
// Bound by the chain of memory round trips: lengths and seats, pages held,
// table entries, the ticket. Map and release together: 64 requests of up to
// 4096 tokens 10.6 us, 1024 of up to 32,768 tokens (a million table entries)
// 14.0 us, 32 prompts of up to 8192 tokens 11.3 us. With blocks of 256
// threads, a block to 1024 table entries, the second took 35 us.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "serve.h"

namespace specv {

constexpr int kKvThreads = 1024, kKvWarps = kKvThreads / 32;
constexpr int kPiece = 256;                       // table entries of one warp's step, eight to a lane
constexpr int kPer = SPEC_MAX_B / kKvThreads;     // requests of one thread at most
constexpr int kPadding = -1, kRefused = -2;       // KvShared::seat of a request without a seat, of one outside the table

struct KvShared {
  int* off;    // [B + 1] map: offsets
  int* scan;   // [B + 1] exclusive scan of the pages needed / released
  int* ctx;    // [B] map: ctx_len
  int* own;    // [B] pages held
  int* seat;   // [B] seat; negative: nothing to do for this request (map: kPadding or kRefused)
  int* pages;  // [B] map: pages of the request after the step, -1 when refused; release: pages kept
  uint32_t *once, *twice;  // seats that some / more than one request names
};

__host__ __device__ inline size_t kv_shared_bytes(int B, int seats) {
  return sizeof(int) * (static_cast<size_t>(6) * B + 2) + 2 * sizeof(uint32_t) * ((static_cast<size_t>(seats) + 31) / 32);
}

__device__ __forceinline__ KvShared carve(int* base, int B, int seats) {
  KvShared s;
  s.off = base;
  s.scan = s.off + B + 1;
  s.ctx = s.scan + B + 1;
  s.own = s.ctx + B;
  s.seat = s.own + B;
  s.pages = s.seat + B;
  s.once = reinterpret_cast<uint32_t*>(s.pages + B);
  s.twice = s.once + (seats + 31) / 32;
  return s;
}

__device__ __forceinline__ void clear_marks(const KvShared& s, int seats) {
  for (int w = threadIdx.x; w < (seats + 31) / 32; w += kKvThreads) s.once[w] = s.twice[w] = 0u;
}
__device__ __forceinline__ void mark(const KvShared& s, int seat) {
  const uint32_t bit = 1u << (seat & 31);
  if (atomicOr(&s.once[seat >> 5], bit) & bit) atomicOr(&s.twice[seat >> 5], bit);
}
__device__ __forceinline__ bool named_twice(const KvShared& s, int seat) {
  return s.twice[seat >> 5] >> (seat & 31) & 1;
}

// Exclusive scan over the block's threads of one number each; the total goes to every thread. One barrier.
__device__ __forceinline__ int block_scan(int x, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  const int sum = s_warp[lane];  // kKvWarps == 32
  int all = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += t;
  }
  total = __shfl_sync(0xffffffffu, all, 31);
  return __shfl_sync(0xffffffffu, all - sum, warp) + incl - x;
}
static_assert(kKvWarps == 32, "block_scan: one warp scans the warps' sums");

// Last block of the grid (every thread gets the answer); resets the ticket.
__device__ __forceinline__ bool last_block(int* ticket, int* s_last) {
  if (gridDim.x == 1) return true;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    *s_last = atomicAdd(ticket, 1) == static_cast<int>(gridDim.x) - 1;
    if (*s_last) {
      *ticket = 0;
      __threadfence();
    }
  }
  __syncthreads();
  return *s_last != 0;
}

__global__ void __launch_bounds__(kKvThreads, 1) k_kv_map(const KvArgs a) {
  extern __shared__ int smem[];
  __shared__ int s_warp[kKvWarps];
  __shared__ int s_flag, s_bad, s_last, s_used;
  const int tid = threadIdx.x, lane = tid & 31, B = a.B, mp = a.p.max_pages, ps = a.p.page_size;
  const KvShared s = carve(smem, B, a.p.seats);
  if (tid == 0) s_flag = s_bad = s_used = 0;
  clear_marks(s, a.p.seats);
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int fc = a.p.free_count[0];
  const int per = (B + kKvThreads - 1) / kKvThreads, b0 = tid * per;  // the thread's requests: b0 ... b0 + per - 1
  int bad = tid == 0 && (fc < 0 || fc > a.p.n_pages), flag = 0;
  for (int k = 0; k < per; ++k) {
    const int b = b0 + k;
    if (b >= B) break;
    const int o = a.offsets[b], end = a.offsets[b + 1], ctx = a.ctx_len[b];
    int seat = a.seats ? a.seats[b] : b;
    bad |= o < 0 || end < o || end > a.N;
    if (seat < 0) {
      seat = kPadding;  // every negative seat of the caller's
    } else if (seat >= a.p.seats) {
      flag |= kFlagIndex;
      seat = kRefused;
    }
    s.off[b] = o;
    if (b == B - 1) s.off[B] = end;
    s.ctx[b] = ctx;
    s.seat[b] = seat;
    s.own[b] = seat >= 0 ? a.p.owned[seat] : 0;
    if (seat >= 0) mark(s, seat);
  }
  if (bad) s_bad = 1;
  __syncthreads();
  bad = s_bad;
  int need[kPer], mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    need[k] = 0;
    const int b = b0 + k;
    if (k >= per || b >= B) continue;
    const int seat = s.seat[b], own = s.own[b];
    int pages = -1;
    if (seat == kPadding) {
      pages = 0;  // no request here
    } else if (seat >= 0) {
      const int64_t total = static_cast<int64_t>(s.ctx[b]) + a.offsets[b + 1] - s.off[b];
      const int64_t want = (total + ps - 1) / ps;
      if (named_twice(s, seat)) flag |= kFlagIndex;
      else if (s.ctx[b] < 0 || total > 0x7fffffff || own < 0 || own > mp) flag |= kFlagLengths;
      else if (want > mp) flag |= kFlagPages;
      else {
        pages = static_cast<int>(want);
        need[k] = max(0, pages - own);
      }
    }
    if (bad) {
      pages = -1;
      need[k] = 0;
    }
    s.pages[b] = pages;
    mine += need[k];
  }
  int asked, run = block_scan(mine, s_warp, asked), used = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = b0 + k;
    if (k >= per || b >= B) continue;
    s.scan[b] = run;
    run += need[k];
    if (need[k] == 0) continue;
    if (run > fc) {  // the pages are not left; requests that need none go on
      s.pages[b] = -1;
      flag |= kFlagPages;
    } else {
      used = run;  // granted requests are those whose running total fits
    }
  }
  if (flag) atomicOr(&s_flag, flag);
  if (used) atomicMax(&s_used, used);
  __syncthreads();

  // tokens
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kKvThreads;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kKvThreads + tid; t < a.N; t += stride) {
    int64_t slot = -1;
    int pos = 0;
    if (!bad && t >= s.off[0] && t < s.off[B]) {
      int lo = 0, hi = B - 1;  // last request with offset <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.off[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int b = lo;
      if (s.pages[b] > 0) {
        pos = s.ctx[b] + static_cast<int>(t - s.off[b]);
        const int j = pos / ps;
        const int page = j < s.own[b] ? a.p.page_table[static_cast<int64_t>(s.seat[b]) * mp + j]
                                      : a.p.free_pages[fc - 1 - (s.scan[b] + j - s.own[b])];
        slot = static_cast<int64_t>(page) * ps + (pos - j * ps);
      }
    }
    a.kv_slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }

  // table entries: one warp to a piece of a request's row
  const int pieces = (mp + kPiece - 1) / kPiece;
  const int items = B * pieces, warps = gridDim.x * kKvWarps;
  for (int it = (tid >> 5) * gridDim.x + blockIdx.x; it < items; it += warps) {
    const int b = it / pieces, c = (it - b * pieces) * kPiece;
    const int own = s.own[b], end = min(s.pages[b], c + kPiece);
    const int start = a.block_table ? c : max(own, c);
    if (start >= end) continue;
    int32_t* row = a.p.page_table + static_cast<int64_t>(s.seat[b]) * mp;
    int page[kPiece / 32];
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k) {
      const int j = start + lane + 32 * k;
      if (j < end) page[k] = j < own ? row[j] : a.p.free_pages[fc - 1 - (s.scan[b] + j - own)];
    }
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k) {
      const int j = start + lane + 32 * k;
      if (j >= end) continue;
      if (j >= own) row[j] = page[k];
      if (a.block_table) a.block_table[static_cast<int64_t>(b) * mp + j] = page[k];
    }
  }

  if (!last_block(a.ticket, &s_last)) return;
  for (int k = 0; k < per; ++k) {
    const int b = b0 + k;
    if (b >= B) break;
    const int pages = s.pages[b], seat = s.seat[b];
    a.seq_len[b] = pages < 0 ? -1 : seat < 0 ? 0 : s.ctx[b] + (s.off[b + 1] - s.off[b]);
    if (seat >= 0 && pages > s.own[b]) a.p.owned[seat] = pages;
  }
  if (tid == 0) {
    if (s_used) a.p.free_count[0] = fc - s_used;
    const int f = bad ? kFlagLengths : s_flag;
    if (f) atomicOr(a.status, f);
  }
}

__global__ void __launch_bounds__(kKvThreads, 1) k_kv_release(const KvArgs a) {
  extern __shared__ int smem[];
  __shared__ int s_warp[kKvWarps];
  __shared__ int s_flag, s_last;
  const int tid = threadIdx.x, lane = tid & 31, B = a.B, mp = a.p.max_pages, ps = a.p.page_size;
  const KvShared s = carve(smem, B, a.p.seats);
  if (tid == 0) s_flag = 0;
  clear_marks(s, a.p.seats);
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int fc = a.p.free_count[0];
  const int per = (B + kKvThreads - 1) / kKvThreads, b0 = tid * per;
  int flag = 0;
  for (int k = 0; k < per; ++k) {
    const int b = b0 + k;
    if (b >= B) break;
    int seat = a.seats ? a.seats[b] : b;
    if (seat >= a.p.seats) {
      flag |= kFlagIndex;
      seat = -1;
    }
    s.seat[b] = seat;
    s.own[b] = seat >= 0 ? a.p.owned[seat] : 0;
    s.pages[b] = a.ctx_len ? a.ctx_len[b] : 0;  // tokens to keep, until it is known that they make sense
    if (seat >= 0) mark(s, seat);
  }
  __syncthreads();
  int mine = 0;
  for (int k = 0; k < per; ++k) {
    const int b = b0 + k;
    if (b >= B) break;
    const int seat = s.seat[b], keep = s.pages[b];
    int own = s.own[b], kept = 0;
    if (seat < 0) {
      own = 0;
    } else if (named_twice(s, seat)) {
      flag |= kFlagIndex;
      own = 0;
    } else if (keep < 0 || own < 0 || own > mp) {
      flag |= kFlagLengths;
      own = 0;
    } else {
      kept = static_cast<int>(min(static_cast<int64_t>(own), (static_cast<int64_t>(keep) + ps - 1) / ps));
    }
    s.own[b] = own;
    s.pages[b] = kept;
    mine += own - kept;
  }
  int back, run = block_scan(mine, s_warp, back);
  for (int k = 0; k < per; ++k) {
    const int b = b0 + k;
    if (b >= B) break;
    s.scan[b] = run;
    run += s.own[b] - s.pages[b];
  }
  if (flag) atomicOr(&s_flag, flag);
  __syncthreads();
  // more pages than the pool has room for: the tables are not this pool's, nothing moves
  const bool bad = fc < 0 || back > a.p.n_pages - fc;
  if (!bad) {
    const int pieces = (mp + kPiece - 1) / kPiece;
    const int items = B * pieces, warps = gridDim.x * kKvWarps;
    for (int it = (tid >> 5) * gridDim.x + blockIdx.x; it < items; it += warps) {
      const int b = it / pieces, c = (it - b * pieces) * kPiece;
      const int kept = s.pages[b], start = max(kept, c), end = min(s.own[b], c + kPiece);
      if (start >= end) continue;
      int32_t* row = a.p.page_table + static_cast<int64_t>(s.seat[b]) * mp;
      for (int j = start + lane; j < end; j += 32) {
        a.p.free_pages[fc + s.scan[b] + j - kept] = row[j];
        row[j] = -1;
      }
    }
  }
  if (!last_block(a.ticket, &s_last)) return;
  if (!bad)
    for (int k = 0; k < per; ++k) {
      const int b = b0 + k;
      if (b >= B) break;
      if (s.own[b] > s.pages[b]) a.p.owned[s.seat[b]] = s.pages[b];
    }
  if (tid == 0) {
    if (!bad && back) a.p.free_count[0] = fc + back;
    const int f = bad ? kFlagLengths : s_flag;
    if (f) atomicOr(a.status, f);
  }
}

namespace {

// One block per SM at most; as many as have a token for each thread or a piece of the tables for each warp.
cudaError_t launch_kv(void (*k)(KvArgs), const KvArgs& a, cudaStream_t st) {
  const size_t smem = kv_shared_bytes(a.B, a.p.seats);
  if (smem > 40 * 1024) {  // the static arrays take less than 8 KiB more
    // always the most that a call can need: another host thread may be between its own setting and launch
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kv_shared_bytes(SPEC_MAX_B, SPEC_MAX_SEATS)));
    if (e != cudaSuccess) return e;
  }
  const int64_t items = static_cast<int64_t>(a.B) * ((a.p.max_pages + kPiece - 1) / kPiece);
  const int64_t blocks = std::min<int64_t>(
      148, std::max<int64_t>((a.N + kKvThreads - 1) / kKvThreads, (items + kKvWarps - 1) / kKvWarps));
  return launch_pdl(k, dim3(static_cast<unsigned>(std::max<int64_t>(1, blocks))), dim3(kKvThreads), smem, st, a);
}

}  // namespace

cudaError_t launch_kv_map(const KvArgs& a, cudaStream_t st) { return launch_kv(k_kv_map, a, st); }
cudaError_t launch_kv_release(const KvArgs& a, cudaStream_t st) { return launch_kv(k_kv_release, a, st); }

}  // namespace specv
