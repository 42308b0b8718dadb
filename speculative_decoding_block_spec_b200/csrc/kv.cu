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
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "serve.h"

namespace specv {

constexpr int kChunk = 1024;  // table entries of one work item

struct KvShared {
  int* off;    // [B + 1] map: offsets
  int* ctx;    // [B] map: ctx_len
  int* own;    // [B] pages held
  int* scan;   // [B + 1] pages needed / released, then their exclusive scan
  int* seat;   // [B] seat, or -1: nothing to do for this request
  int* pages;  // [B] map: pages of the request after the step, -1 when refused; release: pages kept
};

__host__ __device__ inline size_t kv_shared_bytes(int B, int seats) {
  return sizeof(int) * (static_cast<size_t>(6) * B + 2) + 2 * sizeof(uint32_t) * ((static_cast<size_t>(seats) + 31) / 32);
}

// Marks every seat that two requests name; returns whether request b's is one. Whole block.
__device__ __forceinline__ void mark_seats(const int* seat, int B, int seats, uint32_t* once, uint32_t* twice) {
  const int words = (seats + 31) / 32;
  for (int w = threadIdx.x; w < words; w += kThreads) once[w] = twice[w] = 0u;
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += kThreads) {
    const int s = seat[b];
    if (s < 0) continue;
    const uint32_t bit = 1u << (s & 31);
    if (atomicOr(&once[s >> 5], bit) & bit) atomicOr(&twice[s >> 5], bit);
  }
  __syncthreads();
}

// Last block of the grid (every thread gets the answer); resets the ticket.
__device__ __forceinline__ bool last_block(int* ticket, int* s_last) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const int t = atomicAdd(ticket, 1);
    *s_last = t == static_cast<int>(gridDim.x) - 1;
    if (*s_last) {
      *ticket = 0;
      __threadfence();
    }
  }
  __syncthreads();
  return *s_last != 0;
}

__device__ __forceinline__ KvShared carve(int* base, int B) {
  KvShared s;
  s.off = base;
  s.scan = s.off + B + 1;
  s.ctx = s.scan + B + 1;
  s.own = s.ctx + B;
  s.seat = s.own + B;
  s.pages = s.seat + B;
  return s;
}

__global__ void __launch_bounds__(kThreads) k_kv_map(const KvArgs a) {
  extern __shared__ int smem[];
  __shared__ int s_tmp[kWarps + 1];
  __shared__ int s_flag, s_bad, s_last;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, B = a.B, mp = a.p.max_pages, ps = a.p.page_size;
  const KvShared s = carve(smem, B);
  uint32_t* once = reinterpret_cast<uint32_t*>(s.pages + B);
  uint32_t* twice = once + (a.p.seats + 31) / 32;
  if (tid == 0) s_flag = s_bad = 0;
  __syncthreads();
  const int fc = a.p.free_count[0];
  for (int b = tid; b <= B; b += kThreads) {
    const int o = a.offsets[b];
    s.off[b] = o;
    if (o < 0 || o > a.N || (b > 0 && a.offsets[b - 1] > o)) s_bad = 1;
    if (b == B) continue;
    s.ctx[b] = a.ctx_len[b];
    int seat = a.seats ? a.seats[b] : b;
    if (seat >= a.p.seats) {
      atomicOr(&s_flag, kFlagIndex);
      seat = -2;  // refused
    }
    s.seat[b] = seat;
  }
  if (tid == 0 && (fc < 0 || fc > a.p.n_pages)) s_bad = 1;
  mark_seats(s.seat, B, a.p.seats, once, twice);
  const bool bad = s_bad != 0;
  for (int b = tid; b < B; b += kThreads) {
    const int seat = s.seat[b];
    int pages = -1, own = 0, need = 0;
    if (seat == -1) {
      pages = 0;  // no request here
    } else if (seat >= 0) {
      own = a.p.owned[seat];
      const int64_t total = static_cast<int64_t>(s.ctx[b]) + s.off[b + 1] - s.off[b];
      const int64_t want = (total + ps - 1) / ps;
      if (twice[seat >> 5] >> (seat & 31) & 1) atomicOr(&s_flag, kFlagIndex);
      else if (s.ctx[b] < 0 || total > 0x7fffffff || own < 0 || own > mp) atomicOr(&s_flag, kFlagLengths);
      else if (want > mp) atomicOr(&s_flag, kFlagPages);
      else {
        pages = static_cast<int>(want);
        need = max(0, pages - own);
      }
    }
    if (bad) pages = -1, need = 0;
    s.own[b] = own;
    s.pages[b] = pages;
    s.scan[b] = need;
  }
  __syncthreads();
  const int asked = block_exclusive_scan<kThreads>(s.scan, B, s_tmp);
  if (tid == 0) s.scan[B] = asked;
  __syncthreads();
  // a request whose pages are not left is refused; requests that need none go on
  for (int b = tid; b < B; b += kThreads)
    if (s.scan[b + 1] > s.scan[b] && s.scan[b + 1] > fc) {
      s.pages[b] = -1;
      atomicOr(&s_flag, kFlagPages);
    }
  __syncthreads();

  // tokens
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + tid; t < a.N; t += stride) {
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

  // table entries
  const int chunks = (mp + kChunk - 1) / kChunk;
  const int64_t items = static_cast<int64_t>(B) * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int b = static_cast<int>(it / chunks), c = static_cast<int>(it % chunks);
    const int own = s.own[b], end = min(s.pages[b], (c + 1) * kChunk);
    if (c * kChunk >= end) continue;
    int32_t* row = a.p.page_table + static_cast<int64_t>(s.seat[b]) * mp;
    const int start = a.block_table ? c * kChunk : max(own, c * kChunk);
    for (int j = start + tid; j < end; j += kThreads) {
      int page;
      if (j < own) {
        page = row[j];
      } else {
        page = a.p.free_pages[fc - 1 - (s.scan[b] + j - own)];
        row[j] = page;
      }
      if (a.block_table) a.block_table[static_cast<int64_t>(b) * mp + j] = page;
    }
  }

  if (!last_block(a.ticket, &s_last)) return;
  int used = 0;
  for (int b = tid; b < B; b += kThreads) {
    const int pages = s.pages[b];
    const bool ok = pages >= 0;
    a.seq_len[b] = !ok ? -1 : s.seat[b] < 0 ? 0 : s.ctx[b] + (s.off[b + 1] - s.off[b]);
    if (ok && s.seat[b] >= 0 && pages > s.own[b]) {
      a.p.owned[s.seat[b]] = pages;
      used = max(used, s.scan[b + 1]);  // granted requests are those whose running total fits
    }
  }
  if (tid == 0) s_last = 0;
  __syncthreads();
  if (used) atomicMax(&s_last, used);
  __syncthreads();
  if (tid == 0) {
    if (s_last) a.p.free_count[0] = fc - s_last;
    const int flag = bad ? kFlagLengths : s_flag;
    if (flag) atomicOr(a.status, flag);
  }
}

__global__ void __launch_bounds__(kThreads) k_kv_release(const KvArgs a) {
  extern __shared__ int smem[];
  __shared__ int s_tmp[kWarps + 1];
  __shared__ int s_flag, s_last;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, B = a.B, mp = a.p.max_pages, ps = a.p.page_size;
  const KvShared s = carve(smem, B);
  uint32_t* once = reinterpret_cast<uint32_t*>(s.pages + B);
  uint32_t* twice = once + (a.p.seats + 31) / 32;
  if (tid == 0) s_flag = 0;
  __syncthreads();
  const int fc = a.p.free_count[0];
  for (int b = tid; b < B; b += kThreads) {
    int seat = a.seats ? a.seats[b] : b;
    if (seat >= a.p.seats) {
      atomicOr(&s_flag, kFlagIndex);
      seat = -1;
    }
    s.seat[b] = seat;
  }
  __syncthreads();
  mark_seats(s.seat, B, a.p.seats, once, twice);
  for (int b = tid; b < B; b += kThreads) {
    const int seat = s.seat[b];
    int own = 0, kept = 0;
    if (seat >= 0) {
      own = a.p.owned[seat];
      const int keep = a.ctx_len ? a.ctx_len[b] : 0;
      if (twice[seat >> 5] >> (seat & 31) & 1) {
        atomicOr(&s_flag, kFlagIndex);
        own = 0;
      } else if (keep < 0 || own < 0 || own > mp) {
        atomicOr(&s_flag, kFlagLengths);
        own = 0;
      } else {
        kept = static_cast<int>(min(static_cast<int64_t>(own), (static_cast<int64_t>(keep) + ps - 1) / ps));
      }
    }
    s.own[b] = own;
    s.pages[b] = kept;
    s.scan[b] = own - kept;
  }
  __syncthreads();
  const int back = block_exclusive_scan<kThreads>(s.scan, B, s_tmp);
  // more pages than the pool has room for: the tables are not this pool's, nothing moves
  const bool bad = fc < 0 || back > a.p.n_pages - fc;
  if (!bad) {
    const int chunks = (mp + kChunk - 1) / kChunk;
    const int64_t items = static_cast<int64_t>(B) * chunks;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
      const int b = static_cast<int>(it / chunks), c = static_cast<int>(it % chunks);
      const int kept = s.pages[b], start = max(kept, c * kChunk), end = min(s.own[b], (c + 1) * kChunk);
      int32_t* row = a.p.page_table + static_cast<int64_t>(s.seat[b]) * mp;
      for (int j = start + tid; j < end; j += kThreads) {
        a.p.free_pages[fc + s.scan[b] + j - kept] = row[j];
        row[j] = -1;
      }
    }
  }
  if (!last_block(a.ticket, &s_last)) return;
  if (!bad)
    for (int b = tid; b < B; b += kThreads)
      if (s.own[b] > s.pages[b]) a.p.owned[s.seat[b]] = s.pages[b];
  if (tid == 0) {
    if (!bad && back) a.p.free_count[0] = fc + back;
    const int flag = bad ? kFlagLengths : s_flag;
    if (flag) atomicOr(a.status, flag);
  }
}

namespace {

cudaError_t allow_shared(void (*k)(KvArgs), size_t smem) {
  if (smem <= 40 * 1024) return cudaSuccess;  // the static arrays take less than 8 KiB more
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
}

}  // namespace

cudaError_t launch_kv_map(const KvArgs& a, cudaStream_t st) {
  const size_t smem = kv_shared_bytes(a.B, a.p.seats);
  const cudaError_t e = allow_shared(k_kv_map, smem);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.B) * ((a.p.max_pages + kChunk - 1) / kChunk);
  const int64_t blocks = std::min<int64_t>(148, std::max<int64_t>({1, (a.N + kThreads - 1) / kThreads, items}));
  return launch_pdl(k_kv_map, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), smem, st, a);
}

cudaError_t launch_kv_release(const KvArgs& a, cudaStream_t st) {
  const size_t smem = kv_shared_bytes(a.B, a.p.seats);
  const cudaError_t e = allow_shared(k_kv_release, smem);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.B) * ((a.p.max_pages + kChunk - 1) / kChunk);
  const int64_t blocks = std::min<int64_t>(148, std::max<int64_t>(1, items));
  return launch_pdl(k_kv_release, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), smem, st, a);
}

}  // namespace specv
