// Logit rules (penalties, biases, grammar masks) and the token history that
// the penalties read.
//
// Row i of request b with seat s, for every token v of the vocabulary:
//   c = counts[s, v] + #{k < i : x_k = v},  known = seen[s, v] or v in x_<i
//   z = known ? (x > 0 ? x / r : x * r) : x
//   z = z - f c - p [c > 0] + bias(v);  z = -inf where the mask's bit is 0
// The drafted prefix x_<i is part of the history of row i: that is the
// distribution that plain decoding would have sampled from at that position,
// so verification against the edited rows stays lossless.
//
// Only the tokens that a rule names change. In place, the kernel therefore
// reads the seen bits (V / 8 bytes per request) and edits the named elements
// alone; out of place it streams the row once and edits as it goes.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "serve.h"

namespace specv {

constexpr int kRange = 1024;          // tokens of one warp: 32 words of the bit tables, one per lane
constexpr int kRangeWords = kRange / 32;

template <int DT> __device__ __forceinline__ float load_x(const char* row, int64_t v);
template <> __device__ __forceinline__ float load_x<0>(const char* row, int64_t v) {
  return reinterpret_cast<const float*>(row)[v];
}
template <> __device__ __forceinline__ float load_x<1>(const char* row, int64_t v) {
  return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(row)[v]) << 16);
}
// bf16: one rounding to nearest even of the fp32 result (half a step, 2^-9 of the value's binade).
template <int DT> __device__ __forceinline__ void store_x(char* row, int64_t v, float z);
template <> __device__ __forceinline__ void store_x<0>(char* row, int64_t v, float z) {
  reinterpret_cast<float*>(row)[v] = z;
}
template <> __device__ __forceinline__ void store_x<1>(char* row, int64_t v, float z) {
  unsigned short h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(z));
  reinterpret_cast<unsigned short*>(row)[v] = h;
}
template <int DT> __device__ __forceinline__ void copy_x(char* out, const char* in, int64_t v) {
  if constexpr (DT == 0) reinterpret_cast<float*>(out)[v] = reinterpret_cast<const float*>(in)[v];
  else reinterpret_cast<unsigned short*>(out)[v] = reinterpret_cast<const unsigned short*>(in)[v];
}

// One warp: 1024 tokens of up to `per` rows of one request. Warps own their
// tokens alone, so nothing but __syncwarp orders the accesses.
template <int DT, bool INPLACE>
__global__ void __launch_bounds__(kThreads) k_logit_rules(const RulesArgs a) {
  extern __shared__ float s_bias_all[];  // [kWarps][kRange] when there are biases
  __shared__ uint16_t s_list_all[kWarps][kRange];
  __shared__ uint32_t s_seen_all[kWarps][32], s_draft_all[kWarps][32], s_bset_all[kWarps][32];
  __shared__ int s_tok_all[kWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRange;
  const int64_t V = a.V;
  if (t0 >= V) return;
  const int span = static_cast<int>(min(static_cast<int64_t>(kRange), V - t0));
  const int b = blockIdx.y;
  const int64_t W = (V + 31) / 32, w0 = t0 / 32;
  const bool first = t0 == 0 && blockIdx.z == 0 && lane == 0;

  // the request: a value outside its range leaves all its rows as they were
  int flag = 0;
  const int ell = a.vlen ? a.vlen[b] : a.L;
  if (ell < 0 || ell > a.L) flag |= kFlagVerifyLen;
  const int nrow = ell + a.rows - a.L;
  int64_t row0 = 0;
  if (a.row_off) {
    row0 = a.row_off[b];
    if (!flag && (row0 < 0 || row0 + nrow > a.n_rows)) flag |= kFlagIndex;
  }
  int seat = -1;
  if (a.h.counts) {
    seat = a.seats ? a.seats[b] : b;
    if (seat >= a.h.seats) flag |= kFlagIndex;
  }
  float rep = 1.f, freq = 0.f, pres = 0.f;
  if (seat >= 0 && seat < a.h.seats) {
    if (a.h.repetition) rep = a.h.repetition[seat];
    if (a.h.frequency) freq = a.h.frequency[seat];
    if (a.h.presence) pres = a.h.presence[seat];
    if (!(rep > 0.f && rep < INFINITY && fabsf(freq) < INFINITY && fabsf(pres) < INFINITY)) flag |= kFlagParam;
  }
  int m = -1;
  if (a.mask) {
    m = a.mask_rows ? a.mask_rows[b] : b;
    if (m >= a.n_masks) flag |= kFlagIndex;
  }
  if (flag) {
    if (first) atomicOr(a.status, flag);
    return;
  }
  const int total = a.K * nrow;
  const int q0 = blockIdx.z * a.per, q1 = min(total, q0 + a.per);
  const bool pen = seat >= 0 && (rep != 1.f || freq != 0.f || pres != 0.f);
  const bool bias = seat >= 0 && a.h.n_bias > 0;
  const int64_t es = Elem<DT>::kBytes;
  auto row_of = [&](int z, int i) -> int64_t {
    return a.row_off ? row0 + i : (static_cast<int64_t>(b) * a.K + z) * a.rows + i;
  };

  // the named tokens of this range: seen bits, drafted tokens, biased tokens
  uint32_t* s_seen = s_seen_all[warp];
  uint32_t* s_draft = s_draft_all[warp];
  uint32_t* s_bset = s_bset_all[warp];
  int* s_tok = s_tok_all[warp];
  uint16_t* list = s_list_all[warp];
  float* s_bias = s_bias_all + warp * kRange;
  const bool in = w0 + lane < W;
  s_seen[lane] = pen && in ? a.h.seen[seat * W + w0 + lane] : 0u;
  s_draft[lane] = 0u;
  s_bset[lane] = 0u;
  s_tok[lane] = -1;
  __syncwarp();
  if (pen && lane < a.L) {
    const int64_t x = a.tokens[static_cast<int64_t>(b) * a.L + lane];
    if (x < 0 || x >= V) {
      if (t0 == 0 && blockIdx.z == 0) atomicOr(a.status, kFlagTokenRange);
    } else if (x >= t0 && x < t0 + kRange) {
      s_tok[lane] = static_cast<int>(x - t0);
      atomicOr(&s_draft[(x - t0) >> 5], 1u << (x & 31));
    }
  }
  if (q0 >= q1) return;
  if (bias) {
    const int32_t* bt = a.h.bias_tokens + static_cast<int64_t>(seat) * a.h.n_bias;
    const float* bv = a.h.bias_values + static_cast<int64_t>(seat) * a.h.n_bias;
    for (int e0 = 0; e0 < a.h.n_bias; e0 += 32) {
      const int e = e0 + lane;
      const int64_t x = e < a.h.n_bias ? bt[e] : -1;
      if (x >= V && t0 == 0 && blockIdx.z == 0) atomicOr(a.status, kFlagTokenRange);
      const bool hit = x >= t0 && x < t0 + span;
      const float val = hit ? bv[e] : 0.f;
      // entries of one token add up in list order, whatever lane holds them
      for (uint32_t left = __ballot_sync(0xffffffffu, hit); left; left &= left - 1) {
        const int src = __ffs(left) - 1;
        const int at = __shfl_sync(0xffffffffu, static_cast<int>(x - t0), src);
        const float add = __shfl_sync(0xffffffffu, val, src);
        if (lane == 0) {
          const uint32_t bit = 1u << (at & 31);
          const bool had = s_bset[at >> 5] & bit;
          s_bias[at] = had ? s_bias[at] + add : add;
          s_bset[at >> 5] |= bit;
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  uint32_t word = s_seen[lane] | s_draft[lane] | s_bset[lane];
  if (lane * 32 + 32 > span) word &= lane * 32 >= span ? 0u : (1u << (span - lane * 32)) - 1u;
  int incl = __popc(word);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  const int n = __shfl_sync(0xffffffffu, incl, 31);
  for (int at = incl - __popc(word); word; word &= word - 1)
    list[at++] = static_cast<uint16_t>(lane * 32 + __ffs(word) - 1);
  __syncwarp();

  // rows: the mask's -inf (and the copy, out of place)
  if (!INPLACE || m >= 0) {
    for (int q = q0; q < q1; ++q) {
      const int z = q / nrow, i = q - z * nrow;
      const int64_t r = row_of(z, i);
      const char* src = a.x + (r * V + t0) * es;
      char* dst = a.out + (r * V + t0) * es;
      uint32_t allow = 0xffffffffu;
      if (m >= 0 && in) allow = a.mask[(static_cast<int64_t>(m) * a.mask_len + i) * W + w0 + lane];
      for (int w = 0; w < kRangeWords; ++w) {
        const uint32_t ok = __shfl_sync(0xffffffffu, allow, w);
        const int v = w * 32 + lane;
        if (v < span) {
          if (!(ok >> lane & 1)) store_x<DT>(dst, v, -INFINITY);
          else if (!INPLACE) copy_x<DT>(dst, src, v);
        }
      }
    }
    __syncwarp();
  }

  // the named tokens: up to 32 at a time, the lanes that are left over take further rows
  for (int e0 = 0; e0 < n; e0 += 32) {
    const int take = min(32, n - e0);
    const int groups = 32 / take;
    const int sub = lane / take, e = e0 + lane - sub * take;
    if (sub < groups) {
      const int v = list[e];
      const uint32_t bit = 1u << (v & 31);
      const bool seen = s_seen[v >> 5] & bit;
      const bool biased = s_bset[v >> 5] & bit;
      const int count = seen ? a.h.counts[seat * V + t0 + v] : 0;
      const float add = biased ? s_bias[v] : 0.f;
      uint32_t drafted = 0;
      if (s_draft[v >> 5] & bit)
        for (int k = 0; k < a.L; ++k) drafted |= (s_tok[k] == v ? 1u : 0u) << k;
      for (int q = q0 + sub; q < q1; q += groups) {
        const int z = q / nrow, i = q - z * nrow;
        const int extra = __popc(drafted & (i >= 32 ? 0xffffffffu : (1u << i) - 1u));
        const bool known = seen || extra > 0;
        if (!known && !biased) continue;
        if (m >= 0 && !(a.mask[(static_cast<int64_t>(m) * a.mask_len + i) * W + w0 + (v >> 5)] & bit)) continue;
        const int64_t r = row_of(z, i);
        const float x = load_x<DT>(a.x + (r * V + t0) * es, v);
        const int c = count + extra;
        float y = known ? (x > 0.f ? x / rep : x * rep) : x;
        y = y - freq * static_cast<float>(c) - (c > 0 ? pres : 0.f) + add;
        store_x<DT>(a.out + (r * V + t0) * es, v, y);
      }
    }
    __syncwarp();
  }
}

cudaError_t launch_logit_rules(const RulesArgs& args, int dtype, cudaStream_t st) {
  RulesArgs a = args;
  const int64_t ranges = (a.V + kRange - 1) / kRange;
  const int most = a.K * a.rows;
  a.per = 4;
  const dim3 grid(static_cast<unsigned>((ranges + kWarps - 1) / kWarps), static_cast<unsigned>(a.B),
                  static_cast<unsigned>((most + a.per - 1) / a.per));
  const size_t smem = a.h.counts && a.h.n_bias > 0 ? sizeof(float) * kRange * kWarps : 0;
  const bool inplace = a.x == a.out;
  void (*k)(RulesArgs) = dtype == 0 ? (inplace ? k_logit_rules<0, true> : k_logit_rules<0, false>)
                                    : (inplace ? k_logit_rules<1, true> : k_logit_rules<1, false>);
  if (smem) {  // with the static arrays above 48 KiB
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k, grid, dim3(kThreads), smem, st, a);
}

// ------------------------------------------------------------------ history

// counts[s, t] += 1 and seen[s, t] = 1 for every token t of the batch; integer
// atomics, so the order of the threads does not matter.
//  offsets != NULL: tokens[offsets[b] .. offsets[b + 1]) belong to request b.
//  offsets == NULL: tokens is [B, width].
// Negative tokens are padding.
__global__ void __launch_bounds__(kThreads) k_history_add(const spec_history h, const int32_t* __restrict__ seats,
                                                          int B, const int32_t* __restrict__ tokens, int64_t n,
                                                          const int32_t* __restrict__ offsets, int width, int output,
                                                          int* status) {
  extern __shared__ int s_off[];  // [B + 1]
  __shared__ int s_bad;
  pdl_wait();
  pdl_trigger();
  if (offsets) {
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    for (int b = threadIdx.x; b <= B; b += kThreads) {
      const int o = offsets[b];
      s_off[b] = o;
      if (o < 0 || o > n || (b > 0 && offsets[b - 1] > o)) s_bad = 1;
    }
    __syncthreads();
    if (s_bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, kFlagLengths);
      return;
    }
  }
  const int64_t W = (h.V + 31) / 32;
  int flag = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; t < n;
       t += static_cast<int64_t>(gridDim.x) * kThreads) {
    int b;
    if (offsets) {
      if (t < s_off[0] || t >= s_off[B]) continue;
      int lo = 0, hi = B - 1;  // last request with offset <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_off[mid] <= t) lo = mid; else hi = mid - 1;
      }
      b = lo;
    } else {
      b = static_cast<int>(t / width);
    }
    const int seat = seats ? seats[b] : b;
    const int64_t x = tokens[t];
    if (x < 0 || seat < 0) continue;
    if (seat >= h.seats) { flag |= kFlagIndex; continue; }
    if (x >= h.V) { flag |= kFlagTokenRange; continue; }
    atomicOr(h.seen + seat * W + (x >> 5), 1u << (x & 31));
    if (output) atomicAdd(h.counts + seat * h.V + x, 1);
  }
  if (flag) atomicOr(status, flag);
}

cudaError_t launch_history_add(const spec_history& h, const int32_t* seats, int B, const int32_t* tokens, int64_t n,
                               const int32_t* offsets, int width, int output, int* status, cudaStream_t st) {
  const int64_t blocks = std::min<int64_t>((n + kThreads - 1) / kThreads, 148 * 8);
  const size_t smem = offsets ? sizeof(int) * (B + 1) : 0;
  return launch_pdl(k_history_add, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), smem, st, h, seats, B, tokens, n,
                    offsets, width, output, status);
}

// Empties seats: the counts at the set bits (a count is non-zero only where the bit is set), then the bits.
__global__ void __launch_bounds__(kThreads) k_history_clear(const spec_history h, const int32_t* __restrict__ seats,
                                                            int* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int seat = seats ? seats[b] : b;
  if (seat < 0) return;
  if (seat >= h.seats) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, kFlagIndex);
    return;
  }
  const int64_t W = (h.V + 31) / 32;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  uint32_t* seen = h.seen + seat * W;
  const uint32_t word = w < W ? seen[w] : 0u;
  for (uint32_t left = __ballot_sync(0xffffffffu, word != 0); left; left &= left - 1) {
    const int src = __ffs(left) - 1;
    const uint32_t bits = __shfl_sync(0xffffffffu, word, src);
    const int64_t v = (w - lane + src) * 32 + lane;
    if ((bits >> lane & 1) && v < h.V) h.counts[seat * h.V + v] = 0;
  }
  if (word) seen[w] = 0;
}

cudaError_t launch_history_clear(const spec_history& h, const int32_t* seats, int B, int* status, cudaStream_t st) {
  const int64_t W = (h.V + 31) / 32;
  const dim3 grid(static_cast<unsigned>((W + kThreads - 1) / kThreads), static_cast<unsigned>(B));
  return launch_pdl(k_history_clear, grid, dim3(kThreads), 0, st, h, seats, status);
}

}  // namespace specv
