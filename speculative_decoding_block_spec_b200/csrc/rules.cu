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

constexpr int kChunk = 1024;  // tokens of one warp's step over a row: 32 words of a bit table
constexpr int kListMax = 4096;
constexpr int kRowsMax = SPEC_MAX_K * (SPEC_MAX_L + 1);

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

// The -inf pattern of 16 bytes of logits.
template <int DT> __device__ __forceinline__ uint4 neg_inf16() {
  const uint32_t w = DT == 0 ? 0xff800000u : 0xff80ff80u;
  return make_uint4(w, w, w, w);
}

// Words of `allow` whose groups of E bits are all 0 keep those bits: the
// 16-byte vectors that are forbidden as a whole.
template <int E> __device__ __forceinline__ uint32_t whole_groups(uint32_t forbid) {
  uint32_t t = forbid & (forbid >> 1);
  t &= t >> 2;
  if (E == 8) t &= t >> 4;
  return t & (E == 8 ? 0x01010101u : 0x11111111u);
}

// bf16 pairs / fp32 words of a vector where the mask allows them, -inf elsewhere.
template <int DT> __device__ __forceinline__ uint4 choose(const uint4& v, uint32_t ok) {
  const uint4 f = neg_inf16<DT>();
  if constexpr (DT == 0) {
    return make_uint4(ok & 1 ? v.x : f.x, ok & 2 ? v.y : f.y, ok & 4 ? v.z : f.z, ok & 8 ? v.w : f.w);
  } else {
    auto pick = [&](uint32_t x, uint32_t b) {
      const uint32_t keep = (b & 1 ? 0xffffu : 0u) | (b & 2 ? 0xffff0000u : 0u);
      return (x & keep) | (0xff80ff80u & ~keep);
    };
    return make_uint4(pick(v.x, ok), pick(v.y, ok >> 2), pick(v.z, ok >> 4), pick(v.w, ok >> 6));
  }
}

// One warp's 1024 tokens of one row: -inf where the mask forbids and, out of
// place, the copy. `allow`: the lane's 32 tokens of the mask. 16-byte vectors
// at the output's alignment (the mask is shifted to it), elements at the ends;
// in place, vectors that are forbidden only in part are written by elements.
template <int DT, bool INPLACE>
__device__ __forceinline__ void stream_chunk(const char* src, char* dst, int span, uint32_t allow) {
  constexpr int es = Elem<DT>::kBytes, E = Elem<DT>::kPerVec, NV = kChunk / E / 32;
  const int lane = threadIdx.x & 31;
  const bool vec = INPLACE || ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  if (!vec) {
    for (int w = 0; w < 32; ++w) {
      const uint32_t ok = __shfl_sync(0xffffffffu, allow, w);
      const int o = w * 32 + lane;
      if (o >= span) continue;
      if (ok >> lane & 1) copy_x<DT>(dst, src, o);
      else store_x<DT>(dst, o, -INFINITY);
    }
    return;
  }
  const int head = min(span, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15) / es);
  const int nvec = (span - head) / E;
  uint4 v[INPLACE ? 1 : NV];
  if constexpr (!INPLACE) {
#pragma unroll
    for (int t = 0; t < NV; ++t)
      if (lane + 32 * t < nvec) v[t] = ldg16(src + (head + (lane + 32 * t) * E) * es);
  }
  uint32_t ok = allow;  // bit i: token head + 32 lane + i
  const uint32_t ends = __shfl_sync(0xffffffffu, allow, 0);
  if (head) {
    const uint32_t next = __shfl_down_sync(0xffffffffu, allow, 1);
    ok = __funnelshift_r(ok, lane == 31 ? 0xffffffffu : next, head);
  }
  const int left = span - head - 32 * lane;
  if (left < 32) ok |= left <= 0 ? 0xffffffffu : 0xffffffffu << left;
  const int from = lane / (32 / E), at = lane % (32 / E) * E;  // vector lane + 32 t: bits `at` of lane from + t * E
  if constexpr (INPLACE) {
    const uint32_t whole = whole_groups<E>(~ok);
    if (__any_sync(0xffffffffu, whole)) {
#pragma unroll
      for (int t = 0; t < NV; ++t)
        if (__shfl_sync(0xffffffffu, whole, from + t * E) >> at & 1)
          *reinterpret_cast<uint4*>(dst + (head + (lane + 32 * t) * E) * es) = neg_inf16<DT>();
    }
    for (uint32_t part = ~ok & ~(whole * ((1u << E) - 1u)); part; part &= part - 1)
      store_x<DT>(dst, head + 32 * lane + __ffs(part) - 1, -INFINITY);
    if (lane < head && !(ends >> lane & 1)) store_x<DT>(dst, lane, -INFINITY);
  } else {
    const bool plain = __all_sync(0xffffffffu, ok == 0xffffffffu);
#pragma unroll
    for (int t = 0; t < NV; ++t) {
      uint4 y = v[t];
      if (!plain) y = choose<DT>(y, __shfl_sync(0xffffffffu, ok, from + t * E) >> at);
      if (lane + 32 * t < nvec) *reinterpret_cast<uint4*>(dst + (head + (lane + 32 * t) * E) * es) = y;
    }
    const int tail = head + nvec * E, o = lane < head ? lane : tail + lane - head;  // fewer than 2 E <= 32 elements
    const int w = min(o, kChunk - 1) >> 5;
    const uint32_t mine = __shfl_sync(0xffffffffu, allow, w);
    if (o < span && (lane < head || o >= tail)) {
      if (mine >> (o & 31) & 1) copy_x<DT>(dst, src, o);
      else store_x<DT>(dst, o, -INFINITY);
    }
  }
}

// Block (x, b, z): WPT * 8192 tokens of the vocabulary in rows q0 .. q1 of
// request b.
//
// The ids of real histories crowd in the low end of the vocabulary. A block
// therefore compacts its seen tokens into a list in shared memory and hands
// them to its threads, spare threads taking further rows; a crowded tile is
// spread over the whole block, and over further blocks by rows. Tokens that
// are drafted or biased are taken out of the list and go a slower way.
template <int DT, bool INPLACE, int WPT>
__global__ void __launch_bounds__(kThreads, 6) k_logit_rules(const RulesArgs a) {
  constexpr int kTile = WPT * 32 * kThreads;
  constexpr int es = Elem<DT>::kBytes;
  __shared__ uint32_t s_word[WPT * kThreads];
  __shared__ uint16_t s_list[kListMax];
  __shared__ int64_t s_off[kRowsMax];  // first byte of a row
  __shared__ int16_t s_pos[kRowsMax];
  __shared__ int s_tok[32 + SPEC_MAX_BIAS];  // drafted tokens, then the bias list
  __shared__ float s_val[SPEC_MAX_BIAS];
  __shared__ uint16_t s_special[32 + SPEC_MAX_BIAS];
  __shared__ int s_n, s_ns;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y;
  const int64_t V = a.V, W = (V + 31) / 32;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTile, w0 = t0 / 32;
  const int span = static_cast<int>(min(static_cast<int64_t>(kTile), V - t0));
  const bool first = blockIdx.z == 0 && blockIdx.x == 0;
  if (tid == 0) s_n = s_ns = 0;
  pdl_wait();
  pdl_trigger();

  // the request: a value outside its range leaves all its rows as they were
  const int ell = a.vlen ? a.vlen[b] : a.L;
  const int64_t row0 = a.row_off ? a.row_off[b] : 0;
  const int seat = a.h.counts ? (a.seats ? a.seats[b] : b) : -1;
  const int m = a.mask ? (a.mask_rows ? a.mask_rows[b] : b) : -1;
  const bool sat = seat >= 0 && seat < a.h.seats;
  float rep = 1.f, freq = 0.f, pres = 0.f;
  uint32_t word[WPT];  // words tid, tid + 256, ... of the tile
#pragma unroll
  for (int k = 0; k < WPT; ++k) word[k] = 0u;
  if (sat) {
    if (a.h.repetition) rep = a.h.repetition[seat];
    if (a.h.frequency) freq = a.h.frequency[seat];
    if (a.h.presence) pres = a.h.presence[seat];
    const uint32_t* seen = a.h.seen + seat * W + w0;
#pragma unroll
    for (int k = 0; k < WPT; ++k)
      if ((tid + k * kThreads) * 32 < span) word[k] = seen[tid + k * kThreads];
  }
  const int nrow = ell + a.rows - a.L;
  int flag = 0;
  if (ell < 0 || ell > a.L) flag |= kFlagVerifyLen;
  else if (a.row_off && (row0 < 0 || row0 + nrow > a.n_rows)) flag |= kFlagIndex;
  if ((a.h.counts && seat >= a.h.seats) || (a.mask && m >= a.n_masks)) flag |= kFlagIndex;
  if (!(rep > 0.f && rep < INFINITY && fabsf(freq) < INFINITY && fabsf(pres) < INFINITY)) flag |= kFlagParam;
  if (flag) {
    if (first && tid == 0) atomicOr(a.status, flag);
    return;
  }
  const bool pen = sat && (rep != 1.f || freq != 0.f || pres != 0.f);
  const int n_bias = sat ? a.h.n_bias : 0, n_tok = pen ? ell : 0;
  const int q0 = blockIdx.z * a.per, nq = min(a.K * nrow, q0 + a.per) - q0;
  if (first && tid < n_tok) {
    const int x = a.tokens[static_cast<int64_t>(b) * a.L + tid];
    if (x < 0 || x >= V) atomicOr(a.status, kFlagTokenRange);
  }
  if (nq <= 0 || (INPLACE && !pen && m < 0 && n_bias == 0)) return;
  for (int q = tid; q < nq; q += kThreads) {
    const int z = (q0 + q) / nrow, i = q0 + q - z * nrow;
    const int64_t r = a.row_off ? row0 + i : (static_cast<int64_t>(b) * a.K + z) * a.rows + i;
    s_off[q] = r * V * es;
    s_pos[q] = static_cast<int16_t>(i);
  }
  const uint32_t* mask = a.mask + (m >= 0 ? static_cast<int64_t>(m) * a.mask_len * W : 0);
#pragma unroll
  for (int k = 0; k < WPT; ++k) {
    const int at = (tid + k * kThreads) * 32;
    if (!pen) word[k] = 0u;
    else if (at + 32 > span) word[k] &= at >= span ? 0u : (1u << (span - at)) - 1u;
  }

  // drafted and biased tokens of the tile: out of the list, into s_special
  if (n_tok + n_bias > 0) {
#pragma unroll
    for (int k = 0; k < WPT; ++k) s_word[tid + k * kThreads] = word[k];
  }
  __syncthreads();  // s_n, s_ns, s_off, s_pos, s_word
  if (n_tok + n_bias > 0) {
    for (int e = tid; e < 32 + n_bias; e += kThreads) {
      int x = -1;
      if (e >= 32) {
        x = a.h.bias_tokens[static_cast<int64_t>(seat) * n_bias + e - 32];
        s_val[e - 32] = a.h.bias_values[static_cast<int64_t>(seat) * n_bias + e - 32];
        if (first && x >= V) atomicOr(a.status, kFlagTokenRange);
      } else if (e < n_tok) {
        x = a.tokens[static_cast<int64_t>(b) * a.L + e];
      }
      s_tok[e] = x;
      if (x >= t0 && x < t0 + span) {
        s_special[atomicAdd(&s_ns, 1)] = static_cast<uint16_t>(e);
        atomicAnd(&s_word[(x - t0) >> 5], ~(1u << (x & 31)));
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WPT; ++k) word[k] = s_word[tid + k * kThreads];
  }
  int mine = 0;
#pragma unroll
  for (int k = 0; k < WPT; ++k) mine += __popc(word[k]);
  int rank = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, rank, o);
    if (lane >= o) rank += t;
  }
  int base = 0;
  if (lane == 31 && rank) base = atomicAdd(&s_n, rank);  // the warps' order is free: tokens are independent
  rank = __shfl_sync(0xffffffffu, base, 31) + rank - mine;

  if (!INPLACE || m >= 0) {
    for (int c = warp; c * kChunk < span; c += kWarps) {
      const int wspan = min(kChunk, span - c * kChunk);
      const int64_t w = w0 + c * 32 + lane;
      for (int q = 0; q < nq; ++q) {
        const uint32_t allow = m >= 0 && w < W ? mask[s_pos[q] * W + w] : 0xffffffffu;
        const int64_t off = s_off[q] + (t0 + c * kChunk) * es;
        stream_chunk<DT, INPLACE>(a.x + off, a.out + off, wspan, allow);
      }
    }
  }

  // the list, in rounds of kListMax tokens (one, unless the history holds most of the vocabulary)
  __syncthreads();  // s_n; out of place: the copies come before the edits
  const int n = s_n;
  for (int l0 = 0; l0 < n; l0 += kListMax) {
    if (l0) __syncthreads();
    int at = rank - l0;
#pragma unroll
    for (int k = 0; k < WPT; ++k)
      for (uint32_t left = word[k]; left; left &= left - 1, ++at)
        if (at >= 0 && at < kListMax)
          s_list[at] = static_cast<uint16_t>((tid + k * kThreads) * 32 + __ffs(left) - 1);
    __syncthreads();
    const int ln = min(kListMax, n - l0);
    for (int e0 = 0; e0 < ln; e0 += kThreads) {
      const int take = min(kThreads, ln - e0);
      const int groups = kThreads / take, sub = tid / take;
      if (sub >= groups) continue;
      const int64_t v = t0 + s_list[e0 + tid - sub * take];
      const int c = a.h.counts[seat * V + v];
      const char* x = a.x + v * es;
      char* y = a.out + v * es;
      for (int q = sub; q < nq; q += 4 * groups) {  // four rows' loads in flight
        float f[4];
        bool on[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = q + k * groups;
          on[k] = r < nq;
          if (on[k] && m >= 0) on[k] = mask[s_pos[r] * W + (v >> 5)] >> (v & 31) & 1;
          if (on[k]) f[k] = load_x<DT>(x + s_off[r], 0);
        }
        const float minus = freq * static_cast<float>(c) + (c > 0 ? pres : 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (on[k]) store_x<DT>(y + s_off[q + k * groups], 0, (f[k] > 0.f ? f[k] / rep : f[k] * rep) - minus);
      }
    }
  }

  // drafted and biased tokens: the first of the entries that name a token speaks for all, in list order
  const int ns = s_ns;
  for (int e0 = 0; e0 < ns; e0 += kThreads) {
    const int take = min(kThreads, ns - e0);
    const int groups = kThreads / take, sub = tid / take;
    if (sub >= groups) continue;
    const int self = s_special[e0 + tid - sub * take];
    const int64_t v = s_tok[self];
    uint32_t drafted = 0u;
    bool mute = false;
    for (int k = 0; k < n_tok; ++k)
      if (s_tok[k] == v) {
        drafted |= 1u << k;
        mute |= k < self;
      }
    float add = 0.f;
    for (int k = 0; k < n_bias && !mute; ++k)
      if (s_tok[32 + k] == v) {
        add += s_val[k];
        mute = 32 + k < self;
      }
    if (mute) continue;
    const bool seen = pen && (a.h.seen[seat * W + (v >> 5)] >> (v & 31) & 1);
    const int count = seen ? a.h.counts[seat * V + v] : 0;
    for (int q = sub; q < nq; q += groups) {
      const int i = s_pos[q];
      const int extra = __popc(drafted & (i >= 32 ? 0xffffffffu : (1u << i) - 1u)), c = count + extra;
      const bool known = seen || extra > 0;
      if (!known && add == 0.f) continue;
      if (m >= 0 && !(mask[i * W + (v >> 5)] >> (v & 31) & 1)) continue;
      const float f = load_x<DT>(a.x + s_off[q], v);
      const float g = known ? (f > 0.f ? f / rep : f * rep) : f;
      store_x<DT>(a.out + s_off[q], v, g - freq * static_cast<float>(c) - (c > 0 ? pres : 0.f) + add);
    }
  }
}

template <int WPT>
cudaError_t launch_tiles(RulesArgs a, int dtype, cudaStream_t st) {
  const int64_t x = (a.V + WPT * 32 * kThreads - 1) / (WPT * 32 * kThreads);
  const int most = a.K * a.rows;
  const int64_t want = 148 * 12;  // two waves of 6 blocks on 148 SMs, by splitting rows
  const int z = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, want / (x * a.B))));
  a.per = (most + z - 1) / z;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(a.B), static_cast<unsigned>((most + a.per - 1) / a.per));
  const bool inplace = a.x == a.out;
  void (*k)(RulesArgs) = dtype == 0 ? (inplace ? k_logit_rules<0, true, WPT> : k_logit_rules<0, false, WPT>)
                                    : (inplace ? k_logit_rules<1, true, WPT> : k_logit_rules<1, false, WPT>);
  return launch_pdl(k, grid, dim3(kThreads), 0, st, a);
}

cudaError_t launch_logit_rules(const RulesArgs& a, int dtype, cudaStream_t st) {
  const bool streams = a.x != a.out || a.mask;
  return streams ? launch_tiles<1>(a, dtype, st) : launch_tiles<4>(a, dtype, st);
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
