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

constexpr int kTile = 32 * kThreads;   // tokens of one block: one word of the bit tables per thread
constexpr int kWarpTile = 32 * 32;     // of one warp
constexpr int kRowsMax = SPEC_MAX_K * (SPEC_MAX_L + 1);
static_assert(SPEC_MAX_BIAS * 8 <= kTile * 2, "the bias list is staged in the token list's shared memory");

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

// One warp's 1024 tokens of one row: out of place the copy, and -inf where the
// mask forbids. `allow` and `skip` are the lane's words of the mask and of the
// tokens that another block writes (out of place only). Whole 16-byte vectors
// of the output's alignment, single elements at both ends.
template <int DT, bool INPLACE>
__device__ __forceinline__ void stream_row(const char* src, char* dst, int span, uint32_t allow, uint32_t skip) {
  constexpr int es = Elem<DT>::kBytes, E = Elem<DT>::kPerVec;
  const int lane = threadIdx.x & 31;
  const bool vec = INPLACE || ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  const int head = vec ? min(span, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15) / es) : span;
  const int nvec = (span - head) / E;
  uint4 v[kWarpTile / E / 32];
  if constexpr (!INPLACE) {
#pragma unroll
    for (int t = 0; t < kWarpTile / E / 32; ++t)
      if (lane + 32 * t < nvec) v[t] = ldg16(src + (head + (lane + 32 * t) * E) * es);
  }
  skip &= allow;  // a forbidden token is -inf whoever owns it
  const bool plain = __all_sync(0xffffffffu, allow == 0xffffffffu && skip == 0u);
  if (INPLACE && plain) return;
#pragma unroll
  for (int t = 0; t < kWarpTile / E / 32; ++t) {
    const int j = lane + 32 * t, o = min(head + j * E, kWarpTile - 1);
    uint32_t ok = (1u << E) - 1u, no = 0u;
    if (!plain) {  // bits o ... o + E - 1 of the warp's 32 words
      const int w = o >> 5, w1 = min(w + 1, 31);
      ok &= __funnelshift_r(__shfl_sync(0xffffffffu, allow, w), __shfl_sync(0xffffffffu, allow, w1), o & 31);
      if constexpr (!INPLACE)
        no = ((1u << E) - 1u) &
             __funnelshift_r(__shfl_sync(0xffffffffu, skip, w), __shfl_sync(0xffffffffu, skip, w1), o & 31);
    }
    if (j >= nvec) continue;
    char* at = dst + o * es;
    if (ok == 0u) {
      *reinterpret_cast<uint4*>(at) = neg_inf16<DT>();
    } else if (ok == (1u << E) - 1u && no == 0u) {
      if constexpr (!INPLACE) *reinterpret_cast<uint4*>(at) = v[t];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (!(ok >> e & 1)) store_x<DT>(at, e, -INFINITY);
        else if (!INPLACE && !(no >> e & 1)) copy_x<DT>(at, src + o * es, e);
      }
    }
  }
  // the elements before the first and behind the last vector
  const int tail = head + nvec * E;
  for (int k0 = 0; k0 < head + span - tail; k0 += 32) {
    const int k = k0 + lane, o = k < head ? k : tail + k - head;
    const bool in = o < span;
    const int w = min(o, kWarpTile - 1) >> 5;
    const uint32_t ok = __shfl_sync(0xffffffffu, allow, w), no = __shfl_sync(0xffffffffu, skip, w);
    if (!in) continue;
    if (!(ok >> (o & 31) & 1)) store_x<DT>(dst, o, -INFINITY);
    else if (!INPLACE && !(no >> (o & 31) & 1)) copy_x<DT>(dst, src, o);
  }
}

// Blocks (x, b, z): 8192 tokens of the vocabulary (or, behind those, 256
// entries of the request's bias list) in rows q0 .. q1 of request b. A token
// with a bias belongs to the bias block, every other one to its tile's block.
//
// A tile's block compacts its named tokens (seen or drafted) into a list in
// shared memory and hands them to the threads, spare threads taking further
// rows: the ids of real histories crowd in a few tiles, and the list spreads a
// crowded tile over the whole block.
template <int DT, bool INPLACE>
__global__ void __launch_bounds__(kThreads) k_logit_rules(const RulesArgs a) {
  __shared__ __align__(16) uint16_t s_list[kTile];
  __shared__ uint32_t s_draft[kThreads], s_excl[kThreads];
  __shared__ int s_tok[32];
  __shared__ int64_t s_row[kRowsMax];
  __shared__ int16_t s_pos[kRowsMax];
  __shared__ int s_n;
  constexpr int es = Elem<DT>::kBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y;
  const int64_t V = a.V, W = (V + 31) / 32;
  const int tiles = static_cast<int>((V + kTile - 1) / kTile);
  const bool bias_block = static_cast<int>(blockIdx.x) >= tiles;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTile, w0 = t0 / 32;
  const bool first = blockIdx.z == 0 && blockIdx.x == 0;
  s_draft[tid] = s_excl[tid] = 0u;
  if (tid < 32) s_tok[tid] = -1;
  if (tid == 0) s_n = 0;
  pdl_wait();
  pdl_trigger();

  // the request: a value outside its range leaves all its rows as they were
  const int ell = a.vlen ? a.vlen[b] : a.L;
  const int64_t row0 = a.row_off ? a.row_off[b] : 0;
  const int seat = a.h.counts ? (a.seats ? a.seats[b] : b) : -1;
  const int m = a.mask ? (a.mask_rows ? a.mask_rows[b] : b) : -1;
  const bool sat = seat >= 0 && seat < a.h.seats;
  float rep = 1.f, freq = 0.f, pres = 0.f;
  uint32_t seen = 0u;
  if (sat) {
    if (a.h.repetition) rep = a.h.repetition[seat];
    if (a.h.frequency) freq = a.h.frequency[seat];
    if (a.h.presence) pres = a.h.presence[seat];
    if (!bias_block && w0 + tid < W) seen = a.h.seen[seat * W + w0 + tid];
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
  const int n_bias = sat ? a.h.n_bias : 0;
  const int q0 = blockIdx.z * a.per, q1 = min(a.K * nrow, q0 + a.per), nq = q1 - q0;
  if (pen && first && tid < ell) {
    const int x = a.tokens[static_cast<int64_t>(b) * a.L + tid];
    if (x < 0 || x >= V) atomicOr(a.status, kFlagTokenRange);
  }
  if (nq <= 0 || (INPLACE && !pen && m < 0 && !bias_block)) return;
  for (int q = tid; q < nq; q += kThreads) {
    const int z = (q0 + q) / nrow, i = q0 + q - z * nrow;
    s_row[q] = a.row_off ? row0 + i : (static_cast<int64_t>(b) * a.K + z) * a.rows + i;
    s_pos[q] = static_cast<int16_t>(i);
  }
  const uint32_t* mask = a.mask + (m >= 0 ? static_cast<int64_t>(m) * a.mask_len * W : 0);

  // the value of token v (named, known to the rules by count0 / add / drafted) in row q, and whether it changes
  auto edit = [&](float x, bool was_seen, int count0, uint32_t drafted, float add, int i) -> float {
    const int extra = __popc(drafted & (i >= 32 ? 0xffffffffu : (1u << i) - 1u));
    const int c = count0 + extra;
    float y = was_seen || extra > 0 ? (x > 0.f ? x / rep : x * rep) : x;
    return y - freq * static_cast<float>(c) - (c > 0 ? pres : 0.f) + add;
  };
  // all rows of one token for the threads sub, sub + groups, ...: four rows' loads in flight
  auto rows_of = [&](int64_t v, int sub, int groups, bool was_seen, uint32_t drafted, float add, bool biased) {
    const int count0 = was_seen ? a.h.counts[seat * V + v] : 0;
    const uint32_t bit = 1u << (v & 31);
    for (int q = sub; q < nq; q += 4 * groups) {
      float x[4];
      bool on[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = q + k * groups;
        on[k] = r < nq;
        if (!on[k]) continue;
        const int i = s_pos[r];
        if (!was_seen && !biased && !(drafted & (i >= 32 ? 0xffffffffu : (1u << i) - 1u))) on[k] = false;
        else if (m >= 0) on[k] = mask[i * W + (v >> 5)] & bit;
        if (on[k]) x[k] = load_x<DT>(a.x + s_row[r] * V * es, v);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (on[k]) store_x<DT>(a.out + s_row[q + k * groups] * V * es, v,
                               edit(x[k], was_seen, count0, drafted, add, s_pos[q + k * groups]));
    }
  };
  auto drafted_of = [&](int64_t v) -> uint32_t {
    uint32_t d = 0;
    for (int k = 0; k < ell; ++k) d |= (s_tok[k] == v ? 1u : 0u) << k;
    return d;
  };

  if (bias_block) {
    int* tok = reinterpret_cast<int*>(s_list);
    float* val = reinterpret_cast<float*>(s_list) + SPEC_MAX_BIAS;
    for (int e = tid; e < n_bias; e += kThreads) {
      tok[e] = a.h.bias_tokens[static_cast<int64_t>(seat) * n_bias + e];
      val[e] = a.h.bias_values[static_cast<int64_t>(seat) * n_bias + e];
      if (tok[e] >= V && blockIdx.z == 0) atomicOr(a.status, kFlagTokenRange);
    }
    if (pen && tid < ell) s_tok[tid] = a.tokens[static_cast<int64_t>(b) * a.L + tid];
    __syncthreads();
    const int e0 = (static_cast<int>(blockIdx.x) - tiles) * kThreads;
    const int take = min(kThreads, n_bias - e0);
    if (take <= 0) return;
    const int groups = kThreads / take, sub = tid / take, e = e0 + tid - sub * take;
    if (sub >= groups) return;
    const int v = tok[e];
    if (v < 0 || v >= V) return;
    // the first entry of a token speaks for all of them and adds them up in list order
    float add = 0.f;
    for (int k = 0; k < n_bias; ++k) {
      if (tok[k] != v) continue;
      if (k < e) return;
      add += val[k];
    }
    const bool was_seen = pen && (a.h.seen[seat * W + (v >> 5)] >> (v & 31) & 1);
    rows_of(v, sub, groups, was_seen, pen ? drafted_of(v) : 0u, add, true);
    return;
  }

  const int span = static_cast<int>(min(static_cast<int64_t>(kTile), V - t0));
  __syncthreads();
  if (pen && tid < ell) {  // the drafted tokens that a processed row can hold
    const int64_t x = a.tokens[static_cast<int64_t>(b) * a.L + tid];
    if (x >= t0 && x < t0 + span) {
      s_tok[tid] = static_cast<int>(x);
      atomicOr(&s_draft[(x - t0) >> 5], 1u << (x & 31));
    }
  }
  for (int e = tid; e < n_bias; e += kThreads) {
    const int64_t x = a.h.bias_tokens[static_cast<int64_t>(seat) * n_bias + e];
    if (x >= t0 && x < t0 + span) atomicOr(&s_excl[(x - t0) >> 5], 1u << (x & 31));
  }
  __syncthreads();
  if (pen) {
    uint32_t word = (seen | s_draft[tid]) & ~s_excl[tid];
    if (tid * 32 + 32 > span) word &= tid * 32 >= span ? 0u : (1u << (span - tid * 32)) - 1u;
    const int mine = __popc(word);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    int at = 0;
    if (lane == 31) at = atomicAdd(&s_n, incl);  // the warps' order in the list is free: tokens are independent
    at = __shfl_sync(0xffffffffu, at, 31) + incl - mine;
    for (uint32_t left = word; left; left &= left - 1)
      s_list[at++] = static_cast<uint16_t>(tid * 32 + __ffs(left) - 1);
  }
  // seen bits of the list's tokens, for the threads that take them
  const uint32_t excl = s_excl[tid];
  __syncthreads();
  s_excl[tid] = seen;
  if (!INPLACE || m >= 0) {
    const int wspan = min(kWarpTile, span - warp * kWarpTile);
    if (wspan > 0) {
      const int64_t at = t0 + warp * kWarpTile;
      for (int q = 0; q < nq; ++q) {
        uint32_t allow = 0xffffffffu;
        if (m >= 0 && w0 + tid < W) allow = mask[s_pos[q] * W + w0 + tid];
        const int64_t off = (s_row[q] * V + at) * es;
        stream_row<DT, INPLACE>(a.x + off, a.out + off, wspan, allow, excl);
      }
    }
  }
  __syncthreads();  // out of place: the copies come before the edits
  const int n = s_n;
  for (int e0 = 0; e0 < n; e0 += kThreads) {
    const int take = min(kThreads, n - e0);
    const int groups = kThreads / take, sub = tid / take;
    if (sub >= groups) continue;
    const int v = s_list[e0 + tid - sub * take];
    const uint32_t bit = 1u << (v & 31);
    rows_of(t0 + v, sub, groups, s_excl[v >> 5] & bit, s_draft[v >> 5] & bit ? drafted_of(t0 + v) : 0u, 0.f, false);
  }
}

cudaError_t launch_logit_rules(const RulesArgs& args, int dtype, cudaStream_t st) {
  RulesArgs a = args;
  const int64_t tiles = (a.V + kTile - 1) / kTile;
  const int n_bias = a.h.counts ? a.h.n_bias : 0;
  const int64_t x = tiles + (n_bias + kThreads - 1) / kThreads;
  const int most = a.K * a.rows;
  // Rows are split over blocks until the grid fills the GPU twice (148 SMs of 8 blocks).
  const int64_t want = 148 * 16;
  const int z = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, want / (x * a.B))));
  a.per = (most + z - 1) / z;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(a.B), static_cast<unsigned>((most + a.per - 1) / a.per));
  const bool inplace = a.x == a.out;
  void (*k)(RulesArgs) = dtype == 0 ? (inplace ? k_logit_rules<0, true> : k_logit_rules<0, false>)
                                    : (inplace ? k_logit_rules<1, true> : k_logit_rules<1, false>);
  return launch_pdl(k, grid, dim3(kThreads), 0, st, a);
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
