// Logit rules (penalties, biases, grammar masks) and the token history that
// the penalties read.
//
// Row i of request b with seat s, for every token v of the vocabulary:
//   c = counts[s, v] + #{k < i : x_k = v},  known = seen[s, v] or v in x_<i
//   z = known ? (x > 0 ? x / r : x * r) : x
//   z = z - f c - p [c > 0] + bias(v);  z = -inf where the mask's bit is 0
// The drafted prefix x_<i is part of the history of row i: the edited target
// row is the distribution that plain decoding would have sampled from at that
// position. Verification keeps it for any proposal q, as long as q is the one
// that x_i was drawn from: draft rows are edited only where the drafter itself
// drew x_i from the row edited with x_<i.
//
// Only the tokens that a rule names change. Two kernels, each launched where
// it has work:
//  k_rules_stream  what touches whole rows: the mask's -inf, and the copy out
//    of place. Bound by HBM: 544 rows of 151,936 bf16 tokens are copied in
//    54.4 us (6.1 TB/s, a plain copy 51.5) and overwritten with -inf in 30.
//  k_rules_edit    the named elements. It reads the seen bits (V / 8 bytes a
//    request) and the counts and logits that they name. Its time goes into
//    waiting for scattered loads: 2048 draft rows with about 1000 named tokens
//    each take 53 us, in which DRAM delivers 117 MB for 4 MB of elements, at
//    38 % of its rate. With r = 1 only counted, drafted and biased tokens are
//    written: 39 us. Ids spread evenly share fewer lines: 118 and 79 us.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "serve.h"

namespace specv {

constexpr int kChunk = 1024;  // tokens of one warp's step over a row: 32 words of a bit table
constexpr int kEditThreads = 512;
constexpr int kEditTile = 10 * 32 * kEditThreads;  // tokens of the edit kernel's tile: 163,840
constexpr int kListMax = 4096;  // seen tokens that are taken at a time
constexpr float kRepMin = 0x1p-100f;  // 2^-100 <= r <= 2^100: 1 / r is a normal number
constexpr int kRowsMax = SPEC_MAX_K * (SPEC_MAX_L + 1);

template <int DT> __device__ __forceinline__ float load_x(const char* row, int64_t v);
template <> __device__ __forceinline__ float load_x<0>(const char* row, int64_t v) {
  return reinterpret_cast<const float*>(row)[v];
}
template <> __device__ __forceinline__ float load_x<1>(const char* row, int64_t v) {
  return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(row)[v]) << 16);
}
// bf16: one rounding to nearest even of the fp32 result, at most 2^-8 of the value.
template <int DT> __device__ __forceinline__ void store_x(char* row, int64_t v, float z);
template <> __device__ __forceinline__ void store_x<0>(char* row, int64_t v, float z) {
  reinterpret_cast<float*>(row)[v] = z;
}
template <> __device__ __forceinline__ void store_x<1>(char* row, int64_t v, float z) {
  unsigned short h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(z));
  reinterpret_cast<unsigned short*>(row)[v] = h;
}
template <int DT> struct Bits { using type = uint32_t; };  // elements that are moved, not computed, keep their bits
template <> struct Bits<1> { using type = unsigned short; };
template <int DT> __device__ __forceinline__ void copy_x(char* out, const char* in, int64_t v) {
  using Raw = typename Bits<DT>::type;
  reinterpret_cast<Raw*>(out)[v] = reinterpret_cast<const Raw*>(in)[v];
}

// The -inf pattern of 16 bytes of logits.
template <int DT> __device__ __forceinline__ uint4 neg_inf16() {
  const uint32_t w = DT == 0 ? 0xff800000u : 0xff80ff80u;
  return make_uint4(w, w, w, w);
}

// The lowest bit of every group of E bits of `forbid` that is all ones: the
// 16-byte vectors that are forbidden whole.
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

// In place, vectors that the mask forbids in part, read, changed and written
// back (their other elements are this warp's alone). Kept out of line: few
// masks need it, and it would cost the others registers.
template <int DT>
__device__ __noinline__ void mask_partial(char* dst, int nvec, uint32_t ok) {
  constexpr int E = Elem<DT>::kPerVec;
  const int lane = threadIdx.x & 31;
  for (int t = 0; t < kChunk / E / 32; ++t) {
    const uint32_t g = __shfl_sync(0xffffffffu, ok, lane / (32 / E) + t * E) >> (lane % (32 / E) * E) & ((1u << E) - 1u);
    uint4* at = reinterpret_cast<uint4*>(dst + t * 32 * 16);
    if (lane + 32 * t < nvec && g != 0u && g != (1u << E) - 1u) *at = choose<DT>(*at, g);
  }
}

// One warp's 1024 tokens of one row: -inf where the mask forbids and, out of
// place, the copy. `allow`: the lane's 32 tokens of the mask. 16-byte vectors
// at the output's alignment (the mask is shifted to it), elements at the ends.
//
// In place, vectors that are forbidden whole are stored whole, and those that
// are forbidden in part by elements while a lane has at most kPops stores to
// make, else by reading them. 544 rows of 151,936 bf16 tokens, us:
//   forbidden            by elements   by reading
//   2 % at random             34           59
//   all but 100 tokens        37           41
//   half, at random          217           72
template <int DT, bool INPLACE>
__device__ __forceinline__ void stream_chunk(const char* src, char* dst, int span, uint32_t allow) {
  constexpr int es = Elem<DT>::kBytes, E = Elem<DT>::kPerVec, NV = kChunk / E / 32, kPops = 8;
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
  if (INPLACE && __all_sync(0xffffffffu, allow == 0xffffffffu)) return;
  const int head = min(span, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15) / es);
  const int nvec = (span - head) / E;
  src += (head + lane * E) * es;  // the lane's first vector
  dst += (head + lane * E) * es;
  constexpr int kStep = 32 * 16, kFly = 4;  // bytes from vector to vector; vectors in flight per lane
  if (INPLACE && head == 0 && span == kChunk && __all_sync(0xffffffffu, allow == 0u)) {
#pragma unroll
    for (int t = 0; t < NV; ++t) *reinterpret_cast<uint4*>(dst + t * kStep) = neg_inf16<DT>();
    return;
  }
  uint4 v[kFly];
  if constexpr (!INPLACE) {
#pragma unroll
    for (int t = 0; t < kFly; ++t)
      if (lane + 32 * t < nvec) v[t] = ldg16(src + t * kStep);
  }
  uint32_t ok = allow;  // bit i: token head + 32 lane + i
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
          *reinterpret_cast<uint4*>(dst + t * kStep) = neg_inf16<DT>();
    }
    uint32_t part = ~ok & ~(whole * ((1u << E) - 1u));
    uint32_t two = DT == 1 ? part & part >> 1 & 0x55555555u : 0u;  // aligned bf16 pairs
    if (__any_sync(0xffffffffu, __popc(part) - __popc(two) > kPops)) {
      mask_partial<DT>(dst, nvec, ok);
      // what is left are the elements behind the last vector
      const int behind = nvec * E - 32 * lane;
      part &= behind >= 32 ? 0u : behind <= 0 ? 0xffffffffu : 0xffffffffu << behind;
      two &= part;  // a pair lies on one side: nvec * E is even
    }
    char* own = dst + 32 * lane * es - lane * 16;  // the lane's 32 tokens
    part &= ~(two * 3u);
    for (; two; two &= two - 1) *reinterpret_cast<uint32_t*>(own + (__ffs(two) - 1) * es) = 0xff80ff80u;
    for (; part; part &= part - 1) store_x<DT>(own, __ffs(part) - 1, -INFINITY);
    if (head) {
      const uint32_t ends = __shfl_sync(0xffffffffu, allow, 0);
      if (lane < head && !(ends >> lane & 1)) store_x<DT>(dst, lane - head - lane * E, -INFINITY);
    }
  } else {
    const bool plain = __all_sync(0xffffffffu, ok == 0xffffffffu);
#pragma unroll
    for (int t0 = 0; t0 < NV; t0 += kFly) {
#pragma unroll
      for (int t = 0; t < kFly; ++t) {
        uint4 y = v[t];
        if (!plain) y = choose<DT>(y, __shfl_sync(0xffffffffu, ok, from + (t0 + t) * E) >> at);
        if (lane + 32 * (t0 + t) < nvec) *reinterpret_cast<uint4*>(dst + (t0 + t) * kStep) = y;
        if (t0 + kFly < NV && lane + 32 * (t0 + kFly + t) < nvec) v[t] = ldg16(src + (t0 + kFly + t) * kStep);
      }
    }
    // elements before the first and behind the last vector: fewer than 2 E <= 16, one to a lane
    const int tail = head + nvec * E, o = lane < head ? lane : tail + lane - head;
    const uint32_t mine = __shfl_sync(0xffffffffu, allow, min(o, kChunk - 1) >> 5);
    if (o < span) {
      const int rel = o - head - lane * E;
      if (mine >> (o & 31) & 1) copy_x<DT>(dst, src, rel);
      else store_x<DT>(dst, rel, -INFINITY);
    }
  }
}

// What a block needs to know of its request. A value outside its range leaves
// all the request's rows as they were; `flag` says which it was.
struct Request {
  int nrow, ell, seat, m, flag;
  int64_t row0;
  float rep, freq, pres;
  bool sat, pen;
};
__device__ __forceinline__ Request load_request(const RulesArgs& a, int b) {
  Request r;
  r.ell = a.vlen ? a.vlen[b] : a.L;
  r.row0 = a.row_off ? a.row_off[b] : 0;
  r.seat = a.h.counts ? (a.seats ? a.seats[b] : b) : -1;
  r.m = a.mask ? (a.mask_rows ? a.mask_rows[b] : b) : -1;
  r.sat = r.seat >= 0 && r.seat < a.h.seats;
  r.rep = 1.f;
  r.freq = r.pres = 0.f;
  if (r.sat) {
    if (a.h.repetition) r.rep = a.h.repetition[r.seat];
    if (a.h.frequency) r.freq = a.h.frequency[r.seat];
    if (a.h.presence) r.pres = a.h.presence[r.seat];
  }
  r.nrow = r.ell + a.rows - a.L;
  r.flag = 0;
  if (r.ell < 0 || r.ell > a.L) r.flag |= kFlagVerifyLen;
  else if (a.row_off && (r.row0 < 0 || r.row0 + r.nrow > a.n_rows)) r.flag |= kFlagIndex;
  if ((a.h.counts && r.seat >= a.h.seats) || (a.mask && r.m >= a.n_masks)) r.flag |= kFlagIndex;
  if (!(r.rep >= kRepMin && r.rep <= 1.f / kRepMin && fabsf(r.freq) < INFINITY && fabsf(r.pres) < INFINITY))
    r.flag |= kFlagParam;
  r.pen = r.sat && (r.rep != 1.f || r.freq != 0.f || r.pres != 0.f);
  return r;
}
// First byte of row q of the request, q = z * nrow + i (z: branch); i is the position.
template <int DT>
__device__ __forceinline__ int64_t row_byte(const RulesArgs& a, const Request& r, int b, int q, int& i) {
  const int z = q / r.nrow;
  i = q - z * r.nrow;
  const int64_t row = a.row_off ? r.row0 + i : (static_cast<int64_t>(b) * a.K + z) * a.rows + i;
  return row * a.V * Elem<DT>::kBytes;
}

// Block (x, b, q): chunks x * per ... of row q of request b, one after the
// other to its warps, the masks of the next four chunks on their way.
template <int DT, bool INPLACE>
__global__ void __launch_bounds__(kThreads, 6) k_rules_stream(const RulesArgs a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const Request r = load_request(a, b);
  if (r.flag) {
    if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) atomicOr(a.status, r.flag);
    return;
  }
  const int q = blockIdx.z;
  if (q >= a.K * r.nrow || (INPLACE && r.m < 0)) return;
  int i;
  const int64_t row = row_byte<DT>(a, r, b, q, i);
  const int chunks = static_cast<int>((a.V + kChunk - 1) / kChunk);
  const int end = min(chunks, (static_cast<int>(blockIdx.x) + 1) * a.per);
  int c = blockIdx.x * a.per + (threadIdx.x >> 5);
  const int W = static_cast<int>((a.V + 31) / 32);
  const uint32_t* mask = a.mask + (static_cast<int64_t>(r.m) * a.mask_len + i) * W;
  auto allowed = [&](int chunk) {
    const int w = chunk * 32 + lane;
    return r.m >= 0 && chunk < end && w < W ? mask[w] : 0xffffffffu;
  };
  uint32_t allow[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) allow[k] = allowed(c + k * kWarps);
#pragma unroll 1
  for (; c < end; c += kWarps) {
    const int64_t t0 = static_cast<int64_t>(c) * kChunk, off = row + t0 * Elem<DT>::kBytes;
    const uint32_t now = allow[0];
    allow[0] = allow[1];
    allow[1] = allow[2];
    allow[2] = allow[3];
    allow[3] = allowed(c + 4 * kWarps);
    stream_chunk<DT, INPLACE>(a.x + off, a.out + off, static_cast<int>(min(static_cast<int64_t>(kChunk), a.V - t0)), now);
  }
}

// The drafted and biased tokens of a request ("special"), in dynamic shared
// memory: entry e < 32 is drafted token e, entry 32 + k bias entry k.
struct Special {
  int* v;             // token, relative to the tile; negative: not in it
  float* add;         // bias value; an owner's: the sum of its token's
  uint32_t* drafted;  // an owner's: bit k, drafted at position k
  int* count;         // an owner's: its count, -1 when not seen
  int* twice;         // entries whose token another one had named already
  uint16_t* owner;    // entries that speak for their token
};
constexpr int kSpecialBytes = 5 * 4 + 2;
__device__ __forceinline__ Special carve_special(char* base, int n) {
  Special s;
  s.v = reinterpret_cast<int*>(base);
  s.add = reinterpret_cast<float*>(s.v + n);
  s.drafted = reinterpret_cast<uint32_t*>(s.add + n);
  s.count = reinterpret_cast<int*>(s.drafted + n);
  s.twice = s.count + n;
  s.owner = reinterpret_cast<uint16_t*>(s.twice + n);
  return s;
}

// Block (b, z): rows q0 .. q1 of request b over the whole vocabulary; reads
// a.x, writes the named tokens of a.out. COPY: the rows are copied and masked
// first.
//
// A block takes the whole vocabulary, in tiles of kEditTile tokens, one for
// vocabularies up to 163,840. Measured with log-uniform ids (a vocabulary
// ordered by frequency), 256 decoding rows, histories of 4000 tokens: 23 us;
// by blocks of 8192 and of 32,768 tokens, of which one had most of the work,
// 40 and 27. With ids spread evenly, where such blocks would have had equal
// work, only this form was measured: 40 us. Each further tile builds a list of
// its own: 23.8 us at V = 163,840, 26.2 at 163,841, 30.7 at 262,144. A block
// compacts the seen tokens into a list in shared memory and spreads list x
// rows over its threads, two elements in flight per thread: on 2048 draft
// rows four cost 2 % more and eight 11 %, as longer bursts of scattered
// sectors only queue. Drafted and biased tokens, whose value differs from row
// to row or has a sum in it, are kept apart.
template <int DT, bool COPY>
__global__ void __launch_bounds__(kEditThreads, 2) k_rules_edit(const RulesArgs a) {
  constexpr int NT = kEditThreads, WPT = kEditTile / 32 / NT, kBatch = 2;  // WPT words of the bit table per thread
  static_assert(WPT <= 16, "the search over a thread's words takes steps of 8, 4, 2, 1");
  constexpr int es = Elem<DT>::kBytes;
  extern __shared__ __align__(16) char s_dyn[];
  uint32_t* s_word = reinterpret_cast<uint32_t*>(s_dyn);              // [WPT * NT] the tile's seen bits
  uint32_t* s_claim = s_word + WPT * NT;                              // [WPT * NT] bits of special tokens
  int* s_list = reinterpret_cast<int*>(s_claim + WPT * NT);           // [kListMax]
  float* s_minus = reinterpret_cast<float*>(s_list + kListMax);       // [kListMax] f c + p [c > 0] of the list's tokens
  const Special sp = carve_special(reinterpret_cast<char*>(s_minus + kListMax), a.special);
  __shared__ int64_t s_off[kRowsMax];     // first byte of a row
  __shared__ int16_t s_pos[kRowsMax];
  __shared__ int s_rank[NT], s_warp[NT / 32];
  __shared__ int s_nt, s_no;
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = blockIdx.x;
  const int64_t V = a.V, W = (V + 31) / 32;
  const bool special = a.L + a.h.n_bias > 0;
  for (int w = tid; special && w < WPT * NT; w += NT) s_claim[w] = 0u;
  if (tid == 0) s_nt = s_no = 0;
  pdl_wait();
  pdl_trigger();

  const Request r = load_request(a, b);
  const int seat = r.seat, m = r.m, n_bias = r.sat ? a.h.n_bias : 0;
  const uint32_t* seen = a.h.seen + seat * W;
  const int32_t* counts = a.h.counts + seat * V;
  int entry = -1;  // a special entry: token and bias
  float value = 0.f;
  auto load_entry = [&](int e) {
    entry = -1;
    value = 0.f;
    if (e < 32) {
      if (e < min(r.ell, a.L)) entry = a.tokens[static_cast<int64_t>(b) * a.L + e];
    } else if (e < 32 + n_bias) {
      entry = a.h.bias_tokens[static_cast<int64_t>(seat) * n_bias + e - 32];
      value = a.h.bias_values[static_cast<int64_t>(seat) * n_bias + e - 32];
    }
  };
  // the first tile's words and the first entries need the seat alone: they are asked for before the penalties are known
  uint32_t word[WPT];
#pragma unroll
  for (int k = 0; k < WPT; ++k)
    word[k] = r.sat && (tid + k * NT) * 32 < V ? seen[tid + k * NT] : 0u;
  load_entry(tid);
  if (r.flag) {
    if (blockIdx.y == 0 && tid == 0) atomicOr(a.status, r.flag);
    return;
  }
  const bool pen = r.pen;
  // x / r as x times the rounded 1 / r: one more rounding of 2^-24, for a division less per element
  const float rep = r.rep, inv = 1.f / r.rep, freq = r.freq, pres = r.pres;
  const bool counted = pen && (freq != 0.f || pres != 0.f);  // the repetition penalty needs the seen bits alone
  const int n_tok = pen ? r.ell : 0;
  const int q0 = blockIdx.y * a.per, nq = min(a.K * r.nrow, q0 + a.per) - q0;
  if (blockIdx.y == 0 && tid < n_tok && (entry < 0 || entry >= V)) atomicOr(a.status, kFlagTokenRange);
  if (nq <= 0 || (!COPY && !pen && n_bias == 0)) return;
  const uint32_t* mask = a.mask + (m >= 0 ? static_cast<int64_t>(m) * a.mask_len * W : 0);
  for (int q = tid; q < nq; q += NT) {
    int i;
    s_off[q] = row_byte<DT>(a, r, b, q0 + q, i);
    s_pos[q] = static_cast<int16_t>(i);
  }

  if constexpr (COPY) {  // the block's rows, while they will be in L2 for the edits; tiles begin with a barrier
    __syncthreads();
    const int chunks = static_cast<int>((V + kChunk - 1) / kChunk);
    for (int q = 0; q < nq; ++q) {
      const uint32_t* row_mask = mask + s_pos[q] * W;
#pragma unroll 1
      for (int c = tid >> 5; c < chunks; c += NT / 32) {
        const int w = c * 32 + lane;
        const uint32_t allow = m >= 0 && w < W ? row_mask[w] : 0xffffffffu;
        const int64_t at = static_cast<int64_t>(c) * kChunk, off = s_off[q] + at * es;
        stream_chunk<DT, false>(a.x + off, a.out + off, static_cast<int>(min(static_cast<int64_t>(kChunk), V - at)), allow);
      }
    }
    if (!pen && n_bias == 0) return;
  }

  for (int64_t t0 = 0; t0 < V; t0 += kEditTile) {
    const int span = static_cast<int>(min(static_cast<int64_t>(kEditTile), V - t0));
    const int64_t w0 = t0 / 32;
    if (t0) {  // a further tile: the last one's shared memory is free
      __syncthreads();
      for (int w = tid; special && w < WPT * NT; w += NT) s_claim[w] = 0u;
      if (tid == 0) s_nt = s_no = 0;
    }
    if (t0) {
#pragma unroll
      for (int k = 0; k < WPT; ++k)
        word[k] = (tid + k * NT) * 32 < span ? seen[w0 + tid + k * NT] : 0u;
    }
#pragma unroll
    for (int k = 0; k < WPT; ++k) s_word[tid + k * NT] = pen ? word[k] : 0u;
    __syncthreads();  // s_claim, s_word, s_nt, s_no, s_off, s_pos
    if (n_tok + n_bias > 0) {
      uint32_t mine = 0u;  // entries this thread was the first to name
      for (int e = tid, j = 0; e < 32 + n_bias; e += NT, ++j) {
        if (j || t0) load_entry(e);
        const int64_t x = e < 32 && e >= n_tok ? -1 : entry;
        const float add = value;
        if (e >= 32 && x >= V && blockIdx.y == 0 && t0 == 0) atomicOr(a.status, kFlagTokenRange);
        const bool in = x >= t0 && x < t0 + span;
        const int v = in ? static_cast<int>(x - t0) : -1;
        sp.v[e] = v;
        sp.add[e] = add;
        if (in) {
          const uint32_t bit = 1u << (v & 31);
          if (atomicOr(&s_claim[v >> 5], bit) & bit) sp.twice[atomicAdd(&s_nt, 1)] = e;
          else mine |= 1u << j;
        }
      }
      __syncthreads();
      // One entry of a token, whichever came first, speaks for it: it collects the positions the token is drafted at
      // and its biases, added up in list order.
      const int nt = s_nt;
      for (int e = tid, j = 0; e < 32 + n_bias; e += NT, ++j) {
        if (!(mine >> j & 1)) continue;
        const int v = sp.v[e];
        uint32_t drafted = e < 32 ? 1u << e : 0u;
        const uint32_t bits = pen ? seen[w0 + (v >> 5)] : 0u;
        const int stored = counted ? counts[t0 + v] : 0;  // on its way beside the bits: 0 where the bit is not set
        const int count = bits >> (v & 31) & 1 ? stored : -1;
        int biases = e >= 32;
        float add = sp.add[e];
        for (int k = 0; k < nt; ++k) {
          const int o = sp.twice[k];
          if (sp.v[o] != v) continue;
          if (o < 32) {
            drafted |= 1u << o;
          } else {
            add = biases++ ? add + sp.add[o] : sp.add[o];
          }
        }
        if (biases > 2) {  // of two, the order does not matter
          add = 0.f;
          for (int k = 32; k < 32 + n_bias; ++k)
            if (sp.v[k] == v) add += sp.add[k];
        }
        sp.add[e] = add;  // no other thread reads the entries of this token
        sp.drafted[e] = drafted;
        sp.count[e] = count;
        sp.owner[atomicAdd(&s_no, 1)] = static_cast<uint16_t>(e);
      }
    }
    // seen tokens by rank: thread t counts words t * WPT ...; s_rank[t] is the rank of its first token
    int mine = 0;
    for (int k = 0; k < WPT; ++k) {
      const int w = tid * WPT + k, left = span - w * 32;
      uint32_t bits = left > 0 ? s_word[w] : 0u;
      if (special) bits &= ~s_claim[w];
      if (left < 32 && left > 0) bits &= (1u << left) - 1u;
      s_word[w] = bits;
      mine += __popc(bits);
    }
    int rank = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, rank, o);
      if (lane >= o) rank += t;
    }
    if (lane == 31) s_warp[tid >> 5] = rank;
    __syncthreads();  // s_warp, s_no
    {
      const int sum = lane < NT / 32 ? s_warp[lane] : 0;
      int all = sum;
#pragma unroll
      for (int o = 1; o < NT / 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += t;
      }
      rank += __shfl_sync(0xffffffffu, all - sum, tid >> 5);
      s_rank[tid] = rank - mine;
      mine = __shfl_sync(0xffffffffu, all, NT / 32 - 1);
    }
    for (int k = 0, to = s_rank[tid]; k < WPT; ++k) {
      s_claim[tid * WPT + k] = to;
      to += __popc(s_word[tid * WPT + k]);
    }
    __syncthreads();  // s_rank, s_word, s_claim: from here on, ranks of words

    // named tokens x rows; the list in rounds of kListMax (one, unless the history is very long)
    const int n = mine, no = s_no;
    for (int l0 = 0; l0 == 0 || l0 < n; l0 += kListMax) {
      const int ln = min(kListMax, n - l0);
      if (ln == 0 && no == 0) break;
      if (l0) __syncthreads();
      // the token of rank j: a search over the threads' ranks, then over the thread's words, then over the word's bits
      // (each word writing its own tokens in a loop over its bits diverges: 1.7 us for 200 tokens, this 0.7)
#pragma unroll 1
      for (int e = tid; e < ln; e += NT) {
        const int j = l0 + e;
        int lo = 0;
#pragma unroll
        for (int step = NT / 2; step > 0; step >>= 1)
          if (s_rank[lo + step] <= j) lo += step;
        int w = lo * WPT;
        const int last = w + WPT - 1;
#pragma unroll
        for (int step = 8; step > 0; step >>= 1)
          if (w + step <= last && static_cast<int>(s_claim[w + step]) <= j) w += step;
        int left = j - static_cast<int>(s_claim[w]);
        uint32_t bits = s_word[w];
        int at = 0;
#pragma unroll
        for (int half = 16; half > 0; half >>= 1) {
          const int low = __popc(bits & ((1u << half) - 1u));
          if (left >= low) {
            left -= low;
            at += half;
            bits >>= half;
          }
        }
        s_list[e] = w * 32 + at;
      }
      if (ln > 0) __syncthreads();
      const char* x = a.x + t0 * es;
      char* y = a.out + t0 * es;
      const int dq = ln ? NT / ln : 0, de = NT - dq * ln;  // a step of NT elements
      int e = ln ? tid % ln : 0, q = ln ? tid / ln : nq;
      for (bool begin = true;; begin = false) {
        float f[kBatch];
        uint32_t on = 0u;
        int e2 = e, q2 = q;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (q < nq) {
            const int v = s_list[e];
            if (m < 0 || (mask[s_pos[q] * W + w0 + (v >> 5)] >> (v & 31) & 1)) {
              on |= 1u << k;
              f[k] = load_x<DT>(x + s_off[q], v);
            }
          }
          q += dq;
          e += de;
          if (e >= ln) {
            e -= ln;
            ++q;
          }
        }
        if (begin) {  // while the first elements are on their way: special tokens, then the counts
#pragma unroll 1
          for (int j = tid; j < no * nq; j += NT) {
            const int row = j / no, o = sp.owner[j - row * no], v = sp.v[o], i = s_pos[row];
            const int extra = __popc(sp.drafted[o] & (i >= 32 ? 0xffffffffu : (1u << i) - 1u));
            const int c = max(sp.count[o], 0) + extra;
            const bool known = sp.count[o] >= 0 || extra > 0;
            const float add = sp.add[o], minus = freq * static_cast<float>(c) + (c > 0 ? pres : 0.f);
            if (((!known || rep == 1.f) && minus == 0.f && add == 0.f) || l0) continue;  // x stays, bit by bit
            if (m >= 0 && !(mask[i * W + w0 + (v >> 5)] >> (v & 31) & 1)) continue;
            const float g = load_x<DT>(x + s_off[row], v);
            store_x<DT>(y + s_off[row], v, (known ? g * (g > 0.f ? inv : rep) : g) - minus + add);
          }
#pragma unroll 1
          for (int j = tid; j < ln; j += 4 * NT) {
            int c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = counted && j + k * NT < ln ? counts[t0 + s_list[j + k * NT]] : 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (j + k * NT < ln) s_minus[j + k * NT] = freq * static_cast<float>(c[k]) + (c[k] > 0 ? pres : 0.f);
          }
          __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          // with r = 1 tokens that are not counted stay, bit by bit (x * 1 - 0 would lose a NaN's payload)
          if ((on >> k & 1) && (rep != 1.f || s_minus[e2] != 0.f))
            store_x<DT>(y + s_off[q2], s_list[e2], f[k] * (f[k] > 0.f ? inv : rep) - s_minus[e2]);
          q2 += dq;
          e2 += de;
          if (e2 >= ln) {
            e2 -= ln;
            ++q2;
          }
        }
        if (q >= nq) break;
      }
    }
  }
}

static size_t edit_shared(int special) {
  return kEditTile / 4 + kListMax * 8 + static_cast<size_t>(special) * kSpecialBytes;
}

cudaError_t launch_logit_rules(const RulesArgs& args, int dtype, cudaStream_t st) {
  RulesArgs a = args;
  const int most = a.K * a.rows;
  const bool inplace = a.x == a.out;
  // Out of place, many long rows are copied by the edit kernel itself: the edits find part of them in L2. Fewer leave
  // SMs idle, and short ones most of a block's warps. bf16, 800 tokens of history, one launch / two launches, us:
  //   1088 rows of 65,536: 67 / 78    512 of 65,536: 38 / 41    300 of 151,936: 54 / 50
  //   1088 rows of 16,384: 28 / 30    1088 of 8192: 21 / 19     1562 of 1141: 18 / 14
  const bool fused = !inplace && a.h.counts && static_cast<int64_t>(a.B) * most >= 148 * 3 && a.V >= 16 * kChunk;
  if ((!inplace && !fused) || (inplace && a.mask)) {
    // a row is cut until the grid has 4 blocks for each of the GPU's 148 x 6 slots, 8 chunks (one per warp) at least;
    // copies, which have their data to wait for, into those
    const int64_t chunks = (a.V + kChunk - 1) / kChunk, rows = static_cast<int64_t>(a.B) * most;
    const int64_t cut = std::max<int64_t>(1, std::min<int64_t>((chunks + kWarps - 1) / kWarps, 148 * 24 / rows));
    a.per = inplace ? static_cast<int>((chunks + cut - 1) / cut) : kWarps;
    const dim3 grid(static_cast<unsigned>((chunks + a.per - 1) / a.per), static_cast<unsigned>(a.B),
                    static_cast<unsigned>(most));
    void (*k)(RulesArgs) = dtype == 0 ? (inplace ? k_rules_stream<0, true> : k_rules_stream<0, false>)
                                      : (inplace ? k_rules_stream<1, true> : k_rules_stream<1, false>);
    const cudaError_t e = launch_pdl(k, grid, dim3(kThreads), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  if (!a.h.counts) return cudaSuccess;
  // Blocks of a request: the GPU's 296 slots filled once, where every row is there; with lengths known on the device
  // alone, half as many again, as some find no row. 2048 draft rows 52.2 us by 2 blocks per SM, 56.4 by 3; 544 packed
  // target rows 52.2 and 48.7.
  const int slots = 148 * (fused ? 4 : a.vlen ? 3 : 2);
  const int z = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, slots / a.B)));
  a.per = (most + z - 1) / z;
  a.special = 32 + a.h.n_bias;
  const dim3 grid(static_cast<unsigned>(a.B), static_cast<unsigned>((most + a.per - 1) / a.per));
  const size_t smem = edit_shared(a.special);
  void (*k)(RulesArgs) = dtype == 0 ? (fused ? k_rules_edit<0, true> : k_rules_edit<0, false>)
                                    : (fused ? k_rules_edit<1, true> : k_rules_edit<1, false>);
  // always the most that a call can need: another host thread may be between its own setting and launch
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(edit_shared(32 + SPEC_MAX_BIAS)));
  return e != cudaSuccess ? e : launch_pdl(k, grid, dim3(kEditThreads), smem, st, a);
}

// ------------------------------------------------------------------ history

// counts[s, t] += 1 and seen[s, t] = 1 for every token t of the batch; integer
// atomics, so the order of the threads does not matter.
//  offsets != NULL: tokens[offsets[b] .. offsets[b + 1]) belong to request b.
//  offsets == NULL: tokens is [B, width].
// Negative tokens are padding.
//
// A block takes 1024 tokens. Atomics on one address queue up, and a prompt may
// name a few ids again and again: a block whose tokens belong to one request
// first collects the bits of the ids below kHot in shared memory and then
// writes each word once. 32 prompts of up to 8192 tokens, with clearing their
// seats, us by global atomics alone / so:
//   one id throughout            13.2 / 6.8
//   log-uniform ids of 151,936    9.5 / 8.7    of 262,144   11.1 / 11.8
//   ids spread evenly             8.7 / 9.5    of 262,144   12.3 / 13.6
// It is kept for the first line: what a prompt repeats is the user's choice.
constexpr int kAddTokens = 4;     // per thread
constexpr int kHot = 32 * 2 * kThreads;

__global__ void __launch_bounds__(kThreads) k_history_add(const spec_history h, const int32_t* __restrict__ seats,
                                                          int B, const int32_t* __restrict__ tokens, int64_t n,
                                                          const int32_t* __restrict__ offsets, int width, int output,
                                                          int* status) {
  extern __shared__ int s_off[];  // [B + 1], then the requests' seats [B]
  int* s_seat = s_off + B + 1;
  __shared__ uint32_t s_hot[kHot / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (tid == 0) s_bad = 0;
  for (int w = tid; offsets && w < kHot / 32; w += kThreads) s_hot[w] = 0u;
  pdl_wait();
  pdl_trigger();
  const int per = offsets ? kAddTokens : 1;  // a step's tokens are few: one to a thread
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kThreads * per;
  int x[kAddTokens];
#pragma unroll
  for (int k = 0; k < kAddTokens; ++k) {
    const int64_t t = t0 + tid + k * kThreads;
    x[k] = k < per && t < n ? tokens[t] : -1;
  }
  if (offsets) {
    __syncthreads();
    for (int b = tid; b <= B; b += kThreads) {
      const int o = offsets[b];
      s_off[b] = o;
      if (b < B) s_seat[b] = seats ? seats[b] : b;
      if (o < 0 || o > n || (b > 0 && offsets[b - 1] > o)) s_bad = 1;
    }
    __syncthreads();
    if (s_bad) {
      if (blockIdx.x == 0 && tid == 0) atomicOr(status, kFlagLengths);
      return;
    }
  }
  auto request_of = [&](int64_t t) {
    if (!offsets) return static_cast<int>(t / width);
    int lo = 0, hi = B - 1;  // last request with offset <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_off[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  const int64_t W = (h.V + 31) / 32;
  const int b0 = request_of(t0);
  const bool whole = offsets && request_of(min(t0 + kThreads * kAddTokens, n) - 1) == b0;  // one request's block
  int flag = 0;
#pragma unroll
  for (int k = 0; k < kAddTokens; ++k) {
    const int64_t t = t0 + tid + k * kThreads;
    if (x[k] < 0 || (offsets && (t < s_off[0] || t >= s_off[B]))) continue;
    const int b = whole ? b0 : request_of(t);
    const int seat = offsets ? s_seat[b] : seats ? seats[b] : b;
    if (seat < 0) continue;
    if (seat >= h.seats) { flag |= kFlagIndex; continue; }
    if (x[k] >= h.V) { flag |= kFlagTokenRange; continue; }
    const uint32_t bit = 1u << (x[k] & 31);
    if (whole && x[k] < kHot) {
      if (!(s_hot[x[k] >> 5] & bit)) atomicOr(&s_hot[x[k] >> 5], bit);
    } else {
      atomicOr(h.seen + seat * W + (x[k] >> 5), bit);
    }
    if (output) atomicAdd(h.counts + seat * h.V + x[k], 1);
  }
  if (flag) atomicOr(status, flag);
  if (!whole) return;
  __syncthreads();
  const int hot_seat = s_seat[b0];  // in range wherever a bit was collected
  for (int w = tid; w < kHot / 32; w += kThreads)
    if (s_hot[w]) atomicOr(h.seen + hot_seat * W + w, s_hot[w]);
}

cudaError_t launch_history_add(const spec_history& h, const int32_t* seats, int B, const int32_t* tokens, int64_t n,
                               const int32_t* offsets, int width, int output, int* status, cudaStream_t st) {
  const int64_t per = kThreads * (offsets ? kAddTokens : 1), blocks = (n + per - 1) / per;
  const size_t smem = offsets ? sizeof(int) * (2 * B + 1) : 0;  // 32 KiB at most
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
