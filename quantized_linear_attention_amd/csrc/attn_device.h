// attn_device.h — what the softmax layers' kernels share (attn.hip,
// attn_long.hip): element loads and stores, attention over chunks of the 4-bit
// cache with its kernels for few and for many query rows and the join of their
// parts, and the host's checks of a cache and of strided rows.
#pragma once
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>
#include <string.h>

#include "stq.h"
#include "stq_device.h"

using namespace stq;

namespace {

typedef f16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int E_MIN = -23, E_MAX = 13;   // exponents of the cache's scales

__device__ __forceinline__ float bits_f(uint32_t u) { return __uint_as_float(u); }

// Division by an argument of the call, its reciprocal taken on the host: floor(2^32
// / by) is at most one step short for every 32-bit x.  (The compiler's division
// is a chain of some 40 instructions; five of them at a kernel's start and end
// cost 0.7 us of the 9.6 of one short request.  k_attend_tiles keeps the
// compiler's: they are nothing of its time, and its loop came out slower with
// these, 239 us for 227.)
struct Div { uint32_t by, inv; };
Div div_of(int64_t by) {
  Div d;
  d.by = by < 1 ? 1u : (uint32_t)by;
  d.inv = d.by == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / d.by);
  return d;
}
__device__ __forceinline__ int quot(uint32_t x, Div d) {
  const uint32_t q = __umulhi(x, d.inv);
  return (int)(q + (x - q * d.by >= d.by ? 1u : 0u));
}

// A 16-byte load that leaves no trace in the caches (once = true: data that no
// one reads again) or an ordinary one.
template <bool ONCE, typename T>
__device__ __forceinline__ T load16(const T* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(p);
  else return *p;
}
// A 16-byte store past the caches (PAST: an output larger than they are) or into them.
template <bool PAST, typename T>
__device__ __forceinline__ void store16(T* p, T v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// Eight consecutive elements as binary32 (16-byte loads; 2 of them for fp32).
template <int TYPE, bool ONCE = false>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* x) {
  if constexpr (TYPE == STQ_FP32) {
    const f32x4* p = (const f32x4*)((const float*)base + at);
    const f32x4 a = load16<ONCE>(p), b = load16<ONCE>(p + 1);
#pragma unroll
    for (int i = 0; i < 4; i++) { x[i] = a[i]; x[4 + i] = b[i]; }
  } else {
    const u32x4 a = load16<ONCE>((const u32x4*)((const uint16_t*)base + at));
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (TYPE == STQ_BF16) {
        x[2 * i] = bits_f(a[i] << 16);
        x[2 * i + 1] = bits_f(a[i] & 0xFFFF0000u);
      } else {
        const f16x2 h = as_h2(a[i]);
        x[2 * i] = (float)h[0];
        x[2 * i + 1] = (float)h[1];
      }
    }
  }
}
// two binary32 values as a pair of 16-bit elements, to nearest even (NaN stays NaN)
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (TYPE == STQ_BF16) {
    const __bf16 x = (__bf16)a, y = (__bf16)b;
    return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
  } else {
    return h2_bits((f16x2){(f16)a, (f16)b});
  }
}
template <int TYPE, bool PAST = false>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* x) {
  if constexpr (TYPE == STQ_FP32) {
    f32x4* p = (f32x4*)((float*)base + at);
    store16<PAST>(p, (f32x4){x[0], x[1], x[2], x[3]});
    store16<PAST>(p + 1, (f32x4){x[4], x[5], x[6], x[7]});
  } else {
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; i++) a[i] = pack2<TYPE>(x[2 * i], x[2 * i + 1]);
    store16<PAST>((u32x4*)((uint16_t*)base + at), a);
  }
}

// ------------------------------------------------------------- attention
struct AttnArgs {
  const uint8_t* cache;
  const int32_t *table, *tok_start, *len;
  const void* q;
  void* o;
  float *po, *pml;          // partial results: [split][row][D], [split][row][2]
  int n_req, n_tok, hq, hkv, group, T, n_blocks, cols, max_new, window, sink, splits, per, tiles;
  Div by_hkv, by_group, by_max_new, by_per;
  int64_t qs, os;
  float scale;
};

// What a call's chunks are: SPAN all that a request's rows see; LIST the blocks
// that a token's and head's list names (one query token a workgroup); PREFIX the
// tokens that a group of requests shares, for the rows of all of them; SUFFIX
// those of a request behind what its group shares.
enum Mode { SPAN, LIST, PREFIX, SUFFIX };              // (attend_rows has both of the last as SUFFIX)

struct LongArgs : AttnArgs {
  const int32_t* sel;                    // LIST: [n_tok][hkv][n_sel] block columns
  int n_sel;
  const int32_t *group_start, *prefix;   // PREFIX and SUFFIX: [n_groups + 1], [n_groups]
  int n_groups, pre_per;                 // chunks of a prefix' part at least
  int slot0;                             // parts of a prefix at most; in the workspace those of the requests' own tokens follow
  int pre_fill;                          // workgroups of a head that fill the card
  int pre_units;                         // SUFFIX: workgroups (times heads) that take a prefix' part
  int pre_blocks;                        // PREFIX: workgroups that do; the others take the requests' own tokens
  int32_t* shared;                       // [n_req] tokens that the request's group shares, then the chunks of a prefix' part
};
template <int MODE> using ArgsOf = std::conditional_t<MODE == SPAN, AttnArgs, LongArgs>;

// Chunks of 32 positions that some row of positions [p0, p1] sees: the first
// n_low chunks (always-visible tokens), then chunks from lo on, `total` in all.
struct Span { int n_low, lo, total; };
__device__ __forceinline__ Span span_of(int p0, int p1, int window, int sink) {
  Span s;
  if (p1 < 0) { s.n_low = s.lo = s.total = 0; return s; }
  const int first = window > 0 ? max(0, p0 - window + 1) : 0;
  s.lo = first >> 5;
  s.n_low = min((min(sink, p1 + 1) + 31) >> 5, s.lo);
  s.total = s.n_low + (p1 >> 5) + 1 - s.lo;
  return s;
}
// First row, rows, position of query 0.  Query tokens behind the last row of q
// count for the positions (no row lies before -2^28: there are at most 2^28).
struct Req { int first, n_new, base; };
__device__ __forceinline__ Req req_of(const AttnArgs& A, int start, int end, int len) {
  start = max(start, 0);
  end = max(end, start);
  len = (int)min((int64_t)max(len, 0), (int64_t)A.cols * A.T);
  Req r;
  r.first = min(start, A.n_tok);
  r.n_new = min(end, A.n_tok) - r.first;
  r.base = max(len - (end - start), -(1 << 28));
  return r;
}
__device__ __forceinline__ Req req_args(const AttnArgs& A, int i) {
  return req_of(A, ld_const(A.tok_start + i), ld_const(A.tok_start + i + 1), ld_const(A.len + i));
}

// What the workgroups of requests that share prefixes have to know of the whole
// batch, by all lanes of a wave: `Members` of a group g are requests [s, e) with
// query rows [first, last) of q; they share `len` tokens: whole blocks, and none
// behind the first new token of any member that has one, so that every row sees
// all of them.  Up to 256 requests in 64 groups are loaded at once, one request or
// group a lane, and the rest is exchanged between lanes: a chain of one load
// instead of three or four (the prefixes' part of 60 requests behind two of them 24.6
// -> 23.2 us).  More are looked up by every workgroup, a load behind another: 256 -> 257
// requests behind one prefix of 2,048 tokens 51.9 -> 57.0 us (attention without sharing 64.8
// -> 70.1), 64 -> 65 groups of one request behind 1,024 23.8 -> 27.1 (15.5 -> 17.5).
struct Members { int s, e, first, last, len; };
__device__ __forceinline__ int wave_max_i(int x);
struct Whole {
  static constexpr int N = 4;                          // registers of 64 requests
  const LongArgs& A;
  bool fits;
  int start[N + 1], end[N], base[N];                   // base: position of the first new token, the largest without one
  int g0, g1, pre;                                     // lane = group
  __device__ __forceinline__ explicit Whole(const LongArgs& args) : A(args) {
    const int lane = threadIdx.x & 63;
    fits = A.n_req <= 64 * N && A.n_groups <= 64 && A.n_groups > 0;
    if (!fits) return;
    g0 = A.group_start[min(lane, A.n_groups)];
    g1 = A.group_start[min(lane + 1, A.n_groups)];
    pre = A.prefix[min(lane, A.n_groups - 1)];
    int len[N];
#pragma unroll
    for (int r = 0; r <= N; r++) start[r] = 64 * r <= A.n_req ? A.tok_start[min(64 * r + lane, A.n_req)] : 0;
#pragma unroll
    for (int r = 0; r < N; r++) {
      end[r] = 64 * r < A.n_req ? A.tok_start[min(64 * r + lane + 1, A.n_req)] : 0;
      len[r] = 64 * r < A.n_req ? A.len[min(64 * r + lane, A.n_req - 1)] : 0;
    }
#pragma unroll
    for (int r = 0; r < N; r++) base[r] = end[r] > start[r] ? req_of(A, start[r], end[r], len[r]).base : INT32_MAX;
    g0 = min(max(g0, 0), A.n_req);
    g1 = min(max(g1, g0), A.n_req);
    pre = shared_blocks(pre);
  }
  __device__ __forceinline__ int shared_blocks(int x) const { return (int)min((int64_t)max(x, 0), (int64_t)A.cols * A.T) & ~(A.T - 1); }
  // tok_start of request x (any lane's own)
  __device__ __forceinline__ int start_at(int x) const {
    int v = __shfl(start[0], x & 63, 64);
#pragma unroll
    for (int r = 1; r <= N; r++) {
      if (64 * r > A.n_req) break;
      const int y = __shfl(start[r], x & 63, 64);
      v = x >> 6 == r ? y : v;
    }
    return v;
  }
  __device__ __forceinline__ Members group(int g) const {
    Members m;
    int least = INT32_MAX;
    if (fits) {
      m.s = __builtin_amdgcn_readlane(g0, g);
      m.e = __builtin_amdgcn_readlane(g1, g);
      m.len = __builtin_amdgcn_readlane(pre, g);
#pragma unroll
      for (int r = 0; r < N; r++) {
        const int x = 64 * r + (int)(threadIdx.x & 63);
        least = min(least, x >= m.s && x < m.e ? base[r] : INT32_MAX);
      }
      m.first = __builtin_amdgcn_readfirstlane(start_at(m.s));
      m.last = __builtin_amdgcn_readfirstlane(start_at(m.e));
    } else {
      m.s = min(max(ld_const(A.group_start + g), 0), A.n_req);
      m.e = min(max(ld_const(A.group_start + g + 1), m.s), A.n_req);
      m.len = shared_blocks(ld_const(A.prefix + g));
      for (int b = m.s; b < m.e; b += 64) {
        const int i = min(b + (int)(threadIdx.x & 63), m.e - 1);
        const int x = A.tok_start[i], y = A.tok_start[i + 1];
        if (y > x) least = min(least, req_of(A, x, y, A.len[i]).base);
      }
      m.first = A.tok_start[m.s];
      m.last = A.tok_start[m.e];
    }
    m.first = min(max(m.first, 0), A.n_tok);
    m.last = min(max(m.last, m.first), A.n_tok);
    m.len = max(min(m.len, -wave_max_i(-least)), 0) & ~(A.T - 1);
    return m;
  }
  // What request i shares (0 in no group).  The group that holds it is the last one
  // that starts at or before it.
  __device__ __forceinline__ int shared_of(int i) const {
    int g = -1;
    if (fits) {
      g = __builtin_popcountll(__builtin_amdgcn_ballot_w64((int)(threadIdx.x & 63) < A.n_groups && g0 <= i)) - 1;
    } else {
      for (int b = 0; b < A.n_groups; b += 64) {
        const int x = b + (int)(threadIdx.x & 63);
        const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(x < A.n_groups && A.group_start[min(x, A.n_groups - 1)] <= i));
        if (n > 0) g = b + n - 1;
      }
    }
    if (g < 0) return 0;
    const Members m = group(g);
    return i < m.e ? m.len : 0;
  }
  // The x-th part of all prefixes' work: group, tile of its rows, part of its chunks
  // and how many chunks a part has, the same for all.  Parts are sized by what all
  // groups together have to do, so that the card is filled once (four groups of
  // 11,648 to 16,384 shared tokens with 619 query tokens: 235 us in parts by the
  // longest prefix alone, 203 so; one line of all tiles' chunks cut evenly takes 275,
  // since a part's tiles no longer read the same tokens at one time).
  struct Part { int g, tile, sp, per; };
  __device__ __forceinline__ bool part(int rows_of_tile, int x, Part* r) const {
    const int lane = threadIdx.x & 63;
    float total = 0.0f;
    int most = 0;
    auto of = [&](int b, int* tiles, int* chunks) {      // of group b + lane
      int s = g0, e = g1, first, last, share = pre;
      if (fits) {
        first = start_at(s);
        last = start_at(e);
      } else {
        const int y = min(b + lane, A.n_groups - 1);
        s = min(max(A.group_start[y], 0), A.n_req);
        e = min(max(A.group_start[y + 1], s), A.n_req);
        share = shared_blocks(A.prefix[y]);
        first = A.tok_start[s];
        last = A.tok_start[e];
      }
      first = min(max(first, 0), A.n_tok);
      last = min(max(last, first), A.n_tok);
      const bool on = b + lane < A.n_groups && share > 0;
      *tiles = on ? (int)(((int64_t)(last - first) * A.group + rows_of_tile - 1) / rows_of_tile) : 0;
      *chunks = on ? share >> 5 : 0;
    };
    int tiles, chunks;
    for (int b = 0; b < A.n_groups; b += 64) {
      of(b, &tiles, &chunks);
      total += wave_sum((float)tiles * (float)chunks);
      most = max(most, wave_max_i(chunks));
    }
    const int fill = (int)__builtin_fminf(total / A.pre_fill, 0x1p30f);
    r->per = (max(max(fill, A.pre_per), (most + A.slot0 - 1) / A.slot0) + 3) & ~3;
    // (whole parts are more than the total says: no second round of a few workgroups)
    for (int n = 0; r->per < most; n++) {
      int count = 0;
      for (int b = 0; b < A.n_groups; b += 64) {
        if (A.n_groups > 64) of(b, &tiles, &chunks);
        count += wave_sum_i(tiles * ((chunks + r->per - 1) / r->per));
      }
      if (count <= A.pre_fill) break;
      r->per = n < 24 ? r->per + max((r->per >> 4) & ~3, 4) : (most + 3) & ~3;
    }
    for (int b = 0; b < A.n_groups; b += 64) {
      if (A.n_groups > 64) of(b, &tiles, &chunks);
      const int parts = (chunks + r->per - 1) / r->per, mine = tiles * parts;
      int sum = mine;                                    // inclusive
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(sum, d, 64);
        if (lane >= d) sum += y;
      }
      const int all = __builtin_amdgcn_readlane(sum, 63);
      if (x < all) {
        const int k = __builtin_ctzll(__builtin_amdgcn_ballot_w64(sum > x));
        const int y = x - (__builtin_amdgcn_readlane(sum, k) - __builtin_amdgcn_readlane(mine, k)), t = __builtin_amdgcn_readlane(tiles, k);
        r->g = b + k;
        r->sp = y / t;                                   // (the tiles of a part side by side: they read the same tokens)
        r->tile = y - r->sp * t;
        return true;
      }
      x -= all;
    }
    return false;
  }
};
// Entries of a list up to its last one that names a block the token at position
// p may see.  By all lanes of a wave.
__device__ __forceinline__ bool listed(const LongArgs& A, int col, int p) { return col >= 0 && col < A.cols && (int64_t)col * A.T <= p; }
__device__ __forceinline__ int entries_of(const LongArgs& A, const int32_t* list, int p) {
  int n = 0;
  for (int b = 0; b < A.n_sel; b += 64) {
    const int x = b + (int)(threadIdx.x & 63);
    const uint64_t on = __builtin_amdgcn_ballot_w64(x < A.n_sel && listed(A, list[min(x, A.n_sel - 1)], p));
    if (on) n = b + 64 - __builtin_clzll(on);
  }
  return n;
}

// Chunks of one part of a request's work: the host's size for a request of the
// stated longest length, more for a request that is longer than that (a
// multiple of four: one per wave).  Shorter requests have fewer parts, all of
// one size.
__device__ __forceinline__ int split_chunks(const AttnArgs& A, int total) {
  if (total <= A.per * A.splits) return A.per;
  return ((total + A.splits - 1) / A.splits + 3) & ~3;
}

__device__ __forceinline__ float max_quads(float x) {   // over the four 16-lane groups
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __builtin_fmaxf(bits_f(a[0]), bits_f(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_fmaxf(bits_f(b[0]), bits_f(b[1]));
}
__device__ __forceinline__ float sum_quads(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = bits_f(a[0]) + bits_f(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return bits_f(b[0]) + bits_f(b[1]);
}

__device__ __forceinline__ int wave_max_i(int x) {
  x = max(x, dppi<0xB1>(x));
  x = max(x, dppi<0x4E>(x));
  x = max(x, dppi<0x141>(x));
  x = max(x, dppi<0x140>(x));
  return max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
             max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
}
__device__ __forceinline__ float wave_max(float x) {
  x = __builtin_fmaxf(x, dpp<0xB1>(x));
  x = __builtin_fmaxf(x, dpp<0x4E>(x));
  x = __builtin_fmaxf(x, dpp<0x141>(x));
  x = __builtin_fmaxf(x, dpp<0x140>(x));
  return max_quads(x);
}

constexpr float NEG_INF = -__builtin_inff();

// Power of two that brings a row's largest magnitude m into [2^14, 2^15), and
// the factor that turns products of such rows into base-2 logits.
__device__ __forceinline__ int q_shift(float m) {
  return m > 0.0f && m < __builtin_inff() ? 15 - __builtin_amdgcn_frexp_expf(m) : 0;
}
// (Kept normal, and at most 2^80: two products that differ are 2^-48 apart at
// least, which is 2^32 logits then, and products of 2^38 stay finite.)
__device__ __forceinline__ float q_factor(float scale, int e) {
  const float c = __builtin_ldexpf(__builtin_fabsf(scale), -e) * 1.44269504088896340736f;
  return __builtin_fminf(__builtin_fmaxf(c, 1.17549435e-38f), 0x1p80f);
}

// A wave's query rows as matrix operands: row n = lane % 16 of tile nt, the
// channels (D/4) G .. + D/4 of lane group G = lane / 16, in binary16 scaled by
// a power of two that puts the row's largest magnitude in [2^14, 2^15) (exact
// for bf16 and fp16 queries down to 2^-29 of that magnitude).  c: the factor
// from scaled products to base-2 logits, kept positive (a negative scale
// turns the queries' signs) and normal.
template <int D, int TYPE>
__device__ __forceinline__ void load_q(const AttnArgs& A, int64_t at, f16x8* q, float* c) {
  float x[D / 4];
#pragma unroll
  for (int i = 0; i < D / 32; i++) load8<TYPE>(A.q, at + 8 * i, x + 8 * i);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 4; i++) m = __builtin_fmaxf(m, __builtin_fabsf(x[i]));
  m = max_quads(m);
  const int e = q_shift(m);
  const float sign = A.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < D / 32; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) q[i][j] = (f16)(sign * __builtin_ldexpf(x[8 * i + j], e));
  *c = q_factor(A.scale, e);
}

// One chunk (32 cached tokens of one head) as a wave loads it.  Element e of
// lane group G stands for token token_of(G, e): row 4G + e % 4 of key tile e / 4,
// so that the two tiles' products leave lane group G with the eight tokens of
// its query row that the product with the values wants from it.  At D = 128
// the tokens of a lane group are every other one, so that each load covers
// whole 128-byte lines (two tokens' codes) and may pass the caches by: 8
// requests of 32,768 to 131,072 tokens 164 us, 148 so, 161 past the caches with
// half lines.  At D = 64 eight tokens in turn are faster (64 requests of 2,048
// to 8,191 tokens: 51.6 us, 56 with four groups' tokens side by side).
template <int D>
__host__ __device__ constexpr int token_of(int G, int e) {
  return D == 128 ? 16 * (G >> 1) + 2 * e + (G & 1) : 8 * G + e;
}
// Keys: lane (m, G) holds the channels (D/4) G .. of row m.  Values: lane (m,
// G) holds the channels (D/16) m .. of its group's tokens.
template <int D>
struct Chunk {
  static constexpr int KD = D / 32;                    // dwords of keys per tile and lane
  static constexpr int VS = D == 128 ? 4 : 2;          // dwords of scales from the group's first token on
  static constexpr int STEP = token_of<D>(0, 1);       // tokens from one element to the next
  uint32_t k[2][KD], v[8];
  uint32_t ks[2];                                      // the scale of this lane's row is byte token_of % 4
  uint32_t vs[VS];
};

// A lane's places in a chunk, the same for every chunk (bytes from the chunk's
// first key code, value code, key scale, value scale).
template <int D>
struct Places {
  uint32_t k, v, ks, vs;
  __device__ __forceinline__ explicit Places(int T) {
    const int lane = threadIdx.x & 63, m = lane & 15, G = lane >> 4, r = token_of<D>(m >> 2, m & 3);
    k = r * (D / 2) + G * (D / 8);
    ks = (G * (D / 4) / 32) * T + (r & ~3);
    v = token_of<D>(G, 0) * (D / 2) + m * (D / 32);
    vs = (m * (D / 16) / 32) * T + (token_of<D>(G, 0) & ~7);
  }
};
template <int D, bool ONCE>
__device__ __forceinline__ void load_keys(Chunk<D>& C, const Places<D>& W, const uint8_t* codes, const uint8_t* scales) {
#pragma unroll
  for (int u = 0; u < 2; u++) {
    const int t = 4 * Chunk<D>::STEP * u;
    if constexpr (D == 128) {
      const u32x4 w = load16<ONCE>((const u32x4*)(codes + (W.k + t * (D / 2))));
#pragma unroll
      for (int i = 0; i < 4; i++) C.k[u][i] = w[i];
    } else {
      const u32x2 w = load16<ONCE>((const u32x2*)(codes + (W.k + t * (D / 2))));
      C.k[u][0] = w[0];
      C.k[u][1] = w[1];
    }
    C.ks[u] = *(const uint32_t*)(scales + (W.ks + t));
  }
}
template <int D, bool ONCE>
__device__ __forceinline__ void load_values(Chunk<D>& C, const Places<D>& W, const uint8_t* codes, const uint8_t* scales) {
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const uint8_t* p = codes + (W.v + Chunk<D>::STEP * j * (D / 2));
    if constexpr (D == 128) C.v[j] = load16<ONCE>((const uint32_t*)p);
    else C.v[j] = load16<ONCE>((const uint16_t*)p);
  }
  if constexpr (D == 128) {
    const u32x4 s = *(const u32x4*)(scales + W.vs);
#pragma unroll
    for (int i = 0; i < 4; i++) C.vs[i] = s[i];
  } else {
    const u32x2 s = *(const u32x2*)(scales + W.vs);
    C.vs[0] = s[0];
    C.vs[1] = s[1];
  }
}

// Scale byte j of a dword where v_cvt_scalef32_* takes a scale: in the
// exponent field of a binary32 (the conversion reads nothing else of it, and
// gives NaN for the byte 255).
template <int J>
__device__ __forceinline__ float scale_of(uint32_t w) {
  if constexpr (J < 3) return bits_f(w << (23 - 8 * J));
  else return bits_f(w >> 1);
}
template <int J>
__device__ __forceinline__ uint32_t cvt2(uint32_t w, float s) {   // codes 2J, 2J+1 of w as a binary16 pair
  return h2_bits(__builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, J)));
}
__device__ __forceinline__ f16x8 frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(f16x8, (u32x4){a, b, c, d});
}

// What a row's weights are relative to, 2^(product * c - mc).  A weight at the
// reference is 2^LIFT, and the reference follows the row's largest product only
// when a weight would pass 2^(LIFT + 8) = 2^15, which binary16 still holds (the
// sums are binary32, and a quotient does not mind): that spares most steps the
// exchange between lanes and the rescaling of the sums.  The lift is for the small
// weights: binary16 is subnormal below 2^-14, with steps of 2^-24, so without it
// thousands of tokens at 2^-20 of a dominant one (16 nats) lose much of their sum
// (16,390 tokens 14 nats below four: outputs off by 3.7 %, by 48 % at 16.6 nats).
// With it weights are normal down to 2^-21 of the largest at least, and below that
// off by 2^-31 of it at most.
constexpr float LIFT = 7.0f, MOVE = 8.0f;
struct Ref {
  float m, mc, over;       // the product it stands at, times c; products above `over` move it
  __device__ __forceinline__ void init() { m = over = NEG_INF; mc = 0.0f; }
  // Nothing seen yet: any finite reference will do, every weight is 2^-inf.
  __device__ __forceinline__ float at() const { return m == NEG_INF ? 0.0f : m; }
  // to the product x; the factor of what was summed so far
  __device__ __forceinline__ float move(float x, float c) {
    const float from = m;
    m = x;
    mc = __builtin_fmaf(at(), c, -LIFT);
    over = x + MOVE * __builtin_amdgcn_rcpf(c);
    return __builtin_amdgcn_exp2f((from - at()) * c);
  }
  // mc is off by half a step of its own, the same for all of a row's weights,
  // which their quotient does not mind; but past 2^22 that begins to leave the
  // weights' range (at 2^24 by 2^1).  Such rows' waves take the reference from
  // the products before they are multiplied.
  __device__ __forceinline__ bool steep() const { return __builtin_fabsf(mc) >= 0x1p22f; }
};

// x *= f for `count` registers from V`first` on, where any lane of `far` is set.
// The branch lies inside the statement and the accumulators at registers of
// their own: as an `if` around the products, the compiler kept the two sides'
// accumulators apart and copied one to the other in every step, which costs as
// much as the rescaling.  (The waits cover a matrix instruction's result read
// by the multiplications, and theirs read by the next.)
#define SCALE_WHERE(far, f, first, count, ...)                                                         \
  asm volatile("s_cmp_eq_u64 %[m], 0\n\ts_cbranch_scc1 .Lkeep%=\n\ts_nop 15\n\ts_nop 7\n\t"            \
               ".set stq_v, " #first "\n\t.rept " #count "\n\tv_mul_f32 v[stq_v], v[stq_v], %[x]\n\t" \
               ".set stq_v, stq_v+1\n\t.endr\n\ts_nop 4\n.Lkeep%=:"                                  \
               : __VA_ARGS__ : [m] "s"(far), [x] "v"(f) : "scc")
#define AT(r) "+{v[" #r "]}"

// Two weights as a binary16 pair.  Outputs of binary16: to nearest.  bfloat16
// outputs take the truncating conversion (one instruction at full rate against
// one at half): off by 2^-10 of a weight at most where the output's own
// rounding is 2^-8 (and by 2^-31 of the row's largest below 2^-21 of it: see
// Ref), and the weights' sum takes the same truncated values.
template <int TYPE>
__device__ __forceinline__ f16x2 weights(float a, float b) {
  if constexpr (TYPE == STQ_BF16) return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(a, b));
  else return (f16x2){(f16)a, (f16)b};
}

// Keys of a chunk and queries -> products s (tile u: elements 4u ..).
template <int D, int NT>
__device__ __forceinline__ void key_products(const Chunk<D>& C, const f16x8 (*q)[D / 32], f32x4 (*s)[2]) {
#pragma unroll
  for (int u = 0; u < 2; u++) {
    const float sc = scale_of<0>(C.ks[u] >> (8 * (token_of<D>((threadIdx.x >> 2) & 3, threadIdx.x & 3) & 3)));
#pragma unroll
    for (int nt = 0; nt < NT; nt++) s[nt][u] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D / 32; i++) {
      const uint32_t w = C.k[u][i];
      const f16x8 kf = frag(cvt2<0>(w, sc), cvt2<1>(w, sc), cvt2<2>(w, sc), cvt2<3>(w, sc));
#pragma unroll
      for (int nt = 0; nt < NT; nt++) s[nt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[nt][i], s[nt][u], 0, 0, 0);
    }
  }
}
// Values of a chunk and weights: o += V^T P, tile c element i = channel
// (D/16)(4G + i) + c of query row lane % 16.  Pairs of tokens of one channel
// are put together from pairs of channels of one token.
template <int D, int NT>
__device__ __forceinline__ void value_products(const Chunk<D>& C, bool full, const f16x8* P, f32x4 (*o)[D / 16]) {
  float vs[8];
  if constexpr (D == 128) {                            // byte 2 (j % 2) + G % 2 to bits 23 .., by rotation
    const uint32_t odd = (threadIdx.x >> 1) & 8;
#pragma unroll
    for (int j = 0; j < 8; j++)
      vs[j] = bits_f(__builtin_amdgcn_alignbit(C.vs[j >> 1], C.vs[j >> 1], 9 + 16 * (j & 1) + odd));
  } else {
    vs[0] = scale_of<0>(C.vs[0]); vs[1] = scale_of<1>(C.vs[0]); vs[2] = scale_of<2>(C.vs[0]); vs[3] = scale_of<3>(C.vs[0]);
    vs[4] = scale_of<0>(C.vs[1]); vs[5] = scale_of<1>(C.vs[1]); vs[6] = scale_of<2>(C.vs[1]); vs[7] = scale_of<3>(C.vs[1]);
  }
  if (!full) {    // unwritten bytes behind the last token: any finite value, their weights are 0
#pragma unroll
    for (int j = 0; j < 8; j++) vs[j] = bits_f(min(__float_as_uint(vs[j]) & 0x7F800000u, (uint32_t)(E_MAX + 127) << 23));
  }
#pragma unroll
  for (int b = 0; b < D / 32; b++) {                   // bytes of one token and lane
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t x, y;
      if (b == 0) { x = cvt2<0>(C.v[2 * j], vs[2 * j]); y = cvt2<0>(C.v[2 * j + 1], vs[2 * j + 1]); }
      else if (b == 1) { x = cvt2<1>(C.v[2 * j], vs[2 * j]); y = cvt2<1>(C.v[2 * j + 1], vs[2 * j + 1]); }
      else if (b == 2) { x = cvt2<2>(C.v[2 * j], vs[2 * j]); y = cvt2<2>(C.v[2 * j + 1], vs[2 * j + 1]); }
      else { x = cvt2<3>(C.v[2 * j], vs[2 * j]); y = cvt2<3>(C.v[2 * j + 1], vs[2 * j + 1]); }
      lo[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
      hi[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
    }
    const f16x8 fl = frag(lo[0], lo[1], lo[2], lo[3]), fh = frag(hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      o[nt][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fl, P[nt], o[nt][2 * b], 0, 0, 0);
      o[nt][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fh, P[nt], o[nt][2 * b + 1], 0, 0, 0);
    }
  }
}

// o *= f of tile nt where any lane of `far` is set (accumulators of 16 rows and
// D channels: D/4 registers)
template <int D, int NT>
__device__ __forceinline__ void scale_rows(uint64_t far, float f, f32x4 (*o)[D / 16], int nt) {
  if constexpr (D == 128) {
    f32x4* x = o[nt];
    if (nt == 0)
      SCALE_WHERE(far, f, 96, 32, AT(96:99)(x[0]), AT(100:103)(x[1]), AT(104:107)(x[2]), AT(108:111)(x[3]),
                  AT(112:115)(x[4]), AT(116:119)(x[5]), AT(120:123)(x[6]), AT(124:127)(x[7]));
    else
      SCALE_WHERE(far, f, 128, 32, AT(128:131)(x[0]), AT(132:135)(x[1]), AT(136:139)(x[2]), AT(140:143)(x[3]),
                  AT(144:147)(x[4]), AT(148:151)(x[5]), AT(152:155)(x[6]), AT(156:159)(x[7]));
  } else {
    f32x4* x = o[nt];
    if (nt == 0)
      SCALE_WHERE(far, f, 96, 16, AT(96:99)(x[0]), AT(100:103)(x[1]), AT(104:107)(x[2]), AT(108:111)(x[3]));
    else
      SCALE_WHERE(far, f, 112, 16, AT(112:115)(x[0]), AT(116:119)(x[1]), AT(120:123)(x[2]), AT(124:127)(x[3]));
  }
}

// Few query rows per key/value head (a token's head group, drafted tokens):
// the cache's bytes bound the work, so nothing is staged.  One workgroup =
// one (request, head, tile of 16 NT rows, split of the cache); its NWV
// waves take every NWV-th chunk straight from memory into the operands'
// registers and join their running softmaxes through LDS at the end.
// Measured (32 heads over 8, d = 128, one token): 8 requests of 32,768 to
// 131,072 tokens 147 us for 777 MB of codes and scales = 5.3 TB/s; 64 of 2,048 to
// 8,191 tokens 71 us = 5.1 TB/s (a plain read past the caches runs at 7.0, a
// copy at 5.16; the vector units are busy 40 % of the time, the rest is the
// chain of a chunk: keys, products, weights, products); one of 1,021 tokens
// 8.9 us.  Three tokens of 8 heads each over windows of 1,024 at d = 64, 128
// requests: 17.1 us, the vector units busy 29 % of them: two waves a SIMD, and
// each chunk of a wave waits for its own loads.  Rows from 17 on: 16 requests of
// up to 8,192 tokens 24 rows 40 us, 36 rows 41, 64 rows 60 (the bytes take 17 to 20):
// at 191 registers two workgroups a CU, and each tile of 32 rows reads and
// unpacks the cache for itself.
template <int D, int TYPE, int NT, int NWV, bool ONCE, int MODE>
__device__ __forceinline__ void attend_rows(const ArgsOf<MODE>& A, uint32_t bx, int by, int bz, f32x4 (*so)[NT * (D / 16)][64], f32x2 (*sml)[NT][16]) {
  constexpr int NC = D / 16;
  const int lane = threadIdx.x & 63, n = lane & 15, G = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  // the splits slowest: a short request has none of the last ones, and
  // neighbouring workgroups go to different XCDs
  int i = quot(bx, A.by_hkv), tile = by;
  const int h = bx - i * A.hkv;
  int sp = bz;
  Req R;
  int shared = 0, pre_per = 0;
  bool pre = false;            // SUFFIX: a tile of rows of a whole group over what they share
  if constexpr (MODE == SUFFIX) {
    const Whole whole_batch(A);
    if (i < A.pre_units) {
      if (tile > 0 || sp > 0) return;
      pre = true;
      Whole::Part part;
      const bool on = whole_batch.part(16 * NT, i, &part);
      if (bx == 0 && threadIdx.x == 0) A.shared[A.n_req] = part.per;
      if (!on) return;
      const Members m = whole_batch.group(part.g);
      tile = part.tile;
      sp = part.sp;
      pre_per = part.per;
      R.first = m.first;
      R.n_new = m.last - m.first;
      R.base = m.len;                                    // (no row lies before what is shared)
      i = m.s;                                           // by the table of the first
    } else {
      i -= A.pre_units;
      R = req_args(A, i);
      shared = whole_batch.shared_of(i);
    }
  } else if constexpr (MODE == LIST) {
    const int x = i;
    i = quot(x, A.by_max_new);
    const int j = x - i * A.max_new;
    R = req_args(A, i);
    if (j >= R.n_new) return;
    R.first += j;
    R.base += j;
    R.n_new = 1;
  } else {
    R = req_args(A, i);
  }
  const int fresh = pre ? R.n_new : min(R.n_new, A.max_new), rows = fresh * A.group, row0 = tile * 16 * NT;
  if (row0 >= rows) return;
  int p0 = R.base, p1 = R.base + fresh - 1;             // positions of the tile's first and last row
  if (MODE == SPAN || (MODE == SUFFIX && !pre))
    if (A.tiles > 1) {
      p0 = R.base + quot(row0, A.by_group);
      p1 = R.base + quot(min(row0 + 16 * NT, rows) - 1, A.by_group);
    }
  Span sn = {0, 0, 0};
  int per = A.per;
  const int32_t* list = nullptr;
  if constexpr (MODE == SPAN) {
    sn = span_of(p0, p1, A.window, A.sink);
    per = split_chunks(A, sn.total);
  } else if constexpr (MODE == LIST) {
    list = A.sel + ((int64_t)R.first * A.hkv + h) * A.n_sel;
    sn.total = entries_of(A, list, p0) * (A.T >> 5);
    per = split_chunks(A, sn.total);
  } else if (pre) {
    sn.total = R.base >> 5;
    per = pre_per;
  } else {
    if (h == 0 && tile == 0 && sp == 0 && threadIdx.x == 0) A.shared[i] = shared;
    sn.lo = shared >> 5;
    sn.total = max((p1 >> 5) + 1 - sn.lo, 0);
    per = split_chunks(A, sn.total);
  }
  const int window = MODE == SPAN ? A.window : 0, sink = MODE == SPAN ? A.sink : 0;
  const int c0 = sp * per, c1 = min(c0 + per, sn.total);
  if (c0 >= c1 && (sp > 0 || pre)) return;
  // one part: its result is the output's
  const bool whole = !pre && sn.total <= per && (MODE != SUFFIX || sn.lo == 0);
  if constexpr (MODE == SUFFIX) sp += pre ? 0 : A.slot0;  // (a prefix' parts come first in the workspace)

  const int32_t* tab = A.table + (int64_t)i * A.cols;
  const int blk_shift = 31 - __builtin_clz(A.T) - 5;    // chunks of a block, as a power of two
  auto chunk_at = [&](int k) { return k < sn.n_low ? k : sn.lo + k - sn.n_low; };
  // The table entries of a wave's next 64 chunks lie in its lanes, so that no
  // chunk's loads wait for a load of their own.
  Chunk<D> C;
  const Places<D> W(A.T);
  const uint32_t block_bytes = (uint32_t)A.T * D / 16 * 17;
  int k = c0 + wave, ahead = 0, entry = 0, first_of = 0;
  struct Next { const uint8_t* base; uint32_t off; bool dead; int t; };
  // Where chunk kf lies.  Past the end the last chunk once more: the loads are
  // always made (from the cache then); with a branch around them the compiler has to
  // wait for all of them at the first use of any.
  auto locate = [&](int kf) {
    if ((ahead & 63) == 0) {
      if constexpr (MODE == LIST) {
        const int kk = min(kf + NWV * lane, c1 - 1), col = list[kk >> blk_shift];
        const bool on = listed(A, col, p0);
        entry = tab[on ? col : 0];
        if (!on) entry = -1;
        first_of = (on ? col * A.T : 0) + 32 * (kk & ((1 << blk_shift) - 1));
        asm volatile("" : "+v"(first_of));
      } else {
        entry = tab[chunk_at(min(kf + NWV * lane, c1 - 1)) >> blk_shift];
      }
      asm volatile("" : "+v"(entry));     // (waited for here, not behind the branch, where it would hold up every step)
    }
    Next x;
    const int blk = __builtin_amdgcn_readlane(entry, ahead & 63);
    x.dead = (uint32_t)blk >= (uint32_t)A.n_blocks;    // no block: no visible token (block 0 is read in its place)
    if constexpr (MODE == LIST) {
      x.t = __builtin_amdgcn_readlane(first_of, ahead & 63);
      x.off = x.t & (A.T - 1);
    } else {
      x.off = (chunk_at(min(kf, c1 - 1)) * 32) & (A.T - 1);
    }
    x.base = A.cache + ((uint64_t)(uint32_t)(x.dead ? 0 : blk) * A.hkv + h) * block_bytes;
    ahead++;
    return x;
  };
  auto keys = [&](const Next& x) {
    load_keys<D, ONCE>(C, W, x.base + x.off * (D / 2), x.base + A.T * D + x.off);
  };
  auto values = [&](const Next& x) {
    load_values<D, ONCE>(C, W, x.base + A.T * (D / 2) + x.off * (D / 2), x.base + A.T * D + A.T * (D / 32) + x.off);
  };
  Next at;
  at.dead = true;
  if (k < c1) {
    at = locate(k);
    keys(at);
    values(at);
  }
  f16x8 q[NT][D / 32];
  float cf[NT];
  int pos[NT];
  int64_t grow[NT];            // row of q and o as (token, head) index, -1 outside
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    // rows past the last compute the last one again and are not written
    const int r = min(row0 + 16 * nt + n, rows - 1), j = quot(r, A.by_group), g = r - j * A.group;
    grow[nt] = row0 + 16 * nt + n < rows ? (int64_t)(R.first + j) * A.hq + h * A.group + g : -1;
    pos[nt] = R.base + j;
    load_q<D, TYPE>(A, (int64_t)(R.first + j) * A.qs + (int64_t)(h * A.group + g) * D + G * (D / 4), q[nt], &cf[nt]);
  }
  Ref ref[NT];
  uint64_t steep[NT];
  float l[NT];             // this lane group's part of the sum
  f32x4 o[NT][NC];
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    ref[nt].init();
    steep[nt] = 0;
    l[nt] = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; c++) o[nt][c] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }
  // One set of registers for the codes: the next chunk's keys are asked for as
  // soon as this one's are unpacked, its values likewise; the other waves of
  // the SIMD cover what that does not (a second set takes the registers of one or
  // two waves: 147 -> 162 us and 73 -> 77 for the long and the ragged batch).
  while (k < c1) {
    const int t0 = MODE == LIST ? at.t : chunk_at(k) * 32, t1 = t0 + 31;
    const bool dead = at.dead, full = !dead && t1 <= p0 && (window == 0 || t0 > p1 - window || t1 < sink);
    k += NWV;
    f32x4 s[NT][2];
    key_products<D, NT>(C, q, s);
    at = locate(k);
    keys(at);
    f16x8 P[NT];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      if (!full) {
        const int low = window == 0 ? -1 : pos[nt] - window, last = dead ? -1 : pos[nt];
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int t = t0 + token_of<D>(G, e);
          const int see = (int)(t <= last) & ((int)(t > low) | (int)(t < sink));
          s[nt][e >> 2][e & 3] = see ? s[nt][e >> 2][e & 3] : NEG_INF;
        }
      }
      float m = s[nt][0][0];
#pragma unroll
      for (int e = 1; e < 8; e++) m = __builtin_fmaxf(m, s[nt][e >> 2][e & 3]);
      const uint64_t far = __builtin_amdgcn_ballot_w64(m > ref[nt].over);
      float f = 1.0f;
      if (far) {
        f = ref[nt].move(__builtin_fmaxf(ref[nt].m, max_quads(m)), cf[nt]);
        steep[nt] = __builtin_amdgcn_ballot_w64(ref[nt].steep());
      }
      l[nt] *= f;
      scale_rows<D, NT>(far, f, o, nt);
      float mc = ref[nt].mc;
      if (steep[nt]) {
        mc = -LIFT;
#pragma unroll
        for (int e = 0; e < 8; e++) s[nt][e >> 2][e & 3] -= ref[nt].at();
      }
      // Weights to binary16 in pairs; the sum takes the same rounded weights, so
      // that a weight's rounding moves o by its own part only.
      uint32_t pk[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nt][e >> 1][2 * (e & 1)], cf[nt], -mc));
        const float b2 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nt][e >> 1][2 * (e & 1) + 1], cf[nt], -mc));
        const f16x2 hh = weights<TYPE>(a, b2);
        pk[e] = h2_bits(hh);
        l[nt] = __builtin_amdgcn_fdot2(hh, (f16x2){(f16)1.0f, (f16)1.0f}, l[nt], false);
      }
      P[nt] = frag(pk[0], pk[1], pk[2], pk[3]);
    }
    value_products<D, NT>(C, full, P, o);
    values(at);
  }
  if constexpr (NWV == 1) {    // a wave on its own takes whole lists: a lane holds channels (D/16)(4G + i) .. in tiles 0 ..
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const float L = sum_quads(l[nt]);
      if (grow[nt] < 0) continue;
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      const int64_t t = R.first + quot(row0 + 16 * nt + n, A.by_group);
      uint16_t* out = (uint16_t*)A.o + t * A.os + (grow[nt] - t * A.hq) * D + NC * 4 * G;
#pragma unroll
      for (int i4 = 0; i4 < 4; i4++) {
        uint32_t y[NC / 2];
#pragma unroll
        for (int c = 0; c < NC / 2; c++) y[c] = pack2<TYPE>(o[nt][2 * c][i4] * inv, o[nt][2 * c + 1][i4] * inv);
        if constexpr (NC == 8) *(u32x4*)(out + NC * i4) = (u32x4){y[0], y[1], y[2], y[3]};
        else *(u32x2*)(out + NC * i4) = (u32x2){y[0], y[1]};
      }
    }
    return;
  }
  // Join the waves through LDS, each of them a share of the channels: the
  // waves' sums are rescaled to the row's largest product where they are read.
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    l[nt] = sum_quads(l[nt]);
    if (G == 0) sml[wave][nt][n] = (f32x2){ref[nt].m, l[nt]};
#pragma unroll
    for (int c = 0; c < NC; c++) so[wave][nt * NC + c][lane] = o[nt][c];
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    if (grow[nt] < 0) continue;
    f32x2 ml[NWV];
    float M = NEG_INF;
#pragma unroll
    for (int w = 0; w < NWV; w++) {
      ml[w] = sml[w][nt][n];
      M = __builtin_fmaxf(M, ml[w][0]);
    }
    const float M0 = M == NEG_INF ? 0.0f : M;
    float L = 0.0f, f[NWV];
#pragma unroll
    for (int w = 0; w < NWV; w++) {
      f[w] = __builtin_amdgcn_exp2f((ml[w][0] - M0) * cf[nt]);
      L = __builtin_fmaf(ml[w][1], f[w], L);
    }
    // tiles CW * wave ..: channels (D/16)(4G + i) + c
    constexpr int CW = NC > NWV ? NC / NWV : 1;
    if (CW * wave >= NC) break;
    f32x4 x[CW];
#pragma unroll
    for (int c = 0; c < CW; c++) {
      x[c] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NWV; w++) {
        const f32x4 y = so[w][nt * NC + CW * wave + c][lane];
#pragma unroll
        for (int i4 = 0; i4 < 4; i4++) x[c][i4] = __builtin_fmaf(y[i4], f[w], x[c][i4]);
      }
    }
    const int ch0 = NC * 4 * G + CW * wave;
    if (whole) {
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      const int64_t t = R.first + quot(row0 + 16 * nt + n, A.by_group);
      uint16_t* out = (uint16_t*)A.o + t * A.os + (grow[nt] - t * A.hq) * D + ch0;
#pragma unroll
      for (int i4 = 0; i4 < 4; i4++) {
        if constexpr (CW == 2) *(uint32_t*)(out + NC * i4) = pack2<TYPE>(x[0][i4] * inv, x[1][i4] * inv);
        else out[NC * i4] = (uint16_t)pack2<TYPE>(x[0][i4] * inv, 0.0f);
      }
    } else {
      const int64_t row = (int64_t)sp * A.n_tok * A.hq + grow[nt];
      // (parts of a shared prefix may come from k_attend_tiles, whose sums count from the reference's lift)
      const float at_m = MODE == SPAN ? M * cf[nt] : M == NEG_INF ? NEG_INF : __builtin_fmaf(M, cf[nt], -LIFT);
      if (G == 0 && wave == 0) *(f32x2*)(A.pml + 2 * row) = (f32x2){at_m, L};
      float* out = A.po + row * D + ch0;
#pragma unroll
      for (int i4 = 0; i4 < 4; i4++) {
        if constexpr (CW == 2) *(f32x2*)(out + NC * i4) = (f32x2){x[0][i4], x[1][i4]};
        else out[NC * i4] = x[0][i4];
      }
    }
  }
}

template <int D, int TYPE, int NT, int NWV, bool ONCE, int MODE = SPAN>
__global__ void __launch_bounds__(64 * NWV, NWV == 16 ? 4 : 2) k_attend_rows(ArgsOf<MODE> A) {
  __shared__ f32x4 so[NWV][NT * (D / 16)][64];
  __shared__ f32x2 sml[NWV][NT][16];
  attend_rows<D, TYPE, NT, NWV, ONCE, MODE>(A, blockIdx.x, blockIdx.y, blockIdx.z, so, sml);
}

// Many query rows per key/value head (prompts): the matrix products bound the
// work.  One workgroup = one (request, head, tile of 128 rows, split), each wave
// 32 rows.  Tiles of 64 cached tokens (two chunks) go through LDS as
// binary16, unpacked once for all the waves, double buffered: while the waves
// work on one tile, the next one's bytes are converted and the one after it
// is on its way from memory.  One barrier per tile.
//
// Products as in k_attend_rows (transposed, so that a lane keeps one query
// row's statistics), on the 32x32x16 shape: lane n = lane % 32 is query row
// n, and lane half G holds tokens 8a + 4G + b (b < 4) of a 32-token chunk in
// elements 4a + b.  Eight consecutive elements are the operand of a product
// over 16 tokens; the values meet it through ds_read_tr16_b64, which gives
// lane i of 16 lanes channel i of four tokens whose 16-channel rows the lanes
// address (lane 4t + c: channels 4c.. of token t).
//
// Measured (4 prompts of 1,078 to 2,048 tokens over up to 2,048 cached ones, 32
// heads over 8, d = 128): 236 us = 905 TFLOP/s (226 to 238 by the card's clocks), where a library product of
// 8,192 x 8,192 x 8,192 in binary16 runs at 1,150.  A tile costs a wave about
// 1,000 cycles of matrix instructions and as many of vector ones (32 exp2 at
// half rate, the conversions, the sums), which share the SIMD's issue with the
// other wave's; 256 registers allow two.  (Eight waves over 256 rows, one
// workgroup a CU: 441 us, its waves wait for each other in step; products one
// chunk ahead instead of a tile: 268 against 253.)
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __fp16 fp16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) fp16x4 lds_fp16x4;

// 16-byte slot of (token t of 64, channels 8c ..).  The channel part is xored
// with bits of the token so that the 16 lanes of a read phase touch 16 different
// slots of the banks (a write phase is eight lanes: see `tk`); as xors the places of a lane's other
// channels are its first place with constant bits turned.
template <int D>
__device__ __forceinline__ int k_slot(int t, int c) {
  if constexpr (D == 128) return t * 16 + (c ^ (t & 15));
  else return t * 8 + (c ^ ((t >> 1) & 7));
}
template <int D>
__device__ __forceinline__ int v_slot(int t, int c) {
  if constexpr (D == 128) return t * 16 + (c ^ (4 * (t & 3) + ((t >> 2) & 3)));
  else return t * 8 + (c ^ (4 * ((t >> 1) & 1) + ((t >> 2) & 3)));
}

__device__ __forceinline__ float max_halves(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_fmaxf(bits_f(a[0]), bits_f(a[1]));
}

// The x-th tile of a batch: request and first row.  Of up to 64 requests (one a
// lane) the tiles come by the position they end at, in bands a tile high, the
// latest first: they have the most to see, and a list that goes from long to
// short leaves the least of the card idle at its end; no workgroup but the
// last ones is without a tile.  (Requests in their own order met the same shader
// engine again and again, since workgroups are dealt to the XCDs and engines
// in turn: 4 prompts of 1,078 to 2,048 tokens 488 us, rotated from level to level
// 325; a loop of 253 us rotated took 234 so.)
// More requests: each one's last tile first, the requests rotated from level to level.
__device__ __forceinline__ bool tile_of(const AttnArgs& A, int rows_of_tile, int x, int* req, int* row0) {
  if (A.n_req > 64) {
    const int level = x / A.n_req;
    const int i = (x % A.n_req + (level >> 1)) % A.n_req;
    const Req R = req_args(A, i);
    *req = i;
    *row0 = ((min(R.n_new, A.max_new) * A.group + rows_of_tile - 1) / rows_of_tile - 1 - level) * rows_of_tile;
    return *row0 >= 0;
  }
  const int lane = threadIdx.x & 63, i = min(lane, A.n_req - 1);
  const Req R = req_of(A, A.tok_start[i], A.tok_start[i + 1], A.len[i]);
  const int fresh = min(R.n_new, A.max_new);
  const int tiles = lane < A.n_req ? (fresh * A.group + rows_of_tile - 1) / rows_of_tile : 0;
  const int last = tiles > 0 ? R.base + fresh : -(1 << 30);    // behind the last query's position
  const int band = max(rows_of_tile / A.group, 1);
  const int top = wave_max_i(last);                      // (by all lanes)
  const int skip = tiles > 0 ? (top - last) / band : 0;  // bands above the request's first
  int lo = 0, hi = wave_max_i(skip + tiles);
  if (x >= wave_sum_i(tiles)) return false;
  while (hi - lo > 1) {                                  // the band that holds tile x: at most x tiles lie above it
    const int mid = (lo + hi) >> 1;
    if (wave_sum_i(min(max(mid - skip, 0), tiles)) <= x) lo = mid; else hi = mid;
  }
  uint64_t in = __builtin_amdgcn_ballot_w64(lo >= skip && lo < skip + tiles);
  for (int k = x - wave_sum_i(min(max(lo - skip, 0), tiles)); k > 0; k--) in &= in - 1;
  *req = __builtin_ctzll(in);
  *row0 = (__builtin_amdgcn_readlane(tiles, *req) - 1 - (lo - __builtin_amdgcn_readlane(skip, *req))) * rows_of_tile;
  return true;
}

constexpr int TILE_WAVES = 4;
template <int D, int TYPE, int MODE = SPAN>
__global__ void __launch_bounds__(64 * TILE_WAVES, 2) k_attend_tiles(ArgsOf<MODE> A) {
  constexpr int ROWS = 32 * TILE_WAVES;
  constexpr int KSTEP = D / 16, NC = D / 32;
  __shared__ __attribute__((aligned(16))) uint8_t lds_k[2][64 * D * 2], lds_v[2][64 * D * 2];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, G = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int b = blockIdx.x;
  if constexpr (MODE == PREFIX) {
    // Behind the prefixes' parts, where there are few rows of a request's own, these
    // too: they wait for memory where the others wait for the matrix cores.
    if (b >= A.pre_blocks) {
      const uint32_t x = b - A.pre_blocks, sp = x / (uint32_t)(A.n_req * A.hkv);
      attend_rows<D, TYPE, 1, 4, false, SUFFIX>(A, x - sp * (uint32_t)(A.n_req * A.hkv), 0, sp, (f32x4(*)[D / 16][64])lds_k[0], (f32x2(*)[1][16])lds_v[0]);
      return;
    }
  }
  // heads fastest: a head's workgroups share an XCD where the heads are a
  // multiple of 8
  const int h = b % A.hkv; b /= A.hkv;
  int sp = MODE == PREFIX ? 0 : b % A.splits;
  int i, row0, shared = 0, pre_per = 0;
  Req R;
  if constexpr (MODE == PREFIX) {
    const Whole whole_batch(A);
    Whole::Part part;
    const bool on = whole_batch.part(ROWS, b, &part);
    if (blockIdx.x == 0 && tid == 0) A.shared[A.n_req] = part.per;
    if (!on) return;
    const Members m = whole_batch.group(part.g);
    row0 = part.tile * ROWS;
    sp = part.sp;
    pre_per = part.per;
    R.first = m.first;
    R.n_new = m.last - m.first;
    R.base = m.len;                                      // (no row lies before what is shared)
    i = m.s;                                             // by the table of the first
  } else {
    if (!tile_of(A, ROWS, b / A.splits, &i, &row0)) return;
    R = req_args(A, i);
    if constexpr (MODE == SUFFIX) shared = Whole(A).shared_of(i);
  }
  const int rows = (MODE == PREFIX ? R.n_new : min(R.n_new, A.max_new)) * A.group;
  if (row0 < 0 || row0 >= rows) return;
  const int p0 = R.base + row0 / A.group, p1 = R.base + (min(row0 + ROWS, rows) - 1) / A.group;
  Span sn = {0, 0, 0};
  int per;
  if constexpr (MODE == SPAN) {
    sn = span_of(p0, p1, A.window, A.sink);
    per = split_chunks(A, sn.total);
  } else if constexpr (MODE == PREFIX) {
    sn.total = R.base >> 5;
    per = pre_per;
  } else {
    if (h == 0 && row0 == 0 && sp == 0 && tid == 0) A.shared[i] = shared;
    sn.lo = shared >> 5;
    sn.total = max((p1 >> 5) + 1 - sn.lo, 0);
    per = split_chunks(A, sn.total);
  }
  const int window = MODE == SPAN ? A.window : 0, sink = MODE == SPAN ? A.sink : 0;
  const int c0 = sp * per, c1 = min(c0 + per, sn.total);
  if (c0 >= c1 && (sp > 0 || MODE == PREFIX)) return;
  const int parts = MODE == PREFIX || (MODE == SUFFIX && sn.lo > 0) ? 2 : (sn.total + per - 1) / per;
  if constexpr (MODE == SUFFIX) sp += A.slot0;          // (a prefix' parts come first in the workspace)

  // the wave's rows
  const bool on = row0 + 32 * wave + n < rows;         // rows past the last compute the last one again and are not written
  const int r = min(row0 + 32 * wave + n, rows - 1), j = r / A.group, g = r - j * A.group;
  const int pw1 = R.base + (min(row0 + 32 * wave + 32, rows) - 1) / A.group;
  const int pw0 = min(R.base + (row0 + 32 * wave) / A.group, pw1), pos = R.base + j;
  f16x8 q[KSTEP];
  float cf;
  auto queries = [&] {
    float x[D / 2];
    const int64_t at = (int64_t)(R.first + j) * A.qs + (int64_t)(h * A.group + g) * D + 8 * G;
#pragma unroll
    for (int s = 0; s < KSTEP; s++) load8<TYPE>(A.q, at + 16 * s, x + 8 * s);
    float m = 0.0f;
#pragma unroll
    for (int u = 0; u < D / 2; u++) m = __builtin_fmaxf(m, __builtin_fabsf(x[u]));
    m = max_halves(m);
    const int e = q_shift(m);
    const float sign = A.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
    for (int s = 0; s < KSTEP; s++)
#pragma unroll
      for (int u = 0; u < 8; u++) q[s][u] = (f16)(sign * __builtin_ldexpf(x[8 * s + u], e));
    cf = q_factor(A.scale, e);
  };
  if (MODE == SPAN) queries();
  f32x16 o[NC];
#pragma unroll
  for (int c = 0; c < NC; c++)
#pragma unroll
    for (int u = 0; u < 16; u++) o[c][u] = 0.0f;
  Ref ref;
  ref.init();
  uint64_t steep = 0;
  float L = 0.0f;

  const int32_t* tab = A.table + (int64_t)i * A.cols;
  const int T = A.T, blk_shift = 31 - __builtin_clz(T) - 5;
  auto chunk_at = [&](int k) { return k < sn.n_low ? k : sn.lo + k - sn.n_low; };
  // This thread's piece of a tile's keys and of its values: a quarter of a
  // token's codes; waves 0 and 1 chunk k's, 2 and 3 chunk k + 1's, 16 tokens
  // each.  Which lane takes which piece is chosen so that eight lanes in turn,
  // which a 16-byte write to LDS serves at once, meet eight different slots of
  // the banks' 128 bytes (tokens or pieces in order: two-way conflicts, 13 % of
  // the LDS' time).
  constexpr int PS = D / 32;                           // dwords, and slots, of a piece
  const int half = wave >> 1;
  auto bit = [&](int x) { return (lane >> x) & 1; };
  const int ck = D == 128 ? bit(0) + 2 * bit(3) : bit(0) + 2 * bit(1), cv = ck;
  const int tk = 16 * (wave & 1) + 8 * bit(5) + 4 * bit(4) + (D == 128 ? 2 * bit(2) + bit(1) : 2 * bit(2) + bit(3));
  const int tv = 16 * (wave & 1) + (D == 128 ? 8 * bit(2) + 4 * bit(1) + 2 * bit(5) + bit(4) : 8 * bit(5) + 4 * bit(2) + 2 * bit(4) + bit(3));
  const uint32_t kc_at = tk * (D / 2) + 4 * PS * ck, ks_at = T * D + (PS * ck / 4) * T + tk;
  const uint32_t vc_at = T * (D / 2) + tv * (D / 2) + 4 * PS * cv, vs_at = T * D + T * (D / 32) + (PS * cv / 4) * T + tv;
  const uint32_t k_put = 16 * k_slot<D>(32 * half + tk, PS * ck), v_put = 16 * v_slot<D>(32 * half + tv, PS * cv);
  const uint32_t block_bytes = (uint32_t)T * D / 16 * 17;
  int ahead = 0, entry = 0;
  // A tile: chunks k, k + 1; gone: which of them hold no visible token because
  // they lie past the end or in no block.
  struct Tile { int k; uint32_t blk[2]; int gone; };
  auto locate = [&](int k) {
    if ((ahead & 63) == 0) {
      entry = tab[chunk_at(min(k + lane, c1 - 1)) >> blk_shift];
      asm volatile("" : "+v"(entry));
    }
    const uint32_t e0 = __builtin_amdgcn_readlane(entry, ahead & 63), e1 = __builtin_amdgcn_readlane(entry, (ahead & 63) + 1);
    ahead += 2;
    Tile x;
    x.k = k;
    x.gone = (e0 >= (uint32_t)A.n_blocks || k >= c1 ? 1 : 0) | (e1 >= (uint32_t)A.n_blocks || k + 1 >= c1 ? 2 : 0);
    x.blk[0] = e0 < (uint32_t)A.n_blocks ? e0 : 0;
    x.blk[1] = e1 < (uint32_t)A.n_blocks ? e1 : 0;
    return x;
  };
  typedef uint32_t piece_t __attribute__((ext_vector_type(PS)));
  piece_t kraw, vraw;
  uint32_t ksb, vsb;
  auto base_of = [&](const Tile& x) {                  // this wave's chunk: its head's bytes from the chunk's first token slot on
    const uint32_t off = (chunk_at(min(x.k + half, c1 - 1)) * 32) & (T - 1);
    return A.cache + ((uint64_t)(half ? x.blk[1] : x.blk[0]) * A.hkv + h) * block_bytes + off;
  };
  auto off_of = [&](const Tile& x) { return (uint32_t)((chunk_at(min(x.k + half, c1 - 1)) * 32) & (T - 1)) * (D / 2 - 1); };
  auto fetch = [&](const Tile& x, uint32_t code_at, uint32_t scale_at, piece_t& raw, uint32_t& sb) {
    const uint8_t* p = base_of(x);
    raw = *(const piece_t*)(p + off_of(x) + code_at);
    sb = p[scale_at];
  };
  auto put = [&](uint8_t* buf, uint32_t at, const piece_t& raw, float sc) {
#pragma unroll
    for (int x = 0; x < PS; x++)
      *(u32x4*)(buf + (at ^ (16 * x))) = (u32x4){cvt2<0>(raw[x], sc), cvt2<1>(raw[x], sc), cvt2<2>(raw[x], sc), cvt2<3>(raw[x], sc)};
  };
  // (Unwritten bytes behind the last token must not be NaN or infinite as
  // values, their weights are 0; keys keep the NaN of scale byte 255.)
  auto fetch_k = [&](const Tile& x) { fetch(x, kc_at, ks_at, kraw, ksb); };
  auto fetch_v = [&](const Tile& x) { fetch(x, vc_at, vs_at, vraw, vsb); };
  auto put_k = [&](int b) { put(lds_k[b], k_put, kraw, scale_of<0>(ksb)); };
  auto put_v = [&](int b) { put(lds_v[b], v_put, vraw, scale_of<0>(min(vsb, (uint32_t)(E_MAX + 127)))); };
  // in the loop: the values of the next tile and the keys of the one after it
  // move to buffers vb and kb, the ones behind them (tiles xv, xk) are asked for
  auto stage = [&](int vb, int kb, const Tile& xv, const Tile& xk) {
    put_v(vb);
    put_k(kb);
    fetch_v(xv);
    fetch_k(xk);
  };
  // Where this lane reads: keys (token n, channels 8G .., and 16x more), values
  // (tokens 4G + .. and 8 more; four channels, and 32c more); other tokens of
  // the tile lie whole rows on.
  const uint32_t k_at = 16 * k_slot<D>(n, G);
  const int vt = 4 * G + ((lane >> 2) & 3), vch = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const uint32_t v_at[2] = {16u * v_slot<D>(vt, vch >> 3) + 8 * ((vch >> 2) & 1), 16u * v_slot<D>(vt + 8, vch >> 3) + 8 * ((vch >> 2) & 1)};
  auto key_tile = [&](const uint8_t* buf, f32x16* s) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
#pragma unroll
      for (int x = 0; x < 16; x++) s[u][x] = 0.0f;
#pragma unroll
      for (int x = 0; x < KSTEP; x++) {
        const f16x8 kf = *(const f16x8*)(buf + u * 32 * D * 2 + (k_at ^ (32 * x)));
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, q[x], s[u], 0, 0, 0);
      }
    }
  };
  // One tile: its products s become weights and meet its values, while the
  // matrix cores make the next tile's products sn (nothing of one waits for the
  // other, so the compiler interleaves them).
  auto work = [&](const Tile& x, f32x16* s, f32x16* sn, const uint8_t* next_k, const uint8_t* v, auto&& move_on) {
    const int ta = chunk_at(x.k) * 32, tb = chunk_at(min(x.k + 1, c1 - 1)) * 32;
    const bool in_a = window == 0 || ta > pw1 - window || ta + 31 < sink;
    const bool in_b = window == 0 || tb > pw1 - window || tb + 31 < sink;
    if (x.gone || (MODE != PREFIX && tb + 31 > pw0) || !in_a || !in_b) {
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const int t0 = (u ? tb : ta) + 4 * G, low = window == 0 ? -1 : pos - window;
        const int last = x.gone & (1 << u) ? -1 : pos;
#pragma unroll
        for (int e = 0; e < 16; e++) {
          const int t = t0 + 8 * (e >> 2) + (e & 3);
          const int see = (int)(t <= last) & ((int)(t > low) | (int)(t < sink));
          s[u][e] = see ? s[u][e] : NEG_INF;
        }
      }
    }
    float m = s[0][0];
#pragma unroll
    for (int e = 1; e < 32; e++) m = __builtin_fmaxf(m, s[e >> 4][e & 15]);
    const uint64_t far = __builtin_amdgcn_ballot_w64(m > ref.over);
    float f = 1.0f;
    if (far) {
      f = ref.move(__builtin_fmaxf(ref.m, max_halves(m)), cf);
      steep = __builtin_amdgcn_ballot_w64(ref.steep());
    }
    L *= f;
    if constexpr (NC == 4)
      SCALE_WHERE(far, f, 192, 64, AT(192:207)(o[0]), AT(208:223)(o[1]), AT(224:239)(o[2]), AT(240:255)(o[3]));
    else
      SCALE_WHERE(far, f, 128, 32, AT(128:143)(o[0]), AT(144:159)(o[1]));
    float mc = ref.mc;
    if (steep) {
      mc = -LIFT;
#pragma unroll
      for (int e = 0; e < 32; e++) s[e >> 4][e & 15] -= ref.at();
    }
    // (the wave that has matrix work goes first: 234 -> 229 us)
    __builtin_amdgcn_s_setprio(1);
    key_tile(next_k, sn);
    f16x8 P[2][2];
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int y = 0; y < 2; y++) {                     // 16 tokens
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][8 * y + 2 * e], cf, -mc));
          const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][8 * y + 2 * e + 1], cf, -mc));
          const f16x2 hh = weights<TYPE>(e0, e1);
          pk[e] = h2_bits(hh);
          L = __builtin_amdgcn_fdot2(hh, (f16x2){(f16)1.0f, (f16)1.0f}, L, false);
        }
        P[u][y] = frag(pk[0], pk[1], pk[2], pk[3]);
      }
    move_on();
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int y = 0; y < 2; y++)
#pragma unroll
        for (int c = 0; c < NC; c++) {
          const uint8_t* at = v + (32 * u + 16 * y) * D * 2;
          const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4*)(at + (v_at[0] ^ (64 * c)))));
          const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_fp16x4*)(at + (v_at[1] ^ (64 * c)))));
          o[c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(frag(lo[0], lo[1], hi[0], hi[1]), P[u][y], o[c], 0, 0, 0);
        }
    __builtin_amdgcn_s_setprio(0);
  };
  if (MODE != SPAN && c0 >= c1) cf = 0.0f;
  if (c0 < c1) {
    Tile t0 = locate(c0), t1 = locate(c0 + 2), t2 = locate(c0 + 4);
    fetch_k(t0);
    fetch_v(t0);
    if (MODE != SPAN) queries();                        // (short parts: their loads on the way together)
    put_k(0);
    put_v(0);
    fetch_k(t1);
    fetch_v(t1);
    put_k(1);
    fetch_k(t2);
    __syncthreads();
    f32x16 sa[2], sb[2];
    key_tile(lds_k[0], sa);
    __syncthreads();
    // in LDS: the values of tile t0, the keys of t1; in registers: the values of
    // t1, the keys of t2
    for (int k = c0; k < c1; k += 4) {
      const Tile t3 = locate(k + 6);
      work(t0, sa, sb, lds_k[1], lds_v[0], [&] { stage(1, 0, t2, t3); });
      __syncthreads();
      if (k + 2 >= c1) break;
      const Tile t4 = locate(k + 8);
      work(t1, sb, sa, lds_k[0], lds_v[1], [&] { stage(0, 1, t3, t4); });
      __syncthreads();
      t0 = t2;
      t1 = t3;
      t2 = t4;
    }
  }
  {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(L), __float_as_uint(L), false, false);
    L = bits_f(a[0]) + bits_f(a[1]);
  }
  if (!on) return;
  // element 4a + b of tile c: channel 32c + 8a + 4G + b
  if (parts <= 1) {
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint16_t* out = (uint16_t*)A.o + (int64_t)(R.first + j) * A.os + (int64_t)(h * A.group + g) * D + 4 * G;
#pragma unroll
    for (int c = 0; c < NC; c++)
#pragma unroll
      for (int a = 0; a < 4; a++)
        *(u32x2*)(out + 32 * c + 8 * a) = (u32x2){pack2<TYPE>(o[c][4 * a] * inv, o[c][4 * a + 1] * inv),
                                                  pack2<TYPE>(o[c][4 * a + 2] * inv, o[c][4 * a + 3] * inv)};
  } else {
    const int64_t row = (int64_t)sp * A.n_tok * A.hq + (int64_t)(R.first + j) * A.hq + h * A.group + g;
    if (G == 0) {
      A.pml[2 * row] = ref.m == NEG_INF ? NEG_INF : ref.mc;
      A.pml[2 * row + 1] = L;
    }
    float* out = A.po + row * D + 4 * G;
#pragma unroll
    for (int c = 0; c < NC; c++)
#pragma unroll
      for (int a = 0; a < 4; a++)
        *(f32x4*)(out + 32 * c + 8 * a) = (f32x4){o[c][4 * a], o[c][4 * a + 1], o[c][4 * a + 2], o[c][4 * a + 3]};
  }
}

// Join the splits of one row: one wave per row, its channels over the lanes,
// the splits in order.
template <int D, int TYPE, int MODE = SPAN>
__global__ void __launch_bounds__(256) k_attend_join(ArgsOf<MODE> A, int tile_shift) {
  const int lane = threadIdx.x & 63;
  const int hd = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
  if (hd >= A.hq) return;
  const int i = quot(blockIdx.x, A.by_max_new), j = blockIdx.x - i * A.max_new;
  const Req R = req_args(A, i);
  const int fresh = min(R.n_new, A.max_new), rows = fresh * A.group;
  if (j >= fresh) return;
  int p0 = R.base, p1 = R.base + fresh - 1;             // as the tile's workgroups had them
  if (MODE != LIST && A.tiles > 1) {
    const int row0 = ((j * A.group + hd - quot(hd, A.by_group) * A.group) >> tile_shift) << tile_shift;
    p0 = R.base + quot(row0, A.by_group);
    p1 = R.base + quot(min(row0 + (1 << tile_shift), rows) - 1, A.by_group);
  }
  Span sn = {0, 0, 0};
  if constexpr (MODE == SPAN) {
    sn = span_of(p0, p1, A.window, A.sink);
  } else if constexpr (MODE == LIST) {
    sn.total = entries_of(A, A.sel + ((int64_t)(R.first + j) * A.hkv + quot(hd, A.by_group)) * A.n_sel, R.base + j) * (A.T >> 5);
  } else {
    sn.lo = ld_const(A.shared + i) >> 5;
    sn.total = max((p1 >> 5) + 1 - sn.lo, 0);
  }
  const int per = split_chunks(A, sn.total);
  if (sn.total <= per && (MODE != SUFFIX || sn.lo == 0)) return;   // written by its only part
  int parts = per == A.per ? quot(sn.total + per - 1, A.by_per) : (sn.total + per - 1) / per, shared_parts = 0, gap = 0;
  if constexpr (MODE == SUFFIX) {
    const int pre = sn.lo > 0 ? ld_const(A.shared + A.n_req) : 1;
    shared_parts = (sn.lo + pre - 1) / pre;
    parts += shared_parts;
    gap = A.slot0 - shared_parts;
  }
  auto at = [&](int s) { return MODE == SUFFIX && s >= shared_parts ? s + gap : s; };
  const int64_t stride = (int64_t)A.n_tok * A.hq, row = (int64_t)(R.first + j) * A.hq + hd;
  // statistics: part s on lane s (and s + 64)
  const f32x2 none = {NEG_INF, 0.0f};
  const f32x2* ml = (const f32x2*)A.pml + row;
  const f32x2 m0 = lane < parts ? ml[at(lane) * stride] : none, m1 = lane + 64 < parts ? ml[at(lane + 64) * stride] : none;
  // N parts from s on are under way at a time (the last one again where there
  // are fewer, not added): the first eight along with the statistics
  const float* po = A.po + row * D + lane * (D / 64);
  constexpr int FIRST = 8, MORE = 24;
  float y[MORE][D / 64];
  auto ask = [&](auto N, int s) {
#pragma unroll
    for (int e = 0; e < N; e++)
#pragma unroll
      for (int u = 0; u < D / 64; u++) y[e][u] = po[at(min(s + e, parts - 1)) * stride * D + u];
  };
  ask(std::integral_constant<int, FIRST>(), 0);
  float M = wave_max(__builtin_fmaxf(m0[0], m1[0]));
  if (M == NEG_INF) M = 0.0f;
  const float f0 = __builtin_amdgcn_exp2f(m0[0] - M), f1 = __builtin_amdgcn_exp2f(m1[0] - M);
  const float L = wave_sum(__builtin_fmaf(f0, m0[1], f1 * m1[1]));
  float x[D / 64];
#pragma unroll
  for (int u = 0; u < D / 64; u++) x[u] = 0.0f;
  auto add = [&](auto N, int s) {
#pragma unroll
    for (int e = 0; e < N; e++) {
      const float f = bits_f(__builtin_amdgcn_readlane(__float_as_uint(s + e < 64 ? f0 : f1), (s + e) & 63));
#pragma unroll
      for (int u = 0; u < D / 64; u++) x[u] = s + e < parts ? __builtin_fmaf(f, y[e][u], x[u]) : x[u];
    }
  };
  add(std::integral_constant<int, FIRST>(), 0);
  for (int s = FIRST; s < parts; s += MORE) {
    ask(std::integral_constant<int, MORE>(), s);
    add(std::integral_constant<int, MORE>(), s);
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint16_t* o = (uint16_t*)A.o + (int64_t)(R.first + j) * A.os + hd * D + lane * (D / 64);
  if constexpr (D == 128) *(uint32_t*)o = pack2<TYPE>(x[0] * inv, x[1] * inv);
  else *o = (uint16_t)pack2<TYPE>(x[0] * inv, 0.0f);
}

// ------------------------------------------------------------------ host
bool kv_ok(const stq_kv_desc* d) {
  return d && d->n_blocks >= 1 && d->n_kv_heads >= 1 && d->n_kv_heads <= 4096 && (d->d == 64 || d->d == 128) &&
         (d->block_tokens == 32 || d->block_tokens == 64 || d->block_tokens == 128 || d->block_tokens == 256);
}
uint64_t kv_size(const stq_kv_desc* d) {
  return (uint64_t)d->n_blocks * d->n_kv_heads * ((uint64_t)d->block_tokens * d->d * 17 / 16);
}
stq_status kv_check(const stq_kv_desc* d, const void* cache, size_t bytes) {
  if (!kv_ok(d)) return STQ_ERR_ARG;
  if (!cache || ((uintptr_t)cache & 15u) || bytes < kv_size(d)) return STQ_ERR_LAYOUT;
  return STQ_OK;
}
// A launch takes fewer than 2^32 threads in one direction; calls on more tokens go in slices.
constexpr int64_t MOST_THREADS = (1ll << 32) - 1, MOST_GROUPS = 1 << 23;
// The L2s of the eight dies together: a larger output cannot stay there for its
// reader, and stored past them it leaves room and saves their write-back
// (16,381 tokens of 40 heads normed 74.8 -> 67.8 us with loads past them as
// well, 32,749 tokens' values read back with the write before it 39.8 -> 29.2).
constexpr int64_t CACHE_BYTES = 32 << 20;
bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }
int elem_bytes(int type) { return type == STQ_FP32 ? 4 : 2; }
bool stride_ok(int64_t stride, int64_t least, int type) {
  return stride >= least && stride < (1ll << 40) && (stride * elem_bytes(type)) % 16 == 0;
}
// n rows of `bytes` bytes each, `step` bytes apart
struct Rows { const void* p; int64_t step, bytes; };
// Whether two tensors of n rows share a byte.  Rows of one buffer side by side
// (one step) are told apart exactly; with two steps, ranges that meet count.
bool meet(const Rows& a, const Rows& b, int64_t n) {
  const int64_t x = (int64_t)(uintptr_t)a.p, y = (int64_t)(uintptr_t)b.p;
  if (x + (n - 1) * a.step + a.bytes <= y || y + (n - 1) * b.step + b.bytes <= x) return false;
  if (a.step != b.step) return true;
  const int64_t gap = ((y - x) % a.step + a.step) % a.step;      // from a row of a to the next of b
  return gap < a.bytes || gap > a.step - b.bytes;
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.step == b.step && a.bytes == b.bytes; }
stq_status launched() { return hipGetLastError() == hipSuccess ? STQ_OK : STQ_ERR_HIP; }

// Positions lie in [-2^28, 2^30): a window of 2^30 is no limit, and the kernels'
// differences of the two stay in 32 bits.
constexpr int32_t MOST_WINDOW = 1 << 30;
bool attend_ok(const stq_kv_desc* d, const stq_attend_desc* a) {
  return a && a->n_req >= 0 && a->n_tok >= 0 && a->n_tok <= (1 << 28) && a->n_heads >= 1 && a->n_heads % d->n_kv_heads == 0 &&
         a->n_heads <= 65536 && (a->type == STQ_BF16 || a->type == STQ_FP16) && a->table_cols >= 1 &&
         (int64_t)a->table_cols * d->block_tokens <= (1ll << 30) && a->max_new >= 1 && a->max_len >= 1 &&
         a->window >= 0 && a->n_sink >= 0 && isfinite(a->scale);
}
struct Split { int tiles, tile_rows, splits, per, waves; bool staged, once; };
// Query rows per key/value head up to which each wave unpacks the cache for
// itself, 32 rows at a time; above, it is staged through LDS for 128 rows (16
// requests of up to 8,192 tokens, 8 heads, d = 128: 36 rows 41 against 63 us
// staged, 64 rows 60 against 67, 96 rows 76 against 70, 128 rows 90 against 76;
// 64 requests of up to 2,048: 64 rows 54 against 62, 96 rows 67 against 63; d = 64,
// 16 requests: 64 rows 45 against 58, 96 rows 56 against 60, 128 rows 68 against 63).
constexpr int STAGED_ROWS = 64;
// A part of a request's work has its own start (three dependent loads) and end
// (the joins), about 5 us.  Few workgroups are split down to 12 chunks, three a
// wave, until every CU holds two (1 x 16,000 tokens of 8 heads 13.9 us in parts of
// 8 chunks, 11.4 of 12, 12.0 of 16; 8 x 2,000 11.0, 9.9, 10.9; 1 x 2,000 8.0,
// 8.7, 9.8; 8 x 6,000 14.7 at two workgroups a CU, 16.1 at three); many only into parts of 48 chunks and up, which even
// out ragged lengths, and until every CU has eight of them (64 requests of 2,048
// to 8,191 tokens, 8 heads: 78 us at four workgroups a CU, 73 to 74 at six to
// sixteen; 83 whole and 91 in parts of 24 chunks before the loads past the
// caches; 8 requests of 32,768 to 131,072 tokens: 156 us at four, 153 at six, 146
// at eight, 150 at ten, 152 at sixteen).
constexpr int64_t CUS = 256, FEW_GROUPS = 512, FEW_CHUNKS = 12, MANY_GROUPS = 2048, MANY_CHUNKS = 48, MOST_SPLITS = 128;
// (sixteen: whether the caller has a kernel of sixteen waves, and would need no second launch)
void cut(Split* x, int64_t base, int64_t chunks, int64_t few_chunks = FEW_CHUNKS, bool sixteen = true) {
  Split& s = *x;
  auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
  int64_t k = 1;
  if (base > 0) {
    const int64_t few = least(FEW_GROUPS / base, chunks / few_chunks), many = least(MANY_GROUPS / base, chunks / MANY_CHUNKS);
    k = least(few > many ? few : many, MOST_SPLITS);
    if (k < 1) k = 1;
  }
  // One workgroup a CU or fewer, and requests that would be split in two (in up to
  // five where the workgroups are half the CUs and more): sixteen waves and no
  // second launch.  Below that four waves need none either.  Four waves against
  // sixteen, us on the GPU, 8 heads, d = 128: 1 request of 640 tokens 6.9, 7.7;
  // 736 7.6, 8.0; 768 8.1, 8.0; 960 8.7, 8.8 (a call 9.9, 8.8); 1,100 9.3, 9.1;
  // 1,216 8.7, 9.4; 1,500 8.9, 10.6.  32 requests of 736 9.1, 9.7; 768 11.6, 9.8; 2,000
  // 16.9, 14.1; 16 of 640 7.3, 8.1; 1,100 10.5, 10.1; 1,900 12.7, 12.5; 2,048 12.9,
  // 13.1.  (d = 64 gains from 640 on: 20 requests of 640 6.3, 6.2, of 2,048 11.9, 10.3.)
  s.waves = 4;
  if (sixteen && s.tile_rows == 16 && base <= CUS && chunks >= 2 * FEW_CHUNKS && chunks < (2 * base >= CUS ? 65 : 3 * FEW_CHUNKS)) {
    s.waves = 16;
    k = 1;
  }
  s.per = (int)(((chunks + k - 1) / k + 3) & ~3ll);
  s.splits = (int)((chunks + s.per - 1) / s.per);
}

}  // namespace
