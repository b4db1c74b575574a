// attn.hip — gfx950 kernels and C ABI of the softmax layers' operators
// (contract: include/stq.h, "THE SOFTMAX LAYERS OF A HYBRID MODEL"): the
// block plan, the norm and rotation of queries and keys, the 4-bit key/value
// cache and attention over it.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "stq.h"
#include "stq_device.h"

using namespace stq;

namespace {

typedef f16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int E_MIN = -23, E_MAX = 13;   // exponents of the cache's scales

__device__ __forceinline__ float bits_f(uint32_t u) { return __uint_as_float(u); }

// Eight consecutive elements as binary32 (16-byte loads; 2 of them for fp32).
template <int TYPE>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* x) {
  if constexpr (TYPE == STQ_FP32) {
    const f32x4* p = (const f32x4*)((const float*)base + at);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; i++) { x[i] = a[i]; x[4 + i] = b[i]; }
  } else {
    const u32x4 a = *(const u32x4*)((const uint16_t*)base + at);
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
template <int TYPE>
__device__ __forceinline__ void store8(void* base, int64_t at, const float* x) {
  if constexpr (TYPE == STQ_FP32) {
    f32x4* p = (f32x4*)((float*)base + at);
    p[0] = (f32x4){x[0], x[1], x[2], x[3]};
    p[1] = (f32x4){x[4], x[5], x[6], x[7]};
  } else {
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; i++) a[i] = pack2<TYPE>(x[2 * i], x[2 * i + 1]);
    *(u32x4*)((uint16_t*)base + at) = a;
  }
}

// ------------------------------------------------------------ block plan
//
// Every workgroup scans all n requests by itself (8 n bytes from the L2 and
// two scans in LDS), so the plan needs one launch and no traffic between
// workgroups; then the new table entries and the new tokens are dealt out
// over all threads.  A new token's block is taken from the free list, not
// from the table entry that another workgroup may still be writing.
constexpr int PLAN_MAX = 4096, PLAN_NT = 512;

struct PlanArgs {
  const int32_t *cached, *fresh, *free_list;
  int n, n_free, n_blocks, T, cols, n_tok;
  int32_t* table;
  int32_t *tok_start, *len, *pos, *used;
  int64_t* slot;
};

// largest i in [0, n) with start[i] <= x (start non-decreasing, start[0] = 0):
// the request that owns element x of a flattened list (empty requests skipped)
__device__ __forceinline__ int owner(const uint32_t* start, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(PLAN_NT) k_kv_plan(PlanArgs A) {
  extern __shared__ uint32_t sm[];
  const int n = A.n, tid = threadIdx.x;
  uint32_t* tok0 = sm;                 // [n + 1] first new token of request i
  uint32_t* blk0 = sm + n + 1;         // [n + 1] first new block of request i
  uint32_t* tot = blk0 + n + 1;        // [2][PLAN_NT / 64] totals of the waves
  const int T = A.T, cap = A.cols;
  constexpr int NW = PLAN_NT / 64;
  uint32_t run_t = 0, run_b = 0;
  for (int base = 0; base < n; base += PLAN_NT) {
    const int i = base + tid;
    uint32_t m = 0, add = 0;
    if (i < n) {
      const int64_t c = max(A.cached[i], 0);
      m = (uint32_t)max(A.fresh[i], 0);
      const int64_t have = min((c + T - 1) / T, (int64_t)cap), need = min((c + m + T - 1) / T, (int64_t)cap);
      add = (uint32_t)(need - have);
      if (blockIdx.x == 0) A.len[i] = (int32_t)min(c + (int64_t)m, (int64_t)INT32_MAX);
    }
    uint32_t st = m, sb = add;         // inclusive scans over the wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t a = __shfl_up(st, d, 64), b = __shfl_up(sb, d, 64);
      if ((tid & 63) >= d) { st += a; sb += b; }
    }
    if ((tid & 63) == 63) { tot[tid >> 6] = st; tot[NW + (tid >> 6)] = sb; }
    __syncthreads();
    uint32_t bt = run_t, bb = run_b;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      const uint32_t a = tot[w], b = tot[NW + w];
      if (w < (tid >> 6)) { bt += a; bb += b; }
      run_t += a;
      run_b += b;
    }
    if (i < n) { tok0[i] = bt + st - m; blk0[i] = bb + sb - add; }
    __syncthreads();
  }
  if (tid == 0) { tok0[n] = run_t; blk0[n] = run_b; }
  __syncthreads();
  const uint32_t step = gridDim.x * PLAN_NT, first = blockIdx.x * PLAN_NT + tid;
  for (uint32_t i = first; i <= (uint32_t)n; i += step) A.tok_start[i] = (int32_t)tok0[i];
  if (blockIdx.x == 0 && tid == 0) A.used[0] = (int32_t)run_b;
  for (uint32_t u = first; u < run_b; u += step) {
    const int i = owner(blk0, n, u);
    const int have = (int)(((int64_t)max(A.cached[i], 0) + T - 1) / T);
    const int64_t col = (int64_t)have + (u - blk0[i]);
    if (col < cap) A.table[(int64_t)i * cap + col] = u < (uint32_t)A.n_free ? A.free_list[u] : -1;
  }
  for (uint32_t t = first; t < (uint32_t)A.n_tok; t += step) {
    int32_t pos = -1;
    int64_t slot = -1;
    if (t < run_t) {
      const int i = owner(tok0, n, t);
      const int64_t c = max(A.cached[i], 0), p = c + (t - tok0[i]);
      const int64_t have = (c + T - 1) / T, col = p / T;
      pos = (int32_t)min(p, (int64_t)INT32_MAX);
      if (col < cap) {
        const uint32_t u = blk0[i] + (uint32_t)(col - have);
        const int blk = col < have ? A.table[(int64_t)i * cap + col] : (u < (uint32_t)A.n_free ? A.free_list[u] : -1);
        if ((uint32_t)blk < (uint32_t)A.n_blocks) slot = (int64_t)blk * T + p % T;
      }
    }
    A.pos[t] = pos;
    A.slot[t] = slot;
  }
}

// ------------------------------------------------- norm and rotation
//
// One row (head of a token) on D/8 lanes of eight channels each: the row
// stays in registers between its only load and its only store.  A wave takes
// 64/(D/8) heads of one token at a time, so that the token's cosines and sines
// are loaded once per lane and serve all its heads.
struct NormArgs {
  const void *q, *k;
  void *qo, *ko;
  const float *wq, *wk, *cs;
  const int32_t* pos;
  int n_tok, hq, hk, n_rot, n_pos, norm, adjacent;
  float eps;
  int64_t qs, ks, qos, kos;
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {   // over LPR consecutive lanes, every lane the same result
  x = x + dpp<0xB1>(x);
  x = x + dpp<0x4E>(x);
  x = x + dpp<0x141>(x);
  if (LPR >= 16) x = x + dpp<0x140>(x);
  if (LPR >= 32) x = x + __shfl_xor(x, 16, 64);
  return x;
}

template <int D, int IN, int OUT>
__global__ void __launch_bounds__(256) k_qk_norm_rope(NormArgs A) {
  constexpr int LPR = D / 8, RPW = 64 / LPR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane % LPR, c0 = 8 * li;
  const int64_t t = blockIdx.x;
  const int rows = A.hq + A.hk, R = A.n_rot;
  float cs[8], sn[8];
  bool turn = false;
  if (R > 0) {
    const int p = A.pos[t];
    if ((uint32_t)p >= (uint32_t)A.n_pos) return;    // a padded row (the whole workgroup's token)
    turn = c0 < R;
    if (turn) {
      const float* row = A.cs + (int64_t)p * R;
      if (A.adjacent) {                               // pair i: channels 2i, 2i + 1
#pragma unroll
        for (int i = 0; i < 4; i++) {
          cs[2 * i] = cs[2 * i + 1] = row[c0 / 2 + i];
          const float s = row[R / 2 + c0 / 2 + i];
          sn[2 * i] = -s;
          sn[2 * i + 1] = s;
        }
      } else {                                        // pair i: channels i, i + R/2
        const bool low = c0 < R / 2;
        const int b = low ? c0 : c0 - R / 2;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          cs[i] = row[b + i];
          const float s = row[R / 2 + b + i];
          sn[i] = low ? -s : s;
        }
      }
    }
  }
  // lane of the other half of a pair (halves); a row's rotated lanes are 0 .. R/8-1
  const int mate = turn ? (lane - li) + (c0 < R / 2 ? li + R / 16 : li - R / 16) : lane;
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    wq[i] = A.wq ? A.wq[c0 + i] : 1.0f;
    wk[i] = A.wk ? A.wk[c0 + i] : 1.0f;
  }
  for (int h0 = wave * RPW; h0 < rows; h0 += 4 * RPW) {
    const int h = h0 + lane / LPR;
    const bool on = h < rows, isq = h < A.hq;
    float x[8];
    if (on) {
      if (isq) load8<IN>(A.q, t * A.qs + (int64_t)h * D + c0, x);
      else load8<IN>(A.k, t * A.ks + (int64_t)(h - A.hq) * D + c0, x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) x[i] = 0.0f;
    }
    if (A.norm != STQ_NORM_NONE) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i++) s = __builtin_fmaf(x[i], x[i], s);
      s = row_sum<LPR>(s);
      if (A.norm == STQ_NORM_RMS) s *= 1.0f / D;
      const float f = 1.0f / __builtin_sqrtf(s + A.eps);
#pragma unroll
      for (int i = 0; i < 8; i++) x[i] *= f;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] *= isq ? wq[i] : wk[i];
    if (R > 0) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = A.adjacent ? x[i ^ 1] : __shfl(x[i], mate, 64);
      if (turn) {
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = __builtin_fmaf(x[i], cs[i], y[i] * sn[i]);
      }
    }
    if (on) {
      if (isq) store8<OUT>(A.qo, t * A.qos + (int64_t)h * D + c0, x);
      else store8<OUT>(A.ko, t * A.kos + (int64_t)(h - A.hq) * D + c0, x);
    }
  }
}

// ------------------------------------------------------- key/value cache
struct StoreArgs {
  uint8_t* cache;
  const int64_t* slot;
  const void *k, *v;
  void *ko, *vo;
  int n_tok, heads, T;
  int64_t n_slots, ks, vs;
};

// Exponent of a 32-channel block's scale: least e with m <= 6 * 2^e (finite m
// > 0), i.e. with m = f * 2^x, f in [1, 2): x - 2 for f <= 1.5, else x - 1.
__device__ __forceinline__ int scale_exp(float m) {
  const uint32_t u = __float_as_uint(m);
  const int x = (int)(u >> 23) - 127;                  // (a subnormal m gives -127: held at E_MIN)
  const int e = (u & 0x7FFFFFu) > 0x400000u ? x - 1 : x - 2;
  return m == 0.0f ? 0 : min(max(e, E_MIN), E_MAX);
}
// Code of |y| (already divided by the scale) with y's sign: nearest of
// 0 .5 1 1.5 2 3 4 6, ties to the even code.
__device__ __forceinline__ uint32_t code_of(float y) {
  const float a = __builtin_fabsf(y);
  uint32_t c = (uint32_t)(a > 0.25f) + (uint32_t)(a >= 0.75f) + (uint32_t)(a > 1.25f) + (uint32_t)(a >= 1.75f) +
               (uint32_t)(a > 2.5f) + (uint32_t)(a >= 3.5f) + (uint32_t)(a > 5.0f);
  return c | ((c != 0 && y < 0.0f) ? 8u : 0u);
}
// eight channels as one dword of codes; the block's largest magnitude over its four lanes
__device__ __forceinline__ uint32_t codes8(const float* x, int* e_out) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) m = __builtin_fmaxf(m, __builtin_fabsf(x[i]));
  m = rb_max_pos<4>(m);
  const int e = scale_exp(m);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) w |= code_of(__builtin_ldexpf(x[i], -e)) << (4 * i);
  *e_out = e;
  return w;
}

// One (token, head) on D/8 lanes, keys and values together (the NaN rule needs both).
template <int D, int TYPE>
__global__ void __launch_bounds__(256) k_kv_store(StoreArgs A) {
  constexpr int LPR = D / 8, RPB = 256 / LPR;
  const int li = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  const int64_t t = row / A.heads;
  const int h = (int)(row - t * A.heads);
  const bool on = t < A.n_tok;
  const int64_t slot = on ? A.slot[t] : -1;
  const bool live = slot >= 0 && slot < A.n_slots;
  float k[8], v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) k[i] = v[i] = 0.0f;
  if (live) {
    load8<TYPE>(A.k, t * A.ks + (int64_t)h * D + 8 * li, k);
    load8<TYPE>(A.v, t * A.vs + (int64_t)h * D + 8 * li, v);
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; i++) bad |= !(__builtin_fabsf(k[i]) < __builtin_inff()) || !(__builtin_fabsf(v[i]) < __builtin_inff());
  const uint64_t any = __ballot(bad);
  const int l0 = (threadIdx.x & 63) - li;
  const bool poison = ((any >> l0) & ((1ull << LPR) - 1)) != 0;
  if (poison) {
#pragma unroll
    for (int i = 0; i < 8; i++) k[i] = v[i] = 0.0f;
  }
  int ek, ev;
  const uint32_t ck = codes8(k, &ek), cv = codes8(v, &ev);
  if (!live) return;
  const int T = A.T, off = (int)(slot % T);
  uint8_t* hb = A.cache + ((slot / T) * A.heads + h) * ((int64_t)T * D * 17 / 16);
  *(uint32_t*)(hb + off * (D / 2) + 4 * li) = ck;
  *(uint32_t*)(hb + T * (D / 2) + off * (D / 2) + 4 * li) = cv;
  if ((li & 3) == 0) {
    uint8_t* sc = hb + T * D + (li >> 2) * T + off;
    sc[0] = poison ? 255 : (uint8_t)(ek + 127);
    sc[T * (D / 32)] = (uint8_t)(ev + 127);
  }
}

// eight codes of a dword as binary32 values
__device__ __forceinline__ void values8(uint32_t w, uint32_t sbyte, float* x) {
  const float sc = sbyte == 255 ? __builtin_nanf("") : bits_f(sbyte << 23);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t c = (w >> (4 * i)) & 7u;
    // magnitude: exponent bits c >> 1, mantissa bit c & 1; below 2 the codes are 0 and 0.5
    const float m = c < 2 ? 0.5f * c : bits_f(((126u + (c >> 1)) << 23) | ((c & 1u) << 22));
    x[i] = (((w >> (4 * i)) & 8u) ? -m : m) * sc;
  }
}

template <int D, int TYPE>
__global__ void __launch_bounds__(256) k_kv_fetch(StoreArgs A) {
  constexpr int LPR = D / 8, RPB = 256 / LPR;
  const int li = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  const int64_t t = row / A.heads;
  const int h = (int)(row - t * A.heads);
  if (t >= A.n_tok) return;
  const int64_t slot = A.slot[t];
  if (slot < 0 || slot >= A.n_slots) return;
  const int T = A.T, off = (int)(slot % T);
  const uint8_t* hb = A.cache + ((slot / T) * A.heads + h) * ((int64_t)T * D * 17 / 16);
  const uint32_t ck = *(const uint32_t*)(hb + off * (D / 2) + 4 * li);
  const uint32_t cv = *(const uint32_t*)(hb + T * (D / 2) + off * (D / 2) + 4 * li);
  const uint8_t* sc = hb + T * D + (li >> 2) * T + off;
  float x[8];
  values8(ck, sc[0], x);
  store8<TYPE>(A.ko, row * D + 8 * li, x);
  values8(cv, sc[T * (D / 32)], x);
  store8<TYPE>(A.vo, row * D + 8 * li, x);
}

// ------------------------------------------------------------- attention
struct AttnArgs {
  const uint8_t* cache;
  const int32_t *table, *tok_start, *len;
  const void* q;
  void* o;
  float *po, *pml;          // partial results: [split][row][D], [split][row][2]
  int n_req, n_tok, hq, hkv, group, T, n_blocks, cols, max_new, window, sink, splits, tiles;
  int64_t qs, os;
  float scale_log2;
};

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
// Chunks of one split: the work is cut into `splits` equal parts, but not
// below SPLIT_MIN chunks; a part holds a multiple of four (one per wave).
constexpr int SPLIT_MIN = 8;
__device__ __forceinline__ int split_chunks(int total, int splits) {
  return max((((total + splits - 1) / splits) + 3) & ~3, SPLIT_MIN);
}
struct Req { int first, n_new, len, base; };   // first row, query tokens, cached tokens, position of query 0
__device__ __forceinline__ Req req_args(const AttnArgs& A, int i) {
  Req r;
  r.first = min(max(ld_const(A.tok_start + i), 0), A.n_tok);
  const int end = min(max(ld_const(A.tok_start + i + 1), r.first), A.n_tok);
  r.n_new = end - r.first;
  r.len = (int)min((int64_t)max(ld_const(A.len + i), 0), (int64_t)A.cols * A.T);
  r.base = r.len - r.n_new;
  return r;
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

constexpr float NEG_INF = -__builtin_inff();

// Power of two that brings a row's largest magnitude m into [2^14, 2^15), and
// the factor that turns products of such rows into base-2 logits.
__device__ __forceinline__ int q_shift(float m) {
  return m > 0.0f && m < __builtin_inff() ? 15 - __builtin_amdgcn_frexp_expf(m) : 0;
}
__device__ __forceinline__ float q_factor(float scale_log2, int e) {
  return __builtin_fmaxf(__builtin_ldexpf(__builtin_fabsf(scale_log2), -e), 1.17549435e-38f);
}

// A wave's query rows as matrix operands: row n = lane % 16 of tile nt, the
// channels (D/4) G .. + D/4 of lane group G = lane / 16, in binary16 scaled by
// a power of two that puts the row's largest magnitude in [2^14, 2^15) (exact
// for bf16 and fp16 queries down to 2^-29 of that magnitude).  c: the factor
// from scaled products to base-2 logits, kept positive (a negative scale
// turns the queries' signs) and normal.
template <int D, int TYPE>
__device__ __forceinline__ void load_q(const AttnArgs& A, bool on, int64_t at, f16x8* q, float* c) {
  float x[D / 4];
#pragma unroll
  for (int i = 0; i < D / 32; i++) {
    if (on) load8<TYPE>(A.q, at + 8 * i, x + 8 * i);
    else
#pragma unroll
      for (int j = 0; j < 8; j++) x[8 * i + j] = 0.0f;
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 4; i++) m = __builtin_fmaxf(m, __builtin_fabsf(x[i]));
  m = max_quads(m);
  const int e = q_shift(m);
  const float sign = A.scale_log2 < 0.0f ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < D / 32; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) q[i][j] = (f16)(sign * __builtin_ldexpf(x[8 * i + j], e));
  *c = q_factor(A.scale_log2, e);
}

// One chunk (32 cached tokens of one head) as a wave loads it.  Token 8G' + i
// (i < 4) is row 4G' + i of key tile 0, token 8G' + 4 + i that row of tile 1:
// the two tiles' products then leave lane group G with the eight tokens
// 8G .. 8G+7 of its query row, which is the operand that the product with
// the values wants.  Keys: lane (m, G) holds the channels (D/4) G .. of row m.
// Values: lane (m, G) holds the channels (D/16) m .. of tokens 8G .. 8G+7.
template <int D>
struct Chunk {
  static constexpr int KD = D / 32;                    // dwords of keys per tile and lane
  static constexpr int KS = D > 128 ? 2 : 1;           // key scales per tile and lane
  uint32_t k[2][KD], v[8];
  uint32_t ks[2];
  uint32_t vs[2];
  bool dead;                                           // its block's table entry is no block
};

template <int D>
__device__ __forceinline__ void load_chunk(const AttnArgs& A, Chunk<D>& C, int blk, int h, int chunk) {
  const int lane = threadIdx.x & 63, m = lane & 15, G = lane >> 4;
  const int T = A.T, off = (chunk * 32) & (T - 1);
  C.dead = (uint32_t)blk >= (uint32_t)A.n_blocks;
  const uint8_t* hb = A.cache + ((int64_t)(C.dead ? 0 : blk) * A.hkv + h) * (T * D / 16 * 17);
  const uint8_t* kc = hb + off * (D / 2);
  const uint8_t* vc = kc + T * (D / 2);
  const uint8_t* ksc = hb + T * D + off;
  const uint8_t* vsc = ksc + T * (D / 32);
  const int r = 8 * (m >> 2) + (m & 3);
#pragma unroll
  for (int u = 0; u < 2; u++) {
    const uint8_t* p = kc + (r + 4 * u) * (D / 2) + G * (D / 8);
    if constexpr (D == 128) {
      const u32x4 w = *(const u32x4*)p;
#pragma unroll
      for (int i = 0; i < 4; i++) C.k[u][i] = w[i];
    } else {
      const u32x2 w = *(const u32x2*)p;
      C.k[u][0] = w[0];
      C.k[u][1] = w[1];
    }
    C.ks[u] = ksc[(G * (D / 4) / 32) * T + r + 4 * u];
  }
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const uint8_t* p = vc + (8 * G + j) * (D / 2) + m * (D / 32);
    if constexpr (D == 128) C.v[j] = *(const uint32_t*)p;
    else C.v[j] = *(const uint16_t*)p;
  }
  const u32x2 s = *(const u32x2*)(vsc + (m * (D / 16) / 32) * T + 8 * G);
  C.vs[0] = s[0];
  C.vs[1] = s[1];
}

// Scale byte j of a dword where v_cvt_scalef32_* takes a scale: in the
// exponent field of a binary32 (the conversion reads nothing else of it, and
// gives NaN for the byte 255).
template <int J>
__device__ __forceinline__ float scale_of(uint32_t w) {
  return bits_f(J < 3 ? w << (23 - 8 * J) : w >> 1);
}
template <int J>
__device__ __forceinline__ uint32_t cvt2(uint32_t w, float s) {   // codes 2J, 2J+1 of w as a binary16 pair
  return h2_bits(__builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, J)));
}
__device__ __forceinline__ f16x8 frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(f16x8, (u32x4){a, b, c, d});
}

// Running softmax of a wave's 16-row tiles: o is the transposed product, tile
// c element i = channel (D/16)(4G + i) + c of query row n = lane % 16.
template <int D, int NT>
struct Acc {
  f32x4 o[NT][D / 16];
  float m[NT], l[NT];      // largest scaled product (all lane groups alike), this lane group's part of the sum
};

template <int D, int NT, bool MASK>
__device__ __forceinline__ void chunk_step(const AttnArgs& A, const Chunk<D>& C, const f16x8 (*q)[D / 32], const float* c,
                                           const int* p, int chunk, Acc<D, NT>& S) {
  const int G = (threadIdx.x & 63) >> 4;
  f32x4 s[NT][2];
#pragma unroll
  for (int u = 0; u < 2; u++) {
    const float sc = scale_of<0>(C.ks[u]);
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
  f16x8 P[NT];
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    if (MASK) {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int t = chunk * 32 + 8 * G + e;
        const bool see = t <= p[nt] && (A.window == 0 || t > p[nt] - A.window || t < A.sink) && !C.dead;
        s[nt][e >> 2][e & 3] = see ? s[nt][e >> 2][e & 3] : NEG_INF;
      }
    }
    float m = s[nt][0][0];
#pragma unroll
    for (int e = 1; e < 8; e++) m = __builtin_fmaxf(m, s[nt][e >> 2][e & 3]);
    m = __builtin_fmaxf(S.m[nt], max_quads(m));
    // nothing seen so far: any finite reference will do, every weight is 2^-inf
    const float mc = m == NEG_INF ? 0.0f : m * c[nt];
    if (__any(m > S.m[nt])) {
      const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(S.m[nt], c[nt], -mc));
      S.l[nt] *= f;
#pragma unroll
      for (int i = 0; i < D / 16; i++) S.o[nt][i] *= f;
      S.m[nt] = m;
    }
    // Weights to binary16 in pairs; the sum takes the same rounded weights, so
    // that a weight's rounding moves o by its own part only.
    uint32_t pk[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nt][e >> 1][2 * (e & 1)], c[nt], -mc));
      const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[nt][e >> 1][2 * (e & 1) + 1], c[nt], -mc));
      const f16x2 h = {(f16)a, (f16)b};
      pk[e] = h2_bits(h);
      S.l[nt] = __builtin_amdgcn_fdot2(h, (f16x2){(f16)1.0f, (f16)1.0f}, S.l[nt], false);
    }
    P[nt] = frag(pk[0], pk[1], pk[2], pk[3]);
  }
  // Values: pairs of tokens of one channel, from pairs of channels of one token.
  float vs[8];
  vs[0] = scale_of<0>(C.vs[0]); vs[1] = scale_of<1>(C.vs[0]); vs[2] = scale_of<2>(C.vs[0]); vs[3] = scale_of<3>(C.vs[0]);
  vs[4] = scale_of<0>(C.vs[1]); vs[5] = scale_of<1>(C.vs[1]); vs[6] = scale_of<2>(C.vs[1]); vs[7] = scale_of<3>(C.vs[1]);
  if (MASK) {     // unwritten bytes behind the last token: any finite value, their weights are 0
#pragma unroll
    for (int j = 0; j < 8; j++) vs[j] = bits_f(min(__float_as_uint(vs[j]) & 0x7F800000u, (uint32_t)(E_MAX + 127) << 23));
  }
  constexpr int NB = D / 32;                            // bytes of one token and lane
#pragma unroll
  for (int b = 0; b < NB; b++) {
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
      S.o[nt][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fl, P[nt], S.o[nt][2 * b], 0, 0, 0);
      S.o[nt][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fh, P[nt], S.o[nt][2 * b + 1], 0, 0, 0);
    }
  }
}

// Few query rows per key/value head (a token's head group, drafted tokens):
// the cache's bytes bound the work, so nothing is staged.  One workgroup =
// one (request, head, tile of 16 NT rows, split of the cache); its four
// waves take every fourth chunk straight from memory into the operands'
// registers and join their running softmaxes through LDS at the end.
template <int D, int TYPE, int NT>
__global__ void __launch_bounds__(256) k_attend_rows(AttnArgs A) {
  constexpr int NC = D / 16;
  __shared__ f32x4 so[2][NT * NC][64];
  __shared__ float sml[4][NT][16][2];
  const int lane = threadIdx.x & 63, n = lane & 15, G = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  int b = blockIdx.x;
  const int sp = b % A.splits; b /= A.splits;
  const int tile = b % A.tiles; b /= A.tiles;
  const int h = b % A.hkv, i = b / A.hkv;
  const Req R = req_args(A, i);
  const int row0 = tile * 16 * NT, rows = min(R.n_new, A.max_new) * A.group;
  if (row0 >= rows) return;
  const int j1 = (min(row0 + 16 * NT, rows) - 1) / A.group;
  const int p0 = R.base + row0 / A.group, p1 = R.base + j1;
  const Span sn = span_of(p0, p1, A.window, A.sink);
  const int per = split_chunks(sn.total, A.splits);
  const int c0 = sp * per, c1 = min(c0 + per, sn.total);
  if (c0 >= c1 && sp > 0) return;
  const int parts = (sn.total + per - 1) / per;

  f16x8 q[NT][D / 32];
  float cf[NT];
  int pos[NT];
  int64_t grow[NT];            // row of q and o as (token, head) index, -1 outside
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    const int r = row0 + 16 * nt + n, j = r / A.group, g = r - j * A.group;
    const bool on = r < rows;
    grow[nt] = on ? (int64_t)(R.first + j) * A.hq + h * A.group + g : -1;
    pos[nt] = on ? R.base + j : p1;
    load_q<D, TYPE>(A, on, (int64_t)(R.first + j) * A.qs + (int64_t)(h * A.group + g) * D + G * (D / 4), q[nt], &cf[nt]);
  }
  Acc<D, NT> S;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    S.m[nt] = NEG_INF;
    S.l[nt] = 0.0f;
#pragma unroll
    for (int k = 0; k < NC; k++) S.o[nt][k] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int32_t* tab = A.table + (int64_t)i * A.cols;
  const int per_blk = A.T >> 5;
  auto chunk_at = [&](int k) { return k < sn.n_low ? k : sn.lo + k - sn.n_low; };
  Chunk<D> C[2];
  int k = c0 + wave;
  if (k < c1) load_chunk<D>(A, C[0], ld_const(tab + chunk_at(k) / per_blk), h, chunk_at(k));
  auto one = [&](const Chunk<D>& X, int kk) {
    const int ch = chunk_at(kk), t0 = ch * 32, t1 = t0 + 31;
    const bool full = !X.dead && t1 <= p0 && (A.window == 0 || t0 > p1 - A.window || t1 < A.sink);
    if (full) chunk_step<D, NT, false>(A, X, q, cf, pos, ch, S);
    else chunk_step<D, NT, true>(A, X, q, cf, pos, ch, S);
  };
  while (k < c1) {
    if (k + 4 < c1) load_chunk<D>(A, C[1], ld_const(tab + chunk_at(k + 4) / per_blk), h, chunk_at(k + 4));
    one(C[0], k);
    if (k + 4 >= c1) break;
    if (k + 8 < c1) load_chunk<D>(A, C[0], ld_const(tab + chunk_at(k + 8) / per_blk), h, chunk_at(k + 8));
    one(C[1], k + 4);
    k += 8;
  }
  // Join the waves: each row's largest product, every wave rescaled to it, then
  // 2 -> 0 and 3 -> 1, 1 -> 0 (a fixed order).
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    S.l[nt] = sum_quads(S.l[nt]);
    if (G == 0) { sml[wave][nt][n][0] = S.m[nt]; sml[wave][nt][n][1] = S.l[nt]; }
  }
  __syncthreads();
  float M[NT], L[NT];
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    M[nt] = NEG_INF;
#pragma unroll
    for (int w = 0; w < 4; w++) M[nt] = __builtin_fmaxf(M[nt], sml[w][nt][n][0]);
    const float mc = M[nt] == NEG_INF ? 0.0f : M[nt] * cf[nt];
    L[nt] = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; w++) L[nt] += sml[w][nt][n][1] * __builtin_amdgcn_exp2f(__builtin_fmaf(sml[w][nt][n][0], cf[nt], -mc));
    const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(S.m[nt], cf[nt], -mc));
#pragma unroll
    for (int c = 0; c < NC; c++) S.o[nt][c] *= f;
  }
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    if (wave >= step && wave < 2 * step) {
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int c = 0; c < NC; c++) so[wave - step][nt * NC + c][lane] = S.o[nt][c];
    }
    __syncthreads();
    if (wave < step) {
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int c = 0; c < NC; c++) S.o[nt][c] += so[wave][nt * NC + c][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    if (grow[nt] < 0) continue;
    // this lane's channels: (D/16)(4G + i) + c, consecutive
    if (parts <= 1) {
      const float inv = L[nt] == 0.0f ? 0.0f : 1.0f / L[nt];
      const int64_t t = grow[nt] / A.hq, hd = grow[nt] - t * A.hq;
      const int64_t at = t * A.os + hd * D + G * (D / 4);
#pragma unroll
      for (int e = 0; e < D / 32; e++) {
        float x[8];
#pragma unroll
        for (int u = 0; u < 8; u++) x[u] = S.o[nt][(8 * e + u) % NC][(8 * e + u) / NC] * inv;
        store8<TYPE>(A.o, at + 8 * e, x);
      }
    } else {
      const int64_t row = (int64_t)sp * A.n_tok * A.hq + grow[nt];
      if (G == 0) {
        A.pml[2 * row] = M[nt] == NEG_INF ? NEG_INF : M[nt] * cf[nt];
        A.pml[2 * row + 1] = L[nt];
      }
#pragma unroll
      for (int e = 0; e < D / 32; e++) {
        float x[8];
#pragma unroll
        for (int u = 0; u < 8; u++) x[u] = S.o[nt][(8 * e + u) % NC][(8 * e + u) / NC];
        store8<STQ_FP32>(A.po, row * D + G * (D / 4) + 8 * e, x);
      }
    }
  }
}

// Many query rows per key/value head (prompts): the matrix products bound the
// work.  One workgroup = one (request, head, tile of 32 NW rows, split), each
// wave 32 rows.  Tiles of 64 cached tokens (two chunks) go through LDS as
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
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __fp16 fp16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) fp16x4 lds_fp16x4;

// 16-byte slot of (token t of 64, channels 8c ..): rows rotated so that the 16
// lanes of a read or write phase touch 16 different slots of the banks.
template <int D>
__device__ __forceinline__ int k_slot(int t, int c) {
  if constexpr (D == 128) return t * 16 + ((c + t) & 15);
  else return t * 8 + ((c + (t >> 1)) & 7);
}
template <int D>
__device__ __forceinline__ int v_slot(int t, int c) {
  if constexpr (D == 128) return t * 16 + ((c + 4 * (t & 3) + ((t >> 2) & 3)) & 15);
  else return t * 8 + ((c + 4 * ((t >> 1) & 1) + ((t >> 2) & 3)) & 7);
}

__device__ __forceinline__ float max_halves(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_fmaxf(bits_f(a[0]), bits_f(a[1]));
}

template <int D, int TYPE, int NW>
__global__ void __launch_bounds__(64 * NW, 2) k_attend_tiles(AttnArgs A) {
  constexpr int NT = 64 * NW, ROWS = 32 * NW;
  constexpr int KP = 2 * D;                            // 16-byte pieces of a tile's key codes (32 channels of a token)
  constexpr int NP = (2 * KP + NT - 1) / NT;           // pieces of keys and values per thread
  constexpr int KSTEP = D / 16, NC = D / 32;
  __shared__ u32x4 sk[2][64 * D / 8], sv[2][64 * D / 8];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, G = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // (request, head) pairs fastest, the tiles with the most to see first: a pair's
  // workgroups share an XCD where the pairs are a multiple of 8
  int b = blockIdx.x;
  const int pairs = A.n_req * A.hkv, pair = b % pairs; b /= pairs;
  const int sp = b % A.splits, tile = A.tiles - 1 - b / A.splits;
  const int h = pair % A.hkv, i = pair / A.hkv;
  const Req R = req_args(A, i);
  const int row0 = tile * ROWS, rows = min(R.n_new, A.max_new) * A.group;
  if (row0 >= rows) return;
  const int p0 = R.base + row0 / A.group, p1 = R.base + (min(row0 + ROWS, rows) - 1) / A.group;
  const Span sn = span_of(p0, p1, A.window, A.sink);
  const int per = split_chunks(sn.total, A.splits);
  const int c0 = sp * per, c1 = min(c0 + per, sn.total);
  if (c0 >= c1 && sp > 0) return;
  const int parts = (sn.total + per - 1) / per;

  // the wave's rows
  const int r = row0 + 32 * wave + n, j = r / A.group, g = r - j * A.group;
  const bool on = r < rows;
  const int pw1 = R.base + (min(row0 + 32 * wave + 32, rows) - 1) / A.group;
  const int pw0 = min(R.base + (row0 + 32 * wave) / A.group, pw1), pos = on ? R.base + j : pw1;
  f16x8 q[KSTEP];
  float cf;
  {
    float x[D / 2];
    const int64_t at = (int64_t)(R.first + j) * A.qs + (int64_t)(h * A.group + g) * D + 8 * G;
#pragma unroll
    for (int s = 0; s < KSTEP; s++) {
      if (on) load8<TYPE>(A.q, at + 16 * s, x + 8 * s);
      else
#pragma unroll
        for (int u = 0; u < 8; u++) x[8 * s + u] = 0.0f;
    }
    float m = 0.0f;
#pragma unroll
    for (int u = 0; u < D / 2; u++) m = __builtin_fmaxf(m, __builtin_fabsf(x[u]));
    m = max_halves(m);
    const int e = q_shift(m);
    const float sign = A.scale_log2 < 0.0f ? -1.0f : 1.0f;
#pragma unroll
    for (int s = 0; s < KSTEP; s++)
#pragma unroll
      for (int u = 0; u < 8; u++) q[s][u] = (f16)(sign * __builtin_ldexpf(x[8 * s + u], e));
    cf = q_factor(A.scale_log2, e);
  }
  f32x16 o[NC];
#pragma unroll
  for (int c = 0; c < NC; c++)
#pragma unroll
    for (int u = 0; u < 16; u++) o[c][u] = 0.0f;
  float M = NEG_INF, L = 0.0f;

  const int32_t* tab = A.table + (int64_t)i * A.cols;
  const int per_blk = A.T >> 5, T = A.T;
  auto chunk_at = [&](int k) { return k < sn.n_low ? k : sn.lo + k - sn.n_low; };
  u32x4 raw[NP];
  uint32_t sb[NP];
  // this thread's pieces of chunks k, k + 1
  auto fetch = [&](int k) {
#pragma unroll
    for (int s = 0; s < NP; s++) {
      const int p = tid + s * NT;
      if (2 * KP % NT && p >= 2 * KP) break;
      const bool isv = p >= KP;
      const int pp = isv ? p - KP : p;
      const int u = pp / D, w = pp % D;                  // chunk, piece of it: D pieces
      // keys: pieces of a token side by side; values: tokens side by side (the bank layouts of the writes)
      const int t = isv ? w & 31 : w / (D / 32), c = isv ? w >> 5 : w % (D / 32);
      const int ch = chunk_at(min(k + u, c1 - 1));
      int blk = ld_const(tab + ch / per_blk);
      blk = (uint32_t)blk < (uint32_t)A.n_blocks ? blk : 0;
      const int off = ((ch * 32) & (T - 1)) + t;
      const uint8_t* hb = A.cache + ((int64_t)blk * A.hkv + h) * (T * D / 16 * 17);
      raw[s] = *(const u32x4*)(hb + (isv ? T * (D / 2) : 0) + off * (D / 2) + 16 * c);
      sb[s] = hb[T * D + (isv ? T * (D / 32) : 0) + c * T + off];
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int s = 0; s < NP; s++) {
      const int p = tid + s * NT;
      if (2 * KP % NT && p >= 2 * KP) break;
      const bool isv = p >= KP;
      const int pp = isv ? p - KP : p;
      const int u = pp / D, w = pp % D;
      const int t = 32 * u + (isv ? w & 31 : w / (D / 32)), c = 4 * (isv ? w >> 5 : w % (D / 32));
      // values: unwritten bytes behind the last token must not be NaN or infinite, their weights are 0
      const float sc = scale_of<0>(isv ? min(sb[s], (uint32_t)(E_MAX + 127)) : sb[s]);
#pragma unroll
      for (int x = 0; x < 4; x++) {
        const uint32_t d = raw[s][x];
        const u32x4 v = {cvt2<0>(d, sc), cvt2<1>(d, sc), cvt2<2>(d, sc), cvt2<3>(d, sc)};
        if (isv) sv[buf][v_slot<D>(t, c + x)] = v;
        else sk[buf][k_slot<D>(t, c + x)] = v;
      }
    }
  };
  auto block_of = [&](int k) { return ld_const(tab + chunk_at(k) / per_blk); };
  // rows that see all of chunk k
  auto whole = [&](int k) {
    if (k >= c1 || (uint32_t)block_of(k) >= (uint32_t)A.n_blocks) return false;
    const int t0 = chunk_at(k) * 32, t1 = t0 + 31;
    return t1 <= pw0 && (A.window == 0 || t0 > pw1 - A.window || t1 < A.sink);
  };
  if (c0 < c1) {
    fetch(c0);
    put(0);
    if (c0 + 2 < c1) fetch(c0 + 2);
    __syncthreads();
    int buf = 0;
    for (int k = c0; k < c1; k += 2, buf ^= 1) {
      if (k + 2 < c1) {
        put(buf ^ 1);
        if (k + 4 < c1) fetch(k + 4);
      }
      if (chunk_at(k) * 32 <= pw1) {                    // else every token lies behind the wave's rows
        f32x16 s[2];
#pragma unroll
        for (int u = 0; u < 2; u++) {
#pragma unroll
          for (int x = 0; x < 16; x++) s[u][x] = 0.0f;
#pragma unroll
          for (int x = 0; x < KSTEP; x++) {
            const f16x8 kf = __builtin_bit_cast(f16x8, sk[buf][k_slot<D>(32 * u + n, 2 * x + G)]);
            s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, q[x], s[u], 0, 0, 0);
          }
        }
        if (!(whole(k) && whole(k + 1))) {
#pragma unroll
          for (int u = 0; u < 2; u++) {
            const bool there = k + u < c1 && (uint32_t)block_of(min(k + u, c1 - 1)) < (uint32_t)A.n_blocks;
            const int t0 = chunk_at(min(k + u, c1 - 1)) * 32 + 4 * G;
#pragma unroll
            for (int x = 0; x < 16; x++) {
              const int t = t0 + 8 * (x >> 2) + (x & 3);
              const bool see = t <= pos && (A.window == 0 || t > pos - A.window || t < A.sink) && there;
              s[u][x] = see ? s[u][x] : NEG_INF;
            }
          }
        }
        float m = s[0][0];
#pragma unroll
        for (int x = 1; x < 32; x++) m = __builtin_fmaxf(m, s[x >> 4][x & 15]);
        m = __builtin_fmaxf(M, max_halves(m));
        const float mc = m == NEG_INF ? 0.0f : m * cf;
        if (__any(m > M)) {
          const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(M, cf, -mc));
          L *= f;
#pragma unroll
          for (int c = 0; c < NC; c++)
#pragma unroll
            for (int x = 0; x < 16; x++) o[c][x] *= f;
          M = m;
        }
#pragma unroll
        for (int u = 0; u < 2; u++) {
#pragma unroll
          for (int y = 0; y < 2; y++) {                 // 16 tokens
            uint32_t pk[4];
#pragma unroll
            for (int x = 0; x < 4; x++) {
              const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][8 * y + 2 * x], cf, -mc));
              const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][8 * y + 2 * x + 1], cf, -mc));
              const f16x2 hh = {(f16)e0, (f16)e1};
              pk[x] = h2_bits(hh);
              L = __builtin_amdgcn_fdot2(hh, (f16x2){(f16)1.0f, (f16)1.0f}, L, false);
            }
            const f16x8 P = frag(pk[0], pk[1], pk[2], pk[3]);
#pragma unroll
            for (int c = 0; c < NC; c++) {
              const int t = 32 * u + 16 * y + 4 * G + ((lane >> 2) & 3);
              const int cb = 32 * c + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);   // channels cb .. cb + 3
              u32x4* base = sv[buf];
              const fp16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4f16(
                  (lds_fp16x4*)((uint8_t*)(base + v_slot<D>(t, cb >> 3)) + 8 * ((cb >> 2) & 1)));
              const fp16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4f16(
                  (lds_fp16x4*)((uint8_t*)(base + v_slot<D>(t + 8, cb >> 3)) + 8 * ((cb >> 2) & 1)));
              const u32x2 a = __builtin_bit_cast(u32x2, lo), d = __builtin_bit_cast(u32x2, hi);
              o[c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(frag(a[0], a[1], d[0], d[1]), P, o[c], 0, 0, 0);
            }
          }
        }
      }
      __syncthreads();
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
      A.pml[2 * row] = M == NEG_INF ? NEG_INF : M * cf;
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
template <int D, int TYPE>
__global__ void __launch_bounds__(256) k_attend_join(AttnArgs A, int tile_rows) {
  const int lane = threadIdx.x & 63;
  int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int hd = (int)(b % A.hq); b /= A.hq;
  const int j = (int)(b % A.max_new), i = (int)(b / A.max_new);
  if (i >= A.n_req) return;
  const Req R = req_args(A, i);
  if (j >= R.n_new) return;
  const int row0 = (j * A.group + hd % A.group) / tile_rows * tile_rows, rows = min(R.n_new, A.max_new) * A.group;
  const int j1 = (min(row0 + tile_rows, rows) - 1) / A.group;
  const Span sn = span_of(R.base + row0 / A.group, R.base + j1, A.window, A.sink);
  const int per = split_chunks(sn.total, A.splits), parts = (sn.total + per - 1) / per;
  if (parts <= 1) return;                              // written by its only part
  const int64_t stride = (int64_t)A.n_tok * A.hq, row = (int64_t)(R.first + j) * A.hq + hd;
  float M = NEG_INF;
  for (int s = 0; s < parts; s++) M = __builtin_fmaxf(M, A.pml[2 * (s * stride + row)]);
  if (M == NEG_INF) M = 0.0f;
  float L = 0.0f, x[D / 64];
#pragma unroll
  for (int u = 0; u < D / 64; u++) x[u] = 0.0f;
  for (int s = 0; s < parts; s++) {
    const int64_t at = s * stride + row;
    const float f = __builtin_amdgcn_exp2f(A.pml[2 * at] - M);
    L = __builtin_fmaf(f, A.pml[2 * at + 1], L);
#pragma unroll
    for (int u = 0; u < D / 64; u++) x[u] = __builtin_fmaf(f, A.po[at * D + lane * (D / 64) + u], x[u]);
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
bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }
int elem_bytes(int type) { return type == STQ_FP32 ? 4 : 2; }
bool stride_ok(int64_t stride, int64_t least, int type) {
  return stride >= least && stride < (1ll << 40) && (stride * elem_bytes(type)) % 16 == 0;
}
stq_status launched() { return hipGetLastError() == hipSuccess ? STQ_OK : STQ_ERR_HIP; }

bool attend_ok(const stq_kv_desc* d, const stq_attend_desc* a) {
  return a && a->n_req >= 0 && a->n_tok >= 0 && a->n_heads >= 1 && a->n_heads % d->n_kv_heads == 0 &&
         a->n_heads <= 65536 && (a->type == STQ_BF16 || a->type == STQ_FP16) && a->table_cols >= 1 &&
         (int64_t)a->table_cols * d->block_tokens <= (1ll << 30) && a->max_new >= 1 && a->max_len >= 1 &&
         a->window >= 0 && a->n_sink >= 0 && isfinite(a->scale);
}
struct Split { int tiles, tile_rows, splits; bool staged; };
// Query rows per key/value head from which the cache is staged through LDS.
constexpr int STAGED_ROWS = 64;
constexpr int TILE_WAVES = 4;
// Workgroups wanted in all: enough for every CU to hold several and for ragged lengths to even out.
constexpr int64_t WANT_GROUPS = 1536;
Split split_of(const stq_kv_desc* d, const stq_attend_desc* a) {
  Split s;
  const int64_t rows = (int64_t)a->max_new * (a->n_heads / d->n_kv_heads);
  s.staged = rows > STAGED_ROWS;
  s.tile_rows = s.staged ? 32 * TILE_WAVES : 16;
  s.tiles = (int)((rows + s.tile_rows - 1) / s.tile_rows);
  const int64_t base = (int64_t)a->n_req * d->n_kv_heads * s.tiles;
  int64_t seen = a->max_len;
  if (a->window > 0) seen = seen < (int64_t)a->window + a->n_sink + 64 ? seen : (int64_t)a->window + a->n_sink + 64;
  const int64_t chunks = (seen + 31) / 32;
  int64_t k = base > 0 ? WANT_GROUPS / base : 1;
  const int64_t most = chunks / SPLIT_MIN;
  if (k > most) k = most;
  if (k > 64) k = 64;
  s.splits = k < 1 ? 1 : (int)k;
  return s;
}

template <int D, int TYPE>
void launch_attend(AttnArgs& A, const Split& s, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)A.n_req * A.hkv * A.tiles * A.splits);
  if (s.staged) hipLaunchKernelGGL((k_attend_tiles<D, TYPE, TILE_WAVES>), dim3(grid), dim3(64 * TILE_WAVES), 0, st, A);
  else hipLaunchKernelGGL((k_attend_rows<D, TYPE, 1>), dim3(grid), dim3(256), 0, st, A);
  if (A.splits > 1) {
    const int64_t rows = (int64_t)A.n_req * A.max_new * A.hq;
    hipLaunchKernelGGL((k_attend_join<D, TYPE>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, A, s.tile_rows);
  }
}

template <int D, int IN>
void launch_norm(const NormArgs& A, int out, hipStream_t st) {
  const dim3 g((unsigned)A.n_tok), b(256);
  if (out == STQ_FP32) hipLaunchKernelGGL((k_qk_norm_rope<D, IN, STQ_FP32>), g, b, 0, st, A);
  else hipLaunchKernelGGL((k_qk_norm_rope<D, IN, IN>), g, b, 0, st, A);
}
template <int D>
void launch_norm_in(const NormArgs& A, int in, int out, hipStream_t st) {
  if (in == STQ_BF16) launch_norm<D, STQ_BF16>(A, out, st);
  else if (in == STQ_FP16) launch_norm<D, STQ_FP16>(A, out, st);
  else launch_norm<D, STQ_FP32>(A, out, st);
}

template <int D>
void launch_kv(const StoreArgs& A, int type, bool store, hipStream_t st) {
  constexpr int RPB = 256 / (D / 8);
  const dim3 g((unsigned)(((int64_t)A.n_tok * A.heads + RPB - 1) / RPB)), b(256);
  if (store) {
    if (type == STQ_BF16) hipLaunchKernelGGL((k_kv_store<D, STQ_BF16>), g, b, 0, st, A);
    else if (type == STQ_FP16) hipLaunchKernelGGL((k_kv_store<D, STQ_FP16>), g, b, 0, st, A);
    else hipLaunchKernelGGL((k_kv_store<D, STQ_FP32>), g, b, 0, st, A);
  } else {
    if (type == STQ_BF16) hipLaunchKernelGGL((k_kv_fetch<D, STQ_BF16>), g, b, 0, st, A);
    else if (type == STQ_FP16) hipLaunchKernelGGL((k_kv_fetch<D, STQ_FP16>), g, b, 0, st, A);
    else hipLaunchKernelGGL((k_kv_fetch<D, STQ_FP32>), g, b, 0, st, A);
  }
}

}  // namespace

extern "C" {

size_t stq_kv_bytes(const stq_kv_desc* d) { return kv_ok(d) ? (size_t)kv_size(d) : 0; }

stq_status stq_kv_plan(int32_t n, const int32_t* cached, const int32_t* fresh, const int32_t* free_list, int32_t n_free,
                       int32_t n_blocks, int32_t block_tokens, int32_t* table, int32_t table_cols, int32_t n_tok,
                       int32_t* tok_start, int32_t* len, int32_t* pos, int64_t* slot, int32_t* used, hipStream_t st) {
  if (n < 1 || n > PLAN_MAX || n_free < 0 || n_blocks < 1 || table_cols < 1 || n_tok < 0) return STQ_ERR_ARG;
  if (block_tokens != 32 && block_tokens != 64 && block_tokens != 128 && block_tokens != 256) return STQ_ERR_ARG;
  if (!cached || !fresh || (n_free > 0 && !free_list) || !table || !tok_start || !len || !used) return STQ_ERR_ARG;
  if (n_tok > 0 && (!pos || !slot)) return STQ_ERR_ARG;
  PlanArgs A;
  A.cached = cached; A.fresh = fresh; A.free_list = free_list;
  A.n = n; A.n_free = n_free; A.n_blocks = n_blocks; A.T = block_tokens; A.cols = table_cols; A.n_tok = n_tok;
  A.table = table; A.tok_start = tok_start; A.len = len; A.pos = pos; A.slot = slot; A.used = used;
  int64_t g = ((int64_t)n_tok + 2 * PLAN_NT - 1) / (2 * PLAN_NT);
  g = g < 1 ? 1 : (g > 256 ? 256 : g);
  const unsigned lds = 4u * (2u * (n + 1) + 2u * (PLAN_NT / 64));
  hipLaunchKernelGGL(k_kv_plan, dim3((unsigned)g), dim3(PLAN_NT), lds, st, A);
  return launched();
}

stq_status stq_qk_norm_rope(const stq_norm_desc* d, const void* q, const void* k, const float* wq, const float* wk,
                            const int32_t* pos, const float* cos_sin, void* qo, void* ko, hipStream_t st) {
  if (!d || d->n_tok < 0 || d->n_q_heads < 1 || d->n_k_heads < 0 || d->n_q_heads > 65536 || d->n_k_heads > 65536)
    return STQ_ERR_ARG;
  if (d->d != 64 && d->d != 128 && d->d != 256) return STQ_ERR_ARG;
  if (d->in_type < STQ_BF16 || d->in_type > STQ_FP32) return STQ_ERR_ARG;
  if (d->out_type != d->in_type && d->out_type != STQ_FP32) return STQ_ERR_ARG;
  if (d->norm < STQ_NORM_NONE || d->norm > STQ_NORM_L2) return STQ_ERR_ARG;
  if (d->norm != STQ_NORM_NONE && !(d->eps > 0.0f && isfinite(d->eps))) return STQ_ERR_ARG;
  if (d->n_rot < 0 || d->n_rot > d->d || d->n_rot % 16) return STQ_ERR_ARG;
  if (d->rot_pairs != STQ_ROT_HALVES && d->rot_pairs != STQ_ROT_ADJACENT) return STQ_ERR_ARG;
  if (d->n_rot > 0 && d->n_pos < 1) return STQ_ERR_ARG;
  if (d->n_tok == 0) return STQ_OK;
  if (!q || !qo || (d->n_k_heads > 0 && (!k || !ko)) || (d->n_rot > 0 && (!pos || !cos_sin))) return STQ_ERR_ARG;
  const int64_t qw = (int64_t)d->n_q_heads * d->d, kw = (int64_t)d->n_k_heads * d->d;
  if (!aligned(q) || !aligned(qo) || !aligned(wq) || !aligned(wk) || !aligned(cos_sin) || !stride_ok(d->q_stride, qw, d->in_type) ||
      !stride_ok(d->q_out_stride, qw, d->out_type))
    return STQ_ERR_LAYOUT;
  if (d->n_k_heads > 0 && (!aligned(k) || !aligned(ko) || !stride_ok(d->k_stride, kw, d->in_type) ||
                           !stride_ok(d->k_out_stride, kw, d->out_type)))
    return STQ_ERR_LAYOUT;
  if ((q == qo && (d->q_stride != d->q_out_stride || d->in_type != d->out_type)) ||
      (d->n_k_heads > 0 && k == ko && (d->k_stride != d->k_out_stride || d->in_type != d->out_type)))
    return STQ_ERR_ARG;
  NormArgs A;
  A.q = q; A.k = k; A.qo = qo; A.ko = ko; A.wq = wq; A.wk = wk; A.cs = cos_sin; A.pos = pos;
  A.n_tok = d->n_tok; A.hq = d->n_q_heads; A.hk = d->n_k_heads; A.n_rot = d->n_rot; A.n_pos = d->n_pos; A.norm = d->norm;
  A.adjacent = d->rot_pairs == STQ_ROT_ADJACENT; A.eps = d->eps;
  A.qs = d->q_stride; A.ks = d->k_stride; A.qos = d->q_out_stride; A.kos = d->k_out_stride;
  if (d->d == 64) launch_norm_in<64>(A, d->in_type, d->out_type, st);
  else if (d->d == 128) launch_norm_in<128>(A, d->in_type, d->out_type, st);
  else launch_norm_in<256>(A, d->in_type, d->out_type, st);
  return launched();
}

stq_status stq_kv_store(const stq_kv_desc* d, void* cache, size_t bytes, const int64_t* slot, int32_t n_tok, const void* k,
                        const void* v, int64_t k_stride, int64_t v_stride, int32_t type, hipStream_t st) {
  const stq_status s = kv_check(d, cache, bytes);
  if (s != STQ_OK) return s;
  if (n_tok < 0 || type < STQ_BF16 || type > STQ_FP32) return STQ_ERR_ARG;
  if (n_tok == 0) return STQ_OK;
  if (!slot || !k || !v) return STQ_ERR_ARG;
  const int64_t w = (int64_t)d->n_kv_heads * d->d;
  if (!aligned(k) || !aligned(v) || !stride_ok(k_stride, w, type) || !stride_ok(v_stride, w, type)) return STQ_ERR_LAYOUT;
  StoreArgs A;
  memset(&A, 0, sizeof(A));
  A.cache = (uint8_t*)cache; A.slot = slot; A.k = k; A.v = v; A.n_tok = n_tok; A.heads = d->n_kv_heads;
  A.T = d->block_tokens; A.n_slots = (int64_t)d->n_blocks * d->block_tokens; A.ks = k_stride; A.vs = v_stride;
  if (d->d == 64) launch_kv<64>(A, type, true, st);
  else launch_kv<128>(A, type, true, st);
  return launched();
}

stq_status stq_kv_fetch(const stq_kv_desc* d, const void* cache, size_t bytes, const int64_t* slot, int32_t n_tok,
                        void* k_out, void* v_out, int32_t type, hipStream_t st) {
  const stq_status s = kv_check(d, cache, bytes);
  if (s != STQ_OK) return s;
  if (n_tok < 0 || type < STQ_BF16 || type > STQ_FP32) return STQ_ERR_ARG;
  if (n_tok == 0) return STQ_OK;
  if (!slot || !k_out || !v_out) return STQ_ERR_ARG;
  if (!aligned(k_out) || !aligned(v_out)) return STQ_ERR_LAYOUT;
  StoreArgs A;
  memset(&A, 0, sizeof(A));
  A.cache = (uint8_t*)cache; A.slot = slot; A.ko = k_out; A.vo = v_out; A.n_tok = n_tok; A.heads = d->n_kv_heads;
  A.T = d->block_tokens; A.n_slots = (int64_t)d->n_blocks * d->block_tokens;
  if (d->d == 64) launch_kv<64>(A, type, false, st);
  else launch_kv<128>(A, type, false, st);
  return launched();
}

size_t stq_kv_attend_bytes(const stq_kv_desc* d, const stq_attend_desc* a) {
  if (!kv_ok(d) || !attend_ok(d, a)) return 0;
  const Split s = split_of(d, a);
  if (s.splits <= 1) return 0;
  return (size_t)s.splits * a->n_tok * a->n_heads * (d->d + 2) * 4;
}

stq_status stq_kv_attend(const stq_kv_desc* d, const void* cache, size_t bytes, const stq_attend_desc* a,
                         const int32_t* table, const int32_t* tok_start, const int32_t* len, const void* q, void* o,
                         void* work, size_t work_bytes, hipStream_t st) {
  const stq_status s = kv_check(d, cache, bytes);
  if (s != STQ_OK) return s;
  if (!attend_ok(d, a)) return STQ_ERR_ARG;
  if (a->n_req == 0 || a->n_tok == 0) return STQ_OK;
  if (!table || !tok_start || !len || !q || !o) return STQ_ERR_ARG;
  const int64_t w = (int64_t)a->n_heads * d->d;
  if (!aligned(q) || !aligned(o) || !stride_ok(a->q_stride, w, a->type) || !stride_ok(a->o_stride, w, a->type))
    return STQ_ERR_LAYOUT;
  const Split sp = split_of(d, a);
  const size_t need = stq_kv_attend_bytes(d, a);
  if (need > 0 && (!work || !aligned(work) || work_bytes < need)) return STQ_ERR_LAYOUT;
  if ((int64_t)a->n_req * d->n_kv_heads * sp.tiles * sp.splits > INT32_MAX ||
      (int64_t)a->n_req * a->max_new * a->n_heads > INT32_MAX)
    return STQ_ERR_UNSUPPORTED;
  AttnArgs A;
  A.cache = (const uint8_t*)cache; A.table = table; A.tok_start = tok_start; A.len = len; A.q = q; A.o = o;
  A.n_req = a->n_req; A.n_tok = a->n_tok; A.hq = a->n_heads; A.hkv = d->n_kv_heads; A.group = a->n_heads / d->n_kv_heads;
  A.T = d->block_tokens; A.n_blocks = d->n_blocks; A.cols = a->table_cols; A.max_new = a->max_new; A.window = a->window;
  A.sink = a->n_sink; A.splits = sp.splits; A.tiles = sp.tiles; A.qs = a->q_stride; A.os = a->o_stride;
  A.scale_log2 = a->scale * 1.44269504088896340736f;
  A.po = (float*)work;
  A.pml = A.po + (int64_t)sp.splits * a->n_tok * a->n_heads * d->d;
  if (d->d == 64) {
    if (a->type == STQ_BF16) launch_attend<64, STQ_BF16>(A, sp, st);
    else launch_attend<64, STQ_FP16>(A, sp, st);
  } else {
    if (a->type == STQ_BF16) launch_attend<128, STQ_BF16>(A, sp, st);
    else launch_attend<128, STQ_FP16>(A, sp, st);
  }
  return launched();
}

}  // extern "C"
