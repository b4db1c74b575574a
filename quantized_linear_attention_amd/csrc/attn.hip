// attn.hip — gfx950 kernels and C ABI of the softmax layers' operators
// (contract: include/stq.h, "THE SOFTMAX LAYERS OF A HYBRID MODEL"): the
// block plan, the norm and rotation of queries and keys, the 4-bit key/value
// cache and attention over it.
#include "attn_device.h"

namespace {

// ------------------------------------------------------------ block plan
//
// Latency bound: a chain of one read of the counts, the scans, a search and the
// writes (64 requests of one token 3.8 us, 512 requests with 33,000 tokens 5.7
// us, of which a launch alone takes 2).
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
  int32_t* old = (int32_t*)(blk0 + n + 1);         // [n] cached tokens
  uint32_t* tot = blk0 + n + 1 + n;    // [2][PLAN_NT / 64] totals of the waves
  const int T = A.T, lg = 31 - __builtin_clz(T), cap = A.cols;    // (a power of two: shifts for the 64-bit divisions)
  constexpr int NW = PLAN_NT / 64;
  uint32_t run_t = 0, run_b = 0;
  for (int base = 0; base < n; base += PLAN_NT) {
    const int i = base + tid;
    uint32_t m = 0, add = 0;
    int32_t c = 0;
    if (i < n) {
      c = max(A.cached[i], 0);
      m = (uint32_t)max(A.fresh[i], 0);
      const int64_t have = min(((int64_t)c + T - 1) >> lg, (int64_t)cap);
      const int64_t need = min(((int64_t)c + m + T - 1) >> lg, (int64_t)cap);
      add = (uint32_t)(need - have);
      if (blockIdx.x == 0) A.len[i] = (int32_t)min((int64_t)c + m, (int64_t)INT32_MAX);
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
    if (i < n) { tok0[i] = bt + st - m; blk0[i] = bb + sb - add; old[i] = c; }
    __syncthreads();
  }
  if (tid == 0) { tok0[n] = run_t; blk0[n] = run_b; }
  __syncthreads();
  const uint32_t step = gridDim.x * PLAN_NT, first = blockIdx.x * PLAN_NT + tid;
  for (uint32_t i = first; i <= (uint32_t)n; i += step) A.tok_start[i] = (int32_t)tok0[i];
  if (blockIdx.x == 0 && tid == 0) A.used[0] = (int32_t)run_b;
  for (uint64_t v = first; v < run_b; v += step) {       // (64 bits: garbage counts must not keep it going)
    const uint32_t u = (uint32_t)v;
    const int i = owner(blk0, n, u);
    const int have = (int)(((int64_t)old[i] + T - 1) >> lg);
    const int64_t col = (int64_t)have + (u - blk0[i]);
    if (col < cap) A.table[(int64_t)i * cap + col] = u < (uint32_t)A.n_free ? A.free_list[u] : -1;
  }
  for (uint32_t t = first; t < (uint32_t)A.n_tok; t += step) {
    int32_t pos = -1;
    int64_t slot = -1;
    if (t < run_t) {
      const int i = owner(tok0, n, t);
      const int64_t c = old[i], p = c + (t - tok0[i]);
      const int64_t have = (c + T - 1) >> lg, col = p >> lg;
      pos = (int32_t)min(p, (int64_t)INT32_MAX);
      if (col < cap) {
        const uint32_t u = blk0[i] + (uint32_t)(col - have);
        const int blk = col < have ? A.table[(int64_t)i * cap + col] : (u < (uint32_t)A.n_free ? A.free_list[u] : -1);
        if ((uint32_t)blk < (uint32_t)A.n_blocks) slot = (int64_t)blk * T + (p & (T - 1));
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
// 64/(D/8) heads of one token at a time and all of a token's where there are
// tokens enough (`per_tok` waves share a token's heads else), so that the
// token's cosines and sines are loaded once for many rows; two such sets of
// rows are under way at once.  A rotation's other half of a pair comes from
// another lane by DPP (through LDS, as __shfl goes, the exchange alone took
// longer than the memory: 137 us for 16,381 tokens of 40 heads).
// Memory bound: those 16,381 tokens take 67 us, 5.0 TB/s read and written (a
// copy of 1 GiB runs at 5.16); 64 tokens 4.7 us.
struct NormArgs {
  const void *q, *k;
  void *qo, *ko;
  const float *wq, *wk, *cs;
  const int32_t* pos;
  int n_tok, hq, hk, n_rot, n_pos, norm, adjacent, per_tok;
  Div by_per_tok;
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

// x of the lane m lanes up or down (m = half the lanes of the rotated
// channels; lanes in pairs of groups of m)
__device__ __forceinline__ float across(float x, int m, int mate) {
  const int v = __builtin_bit_cast(int, x);
  if (m == 8) return dpp<0x128>(x);                    // row_ror:8
  if (m == 4)                                          // lanes 0-3 from 4 up, 4-7 from 4 down, and so on
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_amdgcn_update_dpp(0, v, 0x104, 0xF, 0x5, false), v, 0x114, 0xF, 0xA, false));
  if (m == 2) return dpp<0x4E>(x);
  if (m == 1) return dpp<0xB1>(x);
  return __shfl(x, mate, 64);
}

template <int D, int IN, int OUT, bool PAST>
__global__ void __launch_bounds__(256) k_qk_norm_rope(NormArgs A) {
  constexpr int LPR = D / 8, RPW = 64 / LPR, U = 2;
  const int lane = threadIdx.x & 63;
  const int li = lane % LPR, c0 = 8 * li;
  const int gw = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  const int tok = quot(gw, A.by_per_tok), part = gw - tok * A.per_tok;
  if (tok >= A.n_tok) return;
  const int64_t t = tok;
  const int rows = A.hq + A.hk, R = A.n_rot, step = A.per_tok * RPW;
  // rows of set x: first + x * step; past the end the last row, not stored
  const int first = part * RPW + lane / LPR;
  float x[U][8];
  auto load = [&](int h, float* y) {
    h = min(h, rows - 1);
    if (h < A.hq) load8<IN, true>(A.q, t * A.qs + (int64_t)h * D + c0, y);
    else load8<IN, true>(A.k, t * A.ks + (int64_t)(h - A.hq) * D + c0, y);
  };
#pragma unroll
  for (int u = 0; u < U; u++) load(first + u * step, x[u]);
  float cs[8], sn[8];
  bool turn = false;
  if (R > 0) {
    const int p = ld_const(A.pos + t);
    if ((uint32_t)p >= (uint32_t)A.n_pos) return;      // a padded row: the whole token
    turn = c0 < R;
    if (turn) {
      const float* row = A.cs + (int64_t)p * R;
      if (A.adjacent) {                                // pair i: channels 2i, 2i + 1
        const f32x4 c = *(const f32x4*)(row + c0 / 2), s = *(const f32x4*)(row + R / 2 + c0 / 2);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          cs[2 * i] = cs[2 * i + 1] = c[i];
          sn[2 * i] = -s[i];
          sn[2 * i + 1] = s[i];
        }
      } else {                                         // pair i: channels i, i + R/2
        const bool low = c0 < R / 2;
        const float* r = row + (low ? c0 : c0 - R / 2);
        load8<STQ_FP32>(r, 0, cs);
        load8<STQ_FP32>(r, R / 2, sn);
        if (low)
#pragma unroll
          for (int i = 0; i < 8; i++) sn[i] = -sn[i];
      }
    }
  }
  // halves: the lane with the other half of this lane's pairs; a row's rotated lanes are 0 .. R/8-1
  const int m = R / 16;
  const int mate = turn ? (lane - li) + (c0 < R / 2 ? li + m : li - m) : lane;
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; i++) wq[i] = wk[i] = 1.0f;
  if (A.wq) load8<STQ_FP32>(A.wq, c0, wq);
  if (A.wk) load8<STQ_FP32>(A.wk, c0, wk);
  auto row = [&](int h, float* y) {
    if (A.norm != STQ_NORM_NONE) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; i++) s = __builtin_fmaf(y[i], y[i], s);
      s = row_sum<LPR>(s);
      if (A.norm == STQ_NORM_RMS) s *= 1.0f / D;
      const float f = 1.0f / __builtin_sqrtf(s + A.eps);
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] *= f;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] *= h < A.hq ? wq[i] : wk[i];
    if (R > 0) {
      float z[8];
      if (A.adjacent) {
#pragma unroll
        for (int i = 0; i < 8; i++) z[i] = y[i ^ 1];
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) z[i] = across(y[i], m, mate);
      }
      if (turn) {
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = __builtin_fmaf(y[i], cs[i], z[i] * sn[i]);
      }
    }
    if (h < rows) {
      if (h < A.hq) store8<OUT, PAST>(A.qo, t * A.qos + (int64_t)h * D + c0, y);
      else store8<OUT, PAST>(A.ko, t * A.kos + (int64_t)(h - A.hq) * D + c0, y);
    }
  };
  for (int h = first; h - lane / LPR < rows; h += U * step) {
    float next[U][8];
#pragma unroll
    for (int u = 0; u < U; u++) load(h + (U + u) * step, next[u]);
#pragma unroll
    for (int u = 0; u < U; u++) row(h + u * step, x[u]);
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int i = 0; i < 8; i++) x[u][i] = next[u][i];
  }
}

// ------------------------------------------------------- key/value cache
struct StoreArgs {
  uint8_t* cache;
  const int64_t* slot;
  const void *k, *v;
  void *ko, *vo;
  int n_tok, heads, T;
  Div by_heads;
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
// eight channels as one dword of codes; the block's largest magnitude over its
// four lanes.  The conversion divides by the scale, rounds to nearest with ties
// to the even code and saturates (tests/test_gpu_attn.py goes through every
// level, midpoint and neighbour at every exponent).
__device__ __forceinline__ uint32_t codes8(const float* x, int* e_out) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) m = __builtin_fmaxf(m, __builtin_fabsf(x[i]));
  m = rb_max_pos<4>(m);
  const int e = scale_exp(m);
  const float sc = bits_f((uint32_t)(e + 127) << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], sc, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], sc, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], sc, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], sc, 3);
  *e_out = e;
  return w;
}

// Memory bound: 32,749 tokens of 8 heads at d = 64 written from binary16 and
// read back as bfloat16 take 29 us for 170 MB (the codes in between stay in
// the caches), 512 tokens 4.5 us in two launches.
//
// One (token, head) on D/8 lanes, keys and values together (the NaN rule needs
// both).  A workgroup takes consecutive tokens of one head, whose codes and
// scales lie side by side where the slots do; the heads come fastest, so that
// the workgroups at work share the tokens' rows.
struct StoreAt { int64_t t; int h, li; bool on; };
template <int D>
__device__ __forceinline__ StoreAt store_at(const StoreArgs& A) {
  constexpr int LPR = D / 8, RPB = 256 / LPR;
  StoreAt s;
  const uint32_t tile = quot(blockIdx.x, A.by_heads);
  s.h = (int)(blockIdx.x - tile * (uint32_t)A.heads);
  s.li = threadIdx.x % LPR;
  s.t = (int64_t)tile * RPB + threadIdx.x / LPR;
  s.on = s.t < A.n_tok;
  return s;
}
// first byte of the slot's block for this head, and the slot's place in it
template <int D>
__device__ __forceinline__ uint8_t* block_at(const StoreArgs& A, int64_t slot, int h, int* off) {
  const int shift = 31 - __builtin_clz(A.T);
  *off = (int)(slot & (A.T - 1));
  return A.cache + ((slot >> shift) * A.heads + h) * ((int64_t)A.T * D / 16 * 17);
}

template <int D, int TYPE>
__global__ void __launch_bounds__(256) k_kv_store(StoreArgs A) {
  constexpr int LPR = D / 8;
  const StoreAt s = store_at<D>(A);
  const int li = s.li;
  const int64_t t = s.on ? s.t : A.n_tok - 1;          // (lanes past the end read the last token's row again)
  const int64_t slot = A.slot[t];
  const bool live = s.on && slot >= 0 && slot < A.n_slots;
  float k[8], v[8];
  load8<TYPE>(A.k, t * A.ks + (int64_t)s.h * D + 8 * li, k);
  load8<TYPE>(A.v, t * A.vs + (int64_t)s.h * D + 8 * li, v);
  // 0 * x is 0 for every finite x, NaN for the others
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) z = __builtin_fmaf(k[i], 0.0f, __builtin_fmaf(v[i], 0.0f, z));
  const uint64_t any = __ballot(z != z);
  const int l0 = (threadIdx.x & 63) - li;
  const bool poison = ((any >> l0) & ((1ull << LPR) - 1)) != 0;
  if (poison) {
#pragma unroll
    for (int i = 0; i < 8; i++) k[i] = v[i] = 0.0f;
  }
  int ek, ev;
  const uint32_t ck = codes8(k, &ek), cv = codes8(v, &ev);
  if (!live) return;
  const int T = A.T;
  int off;
  uint8_t* hb = block_at<D>(A, slot, s.h, &off);
  *(uint32_t*)(hb + off * (D / 2) + 4 * li) = ck;
  *(uint32_t*)(hb + T * (D / 2) + off * (D / 2) + 4 * li) = cv;
  if ((li & 3) == 0) {
    uint8_t* sc = hb + T * D + (li >> 2) * T + off;
    sc[0] = poison ? 255 : (uint8_t)(ek + 127);
    sc[T * (D / 32)] = (uint8_t)(ev + 127);
  }
}

// eight codes of a dword as elements: the conversion's binary16 pairs are
// exact, and NaN for scale byte 255
template <int TYPE, bool PAST>
__device__ __forceinline__ void fetch8(uint32_t w, uint32_t sbyte, void* out, int64_t at) {
  const float sc = bits_f(sbyte << 23);
  uint32_t h[4];
  h[0] = h2_bits(__builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 0)));
  h[1] = h2_bits(__builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 1)));
  h[2] = h2_bits(__builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 2)));
  h[3] = h2_bits(__builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 3)));
  if constexpr (TYPE == STQ_FP16) {
    store16<PAST>((u32x4*)((uint16_t*)out + at), (u32x4){h[0], h[1], h[2], h[3]});
  } else {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = (float)as_h2(h[i >> 1])[i & 1];
    store8<TYPE, PAST>(out, at, x);
  }
}

template <int D, int TYPE, bool PAST>
__global__ void __launch_bounds__(256) k_kv_fetch(StoreArgs A) {
  const StoreAt s = store_at<D>(A);
  if (!s.on) return;
  const int li = s.li;
  const int64_t slot = A.slot[s.t];
  if (slot < 0 || slot >= A.n_slots) return;
  const int T = A.T;
  int off;
  const uint8_t* hb = block_at<D>(A, slot, s.h, &off);
  const uint32_t ck = *(const uint32_t*)(hb + off * (D / 2) + 4 * li);
  const uint32_t cv = *(const uint32_t*)(hb + T * (D / 2) + off * (D / 2) + 4 * li);
  const uint8_t* sc = hb + T * D + (li >> 2) * T + off;
  const uint32_t sk = sc[0], sv = sc[T * (D / 32)];
  const int64_t at = (s.t * A.heads + s.h) * D + 8 * li;
  fetch8<TYPE, PAST>(ck, sk, A.ko, at);
  fetch8<TYPE, PAST>(cv, sv, A.vo, at);
}

// ------------------------------------------------------------------ host

// A cache larger than the last-level cache is read past the caches at d = 128:
// nothing of it would be there at the next call (rates at 32 heads over 8: 570
// MB of pages 78 -> 73 us, 1.1 GB 161 -> 146, three times the rows per head 109
// -> 106; 139 MB, which the next call finds again, 22.4 -> 23.1; d = 64, whose
// loads cover half lines, 50 -> 54 and stays as it is).
constexpr int64_t LAST_CACHE_BYTES = 256 << 20;
Split split_of(const stq_kv_desc* d, const stq_attend_desc* a) {
  Split s;
  const int64_t rows = (int64_t)a->max_new * (a->n_heads / d->n_kv_heads);
  s.staged = rows > STAGED_ROWS;
  s.tile_rows = s.staged ? 32 * TILE_WAVES : rows > 16 ? 32 : 16;
  s.tiles = (int)((rows + s.tile_rows - 1) / s.tile_rows);
  const int64_t base = (int64_t)a->n_req * d->n_kv_heads * s.tiles;
  int64_t seen = a->max_len;
  if (a->window > 0) seen = seen < (int64_t)a->window + a->n_sink + 64 ? seen : (int64_t)a->window + a->n_sink + 64;
  const int64_t chunks = (seen + 31) / 32;
  s.once = d->d == 128 && (double)chunks * 32 * 17 / 16 * d->d * d->n_kv_heads * a->n_req > (double)LAST_CACHE_BYTES;
  cut(&s, base, chunks);
  return s;
}

template <int D, int TYPE, bool ONCE>
void launch_rows(AttnArgs& A, const Split& s, hipStream_t st) {
  const dim3 grid((unsigned)(A.n_req * A.hkv), (unsigned)A.tiles, (unsigned)A.splits);
  if (s.tile_rows == 32) hipLaunchKernelGGL((k_attend_rows<D, TYPE, 2, 4, ONCE>), grid, dim3(256), 0, st, A);
  else if (s.waves == 16) hipLaunchKernelGGL((k_attend_rows<D, TYPE, 1, 16, false>), grid, dim3(1024), 0, st, A);
  else hipLaunchKernelGGL((k_attend_rows<D, TYPE, 1, 4, ONCE>), grid, dim3(256), 0, st, A);
}
template <int D, int TYPE>
void launch_attend(AttnArgs& A, const Split& s, hipStream_t st) {
  const unsigned grid = (unsigned)((int64_t)A.n_req * A.hkv * A.tiles * A.splits);
  if (s.staged) hipLaunchKernelGGL((k_attend_tiles<D, TYPE>), dim3(grid), dim3(64 * TILE_WAVES), 0, st, A);
  else if (s.once) launch_rows<D, TYPE, D == 128>(A, s, st);
  else launch_rows<D, TYPE, false>(A, s, st);
  if (A.splits > 1) {
    const dim3 rows((unsigned)(A.n_req * A.max_new), (unsigned)((A.hq + 3) / 4));
    hipLaunchKernelGGL((k_attend_join<D, TYPE>), rows, dim3(256), 0, st, A, __builtin_ctz(s.tile_rows));
  }
}

constexpr int64_t NORM_WAVES = 8192;
template <int D, int IN, int OUT>
void launch_norm(const NormArgs& A, bool past, hipStream_t st) {
  const dim3 g((unsigned)(((int64_t)A.n_tok * A.per_tok + 3) / 4)), b(256);
  if (past) hipLaunchKernelGGL((k_qk_norm_rope<D, IN, OUT, true>), g, b, 0, st, A);
  else hipLaunchKernelGGL((k_qk_norm_rope<D, IN, OUT, false>), g, b, 0, st, A);
}
template <int D, int IN>
void launch_norm_out(const NormArgs& A, int out, bool past, hipStream_t st) {
  if (out == STQ_FP32) launch_norm<D, IN, STQ_FP32>(A, past, st);
  else launch_norm<D, IN, IN>(A, past, st);
}
template <int D>
void launch_norm_in(const NormArgs& A, int in, int out, bool past, hipStream_t st) {
  if (in == STQ_BF16) launch_norm_out<D, STQ_BF16>(A, out, past, st);
  else if (in == STQ_FP16) launch_norm_out<D, STQ_FP16>(A, out, past, st);
  else launch_norm_out<D, STQ_FP32>(A, out, past, st);
}

template <int D, int TYPE>
void launch_kv_type(StoreArgs A, bool store, hipStream_t st) {
  constexpr int RPB = 256 / (D / 8);
  const int64_t all = A.n_tok, slice = MOST_GROUPS / A.heads * RPB, w = (int64_t)A.heads * D;
  const bool past = 2 * all * w * elem_bytes(TYPE) > CACHE_BYTES;
  const StoreArgs F = A;
  for (int64_t t = 0; t < all; t += slice) {
    A.n_tok = (int)(all - t < slice ? all - t : slice);
    A.slot = F.slot + t;
    const dim3 g((unsigned)(((int64_t)A.n_tok + RPB - 1) / RPB * A.heads)), b(256);
    if (store) {
      A.k = (const char*)F.k + t * A.ks * elem_bytes(TYPE);
      A.v = (const char*)F.v + t * A.vs * elem_bytes(TYPE);
      hipLaunchKernelGGL((k_kv_store<D, TYPE>), g, b, 0, st, A);
    } else {
      A.ko = (char*)F.ko + t * w * elem_bytes(TYPE);
      A.vo = (char*)F.vo + t * w * elem_bytes(TYPE);
      if (past) hipLaunchKernelGGL((k_kv_fetch<D, TYPE, true>), g, b, 0, st, A);
      else hipLaunchKernelGGL((k_kv_fetch<D, TYPE, false>), g, b, 0, st, A);
    }
  }
}
template <int D>
void launch_kv(const StoreArgs& A, int type, bool store, hipStream_t st) {
  if (type == STQ_BF16) launch_kv_type<D, STQ_BF16>(A, store, st);
  else if (type == STQ_FP16) launch_kv_type<D, STQ_FP16>(A, store, st);
  else launch_kv_type<D, STQ_FP32>(A, store, st);
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
  // every workgroup reads the counts and the free list while others write
  const struct { const void* p; int64_t bytes; } in[] = {{cached, 4ll * n}, {fresh, 4ll * n}, {free_list, 4ll * n_free}},
      out[] = {{table, 4ll * n * table_cols}, {tok_start, 4ll * (n + 1)}, {len, 4ll * n}, {pos, 4ll * n_tok},
               {slot, 8ll * n_tok}, {used, 4}};
  for (const auto& x : in)
    for (const auto& y : out)
      if ((uintptr_t)x.p < (uintptr_t)y.p + y.bytes && (uintptr_t)y.p < (uintptr_t)x.p + x.bytes) return STQ_ERR_ARG;
  PlanArgs A;
  A.cached = cached; A.fresh = fresh; A.free_list = free_list;
  A.n = n; A.n_free = n_free; A.n_blocks = n_blocks; A.T = block_tokens; A.cols = table_cols; A.n_tok = n_tok;
  A.table = table; A.tok_start = tok_start; A.len = len; A.pos = pos; A.slot = slot; A.used = used;
  int64_t g = ((int64_t)n_tok + 2 * PLAN_NT - 1) / (2 * PLAN_NT);
  g = g < 1 ? 1 : (g > 256 ? 256 : g);
  const unsigned lds = 4u * (2u * (n + 1) + n + 2u * (PLAN_NT / 64));
  hipLaunchKernelGGL(k_kv_plan, dim3((unsigned)g), dim3(PLAN_NT), lds, st, A);
  return launched();
}

stq_status stq_qk_norm_rope(const stq_norm_desc* d, const void* q, const void* k, const float* wq, const float* wk,
                            const int32_t* pos, const float* cos_sin, void* qo, void* ko, hipStream_t st) {
  if (!d || d->n_tok < 0 || d->n_tok > (1 << 28) || d->n_q_heads < 1 || d->n_k_heads < 0 || d->n_q_heads > 65536 || d->n_k_heads > 65536)
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
  const int ib = elem_bytes(d->in_type), ob = elem_bytes(d->out_type);
  const Rows rq = {q, d->q_stride * ib, qw * ib}, rqo = {qo, d->q_out_stride * ob, qw * ob}, rk = {k, d->k_stride * ib, kw * ib},
             rko = {ko, d->k_out_stride * ob, kw * ob};
  if (!same(rq, rqo) && meet(rq, rqo, d->n_tok)) return STQ_ERR_ARG;
  if (d->n_k_heads > 0 && ((!same(rk, rko) && meet(rk, rko, d->n_tok)) || meet(rk, rqo, d->n_tok) || meet(rq, rko, d->n_tok) ||
                           meet(rqo, rko, d->n_tok)))
    return STQ_ERR_ARG;
  NormArgs A;
  A.q = q; A.k = k; A.qo = qo; A.ko = ko; A.wq = wq; A.wk = wk; A.cs = cos_sin; A.pos = pos;
  A.n_tok = d->n_tok; A.hq = d->n_q_heads; A.hk = d->n_k_heads; A.n_rot = d->n_rot; A.n_pos = d->n_pos; A.norm = d->norm;
  A.adjacent = d->rot_pairs == STQ_ROT_ADJACENT; A.eps = d->eps;
  A.qs = d->q_stride; A.ks = d->k_stride; A.qos = d->q_out_stride; A.kos = d->k_out_stride;
  const bool past = (int64_t)A.n_tok * (A.hq + A.hk) * d->d * elem_bytes(d->out_type) > CACHE_BYTES;
  // waves of one token: as many as fill the card, each with two sets of rows at least
  const int sets = (A.hq + A.hk + 512 / d->d - 1) / (512 / d->d);
  A.per_tok = (int)((NORM_WAVES + A.n_tok - 1) / A.n_tok);
  if (A.per_tok > (sets + 1) / 2) A.per_tok = (sets + 1) / 2;
  A.by_per_tok = div_of(A.per_tok);
  const int64_t slice = A.per_tok > 1 ? d->n_tok : 4 * MOST_GROUPS;     // (several waves a token: 16,384 waves at most)
  for (int64_t t = 0; t < d->n_tok; t += slice) {
    A.n_tok = (int)(d->n_tok - t < slice ? d->n_tok - t : slice);
    A.q = (const char*)q + t * d->q_stride * ib;
    A.qo = (char*)qo + t * d->q_out_stride * ob;
    if (k) A.k = (const char*)k + t * d->k_stride * ib;
    if (ko) A.ko = (char*)ko + t * d->k_out_stride * ob;
    if (pos) A.pos = pos + t;
    if (d->d == 64) launch_norm_in<64>(A, d->in_type, d->out_type, past, st);
    else if (d->d == 128) launch_norm_in<128>(A, d->in_type, d->out_type, past, st);
    else launch_norm_in<256>(A, d->in_type, d->out_type, past, st);
  }
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
  A.cache = (uint8_t*)cache; A.slot = slot; A.k = k; A.v = v; A.n_tok = n_tok; A.heads = d->n_kv_heads; A.by_heads = div_of(A.heads);
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
  A.cache = (uint8_t*)cache; A.slot = slot; A.ko = k_out; A.vo = v_out; A.n_tok = n_tok; A.heads = d->n_kv_heads; A.by_heads = div_of(A.heads);
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
  const Rows rq = {q, a->q_stride * 2, w * 2}, ro = {o, a->o_stride * 2, w * 2};
  if (!same(rq, ro) && meet(rq, ro, a->n_tok)) return STQ_ERR_ARG;
  const Split sp = split_of(d, a);
  const size_t need = stq_kv_attend_bytes(d, a);
  if (need > 0 && (!work || !aligned(work) || work_bytes < need)) return STQ_ERR_LAYOUT;
  const int64_t groups = (int64_t)a->n_req * d->n_kv_heads;
  if ((int64_t)a->n_req * a->max_new * a->n_heads > INT32_MAX ||
      (sp.staged ? groups * sp.tiles * sp.splits * 64 * TILE_WAVES : groups * 64 * sp.waves) > MOST_THREADS ||
      (sp.splits > 1 && (int64_t)a->n_req * a->max_new * 256 > MOST_THREADS))
    return STQ_ERR_UNSUPPORTED;
  AttnArgs A;
  A.cache = (const uint8_t*)cache; A.table = table; A.tok_start = tok_start; A.len = len; A.q = q; A.o = o;
  A.n_req = a->n_req; A.n_tok = a->n_tok; A.hq = a->n_heads; A.hkv = d->n_kv_heads; A.group = a->n_heads / d->n_kv_heads;
  A.T = d->block_tokens; A.n_blocks = d->n_blocks; A.cols = a->table_cols; A.max_new = a->max_new;
  A.window = a->window < MOST_WINDOW ? a->window : MOST_WINDOW;
  A.sink = a->n_sink < MOST_WINDOW ? a->n_sink : MOST_WINDOW;
  A.splits = sp.splits; A.per = sp.per; A.tiles = sp.tiles;
  A.by_hkv = div_of(A.hkv); A.by_group = div_of(A.group); A.by_max_new = div_of(A.max_new); A.by_per = div_of(A.per);
  A.qs = a->q_stride; A.os = a->o_stride;
  A.scale = a->scale;
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
