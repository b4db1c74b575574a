// attn_long.hip — gfx950 kernels and C ABI of the softmax layers' operators for
// long contexts (contract: include/stq.h, "LONG CONTEXTS"): bounds of a block's
// keys, scores of the blocks for a query, their selection, attention over the
// selected blocks, and attention of requests that share a prefix.
#include "attn_device.h"

namespace {

// ------------------------------------------------------- bounds of keys
//
// Per channel the least and the largest of a block's keys, as the upper byte
// of binary16 (E5M2), rounded outward: cached keys are exact in binary16 and
// have two significant bits of E5M2's three, so a bound is the key itself from
// 2^-14 on.  A block with a poisoned key gets NaN.
//
// One wave takes one (block, head).  A lane reads the 16 bytes of one token's
// 32 channels of a scale; tokens of a pass lie on lane bits 0, 1, 4, 5 (and 3
// at d = 64), channel groups on bit 2 (and 3), so that the joins over tokens
// are register swaps (permlane32 and 16, each halving what a lane holds) and
// DPP steps.  Lanes past the last token read the last one again.  All of a block's
// loads are asked for at once.  A chain of counts, table and keys bounds it: the
// blocks of 22,871 tokens of 8 heads (d = 128) 7.7 us for 13.3 MB, 1.7 TB/s; 512
// blocks scattered over 2.9 GB of pages 12.6 us for 10.4 MB, where a launch alone takes 2
// (half of its waves have no block: one token may touch two; 329 misses of
// the CUs' address translation a launch against 29).
struct BoundsArgs {
  const uint8_t* cache;
  const int32_t *table, *tok_start, *len;
  uint8_t* bounds;
  int n_req, hkv, T, n_blocks, cols, max_new, span;
  Div by_span;
};

__device__ __forceinline__ f16x2 min2(f16x2 a, f16x2 b) { return __builtin_elementwise_min(a, b); }
__device__ __forceinline__ f16x2 max2(f16x2 a, f16x2 b) { return __builtin_elementwise_max(a, b); }
template <bool MAX>
__device__ __forceinline__ f16x2 best2(f16x2 a, f16x2 b) {
  if constexpr (MAX) return max2(a, b);
  else return min2(a, b);
}
// N pairs of every lane -> N / 2: the two halves of the wave (rows of 16 lanes)
// join theirs, the lower lanes keep the first half of the pairs, the upper the second
template <bool MAX, int N>
__device__ __forceinline__ void halve32(f16x2* x) {
#pragma unroll
  for (int i = 0; i < N / 2; i++) {
    auto r = __builtin_amdgcn_permlane32_swap(h2_bits(x[i]), h2_bits(x[i + N / 2]), false, false);
    x[i] = best2<MAX>(as_h2(r[0]), as_h2(r[1]));
  }
}
template <bool MAX, int N>
__device__ __forceinline__ void halve16(f16x2* x) {
#pragma unroll
  for (int i = 0; i < N / 2; i++) {
    auto r = __builtin_amdgcn_permlane16_swap(h2_bits(x[i]), h2_bits(x[i + N / 2]), false, false);
    x[i] = best2<MAX>(as_h2(r[0]), as_h2(r[1]));
  }
}
template <bool MAX, int CTRL>
__device__ __forceinline__ f16x2 join2(f16x2 x) {
  return best2<MAX>(x, as_h2((uint32_t)dppi<CTRL>((int)h2_bits(x))));
}
// the upper bytes of four pairs' eight numbers, moved outward where the lower byte has bits
template <bool UP>
__device__ __forceinline__ u32x2 outward(const f16x2* x) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t u = (h2_bits(x[i >> 1]) >> (16 * (i & 1))) & 0xFFFFu;
    b[i] = ((u < 0x8000u) == UP ? u + 0xFFu : u) >> 8;
  }
  return (u32x2){b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24};
}

template <int D>
__global__ void __launch_bounds__(256) k_kv_bounds(BoundsArgs A) {
  constexpr int PASS = D == 128 ? 16 : 32;             // tokens of one load of the wave
  const int lane = threadIdx.x & 63;
  const int h = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
  if (h >= A.hkv) return;
  const int i = quot(blockIdx.x, A.by_span), c = blockIdx.x - i * A.span;
  const int T = A.T, shift = 31 - __builtin_clz(T);
  const int start = ld_const(A.tok_start + i), fresh = max(ld_const(A.tok_start + i + 1) - start, 0);
  const int len = (int)min((int64_t)max(ld_const(A.len + i), 0), (int64_t)A.cols << shift);
  const int64_t base = (int64_t)len - fresh, end = min(base + min(fresh, A.max_new), (int64_t)len);
  const int64_t col = (max(base, (int64_t)0) >> shift) + c;
  if (fresh == 0 || end <= 0 || col << shift >= end) return;
  const int blk = ld_const(A.table + (int64_t)i * A.cols + col);
  if ((uint32_t)blk >= (uint32_t)A.n_blocks) return;
  const int last = (int)min((int64_t)T, len - (col << shift)) - 1;
  const uint64_t unit = (uint64_t)(uint32_t)blk * A.hkv + h;
  const uint8_t* page = A.cache + unit * ((uint64_t)T * D / 16 * 17);
  const int cg = (lane >> 2) & (D / 32 - 1);
  const int tok = (lane & 3) | (D == 128 ? (lane >> 4) << 2 : (lane >> 3) << 2);
  f16x2 lo[16], hi[16];
#pragma unroll
  for (int x = 0; x < 16; x++) {
    lo[x] = as_h2(0x7C007C00u);
    hi[x] = as_h2(0xFC00FC00u);
  }
  uint32_t worst = 0;
  constexpr int U = 4;                                 // passes under way at once
  for (int t0 = 0; t0 <= last; t0 += U * PASS) {
    u32x4 w[U];
    uint32_t sb[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int t = min(t0 + u * PASS + tok, last);
      w[u] = *(const u32x4*)(page + t * (D / 2) + 16 * cg);
      sb[u] = page[T * D + cg * T + t];
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      worst = max(worst, sb[u]);
      const float sc = bits_f(sb[u] << 23);
#pragma unroll
      for (int x = 0; x < 4; x++) {
        const uint32_t p[4] = {cvt2<0>(w[u][x], sc), cvt2<1>(w[u][x], sc), cvt2<2>(w[u][x], sc), cvt2<3>(w[u][x], sc)};
#pragma unroll
        for (int y = 0; y < 4; y++) {
          lo[4 * x + y] = min2(lo[4 * x + y], as_h2(p[y]));
          hi[4 * x + y] = max2(hi[4 * x + y], as_h2(p[y]));
        }
      }
    }
  }
  halve32<false, 16>(lo);
  halve32<true, 16>(hi);
  halve16<false, 8>(lo);
  halve16<true, 8>(hi);
#pragma unroll
  for (int x = 0; x < 4; x++) {
    lo[x] = join2<false, 0x4E>(join2<false, 0xB1>(lo[x]));
    hi[x] = join2<true, 0x4E>(join2<true, 0xB1>(hi[x]));
    if (D == 64) {
      lo[x] = join2<false, 0x128>(lo[x]);
      hi[x] = join2<true, 0x128>(hi[x]);
    }
  }
  const bool poison = __builtin_amdgcn_ballot_w64(worst == 255) != 0;
  // channels 32 cg + 16 (lane bit 5) + 8 (bit 4) .. + 7: the lower bounds by the first lane of four, the upper by the second
  if ((lane & 3) > 1 || (D == 64 && (lane & 8))) return;
  const u32x2 b = lane & 1 ? outward<true>(hi) : outward<false>(lo);
  const u32x2 nan = {0x7F7F7F7Fu, 0x7F7F7F7Fu};
  *(u32x2*)(A.bounds + unit * (2 * D) + (lane & 1) * D + 32 * cg + 16 * (lane >> 5) + 8 * ((lane >> 4) & 1)) = poison ? nan : b;
}

// ------------------------------------------------------ scores of blocks
//
// max over a head group's queries x = scale * q of sum_c max(x_c lo_c, x_c hi_c)
// = x+ . hi + x- . lo: a matrix product over 2 d terms, the bounds (as binary16:
// a byte shifted up) against the queries' positive and negative parts.  Rows of a
// tile: 16 blocks; columns: the heads of a token side by side, the last one
// repeated up to a power of two (a maximum does not mind), so that the group's
// maximum is DPP steps.  Products are exact in binary32.
//
// Memory and latency bound: 64 requests of 8,839 to 32,768 tokens in blocks of
// 64, 32 heads over 8, d = 128: 14 us for 42 MB (3.0 TB/s; the chain of counts,
// table, bounds and store is 5 us of it).  A wave takes four tiles of blocks there:
// 16.6 us with one, 14.9 with two, 15.3 with eight.
struct ScoreArgs : AttnArgs {
  const uint8_t* bounds;
  float* score;
  int rows_shift, tile_run;      // log2 of a token's columns; tiles of 16 blocks that a wave takes in turn
};

__device__ __forceinline__ uint32_t up2(uint32_t w, uint32_t sel) { return __builtin_amdgcn_perm(0u, w, sel); }
// 16 bytes as two operands of eight binary16 numbers
__device__ __forceinline__ void widen(u32x4 w, f16x8* f) {
#pragma unroll
  for (int y = 0; y < 2; y++)
    f[y] = frag(up2(w[2 * y], 0x010C000Cu), up2(w[2 * y], 0x030C020Cu), up2(w[2 * y + 1], 0x010C000Cu), up2(w[2 * y + 1], 0x030C020Cu));
}

// A lane's channels of N query rows, as they lie in memory (16 bytes: eight channels).
template <int D, int N> struct Raw { u32x4 w[N][D / 32]; };
template <int D, int N>
__device__ __forceinline__ void load_raw(const ScoreArgs& A, int64_t at, Raw<D, N>& x, int n) {
  const uint16_t* p = (const uint16_t*)A.q + at;
#pragma unroll
  for (int y = 0; y < D / 64; y++) {
    x.w[n][2 * y] = *(const u32x4*)(p + 64 * y);
    x.w[n][2 * y + 1] = *(const u32x4*)(p + 64 * y + 8);
  }
}
// Their positive and negative parts as operands.  binary16 queries go in as they
// are; bfloat16 ones times a power of two that brings the rows' largest magnitude
// to [2^14, 2^15) (times 2^127 at most: smaller ones are exact in binary16's
// subnormals then): exact down to 2^-29 of it.  *ex: the power of two that the
// products are to be multiplied with, beside the scale's mantissa.
template <int D, int TYPE, int N>
__device__ __forceinline__ void signed_parts(const ScoreArgs& A, const Raw<D, N>& x, f16x8 (*qp)[D / 32], f16x8 (*qn)[D / 32], int* ex) {
  float by = 1.0f;
  *ex = __builtin_amdgcn_frexp_expf(A.scale);
  if constexpr (TYPE == STQ_BF16) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
      for (int i = 0; i < D / 32; i++)
#pragma unroll
        for (int u = 0; u < 4; u++) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x.w[n][i][u] & 0x7FFF7FFFu));
    const int e = min(q_shift(max_quads(bits_f((uint32_t)max(m[0], m[1]) << 16))), 127);
    by = __builtin_ldexpf(A.scale < 0.0f ? -1.0f : 1.0f, e);
    *ex -= e;
  }
  const uint32_t turned = A.scale < 0.0f ? 0x80008000u : 0u;
  const f16x2 zero = {(f16)0.0f, (f16)0.0f};
#pragma unroll
  for (int n = 0; n < N; n++)
#pragma unroll
    for (int i = 0; i < D / 32; i++) {
      uint32_t p[4], q[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const uint32_t w = x.w[n][i][u];
        f16x2 v;
        if constexpr (TYPE == STQ_BF16) v = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(bits_f(w << 16) * by, bits_f(w & 0xFFFF0000u) * by));
        else v = as_h2(w ^ turned);
        p[u] = h2_bits(max2(v, zero));
        q[u] = h2_bits(min2(v, zero));
      }
      qp[n][i] = frag(p[0], p[1], p[2], p[3]);
      qn[n][i] = frag(q[0], q[1], q[2], q[3]);
    }
}

template <int D, int TYPE>
__global__ void __launch_bounds__(256) k_kv_score(ScoreArgs A) {
  constexpr int LD = D / 64;                           // 16-byte loads of one bound
  const int lane = threadIdx.x & 63, n = lane & 15, G = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int i = quot(blockIdx.x, A.by_hkv), h = blockIdx.x - i * A.hkv;
  const Req R = req_args(A, i);
  const int fresh = min(R.n_new, A.max_new), rs = A.rows_shift, TOK = 16 >> rs, tok0 = blockIdx.y * TOK;
  if (tok0 >= fresh) return;
  const int shift = 31 - __builtin_clz(A.T);
  const int p1 = R.base + min(tok0 + TOK, fresh) - 1;
  if (p1 < 0) return;
  const int total = min((p1 >> shift) + 1, A.cols);     // blocks that the last of these tokens sees
  const int32_t* tab = A.table + (int64_t)i * A.cols;
  const int run = 16 * A.tile_run, step = gridDim.z * 4 * run;
  for (int hc = 0; hc < A.group; hc += 16) {            // sixteen heads of the group at a time
    bool ready = false;
    f16x8 qp[1][D / 32], qn[1][D / 32];
    float mul;
    int ex, top;                                       // top: the token's last block (-1: not this lane's to write)
    int64_t to;
    for (int b1 = (blockIdx.z * 4 + wave) * run; b1 < total; b1 += step) {
      const int b2 = min(b1 + run, total);
      u32x4 w[2 * LD];
      bool dead;
      auto load = [&](int b) {
        const int blk = tab[min(b + n, b2 - 1)];
        dead = (uint32_t)blk >= (uint32_t)A.n_blocks;
        const uint8_t* p = A.bounds + ((uint64_t)(uint32_t)(dead ? 0 : blk) * A.hkv + h) * (2 * D) + 16 * G;
#pragma unroll
        for (int x = 0; x < 2 * LD; x++) w[x] = *(const u32x4*)(p + 64 * x);
      };
      load(b1);
      if (!ready) {
        ready = true;
        const int j = tok0 + (n >> rs), jj = min(j, fresh - 1);
        const int g = min(hc + (n & ((1 << rs) - 1)), A.group - 1);
        const int64_t at = (int64_t)(R.first + jj) * A.qs + (int64_t)(h * A.group + g) * D + 16 * G;
        Raw<D, 1> x;
        load_raw<D>(A, at, x, 0);
        signed_parts<D, TYPE, 1>(A, x, qp, qn, &ex);
        mul = __builtin_amdgcn_frexp_mantf(__builtin_fabsf(A.scale));
        const int p = R.base + jj;
        top = j < fresh && (n & ((1 << rs) - 1)) == 0 ? min(p >> shift, A.cols - 1) : -1;
        to = ((int64_t)(R.first + jj) * A.hkv + h) * A.cols;
      }
      for (int b = b1; b < b2; b += 16) {
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < 2 * LD; x++) {
          f16x8 f[2];
          widen(w[x], f);
#pragma unroll
          for (int y = 0; y < 2; y++)
            s = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[y], x < LD ? qn[0][2 * x + y] : qp[0][2 * (x - LD) + y], s, 0, 0, 0);
        }
        const uint32_t gone = (uint32_t)__builtin_amdgcn_ballot_w64(dead) & 0xFFFFu;
        if (b + 16 < b2) load(b + 16);
        f32x4 v;
#pragma unroll
        for (int u = 0; u < 4; u++) {
          float y = __builtin_ldexpf(s[u] * mul, ex);
          if (rs > 0) y = __builtin_fmaxf(y, dpp<0xB1>(y));
          if (rs > 1) y = __builtin_fmaxf(y, dpp<0x4E>(y));
          if (rs > 2) y = __builtin_fmaxf(y, dpp<0x141>(y));
          if (rs > 3) y = __builtin_fmaxf(y, dpp<0x140>(y));
          v[u] = (gone >> (4 * G + u)) & 1 ? NEG_INF : y;
        }
        const int b4 = b + 4 * G;
        if (b4 > top) continue;
        typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
        float* out = A.score + to + b4;
        if (hc > 0)                                    // what this lane has written for the heads before
#pragma unroll
          for (int u = 0; u < 4; u++)
            if (b4 + u <= top) v[u] = __builtin_fmaxf(v[u], out[u]);
        if (b4 + 3 <= top) {
          *(f32x4_a4*)out = v;
        } else {
#pragma unroll
          for (int u = 0; u < 4; u++)
            if (b4 + u <= top) out[u] = v[u];
        }
      }
    }
  }
}

// Many tokens of a request: the products bound the work.  Columns of a product
// are sixteen tokens, and HT products side by side are heads of the group, so that
// the group's maximum is taken between a lane's own registers; a wave holds TT
// such sets of tokens (HT TT products to each widened bound) and goes over the
// blocks that they see.  One power of two scales all of a token's HT queries.
//
// Two prompts of 2,048 and 2,020 tokens behind 14,336 and 8,185, 32 heads over 8, d =
// 128: 27 us for 59 MB and 12.8 GFLOP (70 us by the kernel above, whose columns
// are mostly repeated queries there).  Half of a wave's life is waiting: 33 MB of
// queries come in before its first product and two waves a SIMD fill the registers;
// the matrix cores are busy 20 % of the time.  Waves that take all of a request's
// blocks are the fastest (16 tiles 27 us, 8 33, 4 41: each converts the queries).
template <int D, int TYPE, int HT, int TT>
__global__ void __launch_bounds__(256, 2) k_kv_score_wide(ScoreArgs A) {
  constexpr int LD = D / 64, NT = HT * TT;
  const int lane = threadIdx.x & 63, n = lane & 15, G = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int i = quot(blockIdx.x, A.by_hkv), h = blockIdx.x - i * A.hkv;
  const Req R = req_args(A, i);
  const int fresh = min(R.n_new, A.max_new), tok0 = (blockIdx.y * 4 + wave) * 16 * TT;
  if (tok0 >= fresh) return;
  const int shift = 31 - __builtin_clz(A.T);
  const int p1 = R.base + min(tok0 + 16 * TT, fresh) - 1;
  if (p1 < 0) return;
  const int total = min((p1 >> shift) + 1, A.cols);     // blocks that the last of these tokens sees
  const int32_t* tab = A.table + (int64_t)i * A.cols;
  const int run = 16 * A.tile_run, step = gridDim.z * run;
  struct Tile { u32x4 w[2 * LD]; bool dead; } tile[2];
  __shared__ int entry[4][256];
  // The table entries of 256 blocks of a run, in LDS of the wave's own: asked for
  // tile by tile, each would wait for the scores stored before it.
  int from = 0;
  auto look = [&](int b) {
    from = b;
    int x[4];
#pragma unroll
    for (int y = 0; y < 4; y++) x[y] = tab[min(b + 64 * y + lane, total - 1)];
#pragma unroll
    for (int y = 0; y < 4; y++) entry[wave][64 * y + lane] = x[y];
    lds_wave_fence();
  };
  auto load = [&](Tile& x, int b) {
    if (b < from || b >= from + 256) look(b);
    const int blk = entry[wave][b - from + n];
    const bool dead = (uint32_t)blk >= (uint32_t)A.n_blocks;
    const uint8_t* p = A.bounds + ((uint64_t)(uint32_t)(dead ? 0 : blk) * A.hkv + h) * (2 * D) + 16 * G;
#pragma unroll
    for (int y = 0; y < 2 * LD; y++) x.w[y] = *(const u32x4*)(p + 64 * y);
    x.dead = dead;
  };
  int top[TT];                                         // the token's last block (-1: none)
  int64_t to[TT];
#pragma unroll
  for (int tt = 0; tt < TT; tt++) {
    const int j = tok0 + 16 * tt + n, p = R.base + j;
    top[tt] = j < fresh && p >= 0 ? min(p >> shift, A.cols - 1) : -1;
    to[tt] = ((int64_t)(R.first + min(j, fresh - 1)) * A.hkv + h) * A.cols + 4 * G;
  }
  for (int hc = 0; hc < A.group; hc += HT) {            // HT heads of the group at a time
    int b = blockIdx.z * run, b1 = b;
    if (b >= total) return;
    auto behind = [&](int x) { return x + 16 < b1 + run ? x + 16 : (b1 += step); };   // (past `total`: the end)
    int next = behind(b);
    look(b);
    load(tile[0], b);
    if (next < total) load(tile[1], next);
    f16x8 qp[NT][D / 32], qn[NT][D / 32];
    int ex[TT];
#pragma unroll
    for (int tt = 0; tt < TT; tt++) {
      const int jj = min(tok0 + 16 * tt + n, fresh - 1);
      Raw<D, HT> x;
#pragma unroll
      for (int g = 0; g < HT; g++)
        load_raw<D>(A, (int64_t)(R.first + jj) * A.qs + (int64_t)(h * A.group + min(hc + g, A.group - 1)) * D + 16 * G, x, g);
      signed_parts<D, TYPE, HT>(A, x, &qp[tt * HT], &qn[tt * HT], &ex[tt]);
    }
    const float mul = __builtin_amdgcn_frexp_mantf(__builtin_fabsf(A.scale));
    // one tile of sixteen blocks; the bounds of the one behind the next are asked
    // for before its scores are stored, since waits count both in order
    auto work = [&](Tile& x, int b, int ahead) {
      f32x4 s[NT];
#pragma unroll
      for (int nt = 0; nt < NT; nt++) s[nt] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int z = 0; z < 2 * LD; z++) {
        f16x8 f[2];
        widen(x.w[z], f);
#pragma unroll
        for (int y = 0; y < 2; y++)
#pragma unroll
          for (int nt = 0; nt < NT; nt++)
            s[nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[y], z < LD ? qn[nt][2 * z + y] : qp[nt][2 * (z - LD) + y], s[nt], 0, 0, 0);
      }
      const uint32_t gone = ((uint32_t)__builtin_amdgcn_ballot_w64(x.dead) & 0xFFFFu) >> (4 * G);
      if (ahead < total) load(x, ahead);
#pragma unroll
      for (int tt = 0; tt < TT; tt++) {
        const int b4 = b + 4 * G;
        f32x4 v;
#pragma unroll
        for (int u = 0; u < 4; u++) {
          float y = s[tt * HT][u];
#pragma unroll
          for (int g = 1; g < HT; g++) y = __builtin_fmaxf(y, s[tt * HT + g][u]);
          v[u] = (gone >> u) & 1 ? NEG_INF : __builtin_ldexpf(y * mul, ex[tt]);
        }
        if (b4 > top[tt]) continue;
        typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
        float* out = A.score + to[tt] + b;
        if (hc > 0)                                    // what this lane has written for the heads before
#pragma unroll
          for (int u = 0; u < 4; u++)
            if (b4 + u <= top[tt]) v[u] = __builtin_fmaxf(v[u], out[u]);
        if (b4 + 3 <= top[tt]) {
          *(f32x4_a4*)out = v;
        } else {
#pragma unroll
          for (int u = 0; u < 4; u++)
            if (b4 + u <= top[tt]) out[u] = v[u];
        }
      }
    };
    while (true) {
      int ahead = behind(next);
      work(tile[0], b, ahead);
      if (next >= total) break;
      b = next;
      next = ahead;
      ahead = behind(next);
      work(tile[1], b, ahead);
      if (next >= total) break;
      b = next;
      next = ahead;
    }
  }
}

// --------------------------------------------------- selection of blocks
//
// The `want` largest of a row's scores beside the blocks that are always taken,
// by a threshold on the scores' bits in the order of integers: the number of
// keys above a trial threshold (compares, ballots and population counts, so that
// the search itself runs on the scalar unit) says on which side to go on; trials
// are interpolated between the counts at both ends (every fifth halves the
// range), and from the fifth on the end that moves goes to the next key.  A count
// that meets `want` ends it, or a range of one key, whose equal ones are taken in
// order: 6 to 8 trials for rows of 230 to 2,000 scores, equal ones among them,
// where one bit a trial takes 15 to 18.  The places of the taken blocks are
// population counts of the ballots below, so the list is ascending and the same
// whatever the split.
//
// W waves a row, each with M blocks a lane: block 64 (M wave + m) + lane.
//
// Instruction bound: 32,544 rows of up to 256 scores 29 us (0.34 us a thousand rows
// and wave slot; 340 vector instructions a row and as many scalar ones), 512 rows of
// 138 to 512 7.6 us, of which the launch and the row's loads are five.  Four rows a
// wave with sums over sixteen lanes: 27 us, but 8.1 us for the 512 rows; one bit a
// trial: 53 and 8.6 us.
struct SelectArgs {
  const float* score;
  const int32_t *tok_start, *len;
  int32_t* sel;
  int n_req, n_tok, hkv, T, cols, n_sel, n_first, n_last, max_new;
  Div by_hkv, by_max_new;
};

template <int W, int M>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W) k_kv_select(SelectArgs A) {
  __shared__ uint32_t meet_at[2][W];
  int turn = 0;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int w = W == 1 ? 0 : wave;
  // one number a wave -> f over the row's waves; `before`: over those ahead of this one
  auto all_waves = [&](uint32_t x, auto f, uint32_t none, uint32_t* before) {
    if constexpr (W == 1) {
      *before = none;
      return x;
    } else {
      if (lane == 0) meet_at[turn][wave] = x;
      __syncthreads();
      uint32_t y = none, z = none;
#pragma unroll
      for (int v = 0; v < W; v++) {
        const uint32_t u = meet_at[turn][v];
        if (v < wave) z = f(z, u);
        y = f(y, u);
      }
      turn ^= 1;
      *before = __builtin_amdgcn_readfirstlane(z);
      return (uint32_t)__builtin_amdgcn_readfirstlane(y);
    }
  };
  auto plus = [](uint32_t a, uint32_t b) { return a + b; };
  auto top = [](uint32_t a, uint32_t b) { return max(a, b); };
  auto wave_top = [](uint32_t x) { return (uint32_t)wave_max_i((int)(x ^ 0x80000000u)) ^ 0x80000000u; };
  uint32_t before;

  const uint32_t row = W == 1 ? blockIdx.x * 4 + wave : blockIdx.x;
  const int x = quot(row, A.by_hkv), h = row - x * A.hkv;
  const int i = quot(x, A.by_max_new), j = x - i * A.max_new;
  if (i >= A.n_req) return;
  const int start = max(ld_const(A.tok_start + i), 0), end = max(ld_const(A.tok_start + i + 1), start);
  const int shift = 31 - __builtin_clz(A.T);
  const int len = (int)min((int64_t)max(ld_const(A.len + i), 0), (int64_t)A.cols << shift);
  if (j >= min(min(end, A.n_tok) - start, A.max_new)) return;
  const int p = max(len - (end - start), -(1 << 28)) + j;
  const int nb = p < 0 ? 0 : min((p >> shift) + 1, A.cols);         // blocks that the token sees
  const int64_t at = (int64_t)(start + j) * A.hkv + h;
  const float* in = A.score + at * A.cols;
  int32_t* out = A.sel + at * A.n_sel;
  const int last0 = max(nb - A.n_last, 0), first1 = min(nb, A.n_first);    // blocks below first1 and from last0 on are taken
  const int must = first1 + nb - max(last0, first1);
  const int want = min(A.n_sel, nb) - must;
  // Keys in the order of integers: 0 for what is no candidate (taken already, not
  // seen, -inf), the largest for NaN; -0 counts as 0.
  uint32_t key[M];
  const int b0 = 64 * M * w + lane;
#pragma unroll
  for (int m = 0; m < M; m++) key[m] = __float_as_uint(in[max(min(b0 + 64 * m, nb - 1), 0)]);
  uint32_t big = 0, small = 0;
#pragma unroll
  for (int m = 0; m < M; m++) {
    const int b = b0 + 64 * m;
    uint32_t u = key[m];
    const bool nan = (u & 0x7FFFFFFFu) > 0x7F800000u, none = u == 0xFF800000u || b < first1 || b >= last0;
    if (u == 0x80000000u) u = 0;
    u = (int)u < 0 ? ~u : u | 0x80000000u;
    key[m] = none ? 0u : nan ? 0xFFFFFFFFu : u;
    big = max(big, key[m]);
    small = max(small, 0u - key[m]);                    // (the least but 0, turned over)
  }
  auto above = [&](uint32_t t) {
    uint32_t c = 0;
#pragma unroll
    for (int m = 0; m < M; m++) c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[m] > t));
    return (int)all_waves(c, plus, 0u, &before);
  };
  // count(key > lo) > want > count(key > hi); t and need: what the search ends with
  int flo = above(0), fhi = 0, need = 0;
  uint32_t t = want > 0 ? 0u : 0xFFFFFFFFu;
  if (want > 0 && flo > want) {
    uint32_t hi = all_waves(wave_top(big), top, 0u, &before);
    uint32_t lo = 0u - all_waves(wave_top(small), top, 0u, &before) - 1;
    for (int trial = 0;; trial++) {
      const uint32_t width = hi - lo;
      if (width == 1) {
        t = hi;
        need = want - fhi;
        break;
      }
      uint32_t off = width >> 1;                        // (a float's 24 bits of the range: any trial between the ends will do)
      if (trial % 5 != 4) off = (uint32_t)((float)width * ((float)(flo - want) * __builtin_amdgcn_rcpf((float)(flo - fhi))));
      const uint32_t mid = __builtin_amdgcn_readfirstlane(lo + min(max(off, 1u), width - 1));
      const int f = above(mid);
      if (f == want) {
        t = mid;
        break;
      }
      uint32_t to = mid;
      if (trial >= 4) {                                 // the next key that there is: equal keys end the search then
        const uint32_t turned = f > want ? 0xFFFFFFFFu : 0u, most = f > want ? ~mid - 1 : mid;
        uint32_t y = 0;
#pragma unroll
        for (int m = 0; m < M; m++) {
          const uint32_t k = key[m] ^ turned;
          y = max(y, k <= most ? k : 0u);
        }
        y = all_waves(wave_top(y), top, 0u, &before);
        to = f > want ? ~y - 1 : y;
      }
      if (f > want) {
        lo = to;
        flo = f;
      } else {
        hi = to;
        fhi = f;
      }
    }
  }
  // Of the equal ones the first `need`, then the places of what is taken.
  const auto low = [&](uint64_t mask) { return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0)); };
  uint64_t take[M];
  int seen = 0, mine = 0;
  if (need > 0) {                                       // equal ones in the waves ahead
    uint32_t c = 0;
#pragma unroll
    for (int m = 0; m < M; m++) c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[m] == t));
    all_waves(c, plus, 0u, &before);
    seen = (int)before;
  }
#pragma unroll
  for (int m = 0; m < M; m++) {
    const int b = b0 + 64 * m;
    bool on = key[m] > t || (b < nb && (b < first1 || b >= last0));
    if (need > 0) {
      const uint64_t same = __builtin_amdgcn_ballot_w64(key[m] == t);
      on = on || (key[m] == t && seen + low(same) < need);
      seen += __builtin_popcountll(same);
    }
    take[m] = __builtin_amdgcn_ballot_w64(on);
    mine += __builtin_popcountll(take[m]);
  }
  const int total = (int)all_waves((uint32_t)mine, plus, 0u, &before);
  int pos = (int)before;
#pragma unroll
  for (int m = 0; m < M; m++) {
    if ((take[m] >> lane) & 1) out[pos + low(take[m])] = b0 + 64 * m;
    pos += __builtin_popcountll(take[m]);
  }
  for (int y = total + 64 * w + lane; y < A.n_sel; y += 64 * W) out[y] = -1;
}

// ------------------------------------------------------------------ host
bool touch(const void* a, int64_t an, const void* b, int64_t bn) {
  return a && b && (uintptr_t)a < (uintptr_t)b + bn && (uintptr_t)b < (uintptr_t)a + an;
}
bool long_ok(const stq_kv_desc* d, const stq_attend_desc* a) { return attend_ok(d, a) && a->window == 0 && a->n_sink == 0; }
uint64_t bounds_size(const stq_kv_desc* d) { return (uint64_t)d->n_blocks * d->n_kv_heads * 2 * d->d; }

void fill(AttnArgs& A, const stq_kv_desc* d, const void* cache, const stq_attend_desc* a, const int32_t* table,
          const int32_t* tok_start, const int32_t* len, const void* q, void* o, const Split& sp) {
  A.cache = (const uint8_t*)cache; A.table = table; A.tok_start = tok_start; A.len = len; A.q = q; A.o = o;
  A.po = A.pml = nullptr;
  A.n_req = a->n_req; A.n_tok = a->n_tok; A.hq = a->n_heads; A.hkv = d->n_kv_heads; A.group = a->n_heads / d->n_kv_heads;
  A.T = d->block_tokens; A.n_blocks = d->n_blocks; A.cols = a->table_cols; A.max_new = a->max_new;
  A.window = A.sink = 0;
  A.splits = sp.splits; A.per = sp.per; A.tiles = sp.tiles;
  A.by_hkv = div_of(A.hkv); A.by_group = div_of(A.group); A.by_max_new = div_of(A.max_new); A.by_per = div_of(A.per);
  A.qs = a->q_stride; A.os = a->o_stride;
  A.scale = a->scale;
}

// Work of the blocks' attention: by what a whole list holds.  Few workgroups are
// split into parts of 8 chunks (one request, 32 blocks of 64 tokens, 8 heads: 9.8 us
// on the GPU, 11 in parts of 12 and more, 10.3 of 4).  Where cut() gives sixteen waves,
// they spare the second launch: parts against sixteen waves, us a call and (on the
// GPU), blocks of 64 tokens, 8 heads, d = 128: one request, 12 blocks 12.9 (8.8), 9.8
// (9.4); 17 12.8 (9.0), 10.0 (10.7); 8 requests, 17 12.6 (10.1), 10.4 (10.5); 16
// requests, 12 12.6 (11.8), 9.9 (10.7); 32 14.6 (15.1), 13.6 (14.8); 32 requests, 12 13.4
// (13.7), 11.1 (11.3); 32 20.2 (20.4), 16.4 (17.0).  (In parts on both sides of
// that: one request, 8 blocks 12.8, 18 12.7; 32 requests, 33 blocks 20.0.)
// From 2,048 (token, head) pairs on each has one wave, which needs no join through LDS
// and starts once instead of four times: 16 blocks of 64 tokens at d = 128, prompts of
// 256 tokens 35.2 us by four waves, 35.5 by one; 512 63.3, 58.6; 1,024 120.7, 105.1 (64
// blocks 383, 388; 4 blocks 56, 36); 256 requests of one token 58.6, 55.4; but 128
// tokens 21.2, 25.9.
constexpr int64_t FEW_LISTED = 8;
Split blocks_split(const stq_kv_desc* d, const stq_attend_desc* a, int n_sel) {
  Split s;
  const int64_t rows = a->n_heads / d->n_kv_heads;
  s.staged = s.once = false;
  s.tile_rows = rows > 16 ? 32 : 16;
  s.tiles = (int)((rows + s.tile_rows - 1) / s.tile_rows);
  const int64_t base = (int64_t)a->n_req * a->max_new * d->n_kv_heads * s.tiles;
  cut(&s, base, (int64_t)n_sel * d->block_tokens / 32, FEW_LISTED);
  // (a wave on its own writes no parts: of so many workgroups none is split)
  static_assert(FEW_GROUPS <= MANY_GROUPS, "cut() splits none of MANY_GROUPS workgroups");
  if (s.tile_rows == 16 && base >= MANY_GROUPS) s.waves = 1;
  return s;
}

// Parts of the requests' own tokens, and room for those of the shared prefixes:
// sized on the device by what the groups have to do (Whole::part), from `per`
// chunks up and at most `slots` of them.
struct Shares { Split own; bool staged, both; int tile_rows, slots, per; int64_t pre_units; };
constexpr int64_t MOST_PARTS = 64, PRE_GROUPS = 512;   // (the join holds 128 parts' statistics in its lanes)
Shares shares_of(const stq_kv_desc* d, const stq_attend_desc* a, const stq_shared_desc* g) {
  Shares s;
  const int64_t group = a->n_heads / d->n_kv_heads, rows = (int64_t)a->max_new * group;
  s.own.once = false;
  s.own.staged = rows > STAGED_ROWS;
  s.own.tile_rows = s.own.staged ? 32 * TILE_WAVES : rows > 16 ? 32 : 16;
  s.own.tiles = (int)((rows + s.own.tile_rows - 1) / s.own.tile_rows);
  // (four waves at any length: the prefixes' parts are joined in a second launch anyhow.  Split in parts against
  // whole, us on the GPU, 8 heads, d = 128, behind 2,048 tokens: 4 requests of up to 1,000 own tokens 13.3, 15.7; 16 of 800
  // 16.5, 17.0, of 1,200 19.1, 18.5, of 2,000 21.6, 22.4; 32 of 2,000 23.2, 25.8; 16 of 1,500 behind 8,192 23.5, 25.4)
  cut(&s.own, (int64_t)a->n_req * d->n_kv_heads * s.own.tiles, ((int64_t)a->max_len + 31) / 32, FEW_CHUNKS, false);
  if (s.own.splits > MOST_PARTS) {
    const int64_t chunks = (int64_t)s.own.per * s.own.splits;
    s.own.per = (int)(((chunks + MOST_PARTS - 1) / MOST_PARTS + 3) & ~3ll);
    s.own.splits = (int)((chunks + s.own.per - 1) / s.own.per);
  }
  const int64_t all = (int64_t)a->n_tok * group;        // rows of all groups, and of one on average
  s.staged = g->n_groups > 0 && (s.own.staged || all / g->n_groups > STAGED_ROWS);
  // The requests' own tokens, few rows each, in the same launch as the staged prefixes:
  // 60 requests behind prefixes of 8,192 and 4,416 tokens 46 us in two, 38 in one; 64 behind
  // one of 8,192 44, 37; 128 59, 58; 619 query tokens behind four of 11,648 to 16,384 280, 262.
  s.both = s.staged && s.own.tile_rows == 16;
  s.tile_rows = s.staged ? 32 * TILE_WAVES : s.own.tile_rows;
  const int64_t tiles = (all + s.tile_rows - 1) / s.tile_rows, fill = (PRE_GROUPS + d->n_kv_heads - 1) / d->n_kv_heads;
  s.pre_units = g->n_groups > 0 ? fill + tiles + g->n_groups : 0;
  // (prefix kernel and join of 64 requests behind 2,048 tokens: parts of 8 chunks 23 us, of 12 24, of 16 26;
  // behind 8,192 34, 34, 32; 98 in four groups behind 5,184 to 8,192 48, 40, 39)
  s.per = 12;
  const int64_t chunks = (int64_t)g->max_prefix / 32 + 1;
  int64_t slots = 2 * fill / (tiles > 0 ? tiles : 1) + 1;
  if (slots > (chunks + s.per - 1) / s.per) slots = (chunks + s.per - 1) / s.per;
  const int64_t room = s.own.splits < 32 ? 32 - s.own.splits : MOST_PARTS;       // (the join asks for 32 parts at once)
  s.slots = (int)(slots > room ? room : slots);
  return s;
}

template <int D, int TYPE>
void launch_blocks(const LongArgs& A, const Split& s, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)A.n_req * A.max_new * A.hkv), (unsigned)A.tiles, (unsigned)A.splits);
  if (s.waves == 1) hipLaunchKernelGGL((k_attend_rows<D, TYPE, 1, 1, false, LIST>), grid, dim3(64), 0, st, A);
  else if (s.tile_rows == 32) hipLaunchKernelGGL((k_attend_rows<D, TYPE, 2, 4, false, LIST>), grid, dim3(256), 0, st, A);
  else if (s.waves == 16) hipLaunchKernelGGL((k_attend_rows<D, TYPE, 1, 16, false, LIST>), grid, dim3(1024), 0, st, A);
  else hipLaunchKernelGGL((k_attend_rows<D, TYPE, 1, 4, false, LIST>), grid, dim3(256), 0, st, A);
  if (A.splits > 1) {
    const dim3 rows((unsigned)(A.n_req * A.max_new), (unsigned)((A.hq + 3) / 4));
    hipLaunchKernelGGL((k_attend_join<D, TYPE, LIST>), rows, dim3(256), 0, st, A, 0);
  }
}

template <int D, int TYPE>
void launch_shared(LongArgs& A, const Shares& s, hipStream_t st) {
  if (s.staged) {
    A.pre_blocks = (int)(s.pre_units * A.hkv);
    const int64_t more = s.both ? (int64_t)A.n_req * A.hkv * A.splits : 0;
    hipLaunchKernelGGL((k_attend_tiles<D, TYPE, PREFIX>), dim3((unsigned)(A.pre_blocks + more)), dim3(64 * TILE_WAVES), 0, st, A);
  }
  if (s.own.staged) {
    const unsigned grid = (unsigned)((int64_t)A.n_req * A.hkv * A.tiles * A.splits);
    hipLaunchKernelGGL((k_attend_tiles<D, TYPE, SUFFIX>), dim3(grid), dim3(64 * TILE_WAVES), 0, st, A);
  } else if (!s.both) {                                 // and prefixes of few rows, in one launch
    A.pre_units = s.staged ? 0 : (int)s.pre_units;
    const dim3 grid((unsigned)((A.n_req + A.pre_units) * A.hkv), (unsigned)A.tiles, (unsigned)A.splits);
    if (s.own.tile_rows == 32) hipLaunchKernelGGL((k_attend_rows<D, TYPE, 2, 4, false, SUFFIX>), grid, dim3(256), 0, st, A);
    else hipLaunchKernelGGL((k_attend_rows<D, TYPE, 1, 4, false, SUFFIX>), grid, dim3(256), 0, st, A);
  }
  if (A.n_groups > 0 || A.splits > 1) {
    const dim3 rows((unsigned)(A.n_req * A.max_new), (unsigned)((A.hq + 3) / 4));
    hipLaunchKernelGGL((k_attend_join<D, TYPE, SUFFIX>), rows, dim3(256), 0, st, A, __builtin_ctz(s.own.tile_rows));
  }
}

// Sixteen tokens a product from 16 new tokens on (k_kv_score_wide: below, its columns
// would be tokens that are not there), else a token's heads side by side.
struct Scores { bool wide; int ht, tt, shift; int64_t ys, z; };
Scores scores_of(const AttnArgs& A, int max_len, int* tile_run) {
  Scores s;
  s.shift = 0;
  while (s.shift < 4 && (1 << s.shift) < A.group) s.shift++;
  s.wide = A.max_new >= 16;
  s.ht = A.group >= 3 ? 4 : A.group;
  s.tt = 4 / s.ht;
  const int64_t toks = s.wide ? 64 * s.tt : 16 >> s.shift;            // tokens of a workgroup
  s.ys = (A.max_new + toks - 1) / toks;
  int64_t cols = ((int64_t)max_len + A.T - 1) / A.T;
  if (cols > A.cols) cols = A.cols;
  const int64_t tiles = (cols + 15) / 16, groups = (int64_t)A.n_req * A.hkv * s.ys;
  // (as many waves as the card holds: two workgroups a CU there, four waves a SIMD here)
  int64_t run = s.wide ? tiles * groups / 512 : tiles * groups / 4096;
  *tile_run = (int)(run < 1 ? 1 : run > 8 && !s.wide ? 8 : run > tiles ? tiles : run);
  const int64_t per = s.wide ? *tile_run : 4 * *tile_run;
  s.z = (tiles + per - 1) / per;
  if (s.z > 65535) s.z = 65535;                                        // (the kernels go round)
  return s;
}
template <int D, int TYPE>
void launch_score(const ScoreArgs& A, const Scores& s, hipStream_t st) {
  const dim3 grid((unsigned)(A.n_req * A.hkv), (unsigned)s.ys, (unsigned)s.z);
  if (!s.wide) hipLaunchKernelGGL((k_kv_score<D, TYPE>), grid, dim3(256), 0, st, A);
  else if (s.ht == 4) hipLaunchKernelGGL((k_kv_score_wide<D, TYPE, 4, 1>), grid, dim3(256), 0, st, A);
  else if (s.ht == 2) hipLaunchKernelGGL((k_kv_score_wide<D, TYPE, 2, 2>), grid, dim3(256), 0, st, A);
  else hipLaunchKernelGGL((k_kv_score_wide<D, TYPE, 1, 4>), grid, dim3(256), 0, st, A);
}

}  // namespace

extern "C" {

size_t stq_kv_bounds_bytes(const stq_kv_desc* d) { return kv_ok(d) ? (size_t)bounds_size(d) : 0; }

stq_status stq_kv_bounds(const stq_kv_desc* d, const void* cache, size_t bytes, int32_t n_req, int32_t max_new,
                         const int32_t* table, int32_t table_cols, const int32_t* tok_start, const int32_t* len,
                         void* bounds, hipStream_t st) {
  const stq_status s = kv_check(d, cache, bytes);
  if (s != STQ_OK) return s;
  if (n_req < 0 || max_new < 1 || table_cols < 1 || (int64_t)table_cols * d->block_tokens > (1ll << 30)) return STQ_ERR_ARG;
  if (n_req == 0) return STQ_OK;
  if (!table || !tok_start || !len || !bounds) return STQ_ERR_ARG;
  if (!aligned(bounds)) return STQ_ERR_LAYOUT;
  if (touch(bounds, (int64_t)bounds_size(d), cache, (int64_t)kv_size(d))) return STQ_ERR_ARG;
  BoundsArgs A;
  A.cache = (const uint8_t*)cache; A.table = table; A.tok_start = tok_start; A.len = len; A.bounds = (uint8_t*)bounds;
  A.n_req = n_req; A.hkv = d->n_kv_heads; A.T = d->block_tokens; A.n_blocks = d->n_blocks; A.cols = table_cols; A.max_new = max_new;
  const int64_t span = ((int64_t)max_new - 1) / d->block_tokens + 2;       // blocks that so many tokens touch at most
  A.span = (int)(span < table_cols ? span : table_cols);
  A.by_span = div_of(A.span);
  if ((int64_t)n_req * A.span * 256 > MOST_THREADS) return STQ_ERR_UNSUPPORTED;
  const dim3 g((unsigned)(n_req * A.span), (unsigned)((A.hkv + 3) / 4)), b(256);
  if (d->d == 64) hipLaunchKernelGGL((k_kv_bounds<64>), g, b, 0, st, A);
  else hipLaunchKernelGGL((k_kv_bounds<128>), g, b, 0, st, A);
  return launched();
}

stq_status stq_kv_score(const stq_kv_desc* d, const stq_attend_desc* a, const void* bounds, const int32_t* table,
                        const int32_t* tok_start, const int32_t* len, const void* q, float* score, hipStream_t st) {
  if (!kv_ok(d) || !long_ok(d, a)) return STQ_ERR_ARG;
  if (a->n_req == 0 || a->n_tok == 0) return STQ_OK;
  if (!bounds || !table || !tok_start || !len || !q || !score) return STQ_ERR_ARG;
  const int64_t w = (int64_t)a->n_heads * d->d;
  if (!aligned(bounds) || !aligned(q) || !aligned(score) || !stride_ok(a->q_stride, w, a->type)) return STQ_ERR_LAYOUT;
  const int64_t out = (int64_t)a->n_tok * d->n_kv_heads * a->table_cols * 4;
  if (touch(score, out, bounds, (int64_t)bounds_size(d)) || touch(score, out, q, ((a->n_tok - 1) * a->q_stride + w) * 2)) return STQ_ERR_ARG;
  Split none;
  none.splits = none.per = none.tiles = 1;
  ScoreArgs A;
  fill(A, d, nullptr, a, table, tok_start, len, q, nullptr, none);
  A.bounds = (const uint8_t*)bounds; A.score = score;
  const Scores sc = scores_of(A, a->max_len, &A.tile_run);
  A.rows_shift = sc.shift;
  if ((int64_t)a->n_req * A.hkv * 256 > MOST_THREADS || sc.ys > 65535) return STQ_ERR_UNSUPPORTED;
  if (d->d == 64) {
    if (a->type == STQ_BF16) launch_score<64, STQ_BF16>(A, sc, st);
    else launch_score<64, STQ_FP16>(A, sc, st);
  } else {
    if (a->type == STQ_BF16) launch_score<128, STQ_BF16>(A, sc, st);
    else launch_score<128, STQ_FP16>(A, sc, st);
  }
  return launched();
}

stq_status stq_kv_select(const stq_select_desc* c, const int32_t* tok_start, const int32_t* len, const float* score,
                         int32_t* sel, hipStream_t st) {
  if (!c || c->n_req < 0 || c->n_tok < 0 || c->n_tok > (1 << 28) || c->n_kv_heads < 1 || c->n_kv_heads > 4096) return STQ_ERR_ARG;
  if (c->block_tokens != 32 && c->block_tokens != 64 && c->block_tokens != 128 && c->block_tokens != 256) return STQ_ERR_ARG;
  if (c->table_cols < 1 || (int64_t)c->table_cols * c->block_tokens > (1ll << 30) || c->max_new < 1) return STQ_ERR_ARG;
  if (c->n_sel < 1 || c->n_first < 0 || c->n_last < 0 || (int64_t)c->n_first + c->n_last > c->n_sel) return STQ_ERR_ARG;
  if (c->table_cols > 32768) return STQ_ERR_UNSUPPORTED;
  if (c->n_req == 0 || c->n_tok == 0) return STQ_OK;
  if (!tok_start || !len || !score || !sel) return STQ_ERR_ARG;
  if (!aligned(score) || !aligned(sel)) return STQ_ERR_LAYOUT;
  const int64_t rows = (int64_t)c->n_tok * c->n_kv_heads;
  if (touch(sel, rows * c->n_sel * 4, score, rows * c->table_cols * 4)) return STQ_ERR_ARG;
  SelectArgs A;
  A.score = score; A.tok_start = tok_start; A.len = len; A.sel = sel;
  A.n_req = c->n_req; A.n_tok = c->n_tok; A.hkv = c->n_kv_heads; A.T = c->block_tokens; A.cols = c->table_cols;
  A.n_sel = c->n_sel; A.n_first = c->n_first; A.n_last = c->n_last; A.max_new = c->max_new;
  A.by_hkv = div_of(A.hkv); A.by_max_new = div_of(A.max_new);
  const int64_t units = (int64_t)c->n_req * c->max_new * c->n_kv_heads;
  const int64_t groups = A.cols <= 2048 ? (units + 3) / 4 : units;    // four rows a workgroup, or one
  if (units > INT32_MAX || groups * (A.cols <= 2048 ? 256 : 1024) > MOST_THREADS) return STQ_ERR_UNSUPPORTED;
  const dim3 g((unsigned)groups);
  if (A.cols <= 64) hipLaunchKernelGGL((k_kv_select<1, 1>), g, dim3(256), 0, st, A);
  else if (A.cols <= 256) hipLaunchKernelGGL((k_kv_select<1, 4>), g, dim3(256), 0, st, A);
  else if (A.cols <= 512) hipLaunchKernelGGL((k_kv_select<1, 8>), g, dim3(256), 0, st, A);
  else if (A.cols <= 2048) hipLaunchKernelGGL((k_kv_select<1, 32>), g, dim3(256), 0, st, A);
  else if (A.cols <= 8192) hipLaunchKernelGGL((k_kv_select<16, 8>), g, dim3(1024), 0, st, A);
  else hipLaunchKernelGGL((k_kv_select<16, 32>), g, dim3(1024), 0, st, A);
  return launched();
}

size_t stq_kv_attend_blocks_bytes(const stq_kv_desc* d, const stq_attend_desc* a, int32_t n_sel) {
  if (!kv_ok(d) || !long_ok(d, a) || n_sel < 1 || (int64_t)n_sel * d->block_tokens > (1ll << 30)) return 0;
  const Split s = blocks_split(d, a, n_sel);
  return s.splits <= 1 ? 0 : (size_t)s.splits * a->n_tok * a->n_heads * (d->d + 2) * 4;
}

stq_status stq_kv_attend_blocks(const stq_kv_desc* d, const void* cache, size_t bytes, const stq_attend_desc* a,
                                int32_t n_sel, const int32_t* table, const int32_t* tok_start, const int32_t* len,
                                const int32_t* sel, const void* q, void* o, void* work, size_t work_bytes, hipStream_t st) {
  const stq_status s = kv_check(d, cache, bytes);
  if (s != STQ_OK) return s;
  if (!long_ok(d, a) || n_sel < 1 || (int64_t)n_sel * d->block_tokens > (1ll << 30)) return STQ_ERR_ARG;
  if (a->n_req == 0 || a->n_tok == 0) return STQ_OK;
  if (!table || !tok_start || !len || !sel || !q || !o) return STQ_ERR_ARG;
  const int64_t w = (int64_t)a->n_heads * d->d;
  if (!aligned(sel) || !aligned(q) || !aligned(o) || !stride_ok(a->q_stride, w, a->type) || !stride_ok(a->o_stride, w, a->type))
    return STQ_ERR_LAYOUT;
  const Rows rq = {q, a->q_stride * 2, w * 2}, ro = {o, a->o_stride * 2, w * 2};
  if (!same(rq, ro) && meet(rq, ro, a->n_tok)) return STQ_ERR_ARG;
  if (touch(o, ((a->n_tok - 1) * a->o_stride + w) * 2, sel, (int64_t)a->n_tok * d->n_kv_heads * n_sel * 4)) return STQ_ERR_ARG;
  const Split sp = blocks_split(d, a, n_sel);
  const size_t need = stq_kv_attend_blocks_bytes(d, a, n_sel);
  if (need > 0 && (!work || !aligned(work) || work_bytes < need)) return STQ_ERR_LAYOUT;
  const int64_t units = (int64_t)a->n_req * a->max_new;
  if (units * a->n_heads > INT32_MAX || units * d->n_kv_heads * 64 * sp.waves > MOST_THREADS || (sp.splits > 1 && units * 256 > MOST_THREADS))
    return STQ_ERR_UNSUPPORTED;
  LongArgs A;
  fill(A, d, cache, a, table, tok_start, len, q, o, sp);
  A.sel = sel; A.n_sel = n_sel;
  A.group_start = A.prefix = nullptr; A.shared = nullptr;
  A.n_groups = A.pre_per = A.slot0 = A.pre_units = A.pre_blocks = 0;
  A.pre_fill = 0;
  A.po = (float*)work;
  A.pml = A.po + (int64_t)sp.splits * a->n_tok * a->n_heads * d->d;
  if (d->d == 64) {
    if (a->type == STQ_BF16) launch_blocks<64, STQ_BF16>(A, sp, st);
    else launch_blocks<64, STQ_FP16>(A, sp, st);
  } else {
    if (a->type == STQ_BF16) launch_blocks<128, STQ_BF16>(A, sp, st);
    else launch_blocks<128, STQ_FP16>(A, sp, st);
  }
  return launched();
}

size_t stq_kv_attend_shared_bytes(const stq_kv_desc* d, const stq_attend_desc* a, const stq_shared_desc* g) {
  if (!kv_ok(d) || !long_ok(d, a) || !g || g->n_groups < 0 || g->max_prefix < 0) return 0;
  const Shares s = shares_of(d, a, g);
  return (size_t)(s.own.splits + s.slots) * a->n_tok * a->n_heads * (d->d + 2) * 4 + ((size_t)a->n_req * 4 + 19) / 16 * 16;
}

stq_status stq_kv_attend_shared(const stq_kv_desc* d, const void* cache, size_t bytes, const stq_attend_desc* a,
                                const stq_shared_desc* g, const int32_t* table, const int32_t* tok_start, const int32_t* len,
                                const int32_t* group_start, const int32_t* prefix, const void* q, void* o, void* work,
                                size_t work_bytes, hipStream_t st) {
  const stq_status s = kv_check(d, cache, bytes);
  if (s != STQ_OK) return s;
  if (!long_ok(d, a) || !g || g->n_groups < 0 || g->max_prefix < 0) return STQ_ERR_ARG;
  if (a->n_req == 0 || a->n_tok == 0) return STQ_OK;
  if (!table || !tok_start || !len || (g->n_groups > 0 && (!group_start || !prefix)) || !q || !o) return STQ_ERR_ARG;
  const int64_t w = (int64_t)a->n_heads * d->d;
  if (!aligned(q) || !aligned(o) || !stride_ok(a->q_stride, w, a->type) || !stride_ok(a->o_stride, w, a->type))
    return STQ_ERR_LAYOUT;
  const Rows rq = {q, a->q_stride * 2, w * 2}, ro = {o, a->o_stride * 2, w * 2};
  if (!same(rq, ro) && meet(rq, ro, a->n_tok)) return STQ_ERR_ARG;
  const Shares sp = shares_of(d, a, g);
  const size_t need = stq_kv_attend_shared_bytes(d, a, g);
  if (!work || !aligned(work) || work_bytes < need) return STQ_ERR_LAYOUT;
  const int64_t groups = (int64_t)a->n_req * d->n_kv_heads, pre = sp.pre_units * d->n_kv_heads;
  if ((int64_t)a->n_req * a->max_new * a->n_heads > INT32_MAX || (int64_t)a->n_tok * a->n_heads > INT32_MAX ||
      (sp.own.staged ? groups * sp.own.tiles * sp.own.splits : groups) * 256 > MOST_THREADS ||
      (groups * sp.own.splits + pre) * 256 > MOST_THREADS || (int64_t)a->n_req * a->max_new * 256 > MOST_THREADS)
    return STQ_ERR_UNSUPPORTED;
  LongArgs A;
  fill(A, d, cache, a, table, tok_start, len, q, o, sp.own);
  A.sel = nullptr; A.n_sel = 0;
  A.group_start = group_start; A.prefix = prefix;
  A.n_groups = g->n_groups; A.pre_per = sp.per; A.slot0 = sp.slots; A.pre_units = A.pre_blocks = 0;
  A.pre_fill = (int)((PRE_GROUPS + d->n_kv_heads - 1) / d->n_kv_heads);
  const int64_t rows = (int64_t)(sp.own.splits + sp.slots) * a->n_tok * a->n_heads;
  A.po = (float*)work;
  A.pml = A.po + rows * d->d;
  A.shared = (int32_t*)(A.pml + 2 * rows);
  if (d->d == 64) {
    if (a->type == STQ_BF16) launch_shared<64, STQ_BF16>(A, sp, st);
    else launch_shared<64, STQ_FP16>(A, sp, st);
  } else {
    if (a->type == STQ_BF16) launch_shared<128, STQ_BF16>(A, sp, st);
    else launch_shared<128, STQ_FP16>(A, sp, st);
  }
  return launched();
}

}  // extern "C"
