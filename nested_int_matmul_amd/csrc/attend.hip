// Attention over the 8-bit key/value cache.
//
//   t_j = scale * <q, k_j> * k_scale(page of j)   (optionally capped)
//   out = sum_j exp(t_j - m) v_scale v_j / sum_j exp(t_j - m)
//
// in one pass over the keys with a running reference m and running sums.
// Everything is kept transposed (keys x rows, then dims x rows), so that the
// probabilities leave the first product in the registers where the second
// one wants them:
//   S^T [16 keys x 16 rows] = K [16 x dim] Q^T       (A = codes of k)
//   O^T [16 dims x 16 rows] += V^T [16 x 32 keys] P^T  (A = codes of v)
// A row is one (token, query head of the group); a lane holds row lane % 16.
// The order of the keys in a contraction is free as long as both operands
// agree: with L = 16 (tiles of 64 keys) or 8 (of 32), MFMA t of a tile takes
// as its 16 rows the keys L (r / 4) + 4 t + r % 4, which leaves lane group
// g = lane / 16 with the scores of keys L g .. L g + L - 1: all of one page (a
// page is 16 tokens or more, so one k scale and one v scale a lane), and the L
// consecutive bytes that it loads of each dim of v.  No score and no code goes
// through LDS.  (So for few rows; many rows share their codes through LDS.)
//
// Codes become fp16 exactly (int8 and e4m3 both fit), q becomes fp16 after
// its row is multiplied by a power of two that brings its largest entry to
// 2^14 (entries 2^-29 of that and above keep all their bits), the products
// accumulate in fp32.  Probabilities are rounded to fp16, in units of a
// reference that stays within 2^8 of the row's maximum: off by at most
// 2^-11 of each, an eighth of the result's own rounding to bf16 (2^-8).
#include "kv_device.h"

namespace mq {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNoRef = -1e30f;  // reference of a row that has seen no key
// The reference moves only when a score exceeds it by this much (in log2):
// exp2 stays below 2^8, far from fp16's 2^16, and most tiles need no
// exchange between lanes and no rescaling.
constexpr float kSlack = 8.f;

// Eight codes to an operand of eight fp16.
template <bool E4M3>
__device__ __forceinline__ f16x8 codes_to_f16(uint32_t w0, uint32_t w1) {
  union {
    f16x2 h[4];
    f16x8 v;
  } r;
  const uint32_t w[2] = {w0, w1};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (E4M3) {
      r.h[2 * i] = __builtin_bit_cast(
          f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w[i], 1.f, false));
      r.h[2 * i + 1] = __builtin_bit_cast(
          f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w[i], 1.f, true));
    } else {
      // byte c + 128 under the fp16 exponent of 1024 is 1152 + c
      const f16x2 off = {(_Float16)1152.f, (_Float16)1152.f};
      const uint32_t u = w[i] ^ 0x80808080u;
      const uint32_t p0 = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
      const uint32_t p1 = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
      r.h[2 * i] = __builtin_bit_cast(f16x2, p0) - off;
      r.h[2 * i + 1] = __builtin_bit_cast(f16x2, p1) - off;
    }
  }
  return r.v;
}

// tanh(z) = 1 - 2 / (e^2z + 1), by its series where that cancels (cut below
// 2^-29 of it).
__device__ __forceinline__ float capped(float z) {
  const float e2 = __builtin_amdgcn_exp2f(2.f * kLog2e * fabsf(z));
  const float big = copysignf(fmaf(-2.f, __builtin_amdgcn_rcpf(e2 + 1.f), 1.f), z);
  const float zz = z * z;
  const float small = z * (1.f + zz * (-1.f / 3.f + zz * (2.f / 15.f + zz * (-17.f / 315.f))));
  return fabsf(z) < 0.125f ? small : big;
}

// Keys [lo, hi) of the token at position pos (positions are below 2^30).
struct Keys {
  int lo, hi;
};
__device__ __forceinline__ Keys keys_of(const AttendArgs& a, int64_t pos, int held) {
  Keys k;
  k.hi = a.causal && pos + 1 < held ? (int)(pos + 1) : held;
  k.lo = 0;
  if (a.window > 0 && pos - a.window + 1 > 0)
    k.lo = pos - a.window + 1 < held ? (int)(pos - a.window + 1) : held;
  if (pos < 0 || k.hi < 0) k.hi = 0;
  return k;
}

// What the rows [row_a, row_b) of a (sequence, head) see together, as pieces
// of a.part.piece tokens from a 64-aligned start.
struct Span {
  int lo, hi;  // lo a multiple of 64; lo >= hi: no key
  int pieces;
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, const SeqSpan& sp, int held,
                                        int tok_a, int tok_b) {
  Span r;
  const Keys f = keys_of(a, sp.start + tok_a, held), l = keys_of(a, sp.start + tok_b, held);
  r.lo = f.lo & ~63;
  r.hi = l.hi;
  r.pieces = r.hi > r.lo ? (r.hi - r.lo + a.part.piece - 1) / a.part.piece : 0;
  return r;
}
// row / group: rows are below 2^26 and groups at most 2^10, so a product with
// ceil(2^36 / group) is off by less than 1 / group of a unit.
__device__ __forceinline__ int token_of(const AttendArgs& a, int row) {
  return (int)(((uint64_t)(uint32_t)row * a.group_mul) >> 36);
}
// Where a row's partial results are within a piece's: few rows of a sequence
// and head lie together (a batch may have many more rows than those), many
// rows as in the output.
__device__ __forceinline__ int64_t part_row(const AttendArgs& a, int s, int kvh, int row,
                                            int64_t out_row) {
  return a.part.tile <= 32 ? ((int64_t)s * a.cache.heads + kvh) * a.part.tile + row : out_row;
}
// (blockIdx.y + blockIdx.z) % pieces.  Workgroups are dealt to the parts of the
// chip in turn, those that find nothing too: were every sequence's first piece
// the first of a multiple of four, one part would get the pieces that all
// sequences have and another those that few have (32 sequences of up to 16384
// tokens in 16 pieces each: 102.3 us, turned 99.6; with the pieces outermost
// 127).
__device__ __forceinline__ int turned_piece(const AttendPart& p) {
  const uint32_t z = blockIdx.z;
  const int i = (int)(blockIdx.y + (z - p.pieces * (uint32_t)(((uint64_t)z * p.turn) >> 31)));
  return i < p.pieces ? i : i - p.pieces;
}
__device__ __forceinline__ int held_of(const AttendArgs& a, int s) {
  const int len = a.batch.kv_len[s];
  const int room = a.batch.table_pages * a.cache.block;
  return len < room ? len : room;
}

}  // namespace

// ------------------------------------------------------------- few rows
//
// ROWS * 16 rows a workgroup, NW waves that share them and take the piece's
// tiles in turn, each with sums of its own, joined through LDS at the end;
// pieces are joined by join_kernel.  Bound by the codes' bytes: 464 MB of 32
// sequences in 96 us with the join (4.8 TB/s, nearly the rate of a large
// copy), one sequence of 131072 tokens (268 MB) in 56 us.  Short spans are
// bound by the way of a piece: lengths, table, codes, two products, the join
// (one token over 700: 7 us, and 3 for the join).
//   few_waves: waves of a SIMD that the registers are cut for (k and v of a
// tile, the outputs, the queries).
constexpr int few_waves(int dim, int rows, int kt) {
  return dim * (rows + kt / 32) <= 256 ? 3 : dim * (rows + kt / 32) <= 512 ? 2 : 1;
}

template <int DIM, int ROWS, int KT, int NW, bool E4M3, bool CAP>
__global__ void __launch_bounds__(NW * 64)
    __attribute__((amdgpu_waves_per_eu(few_waves(DIM, ROWS, KT)))) attend_few_kernel(AttendArgs a) {
  constexpr int C = DIM / 64;   // 64-dim chunks of a key
  constexpr int DT = DIM / 16;  // 16-dim tiles of the output
  constexpr int NT = KT / 16;   // 16-key products of a tile
  constexpr int KL = KT / 4;    // consecutive keys of a lane: 16 or 8
  __shared__ float lds_o[NW][16][DIM + 4];
  __shared__ float lds_ml[NW][ROWS * 16][2];

  const int s = blockIdx.z;
  const int kvh = blockIdx.x;
  const int piece = turned_piece(a.part);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r16 = lane & 15;

  // The pages are known one tile ahead of the codes, and a tile's codes are
  // loaded as soon as the registers of the one before are free: k's after the
  // first product, v's after the second.  Table entries are loaded without
  // waiting for the lengths (without a window a piece's first key does not
  // depend on them) and judged when both are there.
  const int block = a.cache.block;
  const int shift = __builtin_ctz(block);
  const int* const table = a.batch.page_table + (int64_t)s * a.batch.table_pages;
  // table entries of the 16 keys whose k this lane loads, and of its scores and v
  int pk = -1, pv = -1;
  auto pages = [&](int key0) {
    const int ik = (key0 + KL * (r16 >> 2)) >> shift, iv = (key0 + KL * g) >> shift;
    pk = ik < a.batch.table_pages ? table[ik] : -1;
    pv = iv < a.batch.table_pages ? table[iv] : -1;
  };
  if (a.window == 0) pages(piece * a.part.piece + KT * wave);

  const SeqSpan sp = seq_span(a.batch, s);
  const int rows = sp.n * a.group;  // rows of this sequence and head
  if (rows <= a.part.over || rows > a.part.upto) return;
  const int held = held_of(a, s);
  const Span span = span_of(a, sp, held, 0, token_of(a, rows - 1));
  if (piece > 0 && piece >= span.pieces) return;

  const int begin = span.lo + piece * a.part.piece;
  const int stop = begin + a.part.piece < span.hi ? begin + a.part.piece : span.hi;
  const int head_bytes = block * DIM;
  const int64_t page_bytes = (int64_t)head_bytes * a.cache.heads;
  const uint8_t* const kbase = a.cache.k + (int64_t)kvh * head_bytes + (r16 & 3) * DIM + 16 * g;
  const uint8_t* const vbase = a.cache.v + (int64_t)kvh * head_bytes + r16 * block;
  u32x4 kc[NT][C];
  uint32_t vc[DT][KL / 4];
  float ks, vs;
  // entries of keys beyond the piece, or outside the pool, are no pages
  auto judge = [&](int key0) {
    if (key0 + KL * (r16 >> 2) >= stop || pk >= a.cache.pages) pk = -1;
    if (key0 + KL * g >= stop || pv >= a.cache.pages) pv = -1;
  };
  auto load_k = [&](int key0) {
    const uint8_t* p = kbase + (pk < 0 ? 0 : pk) * page_bytes +
                       ((key0 + KL * (r16 >> 2)) & (block - 1)) * DIM;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < C; ++c)
        kc[t][c] = *reinterpret_cast<const u32x4*>(p + 4 * t * DIM + 64 * c);
    ks = a.cache.k_scale[(int64_t)(pv < 0 ? 0 : pv) * a.cache.heads + kvh];
  };
  auto load_v = [&](int key0) {
    const uint8_t* p = vbase + (pv < 0 ? 0 : pv) * page_bytes + ((key0 + KL * g) & (block - 1));
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      if (KL == 16) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p + 16 * d * block);
        vc[d][0] = w[0], vc[d][1] = w[1], vc[d][KL / 4 - 2] = w[2], vc[d][KL / 4 - 1] = w[3];
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p + 16 * d * block);
        vc[d][0] = w[0], vc[d][1] = w[1];
      }
    }
    vs = a.cache.v_scale[(int64_t)(pv < 0 ? 0 : pv) * a.cache.heads + kvh];
  };
  const int first_key = begin + KT * wave;
  if (first_key < stop) {
    if (a.window != 0) pages(first_key);
    judge(first_key);
    load_k(first_key);
    load_v(first_key);
  }

  // ---- this lane's rows: the queries as fp16, and the keys they see
  f16x8 q[ROWS][C][2];
  float qf[ROWS];
  int see_lo[ROWS], see_hi[ROWS];
#pragma unroll
  for (int rt = 0; rt < ROWS; ++rt) {
    const int row = rt * 16 + r16;
    const bool real = row < rows;
    const int tok = real ? token_of(a, row) : 0;
    const int head = kvh * a.group + (real ? row - tok * a.group : 0);
    const uint16_t* qp = a.q + (int64_t)(sp.row0 + tok) * a.q_stride + (int64_t)head * DIM;
    u32x4 raw[C][2];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        raw[c][h] = real ? *reinterpret_cast<const u32x4*>(qp + 64 * c + 16 * g + 8 * h)
                         : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = raw[c][h][e] & 0x7fffu, y = (raw[c][h][e] >> 16) & 0x7fffu;
          top = x > top ? x : top;
          top = y > top ? y : top;
        }
      }
    uint32_t o = __shfl_xor(top, 16);
    top = o > top ? o : top;
    o = __shfl_xor(top, 32);
    top = o > top ? o : top;
    int e = (int)(top >> 7) - 127;       // exponent of the row's largest entry
    e = e < -100 ? -100 : (e > 127 ? 14 : e);  // (no scaling of rows with inf or NaN)
    const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
    qf[rt] = __uint_as_float((uint32_t)(e - 14 + 127) << 23) * a.scale;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t pair = raw[c][h][j >> 1];
          const float x = __uint_as_float((j & 1) ? pair & 0xffff0000u : pair << 16);
          q[rt][c][h][j] = (_Float16)(x * up);
        }
    const Keys k = keys_of(a, sp.start + tok, held);
    see_lo[rt] = k.lo;
    see_hi[rt] = real ? k.hi : 0;
  }
  // keys that every real row sees: no mask needed there
  const Keys first = keys_of(a, sp.start, held);
  const Keys last = keys_of(a, sp.start + token_of(a, rows - 1), held);

  f32x4 acc[ROWS][DT];
  float ref[ROWS], sum[ROWS];
#pragma unroll
  for (int rt = 0; rt < ROWS; ++rt) {
    ref[rt] = kNoRef;
    sum[rt] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[rt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  float vref = 0.f, vinv = 0.f;  // unit of the v scales in acc

  const float icap = CAP ? 1.f / a.softcap : 0.f;
  for (int key0 = first_key; key0 < stop; key0 += KT * NW) {
    const int kv0 = key0 + KL * g;
    const bool here = pv >= 0;
    const bool masked =
        key0 < last.lo || key0 + KT > first.hi || key0 + KT > stop || __any(!here);
    const int next = key0 + KT * NW;
    const bool more = next < stop;
    if (more) pages(next);

    // ---- scores
    f32x4 sc[ROWS][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int rt = 0; rt < ROWS; ++rt) sc[rt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      f16x8 op[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          op[t][h] = codes_to_f16<E4M3>(kc[t][c][2 * h], kc[t][c][2 * h + 1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int rt = 0; rt < ROWS; ++rt)
            sc[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(op[t][h], q[rt][c][h], sc[rt][t], 0,
                                                               0, 0);
    }
    const float ks_now = ks;
    if (more) {
      judge(next);
      load_k(next);
    }
    // ---- mask: keys beyond the sequence, and bytes there (never written)
    // must not reach the products as NaN
    int live = KL;  // of this lane's keys, those that are held
    if (masked) {
      const int n = stop - kv0;
      live = !here || n <= 0 ? 0 : (n < KL ? n : KL);
      if (live == 0) vs = 0.f;
    }
    // ---- unit of v
    if (__any(vs > vref)) {
      float m = vs;
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      m = fmaxf(m, vref);
      const float f = vref / m;
#pragma unroll
      for (int rt = 0; rt < ROWS; ++rt)
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[rt][d] = acc[rt][d] * f;
      vref = m;
      vinv = 1.f / m;
    }
    const float vw = vs * vinv;
    // ---- probabilities
    f16x8 p[ROWS][KT / 32];
#pragma unroll
    for (int rt = 0; rt < ROWS; ++rt) {
      const float f = ks_now * qf[rt] * (CAP ? icap : kLog2e);
      float x[KL];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y = sc[rt][t][i] * f;
          if (CAP) {
            y = capped(y) * (a.softcap * kLog2e);
          }
          x[4 * t + i] = y;
        }
      if (masked) {
#pragma unroll
        for (int i = 0; i < KL; ++i) {
          const int j = kv0 + i;
          if (i >= live || j < see_lo[rt] || j >= see_hi[rt]) x[i] = -INFINITY;
        }
      }
      float top = x[0];
#pragma unroll
      for (int i = 1; i < KL; ++i) top = fmaxf(top, x[i]);
      if (__any(top > ref[rt] + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m = fmaxf(top, ref[rt]);
        const float f2 = __builtin_amdgcn_exp2f(ref[rt] - m);
        ref[rt] = m;
        sum[rt] *= f2;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[rt][d] = acc[rt][d] * f2;
      }
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        const float e = __builtin_amdgcn_exp2f(x[i] - ref[rt]);
        sum[rt] += e;
        p[rt][i >> 3][i & 7] = (_Float16)(e * vw);
      }
    }
    if (masked && E4M3) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < KL / 4; ++e) {
          const int keep = live - 4 * e;
          vc[d][e] &= keep >= 4 ? 0xffffffffu : (keep <= 0 ? 0u : (1u << (8 * keep)) - 1);
        }
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int d = 0; d < DT; d += 2) {
      f16x8 op[2][KT / 32];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int h = 0; h < KT / 32; ++h)
          op[e][h] = codes_to_f16<E4M3>(vc[d + e][2 * h], vc[d + e][2 * h + 1]);
#pragma unroll
      for (int h = 0; h < KT / 32; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int rt = 0; rt < ROWS; ++rt)
            acc[rt][d + e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(op[e][h], p[rt][h],
                                                                    acc[rt][d + e], 0, 0, 0);
    }
    if (more) load_v(next);
  }

  // ---- join the waves: reference and sum of every row, then the outputs
#pragma unroll
  for (int rt = 0; rt < ROWS; ++rt) {
    sum[rt] += __shfl_xor(sum[rt], 16);
    sum[rt] += __shfl_xor(sum[rt], 32);
    if (g == 0) {
      lds_ml[wave][rt * 16 + r16][0] = ref[rt];
      lds_ml[wave][rt * 16 + r16][1] = sum[rt];
    }
  }
  __syncthreads();
  const bool direct = span.pieces <= 1;
#pragma unroll
  for (int rt = 0; rt < ROWS; ++rt) {
    float m = kNoRef, l = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, lds_ml[w][rt * 16 + r16][0]);
#pragma unroll
    for (int w = 0; w < NW; ++w)
      l += lds_ml[w][rt * 16 + r16][1] * __builtin_amdgcn_exp2f(lds_ml[w][rt * 16 + r16][0] - m);
    // (a NaN reference cannot be: fmaxf drops it; its sum is NaN)
    const float f = __builtin_amdgcn_exp2f(ref[rt] - m) * vref;
    if (rt > 0) __syncthreads();
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const f32x4 o = acc[rt][d] * f;
      *reinterpret_cast<f32x4*>(&lds_o[wave][r16][16 * d + 4 * g]) = o;
    }
    __syncthreads();
    // 16 rows x DIM outputs over NW * 64 threads, four at a time
    for (int i = threadIdx.x; i < 16 * (DIM / 4); i += NW * 64) {
      const int rr = i / (DIM / 4), d = (i % (DIM / 4)) * 4;
      const int row = rt * 16 + rr;
      if (row >= rows) continue;
      f32x4 o = *reinterpret_cast<f32x4*>(&lds_o[0][rr][d]);
#pragma unroll
      for (int w = 1; w < NW; ++w) o = o + *reinterpret_cast<f32x4*>(&lds_o[w][rr][d]);
      float mm = kNoRef, ll = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) mm = fmaxf(mm, lds_ml[w][rt * 16 + rr][0]);
#pragma unroll
      for (int w = 0; w < NW; ++w)
        ll += lds_ml[w][rt * 16 + rr][1] * __builtin_amdgcn_exp2f(lds_ml[w][rt * 16 + rr][0] - mm);
      const int tok = token_of(a, row);
      const int64_t out_row =
          (int64_t)(sp.row0 + tok) * a.q_heads + kvh * a.group + (row - tok * a.group);
      if (direct) {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        u32x2 b;
        b[0] = bf16_pair(o[0] * inv, o[1] * inv);
        b[1] = bf16_pair(o[2] * inv, o[3] * inv);
        if (ll == 0.f) b = u32x2{0, 0};
        *reinterpret_cast<u32x2*>(a.out + out_row * DIM + d) = b;
        if (a.lse && d == 0) a.lse[out_row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      } else {
        const int64_t at = piece * a.part.step + part_row(a, s, kvh, row, out_row);
        *reinterpret_cast<f32x4*>(a.part.o + at * DIM + d) = o;
        if (d == 0) {
          a.part.ml[2 * at] = mm;
          a.part.ml[2 * at + 1] = ll;
        }
      }
    }
  }
}

// ------------------------------------------------------------ many rows
//
// NW waves of 32 rows each (32x32x16 products), one 64-key tile after the
// other for all of them.  The tile's codes are converted to fp16 once for the
// workgroup and staged through LDS as operand fragments (two buffers each for
// k and v, one barrier a tile); a lane's fragment is 16 consecutive bytes, and
// fragments are permuted within groups of eight lanes (an XOR with the
// fragment's index) so that both the staging stores and the operand loads
// touch all banks evenly.  The 32 key rows of an S^T product are ordered so
// that a lane (row lane % 32, half h = lane / 32) gets keys 16 e + 8 h + 0..7
// of the tile in registers 8 e .. 8 e + 7: eight consecutive keys of one
// 16-key group, the operand of the second product as it stands.  A 16-key
// group lies in one page, so its scales are the same for all lanes.
// Two prompts of up to 2048 tokens behind up to 6144 (32 heads of 128 over 8):
// 430 us, 870 TFLOP/s; unstaged, with 64 rows a workgroup, 976.
//
// What bounds it is the vector unit beside the matrix unit: an exp2 (four
// issue slots), a multiply-add, an addition, half a maximum and half a
// conversion a score, about as long as the two products take.  So the scores
// of the next tile are computed while this tile's probabilities are (matrix
// and vector instructions of one wave in the same stretch of code), and the
// next codes are converted beside the second product.
//
// The v scale of a group goes into the exponent, p = exp2(t + log2 v_scale -
// ref), so that probabilities need no further factor; the row's sum takes
// (sum of the group's p) / v_scale.  A page of zeros (scale 0) is given the
// scale of the page before it (2^-100 if there is none): any would do.
template <int DIM, int NW, bool E4M3, bool CAP>
__global__ void __launch_bounds__(NW * 64)
    __attribute__((amdgpu_waves_per_eu(DIM == 256 ? 1 : 2))) attend_many_kernel(AttendArgs a) {
  constexpr int T = NW * 64;      // threads
  constexpr int KS = DIM / 16;    // 16-dim steps of the first product
  constexpr int DT = DIM / 32;    // 32-dim tiles of the output
  constexpr int KC = 64 * KS / T; // 16-code pieces of k (and of v) a thread
  static_assert(64 * KS % T == 0, "pieces");
  __shared__ u32x4 lds_k[2][2][KS][64];
  __shared__ u32x4 lds_v[2][4][DT][64];
  // of a tile's four 16-key groups: k scale, log2 and inverse of the v scale,
  // v scale, keys held
  __shared__ float lds_ks[2][4], lds_lv[2][4], lds_iv[2][4], lds_vs[2][4];
  __shared__ int lds_live[2][4];

  const int s = blockIdx.z;
  const int kvh = blockIdx.x % a.cache.heads;
  const SeqSpan sp = seq_span(a.batch, s);
  const int rows = sp.n * a.group;
  if (rows <= a.part.over || rows > a.part.upto) return;
  const int tiles = (rows + NW * 32 - 1) / (NW * 32);
  // last rows first: with a causal mask they see the most keys
  const int row_tile = tiles - 1 - (int)(blockIdx.x / a.cache.heads);
  if (row_tile < 0) return;
  const int row_base = row_tile * (NW * 32);
  const int row_last = row_base + NW * 32 < rows ? row_base + NW * 32 - 1 : rows - 1;
  const int held = held_of(a, s);
  const Span span = span_of(a, sp, held, token_of(a, row_base), token_of(a, row_last));
  const int piece = blockIdx.y;
  if (piece > 0 && piece >= span.pieces) return;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r32 = lane & 31;

  // ---- this lane's row
  const int row = row_base + wave * 32 + r32;
  const bool real = row < rows;
  const int tok = real ? token_of(a, row) : 0;
  const int head = kvh * a.group + (real ? row - tok * a.group : 0);
  f16x8 q[KS];
  float qf;
  {
    const uint16_t* qp = a.q + (int64_t)(sp.row0 + tok) * a.q_stride + (int64_t)head * DIM + 8 * h;
    u32x4 raw[KS];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      raw[k] = real ? *reinterpret_cast<const u32x4*>(qp + 16 * k) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = raw[k][e] & 0x7fffu, y = (raw[k][e] >> 16) & 0x7fffu;
        top = x > top ? x : top;
        top = y > top ? y : top;
      }
    }
    const uint32_t o = __shfl_xor(top, 32);
    top = o > top ? o : top;
    int e = (int)(top >> 7) - 127;
    e = e < -100 ? -100 : (e > 127 ? 14 : e);
    // (a negative scale turns the queries round, so that factors are >= 0)
    const float up = copysignf(__uint_as_float((uint32_t)(14 - e + 127) << 23), a.scale);
    qf = __uint_as_float((uint32_t)(e - 14 + 127) << 23) * fabsf(a.scale);
    qf *= CAP ? 1.f / a.softcap : kLog2e;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t pair = raw[k][j >> 1];
        const float x = __uint_as_float((j & 1) ? pair & 0xffff0000u : pair << 16);
        q[k][j] = (_Float16)(x * up);
      }
  }
  const Keys see = keys_of(a, sp.start + tok, held);
  // keys that some, and that all, of this wave's rows see
  const int wrow = row_base + wave * 32;
  const int wlast = wrow + 31 < rows ? wrow + 31 : rows - 1;
  const bool wreal = wrow < rows;
  const Keys wf = keys_of(a, sp.start + (wreal ? token_of(a, wrow) : 0), held);
  const Keys wl = keys_of(a, sp.start + (wreal ? token_of(a, wlast) : 0), held);

  const int begin = span.lo + piece * a.part.piece;
  const int stop = begin + a.part.piece < span.hi ? begin + a.part.piece : span.hi;
  const int n_tiles = stop > begin ? (stop - begin + 63) >> 6 : 0;
  const int block = a.cache.block, shift = __builtin_ctz(block);
  const int head_bytes = block * DIM;
  const uint32_t page_bytes = (uint32_t)head_bytes * a.cache.heads;
  const uint8_t* const kbase = a.cache.k + (int64_t)kvh * head_bytes;
  const uint8_t* const vbase = a.cache.v + (int64_t)kvh * head_bytes;
  const int* const table = a.batch.page_table + (int64_t)s * a.batch.table_pages;

  f32x16 acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) acc[d] = f32x16{};
  float ref = kNoRef, sum = 0.f, vlast = kMinScale;

  // ---- staging.  Thread tid converts k's piece (key c / KS, 16-dim step
  // c % KS) and v's piece (dim c / 4, 16-key group c % 4), c = tid + i T; the
  // 16-key group of its k is the same for the whole wave.
  u32x4 kc[KC], vc[KC];
  float ksc = 0.f, vsc = 0.f;
  struct Pages {
    int p[4];  // of a tile's 16-key groups, -1: none
  };
  // this tile's table entries, group lane % 4
  auto entries = [&](int t) {
    const int key = begin + 64 * t + 16 * (lane & 3);
    const int p = table[(key < stop ? key : stop - 1) >> shift];
    return key < stop ? p : -1;
  };
  auto pages_of = [&](int v) {
    Pages r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = __builtin_amdgcn_readlane(v, e);
      r.p[e] = p < 0 || p >= a.cache.pages ? -1 : p;
    }
    return r;
  };
  auto group_of = [&](const Pages& p) {  // the entry of group tid % 4
    const int x = (tid & 1) ? p.p[1] : p.p[0], y = (tid & 1) ? p.p[3] : p.p[2];
    return (tid & 2) ? y : x;
  };
  auto load_k = [&](const Pages& p, int t) {
    const int at = (begin + 64 * t) & (block - 1);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int c = tid + i * T;
      const int e = (wave * (64 / KS) + i * (T / KS)) >> 4;  // group of key c / KS
      const int x = (e & 1) ? p.p[1] : p.p[0], y = (e & 1) ? p.p[3] : p.p[2];
      const int pg = (e & 2) ? y : x;
      const uint8_t* from = kbase + (uint64_t)(uint32_t)(pg < 0 ? 0 : pg) * page_bytes + at * DIM;
      kc[i] = *reinterpret_cast<const u32x4*>(
          from + (uint32_t)(((c / KS) & (block - 1)) * DIM + 16 * (c % KS)));
    }
  };
  auto load_v = [&](const Pages& p, int t) {
    const int at = (begin + 64 * t) & (block - 1);
    const int pg = group_of(p);
    const int64_t first = (int64_t)(uint64_t)(uint32_t)(pg < 0 ? 0 : pg) * page_bytes;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int c = tid + i * T;
      vc[i] = *reinterpret_cast<const u32x4*>(
          vbase + first + (uint32_t)((c >> 2) * block + at + ((16 * (c & 3)) & (block - 1))));
    }
    const int64_t hp = (int64_t)(pg < 0 ? 0 : pg) * a.cache.heads + kvh;
    ksc = a.cache.k_scale[hp];
    vsc = a.cache.v_scale[hp];
  };
  auto live_of = [&](int pg, int t) {  // keys held of group tid % 4
    const int n = stop - (begin + 64 * t + 16 * (tid & 3));
    return pg < 0 || n <= 0 ? 0 : (n < 16 ? n : 16);
  };
  auto store_k = [&](int buf) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int c = tid + i * T;
      const int key = c / KS, ks = c % KS;
      // row of the S^T product that gives this key: see above
      const int e = key & 15, m = (key & 16) | ((e & 8) >> 1) | ((e & 4) << 1) | (e & 3);
      const int sw = KS == 4 ? 2 * ks : ks & 7;
      lds_k[buf][key >> 5][ks][m ^ sw] =
          __builtin_bit_cast(u32x4, codes_to_f16<E4M3>(kc[i][0], kc[i][1]));
      lds_k[buf][key >> 5][ks][(32 + m) ^ sw] =
          __builtin_bit_cast(u32x4, codes_to_f16<E4M3>(kc[i][2], kc[i][3]));
    }
  };
  auto store_v = [&](int buf) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int c = tid + i * T;
      const int dim = c >> 2, kst = c & 3;
      lds_v[buf][kst][dim >> 5][(dim & 31) ^ (2 * kst)] =
          __builtin_bit_cast(u32x4, codes_to_f16<E4M3>(vc[i][0], vc[i][1]));
      lds_v[buf][kst][dim >> 5][(32 + (dim & 31)) ^ (2 * kst)] =
          __builtin_bit_cast(u32x4, codes_to_f16<E4M3>(vc[i][2], vc[i][3]));
    }
  };
  // the tile's scales and keys held
  auto store_facts = [&](int buf, int live) {
    if (tid < 4) {
      const float vs = live > 0 ? vsc : 0.f;
      lds_ks[buf][tid] = ksc;
      lds_vs[buf][tid] = vs;
      lds_lv[buf][tid] = __builtin_amdgcn_logf(vs);
      lds_iv[buf][tid] = 1.f / vs;
      lds_live[buf][tid] = live;
    }
  };
  // bytes of v beyond the sequence must not become NaN
  auto cut_v = [&](int live) {
    if (__any(live < 16)) {
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int keep = live - 4 * w;
          vc[i][w] &= keep >= 4 ? 0xffffffffu : (keep <= 0 ? 0u : (1u << (8 * keep)) - 1);
        }
    }
  };
  auto scores = [&](int buf, f32x16& s0, f32x16& s1) {
    s0 = f32x16{};
    s1 = f32x16{};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int at = lane ^ (KS == 4 ? 2 * k : k & 7);
      s0 = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, lds_k[buf][0][k][at]),
                                                  q[k], s0, 0, 0, 0);
      s1 = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, lds_k[buf][1][k][at]),
                                                  q[k], s1, 0, 0, 0);
    }
  };

  // State at the head of tile t: k(t + 1), v(t) and v's facts in LDS, the
  // scores of t in registers, the codes of k(t + 2) and v(t + 1) on their way,
  // pages known to t + 2 and the entries of t + 3 on their way.
  Pages ahead;
  int entry, live_next;
  f32x16 sc0 = {}, sc1 = {};
  if (n_tiles > 0) {
    const int e0 = entries(0), e1 = entries(1), e2 = entries(2);
    entry = entries(3);
    Pages p0 = pages_of(e0), p1 = pages_of(e1);
    ahead = pages_of(e2);
    load_k(p0, 0);
    load_v(p0, 0);
    const int live0 = live_of(group_of(p0), 0);
    cut_v(live0);
    store_k(0);
    store_v(0);
    store_facts(0, live0);
    load_k(p1, 1);
    load_v(p1, 1);
    live_next = live_of(group_of(p1), 1);
    store_k(1);
    load_k(ahead, 2);
    __syncthreads();
    scores(0, sc0, sc1);
  }

  auto stage = [&](int t) {  // k(t + 2), v(t + 1); loads of k(t + 3), v(t + 2)
    store_k(t & 1);
    store_v((t & 1) ^ 1);
    const Pages p = pages_of(entry);
    load_k(p, t + 3);
    load_v(ahead, t + 2);
    live_next = live_of(group_of(ahead), t + 2);
    ahead = p;
    entry = entries(t + 4);
  };
  if (!wreal) {  // a wave without rows only stages
    for (int t = 0; t < n_tiles; ++t) {
      __syncthreads();
      cut_v(live_next);
      store_facts((t & 1) ^ 1, live_next);
      stage(t);
    }
    return;
  }
  for (int t = 0; t < n_tiles; ++t) {
    const int buf = t & 1, key0 = begin + 64 * t;
    __syncthreads();
    cut_v(live_next);
    store_facts(buf ^ 1, live_next);
#define SC(j) ((j) < 16 ? sc0[(j) & 15] : sc1[(j) & 15])
    float f[4], lv[4], iv[4];
    bool full = true, zero = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // (not 0, so that it keeps a masked key's -infinity: a page of zeros)
      f[e] = fmaxf(lds_ks[buf][e] * qf, 0x1p-120f);
      lv[e] = lds_lv[buf][e];
      iv[e] = lds_iv[buf][e];
      full = full && lds_live[buf][e] == 16;
      zero = zero || !(lv[e] > -200.f);
    }
    if (zero) {  // the same in all lanes
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float vs = lds_vs[buf][e];
        if (vs > 0.f) {
          vlast = vs;
        } else {
          lv[e] = __builtin_amdgcn_logf(vlast);
          iv[e] = 1.f / vlast;
        }
      }
    } else {
      vlast = lds_vs[buf][3];
    }
    if (CAP) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = capped(SC(8 * e + i) * f[e]) * (a.softcap * kLog2e);
          if (e < 2) sc0[8 * e + i] = x; else sc1[8 * (e & 1) + i] = x;
        }
        f[e] = 1.f;
      }
    }
    if (!full || key0 < wl.lo || key0 + 64 > wf.hi) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int live = lds_live[buf][e];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = key0 + 16 * e + 8 * h + i;
          if (8 * h + i >= live || j < see.lo || j >= see.hi)
            if (e < 2) sc0[8 * e + i] = -INFINITY; else sc1[8 * (e & 1) + i] = -INFINITY;
        }
      }
    }
    // ---- reference
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float m = SC(8 * e);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, SC(8 * e + i));
      top = fmaxf(top, fmaf(m, f[e], lv[e]));
    }
    if (__any(top > ref + kSlack)) {
      top = fmaxf(top, __shfl_xor(top, 32));
      const float m = fmaxf(top, ref);
      const float g = __builtin_amdgcn_exp2f(ref - m);
      ref = m;
      sum *= g;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] = acc[d] * g;
    }
    // ---- probabilities, and the next tile's scores (of the last tile's
    // successor too: they are not used)
    f32x16 nx0, nx1;
    scores(buf ^ 1, nx0, nx1);
    f16x8 p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c = lv[e] - ref;
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float x = __builtin_amdgcn_exp2f(fmaf(SC(8 * e + i), f[e], c));
        const float y = __builtin_amdgcn_exp2f(fmaf(SC(8 * e + i + 1), f[e], c));
        part += x + y;
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f16x2 xy = __builtin_convertvector(f32x2{x, y}, f16x2);
        p[e][i] = xy[0];
        p[e][i + 1] = xy[1];
      }
      sum = fmaf(part, iv[e], sum);
    }
    sc0 = nx0;
    sc1 = nx1;
    // ---- O^T += V^T P^T, and the next codes
    stage(t);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int d = 0; d < DT; ++d)
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            __builtin_bit_cast(f16x8, lds_v[buf][e][d][lane ^ (2 * e)]), p[e], acc[d], 0, 0, 0);
  }
#undef SC

  sum += __shfl_xor(sum, 32);
  if (!real) return;
  const int64_t out_row = (int64_t)(sp.row0 + tok) * a.q_heads + head;
  if (span.pieces <= 1) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* o = a.out + out_row * DIM + 4 * h;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u32x2 b;
        b[0] = bf16_pair(acc[d][4 * i] * inv, acc[d][4 * i + 1] * inv);
        b[1] = bf16_pair(acc[d][4 * i + 2] * inv, acc[d][4 * i + 3] * inv);
        if (sum == 0.f) b = u32x2{0, 0};
        *reinterpret_cast<u32x2*>(o + 32 * d + 8 * i) = b;
      }
    if (a.lse && h == 0) a.lse[out_row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
  } else {
    const int64_t at = piece * a.part.step + part_row(a, s, kvh, row, out_row);
    float* o = a.part.o + at * DIM + 4 * h;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(o + 32 * d + 8 * i) =
            f32x4{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]};
    if (h == 0) {
      a.part.ml[2 * at] = ref;
      a.part.ml[2 * at + 1] = sum;
    }
  }
}

// ------------------------------------------------------------- the join
//
// Threads of L = DIM / 4 a row hold four outputs each.
//   Few rows have many pieces: a workgroup for each, whose 256 / L groups of
// threads take the pieces in turn, each with a reference and a sum of its own,
// joined through LDS.
//   Many rows have few pieces: 256 / L rows a workgroup, each of which searches
// for its sequence among the batch's.  (A workgroup a row, over a grid of the
// longest prompt's rows for every sequence, took 1.1 ns a workgroup only to
// start them: 8 prompts of 512 tokens 150 us.)
//   One launch for both, whose first few_blocks workgroups are for few rows.
template <int DIM>
struct Joined {
  float m = kNoRef, sum = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
};
template <int DIM>
__device__ __forceinline__ void join_pieces(const AttendPart& p, int64_t first, int from, int by,
                                            int pieces, int l, Joined<DIM>& r) {
  for (int i0 = from; i0 < pieces; i0 += 4 * by) {
    float mi[4], si[4];
    f32x4 oi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * by;
      const int64_t at = first + (i < pieces ? i : i0) * p.step;
      mi[j] = p.ml[2 * at];
      si[j] = p.ml[2 * at + 1];
      oi[j] = *reinterpret_cast<const f32x4*>(p.o + at * DIM + 4 * l);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i0 + j * by >= pieces) continue;
      const float top = fmaxf(r.m, mi[j]);
      const float f = __builtin_amdgcn_exp2f(r.m - top), fi = __builtin_amdgcn_exp2f(mi[j] - top);
      r.sum = r.sum * f + si[j] * fi;
      r.o = r.o * f + oi[j] * fi;
      r.m = top;
    }
  }
}
template <int DIM>
__device__ __forceinline__ void put_joined(const AttendArgs& a, int64_t out_row, int l,
                                           const Joined<DIM>& r) {
  const float inv = r.sum == 0.f ? 0.f : 1.f / r.sum;
  u32x2 b;
  b[0] = bf16_pair(r.o[0] * inv, r.o[1] * inv);
  b[1] = bf16_pair(r.o[2] * inv, r.o[3] * inv);
  if (r.sum == 0.f) b = u32x2{0, 0};
  *reinterpret_cast<u32x2*>(a.out + out_row * DIM + 4 * l) = b;
  if (a.lse && l == 0)
    a.lse[out_row] = r.sum == 0.f ? -INFINITY : (r.m + log2f(r.sum)) * kLn2;
}

template <int DIM>
__global__ void __launch_bounds__(256)
    join_kernel(AttendArgs a, AttendPlan plan, int few_rows, int few_blocks) {
  constexpr int L = DIM / 4, G = 256 / L;
  __shared__ f32x4 lds_o[G][L];
  __shared__ float lds_ml[G][2];
  const int kvh = blockIdx.y, bx = blockIdx.x;
  const int l = threadIdx.x % L, pg = threadIdx.x / L;
  const bool is_few = bx < few_blocks;
  int s, row;
  if (is_few) {
    s = bx / few_rows;
    row = bx - s * few_rows;
  } else {
    const int64_t all = (int64_t)(bx - few_blocks) * G + pg;
    if (all >= a.batch.rows * a.group) return;
    const int at = (int)((uint32_t)all / (uint32_t)a.group);
    int end = a.batch.seqs;
    for (s = 0; end - s > 1;) {
      const int mid = (s + end) >> 1;
      if (a.batch.q_start[mid] <= at)
        s = mid;
      else
        end = mid;
    }
    row = (int)(all - (int64_t)seq_span(a.batch, s).row0 * a.group);
  }
  const SeqSpan sp = seq_span(a.batch, s);
  const int rows = sp.n * a.group;
  if (row < 0 || row >= rows) return;
  a.part = plan.part[0];
  for (int i = 1; i < plan.parts; ++i)
    if (rows > plan.part[i].over) a.part = plan.part[i];
  if (is_few != (a.part.tile <= 32)) return;
  const int held = held_of(a, s);
  const int tile = a.part.tile;
  for (; row < rows; row += is_few ? few_rows : rows) {
    const int row_base = row / tile * tile;
    const int row_last = row_base + tile < rows ? row_base + tile - 1 : rows - 1;
    const Span span = span_of(a, sp, held, token_of(a, row_base), token_of(a, row_last));
    if (span.pieces <= 1) return;  // written already (a few rows' span is the same for all)
    const int tok = token_of(a, row);
    const int64_t out_row =
        (int64_t)(sp.row0 + tok) * a.q_heads + kvh * a.group + (row - tok * a.group);
    const int64_t first = part_row(a, s, kvh, row, out_row);
    Joined<DIM> r;
    if (!is_few) {
      join_pieces<DIM>(a.part, first, 0, 1, span.pieces, l, r);
      put_joined<DIM>(a, out_row, l, r);
      return;
    }
    join_pieces<DIM>(a.part, first, pg, G, span.pieces, l, r);
    if (l == 0) {
      lds_ml[pg][0] = r.m;
      lds_ml[pg][1] = r.sum;
    }
    lds_o[pg][l] = r.o;
    __syncthreads();
    if (pg == 0) {
      r = Joined<DIM>();
#pragma unroll
      for (int i = 0; i < G; ++i) r.m = fmaxf(r.m, lds_ml[i][0]);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float f = __builtin_amdgcn_exp2f(lds_ml[i][0] - r.m);
        r.sum += lds_ml[i][1] * f;
        r.o = r.o + lds_o[i][l] * f;
      }
      put_joined<DIM>(a, out_row, l, r);
    }
    __syncthreads();
  }
}

namespace {

constexpr int many_waves(int dim) { return dim == 128 ? 8 : 4; }
constexpr int kFewWaves = 4;

// Keys of a wave's tile: 32 leave dim 256 two waves a SIMD (16 sequences of 8192 tokens:
// 68 -> 55 us, eight sequences of five drafted tokens 34 -> 24 us) and dim 64 four (10.2 ->
// 9.6 us); at dim 128 64 keys keep two waves and more bytes in flight (32 sequences: 103
// against 107 us).
constexpr int few_keys(int dim) { return dim == 128 ? 64 : 32; }

template <int DIM, int ROWS, int NW, int KT>
hipError_t few(const AttendArgs& a, dim3 grid, hipStream_t s) {
  const dim3 block(NW * 64);
  const bool cap = a.softcap > 0.f;
  if (a.cache.e4m3) {
    if (cap)
      hipLaunchKernelGGL((attend_few_kernel<DIM, ROWS, KT, NW, true, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((attend_few_kernel<DIM, ROWS, KT, NW, true, false>), grid, block, 0, s, a);
  } else {
    if (cap)
      hipLaunchKernelGGL((attend_few_kernel<DIM, ROWS, KT, NW, false, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((attend_few_kernel<DIM, ROWS, KT, NW, false, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

template <int DIM>
hipError_t many(const AttendArgs& a, dim3 grid, hipStream_t s) {
  constexpr int NW = many_waves(DIM);
  const dim3 block(NW * 64);
  const bool cap = a.softcap > 0.f;
  if (a.cache.e4m3) {
    if (cap)
      hipLaunchKernelGGL((attend_many_kernel<DIM, NW, true, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((attend_many_kernel<DIM, NW, true, false>), grid, block, 0, s, a);
  } else {
    if (cap)
      hipLaunchKernelGGL((attend_many_kernel<DIM, NW, false, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((attend_many_kernel<DIM, NW, false, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

template <int DIM>
hipError_t attend_part(AttendArgs& a, const AttendPart& part, hipStream_t s) {
  a.part = part;
  const int tile = part.tile;
  const int64_t most = (int64_t)a.batch.max_new * a.group;
  const int64_t tiles = tile > 32 ? (most + tile - 1) / tile : 1;
  const dim3 grid((unsigned)(a.cache.heads * tiles), (unsigned)part.pieces,
                  (unsigned)a.batch.seqs);
  constexpr int KT = few_keys(DIM);
  return tile == 16   ? few<DIM, 1, kFewWaves, KT>(a, grid, s)
         : tile == 32 ? few<DIM, 2, kFewWaves, KT>(a, grid, s)
                      : many<DIM>(a, grid, s);
}

template <int DIM>
hipError_t attend_dim(AttendArgs& a, const AttendPlan& plan, hipStream_t s) {
  int64_t few_blocks = 0, many_blocks = 0;
  constexpr int G = 256 / (DIM / 4);  // rows of a workgroup of the join
  const int64_t most = (int64_t)a.batch.max_new * a.group;
  // workgroups of the join for a sequence and head of few rows; beside prompts
  // eight that take the rows in turn (32 that mostly find none cost 25 us for
  // 200 sequences)
  const int64_t few_rows = most <= 32 ? most : 8;
  // (prompts first: they run longest)
  for (int i = plan.parts - 1; i >= 0; --i) {
    const AttendPart& p = plan.part[i];
    const hipError_t e = attend_part<DIM>(a, p, s);
    if (e != hipSuccess) return e;
    if (p.pieces <= 1) continue;
    if (p.tile <= 32)
      few_blocks = few_rows * a.batch.seqs;
    else
      many_blocks = (a.batch.rows * a.group + G - 1) / G;
  }
  if (few_blocks + many_blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((join_kernel<DIM>),
                     dim3((unsigned)(few_blocks + many_blocks), (unsigned)a.cache.heads),
                     dim3(256), 0, s, a, plan, (int)few_rows, (int)few_blocks);
  return hipGetLastError();
}

// Pieces of the longest span a row can see.  The lengths are not known here.
//   Few rows: two workgroups a CU, counting every sequence.  With several
// sequences more pieces keep the long ones from running on behind the short
// ones, but each has a start and a join, which cost about as much as 256
// tokens.  A place on the chip with W = groups * keys / 512 tokens to read
// takes W (1 + 256 / piece) + piece / 2: least at piece^2 = 512 W, which is
// (keys / piece)^2 = keys / groups; taken to the next power of two (others
// fall unevenly on the chip).  32 sequences of up to 16384 tokens: 4 pieces
// 112 us, 8 (this rule) 95.8, 12 99.7, 16 99.6; 128 of 8192: 4 (this rule)
// 397, 16 452.
//   Many rows: one workgroup a CU, which is what fits of them at dim 128 (2048
// tokens behind 2048, 32 heads of 128: one piece 146 us, two 222).  Counted are
// the rows of the batch, not the longest prompt's for every sequence, by which
// one prompt among single tokens would pass for 32 prompts and stay whole (512
// tokens over 4096, seven single ones beside it: 106 us, by its rows 74).
//   384 tokens a piece where that still fills the chip, 256 where it does not;
// and few rows of a short span are not cut at all, since the join costs as much
// as two or three turns of a workgroup and more where there are many (one token
// over 500: 8.7 us against 10.3, over 1000 12.4 against 10.5; 16 over 700 10.7
// against 13.2, over 1000 14.1 against 13.5; 64 over 1000 24.0 against 32.9).
void plan_part(const AttendArgs& a, int tile, int over, int upto, AttendPlan* plan) {
  AttendPart* const p = &plan->part[plan->parts++];
  p->tile = tile;
  p->over = over;
  p->upto = upto;
  int64_t keys = (int64_t)a.batch.table_pages * a.cache.block;
  if (a.window > 0 && a.window + a.batch.max_new + 64 < keys)
    keys = a.window + a.batch.max_new + 64;
  int64_t tiles = a.batch.seqs;
  if (tile > 32) {
    const int64_t most = (int64_t)a.batch.max_new * a.group, all = a.batch.rows * a.group;
    tiles *= (most + tile - 1) / tile;
    if (tiles > (all + tile - 1) / tile) tiles = (all + tile - 1) / tile;
    if (tiles < 1) tiles = 1;
  }
  const int64_t groups = tiles * a.cache.heads;
  const int64_t step = few_keys(a.cache.dim) * kFewWaves;  // few rows: keys of a workgroup's turn
  const int64_t want = tile > 32 ? 256 : 512;
  int64_t pieces = (want + groups - 1) / groups;
  if (tile <= 32 && a.batch.seqs > 1) {
    int64_t split = 1;
    while (split * split * groups < keys) split *= 2;
    if (pieces < split) pieces = split;
  }
  const int64_t least = groups * keys >= 512 * 256 ? 384 : 256;
  if (pieces > (keys + least - 1) / least) pieces = (keys + least - 1) / least;
  const int64_t half_turns = groups >= 256 ? 8 : groups >= 64 ? 6 : 5;
  if (tile <= 32 && 2 * keys <= half_turns * step) pieces = 1;
  const int64_t grain = tile <= 32 ? step : 64;
  p->piece = (int)(((keys + pieces - 1) / pieces + grain - 1) / grain * grain);
  p->pieces = (int)((keys + p->piece - 1) / p->piece);
  p->turn = (uint32_t)((((uint64_t)1 << 31) + p->pieces - 1) / p->pieces);
  p->step = tile <= 32 ? (int64_t)a.batch.seqs * a.cache.heads * tile : a.batch.rows * a.q_heads;
}

}  // namespace

// Up to 32 rows of a sequence and head share the codes' way through one wave's
// registers; more are worth converting the codes once for all of them.  Where
// prompts and steps come in one batch, each kind has a launch of its own: 512
// tokens over 4096 with 31 single tokens over 8192 take 212 us (936 if all go
// the prompts' way), with seven times six drafted tokens over 4096 81 us (168
// if only up to 16 rows go the other way).  Two prompts of 64 tokens pay 1.5 of
// 28 us for a launch that finds nothing.
AttendPlan attend_plan(const AttendArgs& a, void* workspace) {
  AttendPlan r{};
  const int64_t most = (int64_t)a.batch.max_new * a.group;
  const bool several = a.batch.seqs > 1;
  if (most <= 32 || several) plan_part(a, most <= 16 ? 16 : 32, 0, 32, &r);
  if (most > 32) plan_part(a, many_waves(a.cache.dim) * 32, several ? 32 : 0, 0x7fffffff, &r);
  float* at = static_cast<float*>(workspace);
  for (int i = 0; i < r.parts; ++i) {
    AttendPart* const p = &r.part[i];
    if (p->pieces <= 1) continue;
    const size_t rows = (size_t)p->pieces * p->step;
    // (each begins 16-byte aligned)
    const size_t floats = (rows * (a.cache.dim + 2) + 3) & ~(size_t)3;
    r.bytes += floats * sizeof(float);
    if (!at) continue;
    p->o = at;
    p->ml = at + rows * a.cache.dim;
    at += floats;
  }
  return r;
}

hipError_t launch_attend(AttendArgs& a, const AttendPlan& plan, hipStream_t s) {
  if (a.batch.rows == 0) return hipSuccess;
  switch (a.cache.dim) {
    case 64: return attend_dim<64>(a, plan, s);
    case 128: return attend_dim<128>(a, plan, s);
    case 256: return attend_dim<256>(a, plan, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mq
