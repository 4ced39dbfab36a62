// Rotary positions, and the 8-bit key/value cache: written with its scales
// found on the way, and read back.  All three move bytes: their floor is the
// activations in and the codes (or values) out.
#include "kv_device.h"

namespace mq {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ mq_rope
//
// A thread owns one unit (eight entries, four pairs) of one token and walks
// over `per` heads, four at a time in flight, so the four float64 sines and
// cosines (about 45 instructions a pair) are found once for all of them; the
// angles do not depend on the head.  Lanes of a wave hold consecutive units:
// 8 or 16 bytes each, whole lines together.  8192 tokens of 32 x 128 bf16 (134
// MB in and out): 26 us, 5.1 TB/s, the rate of a large copy.
template <bool F32>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeSpec r, const int* positions,
                                                        const void* x, int64_t x_stride,
                                                        int64_t rows, int heads, int dim,
                                                        uint16_t* out, int64_t out_stride,
                                                        int per) {
  const int units = dim >> 3;
  const int slots = kThreads / units;
  const int u = threadIdx.x % units, slot = threadIdx.x / units;
  const int64_t row = (int64_t)blockIdx.x * slots + slot;
  if (slot >= slots || row >= rows) return;
  const Unit un = unit_of(u, r.rot, r.interleaved);
  const int h0 = blockIdx.y * per, h1 = h0 + per < heads ? h0 + per : heads;
  Turn turn;
  RawUnit<F32> raw[4];
  const int pos = positions[row];
  for (int h = h0; h < h1; h += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (h + j < h1) raw[j] = load_unit<F32>(x, row * x_stride + (int64_t)(h + j) * dim, un);
    if (h == h0 && un.turns) turn.at(r, un, (double)pos, r.factor);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (h + j >= h1) continue;
      float v[8];
      numbers_of_unit<F32>(raw[j], v);
      if (un.turns) turn_unit(v, turn.c, turn.s, r.interleaved);
      uint32_t w[4];
      pack_unit(v, w);
      uint16_t* o = out + row * out_stride + (int64_t)(h + j) * dim;
      *reinterpret_cast<u32x2*>(o + un.lo) = u32x2{w[0], w[1]};
      *reinterpret_cast<u32x2*>(o + un.hi) = u32x2{w[2], w[3]};
    }
  }
}

hipError_t launch_rope(const RopeSpec& r, const int* positions, const void* x, bool f32,
                       int64_t x_stride, int64_t rows, int heads, int dim, uint16_t* out,
                       int64_t out_stride, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int slots = kThreads / (dim / 8);
  const int64_t groups = (rows + slots - 1) / slots;
  // heads of a thread: as many as leave 512 workgroups (two a CU)
  int per = 8;
  while (per > 1 && groups * ((heads + per - 1) / per) < 512) per >>= 1;
  while ((heads + per - 1) / per > 65535) per <<= 1;
  const dim3 grid((unsigned)groups, (unsigned)((heads + per - 1) / per));
  if (f32)
    hipLaunchKernelGGL(rope_kernel<true>, grid, dim3(kThreads), 0, s, r, positions, x, x_stride,
                       rows, heads, dim, out, out_stride, per);
  else
    hipLaunchKernelGGL(rope_kernel<false>, grid, dim3(kThreads), 0, s, r, positions, x, x_stride,
                       rows, heads, dim, out, out_stride, per);
  return hipGetLastError();
}

// --------------------------------------------------------- mq_cache_append
//
// One workgroup per (sequence, page that gets tokens, head, k or v): the
// page's new values stay in registers as bf16 (at most 32 dwords a thread)
// between finding the scale and rounding to codes, so they are read once, and
// no other workgroup touches the page's scale or codes.  Eight tokens' loads
// (four of fp32) are in flight before the first is used, the first of them
// before the page is known.  k's angles of a thread advance by a constant
// step, so its sines and cosines follow by one complex product a token in
// place of an evaluation, and its first ones from a table of the page's first
// position and of one position (turn_table).
// v is held dim-major: pages that get 16 tokens or more go through LDS, four
// tokens of a dim to a dword, and leave in 16-byte pieces; fewer tokens go out
// as single bytes.
// 8192 tokens of 8 x 256 with 16 heads of queries turned (235 MB): 67 us from
// HBM, 56 where the activations are still in the last-level cache (3.5 and 4.2
// TB/s); the turns, in float64, take 9 of them.  A step of 32 tokens: 5 us, a
// chain of dependent loads (lengths, table, scale) and two barriers.
//
// The queries' workgroups (blockIdx.y >= 2 * heads) take eight tokens of the
// same page each, all heads.

constexpr int kQueryTokens = 8;

// at most eight tokens of one page, all query heads
template <int DIM, int T, bool F32>
__device__ __forceinline__ void append_queries(const RopeSpec& r, const SeqSpan& sp, int64_t lo,
                                               int64_t hi, const void* q, int64_t q_stride,
                                               int q_heads, uint16_t* q_out, double* table) {
  constexpr int U = DIM / 8, SLOTS = T / U;
  const int u = threadIdx.x % U, slot = threadIdx.x / U;
  const int hs = q_heads < SLOTS ? q_heads : SLOTS;  // heads side by side
  const int toks = SLOTS / hs;                       // tokens side by side
  const int head0 = slot % hs, tok0 = slot / hs;
  const Unit un = unit_of(u, r.freq ? r.rot : 0, r.interleaved);
  Turn turn, step;
  if (r.freq) {
    turn_table(table, r, (double)lo);
    if (un.turns) {
      // turn at lo + tok0, step of toks positions
      turn.from_table(table, un);
      if (hi - lo > 1) {
        Turn power;
        power.from_table(table + r.rot, un);
#pragma unroll
        for (int i = 0; i < 4; ++i) step.c[i] = 1.0, step.s[i] = 0.0;
        for (int b = 1; b <= toks; b <<= 1) {
          if (tok0 & b) turn.advance(power);
          if (toks & b) step.advance(power);
          const Turn p = power;
          power.advance(p);
        }
      }
    }
  }
  if (tok0 >= toks) return;
  for (int64_t pos = lo + tok0; pos < hi; pos += toks) {
    const int64_t row = sp.row0 + (pos - sp.start);
    for (int h = head0; h < q_heads; h += 4 * hs) {
      RawUnit<F32> raw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (h + j * hs < q_heads)
          raw[j] = load_unit<F32>(q, row * q_stride + (int64_t)(h + j * hs) * DIM, un);
      if (h == head0 && un.turns && pos != lo + tok0) turn.advance(step);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (h + j * hs >= q_heads) continue;
        float v[8];
        numbers_of_unit<F32>(raw[j], v);
        if (un.turns) turn_unit(v, turn.c, turn.s, r.interleaved);
        uint32_t w[4];
        pack_unit(v, w);
        uint16_t* o = q_out + (row * q_heads + h + j * hs) * DIM;
        *reinterpret_cast<u32x2*>(o + un.lo) = u32x2{w[0], w[1]};
        *reinterpret_cast<u32x2*>(o + un.hi) = u32x2{w[2], w[3]};
      }
    }
  }
}

// Threads of a page's workgroup: at most 64 values each.
constexpr int append_threads(int dim, int block) { return dim * block > 16384 ? 512 : 256; }

template <int DIM, int BLOCK, bool F32>
__global__ void __launch_bounds__(append_threads(DIM, BLOCK))
append_kernel(KvCache cache, KvBatch b, RopeSpec r, const void* k, const void* v,
              int64_t kv_stride, const void* q, int64_t q_stride, int q_heads, uint16_t* q_out) {
  constexpr int T = append_threads(DIM, BLOCK);
  constexpr int U = DIM / 8, SLOTS = T / U;
  constexpr int STEPS = BLOCK / SLOTS > 0 ? BLOCK / SLOTS : 1;
  constexpr int ONCE = F32 ? 4 : 8;            // steps loaded before the first is used
  constexpr int G = STEPS < 4 ? STEPS : 4;     // consecutive tokens a thread has of v
  constexpr int PITCH = BLOCK + 4;             // bytes of a dim's row in LDS
  // v's codes on their way to dim-major, or k's and q's table of turns
  __shared__ __align__(16) uint32_t tile[DIM * PITCH / 4];
  static_assert(sizeof(tile) >= 16 * DIM, "turns of DIM / 2 pairs, twice");
  double* const table = reinterpret_cast<double*>(tile);
  __shared__ uint32_t wave_max[T / 64];

  const int seq = blockIdx.z;
  const SeqSpan sp = seq_span(b, seq);
  const int64_t end = sp.start + sp.n;
  const int64_t first = sp.start < 0 ? 0 : sp.start;
  const int64_t pi = first / BLOCK + blockIdx.x;
  const int64_t base = pi * BLOCK;
  int64_t lo = base > first ? base : first;
  int64_t hi = base + BLOCK < end ? base + BLOCK : end;
  if (lo >= hi) return;
  if ((int)blockIdx.y >= 2 * cache.heads) {
    // queries of positions without a page are written too: they are rows
    const int part = blockIdx.y - 2 * cache.heads;
    lo = lo > base + part * kQueryTokens ? lo : base + part * kQueryTokens;
    const int64_t last = base + (part + 1) * kQueryTokens;
    hi = hi < last ? hi : last;
    if (lo < hi) 
      append_queries<DIM, T, F32>(r, sp, lo, hi, q, q_stride, q_heads, q_out, table);
    return;
  }
  const int page = page_of(b, seq, pi, cache.pages);
  const int head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const bool e4m3 = cache.e4m3;
  const int tid = threadIdx.x, u = tid % U, slot = tid / U;
  const int used = (int)(lo - base);  // earlier tokens of the page
  const int fill = (int)(hi - base);

  // ---- the page's new values as bf16, and their largest magnitude
  const Unit un = is_v ? unit_of(u, 0, false) : unit_of(u, r.freq ? r.rot : 0, r.interleaved);
  // place in the page of this thread's j-th token
  auto place = [&](int j) {
    return is_v ? (j / G) * (G * SLOTS) + slot * G + j % G : slot + j * SLOTS;
  };
  const void* src = is_v ? v : k;
  const int64_t at0 = (sp.row0 + (base - sp.start)) * kv_stride + (int64_t)head * DIM;
  uint32_t w[STEPS][4];
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 pair_top = {0, 0};
  Turn turn, step;
  const bool single = fill - used == 1;
  int64_t ph = 0;
  float was = 0.f;
#pragma unroll
  for (int j0 = 0; j0 < STEPS; j0 += ONCE) {
    RawUnit<F32> raw[ONCE];
#pragma unroll
    for (int j = j0; j < j0 + ONCE && j < STEPS; ++j) {
      const int t = place(j);
      if (t >= used && t < fill) raw[j - j0] = load_unit<F32>(src, at0 + t * kv_stride, un);
    }
    if (j0 == 0) {
      // (of the pool's first page where there is none: not used)
      ph = (int64_t)(page < 0 ? 0 : page) * cache.heads + head;
      if (used > 0) was = (is_v ? cache.v_scale : cache.k_scale)[ph];
    }
    if (j0 == 0 && !is_v && r.freq) {
      // (a single token: its own turn)
      turn_table(table, r, (double)(single ? base + used : base));
      if (un.turns && single) {
        turn.from_table(table, un);
      } else if (un.turns) {
        // turn at base + slot; the step of SLOTS positions is what is left of
        // one position's after its squarings
        turn.from_table(table, un);
        step.from_table(table + r.rot, un);
#pragma unroll
        for (int b = 1; b < SLOTS; b <<= 1) {
          turn.advance_if(slot & b, step);
          const Turn p = step;
          step.advance(p);
        }
      }
    }
#pragma unroll
    for (int j = j0; j < j0 + ONCE && j < STEPS; ++j) {
      const int t = place(j);
      if (t >= used && t < fill) {
        if (F32 || un.turns) {
          float x[8];
          numbers_of_unit<F32>(raw[j - j0], x);
          if (un.turns) turn_unit(x, turn.c, turn.s, r.interleaved);
          pack_unit(x, w[j]);
        } else {
          w[j][0] = raw[j - j0].lo[0];
          w[j][1] = raw[j - j0].lo[1];
          w[j][2] = raw[j - j0].hi[0];
          w[j][3] = raw[j - j0].hi[1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pair_top = __builtin_elementwise_max(
              pair_top, __builtin_bit_cast(u16x2, w[j][i] & 0x7fff7fffu));
      }
      if (un.turns && !single && j + 1 < STEPS) turn.advance(step);
    }
  }
  if (page < 0) return;  // (uniform: the page is the workgroup's)
  float* scale_at = (is_v ? cache.v_scale : cache.k_scale) + ph;
  uint8_t* codes = (is_v ? cache.v : cache.k) + ph * (DIM * BLOCK);
  uint32_t top = pair_top[0] > pair_top[1] ? pair_top[0] : pair_top[1];
  // the largest of the workgroup; if some value is no number, of the numbers
  bool odd = false;
  for (int round = 0; round < 2; ++round) {
    for (int off = 32; off > 0; off >>= 1) {
      const uint32_t o = __shfl_xor(top, off);
      top = o > top ? o : top;
    }
    if (round > 0) __syncthreads();
    if ((tid & 63) == 0) wave_max[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T / 64; ++i) top = wave_max[i] > top ? wave_max[i] : top;
    if (top < 0x7f80u) break;
    odd = true;
    top = 0;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const int t = place(j);
      if (t < used || t >= fill) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t m = (w[j][i >> 1] >> (16 * (i & 1))) & 0x7fffu;
        top = m < 0x7f80u && m > top ? m : top;
      }
    }
  }
  float now = __uint_as_float(top << 16) * kv_inv_qmax(e4m3);
  if (now < kMinScale) now = 0.f;
  const bool grows = used > 0 && now > was;
  if (used > 0 && !grows) now = was;
  if (tid == 0) *scale_at = now;

  // ---- earlier codes, where the scale grows
  if (grows) {
    const double ratio = (double)was / (double)now;
    if (!is_v) {
      for (int i = tid; i < used * (DIM / 4); i += T) {
        uint32_t* p = reinterpret_cast<uint32_t*>(codes) + i;
        *p = recode(*p, e4m3, ratio);
      }
    } else {
      // four tokens of a dim at a time; those at or beyond `used` keep their
      // bytes here (this workgroup writes them below)
      const int per = (used + 3) / 4;
      for (int i = tid; i < per * DIM; i += T) {
        const int d = i / per, t = (i % per) * 4;
        uint32_t* p = reinterpret_cast<uint32_t*>(codes + d * BLOCK + t);
        const uint32_t before = *p, after = recode(before, e4m3, ratio);
        const int keep = used - t;
        const uint32_t m = keep >= 4 ? 0xffffffffu : (1u << (8 * keep)) - 1;
        *p = (after & m) | (before & ~m);
      }
    }
    __syncthreads();
  }

  // ---- the new codes
  const float rs = now > 0.f ? 1.f / now : 0.f;
  const bool through_lds = is_v && fill - used >= 16;
  // a dim's row in LDS is turned by a multiple of eight dims' distance, so
  // that the lanes of a wave, eight dims apart, meet different banks
  constexpr int SKEW = 64 / U, WORDS = BLOCK / 4;
#pragma unroll
  for (int j0 = 0; j0 < STEPS; j0 += G) {
    uint32_t out[G][2];
#pragma unroll
    for (int j = j0; j < j0 + G; ++j) {
      const int t = place(j);
      out[j - j0][0] = out[j - j0][1] = 0;
      if (t < used || t >= fill) continue;
      if (now > 0.f) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t pair = w[j][i >> 1];
          x[i] = __uint_as_float((i & 1) ? pair & 0xffff0000u : pair << 16);
        }
        if (odd) {  // infinity: the largest code, NaN: 0
          const float most = now * (e4m3 ? 448.f : 127.f);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[i] = x[i] != x[i] ? 0.f : fminf(fmaxf(x[i], -most), most);
        }
        codes_of_values(x, now, rs, e4m3, out[j - j0]);
      }
      if (!is_v) {
        *reinterpret_cast<uint32_t*>(codes + t * DIM + un.lo) = out[j - j0][0];
        *reinterpret_cast<uint32_t*>(codes + t * DIM + un.hi) = out[j - j0][1];
      } else if (!through_lds) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          codes[(8 * u + i) * BLOCK + t] = (uint8_t)(out[j - j0][i >> 2] >> (8 * (i & 3)));
      }
    }
    if (through_lds) {
      const int t = place(j0);
      const int word = ((t >> 2) + SKEW * (u >> 3)) & (WORDS - 1);
      uint8_t* to = reinterpret_cast<uint8_t*>(tile) + 8 * u * PITCH + 4 * word + (t & 3);
      if (t < BLOCK) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t p = 0;
#pragma unroll
          for (int j = 0; j < G; ++j) p |= ((out[j][i >> 2] >> (8 * (i & 3))) & 0xffu) << (8 * j);
          if (G == 4)
            *reinterpret_cast<uint32_t*>(to + i * PITCH) = p;
          else if (G == 2)
            *reinterpret_cast<uint16_t*>(to + i * PITCH) = (uint16_t)p;
          else
            to[i * PITCH] = (uint8_t)p;
        }
      }
    }
  }
  if (!through_lds) return;
  __syncthreads();
  for (int i = tid; i < DIM * (BLOCK / 16); i += T) {
    const int d = i / (BLOCK / 16), t = (i % (BLOCK / 16)) * 16;
    if (t + 16 <= used || t >= fill) continue;
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      p[e] = tile[d * (PITCH / 4) + (((t >> 2) + e + SKEW * (d >> 6)) & (WORDS - 1))];
    uint8_t* to = codes + d * BLOCK + t;
    if (t >= used && t + 16 <= fill) {
      *reinterpret_cast<u32x4*>(to) = u32x4{p[0], p[1], p[2], p[3]};
    } else {
      for (int e = 0; e < 16; ++e)
        if (t + e >= used && t + e < fill) to[e] = (uint8_t)(p[e >> 2] >> (8 * (e & 3)));
    }
  }
}

namespace {

// Pages that max_new tokens can touch.
int64_t pages_touched(const KvBatch& b, int block) {
  return ((int64_t)b.max_new + block - 2) / block + 1;
}

template <int DIM>
hipError_t append_dim(const KvCache& c, const KvBatch& b, const RopeSpec& r, const void* k,
                      const void* v, int64_t kv_stride, const void* q, int64_t q_stride,
                      int q_heads, bool f32, uint16_t* q_out, hipStream_t s) {
  const int q_parts = q ? c.block / kQueryTokens : 0;
  const dim3 grid((unsigned)pages_touched(b, c.block), (unsigned)(2 * c.heads + q_parts),
                  (unsigned)b.seqs);
#define MQ_APPEND(BLOCK)                                                                        \
  case BLOCK:                                                                                   \
    if (f32)                                                                                    \
      hipLaunchKernelGGL((append_kernel<DIM, BLOCK, true>), grid,                               \
                         dim3(append_threads(DIM, BLOCK)), 0, s, c, b,                          \
                         r, k, v, kv_stride, q, q_stride, q_heads, q_out);                      \
    else                                                                                        \
      hipLaunchKernelGGL((append_kernel<DIM, BLOCK, false>), grid,                              \
                         dim3(append_threads(DIM, BLOCK)), 0, s, c, b,                          \
                         r, k, v, kv_stride, q, q_stride, q_heads, q_out);                      \
    break
  switch (c.block) {
    MQ_APPEND(16);
    MQ_APPEND(32);
    MQ_APPEND(64);
    MQ_APPEND(128);
    default: return hipErrorInvalidValue;
  }
#undef MQ_APPEND
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const KvCache& c, const KvBatch& b, const RopeSpec& r,
                               const void* k, const void* v, int64_t kv_stride, const void* q,
                               int64_t q_stride, int q_heads, bool f32, uint16_t* q_out,
                               hipStream_t s) {
  if (b.rows == 0) return hipSuccess;
  switch (c.dim) {
    case 64: return append_dim<64>(c, b, r, k, v, kv_stride, q, q_stride, q_heads, f32, q_out, s);
    case 128: return append_dim<128>(c, b, r, k, v, kv_stride, q, q_stride, q_heads, f32, q_out, s);
    case 256: return append_dim<256>(c, b, r, k, v, kv_stride, q, q_stride, q_heads, f32, q_out, s);
    default: return hipErrorInvalidValue;
  }
}

// ----------------------------------------------------------- mq_cache_read
//
// One workgroup per (sequence, page, head, k or v).  Eight codes of k and 16
// of v a load; v is turned from dim-major through LDS.  Four sequences of up to
// 16384 tokens, 8 x 128 to bf16 (286 MB): 51 us on the GPU, 5.6 TB/s.
template <int DIM, int BLOCK>
__global__ void __launch_bounds__(kThreads) read_kernel(KvCache cache, KvBatch b, void* k_out,
                                                        void* v_out, bool f32) {
  constexpr int U = DIM / 8, SLOTS = kThreads / U;
  constexpr int PITCH = BLOCK + 4;
  __shared__ uint32_t tile[DIM * PITCH / 4];
  const int seq = blockIdx.z;
  const int head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  void* out = is_v ? v_out : k_out;
  if (!out) return;
  const SeqSpan sp = seq_span(b, seq);
  const int64_t end = sp.start + sp.n;
  // position index of the first row's page, rounded down (it may be negative)
  const int64_t pi = (sp.start >= 0 ? sp.start / BLOCK : -((-sp.start + BLOCK - 1) / BLOCK)) +
                     blockIdx.x;
  const int64_t base = pi * BLOCK;
  const int64_t lo = base > sp.start ? base : sp.start;
  const int64_t hi = base + BLOCK < end ? base + BLOCK : end;
  if (lo >= hi) return;
  const int page = page_of(b, seq, pi, cache.pages);
  const bool e4m3 = cache.e4m3;
  const int tid = threadIdx.x, u = tid % U, slot = tid / U;
  const int64_t ph = (int64_t)(page < 0 ? 0 : page) * cache.heads + head;
  const uint8_t* codes = (is_v ? cache.v : cache.k) + ph * (DIM * BLOCK);
  const float scale = page < 0 ? 0.f : (is_v ? cache.v_scale : cache.k_scale)[ph];
  if (is_v && page >= 0) {
    for (int i = tid; i < DIM * BLOCK / 16; i += kThreads) {
      const int d = i / (BLOCK / 16), t = (i % (BLOCK / 16)) * 16;
      const u32x4 p = *reinterpret_cast<const u32x4*>(codes + d * BLOCK + t);
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[(d * PITCH + t) / 4 + e] = p[e];
    }
    __syncthreads();
  }
  for (int64_t pos = lo + slot; pos < hi; pos += SLOTS) {
    const int t = (int)(pos - base);
    uint32_t p[2] = {0, 0};
    if (page >= 0) {
      if (is_v) {
        const uint8_t* from = reinterpret_cast<const uint8_t*>(tile);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          p[i >> 2] |= (uint32_t)from[(8 * u + i) * PITCH + t] << (8 * (i & 3));
      } else {
        const u32x2 a = *reinterpret_cast<const u32x2*>(codes + t * DIM + 8 * u);
        p[0] = a[0];
        p[1] = a[1];
      }
    }
    float y[8];
    numbers_of(p[0], e4m3, y);
    numbers_of(p[1], e4m3, y + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= scale;
    const int64_t row = sp.row0 + (pos - sp.start);
    const int64_t at = (row * cache.heads + head) * DIM + 8 * u;
    if (f32) {
      f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + at);
      o[0] = f32x4{y[0], y[1], y[2], y[3]};
      o[1] = f32x4{y[4], y[5], y[6], y[7]};
    } else {
      uint32_t w[4];
      pack_unit(y, w);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + at) = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
}

namespace {

template <int DIM>
hipError_t read_dim(const KvCache& c, const KvBatch& b, void* k_out, void* v_out, bool f32,
                    hipStream_t s) {
  const dim3 grid((unsigned)pages_touched(b, c.block), (unsigned)(2 * c.heads), (unsigned)b.seqs);
#define MQ_READ(BLOCK)                                                                         \
  case BLOCK:                                                                                  \
    hipLaunchKernelGGL((read_kernel<DIM, BLOCK>), grid, dim3(kThreads), 0, s, c, b, k_out,     \
                       v_out, f32);                                                            \
    break
  switch (c.block) {
    MQ_READ(16);
    MQ_READ(32);
    MQ_READ(64);
    MQ_READ(128);
    default: return hipErrorInvalidValue;
  }
#undef MQ_READ
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_read(const KvCache& c, const KvBatch& b, void* k_out, void* v_out,
                             bool f32, hipStream_t s) {
  if (b.rows == 0) return hipSuccess;
  switch (c.dim) {
    case 64: return read_dim<64>(c, b, k_out, v_out, f32, s);
    case 128: return read_dim<128>(c, b, k_out, v_out, f32, s);
    case 256: return read_dim<256>(c, b, k_out, v_out, f32, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mq
