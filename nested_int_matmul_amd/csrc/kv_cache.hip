// Rotary positions, and the 8-bit key/value cache: written with its scales
// found on the way, and read back.  All three move bytes: their floor is the
// activations in and the codes (or values) out.
#include "kv_device.h"

namespace mq {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ mq_rope
//
// A thread owns one unit (eight entries, four pairs) of one token and walks
// over `per` heads, so the four float64 sines and cosines (about 45
// instructions a pair) are found once for all of them; their angles do not
// depend on the head.  Lanes of a wave hold consecutive units: 8 or 16 bytes
// each, whole lines together.
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeSpec r, const int* positions,
                                                        const void* x, bool f32, int64_t x_stride,
                                                        int64_t rows, int heads, int dim,
                                                        uint16_t* out, int64_t out_stride,
                                                        int per) {
  const int units = dim >> 3;
  const int slots = kThreads / units;
  const int u = threadIdx.x % units, slot = threadIdx.x / units;
  const int64_t row = (int64_t)blockIdx.x * slots + slot;
  if (slot >= slots || row >= rows) return;
  const Unit un = unit_of(u, r.rot, r.interleaved);
  double c[4], s[4];
  if (un.turns) {
    const double pos = (double)positions[row];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sincos64(pos * r.freq[un.pair0 + i], &s[i], &c[i]);
      s[i] *= r.factor;
      c[i] *= r.factor;
    }
  }
  const int h0 = blockIdx.y * per, h1 = h0 + per < heads ? h0 + per : heads;
  for (int h = h0; h < h1; ++h) {
    float v[8];
    load_unit(x, f32, row * x_stride + (int64_t)h * dim, un, v);
    if (un.turns) turn_unit(v, c, s, r.interleaved);
    uint32_t w[4];
    pack_unit(v, w);
    uint16_t* o = out + row * out_stride + (int64_t)h * dim;
    *reinterpret_cast<u32x2*>(o + un.lo) = u32x2{w[0], w[1]};
    *reinterpret_cast<u32x2*>(o + un.hi) = u32x2{w[2], w[3]};
  }
}

hipError_t launch_rope(const RopeSpec& r, const int* positions, const void* x, bool f32,
                       int64_t x_stride, int64_t rows, int heads, int dim, uint16_t* out,
                       int64_t out_stride, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int slots = kThreads / (dim / 8);
  const int64_t groups = (rows + slots - 1) / slots;
  // heads of a thread: as many as leave 2048 workgroups (eight a CU)
  int per = 16;
  while (per > 1 && groups * ((heads + per - 1) / per) < 2048) per >>= 1;
  while ((heads + per - 1) / per > 65535) per <<= 1;
  const dim3 grid((unsigned)groups, (unsigned)((heads + per - 1) / per));
  hipLaunchKernelGGL(rope_kernel, grid, dim3(kThreads), 0, s, r, positions, x, f32, x_stride,
                     rows, heads, dim, out, out_stride, per);
  return hipGetLastError();
}

// --------------------------------------------------------- mq_cache_append
//
// One workgroup per (sequence, page that gets tokens, head, k or v): the
// page's new values stay in registers as bf16 (at most 64 dwords a thread)
// between finding the scale and rounding to codes, so they are read once, and
// no other workgroup touches the page's scale or codes.  A thread owns one
// unit of every (256 / units)-th token; k's angles of a thread advance by a
// constant step, so its sines and cosines follow by one complex product a
// token in float64 (error below 2^-48 over a page) in place of an evaluation.
// v is held dim-major: pages that get 16 tokens or more go through LDS and
// leave in 16-byte pieces, fewer tokens go out as single bytes.
//
// The queries' workgroups (blockIdx.y >= 2 * heads) take eight tokens of the
// same page each, all heads.

// eight tokens of one page, all query heads
template <int DIM>
__device__ __forceinline__ void append_queries(const KvBatch& b, const RopeSpec& r,
                                               const SeqSpan& sp, int64_t lo, int64_t hi,
                                               const void* q, int64_t q_stride, int q_heads,
                                               bool f32, uint16_t* q_out) {
  constexpr int U = DIM / 8, SLOTS = kThreads / U;
  const int u = threadIdx.x % U, slot = threadIdx.x / U;
  const int hs = q_heads < SLOTS ? q_heads : SLOTS;  // heads side by side
  const int toks = SLOTS / hs;                       // tokens side by side
  const int head0 = slot % hs, tok0 = slot / hs;
  if (tok0 >= toks) return;
  const Unit un = unit_of(u, r.rot, r.interleaved);
  const bool turns = r.freq && un.turns;
  for (int64_t pos = lo + tok0; pos < hi; pos += toks) {
    double c[4], s[4];
    if (turns) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sincos64((double)pos * r.freq[un.pair0 + i], &s[i], &c[i]);
        s[i] *= r.factor;
        c[i] *= r.factor;
      }
    }
    const int64_t row = sp.row0 + (pos - sp.start);
    for (int h = head0; h < q_heads; h += hs) {
      float v[8];
      load_unit(q, f32, row * q_stride + (int64_t)h * DIM, un, v);
      if (turns) turn_unit(v, c, s, r.interleaved);
      uint32_t w[4];
      pack_unit(v, w);
      uint16_t* o = q_out + (row * q_heads + h) * DIM;
      *reinterpret_cast<u32x2*>(o + un.lo) = u32x2{w[0], w[1]};
      *reinterpret_cast<u32x2*>(o + un.hi) = u32x2{w[2], w[3]};
    }
  }
}

constexpr int kQueryTokens = 8;

// a bf16 pattern's value as a quotient's dividend, and whether it is a number
__device__ __forceinline__ float code_quotient(uint32_t bits, float s, float rs) {
  const uint32_t mag = bits & 0x7fffu;
  if (mag >= 0x7f80u)  // infinity: beyond every code, NaN: 0
    return mag > 0x7f80u ? 0.f : ((bits & 0x8000u) ? -1e9f : 1e9f);
  return exact_quotient(__uint_as_float(bits << 16), s, rs);
}

template <int DIM, int BLOCK>
__global__ void __launch_bounds__(kThreads) append_kernel(KvCache cache, KvBatch b, RopeSpec r,
                                                          const void* k, const void* v,
                                                          int64_t kv_stride, const void* q,
                                                          int64_t q_stride, int q_heads, bool f32,
                                                          uint16_t* q_out) {
  constexpr int U = DIM / 8, SLOTS = kThreads / U;
  constexpr int STEPS = BLOCK / SLOTS > 0 ? BLOCK / SLOTS : 1;
  constexpr int PITCH = BLOCK + 4;  // bytes of a dim's row in LDS
  __shared__ uint32_t tile[DIM * PITCH / 4];
  __shared__ uint32_t wave_max[kThreads / 64];

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
    if (lo < hi) append_queries<DIM>(b, r, sp, lo, hi, q, q_stride, q_heads, f32, q_out);
    return;
  }
  const int page = page_of(b, seq, pi, cache.pages);
  if (page < 0) return;
  const int head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const bool e4m3 = cache.e4m3;
  const int tid = threadIdx.x, u = tid % U, slot = tid / U;
  const int64_t ph = (int64_t)page * cache.heads + head;
  float* scale_at = (is_v ? cache.v_scale : cache.k_scale) + ph;
  uint8_t* codes = (is_v ? cache.v : cache.k) + ph * (DIM * BLOCK);
  const int used = (int)(lo - base);  // earlier tokens of the page
  const int fill = (int)(hi - base);
  const float was = used > 0 ? *scale_at : 0.f;

  // ---- the page's new values as bf16, and their largest magnitude
  const Unit un = is_v ? unit_of(u, 0, false) : unit_of(u, r.freq ? r.rot : 0, r.interleaved);
  uint32_t w[STEPS][4];
  uint32_t top = 0;
  double c[4], s[4], dc[4], ds[4];
  if (un.turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double f = r.freq[un.pair0 + i];
      sincos64((double)(base + slot) * f, &s[i], &c[i]);
      s[i] *= r.factor;
      c[i] *= r.factor;
      if (STEPS > 1) sincos64((double)SLOTS * f, &ds[i], &dc[i]);
    }
  }
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int t = slot + j * SLOTS;
    if (t >= used && t < fill) {
      float x[8];
      const int64_t row = sp.row0 + (base + t - sp.start);
      load_unit(is_v ? v : k, f32, row * kv_stride + (int64_t)head * DIM, un, x);
      if (un.turns) turn_unit(x, c, s, r.interleaved);
      pack_unit(x, w[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[j][i] & 0x7fffu, d = (w[j][i] >> 16) & 0x7fffu;
        top = a < 0x7f80u && a > top ? a : top;
        top = d < 0x7f80u && d > top ? d : top;
      }
    }
    if (un.turns && j + 1 < STEPS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double nc = c[i] * dc[i] - s[i] * ds[i];
        s[i] = s[i] * dc[i] + c[i] * ds[i];
        c[i] = nc;
      }
    }
  }
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = __shfl_xor(top, off);
    top = o > top ? o : top;
  }
  if ((tid & 63) == 0) wave_max[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) top = wave_max[i] > top ? wave_max[i] : top;
  float now = __uint_as_float(top << 16) * kv_inv_qmax(e4m3);
  if (now < kMinScale) now = 0.f;
  const bool grows = used > 0 && now > was;
  if (used > 0 && !grows) now = was;
  if (tid == 0) *scale_at = now;

  // ---- earlier codes, where the scale grows
  if (grows) {
    if (!is_v) {
      for (int i = tid; i < used * (DIM / 4); i += kThreads) {
        uint32_t* p = reinterpret_cast<uint32_t*>(codes) + i;
        *p = recode(*p, e4m3, was, now);
      }
    } else {
      // four tokens of a dim at a time; those at or beyond `used` keep their
      // bytes here (this workgroup writes them below)
      const int per = (used + 3) / 4;
      for (int i = tid; i < per * DIM; i += kThreads) {
        const int d = i / per, t = (i % per) * 4;
        uint32_t* p = reinterpret_cast<uint32_t*>(codes + d * BLOCK + t);
        const uint32_t before = *p, after = recode(before, e4m3, was, now);
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
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int t = slot + j * SLOTS;
    if (t < used || t >= fill) continue;
    uint32_t out[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t pair = w[j][2 * half + (i >> 1)];
        const uint32_t bits = (i & 1) ? pair >> 16 : pair & 0xffffu;
        y[i] = now > 0.f ? code_quotient(bits, now, rs) : 0.f;
      }
      out[half] = codes_of(y, e4m3);
    }
    if (!is_v) {
      *reinterpret_cast<uint32_t*>(codes + t * DIM + un.lo) = out[0];
      *reinterpret_cast<uint32_t*>(codes + t * DIM + un.hi) = out[1];
    } else {
      uint8_t* to = through_lds ? reinterpret_cast<uint8_t*>(tile) : codes;
      const int pitch = through_lds ? PITCH : BLOCK;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        to[(8 * u + i) * pitch + t] = (uint8_t)(out[i >> 2] >> (8 * (i & 3)));
    }
  }
  if (!through_lds) return;
  __syncthreads();
  for (int i = tid; i < DIM * (BLOCK / 16); i += kThreads) {
    const int d = i / (BLOCK / 16), t = (i % (BLOCK / 16)) * 16;
    if (t + 16 <= used || t >= fill) continue;
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = tile[(d * PITCH + t) / 4 + e];
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
    hipLaunchKernelGGL((append_kernel<DIM, BLOCK>), grid, dim3(kThreads), 0, s, c, b, r, k, v,  \
                       kv_stride, q, q_stride, q_heads, f32, q_out);                            \
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
// One workgroup per (sequence, page, head, k or v).  Four codes a load; v is
// turned from dim-major through LDS.
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
