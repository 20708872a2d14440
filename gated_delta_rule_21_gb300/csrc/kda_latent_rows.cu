// kda_latent_rows.cu -- the position rotation, and new tokens into the paged
// cache (kda_rotate, kda_latent_append).
//
// Both move rows once and are bound by memory.  A token's angles serve all its
// heads, so a CTA takes a few tokens, makes their cos and sin once in shared
// memory and then goes over the heads with 16-byte accesses.  8192 tokens of 32 heads
// of 64: 11.3 us, 5.9 TB/s; prompts of 4 x up to 2048 tokens with a latent of 512: 16 to 19 us.
//
// The angle t * f is reduced in integers: f / 2 pi modulo 1 in units of 2^-64, times t
// modulo 2^64, is the fraction of a turn (off by t units at most); what is left goes
// to sincospi in fp32.  (The card's 64-bit floating point is too slow for this: a
// prompt's angles took 5 of 18 us in it.)
#include <string.h>

#include "kda_latent.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;   // of a vector (dim <= 256)

struct RotateParams {
  int B, T, H, dim;
  int pairs, inverse;
  Strides x_s, y_s;
  const void *x;
  const int *positions;
  const float *freq;
  void *y;
  int tokens;            // of a CTA
  // append
  const void *latent, *kr;
  Strides lat_s, kr_s;
  void *cache;
  const int *table, *lengths, *fresh;
  int C, max_pages, n_pages, page;
  long long page_stride, token_stride;
};

// The fraction of a turn that f is worth, in 2^-64: f / 2 pi modulo 1.  f is m 2^(e - 150)
// with 24 bits of m; 1 / 2 pi stands in 126 bits, and the bits of the product from
// 2^-64 up to 2^-1 are cut out.
__device__ __forceinline__ unsigned long long fraction(float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = (int)(u >> 23 & 255u);
  const unsigned long long m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
  // floor(2^128 / 2 pi)
  constexpr unsigned long long hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;
  const unsigned long long p0 = m * lo, p1 = __umul64hi(m, lo), q0 = m * hi, q1 = __umul64hi(m, hi);
  const unsigned long long w0 = p0, w1 = p1 + q0, w2 = q1 + (w1 < p1 ? 1ull : 0ull);
  const int s = 214 - (e ? e : 1);          // the bit of the product that is worth 2^-64
  if (s < 0 || s >= 192) return 0;
  const int k = s & 63;
  const unsigned long long a = s < 64 ? w0 : s < 128 ? w1 : w2;
  const unsigned long long b = s < 64 ? w1 : s < 128 ? w2 : 0ull;
  const unsigned long long r = k ? a >> k | b << (64 - k) : a;
  return u >> 31 ? 0ull - r : r;
}

__device__ __forceinline__ float2 turn(unsigned long long unit, float f, int t, bool inverse) {
  if (!finite(f)) return make_float2(f - f, f - f);
  const long long part = (long long)(unit * (unsigned long long)(long long)t);
  float s, c;
  sincospif((float)part * 0x1p-63f, &s, &c);               // half turns in [-1, 1]
  return make_float2(c, inverse ? -s : s);
}

// N values that are read at once, or (one pair a thread) one by one.
template <typename T, int N, bool kWide>
struct alignas(kWide ? sizeof(T) * N : sizeof(T)) Vec {
  T v[N];
};

// P pairs of a vector: 2 P values side by side, or P of each half.
template <typename T, int P, bool kPairs>
struct Some {
  using Piece = Vec<T, kPairs ? 2 * P : P, (P > 1)>;
  Piece u, v;
  __device__ __forceinline__ void load(const T *x, int i, int half) {
    if (kPairs) {
      u = *reinterpret_cast<const Piece *>(x + 2 * i);
    } else {
      u = *reinterpret_cast<const Piece *>(x + i);
      v = *reinterpret_cast<const Piece *>(x + i + half);
    }
  }
  __device__ __forceinline__ void turn(const float2 *cs) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      T &x = kPairs ? u.v[2 * j] : u.v[j], &y = kPairs ? u.v[2 * j + 1] : v.v[j];
      const float a = to_f32(x), b = to_f32(y);
      x = from_f32<T>(a * cs[j].x - b * cs[j].y);
      y = from_f32<T>(b * cs[j].x + a * cs[j].y);
    }
  }
  __device__ __forceinline__ void store(T *y, int i, int half) const {
    if (kPairs) {
      *reinterpret_cast<Piece *>(y + 2 * i) = u;
    } else {
      *reinterpret_cast<Piece *>(y + i) = u;
      *reinterpret_cast<Piece *>(y + i + half) = v;
    }
  }
};

struct Token {
  long long x, y, kr, lat;   // element offsets of its rows
  long long place;           // in the cache; -1: nowhere
  int at;                    // position; append: -1: not there
};

// P: pairs a thread takes at once (1: any alignment).  kAppend: the tokens' keys and
// latents go to the cache as well.  A thread keeps its pairs and goes over the
// (token, head) rows, four on their way at a time.
template <typename T, int P, bool kPairs, bool kAppend>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateParams p) {
  extern __shared__ float2 cs[];               // [tokens][dim / 2]
  __shared__ Token tok[kThreads];
  const int tid = threadIdx.x, half = p.dim / 2;
  const long long all = (long long)p.B * p.T, first = (long long)blockIdx.x * p.tokens;
  const int n = (int)(all - first < p.tokens ? all - first : p.tokens);
  if (tid < n) {
    const int b = (int)((first + tid) / p.T), t = (int)((first + tid) % p.T);
    Token k;
    k.x = b * p.x_s.b + t * p.x_s.t;
    k.y = b * p.y_s.b + t * p.y_s.t;
    k.at = t;
    if (kAppend) {
      k.kr = b * p.kr_s.b + t * p.kr_s.t;
      k.lat = b * p.lat_s.b + t * p.lat_s.t;
      k.place = k.at = -1;
      const int f = p.fresh ? p.fresh[b] : p.T;
      const int fresh = f < 0 ? 0 : f > p.T ? p.T : f;
      const long long q = (long long)p.lengths[b] - fresh + t;
      if (t < fresh && q >= 0) {
        k.at = (int)q;
        if (q / p.page < p.max_pages) {
          const int pg = p.table[(size_t)b * p.max_pages + q / p.page];
          if (pg >= 0 && pg < p.n_pages)
            k.place = pg * p.page_stride + (q % p.page) * p.token_stride;
        }
      }
    } else if (p.positions) {
      k.at = p.positions[first + tid];
    }
    tok[tid] = k;
  }
  __syncthreads();
  if (p.freq) {
    for (int i = tid; i < n * half; i += kThreads) {
      const float f = p.freq[i % half];
      cs[i] = turn(fraction(f), f, tok[i / half].at, p.inverse != 0);
    }
    __syncthreads();
  }
  using Part = Some<T, P, kPairs>;
  const int steps = half / P;
  if (p.x) {
    const int lanes = steps < kThreads ? steps : kThreads, row0 = tid / lanes,
              step = kThreads / lanes, j = (tid % lanes) * P;
    constexpr int U = 4;
    int k[U], h[U];
    int ck = row0 / p.H, ch = row0 % p.H;
    const int dk = step / p.H, dh = step % p.H;
    const T *x = static_cast<const T *>(p.x);
    T *y = static_cast<T *>(p.y);
    if (row0 < step) {
      while (ck < n) {
        Part part[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          k[u] = ck;
          h[u] = ch;
          if (ck < n) part[u].load(x + tok[ck].x + ch * p.x_s.h, j, half);
          ck += dk;
          ch += dh;
          if (ch >= p.H) ch -= p.H, ++ck;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (k[u] >= n) break;
          const Token &t = tok[k[u]];
          if (!kAppend || t.at >= 0) part[u].turn(cs + k[u] * half + j);
          part[u].store(y + t.y + h[u] * p.y_s.h, j, half);
        }
      }
    }
  }
  if (kAppend) {
    for (int i = tid; i < n * steps; i += kThreads) {
      const int k = i / steps, j = (i % steps) * P;
      if (tok[k].place < 0) continue;
      Part part;
      part.load(static_cast<const T *>(p.kr) + tok[k].kr, j, half);
      if (p.freq) part.turn(cs + k * half + j);
      part.store(static_cast<T *>(p.cache) + tok[k].place + p.C, j, half);
    }
    constexpr int W = P == 1 ? 1 : 16 / (int)sizeof(T);
    using Piece = Vec<T, W, (P > 1)>;
    const int words = p.C / W;
    const int lanes = words < kThreads ? words : kThreads, rows = kThreads / lanes;
    if (tid < rows * lanes) {
      for (int k = tid / lanes; k < n; k += rows) {
        if (tok[k].place < 0) continue;
        const T *x = static_cast<const T *>(p.latent) + tok[k].lat;
        T *y = static_cast<T *>(p.cache) + tok[k].place;
        for (int i = tid % lanes; i < words; i += lanes)
          *reinterpret_cast<Piece *>(y + i * W) = *reinterpret_cast<const Piece *>(x + i * W);
      }
    }
  }
}

bool multiple(const void *p, long long bytes) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0;
}

template <typename T, bool kAppend>
cudaError_t launch(RotateParams p, bool wide, cudaStream_t cs) {
  const int half = p.dim / 2;
  const long long all = (long long)p.B * p.T;
  // as many tokens as make one angle a thread, fewer where SMs would stay idle
  int tokens = half ? kThreads / half : 8;
  if (tokens < 1) tokens = 1;
  const long long fill = (all + 4 * 152 - 1) / (4 * 152);
  if (tokens > fill) tokens = (int)fill;
  p.tokens = tokens;
  const long long grid = (all + tokens - 1) / tokens;
  const size_t smem = sizeof(float2) * (size_t)tokens * half;
  constexpr int P = 8 / (int)sizeof(T);        // pairs in 16 bytes
  const unsigned g = (unsigned)grid;
  if (wide && p.pairs) rotate_kernel<T, P, true, kAppend><<<g, kThreads, smem, cs>>>(p);
  else if (wide) rotate_kernel<T, 2 * P, false, kAppend><<<g, kThreads, smem, cs>>>(p);
  else if (p.pairs) rotate_kernel<T, 1, true, kAppend><<<g, kThreads, smem, cs>>>(p);
  else rotate_kernel<T, 1, false, kAppend><<<g, kThreads, smem, cs>>>(p);
  return cudaGetLastError();
}

// Whether every 16-byte piece of a tensor is aligned.
bool wide_ok(const void *p, const Strides &s, int esize) {
  return multiple(p, 16) && (s.b * esize) % 16 == 0 && (s.t * esize) % 16 == 0 &&
         (s.h * esize) % 16 == 0;
}

// Whether rows of n values lie over each other for a stride of their own.
bool over(long long stride, int count, int n) { return count > 1 && stride < n && stride > -n; }

bool dtype_ok(kda_dtype d) { return d == KDA_DTYPE_F32 || d == KDA_DTYPE_BF16; }

}  // namespace
}  // namespace latent
}  // namespace kda

using namespace kda;
using namespace kda::latent;

extern "C" {

kda_status kda_rotate(const kda_rotate_desc *d, const void *x, const int32_t *positions,
                      const float *inv_freq, void *y, kda_stream_t stream) {
  if (!d || d->B < 1 || d->T < 1 || d->H < 1 || d->dim < 1 || !dtype_ok(d->dtype))
    return KDA_ERR_INVALID_ARG;
  if (!x || !inv_freq || !y) return KDA_ERR_INVALID_ARG;
  if (d->dim % 2 || d->dim > 2 * kMaxPairs) return KDA_ERR_UNSUPPORTED;
  if ((long long)d->B * d->T >= (1ll << 31) || d->H >= (1 << 20)) return KDA_ERR_UNSUPPORTED;
  if (over(d->y_stride_b, d->B, d->dim) || over(d->y_stride_t, d->T, d->dim) ||
      over(d->y_stride_h, d->H, d->dim))
    return KDA_ERR_INVALID_ARG;
  const int es = d->dtype == KDA_DTYPE_BF16 ? 2 : 4;
  if (!multiple(x, es) || !multiple(y, es) || !multiple(inv_freq, 4) || !multiple(positions, 4))
    return KDA_ERR_ALIGNMENT;
  RotateParams p;
  memset(&p, 0, sizeof(p));
  p.B = d->B; p.T = d->T; p.H = d->H; p.dim = d->dim;
  p.pairs = d->pairs; p.inverse = d->inverse;
  p.x_s = strides_of(d->B, d->T, d->H, d->x_stride_b, d->x_stride_t, d->x_stride_h);
  p.y_s = strides_of(d->B, d->T, d->H, d->y_stride_b, d->y_stride_t, d->y_stride_h);
  p.x = x; p.positions = positions; p.freq = inv_freq; p.y = y;
  const bool wide = wide_ok(x, p.x_s, es) && wide_ok(y, p.y_s, es) &&
                    d->dim % ((d->pairs ? 16 : 32) / es) == 0;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = es == 2 ? launch<__nv_bfloat16, false>(p, wide, cs)
                                : launch<float, false>(p, wide, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_latent_append(const kda_latent_cache *s, const void *latent, const void *k_rope,
                             const void *q_rope, const float *inv_freq, int pairs,
                             const int32_t *page_table, const int32_t *lengths,
                             const int32_t *new_tokens, void *cache, void *q_out,
                             kda_stream_t stream) {
  if (!s || s->B < 1 || s->T < 1 || s->H < 1 || s->max_pages < 1 || s->n_pages < 1 ||
      s->page_size < 1 || s->C < 1 || s->R < 0 || !dtype_ok(s->dtype))
    return KDA_ERR_INVALID_ARG;
  if (!latent || !page_table || !lengths || !cache) return KDA_ERR_INVALID_ARG;
  if ((s->R > 0) != (k_rope != nullptr)) return KDA_ERR_INVALID_ARG;
  if ((q_rope != nullptr) != (q_out != nullptr)) return KDA_ERR_INVALID_ARG;
  if (q_rope && !inv_freq) return KDA_ERR_INVALID_ARG;
  if (inv_freq && s->R == 0) return KDA_ERR_INVALID_ARG;
  if (s->C > 4096 || s->R % 2 || s->R > 2 * kMaxPairs) return KDA_ERR_UNSUPPORTED;
  if ((long long)s->B * s->T >= (1ll << 31) || s->H >= (1 << 20)) return KDA_ERR_UNSUPPORTED;
  if (over(s->page_stride, s->n_pages, s->C + s->R) ||
      over(s->token_stride, s->page_size, s->C + s->R))
    return KDA_ERR_INVALID_ARG;
  const int es = s->dtype == KDA_DTYPE_BF16 ? 2 : 4;
  for (const void *ptr : {latent, k_rope, q_rope, (const void *)cache, (const void *)q_out})
    if (!multiple(ptr, es)) return KDA_ERR_ALIGNMENT;
  for (const void *ptr : {(const void *)inv_freq, (const void *)page_table, (const void *)lengths,
                          (const void *)new_tokens})
    if (!multiple(ptr, 4)) return KDA_ERR_ALIGNMENT;
  RotateParams p;
  memset(&p, 0, sizeof(p));
  p.B = s->B; p.T = s->T; p.H = s->H; p.dim = s->R; p.pairs = pairs;
  p.x_s = strides_of(s->B, s->T, s->H, s->q_rope_stride_b, s->q_rope_stride_t, s->q_rope_stride_h);
  p.y_s = {(long long)s->T * s->H * s->R, (long long)s->H * s->R, s->R};
  p.x = q_rope; p.freq = inv_freq; p.y = q_out;
  p.latent = latent; p.kr = k_rope; p.cache = cache;
  p.lat_s = strides_of(s->B, s->T, 1, s->latent_stride_b, s->latent_stride_t, 0);
  p.kr_s = strides_of(s->B, s->T, 1, s->k_rope_stride_b, s->k_rope_stride_t, 0);
  p.table = page_table; p.lengths = lengths; p.fresh = new_tokens;
  p.C = s->C; p.max_pages = s->max_pages; p.n_pages = s->n_pages; p.page = s->page_size;
  p.page_stride = s->n_pages > 1 ? s->page_stride : 0;
  p.token_stride = s->page_size > 1 ? s->token_stride : 0;
  const Strides cache_s = {p.page_stride, p.token_stride, s->C};
  const bool wide = (!q_rope || (wide_ok(q_rope, p.x_s, es) && wide_ok(q_out, p.y_s, es))) &&
                    (!k_rope || wide_ok(k_rope, p.kr_s, es)) && wide_ok(latent, p.lat_s, es) &&
                    wide_ok(cache, cache_s, es) && s->R % ((pairs ? 16 : 32) / es) == 0;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = es == 2 ? launch<__nv_bfloat16, true>(p, wide, cs)
                                : launch<float, true>(p, wide, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
