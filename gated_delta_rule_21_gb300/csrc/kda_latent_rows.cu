// kda_latent_rows.cu -- the position rotation, and new tokens into the paged
// cache (kda_rotate, kda_latent_append).
//
// Both move rows once and are bound by memory.  A token's angles serve all its
// heads, so a CTA takes a few tokens, makes their cos and sin once in shared
// memory and then goes over the heads with 16-byte accesses.
//
// The angle t * f is reduced in integers: f / 2 pi modulo 1 as a fraction of
// 2^64, times t modulo 2^64, is the turn exactly but for the 53 bits of
// f / 2 pi; what is left goes to sincospi in fp32.
#include <string.h>

#include "kda_latent.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;   // of a vector (dim <= 256)
constexpr double kInv2Pi = 0.15915494309189533577;

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

__device__ __forceinline__ float2 turn(float f, int t, bool inverse) {
  if (!finite(f)) return make_float2(f - f, f - f);
  const double r = (double)f * kInv2Pi;
  const double frac = r - floor(r);                        // [0, 1)
  const unsigned long long unit =                          // of 2^64, in two halves
      ((unsigned long long)(frac * 4294967296.0) << 32) |
      (unsigned long long)((frac * 4294967296.0 - floor(frac * 4294967296.0)) * 4294967296.0);
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

// P pairs from pair i of a vector, rotated (cs NULL: copied).
template <typename T, int P>
__device__ __forceinline__ void rotate_pairs(const T *x, T *y, int i, int dim, int pairs,
                                             const float2 *cs) {
  float a[P], b[P];
  using Pairs = Vec<T, 2 * P, (P > 1)>;
  using Half = Vec<T, P, (P > 1)>;
  if (pairs) {
    const Pairs v = *reinterpret_cast<const Pairs *>(x + 2 * i);
    Pairs w;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      a[j] = to_f32(v.v[2 * j]);
      b[j] = to_f32(v.v[2 * j + 1]);
      const float2 z = cs ? cs[i + j] : make_float2(1.f, 0.f);
      w.v[2 * j] = cs ? from_f32<T>(a[j] * z.x - b[j] * z.y) : v.v[2 * j];
      w.v[2 * j + 1] = cs ? from_f32<T>(b[j] * z.x + a[j] * z.y) : v.v[2 * j + 1];
    }
    *reinterpret_cast<Pairs *>(y + 2 * i) = w;
  } else {
    const Half u = *reinterpret_cast<const Half *>(x + i);
    const Half v = *reinterpret_cast<const Half *>(x + i + dim / 2);
    Half lo, hi;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      a[j] = to_f32(u.v[j]);
      b[j] = to_f32(v.v[j]);
      const float2 z = cs ? cs[i + j] : make_float2(1.f, 0.f);
      lo.v[j] = cs ? from_f32<T>(a[j] * z.x - b[j] * z.y) : u.v[j];
      hi.v[j] = cs ? from_f32<T>(b[j] * z.x + a[j] * z.y) : v.v[j];
    }
    *reinterpret_cast<Half *>(y + i) = lo;
    *reinterpret_cast<Half *>(y + i + dim / 2) = hi;
  }
}

// P: pairs a thread takes at once (1: any alignment).  kAppend: the tokens'
// keys and latents go to the cache as well.
template <typename T, int P, bool kAppend>
__global__ void __launch_bounds__(kThreads) rotate_kernel(RotateParams p) {
  extern __shared__ float2 cs[];               // [tokens][dim / 2]
  __shared__ int pos[kThreads];
  __shared__ long long place[kThreads];        // of a token in the cache, -1: nowhere
  const int tid = threadIdx.x, half = p.dim / 2;
  const long long all = (long long)p.B * p.T, first = (long long)blockIdx.x * p.tokens;
  const int n = (int)(all - first < p.tokens ? all - first : p.tokens);
  if (tid < n) {
    const int b = (int)((first + tid) / p.T), t = (int)((first + tid) % p.T);
    int at = t;
    if (kAppend) {
      const int f = p.fresh ? p.fresh[b] : p.T;
      const int fresh = f < 0 ? 0 : f > p.T ? p.T : f;
      const long long q = (long long)p.lengths[b] - fresh + t;
      long long where = -1;
      at = -1;
      if (t < fresh && q >= 0) {
        at = (int)q;
        if (q / p.page < p.max_pages) {
          const int pg = p.table[(size_t)b * p.max_pages + q / p.page];
          if (pg >= 0 && pg < p.n_pages)
            where = pg * p.page_stride + (q % p.page) * p.token_stride;
        }
      }
      place[tid] = where;
    } else if (p.positions) {
      at = p.positions[first + tid];
    }
    pos[tid] = at;
  }
  __syncthreads();
  if (p.freq)
    for (int i = tid; i < n * half; i += kThreads)
      cs[i] = turn(p.freq[i % half], pos[i / half], p.inverse != 0);
  __syncthreads();
  if (p.x) {
    const int steps = half / P, row = p.H * steps;
    for (long long i = tid; i < (long long)n * row; i += kThreads) {
      const int k = (int)(i / row), r = (int)(i % row), h = r / steps, j = (r % steps) * P;
      const int b = (int)((first + k) / p.T), t = (int)((first + k) % p.T);
      const bool turned = p.freq && (!kAppend || pos[k] >= 0);
      rotate_pairs<T, P>(static_cast<const T *>(p.x) + b * p.x_s.b + t * p.x_s.t + h * p.x_s.h,
                         static_cast<T *>(p.y) + b * p.y_s.b + t * p.y_s.t + h * p.y_s.h, j,
                         p.dim, p.pairs, turned ? cs + k * half : nullptr);
    }
  }
  if (kAppend) {
    const int steps = half / P;
    for (int i = tid; i < n * steps; i += kThreads) {
      const int k = i / steps, j = (i % steps) * P;
      if (place[k] < 0) continue;
      const int b = (int)((first + k) / p.T), t = (int)((first + k) % p.T);
      rotate_pairs<T, P>(static_cast<const T *>(p.kr) + b * p.kr_s.b + t * p.kr_s.t,
                         static_cast<T *>(p.cache) + place[k] + p.C, j, p.dim, p.pairs,
                         p.freq ? cs + k * half : nullptr);
    }
    constexpr int W = P == 1 ? 1 : 16 / (int)sizeof(T);
    const int words = p.C / W;
    for (int i = tid; i < n * words; i += kThreads) {
      const int k = i / words, j = (i % words) * W;
      if (place[k] < 0) continue;
      const int b = (int)((first + k) / p.T), t = (int)((first + k) % p.T);
      using Piece = Vec<T, W, (P > 1)>;
      *reinterpret_cast<Piece *>(static_cast<T *>(p.cache) + place[k] + j) =
          *reinterpret_cast<const Piece *>(static_cast<const T *>(p.latent) + b * p.lat_s.b +
                                           t * p.lat_s.t + j);
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
  if (wide && p.pairs) rotate_kernel<T, P, kAppend><<<(unsigned)grid, kThreads, smem, cs>>>(p);
  else if (wide) rotate_kernel<T, 2 * P, kAppend><<<(unsigned)grid, kThreads, smem, cs>>>(p);
  else rotate_kernel<T, 1, kAppend><<<(unsigned)grid, kThreads, smem, cs>>>(p);
  return cudaGetLastError();
}

// Whether every 16-byte piece of a tensor is aligned.
bool wide_ok(const void *p, const Strides &s, int esize) {
  return multiple(p, 16) && (s.b * esize) % 16 == 0 && (s.t * esize) % 16 == 0 &&
         (s.h * esize) % 16 == 0;
}

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
  const int es = d->dtype == KDA_DTYPE_BF16 ? 2 : 4;
  if (!multiple(x, es) || !multiple(y, es) || !multiple(inv_freq, 4) || !multiple(positions, 4))
    return KDA_ERR_ALIGNMENT;
  RotateParams p;
  memset(&p, 0, sizeof(p));
  p.B = d->B; p.T = d->T; p.H = d->H; p.dim = d->dim;
  p.pairs = d->pairs; p.inverse = d->inverse;
  p.x_s = {d->x_stride_b, d->x_stride_t, d->x_stride_h};
  p.y_s = {d->y_stride_b, d->y_stride_t, d->y_stride_h};
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
  const int es = s->dtype == KDA_DTYPE_BF16 ? 2 : 4;
  for (const void *ptr : {latent, k_rope, q_rope, (const void *)cache, (const void *)q_out})
    if (!multiple(ptr, es)) return KDA_ERR_ALIGNMENT;
  for (const void *ptr : {(const void *)inv_freq, (const void *)page_table, (const void *)lengths,
                          (const void *)new_tokens})
    if (!multiple(ptr, 4)) return KDA_ERR_ALIGNMENT;
  RotateParams p;
  memset(&p, 0, sizeof(p));
  p.B = s->B; p.T = s->T; p.H = s->H; p.dim = s->R; p.pairs = pairs;
  p.x_s = {s->q_rope_stride_b, s->q_rope_stride_t, s->q_rope_stride_h};
  p.y_s = {(long long)s->T * s->H * s->R, (long long)s->H * s->R, s->R};
  p.x = q_rope; p.freq = inv_freq; p.y = q_out;
  p.latent = latent; p.kr = k_rope; p.cache = cache;
  p.lat_s = {s->latent_stride_b, s->latent_stride_t, 0};
  p.kr_s = {s->k_rope_stride_b, s->k_rope_stride_t, 0};
  p.table = page_table; p.lengths = lengths; p.fresh = new_tokens;
  p.C = s->C; p.max_pages = s->max_pages; p.n_pages = s->n_pages; p.page = s->page_size;
  p.page_stride = s->page_stride; p.token_stride = s->token_stride;
  const Strides cache_s = {s->page_stride, s->token_stride, s->C};
  const bool wide = (!q_rope || (wide_ok(q_rope, p.x_s, es) && wide_ok(q_out, p.y_s, es))) &&
                    (!k_rope || wide_ok(k_rope, p.kr_s, es)) && wide_ok(latent, p.lat_s, es) &&
                    wide_ok(cache, cache_s, es) && s->R % ((pairs ? 16 : 32) / es) == 0;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = es == 2 ? launch<__nv_bfloat16, true>(p, wide, cs)
                                : launch<float, true>(p, wide, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
