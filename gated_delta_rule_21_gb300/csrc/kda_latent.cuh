// kda_latent.cuh -- shared by the latent attention's translation units:
// parameter blocks, the division of a cache's tokens over the SMs, and the
// rows that are computed one by one where a product held values that are not
// finite.  Internal to libkda.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_internal.cuh"

namespace kda {
namespace latent {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Strides {
  long long b, t, h;
};
// The stride of a dimension of 1 is not the caller's to say.
inline Strides strides_of(int B, int T, int H, long long b, long long t, long long h) {
  return {B > 1 ? b : 0, T > 1 ? t : 0, H > 1 ? h : 0};
}

// ---- the expanded form ------------------------------------------------------
struct Prompt {
  int B, T, H, K, R, V;
  const void *q, *qr, *k, *kr, *v;
  Strides q_s, qr_s, k_s, kr_s, v_s;     // (kr_s.h is 0)
  float scale;
  int fours;                             // 4 values of a row can be read at once
  // of each token: the first token of its run, and one past the run's last.
  // Padding has start = t + 1, end = t.  NULL: one run a row.  Both rise along
  // a row.
  const int *start, *end;
  void *o;
  float *lse;
  // backward
  const void *d_o;
  const float *delta;                    // [B,H,T]: d_o . o
  void *dq, *dqr, *dk, *dkr, *dv;
  float *dkr_part;                       // [B,T,H,R]: each head's part of dk_rope
  uint32_t *status;
};

__device__ __forceinline__ int run_start(const Prompt &p, int b, int t) {
  return p.start ? p.start[(size_t)b * p.T + t] : 0;
}
__device__ __forceinline__ int run_end(const Prompt &p, int b, int t) {
  return p.end ? p.end[(size_t)b * p.T + t] : p.T;
}

template <typename T>
__device__ __forceinline__ const T *at(const void *base, const Strides &s, int b, int t, int h) {
  return static_cast<const T *>(base) + b * s.b + t * s.t + h * s.h;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A warp's dot product of two rows of n values.
template <typename T>
__device__ __forceinline__ float dot(const T *a, const T *b, int n, int lane) {
  float s = 0.f;
  for (int i = lane; i < n; i += 32) s = fmaf(to_f32(a[i]), to_f32(b[i]), s);
  return s;
}

template <typename T>
__device__ __forceinline__ float score(const Prompt &p, int b, int h, int i, int j, int lane) {
  float s = dot(at<T>(p.q, p.q_s, b, i, h), at<T>(p.k, p.k_s, b, j, h), p.K, lane);
  if (p.R) s += dot(at<T>(p.qr, p.qr_s, b, i, h), at<T>(p.kr, p.kr_s, b, j, 0), p.R, lane);
  return warp_sum(s) * p.scale;
}

// o of a row whose weights sum up to 0: 0 where it sees nothing; where all that it sees has
// a score of minus infinity, which softmax gives no weights, NaN.
__device__ __forceinline__ float no_weights(bool sees) { return sees ? NAN : 0.f; }

// The tiles multiply masked weights of 0 with what stands there, and 0 times
// infinity is NaN.  A row whose sum came out not finite is made again by these,
// key by key over what it sees; a row that is not finite by itself stays so (and is done
// with at its first weight that is NaN).
// One warp a row; V, K <= 128, R <= 64.
template <typename T>
__device__ __noinline__ void forward_row(const Prompt &p, int b, int h, int i, int lane) {
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int start = run_start(p, b, i);
  for (int j = start; j <= i; ++j) {
    const float s = score<T>(p, b, h, i, j, lane);
    const float mn = s > m ? s : m;
    const float c = m == mn ? 1.f : expf(m - mn), w = s == -INFINITY ? 0.f : expf(s - mn);
    const T *v = at<T>(p.v, p.v_s, b, j, h);
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 32 * e < p.V) acc[e] = acc[e] * c + w * to_f32(v[lane + 32 * e]);
    m = mn;
    if (l != l) break;      // so is everything from here on
  }
  T *o = static_cast<T *>(p.o) + (((size_t)b * p.T + i) * p.H + h) * p.V;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < p.V)
      o[lane + 32 * e] = from_f32<T>(l == 0.f ? no_weights(start <= i) : acc[e] / l);
  if (p.lse && lane == 0) p.lse[((size_t)b * p.H + h) * p.T + i] = m + logf(l);
}

// d s_ij without the scale, and p_ij through w.
template <typename T>
__device__ __forceinline__ float dscore(const Prompt &p, int b, int h, int i, int j, int lane,
                                        float &w) {
  const size_t at_i = ((size_t)b * p.H + h) * p.T + i;
  w = expf(score<T>(p, b, h, i, j, lane) - p.lse[at_i]);
  const T *up = static_cast<const T *>(p.d_o) + (((size_t)b * p.T + i) * p.H + h) * p.V;
  const float dp = warp_sum(dot(up, at<T>(p.v, p.v_s, b, j, h), p.V, lane));
  return w * (dp - p.delta[at_i]);
}

template <typename T>
__device__ __noinline__ void query_grad_row(const Prompt &p, int b, int h, int i, int lane) {
  float acc[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = run_start(p, b, i); j <= i; ++j) {
    float w;
    const float ds = dscore<T>(p, b, h, i, j, lane, w);
    const T *k = at<T>(p.k, p.k_s, b, j, h), *kr = at<T>(p.kr, p.kr_s, b, j, 0);
#pragma unroll
    for (int e = 0; e < 6; ++e) {
      const int c = lane + 32 * e;
      if (c < p.K + p.R) acc[e] += ds * to_f32(c < p.K ? k[c] : kr[c - p.K]);
    }
    if (ds != ds) break;
  }
  const size_t row = ((size_t)b * p.T + i) * p.H + h;
  T *dq = static_cast<T *>(p.dq) + row * p.K, *dqr = static_cast<T *>(p.dqr) + row * p.R;
#pragma unroll
  for (int e = 0; e < 6; ++e) {
    const int c = lane + 32 * e;
    if (c < p.K) dq[c] = from_f32<T>(acc[e] * p.scale);
    else if (c < p.K + p.R) dqr[c - p.K] = from_f32<T>(acc[e] * p.scale);
  }
}

template <typename T>
__device__ __noinline__ void key_grad_row(const Prompt &p, int b, int h, int j, int lane) {
  float acc[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, av[4] = {0.f, 0.f, 0.f, 0.f};
  const int end = run_end(p, b, j);
  for (int i = j; i < end; ++i) {
    float w;
    const float ds = dscore<T>(p, b, h, i, j, lane, w);
    const T *q = at<T>(p.q, p.q_s, b, i, h), *qr = at<T>(p.qr, p.qr_s, b, i, h);
    const T *up = static_cast<const T *>(p.d_o) + (((size_t)b * p.T + i) * p.H + h) * p.V;
#pragma unroll
    for (int e = 0; e < 6; ++e) {
      const int c = lane + 32 * e;
      if (c < p.K + p.R) acc[e] += ds * to_f32(c < p.K ? q[c] : qr[c - p.K]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 32 * e < p.V) av[e] += w * to_f32(up[lane + 32 * e]);
    if (w != w) break;
  }
  const size_t row = ((size_t)b * p.T + j) * p.H + h;
  T *dk = static_cast<T *>(p.dk) + row * p.K, *dv = static_cast<T *>(p.dv) + row * p.V;
  float *part = p.dkr_part + row * p.R;
#pragma unroll
  for (int e = 0; e < 6; ++e) {
    const int c = lane + 32 * e;
    if (c < p.K) dk[c] = from_f32<T>(acc[e] * p.scale);
    else if (c < p.K + p.R) part[c - p.K] = acc[e] * p.scale;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < p.V) dv[lane + 32 * e] = from_f32<T>(av[e]);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// ---- the absorbed form ------------------------------------------------------
constexpr int kRows = 32;        // rows (new token, head) that share a pass over the cache
constexpr int kParts = 152;      // CTAs the work is cut for: one for each SM of a GB300

struct Step {
  int B, T, H, C, R;
  int max_pages, n_pages, page;
  int row_tiles;                 // ceil(T * H / kRows)
  int tile;                      // tokens of the cache in one unit of work
  int extra;                     // units that beginning and ending a row tile is worth
  long long page_stride, token_stride;
  const void *q, *qr, *cache;
  Strides q_s, qr_s;
  const int *table, *lengths, *fresh;
  float scale;
  void *o;
  float *lse;
  int2 *plan;                    // [B][row_tiles]: the first and last part of a row tile, the
                                 // first one as its slot; {-1, rows}: it was written whole,
                                 // these of its rows (as bits) without weights
  float *parts;                  // [2 * kParts][kRows][C]: sums, not yet divided
  float *stats;                  // [2 * kParts][kRows][2]: maximum (of scale log2e s) and sum
  uint32_t *status;
};

// Tokens of sequence b that the table has room for, its length, and its new tokens.
struct Seq {
  int length, held, fresh;
};
__device__ __forceinline__ Seq seq_of(const Step &p, int b) {
  Seq s;
  s.length = p.lengths[b];
  const int f = p.fresh ? p.fresh[b] : p.T;
  s.fresh = f < 0 ? 0 : f > p.T ? p.T : f;
  const long long room = (long long)p.max_pages * p.page;
  s.held = s.length < 0 ? 0 : s.length > room ? (int)room : s.length;
  if (s.fresh == 0) s.held = 0;
  return s;
}
// Tokens that row r (new token r / H) of a sequence sees: [0, seen).
__device__ __forceinline__ int seen(const Step &p, const Seq &s, int r) {
  const int t = r / p.H;
  if (t >= s.fresh) return 0;
  const long long n = (long long)s.length - s.fresh + t + 1;
  return n < 0 ? 0 : n > s.held ? s.held : (int)n;
}
__device__ __forceinline__ int tiles_of(const Step &p, const Seq &s) {
  return (s.held + p.tile - 1) / p.tile;
}

// Units are numbered by sequence, row tile and tile of tokens, `extra` ones in front of
// a row tile's first; CTA g takes [begin(g), begin(g + 1)) of `total`.  No CTA between
// two that have work is idle.
__device__ __forceinline__ long long parts_used(long long total) {
  return total < kParts ? total : kParts;
}
__device__ __forceinline__ long long part_begin(long long total, int g) {
  const long long n = parts_used(total);
  return g >= n ? total : total * g / n;
}
__device__ __forceinline__ long long units_of(const Step &p, const Seq &s) {
  return s.held ? (long long)(tiles_of(p, s) + p.extra) * p.row_tiles : 0;
}

// The first unit of this CTA: sequence, and units into it.  All threads call; `tmp`
// has 36 words.
struct Work {
  long long unit, end, total;    // (total: of all CTAs)
  int b;
  long long off;
};
__device__ __forceinline__ Work find_work(const Step &p, long long *tmp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x, g = blockIdx.x;
  long long total = 0;
  if (p.B > n) {            // else one pass over the sequences shows the total too
    for (int b = tid; b < p.B; b += n) total += units_of(p, seq_of(p, b));
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) tmp[warp] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < (n >> 5); ++w) total += tmp[w];
  }
  Work x = {0, 0, 0, 0, 0};
  long long base = 0;
  for (int b0 = 0; b0 < p.B; b0 += n) {
    if (b0 || p.B > n) __syncthreads();
    const int b = b0 + tid;
    const long long mine = b < p.B ? units_of(p, seq_of(p, b)) : 0;
    long long up = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += y;
    }
    if (lane == 31) tmp[warp] = up;
    __syncthreads();
    long long all = base;
    for (int w = 0; w < (n >> 5); ++w) {
      if (w < warp) up += tmp[w];
      all += tmp[w];
    }
    if (p.B <= n) total = all;
    if (b0 == 0) {
      x.unit = part_begin(total, g);
      x.end = part_begin(total, g + 1);
    }
    const long long before = base + up - mine;
    if (mine && x.unit >= before && x.unit < before + mine) {
      tmp[33] = b;
      tmp[34] = x.unit - before;
    }
    base = all;
  }
  __syncthreads();
  x.total = total;
  if (x.unit < x.end) {
    x.b = (int)tmp[33];
    x.off = tmp[34];
  }
  return x;
}

// A sequence's tiles [j0, j0 + n) for the rows of row tile rt.
struct Segment {
  int b, rt, j0, n;
  bool whole;
  int slot;                      // where a part leaves its sums
  Seq s;
};
struct Cursor {
  Work x;
  bool first;
  __device__ __forceinline__ bool next(const Step &p, Segment &g) {
    while (x.unit < x.end) {
      g.s = seq_of(p, x.b);
      if (x.off >= units_of(p, g.s)) {
        ++x.b;
        x.off = 0;
        continue;
      }
      const int tiles = tiles_of(p, g.s), per = tiles + p.extra;
      g.b = x.b;
      g.rt = 0;
      int at = (int)x.off;
      if (p.row_tiles > 1) {
        g.rt = (int)(x.off / per);
        at = (int)(x.off % per);
      }
      const int n = (int)min((long long)(per - at), x.end - x.unit);
      x.unit += n;
      x.off += n;
      g.j0 = max(at - p.extra, 0);
      g.n = max(at + n - p.extra, 0) - g.j0;
      if (g.n == 0) continue;
      g.whole = g.n == tiles;
      // a part that does not begin its CTA's work ends it
      g.slot = 2 * blockIdx.x + (first ? 0 : 1);
      first = false;
      return true;
    }
    return false;
  }
  // What the kernel that joins the parts has to know (one thread).
  __device__ __forceinline__ static void note(const Step &p, const Segment &g) {
    int2 *d = p.plan + (size_t)g.b * p.row_tiles + g.rt;
    if (g.whole) *d = make_int2(-1, 0);
    else if (g.j0 == 0) d->x = g.slot;
    else if (g.j0 + g.n == tiles_of(p, g.s)) d->y = blockIdx.x;
  }
  // Of 16 rows (behind note): what they see is left to that kernel to look up.
  __device__ __forceinline__ static void note_none(const Step &p, const Segment &g, int half,
                                                   unsigned rows) {
    int2 *d = p.plan + (size_t)g.b * p.row_tiles + g.rt;
    reinterpret_cast<unsigned short *>(&d->y)[half] = (unsigned short)rows;
  }
};

// Whether any of the first n tokens of sequence b has a page.  One warp.
inline __device__ __noinline__ bool any_there(const Step &p, int b, int n, int lane) {
  const int pages = n / p.page + (n % p.page != 0);
  for (int i = 0; i < pages; i += 32) {
    const int pg = i + lane < pages ? p.table[(size_t)b * p.max_pages + i + lane] : -1;
    if (__any_sync(0xffffffffu, pg >= 0 && pg < p.n_pages)) return true;
  }
  return false;
}

// The absorbed form's counterpart of forward_row: row r of sequence b, which sees n
// tokens.  One warp.
template <typename T>
__device__ __noinline__ void step_row(const Step &p, int b, int r, int n, int lane) {
  const int t = r / p.H, h = r % p.H;
  const T *q = at<T>(p.q, p.q_s, b, t, h);
  const T *qr = p.R ? at<T>(p.qr, p.qr_s, b, t, h) : nullptr;
  float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  bool any = false;
  for (int j = 0; j < n; ++j) {
    const int pg = p.table[(size_t)b * p.max_pages + j / p.page];
    if (pg < 0 || pg >= p.n_pages) continue;
    any = true;
    const T *c = static_cast<const T *>(p.cache) + pg * p.page_stride +
                 (long long)(j % p.page) * p.token_stride;
    float s = dot(q, c, p.C, lane);
    if (p.R) s += dot(qr, c + p.C, p.R, lane);
    s = warp_sum(s) * p.scale;
    const float mn = s > m ? s : m;
    const float f = m == mn ? 1.f : expf(m - mn), w = s == -INFINITY ? 0.f : expf(s - mn);
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (lane + 32 * e < p.C) acc[e] = acc[e] * f + w * to_f32(c[lane + 32 * e]);
    m = mn;
    if (l != l) break;
  }
  T *o = static_cast<T *>(p.o) + (((size_t)b * p.T + t) * p.H + h) * p.C;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (lane + 32 * e < p.C)
      o[lane + 32 * e] = from_f32<T>(l == 0.f ? no_weights(any) : acc[e] / l);
  if (p.lse && lane == 0) p.lse[((size_t)b * p.H + h) * p.T + t] = m + logf(l);
}

// Rows that see up to so many keys have their D = d_o . o made from the products (tensor
// cores).
constexpr int kExactKeys = 1024;

// ---- launchers --------------------------------------------------------------
bool prompt_tc_ok(const Prompt &p);       // alignment and strides
cudaError_t launch_prompt_tc(const Prompt &p, cudaStream_t s);
cudaError_t launch_prompt_bwd_tc(const Prompt &p, cudaStream_t s);
bool step_tc_ok(const Step &p);           // (bf16) alignment, strides and pages
cudaError_t launch_step_tc(const Step &p, cudaStream_t s);

}  // namespace latent
}  // namespace kda
