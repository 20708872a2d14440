// kda_latent.cu -- the expanded latent attention: entry points, the table of
// runs, the small kernels around the backward, and the fp32 kernels on the
// CUDA cores, which serve every type and layout.
//
// CUDA cores: a CTA of 512 threads holds 64 queries (forward, gradient of the
// queries) or 64 keys (gradients of keys and values) of one head in shared
// memory as fp32 and walks the other side in tiles of 64.  A thread makes a
// 2 x 4 piece of the tile of scores with packed multiply-adds (two terms of the
// sum at once) and 2 rows of the outputs.  What bounds it: the way of the longest
// row, tile after tile.  Rows of 997 tokens, 18 heads of 64 + 32: 392 us forward and
// backward (256 threads, one stage and the two gradients one after the other 971).
#include <string.h>

#include "kda_f32x2.cuh"
#include "kda_latent.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kThreads = 512;
constexpr int kBlk = 64;          // rows of a tile, either side
constexpr int kRt = 2;            // rows of a thread
constexpr int kLdP = kBlk + 4;    // of a tile of weights

__device__ __forceinline__ float4 four(const float *x) {
  return *reinterpret_cast<const float4 *>(x);
}
__device__ __forceinline__ float4 four(const __nv_bfloat16 *x) {
  const uint2 u = *reinterpret_cast<const uint2 *>(x);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

// Rows of one head, [x | xr] of n and nr values; fours: 4 values can be read at once.
template <typename T>
struct Side {
  const T *x, *xr;
  long long st, str;
  int n, nr, fours;
  // Rows t0 .. t0 + 63 as fp32, zeros from row `lim` on, 16 threads a row.  fp32 values
  // come by asynchronous copies.
  __device__ __forceinline__ void load(float *dst, int ld, int t0, int lim) const {
    const int w = n + nr, r0 = threadIdx.x >> 4, c0 = 4 * (threadIdx.x & 15);
#pragma unroll
    for (int i = 0; i < kRt; ++i) {
      const int r = r0 + kThreads / 16 * i, t = t0 + r;
      const T *a = x + t * st, *b = xr + t * str - n;
      for (int c = c0; c < w; c += 64) {
        const T *y = (c < n ? a : b) + c;
        float *d = dst + r * ld + c;
        if (sizeof(T) == 4 && fours) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           (uint32_t)__cvta_generic_to_shared(d)),
                       "l"(t < lim ? y : x), "r"(t < lim ? 16 : 0)
                       : "memory");
        } else {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (t < lim)
            v = fours ? four(y)
                      : make_float4(to_f32(y[0]), to_f32(y[1]), to_f32(y[2]), to_f32(y[3]));
          *reinterpret_cast<float4 *>(d) = v;
        }
      }
    }
  }
};
template <typename T>
__device__ __forceinline__ Side<T> keys_side(const Prompt &p, int b, int h) {
  return {at<T>(p.k, p.k_s, b, 0, h), at<T>(p.kr, p.kr_s, b, 0, 0), p.k_s.t, p.kr_s.t, p.K, p.R,
          p.fours};
}
template <typename T>
__device__ __forceinline__ Side<T> queries_side(const Prompt &p, int b, int h) {
  return {at<T>(p.q, p.q_s, b, 0, h), at<T>(p.qr, p.qr_s, b, 0, h), p.q_s.t, p.qr_s.t, p.K, p.R,
          p.fours};
}
template <typename T>
__device__ __forceinline__ Side<T> values_side(const Prompt &p, int b, int h) {
  return {at<T>(p.v, p.v_s, b, 0, h), nullptr, p.v_s.t, 0, p.V, 0, p.fours};
}
template <typename T>
__device__ __forceinline__ Side<T> up_side(const Prompt &p, int b, int h) {
  return {static_cast<const T *>(p.d_o) + ((size_t)b * p.T * p.H + h) * p.V, nullptr,
          (long long)p.H * p.V, 0, p.V, 0, 1};
}
__device__ __forceinline__ void copies_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last `kBut` groups are in.
template <int kBut>
__device__ __forceinline__ void copies_in() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kBut) : "memory");
}

// The other side's tiles from t0 up to `last`: while work(t, stage) goes over one, the next
// one is on its way where the shared memory has two stages.
template <typename L, typename W>
__device__ __forceinline__ void walk(int t0, int last, int stages, L load, W work) {
  int st = 0;
  if (t0 < last) load(t0, 0);
  copies_sent();
  for (; t0 < last; t0 += kBlk) {
    const bool more = t0 + kBlk < last;
    if (stages == 2) {
      if (more) load(t0 + kBlk, st ^ 1);
      copies_sent();
      copies_in<1>();
    } else {
      copies_in<0>();
    }
    __syncthreads();
    work(t0, st);
    __syncthreads();
    if (stages == 2) {
      st ^= 1;
    } else if (more) {
      load(t0 + kBlk, 0);
      copies_sent();
    }
  }
  copies_in<0>();
}

// s[i][j] = sum_c a[2 ty + i][c] b[tx + 16 j][c] over n (a multiple of 4) values.
__device__ __forceinline__ void rows_by_rows(const float *a, int lda, const float *b, int ldb,
                                             int n, int ty, int tx, float (&s)[kRt][4]) {
  u64 acc[kRt][4];
#pragma unroll
  for (int i = 0; i < kRt; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
  a += kRt * ty * lda;
  b += tx * ldb;
#pragma unroll 2
  for (int c = 0; c < n; c += 4) {
    ulonglong2 x[kRt], y[4];
#pragma unroll
    for (int i = 0; i < kRt; ++i) x[i] = *reinterpret_cast<const ulonglong2 *>(a + i * lda + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2 *>(b + 16 * j * ldb + c);
#pragma unroll
    for (int i = 0; i < kRt; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fma2(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fma2(x[i].y, y[j].y, acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < kRt; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      upk2(acc[i][j], lo, hi);
      s[i][j] = lo + hi;
    }
}

// acc[i][q] += sum_k w[2 ty + i][k] y[k][4 tx + 64 q ..] over the tile's 64 k, for q < N.
template <int N, int M>
__device__ __forceinline__ void weights_by_some(const float *w, const float *y, int ld, int n,
                                                int ty, int tx, u64 (&acc)[kRt][M][2]) {
  w += kRt * ty * kLdP;
  const float *at[N];
#pragma unroll
  for (int q = 0; q < N; ++q) at[q] = y + 4 * tx + 64 * q;
  if (4 * tx + 64 * (N - 1) >= n) at[N - 1] = y;     // (its sums are not used)
#pragma unroll 2
  for (int k = 0; k < kBlk; k += 4) {
    float4 c[kRt];
#pragma unroll
    for (int i = 0; i < kRt; ++i) c[i] = *reinterpret_cast<const float4 *>(w + i * kLdP + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(at[q] + (k + kk) * ld);
#pragma unroll
        for (int i = 0; i < kRt; ++i) {
          const float f = kk == 0 ? c[i].x : kk == 1 ? c[i].y : kk == 2 ? c[i].z : c[i].w;
          const u64 ff = pk2(f, f);
          acc[i][q][0] = fma2(ff, v.x, acc[i][q][0]);
          acc[i][q][1] = fma2(ff, v.y, acc[i][q][1]);
        }
      }
  }
}
template <int M>
__device__ __forceinline__ void weights_by_rows(const float *w, const float *y, int ld, int n,
                                                int ty, int tx, u64 (&acc)[kRt][M][2]) {
  if (n <= 64) weights_by_some<1>(w, y, ld, n, ty, tx, acc);
  else if (n <= 128) weights_by_some<2>(w, y, ld, n, ty, tx, acc);
  else if (M > 2) weights_by_some<M>(w, y, ld, n, ty, tx, acc);
}

template <int N>
__device__ __forceinline__ void clear(u64 (&acc)[kRt][N][2]) {
#pragma unroll
  for (int i = 0; i < kRt; ++i)
#pragma unroll
    for (int q = 0; q < N; ++q) acc[i][q][0] = acc[i][q][1] = 0;
}

// Maximum and sum over the 16 threads that share rows.
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A CTA's tile, head and row; the longest rows of tiles come first.
struct Where {
  int t0, h, b;
};
__device__ __forceinline__ Where where(const Prompt &p, bool last_first) {
  const int tiles = (p.T + kBlk - 1) / kBlk;
  const unsigned x = blockIdx.x, per = (unsigned)(p.B * p.H);
  const int tile = (int)(x / per), r = (int)(x % per);
  return {(last_first ? tiles - 1 - tile : tile) * kBlk, r % p.H, r / p.H};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) prompt_fwd_kernel(const Prompt p, int stages) {
  extern __shared__ __align__(16) float sm[];
  const int D = p.K + p.R, ldq = D + 4, ldv = p.V + 4;
  float *sq = sm, *sp = sq + kBlk * ldq, *ring = sp + kBlk * kLdP;
  const int stage = kBlk * (ldq + ldv);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Where at0 = where(p, true);
  const int b = at0.b, h = at0.h, t0 = at0.t0;
  const Side<T> keys = keys_side<T>(p, b, h), values = values_side<T>(p, b, h);
  queries_side<T>(p, b, h).load(sq, ldq, t0, p.T);
  int lo[kRt];
#pragma unroll
  for (int i = 0; i < kRt; ++i)
    lo[i] = t0 + kRt * ty + i < p.T ? run_start(p, b, t0 + kRt * ty + i) : 0x7fffffff;
  float m[kRt], l[kRt];
  u64 acc[kRt][2][2];
  clear(acc);
#pragma unroll
  for (int i = 0; i < kRt; ++i) m[i] = -INFINITY, l[i] = 0.f;
  const float scale = p.scale * kLog2e;
  const int last = min(p.T, t0 + kBlk);
  auto load = [&](int j0, int st) {
    keys.load(ring + st * stage, ldq, j0, p.T);
    values.load(ring + st * stage + kBlk * ldq, ldv, j0, p.T);
  };
  walk(run_start(p, b, t0) / kBlk * kBlk, last, stages, load, [&](int j0, int st) {
    const float *sk = ring + st * stage, *sv = sk + kBlk * ldq;
    float s[kRt][4];
    rows_by_rows(sq, ldq, sk, ldq, D, ty, tx, s);
#pragma unroll
    for (int i = 0; i < kRt; ++i) {
      const int t = t0 + kRt * ty + i;
      float top = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = j0 + tx + 16 * j;
        s[i][j] = k >= lo[i] && k <= t ? s[i][j] * scale : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
      top = row_max(top);
      const float base = top == -INFINITY ? 0.f : top, f = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = exp2f(s[i][j] - base);
        sum += w;
        sp[(kRt * ty + i) * kLdP + tx + 16 * j] = w;
      }
      l[i] = l[i] * f + row_sum(sum);
      m[i] = top;
      const u64 ff = pk2(f, f);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        acc[i][q][0] = mul2(acc[i][q][0], ff);
        acc[i][q][1] = mul2(acc[i][q][1], ff);
      }
    }
    __syncwarp();   // the rows of a warp are its own
    weights_by_rows(sp, sv, ldv, p.V, ty, tx, acc);
  });
#pragma unroll
  for (int i = 0; i < kRt; ++i) {
    const int t = t0 + kRt * ty + i;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i], none = no_weights(lo[i] <= t);
    bool bad = false;
    if (t < p.T) {
      T *o = static_cast<T *>(p.o) + (((size_t)b * p.T + t) * p.H + h) * p.V;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (4 * tx + 64 * q >= p.V) continue;
        float x[4];
        upk2(acc[i][q][0], x[0], x[1]);
        upk2(acc[i][q][1], x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = l[i] == 0.f ? none : x[e] * inv;
          bad |= !finite(y);
          o[4 * tx + 64 * q + e] = from_f32<T>(y);
        }
      }
      if (p.lse && tx == 0)
        p.lse[((size_t)b * p.H + h) * p.T + t] =
            l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
    const unsigned which = __ballot_sync(0xffffffffu, bad);
    __syncwarp();
    if (which & 0xffffu) forward_row<T>(p, b, h, t0 + 2 * kRt * (tid >> 5) + i, tid & 31);
    if (which & 0xffff0000u) forward_row<T>(p, b, h, t0 + 2 * kRt * (tid >> 5) + kRt + i, tid & 31);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) prompt_dkv_kernel(const Prompt p, int stages) {
  extern __shared__ __align__(16) float sm[];
  start_next();
  const int D = p.K + p.R, ldq = D + 4, ldv = p.V + 4;
  float *sk = sm, *sv = sk + kBlk * ldq, *sp = sv + kBlk * ldv, *sd = sp + kBlk * kLdP,
        *ring = sd + kBlk * kLdP;
  const int stage = kBlk * (ldq + ldv);
  __shared__ float s_lse[2][kBlk], s_delta[2][kBlk];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Where at0 = where(p, false);
  const int b = at0.b, h = at0.h, t0 = at0.t0;
  const Side<T> queries = queries_side<T>(p, b, h), up = up_side<T>(p, b, h);
  keys_side<T>(p, b, h).load(sk, ldq, t0, p.T);
  values_side<T>(p, b, h).load(sv, ldv, t0, p.T);
  int end[kRt];
#pragma unroll
  for (int i = 0; i < kRt; ++i)
    end[i] = t0 + kRt * ty + i < p.T ? run_end(p, b, t0 + kRt * ty + i) : 0;
  const int last = run_end(p, b, min(p.T, t0 + kBlk) - 1);
  u64 ak[kRt][3][2], av[kRt][2][2];
  clear(ak);
  clear(av);
  const float scale = p.scale * kLog2e;
  auto load = [&](int i0, int st) {
    queries.load(ring + st * stage, ldq, i0, p.T);
    up.load(ring + st * stage + kBlk * ldq, ldv, i0, p.T);
    if (tid < kBlk && i0 + tid < p.T) {
      const size_t r = ((size_t)b * p.H + h) * p.T + i0 + tid;
      s_lse[st][tid] = p.lse[r] * kLog2e;
      s_delta[st][tid] = p.delta[r];
    }
  };
  walk(t0, last, stages, load, [&](int i0, int st) {
    const float *sq = ring + st * stage, *su = sq + kBlk * ldq;
    float s[kRt][4], dp[kRt][4];
    rows_by_rows(sk, ldq, sq, ldq, D, ty, tx, s);
    rows_by_rows(sv, ldv, su, ldv, p.V, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < kRt; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 16 * j, t = i0 + c;
        const bool on = t >= t0 + kRt * ty + i && t < end[i];
        const float w = on ? exp2f(s[i][j] * scale - s_lse[st][c]) : 0.f;
        sp[(kRt * ty + i) * kLdP + c] = w;
        sd[(kRt * ty + i) * kLdP + c] = on ? w * (dp[i][j] - s_delta[st][c]) : 0.f;
      }
    __syncwarp();
    weights_by_rows(sp, su, ldv, p.V, ty, tx, av);
    weights_by_rows(sd, sq, ldq, D, ty, tx, ak);
  });
#pragma unroll
  for (int i = 0; i < kRt; ++i) {
    const int t = t0 + kRt * ty + i;
    const size_t row = ((size_t)b * p.T + t) * p.H + h;
    bool bad = false;
    if (t < p.T) {
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 4 * tx + 64 * q + e;
          float x[2];
          upk2(ak[i][q][e >> 1], x[0], x[1]);
          const float y = x[e & 1] * p.scale;
          if (c < D) bad |= !finite(y);
          if (c < p.K) static_cast<T *>(p.dk)[row * p.K + c] = from_f32<T>(y);
          else if (c < D) p.dkr_part[row * p.R + c - p.K] = y;
          if (q < 2 && c < p.V) {
            upk2(av[i][q < 2 ? q : 0][e >> 1], x[0], x[1]);
            bad |= !finite(x[e & 1]);
            static_cast<T *>(p.dv)[row * p.V + c] = from_f32<T>(x[e & 1]);
          }
        }
    }
    const unsigned which = __ballot_sync(0xffffffffu, bad);
    __syncwarp();
    if (which & 0xffffu) key_grad_row<T>(p, b, h, t0 + 2 * kRt * (tid >> 5) + i, tid & 31);
    if (which & 0xffff0000u) key_grad_row<T>(p, b, h, t0 + 2 * kRt * (tid >> 5) + kRt + i, tid & 31);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) prompt_dq_kernel(const Prompt p, int stages) {
  extern __shared__ __align__(16) float sm[];
  const int D = p.K + p.R, ldq = D + 4, ldv = p.V + 4;
  float *sq = sm, *su = sq + kBlk * ldq, *sd = su + kBlk * ldv, *ring = sd + kBlk * kLdP;
  const int stage = kBlk * (ldq + ldv);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Where at0 = where(p, true);
  const int b = at0.b, h = at0.h, t0 = at0.t0;
  const Side<T> keys = keys_side<T>(p, b, h), values = values_side<T>(p, b, h);
  queries_side<T>(p, b, h).load(sq, ldq, t0, p.T);
  up_side<T>(p, b, h).load(su, ldv, t0, p.T);
  int lo[kRt];
  float lse[kRt], delta[kRt];
#pragma unroll
  for (int i = 0; i < kRt; ++i) {
    const int t = t0 + kRt * ty + i;
    lo[i] = t < p.T ? run_start(p, b, t) : 0x7fffffff;
    const size_t r = ((size_t)b * p.H + h) * p.T + min(t, p.T - 1);
    lse[i] = p.lse[r] * kLog2e;
    delta[i] = p.delta[r];
  }
  u64 acc[kRt][3][2];
  clear(acc);
  const float scale = p.scale * kLog2e;
  const int last = min(p.T, t0 + kBlk);
  auto load = [&](int j0, int st) {
    keys.load(ring + st * stage, ldq, j0, p.T);
    values.load(ring + st * stage + kBlk * ldq, ldv, j0, p.T);
  };
  walk(run_start(p, b, t0) / kBlk * kBlk, last, stages, load, [&](int j0, int st) {
    const float *sk = ring + st * stage, *sv = sk + kBlk * ldq;
    float s[kRt][4], dp[kRt][4];
    rows_by_rows(sq, ldq, sk, ldq, D, ty, tx, s);
    rows_by_rows(su, ldv, sv, ldv, p.V, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < kRt; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = j0 + tx + 16 * j;
        const bool on = k >= lo[i] && k <= t0 + kRt * ty + i;
        sd[(kRt * ty + i) * kLdP + tx + 16 * j] =
            on ? exp2f(s[i][j] * scale - lse[i]) * (dp[i][j] - delta[i]) : 0.f;
      }
    __syncwarp();
    weights_by_rows(sd, sk, ldq, D, ty, tx, acc);
  });
#pragma unroll
  for (int i = 0; i < kRt; ++i) {
    const int t = t0 + kRt * ty + i;
    const size_t row = ((size_t)b * p.T + t) * p.H + h;
    bool bad = false;
    if (t < p.T) {
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 4 * tx + 64 * q + e;
          float x[2];
          upk2(acc[i][q][e >> 1], x[0], x[1]);
          const float y = x[e & 1] * p.scale;
          if (c < D) bad |= !finite(y);
          if (c < p.K) static_cast<T *>(p.dq)[row * p.K + c] = from_f32<T>(y);
          else if (c < D) static_cast<T *>(p.dqr)[row * p.R + c - p.K] = from_f32<T>(y);
        }
    }
    const unsigned which = __ballot_sync(0xffffffffu, bad);
    __syncwarp();
    if (which & 0xffffu) query_grad_row<T>(p, b, h, t0 + 2 * kRt * (tid >> 5) + i, tid & 31);
    if (which & 0xffff0000u) query_grad_row<T>(p, b, h, t0 + 2 * kRt * (tid >> 5) + kRt + i, tid & 31);
  }
  if (blockIdx.x == 0) after_previous();
}

// ---- runs -------------------------------------------------------------------
// Where each token's run begins and ends, one CTA a row.  A warp takes 8 rows of 32
// tokens; a vote shows where a row's runs begin and end, so the latest beginning and the
// next end are bit searches.  One row of 8192 tokens 5 us (8 tokens a thread, whose loads and
// stores lie 32 bytes apart, 13).
constexpr int kRunThreads = 1024, kRunRows = 8, kRunChunk = kRunThreads * kRunRows;

// The starts and / or the ends of tokens t0 .. t0 + 8191; carry_start is the start that
// holds before them, carry_end the end that holds behind them.
template <bool kStart, bool kEnd>
__device__ __forceinline__ void run_chunk(const int *ids, int T, int *start, int *end, int t0,
                                          int &carry_start, int &carry_end) {
  __shared__ int s_top[kRunThreads / 32], s_low[kRunThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = t0 + warp * 32 * kRunRows;
  int id[kRunRows];
#pragma unroll
  for (int i = 0; i < kRunRows; ++i) {
    const int t = w0 + 32 * i + lane;
    id[i] = t < T ? ids[t] : 0;
  }
  const int prev = w0 > 0 && w0 <= T ? ids[w0 - 1] : 0;      // around the warp's tokens
  const int next = w0 + 32 * kRunRows < T ? ids[w0 + 32 * kRunRows] : 0;
  unsigned begins[kRunRows], ends[kRunRows];
  int top = 0, low = T;
#pragma unroll
  for (int i = 0; i < kRunRows; ++i) {
    const int t = w0 + 32 * i + lane;
    int before = __shfl_up_sync(0xffffffffu, id[i], 1);
    int behind = __shfl_down_sync(0xffffffffu, id[i], 1);
    const int left = i ? __shfl_sync(0xffffffffu, id[i ? i - 1 : 0], 31) : prev;
    const int right = i + 1 < kRunRows ? __shfl_sync(0xffffffffu, id[i + 1 < kRunRows ? i + 1 : 0], 0) : next;
    if (lane == 0) before = left;
    if (lane == 31) behind = right;
    begins[i] = __ballot_sync(0xffffffffu, t < T && id[i] != before);
    ends[i] = __ballot_sync(0xffffffffu, t < T && id[i] != behind);
    if (begins[i]) top = w0 + 32 * i + 31 - __clz(begins[i]);
    if (ends[i] && low == T) low = w0 + 32 * i + __ffs(ends[i]);
  }
  if (lane == 0) {
    s_top[warp] = top;
    s_low[warp] = low;
  }
  __syncthreads();
  int from = max(carry_start, __reduce_max_sync(0xffffffffu, lane < warp ? s_top[lane] : 0));
  int to = min(carry_end, __reduce_min_sync(0xffffffffu, lane > warp ? s_low[lane] : T));
#pragma unroll
  for (int i = 0; i < kRunRows; ++i) {
    const int t = w0 + 32 * i + lane;
    const unsigned m = begins[i] & (0xffffffffu >> (31 - lane));
    if (kStart && t < T)
      start[t] = id[i] == 0 ? t + 1 : m ? w0 + 32 * i + 31 - __clz(m) : from;
    if (begins[i]) from = w0 + 32 * i + 31 - __clz(begins[i]);
  }
#pragma unroll
  for (int i = kRunRows - 1; i >= 0; --i) {
    const int t = w0 + 32 * i + lane;
    const unsigned m = ends[i] & (0xffffffffu << lane);
    if (kEnd && t < T) end[t] = id[i] == 0 ? t : m ? w0 + 32 * i + __ffs(m) : to;
    if (ends[i]) to = w0 + 32 * i + __ffs(ends[i]);
  }
  carry_start = max(carry_start, __reduce_max_sync(0xffffffffu, s_top[lane]));
  carry_end = min(carry_end, __reduce_min_sync(0xffffffffu, s_low[lane]));
  __syncthreads();
}

__global__ void __launch_bounds__(kRunThreads) runs_kernel(const int *ids, int T, int *start,
                                                           int *end) {
  start_next();
  const size_t row = (size_t)blockIdx.x * T;
  int a = 0, z = T;
  if (T <= kRunChunk) {
    run_chunk<true, true>(ids + row, T, start + row, end + row, 0, a, z);
    return;
  }
  for (int t0 = 0; t0 < T; t0 += kRunChunk)
    run_chunk<true, false>(ids + row, T, start + row, end + row, t0, a, z);
  a = 0, z = T;
  for (int t0 = (T - 1) / kRunChunk * kRunChunk; t0 >= 0; t0 -= kRunChunk)
    run_chunk<false, true>(ids + row, T, start + row, end + row, t0, a, z);
}

// ---- around the backward ----------------------------------------------------
constexpr int kSmall = 256;       // threads

// delta[b][h][t] = d_o . o, 8 lanes a row.  Bound by memory: 8192 tokens of 32 heads of 128
// 24 us, 5.6 TB/s.
template <typename T>
__global__ void __launch_bounds__(kSmall) delta_kernel(Prompt p) {
  const long long rows = (long long)p.B * p.T * p.H;
  const long long r = (long long)blockIdx.x * (kSmall / 8) + threadIdx.x / 8;
  float s = 0.f;
  if (r < rows) {
    const T *o = static_cast<const T *>(p.o) + r * p.V,
            *u = static_cast<const T *>(p.d_o) + r * p.V;
    constexpr int W = 16 / (int)sizeof(T);
    struct alignas(16) Piece {
      T v[W];
    };
    for (int c = (threadIdx.x & 7) * W; c < p.V; c += 8 * W) {
      const Piece x = *reinterpret_cast<const Piece *>(o + c);
      const Piece y = *reinterpret_cast<const Piece *>(u + c);
#pragma unroll
      for (int e = 0; e < W; ++e) s = fmaf(to_f32(x.v[e]), to_f32(y.v[e]), s);
    }
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (r < rows && (threadIdx.x & 7) == 0) {
    const int h = (int)(r % p.H);
    const long long bt = r / p.H;
    const int t = (int)(bt % p.T), b = (int)(bt / p.T);
    const_cast<float *>(p.delta)[((size_t)b * p.H + h) * p.T + t] = s;
  }
}

// dk_rope = the sum of the heads' parts, in the order of the heads.  8192 tokens of 32 heads:
// 20 us for 68 MB, a third of it launch and latency.
template <typename T>
__global__ void __launch_bounds__(kSmall) rope_sum_kernel(Prompt p) {
  const int quads = p.R / 4;
  const long long i = (long long)blockIdx.x * kSmall + threadIdx.x;
  if (i >= (long long)p.B * p.T * quads) return;
  const float4 *x = reinterpret_cast<const float4 *>(p.dkr_part) + i / quads * p.H * quads +
                    i % quads;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int h = 0; h < p.H; ++h) {
    const float4 y = x[(size_t)h * quads];
    s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
  }
  T *d = static_cast<T *>(p.dkr) + 4 * i;
  d[0] = from_f32<T>(s.x);
  d[1] = from_f32<T>(s.y);
  d[2] = from_f32<T>(s.z);
  d[3] = from_f32<T>(s.w);
}

constexpr size_t kMaxSmem = 226 * 1024;

// `held`: rows of a tile's width that stay, beside one or two stages of the other side.
template <typename K>
cudaError_t launch_tiles(K kern, const Prompt &p, size_t held, cudaStream_t cs, bool beside = false) {
  const size_t stage = sizeof(float) * kBlk * (size_t)(p.K + p.R + 4 + p.V + 4);
  held *= sizeof(float);
  const int stages = held + 2 * stage <= kMaxSmem ? 2 : 1;
  const size_t smem = held + stages * stage;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  const unsigned tiles = (unsigned)((p.T + kBlk - 1) / kBlk);
  if (beside) return launch_next(kern, dim3(tiles * p.B * p.H), kThreads, smem, cs, p, stages);
  kern<<<tiles * p.B * p.H, kThreads, smem, cs>>>(p, stages);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_simt(const Prompt &p, cudaStream_t cs) {
  const size_t q = (size_t)kBlk * (p.K + p.R + 4);
  return launch_tiles(prompt_fwd_kernel<T>, p, q + kBlk * kLdP, cs);
}

// The gradients of the queries need nothing of those of the keys and values: their
// kernel begins once all CTAs of the other one have begun, on the SMs that these leave.
// One of its CTAs ends after the other kernel has, so what follows waits for both.
template <typename T>
cudaError_t backward(const Prompt &p, bool tc, cudaStream_t cs) {
  cudaError_t e = cudaSuccess;
  if (!tc || p.T > kExactKeys) {     // (the tensor cores' path makes the rest by itself)
    const long long rows = (long long)p.B * p.T * p.H;
    delta_kernel<T><<<(unsigned)((rows + kSmall / 8 - 1) / (kSmall / 8)), kSmall, 0, cs>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (tc) {
    e = launch_prompt_bwd_tc(p, cs);
  } else {
    const size_t q = (size_t)kBlk * (p.K + p.R + 4), v = (size_t)kBlk * (p.V + 4),
                 w = (size_t)kBlk * kLdP;
    e = launch_tiles(prompt_dkv_kernel<T>, p, q + v + 2 * w, cs);
    if (e == cudaSuccess) e = launch_tiles(prompt_dq_kernel<T>, p, q + v + w, cs, true);
  }
  if (e != cudaSuccess || p.R == 0) return e;
  const long long quads = (long long)p.B * p.T * (p.R / 4);
  rope_sum_kernel<T><<<(unsigned)((quads + kSmall - 1) / kSmall), kSmall, 0, cs>>>(p);
  return cudaGetLastError();
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

kda_status check(const kda_latent_shape *s) {
  if (!s || s->B < 1 || s->T < 1 || s->H < 1) return KDA_ERR_INVALID_ARG;
  if (s->dtype != KDA_DTYPE_F32 && s->dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
  for (int d : {s->K, s->V})
    if (d != 32 && d != 64 && d != 128) return KDA_ERR_UNSUPPORTED;
  if (s->R != 0 && s->R != 32 && s->R != 64) return KDA_ERR_UNSUPPORTED;
  if ((long long)s->B * s->T >= (1ll << 31) || (long long)s->B * s->H >= (1ll << 31) ||
      (double)s->B * s->T * s->H * (s->K + s->R) >= 2147483648.0)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// Of the workspace, after its header.
size_t table_bytes(const kda_latent_shape *s) {
  return align_up(sizeof(int) * (size_t)s->B * s->T, 256);
}
size_t delta_bytes(const kda_latent_shape *s) {
  return align_up(sizeof(float) * (size_t)s->B * s->T * s->H, 256);
}

Prompt make(const kda_latent_shape *s, const void *q, const void *q_rope, const void *k,
            const void *k_rope, const void *v, float scale, void *workspace) {
  Prompt p;
  memset(&p, 0, sizeof(p));
  p.B = s->B; p.T = s->T; p.H = s->H; p.K = s->K; p.R = s->R; p.V = s->V;
  p.q = q; p.qr = q_rope; p.k = k; p.kr = k_rope; p.v = v;
  auto of = [&](long long b, long long t, long long h) {
    return strides_of(s->B, s->T, s->H, b, t, h);
  };
  p.q_s = of(s->q_stride_b, s->q_stride_t, s->q_stride_h);
  p.k_s = of(s->k_stride_b, s->k_stride_t, s->k_stride_h);
  p.v_s = of(s->v_stride_b, s->v_stride_t, s->v_stride_h);
  if (s->R) {
    p.qr_s = of(s->q_rope_stride_b, s->q_rope_stride_t, s->q_rope_stride_h);
    p.kr_s = of(s->k_rope_stride_b, s->k_rope_stride_t, 0);
  }
  p.scale = scale;
  p.status = &static_cast<WsHeader *>(workspace)->status;
  const uintptr_t bytes = s->dtype == KDA_DTYPE_BF16 ? 8 : 16;
  p.fours = 1;
  for (const void *x : {q, q_rope, k, k_rope, v})
    if (reinterpret_cast<uintptr_t>(x) % bytes) p.fours = 0;
  for (const Strides &x : {p.q_s, p.qr_s, p.k_s, p.kr_s, p.v_s})
    if ((x.b | x.t | x.h) & 3) p.fours = 0;
  return p;
}

kda_status check_call(const kda_latent_shape *s, const void *q, const void *q_rope, const void *k,
                      const void *k_rope, const void *v, float scale, const int32_t *segment_ids,
                      kda_impl impl) {
  const kda_status st = check(s);
  if (st != KDA_OK) return st;
  if (!q || !k || !v || !(fabsf(scale) < INFINITY)) return KDA_ERR_INVALID_ARG;
  if ((s->R > 0) != (q_rope != nullptr) || (s->R > 0) != (k_rope != nullptr))
    return KDA_ERR_INVALID_ARG;
  if (impl != KDA_IMPL_AUTO && impl != KDA_IMPL_SIMT && impl != KDA_IMPL_TC)
    return KDA_ERR_INVALID_ARG;
  if (impl == KDA_IMPL_TC && s->dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  const uintptr_t es = s->dtype == KDA_DTYPE_BF16 ? 2 : 4;
  for (const void *x : {q, q_rope, k, k_rope, v})
    if (!aligned(x, es)) return KDA_ERR_ALIGNMENT;
  if (!aligned(segment_ids, 4)) return KDA_ERR_ALIGNMENT;
  return KDA_OK;
}

kda_status check_workspace(const kda_latent_shape *s, int backward, const void *workspace,
                           size_t bytes) {
  if (!workspace || bytes < kda_latent_workspace_size(s, backward)) return KDA_ERR_WORKSPACE;
  return aligned(workspace, 256) ? KDA_OK : KDA_ERR_ALIGNMENT;
}

cudaError_t find_runs(Prompt &p, const int32_t *segment_ids, const kda_latent_shape *s,
                      void *workspace, cudaStream_t cs) {
  if (!segment_ids) return cudaSuccess;
  int *start = reinterpret_cast<int *>(static_cast<char *>(workspace) + sizeof(WsHeader));
  int *end = start + table_bytes(s) / sizeof(int);
  runs_kernel<<<(unsigned)s->B, kRunThreads, 0, cs>>>(segment_ids, s->T, start, end);
  p.start = start;
  p.end = end;
  return cudaGetLastError();
}

// Whether the tensor cores take the call; *st is a refusal of KDA_IMPL_TC.  (The largest
// product is the largest score only where the scale is not negative.)
bool use_tc(const kda_latent_shape *s, const Prompt &p, kda_impl impl, kda_status *st) {
  if (impl == KDA_IMPL_SIMT || s->dtype != KDA_DTYPE_BF16) return false;
  const bool sign = p.scale >= 0.f, layout = prompt_tc_ok(p);
  if (impl == KDA_IMPL_TC && !(sign && layout))
    *st = sign ? KDA_ERR_ALIGNMENT : KDA_ERR_UNSUPPORTED;
  return sign && layout;
}

}  // namespace
}  // namespace latent
}  // namespace kda

using namespace kda;
using namespace kda::latent;

extern "C" {

size_t kda_latent_workspace_size(const kda_latent_shape *s, int backward) {
  if (check(s) != KDA_OK) return 0;
  size_t n = sizeof(WsHeader) + 2 * table_bytes(s);
  if (backward)
    n += delta_bytes(s) + align_up(sizeof(float) * (size_t)s->B * s->T * s->H * s->R, 256);
  return n;
}

kda_status kda_latent_fwd(const kda_latent_shape *s, const void *q, const void *q_rope,
                          const void *k, const void *k_rope, const void *v, float scale,
                          const int32_t *segment_ids, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, kda_impl impl, kda_stream_t stream) {
  kda_status st = check_call(s, q, q_rope, k, k_rope, v, scale, segment_ids, impl);
  if (st != KDA_OK) return st;
  if (!o) return KDA_ERR_INVALID_ARG;
  if (!aligned(o, 16) || !aligned(lse, 4)) return KDA_ERR_ALIGNMENT;
  st = check_workspace(s, 0, workspace, workspace_bytes);
  if (st != KDA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  Prompt p = make(s, q, q_rope, k, k_rope, v, scale, workspace);
  p.o = o;
  p.lse = lse;
  const bool tc = use_tc(s, p, impl, &st);
  if (st != KDA_OK) return st;
  cudaError_t e = find_runs(p, segment_ids, s, workspace, cs);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  e = tc ? launch_prompt_tc(p, cs)
      : s->dtype == KDA_DTYPE_BF16 ? forward_simt<__nv_bfloat16>(p, cs)
                                   : forward_simt<float>(p, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_latent_bwd(const kda_latent_shape *s, const void *q, const void *q_rope,
                          const void *k, const void *k_rope, const void *v, float scale,
                          const int32_t *segment_ids, const void *o, const float *lse,
                          const void *d_o, void *dq, void *dq_rope, void *dk, void *dk_rope,
                          void *dv, void *workspace, size_t workspace_bytes, kda_impl impl,
                          kda_stream_t stream) {
  kda_status st = check_call(s, q, q_rope, k, k_rope, v, scale, segment_ids, impl);
  if (st != KDA_OK) return st;
  if (!o || !lse || !d_o || !dq || !dk || !dv) return KDA_ERR_INVALID_ARG;
  if ((s->R > 0) != (dq_rope != nullptr) || (s->R > 0) != (dk_rope != nullptr))
    return KDA_ERR_INVALID_ARG;
  for (const void *x : {o, d_o, (const void *)dq, (const void *)dq_rope, (const void *)dk,
                        (const void *)dk_rope, (const void *)dv})
    if (!aligned(x, 16)) return KDA_ERR_ALIGNMENT;
  if (!aligned(lse, 4)) return KDA_ERR_ALIGNMENT;
  st = check_workspace(s, 1, workspace, workspace_bytes);
  if (st != KDA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  Prompt p = make(s, q, q_rope, k, k_rope, v, scale, workspace);
  p.o = const_cast<void *>(o);
  p.lse = const_cast<float *>(lse);
  p.d_o = d_o;
  p.dq = dq; p.dqr = dq_rope; p.dk = dk; p.dkr = dk_rope; p.dv = dv;
  char *ws = static_cast<char *>(workspace) + sizeof(WsHeader) + 2 * table_bytes(s);
  p.delta = reinterpret_cast<float *>(ws);
  p.dkr_part = reinterpret_cast<float *>(ws + delta_bytes(s));
  const bool tc = use_tc(s, p, impl, &st);
  if (st != KDA_OK) return st;
  cudaError_t e = find_runs(p, segment_ids, s, workspace, cs);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  e = s->dtype == KDA_DTYPE_BF16 ? backward<__nv_bfloat16>(p, tc, cs)
                                 : backward<float>(p, false, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
