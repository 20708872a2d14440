// kda_norm.cu -- the norms before and after a block, fused with the block's
// gate and residual scale, forward and backward.
//
// Per row of D values (fp32 throughout, one rounding at each output):
//
//     n1 = y * s1,   s1 = (mean(y^2) + eps)^-1/2
//     out = residual + scale * act(gate) * n1 * w_post
//     n2 = out * s2, s2 = (mean(out^2) + eps)^-1/2
//     x   = n2 * w_pre
//
// Backward, with c2 = mean(d_x w_pre n2) and r = d_out + s2 (d_x w_pre - n2 c2)
// the whole gradient of `out`:
//
//     d_residual = r          d_gate = scale * n1 w_post * act'(gate) * r
//     dw_post = sum_rows scale act(gate) r n1       dw_pre = sum_rows d_x n2
//     dy = s1 (t - n1 c1),  t = scale act(gate) w_post r,  c1 = mean(t n1)
//
// c1 needs c2, but with q = scale act(gate) w_post n1 it is
// mean(q (d_out + s2 d_x w_pre)) - s2 c2 mean(q n2): three sums of one pass,
// so a row costs one reduction and its inputs are read once.
//
// Both kernels are bound by HBM.  A row belongs to `tpr` threads (a power of
// two up to a warp, else whole warps), each owning VEC-wide pieces of 16
// bytes tpr apart; a CTA holds rg = 256 / tpr rows when a row needs fewer
// than 256 threads.  Rows whose length or pointers do not allow 16-byte
// accesses take the same code with VEC = 1.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kMaxDim = 16384;
constexpr int kBlock = 256;        // threads when a row needs at most these
constexpr int kStages = 2;         // rows staged per thread in the backward
constexpr size_t kStageMax = 200 * 1024;   // longer rows are read directly

enum { kGateNone = 0, kGateEach = 1, kGateGroup = 2 };

// How a row is laid over threads.
struct Layout {
  int vec;      // elements per access (16 bytes, or 1)
  int items;    // accesses per thread and row
  int tpr;      // threads per row
  int rg;       // rows per CTA
};

Layout layout_for(int D, int elt, bool vector_ok) {
  Layout l;
  l.vec = vector_ok && D % (16 / elt) == 0 ? 16 / elt : 1;
  const int n = D / l.vec;
  const int most = l.vec > 1 ? 512 : 1024;     // threads of one row
  l.items = l.vec > 1 ? 1 : 4;
  while (l.items * most < n) l.items *= l.vec > 1 ? 2 : 4;
  int t = (n + l.items - 1) / l.items;
  if (t > 32) {
    t = (t + 31) / 32 * 32;
  } else {
    int p = 4;
    while (p < t) p *= 2;
    t = p;
  }
  l.tpr = t;
  l.rg = t <= kBlock ? kBlock / t : 1;
  return l;
}

// VEC elements as fp32.
template <typename T, int VEC>
struct Piece;
template <>
struct Piece<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void get(const Raw &a, float (&f)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw put(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Piece<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void get(const Raw &a, float (&f)[4]) {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  }
  static __device__ __forceinline__ Raw put(const float (&f)[4]) {
    return make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <typename T>
struct Piece<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ void get(const Raw &a, float (&f)[1]) { f[0] = to_f32(a); }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return from_f32<T>(f[0]); }
};

template <int VEC>
__device__ __forceinline__ void load_w(const float *w, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = *w;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 a = *reinterpret_cast<const float4 *>(w + i);
      f[i] = a.x; f[i + 1] = a.y; f[i + 2] = a.z; f[i + 3] = a.w;
    }
  }
}

// act(a), and its derivative when DER.  The sigmoid takes the approximate
// exp2 and reciprocal (a few fp32 ulp); tanh needs tanhf, whose relative
// error holds near 0 too.
template <bool DER>
__device__ __forceinline__ void gate_value(float a, int act, float &v, float &d) {
  if (act == KDA_GATE_TANH) {
    v = tanhf(a);
    if (DER) d = 1.f - v * v;
    return;
  }
  if (act == KDA_GATE_NONE) {
    v = a;
    if (DER) d = 1.f;
    return;
  }
  const float s = __fdividef(1.f, 1.f + __expf(-a));
  if (act == KDA_GATE_SIGMOID) {
    v = s;
    if (DER) d = s * (1.f - s);
  } else {
    v = a * s;
    if (DER) d = s * (1.f + a * (1.f - s));
  }
}

// Sums of N values over the tpr threads of a row, in every thread of the
// row.  `slot` alternates between two buffers, so one barrier is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float (*red)[N][32], int &slot) {
  const int lim = tpr < 32 ? tpr : 32;
  for (int off = lim >> 1; off; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  if (tpr > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[slot][i][warp] = v[i];
    __syncthreads();
    const int nw = tpr >> 5, first = warp / nw * nw;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = lane < nw ? red[slot][i][first + lane] : 0.f;
#pragma unroll
      for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      v[i] = s;
    }
    slot ^= 1;
  }
}

struct NormParams {
  long long R;
  int D, tpr, rg, act;
  float scale, eps, inv_d;
  unsigned rows_per_gate;
  const void *y, *res, *gate;
  const float *w_post, *w_pre;
  void *out, *x;
  float *stats;                 // [2][R]: s1, s2
};

// One row per row group at a time, rows gridDim.x * rg apart.  The weights
// stay in registers; every input element is read once and kept as `out`.
template <typename T, int VEC, int ITEMS>
__global__ void __launch_bounds__(VEC > 1 ? 512 : 1024) norm_fwd_kernel(const NormParams p) {
  using P = Piece<T, VEC>;
  using Raw = typename P::Raw;
  __shared__ float red[2][1][32];
  const int tid = threadIdx.x, tpr = p.tpr, rg = p.rg;
  const int group = tid / tpr, lane = tid - group * tpr;
  int slot = 0;
  for (long long r0 = (long long)blockIdx.x * rg; r0 < p.R; r0 += (long long)gridDim.x * rg) {
    const long long row = r0 + group;
    const bool live = row < p.R;
    const size_t base = (size_t)row * p.D;
    const size_t gbase = p.gate && live ? (size_t)((unsigned)row / p.rows_per_gate) * p.D : 0;
    Raw ry[ITEMS], rr[ITEMS], rgt[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (lane + i * tpr) * VEC;
      if (live && c < p.D) {
        ry[i] = *reinterpret_cast<const Raw *>((const T *)p.y + base + c);
        if (p.gate) rgt[i] = *reinterpret_cast<const Raw *>((const T *)p.gate + gbase + c);
        if (p.res) rr[i] = *reinterpret_cast<const Raw *>((const T *)p.res + base + c);
      }
    }
    float v[ITEMS][VEC], ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const bool ok = live && (lane + i * tpr) * VEC < p.D;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
      if (ok) P::get(ry[i], v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss[0] += v[i][e] * v[i][e];
    }
    row_sum(ss, tpr, red, slot);
    const float s1 = rsqrtf(ss[0] * p.inv_d + p.eps), k = s1 * p.scale;
    ss[0] = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (lane + i * tpr) * VEC;
      if (live && c < p.D) {
        float w[VEC], a[VEC], d;
        load_w<VEC>(p.w_post + c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= k * w[e];
        if (p.gate) {
          P::get(rgt[i], a);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            gate_value<false>(a[e], p.act, a[e], d);
            v[i][e] *= a[e];
          }
        }
        if (p.res) {
          P::get(rr[i], a);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] += a[e];
        }
        *reinterpret_cast<Raw *>((T *)p.out + base + c) = P::put(v[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[0] += v[i][e] * v[i][e];
      }
    }
    float s2 = 0.f;
    if (p.w_pre) {
      row_sum(ss, tpr, red, slot);
      s2 = rsqrtf(ss[0] * p.inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = (lane + i * tpr) * VEC;
        if (live && c < p.D) {
          float w[VEC];
          load_w<VEC>(p.w_pre + c, w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] *= s2 * w[e];
          *reinterpret_cast<Raw *>((T *)p.x + base + c) = P::put(v[i]);
        }
      }
    }
    if (p.stats && live && lane == 0) {
      p.stats[row] = s1;
      p.stats[p.R + row] = s2;
    }
  }
}

struct NormBwdParams {
  NormParams f;
  const void *d_out, *d_x;
  void *dy, *d_res, *d_gate;
  float *part_post, *part_pre, *part_gate;   // [units][D]
  long long gate_rows;
  int splits;      // units per gate row (group gates), 0: whole gate rows per unit
  int n_in;        // input arrays staged per row
  int stages;      // kStages, or 0: inputs are read directly
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

// Sums `acc` over the CTA's row groups and hands the totals of the first
// group's columns to `put(column, values)`.  Uniform over the CTA.
template <int VEC, int ITEMS, typename F>
__device__ __forceinline__ void flush(float (&acc)[ITEMS][VEC], int tpr, int rg, int group,
                                      int lane, int D, float *buf, F put) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = (lane + i * tpr) * VEC;
    if (rg > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) buf[threadIdx.x * VEC + e] = acc[i][e];
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < rg; ++g)
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[i][e] += buf[(g * tpr + lane) * VEC + e];
    }
    if (group == 0 && c < D) put(c, acc[i]);
  }
}

// A unit (CTA) owns a contiguous range of rows, keeps its sums of dw_post,
// dw_pre and (group gates) d_gate in registers and writes them once; the
// units' sums are added in a fixed order by norm_sum_kernel, so no result
// depends on timing.  A thread copies its own pieces of the next row to
// shared memory (cp.async) while it works on this one.
template <typename T, int VEC, int ITEMS, int GATE>
__global__ void __launch_bounds__(VEC > 1 ? 512 : 1024) norm_bwd_kernel(const NormBwdParams q) {
  using P = Piece<T, VEC>;
  using Raw = typename P::Raw;
  constexpr bool kAsync = VEC > 1;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][3][32];
  const NormParams &p = q.f;
  const int tid = threadIdx.x, tpr = p.tpr, rg = p.rg, nthr = blockDim.x;
  const int group = tid / tpr, lane = tid - group * tpr;
  float *buf = reinterpret_cast<float *>(smem);
  Raw *stage = reinterpret_cast<Raw *>(smem + (rg > 1 ? sizeof(float) * nthr * VEC : 0));
  int slot = 0;

  float dw1[ITEMS][VEC] = {}, dw2[ITEMS][VEC] = {};
  constexpr int GI = GATE == kGateGroup ? ITEMS : 1;
  // the gate rows [g_lo, g_hi) of this unit, or its part of one gate row
  long long g_lo = 0, g_hi = 1;
  if (GATE == kGateGroup) {
    if (q.splits) {
      g_lo = blockIdx.x / q.splits;
      g_hi = g_lo + 1;
    } else {
      g_lo = (long long)blockIdx.x * q.gate_rows / gridDim.x;
      g_hi = (long long)(blockIdx.x + 1) * q.gate_rows / gridDim.x;
    }
  }
  for (long long g = g_lo; g < g_hi; ++g) {
    long long lo, hi;
    if (GATE == kGateGroup) {
      const long long n = p.rows_per_gate, s = q.splits ? blockIdx.x % q.splits : 0,
                      m = q.splits ? q.splits : 1;
      lo = g * n + s * n / m;
      hi = g * n + (s + 1) * n / m;
    } else {
      lo = (long long)blockIdx.x * p.R / gridDim.x;
      hi = (long long)(blockIdx.x + 1) * p.R / gridDim.x;
    }
    float ga[GI][VEC], gd[GI][VEC], dg[GI][VEC];
    if (GATE == kGateGroup) {
#pragma unroll
      for (int i = 0; i < GI; ++i) {
        const int c = (lane + i * tpr) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) dg[i][e] = ga[i][e] = gd[i][e] = 0.f;
        if (c < p.D) {
          float a[VEC];
          P::get(*reinterpret_cast<const Raw *>((const T *)p.gate + (size_t)g * p.D + c), a);
#pragma unroll
          for (int e = 0; e < VEC; ++e) gate_value<true>(a[e], p.act, ga[i][e], gd[i][e]);
        }
      }
    }
    auto fetch = [&](long long row, int st) {
      if constexpr (kAsync) {
        if (q.stages && row < hi) {
          const size_t base = (size_t)row * p.D;
#pragma unroll
          for (int i = 0; i < ITEMS; ++i) {
            const int c = (lane + i * tpr) * VEC;
            if (c < p.D) {
              Raw *d = stage + (size_t)(st * ITEMS + i) * q.n_in * nthr + tid;
              cp_async16(d, (const T *)p.y + base + c); d += nthr;
              if (q.d_out) { cp_async16(d, (const T *)q.d_out + base + c); d += nthr; }
              if (q.d_x) { cp_async16(d, (const T *)q.d_x + base + c); d += nthr; }
              if (p.res) { cp_async16(d, (const T *)p.res + base + c); d += nthr; }
              if (GATE == kGateEach) cp_async16(d, (const T *)p.gate + base + c);
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
    };
    int st = 0;
    fetch(lo + group, 0);
    for (long long r0 = lo; r0 < hi; r0 += rg) {
      const long long row = r0 + group;
      const bool live = row < hi;
      fetch(row + rg, st ^ 1);
      float s1 = 0.f, s2 = 0.f;
      if (live) {
        s1 = p.stats[row];
        s2 = p.stats[p.R + row];
      }
      if constexpr (kAsync) asm volatile("cp.async.wait_group 1;" ::: "memory");
      const size_t base = (size_t)row * p.D;
      // n1, n2, the incoming gradients, act(gate) and its derivative
      float n1[ITEMS][VEC], n2[ITEMS][VEC], go[ITEMS][VEC], gx[ITEMS][VEC], a[ITEMS][VEC],
          da[ITEMS][VEC], sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = (lane + i * tpr) * VEC;
        const bool ok = live && c < p.D;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          n1[i][e] = n2[i][e] = go[i][e] = gx[i][e] = a[i][e] = da[i][e] = 0.f;
        if (ok) {
          float w1[VEC], w2[VEC], t[VEC];
          const Raw *sp = stage + (size_t)(st * ITEMS + i) * q.n_in * nthr + tid;
          auto next = [&](const void *src) {
            if (kAsync && q.stages) {
              const Raw v = *sp;
              sp += nthr;
              return v;
            }
            return *reinterpret_cast<const Raw *>((const T *)src + base + c);
          };
          P::get(next(p.y), n1[i]);
          if (q.d_out) P::get(next(q.d_out), go[i]);
          if (q.d_x) P::get(next(q.d_x), gx[i]);
          if (p.res) P::get(next(p.res), n2[i]);
          if (GATE == kGateEach) {
            P::get(next(p.gate), t);
#pragma unroll
            for (int e = 0; e < VEC; ++e) gate_value<true>(t[e], p.act, a[i][e], da[i][e]);
          }
          load_w<VEC>(p.w_post + c, w1);
          if (p.w_pre) load_w<VEC>(p.w_pre + c, w2);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if (GATE == kGateNone) a[i][e] = 1.f;
            if (GATE == kGateGroup) a[i][e] = ga[i < GI ? i : 0][e];
            n1[i][e] *= s1;
            const float qv = p.scale * a[i][e] * w1[e] * n1[i][e];
            n2[i][e] = (n2[i][e] + qv) * s2;
            const float gw = p.w_pre ? gx[i][e] * w2[e] : 0.f;
            sum[0] += gw * n2[i][e];
            sum[1] += qv * (go[i][e] + s2 * gw);
            sum[2] += qv * n2[i][e];
          }
        }
      }
      row_sum(sum, tpr, red, slot);
      const float c2 = sum[0] * p.inv_d;
      const float c1 = (sum[1] - s2 * c2 * sum[2]) * p.inv_d;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = (lane + i * tpr) * VEC;
        if (live && c < p.D) {
          float w1[VEC], w2[VEC], oy[VEC], og[VEC];
          load_w<VEC>(p.w_post + c, w1);
          if (p.w_pre) load_w<VEC>(p.w_pre + c, w2);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float r = go[i][e];
            if (p.w_pre) r += s2 * (gx[i][e] * w2[e] - n2[i][e] * c2);
            dw2[i][e] += gx[i][e] * n2[i][e];
            const float sr = p.scale * r, ar = a[i][e] * sr;
            dw1[i][e] += ar * n1[i][e];
            const float ug = sr * n1[i][e] * w1[e];
            if (GATE == kGateEach) og[e] = ug * da[i][e];
            if (GATE == kGateGroup) dg[i < GI ? i : 0][e] += ug * gd[i < GI ? i : 0][e];
            oy[e] = s1 * (ar * w1[e] - n1[i][e] * c1);
            go[i][e] = r;
          }
          *reinterpret_cast<Raw *>((T *)q.dy + base + c) = P::put(oy);
          if (q.d_res) *reinterpret_cast<Raw *>((T *)q.d_res + base + c) = P::put(go[i]);
          if (GATE == kGateEach && q.d_gate)
            *reinterpret_cast<Raw *>((T *)q.d_gate + base + c) = P::put(og);
        }
      }
      st ^= 1;
    }
    if constexpr (kAsync) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (GATE == kGateGroup && q.d_gate)
      flush<VEC, GI>(dg, tpr, rg, group, lane, p.D, buf, [&](int c, float (&v)[VEC]) {
        if (q.splits) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) q.part_gate[(size_t)blockIdx.x * p.D + c + e] = v[e];
        } else {
          *reinterpret_cast<Raw *>((T *)q.d_gate + (size_t)g * p.D + c) = P::put(v);
        }
      });
  }
  flush<VEC, ITEMS>(dw1, tpr, rg, group, lane, p.D, buf, [&](int c, float (&v)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) q.part_post[(size_t)blockIdx.x * p.D + c + e] = v[e];
  });
  if (p.w_pre)
    flush<VEC, ITEMS>(dw2, tpr, rg, group, lane, p.D, buf, [&](int c, float (&v)[VEC]) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) q.part_pre[(size_t)blockIdx.x * p.D + c + e] = v[e];
    });
}

// Column sums of the units' partials: blockIdx.y 0 dw_post, 1 dw_pre, 2 + g
// gate row g.  32 columns x 32 row lanes, always in the same order.
template <typename T>
__global__ void __launch_bounds__(1024)
    norm_sum_kernel(const float *part_post, const float *part_pre, const float *part_gate,
                    float *dw_post, float *dw_pre, T *d_gate, int units, int splits, int D) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  const int what = blockIdx.y;
  if (what == 1 && !part_pre) return;
  const float *src = what == 0 ? part_post
                     : what == 1 ? part_pre
                                 : part_gate + (size_t)(what - 2) * splits * D;
  const int n = what < 2 ? units : splits;
  float v = 0.f;
  if (c < D)
#pragma unroll 4
    for (int u = y; u < n; u += 32) v += src[(size_t)u * D + c];
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && c < D) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][x];
    if (what == 0) dw_post[c] = v;
    else if (what == 1) dw_pre[c] = v;
    else d_gate[(size_t)(what - 2) * D + c] = from_f32<T>(v);
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

kda_status check_desc(const kda_norm_desc *d, bool has_gate) {
  if (!d || d->rows < 1 || d->dim < 1) return KDA_ERR_INVALID_ARG;
  if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
  if (d->gate_act < KDA_GATE_NONE || d->gate_act > KDA_GATE_TANH) return KDA_ERR_INVALID_ARG;
  if (!(d->scale == d->scale) || !(d->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
  if (has_gate && (d->gate_rows < 1 || d->rows % d->gate_rows)) return KDA_ERR_INVALID_ARG;
  if (d->dim > kMaxDim || d->rows >= (1ll << 31)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

NormParams params_of(const kda_norm_desc *d, const Layout &l, const void *y, const float *w_post,
                     const void *res, const void *gate, const float *w_pre) {
  NormParams p = {};
  p.R = d->rows; p.D = d->dim; p.tpr = l.tpr; p.rg = l.rg; p.act = d->gate_act;
  p.scale = d->scale; p.eps = d->eps; p.inv_d = 1.f / (float)d->dim;
  p.rows_per_gate = gate ? (unsigned)(d->rows / d->gate_rows) : 1u;
  p.y = y; p.res = res; p.gate = gate; p.w_post = w_post; p.w_pre = w_pre;
  return p;
}

// Units (CTAs) of the backward: two for each of the 152 SMs, four where a
// CTA holds several rows, and no more than there are row groups.
int units_for(const kda_norm_desc *d, const Layout &l) {
  const long long most = 152ll * (l.rg > 1 ? 4 : 2);
  const long long n = (d->rows + l.rg - 1) / l.rg;
  return (int)(n < most ? n : most);
}
// Group gates: units per gate row when there are fewer gate rows than units
// (0: every unit has whole gate rows).
int splits_for(const kda_norm_desc *d, const Layout &l, int units) {
  if (d->gate_rows >= units) return 0;
  long long s = units / d->gate_rows;
  const long long per = d->rows / d->gate_rows, most = (per + l.rg - 1) / l.rg;
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s);
}

template <typename T, int VEC, int ITEMS>
cudaError_t launch_fwd_t(const NormParams &p, cudaStream_t stream) {
  auto kern = norm_fwd_kernel<T, VEC, ITEMS>;
  const int threads = p.tpr * p.rg;
  int per_sm = 1;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0);
  if (e != cudaSuccess) return e;
  const long long n = (p.R + p.rg - 1) / p.rg, most = (long long)num_sms() * per_sm;
  kern<<<(unsigned)(n < most ? n : most), threads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int VEC, int ITEMS, int GATE>
cudaError_t launch_bwd_t(NormBwdParams q, int units, cudaStream_t stream) {
  auto kern = norm_bwd_kernel<T, VEC, ITEMS, GATE>;
  const int threads = q.f.tpr * q.f.rg;
  size_t smem = q.f.rg > 1 ? sizeof(float) * threads * VEC : 0;
  const size_t staged = VEC > 1 ? (size_t)kStages * ITEMS * q.n_in * threads * 16 : 0;
  if (staged && staged <= kStageMax) {
    q.stages = kStages;
    smem += staged;
  }
  if (smem > 32 * 1024) {   // with the static arrays, above the default 48 KB
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<units, threads, smem, stream>>>(q);
  return cudaGetLastError();
}

template <typename T, int VEC, int ITEMS>
cudaError_t launch_bwd_g(const NormBwdParams &q, int gate, int units, cudaStream_t stream) {
  if (gate == kGateNone) return launch_bwd_t<T, VEC, ITEMS, kGateNone>(q, units, stream);
  if (gate == kGateEach) return launch_bwd_t<T, VEC, ITEMS, kGateEach>(q, units, stream);
  return launch_bwd_t<T, VEC, ITEMS, kGateGroup>(q, units, stream);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_block_norm_fwd(const kda_norm_desc *d, const void *y, const float *w_post,
                              const void *residual, const void *gate, const float *w_pre,
                              void *out, void *x, float *stats, kda_stream_t stream) {
  const kda_status st = check_desc(d, gate != nullptr);
  if (st != KDA_OK) return st;
  if (!y || !w_post || !out || (w_pre != nullptr) != (x != nullptr)) return KDA_ERR_INVALID_ARG;
  const bool bf16 = d->dtype == KDA_DTYPE_BF16;
  bool vec = true;
  for (const void *ptr : {y, (const void *)w_post, residual, gate, (const void *)w_pre,
                          (const void *)out, (const void *)x})
    vec = vec && aligned16(ptr);
  const Layout l = layout_for(d->dim, bf16 ? 2 : 4, vec);
  NormParams p = params_of(d, l, y, w_post, residual, gate, w_pre);
  p.out = out; p.x = x; p.stats = stats;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorNotSupported;
  using B = __nv_bfloat16;
  if (l.vec > 1 && bf16)
    e = l.items == 1 ? launch_fwd_t<B, 8, 1>(p, cs) : l.items == 2 ? launch_fwd_t<B, 8, 2>(p, cs)
                                                                   : launch_fwd_t<B, 8, 4>(p, cs);
  else if (l.vec > 1)
    e = l.items == 1   ? launch_fwd_t<float, 4, 1>(p, cs)
        : l.items == 2 ? launch_fwd_t<float, 4, 2>(p, cs)
        : l.items == 4 ? launch_fwd_t<float, 4, 4>(p, cs)
                       : launch_fwd_t<float, 4, 8>(p, cs);
  else if (bf16)
    e = l.items == 4 ? launch_fwd_t<B, 1, 4>(p, cs) : launch_fwd_t<B, 1, 16>(p, cs);
  else
    e = l.items == 4 ? launch_fwd_t<float, 1, 4>(p, cs) : launch_fwd_t<float, 1, 16>(p, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_block_norm_bwd_workspace_size(const kda_norm_desc *d, int has_gate) {
  if (check_desc(d, has_gate != 0) != KDA_OK) return 0;
  // the largest over the layouts, since types and pointers choose between them
  size_t n = 0;
  for (int v = 0; v < 3; ++v) {
    const Layout l = layout_for(d->dim, v == 1 ? 2 : 4, v != 0);
    size_t units = (size_t)units_for(d, l), gate_units = 0;
    if (has_gate && d->gate_rows < d->rows) {
      const int s = splits_for(d, l, (int)units);
      if (s) gate_units = units = (size_t)(s * d->gate_rows);
    }
    const size_t m = (2 * units + gate_units) * (size_t)d->dim * sizeof(float);
    if (m > n) n = m;
  }
  return align_up(n, 256);
}

kda_status kda_block_norm_bwd(const kda_norm_desc *d, const void *y, const float *w_post,
                              const void *residual, const void *gate, const float *w_pre,
                              const float *stats, const void *d_out, const void *d_x, void *dy,
                              void *d_residual, void *d_gate, float *dw_post, float *dw_pre,
                              void *workspace, size_t workspace_bytes, kda_stream_t stream) {
  const kda_status st = check_desc(d, gate != nullptr);
  if (st != KDA_OK) return st;
  if (!y || !w_post || !stats || !dy || !dw_post || (!d_out && !d_x)) return KDA_ERR_INVALID_ARG;
  if ((w_pre != nullptr) != (dw_pre != nullptr) || (d_x && !w_pre)) return KDA_ERR_INVALID_ARG;
  if ((d_residual && !residual) || (d_gate && !gate)) return KDA_ERR_INVALID_ARG;
  const size_t need = kda_block_norm_bwd_workspace_size(d, gate != nullptr);
  if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KDA_ERR_ALIGNMENT;
  const bool bf16 = d->dtype == KDA_DTYPE_BF16;
  bool vec = true;
  for (const void *ptr : {y, (const void *)w_post, residual, gate, (const void *)w_pre, d_out, d_x,
                          (const void *)dy, (const void *)d_residual, (const void *)d_gate})
    vec = vec && aligned16(ptr);
  const Layout l = layout_for(d->dim, bf16 ? 2 : 4, vec);
  NormBwdParams q = {};
  q.f = params_of(d, l, y, w_post, residual, gate, w_pre);
  q.f.stats = const_cast<float *>(stats);
  q.d_out = d_out; q.d_x = d_x; q.dy = dy; q.d_res = d_residual; q.d_gate = d_gate;
  q.gate_rows = gate ? d->gate_rows : 0;
  const int mode = !gate ? kGateNone : d->gate_rows == d->rows ? kGateEach : kGateGroup;
  q.n_in = 1 + (d_out != nullptr) + (d_x != nullptr) + (residual != nullptr) + (mode == kGateEach);
  int units = units_for(d, l);
  if (mode == kGateGroup) {
    q.splits = splits_for(d, l, units);
    if (q.splits) units = (int)(q.splits * d->gate_rows);
  }
  float *ws = static_cast<float *>(workspace);
  q.part_post = ws;
  q.part_pre = ws + (size_t)units * d->dim;
  q.part_gate = ws + (size_t)2 * units * d->dim;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorNotSupported;
  using B = __nv_bfloat16;
  if (l.vec > 1 && bf16)
    e = l.items == 1   ? launch_bwd_g<B, 8, 1>(q, mode, units, cs)
        : l.items == 2 ? launch_bwd_g<B, 8, 2>(q, mode, units, cs)
                       : launch_bwd_g<B, 8, 4>(q, mode, units, cs);
  else if (l.vec > 1)
    e = l.items == 1   ? launch_bwd_g<float, 4, 1>(q, mode, units, cs)
        : l.items == 2 ? launch_bwd_g<float, 4, 2>(q, mode, units, cs)
        : l.items == 4 ? launch_bwd_g<float, 4, 4>(q, mode, units, cs)
                       : launch_bwd_g<float, 4, 8>(q, mode, units, cs);
  else if (bf16)
    e = l.items == 4 ? launch_bwd_g<B, 1, 4>(q, mode, units, cs)
                     : launch_bwd_g<B, 1, 16>(q, mode, units, cs);
  else
    e = l.items == 4 ? launch_bwd_g<float, 1, 4>(q, mode, units, cs)
                     : launch_bwd_g<float, 1, 16>(q, mode, units, cs);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  const bool gate_parts = mode == kGateGroup && q.splits && d_gate;
  const dim3 grid((d->dim + 31) / 32, 2 + (gate_parts ? (unsigned)d->gate_rows : 0));
  const float *pre = w_pre ? q.part_pre : nullptr;
  if (bf16)
    norm_sum_kernel<B><<<grid, 1024, 0, cs>>>(q.part_post, pre, q.part_gate, dw_post, dw_pre,
                                              (B *)d_gate, units, q.splits, d->dim);
  else
    norm_sum_kernel<float><<<grid, 1024, 0, cs>>>(q.part_post, pre, q.part_gate, dw_post, dw_pre,
                                                  (float *)d_gate, units, q.splits, d->dim);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
