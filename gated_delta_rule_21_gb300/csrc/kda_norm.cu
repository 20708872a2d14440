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
// accesses take the same code with VEC = 2 (bf16 rows of even length) or 1.
#include <type_traits>

#include "kda_f32x2.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kMaxDim = 16384;
constexpr int kBlock = 256;        // threads when a row needs at most these
constexpr int kStages = 3;         // rows staged per thread in the backward
constexpr size_t kStageMax = 200 * 1024;   // longer rows are read directly

enum { kGateNone = 0, kGateEach = 1, kGateGroup = 2 };

// How a row is laid over threads.
struct Layout {
  int vec;      // elements per access: 16 bytes, 2 (bf16, even rows) or 1
  int items;    // accesses per thread and row
  int tpr;      // threads per row
  int rg;       // rows per CTA
};

// Forward: 16 elements per thread, so that a row's two reductions weigh little
// (at 8, 4096 bf16 elements took 87 us for 8192 rows, bound by issue).
// Backward: 8, whose intermediate values then stay in registers.
Layout layout_for(int D, int elt, bool vector_ok, bool forward) {
  Layout l;
  l.vec = !vector_ok ? 1 : D % (16 / elt) == 0 ? 16 / elt : elt == 2 && D % 2 == 0 ? 2 : 1;
  const int n = D / l.vec;
  const int most = l.vec > 2 ? 512 : 1024;     // threads of one row
  // the kernels' numbers of accesses: 1, 2, 4, 8; vec 2: 2, 8; vec 1: 4, 16
  l.items = l.vec > 2 ? (forward ? 16 / l.vec : 1) : l.vec == 2 ? 2 : 4;
  while (l.items * most < n) l.items *= l.vec > 2 ? 2 : 4;
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

// One or two fp32 values: pairs use the packed f32x2 instructions, which
// halve the arithmetic a row costs.
struct P1 { float v; };
struct P2 { u64 v; };
__device__ __forceinline__ P1 mul(P1 a, P1 b) { return {a.v * b.v}; }
__device__ __forceinline__ P1 add(P1 a, P1 b) { return {a.v + b.v}; }
__device__ __forceinline__ P1 fma(P1 a, P1 b, P1 c) { return {fmaf(a.v, b.v, c.v)}; }
__device__ __forceinline__ float total(P1 a) { return a.v; }
__device__ __forceinline__ P2 mul(P2 a, P2 b) { return {mul2(a.v, b.v)}; }
__device__ __forceinline__ P2 add(P2 a, P2 b) { return {add2(a.v, b.v)}; }
__device__ __forceinline__ P2 fma(P2 a, P2 b, P2 c) { return {fma2(a.v, b.v, c.v)}; }
__device__ __forceinline__ float total(P2 a) {
  float x, y;
  upk2(a.v, x, y);
  return x + y;
}
template <typename P> __device__ __forceinline__ P both(float a);
template <> __device__ __forceinline__ P1 both<P1>(float a) { return {a}; }
template <> __device__ __forceinline__ P2 both<P2>(float a) { return {pk2(a, a)}; }

// VEC elements in memory (Raw) and in registers (E values of type P).
template <typename T, int VEC>
struct Piece {
  static_assert(VEC * sizeof(T) == 16 || (VEC == 2 && sizeof(T) == 2), "accesses");
  using Raw = typename std::conditional<VEC * sizeof(T) == 16, uint4, uint32_t>::type;
  using P = P2;
  static constexpr int E = VEC / 2;
  static __device__ __forceinline__ void get(const Raw &a, P2 (&f)[E]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&a);
#pragma unroll
    for (int i = 0; i < E; ++i)
      f[i].v = sizeof(T) == 4
                   ? pk2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]))
                   : pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ Raw put(const P2 (&f)[E]) {
    Raw a;
    uint32_t *w = reinterpret_cast<uint32_t *>(&a);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      float x, y;
      upk2(f[i].v, x, y);
      if (sizeof(T) == 4) {
        w[2 * i] = __float_as_uint(x);
        w[2 * i + 1] = __float_as_uint(y);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    return a;
  }
  static __device__ __forceinline__ void weight(const float *w, P2 (&f)[E]) {
    if constexpr (VEC == 2) {
      const float2 a = *reinterpret_cast<const float2 *>(w);
      f[0].v = pk2(a.x, a.y);
    } else {
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float4 a = *reinterpret_cast<const float4 *>(w + 2 * i);
        f[i].v = pk2(a.x, a.y);
        f[i + 1].v = pk2(a.z, a.w);
      }
    }
  }
  static __device__ __forceinline__ void store(float *w, const P2 (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) upk2(f[i].v, w[2 * i], w[2 * i + 1]);
  }
};
template <typename T>
struct Piece<T, 1> {
  using Raw = T;
  using P = P1;
  static constexpr int E = 1;
  static __device__ __forceinline__ void get(const Raw &a, P1 (&f)[1]) { f[0].v = to_f32(a); }
  static __device__ __forceinline__ Raw put(const P1 (&f)[1]) { return from_f32<T>(f[0].v); }
  static __device__ __forceinline__ void weight(const float *w, P1 (&f)[1]) { f[0].v = *w; }
  static __device__ __forceinline__ void store(float *w, const P1 (&f)[1]) { *w = f[0].v; }
};

__device__ __forceinline__ float sfu_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sfu_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// act(a), and its derivative when DER, from the approximate exp2 and
// reciprocal (a few fp32 ulp).  tanh a = 1 - 2 / (1 + e^2a) loses digits near
// 0: below 0.3 it is its Taylor series to a^9, whose rest is 6e-8 of it.
template <bool DER, int ACT>
__device__ __forceinline__ void gate_one(float a, float &v, float &d) {
  if (ACT == KDA_GATE_TANH) {
    const float q = a * a;
    const float s = a + a * q * (-1.f / 3 + q * (2.f / 15 + q * (-17.f / 315 + q * (62.f / 2835))));
    const float l = 1.f - 2.f * sfu_rcp(1.f + sfu_ex2(2.f * kLog2e * a));
    v = q < 0.09f ? s : l;
    if (DER) d = 1.f - v * v;
    return;
  }
  const float s = sfu_rcp(1.f + sfu_ex2(-kLog2e * a));
  if (ACT == KDA_GATE_SIGMOID) {
    v = s;
    if (DER) d = s * (1.f - s);
  } else {
    v = a * s;
    if (DER) d = s * (1.f + a * (1.f - s));
  }
}
template <bool DER, int ACT>
__device__ __forceinline__ void gate_one(P1 a, P1 &v, P1 &d) {
  gate_one<DER, ACT>(a.v, v.v, d.v);
}
template <bool DER, int ACT>
__device__ __forceinline__ void gate_one(P2 a, P2 &v, P2 &d) {
  float x, y, vx, vy, dx = 0.f, dy = 0.f;
  upk2(a.v, x, y);
  gate_one<DER, ACT>(x, vx, dx);
  gate_one<DER, ACT>(y, vy, dy);
  v.v = pk2(vx, vy);
  if (DER) d.v = pk2(dx, dy);
}
// a[] becomes act(a[]), d[] the derivative; one branch for all of them.
template <bool DER, typename P, int E>
__device__ __forceinline__ void gate_values(int act, P (&a)[E], P (&d)[E]) {
  if (act == KDA_GATE_SILU) {
#pragma unroll
    for (int e = 0; e < E; ++e) gate_one<DER, KDA_GATE_SILU>(a[e], a[e], d[e]);
  } else if (act == KDA_GATE_SIGMOID) {
#pragma unroll
    for (int e = 0; e < E; ++e) gate_one<DER, KDA_GATE_SIGMOID>(a[e], a[e], d[e]);
  } else if (act == KDA_GATE_TANH) {
#pragma unroll
    for (int e = 0; e < E; ++e) gate_one<DER, KDA_GATE_TANH>(a[e], a[e], d[e]);
  } else if (DER) {
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] = both<P>(1.f);
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
    for (int i = 0; i < N; ++i) v[i] = lane < nw ? red[slot][i][first + lane] : 0.f;
    // the values lie in the first nw lanes; the sum is needed in all
    if (nw <= 8) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int off = 4; off; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
        v[i] = __shfl_sync(0xffffffffu, v[i], 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int off = 16; off; off >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
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
  int n_in;        // input arrays staged per row
  int stages;      // kStages, or 0: inputs are read where they are used
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's own pieces of the rows to come, copied to shared memory
// kStages - 1 rows ahead.  With stages = 0 (rows too long, or accesses of
// less than 16 bytes) pieces are read where they are used.
template <typename T, int VEC, int ITEMS>
struct Stage {
  using Raw = typename Piece<T, VEC>::Raw;
  static constexpr bool kAsync = sizeof(Raw) == 16;
  Raw *base;
  int n_in, nthr, stages, D, lane, tpr;

  template <typename... A>
  __device__ __forceinline__ void fetch(int st, bool live, size_t row, const A *...arrays) const {
    if constexpr (kAsync) {
      if (stages && live) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int c = (lane + i * tpr) * VEC;
          if (c < D) {
            Raw *d = base + (size_t)(st * ITEMS + i) * n_in * nthr;
            ((arrays ? (cp_async16(d, static_cast<const T *>(arrays) + row + c), d += nthr) : d), ...);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  // piece `i` of input number `k` (which is `array`)
  __device__ __forceinline__ Raw get(int st, int i, int k, const void *array, size_t row) const {
    if (kAsync && stages) return base[((size_t)(st * ITEMS + i) * n_in + k) * nthr];
    return *reinterpret_cast<const Raw *>(static_cast<const T *>(array) + row +
                                          (lane + i * tpr) * VEC);
  }
};

// A CTA owns a contiguous range of rows, one row per row group at a time; of
// a gate row shared by rows act(gate) is made once.
template <typename T, int VEC, int ITEMS, int GATE>
__global__ void __launch_bounds__(VEC > 2 ? 512 : 1024) norm_fwd_kernel(const NormParams p) {
  using Pc = Piece<T, VEC>;
  using P = typename Pc::P;
  using Raw = typename Pc::Raw;
  constexpr int E = Pc::E;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][1][32];
  const int tid = threadIdx.x, tpr = p.tpr, rg = p.rg;
  const int group = tid / tpr, lane = tid - group * tpr;
  const Stage<T, VEC, ITEMS> in = {reinterpret_cast<Raw *>(smem) + tid, p.n_in, (int)blockDim.x,
                                   p.stages, p.D, lane, tpr};
  const int k_res = 1, k_gate = 1 + (p.res != nullptr);
  int slot = 0, st = 0;
  const long long lo = (long long)blockIdx.x * p.R / gridDim.x,
                  hi = (long long)(blockIdx.x + 1) * p.R / gridDim.x;
  auto fetch = [&](long long row, int s) {
    in.fetch(s, row < hi, (size_t)row * p.D, (const T *)p.y, (const T *)p.res,
             GATE == kGateEach ? (const T *)p.gate : (const T *)nullptr);
  };
  constexpr int GI = GATE == kGateGroup ? ITEMS : 1;
  P ga[GI][E];
  unsigned ga_row = ~0u;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(lo + group + s * rg, s);
  for (long long r0 = lo; r0 < hi; r0 += rg) {
    const long long row = r0 + group;
    const bool live = row < hi;
    const size_t at = (size_t)row * p.D;
    fetch(row + (kStages - 1) * rg, st == 0 ? kStages - 1 : st - 1);
    if (GATE == kGateGroup && live) {
      const unsigned g = (unsigned)row / p.rows_per_gate;
      if (g != ga_row) {
        ga_row = g;
#pragma unroll
        for (int i = 0; i < GI; ++i) {
          const int c = (lane + i * tpr) * VEC;
          P d[E];
          if (c < p.D) {
            Pc::get(*reinterpret_cast<const Raw *>((const T *)p.gate + (size_t)g * p.D + c), ga[i]);
            gate_values<false>(p.act, ga[i], d);
          }
        }
      }
    }
    if (in.kAsync) cp_async_wait<kStages - 1>();
    P v[ITEMS][E], acc = both<P>(0.f);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = both<P>(0.f);
      if (live && (lane + i * tpr) * VEC < p.D) Pc::get(in.get(st, i, 0, p.y, at), v[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc = fma(v[i][e], v[i][e], acc);
    }
    float ss[1] = {total(acc)};
    row_sum(ss, tpr, red, slot);
    const float s1 = rsqrtf(ss[0] * p.inv_d + p.eps);
    const P k = both<P>(s1 * p.scale);
    acc = both<P>(0.f);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = (lane + i * tpr) * VEC;
      if (live && c < p.D) {
        P w[E], a[E];
        Pc::weight(p.w_post + c, w);
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = mul(mul(v[i][e], k), w[e]);
        if (GATE == kGateEach) {
          Pc::get(in.get(st, i, k_gate, p.gate, at), a);
          P d[E];
          gate_values<false>(p.act, a, d);
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = mul(v[i][e], a[e]);
        }
        if (GATE == kGateGroup)
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = mul(v[i][e], ga[i < GI ? i : 0][e]);
        if (p.res) {
          Pc::get(in.get(st, i, k_res, p.res, at), a);
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = add(v[i][e], a[e]);
        }
        *reinterpret_cast<Raw *>((T *)p.out + at + c) = Pc::put(v[i]);
#pragma unroll
        for (int e = 0; e < E; ++e) acc = fma(v[i][e], v[i][e], acc);
      }
    }
    float s2 = 0.f;
    if (p.w_pre) {
      ss[0] = total(acc);
      row_sum(ss, tpr, red, slot);
      s2 = rsqrtf(ss[0] * p.inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = (lane + i * tpr) * VEC;
        if (live && c < p.D) {
          P w[E];
          Pc::weight(p.w_pre + c, w);
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = mul(mul(v[i][e], both<P>(s2)), w[e]);
          *reinterpret_cast<Raw *>((T *)p.x + at + c) = Pc::put(v[i]);
        }
      }
    }
    if (p.stats && live && lane == 0) {
      p.stats[row] = s1;
      p.stats[p.R + row] = s2;
    }
    st = st + 1 == kStages ? 0 : st + 1;
  }
  if (in.kAsync) cp_async_wait<0>();
}

struct NormBwdParams {
  NormParams f;
  const void *d_out, *d_x;
  void *dy, *d_res, *d_gate;
  float *part_post, *part_pre, *part_gate;   // [units][D]
  long long gate_rows;
  int splits;      // units per gate row (group gates), 0: whole gate rows per unit
};

// Sums `acc` over the CTA's row groups and hands the totals to the first
// group's threads: put(column, values).  Uniform over the CTA.
template <typename Pc, int ITEMS, int VEC, typename F>
__device__ __forceinline__ void flush(typename Pc::P (&acc)[ITEMS][Pc::E], int tpr, int rg,
                                      int group, int lane, int D, typename Pc::P *buf, F put) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = (lane + i * tpr) * VEC;
    if (rg > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < Pc::E; ++e) buf[threadIdx.x * Pc::E + e] = acc[i][e];
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < rg; ++g)
#pragma unroll
          for (int e = 0; e < Pc::E; ++e)
            acc[i][e] = add(acc[i][e], buf[(g * tpr + lane) * Pc::E + e]);
    }
    if (group == 0 && c < D) put(i, c, acc[i]);
  }
}

// A unit (CTA) owns a contiguous range of rows, keeps its column sums in
// registers and writes them once; the units' sums are added in a fixed order
// by norm_sum_kernel, so no result depends on timing.
//
// With m = out, v = d_out + s2 d_x w_pre and q = aw n1 (aw = scale act(gate)
// w_post), a row needs sum(d_x w_pre m), sum(q v) and sum(q m); then
//   r = v - k m,  dy = s1 (aw r - c1 n1),
// and the column sums of r n1 give dw_post and (gate rows shared by rows,
// where act(gate) is a factor of the column) d_gate at once.  One piece per
// thread keeps these values for the second pass over the row, more pieces
// make them again from the staged inputs.
template <typename T, int VEC, int ITEMS, int GATE>
__global__ void __launch_bounds__(VEC > 2 ? 512 : 1024) norm_bwd_kernel(const NormBwdParams q) {
  using Pc = Piece<T, VEC>;
  using P = typename Pc::P;
  using Raw = typename Pc::Raw;
  constexpr int E = Pc::E;
  constexpr bool kKeep = ITEMS == 1;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][3][32];
  const NormParams &p = q.f;
  const int tid = threadIdx.x, tpr = p.tpr, rg = p.rg, nthr = blockDim.x;
  const int group = tid / tpr, lane = tid - group * tpr;
  P *buf = reinterpret_cast<P *>(smem);
  const Stage<T, VEC, ITEMS> in = {
      reinterpret_cast<Raw *>(smem + (rg > 1 ? sizeof(float) * nthr * VEC : 0)) + tid,
      p.n_in, nthr, p.stages, p.D, lane, tpr};
  const int k_out = 1, k_x = k_out + (q.d_out != nullptr), k_res = k_x + (q.d_x != nullptr),
            k_gate = k_res + (p.res != nullptr);
  int slot = 0;

  P dw1[ITEMS][E], dw2[ITEMS][E], w1k[1][E], w2k[1][E];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) dw1[i][e] = dw2[i][e] = both<P>(0.f);
  const P scale = both<P>(p.scale);
  // scale * w_post and w_pre of a piece
  auto weights = [&](int i, P(&w1)[E], P(&w2)[E]) {
    const int c = (lane + i * tpr) * VEC;
#pragma unroll
    for (int e = 0; e < E; ++e) w1[e] = w2[e] = both<P>(0.f);
    if (c < p.D) {
      Pc::weight(p.w_post + c, w1);
      if (p.w_pre) Pc::weight(p.w_pre + c, w2);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) w1[e] = mul(w1[e], scale);
  };
  if (kKeep) weights(0, w1k[0], w2k[0]);

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
    // group gates: act(gate) of the unit's pieces, and the sums of r n1
    constexpr int GI = GATE == kGateGroup ? ITEMS : 1;
    P ga[GI][E], es[GI][E];
    if (GATE == kGateGroup) {
#pragma unroll
      for (int i = 0; i < GI; ++i) {
        const int c = (lane + i * tpr) * VEC;
#pragma unroll
        for (int e = 0; e < E; ++e) es[i][e] = ga[i][e] = both<P>(0.f);
        if (c < p.D) {
          P d[E];
          Pc::get(*reinterpret_cast<const Raw *>((const T *)p.gate + (size_t)g * p.D + c), ga[i]);
          gate_values<false>(p.act, ga[i], d);
        }
      }
    }
    auto fetch = [&](long long row, int s) {
      in.fetch(s, row < hi, (size_t)row * p.D, (const T *)p.y, (const T *)q.d_out,
               (const T *)q.d_x, (const T *)p.res,
               GATE == kGateEach ? (const T *)p.gate : (const T *)nullptr);
    };
    int st = 0;
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(lo + group + s * rg, s);
    for (long long r0 = lo; r0 < hi; r0 += rg) {
      const long long row = r0 + group;
      const bool live = row < hi;
      const size_t at = (size_t)row * p.D;
      float s1 = 0.f, s2 = 0.f;
      if (live) {
        s1 = p.stats[row];
        s2 = p.stats[p.R + row];
      }
      fetch(row + (kStages - 1) * rg, st == 0 ? kStages - 1 : st - 1);
      if (in.kAsync) cp_async_wait<kStages - 1>();
      // n1, m, v, d_x, act(gate) and its derivative of a piece
      auto front = [&](int i, const P(&w1)[E], const P(&w2)[E], P(&n1)[E], P(&m)[E], P(&v)[E],
                       P(&gx)[E], P(&a)[E], P(&da)[E], P(&qv)[E]) {
        Pc::get(in.get(st, i, 0, p.y, at), n1);
        if (q.d_out) Pc::get(in.get(st, i, k_out, q.d_out, at), v);
        else
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = both<P>(0.f);
        if (q.d_x) Pc::get(in.get(st, i, k_x, q.d_x, at), gx);
        else
#pragma unroll
          for (int e = 0; e < E; ++e) gx[e] = both<P>(0.f);
        if (p.res) Pc::get(in.get(st, i, k_res, p.res, at), m);
        else
#pragma unroll
          for (int e = 0; e < E; ++e) m[e] = both<P>(0.f);
        if (GATE == kGateEach) {
          Pc::get(in.get(st, i, k_gate, p.gate, at), a);
          gate_values<true>(p.act, a, da);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          n1[e] = mul(n1[e], both<P>(s1));
          qv[e] = mul(w1[e], n1[e]);
          if (GATE == kGateEach) qv[e] = mul(qv[e], a[e]);
          if (GATE == kGateGroup) qv[e] = mul(qv[e], ga[i < GI ? i : 0][e]);
          m[e] = add(m[e], qv[e]);
          v[e] = fma(mul(gx[e], w2[e]), both<P>(s2), v[e]);
        }
      };
      P n1[1][E], m[1][E], v[1][E], gx[1][E], a[1][E], da[1][E];
      P acc0 = both<P>(0.f), acc1 = acc0, acc2 = acc0;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if (live && (lane + i * tpr) * VEC < p.D) {
          P w1[E], w2[E], qv[E];
          if (!kKeep) weights(i, w1, w2);
          front(i, kKeep ? w1k[0] : w1, kKeep ? w2k[0] : w2, n1[0], m[0], v[0], gx[0], a[0], da[0],
                qv);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            acc0 = fma(mul(gx[0][e], kKeep ? w2k[0][e] : w2[e]), m[0][e], acc0);
            acc1 = fma(qv[e], v[0][e], acc1);
            acc2 = fma(qv[e], m[0][e], acc2);
          }
        }
      }
      float sum[3] = {total(acc0), total(acc1), total(acc2)};
      row_sum(sum, tpr, red, slot);
      const float k = s2 * s2 * s2 * sum[0] * p.inv_d;   // s2 c2, times s2: r = v - k m
      const float c1 = (sum[1] - k * sum[2]) * p.inv_d;
      const P nk = both<P>(-k), nc = both<P>(-c1 * s1), ps1 = both<P>(s1), ps2 = both<P>(s2);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = (lane + i * tpr) * VEC;
        if (live && c < p.D) {
          P w1[E], w2[E], oy[E], og[E], qv[E];
          if (!kKeep) {
            weights(i, w1, w2);
            front(i, w1, w2, n1[0], m[0], v[0], gx[0], a[0], da[0], qv);
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const P w = kKeep ? w1k[0][e] : w1[e];
            dw2[i][e] = fma(mul(gx[0][e], ps2), m[0][e], dw2[i][e]);
            v[0][e] = fma(m[0][e], nk, v[0][e]);            // r
            P aw = w;
            if (GATE == kGateEach) {
              const P x = mul(v[0][e], n1[0][e]);
              dw1[i][e] = fma(a[0][e], x, dw1[i][e]);
              og[e] = mul(mul(w, da[0][e]), x);
              aw = mul(w, a[0][e]);
            } else if (GATE == kGateGroup) {
              es[i < GI ? i : 0][e] = fma(v[0][e], n1[0][e], es[i < GI ? i : 0][e]);
              aw = mul(w, ga[i < GI ? i : 0][e]);
            } else {
              dw1[i][e] = fma(v[0][e], n1[0][e], dw1[i][e]);
            }
            oy[e] = fma(mul(aw, v[0][e]), ps1, mul(n1[0][e], nc));
          }
          *reinterpret_cast<Raw *>((T *)q.dy + at + c) = Pc::put(oy);
          if (q.d_res) *reinterpret_cast<Raw *>((T *)q.d_res + at + c) = Pc::put(v[0]);
          if (GATE == kGateEach && q.d_gate)
            *reinterpret_cast<Raw *>((T *)q.d_gate + at + c) = Pc::put(og);
        }
      }
      st = st + 1 == kStages ? 0 : st + 1;
    }
    if (in.kAsync) cp_async_wait<0>();
    if constexpr (GATE == kGateGroup) {
#pragma unroll
      for (int i = 0; i < GI; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) dw1[i][e] = fma(ga[i][e], es[i][e], dw1[i][e]);
      if (q.d_gate)
        flush<Pc, GI, VEC>(es, tpr, rg, group, lane, p.D, buf, [&](int i, int c, P(&s)[E]) {
          P w1[E], w2[E], a[E], d[E];
          weights(i, w1, w2);
          Pc::get(*reinterpret_cast<const Raw *>((const T *)p.gate + (size_t)g * p.D + c), a);
          gate_values<true>(p.act, a, d);
#pragma unroll
          for (int e = 0; e < E; ++e) a[e] = mul(mul(w1[e], d[e]), s[e]);
          if (q.splits) Pc::store(q.part_gate + (size_t)blockIdx.x * p.D + c, a);
          else *reinterpret_cast<Raw *>((T *)q.d_gate + (size_t)g * p.D + c) = Pc::put(a);
        });
    }
  }
  flush<Pc, ITEMS, VEC>(dw1, tpr, rg, group, lane, p.D, buf, [&](int i, int c, P(&s)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = mul(s[e], scale);
    Pc::store(q.part_post + (size_t)blockIdx.x * p.D + c, s);
  });
  if (p.w_pre)
    flush<Pc, ITEMS, VEC>(dw2, tpr, rg, group, lane, p.D, buf, [&](int i, int c, P(&s)[E]) {
      Pc::store(q.part_pre + (size_t)blockIdx.x * p.D + c, s);
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
#pragma unroll 8
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

// Units (CTAs) of the backward: as many as are resident on 152 SMs at up to
// 128 registers per thread, and no more than there are row groups.
int units_for(const kda_norm_desc *d, const Layout &l) {
  const long long most = 152ll * (l.tpr * l.rg > 256 ? 1 : 2);
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

// Dynamic shared memory of the staged rows (and p.stages).
template <typename T, int VEC, int ITEMS>
size_t stage_bytes(NormParams &p, int threads) {
  if (VEC * sizeof(T) != 16) return 0;
  const size_t n = (size_t)kStages * ITEMS * p.n_in * threads * 16;
  if (n > kStageMax) return 0;
  p.stages = kStages;
  return n;
}
template <typename K>
cudaError_t allow_smem(K kern, size_t smem) {
  // with the static arrays, above the default 48 KB
  return smem > 32 * 1024
             ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
             : cudaSuccess;
}

template <typename T, int VEC, int ITEMS, int GATE>
cudaError_t launch_fwd_g(NormParams p, cudaStream_t stream) {
  auto kern = norm_fwd_kernel<T, VEC, ITEMS, GATE>;
  const int threads = p.tpr * p.rg;
  const size_t smem = stage_bytes<T, VEC, ITEMS>(p, threads);
  cudaError_t e = allow_smem(kern, smem);
  int per_sm = 1;
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
  if (e != cudaSuccess) return e;
  const long long n = (p.R + p.rg - 1) / p.rg, most = (long long)num_sms() * per_sm;
  kern<<<(unsigned)(n < most ? n : most), threads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int VEC, int ITEMS>
cudaError_t launch_fwd_t(const NormParams &p, int gate, cudaStream_t stream) {
  if (gate == kGateNone) return launch_fwd_g<T, VEC, ITEMS, kGateNone>(p, stream);
  if (gate == kGateEach) return launch_fwd_g<T, VEC, ITEMS, kGateEach>(p, stream);
  return launch_fwd_g<T, VEC, ITEMS, kGateGroup>(p, stream);
}

template <typename T, int VEC, int ITEMS, int GATE>
cudaError_t launch_bwd_t(NormBwdParams q, int units, cudaStream_t stream) {
  auto kern = norm_bwd_kernel<T, VEC, ITEMS, GATE>;
  const int threads = q.f.tpr * q.f.rg;
  const size_t smem = (q.f.rg > 1 ? sizeof(float) * threads * VEC : 0) +
                      stage_bytes<T, VEC, ITEMS>(q.f, threads);
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
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
  const Layout l = layout_for(d->dim, bf16 ? 2 : 4, vec, true);
  NormParams p = params_of(d, l, y, w_post, residual, gate, w_pre);
  p.out = out; p.x = x; p.stats = stats;
  const int mode = !gate ? kGateNone : d->gate_rows == d->rows ? kGateEach : kGateGroup;
  p.n_in = 1 + (residual != nullptr) + (mode == kGateEach);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorNotSupported;
  using B = __nv_bfloat16;
  if (l.vec > 2 && bf16)
    e = l.items == 2 ? launch_fwd_t<B, 8, 2>(p, mode, cs) : launch_fwd_t<B, 8, 4>(p, mode, cs);
  else if (l.vec > 2)
    e = l.items == 4 ? launch_fwd_t<float, 4, 4>(p, mode, cs) : launch_fwd_t<float, 4, 8>(p, mode, cs);
  else if (l.vec == 2)
    e = l.items == 2 ? launch_fwd_t<B, 2, 2>(p, mode, cs) : launch_fwd_t<B, 2, 8>(p, mode, cs);
  else if (bf16)
    e = l.items == 4 ? launch_fwd_t<B, 1, 4>(p, mode, cs) : launch_fwd_t<B, 1, 16>(p, mode, cs);
  else
    e = l.items == 4 ? launch_fwd_t<float, 1, 4>(p, mode, cs) : launch_fwd_t<float, 1, 16>(p, mode, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_block_norm_bwd_workspace_size(const kda_norm_desc *d, int has_gate) {
  if (check_desc(d, has_gate != 0) != KDA_OK) return 0;
  // the largest over the layouts, since types and pointers choose between them
  size_t n = 0;
  for (int v = 0; v < 3; ++v) {
    const Layout l = layout_for(d->dim, v == 1 ? 2 : 4, v != 0, false);
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
  const Layout l = layout_for(d->dim, bf16 ? 2 : 4, vec, false);
  NormBwdParams q = {};
  q.f = params_of(d, l, y, w_post, residual, gate, w_pre);
  q.f.stats = const_cast<float *>(stats);
  q.d_out = d_out; q.d_x = d_x; q.dy = dy; q.d_res = d_residual; q.d_gate = d_gate;
  q.gate_rows = gate ? d->gate_rows : 0;
  const int mode = !gate ? kGateNone : d->gate_rows == d->rows ? kGateEach : kGateGroup;
  q.f.n_in = 1 + (d_out != nullptr) + (d_x != nullptr) + (residual != nullptr) + (mode == kGateEach);
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
  if (l.vec > 2 && bf16)
    e = l.items == 1   ? launch_bwd_g<B, 8, 1>(q, mode, units, cs)
        : l.items == 2 ? launch_bwd_g<B, 8, 2>(q, mode, units, cs)
                       : launch_bwd_g<B, 8, 4>(q, mode, units, cs);
  else if (l.vec > 2)
    e = l.items == 1   ? launch_bwd_g<float, 4, 1>(q, mode, units, cs)
        : l.items == 2 ? launch_bwd_g<float, 4, 2>(q, mode, units, cs)
        : l.items == 4 ? launch_bwd_g<float, 4, 4>(q, mode, units, cs)
                       : launch_bwd_g<float, 4, 8>(q, mode, units, cs);
  else if (l.vec == 2)
    e = l.items == 2 ? launch_bwd_g<B, 2, 2>(q, mode, units, cs)
                     : launch_bwd_g<B, 2, 8>(q, mode, units, cs);
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
