// kda_norm.cuh -- what the block norms' forward and backward kernels share:
// how a row lies over threads, pairs of values, gates, row sums, the staged
// rows.  Internal.
#pragma once

#include <type_traits>

#include "kda_f32x2.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace norm {

constexpr int kMaxDim = 16384;
constexpr int kBlock = 256;        // threads of a CTA that holds several rows

enum { kGateNone = 0, kGateEach = 1, kGateGroup = 2 };

// A row belongs to `tpr` threads (a power of two up to a warp, else whole
// warps), each owning `items` pieces of `vec` elements that lie tpr pieces
// apart; a CTA holds `rg` rows when a row needs fewer than 256 threads.
struct Layout {
  int vec;      // elements per access: 16 bytes, 2 (bf16, even rows); 1: fp32, or pairs
                // of bf16 whose rows need not begin on a word
  int items, tpr, rg;
  int bs;       // most threads of the kernel
};

// A kernel that is built: pieces of `vec` elements, `items` of them per thread,
// CTAs of up to `bs` threads.
struct Built {
  int elt, vec, items, bs;
};

// The first kernel whose CTA covers a row.
template <int N>
Layout layout_for(const Built (&built)[N], int D, int elt, bool vector_ok) {
  Layout l;
  l.vec = !vector_ok ? 1 : D % (16 / elt) == 0 ? 16 / elt : elt == 2 && D % 2 == 0 ? 2 : 1;
  const int n = l.vec == 1 && elt == 2 ? (D + 1) / 2 : D / l.vec;
  for (const Built &k : built)
    if (k.elt == elt && k.vec == l.vec && k.items * k.bs >= n) {
      l.items = k.items;
      l.bs = k.bs;
      break;
    }
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

kda_status check_desc(const kda_norm_desc *d, bool has_gate);
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline int gate_mode(const kda_norm_desc *d, const void *gate) {
  return !gate ? kGateNone : d->gate_rows == d->rows ? kGateEach : kGateGroup;
}
inline NormParams params_of(const kda_norm_desc *d, const Layout &l, const void *y,
                            const float *w_post, const void *res, const void *gate,
                            const float *w_pre) {
  NormParams p = {};
  p.R = d->rows; p.D = d->dim; p.tpr = l.tpr; p.rg = l.rg; p.act = d->gate_act;
  p.scale = d->scale; p.eps = d->eps; p.inv_d = 1.f / (float)d->dim;
  p.rows_per_gate = gate ? (unsigned)(d->rows / d->gate_rows) : 1u;
  p.y = y; p.res = res; p.gate = gate; p.w_post = w_post; p.w_pre = w_pre;
  return p;
}
template <typename K>
cudaError_t allow_smem(K kern, size_t smem) {
  // with the static arrays, above the default 48 KB
  return smem > 32 * 1024
             ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
             : cudaSuccess;
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

// A piece of kStep elements in memory (Raw) and in registers (E values of type
// P).  `whole` is false for a ragged piece of which only the first element lies
// in the row; its second one reads as 0 and is not written.
template <typename T, int VEC>
struct Piece {
  static_assert(VEC * sizeof(T) == 16 || (VEC == 2 && sizeof(T) == 2), "accesses");
  using Raw = typename std::conditional<VEC * sizeof(T) == 16, uint4, uint32_t>::type;
  using P = P2;
  static constexpr int E = VEC / 2, kStep = VEC;
  static constexpr bool kRagged = false;
  static __device__ __forceinline__ void get(const Raw &a, P2 (&f)[E]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&a);
#pragma unroll
    for (int i = 0; i < E; ++i)
      f[i].v = sizeof(T) == 4
                   ? pk2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]))
                   : pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ Raw read(const void *p, bool) {
    return *static_cast<const Raw *>(p);
  }
  static __device__ __forceinline__ void write(void *p, const P2 (&f)[E], bool) {
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
    *static_cast<Raw *>(p) = a;
  }
  static __device__ __forceinline__ void weight(const float *w, P2 (&f)[E], bool) {
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
  static __device__ __forceinline__ void store(float *w, const P2 (&f)[E], bool) {
#pragma unroll
    for (int i = 0; i < E; ++i) upk2(f[i].v, w[2 * i], w[2 * i + 1]);
  }
};
template <>
struct Piece<float, 1> {
  using Raw = float;
  using P = P1;
  static constexpr int E = 1, kStep = 1;
  static constexpr bool kRagged = false;
  static __device__ __forceinline__ void get(const Raw &a, P1 (&f)[1]) { f[0].v = a; }
  static __device__ __forceinline__ Raw read(const void *p, bool) {
    return *static_cast<const float *>(p);
  }
  static __device__ __forceinline__ void write(void *p, const P1 (&f)[1], bool) {
    *static_cast<float *>(p) = f[0].v;
  }
  static __device__ __forceinline__ void weight(const float *w, P1 (&f)[1], bool) { f[0].v = *w; }
  static __device__ __forceinline__ void store(float *w, const P1 (&f)[1], bool) { *w = f[0].v; }
};
template <>
struct Piece<__nv_bfloat16, 1> {
  using Raw = uint32_t;
  using P = P2;
  static constexpr int E = 1, kStep = 2;
  static constexpr bool kRagged = true;
  static __device__ __forceinline__ void get(const Raw &a, P2 (&f)[1]) {
    f[0].v = pk2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
  static __device__ __forceinline__ Raw read(const void *p, bool whole) {
    const unsigned short *h = static_cast<const unsigned short *>(p);
    return (uint32_t)h[0] | (whole ? (uint32_t)h[1] << 16 : 0u);
  }
  static __device__ __forceinline__ void write(void *p, const P2 (&f)[1], bool whole) {
    float x, y;
    upk2(f[0].v, x, y);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const uint32_t a = *reinterpret_cast<const uint32_t *>(&h);
    unsigned short *o = static_cast<unsigned short *>(p);
    if (whole && (reinterpret_cast<uintptr_t>(p) & 2) == 0) {
      *reinterpret_cast<uint32_t *>(o) = a;
    } else {
      o[0] = (unsigned short)a;
      if (whole) o[1] = (unsigned short)(a >> 16);
    }
  }
  static __device__ __forceinline__ void weight(const float *w, P2 (&f)[1], bool whole) {
    f[0].v = pk2(w[0], whole ? w[1] : 0.f);
  }
  static __device__ __forceinline__ void store(float *w, const P2 (&f)[1], bool whole) {
    float x, y;
    upk2(f[0].v, x, y);
    w[0] = x;
    if (whole) w[1] = y;
  }
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

// Sums over the tpr threads of a row, in every thread of the row.  `slot`
// alternates between two buffers, so one barrier is enough.
__device__ __forceinline__ float row_sum(float v, int tpr, float (*red)[32], int &slot) {
  if (tpr < 32) {
    for (int off = tpr >> 1; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (tpr > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[slot][warp] = v;
    __syncthreads();
    const int nw = tpr >> 5, first = warp / nw * nw;
    v = lane < nw ? red[slot][first + lane] : 0.f;
    if (nw <= 8) {
#pragma unroll
      for (int off = 4; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      v = __shfl_sync(0xffffffffu, v, 0);
    } else {
#pragma unroll
      for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    }
    slot ^= 1;
  }
  return v;
}

// Three sums at once.  In a warp the lanes split the values after the first
// exchange, so that six shuffles do instead of fifteen, and likewise over
// the warps.
__device__ __forceinline__ void row_sum3(float (&v)[3], int tpr, float (*red)[4][32], int &slot) {
  if (tpr < 32) {
    for (int off = tpr >> 1; off; off >>= 1)
#pragma unroll
      for (int i = 0; i < 3; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // lanes 0..7 end with value 0, 8..15 value 1, 16..23 value 2, 24..31 zero
  float x = lane & 16 ? v[2] : v[0], y = lane & 16 ? 0.f : v[1];
  x += __shfl_xor_sync(0xffffffffu, lane & 16 ? v[0] : v[2], 16);
  y += __shfl_xor_sync(0xffffffffu, lane & 16 ? v[1] : 0.f, 16);
  float z = lane & 8 ? y : x;
  z += __shfl_xor_sync(0xffffffffu, lane & 8 ? x : y, 8);
#pragma unroll
  for (int off = 4; off; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
  if (tpr > 32) {
    if ((lane & 7) == 0) red[slot][lane >> 3][warp] = z;
    __syncthreads();
    const int nw = tpr >> 5, first = warp / nw * nw;
    z = 0.f;
    for (int w = lane & 7; w < nw; w += 8) z += red[slot][lane >> 3][first + w];
#pragma unroll
    for (int off = 4; off; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    slot ^= 1;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) v[i] = __shfl_sync(0xffffffffu, z, 8 * i);
}

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The rows to come, copied to shared memory NS - 1 ahead (NS = 0: inputs are
// read where they are used).  Pieces of 4 or 16 bytes: a thread copies its
// own, [stage][input][item][BS threads], and no barrier guards them.  Ragged
// rows start in the middle of a word: their words are copied by whoever
// comes, [stage][input][row group][row], and one barrier per row lets every
// thread read its elements.
template <typename T, int VEC, int ITEMS, int NIN, int BS, int NS>
struct Stage {
  using Pc = Piece<T, VEC>;
  using Raw = typename Pc::Raw;
  static constexpr bool kShared = Pc::kRagged;
  unsigned char *base;  // of this thread, or of its row group
  const char *src[NIN]; // the inputs, null where absent
  int lane, tpr, D;
  int pitch;            // kShared: bytes between the stages' inputs

  static __host__ __device__ int row_pitch(int D) { return (2 * D + 2 + 15) / 16 * 16; }
  static size_t bytes(int D, int rg) {
    if (NS == 0) return 0;
    return kShared ? (size_t)NS * NIN * rg * row_pitch(D)
                   : (size_t)NS * NIN * ITEMS * BS * sizeof(Raw);
  }
  __device__ __forceinline__ void init(unsigned char *smem, int tid, int group, int rg) {
    base = kShared ? smem + (size_t)group * row_pitch(D) : smem + tid * sizeof(Raw);
    pitch = rg * row_pitch(D);
  }

  // Byte of a ragged row's first element within its first word.
  __device__ __forceinline__ int odd(int k, long long row) const {
    return (int)((reinterpret_cast<uintptr_t>(src[k]) ^ (uintptr_t)((row & D) << 1)) & 2);
  }
  // row: its number; bytes: the thread's first piece; step: between pieces
  __device__ __forceinline__ void fetch(int st, bool live, const bool (&has)[ITEMS], long long row,
                                        long long bytes, int step) const {
    if constexpr (NS > 0) {
      if (live) {
        if constexpr (kShared) {
          const long long start = row * D * 2;
#pragma unroll
          for (int k = 0; k < NIN; ++k)
            if (src[k]) {
              const char *s = src[k] + start;
              // whole words by cp.async, a half word at either end by hand;
              // element c lies at byte 2 c + (address of the row & 2)
              const int o = odd(k, row);
              unsigned char *d = base + (st * NIN + k) * pitch;
              const int words = (2 * D - o) / 4;
              const uint32_t ds = (uint32_t)__cvta_generic_to_shared(d) + 2 * o;
              for (int w = lane; w < words; w += tpr) cp_async4(ds + 4 * w, s + o + 4 * w);
              if (o && lane == 0) *reinterpret_cast<T *>(d + 2) = *reinterpret_cast<const T *>(s);
              if (2 * D - o - 4 * words && lane == tpr - 1)
                *reinterpret_cast<T *>(d + o + 2 * D - 2) =
                    *reinterpret_cast<const T *>(s + 2 * D - 2);
            }
        } else {
          const uint32_t d = (uint32_t)__cvta_generic_to_shared(base) +
                             (uint32_t)(st * NIN * ITEMS * BS * sizeof(Raw));
#pragma unroll
          for (int k = 0; k < NIN; ++k)
            if (src[k]) {
#pragma unroll
              for (int i = 0; i < ITEMS; ++i)
                if (has[i]) {
                  const uint32_t to = d + (uint32_t)((k * ITEMS + i) * BS * sizeof(Raw));
                  const char *from = src[k] + bytes + (long long)i * step;
                  if constexpr (sizeof(Raw) == 16) cp_async16(to, from);
                  else cp_async4(to, from);
                }
            }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  // Asks for a row to come and waits for the present one.
  template <typename F>
  __device__ __forceinline__ void turn(F ask) const {
    if constexpr (NS > 0 && kShared) {
      static_assert(NS == 2, "one row ahead");
      cp_async_wait<0>();
      __syncthreads();       // the row is there, the one before is read
      ask();
    } else if constexpr (NS > 0) {
      ask();
      cp_async_wait<NS - 1>();
    }
  }
  __device__ __forceinline__ Raw get(int st, int k, int i, bool whole, long long row,
                                     long long bytes, int step) const {
    if constexpr (NS > 0 && kShared)
      return Pc::read(base + (st * NIN + k) * pitch + odd(k, row) + 4 * (lane + i * tpr), whole);
    else if constexpr (NS > 0)
      return Pc::read(base + ((st * NIN + k) * ITEMS + i) * BS * sizeof(Raw), true);
    else
      return Pc::read(src[k] + bytes + (long long)i * step, whole);
  }
};

}  // namespace norm
}  // namespace kda
