// kda_step.cu -- one new token per sequence, on states held in a cache.
//
// Both steps read a sequence's fp32 state [keys][columns] of each head once
// and write it once, which is what bounds them (HBM).  With a the decay:
//
//   ssm_step   S = e^{d A} S + d B (outer) x,  y = (C^T S + D x) SiLU(z)
//              d = softplus(dt + dt_bias); x, B, C from the convolution
//   kda_step   S' = e^g S,  r = v - k^T S',  S = S' + beta k (outer) r,
//              o = scale q^T S = scale (q^T S' + beta (q . k) r)
//
// The second form of o needs only sums over the decayed state, so each step
// is one pass: load the tile, one reduction over the keys, store the tile.
//
// A unit is a tile of TC columns of one (sequence, head); a CTA of 256 threads
// walks units gridDim.x apart.  A thread owns 4 adjacent columns of every
// (1024 / TC)-th key row, so a warp's 16-byte accesses cover whole row
// segments.  While a unit is computed, the next one's state is on its way
// to shared memory (each thread copies its own pieces, so no barrier guards
// them) and its inputs to registers: without that the two barriers of a unit
// left the memory idle (119 and 112 us for the sizes below).
//
// Measured: ssm_step, 128 sequences of 64 heads, 128 x 64 states (537 MB of
// states read and written): 90 us, 88 % of the copy bandwidth; kda_step, 120
// sequences of 32 heads, 128 x 128 (503 MB): 93 us, 80 %; what is left there is
// the two sums of a unit, which have to end before its first store.
//
// The short convolution's cache [3][channels] is moved on in place.  The
// channels of B and C (of q and k) are read by several CTAs, so the last CTA
// of a group to have read them, found by a counter in the workspace, moves
// them; nobody waits.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kTap = 4;             // taps of the convolution
constexpr int kWave = kThreads * 4; // state elements per access of a CTA

// SiLU from the approximate exp2 and reciprocal (a few fp32 ulp).
__device__ __forceinline__ float silu(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return x * r;
}

// The units of a CTA: a fixed column tile of the (sequence, head) pairs that
// lie `pairs` apart (all without a division per unit).
struct Walk {
  int H, B, db, dh;       // pairs = db * H + dh
  int tiles, log_tiles;
};
struct Place {
  int b, h;
  __device__ __forceinline__ void advance(const Walk &w) {
    b += w.db;
    h += w.dh;
    if (h >= w.H) {
      h -= w.H;
      ++b;
    }
  }
};

// Thread 0 counts its CTA in, after a barrier that ends the CTA's reads, and
// sets *flag to whether it is the last of `total`, which also resets the
// counter.  The CTA goes on meanwhile and reads the flag after a later barrier.
// No fence: what is ordered are reads before another CTA's writes, and the
// reads are over when their values have gone through the barrier (fences
// here cost 1 us of latency, and a unit's worth of time under load).
__device__ __forceinline__ void arrive(uint32_t *counter, uint32_t total, int *flag) {
  if (threadIdx.x == 0) {
    const uint32_t n = atomicAdd(counter, 1u);
    if (n + 1 == total) *counter = 0;
    *flag = n + 1 == total;
  }
}

// One channel of the convolution at the new token: the input, the cached
// ones (oldest first), the taps.
template <typename T>
struct Channel {
  T x, c0, c1, c2;
  float4 w;
  float bias;

  __device__ __forceinline__ void load(const T *px, const T *cache, size_t stride, const float *pw,
                                       const float *pb) {
    x = *px;
    if (cache) {
      c0 = cache[0];
      c1 = cache[stride];
      c2 = cache[2 * stride];
      w = *reinterpret_cast<const float4 *>(pw);
      bias = pb ? *pb : 0.f;
    }
  }
  __device__ __forceinline__ float value() const {
    return silu(w.w * to_f32(x) + w.z * to_f32(c2) + w.y * to_f32(c1) + w.x * to_f32(c0) + bias);
  }
  __device__ __forceinline__ void shift(T *cache, size_t stride) const {
    cache[0] = c1;
    cache[stride] = c2;
    cache[2 * stride] = x;
  }
};
// Sums of `v` over the threads of a warp that own the same columns.
template <int TC>
__device__ __forceinline__ void sum_rows(float4 &v) {
#pragma unroll
  for (int off = TC / 4; off < 32; off <<= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, off);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, off);
  }
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

struct SsmStepParams {
  Walk walk;
  int H, P, N, G, n_slots, channels;
  float inv_hpg;          // G / H
  const void *xbc, *z, *dt;
  long long xbc_stride, z_stride, dt_stride;
  const float *w, *bias, *A, *D, *dt_bias;
  void *conv;
  float *state;
  const int32_t *slots;
  void *y;
  uint32_t *counters;
};

// IT = accesses per thread: N * TC / 1024.
template <typename T, int N, int TC>
__global__ void __launch_bounds__(kThreads, 3) ssm_step_kernel(const SsmStepParams p) {
  constexpr int IT = N * TC / kWave, RG = kWave / TC, CH = 2 * N + TC;
  constexpr int NC = (CH + kThreads - 1) / kThreads;      // channels per thread
  extern __shared__ __align__(16) float4 stage[];         // [2][IT][kThreads]
  __shared__ float sB[2][N], sC[2][N], sx[2][TC];
  __shared__ __align__(16) float red[kThreads / 32][TC];   // written as float4
  __shared__ int flag;
  const int tid = threadIdx.x, col = (tid * 4) % TC, row = tid * 4 / TC;

  const int c0 = (blockIdx.x & (p.walk.tiles - 1)) * TC;
  struct Unit {
    Place at;
    int slot, g;
    Channel<T> ch[NC];
    float dt, A, z;
  };
  // number of the unit's channel i: of B, of C, of the tile's columns of x
  auto channel = [&](const Unit &n, int i) {
    return i < 2 * N ? p.H * p.P + n.g * N + (i < N ? i : p.G * N + i - N)
                     : n.at.h * p.P + c0 + i - 2 * N;
  };
  auto state_of = [&](const Unit &n) {
    return p.state + (((size_t)n.slot * p.H + n.at.h) * N + row) * p.P + c0 + col;
  };
  auto conv_of = [&](const Unit &n) {
    return static_cast<T *>(p.conv) + (size_t)n.slot * (kTap - 1) * p.channels;
  };
  auto slot_of = [&](const Place &w) {
    int s = -1;
    if (w.b < p.walk.B) s = p.slots ? p.slots[w.b] : w.b;
    return s < p.n_slots ? s : -1;
  };
  auto load = [&](Unit &n, const Place &at, int slot, int st) {
    n.at = at;
    n.slot = slot;
    if (slot >= 0) {
      n.g = (int)((at.h + 0.5f) * p.inv_hpg);
      const float *s = state_of(n);
#pragma unroll
      for (int i = 0; i < IT; ++i)
        cp_async16(stage + (st * IT + i) * kThreads + tid, s + (size_t)i * RG * p.P);
      const T *x = static_cast<const T *>(p.xbc) + (size_t)at.b * p.xbc_stride;
      const T *conv = conv_of(n);
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int i = tid + k * kThreads;
        if (i < CH) {
          const int c = channel(n, i);
          n.ch[k].load(x + c, conv + c, p.channels, p.w + 4 * (size_t)c,
                       p.bias ? p.bias + c : nullptr);
        }
      }
      n.dt = to_f32(static_cast<const T *>(p.dt)[(size_t)at.b * p.dt_stride + at.h]) +
             (p.dt_bias ? p.dt_bias[at.h] : 0.f);
      n.A = p.A[at.h];
      if (p.z && tid < TC)
        n.z = to_f32(static_cast<const T *>(
            p.z)[(size_t)at.b * p.z_stride + at.h * p.P + c0 + tid]);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto work = [&](const Unit &now, int st) {
    T *y = static_cast<T *>(p.y) + ((size_t)now.at.b * p.H + now.at.h) * p.P + c0;
    if (now.slot < 0) {           // idle (uniform)
      // the next unit writes the sx that the one before this still reads
      __syncthreads();
      if (tid < TC) y[tid] = from_f32<T>(0.f);
      return;
    }
    T *conv = conv_of(now);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int i = tid + k * kThreads;
      if (i < CH) {
        const float v = now.ch[k].value();
        (i < N ? sB[st][i] : i < 2 * N ? sC[st][i - N] : sx[st][i - 2 * N]) = v;
        if (i >= 2 * N) now.ch[k].shift(conv + channel(now, i), p.channels);  // its own channels
      }
    }
    const float d = fmaxf(now.dt, 0.f) + log1pf(expf(-fabsf(now.dt)));
    const float a = expf(d * now.A);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    arrive(p.counters + (size_t)now.at.b * p.G + now.g, (uint32_t)(p.H / p.G * p.walk.tiles),
           &flag);

    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float x0 = d * sx[st][col], x1 = d * sx[st][col + 1], x2 = d * sx[st][col + 2],
                x3 = d * sx[st][col + 3];
    float *s = state_of(now);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      float4 v = stage[(st * IT + i) * kThreads + tid];
      const float bn = sB[st][row + i * RG], cn = sC[st][row + i * RG];
      v.x = a * v.x + bn * x0;
      v.y = a * v.y + bn * x1;
      v.z = a * v.z + bn * x2;
      v.w = a * v.w + bn * x3;
      *reinterpret_cast<float4 *>(s + (size_t)i * RG * p.P) = v;
      acc.x += cn * v.x;
      acc.y += cn * v.y;
      acc.z += cn * v.z;
      acc.w += cn * v.w;
    }
    sum_rows<TC>(acc);
    if ((tid & 31) < TC / 4) *reinterpret_cast<float4 *>(&red[tid >> 5][col]) = acc;
    __syncthreads();
    if (flag) {   // the last of the group: its B and C channels
#pragma unroll
      for (int k = 0; k < NC; ++k)
        if (tid + k * kThreads < 2 * N)
          now.ch[k].shift(conv + channel(now, tid + k * kThreads), p.channels);
    }
    if (tid < TC) {
      float o = 0.f;
#pragma unroll
      for (int r = 0; r < kThreads / 32; ++r) o += red[r][tid];
      if (p.D) o += p.D[now.at.h] * sx[st][tid];
      if (p.z) o *= silu(now.z);
      y[tid] = from_f32<T>(o);
    }
  };

  // the slot is read two units ahead, the rest one
  Unit u0, u1;
  Place at = {(int)(blockIdx.x >> p.walk.log_tiles) / p.H,
              (int)(blockIdx.x >> p.walk.log_tiles) % p.H};
  load(u0, at, slot_of(at), 0);
  at.advance(p.walk);
  int slot = slot_of(at);
  auto next = [&](Unit &n, int st) {
    const Place here = at;
    const int s = slot;
    at.advance(p.walk);
    slot = slot_of(at);
    load(n, here, s, st);
  };
  while (true) {
    next(u1, 1);
    work(u0, 0);
    if (u1.at.b >= p.walk.B) break;
    next(u0, 0);
    work(u1, 1);
    if (u0.at.b >= p.walk.B) break;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

struct KdaStepParams {
  Walk walk;
  int H, K, V, n_slots, l2norm;
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const float *g, *beta, *w;
  float scale;
  void *conv;
  float *state;
  const int32_t *slots;
  void *o;
  uint32_t *counters;
};

template <typename T, int K, int TC>
__global__ void __launch_bounds__(kThreads, 3) kda_step_kernel(const KdaStepParams p) {
  constexpr int IT = K * TC / kWave, RG = kWave / TC, CH = 2 * K + TC;
  constexpr int NC = (CH + kThreads - 1) / kThreads;
  extern __shared__ __align__(16) float4 stage[];         // [2][IT][kThreads]
  __shared__ float sq[2][K], sk[2][K], sg[2][K], dots[3];
  __shared__ __align__(16) float sv[2][TC];                // read as float4
  __shared__ float4 sums[2][kThreads / 32][TC / 4];
  __shared__ int flag[2];
  const int tid = threadIdx.x, col = (tid * 4) % TC, row = tid * 4 / TC;
  const int channels = p.H * (2 * K + p.V);

  const int c0 = (blockIdx.x & (p.walk.tiles - 1)) * TC;
  struct Unit {
    Place at;
    int slot;
    Channel<T> ch[NC];
    float g, beta;
  };
  // input and number of channel i of the unit: of q, of k, of the tile's
  // columns of v
  auto input = [&](const Unit &n, int i) {
    return i < K ? static_cast<const T *>(p.q) + (size_t)n.at.b * p.q_stride + n.at.h * K + i
           : i < 2 * K
               ? static_cast<const T *>(p.k) + (size_t)n.at.b * p.k_stride + n.at.h * K + i - K
               : static_cast<const T *>(p.v) + (size_t)n.at.b * p.v_stride + n.at.h * p.V + c0 +
                     i - 2 * K;
  };
  auto channel = [&](const Unit &n, int i) {
    return i < K ? n.at.h * K + i
           : i < 2 * K ? p.H * K + n.at.h * K + i - K
                       : 2 * p.H * K + n.at.h * p.V + c0 + i - 2 * K;
  };
  auto state_of = [&](const Unit &n) {
    return p.state + (((size_t)n.slot * p.H + n.at.h) * K + row) * p.V + c0 + col;
  };
  auto conv_of = [&](const Unit &n) {
    return p.conv ? static_cast<T *>(p.conv) + (size_t)n.slot * (kTap - 1) * channels : nullptr;
  };
  auto slot_of = [&](const Place &w) {
    int s = -1;
    if (w.b < p.walk.B) s = p.slots ? p.slots[w.b] : w.b;
    return s < p.n_slots ? s : -1;
  };
  auto load = [&](Unit &n, const Place &at, int slot, int st) {
    n.at = at;
    n.slot = slot;
    if (slot >= 0) {
      const float *s = state_of(n);
#pragma unroll
      for (int i = 0; i < IT; ++i)
        cp_async16(stage + (st * IT + i) * kThreads + tid, s + (size_t)i * RG * p.V);
      const T *conv = conv_of(n);
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int i = tid + k * kThreads;
        if (i < CH) {
          const int c = channel(n, i);
          n.ch[k].load(input(n, i), conv ? conv + c : nullptr, channels, p.w + 4 * (size_t)c,
                       nullptr);
        }
      }
      const size_t bh = (size_t)at.b * p.H + at.h;
      if (tid < K) n.g = p.g[bh * K + tid];
      n.beta = p.beta[bh];
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto work = [&](const Unit &now, int st) {
    T *o = static_cast<T *>(p.o) + ((size_t)now.at.b * p.H + now.at.h) * p.V + c0;
    if (now.slot < 0) {           // idle (uniform)
      // the next unit writes the arrays that the one before this still reads
      __syncthreads();
      if (tid < TC) o[tid] = from_f32<T>(0.f);
      return;
    }
    T *conv = conv_of(now);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int i = tid + k * kThreads;
      if (i < CH) {
        const float v = conv ? now.ch[k].value() : to_f32(now.ch[k].x);
        (i < K ? sq[st][i] : i < 2 * K ? sk[st][i - K] : sv[st][i - 2 * K]) = v;
        if (conv && i >= 2 * K) now.ch[k].shift(conv + channel(now, i), channels);
      }
    }
    if (tid < K) sg[st][tid] = expf(now.g);
    if (tid == 0) flag[st] = 0;
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();

    if (conv)
      arrive(p.counters + (size_t)now.at.b * p.H + now.at.h, (uint32_t)p.walk.tiles, &flag[st]);

    // sums of the decayed state against k and q, not yet normalised
    float4 ak = make_float4(0.f, 0.f, 0.f, 0.f), aq = ak;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = row + i * RG;
      const float e = sg[st][r], kn = sk[st][r], qn = sq[st][r];
      const float4 v = stage[(st * IT + i) * kThreads + tid];
      const float ek = e * kn, eq = e * qn;
      ak.x += ek * v.x; ak.y += ek * v.y; ak.z += ek * v.z; ak.w += ek * v.w;
      aq.x += eq * v.x; aq.y += eq * v.y; aq.z += eq * v.z; aq.w += eq * v.w;
    }
    sum_rows<TC>(ak);
    sum_rows<TC>(aq);
    if ((tid & 31) < TC / 4) {
      sums[0][tid >> 5][col / 4] = ak;
      sums[1][tid >> 5][col / 4] = aq;
    }
    if (tid >= kThreads - 32) {   // |q|^2, |k|^2, q . k
      float n[3] = {0.f, 0.f, 0.f};
      for (int i = tid & 31; i < K; i += 32) {
        n[0] += sq[st][i] * sq[st][i];
        n[1] += sk[st][i] * sk[st][i];
        n[2] += sq[st][i] * sk[st][i];
      }
#pragma unroll
      for (int off = 16; off; off >>= 1)
#pragma unroll
        for (int j = 0; j < 3; ++j) n[j] += __shfl_xor_sync(0xffffffffu, n[j], off);
      if ((tid & 31) < 3) dots[tid & 31] = (tid & 31) == 0 ? n[0] : (tid & 31) == 1 ? n[1] : n[2];
    }
    __syncthreads();
    const float nq = p.l2norm ? rsqrtf(dots[0] + 1e-6f) : 1.f;
    const float nk = p.l2norm ? rsqrtf(dots[1] + 1e-6f) : 1.f;
    // every thread adds the sums of its own columns: no barrier after this
    ak = aq = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kThreads / 32; ++r) {
      const float4 a = sums[0][r][col / 4], q = sums[1][r][col / 4];
      ak.x += a.x; ak.y += a.y; ak.z += a.z; ak.w += a.w;
      aq.x += q.x; aq.y += q.y; aq.z += q.z; aq.w += q.w;
    }
    const float4 v4 = *reinterpret_cast<const float4 *>(&sv[st][col]);
    // nk times beta times the residual
    const float bk = now.beta * nk, qk = p.scale * nq * dots[2], qs = p.scale * nq;
    const float4 r4 = make_float4(bk * (v4.x - nk * ak.x), bk * (v4.y - nk * ak.y),
                                  bk * (v4.z - nk * ak.z), bk * (v4.w - nk * ak.w));
    if (row == 0) {
      o[col] = from_f32<T>(qs * aq.x + qk * r4.x);
      o[col + 1] = from_f32<T>(qs * aq.y + qk * r4.y);
      o[col + 2] = from_f32<T>(qs * aq.z + qk * r4.z);
      o[col + 3] = from_f32<T>(qs * aq.w + qk * r4.w);
    }
    float *s = state_of(now);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const float kn = sk[st][row + i * RG], e = sg[st][row + i * RG];
      float4 v = stage[(st * IT + i) * kThreads + tid];   // (its registers are worth more)
      v.x = e * v.x + kn * r4.x;
      v.y = e * v.y + kn * r4.y;
      v.z = e * v.z + kn * r4.z;
      v.w = e * v.w + kn * r4.w;
      *reinterpret_cast<float4 *>(s + (size_t)i * RG * p.V) = v;
    }
    if (flag[st]) {   // the last tile of the head: its q and k channels
#pragma unroll
      for (int k = 0; k < NC; ++k)
        if (tid + k * kThreads < 2 * K)
          now.ch[k].shift(conv + channel(now, tid + k * kThreads), channels);
    }
  };

  // the slot is read two units ahead, the rest one
  Unit u0, u1;
  Place at = {(int)(blockIdx.x >> p.walk.log_tiles) / p.H,
              (int)(blockIdx.x >> p.walk.log_tiles) % p.H};
  load(u0, at, slot_of(at), 0);
  at.advance(p.walk);
  int slot = slot_of(at);
  auto next = [&](Unit &n, int st) {
    const Place here = at;
    const int s = slot;
    at.advance(p.walk);
    slot = slot_of(at);
    load(n, here, s, st);
  };
  while (true) {
    next(u1, 1);
    work(u0, 0);
    if (u1.at.b >= p.walk.B) break;
    next(u0, 0);
    work(u1, 1);
    if (u0.at.b >= p.walk.B) break;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Columns per unit: 32 while that leaves no more than one unit for each SM (one
// sequence of 32 heads of 128: 3.3 and 3.5 us, with 64 columns 3.5 and 3.7), else
// up to 64, a tile of 32 KB at 128 keys (4 sequences: 4.6 and 5.1 us, with 32
// columns 5.7 and 6.4; the sizes above 102 and 129 us with 32).
int tile_for(int B, int H, int cols, int sms) {
  const long long small = (long long)B * H * (cols / 32);
  return small <= sms || cols == 32 ? 32 : 64;
}

// Three CTAs fit an SM (registers, and two staged tiles each).
template <typename K, typename P>
cudaError_t launch(K kern, P &p, int B, int keys, int cols, int tc, int sms, cudaStream_t cs) {
  const int tiles = cols / tc;
  const long long units = (long long)B * p.H * tiles;
  const int most = 3 * sms / tiles * tiles;
  const int grid = (int)(units < most ? units : most), pairs = grid / tiles;
  p.walk = {p.H, B, pairs / p.H, pairs % p.H, tiles, tiles == 1 ? 0 : tiles == 2 ? 1 : 2};
  const size_t smem = (size_t)2 * keys * tc * sizeof(float);
  if (smem > 16 * 1024) {   // with the static arrays, above the default 48 KB
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<(unsigned)grid, kThreads, smem, cs>>>(p);
  return cudaGetLastError();
}

template <typename T, int N>
cudaError_t launch_ssm_step(SsmStepParams p, int B, cudaStream_t cs) {
  const int sms = num_sms(), tc = tile_for(B, p.H, p.P, sms);
  p.inv_hpg = (float)p.G / (float)p.H;
  return tc == 32 ? launch(ssm_step_kernel<T, N, 32>, p, B, N, p.P, 32, sms, cs)
                  : launch(ssm_step_kernel<T, N, 64>, p, B, N, p.P, 64, sms, cs);
}

template <typename T, int K>
cudaError_t launch_kda_step(KdaStepParams p, int B, cudaStream_t cs) {
  const int sms = num_sms(), tc = tile_for(B, p.H, p.V, sms);
  return tc == 32 ? launch(kda_step_kernel<T, K, 32>, p, B, K, p.V, 32, sms, cs)
                  : launch(kda_step_kernel<T, K, 64>, p, B, K, p.V, 64, sms, cs);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

}  // namespace

kda_status check_ssm_shape(const kda_ssm_shape *s) {
  if (!s || s->B < 1 || s->T < 1 || s->H < 1 || s->G < 1) return KDA_ERR_INVALID_ARG;
  if (s->dtype != KDA_DTYPE_F32 && s->dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
  if (s->H % s->G) return KDA_ERR_INVALID_ARG;
  if (!dim_ok(s->P) || !dim_ok(s->N)) return KDA_ERR_UNSUPPORTED;
  const long long ch = (long long)s->H * s->P + 2ll * s->G * s->N;
  if (ch >= (1ll << 24) || (long long)s->B * s->T * s->H * 4 >= (1ll << 31))
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_step_workspace_size(int B, int H) {
  if (B < 1 || H < 1 || (long long)B * H >= (1ll << 29)) return 0;
  return align_up(sizeof(WsHeader) + sizeof(uint32_t) * (size_t)B * H, 256);
}

kda_status kda_ssm_step(const kda_ssm_shape *s, const void *xbc, const void *dt, const void *z,
                        const float *w, const float *bias, const float *A, const float *D,
                        const float *dt_bias, const int32_t *slots, int n_slots, void *conv_state,
                        float *state, void *y, void *workspace, size_t workspace_bytes,
                        kda_stream_t stream) {
  const kda_status st = check_ssm_shape(s);
  if (st != KDA_OK) return st;
  if (!xbc || !dt || !w || !A || !conv_state || !state || !y || n_slots < 1)
    return KDA_ERR_INVALID_ARG;
  if (s->T != 1 || (!slots && n_slots < s->B)) return KDA_ERR_INVALID_ARG;
  for (const void *ptr : {(const void *)w, (const void *)state})
    if (!aligned(ptr, 16)) return KDA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kda_step_workspace_size(s->B, s->H)) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KDA_ERR_ALIGNMENT;
  SsmStepParams p = {};
  p.H = s->H; p.P = s->P; p.N = s->N; p.G = s->G; p.n_slots = n_slots;
  p.channels = s->H * s->P + 2 * s->G * s->N;
  p.xbc = xbc; p.z = z; p.dt = dt;
  p.xbc_stride = s->xbc_stride_b; p.z_stride = s->z_stride_b; p.dt_stride = s->dt_stride_b;
  p.w = w; p.bias = bias; p.A = A; p.D = D; p.dt_bias = dt_bias;
  p.conv = conv_state; p.state = state; p.slots = slots; p.y = y;
  p.counters = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + sizeof(WsHeader));
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  using B16 = __nv_bfloat16;
  cudaError_t e;
  if (s->dtype == KDA_DTYPE_BF16)
    e = s->N == 32   ? launch_ssm_step<B16, 32>(p, s->B, cs)
        : s->N == 64 ? launch_ssm_step<B16, 64>(p, s->B, cs)
                     : launch_ssm_step<B16, 128>(p, s->B, cs);
  else
    e = s->N == 32   ? launch_ssm_step<float, 32>(p, s->B, cs)
        : s->N == 64 ? launch_ssm_step<float, 64>(p, s->B, cs)
                     : launch_ssm_step<float, 128>(p, s->B, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_step(const kda_shape *s, const void *q, const void *k, const void *v,
                    long long q_stride, long long k_stride, long long v_stride, const float *g,
                    const float *beta, float scale, const float *conv_w, void *conv_state,
                    int l2norm_qk, const int32_t *slots, int n_slots, float *state, void *o,
                    void *workspace, size_t workspace_bytes, kda_stream_t stream) {
  const kda_status st = check_shape(s);
  if (st != KDA_OK) return st;
  if (!q || !k || !v || !g || !beta || !state || !o || n_slots < 1) return KDA_ERR_INVALID_ARG;
  if (s->T != 1 || (!slots && n_slots < s->B)) return KDA_ERR_INVALID_ARG;
  if ((conv_w != nullptr) != (conv_state != nullptr)) return KDA_ERR_INVALID_ARG;
  if (!(scale == scale)) return KDA_ERR_INVALID_ARG;
  for (const void *ptr : {(const void *)conv_w, (const void *)state})
    if (!aligned(ptr, 16)) return KDA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kda_step_workspace_size(s->B, s->H)) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KDA_ERR_ALIGNMENT;
  KdaStepParams p = {};
  p.H = s->H; p.K = s->K; p.V = s->V; p.n_slots = n_slots; p.l2norm = l2norm_qk;
  p.q = q; p.k = k; p.v = v;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.g = g; p.beta = beta; p.scale = scale; p.w = conv_w; p.conv = conv_state; p.state = state;
  p.slots = slots; p.o = o;
  p.counters = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + sizeof(WsHeader));
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  using B16 = __nv_bfloat16;
  cudaError_t e;
  if (s->qkv_dtype == KDA_DTYPE_BF16)
    e = s->K == 32   ? launch_kda_step<B16, 32>(p, s->B, cs)
        : s->K == 64 ? launch_kda_step<B16, 64>(p, s->B, cs)
                     : launch_kda_step<B16, 128>(p, s->B, cs);
  else
    e = s->K == 32   ? launch_kda_step<float, 32>(p, s->B, cs)
        : s->K == 64 ? launch_kda_step<float, 64>(p, s->B, cs)
                     : launch_kda_step<float, 128>(p, s->B, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
