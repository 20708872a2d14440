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
// A CTA of 256 threads owns a tile of TC columns of one (sequence, head).  A
// thread owns 4 adjacent columns of every (1024 / TC)-th key row, so a warp's
// 16-byte accesses cover whole row segments, and all of a thread's loads
// are issued before anything else.
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

__device__ __forceinline__ float silu(float x) { return x / (1.f + expf(-x)); }

// Thread 0 counts its CTA in, after a barrier that ends the CTA's reads, and
// sets *flag to whether it is the last of `total`, which also resets the
// counter.  The CTA goes on meanwhile and reads the flag after a later barrier.
__device__ __forceinline__ void arrive(uint32_t *counter, uint32_t total, int *flag) {
  if (threadIdx.x == 0) {
    __threadfence();
    const uint32_t n = atomicAdd(counter, 1u);
    if (n + 1 == total) *counter = 0;
    *flag = n + 1 == total;
    __threadfence();
  }
}

// One channel of the convolution at the new token: c[3] are the cached
// inputs, oldest first.
template <typename T>
__device__ __forceinline__ float conv_token(const T *cache, size_t stride, const float4 w, float b,
                                            float x) {
  const float a0 = to_f32(cache[0]), a1 = to_f32(cache[stride]), a2 = to_f32(cache[2 * stride]);
  return silu(w.w * x + w.z * a2 + w.y * a1 + w.x * a0 + b);
}
template <typename T>
__device__ __forceinline__ void shift_channel(T *cache, size_t stride, T x) {
  cache[0] = cache[stride];
  cache[stride] = cache[2 * stride];
  cache[2 * stride] = x;
}

struct SsmStepParams {
  int H, P, N, G, tiles, n_slots, channels;
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
__global__ void __launch_bounds__(kThreads, 4) ssm_step_kernel(const SsmStepParams p) {
  constexpr int IT = N * TC / kWave, RG = kWave / TC;
  __shared__ float sB[N], sC[N], sx[TC], red[RG][TC];
  __shared__ int flag;
  const int tid = threadIdx.x;
  const int tile = blockIdx.x % p.tiles, bh = blockIdx.x / p.tiles;
  const int h = bh % p.H, b = bh / p.H, c0 = tile * TC;
  const int slot = p.slots ? p.slots[b] : b;
  T *y = static_cast<T *>(p.y) + ((size_t)b * p.H + h) * p.P + c0;
  if (slot < 0 || slot >= p.n_slots) {
    if (tid < TC) y[tid] = from_f32<T>(0.f);
    return;
  }
  const int col = (tid * 4) % TC, row = tid * 4 / TC;
  float *s = p.state + (((size_t)slot * p.H + h) * N + row) * p.P + c0 + col;
  float4 v[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i)
    v[i] = *reinterpret_cast<const float4 *>(s + (size_t)i * RG * p.P);

  const int g = h / (p.H / p.G);
  const T *x = static_cast<const T *>(p.xbc) + (size_t)b * p.xbc_stride;
  T *conv = static_cast<T *>(p.conv) + (size_t)slot * (kTap - 1) * p.channels;
  const float dr = to_f32(static_cast<const T *>(p.dt)[(size_t)b * p.dt_stride + h]) +
                   (p.dt_bias ? p.dt_bias[h] : 0.f);
  const int cx = h * p.P + c0, cb = p.H * p.P + g * N, cc = cb + p.G * N;
  for (int i = tid; i < 2 * N + TC; i += kThreads) {
    const int c = i < N ? cb + i : i < 2 * N ? cc + i - N : cx + i - 2 * N;
    const T xn = x[c];
    const float u = conv_token(conv + c, p.channels, *reinterpret_cast<const float4 *>(p.w + 4 * c),
                               p.bias ? p.bias[c] : 0.f, to_f32(xn));
    (i < N ? sB[i] : i < 2 * N ? sC[i - N] : sx[i - 2 * N]) = u;
    if (i >= 2 * N) shift_channel(conv + c, p.channels, xn);   // this CTA's own channels
  }
  const float d = fmaxf(dr, 0.f) + log1pf(expf(-fabsf(dr)));
  const float a = expf(d * p.A[h]);
  uint32_t *counter = p.counters + (size_t)b * p.G + g;
  __syncthreads();
  arrive(counter, (uint32_t)(p.H / p.G * p.tiles), &flag);

  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float x0 = d * sx[col], x1 = d * sx[col + 1], x2 = d * sx[col + 2], x3 = d * sx[col + 3];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const float bn = sB[row + i * RG], cn = sC[row + i * RG];
    v[i].x = a * v[i].x + bn * x0;
    v[i].y = a * v[i].y + bn * x1;
    v[i].z = a * v[i].z + bn * x2;
    v[i].w = a * v[i].w + bn * x3;
    *reinterpret_cast<float4 *>(s + (size_t)i * RG * p.P) = v[i];
    acc.x += cn * v[i].x;
    acc.y += cn * v[i].y;
    acc.z += cn * v[i].z;
    acc.w += cn * v[i].w;
  }
  *reinterpret_cast<float4 *>(&red[row][col]) = acc;
  __syncthreads();
  if (flag) {   // the last of the group: its B and C channels
    for (int i = tid; i < 2 * N; i += kThreads) {
      const int c = i < N ? cb + i : cc + i - N;
      shift_channel(conv + c, p.channels, x[c]);
    }
  }
  if (tid < TC) {
    float o = 0.f;
#pragma unroll
    for (int r = 0; r < RG; ++r) o += red[r][tid];
    if (p.D) o += p.D[h] * sx[tid];
    if (p.z) o *= silu(to_f32(static_cast<const T *>(p.z)[(size_t)b * p.z_stride + cx + tid]));
    y[tid] = from_f32<T>(o);
  }
}

struct KdaStepParams {
  int H, K, V, tiles, n_slots, l2norm;
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
__global__ void __launch_bounds__(kThreads, 4) kda_step_kernel(const KdaStepParams p) {
  constexpr int IT = K * TC / kWave, RG = kWave / TC;
  __shared__ float sq[K], sk[K], sg[K], sv[TC], rk[RG][TC], rq[RG][TC], srk[TC], dots[3];
  __shared__ int flag;
  const int tid = threadIdx.x;
  const int tile = blockIdx.x % p.tiles, bh = blockIdx.x / p.tiles;
  const int h = bh % p.H, b = bh / p.H, c0 = tile * TC;
  const int slot = p.slots ? p.slots[b] : b;
  T *o = static_cast<T *>(p.o) + ((size_t)b * p.H + h) * p.V + c0;
  if (slot < 0 || slot >= p.n_slots) {
    if (tid < TC) o[tid] = from_f32<T>(0.f);
    return;
  }
  const int col = (tid * 4) % TC, row = tid * 4 / TC;
  float *s = p.state + (((size_t)slot * p.H + h) * K + row) * p.V + c0 + col;
  float4 v[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i)
    v[i] = *reinterpret_cast<const float4 *>(s + (size_t)i * RG * p.V);

  const T *q = static_cast<const T *>(p.q) + (size_t)b * p.q_stride + h * K;
  const T *k = static_cast<const T *>(p.k) + (size_t)b * p.k_stride + h * K;
  const T *vv = static_cast<const T *>(p.v) + (size_t)b * p.v_stride + h * p.V + c0;
  const int channels = p.H * (2 * K + p.V);
  T *conv = p.conv ? static_cast<T *>(p.conv) + (size_t)slot * (kTap - 1) * channels : nullptr;
  const int cq = h * K, ck = p.H * K + h * K, cv = 2 * p.H * K + h * p.V + c0;
  for (int i = tid; i < 2 * K + TC; i += kThreads) {
    const T xn = i < K ? q[i] : i < 2 * K ? k[i - K] : vv[i - 2 * K];
    float u = to_f32(xn);
    if (conv) {
      const int c = i < K ? cq + i : i < 2 * K ? ck + i - K : cv + i - 2 * K;
      u = conv_token(conv + c, channels, *reinterpret_cast<const float4 *>(p.w + 4 * c), 0.f, u);
      if (i >= 2 * K) shift_channel(conv + c, channels, xn);
    }
    (i < K ? sq[i] : i < 2 * K ? sk[i - K] : sv[i - 2 * K]) = u;
  }
  for (int i = tid; i < K; i += kThreads) sg[i] = expf(p.g[((size_t)b * p.H + h) * K + i]);
  const float beta = p.beta[(size_t)b * p.H + h];
  if (tid == 0) flag = 0;
  __syncthreads();
  if (conv) arrive(p.counters + (size_t)b * p.H + h, (uint32_t)p.tiles, &flag);

  // sums of the decayed state against k and q, not yet normalised
  float4 ak = make_float4(0.f, 0.f, 0.f, 0.f), aq = ak;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = row + i * RG;
    const float e = sg[r], kn = sk[r], qn = sq[r];
    v[i].x *= e; v[i].y *= e; v[i].z *= e; v[i].w *= e;
    ak.x += kn * v[i].x; ak.y += kn * v[i].y; ak.z += kn * v[i].z; ak.w += kn * v[i].w;
    aq.x += qn * v[i].x; aq.y += qn * v[i].y; aq.z += qn * v[i].z; aq.w += qn * v[i].w;
  }
  *reinterpret_cast<float4 *>(&rk[row][col]) = ak;
  *reinterpret_cast<float4 *>(&rq[row][col]) = aq;
  if (tid >= kThreads - 32) {   // |q|^2, |k|^2, q . k
    float n[3] = {0.f, 0.f, 0.f};
    for (int i = tid & 31; i < K; i += 32) {
      n[0] += sq[i] * sq[i];
      n[1] += sk[i] * sk[i];
      n[2] += sq[i] * sk[i];
    }
#pragma unroll
    for (int off = 16; off; off >>= 1)
#pragma unroll
      for (int j = 0; j < 3; ++j) n[j] += __shfl_xor_sync(0xffffffffu, n[j], off);
    if ((tid & 31) < 3) dots[tid & 31] = (tid & 31) == 0 ? n[0] : (tid & 31) == 1 ? n[1] : n[2];
  }
  __syncthreads();
  if (flag) {
    for (int i = tid; i < 2 * K; i += kThreads)
      shift_channel(conv + (i < K ? cq + i : ck + i - K), channels, i < K ? q[i] : k[i - K]);
  }
  const float nq = p.l2norm ? rsqrtf(dots[0] + 1e-6f) : 1.f;
  const float nk = p.l2norm ? rsqrtf(dots[1] + 1e-6f) : 1.f;
  if (tid < TC) {
    float ks = 0.f, qs = 0.f;
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      ks += rk[r][tid];
      qs += rq[r][tid];
    }
    const float br = beta * (sv[tid] - nk * ks);     // beta times the residual
    srk[tid] = nk * br;
    o[tid] = from_f32<T>(p.scale * nq * (qs + nk * dots[2] * br));
  }
  __syncthreads();
  const float4 r4 = *reinterpret_cast<const float4 *>(&srk[col]);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const float kn = sk[row + i * RG];
    v[i].x += kn * r4.x; v[i].y += kn * r4.y; v[i].z += kn * r4.z; v[i].w += kn * r4.w;
    *reinterpret_cast<float4 *>(s + (size_t)i * RG * p.V) = v[i];
  }
}

// Columns per CTA: 32 while that leaves no more than two CTAs for each SM,
// else up to 64 (a tile of 32 KB at 128 keys: four CTAs fit an SM).
int tile_for(int B, int H, int cols) {
  const long long small = (long long)B * H * (cols / 32);
  return small <= 2ll * num_sms() || cols == 32 ? 32 : 64;
}

template <typename T, int N>
cudaError_t launch_ssm_step(SsmStepParams p, int B, cudaStream_t cs) {
  const int tc = tile_for(B, p.H, p.P);
  p.tiles = p.P / tc;
  const unsigned grid = (unsigned)(B * p.H * p.tiles);
  if (tc == 32) ssm_step_kernel<T, N, 32><<<grid, kThreads, 0, cs>>>(p);
  else ssm_step_kernel<T, N, 64><<<grid, kThreads, 0, cs>>>(p);
  return cudaGetLastError();
}

template <typename T, int K>
cudaError_t launch_kda_step(KdaStepParams p, int B, cudaStream_t cs) {
  const int tc = tile_for(B, p.H, p.V);
  p.tiles = p.V / tc;
  const unsigned grid = (unsigned)(B * p.H * p.tiles);
  if (tc == 32) kda_step_kernel<T, K, 32><<<grid, kThreads, 0, cs>>>(p);
  else kda_step_kernel<T, K, 64><<<grid, kThreads, 0, cs>>>(p);
  return cudaGetLastError();
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
