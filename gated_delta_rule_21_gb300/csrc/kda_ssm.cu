// kda_ssm.cu -- the selective state space operator on prompts: short causal
// convolution, SiLU, scan, skip and gate.  Entry points, the row table, and
// the fp32 CUDA-core kernel that serves every shape and type.
//
//     u = SiLU(conv(xbc) + bias) = (x | B | C);   d = softplus(dt + dt_bias)
//     S = e^{d A} S + d B (outer) x               S: [N][P] per head, fp32
//     y = (C^T S + D x) SiLU(z)
#include <string.h>

#include "kda_ssm.cuh"

namespace kda {
namespace {

__device__ __forceinline__ int block_min(int v, int *red) {
  v = __reduce_min_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < (int)blockDim.x / 32; ++i) v = min(v, red[i]);
  return v;
}

// One CTA per row: its first run and its last token.
__global__ void __launch_bounds__(1024) ssm_rows_kernel(const SsmParams p) {
  __shared__ int red[32];
  const int b = blockIdx.x;
  const int32_t *ids = p.segment_ids + (size_t)b * p.T;
  SsmRow row = {0, p.T, p.T - 1, 0};
  int f = p.T, l = p.T;   // l: T - 1 - last
#pragma unroll 8
  for (int t = threadIdx.x; t < p.T; t += 1024)
    if (ids[t] != 0) {
      f = min(f, t);
      l = min(l, p.T - 1 - t);
    }
  row.first = block_min(f, red);
  row.last = p.T - 1 - block_min(l, red);
  int e = p.T;
  if (row.first < p.T) {
    const int id = ids[row.first];
#pragma unroll 8
    for (int t = threadIdx.x; t < p.T; t += 1024)
      if (t > row.first && ids[t] != id) e = min(e, t);
  }
  row.first_end = block_min(e, red);
  if (threadIdx.x == 0) p.rows[b] = row;
}

__device__ __forceinline__ SsmRow simt_row(const SsmParams &p, int b) {
  if (p.segment_ids) return p.rows[b];
  SsmRow r = {0, p.T, p.T - 1, 0};
  return r;
}

constexpr int kThreads = 256, kCols = 32, kTok = 32, kWarps = kThreads / 32;

// One CTA per (row, head, 32 columns), token by token in fp32.  Warp w holds
// states [w N / 8, (w + 1) N / 8) of column `lane` in registers; 32 tokens of
// B, C and d x are made in shared memory at a time, and the warps' shares of
// y are added there.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) ssm_simt_kernel(const SsmParams p) {
  constexpr int NS = N / kWarps;
  extern __shared__ __align__(16) float sm[];
  float *sB = sm, *sC = sB + kTok * N, *sX = sC + kTok * N, *sY = sX + kTok * kCols;
  __shared__ float sa[kTok], sd[kTok];
  __shared__ int sreset[kTok], slive[kTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = p.P / kCols, tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int h = bh % p.H, b = bh / p.H, c0 = tile * kCols, g = h / (p.H / p.G);
  const int32_t *ids = p.segment_ids ? p.segment_ids + (size_t)b * p.T : nullptr;
  const SsmRow row = simt_row(p, b);
  const T *x = static_cast<const T *>(p.xbc) + (size_t)b * p.xbc_sb;
  const T *past = p.conv_state
                      ? static_cast<const T *>(p.conv_state) +
                            (size_t)b * (kSsmTaps - 1) * p.channels
                      : nullptr;
  const int cx = h * p.P + c0, cb = p.H * p.P + g * N, cc = cb + p.G * N;
  const float A = p.A[h], D = p.D ? p.D[h] : 0.f, db = p.dt_bias ? p.dt_bias[h] : 0.f;
  float s[NS];
  const size_t state = (((size_t)b * p.H + h) * N + warp * NS) * p.P + c0 + lane;
#pragma unroll
  for (int j = 0; j < NS; ++j)
    s[j] = p.initial_state ? p.initial_state[state + (size_t)j * p.P] : 0.f;
  for (int t0 = 0; t0 < p.T; t0 += kTok) {
    const int n = min(kTok, p.T - t0);
    __syncthreads();
    if (tid < n) {
      const SsmToken k = ssm_token(ids, t0 + tid, p.T, row);
      const T *dt = static_cast<const T *>(p.dt) + (size_t)b * p.dt_sb +
                    (long long)(t0 + tid) * p.dt_st;
      const float d = k.live ? ssm_softplus(to_f32(dt[h]) + db) : 0.f;
      sd[tid] = d;
      sa[tid] = expf(d * A);
      sreset[tid] = k.reset;
      slive[tid] = k.live;
    }
    __syncthreads();
    for (int i = tid; i < n * (2 * N + kCols); i += kThreads) {
      const int t = i / (2 * N + kCols), j = i - t * (2 * N + kCols);
      const int c = j < N ? cb + j : j < 2 * N ? cc + j - N : cx + j - 2 * N;
      float u = 0.f;
      if (slive[t]) {
        const SsmToken k = ssm_token(ids, t0 + t, p.T, row);
        u = p.bias ? p.bias[c] : 0.f;
#pragma unroll
        for (int age = 0; age < kSsmTaps; ++age)
          u += p.w[4 * c + 3 - age] *
               ssm_tap(x, p.xbc_st, past, p.channels, c, t0 + t, age, k);
        u = u / (1.f + expf(-u));
      }
      if (j < N) sB[t * N + j] = u * sd[t];
      else if (j < 2 * N) sC[t * N + j - N] = u;
      else sX[t * kCols + j - 2 * N] = u;
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      float a = sa[t], acc = 0.f;
      if (sreset[t]) a = 0.f;
      const float xv = sX[t * kCols + lane];
      const float *pb = sB + t * N + warp * NS, *pc = sC + t * N + warp * NS;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        // a reset drops the state whatever it holds
        s[j] = (sreset[t] ? 0.f : a * s[j]) + pb[j] * xv;
        acc += pc[j] * s[j];
      }
      sY[(warp * kTok + t) * kCols + lane] = acc;
    }
    __syncthreads();
    for (int i = tid; i < n * kCols; i += kThreads) {
      const int t = i / kCols, c = i % kCols;
      float v = 0.f;
      if (slive[t]) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sY[(w * kTok + t) * kCols + c];
        v += D * sX[t * kCols + c];
        if (p.z) {
          const float zv = to_f32(static_cast<const T *>(
              p.z)[(size_t)b * p.z_sb + (long long)(t0 + t) * p.z_st + cx + c]);
          v *= zv / (1.f + expf(-zv));
        }
      }
      static_cast<T *>(p.y)[(((size_t)b * p.T + t0 + t) * p.H + h) * p.P + c0 + c] =
          from_f32<T>(v);
    }
  }
  if (p.conv_out) {      // head h moves its share of the channels
    const SsmToken k = ssm_token(ids, row.last, p.T, row);
    T *out = static_cast<T *>(p.conv_out) + (size_t)b * (kSsmTaps - 1) * p.channels;
    const int ctas = p.H * tiles, me = h * tiles + tile;
    for (int c = me * kThreads + tid; c < p.channels; c += ctas * kThreads)
#pragma unroll
      for (int i = 0; i < kSsmTaps - 1; ++i)
        out[(size_t)i * p.channels + c] =
            ssm_cached(x, p.xbc_st, past, p.channels, c, i, row.last, k);
  }
  if (p.final_state) {
#pragma unroll
    for (int j = 0; j < NS; ++j) p.final_state[state + (size_t)j * p.P] = s[j];
  }
}

template <typename T, int N>
cudaError_t launch_simt(const SsmParams &p, cudaStream_t cs) {
  const size_t smem = sizeof(float) * (2 * kTok * N + kTok * kCols * (1 + kWarps));
  const cudaError_t e = cudaFuncSetAttribute(
      ssm_simt_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  ssm_simt_kernel<T, N><<<(unsigned)(p.B * p.H * (p.P / kCols)), kThreads, smem, cs>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt_t(const SsmParams &p, cudaStream_t cs) {
  return p.N == 32 ? launch_simt<T, 32>(p, cs) : p.N == 64 ? launch_simt<T, 64>(p, cs)
                                                           : launch_simt<T, 128>(p, cs);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t rows_bytes(int B) { return align_up(sizeof(WsHeader) + sizeof(SsmRow) * (size_t)B, 256); }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_ssm_fwd_workspace_size(const kda_ssm_shape *s, kda_impl impl) {
  if (check_ssm_shape(s) != KDA_OK) return 0;
  const bool bf16 = s->dtype == KDA_DTYPE_BF16;
  if (impl == KDA_IMPL_SIMT || (impl == KDA_IMPL_AUTO && !bf16)) return rows_bytes(s->B);
  if ((impl != KDA_IMPL_AUTO && impl != KDA_IMPL_TC) || !bf16) return 0;
  SsmParams p = {};
  p.B = s->B; p.T = s->T; p.H = s->H; p.P = s->P; p.N = s->N; p.G = s->G;
  return rows_bytes(s->B) + ssm_tc_bytes(p);
}

kda_status kda_ssm_fwd(const kda_ssm_shape *s, const void *xbc, const void *dt, const void *z,
                       const float *w, const float *bias, const float *A, const float *D,
                       const float *dt_bias, const float *initial_state, const void *conv_state,
                       const int32_t *segment_ids, void *y, float *final_state, void *conv_out,
                       void *workspace, size_t workspace_bytes, kda_impl impl,
                       kda_stream_t stream) {
  const kda_status st = check_ssm_shape(s);
  if (st != KDA_OK) return st;
  if (!xbc || !dt || !w || !A || !y) return KDA_ERR_INVALID_ARG;
  if (impl != KDA_IMPL_AUTO && impl != KDA_IMPL_SIMT && impl != KDA_IMPL_TC &&
      impl != KDA_IMPL_SPLIT)
    return KDA_ERR_INVALID_ARG;
  const size_t need = kda_ssm_fwd_workspace_size(s, impl);
  if (need == 0) return KDA_ERR_UNSUPPORTED;
  for (const void *ptr : {xbc, z, (const void *)w, (const void *)initial_state, conv_state,
                          (const void *)y, (const void *)final_state, (const void *)conv_out})
    if (!aligned(ptr, 16)) return KDA_ERR_ALIGNMENT;
  const int per16 = s->dtype == KDA_DTYPE_BF16 ? 8 : 4;
  for (long long stride : {s->xbc_stride_b, s->xbc_stride_t, z ? s->z_stride_b : 0,
                           z ? s->z_stride_t : 0})
    if (stride % per16) return KDA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KDA_ERR_ALIGNMENT;
  SsmParams p;
  memset(&p, 0, sizeof(p));
  p.B = s->B; p.T = s->T; p.H = s->H; p.P = s->P; p.N = s->N; p.G = s->G;
  p.channels = s->H * s->P + 2 * s->G * s->N;
  p.xbc = xbc; p.z = z; p.dt = dt;
  p.xbc_sb = s->xbc_stride_b; p.xbc_st = s->xbc_stride_t;
  p.z_sb = s->z_stride_b; p.z_st = s->z_stride_t;
  p.dt_sb = s->dt_stride_b; p.dt_st = s->dt_stride_t;
  p.w = w; p.bias = bias; p.A = A; p.D = D; p.dt_bias = dt_bias;
  p.initial_state = initial_state; p.conv_state = conv_state; p.segment_ids = segment_ids;
  p.y = y; p.final_state = final_state; p.conv_out = conv_out;
  p.rows = reinterpret_cast<SsmRow *>(static_cast<char *>(workspace) + sizeof(WsHeader));
  p.ws = static_cast<unsigned char *>(workspace) + rows_bytes(s->B);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = s->dtype == KDA_DTYPE_BF16;
  cudaError_t e = cudaSuccess;
  if (segment_ids) {
    ssm_rows_kernel<<<s->B, 1024, 0, cs>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return KDA_ERR_CUDA;
  }
  if (bf16 && impl != KDA_IMPL_SIMT)
    e = launch_ssm_tc(p, &reinterpret_cast<WsHeader *>(workspace)->status, cs);
  else
    e = bf16 ? launch_simt_t<__nv_bfloat16>(p, cs) : launch_simt_t<float>(p, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
