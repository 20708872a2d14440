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
  start_next();
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

// How a row is cut for the CUDA-core kernel: `segs` segments of `len` tokens
// (a multiple of kTok), as many as fill the GPU four times over.  With more
// than one, a first pass runs every segment but the last from a zero state,
// the states that enter the segments are chained, and a second pass makes y:
// twice the work on the states, but a short row of few heads no longer waits
// for one chain of tokens (3 rows of 997 tokens, 6 heads: 576 us in one chain,
// 42 us in segments of 32 tokens).  152 SMs, and not what this device has: the
// workspace's size goes by it, which may be asked for where there is no device.
struct SimtCut {
  int segs, len;
};
SimtCut simt_cut(int B, int T, int H, int P) {
  const long long chains = (long long)B * H * (P / kCols), want = (4 * 152 + chains - 1) / chains;
  const int most = (T + kTok - 1) / kTok;
  const int n = (int)(want < most ? want : most);
  SimtCut c;
  c.len = ((T + n - 1) / n + kTok - 1) / kTok * kTok;
  c.segs = (T + c.len - 1) / c.len;
  return c;
}

// One CTA per (segment, row, head, 32 columns), token by token in fp32.  Warp
// w holds states [w N / 8, (w + 1) N / 8) of column `lane` in registers; 32
// tokens of B, C and x are made in shared memory at a time, and the warps'
// shares of y are added there.  FIRST: the first pass (states and decays only).
template <typename T, int N, bool FIRST>
__global__ void __launch_bounds__(kThreads) ssm_simt_kernel(const SsmParams p, const SimtCut cut,
                                                            float *seg_state, float *seg_decay) {
  constexpr int NS = N / kWarps;
  extern __shared__ __align__(16) float sm[];
  float *sB = sm, *sC = sB + kTok * N, *sX = sC + kTok * N, *sY = sX + kTok * kCols;
  __shared__ float sa[kTok], sd[kTok];
  __shared__ int smark[kTok];            // place | first << 2 | live << 3 | reset << 4
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = p.P / kCols, tile = blockIdx.x % tiles, bh = blockIdx.x / tiles % (p.B * p.H);
  const int seg = blockIdx.x / tiles / (p.B * p.H);
  const int h = bh % p.H, b = bh / p.H, c0 = tile * kCols, g = h / (p.H / p.G);
  const int32_t *ids = p.segment_ids ? p.segment_ids + (size_t)b * p.T : nullptr;
  if (FIRST) start_next();
  const SsmRow row = simt_row(p, b);
  const T *x = static_cast<const T *>(p.xbc) + (size_t)b * p.xbc_sb;
  const T *past = p.conv_state
                      ? static_cast<const T *>(p.conv_state) +
                            (size_t)b * (kSsmTaps - 1) * p.channels
                      : nullptr;
  const int cx = h * p.P + c0, cb = p.H * p.P + g * N, cc = cb + p.G * N;
  const float A = p.A[h], D = p.D ? p.D[h] : 0.f, db = p.dt_bias ? p.dt_bias[h] : 0.f;
  const size_t mine = (size_t)(warp * NS) * p.P + c0 + lane, per = (size_t)N * p.P;
  const float *enter = cut.segs > 1 ? seg_state + ((size_t)seg * p.B * p.H + bh) * per
                       : p.initial_state ? p.initial_state + (size_t)bh * per : nullptr;
  float s[NS], decay = 1.f;
  bool dropped = false;
#pragma unroll
  for (int j = 0; j < NS; ++j) s[j] = 0.f;
  const int end = min(p.T, (seg + 1) * cut.len);
  for (int t0 = seg * cut.len; t0 < end; t0 += kTok) {
    const int n = min(kTok, end - t0);
    __syncthreads();
    if (tid < kTok) {
      SsmToken k = {};
      float d = 0.f;
      if (tid < n) {
        k = ssm_token(ids, t0 + tid, p.T, row);
        const T *dt = static_cast<const T *>(p.dt) + (size_t)b * p.dt_sb +
                      (long long)(t0 + tid) * p.dt_st;
        if (k.live) d = ssm_softplus(to_f32(dt[h]) + db);
      }
      sd[tid] = d;
      sa[tid] = expf(d * A);
      smark[tid] = k.place | (k.first ? 4 : 0) | (k.live ? 8 : 0) | (k.reset ? 16 : 0);
    }
    // any token that cuts a window or drops the state?
    const bool cut_here = __syncthreads_or(tid < n && smark[tid] != (8 | (kSsmTaps - 1)) &&
                                           smark[tid] != (12 | (kSsmTaps - 1)));
    // a thread takes a channel and 8 tokens at a time
    constexpr int kStrip = 8, CH = 2 * N + kCols;
    for (int i = tid; i < CH * (kTok / kStrip); i += kThreads) {
      const int j = i % CH, s0 = i / CH * kStrip;
      if (FIRST && j >= N && j < 2 * N) continue;      // C is not needed
      const int c = j < N ? cb + j : j < 2 * N ? cc + j - N : cx + j - 2 * N;
      const float4 w = *reinterpret_cast<const float4 *>(p.w + 4 * (size_t)c);
      const float bias = p.bias ? p.bias[c] : 0.f;
      const T *xc = x + (long long)(t0 + s0) * p.xbc_st + c;
      float in[kStrip + kSsmTaps - 1];                 // with the 3 inputs before
#pragma unroll
      for (int k = 0; k < kStrip + kSsmTaps - 1; ++k) {
        const int t = s0 + k - (kSsmTaps - 1);
        in[k] = t0 + t >= 0 && t < n
                    ? to_f32(xc[(long long)(k - (kSsmTaps - 1)) * p.xbc_st]) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kStrip; ++k) {
        const int t = s0 + k;
        float a0 = in[k], a1 = in[k + 1], a2 = in[k + 2];
        const int mark = smark[t];
        if (cut_here) {
          const int place = mark & 3;
          const bool old = (mark & 4) && past;
          auto cached = [&](int age) {
            return old ? to_f32(past[(size_t)(kSsmTaps - 1 + place - age) * p.channels + c]) : 0.f;
          };
          if (place < 3) a0 = cached(3);
          if (place < 2) a1 = cached(2);
          if (place < 1) a2 = cached(1);
        }
        float u = bias + w.w * in[k + 3] + w.z * a2 + w.y * a1 + w.x * a0;
        u = mark & 8 ? u / (1.f + expf(-u)) : 0.f;
        if (j < N) sB[t * N + j] = u * sd[t];
        else if (j < 2 * N) sC[t * N + j - N] = u;
        else sX[t * kCols + j - 2 * N] = u;
      }
    }
    __syncthreads();
    if (!FIRST && t0 == seg * cut.len) {
      after_previous();          // the states of the segments
      if (enter)
#pragma unroll
        for (int j = 0; j < NS; ++j) s[j] = enter[mine + (size_t)j * p.P];
    }
    // tokens past the segment's end have d = 0: they leave the state alone
    auto scan = [&](int t, bool reset) {
      const float a = sa[t], xv = sX[t * kCols + lane];
      const float4 *pb = reinterpret_cast<const float4 *>(sB + t * N + warp * NS),
                   *pc = reinterpret_cast<const float4 *>(sC + t * N + warp * NS);
      if (reset) {               // drops the state whatever it holds
        dropped = true;
#pragma unroll
        for (int j = 0; j < NS; ++j) s[j] = 0.f;
      }
      if (FIRST) decay *= a;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NS / 4; ++j) {
        const float4 bv = pb[j];
        s[4 * j] = fmaf(a, s[4 * j], bv.x * xv);
        s[4 * j + 1] = fmaf(a, s[4 * j + 1], bv.y * xv);
        s[4 * j + 2] = fmaf(a, s[4 * j + 2], bv.z * xv);
        s[4 * j + 3] = fmaf(a, s[4 * j + 3], bv.w * xv);
        if (!FIRST) {
          const float4 cv = pc[j];
          acc.x += cv.x * s[4 * j];
          acc.y += cv.y * s[4 * j + 1];
          acc.z += cv.z * s[4 * j + 2];
          acc.w += cv.w * s[4 * j + 3];
        }
      }
      if (!FIRST) sY[(warp * kTok + t) * kCols + lane] = (acc.x + acc.y) + (acc.z + acc.w);
    };
    if (cut_here) {
#pragma unroll 1
      for (int t = 0; t < kTok; ++t) scan(t, (smark[t] & 16) != 0);
    } else {
#pragma unroll 4
      for (int t = 0; t < kTok; ++t) scan(t, false);
    }
    if (FIRST) continue;
    __syncthreads();
    for (int i = tid; i < n * kCols; i += kThreads) {
      const int t = i / kCols, c = i % kCols;
      float v = 0.f;
      if (smark[t] & 8) {
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
  if (FIRST) {     // what the segment adds to the state that enters the next
    float *out = seg_state + ((size_t)(seg + 1) * p.B * p.H + bh) * per;
#pragma unroll
    for (int j = 0; j < NS; ++j) out[mine + (size_t)j * p.P] = s[j];
    if (tid == 0 && tile == 0)
      seg_decay[(size_t)seg * p.B * p.H + bh] = dropped ? -1.f : decay;
    return;
  }
  if (seg + 1 < cut.segs) return;
  if (p.conv_out) {      // the last segments' CTAs share a row's channels
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
    for (int j = 0; j < NS; ++j) p.final_state[(size_t)bh * per + mine + (size_t)j * p.P] = s[j];
  }
}

// The states that enter the segments, in place: S_0 is the initial state,
// S_{i+1} = decay_i S_i + what segment i added.  A decay of -1: a reset.
__global__ void __launch_bounds__(256)
    ssm_simt_chain_kernel(const float *initial, float *seg_state, const float *seg_decay, int segs,
                          int heads, size_t per) {
  start_next();
  after_previous();
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, n = (size_t)heads * per;
  if (i >= n) return;
  const int bh = (int)(i / per);
  float s = initial ? initial[i] : 0.f;
  seg_state[i] = s;
  constexpr int kBatch = 8;          // loads in flight
  for (int k0 = 0; k0 + 1 < segs; k0 += kBatch) {
    float a[kBatch], v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k0 + k + 1 < segs) {
        a[k] = seg_decay[(size_t)(k0 + k) * heads + bh];
        v[k] = seg_state[(size_t)(k0 + k + 1) * n + i];
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k0 + k + 1 < segs) {
        // a reset drops the state whatever it holds; a decay that underflows
        // does not: a NaN stays one
        s = (a[k] < 0.f ? 0.f : a[k] * s) + v[k];
        seg_state[(size_t)(k0 + k + 1) * n + i] = s;
      }
  }
}

template <typename T, int N>
cudaError_t launch_simt(const SsmParams &p, cudaStream_t cs) {
  const size_t smem = sizeof(float) * (2 * kTok * N + kTok * kCols * (1 + kWarps));
  const SimtCut cut = simt_cut(p.B, p.T, p.H, p.P);
  const unsigned chains = (unsigned)(p.B * p.H * (p.P / kCols));
  float *state = reinterpret_cast<float *>(p.ws);
  float *decay = state + (size_t)cut.segs * p.B * p.H * N * p.P;
  cudaError_t e = cudaFuncSetAttribute(ssm_simt_kernel<T, N, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(ssm_simt_kernel<T, N, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (cut.segs > 1) {
    ssm_simt_kernel<T, N, true>
        <<<chains * (cut.segs - 1), kThreads, smem, cs>>>(p, cut, state, decay);
    const size_t per = (size_t)N * p.P, n = (size_t)p.B * p.H * per;
    e = cudaGetLastError();
    if (e == cudaSuccess)
      e = launch_next(ssm_simt_chain_kernel, (unsigned)((n + 255) / 256), 256, 0, cs,
                      p.initial_state, state, decay, cut.segs, p.B * p.H, per);
    return e != cudaSuccess ? e
                            : launch_next(ssm_simt_kernel<T, N, false>, chains * cut.segs,
                                          kThreads, smem, cs, p, cut, state, decay);
  }
  ssm_simt_kernel<T, N, false><<<chains * cut.segs, kThreads, smem, cs>>>(p, cut, state, decay);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_simt_t(const SsmParams &p, cudaStream_t cs) {
  return p.N == 32 ? launch_simt<T, 32>(p, cs) : p.N == 64 ? launch_simt<T, 64>(p, cs)
                                                           : launch_simt<T, 128>(p, cs);
}

// The segments' states and decays.
size_t simt_bytes(const kda_ssm_shape *s) {
  const SimtCut cut = simt_cut(s->B, s->T, s->H, s->P);
  if (cut.segs == 1) return 0;
  return align_up(sizeof(float) * (size_t)cut.segs * s->B * s->H * ((size_t)s->N * s->P + 1), 256);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// AUTO: the tensor cores, but for long rows of few heads, whose chain of blocks
// no other CTA hides (bf16, one row of 8192 tokens, N = 64: 1 head of 32 115 us
// against 43 on the CUDA cores, 8 heads 119 against 125, 18 heads 133 against 240;
// 4 heads of 1024 tokens 28 against 24; N = 128, 2000 tokens 43 against 43).  In fp32, where they round more (4e-7 against 1e-7), from the
// size on at which they take about half the time (one row of 8192 tokens, 32 heads
// of 128, N = 128: 0.40 ms against 3.6; 3 rows of 700 tokens, 6 heads of 64: 39 us
// against 98; of 997 tokens, heads of 32, N = 64: 37 against 39).
bool use_tc(const kda_ssm_shape *s, kda_impl impl) {
  if (impl != KDA_IMPL_AUTO) return impl == KDA_IMPL_TC;
  const long long states = (long long)s->B * s->H * s->P * s->N;
  if (s->dtype == KDA_DTYPE_F32 && states * s->T <= (1ll << 26)) return false;
  return s->T < 16 * s->N || states > (1ll << 14);
}

size_t rows_bytes(int B) { return align_up(sizeof(WsHeader) + sizeof(SsmRow) * (size_t)B, 256); }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_ssm_fwd_workspace_size(const kda_ssm_shape *s, kda_impl impl) {
  if (check_ssm_shape(s) != KDA_OK) return 0;
  const bool bf16 = s->dtype == KDA_DTYPE_BF16;
  if (impl != KDA_IMPL_AUTO && impl != KDA_IMPL_SIMT && impl != KDA_IMPL_TC) return 0;
  if (!use_tc(s, impl)) return rows_bytes(s->B) + simt_bytes(s);
  SsmParams p = {};
  p.B = s->B; p.T = s->T; p.H = s->H; p.P = s->P; p.N = s->N; p.G = s->G;
  return rows_bytes(s->B) + ssm_tc_bytes(p, !bf16);
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
  // the CUDA-core kernel reads single elements but for w; AUTO asks for what the
  // tensor cores need at any size
  if (!aligned(w, 16)) return KDA_ERR_ALIGNMENT;
  if (impl != KDA_IMPL_SIMT) {
    for (const void *ptr : {xbc, z, (const void *)initial_state, conv_state, (const void *)y,
                            (const void *)final_state, (const void *)conv_out})
      if (!aligned(ptr, 16)) return KDA_ERR_ALIGNMENT;
    const int per16 = s->dtype == KDA_DTYPE_BF16 ? 8 : 4;
    for (long long stride : {s->xbc_stride_b, s->xbc_stride_t, z ? s->z_stride_b : 0,
                             z ? s->z_stride_t : 0})
      if (stride % per16) return KDA_ERR_ALIGNMENT;
  }
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
  if (use_tc(s, impl))
    e = launch_ssm_tc(p, !bf16, &reinterpret_cast<WsHeader *>(workspace)->status, cs);
  else
    e = bf16 ? launch_simt_t<__nv_bfloat16>(p, cs) : launch_simt_t<float>(p, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
