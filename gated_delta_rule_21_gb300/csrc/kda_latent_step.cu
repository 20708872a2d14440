// kda_latent_step.cu -- the absorbed latent attention over the paged cache:
// entry point, the kernel on the CUDA cores and the one that joins the parts.
//
// The tokens of all sequences are cut into tiles of 128 (on the CUDA cores of 32), and the tiles
// evenly into one part for each SM, so a part may hold the end of one sequence, whole
// ones and the beginning of another.  Whole sequences are written at once;
// of the others each part leaves its sums with the softmax's maximum and sum, and
// a second kernel joins them.  The cut goes by the lengths on the device: a call
// that was captured into a graph follows the lengths that it finds.
#include <string.h>

#include "kda_f32x2.cuh"
#include "kda_latent.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 32;          // tokens in shared memory at once
constexpr int kLdW = kTokens + 4;

// CUDA cores, fp32.  The 32 rows of queries and 32 tokens lie in shared memory;
// a warp makes the scores of its 4 rows and their sums over the latents.  The tokens are
// cut in tiles of 32 (three texts of up to 997 tokens, 24 rows of 160 values: 21 us with
// the join, with tiles of 128 44); what bounds it is the latency of a tile's steps.
template <typename T>
__global__ void __launch_bounds__(kThreads) step_simt_kernel(Step p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ long long tmp[36];
  __shared__ int place[kTokens];
  const int D = p.C + p.R, ld = D + 4;
  float *sq = sm, *sc = sq + kRows * ld, *sw = sc + kTokens * ld;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lane = tid & 31, warp = tid >> 5;
  Cursor cur = {find_work(p, tmp), true};
  const float scale = p.scale * kLog2e;
  Segment g{};
  while (cur.next(p, g)) {
    const Seq &s = g.s;
    const bool whole = g.whole;
    const int r0 = g.rt * kRows, rows = p.T * p.H;
    if (tid == 0) Cursor::note(p, g);
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kThreads) {
      const int r = r0 + i / D, c = i % D;
      float v = 0.f;
      if (r < rows)
        v = to_f32(c < p.C ? at<T>(p.q, p.q_s, g.b, r / p.H, r % p.H)[c]
                           : at<T>(p.qr, p.qr_s, g.b, r / p.H, r % p.H)[c - p.C]);
      sq[i / D * ld + c] = v;
    }
    int lim[2];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 2 * ty + i;
      lim[i] = r < rows ? seen(p, s, r) : 0;
    }
    u64 acc[4][4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][q][0] = acc[i][q][1] = 0;
    const int stop = min(s.held, (g.j0 + g.n) * p.tile);
    for (int k0 = g.j0 * p.tile; k0 < stop; k0 += kTokens) {
      __syncthreads();
      if (tid < kTokens) {      // -1: not there
        const int k = k0 + tid;
        const int pg = k < s.held ? p.table[(size_t)g.b * p.max_pages + k / p.page] : -1;
        place[tid] = pg >= 0 && pg < p.n_pages ? pg : -1;
      }
      __syncthreads();
#pragma unroll
      for (int i = warp; i < kTokens; i += kThreads / 32) {   // a warp a token
        const bool there = place[i] >= 0;
        const T *c = static_cast<const T *>(p.cache) + (there ? place[i] * p.page_stride : 0) +
                     (there ? (long long)((k0 + i) % p.page) * p.token_stride : 0);
#pragma unroll 5
        for (int e = lane; e < D; e += 32) sc[i * ld + e] = there ? to_f32(c[e]) : 0.f;
      }
      __syncthreads();
      u64 a2[2][2] = {{0, 0}, {0, 0}};
      const float *a = sq + 2 * ty * ld, *b = sc + tx * ld;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        ulonglong2 u[2], v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          u[i] = *reinterpret_cast<const ulonglong2 *>(a + i * ld + c);
          v[i] = *reinterpret_cast<const ulonglong2 *>(b + 16 * i * ld + c);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            a2[i][j] = fma2(u[i].x, v[j].x, a2[i][j]);
            a2[i][j] = fma2(u[i].y, v[j].y, a2[i][j]);
          }
      }
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[2], top = m[i];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float lo, hi;
          upk2(a2[i][j], lo, hi);
          const int k = tx + 16 * j;
          v[j] = k0 + k < lim[i] && place[k] >= 0 ? (lo + hi) * scale : -INFINITY;
          top = fmaxf(top, v[j]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.f : top;
        f[i] = exp2f(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float w = exp2f(v[j] - base);
          sum += w;
          sw[(2 * ty + i) * kLdW + tx + 16 * j] = w;
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * f[i] + sum;
        m[i] = top;
      }
      __syncwarp();
      // rows 4 warp + i: their factors stand in lanes 0 (i < 2) and 16
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g = __shfl_sync(0xffffffffu, f[i & 1], (i >> 1) * 16);
        const u64 gg = pk2(g, g);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[i][q][0] = mul2(acc[i][q][0], gg);
          acc[i][q][1] = mul2(acc[i][q][1], gg);
        }
      }
      const float *w = sw + 4 * warp * kLdW, *y = sc + 4 * lane;
#pragma unroll 2
      for (int k = 0; k < kTokens; ++k) {
        u64 ww[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = w[i * kLdW + k];
          ww[i] = pk2(e, e);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (128 * q >= p.C) continue;
          const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(y + k * ld + 128 * q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[i][q][0] = fma2(ww[i], v.x, acc[i][q][0]);
            acc[i][q][1] = fma2(ww[i], v.y, acc[i][q][1]);
          }
        }
      }
      __syncwarp();
    }
    const int slot = g.slot;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = 4 * warp + i, r = r0 + rr;
      const float mi = __shfl_sync(0xffffffffu, m[i & 1], (i >> 1) * 16);
      const float li = __shfl_sync(0xffffffffu, l[i & 1], (i >> 1) * 16);
      if (r >= rows) continue;
      bool bad = false;
      float none = 0.f;
      if (whole && li == 0.f) {
        const int n = seen(p, s, r);
        none = no_weights(n > 0 && any_there(p, g.b, n, lane));
      }
      const int t = r / p.H, h = r % p.H;
      T *o = static_cast<T *>(p.o) + (((size_t)g.b * p.T + t) * p.H + h) * p.C;
      float *part = p.parts + ((size_t)slot * kRows + rr) * p.C;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (128 * q >= p.C) continue;
        float v[4];
        upk2(acc[i][q][0], v[0], v[1]);
        upk2(acc[i][q][1], v[2], v[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 128 * q + 4 * lane + e;
          if (whole) {
            const float z = li == 0.f ? none : v[e] / li;
            bad |= !finite(z);
            o[c] = from_f32<T>(z);
          } else {
            part[c] = v[e];
          }
        }
      }
      if (lane == 0) {
        if (!whole) {
          p.stats[2 * ((size_t)slot * kRows + rr)] = mi;
          p.stats[2 * ((size_t)slot * kRows + rr) + 1] = li;
        } else if (p.lse) {
          p.lse[((size_t)g.b * p.H + h) * p.T + t] =
              li == 0.f ? -INFINITY : (mi + log2f(li)) * kLn2;
        }
      }
      if (whole && p.T > 1 && __any_sync(0xffffffffu, bad)) {
        __syncwarp();
        step_row<T>(p, g.b, r, seen(p, s, r), lane);
      }
    }
  }
}

// Joins the parts of one row, p.C / 4 threads a row with four channels each.  kGroups
// of them share the parts of one row (where there are few rows with many parts), or
// with kGroups 1 take a row each.
template <typename T, int kGroups>
__global__ void __launch_bounds__(512) join_kernel(Step p, int block_rows) {
  __shared__ float4 sums[kGroups > 1 ? 512 : 1];
  __shared__ float s_l[kGroups];
  const int cols = p.C / 4, lane = threadIdx.x & 31, col = threadIdx.x % cols,
            group = kGroups > 1 ? threadIdx.x / cols : 0;
  const int rows = p.T * p.H;
  const unsigned index = blockIdx.x * (unsigned)block_rows +
                         (kGroups > 1 ? 0u : threadIdx.x / (unsigned)cols);
  after_previous();
  if (index >= (unsigned)p.B * (unsigned)rows) return;    // (a row's threads are whole warps)
  const int b = (int)(index / (unsigned)rows), r = (int)(index % (unsigned)rows);
  const int t = r / p.H, h = r % p.H;
  const Seq s = seq_of(p, b);
  const int2 range = p.plan[(size_t)b * p.row_tiles + r / kRows];
  T *o = static_cast<T *>(p.o) + (((size_t)b * p.T + t) * p.H + h) * p.C;
  float *lse = p.lse ? p.lse + ((size_t)b * p.H + h) * p.T + t : nullptr;
  if (s.held == 0) {
    if (group == 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[4 * col + e] = from_f32<T>(0.f);
      if (col == 0 && lse) *lse = -INFINITY;
    }
    return;
  }
  auto none = [&] {        // a row without weights: four channels a thread
    const int n = seen(p, s, r);
    if (n > 0 && any_there(p, b, n, lane))
      for (int e = 0; e < 4; ++e) o[4 * col + e] = from_f32<T>(no_weights(true));
  };
  if (range.x < 0) {
    if (group == 0 && range.y >> r % kRows & 1) none();
    return;
  }
  const int first = range.x, g0 = first >> 1, g1 = range.y;
  auto slot = [&](int g) { return (size_t)(g == g0 ? first : 2 * g) * kRows + r % kRows; };
  const float2 *stats = reinterpret_cast<const float2 *>(p.stats);
  float m = -INFINITY;
  for (int g = g0 + lane; g <= g1; g += 32) m = fmaxf(m, stats[slot(g)].x);
#pragma unroll
  for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  const float base = m == -INFINITY ? 0.f : m;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 8
  for (int g = g0 + group; g <= g1; g += kGroups) {
    const size_t k = slot(g);
    const float2 z = stats[k];
    const float4 x = reinterpret_cast<const float4 *>(p.parts)[k * cols + col];
    const float f = exp2f(z.x - base);
    l = fmaf(f, z.y, l);
    a.x = fmaf(f, x.x, a.x); a.y = fmaf(f, x.y, a.y);
    a.z = fmaf(f, x.z, a.z); a.w = fmaf(f, x.w, a.w);
  }
  if (kGroups > 1) {
    sums[threadIdx.x] = a;
    if (col == 0) s_l[group] = l;
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      const float4 x = sums[g * cols + col];
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      l += s_l[g];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float v[4] = {a.x, a.y, a.z, a.w};
  bool bad = false;
  struct alignas(4 * sizeof(T)) Four {
    T x[4];
  } w;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float z = l == 0.f ? 0.f : v[e] * inv;
    bad |= !finite(z);
    w.x[e] = from_f32<T>(z);
  }
  *reinterpret_cast<Four *>(o + 4 * col) = w;
  if (l == 0.f) none();    // (all threads of the row or none)
  if (col == 0 && lse) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  if (p.T == 1) return;   // every row sees what the others see
  // a row with a value that is not finite, again; its warps write the same values
  const int named = 1 + (kGroups > 1 ? 0 : threadIdx.x / cols);
  int any = bad ? 1 : 0;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
               "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
               : "=r"(any)
               : "r"(any), "r"(named), "r"(cols)
               : "memory");
  if (any) step_row<T>(p, b, r, seen(p, s, r), lane);
}

template <typename T>
cudaError_t launch_simt(const Step &p, cudaStream_t cs) {
  const size_t smem = sizeof(float) * ((size_t)(kRows + kTokens) * (p.C + p.R + 4) + kRows * kLdW);
  cudaError_t e = cudaFuncSetAttribute(step_simt_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  step_simt_kernel<T><<<kParts, kThreads, smem, cs>>>(p);
  return cudaGetLastError();
}

// A row has about 152 / (sequences x row tiles) parts.  From 16 of these on four groups of
// threads share them (one text of 32768 tokens 20 us, with a group a row 31; four of
// 16384 22 and 26), with fewer a row has one group (16 texts of 2000 tokens 19 us, with
// four groups 24; 120 of 4096 126 and 160).
template <typename T>
cudaError_t launch_join(const Step &p, cudaStream_t cs) {
  const int cols = p.C / 4;
  const long long rows = (long long)p.B * p.T * p.H;
  if ((long long)p.B * p.row_tiles * 16 <= kParts)
    return launch_next(join_kernel<T, 4>, dim3((unsigned)rows), (unsigned)(cols * 4), 0, cs, p, 1);
  const int block_rows = 256 / cols;
  return launch_next(join_kernel<T, 1>, dim3((unsigned)((rows + block_rows - 1) / block_rows)), 256u,
                     0, cs, p, block_rows);
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

kda_status check(const kda_latent_cache *s) {
  if (!s || s->B < 1 || s->T < 1 || s->H < 1 || s->max_pages < 1 || s->n_pages < 1 ||
      s->page_size < 1)
    return KDA_ERR_INVALID_ARG;
  if (s->dtype != KDA_DTYPE_F32 && s->dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
  if (s->C != 128 && s->C != 256 && s->C != 512) return KDA_ERR_UNSUPPORTED;
  if (s->R != 0 && s->R != 32 && s->R != 64) return KDA_ERR_UNSUPPORTED;
  if ((double)s->B * s->T * s->H >= 2147483648.0 || (long long)s->T * s->H >= (1ll << 24) ||
      (double)s->max_pages * s->page_size >= 2147483000.0)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

size_t plan_bytes(const kda_latent_cache *s) {
  return align_up(sizeof(int2) * (size_t)s->B * (((size_t)s->T * s->H + kRows - 1) / kRows), 256);
}

}  // namespace
}  // namespace latent
}  // namespace kda

using namespace kda;
using namespace kda::latent;

extern "C" {

size_t kda_latent_step_workspace_size(const kda_latent_cache *s) {
  if (!s || s->B < 1 || s->T < 1 || s->H < 1) return 0;
  if (s->C != 128 && s->C != 256 && s->C != 512) return 0;
  return sizeof(WsHeader) + plan_bytes(s) + sizeof(float) * 2 * kParts * kRows * (s->C + 2);
}

kda_status kda_latent_step(const kda_latent_cache *s, const void *q, const void *q_rope,
                           const void *cache, const int32_t *page_table, const int32_t *lengths,
                           const int32_t *new_tokens, float scale, void *o, float *lse,
                           void *workspace, size_t workspace_bytes, kda_impl impl,
                           kda_stream_t stream) {
  const kda_status st = check(s);
  if (st != KDA_OK) return st;
  if (!q || !cache || !page_table || !lengths || !o || !(fabsf(scale) < INFINITY))
    return KDA_ERR_INVALID_ARG;
  if ((s->R > 0) != (q_rope != nullptr)) return KDA_ERR_INVALID_ARG;
  if (impl != KDA_IMPL_AUTO && impl != KDA_IMPL_SIMT && impl != KDA_IMPL_TC)
    return KDA_ERR_INVALID_ARG;
  const bool bf16 = s->dtype == KDA_DTYPE_BF16;
  for (const void *x : {q, q_rope, cache})
    if (!aligned(x, bf16 ? 2 : 4)) return KDA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_table, (const void *)lengths,
                        (const void *)new_tokens, (const void *)lse})
    if (!aligned(x, 4)) return KDA_ERR_ALIGNMENT;
  if (!aligned(o, 16)) return KDA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kda_latent_step_workspace_size(s)) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KDA_ERR_ALIGNMENT;
  Step p;
  memset(&p, 0, sizeof(p));
  p.B = s->B; p.T = s->T; p.H = s->H; p.C = s->C; p.R = s->R;
  p.max_pages = s->max_pages; p.n_pages = s->n_pages; p.page = s->page_size;
  p.row_tiles = (int)(((long long)s->T * s->H + kRows - 1) / kRows);
  p.page_stride = s->n_pages > 1 ? s->page_stride : 0;
  p.token_stride = s->page_size > 1 ? s->token_stride : 0;
  p.q = q; p.qr = q_rope; p.cache = cache;
  p.q_s = strides_of(s->B, s->T, s->H, s->q_stride_b, s->q_stride_t, s->q_stride_h);
  if (q_rope)
    p.qr_s = strides_of(s->B, s->T, s->H, s->q_rope_stride_b, s->q_rope_stride_t,
                        s->q_rope_stride_h);
  p.table = page_table; p.lengths = lengths; p.fresh = new_tokens;
  p.scale = scale;
  p.o = o; p.lse = lse;
  char *ws = static_cast<char *>(workspace);
  p.status = &reinterpret_cast<WsHeader *>(ws)->status;
  p.plan = reinterpret_cast<int2 *>(ws + sizeof(WsHeader));
  p.parts = reinterpret_cast<float *>(ws + sizeof(WsHeader) + plan_bytes(s));
  p.stats = p.parts + (size_t)2 * kParts * kRows * s->C;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const bool can = bf16 && step_tc_ok(p);
  if (impl == KDA_IMPL_TC && !can) return KDA_ERR_UNSUPPORTED;
  const bool tc = can && impl != KDA_IMPL_SIMT;
  p.tile = tc ? 128 : kTokens;
  // (With 1, 3 and 5: 120 texts of up to 8192 tokens 131, 127.5, 132 us; 64 of them 80, 77, 77;
  // 300 of up to 2000 110, 104, 109; 16 of up to 32768 67, 69, 68; 16 of 2000 19.6, 19.3, 22.6;
  // 120 of 500 33, 31, 30; 8 of 5000 with 64 heads 31, 29, 29)
  p.extra = 3;
  cudaError_t e = tc ? launch_step_tc(p, cs)
                  : bf16 ? launch_simt<__nv_bfloat16>(p, cs)
                         : launch_simt<float>(p, cs);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  e = bf16 ? launch_join<__nv_bfloat16>(p, cs) : launch_join<float>(p, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
