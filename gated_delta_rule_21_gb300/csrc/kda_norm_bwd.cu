// kda_norm_bwd.cu -- the gradients of the block norms (kda_norm.cu has the
// formulas).
#include "kda_norm.cuh"

namespace kda {
namespace norm {
namespace {

struct NormBwdParams {
  NormParams f;
  const void *d_out, *d_x;
  void *dy, *d_res, *d_gate;
  float *part_post, *part_pre, *part_gate;   // [units][D]
  long long gate_rows;
  int staged;      // bytes of staged rows
  int splits;      // units per gate row (group gates), 0: whole gate rows per unit
};

// Sums `acc` over the CTA's row groups and hands the totals to the first
// group's threads: put(column, values).  Uniform over the CTA.
template <typename Pc, int ITEMS, typename F>
__device__ __forceinline__ void flush(typename Pc::P (&acc)[ITEMS][Pc::E], int tpr, int rg,
                                      int group, int lane, int D, typename Pc::P *buf, F put) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = (lane + i * tpr) * Pc::kStep;
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
//   r = v - s2^3 mean(d_x w_pre m) m,  dy = s1 (aw r - c1 n1),
// and the column sums of r n1 give dw_post and (gate rows shared by rows,
// where act(gate) is a factor of the column) d_gate at once.  One piece per
// thread keeps these values for the second pass over the row, more pieces
// make them again from the staged inputs.
template <typename T, int VEC, int ITEMS, int GATE, int BS, int NS>
__global__ void __launch_bounds__(BS) norm_bwd_kernel(const NormBwdParams q) {
  using Pc = Piece<T, VEC>;
  using P = typename Pc::P;
  constexpr int E = Pc::E, W = Pc::kStep, kOut = 1, kX = 2, kRes = 3, kGate = GATE == kGateEach ? 4 : 0;
  constexpr bool kKeep = ITEMS * W <= 8;      // these stay in registers between the passes
  constexpr int KI = kKeep ? ITEMS : 1;
  using In = Stage<T, VEC, ITEMS, GATE == kGateEach ? 5 : 4, BS, NS>;
  constexpr int kAhead = NS > 0 ? NS - 1 : 0;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][4][32];
  const NormParams &p = q.f;
  const int tid = threadIdx.x, tpr = p.tpr, rg = p.rg;
  const int group = tid / tpr, lane = tid - group * tpr;
  start_next();          // norm_sum_kernel
  P *buf = reinterpret_cast<P *>(smem + q.staged);         // for flush, when rg > 1
  const int step = tpr * W * (int)sizeof(T);             // bytes between a thread's pieces
  const long long row_bytes = (long long)p.D * sizeof(T);
  In in;
  in.lane = lane;
  in.tpr = tpr;
  in.D = p.D;
  in.init(smem, tid, group, rg);
  in.src[0] = (const char *)p.y;
  in.src[kOut] = (const char *)q.d_out;
  in.src[kX] = (const char *)q.d_x;
  in.src[kRes] = (const char *)p.res;
  if constexpr (GATE == kGateEach) in.src[kGate] = (const char *)p.gate;
  bool has[ITEMS], whole[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    has[i] = (lane + i * tpr) * W < p.D;
    whole[i] = !Pc::kRagged || (lane + i * tpr) * W + W <= p.D;
  }
  int slot = 0;

  P dw1[ITEMS][E], dw2[ITEMS][E], w1k[KI][E], w2k[KI][E];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) dw1[i][e] = dw2[i][e] = both<P>(0.f);
  const P scale = both<P>(p.scale);
  // scale * w_post and w_pre of a piece
  auto weights = [&](int i, P(&w1)[E], P(&w2)[E]) {
    const int c = (lane + i * tpr) * W;
#pragma unroll
    for (int e = 0; e < E; ++e) w1[e] = w2[e] = both<P>(0.f);
    if (c < p.D) {
      Pc::weight(p.w_post + c, w1, whole[i]);
      if (p.w_pre) Pc::weight(p.w_pre + c, w2, whole[i]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) w1[e] = mul(w1[e], scale);
  };
  if (kKeep)
#pragma unroll
    for (int i = 0; i < KI; ++i) weights(i, w1k[i], w2k[i]);

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
        const int c = (lane + i * tpr) * W;
#pragma unroll
        for (int e = 0; e < E; ++e) es[i][e] = ga[i][e] = both<P>(0.f);
        if (c < p.D) {
          P d[E];
          Pc::get(Pc::read((const T *)p.gate + (size_t)g * p.D + c, whole[i]), ga[i]);
          gate_values<false>(p.act, ga[i], d);
        }
      }
    }
    int st = 0;
    long long at = (lo + group) * row_bytes + (long long)lane * W * sizeof(T);
    const long long advance = rg * row_bytes;
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
      in.fetch(s, lo + group + s * rg < hi, has, lo + group + s * rg, at + s * advance, step);
    for (long long row = lo + group; row - group < hi; row += rg, at += advance) {
      const bool live = row < hi;
      float s1 = 0.f, s2 = 0.f;
      if (live) {
        s1 = p.stats[row];
        s2 = p.stats[p.R + row];
      }
      in.turn([&]() {
        in.fetch(st == 0 ? kAhead : st - 1, row + kAhead * rg < hi, has, row + kAhead * rg,
                 at + kAhead * advance, step);
      });
      // n1, m, v, d_x, act(gate) and its derivative of a piece
      auto front = [&](int i, const P(&w1)[E], const P(&w2)[E], P(&n1)[E], P(&m)[E], P(&v)[E],
                       P(&gx)[E], P(&a)[E], P(&da)[E], P(&qv)[E]) {
        Pc::get(in.get(st, 0, i, whole[i], row, at, step), n1);
        if (q.d_out) Pc::get(in.get(st, kOut, i, whole[i], row, at, step), v);
        else
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = both<P>(0.f);
        if (q.d_x) Pc::get(in.get(st, kX, i, whole[i], row, at, step), gx);
        else
#pragma unroll
          for (int e = 0; e < E; ++e) gx[e] = both<P>(0.f);
        if (p.res) Pc::get(in.get(st, kRes, i, whole[i], row, at, step), m);
        else
#pragma unroll
          for (int e = 0; e < E; ++e) m[e] = both<P>(0.f);
        if (GATE == kGateEach) {
          Pc::get(in.get(st, kGate, i, whole[i], row, at, step), a);
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
      P n1[KI][E], m[KI][E], v[KI][E], gx[KI][E], a[KI][E], da[KI][E];
      P acc0 = both<P>(0.f), acc1 = acc0, acc2 = acc0;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if (live && has[i]) {
          const int k = kKeep ? i : 0;
          P w1[E], w2[E], qv[E];
          if (!kKeep) weights(i, w1, w2);
          front(i, kKeep ? w1k[k] : w1, kKeep ? w2k[k] : w2, n1[k], m[k], v[k], gx[k], a[k], da[k],
                qv);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            acc0 = fma(mul(gx[k][e], kKeep ? w2k[k][e] : w2[e]), m[k][e], acc0);
            acc1 = fma(qv[e], v[k][e], acc1);
            acc2 = fma(qv[e], m[k][e], acc2);
          }
        }
      }
      float sum[3] = {total(acc0), total(acc1), total(acc2)};
      row_sum3(sum, tpr, red, slot);
      // s2 c2, times s2: r = v - kc m (in this order: the cube of s2 may overflow)
      const float kc = s2 * (s2 * (s2 * sum[0] * p.inv_d));
      const float c1 = (sum[1] - kc * sum[2]) * p.inv_d;
      const P nk = both<P>(-kc), nc = both<P>(-c1 * s1), ps1 = both<P>(s1), ps2 = both<P>(s2);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const long long o = at + (long long)i * step;
        if (live && has[i]) {
          const int k = kKeep ? i : 0;
          P w1[E], w2[E], oy[E], og[E], qv[E];
          if (!kKeep) {
            weights(i, w1, w2);
            front(i, w1, w2, n1[k], m[k], v[k], gx[k], a[k], da[k], qv);
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const P w = kKeep ? w1k[k][e] : w1[e];
            dw2[i][e] = fma(mul(gx[k][e], ps2), m[k][e], dw2[i][e]);
            v[k][e] = fma(m[k][e], nk, v[k][e]);            // r
            P aw = w;
            if (GATE == kGateEach) {
              const P x = mul(v[k][e], n1[k][e]);
              dw1[i][e] = fma(a[k][e], x, dw1[i][e]);
              og[e] = mul(mul(w, da[k][e]), x);
              aw = mul(w, a[k][e]);
            } else if (GATE == kGateGroup) {
              es[i < GI ? i : 0][e] = fma(v[k][e], n1[k][e], es[i < GI ? i : 0][e]);
              aw = mul(w, ga[i < GI ? i : 0][e]);
            } else {
              dw1[i][e] = fma(v[k][e], n1[k][e], dw1[i][e]);
            }
            oy[e] = fma(mul(aw, v[k][e]), ps1, mul(n1[k][e], nc));
          }
          Pc::write((char *)q.dy + o, oy, whole[i]);
          if (q.d_res) Pc::write((char *)q.d_res + o, v[k], whole[i]);
          if (GATE == kGateEach && q.d_gate)
            Pc::write((char *)q.d_gate + o, og, whole[i]);
        }
      }
      st = st == kAhead ? 0 : st + 1;
    }
    if (NS > 0) cp_async_wait<0>();
    if (In::kShared && NS > 0) __syncthreads();     // the last row is read
    if constexpr (GATE == kGateGroup) {
#pragma unroll
      for (int i = 0; i < GI; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) dw1[i][e] = fma(ga[i][e], es[i][e], dw1[i][e]);
      if (q.d_gate)
        flush<Pc, GI>(es, tpr, rg, group, lane, p.D, buf, [&](int i, int c, P(&s)[E]) {
          P w1[E], w2[E], a[E], d[E];
          weights(i, w1, w2);
          Pc::get(Pc::read((const T *)p.gate + (size_t)g * p.D + c, whole[i]), a);
          gate_values<true>(p.act, a, d);
#pragma unroll
          for (int e = 0; e < E; ++e) a[e] = mul(mul(w1[e], d[e]), s[e]);
          if (q.splits) Pc::store(q.part_gate + (size_t)blockIdx.x * p.D + c, a, whole[i]);
          else Pc::write((T *)q.d_gate + (size_t)g * p.D + c, a, whole[i]);
        });
    }
  }
  flush<Pc, ITEMS>(dw1, tpr, rg, group, lane, p.D, buf, [&](int i, int c, P(&s)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = mul(s[e], scale);
    Pc::store(q.part_post + (size_t)blockIdx.x * p.D + c, s, whole[i]);
  });
  if (p.w_pre)
    flush<Pc, ITEMS>(dw2, tpr, rg, group, lane, p.D, buf, [&](int i, int c, P(&s)[E]) {
      Pc::store(q.part_pre + (size_t)blockIdx.x * p.D + c, s, whole[i]);
    });
}

// Column sums of the units' partials: blockIdx.y 0 dw_post, 1 dw_pre, 2 + g
// gate row g.  32 columns x 32 row lanes, always in the same order.
template <typename T>
__global__ void __launch_bounds__(1024)
    norm_sum_kernel(const float *part_post, const float *part_pre, const float *part_gate,
                    float *dw_post, float *dw_pre, T *d_gate, int units, int splits, int D) {
  __shared__ float s[32][33];
  after_previous();
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

constexpr Built kBuilt[] = {{2, 8, 1, 256}, {2, 8, 1, 512}, {2, 8, 2, 512}, {2, 8, 4, 512},
                            {2, 2, 4, 256}, {2, 2, 4, 512}, {2, 2, 8, 1024},
                            {2, 1, 4, 256}, {2, 1, 4, 512}, {2, 1, 8, 1024},
                            {4, 4, 1, 256}, {4, 4, 1, 512}, {4, 4, 2, 512}, {4, 4, 4, 512},
                            {4, 4, 8, 512}, {4, 1, 4, 256}, {4, 1, 4, 512}, {4, 1, 16, 1024}};

// Units (CTAs) of the backward: as many as are resident on 152 SMs at up to
// 128 registers per thread, and no more than there are row groups.  (152 and not
// what this device has: the workspace's size goes by it, and may be asked for
// where there is no device.)
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

template <typename T, int VEC, int ITEMS, int GATE, int BS, int NS>
cudaError_t launch_g(NormBwdParams q, int units, cudaStream_t stream) {
  auto kern = norm_bwd_kernel<T, VEC, ITEMS, GATE, BS, NS>;
  const int threads = q.f.tpr * q.f.rg;
  q.staged = (int)Stage<T, VEC, ITEMS, GATE == kGateEach ? 5 : 4, BS, NS>::bytes(q.f.D, q.f.rg);
  const size_t smem = q.staged + (q.f.rg > 1 ? sizeof(float) * threads * Piece<T, VEC>::kStep : 0);
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  kern<<<units, threads, smem, stream>>>(q);
  return cudaGetLastError();
}
template <typename T, int VEC, int ITEMS, int BS, int NS>
cudaError_t launch(const NormBwdParams &q, int gate, int units, cudaStream_t s) {
  if (gate == kGateNone) return launch_g<T, VEC, ITEMS, kGateNone, BS, NS>(q, units, s);
  if (gate == kGateEach) return launch_g<T, VEC, ITEMS, kGateEach, BS, NS>(q, units, s);
  return launch_g<T, VEC, ITEMS, kGateGroup, BS, NS>(q, units, s);
}

}  // namespace
}  // namespace norm
}  // namespace kda

using namespace kda;
using namespace kda::norm;

extern "C" {

size_t kda_block_norm_bwd_workspace_size(const kda_norm_desc *d, int has_gate) {
  if (check_desc(d, has_gate != 0) != KDA_OK) return 0;
  // the largest over the layouts, since types and pointers choose between them
  size_t n = 0;
  for (int v = 0; v < 4; ++v) {
    const Layout l = layout_for(kBuilt, d->dim, v < 2 ? 2 : 4, v % 2 != 0);
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
  const Layout l = layout_for(kBuilt, d->dim, bf16 ? 2 : 4, vec);
  NormBwdParams q = {};
  q.f = params_of(d, l, y, w_post, residual, gate, w_pre);
  q.f.stats = const_cast<float *>(stats);
  q.d_out = d_out; q.d_x = d_x; q.dy = dy; q.d_res = d_residual; q.d_gate = d_gate;
  q.gate_rows = gate ? d->gate_rows : 0;
  const int mode = gate_mode(d, gate);
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
  const bool small = l.bs == 256;
  if (l.vec == 8)
    e = l.items == 4   ? launch<B, 8, 4, 512, 0>(q, mode, units, cs)
        : l.items == 2 ? launch<B, 8, 2, 512, 2>(q, mode, units, cs)
        : small        ? launch<B, 8, 1, 256, 3>(q, mode, units, cs)
                       : launch<B, 8, 1, 512, 3>(q, mode, units, cs);
  else if (l.vec == 4)
    e = l.items == 8   ? launch<float, 4, 8, 512, 0>(q, mode, units, cs)
        : l.items == 4 ? launch<float, 4, 4, 512, 0>(q, mode, units, cs)
        : l.items == 2 ? launch<float, 4, 2, 512, 2>(q, mode, units, cs)
        : small        ? launch<float, 4, 1, 256, 3>(q, mode, units, cs)
                       : launch<float, 4, 1, 512, 3>(q, mode, units, cs);
  else if (l.vec == 2)
    e = l.items == 8 ? launch<B, 2, 8, 1024, 0>(q, mode, units, cs)
        : small      ? launch<B, 2, 4, 256, 3>(q, mode, units, cs)
                     : launch<B, 2, 4, 512, 3>(q, mode, units, cs);
  else if (bf16)
    e = l.items == 8 ? launch<B, 1, 8, 1024, 0>(q, mode, units, cs)
        : small      ? launch<B, 1, 4, 256, 2>(q, mode, units, cs)
                     : launch<B, 1, 4, 512, 2>(q, mode, units, cs);
  else
    e = l.items == 16 ? launch<float, 1, 16, 1024, 0>(q, mode, units, cs)
        : small       ? launch<float, 1, 4, 256, 3>(q, mode, units, cs)
                      : launch<float, 1, 4, 512, 2>(q, mode, units, cs);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  const bool gate_parts = mode == kGateGroup && q.splits && d_gate;
  const dim3 grid((d->dim + 31) / 32, 2 + (gate_parts ? (unsigned)d->gate_rows : 0));
  const float *pre = w_pre ? q.part_pre : nullptr;
  e = bf16 ? launch_next(norm_sum_kernel<B>, grid, 1024, 0, cs, q.part_post, pre, q.part_gate,
                         dw_post, dw_pre, (B *)d_gate, units, q.splits, d->dim)
           : launch_next(norm_sum_kernel<float>, grid, 1024, 0, cs, q.part_post, pre, q.part_gate,
                         dw_post, dw_pre, (float *)d_gate, units, q.splits, d->dim);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
