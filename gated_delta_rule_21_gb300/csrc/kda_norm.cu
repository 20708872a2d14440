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
// The forward is bound by HBM: 8192 rows of 4096 bf16 with a gate per row in
// 64 us, 77 % of the copy bandwidth.  The backward has 512 threads and 128
// registers on an SM and waits for its row's sums: the same rows in 103 us
// (67 %), 131072 rows of 128 in 39 us.  Rows whose length or pointers do not
// allow 16-byte accesses take the same code with pieces of 4 bytes (5049 rows of
// 2292: 45 us); bf16 rows of odd length, which begin in the middle of a word,
// are joined in shared memory (of 2291: 61 us).
// This file: the forward; kda_norm_bwd.cu: the backward.
#include "kda_norm.cuh"

namespace kda {
namespace norm {
namespace {

// A CTA owns a contiguous range of rows, one row per row group at a time; of
// a gate row shared by rows act(gate) is made once.  A thread has 16 elements
// of a row, so that a row's two reductions weigh little (8192 rows of 4096 bf16:
// 64 us; with 8 elements 69).
template <typename T, int VEC, int ITEMS, int GATE, int BS, int NS>
__global__ void __launch_bounds__(BS) norm_fwd_kernel(const NormParams p) {
  using Pc = Piece<T, VEC>;
  using P = typename Pc::P;
  constexpr int E = Pc::E, W = Pc::kStep, kRes = 1, kGate = 2;
  using In = Stage<T, VEC, ITEMS, GATE == kGateEach ? 3 : 2, BS, NS>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][32];
  const int tid = threadIdx.x, tpr = p.tpr, rg = p.rg;
  const int group = tid / tpr, lane = tid - group * tpr;
  const int step = tpr * W * (int)sizeof(T);        // bytes between a thread's pieces
  const long long row_bytes = (long long)p.D * sizeof(T);
  In in;
  in.lane = lane;
  in.tpr = tpr;
  in.D = p.D;
  in.init(smem, tid, group, rg);
  in.src[0] = (const char *)p.y;
  in.src[kRes] = (const char *)p.res;
  if constexpr (GATE == kGateEach) in.src[kGate] = (const char *)p.gate;
  bool has[ITEMS], whole[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    has[i] = (lane + i * tpr) * W < p.D;
    whole[i] = !Pc::kRagged || (lane + i * tpr) * W + W <= p.D;
  }
  const float *w_post = p.w_post + lane * W, *w_pre = p.w_pre ? p.w_pre + lane * W : nullptr;
  const int wstep = tpr * W;
  int slot = 0, st = 0;
  const long long lo = (long long)blockIdx.x * p.R / gridDim.x,
                  hi = (long long)(blockIdx.x + 1) * p.R / gridDim.x;
  constexpr int GI = GATE == kGateGroup ? ITEMS : 1, kAhead = NS > 0 ? NS - 1 : 0;
  P ga[GI][E];
  unsigned ga_row = ~0u;
  long long at = (lo + group) * row_bytes + (long long)lane * W * sizeof(T);
  const long long advance = rg * row_bytes;
#pragma unroll
  for (int s = 0; s < kAhead; ++s)
    in.fetch(s, lo + group + s * rg < hi, has, lo + group + s * rg, at + s * advance, step);
  for (long long row = lo + group; row - group < hi; row += rg, at += advance) {
    const bool live = row < hi;
    in.turn([&]() {
      in.fetch(st == 0 ? kAhead : st - 1, row + kAhead * rg < hi, has, row + kAhead * rg,
               at + kAhead * advance, step);
    });
    if (GATE == kGateGroup && live) {
      const unsigned g = (unsigned)row / p.rows_per_gate;
      if (g != ga_row) {
        ga_row = g;
#pragma unroll
        for (int i = 0; i < GI; ++i) {
          P d[E];
          if (has[i]) {
            Pc::get(Pc::read((const char *)p.gate + g * row_bytes +
                                 (long long)lane * W * sizeof(T) + i * step,
                             whole[i]),
                    ga[i]);
            gate_values<false>(p.act, ga[i], d);
          }
        }
      }
    }
    P v[ITEMS][E], acc = both<P>(0.f);
    if (live) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (has[i]) {
          Pc::get(in.get(st, 0, i, whole[i], row, at, step), v[i]);
#pragma unroll
          for (int e = 0; e < E; ++e) acc = fma(v[i][e], v[i][e], acc);
        }
    }
    const float s1 = rsqrtf(row_sum(total(acc), tpr, red, slot) * p.inv_d + p.eps);
    const P k = both<P>(s1 * p.scale);
    acc = both<P>(0.f);
    if (live) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        if (has[i]) {
          P w[E], a[E];
          Pc::weight(w_post + i * wstep, w, whole[i]);
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = mul(v[i][e], mul(w[e], k));
          if (GATE == kGateEach) {
            P d[E];
            Pc::get(in.get(st, kGate < (GATE == kGateEach ? 3 : 2) ? kGate : 0, i, whole[i], row, at, step), a);
            gate_values<false>(p.act, a, d);
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = mul(v[i][e], a[e]);
          }
          if (GATE == kGateGroup)
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = mul(v[i][e], ga[i < GI ? i : 0][e]);
          if (p.res) {
            Pc::get(in.get(st, kRes, i, whole[i], row, at, step), a);
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = add(v[i][e], a[e]);
          }
          Pc::write((char *)p.out + at + (long long)i * step, v[i], whole[i]);
#pragma unroll
          for (int e = 0; e < E; ++e) acc = fma(v[i][e], v[i][e], acc);
        }
    }
    float s2 = 0.f;
    if (w_pre) {
      s2 = rsqrtf(row_sum(total(acc), tpr, red, slot) * p.inv_d + p.eps);
      if (live) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
          if (has[i]) {
            P w[E];
            Pc::weight(w_pre + i * wstep, w, whole[i]);
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = mul(v[i][e], mul(w[e], both<P>(s2)));
            Pc::write((char *)p.x + at + (long long)i * step, v[i], whole[i]);
          }
      }
    }
    if (p.stats && live && lane == 0) {
      p.stats[row] = s1;
      p.stats[p.R + row] = s2;
    }
    st = st == kAhead ? 0 : st + 1;
  }
  if (NS > 0) cp_async_wait<0>();
}

template <typename T, int VEC, int ITEMS, int GATE, int BS, int NS>
cudaError_t launch_g(const NormParams &p, cudaStream_t stream) {
  auto kern = norm_fwd_kernel<T, VEC, ITEMS, GATE, BS, NS>;
  const int threads = p.tpr * p.rg;
  const size_t smem = Stage<T, VEC, ITEMS, GATE == kGateEach ? 3 : 2, BS, NS>::bytes(p.D, p.rg);
  cudaError_t e = allow_smem(kern, smem);
  int per_sm = 1;
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
  if (e != cudaSuccess) return e;
  const long long n = (p.R + p.rg - 1) / p.rg, most = (long long)num_sms() * per_sm;
  kern<<<(unsigned)(n < most ? n : most), threads, smem, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, int VEC, int ITEMS, int BS, int NS>
cudaError_t launch(const NormParams &p, int gate, cudaStream_t s) {
  if (gate == kGateNone) return launch_g<T, VEC, ITEMS, kGateNone, BS, NS>(p, s);
  if (gate == kGateEach) return launch_g<T, VEC, ITEMS, kGateEach, BS, NS>(p, s);
  return launch_g<T, VEC, ITEMS, kGateGroup, BS, NS>(p, s);
}

}  // namespace

kda_status check_desc(const kda_norm_desc *d, bool has_gate) {
  if (!d || d->rows < 1 || d->dim < 1) return KDA_ERR_INVALID_ARG;
  if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
  if (d->gate_act < KDA_GATE_NONE || d->gate_act > KDA_GATE_TANH) return KDA_ERR_INVALID_ARG;
  if (!(d->scale == d->scale) || !(d->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
  if (has_gate && (d->gate_rows < 1 || d->rows % d->gate_rows)) return KDA_ERR_INVALID_ARG;
  if (d->dim > kMaxDim || d->rows >= (1ll << 31)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace norm
}  // namespace kda

using namespace kda;
using namespace kda::norm;

extern "C" kda_status kda_block_norm_fwd(const kda_norm_desc *d, const void *y,
                                         const float *w_post, const void *residual,
                                         const void *gate, const float *w_pre, void *out, void *x,
                                         float *stats, kda_stream_t stream) {
  const kda_status st = check_desc(d, gate != nullptr);
  if (st != KDA_OK) return st;
  if (!y || !w_post || !out || (w_pre != nullptr) != (x != nullptr)) return KDA_ERR_INVALID_ARG;
  // stats are for the backward, which reads the residual: it must outlive this call
  if (stats && out == residual) return KDA_ERR_INVALID_ARG;
  const bool bf16 = d->dtype == KDA_DTYPE_BF16;
  bool vec = true;
  for (const void *ptr : {y, (const void *)w_post, residual, gate, (const void *)w_pre,
                          (const void *)out, (const void *)x})
    vec = vec && aligned16(ptr);
  static const Built built[] = {{2, 8, 2, 256}, {2, 8, 2, 512}, {2, 8, 4, 512},
                                {2, 2, 4, 512}, {2, 2, 8, 1024}, {2, 1, 4, 512}, {2, 1, 8, 1024},
                                {4, 4, 2, 256}, {4, 4, 2, 512}, {4, 4, 4, 512}, {4, 4, 8, 512},
                                {4, 1, 8, 256}, {4, 1, 8, 512}, {4, 1, 16, 1024}};
  const Layout l = layout_for(built, d->dim, bf16 ? 2 : 4, vec);
  NormParams p = params_of(d, l, y, w_post, residual, gate, w_pre);
  p.out = out; p.x = x; p.stats = stats;
  const int mode = gate_mode(d, gate);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  using B = __nv_bfloat16;
  if (l.vec == 8)
    e = l.items == 4   ? launch<B, 8, 4, 512, 0>(p, mode, cs)
        : l.bs == 256  ? launch<B, 8, 2, 256, 2>(p, mode, cs)
                       : launch<B, 8, 2, 512, 3>(p, mode, cs);
  else if (l.vec == 4)
    e = l.items == 8   ? launch<float, 4, 8, 512, 0>(p, mode, cs)
        : l.items == 4 ? launch<float, 4, 4, 512, 0>(p, mode, cs)
        : l.bs == 256  ? launch<float, 4, 2, 256, 3>(p, mode, cs)
                       : launch<float, 4, 2, 512, 3>(p, mode, cs);
  else if (l.vec == 2)
    e = l.bs == 512 ? launch<B, 2, 4, 512, 2>(p, mode, cs) : launch<B, 2, 8, 1024, 0>(p, mode, cs);
  else if (bf16)
    e = l.bs == 512 ? launch<B, 1, 4, 512, 2>(p, mode, cs) : launch<B, 1, 8, 1024, 2>(p, mode, cs);
  else
    e = l.items == 16 ? launch<float, 1, 16, 1024, 0>(p, mode, cs)
        : l.bs == 256 ? launch<float, 1, 8, 256, 3>(p, mode, cs)
                      : launch<float, 1, 8, 512, 2>(p, mode, cs);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
