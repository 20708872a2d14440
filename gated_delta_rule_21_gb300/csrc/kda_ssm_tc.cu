// kda_ssm_tc.cu -- the selective state space operator on prompts, on the
// tensor cores (tcgen05): bf16 or fp32 activations, N, P in {32, 64, 128}.
//
// In blocks of 128 tokens, with c_r the sum of d A over a block's tokens up to
// r and S the state that enters the block,
//     y_r  = e^{c_r} C_r^T S + sum_{j <= r} (C_r . B_j) e^{c_r - c_j} d_j x_j
//     S'   = e^{c_127} S + sum_j e^{c_127 - c_j} d_j B_j (outer) x_j
// so a block is three products of 128 rows and the state is carried from
// block to block.  Three launches:
//   1. ssm_prep_kernel: the convolution of B and C into operand tiles, and per
//      token and head the factors above (all blocks in parallel).
//   2. ssm_state_kernel: one CTA per (row, head, column tile) walks the blocks:
//      the convolution of x, S' and, for each block, the S that enters it.
//   3. ssm_out_kernel: y of every (block, head), all in parallel.
//
// Rounding.  The final state is carried to tokens and on, so S' is formed to
// fp32 grade: B and the scaled x are each split into two fp16 parts, scaled by
// powers of two for each few channels of a block (22 bits of what is not 2^18 times
// smaller than the largest), all four products are added and S is updated in fp32
// registers, never in the accumulator: 1.5e-7 of the state's norm off, either type,
// as fp32 arithmetic is (two bf16 parts: 3.4e-6, and 20 us less of the 361 below).
// y of bf16 inputs is rounded to bf16 at the end (1.7e-3).  Of its products'
// operands x and the 128 x 128 matrix of factors, scaled by rows, are fp16 (2^-12
// each; x is also what D multiplies), C, B and S bf16, whose errors average out
// over the sums: 1.8e-3 to 2.2e-3 in all (all in bf16: 2.5e-3 to 2.9e-3, half of it
// from D x).  With fp32 inputs each is split in two of its kind and all four
// products added, C and B of C B^T in three, the small products first, since the
// accumulator loses bits at its own size (2e-7 to 7e-7, where an entering state
// is most of y; C and B in two parts 2.5e-6, the large products first 1.2e-6).
//
// What bounds it: 2 rows of 8192 tokens, 64 heads of 64, N = 128: prep 61 us,
// state 158 us, out 142 us; the row of 8192 tokens of 32 heads of 128 in 25
// segments: 16, 129 and 70 us.  The state kernel is a chain of 64 blocks on 128
// SMs, each its convolution's instructions and two barriers long; the other two
// are at the rate of their instructions and of exp2 and reciprocals.  (The
// first kernels of this form took 9.8 and 9.5 ms on the CUDA cores.)
#include <cuda_fp16.h>
#include <math_constants.h>

#include <type_traits>

#include "kda_ssm.cuh"
#include "kda_tc_common.cuh"
#include "kda_f32x2.cuh"

namespace kda {
namespace {

using namespace tc;
using bf16 = __nv_bfloat16;

constexpr int kQ = 128;            // tokens per block

// Tiles hold a block's tokens in slots, the 32 tokens of a quarter transposed
// as 8 strips of 4: the products sum over tokens in any order, and so a lane
// that convolves 4 consecutive tokens writes them 128 bytes apart while 8
// lanes write 8 neighbouring slots (no bank conflicts, no index arithmetic).
__host__ __device__ constexpr int slot_of(int token) {
  return (token & ~31) + 8 * (token & 3) + (token >> 2 & 7);
}
__host__ __device__ constexpr int token_of(int slot) {
  return (slot & ~31) + 4 * (slot & 7) + (slot >> 3 & 3);
}
constexpr int kPrep = 512;         // threads of a prep CTA
constexpr int kConv = 512;         // threads that run the convolution of x

// What the kernels hand to one another, in the workspace.
struct TcBufs {
  int nb;                          // blocks per row
  unsigned char *bhi, *blo;        // [B][nb][G] tiles (slot, state), op_off(slot, n, N): B
                                   // in two scaled fp16 parts, for the state
  unsigned char *bt, *ct;          // likewise B and C in bf16, for y
  unsigned char *xt;               // [B][nb][H] tiles of x in scaled fp16, mn_off(p, slot, 128)
  int xch;                         // channels that share a scale of x
  float *xinv;                     // [B][nb][H][P / xch]: what 1 in xt stands for
  unsigned char *st;               // [B][nb][H] tiles of entering states, mn_off(p, n, N)
  unsigned char *btlo, *clo, *xlo, *slo;  // fp32 inputs: the second parts of bt, ct, xt, st
  unsigned char *bt3, *c3;                // and the third of bt and ct
  unsigned char *bexp;             // [B][nb][G][N]: the exponent (as in a float) of what 1 in
                                   // bhi and blo stands for
  float *ein, *cum, *cumj;         // [B][H][nb * 128] by slot, see prep_factors
  float *cum_lo, *cumj_lo;         // fp32 inputs: what cum and cumj leave of the sums
  float *wst;                      // likewise, by token
  float *dlog;                     // [B][H][nb]: a whole log2 above the finite d
  float4 *dec;                     // [B][H][nb]: e^{c_127}, or -1: the block resets the state;
                                   // what 1 in wst stands for; 0, 0
  int *run;                        // [B][nb * 128] by slot: resets so far in the block, -1: padding
  unsigned char *tok;              // [B][nb * 128] by token: token_mark
  int *flags;                      // [B][nb]: kPlain, kResets
  uint32_t *status;
};
// flags of a block
constexpr int kPlain = 1;          // every token has its whole window in the staged rows
constexpr int kResets = 2;         // a run that is not the row's first starts in it

size_t layout_bufs(const SsmParams &p, bool f32, unsigned char *base, TcBufs *t) {
  const int nb = (p.T + kQ - 1) / kQ;
  const size_t bt = (size_t)p.B * nb, toks = bt * kQ;
  size_t off = 0;
  auto take = [&](size_t n) {
    unsigned char *q = base + off;
    off += align_up(n, 256);
    return q;
  };
  t->nb = nb;
  t->bhi = take(bt * p.G * kQ * p.N * 2);
  t->blo = take(bt * p.G * kQ * p.N * 2);
  t->bt = take(bt * p.G * kQ * p.N * 2);
  t->ct = take(bt * p.G * kQ * p.N * 2);
  t->bexp = take(bt * p.G * p.N);
  t->xt = take(bt * p.H * kQ * p.P * 2);
  t->xinv = (float *)take(bt * p.H * p.P * 2);
  t->st = take(bt * p.H * p.N * p.P * 2);
  t->btlo = take(f32 ? bt * p.G * kQ * p.N * 2 : 0);
  t->bt3 = take(f32 ? bt * p.G * kQ * p.N * 2 : 0);
  t->c3 = take(f32 ? bt * p.G * kQ * p.N * 2 : 0);
  t->clo = take(f32 ? bt * p.G * kQ * p.N * 2 : 0);
  t->xlo = take(f32 ? bt * p.H * kQ * p.P * 2 : 0);
  t->slo = take(f32 ? bt * p.H * p.N * p.P * 2 : 0);
  t->cum_lo = (float *)take(f32 ? toks * p.H * 4 : 0);
  t->cumj_lo = (float *)take(f32 ? toks * p.H * 4 : 0);
  t->ein = (float *)take(toks * p.H * 4);
  t->wst = (float *)take(toks * p.H * 4);
  t->cum = (float *)take(toks * p.H * 4);
  t->cumj = (float *)take(toks * p.H * 4);
  t->dlog = (float *)take(bt * p.H * 4);
  t->dec = (float4 *)take(bt * p.H * 16);
  t->run = (int *)take(toks * 4);
  t->tok = take(toks);
  t->flags = (int *)take(bt * 4);
  return off;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^k with `bound` / 2^k in [2^14, 2^15), as far as 2^k and its inverse are normal.
__device__ __forceinline__ float to_2p15(float bound) {
  const int e = (int)(__float_as_uint(bound) >> 23 & 255u) - 14;
  return __uint_as_float((uint32_t)min(max(e, 14), 240) << 23);
}

// ---------------------------------------------------------------------------
// The convolution of a tile of TP channels x 128 tokens by NT threads.  The
// tile's rows and the 3 before it are staged by cp.async; a warp owns CH
// channels and a lane 4 consecutive tokens.  Channels are kept in pairs for
// the packed arithmetic.
template <int BYTES>
using Word = typename std::conditional<
    BYTES == 16, uint4, typename std::conditional<BYTES == 8, uint2, uint32_t>::type>::type;

template <typename T, int TP, int CH, int NT>
struct Conv {
  static_assert(TP / CH * 32 == NT, "one warp per CH channels");
  static_assert(TP * sizeof(T) == 128 || TP * sizeof(T) == 64, "row bytes");
  static constexpr int E = CH / 2;                         // pairs of channels per lane
  static constexpr int kStrip = 4;
  static constexpr int kRows = kQ + kSsmTaps - 1;
  static constexpr uint32_t kRowBytes = TP * sizeof(T);
  static constexpr uint32_t kPad = kRowBytes == 128 ? 0 : 4;       // bytes per row, off()
  static constexpr uint32_t kBytes = kRows * kRowBytes + (kRows + 3) / 4 * 4 * kPad;
  using Raw = Word<CH * sizeof(T)>;

  // The lanes of a warp read rows 4 apart: rows of 128 bytes are permuted in
  // 16-byte pieces by the row's strip, strips of 64-byte rows lie 16 bytes
  // further apart than their rows fill (either way over 8 places of 16
  // bytes; over 4, the packed row of 32 heads took 7 us longer).
  static __device__ __forceinline__ uint32_t off(int row, int piece16) {
    return kRowBytes == 128
               ? (uint32_t)(row * 128 + ((piece16 ^ (row >> 2 & 7)) << 4))
               : (uint32_t)(row * 64 + (row >> 2) * 16 + (piece16 << 4));
  }
  static __device__ __forceinline__ void unpack(const Raw &a, u64 (&x)[E]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(&a);
#pragma unroll
    for (int i = 0; i < E; ++i)
      x[i] = sizeof(T) == 4
                 ? pk2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]))
                 : pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }

  // A warp's bound on its values and its bias, in shared memory: with 64 columns the
  // state kernel has no register left for them, and with all of the SM's shared
  // memory taken a spilled one comes from L2 (2 x 8192 tokens: 158 us, with
  // seven of them spilled 167).  Two channels keep their bias.
  struct Consts {
    float2 bound;        // |u| <= bound.x max|x| + bound.y
    float bias[CH];
  };
  static constexpr bool kKeep = E == 1;
  u64 wt[kSsmTaps][E], kept;

  // Loads the weights; lane 0 writes *c, to be read after a barrier.
  __device__ __forceinline__ void weights(const SsmParams &p, int channel, int lane, Consts *c) {
    float gain = 0.f, base = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float4 a = *reinterpret_cast<const float4 *>(p.w + 4 * (size_t)(channel + 2 * i));
      const float4 b = *reinterpret_cast<const float4 *>(p.w + 4 * (size_t)(channel + 2 * i + 1));
      wt[0][i] = pk2(a.x, b.x);
      wt[1][i] = pk2(a.y, b.y);
      wt[2][i] = pk2(a.z, b.z);
      wt[3][i] = pk2(a.w, b.w);
      const float b0 = p.bias ? p.bias[channel + 2 * i] : 0.f,
                  b1 = p.bias ? p.bias[channel + 2 * i + 1] : 0.f;
      if (kKeep) kept = pk2(b0, b1);
      else if (lane == 0) c->bias[2 * i] = b0, c->bias[2 * i + 1] = b1;
      gain = fmaxf(gain, fmaxf(fabsf(a.x) + fabsf(a.y) + fabsf(a.z) + fabsf(a.w),
                               fabsf(b.x) + fabsf(b.y) + fabsf(b.z) + fabsf(b.w)));
      base = fmaxf(base, fmaxf(fabsf(b0), fabsf(b1)));
    }
    if (lane == 0) c->bound = make_float2(gain, base);
  }

  // x: the row's token 0 at the tile's channel; past: the convolution's cache
  // there, or null (zeros).  The rows before the row's first run (from token
  // `first` on) are outside the row or padding, which nothing reads: they
  // are staged from the cache, so that the first run's windows are whole.
  // A thread copies one 16-byte piece of every kStep-th row.
  static __device__ __forceinline__ void stage(uint32_t dst, const T *x, long long st,
                                               const T *past, int channels, int t0, int len,
                                               int first, int tid) {
    constexpr int kP16 = kRowBytes / 16, kStep = NT / kP16, kEl = 16 / sizeof(T);
    static_assert(kStep % 32 == 0, "the rows of a thread are permuted alike");
    const int piece = tid % kP16, row0 = tid / kP16;
    const T *src = x + (long long)(t0 - (kSsmTaps - 1) + row0) * st + piece * kEl;
    dst += off(row0, piece);
    if (t0 - (kSsmTaps - 1) >= first && t0 + kQ <= len) {       // every row is there
#pragma unroll
      for (int k = 0; k < (kRows + kStep - 1) / kStep; ++k, src += (long long)kStep * st)
        if ((k + 1) * kStep <= kRows || row0 + k * kStep < kRows)
          cp_async16(dst + k * kStep * (kRowBytes + kPad), src);
    } else {
#pragma unroll 1
      for (int k = 0; k < (kRows + kStep - 1) / kStep; ++k, src += (long long)kStep * st) {
        const int row = row0 + k * kStep, t = t0 - (kSsmTaps - 1) + row;
        if (row < kRows) {
          bool ok = t >= first && t < len;
          const T *from = ok ? src : x;
          if (t < first && past && t >= first - (kSsmTaps - 1)) {
            from = past + (size_t)(kSsmTaps - 1 + t - first) * channels + piece * kEl;
            ok = true;
          }
          cp_async16(dst + k * kStep * (kRowBytes + kPad), from, ok);
        }
      }
    }
    cp_async_commit();
  }

  // f(i, u, inv): u inv = SiLU(conv) of channels [CH warp, CH (warp + 1)) of the
  // tile at the lane's i-th token, 4 lane + i.  CUT: windows end where a run
  // starts, and padding gives 0; tok holds the tokens' windows.
  //
  // inv is 1, or with `scaled` a power of two that keeps |u| of the warp's channels
  // and the block's tokens below 2^15, by the largest finite input: what u is in
  // fp16 then has 11 bits, and two parts of it 22, down to 2^-29 of the largest.
  // The scale costs no instruction per value (1 / (1 + e) is made with it).
  // Returns inv.
  template <bool CUT, typename F>
  __device__ __forceinline__ float run(const unsigned char *rows, int warp, int lane,
                                       const unsigned char *tok, const Consts *c,
                                       bool scaled, F f) const {
    const int at = warp * CH * (int)sizeof(T);
    // rows 4 lane .. 4 lane + 6: two permutations
    const unsigned char *lo = rows + off(4 * lane, at / 16) + at % 16;
    const unsigned char *hi = rows + off(4 * lane + 4, at / 16) + at % 16;
    const uint32_t marks = CUT ? *reinterpret_cast<const uint32_t *>(tok + 4 * lane) : 0;
    uint32_t live = 0x7f;                 // rows that a token's window holds
    if (CUT && scaled) {
      live = 0;
#pragma unroll
      for (int i = 0; i < kStrip; ++i) {
        const int k = marks >> (8 * i), place = k & 3;
        if (k & 8) live |= ((2u << place) - 1) << (i + 3 - place);
      }
    }
    u64 x[kStrip + kSsmTaps - 1][E];
    uint32_t top = 0, top2 = 0;           // of |x|: a float's bits, or two bf16
#pragma unroll
    for (int i = 0; i < kStrip + kSsmTaps - 1; ++i) {
      const Raw r =
          *reinterpret_cast<const Raw *>(i < 4 ? lo + i * kRowBytes : hi + (i - 4) * kRowBytes);
      unpack(r, x[i]);
      if (scaled && (live >> i & 1)) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&r);
        constexpr int kWords = (int)sizeof(Raw) / 4;
#pragma unroll
        for (int e = 0; e < kWords; e += 2) {
          top = larger(top, w[e]);
          if (e + 1 < kWords) top2 = larger(top2, w[e + 1]);
        }
      }
    }
    const float inv = scaled ? fit(larger(top, top2), lo, hi, live, c->bound) : 1.f;
    const uint32_t bias = smem_u32(c->bias);
    const u64 one = pk2(inv, inv);
#pragma unroll
    for (int i = 0; i < kStrip; ++i) {
      u64 u[E];
      if (CUT) {
        const int k = marks >> (8 * i), place = k & 3;
        u64 a[3][E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          a[0][e] = place >= 3 ? x[i][e] : 0;        // (0 is a pair of zeros)
          a[1][e] = place >= 2 ? x[i + 1][e] : 0;
          a[2][e] = place >= 1 ? x[i + 2][e] : 0;
        }
        taps(a[0], a[1], a[2], x[i + 3], bias, one, u);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] = k & 8 ? u[e] : 0;
      } else {
        taps(x[i], x[i + 1], x[i + 2], x[i + 3], bias, one, u);
      }
      f(i, u, inv);
    }
    return inv;
  }

 private:
  // inv for the largest |x| of the warp: top, or where that is not finite what the
  // live rows hold.
  __device__ __forceinline__ float fit(uint32_t top, const unsigned char *lo,
                                       const unsigned char *hi, uint32_t live,
                                       float2 bound) const {
    if (sizeof(T) == 2) top = max(top << 16, top & 0xffff0000u);
    top = __reduce_max_sync(0xffffffffu, top);
    if (top >= 0x7f800000u) {
      top = 0;
#pragma unroll 1
      for (int i = 0; i < kStrip + kSsmTaps - 1; ++i) {
        u64 x[E];
        unpack(*reinterpret_cast<const Raw *>(i < 4 ? lo + i * kRowBytes : hi + (i - 4) * kRowBytes),
               x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t a = (uint32_t)x[e] & 0x7fffffffu, b = (uint32_t)(x[e] >> 32) & 0x7fffffffu;
          if (live >> i & 1)
            top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
    }
    return to_2p15(fmaf(bound.x, __uint_as_float(top), bound.y));
  }
  // The larger magnitudes: bits of a float, or two bf16.  NaN loses or comes out
  // above every number.
  static __device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t w) {
    if (sizeof(T) == 4) return max(m, w & 0x7fffffffu);
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&m),
                                     __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w)));
    return *reinterpret_cast<const uint32_t *>(&r);
  }
  __device__ __forceinline__ void taps(const u64 (&a)[E], const u64 (&b)[E], const u64 (&c)[E],
                                       const u64 (&x)[E], uint32_t bias, u64 one,
                                       u64 (&u)[E]) const {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      u64 v = kept;
      if (!kKeep)    // (volatile: read for each token)
        asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(bias + 8 * i));
      v = fma2(wt[0][i], a[i], fma2(wt[1][i], b[i], fma2(wt[2][i], c[i], fma2(wt[3][i], x[i], v))));
      float e0, e1, d0, d1;
      upk2(mul2(v, pk2(-kLog2e, -kLog2e)), e0, e1);
      upk2(fma2(pk2(ex2(e0), ex2(e1)), one, one), d0, d1);
      u[i] = mul2(v, pk2(rcp(d0), rcp(d1)));
    }
  }
};

using Unpack8 = Conv<bf16, 64, 8, 256>;      // for its unpack

// Pairs as bf16 (R: uint4 or uint2), and v less what such a part holds.
template <typename R, int E>
__device__ __forceinline__ R pack(const u64 (&v)[E]) {
  R r;
  uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    float a, b;
    upk2(v[i], a, b);
    w[i] = pack_bf16(a, b);
  }
  return r;
}
template <typename R, int E>
__device__ __forceinline__ void less(const R &part, u64 (&v)[E]) {
  const uint32_t *h = reinterpret_cast<const uint32_t *>(&part);
#pragma unroll
  for (int i = 0; i < E; ++i)
    v[i] = fma2(pk2(__uint_as_float(h[i] << 16), __uint_as_float(h[i] & 0xffff0000u)),
                pk2(-1.f, -1.f), v[i]);
}

// Pairs as two parts in fp16.
template <typename R, int E>
__device__ __forceinline__ void split16(const u64 (&v)[E], R &hi, R &lo) {
  __half2 *h = reinterpret_cast<__half2 *>(&hi), *l = reinterpret_cast<__half2 *>(&lo);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    float a, b;
    upk2(v[i], a, b);
    h[i] = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h[i]);
    upk2(fma2(pk2(f.x, f.y), pk2(-1.f, -1.f), v[i]), a, b);
    l[i] = __floats2half2_rn(a, b);
  }
}
template <typename R, int E>
__device__ __forceinline__ R pack16(const u64 (&v)[E]) {
  R r;
  __half2 *h = reinterpret_cast<__half2 *>(&r);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    float a, b;
    upk2(v[i], a, b);
    h[i] = __floats2half2_rn(a, b);
  }
  return r;
}
__device__ __forceinline__ void unpack16(const uint4 &a, u64 (&x)[4]) {
  const __half2 *h = reinterpret_cast<const __half2 *>(&a);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[i] = pk2(f.x, f.y);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                    pack_bf16(v[6], v[7]));
}

// What `hi` leaves of the values.
__device__ __forceinline__ void rest8(const uint4 &hi, float (&v)[8]) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] -= __uint_as_float(h[i] << 16);
    v[2 * i + 1] -= __uint_as_float(h[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ SsmRow row_of(const SsmParams &p, int b) {
  if (p.segment_ids) return p.rows[b];
  SsmRow r = {0, p.T, p.T - 1, 0};
  return r;
}
template <typename T>
__device__ __forceinline__ const T *past_of(const SsmParams &p, int b) {
  return p.conv_state ? static_cast<const T *>(p.conv_state) +
                            (size_t)b * (kSsmTaps - 1) * p.channels
                      : nullptr;
}

// Token t's window in the staged rows: how many tokens of its run precede it
// there (all 3 in the row's first run, see Conv::stage), whether it counts.
__device__ __forceinline__ unsigned char token_mark(const SsmToken &k) {
  return (unsigned char)((k.first ? kSsmTaps - 1 : k.place) | (k.live ? 8 : 0));
}
constexpr unsigned char kWhole = (kSsmTaps - 1) | 8;

// ---------------------------------------------------------------------------
// 1. prep

struct Two {       // hi + lo, |lo| at most half a step of hi
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}

// Per token and head of a block, a = d A log2(e):
//   cum  = sum of a up to the token            cumj = cum - log2 d
//   ein  = 2^cum where the entering state reaches the token, else 0
//   wst  = d 2^(sum of a after the token) where the token reaches the state
//          that leaves the block, else -0 (summed from the end: exact where
//          it matters); over a power of two that leaves the largest below 1
// A warp takes a head, a lane 4 tokens.  For fp32 inputs the sums up to a token
// are made and kept in two floats: a factor e^(c_r - c_j) is as exact as the
// difference, however far the sums have run.  (64-bit sums took 40 us.)  For bf16
// inputs they are kept in one, so c_r - c_j is off by a step of the sum or a few:
// 6e-5 each at kWide.  Beyond it the sums are made in two floats and rounded
// once, and a token's a counts down to kFar only: the sum stays above -2^15, one
// step is 2^-9 and a factor, of three sums rounded so, off by 2e-3 at most, half a
// step of bf16.
// The largest finite width of four.
__device__ __forceinline__ float finite_max(const float4 &w) {
  auto in = [](float v) { return v > 0.f && v < CUDART_INF_F ? v : 0.f; };
  return fmaxf(fmaxf(in(w.x), in(w.y)), fmaxf(in(w.z), in(w.w)));
}

constexpr float kFar = -256.f;     // 2^kFar is 0 beside any fp32 value, as 2^a below it is
constexpr float kWide = 1024.f;
template <typename T>
__device__ __forceinline__ void prep_factors(const SsmParams &p, const TcBufs &t, int b, int blk,
                                             unsigned char *smem) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blk * kQ;
  const int32_t *ids = p.segment_ids ? p.segment_ids + (size_t)b * p.T : nullptr;
  int *srun = reinterpret_cast<int *>(smem);                   // [128]
  int *scount = srun + kQ;                                     // resets per warp
  float *sdt = reinterpret_cast<float *>(scount + 8);          // [128][33]
  const SsmRow row = row_of(p, b);
  int n = 0, plain = 1;
  SsmToken k = {};
  if (tid < kQ) {
    k = ssm_token(ids, t0 + tid, p.T, row);
    const unsigned m = __ballot_sync(0xffffffffu, k.reset);
    n = __popc(m & (0xffffffffu >> (31 - lane)));
    if (lane == 0) scount[warp] = __popc(m);
    plain = t0 + tid >= p.T || token_mark(k) == kWhole;
  }
  plain = __syncthreads_and(plain);
  if (tid < kQ) {
    for (int w = 0; w < warp; ++w) n += scount[w];
    srun[tid] = n;
    const size_t at = (size_t)b * t.nb * kQ + t0 + tid;
    t.run[at - tid + slot_of(tid)] = k.live ? n : -1;
    t.tok[at] = token_mark(k);
  }
  if (tid == 0) {
    const int resets = scount[0] + scount[1] + scount[2] + scount[3];
    t.flags[(size_t)b * t.nb + blk] = (plain ? kPlain : 0) | (resets ? kResets : 0);
  }
  constexpr bool kF32 = sizeof(T) == 4;
  const T *dt = static_cast<const T *>(p.dt) + (size_t)b * p.dt_sb;
  for (int h0 = 0; h0 < p.H; h0 += 32) {
    const int nh = min(32, p.H - h0);
    __syncthreads();
    for (int i = tid; i < kQ * 32; i += blockDim.x) {
      const int tt = i >> 5, hh = i & 31;
      float d = 0.f;
      if (hh < nh && t0 + tt < p.T && ssm_id(ids, t0 + tt, p.T) != 0)
        d = ssm_softplus(to_f32(dt[(long long)(t0 + tt) * p.dt_st + h0 + hh]) +
                         (p.dt_bias ? p.dt_bias[h0 + hh] : 0.f));
      sdt[tt * 33 + hh] = d;
    }
    __syncthreads();
    for (int hh = warp; hh < nh; hh += kPrep / 32) {
      // A log2(e) in two floats
      const float A = p.A[h0 + hh], a2 = A * kLog2e;
      const float a2_lo = fmaf(A, kLog2e, -a2) + A * 1.9259629911266175e-8f;
      float d[4], suf[4];
      Two a[4], pre[4], before;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i] = sdt[(lane * 4 + i) * 33 + hh];
        // a width that is not finite reaches its run's tokens by cumj and wst; in
        // the sums it would reach every token after it
        const float f = d[i] * a2;
        const bool in = d[i] > 0.f && d[i] < CUDART_INF_F, far = f < kFar;
        a[i].hi = !in ? 0.f : far ? kFar : f;
        a[i].lo = kF32 && in && !far ? fmaf(d[i], a2, -f) + d[i] * a2_lo : 0.f;
      }
      float total;
      auto prefix = [&](auto two) {      // pre: in the lane; before: the lanes before
        constexpr bool k2 = decltype(two)::value;
        auto plus = [](Two u, Two v) { return k2 ? add(u, v) : Two{u.hi + v.hi, 0.f}; };
        pre[0] = a[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) pre[i] = plus(pre[i - 1], a[i]);
        before = pre[3];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          Two u = {__shfl_up_sync(0xffffffffu, before.hi, o), 0.f};
          if (k2) u.lo = __shfl_up_sync(0xffffffffu, before.lo, o);
          if (lane >= o) before = plus(before, u);
        }
        total = __shfl_sync(0xffffffffu, before.hi, 31);
        before.hi = __shfl_up_sync(0xffffffffu, before.hi, 1);
        if (k2) before.lo = __shfl_up_sync(0xffffffffu, before.lo, 1);
        if (lane == 0) before = {0.f, 0.f};
      };
      prefix(std::integral_constant<bool, kF32>{});
      const bool wide = !kF32 && total < -kWide;
      if (wide) prefix(std::true_type{});
      suf[3] = 0.f;
#pragma unroll
      for (int i = 2; i >= 0; --i) suf[i] = suf[i + 1] + a[i + 1].hi;
      float after = pre[3].hi;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float v = __shfl_down_sync(0xffffffffu, after, o);
        if (lane + o < 32) after += v;
      }
      after = __shfl_down_sync(0xffffffffu, after, 1);
      if (lane == 31) after = 0.f;
      const int last = srun[kQ - 1];
      const size_t at = (((size_t)b * p.H + h0 + hh) * t.nb + blk) * kQ;
      float4 wst;
      float *fw = &wst.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int run = srun[lane * 4 + i];
        const size_t s = at + slot_of(lane * 4 + i);
        const float l = log2f(d[i]);           // d = 0: -inf, a factor of 0
        if (kF32 || wide) {
          const Two c = add(before, pre[i]), j = two_sum(c.hi, -l);
          const float rest = j.lo + c.lo;
          t.ein[s] = run == 0 ? exp2f(c.hi) : 0.f;
          t.cum[s] = c.hi;
          t.cumj[s] = d[i] == 0.f ? CUDART_INF_F : kF32 ? j.hi : j.hi + rest;
          if (kF32) {
            t.cum_lo[s] = c.lo;
            t.cumj_lo[s] = d[i] == 0.f ? 0.f : rest;
          }
        } else {
          const float c = before.hi + pre[i].hi;
          t.ein[s] = run == 0 ? exp2f(c) : 0.f;
          t.cum[s] = c;
          t.cumj[s] = c - l;
        }
        fw[i] = run == last ? d[i] * exp2f(suf[i] + after) : -0.f;
      }
      const float winv = 32768.f * to_2p15(__uint_as_float(__reduce_max_sync(
                                       0xffffffffu, __float_as_uint(finite_max(wst)))));
      const float scale = __uint_as_float((254u << 23) - __float_as_uint(winv));
      *reinterpret_cast<float4 *>(t.wst + at + lane * 4) =
          make_float4(wst.x * scale, wst.y * scale, wst.z * scale, wst.w * scale);
      const uint32_t widest = __reduce_max_sync(
          0xffffffffu, __float_as_uint(finite_max(make_float4(d[0], d[1], d[2], d[3]))));
      if (lane == 0) {
        const size_t o = ((size_t)b * p.H + h0 + hh) * t.nb + blk;
        t.dec[o] = make_float4(last == 0 ? exp2f(total) : -1.f, winv, 0.f, 0.f);
        t.dlog[o] = (float)((int)(widest >> 23) - 126);
      }
    }
  }
}

// Channels per warp in prep: 8 bytes of them.
template <typename T>
constexpr int kPrepCh = 8 / (int)sizeof(T);
template <typename T, int TP>
using PrepConv = Conv<T, TP, kPrepCh<T>, TP / kPrepCh<T> * 32>;

// The convolution of TP channels of B or C of the blocks [blk, end) into their
// operand tiles, the next block's rows on their way.
template <typename T, int TP, bool is_c>
__device__ __forceinline__ void prep_conv(const SsmParams &p, const TcBufs &t, int b, int blk,
                                          int end, int g, int part, unsigned char *smem) {
  const int tid = threadIdx.x;
  const int n0 = part * TP;
  const int ch = p.H * p.P + (is_c ? p.G * p.N : 0) + g * p.N + n0;
  const SsmRow row = row_of(p, b);
  const T *past = past_of<T>(p, b);
  const T *x = static_cast<const T *>(p.xbc) + (size_t)b * p.xbc_sb + ch;
  using Cv = PrepConv<T, TP>;
  using Out = Word<2 * kPrepCh<T>>;
  const int warp = tid >> 5, lane = tid & 31, wch = warp * kPrepCh<T>;
  const bool mine = warp < TP / kPrepCh<T>;   // 32 bf16 channels take half the warps
  auto stage = [&](int i) {
    if (mine && i < end)
      Cv::stage(smem_u32(smem) + (i & 1) * Cv::kBytes, x, p.xbc_st, past ? past + ch : nullptr,
                p.channels, i * kQ, p.T, row.first, tid);
  };
  stage(blk);
  Cv cv;
  auto *consts = reinterpret_cast<typename Cv::Consts *>(smem + 2 * (Cv::kBytes + kQ)) + warp;
  if (mine) cv.weights(p, ch + wch, lane, consts);
  for (; blk < end; ++blk) {
    // whether any token's window leaves the staged rows
    unsigned char *stok = smem + 2 * Cv::kBytes + (blk & 1) * kQ;
    int plain = 1;
    if (p.segment_ids && tid < kQ) {
      const int at = blk * kQ + tid;
      stok[tid] = token_mark(ssm_token(p.segment_ids + (size_t)b * p.T, at, p.T, row));
      plain = at >= p.T || stok[tid] == kWhole;
    }
    cp_async_wait_all();
    plain = __syncthreads_and(plain);
    stage(blk + 1);
    if (!mine) continue;
    // the lane's i-th token: row 8 i + lane % 8 of quarter lane / 8
    const size_t tile = (((size_t)b * t.nb + blk) * p.G + g) * kQ * p.N * 2 +
                        (size_t)(lane >> 3) * 4 * p.N * 16 + (lane & 7) * 16 +
                        (n0 + wch) / 8 * 128 + wch % 8 * 2;
    auto put = [&](int i, u64(&u)[Cv::E], float inv) {
      const size_t o = tile + (size_t)i * p.N * 16;
      Out hi, lo;
      if (!is_c) {
        split16(u, hi, lo);
        *reinterpret_cast<Out *>(t.bhi + o) = hi;
        *reinterpret_cast<Out *>(t.blo + o) = lo;
#pragma unroll
        for (int e = 0; e < Cv::E; ++e) u[e] = mul2(u[e], pk2(inv, inv));
      }
      hi = pack<Out>(u);
      *reinterpret_cast<Out *>((is_c ? t.ct : t.bt) + o) = hi;
      if (sizeof(T) == 4) {
        less(hi, u);
        lo = pack<Out>(u);
        *reinterpret_cast<Out *>((is_c ? t.clo : t.btlo) + o) = lo;
        less(lo, u);
        *reinterpret_cast<Out *>((is_c ? t.c3 : t.bt3) + o) = pack<Out>(u);
      }
    };
    const unsigned char *rows = smem + (blk & 1) * Cv::kBytes;
    const float inv =
        plain ? cv.template run<false>(rows, warp, lane, stok, consts, !is_c, put)
              : cv.template run<true>(rows, warp, lane, stok, consts, !is_c, put);
    if (!is_c && lane < kPrepCh<T>)
      t.bexp[(((size_t)b * t.nb + blk) * p.G + g) * p.N + n0 + wch + lane] =
          (unsigned char)(__float_as_uint(inv) >> 23);
  }
}

// The inputs that the convolution's cache holds after the row.
template <typename T>
__device__ __forceinline__ void prep_cache(const SsmParams &p, int b, int part) {
  const SsmRow row = row_of(p, b);
  const T *x = static_cast<const T *>(p.xbc) + (size_t)b * p.xbc_sb, *past = past_of<T>(p, b);
  SsmToken k = ssm_token(p.segment_ids ? p.segment_ids + (size_t)b * p.T : nullptr, row.last, p.T,
                         row);
  const int c = part * kPrep + threadIdx.x;
  if (c >= p.channels) return;
  T *out = static_cast<T *>(p.conv_out) + (size_t)b * (kSsmTaps - 1) * p.channels + c;
#pragma unroll
  for (int i = 0; i < kSsmTaps - 1; ++i)
    out[(size_t)i * p.channels] = ssm_cached(x, p.xbc_st, past, p.channels, c, i, row.last, k);
}

// CTAs [0, B nb) make the factors, the next ones the tiles of B or C of `run`
// blocks each, the last ones the convolution's cache.
template <typename T, int TP>
__global__ void __launch_bounds__(kPrep, 2)
    ssm_prep_kernel(const SsmParams p, const TcBufs t, int run) {
  extern __shared__ __align__(128) unsigned char smem[];
  start_next();
  after_previous();      // the row table
  int u = blockIdx.x;
  if (u < p.B * t.nb) {
    prep_factors<T>(p, t, u / t.nb, u % t.nb, smem);
    return;
  }
  u -= p.B * t.nb;
  const int runs = (t.nb + run - 1) / run, parts = 2 * p.N / TP, tiles = p.B * runs * p.G * parts;
  if (u < tiles) {
    const int part = u % parts;
    u /= parts;
    const int g = u % p.G;
    u /= p.G;
    const int blk = u % runs * run;
    if (part < p.N / TP)
      prep_conv<T, TP, false>(p, t, u / runs, blk, min(blk + run, t.nb), g, part, smem);
    else
      prep_conv<T, TP, true>(p, t, u / runs, blk, min(blk + run, t.nb), g, part - p.N / TP, smem);
    return;
  }
  u -= tiles;
  const int caches = (p.channels + kPrep - 1) / kPrep;
  prep_cache<T>(p, u / caches, u % caches);
}

// ---------------------------------------------------------------------------
// 2. states

// Barrier of the convolving threads; whether any of them says so.
__device__ __forceinline__ bool any_of_conv(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kConv)
      : "memory");
  return r != 0;
}

// Shared memory of ssm_state_kernel.
template <typename T, int TP>
struct StateSmem {
  using Cv = Conv<T, TP, TP / 16, kConv>;
  static constexpr uint32_t kX = 0;                                 // 2 x [hi | lo] tiles
  static constexpr uint32_t kXBytes = kQ * TP * 2 * 2;
  static constexpr uint32_t kB = kX + 2 * kXBytes;                  // 2 x (hi, lo) tiles
  static constexpr uint32_t kBBytes = 2 * kQ * 128 * 2;
  static constexpr uint32_t kRows = kB + 2 * kBBytes;               // 2 staged tiles of x
  static constexpr uint32_t kW = kRows + 2 * Cv::kBytes;      // 2 x wst
  static constexpr uint32_t kXinv = kW + 2 * kQ * 4;          // 4 x [16]: 1 in kX, by warp
  static constexpr uint32_t kBexp = kXinv + 4 * 16 * 4;       // 4 x [128]: bexp
  static constexpr uint32_t kDec = kBexp + 4 * 128;           // 4 x dec
  static constexpr uint32_t kConsts = kDec + 4 * 16;          // by warp
  static constexpr uint32_t kBar = kConsts + 16 * sizeof(typename Cv::Consts);
  static constexpr uint32_t kTmem = kBar + 48;
  static constexpr uint32_t kBytes = kTmem + 16;
  static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
};

// Whether a token's wst says that its run ends before the block does.
__device__ __forceinline__ bool ends_before(float wst) {
  return __float_as_uint(wst) == 0x80000000u;
}

// What the tokens that reach the state (f: wst, by token) add to row n of it in
// the columns of the operand tile at x, in place of the products.
template <int TP, int COLS>
__device__ __forceinline__ void tokens_of_state(const unsigned char *x, const unsigned char *bhi,
                                                const unsigned char *blo, const float *f, int n,
                                                int N, float (&add)[COLS]) {
#pragma unroll
  for (int k = 0; k < COLS; ++k) add[k] = 0.f;
#pragma unroll 1
  for (int j = 0; j < kQ; ++j) {
    if (ends_before(f[token_of(j)])) continue;
    const uint32_t o = op_off(j, n, N);
    const float b = __half2float(*reinterpret_cast<const __half *>(bhi + o)) +
                    __half2float(*reinterpret_cast<const __half *>(blo + o));
#pragma unroll
    for (int k = 0; k < COLS; ++k) {
      const unsigned char *v = x + mn_off(k, j, kQ);
      add[k] = fmaf(b, __half2float(*reinterpret_cast<const __half *>(v)) +
                           __half2float(*reinterpret_cast<const __half *>(v + TP / 8 * 2048)),
                    add[k]);
    }
  }
}

// 512 threads run the convolution, keep S and write it; one more warp copies
// the tiles of B and issues the products.  Per block i the threads
//   convolve x into the operand buffer i % 2 while the products of block
//   i - 1 run, then wait for those, write the S that entered block i - 1 and
//   update it.
// A thread holds TP / 4 columns of one state row (its TMEM lane).  (With 256
// threads, two warps on a scheduler, a block took 3.7 us instead of 2.2.)
// IDS: rows have segment ids (without them every block is plain, and the
// kernel keeps its registers).
template <typename T, int TP, bool IDS>
__global__ void __launch_bounds__(kConv + 32, 1)
    ssm_state_kernel(const SsmParams p, const TcBufs t) {
  using L = StateSmem<T, TP>;
  using Cv = typename L::Cv;
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kCols = TP / 4;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar_x = sb + L::kBar, bar_b = bar_x + 16, bar_d = bar_x + 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = p.P / TP, tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int h = bh % p.H, b = bh / p.H, g = h / (p.H / p.G), c0 = tile * TP;
  const int nb = t.nb, N = p.N;
  if (warp == 0) tmem_alloc(sb + L::kTmem, 4 * TP);
  if (tid == 0) {
    mbar_init(bar_x, kConv);
    mbar_init(bar_x + 8, kConv);
    mbar_init(bar_b, 1);
    mbar_init(bar_b + 8, 1);
    mbar_init(bar_d, 2);           // the products, and that what came with B is there
    mbar_init(bar_d + 8, 2);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kTmem);
  start_next();

  if (warp == kConv / 32) {
    if (lane == 0) {
      after_previous();
      const uint32_t tb = (uint32_t)(kQ * N * 2);
      auto load = [&](int i) {
        const size_t o = (((size_t)b * nb + i) * p.G + g) * tb;
        const uint32_t bar = bar_b + 8u * (i & 1), dst = sb + L::kB + (i & 1) * L::kBBytes;
        mbar_expect_tx(bar, 2 * tb + N + 16);
        bulk_load(dst, t.bhi + o, tb, bar);
        bulk_load(dst + tb, t.blo + o, tb, bar);
        // what finish(i) needs; block i - 4's is read by then (as is its xinv)
        bulk_load(sb + L::kBexp + (i & 3) * 128, t.bexp + (((size_t)b * nb + i) * p.G + g) * N, N,
                  bar);
        bulk_load(sb + L::kDec + (i & 3) * 16, t.dec + ((size_t)b * p.H + h) * nb + i, 16, bar);
      };
      const float4 *xinv = reinterpret_cast<const float4 *>(smem + L::kXinv);
      const int scales = p.P / (TP / 16);          // of a head: P / xch
      float4 *xinv_out =
          reinterpret_cast<float4 *>(t.xinv + ((size_t)b * nb * p.H + h) * scales + tile * 16);
      int loaded = 0, landed = 0, issued = 0, done = 0;
      bool ok = true;
      for (; loaded < 2 && loaded < nb; ++loaded) load(loaded);
      for (int i = 0; i < nb && ok; ++i) {
        ok = mbar_wait(bar_b + 8u * (i & 1), (i >> 1) & 1);
        if (!ok) break;
        ++landed;
        ok = mbar_wait(bar_x + 8u * (i & 1), (i >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (i & 1) * 2 * TP;
        const uint32_t bt = sb + L::kB + (i & 1) * L::kBBytes;
        const Opnd x = {sb + L::kX + (i & 1) * L::kXBytes, 128, kQ * 16};
        const Opnd bh_ = {bt, (uint32_t)N * 16, 128}, bl_ = {bt + tb, (uint32_t)N * 16, 128};
        // the small products first: a sum in the accumulator loses bits at its size
        mma_k<true>(d, bl_, 1, x, 1, kQ / 16, 2 * TP, false);
        mma_k<true>(d, bh_, 1, x, 1, kQ / 16, 2 * TP, true);
        mma_commit(bar_d + 8u * (i & 1));
        mbar_arrive(bar_d + 8u * (i & 1));
        ++issued;
#pragma unroll
        for (int k = 0; k < 4; ++k)      // the scales of x, for ssm_out_kernel
          xinv_out[(size_t)i * p.H * scales / 4 + k] = xinv[(i & 3) * 4 + k];
        if (i > 0 && loaded < nb) {      // block i - 1's tiles are free once it is done
          ok = mbar_wait(bar_d + 8u * ((i - 1) & 1), ((i - 1) >> 1) & 1);
          if (!ok) break;
          ++done;
          load(loaded++);
        }
      }
      if (!ok) set_status(t.status, KDA_DEVICE_TIMEOUT);
      // nothing of this warp's is in flight when it leaves
      for (int i = landed; i < loaded; ++i) mbar_wait(bar_b + 8u * (i & 1), (i >> 1) & 1);
      for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i)
        mbar_wait(bar_d + 8u * (i & 1), (i >> 1) & 1);
    }
    __syncwarp();
  } else {
    const T *past = past_of<T>(p, b);
    const int ch = h * p.P + c0;
    const T *x = static_cast<const T *>(p.xbc) + (size_t)b * p.xbc_sb + ch;
    const T *before = past ? past + ch : nullptr;
    const float *wst = t.wst + ((size_t)b * p.H + h) * nb * kQ;
    Cv cv;
    const int wch = warp * (TP / 16);
    auto *consts = reinterpret_cast<typename Cv::Consts *>(smem + L::kConsts) + warp;
    cv.weights(p, ch + wch, lane, consts);
    const int n = 32 * (warp & 3) + lane, col0 = (warp >> 2) * kCols;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + col0;
    const size_t state = (((size_t)b * p.H + h) * N + n) * p.P + c0 + col0;
    float s[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) s[i] = 0.f;
    if (p.initial_state && n < N) {
#pragma unroll
      for (int i = 0; i < kCols; i += 4)
        *reinterpret_cast<float4 *>(s + i) =
            *reinterpret_cast<const float4 *>(p.initial_state + state + i);
    }
    after_previous();
    const int first = IDS ? p.rows[b].first : 0;
    auto stage = [&](int i) {
      if (i < nb) {
        if (tid < kQ / 4)
          cp_async16(sb + L::kW + (i & 1) * kQ * 4 + tid * 16, wst + (size_t)i * kQ + tid * 4);
        Cv::stage(sb + L::kRows + (i & 1) * Cv::kBytes, x, p.xbc_st, before, p.channels, i * kQ,
                  p.T, first, tid);
      }
    };
    bool bad = false;
    // the state after block i, once its products are done
    auto finish = [&](int i) {
      if (n < N) {
        const size_t at = ((((size_t)b * nb + i) * p.H + h) * N) * p.P * 2 +
                          (size_t)((c0 + col0) / 8) * N * 16 + (n >> 3) * 128 + (n & 7) * 16;
#pragma unroll
        for (int k = 0; k < kCols; k += 8) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = s[k + e];
          const size_t o = at + (size_t)(k / 8) * N * 16;
          const uint4 hi = pack8(v);
          *reinterpret_cast<uint4 *>(t.st + o) = hi;
          if constexpr (kF32) {
            rest8(hi, v);
            *reinterpret_cast<uint4 *>(t.slo + o) = pack8(v);
          }
        }
      }
      if (!mbar_wait(bar_d + 8u * (i & 1), (i >> 1) & 1)) {
        bad = true;
        set_status(t.status, KDA_DEVICE_TIMEOUT);
      }
      tc_fence_after();
      const float2 d = *reinterpret_cast<const float2 *>(smem + L::kDec + (i & 3) * 16);
      const bool drop = IDS && d.x < 0.f;      // a reset drops the state whatever it holds
      const float a = drop ? 0.f : d.x;
      // the columns are those that four warps convolve
      const float4 xi = *reinterpret_cast<const float4 *>(
          smem + L::kXinv + ((i & 3) * 16 + col0 / (TP / 16)) * 4);
      const float bi = d.y * __uint_as_float((uint32_t)smem[L::kBexp + (i & 3) * 128 + (n & (N - 1))]
                                             << 23);
      const float inv[4] = {bi * xi.x, bi * xi.y, bi * xi.z, bi * xi.w};
      // 8 columns at a time: all 16 at once cost the convolution its registers
#pragma unroll
      for (int k0 = 0; k0 < kCols; k0 += 8) {
        uint32_t hi[8], lo[8];
        tmem_ld8_nw(tl + (i & 1) * 2 * TP + k0, hi);
        tmem_ld8_nw(tl + (i & 1) * 2 * TP + TP + k0, lo);
        tmem_wait_ld();
        reg_fence8(hi);
        reg_fence8(lo);
        float add[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) add[k] = __uint_as_float(hi[k]) + __uint_as_float(lo[k]);
        if (drop) {
          // B of a run that ended may be NaN or infinite, which times 0 is NaN: then
          // the tokens that reach the state are added up one by one
          float odd = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            s[k0 + k] = 0.f;
            odd = fmaf(add[k], 0.f, odd);
          }
          if (__any_sync(0xffffffffu, odd != 0.f) && n < N)
            tokens_of_state<TP>(smem + L::kX + (i & 1) * L::kXBytes + (col0 + k0) / 8 * 2048,
                                t.bhi + (((size_t)b * nb + i) * p.G + g) * kQ * N * 2,
                                t.blo + (((size_t)b * nb + i) * p.G + g) * kQ * N * 2,
                                wst + (size_t)i * kQ, n, N, add);
        }
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float v = inv[(k0 + k) / (kCols / 4)];
          const u64 r = fma2(pk2(a, a), pk2(s[k0 + k], s[k0 + k + 1]),
                             mul2(pk2(v, v), pk2(add[k], add[k + 1])));
          upk2(r, s[k0 + k], s[k0 + k + 1]);
        }
      }
      tc_fence_before();
    };
    stage(0);
    // the next block's flags, loaded early
    int flags = IDS ? t.flags[(size_t)b * nb] : kPlain, flags_next = kPlain;
    int i = 0;
    for (; i < nb; ++i, flags = flags_next) {
      cp_async_wait_all();
      if (any_of_conv(bad)) break;   // a wait ran out somewhere: all leave
      stage(i + 1);
      if (IDS) flags_next = i + 1 < nb ? t.flags[(size_t)b * nb + i + 1] : 0;
      const float *w = reinterpret_cast<const float *>(smem + L::kW + (i & 1) * kQ * 4);
      // the lane's i-th token: slot 8 i + lane % 8 of quarter lane / 8
      using Out = Word<2 * (TP / 16)>;
      const uint32_t at = (uint32_t)(wch / 8 * 2048 + wch % 8 * 2 + (lane >> 3) * 512 +
                                     (lane & 7) * 16);
      unsigned char *xo = smem + L::kX + (i & 1) * L::kXBytes + at;
      const size_t xt = (((size_t)b * nb + i) * p.H + h) * kQ * p.P * 2 +
                        (size_t)(c0 / 8) * 2048 + at;
      const float4 w4 = *reinterpret_cast<const float4 *>(w + 4 * lane);
      auto put = [&](int k, u64(&u)[Cv::E], bool cut) {
        Out hi, lo;
        if constexpr (kF32) {
          split16(u, hi, lo);
          *reinterpret_cast<Out *>(t.xlo + xt + k * 128) = lo;
        } else {
          hi = pack16<Out>(u);
        }
        *reinterpret_cast<Out *>(t.xt + xt + k * 128) = hi;
        const float f = k == 0 ? w4.x : k == 1 ? w4.y : k == 2 ? w4.z : w4.w;
#pragma unroll
        for (int e = 0; e < Cv::E; ++e) {
          u[e] = mul2(u[e], pk2(f, f));
          // a token that does not reach the state adds nothing, whatever it holds
          if (cut && ends_before(f)) u[e] = pk2(0.f, 0.f);
        }
        split16(u, hi, lo);
        *reinterpret_cast<Out *>(xo + k * 128) = hi;
        *reinterpret_cast<Out *>(xo + TP / 8 * 2048 + k * 128) = lo;
      };
      const unsigned char *rows = smem + L::kRows + (i & 1) * Cv::kBytes;
      const unsigned char *tok = t.tok + ((size_t)b * nb + i) * kQ;
      const float inv =
          !IDS || (flags & kPlain)
              ? cv.template run<false>(
                    rows, warp, lane, tok, consts, true,
                    [&](int k, u64(&u)[Cv::E], float) { put(k, u, false); })
              : cv.template run<true>(
                    rows, warp, lane, tok, consts, true,
                    [&](int k, u64(&u)[Cv::E], float) { put(k, u, true); });
      if (lane == 0) reinterpret_cast<float *>(smem + L::kXinv)[(i & 3) * 16 + warp] = inv;
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(bar_x + 8u * (i & 1));
      if (i > 0) finish(i - 1);
    }
    cp_async_wait_all();
    if (i == nb) {
      any_of_conv(false);            // what the other threads made of the last block's x
      finish(nb - 1);
    }
    if (p.final_state && n < N) {
#pragma unroll
      for (int k = 0; k < kCols; k += 4)
        *reinterpret_cast<float4 *>(p.final_state + state + k) =
            make_float4(s[k], s[k + 1], s[k + 2], s[k + 3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 4 * TP);
}

// ---------------------------------------------------------------------------
// 3. outputs

// Shared memory of ssm_out_kernel: C; B, then the matrix of factors; x; the
// entering state; z, then y.  With fp32 inputs every operand has a second part
// right after it (C, F at kPart bytes, x and S next to each other as PT more
// columns).
template <typename T, int PT>
struct OutSmem {
  static constexpr uint32_t kParts = sizeof(T) == 4 ? 2 : 1;
  static constexpr uint32_t kPart = kQ * 128 * 2;
  static constexpr uint32_t kC = 0;
  static constexpr uint32_t kF = kC + kParts * kPart;
  static constexpr uint32_t kX = kF + kParts * kPart;
  static constexpr uint32_t kS = kX + kParts * kQ * PT * 2;
  static constexpr uint32_t kZ = kS + kParts * kQ * PT * 2;
  // fp32 inputs: until C B^T is made, the third parts of C and B lie from kX on
  static constexpr uint32_t kThird = kX;
  static constexpr uint32_t kEnd = kZ + kQ * PT * sizeof(T),
                            kFull = kThird + (kParts - 1) * 2 * kPart;
  static constexpr uint32_t kCum = kEnd > kFull ? kEnd : kFull;     // cumj [128]
  static constexpr uint32_t kCumLo = kCum + kQ * 4;                 // its rest, fp32 inputs
  static constexpr uint32_t kRun = kCumLo + (kParts - 1) * kQ * 4;  // runs, one byte each
  static constexpr uint32_t kXinv = kRun + kQ;                      // [PT / 2]: 1 in x
  static constexpr uint32_t kBar = kXinv + PT * 2;
  static constexpr uint32_t kTmem = kBar + 32;
  static constexpr uint32_t kBytes = kTmem + 16;
};
// Two CTAs of bf16 inputs on an SM (1 KB of each is the system's).
static_assert(2 * (OutSmem<bf16, 64>::kBytes + 1024) <= 228 * 1024, "shared memory of an SM");

// A row is a slot, and so is a column of C B^T and of the factors; slot l of a
// quarter is its token 4 (l % 8) + l / 8.  One CTA per (row, block, group,
// `heads` of its heads); TMEM holds C B^T of the block, shared by the heads,
// and the two parts of y of PT columns.  Two CTAs fit an SM.
//
// An item is PT columns of a head.  What it needs is asked for an item ahead,
// each buffer as soon as its last reader is done: S after C S, x after the
// epilogue, z after the last y has left, the row's factors into registers.
// (With S, x and z asked for when they were needed an item took 5 us of a
// CTA's time; two waves of CTAs on 8192 tokens of 64 heads 151 us.)
template <typename T, int PT>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 1 : 2)
    ssm_out_kernel(const SsmParams p, const TcBufs t, int heads) {
  using L = OutSmem<T, PT>;
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kCols = PT * L::kParts;      // TMEM columns of each part of y
  static_assert(128 + 2 * kCols <= 256, "tensor memory");
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar_cb = sb + L::kBar, bar_x = bar_cb + 8, bar_s = bar_cb + 16,
                 bar_m = bar_cb + 24;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3, half = warp >> 2, r = 32 * quad + lane;
  const int r_token = token_of(lane);       // within the quarter
  const int nb = t.nb, N = p.N, hg = p.H / p.G, per = (hg + heads - 1) / heads;
  int u = blockIdx.x;
  const int part = u % per;
  u /= per;
  const int g = u % p.G;
  u /= p.G;
  const int blk = u % nb, b = u / nb, t0 = blk * kQ;
  const int h_lo = g * hg + part * heads, h_hi = min(h_lo + heads, (g + 1) * hg);
  const int subs = p.P / PT;
  const int n_items = (h_hi - h_lo) * subs;
  if (warp == 0) tmem_alloc(sb + L::kTmem, 256);
  if (tid == 0) {
    mbar_init(bar_cb, 1);
    mbar_init(bar_x, 1);
    mbar_init(bar_s, 1);
    mbar_init(bar_m, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kTmem);
  after_previous();
  const uint32_t t_cb = tmem, t_yi = tmem + 128, t_yx = tmem + 128 + kCols;
  const uint32_t lanes = (uint32_t)(32 * quad) << 16;
  uint32_t n_m = 0;       // commits waited for
  bool bad = false;       // a wait ran out
  auto give_up = [&]() {
    bad = true;
    set_status(t.status, KDA_DEVICE_TIMEOUT);
  };
  auto wait_mma = [&]() {
    if (!mbar_wait(bar_m, n_m & 1)) give_up();
    ++n_m;
    tc_fence_after();
  };
  const uint32_t tile = (uint32_t)(kQ * N * 2);
  auto x_of = [&](int k) {      // item k's x, in the buffers of x
    const size_t at = ((size_t)b * nb + blk) * p.H + h_lo + k / subs;
    return at * kQ * p.P * 2 + (size_t)(k % subs * PT) * kQ * 2;
  };
  auto load_x = [&](int k) {
    mbar_expect_tx(bar_x, (uint32_t)(kQ * PT * 2) * L::kParts);
    bulk_load(sb + L::kX, t.xt + x_of(k), kQ * PT * 2, bar_x);
    if (kF32) bulk_load(sb + L::kX + kQ * PT * 2, t.xlo + x_of(k), kQ * PT * 2, bar_x);
  };
  auto load_s = [&](int k) {
    const size_t at = ((size_t)b * nb + blk) * p.H + h_lo + k / subs;
    const size_t os = at * N * p.P * 2 + (size_t)(k % subs * PT) * N * 2;
    mbar_expect_tx(bar_s, (uint32_t)(N * PT * 2) * L::kParts);
    bulk_load(sb + L::kS, t.st + os, N * PT * 2, bar_s);
    if (kF32) bulk_load(sb + L::kS + N * PT * 2, t.slo + os, N * PT * 2, bar_s);
  };
  int n_x = 0, n_s = 0;         // thread 0: loads of x and S asked for
  if (tid == 0) {
    const size_t o = (((size_t)b * nb + blk) * p.G + g) * tile;
    mbar_expect_tx(bar_cb, 2 * tile * (kF32 ? 3 : 1));
    bulk_load(sb + L::kC, t.ct + o, tile, bar_cb);
    bulk_load(sb + L::kF, t.bt + o, tile, bar_cb);
    if (kF32) {
      bulk_load(sb + L::kC + L::kPart, t.clo + o, tile, bar_cb);
      bulk_load(sb + L::kF + L::kPart, t.btlo + o, tile, bar_cb);
      bulk_load(sb + L::kThird, t.c3 + o, tile, bar_cb);
      bulk_load(sb + L::kThird + L::kPart, t.bt3 + o, tile, bar_cb);
    } else {
      load_s(n_s++);
      load_x(n_x++);
    }
  }
  const int flags = t.flags[(size_t)b * nb + blk];
  const int run = t.run[((size_t)b * nb + blk) * kQ + r];
  signed char *srun = reinterpret_cast<signed char *>(smem + L::kRun);   // at most 128 resets
  if (half == 0) srun[r] = (signed char)run;
  float *scumj = reinterpret_cast<float *>(smem + L::kCum);
  float *scumj_lo = reinterpret_cast<float *>(smem + L::kCumLo);
  // the factors of the next item's head: of row r, and of column tid
  float ein = 0.f, cr = 0.f, cl = 0.f, cj = 0.f, cjl = 0.f, dlog = 0.f, xi = 0.f;
  auto factors = [&](int k) {
    const size_t at = (((size_t)b * p.H + h_lo + k / subs) * nb + blk) * kQ;
    ein = t.ein[at + r];
    cr = t.cum[at + r];
    if (kF32) cl = t.cum_lo[at + r];
    if (tid < kQ) {
      cj = t.cumj[at + tid];
      if (kF32) cjl = t.cumj_lo[at + tid];
    }
    dlog = t.dlog[((size_t)b * p.H + h_lo + k / subs) * nb + blk];
    if (tid < PT / 2)
      xi = t.xinv[((((size_t)b * nb + blk) * p.H + h_lo + k / subs) * p.P + k % subs * PT + 2 * tid) /
                  t.xch];
  };
  factors(0);
  const Opnd opC = {sb + L::kC, 128, (uint32_t)N * 16};
  const Opnd opC2 = {sb + L::kC + L::kPart, 128, (uint32_t)N * 16};
  if (!mbar_wait(bar_cb, 0)) give_up();
  if (tid == 0 && !bad) {
    const Opnd opB = {sb + L::kF, 128, (uint32_t)N * 16};
    if (kF32) {        // (the small products first)
      const Opnd opB2 = {sb + L::kF + L::kPart, 128, (uint32_t)N * 16};
      const Opnd opC3 = {sb + L::kThird, 128, (uint32_t)N * 16};
      const Opnd opB3 = {sb + L::kThird + L::kPart, 128, (uint32_t)N * 16};
      mma_k(t_cb, opC, 0, opB3, 0, N / 16, 128, false);
      mma_k(t_cb, opC3, 0, opB, 0, N / 16, 128, true);
      mma_k(t_cb, opC2, 0, opB2, 0, N / 16, 128, true);
      mma_k(t_cb, opC, 0, opB2, 0, N / 16, 128, true);
      mma_k(t_cb, opC2, 0, opB, 0, N / 16, 128, true);
    }
    mma_k(t_cb, opC, 0, opB, 0, N / 16, 128, kF32);
    mma_commit(bar_m);
  }
  wait_mma();
  if (kF32 && tid == 0 && !bad) {      // where the third parts were
    load_s(n_s++);
    load_x(n_x++);
  }
  // A row's factors are kept in fp16, over the power of two that leaves the row of
  // C B^T below 2^15 times the head's widest d: 11 bits of what is not 2^29 times
  // smaller.  The row's largest finite value, by its two threads:
  float *stop = reinterpret_cast<float *>(smem + L::kZ);      // [2][128]
  auto row_top = [&](bool filter) {
    float m = 0.f;
#pragma unroll 1
    for (int q = half; q < 2 * quad + 2; q += 2) {
      float v[16];
      tmem_ld16(t_cb + lanes + 16 * q, v);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (!filter || fabsf(v[e]) < CUDART_INF_F) m = fmaxf(m, fabsf(v[e]));
    }
    return m;
  };
  float top = row_top(false);
  if (__any_sync(0xffffffffu, !(top < CUDART_INF_F))) top = row_top(true);
  stop[half * kQ + r] = top;
  __syncthreads();
  const float row_inv = to_2p15(fmaxf(top, stop[(half ^ 1) * kQ + r]));
  const float row_log = (float)((int)(__float_as_uint(row_inv) >> 23) - 127);
  float f_inv = 0.f;            // what 1 in the factors of row r stands for
  // entries above the diagonal's 32-row steps are never written again
  for (int i = tid; i < (int)(L::kParts * L::kPart / 16); i += 256)
    *reinterpret_cast<uint4 *>(smem + L::kF + i * 16) = make_uint4(0, 0, 0, 0);

  // z and y: 16-byte pieces of a [128][PT] tile, a thread copies piece q0 of
  // slots s0, s0 + kStep, ..
  constexpr int kP16 = PT * (int)sizeof(T) / 16, kStep = 256 / kP16, kEl = 16 / (int)sizeof(T);
  auto piece = [&](int row, int q) {
    return (uint32_t)(L::kZ + row * kP16 * 16 + ((q ^ (kP16 == 8 ? row & 7 : row >> 1 & 3)) << 4));
  };
  const int q0 = tid % kP16, s0 = tid / kP16;
  for (int k = 0; k < n_items; ++k) {
    const int h = h_lo + k / subs, c = k % subs * PT, ch = h * p.P + c;
    if (tid == 0 && !bad) {
      if (mbar_wait(bar_s, k & 1)) {
        const Opnd opS = {sb + L::kS, 128, (uint32_t)N * 16};
        if (kF32) mma_k(t_yi, opC2, 0, opS, 1, N / 16, kCols, false);
        mma_k(t_yi, opC, 0, opS, 1, N / 16, kCols, kF32);
        mma_commit(bar_m);
      } else {
        give_up();
      }
    }
    if (c == 0 && tid < kQ) {
      scumj[tid] = cj;
      if (kF32) scumj_lo[tid] = cjl;
    }
    if (tid < PT / 2) reinterpret_cast<float *>(smem + L::kXinv)[tid] = xi;
    if (__syncthreads_or(bad)) break;         // cumj is there, the last y has left
    if (p.z) {
      const T *z = static_cast<const T *>(p.z) + (size_t)b * p.z_sb + (long long)t0 * p.z_st + ch +
                   q0 * kEl;
#pragma unroll
      for (int s = s0; s < kQ; s += kStep) {
        const int tok = token_of(s);
        const bool ok = t0 + tok < p.T;
        cp_async16(sb + piece(s, q0), z + (ok ? (long long)tok * p.z_st : 0), ok);
      }
      cp_async_commit();
    }
    const float ein_now = ein;
    if (c == 0) {
      // factors of the head: row r, 16 columns at a time, up to the diagonal
      // over f_inv, the row's and the head's power of two
      f_inv = row_inv * __uint_as_float((uint32_t)(127 + (int)dlog) << 23);
      const Two cs = kF32 ? two_sum(cr, -(row_log + dlog)) : Two{cr - (row_log + dlog), 0.f};
      const float cls = cl + cs.lo;
      const u64 cr2 = pk2(cs.hi, cs.hi), cl2 = pk2(cls, cls), neg = pk2(-1.f, -1.f);
#pragma unroll 1
      for (int q = half; q < 2 * quad + 2; q += 2) {
        float v[16];
        tmem_ld16(t_cb + lanes + 16 * q, v);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const ulonglong2 j = *reinterpret_cast<const ulonglong2 *>(scumj + 16 * q + e);
          float f[4];
          u64 d0 = fma2(j.x, neg, cr2), d1 = fma2(j.y, neg, cr2);
          if (kF32) {
            const ulonglong2 jl = *reinterpret_cast<const ulonglong2 *>(scumj_lo + 16 * q + e);
            d0 = add2(d0, fma2(jl.x, neg, cl2));
            d1 = add2(d1, fma2(jl.y, neg, cl2));
          }
          upk2(d0, f[0], f[1]);
          upk2(d1, f[2], f[3]);
          const u64 lo = mul2(pk2(v[e], v[e + 1]), pk2(ex2(f[0]), ex2(f[1])));
          const u64 hi = mul2(pk2(v[e + 2], v[e + 3]), pk2(ex2(f[2]), ex2(f[3])));
          upk2(lo, v[e], v[e + 1]);
          upk2(hi, v[e + 2], v[e + 3]);
        }
        if (q >= 2 * quad) {     // the diagonal's quarter: later tokens do not count
          const int last = r_token - 2 * (q & 1);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (token_of(e) > last) v[e] = 0.f;
        }
        if (flags & kResets) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (srun[16 * q + e] != (signed char)run) v[e] = 0.f;
        }
        unsigned char *f = smem + L::kF + (r & 7) * 16 + (r >> 3) * 2048 + 2 * q * 128;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          float a[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) a[e] = v[8 * o + e];
          const u64 w[4] = {pk2(a[0], a[1]), pk2(a[2], a[3]), pk2(a[4], a[5]), pk2(a[6], a[7])};
          uint4 hi, lo;
          if constexpr (kF32) {
            split16(w, hi, lo);
            *reinterpret_cast<uint4 *>(f + L::kPart + 128 * o) = lo;
          } else {
            hi = pack16<uint4>(w);
          }
          *reinterpret_cast<uint4 *>(f + 128 * o) = hi;
        }
      }
      fence_proxy_async();
    }
    if (k + 1 < n_items) factors(k + 1);
    wait_mma();                    // C S is done
    tc_fence_before();
    if (__syncthreads_or(bad)) break;
    if (tid == 0) {
      if (k + 1 < n_items) load_s(n_s++);
      if (mbar_wait(bar_x, k & 1)) {
        const Opnd opF = {sb + L::kF, 128, kQ * 16}, opX = {sb + L::kX, 128, kQ * 16};
        if (kF32) {
          const Opnd opF2 = {sb + L::kF + L::kPart, 128, kQ * 16};
          mma_k<true>(t_yx, opF2, 0, opX, 1, kQ / 16, kCols, false);
        }
        mma_k<true>(t_yx, opF, 0, opX, 1, kQ / 16, kCols, kF32);
        mma_commit(bar_m);
        if (k + 1 < n_items) {
          prefetch_l2(t.xt + x_of(k + 1), kQ * PT * 2);
          if (kF32) prefetch_l2(t.xlo + x_of(k + 1), kQ * PT * 2);
        }
      } else {
        give_up();
      }
    }
    wait_mma();
    if (!mbar_wait(bar_x, k & 1)) give_up();      // (x is there: it is read below)
    cp_async_wait_all();
    if (__syncthreads_or(bad)) break;
    // y of row r, columns [half PT / 2, (half + 1) PT / 2)
    const float D = p.D ? p.D[h] : 0.f;
    const u64 ein2 = pk2(ein_now, ein_now), D2 = pk2(D, D), f_inv2 = pk2(f_inv, f_inv);
#pragma unroll
    for (int e0 = 0; e0 < PT / 2; e0 += 16) {
      const int col = half * (PT / 2) + e0;
      float yi[16], yx[16];
      tmem_ld16x2(t_yi + lanes + col, t_yx + lanes + col, yi, yx);
      if (kF32) {           // the products with the second parts
        float vi[16], vx[16];
        tmem_ld16x2(t_yi + lanes + PT + col, t_yx + lanes + PT + col, vi, vx);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          yi[e] += vi[e];
          yx[e] += vx[e];
        }
      }
      if ((flags & kResets) && run > 0)            // the entering state does not reach the
#pragma unroll
        for (int e = 0; e < 16; ++e) yi[e] = 0.f;  // token, whatever it holds
      // x of a later token or another run may be NaN or infinite, which times 0 is
      // NaN: then the tokens that reach row r are added up one by one
      u64 odd = 0;
#pragma unroll
      for (int e = 0; e < 16; e += 2) odd = fma2(pk2(yx[e], yx[e + 1]), 0, odd);
      if (__any_sync(0xffffffffu, (odd & 0x7fffffff7fffffffull) != 0)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) yx[e] = 0.f;
#pragma unroll 1
        for (int j = 0; j < kQ; ++j) {
          if (token_of(j) > 32 * quad + r_token ||
              ((flags & kResets) && srun[j] != (signed char)run))
            continue;
          const unsigned char *fp = smem + L::kF + op_off(r, j, kQ),
                              *xp = smem + L::kX + mn_off(col, j, kQ);
          float f = __half2float(*reinterpret_cast<const __half *>(fp));
          if (kF32) f += __half2float(*reinterpret_cast<const __half *>(fp + L::kPart));
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const unsigned char *v = xp + mn_off(e, 0, kQ);
            float x = __half2float(*reinterpret_cast<const __half *>(v));
            if (kF32) x += __half2float(*reinterpret_cast<const __half *>(v + kQ * PT * 2));
            yx[e] = fmaf(f, x, yx[e]);
          }
        }
      }
      float xinv[8];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<float4 *>(xinv + 4 * q) =
            *reinterpret_cast<const float4 *>(smem + L::kXinv + col * 2 + 16 * q);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        u64 x[4], z[4], y[4];
        const unsigned char *xp = smem + L::kX + (col / 8 + q) * 2048 + (r >> 3) * 128 + (r & 7) * 16;
        unpack16(*reinterpret_cast<const uint4 *>(xp), x);
        if (kF32) {
          unpack16(*reinterpret_cast<const uint4 *>(xp + kQ * PT * 2), z);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = add2(x[e], z[e]);
        }
        // the 8 columns are one piece of z and y, or two of fp32
        unsigned char *zp = smem + piece(r, (col / 8 + q) * (8 / kEl));
        unsigned char *zp2 = smem + piece(r, (col / 8 + q) * (8 / kEl) + (kF32 ? 1 : 0));
        if (p.z) {
          if constexpr (kF32) {
            const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(zp),
                             d = *reinterpret_cast<const ulonglong2 *>(zp2);
            z[0] = a.x; z[1] = a.y; z[2] = d.x; z[3] = d.y;
          } else {
            Unpack8::unpack(*reinterpret_cast<const uint4 *>(zp), z);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 8 * q + 2 * e;
          const u64 v = fma2(f_inv2, pk2(yx[i], yx[i + 1]), mul2(D2, x[e]));
          y[e] = fma2(pk2(xinv[4 * q + e], xinv[4 * q + e]), v, mul2(ein2, pk2(yi[i], yi[i + 1])));
          if (p.z) {
            float a, d, d0, d1;
            upk2(mul2(z[e], pk2(-kLog2e, -kLog2e)), a, d);
            upk2(add2(pk2(1.f, 1.f), pk2(ex2(a), ex2(d))), d0, d1);
            y[e] = mul2(mul2(y[e], z[e]), pk2(rcp(d0), rcp(d1)));
          }
          if (run < 0) y[e] = 0;
        }
        if constexpr (kF32) {
          *reinterpret_cast<ulonglong2 *>(zp) = make_ulonglong2(y[0], y[1]);
          *reinterpret_cast<ulonglong2 *>(zp2) = make_ulonglong2(y[2], y[3]);
        } else {
          *reinterpret_cast<uint4 *>(zp) = pack<uint4>(y);
        }
      }
    }
    tc_fence_before();
    fence_proxy_async();
    __syncthreads();               // x is read, y is whole
    if (tid == 0) {
      tc_fence_after();
      if (k + 1 < n_items) load_x(n_x++);
    }
    T *y = static_cast<T *>(p.y) + ((size_t)b * p.T + t0) * p.H * p.P + ch + q0 * kEl;
#pragma unroll
    for (int s = s0; s < kQ; s += kStep) {
      const int tok = token_of(s);
      if (t0 + tok < p.T)
        *reinterpret_cast<uint4 *>(y + (size_t)tok * p.H * p.P) =
            *reinterpret_cast<const uint4 *>(smem + piece(s, q0));
    }
  }
  if (__syncthreads_or(bad)) {     // nothing is in flight when the CTA leaves
    if (tid == 0) {
      mbar_wait(bar_cb, 0);
      mbar_wait(bar_x, (n_x - 1) & 1);
      mbar_wait(bar_s, (n_s - 1) & 1);
    }
    mbar_wait(bar_m, (n_m - 1) & 1);
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 256);
}

template <typename T, int TP>
cudaError_t launch_prep(const SsmParams &p, const TcBufs &t, cudaStream_t cs) {
  size_t smem = 2 * (PrepConv<T, TP>::kBytes + kQ) + 16 * sizeof(typename PrepConv<T, TP>::Consts);
  const size_t f = (kQ + 8) * 4 + kQ * 33 * 4;
  if (f > smem) smem = f;
  // blocks per CTA: up to 8, as long as three waves of CTAs are left (2 rows of
  // 8192 tokens, 8 groups: 4 blocks take 14 us less than 1; one row, one group: 8
  // take 8 us more)
  const long long tiles = (long long)p.B * t.nb * p.G * (2 * p.N / TP);
  long long run = tiles / (6ll * num_sms());
  run = run < 1 ? 1 : run > 8 ? 8 : run;
  const int runs = (int)((t.nb + run - 1) / run);
  const int caches = p.conv_out ? (p.channels + kPrep - 1) / kPrep : 0;
  const unsigned grid = (unsigned)(p.B * (t.nb + runs * p.G * (2 * p.N / TP) + caches));
  if (p.segment_ids)
    return launch_next(ssm_prep_kernel<T, TP>, grid, kPrep, smem, cs, p, t, (int)run);
  ssm_prep_kernel<T, TP><<<grid, kPrep, smem, cs>>>(p, t, (int)run);
  return cudaGetLastError();
}

template <typename T, int TP, bool IDS>
cudaError_t launch_state_i(const SsmParams &p, const TcBufs &t, cudaStream_t cs) {
  auto kern = ssm_state_kernel<T, TP, IDS>;
  constexpr int smem = (int)StateSmem<T, TP>::kBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_next(kern, (unsigned)(p.B * p.H * (p.P / TP)), kConv + 32, smem, cs, p, t);
}
template <typename T, int TP>
cudaError_t launch_state(const SsmParams &p, const TcBufs &t, cudaStream_t cs) {
  return p.segment_ids ? launch_state_i<T, TP, true>(p, t, cs)
                       : launch_state_i<T, TP, false>(p, t, cs);
}

template <typename T, int PT>
cudaError_t launch_out(const SsmParams &p, const TcBufs &t, cudaStream_t cs) {
  constexpr int smem = (int)OutSmem<T, PT>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(ssm_out_kernel<T, PT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // heads per CTA: up to 4, as long as the CTAs fill the GPU twice over (8 and
  // 16 take as long: 140 us for 2 rows of 8192 tokens of 64 heads)
  const int hg = p.H / p.G;
  int heads = 4;
  auto ctas = [&](int n) { return (long long)p.B * t.nb * p.G * ((hg + n - 1) / n); };
  while (heads > 1 && ctas(heads) < 4ll * num_sms()) heads /= 2;
  return launch_next(ssm_out_kernel<T, PT>, (unsigned)ctas(heads), 256, smem, cs, p, t, heads);
}

}  // namespace

size_t ssm_tc_bytes(const SsmParams &p, bool f32) {
  TcBufs t;
  return layout_bufs(p, f32, nullptr, &t);
}

cudaError_t launch_ssm_tc(const SsmParams &p, bool f32, uint32_t *status, cudaStream_t cs) {
  TcBufs t;
  layout_bufs(p, f32, p.ws, &t);
  t.status = status;
  cudaError_t e;
  t.xch = 2;
  if (f32) {       // twice the operands: tiles of 32 columns throughout
    e = launch_prep<float, 32>(p, t, cs);
    if (e == cudaSuccess) e = launch_state<float, 32>(p, t, cs);
    return e == cudaSuccess ? launch_out<float, 32>(p, t, cs) : e;
  }
  e = p.N == 32 ? launch_prep<bf16, 32>(p, t, cs) : launch_prep<bf16, 64>(p, t, cs);
  if (e != cudaSuccess) return e;
  // 64-column tiles halve the traffic of B's tiles (2 rows of 64 heads of 64
  // columns: 158 us; measured before the scales 141, with 32 columns 246); 32
  // where half the SMs would have no CTA (a packed row of 32 heads of 128 columns:
  // 129 us; before the scales 118, with 64 columns 156)
  const bool narrow = p.P == 32 || (long long)p.B * p.H * (p.P / 64) * 2 <= num_sms();
  t.xch = narrow ? 2 : 4;            // a state kernel's warp's channels
  e = narrow ? launch_state<bf16, 32>(p, t, cs) : launch_state<bf16, 64>(p, t, cs);
  if (e != cudaSuccess) return e;
  return p.P == 32 ? launch_out<bf16, 32>(p, t, cs) : launch_out<bf16, 64>(p, t, cs);
}

}  // namespace kda
