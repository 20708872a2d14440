// kda_latent_bwd_tc.cu -- the expanded latent attention's gradients on the tensor
// cores.
//
// With D_i = d_o_i . o_i, p_ij = exp(s_ij - lse_i) and ds_ij = p_ij (d_o_i . v_j - D_i):
//     dv_j = sum_i p_ij d_o_i,   dk_j = scale sum_i ds_ij q_i,   dq_i = scale sum_j ds_ij k_j
// Two kernels of one shape (and a third for D of queries with few keys), which make s and
// ds twice so that every sum stays in
// one CTA's tensor memory: no atomics, no sums in global memory but the heads' parts of
// dk_rope.  A CTA holds 128 rows of one side of one head (keys and values, or queries
// and d_o) and walks the other side in tiles of 64:
//     S = X1 Y1^T, dP = X2 Y2^T     128 x 64
//     dX1 += dS Y1, dX2 += P Y2     (dX2 for the values alone)
// P and dS are rounded to bf16, the type of the inputs that they meet in a product
// (gradients 2.3e-3 off in the 2-norm, 1.7e-3 of it their own rounding); S, dP, D and all sums are
// fp32.  P and dS lie in tensor memory where S was, S twice, so that S of the next
// tile is made while the rows' threads work on this one, and dP of the next one comes
// first when they are done: the products then hide behind the exponentials.
//
// Shared memory (200 KB): 5 chunks of 16 KB of X, 3 stages of 5 chunks of 8 KB of Y.
// Tensor memory: S twice and dP of 64 columns, dX1 192, dX2 128; for the queries, without
// dX2, X1 instead, whose chunks make room for a fourth stage.
//
// A row of 8192 tokens, 32 heads of 128 + 64: keys and values 910 to 925 us (with fewer
// registers, and what a column needs read after the wait, 1050), queries 778 (with X1 in
// shared memory and three stages 886), D 29.  What bounds them: the products (an instruction
// of N 64 takes 44 cycles with both operands in shared memory, 29 with one: 1400 of 1800
// cycles a tile for the keys) and, as far as their bytes and those cycles tell, the tiles
// of the other side: 40 KB a tile on every SM, 5.45 GB for the keys, come to 6 TB/s out of L2.
#include "kda_f32x2.cuh"
#include "kda_latent_tc.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kOuter = 128, kInner = 64;
constexpr int kMaxStages = 4;
constexpr uint32_t kXChunkB = kOuter * kRowBytes, kYChunkB = kInner * kRowBytes;
constexpr uint32_t kStageB = 5 * kYChunkB;
constexpr uint32_t kOffY = 5 * kXChunkB, kOffC = kOffY + 3 * kStageB;
constexpr uint32_t kSmem = kOffC + 4096 + 1024;
constexpr int kThreads = 384;                  // 8 warps of rows; copies, products, two idle ones
constexpr uint32_t kTdP = 128, kTX1 = 192, kTX2 = 384;   // columns; X1 itself where dX2 is not made

struct Maps {
  CUtensorMap x1, x1r, x2, y1, y1r, y2;
};

struct Control {
  uint64_t x_full, x_moved, y_full[kMaxStages], y_empty[kMaxStages], s_full, ds_ready, done, drain;
  uint32_t tmem;
  int fail;
  unsigned bad[8];
  alignas(16) float stat[8][2][32];      // read four at a time
};

// What a launch makes.  kDelta: D of queries that see at most kExactKeys keys, as
// sum_j p_ij (d_o_i . v_j) / sum_j p_ij.  D from the stored o has o's rounding, whose part of
// ds = p (dp - D) is the larger the fewer keys a query sees (dq and dk of rows of 40
// tokens 2.9e-3 off in the 2-norm, with this 2.3e-3, 1.7e-3 of it their own rounding; of
// 1000 tokens 2.6e-3 and 2.3e-3).  Whether a query is one of them hangs on it alone: a CTA
// walks the keys from the first one that such a query of its rows sees, at most
// kExactKeys + 127 of them, and leaves D of the other rows as it is.
enum What { kKeysOf, kQueriesOf, kDelta };
__device__ __forceinline__ bool few_keys(int start, int row) {
  return start <= row && row - start < kExactKeys;
}

template <What kWhat>
__global__ void __launch_bounds__(kThreads, 1)
prompt_bwd_tc_kernel(const __grid_constant__ Maps maps, const Prompt p) {
  constexpr bool kKeys = kWhat == kKeysOf;
  constexpr int kStages = kKeys ? 3 : 4;
  extern __shared__ __align__(1024) unsigned char raw[];
  unsigned char *smem = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
  Control &c = *reinterpret_cast<Control *>(smem + kOffC);
  const uint32_t s0 = tc::smem_u32(smem);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  int tiles = (p.T + kOuter - 1) / kOuter;
  if (kWhat == kDelta && !p.start) tiles = min(tiles, kExactKeys / kOuter);
  // one head after another, its longest rows first
  const int bh = (int)(blockIdx.x / (unsigned)tiles), order = (int)(blockIdx.x % (unsigned)tiles);
  const int t0 = (kKeys ? order : tiles - 1 - order) * kOuter;
  const int b = bh / p.H, h = bh % p.H;
  const int nk = (p.K + kChunkCols - 1) / kChunkCols, nc = nk + (p.R > 0 ? 1 : 0);
  const int nv = (p.V + kChunkCols - 1) / kChunkCols;
  const int t_last = min(p.T, t0 + kOuter) - 1;
  // tiles of the other side
  int first_key = kKeys ? t0 : run_start(p, b, t0);
  if (kWhat == kDelta) {       // (every warp looks at all rows; starts rise along them)
    first_key = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kOuter / 32; ++i) {
      const int row = t0 + 32 * i + lane;
      const int start = row < p.T ? run_start(p, b, row) : 0x7fffffff;
      if (few_keys(start, row)) first_key = min(first_key, start);
    }
    first_key = __reduce_min_sync(0xffffffffu, first_key);
    if (first_key == 0x7fffffff) return;
  }
  const int first = first_key / kInner;
  const int stop = kKeys ? (run_end(p, b, t_last) + kInner - 1) / kInner : t_last / kInner + 1;
  const int n = stop > first ? stop - first : 0;
  auto bar = [](uint64_t &x) { return tc::smem_u32(&x); };
  if (tid == 0) {
    tc::mbar_init(bar(c.x_full), 1);
    tc::mbar_init(bar(c.x_moved), 256);
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(bar(c.y_full[i]), 1);
      tc::mbar_init(bar(c.y_empty[i]), 1);
    }
    tc::mbar_init(bar(c.s_full), 1);
    tc::mbar_init(bar(c.ds_ready), 256);
    tc::mbar_init(bar(c.done), 1);
    tc::mbar_init(bar(c.drain), 1);
    c.fail = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(tc::smem_u32(&c.tmem), 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (kKeys) start_next();
  const uint32_t tmem = c.tmem;
  const Waits wait(&c.fail, p.T);
  // the fourth stage lies where X1 was
  auto stage_at = [&](int s) { return s < 3 ? s0 + kOffY + (uint32_t)s * kStageB : s0; };

  if (warp >= 8) {
    few_registers();
    if (warp == 8) {
    // ---- copies: one thread ----
    if (lane == 0 && n > 0) {
      // (keys' rope part is shared by the heads)
      const int xr_h = kKeys ? 0 : h, yr_h = kKeys ? h : 0;
      tc::mbar_expect_tx(bar(c.x_full), (uint32_t)(nc + nv) * kXChunkB);
      for (int i = 0; i < nk; ++i)
        tma_load_4d(s0 + (uint32_t)i * kXChunkB, &maps.x1, i * kChunkCols, h, t0, b,
                    bar(c.x_full));
      if (nc > nk)
        tma_load_4d(s0 + (uint32_t)nk * kXChunkB, &maps.x1r, 0, xr_h, t0, b, bar(c.x_full));
      for (int i = 0; i < nv; ++i)
        tma_load_4d(s0 + (uint32_t)(3 + i) * kXChunkB, &maps.x2, i * kChunkCols, h, t0, b,
                    bar(c.x_full));
      bool ok = true;
      int i = 0;
      for (; i < n; ++i) {
        const int s = i % kStages, y0 = (first + i) * kInner;
        ok = wait(bar(c.y_empty[s]), (uint32_t)(i / kStages + 1) & 1);
        if (ok && i == 3 && !kKeys) ok = wait(bar(c.x_moved), 0);
        if (!ok) break;
        const uint32_t d = stage_at(s);
        tc::mbar_expect_tx(bar(c.y_full[s]), (uint32_t)(nc + nv) * kYChunkB);
        for (int e = 0; e < nk; ++e)
          tma_load_4d(d + (uint32_t)e * kYChunkB, &maps.y1, e * kChunkCols, h, y0, b,
                      bar(c.y_full[s]));
        if (nc > nk)
          tma_load_4d(d + (uint32_t)nk * kYChunkB, &maps.y1r, 0, yr_h, y0, b, bar(c.y_full[s]));
        for (int e = 0; e < nv; ++e)
          tma_load_4d(d + (uint32_t)(3 + e) * kYChunkB, &maps.y2, e * kChunkCols, h, y0, b,
                      bar(c.y_full[s]));
      }
      if (c.fail) {   // what is on its way comes in before the CTA ends
        tc::mbar_wait(bar(c.x_full), 0);
        for (int k = max(0, i - kStages); k < i; ++k)
          tc::mbar_wait(bar(c.y_full[k % kStages]), (uint32_t)(k / kStages) & 1);
      }
    }
    __syncwarp();
    } else if (warp == 9) {
    // ---- products: one thread ----
    if (n > 0 && elect_one()) {
      const uint32_t id_s = tc::idesc_bf16(kOuter, kInner, 0, 0),
                     id_x1 = tc::idesc_bf16(kOuter, nc * kChunkCols, 0, 1),
                     id_x2 = tc::idesc_bf16(kOuter, nv * kChunkCols, 0, 1);
      auto scores = [&](int i) {        // S of tile i
        const uint32_t y = stage_at(i % kStages);
        const uint64_t dx = swizzled_desc(s0, 16), dy = swizzled_desc(y, 16);
        for (int e = 0; e < nc; ++e) {
          const uint64_t x = dx + kXChunkB / 16 * e, z = dy + kYChunkB / 16 * e;
          const uint32_t old = e > 0 ? 1u : 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (kKeys)
              tc::mma_bf16(tmem + kInner * (i & 1), x + kStepK * k, z + kStepK * k, id_s,
                           k > 0 ? 1u : old);
            else
              mma_bf16_ts(tmem + kInner * (i & 1), tmem + kTX2 + 32 * e + 8 * k, z + kStepK * k, id_s,
                          k > 0 ? 1u : old);
          }
        }
      };
      auto dp = [&](int i) {
        const uint32_t y = stage_at(i % kStages);
        const uint64_t dx = swizzled_desc(s0 + 3 * kXChunkB, 16),
                       dy = swizzled_desc(y + 3 * kYChunkB, 16);
        for (int e = 0; e < nv; ++e) {
          const uint64_t x = dx + kXChunkB / 16 * e, z = dy + kYChunkB / 16 * e;
          const uint32_t old = e > 0 ? 1u : 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_bf16(tmem + kTdP, x + kStepK * k, z + kStepK * k, id_s, k > 0 ? 1u : old);
        }
      };
      auto loaded = [&](int i) {
        return wait(bar(c.y_full[i % kStages]), (uint32_t)(i / kStages) & 1);
      };
      bool ok = wait(bar(c.x_full), 0) && (kKeys || wait(bar(c.x_moved), 0)) && loaded(0);
      if (!kKeys) tc::tc_fence_after();
      if (ok) {
        scores(0);
        dp(0);
        tc::mma_commit(bar(c.s_full));
      }
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n) {
          ok = loaded(i + 1);
          if (!ok) break;
          scores(i + 1);
        }
        ok = wait(bar(c.ds_ready), (uint32_t)i & 1);
        if (!ok) break;
        tc::tc_fence_after();
        if (i + 1 < n) {
          dp(i + 1);
          tc::mma_commit(bar(c.s_full));
        }
        if (kWhat != kDelta) {
          // steps of 16 rows of Y: the two halves of 32 stand 32 columns apart
          const uint32_t y = stage_at(i % kStages);
          const uint32_t w = tmem + kInner * (i & 1), old = i > 0 ? 1u : 0u;
          const uint64_t dy = swizzled_desc(y, kYChunkB);
          if (kKeys) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma_bf16_ts(tmem + kTX2, w + 32 * (e >> 1) + 8 * (e & 1),
                          dy + 3 * kYChunkB / 16 + kStepRows * e, id_x2, e > 0 ? 1u : old);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma_bf16_ts(tmem + kTX1, w + 16 + 32 * (e >> 1) + 8 * (e & 1), dy + kStepRows * e, id_x1,
                        e > 0 ? 1u : old);
        }
        tc::mma_commit(bar(c.y_empty[i % kStages]));
      }
      if (ok) tc::mma_commit(bar(c.done));
      if (c.fail) {
        tc::mma_commit(bar(c.drain));
        tc::mbar_wait(bar(c.drain), 0);
      }
    }
    __syncwarp();
    }
  } else {
    many_registers();
    // ---- rows: two threads a row, 32 columns each ----
    const int half = warp >> 2, row = t0 + (tid & 127);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const float scale = p.scale * kLog2e;
    const size_t head = ((size_t)b * p.H + h) * p.T;
    // kKeys: columns (queries) [row, to); else columns (keys) [from, row]
    int from = 0x7fffffff, to = 0;
    if (row < p.T) {
      from = kKeys ? row : run_start(p, b, row);
      to = kKeys ? run_end(p, b, row) : row + 1;
    }
    // columns that every row sees
    const int all_from = kKeys ? t_last : run_start(p, b, t_last);
    const int all_to = t_last - t0 + 1 < kOuter ? 0 : kKeys ? run_end(p, b, t0) : t0 + 1;
    if (!kKeys && n > 0) {
      // X1 to tensor memory: its products then read one operand from shared memory, and
      // its place takes another stage
      wait(bar(c.x_full), 0);
      __syncwarp();
      for (int g = half; g < 2 * nc; g += 2) {      // 32 channels
        uint32_t x[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 v = *reinterpret_cast<const uint4 *>(
              smem + (uint32_t)(g >> 1) * kXChunkB + piece_off(tid & 127, 4 * (g & 1) + e));
          x[4 * e] = v.x;
          x[4 * e + 1] = v.y;
          x[4 * e + 2] = v.z;
          x[4 * e + 3] = v.w;
        }
        tmem_st16(tmem + kTX2 + 16 * g + lanes, x);
      }
      tmem_wait_st();
      tc::tc_fence_before();
      tc::mbar_arrive(bar(c.x_moved));
    }
    float lse = 0.f, delta = 0.f, next_lse = 0.f, next_delta = 0.f;
    auto fetch = [&](int i) {
      const int y = (first + i) * kInner + 32 * half + lane;
      next_lse = y < p.T ? p.lse[head + y] * kLog2e : 0.f;
      next_delta = y < p.T ? p.delta[head + y] : 0.f;
    };
    if (kKeys) {
      if (n > 0) fetch(0);
    } else if (row < p.T) {
      lse = p.lse[head + row] * kLog2e;
      if (kWhat == kQueriesOf) delta = p.delta[head + row];
    }
    u64 sum_w = 0, sum_g = 0;           // of p and p dp
    for (int i = 0; i < n; ++i) {
      const int y0 = (first + i) * kInner + 32 * half;
      float2 st[16], de[16];
      if (kKeys) {
        __syncwarp();
        c.stat[warp][0][lane] = -next_lse;
        c.stat[warp][1][lane] = -next_delta;
        __syncwarp();
        if (i + 1 < n) fetch(i + 1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 a = reinterpret_cast<const float4 *>(c.stat[warp][0])[e];
          const float4 g = reinterpret_cast<const float4 *>(c.stat[warp][1])[e];
          st[2 * e] = make_float2(a.x, a.y);
          st[2 * e + 1] = make_float2(a.z, a.w);
          de[2 * e] = make_float2(g.x, g.y);
          de[2 * e + 1] = make_float2(g.z, g.w);
        }
      }
      wait(bar(c.s_full), (uint32_t)i & 1);
      __syncwarp();
      tc::tc_fence_after();
      uint32_t s[32], d[32];
      const uint32_t t_s = tmem + kInner * (i & 1) + 32 * half + lanes;
      tmem_ld32_nw(t_s, s);
      tmem_ld32_nw(tmem + kTdP + 32 * half + lanes, d);
      tc::tmem_wait_ld();
      reg_fence32(s);
      reg_fence32(d);
      const uint32_t on = column_bits(from, to, y0);
      const bool whole = (y0 >= all_from && y0 + 32 <= all_to) ||
                         __all_sync(0xffffffffu, on == 0xffffffffu);
      uint32_t pw[16], dw[16];
      const u64 sc = pk2(scale, scale), nl = pk2(-lse, -lse), nd = pk2(-delta, -delta);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float w0, w1, g0, g1;
        upk2(fma2(pk2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sc,
                  kKeys ? pk2(st[e].x, st[e].y) : nl),
             w0, w1);
        w0 = tc::ex2(w0);
        w1 = tc::ex2(w1);
        upk2(mul2(pk2(w0, w1),
                  add2(pk2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])),
                       kKeys ? pk2(de[e].x, de[e].y) : nd)),
             g0, g1);
        if (!whole) {
          const bool on0 = on >> (2 * e) & 1u, on1 = on >> (2 * e + 1) & 1u;
          w0 = on0 ? w0 : 0.f;
          g0 = on0 ? g0 : 0.f;
          w1 = on1 ? w1 : 0.f;
          g1 = on1 ? g1 : 0.f;
        }
        if (kWhat == kDelta) {
          sum_w = add2(sum_w, pk2(w0, w1));
          sum_g = add2(sum_g, pk2(g0, g1));
        }
        pw[e] = tc::pack_bf16(w0, w1);
        dw[e] = tc::pack_bf16(g0, g1);
      }
      if (kWhat != kDelta) {
        if (kKeys) tmem_st16(t_s, pw);
        tmem_st16(t_s + 16, dw);
        tmem_wait_st();
      }
      tc::tc_fence_before();
      tc::mbar_arrive(bar(c.ds_ready));
    }
    if (kWhat == kDelta) {
      if (n > 0) wait(bar(c.done), 0);
      float a, d;
      upk2(sum_w, a, d);
      c.stat[warp][0][lane] = a + d;
      upk2(sum_g, a, d);
      c.stat[warp][1][lane] = a + d;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (half == 0 && row < p.T && few_keys(from, row)) {
        const float w = c.stat[warp][0][lane] + c.stat[warp + 4][0][lane];
        const float g = c.stat[warp][1][lane] + c.stat[warp + 4][1][lane];
        const_cast<float *>(p.delta)[head + row] = w == 0.f ? 0.f : g / w;
      }
    } else {
      // ---- the sums, 32 columns at a time, the halves in turn ----
      if (n > 0) {
        wait(bar(c.done), 0);
        __syncwarp();
        tc::tc_fence_after();
      }
      bool bad = false;
      const size_t at_row = ((size_t)b * p.T + row) * p.H + h;
      for (int q = half; q < 2 * nc + (kKeys ? 2 * nv : 0); q += 2) {
        const bool is_x2 = q >= 2 * nc, is_rope = !is_x2 && q >= 2 * nk;
        const int col = 32 * (is_x2 ? q - 2 * nc : is_rope ? q - 2 * nk : q);
        const int width = is_x2 ? p.V : is_rope ? p.R : p.K;
        uint32_t x[32];
        if (n > 0) {
          tmem_ld32_wait(tmem + lanes + (is_x2 ? kTX2 + 32 * (q - 2 * nc) : kTX1 + 32 * q), x);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0;
        }
        if (col < width && row < p.T) {
          const float f = is_x2 ? 1.f : p.scale;
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            y[i] = __uint_as_float(x[i]) * f;
            bad |= !finite(y[i]);
          }
          if (kKeys && is_rope) {
            float4 *o = reinterpret_cast<float4 *>(p.dkr_part + at_row * p.R + col);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              o[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          } else {
            void *base = is_x2 ? p.dv : kKeys ? p.dk : is_rope ? p.dqr : p.dq;
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(base) + at_row * width + col);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[i] = make_uint4(tc::pack_bf16(y[8 * i], y[8 * i + 1]),
                                tc::pack_bf16(y[8 * i + 2], y[8 * i + 3]),
                                tc::pack_bf16(y[8 * i + 4], y[8 * i + 5]),
                                tc::pack_bf16(y[8 * i + 6], y[8 * i + 7]));
          }
        }
        __syncwarp();
      }
      const unsigned which = __ballot_sync(0xffffffffu, bad);
      if (lane == 0) c.bad[warp] = which;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      // rows that were not finite, again: 16 of each 32 by either half
      unsigned again = (c.bad[warp & 3] | c.bad[(warp & 3) + 4]) & (half ? 0xffff0000u : 0xffffu);
      for (; again; again &= again - 1) {
        const int r = row - lane + __ffs(again) - 1;
        if (kKeys) key_grad_row<__nv_bfloat16>(p, b, h, r, lane);
        else query_grad_row<__nv_bfloat16>(p, b, h, r, lane);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (tid == 0 && c.fail) set_status(p.status, KDA_DEVICE_TIMEOUT);
  if (warp == 9) tc::tmem_dealloc(tmem, 512);
  if (kWhat == kQueriesOf && blockIdx.x == 0) after_previous();
}

template <What kWhat>
cudaError_t launch(const Maps &m, const Prompt &p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(prompt_bwd_tc_kernel<kWhat>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  unsigned tiles = (unsigned)((p.T + kOuter - 1) / kOuter);
  if (kWhat == kDelta && !p.start && tiles > kExactKeys / kOuter) tiles = kExactKeys / kOuter;
  const unsigned grid = tiles * (unsigned)(p.B * p.H);
  if (kWhat == kQueriesOf)
    return launch_next(prompt_bwd_tc_kernel<kWhat>, dim3(grid), kThreads, kSmem, s, m, p);
  prompt_bwd_tc_kernel<kWhat><<<grid, kThreads, kSmem, s>>>(m, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_bwd_tc(const Prompt &p, cudaStream_t s) {
  const Strides up = {(long long)p.T * p.H * p.V, (long long)p.H * p.V, p.V};
  Maps keys, queries;
  // each tensor as rows of a CTA (128) in one kernel and as the other side (64) in the other
  if (!prompt_map(&keys.x1, p.k, p.k_s, p, p.H, p.K, kOuter) ||
      !prompt_map(&keys.x2, p.v, p.v_s, p, p.H, p.V, kOuter) ||
      !prompt_map(&keys.y1, p.q, p.q_s, p, p.H, p.K, kInner) ||
      !prompt_map(&keys.y2, p.d_o, up, p, p.H, p.V, kInner) ||
      !prompt_map(&queries.x1, p.q, p.q_s, p, p.H, p.K, kOuter) ||
      !prompt_map(&queries.x2, p.d_o, up, p, p.H, p.V, kOuter) ||
      !prompt_map(&queries.y1, p.k, p.k_s, p, p.H, p.K, kInner) ||
      !prompt_map(&queries.y2, p.v, p.v_s, p, p.H, p.V, kInner))
    return cudaErrorInvalidValue;
  keys.x1r = keys.y1r = queries.x1r = queries.y1r = keys.x1;
  if (p.R && (!prompt_map(&keys.x1r, p.kr, p.kr_s, p, 1, p.R, kOuter) ||
              !prompt_map(&keys.y1r, p.qr, p.qr_s, p, p.H, p.R, kInner) ||
              !prompt_map(&queries.x1r, p.qr, p.qr_s, p, p.H, p.R, kOuter) ||
              !prompt_map(&queries.y1r, p.kr, p.kr_s, p, 1, p.R, kInner)))
    return cudaErrorInvalidValue;
  cudaError_t e = launch<kDelta>(queries, p, s);
  if (e == cudaSuccess) e = launch<kKeysOf>(keys, p, s);
  return e != cudaSuccess ? e : launch<kQueriesOf>(queries, p, s);
}

}  // namespace latent
}  // namespace kda
