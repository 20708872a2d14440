// kda_latent_step_tc.cu -- the absorbed latent attention on the tensor cores.
//
// A CTA walks its part of the cache in tiles of 128 tokens.  Both products have
// the tokens' latents as the wide operand and the 32 rows (token, head) that share
// the pass as the narrow one, so no part of an instruction is padding:
//     S^T [128 tokens x 32]  = latents [128 x (C + R)] . q^T          (K: channels)
//     O^T [C latents x 32]  += latents^T [C x 128 tokens] . P^T       (K: tokens)
// A tile is read from memory once and lies in shared memory as chunks of 64
// channels in the 128-byte swizzle, which serve S^T as they are and O^T
// transposed.  Two chunks (128 latents: the M of one O^T block) are one slot of a
// ring; a slot is free when O^T's block has read it, so the next tile comes in
// while this one is worked on.
//
// P is rounded to bf16 because both operands of an instruction have one type and the
// latents are bf16 (o 1.8e-3 off in the 2-norm, 1.6e-3 of it its own rounding); maxima, sums and
// O^T are fp32.
//
// Threads: warps 0 to 7 the softmax, two threads a token with 16 rows each (the running
// maxima of the rows are the same in all of them, and only move when a score exceeds
// them by 2^8, so the sums in tensor memory are hardly ever scaled); warp 8 the copies;
// warp 9 the products.
//
// What bounds it: memory, where a row tile reads its own texts (120 texts of up to 8192
// tokens, 576 MB: 128 us with the join in a graph, 4.5 TB/s; with cold caches this kernel 117,
// the join 19), and the chain of a tile where row tiles share them (two texts of 131072, 64
// heads: 84 us, 2.8 us a tile: S 2000 cycles, softmax 1100, O 1500).  One text of 1000 tokens: 14
// us with the join.
#include "kda_latent_tc.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kTile = 128;               // tokens
constexpr int kThreads = 320;
constexpr int kSoftmax = 256;            // threads
constexpr int kMine = kRows / 2;         // rows of a softmax thread
constexpr uint32_t kChunkB = kTile * kRowBytes;        // 16 KB
constexpr uint32_t kPairB = 2 * kChunkB;
constexpr int kRing = 11;                // chunks in shared memory
constexpr int kMaxPairs = 5, kMaxRopes = 3;
constexpr uint32_t kQChunkB = kRows * kRowBytes;       // 4 KB
constexpr uint32_t kQB = 9 * kQChunkB;
constexpr uint32_t kPB = kTile * kRows * 2;            // 8 KB
constexpr uint32_t kSmem = kRing * kChunkB + kQB + kPB + 1024;
constexpr int kTmemCols = 256;           // S twice (2 x 32), O^T (4 x 32)
constexpr float kSlack = 8.f;            // octaves a score may exceed the maximum by

struct Ring {
  int pairs, ropes;                      // slots; pairs * 2 + ropes <= kRing
  int npair;                             // of a tile: C / 128
  int box;                               // tokens of a copy
};

struct Control {
  uint64_t full[kMaxPairs], empty[kMaxPairs], rfull[kMaxRopes], rempty[kMaxRopes];
  uint64_t s_full[2], q_ready, p_ready, o_done, drain;
  uint32_t tmem;
  int fail;
  unsigned bad[8];
  float top[4][kRows], sum[4][kRows], val[kRows];
  int lim[kRows];
  long long tmp[36];
};

// 16 values a lane, reduced over the warp: lanes l and l + 16 get column l's.
template <bool kMax>
__device__ __forceinline__ float columns(float (&v)[kMine], int lane) {
#pragma unroll
  for (int o = kMine / 2; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
      const float got = __shfl_xor_sync(0xffffffffu, give, o);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return kMax ? fmaxf(v[0], got) : v[0] + got;
}

__device__ __forceinline__ void softmax_barrier() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}
// Of the threads that have the same rows.
__device__ __forceinline__ void half_barrier(int half) {
  asm volatile("bar.sync %0, 128;" ::"r"(2 + half) : "memory");
}

// Whether the next tile is fetched into L2 while the slots that it will take are in use: where
// the row tiles of a text walk it in step, that is, each takes a whole number of parts and two
// CTAs are at the same tile at the same time.  In step: 64 heads, two texts of 131072 tokens
// 83 us, without 88; 19 of 13440 83 and 90; 128 heads, two of 65280 83 and 85.5.  Out of step
// it would cost 2 to 20 %: 64 heads, 32 texts of up to 16384 tokens 111 us, without 103; 12 of 21504
// 114.5 and 109; and so it would where one text has two row tiles (262272 tokens: 96 and 89).
__device__ __forceinline__ bool in_step(const Step &p, const Segment &g, long long total) {
  return p.B * p.row_tiles > 2 && (tiles_of(p, g.s) + p.extra) * parts_used(total) % total == 0;
}

__global__ void __launch_bounds__(kThreads, 1)
step_tc_kernel(const __grid_constant__ CUtensorMap map, const Step p, const Ring ring) {
  extern __shared__ __align__(1024) unsigned char raw[];
  __shared__ Control c;
  unsigned char *smem = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t s_ring = tc::smem_u32(smem);
  const uint32_t s_rope = s_ring + (uint32_t)ring.pairs * kPairB;
  const uint32_t s_q = s_ring + kRing * kChunkB, s_p = s_q + kQB;
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  if (tid == 0) {
    for (int i = 0; i < kMaxPairs; ++i) {
      tc::mbar_init(bar(c.full[i]), 1);
      tc::mbar_init(bar(c.empty[i]), 1);
    }
    for (int i = 0; i < kMaxRopes; ++i) {
      tc::mbar_init(bar(c.rfull[i]), 1);
      tc::mbar_init(bar(c.rempty[i]), 1);
    }
    tc::mbar_init(bar(c.s_full[0]), 1);
    tc::mbar_init(bar(c.s_full[1]), 1);
    tc::mbar_init(bar(c.q_ready), kSoftmax);
    tc::mbar_init(bar(c.p_ready), kSoftmax);
    tc::mbar_init(bar(c.o_done), 1);
    tc::mbar_init(bar(c.drain), 1);
    c.fail = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(tc::smem_u32(&c.tmem), kTmemCols);
  Cursor cur = {find_work(p, c.tmp), true};     // (its barriers cover the above)
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  start_next();
  const uint32_t tmem = c.tmem, t_o = tmem + 2 * kRows;
  const bool rope = p.R > 0;
  const Waits wait(&c.fail, (long long)p.max_pages * p.page);
  Segment g{};

  if (warp == 8) {
    // ---- copies: lane k has the tile's k-th box of tokens ----
    const int boxes = kTile / ring.box;
    const int log_page = __ffs(p.page) - 1;
    Slot pr = {0, 0}, rr = {0, 0};
    int np = 0, nr = 0;                    // copied, up to the slots there are
    bool ok = true;
    auto page_of = [&](int t) {            // -1: not there
      int pg = -1;
      if (lane < boxes && t < g.s.held) pg = p.table[(size_t)g.b * p.max_pages + (t >> log_page)];
      return pg >= 0 && pg < p.n_pages ? pg : -1;
    };
    int next = -1;
    while (ok && cur.next(p, g)) {
      bool ahead = false;
      for (int i = 0; ok && i < g.n; ++i) {
        const int t0 = (g.j0 + i) * kTile + lane * ring.box;
        if (i == 0) next = page_of(t0);
        const int pg = next;
        const bool there = pg >= 0;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, there)) *
                               (uint32_t)ring.box * kRowBytes;
        const int in_page = t0 & (p.page - 1);
        // the first pair, the rope chunk, the other pairs
        for (int k = 0; k < ring.npair; ++k) {
          ok = __all_sync(0xffffffffu, wait(bar(c.empty[pr.at]), pr.lap ^ 1u));
          if (!ok) break;
          const uint32_t full = bar(c.full[pr.at]);
          if (lane == 0) tc::mbar_expect_tx(full, 2 * bytes);
          __syncwarp();
          if (there) {
            const uint32_t dst = s_ring + (uint32_t)pr.at * kPairB + (uint32_t)lane * (uint32_t)ring.box * kRowBytes;
            tma_load_3d(dst, &map, k * 2 * kChunkCols, in_page, pg, full);
            tma_load_3d(dst + kChunkB, &map, (k * 2 + 1) * kChunkCols, in_page, pg, full);
          }
          pr.next(ring.pairs);
          np = min(np + 1, ring.pairs);
          if (k > 0) continue;
          next = i + 1 < g.n ? page_of(t0 + kTile) : -1;
          if (i == 0 && p.row_tiles > 1) ahead = in_step(p, g, cur.x.total);
          if (ahead && next >= 0)
            for (int x = 0; x < p.C + p.R; x += kChunkCols)
              tma_prefetch_3d(&map, x, (t0 + kTile) & (p.page - 1), next);
          if (!rope) continue;
          ok = __all_sync(0xffffffffu, wait(bar(c.rempty[rr.at]), rr.lap ^ 1u));
          if (!ok) break;
          const uint32_t rfull = bar(c.rfull[rr.at]);
          if (lane == 0) tc::mbar_expect_tx(rfull, bytes);
          __syncwarp();
          if (there)
            tma_load_3d(s_rope + (uint32_t)rr.at * kChunkB + (uint32_t)lane * (uint32_t)ring.box * kRowBytes,
                        &map, p.C, in_page, pg, rfull);
          rr.next(ring.ropes);
          nr = min(nr + 1, ring.ropes);
        }
      }
    }
    if (c.fail) {   // what is on its way comes in before the CTA ends
      auto drain = [](uint64_t *full, Slot s, int slots, int n) {
        for (; n > 0; --n) {               // the last n, from the latest back
          if (--s.at < 0) {
            s.at = slots - 1;
            s.lap ^= 1u;
          }
          tc::mbar_wait(tc::smem_u32(full + s.at), s.lap);
        }
      };
      drain(c.full, pr, ring.pairs, np);
      drain(c.rfull, rr, ring.ropes, nr);
    }
  } else if (warp == 9) {
    // ---- products: one thread ----
    if (elect_one()) {
      constexpr uint32_t id_s = tc::idesc_bf16(kTile, kRows, 0, 0),
                         id_o = tc::idesc_bf16(128, kRows, 1, 1);
      const uint64_t dp = tc::smem_desc(s_p, kTile * 16), dq0 = swizzled_desc(s_q, 16);
      // S (+)= a chunk of 64 channels
      auto chunk = [&](uint32_t t_s, uint32_t a, uint64_t dq, uint32_t old) {
        const uint64_t da = swizzled_desc(a, 16);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tc::mma_bf16(t_s, da + kStepK * e, dq + kStepK * e, id_s, e > 0 ? 1u : old);
      };
      Slot pr = {0, 0}, rr = {0, 0};
      uint32_t nt = 0, ns = 0;
      bool ok = true;
      while (ok && cur.next(p, g)) {
        ok = wait(bar(c.q_ready), ns & 1);
        ++ns;
        tc::tc_fence_after();
        // S of the next tile begins (its first pair and its rope chunk) while the
        // softmax works on this one, and goes on when O^T has made room for the rest
        Slot in = pr;
        auto begin = [&](uint32_t t) {
          const uint32_t t_s = tmem + (t & 1) * kRows;
          if (!wait(bar(c.full[in.at]), in.lap)) return false;
          const uint32_t a = s_ring + (uint32_t)in.at * kPairB;
          chunk(t_s, a, dq0, 0u);
          chunk(t_s, a + kChunkB, dq0 + kQChunkB / 16, 1u);
          in.next(ring.pairs);
          if (!rope) return true;
          if (!wait(bar(c.rfull[rr.at]), rr.lap)) return false;
          chunk(t_s, s_rope + (uint32_t)rr.at * kChunkB,
                dq0 + (uint64_t)(2 * ring.npair) * (kQChunkB / 16), 1u);
          tc::mma_commit(bar(c.rempty[rr.at]));
          rr.next(ring.ropes);
          return true;
        };
        ok = ok && begin(nt);
        for (int i = 0; ok && i < g.n; ++i, ++nt) {
          const uint32_t t_s = tmem + (nt & 1) * kRows;
          for (int k = 1; k < ring.npair; ++k) {
            ok = wait(bar(c.full[in.at]), in.lap);
            if (!ok) break;
            const uint32_t a = s_ring + (uint32_t)in.at * kPairB;
            const uint64_t dq = dq0 + (uint64_t)(2 * k) * (kQChunkB / 16);
            chunk(t_s, a, dq, 1u);
            chunk(t_s, a + kChunkB, dq + kQChunkB / 16, 1u);
            in.next(ring.pairs);
          }
          if (!ok) break;
          tc::mma_commit(bar(c.s_full[nt & 1]));
          if (i + 1 < g.n) ok = begin(nt + 1);
          ok = ok && wait(bar(c.p_ready), nt & 1);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t old = i > 0 ? 1u : 0u;
          for (int m = 0; m < ring.npair; ++m) {
            const uint64_t da = swizzled_desc(s_ring + (uint32_t)pr.at * kPairB, kChunkB);
#pragma unroll
            for (int e = 0; e < kTile / 16; ++e)
              tc::mma_bf16(t_o + (uint32_t)m * kRows, da + kStepRows * e, dp + 256 / 16 * e, id_o,
                           e > 0 ? 1u : old);
            tc::mma_commit(bar(c.empty[pr.at]));
            pr.next(ring.pairs);
          }
          tc::mma_commit(bar(c.o_done));
        }
      }
      if (c.fail) {
        tc::mma_commit(bar(c.drain));
        tc::mbar_wait(bar(c.drain), 0);
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: token tid & 127 of a tile, rows 16 half .. ----
    const int half = warp >> 2, token = tid & 127, quad = warp & 3;
    const float scale = p.scale * kLog2e;
    const int rows = p.T * p.H, log_page = __ffs(p.page) - 1;
    const uint32_t lanes = (uint32_t)quad << 21, col0 = (uint32_t)(kMine * half);
    Slot pr = {0, 0};
    uint32_t nt = 0;
    while (cur.next(p, g)) {
      const int r0 = g.rt * kRows;
      if (tid == 0) Cursor::note(p, g);
      // the queries, 8 channels a thread at a time, all on their way at once
      {
        const int r = r0 + lane, t = r / p.H, h = r - t * p.H;
        const bool live = r < rows;
        const unsigned long long q = live ? (unsigned long long)at<__nv_bfloat16>(p.q, p.q_s, g.b, t, h) : 0;
        const unsigned long long qr =
            live && rope ? (unsigned long long)at<__nv_bfloat16>(p.qr, p.qr_s, g.b, t, h) : 0;
        if (warp == 0) c.lim[lane] = live ? seen(p, g.s, r) : 0;
        const bool wide = __all_sync(0xffffffffu, ((q | qr) & 15) == 0);
        const int pieces = (p.C + (rope ? kChunkCols : 0)) / 8, held = (p.C + p.R) / 8;
#pragma unroll
        for (int k = 0; k < kRows / 8; ++k) {
          const int rr = warp + 8 * k;
          const unsigned long long q1 = __shfl_sync(0xffffffffu, q, rr),
                                   r1 = __shfl_sync(0xffffffffu, qr, rr);
          const uint32_t dst = s_q + (uint32_t)rr * kRowBytes;
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            const int i = lane + 32 * e;
            if (i >= pieces) break;
            const unsigned long long x = (i < p.C / 8 ? q1 + 16ull * i : r1 + 16ull * (i - p.C / 8));
            const uint32_t d = dst + (uint32_t)(i >> 3) * kQChunkB + (((i & 7) ^ (rr & 7)) << 4);
            if (q1 == 0 || i >= held) {
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(d), "r"(0) : "memory");
            } else if (wide) {
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(x) : "memory");
            } else {
              const unsigned short *u = reinterpret_cast<const unsigned short *>(x);
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) w[y] = u[2 * y] | (uint32_t)u[2 * y + 1] << 16;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(d), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      tc::fence_proxy_async();
      tc::mbar_arrive(bar(c.q_ready));
      softmax_barrier();
      float nb[kMine], l[kMine];
#pragma unroll
      for (int r = 0; r < kMine; ++r) nb[r] = 0.f, l[r] = 0.f;
      float mine = -INFINITY;       // the maximum that row col0 + (lane & 15) is scaled by
      for (int i = 0; i < g.n; ++i, ++nt) {
        const int k = (g.j0 + i) * kTile + token;
        int pg = -1;
        if (k < g.s.held) pg = p.table[(size_t)g.b * p.max_pages + (k >> log_page)];
        const bool there = pg >= 0 && pg < p.n_pages;
        wait(bar(c.s_full[nt & 1]), (nt >> 1) & 1);
        __syncwarp();
        tc::tc_fence_after();
        float v[kMine], w[kMine];
        tc::tmem_ld16(tmem + (nt & 1) * kRows + col0 + lanes, v);
#pragma unroll
        for (int r = 0; r < kMine; ++r) v[r] = there ? v[r] * scale : -INFINITY;
        if (p.T > 1) {
#pragma unroll
          for (int r = 0; r < kMine; ++r) v[r] = k < c.lim[col0 + r] ? v[r] : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < kMine; ++r) w[r] = v[r];
        const float top1 = columns<true>(w, lane);
        c.top[quad][col0 + (lane & 15)] = top1;
        half_barrier(half);
        const int mc = (int)col0 + (lane & 15);
        const float top = fmaxf(fmaxf(c.top[0][mc], c.top[1][mc]),
                                fmaxf(c.top[2][mc], c.top[3][mc]));
        const bool over = top > mine + kSlack;
        // O^T of the tile before has read P, and its sums stand still
        if (i > 0) wait(bar(c.o_done), (nt - 1) & 1);
        __syncwarp();
        if (__any_sync(0xffffffffu, over)) {
          const float now = fmaxf(mine, top);
          const float f = now == mine ? 1.f : exp2f(mine - now);
          mine = now;
          const float base = now == -INFINITY ? 0.f : now;
          float fr[kMine];
#pragma unroll
          for (int r = 0; r < kMine; ++r) {
            fr[r] = __shfl_sync(0xffffffffu, f, r);
            nb[r] = __shfl_sync(0xffffffffu, base, r);
            l[r] *= fr[r];
          }
          if (i > 0) {
            tc::tc_fence_after();
            for (int m = 0; m < ring.npair; ++m) {
              float x[kMine];
              uint32_t y[kMine];
              const uint32_t t = t_o + (uint32_t)m * kRows + col0 + lanes;
              tc::tmem_ld16(t, x);
#pragma unroll
              for (int r = 0; r < kMine; ++r) y[r] = __float_as_uint(x[r] * fr[r]);
              tmem_st16(t, y);
            }
            tmem_wait_st();
            tc::tc_fence_before();
          }
        }
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
          v[r] = tc::ex2(v[r] - nb[r]);
          l[r] += v[r];
        }
#pragma unroll
        for (int e = 0; e < kMine / 8; ++e) {
          const float x[8] = {v[8 * e],     v[8 * e + 1], v[8 * e + 2], v[8 * e + 3],
                              v[8 * e + 4], v[8 * e + 5], v[8 * e + 6], v[8 * e + 7]};
          tc::st_bf16x8(smem, (s_p - s_ring) + tc::mn_off((int)col0 + 8 * e, token, kTile), x);
        }
        // a token that is not there has a weight of 0: what lies in its place must
        // not be NaN (a chunk of each pair by either thread)
        if (!there) {
          const uint4 zero = make_uint4(0, 0, 0, 0);
          Slot in = pr;
          for (int m = 0; m < ring.npair; ++m) {
            wait(bar(c.full[in.at]), in.lap);
            unsigned char *d = smem + (uint32_t)in.at * kPairB + (uint32_t)half * kChunkB +
                               (uint32_t)token * kRowBytes;
            for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4 *>(d + 16 * e) = zero;
            in.next(ring.pairs);
          }
        }
        for (int m = 0; m < ring.npair; ++m) pr.next(ring.pairs);
        tc::fence_proxy_async();
        tc::tc_fence_before();
        tc::mbar_arrive(bar(c.p_ready));
      }
      // ---- the segment's end: O^T lane `token` of block m is latent 128 m + token ----
#pragma unroll
      for (int r = 0; r < kMine; ++r) nb[r] = l[r];
      const float part_l = columns<false>(nb, lane);
      const int mc = (int)col0 + (lane & 15);
      c.sum[quad][mc] = part_l;
      half_barrier(half);
      const float total = c.sum[0][mc] + c.sum[1][mc] + c.sum[2][mc] + c.sum[3][mc];
      if (quad == 0 && lane < 16) {
        const int r = r0 + mc;
        if (!g.whole) {
          reinterpret_cast<float2 *>(p.stats)[(size_t)g.slot * kRows + mc] = make_float2(mine, total);
        } else if (p.lse && r < rows) {
          p.lse[((size_t)g.b * p.H + r % p.H) * p.T + r / p.H] =
              total == 0.f ? -INFINITY : (mine + log2f(total)) * kLn2;
        }
        c.val[mc] = g.whole ? (total == 0.f ? 0.f : 1.f / total) : 1.f;
        const unsigned none = __ballot_sync(0xffffu, total == 0.f);
        if (g.whole && lane == 0) Cursor::note_none(p, g, half, none);
      }
      wait(bar(c.o_done), (nt - 1) & 1);
      half_barrier(half);
      tc::tc_fence_after();
      unsigned bad = 0;
      for (int m = 0; m < ring.npair; ++m) {
        float x[kMine];
        tc::tmem_ld16(t_o + (uint32_t)m * kRows + col0 + lanes, x);
        const int ch = m * 128 + token;
        if (g.whole) {
          __nv_bfloat16 *o =
              static_cast<__nv_bfloat16 *>(p.o) + ((size_t)g.b * rows + r0 + col0) * p.C + ch;
#pragma unroll
          for (int r = 0; r < kMine; ++r) {
            if (r0 + (int)col0 + r >= rows) break;
            const float f = c.val[col0 + r];
            const float y = f == 0.f ? 0.f : x[r] * f;
            if (!finite(y)) bad |= 1u << r;
            o[(size_t)r * p.C] = __float2bfloat16_rn(y);
          }
        } else {
          float *d = p.parts + ((size_t)g.slot * kRows + col0) * p.C + ch;
#pragma unroll
          for (int r = 0; r < kMine; ++r) d[(size_t)r * p.C] = x[r];
        }
      }
      tc::tc_fence_before();
      if (g.whole && p.T > 1) {
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (lane == 0) c.bad[warp] = bad;
        softmax_barrier();
        bad = c.bad[0] | c.bad[1] | c.bad[2] | c.bad[3] |
              (c.bad[4] | c.bad[5] | c.bad[6] | c.bad[7]) << kMine;
        for (int r = warp; r < kRows; r += 8)
          if (bad >> r & 1) step_row<__nv_bfloat16>(p, g.b, r0 + r, c.lim[r], lane);
      }
      softmax_barrier();      // c.lim, c.val and c.sum are written again
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (tid == 0 && c.fail) set_status(p.status, KDA_DEVICE_TIMEOUT);
  if (warp == 9) tc::tmem_dealloc(tmem, kTmemCols);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

}  // namespace

bool make_swizzled_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims,
                       const long long *strides, const uint32_t *box) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[4], st[3];
  cuuint32_t bx[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    bx[i] = box[i];
    if (i) st[i - 1] = (cuuint64_t)strides[i - 1] * 2;
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), d, st,
            bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool step_tc_ok(const Step &p) {
  return (reinterpret_cast<uintptr_t>(p.cache) & 15) == 0 && p.page >= 8 &&
         (p.page & (p.page - 1)) == 0 && p.token_stride >= p.C + p.R && p.token_stride % 8 == 0 &&
         (p.n_pages == 1 || (p.page_stride > 0 && p.page_stride % 8 == 0)) &&
         p.token_stride < (1ll << 38) && p.page_stride < (1ll << 38);
}

cudaError_t launch_step_tc(const Step &p, cudaStream_t s) {
  Ring r;
  r.npair = p.C / 128;
  // as many tiles ahead as fit: half of the next one beside 512 latents
  r.pairs = p.C == 512 ? 5 : 4;
  r.ropes = p.C == 512 ? 1 : 3;
  r.box = p.page < kTile ? p.page : kTile;
  CUtensorMap map;
  const uint64_t dims[3] = {(uint64_t)(p.C + p.R), (uint64_t)p.page, (uint64_t)p.n_pages};
  const long long strides[2] = {p.token_stride,
                                p.n_pages == 1 ? p.page * p.token_stride : p.page_stride};
  const uint32_t box[3] = {kChunkCols, (uint32_t)r.box, 1};
  if (!make_swizzled_map(&map, p.cache, 3, dims, strides, box)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(step_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSmem);
  if (e != cudaSuccess) return e;
  step_tc_kernel<<<kParts, kThreads, kSmem, s>>>(map, p, r);
  return cudaGetLastError();
}

}  // namespace latent
}  // namespace kda
