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
// Threads: warps 0 to 3 the softmax, a thread a token (the running maxima of the 32
// rows are the same in all of them, and only move when a score exceeds them by
// 2^8, so the sums in tensor memory are hardly ever scaled); warp 4 the copies; warp
// 5 the products.
#include "kda_latent_tc.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kThreads = 192;
constexpr int kSoftmax = 128;            // threads
constexpr uint32_t kChunkB = kTile * kRowBytes;        // 16 KB
constexpr uint32_t kPairB = 2 * kChunkB;
constexpr int kRing = 11;                // chunks in shared memory
constexpr int kMaxPairs = 5, kMaxRopes = 5;
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
  unsigned bad[4];
  float top[4][kRows], sum[4][kRows], val[kRows];
  int lim[kRows];
  long long tmp[36];
};

// A sequence's tiles [j0, j0 + n) for the rows of row tile rt.
struct Segment {
  int b, rt, j0, n;
  bool whole, first;
  Seq s;
};
struct Cursor {
  Work x;
  bool first;
  __device__ __forceinline__ bool next(const Step &p, Segment &g) {
    while (x.unit < x.end) {
      g.s = seq_of(p, x.b);
      const int tiles = tiles_of(g.s);
      if (x.off >= (long long)tiles * p.row_tiles) {
        ++x.b;
        x.off = 0;
        continue;
      }
      g.b = x.b;
      g.rt = (int)(x.off / tiles);
      g.j0 = (int)(x.off % tiles);
      g.n = (int)min((long long)(tiles - g.j0), x.end - x.unit);
      g.whole = g.n == tiles;
      g.first = first;
      first = false;
      x.unit += g.n;
      x.off += g.n;
      return true;
    }
    return false;
  }
};

// 32 values a lane, reduced over the warp: lane l gets column l's.
template <bool kMax>
__device__ __forceinline__ float columns(float (&v)[kRows], int lane) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
      const float got = __shfl_xor_sync(0xffffffffu, give, o);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

__device__ __forceinline__ void softmax_barrier() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
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
  if (warp == 5) tc::tmem_alloc(tc::smem_u32(&c.tmem), kTmemCols);
  Cursor cur = {find_work(p, c.tmp), true};     // (its barriers cover the above)
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  start_next();
  const uint32_t tmem = c.tmem, t_o = tmem + 2 * kRows;
  const bool rope = p.R > 0;
  volatile int *fail = &c.fail;
  Segment g;

  if (warp == 4) {
    // ---- copies: lane k has the tile's k-th box of tokens ----
    const int boxes = kTile / ring.box;
    const int log_page = __ffs(p.page) - 1;
    Slot pr = {0, 0}, rr = {0, 0};
    int np = 0, nr = 0;                    // copied, up to the slots there are
    bool ok = true;
    while (ok && cur.next(p, g)) {
      for (int i = 0; ok && i < g.n; ++i) {
        const int t0 = (g.j0 + i) * kTile + lane * ring.box;
        int pg = -1;
        if (lane < boxes && t0 < g.s.held) pg = p.table[(size_t)g.b * p.max_pages + (t0 >> log_page)];
        const bool there = pg >= 0 && pg < p.n_pages;
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, there)) *
                               (uint32_t)ring.box * kRowBytes;
        const int in_page = t0 & (p.page - 1);
        // the first pair, the rope chunk, the other pairs
        for (int k = 0; k < ring.npair; ++k) {
          ok = __all_sync(0xffffffffu, wait_or_fail(bar(c.empty[pr.at]), pr.lap ^ 1u, fail));
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
          if (k > 0 || !rope) continue;
          ok = __all_sync(0xffffffffu, wait_or_fail(bar(c.rempty[rr.at]), rr.lap ^ 1u, fail));
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
    if (*fail) {   // what is on its way comes in before the CTA ends
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
  } else if (warp == 5) {
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
        ok = wait_or_fail(bar(c.q_ready), ns & 1, fail);
        ++ns;
        tc::tc_fence_after();
        for (int i = 0; ok && i < g.n; ++i, ++nt) {
          const uint32_t t_s = tmem + (nt & 1) * kRows;
          Slot in = pr;
          for (int k = 0; k < ring.npair; ++k) {
            ok = wait_or_fail(bar(c.full[in.at]), in.lap, fail);
            if (!ok) break;
            const uint32_t a = s_ring + (uint32_t)in.at * kPairB;
            const uint64_t dq = dq0 + (uint64_t)(2 * k) * (kQChunkB / 16);
            chunk(t_s, a, dq, k > 0 ? 1u : 0u);
            chunk(t_s, a + kChunkB, dq + kQChunkB / 16, 1u);
            in.next(ring.pairs);
            if (k > 0 || !rope) continue;
            ok = wait_or_fail(bar(c.rfull[rr.at]), rr.lap, fail);
            if (!ok) break;
            chunk(t_s, s_rope + (uint32_t)rr.at * kChunkB,
                  dq0 + (uint64_t)(2 * ring.npair) * (kQChunkB / 16), 1u);
            tc::mma_commit(bar(c.rempty[rr.at]));
            rr.next(ring.ropes);
          }
          if (!ok) break;
          tc::mma_commit(bar(c.s_full[nt & 1]));
          ok = wait_or_fail(bar(c.p_ready), nt & 1, fail);
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
      if (*fail) {
        tc::mma_commit(bar(c.drain));
        tc::mbar_wait(bar(c.drain), 0);
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: thread tid has token tid of a tile ----
    const float scale = p.scale * kLog2e;
    const int rows = p.T * p.H;
    const uint32_t my_lane = (uint32_t)warp << 21;       // 32 lanes a warp
    const int log_page = __ffs(p.page) - 1;
    Slot pr = {0, 0};
    uint32_t nt = 0;
    while (cur.next(p, g)) {
      const int r0 = g.rt * kRows;
      // the queries, 8 channels a thread at a time, all on their way at once
      const int pieces = (p.C + (rope ? kChunkCols : 0)) / 8;
      for (int rr = warp; rr < kRows; rr += 4) {
        const int r = r0 + rr, t = r / p.H, h = r % p.H;
        const bool live = r < rows;
        const __nv_bfloat16 *q = live ? at<__nv_bfloat16>(p.q, p.q_s, g.b, t, h) : nullptr;
        const __nv_bfloat16 *qr =
            live && rope ? at<__nv_bfloat16>(p.qr, p.qr_s, g.b, t, h) : nullptr;
        const bool wide = ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(qr)) & 15) == 0;
        for (int i = lane; i < pieces; i += 32) {
          const int ch = i * 8;
          const __nv_bfloat16 *x = ch < p.C ? q + ch : qr + (ch - p.C);
          const uint32_t off = (s_q - s_ring) + (uint32_t)(ch / kChunkCols) * kQChunkB +
                               piece_off(rr, (ch % kChunkCols) / 8);
          if (live && ch < p.C + p.R && wide) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s_ring + off), "l"(x)
                         : "memory");
            continue;
          }
          uint32_t w[4] = {0, 0, 0, 0};
          if (live && ch < p.C + p.R) {
            const unsigned short *u = reinterpret_cast<const unsigned short *>(x);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = u[2 * e] | (uint32_t)u[2 * e + 1] << 16;
          }
          *reinterpret_cast<uint4 *>(smem + off) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (tid < kRows) c.lim[tid] = r0 + tid < rows ? seen(p, g.s, r0 + tid) : 0;
      tc::fence_proxy_async();
      tc::mbar_arrive(bar(c.q_ready));
      softmax_barrier();
      float nb[kRows], l[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) nb[r] = 0.f, l[r] = 0.f;
      float mine = -INFINITY;             // the maximum that row `lane` is scaled by
      for (int i = 0; i < g.n; ++i, ++nt) {
        const int k = (g.j0 + i) * kTile + tid;
        int pg = -1;
        if (k < g.s.held) pg = p.table[(size_t)g.b * p.max_pages + (k >> log_page)];
        const bool there = pg >= 0 && pg < p.n_pages;
        wait_or_fail(bar(c.s_full[nt & 1]), (nt >> 1) & 1, fail);
        __syncwarp();
        tc::tc_fence_after();
        uint32_t u[32];
        tmem_ld32_wait(tmem + (nt & 1) * kRows + my_lane, u);
        float v[kRows], w[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) v[r] = there ? __uint_as_float(u[r]) * scale : -INFINITY;
        if (p.T > 1) {
#pragma unroll
          for (int r = 0; r < kRows; ++r) v[r] = k < c.lim[r] ? v[r] : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) w[r] = v[r];
        const float top1 = columns<true>(w, lane);
        c.top[warp][lane] = top1;
        softmax_barrier();
        const float top = fmaxf(fmaxf(c.top[0][lane], c.top[1][lane]),
                                fmaxf(c.top[2][lane], c.top[3][lane]));
        const bool over = top > mine + kSlack;
        // O^T of the tile before has read P, and its sums stand still
        if (i > 0) wait_or_fail(bar(c.o_done), (nt - 1) & 1, fail);
        __syncwarp();
        if (__any_sync(0xffffffffu, over)) {
          const float now = fmaxf(mine, top);
          const float f = now == mine ? 1.f : exp2f(mine - now);
          mine = now;
          const float base = now == -INFINITY ? 0.f : now;
          float fr[kRows];
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            fr[r] = __shfl_sync(0xffffffffu, f, r);
            nb[r] = __shfl_sync(0xffffffffu, base, r);
            l[r] *= fr[r];
          }
          if (i > 0) {
            tc::tc_fence_after();
            for (int m = 0; m < ring.npair; ++m) {
              uint32_t x[32];
              tmem_ld32_wait(t_o + (uint32_t)m * kRows + my_lane, x);
#pragma unroll
              for (int r = 0; r < kRows; ++r)
                x[r] = __float_as_uint(__uint_as_float(x[r]) * fr[r]);
              tmem_st32(t_o + (uint32_t)m * kRows + my_lane, x);
            }
            tmem_wait_st();
            tc::tc_fence_before();
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          v[r] = tc::ex2(v[r] - nb[r]);
          l[r] += v[r];
        }
#pragma unroll
        for (int e = 0; e < kRows / 8; ++e) {
          const float x[8] = {v[8 * e],     v[8 * e + 1], v[8 * e + 2], v[8 * e + 3],
                              v[8 * e + 4], v[8 * e + 5], v[8 * e + 6], v[8 * e + 7]};
          tc::st_bf16x8(smem, (s_p - s_ring) + tc::mn_off(8 * e, tid, kTile), x);
        }
        // a token that is not there has a weight of 0: what lies in its place must
        // not be NaN
        if (!there) {
          const uint4 zero = make_uint4(0, 0, 0, 0);
          Slot in = pr;
          for (int m = 0; m < ring.npair; ++m) {
            wait_or_fail(bar(c.full[in.at]), in.lap, fail);
            unsigned char *d = smem + (uint32_t)in.at * kPairB + (uint32_t)tid * kRowBytes;
            for (int e = 0; e < 8; ++e) {
              *reinterpret_cast<uint4 *>(d + 16 * e) = zero;
              *reinterpret_cast<uint4 *>(d + kChunkB + 16 * e) = zero;
            }
            in.next(ring.pairs);
          }
        }
        for (int m = 0; m < ring.npair; ++m) pr.next(ring.pairs);
        tc::fence_proxy_async();
        tc::tc_fence_before();
        tc::mbar_arrive(bar(c.p_ready));
      }
      // ---- the segment's end: O^T lane tid of block m is latent 128 m + tid ----
#pragma unroll
      for (int r = 0; r < kRows; ++r) nb[r] = l[r];
      const float part_l = columns<false>(nb, lane);
      c.sum[warp][lane] = part_l;
      softmax_barrier();
      const float total = c.sum[0][lane] + c.sum[1][lane] + c.sum[2][lane] + c.sum[3][lane];
      const int slot = 2 * blockIdx.x + (g.first ? 0 : 1);
      if (warp == 0) {
        const int r = r0 + lane;
        if (!g.whole) {
          p.stats[2 * ((size_t)slot * kRows + lane)] = mine;
          p.stats[2 * ((size_t)slot * kRows + lane) + 1] = total;
        } else if (p.lse && r < rows) {
          p.lse[((size_t)g.b * p.H + r % p.H) * p.T + r / p.H] =
              total == 0.f ? -INFINITY : (mine + log2f(total)) * kLn2;
        }
        c.val[lane] = g.whole ? (total == 0.f ? 0.f : 1.f / total) : 1.f;
      }
      wait_or_fail(bar(c.o_done), (nt - 1) & 1, fail);
      softmax_barrier();
      tc::tc_fence_after();
      unsigned bad = 0;
      for (int m = 0; m < ring.npair; ++m) {
        uint32_t x[32];
        tmem_ld32_wait(t_o + (uint32_t)m * kRows + my_lane, x);
        const int ch = m * 128 + tid;
        if (g.whole) {
          __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + ((size_t)g.b * rows + r0) * p.C + ch;
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            if (r0 + r >= rows) break;
            const float f = c.val[r];
            const float y = f == 0.f ? 0.f : __uint_as_float(x[r]) * f;
            if (!finite(y)) bad |= 1u << r;
            o[(size_t)r * p.C] = __float2bfloat16_rn(y);
          }
        } else {
          float *d = p.parts + (size_t)slot * kRows * p.C + ch;
#pragma unroll
          for (int r = 0; r < kRows; ++r) d[(size_t)r * p.C] = __uint_as_float(x[r]);
        }
      }
      tc::tc_fence_before();
      if (g.whole && p.T > 1) {
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (lane == 0) c.bad[warp] = bad;
        softmax_barrier();
        bad = c.bad[0] | c.bad[1] | c.bad[2] | c.bad[3];
        for (int r = warp; r < kRows; r += 4)
          if (bad >> r & 1) step_row<__nv_bfloat16>(p, g.b, r0 + r, c.lim[r], lane);
      }
      softmax_barrier();      // c.lim, c.val and c.sum are written again
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (tid == 0 && c.fail) set_status(p.status, KDA_DEVICE_TIMEOUT);
  if (warp == 5) tc::tmem_dealloc(tmem, kTmemCols);
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
  r.pairs = p.C == 512 ? 5 : p.C == 256 ? 4 : 3;
  r.ropes = p.C == 512 ? 1 : p.C == 256 ? 2 : 3;
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
