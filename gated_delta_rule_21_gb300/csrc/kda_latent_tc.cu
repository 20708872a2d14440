// kda_latent_tc.cu -- the expanded latent attention on the tensor cores, forward.
//
// A CTA has 256 queries of one head, as two tiles A and B of 128, and walks the
// keys in tiles of 128:
//     S = [Q | Qr] [K | Kr]^T    128 x 128, K: up to 192 channels
//     O += P V                   128 x V, P (bf16) in tensor memory over S
// One thread issues the products in the order PV_A, S_A of the next keys, PV_B, S_B of
// the next keys, so that the softmax of one tile runs beside the products of the
// other.  A softmax thread has a row of its own; the maximum that a row is scaled by
// moves only when a score exceeds it by 2^8, so O is hardly ever scaled.
//
// P is rounded to bf16 because both operands of an instruction have one type and V is bf16:
// o comes out 1.8e-3 to 2.1e-3 off in the 2-norm, where its own rounding alone makes 1.6e-3.
// The maximum, the sum of the weights (not rounded) and O are fp32.
//
// Shared memory (224 KB): the queries (3 chunks of 16 KB a tile), 4 chunks of keys, 2
// tiles of values (5 chunks and 3 chunks: 620 us instead of 485 for the row below).
// Tensor memory: S_A, S_B, O_A, O_B, 128 columns each.
//
// What bounds it: the products, 2300 of 3800 cycles a pair of tiles (58 cycles an
// instruction of N 128), and waiting for keys, which have no room to come earlier: a row of
// 8192 tokens, 32 heads of 128 + 64, 485 to 500 us (74 % of the measured rate of a large
// matrix product).  Where queries see few keys the softmax does: 25 packed runs 110 us.
#include "kda_f32x2.cuh"
#include "kda_latent_tc.cuh"

namespace kda {
namespace latent {
namespace {

constexpr int kRowsQ = 128;                     // of a tile, queries and keys
constexpr uint32_t kChunkB = kRowsQ * kRowBytes;   // 16 KB
constexpr int kKSlots = 4, kVSlots = 2;
constexpr int kThreads = 384;                   // A, B; copies, products, items and an idle warp
constexpr uint32_t kOffK = 6 * kChunkB, kOffV = kOffK + kKSlots * kChunkB;
constexpr uint32_t kOffC = kOffV + kVSlots * 2 * kChunkB;
constexpr uint32_t kFwdSmem = kOffC + 1024 + 1024;
constexpr float kSlack = 8.f;                   // octaves

struct Maps {
  CUtensorMap q, qr, k, kr, v;
};

// Key tiles [lo, hi) that a query tile sees.
struct Range {
  int lo, hi;
};
// Two query tiles of one head, and the key tiles that either sees.
struct Item {
  int b, h, pair;              // pair < 0: no more
  Range r[2];
  int all_lo[2];               // every row of a tile sees the keys from here on
  int jl, jh;
  __device__ __forceinline__ bool has(int x) const { return r[x].lo < r[x].hi; }
  __device__ __forceinline__ bool active(int x, int j) const {
    return j >= (x ? r[1].lo : r[0].lo) && j < (x ? r[1].hi : r[0].hi);
  }
};

struct FwdControl {
  uint64_t q_full[2], q_empty[2], k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots],
      v_empty[kVSlots];
  uint64_t s_full[2], p_ready[2], o_done[2], o_free[2], drain;
  uint64_t claim, item_full, item_empty;
  uint4 claimed;
  Item item;
  uint32_t tmem;
  int fail;
};

__device__ __forceinline__ Range keys_of(const Prompt &p, int b, int t) {
  if (t * kRowsQ >= p.T) return {0, 0};
  const int lo = run_start(p, b, t * kRowsQ) / kRowsQ;
  return {lo, lo > t ? lo : t + 1};
}
__device__ __forceinline__ Item make_item(const Prompt &p, unsigned index, int pairs) {
  // a head's keys stay in L2 while its queries are worked on, the longest first
  const int bh = (int)(index / (unsigned)pairs);
  Item m;
  m.pair = pairs - 1 - (int)(index % (unsigned)pairs);
  m.b = bh / p.H;
  m.h = bh % p.H;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = 2 * m.pair + x;
    m.r[x] = keys_of(p, m.b, t);
    m.all_lo[x] = t * kRowsQ < p.T ? run_start(p, m.b, min(p.T, (t + 1) * kRowsQ) - 1) : 0;
  }
  const bool a = m.has(0), z = m.has(1);
  m.jl = a && z ? min(m.r[0].lo, m.r[1].lo) : a ? m.r[0].lo : z ? m.r[1].lo : 0;
  m.jh = a && z ? max(m.r[0].hi, m.r[1].hi) : a ? m.r[0].hi : z ? m.r[1].hi : 0;
  return m;
}

// Asks for a CTA of this launch that has not begun; the answer comes to `dst` (16 bytes).
__device__ __forceinline__ void claim_next(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(dst),
      "r"(bar)
      : "memory");
}
// Whether there was one, and its index.
__device__ __forceinline__ bool claimed(uint32_t src, unsigned &index) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(src)
      : "memory");
  index = x;
  return ok != 0;
}

__global__ void __launch_bounds__(kThreads, 1)
prompt_fwd_tc_kernel(const __grid_constant__ Maps maps, const Prompt p) {
  extern __shared__ __align__(1024) unsigned char raw[];
  unsigned char *smem = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
  FwdControl &c = *reinterpret_cast<FwdControl *>(smem + kOffC);
  const uint32_t s0 = tc::smem_u32(smem);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int pairs = (p.T + 2 * kRowsQ - 1) / (2 * kRowsQ);
  const int nk = (p.K + kChunkCols - 1) / kChunkCols, nc = nk + (p.R > 0 ? 1 : 0);
  const int nv = (p.V + kChunkCols - 1) / kChunkCols;
  auto bar = [](uint64_t &x) { return tc::smem_u32(&x); };
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(c.q_full[i]), 1);
      tc::mbar_init(bar(c.q_empty[i]), 1);
      tc::mbar_init(bar(c.v_full[i]), 1);
      tc::mbar_init(bar(c.v_empty[i]), 1);
      tc::mbar_init(bar(c.s_full[i]), 1);
      tc::mbar_init(bar(c.p_ready[i]), 128);
      tc::mbar_init(bar(c.o_done[i]), 1);
      tc::mbar_init(bar(c.o_free[i]), 128);
    }
    for (int i = 0; i < kKSlots; ++i) {
      tc::mbar_init(bar(c.k_full[i]), 1);
      tc::mbar_init(bar(c.k_empty[i]), 1);
    }
    tc::mbar_init(bar(c.drain), 1);
    tc::mbar_init(bar(c.claim), 1);
    tc::mbar_init(bar(c.item_full), 1);
    tc::mbar_init(bar(c.item_empty), 256 + 2);
    c.fail = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(tc::smem_u32(&c.tmem), 512);
  after_previous();        // the table of runs
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = c.tmem;
  const Waits wait(&c.fail, p.T);
  // the next item, by every thread that works on them
  auto next_item = [&](Item &m, uint32_t round) {
    const bool ok = wait(bar(c.item_full), round & 1);
    m = c.item;
    if (!ok) m.pair = -1;
    tc::mbar_arrive(bar(c.item_empty));
    return m.pair >= 0;
  };

  if (warp >= 8) {
    few_registers();
    if (warp == 10) {
      // ---- items: this CTA's own, then those of CTAs that have not begun ----
      if (lane == 0) {
        bool ok = true;
        unsigned index = blockIdx.x;
        for (uint32_t round = 0; ok; ++round) {
          if (round > 0) {
            // (asked for once everyone has begun the item before)
            if (!wait(bar(c.item_empty), (round - 1) & 1)) break;
            tc::mbar_expect_tx(bar(c.claim), 16);
            claim_next(tc::smem_u32(&c.claimed), bar(c.claim));
            if (!wait(bar(c.claim), (round - 1) & 1)) break;
            ok = claimed(tc::smem_u32(&c.claimed), index);
            tc::fence_proxy_async();
          }
          if (ok) c.item = make_item(p, index, pairs);
          else c.item.pair = -1;
          tc::mbar_arrive(bar(c.item_full));
        }
      }
      __syncwarp();
    } else if (warp == 8) {
      // ---- copies ----
      if (lane == 0) {
        uint32_t kn = 0, vn = 0, qn[2] = {0, 0};
        bool ok = true;
        Item m{};
        auto load_q = [&](int x) {
          ok = wait(bar(c.q_empty[x]), (qn[x] + 1) & 1);
          if (!ok) return;
          const int t = (2 * m.pair + x) * kRowsQ;
          const uint32_t full = bar(c.q_full[x]);
          tc::mbar_expect_tx(full, (uint32_t)nc * kChunkB);
          for (int i = 0; i < nk; ++i)
            tma_load_4d(s0 + (uint32_t)(3 * x + i) * kChunkB, &maps.q, i * kChunkCols, m.h, t, m.b,
                        full);
          if (nc > nk)
            tma_load_4d(s0 + (uint32_t)(3 * x + nk) * kChunkB, &maps.qr, 0, m.h, t, m.b, full);
          ++qn[x];
        };
        auto load_k = [&](int j) {
          for (int i = 0; i < nc; ++i, ++kn) {
            const uint32_t s = kn % kKSlots;
            ok = wait(bar(c.k_empty[s]), (kn / kKSlots + 1) & 1);
            if (!ok) return;
            const uint32_t full = bar(c.k_full[s]), d = s0 + kOffK + s * kChunkB;
            tc::mbar_expect_tx(full, kChunkB);
            if (i < nk) tma_load_4d(d, &maps.k, i * kChunkCols, m.h, j * kRowsQ, m.b, full);
            else tma_load_4d(d, &maps.kr, 0, 0, j * kRowsQ, m.b, full);
          }
        };
        for (uint32_t round = 0; ok && next_item(m, round); ++round) {
          if (m.jl >= m.jh) continue;
          if (m.has(0)) load_q(0);
          if (ok) load_k(m.jl);
          if (ok && m.has(1)) load_q(1);
          for (int j = m.jl; ok && j < m.jh; ++j) {
            const uint32_t s = vn % kVSlots;
            ok = wait(bar(c.v_empty[s]), (vn / kVSlots + 1) & 1);
            if (!ok) break;
            const uint32_t full = bar(c.v_full[s]);
            tc::mbar_expect_tx(full, (uint32_t)nv * kChunkB);
            for (int i = 0; i < nv; ++i)
              tma_load_4d(s0 + kOffV + (2 * s + (uint32_t)i) * kChunkB, &maps.v, i * kChunkCols, m.h,
                          j * kRowsQ, m.b, full);
            ++vn;
            if (j + 1 < m.jh) load_k(j + 1);
          }
        }
        if (c.fail) {   // what is on its way comes in before the CTA ends
          for (int x = 0; x < 2; ++x)
            if (qn[x]) tc::mbar_wait(bar(c.q_full[x]), (qn[x] - 1) & 1);
          for (uint32_t k = kn > kKSlots ? kn - kKSlots : 0; k < kn; ++k)
            tc::mbar_wait(bar(c.k_full[k % kKSlots]), (k / kKSlots) & 1);
          for (uint32_t k = vn > kVSlots ? vn - kVSlots : 0; k < vn; ++k)
            tc::mbar_wait(bar(c.v_full[k % kVSlots]), (k / kVSlots) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---- products: one thread ----
      if (elect_one()) {
        constexpr uint32_t id_s = tc::idesc_bf16(128, 128, 0, 0);
        const uint32_t id_o = tc::idesc_bf16(128, nv * kChunkCols, 0, 1);
        bool ok = true;
        // of all items: products S, and items, of a tile; key chunks and value tiles
        uint32_t sn[2] = {0, 0}, qn[2] = {0, 0}, kn = 0, vn = 0;
        Item m{};
        for (uint32_t round = 0; ok && next_item(m, round); ++round) {
          for (int j = m.jl - 1; ok && j < m.jh; ++j) {
            const bool now = j >= m.jl;
            for (int x = 0; ok && x < 2; ++x) {
              const int lo = x ? m.r[1].lo : m.r[0].lo, hi = x ? m.r[1].hi : m.r[0].hi;
              const bool on = now && j >= lo && j < hi;
              if (on) {
                // the rows of the item before have been read
                if (j == lo) ok = wait(bar(c.o_free[x]), qn[x] & 1);
                ok = ok && wait(bar(c.p_ready[x]), (sn[x] - 1) & 1) &&
                     wait(bar(c.v_full[vn % kVSlots]), (vn / kVSlots) & 1);
                if (!ok) break;
                tc::tc_fence_after();
                const uint64_t dv =
                    swizzled_desc(s0 + kOffV + 2 * (vn % kVSlots) * kChunkB, kChunkB);
                const uint32_t old = j > lo ? 1u : 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  mma_bf16_ts(tmem + 256 + 128 * x, tmem + 128 * x + 8 * e, dv + kStepRows * e,
                              id_o, e > 0 ? 1u : old);
              }
              if (j + 1 >= lo && j + 1 < hi) {
                if (j + 1 == lo) {
                  ok = wait(bar(c.q_full[x]), qn[x] & 1);
                  if (!ok) break;
                  ++qn[x];
                }
                const bool last = x == 1 || !m.active(1, j + 1);
                for (int i = 0; i < nc; ++i) {
                  const uint32_t k = kn + (uint32_t)i, s = k % kKSlots;
                  ok = wait(bar(c.k_full[s]), (k / kKSlots) & 1);
                  if (!ok) break;
                  const uint64_t da = swizzled_desc(s0 + (uint32_t)(3 * x + i) * kChunkB, 16),
                                 dk = swizzled_desc(s0 + kOffK + s * kChunkB, 16);
                  const uint32_t old = i > 0 ? 1u : 0u;
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    tc::mma_bf16(tmem + 128 * x, da + kStepK * e, dk + kStepK * e, id_s,
                                 e > 0 ? 1u : old);
                  if (last) tc::mma_commit(bar(c.k_empty[s]));
                }
                if (!ok) break;
                tc::mma_commit(bar(c.s_full[x]));
                ++sn[x];
                if (j + 2 == hi) tc::mma_commit(bar(c.q_empty[x]));
                if (last) kn += (uint32_t)nc;
              }
              if (on && j + 1 == hi) tc::mma_commit(bar(c.o_done[x]));
            }
            if (ok && now) {
              tc::mma_commit(bar(c.v_empty[vn % kVSlots]));
              ++vn;
            }
          }
        }
        if (c.fail) {
          tc::mma_commit(bar(c.drain));
          tc::mbar_wait(bar(c.drain), 0);
        }
      }
      __syncwarp();
    }
  } else {
    many_registers();
    // ---- softmax: a row a thread ----
    const int x = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t t_s = tmem + 128 * x + lanes, t_o = tmem + 256 + 128 * x + lanes;
    // (Not negative.  At 0 the products are set to 0 before the mask, whose -inf times 0
    // would be NaN and every row made again key by key: a call on 2048 tokens of 4 heads takes
    // 59 us, so 78 ms.)
    const float scale = p.scale == 0.f ? 1.f : p.scale * kLog2e;
    const u64 scale2 = pk2(scale, scale);
    uint32_t sn = 0, items = 0;
    Item m0{};
    for (uint32_t round = 0; __all_sync(0xffffffffu, next_item(m0, round)); ++round) {
      const int b = m0.b, h = m0.h, tile = 2 * m0.pair + x, row = tile * kRowsQ + (tid & 127);
      const Range r = x ? m0.r[1] : m0.r[0];
      const int all_lo = x ? m0.all_lo[1] : m0.all_lo[0];
      const int lo = row < p.T ? run_start(p, b, row) : 0x7fffffff;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = r.lo; j < r.hi; ++j, ++sn) {
        wait(bar(c.s_full[x]), sn & 1);
        __syncwarp();
        tc::tc_fence_after();
        uint32_t u[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32_nw(t_s + 32 * i, u[i]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) reg_fence32(u[i]);
        if (p.scale == 0.f) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            u[i >> 5][i & 31] = __float_as_uint(__uint_as_float(u[i >> 5][i & 31]) * 0.f);
        }
        if (j == tile || j * kRowsQ < all_lo) {
          // a warp's rows see most groups of 32 keys whole or not at all
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t on = column_bits(lo, row + 1, j * kRowsQ + 32 * i);
            if (!__all_sync(0xffffffffu, on == 0xffffffffu)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(on >> e & 1u)) u[i][e] = 0xff800000u;   // -inf
            }
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 128; ++i) top = fmaxf(top, __uint_as_float(u[i >> 5][i & 31]));
        top *= scale;
        const bool over = top > m + kSlack;
        if (__any_sync(0xffffffffu, over)) {
          const float now = over ? top : m;
          const float f = over ? exp2f(m - now) : 1.f;
          m = now;
          l *= f;
          if (j > r.lo) {      // PV of the keys before is done: S of these came after it
#pragma unroll 1
            for (int q = 0; q < 2 * nv; ++q) {
              uint32_t o[32];
              tmem_ld32_wait(t_o + 32 * q, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(t_o + 32 * q, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        const u64 nb = pk2(-base, -base);
        u64 sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, d;
            upk2(fma2(pk2(__uint_as_float(u[i][2 * e]), __uint_as_float(u[i][2 * e + 1])), scale2,
                      nb),
                 a, d);
            a = tc::ex2(a);
            d = tc::ex2(d);
            sum = add2(sum, pk2(a, d));
            w[e] = tc::pack_bf16(a, d);
          }
          tmem_st16(t_s + 16 * i, w);
        }
        float a, d;
        upk2(sum, a, d);
        l += a + d;
        tmem_wait_st();
        tc::tc_fence_before();
        tc::mbar_arrive(bar(c.p_ready[x]));
      }
      // ---- the rows ----
      const bool any = r.lo < r.hi;
      if (any) {
        wait(bar(c.o_done[x]), items & 1);
        __syncwarp();
        tc::tc_fence_after();
        ++items;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l, none = no_weights(lo <= row);
      bool bad = false;
      __nv_bfloat16 *o =
          static_cast<__nv_bfloat16 *>(p.o) + (((size_t)b * p.T + row) * p.H + h) * p.V;
#pragma unroll 1
      for (int q = 0; q < p.V / 32; ++q) {
        uint32_t y[32];
        if (any) {
          tmem_ld32_wait(t_o + 32 * q, y);
          if (q + 1 == p.V / 32) {     // the next item's products may write there
            tc::tc_fence_before();
            tc::mbar_arrive(bar(c.o_free[x]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = 0;
        }
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a = l == 0.f ? none : __uint_as_float(y[2 * i]) * inv;
          const float d = l == 0.f ? none : __uint_as_float(y[2 * i + 1]) * inv;
          bad |= !finite(a) || !finite(d);
          w[i] = tc::pack_bf16(a, d);
        }
        if (row < p.T) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint4 *>(o + 32 * q)[i] =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        __syncwarp();
      }
      __syncwarp();
      if (p.lse && row < p.T)
        p.lse[((size_t)b * p.H + h) * p.T + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      unsigned which = __ballot_sync(0xffffffffu, bad && row < p.T);
      __syncwarp();
      for (; which; which &= which - 1)
        forward_row<__nv_bfloat16>(p, b, h, row - lane + __ffs(which) - 1, lane);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (tid == 0 && c.fail) set_status(p.status, KDA_DEVICE_TIMEOUT);
  if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

bool stride_ok(long long s, int n) { return n == 1 || (s > 0 && s % 8 == 0 && s < (1ll << 38)); }
bool tensor_ok(const void *x, const Strides &s, const Prompt &p, bool heads) {
  return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && stride_ok(s.b, p.B) &&
         stride_ok(s.t, p.T) && (!heads || stride_ok(s.h, p.H));
}

}  // namespace

// (The stride of a dimension of 1 is never used.)
bool prompt_map(CUtensorMap *m, const void *x, const Strides &s, const Prompt &p, int heads, int n,
                int rows) {
  const uint64_t dims[4] = {(uint64_t)n, (uint64_t)heads, (uint64_t)p.T, (uint64_t)p.B};
  const long long strides[3] = {heads > 1 ? s.h : 8, p.T > 1 ? s.t : 8, p.B > 1 ? s.b : 8};
  const uint32_t box[4] = {kChunkCols, 1, (uint32_t)rows, 1};
  return make_swizzled_map(m, x, 4, dims, strides, box);
}

bool prompt_tc_ok(const Prompt &p) {
  return tensor_ok(p.q, p.q_s, p, true) && tensor_ok(p.k, p.k_s, p, true) &&
         tensor_ok(p.v, p.v_s, p, true) &&
         (p.R == 0 || (tensor_ok(p.qr, p.qr_s, p, true) && tensor_ok(p.kr, p.kr_s, p, false)));
}

cudaError_t launch_prompt_tc(const Prompt &p, cudaStream_t s) {
  Maps m;
  if (!prompt_map(&m.q, p.q, p.q_s, p, p.H, p.K, kRowsQ) ||
      !prompt_map(&m.k, p.k, p.k_s, p, p.H, p.K, kRowsQ) ||
      !prompt_map(&m.v, p.v, p.v_s, p, p.H, p.V, kRowsQ))
    return cudaErrorInvalidValue;
  m.qr = m.kr = m.q;
  if (p.R && (!prompt_map(&m.qr, p.qr, p.qr_s, p, p.H, p.R, kRowsQ) ||
              !prompt_map(&m.kr, p.kr, p.kr_s, p, 1, p.R, kRowsQ)))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(prompt_fwd_tc_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFwdSmem);
  if (e != cudaSuccess) return e;
  const unsigned pairs = (unsigned)((p.T + 2 * kRowsQ - 1) / (2 * kRowsQ));
  const unsigned grid = pairs * (unsigned)(p.B * p.H);
  if (p.start)             // it gets ready while the table of runs is made
    return launch_next(prompt_fwd_tc_kernel, dim3(grid), kThreads, kFwdSmem, s, m, p);
  prompt_fwd_tc_kernel<<<grid, kThreads, kFwdSmem, s>>>(m, p);
  return cudaGetLastError();
}

}  // namespace latent
}  // namespace kda
