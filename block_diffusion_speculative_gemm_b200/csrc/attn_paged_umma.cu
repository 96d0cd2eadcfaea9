// Paged chunk attention for many rows per kv head (prompts, long chunks) on
// the 5th-generation tensor cores: the formulas of attn_paged.cu with a
// thread per row.
//
// An item is two query tiles of 128 rows (tokens x query heads of a kv head)
// against 128-key tiles.  S = Q K^T (UMMA 128 x 128) lands in TMEM; a softmax
// thread owns one row, i.e. one TMEM lane, so the row maximum and sum need no
// exchange; it writes P over the first half of S's columns in the operand
// type, and O += P V takes P straight from TMEM (A operand) with V as the
// MN-major B operand.  Per CTA (one per SM):
//
//   warps 0-3, 4-7  softmax of query tile 0 and 1, and their results
//   warp 8          TMA: K and V tiles through one ring of slots, Q per item
//   warp 9          MMA issue: QK0(j), PV1(j-1), QK1(j), PV0(j), ...
//
// so the tensor cores work on one query tile while the other one is in its
// softmax.  S of a tile is overwritten by the next product only after P of it
// has been read, which the issue order alone guarantees.  O is rescaled in
// TMEM only when a row's maximum grew by more than 2^8 since its reference was
// set (weights then stay below 2^8, exact enough in fp32 sums and inside
// fp16); normalisation happens once, at the end.
//
// Bound by the tensor cores and, equally, by the exponentials: 4 x 128 x 128 x
// HD flop and 2 x 128 x 128 exponentials per pair of tiles.
#include <algorithm>

#include "attn_paged.cuh"

namespace dflash {

namespace {

constexpr int kKT = 128;          // keys per tile
constexpr int kQT = 128;          // rows per query tile
constexpr int kThreads = 384;     // three warpgroups: softmax 0, softmax 1, TMA + MMA
constexpr int kMaxSlots = 12;
constexpr float kLazy = 8.f;      // log2 growth of a row's maximum before O is rescaled
// registers per thread: 168 at launch; 216 + 216 + 72 = 3 x 168
constexpr int kRegSoftmax = 216, kRegOther = 72;

template <int HD> constexpr int tile_bytes() { return kKT * HD * 2; }

// A split item's description for the joining kernel, one per CTA: the item
// that begins in the CTA's range and ends in another's.
struct JoinItem {
  int valid, row0, tok0, tokens, h, last, late, pad;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzled
// layout: 64 MN-contiguous elements per 128-byte row, rows along K, 8-row
// groups 1024 bytes apart, 64-element column halves `lbo` bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem]: A's rows are TMEM lanes, two 16-bit values a column.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

#define R4(a, i) "=f"(a[i]), "=f"(a[i + 1]), "=f"(a[i + 2]), "=f"(a[i + 3])
#define R16(a, i) R4(a, i), R4(a, i + 4), R4(a, i + 8), R4(a, i + 12)
#define W4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
#define W16(a, i) W4(a, i), W4(a, i + 4), W4(a, i + 8), W4(a, i + 12)

// 64 consecutive fp32 columns of this thread's TMEM lane into v[base..]; the
// values are there when it returns.
template <int BASE, int N>
__device__ __forceinline__ void tmem_ld64(uint32_t addr, float (&v)[N]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,"
      "%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : R16(v, BASE), R16(v, BASE + 16), R16(v, BASE + 32), R16(v, BASE + 48)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32f(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : R16(v, 0), R16(v, 16)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      W16(v, 0), W16(v, 16)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_umma_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ PagedAttnArgs a, int box, int slots,
                           JoinItem* join) {
  pdl_trigger();
  constexpr bool kBf16 = sizeof(T) == 2 && !__is_same(T, __half);
  constexpr int kTile = tile_bytes<HD>();
  constexpr int kHalfTile = kKT * 128;  // one 64-column half
  constexpr int kHalves = HD / 64;
  constexpr uint32_t kColS = 0, kColO = 256;  // S0, S1 (P over their first halves), O0, O1
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  // Q tiles, the ring, the units of the batch's requests
  uint8_t* ring = smem + 2 * kTile;
  long long* pre = reinterpret_cast<long long*>(ring + slots * kTile);
  __shared__ __align__(8) uint64_t bars[2 * kMaxSlots + 9];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto full = [&](int s) { return bar(s); };
  auto empty = [&](int s) { return bar(kMaxSlots + s); };
  constexpr int kB = 2 * kMaxSlots;
  auto s_full = [&](int x) { return bar(kB + x); };
  auto p_full = [&](int x) { return bar(kB + 2 + x); };
  auto o_full = [&](int x) { return bar(kB + 4 + x); };
  const uint32_t q_full = bar(kB + 6), q_empty = bar(kB + 7), all_done = bar(kB + 8);
  if (tid == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), 4);  // the query tile's warps
      mbar_init(o_full(x), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(all_done, 1);
    fence_barrier_init();
    s_abort = 0;
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  pdl_wait();
  if (tid == 0) join[blockIdx.x].valid = 0;
  tc_fence_before();
  attn_plan<HD, kKT>(a, pre);  // ends with a barrier
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // a bounded wait that also gives up once another warp has given up
  auto wait = [&](uint32_t b, uint32_t parity) -> bool {
    if (mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(b, parity)) {
      if (*(volatile int*)&s_abort || global_ns() - t0 > kWaitNs) {
        *(volatile int*)&s_abort = 1;
        return false;
      }
    }
    return true;
  };
  auto wait_warp = [&](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(b, parity));
  };
  bool ok = true;
  const int ipq = a.ipt / 2;  // tokens per query tile
  const uint32_t s_q = smem_u32(smem), s_ring = smem_u32(ring);

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == 8) {
      // ---------------------------------------------------------- TMA
      AttnWalk<kKT> w(a, pre);
      const int rows_all = a.n_pages * a.nkv * a.page;  // past the pools: TMA fills zeros
      const int per = kKT / box;
      int it = 0, seg = 0;
      for (; !w.done() && ok; w.next(), ++seg) {
        const int32_t* tab = a.table + (int64_t)w.r * a.max_pages;
        int ent = 0, ent_base = -1;
        for (int kt = w.kbeg; kt < w.kend && ok; ++kt) {
          // the pool rows of the tile's boxes, looked up 32 boxes at a time
          const int b0 = (kt - w.kbeg) * per;
          if (ent_base < 0 || b0 + per > ent_base + 32) {
            ent_base = b0;
            const int key = w.kbeg * kKT + (b0 + lane) * box;
            int y = rows_all;
            if (key < w.q.len) {
              const int e = tab[key / a.page];
              if (e >= 0 && e < a.n_pages) y = (e * a.nkv + w.h) * a.page + key % a.page;
            }
            if (!DFLASH_CHECK(y >= 0 && y <= rows_all, a.err)) y = rows_all;
            ent = y;
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++it) {
            const int s = it % slots;
            if (it >= slots) {
              ok = wait_warp(empty(s), ((it / slots) - 1) & 1);
              if (!ok) break;
            }
            if (lane == 0) mbar_arrive_expect_tx(full(s), kTile);
            __syncwarp();
            for (int b = 0; b < per; ++b) {
              const int y = __shfl_sync(0xffffffffu, ent, b0 + b - ent_base);
              if (lane < kHalves)
                tma_load_2d(s_ring + s * kTile + b * box * 128 + lane * kHalfTile,
                            kv ? &tmV : &tmK, full(s), lane * 64, y, policy_evict_last());
            }
            if (kt == w.kbeg && kv == 0) {
              // the item's queries, behind its first keys: the last products of the
              // segment before release the buffer
              if (seg > 0 && !wait_warp(q_empty, (seg - 1) & 1)) {
                ok = false;
                break;
              }
              if (lane == 0) {
                const int nx = w.tokens() > ipq ? 2 : 1;
                mbar_arrive_expect_tx(q_full, nx * kHalves * ipq * a.G * 128);
                for (int x = 0; x < nx; ++x)
                  for (int hf = 0; hf < kHalves; ++hf)
                    tma_load_3d(s_q + x * kTile + hf * kHalfTile, &tmQ, q_full, hf * 64,
                                w.h * a.G, w.q.row0 + w.t * a.ipt + x * ipq);
              }
              __syncwarp();
            }
          }
        }
      }
      // the copies in flight land before the CTA may end
      for (int j = max(0, it - slots); j < it; ++j)
        ok &= mbar_wait(full(j % slots), (j / slots) & 1);
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA
      AttnWalk<kKT> w(a, pre);
      const uint32_t id_s = idesc_f16kind(kQT, kKT, kBf16);
      const uint32_t id_o = idesc_f16kind(kQT, HD, kBf16) | (1u << 16);  // B MN-major
      int it = 0, seg = 0;             // ring position, segments so far
      int tiles = 0, tiles1 = 0;       // key tiles so far, those of query tile 1
      auto qk = [&](int x, int slot) {
        const uint64_t dq = smem_desc_sw128(s_q + x * kTile);
        const uint64_t dk = smem_desc_sw128(s_ring + slot * kTile);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint64_t off = (uint64_t)((ks >> 2) * (kHalfTile >> 4) + (ks & 3) * 2);
          umma_f16(tmem + kColS + x * 128, dq + off, dk + off, id_s, ks > 0 ? 1u : 0u);
        }
        umma_commit(s_full(x));
      };
      auto pv = [&](int x, int slot, bool first) {
        const uint64_t dv = desc_mn(s_ring + slot * kTile, kHalfTile);
#pragma unroll
        for (int ks = 0; ks < kKT / 16; ++ks)
          umma_f16_ts(tmem + kColO + x * 128, tmem + kColS + x * 128 + ks * 8,
                      dv + (uint64_t)(ks * 128), id_o, (!first || ks > 0) ? 1u : 0u);
      };
      for (; !w.done() && ok; w.next(), ++seg) {
        const bool two = w.tokens() > ipq;
        const int n = w.kend - w.kbeg;
        if (!wait_warp(q_full, seg & 1)) { ok = false; break; }
        for (int j = 0; j < n; ++j, ++tiles) {
          const int sk = (it + 2 * j) % slots, sv = (it + 2 * j + 1) % slots;
          if (!wait_warp(full(sk), ((it + 2 * j) / slots) & 1)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) qk(0, sk);
          if (two && j > 0) {
            if (!wait_warp(p_full(1), (tiles1++) & 1)) { ok = false; break; }
            tc_fence_after();
            const int sp = (it + 2 * j - 1) % slots;
            if (lane == 0) {
              pv(1, sp, j == 1);
              umma_commit(empty(sp));
            }
          }
          if (lane == 0) {
            if (two) qk(1, sk);
            umma_commit(empty(sk));
            if (j + 1 == n) umma_commit(q_empty);
          }
          if (!wait_warp(full(sv), ((it + 2 * j + 1) / slots) & 1)) { ok = false; break; }
          const int live = w.q.len - (w.kbeg + j) * kKT;  // keys of this tile below the end
          if (live < kKT) {
            // rows past the request's keys hold whatever the page held: as zeros
            // they add nothing (their weights are 0, but 0 x NaN is not)
            const int rows = kKT - max(live, 0);
            for (int c = lane; c < rows * 8 * kHalves; c += 32) {
              const int hf = c / (rows * 8), o = c % (rows * 8);
              *reinterpret_cast<uint4*>(ring + sv * kTile + hf * kHalfTile + (kKT - rows) * 128 +
                                        o * 16) = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          if (!wait_warp(p_full(0), tiles & 1)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
            pv(0, sv, j == 0);
            if (!two) umma_commit(empty(sv));
            if (j + 1 == n) umma_commit(o_full(0));
          }
        }
        if (!ok) break;
        if (two) {
          if (!wait_warp(p_full(1), (tiles1++) & 1)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
            const int sp = (it + 2 * n - 1) % slots;
            pv(1, sp, n == 1);
            umma_commit(empty(sp));
            umma_commit(o_full(1));
          }
        }
        it += 2 * n;
      }
      // the products in flight end before TMEM is freed
      if (lane == 0) umma_commit(all_done);
      __syncwarp();
      ok &= mbar_wait(all_done, 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
    AttnWalk<kKT> w(a, pre);
    const int x = warp >> 2;
    const int lr = tid & 127;  // row of the query tile = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + kColS + x * 128 + lanes, tO = tmem + kColO + x * 128 + lanes;
    const float c = a.scale_log2;
    int tiles = 0, seg = 0;
    int checked = -1;
    bool mapped = false;
    // Query tile 1 sits out the segments that do not need it: its barriers then
    // do not complete a phase, and its own counts of tiles and segments go with them.
    for (; !w.done() && ok; w.next()) {
      if (w.r != checked) {
        checked = w.r;
        mapped = pages_mapped(a, w.r, w.q, lane);
        if (!mapped && lane == 0) set_error(a.err, DFLASH_DEV_PAGE);
      }
      const int tok0 = w.t * a.ipt;
      const bool whole = w.whole();
      if (tid == 0 && !whole && w.kbeg == w.k0) {
        const int last = w.cta_last();
        JoinItem d;
        d.valid = mapped;
        d.row0 = w.q.row0;
        d.tok0 = tok0;
        d.tokens = w.tokens();
        d.h = w.h;
        d.last = last;
        d.late = w.first ? 0 : 1;
        d.pad = 0;
        join[blockIdx.x] = d;
      }
      const int mine = w.tokens() - x * ipq;  // tokens of this query tile
      if (mine <= 0) continue;
      const int rows = min(mine, ipq) * a.G;
      const int tk = tok0 + x * ipq + min(lr, rows - 1) / a.G, hg = min(lr, rows - 1) % a.G;
      const bool valid = lr < rows;
      const int p = w.q.st + tk;
      const int lo = row_lo(a, p), hi = row_hi(a, w.q, p);
      // every row of the query tile sees the keys [all_lo, all_hi)
      const int all_hi = row_hi(a, w.q, w.q.st + tok0 + x * ipq);
      const int all_lo = row_lo(a, w.q.st + tok0 + x * ipq + min(mine, ipq) - 1);
      float m = -INFINITY, l = 0.f;  // reference maximum (log2 units), sum
      for (int kt = w.kbeg; kt < w.kend; ++kt, ++tiles) {
        if (!wait_warp(s_full(x), tiles & 1)) { ok = false; break; }
        tc_fence_after();
        float s[128];
        tmem_ld64<0>(tS, s);
        tmem_ld64<64>(tS + 64, s);
        const int k0 = kt * kKT;
        if (k0 < all_lo || k0 + kKT > all_hi) {
          const int l0 = lo - k0, h0 = hi - k0;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i < l0 || i >= h0) s[i] = -INFINITY;
        }
        float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
        for (int i = 4; i < 128; i += 4) {
          mx0 = fmaxf(mx0, s[i]);
          mx1 = fmaxf(mx1, s[i + 1]);
          mx2 = fmaxf(mx2, s[i + 2]);
          mx3 = fmaxf(mx3, s[i + 3]);
        }
        const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * c;
        if (__any_sync(0xffffffffu, valid && mx > m + kLazy)) {
          const float mn = fmaxf(m, mx);
          const float f = mn == -INFINITY ? 1.f : ex2_ftz(m - mn);
          m = mn;
          l *= f;
          // S of this tile was issued behind the product of the tile before, so O
          // is complete
          if (kt > w.kbeg) {
#pragma unroll 1
            for (int cc = 0; cc < HD; cc += 32) {
              float o[32];
              uint32_t u[32];
              tmem_ld32f(tO + cc, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
              tmem_st32(tO + cc, u);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float e0 = ex2_ftz(fmaf(s[hf * 64 + 2 * i], c, -ref));
            const float e1 = ex2_ftz(fmaf(s[hf * 64 + 2 * i + 1], c, -ref));
            l0 += e0;
            l1 += e1;
            // rounded to the operand type: relative error at most half a step per weight
            u[i] = pack2<T>(e0, e1);
          }
          tmem_st32(tS + hf * 32, u);
        }
        l += l0 + l1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(x));
      }
      if (!ok) break;

      // ---------------------------------------------------------- end of a segment
      if (!wait_warp(o_full(x), seg & 1)) { ok = false; break; }
      ++seg;
      tc_fence_after();
      T* outp = static_cast<T*>(a.out) + (int64_t)(w.q.row0 + tk) * a.out_stride +
                (int64_t)(w.h * a.G + hg) * HD;
      const size_t pr = (size_t)w.slot() * a.tile_rows + x * kQT + lr;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      bool fin = true;
#pragma unroll 1
      for (int cc = 0; cc < HD; cc += 32) {
        float o[32];
        tmem_ld32f(tO + cc, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) fin &= isfinite(o[i]);
        if (!valid) continue;
        if (whole) {
          if (mapped) {
            uint4* dst = reinterpret_cast<uint4*>(outp + cc);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack2<T>(o[8 * i] * inv, o[8 * i + 1] * inv),
                                  pack2<T>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                  pack2<T>(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                  pack2<T>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(a.part_o + pr * HD + cc);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      tc_fence_before();
      if (valid && !whole)
        *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m, l);
      if (valid && whole && mapped && a.lse)
        a.lse[(int64_t)(w.q.row0 + tk) * a.nq + w.h * a.G + hg] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      unsigned odd = __ballot_sync(0xffffffffu, !fin && valid && !isnan(l));
      __syncwarp();
      for (; odd && mapped; odd &= odd - 1) {
        const int src = __ffs(odd) - 1;
        const float mr = __shfl_sync(0xffffffffu, m, src), lr2 = __shfl_sync(0xffffffffu, l, src);
        const int tk2 = __shfl_sync(0xffffffffu, tk, src), hg2 = __shfl_sync(0xffffffffu, hg, src);
        float acc[HD / 32];
        if (!masked_key_fallback<T, HD, kKT>(a, w.r, w.h, w.q, w.kbeg, w.kend, tk2, hg2,
                                             mr == -INFINITY ? 0.f : mr, lane, acc))
          continue;
        T* o2 = static_cast<T*>(a.out) + (int64_t)(w.q.row0 + tk2) * a.out_stride +
                (int64_t)(w.h * a.G + hg2) * HD;
        const size_t pr2 = (size_t)w.slot() * a.tile_rows + x * kQT + (warp & 3) * 32 + src;
#pragma unroll
        for (int d = 0; d < HD / 32; ++d) {
          const int col = lane * (HD / 32) + d;
          if (whole)
            o2[col] = from_f<T>(lr2 == 0.f ? 0.f : acc[d] / lr2);
          else
            a.part_o[pr2 * HD + col] = acc[d];
        }
      }
    }
  }
  if (!ok && lane == 0) set_error(a.err, DFLASH_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the partials of the items that several CTAs shared: block (c, y) does
// rows [32 y, 32 y + 32) of the item that begins in CTA c's range, 8 threads a
// row, its pieces in CTA order.
template <typename T, int HD>
__global__ void __launch_bounds__(256)
    attn_join_kernel(const __grid_constant__ PagedAttnArgs a, const JoinItem* join) {
  pdl_trigger();
  pdl_wait();
  const JoinItem d = join[blockIdx.x];
  if (!d.valid) return;
  const int ipq = a.ipt / 2;
  const int row = blockIdx.y * 32 + (threadIdx.x >> 3), x = row / kQT, lr = row % kQT;
  const int mine = min(d.tokens - x * ipq, ipq);
  if (lr >= mine * a.G) return;
  const int c0 = blockIdx.x, sub = threadIdx.x & 7;
  auto at = [&](int cta) {
    return (size_t)(2 * cta + (cta == c0 ? d.late : 0)) * a.tile_rows + row;
  };
  float M = -INFINITY;
  for (int cta = c0; cta <= d.last; ++cta) M = fmaxf(M, __ldcg(a.part_ml + at(cta) * 2));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  constexpr int V = HD / 32;  // float4 a thread: columns 4 (sub + 8 i)
  float4 acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int cta = c0; cta <= d.last; ++cta) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + at(cta) * 2));
    const float f = ex2_ftz(ml.x - ref);
    L += ml.y * f;
    const float4* src = reinterpret_cast<const float4*>(a.part_o + at(cta) * HD) + sub;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float4 v = __ldcg(src + 8 * i);
      acc[i].x += v.x * f;
      acc[i].y += v.y * f;
      acc[i].z += v.z * f;
      acc[i].w += v.w * f;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t tok = d.row0 + d.tok0 + x * ipq + lr / a.G;
  const int head = d.h * a.G + lr % a.G;
  T* dst = static_cast<T*>(a.out) + tok * a.out_stride + (int64_t)head * HD;
#pragma unroll
  for (int i = 0; i < V; ++i)
    *reinterpret_cast<uint2*>(dst + 4 * (sub + 8 * i)) =
        make_uint2(pack2<T>(acc[i].x * inv, acc[i].y * inv),
                   pack2<T>(acc[i].z * inv, acc[i].w * inv));
  if (a.lse && sub == 0)
    a.lse[tok * a.nq + head] =
        L == 0.f ? -INFINITY : (ref + log2f(L)) * 0.6931471805599453f;
}

template <typename T, int HD>
int launch_umma(const PagedAttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                const CUtensorMap& tv, int box, void* join, cudaStream_t s) {
  constexpr int kLimit = 227 * 1024 - 1024;  // dynamic, beside the barriers
  const int fixed = 1024 + 2 * tile_bytes<HD>() + a.batch * 8;
  const int slots = std::min(kMaxSlots, (kLimit - fixed) / tile_bytes<HD>());
  if (slots < 4) return DFLASH_EUNSUPPORTED;
  static SmemLimit limit;
  if (!limit.raise(reinterpret_cast<const void*>(attn_paged_umma_kernel<T, HD>), kLimit))
    return DFLASH_ECUDA;
  const int ctas = attn_paged_umma_ctas();
  if (launch_pdl(attn_paged_umma_kernel<T, HD>, dim3(ctas), dim3(kThreads),
                 (size_t)fixed + (size_t)slots * tile_bytes<HD>(), s, 1, tq, tk, tv, a, box, slots,
                 static_cast<JoinItem*>(join)) != cudaSuccess)
    return DFLASH_ECUDA;
  const cudaError_t e = launch_pdl(attn_join_kernel<T, HD>, dim3(ctas, 2 * kQT / 32), dim3(256), 0,
                                   s, 1, a, static_cast<const JoinItem*>(join));
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ECUDA;
}

}  // namespace

int attn_paged_umma_ctas() { return num_sms(); }
size_t attn_paged_join_bytes() { return (size_t)attn_paged_umma_ctas() * sizeof(JoinItem); }

int launch_attn_paged_umma(const PagedAttnArgs& a, int hd, int dtype, void* join, cudaStream_t s) {
  // boxes of whole pages, or of (part of) the tile where a page holds it
  const int box = a.page % 128 == 0 ? 128 : a.page % 64 == 0 ? 64 : a.page;
  const int64_t rows = (int64_t)a.n_pages * a.nkv * a.page;
  CUtensorMap tq, tk, tv;
  if (!encode_2d(&tk, a.k_pool, rows, hd, hd, box, dtype) ||
      !encode_2d(&tv, a.v_pool, rows, hd, hd, box, dtype) ||
      !encode_rows3(&tq, a.q, a.n_rows, a.nq, hd, a.q_stride, a.G, a.ipt / 2, dtype))
    return DFLASH_ECUDA;
  TimedScope ts(s, TC_ATTN);
  if (dtype == DFLASH_BF16)
    return hd == 128 ? launch_umma<__nv_bfloat16, 128>(a, tq, tk, tv, box, join, s)
                     : launch_umma<__nv_bfloat16, 64>(a, tq, tk, tv, box, join, s);
  return hd == 128 ? launch_umma<__half, 128>(a, tq, tk, tv, box, join, s)
                   : launch_umma<__half, 64>(a, tq, tk, tv, box, join, s);
}

}  // namespace dflash
