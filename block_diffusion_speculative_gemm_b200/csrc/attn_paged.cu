// Paged chunk attention for at most 16 rows per kv head and request (single
// tokens, mostly): softmax(scale Q K^T) V over a paged cache in one pass, on
// mma.sync m16n8k16 with fp32 accumulators.
//
//   S = Q K^T;  m' = max(m, max S);  P = 2^(S c - m' c), c = scale log2(e);
//   l' = l 2^((m - m') c) + sum P;   O' = O 2^((m - m') c) + P V
//
// A CTA is one producer warp, which finds the CTA's segments, describes them to
// the others, and streams 64-key K and V tiles into a ring of shared-memory slots
// with TMA (one box per page piece), and four compute warps, which split the keys
// of every tile and are joined at the end of a segment.  The softmax state and O
// stay in registers, Q too, P goes from the S accumulators to the next product's
// operand without leaving the thread.  Bound by memory: the keys and values of an
// item are read once for all its rows, 4 rows flop per byte.  The producer runs on
// over segment boundaries, so the ring stays full while a segment is finished, and
// two CTAs share an SM; at head_dim 128 the requests' sums of units leave room for one
// from 198 requests on, which streams as fast (198 single tokens 297 us, 197 294).
// 32 single tokens behind 512 to 4096 keys (32 query, 8 key heads of 128): 50 us, 5.3
// TB/s with start and end, 256 of them 6.3 TB/s; one token behind 2048 keys: 12.5 us, a
// chain of loads (lengths, page table, keys, partials).
//
// Every CTA has the same number of key tiles (attn_paged.cuh); an item shared
// by several CTAs is left as partials (O, max, sum), and the CTA that counts
// itself last joins them in CTA order, so results do not depend on timing.
#include <algorithm>

#include "attn_paged.cuh"

namespace dflash {

namespace {

constexpr int kKL = 6, kKT = 1 << kKL;    // keys per tile
constexpr int kCompute = 128;             // compute threads
constexpr int kThreads = kCompute + 32;
constexpr int kSlots = 6;                 // ring slots, each a K or a V tile
constexpr int kPassCols = 64;             // O columns joined at a time

template <int HD> constexpr int slot_bytes() { return kKT * HD * 2; }
constexpr int kPassRow = kPassCols + 8;   // eight rows side by side meet no bank twice
constexpr int kScratch = 3 * 16 * kPassRow * 4;
constexpr int kSegs = 4;                  // segments described ahead

// A segment of the CTA's work, as the producer describes it.
struct Seg {
  int more;               // 0: the end
  int r, h, row0, st, n, len;
  int tok0, tokens;
  int kbeg, kend, whole;
  int slot;               // partial slot
  // known by seg_info: the request's pages are mapped; the CTAs that share the item,
  // its place in c0
  int mapped, c0, c1, late;
};

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4],
                                                 uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void bar_compute() {
  asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory");
}
// The same barrier; true on every thread when any thread brought `v` true.
__device__ __forceinline__ bool bar_compute_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kCompute)
      : "memory");
  return r != 0;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 2)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ PagedAttnArgs a, int box) {
  pdl_trigger();
  constexpr int NK = 4;               // key groups, one a warp
  constexpr int KW = kKT / NK;        // keys of a tile per warp
  constexpr int kNT = KW / 8;         // S column blocks
  constexpr int kSlot = slot_bytes<HD>();
  constexpr int kHalfTile = kKT * 128;  // one 64-column half of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  float* scratch = reinterpret_cast<float*>(smem + kSlots * kSlot);
  long long* pre = reinterpret_cast<long long*>(smem + kSlots * kSlot + kScratch);
  __shared__ __align__(8) uint64_t bars[2 * kSlots + 3 * kSegs];
  __shared__ Seg segs[kSegs];
  __shared__ float s_ml[4][16][2];
  __shared__ int s_abort, s_last;
  __shared__ int s_taken;  // values of the segment were taken out (ItemKeys)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t s_base = smem_u32(smem);
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[kSlots + s]); };
  auto seg_full = [&](int k) { return smem_u32(&bars[2 * kSlots + k % kSegs]); };
  auto seg_empty = [&](int k) { return smem_u32(&bars[2 * kSlots + kSegs + k % kSegs]); };
  auto seg_info = [&](int k) { return smem_u32(&bars[2 * kSlots + 2 * kSegs + k % kSegs]); };
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 4);
    }
    for (int k = 0; k < kSegs; ++k) {
      mbar_init(seg_full(k), 1);
      mbar_init(seg_empty(k), 4);
      mbar_init(seg_info(k), 1);
    }
    fence_barrier_init();
    s_abort = 0;
    s_taken = 0;
  }
  if (tid < 2) tma_prefetch_desc(tid == 0 ? &tmK : &tmV);
  __syncthreads();
  pdl_wait();
  if (a.batch > 32) attn_plan<HD, kKL>(a, pre);  // ends with a barrier

  // a bounded wait that also gives up once another warp has given up
  auto wait = [&](uint32_t b, uint32_t parity) -> bool {
    if (mbar_try_wait_nap(b, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait_nap(b, parity)) {
      if (*(volatile int*)&s_abort || global_ns() - t0 > kWaitNs) {
        *(volatile int*)&s_abort = 1;
        return false;
      }
    }
    return true;
  };
  bool ok = true;
  const int rows_all = a.n_pages * a.nkv * a.page;  // a row past the pools: TMA fills zeros

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = policy_evict_first();
    const int per = kKT / box, per_log2 = __ffs(per) - 1;  // boxes a tile, at most 4
    int it = 0;                 // ring position
    int checked = -1;
    bool mapped = false;
    if (a.batch <= 32) attn_plan_warp<HD, kKL>(a, pre);
    AttnWalk<kKL> w(a, pre);
    for (int k = 0; ok; w.next(), ++k) {
      if (k >= kSegs &&
          !__all_sync(0xffffffffu, wait(seg_empty(k), (uint32_t)(k / kSegs - 1) & 1))) {
        ok = false;
        break;
      }
      Seg& d = segs[k % kSegs];
      if (w.done()) {
        if (lane == 0) {
          d.more = 0;
          mbar_arrive(seg_full(k));
        }
        break;
      }
      const int32_t* tab = a.table + (int64_t)w.r * a.max_pages;
      // the pool rows of the segment's boxes b0 .. b0 + 31, a lane each
      auto lookup = [&](int b0) -> int {
        const int key = w.kbeg * kKT + (b0 + lane) * box;
        int y = rows_all;
        if (key < w.q.len && b0 < (w.kend - w.kbeg) * per) {
          const int pg = a.by_page.div(key), e = tab[pg];
          if (e >= 0 && e < a.n_pages) y = (e * a.nkv + w.h) * a.page + key - pg * a.page;
        }
        if (!DFLASH_CHECK(y >= 0 && y <= rows_all, a.err)) y = rows_all;
        return y;
      };
      int ent = lookup(0), ahead = lookup(32);  // these boxes, the next ones
      auto describe = [&]() {
        const bool whole = w.whole();
        if (lane == 0) {
          d.more = 1;
          d.r = w.r;
          d.h = w.h;
          d.row0 = w.q.row0;
          d.st = w.q.st;
          d.n = w.q.n;
          d.len = w.q.len;
          d.tok0 = w.t * a.ipt;
          d.tokens = w.tokens();
          d.kbeg = w.kbeg;
          d.kend = w.kend;
          d.whole = whole;
          d.slot = w.slot();
          mbar_arrive(seg_full(k));
        }
        __syncwarp();
        // what takes longer and is needed at the end of the segment only
        if (w.r != checked) {
          checked = w.r;
          mapped = pages_mapped(a, w.r, w.q, lane);
          if (!mapped && lane == 0) set_error(a.err, DFLASH_DEV_PAGE);
        }
        if (lane == 0) {
          d.mapped = mapped;
          if (!whole) {
            const int c0 = w.cta_first();
            d.c0 = c0;
            d.c1 = w.cta_last();
            d.late = w.later_in(c0);
          }
          mbar_arrive(seg_info(k));
        }
        __syncwarp();
      };
      for (int kt = w.kbeg; kt < w.kend && ok; ++kt) {
        const int b0 = ((kt - w.kbeg) * per) & 31;  // a tile's boxes divide 32
        if (kt > w.kbeg && b0 == 0) {
          ent = ahead;
          ahead = lookup((kt - w.kbeg) * per + 32);
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++it) {
          // the description behind the first tile that has room (the compute warps
          // free no slot before they have it)
          if (kt == w.kbeg && kv == 0 && it >= kSlots) describe();
          const int s = it % kSlots;
          if (it >= kSlots) {
            ok = __all_sync(0xffffffffu, wait(empty(s), ((it / kSlots) - 1) & 1));
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive_expect_tx(full(s), kSlot);
          __syncwarp();
          // the tile's boxes side by side, a lane each
          const int hf = lane >> per_log2, b = lane & (per - 1);
          const int y = __shfl_sync(0xffffffffu, ent, b0 + b);
          if (hf < HD / 64)
            tma_load_2d(s_base + s * kSlot + b * box * 128 + hf * kHalfTile, kv ? &tmV : &tmK,
                        full(s), hf * 64, y, pol);
          if (kt == w.kbeg && kv == 1 && it < kSlots) describe();
        }
      }
    }
    // the copies in flight land before the CTA may end
    for (int j = max(0, it - kSlots); j < it; ++j) ok &= mbar_wait(full(j % kSlots), (j / kSlots) & 1);
  } else {
    // ------------------------------------------------------------ compute
    const int wk = warp;
    const int g8 = lane >> 2, t2 = (lane & 3) * 2;
    const T* qg = static_cast<const T*>(a.q);
    // ldmatrix addresses: K rows are keys (operand as stored), V transposed
    const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
    const int vr = (lane & 7) + (((lane >> 3) & 1) << 3), vc = lane >> 4;
    int it = 0;
    for (int seg = 0;; ++seg) {
      // a wait that gave up ends all compute warps together, at the next meeting
      ok = __all_sync(0xffffffffu, wait(seg_full(seg), (uint32_t)(seg / kSegs) & 1));
      if (bar_compute_or(!ok)) {
        ok = false;
        break;
      }
      const Seg& w = segs[seg % kSegs];
      if (!w.more) break;
      const AttnReq q = {w.row0, w.n, w.st, w.len};
      const int tok0 = w.tok0, R = w.tokens * a.G, kbeg = w.kbeg, kend = w.kend;
      // this thread's two rows: token, query head within the group
      int row[2], tok[2], hg[2], lo[2], hi[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        row[j] = g8 + 8 * j;
        const int rr = min(row[j], R - 1);
        tok[j] = tok0 + a.by_g.div(rr);
        hg[j] = rr - (tok[j] - tok0) * a.G;
        lo[j] = row_lo(a, q.st + tok[j]);
        hi[j] = row_hi(a, q, q.st + tok[j]);
      }
      uint32_t qf[HD / 16][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const T* src = qg + (int64_t)(q.row0 + tok[j]) * a.q_stride +
                       (int64_t)(w.h * a.G + hg[j]) * HD + t2;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          qf[ks][j] = *reinterpret_cast<const uint32_t*>(src + ks * 16);
          qf[ks][j + 2] = *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8);
        }
      }
      const ItemKeys keys(a, q, tok0, w.tokens);
      float o[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < HD / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

      for (int kt = kbeg; kt < kend && ok; ++kt, it += 2) {
        const int sk = it % kSlots, sv = (it + 1) % kSlots;
        if (!__all_sync(0xffffffffu, wait(full(sk), (it / kSlots) & 1))) { ok = false; break; }
        const int key0 = kt * kKT + wk * KW;  // this warp's first key
        const uint32_t kb = s_base + sk * kSlot + (uint32_t)(wk * KW) * 128;
        float sc[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
          for (int n = 0; n < kNT; n += 2) {
            uint32_t b[4];
            const int rr = n * 8 + kr, ch = (ks & 3) * 2 + kc;
            ldsm4(b, kb + (ks >> 2) * kHalfTile + rr * 128 + ((ch ^ (rr & 7)) << 4));
            mma16816<T>(sc[n], qf[ks], b[0], b[1]);
            mma16816<T>(sc[n + 1], qf[ks], b[2], b[3]);
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(sk));
        const bool edge = key0 < keys.all_lo || key0 + KW > keys.all_hi;
        if (edge) {
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + n * 8 + t2 + (e & 1);
              if (key < lo[e >> 1] || key >= hi[e >> 1]) sc[n][e] = -INFINITY;
            }
        }
        float alpha[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = m[j];
#pragma unroll
          for (int n = 0; n < kNT; ++n)
            mx = fmaxf(mx, fmaxf(sc[n][2 * j], sc[n][2 * j + 1]) * a.scale_log2);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float ref = mx == -INFINITY ? 0.f : mx;
          alpha[j] = ex2_ftz(m[j] - ref);  // 0 while nothing was seen
          m[j] = mx;
          l[j] *= alpha[j];
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float pv = ex2_ftz(fmaf(sc[n][2 * j + e], a.scale_log2, -ref));
              sc[n][2 * j + e] = pv;
              l[j] += pv;
            }
        }
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= alpha[e >> 1];

        if (!__all_sync(0xffffffffu, wait(full(sv), ((it + 1) / kSlots) & 1))) {
          ok = false;
          break;
        }
        const uint32_t vb = s_base + sv * kSlot + (uint32_t)(wk * KW) * 128;
        if (edge) {
          const int k0 = kt * kKT;
          edge_values<T, HD, kKT>(smem + sv * kSlot, wk * KW, wk * KW + KW, keys.lo - k0,
                                  keys.hi - k0, keys.all_lo - k0, keys.all_hi - k0, lane,
                                  &s_taken);
          // the slot's next tile comes by TMA
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
#pragma unroll
        for (int k2 = 0; k2 < KW / 16; ++k2) {
          // P rounded to the operand type: relative error at most half a step per weight
          const uint32_t pf[4] = {
              pack2<T>(sc[2 * k2][0], sc[2 * k2][1]), pack2<T>(sc[2 * k2][2], sc[2 * k2][3]),
              pack2<T>(sc[2 * k2 + 1][0], sc[2 * k2 + 1][1]),
              pack2<T>(sc[2 * k2 + 1][2], sc[2 * k2 + 1][3])};
#pragma unroll
          for (int d = 0; d < HD / 16; ++d) {
            uint32_t b[4];
            const int rr = k2 * 16 + vr, ch = (d & 3) * 2 + vc;
            ldsm4t(b, vb + (d >> 2) * kHalfTile + rr * 128 + ((ch ^ (rr & 7)) << 4));
            mma16816<T>(o[2 * d], pf, b[0], b[1]);
            mma16816<T>(o[2 * d + 1], pf, b[2], b[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(sv));
      }
      // ---------------------------------------------------------- end of a segment
      // a wait that gave up ends all compute warps here, together
      ok = ok && __all_sync(0xffffffffu, wait(seg_info(seg), (uint32_t)(seg / kSegs) & 1));
      if (bar_compute_or(!ok)) {
        ok = false;
        break;
      }
      const bool mapped = w.mapped;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
        l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
      }
      bool add_back;  // values were taken out
      {               // join the key groups
        if ((lane & 3) == 0)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            s_ml[warp][g8 + 8 * j][0] = m[j];
            s_ml[warp][g8 + 8 * j][1] = l[j];
          }
        bar_compute();
        add_back = s_taken != 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int k = 0; k < NK; ++k) M = fmaxf(M, s_ml[k][g8 + 8 * j][0]);
          const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
          for (int k = 0; k < NK; ++k)
            L += s_ml[k][g8 + 8 * j][1] * ex2_ftz(s_ml[k][g8 + 8 * j][0] - ref);
          const float f = ex2_ftz(m[j] - ref);
          m[j] = M;
          l[j] = L;
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) {
            o[i][2 * j] *= f;
            o[i][2 * j + 1] *= f;
          }
        }
#pragma unroll
        for (int pass = 0; pass < HD / kPassCols; ++pass) {
          constexpr int kB = kPassCols / 8;
          if (wk > 0) {
            float* dst = scratch + (wk - 1) * 16 * kPassRow;
#pragma unroll
            for (int i = 0; i < kB; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (row[j] < R)
                  *reinterpret_cast<float2*>(dst + (g8 + 8 * j) * kPassRow + i * 8 + t2) =
                      make_float2(o[pass * kB + i][2 * j], o[pass * kB + i][2 * j + 1]);
          }
          bar_compute();
          if (wk == 0) {
#pragma unroll
            for (int k = 1; k < NK; ++k) {
              const float* src = scratch + (k - 1) * 16 * kPassRow;
#pragma unroll
              for (int i = 0; i < kB; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  if (row[j] >= R) continue;
                  const float2 v = *reinterpret_cast<const float2*>(
                      src + (g8 + 8 * j) * kPassRow + i * 8 + t2);
                  o[pass * kB + i][2 * j] += v.x;
                  o[pass * kB + i][2 * j + 1] += v.y;
                }
            }
          }
          bar_compute();
        }
      }
      const bool whole = w.whole;
      T* outp = static_cast<T*>(a.out);
      if (wk == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (row[j] >= R) continue;
          if (whole) {
            if (mapped) {
              const float inv = l[j] == 0.f ? 0.f : 1.f / l[j];
              T* dst = outp + (int64_t)(q.row0 + tok[j]) * a.out_stride +
                       (int64_t)(w.h * a.G + hg[j]) * HD + t2;
#pragma unroll
              for (int i = 0; i < HD / 8; ++i)
                *reinterpret_cast<uint32_t*>(dst + i * 8) =
                    pack_result<T>(o[i][2 * j] * inv, o[i][2 * j + 1] * inv);
              if (a.lse && (lane & 3) == 0)
                a.lse[(int64_t)(q.row0 + tok[j]) * a.nq + w.h * a.G + hg[j]] =
                    l[j] == 0.f ? -INFINITY : (m[j] + log2f(l[j])) * 0.6931471805599453f;
            }
          } else {
            const size_t pr = (size_t)w.slot * a.tile_rows + row[j];
#pragma unroll
            for (int i = 0; i < HD / 8; ++i)
              *reinterpret_cast<float2*>(a.part_o + pr * HD + i * 8 + t2) =
                  make_float2(o[i][2 * j], o[i][2 * j + 1]);
            if ((lane & 3) == 0)
              *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m[j], l[j]);
          }
        }
        __syncwarp();
        if (add_back) {
          // row i from the lanes 4 (i % 8) .. + 3, which hold it, to lane i
          const float m0 = __shfl_sync(0xffffffffu, m[0], (lane & 7) * 4);
          const float m1 = __shfl_sync(0xffffffffu, m[1], (lane & 7) * 4);
          const int ti = a.by_g.div(lane), gi = lane - ti * a.G;
          void* dst = nullptr;
          if (lane < R && mapped && whole)
            dst = outp + (int64_t)(q.row0 + tok0 + ti) * a.out_stride +
                  (int64_t)(w.h * a.G + gi) * HD;
          else if (lane < R && mapped)
            dst = a.part_o + ((size_t)w.slot * a.tile_rows + lane) * HD;
          add_taken_out<T, HD>(a, w.r, w.h, q, tok0, w.tokens, kbeg * kKT, kend * kKT, lane,
                               tok0 + ti, gi, lane < 8 ? m0 : m1, dst, !whole, 0, HD);
          if (lane == 0) s_taken = 0;  // all have read it; set again behind the next meeting
        }
      }
      if (!whole) {
        // the CTA that finishes last joins the item's partials in CTA order
        __threadfence();
        bar_compute();
        const int c0 = w.c0, c1 = w.c1, late = w.late;
        auto slot_row = [&](int x, int rr) {
          return (size_t)(2 * x + (x == c0 ? late : 0)) * a.tile_rows + rr;
        };
        if (tid == 0) {
          const unsigned old = atomicAdd(a.cnt + c0, 1u);
          s_last = old == (unsigned)(c1 - c0);
          if (s_last) a.cnt[c0] = 0;
        }
        bar_compute();
        if (s_last && mapped) {
          __threadfence();
          // a warp a row: the lanes take the partials' maxima and sums side by side,
          // then columns
          for (int rr = warp; rr < R; rr += 4) {
            constexpr int V = HD / 32, B = 16;
            float v[B][V];  // sixteen partials on their way at once
            auto fetch = [&](int x0) {
#pragma unroll
              for (int i = 0; i < B; ++i) {
                const float* src = a.part_o + slot_row(min(x0 + i, c1), rr) * HD + lane * V;
                if constexpr (V == 4)
                  *reinterpret_cast<float4*>(v[i]) = __ldcg(reinterpret_cast<const float4*>(src));
                else
                  *reinterpret_cast<float2*>(v[i]) = __ldcg(reinterpret_cast<const float2*>(src));
              }
            };
            auto stats = [&](int x) {
              return x <= c1 ? __ldcg(reinterpret_cast<const float2*>(a.part_ml +
                                                                      slot_row(x, rr) * 2))
                             : make_float2(-INFINITY, 0.f);
            };
            float2 ml = stats(c0 + lane);
            fetch(c0);
            float M = ml.x;
            for (int x0 = c0 + 32; x0 <= c1; x0 += 32) M = fmaxf(M, stats(x0 + lane).x);
            M = warp_max(M);
            const float ref = M == -INFINITY ? 0.f : M;
            float L = 0.f, acc[V];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.f;
            for (int x0 = c0; x0 <= c1; x0 += B) {
              if (x0 > c0) {
                if (((x0 - c0) & 31) == 0) ml = stats(x0 + lane);
                fetch(x0);
              }
              const float f = ex2_ftz(ml.x - ref);
              if (((x0 - c0) & 31) == 0) L += warp_sum(ml.y * f);
#pragma unroll
              for (int i = 0; i < B; ++i) {
                const float g = __shfl_sync(0xffffffffu, f, ((x0 - c0) & 31) + i);
                if (x0 + i > c1) continue;
#pragma unroll
                for (int d = 0; d < V; ++d) acc[d] += v[i][d] * g;
              }
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int ti = a.by_g.div(rr), tk = tok0 + ti, hh = w.h * a.G + rr - ti * a.G;
            T* dst = outp + (int64_t)(q.row0 + tk) * a.out_stride + (int64_t)hh * HD + lane * V;
#pragma unroll
            for (int i = 0; i < V; i += 2)
              *reinterpret_cast<uint32_t*>(dst + i) =
                  pack_result<T>(acc[i] * inv, acc[i + 1] * inv);
            if (a.lse && lane == 0)
              a.lse[(int64_t)(q.row0 + tk) * a.nq + hh] =
                  L == 0.f ? -INFINITY : (ref + log2f(L)) * 0.6931471805599453f;
          }
        }
        bar_compute();  // s_last is reused
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(seg_empty(seg));
    }
  }
  if (!ok && lane == 0) set_error(a.err, DFLASH_DEV_TIMEOUT);
}

template <typename T, int HD>
int launch_one(const PagedAttnArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int box,
               cudaStream_t s) {
  constexpr int kFixed = 1024 + kSlots * slot_bytes<HD>() + kScratch;
  static SmemLimit limit;
  if (!limit.raise(reinterpret_cast<const void*>(attn_paged_kernel<T, HD>),
                   kFixed + kPagedMaxBatch * 8))
    return DFLASH_ECUDA;
  const cudaError_t e =
      launch_pdl(attn_paged_kernel<T, HD>, dim3(attn_paged_ctas()), dim3(kThreads),
                 (size_t)kFixed + (size_t)a.batch * 8, s, 1, tk, tv, a, box);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ECUDA;
}

}  // namespace

int attn_paged_ctas() { return 2 * num_sms(); }

int launch_attn_paged(const PagedAttnArgs& a, int hd, int dtype, cudaStream_t s) {
  // boxes of whole pages, or of the tile where a page holds it
  const int box = std::min(a.page, kKT);
  const int64_t rows = (int64_t)a.n_pages * a.nkv * a.page;
  CUtensorMap tk, tv;
  if (!encode_2d(&tk, a.k_pool, rows, hd, hd, box, dtype) ||
      !encode_2d(&tv, a.v_pool, rows, hd, hd, box, dtype))
    return DFLASH_ECUDA;
  TimedScope ts(s, TC_ATTN);
  if (dtype == DFLASH_BF16)
    return hd == 128 ? launch_one<__nv_bfloat16, 128>(a, tk, tv, box, s)
                     : launch_one<__nv_bfloat16, 64>(a, tk, tv, box, s);
  return hd == 128 ? launch_one<__half, 128>(a, tk, tv, box, s)
                   : launch_one<__half, 64>(a, tk, tv, box, s);
}

}  // namespace dflash
