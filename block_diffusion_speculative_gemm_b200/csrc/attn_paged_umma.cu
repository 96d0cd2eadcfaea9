// Paged chunk attention on the 5th-generation tensor cores: the formulas of
// attn_paged.cu with a thread per row.
//
// The CTA works on two tiles of S = Q K^T at a time, 128 rows x 128 keys each
// (UMMA into TMEM).  An item that fills both query tiles meets one run of 128
// keys with both of them; one that has a single query tile meets two runs of
// 128 keys, each with its own accumulators, joined at the end of the segment.
// A softmax thread owns one row of a tile, i.e. one TMEM lane, so the row
// maximum and sum need no exchange; it writes P over the first half of S's
// columns in the operand type, and O += P V takes P straight from TMEM (A
// operand) with V as the MN-major B operand.  Per CTA (one per SM):
//
//   warps 0-3, 4-7  softmax of tile 0 and 1, and their results
//   warp 8          TMA: K and V tiles through one ring of slots, Q per item
//   warps 9, 10     the products of tile 0 and 1: S(j), then O += P(j) V
//   warp 11         the CTA's segments, described ahead of the others' work
//
// so the tensor cores work on one tile while the other one is in its softmax.
// S of a tile is overwritten by the next product only after P of it has been
// read, which the issue order alone guarantees.  Half of P is handed over while the
// exponentials of the other half run.  O is rescaled in TMEM only when a row's
// maximum grew by more than 2^8 since its reference was set (weights then stay below
// 2^8, exact enough in fp32 sums and inside fp16); normalisation happens once, at the
// end.
//
// Bound by the tensor cores and, equally, by the exponentials: 4 x 128 x 128 x
// HD flop and 128 x 128 exponentials a tile, 1024 cycles each at head_dim 128; a step
// of both tiles takes about 3000 cycles, since a tile's S, softmax and P V follow one
// another.  On new inputs each time, a prompt of 8192 tokens (32 query, 8 key heads of
// 128) takes 528 us, 1.04 PFLOP/s at the clocks that the power limit leaves; 4 blocks of
// 16 behind 32768 keys 106 us, 5.1 TB/s; 32 blocks of 8 behind 512 to 4096 keys 58 us.
// (Evaluating a quarter of the exponentials by a polynomial on the FMA pipe was
// slower: 512 us against 497 for a prompt of 8192 tokens; its instructions cost
// more issue slots than the special-function unit's time is worth.)
#include <algorithm>

#include "attn_paged.cuh"

namespace dflash {

namespace {

constexpr int kKT = 128;          // keys per tile of S
constexpr int kQT = 128;          // rows per query tile
constexpr int kSoftmaxWarps = 8;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kPlanWarp = 11;
constexpr int kThreads = 384;     // the last four warps: a warpgroup of their own
constexpr int kMaxSlots = 12;
constexpr int kSegs = 2;          // segments described ahead
constexpr int kBars = 2 * kMaxSlots + 8 + 3 * kSegs + 3 + 4 + 2;
constexpr float kLazy = 8.f;      // log2 growth of a row's maximum before O is rescaled
// registers per thread: 168 at launch; 2 x 216 + 72 = 3 x 168
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

// The products, issued by the lanes whose `on` is set (one lane) with the whole
// warp converged: control flow and operands then are uniform over the warp, and
// the instruction's operands stay in uniform registers.  In a branch of one lane
// each of the eight instructions of a product took 120 to 170 cycles to issue,
// more than the 64 that it runs.
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void umma_ss(uint32_t on, uint32_t d_tmem, uint64_t adesc,
                                        uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: A's rows are TMEM lanes, two 16-bit values a column.
__device__ __forceinline__ void umma_ts(uint32_t on, uint32_t d_tmem, uint32_t a_tmem,
                                        uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar),
      "r"(on)
      : "memory");
}
// Arrival of the lanes whose `on` is set, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(on)
      : "memory");
}
// 1 in one lane of the warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(r));
  return r;
}
// A value that all lanes hold alike, as one the compiler knows to be uniform.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// 32 consecutive bytes: one wide store, or two where they may start on 16 bytes.
__device__ __forceinline__ void store32(void* dst, const uint32_t* u, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

#define R4(a, i) "=f"(a[i]), "=f"(a[i + 1]), "=f"(a[i + 2]), "=f"(a[i + 3])
#define R16(a, i) R4(a, i), R4(a, i + 4), R4(a, i + 8), R4(a, i + 12)
#define W4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
#define W16(a, i) W4(a, i), W4(a, i + 4), W4(a, i + 8), W4(a, i + 12)

// Consecutive fp32 columns of this thread's TMEM lane; the values are there when
// it returns.
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : R16(v, 0)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : R16(v, 0), R16(v, 16)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
      "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
      "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : R16(v, 0), R16(v, 16), R16(v, 32), R16(v, 48), R16(v, 64), R16(v, 80), R16(v, 96), R16(v, 112)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      W16(v, 0)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The largest of three that are not NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Keys [32 B, 32 B + 32) of a row's scores: weights 2^(c s - ref) rounded to the
// operand type into u, their unrounded sum into l0 + l1 (pairs).
template <typename T>
__device__ __forceinline__ void weights32(const float* s, uint64_t c2, uint64_t nref2,
                                          uint32_t* u, uint64_t& l0, uint64_t& l1) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t x = fma2(pair(s[2 * i], s[2 * i + 1]), c2, nref2);
    float e0, e1;
    unpair(x, e0, e1);
    e0 = ex2_ftz(e0);
    e1 = ex2_ftz(e1);
    const uint64_t e = pair(e0, e1);
    if (i & 1) l1 = add2(l1, e); else l0 = add2(l0, e);
    // rounded to the operand type: relative error at most half a step per weight
    u[i] = pack2<T>(e0, e1);
  }
}

// A row's weights, into TMEM columns tS.., and their sum; p_half is told of the
// first 64 keys' (late enough that nothing waits for the stores), p_full of all.
// No branch inside, so that the instructions of all 128 keys can overlap.
template <typename T>
__device__ __forceinline__ void tile_weights(const float (&s)[128], uint64_t c2, uint64_t nref2,
                                             uint32_t tS, uint32_t on, uint32_t p_half,
                                             uint32_t p_full, uint64_t& l0, uint64_t& l1) {
  uint32_t u[4][16];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    weights32<T>(s + 32 * c, c2, nref2, u[c], l0, l1);
    if (c < 2) tmem_st(tS + c * 16, u[c]);
    if (c == 2) {
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_if(on, p_half);
      tmem_st(tS + c * 16, u[c]);
    }
    if (c == 3) {
      tmem_st(tS + c * 16, u[c]);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_if(on, p_full);
    }
  }
}

// A segment of the CTA's work, as the planning warp describes it to the others.
// two: tile x is query tile x against run j of 128 keys, j < runs.  Otherwise
// tile x is the one query tile against run 2 j + x, the last of which may be
// missing for x = 1.
struct Seg {
  int more;        // 0: the end
  int two, whole;  // whole: the segment is all of its item
  int r, h, row0, st, len;
  int tok0, tokens;
  int run0, runs;
  int slot;        // partial slot
  int mapped;      // the request's pages are (known by seg_info)
  int taken;       // values were taken out of keys that not every row sees (by o_full)
  __device__ int steps(int x) const { return two ? runs : (runs + 1 - x) >> 1; }
  __device__ int run(int x, int j) const { return run0 + (two ? j : 2 * j + x); }
};

// Shared memory beside the tiles.
struct Fixed {
  float2 row[2][kQT];  // what the two threads of a row exchange
  uint64_t bars[kBars];
  Seg seg[kSegs];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Fixed) % 8 == 0, "the units follow");

// A position of the ring, by counting: a division by the number of slots would
// take longer than a product's instructions.
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  __device__ void next(int slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

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
  // Q tiles, the ring, the fixed part, the units of the batch's requests
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + 2 * kTile;
  Fixed& fx = *reinterpret_cast<Fixed*>(ring + slots * kTile);
  long long* pre = reinterpret_cast<long long*>(&fx + 1);

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  auto bar = [&](int i) { return smem_u32(&fx.bars[i]); };
  auto full = [&](int s) { return bar(s); };
  auto empty = [&](int s) { return bar(kMaxSlots + s); };
  constexpr int kB = 2 * kMaxSlots;
  auto s_full = [&](int x) { return bar(kB + x); };
  auto p_half = [&](int x) { return bar(kB + 2 + x); };
  auto p_full = [&](int x) { return bar(kB + 4 + x); };
  auto o_full = [&](int x) { return bar(kB + 6 + x); };
  auto seg_full = [&](int k) { return bar(kB + 8 + k % kSegs); };
  auto seg_info = [&](int k) { return bar(kB + 8 + kSegs + k % kSegs); };
  auto seg_empty = [&](int k) { return bar(kB + 8 + 2 * kSegs + k % kSegs); };
  const uint32_t q_full = bar(kB + 8 + 3 * kSegs), q_empty = bar(kB + 9 + 3 * kSegs);
  const uint32_t all_done = bar(kB + 10 + 3 * kSegs);
  // meetings of the two softmax warps that hold the same rows
  auto met_rows = [&](int quarter) { return bar(kB + 11 + 3 * kSegs + quarter); };
  auto s_read = [&](int x) { return bar(kB + 15 + 3 * kSegs + x); };
  if (tid == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 2);  // the warps of both tiles' products
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full(x), 1);
      mbar_init(p_half(x), 4);  // the tile's warps
      mbar_init(p_full(x), 4);
      mbar_init(o_full(x), 2);  // the products, and what their warp wrote
      mbar_init(s_read(x), 4);
    }
    for (int k = 0; k < kSegs; ++k) {
      mbar_init(seg_full(k), 1);
      mbar_init(seg_info(k), 1);
      mbar_init(seg_empty(k), kSoftmaxWarps + 3);
    }
    for (int i = 0; i < 4; ++i) mbar_init(met_rows(i), 2);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    mbar_init(all_done, 2);
    fence_barrier_init();
    fx.abort = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&fx.tmem), 512);
    tmem_relinquish();
  }
  if (tid < 3) tma_prefetch_desc(tid == 0 ? &tmQ : tid == 1 ? &tmK : &tmV);
  pdl_wait();
  if (tid == 0) join[blockIdx.x].valid = 0;
  tc_fence_before();
  if (a.batch > 32)
    attn_plan<HD, 0>(a, pre);  // ends with a barrier
  else
    __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's: they start at 0

  // a bounded wait that also gives up once another warp has given up; a test
  // that finds the phase incomplete sleeps for a while, so that waiting warps
  // leave the issue slots to the others
  auto wait = [&](uint32_t b, uint32_t parity) -> bool {
    if (mbar_try_wait_nap(b, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait_nap(b, parity)) {
      if (*(volatile int*)&fx.abort || global_ns() - t0 > kWaitNs) {
        *(volatile int*)&fx.abort = 1;
        return false;
      }
    }
    return true;
  };
  auto wait_warp = [&](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(b, parity));
  };
  auto phase = [](int k) { return (uint32_t)(k / kSegs) & 1; };
  // swizzled tiles start on 1024 bytes, as the symbol's alignment asks
  bool ok = true;
  const bool placed = (smem_u32(smem) & 1023) == 0 && fx.tmem == tmem;
  if (!placed) ok = false;
  const uint32_t s_q = smem_u32(smem), s_ring = smem_u32(ring);

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == kPlanWarp) {
      // ---------------------------------------------------------- segments
      int checked = -1, k = 0;
      bool mapped = false;
      if (ok) {
        if (a.batch <= 32) attn_plan_warp<HD, 0>(a, pre);
        AttnWalk<0> w(a, pre);
        for (;; ++k) {
          if (k >= kSegs && !wait_warp(seg_empty(k), phase(k - kSegs))) { ok = false; break; }
          Seg& d = fx.seg[k % kSegs];
          if (w.done()) {
            if (lane == 0) {
              d.more = 0;
              mbar_arrive(seg_full(k));
            }
            break;
          }
          const bool two = w.tokens() > a.ipq, whole = w.whole();
          const int tok0 = w.t * a.ipt, tokens = w.tokens();
          if (lane == 0) {
            d.more = 1;
            d.two = two;
            d.whole = whole;
            d.r = w.r;
            d.h = w.h;
            d.row0 = w.q.row0;
            d.st = w.q.st;
            d.len = w.q.len;
            d.tok0 = tok0;
            d.tokens = tokens;
            d.run0 = two ? w.kbeg : max(w.kbeg * 2, w.x.lo >> 7);
            d.runs = (two ? w.kend : min(w.kend * 2, ((w.x.hi - 1) >> 7) + 1)) - d.run0;
            d.slot = w.slot();
            d.taken = 0;
            mbar_arrive(seg_full(k));
          }
          __syncwarp();
          if (w.r != checked) {
            checked = w.r;
            mapped = pages_mapped(a, w.r, w.q, lane);
            if (!mapped && lane == 0) set_error(a.err, DFLASH_DEV_PAGE);
          }
          if (lane == 0) {
            d.mapped = mapped;
            mbar_arrive(seg_info(k));
            if (!whole && w.kbeg == w.x.k0) {
              JoinItem ji;
              ji.valid = mapped;
              ji.row0 = w.q.row0;
              ji.tok0 = tok0;
              ji.tokens = tokens;
              ji.h = w.h;
              ji.last = w.cta_last();
              ji.late = w.slot() & 1;
              ji.pad = 0;
              join[blockIdx.x] = ji;
            }
          }
          w.next();
        }
      }
    } else if (warp == kTmaWarp) {
      // ---------------------------------------------------------- TMA
      const int rows_all = a.n_pages * a.nkv * a.page;  // past the pools: TMA fills zeros
      const int per = kKT / box, per_log2 = __ffs(per) - 1;  // boxes a tile, at most 8
      RingPos at;
      int it = 0, k = 0;  // tiles asked for, segments
      for (; ok; ++k) {
        if (!wait_warp(seg_full(k), phase(k))) { ok = false; break; }
        const Seg g = fx.seg[k % kSegs];
        if (!g.more) break;
        // keys that one query tile reads pass through once
        const uint64_t pol = g.two ? policy_evict_last() : policy_evict_first();
        const int32_t* tab = a.table + (int64_t)g.r * a.max_pages;
        // the pool rows of the segment's boxes b0 .. b0 + 31, a lane each
        auto lookup = [&](int b0) -> int {
          const int key = g.run0 * kKT + (b0 + lane) * box;
          int y = rows_all;
          if (key < g.len && b0 < g.runs * per) {
            const int pg = a.by_page.div(key), e = tab[pg];
            if (e >= 0 && e < a.n_pages) y = (e * a.nkv + g.h) * a.page + key - pg * a.page;
          }
          if (!DFLASH_CHECK(y >= 0 && y <= rows_all, a.err)) y = rows_all;
          return y;
        };
        int ent = lookup(0), ahead = lookup(32);  // these boxes, the next ones
        const int quad = g.two ? 1 : 2;  // runs per step; a step's boxes divide 32
        for (int j = 0; j < g.runs && ok; j += quad) {
          const int b0 = (j * per) & 31;
          if (j > 0 && b0 == 0) {
            ent = ahead;
            ahead = lookup(j * per + 32);
          }
          const int nr = min(quad, g.runs - j);
          for (int o = 0; o < 2 * nr; ++o, ++it) {  // K of the step's runs, then V
            const int kv = o >= nr, run = kv ? o - nr : o;
            const int s = at.slot;
            if (it >= slots) {
              ok = wait_warp(empty(s), at.phase ^ 1);
              if (!ok) break;
            }
            at.next(slots);
            if (lane == 0) mbar_arrive_expect_tx(full(s), kTile);
            __syncwarp();
            // the tile's boxes side by side, a lane each
            const int hf = lane >> per_log2, b = lane & (per - 1);
            const int y = __shfl_sync(0xffffffffu, ent, b0 + run * per + b);
            if (hf < kHalves)
              tma_load_2d(s_ring + s * kTile + b * box * 128 + hf * kHalfTile, kv ? &tmV : &tmK,
                          full(s), hf * 64, y, pol);
            if (j == 0 && o == 0) {
              // the item's queries, behind its first keys: the last products of the
              // segment before release the buffer
              if (k > 0 && !wait_warp(q_empty, (k - 1) & 1)) {
                ok = false;
                ++it;  // this slot's copies are in flight
                break;
              }
              if (lane == 0) {
                const int nx = g.two ? 2 : 1;
                mbar_arrive_expect_tx(q_full, nx * kHalves * a.ipq * a.G * 128);
                for (int x = 0; x < nx; ++x)
                  for (int hf = 0; hf < kHalves; ++hf)
                    tma_load_3d(s_q + x * kTile + hf * kHalfTile, &tmQ, q_full, hf * 64,
                                g.h * a.G, g.row0 + g.tok0 + x * a.ipq);
              }
              __syncwarp();
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty(k));
      }
      // the copies in flight land before the CTA may end
      for (int j = max(0, it - slots); j < it; ++j)
        ok &= mbar_wait(full(j % slots), (j / slots) & 1);
      if (k > 0) ok &= mbar_wait(q_full, (k - 1) & 1);
    } else {
      // ---------------------------------------------------------- MMA of tile x
      const int x = warp - kMmaWarp;
      const uint32_t on = elect_one();
      const uint32_t id_s = idesc_f16kind(kQT, kKT, kBf16);
      const uint32_t id_o = idesc_f16kind(kQT, HD, kBf16) | (1u << 16);  // B MN-major
      const uint32_t t_s = tmem + kColS + x * 128, t_o = tmem + kColO + x * 128;
      // Both warps visit every ring position in order and release it once, also the
      // tiles that only the other one multiplies with.
      RingPos at;
      int done = 0;       // tiles so far
      int other = 0;      // of the other tile
      bool turn = false;  // tile 0: the step before had a tile 1
      auto pass = [&]() -> bool {
        if (!wait_warp(full(at.slot), at.phase)) return false;
        if (lane == 0) mbar_arrive(empty(at.slot));
        at.next(slots);
        return true;
      };
      // The tiles take turns: a tile's next scores start when the other one's threads
      // have read theirs, so that one is in its exponentials while the products of
      // the other run.  Left alone they fall into step, and wait for the
      // special-function unit and for the products together.  Tile 1 waits in every
      // step of tile 0, tile 0 after every step of tile 1, so that neither passes
      // over a phase.
      auto take_turn = [&]() -> bool {
        return x == 0 && !turn ? true : wait_warp(s_read(x ^ 1), (other - 1 + x) & 1);
      };
      for (int k = 0; ok; ++k) {
        if (!wait_warp(seg_full(k), phase(k))) { ok = false; break; }
        Seg& g = fx.seg[k % kSegs];
        if (!uniform(g.more)) break;
        const bool two = uniform(g.two);
        const ItemKeys ik(a, {0, 0, g.st, g.len}, g.tok0, g.tokens);
        const int lo = uniform(ik.lo), hi = uniform(ik.hi);
        const int all_lo = uniform(ik.all_lo), all_hi = uniform(ik.all_hi);
        const int n = uniform(g.steps(x)), n0 = uniform(g.steps(0)), n1 = uniform(g.steps(1));
        const int run0 = uniform(g.run0), len = uniform(g.len);
        const uint64_t dq = smem_desc_sw128(s_q + (two ? x : 0) * kTile);
        if (!wait_warp(q_full, k & 1)) { ok = false; break; }
        if (n == 0 && lane == 0) mbar_arrive(q_empty);
        int sk = 0;  // slot of the step's K tile
        auto k_ready = [&]() -> bool {
          if (x == 1 && !two && !pass()) return false;
          if (!wait_warp(full(at.slot), at.phase)) return false;
          sk = at.slot;
          at.next(slots);
          return take_turn();
        };
        if (n > 0 && !(ok = k_ready())) break;
        for (int j = 0; j < n; ++j, ++done) {
          const bool both = j < n1;  // both tiles take part
          tc_fence_after();
          const uint64_t dk = smem_desc_sw128(s_ring + sk * kTile);
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            const uint64_t off = (uint64_t)((ks >> 2) * (kHalfTile >> 4) + (ks & 3) * 2);
            umma_ss(on, t_s, dq + off, dk + off, id_s, ks > 0 ? 1u : 0u);
          }
          umma_commit_if(on, s_full(x));
          umma_commit_if(on, empty(sk));
          if (j + 1 == n) umma_commit_if(on, q_empty);

          if (!two && (x == 1 || both) && !(ok = pass())) break;
          const int sv = at.slot;
          if (!(ok = wait_warp(full(sv), at.phase))) break;
          at.next(slots);
          const int key0 = (run0 + (two ? j : 2 * j + x)) * kKT;
          if (key0 < all_lo || key0 + kKT > all_hi) {
            // With two query tiles both warps do this, on the same tile.
            edge_values<T, HD, kKT>(ring + sv * kTile, 0, kKT, lo - key0, hi - key0,
                                    all_lo - key0, all_hi - key0, lane, &g.taken);
            // also where the other tile's warp was first to take them out
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          // O (+)= P V, each half of P as soon as it is there
          const uint64_t dv = desc_mn(s_ring + sv * kTile, kHalfTile);
          if (!(ok = wait_warp(p_half(x), done & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_ts(on, t_o, t_s + ks * 8, dv + (uint64_t)(ks * 128), id_o,
                    (j > 0 || ks > 0) ? 1u : 0u);
          // all that the next step needs, so that its scores follow at once
          turn = both;
          other += x == 1 || both;
          if (!two && x == 0 && both && !(ok = pass())) break;
          if (j + 1 < n && !(ok = k_ready())) break;
          if (!(ok = wait_warp(p_full(x), done & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 4; ks < 8; ++ks)
            umma_ts(on, t_o, t_s + ks * 8, dv + (uint64_t)(ks * 128), id_o, 1u);
          umma_commit_if(on, empty(sv));
          if (j + 1 == n) {
            mbar_arrive_if(on, o_full(x));
            umma_commit_if(on, o_full(x));
          }
        }
        if (!ok) break;
        if (n < n0) {  // a last step without tile 1
          if (!(ok = pass() && take_turn() && pass())) break;
          ++other;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty(k));
      }
      // the products in flight end before TMEM is freed
      umma_commit_if(on, all_done);
      __syncwarp();
      ok &= mbar_wait(all_done, 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
    const int x = warp >> 2, quarter = warp & 3;
    const uint32_t on = elect_one();
    const int lr = tid & 127;  // row of the query tile = TMEM lane
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + kColS + x * 128 + lanes, tO = tmem + kColO + lanes;
    int tiles = 0;   // of tile x so far
    int seg1 = 0;    // segments with a tile 1 so far
    int n_rows = 0;  // meetings so far
    // bounded, as every wait: a warp that gave up does not come
    auto meet_rows = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(met_rows(quarter));
      return wait_warp(met_rows(quarter), (n_rows++) & 1);
    };
    for (int k = 0; ok; ++k) {
      if (!wait_warp(seg_full(k), phase(k))) { ok = false; break; }
      const Seg& g = fx.seg[k % kSegs];
      if (!g.more) break;
      const bool two = g.two;
      const int qtok = g.tok0 + (two ? x * a.ipq : 0);  // first token of the query tile
      const int mine = min(g.tokens - (qtok - g.tok0), a.ipq), rows = mine * a.G;
      const bool valid = lr < rows, live = quarter * 32 < rows;
      const int n = g.steps(x), run0 = g.run(x, 0) * kKT, hop = two ? kKT : 2 * kKT;
      const AttnReq q = {0, 0, 0, g.len};
      int lo, hi;  // the keys that the row sees
      {
        const int p = g.st + qtok + a.by_g.div(min(lr, rows - 1));
        lo = row_lo(a, p);
        hi = row_hi(a, q, p);
      }
      // every row of the query tile sees the keys [all_lo, all_hi)
      const int all_hi = row_hi(a, q, g.st + qtok);
      const int all_lo = row_lo(a, g.st + qtok + mine - 1);
      float m = -INFINITY;      // reference maximum (log2 units)
      uint64_t l0 = 0, l1 = 0;  // sums
      for (int j = 0; j < n; ++j, ++tiles) {
        if (!wait_warp(s_full(x), tiles & 1)) { ok = false; break; }
        if (live) {
          tc_fence_after();
          float s[128];
          tmem_ld(tS, s);
          mbar_arrive_if(on, s_read(x));
          const int k0 = run0 + j * hop;
          if (k0 < all_lo || k0 + kKT > all_hi) {
            const int b0 = lo - k0, b1 = hi - k0;
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i < b0 || i >= b1) s[i] = -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < 124; i += 8)
#pragma unroll
            for (int c = 0; c < 4; ++c) mx[c] = max3(mx[c], s[i + 2 * c], s[i + 2 * c + 1]);
          mx[0] = max3(mx[0], s[124], s[125]);
          mx[1] = max3(mx[1], s[126], s[127]);
          const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale_log2;
          if (__any_sync(0xffffffffu, valid && mt > m + kLazy)) {
            const float mn = fmaxf(m, mt);
            const float f = mn == -INFINITY ? 1.f : ex2_ftz(m - mn);
            m = mn;
            l0 = mul2(l0, pair(f, f));
            l1 = mul2(l1, pair(f, f));
            // S of this tile was issued behind the product of the tile before, so O
            // is complete
            if (j > 0) {
#pragma unroll 1
              for (int cc = 0; cc < HD; cc += 16) {
                float o[16];
                uint32_t u[16];
                tmem_ld(tO + x * 128 + cc, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * f);
                tmem_st(tO + x * 128 + cc, u);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t c2 = pair(a.scale_log2, a.scale_log2), r2 = pair(-ref, -ref);
          tile_weights<T>(s, c2, r2, tS, on, p_half(x), p_full(x), l0, l1);
        } else {
          // no row of this warp is in use: its part of P is never read
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(s_read(x));
            mbar_arrive(p_half(x));
            mbar_arrive(p_full(x));
          }
        }
      }
      if (!ok) break;

      // ---------------------------------------------------------- end of a segment
      // Where both tiles hold the same row over different keys, its two threads
      // exchange maximum and sum, and each finishes half of the columns.
      const bool has1 = g.steps(1) > 0, whole = g.whole;
      const int nc = two ? HD : HD / 2, c0 = two ? 0 : x * nc;
      if (!wait_warp(seg_info(k), phase(k))) { ok = false; break; }
      const bool mapped = g.mapped;
      // With two query tiles the tiles run independently, and a thread waits for its
      // own accumulator only.  Otherwise the meeting makes sure that the other tile
      // has come to the end of this segment, neither less nor more, before its
      // accumulator is waited for.
      if (n > 0 && !wait_warp(o_full(x), (x ? seg1 : k) & 1)) { ok = false; break; }
      float l, f0 = 1.f, f1 = 0.f;  // the row's sum; weights of tile 0 (x when two) and tile 1
      {
        float e0, e1;
        unpair(add2(l0, l1), e0, e1);
        l = e0 + e1;
      }
      if (!two) {
        fx.row[x][lr] = make_float2(m, l);
        if (!meet_rows()) { ok = false; break; }
        if (x == 1 && !wait_warp(o_full(0), k & 1)) { ok = false; break; }
        if (x == 0 && has1 && !wait_warp(o_full(1), seg1 & 1)) { ok = false; break; }
        const float2 r0 = fx.row[0][lr], r1 = fx.row[1][lr];
        m = fmaxf(r0.x, r1.x);
        const float ref = m == -INFINITY ? 0.f : m;
        f0 = ex2_ftz(r0.x - ref);
        f1 = ex2_ftz(r1.x - ref);
        l = r0.y * f0 + r1.y * f1;
      }
      seg1 += has1;
      tc_fence_after();
      // the row's token and head among those of the kv head
      const int ti = a.by_g.div(min(lr, rows - 1)), tk = qtok + ti;
      const int hd = g.h * a.G + min(lr, rows - 1) - ti * a.G;
      const int64_t orow = g.row0 + tk;
      T* outp = static_cast<T*>(a.out) + orow * a.out_stride + (int64_t)hd * HD;
      const size_t pr = (size_t)g.slot * a.tile_rows + (two ? x * kQT : 0) + lr;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool put = valid && mapped;
      if (live) {
#pragma unroll 1
        for (int cc = c0; cc < c0 + nc; cc += 32) {
          float o[32];
          tmem_ld(tO + (two ? x * 128 : 0) + cc, o);
          if (!two) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f0;
            if (has1) {
              float o1[32];
              tmem_ld(tO + 128 + cc, o1);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], f1, o[i]);
            }
          }
          if (!put) continue;
          if (whole) {
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = pack_result<T>(o[2 * i] * inv, o[2 * i + 1] * inv);
            store32(outp + cc, u, a.wide_out);
            store32(outp + cc + 16, u + 8, a.wide_out);
          } else {
            uint32_t u[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) store32(a.part_o + pr * HD + cc + 8 * i, u + 8 * i, true);
          }
        }
      }
      tc_fence_before();
      if (put && c0 == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(a.part_ml + pr * 2) = make_float2(m, l);
        else if (a.lse)
          a.lse[orow * a.nq + hd] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
      if (g.taken && mapped && live) {
        __syncwarp();
        void* dst = nullptr;
        if (put) dst = whole ? static_cast<void*>(outp) : a.part_o + pr * HD;
        add_taken_out<T, HD>(a, g.r, g.h, {g.row0, 0, g.st, g.len}, g.tok0, g.tokens,
                             g.run0 * kKT, (g.run0 + g.runs) * kKT, lane, tk, hd - g.h * a.G, m,
                             dst, !whole, c0, c0 + nc);
      }
      // both threads of a row have read maximum, sum and accumulators
      if (!two && !meet_rows()) { ok = false; break; }
      __syncwarp();
      if (lane == 0) mbar_arrive(seg_empty(k));
    }
  }
  if (!ok && lane == 0) set_error(a.err, placed ? DFLASH_DEV_TIMEOUT : DFLASH_DEV_CHECK);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Joins the partials of the items that several CTAs shared: block (c, y) does
// rows [32 y, 32 y + 32) of the item that begins in CTA c's range, 8 threads a
// row, its pieces in CTA order, four on their way at once: what it costs is the
// latency of its loads.
template <typename T, int HD>
__global__ void __launch_bounds__(256)
    attn_join_kernel(const __grid_constant__ PagedAttnArgs a, const JoinItem* join) {
  pdl_trigger();
  pdl_wait();
  const JoinItem d = join[blockIdx.x];
  if (!d.valid) return;
  const int ipq = a.ipq;
  const int row = blockIdx.y * 32 + (threadIdx.x >> 3), x = row / kQT, lr = row % kQT;
  const int mine = min(d.tokens - x * ipq, ipq);
  if (lr >= mine * a.G) return;
  const int c0 = blockIdx.x, sub = threadIdx.x & 7;
  auto at = [&](int cta) {
    return (size_t)(2 * cta + (cta == c0 ? d.late : 0)) * a.tile_rows + row;
  };
  float M = -INFINITY, ref = 0.f, L = 0.f;
  constexpr int V = HD / 32, B = 4;  // float4 a thread: columns 4 (sub + 8 i); pieces at a time
  float4 acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int cta = c0; cta <= d.last; cta += B) {
    float2 ml[B];
    float4 v[B][V];
#pragma unroll
    for (int e = 0; e < B; ++e) {
      ml[e] = make_float2(-INFINITY, 0.f);
      if (cta + e > d.last) continue;
      const size_t from = at(cta + e);
      ml[e] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + from * 2));
      const float4* src = reinterpret_cast<const float4*>(a.part_o + from * HD) + sub;
#pragma unroll
      for (int i = 0; i < V; ++i) v[e][i] = __ldcg(src + 8 * i);
    }
    const float before = M;
#pragma unroll
    for (int e = 0; e < B; ++e) M = fmaxf(M, ml[e].x);
    ref = M == -INFINITY ? 0.f : M;
    const float g = ex2_ftz(before - ref);
    L *= g;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[i].x *= g;
      acc[i].y *= g;
      acc[i].z *= g;
      acc[i].w *= g;
    }
#pragma unroll
    for (int e = 0; e < B; ++e) {
      if (cta + e > d.last) continue;
      const float f = ex2_ftz(ml[e].x - ref);
      L += ml[e].y * f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc[i].x += v[e][i].x * f;
        acc[i].y += v[e][i].y * f;
        acc[i].z += v[e][i].z * f;
        acc[i].w += v[e][i].w * f;
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t tok = d.row0 + d.tok0 + x * ipq + lr / a.G;
  const int head = d.h * a.G + lr % a.G;
  T* dst = static_cast<T*>(a.out) + tok * a.out_stride + (int64_t)head * HD;
#pragma unroll
  for (int i = 0; i < V; ++i)
    *reinterpret_cast<uint2*>(dst + 4 * (sub + 8 * i)) =
        make_uint2(pack_result<T>(acc[i].x * inv, acc[i].y * inv),
                   pack_result<T>(acc[i].z * inv, acc[i].w * inv));
  if (a.lse && sub == 0)
    a.lse[tok * a.nq + head] =
        L == 0.f ? -INFINITY : (ref + log2f(L)) * 0.6931471805599453f;
}

template <typename T, int HD>
int launch_umma(const PagedAttnArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                const CUtensorMap& tv, int box, void* join, cudaStream_t s) {
  constexpr int kLimit = 227 * 1024;
  const int fixed = 2 * tile_bytes<HD>() + (int)sizeof(Fixed) + a.batch * 8;
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
      !encode_rows3(&tq, a.q, a.n_rows, a.nq, hd, a.q_stride, a.G, a.ipq, dtype))
    return DFLASH_ECUDA;
  TimedScope ts(s, TC_ATTN);
  if (dtype == DFLASH_BF16)
    return hd == 128 ? launch_umma<__nv_bfloat16, 128>(a, tq, tk, tv, box, join, s)
                     : launch_umma<__nv_bfloat16, 64>(a, tq, tk, tv, box, join, s);
  return hd == 128 ? launch_umma<__half, 128>(a, tq, tk, tv, box, join, s)
                   : launch_umma<__half, 64>(a, tq, tk, tv, box, join, s);
}

}  // namespace dflash
