// Paged chunk attention, shared by its kernels: the call's arguments, which
// keys a row sees, and the division of the work.
//
// A request's rows are its new tokens x the G = n_q / n_kv query heads of a kv
// head, packed token-major (row i * G + g), so that one pass over a kv head's
// keys serves all of them.  An item is (request, kv head, tile of `ipt` tokens)
// and costs as many units as it has key tiles of 2^KL keys, and a few more for
// its start and end (kItemUnits, the last units of the item).  The kernels are
// templates over KL; KL = 0 stands for the tcgen05 kernel's choice by item: 128
// keys where the item fills both query tiles, 256 where it has one, which then
// meets two runs of 128 keys at a time.  The units of all items, in
// order, are cut into one equal range per CTA: every CTA streams the same
// number of key tiles however ragged the batch is, at most two of its items
// are shared with other CTAs (its first and its last), and nothing about the
// lengths has to be known on the host.  A CTA finds its range by summing the
// batch's units itself, which costs one pass over the lengths and saves a
// planning launch.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace dflash {

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A pair of results.  An average of fp16 values never leaves their range, but its weights
// are rounded and the sum they are divided by is not, which could take it past the
// largest value by 2^-11 of it: finite results are held inside the range.
template <typename T> __device__ __forceinline__ uint32_t pack_result(float lo, float hi) {
  if constexpr (__is_same(T, __half)) {
    if (fabsf(lo) < INFINITY) lo = fminf(fmaxf(lo, -65504.f), 65504.f);
    if (fabsf(hi) < INFINITY) hi = fminf(fmaxf(hi, -65504.f), 65504.f);
  }
  return pack2<T>(lo, hi);
}

// Quotients by a number that is known at launch, for dividends below 2^31
// (Granlund and Montgomery: with 2^s >= d and m = ceil(2^(31+s) / d), n / d is
// floor(n m / 2^(31+s))).
struct FastDiv {
  unsigned m;
  int s;  // -1: d = 1
  FastDiv() = default;
  explicit FastDiv(int d) : m(0), s(-1) {
    if (d == 1) return;
    while ((1LL << (s + 1)) < d) ++s;  // s + 1 = ceil(log2 d)
    m = (unsigned)(((1ULL << (32 + s)) + d - 1) / d);
  }
  __device__ __forceinline__ int div(int n) const {
    return s < 0 ? n : (int)(__umulhi((unsigned)n, m) >> s);
  }
};

struct PagedAttnArgs {
  const void* q;
  int64_t q_stride;
  const int32_t *cu, *start, *kv_len;  // kv_len null: start + rows
  int batch, n_rows, nq, nkv, G;
  const int32_t* table;
  int max_pages, page, n_pages;
  float scale_log2;  // score scale times log2(e)
  int causal, window;
  void* out;
  int64_t out_stride;
  int wide_out;      // rows of out start on 32 bytes
  float* lse;        // [n_rows][nq] or null
  int ipt;           // tokens per item
  int ipq;           // tokens per query tile (tcgen05 kernel: ipt = 2 ipq)
  int tile_rows;     // rows of an item's partial (>= ipt * G)
  float *part_o, *part_ml;  // slot s: [tile_rows][HD] and [tile_rows][2] (max in log2 units, sum)
  unsigned* cnt;     // one zeroed counter per CTA
  int32_t* err;
  const void *k_pool, *v_pool;
  FastDiv by_g, by_ipt, by_page;  // divisors G, ipt, page
};

struct AttnReq {
  int row0, n, st, len;
};

// Request r's lengths; the return value is DFLASH_OK's 0 or the error bits of
// a request that must not be touched.
__device__ __forceinline__ int attn_req(const PagedAttnArgs& a, int r, AttnReq& q) {
  q.row0 = a.cu[r];
  const int end = a.cu[r + 1];
  q.st = a.start[r];
  if (out_of_order(q.row0, end, a.n_rows)) return DFLASH_DEV_ROWS;
  q.n = end - q.row0;
  q.len = 0;
  if (q.n == 0) return 0;  // a free place of a padded batch: its lengths are not looked at
  const int64_t last = (int64_t)q.st + q.n;
  const int64_t len = a.kv_len ? (int64_t)a.kv_len[r] : last;
  if (q.st < 0 || last > 0x7fffffff || len < 0 || len > (int64_t)a.max_pages * a.page)
    return DFLASH_DEV_CTX_CAP;
  q.len = (int)len;
  return 0;
}

// Keys [lo, hi) that a token at position p sees.
__device__ __forceinline__ int row_lo(const PagedAttnArgs& a, int p) {
  return a.window > 0 ? max(0, p - a.window + 1) : 0;
}
__device__ __forceinline__ int row_hi(const PagedAttnArgs& a, const AttnReq& q, int p) {
  return a.causal ? min(q.len, p + 1) : q.len;
}

// Item tile t: the keys [lo, hi) its rows see, and the key tiles [k0, k1) that
// hold them (none when no row of it sees a key).
struct TileRange {
  int lo, hi, k0, k1;
};
template <int KL>
__device__ __forceinline__ TileRange tile_range(const PagedAttnArgs& a, const AttnReq& q, int t) {
  const int i0 = t * a.ipt, i1 = min(q.n, i0 + a.ipt);
  const int kl = KL > 0 ? KL : i1 - i0 > a.ipq ? 7 : 8;
  TileRange x;
  x.lo = row_lo(a, q.st + i0);
  x.hi = row_hi(a, q, q.st + i1 - 1);
  x.k0 = x.lo >> kl;
  x.k1 = x.hi > x.lo ? ((x.hi - 1) >> kl) + 1 : x.k0;
  return x;
}

// What starting and finishing an item takes, in key tiles: about 4500 cycles
// against 3200 a tile in the tcgen05 kernel, 3 tiles of 64 keys in the other one.
// An 8192-token prompt, whose first items have one tile and whose last ones 64, has
// an uneven end without it (501 us against 470).
template <int KL> constexpr int kItemUnits = KL > 0 ? 3 : 1;
template <int KL> __device__ __forceinline__ int item_units(const TileRange& x) {
  return x.k1 > x.k0 ? x.k1 - x.k0 + kItemUnits<KL> : 0;
}

// Quotient of two non-negative numbers, by the short 32-bit division where both fit.
__device__ __forceinline__ long long quot(long long n, long long d) {
  if (((n | d) >> 32) == 0) return (unsigned)n / (unsigned)d;
  return n / d;
}

__device__ __forceinline__ int attn_tiles(const PagedAttnArgs& a, int n) {
  return a.by_ipt.div(n + a.ipt - 1);
}

// Rows of item tile t that see no key: output 0, log-sum-exp -inf.  Called by a warp.
template <int HD>
__device__ void zero_rows(const PagedAttnArgs& a, const AttnReq& q, int t, int lane) {
  const int i0 = t * a.ipt, i1 = min(q.n, i0 + a.ipt);
  for (int i = i0; i < i1; ++i) {
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                        (int64_t)(q.row0 + i) * a.out_stride);
    for (int c = lane; c < a.nq * HD / 8; c += 32) o[c] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int c = lane; c < a.nq; c += 32) a.lse[(int64_t)(q.row0 + i) * a.nq + c] = -INFINITY;
  }
}

// True when every page that request q's rows may read is mapped.  Called by a
// warp; the answer is the same in every CTA that works on the request.
__device__ __forceinline__ bool pages_mapped(const PagedAttnArgs& a, int r, const AttnReq& q,
                                             int lane) {
  const int lo = row_lo(a, q.st), hi = row_hi(a, q, q.st + q.n - 1);
  bool bad = false;
  if (hi > lo) {
    const int32_t* tab = a.table + (int64_t)r * a.max_pages;
    const int last = a.by_page.div(hi - 1);
#pragma unroll 4
    for (int k = a.by_page.div(lo) + lane; k <= last; k += 32) {
      const int e = tab[k];
      bad |= e < 0 || e >= a.n_pages;
    }
  }
  return !__any_sync(0xffffffffu, bad);
}

// Units of request r for one kv head, by a warp; items without keys are written
// here, by one CTA each.
template <int HD, int KL>
__device__ long long attn_units(const PagedAttnArgs& a, int r, const AttnReq& q, int lane) {
  const int nt = attn_tiles(a, q.n);
  const bool mine = (int)(r % gridDim.x) == (int)blockIdx.x;
  long long u = 0;
  for (int t0 = 0; t0 < nt; t0 += 32) {
    int k = 0;
    if (t0 + lane < nt) k = item_units<KL>(tile_range<KL>(a, q, t0 + lane));
    u += k;
    if (mine) {
      unsigned e = __ballot_sync(0xffffffffu, t0 + lane < nt && k == 0);
      if (e && !pages_mapped(a, r, q, lane)) e = 0;
      for (; e; e &= e - 1) zero_rows<HD>(a, q, t0 + __ffs(e) - 1, lane);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
  return u;
}

// Largest batch of a call: the prefix sums of every request sit in shared memory.
constexpr int kPagedMaxBatch = 4096;
// Largest row count: row and item arithmetic stays inside 31 bits.
constexpr int kPagedMaxRows = 1 << 30;

// Fills pre[r] with the units of requests 0..r (every thread of the CTA; ends
// with a barrier).  Requests with bad lengths or rows out of order have none and set
// their error bits; items without keys have none and are written here, by one CTA
// each.
template <int HD, int KL>
__device__ void attn_plan(const PagedAttnArgs& a, long long* pre) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthr = blockDim.x, nw = nthr >> 5;
  constexpr int kFew = 4;  // item tiles a single thread adds up
  bool spread = false, order = true;
  for (int r = tid; r < a.batch; r += nthr) {
    AttnReq q;
    long long u = 0;
    const int bad = attn_req(a, r, q);
    if (bad) {
      order &= bad != DFLASH_DEV_ROWS;
      if ((int)(r % gridDim.x) == (int)blockIdx.x) set_error(a.err, bad);
    } else {
      const int nt = attn_tiles(a, q.n);
      bool empty = false;
      for (int t = 0; t < min(nt, kFew); ++t) {
        const TileRange x = tile_range<KL>(a, q, t);
        u += item_units<KL>(x);
        empty |= x.k1 == x.k0;
      }
      if (nt > kFew || empty) {
        u = -1;
        spread = true;
      }
    }
    pre[r] = u;
  }
  if (__syncthreads_or(spread || !order)) {
    if (__syncthreads_or(!order)) {  // the requests that overlap earlier ones
      if (warp == 0)
        each_request_order(a.cu, a.batch, a.n_rows, lane, [&](int r, bool ok, int, int) {
          if (r < a.batch && !ok) {
            pre[r] = 0;
            if ((int)(r % gridDim.x) == (int)blockIdx.x) set_error(a.err, DFLASH_DEV_ROWS);
          }
        });
      __syncthreads();
    }
    for (int r = warp; r < a.batch; r += nw) {
      if (pre[r] >= 0) continue;
      AttnReq q;
      attn_req(a, r, q);
      const long long u = attn_units<HD, KL>(a, r, q, lane);
      __syncwarp();
      if (lane == 0) pre[r] = u;
    }
    __syncthreads();
  }
  if (warp == 0) {
    long long carry = 0;
    for (int r0 = 0; r0 < a.batch; r0 += 32) {
      const int r = r0 + lane;
      long long v = r < a.batch ? pre[r] * a.nkv : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long w = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += w;
      }
      v += carry;
      if (r < a.batch) pre[r] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
}

// The same for at most 32 requests, by one warp without a barrier: a lane a
// request.  Only the warp that walks needs the result.
template <int HD, int KL>
__device__ void attn_plan_warp(const PagedAttnArgs& a, long long* pre) {
  const int lane = threadIdx.x & 31;
  constexpr int kFew = 4;
  AttnReq q = {0, 0, 0, 0};
  long long u = 0;
  bool spread = false, order = true;
  if (lane < a.batch) {
    const int bad = attn_req(a, lane, q);
    if (bad) {
      order = bad != DFLASH_DEV_ROWS;
      if ((int)(lane % gridDim.x) == (int)blockIdx.x) set_error(a.err, bad);
    } else {
      const int nt = attn_tiles(a, q.n);
      spread = nt > kFew;
      for (int t = 0; t < min(nt, kFew); ++t) {
        const TileRange x = tile_range<KL>(a, q, t);
        u += item_units<KL>(x);
        spread |= x.k1 == x.k0;
      }
    }
  }
  if (!__all_sync(0xffffffffu, order))  // the requests that overlap earlier ones
    each_request_order(a.cu, a.batch, a.n_rows, lane, [&](int r, bool ok, int, int) {
      if (r < a.batch && !ok) {
        u = 0;
        spread = false;
        if ((int)(r % gridDim.x) == (int)blockIdx.x) set_error(a.err, DFLASH_DEV_ROWS);
      }
    });
  for (unsigned todo = __ballot_sync(0xffffffffu, spread); todo; todo &= todo - 1) {
    const int r = __ffs(todo) - 1;
    AttnReq o;
    o.row0 = __shfl_sync(0xffffffffu, q.row0, r);
    o.n = __shfl_sync(0xffffffffu, q.n, r);
    o.st = __shfl_sync(0xffffffffu, q.st, r);
    o.len = __shfl_sync(0xffffffffu, q.len, r);
    const long long v = attn_units<HD, KL>(a, r, o, lane);
    if (lane == r) u = v;
  }
  u *= a.nkv;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long w = __shfl_up_sync(0xffffffffu, u, d);
    if (lane >= d) u += w;
  }
  if (lane < a.batch) pre[lane] = u;
  __syncwarp();
}

// The division of W units over N CTAs: the first W % N ranges have one unit more
// than the others.
struct UnitSplit {
  long long each, rest;
  __device__ UnitSplit(long long W, int N) {
    each = quot(W, N);
    rest = W - each * N;
  }
  __device__ long long begin(int c) const { return each * c + min((long long)c, rest); }
  __device__ int owner(long long u) const {
    const long long wide = rest * (each + 1);
    return u < wide ? (int)quot(u, each + 1) : (int)(rest + quot(u - wide, each));
  }
};

// A CTA's walk over its range, one segment (a run of key tiles of one item) at
// a time.  Every warp role walks on its own; all lanes of a warp take part.
template <int KL>
struct AttnWalk {
  const PagedAttnArgs& a;
  const long long* pre;
  long long u, u_end;     // position, end of the range
  int c;
  UnitSplit split;
  // the current segment
  AttnReq q;
  int r, h, t;
  int kbeg, kend;         // key tiles of the segment
  TileRange x;            // its item's keys and key tiles
  int off, take;          // units of the item before the segment, units of the segment

  __device__ static int ranges(const PagedAttnArgs& a, long long W) {
    return (int)max(1LL, min((long long)gridDim.x, W));  // every range has at least one unit
  }
  __device__ AttnWalk(const PagedAttnArgs& a_, const long long* pre_)
      : a(a_), pre(pre_), split(pre_[a_.batch - 1], ranges(a_, pre_[a_.batch - 1])) {
    c = blockIdx.x;
    const long long W = pre[a.batch - 1];
    u = u_end = 0;
    if (c >= W) return;
    u = split.begin(c);
    u_end = split.begin(c + 1);
    // the request: first r with pre[r] > u
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] > u) hi = mid; else lo = mid + 1;
    }
    r = lo;
    attn_req(a, r, q);
    const long long base = r ? pre[r - 1] : 0;
    const long long per = quot(pre[r] - base, a.nkv);
    h = (int)quot(u - base, per);
    long long rem = (u - base) - h * per;
    // the item tile: 32 at a time
    const int lane = threadIdx.x & 31, nt = attn_tiles(a, q.n);
    t = 0;
    for (int t0 = 0; nt > 1; t0 += 32) {
      int k = 0;
      if (t0 + lane < nt) {
        k = item_units<KL>(tile_range<KL>(a, q, t0 + lane));
      }
      long long v = k;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long w = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += w;
      }
      const unsigned past = __ballot_sync(0xffffffffu, v > rem);
      if (past == 0 && t0 + 32 < nt) {
        rem -= __shfl_sync(0xffffffffu, v, 31);
        continue;
      }
      const int l = past ? __ffs(past) - 1 : 31;
      t = t0 + l;
      rem -= __shfl_sync(0xffffffffu, v - k, l);
      break;
    }
    set_item((int)rem);
    if (kbeg == kend) next();  // the range begins behind the item's last tile
  }
  __device__ bool done() const { return u >= u_end; }
  __device__ void set_item(int skip) {
    x = tile_range<KL>(a, q, t);
    const int n = x.k1 - x.k0;
    off = skip;
    take = (int)min((long long)item_units<KL>(x) - skip, u_end - u);
    kbeg = x.k0 + min(skip, n);
    kend = x.k0 + min(skip + take, n);
  }
  __device__ void next() {
    u += take;
    if (u >= u_end) return;
    int nt = attn_tiles(a, q.n);
    do {
      if (++t >= nt) {
        t = 0;
        if (++h >= a.nkv) {
          h = 0;
          do ++r; while (pre[r] == pre[r - 1]);
          attn_req(a, r, q);
          nt = attn_tiles(a, q.n);
        }
      }
      set_item(0);
    } while (kbeg == kend);
  }
  __device__ bool whole() const { return kbeg == x.k0 && kend == x.k1; }
  // the CTAs that share the item's tiles, and the partial slot of CTA x among them:
  // 2 x for what begins its range, 2 x + 1 for a later segment
  __device__ long long item_begin() const { return u - off; }
  __device__ int cta_first() const { return split.owner(item_begin()); }
  __device__ int cta_last() const { return split.owner(item_begin() + (x.k1 - x.k0) - 1); }
  __device__ int slot() const { return 2 * c + (u != split.begin(c) ? 1 : 0); }
  // 1 when the item is not what begins the range of CTA c0 = cta_first()
  __device__ int later_in(int c0) const { return item_begin() != split.begin(c0) ? 1 : 0; }
  __device__ int tokens() const { return min(a.ipt, q.n - t * a.ipt); }
};

// Keys that only some rows of an item see.  The tensor-core pass multiplies the
// weight of a key that a row does not see, exactly 0, with the key's values, and 0
// times an infinity or NaN would poison the row.  So the values of keys that no row of
// the item sees are replaced by zeros before the product, and of keys that some rows
// see the values that are not finite are taken out (as zeros); add_taken_out then adds
// them to the rows that do see their key.
struct ItemKeys {
  int lo, hi;          // some row sees the keys [lo, hi)
  int all_lo, all_hi;  // all rows see [all_lo, all_hi), which may be empty (all_lo >= all_hi)
  __device__ ItemKeys(const PagedAttnArgs& a, const AttnReq& q, int tok0, int tokens)
      : lo(row_lo(a, q.st + tok0)),
        hi(row_hi(a, q, q.st + tok0 + tokens - 1)),
        all_lo(row_lo(a, q.st + tok0 + tokens - 1)),
        all_hi(row_hi(a, q, q.st + tok0)) {}
};

// The halves of a pair of 16-bit values that are not finite.
template <typename T> __device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  constexpr uint32_t E = __is_same(T, __half) ? 0x7c00u : 0x7f80u;
  return ((v & E) == E ? 0xffffu : 0u) | ((v & (E << 16)) == (E << 16) ? 0xffff0000u : 0u);
}

// Takes the values that are not finite out of the rows [r0, r1) of a tile of values in
// shared memory (swizzled 128-byte rows, 64-column halves KT rows apart), and says so in
// *taken before it does: another warp that finds them gone finds *taken set.  Called by
// a warp.  0 x v + sum stays 0 as long as every v is finite.
template <typename T, int HD, int KT>
__device__ __forceinline__ void take_out(uint8_t* tile, int r0, int r1, int lane, int* taken) {
  using T2 = std::conditional_t<__is_same(T, __half), __half2, __nv_bfloat162>;
  const uint32_t zero = 0;
  const T2 z = *reinterpret_cast<const T2*>(&zero);
  T2 sum[4] = {z, z, z, z};
#pragma unroll 1
  for (int c = r0 * 8 + lane; c < r1 * 8; c += 32)
#pragma unroll
    for (int hf = 0; hf < HD / 64; ++hf) {
      const uint4 w = *reinterpret_cast<const uint4*>(tile + hf * KT * 128 + c * 16);
      const T2* v = reinterpret_cast<const T2*>(&w);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = __hfma2(v[i], z, sum[i]);
    }
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bits |= *reinterpret_cast<const uint32_t*>(&sum[i]);
  __threadfence_block();
  if (!__any_sync(0xffffffffu, (bits & 0x7fff7fffu) != 0)) return;
  if (lane == 0) *(volatile int*)taken = 1;
  __threadfence_block();
  __syncwarp();
#pragma unroll 1
  for (int c = r0 * 8 + lane; c < r1 * 8; c += 32)
#pragma unroll 1
    for (int hf = 0; hf < HD / 64; ++hf) {
      uint32_t* w = reinterpret_cast<uint32_t*>(tile + hf * KT * 128 + c * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] &= ~not_finite<T>(w[i]);
    }
}

// Zeros in the rows [r0, r1) of such a tile.
template <int HD, int KT>
__device__ __forceinline__ void zero_values(uint8_t* tile, int r0, int r1, int lane) {
#pragma unroll 1
  for (int c = r0 * 8 + lane; c < r1 * 8; c += 32)
#pragma unroll
    for (int hf = 0; hf < HD / 64; ++hf)
      *reinterpret_cast<uint4*>(tile + hf * KT * 128 + c * 16) = make_uint4(0, 0, 0, 0);
}

// The rows [b0, b1) of a tile of values with keys that not every row of the item sees
// (ItemKeys, relative to the tile's first key).  Called by a warp.
template <typename T, int HD, int KT>
__device__ __forceinline__ void edge_values(uint8_t* tile, int b0, int b1, int lo, int hi,
                                            int all_lo, int all_hi, int lane, int* taken) {
  lo = max(b0, min(lo, b1));
  hi = max(lo, min(hi, b1));
  all_lo = max(lo, min(all_lo, hi));
  all_hi = max(all_lo, min(all_hi, hi));
  zero_values<HD, KT>(tile, b0, lo, lane);
  zero_values<HD, KT>(tile, hi, b1, lane);
  if (lo < all_lo) take_out<T, HD, KT>(tile, lo, all_lo, lane, taken);
  if (all_hi < hi) take_out<T, HD, KT>(tile, all_hi, hi, lane, taken);
}

// Adds what was taken out of the keys [from, to) of an item of `tokens` tokens from
// tok0 on, to the columns [c0, c1) of its rows: w v for every value v that is not
// finite of a key that the row sees.  A row a lane: its token, its query head within
// the group, its reference maximum in log2 units and where its columns are (null: not
// written), fp32 in a partial and T in the output.  At most 2 (tokens - 1) keys are
// looked at, however long the context is.  Called by a warp.
template <typename T, int HD>
__device__ __noinline__ void add_taken_out(const PagedAttnArgs& a, int r, int h,
                                           AttnReq q, int tok0, int tokens, int from, int to,
                                           int lane, int tok, int g, float ref,
                                           void* dst, bool partial, int c0, int c1) {
  constexpr int V = HD / 32;
  const ItemKeys keys(a, q, tok0, tokens);
  from = max(from, keys.lo);
  to = min(to, keys.hi);
  const int32_t* tab = a.table + (int64_t)r * a.max_pages;
  const unsigned on = __ballot_sync(0xffffffffu, dst != nullptr);
  const int col = lane * V;
  for (int key = from; key < to; ++key) {
    if (key >= keys.all_lo && key < keys.all_hi) {
      key = keys.all_hi - 1;
      continue;
    }
    const int pg = a.by_page.div(key), e = tab[pg];
    if (e < 0 || e >= a.n_pages) continue;
    const int64_t at = (((int64_t)e * a.nkv + h) * a.page + key - pg * a.page) * HD + col;
    const T* vr = static_cast<const T*>(a.v_pool) + at;
    const T* kr = static_cast<const T*>(a.k_pool) + at;
    float v[V], k[V];
    bool odd = false;
#pragma unroll
    for (int d = 0; d < V; ++d) {
      v[d] = to_f(vr[d]);
      odd |= !isfinite(v[d]);
    }
    if (!__any_sync(0xffffffffu, odd)) continue;
#pragma unroll
    for (int d = 0; d < V; ++d) k[d] = to_f(kr[d]);
    const int p = q.st + tok;
    unsigned sees = on & __ballot_sync(0xffffffffu, key >= row_lo(a, p) && key < row_hi(a, q, p));
    for (; sees; sees &= sees - 1) {
      const int i = __ffs(sees) - 1;
      const int ti = __shfl_sync(0xffffffffu, tok, i), gi = __shfl_sync(0xffffffffu, g, i);
      const float ri = __shfl_sync(0xffffffffu, ref, i);
      void* di = reinterpret_cast<void*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), i));
      const T* qr = static_cast<const T*>(a.q) + (int64_t)(q.row0 + ti) * a.q_stride +
                    (int64_t)(h * a.G + gi) * HD + col;
      float s = 0.f;
#pragma unroll
      for (int d = 0; d < V; ++d) s += to_f(qr[d]) * k[d];
      const float w = ex2_ftz(fmaf(warp_sum(s), a.scale_log2, -ri));
#pragma unroll
      for (int d = 0; d < V; ++d) {
        if (isfinite(v[d]) || col + d < c0 || col + d >= c1) continue;
        if (partial) {
          static_cast<float*>(di)[col + d] += w * v[d];
        } else {
          T* o = static_cast<T*>(di) + col + d;
          *o = from_f<T>(to_f(*o) + w * v[d]);
        }
      }
    }
  }
}

}  // namespace dflash
