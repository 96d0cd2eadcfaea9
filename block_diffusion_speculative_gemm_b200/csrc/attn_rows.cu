// Row operators in front of a paged attention call: per-head RMSNorm with the
// rotate-half position rotation (queries and keys), and the append of a
// chunk's keys (normalised, rotated) and values to a paged K/V cache.
//
//   norm(x)    = x * rsqrt(mean(x^2) + eps) * g            (g null: x unchanged)
//   rope(y, p) = (a cos - b sin, b cos + a sin), y = (a, b) in halves, cos and
//                sin the table rows of position p          (no table: y unchanged)
//
// A head row is held by head_dim / 16 lanes, a lane with 8 consecutive values
// of each half, so a rotation pair never leaves its thread, the norm's sum
// takes 2 or 3 shuffles, and every global access is 16 bytes.  A group of
// lanes stays on one row and walks over its heads (kUnroll of them in flight), so
// the table row sits in registers.  Sums and products are fp32; each value is
// rounded once, when it is stored.  Bound by memory: every value is read once
// and written once.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace dflash {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // heads a lane group has in flight

// 8 elements as raw 16-byte words, loaded now and converted later.
template <typename T> struct Raw8 {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const T* h = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f(h[i]);
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// 8 elements of shared memory.
template <typename T> __device__ __forceinline__ void lds8(const T* p, float (&v)[8]) {
  Raw8<T> r;
  r.w = *reinterpret_cast<const uint4*>(p);
  r.get(v);
}
template <> __device__ __forceinline__ void lds8<float>(const float* p, float (&v)[8]) {
  Raw8<float> r;
  r.a = reinterpret_cast<const float4*>(p)[0];
  r.b = reinterpret_cast<const float4*>(p)[1];
  r.get(v);
}

// Rounds and stores 8 values; true when one does not fit the element type.
template <typename T>
__device__ __forceinline__ bool put8(T* dst, const float (&v)[8]) {
  T h[8];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = from_f<T>(v[i]);
    bad |= narrow_bad<T>(v[i]);
  }
  *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(h);
  return bad;
}
template <>
__device__ __forceinline__ bool put8<float>(float* dst, const float (&v)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
  return false;
}

// A lane's part of a head in pairs: 8 values of each half.  Both kernels use the
// same steps, so that a row's bits do not depend on which of them takes it.
struct HeadPart {
  uint64_t a[4], b[4];
  __device__ __forceinline__ void set(const float (&y1)[8], const float (&y2)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = pair(y1[2 * k], y1[2 * k + 1]);
      b[k] = pair(y2[2 * k], y2[2 * k + 1]);
    }
  }
  __device__ __forceinline__ void get(float (&y1)[8], float (&y2)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      unpair(a[k], y1[2 * k], y1[2 * k + 1]);
      unpair(b[k], y2[2 * k], y2[2 * k + 1]);
    }
  }
  __device__ __forceinline__ float sum_of_squares() const {
    uint64_t q = mul2(a[0], a[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) q = fma2(a[k], a[k], q);
#pragma unroll
    for (int k = 0; k < 4; ++k) q = fma2(b[k], b[k], q);
    float s0, s1;
    unpair(q, s0, s1);
    return s0 + s1;
  }
  __device__ __forceinline__ void scale(float inv, const uint64_t (&g)[8]) {
    const uint64_t f = pair(inv, inv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = mul2(mul2(a[k], f), g[k]);
      b[k] = mul2(mul2(b[k], f), g[4 + k]);
    }
  }
  // cs, sn: cosines and sines in pairs
  __device__ __forceinline__ void rotate(const uint64_t (&cs)[4], const uint64_t (&sn)[4]) {
    const uint64_t minus = pair(-1.f, -1.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t u = a[k];
      a[k] = fma2(u, cs[k], mul2(mul2(b[k], minus), sn[k]));
      b[k] = fma2(b[k], cs[k], mul2(u, sn[k]));
    }
  }
};

// What a warp learns about a row: its request's rows and first position.
struct RowOwner {
  int req, row0, n, st;
  int total;  // cu_rows[batch]
  bool order; // cu_rows ascends inside the rows (as far as this search saw it)
};

// The request that holds `row` (the last one whose first row is <= row), by a
// search over 32 probes a round: one round up to 32 requests, two up to 1024.
// Where cu_rows does not ascend the answer means nothing: owner_in_order has it then.
__device__ __forceinline__ RowOwner find_owner(const int32_t* cu, const int32_t* start, int batch,
                                               int n_rows, int row, int lane) {
  RowOwner o;
  o.order = true;
  if (batch <= 32) {
    const int l = min(lane, batch - 1);
    const int a = cu[l], b = cu[l + 1], st = start[l];
    const unsigned le = __ballot_sync(0xffffffffu, lane < batch && a <= row);
    o.order = __all_sync(0xffffffffu, !out_of_order(a, b, n_rows));
    o.req = le ? 31 - __clz(le) : 0;
    o.row0 = __shfl_sync(0xffffffffu, a, o.req);
    o.n = __shfl_sync(0xffffffffu, b, o.req) - o.row0;
    o.st = __shfl_sync(0xffffffffu, st, o.req);
    o.total = __shfl_sync(0xffffffffu, b, batch - 1);
    return o;
  }
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, i < n && cu[lo + min(i, n - 1)] <= row);
    const int k = le ? 31 - __clz(le) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  o.req = lo;
  o.row0 = cu[lo];
  o.n = cu[lo + 1] - o.row0;
  o.st = start[lo];
  o.total = cu[batch];
  return o;
}

// The requests in order that hold the rows [first, first + 32): own(r, a, b) on every
// lane of the warp for each of them.
template <typename F>
__device__ void owners_in_order(const int32_t* cu, int batch, int n_rows, int first, int lane,
                                F own) {
  each_request_order(cu, batch, n_rows, lane, [&](int r, bool ok, int a, int b) {
    for (unsigned hit = __ballot_sync(0xffffffffu, ok && a < first + 32LL && b > first && b > a);
         hit; hit &= hit - 1) {
      const int src = __ffs(hit) - 1;
      own(__shfl_sync(0xffffffffu, r, src), __shfl_sync(0xffffffffu, a, src),
          __shfl_sync(0xffffffffu, b, src));
    }
  });
}

struct RowArgs {
  const void *a, *b;          // [n_rows][heads][HD], row strides in elements
  int64_t a_stride, b_stride;
  const void *g_a, *g_b;      // [HD] of the inputs' type, or null: no norm
  float eps;
  const float* rope;          // [2][max_pos][HD / 2] cos then sin, or null
  int max_pos;
  const int32_t *cu, *start;
  int batch, n_rows, n_a, n_b;
  int groups_log2;            // lane groups per row
  void *oa, *ob;              // dense rows (kPaged false): row strides oa_stride, ob_stride
  int64_t oa_stride, ob_stride;
  const int32_t* table;       // paged (kPaged true): oa = K pool, ob = V pool
  int max_pages, page, n_pages;
  int32_t* err;
};

// kPaged false: a = queries, b = keys, both normalised and rotated into dense
// rows.  kPaged true: a = keys (normalised, rotated), b = values (copied), into
// the pages of [n_pages][heads][page][HD] pools.
template <typename TI, typename TO, int HD, bool kPaged>
__global__ void __launch_bounds__(kThreads) attn_rows_kernel(const RowArgs p) {
  pdl_trigger();
  pdl_wait();
  constexpr int kLanes = HD / 16, kHalf = HD / 2;
  const int tid = threadIdx.x, lane = tid & 31;
  const int grp = tid / kLanes, i0 = (tid % kLanes) * 8;
  const int gpr = 1 << p.groups_log2;  // at least 8, so that a warp's groups share their row
  const int row = blockIdx.x * ((kThreads / kLanes) >> p.groups_log2) + (grp >> p.groups_log2);
  const int hg = grp & (gpr - 1);
  const int nh = p.n_a + p.n_b;

  Raw8<TI> x[kUnroll][2];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * gpr;
      if (h < nh) {
        const TI* src = h < p.n_a
            ? static_cast<const TI*>(p.a) + (int64_t)row * p.a_stride + (int64_t)h * HD
            : static_cast<const TI*>(p.b) + (int64_t)row * p.b_stride + (int64_t)(h - p.n_a) * HD;
        x[u][0].load(src + i0);
        x[u][1].load(src + i0 + kHalf);
      }
    }
  };
  if (row < p.n_rows) fetch(hg);  // in flight while the row's request is looked up

  RowOwner o = find_owner(p.cu, p.start, p.batch, p.n_rows, row, lane);
  bool order = o.order;
  if (p.batch > 32) {  // the search saw a part of cu_rows only
    for (int r = tid; r < p.batch; r += kThreads)
      order &= !out_of_order(p.cu[r], p.cu[r + 1], p.n_rows);
    order = __syncthreads_and(order);
  }
  if (row >= p.n_rows) return;
  if (!order) {
    if (lane == 0) set_error(p.err, DFLASH_DEV_ROWS);
    o.n = 0;
    owners_in_order(p.cu, p.batch, p.n_rows, row, lane, [&](int r, int a, int b) {
      if (row < a || row >= b) return;
      o.req = r;
      o.row0 = a;
      o.n = b - a;
      o.st = p.start[r];
    });
    if (o.n == 0) return;
  } else {
    if (row >= o.total) return;  // padding behind the last request
    if (row < o.row0) {          // in front of the first one
      if (lane == 0) set_error(p.err, DFLASH_DEV_ROWS);
      return;
    }
  }
  // the whole request has to fit the table and the cache, else none of its rows is written
  const int64_t last = (int64_t)o.st + o.n - 1;
  int64_t cap = p.rope ? p.max_pos : INT64_MAX;
  if (kPaged) cap = min(cap, (int64_t)p.max_pages * p.page);
  if (o.st < 0 || last >= cap) {
    if (lane == 0) set_error(p.err, DFLASH_DEV_CTX_CAP);
    return;
  }
  const int pos = o.st + (row - o.row0);
  uint64_t cs[4], sn[4];
  if (p.rope) {
    const float* t = p.rope + (int64_t)pos * kHalf + i0;
    Raw8<float> c, s;
    c.load(t);
    s.load(t + (int64_t)p.max_pos * kHalf);
    float cv[8], sv[8];
    c.get(cv);
    s.get(sv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      cs[k] = pair(cv[2 * k], cv[2 * k + 1]);
      sn[k] = pair(sv[2 * k], sv[2 * k + 1]);
    }
  }
  int64_t slot = 0;  // paged: pool row of head 0
  if (kPaged) {
    const int32_t* tab = p.table + (int64_t)o.req * p.max_pages;
    bool bad = false;
    for (int k = o.st / p.page + lane; k <= (int)(last / p.page); k += 32) {
      const int e = tab[k];
      bad |= e < 0 || e >= p.n_pages;
    }
    const int e = tab[pos / p.page];
    if (__any_sync(0xffffffffu, bad)) {
      if (lane == 0) set_error(p.err, DFLASH_DEV_PAGE);
      return;
    }
    slot = (int64_t)e * p.n_a * p.page + pos % p.page;
  }

  bool bad = false;
  for (int h0 = hg;;) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * gpr;
      // every lane of the warp takes the shuffles; h is uniform over a group's lanes
      const bool live = h < nh, is_a = h < p.n_a;
      float y1[8], y2[8];
      HeadPart y;
      if (live) {
        x[u][0].get(y1);
        x[u][1].get(y2);
        y.set(y1, y2);
      }
      const TI* g = static_cast<const TI*>(is_a ? p.g_a : p.g_b);
      if (p.g_a != nullptr || p.g_b != nullptr) {
        float ss = live ? y.sum_of_squares() : 0.f;
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        if (live && g != nullptr) {
          Raw8<TI> gr;
          float gv[8];
          uint64_t g2[8];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            gr.load(g + half * kHalf + i0);
            gr.get(gv);
#pragma unroll
            for (int k = 0; k < 4; ++k) g2[half * 4 + k] = pair(gv[2 * k], gv[2 * k + 1]);
          }
          y.scale(rsqrtf(ss / HD + p.eps), g2);
        }
      }
      if (!live) continue;
      if (p.rope && (is_a || !kPaged)) y.rotate(cs, sn);
      y.get(y1, y2);
      TO* dst;
      if (kPaged) {
        const int64_t d = slot + (int64_t)(is_a ? h : h - p.n_a) * p.page;
        if (!DFLASH_CHECK(d >= 0 && d < (int64_t)p.n_pages * p.n_a * p.page, p.err)) continue;
        dst = static_cast<TO*>(is_a ? p.oa : p.ob) + d * HD;
      } else {
        dst = is_a ? static_cast<TO*>(p.oa) + (int64_t)row * p.oa_stride + (int64_t)h * HD
                   : static_cast<TO*>(p.ob) + (int64_t)row * p.ob_stride +
                         (int64_t)(h - p.n_a) * HD;
      }
      bad |= put8<TO>(dst + i0, y1) | put8<TO>(dst + i0 + kHalf, y2);
    }
    // uniform over the warp: its groups' first heads differ by less than gpr
    h0 += kUnroll * gpr;
    if (h0 - hg >= nh) break;
    fetch(h0);
  }
  if (bad) set_error(p.err, DFLASH_DEV_RANGE);
}


// ---------------------------------------------------------------- many rows
// The same operators for many rows.  A CTA has a range of rows; one warp looks up
// each row's request, position and page, and brings the row and its line of the
// rotation table into a ring of shared-memory stages by bulk copies, so that no
// load of the compute warps waits for another one and 100 KB and more are in
// flight per SM without a register.  Compute warp w of W takes the rows w, w + W, ...
// in two stages of its own (a stage that changed hands could be waited for a whole
// round early) and writes its results straight from registers.  16384 rows of 32
// query and 8 key heads of 128 bf16: 65 us (5.3 TB/s), against 91 with a thread's
// loads behind its lookups; their append to a bf16 cache 28 us against 50.  The ring
// holds whole rows, at least 16: rows of more than 53 heads of 128 in 16 bits or 26 in
// fp32 (about twice as many of 64) take the other kernel (64 / 8 bf16 132 us, 32 / 8 fp32 133 us,
// 4.6 and 5.1 TB/s).
constexpr int kStreamMax = 32;  // stages, two a warp
constexpr int kStreamSmem = 220 * 1024;

struct StreamRow {
  int row;       // -1: nothing to do
  int pad;
  int64_t slot;  // paged: pool row of head 0
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Bytes of a stage: a row's heads, then its cosines and sines.
template <typename TI, int HD> __host__ __device__ constexpr int stream_stage(int heads) {
  return heads * HD * (int)sizeof(TI) + HD * 4;
}

template <typename TI, typename TO, int HD, bool kPaged>
__global__ void __launch_bounds__(kStreamMax / 2 * 32 + 32)
    attn_rows_stream_kernel(const RowArgs p, int stages, int pass) {
  pdl_trigger();
  constexpr int kLanes = HD / 16, kHalf = HD / 2, kHeads = 32 / kLanes;  // heads a warp takes at once
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2 * kStreamMax];
  __shared__ StreamRow info[kStreamMax];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = stages / 2;
  const int nh = p.n_a + p.n_b, stage = stream_stage<TI, HD>(nh);
  const uint32_t base = smem_u32(smem);
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[kStreamMax + s]); };
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    fence_barrier_init();
  }
  pdl_wait();
  bool order = true;
  for (int r = tid; r < p.batch; r += blockDim.x)
    order &= !out_of_order(p.cu[r], p.cu[r + 1], p.n_rows);
  order = __syncthreads_and(order);
  const int r_begin = (int)((int64_t)p.n_rows * blockIdx.x / gridDim.x);
  const int count = (int)((int64_t)p.n_rows * (blockIdx.x + 1) / gridDim.x) - r_begin;
  bool ok = true;

  if (warp == warps) {
    // ------------------------------------------------------------ loads
    const int total = p.cu[p.batch];
    if (!order && lane == 0) set_error(p.err, DFLASH_DEV_ROWS);
    int checked = -1;     // the request whose pages were looked through
    bool mapped = true;
    int s = 0, phase = 1;  // stage, parity of its last release (none yet)
    int i = 0;
    for (; i < count && ok; i += 32) {
      // a row per lane: its request (the last one that starts at or before it)
      const int row = r_begin + i + lane;
      int req = 0, row0 = 0, n = 0, st = 0;
      bool good = i + lane < count && (row < total || !order);
      if (!order) {
        owners_in_order(p.cu, p.batch, p.n_rows, r_begin + i, lane, [&](int r, int a, int b) {
          if (row < a || row >= b) return;
          req = r;
          row0 = a;
          n = b - a;
          st = p.start[r];
        });
        good = good && n > 0;
      } else if (good) {
        int lo = 0, hi = p.batch - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.cu[mid] <= row) lo = mid; else hi = mid - 1;
        }
        req = lo;
        row0 = p.cu[lo];
        n = p.cu[lo + 1] - row0;
        st = p.start[lo];
        if (row < row0) {  // in front of the first request
          set_error(p.err, DFLASH_DEV_ROWS);
          good = false;
        }
      }
      // the whole request has to fit the table and the cache, else none of its rows is written
      const int64_t last = (int64_t)st + n - 1;
      int64_t cap = p.rope ? p.max_pos : INT64_MAX;
      if (kPaged) cap = min(cap, (int64_t)p.max_pages * p.page);
      if (good && (st < 0 || last >= cap)) {
        set_error(p.err, DFLASH_DEV_CTX_CAP);
        good = false;
      }
      const int pos = st + (row - row0);
      int64_t slot = 0;
      if (kPaged) {
        // every request among the 32 rows once
        for (unsigned todo = __ballot_sync(0xffffffffu, good); todo;) {
          const int src = __ffs(todo) - 1, rq = __shfl_sync(0xffffffffu, req, src);
          if (rq != checked) {
            const int first = __shfl_sync(0xffffffffu, st, src);
            const int end = __shfl_sync(0xffffffffu, (int)last, src);
            const int32_t* tab = p.table + (int64_t)rq * p.max_pages;
            bool bad = false;
            for (int k = first / p.page + lane; k <= end / p.page; k += 32) {
              const int e = tab[k];
              bad |= e < 0 || e >= p.n_pages;
            }
            mapped = !__any_sync(0xffffffffu, bad);
            checked = rq;
            if (!mapped && lane == 0) set_error(p.err, DFLASH_DEV_PAGE);
          }
          const bool mine = good && req == rq;
          todo &= ~__ballot_sync(0xffffffffu, mine);
          if (mine && !mapped) good = false;
        }
        if (good) {
          const int pg = pos / p.page;
          const int e = p.table[(int64_t)req * p.max_pages + pg];
          slot = (int64_t)e * p.n_a * p.page + pos - pg * p.page;
        }
      }
      // `pass` lanes at a time bring their rows, each into a stage of its own
      for (int j = 0; j < 32 && i + j < count; j += pass) {
        const bool mine = lane >= j && lane < j + pass && i + lane < count;
        int sl = s + lane - j, ph = phase;
        if (sl >= stages) {
          sl -= stages;
          ph ^= 1;
        }
        if (!__all_sync(0xffffffffu,
                        !mine || i + lane < stages || mbar_wait_nap(empty(sl), ph))) {
          ok = false;
          break;
        }
        if (mine) {
          info[sl].row = good ? row : -1;
          info[sl].slot = slot;
          if (!good) {
            mbar_arrive(full(sl));
          } else {
            const uint32_t dst = base + (uint32_t)(sl * stage);
            const uint32_t an = p.n_a * HD * sizeof(TI), bn = p.n_b * HD * sizeof(TI);
            mbar_arrive_expect_tx(full(sl), an + bn + (p.rope ? HD * 4 : 0));
            if (an) bulk_load(dst, static_cast<const TI*>(p.a) + row * p.a_stride, an, full(sl));
            if (bn)
              bulk_load(dst + an, static_cast<const TI*>(p.b) + row * p.b_stride, bn, full(sl));
            if (p.rope) {
              const float* t = p.rope + (int64_t)pos * kHalf;
              bulk_load(dst + an + bn, t, kHalf * 4, full(sl));
              bulk_load(dst + an + bn + kHalf * 4, t + (int64_t)p.max_pos * kHalf, kHalf * 4,
                        full(sl));
            }
          }
        }
        __syncwarp();
        s += min(pass, count - i - j);
        if (s >= stages) {
          s -= stages;
          phase ^= 1;
        }
      }
    }
    // after a wait that gave up: the copies in flight land before the CTA may end
    if (!ok)
      for (int k = 0; k < stages; ++k) mbar_wait(full(k), k < s ? phase ^ 1 : phase);
  } else {
    // ------------------------------------------------------------ rows
    const int i0 = (lane % kLanes) * 8, hg = lane / kLanes;
    uint64_t ga[8], gb[8];  // gains of this lane's columns, in pairs
    auto gains = [&](const void* g, uint64_t (&v)[8]) {
      Raw8<TI> r;
      float t[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (g != nullptr) {
          r.load(static_cast<const TI*>(g) + half * kHalf + i0);
          r.get(t);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[half * 4 + i] = g != nullptr ? pair(t[2 * i], t[2 * i + 1]) : pair(1.f, 1.f);
      }
    };
    gains(p.g_a, ga);
    if (!kPaged) gains(p.g_b, gb);
    bool bad = false;
    int s = warp, phase = 0;
    for (int i = warp; i < count; i += warps) {
      if (!__all_sync(0xffffffffu, mbar_wait_nap(full(s), phase))) {
        ok = false;
        break;
      }
      const int64_t row = info[s].row, slot = info[s].slot;
      if (row >= 0) {
        const uint8_t* x = smem + s * stage;
        uint64_t cs[4], sn[4];
        if (p.rope) {
          const float* t = reinterpret_cast<const float*>(x + nh * HD * sizeof(TI)) + i0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 c = *reinterpret_cast<const float2*>(t + 2 * k);
            const float2 v = *reinterpret_cast<const float2*>(t + kHalf + 2 * k);
            cs[k] = pair(c.x, c.y);
            sn[k] = pair(v.x, v.y);
          }
        }
#pragma unroll 1
        for (int h0 = 0; h0 < nh; h0 += kHeads) {
          const int h = h0 + hg;
          const bool live = h < nh, is_a = h < p.n_a;
          float y1[8], y2[8];
          const TI* src = reinterpret_cast<const TI*>(x) + min(h, nh - 1) * HD + i0;
          lds8(src, y1);
          lds8(src + kHalf, y2);
          HeadPart y;
          y.set(y1, y2);
          if (p.g_a != nullptr || (!kPaged && p.g_b != nullptr)) {
            float ss = y.sum_of_squares();
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            if (is_a ? p.g_a != nullptr : !kPaged && p.g_b != nullptr) {
              const float inv = rsqrtf(ss / HD + p.eps);
              if (is_a || kPaged) y.scale(inv, ga); else y.scale(inv, gb);
            }
          }
          if (!live) continue;
          if (p.rope && (is_a || !kPaged)) y.rotate(cs, sn);
          y.get(y1, y2);
          TO* dst;
          if (kPaged) {
            const int64_t d = slot + (int64_t)(is_a ? h : h - p.n_a) * p.page;
            if (!DFLASH_CHECK(d >= 0 && d < (int64_t)p.n_pages * p.n_a * p.page, p.err)) continue;
            dst = static_cast<TO*>(is_a ? p.oa : p.ob) + d * HD;
          } else {
            dst = is_a ? static_cast<TO*>(p.oa) + row * p.oa_stride + (int64_t)h * HD
                       : static_cast<TO*>(p.ob) + row * p.ob_stride + (int64_t)(h - p.n_a) * HD;
          }
          bad |= put8<TO>(dst + i0, y1) | put8<TO>(dst + i0 + kHalf, y2);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
      s += warps;
      if (s >= stages) {
        s -= stages;
        phase ^= 1;
      }
    }
    if (bad) set_error(p.err, DFLASH_DEV_RANGE);
  }
  if (!ok && lane == 0) set_error(p.err, DFLASH_DEV_TIMEOUT);
}

template <typename TI, typename TO, int HD, bool kPaged>
int launch_stream(const RowArgs& a, int stages, int stage, cudaStream_t s) {
  const auto kernel = attn_rows_stream_kernel<TI, TO, HD, kPaged>;
  static SmemLimit limit;
  if (!limit.raise(reinterpret_cast<const void*>(kernel), kStreamSmem)) return DFLASH_ECUDA;
  const cudaError_t e = launch_pdl(kernel, dim3(num_sms()), dim3(stages / 2 * 32 + 32),
                                   (size_t)stages * stage, s, 1, a, stages,
                                   stages <= 20 ? 4 : 8);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ECUDA;
}

template <typename TI, typename TO, bool kPaged>
int launch_rows(const RowArgs& a0, int hd, cudaStream_t s) {
  RowArgs a = a0;
  const int groups = kThreads / (hd / 16);
  TimedScope ts(s, TC_ROW);
  if (a.n_rows > 8 * num_sms()) {
    const int heads = a.n_a + a.n_b;
    const int64_t stage = hd == 128 ? stream_stage<TI, 128>(std::min(heads, 4096))
                                    : stream_stage<TI, 64>(std::min(heads, 4096));
    const int stages = (int)std::min<int64_t>(kStreamMax, kStreamSmem / stage) & ~1;
    if (stages >= 16)
      return hd == 128 ? launch_stream<TI, TO, 128, kPaged>(a, stages, (int)stage, s)
                       : launch_stream<TI, TO, 64, kPaged>(a, stages, (int)stage, s);
  }
  // Few rows: a CTA per row, so that a row's heads run side by side.  Many
  // rows: 8 groups a row, which then keep the table row over several heads.
  a.groups_log2 = a.n_rows <= 8 * num_sms() ? (hd == 128 ? 5 : 6) : 3;
  const int rows = groups >> a.groups_log2;
  const dim3 grid((a.n_rows + rows - 1) / rows);
  const cudaError_t e =
      hd == 128 ? launch_pdl(attn_rows_kernel<TI, TO, 128, kPaged>, grid, dim3(kThreads), 0, s, 1, a)
                : launch_pdl(attn_rows_kernel<TI, TO, 64, kPaged>, grid, dim3(kThreads), 0, s, 1, a);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ECUDA;
}

}  // namespace

int launch_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                        int dtype, const void* g_q, const void* g_k, float eps, const float* rope,
                        int max_pos, const int32_t* cu, const int32_t* start, int batch,
                        int n_rows, int n_q, int n_kv, int hd, void* q_out, int64_t q_out_stride,
                        void* k_out, int64_t k_out_stride, int32_t* err, cudaStream_t s) {
  RowArgs a = {q, k, q_stride, k_stride, g_q, g_k, eps, rope, max_pos, cu, start, batch, n_rows,
               n_q, n_kv, 0, q_out, k_out, q_out_stride, k_out_stride, nullptr, 0, 0, 0, err};
  if (dtype == DFLASH_BF16) return launch_rows<__nv_bfloat16, __nv_bfloat16, false>(a, hd, s);
  if (dtype == DFLASH_F16) return launch_rows<__half, __half, false>(a, hd, s);
  return launch_rows<float, float, false>(a, hd, s);
}

int launch_kv_append_paged(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           int dtype, const void* g_k, float eps, const float* rope, int max_pos,
                           const int32_t* cu, const int32_t* start, int batch, int n_rows,
                           int n_kv, int hd, void* k_pool, void* v_pool, int cache_dtype,
                           const KvPages& pg, int32_t* err, cudaStream_t s) {
  RowArgs a = {k, v, k_stride, v_stride, g_k, nullptr, eps, rope, max_pos, cu, start, batch,
               n_rows, n_kv, n_kv, 0, k_pool, v_pool, 0, 0, pg.table, pg.max_pages, pg.page,
               pg.n_pages, err};
  const bool b = cache_dtype == DFLASH_BF16;
  if (dtype == DFLASH_BF16)
    return b ? launch_rows<__nv_bfloat16, __nv_bfloat16, true>(a, hd, s)
             : launch_rows<__nv_bfloat16, __half, true>(a, hd, s);
  if (dtype == DFLASH_F16)
    return b ? launch_rows<__half, __nv_bfloat16, true>(a, hd, s)
             : launch_rows<__half, __half, true>(a, hd, s);
  return b ? launch_rows<float, __nv_bfloat16, true>(a, hd, s)
           : launch_rows<float, __half, true>(a, hd, s);
}

}  // namespace dflash
