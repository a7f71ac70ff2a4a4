// The paged key/value cache: page tables from request lengths, and the write
// of entries into pages.
//
// Source of the entries: "Maglev: Sliding Recurrent Memory", paper.rainbus.top,
// 方法步骤详情 (k_rec = RMSNorm(W_k^rec m'_{t-1}), both keys RoPE-rotated, gates
// g = 2 sigmoid(a)) and 前置知识 (the cache is that of plain attention).
#include "paged.cuh"

namespace maglev {
namespace {

// ---------------------------------------------------------------------------
// Page tables. A finished request (new < 0) gives the pages of its held(b) =
// ceil(ctx / page_size) columns back, from the first that is not negative on (the ones
// before it were given back when a window had passed them); the others need need(b) =
// ceil((ctx + new) / page_size) - held(b). With the stack of free pages
// S = free[0..n) followed by the returned pages, request b is served when the
// inclusive prefix sum of need up to b is at most |S| (or need(b) == 0), and
// page i of all pages handed out is S[|S| - 1 - i]. So one prefix sum over the
// requests places every page, and then every token row is independent.
//
// What bounds it is latency: a few KB are read and 16 bytes a token written. So the
// plan (one block: prefix sums over the requests) takes one barrier a sum, the
// fill (a thread per token row) finds its requests by block-wide counts instead of a
// chain of probes, and is scheduled while the plan runs. Up to ONE_LAUNCH_ROWS rows
// the plan's block does the rows itself. GPU time: 64 single tokens 3.3 us, 96
// prompts and ends (74 k rows) 6.2 us, 2048 requests (52 k rows) 10.7 us.
// ---------------------------------------------------------------------------
struct PlanTotals {
  int64_t n_old, avail, left;  // free pages before, with the returned ones, after
  int finished;                // requests
};
struct PlanViews {
  PlanTotals* totals;
  int2* req;  // [B] first position of a served request's tokens (else -1), pages handed out to earlier requests
  int4* fin;  // [finished] pages returned up to and with a finished request, which it is, its first column with a page
};
__device__ __forceinline__ PlanViews plan_views(void* ws, int B) {
  char* p = static_cast<char*>(ws);
  PlanViews v;
  v.totals = reinterpret_cast<PlanTotals*>(p);
  v.fin = reinterpret_cast<int4*>(p + 256);
  v.req = reinterpret_cast<int2*>(v.fin + B);
  return v;
}

constexpr int PLAN_THREADS = 1024;  // at most
constexpr int PLAN_EACH = 2;        // requests of a thread, kept in registers
constexpr int FILL_ROWS = 256;      // token rows (and threads) of a block of the fill

// Exclusive prefix sums of x and y over the block, one barrier; sums of x stop at
// `most` (saturating addition is associative). sums [32] is used once.
__device__ __forceinline__ uint2 block_exclusive(uint2 v, uint32_t most, uint2* sums, uint2* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  auto scan = [&](uint2 z) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, z.x, o), y = __shfl_up_sync(0xffffffffu, z.y, o);
      if (lane >= o) z = make_uint2(min(z.x + x, most), z.y + y);
    }
    return z;
  };
  auto from = [&](uint2 z, int l) {
    return make_uint2(__shfl_sync(0xffffffffu, z.x, l), __shfl_sync(0xffffffffu, z.y, l));
  };
  const uint2 inc = scan(v);
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  // every warp sums the warps' sums for itself
  const uint2 all = scan(lane < (int)blockDim.x / 32 ? sums[lane] : make_uint2(0, 0));
  *total = from(all, 31);
  const uint2 before = from(all, warp > 0 ? warp - 1 : 0), own = from(inc, lane > 0 ? lane - 1 : 0);
  uint2 r = lane > 0 ? own : make_uint2(0, 0);
  if (warp > 0) r = make_uint2(min(r.x + before.x, most), r.y + before.y);
  return r;
}

// The first b in [lo, hi) with x(b) > t (hi if none): x is non-decreasing.
template <typename X, typename V>
__device__ __forceinline__ int first_above(X x, int lo, int hi, V t) {
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (x(mid) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}
// The same for two values t <= u and the whole block: each round reads a value a
// thread and counts, so B requests take log(B) / log(threads) rounds of loads.
__device__ __forceinline__ void block_first_above(const int64_t* x, int n, int64_t t, int64_t u, int* at, int* au) {
  int lo[2] = {0, 0}, len[2] = {n, n};
  while (len[0] > 0 || len[1] > 0) {
    int64_t v[2];
    int step[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // thread i stands for the `step` values from i * step
      step[e] = (len[e] + (int)blockDim.x - 1) / (int)blockDim.x;
      const int i = ((int)threadIdx.x + 1) * step[e] - 1;
      v[e] = (int)threadIdx.x * step[e] < len[e] ? x[lo[e] + (i < len[e] ? i : len[e] - 1)] : INT64_MAX;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int before = __syncthreads_count(v[e] <= (e ? u : t)) * step[e];  // values in shares that lie before
      lo[e] += before < len[e] ? before : len[e];
      len[e] = step[e] > 1 && before < len[e] ? (len[e] - before < step[e] ? len[e] - before : step[e]) : 0;
    }
  }
  *at = lo[0];
  *au = lo[1];
}

// Page k of the pages that finished requests return (request, then column order).
__device__ __forceinline__ int returned_page(const PageTablesArgs& a, const int4* fin, int finished, int k) {
  const int i = first_above([&](int j) { return fin[j].x; }, 0, finished, k);
  if (i >= finished) return -1;
  return a.block_table[(int64_t)fin[i].y * a.max_pages + fin[i].z + (k - (i > 0 ? fin[i - 1].x : 0))];
}

// Row b's first column. Negative columns come first, so where it names a page the row is whole.
__device__ __forceinline__ int first_column(const PageTablesArgs& a, int b) {
  return a.block_table[(int64_t)b * a.max_pages];
}
// The first of row b's `held` columns that is not negative (held, if there is none), where the very first one is
// negative: searched by 8 columns at a time.
__device__ __forceinline__ int first_page(const PageTablesArgs& a, int b, int held) {
  const int32_t* row = a.block_table + (int64_t)b * a.max_pages;
  int lo = 1, len = held - 1;  // it lies in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 7) / 8;
    int negative = 0;  // shares [lo + u step, lo + (u + 1) step) of which even the last column is
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = (u + 1) * step - 1;
      negative += u * step < len && row[lo + (i < len ? i : len - 1)] < 0;
    }
    const int before = negative * step < len ? negative * step : len;
    lo += before;
    len = before < len ? min(step - 1, len - before) : 0;
  }
  return lo;
}

// What a fill needs of the requests that its rows belong to.
struct FillRequests {
  int end[FILL_ROWS + 1];  // where their rows end, from the fill's first row; [0]: where the first request's begin
  int2 at[FILL_ROWS];      // start, need_ex
  int4 fin[FILL_ROWS];     // finished requests, if there are no more
};
// The finished requests, staged (a barrier has to follow before they are used).
__device__ __forceinline__ const int4* stage_finished(const PlanViews& w, int finished, FillRequests& f) {
  if (finished > FILL_ROWS) return w.fin;
  for (int i = threadIdx.x; i < finished; i += blockDim.x) f.fin[i] = w.fin[i];
  return f.fin;
}

// Token rows [t0, t0 + FILL_ROWS) of the map, and with them the table columns whose
// page a row is the first of.
__device__ void fill_rows(const PageTablesArgs& a, const PlanViews& w, const PlanTotals& tot, const int4* fin, int shift,
                          int64_t t0, FillRequests& f, int* err) {
  const int64_t t1 = t0 + FILL_ROWS < a.n_tokens ? t0 + FILL_ROWS : a.n_tokens;
  int b0 = 0, b1 = 0;  // the requests these rows belong to
  if (a.pad == 0) block_first_above(a.cu_tokens + 1, a.B, t0, t1 - 1, &b0, &b1);
  const bool staged = a.pad == 0 && b1 - b0 < FILL_ROWS;  // not with that many requests without rows between
  if (staged) {
    for (int i = threadIdx.x; i <= b1 - b0 + 1 && b0 + i <= a.B; i += blockDim.x) {
      f.end[i] = (int)(a.cu_tokens[b0 + i] - t0);
      if (i <= b1 - b0 && b0 + i < a.B) f.at[i] = w.req[b0 + i];
    }
  }
  __syncthreads();
  for (int64_t t = t0 + threadIdx.x; t < t1; t += blockDim.x) {
    int b;
    int2 at = make_int2(-1, 0);
    int64_t i = 0;
    if (staged) {
      const int x = (int)(t - t0), k = first_above([&](int j) { return f.end[j + 1]; }, 0, b1 - b0, x);
      b = b0 + k;
      if (b < a.B) {
        i = x - f.end[k];
        at = f.at[k];
      }
    } else if (a.pad > 0) {
      b = (int)(t / a.pad);
      i = t - b * a.pad;
      if (i < a.new_len[b]) at = w.req[b];
    } else {
      b = first_above([&](int j) { return a.cu_tokens[j + 1]; }, b0, b1, t);
      if (b < a.B) {
        i = t - a.cu_tokens[b];
        at = w.req[b];
      }
    }
    const int start = at.x, need_ex = at.y;
    int64_t p = -1, slot = -1;
    if (start >= 0) {
      p = start + i;
      const int col = (int)(p >> shift), held = (start + a.page_size - 1) >> shift;
      int32_t* row = a.block_table + (int64_t)b * a.max_pages;
      int page;
      if (col < held) {
        page = row[col];  // the last page the request held already
      } else {
        const int64_t s = tot.avail - 1 - (need_ex + (col - held));
        page = s < tot.n_old ? a.free_pages[s] : returned_page(a, fin, tot.finished, (int)(s - tot.n_old));
        if ((p & (a.page_size - 1)) == 0) row[col] = page;  // the page's first token names it in the table
      }
      if (page >= 0 && page < a.num_pages) {
        slot = ((int64_t)page << shift) + (p & (a.page_size - 1));
      } else {
        record_error(err, DEV_BOUNDS);
        p = -1;
      }
    }
    a.pos[t] = p;
    a.slots[t] = slot;
  }
}

// Returned pages that no request took stay on the stack: entries n_old..left-1.
__device__ void push_returned(const PageTablesArgs& a, const PlanTotals& tot, const int4* fin, int64_t first, int64_t step,
                              int* err) {
  for (int64_t j = tot.n_old + first; j < tot.left; j += step) {
    if (j >= a.num_pages) {  // more pages returned than the pool has
      record_error(err, DEV_BOUNDS);
      break;
    }
    int page = returned_page(a, fin, tot.finished, (int)(j - tot.n_old));
    if (page < 0 || page >= a.num_pages) {  // of a finished row: no page of the pool
      record_error(err, DEV_BOUNDS);
      page = -1;
    }
    a.free_pages[j] = page;
  }
}

// One block. It takes the requests in chunks of PLAN_EACH per thread (one chunk, where
// there are no more). With `fill` it also does the (few) token rows.
__global__ void __launch_bounds__(PLAN_THREADS) page_plan_kernel(PageTablesArgs a, void* ws, int shift, int fill,
                                                                 int* err) {
  __shared__ uint2 sums[4][32];
  __shared__ FillRequests requests;
  wait_for_last();
  let_next_start();
  const PlanViews w = plan_views(ws, a.B);
  const int tid = threadIdx.x, chunk = PLAN_EACH * blockDim.x;
  const int cap = a.max_pages << shift;  // at most 2^30, like n_tokens
  const uint32_t most = (uint32_t)a.n_tokens + 1;
  auto pages_of = [&](int len) { return (len + a.page_size - 1) >> shift; };
  // a request with a length outside its row is not served (cap + 1), and gives nothing back
  auto clip = [&](int64_t c) { return c < 0 || c > cap ? cap + 1 : (int)c; };
  auto held_of = [&](int c) { return c > cap ? 0 : pages_of(c); };
  int n_old = *a.n_free, released = 0;
  if (a.B > chunk) {  // pages come back before any is handed out
    uint2 total;
    uint32_t rel = 0;
    for (int b = tid; b < a.B; b += blockDim.x) {
      if (a.new_len[b] >= 0) continue;
      const int held = held_of(clip(a.ctx_len[b]));
      rel += held > 0 && first_column(a, b) < 0 ? held - first_page(a, b, held) : held;
    }
    block_exclusive(make_uint2(0, rel), most, sums[3], &total);
    released = total.y;
  }
  uint32_t rows_before = 0, fin_before = 0, back_before = 0, need_before = 0, taken = 0;  // of earlier chunks
  for (int base = 0; base < a.B; base += chunk) {
    const int b0 = base + tid * PLAN_EACH;
    int c[PLAN_EACH], held[PLAN_EACH], lead[PLAN_EACH];  // lead: columns that a finished request's pages begin behind
    uint32_t rows[PLAN_EACH];  // one row more than there are is as bad as any number of them
    bool done[PLAN_EACH];
    int64_t ctx[PLAN_EACH];
    uint2 v = make_uint2(0, 0), total;
#pragma unroll
    for (int e = 0; e < PLAN_EACH; ++e) {
      const bool in = b0 + e < a.B;
      const int64_t n = in ? a.new_len[b0 + e] : 0;
      ctx[e] = in ? a.ctx_len[b0 + e] : 0;
      c[e] = clip(ctx[e]);
      held[e] = held_of(c[e]);
      done[e] = n < 0;
      rows[e] = n < 0 ? 0 : (n > a.n_tokens ? most : (uint32_t)n);
      v.x = min(v.x + rows[e], most);
      v.y += done[e];
      if (c[e] > cap) record_error(err, DEV_BOUNDS);
    }
#pragma unroll
    for (int e = 0; e < PLAN_EACH; ++e) lead[e] = done[e] && held[e] > 0 ? first_column(a, b0 + e) : 0;
    if (base > 0) __syncthreads();  // the sums of the last chunk have been read
    uint2 at = block_exclusive(v, most, sums[0], &total);
    at.x = min(at.x + rows_before, most);
    rows_before = min(rows_before + total.x, most);
    uint32_t fin_ex = at.y + fin_before;
    fin_before += total.y;
    uint32_t end[PLAN_EACH], need[PLAN_EACH], mine = 0, back = 0;
    bool fits[PLAN_EACH];
#pragma unroll
    for (int e = 0; e < PLAN_EACH; ++e) {
      at.x = min(at.x + rows[e], most);
      end[e] = at.x;
      fits[e] = b0 + e < a.B && !done[e] && c[e] <= cap && rows[e] <= (uint32_t)(cap - c[e]) &&
                (a.pad ? rows[e] <= a.pad : end[e] < most);
      need[e] = fits[e] ? pages_of(c[e] + (int)rows[e]) - held[e] : 0;
      mine += need[e];
      lead[e] = lead[e] < 0 ? first_page(a, b0 + e, held[e]) : 0;  // its load has had the barrier's time
      back += done[e] ? held[e] - lead[e] : 0;
    }
    const uint2 pre = block_exclusive(make_uint2(back, mine), ~0u, sums[1], &total);
    uint32_t back_ex = back_before + pre.x, need_ex = need_before + pre.y;
    back_before += total.x;
    need_before += total.y;
    if (a.B <= chunk) released = back_before;
    if (base == 0) {
      if (n_old < 0 || n_old > a.num_pages) {
        if (tid == 0) record_error(err, DEV_BOUNDS);
        n_old = n_old < 0 ? 0 : a.num_pages;
      }
      if (tid == 0) a.cu_tokens[0] = 0;
    }
#pragma unroll
    for (int e = 0; e < PLAN_EACH; ++e) {
      const int b = b0 + e;
      if (b >= a.B) break;
      const bool served = fits[e] && (need[e] == 0 || (int64_t)need_ex + need[e] <= (int64_t)n_old + released);
      if (done[e]) {
        back_ex += held[e] - lead[e];
        w.fin[fin_ex++] = make_int4((int)back_ex, b, lead[e], 0);
      }
      a.cu_tokens[b + 1] = end[e] < most ? end[e] : a.n_tokens;
      a.seq_len[b] = done[e] ? 0 : (served ? ctx[e] + rows[e] : ctx[e]);
      w.req[b] = make_int2(served ? c[e] : -1, (int)need_ex);
      need_ex += need[e];
      taken += served ? need[e] : 0;
    }
  }
  uint2 total;
  block_exclusive(make_uint2(0, taken), most, sums[2], &total);
  const int64_t avail = (int64_t)n_old + released;
  const PlanTotals tot{n_old, avail, avail - (int)total.y, (int)fin_before};
  if (tid == 0) {
    *w.totals = tot;
    *a.n_free_out = (int)(tot.left < a.num_pages ? tot.left : a.num_pages);
  }
  if (!fill) return;
  __syncthreads();  // the plan is visible to the block
  const int4* fin = stage_finished(w, tot.finished, requests);
  __syncthreads();
  for (int64_t t0 = 0; t0 < a.n_tokens; t0 += FILL_ROWS) {
    if (t0 > 0) __syncthreads();  // the requests of the last rows have been read
    fill_rows(a, w, tot, fin, shift, t0, requests, err);
  }
  push_returned(a, tot, fin, tid, blockDim.x, err);
}

__global__ void __launch_bounds__(FILL_ROWS) page_fill_kernel(PageTablesArgs a, void* ws, int shift, int* err) {
  __shared__ FillRequests requests;
  const PlanViews w = plan_views(ws, a.B);
  wait_for_last();  // the plan is written
  const PlanTotals tot = *w.totals;
  const int4* fin = stage_finished(w, tot.finished, requests);
  fill_rows(a, w, tot, fin, shift, (int64_t)blockIdx.x * FILL_ROWS, requests, err);  // has a barrier before it reads fin
  push_returned(a, tot, fin, (int64_t)blockIdx.x * FILL_ROWS + threadIdx.x, (int64_t)gridDim.x * FILL_ROWS, err);
}

// ---------------------------------------------------------------------------
// Entries into pages. A thread owns 8 RoPE pairs of one (token, head) row:
// channels [8u, 8u+8) and [hd/2 + 8u, hd/2 + 8u + 8), loaded and stored 16 bytes
// at a time; hd/16 threads cover a row and reduce its RMS with shuffles. A thread
// keeps its head (and gates) and goes through the block's tokens, `pass` of them
// at a time; their angles (double products, shared by the heads) are formed once
// into shared memory while the first loads are on their way. Bound by HBM, of 10 x 128:
// 65536 rotated rows in bf16 take 107 us (0.94 of the copy rate), 32768 in fp32 106
// (0.95); mixed ones in bf16 83 us for 32768 (0.91) and 26 for 8192 (0.73: about three
// waves of blocks), in fp32 158 (0.95) and 45 (0.85); 64 rows 2.8 us.
// ---------------------------------------------------------------------------
enum { WRITE_COPY = 0, WRITE_ROPE = 1, WRITE_MIX = 2 };
constexpr int WRITE_THREADS = 256;
constexpr int WRITE_TURNS = 2048;  // angles of a block: 32 tokens of hd 128, 64 of hd 64

// 8 elements as they are stored, so that all loads are in flight before any arithmetic.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void store_raw8(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}

template <typename T, int HD, int MODE>
__global__ void __launch_bounds__(WRITE_THREADS, sizeof(T) == 2 ? 3 : 2) paged_write_kernel(
    PagedShape s, const __grid_constant__ RopeFreqs rf, int shift, int64_t n, int tile, int heads, int pass,
    const int64_t* slots, const int64_t* pos, const T* k, const T* v, const T* Rk, const T* Rv, const float* gates, T* kp,
    T* vp, int* err) {
  constexpr int HALF = HD / 2, TPR = HD / 16;
  __shared__ float2 turn[MODE == WRITE_COPY ? 1 : WRITE_TURNS];
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const int ntok = (int)(n - t0 < tile ? n - t0 : tile);
  const int64_t nslots = (int64_t)s.num_pages << shift;
  wait_for_last();
  const int u = threadIdx.x % TPR, row = threadIdx.x / TPR, h = blockIdx.y * heads + row % heads;
  const bool mine = row < heads * pass && h < s.Hkv;
  float gkl = 1.f, gkr = 0.f, gvl = 1.f, gvr = 0.f;
  Raw8<T> k1{}, k2{}, v1{}, v2{}, r1{}, r2{}, w1{}, w2{};
  int64_t slot = -1;
  auto load = [&](int tt) {  // every load of token tt's piece; slot < 0: nothing to write
    slot = -1;
    if (!mine || tt >= ntok) return;
    slot = slots[t0 + tt];
    if (MODE != WRITE_COPY && pos[t0 + tt] < 0) slot = -1;
    if (slot >= nslots) {
      if (u == 0) record_error(err, DEV_BOUNDS);
      slot = -1;
    }
    const int64_t src = ((t0 + tt) * s.Hkv + h) * HD + 8 * u;
    k1 = raw8(k + src);
    k2 = raw8(k + src + HALF);
    v1 = raw8(v + src);
    v2 = raw8(v + src + HALF);
    if (MODE == WRITE_MIX) {
      r1 = raw8(Rk + src);
      r2 = raw8(Rk + src + HALF);
      w1 = raw8(Rv + src);
      w2 = raw8(Rv + src + HALF);
    }
  };
  load(row / heads);
  if (MODE == WRITE_MIX && mine) {
    gkl = gate_value(gates[h]);
    gkr = gate_value(gates[s.Hkv + h]);
    gvl = gate_value(gates[s.vg * s.Hkv + h]);
    gvr = gate_value(gates[(s.vg + 1) * s.Hkv + h]);
  }
  if (MODE != WRITE_COPY) {
    // pairs 8u + e of a token at [e / 2][u][e % 2]: the lanes of a row read side by side
    for (int i = threadIdx.x; i < ntok * HALF; i += WRITE_THREADS) {
      const int c = i % HALF, e = c % 8;
      turn[i - c + (e / 2 * TPR + c / 8) * 2 + e % 2] = rope_turn(pos[t0 + i / HALF], rf.turns[c]);
    }
    __syncthreads();
  }
  for (int tt = row / heads; tt - row / heads < ntok; tt += pass) {  // whole blocks: the RMS sums shuffle
    float x1[8], x2[8], y1[8], y2[8];
    float rinv = 0.f;
    if (MODE == WRITE_MIX) {
      load8f(reinterpret_cast<const T*>(&r1), y1);
      load8f(reinterpret_cast<const T*>(&r2), y2);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += y1[e] * y1[e] + y2[e] * y2[e];
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      rinv = gkr * rsqrtf(ss / HD + s.eps);
    }
    if (slot >= 0) {
      const int64_t dst = ((((slot >> shift) * s.Hkv + h) << shift) + (slot & (s.page_size - 1))) * HD + 8 * u;
      if (MODE == WRITE_COPY) {
        store_raw8(kp + dst, k1);
        store_raw8(kp + dst + HALF, k2);
      } else {
        load8f(reinterpret_cast<const T*>(&k1), x1);
        load8f(reinterpret_cast<const T*>(&k2), x2);
        const float4* tw = reinterpret_cast<const float4*>(turn + tt * HALF) + u;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 w = tw[e / 2 * TPR];  // two pairs' angles
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float cs = i ? w.z : w.x, sn = i ? w.w : w.y;
            // both keys turn by the same angle, so the mix comes first
            float p = x1[e + i], q = x2[e + i];
            if (MODE == WRITE_MIX) {
              p = gkl * p + rinv * y1[e + i];
              q = gkl * q + rinv * y2[e + i];
            }
            x1[e + i] = p * cs - q * sn;
            x2[e + i] = p * sn + q * cs;
          }
        }
        store8f(kp + dst, x1);
        store8f(kp + dst + HALF, x2);
      }
      if (MODE != WRITE_MIX) {
        store_raw8(vp + dst, v1);
        store_raw8(vp + dst + HALF, v2);
      } else {
        load8f(reinterpret_cast<const T*>(&v1), x1);
        load8f(reinterpret_cast<const T*>(&v2), x2);
        load8f(reinterpret_cast<const T*>(&w1), y1);
        load8f(reinterpret_cast<const T*>(&w2), y2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x1[e] = gvl * x1[e] + gvr * y1[e];
          x2[e] = gvl * x2[e] + gvr * y2[e];
        }
        store8f(vp + dst, x1);
        store8f(vp + dst + HALF, x2);
      }
    }
    load(tt + pass);
  }
}

template <typename T, int HD>
cudaError_t write_pages(const PagedShape& s, int64_t n, const int64_t* slots, const int64_t* pos, const void* k,
                        const void* v, const void* Rk, const void* Rv, const float* gates, void* kp, void* vp, int* err,
                        cudaStream_t st) {
  constexpr int ROWS = WRITE_THREADS / (HD / 16), MOST = WRITE_TURNS / (HD / 2);
  const int heads = s.Hkv < ROWS ? s.Hkv : ROWS, pass = ROWS / heads;  // of a block; tokens at a time
  // two passes a block: one leaves the angles uncovered, four leave a ragged last wave
  // (10 x 128 with 1, 2, 4 passes: 8192 mixed rows in bf16 26.9, 25.9, 27.0 us, 16384 48.4,
  // 45.0, 47.1, in fp32 85.6, 83.5, 82.2; 65536 rotated in bf16 114.4, 107.8, 106.9, 4096
  // 9.5, 10.2, 10.2)
  int tile = pass * 2 < MOST ? pass * 2 : MOST;
  while (tile > 1 && n < (int64_t)tile * 4 * num_sms()) tile /= 2;  // few tokens: spread them over the SMs
  const dim3 blocks((unsigned)((n + tile - 1) / tile), (unsigned)((s.Hkv + heads - 1) / heads));
  const RopeFreqs& rf = rope_freqs(HD, s.log2_base);
  const int shift = log2_of(s.page_size);
  auto go = [&](auto kern) {
    return launch_dependent(kern, blocks, WRITE_THREADS, 0, st, s, rf, shift, n, tile, heads, pass, slots, pos,
                            (const T*)k, (const T*)v, (const T*)Rk, (const T*)Rv, gates, (T*)kp, (T*)vp, err);
  };
  if (!pos) return go(paged_write_kernel<T, HD, WRITE_COPY>);
  if (!s.inject) return go(paged_write_kernel<T, HD, WRITE_ROPE>);
  return go(paged_write_kernel<T, HD, WRITE_MIX>);
}

// Token rows that the plan's block fills itself: 512 single tokens take it 4.8 us, 1024
// packed rows 6.2 to 7.3 us against 4.5 to 5 with the second launch.
constexpr int64_t ONE_LAUNCH_ROWS = 512;

}  // namespace

size_t page_tables_workspace_bytes(int B) { return 256 + (size_t)B * (sizeof(int4) + sizeof(int2)); }

int page_tables_kernels(int64_t n_tokens) { return n_tokens <= ONE_LAUNCH_ROWS ? 1 : 2; }

cudaError_t launch_page_tables(const PageTablesArgs& a, void* workspace, int* err, cudaStream_t st) {
  const int shift = log2_of(a.page_size);
  const int one = a.n_tokens <= ONE_LAUNCH_ROWS;
  int threads = (a.B + PLAN_EACH - 1) / PLAN_EACH;  // few requests: fewer warps to sum over
  if (one && a.n_tokens > threads) threads = (int)a.n_tokens;
  threads = threads < 64 ? 64 : threads > PLAN_THREADS ? PLAN_THREADS : (threads + 31) / 32 * 32;
  cudaError_t e = launch_dependent(page_plan_kernel, dim3(1), threads, 0, st, a, workspace, shift, one, err);
  if (e != cudaSuccess || one) return e;
  return launch_dependent(page_fill_kernel, dim3((unsigned)((a.n_tokens + FILL_ROWS - 1) / FILL_ROWS)), FILL_ROWS, 0, st,
                          a, workspace, shift, err);
}

cudaError_t launch_paged_write(const PagedShape& s, int64_t n, const int64_t* slots, const int64_t* pos, const void* k,
                               const void* v, const void* Rk, const void* Rv, const float* gates, void* k_pages,
                               void* v_pages, int* err, cudaStream_t st) {
  if (s.dtype == 1 && s.hd == 128)
    return write_pages<bf16, 128>(s, n, slots, pos, k, v, Rk, Rv, gates, k_pages, v_pages, err, st);
  if (s.dtype == 1 && s.hd == 64)
    return write_pages<bf16, 64>(s, n, slots, pos, k, v, Rk, Rv, gates, k_pages, v_pages, err, st);
  if (s.dtype == 0 && s.hd == 128)
    return write_pages<float, 128>(s, n, slots, pos, k, v, Rk, Rv, gates, k_pages, v_pages, err, st);
  if (s.dtype == 0 && s.hd == 64)
    return write_pages<float, 64>(s, n, slots, pos, k, v, Rk, Rv, gates, k_pages, v_pages, err, st);
  return cudaErrorInvalidValue;
}

}  // namespace maglev
