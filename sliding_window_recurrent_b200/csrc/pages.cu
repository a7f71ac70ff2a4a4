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
// Page tables. A finished request (new < 0) gives its held(b) =
// ceil(ctx / page_size) pages back; the others need need(b) =
// ceil((ctx + new) / page_size) - held(b). With the stack of free pages
// S = free[0..n) followed by the returned pages, request b is served when the
// inclusive prefix sum of need up to b is at most |S| (or need(b) == 0), and
// page i of all pages handed out is S[|S| - 1 - i]. So one prefix sum over the
// requests places every page, and then every token row is independent.
//
// The plan (one block: prefix sums over the requests) and the fill (a thread
// per token row) are one launch when one block can do both, else two.
// ---------------------------------------------------------------------------
struct PlanTotals {
  int64_t n_old, avail, left;  // free pages before, with the returned ones, after
};
struct PlanViews {
  PlanTotals* totals;
  int64_t* start;  // [B] first position of a served request's tokens, else -1
  int* need_ex;    // [B] pages handed out to earlier requests
  int* rel_ex;     // [B+1] pages returned by earlier requests
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
__host__ __device__ inline PlanViews plan_views(void* ws, int B) {
  char* p = static_cast<char*>(ws);
  PlanViews v;
  v.totals = reinterpret_cast<PlanTotals*>(p);
  v.start = reinterpret_cast<int64_t*>(p + 256);
  v.need_ex = reinterpret_cast<int*>(p + 256 + up256((size_t)B * 8));
  v.rel_ex = v.need_ex + B;
  return v;
}

constexpr int PLAN_THREADS = 1024;
constexpr int FILL_THREADS = 256;
constexpr int FILL_ROWS = 1024;  // token rows of one block of the fill

// Exclusive prefix sum over the block; *total receives the block's sum.
template <typename T>
__device__ __forceinline__ T block_exclusive(T x, T* sums /* [33] shared */, T* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  T inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // the sums of an earlier call have been read
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const T w = lane < PLAN_THREADS / 32 ? sums[lane] : T(0);
    T winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += y;
    }
    sums[lane] = winc - w;
    if (lane == 31) sums[32] = winc;
  }
  __syncthreads();
  *total = sums[32];
  return sums[warp] + inc - x;
}

// The first b in [lo, hi) with x[b] > t (hi if none): x is non-decreasing.
template <typename T>
__device__ __forceinline__ int first_above(const T* x, int lo, int hi, int64_t t) {
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if ((int64_t)x[mid] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Page k of the pages that finished requests return (request, then column order).
__device__ __forceinline__ int returned_page(const PageTablesArgs& a, const PlanViews& w, int64_t k) {
  const int r = first_above(w.rel_ex + 1, 0, a.B, k);
  if (r >= a.B) return -1;
  return a.block_table[(int64_t)r * a.max_pages + (k - w.rel_ex[r])];
}

// Token rows [t0, t0 + rows) of the map, and with them the table columns whose
// page a row is the first of.
__device__ void fill_rows(const PageTablesArgs& a, const PlanViews& w, int shift, int64_t t0, int rows, int* range,
                          int* err) {
  const int64_t t1 = t0 + rows < a.n_tokens ? t0 + rows : a.n_tokens;
  const PlanTotals tot = *w.totals;
  if (a.pad == 0) {  // the requests these rows belong to
    if (threadIdx.x == 0) range[0] = first_above(a.cu_tokens + 1, 0, a.B, t0);
    if (threadIdx.x == 32) range[1] = first_above(a.cu_tokens + 1, 0, a.B, t1 - 1);
    __syncthreads();
  }
  for (int64_t t = t0 + threadIdx.x; t < t1; t += blockDim.x) {
    int b;
    int64_t i;
    bool live;
    if (a.pad == 0) {
      b = first_above(a.cu_tokens + 1, range[0], range[1], t);
      live = b < a.B && t < a.cu_tokens[a.B];
      i = live ? t - a.cu_tokens[b] : 0;
    } else {
      b = (int)(t / a.pad);
      i = t - (int64_t)b * a.pad;
      live = i < a.new_len[b];
    }
    const int64_t start = live ? w.start[b] : -1;
    int64_t p = -1, slot = -1;
    if (start >= 0) {
      p = start + i;
      const int64_t col = p >> shift, held = (start + a.page_size - 1) >> shift;
      int32_t* row = a.block_table + (int64_t)b * a.max_pages;
      int page;
      if (col < held) {
        page = row[col];  // the last page the request held already
      } else {
        const int64_t s = tot.avail - 1 - (w.need_ex[b] + (col - held));
        page = s < tot.n_old ? a.free_pages[s] : returned_page(a, w, s - tot.n_old);
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
__device__ void push_returned(const PageTablesArgs& a, const PlanViews& w, int64_t first, int64_t step, int* err) {
  const PlanTotals tot = *w.totals;
  for (int64_t j = tot.n_old + first; j < tot.left; j += step) {
    if (j >= a.num_pages) {  // more pages returned than the pool has
      record_error(err, DEV_BOUNDS);
      break;
    }
    a.free_pages[j] = returned_page(a, w, j - tot.n_old);
  }
}

// One block. The prefix sums run over chunks of 1024 requests, so B is not
// bounded by the block; with `fill` it also does the (few) token rows.
__global__ void __launch_bounds__(PLAN_THREADS) page_plan_kernel(PageTablesArgs a, void* ws, int shift, int fill,
                                                                 int* err) {
  __shared__ int64_t sums64[33];
  __shared__ int sums32[33];
  __shared__ int range[2];
  const PlanViews w = plan_views(ws, a.B);
  const int tid = threadIdx.x;
  const int64_t cap = (int64_t)a.max_pages << shift;
  auto held_of = [&](int64_t c) -> int {  // pages of c cached tokens; lengths outside the row are cut
    c = c < 0 ? 0 : (c > cap ? cap : c);
    return (int)((c + a.page_size - 1) >> shift);
  };
  int mine = 0, released;
  for (int b = tid; b < a.B; b += PLAN_THREADS)
    if (a.new_len[b] < 0) mine += held_of(a.ctx_len[b]);
  block_exclusive(mine, sums32, &released);
  int64_t n_old = *a.n_free;
  if (n_old < 0 || n_old > a.num_pages) {
    if (tid == 0) record_error(err, DEV_BOUNDS);
    n_old = n_old < 0 ? 0 : a.num_pages;
  }
  const int64_t avail = n_old + released;
  int64_t rows_before = 0, need_before = 0;
  int rel_before = 0, taken = 0;
  for (int base = 0; base < a.B; base += PLAN_THREADS) {
    const int b = base + tid;
    const bool in = b < a.B;
    const int64_t c = in ? a.ctx_len[b] : 0, n = in ? a.new_len[b] : 0;
    const bool done = n < 0;
    // one row more than there are is as bad as any number of them, and keeps the sum small
    const int64_t rows = n < 0 ? 0 : (n > a.n_tokens ? a.n_tokens + 1 : n);
    const int held = held_of(c);
    int64_t chunk_rows, chunk_need;
    int chunk_rel;
    const int64_t row_end = rows_before + block_exclusive(rows, sums64, &chunk_rows) + rows;
    const int rel_ex = rel_before + block_exclusive(done ? held : 0, sums32, &chunk_rel);
    const bool fits = in && !done && c >= 0 && c <= cap - rows && (a.pad ? rows <= a.pad : row_end <= a.n_tokens);
    const int need = fits ? held_of(c + rows) - held : 0;
    const int64_t need_ex = need_before + block_exclusive((int64_t)need, sums64, &chunk_need);
    const bool served = fits && (need == 0 || need_ex + need <= avail);
    if (in) {
      if (b == 0) a.cu_tokens[0] = 0;
      a.cu_tokens[b + 1] = row_end < a.n_tokens ? row_end : a.n_tokens;
      a.seq_len[b] = done ? 0 : (served ? c + rows : c);
      w.start[b] = served ? c : -1;
      w.need_ex[b] = served ? (int)need_ex : 0;
      if (b == 0) w.rel_ex[0] = 0;
      w.rel_ex[b + 1] = rel_ex + (done ? held : 0);
    }
    if (served) taken += need;
    rows_before += chunk_rows;
    need_before += chunk_need;
    rel_before += chunk_rel;
  }
  int all_taken;
  block_exclusive(taken, sums32, &all_taken);
  if (tid == 0) {
    const int64_t left = avail - all_taken;
    *w.totals = PlanTotals{n_old, avail, left};
    *a.n_free_out = (int)(left < a.num_pages ? left : a.num_pages);
  }
  if (!fill) return;
  __syncthreads();  // the plan is visible to the block
  if (a.n_tokens > 0) fill_rows(a, w, shift, 0, (int)a.n_tokens, range, err);
  push_returned(a, w, tid, PLAN_THREADS, err);
}

__global__ void __launch_bounds__(FILL_THREADS) page_fill_kernel(PageTablesArgs a, void* ws, int shift, int* err) {
  __shared__ int range[2];
  const PlanViews w = plan_views(ws, a.B);
  fill_rows(a, w, shift, (int64_t)blockIdx.x * FILL_ROWS, FILL_ROWS, range, err);
  push_returned(a, w, (int64_t)blockIdx.x * FILL_THREADS + threadIdx.x, (int64_t)gridDim.x * FILL_THREADS, err);
}

// ---------------------------------------------------------------------------
// Entries into pages. A thread owns 8 RoPE pairs of one (token, head) row:
// channels [8u, 8u+8) and [hd/2 + 8u, hd/2 + 8u + 8), loaded and stored 16
// bytes at a time; hd/16 threads cover a row and reduce its RMS with shuffles.
// A block takes `tile` tokens; their angles (double products, shared by the
// heads) are formed once into shared memory.
// ---------------------------------------------------------------------------
enum { WRITE_COPY = 0, WRITE_ROPE = 1, WRITE_MIX = 2 };
constexpr int WRITE_THREADS = 256;
constexpr int WRITE_TILE = 16;  // the most tokens of a block

template <typename T, int HD, int MODE>
__global__ void __launch_bounds__(WRITE_THREADS) paged_write_kernel(
    PagedShape s, RopeFreqs rf, int shift, int64_t n, int tile, const int64_t* __restrict__ slots,
    const int64_t* __restrict__ pos, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ Rk,
    const T* __restrict__ Rv, const float* __restrict__ gates, T* __restrict__ kp, T* __restrict__ vp, int* err) {
  constexpr int HALF = HD / 2, TPR = HD / 16;
  __shared__ float2 turn[MODE == WRITE_COPY ? 1 : WRITE_TILE * HALF];
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const int ntok = (int)(n - t0 < tile ? n - t0 : tile);
  if (MODE != WRITE_COPY) {
    for (int i = threadIdx.x; i < ntok * HALF; i += WRITE_THREADS)
      turn[i] = rope_turn(pos[t0 + i / HALF], rf.turns[i % HALF]);
    __syncthreads();
  }
  const int64_t nslots = (int64_t)s.num_pages << shift;
  const int items = ntok * s.Hkv * TPR;
  for (int i0 = 0; i0 < items; i0 += WRITE_THREADS) {  // whole warps: the RMS sums shuffle
    const int i = i0 + threadIdx.x;
    const int u = i % TPR, row = i / TPR;
    bool live = i < items;
    const int tt = live ? row / s.Hkv : 0, h = live ? row % s.Hkv : 0;
    const int64_t slot = slots[t0 + tt];
    if (live && slot >= nslots) {
      if (u == 0) record_error(err, DEV_BOUNDS);
      live = false;
    }
    live = live && slot >= 0 && (MODE == WRITE_COPY || pos[t0 + tt] >= 0);
    const int64_t src = ((t0 + tt) * s.Hkv + h) * HD + 8 * u;
    float k1[8], k2[8], v1[8], v2[8], r1[8], r2[8];
    float ss = 0.f;
    if (live) {
      load8f(k + src, k1);
      load8f(k + src + HALF, k2);
      load8f(v + src, v1);
      load8f(v + src + HALF, v2);
      if (MODE == WRITE_MIX) {
        load8f(Rk + src, r1);
        load8f(Rk + src + HALF, r2);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += r1[e] * r1[e] + r2[e] * r2[e];
      }
    }
    if (MODE == WRITE_MIX) {
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (!live) continue;
    if (MODE != WRITE_COPY) {
      const float rinv = MODE == WRITE_MIX ? rsqrtf(ss / HD + s.eps) : 0.f;
      float gkl = 1.f, gkr = 0.f;
      if (MODE == WRITE_MIX) {
        gkl = gate_value(gates[h]);
        gkr = gate_value(gates[s.Hkv + h]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = turn[tt * HALF + 8 * u + e];
        float a = k1[e] * w.x - k2[e] * w.y, b = k1[e] * w.y + k2[e] * w.x;
        if (MODE == WRITE_MIX) {
          const float x = r1[e] * rinv, y = r2[e] * rinv;
          a = gkl * a + gkr * (x * w.x - y * w.y);
          b = gkl * b + gkr * (x * w.y + y * w.x);
        }
        k1[e] = a;
        k2[e] = b;
      }
    }
    if (MODE == WRITE_MIX) {
      const float gvl = gate_value(gates[s.vg * s.Hkv + h]), gvr = gate_value(gates[(s.vg + 1) * s.Hkv + h]);
      load8f(Rv + src, r1);
      load8f(Rv + src + HALF, r2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v1[e] = gvl * v1[e] + gvr * r1[e];
        v2[e] = gvl * v2[e] + gvr * r2[e];
      }
    }
    const int64_t dst = ((((slot >> shift) * s.Hkv + h) << shift) + (slot & (s.page_size - 1))) * HD + 8 * u;
    store8f(kp + dst, k1);
    store8f(kp + dst + HALF, k2);
    store8f(vp + dst, v1);
    store8f(vp + dst + HALF, v2);
  }
}

template <typename T, int HD>
cudaError_t write_pages(const PagedShape& s, int64_t n, const int64_t* slots, const int64_t* pos, const void* k,
                        const void* v, const void* Rk, const void* Rv, const float* gates, void* kp, void* vp, int* err,
                        cudaStream_t st) {
  int tile = WRITE_TILE;
  while (tile > 1 && n < (int64_t)tile * 2 * num_sms()) tile /= 2;  // few tokens: spread them over the SMs
  const unsigned blocks = (unsigned)((n + tile - 1) / tile);
  const RopeFreqs rf = rope_freqs(HD, s.log2_base);
  const int shift = log2_of(s.page_size);
  auto go = [&](auto kern) {
    kern<<<blocks, WRITE_THREADS, 0, st>>>(s, rf, shift, n, tile, slots, pos, (const T*)k, (const T*)v, (const T*)Rk,
                                           (const T*)Rv, gates, (T*)kp, (T*)vp, err);
  };
  if (!pos) go(paged_write_kernel<T, HD, WRITE_COPY>);
  else if (!s.inject) go(paged_write_kernel<T, HD, WRITE_ROPE>);
  else go(paged_write_kernel<T, HD, WRITE_MIX>);
  return cudaGetLastError();
}

// Token rows that one block of the plan fills itself instead of a second launch.
constexpr int64_t ONE_LAUNCH_ROWS = 4096;

}  // namespace

size_t page_tables_workspace_bytes(int B) { return 256 + up256((size_t)B * 8) + up256(((size_t)2 * B + 1) * 4); }

int page_tables_kernels(int64_t n_tokens) { return n_tokens <= ONE_LAUNCH_ROWS ? 1 : 2; }

cudaError_t launch_page_tables(const PageTablesArgs& a, void* workspace, int* err, cudaStream_t st) {
  const int shift = log2_of(a.page_size);
  const int one = a.n_tokens <= ONE_LAUNCH_ROWS;
  page_plan_kernel<<<1, PLAN_THREADS, 0, st>>>(a, workspace, shift, one, err);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || one) return e;
  page_fill_kernel<<<(unsigned)((a.n_tokens + FILL_ROWS - 1) / FILL_ROWS), FILL_THREADS, 0, st>>>(a, workspace, shift,
                                                                                                  err);
  return cudaGetLastError();
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
