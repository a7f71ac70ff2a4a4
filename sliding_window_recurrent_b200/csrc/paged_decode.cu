// One decode step over a paged key/value cache: the paged form of the ring
// step in decode.cu, for sequences of any length and grouped key/value heads.
//
// Source: "Maglev: Sliding Recurrent Memory", paper.rainbus.top, 研究动机 (the
// decoder reads a window of entries and the memory) and 前置知识 (KV cache:
// the memory rides in the existing entries); the prefiller's full layers read
// every entry (window 0).
//
// Mathematics. For a query row q (rotated, scaled to log2 units) and any split of
// its keys into parts, each part keeps (m, l, o): a reference m >= is not needed
// to be the exact maximum, l = sum 2^(s_j - m), o = sum 2^(s_j - m) v_j. Parts join
// by M = max m_i, l = sum 2^(m_i - M) l_i, o likewise, out = o / l.
//
// Split. The cache is read once and nothing else is large, so the kernel is bound
// by HBM and has to keep every SM streaming whatever the lengths are. A unit is a
// (sequence, key/value head, group of query heads) and is cut into steps of 16
// keys (one page holds a whole number of steps). All steps of all units, in
// order, are dealt to the blocks of a persistent grid in equal contiguous
// ranges: a block's range covers whole units and at most two partial ones, each
// warp takes every NW-th step of it. A partial unit's (m, l, o) goes to the
// workspace, and the block that completes the unit's count joins the parts in
// block order, so results do not depend on which block came last.
//
// Streaming. A warp owns a ring of stages in shared memory (K and V of one step)
// filled by its own 16-byte asynchronous copies; no block-wide barrier
// stands between a copy and its use, and copies run ahead across units.
#include "paged.cuh"

namespace maglev {
namespace {

constexpr int KSTEP = 16;  // keys of a step

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes to shared memory; bytes = 0 fills with zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
// x - bf16(x): exact in fp32, so bf16(x) + bf16(x - bf16(x)) carries 16 bits of x.
__device__ __forceinline__ float rest(float x) { return x - __bfloat162float(__float2bfloat16_rn(x)); }

// A running reference may lie this far (log2 units) below the maximum before it
// moves: weights stay below 2^8, and the rescaling of o becomes rare.
constexpr float SLACK = 8.0f;

// Where a step's entries lie in shared memory: rows of HD elements, the 16-byte
// pieces of row r permuted by r & 7 so that a column of pieces hits every bank.
template <typename T, int HD>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return (uint32_t)(r * HD * (int)sizeof(T) + ((c ^ (r & 7)) << 4));
}

// ---------------------------------------------------------------------------
// bf16: 16 keys x up to 8 NT query heads on the tensor cores. S^T = K q^T and
// O^T = V^T P^T take the keys (the channels) as the instruction's 16 rows and the
// heads as its columns: with one head to a key head the heads are the side to
// pad, and 8 columns is the least it can be padded to. The step is bound by HBM
// (8 KB per 16 keys), which leaves room to carry q and P as two bf16 parts
// each: S and O then are fp32-accurate and the only rounding is the output's.
// ---------------------------------------------------------------------------
template <int HD, int NT>
struct MmaTile {
  static constexpr int HEADS = 8 * NT, KS = HD / 16;
  static constexpr int QROW = HD + 8;                 // padded: fragment loads hit every bank
  static constexpr int Q_BYTES = 2 * HEADS * QROW * 2;  // upper parts, then lower parts
  static constexpr int SCRATCH = 0;
  float o[KS][NT][4];
  float m[NT][2], l[NT][2];
  uint32_t qh[KS][NT][2], ql[KS][NT][2];

  __device__ __forceinline__ static void put_q(char* qs, int j, int c, float x) {
    bf16* q = reinterpret_cast<bf16*>(qs);
    q[j * QROW + c] = __float2bfloat16_rn(x);
    q[(HEADS + j) * QROW + c] = __float2bfloat16_rn(rest(x));
  }
  __device__ __forceinline__ void begin(const char* qs) {
    const int g = (threadIdx.x % 32) / 4, t = threadIdx.x % 4;
    const bf16* q = reinterpret_cast<const bf16*>(qs);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bf16* p = q + (n * 8 + g) * QROW + 16 * k + 2 * t;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qh[k][n][e] = *reinterpret_cast<const uint32_t*>(p + 8 * e);
          ql[k][n][e] = *reinterpret_cast<const uint32_t*>(p + HEADS * QROW + 8 * e);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][n][e] = 0.f;
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
  }
  // live(r): whether key r of the step takes part; all: every key does
  template <typename Live>
  __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, bool all, Live live, char*, const char*, int) {
    const int lane = threadIdx.x % 32, g = lane / 4;
    float s[NT][4], s2[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
    const int kr = lane & 15;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t a[4];
      ldsm4(a, ks + piece<bf16, HD>(kr, 2 * k + (lane >> 4)));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(s[n], a, qh[k][n][0], qh[k][n][1]);
        mma16816(s2[n], a, ql[k][n][0], ql[k][n][1]);
      }
    }
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] += s2[n][e];
        if (!all && !live(g + (e & 2) * 4)) s[n][e] = -INFINITY;
        grow |= s[n][e] > m[n][e & 1] + SLACK;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          const float mn = fmaxf(m[n][e], x);
          const float a = m[n][e] == -INFINITY ? 0.f : pow2(m[n][e] - mn);
          m[n][e] = mn;
          l[n][e] *= a;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            o[k][n][e] *= a;
            o[k][n][e + 2] *= a;
          }
        }
    }
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float r = m[n][e & 1];
        w[e] = pow2(s[n][e] - (r == -INFINITY ? 0.f : r));
        l[n][e & 1] += w[e];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ph[n][e] = transpose8x8(pack2(w[2 * e], w[2 * e + 1]));
        pl[n][e] = transpose8x8(pack2(rest(w[2 * e]), rest(w[2 * e + 1])));
      }
    }
    const int vr = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t a[4];
      ldsm4_trans(a, vs + piece<bf16, HD>(vr, 2 * k + ((lane >> 3) & 1)));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(o[k][n], a, ph[n][0], ph[n][1]);
        mma16816(o[k][n], a, pl[n][0], pl[n][1]);
      }
    }
  }
  // the warp's references and sums, then (scaled to the block's references M) its outputs
  __device__ __forceinline__ void put_ml(float* wm, float* wl) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[n][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (lane < 4) {
          wm[n * 8 + 2 * lane + e] = m[n][e];
          wl[n * 8 + 2 * lane + e] = x;
        }
      }
  }
  template <int ROW>
  __device__ __forceinline__ void put_o(float* wo, const float* f, int heads) {
    const int g = (threadIdx.x % 32) / 4, t = threadIdx.x % 4;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = n * 8 + 2 * t + e;
        if (j >= heads) continue;
        const float a = f[j];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          wo[j * ROW + 16 * k + g] = o[k][n][e] * a;
          wo[j * ROW + 16 * k + g + 8] = o[k][n][e + 2] * a;
        }
      }
  }
};

// ---------------------------------------------------------------------------
// fp32 on the CUDA cores: a lane owns half a key's channels for the scores
// and four channels for the outputs, each 16-byte piece read once for all heads.
// ---------------------------------------------------------------------------
template <int HD>
struct SimtTile {
  static constexpr int HEADS = 4, PIECES = HD / 4;
  static constexpr int Q_BYTES = HEADS * HD * 4;
  static constexpr int SCRATCH = HEADS * KSTEP * 4;  // a warp's weights of a step
  static constexpr int SPLIT = 32 / PIECES > 0 ? 32 / PIECES : 1;  // lanes that share a piece (hd 64: 2)
  float o[HEADS][4];
  float m[HEADS], l[HEADS];

  __device__ __forceinline__ static void put_q(char* qs, int j, int c, float x) {
    reinterpret_cast<float*>(qs)[j * HD + c] = x;
  }
  __device__ __forceinline__ void begin(const char*) {
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    }
  }
  __device__ __forceinline__ static float4 lds4(uint32_t a) {
    float4 r;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(a) : "memory");
    return r;
  }
  template <typename Live>
  __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, bool all, Live live, char* scratch, const char* qs,
                                       int heads) {
    const int lane = threadIdx.x % 32, r = lane & 15, half = lane >> 4;
    const float4* q = reinterpret_cast<const float4*>(qs);
    float s[HEADS];
#pragma unroll
    for (int j = 0; j < HEADS; ++j) s[j] = 0.f;
#pragma unroll
    for (int i = 0; i < PIECES / 2; ++i) {
      const int c = half * (PIECES / 2) + i;
      const float4 x = lds4(ks + piece<float, HD>(r, c));
#pragma unroll
      for (int j = 0; j < HEADS; ++j)
        if (j < heads) {
          const float4 y = q[j * PIECES + c];
          s[j] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[j]))));
        }
    }
    float* w = reinterpret_cast<float*>(scratch);
    const bool on = all || live(r);
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
      if (j >= heads) break;
      s[j] += __shfl_xor_sync(0xffffffffu, s[j], 16);
      if (!on) s[j] = -INFINITY;
      if (__any_sync(0xffffffffu, s[j] > m[j] + SLACK)) {
        float x = s[j];
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        const float mn = fmaxf(m[j], x);
        const float a = m[j] == -INFINITY ? 0.f : exp2f(m[j] - mn);
        m[j] = mn;
        l[j] *= a;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= a;
      }
      const float p = exp2f(s[j] - (m[j] == -INFINITY ? 0.f : m[j]));
      l[j] += p;  // both halves keep the same sum
      if (half == 0) w[j * KSTEP + r] = p;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < KSTEP / SPLIT; ++i) {
      const int k = i * SPLIT + (SPLIT > 1 ? lane / PIECES : 0);
      const float4 x = lds4(vs + piece<float, HD>(k, lane % PIECES));
#pragma unroll
      for (int j = 0; j < HEADS; ++j)
        if (j < heads) {
          const float p = w[j * KSTEP + k];
          o[j][0] = fmaf(p, x.x, o[j][0]);
          o[j][1] = fmaf(p, x.y, o[j][1]);
          o[j][2] = fmaf(p, x.z, o[j][2]);
          o[j][3] = fmaf(p, x.w, o[j][3]);
        }
    }
  }
  __device__ __forceinline__ void put_ml(float* wm, float* wl) {
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
      float x = l[j];
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if (threadIdx.x % 32 == 0) {
        wm[j] = m[j];
        wl[j] = x;
      }
    }
  }
  template <int ROW>
  __device__ __forceinline__ void put_o(float* wo, const float* f, int heads) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
      if (j >= heads) break;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = o[j][e];
        if (SPLIT > 1) x[e] += __shfl_xor_sync(0xffffffffu, x[e], 16);
        x[e] *= f[j];
      }
      if (lane < PIECES) *reinterpret_cast<float4*>(wo + j * ROW + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
};

// ---------------------------------------------------------------------------
struct DecodeArgs {
  const int64_t* pos;
  const void *q, *k, *v, *krec, *vrec;
  const float* gates;
  const int32_t* table;
  void *kp, *vp, *out;
  float* parts;    // [grid][2][HEADS][hd + 2]
  int* counters;   // [B * units], zero between calls
  int shift;       // log2 of the page size
  int heads, units;  // query heads of a unit (the last may have fewer), units of a sequence
  float scale_log2;
  int* err;
};

constexpr int PART_HEADS = 16, PART_ROW = 130;  // the largest part: 16 heads of 128 channels, m and l
constexpr int MIN_STEPS = 8;                    // fewest steps of a block's range

// A sequence's steps and the unit a global step lies in.
struct Cursor {
  int b, hu;         // sequence, unit within it
  int p, lo, s0, n;  // its position, first key, first step, steps (of each unit)
  int64_t base;      // global step of the unit's first one
};

template <typename T, int HD, typename Tile, int NW, int STAGES, int OCC>
__global__ void __launch_bounds__(NW * 32, OCC) paged_decode_kernel(PagedShape s, DecodeArgs a,
                                                                  const __grid_constant__ RopeFreqs rf) {
  constexpr int HALF = HD / 2, THREADS = NW * 32, HEADS = Tile::HEADS;
  constexpr int CPR = HD * (int)sizeof(T) / 16;            // 16-byte pieces of an entry
  constexpr int KV = KSTEP * HD * (int)sizeof(T);          // K (or V) bytes of a step
  constexpr int OROW = HD + 4;                             // merge rows: four columns of one key row hit every bank
  extern __shared__ __align__(128) char sm[];
  char* qs = sm + NW * STAGES * 2 * KV;
  T* kn = reinterpret_cast<T*>(qs + Tile::Q_BYTES);        // the new entry, as stored
  T* vn = kn + HD;
  float2* turn = reinterpret_cast<float2*>(vn + HD);       // angles of the current sequence's position
  char* scratch = reinterpret_cast<char*>(turn + HALF) + (threadIdx.x / 32) * Tile::SCRATCH;
  float* wm = reinterpret_cast<float*>(reinterpret_cast<char*>(turn + HALF) + NW * Tile::SCRATCH);  // [NW][HEADS]
  float* wl = wm + NW * HEADS;
  float* wo = wl + NW * HEADS;                             // [NW][heads][OROW]
  __shared__ int64_t sums[NW];
  __shared__ int sh_b, sh_last;
  __shared__ int64_t sh_base;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t cap = (int64_t)s.max_pages << a.shift;
  T* kp = static_cast<T*>(a.kp);
  T* vp = static_cast<T*>(a.vp);
  T* out = static_cast<T*>(a.out);

  // steps of sequence b (0: not running)
  auto steps_of = [&](int b, int* pp, int* plo, int* ps0) -> int {
    const int64_t p = a.pos[b];
    if (p < 0 || p >= cap) return 0;
    *pp = (int)p;
    *plo = s.window > 0 && p >= s.window ? (int)p - s.window + 1 : 0;
    *ps0 = *plo / KSTEP;
    return (int)p / KSTEP - *ps0 + 1;
  };

  // sequences that are not running: zeros
  for (int b = blockIdx.x; b < s.B; b += gridDim.x) {
    const int64_t p = a.pos[b];
    if (p >= 0 && p < cap) continue;
    if (p >= cap && tid == 0) record_error(a.err, DEV_BOUNDS);
    for (int i = tid; i < s.H * HD; i += THREADS) out[(int64_t)b * s.H * HD + i] = from_f<T>(0.f);
  }

  // this block's range of the global steps, and the sequence it begins in
  int64_t r0, r1, per;
  {
    const int chunk = (s.B + THREADS - 1) / THREADS;
    const int b0 = tid * chunk, b1 = b0 + chunk < s.B ? b0 + chunk : s.B;
    int d0, d1, d2;
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += steps_of(b, &d0, &d1, &d2);
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    total *= a.units;
    per = (total + gridDim.x - 1) / gridDim.x;
    if (per < MIN_STEPS) per = MIN_STEPS;
    per = (per + NW - 1) / NW * NW;
    r0 = per * blockIdx.x;
    r1 = r0 + per < total ? r0 + per : total;
    if (r0 >= r1) return;
    int64_t at = (before + inc - mine) * a.units;
    if (r0 >= at && r0 < at + mine * a.units) {
      int b = b0;
      for (;; ++b) {
        const int64_t n = (int64_t)steps_of(b, &d0, &d1, &d2) * a.units;
        if (r0 < at + n) break;
        at += n;
      }
      sh_b = b;
      sh_base = at;
    }
    __syncthreads();
  }
  Cursor cur;  // the unit being worked on
  cur.b = sh_b;
  cur.n = steps_of(cur.b, &cur.p, &cur.lo, &cur.s0);
  cur.hu = (int)((r0 - sh_base) / cur.n);
  cur.base = sh_base + (int64_t)cur.hu * cur.n;
  auto seek = [&](Cursor& c, int64_t t) {  // moves on to the unit of step t < r1
    while (t >= c.base + c.n) {
      c.base += c.n;
      if (++c.hu == a.units) {
        c.hu = 0;
        do c.n = steps_of(++c.b, &c.p, &c.lo, &c.s0);
        while (c.n == 0);
      }
    }
  };
  const int groups = a.units / s.Hkv;  // units of a key/value head

  // ---- the warp's copies
  Cursor ahead = cur;
  int64_t ti = r0 + warp;  // the next step to copy
  int page = -1;           // its page, looked up one step before it is needed
  uint32_t bad = 0;        // stages whose page lies outside the pool
  auto look = [&]() {
    if (ti >= r1) return;
    seek(ahead, ti);
    const int key = (ahead.s0 + (int)(ti - ahead.base)) * KSTEP;
    page = a.table[(int64_t)ahead.b * s.max_pages + (key >> a.shift)];
  };
  const uint32_t stage0 = smem_u32(sm) + warp * STAGES * 2 * KV;
  auto issue = [&](int st) {
    if (ti < r1) {
      const int key = (ahead.s0 + (int)(ti - ahead.base)) * KSTEP;
      const int hk = ahead.hu / groups;
      const bool ok = page >= 0 && page < s.num_pages;
      // keys [from, to) of the step lie in the cache; the new entry (position p) does not
      const int from = ok ? ahead.lo - key : KSTEP, to = ok ? ahead.p - key : 0;
      const int64_t e = ((((int64_t)(ok ? page : 0) * s.Hkv + hk) << a.shift) + (key & (s.page_size - 1))) * HD;
      const char* gk = reinterpret_cast<const char*>(kp + e);
      const char* gv = reinterpret_cast<const char*>(vp + e);
      const uint32_t dk = stage0 + st * 2 * KV, dv = dk + KV;
#pragma unroll
      for (int i = 0; i < KSTEP * CPR / 32; ++i) {
        const int x = i * 32 + lane, r = x / CPR, c = x % CPR;
        const int bytes = r >= from && r < to ? 16 : 0;
        copy16(dk + piece<T, HD>(r, c), gk + x * 16, bytes);
        copy16(dv + piece<T, HD>(r, c), gv + x * 16, bytes);
      }
      bad = ok ? bad & ~(1u << st) : bad | (1u << st);
      if (!ok && lane == 0) record_error(a.err, DEV_BOUNDS);
      ti += NW;
      look();
    }
    copy_commit();
  };
  look();
#pragma unroll
  for (int st = 0; st < STAGES; ++st) issue(st);

  // ---- the range's units in order
  Tile tile;
  int st = 0;
  int turned = -1;
  int64_t t = r0 + warp;  // the warp's next step to work on
  for (int64_t at = r0; at < r1;) {
    seek(cur, at);
    const int64_t end = cur.base + cur.n < r1 ? cur.base + cur.n : r1;  // steps [at, end) of the unit
    const int hk = cur.hu / groups;
    const int h0 = hk * (s.H / s.Hkv) + (cur.hu % groups) * a.heads;
    const int heads = min(a.heads, (hk + 1) * (s.H / s.Hkv) - h0);
    const bool has_new = end == cur.base + cur.n;
    __syncthreads();  // the last unit's q and merge rows have been read
    if (turned != cur.b) {
      for (int c = tid; c < HALF; c += THREADS) turn[c] = rope_turn(cur.p, rf.inv_freq[c]);
      turned = cur.b;
      __syncthreads();
    }
    for (int i = tid; i < HEADS * HALF; i += THREADS) {
      const int j = i / HALF, c = i % HALF;
      float x = 0.f, y = 0.f;
      if (j < heads) {
        const T* q = static_cast<const T*>(a.q) + ((int64_t)cur.b * s.H + h0 + j) * HD;
        const float q1 = to_f(q[c]), q2 = to_f(q[c + HALF]);
        const float2 w = turn[c];
        x = (q1 * w.x - q2 * w.y) * a.scale_log2;
        y = (q1 * w.y + q2 * w.x) * a.scale_log2;
      }
      Tile::put_q(qs, j, c, x);
      Tile::put_q(qs, j, c + HALF, y);
    }
    if (has_new) {
      const int64_t row = ((int64_t)cur.b * s.Hkv + hk) * HD;
      int pg = -1;
      if (cur.hu % groups == 0) pg = a.table[(int64_t)cur.b * s.max_pages + (cur.p >> a.shift)];
      const bool store = pg >= 0 && pg < s.num_pages;  // a bad page is recorded where its step is copied
      const int64_t e = ((((int64_t)(store ? pg : 0) * s.Hkv + hk) << a.shift) + (cur.p & (s.page_size - 1))) * HD;
      for (int c = tid; c < HALF; c += THREADS) {
        const float2 w = turn[c];
        const T *k = static_cast<const T*>(a.k) + row, *v = static_cast<const T*>(a.v) + row;
        const float k1 = to_f(k[c]), k2 = to_f(k[c + HALF]);
        float a1 = k1 * w.x - k2 * w.y, a2 = k1 * w.y + k2 * w.x;
        float v1 = to_f(v[c]), v2 = to_f(v[c + HALF]);
        if (s.inject) {
          const T *kr = static_cast<const T*>(a.krec) + row, *vr = static_cast<const T*>(a.vrec) + row;
          const float gkl = gate_value(a.gates[hk]), gkr = gate_value(a.gates[s.Hkv + hk]);
          const float gvl = gate_value(a.gates[s.vg * s.Hkv + hk]), gvr = gate_value(a.gates[(s.vg + 1) * s.Hkv + hk]);
          a1 = gkl * a1 + gkr * to_f(kr[c]);
          a2 = gkl * a2 + gkr * to_f(kr[c + HALF]);
          v1 = gvl * v1 + gvr * to_f(vr[c]);
          v2 = gvl * v2 + gvr * to_f(vr[c + HALF]);
        }
        kn[c] = from_f<T>(a1);  // the step attends to exactly what it stores
        kn[c + HALF] = from_f<T>(a2);
        vn[c] = from_f<T>(v1);
        vn[c + HALF] = from_f<T>(v2);
        if (store) {
          kp[e + c] = from_f<T>(a1);
          kp[e + c + HALF] = from_f<T>(a2);
          vp[e + c] = from_f<T>(v1);
          vp[e + c + HALF] = from_f<T>(v2);
        }
      }
    }
    __syncthreads();
    tile.begin(qs);
    for (; t < end; t += NW) {
      const int key = (cur.s0 + (int)(t - cur.base)) * KSTEP;
      const uint32_t ks = stage0 + st * 2 * KV, vs = ks + KV;
      copy_wait<STAGES - 1>();
      __syncwarp();
      const int from = cur.lo - key, to = cur.p - key;  // keys [from, to] take part
      const bool gone = bad >> st & 1;
      if (to < KSTEP) {  // the new entry goes where its page holds it
        char* row = sm + (ks - smem_u32(sm));
        for (int c = lane; c < CPR; c += 32) {
          *reinterpret_cast<uint4*>(row + piece<T, HD>(to, c)) = reinterpret_cast<const uint4*>(kn)[c];
          *reinterpret_cast<uint4*>(row + KV + piece<T, HD>(to, c)) = reinterpret_cast<const uint4*>(vn)[c];
        }
        __syncwarp();
      }
      tile.step(
          ks, vs, from <= 0 && to >= KSTEP - 1 && !gone,
          [&](int r) { return r == to || (!gone && r >= from && r < to); }, scratch, qs, heads);
      __syncwarp();  // every lane has read the stage
      issue(st);
      st = st + 1 == STAGES ? 0 : st + 1;
    }
    // the warps' parts to one
    tile.put_ml(wm + warp * HEADS, wl + warp * HEADS);
    __syncthreads();
    float* f = wl + NW * HEADS + NW * a.heads * OROW + warp * HEADS;  // the warp's factors
    if (lane < heads) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w * HEADS + lane]);
      const float mine = wm[warp * HEADS + lane];
      f[lane] = mine == -INFINITY ? 0.f : pow2(mine - M);
    }
    __syncwarp();
    tile.template put_o<OROW>(wo + warp * a.heads * OROW, f, heads);
    __syncthreads();
    const bool whole = at == cur.base && has_new;
    const float* fac = wl + NW * HEADS + NW * a.heads * OROW;
    float* part = a.parts + ((int64_t)blockIdx.x * 2 + (at == r0 ? 0 : 1)) * PART_HEADS * PART_ROW;
    for (int i = tid; i < heads * HD; i += THREADS) {
      const int j = i / HD, c = i % HD;
      float O = 0.f, L = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        O += wo[(w * a.heads + j) * OROW + c];
        L += wl[w * HEADS + j] * fac[w * HEADS + j];
      }
      if (whole) {
        out[((int64_t)cur.b * s.H + h0 + j) * HD + c] = from_f<T>(L > 0.f || L != L ? O / L : 0.f);
      } else {
        part[j * PART_ROW + 2 + c] = O;
        if (c == 0) {
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w * HEADS + j]);
          part[j * PART_ROW] = M;
          part[j * PART_ROW + 1] = L;
        }
      }
    }
    if (!whole) {
      const int c0 = (int)(cur.base / per), c1 = (int)((cur.base + cur.n - 1) / per);  // blocks with a part
      int* counter = a.counters + (int64_t)cur.b * a.units + cur.hu;
      __syncthreads();
      if (tid == 0) {
        __threadfence();  // the block's part before its count (the fence is cumulative over the barrier)
        sh_last = atomicAdd(counter, 1) == c1 - c0;
        if (sh_last) {
          __threadfence();
          *counter = 0;  // ready for the next call
        }
      }
      __syncthreads();
      if (sh_last) {
        auto part_of = [&](int c) {  // block c's part of this unit
          return a.parts + ((int64_t)c * 2 + (per * c >= cur.base ? 0 : 1)) * PART_HEADS * PART_ROW;
        };
        for (int i = tid; i < heads * HD; i += THREADS) {
          const int j = i / HD, c = i % HD;
          float M = -INFINITY, L = 0.f, O = 0.f;
          for (int x = c0; x <= c1; ++x) M = fmaxf(M, __ldcg(part_of(x) + j * PART_ROW));
          for (int x = c0; x <= c1; ++x) {
            const float* pr = part_of(x) + j * PART_ROW;
            const float mx = __ldcg(pr);
            const float w = mx == -INFINITY ? 0.f : pow2(mx - M);
            L += w * __ldcg(pr + 1);
            O += w * __ldcg(pr + 2 + c);
          }
          out[((int64_t)cur.b * s.H + h0 + j) * HD + c] = from_f<T>(L > 0.f || L != L ? O / L : 0.f);
        }
      }
    }
    at = end;
  }
}

int units_of(const PagedShape& s, int heads) {  // units of a sequence
  const int group = s.H / s.Hkv;
  return s.Hkv * ((group + heads - 1) / heads);
}
// Query heads of a unit: as many of a key/value head's as a tile takes.
int tile_heads(const PagedShape& s) {
  if (s.dtype == 0) return 4;
  return s.H / s.Hkv > 8 ? 16 : 8;
}
constexpr int MAX_OCC = 3;  // resident blocks per SM, at most
size_t parts_bytes() { return (size_t)num_sms() * MAX_OCC * 2 * PART_HEADS * PART_ROW * sizeof(float); }

template <typename T, int HD, typename Tile, int NW, int STAGES, int OCC>
cudaError_t run(const PagedShape& s, DecodeArgs a, cudaStream_t st) {
  const int group = s.H / s.Hkv;
  a.heads = group < Tile::HEADS ? group : Tile::HEADS;
  a.units = units_of(s, Tile::HEADS);
  const size_t smem = (size_t)NW * STAGES * 2 * KSTEP * HD * sizeof(T) + Tile::Q_BYTES + 2 * HD * sizeof(T) +
                      HD / 2 * sizeof(float2) + NW * Tile::SCRATCH + 3 * NW * Tile::HEADS * sizeof(float) +
                      (size_t)NW * a.heads * (HD + 4) * sizeof(float);
  auto kern = paged_decode_kernel<T, HD, Tile, NW, STAGES, OCC>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int occ = (int)(227 * 1024 / (smem + 1024)) < OCC ? (int)(227 * 1024 / (smem + 1024)) : OCC;
  // steps there can be at most, from the sizes alone
  int64_t keys = (int64_t)s.max_pages * s.page_size;
  if (s.window > 0 && s.window + KSTEP < keys) keys = s.window + KSTEP;
  const int64_t steps = (keys + KSTEP - 1) / KSTEP * a.units * s.B;
  int64_t grid = (int64_t)num_sms() * occ;
  if (grid > (steps + MIN_STEPS - 1) / MIN_STEPS) grid = (steps + MIN_STEPS - 1) / MIN_STEPS;
  kern<<<(unsigned)grid, NW * 32, smem, st>>>(s, a, rope_freqs(HD, s.log2_base));
  return cudaGetLastError();
}

}  // namespace

// The parts have the same size for every shape, so that calls of different
// shapes can use one workspace in turn: the counters behind them stay zero.
size_t paged_decode_workspace_bytes(const PagedShape& s) {
  return parts_bytes() + (size_t)s.B * units_of(s, tile_heads(s)) * sizeof(int);
}

cudaError_t launch_paged_decode(const PagedShape& s, const int64_t* pos, const void* q, const void* k, const void* v,
                                const void* krec, const void* vrec, const float* gates, const int32_t* block_table,
                                void* k_pages, void* v_pages, void* out, void* workspace, int* err, cudaStream_t st) {
  DecodeArgs a{};
  a.pos = pos;
  a.q = q;
  a.k = k;
  a.v = v;
  a.krec = krec;
  a.vrec = vrec;
  a.gates = gates;
  a.table = block_table;
  a.kp = k_pages;
  a.vp = v_pages;
  a.out = out;
  a.parts = static_cast<float*>(workspace);
  a.counters = reinterpret_cast<int*>(static_cast<char*>(workspace) + parts_bytes());
  a.shift = log2_of(s.page_size);
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)s.hd);
  a.err = err;
  const bool wide = tile_heads(s) == 16;
  if (s.dtype == 1 && s.hd == 128)
    return wide ? run<bf16, 128, MmaTile<128, 2>, 4, 2, 2>(s, a, st) : run<bf16, 128, MmaTile<128, 1>, 4, 2, 3>(s, a, st);
  if (s.dtype == 1 && s.hd == 64)
    return wide ? run<bf16, 64, MmaTile<64, 2>, 4, 4, 2>(s, a, st) : run<bf16, 64, MmaTile<64, 1>, 4, 4, 3>(s, a, st);
  if (s.dtype == 0 && s.hd == 128) return run<float, 128, SimtTile<128>, 4, 2, 1>(s, a, st);
  if (s.dtype == 0 && s.hd == 64) return run<float, 64, SimtTile<64>, 4, 2, 3>(s, a, st);
  return cudaErrorInvalidValue;
}

}  // namespace maglev
