// One decode step over a paged key/value cache: the paged form of the ring
// step in decode.cu, for sequences of any length and grouped key/value heads.
//
// Source: "Maglev: Sliding Recurrent Memory", paper.rainbus.top, 研究动机 (the
// decoder reads a window of entries and the memory) and 前置知识 (KV cache:
// the memory rides in the existing entries); the prefiller's full layers read
// every entry (window 0).
//
// Mathematics. For a query row q (rotated, scaled to log2 units) and any split of
// its keys into parts, each part keeps (m, l, o): a reference m near the maximum
// of its scores s_j, l = sum 2^(s_j - m), o = sum 2^(s_j - m) v_j. Parts join by
// M = max m_i, l = sum 2^(m_i - M) l_i, o likewise, out = o / l.
//
// Split. The cache is read once and nothing else is large, so the kernel is bound
// by HBM and has to keep every SM streaming whatever the lengths are. A unit is a
// (sequence, key/value head, group of query heads) and is cut into steps of 16
// keys (a page holds a whole number of steps). All steps of all units, in order,
// are dealt to the warps of the grid in equal contiguous ranges (a unit weighs a few
// steps more than it has, for its query and its end). A warp works alone: it
// streams its steps through its own ring of shared-memory stages (16-byte
// asynchronous copies that run ahead across units), keeps (m, l, o) in registers,
// writes the outputs of units that lie in its range, and leaves parts (m, l, o) of
// the at most two that do not in the workspace. A second kernel, whose blocks are
// scheduled while the first one ends, joins the parts in the order of the keys:
// the same bits whatever ran first, and no block waits for another. (Ranges dealt at
// run time to even out the SMs' speeds: more parts and restarts, 108 to 113 us against
// 109 at 64 ragged sequences, 103 to 113 against 99 at 8 long ones.)
//
// Measured (one B200, GPU time in a graph; share of the bytes' time at 6535 GB/s):
//   64 sequences of 64..4096, 10 heads of 128, bf16          109.6 us  0.95
//   8 of 8192..65536, 32 query heads on 4 of 128, bf16        98.6 us  0.94
//   64 of 128..8192, window 512, 10 of 128, bf16              34.7 us  0.73
//   2 of 15005, 30010, 8 on 4 heads of 64, fp32               24.1 us  0.58
//   1 of 190, 10 of 128, bf16                                  7.6 us  (latency)
// Beside the streaming each call pays about 3.5 us from the launch to the first data
// (positions, page numbers and entries are three loads that depend on one another),
// 2 us for the join, and what the slowest SM takes longer than the average (3 to 8 us).
// More than 8 (fp32: 4) query heads to a key/value head are shared by a team of two or
// four warps, each with its own heads, over one ring of stages: the cache is read
// once for up to 32 (16) heads. Heads come in eights (fours): with 9 to 15, or 17 to 24,
// a warp of the team has little to do. Their arithmetic then is what binds: 0.76 of the
// bytes' time at 16 heads of 128, 0.43 at 24, 0.66 at 8 in fp32 (0.72, 0.42, 0.45 with
// wider tiles or several passes).
// Eight warps with two 8 KB stages each (128 KB in flight on an SM) are what HBM
// needs; with twelve the SMs' shares drift apart and the slowest ends 20% late.
#include "paged.cuh"
#include "paged_grid.h"

namespace maglev {
namespace {

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
// x = upper part + rest: the largest bf16 number nearer to zero than x, and what is left
// (at most one step of bf16), rounded to nearest. Together they carry x to 2^-16. Both
// have x's sign, and the rest of an x that is not zero is not zero either: an infinite key
// or value times both parts then is the infinity that it is times x, where inf * 0 or
// inf - inf would be a NaN. Of a bf16 number the sum is exact, and zero stays zero.
__device__ __forceinline__ uint32_t below(float x) {  // its upper 16 bits are the upper part's
  const uint32_t u = __float_as_uint(x);
  return u - ((u & 0x7fffffffu) != 0);
}
__device__ __forceinline__ uint32_t upper2(float x, float y) { return __byte_perm(below(x), below(y), 0x7632); }
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float rest(float x) { return x - __uint_as_float(below(x) & 0xffff0000u); }
__device__ __forceinline__ uint32_t rest2(float x, float y) { return pack2(rest(x), rest(y)); }

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
// bf16: 16 keys x some query heads on the tensor cores. S^T = K q^T and O^T = V^T P^T
// take the keys (the channels) as the instruction's 16 rows and the heads as its
// columns: with one head to a key head the heads are the side to pad, and 8
// columns is the least it can be padded to. The step is bound by HBM (8 KB per 16
// keys, up to 8 heads), which leaves room to carry q and P as two bf16 parts each, that
// is to 2^-16: a score errs by up to 2^-16 |q| |k| / sqrt(hd), a weight by that and 2^-16
// of itself. For scores of some tens that is far below the output's rounding (2^-8); it
// reaches it where |q| |k| / sqrt(hd) is some hundreds. The 8 NT columns hold
// both parts: up to 4 heads in one tile (columns 0-3 the upper, 4-7 the lower
// parts), 8 heads in two (the upper parts in the first).
// ---------------------------------------------------------------------------
template <int HD, int NT>
struct MmaTile {
  static constexpr int HEADS = 4 * NT, KS = HD / 16;
  static constexpr int WARP_BYTES = 0;
  static constexpr bool ONE = NT == 1;         // both parts in one tile
  static constexpr int NH = ONE ? 1 : NT / 2;  // tiles of scores
  float o[KS][NH][4];
  float m[NH][2], l[NH][2];
  uint32_t q[KS][NT][2];

  // Head of this lane's column e (of 2) in score tile n, and of its row in a B fragment.
  __device__ __forceinline__ static int col_head(int n, int e) {
    const int t = threadIdx.x % 4;
    return ONE ? 2 * (t & 1) + e : 8 * n + 2 * t + e;
  }
  __device__ __forceinline__ static int row_head(int n) {
    const int g = (threadIdx.x % 32) / 4;
    return ONE ? g & 3 : 8 * n + g;
  }
  // The raw q rows as B fragments; then, with the angles, rotated, scaled and split.
  __device__ __forceinline__ void load_q(const bf16* src, int heads) {
    const int t = threadIdx.x % 4;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          q[k][n][e] = row_head(n) < heads
                           ? *reinterpret_cast<const uint32_t*>(src + row_head(n) * HD + 16 * k + 8 * e + 2 * t)
                           : 0u;
  }
  __device__ __forceinline__ void begin(const float2* turn, float scale, char*, int) {
    const int t = threadIdx.x % 4;
    const bool lower = threadIdx.x & 16;  // ONE: this lane's column holds lower parts
#pragma unroll
    for (int k = 0; k < KS / 2; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 w = *reinterpret_cast<const float4*>(turn + 16 * k + 8 * e + 2 * t);  // two channels' angles
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q[k][n][e]));
          const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q[k + KS / 2][n][e]));
          const float x0 = (a.x * w.x - b.x * w.y) * scale, x1 = (a.y * w.z - b.y * w.w) * scale;
          const float y0 = (a.x * w.y + b.x * w.x) * scale, y1 = (a.y * w.w + b.y * w.z) * scale;
          if (ONE) {
            q[k][n][e] = lower ? rest2(x0, x1) : upper2(x0, x1);
            q[k + KS / 2][n][e] = lower ? rest2(y0, y1) : upper2(y0, y1);
          } else {
            q[k][n][e] = upper2(x0, x1);
            q[k + KS / 2][n][e] = upper2(y0, y1);
            q[k][NT - NH + n][e] = rest2(x0, x1);
            q[k + KS / 2][NT - NH + n][e] = rest2(y0, y1);
          }
        }
      }
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][n][e] = 0.f;
    }
  }
  // live(r): whether key r of the step takes part; all: every key does
  template <typename Live>
  __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, bool all, Live live, char*, int) {
    const int lane = threadIdx.x % 32, g = lane / 4;
    float s[NH][4], s2[NH][4];  // two chains of products, short enough to hide
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
    const int kr = lane & 15;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t a[4];
      ldsm4(a, ks + piece<bf16, HD>(kr, 2 * k + (lane >> 4)));
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if (ONE) {
          mma16816(k & 1 ? s2[n] : s[n], a, q[k][n][0], q[k][n][1]);
        } else {
          mma16816(s[n], a, q[k][n][0], q[k][n][1]);
          mma16816(s2[n], a, q[k][NT - NH + n][0], q[k][NT - NH + n][1]);
        }
      }
    }
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] += s2[n][e];
        if (ONE) s[n][e] += __shfl_xor_sync(0xffffffffu, s[n][e], 2);
      }
    if (!all) {  // a branch of its own: most steps are whole
      const bool on[2] = {live(g), live(g + 8)};
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!on[e / 2]) s[n][e] = -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) grow |= s[n][e] > m[n][e & 1] + SLACK;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NH; ++n)
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
    uint32_t ph[NH][2], pl[NH][2];
    const bool lower = threadIdx.x & 2;
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float r = m[n][e & 1];
        w[e] = pow2(s[n][e] - (r == -INFINITY ? 0.f : r));
        l[n][e & 1] += w[e];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (ONE) {
          ph[n][e] = transpose8x8(lower ? rest2(w[2 * e], w[2 * e + 1]) : upper2(w[2 * e], w[2 * e + 1]));
        } else {
          ph[n][e] = transpose8x8(upper2(w[2 * e], w[2 * e + 1]));
          pl[n][e] = transpose8x8(rest2(w[2 * e], w[2 * e + 1]));
        }
      }
    }
    const int vr = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t a[4];
      ldsm4_trans(a, vs + piece<bf16, HD>(vr, 2 * k + ((lane >> 3) & 1)));
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        mma16816(o[k][n], a, ph[n][0], ph[n][1]);
        if (!ONE) mma16816(o[k][n], a, pl[n][0], pl[n][1]);
      }
    }
  }
  // sums over the lanes that share a head
  __device__ __forceinline__ void finish(int heads) {
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
      if (ONE) {  // upper and lower parts; a single head lies in the even columns
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; e += 2) o[k][n][e] += __shfl_xor_sync(0xffffffffu, o[k][n][e], 2);
        if (heads > 1) {
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 1; e < 4; e += 2) o[k][n][e] += __shfl_xor_sync(0xffffffffu, o[k][n][e], 2);
        }
      }
    }
  }
  // f(head, m, l) from one lane of each head
  template <typename F>
  __device__ __forceinline__ void each_head(int heads, F f) {
    if (threadIdx.x % 32 < (ONE ? 2 : 4)) {
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (col_head(n, e) < heads) f(col_head(n, e), m[n][e], l[n][e]);
    }
  }
  // f(head, channel, value * factor(l)) from the lane that holds it
  template <typename R, typename F>
  __device__ __forceinline__ void each_out(int heads, R factor, F f) {
    const int g = (threadIdx.x % 32) / 4;
    if (ONE && (threadIdx.x & 2)) return;
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = col_head(n, e);
        if (j >= heads) continue;
        const float r = factor(l[n][e]);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          f(j, 16 * k + g, o[k][n][e] * r);
          f(j, 16 * k + g + 8, o[k][n][e + 2] * r);
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
  static constexpr int WARP_BYTES = HEADS * (HD + KSTEP) * 4;  // a warp's q rows, and its weights of a step
  static constexpr int SPLIT = 32 / PIECES > 0 ? 32 / PIECES : 1;  // lanes that share a piece (hd 64: 2)
  float o[HEADS][4];
  float m[HEADS], l[HEADS];

  float q1[HEADS][HD / 64], q2[HEADS][HD / 64];

  __device__ __forceinline__ void load_q(const float* q, int heads) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < HEADS; ++j)
#pragma unroll
      for (int r = 0; r < HD / 64; ++r) {
        q1[j][r] = j < heads ? q[j * HD + lane + 32 * r] : 0.f;
        q2[j][r] = j < heads ? q[j * HD + HD / 2 + lane + 32 * r] : 0.f;
      }
  }
  __device__ __forceinline__ void begin(const float2* turn, float scale, char* room, int) {
    const int lane = threadIdx.x % 32;
    float* q = reinterpret_cast<float*>(room);
#pragma unroll
    for (int r = 0; r < HD / 64; ++r) {
      const float2 w = turn[lane + 32 * r];
#pragma unroll
      for (int j = 0; j < HEADS; ++j) {
        q[j * HD + lane + 32 * r] = (q1[j][r] * w.x - q2[j][r] * w.y) * scale;
        q[j * HD + HD / 2 + lane + 32 * r] = (q1[j][r] * w.y + q2[j][r] * w.x) * scale;
      }
    }
    __syncwarp();
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
  __device__ __forceinline__ void step(uint32_t ks, uint32_t vs, bool all, Live live, char* room, int heads) {
    const int lane = threadIdx.x % 32, r = lane & 15, half = lane >> 4;
    const float4* q = reinterpret_cast<const float4*>(room);
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
    float* w = reinterpret_cast<float*>(room) + HEADS * HD;
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
  __device__ __forceinline__ void finish(int) {
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], d);
      if (SPLIT > 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] += __shfl_xor_sync(0xffffffffu, o[j][e], 16);
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each_head(int heads, F f) {
    if (threadIdx.x % 32 == 0) {
#pragma unroll
      for (int j = 0; j < HEADS; ++j)
        if (j < heads) f(j, m[j], l[j]);
    }
  }
  template <typename R, typename F>
  __device__ __forceinline__ void each_out(int heads, R factor, F f) {
    const int lane = threadIdx.x % 32;
    if (lane >= PIECES) return;
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
      if (j >= heads) break;
      const float r = factor(l[j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) f(j, 4 * lane + e, o[j][e] * r);
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
  float* parts;      // [teams][2][heads][PART_ROW]
  int teams;         // of the grid
  double inv_teams;
  int shift;         // log2 of the page size
  int heads, units;  // query heads of a unit (the last may have fewer), units of a sequence
  float scale_log2;
  int* err;
};

constexpr int PART_M = 128, PART_ROW = 132;  // a part's row: up to 128 channels, then m and l
// Position, first key, first step and cost of one unit of sequence b (cost 0: not
// running). Its steps are the last cost - UNIT_COST of the cost's.
struct Sequence {
  int p, lo, s0, cost;
};
__device__ __forceinline__ Sequence sequence_at(const PagedShape& s, const DecodeArgs& a, int64_t p) {
  Sequence r{0, 0, 0, 0};
  if (p < 0 || p >= (int64_t)s.max_pages << a.shift) return r;
  r.p = (int)p;
  r.lo = s.window > 0 && p >= s.window ? (int)p - s.window + 1 : 0;
  r.s0 = r.lo / KSTEP;
  r.cost = r.p / KSTEP - r.s0 + 1 + UNIT_COST;
  return r;
}

// A position; EARLY: read before this kernel has waited for the last one. The kernel before has waited for whatever wrote
// the positions, so they lie in L2, but only a wait of its own says that this SM's L1 holds nothing older.
template <bool EARLY>
__device__ __forceinline__ int64_t position(const DecodeArgs& a, int b) {
  return EARLY ? (int64_t)__ldcg(reinterpret_cast<const long long*>(a.pos) + b) : a.pos[b];
}
template <bool EARLY = false>
__device__ __forceinline__ Sequence sequence(const PagedShape& s, const DecodeArgs& a, int b) {
  return sequence_at(s, a, position<EARLY>(a, b));
}

// The costs of all units in order make one line, which is cut into equal ranges.
// It follows from the positions alone: every block of both kernels forms the same
// sums. Thread i covers `chunk` sequences from i * chunk.
template <int THREADS, int TEAMS>
struct Plan {
  int64_t before[THREADS];  // costs (of one unit each) of the sequences before thread i's
  int64_t sums[THREADS / 32];
  int owner[TEAMS];  // the thread whose sequences hold where the block's team i begins
};
// What a thread keeps of it.
struct Steps {
  int64_t total, per;  // cost of all units, of a team's range
  int chunk;
};
template <bool EARLY, int THREADS, int TEAMS>
__device__ __forceinline__ Steps form_plan(Plan<THREADS, TEAMS>& plan, const PagedShape& s, const DecodeArgs& a) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  Steps r;
  r.chunk = (s.B + THREADS - 1) / THREADS;
  int64_t mine = 0;
  const int b0 = tid * r.chunk, b1 = b0 + r.chunk < s.B ? b0 + r.chunk : s.B;
  for (int b = b0; b < b1; b += 8) {
    int64_t p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = b + e < b1 ? position<EARLY>(a, b + e) : -1;
#pragma unroll
    for (int e = 0; e < 8; ++e) mine += sequence_at(s, a, p[e]).cost;
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) plan.sums[warp] = inc;
  __syncthreads();
  int64_t at = inc - mine;
  r.total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) at += plan.sums[w];
    r.total += plan.sums[w];
  }
  plan.before[tid] = at;
  r.total *= a.units;
  // total / teams, rounded up (a 64-bit division would take 0.3 us here)
  r.per = r.total > 0 ? (int64_t)((double)(r.total - 1) * a.inv_teams) + 1 : 1;
  if (r.per * a.teams < r.total) ++r.per;
  at *= a.units;
  mine *= a.units;
#pragma unroll
  for (int i = 0; i < TEAMS; ++i) {
    const int64_t t = r.per * ((int64_t)blockIdx.x * TEAMS + i) - at;
    if (t >= 0 && t < mine) plan.owner[i] = tid;
  }
  __syncthreads();
  return r;
}

// The unit that a place on the line lies in: sequence, unit within it, where it begins.
struct Cursor {
  int b, hu;
  Sequence q;
  int64_t base;
};
// The one of place t, which thread `owner`'s sequences hold.
template <typename P>
__device__ __forceinline__ Cursor locate(const P& plan, const Steps& steps, const PagedShape& s,
                                         const DecodeArgs& a, int owner, int64_t t) {
  Cursor c;
  c.b = owner * steps.chunk;
  int64_t at = plan.before[owner] * a.units;
  for (;; ++c.b) {
    c.q = sequence(s, a, c.b);
    if (t < at + (int64_t)c.q.cost * a.units) break;
    at += (int64_t)c.q.cost * a.units;
  }
  const int64_t rest = t - at;
  c.hu = (int)((float)rest / (float)c.q.cost);  // off by one at most: units are few
  if ((int64_t)c.hu * c.q.cost > rest) --c.hu;
  if ((int64_t)(c.hu + 1) * c.q.cost <= rest) ++c.hu;
  c.base = at + (int64_t)c.hu * c.q.cost;
  return c;
}
// Moves on to the next unit.
__device__ __forceinline__ void next_unit(Cursor& c, const PagedShape& s, const DecodeArgs& a) {
  c.base += c.q.cost;
  if (++c.hu < a.units) return;
  c.hu = 0;
  do c.q = sequence(s, a, ++c.b);
  while (c.q.cost == 0);
}

// TW warps form a team that shares its steps' stages and takes Tile::HEADS heads each.
template <typename T, int HD, typename Tile, int TW, int NW, int STAGES, int OCC>
__global__ void __launch_bounds__(NW * 32, OCC) paged_decode_kernel(PagedShape s, DecodeArgs a,
                                                                  const __grid_constant__ RopeFreqs rf) {
  constexpr int HALF = HD / 2, NP = HALF / 32;
  constexpr int CPR = HD * (int)sizeof(T) / 16;    // 16-byte pieces of an entry
  constexpr int KV = KSTEP * HD * (int)sizeof(T);  // K (or V) bytes of a step
  constexpr int TEAMS = NW / TW;
  extern __shared__ __align__(128) char sm[];
  __shared__ Plan<NW * 32, TEAMS> plan;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, team = warp / TW, rank = warp % TW;
  char* stages = sm + team * STAGES * 2 * KV;
  char* after = sm + TEAMS * STAGES * 2 * KV;
  char* room = after + warp * Tile::WARP_BYTES;
  T* entry = reinterpret_cast<T*>(after + NW * Tile::WARP_BYTES) + warp * 2 * HD;  // the new K, V
  float2* turn = reinterpret_cast<float2*>(after + NW * (Tile::WARP_BYTES + 2 * HD * sizeof(T))) + warp * HALF;
  auto team_sync = [&]() {
    if (TW == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TW * 32) : "memory");
  };
  T* kp = static_cast<T*>(a.kp);
  T* vp = static_cast<T*>(a.vp);
  T* out = static_cast<T*>(a.out);

  wait_for_last();
  let_next_start();  // the join's blocks may take the places that come free
  const Steps steps = form_plan<false>(plan, s, a);
  const int64_t per = steps.per, total = steps.total;
  const int me = blockIdx.x * TEAMS + team;
  const int64_t t0 = per * me, t1 = t0 + per < total ? t0 + per : total;  // the team's range
  if (t0 >= t1) return;
  const int groups = a.units / s.Hkv, per_kv = s.H / s.Hkv;  // units, query heads of a key/value head
  Cursor cur = locate(plan, steps, s, a, plan.owner[team], t0);  // the unit being worked on
  // [begin, end) of a unit's steps lie in the range
  auto begin_of = [&](const Cursor& c) { return c.base + UNIT_COST > t0 ? c.base + UNIT_COST : t0; };
  auto end_of = [&](const Cursor& c) { return c.base + c.q.cost < t1 ? c.base + c.q.cost : t1; };
  if (begin_of(cur) >= t1) return;  // the last unit's steps are the next team's

  // ---- copies
  Cursor ahead = cur;
  int akey, aleft, ahk;    // the next step's first key, the steps left of its unit (0: of the range), its key/value head
  const int32_t* arow;     // its row of the block table
  int page;                // its page, looked up one step before it is needed
  uint32_t bad = 0;        // stages whose page lies outside the pool
  auto enter = [&]() {     // the copies reach unit `ahead`
    const int64_t t = begin_of(ahead);
    akey = (ahead.q.s0 + (int)(t - ahead.base - UNIT_COST)) * KSTEP;
    aleft = (int)(end_of(ahead) - t);
    ahk = ahead.hu / groups;
    arow = a.table + (int64_t)ahead.b * s.max_pages;
  };
  enter();
  page = arow[akey >> a.shift];
  const uint32_t stage0 = smem_u32(stages);
  // a lane's i-th piece of a step's K or V lies HOP i bytes on, and goes to HOP i + put[i % PUTS]
  constexpr int HOP = 512 * TW, PERIOD = CPR / 4, PUTS = PERIOD > TW ? PERIOD / TW : 1, PIECES = KSTEP * CPR / 32 / TW;
  uint32_t put[PUTS];
#pragma unroll
  for (int i = 0; i < PUTS; ++i) {
    const int x = (i * TW + rank) * 32 + lane;
    put[i] = piece<T, HD>(x / CPR, x % CPR) - HOP * i;
  }
  auto issue = [&](int st) {
    if (aleft > 0) {
      const bool ok = page >= 0 && page < s.num_pages;
      // keys [from, to) of the step lie in the cache; the new entry (position p) does not
      const int from = ok ? ahead.q.lo - akey : KSTEP, to = ok ? ahead.q.p - akey : 0;
      const int64_t e = ((((int64_t)(ok ? page : 0) * s.Hkv + ahk) << a.shift) + (akey & (s.page_size - 1))) * HD +
                        (rank * 32 + lane) * (16 / (int)sizeof(T));
      const char* gk = reinterpret_cast<const char*>(kp + e);
      const char* gv = reinterpret_cast<const char*>(vp + e);
      const uint32_t dk = stage0 + st * 2 * KV;
      if (from <= 0 && to >= KSTEP) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          copy16(dk + put[i % PUTS] + HOP * i, gk + HOP * i, 16);
          copy16(dk + put[i % PUTS] + HOP * i + KV, gv + HOP * i, 16);
        }
      } else {
        for (int i = 0; i < PIECES; ++i) {
          const int x = (i * TW + rank) * 32 + lane, r = x / CPR;
          const int bytes = r >= from && r < to ? 16 : 0;
          copy16(dk + piece<T, HD>(r, x % CPR), gk + HOP * i, bytes);
          copy16(dk + piece<T, HD>(r, x % CPR) + KV, gv + HOP * i, bytes);
        }
      }
      bad = ok ? bad & ~(1u << st) : bad | (1u << st);
      if (!ok && lane == 0) record_error(a.err, DEV_BOUNDS);
      akey += KSTEP;
      if (--aleft == 0 && ahead.base + ahead.q.cost + UNIT_COST < t1) {
        next_unit(ahead, s, a);
        enter();
      }
      if (aleft > 0) page = arow[akey >> a.shift];
    }
    copy_commit();
  };
  int turned = -1;
  auto turn_to = [&](const Cursor& c) {  // the angles of its sequence's position
    if (turned == c.b) return;
    turned = c.b;
    __syncwarp();  // the last ones have been read
#pragma unroll
    for (int r = 0; r < NP; ++r) turn[lane + 32 * r] = rope_turn(c.q.p, rf.turns[lane + 32 * r]);
    __syncwarp();
  };
  turn_to(cur);  // while the first page number is on its way
#pragma unroll
  for (int st = 0; st < STAGES; ++st) issue(st);

  // ---- the range's units in order
  Tile tile;
  int st = 0;
  for (;;) {
    const int64_t t = begin_of(cur), end = end_of(cur);  // steps [t, end) of the unit
    const int hk = cur.hu / groups;
    const int h0 = hk * per_kv + (cur.hu % groups) * a.heads;
    const int first = h0 + rank * Tile::HEADS;  // the warp's heads (none: the unit has fewer)
    const int unit_heads = min(a.heads, (hk + 1) * per_kv - h0);
    const int heads = TW == 1 ? unit_heads : min(Tile::HEADS, unit_heads - rank * Tile::HEADS);
    const bool has_new = end == cur.base + cur.q.cost, whole = t == cur.base + UNIT_COST && has_new;
    // every load of the unit at once: the query rows, and the new entry's parts
    const int64_t row = ((int64_t)cur.b * s.Hkv + hk) * HD;
    float k1[NP], k2[NP], v1[NP], v2[NP], kr1[NP], kr2[NP], vr1[NP], vr2[NP], ga = 0.f, gb = 0.f, gc = 0.f, gd = 0.f;
    int pg = -1;
    tile.load_q(static_cast<const T*>(a.q) + ((int64_t)cur.b * s.H + first) * HD, heads);
    if (has_new && rank == 0) {
      const T *k = static_cast<const T*>(a.k) + row, *v = static_cast<const T*>(a.v) + row;
      const T *kr = static_cast<const T*>(a.krec) + row, *vr = static_cast<const T*>(a.vrec) + row;
      if (cur.hu % groups == 0) pg = a.table[(int64_t)cur.b * s.max_pages + (cur.q.p >> a.shift)];
#pragma unroll
      for (int r = 0; r < NP; ++r) {
        const int c = lane + 32 * r;
        k1[r] = to_f(k[c]);
        k2[r] = to_f(k[c + HALF]);
        v1[r] = to_f(v[c]);
        v2[r] = to_f(v[c + HALF]);
        if (s.inject) {
          kr1[r] = to_f(kr[c]);
          kr2[r] = to_f(kr[c + HALF]);
          vr1[r] = to_f(vr[c]);
          vr2[r] = to_f(vr[c + HALF]);
        }
      }
      if (s.inject) {
        ga = a.gates[hk];
        gb = a.gates[s.Hkv + hk];
        gc = a.gates[s.vg * s.Hkv + hk];
        gd = a.gates[(s.vg + 1) * s.Hkv + hk];
      }
    }
    turn_to(cur);
    tile.begin(turn, a.scale_log2, room, heads);
    if (has_new && rank == 0) {
      const bool store = pg >= 0 && pg < s.num_pages;  // a bad page is recorded where its step is copied
      const int64_t e = ((((int64_t)(store ? pg : 0) * s.Hkv + hk) << a.shift) + (cur.q.p & (s.page_size - 1))) * HD;
#pragma unroll
      for (int r = 0; r < NP; ++r) {
        const int c = lane + 32 * r;
        const float2 w = turn[c];
        float x1 = k1[r] * w.x - k2[r] * w.y, x2 = k1[r] * w.y + k2[r] * w.x, y1 = v1[r], y2 = v2[r];
        if (s.inject) {
          const float gkl = gate_value(ga), gkr = gate_value(gb), gvl = gate_value(gc), gvr = gate_value(gd);
          x1 = gkl * x1 + gkr * kr1[r];
          x2 = gkl * x2 + gkr * kr2[r];
          y1 = gvl * y1 + gvr * vr1[r];
          y2 = gvl * y2 + gvr * vr2[r];
        }
        const T e1 = from_f<T>(x1), e2 = from_f<T>(x2), f1 = from_f<T>(y1), f2 = from_f<T>(y2);
        entry[c] = e1;  // the step attends to exactly what it stores
        entry[c + HALF] = e2;
        entry[HD + c] = f1;
        entry[HD + c + HALF] = f2;
        if (store) {
          kp[e + c] = e1;
          kp[e + c + HALF] = e2;
          vp[e + c] = f1;
          vp[e + c + HALF] = f2;
        }
      }
      __syncwarp();
    }
    int key = (cur.q.s0 + (int)(t - cur.base - UNIT_COST)) * KSTEP;
    const int key_end = key + (int)(end - t) * KSTEP;
#pragma unroll 1
    for (; key < key_end; key += KSTEP) {
      const uint32_t ks = stage0 + st * 2 * KV, vs = ks + KV;
      copy_wait<STAGES - 1>();
      team_sync();  // the team's copies of the stage have landed
      const int from = cur.q.lo - key, to = cur.q.p - key;  // keys [from, to] take part
      const bool gone = bad >> st & 1;
      if (to < KSTEP) {  // the new entry goes where its page holds it
        if (rank == 0) {
          char* dst = stages + st * 2 * KV;
          for (int c = lane; c < CPR; c += 32) {
            *reinterpret_cast<uint4*>(dst + piece<T, HD>(to, c)) = reinterpret_cast<const uint4*>(entry)[c];
            *reinterpret_cast<uint4*>(dst + KV + piece<T, HD>(to, c)) = reinterpret_cast<const uint4*>(entry + HD)[c];
          }
        }
        team_sync();
      }
      if (TW == 1 || heads > 0)
        tile.step(
            ks, vs, from <= 0 && to >= KSTEP - 1 && !gone,
            [&](int r) { return r == to || (!gone && r >= from && r < to); }, room, heads);
      team_sync();  // every lane has read the stage
      issue(st);
      st = st + 1 == STAGES ? 0 : st + 1;
    }
    tile.finish(heads);
    if (whole) {
      T* d = out + ((int64_t)cur.b * s.H + first) * HD;
      tile.each_out(
          heads, [](float l) { return 1.f / l; },  // (no weight at all: 0 * inf, as the formula has it)
          [&](int j, int c, float x) { d[j * HD + c] = from_f<T>(x); });
    } else {
      // the unit that holds the range's first place, or the one that goes on behind its last
      float* part = a.parts + (((int64_t)me * 2 + (cur.base + UNIT_COST <= t0 ? 0 : 1)) * a.heads + first - h0) * PART_ROW;
      tile.each_out(
          heads, [](float) { return 1.f; }, [&](int j, int c, float x) { part[j * PART_ROW + c] = x; });
      tile.each_head(heads, [&](int j, float m, float l) {
        *reinterpret_cast<float2*>(part + j * PART_ROW + PART_M) = make_float2(m, l);
      });
    }
    if (cur.base + cur.q.cost + UNIT_COST >= t1) break;
    next_unit(cur, s, a);
  }
}

// ---------------------------------------------------------------------------
// The outputs of units in several teams' ranges, and zeros for sequences that are
// not running. A block's warps are divided among its (sequence, query head)s; one with
// very many parts they take together. A lane owns four channels: what counts is the
// latency of parts in L2.
// ---------------------------------------------------------------------------
constexpr int JOIN_WARPS = 8;
constexpr int FLY = 8;  // parts of a lane in flight

// (m, l, o) of four channels over some of a unit's parts.
struct Joined {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float m2, float l2, float4 o2) {
    const float mn = fmaxf(m, m2), r = mn == -INFINITY ? 0.f : mn, f = pow2(m - r), f2 = pow2(m2 - r);
    l = l * f + l2 * f2;
    o.x = o.x * f + o2.x * f2;
    o.y = o.y * f + o2.y * f2;
    o.z = o.z * f + o2.z * f2;
    o.w = o.w * f + o2.w * f2;
    m = mn;
  }
};
// Where the parts of a head lie: the first one, the others `stride` apart from `rest` on.
struct Parts {
  const float *first, *rest;
  int np;
};

// Parts x1, x1 + step, ... of a head, channels c..c+3.
__device__ __forceinline__ Joined join_parts(const Parts& p, int64_t stride, int c, int x1, int step) {
  Joined r{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
  for (int x0 = x1; x0 < p.np; x0 += FLY * step) {
    float2 ml[FLY];
    float4 y[FLY];
#pragma unroll
    for (int u = 0; u < FLY; ++u) {
      const int x = x0 + u * step;
      ml[u] = make_float2(-INFINITY, 0.f);
      if (x < p.np) {
        const float* part = x == 0 ? p.first : p.rest + x * stride;
        ml[u] = __ldcg(reinterpret_cast<const float2*>(part + PART_M));
        y[u] = __ldcg(reinterpret_cast<const float4*>(part + c));
      }
    }
    float mn = r.m;
#pragma unroll
    for (int u = 0; u < FLY; ++u) mn = fmaxf(mn, ml[u].x);
    const float ref = mn == -INFINITY ? 0.f : mn, f = pow2(r.m - ref);
    r.l *= f;
    r.o.x *= f;
    r.o.y *= f;
    r.o.z *= f;
    r.o.w *= f;
    r.m = mn;
#pragma unroll
    for (int u = 0; u < FLY; ++u) {
      if (x0 + u * step >= p.np) break;
      const float w = pow2(ml[u].x - ref);
      r.l += w * ml[u].y;
      r.o.x += w * y[u].x;
      r.o.y += w * y[u].y;
      r.o.z += w * y[u].z;
      r.o.w += w * y[u].w;
    }
  }
  return r;
}

template <typename T, int HD>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 2) paged_join_kernel(PagedShape s, DecodeArgs a, int per_block) {
  constexpr int NW = JOIN_WARPS, V = HD / 4, SHARE = 32 / V;  // lanes that share four channels (hd 64: 2)
  __shared__ Plan<NW * 32, 0> plan;
  __shared__ Parts parts[NW];
  __shared__ float4 so[NW][V];
  __shared__ float sm[NW], sl[NW];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = lane % V * 4;
  const int each = NW / per_block, rank = warp % each;  // warps of a head
  const int longest = 4 * FLY * SHARE * each;                               // parts they take alone: four loads' time
  const Steps steps = form_plan<true>(plan, s, a);  // reads nothing that the first kernel writes
  const int64_t heads = (int64_t)s.B * s.H, stride = (int64_t)2 * a.heads * PART_ROW;  // from team to team
  const int groups = a.units / s.Hkv, per_kv = s.H / s.Hkv;
  bool waited = false;
  for (int64_t at = (int64_t)blockIdx.x * per_block; at < heads; at += (int64_t)gridDim.x * per_block) {
    const int64_t head = at + warp / each;
    const bool mine = head < heads;
    Parts p{nullptr, nullptr, 1};
    if (mine) {
      const int b = (int)(head / s.H), h = (int)(head % s.H), hk = h / per_kv, in_kv = h - hk * per_kv;
      const Sequence q = sequence<true>(s, a, b);
      const int i = b / steps.chunk;
      int64_t base = plan.before[i];
      for (int x = i * steps.chunk; x < b; ++x) base += sequence<true>(s, a, x).cost;
      // the unit's first step, and the teams that have steps of it
      base = base * a.units + (int64_t)(hk * groups + in_kv / a.heads) * q.cost + UNIT_COST;
      const int w0 = (int)(base / steps.per);
      p.np = q.cost ? (int)((base + q.cost - UNIT_COST - 1) / steps.per) - w0 + 1 : 0;
      p.rest = a.parts + w0 * stride + in_kv % a.heads * PART_ROW;
      p.first = p.rest + (base > steps.per * w0 ? stride / 2 : 0);  // behind other units of team w0's range
      if (p.np == 0 && rank == 0 && lane == 0 && position<true>(a, b) >= 0) record_error(a.err, DEV_BOUNDS);  // beyond the table
    }
    if (!waited) wait_for_last();  // the parts are written
    waited = true;
    // (the barrier also ends the last round's use of the shared rows)
    const int help = __syncthreads_or(p.np > longest) ? per_block : 0;
    if (help) {
      if (rank == 0 && lane == 0) parts[warp / each] = p;
      __syncthreads();
    }
    Joined r{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
    for (int i = 0; i <= help; ++i) {  // the heads with the most parts by the whole block, then each its own
      const bool together = i < help;
      if (together && parts[i].np <= longest) continue;
      Joined x{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      Parts of = p;  // (by value: a choice between the two places would keep p in memory)
      if (together) of = parts[i];
      if (together || (p.np > 1 && p.np <= longest))
        x = join_parts(of, stride, c, (together ? warp : rank) * SHARE + lane / V,
                       (together ? NW : each) * SHARE);
      if (SHARE > 1)  // lanes with the same channels
        x.add(__shfl_down_sync(0xffffffffu, x.m, 16), __shfl_down_sync(0xffffffffu, x.l, 16),
              make_float4(__shfl_down_sync(0xffffffffu, x.o.x, 16), __shfl_down_sync(0xffffffffu, x.o.y, 16),
                          __shfl_down_sync(0xffffffffu, x.o.z, 16), __shfl_down_sync(0xffffffffu, x.o.w, 16)));
      if (!together && each == 1) {
        if (p.np <= longest) r = x;
        break;
      }
      if (lane < V) so[warp][lane] = x.o;
      if (lane == 0) {
        sm[warp] = x.m;
        sl[warp] = x.l;
      }
      __syncthreads();
      if (lane < V && (together ? warp == i * each : rank == 0 && p.np <= longest))
        for (int w = together ? 0 : warp, n = together ? NW : each; n > 0; ++w, --n) r.add(sm[w], sl[w], so[w][lane]);
      __syncthreads();
    }
    if (!mine || p.np == 1 || rank != 0 || lane >= V) continue;  // np == 1: its team has written it
    T* out = static_cast<T*>(a.out) + head * HD;
    const float f = p.np == 0 ? 0.f : 1.f / r.l;
    out[c] = from_f<T>(r.o.x * f);
    out[c + 1] = from_f<T>(r.o.y * f);
    out[c + 2] = from_f<T>(r.o.z * f);
    out[c + 3] = from_f<T>(r.o.w * f);
  }
}

int units_of(const PagedShape& s, int heads) {  // units of a sequence
  const int group = s.H / s.Hkv;
  return s.Hkv * ((group + heads - 1) / heads);
}
// Query heads of a unit: as many of a key/value head's as a tile takes, or two or
// four tiles of a team where there are more.
int unit_heads(const PagedShape& s) {
  const int group = s.H / s.Hkv, most = s.dtype == 0 ? 16 : 32;
  int n = 4;
  while (n < group && n < most) n *= 2;
  return n;
}
constexpr int MAX_WARPS = 12;  // of an SM, at most

template <typename T, int HD, typename Tile, int TW, int NW, int STAGES, int OCC>
cudaError_t run(const PagedShape& s, DecodeArgs a, cudaStream_t st) {
  static_assert(NW * OCC <= MAX_WARPS, "the workspace holds the parts of MAX_WARPS warps an SM");
  constexpr int TEAMS = NW / TW;
  const int group = s.H / s.Hkv;
  a.heads = group < TW * Tile::HEADS ? group : TW * Tile::HEADS;
  a.units = units_of(s, TW * Tile::HEADS);
  constexpr size_t smem = (size_t)TEAMS * STAGES * 2 * KSTEP * HD * sizeof(T) +
                          (size_t)NW * (Tile::WARP_BYTES + 2 * HD * sizeof(T) + HD / 2 * sizeof(float2));
  static_assert((smem + sizeof(Plan<NW * 32, TEAMS>) + 1024) * OCC <= 228 * 1024, "OCC blocks share an SM's memory");
  auto kern = paged_decode_kernel<T, HD, Tile, TW, NW, STAGES, OCC>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = decode_blocks(s.B, a.units, s.max_pages, s.page_size, s.window, TEAMS, (int64_t)num_sms() * OCC);
  a.teams = (int)grid * TEAMS;
  a.inv_teams = 1.0 / a.teams;
  e = launch_dependent(kern, dim3((unsigned)grid), NW * 32, smem, st, s, a, rope_freqs(HD, s.log2_base));
  if (e != cudaSuccess) return e;
  // the join: scheduled as the first kernel ends, its blocks wait for that before they read a part
  const int64_t heads = (int64_t)s.B * s.H, blocks = 2 * num_sms();
  int per_block = 1;  // heads of a block: 1, 2, 4 or 8
  while (per_block < JOIN_WARPS && per_block * blocks < heads) per_block *= 2;
  const int64_t need = (heads + per_block - 1) / per_block;
  return launch_dependent(paged_join_kernel<T, HD>, dim3((unsigned)(need < blocks ? need : blocks)), JOIN_WARPS * 32, 0,
                          st, s, a, per_block);
}

}  // namespace

size_t paged_decode_workspace_bytes(const PagedShape& s) {
  const int group = s.H / s.Hkv, most = unit_heads(s), warps = most / (s.dtype == 0 ? 4 : 8);  // of a team
  return (size_t)num_sms() * (MAX_WARPS / (warps > 1 ? warps : 1)) * 2 * (group < most ? group : most) * PART_ROW *
         sizeof(float);
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
  a.shift = log2_of(s.page_size);
  a.scale_log2 = 1.4426950408889634f / sqrtf((float)s.hd);
  a.err = err;
  const int heads = unit_heads(s);
  if (s.dtype == 1 && s.hd == 128) {
    if (heads == 4) return run<bf16, 128, MmaTile<128, 1>, 1, 4, 2, 2>(s, a, st);
    if (heads == 8) return run<bf16, 128, MmaTile<128, 2>, 1, 4, 2, 2>(s, a, st);
    if (heads == 16) return run<bf16, 128, MmaTile<128, 2>, 2, 4, 3, 3>(s, a, st);
    return run<bf16, 128, MmaTile<128, 2>, 4, 4, 6, 3>(s, a, st);
  }
  if (s.dtype == 1 && s.hd == 64) {
    if (heads == 4) return run<bf16, 64, MmaTile<64, 1>, 1, 4, 2, 3>(s, a, st);
    if (heads == 8) return run<bf16, 64, MmaTile<64, 2>, 1, 4, 3, 2>(s, a, st);
    if (heads == 16) return run<bf16, 64, MmaTile<64, 2>, 2, 4, 4, 3>(s, a, st);
    return run<bf16, 64, MmaTile<64, 2>, 4, 4, 6, 3>(s, a, st);
  }
  if (s.dtype == 0 && s.hd == 128) {
    if (heads == 4) return run<float, 128, SimtTile<128>, 1, 4, 2, 1>(s, a, st);
    if (heads == 8) return run<float, 128, SimtTile<128>, 2, 4, 2, 2>(s, a, st);
    return run<float, 128, SimtTile<128>, 4, 4, 2, 3>(s, a, st);
  }
  if (s.dtype == 0 && s.hd == 64) {
    if (heads == 4) return run<float, 64, SimtTile<64>, 1, 4, 2, 2>(s, a, st);
    if (heads == 8) return run<float, 64, SimtTile<64>, 2, 4, 3, 3>(s, a, st);
    return run<float, 64, SimtTile<64>, 4, 4, 4, 3>(s, a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace maglev
