// One decode step over a paged key/value cache: the paged form of the ring
// step in decode.cu, for sequences of any length and grouped key/value heads.
//
// Source: "Maglev: Sliding Recurrent Memory", paper.rainbus.top, 研究动机 (the
// decoder reads a window of entries and the memory) and 前置知识 (KV cache:
// the memory rides in the existing entries); the prefiller's full layers read
// every entry (window 0).
#include "paged.cuh"

namespace maglev {
namespace {

constexpr int PD_THREADS = 256;

// One block per (sequence, query head); each warp walks every eighth key with
// an online softmax (log2 units) over them, the lanes holding the channels.
template <typename T, int HD>
__global__ void __launch_bounds__(PD_THREADS) paged_decode_kernel(
    PagedShape s, RopeFreqs rf, int shift, const int64_t* __restrict__ pos, const T* __restrict__ q,
    const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ krec, const T* __restrict__ vrec,
    const float* __restrict__ gates, const int32_t* __restrict__ table, T* __restrict__ kp, T* __restrict__ vp,
    T* __restrict__ out, float scale_log2, int* err) {
  constexpr int HALF = HD / 2, NW = PD_THREADS / 32, CPL = HD / 32;
  __shared__ float qs[HD], kn[HD], vn[HD];
  __shared__ float wm[NW], wl[NW], wo[NW][HD];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int b = blockIdx.x / s.H, h = blockIdx.x % s.H, group = s.H / s.Hkv, hk = h / group;
  const int64_t p = pos[b];
  const int64_t qrow = (int64_t)blockIdx.x * HD, krow = ((int64_t)b * s.Hkv + hk) * HD;
  if (p < 0 || p >= ((int64_t)s.max_pages << shift)) {
    if (p >= 0 && tid == 0) record_error(err, DEV_BOUNDS);
    if (tid < HD) out[qrow + tid] = from_f<T>(0.f);
    return;
  }
  if (tid < HALF) {
    const int c = tid;
    const float2 w = rope_turn(p, rf.inv_freq[c]);
    const float q1 = to_f(q[qrow + c]), q2 = to_f(q[qrow + c + HALF]);
    qs[c] = (q1 * w.x - q2 * w.y) * scale_log2;
    qs[c + HALF] = (q1 * w.y + q2 * w.x) * scale_log2;
    const float k1 = to_f(k[krow + c]), k2 = to_f(k[krow + c + HALF]);
    float a1 = k1 * w.x - k2 * w.y, a2 = k1 * w.y + k2 * w.x;
    float v1 = to_f(v[krow + c]), v2 = to_f(v[krow + c + HALF]);
    if (s.inject) {
      const float gkl = gate_value(gates[hk]), gkr = gate_value(gates[s.Hkv + hk]);
      const float gvl = gate_value(gates[s.vg * s.Hkv + hk]), gvr = gate_value(gates[(s.vg + 1) * s.Hkv + hk]);
      a1 = gkl * a1 + gkr * to_f(krec[krow + c]);
      a2 = gkl * a2 + gkr * to_f(krec[krow + c + HALF]);
      v1 = gvl * v1 + gvr * to_f(vrec[krow + c]);
      v2 = gvl * v2 + gvr * to_f(vrec[krow + c + HALF]);
    }
    kn[c] = to_f(from_f<T>(a1));  // the step attends to exactly what it stores
    kn[c + HALF] = to_f(from_f<T>(a2));
    vn[c] = to_f(from_f<T>(v1));
    vn[c + HALF] = to_f(from_f<T>(v2));
  }
  __syncthreads();
  const int32_t* row = table + (int64_t)b * s.max_pages;
  auto entry = [&](int64_t j) -> int64_t {  // element offset of position j's entry, -1 outside the pool
    const int page = row[j >> shift];
    if (page < 0 || page >= s.num_pages) return -1;
    return ((((int64_t)page * s.Hkv + hk) << shift) + (j & (s.page_size - 1))) * HD;
  };
  if (h % group == 0 && tid < HD) {
    const int64_t e = entry(p);
    if (e >= 0) {
      kp[e + tid] = from_f<T>(kn[tid]);
      vp[e + tid] = from_f<T>(vn[tid]);
    } else if (tid == 0) {
      record_error(err, DEV_BOUNDS);
    }
  }
  const int64_t lo = s.window > 0 && p >= s.window ? p - s.window + 1 : 0;
  float m = -INFINITY, l = 0.f, o[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) o[c] = 0.f;
  for (int64_t j = lo + warp; j <= p; j += NW) {
    const int64_t e = j == p ? 0 : entry(j);
    if (e < 0) {
      if (lane == 0) record_error(err, DEV_BOUNDS);
      continue;
    }
    float d = 0.f, vv[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int ch = lane + 32 * c;
      d = fmaf(qs[ch], j == p ? kn[ch] : to_f(kp[e + ch]), d);
      vv[c] = j == p ? vn[ch] : to_f(vp[e + ch]);
    }
    d = warp_sum(d);
    const float mn = fmaxf(m, d);
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float pr = mn == -INFINITY ? 0.f : exp2f(d - mn);
    l = l * alpha + pr;
#pragma unroll
    for (int c = 0; c < CPL; ++c) o[c] = o[c] * alpha + pr * vv[c];
    m = mn;
  }
#pragma unroll
  for (int c = 0; c < CPL; ++c) wo[warp][lane + 32 * c] = o[c];
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
  __syncthreads();
  if (tid < HD) {
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w]);
    for (int w = 0; w < NW; ++w) {
      const float a = wm[w] == -INFINITY ? 0.f : exp2f(wm[w] - M);
      L += a * wl[w];
      O += a * wo[w][tid];
    }
    out[qrow + tid] = from_f<T>(O / L);
  }
}

}  // namespace

size_t paged_decode_workspace_bytes(const PagedShape&) { return 0; }

cudaError_t launch_paged_decode(const PagedShape& s, const int64_t* pos, const void* q, const void* k, const void* v,
                                const void* krec, const void* vrec, const float* gates, const int32_t* block_table,
                                void* k_pages, void* v_pages, void* out, void*, int* err, cudaStream_t st) {
  const RopeFreqs rf = rope_freqs(s.hd, s.log2_base);
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)s.hd);
  const int shift = log2_of(s.page_size);
  auto go = [&](auto kern, auto t) {
    using T = decltype(t);
    kern<<<(unsigned)(s.B * s.H), PD_THREADS, 0, st>>>(s, rf, shift, pos, (const T*)q, (const T*)k, (const T*)v,
                                                      (const T*)krec, (const T*)vrec, gates, block_table, (T*)k_pages,
                                                      (T*)v_pages, (T*)out, scale_log2, err);
  };
  if (s.dtype == 1 && s.hd == 128) go(paged_decode_kernel<bf16, 128>, bf16());
  else if (s.dtype == 1 && s.hd == 64) go(paged_decode_kernel<bf16, 64>, bf16());
  else if (s.dtype == 0 && s.hd == 128) go(paged_decode_kernel<float, 128>, 0.f);
  else if (s.dtype == 0 && s.hd == 64) go(paged_decode_kernel<float, 64>, 0.f);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace maglev
