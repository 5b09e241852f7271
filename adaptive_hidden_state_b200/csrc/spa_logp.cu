// Log probabilities of given tokens with the entropy and the most likely
// alternatives of each row of logits, in one pass over the logits.
//
// Per row, with m = max x: S = sum e^(x-m), T = sum e^(x-m) (x-m), both kept
// in fp32 by every thread against its own running maximum and re-scaled when
// that grows; log p(i) = (x_i - m) - log S and H = log S - T / S, a sum of two
// terms that are never negative, so a sharp row loses nothing by cancellation.
//
// The `top` largest: each warp keeps its best 32 in order, one per lane.  An
// element enters only if it beats the warp's `top`-th best; a thread first
// compares the maximum of its whole tile, and the warps share the best such
// bound, so nearly every tile is passed by one comparison.  The order (larger
// value, then lower id) is total, so the result depends on no timing.
//
// Bound by HBM: 4 or 2 bytes per logit.  A row is read by a cluster of 1 to 8
// CTAs, whose statistics and lists meet in distributed shared memory: no
// scratch, no second launch.
#include "spa_device.cuh"

namespace spa {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpUnroll = 4;  // 16-byte loads in flight per thread
constexpr float kLog2e = 1.4426950408889634f;

struct LpStat {
  float m, s, t;
};
// Sum of two partial statistics against the larger maximum.  A part without
// elements (m = -inf, s = 0) adds nothing; NaN sums stay NaN.
__device__ __forceinline__ LpStat lp_merge(const LpStat& a, const LpStat& b) {
  LpStat r;
  r.m = fmaxf(a.m, b.m);
  const float ref = r.m == -INFINITY ? 0.f : r.m;
  const float fa = exp2f((a.m - ref) * kLog2e), fb = exp2f((b.m - ref) * kLog2e);
  // e^(m_a - m) is 0 long before the difference reaches the clamp
  const float da = fmaxf(a.m - ref, -1e4f), db = fmaxf(b.m - ref, -1e4f);
  r.s = fa * a.s + fb * b.s;
  r.t = fa * (a.t + a.s * da) + fb * (b.t + b.s * db);
  return r;
}

// Order-preserving map of floats to signed integers (for atomicMax).
__device__ __forceinline__ int lp_key(float v) {
  const int u = __float_as_int(v);
  return u ^ ((u >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float lp_unkey(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

__device__ __forceinline__ bool lp_better(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

// A warp's ordered list (lane i holds the i-th best) and its `top`-th entry.
struct LpList {
  float v = -INFINITY, tv = -INFINITY;
  int i = 0x7FFFFFFF, ti = 0x7FFFFFFF;
  __device__ __forceinline__ void insert(float cv, int ci, int top, int lane) {
    const int pos = __popc(__ballot_sync(0xffffffffu, lp_better(v, i, cv, ci)));
    const float uv = __shfl_up_sync(0xffffffffu, v, 1);
    const int ui = __shfl_up_sync(0xffffffffu, i, 1);
    if (lane > pos) { v = uv; i = ui; }
    if (lane == pos) { v = cv; i = ci; }
    tv = __shfl_sync(0xffffffffu, v, top - 1);
    ti = __shfl_sync(0xffffffffu, i, top - 1);
  }
  // Every lane's candidate (where `is` holds), in lane order.
  __device__ __forceinline__ void offer(bool is, float cv, int ci, int top, int lane) {
    uint32_t mask = __ballot_sync(0xffffffffu, is && lp_better(cv, ci, tv, ti));
    while (mask) {
      const int src = __ffs(mask) - 1;
      mask &= mask - 1;
      const float sv = __shfl_sync(0xffffffffu, cv, src);
      const int si = __shfl_sync(0xffffffffu, ci, src);
      if (lp_better(sv, si, tv, ti)) insert(sv, si, top, lane);
    }
  }
};

template <typename T> struct LpVec;
template <> struct LpVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
  }
};
template <> struct LpVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};

// NE elements per thread (absent ones -inf): id(i) is element i's column,
// ascending in i.
template <int NE, typename IdFn>
__device__ __forceinline__ void lp_tile(const float (&x)[NE], IdFn id, LpStat& st, LpList& list, int* s_cut,
                                        int top, int lane) {
  float tm = x[0];
#pragma unroll
  for (int i = 1; i < NE; ++i) tm = fmaxf(tm, x[i]);
  if (tm > st.m) {
    const LpStat none = {tm, 0.f, 0.f};
    st = lp_merge(st, none);
  }
  const float ref = st.m == -INFINITY ? 0.f : st.m;
  float s = 0.f, t = 0.f;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const float d = x[i] - ref, e = exp2f(d * kLog2e);
    s += e;
    t = fmaf(e, fmaxf(d, -1e4f), t);
  }
  st.s += s;
  st.t += t;
  if (top == 0) return;
  float cut = lp_unkey(*reinterpret_cast<volatile int*>(s_cut));
  const bool maybe = tm >= cut && tm > -INFINITY && lp_better(tm, id(0), list.tv, list.ti);
  if (!__any_sync(0xffffffffu, maybe)) return;
  if (list.tv == -INFINITY) {
    // a bound for a list that is not full yet: the top-th largest of the lanes' maxima
    int rank = 0;
#pragma unroll
    for (int q = 0; q < 32; ++q) {
      const float o = __shfl_sync(0xffffffffu, tm, q);
      rank += o > tm || (o == tm && q < lane);
    }
    const uint32_t at = __ballot_sync(0xffffffffu, rank == top - 1);
    if (at) cut = fmaxf(cut, __shfl_sync(0xffffffffu, tm, __ffs(at) - 1));
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) list.offer(x[i] >= cut && x[i] > -INFINITY, x[i], id(i), top, lane);
  if (lane == 0 && list.tv > cut) atomicMax(s_cut, lp_key(list.tv));
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logp_kernel(const LogpParams p, int C) {
  constexpr int VN = LpVec<T>::N;
  __shared__ float s_stat[kLpWarps][3];
  __shared__ float s_lv[kLpWarps][32];
  __shared__ int s_li[kLpWarps][32];
  __shared__ float s_out[3];  // this CTA's statistics and list, read by the cluster's first CTA
  __shared__ float s_ov[32];
  __shared__ int s_oi[32];
  __shared__ int s_cut;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)(blockIdx.x % C);
  const long long row = blockIdx.x / C;
  if (tid == 0) s_cut = lp_key(-INFINITY);
  __syncthreads();
  const T* x = reinterpret_cast<const T*>(p.logits) + row * p.ld;
  const int top = p.top;
  // whole 16-byte vectors, and the elements before and after them
  const int mis = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int head = min(mis ? VN - mis : 0, p.V);
  const int nv = (p.V - head) / VN, tail0 = head + nv * VN;
  const int v0 = (int)((long long)nv * rank / C), v1 = (int)((long long)nv * (rank + 1) / C);
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);

  LpStat st = {-INFINITY, 0.f, 0.f};
  LpList list;
  if (rank == 0 && head) {
    const float v[1] = {tid < head ? to_f(x[tid]) : -INFINITY};
    if (warp == 0) lp_tile<1>(v, [&](int) { return tid; }, st, list, &s_cut, top, lane);
  }
  for (int b0 = v0; b0 < v1; b0 += kLpThreads * kLpUnroll) {
    uint4 w[kLpUnroll];
    float v[kLpUnroll * VN];
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      const int i = b0 + u * kLpThreads + tid;
      if (i < v1) w[u] = __ldg(xv + i);
    }
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
      if (b0 + u * kLpThreads + tid < v1) {
        LpVec<T>::unpack(w[u], v + u * VN);
      } else {
#pragma unroll
        for (int e = 0; e < VN; ++e) v[u * VN + e] = -INFINITY;
      }
    }
    const int first = head + (b0 + tid) * VN;
    lp_tile<kLpUnroll * VN>(v, [&](int i) { return first + (i / VN) * kLpThreads * VN + i % VN; }, st, list,
                            &s_cut, top, lane);
  }
  if (rank == C - 1 && tail0 < p.V) {
    const float v[1] = {tail0 + tid < p.V ? to_f(x[tail0 + tid]) : -INFINITY};
    if (warp == 0) lp_tile<1>(v, [&](int) { return tail0 + tid; }, st, list, &s_cut, top, lane);
  }

  // lanes, warps, CTAs of the cluster, each in a fixed order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    LpStat b;
    b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, st.t, o);
    st = lp_merge(st, b);
  }
  if (lane == 0) {
    s_stat[warp][0] = st.m; s_stat[warp][1] = st.s; s_stat[warp][2] = st.t;
  }
  s_lv[warp][lane] = list.v;
  s_li[warp][lane] = list.i;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < kLpWarps; ++w) {
      const LpStat b = {s_stat[w][0], s_stat[w][1], s_stat[w][2]};
      st = lp_merge(st, b);
      if (top) list.offer(lane < top && s_lv[w][lane] > -INFINITY, s_lv[w][lane], s_li[w][lane], top, lane);
    }
    if (lane == 0) { s_out[0] = st.m; s_out[1] = st.s; s_out[2] = st.t; }
    s_ov[lane] = list.v;
    s_oi[lane] = list.i;
  }
  if (C > 1) {
    cluster_sync();
    if (rank == 0 && warp == 0) {
      for (int q = 1; q < C; ++q) {
        LpStat b;
        b.m = ld_dsmem_f32(mapa_shared(smem_u32(&s_out[0]), q));
        b.s = ld_dsmem_f32(mapa_shared(smem_u32(&s_out[1]), q));
        b.t = ld_dsmem_f32(mapa_shared(smem_u32(&s_out[2]), q));
        const float cv = ld_dsmem_f32(mapa_shared(smem_u32(&s_ov[lane]), q));
        const int ci = __float_as_int(ld_dsmem_f32(mapa_shared(smem_u32(&s_oi[lane]), q)));
        st = lp_merge(st, b);
        if (top) list.offer(lane < top && cv > -INFINITY, cv, ci, top, lane);
      }
    }
  }
  if (rank == 0 && warp == 0) {
    const bool none = st.m == -INFINITY && st.s == 0.f;  // every logit is -inf
    const float logS = logf(st.s);
    if (lane == 0) {
      const int tok = p.tok[row];
      float lp = __int_as_float(0x7FC00000);
      if (tok < 0 || tok >= p.V) report_error(p.err, DEVERR_INDEX, 721);
      else lp = none ? -INFINITY : (to_f(x[tok]) - st.m) - logS;
      p.logp[row] = lp;
      p.entropy[row] = none ? 0.f : logS - st.t / st.s;
    }
    if (lane < top) {
      const bool has = list.v > -INFINITY;
      p.top_id[row * top + lane] = has ? list.i : -1;
      p.top_logp[row * top + lane] = has ? (list.v - st.m) - logS : -INFINITY;
    }
  }
  if (C > 1) cluster_sync();  // the other CTAs' shared memory stays until it has been read
}

cudaError_t launch_token_logprobs(int dtype, const LogpParams& p, int rows, int num_sms, cudaStream_t stream) {
  int C = 1;
  while (C < 8 && (long long)rows * C < 4LL * num_sms && p.V / (2 * C) >= 4096) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * C);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return dtype == 1 ? cudaLaunchKernelEx(&cfg, logp_kernel<__nv_bfloat16>, p, C)
                    : cudaLaunchKernelEx(&cfg, logp_kernel<float>, p, C);
}

}  // namespace spa
