// 8-bit K/V cache: rows quantised as they are written, and read back.
//
// Both move each byte once and are bound by HBM at the sizes of a fill or of
// a batched step, by launch latency below a few MB.
#include <cstring>

#include "spa_q8.cuh"

namespace spa {

constexpr int kQwThreads = 256;
constexpr int kQwChunks = 4;  // 16-element chunks a thread holds: 128 rows x 128 elements / 16 / 256

template <typename T> struct Chunk16;  // 16 consecutive elements in registers, as loaded
template <> struct Chunk16<__nv_bfloat16> {
  uint4 r[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r[0] = __ldg(reinterpret_cast<const uint4*>(p));
    r[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(r);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
};
template <> struct Chunk16<float> {
  float4 r[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ float get(int i) const { return reinterpret_cast<const float*>(r)[i]; }
};

// One CTA = one block of tokens of one head of K or of V.  It finds which of
// the block's rows are written (row map in shared memory: the last of equal
// indices wins, whatever their order), holds the new rows and the remaining
// rows' codes in registers, takes the largest magnitude, and writes the new
// codes; the remaining rows are written only when the scale changes.  A block
// that gets no row is left untouched.
template <typename T, int FMT>
__global__ void __launch_bounds__(kQwThreads) q8_write_kernel(const Q8WriteParams p) {
  __shared__ int s_row[128];
  __shared__ int s_any;
  __shared__ float s_red[kQwThreads / 32];
  __shared__ float s_amax;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, nthr = blockDim.x;
  const int j = blockIdx.x, h = blockIdx.y >> 1, is_v = blockIdx.y & 1, b = blockIdx.z;
  const int r0 = j * p.block, rows = min(p.block, p.N - r0);
  const size_t width = (size_t)p.n_kv * p.hd;
  for (int i = tid; i < rows; i += nthr) s_row[i] = (p.idx || r0 + i >= p.k) ? -1 : r0 + i;
  if (tid == 0) s_any = 0;
  __syncthreads();
  if (p.idx) {
    const int32_t* ib = p.idx + (size_t)b * p.k;
    bool any = false;
    for (int i = tid; i < p.k; i += nthr) {
      const int r = __ldg(ib + i);
      if ((unsigned)(r - r0) < (unsigned)rows) {
        atomicMax(&s_row[r - r0], i);
        any = true;
      } else if ((r < 0 || r >= p.N) && j == 0 && blockIdx.y == 0) {
        report_error(p.err, DEVERR_INDEX, 701);
      }
    }
    if (any) s_any = 1;
    __syncthreads();
    if (!s_any) return;
  } else if (r0 >= p.k) {
    return;
  }
  const T* src = reinterpret_cast<const T*>(is_v ? p.v_rows : p.k_rows);
  uint8_t* codes = (is_v ? p.v_codes : p.k_codes) + ((size_t)b * p.N + r0) * width + (size_t)h * p.hd;
  float* scale = (is_v ? p.v_scale : p.k_scale) + ((size_t)b * gridDim.x + j) * p.n_kv + h;
  const float s_old = *scale;
  const int cpr = p.hd / 16, total = rows * cpr;
  const size_t src_rows = p.indexed ? (size_t)p.N : (size_t)p.k;

  Chunk16<T> x[kQwChunks];
  int from[kQwChunks];  // source row, -1: a remaining row (its codes in x), -2: nothing
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int q = 0; q < kQwChunks; ++q) {
    const int c = tid + q * nthr;
    from[q] = -2;
    if (c < total) {
      const int r = c / cpr, col = (c % cpr) * 16;
      from[q] = s_row[r];
      if (from[q] >= 0) {
        const size_t sr = (size_t)b * src_rows + (p.indexed ? r0 + r : from[q]);
        x[q].load(src + sr * width + (size_t)h * p.hd + col);
      } else {
        *reinterpret_cast<uint4*>(x[q].r) = *reinterpret_cast<const uint4*>(codes + (size_t)r * width + col);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kQwChunks; ++q) {
    if (from[q] >= 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float a = fabsf(x[q].get(i));
        if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
        else bad = true;
      }
    } else if (from[q] == -1 && s_old != 0.f) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(x[q].r);
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(q8_value<FMT>((w[i >> 2] >> (8 * (i & 3))) & 0xFFu)));
      amax = fmaxf(amax, m * s_old);
    }
  }
  if (bad) report_error(p.err, DEVERR_VALUE, 702);
  amax = warp_max(amax);
  if ((tid & 31) == 0) s_red[tid >> 5] = amax;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < nthr / 32; ++w) amax = fmaxf(amax, s_red[w]);
    s_amax = amax;
    *scale = q8_scale<FMT>(amax);  // every thread has read s_old before the barrier above
  }
  __syncthreads();
  const float s = q8_scale<FMT>(s_amax);
  const float inv = s > 0.f ? q8_inverse(s) : 0.f;
#pragma unroll
  for (int q = 0; q < kQwChunks; ++q) {
    if (from[q] == -2 || (from[q] == -1 && s == s_old)) continue;
    const int c = tid + q * nthr;
    float v[16];
    if (from[q] >= 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float a = x[q].get(i);
        v[i] = fabsf(a) <= 3.402823466e38f ? a * inv : 0.f;
      }
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(x[q].r);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = s_old != 0.f ? q8_value<FMT>((w[i >> 2] >> (8 * (i & 3))) & 0xFFu) * s_old * inv : 0.f;
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = q8_encode2<FMT>(v[4 * i], v[4 * i + 1]) | (q8_encode2<FMT>(v[4 * i + 2], v[4 * i + 3]) << 16);
    *reinterpret_cast<uint4*>(codes + (size_t)(c / cpr) * width + (c % cpr) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// One thread = 16 codes of one row of K or of V.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) q8_read_kernel(const Q8ReadParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int width = p.n_kv * p.hd, cpr = width / 16;
  const long long total = (long long)p.B * p.k * cpr;
  const int is_v = blockIdx.y;
  const int nb = (p.N + p.block - 1) / p.block;
  const long long c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= total) return;
  const long long t = c / cpr;
  const int col = (int)(c - t * cpr) * 16;
  const long long b = t / p.k;
  const int i = (int)(t - b * p.k);
  const int r = p.idx ? __ldg(p.idx + t) : i;
  if (r < 0 || r >= p.N) {
    report_error(p.err, DEVERR_INDEX, 703);
    return;
  }
  const uint8_t* codes = (is_v ? p.v_codes : p.k_codes) + ((size_t)b * p.N + r) * width + col;
  const float s = __ldg((is_v ? p.v_scale : p.k_scale) + ((size_t)b * nb + r / p.block) * p.n_kv + col / p.hd);
  const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(codes));
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  T* out = reinterpret_cast<T*>(is_v ? p.v_out : p.k_out) + (size_t)t * width + col;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float4 v;
    v.x = s != 0.f ? q8_value<FMT>(w[q] & 0xFFu) * s : 0.f;
    v.y = s != 0.f ? q8_value<FMT>((w[q] >> 8) & 0xFFu) * s : 0.f;
    v.z = s != 0.f ? q8_value<FMT>((w[q] >> 16) & 0xFFu) * s : 0.f;
    v.w = s != 0.f ? q8_value<FMT>(w[q] >> 24) * s : 0.f;
    store4(out + 4 * q, v);
  }
}

cudaError_t launch_q8_write(int dtype, int fmt, const Q8WriteParams& p, cudaStream_t stream) {
  const int chunks = p.block * p.hd / 16;  // <= kQwThreads * kQwChunks
  const int threads = chunks >= kQwThreads ? kQwThreads : (chunks + 31) / 32 * 32;
  const dim3 grid((p.N + p.block - 1) / p.block, 2 * p.n_kv, p.B);
  if (dtype == 1)
    return fmt == kQ8Int8 ? launch_k(q8_write_kernel<__nv_bfloat16, kQ8Int8>, grid, dim3(threads), 0, stream, p)
                          : launch_k(q8_write_kernel<__nv_bfloat16, kQ8E4m3>, grid, dim3(threads), 0, stream, p);
  return fmt == kQ8Int8 ? launch_k(q8_write_kernel<float, kQ8Int8>, grid, dim3(threads), 0, stream, p)
                        : launch_k(q8_write_kernel<float, kQ8E4m3>, grid, dim3(threads), 0, stream, p);
}

cudaError_t launch_q8_read(int dtype, int fmt, const Q8ReadParams& p, cudaStream_t stream) {
  const long long chunks = (long long)p.B * p.k * (p.n_kv * p.hd / 16);
  const dim3 grid((unsigned)((chunks + 255) / 256), 2);
  if (dtype == 1)
    return fmt == kQ8Int8 ? launch_k(q8_read_kernel<__nv_bfloat16, kQ8Int8>, grid, dim3(256), 0, stream, p)
                          : launch_k(q8_read_kernel<__nv_bfloat16, kQ8E4m3>, grid, dim3(256), 0, stream, p);
  return fmt == kQ8Int8 ? launch_k(q8_read_kernel<float, kQ8Int8>, grid, dim3(256), 0, stream, p)
                        : launch_k(q8_read_kernel<float, kQ8E4m3>, grid, dim3(256), 0, stream, p);
}

}  // namespace spa
