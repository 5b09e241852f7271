// 8-bit K/V cache: rows quantised as they are written, and read back.
//
// Both move each byte once and are bound by HBM at the sizes of a batched
// step, by launch latency below a few MB.  What would bind them otherwise is
// the number of instructions per element, so magnitudes are compared two at
// a time as 16-bit patterns, int8 codes come out of the mantissa of one fused
// multiply-add, and codes go to bf16 in pairs.
#include <cstring>

#include "spa_q8.cuh"

namespace spa {

// 16 consecutive elements in registers, as loaded.  mag: the largest
// magnitude of the finite ones as fp32 bits (bad is set by an infinity or a
// NaN); clean makes those 0.
template <typename T> struct Chunk16;
template <> struct Chunk16<__nv_bfloat16> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
  __device__ __forceinline__ uint32_t most() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m >> 16, m & 0xFFFFu) << 16;
  }
  __device__ __forceinline__ void clean() {
    if (most() < 0x7F800000u) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
      if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
    }
  }
  __device__ __forceinline__ uint32_t mag(bool& bad) {
    uint32_t m = most();
    if (m >= 0x7F800000u) {
      bad = true;
      clean();
      m = most();
    }
    return m;
  }
};
template <> struct Chunk16<float> {
  uint32_t w[16];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
    }
  }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(w[i]); }
  __device__ __forceinline__ uint32_t most() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ void clean() {
    if (most() < 0x7F800000u) return;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] = 0;
  }
  __device__ __forceinline__ uint32_t mag(bool& bad) {
    uint32_t m = most();
    if (m >= 0x7F800000u) {
      bad = true;
      clean();
      m = most();
    }
    return m;
  }
};

// Largest magnitude of codes: two running 16-bit maxima (int8: and minima).
template <int FMT> struct CodesMag {
  uint32_t hi = 0, lo = 0;
  // Adds 16 codes; keep: all ones, or 0 to leave them out.
  __device__ __forceinline__ void add(const uint4& c, uint32_t keep) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (FMT == kQ8E4m3) {  // the 7 low bits are ordered as the magnitudes
        hi = __vmaxu2(__vmaxu2(hi, w[i] & 0x007F007Fu & keep), (w[i] >> 8) & 0x007F007Fu & keep);
      } else {
        const uint32_t v = w[i] & keep;
        const uint32_t a = q8_pair<FMT>(v, v, 0, 1), b = q8_pair<FMT>(v, v, 2, 3);
        hi = __vmaxs2(hi, __vmaxs2(a, b));
        lo = __vmins2(lo, __vmins2(a, b));
      }
    }
  }
  __device__ __forceinline__ uint32_t get() const {
    if constexpr (FMT == kQ8E4m3) return max(hi >> 16, hi & 0xFFFFu);
    const int h = max((int)(int16_t)(hi & 0xFFFFu), (int)hi >> 16);
    const int l = min((int)(int16_t)(lo & 0xFFFFu), (int)lo >> 16);
    return (uint32_t)max(h, -l);
  }
};

// Codes of four values times inv (|value * inv| <= qmax): int8 from the
// mantissa of x inv + 1.5 2^23, which rounds to the nearest integer, ties to even.
template <int FMT> __device__ __forceinline__ uint32_t q8_encode4(const float (&x)[4], float inv) {
  if constexpr (FMT == kQ8Int8) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(fmaf(x[i], inv, 12582912.f));
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
  } else {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return a | (b << 16);
  }
}

// One CTA = one block of tokens and kQwWarps of its (head, K or V) items, a
// warp each (or one item, all warps, where that would leave SMs without
// work).  The CTA finds which of the block's rows are written (row map in
// shared memory: the last of equal indices wins, whatever their order); from
// there on no warp waits for another.  A warp takes the largest magnitude
// over the remaining rows' codes and over the new rows, and then reads the
// new rows again (from L1) and writes their codes; the remaining rows are
// read again and written only when the scale changes.  (One CTA per item,
// its rows in registers, spent five times the instructions: 104 against 46 us
// for 328 of 2048 rows, B = 8, 32 heads of 128.)
//
// The CTAs count the blocks (by_row = 0; one without a new row is left
// untouched), or, when there are fewer rows than blocks, the rows: the first
// row of a block takes it (one row in 65536 tokens x 8 heads, blocks of 128:
// 3.9 against 7.5 us; 64 rows 5.9 / 9.8).
constexpr int kQwWarps = 4, kQwThreads = kQwWarps * 32;
constexpr int kQwUnroll = 8;  // 16-byte loads in flight per lane

template <typename T, int FMT>
__global__ void __launch_bounds__(kQwThreads) q8_write_kernel(const Q8WriteParams p) {
  __shared__ int s_row[128];   // new row of the source, -1: a remaining row
  __shared__ int s_list[128];  // the block's new rows
  __shared__ int s_first, s_new;
  __shared__ uint32_t s_red[2][kQwWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.z;
  const int share = p.share, part = share ? warp : 0;  // share: the warps share one item
  const int item = share ? blockIdx.y : blockIdx.y * kQwWarps + warp, h = item >> 1, is_v = item & 1;
  const int32_t* ib = p.idx ? p.idx + (size_t)b * p.k : nullptr;
  int j = blockIdx.x;
  if (p.by_row) {
    const int r = __ldg(ib + blockIdx.x);
    if (r < 0 || r >= p.N) {
      if (blockIdx.y == 0 && tid == 0) report_error(p.err, DEVERR_INDEX, 701);
      return;
    }
    j = r >> p.block_log2;
  }
  const int r0 = j << p.block_log2, rows = min(1 << p.block_log2, p.N - r0);
  for (int i = tid; i < rows; i += kQwThreads) s_row[i] = (ib || r0 + i >= p.k) ? -1 : r0 + i;
  if (tid == 0) {
    s_first = 0x7FFFFFFF;
    s_new = 0;
  }
  __syncthreads();
  if (ib) {
    int first = 0x7FFFFFFF;
#pragma unroll 4
    for (int i = tid; i < p.k; i += kQwThreads) {
      const int r = __ldg(ib + i);
      if ((unsigned)(r - r0) < (unsigned)rows) {
        atomicMax(&s_row[r - r0], i);
        first = min(first, i);
      } else if (!p.by_row && (r < 0 || r >= p.N) && j == 0 && blockIdx.y == 0) {
        report_error(p.err, DEVERR_INDEX, 701);
      }
    }
    if (first != 0x7FFFFFFF) atomicMin(&s_first, first);
    __syncthreads();
    if (p.by_row ? s_first != (int)blockIdx.x : s_first == 0x7FFFFFFF) return;
  }
  for (int i = tid; i < rows; i += kQwThreads)
    if (s_row[i] >= 0) s_list[atomicAdd(&s_new, 1)] = i;  // their order does not matter
  __syncthreads();
  if (item >= 2 * p.n_kv) return;

  const int n_new = s_new, width = p.n_kv * p.hd;
  const int nb = (p.N + (1 << p.block_log2) - 1) >> p.block_log2;
  float* scale = (is_v ? p.v_scale : p.k_scale) + ((size_t)b * nb + j) * p.n_kv + h;
  const float s_old = *scale;
  // a lane's 16-element pieces: column `col` of rows row, row + step, ...
  const int cpr_log2 = p.hd_log2 - 4;
  const int row = (lane >> cpr_log2) + part * (32 >> cpr_log2), step = (32 >> cpr_log2) * (share ? kQwWarps : 1);
  const int col = (lane & ((1 << cpr_log2) - 1)) << 4;
  uint8_t* codes = (is_v ? p.v_codes : p.k_codes) + ((size_t)b * p.N + r0) * width + (size_t)h * p.hd + col;
  const T* src = reinterpret_cast<const T*>(is_v ? p.v_rows : p.k_rows) +
                 ((size_t)b * (p.indexed ? p.N : p.k) + (p.indexed ? r0 : 0)) * width + (size_t)h * p.hd + col;
  auto new_row = [&](int i) {  // of the source
    const int r = s_list[i];
    return src + (size_t)(p.indexed ? r : s_row[r]) * width;
  };

  CodesMag<FMT> old;
  if (n_new < rows) {
    for (int r = row; r < rows; r += kQwUnroll * step) {
      uint4 c[kQwUnroll];
#pragma unroll
      for (int q = 0; q < kQwUnroll; ++q)
        if (r + q * step < rows) c[q] = *reinterpret_cast<const uint4*>(codes + (size_t)(r + q * step) * width);
#pragma unroll
      for (int q = 0; q < kQwUnroll; ++q)
        if (r + q * step < rows) old.add(c[q], s_row[r + q * step] < 0 ? ~0u : 0u);
    }
  }
  uint32_t mag_new = 0;
  bool bad = false;
  for (int i = row; i < n_new; i += 4 * step) {
    Chunk16<T> x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q * step < n_new) x[q].load(new_row(i + q * step));
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q * step < n_new) mag_new = max(mag_new, x[q].mag(bad));
  }
  if (bad) report_error(p.err, DEVERR_VALUE, 702);
  mag_new = __reduce_max_sync(0xffffffffu, mag_new);
  uint32_t mag_old = __reduce_max_sync(0xffffffffu, old.get());
  if (share) {
    if (lane == 0) {
      s_red[0][warp] = mag_new;
      s_red[1][warp] = mag_old;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQwWarps; ++w) {
      mag_new = max(mag_new, s_red[0][w]);
      mag_old = max(mag_old, s_red[1][w]);
    }
  }
  const float s = q8_scale<FMT>(fmaxf(__uint_as_float(mag_new), s_old != 0.f ? q8_value<FMT>(mag_old) * s_old : 0.f));
  if (lane == 0 && part == 0) *scale = s;  // every thread has read s_old before the reduction above
  const float inv = s > 0.f ? q8_inverse(s) : 0.f;
  for (int i = row; i < n_new; i += 2 * step) {
    Chunk16<T> x[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (i + q * step < n_new) x[q].load(new_row(i + q * step));
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (i + q * step >= n_new) continue;
      x[q].clean();
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v[4] = {x[q].get(4 * e), x[q].get(4 * e + 1), x[q].get(4 * e + 2), x[q].get(4 * e + 3)};
        o[e] = q8_encode4<FMT>(v, inv);
      }
      *reinterpret_cast<uint4*>(codes + (size_t)s_list[i + q * step] * width) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (s == s_old || n_new == rows) return;
#pragma unroll 1
  for (int r = row; r < rows; r += step) {
    if (s_row[r] >= 0) continue;
    uint4* at = reinterpret_cast<uint4*>(codes + (size_t)r * width);
    const uint4 c = *at;
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = s_old != 0.f ? q8_value<FMT>((w[i] >> (8 * e)) & 0xFFu) * s_old : 0.f;
      o[i] = q8_encode4<FMT>(v, inv);
    }
    *at = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// 32 bytes at a 32-byte aligned address (wide), or at a 16-byte aligned one.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// One CTA = one output row of one sequence's K or V (or as many as its 256
// threads cover), 16 codes a thread, written as whole sectors.  2 x 134 M
// codes to bf16 (402 MB): 64 us; with two 16-byte stores 68, with four chunks
// a thread 78 us: many small CTAs keep the stores of one and the loads of the
// next apart.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) q8_read_kernel(const Q8ReadParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int width = p.n_kv * p.hd, cpr = width >> 4;
  const int tpr = min(cpr, 256), rps = 256 / tpr, sub = threadIdx.x / tpr;
  const int is_v = blockIdx.y & 1, b = blockIdx.y >> 1;
  const int i = blockIdx.x * rps + sub;
  if (sub >= rps || i >= p.k) return;
  const int r = p.idx ? __ldg(p.idx + (size_t)b * p.k + i) : i;
  if (r < 0 || r >= p.N) {
    report_error(p.err, DEVERR_INDEX, 703);
    return;
  }
  const int nb = (p.N + (1 << p.block_log2) - 1) >> p.block_log2;
  const uint8_t* codes = (is_v ? p.v_codes : p.k_codes) + ((size_t)b * p.N + r) * width;
  const float* scale = (is_v ? p.v_scale : p.k_scale) + ((size_t)b * nb + (r >> p.block_log2)) * p.n_kv;
  T* out = reinterpret_cast<T*>(is_v ? p.v_out : p.k_out) + ((size_t)b * p.k + i) * width;
  for (int c = threadIdx.x - sub * tpr; c < cpr; c += tpr) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(codes) + c);
    const float s = __ldg(scale + (c >> (p.hd_log2 - 4)));
    uint32_t v[8];
    q8_word_to_bf16<FMT>(w.x, v[0], v[1]);
    q8_word_to_bf16<FMT>(w.y, v[2], v[3]);
    q8_word_to_bf16<FMT>(w.z, v[4], v[5]);
    q8_word_to_bf16<FMT>(w.w, v[6], v[7]);
    if constexpr (sizeof(T) == 2) {
      if ((__float_as_uint(s) & 0xFFFFu) == 0) {
        // the scale is a bf16: the product rounds once, as from fp32
        const __nv_bfloat162 sb = __float2bfloat162_rn(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 t = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v[e]), sb);
          v[e] = *reinterpret_cast<const uint32_t*>(&t);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 t =
              __floats2bfloat162_rn(__uint_as_float(v[e] << 16) * s, __uint_as_float(v[e] & 0xFFFF0000u) * s);
          v[e] = *reinterpret_cast<const uint32_t*>(&t);
        }
      }
      store32(out + (size_t)c * 16, v, p.wide);
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[2 * e] = __float_as_uint(__uint_as_float(v[4 * half + e] << 16) * s);
          f[2 * e + 1] = __float_as_uint(__uint_as_float(v[4 * half + e] & 0xFFFF0000u) * s);
        }
        store32(out + (size_t)c * 16 + 8 * half, f, p.wide);
      }
    }
  }
}

static int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

cudaError_t launch_q8_write(int dtype, int fmt, int block, Q8WriteParams p, int num_sms, cudaStream_t stream) {
  p.block_log2 = log2_of(block);
  p.hd_log2 = log2_of(p.hd);
  const int nb = (p.N + block - 1) / block;
  p.by_row = p.idx && p.k < nb;
  const int blocks = p.by_row ? p.k : p.idx ? nb : (p.k + block - 1) / block;
  // Fewer items than eight warps on each SM: all warps on one item.  A fill
  // of 1024 x 32 x 128 (1024 items): 6.3 against 13.5 us.
  p.share = (long long)blocks * 2 * p.n_kv * p.B < 8LL * num_sms;
  const dim3 grid(blocks, p.share ? 2 * p.n_kv : (2 * p.n_kv + kQwWarps - 1) / kQwWarps, p.B);
  if (dtype == 1)
    return fmt == kQ8Int8 ? launch_k(q8_write_kernel<__nv_bfloat16, kQ8Int8>, grid, dim3(kQwThreads), 0, stream, p)
                          : launch_k(q8_write_kernel<__nv_bfloat16, kQ8E4m3>, grid, dim3(kQwThreads), 0, stream, p);
  return fmt == kQ8Int8 ? launch_k(q8_write_kernel<float, kQ8Int8>, grid, dim3(kQwThreads), 0, stream, p)
                        : launch_k(q8_write_kernel<float, kQ8E4m3>, grid, dim3(kQwThreads), 0, stream, p);
}

cudaError_t launch_q8_read(int dtype, int fmt, int block, Q8ReadParams p, cudaStream_t stream) {
  p.block_log2 = log2_of(block);
  p.hd_log2 = log2_of(p.hd);
  const int cpr = p.n_kv * p.hd / 16, rps = 256 / (cpr < 256 ? cpr : 256);
  p.wide = (reinterpret_cast<uintptr_t>(p.k_out) | reinterpret_cast<uintptr_t>(p.v_out)) % 32 == 0;
  const dim3 grid((p.k + rps - 1) / rps, 2 * p.B);
  if (dtype == 1)
    return fmt == kQ8Int8 ? launch_k(q8_read_kernel<__nv_bfloat16, kQ8Int8>, grid, dim3(256), 0, stream, p)
                          : launch_k(q8_read_kernel<__nv_bfloat16, kQ8E4m3>, grid, dim3(256), 0, stream, p);
  return fmt == kQ8Int8 ? launch_k(q8_read_kernel<float, kQ8Int8>, grid, dim3(256), 0, stream, p)
                        : launch_k(q8_read_kernel<float, kQ8E4m3>, grid, dim3(256), 0, stream, p);
}

}  // namespace spa
