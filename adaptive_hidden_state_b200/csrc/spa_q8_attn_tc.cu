// Tensor-core attention over the 8-bit K/V cache (tcgen05, TMEM), bf16
// queries, head_dim 64 or 128: the kernel for many query rows of a kv head.
//
// One CTA = one or two tiles of 128 query rows of one kv head of one
// sequence, and one contiguous share of its keys, in tiles of 128:
//   warps 0-3, 4-7  softmax of the first and second query tile: thread i owns
//                   row i (TMEM lane i)
//   next 4 warps    conversion: codes go from global memory through registers
//                   (the next tile's loads are in flight while this one is
//                   converted) to bf16 tiles in shared memory, in the swizzled
//                   layout the MMA reads; the block's scale, a power of two, is
//                   multiplied in there, exactly, so the softmax sees plain
//                   keys and values and both query tiles share the work
//   last warp       one thread issues the MMAs: for each key tile and query
//                   tile S = Q K^T (fp32, TMEM), and once the softmax warps
//                   have written P (bf16) over S in TMEM, O += P V with P as
//                   the TMEM operand, so P never touches shared memory
// The order PV0(j-1), QK0(j), PV1(j-1), QK1(j) keeps the tensor core on one
// query tile while the other's softmax runs.  MMAs of one thread execute in
// order, so QK_i(j) overwrites P_i(j-1) after PV_i(j-1) has read it, and the
// commit after QK_i(j) that hands S_i to the softmax also says that O_i is
// complete up to j - 1 and may be re-scaled.
//
// The running maximum is lazy: O is re-scaled only when it grows by more than
// 2^8 (the result is exact for any reference).  Key shares of a query tile
// form a cluster and are joined through distributed shared memory in share
// order, so the result does not depend on timing.
#include <cstring>

#include "spa_q8.cuh"

namespace spa {

constexpr int kTT = 128;                 // query rows of a tile, keys of a tile
constexpr float kTRescale = 8.0f;

template <int HD, int NQ> struct TcCfg {
  static constexpr int kQBytes = kTT * HD * 2;        // one query tile
  static constexpr int kTile = kTT * HD * 2;          // one bf16 K or V tile
  static constexpr int kStages = 2;                   // K ring, V ring
  static constexpr int kThreads = NQ * 128 + 128 + 32;
  static constexpr int kUsed = NQ * kQBytes + 2 * kStages * kTile + 1024;
  // at least 120 KB, so that no SM holds two CTAs that want its tensor memory
  static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
};

struct TcSync {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_done;
  uint32_t tmem;
  int abort, ok;
};

__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) | ((uint64_t)64 << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D[tmem] (+)= A[tmem] * B[smem]: A bf16 pairs in 32-bit columns, K-major.
__device__ __forceinline__ void umma_bf16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  const uint32_t z = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(z), "r"(z), "r"(z), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 codes -> 16 bf16 values times the scale (a power of two or 0: exact).
template <int FMT>
__device__ __forceinline__ void convert16(const uint4& w4, float scale, uint4& lo, uint4& hi) {
  const __nv_bfloat162 sc = __float2bfloat162_rn(scale);
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t t = q8_to_bf162_lo<FMT>(__byte_perm(w[i >> 1], 0, i & 1 ? 0x4342 : 0x4140));
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&t), sc);
    o[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int HD, int FMT, int NQ>
__global__ void __launch_bounds__(TcCfg<HD, NQ>::kThreads, 1) q8_attn_tc_kernel(const Q8AttnParams p) {
  using Cfg = TcCfg<HD, NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + NQ * Cfg::kQBytes;
  uint8_t* sV = sK + Cfg::kStages * Cfg::kTile;
  __shared__ __align__(8) TcSync sy;
  __shared__ float s_m[NQ * kTT], s_l[NQ * kTT];
  __shared__ float s_w[NQ * kTT][8];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kConvWarp = NQ * 4, kMmaWarp = NQ * 4 + 4;
  const int S = p.splits, sp = blockIdx.x % S, h = blockIdx.y, b = blockIdx.z;
  const int row0 = (blockIdx.x / S) * NQ * kTT;  // first query row of this CTA
  const int R = p.k * p.group;
  int* err = p.err;

  if (tid == 0) {
    mbar_init(&sy.q_full, NQ * 128);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sy.k_full[s], 128);
      mbar_init(&sy.k_empty[s], 1);
      mbar_init(&sy.v_full[s], 128);
      mbar_init(&sy.v_empty[s], 1);
      mbar_init(&sy.s_full[s], 1);
      mbar_init(&sy.p_full[s], 128);
    }
    mbar_init(&sy.o_done, 1);
    sy.abort = 0;
    sy.ok = 1;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sy.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();  // the next kernel comes to this SM after the tensor memory has been taken
  const uint32_t tmem = sy.tmem;  // S_i (P_i over it) at columns 128 i, O_i at 256 + 128 i
  griddep_wait();
  int len = p.N;
  if (p.lens) {
    len = __ldg(p.lens + b);
    if (len < 0 || len > p.N) {
      if (tid == 0) report_error(err, DEVERR_INDEX, 731);
      len = min(max(len, 0), p.N);
    }
  }
  const int n_kt = (len + kTT - 1) / kTT;
  const int kt0 = (int)((long long)sp * n_kt / S), kt1 = (int)((long long)(sp + 1) * n_kt / S);
  const int n = kt1 - kt0;  // key tiles of this CTA (may be none)

  if (warp < kConvWarp) {
    // ------------------------------------------------------------ softmax
    const int i = warp >> 2, row = (warp & 3) * 32 + lane;
    // Q rows of this tile, 2 (HD = 128) or 4 per instruction of a warp
    {
      constexpr int CPR = HD / 8;  // 16-byte pieces of a row
      uint8_t* dst = sQ + i * Cfg::kQBytes;
#pragma unroll 8
      for (int it = 0; it < CPR; ++it) {
        const int r = (warp & 3) * 32 + it * (32 / CPR) + lane / CPR, c = lane % CPR;
        const int qr = row0 + i * kTT + r;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (qr < R) {
          const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(p.Q) +
                                     (((size_t)b * p.k + qr / p.group) * p.n_heads + (size_t)h * p.group + qr % p.group) * HD;
          v = __ldg(reinterpret_cast<const uint4*>(src) + c);
        }
        *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
      }
      proxy_fence_smem();
      mbar_arrive_cta(&sy.q_full);
    }
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_base = lane_base + (uint32_t)(i * 128), o_base = lane_base + 256u + (uint32_t)(i * 128);
    const float c = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const bool got = mbar_wait(&sy.s_full[i], j & 1, &sy.abort, err, 732);
      __syncwarp();
      if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
      tc_fence_after();
      const int left = len - (kt0 + j) * kTT;  // keys of this tile that count
      float tmax = -INFINITY;
#pragma unroll 1
      for (int c0 = 0; c0 < kTT; c0 += 32) {
        float x[32];
        tmem_ld32(s_base + (uint32_t)c0, x);
        if (left < c0 + 32) {
#pragma unroll
          for (int q = 0; q < 32; ++q) x[q] = c0 + q < left ? x[q] : -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < 32; q += 2) tmax = max3(tmax, x[q], x[q + 1]);
      }
      tmax *= c;
      if (j == 0) {
        m = tmax;
      } else if (__any_sync(0xffffffffu, tmax > m + kTRescale)) {
        // some row's maximum grew by more than 2^8: the warp re-scales
        const float m_new = fmaxf(m, tmax), f = exp2f(m - m_new);
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 16) {
          uint32_t o[16];
          asm volatile(
              "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
              "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
              : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]),
                "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
              : "r"(o_base + (uint32_t)c0));
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
          tmem_st16(o_base + (uint32_t)c0, o);
        }
        l *= f;
        m = m_new;
      }
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int c0 = 0; c0 < kTT; c0 += 32) {
        float x[32];
        uint32_t w[16];
        tmem_ld32(s_base + (uint32_t)c0, x);
        if (left < c0 + 32) {
#pragma unroll
          for (int q = 0; q < 32; ++q) x[q] = c0 + q < left ? x[q] : -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < 32; q += 2) {
          const float2 y = fma2(make_float2(x[q], x[q + 1]), make_float2(c, c), make_float2(-m, -m));
          const float2 e = make_float2(ex2(y.x), ex2(y.y));
          sum = add2(sum, e);
          const __nv_bfloat162 v = __floats2bfloat162_rn(e.x, e.y);
          w[q >> 1] = *reinterpret_cast<const uint32_t*>(&v);
        }
        tmem_st16(s_base + (uint32_t)(c0 >> 1), w);  // over scores this thread has read
      }
      l += sum.x + sum.y;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_cta(&sy.p_full[i]);
    }
    const bool fin = ok && mbar_wait(&sy.o_done, 0, &sy.abort, err, 733);
    __syncwarp();
    const bool warp_ok = __all_sync(0xffffffffu, fin);
    if (lane == 0 && !warp_ok) atomicAnd(&sy.ok, 0);
    // the tiles' softmax warps agree, and no MMA reads the rings any more
    named_bar_sync(1, NQ * 128);
    if (sy.ok) {
      tc_fence_after();
      const int qr = row0 + i * kTT + row;
      const float inv = l != 0.f ? 1.0f / l : 0.f;
      __nv_bfloat16* dst = nullptr;
      if (S == 1 && qr < R)
        dst = reinterpret_cast<__nv_bfloat16*>(p.O) +
              (((size_t)b * p.k + qr / p.group) * p.n_heads + (size_t)h * p.group + qr % p.group) * HD;
      // key shares: the unnormalised row into the idle rings, 16-byte piece c of row r at piece c ^ (r % 16)
      float* sO = reinterpret_cast<float*>(sK) + (size_t)(i * kTT + row) * HD;
#pragma unroll 1
      for (int c0 = 0; c0 < HD; c0 += 32) {
        float o[32];
        if (n > 0) {
          tmem_ld32(o_base + (uint32_t)c0, o);
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] = 0.f;
        }
        if (S == 1) {
          if (dst) {
#pragma unroll
            for (int q = 0; q < 32; q += 8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(o[q + 2 * e] * inv, o[q + 2 * e + 1] * inv);
                w[e] = *reinterpret_cast<const uint32_t*>(&v);
              }
              *reinterpret_cast<uint4*>(dst + c0 + q) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < 32; q += 4)
            *reinterpret_cast<float4*>(sO + ((((c0 + q) >> 2) ^ (row & 15)) << 2)) =
                make_float4(o[q], o[q + 1], o[q + 2], o[q + 3]);
        }
      }
      if (S > 1) {
        s_m[i * kTT + row] = m;
        s_l[i * kTT + row] = l;
      }
    }
  } else if (warp < kMmaWarp) {
    // --------------------------------------------------------- conversion
    const int t = tid - kConvWarp * 32;
    constexpr int CPR = HD / 16, PER = CPR;  // 16-byte pieces of a row; pieces a thread converts (128 rows / 128 threads)
    constexpr int ROWS = 128 / CPR;          // rows per step of the 128 threads (16 or 32)
    const size_t width = (size_t)p.n_kv * HD;
    const uint8_t* kbase = p.k_codes + (size_t)b * p.N * width + (size_t)h * HD;
    const uint8_t* vbase = p.v_codes + (size_t)b * p.N * width + (size_t)h * HD;
    const int nb = (p.N + (1 << p.block_log2) - 1) >> p.block_log2;
    const float* ksc = p.k_scale + (size_t)b * nb * p.n_kv + h;
    const float* vsc = p.v_scale + (size_t)b * nb * p.n_kv + h;
    const int tr = t / CPR, tc = t % CPR;
    uint4 kr[PER], vr[PER];
    float kf[PER], vf[PER];
    auto fetch = [&](const uint8_t* base, const float* scale, int j, uint4 (&r)[PER], float (&f)[PER]) {
#pragma unroll
      for (int it = 0; it < PER; ++it) {
        const int key = (kt0 + j) * kTT + it * ROWS + tr;
        r[it] = make_uint4(0u, 0u, 0u, 0u);
        f[it] = 0.f;
        if (j < n && key < len) {  // rows past the length are zeros, whatever the cache holds there
          r[it] = __ldg(reinterpret_cast<const uint4*>(base + (size_t)key * width) + tc);
          f[it] = __ldg(scale + (size_t)(key >> p.block_log2) * p.n_kv);
        }
      }
    };
    auto put = [&](uint8_t* tile, const uint4 (&r)[PER], const float (&f)[PER]) {
#pragma unroll
      for (int it = 0; it < PER; ++it) {
        const int row = it * ROWS + tr;
        uint4 lo, hi;
        convert16<FMT>(r[it], f[it], lo, hi);
        uint8_t* dst = tile + (tc >> 2) * 16384 + row * 128;
        const int c0 = (tc & 3) * 2, x = row & 7;
        // lanes of the two halves store their pieces in opposite order: every bank once
        const bool swap = (tc >> 2) & 1;
        *reinterpret_cast<uint4*>(dst + (((c0 + (swap ? 1 : 0)) ^ x) << 4)) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(dst + (((c0 + (swap ? 0 : 1)) ^ x) << 4)) = swap ? lo : hi;
      }
    };
    fetch(kbase, ksc, 0, kr, kf);
    fetch(vbase, vsc, 0, vr, vf);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const int st = j & 1;
      const uint32_t ph = ((j >> 1) - 1) & 1;
      if (j >= 2 && !mbar_wait(&sy.k_empty[st], ph, &sy.abort, err, 734)) break;
      put(sK + st * Cfg::kTile, kr, kf);
      proxy_fence_smem();
      mbar_arrive_cta(&sy.k_full[st]);
      fetch(kbase, ksc, j + 1, kr, kf);
      if (j >= 2 && !mbar_wait(&sy.v_empty[st], ph, &sy.abort, err, 735)) break;
      put(sV + st * Cfg::kTile, vr, vf);
      proxy_fence_smem();
      mbar_arrive_cta(&sy.v_full[st]);
      fetch(vbase, vsc, j + 1, vr, vf);
    }
  } else if (lane == 0) {
    // ---------------------------------------------------------------- MMA
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, HD) | (1u << 16);  // V is MN-major
    const uint64_t dq = smem_desc_sw128(smem_u32(sQ));
    const uint64_t dk = smem_desc_sw128(smem_u32(sK));
    const uint64_t dv = desc_sw128_mn(smem_u32(sV), 16384);
    constexpr uint64_t kTileOff = Cfg::kTile >> 4, kQOff = Cfg::kQBytes >> 4;
    bool ok = n > 0 && mbar_wait(&sy.q_full, 0, &sy.abort, err, 736);
    for (int j = 0; ok && j <= n; ++j) {
      const int st = j & 1, pst = (j - 1) & 1;
      if (j < n && !mbar_wait(&sy.k_full[st], (j >> 1) & 1, &sy.abort, err, 737)) break;
      if (j > 0 && !mbar_wait(&sy.v_full[pst], ((j - 1) >> 1) & 1, &sy.abort, err, 738)) break;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if (j > 0) {
          if (!mbar_wait(&sy.p_full[i], (j - 1) & 1, &sy.abort, err, 739)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(tmem + 256u + i * 128u, tmem + i * 128u + kk * 8u, dv + pst * kTileOff + (uint64_t)(kk * 128),
                         idesc_pv, (j > 1 || kk > 0) ? 1u : 0u);
          if (i == NQ - 1) umma_commit(&sy.v_empty[pst]);
        }
        if (j < n) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint64_t off = (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);
            umma_bf16(tmem + i * 128u, dq + i * kQOff + off, dk + st * kTileOff + off, idesc_qk, kk > 0 ? 1u : 0u);
          }
          umma_commit(&sy.s_full[i]);
          if (i == NQ - 1) umma_commit(&sy.k_empty[st]);
        }
      }
    }
    umma_commit(&sy.o_done);
  }
  __syncwarp();
  __syncthreads();
  if (sy.abort != 0 && tid == 0) mbar_drain_bounded(&sy.o_done, 0, err, 740);  // MMAs in flight, before TMEM is freed
  __syncthreads();
  if (S > 1) {
    // every thread of every CTA passes both cluster barriers, whatever happened before
    cluster_sync();
    const bool good = sy.abort == 0 && sy.ok;
    const int RS = kTT / S;  // rows of each query tile this CTA joins
    if (good && tid < NQ * RS) {
      const int row = (tid / RS) * kTT + sp * RS + tid % RS;
      const uint32_t am = smem_u32(&s_m[row]), al = smem_u32(&s_l[row]);
      float mq[8], lq[8], mm = -INFINITY;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < S) {
          mq[q] = ld_dsmem_f32(mapa_shared(am, (uint32_t)q));
          lq[q] = ld_dsmem_f32(mapa_shared(al, (uint32_t)q));
          mm = fmaxf(mm, mq[q]);
        }
      float L = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < S) {
          mq[q] = mq[q] == -INFINITY && lq[q] == 0.f ? 0.f : exp2f(mq[q] - mm);  // a share without keys adds nothing
          L += mq[q] * lq[q];
        }
      const float inv = L != 0.f ? 1.0f / L : 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < S) s_w[row][q] = mq[q] * inv;
    }
    __syncthreads();
    if (good) {
      constexpr int C4 = HD / 4;
      for (int task = tid; task < NQ * RS * C4; task += Cfg::kThreads) {
        const int ri = task / C4, ch = task % C4;
        const int row = (ri / RS) * kTT + sp * RS + ri % RS, qr = row0 + row;
        if (qr >= R) continue;
        const uint32_t la = smem_u32(reinterpret_cast<float*>(sK) + (size_t)row * HD + ((ch ^ (row & 15)) << 2));
        float4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < S) v[q] = ld_dsmem_f4(mapa_shared(la, (uint32_t)q));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < S) {
            const float w = s_w[row][q];
            acc.x += w * v[q].x; acc.y += w * v[q].y; acc.z += w * v[q].z; acc.w += w * v[q].w;
          }
        store4(reinterpret_cast<__nv_bfloat16*>(p.O) +
                   (((size_t)b * p.k + qr / p.group) * p.n_heads + (size_t)h * p.group + qr % p.group) * HD + ch * 4,
               acc);
      }
    }
    cluster_sync();  // no CTA leaves while its rows are being read
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int HD, int FMT, int NQ>
static cudaError_t launch_tc(Q8AttnParams& p, int splits_most, cudaStream_t stream) {
  using Cfg = TcCfg<HD, NQ>;
  auto kern = q8_attn_tc_kernel<HD, FMT, NQ>;
  cudaError_t e = configure_kernel((const void*)kern, Cfg::kSmem, false);
  if (e != cudaSuccess) return e;
  p.splits = splits_most;
  const int tiles = (p.k * p.group + NQ * kTT - 1) / (NQ * kTT);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * p.splits), p.n_kv, p.B);
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Key shares: doubled while the grid stays within the SMs (one CTA on each,
// by shared memory) and every share keeps a tile.
static int tc_splits(long long ctas, int n_kt, int num_sms) {
  int s = 1;
  while (s < 8 && ctas * s * 2 <= num_sms && n_kt >= s * 2) s *= 2;
  return s;
}

cudaError_t launch_q8_attention_tc(int fmt, int hd, Q8AttnParams p, int num_sms, cudaStream_t stream) {
  const int n_kt = (p.N + kTT - 1) / kTT;
  const long long heads = (long long)p.B * p.n_kv;
  const int t1 = (p.k * p.group + kTT - 1) / kTT, t2 = (t1 + 1) / 2;
  // two query tiles in a CTA share the converted keys and values; one while the single tiles do not fill the SMs
  const bool two = t1 >= 2 && heads * t1 > num_sms / 2;
  const int s = tc_splits(heads * (two ? t2 : t1), n_kt, num_sms);
#define SPA_TC_Q8(HD_, F_) \
  return two ? launch_tc<HD_, F_, 2>(p, s, stream) : launch_tc<HD_, F_, 1>(p, s, stream)
  if (hd == 128) {
    if (fmt == kQ8Int8) SPA_TC_Q8(128, kQ8Int8);
    SPA_TC_Q8(128, kQ8E4m3);
  }
  if (hd == 64) {
    if (fmt == kQ8Int8) SPA_TC_Q8(64, kQ8Int8);
    SPA_TC_Q8(64, kQ8E4m3);
  }
#undef SPA_TC_Q8
  return cudaErrorInvalidValue;
}

}  // namespace spa
