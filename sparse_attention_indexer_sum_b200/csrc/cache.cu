// cache.cu -- what a serving loop runs between its projections and the path:
//  * RMS norm with the residual's addition, its result in bf16 / fp32 and / or e4m3
//    with one scale per 128 values (the arithmetic of quant_e4m3_kernel per group);
//  * latent rows and indexer keys into cache slots (paged or not), with the position
//    rotation applied on the way: bf16, e4m3 or 4-bit microscaled latent rows, bf16 or
//    e4m3 keys.
// Both are bound by memory: every input is read once and every output written once,
// from registers.
#include <type_traits>

#include "ic_device.cuh"
#include "ic_internal.h"

namespace ic {

// ------------------------------------------------------------------ RMS norm
// h = x + residual;  y = h * rsqrt(mean(h^2) + eps) * weight, all in fp32: the sum is
// rounded only where it is stored, and the norm is of the unrounded sum.
//   codes: per group of 128 values, scale = amax / 448 (1 when amax == 0), code =
//   e4m3_rn_satfinite(y / scale), from the unrounded y.

template <typename T>
struct Vec8;  // eight values from / to 16-byte aligned memory
template <>
struct Vec8<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const void* p, long i, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __bfloat1622float2(h[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store(void* p, long i, const float (&v)[8]) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = u;
  }
};
template <>
struct Vec8<float> {
  static __device__ __forceinline__ void load(const void* p, long i, float (&v)[8]) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, long i, const float (&v)[8]) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// The quantiser of a group: scale = amax / 448 (1 when amax == 0), code =
// e4m3_rn_satfinite(x / scale) with the quotient correctly rounded, as in
// quant_e4m3_kernel.  The quotient takes three operations instead of a division: q = x r
// with r the correctly rounded reciprocal of the scale, then one correction by the exact
// remainder, q + (x - q scale) r, which is the correctly rounded quotient (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990) as
// long as the remainder does not underflow.  It can only for |x| < 2^-125; with a scale of
// at least 2^-90 the quotient is then far below the smallest code.  Smaller scales, and
// those that are not finite, take the division.
struct E4m3Scale {
  float scale, rcp;
  bool divide;
  __device__ __forceinline__ explicit E4m3Scale(float amax) {
    scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    rcp = __frcp_rn(scale);
    divide = !(scale >= 0x1p-90f && scale < INFINITY);
  }
  __device__ __forceinline__ float fast(float x) const {
    const float q = x * rcp;
    return fmaf(fmaf(-q, scale, x), rcp, q);
  }
  __device__ __forceinline__ uint32_t code(float x) const {
    return static_cast<uint32_t>(__nv_cvt_float_to_fp8(divide ? __fdiv_rn(x, scale) : fast(x),
                                                       __NV_SATFINITE, __NV_E4M3));
  }
  // The codes of N values (a multiple of 4), four a word.
  template <int N>
  __device__ __forceinline__ void codes(const float* v, uint32_t* w) const {
    if (!divide) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        w[i / 4] = pair(fast(v[i]), fast(v[i + 1])) | (pair(fast(v[i + 2]), fast(v[i + 3])) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        w[i / 4] = pair(__fdiv_rn(v[i], scale), __fdiv_rn(v[i + 1], scale)) |
                   (pair(__fdiv_rn(v[i + 2], scale), __fdiv_rn(v[i + 3], scale)) << 16);
    }
  }
  static __device__ __forceinline__ uint32_t pair(float x, float y) {
    return static_cast<uint32_t>(
        __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3));
  }
};

template <typename F>
__device__ __forceinline__ F block_sum(F v, F* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x / 32;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  F t = (threadIdx.x & 31) < nw ? part[threadIdx.x & 31] : F(0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// The scale 1 / sqrt(mean(h^2) + eps) as up * rstd (y = h * up * rstd * weight).  WIDE: where
// eps does not cover squares that vanish in 32 bits (kNormEps), they are taken and summed in
// 64; up is a power of two that keeps both factors normal numbers where the scale is none.
constexpr float kNormEps = 0x1p-100f;
template <bool WIDE>
struct NormSum {
  using type = typename std::conditional<WIDE, double, float>::type;
  static __device__ __forceinline__ void add(type& s, float v) {
    if constexpr (WIDE)
      s += static_cast<double>(v) * v;
    else
      s = fmaf(v, v, s);
  }
  float up = 1.f, rstd;
  template <typename F>
  __device__ __forceinline__ NormSum(F total, int n, float eps) {
    if constexpr (WIDE) {
      const double r = rsqrt(static_cast<double>(total) / n + eps);
      up = r > 0x1p100 ? 0x1p64f : r < 0x1p-64 ? 0x1p-32f : 1.f;
      rstd = static_cast<float>(r / up);
    } else {
      rstd = rsqrtf(static_cast<float>(total) / static_cast<float>(n) + eps);
    }
  }
  __device__ __forceinline__ float operator()(float h, float w) const {
    if constexpr (WIDE) h *= up;
    return h * rstd * w;
  }
};

// One CTA per row, the row in registers: thread t holds chunks t, t + T, ... of eight
// values (CH of them at most; T = blockDim.x is a multiple of 32, so the 16 chunks of a
// group of 128 lie in one half warp).
// Bound by memory where there are many rows, and then by how many rows are in flight: 32
// registers a thread instead of 40 (a few bytes spilled) take 16384 rows of 7168 with all
// outputs from 190 to 173 us (6.1 TB/s, 0.93 of the measured copy rate), 4096 of 16384 from
// 145 to 109 us.
template <typename T, int CH, bool WIDE>
__global__ void __launch_bounds__(1024, 2) rms_norm_kernel(const RmsNormArgs a) {
  using Sum = NormSum<WIDE>;
  __shared__ typename Sum::type part[32];
  grid_dep_wait();
  const long row = blockIdx.x;
  const int chunks = a.n / 8;
  float v[CH][8];
  typename Sum::type ss = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (c < chunks) {
      Vec8<T>::load(a.x, row * a.ld_x + 8 * c, v[i]);
      if (a.residual) {
        float r[8];
        Vec8<T>::load(a.residual, row * a.ld_r + 8 * c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) Sum::add(ss, v[i][j]);
    }
  }
  const Sum scale(block_sum(ss, part), a.n, a.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < chunks) {
      if (a.h) Vec8<T>::store(a.h, row * a.ld_h + 8 * c, v[i]);
      float w[8];
      if (a.w_f32)
        Vec8<float>::load(a.weight, 8 * c, w);
      else
        Vec8<__nv_bfloat16>::load(a.weight, 8 * c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = scale(v[i][j], w[j]);
      if (a.y) Vec8<T>::store(a.y, row * a.ld_y + 8 * c, v[i]);
    }
    if (a.codes) {
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const E4m3Scale sc(amax);
      if (c < chunks) {
        uint32_t w[2];
        sc.codes<8>(v[i], w);
        *reinterpret_cast<uint2*>(a.codes + row * a.ld_c + 8 * c) = make_uint2(w[0], w[1]);
        if ((c & 15) == 0) a.scales[row * ((a.n + 127) / 128) + c / 16] = sc.scale;
      }
    }
  }
}

// Any length, stride and alignment: one CTA per row, the row read twice (the second
// time from cache), a warp per group of 128 values.  Every element of the second pass
// is read before the same thread writes it, so h may be the residual and y may be x.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) rms_norm_any_kernel(const RmsNormArgs a) {
  __shared__ double part[32];
  grid_dep_wait();
  const long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.ld_r : nullptr;
  // a thread's squares in runs of 16, the runs in 64 bits: in one 32-bit sum the last of
  // millions of terms would round to a fraction of their bits
  double ss = 0.0;
  for (int i = threadIdx.x; i < a.n;) {
    const int end = min(a.n, i + 16 * static_cast<int>(blockDim.x));
    typename NormSum<WIDE>::type run = 0;
#pragma unroll 4
    for (; i < end; i += blockDim.x) {
      float v = static_cast<float>(x[i]);
      if (r) v += static_cast<float>(r[i]);
      NormSum<WIDE>::add(run, v);
    }
    ss += run;
  }
  const NormSum<WIDE> scale(block_sum(ss, part), a.n, a.eps);
  T* h = a.h ? static_cast<T*>(a.h) + row * a.ld_h : nullptr;
  T* y = a.y ? static_cast<T*>(a.y) + row * a.ld_y : nullptr;
  const int lane = threadIdx.x & 31, groups = (a.n + 127) / 128;
  for (int g = threadIdx.x / 32; g < groups; g += blockDim.x / 32) {
    float v[4], amax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 128 * g + 32 * j + lane;
      v[j] = 0.f;
      if (i < a.n) {
        v[j] = static_cast<float>(x[i]);
        if (r) v[j] += static_cast<float>(r[i]);
        if (h) h[i] = static_cast<T>(v[j]);
        const float w = a.w_f32 ? static_cast<const float*>(a.weight)[i]
                                : __bfloat162float(static_cast<const __nv_bfloat16*>(a.weight)[i]);
        v[j] = scale(v[j], w);
        if (y) y[i] = static_cast<T>(v[j]);
      }
      amax = fmaxf(amax, fabsf(v[j]));
    }
    if (a.codes) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const E4m3Scale sc(amax);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 128 * g + 32 * j + lane;
        if (i < a.n) a.codes[row * a.ld_c + i] = static_cast<uint8_t>(sc.code(v[j]));
      }
      if (lane == 0) a.scales[row * groups + g] = sc.scale;
    }
  }
}

template <typename T, bool WIDE>
static cudaError_t launch_rms_norm_t(const RmsNormArgs& a, cudaStream_t stream) {
  const auto ok = [](const void* p, long ld_bytes, unsigned to) {
    return reinterpret_cast<uintptr_t>(p) % to == 0 && ld_bytes % to == 0;
  };
  const long e = sizeof(T);
  const bool vec = a.n % 8 == 0 && a.n <= 16384 && ok(a.x, a.ld_x * e, 16) &&
                   ok(a.residual, a.ld_r * e, 16) && ok(a.h, a.ld_h * e, 16) &&
                   ok(a.y, a.ld_y * e, 16) && ok(a.codes, a.ld_c, 8) && ok(a.weight, 0, 16);
  const dim3 grid(static_cast<unsigned>(a.rows));
  if (!vec) return launch_dep(rms_norm_any_kernel<T, WIDE>, grid, dim3(256), 0, stream, 1, a);
  const int chunks = a.n / 8;
  // Two chunks a thread keep more CTAs, and so rows, in flight where there are rows to fill
  // them (16384 rows of 4096: 96 against 114 us); with few rows one chunk a thread is the
  // shorter way (64 rows: 2.8 against 3.5 us), as it is for short rows.
  const bool two = chunks > 1024 || (chunks > 128 && a.rows >= 4L * num_sms());
  const int per = two ? (chunks + 1) / 2 : chunks;
  const dim3 block(static_cast<unsigned>((per + 31) / 32 * 32));
  return two ? launch_dep(rms_norm_kernel<T, 2, WIDE>, grid, block, 0, stream, 1, a)
             : launch_dep(rms_norm_kernel<T, 1, WIDE>, grid, block, 0, stream, 1, a);
}

ic_status launch_rms_norm(const RmsNormArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return IC_OK;
  // (64 bits for every eps: 190 instead of 173 us on 16384 x 7168 with all outputs)
  const cudaError_t e = a.eps < kNormEps
                            ? a.f32 ? launch_rms_norm_t<float, true>(a, stream)
                                    : launch_rms_norm_t<__nv_bfloat16, true>(a, stream)
                        : a.f32 ? launch_rms_norm_t<float, false>(a, stream)
                                : launch_rms_norm_t<__nv_bfloat16, false>(a, stream);
  ic_status st = cuda_check(e, "rms_norm_kernel launch");
  if (!st) {
    const double m = static_cast<double>(a.rows) * a.n, b = a.f32 ? 4.0 : 2.0;
    trace_launch(kKindRmsNorm, stream,
                 m * (b * (1 + (a.residual != nullptr) + (a.h != nullptr) + (a.y != nullptr)) +
                      (a.codes ? 1.0 : 0.0)) +
                     (a.codes ? 4.0 * a.rows * ((a.n + 127) / 128) : 0.0));
  }
  return st;
}

// ------------------------------------------------------------------ cache append
// A pair (a, b) turned by the position's angle: (a cos - b sin, b cos + a sin).
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float t = a * c - b * s;
  b = fmaf(b, c, a * s);
  a = t;
}

// The e8m0 code of a block of magnitude amax >= 0: the smallest power of two 2^(E - 127)
// with amax / 2^(E - 127) <= 6, so that no value saturates.  amax = m 2^e with m in
// [1, 2): e - 2 if m <= 1.5, else e - 1; the addition carries into the exponent field
// exactly when m > 1.5.  (Rounding e down, the other common rule, clips magnitudes with m
// above 1.5, the block's largest by up to a quarter; its mean squared error is 1 % lower on
// normal data and 8 % on Laplace data.)  A block with an infinity or NaN gets 255 (NaN).
__device__ __forceinline__ unsigned e8m0_code(float amax, bool finite) {
  if (!finite) return 255u;
  const int e = static_cast<int>((__float_as_uint(amax) + 0x3FFFFFu) >> 23) - 2;
  return e > 0 ? static_cast<unsigned>(e) : 0u;
}

// One warp per token.  Latent row (576 values): lane l holds dims 16l..16l+15; the 64
// rotated dims are a pair per lane.  Key (128 values): lane l holds dims 4l..4l+3, of
// which the first 64 are rotated.
// Bound by memory.
template <int FMT>
__global__ void __launch_bounds__(128, 10) cache_append_kernel(const AppendArgs a) {
  grid_dep_wait();
  const long row = static_cast<long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (row >= a.rows) return;
  // every load that does not depend on another goes out first
  const long slot = a.slots[row];
  const long pos = a.rope ? a.pos[row] : 0;
  uint4 u0, u1;
  uint2 ku;
  __nv_bfloat162 rp;  // rotated latent dims: pair (2l, 2l + 1), or (l, l + 32)
  if (a.kv) {
    const __nv_bfloat16* x = a.kv + row * a.ld_kv;
    u0 = *reinterpret_cast<const uint4*>(x + 16 * lane);
    u1 = *reinterpret_cast<const uint4*>(x + 16 * lane + 8);
    if (a.kv_halves)
      rp = __nv_bfloat162(x[512 + lane], x[544 + lane]);
    else
      rp = *reinterpret_cast<const __nv_bfloat162*>(x + 512 + 2 * lane);
  }
  if (a.k) ku = *reinterpret_cast<const uint2*>(a.k + row * a.ld_k + 4 * lane);
  if (slot < 0) return;  // a padded row
  if (slot >= a.num_slots || pos < 0 || (a.rope && pos >= a.rope_rows)) return;
  const bool turn = a.rope != nullptr;
  float rc = 0.f, rs = 0.f;  // cos and sin of angle l
  if (turn) {
    rc = a.rope[pos * 64 + lane];
    rs = a.rope[pos * 64 + 32 + lane];
  }

  if (a.kv) {
    uint8_t* o = a.kv_cache + slot * a.ld_cache;
    if (turn) {
      float2 f = __bfloat1622float2(rp);
      rotate_pair(f.x, f.y, rc, rs);
      rp = __floats2bfloat162_rn(f.x, f.y);
    }
    __nv_bfloat16* ro;
    if constexpr (FMT == kFmtBf16) {
      *reinterpret_cast<uint4*>(o + 32 * lane) = u0;
      *reinterpret_cast<uint4*>(o + 32 * lane + 16) = u1;
      ro = reinterpret_cast<__nv_bfloat16*>(o + 1024);
    } else {
      float v[16];
      const __nv_bfloat162* p0 = reinterpret_cast<const __nv_bfloat162*>(&u0);
      const __nv_bfloat162* p1 = reinterpret_cast<const __nv_bfloat162*>(&u1);
      float amax = 0.f;
      bool finite = true;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(p0[i]), g = __bfloat1622float2(p1[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y, v[8 + 2 * i] = g.x, v[8 + 2 * i + 1] = g.y;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        amax = fmaxf(amax, fabsf(v[i]));
        if constexpr (FMT == kFmtMxf4) finite = finite && fabsf(v[i]) < INFINITY;
      }
      if constexpr (FMT == kFmtE4m3) {
#pragma unroll
        for (int off = 4; off > 0; off >>= 1)  // the 8 lanes of a group of 128
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const E4m3Scale sc(amax);
        uint32_t w[4];
        sc.codes<16>(v, w);
        *reinterpret_cast<uint4*>(o + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
        if ((lane & 7) == 0) *reinterpret_cast<float*>(o + 512 + 4 * (lane / 8)) = sc.scale;
        ro = reinterpret_cast<__nv_bfloat16*>(o + 528);
      } else {
        // the other half of the block of 32
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const unsigned both = __ballot_sync(0xffffffffu, finite);
        const unsigned e = e8m0_code(amax, ((both >> (lane & ~1)) & 3u) == 3u);
        // x 2^(127 - E), exact; E <= 253 for finite blocks
        const float inv = e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
        uint32_t w[2] = {0u, 0u};
        if (e != 255u) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t c = __nv_cvt_float2_to_fp4x2(
                make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_E2M1, cudaRoundNearest);
            w[i / 4] |= (c & 0xFFu) << (8 * (i & 3));
          }
        }
        *reinterpret_cast<uint2*>(o + 8 * lane) = make_uint2(w[0], w[1]);
        if ((lane & 1) == 0) o[256 + lane / 2] = static_cast<uint8_t>(e);
        ro = reinterpret_cast<__nv_bfloat16*>(o + 272);
      }
    }
    if (a.kv_halves) {
      ro[lane] = rp.x;
      ro[32 + lane] = rp.y;
    } else {
      *reinterpret_cast<__nv_bfloat162*>(ro + 2 * lane) = rp;
    }
  }

  if (a.k) {
    const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ku.x));
    const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ku.y));
    float v[4] = {f0.x, f0.y, f1.x, f1.y};
    if (turn) {
      if (a.k_halves) {  // dims 4l + j and 32 + 4l + j: lanes l and l + 8 (l < 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float other = __shfl_xor_sync(0xffffffffu, v[j], 8);
          const float c = __shfl_sync(0xffffffffu, rc, 4 * (lane & 7) + j);
          const float s = __shfl_sync(0xffffffffu, rs, 4 * (lane & 7) + j);
          if (lane < 16) v[j] = lane < 8 ? v[j] * c - other * s : fmaf(v[j], c, other * s);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // pairs 2l, 2l + 1
          const float c = __shfl_sync(0xffffffffu, rc, (2 * lane + j) & 31);
          const float s = __shfl_sync(0xffffffffu, rs, (2 * lane + j) & 31);
          if (lane < 16) rotate_pair(v[2 * j], v[2 * j + 1], c, s);
        }
      }
    }
    if (a.k_fp8) {
      float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      const E4m3Scale sc(amax);
      uint32_t w;
      sc.codes<4>(v, &w);
      *reinterpret_cast<uint32_t*>(a.k_cache + slot * 128 + 4 * lane) = w;
      if (lane == 0) a.k_scale[slot] = sc.scale;
    } else {
      uint2 w;
      *reinterpret_cast<__nv_bfloat162*>(&w.x) = __floats2bfloat162_rn(v[0], v[1]);
      *reinterpret_cast<__nv_bfloat162*>(&w.y) = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(a.k_cache + slot * 256 + 8 * lane) = w;
    }
  }
}

ic_status launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return IC_OK;
  const dim3 grid(static_cast<unsigned>((a.rows + 3) / 4)), block(128);
  const cudaError_t e =
      a.kv_fmt == kFmtMxf4
          ? launch_dep(cache_append_kernel<kFmtMxf4>, grid, block, 0, stream, 1, a)
      : a.kv_fmt == kFmtE4m3
          ? launch_dep(cache_append_kernel<kFmtE4m3>, grid, block, 0, stream, 1, a)
          : launch_dep(cache_append_kernel<kFmtBf16>, grid, block, 0, stream, 1, a);
  ic_status st = cuda_check(e, "cache_append_kernel launch");
  if (!st) {
    double row = 8.0 + (a.rope ? 4.0 + 256.0 : 0.0);
    if (a.kv)
      row += 1152.0 + (a.kv_fmt == kFmtMxf4   ? KV4_ROW_BYTES
                       : a.kv_fmt == kFmtE4m3 ? KV8_ROW_BYTES
                                              : 1152);
    if (a.k) row += 256.0 + (a.k_fp8 ? 132.0 : 256.0);
    trace_launch(kKindCacheAppend, stream, row * static_cast<double>(a.rows));
  }
  return st;
}

}  // namespace ic
