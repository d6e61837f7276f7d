// Activation checkpoints in 8 bits: a layer's saved block held between its
// forward and its backward as Pre, the deviations O - mean and X in 8 bits with
// one power of two for every 32 values, and restored from them.
//
// For a group of 32 values with the largest magnitude m = f 2^E (1 <= f < 2),
// the scale 2^k is the smallest power of two with m <= top 2^k.  int8 (top
// 127): 64 f <= 127 gives k = E - 6, else E - 5; e4m3 (top 448 = 1.75 2^8):
// f <= 1.75 gives k = E - 8, else E - 7.  Multiplying by a power of two is exact,
// so the only rounding of a value is the one to 8 bits.
//
// Memory-bound: the save reads 14d bytes a token and writes 6.19d (bf16
// operands, fp32 residual stream), the restore reads 6.19d and writes 24d; the
// arithmetic is a few instructions a value.
#include <cuda_fp8.h>

#include "args.h"
#include "common.cuh"
#include "internal.h"

namespace hstu {
namespace {

constexpr int kGroup = 32;          // values that share a scale
constexpr int kScaleNaN = 255;
// Largest biased exponent k + 127: the largest with top 2^k in fp32's range.  A
// larger magnitude (within 2^-7 of fp32's end) is held as top 2^k, since the
// multiple of the next scale that it rounds to is 2^128.
template <int FMT> constexpr int kScaleMax = FMT == HSTU_CKPT_INT8 ? 121 + 127 : 119 + 127;

// 2^k for k in [-126, 127].
__device__ __forceinline__ float pow2f(int k) { return __int_as_float((k + 127) << 23); }

// The biased exponent k + 127 of the group whose largest magnitude has these bits.
template <int FMT>
__device__ __forceinline__ int scale_of(uint32_t abs_bits) {
  if (abs_bits >= 0x7f800000u) return kScaleNaN;
  const int E = (int)(abs_bits >> 23);                       // biased; 0 below 2^-126
  const uint32_t f = abs_bits & 0x7fffffu;
  // 127/64 = 1.984375 and 448/256 = 1.75 as fractions of 2^23
  const int k = FMT == HSTU_CKPT_INT8 ? E - 6 + (f > 0x7e0000u) : E - 8 + (f > 0x600000u);
  return min(max(k, 1), kScaleMax<FMT>);
}

// Eight values of a group with this scale in 8 bits (e4m3's conversion saturates by itself).
template <int FMT>
__device__ __forceinline__ uint2 pack8(float (&f)[8], int scale) {
  uint32_t w[2];
  const float inv = pow2f(scale == kScaleNaN ? 0 : 127 - scale);
  if (FMT == HSTU_CKPT_INT8) {
    if (scale == kScaleMax<FMT>) {
      const float top = 127.f * pow2f(kScaleMax<FMT> - 127);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i], -top), top);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // |f inv| <= 127: adding 1.5 2^23 rounds to the nearest whole number
      // (ties to even) and leaves it in the low byte
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(fmaf(f[4 * i + j], inv, 12582912.f));
      w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

template <int FMT>
__device__ __forceinline__ void unpack8(uint2 q, int scale, float (&f)[8]) {
  const float s = scale == kScaleNaN ? __int_as_float(0x7fffffff) : pow2f(scale - 127);
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (FMT == HSTU_CKPT_INT8) {
      const uint32_t u = w[i] ^ 0x80808080u;                 // value + 128 in each byte
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[4 * i + j] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + j)) - 8388736.f) * s;
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * j)), __NV_E4M3);
        const float2 t = __half22float2(__half2(h));
        f[4 * i + 2 * j] = t.x * s;
        f[4 * i + 2 * j + 1] = t.y * s;
      }
    }
  }
}

struct CkptPtrs {
  unsigned char *pre, *dev, *x, *pre_s, *dev_s, *x_s;
  float *mean, *rstd;
};

// One thread for 8 values; units [0, 4n) are Pre's, [4n, 5n) O's, [5n, 6n) X's,
// n = T d / 8.  n is a multiple of 4 (d is one of 32), so a group's four
// lanes are in one part; whole warps run every step (the grid is padded).
template <typename T, int FMT, bool HAS_X>
__global__ void __launch_bounds__(256) ckpt_save_kernel(const T* __restrict__ pre, const float* __restrict__ o,
                                                        const T* __restrict__ x, const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, int64_t rows, int d,
                                                        CkptPtrs c) {
  const int64_t n = rows * (d / 8), total = n * (HAS_X ? 6 : 5);
  const int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = i0; i < rows; i += step) {
    c.mean[i] = mean[i];
    c.rstd[i] = rstd[i];
  }
  const int64_t padded = (total + 31) / 32 * 32;
  for (int64_t i = i0; i < padded; i += step) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    unsigned char *q = c.pre, *s = c.pre_s;
    int64_t u = i;
    if (i < 4 * n) {
      load8(pre + u * 8, f);
    } else if (i < 5 * n) {
      u = i - 4 * n;
      q = c.dev;
      s = c.dev_s;
      load8(o + u * 8, f);
      const float mu = mean[u / (d / 8)];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] -= mu;
    } else if (HAS_X && i < total) {
      u = i - 5 * n;
      q = c.x;
      s = c.x_s;
      load8(x + u * 8, f);
    }
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(f[k]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if (i < total) {
      const int k = scale_of<FMT>(m);
      if ((u & 3) == 0) s[u >> 2] = (unsigned char)k;
      *reinterpret_cast<uint2*>(q + u * 8) = pack8<FMT>(f, k);
    }
  }
}

__device__ __forceinline__ float silu_of(float x) { return x / (1.f + __expf(-x)); }

// One thread for 8 columns of a row: U, V, Q, K, the deviation and X.
template <typename T, int FMT, bool HAS_X>
__global__ void __launch_bounds__(256) ckpt_restore_kernel(CkptPtrs c, const T* __restrict__ gamma,
                                                           const T* __restrict__ beta, int64_t rows, int d,
                                                           T* __restrict__ pre, T* __restrict__ g,
                                                           float* __restrict__ o, T* __restrict__ z,
                                                           T* __restrict__ x, float* __restrict__ mean,
                                                           float* __restrict__ rstd) {
  const int units = d / 8;
  const int64_t total = rows * units;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
    const int64_t r = i / units;
    const int u = (int)(i - r * units);
    const float mu = c.mean[r], rs = c.rstd[r];
    if (u == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
    float gate[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int64_t at = r * 4 * units + p * units + u;
      float f[8], a[8];
      unpack8<FMT>(*reinterpret_cast<const uint2*>(c.pre + at * 8), c.pre_s[at >> 2], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = silu_of(f[k]);
      store8(pre + at * 8, f);
      store8(g + at * 8, a);
      if (p == 0)
#pragma unroll
        for (int k = 0; k < 8; ++k) gate[k] = to_f(from_f<T>(a[k]));
    }
    float dv[8], out[8];
    unpack8<FMT>(*reinterpret_cast<const uint2*>(c.dev + i * 8), c.dev_s[i >> 2], dv);
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = mu + dv[k];
    store8(o + i * 8, out);
    float gm[8], bt[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      gm[k] = 1.f;
      bt[k] = 0.f;
    }
    if (gamma) load8(gamma + u * 8, gm);
    if (beta) load8(beta + u * 8, bt);
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = (dv[k] * rs * gm[k] + bt[k]) * gate[k];
    store8(z + i * 8, out);
    if (HAS_X) {
      unpack8<FMT>(*reinterpret_cast<const uint2*>(c.x + i * 8), c.x_s[i >> 2], out);
      store8(x + i * 8, out);
    }
  }
}

void ckpt_offsets(const hstu_config* c, int64_t T, size_t off[HSTU_CKPT_COUNT + 1]) {
  const size_t d = (size_t)c->d_model, t = (size_t)T;
  const size_t x = c->io_dtype != c->dtype ? t * d : 0;
  const size_t sizes[HSTU_CKPT_COUNT] = {t * 4 * d,          t * d,      x,     t * 4 * d / kGroup,
                                         t * d / kGroup, x / kGroup, t * 4, t * 4};
  size_t o = 0;
  for (int i = 0; i < HSTU_CKPT_COUNT; ++i) {
    off[i] = o;
    o = align_up(o + sizes[i], 256);
  }
  off[HSTU_CKPT_COUNT] = o;
}

CkptPtrs ckpt_ptrs(const hstu_config* c, int64_t T, const void* ckpt) {
  size_t off[HSTU_CKPT_COUNT + 1];
  ckpt_offsets(c, T, off);
  auto* b = static_cast<unsigned char*>(const_cast<void*>(ckpt));
  CkptPtrs p;
  p.pre = b + off[HSTU_CKPT_PRE];
  p.dev = b + off[HSTU_CKPT_DEV];
  p.x = b + off[HSTU_CKPT_X];
  p.pre_s = b + off[HSTU_CKPT_PRE_SCALE];
  p.dev_s = b + off[HSTU_CKPT_DEV_SCALE];
  p.x_s = b + off[HSTU_CKPT_X_SCALE];
  p.mean = reinterpret_cast<float*>(b + off[HSTU_CKPT_MEAN]);
  p.rstd = reinterpret_cast<float*>(b + off[HSTU_CKPT_RSTD]);
  return p;
}

unsigned grid_of(int64_t threads) {
  const int64_t g = (threads + 255) / 256, cap = (int64_t)sm_count() * 32;
  return (unsigned)(g > cap ? cap : g);
}

template <typename T, int FMT, bool HAS_X>
cudaError_t launch_save(const hstu_config* c, const void* saved, int64_t rows, void* ckpt, cudaStream_t s) {
  size_t off[HSTU_SAVED_COUNT + 1];
  saved_offsets(c, rows, off);
  auto* b = static_cast<const unsigned char*>(saved);
  ckpt_save_kernel<T, FMT, HAS_X><<<grid_of(rows * (c->d_model / 8) * (HAS_X ? 6 : 5)), 256, 0, s>>>(
      reinterpret_cast<const T*>(b + off[HSTU_SAVED_PRE]),
      reinterpret_cast<const float*>(b + off[HSTU_SAVED_O]),
      reinterpret_cast<const T*>(b + off[HSTU_SAVED_XLOW]),
      reinterpret_cast<const float*>(b + off[HSTU_SAVED_MEAN]),
      reinterpret_cast<const float*>(b + off[HSTU_SAVED_RSTD]), rows, c->d_model, ckpt_ptrs(c, rows, ckpt));
  count_launch();
  return cudaGetLastError();
}

template <typename T, int FMT, bool HAS_X>
cudaError_t launch_restore(const hstu_config* c, const void* ckpt, const void* gamma, const void* beta,
                           int64_t rows, void* saved, cudaStream_t s) {
  size_t off[HSTU_SAVED_COUNT + 1];
  saved_offsets(c, rows, off);
  auto* b = static_cast<unsigned char*>(saved);
  ckpt_restore_kernel<T, FMT, HAS_X><<<grid_of(rows * (c->d_model / 8)), 256, 0, s>>>(
      ckpt_ptrs(c, rows, ckpt), static_cast<const T*>(gamma), static_cast<const T*>(beta), rows, c->d_model,
      reinterpret_cast<T*>(b + off[HSTU_SAVED_PRE]), reinterpret_cast<T*>(b + off[HSTU_SAVED_G]),
      reinterpret_cast<float*>(b + off[HSTU_SAVED_O]), reinterpret_cast<T*>(b + off[HSTU_SAVED_Z]),
      reinterpret_cast<T*>(b + off[HSTU_SAVED_XLOW]), reinterpret_cast<float*>(b + off[HSTU_SAVED_MEAN]),
      reinterpret_cast<float*>(b + off[HSTU_SAVED_RSTD]));
  count_launch();
  return cudaGetLastError();
}

hstu_status check_format(int32_t f) {
  return f == HSTU_CKPT_INT8 || f == HSTU_CKPT_E4M3 ? HSTU_OK : HSTU_ERR_INVALID;
}

}  // namespace
}  // namespace hstu

using namespace hstu;

// The kernel for the config's types: bf16 with its own copy of X, bf16, fp32.
#define HSTU_CKPT_DISPATCH(FN, FMT, ...)                                     \
  (cfg->dtype == HSTU_F32 ? FN<float, FMT, false>(__VA_ARGS__)               \
   : cfg->io_dtype == HSTU_F32 ? FN<bf16, FMT, true>(__VA_ARGS__)            \
                               : FN<bf16, FMT, false>(__VA_ARGS__))

extern "C" {

hstu_status hstu_checkpoint_layout(const hstu_config* cfg, int64_t T, size_t offsets[HSTU_CKPT_COUNT + 1]) {
  HSTU_TRY(check_cfg(cfg));
  if (T < 0 || !offsets) return HSTU_ERR_INVALID;
  ckpt_offsets(cfg, T, offsets);
  return HSTU_OK;
}

hstu_status hstu_checkpoint_save(const hstu_config* cfg, int32_t format, const void* saved, int64_t T,
                                 void* ckpt, cudaStream_t stream) {
  HSTU_TRY(check_cfg(cfg));
  HSTU_TRY(check_format(format));
  if (T < 0) return HSTU_ERR_INVALID;
  HSTU_TRY(need(saved, T));
  HSTU_TRY(need(ckpt, T));
  if (T == 0) return HSTU_OK;
  prof_begin(HSTU_K_CHECKPOINT, stream);
  const cudaError_t e =
      format == HSTU_CKPT_INT8 ? HSTU_CKPT_DISPATCH(launch_save, HSTU_CKPT_INT8, cfg, saved, T, ckpt, stream)
                               : HSTU_CKPT_DISPATCH(launch_save, HSTU_CKPT_E4M3, cfg, saved, T, ckpt, stream);
  prof_end(HSTU_K_CHECKPOINT, stream);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

hstu_status hstu_checkpoint_restore(const hstu_config* cfg, int32_t format, const void* ckpt,
                                    const void* ln_gamma, const void* ln_beta, int64_t T, void* saved,
                                    cudaStream_t stream) {
  HSTU_TRY(check_cfg(cfg));
  HSTU_TRY(check_format(format));
  if (T < 0) return HSTU_ERR_INVALID;
  HSTU_TRY(need(ckpt, T));
  HSTU_TRY(opt(ln_gamma));
  HSTU_TRY(opt(ln_beta));
  HSTU_TRY(need(saved, T));
  if (T == 0) return HSTU_OK;
  prof_begin(HSTU_K_CHECKPOINT, stream);
  const cudaError_t e = format == HSTU_CKPT_INT8
                            ? HSTU_CKPT_DISPATCH(launch_restore, HSTU_CKPT_INT8, cfg, ckpt, ln_gamma, ln_beta,
                                                 T, saved, stream)
                            : HSTU_CKPT_DISPATCH(launch_restore, HSTU_CKPT_E4M3, cfg, ckpt, ln_gamma, ln_beta,
                                                 T, saved, stream);
  prof_end(HSTU_K_CHECKPOINT, stream);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
