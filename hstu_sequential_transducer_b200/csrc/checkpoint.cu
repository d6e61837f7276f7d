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
// arithmetic is 12 and 17 instructions a value, most of them on pairs.  So the kernels are
// plain streams: many small CTAs, each in one part of the block; a thread
// loads its pieces of 16 bytes (of the wider side) before it works on the first,
// and neighbouring threads hold neighbouring pieces, so that every access covers
// whole 32-byte sectors.
//
// Measured at 131,072 x 1,024, int8, bf16 operands, fp32 residual stream: save 412 us
// (6.6 TB/s; 435 with 2 pieces in flight, 555 with 1), restore 647 us
// (6.3 TB/s; 708 with 4 pieces of V, Q, K and X, 1,216 with 8: the stores of
// few CTAs come in bursts).
#include <cuda_fp8.h>

#include "args.h"
#include "common.cuh"
#include "f32x2.cuh"
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

// The biased exponent k + 127 of the group whose largest magnitude has these
// bits: the exponent, one more for a fraction above 127/64 = 1.984375 or 448/256
// = 1.75 (0x7e0000 and 0x600000 as fractions of 2^23, which the addend carries over).
template <int FMT>
__device__ __forceinline__ int scale_of(uint32_t abs_bits) {
  const int k = FMT == HSTU_CKPT_INT8 ? (int)((abs_bits + 0x1ffffu) >> 23) - 6 : (int)((abs_bits + 0x1fffffu) >> 23) - 8;
  return abs_bits >= 0x7f800000u ? kScaleNaN : min(max(k, 1), kScaleMax<FMT>);
}

// 2^k of a held scale; NaN for a group that holds none.
__device__ __forceinline__ float scale_value(int scale) {
  return scale == kScaleNaN ? __int_as_float(0x7fffffff) : pow2f(scale - 127);
}

// W elements of a 16-byte or 8-byte piece, as pairs.
template <typename T, int W> struct Piece {
  static constexpr int kWords = W * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 4) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
  }
  __device__ __forceinline__ void get(F2 (&f)[W / 2]) const {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      if constexpr (sizeof(T) == 4) f[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
  __device__ __forceinline__ void set(const F2 (&f)[W / 2]) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[2 * i] = __float_as_uint(f[i].x);
        w[2 * i + 1] = __float_as_uint(f[i].y);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
  // The largest magnitude's bits as fp32 (above infinity's for a NaN).
  __device__ __forceinline__ uint32_t largest() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = w[0] & 0x7fffffffu;
#pragma unroll
      for (int i = 1; i < kWords; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    } else {
      uint32_t m = w[0] & 0x7fff7fffu;               // two at a time
#pragma unroll
      for (int i = 1; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
      return max(m << 16, m & 0xffff0000u);
    }
  }
};
// Elements of a 16-byte piece.
template <typename T> constexpr int kPiece = 16 / (int)sizeof(T);

// Two pairs of a group with this scale in 8 bits (e4m3's conversion saturates by itself).
template <int FMT> __device__ __forceinline__ uint32_t pack4(F2 a, F2 b, F2 inv) {
  if (FMT == HSTU_CKPT_INT8) {
    // |a inv| <= 127: adding 1.5 2^23 rounds to the nearest whole number
    // (ties to even) and leaves it in the low byte
    const F2 x = fma(a, inv, both(12582912.f)), y = fma(b, inv, both(12582912.f));
    return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                       __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(mul(a, inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(mul(b, inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <int FMT> __device__ __forceinline__ void unpack4(uint32_t w, F2 s, F2& a, F2& b) {
  if (FMT == HSTU_CKPT_INT8) {
    const uint32_t u = w ^ 0x80808080u;                 // value + 128 in each byte
    uint32_t f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __byte_perm(u, 0x4b000000u, 0x7440 + j);    // 2^23 + value + 128
    a = mul(add(make_float2(__uint_as_float(f[0]), __uint_as_float(f[1])), both(-8388736.f)), s);
    b = mul(add(make_float2(__uint_as_float(f[2]), __uint_as_float(f[3])), both(-8388736.f)), s);
  } else {
    a = mul(__half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3))), s);
    b = mul(__half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3))), s);
  }
}

// W packed 8-bit values.
template <int W> struct Held {
  uint32_t w[W / 4];
  __device__ __forceinline__ void load(const unsigned char* p) {
    if constexpr (W == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ void store(unsigned char* p) const {
    if constexpr (W == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
  template <int FMT> __device__ __forceinline__ void get(int scale, F2 (&f)[W / 2]) const {
    const F2 s = both(scale_value(scale));
#pragma unroll
    for (int i = 0; i < W / 4; ++i) unpack4<FMT>(w[i], s, f[2 * i], f[2 * i + 1]);
  }
};

struct CkptPtrs {
  unsigned char *pre, *dev, *x, *pre_s, *dev_s, *x_s;
  float *mean, *rstd;
};

constexpr int kThreads = 256;
constexpr int kSaveUnroll = 4;       // pieces that a thread has in flight

// The elements of a CTA: [base, base + count) of a part, count at most kThreads
// W U and a multiple of 32; piece i of a thread begins at its element place(i).
template <int W> __device__ __forceinline__ int place(int i) { return W * ((int)threadIdx.x + i * kThreads); }
__device__ __forceinline__ int count_of(int64_t n, int64_t base, int per) { return (int)min((int64_t)per, n - base); }

// Holds a piece at q and its group's scale in scales.  The 32 / W neighbouring
// lanes of a group have elements (`any`), or none of them has; whole warps take part.
template <int FMT, typename T, int W>
__device__ __forceinline__ void hold(F2 (&f)[W / 2], uint32_t largest, bool any, unsigned char* q,
                                     unsigned char* scales, int at) {
#pragma unroll
  for (int o = 16 / W; o > 0; o >>= 1) largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
  if (!any) return;
  const int k = scale_of<FMT>(largest);
  if (FMT == HSTU_CKPT_INT8 && k == kScaleMax<FMT>) {
    const float top = 127.f * pow2f(kScaleMax<FMT> - 127);
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
      f[i] = make_float2(fminf(fmaxf(f[i].x, -top), top), fminf(fmaxf(f[i].y, -top), top));
  }
  const F2 inv = both(pow2f(k == kScaleNaN ? 0 : 127 - k));
  Held<W> h;
#pragma unroll
  for (int i = 0; i < W / 4; ++i) h.w[i] = pack4<FMT>(f[2 * i], f[2 * i + 1], inv);
  h.store(q + at);
  if ((threadIdx.x & (kGroup / W - 1)) == 0) scales[at / kGroup] = (unsigned char)k;
}

// CTA `tile` of an array of n elements.
template <typename T, int FMT>
__device__ __forceinline__ void save_tile(const T* src, int64_t n, int64_t tile, unsigned char* q,
                                          unsigned char* scales) {
  constexpr int W = kPiece<T>, U = kSaveUnroll, kPer = kThreads * W * U;
  const int64_t base = tile * kPer;
  const int count = count_of(n, base, kPer);
  src += base;
  Piece<T, W> in[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    in[i] = {};
    if (place<W>(i) < count) in[i].load(src + place<W>(i));
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    F2 f[W / 2];
    in[i].get(f);
    hold<FMT, T, W>(f, in[i].largest(), place<W>(i) < count, q + base, scales + base / kGroup, place<W>(i));
  }
}

// CTAs [0, tp) hold Pre, [tp, tp + td) the deviations, the others X.
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) ckpt_save_kernel(const T* __restrict__ pre, const float* __restrict__ o,
                                                             const T* __restrict__ x, const float* __restrict__ mean,
                                                             const float* __restrict__ rstd, int64_t rows, int d,
                                                             int64_t tp, int64_t td, CkptPtrs c) {
  const int64_t tile = blockIdx.x, n = rows * d;
  if (tile < tp) {
    save_tile<T, FMT>(pre, 4 * n, tile, c.pre, c.pre_s);
    return;
  }
  if (tile >= tp + td) {
    save_tile<T, FMT>(x, n, tile - tp - td, c.x, c.x_s);
    return;
  }
  constexpr int W = kPiece<float>, U = kSaveUnroll, kPer = kThreads * W * U;
  const int64_t base = (tile - tp) * kPer;
  const int count = count_of(n, base, kPer);
  const RowOf where(base, d);
  o += base;
  mean += where.row0;
  rstd += where.row0;
  Piece<float, W> in[U];
  float mu[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    in[i] = {};
    mu[i] = 0.f;
    if (place<W>(i) < count) {
      const int r = where.rows_after(place<W>(i));
      in[i].load(o + place<W>(i));
      mu[i] = mean[r];
      if (where.col0 + place<W>(i) == r * d) {       // the row's first piece
        c.mean[where.row0 + r] = mu[i];
        c.rstd[where.row0 + r] = rstd[r];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    F2 f[W / 2];
    in[i].get(f);
#pragma unroll
    for (int k = 0; k < W / 2; ++k) f[k] = add(f[k], both(-mu[i]));
    Piece<float, W> p;
    p.set(f);
    hold<FMT, float, W>(f, p.largest(), place<W>(i) < count, c.dev + base, c.dev_s + base / kGroup, place<W>(i));
  }
}

constexpr int kGateUnroll = 2, kRestUnroll = 2;

// Stores a piece of Pre and its SiLU; leaves that, as it is stored, in f.
template <typename T, int W>
__device__ __forceinline__ void store_pre_g(F2 (&f)[W / 2], T* pre, T* g) {
  Piece<T, W> p;
  p.set(f);
  p.store(pre);
#pragma unroll
  for (int k = 0; k < W / 2; ++k) f[k] = mul(f[k], sigmoid2(f[k]));
  p.set(f);
  p.store(g);
  p.get(f);
}

// CTAs [0, tg) restore U with G, O and Z (d columns a row), [tg, tg + tr) V, Q
// and K with G (3d columns a row), the others X.
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) ckpt_restore_kernel(CkptPtrs c, const T* __restrict__ gamma,
                                                                const T* __restrict__ beta, int64_t rows, int d,
                                                                int64_t tg, int64_t tr, T* __restrict__ pre,
                                                                T* __restrict__ g, float* __restrict__ o,
                                                                T* __restrict__ z, T* __restrict__ x,
                                                                float* __restrict__ mean, float* __restrict__ rstd) {
  const int64_t tile = blockIdx.x;
  if (tile < tg) {
    constexpr int W = kPiece<float>, U = kGateUnroll, kPer = kThreads * W * U;
    const int64_t base = tile * kPer;
    const int count = count_of(rows * d, base, kPer);
    const RowOf where(base, d);
    // element e of U is element e + 3d times its row of Pre
    const int64_t pbase = base + 3 * d * where.row0;
    int row[U];
    Held<W> qu[U], qd[U];
    int su[U], sd[U];
    float mu[U], rs[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (place<W>(i) >= count) continue;
      row[i] = where.rows_after(place<W>(i));
      const int at = place<W>(i) + 3 * d * row[i];
      qu[i].load(c.pre + pbase + at);
      qd[i].load(c.dev + base + place<W>(i));
      su[i] = c.pre_s[(pbase + at) / kGroup];
      sd[i] = c.dev_s[base / kGroup + place<W>(i) / kGroup];
      mu[i] = c.mean[where.row0 + row[i]];
      rs[i] = c.rstd[where.row0 + row[i]];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (place<W>(i) >= count) continue;
      const int at = place<W>(i) + 3 * d * row[i], col = where.col0 + place<W>(i) - d * row[i];
      F2 f[W / 2], dv[W / 2], out[W / 2];
      qu[i].template get<FMT>(su[i], f);
      qd[i].template get<FMT>(sd[i], dv);
      store_pre_g<T, W>(f, pre + pbase + at, g + pbase + at);
#pragma unroll
      for (int k = 0; k < W / 2; ++k) out[k] = add(both(mu[i]), dv[k]);
      Piece<float, W> po;
      po.set(out);
      po.store(o + base + place<W>(i));
#pragma unroll
      for (int k = 0; k < W / 2; ++k) out[k] = mul(dv[k], both(rs[i]));
      Piece<T, W> p;
      if (gamma) {
        F2 t[W / 2];
        p.load(gamma + col);
        p.get(t);
#pragma unroll
        for (int k = 0; k < W / 2; ++k) out[k] = mul(out[k], t[k]);
      }
      if (beta) {
        F2 t[W / 2];
        p.load(beta + col);
        p.get(t);
#pragma unroll
        for (int k = 0; k < W / 2; ++k) out[k] = add(out[k], t[k]);
      }
#pragma unroll
      for (int k = 0; k < W / 2; ++k) out[k] = mul(out[k], f[k]);
      p.set(out);
      p.store(z + base + place<W>(i));
      if (col == 0) {
        mean[where.row0 + row[i]] = mu[i];
        rstd[where.row0 + row[i]] = rs[i];
      }
    }
    return;
  }
  constexpr int W = kPiece<T>, U = kRestUnroll, kPer = kThreads * W * U;
  if (tile < tg + tr) {
    const int64_t base = (tile - tg) * kPer;
    const int count = count_of(3 * rows * d, base, kPer);
    const RowOf where(base, 3 * d);
    // element e of V|Q|K is element e + d (its row + 1) of Pre
    const int64_t pbase = base + d * (where.row0 + 1);
    int at[U], s[U];
    Held<W> q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (place<W>(i) >= count) continue;
      at[i] = place<W>(i) + d * where.rows_after(place<W>(i));
      q[i].load(c.pre + pbase + at[i]);
      s[i] = c.pre_s[(pbase + at[i]) / kGroup];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (place<W>(i) >= count) continue;
      F2 f[W / 2];
      q[i].template get<FMT>(s[i], f);
      store_pre_g<T, W>(f, pre + pbase + at[i], g + pbase + at[i]);
    }
    return;
  }
  const int64_t base = (tile - tg - tr) * kPer;
  const int count = count_of(rows * d, base, kPer);
  Held<W> q[U];
  int s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (place<W>(i) >= count) continue;
    q[i].load(c.x + base + place<W>(i));
    s[i] = c.x_s[base / kGroup + place<W>(i) / kGroup];
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (place<W>(i) >= count) continue;
    F2 f[W / 2];
    q[i].template get<FMT>(s[i], f);
    Piece<T, W> p;
    p.set(f);
    p.store(x + base + place<W>(i));
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

// Tiles of `unroll` pieces of W elements a thread in n elements.
int64_t tiles_of(int64_t n, int W, int unroll) {
  const int64_t per = (int64_t)kThreads * W * unroll;
  return (n + per - 1) / per;
}

template <typename T, int FMT>
cudaError_t launch_save(const hstu_config* c, const void* saved, int64_t rows, void* ckpt, cudaStream_t s) {
  size_t off[HSTU_SAVED_COUNT + 1];
  saved_offsets(c, rows, off);
  auto* b = static_cast<const unsigned char*>(saved);
  const int64_t n = rows * c->d_model;
  const int64_t tp = tiles_of(4 * n, kPiece<T>, kSaveUnroll), td = tiles_of(n, kPiece<float>, kSaveUnroll);
  const int64_t tx = c->io_dtype != c->dtype ? tiles_of(n, kPiece<T>, kSaveUnroll) : 0;
  if (tp + td + tx > INT32_MAX) return cudaErrorInvalidValue;
  ckpt_save_kernel<T, FMT><<<(unsigned)(tp + td + tx), kThreads, 0, s>>>(
      reinterpret_cast<const T*>(b + off[HSTU_SAVED_PRE]),
      reinterpret_cast<const float*>(b + off[HSTU_SAVED_O]),
      reinterpret_cast<const T*>(b + off[HSTU_SAVED_XLOW]),
      reinterpret_cast<const float*>(b + off[HSTU_SAVED_MEAN]),
      reinterpret_cast<const float*>(b + off[HSTU_SAVED_RSTD]), rows, c->d_model, tp, td, ckpt_ptrs(c, rows, ckpt));
  count_launch();
  return cudaGetLastError();
}

template <typename T, int FMT>
cudaError_t launch_restore(const hstu_config* c, const void* ckpt, const void* gamma, const void* beta,
                           int64_t rows, void* saved, cudaStream_t s) {
  size_t off[HSTU_SAVED_COUNT + 1];
  saved_offsets(c, rows, off);
  auto* b = static_cast<unsigned char*>(saved);
  const int64_t n = rows * c->d_model;
  const int64_t tg = tiles_of(n, kPiece<float>, kGateUnroll), tr = tiles_of(3 * n, kPiece<T>, kRestUnroll);
  const int64_t tx = c->io_dtype != c->dtype ? tiles_of(n, kPiece<T>, kRestUnroll) : 0;
  if (tg + tr + tx > INT32_MAX) return cudaErrorInvalidValue;
  ckpt_restore_kernel<T, FMT><<<(unsigned)(tg + tr + tx), kThreads, 0, s>>>(
      ckpt_ptrs(c, rows, ckpt), static_cast<const T*>(gamma), static_cast<const T*>(beta), rows, c->d_model, tg, tr,
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

#define HSTU_CKPT_DISPATCH(FN, FMT, ...) \
  (cfg->dtype == HSTU_F32 ? FN<float, FMT>(__VA_ARGS__) : FN<bf16, FMT>(__VA_ARGS__))

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
