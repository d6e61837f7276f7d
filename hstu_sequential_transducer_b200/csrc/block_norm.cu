// The joint between two blocks of a stack: the norm after a block, its gate
// and residual scale, the residual sum and the norm before the next block,
// forward and backward, in one pass over the rows.
//
//   y = x + s (.) (Norm_post(b) (.) act(u)),   h = Norm_pre(y)
//
//   e  = dy + r2 (g - mean(g) - n2 mean(g n2)),  g = dh gamma2, n2 = (y - m2) r2
//   dp = e s act(u),  du = e s p act'(u),        p = n1 gamma1 + beta1
//   db = r1 (q - mean(q) - n1 mean(q n1)),       q = dp gamma1, n1 = (b - m1) r1
//   dgamma1 += sum dp n1, dbeta1 += sum dp, ds += sum e p act(u),
//   dgamma2 += sum dh n2, dbeta2 += sum dh       (no mean(.) term for RMS)
//
// Memory-bound (a token reads 10d bytes and writes 6d in the forward, reads
// 18d and writes 8d in the backward, with bf16 operands and an fp32 residual
// stream).  A team of TPR threads, 8 columns a thread (a power of two below a
// warp, else whole warps), takes R rows at a time: 4 in the forward, 1 or 2 in
// the backward.  The columns stay the same, so the parameters are read once and
// the gradients' sums stay in registers; the R rows give the four sums that are
// joined together (4 means; 2 sums of 2 rows), at half the shuffles of four
// separate ones and one barrier.  The next rows are on their way meanwhile:
// every thread copies its own elements of them into its own slots of shared
// memory (cp.async), so the copies need no barrier.  The parameters' gradients
// are joined over the CTA's teams, written once per CTA and summed over the
// CTAs by a second kernel, always in the same order.
//
// Measured at 131,072 x 1,024, bf16 operands, fp32 residual stream: forward
// 340-343 us (6.3 TB/s; 372 with 4 resident CTAs, which takes registers from
// each), backward 547 us (6.4 TB/s; 599 with 3 CTAs; 566 with one row at a time and 4).
// With a bf16 residual stream 0.7 of the copy rate: half the bytes, but the same joins by
// the same 12 (forward) and 8 (backward) warps on a multiprocessor, which fill neither
// DRAM (45 and 54 %, at 32,768 x 1,024) nor the issue slots (54 and 50 %).
#include "args.h"
#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"

namespace hstu {
namespace {

constexpr int kParams = 5;      // post_gamma, post_beta, res_scale, pre_gamma, pre_beta
constexpr int kFwdRows = 4;     // rows that a team takes at a time in the forward
// Threads of a CTA: one team of 96 or more, else as many teams as 128 threads are.
template <int TPR> constexpr int kThreads = TPR >= 96 ? TPR : 128;
// The backward takes two rows at a time with 8 warps on a multiprocessor, whose
// registers then hold them; teams of 3, 5, 6 or 7 warps do not make 8, and take
// one row at a time with up to 16 warps (d = 1,536: 312 us instead of 348 with one
// team; d = 2,048 the other way round, 299 instead of 321).
constexpr int bwd_rows(int team) { return team == 96 || (team > 128 && team < 256) ? 1 : 2; }
// CTAs of a multiprocessor.
constexpr int fwd_resident(int threads) { return threads > 192 ? 2 : 384 / threads; }
constexpr int bwd_resident(int threads) { return bwd_rows(threads) == 1 ? 512 / threads : 256 / threads; }

// Copies B (16 or 8) bytes from src, or zeros where `any` is false.
template <int B> __device__ __forceinline__ void copy_async(void* dst, const void* src, bool any) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = any ? B : 0;
  if constexpr (B == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// W (4 or 8) elements from p as W / 2 pairs, and back.
template <int W> __device__ __forceinline__ void get(const float* p, F2* f) {
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const float4 u = reinterpret_cast<const float4*>(p)[i];
    f[2 * i] = make_float2(u.x, u.y);
    f[2 * i + 1] = make_float2(u.z, u.w);
  }
}
template <int W> __device__ __forceinline__ void get(const bf16* p, F2* f) {
  uint2 u[W / 4];
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(u) = *reinterpret_cast<const uint4*>(p);
  else
    u[0] = *reinterpret_cast<const uint2*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(u);
#pragma unroll
  for (int i = 0; i < W / 2; ++i) f[i] = __bfloat1622float2(h[i]);
}
template <int W> __device__ __forceinline__ void put(float* p, const F2* f) {
#pragma unroll
  for (int i = 0; i < W / 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
}
template <int W> __device__ __forceinline__ void put(bf16* p, const F2* f) {
  uint2 u[W / 4];
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(u);
#pragma unroll
  for (int i = 0; i < W / 2; ++i) h[i] = __floats2bfloat162_rn(f[i].x, f[i].y);
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(u);
  else
    *reinterpret_cast<uint2*>(p) = u[0];
}
// As they are stored in T.
template <typename T> __device__ __forceinline__ F2 rounded(F2 a) {
  return make_float2(to_f(from_f<T>(a.x)), to_f(from_f<T>(a.y)));
}

// The 8 columns of a team's thread, in P parts of W: neighbouring threads hold
// neighbouring parts, and a part is 16 bytes of the residual stream's type, so
// that a warp's access covers whole 32-byte sectors (8 fp32 columns in a row
// would be two accesses of half sectors: 458 and 813 us instead of 372 and 599).
template <typename IO, int TPR> struct Columns {
  static constexpr int W = 16 / (int)sizeof(IO), P = 8 / W, NT = kThreads<TPR>;
  int col[P];
  bool has[P];
  __device__ __forceinline__ Columns(int lane, int d) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      col[j] = W * (lane + TPR * j);
      has[j] = col[j] < d;
    }
  }
  // A row's elements of this thread into its slots of an array (8 NT elements), or zeros; and back.
  template <typename T> __device__ __forceinline__ void fetch(T* slots, const T* row, bool any) const {
#pragma unroll
    for (int j = 0; j < P; ++j)
      copy_async<W * (int)sizeof(T)>(slots + (j * NT + threadIdx.x) * W, row + (has[j] ? col[j] : 0), any && has[j]);
  }
  template <typename T> __device__ __forceinline__ void take(const T* slots, F2 (&f)[4]) const {
#pragma unroll
    for (int j = 0; j < P; ++j) get<W>(slots + (j * NT + threadIdx.x) * W, f + j * (W / 2));
  }
  template <typename T> __device__ __forceinline__ void store(T* row, const F2 (&f)[4]) const {
#pragma unroll
    for (int j = 0; j < P; ++j)
      if (has[j]) put<W>(row + col[j], f + j * (W / 2));
  }
};

// A parameter's elements, kept packed in their own type; `other` without it, zeros past d.
template <typename T, typename IO, int TPR> struct Param {
  static constexpr int W = Columns<IO, TPR>::W, P = 8 / W;
  __align__(16) T v[8];
  __device__ __forceinline__ void load(const T* p, const Columns<IO, TPR>& c, float other) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (p && c.has[j]) {
        if constexpr (W * sizeof(T) == 16)
          *reinterpret_cast<uint4*>(v + j * W) = *reinterpret_cast<const uint4*>(p + c.col[j]);
        else
          *reinterpret_cast<uint2*>(v + j * W) = *reinterpret_cast<const uint2*>(p + c.col[j]);
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k) v[j * W + k] = from_f<T>(c.has[j] ? other : 0.f);
      }
    }
  }
  __device__ __forceinline__ void pairs(F2 (&f)[4]) const { get<8>(v, f); }
};

template <int TPR> struct Team {
  static constexpr int kTeams = kThreads<TPR> / TPR;
  static constexpr int kWarps = TPR > 32 ? TPR / 32 : 1;
  // Joins N (1, 2 or 4) sums over the team's threads; all of them get the
  // totals.  log2 N exchanges leave each of N groups of lanes with one of the sums.
  // slot: the team's 2 x kWarps x 4 floats; flip alternates, so that a slot
  // is rewritten only after a barrier that follows its last read.
  template <int N> static __device__ __forceinline__ void join(float (&v)[N], float (*slot)[4], int& flip, int team) {
    constexpr int L = TPR < 32 ? TPR : 32, G = L / N;        // lanes that share a sum, at least 1
    const int lane = threadIdx.x & 31;
    float t = v[0];
    if constexpr (N == 4) {
      const bool upper = lane & (L / 2), odd = lane & (L / 4);
      const float a = (upper ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[2], L / 2);
      const float b = (upper ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, upper ? v[1] : v[3], L / 2);
      t = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, L / 4);
    } else if constexpr (N == 2) {
      const bool upper = lane & (L / 2);
      t = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], L / 2);
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if constexpr (TPR <= 32) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = N == 1 ? t : __shfl_sync(0xffffffffu, t, i * G, L);
    } else {
      float(*const s)[4] = slot + flip * kWarps;
      flip ^= 1;
      if (lane % G == 0) s[(threadIdx.x % TPR) / 32][lane / G] = t;
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(TPR) : "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = s[0][i];
#pragma unroll
      for (int k = 1; k < kWarps; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += s[k][i];
    }
  }
};

// act(u) and act'(u), in place of u.
__device__ __forceinline__ void gate8(int act, F2 (&u)[4], F2 (&slope)[4]) {
  if (act == HSTU_GATE_NONE) {
#pragma unroll
    for (int k = 0; k < 4; ++k) slope[k] = both(1.f);
  } else if (act == HSTU_GATE_SIGMOID) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const F2 s = sigmoid2(u[k]);
      u[k] = s;
      slope[k] = mul(s, fma(s, both(-1.f), both(1.f)));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const F2 s = sigmoid2(u[k]);
      slope[k] = mul(s, fma(u[k], fma(s, both(-1.f), both(1.f)), both(1.f)));
      u[k] = mul(u[k], s);
    }
  }
}

template <typename T>
struct FwdArgs {
  int post, pre, act, d;
  float eps;
  const T *gamma1, *beta1, *scale, *gamma2, *beta2;
  const T* gate;
  int64_t gate_stride, rows;
  T* h;
  float4* stats;
};

// Bytes of a row's slots: b, x, u of the forward; dy, dh, y, b, u of the backward.
template <typename T, typename IO, int TPR>
constexpr int kFwdSlots = 8 * (2 * (int)sizeof(IO) + (int)sizeof(T)) * kThreads<TPR>;
template <typename T, typename IO, int TPR>
constexpr int kBwdSlots = 8 * (4 * (int)sizeof(IO) + (int)sizeof(T)) * kThreads<TPR>;

// T: operand type; IO: residual stream's type.
template <typename T, typename IO, int TPR>
__global__ void __launch_bounds__(kThreads<TPR>, fwd_resident(kThreads<TPR>)) block_norm_fwd_kernel(FwdArgs<T> p, const IO* x,
                                                                                const IO* __restrict__ b, IO* y) {
  using W = Team<TPR>;
  constexpr int NT = kThreads<TPR>, R = kFwdRows, kRow = kFwdSlots<T, IO, TPR>;
  extern __shared__ __align__(16) unsigned char ring[];
  // row i's slots of b, x and u
  auto at_b = [&](int i) { return reinterpret_cast<IO*>(ring + i * kRow); };
  auto at_x = [&](int i) { return reinterpret_cast<IO*>(ring + i * kRow) + 8 * NT; };
  auto at_u = [&](int i) { return reinterpret_cast<T*>(at_x(i) + 8 * NT); };
  __shared__ __align__(16) float sums[W::kTeams][2 * W::kWarps][4];
  const int team = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const int d = p.d;
  const Columns<IO, TPR> cols(lane, d);
  const float inv_d = 1.f / (float)d;
  float(*const own)[4] = sums[team];
  int flip = 0;
  // a CTA's teams take the same number of steps; rows [base, base + kRows) are the CTA's next ones
  constexpr int kRows = W::kTeams * R;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t base = (int64_t)blockIdx.x * kRows;
  // The two parts of a step's copies, b and then u and x.  Rows past the end
  // keep what their slots held; nothing that comes of it is kept.
  auto fetch_b = [&](int64_t next) {
    if (b) {
      const bool full = next + kRows <= p.rows;
      const int64_t r0 = next + team * R;
      const IO* pb = b + r0 * d;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (full || r0 + i < p.rows) cols.fetch(at_b(i), pb, true);
        pb += d;
      }
    }
    copy_commit();
  };
  auto fetch_x = [&](int64_t next) {
    const bool full = next + kRows <= p.rows;
    const int64_t r0 = next + team * R;
    const IO* px = x + r0 * d;
    const T* pu = p.gate + r0 * p.gate_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (full || r0 + i < p.rows) {
        cols.fetch(at_x(i), px, true);
        if (p.gate) cols.fetch(at_u(i), pu, true);
      }
      px += d;
      pu += p.gate_stride;
    }
    copy_commit();
  };
  // mean and 1/spread of R rows
  auto row_stats = [&](int kind, const F2 (&v)[R][4], float (&m)[R], float (&r)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) m[i] = r[i] = 0.f;
    if (kind == HSTU_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        F2 t = both(0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (cols.has[k * cols.P / 4]) t = add(t, v[i][k]);
        m[i] = t.x + t.y;
      }
      W::join(m, own, flip, team);
#pragma unroll
      for (int i = 0; i < R; ++i) m[i] *= inv_d;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      F2 t = both(0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (cols.has[k * cols.P / 4]) {
          const F2 c = add(v[i][k], both(-m[i]));
          t = fma(c, c, t);
        }
      r[i] = t.x + t.y;
    }
    W::join(r, own, flip, team);
#pragma unroll
    for (int i = 0; i < R; ++i) r[i] = rsqrtf(r[i] * inv_d + p.eps);
  };
  using Par = Param<T, IO, TPR>;
  auto normalise = [&](F2 (&v)[R][4], const float (&m)[R], const float (&r)[R], const Par& gamma, const Par& beta) {
    F2 g[4], bt[4];
    gamma.pairs(g);
    beta.pairs(bt);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] = fma(mul(add(v[i][k], both(-m[i])), both(r[i])), g[k], bt[k]);
  };
  fetch_b(base);
  fetch_x(base);
  Par gamma1, beta1, scale, gamma2, beta2;
  gamma1.load(p.gamma1, cols, 1.f);
  beta1.load(p.beta1, cols, 0.f);
  scale.load(p.scale, cols, 1.f);
  gamma2.load(p.gamma2, cols, 1.f);
  beta2.load(p.beta2, cols, 0.f);
  for (; base < p.rows; base += step) {
    const int64_t r0 = base + team * R;
    const bool full = base + kRows <= p.rows;
    copy_wait<1>();                    // b is here
    F2 v[R][4];
    float m1[R], r1[R], m2[R], r2[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m1[i] = m2[i] = 0.f;
      r1[i] = r2[i] = 1.f;
    }
    if (b) {
#pragma unroll
      for (int i = 0; i < R; ++i) cols.take(at_b(i), v[i]);
      if (p.post != HSTU_NORM_NONE) {
        row_stats(p.post, v, m1, r1);
        // a part's slots are free once its values have gone into a sum or a store
        fetch_b(base + step);
        normalise(v, m1, r1, gamma1, beta1);
        copy_wait<1>();                // u and x are here
      } else {
        copy_wait<0>();
      }
      F2 sc[4];
      scale.pairs(sc);
      IO* py = y + r0 * d;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        F2 u[4], slope[4];
        if (p.gate) {
          cols.take(at_u(i), u);
          gate8(p.act, u, slope);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[i][k] = mul(v[i][k], u[k]);
        }
        cols.take(at_x(i), u);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = rounded<IO>(fma(sc[k], v[i][k], u[k]));
        if (full || r0 + i < p.rows) cols.store(py, v[i]);
        py += d;
      }
      if (p.post == HSTU_NORM_NONE) fetch_b(base + step);
      fetch_x(base + step);
      if (p.h && p.pre != HSTU_NORM_NONE) row_stats(p.pre, v, m2, r2);
    } else {
      copy_wait<0>();
#pragma unroll
      for (int i = 0; i < R; ++i) cols.take(at_x(i), v[i]);
      if (p.h && p.pre != HSTU_NORM_NONE) row_stats(p.pre, v, m2, r2);
      fetch_b(base + step);
      fetch_x(base + step);
    }
    if (p.h) {
      if (p.pre != HSTU_NORM_NONE) normalise(v, m2, r2, gamma2, beta2);
      T* ph = p.h + r0 * d;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (full || r0 + i < p.rows) cols.store(ph, v[i]);
        ph += d;
      }
    }
    if (p.stats && lane == 0)
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (full || r0 + i < p.rows) p.stats[r0 + i] = make_float4(m1[i], r1[i], m2[i], r2[i]);
  }
}

struct GradPtrs {
  float* p[kParams];
};

template <typename T>
struct BwdArgs {
  int post, pre, act, d;
  const T *gamma1, *beta1, *scale, *gamma2;
  const T* gate;
  int64_t gate_stride, rows;
  const float4* stats;
  T *db, *dgate;
  int64_t dgate_stride;
  float* partial;               // [gridDim.x][5][d]; NULL: not wanted, or one CTA
  GradPtrs grads;               // where a single CTA adds its sums
};

template <typename T, typename IO, int TPR>
__global__ void __launch_bounds__(kThreads<TPR>, bwd_resident(kThreads<TPR>)) block_norm_bwd_kernel(
    BwdArgs<T> p, const IO* __restrict__ y, const IO* __restrict__ b, const IO* dy, const IO* __restrict__ dh,
    IO* dx) {
  using W = Team<TPR>;
  constexpr int NT = kThreads<TPR>, R = bwd_rows(TPR), kRow = kBwdSlots<T, IO, TPR>;
  extern __shared__ __align__(16) unsigned char ring[];
  // row i's slots of dy, dh, y and b (array 0 .. 3) and of u
  auto at = [&](int i, int array) { return reinterpret_cast<IO*>(ring + i * kRow) + array * 8 * NT; };
  auto at_u = [&](int i) { return reinterpret_cast<T*>(at(i, 4)); };
  __shared__ __align__(16) float sums[W::kTeams][2 * W::kWarps][4];
  const int team = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const int d = p.d;
  const Columns<IO, TPR> cols(lane, d);
  const float inv_d = 1.f / (float)d;
  float(*const own)[4] = sums[team];
  int flip = 0;
  // a CTA's teams take the same number of steps; rows [base, base + kRows) are the CTA's next ones
  constexpr int kRows = W::kTeams * R;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t base = (int64_t)blockIdx.x * kRows;
  // The two parts of a step's copies: what gives e, and what it is passed on
  // to.  Rows past the end are zeros (the copy's source is row 0, of which it
  // reads nothing).
  auto fetch_e = [&](int64_t next) {
    const bool full = next + kRows <= p.rows;
    const int64_t r0 = next + team * R;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool row = full || r0 + i < p.rows;
      const int64_t off = row ? (r0 + i) * d : 0;
      if (dy) cols.fetch(at(i, 0), dy + off, row);
      if (dh) {
        cols.fetch(at(i, 1), dh + off, row);
        cols.fetch(at(i, 2), y + off, row);
      }
    }
    copy_commit();
  };
  auto fetch_b = [&](int64_t next) {
    if (b) {
      const bool full = next + kRows <= p.rows;
      const int64_t r0 = next + team * R;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool row = full || r0 + i < p.rows;
        const int64_t r = row ? r0 + i : 0;
        cols.fetch(at(i, 3), b + r * d, row);
        if (p.gate) cols.fetch(at_u(i), p.gate + r * p.gate_stride, row);
      }
    }
    copy_commit();
  };
  fetch_e(base);
  fetch_b(base);
  F2 acc[kParams][4];
#pragma unroll
  for (int i = 0; i < kParams; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[i][k] = both(0.f);
  Param<T, IO, TPR> gamma1, beta1, scale, gamma2;
  gamma1.load(p.gamma1, cols, 1.f);
  beta1.load(p.beta1, cols, 0.f);
  scale.load(p.scale, cols, 1.f);
  gamma2.load(p.gamma2, cols, 1.f);
  float4 next[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = base + team * R + i;
    next[i] = r < p.rows ? p.stats[r] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (; base < p.rows; base += step) {
    const int64_t r0 = base + team * R;
    const bool full = base + kRows <= p.rows;
    float4 st[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      st[i] = next[i];
      next[i] = r0 + step + i < p.rows ? p.stats[r0 + step + i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    copy_wait<1>();                    // dy, dh and y are here
    // Without a row all inputs and statistics are 0, and so is what is summed.
    // Past d the inputs and s are 0: e is not, but nothing of it is passed on.
    F2 e[R][4], up[R][4], n[R][4], lo[R], hi[R];
    float t[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) e[i][k] = up[i][k] = both(0.f);
      if (dy) cols.take(at(i, 0), e[i]);
      if (dh) cols.take(at(i, 1), up[i]);
    }
    if (dh && p.pre != HSTU_NORM_NONE) {
      F2 g[4];
      gamma2.pairs(g);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        cols.take(at(i, 2), n[i]);
        lo[i] = hi[i] = both(0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          n[i][k] = mul(add(n[i][k], both(-st[i].z)), both(st[i].w));
          acc[3][k] = fma(up[i][k], n[i][k], acc[3][k]);
          acc[4][k] = add(acc[4][k], up[i][k]);
          up[i][k] = mul(up[i][k], g[k]);
          lo[i] = add(lo[i], up[i][k]);
          hi[i] = fma(up[i][k], n[i][k], hi[i]);
        }
        t[2 * i] = lo[i].x + lo[i].y;
        t[2 * i + 1] = hi[i].x + hi[i].y;
      }
      W::join(t, own, flip, team);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const F2 level = both(p.pre == HSTU_NORM_LAYER ? -t[2 * i] * inv_d : 0.f), along = both(-t[2 * i + 1] * inv_d);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          e[i][k] = fma(add(fma(n[i][k], along, up[i][k]), level), both(st[i].w), e[i][k]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) e[i][k] = add(e[i][k], up[i][k]);
    }
    if (dx)
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (full || r0 + i < p.rows) cols.store(dx + (r0 + i) * d, e[i]);
    // a part's slots are free once its values have been taken: a thread's loads come before
    // the copies that it starts after them
    fetch_e(base + step);
    copy_wait<1>();                    // b and u are here
    if (b) {
      F2 g[4], bt[4], sc[4];
      gamma1.pairs(g);
      beta1.pairs(bt);
      scale.pairs(sc);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        F2 u[4], slope[4];
        cols.take(at(i, 3), n[i]);
        if (p.gate) {
          cols.take(at_u(i), u);
          gate8(p.act, u, slope);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            u[k] = both(1.f);
            slope[k] = both(0.f);
          }
        }
        lo[i] = hi[i] = both(0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          F2 v = n[i][k];
          if (p.post != HSTU_NORM_NONE) {
            n[i][k] = mul(add(n[i][k], both(-st[i].x)), both(st[i].y));
            v = fma(n[i][k], g[k], bt[k]);
          }
          const F2 dv = mul(e[i][k], sc[k]);
          acc[2][k] = fma(e[i][k], mul(v, u[k]), acc[2][k]);
          slope[k] = mul(mul(dv, v), slope[k]);     // du
          e[i][k] = mul(dv, u[k]);                  // dp
          if (p.post != HSTU_NORM_NONE) {
            acc[0][k] = fma(e[i][k], n[i][k], acc[0][k]);
            acc[1][k] = add(acc[1][k], e[i][k]);
            e[i][k] = mul(e[i][k], g[k]);
            lo[i] = add(lo[i], e[i][k]);
            hi[i] = fma(e[i][k], n[i][k], hi[i]);
          }
        }
        t[2 * i] = lo[i].x + lo[i].y;
        t[2 * i + 1] = hi[i].x + hi[i].y;
        if ((full || r0 + i < p.rows) && p.gate && p.dgate) cols.store(p.dgate + (r0 + i) * p.dgate_stride, slope);
      }
      if (p.post != HSTU_NORM_NONE) W::join(t, own, flip, team);
    }
    fetch_b(base + step);
    if (b && p.db)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (p.post != HSTU_NORM_NONE) {
          const F2 level = both(p.post == HSTU_NORM_LAYER ? -t[2 * i] * inv_d : 0.f), along = both(-t[2 * i + 1] * inv_d);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            e[i][k] = mul(add(fma(n[i][k], along, e[i][k]), level), both(st[i].y));
        }
        if (full || r0 + i < p.rows) cols.store(p.db + (r0 + i) * d, e[i]);
      }
  }
  if (W::kTeams == 1 && p.partial) {
#pragma unroll
    for (int i = 0; i < kParams; ++i) cols.store(p.partial + ((int64_t)blockIdx.x * kParams + i) * d, acc[i]);
    return;
  }
  // joins the teams' sums in the ring, whose last copies hold nothing
  copy_wait<0>();
  float* const all = reinterpret_cast<float*>(ring);          // [kTeams][8 TPR]
  for (int i = 0; i < kParams; ++i) {
    float* const add_to = p.partial ? nullptr : p.grads.p[i];
    if (!p.partial && !add_to) continue;
    __syncthreads();
    cols.store(all + team * 8 * TPR, acc[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += NT) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < W::kTeams; ++w) t += all[w * 8 * TPR + c];
      if (p.partial) p.partial[((int64_t)blockIdx.x * kParams + i) * d + c] = t;
      else add_to[c] += t;
    }
  }
}

// grads.p[i][c] += sum over the CTAs of partial[cta][i][c], in the order of
// the CTAs within each of 32 strips, then of the strips.  Parameters that share
// a gradient (two norms with one gamma) are added one after another by the
// CTAs of the first.
constexpr int kStrips = 32;
__global__ void __launch_bounds__(32 * kStrips) block_norm_join_kernel(const float* __restrict__ partial, int ctas,
                                                                       int d, GradPtrs grads) {
  __shared__ float strip[kStrips][32];
  const int first = blockIdx.y;
  float* const out = grads.p[first];
  if (!out) return;
  for (int i = 0; i < first; ++i)
    if (grads.p[i] == out) return;
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  for (int i = first; i < kParams; ++i) {
    if (grads.p[i] != out) continue;
    const float* src = partial + (int64_t)i * d + c;
    float t = 0.f;
    if (c < d)
#pragma unroll 4
      for (int k = w; k < ctas; k += kStrips) t += src[(int64_t)k * kParams * d];
    strip[w][lane] = t;
    __syncthreads();
    if (w == 0 && c < d) {
#pragma unroll
      for (int k = 1; k < kStrips; ++k) t += strip[k][lane];
      out[c] += t;
    }
    __syncthreads();
  }
}

// Threads of a team, 8 columns each: a power of two below a warp, else warps.
int team_threads(int d) {
  if (d > 256) return (d + 255) / 256 * 32;
  int t = 4;
  while (8 * t < d) t *= 2;
  return t;
}

// CTAs that have rows, at most those that are resident (the backward's workspace
// holds a partial sum of each).
int64_t ctas_of(int d, int64_t T, int rows, int (*resident)(int)) {
  const int team = team_threads(d), threads = team >= 96 ? team : 128, teams = threads / team;
  const int64_t want = (T + teams * rows - 1) / (teams * rows), cap = (int64_t)sm_count() * resident(threads);
  return want < cap ? want : cap;
}
// Two steps are left to one CTA, which adds its sums to the gradients itself
// (4 rows of 1,024: 27 us a call and 9.0 us a graph node; two CTAs and the
// joining launch 30 and 8.3; with three steps the graph's node takes 10.5 and 8.9).
constexpr int kOneCta = 2;
int64_t bwd_ctas(int d, int64_t T) {
  const int64_t ctas = ctas_of(d, T, bwd_rows(team_threads(d)), bwd_resident);
  return ctas <= kOneCta ? 1 : ctas;
}

// 48 KB, the kernel's static arrays included, need no permission.
template <typename K> cudaError_t allow_shared(K* kernel, int bytes) {
  return bytes > 40 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
                           : cudaSuccess;
}

template <typename T, typename IO, int TPR>
cudaError_t launch_fwd(const FwdArgs<T>& p, const void* x, const void* b, void* y, cudaStream_t s) {
  constexpr int kBytes = kFwdRows * kFwdSlots<T, IO, TPR>;
  cudaError_t e = allow_shared(block_norm_fwd_kernel<T, IO, TPR>, kBytes);
  if (e != cudaSuccess) return e;
  const int64_t ctas = ctas_of(p.d, p.rows, kFwdRows, fwd_resident);
  block_norm_fwd_kernel<T, IO, TPR><<<(unsigned)ctas, kThreads<TPR>, kBytes, s>>>(
      p, static_cast<const IO*>(x), static_cast<const IO*>(b), static_cast<IO*>(y));
  count_launch();
  return cudaGetLastError();
}

template <typename T, typename IO>
cudaError_t run_fwd(const hstu_config* c, const hstu_block_norm* n, const void* x, const void* b,
                    const void* gate, int64_t gate_stride, int64_t T_, void* y, void* h, float* stats,
                    cudaStream_t s) {
  FwdArgs<T> p;
  p.post = n->post_kind; p.pre = n->pre_kind; p.act = n->gate_act; p.d = c->d_model; p.eps = c->ln_eps;
  p.gamma1 = static_cast<const T*>(n->post_gamma); p.beta1 = static_cast<const T*>(n->post_beta);
  p.scale = static_cast<const T*>(n->res_scale);
  p.gamma2 = static_cast<const T*>(n->pre_gamma); p.beta2 = static_cast<const T*>(n->pre_beta);
  p.gate = b ? static_cast<const T*>(gate) : nullptr; p.gate_stride = gate_stride; p.rows = T_;
  p.h = static_cast<T*>(h); p.stats = reinterpret_cast<float4*>(stats);
  switch (team_threads(p.d)) {
    case 4: return launch_fwd<T, IO, 4>(p, x, b, y, s);
    case 8: return launch_fwd<T, IO, 8>(p, x, b, y, s);
    case 16: return launch_fwd<T, IO, 16>(p, x, b, y, s);
    case 32: return launch_fwd<T, IO, 32>(p, x, b, y, s);
    case 64: return launch_fwd<T, IO, 64>(p, x, b, y, s);
    case 96: return launch_fwd<T, IO, 96>(p, x, b, y, s);
    case 128: return launch_fwd<T, IO, 128>(p, x, b, y, s);
    case 160: return launch_fwd<T, IO, 160>(p, x, b, y, s);
    case 192: return launch_fwd<T, IO, 192>(p, x, b, y, s);
    case 224: return launch_fwd<T, IO, 224>(p, x, b, y, s);
    default: return launch_fwd<T, IO, 256>(p, x, b, y, s);
  }
}

template <typename T, typename IO, int TPR>
cudaError_t launch_bwd(BwdArgs<T> p, const void* y, const void* b, const void* dy, const void* dh,
                       void* dx, const GradPtrs& grads, cudaStream_t s) {
  constexpr int kBytes = bwd_rows(TPR) * kBwdSlots<T, IO, TPR>;
  cudaError_t e = allow_shared(block_norm_bwd_kernel<T, IO, TPR>, kBytes);
  if (e != cudaSuccess) return e;
  const int ctas = (int)bwd_ctas(p.d, p.rows);
  p.grads = grads;
  if (ctas == 1) p.partial = nullptr;
  block_norm_bwd_kernel<T, IO, TPR><<<(unsigned)ctas, kThreads<TPR>, kBytes, s>>>(
      p, static_cast<const IO*>(y), static_cast<const IO*>(b), static_cast<const IO*>(dy),
      static_cast<const IO*>(dh), static_cast<IO*>(dx));
  count_launch();
  e = cudaGetLastError();
  if (e == cudaSuccess && p.partial) {
    block_norm_join_kernel<<<dim3((unsigned)((p.d + 31) / 32), kParams), 32 * kStrips, 0, s>>>(p.partial, ctas, p.d, grads);
    count_launch();
    e = cudaGetLastError();
  }
  return e;
}

template <typename T, typename IO>
cudaError_t run_bwd(const hstu_config* c, const hstu_block_norm* n, const void* y, const void* b,
                    const void* gate, int64_t gate_stride, const float* stats, const void* dy, const void* dh,
                    int64_t T_, void* dx, void* db, void* dgate, int64_t dgate_stride, const GradPtrs& grads,
                    float* partial, cudaStream_t s) {
  BwdArgs<T> p;
  p.post = n->post_kind; p.pre = n->pre_kind; p.act = n->gate_act; p.d = c->d_model;
  p.gamma1 = static_cast<const T*>(n->post_gamma); p.beta1 = static_cast<const T*>(n->post_beta);
  p.scale = static_cast<const T*>(n->res_scale); p.gamma2 = static_cast<const T*>(n->pre_gamma);
  p.gate = b ? static_cast<const T*>(gate) : nullptr; p.gate_stride = gate_stride; p.rows = T_;
  p.stats = reinterpret_cast<const float4*>(stats);
  p.db = static_cast<T*>(db); p.dgate = static_cast<T*>(dgate); p.dgate_stride = dgate_stride;
  p.partial = partial;
  switch (team_threads(p.d)) {
    case 4: return launch_bwd<T, IO, 4>(p, y, b, dy, dh, dx, grads, s);
    case 8: return launch_bwd<T, IO, 8>(p, y, b, dy, dh, dx, grads, s);
    case 16: return launch_bwd<T, IO, 16>(p, y, b, dy, dh, dx, grads, s);
    case 32: return launch_bwd<T, IO, 32>(p, y, b, dy, dh, dx, grads, s);
    case 64: return launch_bwd<T, IO, 64>(p, y, b, dy, dh, dx, grads, s);
    case 96: return launch_bwd<T, IO, 96>(p, y, b, dy, dh, dx, grads, s);
    case 128: return launch_bwd<T, IO, 128>(p, y, b, dy, dh, dx, grads, s);
    case 160: return launch_bwd<T, IO, 160>(p, y, b, dy, dh, dx, grads, s);
    case 192: return launch_bwd<T, IO, 192>(p, y, b, dy, dh, dx, grads, s);
    case 224: return launch_bwd<T, IO, 224>(p, y, b, dy, dh, dx, grads, s);
    default: return launch_bwd<T, IO, 256>(p, y, b, dy, dh, dx, grads, s);
  }
}

hstu_status check_block_norm(const hstu_config* c, const hstu_block_norm* n) {
  HSTU_TRY(check_cfg(c));
  if (!n || n->reserved != 0) return HSTU_ERR_INVALID;
  if (n->post_kind < HSTU_NORM_NONE || n->post_kind > HSTU_NORM_RMS) return HSTU_ERR_INVALID;
  if (n->pre_kind < HSTU_NORM_NONE || n->pre_kind > HSTU_NORM_RMS) return HSTU_ERR_INVALID;
  if (n->gate_act < HSTU_GATE_NONE || n->gate_act > HSTU_GATE_SILU) return HSTU_ERR_INVALID;
  HSTU_TRY(opt(n->post_gamma));
  HSTU_TRY(opt(n->post_beta));
  HSTU_TRY(opt(n->res_scale));
  HSTU_TRY(opt(n->pre_gamma));
  HSTU_TRY(opt(n->pre_beta));
  return HSTU_OK;
}

// An optional [T][d] array whose rows are `stride` operand elements apart.
hstu_status check_strided(const hstu_config* c, const void* p, int64_t stride) {
  if (!p) return HSTU_OK;
  if (stride < c->d_model) return HSTU_ERR_INVALID;
  if (stride * dtype_size(c->dtype) % 16 != 0) return HSTU_ERR_UNSUPPORTED;
  return opt(p);
}

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

size_t hstu_block_norm_bwd_workspace_size(const hstu_config* cfg, int64_t T) {
  if (check_cfg(cfg) != HSTU_OK || T <= 0) return 0;
  return (size_t)bwd_ctas(cfg->d_model, T) * kParams * (size_t)cfg->d_model * sizeof(float);
}

hstu_status hstu_block_norm_fwd(const hstu_config* cfg, const hstu_block_norm* bn, const void* x,
                                const void* b, const void* gate, int64_t gate_stride, int64_t T, void* y,
                                void* h, float* stats, cudaStream_t stream) {
  HSTU_TRY(check_block_norm(cfg, bn));
  if (T < 0) return HSTU_ERR_INVALID;
  HSTU_TRY(need(x, T));
  HSTU_TRY(opt(b));
  if (b) HSTU_TRY(need(y, T));
  HSTU_TRY(check_strided(cfg, b ? gate : nullptr, gate_stride));
  HSTU_TRY(opt(h));
  HSTU_TRY(opt(stats));
  if (T == 0 || (!b && !h && !stats)) return HSTU_OK;
  prof_begin(HSTU_K_BLOCK_NORM, stream);
  cudaError_t e;
  if (cfg->dtype == HSTU_F32)
    e = run_fwd<float, float>(cfg, bn, x, b, gate, gate_stride, T, y, h, stats, stream);
  else if (cfg->io_dtype == HSTU_F32)
    e = run_fwd<bf16, float>(cfg, bn, x, b, gate, gate_stride, T, y, h, stats, stream);
  else
    e = run_fwd<bf16, bf16>(cfg, bn, x, b, gate, gate_stride, T, y, h, stats, stream);
  prof_end(HSTU_K_BLOCK_NORM, stream);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

hstu_status hstu_block_norm_bwd(const hstu_config* cfg, const hstu_block_norm* bn, const void* y,
                                const void* b, const void* gate, int64_t gate_stride, const float* stats,
                                const void* dy, const void* dh, int64_t T, void* dx, void* db, void* dgate,
                                int64_t dgate_stride, const hstu_block_norm_grads* grads, void* workspace,
                                size_t ws_bytes, cudaStream_t stream) {
  HSTU_TRY(check_block_norm(cfg, bn));
  if (T < 0) return HSTU_ERR_INVALID;
  if (dh) HSTU_TRY(need(y, T));
  HSTU_TRY(opt(b));
  HSTU_TRY(check_strided(cfg, b ? gate : nullptr, gate_stride));
  HSTU_TRY(check_strided(cfg, b && gate ? dgate : nullptr, dgate_stride));
  HSTU_TRY(need(stats, T));
  HSTU_TRY(opt(dy));
  HSTU_TRY(opt(dh));
  HSTU_TRY(opt(dx));
  HSTU_TRY(opt(db));
  GradPtrs g = {};
  bool any = false;
  if (grads) {
    float* const all[kParams] = {grads->post_gamma, grads->post_beta, grads->res_scale, grads->pre_gamma,
                                 grads->pre_beta};
    const int kind[kParams] = {bn->post_kind, bn->post_kind, HSTU_NORM_LAYER, bn->pre_kind, bn->pre_kind};
    for (int i = 0; i < kParams; ++i) {
      HSTU_TRY(meta(all[i], all[i] ? 1 : 0, 4));
      g.p[i] = kind[i] != HSTU_NORM_NONE ? all[i] : nullptr;
      any = any || g.p[i];
      // the same array, or apart
      for (int k = 0; k < i; ++k) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(all[i]), b = reinterpret_cast<uintptr_t>(all[k]);
        if (all[i] && all[k] && a != b && (a < b ? b - a : a - b) < (size_t)cfg->d_model * sizeof(float))
          return HSTU_ERR_INVALID;
      }
    }
  }
  if (T == 0) return HSTU_OK;
  if (any) {
    if (ws_bytes < hstu_block_norm_bwd_workspace_size(cfg, T)) return HSTU_ERR_WORKSPACE;
    HSTU_TRY(need(workspace, 1));
  }
  float* partial = any ? static_cast<float*>(workspace) : nullptr;
  prof_begin(HSTU_K_BLOCK_NORM, stream);
  cudaError_t e;
  if (cfg->dtype == HSTU_F32)
    e = run_bwd<float, float>(cfg, bn, y, b, gate, gate_stride, stats, dy, dh, T, dx, db, dgate, dgate_stride, g,
                              partial, stream);
  else if (cfg->io_dtype == HSTU_F32)
    e = run_bwd<bf16, float>(cfg, bn, y, b, gate, gate_stride, stats, dy, dh, T, dx, db, dgate, dgate_stride, g,
                             partial, stream);
  else
    e = run_bwd<bf16, bf16>(cfg, bn, y, b, gate, gate_stride, stats, dy, dh, T, dx, db, dgate, dgate_stride, g,
                            partial, stream);
  prof_end(HSTU_K_BLOCK_NORM, stream);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
