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
// 16d and writes 8d in the backward, with bf16 operands and an fp32 residual
// stream).  A row is held in registers, 8 elements a thread, by the WPR warps
// of a team; its statistics are joined by shuffles and, for several warps, through
// shared memory.  A thread keeps the same columns for all its rows, so the
// parameters' gradients are summed in its registers, joined over the CTA's teams,
// written once per CTA and summed over the CTAs by a second kernel, always in
// the same order.
#include "args.h"
#include "common.cuh"
#include "internal.h"

namespace hstu {
namespace {

constexpr int kThreads = 256;
constexpr int kParams = 5;      // post_gamma, post_beta, res_scale, pre_gamma, pre_beta

// Joins v[0..N) over the WPR warps of a team; all its threads get the sums.
// slot: 2 x N x WPR floats of the team; *flip alternates, so that a slot is
// rewritten only after a barrier that follows its last read.
template <int WPR, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float* slot, int& flip, int team, int wid) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (WPR == 1) return;
  float* const s = slot + flip * N * WPR;
  flip ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i * WPR + wid] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(WPR * 32) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) t += s[i * WPR + w];
    v[i] = t;
  }
}

// act(u) and act'(u).
__device__ __forceinline__ void gate_of(int act, float u, float& a, float& da) {
  if (act == HSTU_GATE_NONE) {
    a = u;
    da = 1.f;
    return;
  }
  const float s = 1.f / (1.f + __expf(-u));
  if (act == HSTU_GATE_SIGMOID) {
    a = s;
    da = s * (1.f - s);
  } else {
    a = u * s;
    da = s * (1.f + u * (1.f - s));
  }
}

template <typename T>
__device__ __forceinline__ void param8(const T* p, int col, float other, float (&f)[8]) {
  if (p) {
    load8(p + col, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = other;
  }
}

// Mean and 1/spread of a team's row; elements past d (live false) are left out.
template <int WPR>
__device__ __forceinline__ void row_stats(int kind, const float (&a)[8], bool live, float inv_d, float eps,
                                          float* slot, int& flip, int team, int wid, float& m, float& r) {
  m = 0.f;
  if (kind == HSTU_NORM_LAYER) {
    float t[1] = {0.f};
    if (live)
#pragma unroll
      for (int k = 0; k < 8; ++k) t[0] += a[k];
    team_sum<WPR, 1>(t, slot, flip, team, wid);
    m = t[0] * inv_d;
  }
  float t[1] = {0.f};
  if (live)
#pragma unroll
    for (int k = 0; k < 8; ++k) t[0] += (a[k] - m) * (a[k] - m);
  team_sum<WPR, 1>(t, slot, flip, team, wid);
  r = 1.f / sqrtf(t[0] * inv_d + eps);
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

// T: operand type; IO: residual stream's type.
template <typename T, typename IO, int WPR>
__global__ void __launch_bounds__(kThreads) block_norm_fwd_kernel(FwdArgs<T> p, const IO* x,
                                                                  const IO* __restrict__ b, IO* y) {
  constexpr int kTeams = kThreads / 32 / WPR;
  __shared__ float slots[kTeams][2 * WPR];
  const int team = threadIdx.x / (32 * WPR), lane = threadIdx.x % (32 * WPR), wid = lane / 32;
  const int d = p.d, col = lane * 8;
  const bool live = col < d;
  const float inv_d = 1.f / (float)d;
  int flip = 0;
  for (int64_t r = (int64_t)blockIdx.x * kTeams + team; r < p.rows; r += (int64_t)gridDim.x * kTeams) {
    float a[8] = {}, bb[8] = {};
    if (live) load8(x + r * d + col, a);
    float4 st = make_float4(0.f, 1.f, 0.f, 1.f);
    if (b) {
      float u[8] = {};
      if (live) {
        load8(b + r * d + col, bb);
        if (p.gate) load8(p.gate + r * p.gate_stride + col, u);
      }
      if (p.post != HSTU_NORM_NONE)
        row_stats<WPR>(p.post, bb, live, inv_d, p.eps, slots[team], flip, team, wid, st.x, st.y);
      if (live) {
        float g[8], bt[8], sc[8];
        param8(p.gamma1, col, 1.f, g);
        param8(p.beta1, col, 0.f, bt);
        param8(p.scale, col, 1.f, sc);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float v = p.post != HSTU_NORM_NONE ? (bb[k] - st.x) * st.y * g[k] + bt[k] : bb[k];
          if (p.gate) {
            float act, slope;
            gate_of(p.act, u[k], act, slope);
            v *= act;
          }
          a[k] = to_f(from_f<IO>(a[k] + sc[k] * v));
        }
        store8(y + r * d + col, a);
      }
    }
    if (p.h) {
      if (p.pre != HSTU_NORM_NONE)
        row_stats<WPR>(p.pre, a, live, inv_d, p.eps, slots[team], flip, team, wid, st.z, st.w);
      if (live) {
        if (p.pre != HSTU_NORM_NONE) {
          float g[8], bt[8];
          param8(p.gamma2, col, 1.f, g);
          param8(p.beta2, col, 0.f, bt);
#pragma unroll
          for (int k = 0; k < 8; ++k) a[k] = (a[k] - st.z) * st.w * g[k] + bt[k];
        }
        store8(p.h + r * d + col, a);
      }
    }
    if (p.stats && lane == 0) p.stats[r] = st;
  }
}

template <typename T>
struct BwdArgs {
  int post, pre, act, d;
  const T *gamma1, *beta1, *scale, *gamma2;
  const T* gate;
  int64_t gate_stride, rows;
  const float4* stats;
  T *db, *dgate;
  int64_t dgate_stride;
  float* partial;               // [gridDim.x][5][d], or NULL
};

template <typename T, typename IO, int WPR>
__global__ void __launch_bounds__(kThreads) block_norm_bwd_kernel(BwdArgs<T> p, const IO* __restrict__ y,
                                                                  const IO* __restrict__ b, const IO* dy,
                                                                  const IO* __restrict__ dh, IO* dx) {
  constexpr int kTeams = kThreads / 32 / WPR;
  __shared__ float slots[kTeams][2 * 2 * WPR];
  __shared__ float sums[kTeams > 1 ? kTeams : 1][256 * WPR];
  const int team = threadIdx.x / (32 * WPR), lane = threadIdx.x % (32 * WPR), wid = lane / 32;
  const int d = p.d, col = lane * 8;
  const bool live = col < d;
  const float inv_d = 1.f / (float)d;
  int flip = 0;
  float acc[kParams][8] = {};
  for (int64_t r = (int64_t)blockIdx.x * kTeams + team; r < p.rows; r += (int64_t)gridDim.x * kTeams) {
    const float4 st = p.stats[r];
    float e[8] = {};
    if (live && dy) load8(dy + r * d + col, e);
    if (dh) {
      float up[8] = {};
      if (live) load8(dh + r * d + col, up);
      if (p.pre == HSTU_NORM_NONE) {
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] += up[k];
      } else {
        float n[8] = {}, t[2] = {0.f, 0.f};
        if (live) {
          float g[8];
          load8(y + r * d + col, n);
          param8(p.gamma2, col, 1.f, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            n[k] = (n[k] - st.z) * st.w;
            acc[3][k] += up[k] * n[k];
            acc[4][k] += up[k];
            up[k] *= g[k];
            t[0] += up[k];
            t[1] += up[k] * n[k];
          }
        }
        team_sum<WPR, 2>(t, slots[team], flip, team, wid);
        const float level = p.pre == HSTU_NORM_LAYER ? t[0] * inv_d : 0.f, along = t[1] * inv_d;
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] += st.w * (up[k] - level - n[k] * along);
      }
    }
    if (live && dx) store8(dx + r * d + col, e);
    if (!b) continue;
    float n[8] = {}, q[8] = {}, t[2] = {0.f, 0.f};
    if (live) {
      float u[8], g[8], bt[8], sc[8], du[8];
      load8(b + r * d + col, n);
      if (p.gate) load8(p.gate + r * p.gate_stride + col, u);
      param8(p.gamma1, col, 1.f, g);
      param8(p.beta1, col, 0.f, bt);
      param8(p.scale, col, 1.f, sc);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float v = n[k];
        if (p.post != HSTU_NORM_NONE) {
          n[k] = (n[k] - st.x) * st.y;
          v = n[k] * g[k] + bt[k];
        }
        float act = 1.f, slope = 0.f;
        if (p.gate) gate_of(p.act, u[k], act, slope);
        acc[2][k] += e[k] * v * act;
        const float dv = e[k] * sc[k];
        du[k] = dv * v * slope;
        const float dp = dv * act;
        acc[0][k] += dp * n[k];
        acc[1][k] += dp;
        q[k] = p.post != HSTU_NORM_NONE ? dp * g[k] : dp;
        t[0] += q[k];
        t[1] += q[k] * n[k];
      }
      if (p.gate && p.dgate) store8(p.dgate + r * p.dgate_stride + col, du);
    }
    if (p.post != HSTU_NORM_NONE) {
      team_sum<WPR, 2>(t, slots[team], flip, team, wid);
      const float level = p.post == HSTU_NORM_LAYER ? t[0] * inv_d : 0.f, along = t[1] * inv_d;
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] = st.y * (q[k] - level - n[k] * along);
    }
    if (live && p.db) store8(p.db + r * d + col, q);
  }
  if (!p.partial) return;
  float* const out = p.partial + (int64_t)blockIdx.x * kParams * d;
  for (int i = 0; i < kParams; ++i) {
    if (kTeams == 1) {
      if (live)
#pragma unroll
        for (int k = 0; k < 8; ++k) out[i * d + col + k] = acc[i][k];
      continue;
    }
    __syncthreads();
    if (live)
#pragma unroll
      for (int k = 0; k < 8; ++k) sums[team][col + k] = acc[i][k];
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kTeams; ++w) t += sums[w][c];
      out[i * d + c] = t;
    }
  }
}

struct GradPtrs {
  float* p[kParams];
};

// grads.p[i][c] += sum over the CTAs of partial[cta][i][c], in the order of
// the CTAs within each of 8 strips, then of the strips.
__global__ void __launch_bounds__(256) block_norm_join_kernel(const float* __restrict__ partial, int ctas, int d,
                                                              GradPtrs grads) {
  __shared__ float strip[8][32];
  float* const out = grads.p[blockIdx.y];
  if (!out) return;
  const int c = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
  const float* src = partial + (int64_t)blockIdx.y * d + c;
  float t = 0.f;
  if (c < d)
#pragma unroll 8
    for (int i = w; i < ctas; i += 8) t += src[(int64_t)i * kParams * d];
  strip[w][threadIdx.x % 32] = t;
  __syncthreads();
  if (w == 0 && c < d) {
#pragma unroll
    for (int k = 1; k < 8; ++k) t += strip[k][threadIdx.x];
    out[c] += t;
  }
}

int warps_per_row(int d) { return d <= 256 ? 1 : d <= 512 ? 2 : d <= 1024 ? 4 : 8; }

// CTAs of the backward, which bound its workspace: at most two per multiprocessor.
int64_t bwd_ctas(int d, int64_t T) {
  const int teams = kThreads / 32 / warps_per_row(d);
  const int64_t want = (T + teams - 1) / teams, cap = (int64_t)sm_count() * 2;
  return want < cap ? want : cap;
}

template <typename T, typename IO, int WPR>
cudaError_t launch_fwd(const FwdArgs<T>& p, const void* x, const void* b, void* y, cudaStream_t s) {
  constexpr int kTeams = kThreads / 32 / WPR;
  int64_t ctas = (p.rows + kTeams - 1) / kTeams;
  const int64_t cap = (int64_t)sm_count() * 8;
  if (ctas > cap) ctas = cap;
  block_norm_fwd_kernel<T, IO, WPR><<<(unsigned)ctas, kThreads, 0, s>>>(
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
  switch (warps_per_row(p.d)) {
    case 1: return launch_fwd<T, IO, 1>(p, x, b, y, s);
    case 2: return launch_fwd<T, IO, 2>(p, x, b, y, s);
    case 4: return launch_fwd<T, IO, 4>(p, x, b, y, s);
    default: return launch_fwd<T, IO, 8>(p, x, b, y, s);
  }
}

template <typename T, typename IO, int WPR>
cudaError_t launch_bwd(const BwdArgs<T>& p, const void* y, const void* b, const void* dy, const void* dh,
                       void* dx, const GradPtrs& grads, cudaStream_t s) {
  const int ctas = (int)bwd_ctas(p.d, p.rows);
  block_norm_bwd_kernel<T, IO, WPR><<<(unsigned)ctas, kThreads, 0, s>>>(
      p, static_cast<const IO*>(y), static_cast<const IO*>(b), static_cast<const IO*>(dy),
      static_cast<const IO*>(dh), static_cast<IO*>(dx));
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.partial) {
    block_norm_join_kernel<<<dim3((unsigned)((p.d + 31) / 32), kParams), 256, 0, s>>>(p.partial, ctas, p.d, grads);
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
  switch (warps_per_row(p.d)) {
    case 1: return launch_bwd<T, IO, 1>(p, y, b, dy, dh, dx, grads, s);
    case 2: return launch_bwd<T, IO, 2>(p, y, b, dy, dh, dx, grads, s);
    case 4: return launch_bwd<T, IO, 4>(p, y, b, dy, dh, dx, grads, s);
    default: return launch_bwd<T, IO, 8>(p, y, b, dy, dh, dx, grads, s);
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
