// Embedding lookup with scaling, and its gradient by sorted ids.
//
//   out[t] = scale E[id_t]                (zero for an id outside [0, V))
//   dE[v] += scale sum_{t: id_t = v} dout[t]
//
// Both move rows and compute next to nothing: the lookup reads each named row
// and writes T rows (twice with the bf16 copy), the gradient reads T rows and
// writes one for each different id.
//
// Gradient: (id, event) pairs are sorted by id with a stable radix sort of 8
// bits a pass (as many passes as V has digits; ids outside [0, V) become V and
// end up last), so that an item's events are neighbours in their own order.
// A warp then sums a chunk of 32 sorted events: its lanes hold the chunk's
// (id, event) pairs, every row is read once, and each item's sum leaves the
// registers when the id changes.  An item whose events lie in one chunk is
// added to the gradient there; one that crosses into the next chunk leaves a
// partial sum per chunk, and the chunk where it begins adds those up, so no
// item's sum depends on the order of execution and a popular item is read by
// as many warps as it has chunks.
#include "args.h"
#include "common.cuh"
#include "internal.h"

namespace hstu {
namespace {

constexpr int kChunk = 32;           // sorted events of a warp
constexpr int kTile = 2048;          // events of a sorting CTA
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kPerThread = kTile / kSortThreads;
constexpr int kDigits = 256;

// N consecutive elements in one access of N * sizeof(T) bytes.
template <int BYTES> struct Raw;
template <> struct Raw<16> { using U = uint4; };
template <> struct Raw<8> { using U = uint2; };
template <> struct Raw<4> { using U = uint32_t; };
template <> struct Raw<2> { using U = uint16_t; };

template <typename T, int N>
struct Pack {
  union {
    typename Raw<(int)sizeof(T) * N>::U raw;
    T v[N];
  };
  __device__ Pack() {}
  __device__ __forceinline__ void load(const T* p) {
    raw = *reinterpret_cast<const typename Raw<(int)sizeof(T) * N>::U*>(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    *reinterpret_cast<typename Raw<(int)sizeof(T) * N>::U*>(p) = raw;
  }
};

__device__ __forceinline__ int64_t id_at(const void* ids, int id_bytes, int64_t t) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[t] : (int64_t) static_cast<const int32_t*>(ids)[t];
}

// ---------------------------------------------------------------------------
// Lookup: one thread for N columns of a row.
// ---------------------------------------------------------------------------
template <typename TT, typename TO, int N, bool LOW>
__global__ void __launch_bounds__(256) lookup_kernel(const TT* __restrict__ table, int64_t V, int dim,
                                                     int64_t table_stride, const void* __restrict__ ids,
                                                     int id_bytes, int64_t rows, float scale,
                                                     TO* __restrict__ out, int width, int64_t out_stride,
                                                     bf16* __restrict__ low, int64_t low_stride) {
  const int units = width / N;
  const int64_t total = rows * units, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
    const int64_t t = i / units;
    const int c = (int)(i - t * units) * N;
    const int64_t id = id_at(ids, id_bytes, t);
    float f[N];
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = 0.f;
    if (id >= 0 && id < V && c < dim) {     // N divides dim
      Pack<TT, N> a;
      a.load(table + id * table_stride + c);
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = scale * to_f(a.v[k]);
    }
    Pack<TO, N> o;
#pragma unroll
    for (int k = 0; k < N; ++k) o.v[k] = from_f<TO>(f[k]);
    o.store(out + t * out_stride + c);
    if (LOW) {
      Pack<bf16, N> l;
#pragma unroll
      for (int k = 0; k < N; ++k) l.v[k] = from_f<bf16>(f[k]);
      l.store(low + t * low_stride + c);
    }
  }
}

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
// The pair of event t: from the ids in the first pass, from the previous pass
// after it.
struct PairSource {
  const uint2* pairs;
  const void* ids;
  int id_bytes;
  uint32_t V;
  __device__ __forceinline__ uint2 operator()(int64_t t) const {
    if (pairs) return pairs[t];
    const int64_t id = id_at(ids, id_bytes, t);
    return make_uint2(id >= 0 && id < (int64_t)V ? (uint32_t)id : V, (uint32_t)t);
  }
};

__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(PairSource src, int64_t T, int shift,
                                                                 uint32_t* __restrict__ hist) {
  __shared__ uint32_t h[kDigits];
  h[threadIdx.x] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kTile;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t t = base + i * kSortThreads + threadIdx.x;
    if (t < T) atomicAdd(&h[(src(t).x >> shift) & (kDigits - 1)], 1u);
  }
  __syncthreads();
  hist[(int64_t)blockIdx.x * kDigits + threadIdx.x] = h[threadIdx.x];
}

// One CTA a digit: hist[tile][digit] becomes the number of events with this
// digit in earlier tiles; totals[digit] their number in all.
__global__ void __launch_bounds__(256) sort_scan_kernel(uint32_t* __restrict__ hist, int tiles,
                                                        uint32_t* __restrict__ totals) {
  __shared__ uint32_t warp_tot[8];
  __shared__ uint32_t carry;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int base = 0; base < tiles; base += 256) {
    const int i = base + threadIdx.x;
    uint32_t* const p = hist + (int64_t)i * kDigits + blockIdx.x;
    const uint32_t x = i < tiles ? *p : 0u;
    uint32_t v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    uint32_t before = carry;
    for (int w = 0; w < warp; ++w) before += warp_tot[w];
    if (i < tiles) *p = before + v - x;
    __syncthreads();
    if (threadIdx.x == 255) carry = before + v;
    __syncthreads();
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// Moves a tile's pairs to their places: the digit's first place (all lower
// digits), plus its events in earlier tiles, earlier warps of the tile, and
// earlier places of the warp.
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(PairSource src, int64_t T, int shift,
                                                                    const uint32_t* __restrict__ hist,
                                                                    const uint32_t* __restrict__ totals,
                                                                    uint2* __restrict__ out) {
  __shared__ uint32_t count[kSortWarps][kDigits];
  __shared__ uint32_t first[kDigits];
  __shared__ uint32_t warp_tot[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) count[w][tid] = 0;
  // exclusive scan of the digits' totals
  const uint32_t x = totals[tid];
  uint32_t v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; ++w) before += warp_tot[w];
  first[tid] = before + v - x + hist[(int64_t)blockIdx.x * kDigits + tid];
  // rank within the warp, whose events are consecutive
  const int64_t base = (int64_t)blockIdx.x * kTile + warp * (32 * kPerThread);
  uint2 pair[kPerThread];
  uint32_t rank[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t t = base + i * 32 + lane;
    const bool in = t < T;
    pair[i] = in ? src(t) : make_uint2(0, 0);
    const uint32_t digit = (pair[i].x >> shift) & (kDigits - 1);
    const uint32_t peers = __match_any_sync(0xffffffffu, in ? digit : 0x10000u);
    const uint32_t ahead = __popc(peers & ((1u << lane) - 1u));
    const uint32_t seen = in ? count[warp][digit] : 0u;
    __syncwarp();
    if (in && ahead == 0) count[warp][digit] = seen + __popc(peers);
    __syncwarp();
    rank[i] = seen + ahead;
  }
  __syncthreads();
  // over the warps: earlier ones of this digit, and the place where it begins
  uint32_t run = first[tid];
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    const uint32_t n = count[w][tid];
    count[w][tid] = run;
    run += n;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t t = base + i * 32 + lane;
    if (t < T) out[count[warp][(pair[i].x >> shift) & (kDigits - 1)] + rank[i]] = pair[i];
  }
}

// ---------------------------------------------------------------------------
// Rows form: how many items begin before each chunk
// ---------------------------------------------------------------------------
// heads[c] = items whose first event lies in chunk c.
__global__ void __launch_bounds__(256) heads_kernel(const uint2* __restrict__ pairs, int64_t T, uint32_t V,
                                                    int64_t chunks, uint32_t* __restrict__ heads) {
  const int64_t c = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t t = c * kChunk + (threadIdx.x & 31);
  bool head = false;
  if (t < T) {
    const uint32_t k = pairs[t].x;
    head = k < V && (t == 0 || pairs[t - 1].x != k);
  }
  const uint32_t n = __popc(__ballot_sync(0xffffffffu, head));
  if (c < chunks && (threadIdx.x & 31) == 0) heads[c] = n;
}

// heads becomes its exclusive prefix sum; *num_rows the number of items.  One CTA.
__global__ void __launch_bounds__(1024) heads_scan_kernel(uint32_t* __restrict__ heads, int64_t chunks,
                                                          int64_t* __restrict__ num_rows) {
  __shared__ uint32_t warp_tot[32];
  __shared__ uint32_t carry;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int64_t base = 0; base < chunks; base += 1024) {
    const int64_t i = base + threadIdx.x;
    const uint32_t x = i < chunks ? heads[i] : 0u;
    uint32_t v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    uint32_t before = carry;
    for (int w = 0; w < warp; ++w) before += warp_tot[w];
    if (i < chunks) heads[i] = before + v - x;
    __syncthreads();
    if (threadIdx.x == 1023) carry = before + v;
    __syncthreads();
  }
  if (threadIdx.x == 0) *num_rows = carry;
}

// ---------------------------------------------------------------------------
// Sums
// ---------------------------------------------------------------------------
struct SumArgs {
  const uint2* pairs;
  int64_t T, chunks;
  uint32_t V;
  int dim;
  int64_t dout_stride;
  float scale;
  float* dst;                 // dtable or rows
  int64_t dst_stride;
  const uint32_t* heads;      // rows form: items before each chunk; else NULL
  int64_t* row_ids;
  float* partial;             // [chunks][2][dim]
};

// Adds (dense) or writes (rows form) an item's sum.
template <int N>
__device__ __forceinline__ void put_sum(const SumArgs& a, int64_t row, int col, const float (&f)[N]) {
  float* const p = a.dst + row * a.dst_stride + col;
#pragma unroll
  for (int k = 0; k < N; ++k) p[k] = a.heads ? a.scale * f[k] : p[k] + a.scale * f[k];
}

// A warp sums a chunk's columns [32 N y, 32 N (y + 1)); a lane owns N of them.
// partial[c][0]: the sum of the item that came over from the chunk before;
// partial[c][1]: of the one that begins in the chunk and goes on after it.
template <typename T, int N>
__global__ void __launch_bounds__(256) sum_kernel(SumArgs a, const T* __restrict__ dout) {
  const int lane = threadIdx.x & 31;
  const int64_t c = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (c >= a.chunks) return;
  const int64_t t0 = c * kChunk;
  const int n = (int)min((int64_t)kChunk, a.T - t0);
  const uint2 mine = lane < n ? a.pairs[t0 + lane] : make_uint2(a.V, 0);
  const uint32_t before = t0 > 0 ? a.pairs[t0 - 1].x : a.V;
  const uint32_t after = t0 + n < a.T ? a.pairs[t0 + n].x : a.V;
  uint32_t left = __shfl_up_sync(0xffffffffu, mine.x, 1);
  if (lane == 0) left = before;
  const bool real = mine.x < a.V;
  const uint32_t begins = __ballot_sync(0xffffffffu, real && left != mine.x);   // an item's first event
  const int count = __popc(__ballot_sync(0xffffffffu, real));   // padding sorts last
  if (count == 0) return;
  const int col = ((int)blockIdx.y * 32 + lane) * N;
  const bool live = col < a.dim;
  const int64_t first_row = a.heads ? (int64_t)a.heads[c] : 0;
  float acc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) acc[k] = 0.f;
  bool open = (begins & 1u) == 0;       // the running item began before this chunk
  int started = 0;                      // items begun in this chunk so far
  for (int j = 0; j < count; ++j) {
    const uint32_t key = __shfl_sync(0xffffffffu, mine.x, j), ev = __shfl_sync(0xffffffffu, mine.y, j);
    if ((begins >> j) & 1u) ++started;
    if (live) {
      Pack<T, N> p;
      p.load(dout + (int64_t)ev * a.dout_stride + col);
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += to_f(p.v[k]);
    }
    const bool last = j + 1 == count;
    const bool ends = last ? !(count == n && after == key) : ((begins >> (j + 1)) & 1u);
    if (!ends && !last) continue;
    const int64_t row = a.heads ? first_row + started - 1 : (int64_t)key;
    if (live) {
      if (open || !ends) {
        float* const w = a.partial + (c * 2 + (open ? 0 : 1)) * a.dim + col;
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = acc[k];
      } else {
        put_sum<N>(a, row, col, acc);
      }
    }
    if (a.heads && !open && blockIdx.y == 0 && lane == 0) a.row_ids[row] = key;
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    open = false;
  }
}

// A CTA for a chunk: where the chunk's last item begins in it and goes on, adds
// up the item's partial sums.
__global__ void __launch_bounds__(256) join_kernel(SumArgs a) {
  __shared__ float strip[8][32];
  const int64_t c = blockIdx.x, t0 = c * kChunk, end = t0 + kChunk;
  if (end >= a.T) return;
  const uint32_t key = a.pairs[end].x;
  if (key >= a.V || a.pairs[end - 1].x != key) return;               // nothing goes on
  if (a.pairs[t0].x == key && t0 > 0 && a.pairs[t0 - 1].x == key) return;    // it began earlier
  // the chunks that the item came over to: c + 1 .. last (a chunk's first
  // event is the item's as long as the chunk's index does not pass it)
  int64_t lo = c + 1, hi = a.chunks;            // first chunk that does not begin with the item is in (lo, hi]
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.pairs[mid * kChunk].x == key) lo = mid; else hi = mid;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t row = a.heads ? (int64_t)a.heads[c + 1] - 1 : (int64_t)key;
  for (int base = 0; base < a.dim; base += 32) {
    const int col = base + lane;
    float t = 0.f;
    if (col < a.dim) {
      if (w == 0) t = a.partial[(c * 2 + 1) * a.dim + col];
      for (int64_t i = c + 1 + w; i <= lo; i += 8) t += a.partial[i * 2 * a.dim + col];
    }
    strip[w][lane] = t;
    __syncthreads();
    if (w == 0 && col < a.dim) {
#pragma unroll
      for (int k = 1; k < 8; ++k) t += strip[k][lane];
      const float f[1] = {t};
      put_sum<1>(a, row, col, f);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
bool vec_ok(int64_t n, const void* p, int64_t bytes, int64_t stride, int64_t a, int64_t b) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(n * bytes) == 0 && stride % n == 0 && a % n == 0 && b % n == 0;
}

struct BwdLayout {
  size_t a, b, hist, totals, heads, partial, total;
  int64_t tiles, chunks;
};
BwdLayout bwd_layout(int64_t T, int dim) {
  BwdLayout l;
  l.tiles = (T + kTile - 1) / kTile;
  l.chunks = (T + kChunk - 1) / kChunk;
  l.a = 0;
  l.b = align_up(l.a + (size_t)T * 8, 256);
  l.hist = align_up(l.b + (size_t)T * 8, 256);
  l.totals = align_up(l.hist + (size_t)l.tiles * kDigits * 4, 256);
  l.heads = align_up(l.totals + kDigits * 4, 256);
  l.partial = align_up(l.heads + (size_t)l.chunks * 4, 256);
  l.total = align_up(l.partial + (size_t)l.chunks * 2 * (size_t)dim * 4, 256);
  return l;
}

hstu_status check_sizes(int64_t T, int64_t V, int32_t dim) {
  if (T < 0 || V < 1 || dim < 1) return HSTU_ERR_INVALID;
  if (T >= ((int64_t)1 << 31) || V >= ((int64_t)1 << 31) || dim > 65536) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}
hstu_status check_ids(const void* ids, int32_t id_bytes, int64_t T) {
  if (id_bytes != 4 && id_bytes != 8) return HSTU_ERR_INVALID;
  return meta(ids, T, (size_t)id_bytes);
}
hstu_status check_dtype(int32_t t) { return t == HSTU_F32 || t == HSTU_BF16 ? HSTU_OK : HSTU_ERR_INVALID; }

template <typename T>
cudaError_t launch_sum(const SumArgs& a, const void* dout, int n, cudaStream_t s) {
  const T* p = static_cast<const T*>(dout);
  const dim3 grid((unsigned)((a.chunks + 7) / 8), (unsigned)((a.dim + 32 * n - 1) / (32 * n)));
  if (n == 4) sum_kernel<T, 4><<<grid, 256, 0, s>>>(a, p);
  else if (n == 2) sum_kernel<T, 2><<<grid, 256, 0, s>>>(a, p);
  else sum_kernel<T, 1><<<grid, 256, 0, s>>>(a, p);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.chunks > 1) {
    join_kernel<<<(unsigned)a.chunks, 256, 0, s>>>(a);
    count_launch();
    e = cudaGetLastError();
  }
  return e;
}

// The gradient in either form; rows form when row_ids is given.
cudaError_t embedding_bwd(const void* dout, int dout_dtype, int64_t dout_stride, const void* ids, int id_bytes,
                          int64_t T, int64_t V, int dim, float scale, float* dst, int64_t dst_stride,
                          int64_t* row_ids, int64_t* num_rows, void* ws, cudaStream_t s) {
  const BwdLayout l = bwd_layout(T, dim);
  char* const base = static_cast<char*>(ws);
  uint2* pairs[2] = {reinterpret_cast<uint2*>(base + l.a), reinterpret_cast<uint2*>(base + l.b)};
  uint32_t* hist = reinterpret_cast<uint32_t*>(base + l.hist);
  uint32_t* totals = reinterpret_cast<uint32_t*>(base + l.totals);
  uint32_t* heads = reinterpret_cast<uint32_t*>(base + l.heads);
  int bits = 0;
  while (bits < 32 && ((uint64_t)V >> bits) != 0) ++bits;        // keys are 0 .. V
  int cur = 0;
  PairSource src{nullptr, ids, id_bytes, (uint32_t)V};
  for (int shift = 0; shift < bits; shift += 8) {
    sort_hist_kernel<<<(unsigned)l.tiles, kSortThreads, 0, s>>>(src, T, shift, hist);
    sort_scan_kernel<<<kDigits, 256, 0, s>>>(hist, (int)l.tiles, totals);
    sort_scatter_kernel<<<(unsigned)l.tiles, kSortThreads, 0, s>>>(src, T, shift, hist, totals, pairs[cur]);
    count_launch(3);
    src.pairs = pairs[cur];
    cur ^= 1;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (row_ids) {
    heads_kernel<<<(unsigned)((l.chunks + 7) / 8), 256, 0, s>>>(src.pairs, T, (uint32_t)V, l.chunks, heads);
    heads_scan_kernel<<<1, 1024, 0, s>>>(heads, l.chunks, num_rows);
    count_launch(2);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  SumArgs a;
  a.pairs = src.pairs;
  a.T = T;
  a.chunks = l.chunks;
  a.V = (uint32_t)V;
  a.dim = dim;
  a.dout_stride = dout_stride;
  a.scale = scale;
  a.dst = dst;
  a.dst_stride = dst_stride;
  a.heads = row_ids ? heads : nullptr;
  a.row_ids = row_ids;
  a.partial = reinterpret_cast<float*>(base + l.partial);
  const int64_t es = dtype_size(dout_dtype);
  int n = 4;
  while (n > 1 && !vec_ok(n, dout, es, dout_stride, dim, dim)) n >>= 1;
  return dout_dtype == HSTU_BF16 ? launch_sum<bf16>(a, dout, n, s) : launch_sum<float>(a, dout, n, s);
}

template <typename TT, typename TO, bool LOW>
cudaError_t launch_lookup(const void* table, int64_t V, int dim, int64_t table_stride, const void* ids,
                          int id_bytes, int64_t T, float scale, void* out, int width, int64_t out_stride,
                          void* low, int64_t low_stride, cudaStream_t s) {
  int n = 4;
  while (n > 1 && !(vec_ok(n, table, sizeof(TT), table_stride, dim, width) &&
                    vec_ok(n, out, sizeof(TO), out_stride, dim, width) &&
                    (!LOW || vec_ok(n, low, 2, low_stride, dim, width))))
    n >>= 1;
  const int64_t want = (T * (width / n) + 255) / 256, cap = (int64_t)sm_count() * 32;
  const unsigned grid = (unsigned)(want < cap ? want : cap);
  const TT* t = static_cast<const TT*>(table);
  TO* o = static_cast<TO*>(out);
  bf16* l = static_cast<bf16*>(low);
  if (n == 4) lookup_kernel<TT, TO, 4, LOW><<<grid, 256, 0, s>>>(t, V, dim, table_stride, ids, id_bytes, T, scale, o, width, out_stride, l, low_stride);
  else if (n == 2) lookup_kernel<TT, TO, 2, LOW><<<grid, 256, 0, s>>>(t, V, dim, table_stride, ids, id_bytes, T, scale, o, width, out_stride, l, low_stride);
  else lookup_kernel<TT, TO, 1, LOW><<<grid, 256, 0, s>>>(t, V, dim, table_stride, ids, id_bytes, T, scale, o, width, out_stride, l, low_stride);
  count_launch();
  return cudaGetLastError();
}

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status hstu_embedding_fwd(const void* table, int32_t table_dtype, int64_t V, int32_t dim,
                               int64_t table_stride, const void* ids, int32_t id_bytes, int64_t T, float scale,
                               void* out, int32_t out_dtype, int32_t width, int64_t out_stride, void* out_low,
                               int64_t low_stride, cudaStream_t stream) {
  HSTU_TRY(check_sizes(T, V, dim));
  HSTU_TRY(check_dtype(table_dtype));
  HSTU_TRY(check_dtype(out_dtype));
  if (width < dim || table_stride < dim || out_stride < width || (out_low && low_stride < width))
    return HSTU_ERR_INVALID;
  if (width > 65536) return HSTU_ERR_UNSUPPORTED;
  if (out_low && out_dtype != HSTU_F32) return HSTU_ERR_INVALID;
  HSTU_TRY(check_ids(ids, id_bytes, T));
  HSTU_TRY(meta(table, T, (size_t)dtype_size(table_dtype)));
  HSTU_TRY(meta(out, T, (size_t)dtype_size(out_dtype)));
  HSTU_TRY(meta(out_low, out_low ? 1 : 0, 2));
  if (T == 0) return HSTU_OK;
  prof_begin(HSTU_K_EMBED, stream);
  cudaError_t e;
#define HSTU_LOOKUP(TT, TO, LOW)                                                                            \
  launch_lookup<TT, TO, LOW>(table, V, dim, table_stride, ids, id_bytes, T, scale, out, width, out_stride, \
                             out_low, low_stride, stream)
  if (table_dtype == HSTU_F32)
    e = out_dtype == HSTU_BF16 ? HSTU_LOOKUP(float, bf16, false)
        : out_low              ? HSTU_LOOKUP(float, float, true)
                               : HSTU_LOOKUP(float, float, false);
  else
    e = out_dtype == HSTU_BF16 ? HSTU_LOOKUP(bf16, bf16, false)
        : out_low              ? HSTU_LOOKUP(bf16, float, true)
                               : HSTU_LOOKUP(bf16, float, false);
#undef HSTU_LOOKUP
  prof_end(HSTU_K_EMBED, stream);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

size_t hstu_embedding_bwd_workspace_size(int64_t T, int64_t V, int32_t dim) {
  if (check_sizes(T, V, dim) != HSTU_OK || T == 0) return 0;
  return bwd_layout(T, dim).total;
}

hstu_status hstu_embedding_bwd(const void* dout, int32_t dout_dtype, int64_t dout_stride, const void* ids,
                               int32_t id_bytes, int64_t T, int64_t V, int32_t dim, float scale, float* dtable,
                               int64_t dtable_stride, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  HSTU_TRY(check_sizes(T, V, dim));
  HSTU_TRY(check_dtype(dout_dtype));
  if (dout_stride < dim || dtable_stride < dim) return HSTU_ERR_INVALID;
  HSTU_TRY(check_ids(ids, id_bytes, T));
  HSTU_TRY(meta(dout, T, (size_t)dtype_size(dout_dtype)));
  HSTU_TRY(meta(dtable, T, 4));
  if (T == 0) return HSTU_OK;
  if (ws_bytes < bwd_layout(T, dim).total) return HSTU_ERR_WORKSPACE;
  HSTU_TRY(need(workspace, 1));
  prof_begin(HSTU_K_EMBED, stream);
  const cudaError_t e = embedding_bwd(dout, dout_dtype, dout_stride, ids, id_bytes, T, V, dim, scale, dtable,
                                      dtable_stride, nullptr, nullptr, workspace, stream);
  prof_end(HSTU_K_EMBED, stream);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

hstu_status hstu_embedding_bwd_rows(const void* dout, int32_t dout_dtype, int64_t dout_stride, const void* ids,
                                    int32_t id_bytes, int64_t T, int64_t V, int32_t dim, float scale,
                                    int64_t* row_ids, float* rows, int64_t rows_stride, int64_t* d_num_rows,
                                    void* workspace, size_t ws_bytes, cudaStream_t stream) {
  HSTU_TRY(check_sizes(T, V, dim));
  HSTU_TRY(check_dtype(dout_dtype));
  if (dout_stride < dim || rows_stride < dim) return HSTU_ERR_INVALID;
  HSTU_TRY(check_ids(ids, id_bytes, T));
  HSTU_TRY(meta(dout, T, (size_t)dtype_size(dout_dtype)));
  HSTU_TRY(meta(row_ids, T, 8));
  HSTU_TRY(meta(rows, T, 4));
  HSTU_TRY(meta(d_num_rows, 1, 8));
  if (T > 0) {
    if (ws_bytes < bwd_layout(T, dim).total) return HSTU_ERR_WORKSPACE;
    HSTU_TRY(need(workspace, 1));
  }
  prof_begin(HSTU_K_EMBED, stream);
  cudaError_t e;
  if (T == 0)
    e = cudaMemsetAsync(d_num_rows, 0, sizeof(int64_t), stream);
  else
    e = embedding_bwd(dout, dout_dtype, dout_stride, ids, id_bytes, T, V, dim, scale, rows, rows_stride, row_ids,
                      d_num_rows, workspace, stream);
  prof_end(HSTU_K_EMBED, stream);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
