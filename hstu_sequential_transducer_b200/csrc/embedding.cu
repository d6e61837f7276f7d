// Embedding lookup with scaling, and its gradient by sorted ids.
//
//   out[t] = scale E[id_t]                (zero for an id outside [0, V))
//   dE[v] += scale sum_{t: id_t = v} dout[t]
//
// Both move rows and compute next to nothing: the lookup reads each named row
// and writes T rows (twice with the bf16 copy), the gradient reads T rows and
// writes one for each different id.
//
// Gradient: (id, event) pairs are sorted by id with a stable radix sort of up
// to 9 bits a pass (as many passes as V has digits; ids outside [0, V) become V
// and end up last), so that an item's events are neighbours in their own order.
// A warp then sums a chunk of 32 sorted events: its lanes hold the chunk's
// (id, event) pairs, every row is read once, 8 of them in flight, and each
// item's sum leaves the registers when the id changes.  An item whose events lie in
// one chunk is added to the gradient there; one that crosses into the next chunk
// leaves a partial sum per chunk, and the chunk where it begins is put on a list
// whose entries are joined by a last kernel.  No item's sum depends on the
// order of execution, and a popular item is read by as many warps as it has chunks.
#include <algorithm>

#include "args.h"
#include "common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace hstu {
namespace {

constexpr int kChunk = 32;           // sorted events of a warp
constexpr int kBatch = 8;            // rows of a chunk in flight
constexpr int kSuper = 1024;         // sorted events of a CTA that counts items
constexpr int kTile = 4096;          // events of a sorting CTA
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 512;         // of a pass, at most
constexpr int kMaxPasses = 4;
constexpr int kJoinWords = 4;        // counters before the list of items to join, cleared by the sort
constexpr int kAlone = 32;           // an item that goes on for more chunks is a long one
// Up to this many tiles, a CTA of the sort adds up the tiles' counts by itself
// (2 KB of each); above, a kernel of its own scans them once for all CTAs (two
// launches more; whole gradients of 8 columns: 287,928 events 52.7 us by itself, 54.2
// scanned; 400,000 65.0 and 64.6; 1,048,576 140.8 and 124.7).
constexpr int kDirectTiles = 96;
// Up to this many events are sorted by one CTA in one launch, and up to eight
// times as many by a cluster of CTAs, also in one launch (14,001 events in two
// passes: 14 us; as a launch for the counts and one for each pass 21).
constexpr int kSmallSort = 4096;
constexpr int kSortCluster = 8;

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
// Lookup: a thread has kLookups pieces of N columns in flight, neighbouring
// threads neighbouring pieces, in many small CTAs (a training batch of 287,928 rows
// of 1,024 with the bf16 copy: 363 us with one piece a thread and 32 CTAs a
// multiprocessor).
// ---------------------------------------------------------------------------
constexpr int kLookups = 4;
template <typename TT, typename TO, int N, bool LOW>
__global__ void __launch_bounds__(256) lookup_kernel(const TT* __restrict__ table, int64_t V, int dim,
                                                     int64_t table_stride, const void* __restrict__ ids,
                                                     int id_bytes, int64_t rows, float scale,
                                                     TO* __restrict__ out, int width, int64_t out_stride,
                                                     bf16* __restrict__ low, int64_t low_stride) {
  const int units = width / N;
  const int64_t base = (int64_t)blockIdx.x * (256 * kLookups);
  const RowOf where(base, units);
  const int count = (int)min((int64_t)(256 * kLookups), rows * units - base);
  Pack<TT, N> in[kLookups];
  int64_t row[kLookups];
  int col[kLookups];
  bool any[kLookups];
#pragma unroll
  for (int i = 0; i < kLookups; ++i) {
    const int off = i * 256 + (int)threadIdx.x;
    any[i] = false;
    if (off < count) {
      const int r = where.rows_after(off);
      row[i] = where.row0 + r;
      col[i] = (where.col0 + off - r * units) * N;
      const int64_t id = id_at(ids, id_bytes, row[i]);
      any[i] = id >= 0 && id < V && col[i] < dim;     // N divides dim
      if (any[i]) in[i].load(table + id * table_stride + col[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kLookups; ++i) {
    if (i * 256 + (int)threadIdx.x >= count) break;
    float f[N];
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = any[i] ? scale * to_f(in[i].v[k]) : 0.f;
    Pack<TO, N> o;
#pragma unroll
    for (int k = 0; k < N; ++k) o.v[k] = from_f<TO>(f[k]);
    o.store(out + row[i] * out_stride + col[i]);
    if (LOW) {
      Pack<bf16, N> l;
#pragma unroll
      for (int k = 0; k < N; ++k) l.v[k] = from_f<bf16>(f[k]);
      l.store(low + row[i] * low_stride + col[i]);
    }
  }
}

// Rows that allow no wider access than an element: a warp a row, kLookups * 2
// of a lane's columns in flight.
constexpr int kRowFlight = 2 * kLookups;
template <typename TT, typename TO, bool LOW>
__global__ void __launch_bounds__(256) lookup_rows_kernel(const TT* __restrict__ table, int64_t V, int dim,
                                                          int64_t table_stride, const void* __restrict__ ids,
                                                          int id_bytes, int64_t rows, float scale,
                                                          TO* __restrict__ out, int width, int64_t out_stride,
                                                          bf16* __restrict__ low, int64_t low_stride) {
  const int lane = threadIdx.x & 31;
  const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (row >= rows) return;
  const int64_t id = id_at(ids, id_bytes, row);
  const int have = id >= 0 && id < V ? dim : 0;
  const TT* const src = table + (have ? id : 0) * table_stride;
  out += row * out_stride;
  if (LOW) low += row * low_stride;
  for (int c0 = lane; c0 < width; c0 += 32 * kRowFlight) {
    float f[kRowFlight];
#pragma unroll
    for (int i = 0; i < kRowFlight; ++i) f[i] = c0 + 32 * i < have ? to_f(src[c0 + 32 * i]) : 0.f;
#pragma unroll
    for (int i = 0; i < kRowFlight; ++i) {
      const int c = c0 + 32 * i;
      if (c >= width) break;
      const float v = c < have ? scale * f[i] : 0.f;
      out[c] = from_f<TO>(v);
      if (LOW) low[c] = from_f<bf16>(v);
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

// A pass sorts by the digit of `width` bits from `shift` on.
struct Pass {
  int shift, width;
  __device__ __forceinline__ uint32_t digit(uint32_t key) const { return (key >> shift) & ((1u << width) - 1u); }
};

// Counts the first pass's digits of every tile, and clears the counts of the
// later passes and the counters before the list of items to join.
__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(PairSource src, int64_t T, Pass pass, int passes,
                                                                 uint32_t* __restrict__ hist, int64_t pass_stride,
                                                                 uint32_t* __restrict__ joins) {
  __shared__ uint32_t h[kDigits];
  if (threadIdx.x < kDigits) h[threadIdx.x] = 0;
  if (blockIdx.x == 0 && threadIdx.x < kJoinWords) joins[threadIdx.x] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kTile;
#pragma unroll
  for (int i = 0; i < kTile / kSortThreads; ++i) {
    const int64_t t = base + i * kSortThreads + threadIdx.x;
    if (t < T) atomicAdd(&h[pass.digit(src(t).x)], 1u);
  }
  __syncthreads();
  if (threadIdx.x >= kDigits) return;
  uint32_t* const out = hist + (int64_t)blockIdx.x * kDigits + threadIdx.x;
  *out = h[threadIdx.x];
  for (int p = 1; p < passes; ++p) out[p * pass_stride] = 0;
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

// Exclusive prefix sum of x over the CTA's 32 warps.
static_assert(kSortWarps == 32, "a warp's lanes scan the warps' totals");
__device__ __forceinline__ uint32_t block_prefix(uint32_t x, uint32_t* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
  uint32_t w = lane < warp ? warp_tot[lane] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w + v - x;
}

__device__ __forceinline__ void clear_counts(uint32_t (*count)[kDigits]) {
  uint4* const p = reinterpret_cast<uint4*>(count[0]);
#pragma unroll
  for (int i = 0; i < kSortWarps * kDigits / 4 / kSortThreads; ++i)
    p[i * kSortThreads + threadIdx.x] = make_uint4(0, 0, 0, 0);
}
// The thread's digit: its warps' counts become their first places, from `run` on.
__device__ __forceinline__ void warps_first(uint32_t (*count)[kDigits], uint32_t run) {
  uint32_t n[kSortWarps];
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) n[w] = count[w][threadIdx.x];
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    count[w][threadIdx.x] = run;
    run += n[w];
  }
}

// The lanes that have a pair of the same digit, by a vote for each of its bits
// (a pass's launch takes 8.6 us with it, 10.1 with the instruction that matches whole values).
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, int width, bool in) {
  uint32_t peers = __ballot_sync(0xffffffffu, in);
  for (int b = 0; b < width; ++b) {
    const bool one = (digit >> b) & 1u;
    const uint32_t ones = __ballot_sync(0xffffffffu, one);
    peers &= one ? ones : ~ones;
  }
  return peers;
}

// Stable ranks of N pairs a thread: warps hold consecutive runs of 32 N pairs,
// pair i of a lane the one 32 i + lane places on.  rank: the pair's place among
// those of its digit in its warp; count[warp][digit]: how many the warp has.
template <int N>
__device__ __forceinline__ void warp_ranks(const uint32_t (&digit)[N], const bool (&in)[N], int width,
                                           uint32_t (&rank)[N], uint32_t (&peers)[N], uint32_t* count) {
  const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
#pragma unroll
  for (int i = 0; i < N; ++i) peers[i] = same_digit(digit[i], width, in[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t ahead = __popc(peers[i] & below);
    const uint32_t seen = in[i] ? count[digit[i]] : 0u;
    __syncwarp();
    if (in[i] && ahead == 0) count[digit[i]] = seen + __popc(peers[i]);
    __syncwarp();
    rank[i] = seen + ahead;
  }
}

// Moves a tile's pairs to their places: the digit's first place (all lower
// digits), plus its events in earlier tiles, earlier warps of the tile, and
// earlier places of the warp; and counts the next pass's digits of the tile
// where each pair arrives.  DIRECT: hist holds the tiles' counts; otherwise their
// prefix sums and, in totals, their sums.
template <bool DIRECT>
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(PairSource src, int64_t T, Pass pass, int tiles,
                                                                    const uint32_t* __restrict__ hist,
                                                                    const uint32_t* __restrict__ totals,
                                                                    uint2* __restrict__ out, Pass next,
                                                                    uint32_t* __restrict__ next_hist) {
  constexpr int N = kTile / kSortThreads, kGroups = kSortThreads * 4 / kDigits;
  extern __shared__ uint32_t dyn[];
  uint32_t(*const count)[kDigits] = reinterpret_cast<uint32_t(*)[kDigits]>(dyn);       // [kSortWarps]
  __shared__ uint32_t warp_tot[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const int64_t base = (int64_t)blockIdx.x * kTile + warp * (32 * N) + lane;
  uint2 pair[N];
  uint32_t digit[N], rank[N], peers[N];
  bool in[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    in[i] = base + i * 32 < T;
    pair[i] = in[i] ? src(base + i * 32) : make_uint2(0, 0);
    digit[i] = pass.digit(pair[i].x);
  }
  uint32_t all = 0, earlier = 0;        // this digit's events, and those of them in earlier tiles
  if (DIRECT) {
    // a thread adds four digits' counts of every kGroups-th tile
    uint4 sum = make_uint4(0, 0, 0, 0), mine = make_uint4(0, 0, 0, 0);
    const int group = tid / (kDigits / 4), d4 = tid % (kDigits / 4);
    const uint4* const h = reinterpret_cast<const uint4*>(hist) + d4;
    constexpr int kFlight = 9;
    for (int t0 = group; t0 < tiles; t0 += kFlight * kGroups) {
      uint4 v[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int t = min(t0 + i * kGroups, tiles - 1);
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                     : "l"(h + (int64_t)t * (kDigits / 4))
                     : "memory");
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int t = t0 + i * kGroups;
        const uint32_t there = t < tiles ? 0xffffffffu : 0u, m = t < (int)blockIdx.x ? there : 0u;
        sum.x += v[i].x & there; sum.y += v[i].y & there; sum.z += v[i].z & there; sum.w += v[i].w & there;
        mine.x += v[i].x & m; mine.y += v[i].y & m; mine.z += v[i].z & m; mine.w += v[i].w & m;
      }
    }
    static_assert(2 * kGroups <= kSortWarps, "the groups' sums fit the counters");
    reinterpret_cast<uint4*>(count[group])[d4] = sum;
    reinterpret_cast<uint4*>(count[kGroups + group])[d4] = mine;
    __syncthreads();
    if (tid < kDigits)
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        all += count[g][tid];
        earlier += count[kGroups + g][tid];
      }
    __syncthreads();
  } else if (tid < kDigits) {
    all = totals[tid];
    earlier = hist[(int64_t)blockIdx.x * kDigits + tid];
  }
  clear_counts(count);
  const uint32_t run = block_prefix(all, warp_tot) + earlier;      // where the tile's events of this digit go
  warp_ranks<N>(digit, in, pass.width, rank, peers, count[warp]);
  __syncthreads();
  if (tid < kDigits) warps_first(count, run);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t to = in[i] ? count[warp][digit[i]] + rank[i] : 0u;
    if (in[i]) out[to] = pair[i];
    if (next_hist) {
      // the next pass's counter of the pair (after the last one there is none, nor a digit: its shift may be 32)
      const uint32_t at = in[i] ? to / kTile * kDigits + next.digit(pair[i].x) : 0xffffffffu;
      // once for those of the pair's peers that share the first one's counter (a popular item's all do)
      const int first = __ffs(peers[i]) - 1;
      const uint32_t lead = __shfl_sync(0xffffffffu, at, first < 0 ? 0 : first);
      const uint32_t with = __ballot_sync(0xffffffffu, in[i] && at == lead) & peers[i];
      if (in[i] && (at != lead || lane == first)) atomicAdd(next_hist + at, at != lead ? 1u : (uint32_t)__popc(with));
    }
  }
}

// The word at the same place of shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::cluster_addr(p, rank)) : "memory");
  return v;
}

// All passes of a cluster's CTAs, a tile each: they read one another's counts
// from shared memory, and pass on the pairs through the buffers a and b (L2).
__global__ void __launch_bounds__(kSortThreads) sort_cluster_kernel(PairSource src, int T, int bits, int passes,
                                                                    uint2* a, uint2* b,
                                                                    uint32_t* __restrict__ joins) {
  constexpr int N = kTile / kSortThreads;
  extern __shared__ uint32_t dyn[];
  uint32_t(*const count)[kDigits] = reinterpret_cast<uint32_t(*)[kDigits]>(dyn);       // [kSortWarps]
  __shared__ uint32_t tile_count[kDigits];
  __shared__ uint32_t warp_tot[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const uint32_t rank_of_cta = tc::cluster_rank();
  if (blockIdx.x == 0 && tid < kJoinWords) joins[tid] = 0;
  const int base = (int)blockIdx.x * kTile + warp * (32 * N) + lane;
  const int width = (bits + passes - 1) / passes;
  uint2 pair[N];
  uint32_t digit[N], rank[N], peers[N];
  bool in[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    in[i] = base + i * 32 < T;
    pair[i] = in[i] ? src(base + i * 32) : make_uint2(0, 0);
  }
  for (int p = 0; p < passes; ++p) {
    const Pass pass{p * width, width};
    uint2* const to = p & 1 ? b : a;
    clear_counts(count);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) digit[i] = pass.digit(pair[i].x);
    warp_ranks<N>(digit, in, width, rank, peers, count[warp]);
    __syncthreads();
    if (tid < kDigits) {
      uint32_t n = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) n += count[w][tid];
      tile_count[tid] = n;
    }
    tc::cluster_sync();
    uint32_t all = 0, earlier = 0;
    if (tid < kDigits)
      for (uint32_t r = 0; r < gridDim.x; ++r) {
        const uint32_t n = cluster_load(tile_count + tid, r);
        all += n;
        earlier += r < rank_of_cta ? n : 0u;
      }
    const uint32_t run = block_prefix(all, warp_tot) + earlier;
    if (tid < kDigits) warps_first(count, run);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in[i]) to[count[warp][digit[i]] + rank[i]] = pair[i];
    // the counts have been read and the pairs are written, by every CTA
    tc::cluster_sync();
    if (p + 1 < passes)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (in[i]) pair[i] = __ldcg(to + base + i * 32);
  }
}

// All passes of T <= kSmallSort events, in shared memory; with heads, also
// what heads_kernel leaves for the rows form.
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(PairSource src, int T, int bits, int passes,
                                                                  uint2* __restrict__ out,
                                                                  uint32_t* __restrict__ joins,
                                                                  uint32_t* __restrict__ heads,
                                                                  uint32_t* __restrict__ supers,
                                                                  int64_t* __restrict__ num_rows) {
  constexpr int N = kSmallSort / kSortThreads;
  static_assert(kSmallSort / kChunk <= kSortThreads, "a thread counts a chunk");
  extern __shared__ uint32_t dyn[];
  uint32_t(*const count)[kDigits] = reinterpret_cast<uint32_t(*)[kDigits]>(dyn);       // [kSortWarps]
  uint2* const buf = reinterpret_cast<uint2*>(dyn + kSortWarps * kDigits);              // [kSmallSort]
  __shared__ uint32_t warp_tot[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  if (tid < kJoinWords) joins[tid] = 0;
  // consecutive events in consecutive warps, as few rounds as T takes
  const int per = (T + kSortThreads - 1) / kSortThreads;
  const int base = warp * (32 * per) + lane;
  uint2 pair[N];
  uint32_t digit[N], rank[N], peers[N];
  bool in[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    in[i] = i < per && base + i * 32 < T;
    pair[i] = in[i] ? src(base + i * 32) : make_uint2(0, 0);
  }
  const int width = (bits + passes - 1) / passes;
  for (int p = 0; p < passes; ++p) {
    const Pass pass{p * width, width};
    clear_counts(count);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) digit[i] = pass.digit(pair[i].x);
    warp_ranks<N>(digit, in, width, rank, peers, count[warp]);
    __syncthreads();
    uint32_t all = 0;
    if (tid < kDigits)
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) all += count[w][tid];
    const uint32_t run = block_prefix(all, warp_tot);
    if (tid < kDigits) warps_first(count, run);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in[i]) buf[count[warp][digit[i]] + rank[i]] = pair[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in[i]) pair[i] = buf[base + i * 32];
    if (p + 1 < passes) __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (in[i]) out[base + i * 32] = pair[i];
  if (!heads) return;
  uint32_t n = 0;               // items that begin in this thread's chunk
  const int chunks = (T + kChunk - 1) / kChunk;
  if (tid < chunks) {
    uint32_t left = tid > 0 ? buf[tid * kChunk - 1].x : src.V;
    for (int t = tid * kChunk; t < min((tid + 1) * kChunk, T); ++t) {
      const uint32_t k = buf[t].x;
      n += k < src.V && k != left;
      left = k;
    }
  }
  __syncthreads();              // the last pass has read warp_tot
  const uint32_t before = block_prefix(n, warp_tot);
  if (tid < chunks) {
    heads[tid] = before;
    if (tid % (kSuper / kChunk) == 0) supers[tid / (kSuper / kChunk)] = 0;
    if (tid == chunks - 1) *num_rows = before + n;
  }
}

// ---------------------------------------------------------------------------
// Rows form: how many items begin before each chunk
// ---------------------------------------------------------------------------
// heads[c]: items whose first event lies in an earlier chunk of chunk c's
// kSuper events; supers[s]: in earlier kSuper events than number s; *num_rows:
// in all.  A CTA counts kSuper events; the one that finishes last turns the counts
// into prefix sums (*finished, cleared by the sort, tells).
__global__ void __launch_bounds__(kSuper) heads_kernel(const uint2* __restrict__ pairs, int64_t T, uint32_t V,
                                                       int64_t chunks, uint32_t* __restrict__ heads,
                                                       uint32_t* supers, uint32_t* finished,
                                                       int64_t* __restrict__ num_rows) {
  static_assert(kSuper == 32 * 32, "the warps' counts fit a warp");
  __shared__ uint32_t warp_n[32];
  __shared__ uint32_t carry;
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const auto scan = [lane](uint32_t v) {        // inclusive, over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  const int64_t t = (int64_t)blockIdx.x * kSuper + threadIdx.x;
  bool head = false;
  if (t < T) {
    const uint32_t k = pairs[t].x;
    head = k < V && (t == 0 || pairs[t - 1].x != k);
  }
  const uint32_t n = __popc(__ballot_sync(0xffffffffu, head));
  if (lane == 0) warp_n[warp] = n;
  __syncthreads();
  if (warp == 0) {
    const uint32_t x = warp_n[lane], v = scan(x);
    const int64_t c = (int64_t)blockIdx.x * (kSuper / kChunk) + lane;
    if (c < chunks) heads[c] = v - x;
    if (lane == 31) {
      supers[blockIdx.x] = v;
      __threadfence();
      last = atomicAdd(finished, 1u) == gridDim.x - 1;
      carry = 0;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (uint32_t base = 0; base < gridDim.x; base += kSuper) {
    const uint32_t i = base + threadIdx.x;
    const uint32_t x = i < gridDim.x ? __ldcg(supers + i) : 0u, v = scan(x);
    if (lane == 31) warp_n[warp] = v;
    __syncthreads();
    uint32_t w = lane < warp ? warp_n[lane] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    const uint32_t before = carry + w;
    if (i < gridDim.x) supers[i] = before + v - x;
    __syncthreads();
    if (threadIdx.x == kSuper - 1) carry = before + v;
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
  const uint32_t *heads, *supers;      // rows form: items before each chunk; else NULL
  int64_t* row_ids;
  float* partial;             // [chunks][2][dim]
  // Items that cross chunks, by the chunk where they begin: joins[0] short ones
  // from the front of a list of [chunks], joins[1] long ones from its end.
  uint32_t* joins;
  __device__ __forceinline__ uint32_t* list() const { return joins + kJoinWords; }
  // Items that begin before chunk c.
  __device__ __forceinline__ int64_t before(int64_t c) const {
    return (int64_t)supers[c / (kSuper / kChunk)] + heads[c];
  }
};

// The N columns of a lane in a slice of 32 N: neighbours, read and written in
// one access (NEXT), or, where rows allow no wide access, 32 apart.
template <int N, bool NEXT> struct Lane {
  int col, have;        // the first column, and how many of the N there are
  __device__ __forceinline__ explicit Lane(int dim) {
    const int lane = threadIdx.x & 31;
    col = (int)blockIdx.y * 32 * N + (NEXT ? lane * N : lane);
    const int left = dim - col;
    have = left <= 0 ? 0 : NEXT ? N : min(N, (left + 31) / 32);
    if (!have) col = 0;
  }
  // Of a row's elements from this lane's first column on.
  template <typename T> __device__ __forceinline__ void load(const T* p, Pack<T, N>& a) const {
    if constexpr (NEXT) {
      a.load(p);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) a.v[k] = k < have ? p[32 * k] : from_f<T>(0.f);
    }
  }
  __device__ __forceinline__ void load(const float* p, float (&f)[N]) const {
    if constexpr (NEXT) {
      constexpr int M = N > 4 ? 4 : N;
#pragma unroll
      for (int i = 0; i < N; i += M) {
        Pack<float, M> a;
        a.load(p + i);
#pragma unroll
        for (int k = 0; k < M; ++k) f[i + k] = a.v[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = k < have ? p[32 * k] : 0.f;
    }
  }
  __device__ __forceinline__ void store(float* p, const float (&f)[N]) const {
    if constexpr (NEXT) {
      constexpr int M = N > 4 ? 4 : N;
#pragma unroll
      for (int i = 0; i < N; i += M) {
        Pack<float, M> a;
#pragma unroll
        for (int k = 0; k < M; ++k) a.v[k] = f[i + k];
        a.store(p + i);
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < have) p[32 * k] = f[k];
    }
  }
  // load(), where the program says (volatile: the compiler would move each load of a
  // batch down to its use, and wait for every one of them).
  __device__ __forceinline__ void load_now(const float* p, float (&f)[N]) const {
    if constexpr (NEXT && N >= 4) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(f[i]), "=f"(f[i + 1]), "=f"(f[i + 2]), "=f"(f[i + 3])
                     : "l"(p + i)
                     : "memory");
    } else if constexpr (NEXT && N == 2) {
      asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(f[0]), "=f"(f[1]) : "l"(p) : "memory");
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        asm volatile("ld.global.f32 %0, [%1];" : "=f"(f[k]) : "l"(p + 32 * min(k, have - 1)) : "memory");
    }
  }
};

// A warp sums a chunk's columns [32 N y, 32 N (y + 1)).
// partial[c][0]: the sum of the item that came over from the chunk before;
// partial[c][1]: of the one that begins in the chunk and goes on after it.
// ROWS: items are written to their places in the rows form, else added.
template <typename T, int N, bool NEXT, bool ROWS>
__global__ void __launch_bounds__(256) sum_kernel(SumArgs a, const T* __restrict__ dout) {
  const int lane = threadIdx.x & 31;
  const int64_t c = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (c >= a.chunks) return;
  const int64_t t0 = c * kChunk;
  const int n = (int)min((int64_t)kChunk, a.T - t0);
  const uint2 mine = lane < n ? a.pairs[t0 + lane] : make_uint2(a.V, 0);
  const uint32_t before = t0 > 0 ? a.pairs[t0 - 1].x : a.V;
  const uint32_t after = t0 + n < a.T ? a.pairs[t0 + n].x : a.V;
  const uint32_t far = t0 + (kAlone + 1) * kChunk < a.T ? a.pairs[t0 + (kAlone + 1) * kChunk].x : a.V;
  uint32_t left = __shfl_up_sync(0xffffffffu, mine.x, 1), right = __shfl_down_sync(0xffffffffu, mine.x, 1);
  if (lane == 0) left = before;
  if (lane == n - 1) right = after;
  const bool real = mine.x < a.V;
  const uint32_t begins = __ballot_sync(0xffffffffu, real && left != mine.x);   // an item's first event
  const uint32_t ends = __ballot_sync(0xffffffffu, real && right != mine.x);    // an item's last event
  const int count = __popc(__ballot_sync(0xffffffffu, real));   // padding sorts last
  if (count == 0) return;
  const Lane<N, NEXT> cols(a.dim);
  const T* const src = dout + cols.col;
  float* const dst = a.dst + cols.col;
  const int64_t first_row = ROWS ? a.before(c) - 1 : 0;
  float acc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) acc[k] = 0.f;
#pragma unroll 1
  for (int j0 = 0; j0 < count; j0 += kBatch) {
    Pack<T, N> row[kBatch];
    float old[ROWS ? 1 : kBatch][N];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i;
      const uint32_t key = __shfl_sync(0xffffffffu, mine.x, j & 31), ev = __shfl_sync(0xffffffffu, mine.y, j & 31);
      if (j < count && cols.have) {
        cols.load(src + (int64_t)ev * a.dout_stride, row[i]);
        // what the gradient holds of an item that begins and ends in this chunk
        if (!ROWS && (ends >> j & 1u) && (begins & (0xffffffffu >> (31 - j))))
          cols.load(dst + (int64_t)key * a.dst_stride, old[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i;
      if (j >= count) break;
      const uint32_t key = __shfl_sync(0xffffffffu, mine.x, j);
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += to_f(row[i].v[k]);
      const bool end = ends >> j & 1u;
      if (!end && j + 1 < count) continue;
      const uint32_t begun = begins & (0xffffffffu >> (31 - j));      // items begun so far
      if (!begun || !end) {
        if (cols.have) cols.store(a.partial + (c * 2 + (begun ? 1 : 0)) * a.dim + cols.col, acc);
        if (begun && blockIdx.y == 0 && lane == 0) {
          const int is_long = far == key;
          const int64_t i = atomicAdd(a.joins + is_long, 1u);
          a.list()[is_long ? a.chunks - 1 - i : i] = (uint32_t)c;
        }
      } else if (cols.have) {
        const int64_t at = ROWS ? first_row + __popc(begun) : (int64_t)key;
        float f[N];
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = ROWS ? a.scale * acc[k] : old[ROWS ? 0 : i][k] + a.scale * acc[k];
        cols.store(dst + at * a.dst_stride, f);
      }
      if (ROWS && begun && blockIdx.y == 0 && lane == 0) a.row_ids[first_row + __popc(begun)] = key;
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] = 0.f;
    }
  }
}

// Where the item ends that begins in chunk c and goes on: the last chunk that
// begins with its id.  The warp's lanes probe the next 32 chunks, then 32
// places of what is left, until the places are neighbours.
__device__ __forceinline__ int64_t last_chunk(const SumArgs& a, int64_t c, uint32_t key) {
  const int lane = threadIdx.x & 31;
  int64_t last = c + 1, step = 1, end = a.chunks;
  while (true) {
    const int64_t p = last + step * (lane + 1);
    const uint32_t same = __ballot_sync(0xffffffffu, p < end && a.pairs[p * kChunk].x == key);
    const int run = __popc(same);             // the ids are sorted: a run of lanes from the first
    last += step * run;
    if (run == 32) {
      step = (end - last + 31) / 32;          // at least 1: last is a chunk
    } else if (step == 1) {
      return last;
    } else {
      end = min(end, last + step);
      step = (step + 31) / 32;
    }
  }
}

// Adds the partial sums of chunks first, first + STRIDE, ... up to last (at
// least one), kFlight of them in flight; places past the last load that one again.
template <int STRIDE, int kFlight, int N, bool NEXT>
__device__ __forceinline__ void add_partials(const SumArgs& a, int64_t first, int64_t last, const Lane<N, NEXT>& cols,
                                             float (&acc)[N]) {
  const float* p = a.partial + first * 2 * a.dim + cols.col;
  const int64_t step = (int64_t)STRIDE * 2 * a.dim;
  for (int64_t left = (last - first) / STRIDE + 1; left > 0; left -= kFlight, p += kFlight * step) {
    float f[kFlight][N];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) cols.load_now(p + min((int64_t)i, left - 1) * step, f[i]);
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += i < left ? f[i][k] : 0.f;
  }
}

template <bool ROWS, int N, bool NEXT>
__device__ __forceinline__ void put_joined(const SumArgs& a, int64_t c, uint32_t key, const Lane<N, NEXT>& cols,
                                           const float (&acc)[N]) {
  const int64_t at = ROWS ? a.before(c + 1) - 1 : (int64_t)key;
  float* const p = a.dst + at * a.dst_stride + cols.col;
  float f[N];
  if (!ROWS) cols.load(p, f);
#pragma unroll
  for (int k = 0; k < N; ++k) f[k] = ROWS ? a.scale * acc[k] : f[k] + a.scale * acc[k];
  cols.store(p, f);
}

// Joins the partial sums of the listed items, columns [32 N y, 32 N (y + 1)) of
// each: CTAs [0, longs) the long items, one at a time, whose warps add every
// kJoinWarps-th chunk; the others the short ones, a warp each.
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;
template <int N, bool NEXT, bool ROWS>
__global__ void __launch_bounds__(kJoinThreads, N > 4 || !NEXT ? 2 : 3) join_kernel(SumArgs a, unsigned longs) {
  __shared__ float strip[kJoinWarps][32 * N];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const Lane<N, NEXT> cols(a.dim);
  if (blockIdx.x >= longs) {
    const uint32_t items = a.joins[0];
    for (uint32_t i = (blockIdx.x - longs) * kJoinWarps + w; i < items; i += (gridDim.x - longs) * kJoinWarps) {
      const int64_t c = a.list()[i];
      const uint32_t key = a.pairs[(c + 1) * kChunk].x;
      const int64_t last = last_chunk(a, c, key);
      if (!cols.have) continue;
      float acc[N];
      cols.load(a.partial + (c * 2 + 1) * a.dim + cols.col, acc);
      add_partials<1, 4>(a, c + 1, last, cols, acc);
      put_joined<ROWS>(a, c, key, cols, acc);
    }
    return;
  }
  const uint32_t items = a.joins[1];
  for (uint32_t i = blockIdx.x; i < items; i += longs) {
    const int64_t c = a.list()[a.chunks - 1 - i];
    const uint32_t key = a.pairs[(c + 1) * kChunk].x;
    const int64_t last = last_chunk(a, c, key);
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    if (cols.have) {
      if (w == 0) cols.load(a.partial + (c * 2 + 1) * a.dim + cols.col, acc);
      add_partials<kJoinWarps, 8>(a, c + 1 + w, last, cols, acc);     // longer than kJoinWarps chunks
    }
#pragma unroll
    for (int k = 0; k < N; ++k) strip[w][k * 32 + lane] = acc[k];
    __syncthreads();
    if (w == 0 && cols.have) {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int o = 1; o < kJoinWarps; ++o) acc[k] += strip[o][k * 32 + lane];
      put_joined<ROWS>(a, c, key, cols, acc);
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
  size_t a, b, hist, totals, heads, supers, joins, partial, total;
  int64_t tiles, chunks, nsupers;
};
BwdLayout bwd_layout(int64_t T, int dim) {
  BwdLayout l;
  l.tiles = (T + kTile - 1) / kTile;
  l.chunks = (T + kChunk - 1) / kChunk;
  l.nsupers = (T + kSuper - 1) / kSuper;
  l.a = 0;
  l.b = align_up(l.a + (size_t)T * 8, 256);
  l.hist = align_up(l.b + (size_t)T * 8, 256);
  l.totals = align_up(l.hist + (size_t)l.tiles * kDigits * 4 * kMaxPasses, 256);
  l.heads = align_up(l.totals + kDigits * 4, 256);
  l.supers = align_up(l.heads + (size_t)l.chunks * 4, 256);
  l.joins = align_up(l.supers + (size_t)l.nsupers * 4, 256);
  l.partial = align_up(l.joins + kJoinWords * 4 + (size_t)l.chunks * 4, 256);
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

template <typename T, int N, bool NEXT, bool ROWS>
cudaError_t launch_sum_n(const SumArgs& a, const void* dout, cudaStream_t s) {
  const unsigned slices = (unsigned)((a.dim + 32 * N - 1) / (32 * N));
  sum_kernel<T, N, NEXT, ROWS><<<dim3((unsigned)((a.chunks + 7) / 8), slices), 256, 0, s>>>(a, static_cast<const T*>(dout));
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.chunks > 1) {
    // CTAs for as many items as there can be, at most one (long) and two
    // (short) a multiprocessor
    const int64_t sms = sm_count(), most = (sms + slices - 1) / slices;
    const int64_t longs = std::min(most, (a.chunks + kAlone - 1) / kAlone);
    const int64_t shorts = std::min(2 * most, (a.chunks + kJoinWarps - 1) / kJoinWarps);
    join_kernel<N, NEXT, ROWS><<<dim3((unsigned)(longs + shorts), slices), kJoinThreads, 0, s>>>(a, (unsigned)longs);
    count_launch();
    e = cudaGetLastError();
  }
  return e;
}
// N columns a lane: 16 bytes of dout where alignment and width allow, fewer
// rather than idle lanes for narrow rows; where rows allow no wide access, four
// that are 32 apart (201,528 x 333: 184 us, 205 with one).
template <typename T, bool ROWS>
cudaError_t launch_sum(const SumArgs& a, const void* dout, cudaStream_t s) {
  constexpr int kMost = 16 / (int)sizeof(T);
  int n = kMost;
  while (n > 1 && !(vec_ok(n, dout, sizeof(T), a.dout_stride, a.dim, a.dim) &&
                    vec_ok(n < 4 ? n : 4, a.dst, 4, a.dst_stride, a.dim, a.dim) && (n == 2 || a.dim > 16 * n)))
    n >>= 1;
  if constexpr (kMost == 8)
    if (n == 8) return launch_sum_n<T, 8, true, ROWS>(a, dout, s);
  if (n == 4) return launch_sum_n<T, 4, true, ROWS>(a, dout, s);
  if (n == 2) return launch_sum_n<T, 2, true, ROWS>(a, dout, s);
  return a.dim > 64 ? launch_sum_n<T, 4, false, ROWS>(a, dout, s) : launch_sum_n<T, 1, false, ROWS>(a, dout, s);
}

// The gradient in either form; rows form when row_ids is given.
cudaError_t embedding_bwd(const void* dout, int dout_dtype, int64_t dout_stride, const void* ids, int id_bytes,
                          int64_t T, int64_t V, int dim, float scale, float* dst, int64_t dst_stride,
                          int64_t* row_ids, int64_t* num_rows, void* ws, cudaStream_t s) {
  const BwdLayout l = bwd_layout(T, dim);
  char* const base = static_cast<char*>(ws);
  uint2* pairs[2] = {reinterpret_cast<uint2*>(base + l.a), reinterpret_cast<uint2*>(base + l.b)};
  uint32_t* const hist = reinterpret_cast<uint32_t*>(base + l.hist);
  uint32_t* const totals = reinterpret_cast<uint32_t*>(base + l.totals);
  uint32_t* const joins = reinterpret_cast<uint32_t*>(base + l.joins);
  uint32_t* const heads = reinterpret_cast<uint32_t*>(base + l.heads);
  uint32_t* const supers = reinterpret_cast<uint32_t*>(base + l.supers);
  int bits = 0;
  while (((uint64_t)V >> bits) != 0) ++bits;                      // keys are 0 .. V
  const int passes = (bits + 8) / 9, width = (bits + passes - 1) / passes;
  PairSource src{nullptr, ids, id_bytes, (uint32_t)V};
  cudaError_t e = cudaSuccess;
  if (T <= kSmallSort) {
    constexpr int kBytes = kSortWarps * kDigits * 4 + kSmallSort * 8;
    e = cudaFuncSetAttribute(sort_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    sort_small_kernel<<<1, kSortThreads, kBytes, s>>>(src, (int)T, bits, passes, pairs[0], joins,
                                                      row_ids ? heads : nullptr, supers, num_rows);
    count_launch();
    src.pairs = pairs[0];
  } else if (l.tiles <= kSortCluster) {
    constexpr int kBytes = kSortWarps * kDigits * 4;
    e = cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)l.tiles;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)l.tiles);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, sort_cluster_kernel, src, (int)T, bits, passes, pairs[0], pairs[1], joins);
    count_launch();
    if (e != cudaSuccess) return e;
    src.pairs = pairs[(passes - 1) & 1];
  } else {
    const int64_t stride = l.tiles * kDigits;
    constexpr int kBytes = kSortWarps * kDigits * 4;
    const bool direct = l.tiles <= kDirectTiles;
    e = cudaFuncSetAttribute(direct ? sort_scatter_kernel<true> : sort_scatter_kernel<false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    const auto pass = [&](int p) { return Pass{p * width, width}; };
    sort_hist_kernel<<<(unsigned)l.tiles, kSortThreads, 0, s>>>(src, T, pass(0), passes, hist, stride, joins);
    count_launch();
    for (int p = 0; p < passes; ++p) {
      uint32_t* const h = hist + p * stride;
      uint32_t* const next = p + 1 < passes ? h + stride : nullptr;
      if (direct) {
        sort_scatter_kernel<true><<<(unsigned)l.tiles, kSortThreads, kBytes, s>>>(src, T, pass(p), (int)l.tiles, h, totals,
                                                                             pairs[p & 1], pass(p + 1), next);
      } else {
        sort_scan_kernel<<<kDigits, 256, 0, s>>>(h, (int)l.tiles, totals);
        count_launch();
        sort_scatter_kernel<false><<<(unsigned)l.tiles, kSortThreads, kBytes, s>>>(src, T, pass(p), (int)l.tiles, h, totals,
                                                                              pairs[p & 1], pass(p + 1), next);
      }
      count_launch();
      src.pairs = pairs[p & 1];
    }
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
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
  a.heads = heads;
  a.supers = supers;
  a.row_ids = row_ids;
  a.partial = reinterpret_cast<float*>(base + l.partial);
  a.joins = joins;
  if (!row_ids)
    return dout_dtype == HSTU_BF16 ? launch_sum<bf16, false>(a, dout, s) : launch_sum<float, false>(a, dout, s);
  if (T > kSmallSort) {
    heads_kernel<<<(unsigned)l.nsupers, kSuper, 0, s>>>(src.pairs, T, (uint32_t)V, l.chunks, heads, supers, joins + 2,
                                                        num_rows);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return dout_dtype == HSTU_BF16 ? launch_sum<bf16, true>(a, dout, s) : launch_sum<float, true>(a, dout, s);
}

// Rows that allow no wider access go to lookup_rows_kernel from this width on (67
// million elements, fp32 with the bf16 copy: width 33 178 us by pieces, 297 by rows; 65
// 174 and 173; 101 172 and 125; 333 168 and 94).
constexpr int kRowsFrom = 64;
template <typename TT, typename TO, bool LOW>
cudaError_t launch_lookup(const void* table, int64_t V, int dim, int64_t table_stride, const void* ids,
                          int id_bytes, int64_t T, float scale, void* out, int width, int64_t out_stride,
                          void* low, int64_t low_stride, cudaStream_t s) {
  // 16 bytes of the widest side, if alignment and widths allow
  constexpr int kMost = sizeof(TT) == 2 && sizeof(TO) == 2 ? 8 : 4;
  int n = kMost;
  while (n > 1 && !(vec_ok(n, table, sizeof(TT), table_stride, dim, width) &&
                    vec_ok(n, out, sizeof(TO), out_stride, dim, width) &&
                    (!LOW || vec_ok(n, low, 2, low_stride, dim, width))))
    n >>= 1;
  const bool by_rows = n == 1 && width >= kRowsFrom;
  const int64_t ctas = by_rows ? (T + 7) / 8 : (T * (width / n) + 256 * kLookups - 1) / (256 * kLookups);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)ctas;
  const TT* t = static_cast<const TT*>(table);
  TO* o = static_cast<TO*>(out);
  bf16* l = static_cast<bf16*>(low);
  if (by_rows) {
    lookup_rows_kernel<TT, TO, LOW><<<grid, 256, 0, s>>>(t, V, dim, table_stride, ids, id_bytes, T, scale, o, width,
                                                         out_stride, l, low_stride);
    count_launch();
    return cudaGetLastError();
  }
#define HSTU_LAUNCH(N)                                                                                          \
  lookup_kernel<TT, TO, N, LOW><<<grid, 256, 0, s>>>(t, V, dim, table_stride, ids, id_bytes, T, scale, o, width, \
                                                     out_stride, l, low_stride)
  if (n == kMost) HSTU_LAUNCH(kMost);
  else if (n == 4) HSTU_LAUNCH(4);
  else if (n == 2) HSTU_LAUNCH(2);
  else HSTU_LAUNCH(1);
#undef HSTU_LAUNCH
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
