// Embedding of tokens by one range of the vocabulary, and the table's gradient
// by sorted tokens.
//
// The gradient sorts the tokens (stable counting sorts, ops_sort.cuh), cuts
// the sorted places into runs of kRun, and sums each token's rows of a run in
// order.  A token whose places all lie in one run is finished there; the parts
// of one that crosses runs go to the workspace in binary32 and are joined in
// the runs' order by a second kernel.  Every sum has one fixed order, so the
// gradient is the same from call to call.
#include <type_traits>

#include "ops_common.cuh"
#include "ops_sort.cuh"

namespace pl {
namespace {

__device__ __forceinline__ int64_t token_of(const EmbedArgs& a, uint64_t i) {
  return a.wide_tokens ? ((const int64_t*)a.tokens)[i] : (int64_t)((const int32_t*)a.tokens)[i];
}

// Row of the table, or `rows` for a token outside the range.
__device__ __forceinline__ uint64_t row_of(const EmbedArgs& a, uint64_t i) {
  const uint64_t r = (uint64_t)token_of(a, i) - (uint64_t)a.first;  // wraps to a large value below the range
  return r < a.rows ? r : a.rows;
}

// y = scale x the token's row, in binary32, rounded once.  A group of tpt threads
// takes U tokens and keeps one vector of each in flight.  Bound by DRAM, mostly
// its writes: 32768 x 5120 bf16, a quarter of the tokens in the range, 55 us, 6.4
// TB/s.  SHIFT (rows at any address): 4096 x 1537 binary32, 10 us.
template <typename T, bool SHIFT, int U>
__global__ void __launch_bounds__(kRowThreads) embed_kernel(const __grid_constant__ EmbedArgs a, int tpt) {
  op_wait();
  constexpr int V = V16<T>;
  static_assert(!SHIFT || U == 1, "tokens of one thread cut their rows alike");
  const int per = blockDim.x / tpt, lane = threadIdx.x % tpt;
  const uint64_t t0 = (uint64_t)blockIdx.x * per * U + threadIdx.x / tpt;
  const T* x[U];
  bool in[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t t = t0 + u * per, row = t < a.n ? row_of(a, t) : a.rows;
    in[u] = row < a.rows;
    x[u] = (const T*)a.x + row * a.ldx;
  }
  const Cut c = cut_of<T, SHIFT>((T*)a.y + t0 * a.ldy, a.width);
  for (uint64_t v = lane; v < c.nv + c.beside; v += tpt) {
    if (SHIFT && v >= c.nv) {
      const uint64_t e = c.at<V>((uint32_t)(v - c.nv));
      if (t0 < a.n) ((T*)a.y)[t0 * a.ldy + e] = from_f32<T>(ld1_if(x[0] + e, in[0]) * (in[0] ? a.scale : 0.f));
      continue;
    }
    Pack<T, V> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = ld_row_if<T, SHIFT>(x[u] + c.head + v * V, in[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) pin(r[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint64_t t = t0 + u * per;
      if (t >= a.n) continue;
      // a token outside the range is 0, whatever the scale
#pragma unroll
      for (int i = 0; i < V; ++i) r[u].v[i] = from_f32<T>(to_f32(r[u].v[i]) * (in[u] ? a.scale : 0.f));
      st_pack_once<T, V>((T*)a.y + t * a.ldy + c.head + v * V, r[u]);
    }
  }
}

// ------------------------------------------------------- sort of the tokens

// A whole number of T's size: rows that are copied or cleared, whatever they hold.
template <typename T>
using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;

// More tokens than a cluster sorts: one digit of the sort in two launches (about
// 9 us, most of it the launches and the wait of one for the other), of (key,
// index) pairs, or the tokens themselves when in_key is null.  Keys are rows of
// the table; rows = outside, sorted last.
struct SortArgs {
  EmbedArgs e;
  const uint32_t *in_key, *in_idx;
  uint32_t *out_key, *out_idx;
  uint32_t* counts;
  int shift, bits, passes;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint64_t i) {
  return a.in_key ? a.in_key[i] : (uint32_t)row_of(a.e, i);
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortArgs a, uint32_t chunk) {
  op_wait();
  op_next();
  __shared__ uint32_t hist[kSortBins];
  const int bins = 1 << a.bits;
  for (int b = threadIdx.x; b < bins; b += blockDim.x) hist[b] = 0;
  __syncthreads();
  const uint64_t i0 = (uint64_t)blockIdx.x * chunk;
  for (uint32_t i = threadIdx.x; i < chunk && i0 + i < a.e.n; i += blockDim.x)
    atomicAdd(hist + (sort_key(a, i0 + i) >> a.shift & (bins - 1)), 1u);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += blockDim.x) a.counts[(uint64_t)blockIdx.x * bins + b] = hist[b];
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const __grid_constant__ SortArgs a, uint32_t chunk,
                                                                  int ipt) {
  extern __shared__ uint16_t cnt[];
  __shared__ uint32_t base[kSortBins], before[kSortBins], tmp[33];
  const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t i0 = (uint64_t)blockIdx.x * chunk;
  int digit[kSortIpt];
  uint32_t local[kSortIpt], key[kSortIpt];
#pragma unroll
  for (int q = 0; q < kSortIpt; ++q)
    if (q < ipt) {
      const uint64_t i = i0 + (uint64_t)(warp * ipt + q) * 32 + lane;
      key[q] = i < a.e.n ? sort_key(a, i) : 0;
      digit[q] = i < a.e.n ? (int)(key[q] >> a.shift & (bins - 1)) : -1;
    }
  rank_chunk(digit, local, ipt, bins, cnt, [](int, uint32_t) {});
  op_wait();
  sum_chunks(a.counts, gridDim.x, blockIdx.x, bins, base, before);
  uint32_t carry = 0;
  for (int b0 = 0; b0 < bins; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    uint32_t total;
    const uint32_t at = carry + block_exclusive(b < bins ? base[b] : 0, tmp, &total);
    if (b < bins) base[b] = at + before[b];
    carry += total;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kSortIpt; ++q)
    if (q < ipt && digit[q] >= 0) {
      const uint64_t i = i0 + (uint64_t)(warp * ipt + q) * 32 + lane;
      const uint32_t p = base[digit[q]] + cnt[warp * bins + digit[q]] + local[q];
      a.out_key[p] = key[q];
      a.out_idx[p] = a.in_idx ? a.in_idx[i] : (uint32_t)i;
    }
}

// All digits by one cluster.  Its CTAs hold the items in place order, per =
// 1024 x ipt each; a digit reads them into registers, and writes them to their
// new places in all CTAs' shared memory, the last digit to the workspace.
__device__ __forceinline__ void cluster_sort(const SortArgs& a, int ipt, char* shared) {
  const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  __shared__ uint32_t hist[kSortBins], base[kSortBins], tmp[33];
  const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t n = (uint32_t)a.e.n, per = kClusterThreads * ipt, i0 = cluster.block_rank() * per;
  const int log_per = 31 - __clz(per);
  uint32_t *keys = (uint32_t*)shared, *idx = keys + per;
  uint16_t* cnt = (uint16_t*)(idx + per);
  for (int p = 0; p < a.passes; ++p) {
    int digit[kSortIpt];
    uint32_t local[kSortIpt], key[kSortIpt], id[kSortIpt];
#pragma unroll
    for (int q = 0; q < kSortIpt; ++q)
      if (q < ipt) {
        const uint32_t at = (uint32_t)(warp * ipt + q) * 32 + lane, i = i0 + at;
        digit[q] = -1;
        if (i < n) {
          key[q] = p ? keys[at] : (uint32_t)row_of(a.e, i);
          id[q] = p ? idx[at] : i;
          digit[q] = (int)(key[q] >> (p * a.bits) & (bins - 1));
        }
      }
    rank_chunk(digit, local, ipt, bins, cnt, [&](int b, uint32_t c) { hist[b] = c; });
    cluster_bases(hist, bins, base, tmp);
#pragma unroll
    for (int q = 0; q < kSortIpt; ++q)
      if (q < ipt && digit[q] >= 0) {
        const uint32_t to = base[digit[q]] + cnt[warp * bins + digit[q]] + local[q];
        if (p + 1 < a.passes) {
          cluster.map_shared_rank(keys, to >> log_per)[to & (per - 1)] = key[q];
          cluster.map_shared_rank(idx, to >> log_per)[to & (per - 1)] = id[q];
        } else {
          a.out_key[to] = key[q];
          a.out_idx[to] = id[q];
        }
      }
    cluster.sync();
  }
}

// Row r of the table's gradient where no token names it: zero, or the base's
// bits, by `lanes` threads.
template <typename T, bool SHIFT>
__device__ __forceinline__ void fill_row(const EmbedArgs& a, uint64_t r, int lane, int lanes) {
  constexpr int V = V16<T>;
  T* y = (T*)a.y + r * a.ldy;
  const T* b = (const T*)a.base + r * a.ldb;
  const Cut c = cut_of<T, SHIFT>(y, a.width);
  if (!a.base) {
    for (uint64_t v = lane; v < c.nv; v += lanes) st_pack_once<T, V>(y + c.head + v * V, Pack<T, V>{});
  } else {
#pragma unroll 4
    for (uint64_t v = lane; v < c.nv; v += lanes)
      st_pack_once<T, V>(y + c.head + v * V, ld_row_if<T, SHIFT>(b + c.head + v * V, true));
  }
  for (uint32_t i = lane; SHIFT && i < c.beside; i += lanes) {
    const uint64_t e = c.at<V>(i);
    y[e] = a.base ? b[e] : T{};
  }
}

// Fills what no token names of rows r0 .. r1.  The rows that tokens name are
// marked in a bitmap first, by a look at all tokens.
constexpr uint64_t kBitmapRows = 1 << 18;
template <typename T, bool SHIFT>
__device__ __forceinline__ void fill_rows(const EmbedArgs& a, uint64_t r0, uint64_t r1, uint32_t* bits) {
  int lanes = 32;  // per row
  while (lanes > 1 && (uint64_t)lanes / 2 >= a.width / V16<T>) lanes /= 2;
  for (uint64_t s0 = r0; s0 < r1; s0 += kBitmapRows) {
    const uint32_t rows = (uint32_t)min(kBitmapRows, r1 - s0);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < (rows + 31) / 32; i += blockDim.x) bits[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (uint64_t i = threadIdx.x; i < a.n; i += blockDim.x) {
      const uint64_t r = row_of(a, i) - s0;
      if (r < rows) atomicOr(bits + r / 32, 1u << (r % 32));
    }
    __syncthreads();
    for (uint32_t k = threadIdx.x / lanes; k < rows; k += blockDim.x / lanes)
      if (!(bits[k / 32] >> (k % 32) & 1u)) fill_row<T, SHIFT>(a, s0 + k, threadIdx.x % lanes, lanes);
  }
}

// The first cluster sorts, the others fill: that needs no sorted tokens and
// mostly takes longer than the sort.  Bound by DRAM's writes: 16384 tokens beside
// 52000 rows of 4096 bf16 zeros, 82 us, 5.2 TB/s of stores.
template <typename T, bool SHIFT>
__global__ void __launch_bounds__(kClusterThreads) sort_fill_kernel(const __grid_constant__ SortArgs a, int ipt) {
  op_wait();
  op_next();
  extern __shared__ char dyn[];
  const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const uint32_t skip = a.e.n ? cluster.num_blocks() : 0;
  if (blockIdx.x < skip) {
    cluster_sort(a, ipt, dyn);
    return;
  }
  const uint64_t part = blockIdx.x - skip, parts = gridDim.x - skip;
  fill_rows<T, SHIFT>(a.e, a.e.rows * part / parts, a.e.rows * (part + 1) / parts, (uint32_t*)dyn);
}

// ------------------------------------------------------- sums of sorted rows

constexpr int kRun = 32;          // sorted places of one run, at most
constexpr int kSumThreads = 256;  // one vector of the row each, at most

struct SumArgs {
  EmbedArgs e;
  const uint32_t *key, *idx;
  float* part;      // [run][head, tail][width]
  uint64_t runs;
  uint32_t run;     // places of a run
  uint32_t tiles;   // column tiles of a row
  uint64_t fills;   // CTAs that fill kFill rows each, before those that sum
};

// The same as fill_rows where the tokens are sorted already and too many to
// look at: each row is searched among them.
constexpr int kFill = 32;
template <typename TY, int N>
__device__ __forceinline__ void fill_searched(const SumArgs& a, uint64_t r0) {
  __shared__ uint32_t touched;
  if (threadIdx.x < 32) {
    const uint64_t r = r0 + threadIdx.x;
    uint64_t lo = 0, hi = a.e.n;
    while (lo < hi) {
      const uint64_t mid = (lo + hi) / 2;
      if (a.key[mid] < r) lo = mid + 1;
      else hi = mid;
    }
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, r >= a.e.rows || (lo < a.e.n && a.key[lo] == r));
    if (threadIdx.x == 0) touched = m;
  }
  __syncthreads();
  const int warps = blockDim.x / 32;
  for (int k = threadIdx.x / 32; k < kFill; k += warps)
    if (!(touched >> k & 1u)) fill_row<Bits<TY>, N * sizeof(TY) != 16>(a.e, r0 + k, threadIdx.x % 32, 32);
}

template <typename TY, int N>
__device__ __forceinline__ void finish(const SumArgs& a, uint64_t row, uint64_t c, const float (&acc)[N]) {
  Pack<TY, N> o;
  if (a.e.base) {
    // may be the row written next, so not through the read-only path
    o = *reinterpret_cast<const Pack<TY, N>*>((const TY*)a.e.base + row * a.e.ldb + c);
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<TY>(__fadd_rn(to_f32(o.v[i]), acc[i] * a.e.scale));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<TY>(acc[i] * a.e.scale);
  }
  st_pack_once<TY, N>((TY*)a.e.y + row * a.e.ldy + c, o);
}

// N binary32 sums of the workspace, which is 16-byte aligned and no more: in
// accesses of at most 16 bytes.
template <int N>
__device__ __forceinline__ void st_part(float* part, const float (&acc)[N]) {
  constexpr int W = N < 4 ? N : 4;
#pragma unroll
  for (int q = 0; q < N; q += W) {
    Pack<float, W> o;
#pragma unroll
    for (int i = 0; i < W; ++i) o.v[i] = acc[q + i];
    st_pack<float, W>(part + q, o);
  }
}
template <int N>
__device__ __forceinline__ void ld_part(const float* part, float (&x)[N]) {
  constexpr int W = N < 4 ? N : 4;
#pragma unroll
  for (int q = 0; q < N; q += W) {
    const Pack<float, W> r = *reinterpret_cast<const Pack<float, W>*>(part + q);
#pragma unroll
    for (int i = 0; i < W; ++i) x[q + i] = r.v[i];
  }
}

// One run's columns by one thread for each vector: 8 of the run's rows in flight,
// added in the order of their places, and a token's sum written when its places
// end.  Runs of equal length share out the tokens that occur often.  Bound by
// DRAM's reads: 16384 tokens x 4096 bf16, 31 us, 6.4 TB/s (with 16 or 64 places a
// run 7 and 9% slower).
template <typename TX, typename TY, int N>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const __grid_constant__ SumArgs a) {
  op_wait();
  op_next();
  if (blockIdx.x < a.fills) {
    fill_searched<TY, N>(a, (uint64_t)blockIdx.x * kFill);
    return;
  }
  const uint64_t block = blockIdx.x - a.fills;
  __shared__ uint32_t key[kRun + 2], idx[kRun];  // key[1 + i]: place i of the run; its neighbours at the ends
  const uint64_t run = block / a.tiles, p0 = run * a.run;
  const int n = (int)(a.e.n - p0 < a.run ? a.e.n - p0 : a.run);
  const uint32_t none = 0xFFFFFFFFu;
  for (int i = threadIdx.x; i < n + 2; i += blockDim.x) {
    const uint64_t p = p0 + i;  // place p - 1
    key[i] = p >= 1 && p <= a.e.n ? a.key[p - 1] : none;
    if (i >= 1 && i <= n) idx[i - 1] = a.idx[p - 1];
  }
  __syncthreads();
  const uint64_t c = ((block % a.tiles) * blockDim.x + threadIdx.x) * N;
  if (c >= a.e.width) return;
  const uint32_t rows = (uint32_t)a.e.rows;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  bool head = key[0] == key[1];  // the first token's earlier places are in the run before
  constexpr int U = 8;
  for (int q = 0; q < n; q += U) {
    Pack<TX, N> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      x[u] = ld_pack_if<TX, N>((const TX*)a.e.x + (uint64_t)idx[min(q + u, n - 1)] * a.e.ldx + c, q + u < n && key[q + u + 1] < rows);
#pragma unroll
    for (int u = 0; u < U; ++u) pin(x[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (q + u >= n) break;
      const uint32_t k = key[q + u + 1];
      if (k >= rows) break;  // outside: these sort last
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += to_f32(x[u].v[i]);
      const bool more = key[q + u + 2] == k;
      if (more && q + u + 1 < n) continue;
      if (!head && !more) {
        finish<TY, N>(a, k, c, acc);
      } else {
        st_part<N>(a.part + (run * 2 + (head ? 0 : 1)) * a.e.width + c, acc);
      }
      head = false;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
    }
  }
}

// The token whose first place lies in this run and that goes on in the next:
// its tail here, then the heads of the runs that it reaches.  7 us where the most
// frequent of 16384 tokens has a thousand places: three round trips and the
// launch.
template <typename TX, typename TY, int N>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const __grid_constant__ SumArgs a) {
  op_wait();
  const uint64_t run = blockIdx.x / a.tiles, p0 = run * a.run, p1 = p0 + a.run;
  if (p1 >= a.e.n) return;
  // loaded together: one after another they would take three round trips
  const uint32_t k = a.key[p1 - 1], next = a.key[p1], earlier = p0 > 0 ? a.key[p0 - 1] : 0xFFFFFFFFu;
  if (k >= (uint32_t)a.e.rows || next != k || earlier == k) return;
  // how many runs it reaches, so that the loads below need not wait for keys
  __shared__ uint32_t reach;
  if (threadIdx.x == 0) reach = 0;
  __syncthreads();
  for (uint64_t r = run + 1 + threadIdx.x; r < a.runs && a.key[r * a.run] == k; r += blockDim.x)
    atomicMax(&reach, (uint32_t)(r - run));
  __syncthreads();
  const uint64_t c = ((uint64_t)(blockIdx.x % a.tiles) * blockDim.x + threadIdx.x) * N;
  if (c >= a.e.width) return;
  float acc[N];
  const float* part = a.part + (run * 2 + 1) * a.e.width + c;
  ld_part<N>(part, acc);
  part += a.e.width;
  const uint32_t heads = reach;
#pragma unroll 16
  for (uint32_t r = 0; r < heads; ++r) {
    float x[N];
    ld_part<N>(part + (uint64_t)r * 2 * a.e.width, x);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += x[i];
  }
  finish<TY, N>(a, k, c, acc);
}

// Digits of the sort: as few as 10-bit digits allow, of equal size.
void digits_of(uint64_t rows, int* passes, int* bits) {
  int b = 1;
  while (rows >> b) ++b;  // keys 0 .. rows
  *passes = (b + 9) / 10;
  *bits = (b + *passes - 1) / *passes;
}

// Places of a run: 32, or fewer (8 at least) until the runs of 256-thread
// tiles fill the SMs twice.
uint32_t run_of(uint64_t n, uint64_t width) {
  uint32_t run = kRun;
  while (run > 8 && (n + run - 1) / run * ((width + 2047) / 2048) < 2 * 152) run /= 2;
  return run;
}

struct Space {
  uint64_t key[2], idx[2], counts, part, end;
};

Space space_of(uint64_t n, uint64_t rows, uint64_t width) {
  int passes, bits;
  digits_of(rows, &passes, &bits);
  const bool one = n <= kClusterSort;
  const uint64_t run = run_of(n, width), runs = (n + run - 1) / run;
  Space s;
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t p = at;
    at += (bytes + 255) & ~(uint64_t)255;
    return p;
  };
  s.key[0] = take(n * 4);
  s.idx[0] = take(n * 4);
  s.key[1] = take(one ? 0 : n * 4);
  s.idx[1] = take(one ? 0 : n * 4);
  s.counts = take(one ? 0 : sort_chunks(n) * ((uint64_t)4 << bits));
  s.part = take(runs > 1 ? runs * 2 * width * 4 : 0);
  s.end = at;
  return s;
}

template <typename TX, typename TY>
purlin_status sums(const SumArgs& in, cudaStream_t s) {
  // one vector of N elements is loaded from x, base and y and, as binary32, from the workspace
  const uint64_t elems = in.e.ldx | in.e.ldy | in.e.ldb | in.e.width;
  auto fits = [&](int n) {
    return elems % n == 0 && (uintptr_t)in.e.x % (n * sizeof(TX)) == 0 && (uintptr_t)in.e.y % (n * sizeof(TY)) == 0 &&
           (uintptr_t)in.e.base % (n * sizeof(TY)) == 0;
  };
  constexpr int kMost = 16 / (sizeof(TX) > sizeof(TY) ? sizeof(TX) : sizeof(TY));
  auto go = [&](auto n) -> purlin_status {
    constexpr int N = decltype(n)::value;
    SumArgs a = in;
    const uint64_t nv = a.e.width / N;
    a.tiles = (uint32_t)((nv + kSumThreads - 1) / kSumThreads);
    const int threads = (int)((nv + a.tiles * 32 - 1) / (a.tiles * 32)) * 32;
    if (purlin_status st = op_launch(sum_kernel<TX, TY, N>, a.fills + a.runs * a.tiles, threads, 0, s, a)) return st;
    if (a.runs < 2) return PL_OK;
    return op_launch(join_kernel<TX, TY, N>, a.runs * a.tiles, threads, 0, s, a);
  };
  if constexpr (kMost >= 8)
    if (fits(8)) return go(std::integral_constant<int, 8>());
  if (fits(4)) return go(std::integral_constant<int, 4>());
  if (fits(2)) return go(std::integral_constant<int, 2>());
  return go(std::integral_constant<int, 1>());
}

template <typename T>
purlin_status embed_t(const EmbedArgs& a, cudaStream_t s) {
  const uint64_t bits = (uint64_t)(uintptr_t)a.x | (uint64_t)(uintptr_t)a.y | (a.ldx | a.ldy | a.width) * sizeof(T);
  const RowShape c = RowShape::of<T>(a.width, bits % 16 != 0);
  auto go = [&](auto shift, auto u) {
    constexpr int U = decltype(u)::value;
    return op_launch(embed_kernel<T, decltype(shift)::value, U>, c.ctas(a.n, U), c.tpt * c.per, 0, s, a, c.tpt);
  };
  if (bits % 16) return go(std::true_type(), std::integral_constant<int, 1>());
  if (c.ctas(a.n, 4) < kManyCtas) return go(std::false_type(), std::integral_constant<int, 1>());
  return go(std::false_type(), std::integral_constant<int, 4>());
}

// Up to kClusterSort tokens: one launch sorts them and fills the rows that
// none of them names.
purlin_status launch_sort_fill(const SortArgs& a, bool fill, int elem, cudaStream_t s) {
  const EmbedArgs& e = a.e;
  // A fill of 64 MiB or more hides the sort: then few CTAs take many tokens
  // each, because clusters of 2 find places among the others' that clusters of
  // 8 do not (16384 tokens, 512 MiB: 122 against 135 us in all).  Else the sort
  // is what takes the time.
  const uint64_t bytes = fill ? e.rows * e.width * elem : 0;
  const ClusterShape c(e.n, bytes >= (uint64_t)64 << 20 ? kSortIpt : 2);
  // about two rounds of CTAs fill, each at least 16 KiB
  const uint64_t fills = (std::min<uint64_t>(2 * 152, bytes / 16384) + c.ctas - (fill ? 1 : 0)) / c.ctas * c.ctas;
  const uint64_t grid = (e.n ? c.ctas : 0) + (fill ? std::max<uint64_t>(fills, c.ctas) : 0);
  if (grid == 0) return PL_OK;
  const size_t sorted = e.n ? (size_t)8 * kClusterThreads * c.ipt + ((size_t)kClusterThreads / 32 * 2 << a.bits) : 0;
  const size_t smem = std::max<size_t>(sorted, fill ? kBitmapRows / 8 : 0);
  constexpr int kMost = 8 * kClusterThreads * kSortIpt + kClusterThreads / 32 * 2 * kSortBins;
  const uint64_t rows = (uint64_t)(uintptr_t)e.y | (uint64_t)(uintptr_t)e.base | (e.ldy | e.ldb | e.width) * elem;
  auto go = [&](auto fn) -> purlin_status {
    if (purlin_status st = op_smem((const void*)fn, smem, kMost)) return st;
    return op_launch_cluster(c.ctas, fn, grid, kClusterThreads, smem, s, a, c.ipt);
  };
  if (elem == 4) return rows % 16 ? go(sort_fill_kernel<uint32_t, true>) : go(sort_fill_kernel<uint32_t, false>);
  return rows % 16 ? go(sort_fill_kernel<uint16_t, true>) : go(sort_fill_kernel<uint16_t, false>);
}

}  // namespace

size_t embed_grad_bytes(uint64_t tokens, uint64_t rows, uint64_t width) { return (size_t)space_of(tokens, rows, width).end; }

purlin_status launch_embed(const EmbedArgs& a, int dtype, cudaStream_t s) {
  return dtype == PL_F32 ? embed_t<float>(a, s) : embed_t<bf16>(a, s);
}

purlin_status launch_embed_grad(const EmbedArgs& e, int x_dtype, int y_dtype, cudaStream_t s) {
  char* ws = (char*)e.workspace;
  const Space sp = space_of(e.n, e.rows, e.width);
  SortArgs a = {};
  a.e = e;
  digits_of(e.rows, &a.passes, &a.bits);
  a.out_key = (uint32_t*)(ws + sp.key[0]);
  a.out_idx = (uint32_t*)(ws + sp.idx[0]);
  // rows that no token names are left alone where they hold the base already
  const bool fill = e.base != e.y || e.ldb != e.ldy;
  purlin_status st;
  int out = 0;
  uint64_t fills = 0;
  if (e.n <= kClusterSort) {
    if ((st = launch_sort_fill(a, fill, y_dtype == PL_F32 ? 4 : 2, s))) return st;
  } else {
    fills = fill ? (e.rows + kFill - 1) / kFill : 0;
    const uint64_t chunk = sort_chunk(e.n), chunks = sort_chunks(e.n);
    a.counts = (uint32_t*)(ws + sp.counts);
    for (int p = 0; p < a.passes; ++p) {
      a.shift = p * a.bits;
      out = p & 1;
      a.out_key = (uint32_t*)(ws + sp.key[out]);
      a.out_idx = (uint32_t*)(ws + sp.idx[out]);
      const size_t smem = (size_t)(kSortThreads / 32 << a.bits) * sizeof(uint16_t);
      if ((st = op_launch(sort_count_kernel, chunks, kSortThreads, 0, s, a, (uint32_t)chunk))) return st;
      if ((st = op_launch(sort_place_kernel, chunks, kSortThreads, smem, s, a, (uint32_t)chunk, (int)(chunk / kSortThreads)))) return st;
      a.in_key = a.out_key;
      a.in_idx = a.out_idx;
    }
  }
  SumArgs m = {};
  m.e = e;
  m.key = (const uint32_t*)(ws + sp.key[out]);
  m.idx = (const uint32_t*)(ws + sp.idx[out]);
  m.part = (float*)(ws + sp.part);
  m.fills = fills;
  m.run = run_of(e.n, e.width);
  m.runs = (e.n + m.run - 1) / m.run;
  if (x_dtype == PL_F32) return y_dtype == PL_F32 ? sums<float, float>(m, s) : sums<float, bf16>(m, s);
  return y_dtype == PL_F32 ? sums<bf16, float>(m, s) : sums<bf16, bf16>(m, s);
}

}  // namespace pl
