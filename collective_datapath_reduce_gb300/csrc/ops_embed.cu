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

constexpr int kRowThreads = 256;

template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads) embed_kernel(const __grid_constant__ EmbedArgs a, int tpt) {
  op_wait();
  const uint64_t t = (uint64_t)blockIdx.x * (kRowThreads / tpt) + threadIdx.x / tpt;
  if (t >= a.n) return;
  const uint64_t row = row_of(a, t), nv = a.width / N;
  const T* x = (const T*)a.x + row * a.ldx;
  T* y = (T*)a.y + t * a.ldy;
  for (uint64_t v = threadIdx.x % tpt; v < nv; v += tpt) {
    Pack<T, N> r = zero_pack<T, N>();
    if (row < a.rows) {
      r = ld_pack<T, N>(x + v * N);
#pragma unroll
      for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(to_f32(r.v[i]) * a.scale);
    }
    st_pack<T, N>(y + v * N, r);
  }
}

// ------------------------------------------------------- sort of the tokens

// One digit of the sort: (key, index) pairs, or the tokens themselves when
// in_key is null.  Keys are rows of the table; rows = outside, sorted last.
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
  op_wait();
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
  sum_chunks(a.counts, gridDim.x, blockIdx.x, bins, base, before);
  rank_chunk(digit, local, ipt, bins, cnt, [](int, uint32_t) {});
  uint32_t total;
  const uint32_t at = block_exclusive(threadIdx.x < bins ? base[threadIdx.x] : 0, tmp, &total);
  if (threadIdx.x < bins) base[threadIdx.x] = at + before[threadIdx.x];
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

// All digits by one CTA, between two arrays in shared memory.
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(const __grid_constant__ SortArgs a, int ipt) {
  op_wait();
  extern __shared__ uint32_t pair[];  // keys, indexes, then the warps' counters
  __shared__ uint32_t base[kSortBins], tmp[33];
  const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t n = (uint32_t)a.e.n;
  uint32_t *keys = pair, *idx = pair + n;
  uint16_t* cnt = (uint16_t*)(pair + 2 * n);
  for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) {
    keys[i] = (uint32_t)row_of(a.e, i);
    idx[i] = i;
  }
  __syncthreads();
  for (int p = 0; p < a.passes; ++p) {
    int digit[kSortIpt];
    uint32_t local[kSortIpt], key[kSortIpt], id[kSortIpt];
#pragma unroll
    for (int q = 0; q < kSortIpt; ++q)
      if (q < ipt) {
        const uint32_t i = (uint32_t)(warp * ipt + q) * 32 + lane;
        key[q] = i < n ? keys[i] : 0;
        id[q] = i < n ? idx[i] : 0;
        digit[q] = i < n ? (int)(key[q] >> (p * a.bits) & (bins - 1)) : -1;
      }
    rank_chunk(digit, local, ipt, bins, cnt, [&](int b, uint32_t c) { base[b] = c; });
    uint32_t carry = 0;
    for (int b0 = 0; b0 < bins; b0 += blockDim.x) {
      const int b = b0 + threadIdx.x;
      uint32_t total;
      const uint32_t at = carry + block_exclusive(b < bins ? base[b] : 0, tmp, &total);
      if (b < bins) base[b] = at;
      carry += total;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSortIpt; ++q)
      if (q < ipt && digit[q] >= 0) {
        const uint32_t to = base[digit[q]] + cnt[warp * bins + digit[q]] + local[q];
        keys[to] = key[q];
        idx[to] = id[q];
      }
    __syncthreads();
  }
  for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) {
    a.out_key[i] = keys[i];
    a.out_idx[i] = idx[i];
  }
}

// ------------------------------------------------------- sums of sorted rows

constexpr int kRun = 32;          // sorted places of one run
constexpr int kSumThreads = 128;  // one vector of the row each
constexpr int kFill = 32;         // table rows of one CTA that fills untouched rows

struct SumArgs {
  EmbedArgs e;
  const uint32_t *key, *idx;
  float* part;      // [run][head, tail][width]
  uint64_t runs;
  uint32_t tiles;   // column tiles of a row
};

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
  st_pack<TY, N>((TY*)a.e.y + row * a.e.ldy + c, o);
}

// Rows that no token names: zero, or the base's.
template <typename TY, int N>
__device__ void fill_rows(const SumArgs& a, uint64_t block) {
  __shared__ uint32_t touched;
  const uint64_t r0 = block * kFill;
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
  const uint64_t nv = a.e.width / N;
  for (int k = 0; k < kFill; ++k) {
    if (touched >> k & 1u) continue;
    for (uint64_t v = threadIdx.x; v < nv; v += kSumThreads) {
      Pack<TY, N> o = zero_pack<TY, N>();
      if (a.e.base) o = ld_pack<TY, N>((const TY*)a.e.base + (r0 + k) * a.e.ldb + v * N);
      st_pack<TY, N>((TY*)a.e.y + (r0 + k) * a.e.ldy + v * N, o);
    }
  }
}

template <typename TX, typename TY, int N>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const __grid_constant__ SumArgs a) {
  op_wait();
  if (blockIdx.x >= a.runs * a.tiles) {
    fill_rows<TY, N>(a, blockIdx.x - a.runs * a.tiles);
    return;
  }
  __shared__ uint32_t key[kRun + 2], idx[kRun];  // key[1 + i]: place i of the run; its neighbours at the ends
  const uint64_t run = blockIdx.x / a.tiles, p0 = run * kRun;
  const int n = (int)(a.e.n - p0 < kRun ? a.e.n - p0 : kRun);
  const uint32_t none = 0xFFFFFFFFu;
  for (int i = threadIdx.x; i < n + 2; i += kSumThreads) {
    const uint64_t p = p0 + i;  // place p - 1
    key[i] = p >= 1 && p <= a.e.n ? a.key[p - 1] : none;
    if (i >= 1 && i <= n) idx[i - 1] = a.idx[p - 1];
  }
  __syncthreads();
  const uint64_t c = ((uint64_t)(blockIdx.x % a.tiles) * kSumThreads + threadIdx.x) * N;
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
      if (q + u < n && key[q + u + 1] < rows) x[u] = ld_pack<TX, N>((const TX*)a.e.x + (uint64_t)idx[q + u] * a.e.ldx + c);
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
        float* part = a.part + (run * 2 + (head ? 0 : 1)) * a.e.width + c;
        Pack<float, N> o;
#pragma unroll
        for (int i = 0; i < N; ++i) o.v[i] = acc[i];
        st_pack<float, N>(part, o);
      }
      head = false;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
    }
  }
}

// The token whose first place lies in this run and that goes on in the next:
// its tail here, then the heads of the runs that it reaches.
template <typename TX, typename TY, int N>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const __grid_constant__ SumArgs a) {
  op_wait();
  const uint64_t run = blockIdx.x / a.tiles, p0 = run * kRun, p1 = p0 + kRun;
  if (p1 >= a.e.n) return;
  const uint32_t k = a.key[p1 - 1];
  if (k >= (uint32_t)a.e.rows || a.key[p1] != k) return;
  if (p0 > 0 && a.key[p0 - 1] == k) return;  // begun earlier
  const uint64_t c = ((uint64_t)(blockIdx.x % a.tiles) * kSumThreads + threadIdx.x) * N;
  if (c >= a.e.width) return;
  float acc[N];
  {
    const Pack<float, N> x = *reinterpret_cast<const Pack<float, N>*>(a.part + (run * 2 + 1) * a.e.width + c);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = x.v[i];
  }
  for (uint64_t r = run + 1; r < a.runs && a.key[r * kRun] == k; ++r) {
    const Pack<float, N> x = *reinterpret_cast<const Pack<float, N>*>(a.part + r * 2 * a.e.width + c);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += x.v[i];
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

struct Space {
  uint64_t key[2], idx[2], counts, part, end;
};

uint64_t up(uint64_t x) { return (x + 255) & ~(uint64_t)255; }

Space space_of(uint64_t n, uint64_t rows, uint64_t width) {
  int passes, bits;
  digits_of(rows, &passes, &bits);
  const bool small = n <= kSortSmall;
  const uint64_t runs = (n + kRun - 1) / kRun;
  Space s;
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t p = at;
    at += up(bytes);
    return p;
  };
  s.key[0] = take(n * 4);
  s.idx[0] = take(n * 4);
  s.key[1] = take(small ? 0 : n * 4);
  s.idx[1] = take(small ? 0 : n * 4);
  s.counts = take(small ? 0 : sort_chunks(n) * ((uint64_t)4 << bits));
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
    a.tiles = (uint32_t)((a.e.width / N + kSumThreads - 1) / kSumThreads);
    // rows that no token names are left alone when they already hold the base
    const bool fill = a.e.base != a.e.y || a.e.ldb != a.e.ldy;
    const uint64_t fills = fill ? (a.e.rows + kFill - 1) / kFill : 0;
    if (purlin_status st = op_launch(sum_kernel<TX, TY, N>, a.runs * a.tiles + fills, kSumThreads, 0, s, a)) return st;
    if (a.runs < 2) return PL_OK;
    return op_launch(join_kernel<TX, TY, N>, a.runs * a.tiles, kSumThreads, 0, s, a);
  };
  if constexpr (kMost >= 8)
    if (fits(8)) return go(std::integral_constant<int, 8>());
  if (fits(4)) return go(std::integral_constant<int, 4>());
  if (fits(2)) return go(std::integral_constant<int, 2>());
  return go(std::integral_constant<int, 1>());
}

int threads_per_token(uint64_t nv) {
  int t = 32;
  while (t < kRowThreads && (uint64_t)t < nv) t *= 2;
  return t;
}

template <typename T>
purlin_status embed_t(const EmbedArgs& a, cudaStream_t s) {
  const uint64_t bits = (uint64_t)(uintptr_t)a.x | (uint64_t)(uintptr_t)a.y | (a.ldx | a.ldy | a.width) * sizeof(T);
  return with_vec<T>(vec_bytes(bits), [&](auto n) {
    constexpr int N = decltype(n)::value;
    const int tpt = threads_per_token(a.width / N), per = kRowThreads / tpt;
    return op_launch(embed_kernel<T, N>, (a.n + per - 1) / per, kRowThreads, 0, s, a, tpt);
  });
}

purlin_status raise_smem(const void* fn, int bytes) {
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess) return PL_OK;
  (void)cudaGetLastError();
  return PL_ERR_CUDA;
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
  int out = 0;
  purlin_status st;
  if (e.n == 0) {
    out = 0;
  } else if (e.n <= kSortSmall) {
    a.out_key = (uint32_t*)(ws + sp.key[0]);
    a.out_idx = (uint32_t*)(ws + sp.idx[0]);
    const int ipt = (int)((e.n + kSortThreads - 1) / kSortThreads);
    const uint64_t wide = std::max<uint64_t>(e.n, (uint64_t)1 << a.bits);
    const int threads = (int)std::min<uint64_t>(kSortThreads, (wide + 31) / 32 * 32);
    const size_t smem = 8 * e.n + (size_t)(threads / 32 << a.bits) * sizeof(uint16_t);
    constexpr int kMost = 8 * kSortSmall + kSortWarps * kSortBins * 2;
    if ((st = raise_smem((const void*)sort_small_kernel, kMost))) return st;
    if ((st = op_launch(sort_small_kernel, 1, threads, smem, s, a, ipt))) return st;
  } else {
    if ((st = raise_smem((const void*)sort_place_kernel, kSortWarps * kSortBins * 2))) return st;
    const uint64_t chunk = sort_chunk(e.n), chunks = sort_chunks(e.n);
    a.counts = (uint32_t*)(ws + sp.counts);
    for (int p = 0; p < a.passes; ++p) {
      a.shift = p * a.bits;
      out = p & 1;
      a.out_key = (uint32_t*)(ws + sp.key[out]);
      a.out_idx = (uint32_t*)(ws + sp.idx[out]);
      if ((st = op_launch(sort_count_kernel, chunks, kSortThreads, 0, s, a, (uint32_t)chunk))) return st;
      const size_t smem = (size_t)(kSortWarps << a.bits) * sizeof(uint16_t);
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
  m.runs = (e.n + kRun - 1) / kRun;
  if (x_dtype == PL_F32) return y_dtype == PL_F32 ? sums<float, float>(m, s) : sums<float, bf16>(m, s);
  return y_dtype == PL_F32 ? sums<bf16, float>(m, s) : sums<bf16, bf16>(m, s);
}

}  // namespace pl
