// The routing of rows to experts: the sort of a router's choice, the dispatch of
// the tokens' rows and the gradient of their combination.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "internal.h"
#include "launch.h"

#pragma clang fp contract(off)

namespace svdq {
namespace {

using namespace dev;

// ---------------------------------------------------------------------------
// Stable counting sort of the slots by key (the expert, or `experts` for a
// dropped slot).  Slots are cut into chunks, one per workgroup, and a chunk into
// contiguous pieces, one per wave, so that rows are numbered in the order
//     key, chunk, wave, place in the wave's piece.
// sort_count_kernel counts the keys of each chunk; sort_place_kernel starts from
// the counts of all chunks, counts again by wave, and numbers each wave's slots 64
// at a time: the lanes with a slot's key come from one ballot per key bit, its
// rank is the number of them below its lane.  One chunk needs no counts, and one
// launch does it.  Chains of dependent steps bound it, not bytes: 128 slots 3.6 us,
// 98304 slots of 64 experts 3.4 and 9.7 us, 4M slots 58 us (0.87 TB/s).
// ---------------------------------------------------------------------------
constexpr int kSortWaves = kSortThreads / 64;

__device__ __forceinline__ int key_of(const int32_t* __restrict__ expert, int s, int experts) {
  const int e = expert[s];
  return (unsigned)e < (unsigned)experts ? e : experts;
}

// A wave's piece is taken 64 kKeys slots at a time, all of their keys loaded together.
constexpr int kKeys = 8;
static_assert(kKeys * kSortThreads == kSortChunk, "the usual chunk is one load of keys");

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t* __restrict__ expert, int b, int chunk,
                                                                  int experts, int32_t* __restrict__ counts) {
  __shared__ int s_count[SVDQ_MAX_EXPERTS + 1];
  const int tid = (int)threadIdx.x, keys = experts + 1;
  const int lo = (int)blockIdx.x * chunk, hi = min(lo + chunk, b);
  for (int e = tid; e < keys; e += kSortThreads) s_count[e] = 0;
  __syncthreads();
  for (int s0 = lo + tid; s0 < hi; s0 += kKeys * kSortThreads) {
    int key[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int s = s0 + i * kSortThreads;
      key[i] = s < hi ? key_of(expert, s, experts) : -1;
    }
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if (key[i] >= 0) atomicAdd(&s_count[key[i]], 1);
  }
  __syncthreads();
  for (int e = tid; e < keys; e += kSortThreads) counts[(size_t)blockIdx.x * keys + e] = s_count[e];
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t* __restrict__ expert, int b, int k,
                                                                  int chunk, int chunks, int experts, int bits,
                                                                  const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ row_index,
                                                                  int32_t* __restrict__ index) {
  extern __shared__ int s_next[];  // [wave][key]: the wave's count of a key, then its next row
  __shared__ int s_total[kSortWaves];
  const int tid = (int)threadIdx.x, lane = tid & 63, keys = experts + 1;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lo = (int)blockIdx.x * chunk, hi = min(lo + chunk, b);
  const int piece = chunk / kSortWaves;
  const int w0 = min(lo + wave * piece, hi), w1 = min(w0 + piece, hi);
  int key[kKeys];
  auto load_keys = [&](int s0) {  // slot s0 + 64 i + lane; -1 behind the piece
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int s = s0 + 64 * i + lane;
      key[i] = s < w1 ? key_of(expert, s, experts) : -1;
    }
  };
  load_keys(w0);
  for (int e = tid; e < keys * kSortWaves; e += kSortThreads) s_next[e] = 0;
  __syncthreads();
  int* next = s_next + wave * keys;
  for (int s0 = w0;;) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if (key[i] >= 0) atomicAdd(&next[key[i]], 1);
    s0 += 64 * kKeys;
    if (s0 >= w1) break;
    load_keys(s0);
  }
  __syncthreads();
  // rows before a key's first one: a scan over the keys, kSortThreads at a time
  int before = 0;
  for (int e0 = 0; e0 < keys; e0 += kSortThreads) {
    const int e = e0 + tid;
    int total = 0, earlier = 0;  // the key's slots in all chunks, and in those before this one
    if (e < keys) {
      if (counts) {
        for (int c0 = 0; c0 < chunks; c0 += 8) {
          int v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = c0 + i < chunks ? counts[(size_t)(c0 + i) * keys + e] : 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            total += v[i];
            earlier += c0 + i < (int)blockIdx.x ? v[i] : 0;
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) total += s_next[w * keys + e];
      }
    }
    int up = total;  // inclusive scan over the wave
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(up, d);
      up += lane >= d ? v : 0;
    }
    if (lane == 63) s_total[wave] = up;
    __syncthreads();
    int start = before + up - total, all = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      start += w < wave ? s_total[w] : 0;
      all += s_total[w];
    }
    before += all;
    if (e < keys) {
      if (blockIdx.x == 0) offsets[e] = start;  // of key `experts`: the end of the experts' rows
      int row = start + earlier;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const int v = s_next[w * keys + e];
        s_next[w * keys + e] = row;
        row += v;
      }
    }
    __syncthreads();
  }
  if (piece > 64 * kKeys) load_keys(w0);  // (otherwise they are there)
  for (int s0 = w0; s0 < w1;) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      if (s0 + 64 * i >= w1) break;
      const int s = s0 + 64 * i + lane;
      const bool live = key[i] >= 0;
      uint64_t same = __ballot(live);
      for (int d = 0; d < bits; ++d) {
        const uint64_t set = __ballot(key[i] >> d & 1);
        same &= key[i] >> d & 1 ? set : ~set;
      }
      const int rank = __popcll(same & ((1ULL << lane) - 1));
      if (live) {
        const int row = next[key[i]] + rank;
        // the wave's lanes have read their rows before the last lane of each key
        // moves it on: LDS accesses of a wave complete in order
        if (rank + 1 == __popcll(same)) next[key[i]] = row + 1;
        index[s] = key[i] < experts ? row : -1 - row;
        row_index[row] = s / k;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // (the next 64 slots see the moved rows)
    }
    s0 += 64 * kKeys;
    if (s0 < w1) load_keys(s0);
  }
}

// ---------------------------------------------------------------------------
// Dispatch, and the gradient of the combination:
//     drows[index[t,q]] = weight[t,q] x[t],   dweight[t,q] = x[t] . rows[index[t,q]]
// nw waves take a token, each every nw-th chunk of 64 W columns (16 bytes a lane),
// its rows eight at a time, all loads of a chunk together.  x is read once for
// eight rows; a row's elements are read before they are written (drows may be
// rows).  Sums: a lane's own products in order, then the lanes by halves, then
// the waves in order, all in fp32.  Memory bounds both: 4096 x 6 rows of 2048 in bf16,
// dispatch 20.6 us, 5.7 TB/s, gradient 45.5 us, 4.8 TB/s.
// ---------------------------------------------------------------------------
constexpr int kRouteBatch = 8;

typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));

template <bool BF16>
struct RowVector {
  static constexpr int W = BF16 ? 8 : 4;  // columns of 16 bytes
  typedef typename std::conditional<BF16, uint16_t, uint32_t>::type Element;
  typedef typename std::conditional<BF16, u32x4_at2, u32x4_at4>::type Loose;  // gfx950 takes any element's address
  template <bool ONCE>  // read this once only
  static __device__ __forceinline__ u32x4 get(const void* base, long long row, int n, int j) {
    const Element* p = reinterpret_cast<const Element*>(base) + (size_t)row * n + j;
    if (j + W <= n) {
      if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const Loose*>(p));
      return *reinterpret_cast<const Loose*>(p);
    }
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (j + e < n) {
        if constexpr (BF16)
          v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
        else
          v[e] = p[e];
      }
    return v;
  }
  static __device__ __forceinline__ void put(void* base, long long row, int n, int j, const u32x4& v) {
    Element* p = reinterpret_cast<Element*>(base) + (size_t)row * n + j;
    if (j + W <= n) {
      // past the L2: rows come in at their place once, and evicting what is read for them
      // costs more (4096 x 6 rows of 2048, the same every call: gradient bf16 53.6 -> 39.4 us, dispatch fp32
      // 51.4 -> 41.1)
      __builtin_nontemporal_store(v, reinterpret_cast<Loose*>(p));
      return;
    }
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (j + e < n) p[e] = BF16 ? (Element)(v[(e >> 1) & 3] >> (16 * (e & 1))) : (Element)v[e & 3];
  }
  static __device__ __forceinline__ float value(const u32x4& v, int e) {
    if constexpr (BF16) return e & 1 ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]);
    return __uint_as_float(v[e]);
  }
};

template <bool BF16, bool DOT, bool WRITE>
__global__ __launch_bounds__(256) void scatter_rows_kernel(const void* __restrict__ x, int t_count, int n,
                                                           const int32_t* __restrict__ index,
                                                           const float* __restrict__ weight, int k, const void* rows,
                                                           int R, void* drows, float* __restrict__ dweight, int nw) {
  typedef RowVector<BF16> V;
  constexpr int W = V::W;
  __shared__ float s_dot[4][kRouteBatch];
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int part = wave % nw;
  const long long t = (long long)blockIdx.x * (4 / nw) + wave / nw;
  const bool live = t < t_count;
  for (int q0 = 0; q0 < k; q0 += kRouteBatch) {
    int row[kRouteBatch];  // the slot's row: >= 0 used, -1 - r to be cleared, below -R not there
    float w[kRouteBatch], dot[kRouteBatch];
#pragma unroll
    for (int q = 0; q < kRouteBatch; ++q) {
      row[q] = INT32_MIN;
      w[q] = 1.0f;
      dot[q] = 0.0f;
      if (live && q0 + q < k) {
        const int i = index[t * k + q0 + q];
        if (i < R && i >= -R) row[q] = i;
        if (weight) w[q] = weight[t * k + q0 + q];
      }
    }
    if (live)
      for (int j0 = part * 64 * W; j0 < n; j0 += nw * 64 * W) {
        const int j = j0 + lane * W;
        if (j >= n) continue;
        const u32x4 xv = V::template get<false>(x, t, n, j);
        u32x4 rv[kRouteBatch];
        if constexpr (DOT) {
#pragma unroll
          for (int q = 0; q < kRouteBatch; ++q) {
            rv[q] = u32x4{0u, 0u, 0u, 0u};
            if (row[q] >= 0) rv[q] = V::template get<true>(rows, row[q], n, j);
          }
#pragma unroll
          for (int q = 0; q < kRouteBatch; ++q)
            if (row[q] >= 0)  // (a slot without a row adds nothing, whatever x holds)
#pragma unroll
              for (int e = 0; e < W; ++e) dot[q] = __builtin_fmaf(V::value(xv, e), V::value(rv[q], e), dot[q]);
        }
        if constexpr (WRITE) {
#pragma unroll
          for (int q = 0; q < kRouteBatch; ++q) {
            if (row[q] == INT32_MIN) continue;
            u32x4 o = {0u, 0u, 0u, 0u};
            if (row[q] >= 0) {
              if (weight) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if constexpr (BF16)
                    o[e] = pack_bf16x2(w[q] * bf16_lo(xv[e]), w[q] * bf16_hi(xv[e]));
                  else
                    o[e] = __float_as_uint(w[q] * __uint_as_float(xv[e]));
                }
              } else {
                o = xv;
              }
            }
            V::put(drows, row[q] >= 0 ? row[q] : -1 - row[q], n, j, o);
          }
        }
      }
    if constexpr (DOT) {
#pragma unroll
      for (int q = 0; q < kRouteBatch; ++q) {
#pragma unroll
        for (int d = 32; d > 0; d /= 2) dot[q] += __shfl_xor(dot[q], d);
        if (lane == 0) s_dot[wave][q] = dot[q];
      }
      __syncthreads();
      if (live && part == 0 && lane < kRouteBatch && q0 + lane < k) {
        float sum = s_dot[wave][lane];
        for (int p = 1; p < nw; ++p) sum += s_dot[wave + p][lane];
        dweight[t * k + q0 + lane] = sum;
      }
      __syncthreads();
    }
  }
}

}  // namespace

int launch_sort_rows(const int32_t* expert, int b, int k, int experts, int32_t* offsets, int32_t* row_index,
                     int32_t* index, void* ws, void* stream) {
  const SortPlan p = sort_plan(b);
  const int32_t* counts = nullptr;
  if (p.chunks > 1) {
    int32_t* c = reinterpret_cast<int32_t*>(ws);
    const int status = launch_checked(sort_count_kernel, p.chunks, kSortThreads, (hipStream_t)stream, expert, b,
                                      p.chunk, experts, c);
    if (status != 0) return status;
    counts = c;
  }
  const int ok = scratch_free(reinterpret_cast<const void*>(sort_place_kernel));
  if (ok != 0) return ok;
  int bits = 0;
  while (experts >> bits) ++bits;  // keys 0 .. experts
  hipLaunchKernelGGL(sort_place_kernel, dim3((unsigned)p.chunks), dim3(kSortThreads),
                     (size_t)kSortWaves * (experts + 1) * 4, (hipStream_t)stream, expert, b, k, p.chunk, p.chunks,
                     experts, bits, counts, offsets, row_index, index);
  return (int)hipGetLastError();
}

int launch_scatter_rows(const void* x, int t, int n, int dtype, const int32_t* index, const float* weight, int k,
                        const void* rows, int R, void* drows, float* dweight, void* stream) {
  const bool bf = dtype == SVDQ_OUT_BF16;
  const int units = (n + (bf ? 512 : 256) - 1) / (bf ? 512 : 256);  // a wave's chunks in a row
  // Waves of a token: a whole chunk each, or a part where tokens alone do not fill the
  // chip (4096 tokens x 6 rows of 2048, other rows every call: gradient bf16 57 us with
  // one, 60 with two, 50 with four, fp32 105, 108, 91; 4096 x 2 rows of 1001 bf16:
  // dispatch 7.9 with one, 8.8 with two; 300 x 6 rows of 4608 bf16: 18.9, 12.5, 9.8).
  const int whole = n / (bf ? 512 : 256);
  int nw = 1;
  while (nw < 4 && (2 * nw <= whole || (2 * nw <= units && (long long)t * nw < 8 * kMaxCUs))) nw *= 2;
  const int grid = (int)(((long long)t * nw + 3) / 4);
  auto go = [&](auto kernel) {
    return launch_checked(kernel, grid, 256, (hipStream_t)stream, x, t, n, index, weight, k, rows, R, drows, dweight,
                          nw);
  };
  if (dweight && drows) return bf ? go(scatter_rows_kernel<true, true, true>) : go(scatter_rows_kernel<false, true, true>);
  if (dweight) return bf ? go(scatter_rows_kernel<true, true, false>) : go(scatter_rows_kernel<false, true, false>);
  return bf ? go(scatter_rows_kernel<true, false, true>) : go(scatter_rows_kernel<false, false, true>);
}

}  // namespace svdq
