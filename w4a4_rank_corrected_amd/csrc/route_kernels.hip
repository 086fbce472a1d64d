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
// Dispatch, and the weights' gradient of the combination, driven by the tokens:
//     rows[index[t,q]] = weight[t,q] x[t],   dweight[t,q] = x[t] . rows[index[t,q]]
// nw waves take a token, each every nw-th chunk of 64 W columns (16 bytes a lane),
// its rows eight at a time, all loads of a chunk together; x is read once for eight
// rows.  Sums: a lane's own products in order, then the lanes by halves, then the
// waves in order, all in fp32.  Memory bounds it: 4096 x 6 rows of 2048 in bf16,
// dispatch 20.6 us, 5.7 TB/s.
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

// The tokens of workgroup `block` of kWaves waves.  WRITE: dispatch; otherwise the weights' gradient.
template <bool BF16, bool WRITE, int kWaves>
__device__ __forceinline__ void token_part(const void* __restrict__ x, int t_count, int n,
                                           const int32_t* __restrict__ index, const float* __restrict__ weight, int k,
                                           const void* rows, int R, void* out, float* __restrict__ dweight, int nw,
                                           long long block) {
  typedef RowVector<BF16> V;
  constexpr int W = V::W;
  constexpr bool DOT = !WRITE;
  __shared__ float s_dot[kWaves][kRouteBatch];
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int part = wave % nw;
  const long long t = block * (kWaves / nw) + wave / nw;
  const bool live = t < t_count;
  for (int q0 = 0; q0 < k; q0 += kRouteBatch) {
    int row[kRouteBatch];  // the slot's row: >= 0 used, -1 - r to be cleared (dispatch), below -R not there
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
            V::put(out, row[q] >= 0 ? row[q] : -1 - row[q], n, j, o);
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

template <bool BF16, bool WRITE>
__global__ __launch_bounds__(256) void scatter_rows_kernel(const void* __restrict__ x, int t_count, int n,
                                                           const int32_t* __restrict__ index,
                                                           const float* __restrict__ weight, int k, const void* rows,
                                                           int R, void* drows, float* __restrict__ dweight, int nw) {
  token_part<BF16, WRITE, 4>(x, t_count, n, index, weight, k, rows, R, drows, dweight, nw, blockIdx.x);
}

// ---------------------------------------------------------------------------
// The rows' gradient of the combination, driven by the rows:
//     drows[r] = sum over the slots (t,q) that name r, in their order, of weight[t,q] dy[t]
// so that a row that no slot names becomes zero, one that several name gets their sum
// in a fixed order, and a slot that names none touches nothing.  A workgroup takes
// `per` neighbouring rows.  It reads the whole index (all loads of a round together)
// and keeps in LDS the slots that name its rows: one in the row's own entry, further
// ones in a list behind it, which is put into the slots' order; then its waves take
// four chunks of 64 W columns of a row at a time.  Lists longer than kListMost or
// beyond the workgroup's kLinks links are given up: such a row's slots are found by
// reading the index again for each of its chunks.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 512, kGradWaves = kGradThreads / 64;
constexpr int kLinks = 2048, kListMost = 64;
constexpr uint32_t kNone = ~0u, kEnd = ~0u - 1, kMany = ~0u - 2;  // Namer::next: no slot, the list's end, given up
struct Namer {
  uint32_t slot, next;
};

template <bool BF16>
__device__ __forceinline__ void rows_part(const void* __restrict__ dy, int t_count, int n,
                                          const int32_t* __restrict__ index, const float* __restrict__ weight, int k,
                                          int R, void* drows, int per, int block, Namer* named) {
  typedef RowVector<BF16> V;
  constexpr int W = V::W;
  Namer* links = named + per;
  __shared__ uint32_t s_links;
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = block * per, count = min(per, R - r0);
  const size_t total = (size_t)t_count * k;  // at most 2^32 slots: 0 .. 2^32 - 1
  for (int i = tid; i < count; i += kGradThreads) named[i].next = kNone;
  if (tid == 0) s_links = 0;
  __syncthreads();
  auto name = [&](uint32_t row, uint32_t slot) {
    Namer& at = named[row];
    if (atomicCAS(&at.next, kNone, kEnd) == kNone) {
      at.slot = slot;
      return;
    }
    const uint32_t e = atomicAdd(&s_links, 1u);
    if (e < (uint32_t)kLinks) {
      links[e].slot = slot;
      links[e].next = atomicExch(&at.next, e);
    } else {
      atomicExch(&at.next, kMany);  // (links put before it later end in it)
    }
  };
  constexpr int B = 4;  // vectors of four slots a thread has under way
  for (size_t s0 = 0; s0 < total; s0 += 4 * B * kGradThreads) {
    u32x4 v[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const size_t s = s0 + 4 * ((size_t)i * kGradThreads + tid);
      v[i] = u32x4{~0u, ~0u, ~0u, ~0u};
      if (s + 4 <= total) {
        v[i] = *reinterpret_cast<const u32x4_at4*>(index + s);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (s + e < total) v[i][e] = (uint32_t)index[s + e];
      }
    }
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // (what lies outside the R rows lies outside these; a filled-up place is -1)
        const uint32_t row = v[i][e] - (uint32_t)r0;
        if (row < (uint32_t)count) name(row, (uint32_t)(s0 + 4 * ((size_t)i * kGradThreads + tid) + e));
      }
  }
  __syncthreads();
  // lists into the slots' order: the least of the rest to each place
  for (int i = tid; i < count; i += kGradThreads) {
    uint32_t first = named[i].next;
    if (first >= kMany) continue;
    int length = 1;
    for (uint32_t e = first; e < kMany && length <= kListMost; e = links[e].next) {
      ++length;
      if (links[e].next == kMany) length = kListMost + 1;
    }
    if (length > kListMost) {
      named[i].next = kMany;
      continue;
    }
    for (Namer* p = &named[i]; p->next != kEnd; p = &links[p->next]) {
      Namer* least = p;
      for (uint32_t e = p->next; e != kEnd; e = links[e].next)
        if (links[e].slot < least->slot) least = &links[e];
      const uint32_t t = p->slot;
      p->slot = least->slot;
      least->slot = t;
    }
  }
  __syncthreads();
  constexpr int C = 4;  // chunks of a row a wave takes at a time
  const int groups = (n + C * 64 * W - 1) / (C * 64 * W);
  for (long long u = wave; u < (long long)count * groups; u += kGradWaves) {
    const int i = (int)(u / groups), j0 = (int)(u - (long long)i * groups) * C * 64 * W + lane * W;
    const uint32_t slot = __builtin_amdgcn_readfirstlane(named[i].slot);
    const uint32_t next = __builtin_amdgcn_readfirstlane(named[i].next);
    const long long row = r0 + i;
    if (next == kNone || next == kEnd) {
      u32x4 o[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        o[c] = u32x4{0u, 0u, 0u, 0u};
        const int j = j0 + c * 64 * W;
        if (next == kEnd && j < n) o[c] = V::template get<false>(dy, slot / (uint32_t)k, n, j);
      }
      if (weight && next == kEnd) {
        const float w = weight[slot];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (BF16)
              o[c][e] = pack_bf16x2(w * bf16_lo(o[c][e]), w * bf16_hi(o[c][e]));
            else
              o[c][e] = __float_as_uint(w * __uint_as_float(o[c][e]));
          }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = j0 + c * 64 * W;
        if (j < n) V::put(drows, row, n, j, o[c]);
      }
      continue;
    }
#pragma unroll 1
    for (int c = 0; c < C; ++c) {
      const int j = j0 + c * 64 * W;
      float sum[W];
      bool any = false;
      auto add = [&](uint32_t s) {
        const u32x4 v = j < n ? V::template get<false>(dy, s / (uint32_t)k, n, j) : u32x4{0u, 0u, 0u, 0u};
        const float w = weight ? weight[s] : 1.0f;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float p = w * V::value(v, e);
          sum[e] = any ? sum[e] + p : p;
        }
        any = true;
      };
      if (next != kMany) {
        add(slot);
        for (uint32_t e = next; e != kEnd; e = __builtin_amdgcn_readfirstlane(links[e].next))
          add(__builtin_amdgcn_readfirstlane(links[e].slot));
      } else {
        for (size_t s0 = 0; s0 < total; s0 += 64) {
          uint64_t hits = __ballot(s0 + lane < total && index[s0 + lane] == (int32_t)row);
          for (; hits; hits &= hits - 1) add((uint32_t)(s0 + __builtin_ctzll(hits)));
        }
      }
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = BF16 ? pack_bf16x2(sum[2 * e % W], sum[(2 * e + 1) % W]) : __float_as_uint(sum[e]);
      if (j < n) V::put(drows, row, n, j, o);
    }
  }
}

// The gradient in one launch: the first row_blocks workgroups take rows, the others tokens'
// weights (none where dweight is NULL).  4096 x 6 rows of 2048 in bf16: 54.7 us, where
// the rows alone take 32.9 (dy read once for each row that it reaches, by the caches) and
// the weights 21.7; tokens' rows written by the tokens' waves, with the rows of no or
// several slots in a launch before them, 54.8.
template <bool BF16>
__global__ __launch_bounds__(kGradThreads) void combine_grad_kernel(const void* __restrict__ dy, int t_count, int n,
                                                                    const int32_t* __restrict__ index,
                                                                    const float* __restrict__ weight, int k,
                                                                    const void* rows, int R, void* drows,
                                                                    float* __restrict__ dweight, int nw, int per,
                                                                    int row_blocks) {
  extern __shared__ __align__(16) Namer grad_lds[];
  if ((int)blockIdx.x < row_blocks)
    rows_part<BF16>(dy, t_count, n, index, weight, k, R, drows, per, (int)blockIdx.x, grad_lds);
  else
    token_part<BF16, false, kGradWaves>(dy, t_count, n, index, weight, k, rows, R, nullptr, dweight, nw,
                                        (long long)blockIdx.x - row_blocks);
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

namespace {

// Waves of a token: a whole chunk each, or a part where tokens alone do not fill the
// chip (4096 tokens x 6 rows of 2048, other rows every call: gradient bf16 57 us with
// one, 60 with two, 50 with four, fp32 105, 108, 91; 4096 x 2 rows of 1001 bf16:
// dispatch 7.9 with one, 8.8 with two; 300 x 6 rows of 4608 bf16: 18.9, 12.5, 9.8).
int token_waves(int t, int n, bool bf) {
  const int chunk = bf ? 512 : 256, whole = n / chunk, units = (n + chunk - 1) / chunk;
  int nw = 1;
  while (nw < 4 && (2 * nw <= whole || (2 * nw <= units && (long long)t * nw < 8 * kMaxCUs))) nw *= 2;
  return nw;
}

}  // namespace

int launch_scatter_rows(const void* x, int t, int n, int dtype, const int32_t* index, const float* weight, int k,
                        const void* rows, int R, void* drows, float* dweight, void* stream) {
  const bool bf = dtype == SVDQ_OUT_BF16;
  const int nw = token_waves(t, n, bf);
  auto go = [&](auto kernel) {
    return launch_checked(kernel, ((long long)t * nw + 3) / 4, 256, (hipStream_t)stream, x, t, n, index, weight, k, rows, R,
                          drows, dweight, nw);
  };
  if (dweight) return bf ? go(scatter_rows_kernel<true, false>) : go(scatter_rows_kernel<false, false>);
  return bf ? go(scatter_rows_kernel<true, true>) : go(scatter_rows_kernel<false, true>);
}

int launch_combine_grad(const void* dy, int t, int n, int dtype, const int32_t* index, const float* weight, int k,
                        const void* rows, int R, void* drows, float* dweight, void* stream) {
  const bool bf = dtype == SVDQ_OUT_BF16;
  const int nw = token_waves(t, n, bf);
  if (!drows || R == 0) return launch_scatter_rows(dy, t, n, dtype, index, weight, k, rows, R, nullptr, dweight, stream);
  long long tokens = dweight ? ((long long)t * nw + kGradWaves - 1) / kGradWaves : 0;
  if (dweight && drows == rows) {  // all rows are read before any is written
    const int status = launch_scatter_rows(dy, t, n, dtype, index, weight, k, rows, R, nullptr, dweight, stream);
    if (status != 0) return status;
    tokens = 0;
  }
  const GradPlan p = grad_plan(R);
  auto go = [&](auto kernel) {
    if (!launch_fits(p.blocks + tokens, kGradThreads)) return (int)hipErrorInvalidConfiguration;
    const int ok = scratch_free(reinterpret_cast<const void*>(kernel));
    if (ok != 0) return ok;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(p.blocks + tokens)), dim3(kGradThreads),
                       (size_t)(p.per + kLinks) * sizeof(Namer), (hipStream_t)stream, dy, t, n, index, weight, k, rows, R,
                       drows, dweight, nw, p.per, p.blocks);
    return (int)hipGetLastError();
  };
  return bf ? go(combine_grad_kernel<true>) : go(combine_grad_kernel<false>);
}

}  // namespace svdq
