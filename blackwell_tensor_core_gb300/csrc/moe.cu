// The routed rows' way to their experts and back: a stable counting sort of
// the (token, expert) pairs, the dispatch of token rows into expert order,
// the weighted combine into token order, and the gradient of each.
//
// With T tokens, k experts a token and pairs p = t * k + j:
//   sort      order[r] = the pair at sorted row r, position[p] = its inverse,
//             offsets[e] = the first row of expert e (offsets[E] = n, the rows
//             that have an expert; pairs without one are sorted behind them)
//   dispatch  rows[position[p]] = x[t], zero where position[p] >= n
//   combine   y[t] = sum_j w[p] rows[position[p]] over position[p] < n
// and, d for the gradient of a scalar loss,
//   dispatch' dx[t] = sum_j d_rows[position[p]]   (combine without weights)
//   combine'  d_rows[position[p]] = w[p] dy[t],  dw[p] = <dy[t], rows[position[p]]>
// A pair without an expert takes part in none of the sums, whatever its row
// holds (NaN included), and its d_rows and dw are zero.
//
// Every kernel walks the pairs in token order, so that a token's row is read
// once for all its k copies, and adds in the order j = 0 .. k-1 in FP32:
// there are no atomics and results do not depend on the launch.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <mutex>

#include "../../include/bwgemm.h"
#include "launch.h"
#include "params.h"
#include "ptx.cuh"
#include "runtime.h"

namespace bwg {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxColumns = 1 << 30;  // the vectors of a row's blocks are counted in an int

// The int at `p` (this CTA's shared memory) in the shared memory of CTA `rank`.
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  return static_cast<int>(ld_shared_cluster_u32(mapa_shared(smem_u32(p), rank)));
}

// A position outside [0, pairs) is not followed; it is reported through the
// device error word, with the kind of a broken offsets array.
__device__ __forceinline__ void record_bad_position(unsigned long long* err) {
  atomicCAS(err, 0ull, (kFaultBadOffsets << 56) | (static_cast<unsigned long long>(blockIdx.x & 0xFFFFFFu) << 16));
}

// ------------------------------------------------------------------ sort ----
// One cluster of C CTAs of W warps; warp g of all C * W takes the g-th
// contiguous run of pairs.  Pass 1 counts each warp's pairs per expert in a
// shared-memory row of its own (lanes with the same expert are found by votes
// and counted by one of them, so no two lanes write one counter);
// the counts become starts by prefix sums over warps, over CTAs (through
// distributed shared memory) and over experts; pass 2 hands out the rows in
// pair order.
// What bounds it: latency.  The ids are 0.3 MB for the 4096 x 8 layer; one
// launch with its counts on chip replaces three passes through global memory.
// 32768 ids of 32 experts: 6.0 us, with 8 CTAs 7.6; 131072 of 256 experts 15.4 and
// 25.4.  Sums over the warps' counts and the CTAs' totals that waited for one load
// after the other cost the former 5 us.
constexpr int kSortMaxWarps = 32;
constexpr int kSortAhead = 4;    // id loads in flight per lane
constexpr int kSortCtas = 16;    // of the cluster, where the device has room for it; else 8

template <class ID>
__global__ void __launch_bounds__(kSortMaxWarps * 32)
    moe_sort_kernel(const ID* ids, int pairs, int E, int n_cta, int* offsets, int* order, int* position) {
  extern __shared__ int sm[];
  grid_dependency_wait();
  grid_dependents_launch();
  const int W = static_cast<int>(blockDim.x >> 5);
  const int buckets = E + 1;         // bucket E: pairs without an expert
  int* hist = sm;                    // [W][buckets]
  int* total = sm + W * buckets;       // [buckets] this CTA's counts
  int* start = total + buckets;      // [buckets] this CTA's first row in each bucket
  int* part = start + buckets;       // [32] scan partials
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  const uint32_t rank = n_cta > 1 ? cluster_ctarank() : 0u;

  const long long runs = static_cast<long long>(n_cta) * W;
  const long long per = ((pairs + runs - 1) / runs + 31) / 32 * 32;
  const long long first = (static_cast<long long>(rank) * W + warp) * per;
  const long long last = first + per < pairs ? first + per : pairs;
  int* mine = hist + warp * buckets;
  const unsigned below = (1u << lane) - 1u;

  auto load = [&](long long p) -> int {
    if (p >= last) return -1;
    const ID v = ids[p];
    return v >= 0 && v < static_cast<ID>(E) ? static_cast<int>(v) : E;
  };
  // The lanes with this lane's bucket, bit by bit of the bucket's number: 6
  // votes for 32 experts take less time than one match.any (32768 pairs 6.0 us,
  // with match.any 6.5; 131072 of 256 experts 15.4 and 21.4).
  const int bits = 32 - __clz(E);
  auto same_bucket = [&](int key) -> unsigned {
    unsigned same = __ballot_sync(0xffffffffu, key >= 0);
    for (int b = 0; b < bits; ++b) {
      const unsigned set = __ballot_sync(0xffffffffu, (key >> b) & 1);
      same &= (key >> b) & 1 ? set : ~set;
    }
    return same;
  };
  int key[kSortAhead];
#pragma unroll
  for (int a = 0; a < kSortAhead; ++a) key[a] = load(first + 32 * a + lane);
  for (int b = lane; b < buckets; b += 32) mine[b] = 0;
  __syncwarp();
  for (long long p0 = first; p0 < last; p0 += 32 * kSortAhead) {
    if (p0 != first) {
#pragma unroll
      for (int a = 0; a < kSortAhead; ++a) key[a] = load(p0 + 32 * a + lane);
    }
#pragma unroll
    for (int a = 0; a < kSortAhead; ++a) {
      if (p0 + 32 * a >= last) break;
      const unsigned same = same_bucket(key[a]);
      if (key[a] >= 0 && (same & below) == 0) mine[key[a]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // warps' counts -> each warp's start inside the CTA's share of the bucket,
  // a thread a bucket, 8 loads ahead
  for (int b = static_cast<int>(threadIdx.x); b < buckets; b += static_cast<int>(blockDim.x)) {
    int run = 0;
    for (int w0 = 0; w0 < W; w0 += 8) {
      int c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = w0 + i < W ? hist[(w0 + i) * buckets + b] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (w0 + i < W) hist[(w0 + i) * buckets + b] = run;
        run += c[i];
      }
    }
    total[b] = run;
  }
  if (n_cta > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // every CTA: all CTAs' counts, the part of lower ranks, and the exclusive
  // sum over buckets, blockDim.x buckets at a time
  int carry = 0;
  for (int b0 = 0; b0 < buckets; b0 += static_cast<int>(blockDim.x)) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int all = 0, before = 0;
    if (b < buckets) {
      if (n_cta > 1) {
        int v[kSortCtas];
#pragma unroll
        for (int c = 0; c < kSortCtas; ++c) v[c] = c < n_cta ? ld_cluster(total + b, static_cast<uint32_t>(c)) : 0;
#pragma unroll
        for (int c = 0; c < kSortCtas; ++c) {
          if (c < static_cast<int>(rank)) before += v[c];
          all += v[c];
        }
      } else {
        all = total[b];
      }
    }
    int incl = all;
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      int v = lane < W ? part[lane] : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
      }
      part[lane] = v;
    }
    __syncthreads();
    const int excl = carry + (warp > 0 ? part[warp - 1] : 0) + incl - all;
    if (b < buckets) {
      start[b] = excl + before;
      if (rank == 0) offsets[b] = excl;  // for bucket E: the rows that have an expert
    }
    carry += part[31];
    __syncthreads();
  }
  for (long long p0 = first; p0 < last; p0 += 32 * kSortAhead) {
    if (per > 32 * kSortAhead) {  // else the keys are still there
#pragma unroll
      for (int a = 0; a < kSortAhead; ++a) key[a] = load(p0 + 32 * a + lane);
    }
#pragma unroll
    for (int a = 0; a < kSortAhead; ++a) {
      if (p0 + 32 * a >= last) break;
      const unsigned same = same_bucket(key[a]);
      if (key[a] >= 0) {
        const int at = start[key[a]] + mine[key[a]] + __popc(same & below);
        const int p = static_cast<int>(p0 + 32 * a + lane);
        position[p] = at;
        order[at] = p;
      }
      __syncwarp();
      if (key[a] >= 0 && (same & below) == 0) mine[key[a]] += __popc(same);
      __syncwarp();
    }
  }
  // a CTA's counts may be read by its peers until all have passed their sums
  if (n_cta > 1) cluster_sync_all();
}

// ------------------------------------------------------------------ rows ----

struct MoeRows {
  const void* src;      // dispatch: x; combine: rows; combine gradient: dy
  const void* rows_in;  // combine gradient: rows
  void* dst;            // dispatch: rows; combine: y; combine gradient: d_rows
  const float* weights; // combine: [pairs] or nullptr (all 1)
  float* d_weights;
  const int* position;
  const int* kept;      // &offsets[E]
  long long ld_src, ld_rows, ld_dst;  // in elements
  int T, k, vecs;       // vecs: vectors a row
  int pairs;            // T * k: rows of the expert order
  unsigned long long* err;
};

// A vector of VB bytes of elements T, as FP32 values and back.
template <int VB>
struct Raw;
template <>
struct Raw<16> {
  using type = uint4;
};
template <>
struct Raw<4> {
  using type = uint32_t;
};
template <>
struct Raw<2> {
  using type = uint16_t;
};

template <class T, int VB>
union Vec {
  typename Raw<VB>::type raw;
  T e[VB / sizeof(T)];
  __device__ Vec() {}
};

// An operand to be read with ld_global in vectors of VB bytes (the narrow loads
// need no pointer from behind the wait: the gradient of 2049 x 8 rows of 2047 FP32
// 54.9 us, with one 55.9).
template <int VB>
__device__ __forceinline__ const void* input(const void* p) {
  return VB == 16 ? behind_wait(p) : p;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float& d, float v) { d = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half& d, float v) { d = __float2half_rn(v); }

// Block (t, chunk): V vectors of token t per thread, blockDim.x apart, stored to
// its k rows.  The stores are the time; one vector of 16 bytes a thread reaches
// 6.5 TB/s, narrower ones need more of them (2049 x 8 rows of 2047 BF16, 2 bytes
// at a time: 29.2 us with one, 19.0 with 8).
template <int VB>
constexpr int dispatch_vectors() {
  return VB == 16 ? 1 : VB == 4 ? 4 : 8;
}

// Vectors of 4 bytes: the threads of a warp take those that fill one aligned
// line of 128 bytes of the row they store to, whatever its start, so that no
// store splits a sector with another warp's (2049 x 8 rows of 2047 FP32: 25.9 us,
// 33.9 without; with 2 bytes, or in the combine's gradient, whose vectors of dy
// would then be read once a pair, it costs more than it gives).  Vectors to
// skip at row `dst`.
template <int VB>
__device__ __forceinline__ int line_skew(const void* dst) {
  return VB == 4 ? static_cast<int>((reinterpret_cast<uintptr_t>(dst) & 127u) / VB) : 0;
}
template <int VB>
constexpr int most_skew() {
  return VB == 4 ? 128 / VB - 1 : 0;
}

template <int VB>
__global__ void __launch_bounds__(256) moe_dispatch_kernel(const __grid_constant__ MoeRows p, int chunks, int elt) {
  using R = typename Raw<VB>::type;
  constexpr int V = dispatch_vectors<VB>();
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = static_cast<int>(blockIdx.x / static_cast<unsigned>(chunks));
  const int step = static_cast<int>(blockDim.x);
  const int v0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(chunks)) * step * V + static_cast<int>(threadIdx.x);
  const R* src = reinterpret_cast<const R*>(static_cast<const char*>(input<VB>(p.src)) + t * p.ld_src * elt);
  R x[V];
  if constexpr (VB != 4) {
#pragma unroll
    for (int m = 0; m < V; ++m)
      if (v0 + m * step < p.vecs) x[m] = ld_global(src + v0 + m * step);
  }
  const int kept = *p.kept;
  const int* pos = p.position + static_cast<long long>(t) * p.k;
  for (int j = 0; j < p.k; ++j) {
    const int r = pos[j];
    if (static_cast<unsigned>(r) >= static_cast<unsigned>(p.pairs)) {
      if (threadIdx.x == 0) record_bad_position(p.err);
      continue;
    }
    R* dst = reinterpret_cast<R*>(static_cast<char*>(p.dst) + r * p.ld_dst * elt);
    const int v = v0 - line_skew<VB>(dst);
    if constexpr (VB == 4) {
#pragma unroll
      for (int m = 0; m < V; ++m)
        if (static_cast<unsigned>(v + m * step) < static_cast<unsigned>(p.vecs)) x[m] = ld_global(src + v + m * step);
    }
#pragma unroll
    for (int m = 0; m < V; ++m)
      if (static_cast<unsigned>(v + m * step) < static_cast<unsigned>(p.vecs)) dst[v + m * step] = r < kept ? x[m] : R{};
  }
}

// Loads in flight decide how near these two kernels come to the memory's rate,
// so a thread takes P pairs (k, 5 as 6 and 7 as 8; more in turns of 8) of V
// vectors and issues all P * V loads before it uses the first.  Measured for
// 4096 tokens x 8 experts, H = 4096 BF16: the combine 46.0 us (6.5 TB/s) with 8
// loads of 16 bytes a thread and 128 threads a block, 46.9 with 256 threads, 45.2
// with 16 loads, which take 5003 x 6 of H = 2056 from 23.8 to 29.2; the gradient
// 86.6 us (6.6 TB/s) with 16 loads, 88.6 with 8, 94.4 with 256 threads.  Narrower
// vectors: 32 loads for the combine (2049 x 8 rows of 2047 FP32: 25.8 us, 28.7
// with 16), 16 for the gradient (55.2; 53.1 with 32), and for the combine loads
// that leave no line in L1 (2049 x 8 rows of 2047 BF16 21.1 us, 22.3 with them in
// L1; the gradient and the dispatch lose by it).  Checks of the positions between
// the loads cost the combine 15 us.
constexpr int kRowThreads = 128;
template <int VB, int P, bool GRAD>
constexpr int vectors_of() {
  return (GRAD ? 16 : VB == 16 ? 8 : 32) / P;
}

// Block (t, chunk): V vectors of y[t] per thread, blockDim.x apart, from its k rows.
template <class T, int VB, int P>
__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(const __grid_constant__ MoeRows p, int chunks) {
  using R = typename Raw<VB>::type;
  constexpr int N = VB / static_cast<int>(sizeof(T));
  constexpr int V = vectors_of<VB, P, false>();
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = static_cast<int>(blockIdx.x / static_cast<unsigned>(chunks));
  const int step = static_cast<int>(blockDim.x);
  const int v0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(chunks)) * step * V + static_cast<int>(threadIdx.x);
  const int kept = min(*p.kept, p.pairs);
  const long long p0 = static_cast<long long>(t) * p.k;
  const T* rows = static_cast<const T*>(input<VB>(p.src));
  float acc[V][N];
#pragma unroll
  for (int m = 0; m < V; ++m)
#pragma unroll
    for (int i = 0; i < N; ++i) acc[m][i] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += P) {
    Vec<T, VB> x[P][V];
    float w[P];
    int row[P];
    bool has[P], bad = false;
    // all positions and weights, then all rows: nothing between the loads
#pragma unroll
    for (int a = 0; a < P; ++a) {
      row[a] = j0 + a < p.k ? p.position[p0 + j0 + a] : -1;
      w[a] = p.weights != nullptr && j0 + a < p.k ? p.weights[p0 + j0 + a] : 1.f;
    }
#pragma unroll
    for (int a = 0; a < P; ++a) {
      bad |= j0 + a < p.k && static_cast<unsigned>(row[a]) >= static_cast<unsigned>(p.pairs);
      has[a] = row[a] >= 0 && row[a] < kept;
      const R* src = reinterpret_cast<const R*>(rows + (has[a] ? row[a] : 0) * p.ld_src);
#pragma unroll
      for (int m = 0; m < V; ++m)
        if (has[a] && v0 + m * step < p.vecs) x[a][m].raw = ld_global_once(src + v0 + m * step);
    }
    if (bad && threadIdx.x == 0) record_bad_position(p.err);
#pragma unroll
    for (int a = 0; a < P; ++a)
      if (has[a]) {
#pragma unroll
        for (int m = 0; m < V; ++m)
#pragma unroll
          for (int i = 0; i < N; ++i) acc[m][i] = fmaf(w[a], to_f32(x[a][m].e[i]), acc[m][i]);
      }
  }
  R* dst = reinterpret_cast<R*>(static_cast<T*>(p.dst) + t * p.ld_dst);
#pragma unroll
  for (int m = 0; m < V; ++m) {
    if (v0 + m * step < p.vecs) {
      Vec<T, VB> y;
#pragma unroll
      for (int i = 0; i < N; ++i) from_f32(y.e[i], acc[m][i]);
      dst[v0 + m * step] = y.raw;
    }
  }
}

// Block t: d_rows of token t's k rows and the k inner products.
template <class T, int VB, int P>
__global__ void __launch_bounds__(kRowThreads) moe_combine_grad_kernel(const __grid_constant__ MoeRows p) {
  using R = typename Raw<VB>::type;
  constexpr int N = VB / static_cast<int>(sizeof(T));
  constexpr int V = vectors_of<VB, P, true>();
  __shared__ float sums[kRowThreads / 32][P];
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = static_cast<int>(blockIdx.x);
  const int step = static_cast<int>(blockDim.x);
  const int kept = min(*p.kept, p.pairs);
  const long long p0 = static_cast<long long>(t) * p.k;
  const R* dy = reinterpret_cast<const R*>(static_cast<const T*>(input<VB>(p.src)) + t * p.ld_src);
  const T* rows = static_cast<const T*>(input<VB>(p.rows_in));
  for (int j0 = 0; j0 < p.k; j0 += P) {
    int row[P];
    float w[P], dot[P];
    bool bad = false;
#pragma unroll
    for (int a = 0; a < P; ++a) {
      const bool in = j0 + a < p.k;
      row[a] = in ? p.position[p0 + j0 + a] : -1;
      w[a] = in ? p.weights[p0 + j0 + a] : 0.f;
    }
#pragma unroll
    for (int a = 0; a < P; ++a) {
      if (static_cast<unsigned>(row[a]) >= static_cast<unsigned>(p.pairs)) {
        bad |= j0 + a < p.k;
        row[a] = -1;
      }
      dot[a] = 0.f;
    }
    if (bad && threadIdx.x == 0) record_bad_position(p.err);
    const R* from[P];
    R* to[P];
#pragma unroll
    for (int a = 0; a < P; ++a) {
      const int r = max(row[a], 0);
      from[a] = reinterpret_cast<const R*>(rows + r * p.ld_rows);
      to[a] = reinterpret_cast<R*>(static_cast<T*>(p.dst) + r * p.ld_dst);
    }
    for (int v = static_cast<int>(threadIdx.x); v < p.vecs; v += step * V) {
      Vec<T, VB> g[V], x[P][V];
      auto in = [&](int m) { return v + m * step < p.vecs; };
#pragma unroll
      for (int m = 0; m < V; ++m)
        if (in(m)) g[m].raw = ld_global(dy + v + m * step);
#pragma unroll
      for (int a = 0; a < P; ++a)
#pragma unroll
        for (int m = 0; m < V; ++m)
          if (row[a] >= 0 && row[a] < kept && in(m)) x[a][m].raw = ld_global(from[a] + v + m * step);
#pragma unroll
      for (int a = 0; a < P; ++a) {
        if (row[a] < 0) continue;
#pragma unroll
        for (int m = 0; m < V; ++m) {
          if (!in(m)) continue;
          Vec<T, VB> d;
          if (row[a] < kept) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float y = to_f32(g[m].e[i]);
              dot[a] = fmaf(to_f32(x[a][m].e[i]), y, dot[a]);
              from_f32(d.e[i], w[a] * y);
            }
          } else {
            d.raw = R{};
          }
          to[a][v + m * step] = d.raw;
        }
      }
    }
#pragma unroll
    for (int a = 0; a < P; ++a) {
      for (int d = 16; d > 0; d >>= 1) dot[a] += __shfl_xor_sync(0xffffffffu, dot[a], d);
      if ((threadIdx.x & 31u) == 0) sums[threadIdx.x >> 5][a] = dot[a];
    }
    __syncthreads();
    const int a = static_cast<int>(threadIdx.x);
    if (a < P && j0 + a < p.k) {
      float total = 0.f;
      for (int w2 = 0; w2 < step / 32; ++w2) total += sums[w2][a];
      p.d_weights[p0 + j0 + a] = total;
    }
    __syncthreads();
  }
}

// Widest vector (16, 4 or 2 bytes, at least an element) in which every
// row of H elements can be read and written whole.
int vector_bytes(int H, int elt, std::initializer_list<const void*> ptrs, std::initializer_list<long long> lds) {
  uintptr_t bits = static_cast<uintptr_t>(static_cast<long long>(H) * elt);
  for (const void* q : ptrs) bits |= reinterpret_cast<uintptr_t>(q);
  for (long long ld : lds) bits |= static_cast<uintptr_t>(ld * elt);
  return (bits & 15u) == 0 ? 16 : (bits & 3u) == 0 ? 4 : elt;
}

int elt_bytes(int dtype) { return dtype == BWG_OUT_FP32 ? 4 : 2; }

bool dtype_ok(int dtype) { return dtype == BWG_OUT_BF16 || dtype == BWG_OUT_FP16 || dtype == BWG_OUT_FP32; }

bool elt_aligned(const void* q, int elt) { return (reinterpret_cast<uintptr_t>(q) & static_cast<uintptr_t>(elt - 1)) == 0; }

// Arguments that the row kernels share; *empty: nothing to do.
bwg_status check_rows(int dtype, int T, int H, int k, int E, const int* position, const int* offsets, bool* empty) {
  *empty = false;
  if (!dtype_ok(dtype) || T < 0 || H < 0 || k < 1 || E < 1) return BWG_ERR_INVALID_ARG;
  if (E > kMaxExperts || H > kMaxColumns || static_cast<long long>(T) * k > 0x7fffffffLL) return BWG_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) {
    *empty = true;
    return BWG_OK;
  }
  if (position == nullptr || offsets == nullptr) return BWG_ERR_INVALID_ARG;
  return BWG_OK;
}

// Threads of a row block (at most `most`, whole warps) and blocks a row, for
// `per` vectors a thread, the row shared out evenly.
void row_shape(int vecs, int per, int most, int* threads, int* chunks) {
  *chunks = std::max(1, (vecs + most * per - 1) / (most * per));
  const int each = (vecs + *chunks * per - 1) / (*chunks * per);
  *threads = std::max(32, (each + 31) / 32 * 32);
}

template <class T, int VB, int P>
cudaError_t launch_combine_as(const MoeRows& p, cudaStream_t s) {
  int threads, chunks;
  row_shape(p.vecs, vectors_of<VB, P, false>(), kRowThreads, &threads, &chunks);
  const long long blocks = static_cast<long long>(p.T) * chunks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_overlapped(moe_combine_kernel<T, VB, P>, static_cast<unsigned>(blocks), static_cast<unsigned>(threads),
                           0, s, 1, p, chunks);
}

template <class T, int VB, int P>
cudaError_t launch_grad_as(const MoeRows& p, cudaStream_t s) {
  int threads, chunks;
  row_shape(p.vecs, vectors_of<VB, P, true>(), kRowThreads, &threads, &chunks);
  return launch_overlapped(moe_combine_grad_kernel<T, VB, P>, static_cast<unsigned>(p.T),
                           static_cast<unsigned>(threads), 0, s, 1, p);
}

template <class T, int VB>
cudaError_t launch_pairs(bool grad, const MoeRows& p, cudaStream_t s) {
  switch (p.k > 6 ? 8 : p.k > 4 ? 6 : p.k) {
    case 1: return grad ? launch_grad_as<T, VB, 1>(p, s) : launch_combine_as<T, VB, 1>(p, s);
    case 2: return grad ? launch_grad_as<T, VB, 2>(p, s) : launch_combine_as<T, VB, 2>(p, s);
    case 3: return grad ? launch_grad_as<T, VB, 3>(p, s) : launch_combine_as<T, VB, 3>(p, s);
    case 4: return grad ? launch_grad_as<T, VB, 4>(p, s) : launch_combine_as<T, VB, 4>(p, s);
    case 6: return grad ? launch_grad_as<T, VB, 6>(p, s) : launch_combine_as<T, VB, 6>(p, s);
    default: return grad ? launch_grad_as<T, VB, 8>(p, s) : launch_combine_as<T, VB, 8>(p, s);
  }
}

template <class T>
cudaError_t launch_vectors(bool grad, const MoeRows& p, int vb, cudaStream_t s) {
  if (vb == 16) return launch_pairs<T, 16>(grad, p, s);
  if (vb == 4) return launch_pairs<T, 4>(grad, p, s);
  if constexpr (sizeof(T) == 2) return launch_pairs<T, 2>(grad, p, s);
  return cudaErrorInvalidValue;
}

cudaError_t launch_weighted(bool grad, const MoeRows& p, int dtype, int vb, cudaStream_t s) {
  return dtype == BWG_OUT_FP32   ? launch_vectors<float>(grad, p, vb, s)
         : dtype == BWG_OUT_BF16 ? launch_vectors<__nv_bfloat16>(grad, p, vb, s)
                                 : launch_vectors<__half>(grad, p, vb, s);
}

bwg_status run_combine(const void* rows, int dtype, int T, int H, int ldr, int k, const float* weights,
                       const int* position, const int* offsets, int E, void* Y, int ldy, cudaStream_t s) {
  bool empty;
  bwg_status st = check_rows(dtype, T, H, k, E, position, offsets, &empty);
  if (st != BWG_OK || empty) return st;
  if (rows == nullptr || Y == nullptr || ldr < H || ldy < H) return BWG_ERR_INVALID_ARG;
  const int elt = elt_bytes(dtype);
  if (!elt_aligned(rows, elt) || !elt_aligned(Y, elt)) return BWG_ERR_ALIGNMENT;
  Runtime rt;
  if ((st = runtime_device(&rt)) != BWG_OK) return st;
  const int vb = vector_bytes(H, elt, {rows, Y}, {ldr, ldy});
  MoeRows p = {};
  p.src = rows;
  p.dst = Y;
  p.weights = weights;
  p.position = position;
  p.kept = offsets + E;
  p.ld_src = ldr;
  p.ld_dst = ldy;
  p.T = T;
  p.k = k;
  p.pairs = T * k;
  p.err = rt.err;
  p.vecs = static_cast<int>(static_cast<long long>(H) * elt / vb);
  return runtime_status(launch_weighted(false, p, dtype, vb, s));
}

size_t sort_smem(int warps, int E) { return (static_cast<size_t>(warps + 2) * (E + 1) + 32) * sizeof(int); }

// CTAs of the sort's cluster on this device: 16 (beyond the portable size) if
// one such cluster fits with the most shared memory a call takes, else 8.
template <class ID>
cudaError_t sort_ctas(int device, int* n) {
  static std::mutex mu;
  static int known[64];
  if (device >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (known[device] == 0) {
    const void* fn = reinterpret_cast<const void*>(moe_sort_kernel<ID>);
    const size_t smem = sort_smem(kSortMaxWarps, kMaxExperts);
    cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortCtas, 1, 1);
    cfg.blockDim = dim3(kSortMaxWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg) != cudaSuccess) {
      cudaGetLastError();
      clusters = 0;
    }
    known[device] = clusters > 0 ? kSortCtas : 8;
  }
  *n = known[device];
  return cudaSuccess;
}

template <class ID>
cudaError_t launch_sort(const void* ids, int pairs, int E, int* offsets, int* order, int* position, int device,
                        cudaStream_t s) {
  // One CTA up to 2048 pairs (256 experts: 5.0 us), a warp for each 128 of
  // them; a cluster beyond (8192 pairs with 8 CTAs: 6.2 us, one CTA takes 7.7
  // for 4096; 32768 pairs with 16 CTAs 6.0 us, with 8 7.6).
  int n_cta = 1;
  const cudaError_t known = sort_ctas<ID>(device, &n_cta);
  if (known != cudaSuccess) return known;
  if (pairs <= 2048) n_cta = 1;
  const int warps = n_cta > 1 ? kSortMaxWarps : std::min(kSortMaxWarps, std::max(4, (pairs + 127) / 128));
  // (overlapped launches throughout this file: 4096 x 8, H = 4096, sort and
  // dispatch 54.6 -> 52.1 us back to back; a sort of 128 pairs 2.4 -> 2.2)
  return launch_overlapped(moe_sort_kernel<ID>, static_cast<unsigned>(n_cta), static_cast<unsigned>(warps * 32),
                           sort_smem(warps, E), s, static_cast<unsigned>(n_cta), static_cast<const ID*>(ids), pairs, E,
                           n_cta, offsets, order, position);
}

}  // namespace
}  // namespace bwg

using namespace bwg;

extern "C" {

bwg_status moe_sort(const void* expert_ids, int id_bytes, int pairs, int E, int* offsets, int* order, int* position,
                    void* stream) {
  if ((id_bytes != 4 && id_bytes != 8) || pairs < 0 || E < 1 || offsets == nullptr) return BWG_ERR_INVALID_ARG;
  if (E > kMaxExperts) return BWG_ERR_UNSUPPORTED;
  if (pairs > 0 && (expert_ids == nullptr || order == nullptr || position == nullptr)) return BWG_ERR_INVALID_ARG;
  if (!elt_aligned(expert_ids, id_bytes)) return BWG_ERR_ALIGNMENT;
  Runtime rt;
  const bwg_status st = runtime_device(&rt);
  if (st != BWG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return runtime_status(id_bytes == 8 ? launch_sort<long long>(expert_ids, pairs, E, offsets, order, position, rt.device, s)
                                      : launch_sort<int>(expert_ids, pairs, E, offsets, order, position, rt.device, s));
}

bwg_status moe_dispatch(const void* X, int dtype, int T, int H, int ldx, int k, const int* position,
                        const int* offsets, int E, void* rows, int ldr, void* stream) {
  bool empty;
  bwg_status st = check_rows(dtype, T, H, k, E, position, offsets, &empty);
  if (st != BWG_OK || empty) return st;
  if (X == nullptr || rows == nullptr || ldx < H || ldr < H) return BWG_ERR_INVALID_ARG;
  const int elt = elt_bytes(dtype);
  if (!elt_aligned(X, elt) || !elt_aligned(rows, elt)) return BWG_ERR_ALIGNMENT;
  Runtime rt;
  if ((st = runtime_device(&rt)) != BWG_OK) return st;
  const int vb = vector_bytes(H, elt, {X, rows}, {ldx, ldr});
  MoeRows p = {};
  p.src = X;
  p.dst = rows;
  p.position = position;
  p.kept = offsets + E;
  p.ld_src = ldx;
  p.ld_dst = ldr;
  p.T = T;
  p.k = k;
  p.pairs = T * k;
  p.err = rt.err;
  p.vecs = static_cast<int>(static_cast<long long>(H) * elt / vb);
  int threads, chunks;
  row_shape(p.vecs + (vb == 4 ? most_skew<4>() : 0),
            vb == 16 ? dispatch_vectors<16>() : vb == 4 ? dispatch_vectors<4>() : dispatch_vectors<2>(), 256, &threads,
            &chunks);
  const long long blocks = static_cast<long long>(T) * chunks;
  if (blocks > 0x7fffffffLL) return BWG_ERR_UNSUPPORTED;
  const unsigned b = static_cast<unsigned>(blocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto kernel = vb == 16 ? moe_dispatch_kernel<16> : vb == 4 ? moe_dispatch_kernel<4> : moe_dispatch_kernel<2>;
  return runtime_status(launch_overlapped(kernel, b, static_cast<unsigned>(threads), 0, s, 1, p, chunks, elt));
}

bwg_status moe_dispatch_grad(const void* d_rows, int dtype, int T, int H, int ldr, int k, const int* position,
                             const int* offsets, int E, void* dX, int ldx, void* stream) {
  return run_combine(d_rows, dtype, T, H, ldr, k, nullptr, position, offsets, E, dX, ldx,
                     static_cast<cudaStream_t>(stream));
}

bwg_status moe_combine(const void* rows, int dtype, int T, int H, int ldr, int k, const float* weights,
                       const int* position, const int* offsets, int E, void* Y, int ldy, void* stream) {
  if (T > 0 && H > 0 && weights == nullptr) return BWG_ERR_INVALID_ARG;
  return run_combine(rows, dtype, T, H, ldr, k, weights, position, offsets, E, Y, ldy,
                     static_cast<cudaStream_t>(stream));
}

bwg_status moe_combine_grad(const void* dY, const void* rows, int dtype, int T, int H, int ldy, int ldr, int k,
                            const float* weights, const int* position, const int* offsets, int E, void* d_rows,
                            int ld_dr, float* d_weights, void* stream) {
  bool empty;
  bwg_status st = check_rows(dtype, T, H < 1 ? 1 : H, k, E, position, offsets, &empty);
  if (H < 0) return BWG_ERR_INVALID_ARG;
  if (st != BWG_OK || empty) return st;
  if (weights == nullptr || d_weights == nullptr) return BWG_ERR_INVALID_ARG;
  if (H > 0 && (dY == nullptr || rows == nullptr || d_rows == nullptr || ldy < H || ldr < H || ld_dr < H))
    return BWG_ERR_INVALID_ARG;
  const int elt = elt_bytes(dtype);
  if (!elt_aligned(dY, elt) || !elt_aligned(rows, elt) || !elt_aligned(d_rows, elt)) return BWG_ERR_ALIGNMENT;
  Runtime rt;
  if ((st = runtime_device(&rt)) != BWG_OK) return st;
  const int vb = vector_bytes(H, elt, {dY, rows, d_rows}, {ldy, ldr, ld_dr});
  MoeRows p = {};
  p.src = dY;
  p.rows_in = rows;
  p.dst = d_rows;
  p.weights = weights;
  p.d_weights = d_weights;
  p.position = position;
  p.kept = offsets + E;
  p.ld_src = ldy;
  p.ld_rows = ldr;
  p.ld_dst = ld_dr;
  p.T = T;
  p.k = k;
  p.pairs = T * k;
  p.err = rt.err;
  p.vecs = static_cast<int>(static_cast<long long>(H) * elt / vb);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return runtime_status(launch_weighted(true, p, dtype, vb, s));
}

}  // extern "C"
