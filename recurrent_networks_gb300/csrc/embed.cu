// Token embedding with scaling and its gradient by sorted tokens
// (include/rnn.h).
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rnn.h"

namespace rnn {
namespace {

// A vector of VB bytes of the storage type, as fp32 values and back.
template <typename T, int VB> struct Vec {
  static constexpr int N = VB / (int)sizeof(T);
  T v[N];
};
template <int VB> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = unsigned; };
template <> struct Raw<2> { using type = unsigned short; };
template <typename T, int VB> __device__ __forceinline__ Vec<T, VB> load_vec(const T* p) {
  typename Raw<VB>::type r = __ldg((const typename Raw<VB>::type*)p);
  return *(Vec<T, VB>*)&r;
}
template <typename T, int VB> __device__ __forceinline__ void store_vec(T* p, const Vec<T, VB>& v) {
  *(typename Raw<VB>::type*)p = *(const typename Raw<VB>::type*)&v;
}

// A vector's values in fp32, by the pair for bf16 (packed instructions), and back.
template <typename T, int VB> struct Wide {
  static constexpr int P = sizeof(T) == 2 && VB >= 4 ? 2 : 1, W = VB / (int)sizeof(T) / P;
  FV<P> f[W];
  __device__ __forceinline__ void set(const Vec<T, VB>& v) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (P == 2) {
        const uint32_t w = ((const uint32_t*)&v)[i];
        f[i] = FV<P>{{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)}};
      } else {
        f[i].v[0] = to_f(v.v[i]);
      }
    }
  }
  __device__ __forceinline__ void scale(float s) {
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = mul(f[i], splat<P>(s));
  }
  __device__ __forceinline__ Vec<T, VB> get() const {
    Vec<T, VB> v;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (P == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].v[0], f[i].v[P - 1]);
        ((uint32_t*)&v)[i] = *(const uint32_t*)&h;
      } else {
        v.v[i] = from_f<T>(f[i].v[0]);
      }
    }
    return v;
  }
};

// ---- forward --------------------------------------------------------------------
// `lanes` lanes (a power of two) to a token, 16-byte vectors where the rows
// allow, ROWS tokens of a lane group in flight. Bound by out's bytes (the rows of
// frequent tokens come from L2): n=131072 E=1024 bf16 60 us, 5.5 TB/s of the 338
// MB that have to move. Scaling pair by pair in fp32; element by element the
// conversions alone kept 74 % of the issue slots busy.
template <typename T, typename I, int VB>
__global__ void __launch_bounds__(256) embed_fwd_kernel(long long n, int V, int E, int lanes, const I* ids, const T* W,
                                                        float scale, T* out, unsigned* status) {
  constexpr int ROWS = 4;
  using X = Vec<T, VB>;
  const int groups = 256 / lanes, g = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int nv = E / X::N;
  const long long step = (long long)gridDim.x * groups * ROWS;
  for (long long i0 = ((long long)blockIdx.x * groups + g) * ROWS; i0 < n; i0 += step) {
    const T* src[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long long v = i0 + r < n ? (long long)ids[i0 + r] : 0;
      const bool ok = v >= 0 && v < V;
      src[r] = ok ? W + (size_t)v * E : nullptr;
      if (!ok && l == 0 && status) atomicOr(status, STATUS_RANGE);
    }
    for (int e = l; e < nv; e += lanes) {
      X x[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (src[r]) x[r] = load_vec<T, VB>(src[r] + (size_t)e * X::N);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (i0 + r >= n) break;
        Wide<T, VB> w = {};
        if (src[r]) w.set(x[r]);
        if (src[r]) w.scale(scale);
        store_vec<T, VB>(out + (size_t)(i0 + r) * E + (size_t)e * X::N, w.get());
      }
    }
  }
}

// ---- gradient: sorting the tokens --------------------------------------------------
// A token's key is its id, or V (past every row) when it has no gradient. The
// tokens are sorted by key, equal keys in token order: least significant digit
// first, DIGIT_MAX bits at most a pass, each pass a count of the digits of
// every tile of TILE tokens, a scan of the counts in (digit, tile) order and a
// stable scatter, which also counts the next pass's digits by the places it
// writes to. All counts are whole numbers, so nothing depends on timing.
constexpr int SORT_THREADS = 256, SORT_WARPS = SORT_THREADS / 32, SORT_ROUNDS = 4;
constexpr int TILE = SORT_THREADS * SORT_ROUNDS;
constexpr int DIGIT_MAX = 11;

struct SortArgs {
  long long n, pad;
  int V, tiles, shift, bits;
  const void* ids;            // first pass; then kin, pin
  const unsigned *kin, *pin;
  unsigned *kout, *pout;
  unsigned* hist;             // [1 << bits][tiles]
  unsigned* total;            // [1 << bits]
  unsigned* hist_next;        // the next pass's counts (null in the last one)
  unsigned* status;
  uint4* zero;                // this launch's share of dW to clear, by the blocks past the tiles
  size_t zeros;               // 16-byte units
};

template <typename I> __device__ __forceinline__ unsigned key_of(const I* ids, long long i, const SortArgs& p) {
  const long long v = (long long)ids[i];
  const bool ok = v >= 0 && v < p.V;
  if (!ok) atomicOr(p.status, STATUS_RANGE);
  return ok && v != p.pad ? (unsigned)v : (unsigned)p.V;
}
__device__ __forceinline__ bool zero_share(const SortArgs& p, int first) {
  if ((int)blockIdx.x < first) return false;
  const size_t stride = (size_t)(gridDim.x - first) * blockDim.x;
  for (size_t i = (size_t)(blockIdx.x - first) * blockDim.x + threadIdx.x; i < p.zeros; i += stride)
    p.zero[i] = make_uint4(0, 0, 0, 0);
  return true;
}

// The first pass's counts.
template <typename I> __global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(SortArgs p) {
  if (zero_share(p, p.tiles)) return;
  extern __shared__ unsigned count[];
  const int bins = 1 << p.bits;
  for (int d = threadIdx.x; d < bins; d += SORT_THREADS) count[d] = 0;
  __syncthreads();
  const long long base = (long long)blockIdx.x * TILE;
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const long long i = base + r * SORT_THREADS + threadIdx.x;
    if (i < p.n) atomicAdd(&count[key_of((const I*)p.ids, i, p) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += SORT_THREADS) p.hist[(size_t)d * p.tiles + blockIdx.x] = count[d];
}

// Exclusive sums of p.hist along the tiles, in place, a warp a digit; the
// digits' totals go to p.total. Clears the next pass's counts.
__global__ void __launch_bounds__(SORT_THREADS) sort_scan_kernel(SortArgs p) {
  const int bins = 1 << p.bits, blocks = (bins + SORT_WARPS - 1) / SORT_WARPS;
  if (zero_share(p, blocks)) return;
  const int d = blockIdx.x * SORT_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (d >= bins) return;
  unsigned* row = p.hist + (size_t)d * p.tiles;
  unsigned carry = 0;
  for (int base = 0; base < p.tiles; base += 128) {
    unsigned v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = base + q * 32 + lane < p.tiles ? row[base + q * 32 + lane] : 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      unsigned inc = v[q];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      if (base + q * 32 + lane < p.tiles) row[base + q * 32 + lane] = carry + inc - v[q];
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  if (lane == 0) p.total[d] = carry;
  if (p.hist_next)
    for (int t = lane; t < p.tiles; t += 32) p.hist_next[(size_t)d * p.tiles + t] = 0;
}

template <typename I, bool FIRST> __global__ void __launch_bounds__(SORT_THREADS) sort_scatter_kernel(SortArgs p) {
  if (zero_share(p, p.tiles)) return;
  extern __shared__ unsigned place[];  // [SORT_WARPS][bins]: the warp's counts, then where its next key of a digit goes
  __shared__ unsigned warp_sum[SORT_WARPS];
  const int bins = 1 << p.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = threadIdx.x; d < bins * SORT_WARPS; d += SORT_THREADS) place[d] = 0;
  __syncthreads();
  unsigned* mine = place + warp * bins;
  const long long base = (long long)blockIdx.x * TILE + warp * SORT_ROUNDS * 32 + lane;  // a warp's keys are consecutive
  unsigned key[SORT_ROUNDS];
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const long long i = base + r * 32;
    key[r] = i < p.n ? (FIRST ? key_of((const I*)p.ids, i, p) : p.kin[i]) : 0;
    if (i < p.n) atomicAdd(&mine[key[r] >> p.shift & (bins - 1)], 1u);
  }
  // where a digit's keys begin: the sum of the totals of the digits before it
  const int per = (bins + SORT_THREADS - 1) / SORT_THREADS, d0 = min(bins, (int)threadIdx.x * per), d1 = min(bins, d0 + per);
  unsigned sum = 0;
  for (int d = d0; d < d1; ++d) sum += p.total[d];
  unsigned inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  unsigned begin = inc - sum;
  for (int w = 0; w < warp; ++w) begin += warp_sum[w];
  for (int d = d0; d < d1; ++d) {
    unsigned at = begin + p.hist[(size_t)d * p.tiles + blockIdx.x];
    begin += p.total[d];
#pragma unroll
    for (int w = 0; w < SORT_WARPS; ++w) {
      const unsigned c = place[w * bins + d];
      place[w * bins + d] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const long long i = base + r * 32;
    const bool on = i < p.n;
    const unsigned d = on ? key[r] >> p.shift & (bins - 1) : bins;  // lanes past the end match one another alone
    const unsigned peers = __match_any_sync(0xffffffffu, d);
    const unsigned before = __popc(peers & ((1u << lane) - 1));
    unsigned at = 0;
    if (on) at = mine[d] + before;
    __syncwarp();
    if (on && before == 0) mine[d] += __popc(peers);
    __syncwarp();
    if (on) {
      p.kout[at] = key[r];
      if (p.hist_next) atomicAdd(&p.hist_next[(size_t)(key[r] >> (p.shift + p.bits) & (bins - 1)) * p.tiles + at / TILE], 1u);
      p.pout[at] = FIRST ? (unsigned)i : p.pin[i];
    }
  }
}

// ---- gradient: summing the sorted tokens' rows ---------------------------------------
struct SumArgs {
  long long n;
  int V, E, piece, coltiles;
  long long pieces;
  const unsigned *key, *pos;
  const void* dout;
  float scale;
  void* dW;
  float* part;  // [pieces][2][E]: sums of a piece's first id (begun in an earlier piece) and last id (going on in the next)
};

// N fp32 partial sums at p (aligned to their size where N is 4 or 8).
template <int N> __device__ __forceinline__ void store_part(float* p, const float* x) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int q = 0; q < N; q += 4) *(float4*)(p + q) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
  } else {
#pragma unroll
    for (int q = 0; q < N; ++q) p[q] = x[q];
  }
}
template <int N> __device__ __forceinline__ void load_part(const float* p, float* x) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int q = 0; q < N; q += 4) {
      const float4 v = *(const float4*)(p + q);
      x[q] = v.x, x[q + 1] = v.y, x[q + 2] = v.z, x[q + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < N; ++q) x[q] = p[q];
  }
}

// A warp sums `piece` (at most 32) sorted tokens over 32 vectors of columns, in
// order. An id whose tokens all lie in the piece is written to dW; what belongs
// to an id that crosses the piece's ends goes to part. Bound by the gather of
// dout's rows: every lane copies its vector of the next RING rows into its own
// place of a ring in shared memory, so that up to 15 rows a warp are on their
// way while one is added: 56 us for n=131072 E=1024 bf16, 5.6 TB/s (two register
// batches of 4 rows spilled and reached 2.1 TB/s).
constexpr int PIECE_MAX = 32, RING = 16;
template <int VB> __device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  static_assert(VB == 16 || VB == 8 || VB == 4, "cp.async sizes");
  if constexpr (VB == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(VB) : "memory");
}
template <typename T, int VB> __global__ void __launch_bounds__(256) embed_sum_kernel(SumArgs p) {
  using X = Vec<T, VB>;
  __shared__ __align__(16) unsigned char ring[8][RING][32 * VB];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long w = (long long)blockIdx.x * 8 + warp;
  const long long piece = w / p.coltiles;
  if (piece >= p.pieces) return;
  const int col = ((int)(w % p.coltiles) * 32 + lane) * X::N;
  const long long i0 = piece * p.piece;
  const int count = (int)min((long long)p.piece, p.n - i0);
  const unsigned none = 0xffffffffu;
  const unsigned key = lane < count ? __ldg(p.key + i0 + lane) : none;
  const unsigned pos = lane < count ? __ldg(p.pos + i0 + lane) : 0;
  const unsigned prev = i0 > 0 ? __ldg(p.key + i0 - 1) : none;
  const unsigned next = i0 + count < p.n ? __ldg(p.key + i0 + count) : none;
  // the tokens without a gradient come last
  const int sums = __popc(__ballot_sync(0xffffffffu, key < (unsigned)p.V));
  const bool on = col < p.E;
  const T* dout = (const T*)p.dout + col;
  const uint32_t mine = smem_u32(&ring[warp][0][lane * VB]);
  auto ask = [&](int j, unsigned s) {
    if (j < sums && on) {
      if constexpr (VB >= 4)
        copy_async<VB>(mine + j % RING * 32 * VB, dout + (size_t)s * p.E);
      else  // rows of odd width: no asynchronous copy of 2 bytes
        *(X*)&ring[warp][j % RING][lane * VB] = load_vec<T, VB>(dout + (size_t)s * p.E);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int j = 0; j < RING - 1; ++j) ask(j, __shfl_sync(0xffffffffu, pos, j));
  Wide<T, VB> acc = {};
  unsigned cur = none;
  for (int j = 0; j < sums; ++j) {
    ask(j + RING - 1, __shfl_sync(0xffffffffu, pos, (j + RING - 1) & 31));
    const unsigned k = __shfl_sync(0xffffffffu, key, j), after = j + 1 < count ? __shfl_sync(0xffffffffu, key, j + 1) : next;
    asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
    const X x = *(const X*)&ring[warp][j % RING][lane * VB];
    Wide<T, VB> w;
    w.set(x);
    if (k != cur) {
      acc = w;
    } else {
#pragma unroll
      for (int i = 0; i < acc.W; ++i) acc.f[i] = add(acc.f[i], w.f[i]);
    }
    cur = k;
    if (!on || (after == k && j + 1 < count)) continue;
    const bool head = k == prev, tail = after == k;
    if (!head && !tail) {
      acc.scale(p.scale);
      store_vec<T, VB>((T*)p.dW + (size_t)k * p.E + col, acc.get());
    } else {
      store_part<X::N>(p.part + ((size_t)piece * 2 + (head ? 0 : 1)) * p.E + col, (const float*)acc.f);
    }
  }
}

// The ids that cross pieces (16 us of the 122 us backward at n=131072 V=50000
// E=1024, latency: few registers keep four blocks an SM, 21 us with two): a warp
// per piece in which such an id begins, over 32 vectors of columns, adds the
// pieces' sums in order. An id over more than LONG pieces is shared by the
// block's 8 warps, their sums added in order.
template <typename T, int VB> __global__ void __launch_bounds__(256, 4) embed_join_kernel(SumArgs p) {
  using X = Vec<T, VB>;
  constexpr int LONG = 12, N = X::N;
  __shared__ long long long_item[8];
  __shared__ long long long_end[8];
  __shared__ float sums[8][32 * N];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto sum = [&](long long from, long long to, int col, float* acc) {  // the first-id sums of pieces from .. to-1
    for (long long r = from; r < to; r += 4) {
      float v[4][N];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r + k < to) load_part<N>(p.part + (size_t)(r + k) * 2 * p.E + col, v[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r + k < to) {
#pragma unroll
          for (int q = 0; q < N; ++q) acc[q] += v[k][q];
        }
    }
  };
  auto write = [&](unsigned id, int col, const float* acc) {
    X x;
#pragma unroll
    for (int q = 0; q < N; ++q) x.v[q] = from_f<T>(acc[q] * p.scale);
    store_vec<T, VB>((T*)p.dW + (size_t)id * p.E + col, x);
  };
  // a block's warps have neighbouring pieces and the same columns, so that the
  // column tiles of a long id go to different blocks
  const long long piece = blockIdx.x / p.coltiles * 8ll + warp;
  const int col = ((int)(blockIdx.x % p.coltiles) * 32 + lane) * N;
  if (lane == 0) long_item[warp] = -1;
  if (piece + 1 < p.pieces) {
    const long long i1 = (piece + 1) * p.piece;  // the next piece's first token
    const unsigned id = __ldg(p.key + i1 - 1), next = __ldg(p.key + i1);
    const unsigned prev = piece > 0 ? __ldg(p.key + piece * p.piece - 1) : 0xffffffffu;
    if (id < (unsigned)p.V && prev != id && next == id) {
      long long end = piece + 2;  // the id's last piece + 1
      for (bool more = true; more; end += 32) {
        const long long r = end + lane;
        const unsigned same = __ballot_sync(0xffffffffu, r < p.pieces && __ldg(p.key + r * p.piece) == id);
        if (same != 0xffffffffu) {
          end += __ffs(~same) - 1 - 32;
          more = false;
        }
      }
      if (end - piece > LONG) {
        if (lane == 0) {
          long_item[warp] = piece;
          long_end[warp] = end;
        }
      } else if (col < p.E) {
        float acc[N];
        load_part<N>(p.part + ((size_t)piece * 2 + 1) * p.E + col, acc);
        sum(piece + 1, end, col, acc);
        write(id, col, acc);
      }
    }
  }
  __syncthreads();
  for (int s = 0; s < 8; ++s) {
    if (long_item[s] < 0) continue;
    const long long pc = long_item[s], end = long_end[s];
    const int c = col;
    const long long share = (end - pc - 1 + 7) / 8, from = min(end, pc + 1 + warp * share), to = min(end, from + share);
    float acc[N];
#pragma unroll
    for (int q = 0; q < N; ++q) acc[q] = 0.0f;
    if (warp == 0 && c < p.E) load_part<N>(p.part + ((size_t)pc * 2 + 1) * p.E + c, acc);
    if (c < p.E) sum(from, to, c, acc);
#pragma unroll
    for (int q = 0; q < N; ++q) sums[warp][lane * N + q] = acc[q];
    __syncthreads();
    if (warp == 0 && c < p.E) {
      for (int k = 1; k < 8; ++k)
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] += sums[k][lane * N + q];
      write(__ldg(p.key + (pc + 1) * p.piece - 1), c, acc);
    }
    __syncthreads();
  }
}

// Few tokens: one launch. Every block sorts all of them (a bitonic network on
// (key, place) pairs, which differ, so the order is stable) and then writes
// its share of dW, a warp a row (or 1 / split of its columns): the sum of the
// row's tokens, or zeros. Up to FEW tokens, where the longest possible sum, all
// tokens of one id, costs about what the other path's launches do.
constexpr int FEW = 512;
template <typename T, typename I, int VB>
__global__ void __launch_bounds__(256) embed_few_kernel(int n, int V, int E, int split, const I* ids, long long pad, const T* dout,
                                                        float scale, T* dW, unsigned* status) {
  using X = Vec<T, VB>;
  constexpr int N = X::N;
  __shared__ unsigned long long s[FEW];
  int size = 1;
  while (size < n) size *= 2;
  bool range = false;
  for (int i = threadIdx.x; i < size; i += 256) {
    unsigned long long k = ~0ull;
    if (i < n) {
      const long long v = (long long)ids[i];
      const bool ok = v >= 0 && v < V;
      range |= !ok;
      if (ok && v != pad) k = (unsigned long long)v << 32 | (unsigned)i;
    }
    s[i] = k;
  }
  const int any = __syncthreads_or(range);
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = any ? STATUS_RANGE : STATUS_OK;
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      for (int t = threadIdx.x; t < size / 2; t += 256) {
        const int a = 2 * t - (t & (j - 1)), b = a + j;
        const unsigned long long x = s[a], y = s[b];
        if ((x > y) == ((a & k) == 0)) {
          s[a] = y;
          s[b] = x;
        }
      }
      __syncthreads();
    }
  const int lane = threadIdx.x & 31;
  for (long long w = blockIdx.x * 8 + (threadIdx.x >> 5); w < (long long)V * split; w += gridDim.x * 8) {
    const int v = (int)(w / split);
    int lo = 0, hi = n;  // the first token of id v
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if ((s[mid] >> 32) < (unsigned)v) lo = mid + 1;
      else hi = mid;
    }
    for (int col = ((int)(w % split) * 32 + lane) * N; col < E; col += split * 32 * N) {
      float acc[N];
#pragma unroll
      for (int q = 0; q < N; ++q) acc[q] = 0.0f;
      for (int i = lo; i < n && (s[i] >> 32) == (unsigned)v; i += 8) {
        X x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i + k < n && (s[i + k] >> 32) == (unsigned)v)
            x[k] = load_vec<T, VB>(dout + (size_t)(unsigned)s[i + k] * E + col);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i + k < n && (s[i + k] >> 32) == (unsigned)v) {
#pragma unroll
            for (int q = 0; q < N; ++q) acc[q] += to_f(x[k].v[q]);
          }
      }
      X x;
#pragma unroll
      for (int q = 0; q < N; ++q) x.v[q] = from_f<T>(acc[q] * scale);
      store_vec<T, VB>(dW + (size_t)v * E + col, x);
    }
  }
}

// ---- host ----------------------------------------------------------------------------
int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return RNN_OK;
  fprintf(stderr, "librnn_gb300: CUDA error: %s\n", cudaGetErrorString(e));
  return RNN_ECUDA;
}
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
constexpr int EMBED_E_MAX = 1 << 30;  // column numbers and strides stay within 32 bits
bool embed_ok(long long n, int V, int E, int dtype, int id_bytes) {
  return n >= 0 && n < (1ll << 31) && V >= 1 && E >= 1 && E <= EMBED_E_MAX && (dtype == RNN_F32 || dtype == RNN_BF16) &&
         (id_bytes == 4 || id_bytes == 8);
}

struct EmbedPlan {
  int passes, bits, tiles, piece;
  long long pieces;
  size_t hist, list, part, total;  // bytes; a list holds n words
};
EmbedPlan embed_plan(long long n, int V, int E) {
  EmbedPlan z{};
  z.total = 256;
  if (n <= FEW) return z;
  int bits = 0;
  while (((long long)V >> bits) > 0) ++bits;  // keys 0 .. V
  z.passes = (bits + DIGIT_MAX - 1) / DIGIT_MAX;
  z.bits = (bits + z.passes - 1) / z.passes;
  z.tiles = (int)((n + TILE - 1) / TILE);
  // 32 tokens a warp keep the partial sums' traffic low (two fp32 rows for 32
  // rows at most); fewer when the warps would not fill the GPU
  z.piece = PIECE_MAX;
  const long long cols = (E + 255) / 256;
  while (z.piece > 8 && n / z.piece * cols < 8 * device_sms()) z.piece /= 2;
  z.pieces = (n + z.piece - 1) / z.piece;
  z.hist = up256((((size_t)2 * z.tiles + 1) << z.bits) * sizeof(unsigned));  // two passes' counts, and the digits' totals
  z.list = up256((size_t)n * sizeof(unsigned));
  z.part = up256((size_t)z.pieces * 2 * E * sizeof(float));
  z.total = 256 + z.hist + 4 * z.list + z.part;
  return z;
}

template <typename T> int vec_bytes(int E) {
  const size_t row = (size_t)E * sizeof(T);
  return row % 16 == 0 ? 16 : row % 8 == 0 ? 8 : row % 4 == 0 ? 4 : 2;
}

template <typename T, typename I, int VB>
cudaError_t embed_fwd_launch(long long n, int V, int E, const void* ids, const void* W, float scale, void* out,
                             unsigned* status, cudaStream_t st) {
  const int nv = E / Vec<T, VB>::N;
  int lanes = 1;
  while (lanes < nv && lanes < 256) lanes *= 2;
  const long long per_block = 256 / lanes * 4;
  const long long blocks = (n + per_block - 1) / per_block, most = 16ll * device_sms();
  embed_fwd_kernel<T, I, VB><<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(
      n, V, E, lanes, (const I*)ids, (const T*)W, scale, (T*)out, status);
  note_launch();
  return cudaGetLastError();
}

template <typename T, typename I, int VB>
cudaError_t embed_bwd_launch(long long n, int V, int E, const void* ids, long long pad, const void* dout, float scale,
                             void* dW, char* ws, cudaStream_t st) {
  const EmbedPlan z = embed_plan(n, V, E);
  const int sms = device_sms();
  if (n <= FEW) {
    const int coltiles = (E + 32 * Vec<T, VB>::N - 1) / (32 * Vec<T, VB>::N), warps = 16 * sms;
    const int split = V >= warps ? 1 : warps / V < coltiles ? warps / V : coltiles;
    const long long want = ((long long)V * split + 7) / 8;
    const int blocks = want < 2 * sms ? (int)want : 2 * sms;
    embed_few_kernel<T, I, VB><<<blocks, 256, 0, st>>>((int)n, V, E, split, (const I*)ids, pad, (const T*)dout, scale, (T*)dW,
                                                       (unsigned*)ws);
    note_launch();
    return cudaGetLastError();
  }
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return e;
  SortArgs s{};
  s.n = n; s.pad = pad; s.V = V; s.tiles = z.tiles; s.bits = z.bits;
  s.ids = ids;
  s.status = (unsigned*)ws;
  unsigned* const counts = (unsigned*)(ws + 256);
  const size_t count_words = (size_t)z.tiles << z.bits;
  s.total = counts + 2 * count_words;
  unsigned* list[4];
  for (int k = 0; k < 4; ++k) list[k] = (unsigned*)(ws + 256 + z.hist + k * z.list);
  // The sort is a chain of short launches that leaves most of the GPU idle:
  // the blocks past its tiles clear dW meanwhile, a share in each launch.
  const size_t bytes = (size_t)V * E * sizeof(T), units = bytes / 16;
  const int launches = 2 * z.passes + 1;
  const size_t share = (units + launches - 1) / launches;
  if (bytes % 16) {
    e = cudaMemsetAsync((char*)dW + units * 16, 0, bytes % 16, st);
    if (e != cudaSuccess) return e;
  }
  const int smem = SORT_WARPS * (int)sizeof(unsigned) << z.bits;
  for (int pass = 0, launch = 0; pass < z.passes; ++pass) {
    const bool first = pass == 0;
    s.shift = pass * z.bits;
    s.kin = list[pass % 2 * 2];
    s.pin = list[pass % 2 * 2 + 1];
    s.kout = list[(pass + 1) % 2 * 2];
    s.pout = list[(pass + 1) % 2 * 2 + 1];
    auto clear = [&]() {
      const size_t at = share * launch < units ? share * launch : units;
      s.zero = (uint4*)dW + at;
      s.zeros = units - at < share ? units - at : share;
      ++launch;
      const size_t want = (s.zeros + 1023) / 1024;
      return (int)(want < (size_t)4 * sms ? want : (size_t)4 * sms);
    };
    s.hist = counts + pass % 2 * count_words;
    s.hist_next = pass + 1 < z.passes ? counts + (pass + 1) % 2 * count_words : nullptr;
    int more;
    if (first) {
      more = clear();
      sort_count_kernel<I><<<z.tiles + more, SORT_THREADS, smem / SORT_WARPS, st>>>(s);
      note_launch();
    }
    more = clear();
    sort_scan_kernel<<<((1 << z.bits) + SORT_WARPS - 1) / SORT_WARPS + more, SORT_THREADS, 0, st>>>(s);
    more = clear();
    const void* k = first ? (const void*)sort_scatter_kernel<I, true> : (const void*)sort_scatter_kernel<I, false>;
    e = set_smem_attr(k, smem);
    if (e != cudaSuccess) return e;
    if (first) sort_scatter_kernel<I, true><<<z.tiles + more, SORT_THREADS, smem, st>>>(s);
    else sort_scatter_kernel<I, false><<<z.tiles + more, SORT_THREADS, smem, st>>>(s);
    note_launch(2);
  }
  SumArgs a{};
  a.n = n; a.V = V; a.E = E; a.piece = z.piece; a.pieces = z.pieces;
  a.coltiles = (E + 32 * Vec<T, VB>::N - 1) / (32 * Vec<T, VB>::N);
  a.key = s.kout; a.pos = s.pout;
  a.dout = dout; a.scale = scale; a.dW = dW;
  a.part = (float*)(ws + 256 + z.hist + 4 * z.list);
  const unsigned blocks = (unsigned)((z.pieces * a.coltiles + 7) / 8);
  embed_sum_kernel<T, VB><<<blocks, 256, 0, st>>>(a);
  embed_join_kernel<T, VB><<<(unsigned)((z.pieces + 7) / 8 * a.coltiles), 256, 0, st>>>(a);
  note_launch(2);
  return cudaGetLastError();
}

template <typename T, typename I, bool BWD, typename... A> cudaError_t by_vector(long long n, int V, int E, A... a) {
  switch (vec_bytes<T>(E)) {
    case 16:
      if constexpr (BWD) return embed_bwd_launch<T, I, 16>(n, V, E, a...);
      else return embed_fwd_launch<T, I, 16>(n, V, E, a...);
    case 8:
      if constexpr (BWD) return embed_bwd_launch<T, I, 8>(n, V, E, a...);
      else return embed_fwd_launch<T, I, 8>(n, V, E, a...);
    case 4:
      if constexpr (BWD) return embed_bwd_launch<T, I, 4>(n, V, E, a...);
      else return embed_fwd_launch<T, I, 4>(n, V, E, a...);
  }
  if constexpr (sizeof(T) == 2) {
    if constexpr (BWD) return embed_bwd_launch<T, I, 2>(n, V, E, a...);
    else return embed_fwd_launch<T, I, 2>(n, V, E, a...);
  }
  return cudaErrorInvalidValue;  // rows of 4-byte elements are whole 4-byte vectors
}
template <bool BWD, typename... A> int embed_dispatch(int dtype, int id_bytes, long long n, int V, int E, A... a) {
  if (dtype == RNN_BF16)
    return cuda_status(id_bytes == 4 ? by_vector<__nv_bfloat16, int, BWD>(n, V, E, a...)
                                     : by_vector<__nv_bfloat16, long long, BWD>(n, V, E, a...));
  return cuda_status(id_bytes == 4 ? by_vector<float, int, BWD>(n, V, E, a...)
                                   : by_vector<float, long long, BWD>(n, V, E, a...));
}

}  // namespace
}  // namespace rnn

using namespace rnn;

extern "C" {

size_t rnn_embed_bwd_workspace_size(long long n, int V, int E) {
  return embed_ok(n, V, E, RNN_F32, 4) ? embed_plan(n, V, E).total : 0;
}

int rnn_embed_fwd(long long n, int V, int E, int dtype, int id_bytes, const void* ids, const void* W, float scale,
                  void* out, void* status, void* stream) {
  if (!embed_ok(n, V, E, dtype, id_bytes) || !W || (n > 0 && (!ids || !out))) return RNN_EINVAL;
  if (!al16(W) || !al16(out) || ((uintptr_t)status & 3u) || ((uintptr_t)ids & (id_bytes - 1))) return RNN_EINVAL;
  if (n == 0) return RNN_OK;
  return embed_dispatch<false>(dtype, id_bytes, n, V, E, ids, W, scale, out, (unsigned*)status, (cudaStream_t)stream);
}

int rnn_embed_bwd(long long n, int V, int E, int dtype, int id_bytes, const void* ids, long long padding_idx,
                  const void* dout, float scale, void* dW, void* workspace, size_t ws_bytes, void* stream) {
  if (!embed_ok(n, V, E, dtype, id_bytes) || !dW || !workspace || (n > 0 && (!ids || !dout))) return RNN_EINVAL;
  if (!al16(dW) || !al16(dout) || !al16(workspace) || ((uintptr_t)ids & (id_bytes - 1))) return RNN_EINVAL;
  if (ws_bytes < rnn_embed_bwd_workspace_size(n, V, E)) return RNN_ENOSPC;
  return embed_dispatch<true>(dtype, id_bytes, n, V, E, ids, padding_idx, dout, scale, dW, (char*)workspace,
                              (cudaStream_t)stream);
}

}  // extern "C"
