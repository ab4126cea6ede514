// Token embedding with scaling and its gradient by sorted tokens
// (include/rnn.h).
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
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

// ---- forward --------------------------------------------------------------------
// `lanes` lanes (a power of two) to a token, 16-byte vectors where the rows
// allow, ROWS tokens of a lane group in flight.
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
#pragma unroll
        for (int q = 0; q < X::N; ++q) x[r].v[q] = src[r] ? from_f<T>(to_f(x[r].v[q]) * scale) : from_f<T>(0.0f);
        store_vec<T, VB>(out + (size_t)(i0 + r) * E + (size_t)e * X::N, x[r]);
      }
    }
  }
}

// ---- gradient: sorting the tokens --------------------------------------------------
// A token's key is its id, or V (past every row) when it has no gradient. The
// tokens are sorted by key, equal keys in token order: least significant digit
// first, DIGIT_MAX bits at most a pass, each pass a count of the digits of
// every tile of TILE tokens, a scan of the counts in (digit, tile) order and a
// stable scatter. All counts are whole numbers, so nothing depends on timing.
constexpr int SORT_THREADS = 256, SORT_WARPS = SORT_THREADS / 32, SORT_ROUNDS = 16;
constexpr int TILE = SORT_THREADS * SORT_ROUNDS;
constexpr int DIGIT_MAX = 11;

struct SortArgs {
  long long n, pad;
  int V, tiles, shift, bits;
  const void* ids;            // first pass; then kin, pin
  const unsigned *kin, *pin;
  unsigned *kout, *pout;
  unsigned* hist;             // [1 << bits][tiles]
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

template <typename I, bool FIRST> __global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(SortArgs p) {
  if (zero_share(p, p.tiles)) return;
  extern __shared__ unsigned count[];
  const int bins = 1 << p.bits;
  for (int d = threadIdx.x; d < bins; d += SORT_THREADS) count[d] = 0;
  __syncthreads();
  const long long base = (long long)blockIdx.x * TILE;
#pragma unroll
  for (int r = 0; r < SORT_ROUNDS; ++r) {
    const long long i = base + r * SORT_THREADS + threadIdx.x;
    if (i < p.n) {
      const unsigned k = FIRST ? key_of((const I*)p.ids, i, p) : p.kin[i];
      atomicAdd(&count[k >> p.shift & (bins - 1)], 1u);
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += SORT_THREADS) p.hist[(size_t)d * p.tiles + blockIdx.x] = count[d];
}

// Exclusive sum of p.hist in place, one block.
__global__ void __launch_bounds__(1024) sort_scan_kernel(SortArgs p) {
  if (zero_share(p, 1)) return;
  __shared__ unsigned warp_sum[32];
  const size_t total = (size_t)p.tiles << p.bits;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned carry = 0;
  for (size_t base = 0; base < total; base += 4096) {
    const size_t at = base + threadIdx.x * 4;
    unsigned v[4], s = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = at + q < total ? p.hist[at + q] : 0;
      s += v[q];
    }
    unsigned inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    unsigned before = carry, all = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const unsigned t = warp_sum[w];
      if (w < warp) before += t;
      all += t;
    }
    unsigned x = before + inc - s;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (at + q < total) p.hist[at + q] = x;
      x += v[q];
    }
    carry += all;
    __syncthreads();
  }
}

template <typename I, bool FIRST> __global__ void __launch_bounds__(SORT_THREADS) sort_scatter_kernel(SortArgs p) {
  if (zero_share(p, p.tiles)) return;
  extern __shared__ unsigned place[];  // [SORT_WARPS][bins]: the warp's counts, then where its next key of a digit goes
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
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += SORT_THREADS) {
    unsigned at = p.hist[(size_t)d * p.tiles + blockIdx.x];
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

// A warp sums `piece` sorted tokens over 32 vectors of columns, in order. An
// id whose tokens all lie in the piece is written to dW; what belongs to an
// id that crosses the piece's ends goes to part.
template <typename T, int VB> __global__ void __launch_bounds__(256) embed_sum_kernel(SumArgs p) {
  using X = Vec<T, VB>;
  constexpr int AHEAD = 8;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long piece = w / p.coltiles;
  if (piece >= p.pieces) return;
  const int col = ((int)(w % p.coltiles) * 32 + lane) * X::N;
  const long long i0 = piece * p.piece;
  const int count = (int)min((long long)p.piece, p.n - i0);
  const T* dout = (const T*)p.dout;
  const unsigned none = 0xffffffffu;
  const unsigned prev = i0 > 0 ? __ldg(p.key + i0 - 1) : none;
  const unsigned next = i0 + count < p.n ? __ldg(p.key + i0 + count) : none;
  const bool on = col < p.E;
  float acc[X::N];
#pragma unroll
  for (int q = 0; q < X::N; ++q) acc[q] = 0.0f;
  unsigned cur = none;
  auto flush = [&](bool last) {
    if (cur == none || cur >= (unsigned)p.V || !on) return;
    const bool head = cur == prev, tail = last && cur == next;
    if (!head && !tail) {
      X x;
#pragma unroll
      for (int q = 0; q < X::N; ++q) x.v[q] = from_f<T>(acc[q] * p.scale);
      store_vec<T, VB>((T*)p.dW + (size_t)cur * p.E + col, x);
    } else {
      float* out = p.part + ((size_t)piece * 2 + (head ? 0 : 1)) * p.E + col;
#pragma unroll
      for (int q = 0; q < X::N; ++q) out[q] = acc[q];
    }
  };
  for (int b = 0; b < count; b += 32) {
    const int m = min(32, count - b);
    const unsigned k32 = lane < m ? __ldg(p.key + i0 + b + lane) : none;
    const unsigned s32 = lane < m ? __ldg(p.pos + i0 + b + lane) : 0;
    for (int j0 = 0; j0 < m; j0 += AHEAD) {
      X x[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const unsigned k = __shfl_sync(0xffffffffu, k32, j0 + j), s = __shfl_sync(0xffffffffu, s32, j0 + j);
        if (j0 + j < m && k < (unsigned)p.V && on) x[j] = load_vec<T, VB>(dout + (size_t)s * p.E + col);
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (j0 + j >= m) break;
        const unsigned k = __shfl_sync(0xffffffffu, k32, j0 + j);
        if (k != cur) {
          flush(false);
          cur = k;
#pragma unroll
          for (int q = 0; q < X::N; ++q) acc[q] = 0.0f;
        }
        if (k < (unsigned)p.V && on) {
#pragma unroll
          for (int q = 0; q < X::N; ++q) acc[q] += to_f(x[j].v[q]);
        }
      }
    }
  }
  flush(true);
}

// The ids that cross pieces: a warp per piece in which such an id begins, over
// 32 vectors of columns, adds the pieces' sums in order. An id over more than
// LONG pieces is shared by the block's 8 warps, their sums added in order.
template <typename T, int VB> __global__ void __launch_bounds__(256) embed_join_kernel(SumArgs p) {
  using X = Vec<T, VB>;
  constexpr int LONG = 32, N = X::N;
  __shared__ long long long_item[8];
  __shared__ long long long_end[8];
  __shared__ float sums[8][32 * N];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto sum = [&](long long from, long long to, int col, float* acc) {  // the first-id sums of pieces from .. to-1
    long long r = from;
    for (; r + 4 <= to; r += 4) {
      float v[4][N];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < N; ++q) v[k][q] = p.part[(size_t)(r + k) * 2 * p.E + col + q];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] += v[k][q];
    }
    for (; r < to; ++r)
#pragma unroll
      for (int q = 0; q < N; ++q) acc[q] += p.part[(size_t)r * 2 * p.E + col + q];
  };
  auto write = [&](unsigned id, int col, const float* acc) {
    X x;
#pragma unroll
    for (int q = 0; q < N; ++q) x.v[q] = from_f<T>(acc[q] * p.scale);
    store_vec<T, VB>((T*)p.dW + (size_t)id * p.E + col, x);
  };
  const long long w = (long long)blockIdx.x * 8 + warp;
  const long long piece = w / p.coltiles;
  const int col = ((int)(w % p.coltiles) * 32 + lane) * N;
  if (lane == 0) long_item[warp] = -1;
  if (piece + 1 < p.pieces) {
    const long long i1 = (piece + 1) * p.piece;  // the next piece's first token
    const unsigned id = __ldg(p.key + i1 - 1);
    const bool begins = piece == 0 || __ldg(p.key + piece * p.piece - 1) != id;
    if (id < (unsigned)p.V && begins && __ldg(p.key + i1) == id) {
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
          long_item[warp] = w;
          long_end[warp] = end;
        }
      } else if (col < p.E) {
        float acc[N];
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] = p.part[((size_t)piece * 2 + 1) * p.E + col + q];
        sum(piece + 1, end, col, acc);
        write(id, col, acc);
      }
    }
  }
  __syncthreads();
  for (int s = 0; s < 8; ++s) {
    if (long_item[s] < 0) continue;
    const long long pc = long_item[s] / p.coltiles, end = long_end[s];
    const int c = ((int)(long_item[s] % p.coltiles) * 32 + lane) * N;
    const long long share = (end - pc - 1 + 7) / 8, from = min(end, pc + 1 + warp * share), to = min(end, from + share);
    float acc[N];
#pragma unroll
    for (int q = 0; q < N; ++q) acc[q] = warp == 0 && c < p.E ? p.part[((size_t)pc * 2 + 1) * p.E + c + q] : 0.0f;
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
bool embed_ok(long long n, int V, int E, int dtype, int id_bytes) {
  return n >= 0 && n < (1ll << 31) && V >= 1 && E >= 1 && (dtype == RNN_F32 || dtype == RNN_BF16) &&
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
  // 64 tokens a warp keep the partial sums' traffic low; fewer when the warps
  // would not fill the GPU
  z.piece = 64;
  const long long cols = (E + 255) / 256;
  while (z.piece > 8 && n / z.piece * cols < 8 * device_sms()) z.piece /= 2;
  z.pieces = (n + z.piece - 1) / z.piece;
  z.hist = up256(((size_t)z.tiles << z.bits) * sizeof(unsigned));
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
  const int nv = E * (int)sizeof(T) / VB;
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
  s.hist = (unsigned*)(ws + 256);
  unsigned* list[4];
  for (int k = 0; k < 4; ++k) list[k] = (unsigned*)(ws + 256 + z.hist + k * z.list);
  // The sort is a chain of short launches that leaves most of the GPU idle:
  // the blocks past its tiles clear dW meanwhile, a share in each launch.
  const size_t bytes = (size_t)V * E * sizeof(T), units = bytes / 16;
  const int launches = 3 * z.passes;
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
    int more = clear();
    if (first) sort_count_kernel<I, true><<<z.tiles + more, SORT_THREADS, smem / SORT_WARPS, st>>>(s);
    else sort_count_kernel<I, false><<<z.tiles + more, SORT_THREADS, smem / SORT_WARPS, st>>>(s);
    more = clear();
    sort_scan_kernel<<<1 + (more + 3) / 4, 1024, 0, st>>>(s);
    more = clear();
    const void* k = first ? (const void*)sort_scatter_kernel<I, true> : (const void*)sort_scatter_kernel<I, false>;
    e = set_smem_attr(k, smem);
    if (e != cudaSuccess) return e;
    if (first) sort_scatter_kernel<I, true><<<z.tiles + more, SORT_THREADS, smem, st>>>(s);
    else sort_scatter_kernel<I, false><<<z.tiles + more, SORT_THREADS, smem, st>>>(s);
    note_launch(3);
  }
  SumArgs a{};
  a.n = n; a.V = V; a.E = E; a.piece = z.piece; a.pieces = z.pieces;
  a.coltiles = (E + 32 * Vec<T, VB>::N - 1) / (32 * Vec<T, VB>::N);
  a.key = s.kout; a.pos = s.pout;
  a.dout = dout; a.scale = scale; a.dW = dW;
  a.part = (float*)(ws + 256 + z.hist + 4 * z.list);
  const unsigned blocks = (unsigned)((z.pieces * a.coltiles + 7) / 8);
  embed_sum_kernel<T, VB><<<blocks, 256, 0, st>>>(a);
  embed_join_kernel<T, VB><<<blocks, 256, 0, st>>>(a);
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
