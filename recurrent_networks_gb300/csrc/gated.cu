// The gated linear scan: forward, backward and the single-token step, and
// their C entry points (include/rnn.h).
#include <limits.h>
#include <stdio.h>

#include "gated.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rnn.h"

namespace rnn {
namespace {

// Work item: GATED_CHUNK steps of 128 bytes of channels (64 bf16, 32 fp32) of
// one batch row, one CTA. Each of the 8 warps holds 16 consecutive steps, a
// lane 4 bytes of channels. The recurrence is affine in its state, so a warp
// first folds its steps into one map c -> P c + H, the CTA folds the warps'
// maps, and the state that enters the chunk comes from the chunks before it:
// chunks are grouped by `span`; the last chunk of a group publishes the state
// after it, every other chunk its own map as soon as it has it, and a chunk
// starts from the state before its group and applies the maps of the group's
// chunks before it, in their order. The order of the sums is thus fixed, the
// same for any grouping and any batch, and the chain through the chunks has
// one hop per group.
// Published values are 8-byte words (fp32, tag) that are written and read
// whole, so a reader polls the value itself: no fence, and one round trip.
// CTAs stay and take item after item from a counter, in chunk order and only
// when the last one is through its wait, so whatever an item waits for is
// being worked on, however few of the CTAs are running.
constexpr int WARPS = 8, STEPS = GATED_CHUNK / WARPS, THREADS = WARPS * 32;
constexpr int MAX_SPAN = 3;  // log2

struct GatedArgs {
  int B, T, C, chunks;  // C = N D channels
  int tiles_c;          // channel tiles per batch row
  int width;            // channels of a tile: a full row of lanes, or 28 lanes' (see fetch_rows)
  int span;             // log2 of the chunks per group
  int solo;  // one chunk, all CTAs at once: no waits, so block 0 clears the status word itself
  const void* Wx;
  const void* bias;
  const float* s0;
  const unsigned char* reset;
  const int* lengths;
  void* h;
  float* last;
  float* carry;              // [B][chunks][C]: the state before every chunk (the tape)
  signed char* q;            // 8-bit pre-activations: written by the forward, read by the backward
  unsigned char* qs;
  const void* dh;
  const float* dlast;
  void* dWx;
  float* ds0;
  // db, by db_mode: 0 none; 1 each item's sums to dbp [B chunks][G][C], added by
  // a launch of their own; 2 the last item of a channel tile to finish adds
  // them, in the items' order; 3 a CTA has all items of a channel tile
  int db_mode;
  float* dbp;
  void* db;
  unsigned* done;            // [tiles_c], zeroed (mode 2)
  unsigned long long* states;  // [groups, or 2 in turn][tiles][N][32]: the state (or its gradient) that enters a group
  ulonglong2* maps;            // [chunks][tiles][N][32]: the chunks' maps (P, H)
  unsigned* status;
  unsigned* ticket;
  unsigned long long wait_limit_ns;
  // fault injection (rnn_debug_inject_wait): at this chunk (in processing order)
  // of the first tile a wait for a word that nothing writes; -1: off
  int inject_chunk;
  unsigned long long inject_limit_ns;
};

__device__ __forceinline__ int clamp_len(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// Factors of maps are products of sigmoids, so not negative, and a NaN that a
// product or a sum gives is 0x7fffffff: the sign bit is free to mark a reset
// among their steps (-0, or with a NaN among them 0xffffffff). A reset drops what
// came before even where that is an infinity or NaN; a factor that merely
// underflowed to 0 leaves it non-finite.
constexpr unsigned RESET = 0x80000000u;
__device__ __forceinline__ float affine(float f, float x, float u) {
  return (int)__float_as_uint(f) < 0 ? u : fmaf(f, x, u);
}
__device__ __forceinline__ float factor(float a, float b) {
  return __uint_as_float(__float_as_uint(a * b) | ((__float_as_uint(a) | __float_as_uint(b)) & RESET));
}
template <int N> __device__ __forceinline__ FV<N> factor(const FV<N>& a, const FV<N>& b) {
  FV<N> r;
#pragma unroll
  for (int v = 0; v < N; ++v) r.v[v] = factor(a.v[v], b.v[v]);
  return r;
}
template <int N> __device__ __forceinline__ FV<N> affine(const FV<N>& f, const FV<N>& x, const FV<N>& u) {
  FV<N> r;
#pragma unroll
  for (int v = 0; v < N; ++v) r.v[v] = affine(f.v[v], x.v[v], u.v[v]);
  return r;
}
template <int N> __device__ __forceinline__ FV<N> select(bool on, const FV<N>& a, const FV<N>& b) {
  FV<N> r;
#pragma unroll
  for (int v = 0; v < N; ++v) r.v[v] = on ? a.v[v] : b.v[v];
  return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"((uint64_t)map),
               "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// The channels of a lane: 4 bytes of the storage type.
template <typename T> struct Lane;
template <> struct Lane<float> {
  static constexpr int N = 1;
  __device__ static FV<1> unpack(uint32_t v) { return {{__uint_as_float(v)}}; }
  __device__ static uint32_t pack(const FV<1>& x) { return __float_as_uint(x.v[0]); }
};
template <> struct Lane<__nv_bfloat16> {
  static constexpr int N = 2;
  __device__ static FV<2> unpack(uint32_t v) { return {{__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)}}; }
  __device__ static uint32_t pack(const FV<2>& x) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.v[0], x.v[1]);
    return *(const uint32_t*)&h;
  }
};
// N signed bytes as fp32, without the conversion unit: a byte plus 128 in the
// low bits of 2^23 is 2^23 + 128 + q.
__device__ __forceinline__ FV<2> bytes_f(uint32_t w, FV<2>*) {
  w ^= 0x8080u;
  const FV<2> m = {{__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650)), __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7651))}};
  return add(m, splat<2>(-8388736.0f));
}
__device__ __forceinline__ FV<1> bytes_f(uint32_t w, FV<1>*) { return {{(float)(signed char)w}}; }

// A lane's channels at p (n of them inside the row: 0 .. N), and back. `wide`:
// the row starts on 4 bytes.
template <typename T> __device__ __forceinline__ uint32_t load_lane(const T* p, int n, bool wide) {
  if (n <= 0) return 0;
  if (sizeof(T) == 4 || (wide && n == 2)) return __ldg((const uint32_t*)p);
  const unsigned short* q = (const unsigned short*)p;
  return (uint32_t)__ldg(q) | (n == 2 ? (uint32_t)__ldg(q + 1) << 16 : 0u);
}
template <typename T> __device__ __forceinline__ void store_lane(T* p, uint32_t v, int n, bool wide) {
  if (n <= 0) return;
  if (sizeof(T) == 4 || (wide && n == 2)) {
    *(uint32_t*)p = v;
    return;
  }
  unsigned short* q = (unsigned short*)p;
  q[0] = (unsigned short)v;
  if (n == 2) q[1] = (unsigned short)(v >> 16);
}

// The item of this CTA and where it lies.
struct Item {
  int k, tile, b, ch, n, t0, len;  // ch: the lane's first channel, n: how many of its channels exist; t0: the warp's first step
  int ct;                          // the tile's first channel
  int live;                        // the warp's steps that exist
  unsigned rst;                    // bit j: reset at the warp's step j
  bool plain;                      // every step exists, none is a reset
};
// Thread 0 takes an item (the first one: from == blockIdx.x without a counter
// when there is one item a CTA) and works out its place for all, the divisions
// once; x < 0: no more items.
template <bool REVERSE> __device__ __forceinline__ int4 place_of(const GatedArgs& p, unsigned id) {
  const unsigned tiles = (unsigned)p.B * p.tiles_c, k = id / tiles, tile = id % tiles, b = tile / p.tiles_c;
  if (k >= (unsigned)p.chunks) return make_int4(-1, 0, 0, 0);
  return make_int4(REVERSE ? p.chunks - 1 - (int)k : (int)k, (int)tile, (int)b, clamp_len(p.lengths, b, p.T));
}
template <int N> __device__ __forceinline__ Item item_of(const GatedArgs& p, const int4& s) {
  Item it;
  it.k = s.x;
  it.tile = s.y;
  it.b = s.z;
  it.len = s.w;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  it.ct = (it.tile - it.b * p.tiles_c) * p.width;
  it.ch = it.ct + lane * N;
  it.n = min(max(min(p.C, it.ct + p.width) - it.ch, 0), N);
  it.t0 = it.k * GATED_CHUNK + warp * STEPS;
  it.live = min(max(it.len - it.t0, 0), STEPS);
  it.rst = 0;
  if (p.reset) {
    bool r = false;
    if (lane < it.live) r = p.reset[(size_t)it.b * p.T + it.t0 + lane] != 0;
    it.rst = __ballot_sync(0xffffffffu, r);
  }
  it.plain = it.live == STEPS && it.rst == 0;
  return it;
}

// (value, tag) words; the tag is the place of the group or chunk (never 0, the
// cleared value). Relaxed accesses at gpu scope: each 8-byte word is read and
// written whole, and nothing else is ordered by it.
__device__ __forceinline__ unsigned long long word_of(float v, unsigned tag) {
  return (unsigned long long)tag << 32 | __float_as_uint(v);
}
__device__ __forceinline__ float value_of(unsigned long long w) { return __uint_as_float((unsigned)w); }
__device__ __forceinline__ bool is_set(unsigned long long w, unsigned tag) { return (unsigned)(w >> 32) == tag; }
__device__ __forceinline__ unsigned long long ld_word(const unsigned long long* p) {
  unsigned long long w;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(p) : "memory");
  return w;
}
__device__ __forceinline__ void st_word(unsigned long long* p, unsigned long long w) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(w) : "memory");
}

// An affine map x -> P x + H, and first `a`, then `b`.
struct Map {
  float P, H;
};
__device__ __forceinline__ Map then(const Map& a, const Map& b) { return {factor(a.P, b.P), affine(b.P, a.H, b.H)}; }

// How a CTA passes the state through the chunks of a tile; REVERSE: the
// processing order descends. All threads take part, Q neighbouring lanes to a
// channel slot (v, lane): a lane folds M of the warps' maps, scans over the Q
// lanes give what is done to the state before each warp and by the whole
// chunk. (One warp that folded the warps' maps one after the other, with the
// rest of the CTA idle, cost 25 of 247 us at B=32 T=4096 C=1024.)
template <int N, bool REVERSE> struct Chain {
  static constexpr int Q = THREADS / (32 * N), M = WARPS / Q;
  static constexpr int ROW = 32 * N + 2, EROW = 32 * N + 4;  // row lengths that spread the Q lanes over the banks
  static constexpr int RUN = ((1 << MAX_SPAN) + Q - 1) / Q;   // chunks of a group to a lane, at most
  static constexpr unsigned ALL = 0xffffffffu;
  const GatedArgs& p;
  const Item& it;
  bool& failed;
  int o, first, group;  // this chunk's and its group's first chunk's place in processing order, the group's place
  int c, q, ch;         // the slot, the lane's part of it, the slot's channel
  float x;              // the state before the first chunk, then the state that enters the chunk
  unsigned long long early;
  Map mine[M], before, whole;  // the lane's maps, what comes before them, the chunk's
  __device__ __forceinline__ Chain(const GatedArgs& p, const Item& it, bool& failed) : p(p), it(it), failed(failed) {
    o = REVERSE ? p.chunks - 1 - it.k : it.k;
    group = o >> p.span;
    first = group << p.span;
    c = threadIdx.x / Q;
    q = threadIdx.x % Q;
    ch = c % 32 * N < p.width ? it.ct + c % 32 * N + c / 32 : p.C;  // (p.C: a slot without a channel)
  }
  __device__ __forceinline__ size_t at(int i) const {
    return ((size_t)i * ((unsigned)p.B * p.tiles_c) + it.tile) * N * 32 + c;
  }
  // Where the state that enters a group lies. Without groups of several chunks
  // two places in turn do: group g + 2 is written after chunk g + 1 had its
  // state, from chunk g, all of whose lanes had theirs.
  __device__ __forceinline__ unsigned long long* state(int g) const { return p.states + at(p.span ? g : g & 1); }
  // At the start: the state before the first chunk, or the one that enters the
  // group; where it is there already (the usual case with many tiles) the
  // round trip runs beside the tile's load.
  __device__ __forceinline__ void ask(const float* init) {
    x = 0.0f;
    early = 0;
    if (group > 0) early = ld_word(state(group));
    else if (init && ch < p.C) x = __ldg(init + (size_t)it.b * p.C + ch);
  }
  // The warp waits until `get` holds in all lanes, for at most limit_ns. When
  // that runs out the state is whatever was read: the status word tells, this
  // warp's later waits return at once, and the items still go to their end,
  // publishing what they have, so that nobody waits for them in turn.
  template <typename F> __device__ __forceinline__ void wait(F&& get, bool& lost, unsigned long long limit_ns) {
    bool ok = lost || get();
    if (__all_sync(ALL, ok)) return;
    const uint64_t t0 = globaltimer_ns();
    do {
      if (!ok) ok = get();
      if (__any_sync(ALL, globaltimer_ns() - t0 > limit_ns)) {
        atomicOr(p.status, STATUS_TIMEOUT);
        lost = true;
        return;
      }
    } while (!__all_sync(ALL, ok));
  }
  template <typename F> __device__ __forceinline__ void wait(F&& get) { wait(get, failed, p.wait_limit_ns); }
  // Over the Q lanes of a slot, in their order: everything up to and including
  // the lane's m.
  static __device__ __forceinline__ Map scan(Map m, int q) {
#pragma unroll
    for (int d = 1; d < Q; d *= 2) {
      const Map l = {__shfl_up_sync(ALL, m.P, d, Q), __shfl_up_sync(ALL, m.H, d, Q)};
      if (q >= d) m = then(l, m);
    }
    return m;
  }
  static __device__ __forceinline__ Map last_of(const Map& m) {
    return {__shfl_sync(ALL, m.P, Q - 1, Q), __shfl_sync(ALL, m.H, Q - 1, Q)};
  }
  static __device__ __forceinline__ Map shifted(const Map& m, int q) {
    Map l = {__shfl_up_sync(ALL, m.P, 1, Q), __shfl_up_sync(ALL, m.H, 1, Q)};
    if (q == 0) l = {1.0f, 0.0f};
    return l;
  }
  __device__ __forceinline__ int warp_of(int i) const { return REVERSE ? WARPS - 1 - (q * M + i) : q * M + i; }
  // With the lane's maps in `mine`: scans them and publishes the chunk's map
  // for the group's later chunks.
  __device__ __forceinline__ void publish() {
    Map m = mine[0];
#pragma unroll
    for (int i = 1; i < M; ++i) m = then(m, mine[i]);
    m = scan(m, q);
    before = shifted(m, q);
    whole = last_of(m);
    if (o + 1 == first + (1 << p.span) || o + 1 == p.chunks || q != 0) return;
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p.maps + at(o)), "l"(word_of(whole.P, o + 1)),
                 "l"(word_of(whole.H, o + 1))
                 : "memory");
  }
  // Makes x the state that enters the chunk, publishes the one that leaves a
  // group, and hands every warp its own: enter [WARPS][EROW].
  __device__ __forceinline__ void pass(float* enter) {
    if (o == p.inject_chunk && it.tile == 0) {
      bool lost = false;  // (the chunks' own waits are left untouched)
      wait([&]() { return ld_word((const unsigned long long*)p.ticket + 1) != 0; }, lost, p.inject_limit_ns);
    }
    // the group's chunks before this one, a run of them a lane
    const int run = (o - first + Q - 1) / Q, from = first + q * run;
    Map r[RUN];
    if (o > first) {
      if (group > 0 && !is_set(early, group)) early = ld_word(state(group));  // beside the maps' round trip
      ulonglong2 m[RUN];
      wait([&]() {
        bool all = true;
#pragma unroll
        for (int i = 0; i < RUN; ++i)
          if (i < run && from + i < o)
            asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];"
                         : "=l"(m[i].x), "=l"(m[i].y)
                         : "l"(p.maps + at(from + i))
                         : "memory");
#pragma unroll
        for (int i = 0; i < RUN; ++i)
          if (i < run && from + i < o) all &= is_set(m[i].x, from + i + 1) && is_set(m[i].y, from + i + 1);
        return all;
      });
#pragma unroll
      for (int i = 0; i < RUN; ++i) r[i] = {value_of(m[i].x), value_of(m[i].y)};
    }
    if (group > 0) {
      wait([&]() {
        if (!is_set(early, group)) early = ld_word(state(group));
        return is_set(early, group);
      });
      x = value_of(early);
    }
    if (o > first) {
      // one chunk's map after the other, as if the state had come from the
      // chunk before: the bits do not depend on the groups
      for (int l = 0; l * run < o - first; ++l) {
        float y = x;
#pragma unroll
        for (int i = 0; i < RUN; ++i)
          if (i < run && from + i < o) y = affine(r[i].P, y, r[i].H);
        x = __shfl_sync(ALL, y, l, Q);
      }
    }
    if (o + 1 == first + (1 << p.span) && o + 1 < p.chunks && q == 0)
      st_word(state(group + 1), word_of(affine(whole.P, x, whole.H), group + 1));
    float e = affine(before.P, x, before.H);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      enter[warp_of(i) * EROW + c] = e;
      e = affine(mine[i].P, e, mine[i].H);
    }
  }
  // Lane 0 of a slot: the value x at row r of a [rows][C] array.
  __device__ __forceinline__ void store(float* a, size_t r, float v) const {
    if (q == 0 && ch < p.C) a[r * p.C + ch] = v;
  }
};

// A warp's steps of a tile by the lanes' own asynchronous copies, for rows that
// TMA cannot take (or must not, see `solo`). Rows that are no multiple of 16
// bytes start anywhere in one; the tile then has 28 lanes' channels, 112 bytes,
// which lie in the 8 aligned 16-byte pieces that a row's 128-byte place holds.
// They are copied as they lie, 4 rows an instruction, and read with the row's
// shift (Rows). (4-byte copies to the final places took 20 of 51 us forward at
// B=4 T=2048 C=998.) Rows past `live` are not read, nor anything past the end.
template <typename T, int ROWS>
__device__ __forceinline__ void fetch_rows(const GatedArgs& p, const Item& it, const T* src, uint32_t* dst) {
  const int lane = threadIdx.x & 31, rows = it.live * ROWS, piece = lane & 7;
  const int bytes = max(min(p.C - it.ct, p.width), 0) * (int)sizeof(T);
  const size_t all = (size_t)p.B * p.T * ROWS * p.C * sizeof(T);
  const uint32_t to = smem_u32(dst) + piece * 16;
  size_t at = ((((size_t)it.b * p.T + it.t0) * ROWS + (lane >> 3)) * p.C + it.ct) * sizeof(T);
  const size_t step = (size_t)4 * p.C * sizeof(T);
#pragma unroll 4
  for (int r = lane >> 3; r < rows; r += 4, at += step) {
    const size_t from = (at & ~(size_t)15) + piece * 16;
    if (from < at + bytes)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + r * 128), "l"((const char*)src + from),
                   "r"((int)(all - from < 16 ? all - from : 16))
                   : "memory");
  }
}
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();  // the lanes read one another's pieces
}
// The 4-byte words of a lane in a warp's rows of a tile.
template <typename T, int ROWS, bool TMA> struct Rows {
  const uint32_t* at;  // the lane's word of the first row
  unsigned e0, step;   // of a row: elements from the 16-byte boundary, mod 16 bytes; of the next one more
  __device__ __forceinline__ Rows(const GatedArgs& p, const Item& it, const uint32_t* tile) : at(tile + (threadIdx.x & 31)) {
    if (!TMA) {
      e0 = (unsigned)(((size_t)it.b * p.T + it.t0) * ROWS * p.C + it.ct);
      step = (unsigned)p.C;
    }
  }
  __device__ __forceinline__ uint32_t operator()(int r) const {
    if (TMA) return at[r * 32];
    const unsigned e = e0 + r * step;
    if (sizeof(T) == 4) return at[r * 32 + (e & 3)];
    const uint32_t* w = at + r * 32 + ((e & 7) >> 1);
    return e & 1 ? w[0] >> 16 | w[1] << 16 : w[0];
  }
};

// The TMA loads of a warp (its tile, asked for by lane 0) and of the CTA (the
// biases, by thread 0), as every thread follows them: `phase` has the parity of
// each barrier's next load. Once a wait has run out (`failed`) no more are asked
// for, so that no barrier's phases get mixed up, and before the CTA leaves it
// waits (again with the limit) for what is in flight: nothing may be written to
// shared memory that is another CTA's by then.
struct Loads {
  static constexpr unsigned TILE = 1, BIAS = 2;
  unsigned phase = 0;
  bool& failed;
  __device__ __forceinline__ explicit Loads(bool& failed) : failed(failed) {}
  template <unsigned WHICH> __device__ __forceinline__ bool ask(bool wanted) {
    wanted = wanted && !failed;
    if (wanted) phase ^= WHICH;
    return wanted;
  }
  template <unsigned WHICH> __device__ __forceinline__ unsigned last() const { return phase & WHICH ? 0 : 1; }
  template <unsigned WHICH> __device__ __forceinline__ void wait(const GatedArgs& p, uint32_t bar) {
    mbar_wait_bounded<false>(bar, last<WHICH>(), p.wait_limit_ns, p.status, failed);
  }
  // (A barrier that was never asked counts as past the phase before its first.)
  __device__ __forceinline__ void leave(const GatedArgs& p, uint32_t bar, uint32_t bias_bar) {
    if (!failed || threadIdx.x % 32 != 0) return;
    bool late = false;
    mbar_wait_bounded<false>(bar, last<TILE>(), p.wait_limit_ns, nullptr, late);
    late = false;
    if (threadIdx.x == 0) mbar_wait_bounded<false>(bias_bar, last<BIAS>(), p.wait_limit_ns, nullptr, late);
  }
};

// A lane's biases, scaled as the gates want them: from the copy beside the tile
// [G][32] (TMA), or from memory.
template <typename T, int FN, int N, bool TMA>
__device__ __forceinline__ void load_bias(const GatedArgs& p, const Item& it, const uint32_t* copy, FV<N>* bias) {
  constexpr int G = gated_gates(FN);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    uint32_t w = 0;
    if (p.bias) w = TMA ? copy[g * 32 + (threadIdx.x & 31)] : load_lane((const T*)p.bias + (size_t)g * p.C + it.ch, it.n, p.C % 2 == 0);
    bias[g] = mul(Lane<T>::unpack(w), splat<N>(mul_of<FN, N>(g)));
  }
}
// raw pre-activation -> gate value (see mul_of)
template <int FN, int N> __device__ __forceinline__ FV<N> gate(int g, const FV<N>& a, const FV<N>& bias) {
  return mul_of<FN, N>(g) == 1.0f ? add(a, bias) : fma(a, splat<N>(mul_of<FN, N>(g)), bias);
}

template <bool V> struct Flag { static constexpr bool value = V; };
// Steps whose warp has all of them and no reset run without a test per step.
template <typename F> __device__ __forceinline__ void by_mask(const Item& it, F&& f) {
  if (it.plain) f(Flag<false>());
  else f(Flag<true>());
}

// CTAs an SM holds: what the tiles (64 KB linear, 32 KB coupled; the backward's
// and the 8-bit copies' more) and the registers of f and u allow. Measured with
// one more or less: coupled forward 146 us with 4, 163 with 3 (B=32 T=4096
// C=1024 bf16); coupled backward bf16 311 with 2, 404 with 3 (spills), fp32 82
// and 74 (B=16 T=2048 C=512); linear forward 247 with 3, 258 with 2.
template <typename T, int FN, bool Q8> __host__ __device__ constexpr int ctas_per_sm(bool bwd) {
  if (bwd) return FN == GATED_COUPLED && !Q8 && sizeof(T) == 4 ? 3 : 2;
  return Q8 ? 2 : FN == GATED_COUPLED ? 4 : 3;
}

// Forward. Reads Wx once and writes h once: 10 bytes a channel and step for
// linear bf16, so memory bounds it; the arithmetic (three sigmoids, about 24
// issue slots and 6 special-function operations) has to hide behind that. The
// tile is asked for by TMA, a box of 16 steps a warp; pass 1 turns it into f and
// u and the warp's map; the state comes in (Chain); pass 2 runs the recurrence
// and lays h where the tile was, from where one TMA store a warp takes it.
// Without the 8-bit copy u waits in the tile's place of i and g (coupled: f and
// g), which are not read again, so that f alone stays in registers and three
// tiles fit an SM. Measured: B=32 T=4096 C=1024 linear bf16 216 us, 6.22 TB/s,
// 93 % of the copy bandwidth (loads and stores alone, without arithmetic or
// state, 201 us); B=1 T=65537 C=768 120 us, where each tile's chunks wait for one
// another (loads and stores alone 80 us); with the 8-bit copy, which takes the
// shared memory of the third tile, B=8 T=4099 C=1024 120 us, 4.0 TB/s.
template <typename T, int FN, bool Q8, bool TMA>
__global__ void __launch_bounds__(THREADS, (ctas_per_sm<T, FN, Q8>(false)))
    gated_fwd_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap hmap,
                     const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap bmap, GatedArgs p) {
  constexpr int G = gated_gates(FN), N = Lane<T>::N;
  constexpr bool TMAQ = Q8 && TMA;  // (the rows of bytes are 16-byte multiples then, too)
  constexpr int U0 = FN == GATED_LINEAR ? 0 : 1, U1 = FN == GATED_LINEAR ? 2 : 0;  // rows that hold u of channel 0, 1
  extern __shared__ __align__(128) unsigned char smem[];
  uint32_t* tile = (uint32_t*)smem;                                   // [WARPS][STEPS][G][32]
  using Ch = Chain<N, false>;
  uint32_t* bcopy = tile + WARPS * STEPS * G * 32;                    // [G][32]
  float2* maps = (float2*)(bcopy + G * 32);                           // [WARPS][ROW]: slot v * 32 + lane
  float* enter = (float*)(maps + WARPS * Ch::ROW);                    // [WARPS][EROW]: the states that enter the warps
  uint32_t* tops = (uint32_t*)(enter + WARPS * Ch::EROW);             // Q8: [WARPS][G][32]
  unsigned char* qtile = (unsigned char*)(tops + (Q8 ? WARPS * G * 32 : 0));  // Q8: [WARPS][STEPS][G][32 N]
  unsigned long long* bars = (unsigned long long*)(qtile + (Q8 ? WARPS * STEPS * G * 32 * N : 0));  // [WARPS]; the biases'
  int4* shared = (int4*)(bars + WARPS + 2);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bar = smem_u32(bars + warp);
  const uint32_t bbar = smem_u32(bars + WARPS);
  if (TMA && lane == 0) {
    mbar_init(bar, 1);
    if (warp == 0) mbar_init(bbar, 1);
    fence_mbar_init_cluster();
  }
  uint32_t* mine = tile + warp * STEPS * G * 32;
  bool failed = false;
  if (p.solo && blockIdx.x == 0 && threadIdx.x == 0) *p.status = STATUS_OK;
  if (threadIdx.x == 0) *shared = place_of<false>(p, p.solo ? blockIdx.x : atomicAdd(p.ticket, 1u));
  __syncthreads();
  Loads loads(failed);
  while (shared->x >= 0) {
  const Item it = item_of<N>(p, *shared);
  if (TMA) {
    if (loads.ask<Loads::TILE>(it.live > 0) && lane == 0) {
      mbar_arrive_expect_tx(bar, STEPS * G * 128);
      tma_load_4d(smem_u32(mine), &xmap, bar, it.ct, 0, it.t0, it.b);
    }
    if (loads.ask<Loads::BIAS>(p.bias != nullptr) && threadIdx.x == 0) {
      mbar_arrive_expect_tx(bbar, G * 128);
      tma_load_4d(smem_u32(bcopy), &bmap, bbar, it.ct, 0, 0, 0);
    }
  } else {
    fetch_rows<T, G>(p, it, (const T*)p.Wx, mine);
  }
  Ch chain(p, it, failed);
  chain.ask(p.s0);
  FV<N> bias[G];
  if (TMA && p.bias) loads.wait<Loads::BIAS>(p, bbar);
  load_bias<T, FN, N, TMA>(p, it, bcopy, bias);
  if (TMA) {
    if (it.live > 0) loads.wait<Loads::TILE>(p, bar);
  } else {
    fetch_wait();
  }

  const Rows<T, G, TMA> raws(p, it, mine);
  FV<N> f[STEPS], u[Q8 ? STEPS : 1], P = splat<N>(1.0f), H = splat<N>(0.0f);
  uint32_t top[G];
#pragma unroll
  for (int g = 0; g < G; ++g) top[g] = 0;
  by_mask(it, [&](auto mask) {
    constexpr bool MASK = decltype(mask)::value;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const bool on = !MASK || j < it.live, rst = MASK && (it.rst >> j & 1);
      FV<N> z[G], w;
#pragma unroll
      for (int g = 0; g < (FN == GATED_LINEAR && !Q8 ? G - 1 : G); ++g) {  // o is read when it is needed
        const uint32_t raw = raws(j * G + g);
        if (Q8) top[g] = on ? mag_max<T>(top[g], raw) : top[g];
        z[g] = gate<FN>(g, Lane<T>::unpack(raw), bias[g]);
      }
      gated_coeff<FN, N>(z, f[j], w);
      if (MASK) {
        f[j] = select(on, rst ? splat<N>(0.0f) : f[j], splat<N>(1.0f));
        w = select(on, w, splat<N>(0.0f));
      }
      P = MASK ? factor(P, rst ? splat<N>(-0.0f) : f[j]) : mul(P, f[j]);
      H = MASK && rst ? w : fma(f[j], H, w);
      if (Q8) {
        u[j] = w;
      } else {
        if (!TMA) __syncwarp();  // the rows are read across the lanes
        mine[(j * G + U0) * 32 + lane] = __float_as_uint(w.v[0]);
        if (N == 2) mine[(j * G + U1) * 32 + lane] = __float_as_uint(w.v[N - 1]);
      }
    }
  });
#pragma unroll
  for (int v = 0; v < N; ++v) {
    maps[warp * Ch::ROW + v * 32 + lane] = make_float2(P.v[v], H.v[v]);
  }
  if (Q8) {
#pragma unroll
    for (int g = 0; g < G; ++g) tops[(warp * G + g) * 32 + lane] = top[g];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < Ch::M; ++i) {
    const float2 m = maps[chain.warp_of(i) * Ch::ROW + chain.c];
    chain.mine[i] = {m.x, m.y};
  }
  chain.publish();
  const bool wide = p.C % 2 == 0;
  if (Q8) {  // before the wait for the state: the tile in 8 bits
    const int qblocks = (p.T + ACT_BLOCK - 1) / ACT_BLOCK;
    FV<N> inv[G];
    bool huge = false, odd = false;  // a block that saturates, a block that is not finite
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t both = mag_max<T>(top[g], tops[((warp ^ 1) * G + g) * 32 + lane]);
#pragma unroll
      for (int v = 0; v < N; ++v) {
        const unsigned s = act_scale_byte(__uint_as_float(mag_bits<T>(both, v)));
        inv[g].v[v] = act_inv_scale(s);
        huge |= s == 248;
        odd |= s == ACT_NONFINITE;
        if ((warp & 1) == 0 && v < it.n && it.t0 < p.T)
          p.qs[(((size_t)it.b * qblocks + it.t0 / ACT_BLOCK) * G + g) * p.C + it.ch + v] = (unsigned char)s;
      }
    }
    huge = __any_sync(0xffffffffu, huge);
    odd = __any_sync(0xffffffffu, odd);
    unsigned char* qmine = qtile + warp * STEPS * G * 32 * N;
    auto pack = [&](auto mask) {  // MASK: steps that do not exist, saturated or non-finite blocks
      constexpr bool MASK = decltype(mask)::value;
#pragma unroll 4
      for (int j = 0; j < STEPS; ++j)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          FV<N> t = quant(Lane<T>::unpack(raws(j * G + g)), inv[g], MASK && huge);
          if (MASK) {
#pragma unroll
            for (int v = 0; v < N; ++v)
              if (j >= it.live || inv[g].v[v] == 0.0f) t.v[v] = 0.0f;
          }
          if (N == 2) *(unsigned short*)(qmine + (j * G + g) * 64 + lane * 2) = (unsigned short)low_bytes(t.v[0], t.v[N - 1]);
          else qmine[(j * G + g) * 32 + lane] = (unsigned char)__float_as_uint(t.v[0]);
        }
    };
    if (it.live == STEPS && !huge && !odd) pack(Flag<false>());
    else pack(Flag<true>());
    if (TMAQ) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && it.t0 < p.T) {
        tma_store_4d(&qmap, smem_u32(qmine), it.ct, 0, it.t0, it.b);
        bulk_commit_group();
      }
    } else {
      signed char* q = p.q + ((size_t)it.b * p.T + it.t0) * G * p.C + it.ch;
      for (int r = 0; r < STEPS * G && it.t0 + r / G < p.T; ++r)
#pragma unroll
        for (int v = 0; v < N; ++v)
          if (v < it.n) q[(size_t)r * p.C + v] = (signed char)qmine[r * 32 * N + lane * N + v];
    }
  }
  chain.pass(enter);
  if (p.carry) chain.store(p.carry, (size_t)it.b * p.chunks + it.k, chain.x);
  if (p.last && it.k == p.chunks - 1) chain.store(p.last, it.b, affine(chain.whole.P, chain.x, chain.whole.H));
  __syncthreads();
  unsigned next = 0xffffffffu;
  if (threadIdx.x == 0 && !p.solo) next = atomicAdd(p.ticket, 1u);  // on its way beside the last pass
  FV<N> c;
#pragma unroll
  for (int v = 0; v < N; ++v) c.v[v] = enter[warp * Ch::EROW + v * 32 + lane];
  by_mask(it, [&](auto mask) {
    constexpr bool MASK = decltype(mask)::value;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const bool on = !MASK || j < it.live, rst = MASK && (it.rst >> j & 1);
      FV<N> w, y, o;
      if (FN == GATED_LINEAR)
        o = sigmoid(gate<FN>(G - 1, Lane<T>::unpack(raws(j * G + G - 1)), bias[G - 1]));
      if (Q8) {
        w = u[Q8 ? j : 0];
      } else {
        w.v[0] = __uint_as_float(mine[(j * G + U0) * 32 + lane]);
        if (N == 2) w.v[N - 1] = __uint_as_float(mine[(j * G + U1) * 32 + lane]);
      }
      c = MASK && rst ? w : fma(f[j], c, w);
      y = FN == GATED_LINEAR ? mul(o, c) : c;
      if (MASK) y = select(on, y, splat<N>(0.0f));
      // step j's row lies in a step before j (or is row 0 of step 0), all read
      if (!TMA) __syncwarp();
      mine[j * 32 + lane] = Lane<T>::pack(y);
    }
  });
  if (TMA) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && it.t0 < p.T) {
      tma_store_4d(&hmap, smem_u32(mine), it.ct, 0, it.t0, it.b);
      bulk_commit_group();
      bulk_wait_group_read<0>();
    }
  } else {
    T* h = (T*)p.h + ((size_t)it.b * p.T + it.t0) * p.C + it.ch;
    for (int j = 0; j < STEPS && it.t0 + j < p.T; ++j) store_lane(h + (size_t)j * p.C, mine[j * 32 + lane], it.n, wide);
  }
  if (threadIdx.x == 0) *shared = place_of<false>(p, next);
  __syncthreads();
  }
  if (TMA) loads.leave(p, bar, bbar);
}

// Backward: 18 bytes a channel and step for linear bf16 (Wx, dh in; dWx out).
// The states are not stored by the forward but for one in 128: pass 1 evaluates
// the gates and folds the state's and the gradient's maps at once (the
// gradient's from e = o dh, which needs no state), the two enter, the states are
// run forward in registers, and the last pass runs the gradient back with the
// gates evaluated once more (keeping them would take the registers of f and c).
// dWx replaces the pre-activations in the tile and leaves by TMA; with the 8-bit
// tile, whose rows are too short, through a ring of 8 steps. Sums for db stay in
// registers over a warp's steps and are added over warps and items in a fixed
// order. Two 80 KB tiles fit an SM, and the time an item spends outside its loads
// (two passes of about 1.5 us, the state, the store) is what keeps it at 5.5
// TB/s: B=32 T=4096 C=1024 linear bf16 439 us with db, 429 without (362 at the
// copy bandwidth; without special functions 20 us less); fp32 B=16 T=2048 C=512
// 122 us, 4.97 TB/s; int8 checkpoint B=8 T=4099 C=1024 138 us.
template <typename T, int FN, bool Q8, bool TMA>
__global__ void __launch_bounds__(THREADS, (ctas_per_sm<T, FN, Q8>(true)))
    gated_bwd_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap dmap,
                     const __grid_constant__ CUtensorMap omap, const __grid_constant__ CUtensorMap bmap, GatedArgs p) {
  constexpr int G = gated_gates(FN), N = Lane<T>::N;
  constexpr int XB = Q8 ? 32 * N : 128;  // bytes of a row (t, g) of the tile
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* tile = smem;                                          // [WARPS][STEPS][G][XB]
  uint32_t* dtile = (uint32_t*)(tile + WARPS * STEPS * G * XB);        // [WARPS][STEPS][32]
  using Ch = Chain<N, true>;
  uint32_t* bcopy = dtile + WARPS * STEPS * 32;                        // [G][32]
  float2* maps = (float2*)(bcopy + G * 32);                            // [WARPS][ROW]: P, H of the state; slot v * 32 + lane
  float* mapE = (float*)(maps + WARPS * Ch::ROW);                      // [WARPS][EROW]: with P, the gradient's
  float* enter = mapE + WARPS * Ch::EROW;                              // [WARPS][EROW]: the gradients that enter the warps
  float* begin = enter + WARPS * Ch::EROW;                             // [WARPS][EROW]: the states that do
  float* dbs = begin + WARPS * Ch::EROW;                               // [WARPS][G][N][32]
  uint32_t* ring = (uint32_t*)(dbs + WARPS * G * 32 * N);              // Q8: [WARPS][8 steps][G][32]
  uint32_t* omine = ring + (threadIdx.x >> 5) * (Q8 ? 8 * G * 32 : 0);
  unsigned long long* bars = (unsigned long long*)(ring + (Q8 ? WARPS * 8 * G * 32 : 0));
  int4* shared = (int4*)(bars + WARPS + 2);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bar = smem_u32(bars + warp);
  const uint32_t bbar = smem_u32(bars + WARPS);
  if (TMA && lane == 0) {
    mbar_init(bar, 1);
    if (warp == 0) mbar_init(bbar, 1);
    fence_mbar_init_cluster();
  }
  unsigned char* mine = tile + warp * STEPS * G * XB;
  uint32_t* dmine = dtile + warp * STEPS * 32;
  const bool wide = p.C % 2 == 0;
  bool failed = false;
  if (p.solo && blockIdx.x == 0 && threadIdx.x == 0) *p.status = STATUS_OK;
  if (threadIdx.x == 0) *shared = place_of<true>(p, p.solo ? blockIdx.x : atomicAdd(p.ticket, 1u));
  if (!p.dh) {
#pragma unroll
    for (int j = 0; j < STEPS; ++j) dmine[j * 32 + lane] = 0;
  }
  __syncthreads();
  // db's sums over the warps of an item
  auto sum_db = [&](int b, int k, int ct) {
    for (int i = threadIdx.x; i < G * 32 * N; i += THREADS) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s += dbs[w * G * 32 * N + i];
      const int g = i / (32 * N), at = i % 32 * N + i / 32 % N, ch = ct + at;
      if (at < p.width && ch < p.C) {
        if (p.db_mode == 3) ((T*)p.db)[(size_t)g * p.C + ch] = from_f<T>(s);
        else __stcg(p.dbp + (((size_t)b * p.chunks + k) * G + g) * p.C + ch, s);
      }
    }
  };
  int last_b = -1, last_k = 0, last_ct = 0;  // mode 1: the item whose sums wait for the next load
  Loads loads(failed);
  while (shared->x >= 0) {
  const Item it = item_of<N>(p, *shared);
  if (TMA) {
    if (loads.ask<Loads::TILE>(it.live > 0) && lane == 0) {
      mbar_arrive_expect_tx(bar, STEPS * G * XB + (p.dh ? STEPS * 128 : 0));
      tma_load_4d(smem_u32(mine), &xmap, bar, it.ct, 0, it.t0, it.b);
      if (p.dh) tma_load_4d(smem_u32(dmine), &dmap, bar, it.ct, 0, it.t0, it.b);
    }
    if (loads.ask<Loads::BIAS>(p.bias != nullptr) && threadIdx.x == 0) {
      mbar_arrive_expect_tx(bbar, G * 128);
      tma_load_4d(smem_u32(bcopy), &bmap, bbar, it.ct, 0, 0, 0);
    }
  } else {
    if (Q8) {
      const signed char* at = p.q + ((size_t)it.b * p.T + it.t0) * G * p.C + it.ch;
#pragma unroll 8
      for (int r = 0; r < it.live * G; ++r)
#pragma unroll
        for (int v = 0; v < N; ++v)
          mine[r * XB + lane * N + v] = v < it.n ? (unsigned char)__ldg(at + (size_t)r * p.C + v) : 0;
    } else {
      fetch_rows<T, G>(p, it, (const T*)p.Wx, (uint32_t*)mine);
    }
    if (p.dh) fetch_rows<T, 1>(p, it, (const T*)p.dh, dmine);
  }
  Ch chain(p, it, failed);
  chain.ask(p.dlast);
  if (last_b >= 0) sum_db(last_b, last_k, last_ct);
  const float cc = chain.ch < p.C ? __ldg(p.carry + ((size_t)it.b * p.chunks + it.k) * p.C + chain.ch) : 0.0f;  // the state that enters the chunk
  FV<N> bias[G], scale[Q8 ? G : 1];
  if (Q8) {
    const int qblocks = (p.T + ACT_BLOCK - 1) / ACT_BLOCK;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int v = 0; v < N; ++v)
        scale[Q8 ? g : 0].v[v] =
            v < it.n && it.t0 < p.T
                ? mul_of<FN, N>(g) * act_scale(p.qs[(((size_t)it.b * qblocks + it.t0 / ACT_BLOCK) * G + g) * p.C + it.ch + v])
                : 0.0f;
  }
  if (TMA && p.bias) loads.wait<Loads::BIAS>(p, bbar);
  load_bias<T, FN, N, TMA>(p, it, bcopy, bias);
  if (TMA) {
    if (it.live > 0) loads.wait<Loads::TILE>(p, bar);
  } else {
    fetch_wait();
  }

  const Rows<T, G, TMA> raws(p, it, (const uint32_t*)mine);
  const Rows<T, 1, TMA> drows(p, it, dmine);
  auto gate_at = [&](int j, int g) {
    if (Q8) {
      const unsigned char* r = mine + (j * G + g) * XB + lane * N;
      const uint32_t w = N == 2 ? *(const unsigned short*)r : *r;
      return fma(bytes_f(w, (FV<N>*)nullptr), scale[Q8 ? g : 0], bias[g]);
    }
    return gate<FN>(g, Lane<T>::unpack(raws(j * G + g)), bias[g]);
  };

  FV<N> f[STEPS], u[STEPS], P = splat<N>(1.0f), H = splat<N>(0.0f), E = splat<N>(0.0f);
  by_mask(it, [&](auto mask) {
    constexpr bool MASK = decltype(mask)::value;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const bool on = !MASK || j < it.live, rst = MASK && (it.rst >> j & 1);
      FV<N> z[G], e = Lane<T>::unpack(drows(j));
#pragma unroll
      for (int g = 0; g < G; ++g) z[g] = gate_at(j, g);
      gated_coeff<FN, N>(z, f[j], u[j]);
      if (FN == GATED_LINEAR) e = mul(e, sigmoid(z[G - 1]));
      if (MASK) {
        e = select(on, e, splat<N>(0.0f));
        f[j] = select(on, rst ? splat<N>(0.0f) : f[j], splat<N>(1.0f));
        u[j] = select(on, u[j], splat<N>(0.0f));
      }
      // what step j's delta sends out of the warp's first step: f_0 .. f_j times it
      P = MASK ? factor(P, rst ? splat<N>(-0.0f) : f[j]) : mul(P, f[j]);
      H = MASK && rst ? u[j] : fma(f[j], H, u[j]);
      E = MASK ? affine(P, e, E) : fma(P, e, E);
    }
  });
#pragma unroll
  for (int v = 0; v < N; ++v) {
    maps[warp * Ch::ROW + v * 32 + lane] = make_float2(P.v[v], H.v[v]);
    mapE[warp * Ch::EROW + v * 32 + lane] = E.v[v];
  }
  __syncthreads();
  Map own[Ch::M];  // the state's maps of the lane's warps
#pragma unroll
  for (int i = 0; i < Ch::M; ++i) {
    const float2 m = maps[chain.warp_of(i) * Ch::ROW + chain.c];
    own[i] = {m.x, m.y};
    chain.mine[i] = {m.x, mapE[chain.warp_of(i) * Ch::EROW + chain.c]};
  }
  chain.publish();
  {  // the states that enter the warps: the lanes of a slot hold descending warps
    Map m = own[Ch::M - 1];
#pragma unroll
    for (int i = Ch::M - 2; i >= 0; --i) m = then(m, own[i]);
#pragma unroll
    for (int d = 1; d < Ch::Q; d *= 2) {
      const Map l = {__shfl_down_sync(0xffffffffu, m.P, d, Ch::Q), __shfl_down_sync(0xffffffffu, m.H, d, Ch::Q)};
      if (chain.q + d < Ch::Q) m = then(l, m);
    }
    Map l = {__shfl_down_sync(0xffffffffu, m.P, 1, Ch::Q), __shfl_down_sync(0xffffffffu, m.H, 1, Ch::Q)};
    if (chain.q == Ch::Q - 1) l = {1.0f, 0.0f};
    float e = affine(l.P, cc, l.H);
#pragma unroll
    for (int i = Ch::M - 1; i >= 0; --i) {
      begin[chain.warp_of(i) * Ch::EROW + chain.c] = e;
      e = affine(own[i].P, e, own[i].H);
    }
  }
  chain.pass(enter);
  if (p.ds0 && it.k == 0) chain.store(p.ds0, it.b, affine(chain.whole.P, chain.x, chain.whole.H));
  __syncthreads();
  unsigned next = 0xffffffffu;
  if (threadIdx.x == 0 && !p.solo) next = atomicAdd(p.ticket, 1u);  // on its way beside the last pass
  FV<N> c, x;  // the state before the warp's steps, the gradient that reaches it from after them
#pragma unroll
  for (int v = 0; v < N; ++v) {
    c.v[v] = begin[warp * Ch::EROW + v * 32 + lane];
    x.v[v] = enter[warp * Ch::EROW + v * 32 + lane];
  }
  const FV<N> start = c;
  by_mask(it, [&](auto mask) {
    constexpr bool MASK = decltype(mask)::value;
#pragma unroll
    for (int j = 0; j < STEPS; ++j) u[j] = c = MASK && (it.rst >> j & 1) ? u[j] : fma(f[j], c, u[j]);
  });
  FV<N> db[G];
#pragma unroll
  for (int g = 0; g < G; ++g) db[g] = splat<N>(0.0f);
  // dWx leaves through the tile (in place of the pre-activations it came from)
  // and one TMA store a warp; from the registers where the tile holds bytes or
  // TMA cannot take the rows
  constexpr bool staged = !Q8 && TMA, ringed = Q8 && TMA;
  T* out = p.dWx ? (T*)p.dWx + ((size_t)it.b * p.T + it.t0) * G * p.C + it.ch : nullptr;
  by_mask(it, [&](auto mask) {
    constexpr bool MASK = decltype(mask)::value;
#pragma unroll
    for (int j = STEPS - 1; j >= 0; --j) {
      const bool on = !MASK || j < it.live, rst = MASK && (it.rst >> j & 1);
      FV<N> z[G], da[G], d = Lane<T>::unpack(drows(j));
#pragma unroll
      for (int g = 0; g < G; ++g) z[g] = gate_at(j, g);
      FV<N> y = x;
      const FV<N> cp = j > 0 ? u[j > 0 ? j - 1 : 0] : start;
      gated_grad<FN, N>(z, f[j], MASK && rst ? splat<N>(0.0f) : cp, u[j], d, y, da);
      x = MASK ? select(on, rst ? splat<N>(0.0f) : y, x) : y;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (MASK) da[g] = select(on, da[g], splat<N>(0.0f));
        db[g] = add(db[g], da[g]);
        if (staged)
          *(uint32_t*)(mine + (j * G + g) * XB + lane * 4) = Lane<T>::pack(da[g]);
        else if (ringed)
          omine[((j & 7) * G + g) * 32 + lane] = Lane<T>::pack(da[g]);
        else if (out && it.t0 + j < p.T)
          store_lane(out + (size_t)(j * G + g) * p.C, Lane<T>::pack(da[g]), it.n, wide);
      }
      if (ringed && j % 4 == 0) {  // four steps are whole: their store, and the place of the four before is free
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && p.dWx && it.t0 + j < p.T) {
          tma_store_4d(&omap, smem_u32(omine + (j & 4) * G * 32), it.ct, 0, it.t0 + j, it.b);
          bulk_commit_group();
          bulk_wait_group_read<1>();
        }
        __syncwarp();
      }
    }
  });
  if (staged) {  // (the fence also puts the lanes' writes before the next item's load)
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && p.dWx && it.t0 < p.T) {
      tma_store_4d(&omap, smem_u32(mine), it.ct, 0, it.t0, it.b);
      bulk_commit_group();
    }
  }
  if (p.db_mode) {
    float* mine_db = dbs + warp * G * N * 32 + lane;
    const bool more = p.db_mode == 3 && it.b > 0;  // (mode 3: a channel tile's items come in the order of b)
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int v = 0; v < N; ++v) mine_db[(g * N + v) * 32] = more ? mine_db[(g * N + v) * 32] + db[g].v[v] : db[g].v[v];
    if (p.db_mode == 2 || (p.db_mode == 3 && it.b + 1 == p.B)) {
      __syncthreads();
      sum_db(it.b, it.k, it.ct);
    }
    if (p.db_mode == 2) {
      __threadfence();  // this thread's sums, before the count
      __syncthreads();
      if (threadIdx.x == 0) shared[1].x = (int)atomicAdd(p.done + it.ct / p.width, 1u);
      __syncthreads();
      const int rows = p.B * p.chunks;
      if (shared[1].x == rows - 1) {
        __threadfence();
        for (int i = threadIdx.x; i < G * 32 * N; i += THREADS) {
          const int g = i / (32 * N), ch = it.ct + i % (32 * N);
          if (ch >= min(p.C, it.ct + p.width)) continue;
          const float* at = p.dbp + (size_t)g * p.C + ch;
          float s = 0.0f;
#pragma unroll 32
          for (int r = 0; r < rows; ++r) s += __ldcg(at + (size_t)r * G * p.C);
          ((T*)p.db)[(size_t)g * p.C + ch] = from_f<T>(s);
        }
      }
    }
  }
  if (TMA && lane == 0) bulk_wait_group_read<0>();  // the tile is read from until then
  if (threadIdx.x == 0) *shared = place_of<true>(p, p.db_mode == 3 ? it.tile + p.tiles_c : next);
  if (p.db_mode == 1) last_b = it.b, last_k = it.k, last_ct = it.ct;
  __syncthreads();
  }
  if (last_b >= 0) sum_db(last_b, last_k, last_ct);
  if (TMA) loads.leave(p, bar, bbar);
}

template <typename T, int FN, bool Q8> constexpr int fwd_smem() {
  constexpr int G = gated_gates(FN), N = Lane<T>::N, W = 32 * N;
  return WARPS * STEPS * G * 128 + G * 128 + WARPS * (W + 2) * 8 + WARPS * (W + 4) * 4 +
         (Q8 ? WARPS * G * 32 * (4 + STEPS * N) : 0) + WARPS * 8 + 48;
}
template <typename T, int FN, bool Q8> constexpr int bwd_smem() {
  constexpr int G = gated_gates(FN), N = Lane<T>::N, W = 32 * N;
  return WARPS * STEPS * (G * (Q8 ? W : 128) + 128) + G * 128 + WARPS * (W + 2) * 8 + 3 * WARPS * (W + 4) * 4 +
         WARPS * G * W * 4 + (Q8 ? WARPS * 8 * G * 128 : 0) + WARPS * 8 + 48;
}

// db[j] = sum over `rows` of dbp[row][j], in row order within 32 interleaved
// lanes, then the lanes in order.
template <typename T>
__global__ void __launch_bounds__(1024) gated_db_kernel(const float* dbp, T* db, int rows, int cols) {
  __shared__ float red[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + tx;
  float s = 0.0f;
  if (j < cols)
#pragma unroll 8
    for (int r = ty; r < rows; r += 32) s += dbp[(size_t)r * cols + j];
  red[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && j < cols) {
#pragma unroll
    for (int k = 1; k < 32; ++k) s += red[k][tx];
    db[j] = from_f<T>(s);
  }
}

struct StepArgs {
  int rows, C, slots;
  const void* Wx;
  const void* bias;
  const int* slot;
  const float* pool;
  float* pool_out;
  void* h;
  unsigned* status;
};

// One step of many sequences: nothing to share, a thread has the N channels of a
// lane (4 bytes of the storage type) and everything it needs is asked for at
// once. Launch and one round trip bound it: 5 us for 1 to 256 rows of C=1024.
template <typename T, int FN>
__global__ void __launch_bounds__(128) gated_step_kernel(StepArgs p) {
  constexpr int G = gated_gates(FN), N = Lane<T>::N;
  const int lanes = (p.C + N - 1) / N;
  const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
  if (id >= (long long)p.rows * lanes) return;
  const int m = (int)(id / lanes), ch = (int)(id % lanes) * N;
  const int n = min(p.C - ch, N);
  const bool wide = p.C % 2 == 0;
  const int slot = p.slot ? __ldg(p.slot + m) : m;
  FV<N> y = splat<N>(0.0f);
  if (slot >= 0 && slot < p.slots) {
    FV<N> z[G], f, u, c;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      z[g] = Lane<T>::unpack(load_lane((const T*)p.Wx + ((size_t)m * G + g) * p.C + ch, n, wide));
      FV<N> b = Lane<T>::unpack(p.bias ? load_lane((const T*)p.bias + (size_t)g * p.C + ch, n, wide) : 0);
      z[g] = gate<FN>(g, z[g], mul(b, splat<N>(mul_of<FN, N>(g))));
    }
    const size_t at = (size_t)slot * p.C + ch;
#pragma unroll
    for (int v = 0; v < N; ++v) c.v[v] = v < n ? p.pool[at + v] : 0.0f;
    gated_coeff<FN, N>(z, f, u);
    c = fma(f, c, u);
#pragma unroll
    for (int v = 0; v < N; ++v)
      if (v < n) p.pool_out[at + v] = c.v[v];
    y = FN == GATED_LINEAR ? mul(sigmoid(z[G - 1]), c) : c;
  } else if (slot >= p.slots && ch == 0 && p.status) {
    atomicOr(p.status, STATUS_RANGE);
  }
  store_lane((T*)p.h + (size_t)m * p.C + ch, Lane<T>::pack(y), n, wide);
}

// ---- host ----------------------------------------------------------------------
int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return RNN_OK;
  fprintf(stderr, "librnn_gb300: CUDA error: %s\n", cudaGetErrorString(e));
  return RNN_ECUDA;
}
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

bool gated_dims_ok(const rnn_gated_dims_t* d) {
  return d && d->B >= 1 && d->T >= 0 && d->T <= INT_MAX - GATED_CHUNK && d->N >= 1 && d->D >= 1 && (d->function == RNN_LINEAR || d->function == RNN_LINEAR_COUPLED) &&
         (d->dtype == RNN_F32 || d->dtype == RNN_BF16) && (d->checkpoint == RNN_CKPT_NONE || d->checkpoint == RNN_CKPT_INT8) &&
         (long long)d->N * d->D <= (1 << 28) &&
         // one item per 128 steps of 28 (at least) channels
         (double)d->B * (d->N * (double)d->D / 28 + 1) * (d->T / (double)GATED_CHUNK + 1) < 2147483647.0;
}

struct GatedSizes {
  int G, C, chunks, qblocks, width, tiles_c, span, solo, db_mode;
  size_t esize, carry, q, qs, tape;
  // workspace: status, ticket, states, maps, counts (sync: zeroed by every call;
  // solo: the status alone, written by it) | db sums
  size_t sync, states, maps, dbp;
};
GatedSizes gated_sizes(const rnn_gated_dims_t* d) {
  GatedSizes z;
  z.G = gated_gates(d->function);
  z.C = d->N * d->D;
  z.chunks = (d->T + GATED_CHUNK - 1) / GATED_CHUNK;
  z.qblocks = (d->T + ACT_BLOCK - 1) / ACT_BLOCK;
  z.esize = d->dtype == RNN_BF16 ? 2 : 4;
  // whole rows of lanes where rows are 16-byte multiples, else 28 lanes (fetch_rows)
  const int lane = d->dtype == RNN_BF16 ? 2 : 1;
  z.width = (z.C * z.esize) % 16 == 0 ? 32 * lane : 28 * lane;
  z.tiles_c = (z.C + z.width - 1) / z.width;
  const size_t tiles = (size_t)d->B * z.tiles_c;
  // With fewer tiles than SMs, chunks of one tile wait on one another: the more
  // of them run side by side, the more share a hop of the chain. Measured at
  // 12 tiles (B=1 T=65537 C=768, forward): groups of 1, 2, 4, 8, 16, 32 chunks
  // take 310, 167, 124, 119, 121, 126 us; at 128 tiles (B=8 T=4096 C=1024) 1
  // takes 70 us, 2 to 8 74, 32 81.
  const size_t sms = device_sms();
  z.span = 0;
  while (z.span < MAX_SPAN && (tiles << (z.span + 1)) <= sms) ++z.span;
  // A short sequence is all latency: without TMA there is no wait that could
  // run out, and the clearing launch for the status word falls away.
  z.solo = z.chunks == 1 && tiles <= 2 * sms;
  const size_t lanes = tiles * 32 * (d->dtype == RNN_BF16 ? 2 : 1);
  z.carry = up256((size_t)d->B * z.chunks * z.C * sizeof(float));
  const bool q8 = d->checkpoint == RNN_CKPT_INT8;
  z.q = q8 ? up256((size_t)d->B * d->T * z.G * z.C) : 0;
  z.qs = q8 ? up256((size_t)d->B * z.qblocks * z.G * z.C) : 0;
  z.tape = z.carry + z.q + z.qs;
  const size_t groups = z.span ? ((size_t)(z.chunks - 1) >> z.span) + 1 : 2;
  z.states = z.chunks > 1 ? up256(groups * lanes * sizeof(unsigned long long)) : 0;
  z.maps = z.chunks > 1 && z.span > 0 ? up256(z.chunks * lanes * sizeof(ulonglong2)) : 0;
  // db: with few batch rows of one chunk, a CTA takes a channel tile's rows one
  // after the other; with few items, the last one adds the items' sums (32
  // loads in flight, a round trip of a microsecond each); else a launch does
  // (128 items: 24 us after the last one against 6 for the launch).
  const long long rows = (long long)d->B * z.chunks;
  z.db_mode = z.solo && d->B <= 8 ? 3 : !z.solo && rows <= 64 ? 2 : 1;
  z.sync = z.solo ? 256 : 512 + z.states + z.maps + up256(z.tiles_c * sizeof(unsigned));
  z.dbp = z.db_mode == 3 ? 0 : up256((size_t)d->B * z.chunks * z.G * z.C * sizeof(float));
  return z;
}

// [C][rows][T][B] box of one warp's steps; elem: 1, 2 or 4 bytes
cudaError_t tile_map(CUtensorMap* m, const void* base, int elem, const GatedArgs& a, int rows, int width, int steps = STEPS) {
  const unsigned long long dims[4] = {(unsigned long long)a.C, (unsigned long long)rows, (unsigned long long)a.T,
                                      (unsigned long long)a.B};
  const unsigned box[4] = {(unsigned)width, (unsigned)rows, (unsigned)steps, 1};
  return encode_tensor_map(m, base, elem, 4, dims, box);
}

template <typename T, int FN, bool Q8, bool TMA> cudaError_t gated_launch(bool bwd, const GatedArgs& a, cudaStream_t st) {
  constexpr int G = gated_gates(FN), width = 32 * Lane<T>::N;
  CUtensorMap x = {}, d = {}, out = {}, q = {}, bias = {};
  if (TMA) {
    cudaError_t e = bwd && Q8 ? tile_map(&x, a.q, 1, a, G, width) : tile_map(&x, a.Wx, (int)sizeof(T), a, G, width);
    if (e == cudaSuccess && a.bias) {
      const unsigned long long dims[4] = {(unsigned long long)a.C, G, 1, 1};
      const unsigned box[4] = {width, G, 1, 1};
      e = encode_tensor_map(&bias, a.bias, (int)sizeof(T), 4, dims, box);
    }
    if (e == cudaSuccess && bwd && a.dh) e = tile_map(&d, a.dh, (int)sizeof(T), a, 1, width);
    if (e == cudaSuccess && !bwd && Q8) e = tile_map(&q, a.q, 1, a, G, width);
    if (e == cudaSuccess && !bwd) e = tile_map(&out, a.h, (int)sizeof(T), a, 1, width);
    if (e == cudaSuccess && bwd && a.dWx) e = tile_map(&out, a.dWx, (int)sizeof(T), a, G, width, Q8 ? 4 : STEPS);
    if (e != cudaSuccess) return e;
  }
  const unsigned items = (unsigned)((size_t)a.B * a.tiles_c * a.chunks);
  const int smem = bwd ? bwd_smem<T, FN, Q8>() : fwd_smem<T, FN, Q8>();
  const void* k = bwd ? (const void*)gated_bwd_kernel<T, FN, Q8, TMA> : (const void*)gated_fwd_kernel<T, FN, Q8, TMA>;
  cudaError_t e = set_smem_attr(k, smem);
  if (e != cudaSuccess) return e;
  const unsigned most = device_sms() * ctas_per_sm<T, FN, Q8>(bwd);
  const unsigned ctas = bwd && a.db_mode == 3 ? a.tiles_c : a.solo || items < most ? items : most;
  if (bwd) gated_bwd_kernel<T, FN, Q8, TMA><<<ctas, THREADS, smem, st>>>(x, d, out, bias, a);
  else gated_fwd_kernel<T, FN, Q8, TMA><<<ctas, THREADS, smem, st>>>(x, out, q, bias, a);
  note_launch();
  return cudaGetLastError();
}
template <typename T, int FN, bool Q8> cudaError_t gated_launch(bool bwd, const GatedArgs& a, cudaStream_t st) {
  // TMA rows start on 16 bytes
  const bool tma = !a.solo && ((size_t)a.C * (Q8 ? 1 : sizeof(T))) % 16 == 0;
  return tma ? gated_launch<T, FN, Q8, true>(bwd, a, st) : gated_launch<T, FN, Q8, false>(bwd, a, st);
}
template <typename T> cudaError_t gated_launch(int fn, bool q8, bool bwd, const GatedArgs& a, cudaStream_t st) {
  if (fn == GATED_LINEAR)
    return q8 ? gated_launch<T, GATED_LINEAR, true>(bwd, a, st) : gated_launch<T, GATED_LINEAR, false>(bwd, a, st);
  return q8 ? gated_launch<T, GATED_COUPLED, true>(bwd, a, st) : gated_launch<T, GATED_COUPLED, false>(bwd, a, st);
}
cudaError_t gated_launch(const rnn_gated_dims_t* d, bool q8, bool bwd, const GatedArgs& a, cudaStream_t st) {
  return d->dtype == RNN_BF16 ? gated_launch<__nv_bfloat16>(d->function, q8, bwd, a, st)
                              : gated_launch<float>(d->function, q8, bwd, a, st);
}

// What both directions take from the dims and the workspace.
GatedArgs gated_args(const rnn_gated_dims_t* d, const GatedSizes& z, void* workspace) {
  GatedArgs a{};
  a.B = d->B; a.T = d->T; a.C = z.C; a.chunks = z.chunks;
  a.tiles_c = z.tiles_c; a.width = z.width; a.span = z.span; a.solo = z.solo;
  char* ws = (char*)workspace;
  a.status = (unsigned*)ws;
  if (!z.solo) {
    a.ticket = (unsigned*)(ws + 256);
    a.states = (unsigned long long*)(ws + 512);
    a.maps = (ulonglong2*)(ws + 512 + z.states);
    a.done = (unsigned*)(ws + 512 + z.states + z.maps);
  }
  a.wait_limit_ns = wait_limit_ns();
  inject_wait(&a.inject_chunk, &a.inject_limit_ns);
  if (z.solo) a.inject_chunk = -1;
  return a;
}

}  // namespace
}  // namespace rnn

using namespace rnn;

extern "C" {

int rnn_gated_num_gates(int function) {
  return function == RNN_LINEAR || function == RNN_LINEAR_COUPLED ? gated_gates(function) : -1;
}

size_t rnn_gated_tape_size(const rnn_gated_dims_t* d) { return gated_dims_ok(d) ? gated_sizes(d).tape : 0; }

size_t rnn_gated_workspace_size(const rnn_gated_dims_t* d, int kind) {
  if (!gated_dims_ok(d) || (kind != RNN_WS_FWD && kind != RNN_WS_BWD)) return 0;
  const GatedSizes z = gated_sizes(d);
  return z.sync + (kind == RNN_WS_BWD ? z.dbp : 0);
}

int rnn_gated_fwd(const rnn_gated_dims_t* d, const void* Wx, const void* b, const void* state0,
                  const unsigned char* reset, const int* lengths, void* h, void* last, void* tape,
                  void* workspace, size_t ws_bytes, void* stream) {
  if (!gated_dims_ok(d) || !workspace || (d->T > 0 && (!Wx || !h))) return RNN_EINVAL;
  const void* ptrs[] = {Wx, b, state0, h, last, tape, workspace};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (lengths && ((uintptr_t)lengths & 3u)) return RNN_EINVAL;
  if (ws_bytes < rnn_gated_workspace_size(d, RNN_WS_FWD)) return RNN_ENOSPC;
  cudaStream_t st = (cudaStream_t)stream;
  const GatedSizes z = gated_sizes(d);
  int rc = z.solo ? RNN_OK : cuda_status(cudaMemsetAsync(workspace, 0, z.sync, st));
  if (rc) return rc;
  if (d->T == 0) {
    const size_t bytes = (size_t)d->B * z.C * sizeof(float);
    if (!last) return RNN_OK;
    return cuda_status(state0 ? cudaMemcpyAsync(last, state0, bytes, cudaMemcpyDeviceToDevice, st)
                              : cudaMemsetAsync(last, 0, bytes, st));
  }
  GatedArgs a = gated_args(d, z, workspace);
  a.Wx = Wx; a.bias = b; a.s0 = (const float*)state0; a.reset = reset; a.lengths = lengths;
  a.h = h; a.last = (float*)last;
  a.carry = (float*)tape;
  const bool q8 = tape && d->checkpoint == RNN_CKPT_INT8;
  if (q8) {
    a.q = (signed char*)tape + z.carry;
    a.qs = (unsigned char*)tape + z.carry + z.q;
  }
  return cuda_status(gated_launch(d, q8, false, a, st));
}

int rnn_gated_bwd(const rnn_gated_dims_t* d, const void* Wx, const void* b, const unsigned char* reset,
                  const int* lengths, const void* tape, const void* dh, const void* dlast, void* dWx, void* db,
                  void* dstate0, void* workspace, size_t ws_bytes, void* stream) {
  if (!gated_dims_ok(d) || !workspace) return RNN_EINVAL;
  const bool q8 = d->checkpoint == RNN_CKPT_INT8;
  if (d->T > 0 && (!tape || (!q8 && !Wx))) return RNN_EINVAL;
  const void* ptrs[] = {Wx, b, tape, dh, dlast, dWx, db, dstate0, workspace};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (lengths && ((uintptr_t)lengths & 3u)) return RNN_EINVAL;
  if (ws_bytes < rnn_gated_workspace_size(d, RNN_WS_BWD)) return RNN_ENOSPC;
  cudaStream_t st = (cudaStream_t)stream;
  const GatedSizes z = gated_sizes(d);
  int rc = z.solo ? RNN_OK : cuda_status(cudaMemsetAsync(workspace, 0, z.sync, st));
  if (rc) return rc;
  if (d->T == 0) {
    const size_t bytes = (size_t)d->B * z.C * sizeof(float);
    if (dstate0) {
      rc = cuda_status(dlast ? cudaMemcpyAsync(dstate0, dlast, bytes, cudaMemcpyDeviceToDevice, st)
                             : cudaMemsetAsync(dstate0, 0, bytes, st));
      if (rc) return rc;
    }
    return db ? cuda_status(cudaMemsetAsync(db, 0, (size_t)z.G * z.C * z.esize, st)) : RNN_OK;
  }
  GatedArgs a = gated_args(d, z, workspace);
  a.Wx = Wx; a.bias = b; a.reset = reset; a.lengths = lengths;
  a.carry = (float*)tape;
  if (q8) {
    a.q = (signed char*)tape + z.carry;
    a.qs = (unsigned char*)tape + z.carry + z.q;
  }
  a.dh = dh; a.dlast = (const float*)dlast; a.dWx = dWx; a.ds0 = (float*)dstate0;
  a.db = db;
  a.db_mode = db ? z.db_mode : 0;
  a.dbp = (float*)((char*)workspace + z.sync);
  rc = cuda_status(gated_launch(d, q8, true, a, st));
  if (rc || a.db_mode != 1) return rc;
  const int cols = z.G * z.C;
  if (d->dtype == RNN_BF16)
    gated_db_kernel<<<(cols + 31) / 32, 1024, 0, st>>>(a.dbp, (__nv_bfloat16*)db, d->B * z.chunks, cols);
  else
    gated_db_kernel<<<(cols + 31) / 32, 1024, 0, st>>>(a.dbp, (float*)db, d->B * z.chunks, cols);
  note_launch();
  return cuda_status(cudaGetLastError());
}

int rnn_gated_step(int rows, int slots, int N, int D, int function, int dtype, const void* Wx, const void* b,
                   const int* slot, const void* pool, void* pool_out, void* h, void* status, void* stream) {
  if (rows < 0 || slots < 1 || N < 1 || D < 1 || (long long)N * D > (1 << 28) || rnn_gated_num_gates(function) < 0 ||
      (dtype != RNN_F32 && dtype != RNN_BF16) || (!slot && rows > slots))
    return RNN_EINVAL;
  if (!pool || !pool_out || (rows > 0 && (!Wx || !h))) return RNN_EINVAL;
  const void* ptrs[] = {Wx, b, pool, pool_out, h};
  for (const void* p : ptrs)
    if (p && !al16(p)) return RNN_EINVAL;
  if (((uintptr_t)slot & 3u) || ((uintptr_t)status & 3u)) return RNN_EINVAL;
  if (!pools_apart(pool, pool_out, (size_t)slots * N * D * sizeof(float))) return RNN_EINVAL;
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) return RNN_OK;
  StepArgs a{rows, N * D, slots, Wx, b, slot, (const float*)pool, (float*)pool_out, h, (unsigned*)status};
  const int n = dtype == RNN_BF16 ? 2 : 1;
  const unsigned grid = (unsigned)(((long long)rows * ((a.C + n - 1) / n) + 127) / 128);
  if (dtype == RNN_BF16) {
    if (function == RNN_LINEAR) gated_step_kernel<__nv_bfloat16, GATED_LINEAR><<<grid, 128, 0, st>>>(a);
    else gated_step_kernel<__nv_bfloat16, GATED_COUPLED><<<grid, 128, 0, st>>>(a);
  } else {
    if (function == RNN_LINEAR) gated_step_kernel<float, GATED_LINEAR><<<grid, 128, 0, st>>>(a);
    else gated_step_kernel<float, GATED_COUPLED><<<grid, 128, 0, st>>>(a);
  }
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
