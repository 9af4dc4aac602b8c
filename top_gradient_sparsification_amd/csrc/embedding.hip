// Embedding lookup and its gradient on gfx950.
//
// Lookup: out[t] = scale * table[token[t]], a row of zeros where token[t] < 0.
// One pass, bound by HBM: every thread moves four vectors of 16 bytes (of the
// wider of the two types), all four rows' loads in flight before the first
// store.  131,072 rows of 2,048 in bf16 from a table of 128,000: 184 us.  Its
// 32,600 distinct rows are 134 MB, but each of the eight L2s fetches for itself,
// 225 MB if it kept all and 301 as counted: with the 537 MB written 4.6 TB/s of a
// copy's 5.2.  One row: 3 us of a call's 8.
//
// Gradient: out[v] (+)= scale * sum of grad[t] over the places with
// token[t] == v.  Atomic adds would make the sums depend on their order, and a
// frequent token's row would take one add per occurrence; instead
//   1. the places are sorted by token, stably (radix, 8 to 10 bits a pass), so
//      every token's places stand together in ascending order;
//   2. k_grad_chunks: the sorted list is cut into chunks of 8 to 64 places.  A
//      wave takes one chunk for 64 vectors of columns, walks the chunk with
//      eight row loads in flight and keeps the running row sum in registers.  A
//      token whose places all lie inside the chunk is finished there; a sum
//      that continues into a neighbouring chunk goes to a partial row.  Other
//      waves of the same launch write the zeros of rows no token names (a
//      binary search in the sorted tokens finds them);
//   3. k_grad_join: partial rows of tokens that span chunks are added in chunk
//      order.
// Few places of a small table take one launch instead (k_grad_few).
// The order of every sum is fixed by the tokens alone, so results are the same
// bits on every run.  Sums are fp32.
#include <type_traits>

#include "tgs_host.h"
#include "tgs_types.h"

namespace tgs {

// A token outside [-inf, V) is an error: it reads and adds to nothing.
template <class I>
__device__ __forceinline__ int64_t load_token(const I* p, int64_t t) {
  return (int64_t)p[t];
}

// ---------------------------------------------------------------- lookup --
struct LookupArgs {
  const void* tokens;
  const void* table;
  void* out;
  u32* err;
  int64_t T, V, D;
  u32 nv;     // vectors a row
  u64 total;  // T * nv
  float scale;
};

constexpr int kLookupThreads = 256;
constexpr int kLookupUnroll = 4;
// Above this size stores pass the caches by, so that these keep the table's
// frequent rows.  From 128,000 rows of 2,048 in bf16, inputs changing, plain and
// past the caches: 8 MB 8.9 and 9.1 us, 34 MB 14.7 and 12.3, 134 MB 52 and 36, 537
// MB 197 and 185.  What reads a smaller result next still finds it in the caches:
// with an addition over the result 50 MB take 36.3 and 37.6, 67 MB 47.1 and 48.6,
// 100 MB 69.7 and 68.4, 537 MB 374 and 362.
constexpr size_t kStreamingBytes = (size_t)64 << 20;

template <class TI, class TO, class I, int E, bool STREAMING>
__global__ __launch_bounds__(kLookupThreads) void k_lookup(LookupArgs a) {
  const I* tokens = (const I*)a.tokens;
  const TI* table = (const TI*)a.table;
  TO* out = (TO*)a.out;
  const u64 base = (u64)blockIdx.x * (kLookupThreads * kLookupUnroll);
  const u64 row0 = base / a.nv;
  const u32 rest = (u32)(base - row0 * a.nv) + threadIdx.x;
  int64_t tok[kLookupUnroll], row[kLookupUnroll], at[kLookupUnroll];
  Vec<TI, E> x[kLookupUnroll];
#pragma unroll
  for (int u = 0; u < kLookupUnroll; ++u) {
    const u32 i = rest + u * kLookupThreads;
    const u32 q = i / a.nv;
    row[u] = (int64_t)(row0 + q);
    // the last vector of a row ends with the row: it may overlap the one before
    const int64_t c = (int64_t)(i - q * a.nv) * E;
    at[u] = c + E <= a.D ? c : a.D - E;
    tok[u] = row[u] < a.T ? load_token(tokens, row[u]) : -1;
    if (tok[u] >= a.V) {
      atomicOr(a.err, kErrBadInput);
      tok[u] = -1;
    }
  }
#pragma unroll
  for (int u = 0; u < kLookupUnroll; ++u)
    if (tok[u] >= 0) x[u] = load_vec<TI, E>(table + tok[u] * a.D + at[u]);
#pragma unroll
  for (int u = 0; u < kLookupUnroll; ++u) {
    Vec<TO, E> y;
#pragma unroll
    for (int e = 0; e < E; ++e) y.v[e] = from_f32<TO>(tok[u] >= 0 ? to_f32(x[u].v[e]) * a.scale : 0.0f);
    if (row[u] < a.T) {
      if constexpr (STREAMING) store_vec_streaming<TO, E>(out + row[u] * a.D + at[u], y);
      else store_vec<TO, E>(out + row[u] * a.D + at[u], y);
    }
  }
}

// ------------------------------------------------------------------ sort --
// Keys: the token where it lies in [0, V), else V (sorted behind all others).
constexpr int kTokenThreads = 512;
constexpr int kTokenWaves = kTokenThreads / kWave;
constexpr int kDigitBits = 10;
// Sorting workgroups, one for 2,048 places.  131,072 places of 16 columns take 64
// us with 32 of them, 55 with 64, 56 with 128; 1,000,000 238 with 64, 199 with 128,
// 189 with 256, which double the counts that each reads.  Of 1,024 places each
// 16,384 take 36 us instead of 40, 131,072 56 instead of 55.
constexpr int kTokenBlocks = 128;
constexpr int kOneThreads = 1024;
constexpr int kOneWaves = kOneThreads / kWave;
// Places that one workgroup sorts, in one launch: what LDS holds (4,096 of 64
// columns in 25,000 rows: 31 us, 37 by several; 2,500: 27 and 34).
constexpr int kOneMaxT = 4096;

struct SortArgs {
  const void* tokens;
  const u32* keys_in;
  const u32* places_in;
  u32* keys_out;
  u32* places_out;
  u32* hist;  // [blocks][1 << bits]
  u32* err;
  u32 T, V;
  u32 per_wave;  // places a wave handles, a multiple of 64
  int shift, bits, passes;
};

template <class I>
__device__ __forceinline__ u32 token_key(const SortArgs& a, u32 t) {
  const int64_t v = load_token((const I*)a.tokens, t);
  if (v >= (int64_t)a.V) atomicOr(a.err, kErrBadInput);
  return v >= 0 && v < (int64_t)a.V ? (u32)v : a.V;
}

// The lanes of the wave whose digit equals this lane's (inactive lanes must
// hold a digit no active lane has: bit `bits` set).
__device__ __forceinline__ u64 same_digit(u32 d, int bits) {
  u64 m = ~0ull;
  for (int b = 0; b <= bits; ++b) {
    const bool bit = (d >> b) & 1u;
    const u64 with = ballot(bit);
    m &= bit ? with : ~with;
  }
  return m;
}

// Counts of each digit over a block's places.
template <class I, bool FIRST>
__global__ __launch_bounds__(kTokenThreads) void k_sort_count(SortArgs a) {
  __shared__ u32 s_h[1 << kDigitBits];
  const u32 bins = 1u << a.bits;
  for (u32 i = threadIdx.x; i < bins; i += kTokenThreads) s_h[i] = 0;
  __syncthreads();
  const u64 b0 = (u64)blockIdx.x * a.per_wave * kTokenWaves;
  const u64 b1 = min((u64)a.T, b0 + (u64)a.per_wave * kTokenWaves);
  for (u64 t = b0 + threadIdx.x; t < b1; t += kTokenThreads) {
    const u32 key = FIRST ? token_key<I>(a, (u32)t) : a.keys_in[t];
    atomicAdd(&s_h[(key >> a.shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (u32 i = threadIdx.x; i < bins; i += kTokenThreads) a.hist[(u64)blockIdx.x * bins + i] = s_h[i];
}

// Exclusive prefix over the (up to 1024) values s_v[bin] in bin order.
template <int NT>
__device__ __forceinline__ void scan_bins(u32* s_v, u32 bins, u32* s_scan) {
  u32 carry = 0;
  for (u32 b0 = 0; b0 < bins; b0 += NT) {
    const u32 i = b0 + threadIdx.x;
    const u32 v = i < bins ? s_v[i] : 0;
    u32 total;
    const u32 ex = block_exclusive_sum<NT>(v, s_scan, total);
    if (i < bins) s_v[i] = carry + ex;
    carry += total;
  }
  __syncthreads();
}

// Moves a block's places to where the pass puts them: every wave owns a
// contiguous part of the block, so (digit, block, wave, place) is the order.
template <class I, bool FIRST>
__global__ __launch_bounds__(kTokenThreads) void k_sort_move(SortArgs a) {
  __shared__ u32 s_off[kTokenWaves][1 << kDigitBits];
  __shared__ u32 s_base[1 << kDigitBits];
  __shared__ u32 s_scan[kTokenWaves + 1];
  const u32 bins = 1u << a.bits, mask = bins - 1;
  const int w = threadIdx.x / kWave, lane = lane_id();
  for (u32 i = threadIdx.x; i < bins * kTokenWaves; i += kTokenThreads) s_off[i >> a.bits][i & mask] = 0;
  // block base of each digit: all smaller digits, and this digit in earlier blocks
  u32 before[(1 << kDigitBits) / kTokenThreads] = {};
  const u32 nb = gridDim.x;
#pragma unroll
  for (int j = 0; j < (1 << kDigitBits) / kTokenThreads; ++j) {
    const u32 bin = j * kTokenThreads + threadIdx.x;
    u32 all = 0;
    if (bin < bins) {
#pragma unroll 8
      for (u32 b = 0; b < nb; ++b) {
        const u32 c = a.hist[(u64)b * bins + bin];
        if (b < blockIdx.x) before[j] += c;
        all += c;
      }
      s_base[bin] = all;
    }
  }
  __syncthreads();
  const u64 w0 = ((u64)blockIdx.x * kTokenWaves + w) * a.per_wave;
  const u64 w1 = min((u64)a.T, w0 + a.per_wave);
  for (u64 t = w0 + lane; t < w1; t += kWave) {
    const u32 key = FIRST ? token_key<I>(a, (u32)t) : a.keys_in[t];
    atomicAdd(&s_off[w][(key >> a.shift) & mask], 1u);
  }
  scan_bins<kTokenThreads>(s_base, bins, s_scan);
#pragma unroll
  for (int j = 0; j < (1 << kDigitBits) / kTokenThreads; ++j) {
    const u32 bin = j * kTokenThreads + threadIdx.x;
    if (bin < bins) {
      u32 run = s_base[bin] + before[j];
      for (int i = 0; i < kTokenWaves; ++i) {
        const u32 c = s_off[i][bin];
        s_off[i][bin] = run;
        run += c;
      }
    }
  }
  __syncthreads();
  for (u64 t0 = w0; t0 < w1; t0 += kWave) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the offsets that other lanes moved on
    const u64 t = t0 + lane;
    const bool here = t < w1;
    const u32 key = !here ? 0u : FIRST ? token_key<I>(a, (u32)t) : a.keys_in[t];
    const u32 d = here ? (key >> a.shift) & mask : bins;
    const u64 same = same_digit(d, a.bits);
    const u32 rank = __popcll(same & ((1ull << lane) - 1));
    u32 off = 0;
    if (here && rank == 0) {
      off = s_off[w][d];
      s_off[w][d] = off + __popcll(same);
    }
    off = __shfl(off, (int)__ffsll((unsigned long long)same) - 1);
    if (here) {
      a.keys_out[off + rank] = key;
      a.places_out[off + rank] = FIRST ? (u32)t : a.places_in[t];
    }
  }
}

// All passes in one workgroup, for up to kOneMaxT places.
template <class I>
__global__ __launch_bounds__(kOneThreads) void k_sort_one(SortArgs a) {
  __shared__ u32 s_key[2][kOneMaxT];
  __shared__ u16 s_place[2][kOneMaxT];
  __shared__ u32 s_off[kOneWaves][1 << kDigitBits];
  __shared__ u32 s_base[1 << kDigitBits];
  __shared__ u32 s_scan[kOneWaves + 1];
  const u32 T = a.T, bins = 1u << a.bits, mask = bins - 1;
  const int w = threadIdx.x / kWave, lane = lane_id();
  for (u32 t = threadIdx.x; t < T; t += kOneThreads) {
    s_key[0][t] = token_key<I>(a, t);
    s_place[0][t] = (u16)t;
  }
  const u32 w0 = w * a.per_wave, w1 = min(T, w0 + a.per_wave);
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits, from = pass & 1;
    const bool last = pass + 1 == a.passes;
    for (u32 i = threadIdx.x; i < bins * kOneWaves; i += kOneThreads) s_off[i >> a.bits][i & mask] = 0;
    __syncthreads();
    for (u32 t = w0 + lane; t < w1; t += kWave) atomicAdd(&s_off[w][(s_key[from][t] >> shift) & mask], 1u);
    __syncthreads();
    if (threadIdx.x < bins) {
      u32 run = 0;
      for (int i = 0; i < kOneWaves; ++i) {
        const u32 c = s_off[i][threadIdx.x];
        s_off[i][threadIdx.x] = run;
        run += c;
      }
      s_base[threadIdx.x] = run;
    }
    __syncthreads();
    scan_bins<kOneThreads>(s_base, bins, s_scan);
    for (u32 t0 = w0; t0 < w1; t0 += kWave) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the offsets that other lanes moved on
      const u32 t = t0 + lane;
      const bool here = t < w1;
      const u32 key = here ? s_key[from][t] : 0u;
      const u32 d = here ? (key >> shift) & mask : bins;
      const u64 same = same_digit(d, a.bits);
      const u32 rank = __popcll(same & ((1ull << lane) - 1));
      u32 off = 0;
      if (here && rank == 0) {
        off = s_off[w][d];
        s_off[w][d] = off + __popcll(same);
      }
      off = __shfl(off, (int)__ffsll((unsigned long long)same) - 1);
      if (here) {
        const u32 to = s_base[d] + off + rank;
        if (last) {
          a.keys_out[to] = key;
          a.places_out[to] = s_place[from][t];
        } else {
          s_key[from ^ 1][to] = key;
          s_place[from ^ 1][to] = s_place[from][t];
        }
      }
    }
    __syncthreads();
  }
}

// -------------------------------------------------------------- gradient --
struct GradArgs {
  const u32* keys;    // [T] sorted tokens, V where masked
  const u32* places;  // [T]
  const void* grad;
  void* out;
  float* part;  // [2 * chunks][D]: a chunk's sum that began before it, and one that goes on after it
  u32 T, V;
  int64_t D;
  u32 nv;     // vectors a row
  u32 slabs;  // groups of 64 vectors a row
  u32 chunk;  // places a chunk
  u32 chunks;
  u64 waves;       // chunks * slabs
  u32 join0;       // first of a launch's (chunk, slab) pairs to join
  u32 fill_rows;   // rows a zero-filling wave looks at
  float scale;
  int accumulate;
};

constexpr int kGradThreads = 256;
constexpr int kGradWaves = kGradThreads / kWave;
constexpr int kGradFlight = 8;  // row loads in flight

// Column of a lane's vector, and how many of its leading elements belong to
// the vector before it (the last vector of a row ends with the row).
template <int E>
__device__ __forceinline__ int64_t column_of(u32 vec, int64_t D, int* skip) {
  const int64_t c = (int64_t)vec * E;
  *skip = c + E <= D ? 0 : (int)(c + E - D);
  return c - *skip;
}

template <class TO, int E>
__device__ __forceinline__ void put_row(TO* p, const float (&s)[E], float scale, int accumulate, int skip) {
  Vec<TO, E> y;
  if (accumulate) y = load_vec<TO, E>(p);
#pragma unroll
  for (int e = 0; e < E; ++e) y.v[e] = from_f32<TO>(accumulate ? to_f32(y.v[e]) + s[e] * scale : s[e] * scale);
  if (skip == 0) {
    store_vec<TO, E>(p, y);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e >= skip) p[e] = y.v[e];
  }
}

// First place in the sorted keys whose key is not below v.
__device__ __forceinline__ u32 lower_bound(const u32* keys, u32 n, u32 v) {
  u32 lo = 0;
  while (n > 0) {
    const u32 half = n >> 1;
    if (keys[lo + half] < v) {
      lo += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  return lo;
}

template <class TO, int E>
__device__ __forceinline__ void fill_rows(const GradArgs& a, u64 wave) {
  const int lane = lane_id();
  const u64 v0 = wave * a.fill_rows;
  if (v0 >= a.V) return;
  const u64 v = v0 + lane;
  bool empty = false;
  if (lane < (int)a.fill_rows && v < a.V) {
    const u32 at = lower_bound(a.keys, a.T, (u32)v);
    empty = at == a.T || a.keys[at] != (u32)v;
  }
  Vec<TO, E> zero;
#pragma unroll
  for (int e = 0; e < E; ++e) zero.v[e] = from_f32<TO>(0.0f);
  for (u64 m = ballot(empty); m; m &= m - 1) {
    TO* row = (TO*)a.out + (int64_t)(v0 + __ffsll((unsigned long long)m) - 1) * a.D;
    for (u32 vec = lane; vec < a.nv; vec += kWave) {
      const int64_t c = (int64_t)vec * E;
      store_vec<TO, E>(row + (c + E <= a.D ? c : a.D - E), zero);
    }
  }
}

template <class TG, class TO, int E>
__global__ __launch_bounds__(kGradThreads) void k_grad_chunks(GradArgs a) {
  const u32 w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const u64 wave = (u64)blockIdx.x * kGradWaves + w;
  if (wave >= a.waves) {
    if (!a.accumulate) fill_rows<TO, E>(a, wave - a.waves);
    return;
  }
  const u32 slab = (u32)(wave % a.slabs), chunk = (u32)(wave / a.slabs);
  const u64 first = (u64)chunk * a.chunk;
  const u32 n = (u32)min((u64)a.chunk, (u64)a.T - first);
  const u32* keys = a.keys + first;
  const u32* places = a.places + first;
  if (keys[0] == a.V) return;  // masked places only; behind others their rows may be loaded, and are never added
  const u32 vec = slab * kWave + lane_id();
  const bool here = vec < a.nv;
  int skip;
  const int64_t col = column_of<E>(here ? vec : 0, a.D, &skip);
  const TG* grad = (const TG*)a.grad + col;
  // the token before the chunk's first and the one behind its last
  const u32 before = chunk > 0 ? keys[-1] : a.V;
  const u32 behind = first + n < a.T ? keys[n] : a.V;
  bool inside = before != keys[0];  // the running sum began in this chunk
  float s[E] = {};
  for (u32 i0 = 0; i0 < n; i0 += kGradFlight) {
    Vec<TG, E> x[kGradFlight];
    u32 k[kGradFlight + 1];
#pragma unroll
    for (int j = 0; j < kGradFlight; ++j) {
      const u32 i = i0 + j < n ? i0 + j : n - 1;
      k[j] = i0 + j < n ? keys[i] : a.V;
      x[j] = load_vec<TG, E>(grad + (int64_t)places[i] * a.D);
    }
    k[kGradFlight] = i0 + kGradFlight < n ? keys[i0 + kGradFlight] : behind;
#pragma unroll
    for (int j = 0; j < kGradFlight; ++j) {
      if (k[j] == a.V) return;  // only masked places (or none) follow
#pragma unroll
      for (int e = 0; e < E; ++e) s[e] += to_f32(x[j].v[e]);
      const bool at_end = i0 + j + 1 == n;
      const u32 next = at_end ? behind : k[j + 1];
      if (next != k[j] || at_end) {
        const bool goes_on = next == k[j];
        if (here) {
          if (inside && !goes_on) {
            put_row<TO, E>((TO*)a.out + (int64_t)k[j] * a.D + col, s, a.scale, a.accumulate, skip);
          } else {
            float* p = a.part + (int64_t)(2 * (u64)chunk + (inside ? 1 : 0)) * a.D + col;
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (e >= skip) p[e] = s[e];
          }
        }
        inside = true;
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] = 0.0f;
      }
    }
  }
}

// A token that begins in chunk c and goes on: its partial rows, added in chunk
// order by the four waves of a workgroup (a quarter of the chunks each).
template <class TO, int E>
__global__ __launch_bounds__(kGradThreads) void k_grad_join(GradArgs a) {
  __shared__ float s_sum[kGradWaves][kWave][E];
  const u32 id = a.join0 + blockIdx.x, slab = id % a.slabs, chunk = id / a.slabs;
  const u64 end = (u64)(chunk + 1) * a.chunk;  // chunk + 1 < chunks, so end < T
  const u32 key = a.keys[end - 1];
  if (key == a.V || a.keys[end] != key) return;
  if (chunk > 0 && a.keys[(u64)chunk * a.chunk - 1] == key) return;  // began in an earlier chunk
  // the last chunk that holds the token: the places behind it are >= key + 1
  const u32 stop = (u32)end + lower_bound(a.keys + end, a.T - (u32)end, key + 1);
  const u32 last = (stop - 1) / a.chunk;
  const u32 count = last - chunk;  // partial rows behind the first
  const u32 w = threadIdx.x / kWave, vec = slab * kWave + lane_id();
  const bool here = vec < a.nv;
  int skip;
  const int64_t col = column_of<E>(here ? vec : 0, a.D, &skip);
  const u32 per = (count + 1 + kGradWaves - 1) / kGradWaves;
  const u32 c0 = w * per, c1 = min(count + 1, c0 + per);
  float s[E] = {};
#pragma unroll 8
  for (u32 i = c0; i < c1; ++i) {
    const Vec<float, E> x =
        load_vec<float, E>(a.part + (int64_t)(2 * (u64)(chunk + i) + (i == 0 ? 1 : 0)) * a.D + col);
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] += x.v[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_sum[w][lane_id()][e] = s[e];
  __syncthreads();
  if (w != 0 || !here) return;
#pragma unroll
  for (int i = 1; i < kGradWaves; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] += s_sum[i][lane_id()][e];
  put_row<TO, E>((TO*)a.out + (int64_t)key * a.D + col, s, a.scale, a.accumulate, skip);
}

// --------------------------------------------------- gradient, few places --
// Up to kFewMaxT places in one launch, where the table is small too: every workgroup looks through all tokens
// for those of its own rows (at most 64), sorts their places in LDS, stably, and
// writes its rows, zeros included.  No launch waits for another, which is what
// the sorted route's three cost here: 512 places, 1,001 rows of 130:
// 19.7 -> 10.5 us, most of it the call's own time on the host.
struct FewArgs {
  const void* tokens;
  const void* grad;
  void* out;
  u32* err;
  u32 T, V;
  int64_t D;
  u32 nv;        // vectors a row
  u32 slabs;     // groups of 64 vectors a row
  u32 rows;      // a workgroup's
  u32 per_wave;  // places a wave looks through, a multiple of 64
  float scale;
  int accumulate;
};

constexpr u32 kFewMaxT = 2048;
constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / kWave;
constexpr int kFewKeys = kFewMaxT / kFewThreads;  // places a lane
static_assert(kFewMaxT <= 65536, "places are held in 16 bits");
constexpr int kFewFlight = 16;                    // row loads in flight
constexpr u32 kFewHot = 32;                       // places of a row that one wave adds alone

template <class TG, class TO, class I, int E>
__global__ __launch_bounds__(kFewThreads) void k_grad_few(FewArgs a) {
  __shared__ u16 s_place[kFewMaxT];
  __shared__ u32 s_cnt[kFewWaves][kWave];
  __shared__ u32 s_start[kWave + 1];
  __shared__ float s_sum[kFewWaves][kWave][E];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const u32 r0 = blockIdx.x * a.rows, rows = min(a.rows, a.V - r0);
  // keys: the row in this workgroup's, kWave for all others
  const u32 w0 = w * a.per_wave, w1 = min(a.T, w0 + a.per_wave);
  u32 key[kFewKeys], at[kFewKeys];
#pragma unroll
  for (int i = 0; i < kFewKeys; ++i) {
    const u32 t = w0 + i * kWave + lane;
    key[i] = kWave;
    if (t < w1) {
      const int64_t v = load_token((const I*)a.tokens, t);
      if (v >= (int64_t)a.V && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrBadInput);
      if (v >= (int64_t)r0 && v < (int64_t)(r0 + rows)) key[i] = (u32)(v - r0);
    }
  }
  s_cnt[w][lane] = 0;
#pragma unroll
  for (int i = 0; i < kFewKeys; ++i) {
    if (w0 + i * kWave < w1) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the counts that other lanes moved on
      const u64 same = same_digit(key[i], 6);
      const u32 rank = __popcll(same & ((1ull << lane) - 1));
      at[i] = key[i] < kWave ? s_cnt[w][key[i]] + rank : 0;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (key[i] < kWave && rank == 0) s_cnt[w][key[i]] = at[i] + __popcll(same);
    }
  }
  __syncthreads();
  if (w == 0) {
    u32 c = 0;
#pragma unroll
    for (int i = 0; i < kFewWaves; ++i) {
      const u32 n = s_cnt[i][lane];
      s_cnt[i][lane] = c;
      c += n;
    }
    const u32 upto = wave_inclusive_sum(c);
    s_start[lane] = upto - c;
    if (lane == kWave - 1) s_start[kWave] = upto;
  }
  __syncthreads();
  if (s_start[kWave] > 0) {
#pragma unroll
    for (int i = 0; i < kFewKeys; ++i) {
      if (key[i] < kWave) s_place[s_start[key[i]] + s_cnt[w][key[i]] + at[i]] = (u16)(w0 + i * kWave + lane);
    }
    __syncthreads();
  } else if (a.accumulate) {
    return;
  }
  const u32 vec = blockIdx.y * kWave + lane;
  const bool here = vec < a.nv;
  int skip;
  const int64_t col = column_of<E>(here ? vec : 0, a.D, &skip);
  const TG* grad = (const TG*)a.grad + col;
  TO* out = (TO*)a.out + (int64_t)r0 * a.D + col;
  // the sum of places i0 .. i1 - 1 of the sorted list, in their order
  auto add = [&](u32 i0, u32 i1, float(&s)[E]) {
    for (; i0 < i1; i0 += kFewFlight) {
      Vec<TG, E> x[kFewFlight];
#pragma unroll
      for (int j = 0; j < kFewFlight; ++j) {
        if (j < 4 || i0 + j < i1) {
          const u32 p = __builtin_amdgcn_readfirstlane(s_place[min(i0 + j, i1 - 1)]);
          x[j] = load_vec<TG, E>(grad + (int64_t)p * a.D);
        }
      }
#pragma unroll
      for (int j = 0; j < kFewFlight; ++j) {
        if (i0 + j < i1) {
#pragma unroll
          for (int e = 0; e < E; ++e) s[e] += to_f32(x[j].v[e]);
        }
      }
    }
  };
  for (u32 r = w; r < rows; r += kFewWaves) {
    const u32 i0 = __builtin_amdgcn_readfirstlane(s_start[r]), i1 = __builtin_amdgcn_readfirstlane(s_start[r + 1]);
    if (i1 - i0 > kFewHot || (i1 == i0 && a.accumulate)) continue;
    float s[E] = {};
    add(i0, i1, s);
    // a row without places is +0, whatever the scale's sign
    if (here) put_row<TO, E>(out + (int64_t)r * a.D, s, i1 == i0 ? 1.0f : a.scale, a.accumulate, skip);
  }
  if (s_start[kWave] <= kFewHot) return;
  for (u32 r = 0; r < rows; ++r) {  // rows of many places: an eighth of them a wave
    const u32 i0 = __builtin_amdgcn_readfirstlane(s_start[r]), i1 = __builtin_amdgcn_readfirstlane(s_start[r + 1]);
    if (i1 - i0 <= kFewHot) continue;
    const u32 per = (i1 - i0 + kFewWaves - 1) / kFewWaves, b = min(i1, i0 + w * per);
    float s[E] = {};
    add(b, min(i1, b + per), s);
#pragma unroll
    for (int e = 0; e < E; ++e) s_sum[w][lane][e] = s[e];
    __syncthreads();
    if (w == 0 && here) {
#pragma unroll
      for (int i = 1; i < kFewWaves; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] += s_sum[i][lane][e];
      put_row<TO, E>(out + (int64_t)r * a.D, s, a.scale, a.accumulate, skip);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host --
// A launch of 2^32 threads or more is refused by the runtime, after what came
// before it is enqueued.
static u64 most_blocks(int threads) { return 0xFFFFFFFFull / threads; }

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Elements a lane moves at once: 16 bytes of the wider type; single elements
// where a row is shorter than that.
static int vector_of(int64_t D, tgs_dtype a, tgs_dtype b) {
  const int e = dtype_bytes(a) == 2 && dtype_bytes(b) == 2 ? 8 : 4;
  return D >= e ? e : 1;
}

// Rows of a workgroup of k_grad_few: enough groups to give all compute units work.
// With at least 64, 128, 256, 512 and 1,024 groups 1,024 places in 8,000 rows of
// 130 take 20, 14, 11, 9.4 and 9.5 us, 512 in 30,000 rows of 64 14, 14, 14, 9.6
// and 8.6, 512 in 4,000 rows of 512 10, 7.5, 7.4, 8.3 and 8.3.  Two rows a group
// instead of four: 512 in 1,001 rows of 1,024 9.3 and 7.6, in 4,000 of 512 12.3 and
// 8.3, though 2,048 in 1,001 of 130 8.5 and 11.6.
static u32 few_rows(int64_t V) {
  u32 rows = kWave;
  while (rows > 4 && V < (int64_t)rows * 512) rows /= 2;
  return rows;
}
static u32 few_groups(int64_t V) { return (u32)((V + few_rows(V) - 1) / few_rows(V)); }

struct GradPlan {
  int E, bits, passes;
  u32 nv, slabs, chunk, chunks, sort_blocks, per_wave;
  bool few;  // one launch
  bool one;  // one workgroup sorts
  size_t keys[2], places[2], hist, part, total;
};

static bool grad_plan(int64_t T, int64_t V, int64_t D, tgs_dtype tg, tgs_dtype to, GradPlan* p) {
  if (T < 0 || T > INT32_MAX || V < 1 || V > INT32_MAX || D < 1 || D > INT32_MAX) return false;
  p->E = vector_of(D, tg, to);
  // 16-bit gradients to fp32 rows: eight a lane where that leaves fewer groups of 64 lanes a row, and waves
  // enough.  With 25,000 rows, accumulated, four against eight: 2^26 values in rows of 512 103 and 86 us, of 2,048
  // 103 and 81; 2^28 in rows of 2,048 284 and 251.  At 2^25 they are within a tenth of each other (rows of 768 76
  // and 77, written 73 and 75), at 2^24, where eight halves the chunks, written 53 and 61.  Rows of up to 256 would
  // leave half the lanes idle: 2^26 in rows of 64 204 and 215, 2^27 in rows of 256 163 and 171.
  if (p->E == 4 && dtype_bytes(tg) == 2 && D > 256 && T > kFewMaxT && T >= ((int64_t)1 << 26) / D) p->E = 8;
  p->nv = (u32)((D + p->E - 1) / p->E);
  p->slabs = (p->nv + kWave - 1) / kWave;
  // chunks: long enough that partial rows are few, short enough that about
  // 4096 waves (four a SIMD) have work.  For 1,024, 2,048, 4,096, 8,192 and 16,384
  // 16,384 places of 1,024 take 85, 62, 50, 48 and 48 us, 131,072 of 256 103, 103,
  // 78, 69 and 79, of 2,048 302, 303, 302, 302 and 330; each doubling doubles the
  // partial rows' memory too
  p->chunk = 64;
  while (p->chunk > 8 && (u64)T / p->chunk * p->slabs < 4096) p->chunk >>= 1;
  p->chunks = (u32)(((u64)T + p->chunk - 1) / p->chunk);
  int bits = 1;
  while (((u64)1 << bits) < (u64)V + 1) ++bits;  // keys 0 .. V
  p->passes = (bits + kDigitBits - 1) / kDigitBits;
  p->bits = (bits + p->passes - 1) / p->passes;
  p->one = T <= kOneMaxT;
  const u32 groups = few_groups(V);
  // every workgroup looks through all tokens: few of either (1,024 places: 12 against 19 us with 251 workgroups,
  // 20 against 19 with 2,000; 2,048 places: 15 against 20 with 251, 30 against 25 with 2,500)
  const u64 looks = (u64)groups * p->slabs;
  p->few = T <= kFewMaxT && looks <= 2500 && looks * (u64)T <= 2100000;
  if (p->few) {
    p->total = kWorkspaceHeader;
    return true;
  }
  const u32 waves = p->one ? kOneWaves : kTokenWaves;
  u64 blocks = p->one ? 1 : ((u64)T + 2047) / 2048;
  if (blocks > kTokenBlocks) blocks = kTokenBlocks;
  p->sort_blocks = (u32)std::max<u64>(blocks, 1);
  const u64 parts = (u64)p->sort_blocks * waves, per = ((u64)T + parts - 1) / parts;
  p->per_wave = (u32)((per + kWave - 1) / kWave * kWave);
  size_t at = kWorkspaceHeader;
  for (int i = 0; i < 2; ++i) {
    p->keys[i] = at;
    at += up256((size_t)T * 4);
    p->places[i] = at;
    at += up256((size_t)T * 4);
  }
  p->hist = at;
  at += up256(((size_t)kTokenBlocks << kDigitBits) * 4);
  p->part = at;
  at += up256((size_t)p->chunks * 2 * (size_t)D * 4);
  p->total = at;
  return true;
}

template <class F>
static void with_token_dtype(tgs_dtype t, F&& f) {
  if (t == TGS_INT32) f((int32_t*)nullptr);
  else f((int64_t*)nullptr);
}

static tgs_status check_common(const char* what, const void* tokens, tgs_dtype tokens_dtype, int64_t T, int64_t V,
                               int64_t D, tgs_dtype a_dtype, tgs_dtype b_dtype, float scale, const void* workspace,
                               size_t workspace_bytes, size_t need) {
  if (T < 0 || T > INT32_MAX) return fail(TGS_EINVAL, "%s: T=%lld outside [0, 2^31-1]", what, (long long)T);
  if (V < 1 || V > INT32_MAX) return fail(TGS_EINVAL, "%s: V=%lld outside [1, 2^31-1]", what, (long long)V);
  if (D < 1 || D > INT32_MAX) return fail(TGS_EINVAL, "%s: D=%lld outside [1, 2^31-1]", what, (long long)D);
  if (!is_token_dtype(tokens_dtype)) return fail(TGS_EINVAL, "%s: tokens must be int32 or int64", what);
  if (!is_float_dtype(a_dtype) || !is_float_dtype(b_dtype))
    return fail(TGS_EINVAL, "%s: values must be fp32, bf16 or fp16", what);
  if (!(scale - scale == 0.0f)) return fail(TGS_EINVAL, "%s: scale is not finite", what);
  if (T > 0 && !tokens) return fail(TGS_EINVAL, "%s: null tokens", what);
  if (((uintptr_t)tokens & (dtype_bytes(tokens_dtype) - 1)) != 0)
    return fail(TGS_EINVAL, "%s: tokens not aligned to their type", what);
  if (!workspace) return fail(TGS_EINVAL, "%s: null workspace", what);
  if (((uintptr_t)workspace & 255u) != 0) return fail(TGS_EINVAL, "%s: workspace not 256-byte aligned", what);
  if (workspace_bytes < need)
    return fail(TGS_EWORKSPACE, "%s: workspace %zu bytes, need %zu", what, workspace_bytes, need);
  return TGS_OK;
}

static tgs_status check_array(const char* what, const char* name, const void* p, tgs_dtype t, bool needed) {
  if (needed && !p) return fail(TGS_EINVAL, "%s: null %s", what, name);
  if (((uintptr_t)p & (dtype_bytes(t) - 1)) != 0)
    return fail(TGS_EINVAL, "%s: %s not aligned to its type", what, name);
  return TGS_OK;
}

}  // namespace tgs

using namespace tgs;

extern "C" size_t tgs_embedding_lookup_workspace_bytes(int64_t T) {
  return T < 0 || T > INT32_MAX ? 0 : kWorkspaceHeader;
}

extern "C" tgs_status tgs_embedding_lookup(const void* tokens, tgs_dtype tokens_dtype, int64_t T, const void* table,
                                           tgs_dtype table_dtype, int64_t V, int64_t D, float scale, void* out,
                                           tgs_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
  const char* what = "embedding_lookup";
  tgs_status st = check_common(what, tokens, tokens_dtype, T, V, D, table_dtype, out_dtype, scale, workspace,
                               workspace_bytes, kWorkspaceHeader);
  if (st != TGS_OK) return st;
  if ((st = check_array(what, "table", table, table_dtype, T > 0)) != TGS_OK) return st;
  if ((st = check_array(what, "out", out, out_dtype, T > 0)) != TGS_OK) return st;
  const size_t out_bytes = (size_t)T * (size_t)D * dtype_bytes(out_dtype);
  if (overlaps(out, out_bytes, tokens, (size_t)T * dtype_bytes(tokens_dtype)) ||
      overlaps(out, out_bytes, table, (size_t)V * (size_t)D * dtype_bytes(table_dtype)) ||
      overlaps(out, out_bytes, workspace, workspace_bytes))
    return fail(TGS_EINVAL, "%s: out overlaps an input or the workspace", what);
  if (T == 0) return TGS_OK;
  const int E = vector_of(D, table_dtype, out_dtype);
  LookupArgs a{};
  a.tokens = tokens;
  a.table = table;
  a.out = out;
  a.err = (u32*)workspace;
  a.T = T;
  a.V = V;
  a.D = D;
  a.nv = (u32)((D + E - 1) / E);
  a.total = (u64)T * a.nv;
  a.scale = scale;
  const u64 blocks = (a.total + kLookupThreads * kLookupUnroll - 1) / (kLookupThreads * kLookupUnroll);
  if (blocks > most_blocks(kLookupThreads)) return fail(TGS_EINVAL, "%s: T * D too large", what);
  with_token_dtype(tokens_dtype, [&](auto* i) {
    with_float_dtype(table_dtype, [&](auto* ti) {
      with_float_dtype(out_dtype, [&](auto* to) {
        using I = std::remove_pointer_t<decltype(i)>;
        using TI = std::remove_pointer_t<decltype(ti)>;
        using TO = std::remove_pointer_t<decltype(to)>;
        constexpr int W = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4;
        if (E != W) hipLaunchKernelGGL((k_lookup<TI, TO, I, 1, false>), dim3((u32)blocks), dim3(kLookupThreads), 0, stream, a);
        else if (out_bytes > kStreamingBytes) hipLaunchKernelGGL((k_lookup<TI, TO, I, W, true>), dim3((u32)blocks), dim3(kLookupThreads), 0, stream, a);
        else hipLaunchKernelGGL((k_lookup<TI, TO, I, W, false>), dim3((u32)blocks), dim3(kLookupThreads), 0, stream, a);
      });
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TGS_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
  return TGS_OK;
}

extern "C" size_t tgs_embedding_grad_workspace_bytes(int64_t T, int64_t V, int64_t D, tgs_dtype grad_dtype,
                                                     tgs_dtype out_dtype) {
  GradPlan p;
  if (!is_float_dtype(grad_dtype) || !is_float_dtype(out_dtype) || !grad_plan(T, V, D, grad_dtype, out_dtype, &p))
    return 0;
  return p.total;
}

extern "C" tgs_status tgs_embedding_grad(const void* tokens, tgs_dtype tokens_dtype, int64_t T, const void* grad,
                                         tgs_dtype grad_dtype, int64_t V, int64_t D, float scale, void* out,
                                         tgs_dtype out_dtype, int32_t accumulate, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream) {
  const char* what = "embedding_grad";
  GradPlan p{};
  size_t need = 0;
  if (is_float_dtype(grad_dtype) && is_float_dtype(out_dtype) && grad_plan(T, V, D, grad_dtype, out_dtype, &p))
    need = p.total;
  tgs_status st = check_common(what, tokens, tokens_dtype, T, V, D, grad_dtype, out_dtype, scale, workspace,
                               workspace_bytes, need);
  if (st != TGS_OK) return st;
  if ((st = check_array(what, "grad", grad, grad_dtype, T > 0)) != TGS_OK) return st;
  if ((st = check_array(what, "out", out, out_dtype, true)) != TGS_OK) return st;
  const size_t out_bytes = (size_t)V * (size_t)D * dtype_bytes(out_dtype);
  if (overlaps(out, out_bytes, tokens, (size_t)T * dtype_bytes(tokens_dtype)) ||
      overlaps(out, out_bytes, grad, (size_t)T * (size_t)D * dtype_bytes(grad_dtype)) ||
      overlaps(out, out_bytes, workspace, workspace_bytes))
    return fail(TGS_EINVAL, "%s: out overlaps an input or the workspace", what);
  if (T == 0 && accumulate) return TGS_OK;
  if (p.few) {
    FewArgs f{};
    f.tokens = tokens;
    f.grad = grad;
    f.out = out;
    f.err = (u32*)workspace;
    f.T = (u32)T;
    f.V = (u32)V;
    f.D = D;
    f.nv = p.nv;
    f.slabs = p.slabs;
    f.scale = scale;
    f.accumulate = accumulate != 0;
    f.per_wave = (u32)((T + kFewThreads - 1) / kFewThreads) * kWave;
    f.rows = few_rows(V);
    const dim3 grid(few_groups(V), p.slabs);
    with_token_dtype(tokens_dtype, [&](auto* i) {
      with_float_dtype(grad_dtype, [&](auto* tg) {
        with_float_dtype(out_dtype, [&](auto* to) {
          using TG = std::remove_pointer_t<decltype(tg)>;
          using TO = std::remove_pointer_t<decltype(to)>;
          using TI = std::remove_pointer_t<decltype(i)>;
          constexpr int W = sizeof(TG) == 2 && sizeof(TO) == 2 ? 8 : 4;
          if (p.E == W) hipLaunchKernelGGL((k_grad_few<TG, TO, TI, W>), grid, dim3(kFewThreads), 0, stream, f);
          else hipLaunchKernelGGL((k_grad_few<TG, TO, TI, 1>), grid, dim3(kFewThreads), 0, stream, f);
        });
      });
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(TGS_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    return TGS_OK;
  }
  char* ws = (char*)workspace;
  GradArgs a{};
  a.grad = grad;
  a.out = out;
  a.part = (float*)(ws + p.part);
  a.T = (u32)T;
  a.V = (u32)V;
  a.D = D;
  a.nv = p.nv;
  a.slabs = p.slabs;
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  a.waves = (u64)p.chunks * p.slabs;
  // about 32 KB of zeros a wave, 64 rows at most (one binary search a lane)
  a.fill_rows = (u32)std::max<size_t>(1, std::min<size_t>(kWave, 32768 / ((size_t)D * dtype_bytes(out_dtype))));
  a.scale = scale;
  a.accumulate = accumulate != 0;
  const u64 fill = accumulate ? 0 : ((u64)V + a.fill_rows - 1) / a.fill_rows;
  const u64 blocks = (a.waves + fill + kGradWaves - 1) / kGradWaves;
  if (blocks > most_blocks(kGradThreads)) return fail(TGS_EINVAL, "%s: T * D or V * D too large", what);
  // a workgroup each, four times as many as chunk workgroups: past 2^30 places in several launches
  const u32 joins = p.chunks > 1 ? (p.chunks - 1) * p.slabs : 0;
  SortArgs s{};
  s.tokens = tokens;
  s.hist = (u32*)(ws + p.hist);
  s.err = (u32*)workspace;
  s.T = (u32)T;
  s.V = (u32)V;
  s.per_wave = p.per_wave;
  s.bits = p.bits;
  s.passes = p.passes;
  int last = 0;
  if (T > 0) {
    with_token_dtype(tokens_dtype, [&](auto* i) {
      using I = std::remove_pointer_t<decltype(i)>;
      if (p.one) {
        s.keys_out = (u32*)(ws + p.keys[0]);
        s.places_out = (u32*)(ws + p.places[0]);
        hipLaunchKernelGGL((k_sort_one<I>), dim3(1), dim3(kOneThreads), 0, stream, s);
        return;
      }
      for (int pass = 0; pass < p.passes; ++pass) {
        last = pass & 1;
        s.shift = pass * p.bits;
        s.keys_in = (const u32*)(ws + p.keys[last ^ 1]);
        s.places_in = (const u32*)(ws + p.places[last ^ 1]);
        s.keys_out = (u32*)(ws + p.keys[last]);
        s.places_out = (u32*)(ws + p.places[last]);
        if (pass == 0) {
          hipLaunchKernelGGL((k_sort_count<I, true>), dim3(p.sort_blocks), dim3(kTokenThreads), 0, stream, s);
          hipLaunchKernelGGL((k_sort_move<I, true>), dim3(p.sort_blocks), dim3(kTokenThreads), 0, stream, s);
        } else {
          hipLaunchKernelGGL((k_sort_count<int32_t, false>), dim3(p.sort_blocks), dim3(kTokenThreads), 0, stream, s);
          hipLaunchKernelGGL((k_sort_move<int32_t, false>), dim3(p.sort_blocks), dim3(kTokenThreads), 0, stream, s);
        }
      }
    });
  }
  a.keys = (const u32*)(ws + p.keys[last]);
  a.places = (const u32*)(ws + p.places[last]);
  with_float_dtype(grad_dtype, [&](auto* tg) {
    with_float_dtype(out_dtype, [&](auto* to) {
      using TG = std::remove_pointer_t<decltype(tg)>;
      using TO = std::remove_pointer_t<decltype(to)>;
      auto launch = [&](auto width) {
        constexpr int E = decltype(width)::value;
        hipLaunchKernelGGL((k_grad_chunks<TG, TO, E>), dim3((u32)blocks), dim3(kGradThreads), 0, stream, a);
        for (a.join0 = 0; a.join0 < joins;) {
          const u32 n = (u32)std::min<u64>(joins - a.join0, most_blocks(kGradThreads));
          hipLaunchKernelGGL((k_grad_join<TO, E>), dim3(n), dim3(kGradThreads), 0, stream, a);
          a.join0 += n;
        }
      };
      if (p.E == 1) launch(std::integral_constant<int, 1>{});
      else if constexpr (sizeof(TG) == 4) launch(std::integral_constant<int, 4>{});
      else if constexpr (sizeof(TO) == 2) launch(std::integral_constant<int, 8>{});
      else if (p.E == 8) launch(std::integral_constant<int, 8>{});
      else launch(std::integral_constant<int, 4>{});
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TGS_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
  return TGS_OK;
}
