// One pass over a row of logits, and what is made of it.
//
// With d = (x - r) / temperature for a reference score r, a thread keeps the
// sum of e^d and (for the entropy) of d e^d over its elements, relative to a
// reference of its own: its first vector's largest score, replaced only where
// a later score is more than 2^24 times as probable.  That is one exponential
// a value and no running rescale; a row's sums are joined at its largest score.
#pragma once

#include <limits>

#include "tgs_rows.h"

namespace tgs {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
constexpr float kLowest = -3.402823466385288598117e+38f;
constexpr float kInf = __builtin_huge_valf();
constexpr float kRescale = 24.0f;  // powers of two above the reference at which it is replaced

struct Logits {
  const void* p;
  int64_t ld;  // elements from row to row
  u32 V;
  float c2;   // log2(e) / temperature
  float inv;  // 1 / temperature
};

template <class T>
constexpr int kLogitsVector = 16 / sizeof(T);

// A thread's share: sums relative to `ref`, the largest score and the first
// vector that holds it (counted in the thread's own).
struct Share {
  float ref = kLowest, s = 0.0f, w = 0.0f, top = -kInf;
  u32 at = 0;
  float part = -kInf;  // the largest score of the present part
};

// For the search for a row's largest scores its vectors are cut into parts, whose
// largest score each thread leaves behind.
constexpr u32 kParts = 8;
constexpr u32 kUnroll = 4;  // vectors that a thread loads at once

// How elements [c0, c1) of a row lie: vectors of E elements, NT to a step.
struct Span {
  u32 c0, c1;
  template <int STEP>
  __device__ __forceinline__ u32 rounds() const { return (c1 - c0 + kUnroll * STEP - 1) / (kUnroll * STEP); }
  // vectors of a thread that make a part
  template <int STEP>
  __device__ __forceinline__ u32 part() const { return (rounds<STEP>() + kParts - 1) / kParts * kUnroll; }
};

template <int E, bool ENTROPY, bool TOP>
__device__ __forceinline__ void take(const float (&x)[E], u32 j, float c2, Share& h) {
  float top = -kInf;
#pragma unroll
  for (int e = 0; e < E; ++e) top = fmaxf(top, x[e]);
  if constexpr (TOP) {
    if (top > h.top) h.at = j;
    h.part = fmaxf(h.part, top);
  }
  h.top = fmaxf(h.top, top);
  const float step = (h.ref - top) * c2;
  if (step < -kRescale) {
    const float f = __builtin_amdgcn_exp2f(step);
    if (f == 0.0f) {
      h.s *= 0.0f;  // a NaN stays one
      h.w = 0.0f;
    } else {
      if constexpr (ENTROPY) h.w = f * fmaf(h.s, step, h.w);
      h.s *= f;
    }
    h.ref = top;
  }
  float s = 0.0f, w = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float d = (x[e] - h.ref) * c2, p = __builtin_amdgcn_exp2f(d);
    s += p;
    if constexpr (ENTROPY) w = fmaf(p, fmaxf(d, -1024.0f), w);  // 0 where p is, not 0 times infinity
  }
  h.s += s;
  if constexpr (ENTROPY) h.w += w;
}

// Elements [c0, c1) of a row by NT threads; thread t takes the vectors that
// start at c0 + (t + j NT) E.  The last vector is moved back to end with the
// row, so that it too is one load without a branch; what it has in common with
// the one before counts as -inf.  parts: with TOP, [kParts][NT] largest scores.
// kept: where the whole vectors of the first round of a row from column 0 on are
// left, in order.
template <class T, int NT, bool ENTROPY, bool TOP, bool KEEP = false>
__device__ __forceinline__ Share row_pass(const T* row, const Span& sp, float c2, float* parts,
                                          Vec<T, kLogitsVector<T>>* kept = nullptr) {
  constexpr int E = kLogitsVector<T>, U = kUnroll;
  constexpr u32 kStep = NT * E;
  const u32 c0 = sp.c0, c1 = sp.c1;
  Share h;
  if (c1 - c0 < (u32)E) {
    if (threadIdx.x == 0) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = c0 + e < c1 ? to_f32(row[c0 + e]) : -kInf;
      take<E, ENTROPY, TOP>(x, 0, c2, h);
    }
    if constexpr (TOP) parts[threadIdx.x] = h.part;
    return h;
  }
  u32 c = c0 + threadIdx.x * E, j = 0, part = 0, end = TOP ? sp.part<kStep>() : 0;
  for (u32 rest = c1 - c0; rest >= U * kStep; rest -= U * kStep, c += U * kStep) {
    Vec<T, E> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load_vec<T, E>(row + c + u * kStep);
    if constexpr (KEEP) {
      if (j == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) kept[u * NT + threadIdx.x] = v[u];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = to_f32(v[u].v[e]);
      take<E, ENTROPY, TOP>(x, j + u, c2, h);
    }
    j += U;
    if constexpr (TOP) {
      if (j == end) {
        parts[part++ * NT + threadIdx.x] = h.part;
        h.part = -kInf;
        end += sp.part<kStep>();
      }
    }
  }
  Vec<T, E> v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c + u * kStep < c1) v[u] = load_vec<T, E>(row + min(c + u * kStep, c1 - E));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const u32 at = c + u * kStep;
    if (at >= c1) continue;
    const u32 skip = at - min(at, c1 - E);
    if constexpr (KEEP) {
      if (j == 0 && skip == 0) kept[u * NT + threadIdx.x] = v[u];
    }
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = (u32)e >= skip ? to_f32(v[u].v[e]) : -kInf;
    take<E, ENTROPY, TOP>(x, j + u, c2, h);
  }
  if constexpr (TOP) {
    if (part < kParts) parts[part * NT + threadIdx.x] = h.part;
  }
  return h;
}

// A row's (or a slice's) sums relative to its largest score m; m = -inf where
// every score is, and then s = 0.  log_s = log(s).
struct RowSums {
  float m, s, w;
};

template <int NT>
__device__ __forceinline__ RowSums join_shares(const Share& h, float c2, float* lds) {
  float m[1] = {h.top};
  group_reduce<Max, NT>(m, lds);
  float x[2] = {0.0f, 0.0f};
  if (h.s != 0.0f) {
    const float step = (h.ref - m[0]) * c2, f = __builtin_amdgcn_exp2f(step);
    x[0] = h.s * f;
    x[1] = f == 0.0f ? 0.0f : f * fmaf(h.s, step, h.w);
  }
  group_reduce<Sum, NT>(x, lds + NT / kWave);
  return RowSums{m[0], x[0], x[1]};
}
template <int NT>
constexpr int kJoinLds = 3 * (NT / kWave);

// ------------------------------------------------------ largest entries --
// Key of an entry: larger for a larger score, then for a lower index.  -0 counts
// as +0 and a NaN above infinity.  0 stands for no entry.
__device__ __forceinline__ u32 score_order(float x) {
  const u32 b = __float_as_uint(x + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ u64 entry_key(float x, u32 index) { return (u64)score_order(x) << 32 | (0xFFFFFFFEu - index); }
__device__ __forceinline__ u32 key_index(u64 key) { return 0xFFFFFFFEu - (u32)key; }
__device__ __forceinline__ float key_score(u64 key) {
  const u32 o = (u32)(key >> 32);
  if (o == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

constexpr int kMostTop = 64;
constexpr u32 kFewTop = 12;

template <int NT>
struct TopLds {
  static constexpr int kList = NT == kWave ? 512 : 1024;
  u64 keys[NT];
  union {
    u64 list[kList];
    float parts[kParts * NT];  // given up once the owners are known
  };
  u64 out[kMostTop];
  u32 larger[NT];
  u16 owner[kParts * NT];
  u32 owners, listed;
};

// The k <= 64 largest keys of what the threads hold, descending, to s.out (0
// where there are fewer).  `bound` is a key no larger than the thread's largest
// one (0: it holds none); entries_of(owner, j, f) calls f(scores, index of the
// first, skip, n) for item j of thread `owner`, of `count` items at most, whose
// entries are scores skip .. n - 1.  With PARTED thread
// t's items of part i, i each .. (i + 1) each - 1, hold scores up to s.parts[i][t].
//
// No key below the least of k groups' bounds, of 64, is among the k largest.  Few
// groups are found one by one, up to 12, more by counting: 65,536 rows of 1,000 in
// bf16 with 5 alternatives take 89 us, all counted 98.
// The few threads whose own bound reaches it hold all keys that do; their items,
// of parts that reach it, are looked at by the whole workgroup, and the few keys
// found are ranked by counting.  (Looked at by their own threads, a vector's eight
// entries by a few lanes of every wave, 128,000 scores with 20 alternatives took
// 14.7 us where they took 10.9 in this way; the whole kernel now takes 12.3.)  Where they are too many (an order made for it) or
// `all` is set (bounds that NaNs passed by), k rounds over everything find the
// largest below the last.
//
// offer_bound comes first, and a barrier between the two.
template <int NT>
__device__ __forceinline__ void offer_bound(TopLds<NT>& s, u64 bound) {
  const u32 t = threadIdx.x;
  s.keys[t] = bound;
  if (t < kMostTop) s.out[t] = 0;
  if (t == 0) s.owners = s.listed = 0;
}

template <int NT, bool PARTED, class F>
__device__ __forceinline__ void largest_keys(TopLds<NT>& s, u64 bound, u32 count, u32 each, u32 k, bool all,
                                             F&& entries_of) {
  constexpr int W = NT / kWave;
  const u32 t = threadIdx.x, lane = t % kWave, wave = t / kWave;
  // group g: lane g of every wave
  u64 g = s.keys[lane];
#pragma unroll
  for (int i = kWave; i < NT; i += kWave) g = max(g, s.keys[lane + i]);
  const u32 order = (u32)(g >> 32);
  bool taken = false;  // k groups, none of them a lower order's than one left out
  if (k <= kFewTop) {
    u32 rest = order + 1;  // 0 where taken
    for (u32 r = 0; r < k; ++r) {
      const u32 best = wave_max(rest);
      if ((int)lane == __builtin_ctzll(ballot(rest == best))) {
        taken = true;
        rest = 0;
      }
    }
  } else {
    // by counting, the lane in place of the order's last bits
    const u32 rough = (order & ~63u) | (kWave - 1 - lane);
    u32 larger = 0;
#pragma unroll
    for (int i = 0; i < kWave / W; ++i) larger += (u32)__builtin_amdgcn_readlane((int)rough, wave * (kWave / W) + i) > rough;
    if constexpr (W > 1) {
      s.larger[t] = larger;
      __syncthreads();
      larger = 0;
#pragma unroll
      for (int i = 0; i < NT; i += kWave) larger += s.larger[lane + i];
    }
    taken = larger < k;
  }
  // the least of them; 0 where fewer groups hold any
  const u32 least_order = wave_min(taken ? order : ~0u);
  const u32 least_low = wave_min(taken && order == least_order ? (u32)g : ~0u);
  const u64 least = least_order ? (u64)least_order << 32 | least_low : 0;
  if (!all) {
    if (bound >= least && bound != 0) {
      if constexpr (PARTED) {
        for (u32 i = 0; i * each < count; ++i)
          if (score_order(s.parts[i * NT + t]) >= (u32)(least >> 32)) s.owner[atomicAdd(&s.owners, 1u)] = (u16)(i * NT + t);
      } else {
        s.owner[atomicAdd(&s.owners, 1u)] = (u16)t;
      }
    }
    __syncthreads();
    // least as a score and an index: everything where fewer than k groups hold any
    const bool some = least != 0;
    const float floor = some ? key_score(least) : -kInf;
    const u32 until = some ? key_index(least) : ~0u, items = s.owners * each;
    for (u32 i = t; i < items; i += NT) {
      const u32 o = i / each, owner = s.owner[o];
      entries_of(owner % NT, owner / NT * each + (i - o * each), [&](const auto& x, u32 index, u32 skip, u32 n) {
        constexpr u32 N = sizeof(x) / sizeof(x[0]);
        u32 hits = 0;
#pragma unroll
        for (u32 e = 0; e < N; ++e)
          if (e >= skip && e < n && (x[e] > floor || (x[e] == floor && index + e <= until))) hits |= 1u << e;
        if (!hits) return;
        u32 at = atomicAdd(&s.listed, (u32)__builtin_popcount(hits));
#pragma unroll
        for (u32 e = 0; e < N; ++e) {
          if (!(hits >> e & 1)) continue;
          if (at < TopLds<NT>::kList) s.list[at] = entry_key(x[e], index + e);
          ++at;
        }
      });
    }
    __syncthreads();
  }
  const u32 n = s.listed;
  if (!all && n <= TopLds<NT>::kList) {
    for (u32 i = t; i < n; i += NT) {
      const u64 mine = s.list[i];
      u32 rank = 0;
#pragma unroll 8
      for (u32 o = 0; o < n; ++o) rank += s.list[o] > mine;
      if (rank < k) s.out[rank] = mine;
    }
  } else {
    u64 last = ~(u64)0;
    for (u32 r = 0; r < k; ++r) {
      u64 best = 0;
      for (u32 j = 0; j < count; ++j)
        entries_of(t, j, [&](const auto& x, u32 index, u32 skip, u32 m) {
          constexpr u32 N = sizeof(x) / sizeof(x[0]);
#pragma unroll
          for (u32 e = 0; e < N; ++e) {
            const u64 key = entry_key(x[e], index + e);
            if (e >= skip && e < m && key < last && key > best) best = key;
          }
        });
      best = wave_max64(best);
      __syncthreads();
      if (lane_id() == 0) s.keys[t / kWave] = best;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NT / kWave; ++i) best = max(best, s.keys[i]);
      if (t == 0) s.out[r] = best;
      last = best;
    }
  }
  __syncthreads();
}

}  // namespace tgs
