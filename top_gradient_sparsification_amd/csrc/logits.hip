// Losses on rows of logits on gfx950: log probabilities of given tokens with
// entropy and top alternatives, distillation from a teacher's top logits, and
// the gradients of both.
//
//   p = softmax(z / tau) = e^((z - m) / tau) / s,  s = sum e^((z - m) / tau)
//   log p(j) = (z_j - m) / tau - log s
//   H = log s - sum of e^d d / s with d = (z - m) / tau
//   L = sum over slots of q (log q - log p(index)), q = softmax(teacher / tau)
//   gradients: of log p(j)  (onehot(j) - p) / tau
//              of H         -p (log p + H) / tau
//              of L         (p - q) / tau
//
// Bound by HBM: a row is read once on the way out, read and written once on
// the way back.  8,192 rows of 64,000 in bf16: 181 us for the log probabilities
// alone (5.8 TB/s), 188 with the entropy, 197 with 5 alternatives too, 183 for a
// distillation with 64 slots; gradients of 8,192 rows of 32,000 185 to 191 us (5.5 to
// 5.8 TB/s).  An exponential costs a SIMD four cycles where an addition costs one, so
// the pass is kept to one a value and some eight operations besides: the arithmetic
// of bf16 with the entropy is close to what the memory leaves time for.
#include <type_traits>

#include "tgs_softmax.h"

namespace tgs {

constexpr int kRowThreads = 256;
constexpr int kMostSlices = 64;  // of a row, that a wave joins

// What one slice of a row leaves for the join: its sums, and behind all of them
// its largest keys.
struct SliceSums {
  float m, s, w, pad;
};

struct Split {
  u32 slices;  // a row's; 1: nothing is joined
  u32 length;  // elements of a slice, a multiple of every vector
  SliceSums* sums;  // [row][slice]
  u64* keys;        // [row][slice][top]
  u32* arrived;     // [row] workgroups that are done, 0 between calls
};

// Stores a slice's sums where every workgroup of its row sees them.
__device__ __forceinline__ void store_slice(const Split& split, int64_t row, u32 slice, const RowSums& r) {
  float* p = &split.sums[row * split.slices + slice].m;
  st_agent_f32(p, r.m);
  st_agent_f32(p + 1, r.s);
  st_agent_f32(p + 2, r.w);
}

// Whether this workgroup is the last of its row to come here: what the others
// stored at device scope before is there to be loaded at device scope.
__device__ __forceinline__ bool last_of_row(const Split& split, int64_t row, u32* lds) {
  wait_all_memory();
  __syncthreads();
  if (threadIdx.x == 0) {
    const u32 before = add_agent_relaxed(split.arrived + row, 1u);
    if (before == split.slices - 1) st_agent(split.arrived + row, 0u);
    *lds = before;
  }
  __syncthreads();
  return *lds == split.slices - 1;
}

// A row's sums from its slices' (64 at most), by the first wave; every thread gets them.
__device__ __forceinline__ RowSums join_slices(const Split& split, int64_t row, float c2, float* lds) {
  if (threadIdx.x < kWave) {
    RowSums p{-kInf, 0.0f, 0.0f};
    if (threadIdx.x < split.slices) {
      const u32* q = (const u32*)&split.sums[row * split.slices + threadIdx.x];
      p = RowSums{__uint_as_float(ld_agent(q)), __uint_as_float(ld_agent(q + 1)), __uint_as_float(ld_agent(q + 2))};
    }
    const float m = lanes_reduce<Max, kWave>(p.m);
    float s = 0.0f, w = 0.0f;
    if (p.s != 0.0f) {
      const float step = (p.m - m) * c2, f = p.m == m ? 1.0f : __builtin_amdgcn_exp2f(step);
      s = p.s * f;
      w = p.m == m ? p.w : f == 0.0f ? 0.0f : f * fmaf(p.s, step, p.w);
    }
    s = lanes_reduce<Sum, kWave>(s);
    w = lanes_reduce<Sum, kWave>(w);
    if (threadIdx.x == 0) {
      lds[0] = m;
      lds[1] = s;
      lds[2] = w;
    }
  }
  __syncthreads();
  return RowSums{lds[0], lds[1], lds[2]};
}

__device__ __forceinline__ int64_t load_index(const void* p, bool wide, int64_t i) {
  return wide ? ((const int64_t*)p)[i] : (int64_t)((const int32_t*)p)[i];
}

// The index, -1 where it stands for none; one past the row is reported.
__device__ __forceinline__ int load_entry(const void* p, bool wide, int64_t i, u32 V, u32* err) {
  const int64_t v = load_index(p, wide, i);
  if (v >= (int64_t)V) atomicOr(err, kErrBadInput);
  return v >= 0 && v < (int64_t)V ? (int)v : -1;
}

// ----------------------------------------------- log probabilities of tokens --
struct LogprobsArgs {
  Logits z;
  Split split;
  const void* tokens;
  float* logprobs;
  float* stats;    // [T][2]: largest score, log s
  float* entropy;  // or null
  int32_t* top_indices;
  float* top_logprobs;
  u32* err;
  int64_t row0;
  u32 top;
  bool wide;  // 64-bit tokens
};

// The difference is taken of halves, with the same bits where it is no denormal: of
// scores at either end of the type it is no fp32 number, over the temperature it may be.
__device__ __forceinline__ float log_probability(const Logits& z, float x, const RowSums& r, float log_s) {
  return r.s == 0.0f ? -kInf : fmaf(0.5f, x, -0.5f * r.m) * (2.0f * z.inv) - log_s;
}

// One row's results from its sums, by any number of threads.
template <bool ENTROPY>
__device__ __forceinline__ void write_logprobs(const LogprobsArgs& a, int64_t row, int token, float score,
                                               const RowSums& r, const u64* keys) {
  const bool real = token >= 0;
  const float log_s = r.s == 0.0f ? 0.0f : logf(r.s);
  if (threadIdx.x == 0) {
    a.logprobs[row] = real ? log_probability(a.z, score, r, log_s) : 0.0f;
    a.stats[2 * row] = real ? r.m : 0.0f;
    a.stats[2 * row + 1] = real ? log_s : 0.0f;
    if constexpr (ENTROPY) {
      const float h = log_s - r.w / r.s * kLn2;  // roundings may leave less than nothing
      a.entropy[row] = !real || r.s == 0.0f || h < 0.0f ? 0.0f : h;
    }
  }
  for (u32 i = threadIdx.x; i < a.top; i += blockDim.x) {
    const u64 key = real ? keys[i] : 0;
    a.top_indices[row * a.top + i] = real ? (int32_t)key_index(key) : -1;
    a.top_logprobs[row * a.top + i] = real ? log_probability(a.z, key_score(key), r, log_s) : 0.0f;
  }
}

template <class T, int NT, bool ENTROPY, bool TOP, bool SPLIT>
__global__ __launch_bounds__(NT) void k_logprobs(LogprobsArgs a) {
  constexpr int E = kLogitsVector<T>;
  __shared__ float s_red[kJoinLds<NT>];
  __shared__ std::conditional_t<TOP, TopLds<NT>, int> s_top;
  const u32 slices = SPLIT ? a.split.slices : 1, slice = SPLIT ? blockIdx.x % slices : 0;
  const int64_t part = SPLIT ? blockIdx.x / slices : blockIdx.x, row = a.row0 + part;
  const T* z = (const T*)a.z.p + row * a.z.ld;
  const u32 c0 = SPLIT ? slice * a.split.length : 0, c1 = SPLIT ? min(c0 + a.split.length, a.z.V) : a.z.V;
  const Span span{c0, c1};
  float* parts = nullptr;
  if constexpr (TOP) parts = s_top.parts;
  const int64_t given = load_index(a.tokens, a.wide, row);
  // few rows: the pass does not wait for the token, and reads a masked place's row in vain
  const auto masked = [&] {
    if (given >= 0 && given < (int64_t)a.z.V) return false;
    if (given >= 0) atomicOr(a.err, kErrBadInput);
    if (slice == 0) write_logprobs<ENTROPY>(a, row, -1, 0.0f, RowSums{0.0f, 1.0f, 0.0f}, nullptr);
    return true;
  };
  if constexpr (!SPLIT) {
    if (masked()) return;
  }
  const Share h = row_pass<T, NT, ENTROPY, TOP>(z, span, a.z.c2, parts);
  if constexpr (SPLIT) {
    if (masked()) return;
  }
  const int token = (int)given;
  const float score = to_f32(z[token]);
  const u32 first = c0 + threadIdx.x * E, at = first + h.at * (NT * E);
  u64 bound = first < c1 ? entry_key(h.top, min(at + E, c1) - 1) : 0;
  if constexpr (TOP) {
    offer_bound(s_top, bound);
    if constexpr (NT == kWave) __syncthreads();  // else there is one in what comes next
  }
  RowSums r = join_shares<NT>(h, a.z.c2, s_red);
  const u64* keys = nullptr;
  if constexpr (TOP) {
    const u32 count = (c1 - c0 + NT * E - 1) / (NT * E), each = span.part<NT * E>();
    largest_keys<NT, true>(s_top, bound, count, each, a.top, r.s != r.s, [&](u32 owner, u32 j, auto&& f) {
      const u32 c = c0 + (owner + j * NT) * E;
      if (c >= c1) return;
      float x[E];
      if (c1 - c0 < (u32)E) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = c + e < c1 ? to_f32(z[c + e]) : 0.0f;
        f(x, c, 0u, c1 - c);
        return;
      }
      const u32 from = min(c, c1 - E);
      const Vec<T, E> v = load_vec<T, E>(z + from);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = to_f32(v.v[e]);
      f(x, from, c - from, (u32)E);
    });
    keys = s_top.out;
  }
  if constexpr (SPLIT) {
    __shared__ u32 s_last;
    __shared__ float s_sums[3];
    if (threadIdx.x == 0) store_slice(a.split, part, slice, r);
    if constexpr (TOP)
      for (u32 i = threadIdx.x; i < a.top; i += NT) st_agent64(a.split.keys + (part * slices + slice) * a.top + i, keys[i]);
    if (!last_of_row(a.split, part, &s_last)) return;
    r = join_slices(a.split, part, a.z.c2, s_sums);
    if constexpr (TOP) {
      // thread t holds the keys t, t + NT, .. of the slices'
      const u32 n = slices * a.top, count = (n + NT - 1) / NT;
      const u64* all = a.split.keys + part * n;
      constexpr int kHeld = kMostSlices * kMostTop / NT;
      u64 held[kHeld];
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const u32 i = threadIdx.x + j * NT;
        held[j] = i < n ? ld_agent64(all + i) : 0;
      }
      bound = 0;
#pragma unroll
      for (u64 key : held) bound = max(bound, key);
      offer_bound(s_top, bound);
      __syncthreads();
      largest_keys<NT, false>(s_top, bound, count, count, a.top, r.s != r.s, [&](u32 owner, u32 j, auto&& f) {
        const u32 i = owner + j * NT;
        const u64 key = i < n ? ld_agent64(all + i) : 0;
        const float x[1] = {key_score(key)};
        if (key != 0) f(x, key_index(key), 0u, 1u);
      });
    }
  }
  write_logprobs<ENTROPY>(a, row, token, score, r, keys);
}

// ------------------------------------------------------------ way back --
struct LogprobsGradArgs {
  Logits z;
  const void* tokens;
  const float* stats;
  const float* grad;          // of the log probabilities, or null
  const float* entropy;       // with grad_entropy
  const float* grad_entropy;  // or null
  void* out;
  int64_t ld_out;
  u32* err;
  int64_t row0;
  u32 slices, length;
  bool wide, streaming;
};

// Element x's p / tau times its coefficient: (b - a (log p + h)) p, with b and a
// times 1 / tau already; 0 where p is.
struct Coefficients {
  float m, log_s, l2;  // l2: log2 s
  float a, b, h;
};

// Whether every score of a row is -inf: no distribution, gradient 0.  A maximum
// passes NaN by, so a row of nothing else, or of NaN among -inf, has m = -inf too;
// its sum, and so log s, is NaN, and its gradient with them.
__device__ __forceinline__ bool no_scores(float m, float log_s) { return m == -kInf && log_s == log_s; }

template <bool ENTROPY>
__device__ __forceinline__ float slope(const Logits& z, const Coefficients& k, float x) {
  const float d = x - k.m;
  const float p = __builtin_amdgcn_exp2f(fmaf(d, z.c2, -k.l2));
  if constexpr (!ENTROPY) return p * k.b;
  const float lp = fmaxf(fmaf(d, z.inv, -k.log_s), -1024.0f);
  return p * fmaf(-k.a, lp + k.h, k.b);
}

// The first column from c0 on that begins a cache line of out.
template <class T>
constexpr u32 kLine = 128 / sizeof(T);
template <class T>
__device__ __forceinline__ u32 aligned_column(const T* out, u32 c0, u32 c1) {
  const u32 past = (u32)((uintptr_t)(out + c0) / sizeof(T) % kLine<T>);
  return min(c0 + (kLine<T> - past) % kLine<T>, c1);
}

// out = f(z) for columns [c0, c1), a vector's results passed through patch(y,
// its first column) on their way; out may be z.  A wave's vectors begin with a line:
// 4,096 rows of 50,001 in fp16 take 164 us, 181 where they begin with the row, 177
// where with 16 bytes.
// From the end to the start: a pass over the row that came before left its end in
// the caches.
template <class T, int NT, bool KEPT, class F, class P>
__device__ __forceinline__ void map_row(const T* z, T* out, u32 c0, u32 c1, bool streaming,
                                        const Vec<T, kLogitsVector<T>>* kept, F&& f, P&& patch) {
  constexpr int E = kLogitsVector<T>, U = 2;
  constexpr u32 kStep = NT * E;
  const u32 start = aligned_column(out, c0, c1);
  const auto one = [&](const Vec<T, E>& v, u32 at) {
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = f(to_f32(v.v[e]));
    patch(y, at);
    const Vec<T, E> r = round_vec<T, E>(y);
    if (streaming) store_vec_streaming<T, E>(out + at, r);
    else store_vec<T, E>(out + at, r);
  };
  // the elements before the first whole vector and behind the last, a thread each
  const u32 before = start - c0, behind = (c1 - start) % E;
  for (u32 i = threadIdx.x; i < before + behind; i += NT) {
    const u32 at = i < before ? c0 + i : c1 - behind + (i - before);
    float y[1] = {f(to_f32(z[at]))};
    patch(y, at);
    out[at] = round_vec<T, 1>(y).v[0];
  }
  // with KEPT (c0 = 0) the row's first vectors are at hand where out's lines begin with one of them
  const u32 held = KEPT && start % E == 0 ? kUnroll * kStep : 0;
  u32 rounds = (c1 - start) / (U * kStep), c = start + rounds * (U * kStep) + threadIdx.x * E;
  Vec<T, E> v[U];
  if (KEPT && c1 <= held) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * kStep + E <= c1) v[u] = kept[c / E + u * NT];
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * kStep + E <= c1) v[u] = load_vec<T, E>(z + c + u * kStep);
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c + u * kStep + E <= c1) one(v[u], c + u * kStep);
  for (; rounds > 0; --rounds) {
    c -= U * kStep;
    if (KEPT && start + rounds * (U * kStep) <= held) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = kept[c / E + u * NT];
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = load_vec<T, E>(z + c + u * kStep);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) one(v[u], c + u * kStep);
  }
}

template <class T, int NT>
__device__ __forceinline__ void zero_row(T* out, u32 c0, u32 c1, bool streaming) {
  constexpr int E = kLogitsVector<T>;
  const float zero[E] = {};
  const u32 start = aligned_column(out, c0, c1), before = start - c0, behind = (c1 - start) % E;
  for (u32 i = threadIdx.x; i < before + behind; i += NT)
    out[i < before ? c0 + i : c1 - behind + (i - before)] = from_f32<T>(0.0f);
  for (u32 c = start + threadIdx.x * E; c + E <= c1; c += NT * E) {
    if (streaming) store_vec_streaming<T, E>(out + c, round_vec<T, E>(zero));
    else store_vec<T, E>(out + c, round_vec<T, E>(zero));
  }
}

template <class T, int NT, bool ENTROPY>
__global__ __launch_bounds__(NT) void k_logprobs_grad(LogprobsGradArgs a) {
  const u32 slice = a.slices == 1 ? 0 : blockIdx.x % a.slices;
  const int64_t row = a.row0 + (a.slices == 1 ? blockIdx.x : blockIdx.x / a.slices);
  const u32 c0 = slice * a.length, c1 = min(c0 + a.length, a.z.V);
  T* out = (T*)a.out + row * a.ld_out;
  const int token = load_entry(a.tokens, a.wide, row, a.z.V, a.err);
  Coefficients k;
  k.m = a.stats[2 * row];
  k.log_s = a.stats[2 * row + 1];
  if (token < 0 || no_scores(k.m, k.log_s)) {  // masked, or no score above -inf
    zero_row<T, NT>(out, c0, c1, a.streaming);
    return;
  }
  k.l2 = k.log_s * kLog2e;
  const float g = a.grad ? a.grad[row] * a.z.inv : 0.0f;
  k.b = -g;
  k.a = ENTROPY ? a.grad_entropy[row] * a.z.inv : 0.0f;
  k.h = ENTROPY ? a.entropy[row] : 0.0f;
  map_row<T, NT, false>(
      (const T*)a.z.p + row * a.z.ld, out, c0, c1, a.streaming, nullptr, [&](float x) { return slope<ENTROPY>(a.z, k, x); },
      [&](auto& y, u32 at) {
        constexpr u32 N = sizeof(y) / sizeof(y[0]);
        if ((u32)token - at >= N) return;
#pragma unroll
        for (u32 e = 0; e < N; ++e) y[e] += at + e == (u32)token ? g : 0.0f;
      });
}

// ---------------------------------------------------------- distillation --
struct DistillArgs {
  Logits z;
  Split split;
  const void* indices;
  const void* teacher;
  float* loss;
  float* stats;        // or null
  const float* given;  // grad: upstream gradients; step: weights or null
  void* out;
  int64_t ld_out;
  u32* err;
  int64_t row0;
  u32 K;
  int teacher_dtype;
  bool wide, streaming;
};

constexpr int kMostSlots = 1024;

constexpr u32 kHeads = 1024;  // lists of slots, by the vector that an index falls into
constexpr u32 kNoSlot = ~0u;

// The list of a column, of a vector of map_row's by its first, whose whole vectors begin at `start`.
template <class T>
__device__ __forceinline__ u32 head_of(u32 column, u32 start) {
  return (column - start + kLine<T>) / kLogitsVector<T> % kHeads;
}

// The slots of a row in LDS, K of each.
struct Slots {
  float* q;    // probability
  int* index;  // -1: empty
  float* lq;   // for the loss: its log
  float* x;    // for the loss: the row's score there
  float* sum;  // for the gradient: q of all slots with this index, in the first of them
  u32* next;   // for the gradient: the next slot of a list
  u32* head;
  float (*red)[16];
};
template <bool LOSS, bool GRAD>
constexpr size_t slots_bytes(u32 K) {
  return (size_t)K * 4 * (2 + (LOSS ? 2 : 0) + (GRAD ? 2 : 0)) + (GRAD ? kHeads * 4 : 0);
}
template <bool LOSS, bool GRAD>
__device__ __forceinline__ Slots slots_in(float* lds, u32 K, float (*red)[16]) {
  Slots s{};
  s.q = lds;
  s.index = (int*)(lds + K);
  lds += 2 * K;
  if constexpr (LOSS) {
    s.lq = lds;
    s.x = lds + K;
    lds += 2 * K;
  }
  if constexpr (GRAD) {
    s.sum = lds;
    s.next = (u32*)(lds + K);
    s.head = (u32*)(lds + 2 * K);
  }
  s.red = red;
  return s;
}

// Reads a row's slots; for the gradient lists those in [c0, c1).  False where no
// slot has any probability.  Ends with a barrier.
template <class T, int NT, bool LOSS, bool GRAD>
__device__ __forceinline__ bool load_slots(const DistillArgs& a, int64_t row, const T* z, const T* out, u32 c0, u32 c1,
                                           const Slots& s) {
  const u32 start = GRAD ? aligned_column(out, c0, c1) : 0;
  float top[1] = {-kInf}, any[1] = {-kInf};
  if constexpr (GRAD) {
    for (u32 i = threadIdx.x; i < kHeads; i += NT) s.head[i] = kNoSlot;
  }
  for (u32 i = threadIdx.x; i < a.K; i += NT) {
    const int64_t at = row * a.K + i;
    const int index = load_entry(a.indices, a.wide, at, a.z.V, a.err);
    float t = -kInf;
    if (index >= 0) {
      t = a.teacher_dtype == TGS_FP32 ? ((const float*)a.teacher)[at]
          : a.teacher_dtype == TGS_BF16 ? to_f32(((const bf16_t*)a.teacher)[at]) : to_f32(((const fp16_t*)a.teacher)[at]);
      if constexpr (LOSS) s.x[i] = to_f32(z[index]);
    }
    s.index[i] = index;
    s.q[i] = t;
    top[0] = fmaxf(top[0], t);
    if (t != -kInf) any[0] = 1.0f;
  }
  group_reduce<Max, NT>(top, s.red[0]);
  group_reduce<Max, NT>(any, s.red[1]);
  if (any[0] < 0.0f) return false;
  if constexpr (GRAD && NT == kWave) __syncthreads();
  float sum[1] = {0.0f};
  for (u32 i = threadIdx.x; i < a.K; i += NT) {
    const int index = s.index[i];
    const float d = (s.q[i] - top[0]) * a.z.inv, e = index >= 0 ? __builtin_amdgcn_exp2f(d * kLog2e) : 0.0f;
    s.q[i] = e;
    if constexpr (LOSS) s.lq[i] = d;
    if constexpr (GRAD) {
      if (index >= 0 && (u32)index >= c0 && (u32)index < c1)
        s.next[i] = atomicExch(&s.head[head_of<T>((u32)index, start)], i);
    }
    sum[0] += e;
  }
  group_reduce<Sum, NT>(sum, s.red[2]);
  const float scale = 1.0f / sum[0], log_sum = logf(sum[0]);
  for (u32 i = threadIdx.x; i < a.K; i += NT) {
    s.q[i] *= scale;
    if constexpr (LOSS) s.lq[i] -= log_sum;
  }
  __syncthreads();
  if constexpr (GRAD) {
    // an index may stand in several slots: their q are added in the slots' order
    for (u32 i = threadIdx.x; i < a.K; i += NT) {
      const int index = s.index[i];
      if (index < 0 || (u32)index < c0 || (u32)index >= c1) continue;
      bool first = true, others = false;
      for (u32 o = s.head[head_of<T>((u32)index, start)]; o != kNoSlot; o = s.next[o]) {
        if (o == i || s.index[o] != index) continue;
        others = true;
        first = first && i < o;
      }
      float q = first ? s.q[i] : 0.0f;
      if (others && first)
        for (u32 o = i + 1; o < a.K; ++o)
          if (s.index[o] == index) q += s.q[o];
      s.sum[i] = q;
    }
    __syncthreads();
  }
  return true;
}

// The row's loss, in every thread's hands.
template <int NT>
__device__ __forceinline__ float slots_loss(const DistillArgs& a, const RowSums& r, float log_s, const Slots& s) {
  float sum[1] = {0.0f};
  for (u32 i = threadIdx.x; i < a.K; i += NT) {
    const float q = s.q[i];
    if (!(q == 0.0f)) sum[0] = fmaf(q, s.lq[i] - log_probability(a.z, s.x[i], r, log_s), sum[0]);
  }
  group_reduce<Sum, NT>(sum, s.red[3]);
  return sum[0];
}

// A teacher's NaN, which every q then is, goes to the whole row's gradient.
__device__ __forceinline__ Coefficients distill_coefficients(const DistillArgs& a, int64_t row, float m, float log_s,
                                                             const Slots& s) {
  const float g = a.given ? a.given[row] : 1.0f;
  return Coefficients{m, log_s, log_s * kLog2e, 0.0f, fmaf(0.0f, s.q[0], g * a.z.inv), 0.0f};
}

// Whether a row's gradient is 0 because its logits have no distribution; not where
// its teacher's q are NaN.
__device__ __forceinline__ bool no_gradient(float m, float log_s, const Slots& s) {
  return no_scores(m, log_s) && s.q[0] == s.q[0];
}

// out = (p - q) b for columns [c0, c1) of a row.
template <class T, int NT, bool KEPT>
__device__ __forceinline__ void write_distill_grad(const DistillArgs& a, const T* z, T* out, u32 c0, u32 c1,
                                                   const Coefficients& k, const Slots& s,
                                                   const Vec<T, kLogitsVector<T>>* kept) {
  const u32 start = aligned_column(out, c0, c1);
  map_row<T, NT, KEPT>(
      z, out, c0, c1, a.streaming, kept, [&](float x) { return slope<false>(a.z, k, x); },
      [&](auto& y, u32 at) {
        constexpr u32 N = sizeof(y) / sizeof(y[0]);
        for (u32 o = s.head[head_of<T>(at, start)]; o != kNoSlot; o = s.next[o]) {
          const u32 place = (u32)s.index[o] - at;
          const float q = s.sum[o] * k.b;
#pragma unroll
          for (u32 e = 0; e < N; ++e) y[e] -= e == place ? q : 0.0f;
        }
      });
}

__device__ __forceinline__ void write_loss(const DistillArgs& a, int64_t row, float loss, float m, float log_s) {
  if (threadIdx.x != 0) return;
  if (a.loss) a.loss[row] = loss;
  if (a.stats) {
    a.stats[2 * row] = m;
    a.stats[2 * row + 1] = log_s;
  }
}

// The losses; with GRAD the gradient of their weighted sum too, for which the
// row is read again: its first round of vectors, 16 to 64 KB, from LDS, the rest from
// beyond the L2 (8,192 rows of 32,000 in bf16 take 212 us, 243 without LDS; 4,096 of
// 128,000 441 and 492: their rows in flight outgrow the L2, which fetches 1.78 GB where
// the logits are 1.03, and memory and the last cache together give 6.4 TB/s).
template <class T, int NT, bool GRAD>
__global__ __launch_bounds__(NT) void k_distill(DistillArgs a) {
  constexpr bool KEEP = GRAD && NT >= kRowThreads;
  extern __shared__ float s_slots[];
  __shared__ float s_red[kJoinLds<NT>], s_more[4][16];
  __shared__ Vec<T, kLogitsVector<T>> s_kept[KEEP ? kUnroll * NT : 1];
  const Slots s = slots_in<true, GRAD>(s_slots, a.K, s_more);
  const int64_t row = a.row0 + blockIdx.x;
  const T* z = (const T*)a.z.p + row * a.z.ld;
  T* out = GRAD ? (T*)a.out + row * a.ld_out : nullptr;
  if (!load_slots<T, NT, true, GRAD>(a, row, z, out, 0, a.z.V, s)) {
    write_loss(a, row, 0.0f, 0.0f, 0.0f);
    if constexpr (GRAD) zero_row<T, NT>(out, 0, a.z.V, a.streaming);
    return;
  }
  const Share h = row_pass<T, NT, false, false, KEEP>(z, Span{0, a.z.V}, a.z.c2, nullptr, s_kept);
  const RowSums r = join_shares<NT>(h, a.z.c2, s_red);
  const float log_s = r.s == 0.0f ? 0.0f : logf(r.s);
  write_loss(a, row, slots_loss<NT>(a, r, log_s, s), r.m, log_s);
  if constexpr (GRAD) {
    if (no_gradient(r.m, log_s, s)) zero_row<T, NT>(out, 0, a.z.V, a.streaming);
    else write_distill_grad<T, NT, KEEP>(a, z, out, 0, a.z.V, distill_coefficients(a, row, r.m, log_s, s), s, s_kept);
  }
}

// The losses of rows in slices: the last workgroup of a row joins their sums.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_distill_split(DistillArgs a) {
  constexpr int NT = kRowThreads;
  extern __shared__ float s_slots[];
  __shared__ float s_red[kJoinLds<NT>], s_more[4][16];
  __shared__ u32 s_last;
  __shared__ float s_sums[3];
  const Slots s = slots_in<true, false>(s_slots, a.K, s_more);
  const u32 slices = a.split.slices, slice = blockIdx.x % slices;
  const int64_t part = blockIdx.x / slices, row = a.row0 + part;
  const T* z = (const T*)a.z.p + row * a.z.ld;
  const u32 c0 = slice * a.split.length, c1 = min(c0 + a.split.length, a.z.V);
  const Share h = row_pass<T, NT, false, false>(z, Span{c0, c1}, a.z.c2, nullptr);
  const RowSums own = join_shares<NT>(h, a.z.c2, s_red);
  if (threadIdx.x == 0) store_slice(a.split, part, slice, own);
  if (!last_of_row(a.split, part, &s_last)) return;
  if (!load_slots<T, NT, true, false>(a, row, z, nullptr, 0, a.z.V, s)) {
    write_loss(a, row, 0.0f, 0.0f, 0.0f);
    return;
  }
  const RowSums r = join_slices(a.split, part, a.z.c2, s_sums);
  const float log_s = r.s == 0.0f ? 0.0f : logf(r.s);
  write_loss(a, row, slots_loss<NT>(a, r, log_s, s), r.m, log_s);
}

template <class T, int NT>
__global__ __launch_bounds__(NT) void k_distill_grad(DistillArgs a) {
  extern __shared__ float s_slots[];
  __shared__ float s_more[4][16];
  const Slots s = slots_in<false, true>(s_slots, a.K, s_more);
  const u32 slices = a.split.slices, slice = slices == 1 ? 0 : blockIdx.x % slices;
  const int64_t row = a.row0 + (slices == 1 ? blockIdx.x : blockIdx.x / slices);
  const u32 c0 = slice * a.split.length, c1 = min(c0 + a.split.length, a.z.V);
  T* out = (T*)a.out + row * a.ld_out;
  const T* z = (const T*)a.z.p + row * a.z.ld;
  const float m = a.stats[2 * row], log_s = a.stats[2 * row + 1];
  if (!load_slots<T, NT, false, true>(a, row, z, out, c0, c1, s) || no_gradient(m, log_s, s))
    zero_row<T, NT>(out, c0, c1, a.streaming);
  else write_distill_grad<T, NT, false>(a, z, out, c0, c1, distill_coefficients(a, row, m, log_s, s), s, nullptr);
}

// ------------------------------------------------------------------ host --
struct RowPlan {
  u32 slices, length;
};

// Slices of a row for about `groups` workgroups in all, none shorter than one
// round of loads.
static RowPlan row_plan(int64_t T, int64_t V, u32 unit, int64_t groups, int64_t most, int64_t least = 1) {
  const int64_t want = std::max<int64_t>(1, std::min(most, groups / std::max<int64_t>(T, 1)));
  const int64_t per = std::max<int64_t>({(V + want - 1) / want, kUnroll * (int64_t)unit, least});
  const int64_t length = (per + unit - 1) / unit * unit;
  return RowPlan{(u32)((V + length - 1) / length), (u32)std::min<int64_t>(length, (int64_t)1 << 31)};
}

// Rows of up to 320 vectors of 16 bytes are one wave's.  16,384 rows by a wave and
// by a workgroup of four, in bf16: 1,500 log probabilities with 5 alternatives 33 and
// 52 us, their gradient 24 and 32; 2,500 36 and 58, 34 and 39; 4,000 48 and 63, but
// 54 and 49.  In fp32 1,500 scores take 19 and 23 us, 2,500 29 and 28.
static bool short_row(int64_t V, tgs_dtype t) { return V * (int64_t)dtype_bytes(t) <= 320 * 16; }
// The call that reads a row twice keeps fewer rows in flight where they are long, so
// that the second reading finds them in the caches.  In bf16, with 256, 512 and 1,024
// threads, before any of a row was kept in LDS, 8,192 rows of 32,000 take 267, 243 and
// 281 us, 4,096 of 128,000 606, 561 and 491.  With what is kept, 8,192 rows of 9,000
// take 77 us with 256 and 96 with 512, of 20,000 147 with 512 and 194 with 1,024, of
// 64,000 443 with 512 and 421 with 1,024; 2,048 of 50,001 in fp16 110 and 116.
static int step_threads(int64_t V, tgs_dtype t) {
  const int64_t bytes = V * (int64_t)dtype_bytes(t);
  return short_row(V, t) ? kWave : bytes < 32 << 10 ? kRowThreads : bytes < 112 << 10 ? 512 : 1024;
}

// Workgroups of a call whose rows go in slices.  Every slice, and every row's join,
// searches for its own alternatives: of 128,000 scores in bf16 with 20, for 1,024
// and 2,048 workgroups, 128 rows take 19 and 30 us, 256 25 and 32, 900 58 and 66;
// 400 of 50,001 in fp32 with the entropy alone 18.4 and 17.5.  Slices of two vectors
// a thread instead of four: 64 rows 30 and 20 us, one 16.4 and 15.9.
constexpr int64_t kPassGroups = 1024;
static_assert(kPassGroups / 2 <= (int64_t)(sizeof(HeaderHist::hist) / sizeof(u32)), "a counter for every row in slices");

static u32 row_unit(tgs_dtype t) { return kRowThreads * (u32)(16 / dtype_bytes(t)); }
static RowPlan pass_plan(int64_t T, int64_t V, tgs_dtype t) {
  return row_plan(T, V, row_unit(t), kPassGroups, kMostSlices);
}
// Gradients go in short slices, each of four vectors a thread: many workgroups that
// end and are followed by the next in memory reach what few long ones do not.  With
// 4,096, 16,384 and 32,768 workgroups 8,192 rows of 32,000 in bf16 take 207, 208 and
// 189 us, with 64 slots 212, 212 and 184, 2,048 of 128,000 210, 211 and 190; with
// slices of two vectors 198, 219 and 180.  Each slice reads the row's slots, so
// it is 16 times as long as the slots are many at least: with no such bound, 16, 64 and
// 256 times 2,048 rows of 128,000 with 1,024 slots take 269, 231, 224 and 254 us, with
// 512 200, 201, 218 and 230, 8,192 of 32,000 with 256 190, 190, 211 and 218, 512 of
// 128,000 with 512 54, 54, 52 and 70, 64 of them 12.9, 13.0, 15.5 and 52, 2,048 of
// 50,001 with 512 in bf16 99, 99, 97 and 95, in fp32 169, 165, 182 and 175.
static RowPlan grad_plan_of(int64_t T, int64_t V, tgs_dtype t, int64_t K) {
  return row_plan(T, V, row_unit(t), 32768, INT32_MAX, 16 * K);
}

static size_t sums_bytes(int64_t T, const RowPlan& p) {
  return p.slices == 1 ? 0 : round_up_256((size_t)T * p.slices * sizeof(SliceSums));
}
static size_t keys_bytes(int64_t T, const RowPlan& p, int32_t top) {
  return p.slices == 1 ? 0 : round_up_256((size_t)T * p.slices * (size_t)top * 8);
}

static bool row_sizes(int64_t T, int64_t V) { return T >= 0 && T <= INT32_MAX && V >= 1 && V <= INT32_MAX; }

// Rows of V elements every ld elements.
static size_t rows_bytes(int64_t T, int64_t V, int64_t ld, tgs_dtype t) {
  return T == 0 ? 0 : ((size_t)(T - 1) * (size_t)ld + (size_t)V) * dtype_bytes(t);
}

static tgs_status check_logits(const char* what, const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                               float temperature) {
  if (T < 0 || T > INT32_MAX) return fail(TGS_EINVAL, "%s: T=%lld outside [0, 2^31-1]", what, (long long)T);
  if (V < 1 || V > INT32_MAX) return fail(TGS_EINVAL, "%s: V=%lld outside [1, 2^31-1]", what, (long long)V);
  if (ld < V || ld > INT32_MAX) return fail(TGS_EINVAL, "%s: rows %lld elements apart, outside [V, 2^31-1]", what, (long long)ld);
  if (!is_float_dtype(dtype)) return fail(TGS_EINVAL, "%s: logits must be fp32, bf16 or fp16", what);
  if (!(temperature >= 1e-6f && temperature <= 1e6f)) return fail(TGS_EINVAL, "%s: temperature outside [1e-6, 1e6]", what);
  return check_rows_array(what, "logits", logits, dtype_bytes(dtype), T > 0);
}

struct Array {
  const char* name;
  const void* p;
  size_t bytes;
  size_t align;
  bool needed;
};

// Nulls, alignment, and outputs that overlap an input or one another.  `same`:
// the output that may be the logits (the first input) themselves.
template <int NI, int NO>
static tgs_status check_arrays(const char* what, const Array (&in)[NI], const Array (&out)[NO], bool same) {
  for (const Array& x : in)
    if (tgs_status st = check_rows_array(what, x.name, x.p, x.align, x.needed); st != TGS_OK) return st;
  for (const Array& x : out)
    if (tgs_status st = check_rows_array(what, x.name, x.p, x.align, x.needed); st != TGS_OK) return st;
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (!(same && o == 0 && i == 0) && overlaps(out[o].p, out[o].bytes, in[i].p, in[i].bytes))
        return fail(TGS_EINVAL, "%s: %s overlaps %s", what, out[o].name, in[i].name);
    for (int i = 0; i < o; ++i)
      if (overlaps(out[o].p, out[o].bytes, out[i].p, out[i].bytes))
        return fail(TGS_EINVAL, "%s: %s overlaps %s", what, out[o].name, out[i].name);
  }
  return TGS_OK;
}

static Logits logits_of(const void* p, int64_t ld, int64_t V, float temperature) {
  return Logits{p, ld, (u32)V, (float)(1.4426950408889634 / (double)temperature), (float)(1.0 / (double)temperature)};
}

// Launches over rows [row0, row0 + rows), as many as a launch takes.
template <class F>
static void over_rows(int64_t T, int64_t groups_a_row, int threads, F&& f) {
  const int64_t most = std::max<int64_t>(1, most_groups(threads) / groups_a_row);
  for (int64_t row0 = 0; row0 < T; row0 += most) f(row0, std::min(most, T - row0));
}

template <class F>
static void with_flag(bool b, F&& f) {
  if (b) f(std::true_type{});
  else f(std::false_type{});
}

}  // namespace tgs

using namespace tgs;

extern "C" size_t tgs_token_logprobs_workspace_bytes(int64_t T, int64_t V, tgs_dtype dtype, int32_t top) {
  if (!row_sizes(T, V) || !is_float_dtype(dtype) || top < 0 || top > kMostTop || top > V) return 0;
  const RowPlan p = pass_plan(T, V, dtype);
  return kWorkspaceHeader + sums_bytes(T, p) + keys_bytes(T, p, top);
}

extern "C" tgs_status tgs_token_logprobs(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                         const void* tokens, tgs_dtype tokens_dtype, float temperature,
                                         float* logprobs, float* stats, float* entropy, int32_t top,
                                         int32_t* top_indices, float* top_logprobs, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream) {
  const char* what = "token_logprobs";
  tgs_status st = check_logits(what, logits, dtype, T, V, ld, temperature);
  if (st != TGS_OK) return st;
  if (!is_token_dtype(tokens_dtype)) return fail(TGS_EINVAL, "%s: tokens must be int32 or int64", what);
  if (top < 0 || top > kMostTop || top > V)
    return fail(TGS_EINVAL, "%s: top=%d outside [0, min(%d, V)]", what, (int)top, kMostTop);
  const size_t need = tgs_token_logprobs_workspace_bytes(T, V, dtype, top);
  if ((st = check_rows_workspace(what, workspace, workspace_bytes, need)) != TGS_OK) return st;
  const size_t ts = dtype_bytes(tokens_dtype), n = (size_t)T * 4;
  const bool some = T > 0;
  const Array in[] = {{"logits", logits, rows_bytes(T, V, ld, dtype), dtype_bytes(dtype), some},
                      {"tokens", tokens, (size_t)T * ts, ts, some}};
  const Array out[] = {{"logprobs", logprobs, n, 4, some},
                       {"stats", stats, 2 * n, 4, some},
                       {"entropy", entropy, n, 4, false},
                       {"top_indices", top_indices, n * top, 4, some && top > 0},
                       {"top_logprobs", top_logprobs, n * top, 4, some && top > 0},
                       {"the workspace", workspace, workspace_bytes, 256, true}};
  if ((st = check_arrays(what, in, out, false)) != TGS_OK) return st;
  if (T == 0) return TGS_OK;
  const RowPlan p = pass_plan(T, V, dtype);
  char* scratch = (char*)workspace + kWorkspaceHeader;
  LogprobsArgs a{};
  a.z = logits_of(logits, ld, V, temperature);
  a.split = Split{p.slices, p.length, (SliceSums*)scratch, (u64*)(scratch + sums_bytes(T, p)), header_hist(workspace)->hist};
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.stats = stats;
  a.entropy = entropy;
  a.top_indices = top_indices;
  a.top_logprobs = top_logprobs;
  a.err = (u32*)workspace;
  a.top = (u32)top;
  a.wide = tokens_dtype == TGS_INT64;
  with_float_dtype(dtype, [&](auto* z) {
    using Z = std::remove_pointer_t<decltype(z)>;
    with_flag(entropy != nullptr, [&](auto ent) {
      with_flag(top > 0, [&](auto tops) {
        constexpr bool ENT = decltype(ent)::value, TOP = decltype(tops)::value;
        const bool wave = short_row(V, dtype);
        const int threads = wave ? kWave : kRowThreads;
        over_rows(T, p.slices, threads, [&](int64_t row0, int64_t rows) {
          a.row0 = row0;
          const dim3 grid((u32)(rows * p.slices));
          if (wave) hipLaunchKernelGGL((k_logprobs<Z, kWave, ENT, TOP, false>), grid, dim3(kWave), 0, stream, a);
          else if (p.slices == 1) hipLaunchKernelGGL((k_logprobs<Z, kRowThreads, ENT, TOP, false>), grid, dim3(kRowThreads), 0, stream, a);
          else hipLaunchKernelGGL((k_logprobs<Z, kRowThreads, ENT, TOP, true>), grid, dim3(kRowThreads), 0, stream, a);
        });
      });
    });
  });
  return launched(what);
}

extern "C" tgs_status tgs_token_logprobs_grad(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                              const void* tokens, tgs_dtype tokens_dtype, float temperature,
                                              const float* stats, const float* grad_logprobs, const float* entropy,
                                              const float* grad_entropy, void* out, int64_t ld_out, void* workspace,
                                              size_t workspace_bytes, hipStream_t stream) {
  const char* what = "token_logprobs_grad";
  tgs_status st = check_logits(what, logits, dtype, T, V, ld, temperature);
  if (st != TGS_OK) return st;
  if (!is_token_dtype(tokens_dtype)) return fail(TGS_EINVAL, "%s: tokens must be int32 or int64", what);
  if (ld_out < V || ld_out > INT32_MAX) return fail(TGS_EINVAL, "%s: rows of out %lld elements apart", what, (long long)ld_out);
  if (T > 0 && !grad_logprobs && !grad_entropy) return fail(TGS_EINVAL, "%s: no incoming gradient", what);
  if (T > 0 && grad_entropy && !entropy) return fail(TGS_EINVAL, "%s: null entropy", what);
  if ((st = check_rows_workspace(what, workspace, workspace_bytes, kWorkspaceHeader)) != TGS_OK) return st;
  const size_t ts = dtype_bytes(tokens_dtype), n = (size_t)T * 4;
  const bool some = T > 0, same = out == logits && ld_out == ld;
  const Array in[] = {{"logits", logits, rows_bytes(T, V, ld, dtype), dtype_bytes(dtype), some},
                      {"tokens", tokens, (size_t)T * ts, ts, some},
                      {"stats", stats, 2 * n, 4, some},
                      {"grad_logprobs", grad_logprobs, n, 4, false},
                      {"entropy", grad_entropy ? entropy : nullptr, n, 4, false},
                      {"grad_entropy", grad_entropy, n, 4, false}};
  const Array outs[] = {{"out", out, rows_bytes(T, V, ld_out, dtype), dtype_bytes(dtype), some},
                        {"the workspace", workspace, workspace_bytes, 256, true}};
  if ((st = check_arrays(what, in, outs, same)) != TGS_OK) return st;
  if (T == 0) return TGS_OK;
  const RowPlan p = grad_plan_of(T, V, dtype, 0);
  LogprobsGradArgs a{};
  a.z = logits_of(logits, ld, V, temperature);
  a.tokens = tokens;
  a.stats = stats;
  a.grad = grad_logprobs;
  a.entropy = entropy;
  a.grad_entropy = grad_entropy;
  a.out = out;
  a.ld_out = ld_out;
  a.err = (u32*)workspace;
  a.slices = p.slices;
  a.length = p.length;
  a.wide = tokens_dtype == TGS_INT64;
  a.streaming = (size_t)T * V * dtype_bytes(dtype) > kRowsStreamingBytes;
  with_float_dtype(dtype, [&](auto* z) {
    using Z = std::remove_pointer_t<decltype(z)>;
    with_flag(grad_entropy != nullptr, [&](auto ent) {
      constexpr bool ENT = decltype(ent)::value;
      const bool wave = short_row(V, dtype);
      const int threads = wave ? kWave : kRowThreads;
      over_rows(T, p.slices, threads, [&](int64_t row0, int64_t rows) {
        a.row0 = row0;
        const dim3 grid((u32)(rows * p.slices));
        if (wave) hipLaunchKernelGGL((k_logprobs_grad<Z, kWave, ENT>), grid, dim3(kWave), 0, stream, a);
        else hipLaunchKernelGGL((k_logprobs_grad<Z, kRowThreads, ENT>), grid, dim3(kRowThreads), 0, stream, a);
      });
    });
  });
  return launched(what);
}

// The three calls of the distillation: losses (out null), a gradient from the
// forward pass's sums (loss null), both.
static tgs_status distillation(const char* what, const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                               const void* indices, tgs_dtype indices_dtype, const void* teacher,
                               tgs_dtype teacher_dtype, int64_t K, float temperature, bool has_loss, float* loss,
                               bool has_grad, float* stats, const float* given, void* out, int64_t ld_out,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  tgs_status st = check_logits(what, logits, dtype, T, V, ld, temperature);
  if (st != TGS_OK) return st;
  if (!is_token_dtype(indices_dtype)) return fail(TGS_EINVAL, "%s: indices must be int32 or int64", what);
  if (!is_float_dtype(teacher_dtype)) return fail(TGS_EINVAL, "%s: teacher must be fp32, bf16 or fp16", what);
  if (K < 1 || K > kMostSlots) return fail(TGS_EINVAL, "%s: K=%lld outside [1, %d]", what, (long long)K, kMostSlots);
  if (has_grad && (ld_out < V || ld_out > INT32_MAX))
    return fail(TGS_EINVAL, "%s: rows of out %lld elements apart", what, (long long)ld_out);
  const RowPlan p = pass_plan(T, V, dtype), g = grad_plan_of(T, V, dtype, K);
  const size_t need = has_loss ? tgs_distillation_workspace_bytes(T, V, dtype) : kWorkspaceHeader;
  if ((st = check_rows_workspace(what, workspace, workspace_bytes, need)) != TGS_OK) return st;
  const size_t is = dtype_bytes(indices_dtype), es = dtype_bytes(teacher_dtype), n = (size_t)T * 4;
  const bool some = T > 0, same = has_grad && out == logits && ld_out == ld;
  const Array in[] = {{"logits", logits, rows_bytes(T, V, ld, dtype), dtype_bytes(dtype), some},
                      {"indices", indices, (size_t)T * K * is, is, some},
                      {"teacher", teacher, (size_t)T * K * es, es, some},
                      {has_loss ? "weights" : "grad_loss", given, n, 4, some && !has_loss},
                      {"stats", has_loss ? nullptr : stats, 2 * n, 4, some && !has_loss}};
  const Array outs[] = {{"out", has_grad ? out : nullptr, has_grad ? rows_bytes(T, V, ld_out, dtype) : 0, dtype_bytes(dtype),
                         some && has_grad},
                        {"loss", has_loss ? loss : nullptr, n, 4, some && has_loss},
                        {"stats", has_loss ? stats : nullptr, 2 * n, 4, false},
                        {"the workspace", workspace, workspace_bytes, 256, true}};
  if ((st = check_arrays(what, in, outs, same)) != TGS_OK) return st;
  if (T == 0) return TGS_OK;
  char* scratch = (char*)workspace + kWorkspaceHeader;
  DistillArgs a{};
  a.z = logits_of(logits, ld, V, temperature);
  a.indices = indices;
  a.teacher = teacher;
  a.loss = loss;
  a.stats = stats;
  a.given = given;
  a.out = out;
  a.ld_out = ld_out;
  a.err = (u32*)workspace;
  a.K = (u32)K;
  a.teacher_dtype = teacher_dtype;
  a.wide = indices_dtype == TGS_INT64;
  a.streaming = (size_t)T * V * dtype_bytes(dtype) > kRowsStreamingBytes;
  const size_t loss_lds = slots_bytes<true, false>(a.K), grad_lds = slots_bytes<false, true>(a.K),
               both_lds = slots_bytes<true, true>(a.K);
  const bool both = has_loss && has_grad, split = p.slices > 1;
  // split rows' gradients wait for the join
  if (both && split) a.stats = (float*)(scratch + sums_bytes(T, p));
  with_float_dtype(dtype, [&](auto* z) {
    using Z = std::remove_pointer_t<decltype(z)>;
    const bool wave = short_row(V, dtype);
    const int threads = wave ? kWave : kRowThreads;
    if (has_loss) {
      a.split = Split{p.slices, p.length, (SliceSums*)scratch, nullptr, header_hist(workspace)->hist};
      over_rows(T, p.slices, both ? 1024 : threads, [&](int64_t row0, int64_t rows) {
        a.row0 = row0;
        const dim3 grid((u32)(rows * p.slices));
        if (split) {
          hipLaunchKernelGGL((k_distill_split<Z>), grid, dim3(kRowThreads), loss_lds, stream, a);
          return;
        }
        with_flag(both, [&](auto grad) {
          constexpr bool GRAD = decltype(grad)::value;
          const size_t bytes = GRAD ? both_lds : loss_lds;
          const auto launch = [&](auto nt) {
            constexpr int NT = decltype(nt)::value;
            hipLaunchKernelGGL((k_distill<Z, NT, GRAD>), grid, dim3(NT), bytes, stream, a);
          };
          const int nt = GRAD ? step_threads(V, dtype) : threads;
          if (nt == kWave) launch(std::integral_constant<int, kWave>{});
          else if (nt == kRowThreads) launch(std::integral_constant<int, kRowThreads>{});
          else if constexpr (GRAD) {
            if (nt == 512) launch(std::integral_constant<int, 512>{});
            else launch(std::integral_constant<int, 1024>{});
          }
        });
      });
      if (!both || !split) return;
    }
    a.split = Split{g.slices, g.length, nullptr, nullptr, nullptr};
    over_rows(T, g.slices, threads, [&](int64_t row0, int64_t rows) {
      a.row0 = row0;
      const dim3 grid((u32)(rows * g.slices));
      if (wave) hipLaunchKernelGGL((k_distill_grad<Z, kWave>), grid, dim3(kWave), grad_lds, stream, a);
      else hipLaunchKernelGGL((k_distill_grad<Z, kRowThreads>), grid, dim3(kRowThreads), grad_lds, stream, a);
    });
  });
  return launched(what);
}

extern "C" size_t tgs_distillation_workspace_bytes(int64_t T, int64_t V, tgs_dtype dtype) {
  if (!row_sizes(T, V) || !is_float_dtype(dtype)) return 0;
  const RowPlan p = pass_plan(T, V, dtype);
  return kWorkspaceHeader + sums_bytes(T, p) + (p.slices == 1 ? 0 : round_up_256((size_t)T * 8));
}

extern "C" tgs_status tgs_distillation_loss(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                            const void* indices, tgs_dtype indices_dtype, const void* teacher,
                                            tgs_dtype teacher_dtype, int64_t K, float temperature, float* loss,
                                            float* stats, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return distillation("distillation_loss", logits, dtype, T, V, ld, indices, indices_dtype, teacher, teacher_dtype, K,
                      temperature, true, loss, false, stats, nullptr, nullptr, 0, workspace, workspace_bytes, stream);
}

extern "C" tgs_status tgs_distillation_grad(const void* logits, tgs_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                            const void* indices, tgs_dtype indices_dtype, const void* teacher,
                                            tgs_dtype teacher_dtype, int64_t K, float temperature, const float* stats,
                                            const float* grad_loss, void* out, int64_t ld_out, void* workspace,
                                            size_t workspace_bytes, hipStream_t stream) {
  return distillation("distillation_grad", logits, dtype, T, V, ld, indices, indices_dtype, teacher, teacher_dtype, K,
                      temperature, false, nullptr, true, (float*)stats, grad_loss, out, ld_out, workspace,
                      workspace_bytes, stream);
}

extern "C" tgs_status tgs_distillation_loss_and_grad(const void* logits, tgs_dtype dtype, int64_t T, int64_t V,
                                                     int64_t ld, const void* indices, tgs_dtype indices_dtype,
                                                     const void* teacher, tgs_dtype teacher_dtype, int64_t K,
                                                     float temperature, const float* weights, float* loss, void* out,
                                                     int64_t ld_out, void* workspace, size_t workspace_bytes,
                                                     hipStream_t stream) {
  return distillation("distillation_loss_and_grad", logits, dtype, T, V, ld, indices, indices_dtype, teacher,
                      teacher_dtype, K, temperature, true, loss, true, nullptr, weights, out, ld_out, workspace,
                      workspace_bytes, stream);
}
