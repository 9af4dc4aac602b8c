// Layer norm over the last axis and its gradients on gfx950.
//
//   mean = sum x / D,  var = sum (x - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   y = xh w + b with xh = (x - mean) rstd
//   dx = rstd (g w - sum(g w) / D - xh sum(g w xh) / D)
//   dw = sum over rows of g xh,  db = sum over rows of g
//
// Bound by HBM: 8 and 14 operations a value that is read and written once.  A
// row stays in the registers of the lanes that read it (8 lanes to 1,024,
// several vectors each), so that the mean is known before the squares are
// summed and no value is read twice.  Rows that registers do not hold are read
// again, from the caches.  131,072 rows of 2,048 in bf16: 185 us (5.8 TB/s, as a copy);
// 65,536 of 4,096 back, with weight and bias: 297 us (5.4).
#include <type_traits>

#include "tgs_rows.h"

namespace tgs {

struct NormArgs {
  const void* x;
  const void* weight;
  const void* bias;
  void* out;
  float* mean;
  float* rstd;
  int64_t T, row0;
  u32 D;
  int weight_dtype;
  float eps;
  bool streaming;
};

// Where the sum of squares passes fp32's range it is taken of values smaller by this.
constexpr float kShrink = 0x1p-80f;
// Where it falls below, down to where squares are lost or keep few bits, and eps does
// not outweigh it, it is taken of values larger by this.  The mean is small then too:
// values of 2^-20 and more are either equal or 2^-45 apart, with squares of 2^-90.
constexpr float kGrow = 0x1p100f, kFaint = 0x1p-96f, kFaintEps = 0x1p-100f, kFaintMean = 0x1p-20f;
__device__ __forceinline__ bool is_faint(float mean, float squares, float eps) {
  return squares < kFaint && eps < kFaintEps && fabsf(mean) < kFaintMean;
}
// A row's values lie flat where the squares of their distances to the mean sum up to
// no more than they would at a 256th of the mean each.  The roundings of the mean's own
// sum, up to about 20 (more in a long row), would stand out beside such distances: they
// are taken off by the mean of the distances, each of which is exact.
// Three passes more over what the registers hold: 65,536 rows of 1,024 in fp32 about
// 1,000 take 94 us instead of 92, rows of 0.1 alone in bf16 32,768 of 8,192 235 instead
// of 193, 131,072 of 2,048 213 instead of 186.
constexpr float kFlat = 0x1p-8f;
// The squares' sum that a row has to exceed, to be neither flat nor faint.
__device__ __forceinline__ float least_squares(float mean, float D, float eps) {
  const float m = mean * kFlat;
  return fmaxf(m * m * D, eps < kFaintEps ? kFaint : 0.0f);
}

// What a row is normed by: out = (x scale - mean) rstd.
struct Moments {
  float mean, rstd, scale;
};
// From the sum of the squares of x scale - mean.  Of a row of one value the
// variance is eps alone.
__device__ __forceinline__ Moments moments(float mean, float squares, float scale, float D, float eps) {
  if (squares == 0.0f) return Moments{mean / scale, 1.0f / sqrtf(eps), 1.0f};
  return Moments{mean, 1.0f / sqrtf(squares / D + eps * scale * scale), scale};
}

constexpr int norm_threads(int L) { return L > 256 ? L : 256; }

// How a row lies in L lanes of NV vectors of E <= D elements.  Vector i of a lane
// stands for columns c .. c + E - 1; past the row's end it is moved back to end
// with the row, so that it is one load without a branch, and its first `skip`
// elements are another vector's.  Those are computed and stored twice, with the
// same bits, and left out of the sums.
template <int E, int L>
struct Place {
  u32 D, t;
  __device__ __forceinline__ u32 column(int i) const { return (i * L + t) * E; }
  __device__ __forceinline__ bool inside(int i) const { return column(i) < D; }
  __device__ __forceinline__ u32 at(int i) const { return min(column(i), D - E); }
  // the same for the whole launch: no lane's vector i passes the row's end
  __device__ __forceinline__ bool whole(int i) const { return (u32)((i + 1) * L * E) <= D; }
  // calls f(e, counts) with counts = false where the element is another vector's
  template <class F>
  __device__ __forceinline__ void each(int i, F&& f) const {
    if (whole(i)) {
#pragma unroll
      for (int e = 0; e < E; ++e) f(e, true);
    } else {
      const u32 skip = column(i) - at(i);
#pragma unroll
      for (int e = 0; e < E; ++e) f(e, (u32)e >= skip);
    }
  }
};

// Has the compiler read values of narrow types out of their registers again,
// instead of holding each of them in 32 bits from one pass over them to the next.
template <class T, int E, int NV>
__device__ __forceinline__ void forget(Vec<T, E> (&v)[NV]) {
  if constexpr (sizeof(T) * E >= 8) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32 x[sizeof(T) * E / 4];
      __builtin_memcpy(x, &v[i], sizeof(x));
#pragma unroll
      for (u32& y : x) asm volatile("" : "+v"(y));
      __builtin_memcpy(&v[i], x, sizeof(x));
    }
  }
}

// A lane's parameters.
template <int E, int L, int NV>
__device__ __forceinline__ void lane_params(const Place<E, L>& at, const void* p, int dtype, float absent,
                                            float (&w)[NV][E]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) load_params<E>(p, dtype, at.at(i), at.D, absent, w[i]);
}

// A row in L lanes of NV vectors of E elements each; a workgroup takes every
// gridDim.x-th set of rows and keeps its columns' parameters in registers.  Of 16
// lanes a row the compiler is held to six waves a SIMD, where it would take two
// registers too many for them (200,000 rows of 100 in bf16 24.4 us with five waves,
// 21.7 with six).
template <class TX, class TY, int E, int L, int NV>
__global__ __launch_bounds__(norm_threads(L), L == 16 ? 6 : 1) void k_norm(NormArgs a) {
  constexpr int NT = norm_threads(L);
  __shared__ float s_red[4][L > kWave ? L / kWave : 1];
  const Place<E, L> at{a.D, threadIdx.x % L};
  const float D = (float)a.D;
  float w[NV][E], b[NV][E];
  lane_params<E, L, NV>(at, a.weight, a.weight_dtype, 1.0f, w);
  lane_params<E, L, NV>(at, a.bias, a.weight_dtype, 0.0f, b);
  for (int64_t set = blockIdx.x; set * (NT / L) < a.T; set += gridDim.x) {
    const int64_t row = set * (NT / L) + threadIdx.x / L;
    const bool real = row < a.T;
    const TX* x = (const TX*)a.x + (real ? row : 0) * (int64_t)a.D;
    Vec<TX, E> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at.inside(i)) raw[i] = load_vec<TX, E>(x + at.at(i));
    float scale = 1.0f, mean = 0.0f, sum[1], squares[1];
    // of x scale - mean
    const auto add_up = [&](float* lds) {
      sum[0] = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float part = 0.0f;
        at.each(i, [&](int e, bool counts) { part += counts ? fmaf(to_f32(raw[i].v[e]), scale, -mean) : 0.0f; });
        sum[0] += part;
      }
      group_reduce<Sum, L>(sum, lds);
    };
    const auto add_squares = [&] {
      squares[0] = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float part = 0.0f;
        at.each(i, [&](int e, bool counts) {
          const float d = counts ? fmaf(to_f32(raw[i].v[e]), scale, -mean) : 0.0f;
          part = fmaf(d, d, part);
        });
        squares[0] += part;
      }
      group_reduce<Sum, L>(squares, s_red[1]);
    };
    add_up(s_red[0]);
    mean = sum[0] / D;
    forget(raw);
    add_squares();
    float rstd = 1.0f / sqrtf(squares[0] / D + a.eps);
    if (__any(!(squares[0] > least_squares(mean, D, a.eps) && squares[0] < __builtin_huge_valf()))) {
      // the same for a whole workgroup where a row is one
      const bool far = !(squares[0] < __builtin_huge_valf()), faint = is_faint(mean, squares[0], a.eps);
      const bool again = far || faint || (mean != 0.0f && squares[0] <= least_squares(mean, D, a.eps));
      if (__any(again)) {
        const float before = mean;
        if (far) scale = kShrink;
        if (faint) scale = kGrow;
        mean = 0.0f;
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
          add_up(s_red[2 + turn]);
          mean += sum[0] / D;
        }
        add_squares();
        const Moments m = moments(mean, squares[0], scale, D, a.eps);
        mean = again ? m.mean : before;
        rstd = again ? m.rstd : rstd;
        scale = m.scale;
      }
    }
    forget(raw);
    if (real) {
      if (at.t == 0) {
        if (a.mean) a.mean[row] = mean / scale;
        if (a.rstd) a.rstd[row] = rstd * scale;
      }
      TY* out = (TY*)a.out + row * (int64_t)a.D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!at.inside(i)) continue;
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = fmaf(fmaf(to_f32(raw[i].v[e]), scale, -mean) * rstd, w[i][e], b[i][e]);
        const Vec<TY, E> r = round_vec<TY, E>(y);
        if (a.streaming) store_vec_streaming<TY, E>(out + at.at(i), r);
        else store_vec<TY, E>(out + at.at(i), r);
      }
    }
  }
}

// Calls f(e) for the elements of vector [c, c + E) that lie in the row.
template <int E, class F>
__device__ __forceinline__ void in_row(u32 c, u32 n, F&& f) {
  if (c + E <= n) {
#pragma unroll
    for (int e = 0; e < E; ++e) f(e);
  } else if (c < n) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c + e < n) f(e);
  }
}

constexpr int kLongThreads = 1024;

// Rows longer than registers hold: read three times, twice from the caches.  The
// distances to the first mean are summed beside their squares, since its sum takes
// up to D / 4,096 additions a thread.
// out may be x: a thread writes what it alone reads.
template <class TX, class TY, int E>
__global__ __launch_bounds__(kLongThreads) void k_norm_long(NormArgs a) {
  __shared__ float s_red[2][2 * (kLongThreads / kWave)];
  const int64_t row = a.row0 + blockIdx.x;
  const u32 n = a.D;
  const float D = (float)n;
  const TX* x = (const TX*)a.x + row * (int64_t)n;
  float scale = 1.0f, mean = 0.0f, sum[2];
  // of x scale - mean, and of its square
  const auto add_up = [&](float* lds) {
    sum[0] = sum[1] = 0.0f;
    for (u32 c = threadIdx.x * E; c < n; c += kLongThreads * E) {
      const Vec<TX, E> raw = load_part<TX, E>(x, c, n, from_f32<TX>(0.0f));
      float p0 = 0.0f, p1 = 0.0f;
      in_row<E>(c, n, [&](int e) {
        const float d = fmaf(to_f32(raw.v[e]), scale, -mean);
        p0 += d;
        p1 = fmaf(d, d, p1);
      });
      sum[0] += p0;
      sum[1] += p1;
    }
    group_reduce<Sum, kLongThreads>(sum, lds);
  };
  float first[1] = {0.0f};
  for (u32 c = threadIdx.x * E; c < n; c += kLongThreads * E) {
    const Vec<TX, E> raw = load_part<TX, E>(x, c, n, from_f32<TX>(0.0f));
    float part = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) part += to_f32(raw.v[e]);
    first[0] += part;
  }
  group_reduce<Sum, kLongThreads>(first, s_red[0]);
  mean = first[0] / D;
  add_up(s_red[1]);
  float off = sum[0] / D, squares = fmaf(-off * off, D, sum[1]);
  mean += off;
  const bool far = !(sum[1] < __builtin_huge_valf()), faint = is_faint(mean, sum[1], a.eps);
  // the same for the whole workgroup: little is left of the squares without the first mean's error
  if (far || faint || (off != 0.0f && !(squares > 0.5f * sum[1]))) {
    if (far || faint) {
      scale = far ? kShrink : kGrow;
      mean = 0.0f;
    }
    // a mean of other values takes two passes more
#pragma unroll 1
    for (int turn = far || faint ? 0 : 2; turn < 3; ++turn) {
      add_up(s_red[turn % 2]);
      if (turn < 2) mean += sum[0] / D;
    }
    squares = sum[1];
  }
  const Moments m = moments(mean, squares, scale, D, a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = m.mean / m.scale;
    if (a.rstd) a.rstd[row] = m.rstd * m.scale;
  }
  TY* out = (TY*)a.out + row * (int64_t)n;
  for (u32 c = threadIdx.x * E; c < n; c += kLongThreads * E) {
    const Vec<TX, E> raw = load_part<TX, E>(x, c, n, from_f32<TX>(0.0f));
    float w[E], b[E], y[E];
    load_params<E>(a.weight, a.weight_dtype, c, n, 1.0f, w);
    load_params<E>(a.bias, a.weight_dtype, c, n, 0.0f, b);
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = fmaf(fmaf(to_f32(raw.v[e]), m.scale, -m.mean) * m.rstd, w[e], b[e]);
    store_part<TY, E>(out, c, n, round_vec<TY, E>(y), a.streaming);
  }
}

// -------------------------------------------------------------- gradients --
struct NormGradArgs {
  const void* grad;
  const void* x;
  const float* mean;
  const float* rstd;
  const void* weight;
  void* out;
  float* part;  // [groups][2][D] sums of g xh and of g, null without parameters' gradients
  u32* arrived;  // not null: the last workgroup to arrive, counted here, adds the partial rows
  void* grad_weight;
  void* grad_bias;
  int param_dtype;
  int64_t T;
  u32 D;
  int weight_dtype;
  bool streaming;
};

// xh = (x - mean) rstd, of half the difference, which is an fp32 number where the
// whole one may be none.
struct Centre {
  float half_mean, twice_rstd;
  __device__ __forceinline__ Centre(float mean, float rstd) : half_mean(0.5f * mean), twice_rstd(2.0f * rstd) {}
  __device__ __forceinline__ float xh(float x) const { return fmaf(0.5f, x, -half_mean) * twice_rstd; }
};

// Column c of the sums: of weight's gradient, then of bias's.
__device__ __forceinline__ void store_column(void* weight, void* bias, int dtype, u32 D, u32 c, float sum) {
  if (c < D) {
    if (weight) store_param(weight, dtype, c, sum);
  } else if (bias) {
    store_param(bias, dtype, c - D, sum);
  }
}

// A workgroup takes every gridDim.x-th set of NT / L rows and keeps its
// columns' sums of g xh and of g in registers; its sums go to one partial row.
template <class TX, class TY, int E, int L, int NV>
__global__ __launch_bounds__(norm_threads(L)) void k_norm_grad(NormGradArgs a) {
  constexpr int NT = norm_threads(L);
  constexpr int kCols = L * NV * E;
  __shared__ float s_red[2][2 * (L > kWave ? L / kWave : 1)];
  __shared__ float s_cols[L < 256 ? 2 * kCols : 1];
  const Place<E, L> at{a.D, threadIdx.x % L};
  const u32 D = a.D;
  const float inv = 1.0f / (float)D;
  float w[NV][E], dw[NV][E], db[NV][E];
  lane_params<E, L, NV>(at, a.weight, a.weight_dtype, 1.0f, w);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = db[i][e] = 0.0f;
  int turn = 0;
  for (int64_t set = blockIdx.x; set * (NT / L) < a.T; set += gridDim.x, turn ^= 1) {
    const int64_t row = set * (NT / L) + threadIdx.x / L;
    const bool real = row < a.T;
    const int64_t base = (real ? row : 0) * (int64_t)D;
    const TX* x = (const TX*)a.x + base;
    const TY* g = (const TY*)a.grad + base;
    // before the row itself: behind it, the second of them waits for the row (65,536 of 4,096 337 us, not 296)
    const float rstd = a.rstd[real ? row : 0];
    const Centre centre(a.mean[real ? row : 0], rstd);
    Vec<TX, E> rx[NV];
    Vec<TY, E> rg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at.inside(i)) {
        rx[i] = load_vec<TX, E>(x + at.at(i));
        rg[i] = load_vec<TY, E>(g + at.at(i));
      }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float p0 = 0.0f, p1 = 0.0f;
      at.each(i, [&](int e, bool counts) {
        // a row past the last, or another vector's element, may be a NaN, and adds nothing all the same
        const bool on = L < NT ? counts && real : counts;
        const float xh = on ? centre.xh(to_f32(rx[i].v[e])) : 0.0f;
        const float gv = on ? to_f32(rg[i].v[e]) : 0.0f, gw = gv * w[i][e];
        p0 += gw;
        p1 = fmaf(gw, xh, p1);
        dw[i][e] = fmaf(gv, xh, dw[i][e]);
        db[i][e] += gv;
      });
      s[0] += p0;
      s[1] += p1;
    }
    group_reduce<Sum, L>(s, s_red[turn]);
    const float m0 = s[0] * inv, m1 = s[1] * inv;
    forget(rx);
    forget(rg);
    TX* out = (TX*)a.out + base;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!real || !at.inside(i)) continue;
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xh = centre.xh(to_f32(rx[i].v[e])), gw = to_f32(rg[i].v[e]) * w[i][e];
        y[e] = rstd * fmaf(-xh, m1, gw - m0);
      }
      const Vec<TX, E> r = round_vec<TX, E>(y);
      if (a.streaming) store_vec_streaming<TX, E>(out + at.at(i), r);
      else store_vec<TX, E>(out + at.at(i), r);
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * 2 * D;
  if constexpr (L >= 256) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const u32 c = at.at(i);
      at.each(i, [&](int e, bool counts) {
        if (!counts) return;
        part[c + e] = dw[i][e];
        part[(int64_t)D + c + e] = db[i][e];
      });
    }
  } else {
    // groups of a wave first, then the waves in turn
#pragma unroll
    for (int m = L; m < kWave; m *= 2) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          dw[i][e] += __shfl_xor(dw[i][e], m);
          db[i][e] += __shfl_xor(db[i][e], m);
        }
      }
    }
    for (int turn_of = 0; turn_of < NT / kWave; ++turn_of) {
      if (threadIdx.x / kWave == turn_of && lane_id() < L) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const u32 c = at.at(i);
          at.each(i, [&](int e, bool counts) {
            if (!counts) return;
            s_cols[c + e] = dw[i][e] + (turn_of ? s_cols[c + e] : 0.0f);
            s_cols[kCols + c + e] = db[i][e] + (turn_of ? s_cols[kCols + c + e] : 0.0f);
          });
        }
      }
      __syncthreads();
    }
    for (u32 c = threadIdx.x; c < D; c += NT) {
      if (a.arrived) {
        st_agent_f32(part + c, s_cols[c]);
        st_agent_f32(part + D + c, s_cols[kCols + c]);
      } else {
        part[c] = s_cols[c];
        part[(int64_t)D + c] = s_cols[kCols + c];
      }
    }
    if (!a.arrived) return;
    __shared__ u32 s_before;
    wait_all_memory();
    __syncthreads();
    if (threadIdx.x == 0) {
      s_before = add_agent_relaxed(a.arrived, 1u);
      if (s_before == gridDim.x - 1) st_agent(a.arrived, 0u);
    }
    __syncthreads();
    if (s_before != gridDim.x - 1) return;
    for (u32 c = threadIdx.x; c < 2 * D; c += NT) {
      float sum = 0.0f;
#pragma unroll 32
      for (u32 g = 0; g < gridDim.x; ++g) sum += __uint_as_float(ld_agent((const u32*)a.part + (size_t)g * 2 * D + c));
      store_column(a.grad_weight, a.grad_bias, a.param_dtype, D, c, sum);
    }
  }
}

// Rows longer than registers hold: x's gradient, each row read twice.
template <class TX, class TY, int E>
__global__ __launch_bounds__(kLongThreads) void k_norm_grad_long(NormGradArgs a, int64_t row0) {
  __shared__ float s_red[2 * (kLongThreads / kWave)];
  const int64_t row = row0 + blockIdx.x;
  const u32 D = a.D;
  const int64_t at = row * (int64_t)D;
  const TX* x = (const TX*)a.x + at;
  const TY* g = (const TY*)a.grad + at;
  const float rstd = a.rstd[row], inv = 1.0f / (float)D;
  const Centre centre(a.mean[row], rstd);
  float s[2] = {0.0f, 0.0f};
  for (u32 c = threadIdx.x * E; c < D; c += kLongThreads * E) {
    const Vec<TX, E> rx = load_part<TX, E>(x, c, D, from_f32<TX>(0.0f));
    const Vec<TY, E> rg = load_part<TY, E>(g, c, D, from_f32<TY>(0.0f));
    float w[E], p0 = 0.0f, p1 = 0.0f;
    load_params<E>(a.weight, a.weight_dtype, c, D, 1.0f, w);
    in_row<E>(c, D, [&](int e) {
      const float gw = to_f32(rg.v[e]) * w[e];
      p0 += gw;
      p1 = fmaf(gw, centre.xh(to_f32(rx.v[e])), p1);
    });
    s[0] += p0;
    s[1] += p1;
  }
  group_reduce<Sum, kLongThreads>(s, s_red);
  const float m0 = s[0] * inv, m1 = s[1] * inv;
  TX* out = (TX*)a.out + at;
  for (u32 c = threadIdx.x * E; c < D; c += kLongThreads * E) {
    const Vec<TX, E> rx = load_part<TX, E>(x, c, D, from_f32<TX>(0.0f));
    const Vec<TY, E> rg = load_part<TY, E>(g, c, D, from_f32<TY>(0.0f));
    float w[E], y[E];
    load_params<E>(a.weight, a.weight_dtype, c, D, 1.0f, w);
#pragma unroll
    for (int e = 0; e < E; ++e)
      y[e] = rstd * fmaf(-centre.xh(to_f32(rx.v[e])), m1, to_f32(rg.v[e]) * w[e] - m0);
    store_part<TX, E>(out, c, D, round_vec<TX, E>(y), a.streaming);
  }
}

// Such rows' sums by columns: a workgroup takes 256 columns of every
// gridDim.y-th row.  It runs before k_norm_grad_long, which may overwrite x or g.
template <class TX, class TY>
__global__ __launch_bounds__(256) void k_norm_columns(NormGradArgs a) {
  const u32 D = a.D, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= D) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
    const float xh = Centre(a.mean[row], a.rstd[row]).xh(to_f32(((const TX*)a.x)[row * D + c]));
    const float g = to_f32(((const TY*)a.grad)[row * D + c]);
    dw = fmaf(g, xh, dw);
    db += g;
  }
  float* part = a.part + (int64_t)blockIdx.y * 2 * D;
  part[c] = dw;
  part[(int64_t)D + c] = db;
}

// Adds the partial rows, each column's in a fixed order, and rounds the sums.
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void k_norm_join(const float* part, u32 groups, u32 D, void* weight,
                                                            void* bias, int dtype) {
  constexpr u32 W = kJoinThreads / kWave;
  __shared__ float s_sum[W][kWave];
  const int lane = lane_id();
  const u32 w = threadIdx.x / kWave;
  const int64_t width = 2 * (int64_t)D, c = (int64_t)blockIdx.x * kWave + lane;
  float sum = 0.0f;
  if (c < width) {
#pragma unroll 8
    for (u32 g = w; g < groups; g += W) sum += part[g * width + c];
  }
  s_sum[w][lane] = sum;
  __syncthreads();
  if (w == 0 && c < width) {
#pragma unroll
    for (u32 i = 1; i < W; ++i) sum += s_sum[i][lane];
    store_column(weight, bias, dtype, D, (u32)c, sum);
  }
}

// ------------------------------------------------------------------ host --
constexpr int64_t kMostD = (int64_t)1 << 24;  // exact in fp32, and no launch reaches 2^32 threads
// Vectors of a row that registers hold: on the way back they hold the columns' sums too.
constexpr int64_t kMostHeld = 4096;
template <int E>
constexpr int64_t kMostHeldBack = E == 4 ? 4096 : 2048;

// Elements of a vector, lanes of a row and vectors a lane for rows of D: the
// smallest that holds them.  Calls f(E, L, NV) as integral constants; false where
// none does.
template <int E, int64_t MOST, class F>
static bool with_shape(int64_t D, F&& f) {
  const int64_t vectors = (D + E - 1) / E;
  const auto call = [&](auto e, auto l, auto nv) { f(e, l, nv); };
  using std::integral_constant;
  constexpr integral_constant<int, E> e{};
  if (D < E) call(integral_constant<int, 1>{}, integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (vectors <= 8) call(e, integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (vectors <= 32) call(e, integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else if (vectors <= 64) call(e, integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (vectors <= 128) call(e, integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (vectors <= 256) call(e, integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (vectors <= 512) call(e, integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (vectors <= 1024) call(e, integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else if (vectors <= 2048) call(e, integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else if (vectors > MOST) return false;
  else if constexpr (MOST > 2048) call(e, integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  return true;
}

// Workgroups that add up the parameters' gradients, hence partial rows.  With one
// vector a lane, whose five workgroups a unit all reside, 1,280: 1,000,000 rows of
// 64 in bf16 take 134, 102, 83 and 112 us with 512, 768, 1,280 and 1,536, 262,144 of
// 512 273, 212, 168 and 218.  With more vectors 512: 131,072 of 2,048 309, 326 and 311
// with 512, 768 and 1,024, 65,536 of 4,096 304, 318 and 344, 65,536 of 1,024 79, 84
// and 86.  Of 1,024 threads 256: 16,384 rows of 16,384 480, 309 and 328 with 128, 256
// and 512.
//
// Each takes two sets of rows at least, whose partial rows few rows would outweigh:
// with one, two, four and eight 512 rows of 4,096 in bf16 take 21.1, 15.3, 14.8 and
// 19.6 us a call, 512 of 8,192 30, 22.5, 23.3 and 31, 2,048 of 2,048 21.1, 17.9, 20.5
// and 29.5.
//
// `one`: few rows of few columns, whose last workgroup adds the partial rows itself
// instead of a second launch: 13 us a call instead of 15.3 from 64 rows of 64 to 1,024
// of 256, the rule's edge, in fp32 and bf16.  Past it the gain ends: 4,096 rows of 256
// in fp32 take 14.0 and 15.3, 8,192 21.2 and 15.6, 2,048 of 512 15.4 and 15.5, 64 of
// 512 20.8 and 15.4.
template <int E>
static int64_t norm_groups(int64_t T, int64_t D, bool* one) {
  // rows that registers do not hold: 34 MB of partial rows at most, but one
  int64_t rows = 1, most = std::max<int64_t>(1, std::min<int64_t>(64, ((int64_t)1 << 22) / D));
  *one = false;
  with_shape<E, kMostHeldBack<E>>(D, [&](auto, auto l, auto nv) {
    constexpr int NT = norm_threads(decltype(l)::value);
    rows = NT / decltype(l)::value;
    *one = D <= 256 && (T + rows - 1) / rows <= 256;
    most = *one ? 64 : NT > 256 ? 256 : decltype(nv)::value == 1 ? 1280 : 512;
  });
  if (!*one) rows *= 2;
  return std::max<int64_t>(1, std::min(most, (T + rows - 1) / rows));
}

static tgs_status check_norm_sizes(const char* what, int64_t T, int64_t D) {
  if (T < 0 || T > INT32_MAX) return fail(TGS_EINVAL, "%s: T=%lld outside [0, 2^31-1]", what, (long long)T);
  if (D < 1 || D > kMostD) return fail(TGS_EINVAL, "%s: D=%lld outside [1, 2^24]", what, (long long)D);
  return TGS_OK;
}

template <class F>
static void with_two_types(tgs_dtype a, tgs_dtype b, F&& f) {
  with_float_dtype(a, [&](auto* x) { with_float_dtype(b, [&](auto* y) { f(x, y); }); });
}

}  // namespace tgs

using namespace tgs;

extern "C" tgs_status tgs_layer_norm(const void* x, tgs_dtype x_dtype, int64_t T, int64_t D, const void* weight,
                                     const void* bias, tgs_dtype weight_dtype, float eps, void* out,
                                     tgs_dtype out_dtype, float* mean, float* rstd, hipStream_t stream) {
  const char* what = "layer_norm";
  tgs_status st = check_norm_sizes(what, T, D);
  if (st != TGS_OK) return st;
  if (!is_float_dtype(x_dtype) || !is_float_dtype(out_dtype) || ((weight || bias) && !is_float_dtype(weight_dtype)))
    return fail(TGS_EINVAL, "%s: values must be fp32, bf16 or fp16", what);
  if (!(eps >= 0.0f) || !(eps - eps == 0.0f)) return fail(TGS_EINVAL, "%s: eps must be finite and >= 0", what);
  const size_t wa = dtype_bytes(weight || bias ? weight_dtype : TGS_FP32);
  if ((st = check_rows_array(what, "x", x, dtype_bytes(x_dtype), T > 0)) != TGS_OK ||
      (st = check_rows_array(what, "out", out, dtype_bytes(out_dtype), T > 0)) != TGS_OK ||
      (st = check_rows_array(what, "weight", weight, wa, false)) != TGS_OK ||
      (st = check_rows_array(what, "bias", bias, wa, false)) != TGS_OK ||
      (st = check_rows_array(what, "mean", mean, 4, false)) != TGS_OK ||
      (st = check_rows_array(what, "rstd", rstd, 4, false)) != TGS_OK)
    return st;
  const size_t nx = (size_t)T * D * dtype_bytes(x_dtype), no = (size_t)T * D * dtype_bytes(out_dtype);
  const size_t nw = (size_t)D * wa, ns = (size_t)T * 4;
  const bool in_place = x == out && x_dtype == out_dtype;
  if ((!in_place && overlaps(out, no, x, nx)) || overlaps(out, no, weight, nw) || overlaps(out, no, bias, nw))
    return fail(TGS_EINVAL, "%s: out overlaps an input", what);
  for (float* s : {mean, rstd})
    if (overlaps(s, ns, x, nx) || overlaps(s, ns, out, no) || overlaps(s, ns, weight, nw) || overlaps(s, ns, bias, nw))
      return fail(TGS_EINVAL, "%s: mean or rstd overlaps another array", what);
  if (overlaps(mean, ns, rstd, ns)) return fail(TGS_EINVAL, "%s: mean overlaps rstd", what);
  if (T == 0) return TGS_OK;
  NormArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.out = out;
  a.mean = mean;
  a.rstd = rstd;
  a.T = T;
  a.D = (u32)D;
  a.weight_dtype = weight_dtype;
  a.eps = eps;
  a.streaming = no > kRowsStreamingBytes;
  with_two_types(x_dtype, out_dtype, [&](auto* tx, auto* ty) {
    using TX = std::remove_pointer_t<decltype(tx)>;
    using TY = std::remove_pointer_t<decltype(ty)>;
    constexpr int E = sizeof(TX) == 2 && sizeof(TY) == 2 ? 8 : 4;
    const bool held = with_shape<E, kMostHeld>(D, [&](auto e, auto l, auto nv) {
      constexpr int L = decltype(l)::value, NT = norm_threads(L);
      // Workgroups at most.  Of several rows each 8,192 (131,072 rows of 2,048 in bf16 190 us; 193 with 4,096, 197
      // with 16,384).  Of one row, as many as reside: with two and four vectors a thread 1,024 and 768 (65,536 of
      // 4,096 225, 200 and 216 us with 768, 1,024 and 1,536; 32,768 of 8,192 193, 227 and 201 with 768, 1,024 and
      // 1,280), of 1,024 threads 512 and 256 (8,192 of 8,192, fp32 to bf16, 87, 77 and 76 us with 256, 512 and 1,024;
      // with four vectors 4,000 of 20,000 in bf16 122, 134 and 159, 8,192 of 32,768 286, 306 and 315, in fp32 8,192 of
      // 8,200 115, 116 and 117, of 12,288 146, 147 and 148, of 16,384 192, 188 and 186).
      constexpr int64_t kOneRow = decltype(nv)::value == 2 ? (L == 256 ? 1024 : 512) : (L == 256 ? 768 : 256);
      const int64_t sets = (T + NT / L - 1) / (NT / L), most = L <= kWave ? 8192 : kOneRow;
      hipLaunchKernelGGL((k_norm<TX, TY, decltype(e)::value, L, decltype(nv)::value>), dim3((u32)std::min(sets, most)),
                         dim3(NT), 0, stream, a);
    });
    if (!held) {
      const int64_t most = most_groups(kLongThreads);
      for (a.row0 = 0; a.row0 < T; a.row0 += most)
        hipLaunchKernelGGL((k_norm_long<TX, TY, E>), dim3((u32)std::min(most, T - a.row0)), dim3(kLongThreads), 0,
                           stream, a);
    }
  });
  return launched(what);
}

extern "C" size_t tgs_layer_norm_grad_workspace_bytes(int64_t T, int64_t D) {
  if (T < 0 || T > INT32_MAX || D < 1 || D > kMostD) return 0;
  // the types decide how many lanes a row takes: the most of either
  bool one;
  const int64_t groups = std::max(norm_groups<4>(T, D, &one), norm_groups<8>(T, D, &one));
  return kWorkspaceHeader + round_up_256((size_t)groups * 2 * (size_t)D * 4);
}

extern "C" tgs_status tgs_layer_norm_grad(const void* grad, tgs_dtype grad_dtype, const void* x, tgs_dtype x_dtype,
                                          int64_t T, int64_t D, const float* mean, const float* rstd,
                                          const void* weight, tgs_dtype weight_dtype, void* grad_x, void* grad_weight,
                                          void* grad_bias, tgs_dtype param_dtype, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream) {
  const char* what = "layer_norm_grad";
  tgs_status st = check_norm_sizes(what, T, D);
  if (st != TGS_OK) return st;
  const bool params = grad_weight || grad_bias;
  if (!is_float_dtype(x_dtype) || !is_float_dtype(grad_dtype) || (weight && !is_float_dtype(weight_dtype)) ||
      (params && !is_float_dtype(param_dtype)))
    return fail(TGS_EINVAL, "%s: values must be fp32, bf16 or fp16", what);
  const size_t pa = dtype_bytes(params ? param_dtype : TGS_FP32), wa = dtype_bytes(weight ? weight_dtype : TGS_FP32);
  if ((st = check_rows_array(what, "grad", grad, dtype_bytes(grad_dtype), T > 0)) != TGS_OK ||
      (st = check_rows_array(what, "x", x, dtype_bytes(x_dtype), T > 0)) != TGS_OK ||
      (st = check_rows_array(what, "mean", mean, 4, T > 0)) != TGS_OK ||
      (st = check_rows_array(what, "rstd", rstd, 4, T > 0)) != TGS_OK ||
      (st = check_rows_array(what, "weight", weight, wa, false)) != TGS_OK ||
      (st = check_rows_array(what, "grad_x", grad_x, dtype_bytes(x_dtype), T > 0)) != TGS_OK ||
      (st = check_rows_array(what, "grad_weight", grad_weight, pa, false)) != TGS_OK ||
      (st = check_rows_array(what, "grad_bias", grad_bias, pa, false)) != TGS_OK ||
      (st = check_rows_workspace(what, workspace, workspace_bytes, tgs_layer_norm_grad_workspace_bytes(T, D))) != TGS_OK)
    return st;
  struct Span {
    const void* p;
    size_t n;
  };
  const size_t nx = (size_t)T * D * dtype_bytes(x_dtype), ng = (size_t)T * D * dtype_bytes(grad_dtype);
  const Span in[] = {{grad, ng}, {x, nx}, {mean, (size_t)T * 4}, {rstd, (size_t)T * 4}, {weight, (size_t)D * wa}};
  const Span out[] = {{grad_x, nx}, {grad_weight, (size_t)D * pa}, {grad_bias, (size_t)D * pa}, {workspace, workspace_bytes}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i) {
      // x's gradient may take the place of x or of the incoming gradient
      if (o == 0 && (i == 1 || (i == 0 && grad_dtype == x_dtype)) && out[o].p == in[i].p) continue;
      if (overlaps(out[o].p, out[o].n, in[i].p, in[i].n)) return fail(TGS_EINVAL, "%s: an output overlaps an input", what);
    }
    for (int i = 0; i < o; ++i)
      if (overlaps(out[o].p, out[o].n, out[i].p, out[i].n)) return fail(TGS_EINVAL, "%s: outputs overlap", what);
  }
  if (T == 0 && !params) return TGS_OK;
  NormGradArgs a{};
  a.grad = grad;
  a.x = x;
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.out = grad_x;
  a.part = params ? (float*)((char*)workspace + kWorkspaceHeader) : nullptr;
  a.T = T;
  a.D = (u32)D;
  a.weight_dtype = weight_dtype;
  a.streaming = nx > kRowsStreamingBytes;
  a.grad_weight = grad_weight;
  a.grad_bias = grad_bias;
  a.param_dtype = param_dtype;
  int64_t groups = 0;
  bool one = false;
  if (T > 0)
    with_two_types(x_dtype, grad_dtype, [&](auto* tx, auto* ty) {
      using TX = std::remove_pointer_t<decltype(tx)>;
      using TY = std::remove_pointer_t<decltype(ty)>;
      constexpr int E = sizeof(TX) == 2 && sizeof(TY) == 2 ? 8 : 4;
      groups = norm_groups<E>(T, D, &one);
      a.arrived = one && params ? header_hist(workspace)->hist : nullptr;
      const bool held = with_shape<E, kMostHeldBack<E>>(D, [&](auto e, auto l, auto nv) {
        constexpr int L = decltype(l)::value;
        hipLaunchKernelGGL((k_norm_grad<TX, TY, decltype(e)::value, L, decltype(nv)::value>), dim3((u32)groups),
                           dim3(norm_threads(L)), 0, stream, a);
      });
      if (!held) {
        if (params)
          hipLaunchKernelGGL((k_norm_columns<TX, TY>), dim3((u32)((D + 255) / 256), (u32)groups), dim3(256), 0, stream, a);
        const int64_t most = most_groups(kLongThreads);
        for (int64_t row0 = 0; row0 < T; row0 += most)
          hipLaunchKernelGGL((k_norm_grad_long<TX, TY, E>), dim3((u32)std::min(most, T - row0)), dim3(kLongThreads), 0,
                             stream, a, row0);
      }
    });
  if (params && !one)
    hipLaunchKernelGGL(k_norm_join, dim3((u32)((2 * D + kWave - 1) / kWave)), dim3(kJoinThreads), 0, stream, a.part,
                       (u32)groups, (u32)D, grad_weight, grad_bias, param_dtype);
  return launched(what);
}
