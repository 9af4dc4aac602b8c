// Newton-Schulz products of matrices that one workgroup holds in LDS (the
// formulas, and what is rounded, as in orthogonal.hip): a shorter side of 65 to
// 128, and a longer one of up to 384 for bf16 results, 128 for fp32 and fp16.
//
// Such a matrix has 17 launches' worth of steps and little to compute in each:
// one launch does it all, the norm and the momentum included.  X lies in LDS
// column by column (fp16; high and low parts for fp32 and fp16 results) and, in fp32, in
// registers in the layout that the matrix instructions leave: the wave that
// makes a block of the update owns it throughout.  The update reads X as it lies,
// the gram by transposing reads.  Eight waves take the products' blocks of 32 x 32;
// the symmetric products are made whole, so that every wave has the same share.
// 25.7 us at 128 x 128 in bf16, 3.3 of them a step, where launch by launch takes
// 75; 69 against 81 at 128 x 384 and 126 against 290 for 256 of them.  Bound by
// the latency from one phase to the next: the matrix cores are busy a third of it.
#include <type_traits>

#include "tgs_orthogonal.h"

namespace tgs {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kLdsWaves = 8;

struct LdsArgs {
  const void* x;
  float* momentum;
  void* out;
  int64_t count;  // rows * cols
  int rows, cols, tall, nesterov, steps;
  float beta, keep, gain, ca, cb, cc;
  double eps;
};

__device__ __forceinline__ f16v mfma32(h8 a, h8 b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

// Calls f(index, address) for the four values of rows r0..r0 + 3 of X's column
// c that lie inside the matrix.
template <class T, class F>
__device__ __forceinline__ void each4(const LdsArgs& a, T* base, int r0, int c, F&& f) {
  if (a.tall) {  // a row of x holds a column of X
    if (c >= a.rows) return;
    T* p = base + (int64_t)c * a.cols + r0;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r0 + r < a.cols) f(r, p + r);
  } else {
    if (c >= a.cols) return;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r0 + r < a.rows) f(r, base + (int64_t)(r0 + r) * a.cols + c);
  }
}

// Matrices lie in LDS in lines of 128 (a column of X, a row of E or P) of 16
// chunks of 16 bytes; a line's chunks are turned by its index so that neither 16
// lanes that read one chunk of 16 lines nor 32 lanes that transpose 4 lines x 32
// values meet in a bank (padded lines: 90 us for 17 steps of 128 x 128, these: 78).
__device__ __forceinline__ int turn(int line) { return (line & 3) << 2 | (line >> 2 & 1) << 1 | (line >> 3 & 1); }

// 1 / x of a power of two.
__device__ __forceinline__ float inverse(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }

// 4 x NB blocks of 32 x 32 hold the matrix; a wave makes them in pairs, one
// below the other, that share their right operand.
template <int NB, bool SPLIT, class TX, class TW, bool MUON>
__global__ __launch_bounds__(kLdsWaves* kWave, 2) void k_ns_lds(LdsArgs a, StepScales sc) {
  constexpr int MP = 128, NP = 32 * NB, PARTS = SPLIT ? 2 : 1;
  constexpr int UP = 2 * NB / kLdsWaves;  // pairs of X a wave owns
  static_assert(kLdsWaves == 8 && 2 * NB % kLdsWaves == 0, "a pair of E and P a wave");
  // P has its own square where LDS holds three, else it replaces E
  constexpr bool APART = PARTS * MP * 2 * (NP + 2 * MP) <= 150 * 1024;
  __shared__ __align__(16) _Float16 s_x[PARTS][NP * MP], s_e[PARTS][MP * MP], s_p[APART ? PARTS : 1][APART ? MP * MP : 8];
  __shared__ __align__(16) float s_d[MP], s_dp[MP];
  __shared__ double s_sum[kLdsWaves];
  _Float16* ph = APART ? s_p[0] : s_e[0];
  _Float16* pl = APART ? s_p[APART ? PARTS - 1 : 0] : s_e[PARTS - 1];
  const int lane = lane_id(), h = lane >> 5, c32 = lane & 31;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t base = (int64_t)blockIdx.x * a.count;
  const TX* x = (const TX*)a.x + base;
  float* mom = MUON ? a.momentum + base : nullptr;
  TW* out = (TW*)a.out + base;

  // pair u: rows row_of(u).. + 63 of columns col_of(u).. + 31; lane (h, c32) holds
  // rows 8 g + 4 h + r of column c32 of a block at 4 g + r
  auto row_of = [&](int u) { return (u * kLdsWaves + w) / NB * 64; };
  auto col_of = [&](int u) { return (u * kLdsWaves + w) % NB * 32; };
  f16v xf[UP][2];
  double sum = 0.0;
#pragma unroll
  for (int u = 0; u < UP; ++u)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f16v& v = xf[u][b];
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = 0.0f;
      const int r0 = row_of(u) + 32 * b + 4 * h, c = col_of(u) + c32;
#pragma unroll
      for (int g = 0; g < 4; ++g) each4(a, x, r0 + 8 * g, c, [&](int r, const TX* p) { v[4 * g + r] = to_f32(*p); });
      if (MUON) {
        f16v m;
#pragma unroll
        for (int g = 0; g < 4; ++g) each4(a, mom, r0 + 8 * g, c, [&](int r, float* p) { m[4 * g + r] = *p; });
#pragma unroll
        for (int g = 0; g < 4; ++g)
          each4(a, mom, r0 + 8 * g, c, [&](int r, float* p) {
            const float gr = v[4 * g + r], mn = new_momentum(a.beta, m[4 * g + r], gr);
            *p = mn;
            v[4 * g + r] = muon_u(a.nesterov, a.beta, gr, mn);
          });
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) sum = fma((double)v[q], (double)v[q], sum);
    }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) s_sum[w] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < kLdsWaves; ++i) sum += s_sum[i];
  const double inv = 1.0 / (sqrt(sum) + a.eps);

  // Places in lines, all of them a lane's constant with the block's and the
  // index's part turned in or added.
  const int own_line = c32 * 128 + turn(c32) * 8;
  // A block, in fp16, to lines (columns) of LDS.
  auto put = [&](_Float16* hp, _Float16* lp, int col, int row, const f16v& v) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      h4 p, l;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        _Float16 x1, x2;
        split_half(v[4 * g + r], x1, x2);
        p[r] = x1;
        l[r] = x2;
      }
      const int at = col * 128 + (own_line ^ (row + 8 * g)) + 4 * h;
      *(h4*)(hp + at) = p;
      if (SPLIT) *(h4*)(lp + at) = l;
    }
  };
#pragma unroll
  for (int u = 0; u < UP; ++u)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int q = 0; q < 16; ++q) xf[u][b][q] = (float)((double)xf[u][b][q] * inv) * sc.x[0];
      put(s_x[0], s_x[PARTS - 1], col_of(u), row_of(u) + 32 * b, xf[u][b]);
    }
  __syncthreads();

  // Operands of 16 summation indices from k on: 32 rows `row` of a matrix that
  // lies row by row, or 32 columns of one that lies column by column (16 lanes
  // transpose 4 indices x 16 rows twice).
  auto as_rows = [&](const _Float16* p, int row, int k) { return *(const h8*)(p + row * 128 + ((own_line ^ 8 * h) ^ k)); };
  const int line0 = 8 * h + lane % 16 / 4, at0 = c32 / 16 * 16 + lane % 4 * 4;  // k, a multiple of 16, leaves the turn
  const int first = line0 * 128 + (at0 ^ turn(line0) * 8), second = (line0 + 4) * 128 + (at0 ^ turn(line0 + 4) * 8);
  auto as_columns = [&](const _Float16* p, int row, int k) {
    return columns8(p + k * 128 + (first ^ row), p + k * 128 + (second ^ row));
  };
  // Both blocks of a pair, 16 summation indices.
  auto multiply = [&](f16v(&acc)[2], auto&& left, auto&& right) {
    const h8 rh = right(0), l0 = left(0, 0), l1 = left(0, 1);
    if (SPLIT) {
      const h8 rl = right(1);
      acc[0] = mfma32(left(1, 0), rh, mfma32(l0, rl, acc[0]));
      acc[1] = mfma32(left(1, 1), rh, mfma32(l1, rl, acc[1]));
    }
    acc[0] = mfma32(l0, rh, acc[0]);
    acc[1] = mfma32(l1, rh, acc[1]);
  };
  const f16v zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
  const int I = w / 4 * 64, J = w % 4 * 32;  // this wave's pair of E and P
  for (int s = 0; s < a.steps; ++s) {
    // all scales are powers of two
    const float sx = sc.x[s], sa = sc.a[s], sp = sc.p[s], next = sc.x[s + 1];
    // ---- gram: E and D
    {
      f16v acc[2] = {zero, zero};
#pragma unroll 8
      for (int k = 0; k < NP; k += 16)
        multiply(acc, [&](int p, int b) { return as_columns(s_x[p ? PARTS - 1 : 0], I + 32 * b, k); },
                 [&](int p) { return as_columns(s_x[p ? PARTS - 1 : 0], J, k); });
      const float to_a = inverse(sx) * inverse(sx), to_e = to_a * sa;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (I + 32 * b == J) {
          float d = 0.0f;
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const bool here = 8 * (q / 4) + 4 * h + q % 4 == c32;
            d = here ? acc[b][q] : d;
            acc[b][q] = here ? 0.0f : acc[b][q];
          }
          if (c32 / 4 % 2 == h) s_d[J + c32] = d * to_a;
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[b][q] *= to_e;
        put(s_e[0], s_e[PARTS - 1], J, I + 32 * b, acc[b]);
      }
    }
    __syncthreads();
    // ---- square: P from E and D;  P = c E^2 + (c (d_i + d_j) + b) E off the diagonal
    {
      f16v acc[2] = {zero, zero};
#pragma unroll
      for (int k = 0; k < MP; k += 16)
        multiply(acc, [&](int p, int b) { return as_rows(s_e[p ? PARTS - 1 : 0], I + 32 * b, k); },
                 [&](int p) { return as_rows(s_e[p ? PARTS - 1 : 0], J, k); });
      const float from_a = inverse(sa), to_sq = from_a * from_a, dj = s_d[J + c32];
      const float kc = a.cc * to_sq * sp, kd = a.cc * (sp * from_a), kj = fmaf(a.cc, dj, a.cb) * (sp * from_a);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (I + 32 * b == J) {
          float d = 0.0f;
#pragma unroll
          for (int q = 0; q < 16; ++q) d = 8 * (q / 4) + 4 * h + q % 4 == c32 ? acc[b][q] : d;
          // what multiplies X of this scale, to give it in the next one
          if (c32 / 4 % 2 == h) s_dp[J + c32] = (a.ca + fmaf(a.cc, fmaf(dj, dj, d * to_sq), a.cb * dj)) * (next * inverse(sx));
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int row = I + 32 * b + 8 * g + 4 * h, at = J * 128 + (own_line ^ (I + 32 * b + 8 * g)) + 4 * h;
          const h4 eh = *(const h4*)(s_e[0] + at), el = *(const h4*)(s_e[PARTS - 1] + at);
          const f4 di = *(const f4*)(s_d + row);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float e = (float)eh[r] + (SPLIT ? (float)el[r] : 0.0f);
            acc[b][4 * g + r] = fmaf(fmaf(kd, di[r], kj), e, acc[b][4 * g + r] * kc);
          }
        }
        if (I + 32 * b == J) {
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[b][q] = 8 * (q / 4) + 4 * h + q % 4 == c32 ? 0.0f : acc[b][q];
        }
      }
      if (!APART) __syncthreads();  // every wave has read E
#pragma unroll
      for (int b = 0; b < 2; ++b) put(ph, pl, J, I + 32 * b, acc[b]);
    }
    __syncthreads();
    // ---- update: X <- (a + D_P) X + E_P X
    const float to_next = next * inverse(sp) * inverse(sx);
#pragma unroll
    for (int u = 0; u < UP; ++u) {
      const int row = row_of(u), col = col_of(u);
      f16v acc[2] = {zero, zero};
#pragma unroll
      for (int k = 0; k < MP; k += 16)
        multiply(acc, [&](int p, int b) { return as_rows(p ? pl : ph, row + 32 * b, k); },
                 [&](int p) { return as_rows(s_x[p ? PARTS - 1 : 0], col, k); });
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f4 d = *(const f4*)(s_dp + row + 32 * b + 8 * g + 4 * h);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            xf[u][b][4 * g + r] = fmaf(d[r], xf[u][b][4 * g + r], acc[b][4 * g + r] * to_next);
        }
    }
    if (s + 1 == a.steps) break;
    __syncthreads();  // every wave has read X
#pragma unroll
    for (int u = 0; u < UP; ++u)
#pragma unroll
      for (int b = 0; b < 2; ++b) put(s_x[0], s_x[PARTS - 1], col_of(u), row_of(u) + 32 * b, xf[u][b]);
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < UP; ++u)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int r0 = row_of(u) + 32 * b + 4 * h, c = col_of(u) + c32;
      f16v old;
      if (MUON) {
#pragma unroll
        for (int g = 0; g < 4; ++g) each4(a, out, r0 + 8 * g, c, [&](int r, TW* p) { old[4 * g + r] = to_f32(*p); });
      }
#pragma unroll
      for (int g = 0; g < 4; ++g)
        each4(a, out, r0 + 8 * g, c, [&](int r, TW* p) {
          const float v = xf[u][b][4 * g + r];
          *p = from_f32<TW>(MUON ? fmaf(a.keep, old[4 * g + r], a.gain * v) : v);
        });
    }
}

// ------------------------------------------------------------------ host --
bool lds_holds(int64_t rows, int64_t cols, bool split) {
  const int64_t m = std::min(rows, cols), n = std::max(rows, cols);
  return m > kSmallSide && m <= 128 && n <= (split ? 128 : 384);
}

template <bool SPLIT, class TX, class TW, bool MUON>
static void launch_lds(const LdsArgs& a, const StepScales& s, int batch, hipStream_t stream) {
  const int n = std::max(a.rows, a.cols);
  const dim3 grid(batch), block(kLdsWaves * kWave);
  if (SPLIT || n <= 128) {
    hipLaunchKernelGGL((k_ns_lds<4, SPLIT, TX, TW, MUON>), grid, block, 0, stream, a, s);
  } else if constexpr (!SPLIT) {
    if (n <= 256) hipLaunchKernelGGL((k_ns_lds<8, SPLIT, TX, TW, MUON>), grid, block, 0, stream, a, s);
    else hipLaunchKernelGGL((k_ns_lds<12, SPLIT, TX, TW, MUON>), grid, block, 0, stream, a, s);
  }
}

void lds_run(const NsCall& q, const StepScales& s, hipStream_t stream) {
  LdsArgs a{};
  a.x = q.x;
  a.momentum = q.momentum;
  a.out = q.out;
  a.count = q.rows * q.cols;
  a.rows = (int)q.rows;
  a.cols = (int)q.cols;
  a.tall = q.rows > q.cols;
  a.nesterov = q.nesterov;
  a.steps = q.steps;
  a.beta = q.beta;
  a.keep = q.keep;
  a.gain = q.gain;
  a.ca = (float)q.a;
  a.cb = (float)q.b;
  a.cc = (float)q.c;
  a.eps = q.eps;
  with_float_dtype(q.out_dtype, [&](auto* o) {
    using TW = std::remove_pointer_t<decltype(o)>;
    constexpr bool SPLIT = kSplitProducts<TW>;
    if (q.momentum)
      with_float_dtype(q.x_dtype, [&](auto* x) {
        launch_lds<SPLIT, std::remove_pointer_t<decltype(x)>, TW, true>(a, s, (int)q.batch, stream);
      });
    else
      launch_lds<SPLIT, TW, TW, false>(a, s, (int)q.batch, stream);
  });
}

}  // namespace tgs
