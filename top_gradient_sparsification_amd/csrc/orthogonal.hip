// Newton-Schulz orthogonalisation and the Muon step on gfx950.
//
//   X <- G / (|G|_F + eps), then `steps` times
//   A = X X^T,  P = b A + c A^2,  X <- a X + P X
// with X the m x n matrix whose rows are the shorter side (m <= n; a tall G is
// transposed on the way in and out).
//
// Three products a step, all of the form C = L R^T with both operands'
// summation index contiguous, on the fp16 matrix instructions with fp32
// accumulators (k_ns_product):
//   gram     A = X X^T          operands X, X      symmetric: lower tiles only
//   square   A^2 = A A^T        operands A, A      symmetric: lower tiles only
//   update   P X = P (X^T)^T    operands P, X^T
// X is kept in both orders; the update's epilogue writes both.
//
// What is rounded.  The diagonals of A and P are large against the rest near
// the end (A tends to the identity), so they are held apart in fp32 and the
// products see only the off-diagonal part E of A and of P:
//   A = D + E:   A^2 = D^2 + (d_i + d_j) E + E^2,   P X = D_P X + E_P X.
// X itself is held as fp16 high + low part (22 bits) and a + D_P multiplies
// both.  With results of 16 bits the products read the high parts only: the
// result is then 2e-4 to 7e-4 (2-norm) off, below the 1.7e-3 of the final
// rounding, where rounding X, A and P whole gives 1.6e-3 to 3e-3 (fp16) and
// 1.3e-2 to 2.4e-2 (bf16).  With fp32 results every operand is high + low and
// a product is three (high low + low high + high high): as exact as fp32
// products (1.4e-6 to 2.3e-6 against 1.3e-6 to 2.0e-6).
//
// Range.  The singular values of X start in [0, 1]; the host bounds them after
// every step by the polynomial's extrema, and scales X, A and P by powers of
// two so that no entry passes 2^14 and small entries keep their low bits.
#include <cmath>
#include <type_traits>

#include "tgs_orthogonal.h"

namespace tgs {

typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kBK = 64;        // summation indices a stage: rows of 128 bytes in LDS

// ------------------------------------------------------- norm and packing --
struct NormArgs {
  const void* x;    // [batch][rows][cols] matrix or gradient
  float* momentum;  // [batch][rows][cols], or null: x itself is orthogonalised
  double* part;     // [batch][blocks]
  int64_t count;    // rows * cols
  int blocks, nesterov;
  float beta;
};

struct PackArgs {
  const void* x;
  const float* momentum;
  const double* part;
  _Float16* xh;      // [batch][mp][np] high and low parts of X
  _Float16* xl;
  _Float16* th;      // [batch][np][mp] the transpose
  _Float16* tl;      // null: high part only
  int64_t count;     // rows * cols
  int rows, cols, mp, np, blocks;
  int tall;          // rows > cols: X is the transpose of x
  int nesterov;
  float beta, sx;
  double eps;
};

template <class T, bool MUON>
__global__ __launch_bounds__(256) void k_ns_norm(NormArgs a) {
  __shared__ double s_sum[4];
  const int64_t base = (int64_t)blockIdx.y * a.count;
  const T* x = (const T*)a.x + base;
  float* mom = MUON ? a.momentum + base : nullptr;
  double sum = 0.0;
  constexpr int E = 4;
  const int64_t step = (int64_t)gridDim.x * 256 * E;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * E; i < a.count; i += step) {
    if (i + E <= a.count) {
      const Vec<T, E> g = load_vec<T, E>(x + i);
      Vec<float, E> m;
      if (MUON) m = load_vec<float, E>(mom + i);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float v = to_f32(g.v[e]);
        if (MUON) {
          m.v[e] = new_momentum(a.beta, m.v[e], v);
          v = muon_u(a.nesterov, a.beta, v, m.v[e]);
        }
        sum = fma((double)v, (double)v, sum);
      }
      if (MUON) store_vec<float, E>(mom + i, m);
    } else {
      for (int64_t j = i; j < a.count; ++j) {
        float v = to_f32(x[j]);
        if (MUON) {
          const float m = new_momentum(a.beta, mom[j], v);
          mom[j] = m;
          v = muon_u(a.nesterov, a.beta, v, m);
        }
        sum = fma((double)v, (double)v, sum);
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane_id() == 0) s_sum[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.part[(int64_t)blockIdx.y * a.blocks + blockIdx.x] = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
}

void launch_norm(const NsCall& q, double* part, int blocks, hipStream_t stream) {
  NormArgs a{};
  a.x = q.x;
  a.momentum = q.momentum;
  a.part = part;
  a.count = q.rows * q.cols;
  a.blocks = blocks;
  a.nesterov = q.nesterov;
  a.beta = q.beta;
  with_float_dtype(q.x_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const dim3 grid(blocks, (unsigned)q.batch);
    if (q.momentum) hipLaunchKernelGGL((k_ns_norm<T, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_ns_norm<T, false>), grid, dim3(256), 0, stream, a);
  });
}

// One 64 x 64 tile of x: normalised, scaled, written to X and its transpose,
// zeros outside the matrix.  The tile of X lies at (r0, c0) of the padded
// matrix; x is read in its own order and turned in LDS.
template <class T, bool MUON>
__global__ __launch_bounds__(256) void k_ns_pack(PackArgs a) {
  __shared__ float s_t[64][65];
  const int64_t base = (int64_t)blockIdx.z * a.count;
  const T* x = (const T*)a.x + base;
  const float* mom = MUON ? a.momentum + base : nullptr;
  // every wave adds the partial sums itself, in the same order
  double sum = 0.0;
  for (int i = lane_id(); i < a.blocks; i += kWave) sum += a.part[(int64_t)blockIdx.z * a.blocks + i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  const double inv = 1.0 / (sqrt(sum) + a.eps);
  // rows and columns of x's own order
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
#pragma unroll 4
  for (int i = ty; i < 64; i += 4) {
    const int r = r0 + i, c = c0 + tx;
    float v = 0.0f;
    if (r < a.rows && c < a.cols) {
      v = to_f32(x[(int64_t)r * a.cols + c]);
      if (MUON) v = muon_u(a.nesterov, a.beta, v, mom[(int64_t)r * a.cols + c]);
      v = (float)((double)v * inv) * a.sx;
    }
    s_t[i][tx] = v;
  }
  __syncthreads();
  const int64_t plane = (int64_t)blockIdx.z * a.mp * a.np;
  // in x's order: X, or its transpose where x is tall
  const int ld = a.tall ? a.mp : a.np, ldt = a.tall ? a.np : a.mp;
  const int vec = threadIdx.x % 8, line = threadIdx.x / 8;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = half * 32 + line;
    h8 h, l, hx, lx;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      _Float16 p, q;
      split_half(s_t[i][vec * 8 + e], p, q);
      h[e] = p;
      l[e] = q;
      split_half(s_t[vec * 8 + e][i], p, q);
      hx[e] = p;
      lx[e] = q;
    }
    const int64_t at = plane + (int64_t)(r0 + i) * ld + c0 + vec * 8;
    const int64_t att = plane + (int64_t)(c0 + i) * ldt + r0 + vec * 8;
    if (a.tall) {
      *(h8*)(a.th + at) = h;
      if (a.tl) *(h8*)(a.tl + at) = l;
      *(h8*)(a.xh + att) = hx;
      *(h8*)(a.xl + att) = lx;
    } else {
      *(h8*)(a.xh + at) = h;
      *(h8*)(a.xl + at) = l;
      *(h8*)(a.th + att) = hx;
      if (a.tl) *(h8*)(a.tl + att) = lx;
    }
  }
}

// --------------------------------------------------------------- products --
enum Product { kGram, kSquare, kUpdate, kLast };

struct ProductArgs {
  // operands of C = L R^T: [rows][ld], summation length k (a multiple of 64);
  // the low parts lie `low` elements behind the high ones
  const _Float16* l;
  const _Float16* r;
  int64_t l_low, r_low;
  int64_t l_batch, r_batch;  // elements between matrices of a batch
  int ld, k;
  int mp, np;      // C is [mp][mp] (gram, square) or [mp][np]
  int tiles_n;     // column tiles (update)
  float scale;     // accumulator to true value
  // in/out of the epilogues
  float* diag_a;   // [batch][mp] diagonal of A
  float* diag_p;   // [batch][mp] diagonal of P
  _Float16* e;     // gram: out, square: in; off-diagonal part of A, low part e_low behind
  _Float16* p;     // square: out
  int64_t e_low, p_low;
  _Float16* xh;    // update: X in and out
  _Float16* xl;
  _Float16* th;    // update: transpose out
  _Float16* tl;
  float store;     // scale of what is stored
  float load;      // 1 / scale of X or E as read
  float ca, cb, cc;
  // last step
  void* out;       // [batch][rows][cols]: result, or the weights that are updated
  int rows, cols, tall;
  float keep, gain;  // muon: w = keep * w + gain * O
};

// Stage layout: row r of a 64-column stage is 8 chunks of 16 bytes, chunk c at
// place c ^ ((r >> 1) & 7).
__device__ __forceinline__ int chunk_place(int r, int c) { return c ^ ((r >> 1) & 7); }

// 16 bytes a lane from global memory to LDS (base + 16 * lane), asynchronously.
__device__ __forceinline__ void load_to_lds(const _Float16* from, _Float16* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

template <int ROWS, int WAVES>
__device__ __forceinline__ void load_stage(const _Float16* base, const u32 (&off)[ROWS / (8 * WAVES)], _Float16* lds,
                                           int wave) {
#pragma unroll
  for (int i = 0; i < ROWS / (8 * WAVES); ++i) load_to_lds(base + off[i], lds + (i * WAVES + wave) * 8 * kBK);
}

template <int MI, int NI>
__device__ __forceinline__ void multiply_stage(const _Float16* sl, const _Float16* sr, int l_row, int r_row,
                                               f16v (&acc)[MI][NI]) {
  const int lane = lane_id(), i = lane & 31, hi = lane >> 5;
#pragma unroll
  for (int kk = 0; kk < kBK / 16; ++kk) {
    h8 x[MI], y[NI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      const int row = l_row + mi * 32 + i;
      x[mi] = *(const h8*)(sl + row * kBK + chunk_place(row, kk * 2 + hi) * 8);
    }
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const int row = r_row + ni * 32 + i;
      y[ni] = *(const h8*)(sr + row * kBK + chunk_place(row, kk * 2 + hi) * 8);
    }
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[mi], y[ni], acc[mi][ni], 0, 0, 0);
  }
}

// Eight columns of one row of the result, in place in v: the epilogue's values
// in the scale that is stored; written in row order.
template <Product K, bool SPLIT, class TW, bool MUON>
__device__ __forceinline__ void finish_row(const ProductArgs& a, int64_t plane_c, int64_t diag, int row, int col,
                                           float (&v)[8], float d_row) {
  const int ldc = K == kGram || K == kSquare ? a.mp : a.np;
  const int64_t at = plane_c + (int64_t)row * ldc + col;
  if constexpr (K == kGram) {
    h8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = v[e] * a.scale;
      if (row == col + e) a.diag_a[diag + row] = t;
      v[e] = row == col + e ? 0.0f : t * a.store;
      _Float16 p, q;
      split_half(v[e], p, q);
      h[e] = p;
      l[e] = q;
    }
    *(h8*)(a.e + at) = h;
    if (SPLIT) *(h8*)(a.e + a.e_low + at) = l;
  } else if constexpr (K == kSquare) {
    const h8 eh = *(const h8*)(a.e + at);
    h8 el;
    if (SPLIT) el = *(const h8*)(a.e + a.e_low + at);
    h8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float off = ((float)eh[e] + (SPLIT ? (float)el[e] : 0.0f)) * a.load;
      const float sq = v[e] * a.scale;
      const float d_col = a.diag_a[diag + col + e];
      if (row == col + e) a.diag_p[diag + row] = fmaf(a.cc, fmaf(d_row, d_row, sq), a.cb * d_row);
      const float t = fmaf(a.cc, sq, fmaf(a.cc, d_row + d_col, a.cb) * off);
      v[e] = row == col + e ? 0.0f : t * a.store;
      _Float16 p, q;
      split_half(v[e], p, q);
      h[e] = p;
      l[e] = q;
    }
    *(h8*)(a.p + at) = h;
    if (SPLIT) *(h8*)(a.p + a.p_low + at) = l;
  } else {
    const h8 xh = *(const h8*)(a.xh + at), xl = *(const h8*)(a.xl + at);
    h8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = ((float)xh[e] + (float)xl[e]) * a.load;
      v[e] = fmaf(a.ca + d_row, x, v[e] * a.scale) * a.store;
      if (K == kUpdate) {
        _Float16 p, q;
        split_half(v[e], p, q);
        h[e] = p;
        l[e] = q;
      }
    }
    if (K == kUpdate) {
      *(h8*)(a.xh + at) = h;
      *(h8*)(a.xl + at) = l;
    }
  }
}

// Eight consecutive results of the last step, to the caller's array.
template <class TW, bool MUON>
__device__ __forceinline__ void put_result(const ProductArgs& a, int64_t plane_o, int r, int c, const float (&v)[8]) {
  if (r >= a.rows || c >= a.cols) return;
  TW* p = (TW*)a.out + plane_o + (int64_t)r * a.cols + c;
  if (c + 8 <= a.cols) {
    Vec<TW, 8> y;
    if (MUON) y = load_vec<TW, 8>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      y.v[e] = from_f32<TW>(MUON ? fmaf(a.keep, to_f32(y.v[e]), a.gain * v[e]) : v[e]);
    store_vec<TW, 8>(p, y);
  } else {
    for (int e = 0; e < 8 && c + e < a.cols; ++e)
      p[e] = from_f32<TW>(MUON ? fmaf(a.keep, to_f32(p[e]), a.gain * v[e]) : v[e]);
  }
}

template <Product K, bool SPLIT, class TW, bool MUON, int BM, int BN, int WR, int WC>
__global__ __launch_bounds__(WR* WC* kWave) void k_ns_product(ProductArgs a) {
  constexpr int WAVES = WR * WC, WM = BM / WR, WN = BN / WC, MI = WM / 32, NI = WN / 32;
  __shared__ __align__(16) _Float16 s_l0[BM * kBK], s_r0[BN * kBK], s_l1[BM * kBK], s_r1[BN * kBK];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  constexpr bool SYM = K == kGram || K == kSquare;
  int tm, tn;
  if (SYM) {  // the t-th tile of the lower triangle, row by row
    const int t = blockIdx.x;
    tm = (int)((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
    while (tm * (tm + 1) / 2 > t) --tm;
    tn = t - tm * (tm + 1) / 2;
  } else {
    tm = blockIdx.x / a.tiles_n;
    tn = blockIdx.x - tm * a.tiles_n;
  }
  const int batch = blockIdx.y;
  // this lane's part of each stage: 8 rows of 8 chunks a wave and load
  u32 off_l[BM / (8 * WAVES)], off_r[BN / (8 * WAVES)];
#pragma unroll
  for (int i = 0; i < BM / (8 * WAVES); ++i) {
    const int row = (i * WAVES + wave) * 8 + lane / 8;
    off_l[i] = (u32)(row * a.ld + chunk_place(row, lane % 8) * 8);
  }
#pragma unroll
  for (int i = 0; i < BN / (8 * WAVES); ++i) {
    const int row = (i * WAVES + wave) * 8 + lane / 8;
    off_r[i] = (u32)(row * a.ld + chunk_place(row, lane % 8) * 8);
  }
  const _Float16* gl = a.l + (int64_t)batch * a.l_batch + (int64_t)tm * BM * a.ld;
  const _Float16* gr = a.r + (int64_t)batch * a.r_batch + (int64_t)tn * BN * a.ld;
  const int kt = a.k / kBK, nt = SPLIT ? 3 * kt : kt;
  // stage t of the sum: high x low, low x high, high x high where split
  auto load = [&](int t, _Float16* sl, _Float16* sr) {
    int64_t ol, orr;
    if (SPLIT) {
      const int seg = t >= 2 * kt ? 2 : t >= kt ? 1 : 0;
      const int64_t k0 = (int64_t)(t - seg * kt) * kBK;
      ol = k0 + (seg == 1 ? a.l_low : 0);
      orr = k0 + (seg == 0 ? a.r_low : 0);
    } else {
      ol = orr = (int64_t)t * kBK;
    }
    load_stage<BM, WAVES>(gl + ol, off_l, sl, wave);
    load_stage<BN, WAVES>(gr + orr, off_r, sr, wave);
  };
  const int l_row = (wave / WC) * WM, r_row = (wave % WC) * WN;
  f16v acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[mi][ni][q] = 0.0f;
  load(0, s_l0, s_r0);
  __syncthreads();
  for (int t = 0; t < nt; t += 2) {
    if (t + 1 < nt) load(t + 1, s_l1, s_r1);
    multiply_stage<MI, NI>(s_l0, s_r0, l_row, r_row, acc);
    __syncthreads();
    if (t + 1 >= nt) break;
    if (t + 2 < nt) load(t + 2, s_l0, s_r0);
    multiply_stage<MI, NI>(s_l1, s_r1, l_row, r_row, acc);
    __syncthreads();
  }
  // Epilogue: every wave turns its tile in its own part of LDS, 32 rows at a
  // time: once out in row order (16 bytes a lane), once transposed.
  constexpr int LD = WN + 2;
  static_assert(32 * LD * 4 * (WAVES / 4) <= BM * kBK * 2 && BM == BN, "a wave's strip fits its part of a stage");
  _Float16* part = wave * 4 / WAVES == 0 ? s_l0 : wave * 4 / WAVES == 1 ? s_r0 : wave * 4 / WAVES == 2 ? s_l1 : s_r1;
  float* strip = (float*)part + (wave % (WAVES / 4)) * 32 * LD;
  const int64_t diag = (int64_t)batch * a.mp;
  const int64_t plane_c = (int64_t)batch * a.mp * (SYM ? a.mp : a.np);
  const int64_t plane_o = (int64_t)batch * a.rows * a.cols;
  const int row0 = tm * BM + l_row, col0 = tn * BN + r_row;
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int q = 0; q < 16; ++q)
        strip[(8 * (q / 4) + 4 * (lane >> 5) + q % 4) * LD + ni * 32 + (lane & 31)] = acc[mi][ni][q];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    constexpr int VR = WN / 8;  // vectors a row
#pragma unroll
    for (int it = 0; it < 32 * VR / kWave; ++it) {
      const int r = (it * kWave + lane) / VR, c = (it * kWave + lane) % VR * 8;
      float* s = strip + r * LD + c;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = s[e];
      const int row = row0 + mi * 32 + r;
      const float d_row = K == kGram ? 0.0f : (K == kSquare ? a.diag_a : a.diag_p)[diag + row];
      finish_row<K, SPLIT, TW, MUON>(a, plane_c, diag, row, col0 + c, v, d_row);
      if (K == kLast && !a.tall) {
        put_result<TW, MUON>(a, plane_o, row, col0 + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = v[e];
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const bool turned = SYM ? tm != tn : K == kLast ? a.tall != 0 : true;
    if (turned) {
#pragma unroll
      for (int it = 0; it < 32 * VR / kWave; ++it) {
        const int c = (it * kWave + lane) / 4, r = (it * kWave + lane) % 4 * 8;
        float v[8];
        h8 h, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = strip[(r + e) * LD + c];
          _Float16 p, q;
          split_half(v[e], p, q);
          h[e] = p;
          l[e] = q;
        }
        const int row = row0 + mi * 32 + r, col = col0 + c;
        if constexpr (K == kLast) {
          put_result<TW, MUON>(a, plane_o, col, row, v);
        } else {
          const int64_t at = plane_c + (int64_t)col * a.mp + row;
          _Float16* to = K == kGram ? a.e : K == kSquare ? a.p : a.th;
          *(h8*)(to + at) = h;
          if (SPLIT) *(h8*)((K == kGram ? a.e + a.e_low : K == kSquare ? a.p + a.p_low : a.tl) + at) = l;
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// ------------------------------------------------------------------ host --
// 2^e with bound * 2^e <= 2^14.
static float scale_for(double bound) {
  int e = 0;
  if (bound > 0) frexp(bound, &e);  // bound <= 2^e
  return (float)ldexp(1.0, std::max(-60, std::min(40, 14 - e)));
}

// Bounds of |sigma p(sigma^2)| from step to step, singular values in [0, hi].
static bool step_scales(int steps, double a, double b, double c, StepScales* s) {
  double hi = 1.0;
  for (int t = 0; t < steps; ++t) {
    s->x[t] = scale_for(hi);
    s->a[t] = scale_for(hi * hi);
    auto f = [&](double v) { return fabs(v * (a + v * v * (b + v * v * c))); };
    auto g = [&](double q) { return fabs(q * (b + q * c)); };
    const double l = hi * hi;
    double top = f(hi), ptop = g(l);
    if (c != 0) {
      const double q = -b / (2 * c);
      if (q > 0 && q < l) ptop = std::max(ptop, g(q));
      // a + 3 b q + 5 c q^2 = 0
      const double disc = 9 * b * b - 20 * a * c;
      if (disc >= 0)
        for (const double r : {(-3 * b + sqrt(disc)) / (10 * c), (-3 * b - sqrt(disc)) / (10 * c)})
          if (r > 0 && r < l) top = std::max(top, f(sqrt(r)));
    } else if (b != 0) {
      const double q = -a / (3 * b);
      if (q > 0 && q < l) top = std::max(top, f(sqrt(q)));
    }
    s->p[t] = scale_for(ptop);
    hi = top;
    if (!(hi <= 1073741824.0) || !(ptop <= 1073741824.0)) return false;
  }
  s->x[steps] = 1.0f;
  return true;
}

struct NsPlan {
  int m, n, mp, np, tall, tile, blocks;
  bool split, small;
  size_t part, diag_a, diag_p, x, t[2], e, p, total;  // byte offsets
  int64_t x_low, t_low, e_low, p_low;                 // elements between high and low parts
};

static bool ns_plan(int64_t batch, int64_t rows, int64_t cols, bool split, NsPlan* p) {
  if (batch < 1 || batch > 65535 || rows < 1 || cols < 1 || rows > 65536 || cols > 65536) return false;
  p->tall = rows > cols;
  p->m = (int)std::min(rows, cols);
  p->n = (int)std::max(rows, cols);
  p->split = split;
  p->small = p->m <= kSmallSide;
  if (p->small) {
    p->total = small_workspace_bytes(batch, rows, cols);
    return true;
  }
  p->tile = p->m > 512 ? 128 : 64;
  auto up = [](int64_t v, int64_t to) { return (v + to - 1) / to * to; };
  p->mp = (int)up(p->m, p->tile);
  p->np = (int)up(p->n, p->tile);
  p->blocks = (int)std::min<int64_t>(kNormBlocks, up(rows * cols, 4096) / 4096);
  const int64_t xs = batch * p->mp * p->np, as = batch * p->mp * p->mp;
  p->x_low = xs;
  p->t_low = xs;
  p->e_low = p->p_low = as;
  size_t at = kWorkspaceHeader;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += (size_t)up(bytes, 256);
    return here;
  };
  p->part = take(batch * p->blocks * 8);
  p->diag_a = take(batch * p->mp * 4);
  p->diag_p = take(batch * p->mp * 4);
  p->x = take(xs * 4);
  for (size_t& t : p->t) t = take(xs * (split ? 4 : 2));
  p->e = take(as * (split ? 4 : 2));
  p->p = take(as * (split ? 4 : 2));
  p->total = at;
  return true;
}

template <Product K, bool SPLIT, class TW, bool MUON>
static void launch_product(const NsPlan& p, const ProductArgs& a, int batch, hipStream_t stream) {
  const bool sym = K == kGram || K == kSquare;
  const int tm = p.mp / p.tile, tn = p.np / p.tile;
  const dim3 grid(sym ? tm * (tm + 1) / 2 : tm * tn, batch);
  if (p.tile == 128)
    hipLaunchKernelGGL((k_ns_product<K, SPLIT, TW, MUON, 128, 128, 2, 2>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_ns_product<K, SPLIT, TW, MUON, 64, 64, 2, 2>), grid, dim3(256), 0, stream, a);
}

template <bool SPLIT, class TW, bool MUON>
static void run_steps(const NsCall& q, const NsPlan& p, const StepScales& s, char* ws, hipStream_t stream) {
  const int batch = (int)q.batch;
  ProductArgs a{};
  a.mp = p.mp;
  a.np = p.np;
  a.tiles_n = p.np / p.tile;
  a.diag_a = (float*)(ws + p.diag_a);
  a.diag_p = (float*)(ws + p.diag_p);
  a.e = (_Float16*)(ws + p.e);
  a.p = (_Float16*)(ws + p.p);
  a.e_low = p.e_low;
  a.p_low = p.p_low;
  a.xh = (_Float16*)(ws + p.x);
  a.xl = a.xh + p.x_low;
  a.ca = (float)q.a;
  a.cb = (float)q.b;
  a.cc = (float)q.c;
  a.out = q.out;
  a.rows = (int)q.rows;
  a.cols = (int)q.cols;
  a.tall = p.tall;
  a.keep = q.keep;
  a.gain = q.gain;
  for (int t = 0; t < q.steps; ++t) {
    const float sx = s.x[t], sa = s.a[t], sp = s.p[t];
    ProductArgs g = a;
    g.l = g.r = a.xh;
    g.l_low = g.r_low = p.x_low;
    g.l_batch = g.r_batch = (int64_t)p.mp * p.np;
    g.ld = g.k = p.np;
    g.scale = 1.0f / (sx * sx);
    g.store = sa;
    launch_product<kGram, SPLIT, float, false>(p, g, batch, stream);
    g = a;
    g.l = g.r = a.e;
    g.l_low = g.r_low = p.e_low;
    g.l_batch = g.r_batch = (int64_t)p.mp * p.mp;
    g.ld = g.k = p.mp;
    g.scale = 1.0f / (sa * sa);
    g.load = 1.0f / sa;
    g.store = sp;
    launch_product<kSquare, SPLIT, float, false>(p, g, batch, stream);
    g = a;
    g.l = a.p;
    g.l_low = p.p_low;
    g.l_batch = (int64_t)p.mp * p.mp;
    g.r = (const _Float16*)(ws + p.t[t & 1]);
    g.r_low = p.t_low;
    g.r_batch = (int64_t)p.mp * p.np;
    g.th = (_Float16*)(ws + p.t[(t & 1) ^ 1]);
    g.tl = g.th + p.t_low;
    g.ld = g.k = p.mp;
    g.scale = 1.0f / (sp * sx);
    g.load = 1.0f / sx;
    g.store = s.x[t + 1];
    if (t + 1 < q.steps) launch_product<kUpdate, SPLIT, float, false>(p, g, batch, stream);
    else launch_product<kLast, SPLIT, TW, MUON>(p, g, batch, stream);
  }
}

template <bool MUON>
static tgs_status ns_run(const NsCall& q, const NsPlan& p, const StepScales& s, void* workspace, hipStream_t stream) {
  if (p.small) {
    small_run(q, s, workspace, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(TGS_EHIP, "%s: launch failed: %s", q.what, hipGetErrorString(e));
    return TGS_OK;
  }
  char* ws = (char*)workspace;
  PackArgs k{};
  k.x = q.x;
  k.momentum = q.momentum;
  k.part = (const double*)(ws + p.part);
  k.xh = (_Float16*)(ws + p.x);
  k.xl = k.xh + p.x_low;
  k.th = (_Float16*)(ws + p.t[0]);
  k.tl = p.split ? k.th + p.t_low : nullptr;
  k.count = q.rows * q.cols;
  k.rows = (int)q.rows;
  k.cols = (int)q.cols;
  k.mp = p.mp;
  k.np = p.np;
  k.blocks = p.blocks;
  k.tall = p.tall;
  k.nesterov = q.nesterov;
  k.beta = q.beta;
  k.sx = s.x[0];
  k.eps = q.eps;
  launch_norm(q, (double*)(ws + p.part), p.blocks, stream);
  const dim3 tiles((p.tall ? p.mp : p.np) / 64, (p.tall ? p.np : p.mp) / 64, (unsigned)q.batch);
  with_float_dtype(q.x_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    hipLaunchKernelGGL((k_ns_pack<T, MUON>), tiles, dim3(256), 0, stream, k);
  });
  with_float_dtype(q.out_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    run_steps<sizeof(T) == 4, T, MUON>(q, p, s, ws, stream);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TGS_EHIP, "%s: launch failed: %s", q.what, hipGetErrorString(e));
  return TGS_OK;
}

// The checks both entries share; on TGS_OK the plan and scales are set.
static tgs_status ns_check(const NsCall& q, NsPlan* p, StepScales* s, const void* workspace, size_t workspace_bytes) {
  if (!is_float_dtype(q.x_dtype) || !is_float_dtype(q.out_dtype))
    return fail(TGS_EINVAL, "%s: values must be fp32, bf16 or fp16", q.what);
  if (!ns_plan(q.batch, q.rows, q.cols, q.out_dtype == TGS_FP32, p))
    return fail(TGS_EINVAL, "%s: batch=%lld rows=%lld cols=%lld outside [1, 65535], [1, 65536], [1, 65536]", q.what,
                (long long)q.batch, (long long)q.rows, (long long)q.cols);
  if (q.steps < 1 || q.steps > kMaxSteps)
    return fail(TGS_EINVAL, "%s: steps=%d outside [1, %d]", q.what, q.steps, kMaxSteps);
  for (const double v : {q.a, q.b, q.c, q.eps})
    if (!std::isfinite((float)v)) return fail(TGS_EINVAL, "%s: a coefficient or eps is not finite", q.what);
  if (q.eps < 0) return fail(TGS_EINVAL, "%s: eps is negative", q.what);
  if (!step_scales(q.steps, q.a, q.b, q.c, s))
    return fail(TGS_EINVAL, "%s: the coefficients let singular values grow past 2^30", q.what);
  if (!q.x || !q.out) return fail(TGS_EINVAL, "%s: null pointer", q.what);
  if (((uintptr_t)q.x & (dtype_bytes(q.x_dtype) - 1)) != 0 || ((uintptr_t)q.out & (dtype_bytes(q.out_dtype) - 1)) != 0)
    return fail(TGS_EINVAL, "%s: an array is not aligned to its type", q.what);
  if (!workspace) return fail(TGS_EINVAL, "%s: null workspace", q.what);
  if (((uintptr_t)workspace & 255u) != 0) return fail(TGS_EINVAL, "%s: workspace not 256-byte aligned", q.what);
  if (workspace_bytes < p->total)
    return fail(TGS_EWORKSPACE, "%s: workspace %zu bytes, need %zu", q.what, workspace_bytes, p->total);
  const size_t count = (size_t)q.batch * (size_t)q.rows * (size_t)q.cols;
  const size_t xb = count * dtype_bytes(q.x_dtype), ob = count * dtype_bytes(q.out_dtype);
  if (overlaps(q.x, xb, workspace, p->total) || overlaps(q.out, ob, workspace, p->total))
    return fail(TGS_EINVAL, "%s: an array overlaps the workspace", q.what);
  return TGS_OK;
}

}  // namespace tgs

using namespace tgs;

extern "C" size_t tgs_newton_schulz_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, tgs_dtype dtype) {
  NsPlan p;
  return is_float_dtype(dtype) && ns_plan(batch, rows, cols, dtype == TGS_FP32, &p) ? p.total : 0;
}

extern "C" tgs_status tgs_newton_schulz(const void* x, tgs_dtype dtype, int64_t batch, int64_t rows, int64_t cols,
                                        int32_t steps, float a, float b, float c, float eps, void* out,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  NsCall q{};
  q.what = "newton_schulz";
  q.x = x;
  q.x_dtype = q.out_dtype = dtype;
  q.out = out;
  q.batch = batch;
  q.rows = rows;
  q.cols = cols;
  q.steps = steps;
  q.a = a;
  q.b = b;
  q.c = c;
  q.eps = eps;
  NsPlan p;
  StepScales s;
  const tgs_status st = ns_check(q, &p, &s, workspace, workspace_bytes);
  if (st != TGS_OK) return st;
  const size_t bytes = (size_t)batch * (size_t)rows * (size_t)cols * dtype_bytes(dtype);
  if (x != out && overlaps(x, bytes, out, bytes))
    return fail(TGS_EINVAL, "newton_schulz: out overlaps x (it may be x itself)");
  return ns_run<false>(q, p, s, workspace, stream);
}

extern "C" size_t tgs_muon_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, tgs_dtype weight_dtype) {
  return tgs_newton_schulz_workspace_bytes(batch, rows, cols, weight_dtype);
}

extern "C" tgs_status tgs_muon_step(void* weight, tgs_dtype weight_dtype, const void* grad, tgs_dtype grad_dtype,
                                    float* momentum, int64_t batch, int64_t rows, int64_t cols, float lr, float beta,
                                    int32_t nesterov, float weight_decay, int32_t steps, float a, float b, float c,
                                    float eps, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  NsCall q{};
  q.what = "muon_step";
  q.x = grad;
  q.x_dtype = grad_dtype;
  q.momentum = momentum;
  q.out = weight;
  q.out_dtype = weight_dtype;
  q.batch = batch;
  q.rows = rows;
  q.cols = cols;
  q.beta = beta;
  q.nesterov = nesterov != 0;
  q.steps = steps;
  q.a = a;
  q.b = b;
  q.c = c;
  q.eps = eps;
  for (const float v : {lr, beta, weight_decay})
    if (!std::isfinite(v)) return fail(TGS_EINVAL, "muon_step: lr, beta or weight_decay is not finite");
  NsPlan p;
  StepScales s;
  const tgs_status st = ns_check(q, &p, &s, workspace, workspace_bytes);
  if (st != TGS_OK) return st;
  q.keep = (float)(1.0 - (double)lr * weight_decay);
  q.gain = (float)(-(double)lr * sqrt(std::max(1.0, (double)rows / (double)cols)));
  if (!momentum) return fail(TGS_EINVAL, "muon_step: null momentum");
  if (((uintptr_t)momentum & 3u) != 0) return fail(TGS_EINVAL, "muon_step: momentum not aligned to its type");
  const size_t count = (size_t)batch * (size_t)rows * (size_t)cols;
  const size_t wb = count * dtype_bytes(weight_dtype), gb = count * dtype_bytes(grad_dtype), mb = count * 4;
  if (overlaps(weight, wb, grad, gb) || overlaps(weight, wb, momentum, mb) || overlaps(grad, gb, momentum, mb) ||
      overlaps(momentum, mb, workspace, p.total))
    return fail(TGS_EINVAL, "muon_step: weight, grad, momentum and the workspace must not overlap");
  return ns_run<true>(q, p, s, workspace, stream);
}
