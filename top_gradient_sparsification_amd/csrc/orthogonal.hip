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
// A workgroup makes a tile of C: stages of 128 bytes a row of both operands go
// from memory to a ring in LDS (asynchronous loads, one to three stages ahead),
// the operands of the next 16 summation indices are read while these are
// multiplied.  Square tiles of 64 to 256 a side, picked by a model of the time
// (pick_shape).  256 tiles of 256 (4,096 square, update) take 141 us, as a library's
// 4,096 product does (114 us without the epilogue); the symmetric products of
// that size take 253 tiles of 192 rather than 136 of 256, which leave half the
// device idle (four products of 4,096: 1,653 against 1,843 us for the whole
// call).  Small matrices with a long side have few tiles with long sums, so
// workgroups share them (gram of 200 x 8,000: 31 -> 12 us).
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

constexpr int kBK = 64;         // elements of a row a stage: rows of 128 bytes in LDS
constexpr int kSplitCols = 32;  // columns of high parts, then as many of low parts, in a split row

// Where a matrix of rows of ld elements holds (row, col).  Split matrices
// interleave: 32 columns' high parts, then their low parts, so that a stage of
// 128 bytes a row holds both.
template <bool SPLIT>
__device__ __forceinline__ int64_t place_of(int row, int col, int ld) {
  return SPLIT ? (int64_t)row * 2 * ld + (col / kSplitCols) * 2 * kSplitCols + col % kSplitCols : (int64_t)row * ld + col;
}

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
  _Float16* x_out;   // X, then low parts x_low behind
  _Float16* t_out;   // the transpose; with split, low parts as X
  int64_t x_low;
  int64_t count;     // rows * cols
  int rows, cols, mp, np, blocks;
  int split;
  u32* arrived;  // counters to clear
  int arrive;
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
  constexpr int E = 8;
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
  {
    const int64_t i = (((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (i < a.arrive) a.arrived[i] = 0;
  }
  // every workgroup adds the partial sums itself, in the same order
  __shared__ double s_sum[4];
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.blocks; i += 256) sum += a.part[(int64_t)blockIdx.z * a.blocks + i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane_id() == 0) s_sum[threadIdx.x / kWave] = sum;
  __syncthreads();
  sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
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
  // in x's order: X, or its transpose where x is tall
  const int64_t plane = (int64_t)blockIdx.z * a.mp * a.np * (a.split ? 2 : 1);
  const int ld = a.tall ? a.mp : a.np, ldt = a.tall ? a.np : a.mp;
  const int vec = threadIdx.x % 8, line = threadIdx.x / 8;
  auto put = [&](int row, int col, int stride, bool is_x, h8 h, h8 l) {
    _Float16* to = (is_x ? a.x_out : a.t_out) + plane +
                   (a.split ? place_of<true>(row, col, stride) : place_of<false>(row, col, stride));
    *(h8*)to = h;
    if (a.split) *(h8*)(to + kSplitCols) = l;
    else if (is_x) *(h8*)(to + a.x_low) = l;
  };
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
    put(r0 + i, c0 + vec * 8, ld, !a.tall, h, l);
    put(c0 + i, r0 + vec * 8, ldt, a.tall, hx, lx);
  }
}

// --------------------------------------------------------------- products --
enum Product { kGram, kSquare, kUpdate, kLast };

struct ProductArgs {
  // operands of C = L R^T: rows `stride` elements apart, `stages` stages of 64 elements
  const _Float16* l;
  const _Float16* r;
  int64_t l_batch, r_batch;  // elements between matrices of a batch
  int stride, stages;
  int mp, np;      // C is [mp][mp] (gram, square) or [mp][np]
  int tiles, tiles_n;  // tiles a matrix; of them in a row (update)
  int units, share;  // gram, square: stages of all tiles, and of them a workgroup's
  float* sums;       // gram, square: [workgroups][2][B * B] partial sums of tiles that workgroups share
  u32* arrived;      // of their workgroups, per tile; zero between products
  float scale;     // accumulator to true value
  // in/out of the epilogues
  float* diag_a;   // [batch][mp] diagonal of A
  float* diag_p;   // [batch][mp] diagonal of P
  _Float16* e;     // gram: out, square: in; off-diagonal part of A
  _Float16* p;     // square: out
  _Float16* x;     // update: X in and out
  _Float16* t;     // update: transpose out
  int64_t x_low;   // X's low parts behind its high ones (not split)
  float store;     // scale of what is stored
  float load;      // 1 / scale of X or E as read
  float ca, cb, cc;
  // last step
  void* out;       // [batch][rows][cols]: result, or the weights that are updated
  int rows, cols, tall;
  float keep, gain;  // muon: w = keep * w + gain * O
};

// A workgroup's share of a product: a B x B tile, WR x WC waves, a ring of S
// stages in LDS.  SHARE: workgroups take equal runs of the list of all tiles'
// stages (symmetric products).
template <int B_, int WR_, int WC_, int S_, bool SHARE_ = false>
struct Shape {
  static constexpr bool SHARE = SHARE_;
  static constexpr int B = B_, WR = WR_, WC = WC_, S = S_, WAVES = WR_ * WC_;
  static constexpr int WM = B_ / WR_, WN = B_ / WC_, MI = WM / 32, NI = WN / 32;
  static constexpr int LOADS = 2 * B_ / (8 * WAVES);  // 16-byte loads a lane and stage
};

// Stage layout: row r of a 64-element stage is 8 chunks of 16 bytes, chunk c at
// place c ^ ((r >> 1) & 7): 16 lanes that read one chunk of 16 rows then cover
// all 64 banks.
__device__ __forceinline__ int chunk_place(int r, int c) { return c ^ ((r >> 1) & 7); }

// 16 bytes a lane from global memory to LDS (base + 16 * lane), asynchronously.
__device__ __forceinline__ void load_to_lds(const char* from, _Float16* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Waits until at most `left` (0, 1 or 2) stages of N loads each are in flight
// and every read of LDS is done, then meets the other waves: what they loaded
// is there, and what they read may be overwritten.
template <int N>
__device__ __forceinline__ void stage_barrier(int left) {
  if (left >= 2) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * N) : "memory");
  else if (left == 1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
  else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// What the epilogue reads for eight columns of one row, fetched ahead of the
// stores before it (which the compiler must take for changing it).
template <class TW>
struct Fetched {
  h8 hi, lo;       // X, or E
  float d_row;     // of P's diagonal, or A's
  Vec<TW, 8> old;  // weights
};

// Eight columns of one row of the result, in place in v: the epilogue's values
// in the scale that is stored; written in row order.
template <Product K, bool SPLIT, class TW>
__device__ __forceinline__ void finish_row(const ProductArgs& a, int64_t at, int64_t diag, int row, int col,
                                           float (&v)[8], const Fetched<TW>& f, const float (&d_col)[8]) {
  const int64_t x_low = SPLIT ? kSplitCols : a.x_low;
  h8 h, l;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (K == kGram) {
      const float t = v[e] * a.scale;
      if (row == col + e) a.diag_a[diag + row] = t;
      v[e] = row == col + e ? 0.0f : t * a.store;
    } else if constexpr (K == kSquare) {
      const float off = ((float)f.hi[e] + (SPLIT ? (float)f.lo[e] : 0.0f)) * a.load;
      const float sq = v[e] * a.scale;
      if (row == col + e) a.diag_p[diag + row] = fmaf(a.cc, fmaf(f.d_row, f.d_row, sq), a.cb * f.d_row);
      const float t = fmaf(a.cc, sq, fmaf(a.cc, f.d_row + d_col[e], a.cb) * off);
      v[e] = row == col + e ? 0.0f : t * a.store;
    } else {
      const float x = ((float)f.hi[e] + (float)f.lo[e]) * a.load;
      v[e] = fmaf(a.ca + f.d_row, x, v[e] * a.scale) * a.store;
    }
    _Float16 p, q;
    split_half(v[e], p, q);
    h[e] = p;
    l[e] = q;
  }
  if constexpr (K == kUpdate) {
    *(h8*)(a.x + at) = h;
    *(h8*)(a.x + at + x_low) = l;
  } else if constexpr (K != kLast) {
    _Float16* to = (K == kGram ? a.e : a.p) + at;
    *(h8*)to = h;
    if (SPLIT) *(h8*)(to + kSplitCols) = l;
  }
}

// Eight consecutive results of the last step, to the caller's array.
template <class TW, bool MUON>
__device__ __forceinline__ void put_result(const ProductArgs& a, int64_t plane_o, int r, int c, const float (&v)[8],
                                           Vec<TW, 8> old) {
  if (r >= a.rows || c >= a.cols) return;
  TW* p = (TW*)a.out + plane_o + (int64_t)r * a.cols + c;
  if (c + 8 <= a.cols) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      old.v[e] = from_f32<TW>(MUON ? fmaf(a.keep, to_f32(old.v[e]), a.gain * v[e]) : v[e]);
    store_vec<TW, 8>(p, old);
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (c + e < a.cols) p[e] = from_f32<TW>(MUON ? fmaf(a.keep, to_f32(p[e]), a.gain * v[e]) : v[e]);
  }
}

template <Product K, bool SPLIT, class TW, bool MUON, class G>
__global__ __launch_bounds__(G::WAVES* kWave, G::B == 192 ? 1 : 2) void k_ns_product(ProductArgs a) {
  constexpr int B = G::B, S = G::S, WAVES = G::WAVES, WC = G::WC, WM = G::WM, WN = G::WN, MI = G::MI, NI = G::NI;
  constexpr bool SYM = K == kGram || K == kSquare;
  static_assert(S == 2 || S == 4, "ring");
  // one array a stage, so that reads of one are seen not to depend on loads to another
  __shared__ __align__(16) _Float16 s_0[2 * B * kBK], s_1[2 * B * kBK], s_2[S > 2 ? 2 * B * kBK : 8],
      s_3[S > 2 ? 2 * B * kBK : 8];
  __shared__ int s_state;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  // Workgroups go to the 8 XCDs in turn: each XCD takes a run of neighbouring tiles.
  int id = blockIdx.x;
  {
    const int xcd = id % 8, q = gridDim.x / 8, rest = gridDim.x % 8;
    id = xcd * q + min(xcd, rest) + id / 8;
  }
  // Shared tiles: the stages of all tiles form one list and every workgroup takes
  // an equal run of it.  The last workgroup to arrive at a tile that several
  // share adds their sums, in the order of the stages, and goes on to the epilogue.
  const int wg = id, nt = a.stages;
  int unit = G::SHARE ? wg * a.share : 0;
  const int unit_end = G::SHARE ? min(unit + a.share, a.units) : 1;
  while (unit < unit_end) {
    int first = 0, last = nt;  // stages of the tile
    if (G::SHARE) {
      id = unit / nt;
      first = unit - id * nt;
      last = min(nt, first + unit_end - unit);
      unit += last - first;
    } else {
      unit = 1;
    }
    const int tile = id, batch = id / a.tiles;
    id -= batch * a.tiles;
    int tm, tn;
    if (SYM) {  // the id-th tile of the lower triangle, row by row
      tm = (int)((sqrtf(8.0f * id + 1.0f) - 1.0f) * 0.5f);
      while ((tm + 1) * (tm + 2) / 2 <= id) ++tm;
      while (tm * (tm + 1) / 2 > id) --tm;
      tn = id - tm * (tm + 1) / 2;
    } else {  // groups of four tile rows, column by column
      const int group = id / (4 * a.tiles_n), r0 = group * 4, rows = min(4, (a.mp + B - 1) / B - r0);
      id -= group * 4 * a.tiles_n;
      tn = id / rows;
      tm = r0 + id - tn * rows;
    }
    // this lane's part of each stage, in bytes: 8 rows of 8 chunks a wave and load
    constexpr int HALF = G::LOADS / 2;
    u32 off_l[HALF], off_r[HALF];
    const int cols_c = SYM ? a.mp : a.np;  // a tile may hang over: rows past the end are read as the last one
#pragma unroll
    for (int i = 0; i < HALF; ++i) {
      const int row = (i * WAVES + wave) * 8 + lane / 8;
      off_l[i] = (u32)(min(row, a.mp - 1 - tm * B) * a.stride + chunk_place(row, lane % 8) * 8) * 2;
      off_r[i] = (u32)(min(row, cols_c - 1 - tn * B) * a.stride + chunk_place(row, lane % 8) * 8) * 2;
    }
    const char* gl = (const char*)(a.l + batch * a.l_batch + (int64_t)tm * B * a.stride + (int64_t)first * kBK);
    const char* gr = (const char*)(a.r + batch * a.r_batch + (int64_t)tn * B * a.stride + (int64_t)first * kBK);
    const int count = last - first;
    auto ring = [&](int i) -> _Float16* { return i == 0 ? s_0 : i == 1 ? s_1 : i == 2 ? s_2 : s_3; };
    auto load = [&](int t, _Float16* to) {
#pragma unroll
      for (int i = 0; i < HALF; ++i) load_to_lds(gl + (int64_t)t * (kBK * 2) + off_l[i], to + (i * WAVES + wave) * 8 * kBK);
#pragma unroll
      for (int i = 0; i < HALF; ++i)
        load_to_lds(gr + (int64_t)t * (kBK * 2) + off_r[i], to + B * kBK + (i * WAVES + wave) * 8 * kBK);
    };
    // Operands of 16 summation indices: [high, low parts][blocks of 32 rows]
    constexpr int PARTS = SPLIT ? 2 : 1, KK = SPLIT ? 2 : 4;
    const int l_row = (wave / WC) * WM, r_row = (wave % WC) * WN;
    const int i32 = lane & 31, hi = lane >> 5;
    h8 x[2][PARTS][MI], y[2][PARTS][NI];
    auto read = [&](const _Float16* from, int kk, int to) {
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        const int place = chunk_place(i32, p * 4 + kk * 2 + hi) * 8;  // l_row, r_row: multiples of 32
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) x[to][p][mi] = *(const h8*)(from + (l_row + mi * 32 + i32) * kBK + place);
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) y[to][p][ni] = *(const h8*)(from + (B + r_row + ni * 32 + i32) * kBK + place);
      }
    };
    f16v acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[mi][ni][q] = 0.0f;
    auto multiply = [&](int from) {
#pragma unroll
      for (int q = SPLIT ? 0 : 2; q < 3; ++q)  // high low, low high, high high
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[from][q == 1 ? PARTS - 1 : 0][mi],
                                                                 y[from][q == 0 ? PARTS - 1 : 0][ni], acc[mi][ni], 0, 0, 0);
    };
    // One stage: S - 1 stages are in flight while it is multiplied; the operands
    // of the next 16 indices are read while these are multiplied, over the
    // barrier too.
    auto step = [&](auto at, int t) {
      constexpr int b = decltype(at)::value;
      if (t + S - 1 < count) load(t + S - 1, ring((b + S - 1) % S));
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        if (kk + 1 < KK) {
          read(ring(b), kk + 1, (kk + 1) & 1);
        } else {  // behind the last stage this reads what nothing uses
          stage_barrier<G::LOADS>(min(S - 2, count - t - 2));
          read(ring((b + 1) % S), 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);  // the reads stay ahead of the products
        multiply(kk & 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
      if (i < count) load(i, ring(i));
    stage_barrier<G::LOADS>(min(S - 2, count - 1));
    read(ring(0), 0, 0);
    for (int t = 0; t < count; t += S) {
      step(std::integral_constant<int, 0>{}, t);
      if (B > 64 || t + 1 < count) step(std::integral_constant<int, 1>{}, t + 1);  // B > 64: count is even
      if constexpr (S > 2) {
        if (t + 2 < count) step(std::integral_constant<int, 2>{}, t + 2);
        if (t + 3 < count) step(std::integral_constant<int, 3>{}, t + 3);
      }
    }
    if (G::SHARE && count < nt) {
      // Sums pass between workgroups at device scope (stores written through,
      // loads that miss what a nearer cache holds), ordered by the counter.
      constexpr int PAIRS = MI * NI * 8;
      const int w0 = tile * nt / a.share, n = (tile * nt + nt - 1) / a.share - w0 + 1;
      u32* arrived = a.arrived + tile;
      auto slot = [&](int w) {  // a workgroup's only tile that it does not begin is its first one
        const int64_t at = ((int64_t)w * 2 + (w == w0 ? 1 : 0)) * (B * B / 2);
        return (u64*)a.sums + at + threadIdx.x;
      };
      auto pair = [&](int i) -> u64 {
        const f16v& q = acc[i / 8 / NI][i / 8 % NI];
        return (u64)__float_as_uint(q[i % 8 * 2 + 1]) << 32 | __float_as_uint(q[i % 8 * 2]);
      };
      if (threadIdx.x == 0)
        s_state = __hip_atomic_load(arrived, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (u32)(n - 1);
      __syncthreads();
      if (!s_state) {
        u64* to = slot(wg);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i)
          __hip_atomic_store(to + i * (WAVES * kWave), pair(i), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0)
          s_state = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (u32)(n - 1);
        __syncthreads();
        if (!s_state) continue;
      }
      if (threadIdx.x == 0) __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // s = sum over w0, w0 + 1, ...; this workgroup's own part from registers
      constexpr int BATCH = 8;
#pragma unroll
      for (int i0 = 0; i0 < PAIRS; i0 += BATCH) {
        u64 own[BATCH];
        float lo[BATCH], up[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          own[i] = pair(i0 + i);
          lo[i] = up[i] = 0.0f;
        }
        for (int w = w0; w < w0 + n; ++w) {
          const u64* from = slot(w) + i0 * (WAVES * kWave);
          u64 in[BATCH];
#pragma unroll
          for (int i = 0; i < BATCH; ++i)
            in[i] = w == wg ? own[i]
                            : __hip_atomic_load(from + i * (WAVES * kWave), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            lo[i] += __uint_as_float((u32)in[i]);
            up[i] += __uint_as_float((u32)(in[i] >> 32));
          }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          f16v& q = acc[(i0 + i) / 8 / NI][(i0 + i) / 8 % NI];
          q[(i0 + i) % 8 * 2] = lo[i];
          q[(i0 + i) % 8 * 2 + 1] = up[i];
        }
      }
    }
    // Epilogue: every wave turns its tile in its own part of LDS, 32 rows at a
    // time: once out in row order (16 bytes a lane), once transposed.  What it
    // reads is fetched for 32 rows at once, where registers allow while the rows
    // before are worked on.
    constexpr int VR = WN / 8, ITS = 32 * VR / kWave, LD = WN + 2;  // vectors a row; of them a lane
    constexpr int AHEAD = MI <= 2 ? 1 : 0;
    static_assert(WAVES / 2 * 32 * LD * 4 <= 2 * B * kBK * 2, "a wave's strip fits its part of a stage");
    float* strip = (float*)(wave < WAVES / 2 ? s_0 : s_1) + wave % (WAVES / 2) * 32 * LD;
    const int64_t diag = (int64_t)batch * a.mp;
    const int64_t plane_c = (int64_t)batch * a.mp * (SYM ? a.mp : a.np) * PARTS;
    const int64_t plane_o = (int64_t)batch * a.rows * a.cols;
    const int row0 = tm * B + l_row, col0 = tn * B + r_row;
    auto strip_row = [&](int it) { return (it * kWave + lane) / VR; };
    auto strip_col = [&](int it) { return (it * kWave + lane) % VR * 8; };
    auto at_of = [&](int row, int col) { return plane_c + place_of<SPLIT>(row, col, SYM ? a.mp : a.np); };
    Fetched<TW> f[AHEAD + 1][ITS];
    auto fetch = [&](int mi, Fetched<TW>(&to)[ITS]) {
#pragma unroll
      for (int it = 0; it < ITS; ++it) {
        const int row = row0 + mi * 32 + strip_row(it), col = col0 + strip_col(it);
        if (row >= a.mp || col >= cols_c) continue;
        if constexpr (K != kGram) {
          const _Float16* from = (K == kSquare ? a.e : a.x) + at_of(row, col);
          to[it].hi = *(const h8*)from;
          if (SPLIT) to[it].lo = *(const h8*)(from + kSplitCols);
          else if (K != kSquare) to[it].lo = *(const h8*)(from + a.x_low);
          to[it].d_row = (K == kSquare ? a.diag_a : a.diag_p)[diag + row];
        }
        if constexpr (K == kLast && MUON) {
          const int r = a.tall ? col0 + (it * kWave + lane) / 4 : row;
          const int c = a.tall ? row0 + mi * 32 + lane % 4 * 8 : col;
          if (r < a.rows && c + 8 <= a.cols) to[it].old = load_vec<TW, 8>((const TW*)a.out + plane_o + (int64_t)r * a.cols + c);
        }
      }
    };
    // one column for every it where VR divides the wave
    constexpr int COLS = kWave % VR == 0 ? 1 : ITS;
    float d_col[COLS][8];
    if constexpr (K == kSquare) {
#pragma unroll
      for (int it = 0; it < COLS; ++it)
#pragma unroll
        for (int e = 0; e < 8; ++e) d_col[it][e] = a.diag_a[diag + min(col0 + strip_col(it) + e, a.mp - 1)];
    }
    fetch(0, f[0]);
    __syncthreads();
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      if (AHEAD ? mi + 1 < MI : mi > 0) fetch(mi + AHEAD, f[(mi + AHEAD) & AHEAD]);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          strip[(8 * (q / 4) + 4 * (lane >> 5) + q % 4) * LD + ni * 32 + (lane & 31)] = acc[mi][ni][q];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int it = 0; it < ITS; ++it) {
        const int r = strip_row(it), c = strip_col(it);
        float* s = strip + r * LD + c;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s[e];
        const int row = row0 + mi * 32 + r, col = col0 + c;
        if (row >= a.mp || col >= cols_c) continue;
        finish_row<K, SPLIT, TW>(a, at_of(row, col), diag, row, col, v, f[mi & AHEAD][it], d_col[it % COLS]);
        if (K == kLast && !a.tall) {
          put_result<TW, MUON>(a, plane_o, row, col, v, f[mi & AHEAD][it].old);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = v[e];
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const bool turned = SYM ? tm != tn : K == kLast ? a.tall != 0 : true;
      if (turned) {
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const int c = (it * kWave + lane) / 4, r = lane % 4 * 8;
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
          if (row >= a.mp || col >= cols_c) continue;
          if constexpr (K == kLast) {
            put_result<TW, MUON>(a, plane_o, col, row, v, f[mi & AHEAD][it].old);
          } else {
            _Float16* to = (K == kGram ? a.e : K == kSquare ? a.p : a.t) + plane_c + place_of<SPLIT>(col, row, a.mp);
            *(h8*)to = h;
            if (SPLIT) *(h8*)(to + kSplitCols) = l;
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }    if (G::SHARE) __syncthreads();  // the next tile's stages overwrite the strips
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
  int m, n, mp, np, tall, blocks;
  int shape[3];  // of the gram, the square and the update
  int share[2];  // stages of a workgroup in the gram and the square, where tiles are shared
  int arrive;    // counters to clear
  bool split, small;
  size_t part, diag_a, diag_p, x, t[2], e, p, sums, arrived, total;  // byte offsets
  int64_t x_low;  // elements between X's high and low parts (not split)
};

typedef Shape<64, 2, 2, 4> Tile64;
typedef Shape<64, 2, 2, 4, true> Tile64Shared;
typedef Shape<128, 2, 2, 2> Tile128;
typedef Shape<128, 2, 2, 4> Tile128Deep;
typedef Shape<192, 2, 2, 2> Tile192;
typedef Shape<256, 2, 4, 2> Tile256;
enum { k64, k128, k128Deep, k192, k256, k64Shared, kShapes };
constexpr int kTile[kShapes] = {64, 128, 128, 192, 256, 64};

// The shape of a product is the one with the least time by this model, fitted
// to products of 128 to 8,192 a side: `fixed` us for the first stages' way and
// the epilogue, and a time a stage, lower where every workgroup has a compute
// unit of its own.  With more tiles than fit at once the last round costs about
// a third of a round more than its share.
struct ShapeTime {
  int slots;          // workgroups that fit at once
  float fixed, full, alone;  // us, and us a stage: all slots taken, one workgroup a compute unit
  float full_split, alone_split;
};
constexpr ShapeTime kTime[kShapes] = {
    {512, 4.5f, 0.55f, 0.21f, 0.65f, 0.27f},   {512, 8.0f, 1.05f, 0.75f, 1.3f, 0.95f},
    {256, 8.0f, 0.55f, 0.55f, 0.85f, 0.85f},   {256, 11.0f, 1.05f, 1.05f, 1.45f, 1.45f},
    {256, 14.0f, 1.75f, 1.75f, 2.8f, 2.8f},    {512, 12.5f, 0.3f, 0.25f, 0.4f, 0.3f},
};

static int64_t tiles_of(const NsPlan& p, int64_t batch, int shape, bool symmetric) {
  const int64_t tm = (p.mp + kTile[shape] - 1) / kTile[shape], tn = (p.np + kTile[shape] - 1) / kTile[shape];
  return batch * (symmetric ? tm * (tm + 1) / 2 : tm * tn);
}

// Stages a workgroup takes where tiles are shared: at most four workgroups a
// tile, and eight stages at least.
static int64_t pick_share(int64_t tiles, int64_t nt) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(512, std::min(tiles * 4, tiles * nt / 8)));
  return ((tiles * nt + most - 1) / most + 1) / 2 * 2;
}

static int pick_shape(const NsPlan& p, int64_t batch, int64_t k, bool symmetric) {
  const int64_t nt = k * (p.split ? 2 : 1) / kBK;
  int best = k64;
  double least = 1e30;
  for (int i = 0; i < kShapes; ++i) {
    if (i == k64Shared && !symmetric) continue;
    const ShapeTime& t = kTime[i];
    int64_t work = tiles_of(p, batch, i, symmetric), stages = nt;
    if (i == k64Shared) {
      stages = pick_share(work, nt);
      if (stages >= nt) continue;
      work = (work * nt + stages - 1) / stages;
    }
    const double full = p.split ? t.full_split : t.full, alone = p.split ? t.alone_split : t.alone;
    const double us = t.fixed + stages * (work <= 256        ? alone
                                          : work <= t.slots ? full
                                                            : full * ((double)work / t.slots + 0.35));
    if (us < least) least = us, best = i;
  }
  return best;
}

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
  auto up = [](int64_t v, int64_t to) { return (v + to - 1) / to * to; };
  // tiles may hang over, but shapes above 64 take stages in pairs
  p->mp = (int)up(p->m, 128);
  p->np = (int)up(p->n, 128);
  p->shape[0] = pick_shape(*p, batch, p->np, true);
  p->shape[1] = pick_shape(*p, batch, p->mp, true);
  p->shape[2] = pick_shape(*p, batch, p->mp, false);
  p->blocks = norm_blocks(batch, rows * cols);
  const int64_t xs = batch * p->mp * p->np, as = batch * p->mp * p->mp;
  p->x_low = xs;
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
  int64_t runs = 0;
  p->arrive = 0;
  for (int i = 0; i < 2; ++i) {
    if (p->shape[i] != k64Shared) continue;
    const int64_t tiles = tiles_of(*p, batch, k64Shared, true), nt = (int64_t)(i ? p->mp : p->np) * (split ? 2 : 1) / kBK;
    p->share[i] = (int)pick_share(tiles, nt);
    p->arrive = (int)tiles;
    runs = std::max(runs, (tiles * nt + p->share[i] - 1) / p->share[i]);
  }
  p->sums = take(runs * 2 * 64 * 64 * 4);
  p->arrived = take((int64_t)p->arrive * 4);
  p->total = at;
  return true;
}

template <Product K, bool SPLIT, class TW, bool MUON, class G>
static void launch_tiles(const NsPlan& p, ProductArgs a, int64_t batch, hipStream_t stream) {
  const int tm = (p.mp + G::B - 1) / G::B;
  a.tiles_n = (p.np + G::B - 1) / G::B;
  a.tiles = K == kGram || K == kSquare ? tm * (tm + 1) / 2 : tm * a.tiles_n;
  int64_t blocks = a.tiles * batch;
  if (G::SHARE) {
    a.units = (int)(blocks * a.stages);
    a.share = p.share[K == kSquare];
    blocks = (a.units + a.share - 1) / a.share;
  }
  hipLaunchKernelGGL((k_ns_product<K, SPLIT, TW, MUON, G>), dim3((unsigned)blocks), dim3(G::WAVES * kWave), 0,
                     stream, a);
}

template <Product K, bool SPLIT, class TW, bool MUON>
static void launch_product(const NsPlan& p, const ProductArgs& a, int64_t batch, hipStream_t stream) {
  constexpr bool SYM = K == kGram || K == kSquare;
  switch (p.shape[K == kGram ? 0 : K == kSquare ? 1 : 2]) {
    case k128: return launch_tiles<K, SPLIT, TW, MUON, Tile128>(p, a, batch, stream);
    case k128Deep: return launch_tiles<K, SPLIT, TW, MUON, Tile128Deep>(p, a, batch, stream);
    case k192: return launch_tiles<K, SPLIT, TW, MUON, Tile192>(p, a, batch, stream);
    case k256: return launch_tiles<K, SPLIT, TW, MUON, Tile256>(p, a, batch, stream);
    case k64Shared:
      if constexpr (SYM) launch_tiles<K, SPLIT, TW, MUON, Tile64Shared>(p, a, batch, stream);
      return;
    default: return launch_tiles<K, SPLIT, TW, MUON, Tile64>(p, a, batch, stream);
  }
}

template <bool SPLIT, class TW, bool MUON>
static void run_steps(const NsCall& q, const NsPlan& p, const StepScales& s, char* ws, hipStream_t stream) {
  constexpr int PARTS = SPLIT ? 2 : 1;
  ProductArgs a{};
  a.mp = p.mp;
  a.np = p.np;
  a.diag_a = (float*)(ws + p.diag_a);
  a.diag_p = (float*)(ws + p.diag_p);
  a.e = (_Float16*)(ws + p.e);
  a.p = (_Float16*)(ws + p.p);
  a.x = (_Float16*)(ws + p.x);
  a.x_low = p.x_low;
  a.sums = (float*)(ws + p.sums);
  a.arrived = (u32*)(ws + p.arrived);
  a.ca = (float)q.a;
  a.cb = (float)q.b;
  a.cc = (float)q.c;
  a.out = q.out;
  a.rows = (int)q.rows;
  a.cols = (int)q.cols;
  a.tall = p.tall;
  a.keep = q.keep;
  a.gain = q.gain;
  const int64_t x_size = (int64_t)p.mp * p.np * PARTS, a_size = (int64_t)p.mp * p.mp * PARTS;
  for (int t = 0; t < q.steps; ++t) {
    const float sx = s.x[t], sa = s.a[t], sp = s.p[t];
    ProductArgs g = a;
    g.l = g.r = a.x;
    g.l_batch = g.r_batch = x_size;
    g.stride = p.np * PARTS;
    g.stages = g.stride / kBK;
    g.scale = 1.0f / (sx * sx);
    g.store = sa;
    launch_product<kGram, SPLIT, float, false>(p, g, q.batch, stream);
    g = a;
    g.l = g.r = a.e;
    g.l_batch = g.r_batch = a_size;
    g.stride = p.mp * PARTS;
    g.stages = g.stride / kBK;
    g.scale = 1.0f / (sa * sa);
    g.load = 1.0f / sa;
    g.store = sp;
    launch_product<kSquare, SPLIT, float, false>(p, g, q.batch, stream);
    g = a;
    g.l = a.p;
    g.l_batch = a_size;
    g.r = (const _Float16*)(ws + p.t[t & 1]);
    g.r_batch = x_size;
    g.t = (_Float16*)(ws + p.t[(t & 1) ^ 1]);
    g.stride = p.mp * PARTS;
    g.stages = g.stride / kBK;
    g.scale = 1.0f / (sp * sx);
    g.load = 1.0f / sx;
    g.store = s.x[t + 1];
    if (t + 1 < q.steps) launch_product<kUpdate, SPLIT, float, false>(p, g, q.batch, stream);
    else launch_product<kLast, SPLIT, TW, MUON>(p, g, q.batch, stream);
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
  k.x_out = (_Float16*)(ws + p.x);
  k.t_out = (_Float16*)(ws + p.t[0]);
  k.x_low = p.x_low;
  k.split = p.split;
  k.arrived = (u32*)(ws + p.arrived);
  k.arrive = p.arrive;
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
