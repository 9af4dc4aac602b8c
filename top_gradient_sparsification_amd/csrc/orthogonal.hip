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
// A workgroup makes a tile of C: stages of 128 or 256 bytes a row of both
// operands go from memory to a ring in LDS by asynchronous loads, one to three
// stages ahead, and the operands of the next 16 summation indices are read from
// it while these are multiplied.  Tiles are 64 to 256 a side, whichever a model
// of the time finds best (pick_shape): large ones read less from L2 and feed the
// matrix cores better, small ones fill the device.  At 4,096 square the update
// takes 256 tiles of 256 in 142 us; a library's product of that size, which writes
// 2 bytes an entry of its result where this reads and writes 12, takes 114.  The
// clock falls to about 1.7 GHz under it, and fewer cycles no longer shortened it.
// The symmetric products take 253 tiles of 192 in 85 us rather than 136 of 256,
// which leave half the device idle, in 120.  Few tiles with long sums are shared
// by workgroups (the gram of 200 x 8,000 in fp32: 59 -> 28 us).
// Tiles of 64 and 128 are bound by the rate at which a compute unit fills its
// LDS, about 65 GB/s: 1,000 x 1,533 in fp32 takes 13 to 21 us a product.
//
// What is rounded.  The diagonals of A and P are large against the rest near
// the end (A tends to the identity), so they are held apart in fp32 and the
// products see only the off-diagonal part E of A and of P:
//   A = D + E:   A^2 = D^2 + (d_i + d_j) E + E^2,   P X = D_P X + E_P X.
// X itself is held in fp32, in the order of the update's registers, and a + D_P
// multiplies that; the operands are fp16.  With bf16 results the products read
// high parts only: for matrices like gradients the result is then 2e-4 to 8e-4
// (2-norm) off, below the 1.7e-3 of the final rounding, where rounding X, A and P
// whole to fp16 gives 1.2e-3 to 4.3e-3 and to bf16 1.3e-2 to 2.4e-2.  What X's
// rounding puts into directions in which a matrix of low rank is empty grows by
// the first coefficient a step: such a matrix comes out up to 5e-3 off with a
// shorter side of 65, 3e-3 with 128, 2e-3 with 256, 1.4e-3 with 512.  With fp32
// and fp16 results every operand is high + low and a product is three (high low +
// low high + high high): as exact as fp32 products (1.4e-6 to 2.3e-6 against
// 1.3e-6 to 2.0e-6).  fp16 rounds at 2.1e-4, which single products' 2e-4 to 8e-4
// would pass.
//
// Range.  The singular values of X start in [0, 1]; the host bounds them after
// every step by the polynomial's extrema, and scales X, A and P by powers of
// two so that no entry passes 2^14 and small entries keep their low bits.
#include <cmath>
#include <type_traits>

#include "tgs_orthogonal.h"

namespace tgs {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kSplitCols = 32;  // columns of high parts, then as many of low parts, in a split row

// Where a matrix of rows of ld elements holds (row, col).  Split matrices
// interleave: 32 columns' high parts, then their low parts, so that a stage
// holds both.
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
  _Float16* x_out;   // X and its transpose, operands of the products
  _Float16* t_out;
  float* xf;         // X in fp32, in the order of the update's registers
  int tile, tile_rows, tile_cols;  // of the update: a workgroup's, a wave's rows and columns
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
  // rows and columns of x's own order
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  // all of a thread's loads in flight at once: outside the matrix they read its
  // first entry
  T in[16];
  float in_m[MUON ? 16 : 1];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = r0 + ty + 4 * i, c = c0 + tx;
    const int64_t at = r < a.rows && c < a.cols ? (int64_t)r * a.cols + c : 0;
    in[i] = x[at];
    if (MUON) in_m[i] = mom[at];
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
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v = to_f32(in[i]);
    if (MUON) v = muon_u(a.nesterov, a.beta, v, in_m[i]);
    v = (float)((double)v * inv) * a.sx;
    s_t[ty + 4 * i][tx] = r0 + ty + 4 * i < a.rows && c0 + tx < a.cols ? v : 0.0f;
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
  // a wave writes one block of 32 x 32 of X as the update's wave will hold it
  const int bi = threadIdx.x / 128 * 32, bj = threadIdx.x / 64 % 2 * 32;
  const int row = (a.tall ? c0 : r0) + bi, col = (a.tall ? r0 : c0) + bj;
  const int wr = a.tile / a.tile_rows, wc = a.tile / a.tile_cols;
  const int tiles_m = (a.mp + a.tile - 1) / a.tile, tiles_n = (a.np + a.tile - 1) / a.tile;
  const int wave = row % a.tile / a.tile_rows * wc + col % a.tile / a.tile_cols;
  const int block = row % a.tile_rows / 32 * (a.tile_cols / 32) + col % a.tile_cols / 32;
  const int64_t tile = ((int64_t)blockIdx.z * tiles_m + row / a.tile) * tiles_n + col / a.tile;
  f4* to = (f4*)a.xf + ((tile * (wr * wc) + wave) * (a.tile_rows * a.tile_cols / 1024) + block) * 256 + tx;
  const int h = tx >> 5, c32 = tx & 31;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    f4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = bi + 8 * g + 4 * h + r, j = bj + c32;
      v[r] = a.tall ? s_t[j][i] : s_t[i][j];
    }
    to[g * kWave] = v;
  }
}

// --------------------------------------------------------------- products --
enum Product { kGram, kSquare, kUpdate, kLast };

struct ProductArgs {
  // operands of C = L R^T: rows `stride` elements apart
  const _Float16* l;
  const _Float16* r;
  int64_t l_batch, r_batch;  // elements between matrices of a batch
  int stride, stages;  // stages: of BK elements
  int mp, np;      // C is [mp][mp] (gram, square) or [mp][np]
  int tiles, tiles_n;  // tiles a matrix; of them in a row (update)
  int units, share;  // gram, shared tiles: stages of all tiles, and of them a workgroup's
  float* sums;       // [workgroups][2][B * B] partial sums of tiles that workgroups share
  u32* arrived;      // of their workgroups, per tile; zero between products
  float scale;     // accumulator to true value
  // in/out of the epilogues
  float* diag_a;   // [batch][mp] diagonal of A
  float* diag_p;   // [batch][mp] diagonal of P
  _Float16* e;     // gram: out, square: in; off-diagonal part of A
  _Float16* p;     // square: out
  _Float16* x;     // update: X out
  _Float16* t;     // update: transpose out
  float* xf;       // update: X in fp32, in and out, in the order of the registers
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
// stages (the gram).
template <int B_, int WR_, int WC_, int BK_, int S_, bool SHARE_ = false>
struct Shape {
  static constexpr int BK = BK_, CHUNKS = BK_ / 8, ROWS = 64 / CHUNKS;  // elements and chunks of a row a stage, rows a load
  static constexpr bool SHARE = SHARE_;
  static constexpr int EU = 4 * B_ * BK_ * S_ > 80 * 1024 && WR_ * WC_ == 4 ? 1 : 2;  // waves a SIMD that LDS allows
  static constexpr int B = B_, WR = WR_, WC = WC_, S = S_, WAVES = WR_ * WC_;
  static constexpr int WM = B_ / WR_, WN = B_ / WC_, MI = WM / 32, NI = WN / 32;
  static constexpr int LOADS = 2 * B_ / (ROWS * WAVES);  // 16-byte loads a lane and stage
};

// Stage layout: a row is C chunks of 16 bytes, 8 or 16, turned by the row so that
// 16 lanes that read one chunk of 16 rows cover all 64 banks.
template <int C>
__device__ __forceinline__ int chunk_place(int r, int c) { return c ^ (C == 8 ? (r >> 1) & 7 : r & 15); }

// 16 bytes a lane from global memory to LDS (base + 16 * lane), asynchronously.
__device__ __forceinline__ void load_to_lds(const char* from, _Float16* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Waits until at most LEFT loads are in flight and every read of LDS is done,
// then meets the other waves: what they loaded is there, and what they read may
// be overwritten.
template <int LEFT>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
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
__global__ __launch_bounds__(G::WAVES* kWave, G::EU) void k_ns_product(ProductArgs a) {
  constexpr int B = G::B, S = G::S, WAVES = G::WAVES, WC = G::WC, WM = G::WM, WN = G::WN, MI = G::MI, NI = G::NI;
  constexpr bool SYM = K == kGram || K == kSquare;
  static_assert(S >= 2 && S <= 4, "ring");
  constexpr int BK = G::BK, STAGE = 2 * B * BK;
  // one array a stage, so that reads of one are seen not to depend on loads to another
  __shared__ __align__(16) _Float16 s_0[STAGE], s_1[STAGE], s_2[S > 2 ? STAGE : 8], s_3[S > 3 ? STAGE : 8];
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
      const int row = (i * WAVES + wave) * G::ROWS + lane / G::CHUNKS;
      const int chunk = chunk_place<G::CHUNKS>(row, lane % G::CHUNKS);
      off_l[i] = (u32)(min(row, a.mp - 1 - tm * B) * a.stride + chunk * 8) * 2;
      off_r[i] = (u32)(min(row, cols_c - 1 - tn * B) * a.stride + chunk * 8) * 2;
    }
    const char* gl = (const char*)(a.l + batch * a.l_batch + (int64_t)tm * B * a.stride + (int64_t)first * BK);
    const char* gr = (const char*)(a.r + batch * a.r_batch + (int64_t)tn * B * a.stride + (int64_t)first * BK);
    const int count = last - first;
    auto ring = [&](int i) -> _Float16* { return i == 0 ? s_0 : i == 1 ? s_1 : i == 2 ? s_2 : s_3; };
    auto load = [&](int t, _Float16* to, int i) {  // the i-th of a stage's loads
      const int j = i % HALF * WAVES + wave;
      if (i < HALF) load_to_lds(gl + (int64_t)t * (BK * 2) + off_l[i], to + j * 512);
      else load_to_lds(gr + (int64_t)t * (BK * 2) + off_r[i - HALF], to + B * BK + j * 512);
    };
    // Operands of 16 summation indices: [high, low parts][blocks of 32 rows]
    constexpr int PARTS = SPLIT ? 2 : 1, KK = BK / 16 / PARTS;
    const int l_row = (wave / WC) * WM, r_row = (wave % WC) * WN;
    const int i32 = lane & 31, hi = lane >> 5;
    h8 x[2][PARTS][MI], y[2][PARTS][NI];
    constexpr int READS = PARTS * (MI + NI), PRODUCTS = MI * NI * (SPLIT ? 3 : 1);
    auto read = [&](const _Float16* from, int kk, int to, int i) {  // the i-th of the operands
      const int p = i / (MI + NI), j = i % (MI + NI);
      const int chunk = SPLIT ? kk / 2 * 8 + p * 4 + kk % 2 * 2 : kk * 2;
      const int place = chunk_place<G::CHUNKS>(i32, chunk + hi) * 8;  // l_row, r_row: multiples of 32
      if (j < MI) x[to][p][j] = *(const h8*)(from + (l_row + j * 32 + i32) * BK + place);
      else y[to][p][j - MI] = *(const h8*)(from + (B + r_row + (j - MI) * 32 + i32) * BK + place);
    };
    f16v acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[mi][ni][q] = 0.0f;
    auto multiply = [&](int from, int i) {  // the i-th of the products: high low, low high, high high
      const int q = SPLIT ? i / (MI * NI) : 2, mi = i % (MI * NI) / NI, ni = i % NI;
      acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[from][q == 1 ? PARTS - 1 : 0][mi],
                                                           y[from][q == 0 ? PARTS - 1 : 0][ni], acc[mi][ni], 0, 0, 0);
    };
    // One stage: S - 1 stages are in flight while it is multiplied; the operands
    // of the next 16 indices are read while these are multiplied, over the
    // barrier too.  Reads and loads stand between the products one by one: a row
    // of them would hold the wave up at their queue with the matrix cores idle
    // (8,192 x 2,048 in bf16: 1,036 -> 903 us).  Behind the last stage the loads
    // repeat it and the reads give what nothing uses.
    auto step = [&](auto at, int t) {
      constexpr int b = decltype(at)::value;
      const int ahead = min(t + S - 1, count - 1);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const bool inside = kk + 1 < KK;
        if (!inside) stage_barrier<(S - 2) * G::LOADS>();
        const int l0 = inside ? G::LOADS * kk / (KK - 1) : 0, loads = inside ? G::LOADS * (kk + 1) / (KK - 1) - l0 : 0;
        const int ops = READS + loads;
#pragma unroll
        for (int i = 0; i < PRODUCTS; ++i) {
          multiply(kk & 1, i);
#pragma unroll
          for (int j = ops * i / PRODUCTS; j < ops * (i + 1) / PRODUCTS; ++j) {
            if (j < READS) read(ring(inside ? b : (b + 1) % S), inside ? kk + 1 : 0, (kk + 1) & 1, j);
            else load(ahead, ring((b + S - 1) % S), l0 + j - READS);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    // What the epilogue reads: lane (h, c) holds rows 8 g + 4 h + 0..3 of column c of a
    // block.  Fetched for 32 rows at once, while the rows before are worked on; for
    // all rows ahead of the products where there are 32 only.
    constexpr bool EARLY = MI == 1;
    const int h = hi, c32 = i32;
    const int row0 = tm * B + l_row, col0 = tn * B + r_row;
    const float* diag_in = (K == kSquare ? a.diag_a : a.diag_p) + (int64_t)batch * a.mp;
    const int64_t plane = (int64_t)batch * a.mp * cols_c * PARTS;
    _Float16* by_row = (K == kGram ? a.e : K == kSquare ? a.p : a.x) + plane;
    _Float16* by_col = (K == kGram ? a.e : K == kSquare ? a.p : a.t) + plane;
    f4* xf = (f4*)a.xf + (((int64_t)batch * a.tiles + tm * a.tiles_n + tn) * WAVES + wave) * (MI * NI * 4 * kWave) + lane;
    f4 x_in[2][NI][4], d_in[2][4];
    h4 e_in[2][PARTS][NI][4];
    auto fetch = [&](int mi, int to) {
      if (K == kGram || row0 + mi * 32 >= a.mp) return;
#pragma unroll
      for (int g = 0; g < 4; ++g) d_in[to][g] = *(const f4*)(diag_in + row0 + mi * 32 + 8 * g + 4 * h);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        if (col0 + ni * 32 >= cols_c) continue;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if constexpr (K == kSquare) {  // E is symmetric: its row `col`
            const _Float16* from = a.e + plane + place_of<SPLIT>(col0 + ni * 32 + c32, row0 + mi * 32 + 8 * g + 4 * h, a.mp);
            e_in[to][0][ni][g] = *(const h4*)from;
            if (SPLIT) e_in[to][PARTS - 1][ni][g] = *(const h4*)(from + kSplitCols);
          } else {
            x_in[to][ni][g] = xf[((mi * NI + ni) * 4 + g) * kWave];
          }
        }
      }
    };
    float d_col[NI];
    if constexpr (K == kSquare) {
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        const int col = col0 + ni * 32 + c32;
        d_col[ni] = col < cols_c ? diag_in[col] : 0.0f;
      }
    }
    if (EARLY) fetch(0, 0);
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
#pragma unroll
      for (int j = 0; j < G::LOADS; ++j) load(min(i, count - 1), ring(i), j);
    stage_barrier<(S - 2) * G::LOADS>();
#pragma unroll
    for (int j = 0; j < READS; ++j) read(ring(0), 0, 0, j);
    for (int t = 0; t < count; t += S) {
      step(std::integral_constant<int, 0>{}, t);
      if ((S == 2 && B > 64) || t + 1 < count) step(std::integral_constant<int, 1>{}, t + 1);  // B > 64: count is even
      if constexpr (S > 2)
        if (t + 2 < count) step(std::integral_constant<int, 2>{}, t + 2);
      if constexpr (S > 3)
        if (t + 3 < count) step(std::integral_constant<int, 3>{}, t + 3);
    }
    stage_barrier<0>();  // LDS is free for sums and strips
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
    // Epilogue, 32 rows at a time, on the registers as the products leave them:
    // lane (h, c) holds rows 8 g + 4 h + 0..3 of column c of a block.  Results go
    // through the wave's own strip of LDS, column by column in fp16, and out in
    // both orders: runs of 8 rows as they lie, runs of 8 columns by transposing
    // reads.
    constexpr int LDR = 40, LDF = WN + 2;  // a column of a strip, a row of the last step's fp32 strip
    constexpr int STRIP = (32 * LDF * 4 > PARTS * WN * LDR * 2 ? 32 * LDF * 4 : PARTS * WN * LDR * 2) / 2;
    constexpr int PER = WAVES / (S >= 4 ? 4 : 2);  // strips a stage
    static_assert(PER * STRIP <= STAGE, "the waves' strips fit their stages");
    _Float16* strip = ring(wave / PER) + wave % PER * STRIP;
    if (!EARLY) fetch(0, 0);
    __syncthreads();
    const float to_stored = a.scale * a.store;  // powers of two
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      if (row0 + mi * 32 >= a.mp) break;
      if (mi + 1 < MI) fetch(mi + 1, (mi + 1) & 1);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        if (col0 + ni * 32 >= cols_c) continue;
        const bool on_diagonal = SYM && row0 + mi * 32 == col0 + ni * 32;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float sum = acc[mi][ni][4 * g + r];
            if constexpr (K == kGram) {
              v[r] = sum * to_stored;
            } else if constexpr (K == kSquare) {
              const float e = (float)e_in[mi & 1][0][ni][g][r] + (SPLIT ? (float)e_in[mi & 1][PARTS - 1][ni][g][r] : 0.0f);
              const float d = fmaf(a.cc, d_in[mi & 1][g][r] + d_col[ni], a.cb) * (a.load * a.store);
              v[r] = fmaf(d, e, sum * (a.cc * to_stored));
            } else {
              v[r] = fmaf((a.ca + d_in[mi & 1][g][r]) * (a.load * a.store), x_in[mi & 1][ni][g][r], sum * to_stored);
            }
          }
          if (on_diagonal && c32 / 8 == g && c32 / 4 % 2 == h) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (c32 % 4 != r) continue;
              const float sum = acc[mi][ni][4 * g + r] * a.scale;
              const int64_t at = (int64_t)batch * a.mp + row0 + mi * 32 + c32;
              if constexpr (K == kGram) {
                a.diag_a[at] = sum;
              } else if constexpr (K == kSquare) {
                const float d = d_in[mi & 1][g][r];
                a.diag_p[at] = fmaf(a.cc, fmaf(d, d, sum), a.cb * d);
              }
              v[r] = 0.0f;
            }
          }
          if constexpr (K == kLast) {
#pragma unroll
            for (int r = 0; r < 4; ++r) ((float*)strip)[(8 * g + 4 * h + r) * LDF + ni * 32 + c32] = v[r];
          } else {
            if (K == kUpdate) xf[((mi * NI + ni) * 4 + g) * kWave] = v;
            h4 p, q;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              _Float16 x1, x2;
              split_half(v[r], x1, x2);
              p[r] = x1;
              q[r] = x2;
            }
            _Float16* to = strip + (ni * 32 + c32) * LDR + 8 * g + 4 * h;
            *(h4*)to = p;
            if (SPLIT) *(h4*)(to + WN * LDR) = q;
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      constexpr int ITS = WN / 16;  // vectors of 8 a lane
      if constexpr (K == kLast) {
        const int64_t plane_o = (int64_t)batch * a.rows * a.cols;
        const float* rows = (const float*)strip;
        Vec<TW, 8> old[ITS];
        int at_r[ITS], at_c[ITS], in[ITS];
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const int i = it * kWave + lane;
          const int r = a.tall ? i % 4 * 8 : i / (WN / 8), c = a.tall ? i / 4 : i % (WN / 8) * 8;
          at_r[it] = a.tall ? col0 + c : row0 + mi * 32 + r;
          at_c[it] = a.tall ? row0 + mi * 32 + r : col0 + c;
          in[it] = r * LDF + c;
          if (MUON && at_r[it] < a.rows && at_c[it] + 8 <= a.cols)
            old[it] = load_vec<TW, 8>((const TW*)a.out + plane_o + (int64_t)at_r[it] * a.cols + at_c[it]);
        }
        const int stride_v = a.tall ? LDF : 1;
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = rows[in[it] + e * stride_v];
          put_result<TW, MUON>(a, plane_o, at_r[it], at_c[it], v, old[it]);
        }
      } else {
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const int i = it * kWave + lane, c = i / 4, r = i % 4 * 8;
          if (col0 + c >= cols_c) continue;
          _Float16* to = by_col + place_of<SPLIT>(col0 + c, row0 + mi * 32 + r, a.mp);
          *(h8*)to = *(const h8*)(strip + c * LDR + r);
          if (SPLIT) *(h8*)(to + kSplitCols) = *(const h8*)(strip + (WN + c) * LDR + r);
        }
        if (!SYM || tm != tn) {  // a tile on the diagonal is its own transpose
          // 16 lanes transpose 16 rows x 4 columns: lane s reads rows 4 (s % 4).. of
          // column s / 4 and gets row s
          const int s = lane & 15;
#pragma unroll
          for (int it = 0; it < ITS; ++it) {
            const int group = it * 4 + lane / 16, c = group % (WN / 8) * 8, r = group / (WN / 8) * 16;
            _Float16* from = strip + (c + s / 4) * LDR + r + s % 4 * 4;
            const h8 p = columns8(from, from + 4 * LDR);
            h8 q;
            if (SPLIT) q = columns8(from + WN * LDR, from + (WN + 4) * LDR);
            if (col0 + c >= cols_c) continue;
            _Float16* to = by_row + place_of<SPLIT>(row0 + mi * 32 + r + s, col0 + c, cols_c);
            *(h8*)to = p;
            if (SPLIT) *(h8*)(to + kSplitCols) = q;
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if (G::SHARE) __syncthreads();  // the next tile's stages overwrite the strips
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
  int share;     // stages of a workgroup in the gram, where tiles are shared
  int arrive;    // counters to clear
  bool split, small, lds;
  size_t part, diag_a, diag_p, x, t[2], xf, e, p, sums, arrived, total;  // byte offsets
};

typedef Shape<64, 2, 2, 64, 4> Tile64;
typedef Shape<64, 2, 2, 128, 4> Tile64Deep;
typedef Shape<64, 2, 2, 128, 4, true> Tile64Shared;
typedef Shape<128, 2, 2, 64, 2> Tile128;
typedef Shape<128, 2, 2, 64, 4> Tile128Deep;
typedef Shape<192, 2, 2, 64, 2> Tile192;
typedef Shape<256, 2, 4, 64, 2> Tile256;
enum { k64, k64Deep, k128, k128Deep, k192, k256, k64Shared, kShapes };
constexpr int kTile[kShapes] = {64, 64, 128, 128, 192, 256, 64};
constexpr int kWaveRows[] = {Tile64::WM, Tile64Deep::WM, Tile128::WM, Tile128Deep::WM, Tile192::WM, Tile256::WM};
constexpr int kWaveCols[] = {Tile64::WN, Tile64Deep::WN, Tile128::WN, Tile128Deep::WN, Tile192::WN, Tile256::WN};

// The shape of a product is the one with the least time by this model, fitted
// to products of 128 to 8,192 a side: `fixed` us for the first stages' way and
// the epilogue, and a time for 64 summation indices (for 32 with their low
// parts in split products).  Shapes of which two workgroups fit a compute unit
// take longer a stage where they do; then the last of several rounds costs a
// third of a round more than its share, else a whole round.
struct ShapeTime {
  int slots;  // workgroups that fit at once
  struct {
    float fixed, alone, full;  // us, and us a stage: one workgroup a compute unit, all slots taken
  } whole, split;
};
constexpr ShapeTime kTime[kShapes] = {
    {512, {4.0f, 0.36f, 0.5f}, {4.5f, 0.29f, 0.5f}},     // 64
    {256, {4.8f, 0.24f, 0.24f}, {4.8f, 0.22f, 0.22f}},   // 64 deep
    {512, {6.8f, 0.61f, 0.8f}, {11.0f, 0.76f, 1.15f}},   // 128
    {256, {6.0f, 0.48f, 0.48f}, {11.0f, 0.54f, 0.54f}},  // 128 deep
    {256, {11.0f, 0.95f, 0.95f}, {18.0f, 1.2f, 1.2f}},   // 192
    {256, {10.0f, 1.5f, 1.5f}, {17.0f, 2.0f, 2.0f}},     // 256
    {256, {10.0f, 0.24f, 0.24f}, {10.0f, 0.22f, 0.22f}},  // 64 shared
};

static int64_t tiles_of(const NsPlan& p, int64_t batch, int shape, bool symmetric) {
  const int64_t tm = (p.mp + kTile[shape] - 1) / kTile[shape], tn = (p.np + kTile[shape] - 1) / kTile[shape];
  return batch * (symmetric ? tm * (tm + 1) / 2 : tm * tn);
}

// Stages (of 128) a workgroup takes where tiles are shared: as many workgroups as
// make about four a tile, runs of four stages or more.  With one, two, four, eight
// and sixteen a tile the gram lets 256 x 4,096 in bf16 take 169, 146, 132, 135 and
// 135 us, 512 x 8,192 289, 235, 214, 241 and 241, two of 256 x 4,096 in fp32 263,
// 212, 187, 190 and 223, 129 x 2,029 171, 153, 142, 147 and 147, and 200 x 8,000
// 401, 281, 229, 208 and 219.  Runs of two or eight stages and more change nothing.
static int64_t pick_share(int64_t tiles, int64_t nt) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(256, std::min(tiles * 4, tiles * nt / 4)));
  return (tiles * nt + most - 1) / most;
}

static int pick_shape(const NsPlan& p, int64_t batch, int64_t k, Product product) {
  const bool symmetric = product == kGram || product == kSquare;
  const int64_t nt = k * (p.split ? 2 : 1) / 64;
  int best = k64;
  double least = 1e30;
  for (int i = 0; i < kShapes; ++i) {
    if (i == k64Shared && product != kGram) continue;  // a square's sums are too short
    const auto& t = p.split ? kTime[i].split : kTime[i].whole;
    const int slots = kTime[i].slots;
    int64_t work = tiles_of(p, batch, i, symmetric), stages = nt;
    if (i == k64Shared) {
      stages = 2 * pick_share(work, nt / 2);
      if (stages >= nt) continue;
      work = 1;  // one round
    }
    double us;
    if (work <= 256) us = t.fixed + stages * t.alone;
    else if (slots == 256) us = (t.fixed + stages * t.full) * ((work + 255) / 256);
    else us = t.fixed + stages * t.full * (work <= slots ? 1.0 : (double)work / slots + 0.35);
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
  p->lds = lds_holds(rows, cols, split);
  if (p->lds) {
    p->total = kWorkspaceHeader;
    return true;
  }
  auto up = [](int64_t v, int64_t to) { return (v + to - 1) / to * to; };
  // tiles may hang over, but shapes above 64 take stages in pairs
  p->mp = (int)up(p->m, 128);
  p->np = (int)up(p->n, 128);
  p->shape[0] = pick_shape(*p, batch, p->np, kGram);
  p->shape[1] = pick_shape(*p, batch, p->mp, kSquare);
  p->shape[2] = pick_shape(*p, batch, p->mp, kUpdate);
  p->blocks = norm_blocks(batch, rows * cols);
  const int64_t xs = batch * p->mp * p->np, as = batch * p->mp * p->mp;
  size_t at = kWorkspaceHeader;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += (size_t)up(bytes, 256);
    return here;
  };
  p->part = take(batch * p->blocks * 8);
  p->diag_a = take(batch * p->mp * 4);
  p->diag_p = take(batch * p->mp * 4);
  p->x = take(xs * (split ? 4 : 2));
  p->xf = take(tiles_of(*p, batch, p->shape[2], false) * kTile[p->shape[2]] * kTile[p->shape[2]] * 4);
  for (size_t& t : p->t) t = take(xs * (split ? 4 : 2));
  p->e = take(as * (split ? 4 : 2));
  p->p = take(as * (split ? 4 : 2));
  int64_t runs = 0;
  p->arrive = 0;
  if (p->shape[0] == k64Shared) {
    const int64_t tiles = tiles_of(*p, batch, k64Shared, true), nt = (int64_t)p->np * (split ? 2 : 1) / Tile64Shared::BK;
    p->share = (int)pick_share(tiles, nt);
    p->arrive = (int)tiles;
    runs = (tiles * nt + p->share - 1) / p->share;
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
  a.stages = a.stride / G::BK;
  a.tiles = K == kGram || K == kSquare ? tm * (tm + 1) / 2 : tm * a.tiles_n;
  int64_t blocks = a.tiles * batch;
  if (G::SHARE) {
    a.units = (int)(blocks * a.stages);
    a.share = p.share;
    blocks = (a.units + a.share - 1) / a.share;
  }
  hipLaunchKernelGGL((k_ns_product<K, SPLIT, TW, MUON, G>), dim3((unsigned)blocks), dim3(G::WAVES * kWave), 0,
                     stream, a);
}

template <Product K, bool SPLIT, class TW, bool MUON>
static void launch_product(const NsPlan& p, const ProductArgs& a, int64_t batch, hipStream_t stream) {
  switch (p.shape[K == kGram ? 0 : K == kSquare ? 1 : 2]) {
    case k64Deep: return launch_tiles<K, SPLIT, TW, MUON, Tile64Deep>(p, a, batch, stream);
    case k128: return launch_tiles<K, SPLIT, TW, MUON, Tile128>(p, a, batch, stream);
    case k128Deep: return launch_tiles<K, SPLIT, TW, MUON, Tile128Deep>(p, a, batch, stream);
    case k192: return launch_tiles<K, SPLIT, TW, MUON, Tile192>(p, a, batch, stream);
    case k256: return launch_tiles<K, SPLIT, TW, MUON, Tile256>(p, a, batch, stream);
    case k64Shared:
      if constexpr (K == kGram) launch_tiles<K, SPLIT, TW, MUON, Tile64Shared>(p, a, batch, stream);
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
  a.xf = (float*)(ws + p.xf);
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
    g.scale = 1.0f / (sx * sx);
    g.store = sa;
    launch_product<kGram, SPLIT, float, false>(p, g, q.batch, stream);
    g = a;
    g.l = g.r = a.e;
    g.l_batch = g.r_batch = a_size;
    g.stride = p.mp * PARTS;
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
    g.scale = 1.0f / (sp * sx);
    g.load = 1.0f / sx;
    g.store = s.x[t + 1];
    if (t + 1 < q.steps) launch_product<kUpdate, SPLIT, float, false>(p, g, q.batch, stream);
    else launch_product<kLast, SPLIT, TW, MUON>(p, g, q.batch, stream);
  }
}

template <bool MUON>
static tgs_status ns_run(const NsCall& q, const NsPlan& p, const StepScales& s, void* workspace, hipStream_t stream) {
  if (p.small || p.lds) {
    if (p.small) small_run(q, s, workspace, stream);
    else lds_run(q, s, stream);
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
  k.xf = (float*)(ws + p.xf);
  k.tile = kTile[p.shape[2]];
  k.tile_rows = kWaveRows[p.shape[2]];
  k.tile_cols = kWaveCols[p.shape[2]];
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
    run_steps<kSplitProducts<T>, T, MUON>(q, p, s, ws, stream);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TGS_EHIP, "%s: launch failed: %s", q.what, hipGetErrorString(e));
  return TGS_OK;
}

// The checks both entries share; on TGS_OK the plan and scales are set.
static tgs_status ns_check(const NsCall& q, NsPlan* p, StepScales* s, const void* workspace, size_t workspace_bytes) {
  if (!is_float_dtype(q.x_dtype) || !is_float_dtype(q.out_dtype))
    return fail(TGS_EINVAL, "%s: values must be fp32, bf16 or fp16", q.what);
  if (!ns_plan(q.batch, q.rows, q.cols, split_products(q.out_dtype), p))
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
  return is_float_dtype(dtype) && ns_plan(batch, rows, cols, split_products(dtype), &p) ? p.total : 0;
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
