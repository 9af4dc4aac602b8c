// Newton-Schulz products of matrices whose shorter side is at most 64 (the
// formulas, and what is rounded, as in orthogonal.hip, but that with a shorter side
// of up to 32 every type takes the three products, and above the update takes X's
// low parts for every type).
//
// Such a step has little to compute: what costs is the launches and the
// barriers.  Here X stays in registers, in fp32.  A wave owns 16 CB columns of
// the padded MP x n matrix (MP = 32 or 64 rows) in both orders that the 16 x 16
// x 32 matrix instruction takes an operand in, rounded to fp16 parts as it does:
//   rows    lane = row of X, 8 columns      for the gram product X X^T
//   columns lane = column of X, 8 rows      for the update P X
// The instruction's result comes in the layout "lane = column, 4 rows", so its
// registers are, two blocks of 16 taken together, an operand again with its
// summation index in another order (slot (g, 4 b + r) holds index 16 b + 4 g +
// r; both operands use the same order).  P X with P as left operand gives the
// column order; the same registers with the operands exchanged give (P X)^T,
// the row order.  The update is computed both ways and X passes through LDS
// once, at the start, for the order that memory does not have.
//
// Per step: the waves' gram products are added through LDS (lower blocks
// only), E and D are made, the waves share the blocks of E^2, P is written to
// LDS, every wave updates its columns.
//
// Up to 512 columns of 64, or 1,024 of 32, one workgroup holds a whole matrix and
// one launch does everything, the norm and the momentum included.  Longer ones are
// cut into chunks of 256 columns, a workgroup each, and the sum over chunks is
// where a launch ends: norm, first gram, then one launch a step, in which every
// workgroup adds the chunks' gram products itself; X is kept in memory between
// them as the registers' dump.
#include <type_traits>

#include "tgs_orthogonal.h"

namespace tgs {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kSmWaves = 8;
constexpr int kSmThreads = kSmWaves * kWave;

enum SmallStage { kWhole, kFirst, kMiddle, kEnd };

struct SmallArgs {
  const void* x;
  float* momentum;
  void* out;
  const double* part;  // partial sums of squares (chunks > 1)
  f4* gram;            // [2][batch][chunks][lower blocks][64]
  f4* state;           // [batch][chunks][registers][threads]
  int64_t count;       // rows * cols
  tgs_dtype x_dtype, out_dtype;
  int rows, cols, n, tall, nesterov, steps, step, chunks, part_blocks;
  float beta, keep, gain, ca, cb, cc;
  double eps;
};

// Four consecutive elements, those past `left` as zero.
__device__ __forceinline__ f4 load4(const void* p, tgs_dtype t, int64_t at, int left) {
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (left <= 0) return v;
  auto get = [&](auto* q) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(q)>>;
    if (left >= 4) {
      const Vec<T, 4> y = load_vec<T, 4>(q + at);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = to_f32(y.v[r]);
    } else {
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < left) v[r] = to_f32(q[at + r]);
    }
  };
  if (t == TGS_FP32) get((const float*)p);
  else if (t == TGS_BF16) get((const bf16_t*)p);
  else get((const fp16_t*)p);
  return v;
}

__device__ __forceinline__ void store4(void* p, tgs_dtype t, int64_t at, int left, f4 v) {
  if (left <= 0) return;
  auto put = [&](auto* q) {
    using T = std::remove_pointer_t<decltype(q)>;
    if (left >= 4) {
      Vec<T, 4> y;
#pragma unroll
      for (int r = 0; r < 4; ++r) y.v[r] = from_f32<T>(v[r]);
      store_vec<T, 4>(q + at, y);
    } else {
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < left) q[at + r] = from_f32<T>(v[r]);
    }
  };
  if (t == TGS_FP32) put((float*)p);
  else if (t == TGS_BF16) put((bf16_t*)p);
  else put((fp16_t*)p);
}

__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Block pair (I, J), I >= J, of the t-th lower block, row by row.
__device__ __forceinline__ void lower_block(int t, int& I, int& J) {
  I = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
  J = t - I * (I + 1) / 2;
}

template <int RB, int CB, bool SPLIT, SmallStage STAGE>
__global__ __launch_bounds__(kSmThreads) void k_ns_small(SmallArgs a, StepScales sc) {
  constexpr int MP = 16 * RB, KB = RB / 2, CP = CB / 2, NBLK = RB * (RB + 1) / 2, LD = MP + 8;
  constexpr int ND = SPLIT ? 2 : 1;
  __shared__ __align__(16) f4 s_gram[kSmWaves][NBLK][kWave];
  __shared__ __align__(16) _Float16 s_e[ND][MP][LD], s_p[ND][MP][LD];
  __shared__ __align__(16) float s_d[MP], s_dp[MP];
  __shared__ double s_sum[kSmWaves];
  const int tid = threadIdx.x, lane = lane_id(), g = lane >> 4, l16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int chunk = blockIdx.x, batch = blockIdx.y;
  const int j0 = (chunk * kSmWaves + w) * 16 * CB;
  const int waves = min(kSmWaves, (a.n - chunk * kSmWaves * 16 * CB + 16 * CB - 1) / (16 * CB));  // with columns
  const int64_t base = (int64_t)batch * a.count;
  const f4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  // X, times the step's scale, block by block: this lane's column and four rows,
  // and its row and four columns
  f4 xc[RB][CB], xr[RB][CB];
  // the place of this lane's four values of block (rb, c) in memory order
  auto place = [&](int rb, int c, int64_t& at, int& left) {
    const int line = a.tall ? j0 + 16 * c + l16 : 16 * rb + l16;
    const int off = a.tall ? 16 * rb + 4 * g : j0 + 16 * c + 4 * g;
    at = base + (int64_t)line * a.cols + off;
    left = line < a.rows ? a.cols - off : 0;
  };

  f4* state = a.state + ((int64_t)batch * a.chunks + chunk) * (2 * RB * CB) * kSmThreads + tid;

  if constexpr (STAGE == kWhole || STAGE == kFirst) {
    f4 v[RB][CB];
    double sum = 0.0;
    if (w < waves) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          int64_t at;
          int left;
          place(rb, c, at, left);
          v[rb][c] = load4(a.x, a.x_dtype, at, left);
          if (a.momentum) {
            f4 m = load4(a.momentum, TGS_FP32, at, left);
            if (STAGE == kWhole) {
#pragma unroll
              for (int r = 0; r < 4; ++r) m[r] = new_momentum(a.beta, m[r], v[rb][c][r]);
              store4(a.momentum, TGS_FP32, at, left, m);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) v[rb][c][r] = muon_u(a.nesterov, a.beta, v[rb][c][r], m[r]);
          }
          if (STAGE == kWhole)
#pragma unroll
            for (int r = 0; r < 4; ++r) sum = fma((double)v[rb][c][r], (double)v[rb][c][r], sum);
        }
    } else {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int c = 0; c < CB; ++c) v[rb][c] = zero;
    }
    if (STAGE == kFirst)
      for (int i = lane; i < a.part_blocks; i += kWave) sum += a.part[(int64_t)batch * a.part_blocks + i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (STAGE == kWhole) {
      if (lane == 0) s_sum[w] = sum;
      __syncthreads();
      sum = 0.0;
      for (int i = 0; i < kSmWaves; ++i) sum += s_sum[i];
    }
    const double inv = 1.0 / (sqrt(sum) + a.eps);
    const float sx = sc.x[0];
    // the other order: block by block through the wave's own LDS, in lines of 20 so
    // that neither order's accesses meet in a bank
    constexpr int LINE = 20;
    static_assert(2 * 16 * LINE * sizeof(float) <= sizeof(s_gram[0]), "two blocks fit");
    float* turn = (float*)s_gram[w];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        f4 x, y;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = (float)((double)v[rb][c][r] * inv) * sx;
        float* block = turn + (rb * CB + c) % 2 * (16 * LINE);
        *(f4*)(block + l16 * LINE + 4 * g) = x;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = block[(4 * g + r) * LINE + l16];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        xc[rb][c] = a.tall ? x : y;
        xr[rb][c] = a.tall ? y : x;
      }
  } else {
    const f4* p = state;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        xc[rb][c] = *p, p += kSmThreads;
        xr[rb][c] = *p, p += kSmThreads;
      }
  }

  // An operand of two neighbouring blocks: high parts, low parts.
  auto operand = [&](f4 first, f4 second, h8& high, h8& low) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      _Float16 h, l;
      split_half(e < 4 ? first[e] : second[e - 4], h, l);
      high[e] = h;
      low[e] = l;
    }
  };

  // The sums of X X^T's lower blocks over this workgroup's columns; `take` gets
  // four rows of one column each.
  auto gram = [&](auto&& take) {
    f4 acc[NBLK];
#pragma unroll
    for (int t = 0; t < NBLK; ++t) acc[t] = zero;
    if (w < waves) {
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        h8 rh[RB], rl[RB];
#pragma unroll
        for (int I = 0; I < RB; ++I) {
          operand(xr[I][2 * c], xr[I][2 * c + 1], rh[I], rl[I]);
#pragma unroll
          for (int J = 0; J <= I; ++J) {
            f4& q = acc[I * (I + 1) / 2 + J];
            if (SPLIT) q = mfma(rl[I], rh[J], mfma(rh[I], rl[J], q));
            q = mfma(rh[I], rh[J], q);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NBLK; ++t) s_gram[w][t][lane] = acc[t];
    }
    __syncthreads();
    for (int u = tid; u < NBLK * kWave; u += kSmThreads) {
      f4 q = s_gram[0][u / kWave][u % kWave];
      for (int i = 1; i < waves; ++i) q += s_gram[i][u / kWave][u % kWave];
      take(u, q);
    }
  };
  // From a sum: E (both triangles) and D to LDS.
  auto put_e = [&](int u, f4 q, float to_a, float sa) {
    int I, J;
    lower_block(u / kWave, I, J);
    const int ug = (u % kWave) >> 4, i0 = 16 * I + 4 * ug, j = 16 * J + (u & 15);
    h4 h, l;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float t = q[r] * to_a;
      if (i0 + r == j) s_d[j] = t;
      _Float16 x, y;
      split_half(i0 + r == j ? 0.0f : t * sa, x, y);
      h[r] = x;
      l[r] = y;
      if (I != J) {
        s_e[0][i0 + r][j] = x;
        if (SPLIT) s_e[ND - 1][i0 + r][j] = y;
      }
    }
    *(h4*)&s_e[0][j][i0] = h;
    if (SPLIT) *(h4*)&s_e[ND - 1][j][i0] = l;
  };
  // P from E and D, its blocks dealt to the waves.
  auto square = [&](float sa, float sp) {
    const float to_sq = 1.0f / (sa * sa), to_e = 1.0f / sa;
    for (int t = w; t < RB * RB; t += kSmWaves) {
      const int I = t / RB, J = t % RB;
      f4 q = zero;
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const h8 xh = *(const h8*)&s_e[0][16 * I + l16][32 * k + 8 * g];
        const h8 yh = *(const h8*)&s_e[0][16 * J + l16][32 * k + 8 * g];
        if (SPLIT) {
          const h8 xl = *(const h8*)&s_e[ND - 1][16 * I + l16][32 * k + 8 * g];
          const h8 yl = *(const h8*)&s_e[ND - 1][16 * J + l16][32 * k + 8 * g];
          q = mfma(xl, yh, mfma(xh, yl, q));
        }
        q = mfma(xh, yh, q);
      }
      const int i0 = 16 * I + 4 * g, j = 16 * J + l16;
      const h4 eh = *(const h4*)&s_e[0][j][i0], el = *(const h4*)&s_e[ND - 1][j][i0];
      const f4 di = *(const f4*)&s_d[i0];
      const float dj = s_d[j];
      h4 h, l;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = ((float)eh[r] + (SPLIT ? (float)el[r] : 0.0f)) * to_e, sq = q[r] * to_sq;
        if (i0 + r == j) s_dp[j] = fmaf(a.cc, fmaf(dj, dj, sq), a.cb * dj);
        const float p = fmaf(a.cc, sq, fmaf(a.cc, di[r] + dj, a.cb) * e);
        _Float16 x, y;
        split_half(i0 + r == j ? 0.0f : p * sp, x, y);
        h[r] = x;
        l[r] = y;
      }
      *(h4*)&s_p[0][j][i0] = h;
      if (SPLIT) *(h4*)&s_p[ND - 1][j][i0] = l;
    }
  };
  // P's operand for row block rb, slot (g, 4 b + r) = column 32 k + 16 b + 4 g + r.
  auto p_operand = [&](int d, int rb, int k) {
    const h4 x = *(const h4*)&s_p[d][16 * rb + l16][32 * k + 4 * g];
    const h4 y = *(const h4*)&s_p[d][16 * rb + l16][32 * k + 16 + 4 * g];
    return (h8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };
  // X <- (a + D_P) X + E_P X in both orders, or the result in memory's order.  X's
  // low parts are multiplied for bf16 results too: what its rounding puts into
  // directions in which a matrix of low rank is empty grows by the first coefficient
  // a step, and the more the smaller the matrix (64 x 64 of rank 8: 3.0e-3 off, with
  // them 7e-4).  64 x 512 takes 46 us with them, 39 without, 63 with all three
  // products; 64 x 64 takes 23, 20 and 27.
  auto update = [&](float sx, float sp, float next, auto last) {
    constexpr bool LAST = decltype(last)::value;
    const float to_x = next / sx, to_acc = next / (sp * sx);  // powers of two
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      f4 nc[RB], nr[RB];
      h8 ch[KB], cl[KB];
#pragma unroll
      for (int k = 0; k < KB; ++k) operand(xc[2 * k][c], xc[2 * k + 1][c], ch[k], cl[k]);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        f4 qc = zero, qr = zero;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          const h8 ph = p_operand(0, rb, k);
          h8 pl;
          if (SPLIT) pl = p_operand(ND - 1, rb, k);
          if (!LAST || a.tall) {
            if (SPLIT) qc = mfma(pl, ch[k], qc);
            qc = mfma(ph, ch[k], mfma(ph, cl[k], qc));
          }
          if (!LAST || !a.tall) {
            if (SPLIT) qr = mfma(ch[k], pl, qr);
            qr = mfma(ch[k], ph, mfma(cl[k], ph, qr));
          }
        }
        const f4 dc = *(const f4*)&s_dp[16 * rb + 4 * g];
        const float dr = s_dp[16 * rb + l16];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          nc[rb][r] = fmaf((a.ca + dc[r]) * to_x, xc[rb][c][r], qc[r] * to_acc);
          nr[rb][r] = fmaf((a.ca + dr) * to_x, xr[rb][c][r], qr[r] * to_acc);
        }
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        if constexpr (LAST) {
          int64_t at;
          int left;
          place(rb, c, at, left);
          f4 v = a.tall ? nc[rb] : nr[rb];
          if (a.momentum) {
            const f4 old = load4(a.out, a.out_dtype, at, left);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = fmaf(a.keep, old[r], a.gain * v[r]);
          }
          store4(a.out, a.out_dtype, at, left, v);
        } else {
xc[rb][c] = nc[rb];
          xr[rb][c] = nr[rb];
        }
      }
    }
  };
  // The chunks' sums lie in one of two buffers by the step's parity.
  auto chunk_sums = [&](int s) {
    return a.gram + ((int64_t)(s & 1) * gridDim.y + batch) * a.chunks * (NBLK * kWave);
  };
  auto save = [&]() {
    f4* p = state;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        *p = xc[rb][c], p += kSmThreads;
        *p = xr[rb][c], p += kSmThreads;
      }
  };

  if constexpr (STAGE == kWhole) {
    for (int s = 0; s < a.steps; ++s) {
      const float sx = sc.x[s], sa = sc.a[s], sp = sc.p[s], to_a = 1.0f / (sx * sx);
      gram([&](int u, f4 q) { put_e(u, q, to_a, sa); });
      __syncthreads();
      square(sa, sp);
      __syncthreads();
      if (s + 1 < a.steps) {
        if (w < waves) update(sx, sp, sc.x[s + 1], std::false_type{});
      } else {
        if (w < waves) update(sx, sp, 1.0f, std::true_type{});
      }
    }
  } else {
    if constexpr (STAGE != kFirst) {
      const float sx = sc.x[a.step], sa = sc.a[a.step], sp = sc.p[a.step], to_a = 1.0f / (sx * sx);
      const f4* sums = chunk_sums(a.step);
      for (int u = tid; u < NBLK * kWave; u += kSmThreads) {
        f4 q = zero;
#pragma unroll 8
        for (int i = 0; i < a.chunks; ++i) q += sums[(int64_t)i * (NBLK * kWave) + u];
        put_e(u, q, to_a, sa);
      }
      __syncthreads();
      square(sa, sp);
      __syncthreads();
      if (w < waves) update(sx, sp, STAGE == kEnd ? 1.0f : sc.x[a.step + 1], std::integral_constant<bool, STAGE == kEnd>{});
    }
    if constexpr (STAGE != kEnd) {
      f4* to = chunk_sums(STAGE == kFirst ? 0 : a.step + 1) + (int64_t)chunk * (NBLK * kWave);
      gram([&](int u, f4 q) { to[u] = q; });
      save();
    }
  }
}

// ------------------------------------------------------------------ host --
struct SmallPlan {
  int rb, cb, chunks, blocks;
  size_t part, gram, state, total;
};

// Columns a wave: the fewest with which one workgroup holds the matrix and one
// launch does (30 x 512 in bf16 21 us, 35 in chunks; 300 of 64 x 512 99 and 228;
// one of 64 x 512 in fp32 65 and 60 is the exception); else 32, the fewest there
// are, for any batch: with 64, 16 of 64 x 4,096 take 139 us instead of 108, 300
// of 64 x 2,048 966 instead of 895, 1,000 of 30 x 1,100 885 instead of 765, though
// 1,000 of 64 x 1,024 1,452 instead of 1,585.
static SmallPlan small_plan(int64_t batch, int64_t rows, int64_t cols) {
  SmallPlan p{};
  const int64_t m = std::min(rows, cols), n = std::max(rows, cols);
  p.rb = m <= 32 ? 2 : 4;
  const int most = p.rb == 2 ? 8 : 4;
  auto chunks = [&](int cb) { return (n + kSmWaves * 16 * cb - 1) / (kSmWaves * 16 * cb); };
  p.cb = 2;
  if (chunks(most) == 1)
    while (chunks(p.cb) > 1) p.cb *= 2;
  p.chunks = (int)chunks(p.cb);
  p.blocks = norm_blocks(batch, rows * cols);
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  size_t at = kWorkspaceHeader;
  p.part = at;
  p.gram = p.state = at;
  if (p.chunks > 1) {
    at += up((size_t)batch * p.blocks * 8);
    p.gram = at;
    at += up((size_t)2 * batch * p.chunks * (p.rb * (p.rb + 1) / 2) * kWave * sizeof(f4));
    p.state = at;
    at += up((size_t)batch * p.chunks * (2 * p.rb * p.cb) * kSmThreads * sizeof(f4));
  }
  p.total = at;
  return p;
}

size_t small_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) { return small_plan(batch, rows, cols).total; }

template <int RB, int CB, bool SPLIT>
static void launch_small(const SmallPlan& p, SmallArgs a, const StepScales& s, int batch, hipStream_t stream) {
  const dim3 grid(p.chunks, batch), block(kSmThreads);
  if (p.chunks == 1) {
    hipLaunchKernelGGL((k_ns_small<RB, CB, SPLIT, kWhole>), grid, block, 0, stream, a, s);
    return;
  }
  if constexpr (CB == 2) {  // chunks are of 32 columns a wave
    hipLaunchKernelGGL((k_ns_small<RB, CB, SPLIT, kFirst>), grid, block, 0, stream, a, s);
    for (a.step = 0; a.step + 1 < a.steps; ++a.step)
      hipLaunchKernelGGL((k_ns_small<RB, CB, SPLIT, kMiddle>), grid, block, 0, stream, a, s);
    hipLaunchKernelGGL((k_ns_small<RB, CB, SPLIT, kEnd>), grid, block, 0, stream, a, s);
  }
}

template <bool SPLIT>
static void launch_small_any(const SmallPlan& p, const SmallArgs& a, const StepScales& s, int batch, hipStream_t stream) {
  if (p.rb == 2) {
    // three products for bf16 results too: single ones, even with X's low parts in the
    // update, leave up to 3.7e-3 of matrices so small, twice the result's rounding (30 x
    // 1,024 takes 42 us instead of 36, 32 x 32 11.9 instead of 10.5)
    if (p.cb == 2) launch_small<2, 2, true>(p, a, s, batch, stream);
    else if (p.cb == 4) launch_small<2, 4, true>(p, a, s, batch, stream);
    else launch_small<2, 8, true>(p, a, s, batch, stream);
  } else {
    if (p.cb == 2) launch_small<4, 2, SPLIT>(p, a, s, batch, stream);
    else launch_small<4, 4, SPLIT>(p, a, s, batch, stream);
  }
}

void small_run(const NsCall& q, const StepScales& s, void* workspace, hipStream_t stream) {
  const SmallPlan p = small_plan(q.batch, q.rows, q.cols);
  char* ws = (char*)workspace;
  SmallArgs a{};
  a.x = q.x;
  a.momentum = q.momentum;
  a.out = q.out;
  a.part = (const double*)(ws + p.part);
  a.gram = (f4*)(ws + p.gram);
  a.state = (f4*)(ws + p.state);
  a.count = q.rows * q.cols;
  a.x_dtype = q.x_dtype;
  a.out_dtype = q.out_dtype;
  a.rows = (int)q.rows;
  a.cols = (int)q.cols;
  a.n = (int)std::max(q.rows, q.cols);
  a.tall = q.rows > q.cols;
  a.nesterov = q.nesterov;
  a.steps = q.steps;
  a.chunks = p.chunks;
  a.part_blocks = p.blocks;
  a.beta = q.beta;
  a.keep = q.keep;
  a.gain = q.gain;
  a.ca = (float)q.a;
  a.cb = (float)q.b;
  a.cc = (float)q.c;
  a.eps = q.eps;
  if (p.chunks > 1) launch_norm(q, (double*)(ws + p.part), p.blocks, stream);
  if (split_products(q.out_dtype)) launch_small_any<true>(p, a, s, (int)q.batch, stream);
  else launch_small_any<false>(p, a, s, (int)q.batch, stream);
}

}  // namespace tgs
