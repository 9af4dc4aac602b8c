// What the two routes of the Newton-Schulz operators share: the host's plan of
// a call, the scales of its steps, and the small route's entry.
#pragma once

#include <algorithm>
#include <type_traits>

#include "tgs_host.h"
#include "tgs_types.h"

namespace tgs {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));

constexpr int kMaxSteps = 64;

// Operands are high + low fp16 parts and a product is three where the result is
// fp32 or fp16, whose roundings (2^-24, 2^-11) a single fp16 operand's would pass.
inline bool split_products(tgs_dtype t) { return t != TGS_BF16; }
template <class T>
constexpr bool kSplitProducts = !std::is_same<T, bf16_t>::value;

// Powers of two that X (before each step, 1 after the last), A and P are held at.
struct StepScales {
  float x[kMaxSteps + 1], a[kMaxSteps], p[kMaxSteps];
};

struct NsCall {
  const char* what;
  const void* x;  // matrix, or gradient of a Muon step
  tgs_dtype x_dtype;
  float* momentum;  // null: x itself is orthogonalised
  void* out;        // result, or the weights that are updated
  tgs_dtype out_dtype;
  int64_t batch, rows, cols;
  float beta;
  int nesterov;
  float keep, gain;  // w = keep * w + gain * O
  int steps;
  double a, b, c, eps;
};

// v = high + low fp16 part.
__device__ __forceinline__ void split_half(float v, _Float16& h, _Float16& l) {
  h = (_Float16)v;
  l = (_Float16)(v - (float)h);
}

// Eight columns of this lane's row by two transposing LDS reads of four: of 16
// lanes, lane s addresses rows 4 (s % 4).. of column s / 4 and gets row s.
__device__ __forceinline__ h8 columns8(const _Float16* first, const _Float16* second) {
  typedef __attribute__((address_space(3))) s4* Lds;
  union {
    s4 s[2];
    h8 h;
  } u;
  u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)first);
  u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)second);
  return u.h;
}

// The new momentum, and the value that is orthogonalised.
__device__ __forceinline__ float new_momentum(float beta, float m, float g) { return fmaf(beta, m, g); }
__device__ __forceinline__ float muon_u(int nesterov, float beta, float g, float m) {
  return nesterov ? fmaf(beta, m, g) : m;
}

// Partial sums of squares a matrix: 4,096 entries each, at most 1,024 and about
// 2,048 for all matrices of a stack.  2,048 to 16,384 entries, and at most 256 to
// 2,048, change a call by 2% at most (4,096 square 1,574 to 1,580 us, eight of 1,024
// 396 to 405).
inline int norm_blocks(int64_t batch, int64_t count) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(1024, 2048 / batch));
  return (int)std::min(most, (count + 4095) / 4096);
}

// Sums of squares of what is orthogonalised (and the momentum's update): one
// partial sum a workgroup at part[batch][blocks].
void launch_norm(const NsCall& q, double* part, int blocks, hipStream_t stream);

// The route for matrices whose shorter side is at most kSmallSide.
constexpr int kSmallSide = 64;
size_t small_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);
void small_run(const NsCall& q, const StepScales& s, void* workspace, hipStream_t stream);


// The route for matrices that one workgroup holds in LDS.
bool lds_holds(int64_t rows, int64_t cols, bool split);
void lds_run(const NsCall& q, const StepScales& s, hipStream_t stream);

}  // namespace tgs
