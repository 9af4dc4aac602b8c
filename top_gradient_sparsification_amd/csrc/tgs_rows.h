// What the operators over rows (layer norm, the losses on logits) share:
// reductions over part of a wave, a wave or a workgroup, and short vectors of
// a row whose last one may hang over its end.
#pragma once

#include "tgs_host.h"
#include "tgs_types.h"

namespace tgs {

// A launch of 2^32 threads or more is refused by the runtime: longer calls take several.
inline int64_t most_groups(int threads) { return (int64_t)(0xFFFFFFFFull / (unsigned)threads); }

inline size_t round_up_256(size_t x) { return (x + 255) & ~(size_t)255; }

// Results above this size are stored past the caches.
constexpr size_t kRowsStreamingBytes = (size_t)64 << 20;

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f32(float identity, float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(identity), __float_as_int(x), CTRL, ROWS, 0xf, false));
}

struct Sum {
  static constexpr float kIdentity = 0.0f;
  static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
// The larger; of a number and a NaN the number.
struct Max {
  static constexpr float kIdentity = -__builtin_huge_valf();
  static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

// Reduces over groups of L neighbouring lanes, every lane of a group gets the
// same bits.  All lanes of the wave take part.
template <class Op, int L>
__device__ __forceinline__ float lanes_reduce(float x) {
  static_assert(L == 8 || L == 16 || L == 64, "");
  x = Op::of(x, dpp_f32<0xB1, 0xf>(x, x));   // quad_perm 1 0 3 2
  x = Op::of(x, dpp_f32<0x4E, 0xf>(x, x));   // quad_perm 2 3 0 1
  x = Op::of(x, dpp_f32<0x141, 0xf>(x, x));  // row_half_mirror
  if constexpr (L >= 16) x = Op::of(x, dpp_f32<0x140, 0xf>(x, x));  // row_mirror
  if constexpr (L == 64) {
    x = Op::of(x, dpp_f32<0x142, 0xa>(Op::kIdentity, x));  // row_bcast:15 -> rows 1, 3
    x = Op::of(x, dpp_f32<0x143, 0xc>(Op::kIdentity, x));  // row_bcast:31 -> rows 2, 3
    x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
  }
  return x;
}

// Reduces N values a thread over groups of L threads (a power of two; above 64
// the whole workgroup).  lds: N * L / 64 floats, not in use since the last
// barrier but one; calls in a row take alternating ones.
template <class Op, int L, int N>
__device__ __forceinline__ void group_reduce(float (&x)[N], float* lds) {
#pragma unroll
  for (int n = 0; n < N; ++n) x[n] = lanes_reduce<Op, (L < kWave ? L : kWave)>(x[n]);
  if constexpr (L > kWave) {
    constexpr int W = L / kWave;
    const int w = threadIdx.x / kWave;
    if (lane_id() == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) lds[n * W + w] = x[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      x[n] = lds[n * W];
#pragma unroll
      for (int i = 1; i < W; ++i) x[n] = Op::of(x[n], lds[n * W + i]);
    }
  }
}

// Elements c .. c + E - 1 of a row of n, `fill` past its end.
template <class T, int E>
__device__ __forceinline__ Vec<T, E> load_part(const T* row, u32 c, u32 n, T fill) {
  if (c + E <= n) return load_vec<T, E>(row + c);
  Vec<T, E> v;
#pragma unroll
  for (int e = 0; e < E; ++e) v.v[e] = c + e < n ? row[c + e] : fill;
  return v;
}

template <class T, int E>
__device__ __forceinline__ void store_part(T* row, u32 c, u32 n, const Vec<T, E>& v, bool streaming) {
  if (c + E <= n) {
    if (streaming) store_vec_streaming<T, E>(row + c, v);
    else store_vec<T, E>(row + c, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (c + e < n) row[c + e] = v.v[e];
}

// E values rounded to the type, to nearest even (bf16 by pairs, in one instruction).
template <class T, int E>
__device__ __forceinline__ Vec<T, E> round_vec(const float (&x)[E]) {
  Vec<T, E> v;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (std::is_same<T, bf16_t>::value) v.v[e].b = __builtin_bit_cast(u16, (__bf16)x[e]);
    else v.v[e] = from_f32<T>(x[e]);
  }
  return v;
}

// E parameters of a row from column c on, of a type known at run time (the same
// for the whole launch); `absent` where there are none.
template <int E>
__device__ __forceinline__ void load_params(const void* p, int dtype, u32 c, u32 n, float absent, float (&w)[E]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = absent;
  } else if (dtype == TGS_FP32) {
    const Vec<float, E> v = load_part<float, E>((const float*)p, c, n, 0.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = v.v[e];
  } else if (dtype == TGS_BF16) {
    const Vec<bf16_t, E> v = load_part<bf16_t, E>((const bf16_t*)p, c, n, bf16_t{0});
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = to_f32(v.v[e]);
  } else {
    const Vec<fp16_t, E> v = load_part<fp16_t, E>((const fp16_t*)p, c, n, (fp16_t)0.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = to_f32(v.v[e]);
  }
}

__device__ __forceinline__ void store_param(void* p, int dtype, u32 c, float x) {
  if (dtype == TGS_FP32) ((float*)p)[c] = x;
  else if (dtype == TGS_BF16) ((bf16_t*)p)[c] = from_f32<bf16_t>(x);
  else ((fp16_t*)p)[c] = from_f32<fp16_t>(x);
}

// Host: the checks that these operators' arrays have in common.
inline tgs_status check_rows_array(const char* what, const char* name, const void* p, size_t align, bool needed) {
  if (needed && !p) return fail(TGS_EINVAL, "%s: null %s", what, name);
  if (((uintptr_t)p & (align - 1)) != 0) return fail(TGS_EINVAL, "%s: %s not aligned to its type", what, name);
  return TGS_OK;
}

inline tgs_status check_rows_workspace(const char* what, const void* workspace, size_t bytes, size_t need) {
  if (!workspace) return fail(TGS_EINVAL, "%s: null workspace", what);
  if (((uintptr_t)workspace & 255u) != 0) return fail(TGS_EINVAL, "%s: workspace not 256-byte aligned", what);
  if (bytes < need) return fail(TGS_EWORKSPACE, "%s: workspace %zu bytes, need %zu", what, bytes, need);
  return TGS_OK;
}

inline tgs_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TGS_EHIP, "%s: launch failed: %s", what, hipGetErrorString(e));
  return TGS_OK;
}

}  // namespace tgs
