// Element types of the language-model training operators: conversions between
// the stored types (fp32, bf16, fp16) and the fp32 that every operator
// computes in, and loads and stores of short vectors of them.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>

#include "tgs.h"
#include "tgs_internal.h"

namespace tgs {

struct bf16_t {
  u16 b;
};
typedef _Float16 fp16_t;

inline size_t dtype_bytes(tgs_dtype t) {
  switch (t) {
    case TGS_FP32: case TGS_INT32: return 4;
    case TGS_BF16: case TGS_FP16: return 2;
    case TGS_INT64: return 8;
    default: return 0;
  }
}
inline bool is_float_dtype(tgs_dtype t) { return t == TGS_FP32 || t == TGS_BF16 || t == TGS_FP16; }
inline bool is_token_dtype(tgs_dtype t) { return t == TGS_INT32 || t == TGS_INT64; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16_t x) { return __uint_as_float((u32)x.b << 16); }
__device__ __forceinline__ float to_f32(fp16_t x) { return (float)x; }

// Rounds to nearest even; a NaN stays a (quiet) NaN.
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float x) {
  const u32 u = __float_as_uint(x);
  const u32 r = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
  return bf16_t{(u16)((u & 0x7FFFFFFFu) > 0x7F800000u ? ((u >> 16) | 0x40u) : r)};
}
template <>
__device__ __forceinline__ fp16_t from_f32<fp16_t>(float x) { return (fp16_t)x; }

// E consecutive elements at any element-aligned address: one load or store of
// up to 16 bytes (global accesses need no more than the element's alignment).
template <class T, int E>
struct __attribute__((packed, aligned(sizeof(T)))) Vec {
  T v[E];
};

template <class T, int E>
__device__ __forceinline__ Vec<T, E> load_vec(const T* p) { return *(const Vec<T, E>*)p; }

template <class T, int E>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, E>& x) { *(Vec<T, E>*)p = x; }

// The same store with the non-temporal hint, for arrays larger than the caches.
template <class T, int E>
struct VecWords {
  typedef u32 type __attribute__((ext_vector_type(sizeof(T) * E / 4), aligned(sizeof(T))));
};

template <class T, int E>
__device__ __forceinline__ void store_vec_streaming(T* p, const Vec<T, E>& x) {
  if constexpr (sizeof(T) * E >= 8) {
    typename VecWords<T, E>::type w;
    __builtin_memcpy(&w, &x, sizeof(x));
    __builtin_nontemporal_store(w, (typename VecWords<T, E>::type*)p);
  } else {
    store_vec<T, E>(p, x);
  }
}

// Calls f with a null pointer of the element type for a dtype code.
template <class F>
inline void with_float_dtype(tgs_dtype t, F&& f) {
  if (t == TGS_FP32) f((float*)nullptr);
  else if (t == TGS_BF16) f((bf16_t*)nullptr);
  else f((fp16_t*)nullptr);
}

}  // namespace tgs
