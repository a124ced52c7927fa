// gdr_ops.cuh -- what the scan, norm-and-rotation and paged attention kernels share:
// typed loads and stores of a few consecutive elements, and host-side checks.
#pragma once

#include <cuda_bf16.h>
#include <atomic>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "gdr_internal.cuh"

namespace gdr {
namespace ops {

typedef __nv_bfloat16 bf16;

// ------------------------------------------------------------------ device
// V consecutive elements as raw bits, the widest aligned access the count allows.
template <typename T, int V>
struct Raw {
  T v[V];
};
template <>
struct Raw<float, 2> {
  float2 v;
};
template <>
struct Raw<float, 4> {
  float4 v;
};
template <>
struct Raw<bf16, 2> {
  uint32_t v;
};
template <>
struct Raw<bf16, 4> {
  uint2 v;
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
  Raw<T, V> r;
  if constexpr (V == 1)
    r.v[0] = *p;
  else
    r.v = *reinterpret_cast<const decltype(r.v)*>(p);
  return r;
}
// The same, for data that is read once.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_once(const T* p) {
  Raw<T, V> r;
  if constexpr (V == 1)
    r.v[0] = __ldcs(p);
  else
    r.v = __ldcs(reinterpret_cast<const decltype(r.v)*>(p));
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, V>& r) {
  if constexpr (V == 1)
    *p = r.v[0];
  else
    *reinterpret_cast<std::remove_const_t<decltype(r.v)>*>(p) = r.v;
}

__device__ __forceinline__ float2 unpack2(uint32_t b) {
  return make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int V>
__device__ __forceinline__ void to_float(const Raw<T, V>& r, float* f) {
  if constexpr (V == 1) {
    f[0] = static_cast<float>(r.v[0]);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r.v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 p = unpack2(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  } else {
    const float* w = reinterpret_cast<const float*>(&r.v);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = w[i];
  }
}

// Two fp32 operations per instruction, on pairs of registers.
__device__ __forceinline__ unsigned long long bits2(float2 a) {
  return *reinterpret_cast<unsigned long long*>(&a);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<float2*>(&d);
}
// Four consecutive elements as two pairs.
__device__ __forceinline__ void load_pairs(const float* p, float2* f) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = make_float2(v.x, v.y);
  f[1] = make_float2(v.z, v.w);
}
__device__ __forceinline__ void to_pairs(const Raw<float, 4>& r, float2* f) {
  f[0] = make_float2(r.v.x, r.v.y);
  f[1] = make_float2(r.v.z, r.v.w);
}
__device__ __forceinline__ void to_pairs(const Raw<bf16, 4>& r, float2* f) {
  f[0] = unpack2(r.v.x);
  f[1] = unpack2(r.v.y);
}
__device__ __forceinline__ void store_pairs(float* p, const float2* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
}
__device__ __forceinline__ void store_pairs(bf16* p, const float2* f) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y));
}

template <typename T, int V>
__device__ __forceinline__ void load_f(const T* p, float* f) {
  to_float<T, V>(load_raw<T, V>(p), f);
}

template <typename T, int V>
__device__ __forceinline__ void store_f(T* p, const float* f) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2)
      *p = __float2bfloat16_rn(f[0]);
    else
      *p = f[0];
  } else {
    Raw<T, V> r;
    if constexpr (sizeof(T) == 2) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&r.v);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1]);
    } else {
      float* w = reinterpret_cast<float*>(&r.v);
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = f[i];
    }
    *reinterpret_cast<decltype(r.v)*>(p) = r.v;
  }
}

// ------------------------------------------------------------------ host
inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool is_dtype(int d) { return d == GDR_F32 || d == GDR_BF16; }
inline size_t dtype_size(int d) { return d == GDR_BF16 ? 2 : 4; }
// The status of a runtime call; leaves no error for a later one to report.
inline gdr_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return GDR_OK;
  (void)cudaGetLastError();
  return GDR_ERR_CUDA;
}

// A launch; its own status, not the error that an earlier call left behind.
template <typename Fn, typename... Args>
gdr_status launch_kernel(Fn fn, dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  return status_of(cudaLaunchKernelEx(&cfg, fn, args...));
}

// Lets `fn` use `bytes` of dynamic shared memory; asked of the runtime once per kernel (Tag
// names it) and device.
template <typename Tag, typename Fn>
bool allow_smem(Fn fn, int bytes) {
  static std::atomic<unsigned> done;             // a bit per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned bit = dev < 32 ? 1u << dev : 0u;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// A launch that may begin while the kernel before it in the stream still runs; the launched
// kernel waits for that one's results itself (griddepcontrol.wait, in every block).
template <typename Fn, typename... Args>
gdr_status launch_behind(Fn fn, dim3 grid, int threads, cudaStream_t s, Args... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return status_of(cudaLaunchKernelEx(&cfg, fn, args...));
}

// Calls f with a null pointer of the element type that `dtype` names.
template <typename F>
auto with_dtype(int dtype, F f) {
  return dtype == GDR_BF16 ? f(static_cast<bf16*>(nullptr)) : f(static_cast<float*>(nullptr));
}

// The sizes of a paged cache. Zero pages or table columns are an empty cache: its arrays may
// be null, as those of empty tensors are.
inline gdr_status check_cache(const gdr_paged_cache* c) {
  if (!c) return GDR_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->page_size <= 0 || c->HK <= 0 || c->D <= 0 || c->max_pages < 0 ||
      !is_dtype(c->dtype) || c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
    return GDR_ERR_INVALID_ARG;
  if (c->D > 256 || c->HK > (1 << 20)) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}
inline bool has_arrays(const gdr_paged_cache* c, const void* k, const void* v, const void* table) {
  return (c->num_pages == 0 || (k && v)) && (c->max_pages == 0 || table);
}

}  // namespace ops
}  // namespace gdr
