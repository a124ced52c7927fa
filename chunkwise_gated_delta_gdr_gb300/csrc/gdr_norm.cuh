// gdr_norm.cuh -- what gdr_gated.cu and gdr_residual.cu share: rows of a norm held by a group of
// lanes or by a block, their copies ahead of time, sums over a row, gate activations, the weights'
// gradients, and the plan of a launch.
#pragma once

#include "gdr_ops.cuh"
#include "gdr_ptx.cuh"

namespace gdr {
namespace ops {
namespace {

// Every kernel here may be launched while the one before it in the stream still runs, and lets the
// next one be: begin_behind() is the point from which it touches memory (a decode step of
// 64 x 16 heads 4.1 -> 2.5 us a call, of 64 x 2048 channels 4.1 -> 3.3).

constexpr int kMaxThreads = 512;

// Who holds a row, and how. LANES > 0: that many lanes of a warp (8, 16 or 32), several rows
// per warp. LANES == 0: a whole block, whose size follows the row's. A thread holds NV runs of
// V consecutive elements; run c of thread i starts at element (c threads + i) V. V is 8 where
// sizes, strides and bases allow 16-byte accesses, else 1.
// SHIFT: rows of any length whose strides are the dense ones but for multiples of 8 elements, so
// that a row starts `phase` elements behind a 16-byte boundary in every tensor alike. Runs are
// laid along the boundaries, run 0 from element -phase on, and what a run has outside the row is
// masked. A thread's rows all have one phase: its weights' gradients stay in their places.
// (2 x 307 x 3190 with a gate, training step: 147 us element by element, 30 so.)
template <int LANES_, int V_, int NV_, bool SHIFT_ = false>
struct Shape {
  static constexpr int LANES = LANES_, V = V_, NV = NV_, N = V_ * NV_;
  static constexpr bool SHIFT = SHIFT_;
  // Elements that the groups of a block of 256 threads hold.
  static constexpr int kSums = LANES_ ? 256 * N : 1;
  // Copies ahead of time go through shared memory, 16 bytes at a time.
  static constexpr bool kAhead = V_ == 8 && NV_ <= 2;
  // Short rows element by element: the next row's elements are loaded into registers.
  static constexpr bool kRegs = V_ == 1 && NV_ <= 8;
  // Rows past 8192 elements, and long ones element by element, are loaded when they are needed,
  // kGroup runs at a time (3006 rows of 9000 with norm, gate and scale, all bf16, training step: 582
  // us run by run, 477 so).
  static constexpr bool kGroups = !kAhead && !kRegs;
  static constexpr int kGroup = V_ == 1 ? 8 : 2;
};

// V consecutive elements as raw words.
template <typename T, int V>
struct Run {
  uint32_t w[V * sizeof(T) / 4];
};
template <>
struct Run<bf16, 1> {
  bf16 v;
};

template <typename T, int V>
__device__ __forceinline__ void unpack(const Run<T, V>& r, float* f) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2)
      f[0] = __bfloat162float(r.v);
    else
      f[0] = __uint_as_float(r.w[0]);
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 p = unpack2(r.w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __uint_as_float(r.w[i]);
  }
}
// ONLY_READ: nothing writes this memory while the kernel runs, so the load may move before any
// store of it.
template <typename T, int V, bool ONLY_READ = false>
__device__ __forceinline__ void load_run(const T* p, float* f) {
  Run<T, V> r;
  if constexpr (V == 1 && sizeof(T) == 2) {
    r.v = ONLY_READ ? __ldg(p) : *p;
  } else if constexpr (V == 1) {
    r.w[0] = __float_as_uint(ONLY_READ ? __ldg(p) : *p);
  } else {
#pragma unroll
    for (int i = 0; i < V * (int)sizeof(T) / 16; ++i) {
      const uint4* q = reinterpret_cast<const uint4*>(p) + i;
      const uint4 u = ONLY_READ ? __ldg(q) : *q;
      r.w[4 * i] = u.x;
      r.w[4 * i + 1] = u.y;
      r.w[4 * i + 2] = u.z;
      r.w[4 * i + 3] = u.w;
    }
  }
  unpack<T, V>(r, f);
}
template <typename T, int V>
__device__ __forceinline__ void store_run(T* p, const float* f) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2)
      *p = __float2bfloat16_rn(f[0]);
    else
      *p = f[0];
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}
// One element as it lies in memory, and its value. Nothing here waits for the load: with the
// conversion beside it, in one of two branches, every load waited for the one before.
template <bool ONLY_READ>
__device__ __forceinline__ uint32_t load_raw(const void* p, int64_t i, int is_bf16) {
  if (is_bf16) {
    const unsigned short* q = static_cast<const unsigned short*>(p) + i;
    return ONLY_READ ? __ldg(q) : *q;
  }
  const uint32_t* q = static_cast<const uint32_t*>(p) + i;
  return ONLY_READ ? __ldg(q) : *q;
}
__device__ __forceinline__ float raw_value(uint32_t raw, int is_bf16) {
  return __uint_as_float(is_bf16 ? raw << 16 : raw);
}
// A run into memory whose type is known at run time only.
template <int V>
__device__ __forceinline__ void store_any(void* p, int64_t i, int is_bf16, const float* f) {
  if (is_bf16)
    store_run<bf16, V>(static_cast<bf16*>(p) + i, f);
  else
    store_run<float, V>(static_cast<float*>(p) + i, f);
}

// Operations on runs of V elements, in pairs where V is 8 (two fp32 operations per instruction).
template <int V, typename F2, typename F1>
__device__ __forceinline__ void over_run(F2 two, F1 one) {
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < V; i += 2) two(i);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) one(i);
  }
}
__device__ __forceinline__ float2 pair_at(const float* a, int i) { return make_float2(a[i], a[i + 1]); }
__device__ __forceinline__ void put_pair(float* d, int i, float2 v) { d[i] = v.x, d[i + 1] = v.y; }
template <int V>                                 // d = a b
__device__ __forceinline__ void mul_run(float* d, const float* a, const float* b) {
  over_run<V>([&](int i) { put_pair(d, i, mul2(pair_at(a, i), pair_at(b, i))); },
              [&](int i) { d[i] = a[i] * b[i]; });
}
template <int V>                                 // d = s a
__device__ __forceinline__ void scale_run(float* d, const float* a, float s) {
  over_run<V>([&](int i) { put_pair(d, i, mul2(pair_at(a, i), make_float2(s, s))); },
              [&](int i) { d[i] = a[i] * s; });
}
template <int V>                                 // d = a b + c
__device__ __forceinline__ void fma_run(float* d, const float* a, const float* b, const float* c) {
  over_run<V>([&](int i) { put_pair(d, i, fma2(pair_at(a, i), pair_at(b, i), pair_at(c, i))); },
              [&](int i) { d[i] = fmaf(a[i], b[i], c[i]); });
}
template <int V>                                 // d = s a + c
__device__ __forceinline__ void fma_run(float* d, const float* a, float s, const float* c) {
  over_run<V>([&](int i) { put_pair(d, i, fma2(pair_at(a, i), make_float2(s, s), pair_at(c, i))); },
              [&](int i) { d[i] = fmaf(a[i], s, c[i]); });
}
template <int V>                                 // sum of a b
__device__ __forceinline__ float dot_run(const float* a, const float* b) {
  float2 s = make_float2(0.f, 0.f);
  over_run<V>([&](int i) { s = fma2(pair_at(a, i), pair_at(b, i), s); },
              [&](int i) { s.x = fmaf(a[i], b[i], s.x); });
  return s.x + s.y;
}

// The gate a(z) = g zz and its slope g (zz (1 - g) + c): g = 1 / (1 + e^-z) or 1 without an
// activation, zz = z or, for the sigmoid, 1, and c = 1, 0 likewise. (Without an activation the
// slope is 1 outright: the formula would make NaN of an infinite z.)
enum Act { kNone = GDR_ACT_NONE, kSigmoid = GDR_ACT_SIGMOID, kSilu = GDR_ACT_SILU };
// By the approximate 2^x and reciprocal (2^-22 each, and the rounding of z log2(e), half an ulp
// of it); 0 for z < -88.
__device__ __forceinline__ float sigmoid(float z) {
  float e, g;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(1.f + e));
  return g;
}
template <int V>
__device__ __forceinline__ void gate_sigma(float* g, const float* z, int kind) {
#pragma unroll
  for (int e = 0; e < V; ++e) g[e] = kind == kNone ? 1.f : sigmoid(z[e]);
}
template <int V>
__device__ __forceinline__ void gate_open(float* a, const float* g, const float* z, int kind) {
  if (kind == kSigmoid) {
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] = g[e];
  } else {
    mul_run<V>(a, g, z);
  }
}
template <int V>                                 // s may be z
__device__ __forceinline__ void gate_slope(float* s, const float* g, const float* z, int kind) {
  over_run<V>(
      [&](int i) {
        const float2 gp = pair_at(g, i), one = make_float2(1.f, 1.f);
        const float2 h = fma2(gp, make_float2(-1.f, -1.f), one);
        const float2 zh = fma2(pair_at(z, i), h, one);
        put_pair(s, i, kind == kNone ? one : mul2(gp, kind == kSigmoid ? h : zh));
      },
      [&](int i) {
        const float h = 1.f - g[i];
        s[i] = kind == kNone ? 1.f : g[i] * (kind == kSigmoid ? h : fmaf(z[i], h, 1.f));
      });
}

// Sums of K values over a row's threads, known to all of them. A block's sums meet in `red`
// (two halves, taken in turn, so that one barrier per sum is enough).
struct Red {
  float v[2][3][32];
};
template <int LANES, int K>
__device__ __forceinline__ void row_sum(float* s, Red& red, int& turn) {
  constexpr int FIRST = LANES ? LANES / 2 : 16;
#pragma unroll
  for (int o = FIRST; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += __shfl_xor_sync(~0u, s[k], o);
  if constexpr (LANES == 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (warps > 1) {
      if (lane < K) {
        float mine = s[0];
#pragma unroll
        for (int k = 1; k < K; ++k) mine = lane == k ? s[k] : mine;
        red.v[turn][lane][warp] = mine;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        s[k] = lane < warps ? red.v[turn][k][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s[k] += __shfl_xor_sync(~0u, s[k], o);
      }
      turn ^= 1;
    }
  }
}

// Which rows a group takes: rows are (token, head); a group keeps one head, so that the sums
// for that head's weights stay in its registers, and takes every step-th token.
struct Walk {
  int head, tok, step, iters, tid, threads;      // tok: the first; tid of `threads` in the group
  bool on;                                       // whether the group has a head at all
};
template <int LANES>
__device__ __forceinline__ Walk walk_of(int tokens, int H, int groups) {
  Walk w;
  w.threads = LANES ? LANES : blockDim.x;
  w.tid = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x;
  const int gid = LANES ? blockIdx.x * (blockDim.x / (LANES ? LANES : 1)) + threadIdx.x / (LANES ? LANES : 1)
                        : blockIdx.x;
  w.on = gid < groups;                           // groups: a multiple of H
  w.head = gid % H;
  w.tok = gid / H;
  w.step = groups / H;
  w.iters = (tokens + w.step - 1) / w.step;      // of every group alike; rows past the end idle
  return w;
}

// A strided view [B, T, H, D] or a dense one.
struct View {
  const void* p;
  int64_t b, t, h;
  // Of token `tok` of all batch rows; flat: those are one token stride apart, too.
  __device__ __forceinline__ int64_t at(int tok, int T, int flat, int head) const {
    if (flat) return tok * t + head * h;
    const int bi = tok / T;
    return bi * b + (tok - bi * T) * t + head * h;
  }
};
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(at)
               : "memory");
  return u;
}

// A group's copies ahead of time: every thread's own pieces of 16 bytes, in its own places of
// shared memory, so that no barrier is needed between a copy and its use.
struct Ahead {
  uint32_t base, pitch;                          // of this thread; from piece to piece
  int pieces, stages;
  __device__ __forceinline__ Ahead(const char* places, int pieces_, int stages_)
      : base(ptx::smem_u32(places) + threadIdx.x * 16),
        pitch(blockDim.x * 16),
        pieces(pieces_),
        stages(stages_) {}
  __device__ __forceinline__ uint32_t of(int stage) const { return base + stage * pieces * pitch; }
  __device__ __forceinline__ void wait() const {
    if (stages == 3)
      ptx::cp_async_wait<2>();
    else if (stages == 2)
      ptx::cp_async_wait<1>();
    else
      ptx::cp_async_wait<0>();
  }
};

// One tensor of a row. With S::kAhead its runs come from the thread's places in shared memory,
// from `first` on, where fetch() had them copied; with S::kRegs from registers, where fetch() put
// the next row's and advance() made them this one's; else group() brings them.
template <class S, bool ONLY_READ>
struct Row {
  const void* p;                                 // the row's first element
  int is_bf16, first;                            // first: its first piece within a stage
  uint32_t now[S::kRegs ? S::N : S::kGroups ? S::kGroup * S::V : 1], next[S::kRegs ? S::N : 1];
  __device__ __forceinline__ void set(const void* base, int64_t at, int bf, int piece) {
    p = static_cast<const char*>(base) + at * (bf ? 2 : 4);
    is_bf16 = bf;
    first = piece;
  }
  __device__ __forceinline__ int per_run() const { return is_bf16 ? 1 : 2; }
  // D: the row's length.
  __device__ __forceinline__ void fetch(const Ahead& a, uint32_t places, int c, int i, int D) {
    if constexpr (S::kRegs) {
      next[c] = load_raw<ONLY_READ>(p, i, is_bf16);
    } else {
      const int es = is_bf16 ? 2 : 4;
      const uint32_t at = places + (first + c * per_run()) * a.pitch;
      const char* src = static_cast<const char*>(p) + (int64_t)i * es;
      int left = 16 * per_run();                 // bytes of the run
      if (S::SHIFT) left = min(left, (D - i) * es);        // nothing behind the row is read
      ptx::cp_async16(at, src, min(left, 16));
      if (!is_bf16) {
        const bool more = left > 16;
        ptx::cp_async16(at + a.pitch, more ? src + 16 : src, more ? left - 16 : 0);
      }
    }
  }
  __device__ __forceinline__ void advance() {
    if constexpr (S::kRegs)
#pragma unroll
      for (int j = 0; j < S::N; ++j) now[j] = next[j];
  }
  // Runs c .. c + kGroup - 1, all under way at once: zeros behind the row.
  __device__ __forceinline__ void group(const Walk& w, int c, int D) {
    if constexpr (S::kGroups) {
      auto bring = [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
#pragma unroll
        for (int j = 0; j < S::kGroup; ++j) {
          const int i = ((c + j) * w.threads + w.tid) * S::V;
          uint32_t* to = now + j * S::V;
          if constexpr (S::V == 1) {
            to[0] = i < D ? load_raw<ONLY_READ>(p, i, sizeof(T) == 2) : 0u;
          } else {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(p) + i);
#pragma unroll
            for (int k = 0; k < S::V * (int)sizeof(T) / 16; ++k) {
              uint4 u = make_uint4(0, 0, 0, 0);
              if (i < D) u = ONLY_READ ? __ldg(q + k) : q[k];
              to[4 * k] = u.x, to[4 * k + 1] = u.y, to[4 * k + 2] = u.z, to[4 * k + 3] = u.w;
            }
          }
        }
      };
      if (is_bf16)
        bring(static_cast<bf16*>(nullptr));
      else
        bring(static_cast<float*>(nullptr));
    }
  }
  __device__ __forceinline__ void get(const Ahead& a, uint32_t places, int c, int i, int D,
                                      float* f) const {
    if constexpr (S::kAhead) {
      const uint32_t at = places + (first + c * per_run()) * a.pitch;
      const uint4 u = shared16(at);
      if (is_bf16) {
        const Run<bf16, 8> r = {{u.x, u.y, u.z, u.w}};
        unpack<bf16, 8>(r, f);
      } else {
        const uint4 v = shared16(at + a.pitch);
        const Run<float, 8> r = {{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w}};
        unpack<float, 8>(r, f);
      }
      if (S::SHIFT && (i < 0 || i + 8 > D)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i + e < 0 || i + e >= D) f[e] = 0.f;
      }
    } else if constexpr (S::kRegs) {
      f[0] = raw_value(now[c], is_bf16);
    } else if constexpr (S::V == 1) {
      f[0] = raw_value(now[c % S::kGroup], is_bf16);
    } else {
      const uint32_t* u = now + c % S::kGroup * S::V;
      if (is_bf16) {
        const Run<bf16, 8> r = {{u[0], u[1], u[2], u[3]}};
        unpack<bf16, 8>(r, f);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(u[e]);
      }
    }
  }
};
// A run's elements of a vector [D] that all rows share (0 outside it).
template <class S>
__device__ __forceinline__ void load_shared(const float* w, int i, int D, float* f) {
  if constexpr (S::SHIFT) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = i + e >= 0 && i + e < D ? __ldg(w + i + e) : 0.f;
  } else {
    load_run<float, S::V, true>(w + i, f);
  }
}
// The next group of a row's tensors, where run c is its first.
template <class S, typename... Rows>
__device__ __forceinline__ void group_at(const Walk& w, int c, int D, Rows&... rows) {
  if constexpr (S::kGroups)
    if (c % S::kGroup == 0) (rows.group(w, c, D), ...);
}

// A run into a row.
template <class S>
__device__ __forceinline__ void store_row(void* p, size_t row, int i, int D, int is_bf16,
                                          const float* f) {
  if (S::SHIFT && (i < 0 || i + 8 > D)) {
#pragma unroll
    for (int e = 0; e < S::V; ++e)
      if (i + e >= 0 && i + e < D) store_any<1>(p, (int64_t)row + i + e, is_bf16, f + e);
  } else {
    store_any<S::V>(p, (int64_t)row + i, is_bf16, f);
  }
}
// A run of the weights' gradients, whose rows have no alignment of their own with SHIFT.
template <class S>
__device__ __forceinline__ void store_part(float* p, int i, int D, const float* f) {
  if constexpr (S::SHIFT) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e >= 0 && i + e < D) p[i + e] = f[e];
  } else {
    store_run<float, S::V>(p + i, f);
  }
}

// Column sums of part [which][rows][cols] into out<which>. A block takes 8 columns (a sector of
// a row) and its 64 rows of threads share the parts, so that few loads follow one another.
constexpr int kSumCols = 8, kSumRows = 64;
__global__ void __launch_bounds__(kSumCols * kSumRows) column_sum_kernel(const float* part,
                                                                         float* out0, float* out1,
                                                                         float* out2, int rows,
                                                                         int cols) {
  __shared__ float s[kSumRows][kSumCols + 1];
  wait_for_before();                             // the parts are written
  const int x = threadIdx.x % kSumCols, r0 = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + x, which = blockIdx.y;
  float* out = which == 0 ? out0 : which == 1 ? out1 : out2;
  if (!out) return;
  const float* p = part + (size_t)which * rows * cols;
  float v = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int r = r0; r < rows; r += kSumRows) v += p[(size_t)r * cols + c];
  }
  s[r0][x] = v;
  __syncthreads();
#pragma unroll
  for (int n = kSumRows / 2; n > 0; n >>= 1) {
    if (r0 < n) s[r0][x] += s[r0 + n][x];
    __syncthreads();
  }
  if (r0 == 0 && c < cols) out[c] = s[0][x];
}

// A block's part of a weight gradient: its group's sums, or those of its groups added in order,
// element by element (groups of SHIFT have phases of their own); s: S::kSums floats.
template <class S>
__device__ __forceinline__ void block_part(const float* acc, float* s, float* to, const Walk& w,
                                           int phase, int D) {
  if constexpr (S::LANES == 0) {
#pragma unroll
    for (int c = 0; c < S::NV; ++c) {
      const int i = (c * w.threads + w.tid) * S::V - phase;
      if (i < D) store_part<S>(to, i, D, acc + c * S::V);
    }
  } else {
    const int groups = blockDim.x / S::LANES;
    __syncthreads();                             // the last sum's readers are done
#pragma unroll
    for (int c = 0; c < S::NV; ++c)
#pragma unroll
      for (int e = 0; e < S::V; ++e) {
        const int i = (c * w.threads + w.tid) * S::V - phase + e;
        if (i >= 0 && i < D) s[threadIdx.x / S::LANES * D + i] = acc[c * S::V + e];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
      float v = 0.f;
      for (int g = 0; g < groups; ++g) v += s[g * D + i];
      to[i] = v;
    }
  }
}

// ------------------------------------------------------------------ host
constexpr int kSms = 152;
constexpr int kWidest = 16384;                   // elements of a row at most
// Of copies, an SM and a block at most: what does not fit twice goes without a row ahead (the
// residual's backward with 32-bit tensors: 96 threads of 1536 channels, five blocks an SM, 21 KB each).
constexpr int kSmemPerSm = 200 * 1024;
constexpr int kGroupsPerSm = 512;                // threads, of rows in groups of elements
constexpr int kPlainSmem = 24 * 1024;            // fits beside the static part without being asked for

// What a call's kernel looks like: threads of a block, groups and blocks, copies ahead.
struct Plan {
  int lanes, v, nv, threads, groups, blocks, rows;   // rows: of the parts, per weight
  bool shift;
  int pieces, stages, smem;
};

// f(Shape) for a plan.
template <typename F>
auto with_block(const Plan& p, F f) {
  if (p.shift) return f(Shape<0, 8, 2, true>());
  if (p.v == 8) return p.nv == 2 ? f(Shape<0, 8, 2>()) : f(Shape<0, 8, 4>());
  return p.nv == 4    ? f(Shape<0, 1, 4>())
         : p.nv == 8  ? f(Shape<0, 1, 8>())
         : p.nv == 16 ? f(Shape<0, 1, 16>())
                      : f(Shape<0, 1, 32>());
}
// TWO: whether rows of more than 256 elements share a warp.
template <bool TWO, typename F>
auto with_shape(const Plan& p, F f) {
  if (p.lanes == 0) return with_block(p, f);
  if (p.shift)
    return p.lanes == 8    ? f(Shape<8, 8, 1, true>())
           : p.lanes == 16 ? f(Shape<16, 8, 1, true>())
                           : f(Shape<32, 8, 1, true>());
  if (p.v == 1) return f(Shape<32, 1, 8>());
  if constexpr (TWO)
    if (p.nv == 2) return f(Shape<32, 8, 2>());
  return p.lanes == 8    ? f(Shape<8, 8, 1>())
         : p.lanes == 16 ? f(Shape<16, 8, 1>())
                         : f(Shape<32, 8, 1>());
}

// How a call's rows lie: 16-byte accesses fit; fit but for a phase (Shape's SHIFT); or neither.
enum Fit { kVec, kShift, kSingle };

// pieces: 16-byte pieces per run of 8, over all tensors of a row. widest: elements of a row that
// shares a warp, at most (256 where rows have a phase or no alignment). per_sm: threads an SM is
// to hold.
Plan make_plan(int tokens, int H, int D, int pieces, Fit fit, int widest, bool per_head,
               int per_sm) {
  Plan p = {};
  p.shift = fit == kShift && D + 7 <= kMaxThreads * 16;
  const bool vec = fit == kVec || p.shift;
  p.v = vec ? 8 : 1;
  const int span = D + (p.shift ? 7 : 0);        // elements that a row's threads cover
  p.lanes = span > (fit == kVec ? widest : 256) ? 0
            : !vec || span > 128                ? 32
            : span > 64                         ? 16
                                                : 8;
  int per_block = 1;                             // groups of a block
  if (p.lanes) {
    p.nv = !vec ? 8 : span > 256 ? 2 : 1;
    p.threads = 256;
    per_block = p.threads / p.lanes;
  } else {
    // Elements of a thread: 16, 32 in the widest rows; element by element as few as 512 threads
    // allow (more threads have more loads under way: 1776 rows of 4075 with a gate from an odd
    // slice, training step, 124 us with 16 a thread, 70 with 8).
    p.nv = vec                     ? (D <= kMaxThreads * 16 ? 2 : 4)
           : D <= kMaxThreads * 4  ? 4
           : D <= kMaxThreads * 8  ? 8
           : D <= kMaxThreads * 16 ? 16
                                   : 32;
    const int n = p.nv * p.v;
    p.threads = ((span + n - 1) / n + 31) / 32 * 32;
  }
  if (p.lanes == 0 && !vec && p.nv > 8 && per_sm > kGroupsPerSm) per_sm = kGroupsPerSm;
  const long long rows = (long long)tokens * H;
  long long blocks = (rows + per_block - 1) / per_block;
  const long long most = (long long)kSms * (per_sm / p.threads > 1 ? per_sm / p.threads : 1);
  if (blocks > most) blocks = most;
  const long long least = (H + per_block - 1) / per_block;     // a group per head
  if (blocks < least) blocks = least;
  long long groups = blocks * per_block / H * H;
  if (p.shift && groups < rows) {                // steps of 8 tokens, for one phase per group
    const long long unit = 8LL * H;
    groups = groups < unit ? unit : groups / unit * unit;
    blocks = (groups + per_block - 1) / per_block;
  }
  p.blocks = (int)blocks;
  p.groups = (int)groups;
  p.rows = per_head ? p.groups / H : p.blocks;
  p.pieces = pieces * p.nv;
  p.stages = !vec && p.nv <= 8 ? 2 : 1;          // 2: the next row in registers
  if (p.v == 8 && p.nv <= 2) {
    const int stage = p.pieces * p.threads * 16;
    const int resident = per_sm / p.threads > 1 ? per_sm / p.threads : 1;
    p.stages = 3;
    while (p.stages > 1 && (long long)p.stages * stage * resident > kSmemPerSm) --p.stages;
    p.smem = p.stages * stage;
  }
  return p;
}

// The fit of a view [B, T, H, D] (strides of dimensions of one element: 0).
Fit fit_of(const void* p, int B, int T, int H, int D, int64_t b, int64_t t, int64_t h) {
  if (!is_aligned(p, 16)) return kSingle;
  const int64_t row = D, tok = row * H, batch = tok * T;
  if ((B > 1 && (b - batch) % 8) || (T > 1 && (t - tok) % 8) || (H > 1 && (h - row) % 8))
    return kSingle;
  return D % 8 ? kShift : kVec;
}
Fit worse(Fit a, Fit b) { return a > b ? a : b; }

// Column sums of the parts, behind the kernel that writes them.
gdr_status sum_parts(const float* part, float* o0, float* o1, float* o2, int rows, int cols,
                     cudaStream_t s) {
  return launch_behind(column_sum_kernel, dim3((cols + kSumCols - 1) / kSumCols, o1 || o2 ? 3 : 1),
                       kSumCols * kSumRows, s, part, o0, o1, o2, rows, cols);
}
gdr_status zero(float* p, size_t n, cudaStream_t s) {
  return !p || n == 0 ? GDR_OK : status_of(cudaMemsetAsync(p, 0, n * sizeof(float), s));
}

bool bad_eps(float e) { return !(isfinite(e) && e > 0.f); }
bool bad_act(int k) { return k != GDR_ACT_NONE && k != GDR_ACT_SIGMOID && k != GDR_ACT_SILU; }

// Threads that an SM is to hold, as their registers allow: forward; the residual's backward, and
// with a norm, gate or scale per channel (at most the former); the gated norm forward with a phase,
// and backward; gated_rows_kernel, forward and backward. (Residual training step of 2 x 8192 x 4096:
// 197 us with 1024 both ways; 1280 and 1536 forward gave 224 and 243, 768 backward 231. The others
// were not measured beside their neighbours.)
constexpr int kFwdPerSm = 1024, kBwdPerSm = 1024, kFullPerSm = 512;
constexpr int kGatedShiftPerSm = 640, kGatedBwdPerSm = 512;
constexpr int kFwdRowsPerSm = 768, kBwdRowsPerSm = 512;

}  // namespace
}  // namespace ops
}  // namespace gdr
