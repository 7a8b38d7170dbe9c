// Device helpers shared by the kernels that walk token rows (basa_rope.cu,
// basa_gnorm.cu): eight consecutive elements of a row as one unit of loading and
// storing, packed fp32 pairs as the unit of arithmetic, parameters of two types.
// Everything here has internal linkage.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "basa_internal.h"

namespace basa {
namespace {

// ---------------------------------------------------------------------------
// Packed fp32 pairs (sm_100's f32x2 arithmetic): two values an instruction.
// These kernels move about 24 bytes per SM and clock, so the instructions spent
// per value decide whether they keep up with HBM.
// ---------------------------------------------------------------------------
typedef uint64_t f2;

__device__ __forceinline__ f2 pk(float lo, float hi) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 un(f2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float sum2(f2 v) {
  const float2 f = un(v);
  return f.x + f.y;
}

// ---------------------------------------------------------------------------
// Eight consecutive elements
// ---------------------------------------------------------------------------
struct e4m3_t {
  uint8_t bits;
};

template <typename T> struct Raw8;  // as they lie in memory
template <> struct Raw8<__nv_bfloat16> { uint4 a; };
template <> struct Raw8<float> { uint4 a, b; };

__device__ __forceinline__ void load8(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* p) {
  r.a = __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void load8(Raw8<float>& r, const float* p) {
  r.a = __ldcs(reinterpret_cast<const uint4*>(p));
  r.b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
}
__device__ __forceinline__ void zero8(Raw8<__nv_bfloat16>& r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void zero8(Raw8<float>& r) { r.a = r.b = make_uint4(0, 0, 0, 0); }

// Element i of the eight, in fp32.  Exact: a bf16 value is the upper half of
// the fp32 value it stands for.
__device__ __forceinline__ float elem(const Raw8<__nv_bfloat16>& r, int i) {
  const uint32_t w = i < 2 ? r.a.x : i < 4 ? r.a.y : i < 6 ? r.a.z : r.a.w;
  return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}
__device__ __forceinline__ float elem(const Raw8<float>& r, int i) {
  const uint4& v = i < 4 ? r.a : r.b;
  const int k = i & 3;
  return __uint_as_float(k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w);
}
// In order: p[i] = (element 2i, element 2i + 1).
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, f2 (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pk(elem(r, 2 * i), elem(r, 2 * i + 1));
}

// Rounds to nearest even, once, on the way out.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  uint4 r;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = r;
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  float4* o = reinterpret_cast<float4*>(p);
  o[0] = make_float4(f[0], f[1], f[2], f[3]);
  o[1] = make_float4(f[4], f[5], f[6], f[7]);
}
// e4m3: values beyond the type's largest, 448, become 448; NaN stays NaN.
__device__ __forceinline__ void store8(e4m3_t* p, const float (&f)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <typename T>
__device__ __forceinline__ void store8(T* o, const f2 (&p)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = un(p[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
  store8(o, f);
}

// ---------------------------------------------------------------------------
// Asynchronous copies.  Every thread copies its own columns of a row to its own
// bytes of a stage in shared memory and is the only one to read them, so the
// stages need no barrier.  A slot holds one tensor's vectors of a stage, in
// 16-byte pieces, the threads side by side.
// ---------------------------------------------------------------------------
// on = false: sixteen bytes of zeros, and src, any valid address, is not read.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most kAhead of this thread's groups are in flight.
template <int kAhead>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
}

template <typename T>
struct Slot {
  static constexpr int kPieces = (int)sizeof(T) / 2;
  __host__ __device__ static constexpr int bytes(int vectors, int threads) {
    return vectors * kPieces * threads * 16;
  }
  __device__ static __forceinline__ void fetch(uint32_t at, const T* src, int j, int threads,
                                               int tid, bool on) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      copy16(at + ((j * kPieces + p) * threads + tid) * 16,
             reinterpret_cast<const char*>(src) + p * 16, on);
  }
  __device__ static __forceinline__ void take(const char* at, int j, int threads, int tid,
                                              Raw8<T>& r) {
    const uint4* s = reinterpret_cast<const uint4*>(at) + j * kPieces * threads + tid;
    r.a = s[0];
    if constexpr (kPieces == 2) r.b = s[threads];
  }
};

__device__ __forceinline__ uint32_t shared_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------------------
// Parameters (norm weights, modulations) of type bf16 or fp32, eight from
// column `col`, a multiple of 8; `fill` where there are none.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void param8(const void* p, bool bf16, long long col, float fill,
                                       float (&f)[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fill;
  } else if (bf16) {
    Raw8<__nv_bfloat16> r;
    r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + col));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = elem(r, i);
  } else {
    Raw8<float> r;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + col);
    r.a = __ldg(q);
    r.b = __ldg(q + 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = elem(r, i);
  }
}
__device__ __forceinline__ void param8(const void* p, bool bf16, long long col, float fill,
                                       f2 (&v)[4]) {
  float f[8];
  param8(p, bf16, col, fill, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pk(f[2 * i], f[2 * i + 1]);
}
// Eight parameters on their way to L1, so that those of several kinds that a
// kernel takes one after another wait for memory once.
__device__ __forceinline__ void ahead8(const void* p, bool bf16, long long col) {
  if (p)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const char*>(p) +
                                                  col * (bf16 ? 2 : 4)));
}
// Gradients of parameters, in the parameters' type.
__device__ __forceinline__ void store_param8(void* p, bool bf16, long long col, const f2 (&f)[4]) {
  if (bf16)
    store8(static_cast<__nv_bfloat16*>(p) + col, f);
  else
    store8(static_cast<float*>(p) + col, f);
}
__device__ __forceinline__ void store_param(void* p, bool bf16, long long col, float f) {
  if (bf16)
    static_cast<__nv_bfloat16*>(p)[col] = __float2bfloat16_rn(f);
  else
    static_cast<float*>(p)[col] = f;
}

template <int kLanes>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Two sums side by side.
template <int kLanes>
__device__ __forceinline__ float2 lane_sum(float2 v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, v.x, o), y = __shfl_xor_sync(0xffffffffu, v.y, o);
    v.x += x;
    v.y += y;
  }
  return v;
}

// The same value, but one that the compiler takes for a new one: what is formed
// from it inside a loop is not moved ahead of the loop, where it would hold
// registers that the loop does not have.
__device__ __forceinline__ int anew(int v) {
  asm volatile("" : "+r"(v));
  return v;
}
// Keeps the compiler from loading all of a sequence's operands ahead of using
// the first, for the same reason.
__device__ __forceinline__ void one_by_one() { asm volatile("" ::: "memory"); }

// Programmatic dependent launch: a kernel that ends a gradient's sums is launched
// while the one that leaves the partial sums still runs, and waits for it.
__device__ __forceinline__ void dependents_may_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_partial_sums() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
template <typename... P, typename... A>
basa_status launch_dependent(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream,
                             const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess) return BASA_OK;
  cudaGetLastError();  // reported here, not by the next call
  return BASA_ERR_CUDA;
}

// Dynamic shared memory of a CTA at most, of an SM's 228 KB beside static parts and the
// CTAs' own 1 KB.
constexpr int kMostSmem = 224 * 1024;
// Dynamic shared memory beyond what a kernel may use unasked (48 KB with its static
// part) has to be allowed.  What is allowed belongs to the kernel, not to the launch:
// always the same, or a call of another host thread with narrower rows could lower
// it between this and the launch.
template <typename K>
bool allow_smem(K kernel, int smem) {
  if (smem <= 32 * 1024 ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) ==
          cudaSuccess)
    return true;
  cudaGetLastError();
  return false;
}

inline int row_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();  // no device: the workspace sizes of a B200
    return 148;
  }
  return n;
}
// Where a call's tensors lie.  An output may take one input's place where the header
// says so (same address, dense rows, same type); any other byte of an output that
// another output or an input has too would be read or written by two parts of a launch.
struct Overlap {
  struct Rows {
    unsigned long long at, bytes, row, ld;  // first to last byte, of a row, from row to row
    bool out;
    const void* place;  // of an output: the input whose place it may take
  };
  Rows all[24];
  int n = 0;
  // rows of `row` bytes, ld bytes apart (0 or one row: dense)
  void add(const void* p, long long rows, long long row, long long ld, bool out, const void* place) {
    if (!p || rows <= 0 || row <= 0) return;
    const bool one = rows == 1 || ld == row;
    const unsigned long long r = rows, w = row, step = one ? w : ld, bytes = (r - 1) * step + w;
    all[n++] = Rows{(unsigned long long)reinterpret_cast<uintptr_t>(p), bytes, one ? bytes : w,
                    one ? 0 : step, out, place};
  }
  void in(const void* p, long long rows, long long row, long long ld) { add(p, rows, row, ld, false, nullptr); }
  void in(const void* p, long long bytes) { in(p, 1, bytes, 0); }
  void out(const void* p, long long rows, long long row, long long ld, const void* place) {
    add(p, rows, row, ld, true, place);
  }
  void out(const void* p, long long bytes, const void* place = nullptr) { out(p, 1, bytes, 0, place); }
  // Slices of one buffer lie side by side in what the strides have in common.
  static bool meet(const Rows& a, const Rows& b) {
    if (a.at + a.bytes <= b.at || b.at + b.bytes <= a.at) return false;
    unsigned long long g = a.ld, h = b.ld;
    while (h) {
      const unsigned long long t = g % h;
      g = h;
      h = t;
    }
    if (!g) return true;
    const unsigned long long off = b.at >= a.at ? (b.at - a.at) % g : (g - (a.at - b.at) % g) % g;
    return off < a.row || off + b.row > g;
  }
  bool any() const {
    for (int i = 0; i < n; ++i) {
      if (!all[i].out) continue;
      bool taken = false;  // the place of one input, once
      for (int j = 0; j < n; ++j) {
        if (j == i || (all[j].out && j < i) || !meet(all[i], all[j])) continue;
        const bool own = !all[j].out && !taken && all[i].place &&
                         all[j].at == (unsigned long long)reinterpret_cast<uintptr_t>(all[i].place) &&
                         all[i].at == all[j].at && all[i].bytes == all[j].bytes;
        if (!own) return true;
        taken = true;
      }
    }
    return false;
  }
};
inline bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace
}  // namespace basa
