// What stands between a q/k/v projection and the attention calls: RMS norm of q
// and k, rotary positions with three axes, and the copy of q, k, v out of the
// projection's rows into the dense layout the attention reads (basa_qkv_rope),
// with its backward (basa_qkv_rope_bwd) and the table of angles
// (basa_rope_table).
//
// With n = x r w, r = 1 / sqrt(mean(x^2) + eps) (over a head's d values or over
// all heads of a token) and pair (a, b) of n turned by the angle of its axis:
//   forward   (a cos - b sin, a sin + b cos)
//   backward  gn = the output's gradient turned by minus the angle,
//             dx = r (w gn - x r^2 mean(w gn x)),  dw = sum over rows of gn x r.
#include <math.h>
#include <string.h>

#include "row_device.cuh"

namespace basa {
namespace {

struct RopePart {      // one of q, k, v
  const void* x;       // input rows (the forward's input)
  const void* g;       // backward: gradient of the forward's output, dense
  void* o;             // forward: output, dense; backward: gradient of x
  const void* w;       // norm weight, or null
  float* part;         // backward: partial sums of the weight's gradient
  long long ldx, ldg, ldo;
  int heads;
  int chunks;          // CTAs that share a token's heads
  int steps;           // of kHeadsPerWarp heads, per chunk
  float mul;           // e4m3 output: 1 / descale
};

struct RopeArgs {
  RopePart q, k, v;
  const float2* table;
  uint32_t tokens, T, Hg, Wg;
  int nt, nh, nw;      // rotated pairs per axis
  int d;
  float eps;
  int w_bf16;
};

__device__ __forceinline__ RopePart pick(const RopeArgs& a, int part) {
  return part == 0 ? a.q : part == 1 ? a.k : a.v;
}

// The rotation of the eight elements at 8 * sub of a head: element i and its
// partner share cs[pair(i)].  Pairs of neighbours: four angles.  Pairs half the
// rotated width apart: eight, the partner's elements lie in another lane.
template <bool kHalves>
struct Turn {
  static constexpr int kN = kHalves ? 8 : 4;
  int base[kN];
  uint32_t axis;   // two bits a pair; 3: not rotated
  float sign;      // halves: -1 for the first element of a pair, +1 for the second
  int partner;     // halves: lane that holds the partner's elements
  float2 cs[kN];

  __device__ __forceinline__ void init(const RopeArgs& a, int sub, int lanes_per_head) {
    const int pairs = a.nt + a.nh + a.nw;
    const int lane = threadIdx.x & 31;
    int j0 = sub * 4;
    sign = 1.f;
    partner = lane;
    if (kHalves) {
      j0 = sub * 8;
      if (j0 < pairs) {
        sign = -1.f;
        partner = lane + pairs / 8;
      } else if (j0 < 2 * pairs) {
        j0 -= pairs;
        partner = lane - pairs / 8;
      } else {
        j0 = pairs;
      }
    }
    axis = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int j = j0 + i;
      uint32_t ax = 3;
      base[i] = 0;
      if (j < a.nt) {
        ax = 0;
        base[i] = j;
      } else if (j < a.nt + a.nh) {
        ax = 1;
        base[i] = (int)a.T * a.nt + j - a.nt;
      } else if (j < pairs) {
        ax = 2;
        base[i] = (int)a.T * a.nt + (int)a.Hg * a.nh + j - a.nt - a.nh;
      }
      axis |= ax << (2 * i);
    }
  }

  // The angles of token n; dir = -1 turns back.
  __device__ __forceinline__ void load(const RopeArgs& a, uint32_t n, float dir) {
    const uint32_t row = n / a.Wg, x = n - row * a.Wg;
    const uint32_t frame = row / a.Hg, y = row - frame * a.Hg;
    const uint32_t t = frame % a.T;
    const int ot = (int)t * a.nt, oy = (int)y * a.nh, ox = (int)x * a.nw;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t ax = (axis >> (2 * i)) & 3u;
      float2 v = make_float2(1.f, 0.f);
      if (ax != 3u) v = __ldg(a.table + base[i] + (ax == 0u ? ot : ax == 1u ? oy : ox));
      v.y *= kHalves ? dir * sign : dir;
      cs[i] = v;
    }
  }

  __device__ __forceinline__ void apply(float (&f)[8]) const {
    if (kHalves) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_sync(0xffffffffu, f[i], partner);
        f[i] = f[i] * cs[i & (kN - 1)].x + other * cs[i & (kN - 1)].y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = f[2 * i], q = f[2 * i + 1];
        f[2 * i] = p * cs[i].x - q * cs[i].y;
        f[2 * i + 1] = p * cs[i].y + q * cs[i].x;
      }
    }
  }
};

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeBatch = 4;  // steps whose loads are issued together

// Norm over each head, or none.  kLph lanes hold a head, a warp 32 / kLph heads
// (a step); a warp takes the steps of its chunk of one token, then the next
// token, so that a token's angles are read once for all its heads and a
// thread's columns of the weight stay in registers.
template <typename TI, typename TO, int kLph, bool kHalves, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads) rope_head_kernel(RopeArgs a) {
  constexpr int kHpw = 32 / kLph;
  int chunk = blockIdx.y, part = 0;
  if (chunk >= a.q.chunks) {
    chunk -= a.q.chunks;
    part = 1;
    if (chunk >= a.k.chunks) {
      chunk -= a.k.chunks;
      part = 2;
    }
  }
  const RopePart P = pick(a, part);
  const int lane = threadIdx.x & 31, sub = lane % kLph, slot = lane / kLph;
  const int h0 = chunk * P.steps * kHpw + slot;
  const int hend = min(P.heads, (chunk + 1) * P.steps * kHpw);
  const uint32_t stride = gridDim.x * kRopeWarps;
  Turn<kHalves> turn;
  float w[8];
  if (part < 2) {
    turn.init(a, sub, kLph);
    if (kNorm) param8(P.w, a.w_bf16, sub * 8, 1.f, w);
  }
  for (uint32_t n = blockIdx.x * kRopeWarps + threadIdx.x / 32; n < a.tokens; n += stride) {
    const TI* x = static_cast<const TI*>(P.x) + (long long)n * P.ldx + sub * 8;
    TO* o = static_cast<TO*>(P.o) + (long long)n * P.ldo + sub * 8;
    if (part < 2) turn.load(a, n, 1.f);
    for (int s = 0; s < P.steps; s += kRopeBatch) {
      Raw8<TI> raw[kRopeBatch];
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        const int h = h0 + (s + u) * kHpw;
        if (h < hend)
          load8(raw[u], x + h * (kLph * 8));
        else
          zero8(raw[u]);
      }
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        const int h = h0 + (s + u) * kHpw;
        float f[8];
        widen8(raw[u], f);
        if (part < 2) {
          if (kNorm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
            const float r = rsqrtf(lane_sum<kLph>(ss) * (1.f / (kLph * 8)) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= r * w[i];
          }
          turn.apply(f);
        }
        if (sizeof(TO) == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= P.mul;
        }
        if (h < hend) store8(o + h * (kLph * 8), f);
      }
    }
  }
}

constexpr int kRopeBwdBatch = 2;

// Backward of rope_head_kernel, the same walk.  The weight's gradient is summed
// in a thread's own eight columns over all its tokens and heads, then over the
// CTA, and left as one row of partial sums a CTA.
template <typename T, int kLph, bool kHalves, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads) rope_head_bwd_kernel(RopeArgs a) {
  constexpr int kHpw = 32 / kLph;
  constexpr int kD = kLph * 8;
  __shared__ float red[kRopeWarps][kD];
  int chunk = blockIdx.y, part = 0;
  if (chunk >= a.q.chunks) {
    chunk -= a.q.chunks;
    part = 1;
    if (chunk >= a.k.chunks) {
      chunk -= a.k.chunks;
      part = 2;
    }
  }
  const RopePart P = pick(a, part);
  const int lane = threadIdx.x & 31, sub = lane % kLph, slot = lane / kLph;
  const int h0 = chunk * P.steps * kHpw + slot;
  const int hend = min(P.heads, (chunk + 1) * P.steps * kHpw);
  const uint32_t stride = gridDim.x * kRopeWarps;
  Turn<kHalves> turn;
  float w[8], acc[8];
  if (part < 2) {
    turn.init(a, sub, kLph);
    if (kNorm) param8(P.w, a.w_bf16, sub * 8, 1.f, w);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (uint32_t n = blockIdx.x * kRopeWarps + threadIdx.x / 32; n < a.tokens; n += stride) {
    const T* x = static_cast<const T*>(P.x) + (long long)n * P.ldx + sub * 8;
    const T* g = static_cast<const T*>(P.g) + (long long)n * P.ldg + sub * 8;
    T* o = static_cast<T*>(P.o) + (long long)n * P.ldo + sub * 8;
    if (part < 2) turn.load(a, n, -1.f);
    for (int s = 0; s < P.steps; s += kRopeBwdBatch) {
      Raw8<T> rg[kRopeBwdBatch], rx[kRopeBwdBatch];
#pragma unroll
      for (int u = 0; u < kRopeBwdBatch; ++u) {
        const int h = h0 + (s + u) * kHpw;
        zero8(rg[u]);
        zero8(rx[u]);
        if (h < hend) {
          load8(rg[u], g + h * kD);
          if (kNorm && part < 2) load8(rx[u], x + h * kD);
        }
      }
#pragma unroll
      for (int u = 0; u < kRopeBwdBatch; ++u) {
        const int h = h0 + (s + u) * kHpw;
        float f[8];
        widen8(rg[u], f);
        if (part < 2) {
          turn.apply(f);
          if (kNorm) {
            float xf[8];
            widen8(rx[u], xf);
            float ss = 0.f, sd = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              ss = fmaf(xf[i], xf[i], ss);
              sd = fmaf(xf[i], f[i] * w[i], sd);
            }
            ss = lane_sum<kLph>(ss);
            sd = lane_sum<kLph>(sd);
            const float r = rsqrtf(ss * (1.f / kD) + a.eps);
            const float c = sd * (1.f / kD) * r * r;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[i] = fmaf(f[i], xf[i] * r, acc[i]);
              f[i] = r * (f[i] * w[i] - xf[i] * c);
            }
          }
        }
        if (h < hend) store8(o + h * kD, f);
      }
    }
  }
  if (kNorm && part < 2 && P.part) {  // uniform over the CTA
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = acc[i];
#pragma unroll
      for (int m = kLph; m < 32; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
      if (slot == 0) red[threadIdx.x / 32][sub * 8 + i] = v;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < kD; c += kRopeThreads) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kRopeWarps; ++i) v += red[i][c];
      P.part[((long long)blockIdx.x * P.chunks + chunk) * kD + c] = v;
    }
  }
}

constexpr int kTokenMaxThreads = 512;

// Sum over the CTA of one or two values a thread; `buf` alternates between
// calls, so one barrier a call is enough.
__device__ __forceinline__ float2 block_sum(float a, float b, float2 (*red)[16], int buf) {
  a = lane_sum<32>(a);
  b = lane_sum<32>(b);
  if ((threadIdx.x & 31) == 0) red[buf][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
    s.x += red[buf][i].x;
    s.y += red[buf][i].y;
  }
  return s;
}

// Norm over all heads of a token: a CTA holds one token's q, k or v in
// registers (kV vectors of eight a thread), so its rows are read once.
template <typename TI, typename TO, int kV, bool kHalves>
__global__ void __launch_bounds__(kTokenMaxThreads) rope_token_kernel(RopeArgs a) {
  __shared__ float2 red[2][16];
  const int part = blockIdx.y;
  const RopePart P = pick(a, part);
  const int lph = a.d / 8, nvec = P.heads * lph, tid = threadIdx.x;
  const float inv = 1.f / (float)(P.heads * a.d);
  Turn<kHalves> turn;
  if (part < 2) turn.init(a, tid % lph, lph);
  int buf = 0;
  for (uint32_t n = blockIdx.x; n < a.tokens; n += gridDim.x, buf ^= 1) {
    const TI* x = static_cast<const TI*>(P.x) + (long long)n * P.ldx;
    TO* o = static_cast<TO*>(P.o) + (long long)n * P.ldo;
    Raw8<TI> raw[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = j * blockDim.x + tid;
      if (i < nvec)
        load8(raw[j], x + i * 8);
      else
        zero8(raw[j]);
    }
    float r = 1.f;
    if (part < 2) {
      turn.load(a, n, 1.f);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        float f[8];
        widen8(raw[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
      }
      r = rsqrtf(block_sum(ss, 0.f, red, buf).x * inv + a.eps);
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = j * blockDim.x + tid;
      float f[8];
      widen8(raw[j], f);
      if (part < 2) {
        float w[8];
        param8(i < nvec ? P.w : nullptr, a.w_bf16, i * 8, 1.f, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= r * w[e];
        turn.apply(f);
      }
      if (sizeof(TO) == 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= P.mul;
      }
      if (i < nvec) store8(o + i * 8, f);
    }
  }
}

// Backward of rope_token_kernel.  Both sums of a row (x^2 and w gn x) share one
// barrier; a thread's columns of the weight's gradient stay in registers over
// all its tokens and are left as one row of partial sums a CTA.
template <typename T, int kV, bool kHalves>
__global__ void __launch_bounds__(kTokenMaxThreads) rope_token_bwd_kernel(RopeArgs a) {
  __shared__ float2 red[2][16];
  const int part = blockIdx.y;
  const RopePart P = pick(a, part);
  const int lph = a.d / 8, nvec = P.heads * lph, tid = threadIdx.x;
  const float inv = 1.f / (float)(P.heads * a.d);
  Turn<kHalves> turn;
  if (part < 2) turn.init(a, tid % lph, lph);
  float acc[kV][8];
#pragma unroll
  for (int j = 0; j < kV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[j][e] = 0.f;
  int buf = 0;
  for (uint32_t n = blockIdx.x; n < a.tokens; n += gridDim.x, buf ^= 1) {
    const T* x = static_cast<const T*>(P.x) + (long long)n * P.ldx;
    const T* g = static_cast<const T*>(P.g) + (long long)n * P.ldg;
    T* o = static_cast<T*>(P.o) + (long long)n * P.ldo;
    Raw8<T> rx[kV], rg[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = j * blockDim.x + tid;
      zero8(rx[j]);
      zero8(rg[j]);
      if (i < nvec) {
        load8(rg[j], g + i * 8);
        if (part < 2) load8(rx[j], x + i * 8);
      }
    }
    if (part == 2) {
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const int i = j * blockDim.x + tid;
        float f[8];
        widen8(rg[j], f);
        if (i < nvec) store8(o + i * 8, f);
      }
      continue;
    }
    turn.load(a, n, -1.f);
    float gn[kV][8], ss = 0.f, sd = 0.f;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = j * blockDim.x + tid;
      float xf[8], w[8];
      widen8(rg[j], gn[j]);
      turn.apply(gn[j]);
      widen8(rx[j], xf);
      param8(i < nvec ? P.w : nullptr, a.w_bf16, i * 8, 1.f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(xf[e], xf[e], ss);
        sd = fmaf(xf[e], gn[j][e] * w[e], sd);
      }
    }
    const float2 s = block_sum(ss, sd, red, buf);
    const float r = rsqrtf(s.x * inv + a.eps), c = s.y * inv * r * r;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = j * blockDim.x + tid;
      float xf[8], w[8], f[8];
      widen8(rx[j], xf);
      param8(i < nvec ? P.w : nullptr, a.w_bf16, i * 8, 1.f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[j][e] = fmaf(gn[j][e], xf[e] * r, acc[j][e]);
        f[e] = r * (gn[j][e] * w[e] - xf[e] * c);
      }
      if (i < nvec) store8(o + i * 8, f);
    }
  }
  if (part < 2 && P.part) {
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = j * blockDim.x + tid;
      if (i < nvec) store8(P.part + (long long)blockIdx.x * nvec * 8 + i * 8, acc[j]);
    }
  }
}

// out[c] = sum over rows of part[row][c], for two matrices in one launch
// (blockIdx.y).  A CTA owns eight columns; 32 rows are read side by side and
// joined in a fixed order, so equal calls give equal bits.
struct ColSum {
  const float* part;
  void* out;
  int rows, cols;
};
__global__ void __launch_bounds__(256) rope_colsum_kernel(ColSum s0, ColSum s1, int bf16) {
  __shared__ float red[32][9];
  const ColSum s = blockIdx.y ? s1 : s0;
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), lane = threadIdx.x >> 3;
  if (blockIdx.x * 8 >= s.cols || !s.out) return;  // cols is a multiple of 8
  float v = 0.f;
  for (int r = lane; r < s.rows; r += 32) v += s.part[(long long)r * s.cols + c];
  red[lane][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += red[i][threadIdx.x];
    store_param(s.out, bf16, c, v);
  }
}

// One (cos, sin) pair a thread.  Angles and their sine are taken in fp64: at a
// position of thousands an fp32 angle is off by more than the table's rounding.
struct TableArgs {
  float2* out;
  int G[3], n[3];
  double theta, start[3], step[3];
};
__global__ void rope_table_kernel(TableArgs a) {
  int i = blockIdx.x * blockDim.x + threadIdx.x;
#pragma unroll
  for (int ax = 0; ax < 3; ++ax) {
    const int m = a.G[ax] * a.n[ax];
    if (i < m) {
      const int pos = i / a.n[ax], j = i - pos * a.n[ax];
      const double f = pow(a.theta, -(double)j / (double)a.n[ax]);
      double s, c;
      sincos((a.start[ax] + a.step[ax] * pos) * f, &s, &c);
      a.out[i] = make_float2((float)c, (float)s);
      return;
    }
    i -= m;
    a.out += m;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

struct RopeDims {
  long long tokens;
  int heads[2];       // q, k
  long long pairs;
};

bool bad_factor(float f) { return !(f >= 0.f) || isinf(f); }

basa_status check_rope(const basa_rope_params* p, bool bwd, RopeDims* r) {
  if (!p) return BASA_ERR_INVALID_ARG;
  if (p->B < 0 || p->T < 0 || p->Hg < 0 || p->Wg < 0 || p->H < 0 || p->d <= 0)
    return BASA_ERR_INVALID_ARG;
  if (p->Hkv < 0 || (p->Hkv > 0 && p->H % p->Hkv != 0)) return BASA_ERR_INVALID_ARG;
  if (p->dtype != BASA_F32 && p->dtype != BASA_BF16)
    return p->dtype == BASA_FP8_E4M3 ? BASA_ERR_UNSUPPORTED : BASA_ERR_INVALID_ARG;
  if (p->out_dtype != p->dtype && (p->out_dtype != BASA_FP8_E4M3 || bwd))
    return p->out_dtype >= BASA_F32 && p->out_dtype <= BASA_FP8_E4M3 ? BASA_ERR_UNSUPPORTED
                                                                     : BASA_ERR_INVALID_ARG;
  if (p->w_dtype != BASA_F32 && p->w_dtype != BASA_BF16) return BASA_ERR_INVALID_ARG;
  if (p->layout != BASA_ROPE_PAIRS && p->layout != BASA_ROPE_HALVES) return BASA_ERR_INVALID_ARG;
  if (p->norm < BASA_ROPE_NORM_NONE || p->norm > BASA_ROPE_NORM_TOKEN) return BASA_ERR_INVALID_ARG;
  if (p->norm != BASA_ROPE_NORM_NONE && (!(p->eps > 0.f) || isinf(p->eps)))
    return BASA_ERR_INVALID_ARG;
  if (bad_factor(p->q_descale) || bad_factor(p->k_descale) || bad_factor(p->v_descale))
    return BASA_ERR_INVALID_ARG;
  if (p->at < 0 || p->ah < 0 || p->aw < 0 || ((p->at | p->ah | p->aw) & 1))
    return BASA_ERR_INVALID_ARG;
  if (p->d != 32 && p->d != 64 && p->d != 128) return BASA_ERR_UNSUPPORTED;
  const long long rot = (long long)p->at + p->ah + p->aw;
  if (rot > p->d) return BASA_ERR_INVALID_ARG;
  if (p->layout == BASA_ROPE_HALVES && rot % 16 != 0) return BASA_ERR_UNSUPPORTED;
  r->heads[0] = p->H;
  r->heads[1] = p->Hkv > 0 ? p->Hkv : p->H;
  if (p->H > 16384 || (p->norm == BASA_ROPE_NORM_TOKEN && (long long)p->H * p->d > 16384))
    return BASA_ERR_UNSUPPORTED;
  const int64_t in[3] = {p->ldq, p->ldk, p->ldv}, gr[3] = {p->ldgq, p->ldgk, p->ldgv};
  for (int i = 0; i < 3; ++i) {
    const long long row = (long long)r->heads[i > 0] * p->d;
    if (in[i] < 0 || gr[i] < 0 || (in[i] && in[i] < row) || (gr[i] && gr[i] < row))
      return BASA_ERR_INVALID_ARG;
    if (in[i] % 8 || gr[i] % 8) return BASA_ERR_ALIGN;
    if (in[i] > (1LL << 31) || gr[i] > (1LL << 31)) return BASA_ERR_UNSUPPORTED;
  }
  r->tokens = 1;
  const int32_t g[4] = {p->B, p->T, p->Hg, p->Wg};
  for (int i = 0; i < 4; ++i)
    if (g[i] == 0) r->tokens = 0;
  for (int i = 0; i < 4 && r->tokens; ++i) {
    r->tokens *= g[i];
    if (r->tokens > (1LL << 30)) return BASA_ERR_UNSUPPORTED;
  }
  r->pairs = (long long)p->T * (p->at / 2) + (long long)p->Hg * (p->ah / 2) +
             (long long)p->Wg * (p->aw / 2);
  if (r->pairs > (1LL << 30)) return BASA_ERR_UNSUPPORTED;
  return BASA_OK;
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Launch shape: CTAs along the tokens, and the chunks and steps of each part.
struct RopeGrid {
  unsigned x, y;
  int threads, v;
  int chunks[2], steps[2];
};

RopeGrid rope_grid(const basa_rope_params* p, const RopeDims& r, bool with_v, bool bwd) {
  RopeGrid g;
  const int sms = sm_count();
  if (p->norm == BASA_ROPE_NORM_TOKEN) {
    const int nvec = p->H * p->d / 8;  // H >= Hkv
    g.v = nvec <= 128 ? 1 : 4;
    g.threads = ((nvec + g.v - 1) / g.v + 31) / 32 * 32;
    g.chunks[0] = g.chunks[1] = 1;
    g.steps[0] = g.steps[1] = 0;
    g.y = with_v ? 3 : 2;
    const int per_sm = (bwd ? 640 : 1024) / g.threads;
    const long long cap = (long long)sms * (per_sm > 1 ? per_sm : 1);
    g.x = (unsigned)(r.tokens < cap ? r.tokens : cap);
    return g;
  }
  const int hpw = 32 / (p->d / 8);
  const int batch = bwd ? kRopeBwdBatch : kRopeBatch;
  g.threads = kRopeThreads;
  g.v = 0;
  g.y = 0;
  for (int i = 0; i < 2; ++i) {
    const int steps = (r.heads[i] + hpw - 1) / hpw;
    const int want = (steps + 3 * batch - 1) / (3 * batch);
    g.steps[i] = ((steps + want - 1) / want + batch - 1) / batch * batch;
    g.chunks[i] = (steps + g.steps[i] - 1) / g.steps[i];
  }
  g.y = g.chunks[0] + g.chunks[1] + (with_v ? g.chunks[1] : 0);
  const long long need = (r.tokens + kRopeWarps - 1) / kRopeWarps;
  const long long cap = (long long)sms * (bwd ? 4 : 16);
  g.x = (unsigned)(need < cap ? need : cap);
  return g;
}

size_t rope_part_bytes(const basa_rope_params* p, const RopeDims& r, const RopeGrid& g, int i) {
  const size_t cols = p->norm == BASA_ROPE_NORM_TOKEN ? (size_t)r.heads[i] * p->d : (size_t)p->d;
  return up256((size_t)g.x * g.chunks[i] * cols * sizeof(float));
}

template <typename TI, typename TO, int kLph>
void go_head(const RopeGrid& g, const RopeArgs& a, bool halves, bool norm, cudaStream_t st) {
  const dim3 grid(g.x, g.y);
  if (halves && norm) rope_head_kernel<TI, TO, kLph, true, true><<<grid, kRopeThreads, 0, st>>>(a);
  else if (halves) rope_head_kernel<TI, TO, kLph, true, false><<<grid, kRopeThreads, 0, st>>>(a);
  else if (norm) rope_head_kernel<TI, TO, kLph, false, true><<<grid, kRopeThreads, 0, st>>>(a);
  else rope_head_kernel<TI, TO, kLph, false, false><<<grid, kRopeThreads, 0, st>>>(a);
}
template <typename T, int kLph>
void go_head_bwd(const RopeGrid& g, const RopeArgs& a, bool halves, bool norm, cudaStream_t st) {
  const dim3 grid(g.x, g.y);
  if (halves && norm) rope_head_bwd_kernel<T, kLph, true, true><<<grid, kRopeThreads, 0, st>>>(a);
  else if (halves) rope_head_bwd_kernel<T, kLph, true, false><<<grid, kRopeThreads, 0, st>>>(a);
  else if (norm) rope_head_bwd_kernel<T, kLph, false, true><<<grid, kRopeThreads, 0, st>>>(a);
  else rope_head_bwd_kernel<T, kLph, false, false><<<grid, kRopeThreads, 0, st>>>(a);
}
template <typename TI, typename TO>
void go_fwd(const basa_rope_params* p, const RopeGrid& g, const RopeArgs& a, cudaStream_t st) {
  const bool halves = p->layout == BASA_ROPE_HALVES;
  if (p->norm == BASA_ROPE_NORM_TOKEN) {
    const dim3 grid(g.x, g.y);
    if (g.v == 1 && halves) rope_token_kernel<TI, TO, 1, true><<<grid, g.threads, 0, st>>>(a);
    else if (g.v == 1) rope_token_kernel<TI, TO, 1, false><<<grid, g.threads, 0, st>>>(a);
    else if (halves) rope_token_kernel<TI, TO, 4, true><<<grid, g.threads, 0, st>>>(a);
    else rope_token_kernel<TI, TO, 4, false><<<grid, g.threads, 0, st>>>(a);
    return;
  }
  const bool norm = p->norm != BASA_ROPE_NORM_NONE;
  if (p->d == 128) go_head<TI, TO, 16>(g, a, halves, norm, st);
  else if (p->d == 64) go_head<TI, TO, 8>(g, a, halves, norm, st);
  else go_head<TI, TO, 4>(g, a, halves, norm, st);
}
template <typename T>
void go_bwd(const basa_rope_params* p, const RopeGrid& g, const RopeArgs& a, cudaStream_t st) {
  const bool halves = p->layout == BASA_ROPE_HALVES;
  if (p->norm == BASA_ROPE_NORM_TOKEN) {
    const dim3 grid(g.x, g.y);
    if (g.v == 1 && halves) rope_token_bwd_kernel<T, 1, true><<<grid, g.threads, 0, st>>>(a);
    else if (g.v == 1) rope_token_bwd_kernel<T, 1, false><<<grid, g.threads, 0, st>>>(a);
    else if (halves) rope_token_bwd_kernel<T, 4, true><<<grid, g.threads, 0, st>>>(a);
    else rope_token_bwd_kernel<T, 4, false><<<grid, g.threads, 0, st>>>(a);
    return;
  }
  const bool norm = p->norm != BASA_ROPE_NORM_NONE;
  if (p->d == 128) go_head_bwd<T, 16>(g, a, halves, norm, st);
  else if (p->d == 64) go_head_bwd<T, 8>(g, a, halves, norm, st);
  else go_head_bwd<T, 4>(g, a, halves, norm, st);
}

RopeArgs rope_args(const basa_rope_params* p, const RopeDims& r, const RopeGrid& g,
                   const float* table, bool bwd) {
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  a.table = reinterpret_cast<const float2*>(table);
  a.tokens = (uint32_t)r.tokens;
  a.T = (uint32_t)p->T; a.Hg = (uint32_t)p->Hg; a.Wg = (uint32_t)p->Wg;
  a.nt = p->at / 2; a.nh = p->ah / 2; a.nw = p->aw / 2;
  a.d = p->d;
  a.eps = p->eps;
  a.w_bf16 = p->w_dtype == BASA_BF16;
  RopePart* part[3] = {&a.q, &a.k, &a.v};
  const int64_t in[3] = {p->ldq, p->ldk, p->ldv}, gr[3] = {p->ldgq, p->ldgk, p->ldgv};
  const float ds[3] = {p->q_descale, p->k_descale, p->v_descale};
  for (int i = 0; i < 3; ++i) {
    const int j = i > 0;
    const long long row = (long long)r.heads[j] * p->d;
    part[i]->heads = r.heads[j];
    part[i]->chunks = g.chunks[j];
    part[i]->steps = g.steps[j];
    part[i]->ldx = in[i] ? in[i] : row;
    part[i]->ldg = row;
    part[i]->ldo = bwd && gr[i] ? gr[i] : row;
    part[i]->mul = 1.f / (ds[i] > 0.f ? ds[i] : 1.f);
  }
  return a;
}

basa_status launched() { return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA; }

}  // namespace
}  // namespace basa

using namespace basa;

extern "C" {

int64_t basa_rope_table_pairs(const basa_rope_params* p) {
  RopeDims r;
  return check_rope(p, false, &r) == BASA_OK ? (int64_t)r.pairs : 0;
}

basa_status basa_rope_table(float* table, double theta, const double* start, const double* step,
                            const basa_rope_params* p, cudaStream_t stream) {
  NvtxRange nvtx("basa_rope_table");
  RopeDims r;
  basa_status s = check_rope(p, false, &r);
  if (s != BASA_OK) return s;
  if (!(theta > 0.0) || isinf(theta) || !start || !step) return BASA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (!isfinite(start[i]) || !isfinite(step[i])) return BASA_ERR_INVALID_ARG;
  if (r.pairs == 0) return BASA_OK;
  if (!table) return BASA_ERR_INVALID_ARG;
  if (off16(table)) return BASA_ERR_ALIGN;
  TableArgs a;
  a.out = reinterpret_cast<float2*>(table);
  const int G[3] = {p->T, p->Hg, p->Wg}, n[3] = {p->at / 2, p->ah / 2, p->aw / 2};
  for (int i = 0; i < 3; ++i) {
    a.G[i] = G[i];
    a.n[i] = n[i];
    a.start[i] = start[i];
    a.step[i] = step[i];
  }
  a.theta = theta;
  rope_table_kernel<<<(unsigned)((r.pairs + 127) / 128), 128, 0, stream>>>(a);
  return launched();
}

basa_status basa_qkv_rope(const void* q, const void* k, const void* v, const void* q_weight,
                          const void* k_weight, const float* table, void* q_out, void* k_out,
                          void* v_out, const basa_rope_params* p, cudaStream_t stream) {
  NvtxRange nvtx("basa_qkv_rope");
  RopeDims r;
  basa_status s = check_rope(p, false, &r);
  if (s != BASA_OK) return s;
  if (r.tokens * p->H == 0) return BASA_OK;
  if (!q || !k || !q_out || !k_out || (!v != !v_out) || (r.pairs && !table))
    return BASA_ERR_INVALID_ARG;
  if (p->norm == BASA_ROPE_NORM_NONE && (q_weight || k_weight)) return BASA_ERR_INVALID_ARG;
  if (off16(q) || off16(k) || off16(v) || off16(q_weight) || off16(k_weight) || off16(table) ||
      off16(q_out) || off16(k_out) || off16(v_out))
    return BASA_ERR_ALIGN;
  const RopeGrid g = rope_grid(p, r, v != nullptr, false);
  RopeArgs a = rope_args(p, r, g, table, false);
  a.q.x = q; a.k.x = k; a.v.x = v;
  a.q.w = q_weight; a.k.w = k_weight;
  a.q.o = q_out; a.k.o = k_out; a.v.o = v_out;
  const bool low = p->out_dtype == BASA_FP8_E4M3;
  if (p->dtype == BASA_BF16) {
    if (low) go_fwd<__nv_bfloat16, e4m3_t>(p, g, a, stream);
    else go_fwd<__nv_bfloat16, __nv_bfloat16>(p, g, a, stream);
  } else {
    if (low) go_fwd<float, e4m3_t>(p, g, a, stream);
    else go_fwd<float, float>(p, g, a, stream);
  }
  return launched();
}

size_t basa_qkv_rope_bwd_workspace_size(const basa_rope_params* p) {
  RopeDims r;
  if (check_rope(p, true, &r) != BASA_OK || p->norm == BASA_ROPE_NORM_NONE ||
      r.tokens * p->H == 0)
    return 0;
  const RopeGrid g = rope_grid(p, r, true, true);
  return rope_part_bytes(p, r, g, 0) + rope_part_bytes(p, r, g, 1);
}

basa_status basa_qkv_rope_bwd(const void* dq_out, const void* dk_out, const void* dv_out,
                              const void* q, const void* k, const void* q_weight,
                              const void* k_weight, const float* table, void* dq, void* dk,
                              void* dv, void* dq_weight, void* dk_weight, void* workspace,
                              const basa_rope_params* p, cudaStream_t stream) {
  NvtxRange nvtx("basa_qkv_rope_bwd");
  RopeDims r;
  basa_status s = check_rope(p, true, &r);
  if (s != BASA_OK) return s;
  const bool norm = p->norm != BASA_ROPE_NORM_NONE;
  if (!norm && (q_weight || k_weight)) return BASA_ERR_INVALID_ARG;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return BASA_ERR_INVALID_ARG;
  if (off16(q_weight) || off16(k_weight) || off16(dq_weight) || off16(dk_weight))
    return BASA_ERR_ALIGN;
  const bool token = p->norm == BASA_ROPE_NORM_TOKEN;
  const int cols[2] = {token ? r.heads[0] * p->d : p->d, token ? r.heads[1] * p->d : p->d};
  if (r.tokens * p->H == 0) {  // no rows: the weights' gradients are zero
    const size_t es = p->w_dtype == BASA_BF16 ? 2 : 4;
    if (dq_weight && cudaMemsetAsync(dq_weight, 0, cols[0] * es, stream) != cudaSuccess)
      return BASA_ERR_CUDA;
    if (dk_weight && cudaMemsetAsync(dk_weight, 0, cols[1] * es, stream) != cudaSuccess)
      return BASA_ERR_CUDA;
    return BASA_OK;
  }
  if (!dq_out || !dk_out || !dq || !dk || (!dv_out != !dv) || (r.pairs && !table) ||
      (norm && (!q || !k)))
    return BASA_ERR_INVALID_ARG;
  if (off16(dq_out) || off16(dk_out) || off16(dv_out) || off16(q) || off16(k) || off16(table) ||
      off16(dq) || off16(dk) || off16(dv))
    return BASA_ERR_ALIGN;
  const bool sums = dq_weight || dk_weight;
  if (sums && !workspace) return BASA_ERR_WORKSPACE;
  if (sums && off16(workspace)) return BASA_ERR_ALIGN;
  // the grid, and with it the order of the weights' sums, does not go by v
  RopeGrid g = rope_grid(p, r, true, true);
  if (!dv) g.y -= token ? 1 : g.chunks[1];
  RopeArgs a = rope_args(p, r, g, table, true);
  a.q.x = q; a.k.x = k;
  a.q.g = dq_out; a.k.g = dk_out; a.v.g = dv_out;
  a.q.w = q_weight; a.k.w = k_weight;
  a.q.o = dq; a.k.o = dk; a.v.o = dv;
  char* ws = static_cast<char*>(workspace);
  if (dq_weight) a.q.part = reinterpret_cast<float*>(ws);
  if (dk_weight) a.k.part = reinterpret_cast<float*>(ws + rope_part_bytes(p, r, g, 0));
  if (p->dtype == BASA_BF16)
    go_bwd<__nv_bfloat16>(p, g, a, stream);
  else
    go_bwd<float>(p, g, a, stream);
  if (sums) {
    const ColSum c0{a.q.part, dq_weight, (int)g.x * g.chunks[0], cols[0]};
    const ColSum c1{a.k.part, dk_weight, (int)g.x * g.chunks[1], cols[1]};
    rope_colsum_kernel<<<dim3((unsigned)(cols[0] / 8), 2), 256, 0, stream>>>(
        c0, c1, p->w_dtype == BASA_BF16);
  }
  return launched();
}

}  // extern "C"
