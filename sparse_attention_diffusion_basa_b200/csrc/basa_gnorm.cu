// The border between two blocks of a Diffusion Transformer (basa_gated_norm)
// and its backward (basa_gated_norm_bwd).  Per row of C values:
//   u  = y, or post-norm(y) * pw
//   x' = res_scale * x + gate * u
//   h  = (norm(x') * w + b) * (1 + scale) + shift
// with norm(z) = (z - mean) * rstd (layer) or z * rstd (rms, mean = 0).  Backward,
// with xh = norm(x'), yh = post-norm(y), gh and gx the gradients of h and x':
//   a  = gh (1 + scale) w
//   t  = gx + rstd (a - mean(a) - xh mean(a xh))         (rms: no mean(a))
//   dx = res_scale t,  e = gate pw t
//   dy = prstd (e - mean(e) - yh mean(e yh)),  without a post-norm dy = e
//   over the rows of a modulation: A = sum gh xh, S = sum gh, D = sum t yh
//   dscale = w A + b S, dshift = S, dgate = pw D
//   dw = sum (1 + scale) A, db = sum (1 + scale) S, dpw = sum gate D.
//
// Bound by HBM: every row is read and written once.  A CTA takes whole rows, each
// thread the same columns of every row; a CTA's rows are a contiguous range, so a
// modulation row's factors are formed once for many rows, and rows are read ahead
// by asynchronous copies.  Measured on a B200 (copy 6.57 TB/s), device time of the
// call: 75600 rows of 5120, fp32 stream and bf16 branch 787 to 801 us = 5.80 to 5.90
// TB/s (88 to 90% of the copy rate; the first form, unpacked and one row at a time,
// 1172); 14508 rows of 1536 bf16, both norms, a modulation a frame 40 us (68%; about
// 8 us of it start and end); backward of 16384 rows of 5120 bf16 188 us = 5.36 TB/s
// (82%; 273).  A modulation a token is far from that (16384 rows of 5120 bf16: 477 us
// for 179 us of bytes): each team's own factors pass through shared memory.
#include <math.h>
#include <string.h>

#include "row_device.cuh"

namespace basa {
namespace {

constexpr int kMaxC = 8192;
constexpr int kMaxWarps = 20;

struct GnArgs {
  const void *x, *y, *gate, *pw, *w, *b, *scale, *shift;
  void *xo, *h;
  float4* stats;
  // backward: gh and gx in the places of h's and x''s gradients
  const void *gh, *gx;
  const float4* st;
  void *dx, *dy, *dgate, *dscale, *dshift;
  float *part_g, *part_w;   // [grid][2][3][C], [grid][3][C]
  long long ld_gate, ld_scale, ld_shift;
  long long rows, group;    // rows of a modulation
  int C;
  int norm, post;
  float eps, post_eps, res, inv;
  int mod_bf16, w_bf16;
  int depth;                // stages of a read-ahead ring
  int need_y;
  // forward: warps that share a row, rows a CTA works on at a time
  int warps, teams;
  int direct;               // every team keeps the factors of its own row
  int wide;                 // fp32 outputs are aligned to 32 bytes
};

// Waits until at most depth - 1 of this thread's copies are in flight.
__device__ __forceinline__ void ring_wait(int depth) {
  if (depth == 3)
    copy_wait<2>();
  else if (depth == 2)
    copy_wait<1>();
  else
    copy_wait<0>();
}
__device__ __forceinline__ f2 both(float v) { return pk(v, v); }

// ---------------------------------------------------------------------------
// Sums over a row that a team of warps holds.  Every warp leaves its part in
// shared memory and, behind the team's barrier, adds up all parts in order.
// `buf` alternates from sum to sum, so that barrier is the only one.
// ---------------------------------------------------------------------------
struct Team {
  int warps, id;      // of this team
  int threads, tid;   // threads of the team, and this one's number among them
  int lane, warp;     // warp: its number in the team
  float4 (*red)[kMaxWarps];  // [2][warps of the CTA], at this team's first warp
  int buf;

  __device__ __forceinline__ void sync() const {
    if (warps == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
  }
  __device__ __forceinline__ float* next() {
    float* at = reinterpret_cast<float*>(red[buf]);
    buf ^= 1;
    return at;
  }
  // Two sums of one row, or of each of two rows.  Lanes that hold a sum's halves
  // of the warp keep one sum and hand on the others (six exchanges for four
  // sums); every warp then adds up the warps' parts, one a lane.
  __device__ __forceinline__ void sums(const float2 (&v)[1], float2 (&s)[1]) {
    const bool hi = lane & 16;
    float k = (hi ? v[0].y : v[0].x) + __shfl_xor_sync(0xffffffffu, hi ? v[0].x : v[0].y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
    float* at = next();
    if ((lane & 15) == 0) at[2 * warp + (lane >> 4)] = k;
    sync();
    k = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 32 * i < 2 * warps) k += at[lane + 32 * i];
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
    s[0].x = __shfl_sync(0xffffffffu, k, 0);
    s[0].y = __shfl_sync(0xffffffffu, k, 1);
  }
  __device__ __forceinline__ void sums(const float2 (&v)[2], float2 (&s)[2]) {
    const bool hi = lane & 16, mid = lane & 8;
    const float a = (hi ? v[1].x : v[0].x) + __shfl_xor_sync(0xffffffffu, hi ? v[0].x : v[1].x, 16);
    const float b = (hi ? v[1].y : v[0].y) + __shfl_xor_sync(0xffffffffu, hi ? v[0].y : v[1].y, 16);
    float k = (mid ? b : a) + __shfl_xor_sync(0xffffffffu, mid ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
    float* at = next();
    if ((lane & 7) == 0) at[4 * warp + (lane >> 3)] = k;
    sync();
    k = 0.f;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (lane + 32 * i < 4 * warps) k += at[lane + 32 * i];
#pragma unroll
    for (int o = 16; o > 2; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
    s[0].x = __shfl_sync(0xffffffffu, k, 0);
    s[0].y = __shfl_sync(0xffffffffu, k, 1);
    s[1].x = __shfl_sync(0xffffffffu, k, 2);
    s[1].y = __shfl_sync(0xffffffffu, k, 3);
  }
};
static_assert(kMaxWarps <= 24, "Team::sums reads three parts a lane");

// A modulation row's factors for the eight columns from `col`: gate * pw of the
// branch; (1 + scale) * w and (1 + scale) * b + shift of the norm.
__device__ __forceinline__ void gate8(const GnArgs& a, long long g, int col, f2 (&G)[4]) {
  f2 p[4];
  param8(a.gate, a.mod_bf16, g * a.ld_gate + col, 1.f, G);
  if (a.pw) {
    param8(a.pw, a.w_bf16, col, 1.f, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) G[i] = mul2(G[i], p[i]);
  }
}
__device__ __forceinline__ void scale8(const GnArgs& a, long long g, int col, f2 (&S)[4],
                                       f2 (&p)[4]) {
  param8(a.scale, a.mod_bf16, g * a.ld_scale + col, 0.f, p);
#pragma unroll
  for (int i = 0; i < 4; ++i) S[i] = p[i] = add2(p[i], both(1.f));
  if (a.w) {
    f2 w[4];
    param8(a.w, a.w_bf16, col, 1.f, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) S[i] = mul2(S[i], w[i]);
  }
}
__device__ __forceinline__ void affine8(const GnArgs& a, long long g, int col, f2 (&S)[4],
                                        f2 (&B)[4]) {
  f2 p[4];
  scale8(a, g, col, S, p);
  param8(a.shift, a.mod_bf16, g * a.ld_shift + col, 0.f, B);
  if (a.b) {
    f2 b[4];
    param8(a.b, a.w_bf16, col, 0.f, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) B[i] = fma2(b[i], p[i], B[i]);
  }
}
__device__ __forceinline__ void params_ahead(const GnArgs& a, long long g, int col) {
  ahead8(a.gate, a.mod_bf16, g * a.ld_gate + col);
  ahead8(a.pw, a.w_bf16, col);
  ahead8(a.scale, a.mod_bf16, g * a.ld_scale + col);
  ahead8(a.w, a.w_bf16, col);
  ahead8(a.shift, a.mod_bf16, g * a.ld_shift + col);
  ahead8(a.b, a.w_bf16, col);
}
// An array of fp32 factors in shared memory: two 16-byte pieces of a vector, the
// first pieces of all vectors and then the second ones, `half` bytes further.
// One more vector of zeros stands for all vectors past the row's end.
__host__ __device__ constexpr int factor_half(int nvec) { return (nvec + 1) * 16; }
// Stages begin at 128 bytes: a request of an asynchronous copy whose destination
// does not is split (measured: 1.5 times as many at the L2).
__host__ __device__ constexpr int up128(int x) { return (x + 127) & ~127; }
__device__ __forceinline__ void put8(char* at, int half, const f2 (&f)[4]) {
  *reinterpret_cast<ulonglong2*>(at) = make_ulonglong2(f[0], f[1]);
  *reinterpret_cast<ulonglong2*>(at + half) = make_ulonglong2(f[2], f[3]);
}
__device__ __forceinline__ void get8(const char* at, int half, f2 (&f)[4]) {
  const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(at),
                   y = *reinterpret_cast<const ulonglong2*>(at + half);
  f[0] = x.x;
  f[1] = x.y;
  f[2] = y.x;
  f[3] = y.y;
}
// A thread's columns of a row: vector j of eight at col(j), whether it is inside
// the row, and where its factors lie.  Vectors past the row's end are filled
// with zeros on the way in, have factors of zero, are computed with like the
// others (to zeros) and not stored, so the loops over a thread's vectors have no
// branches.  All of it is formed anew where it is used, from few registers: a
// spilled register costs far more than an addition in kernels whose shared
// memory leaves almost no L1.
struct Cols {
  int first, next, C;  // column of vector 0, from vector to vector, columns of a row
  __device__ __forceinline__ Cols(const Team& t, int C_)
      : first(t.tid * 8), next(t.threads * 8), C(C_) {}
  __device__ __forceinline__ int col(int j) const { return first + j * next; }
  __device__ __forceinline__ bool ok(int j) const { return col(j) < C; }
  __device__ __forceinline__ int at(int j) const { return min(col(j), C) * 2; }
};

// One tensor's part of a ring stage: a row's bytes as they lie in memory, up to
// the team's vectors.  bf16: a lane copies its own vectors.  fp32: a vector is
// two 16-byte pieces; the lanes of a warp copy consecutive pieces, not their
// own, so that a request covers whole lines (with a lane's own pieces, 32 bytes
// apart, the L2 sees one request for each piece).
template <typename T, int kV>
struct Part {
  static constexpr int kPieces = (int)sizeof(T) / 2;
  int first;  // element of the lane's first piece
  __device__ __forceinline__ explicit Part(const Team& t)
      : first(kPieces == 1 ? t.tid * 8 : t.warp * 256 + t.lane * 4) {}
  static __host__ __device__ constexpr int bytes(int threads) {
    return kV * threads * kPieces * 16;
  }
  __device__ __forceinline__ void fetch(uint32_t at, const T* row, const Cols& c,
                                        bool on = true) const {
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int e = first + j * c.next + p * 128;
        const bool in = e < c.C && on;
        copy16(at + e * (int)sizeof(T), row + (in ? e : 0), in);
      }
  }
  __device__ __forceinline__ void take(const char* at, int j, const Cols& c, f2 (&f)[4]) const {
    const uint4* s = reinterpret_cast<const uint4*>(at + c.col(j) * (int)sizeof(T));
    Raw8<T> r;
    r.a = s[0];
    if constexpr (kPieces == 2) r.b = s[1];
    widen8(r, f);
  }
};

__device__ __forceinline__ void put_row(__nv_bfloat16* p, const f2 (&f)[4], bool) { store8(p, f); }
// fp32: 32 bytes a lane in one store where the tensor is aligned to them, so
// that no request writes half a sector.
__device__ __forceinline__ void put_row(float* p, const f2 (&f)[4], bool wide) {
  if (wide)
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(f[0]), "l"(f[1]),
                 "l"(f[2]), "l"(f[3])
                 : "memory");
  else
    store8(p, f);
}

// Elements of a row in this warp.
__device__ __forceinline__ float elements_of(const Team& t, int kv, int nvec) {
  int n = 0;
  for (int j = 0; j < kv; ++j) {
    const int left = nvec - j * t.threads - 32 * t.warp;
    n += left < 0 ? 0 : left > 32 ? 32 : left;
  }
  return (float)(8 * n);
}

// (mean, rstd) of a row held kV * 8 values a thread, zeros past the row's end.
// Layer: the squares are taken about each warp's own mean and joined about the
// row's (Chan, Golub and LeVeque's update), so a mean far from zero costs no
// digits and one barrier is enough.  n, inv_n: elements of the warp.
template <int kV>
__device__ __forceinline__ float2 row_stats(const f2 (&f)[kV][4], const Cols& c, int kind,
                                            float eps, float inv, float n, float inv_n, Team& t) {
  f2 q0 = 0, q1 = 0;
  if (kind == BASA_NORM_LAYER) {
    f2 s0 = 0, s1 = 0;
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        s0 = add2(s0, f[j][i]);
        s1 = add2(s1, f[j][i + 1]);
      }
    const float m = lane_sum<32>(sum2(add2(s0, s1))) * inv_n;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const f2 mm = both(c.ok(j) ? -m : 0.f);
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const f2 a = add2(f[j][i], mm), b = add2(f[j][i + 1], mm);
        q0 = fma2(a, a, q0);
        q1 = fma2(b, b, q1);
      }
    }
    float q = lane_sum<32>(sum2(add2(q0, q1)));
    float mean = m;
    if (t.warps > 1) {  // at most eight
      float4* at = reinterpret_cast<float4*>(t.next());
      if (t.lane == 0) at[t.warp] = make_float4(m, q, n, 0.f);
      t.sync();
      const int i = t.lane & 7;
      const float4 w = i < t.warps ? at[i] : make_float4(0.f, 0.f, 0.f, 0.f);
      mean = lane_sum<8>(w.x * w.z) * inv;
      const float d = w.x - mean;
      q = lane_sum<8>(fmaf(w.z * d, d, w.y));
    }
    return make_float2(mean, rsqrtf(q * inv + eps));
  }
#pragma unroll
  for (int j = 0; j < kV; ++j)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      q0 = fma2(f[j][i], f[j][i], q0);
      q1 = fma2(f[j][i + 1], f[j][i + 1], q1);
    }
  float q = lane_sum<32>(sum2(add2(q0, q1)));
  if (t.warps > 1) {
    float* at = t.next();
    if (t.lane == 0) at[t.warp] = q;
    t.sync();
    const int i = t.lane & 7;
    q = lane_sum<8>(i < t.warps ? at[i] : 0.f);
  }
  return make_float2(0.f, rsqrtf(q * inv + eps));
}

// ---------------------------------------------------------------------------
// Forward.  One CTA an SM takes a contiguous range of rows, `teams` rows at a
// time, each in the registers of one team of warps: a row's own sums are a chain
// of exchanges that several rows at a time hide.  The factors of a modulation
// row are combined once, in fp32, into shared memory for all the teams (direct:
// a modulation covers too few rows for that, and each team keeps its own).
// One row at a time a CTA took 939 us for 75600 rows of 5120, teams 791; rows dealt
// to the CTAs in turn instead of in ranges the same there, and 61 us instead of 42
// for 14508 rows of 1536, where each CTA then meets every frame's factors.
// ---------------------------------------------------------------------------
constexpr int kFwdThreads = 512;  // 128 registers each

template <typename TX, typename TY, int kV, bool kBranch, bool kNorm>
__global__ void __launch_bounds__(kFwdThreads, 1)
    gnorm_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ __align__(128) char dyn[];
  __shared__ float4 red[2][kMaxWarps];
  const int nvec = a.C / 8;
  Team t;
  t.warps = a.warps;
  t.lane = threadIdx.x & 31;
  t.id = (threadIdx.x >> 5) / t.warps;
  t.warp = (threadIdx.x >> 5) - t.id * t.warps;
  t.threads = 32 * t.warps;
  t.tid = 32 * t.warp + t.lane;
  t.red = reinterpret_cast<float4(*)[kMaxWarps]>(&red[0][t.id * t.warps]);
  t.buf = 0;
  Cols c(t, a.C);
  Part<TX, kV> px(t);
  Part<TY, kV> py(t);
  const float n = elements_of(t, kV, nvec), inv_n = n > 0.f ? 1.f / n : 0.f;
  const int half = factor_half(nvec), arr = 2 * half;  // bytes of one array of factors
  const int factors = up128(((kBranch ? 1 : 0) + (kNorm ? 2 : 0)) * arr);
  char* const sG = dyn + (a.direct ? t.id * factors : 0);
  char* const sS = sG + (kBranch ? arr : 0);
  char* const sB = sS + (kNorm ? arr : 0);
  const int x_bytes = Part<TX, kV>::bytes(t.threads);
  const int stage = x_bytes + (kBranch ? Part<TY, kV>::bytes(t.threads) : 0);
  char* const ring = dyn + (a.direct ? a.teams : 1) * factors + t.id * a.depth * stage;
  const uint32_t ring_at = shared_u32(ring);
  const int r0 = (int)(a.rows * blockIdx.x / gridDim.x);
  const int r1 = (int)(a.rows * (blockIdx.x + 1) / gridDim.x);
  const long long off = (long long)(r0 + t.id) * a.C, skip = (long long)a.teams * a.C;
  const TX* x = static_cast<const TX*>(a.x) + off;
  const TY* y = kBranch ? static_cast<const TY*>(a.y) + off : nullptr;
  TX* xo = kBranch ? static_cast<TX*>(a.xo) + off : nullptr;
  TY* h = kNorm ? static_cast<TY*>(a.h) + off : nullptr;
  int ahead = r0 + t.id, at_stage = 0;
  auto fetch = [&](int to) {
    __syncwarp();  // every lane has read what the stage held
    if (ahead < r1) {
      px.fetch(ring_at + to, x, c);
      x += skip;
      if (kBranch) {
        py.fetch(ring_at + to + x_bytes, y, c);
        y += skip;
      }
      ahead += a.teams;
    }
    copy_commit();
  };
  auto fill = [&](long long g, int v) {
    f2 S[4] = {0, 0, 0, 0}, B[4] = {0, 0, 0, 0};
    if (v < nvec) params_ahead(a, g, v * 8);
    if (kBranch) {
      if (v < nvec) gate8(a, g, v * 8, S);
      put8(sG + v * 16, half, S);
    }
    if (kNorm) {
      if (v < nvec) affine8(a, g, v * 8, S, B);
      put8(sS + v * 16, half, S);
      put8(sB + v * 16, half, B);
    }
  };
  for (int s = 0; s < a.depth; ++s) fetch(s * stage);
  int r = r0 + t.id;
  for (int seg = r0; seg < r1;) {  // rows of one modulation, or, direct, all rows
    long long g = seg / a.group;
    int end = r1;
    if (!a.direct) {
      end = (int)min((long long)r1, (g + 1) * a.group);
      __syncthreads();
      for (int v = threadIdx.x; v <= nvec; v += blockDim.x) fill(g, v);
      __syncthreads();
    }
    g = -1;
    seg = end;
    for (; r < end; r += a.teams) {
      if (a.direct && r / a.group != g) {
        g = r / a.group;
        t.sync();  // the row before has been read
#pragma unroll 1
        for (int v = t.tid; v <= nvec; v += t.threads) fill(g, v);
        t.sync();
      }
      ring_wait(a.depth);
      __syncwarp();  // what the other lanes have copied
      c.first = anew(c.first);
      px.first = anew(px.first);
      py.first = anew(py.first);
      const char* at = ring + at_stage;
      f2 f[kV][4];
      float2 post = make_float2(0.f, 0.f), pre = make_float2(0.f, 0.f);
      if (kBranch) {
        f2 m = 0, s = both(1.f);
        if (a.post != BASA_NORM_NONE) {
#pragma unroll
          for (int j = 0; j < kV; ++j) py.take(at + x_bytes, j, c, f[j]);
          post = row_stats<kV>(f, c, a.post, a.post_eps, a.inv, n, inv_n, t);
          m = both(-post.x);
          s = both(post.y);
        }
        const f2 res = both(a.res);
        const bool plain = a.post == BASA_NORM_NONE && a.res == 1.f;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          f2 u[4], G[4];
          py.take(at + x_bytes, j, c, u);
          px.take(at, j, c, f[j]);
          get8(sG + c.at(j), half, G);
          if (plain) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[j][i] = fma2(u[i], G[i], f[j][i]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              f[j][i] = fma2(mul2(add2(u[i], m), s), G[i], mul2(res, f[j][i]));
          }
          if (c.ok(j)) put_row(xo + c.col(j), f[j], a.wide);
          one_by_one();
        }
        xo += skip;
      } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) px.take(at, j, c, f[j]);
      }
      fetch(at_stage);  // the row's elements are in registers, their stage is free
      at_stage = at_stage + stage == a.depth * stage ? 0 : at_stage + stage;
      if (kNorm) {
        pre = row_stats<kV>(f, c, a.norm, a.eps, a.inv, n, inv_n, t);
        const f2 m = both(-pre.x), s = both(pre.y);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          f2 S[4], B[4];
          get8(sS + c.at(j), half, S);
          get8(sB + c.at(j), half, B);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[j][i] = fma2(mul2(add2(f[j][i], m), s), S[i], B[i]);
          if (c.ok(j)) put_row(h + c.col(j), f[j], a.wide);
          one_by_one();
        }
        h += skip;
      }
      if (a.stats && t.tid == 0) a.stats[r] = make_float4(pre.x, pre.y, post.x, post.y);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  A CTA is one team and takes a contiguous range of rows, kR at a
// time; a thread's columns of the three sums over rows stay in registers.  Rows
// at a time share the factors read, the waits, the barriers and the addresses,
// and their chains of exchanges run side by side; of one modulation row's
// rows an odd last one has a row of zeros beside it.
// ---------------------------------------------------------------------------
template <int kV>
struct ColSums {
  f2 a[kV][4], s[kV][4], d[kV][4];  // gh xh, gh, t yh
};

// The sums of modulation row g end: into the result where all its rows lay in
// this CTA's range, into the CTA's partial rows otherwise; and, times the
// modulation, into the CTA's partial rows of the weights.
template <int kV, bool kBranch, bool kNorm>
__device__ __forceinline__ void flush(const GnArgs& a, const ColSums<kV>& c, long long g,
                                      bool whole, bool first, bool again) {
  float* pg = a.part_g + ((long long)blockIdx.x * 2 + (first ? 0 : 1)) * 3 * a.C;
  float* pw = a.part_w + (long long)blockIdx.x * 3 * a.C;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (col >= a.C) continue;
    f2 v[4], p[4], q[4];
    params_ahead(a, g, col);
    if (a.part_w) {
      auto add = [&](float* to, const f2(&sum)[4]) {
        f2 old[4];
        if (again) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 o = *reinterpret_cast<const float2*>(to + 2 * i);
            old[i] = pk(o.x, o.y);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = again ? fma2(p[i], sum[i], old[i]) : mul2(p[i], sum[i]);
        store8(to, v);
      };
      if (kNorm) {
        param8(a.scale, a.mod_bf16, g * a.ld_scale + col, 0.f, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = add2(p[i], both(1.f));
        add(pw + col, c.a[j]);
        add(pw + a.C + col, c.s[j]);
      }
      if (kBranch) {
        param8(a.gate, a.mod_bf16, g * a.ld_gate + col, 1.f, p);
        add(pw + 2 * a.C + col, c.d[j]);
      }
    }
    if (whole) {
      if (kNorm && a.dscale) {
        param8(a.w, a.w_bf16, col, 1.f, p);
        param8(a.b, a.w_bf16, col, 0.f, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fma2(p[i], c.a[j][i], mul2(q[i], c.s[j][i]));
        store_param8(a.dscale, a.mod_bf16, g * a.C + col, v);
      }
      if (kNorm && a.dshift) store_param8(a.dshift, a.mod_bf16, g * a.C + col, c.s[j]);
      if (kBranch && a.dgate) {
        param8(a.pw, a.w_bf16, col, 1.f, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(p[i], c.d[j][i]);
        store_param8(a.dgate, a.mod_bf16, g * a.C + col, v);
      }
    } else if (a.part_g) {
      if (kNorm) {
        store8(pg + col, c.a[j]);
        store8(pg + a.C + col, c.s[j]);
      }
      if (kBranch) store8(pg + 2 * a.C + col, c.d[j]);
    }
  }
}

template <typename TX, typename TY, int kV, int kR, int kThreads, bool kBranch, bool kNorm>
__global__ void __launch_bounds__(kThreads, 1)
    gnorm_bwd_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ __align__(128) char dyn[];
  __shared__ float4 red[2][kMaxWarps];
  const int nvec = a.C / 8;
  Team t;
  t.warps = blockDim.x >> 5;
  t.lane = threadIdx.x & 31;
  t.id = 0;
  t.warp = threadIdx.x >> 5;
  t.threads = blockDim.x;
  t.tid = threadIdx.x;
  t.red = red;
  t.buf = 0;
  Cols c(t, a.C);
  Part<TX, kV> lx(t);
  Part<TY, kV> ly(t);
  const int xb = Part<TX, kV>::bytes(t.threads), yb = Part<TY, kV>::bytes(t.threads);
  const int o_y = xb, o_x = o_y + (kBranch ? yb : 0), o_gh = o_x + xb;
  const int row_bytes = kNorm ? o_gh + yb : o_x, stage = kR * row_bytes;
  const int half = factor_half(nvec);
  char* const sG = dyn;
  char* const sS = sG + (kBranch ? 2 * half : 0);
  char* const ring = dyn + up128(4 * half);
  const uint32_t ring_at = shared_u32(ring);
  const int r0 = (int)(a.rows * blockIdx.x / gridDim.x);
  const int r1 = (int)(a.rows * (blockIdx.x + 1) / gridDim.x);
  const long long off = (long long)r0 * a.C;
  long long src = off;  // of the next row to fetch
  // gx and y may be absent: zeros, and the address of an output that is not read
  const bool have_gx = a.gx != nullptr, have_y = a.need_y;
  long long dst = off;  // of the rows at work
  long long g = r0 / a.group;
  int ahead = r0, ahead_end = (int)min((long long)r1, (g + 1) * a.group), at_stage = 0;
  auto fetch = [&](int to) {
    __syncwarp();  // every lane has read what the stage held
    if (ahead < r1) {
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        const uint32_t at = ring_at + to + k * row_bytes;
        const bool on = k == 0 || ahead + k < ahead_end;
        const long long e = src + (on ? k * a.C : 0);
        if (kNorm) {
          lx.fetch(at + o_x, static_cast<const TX*>(a.x) + e, c, on);
          ly.fetch(at + o_gh, static_cast<const TY*>(a.gh) + e, c, on);
        }
        lx.fetch(at, static_cast<const TX*>(have_gx ? a.gx : a.dx) + e, c, on && have_gx);
        if (kBranch)
          ly.fetch(at + o_y, static_cast<const TY*>(have_y ? a.y : a.dy) + e, c, on && have_y);
      }
      const int rows = min(kR, ahead_end - ahead);
      src += rows * a.C;
      ahead += rows;
      if (ahead == ahead_end) ahead_end = (int)min((long long)r1, ahead + a.group);
    }
    copy_commit();
  };
  const int first_end = ahead_end;
  for (int s = 0; s < a.depth; ++s) fetch(s * stage);
  ColSums<kV> sum;
  int end = r0;
  const long long g_first = g;
  bool flushed = false;
  float4 st_next[kR];
  // Of the rows from r on, ahead of their use; zeros beside an odd last row of a
  // modulation (end: of its rows), not the next one's statistics, which may not be
  // finite and would reach this one's sums as 0 * NaN.
  auto stats_of = [&](int r, int end) {
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      st_next[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.st && r + k < (k ? end : r1)) st_next[k] = __ldg(a.st + r + k);
    }
  };
  stats_of(r0, first_end);
  for (int r = r0;;) {
    if (r == end) {
      if (r > r0) {
        flush<kV, kBranch, kNorm>(a, sum, g, g * a.group >= r0 && (g + 1) * a.group <= r,
                                  g == g_first, flushed);
        flushed = true;
      }
      if (r == r1) break;
      if (r1 - r <= a.group) dependents_may_start();
      g = r / a.group;
      end = (int)min((long long)r1, (g + 1) * a.group);
#pragma unroll
      for (int j = 0; j < kV; ++j) {  // each thread reads the factors that it writes
        f2 p[4] = {0, 0, 0, 0}, q[4];
        if (c.ok(j)) params_ahead(a, g, c.col(j));
        if (kBranch) {
          if (c.ok(j)) gate8(a, g, c.col(j), p);
          put8(sG + c.at(j), half, p);
        }
        if (kNorm) {
          if (c.ok(j)) scale8(a, g, c.col(j), p, q);
          put8(sS + c.at(j), half, p);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum.a[j][i] = sum.s[j][i] = sum.d[j][i] = 0;
      }
    }
    float4 st[kR];
    bool on[kR];
    int rows = 0;
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      on[k] = r + k < end;
      rows += on[k] ? 1 : 0;
      st[k] = st_next[k];
    }
    stats_of(r + rows, r + rows < end ? end : (int)min((long long)r1, r + rows + a.group));
    ring_wait(a.depth);
    __syncwarp();  // what the other lanes have copied
    c.first = anew(c.first);
    lx.first = anew(lx.first);
    ly.first = anew(ly.first);
    const char* at = ring + at_stage;
    f2 xh[kR][kV][4], v[kR][kV][4];  // xh; a, then t, then e
    float2 c12[kR];
    if (kNorm) {
      float2 part[kR];
      f2 s1[kR], s2[kR];
#pragma unroll
      for (int k = 0; k < kR; ++k) s1[k] = s2[k] = 0;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        f2 S[4];
        get8(sS + c.at(j), half, S);
#pragma unroll
        for (int k = 0; k < kR; ++k) {
          const f2 m = both(-st[k].x), s = both(st[k].y);
          lx.take(at + k * row_bytes + o_x, j, c, xh[k][j]);
          ly.take(at + k * row_bytes + o_gh, j, c, v[k][j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xh[k][j][i] = mul2(add2(xh[k][j][i], m), s);
            sum.a[j][i] = fma2(v[k][j][i], xh[k][j][i], sum.a[j][i]);
            sum.s[j][i] = add2(sum.s[j][i], v[k][j][i]);
            v[k][j][i] = mul2(v[k][j][i], S[i]);
            s1[k] = add2(s1[k], v[k][j][i]);
            s2[k] = fma2(v[k][j][i], xh[k][j][i], s2[k]);
          }
          one_by_one();
        }
      }
#pragma unroll
      for (int k = 0; k < kR; ++k) part[k] = make_float2(sum2(s1[k]), sum2(s2[k]));
      t.sums(part, c12);
    }
    f2 c1[kR], c2[kR], sk[kR];
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      if (!kNorm) c12[k] = make_float2(0.f, 0.f);
      c1[k] = both(a.norm == BASA_NORM_LAYER ? -c12[k].x * a.inv : 0.f);
      c2[k] = both(-c12[k].y * a.inv);
      sk[k] = both(st[k].y);
    }
    f2 s1[kR], s2[kR];
#pragma unroll
    for (int k = 0; k < kR; ++k) s1[k] = s2[k] = 0;
    const f2 res = both(a.res);
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      f2 G[4];
      if (kBranch) get8(sG + c.at(j), half, G);
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        const char* row = at + k * row_bytes;
        f2 gx[4];
        lx.take(row, j, c, gx);
        if (kNorm) {  // rstd (a - mean(a) - xh mean(a xh)) + gx
#pragma unroll
          for (int i = 0; i < 4; ++i)
            gx[i] = fma2(sk[k], fma2(xh[k][j][i], c2[k], add2(v[k][j][i], c1[k])), gx[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][j][i] = mul2(res, gx[i]);
        if (c.ok(j) && on[k]) put_row(static_cast<TX*>(a.dx) + dst + k * a.C + c.col(j), v[k][j], a.wide);
        if (kBranch) {
          f2 yh[4];
          ly.take(row + o_y, j, c, yh);
          if (a.post == BASA_NORM_NONE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sum.d[j][i] = fma2(gx[i], yh[i], sum.d[j][i]);
              v[k][j][i] = mul2(gx[i], G[i]);
            }
            if (c.ok(j) && on[k]) put_row(static_cast<TY*>(a.dy) + dst + k * a.C + c.col(j), v[k][j], a.wide);
          } else {
            const f2 pm = both(-st[k].z), ps = both(st[k].w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              yh[i] = mul2(add2(yh[i], pm), ps);
              sum.d[j][i] = fma2(gx[i], yh[i], sum.d[j][i]);
              v[k][j][i] = mul2(gx[i], G[i]);
              s1[k] = add2(s1[k], v[k][j][i]);
              s2[k] = fma2(v[k][j][i], yh[i], s2[k]);
            }
          }
        }
        one_by_one();
      }
    }
    if (kBranch && a.post != BASA_NORM_NONE) {
      float2 part[kR];
#pragma unroll
      for (int k = 0; k < kR; ++k) part[k] = make_float2(sum2(s1[k]), sum2(s2[k]));
      t.sums(part, c12);
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        const f2 pm = both(-st[k].z), ps = both(st[k].w);
        const f2 c1 = both(a.post == BASA_NORM_LAYER ? -c12[k].x * a.inv : 0.f),
                 c2 = both(-c12[k].y * a.inv);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          f2 yh[4];
          ly.take(at + k * row_bytes + o_y, j, c, yh);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[k][j][i] = mul2(ps, fma2(mul2(add2(yh[i], pm), ps), c2, add2(v[k][j][i], c1)));
          if (c.ok(j) && on[k]) put_row(static_cast<TY*>(a.dy) + dst + k * a.C + c.col(j), v[k][j], a.wide);
        }
      }
    }
    fetch(at_stage);
    at_stage = at_stage + stage == a.depth * stage ? 0 : at_stage + stage;
    dst += rows * a.C;
    r += rows;
  }
}

// Joins the partial sums of gnorm_bwd_kernel.  A CTA owns eight columns and
// reads 32 partial rows side by side, joined in a fixed order, so equal calls give
// equal bits.  It reads a few MB that still lie in the L2 (8 us cold for 16384 rows of
// 5120) and is launched while the rows' kernel ends.  blockIdx.z = 0:
// the modulation rows whose tokens span several CTAs; blockIdx.y is the
// modulation row, or, where there are more of those than CTAs, the CTA in which
// the row begins (each CTA's range splits at most one that goes on behind it).
// blockIdx.z = 1: the weights, over every CTA.
struct GnJoin {
  const float *part_g, *part_w;
  const void *w, *b, *pw;
  void *dgate, *dscale, *dshift, *dw, *db, *dpw;
  long long rows, group, groups;
  int C, grid, by_group;
  int mod_bf16, w_bf16;
};
__global__ void __launch_bounds__(256) gnorm_join_kernel(GnJoin a) {
  __shared__ float red[3][32][9];
  wait_for_partial_sums();
  const int k = threadIdx.x & 7, lane = threadIdx.x >> 3;
  const int c = blockIdx.x * 8 + k;
  float v[3] = {0.f, 0.f, 0.f};
  long long g = 0;
  if (blockIdx.z == 0) {
    if (!a.part_g) return;
    if (a.by_group) {
      g = blockIdx.y;
    } else {  // the row that holds this CTA's last token
      const long long last = a.rows * (blockIdx.y + 1) / a.grid - 1;
      g = last / a.group;
      if (g * a.group < a.rows * blockIdx.y / a.grid) return;  // began in an earlier CTA
    }
    const long long lo = ((g * a.group + 1) * a.grid - 1) / a.rows;
    const long long hi = ((g + 1) * a.group * a.grid - 1) / a.rows;
    if (lo == hi) return;  // inside one CTA, which has written the result
    // a CTA behind the first one begins inside this row of modulations, so its
    // sums are the CTA's first; in the first one they may be its last
    const bool whole = a.rows * lo / a.grid / a.group == g;
#pragma unroll 4
    for (int i = (int)lo + lane; i <= (int)hi; i += 32) {
      const float* p = a.part_g + (i * 2 + (i == (int)lo && !whole ? 1 : 0)) * 3LL * a.C + c;
#pragma unroll
      for (int s = 0; s < 3; ++s) v[s] += p[s * a.C];
    }
  } else {
    if (blockIdx.y || !a.part_w) return;
#pragma unroll 4
    for (int i = lane; i < a.grid; i += 32) {
      const float* p = a.part_w + (long long)i * 3 * a.C + c;
#pragma unroll
      for (int s = 0; s < 3; ++s) v[s] += p[s * a.C];
    }
  }
#pragma unroll
  for (int s = 0; s < 3; ++s) red[s][lane][k] = v[s];
  __syncthreads();
  if (threadIdx.x >= 24) return;
  const int s = threadIdx.x >> 3;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) t += red[s][i][k];
  if (blockIdx.z) {
    void* o = s == 0 ? a.dw : s == 1 ? a.db : a.dpw;
    if (o) store_param(o, a.w_bf16, c, t);
    return;
  }
  auto param = [&](const void* p, float fill) {
    return !p ? fill
              : a.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c])
                         : static_cast<const float*>(p)[c];
  };
  if (s == 0 && a.dscale) {
    float u = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) u += red[1][i][k];
    store_param(a.dscale, a.mod_bf16, g * a.C + c, fmaf(param(a.w, 1.f), t, param(a.b, 0.f) * u));
  }
  if (s == 1 && a.dshift) store_param(a.dshift, a.mod_bf16, g * a.C + c, t);
  if (s == 2 && a.dgate) store_param(a.dgate, a.mod_bf16, g * a.C + c, param(a.pw, 1.f) * t);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
int round32(int x) { return (x + 31) / 32 * 32; }

basa_status check_gnorm(const basa_gnorm_params* p) {
  if (!p || p->rows < 0 || p->C <= 0 || p->groups < 1) return BASA_ERR_INVALID_ARG;
  if (p->norm < BASA_NORM_NONE || p->norm > BASA_NORM_RMS || p->post_norm < BASA_NORM_NONE ||
      p->post_norm > BASA_NORM_RMS)
    return BASA_ERR_INVALID_ARG;
  if (p->norm != BASA_NORM_NONE && (!(p->eps > 0.f) || isinf(p->eps))) return BASA_ERR_INVALID_ARG;
  if (p->post_norm != BASA_NORM_NONE && (!(p->post_eps > 0.f) || isinf(p->post_eps)))
    return BASA_ERR_INVALID_ARG;
  if (!isfinite(p->res_scale)) return BASA_ERR_INVALID_ARG;
  const int32_t ty[4] = {p->x_dtype, p->dtype, p->mod_dtype, p->w_dtype};
  for (int i = 0; i < 4; ++i)
    if (ty[i] != BASA_F32 && ty[i] != BASA_BF16)
      return ty[i] == BASA_FP8_E4M3 ? BASA_ERR_UNSUPPORTED : BASA_ERR_INVALID_ARG;
  if (p->x_dtype == BASA_BF16 && p->dtype == BASA_F32) return BASA_ERR_UNSUPPORTED;
  if (p->rows % p->groups) return BASA_ERR_SHAPE;
  if (p->C % 8 || p->C > kMaxC || p->rows > (1LL << 30) || p->groups > (1LL << 30))
    return BASA_ERR_UNSUPPORTED;
  const int64_t ld[3] = {p->ld_gate, p->ld_scale, p->ld_shift};
  for (int i = 0; i < 3; ++i) {
    if (ld[i] < 0) return BASA_ERR_INVALID_ARG;
    if (ld[i] % 8) return BASA_ERR_ALIGN;
    if (ld[i] > (1LL << 31)) return BASA_ERR_UNSUPPORTED;
  }
  return BASA_OK;
}

// Bytes of the border's tensors, and the inputs that its two directions share.
struct GnBytes {
  long long x, y, m, w, groups;  // of the rows, of a modulation row, of a weight
  long long ld[3];
  explicit GnBytes(const basa_gnorm_params* p) {
    auto es = [](int t) { return t == BASA_BF16 ? 2LL : 4LL; };
    x = p->rows * p->C * es(p->x_dtype);
    y = p->rows * p->C * es(p->dtype);
    m = p->C * es(p->mod_dtype);
    w = p->C * es(p->w_dtype);
    groups = p->groups;
    const int64_t l[3] = {p->ld_gate, p->ld_scale, p->ld_shift};
    for (int i = 0; i < 3; ++i) ld[i] = l[i] * es(p->mod_dtype);
  }
  void mod(Overlap& o, const void* p, int i) const { o.in(p, ld[i] ? groups : 1, m, ld[i]); }
};

GnArgs gnorm_args(const basa_gnorm_params* p) {
  GnArgs a;
  memset(&a, 0, sizeof(a));
  a.ld_gate = p->ld_gate; a.ld_scale = p->ld_scale; a.ld_shift = p->ld_shift;
  a.rows = p->rows;
  a.group = p->rows / p->groups;
  a.C = p->C;
  a.norm = p->norm; a.post = p->post_norm;
  a.eps = p->eps; a.post_eps = p->post_eps; a.res = p->res_scale;
  a.inv = 1.f / (float)p->C;
  a.mod_bf16 = p->mod_dtype == BASA_BF16;
  a.w_bf16 = p->w_dtype == BASA_BF16;
  return a;
}

template <typename K>
basa_status go(K kernel, const GnArgs& a, unsigned grid, int threads, int smem, cudaStream_t st) {
  if (!allow_smem(kernel, smem)) return BASA_ERR_CUDA;
  kernel<<<grid, threads, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

template <typename TX, typename TY, int kV>
basa_status go_fwd_v(GnArgs a, cudaStream_t st) {
  const bool branch = a.y != nullptr, norm = a.norm != BASA_NORM_NONE;
  const int per_row = 32 * a.warps;
  const int stage = Part<TX, kV>::bytes(per_row) + (branch ? Part<TY, kV>::bytes(per_row) : 0);
  const int sms = row_sm_count();
  const unsigned grid = (unsigned)(a.rows < sms ? a.rows : sms);
  const long long most = (a.rows + grid - 1) / grid;  // rows of a CTA
  const int factors = up128(((branch ? 1 : 0) + (norm ? 2 : 0)) * 2 * factor_half(a.C / 8));
  a.teams = kFwdThreads / per_row;
  if (a.warps > 1 && a.teams > 15) a.teams = 15;  // barriers of a CTA
  if (a.teams > most) a.teams = (int)most;
  a.direct = a.group < 4 * a.teams;
  // shared memory: the factors, once or for each team, and a ring for each team
  const int fit = a.direct ? kMostSmem / (factors + stage) : (kMostSmem - factors) / stage;
  if (a.teams > fit) a.teams = fit;
  const int held = a.direct ? a.teams * factors : factors;
  a.depth = (kMostSmem - held) / (a.teams * stage);
  if (a.depth > 3) a.depth = 3;
  const int smem = held + a.teams * a.depth * stage, threads = a.teams * per_row;
  if (branch && norm) return go(gnorm_kernel<TX, TY, kV, true, true>, a, grid, threads, smem, st);
  if (branch) return go(gnorm_kernel<TX, TY, kV, true, false>, a, grid, threads, smem, st);
  return go(gnorm_kernel<TX, TY, kV, false, true>, a, grid, threads, smem, st);
}
template <typename TX, typename TY>
basa_status go_fwd(GnArgs a, cudaStream_t st) {
  const int nvec = a.C / 8;
  a.warps = (nvec + 159) / 160;
  const int v = (nvec + 32 * a.warps - 1) / (32 * a.warps);
  return v == 5   ? go_fwd_v<TX, TY, 5>(a, st)
         : v == 4 ? go_fwd_v<TX, TY, 4>(a, st)
         : v == 3 ? go_fwd_v<TX, TY, 3>(a, st)
         : v == 2 ? go_fwd_v<TX, TY, 2>(a, st)
                  : go_fwd_v<TX, TY, 1>(a, st);
}

// Launch shape of the backward.  Up to 640 threads, one vector and two rows a
// thread; wider rows, of more than 5120 columns, two vectors and one row.  At
// 16384 rows of 5120 bf16 columns: one vector and two rows 189 us, two vectors
// and two rows (half the warps) 199, one and one 215.
struct BwdShape {
  int v, threads, per_sm, bytes;  // bytes: shared memory beside the ring
  long long grid;
};
BwdShape bwd_shape(const basa_gnorm_params* p) {
  BwdShape s;
  const int nvec = p->C / 8, most = nvec <= 640 ? 640 : 512;
  s.v = nvec <= 640 ? 1 : 2;
  s.threads = round32((nvec + s.v - 1) / s.v);
  s.bytes = up128(4 * factor_half(nvec));
  const int sx = p->x_dtype == BASA_BF16 ? 2 : 4, sy = p->dtype == BASA_BF16 ? 2 : 4;
  const int stage = 2 * s.threads * 8 * 2 * (sx + sy);  // 1 x 2 or 2 x 1 vectors of four rows
  s.per_sm = most / s.threads;
  if (s.per_sm > kMostSmem / (s.bytes + stage + 2048)) s.per_sm = kMostSmem / (s.bytes + stage + 2048);
  if (s.per_sm > 8) s.per_sm = 8;
  if (s.per_sm < 1) s.per_sm = 1;
  long long cap = (long long)row_sm_count() * s.per_sm;
  const long long few = (p->rows + 3) / 4;  // at least four rows a CTA
  if (cap > few) cap = few;
  s.grid = cap < 1 ? 1 : cap;
  return s;
}
size_t part_g_bytes(const basa_gnorm_params* p, const BwdShape& s) {
  return up256((size_t)s.grid * 6 * p->C * sizeof(float));
}
size_t part_w_bytes(const basa_gnorm_params* p, const BwdShape& s) {
  return up256((size_t)s.grid * 3 * p->C * sizeof(float));
}

template <typename TX, typename TY, int kV, int kR, int kThreads>
basa_status go_bwd_t(GnArgs a, const BwdShape& s, cudaStream_t st) {
  const bool branch = a.dy != nullptr, norm = a.norm != BASA_NORM_NONE;
  const int xb = Part<TX, kV>::bytes(s.threads), yb = Part<TY, kV>::bytes(s.threads);
  const int stage = kR * (xb + (branch ? yb : 0) + (norm ? xb + yb : 0));
  a.depth = (kMostSmem / s.per_sm - 2048 - s.bytes) / stage;
  a.depth = a.depth > 3 ? 3 : a.depth < 1 ? 1 : a.depth;
  const int smem = s.bytes + a.depth * stage;
  const unsigned grid = (unsigned)s.grid;
  if (branch && norm)
    return go(gnorm_bwd_kernel<TX, TY, kV, kR, kThreads, true, true>, a, grid, s.threads, smem, st);
  if (branch)
    return go(gnorm_bwd_kernel<TX, TY, kV, kR, kThreads, true, false>, a, grid, s.threads, smem,
              st);
  return go(gnorm_bwd_kernel<TX, TY, kV, kR, kThreads, false, true>, a, grid, s.threads, smem, st);
}
template <typename TX, typename TY>
basa_status go_bwd(const GnArgs& a, const BwdShape& s, cudaStream_t st) {
  return s.v == 1 ? go_bwd_t<TX, TY, 1, 2, 640>(a, s, st) : go_bwd_t<TX, TY, 2, 1, 512>(a, s, st);
}

}  // namespace
}  // namespace basa

using namespace basa;

extern "C" {

basa_status basa_gated_norm(const void* x, const void* y, const void* gate, const void* post_weight,
                            const void* weight, const void* bias, const void* scale,
                            const void* shift, void* x_out, void* h, float* stats,
                            const basa_gnorm_params* p, cudaStream_t stream) {
  NvtxRange nvtx("basa_gated_norm");
  basa_status s = check_gnorm(p);
  if (s != BASA_OK) return s;
  const bool norm = p->norm != BASA_NORM_NONE, post = p->post_norm != BASA_NORM_NONE;
  if (!norm && (h || weight || bias || scale || shift)) return BASA_ERR_INVALID_ARG;
  if (!post && post_weight) return BASA_ERR_INVALID_ARG;
  if (p->rows == 0) return BASA_OK;
  if (!x || (!y && (gate || post || x_out || !norm)) || (y && !x_out) || (norm && !h))
    return BASA_ERR_INVALID_ARG;
  if (off16(x) || off16(y) || off16(gate) || off16(post_weight) || off16(weight) || off16(bias) ||
      off16(scale) || off16(shift) || off16(x_out) || off16(h) || off16(stats))
    return BASA_ERR_ALIGN;
  {
    Overlap o;
    const GnBytes n(p);
    o.in(x, n.x);
    o.in(y, n.y);
    n.mod(o, gate, 0);
    n.mod(o, scale, 1);
    n.mod(o, shift, 2);
    for (const void* w : {post_weight, weight, bias}) o.in(w, n.w);
    o.out(x_out, n.x, x);
    o.out(h, n.y, y);
    o.out(stats, p->rows * 16);
    if (o.any()) return BASA_ERR_INVALID_ARG;
  }
  GnArgs a = gnorm_args(p);
  a.x = x; a.y = y; a.gate = gate; a.pw = post_weight;
  a.w = weight; a.b = bias; a.scale = scale; a.shift = shift;
  a.xo = x_out; a.h = h;
  a.stats = reinterpret_cast<float4*>(stats);
  a.wide = aligned32(x_out) && aligned32(h);
  if (p->x_dtype == BASA_BF16) return go_fwd<__nv_bfloat16, __nv_bfloat16>(a, stream);
  if (p->dtype == BASA_BF16) return go_fwd<float, __nv_bfloat16>(a, stream);
  return go_fwd<float, float>(a, stream);
}

size_t basa_gated_norm_bwd_workspace_size(const basa_gnorm_params* p) {
  if (check_gnorm(p) != BASA_OK || p->rows == 0) return 0;
  const BwdShape s = bwd_shape(p);
  return part_g_bytes(p, s) + part_w_bytes(p, s);
}

basa_status basa_gated_norm_bwd(const void* dh, const void* x_out, const float* stats,
                                const void* y, const void* dx_out, const void* gate,
                                const void* post_weight, const void* weight, const void* bias,
                                const void* scale, void* dx, void* dy, void* dgate,
                                void* dpost_weight, void* dweight, void* dbias, void* dscale,
                                void* dshift, void* workspace, const basa_gnorm_params* p,
                                cudaStream_t stream) {
  NvtxRange nvtx("basa_gated_norm_bwd");
  basa_status s = check_gnorm(p);
  if (s != BASA_OK) return s;
  const bool norm = p->norm != BASA_NORM_NONE, post = p->post_norm != BASA_NORM_NONE;
  if (!norm && (weight || bias || scale || dweight || dbias || dscale || dshift))
    return BASA_ERR_INVALID_ARG;
  if ((post_weight && !post) || (dpost_weight && !post_weight) || (dgate && !gate) ||
      (dweight && !weight) || (dbias && !bias) || (dscale && !scale))
    return BASA_ERR_INVALID_ARG;
  if (off16(gate) || off16(post_weight) || off16(weight) || off16(bias) || off16(scale) ||
      off16(dgate) || off16(dpost_weight) || off16(dweight) || off16(dbias) || off16(dscale) ||
      off16(dshift))
    return BASA_ERR_ALIGN;
  if (p->rows == 0) {  // no rows: the sums over rows are zero
    const size_t me = p->mod_dtype == BASA_BF16 ? 2 : 4, we = p->w_dtype == BASA_BF16 ? 2 : 4;
    void* mods[3] = {dgate, dscale, dshift};
    void* ws[3] = {dpost_weight, dweight, dbias};
    for (int i = 0; i < 3; ++i) {
      if (mods[i] && cudaMemsetAsync(mods[i], 0, (size_t)p->groups * p->C * me, stream) != cudaSuccess)
        return BASA_ERR_CUDA;
      if (ws[i] && cudaMemsetAsync(ws[i], 0, (size_t)p->C * we, stream) != cudaSuccess)
        return BASA_ERR_CUDA;
    }
    return BASA_OK;
  }
  const bool need_y = post || dgate;
  if (!dx || (norm ? !dh || !x_out || !stats : !dx_out || !dy) || (post && (!stats || !dy)) ||
      (!dy && (gate || post)) || (need_y && !y))
    return BASA_ERR_INVALID_ARG;
  if (off16(dh) || off16(x_out) || off16(stats) || off16(y) || off16(dx_out) || off16(dx) ||
      off16(dy))
    return BASA_ERR_ALIGN;
  const bool mods = dgate || dscale || dshift, weights = dpost_weight || dweight || dbias;
  if ((mods || weights) && !workspace) return BASA_ERR_WORKSPACE;
  if ((mods || weights) && off16(workspace)) return BASA_ERR_ALIGN;
  const BwdShape sh = bwd_shape(p);
  {
    Overlap o;
    const GnBytes n(p);
    o.in(dx_out, n.x);
    if (norm) o.in(dh, n.y);
    if (norm) o.in(x_out, n.x);
    if (norm || post) o.in(stats, p->rows * 16);
    if (need_y) o.in(y, n.y);
    n.mod(o, gate, 0);
    n.mod(o, scale, 1);
    for (const void* w : {post_weight, weight, bias}) o.in(w, n.w);
    o.out(dx, n.x, dx_out);
    o.out(dy, n.y);
    for (void* m : {dgate, dscale, dshift}) o.out(m, n.groups * n.m);
    for (void* w : {dpost_weight, dweight, dbias}) o.out(w, n.w);
    if (mods || weights) o.out(workspace, (long long)(part_g_bytes(p, sh) + part_w_bytes(p, sh)));
    if (o.any()) return BASA_ERR_INVALID_ARG;
  }
  GnArgs a = gnorm_args(p);
  a.x = x_out; a.y = y; a.gate = gate; a.pw = post_weight;
  a.w = weight; a.b = bias; a.scale = scale;
  a.gh = dh; a.gx = dx_out;
  a.st = reinterpret_cast<const float4*>(stats);
  a.dx = dx; a.dy = dy;
  a.dgate = dgate; a.dscale = dscale; a.dshift = dshift;
  a.need_y = need_y;
  a.wide = aligned32(dx) && aligned32(dy);
  char* ws = static_cast<char*>(workspace);
  if (mods) a.part_g = reinterpret_cast<float*>(ws);
  if (weights) a.part_w = reinterpret_cast<float*>(ws + part_g_bytes(p, sh));
  if (p->x_dtype == BASA_BF16) s = go_bwd<__nv_bfloat16, __nv_bfloat16>(a, sh, stream);
  else if (p->dtype == BASA_BF16) s = go_bwd<float, __nv_bfloat16>(a, sh, stream);
  else s = go_bwd<float, float>(a, sh, stream);
  if (s != BASA_OK || !(mods || weights)) return s;
  GnJoin j;
  memset(&j, 0, sizeof(j));
  j.part_g = a.part_g; j.part_w = a.part_w;
  j.w = weight; j.b = bias; j.pw = post_weight;
  j.dgate = dgate; j.dscale = dscale; j.dshift = dshift;
  j.dw = dweight; j.db = dbias; j.dpw = dpost_weight;
  j.rows = p->rows; j.group = a.group; j.groups = p->groups;
  j.C = p->C; j.grid = (int)sh.grid;
  j.by_group = p->groups <= sh.grid;
  j.mod_bf16 = a.mod_bf16; j.w_bf16 = a.w_bf16;
  const unsigned gy = !mods ? 1u : (unsigned)(j.by_group ? p->groups : sh.grid);
  return launch_dependent(gnorm_join_kernel, dim3((unsigned)(p->C / 8), gy, weights ? 2 : 1), 256,
                          stream, j);
}

}  // extern "C"
