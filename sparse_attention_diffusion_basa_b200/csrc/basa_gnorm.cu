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
// HBM-bound: every row is read and written once.  A CTA takes whole rows, each
// thread the same columns of every row, so the modulations of a run of rows and
// the column sums of the backward stay in registers; a CTA's rows are a
// contiguous range, read ahead by asynchronous copies.
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
  int depth;                // stages of the read-ahead ring
  int need_y;
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
template <typename T>
__device__ __forceinline__ void take(const char* at, int j, f2 (&f)[4]) {
  Raw8<T> r;
  Slot<T>::take(at, j, blockDim.x, threadIdx.x, r);
  widen8(r, f);
}

// ---------------------------------------------------------------------------
// Sums over a row.  Every warp leaves its part in shared memory and, behind one
// barrier, adds up all warps' parts itself, one a lane.  `buf` alternates from
// sum to sum, so that barrier is the only one.
// ---------------------------------------------------------------------------
struct RowSmem {
  float2 red[2][kMaxWarps];
};

__device__ __forceinline__ float2 share(float2 v, RowSmem& sm, int& buf) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) sm.red[buf][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < (int)(blockDim.x >> 5) ? sm.red[buf][lane] : make_float2(0.f, 0.f);
  buf ^= 1;
  return v;
}

__device__ __forceinline__ float2 row_sum2(f2 a, f2 b, RowSmem& sm, int& buf) {
  const float2 v = lane_sum<32>(make_float2(sum2(a), sum2(b)));
  return lane_sum<32>(share(v, sm, buf));
}

// Elements of a row that warp i holds.
__device__ __forceinline__ float warp_elements(int i, int kv, int nvec) {
  int n = 0;
  for (int j = 0; j < kv; ++j) {
    const int left = nvec - j * (int)blockDim.x - 32 * i;
    n += left < 0 ? 0 : left > 32 ? 32 : left;
  }
  return (float)(8 * n);
}

struct Counts {      // elements of a warp: of this thread's, and of warp number `lane`
  float inv_mine;    // 1 / elements, 0 where there are none
  float lanes, inv_lanes;
};

// (mean, rstd) of a row held kV * 8 values a thread, zeros where ok is false.
// Layer: the squares are taken about each warp's own mean and joined about the
// row's (Chan, Golub and LeVeque's update), so a mean far from zero costs no
// digits and one barrier is enough.
template <int kV>
__device__ __forceinline__ float2 row_stats(const f2 (&f)[kV][4], const bool (&ok)[kV], int kind,
                                            float eps, float inv, const Counts& n, RowSmem& sm,
                                            int& buf) {
  f2 q = pk(0.f, 0.f);
  if (kind == BASA_NORM_LAYER) {
    f2 t = pk(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) t = add2(t, f[j][i]);
    const float s = lane_sum<32>(sum2(t));
    const float m = -s * n.inv_mine;
    const f2 mm = pk(m, m);
#pragma unroll
    for (int j = 0; j < kV; ++j)
      if (ok[j])
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 d = add2(f[j][i], mm);
          q = fma2(d, d, q);
        }
    const float2 v = share(make_float2(s, lane_sum<32>(sum2(q))), sm, buf);
    const float mean = lane_sum<32>(v.x) * inv;
    const float d = v.x * n.inv_lanes - mean;
    const float m2 = lane_sum<32>(fmaf(n.lanes * d, d, v.y));
    return make_float2(mean, rsqrtf(m2 * inv + eps));
  }
#pragma unroll
  for (int j = 0; j < kV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) q = fma2(f[j][i], f[j][i], q);
  const float2 v = share(make_float2(0.f, lane_sum<32>(sum2(q))), sm, buf);
  return make_float2(0.f, rsqrtf(lane_sum<32>(v.y) * inv + eps));
}

__device__ __forceinline__ f2 both(float v) { return pk(v, v); }

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <typename TX, typename TY, int kV, int kThreads, int kCtas, bool kBranch, bool kNorm>
__global__ void __launch_bounds__(kThreads, kCtas) gnorm_kernel(GnArgs a) {
  extern __shared__ __align__(16) char ring[];
  __shared__ RowSmem sm;
  const int tid = threadIdx.x, threads = blockDim.x, nvec = a.C / 8;
  bool ok[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) ok[j] = j * threads + tid < nvec;
  const int next = threads * 8;  // columns from one of a thread's vectors to the next
  Counts cnt;
  {
    const float mine = warp_elements(tid >> 5, kV, nvec);
    cnt.inv_mine = mine > 0.f ? 1.f / mine : 0.f;
    cnt.lanes = (tid & 31) < (threads >> 5) ? warp_elements(tid & 31, kV, nvec) : 0.f;
    cnt.inv_lanes = cnt.lanes > 0.f ? 1.f / cnt.lanes : 0.f;
  }
  const int x_bytes = Slot<TX>::bytes(kV, threads);
  const int stage = x_bytes + (kBranch ? Slot<TY>::bytes(kV, threads) : 0);
  const int r0 = (int)(a.rows * blockIdx.x / gridDim.x);
  const int r1 = (int)(a.rows * (blockIdx.x + 1) / gridDim.x);
  const long long off = (long long)r0 * a.C + tid * 8;
  const TX* x = static_cast<const TX*>(a.x) + off;
  const TY* y = kBranch ? static_cast<const TY*>(a.y) + off : nullptr;
  TX* xo = kBranch ? static_cast<TX*>(a.xo) + off : nullptr;
  TY* h = kNorm ? static_cast<TY*>(a.h) + off : nullptr;
  const uint32_t ring_at = shared_u32(ring);
  int ahead = 0, to_stage = 0;  // rows asked for, and the stage of the next
  auto fetch = [&]() {
    if (r0 + ahead < r1) {
      const uint32_t at = ring_at + to_stage;
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) {
          Slot<TX>::fetch(at, x + j * next, j, threads, tid);
          if (kBranch) Slot<TY>::fetch(at + x_bytes, y + j * next, j, threads, tid);
        }
      x += a.C;
      if (kBranch) y += a.C;
    }
    copy_commit();
    ++ahead;
    to_stage = to_stage + stage == a.depth * stage ? 0 : to_stage + stage;
  };
  for (int s = 0; s < a.depth - 1; ++s) fetch();
  f2 G[kV][4], S[kV][4], B[kV][4];
  long long g_end = r0;
  int buf = 0, at_stage = 0;
  for (int r = r0; r < r1; ++r) {
    fetch();
    if (r >= g_end) {  // another modulation row
      const long long g = r / a.group;
      g_end = (g + 1) * a.group;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const long long c = ok[j] ? tid * 8 + j * next : 0;
        f2 p[4], q[4];
        if (kBranch) {
          param8(a.gate, a.mod_bf16, g * a.ld_gate + c, 1.f, G[j]);
          param8(a.pw, a.w_bf16, c, 1.f, p);
#pragma unroll
          for (int i = 0; i < 4; ++i) G[j][i] = mul2(G[j][i], p[i]);
        }
        if (kNorm) {
          param8(a.scale, a.mod_bf16, g * a.ld_scale + c, 0.f, p);
          param8(a.w, a.w_bf16, c, 1.f, S[j]);
          param8(a.b, a.w_bf16, c, 0.f, B[j]);
          param8(a.shift, a.mod_bf16, g * a.ld_shift + c, 0.f, q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = add2(p[i], both(1.f));
            S[j][i] = mul2(S[j][i], p[i]);
            B[j][i] = fma2(B[j][i], p[i], q[i]);
          }
        }
      }
    }
    ring_wait(a.depth);
    const char* at = ring + at_stage;
    at_stage = at_stage + stage == a.depth * stage ? 0 : at_stage + stage;
    f2 f[kV][4];
    float2 post = make_float2(0.f, 0.f), pre = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[j][i] = 0;
    if (kBranch) {
      f2 u[kV][4];
#pragma unroll
      for (int j = 0; j < kV; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[j][i] = 0;
        if (ok[j]) take<TY>(at + x_bytes, j, u[j]);
      }
      if (a.post != BASA_NORM_NONE) {
        post = row_stats<kV>(u, ok, a.post, a.post_eps, a.inv, cnt, sm, buf);
        const f2 m = both(-post.x), s = both(post.y);
#pragma unroll
        for (int j = 0; j < kV; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) u[j][i] = mul2(add2(u[j][i], m), s);
      }
      const f2 res = both(a.res);
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) {
          take<TX>(at, j, f[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[j][i] = fma2(res, f[j][i], mul2(u[j][i], G[j][i]));
          store8(xo + j * next, f[j]);
        }
      xo += a.C;
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) take<TX>(at, j, f[j]);
    }
    if (kNorm) {
      pre = row_stats<kV>(f, ok, a.norm, a.eps, a.inv, cnt, sm, buf);
      const f2 m = both(-pre.x), s = both(pre.y);
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[j][i] = fma2(mul2(add2(f[j][i], m), s), S[j][i], B[j][i]);
          store8(h + j * next, f[j]);
        }
      h += a.C;
    }
    if (a.stats && tid == 0) a.stats[r] = make_float4(pre.x, pre.y, post.x, post.y);
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
template <int kV>
struct ColSums {
  f2 a[kV][4], s[kV][4], d[kV][4];  // gh xh, gh, t yh
};

// The sums of modulation row g end: into the result where all its rows lay in
// this CTA's range, into the CTA's partial rows otherwise; and, times the
// modulation, into the CTA's partial rows of the weights.
template <int kV, bool kBranch, bool kNorm>
__device__ __forceinline__ void flush(const GnArgs& a, const ColSums<kV>& c, long long g, bool whole,
                                   bool first, bool again) {
  float* pg = a.part_g + ((long long)blockIdx.x * 2 + (first ? 0 : 1)) * 3 * a.C;
  float* pw = a.part_w + (long long)blockIdx.x * 3 * a.C;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (col >= a.C) continue;
    f2 v[4], p[4], q[4];
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

template <typename TX, typename TY, int kV, int kThreads, bool kBranch, bool kNorm>
__global__ void __launch_bounds__(kThreads, 1) gnorm_bwd_kernel(const __grid_constant__ GnArgs a) {
  extern __shared__ __align__(16) char ring[];
  __shared__ RowSmem sm;
  const int tid = threadIdx.x, threads = blockDim.x, nvec = a.C / 8;
  bool ok[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) ok[j] = j * threads + tid < nvec;
  const int next = threads * 8;
  const int xb = Slot<TX>::bytes(kV, threads), yb = Slot<TY>::bytes(kV, threads);
  const int o_y = a.gx ? xb : 0, o_x = o_y + (a.need_y ? yb : 0), o_gh = o_x + xb;
  const int stage = kNorm ? o_gh + yb : o_x;
  const int r0 = (int)(a.rows * blockIdx.x / gridDim.x);
  const int r1 = (int)(a.rows * (blockIdx.x + 1) / gridDim.x);
  long long from = (long long)r0 * a.C + tid * 8, to = from;  // of the next row read, written
  const uint32_t ring_at = shared_u32(ring);
  int ahead = 0, to_stage = 0;
  auto fetch = [&]() {
    if (r0 + ahead < r1) {
      const uint32_t at = ring_at + to_stage;
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) {
          const long long e = from + j * next;
          if (kNorm) {
            Slot<TX>::fetch(at + o_x, static_cast<const TX*>(a.x) + e, j, threads, tid);
            Slot<TY>::fetch(at + o_gh, static_cast<const TY*>(a.gh) + e, j, threads, tid);
          }
          if (a.gx) Slot<TX>::fetch(at, static_cast<const TX*>(a.gx) + e, j, threads, tid);
          if (kBranch && a.need_y)
            Slot<TY>::fetch(at + o_y, static_cast<const TY*>(a.y) + e, j, threads, tid);
        }
      from += a.C;
    }
    copy_commit();
    ++ahead;
    to_stage = to_stage + stage == a.depth * stage ? 0 : to_stage + stage;
  };
  for (int s = 0; s < a.depth - 1; ++s) fetch();
  f2 G[kV][4], S[kV][4];  // gate * pw, (1 + scale) * w
  ColSums<kV> sum;
  long long g = r0 / a.group, g_end = r0;
  const long long g_first = g;
  bool flushed = false;
  int buf = 0, at_stage = 0;
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f), st_next = st;
  if (a.st) st_next = __ldg(a.st + r0);
  for (int r = r0;; ++r) {
    if (r >= g_end || r == r1) {
      if (r > r0) {
        flush<kV, kBranch, kNorm>(a, sum, g, g * a.group >= r0 && (g + 1) * a.group <= r,
                                  g == g_first, flushed);
        flushed = true;
      }
      if (r == r1) break;
      g = r / a.group;
      g_end = (g + 1) * a.group;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const long long c = ok[j] ? tid * 8 + j * next : 0;
        f2 p[4];
        if (kBranch) {
          param8(a.gate, a.mod_bf16, g * a.ld_gate + c, 1.f, G[j]);
          param8(a.pw, a.w_bf16, c, 1.f, p);
#pragma unroll
          for (int i = 0; i < 4; ++i) G[j][i] = mul2(G[j][i], p[i]);
        }
        if (kNorm) {
          param8(a.scale, a.mod_bf16, g * a.ld_scale + c, 0.f, p);
          param8(a.w, a.w_bf16, c, 1.f, S[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) S[j][i] = mul2(S[j][i], add2(p[i], both(1.f)));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum.a[j][i] = sum.s[j][i] = sum.d[j][i] = 0;
      }
    }
    fetch();
    st = st_next;
    if (a.st && r + 1 < r1) st_next = __ldg(a.st + r + 1);
    ring_wait(a.depth);
    const char* at = ring + at_stage;
    at_stage = at_stage + stage == a.depth * stage ? 0 : at_stage + stage;
    f2 t[kV][4];
    if (kNorm) {
      const f2 m = both(-st.x), s = both(st.y);
      f2 xh[kV][4], s1 = 0, s2 = 0;
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) {
          take<TX>(at + o_x, j, xh[j]);
          take<TY>(at + o_gh, j, t[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xh[j][i] = mul2(add2(xh[j][i], m), s);
            sum.a[j][i] = fma2(t[j][i], xh[j][i], sum.a[j][i]);
            sum.s[j][i] = add2(sum.s[j][i], t[j][i]);
            t[j][i] = mul2(t[j][i], S[j][i]);
            s1 = add2(s1, t[j][i]);
            s2 = fma2(t[j][i], xh[j][i], s2);
          }
        }
      const float2 v = row_sum2(s1, s2, sm, buf);
      // t = rstd (a - mean(a) - xh mean(a xh)) + gx
      const f2 c1 = both(a.norm == BASA_NORM_LAYER ? -v.x * a.inv : 0.f), c2 = both(-v.y * a.inv);
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) {
          f2 gx[4] = {0, 0, 0, 0};
          if (a.gx) take<TX>(at, j, gx);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            t[j][i] = fma2(s, add2(fma2(xh[j][i], c2, t[j][i]), c1), gx[i]);
        }
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) take<TX>(at, j, t[j]);
    }
    const f2 res = both(a.res);
#pragma unroll
    for (int j = 0; j < kV; ++j)
      if (ok[j]) {
        f2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(res, t[j][i]);
        store8(static_cast<TX*>(a.dx) + to + j * next, v);
      }
    if (kBranch) {
      if (a.post == BASA_NORM_NONE) {
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (ok[j]) {
            if (a.need_y) {
              f2 y[4];
              take<TY>(at + o_y, j, y);
#pragma unroll
              for (int i = 0; i < 4; ++i) sum.d[j][i] = fma2(t[j][i], y[i], sum.d[j][i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j][i] = mul2(t[j][i], G[j][i]);
          }
      } else {
        const f2 m = both(-st.z), s = both(st.w);
        f2 yh[kV][4], s1 = 0, s2 = 0;
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (ok[j]) {
            take<TY>(at + o_y, j, yh[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              yh[j][i] = mul2(add2(yh[j][i], m), s);
              sum.d[j][i] = fma2(t[j][i], yh[j][i], sum.d[j][i]);
              t[j][i] = mul2(t[j][i], G[j][i]);
              s1 = add2(s1, t[j][i]);
              s2 = fma2(t[j][i], yh[j][i], s2);
            }
          }
        const float2 v = row_sum2(s1, s2, sm, buf);
        const f2 c1 = both(a.post == BASA_NORM_LAYER ? -v.x * a.inv : 0.f), c2 = both(-v.y * a.inv);
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (ok[j])
#pragma unroll
            for (int i = 0; i < 4; ++i)
              t[j][i] = mul2(s, add2(fma2(yh[j][i], c2, t[j][i]), c1));
      }
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (ok[j]) store8(static_cast<TY*>(a.dy) + to + j * next, t[j]);
    }
    to += a.C;
  }
}

// Joins the partial sums of gnorm_bwd_kernel.  A CTA owns eight columns and
// reads 32 partial rows side by side, joined in a fixed order.  blockIdx.z = 0:
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
    for (long long i = lo + lane; i <= hi; i += 32) {
      const bool first = a.rows * i / a.grid / a.group == g;
      const float* p = a.part_g + (i * 2 + !first) * 3 * a.C + c;
#pragma unroll
      for (int s = 0; s < 3; ++s) v[s] += p[s * a.C];
    }
  } else {
    if (blockIdx.y || !a.part_w) return;
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

constexpr int kSmemCta = 220 * 1024;  // of the 227 KB a CTA may have; the rest is static

template <typename K>
basa_status go(K kernel, const GnArgs& a, unsigned grid, int threads, int smem, cudaStream_t st) {
  if (smem > 32 * 1024 &&  // beside the static part, 48 KB are free to take
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return BASA_ERR_CUDA;
  kernel<<<grid, threads, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

template <typename TX, typename TY, int kThreads, int kCtas>
basa_status go_fwd_t(GnArgs a, int threads, cudaStream_t st) {
  const bool branch = a.y != nullptr, norm = a.norm != BASA_NORM_NONE;
  const int stage = Slot<TX>::bytes(2, threads) + (branch ? Slot<TY>::bytes(2, threads) : 0);
  a.depth = 3;
  const int smem = a.depth * stage;
  int per_sm = kSmemCta / (smem + 1024);
  const int by_regs = kThreads * kCtas / threads;
  if (per_sm > by_regs) per_sm = by_regs;
  if (per_sm < 1) per_sm = 1;
  const long long cap = (long long)row_sm_count() * per_sm;
  const unsigned grid = (unsigned)(a.rows < cap ? a.rows : cap);
  if (branch && norm)
    return go(gnorm_kernel<TX, TY, 2, kThreads, kCtas, true, true>, a, grid, threads, smem, st);
  if (branch)
    return go(gnorm_kernel<TX, TY, 2, kThreads, kCtas, true, false>, a, grid, threads, smem, st);
  return go(gnorm_kernel<TX, TY, 2, kThreads, kCtas, false, true>, a, grid, threads, smem, st);
}
template <typename TX, typename TY>
basa_status go_fwd(const GnArgs& a, cudaStream_t st) {
  const int threads = round32((a.C / 8 + 1) / 2);
  if (threads <= 128) return go_fwd_t<TX, TY, 128, 4>(a, threads, st);
  if (threads <= 320) return go_fwd_t<TX, TY, 320, 2>(a, threads, st);
  return go_fwd_t<TX, TY, 512, 1>(a, threads, st);
}

// Launch shape of the backward: vectors a thread and CTAs.  Sums in registers
// cost 40 fp32 a vector, so a thread takes one vector up to 640 threads (102
// registers each), two beyond.
struct BwdShape {
  int v, threads;
  long long grid;
};
BwdShape bwd_shape(const basa_gnorm_params* p) {
  BwdShape s;
  const int nvec = p->C / 8;
  s.v = nvec <= 640 ? 1 : 2;
  s.threads = round32((nvec + s.v - 1) / s.v);
  int per_sm = (s.v == 1 ? 640 : 512) / s.threads;
  if (per_sm > 8) per_sm = 8;
  long long cap = (long long)row_sm_count() * per_sm;
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

template <typename TX, typename TY, int kV, int kThreads>
basa_status go_bwd_v(GnArgs a, const BwdShape& s, cudaStream_t st) {
  const bool branch = a.dy != nullptr, norm = a.norm != BASA_NORM_NONE;
  const int xb = Slot<TX>::bytes(kV, s.threads), yb = Slot<TY>::bytes(kV, s.threads);
  const int stage = (a.gx ? xb : 0) + (a.need_y ? yb : 0) + (norm ? xb + yb : 0);
  const int ctas = (kV == 1 ? 640 : 512) / s.threads;
  const int room = kSmemCta / (ctas < 1 ? 1 : ctas > 8 ? 8 : ctas) - 1024;
  a.depth = room / stage;
  a.depth = a.depth > 3 ? 3 : a.depth < 1 ? 1 : a.depth;
  const int smem = a.depth * stage;
  const unsigned grid = (unsigned)s.grid;
  if (branch && norm)
    return go(gnorm_bwd_kernel<TX, TY, kV, kThreads, true, true>, a, grid, s.threads, smem, st);
  if (branch)
    return go(gnorm_bwd_kernel<TX, TY, kV, kThreads, true, false>, a, grid, s.threads, smem, st);
  return go(gnorm_bwd_kernel<TX, TY, kV, kThreads, false, true>, a, grid, s.threads, smem, st);
}
template <typename TX, typename TY>
basa_status go_bwd(const GnArgs& a, const BwdShape& s, cudaStream_t st) {
  return s.v == 1 ? go_bwd_v<TX, TY, 1, 640>(a, s, st) : go_bwd_v<TX, TY, 2, 512>(a, s, st);
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
  GnArgs a = gnorm_args(p);
  a.x = x; a.y = y; a.gate = gate; a.pw = post_weight;
  a.w = weight; a.b = bias; a.scale = scale; a.shift = shift;
  a.xo = x_out; a.h = h;
  a.stats = reinterpret_cast<float4*>(stats);
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
  GnArgs a = gnorm_args(p);
  a.x = x_out; a.y = y; a.gate = gate; a.pw = post_weight;
  a.w = weight; a.b = bias; a.scale = scale;
  a.gh = dh; a.gx = dx_out;
  a.st = reinterpret_cast<const float4*>(stats);
  a.dx = dx; a.dy = dy;
  a.dgate = dgate; a.dscale = dscale; a.dshift = dshift;
  a.need_y = need_y;
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
  gnorm_join_kernel<<<dim3((unsigned)(p->C / 8), gy, weights ? 2 : 1), 256, 0, stream>>>(j);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

}  // extern "C"
