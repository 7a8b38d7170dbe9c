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
//
// Bound by HBM: every row is read once and written once.  At 6.5 TB/s an SM moves
// 23 bytes a clock, so the kernels also have to spend few instructions a value:
// arithmetic is packed two values an instruction, a lane holds both elements of
// its pairs, a token's angles are gathered once for all its heads, and rows come
// by asynchronous copies that need no registers while they are under way.
// Measured on a B200 (copy 6.57 TB/s), device time of the call: 128 x 128 grid, 24
// heads of 128 in bf16, q, k, v slices of one projection 93.3 us = 6.47 TB/s (98% of
// the copy rate); 21 x 45 x 80 clip, norm over 40 heads, q and k 498 us = 6.22 TB/s
// (95%; the first form, unpacked and with an exchange between lanes a pair, 684);
// backward of two 128 x 128 grids 258 us = 6.25 TB/s (95%; first form 389).
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
  int ctas;            // along the tokens
  int chunks;          // CTAs that share a token's heads
  int steps;           // of 512 / d heads each, per chunk
  float mul, rest;     // e4m3 output: 1 / factor rounded toward zero, and what is left of it
                       // (q and k behind a norm: mul alone, rounded to nearest)
  float inv;           // 1 / values of a token's row
};

struct RopeArgs {
  RopePart part[3];    // q, k, v; read from the parameter bank where they are used
  const float2* table;
  uint32_t tokens, T, Hg, Wg;
  int nt, nh, nw;      // rotated pairs per axis
  int d;
  float eps;
  int w_bf16;
};

// A lane holds sixteen elements of a head: two vectors of eight, at ea and eb.
// They are kept as eight packed pairs A[4], B[4] such that (A[i], B[i]) are the
// first and second elements of rotated pairs, whatever the layout, so that the
// rotation is A' = A cos - B sin, B' = B cos + A sin without a word exchanged
// between lanes:
//   pairs    A the even and B the odd elements of both vectors,
//   halves   A the vector in the first and B the one in the second half of the
//            rotated width (of the rest, two vectors that are not rotated).
struct Lane {
  int ea, eb;   // elements
  int ja, jb;   // rotated pair of A[0] and of A[2]; -1: not rotated
};
template <bool kHalves>
__device__ __forceinline__ Lane lane_of(const RopeArgs& a, int sub) {
  const int pairs = a.nt + a.nh + a.nw;
  Lane l;
  if (kHalves) {
    const int r = pairs / 8;  // lanes of the rotated width
    if (sub < r) {
      l.ea = 8 * sub;
      l.eb = l.ea + pairs;
      l.ja = 8 * sub;
      l.jb = l.ja + 4;
    } else {
      l.ea = 2 * pairs + 8 * (sub - r);
      l.eb = l.ea + (a.d - 2 * pairs) / 2;
      l.ja = l.jb = -1;
    }
  } else {
    l.ea = 8 * sub;
    l.eb = l.ea + a.d / 2;
    l.ja = l.ea / 2;
    l.jb = l.eb / 2;
  }
  return l;
}

template <bool kHalves, typename T>
__device__ __forceinline__ void unpack16(const Raw8<T>& a, const Raw8<T>& b, f2 (&A)[4],
                                         f2 (&B)[4]) {
  if (kHalves) {
    widen8(a, A);
    widen8(b, B);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      A[i] = pk(elem(a, 4 * i), elem(a, 4 * i + 2));
      B[i] = pk(elem(a, 4 * i + 1), elem(a, 4 * i + 3));
      A[i + 2] = pk(elem(b, 4 * i), elem(b, 4 * i + 2));
      B[i + 2] = pk(elem(b, 4 * i + 1), elem(b, 4 * i + 3));
    }
  }
}
template <bool kHalves>
__device__ __forceinline__ void order16(const f2 (&A)[4], const f2 (&B)[4], float (&a)[8],
                                        float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = un(A[i]), q = un(B[i]);
    if (kHalves) {
      a[2 * i] = p.x;
      a[2 * i + 1] = p.y;
      b[2 * i] = q.x;
      b[2 * i + 1] = q.y;
    } else {
      float* f = i < 2 ? a + 4 * i : b + 4 * (i - 2);
      f[0] = p.x;
      f[1] = q.x;
      f[2] = p.y;
      f[3] = q.y;
    }
  }
}
template <bool kHalves, typename TO>
__device__ __forceinline__ void pack16(TO* row, const Lane& l, const f2 (&A)[4], const f2 (&B)[4]) {
  float a[8], b[8];
  order16<kHalves>(A, B, a, b);
  store8(row + l.ea, a);
  store8(row + l.eb, b);
}
// A lane's sixteen weights from element `col` of w on, in the order of A and B.
template <bool kHalves>
__device__ __forceinline__ void weight16(const void* w, bool bf16, int col, const Lane& l,
                                         f2 (&A)[4], f2 (&B)[4]) {
  Raw8<float> a, b;
  float fa[8], fb[8];
  param8(w, bf16, col + l.ea, 1.f, fa);
  param8(w, bf16, col + l.eb, 1.f, fb);
  a.a = make_uint4(__float_as_uint(fa[0]), __float_as_uint(fa[1]), __float_as_uint(fa[2]),
                   __float_as_uint(fa[3]));
  a.b = make_uint4(__float_as_uint(fa[4]), __float_as_uint(fa[5]), __float_as_uint(fa[6]),
                   __float_as_uint(fa[7]));
  b.a = make_uint4(__float_as_uint(fb[0]), __float_as_uint(fb[1]), __float_as_uint(fb[2]),
                   __float_as_uint(fb[3]));
  b.b = make_uint4(__float_as_uint(fb[4]), __float_as_uint(fb[5]), __float_as_uint(fb[6]),
                   __float_as_uint(fb[7]));
  unpack16<kHalves>(a, b, A, B);
}

// Where pair j's angle lies in the table: base + coordinate of its axis * pairs
// of the axis.
struct Spot {
  int base, axis;  // axis 3: not rotated
};
__device__ __forceinline__ Spot spot_of(const RopeArgs& a, int j) {
  const int pairs = a.nt + a.nh + a.nw;
  if (j < 0 || j >= pairs) return {0, 3};
  if (j < a.nt) return {j, 0};
  if (j < a.nt + a.nh) return {(int)a.T * a.nt + j - a.nt, 1};
  return {(int)a.T * a.nt + (int)a.Hg * a.nh + j - a.nt - a.nh, 2};
}

// Grid coordinates of a token, stepped by a fixed number of tokens without a
// division.
struct Coord {
  uint32_t x, y, t, sx, sy, st;
  __device__ __forceinline__ void init(const RopeArgs& a, uint32_t n, uint32_t step) {
    uint32_t q = n / a.Wg;
    x = n - q * a.Wg;
    t = q / a.Hg;
    y = q - t * a.Hg;
    t %= a.T;
    q = step / a.Wg;
    sx = step - q * a.Wg;
    st = q / a.Hg;
    sy = q - st * a.Hg;
    st %= a.T;
  }
  __device__ __forceinline__ void next(const RopeArgs& a) {
    x += sx;
    y += sy;
    t += st;
    if (x >= a.Wg) {
      x -= a.Wg;
      ++y;
    }
    if (y >= a.Hg) {
      y -= a.Hg;
      ++t;
    }
    if (t >= a.T) t -= a.T;
  }
  __device__ __forceinline__ float2 angle(const RopeArgs& a, const Spot& s) const {
    const int off = s.axis == 0 ? (int)t * a.nt : s.axis == 1 ? (int)y * a.nh : (int)x * a.nw;
    return s.axis == 3 ? make_float2(1.f, 0.f) : __ldg(a.table + s.base + off);
  }
};

__device__ __forceinline__ f2 neg2(f2 v) {
  const float2 f = un(v);
  return pk(-f.x, -f.y);
}

// Which of a lane's eight pairs are rotated, a bit each.
template <bool kHalves>
__device__ __forceinline__ uint32_t rotated(const RopeArgs& a, const Lane& l) {
  if (kHalves) return l.ja >= 0 ? 0xffu : 0u;
  const int pairs = a.nt + a.nh + a.nw;
  auto four = [&](int j) { return (1u << min(max(pairs - j, 0), 4)) - 1u; };
  return four(l.ja) | four(l.jb) << 4;
}
// Without a norm: (A, B) become (A C + B N, B C + A S), or, not rotated, stay what they
// were.  Their sine of zero would not do that: 0 * infinity makes a NaN of a neighbour,
// and a zero may lose its sign.  (Under a norm an infinity is its head's loss anyway.)
template <bool kHalves>
__device__ __forceinline__ void turn(f2 (&A)[4], f2 (&B)[4], const f2 (&C)[4], const f2 (&S)[4],
                                     const f2 (&N)[4], uint32_t rot) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 p = fma2(A[i], C[i], mul2(B[i], N[i]));
    const f2 q = fma2(B[i], C[i], mul2(A[i], S[i]));
    if (kHalves) {
      A[i] = rot ? p : A[i];
      B[i] = rot ? q : B[i];
    } else {
      const float2 a0 = un(A[i]), b0 = un(B[i]), a1 = un(p), b1 = un(q);
      const bool x = rot >> (2 * i) & 1, y = rot >> (2 * i) & 2;
      A[i] = pk(x ? a1.x : a0.x, y ? a1.y : a0.y);
      B[i] = pk(x ? b1.x : b0.x, y ? b1.y : b0.y);
    }
  }
}

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;

// Which of q, k, v a CTA works on, the chunk of its heads, and its number among
// the CTAs along the tokens.  Each part has CTAs in proportion to its work.
__device__ __forceinline__ int part_of(const RopeArgs& a, int& chunk, int& cta) {
  int i = blockIdx.x, part = 0;
  while (part < 2 && i >= a.part[part].ctas * a.part[part].chunks) {
    i -= a.part[part].ctas * a.part[part].chunks;
    ++part;
  }
  chunk = i / a.part[part].ctas;
  cta = i - chunk * a.part[part].ctas;
  return part;
}

// An e4m3 output is value / factor, rounded to fp32 and then to e4m3.  Where a value
// has not been scaled before, a product with the factor's reciprocal, itself rounded,
// does not do: quotients of bf16 values lie at ties of e4m3 (0.75 / 0.03 = 25, between
// 24 and 26), and 0.75% of v's values went the other way.  With 1 / factor in two
// terms the quotient is off by at most 2^-46 of itself ahead of its rounding to fp32.
// `rest` is positive, so that an infinity stays one.  A division took 123 us for the
// 128 x 128 grid without a norm, this 77, one product 75.  Behind a norm one product
// is taken into 1 / rms: those values are rounded already and meet a tie by chance
// alone.
__device__ __forceinline__ void divide8(f2 (&A)[4], f2 (&B)[4], const RopePart& P) {
  const f2 m = pk(P.mul, P.mul), rest = pk(P.rest, P.rest);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    A[i] = fma2(A[i], m, mul2(A[i], rest));
    B[i] = fma2(B[i], m, mul2(B[i], rest));
  }
}

// v: rows copied (or narrowed) two heads' worth at a time.
template <typename TI, typename TO, int kLph, bool kHalves>
__device__ __forceinline__ void copy_rows(const TI* x, TO* o, const Lane& l, int h0, int hend,
                                          const RopePart& P) {
  constexpr int kHpw = 32 / kLph, kD = kLph * 16;
  for (int h = h0; h < hend; h += 2 * kHpw) {
    Raw8<TI> ra[2], rb[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (h + u * kHpw < hend) {
        load8(ra[u], x + (h + u * kHpw) * kD + l.ea);
        load8(rb[u], x + (h + u * kHpw) * kD + l.eb);
      }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (h + u * kHpw < hend) {
        f2 A[4], B[4];
        unpack16<kHalves>(ra[u], rb[u], A, B);
        if (sizeof(TO) == 1) divide8(A, B, P);
        pack16<kHalves>(o + (h + u * kHpw) * kD, l, A, B);
      }
  }
}

// A warp's two pairs a lane of one token's angles, gathered ahead of the token
// and then read by the lanes that need them.
struct Gather {
  Coord at;
  Spot spot[2];
  float2 next[2];
  __device__ __forceinline__ void init(const RopeArgs& a, uint32_t n, uint32_t step, int first,
                                       int threads) {
    at.init(a, n, step);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = first + i * threads;
      spot[i] = spot_of(a, j < 64 ? j : -1);
      next[i] = at.angle(a, spot[i]);
    }
  }
  __device__ __forceinline__ void put(float4* to, int first, int threads) const {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (first + i * threads < 64) reinterpret_cast<float2*>(to)[first + i * threads] = next[i];
  }
  // Past the last token the coordinates are those of some token all the same.
  __device__ __forceinline__ void ahead(const RopeArgs& a) {
    at.next(a);
#pragma unroll
    for (int i = 0; i < 2; ++i) next[i] = at.angle(a, spot[i]);
  }
};

__device__ __forceinline__ void angles_of(const float4* cs, const Lane& l, f2 (&C)[4],
                                          f2 (&S)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = i < 2 ? l.ja : l.jb;
    float4 v = make_float4(1.f, 0.f, 1.f, 0.f);
    if (j >= 0) v = cs[j / 2 + (i & 1)];
    C[i] = pk(v.x, v.z);
    S[i] = pk(v.y, v.w);
  }
}

// Stages of a warp's ring: 4 KB of reads in flight a warp, 2 KB for fp32's half
// as many values a byte.
template <typename T> constexpr int kStages = sizeof(T) == 2 ? 4 : 2;

// Norm over each head, or none.  kLph lanes hold a head, a warp 32 / kLph heads
// (a step); a warp takes the steps of its chunk of one token, then the next
// token, so that a token's angles are read once for all its heads.  Rows come
// through a ring of asynchronous copies, private to each lane, that runs ahead
// across tokens.  The norm's weight is folded into the angles:
// A' = r (A (wA cos) - B (wB sin)).  Five CTAs an SM at 96 registers against
// four at 128: 96 and 101 us for the 128 x 128 grid in bf16.  With a norm the fp32
// forms spill there (8 bytes in the pairs layout, 24 in halves) and take 234 us, 79%
// of the copy rate; bf16 in halves spills 8 bytes (95 us).
template <typename TI, typename TO, int kLph, bool kHalves, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, 5)
    rope_head_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kHpw = 32 / kLph, kD = kLph * 16, kDepth = kStages<TI>;
  constexpr int kStage = Slot<TI>::bytes(2, 32);
  __shared__ __align__(16) char rings[kRopeWarps][kDepth * kStage];
  __shared__ float4 cs[kRopeWarps][2][32];
  int chunk, cta;
  const int part = part_of(a, chunk, cta);
  const RopePart& P = a.part[part];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, slot = lane / kLph;
  const int h0 = chunk * P.steps * kHpw + slot;
  const int hend = min(P.heads, (chunk + 1) * P.steps * kHpw);
  const uint32_t stride = P.ctas * kRopeWarps;
  const Lane l = lane_of<kHalves>(a, lane % kLph);
  uint32_t n = cta * kRopeWarps + warp;
  const TI* x = static_cast<const TI*>(P.x) + (long long)n * P.ldx;
  TO* o = static_cast<TO*>(P.o) + (long long)n * P.ldo;
  const long long dx = (long long)stride * P.ldx, dout = (long long)stride * P.ldo;
  if (part == 2) {
    for (; n < a.tokens; n += stride, x += dx, o += dout)
      copy_rows<TI, TO, kLph, kHalves>(x, o, l, h0, hend, P);
    return;
  }
  if (n >= a.tokens) return;  // a whole warp; the kernel has no CTA barrier
  const uint32_t ring = shared_u32(rings[warp]);
  uint32_t fn = n;
  int fh = h0, to = 0;
  auto fetch = [&]() {
    if (fn < a.tokens) {
      const bool on = fh < hend;
      const TI* head = x + (on ? fh : 0) * kD;
      Slot<TI>::fetch(ring + to, head + l.ea, 0, 32, lane, on);
      Slot<TI>::fetch(ring + to, head + l.eb, 1, 32, lane, on);
      fh += kHpw;
      if (fh - slot >= hend) {
        fh = h0;
        fn += stride;
        x += dx;
      }
    }
    copy_commit();
    to = to + kStage == kDepth * kStage ? 0 : to + kStage;
  };
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) fetch();
  Gather ang;
  ang.init(a, n, stride, lane, 32);
  f2 WA[4], WB[4];
  if (kNorm) weight16<kHalves>(P.w, a.w_bf16, 0, l, WA, WB);
  const float mul = sizeof(TO) == 1 ? P.mul : 1.f;
  const uint32_t rot = kNorm ? 0u : rotated<kHalves>(a, l);
  int from = 0, buf = 0;
  for (; n < a.tokens; n += stride, o += dout, buf ^= 1) {
    ang.put(cs[warp][buf], lane, 32);
    __syncwarp();
    ang.ahead(a);
    f2 CA[4], CB[4], SA[4], SB[4];
    angles_of(cs[warp][buf], l, CA, SA);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      CB[i] = CA[i];
      SB[i] = neg2(SA[i]);
      if (kNorm) {
        CA[i] = mul2(CA[i], WA[i]);
        CB[i] = mul2(CB[i], WB[i]);
        SA[i] = mul2(SA[i], WA[i]);
        SB[i] = mul2(SB[i], WB[i]);
      }
    }
    for (int h = h0; h - slot < hend; h += kHpw) {  // the same trip count for a warp
      fetch();
      copy_wait<kDepth - 1>();
      Raw8<TI> ra, rb;
      Slot<TI>::take(rings[warp] + from, 0, 32, lane, ra);
      Slot<TI>::take(rings[warp] + from, 1, 32, lane, rb);
      from = from + kStage == kDepth * kStage ? 0 : from + kStage;
      f2 A[4], B[4];
      unpack16<kHalves>(ra, rb, A, B);
      float r = mul;
      if (kNorm) {
        f2 s0 = mul2(A[0], A[0]), s1 = mul2(B[0], B[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          s0 = fma2(A[i], A[i], s0);
          s1 = fma2(B[i], B[i], s1);
        }
        r *= rsqrtf(lane_sum<kLph>(sum2(add2(s0, s1))) * (1.f / kD) + a.eps);
      }
      if (!kNorm) {
        turn<kHalves>(A, B, CA, SA, SB, rot);
      } else {
        const f2 rr = pk(r, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 p = fma2(A[i], CA[i], mul2(B[i], SB[i]));
          const f2 q = fma2(B[i], CB[i], mul2(A[i], SA[i]));
          A[i] = mul2(p, rr);
          B[i] = mul2(q, rr);
        }
      }
      if (!kNorm && sizeof(TO) == 1) divide8(A, B, P);
      if (h < hend) pack16<kHalves>(o + h * kD, l, A, B);
    }
  }
}

// Backward of rope_head_kernel, the same walk.  The weight's gradient is summed
// in a lane's own sixteen columns over all its tokens and heads, then over the
// CTA, and left as one row of partial sums a CTA.  Four CTAs an SM: 128 registers
// hold the sums and a step without spills (fp32 in the pairs layout at 64 and 128
// elements a head spills 8 bytes); two 128 x 128 grids with 24 heads 258 us.
// Without a norm there are no sums: five CTAs, as forward (128 x 128 grid 96 us; four,
// with the selects of what is not rotated, 100).
template <typename T, int kLph, bool kHalves, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, kNorm ? 4 : 5)
    rope_head_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kHpw = 32 / kLph, kD = kLph * 16, kDepth = kStages<T>;
  constexpr int kStage = Slot<T>::bytes(kNorm ? 4 : 2, 32);
  __shared__ __align__(16) char rings[kRopeWarps][kDepth * kStage];
  __shared__ float4 cs[kRopeWarps][2][32];
  __shared__ float red[kRopeWarps][kD];
  int chunk, cta;
  const int part = part_of(a, chunk, cta);
  const RopePart& P = a.part[part];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, slot = lane / kLph;
  const int h0 = chunk * P.steps * kHpw + slot;
  const int hend = min(P.heads, (chunk + 1) * P.steps * kHpw);
  const uint32_t stride = P.ctas * kRopeWarps;
  const Lane l = lane_of<kHalves>(a, lane % kLph);
  uint32_t n = cta * kRopeWarps + warp;
  const T* g = static_cast<const T*>(P.g) + (long long)n * P.ldg;
  T* o = static_cast<T*>(P.o) + (long long)n * P.ldo;
  const long long dg = (long long)stride * P.ldg, dout = (long long)stride * P.ldo;
  if (part == 2) {
    for (; n < a.tokens; n += stride, g += dg, o += dout)
      copy_rows<T, T, kLph, kHalves>(g, o, l, h0, hend, P);
    return;
  }
  const T* x = kNorm ? static_cast<const T*>(P.x) + (long long)n * P.ldx : nullptr;
  const long long dx = (long long)stride * P.ldx;
  const uint32_t ring = shared_u32(rings[warp]);
  uint32_t fn = n;
  int fh = h0, to = 0;
  auto fetch = [&]() {
    if (fn < a.tokens) {
      const bool on = fh < hend;
      const int head = (on ? fh : 0) * kD;
      Slot<T>::fetch(ring + to, g + head + l.ea, 0, 32, lane, on);
      Slot<T>::fetch(ring + to, g + head + l.eb, 1, 32, lane, on);
      if (kNorm) {
        Slot<T>::fetch(ring + to, x + head + l.ea, 2, 32, lane, on);
        Slot<T>::fetch(ring + to, x + head + l.eb, 3, 32, lane, on);
      }
      fh += kHpw;
      if (fh - slot >= hend) {
        fh = h0;
        fn += stride;
        g += dg;
        if (kNorm) x += dx;
      }
    }
    copy_commit();
    to = to + kStage == kDepth * kStage ? 0 : to + kStage;
  };
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) fetch();
  Gather ang;
  ang.init(a, n, stride, lane, 32);
  f2 WA[4], WB[4], accA[4], accB[4];
  if (kNorm) weight16<kHalves>(P.w, a.w_bf16, 0, l, WA, WB);
#pragma unroll
  for (int i = 0; i < 4; ++i) accA[i] = accB[i] = pk(0.f, 0.f);
  const uint32_t rot = kNorm ? 0u : rotated<kHalves>(a, l);
  int from = 0, buf = 0;
  for (; n < a.tokens; n += stride, o += dout, buf ^= 1) {
    ang.put(cs[warp][buf], lane, 32);
    __syncwarp();
    ang.ahead(a);
    f2 C[4], S[4], N[4];  // N = -S
    angles_of(cs[warp][buf], l, C, S);
#pragma unroll
    for (int i = 0; i < 4; ++i) N[i] = neg2(S[i]);
    for (int h = h0; h - slot < hend; h += kHpw) {  // the same trip count for a warp
      fetch();
      copy_wait<kDepth - 1>();
      const char* at = rings[warp] + from;
      from = from + kStage == kDepth * kStage ? 0 : from + kStage;
      f2 A[4], B[4], GA[4], GB[4];
      Raw8<T> ra, rb;
      Slot<T>::take(at, 0, 32, lane, ra);
      Slot<T>::take(at, 1, 32, lane, rb);
      unpack16<kHalves>(ra, rb, A, B);
      if (kNorm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // turned back
          GA[i] = fma2(A[i], C[i], mul2(B[i], S[i]));
          GB[i] = fma2(B[i], C[i], mul2(A[i], N[i]));
        }
      } else {
        turn<kHalves>(A, B, C, N, S, rot);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          GA[i] = A[i];
          GB[i] = B[i];
        }
      }
      if (kNorm) {
        Slot<T>::take(at, 2, 32, lane, ra);
        Slot<T>::take(at, 3, 32, lane, rb);
        unpack16<kHalves>(ra, rb, A, B);
        f2 s0 = mul2(A[0], A[0]), s1 = mul2(B[0], B[0]);
        f2 d0 = mul2(A[0], mul2(GA[0], WA[0])), d1 = mul2(B[0], mul2(GB[0], WB[0]));
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          s0 = fma2(A[i], A[i], s0);
          s1 = fma2(B[i], B[i], s1);
          d0 = fma2(A[i], mul2(GA[i], WA[i]), d0);
          d1 = fma2(B[i], mul2(GB[i], WB[i]), d1);
        }
        const float2 s =
            lane_sum<kLph>(make_float2(sum2(add2(s0, s1)), sum2(add2(d0, d1))));
        const float r = rsqrtf(s.x * (1.f / kD) + a.eps);
        const float c = -s.y * (1.f / kD) * r * r * r;
        const f2 rr = pk(r, r), cc = pk(c, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 pA = mul2(GA[i], rr), pB = mul2(GB[i], rr);
          accA[i] = fma2(pA, A[i], accA[i]);
          accB[i] = fma2(pB, B[i], accB[i]);
          GA[i] = fma2(pA, WA[i], mul2(A[i], cc));
          GB[i] = fma2(pB, WB[i], mul2(B[i], cc));
        }
      }
      if (h < hend) pack16<kHalves>(o + h * kD, l, GA, GB);
    }
  }
  if (kNorm && P.part) {  // uniform over the CTA
    dependents_may_start();
    float fa[8], fb[8];
    order16<kHalves>(accA, accB, fa, fb);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int m = kLph; m < 32; m <<= 1) {
        fa[i] += __shfl_xor_sync(0xffffffffu, fa[i], m);
        fb[i] += __shfl_xor_sync(0xffffffffu, fb[i], m);
      }
      if (slot == 0) {
        red[warp][l.ea + i] = fa[i];
        red[warp][l.eb + i] = fb[i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < kD; c += kRopeThreads) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kRopeWarps; ++i) v += red[i][c];
      P.part[((long long)cta * P.chunks + chunk) * kD + c] = v;
    }
  }
}

// Norm over all heads of a token: a CTA takes a token's q or k, sixteen elements
// of a head kV times a thread, rows through a ring of asynchronous copies.  A
// token's angles are gathered by one thread a pair into shared memory and read
// behind the barrier that the row's sum needs anyway.  The weights' columns of a
// thread lie in shared memory too (fp32, read by that thread alone): in
// registers they would halve the CTAs of an SM.  Two groups of sixteen a thread
// beyond 2048 columns, fewer barriers and angles a value: 503 us for the 21 x 45 x 80
// clip with 40 heads of 128, one group 640; up to 2048 one, for more rows at a time:
// a clip of 14508 tokens with 12 query and 4 K/V heads 43 us, two groups 49 (33 since
// several teams share a CTA).  Four
// times the SMs in CTAs of each part (three are resident): 503 us, three times 517,
// six times 511.
constexpr int kCs = 5;  // kStages + 1 of bf16
struct TokenSmem {
  float2 red[2][32];
  float4 cs[kCs][32];  // two pairs' (cos, sin), a buffer a token
};

// A token's angles on their way to shared memory, a thread's two pairs, as part
// of the thread's next group of copies: forward, of the token whose row the group
// brings (kDepth - 1 ahead), read behind that token's barrier; backward, of the
// token after the next, read ahead of its own barrier and behind the one before,
// by which every thread has waited for its copies.  Either way a buffer is
// written anew only when the barrier of the token behind its last reader's has
// been passed: kDepth + 1 buffers forward, 3 backward.  Pairs that are not
// rotated are (1, 0) in every buffer from the start.
struct TokenAngles {
  Coord at;
  uint32_t spot[2];  // base of the pair in the table, axis in the two highest bits
  __device__ __forceinline__ void init(const RopeArgs& a, uint32_t n, uint32_t step, int tid,
                                       int threads, TokenSmem& sm) {
    at.init(a, n, step);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = tid + i * threads;
      const Spot s = spot_of(a, j < 64 ? j : -1);
      spot[i] = (uint32_t)s.base | (uint32_t)s.axis << 30;
      if (s.axis == 3 && j < 64) {
#pragma unroll
        for (int b = 0; b < kCs; ++b)
          reinterpret_cast<float2*>(sm.cs[b])[j] = make_float2(1.f, 0.f);
      }
    }
  }
  // Of the coordinates' token, which then move on to the next.
  __device__ __forceinline__ void fetch(const RopeArgs& a, TokenSmem& sm, int buf, int tid,
                                        int threads) {
    if (tid >= 64) return;  // at most 64 pairs: none of them this warp's
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t axis = spot[i] >> 30;
      if (axis != 3u) {
        const int off = axis == 0u ? (int)at.t * a.nt : axis == 1u ? (int)at.y * a.nh
                                                                   : (int)at.x * a.nw;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                         shared_u32(sm.cs[buf]) + (tid + i * threads) * 8),
                     "l"(a.table + (int)(spot[i] & 0x3fffffffu) + off)
                     : "memory");
      }
    }
    at.next(a);
  }
};
__device__ __forceinline__ int after(int cs) { return cs == kCs - 1 ? 0 : cs + 1; }

// A part with fewer heads than q needs fewer warps a token: a CTA then takes
// several tokens side by side, a team of warps each.
constexpr int kMaxTeams = 8;
static_assert(sizeof(TokenSmem) % 128 == 0, "stages begin at 128 bytes");
struct TokenTeam {
  int threads, id, count, tid;  // of a team, this team, teams of the CTA, thread of the team
  __device__ __forceinline__ TokenTeam(int units, int per_thread) {
    threads = min((int)blockDim.x, (units + 32 * per_thread - 1) / (32 * per_thread) * 32);
    count = min((int)blockDim.x / threads, kMaxTeams);
    id = threadIdx.x / threads;
    tid = threadIdx.x - id * threads;
  }
  __device__ __forceinline__ void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
  }
};
// Sums over a team, each warp's left in red and read by all behind the barrier.  One
// sum: teams of up to eight warps read all eight (zeros beyond the team's), wider
// ones exchange once more.  Two sums: always by exchanges, which need fewer
// registers (a spilled one costs the backward 18%).
__device__ __forceinline__ void clear_sums(TokenSmem& sm, const TokenTeam& t) {
  if (t.tid < 16) {
    const int b = t.tid >> 3, i = t.tid & 7;
    if (i >= t.threads >> 5) reinterpret_cast<float*>(sm.red[b])[i] = 0.f;
  }
}
__device__ __forceinline__ float2 part_sum(float2 v, TokenSmem& sm, int buf, const TokenTeam& t) {
  // the lanes of each half keep one of the two sums and hand on the other
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 16;
  float k = (hi ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, hi ? v.x : v.y, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
  float* red = reinterpret_cast<float*>(sm.red[buf]);
  if ((lane & 15) == 0) red[2 * (t.tid >> 5) + (lane >> 4)] = k;
  t.sync();
  k = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < t.threads >> 4) k += red[lane + 32 * i];
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
  return make_float2(__shfl_sync(0xffffffffu, k, 0), __shfl_sync(0xffffffffu, k, 1));
}
__device__ __forceinline__ float part_sum(float v, TokenSmem& sm, int buf, const TokenTeam& t) {
  v = lane_sum<32>(v);
  const int lane = threadIdx.x & 31;
  float* red = reinterpret_cast<float*>(sm.red[buf]);
  if (lane == 0) red[t.tid >> 5] = v;
  t.sync();
  if (t.threads <= 256) {
    const float4* w = reinterpret_cast<const float4*>(red);
    const float4 a = w[0], b = w[1];
    return sum2(add2(add2(pk(a.x, a.y), pk(a.z, a.w)), add2(pk(b.x, b.y), pk(b.z, b.w))));
  }
  return lane_sum<16>((lane & 15) < t.threads >> 5 ? red[lane & 15] : 0.f);
}

// A warp keeps its weights and its stages side by side in shared memory, 512 bytes a
// piece, sixteen a lane: every offset is a constant of the instruction.
// Weights: eight 16-byte pieces for each of a lane's kV groups of sixteen (A's,
// then B's).
__device__ __forceinline__ void put_weights(char* at, int j, int lane, const f2 (&A)[4],
                                            const f2 (&B)[4]) {
  ulonglong2* w = reinterpret_cast<ulonglong2*>(at) + j * 4 * 32 + lane;
  w[0] = make_ulonglong2(A[0], A[1]);
  w[32] = make_ulonglong2(A[2], A[3]);
  w[64] = make_ulonglong2(B[0], B[1]);
  w[96] = make_ulonglong2(B[2], B[3]);
}
// Group j's A (second = 0) or B (1).
__device__ __forceinline__ void get_weights(const char* at, int j, int second, int lane,
                                            f2 (&W)[4]) {
  const ulonglong2* w = reinterpret_cast<const ulonglong2*>(at) + (j * 4 + 2 * second) * 32 + lane;
  ulonglong2 v = w[0];
  W[0] = v.x;
  W[1] = v.y;
  v = w[32];
  W[2] = v.x;
  W[3] = v.y;
}
__host__ __device__ constexpr int weight_bytes(int kv, int threads) { return kv * threads * 64; }

template <typename TI, typename TO, int kV, bool kHalves>
__global__ void __launch_bounds__(512) rope_token_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(128) char dyn[];
  constexpr int kDepth = kStages<TI>;
  int chunk, cta;
  const int part = part_of(a, chunk, cta);
  const RopePart& P = a.part[part];
  const int lph = a.d / 16, units = P.heads * lph;
  const TokenTeam team(units, kV);
  if (team.id >= team.count) return;
  const int tid = team.tid, threads = team.threads;
  TokenSmem& sm = reinterpret_cast<TokenSmem*>(dyn)[team.id];
  const Lane l = lane_of<kHalves>(a, tid % lph);
  const int h0 = tid / lph * a.d, dh = threads / lph * a.d;  // a thread's heads, in elements
  const uint32_t stride = P.ctas * team.count;
  uint32_t n = cta * team.count + team.id, fn = n;
  if (n >= a.tokens) return;  // a whole team
  bool on[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) on[j] = j * threads + tid < units;
  constexpr int stage = Slot<TI>::bytes(2 * kV, 32);
  const int lane = tid & 31;
  char* weights = dyn + team.count * (int)sizeof(TokenSmem) +
                  (team.id * threads + tid) / 32 * (weight_bytes(kV, 32) + kDepth * stage);
  char* ring = weights + weight_bytes(kV, 32);
  const uint32_t ring_at = shared_u32(ring);
  int to = 0, from = 0;
  auto fetch = [&]() {
    if (fn < a.tokens) {
      const TI* x = static_cast<const TI*>(P.x) + (uint64_t)fn * (uint32_t)P.ldx;
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        const TI* head = x + (on[j] ? h0 + j * dh : 0);
        Slot<TI>::fetch(ring_at + to, head + l.ea, 2 * j, 32, lane, on[j]);
        Slot<TI>::fetch(ring_at + to, head + l.eb, 2 * j + 1, 32, lane, on[j]);
      }
      fn += stride;
    }
    copy_commit();
    to = to + stage == kDepth * stage ? 0 : to + stage;
  };
  auto take = [&](int j, f2(&A)[4], f2(&B)[4]) {
    Raw8<TI> ra, rb;
    Slot<TI>::take(ring + from, 2 * j, 32, lane, ra);
    Slot<TI>::take(ring + from, 2 * j + 1, 32, lane, rb);
    unpack16<kHalves>(ra, rb, A, B);
  };
  const float mul = sizeof(TO) == 1 ? P.mul : 1.f;
  if (part == 2) {
#pragma unroll
    for (int s = 0; s < kDepth - 1; ++s) fetch();
    for (; n < a.tokens; n += stride) {
      TO* o = static_cast<TO*>(P.o) + (uint64_t)n * (uint32_t)P.ldo + h0;
      fetch();
      copy_wait<kDepth - 1>();
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        f2 A[4], B[4];
        take(j, A, B);
        if (sizeof(TO) == 1) divide8(A, B, P);
        if (on[j]) pack16<kHalves>(o + j * dh, l, A, B);
      }
      from = from + stage == kDepth * stage ? 0 : from + stage;
    }
    return;
  }
  TokenAngles ang;
  ang.init(a, n, stride, tid, threads, sm);
  clear_sums(sm, team);
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) {
    ang.fetch(a, sm, s, tid, threads);
    fetch();
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    f2 A[4], B[4];
    weight16<kHalves>(on[j] ? P.w : nullptr, a.w_bf16, h0 + j * dh, l, A, B);
    put_weights(weights, j, lane, A, B);
  }
  int buf = 0, cs = 0, cs_to = kDepth - 1;
  for (; n < a.tokens; n += stride, buf ^= 1, cs = after(cs), cs_to = after(cs_to)) {
    copy_wait<kDepth - 2>();  // this token's row and angles
    ang.fetch(a, sm, cs_to, tid, threads);
    fetch();
    f2 A[kV][4], B[kV][4], s = pk(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      take(j, A[j], B[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(B[j][i], B[j][i], fma2(A[j][i], A[j][i], s));
    }
    from = from + stage == kDepth * stage ? 0 : from + stage;
    const float r = mul * rsqrtf(part_sum(sum2(s), sm, buf, team) * P.inv + a.eps);
    const f2 rr = pk(r, r);
    f2 C[4], S[4], N[4];  // N = -S
    angles_of(sm.cs[cs], l, C, S);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      C[i] = mul2(C[i], rr);
      N[i] = mul2(S[i], pk(-r, -r));
      S[i] = mul2(S[i], rr);
    }
    TO* o = static_cast<TO*>(P.o) + (uint64_t)n * (uint32_t)P.ldo + h0;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      f2 WA[4], WB[4];
      get_weights(weights, j, 0, lane, WA);
      get_weights(weights, j, 1, lane, WB);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 p = mul2(A[j][i], WA[i]), q = mul2(B[j][i], WB[i]);
        A[j][i] = fma2(p, C[i], mul2(q, N[i]));
        B[j][i] = fma2(q, C[i], mul2(p, S[i]));
      }
      if (on[j]) pack16<kHalves>(o + j * dh, l, A[j], B[j]);
    }
  }
}

// Backward of rope_token_kernel.  Both sums of a row (x^2 and w gn x) share one
// barrier; a thread's columns of the weight's gradient stay in registers over
// all its tokens and are left as one row of partial sums a team.  Up to 5120
// columns two CTAs of 320 threads share an SM without a spilled register (50 us
// for a clip of 14508 tokens with 12 query and 4 K/V heads of 128, first form 99); up
// to 8192 one CTA; beyond, 64 registers a thread and spills.  What bounds it there is
// latency, not HBM (31.7 us): a barrier and two exchanges a token of 3 KB, and each
// CTA's set-up.
template <typename T, int kThreads, int kCtas, bool kHalves>
__global__ void __launch_bounds__(kThreads, kCtas)
    rope_token_bwd_kernel(const __grid_constant__ RopeArgs a, int depth) {
  extern __shared__ __align__(128) char dyn[];
  int chunk, cta;
  const int part = part_of(a, chunk, cta);
  const RopePart& P = a.part[part];
  const int lph = a.d / 16;
  const TokenTeam team(P.heads * lph, 1);
  if (team.id >= team.count) return;
  const int tid = team.tid, threads = team.threads;
  TokenSmem& sm = reinterpret_cast<TokenSmem*>(dyn)[team.id];
  const Lane l = lane_of<kHalves>(a, tid % lph);
  const bool on = tid < P.heads * lph;
  const int h0 = on ? tid / lph * a.d : 0;
  const uint32_t stride = P.ctas * team.count;
  const uint32_t row = cta * team.count + team.id;  // of partial sums
  uint32_t n = row, fn = n;
  constexpr int stage = Slot<T>::bytes(4, 32);
  const int lane = tid & 31;
  char* weights = dyn + team.count * (int)sizeof(TokenSmem) +
                  (team.id * threads + tid) / 32 * (weight_bytes(1, 32) + depth * stage);
  char* ring = weights + weight_bytes(1, 32);
  const uint32_t ring_at = shared_u32(ring);
  int to = 0, from = 0;
  auto fetch = [&]() {
    if (fn < a.tokens) {
      const T* g = static_cast<const T*>(P.g) + (uint64_t)fn * (uint32_t)P.ldg + h0;
      Slot<T>::fetch(ring_at + to, g + l.ea, 0, 32, lane, on);
      Slot<T>::fetch(ring_at + to, g + l.eb, 1, 32, lane, on);
      if (part < 2) {
        const T* x = static_cast<const T*>(P.x) + (uint64_t)fn * (uint32_t)P.ldx + h0;
        Slot<T>::fetch(ring_at + to, x + l.ea, 2, 32, lane, on);
        Slot<T>::fetch(ring_at + to, x + l.eb, 3, 32, lane, on);
      }
      fn += stride;
    }
    copy_commit();
    to = depth == 2 ? stage - to : 0;
  };
  auto arrive = [&]() {  // the oldest row asked for
    if (depth == 2)
      copy_wait<1>();
    else
      copy_wait<0>();
  };
  auto take = [&](int j, f2(&A)[4], f2(&B)[4]) {
    Raw8<T> ra, rb;
    Slot<T>::take(ring + from, j, 32, lane, ra);
    Slot<T>::take(ring + from, j + 1, 32, lane, rb);
    unpack16<kHalves>(ra, rb, A, B);
  };
  if (part == 2) {
    if (depth == 2) fetch();
    for (; n < a.tokens; n += stride) {
      fetch();
      arrive();
      f2 A[4], B[4];
      take(0, A, B);
      from = depth == 2 ? stage - from : 0;
      if (on) pack16<kHalves>(static_cast<T*>(P.o) + (uint64_t)n * (uint32_t)P.ldo + h0, l, A, B);
    }
    return;
  }
  TokenAngles ang;
  ang.init(a, n, stride, tid, threads, sm);
  ang.fetch(a, sm, 0, tid, threads);
  ang.fetch(a, sm, 1, tid, threads);
  copy_commit();
  f2 accA[4], accB[4];
  {
    f2 A[4], B[4];
    weight16<kHalves>(on ? P.w : nullptr, a.w_bf16, h0, l, A, B);
    put_weights(weights, 0, lane, A, B);
#pragma unroll
    for (int i = 0; i < 4; ++i) accA[i] = accB[i] = pk(0.f, 0.f);
  }
  copy_wait<0>();
  team.sync();  // the first two tokens' angles
  if (depth == 2) fetch();
  int buf = 0, cs = 0;
  for (; n < a.tokens; n += stride, buf ^= 1, cs = after(cs)) {
    // the angles of the token after the next: every thread has waited for them
    // when it comes to the next token's barrier
    ang.fetch(a, sm, after(after(cs)), tid, threads);
    fetch();
    arrive();
    f2 XA[4], XB[4], GA[4], GB[4], s = pk(0.f, 0.f), d = s;
    {
      f2 C[4], S[4], A[4], B[4];
      angles_of(sm.cs[cs], l, C, S);
      take(0, A, B);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        GA[i] = fma2(A[i], C[i], mul2(B[i], S[i]));
        GB[i] = fma2(B[i], C[i], mul2(A[i], neg2(S[i])));
      }
      one_by_one();
      take(2, XA, XB);
#pragma unroll
      for (int i = 0; i < 4; ++i) s = fma2(XB[i], XB[i], fma2(XA[i], XA[i], s));
      one_by_one();
      get_weights(weights, 0, 0, lane, A);
#pragma unroll
      for (int i = 0; i < 4; ++i) d = fma2(XA[i], mul2(GA[i], A[i]), d);
      one_by_one();
      get_weights(weights, 0, 1, lane, B);
#pragma unroll
      for (int i = 0; i < 4; ++i) d = fma2(XB[i], mul2(GB[i], B[i]), d);
    }
    from = depth == 2 ? stage - from : 0;
    const float2 t = part_sum(make_float2(sum2(s), sum2(d)), sm, buf, team);
    const float inv = 1.f / (float)(P.heads * a.d);
    const float r = rsqrtf(t.x * inv + a.eps);
    const float c = -t.y * inv * r * r * r;
    const f2 rr = pk(r, r), cc = pk(c, c);
    f2 W[4];
    get_weights(weights, 0, 0, lane, W);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 p = mul2(GA[i], rr);
      accA[i] = fma2(p, XA[i], accA[i]);
      GA[i] = fma2(p, W[i], mul2(XA[i], cc));
    }
    one_by_one();
    get_weights(weights, 0, 1, lane, W);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 p = mul2(GB[i], rr);
      accB[i] = fma2(p, XB[i], accB[i]);
      GB[i] = fma2(p, W[i], mul2(XB[i], cc));
    }
    if (on) pack16<kHalves>(static_cast<T*>(P.o) + (uint64_t)n * (uint32_t)P.ldo + h0, l, GA, GB);
  }
  dependents_may_start();
  if (P.part && on)
    pack16<kHalves>(P.part + (long long)row * P.heads * a.d + h0, l, accA, accB);
}

// out[c] = sum over rows of part[row][c], for two matrices in one launch
// (blockIdx.y).  A CTA owns eight columns; 128 rows are read side by side and
// joined pairwise, in a fixed order, so equal calls give equal bits.
struct ColSum {
  const float* part;
  void* out;
  int rows, cols;
};
constexpr int kSumLanes = 128;
__global__ void __launch_bounds__(8 * kSumLanes) rope_colsum_kernel(ColSum s0, ColSum s1,
                                                                    int bf16) {
  __shared__ float red[kSumLanes / 4][8], red2[kSumLanes / 16][8];
  wait_for_partial_sums();
  const ColSum s = blockIdx.y ? s1 : s0;
  const int k = threadIdx.x & 7, lane = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 8 + k;
  if (blockIdx.x * 8 >= s.cols || !s.out) return;  // cols is a multiple of 8
  float v = 0.f;
#pragma unroll 8
  for (int r = lane; r < s.rows; r += kSumLanes) v += s.part[(long long)r * s.cols + c];
  auto over_warp = [](float x) {  // the warp's four rows
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
  };
  v = over_warp(v);
  if ((threadIdx.x & 31) < 8) red[warp][k] = v;
  __syncthreads();
  if (threadIdx.x < 2 * kSumLanes) {  // whole warps
    v = over_warp(red[lane][k]);
    if ((threadIdx.x & 31) < 8) red2[warp][k] = v;
  }
  __syncthreads();
  if (threadIdx.x < 8) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kSumLanes / 16; ++i) v += red2[i][k];
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
struct RopeDims {
  long long tokens;
  int heads[2];       // q, k
  long long pairs;
};

bool bad_factor(float f) { return !(f >= 0.f) || isinf(f); }
// Beyond these 1 / factor in two terms would leave fp32's normal numbers.
bool far_factor(float f) { return f > 0.f && (f < 0x1p-100f || f > 0x1p100f); }

basa_status check_rope(const basa_rope_params* p, bool bwd, RopeDims* r) {
  if (!p) return BASA_ERR_INVALID_ARG;
  if (p->B < 0 || p->T < 0 || p->Hg < 0 || p->Wg < 0 || p->H < 0 || p->d <= 0)
    return BASA_ERR_INVALID_ARG;
  if (p->Hkv < 0 || (p->Hkv > 0 && (p->H == 0 || p->H % p->Hkv != 0))) return BASA_ERR_INVALID_ARG;
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
  if (p->out_dtype == BASA_FP8_E4M3 &&
      (far_factor(p->q_descale) || far_factor(p->k_descale) || far_factor(p->v_descale)))
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

// Launch shape.  The CTAs of a part (q, k, v) number in proportion to its steps,
// so that all end together and none carries its set-up for a handful of steps.
struct RopeGrid {
  unsigned x;
  int threads, v;
  int ctas[3], chunks[3], steps[3];
  int teams;    // norm over a token: most teams of a CTA
  int rows[2];  // backward: rows of partial sums of q's and k's weights
};

RopeGrid rope_grid(const basa_rope_params* p, const RopeDims& r, bool with_v, bool bwd) {
  RopeGrid g;
  memset(&g, 0, sizeof(g));
  const int sms = row_sm_count();
  const int heads[3] = {r.heads[0], r.heads[1], r.heads[1]};
  if (p->norm == BASA_ROPE_NORM_TOKEN) {
    const int units = p->H * p->d / 16;  // H >= Hkv
    g.v = bwd || units <= 128 ? 1 : 2;
    g.threads = ((units + g.v - 1) / g.v + 31) / 32 * 32;
    // Several teams to a CTA where one is a few warps: CTAs of a warp or two come and
    // go one by one, and a few CTAs of many warps spread over an SM more evenly.  4800
    // tokens of 8 heads of 64, one team to a CTA and several: 34.8 and 12.3 us, backward
    // 34.9 and 20.5; 14508 tokens with 12 query and 4 K/V heads of 128: 41.0 and 32.8,
    // backward 57.4 and 51.0.
    const int most = bwd ? 192 : 256;
    int q_teams = g.threads < most ? most / g.threads : 1;
    if (q_teams > kMaxTeams) q_teams = kMaxTeams;
    g.threads *= q_teams;
    // Threads of a part on an SM at a time.  Forward, at the 14508 tokens above (one
    // team to a CTA), 640 against 960 and 1280: 41.0, 43.6 and 47.1 us; backward, where
    // more leave more rows of partial sums, 384 against 192 and 576: 51.0, 70.5, 56.1.
    int per_sm = (bwd ? 384 : 640) / g.threads;
    if (per_sm < 1) per_sm = 1;
    for (int i = 0; i < (with_v ? 3 : 2); ++i) {
      const int threads = ((heads[i] * p->d / 16 + g.v - 1) / g.v + 31) / 32 * 32;
      int teams = g.threads / threads;
      if (teams > kMaxTeams) teams = kMaxTeams;
      if (teams > g.teams) g.teams = teams;
      const long long need = (r.tokens + teams - 1) / teams;
      long long ctas = (long long)sms * per_sm * q_teams / teams;
      if (ctas < sms) ctas = sms;
      g.ctas[i] = (int)(need < ctas ? need : ctas);
      g.chunks[i] = 1;
      g.x += g.ctas[i];
      if (i < 2) g.rows[i] = g.ctas[i] * teams;
    }
    return g;
  }
  const int hpw = 512 / p->d;
  g.threads = kRopeThreads;
  int all = 0;
  for (int i = 0; i < (with_v ? 3 : 2); ++i) {
    const int steps = (heads[i] + hpw - 1) / hpw;
    const int want = (steps + 7) / 8;
    g.steps[i] = (steps + want - 1) / want;
    g.chunks[i] = (steps + g.steps[i] - 1) / g.steps[i];
    all += g.steps[i] * g.chunks[i];
  }
  const long long need = (r.tokens + kRopeWarps - 1) / kRopeWarps;
  // Forward, a warp takes as many tokens as make six steps, so long as the SMs have
  // several CTAs each to choose from (budgets of 5, 20 and 40 CTAs an SM were slower
  // than 10); backward, as few CTAs as balance, since each leaves a row of partial
  // sums.
  const long long budget = (long long)sms * (bwd ? 12 : 10);
  for (int i = 0; i < (with_v ? 3 : 2); ++i) {
    const long long ctas = (budget * g.steps[i] + all - 1) / all;
    long long each = need / ctas > 1 ? need / ctas : 1;  // tokens of a warp, for all alike
    const long long most = (5 + g.steps[i]) / g.steps[i];
    if (!bwd && each > most) each = most;
    g.ctas[i] = (int)((need + each - 1) / each);
    g.x += g.ctas[i] * g.chunks[i];
    if (i < 2) g.rows[i] = g.ctas[i] * g.chunks[i];
  }
  return g;
}

size_t rope_part_bytes(const basa_rope_params* p, const RopeDims& r, const RopeGrid& g, int i) {
  const size_t cols = p->norm == BASA_ROPE_NORM_TOKEN ? (size_t)r.heads[i] * p->d : (size_t)p->d;
  return up256((size_t)g.rows[i] * cols * sizeof(float));
}

template <typename TI, typename TO, int kLph>
void go_head(const RopeGrid& g, const RopeArgs& a, bool halves, bool norm, cudaStream_t st) {
  const dim3 grid(g.x);
  if (halves && norm) rope_head_kernel<TI, TO, kLph, true, true><<<grid, kRopeThreads, 0, st>>>(a);
  else if (halves) rope_head_kernel<TI, TO, kLph, true, false><<<grid, kRopeThreads, 0, st>>>(a);
  else if (norm) rope_head_kernel<TI, TO, kLph, false, true><<<grid, kRopeThreads, 0, st>>>(a);
  else rope_head_kernel<TI, TO, kLph, false, false><<<grid, kRopeThreads, 0, st>>>(a);
}
template <typename T, int kLph>
void go_head_bwd(const RopeGrid& g, const RopeArgs& a, bool halves, bool norm, cudaStream_t st) {
  const dim3 grid(g.x);
  if (halves && norm) rope_head_bwd_kernel<T, kLph, true, true><<<grid, kRopeThreads, 0, st>>>(a);
  else if (halves) rope_head_bwd_kernel<T, kLph, true, false><<<grid, kRopeThreads, 0, st>>>(a);
  else if (norm) rope_head_bwd_kernel<T, kLph, false, true><<<grid, kRopeThreads, 0, st>>>(a);
  else rope_head_bwd_kernel<T, kLph, false, false><<<grid, kRopeThreads, 0, st>>>(a);
}
template <typename K, typename... Args>
bool go_token(K kernel, const RopeGrid& g, int smem, cudaStream_t st, const Args&... args) {
  if (!allow_smem(kernel, smem)) return false;
  kernel<<<g.x, g.threads, smem, st>>>(args...);
  return true;
}
template <typename TI, typename TO>
bool go_fwd(const basa_rope_params* p, const RopeGrid& g, const RopeArgs& a, cudaStream_t st) {
  const bool halves = p->layout == BASA_ROPE_HALVES;
  if (p->norm == BASA_ROPE_NORM_TOKEN) {
    const int smem = g.teams * (int)sizeof(TokenSmem) + weight_bytes(g.v, g.threads) +
                     kStages<TI> * Slot<TI>::bytes(2 * g.v, g.threads);
    if (g.v == 1)
      return halves ? go_token(rope_token_kernel<TI, TO, 1, true>, g, smem, st, a)
                    : go_token(rope_token_kernel<TI, TO, 1, false>, g, smem, st, a);
    return halves ? go_token(rope_token_kernel<TI, TO, 2, true>, g, smem, st, a)
                  : go_token(rope_token_kernel<TI, TO, 2, false>, g, smem, st, a);
  }
  const bool norm = p->norm != BASA_ROPE_NORM_NONE;
  if (p->d == 128) go_head<TI, TO, 8>(g, a, halves, norm, st);
  else if (p->d == 64) go_head<TI, TO, 4>(g, a, halves, norm, st);
  else go_head<TI, TO, 2>(g, a, halves, norm, st);
  return true;
}
template <typename T>
bool go_bwd(const basa_rope_params* p, const RopeGrid& g, const RopeArgs& a, cudaStream_t st) {
  const bool halves = p->layout == BASA_ROPE_HALVES;
  if (p->norm == BASA_ROPE_NORM_TOKEN) {
    const int w = g.teams * (int)sizeof(TokenSmem) + weight_bytes(1, g.threads);
    const int stage = Slot<T>::bytes(4, g.threads);
    const int depth = w + 2 * stage <= kMostSmem ? 2 : 1;  // fp32 rows of over 11 K values: 1
    const int smem = w + depth * stage;
    if (g.threads <= 320)
      return halves ? go_token(rope_token_bwd_kernel<T, 320, 2, true>, g, smem, st, a, depth)
                    : go_token(rope_token_bwd_kernel<T, 320, 2, false>, g, smem, st, a, depth);
    if (g.threads <= 512)
      return halves ? go_token(rope_token_bwd_kernel<T, 512, 1, true>, g, smem, st, a, depth)
                    : go_token(rope_token_bwd_kernel<T, 512, 1, false>, g, smem, st, a, depth);
    return halves ? go_token(rope_token_bwd_kernel<T, 1024, 1, true>, g, smem, st, a, depth)
                  : go_token(rope_token_bwd_kernel<T, 1024, 1, false>, g, smem, st, a, depth);
  }
  const bool norm = p->norm != BASA_ROPE_NORM_NONE;
  if (p->d == 128) go_head_bwd<T, 8>(g, a, halves, norm, st);
  else if (p->d == 64) go_head_bwd<T, 4>(g, a, halves, norm, st);
  else go_head_bwd<T, 2>(g, a, halves, norm, st);
  return true;
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
  const int64_t in[3] = {p->ldq, p->ldk, p->ldv}, gr[3] = {p->ldgq, p->ldgk, p->ldgv};
  const float ds[3] = {p->q_descale, p->k_descale, p->v_descale};
  for (int i = 0; i < 3; ++i) {
    const int j = i > 0;
    const long long row = (long long)r.heads[j] * p->d;
    a.part[i].heads = r.heads[j];
    a.part[i].ctas = g.ctas[i];
    a.part[i].chunks = g.chunks[i];
    a.part[i].steps = g.steps[i];
    a.part[i].ldx = in[i] ? in[i] : row;
    a.part[i].ldg = row;
    a.part[i].ldo = bwd && gr[i] ? gr[i] : row;
    a.part[i].inv = 1.f / (float)row;
    const double inv = 1.0 / (ds[i] > 0.f ? (double)ds[i] : 1.0);
    float mul = (float)inv;
    const bool two_terms = i == 2 || p->norm == BASA_ROPE_NORM_NONE;
    if (two_terms && (double)mul > inv) mul = nextafterf(mul, 0.f);
    const float rest = (float)(inv - (double)mul);
    a.part[i].mul = mul;
    a.part[i].rest = rest > 0.f ? rest : 1e-45f;
  }
  return a;
}

int size_of(int dtype) { return dtype == BASA_F32 ? 4 : dtype == BASA_BF16 ? 2 : 1; }
// q, k, v (or their gradients): rows of tensor i at ld elements, 0 = dense.
struct RopeRows {
  long long tokens, row[3], ld[3];  // bytes
  RopeRows(const basa_rope_params* p, const RopeDims& r, int dtype, int64_t lq, int64_t lk, int64_t lv) {
    const int64_t l[3] = {lq, lk, lv};
    tokens = r.tokens;
    for (int i = 0; i < 3; ++i) {
      row[i] = (long long)r.heads[i > 0] * p->d * size_of(dtype);
      ld[i] = l[i] ? l[i] * size_of(dtype) : row[i];
    }
  }
  bool dense(int i) const { return ld[i] == row[i] || tokens == 1; }
};
void add_weights(Overlap& o, const basa_rope_params* p, const RopeDims& r, const void* qw, const void* kw,
                 const void* table, bool out) {
  const void* w[2] = {qw, kw};
  for (int i = 0; i < 2; ++i)
    o.add(w[i], 1, (long long)(p->norm == BASA_ROPE_NORM_TOKEN ? r.heads[i] : 1) * p->d * size_of(p->w_dtype), 0,
          out, nullptr);
  if (r.pairs) o.in(table, r.pairs * 8);
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
  {
    Overlap o;
    const RopeRows from(p, r, p->dtype, p->ldq, p->ldk, p->ldv), to(p, r, p->out_dtype, 0, 0, 0);
    const void *x[3] = {q, k, v}, *y[3] = {q_out, k_out, v_out};
    for (int i = 0; i < 3; ++i) {
      o.in(x[i], r.tokens, from.row[i], from.ld[i]);
      o.out(y[i], r.tokens, to.row[i], to.ld[i],
            p->out_dtype == p->dtype && from.dense(i) ? x[i] : nullptr);
    }
    add_weights(o, p, r, q_weight, k_weight, table, false);
    if (o.any()) return BASA_ERR_INVALID_ARG;
  }
  const RopeGrid g = rope_grid(p, r, v != nullptr, false);
  RopeArgs a = rope_args(p, r, g, table, false);
  a.part[0].x = q; a.part[1].x = k; a.part[2].x = v;
  a.part[0].w = q_weight; a.part[1].w = k_weight;
  a.part[0].o = q_out; a.part[1].o = k_out; a.part[2].o = v_out;
  const bool low = p->out_dtype == BASA_FP8_E4M3;
  const bool ok = p->dtype == BASA_BF16
                      ? (low ? go_fwd<__nv_bfloat16, e4m3_t>(p, g, a, stream)
                             : go_fwd<__nv_bfloat16, __nv_bfloat16>(p, g, a, stream))
                      : (low ? go_fwd<float, e4m3_t>(p, g, a, stream)
                             : go_fwd<float, float>(p, g, a, stream));
  const basa_status l = launched();
  return ok ? l : BASA_ERR_CUDA;
}

size_t basa_qkv_rope_bwd_workspace_size(const basa_rope_params* p) {
  RopeDims r;
  if (check_rope(p, true, &r) != BASA_OK || p->norm == BASA_ROPE_NORM_NONE ||
      r.tokens * p->H == 0)
    return 0;
  size_t n = 0;
  for (int v = 0; v < 2; ++v) {  // with and without v
    const RopeGrid g = rope_grid(p, r, v != 0, true);
    const size_t m = rope_part_bytes(p, r, g, 0) + rope_part_bytes(p, r, g, 1);
    n = m > n ? m : n;
  }
  return n;
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
  const RopeGrid g = rope_grid(p, r, dv != nullptr, true);
  {
    Overlap o;
    const RopeRows x(p, r, p->dtype, p->ldq, p->ldk, p->ldv), go(p, r, p->dtype, 0, 0, 0),
        gx(p, r, p->dtype, p->ldgq, p->ldgk, p->ldgv);
    const void *in[3] = {q, k, nullptr}, *from[3] = {dq_out, dk_out, dv_out}, *to[3] = {dq, dk, dv};
    for (int i = 0; i < 3; ++i) {
      if (norm) o.in(in[i], r.tokens, x.row[i], x.ld[i]);
      o.in(from[i], r.tokens, go.row[i], go.ld[i]);
      o.out(to[i], r.tokens, gx.row[i], gx.ld[i], gx.dense(i) ? from[i] : nullptr);
    }
    add_weights(o, p, r, q_weight, k_weight, table, false);
    add_weights(o, p, r, dq_weight, dk_weight, nullptr, true);
    if (sums) o.out(workspace, (long long)(rope_part_bytes(p, r, g, 0) + rope_part_bytes(p, r, g, 1)));
    if (o.any()) return BASA_ERR_INVALID_ARG;
  }
  RopeArgs a = rope_args(p, r, g, table, true);
  a.part[0].x = q; a.part[1].x = k;
  a.part[0].g = dq_out; a.part[1].g = dk_out; a.part[2].g = dv_out;
  a.part[0].w = q_weight; a.part[1].w = k_weight;
  a.part[0].o = dq; a.part[1].o = dk; a.part[2].o = dv;
  char* ws = static_cast<char*>(workspace);
  if (dq_weight) a.part[0].part = reinterpret_cast<float*>(ws);
  if (dk_weight) a.part[1].part = reinterpret_cast<float*>(ws + rope_part_bytes(p, r, g, 0));
  const bool ok = p->dtype == BASA_BF16 ? go_bwd<__nv_bfloat16>(p, g, a, stream)
                                        : go_bwd<float>(p, g, a, stream);
  if ((s = launched()) != BASA_OK || !ok) return BASA_ERR_CUDA;
  if (sums) {
    const ColSum c0{a.part[0].part, dq_weight, g.rows[0], cols[0]};
    const ColSum c1{a.part[1].part, dk_weight, g.rows[1], cols[1]};
    return launch_dependent(rope_colsum_kernel, dim3((unsigned)(cols[0] / 8), 2), 8 * kSumLanes, stream, c0,
                            c1, (int)(p->w_dtype == BASA_BF16));
  }
  return BASA_OK;
}

}  // extern "C"
