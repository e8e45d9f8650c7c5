// AdamW over many tensors in one launch (decoupled decay):
//   g = grad * scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
// Bound by its bytes: 28 an element with bfloat16 weights and gradients, float32
// masters and moments (60M elements 253 us, 98% of the measured copy rate); 14 with
// float32 weights, bfloat16 gradients and 8-bit moments (120M elements 297 us, 84%:
// the codes' instructions).  Many small tensors: the host, whose
// checks take 0.1 us a tensor.
//
// The tensors' addresses travel as kernel parameters: no table in device memory,
// nothing to copy, and a captured call replays as it was.  The tensors are cut into
// pieces, a warp takes one; a block takes a run of pieces, so that it looks its first
// tensor up once and then walks on.  256 elements, eight a lane, are a block of the
// 8-bit states: its largest value is one redux.sync.  With 8-bit states a piece is
// eight blocks where there are enough of them: their scales are then one 32-byte
// sector, read and written once (one scale at a time, each 4-byte store into a sector
// held the loads of its neighbours up: 348 us for 120M elements, 265 without scales).
// Reading the next block ahead, into registers or shared memory, gave nothing: 32
// warps an SM hide the loads.
//
// 8-bit moments: m and sqrt(v) as e4m3 codes times a float32 scale for each 256
// elements of a tensor (largest magnitude / 448).  Rounding to nearest would never
// move a second moment whose change in one step is smaller than half a code (one in a
// thousand against one in sixteen); instead an element's rounding threshold walks a
// Weyl sequence over the steps, (index * A + t * B + salt) mod 2^32 over 2^32, so
// that in the mean over steps nothing is lost: sqrt(v) of gradients of constant size
// is off by 15% (root mean square) and 0.5% on average at b2 = 0.999, 22% and 9%
// rounded to nearest.  sqrt(v), not v: half the exponents.  A sqrt(v) that is not zero
// does not become zero (m / eps would follow).
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mgg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kFew = 24, kMany = 400;  // tensors of a launch, by parameter size
constexpr int kGroups = 128;
constexpr uint32_t kWalkI = 0x9E3779B1u, kWalkT = 0xC13FA9A9u, kSaltV = 0x80000000u;

struct Entry {
  void* p;
  float* master;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  long long n;
  int wide;  // every address allows vectors of eight elements
};
template <int N>
struct AdamwParams {
  int count, pieces;
  int span;                   // blocks of 256 elements in a piece
  float b1, c1, b2, c2, eps;  // c: 1 - b
  float lr, decay;            // lr where lr_dev is null; weight decay
  double lnb1, lnb2;
  long long step;
  const float* lr_dev;
  const int32_t* step_dev;
  const float* grad_scale;
  // Each block reads these at its start, one after the other, from memory (they are
  // cold): the tensor that holds the first piece of its group of blocks, then the
  // tensors' first pieces from there on.
  unsigned short hint[kGroups];
  int first[N + 1];
  Entry e[N];
};
static_assert(sizeof(AdamwParams<kMany>) <= 32764, "kernel parameters");

__device__ __forceinline__ void bf16s(const uint4& q, float (&v)[8]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
// Eight elements from i on, `wide` as one access, else those below n, 32 apart.
template <bool WIDE>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  static_assert(WIDE, "");
  asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                 "=f"(v[7])
               : "l"(p));
}
template <bool WIDE>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  static_assert(WIDE, "");
  bf16s(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                                            cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
}
template <bool WIDE, typename T>
__device__ __forceinline__ void get(const T* base, long long i, long long n, float (&v)[8]) {
  if constexpr (WIDE) {
    load8<true>(base + i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + 32 * j < n ? static_cast<float>(base[i + 32 * j]) : 0.f;
  }
}
template <bool WIDE, typename T>
__device__ __forceinline__ void put(T* base, long long i, long long n, const float (&v)[8]) {
  if constexpr (WIDE) {
    store8(base + i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + 32 * j < n) base[i + 32 * j] = static_cast<T>(v[j]);
  }
}

// ---------------------------------------------------------------- 8-bit states
// Two e4m3 codes (low half) as floats.
__device__ __forceinline__ void decode2(uint32_t c, float& a, float& b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(c)));
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}\n"
      : "=f"(a), "=f"(b)
      : "r"(h));
}
// Eight codes, as they lie (WIDE) or gathered.
template <bool WIDE>
__device__ __forceinline__ uint2 get_codes(const void* base, long long i, long long n) {
  const uint8_t* q = static_cast<const uint8_t*>(base);
  if constexpr (WIDE) {
    return *reinterpret_cast<const uint2*>(q + i);
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + 32 * j < n) w[j / 4] |= static_cast<uint32_t>(q[i + 32 * j]) << (8 * (j % 4));
    return make_uint2(w[0], w[1]);
  }
}
__device__ __forceinline__ void decode8(uint2 w, float scale, float (&v)[8]) {
  decode2(w.x, v[0], v[1]);
  decode2(w.x >> 16, v[2], v[3]);
  decode2(w.y, v[4], v[5]);
  decode2(w.y >> 16, v[6], v[7]);
#pragma unroll
  for (int j = 0; j < 8; j += 2) unpack2(mul2(pack2(v[j], v[j + 1]), both(scale)), v[j], v[j + 1]);
}
// The largest magnitudes of a block's moments m and r (its root, not negative).  odd:
// a value is not finite, and the largest are those of the others (an element that is
// not finite becomes NaN and leaves its neighbours alone); of m its sum tells.
__device__ __forceinline__ bool largest(const float (&m)[8], const float (&r)[8], float& tm, float& tr) {
  uint32_t top = 0;
  tm = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    top = max(top, __float_as_uint(r[j]));  // (as whole numbers, which keep NaN)
    tm = fmaxf(tm, fabsf(m[j]));
  }
  float s0, s1;
  unpack2(add2(add2(pack2(m[0], m[1]), pack2(m[2], m[3])), add2(pack2(m[4], m[5]), pack2(m[6], m[7]))), s0, s1);
  if (!isfinite(s0 + s1)) top = 0xffffffffu;
  top = __reduce_max_sync(0xffffffffu, top);
  const bool odd = top >= 0x7f800000u;  // (the same in every lane)
  if (odd) {
    top = 0, tm = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (__float_as_uint(r[j]) < 0x7f800000u) top = max(top, __float_as_uint(r[j]));
      if (isfinite(m[j])) tm = fmaxf(tm, fabsf(m[j]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  tr = __uint_as_float(top);
  tm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(tm)));
  return odd;
}
// v's codes: |v| / scale as the bits of a number with four exponent and three
// mantissa bits (times 2^-120, so that e4m3's denormals are float's), 20 bits below
// them, the threshold's 20 bits added, cut off.  The code's eight bits are left on
// the top byte and gathered from there.
template <bool ROOT, bool ONE>
__device__ __forceinline__ uint2 codes(float inv, float tiny, bool odd, const uint32_t (&walk)[8],
                                       const float (&v)[8]) {
  uint32_t b[8], c[8], low = 0xffffffffu;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float y0, y1;
    if (ONE && ROOT) {
      unpack2(mul2(pack2(v[j], v[j + 1]), both(tiny)), y0, y1);
    } else if (ONE) {
      y0 = fabsf(v[j]) * tiny, y1 = fabsf(v[j + 1]) * tiny;
    } else {
      y0 = (fabsf(v[j]) * inv) * 0x1p-120f, y1 = (fabsf(v[j + 1]) * inv) * 0x1p-120f;
    }
    b[j] = __float_as_uint(y0), b[j + 1] = __float_as_uint(y1);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (ROOT) low = min(low, b[j]);
    c[j] = min(walk[j] + b[j], 0x07efffffu);
  }
  if (ROOT && __any_sync(0xffffffffu, low < 0x100000u)) {  // (a root below one code)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (b[j]) c[j] = max(c[j], 0x100000u);
  }
  if (odd) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((__float_as_uint(v[j]) & 0x7fffffffu) >= 0x7f800000u) c[j] = 0x07f00000u;
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t* q = c + 4 * h;
    const uint32_t lo = __byte_perm(q[0] << 4, q[1] << 4, 0x0073), hi = __byte_perm(q[2] << 4, q[3] << 4, 0x0073);
    w[h] = __byte_perm(lo, hi, 0x5410) & 0x7f7f7f7fu;
    if (!ROOT) {
      const float* f = v + 4 * h;
      const uint32_t s0 = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0073),
                     s1 = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0073);
      w[h] |= __byte_perm(s0, s1, 0x5410) & 0x80808080u;
    }
  }
  return make_uint2(w[0], w[1]);
}
template <bool WIDE, bool ROOT>
__device__ __forceinline__ void put_codes(void* base, long long i, long long n, float inv, bool odd,
                                          const uint32_t (&walk)[8], const float (&v)[8]) {
  // one product where the factor is a normal number (up to 28672 as the largest)
  const float tiny = inv * 0x1p-120f;
  const uint2 w = tiny >= 0x1p-126f || inv == 0.f ? codes<ROOT, true>(inv, tiny, odd, walk, v)
                                                  : codes<ROOT, false>(inv, tiny, odd, walk, v);
  uint8_t* q = static_cast<uint8_t*>(base);
  if constexpr (WIDE) {
    *reinterpret_cast<uint2*>(q + i) = w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + 32 * j < n) q[i + 32 * j] = static_cast<uint8_t>((j < 4 ? w.x : w.y) >> (8 * (j % 4)));
  }
}
// Both moments' codes; returns their scales in lanes 0 and 1.  The four divisions (a
// scale and its inverse each) are one: lanes 0 to 3 take one each.
template <bool WIDE>
__device__ __forceinline__ float put_moments(const Entry& e, long long i, uint32_t walk, const float (&m)[8],
                                             const float (&r)[8]) {
  float tm, tr;
  const bool odd = largest(m, r, tm, tr);
  const int lane = threadIdx.x & 31;
  const float t = lane & 1 ? tr : tm;
  const float q = __fdiv_rn(lane & 2 ? 448.f : t, lane & 2 ? t : 448.f);
  float im = __shfl_sync(0xffffffffu, q, 2), ir = __shfl_sync(0xffffffffu, q, 3);
  im = tm > 0x1p-110f ? im : 0.f;
  ir = tr > 0x1p-110f ? ir : 0.f;
  // the thresholds' 20 bits; the salt turns the first of them
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = (walk + static_cast<uint32_t>(WIDE ? j : 32 * j) * kWalkI) >> 12;
  put_codes<WIDE, false>(e.m, i, e.n, im, odd, w, m);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] ^= kSaltV >> 12;
  put_codes<WIDE, true>(e.v, i, e.n, ir, odd, w, r);
  return q;
}

// ---------------------------------------------------------------- the step
// One instruction each, within 2 ulp; a second moment below 1e-38 counts as 0 here.
__device__ __forceinline__ float root(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float inverse(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// a + b, each rounded by itself.  (add2 of two products is contracted to fma2.)
__device__ __forceinline__ F2 sum2(F2 a, F2 b) {
  float a0, a1, b0, b1;
  unpack2(a, a0, a1);
  unpack2(b, b0, b1);
  return pack2(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}
struct Rates {
  float b1, c1, b2, c2, eps, keep, rate, root, gs;
  uint32_t walk;
};

// Eight elements of this lane, of the warp's 256 from `at` on: what is read, then
// the step on it.
template <typename P, typename G, bool MASTER, bool BITS8>
struct Held {
  float p[8], g[8], m[8], v[8];
  uint4 gc;  // eight bfloat16 gradients as they lie
  uint2 mc, vc;
  template <bool WIDE>
  __device__ __forceinline__ void read(const Entry& e, long long at) {
    const int lane = threadIdx.x & 31;
    const long long i = at + (WIDE ? 8 * lane : lane), n = e.n;
    if constexpr (WIDE && sizeof(G) == 2)
      gc = *reinterpret_cast<const uint4*>(static_cast<const G*>(e.g) + i);
    else
      get<WIDE>(static_cast<const G*>(e.g), i, n, g);
    if constexpr (MASTER)
      get<WIDE>(static_cast<const float*>(e.master), i, n, p);
    else
      get<WIDE>(static_cast<const P*>(e.p), i, n, p);
    if constexpr (BITS8) {
      mc = get_codes<WIDE>(e.m, i, n), vc = get_codes<WIDE>(e.v, i, n);
    } else {
      get<WIDE>(static_cast<const float*>(e.m), i, n, m);
      get<WIDE>(static_cast<const float*>(e.v), i, n, v);
    }
  }
  // ms, vs: the block's scales; returns the new ones in lanes 0 and 1
  template <bool WIDE>
  __device__ __forceinline__ float step(const Entry& e, long long at, const Rates& r, float ms, float vs) {
    const int lane = threadIdx.x & 31;
    const long long i = at + (WIDE ? 8 * lane : lane), n = e.n;
    if constexpr (WIDE && sizeof(G) == 2) bf16s(gc, g);
    if constexpr (BITS8) {
      decode8(mc, ms, m);
      decode8(vc, vs, v);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const F2 x = mul2(pack2(g[j], g[j + 1]), both(r.gs));
      F2 mm = mul2(pack2(m[j], m[j + 1]), both(r.b1)), vv = pack2(v[j], v[j + 1]);
      float v0, v1, r0, r1, d0, d1, p0, p1;
      if constexpr (BITS8) {
        // each operation rounded by itself, as the formula is written: the codes are
        // then the same wherever they are computed in f32
        mm = sum2(mm, mul2(x, both(r.c1)));
        vv = sum2(mul2(mul2(vv, vv), both(r.b2)), mul2(mul2(x, x), both(r.c2)));
        unpack2(vv, v0, v1);
        r0 = __fsqrt_rn(v0), r1 = __fsqrt_rn(v1);
      } else {
        mm = fma2(x, both(r.c1), mm);
        vv = fma2(mul2(x, x), both(r.c2), mul2(vv, both(r.b2)));
        unpack2(vv, v0, v1);
        r0 = root(v0), r1 = root(v1);
      }
      unpack2(fma2(pack2(r0, r1), both(r.root), both(r.eps)), d0, d1);
      const F2 u = mul2(mm, pack2(inverse(d0), inverse(d1)));
      unpack2(fma2(both(-r.rate), u, mul2(pack2(p[j], p[j + 1]), both(r.keep))), p0, p1);
      p[j] = p0, p[j + 1] = p1;
      unpack2(mm, m[j], m[j + 1]);
      v[j] = BITS8 ? r0 : v0, v[j + 1] = BITS8 ? r1 : v1;
    }
    if constexpr (MASTER) put<WIDE>(e.master, i, n, p);
    put<WIDE>(static_cast<P*>(e.p), i, n, p);
    if constexpr (BITS8) {
      return put_moments<WIDE>(e, i, r.walk + static_cast<uint32_t>(i) * kWalkI, m, v);
    } else {
      put<WIDE>(static_cast<float*>(e.m), i, n, m);
      put<WIDE>(static_cast<float*>(e.v), i, n, v);
      return 0.f;
    }
  }
};

template <typename P, typename G, bool MASTER, bool BITS8, int N>
__global__ void __launch_bounds__(kThreads, BITS8 ? 4 : 3) adamw_kernel(const __grid_constant__ AdamwParams<N> a) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  const long long t = a.step_dev ? static_cast<long long>(*a.step_dev) : a.step;
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  // 1 - b^t = -expm1(t ln b): no cancellation in the first steps
  const float bc1 = -expm1f(static_cast<float>(static_cast<double>(t) * a.lnb1));
  const float bc2 = -expm1f(static_cast<float>(static_cast<double>(t) * a.lnb2));
  Rates r;
  r.b1 = a.b1, r.c1 = a.c1, r.b2 = a.b2, r.c2 = a.c2, r.eps = a.eps;
  r.keep = 1.f - lr * a.decay;
  r.rate = lr / bc1;
  r.root = rsqrtf(bc2);
  r.gs = a.grad_scale ? *a.grad_scale : 1.f;
  r.walk = static_cast<uint32_t>(t) * kWalkT;
  const int lo = static_cast<int>(static_cast<long long>(blockIdx.x) * a.pieces / gridDim.x);
  const int hi = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * a.pieces / gridDim.x);
  int k = a.hint[static_cast<int>(static_cast<long long>(blockIdx.x) * kGroups / gridDim.x)];
  const int lane = threadIdx.x & 31;
  Held<P, G, MASTER, BITS8> held;
  for (int piece = lo + warp; piece < hi; piece += kWarps) {
    while (a.first[k + 1] <= piece) ++k;
    const Entry e = a.e[k];
    long long at = static_cast<long long>(piece - a.first[k]) * a.span * 256;
    if constexpr (BITS8) {
      const int blocks = static_cast<int>(min(static_cast<long long>(a.span), (e.n - at + 255) >> 8));
      float ms = 0.f, vs = 0.f;  // the piece's scales, a lane each
      if (lane < blocks) ms = e.ms[(at >> 8) + lane], vs = e.vs[(at >> 8) + lane];
      const long long first = at >> 8;
      // lane b's scales become the ones that the step on block b returns
      auto renew = [&](int b, float q) {
        const float m = __shfl_sync(0xffffffffu, q, 0), v = __shfl_sync(0xffffffffu, q, 1);
        if (lane == b) ms = m, vs = v;
      };
      auto of = [&](float s, int b) { return __shfl_sync(0xffffffffu, s, b); };
      for (int b = 0; b < blocks; ++b, at += 256) {
        if (e.wide && at + 256 <= e.n) {
          held.template read<true>(e, at);
          renew(b, held.template step<true>(e, at, r, of(ms, b), of(vs, b)));
        } else {
          held.template read<false>(e, at);
          renew(b, held.template step<false>(e, at, r, of(ms, b), of(vs, b)));
        }
      }
      if (lane < blocks) e.ms[first + lane] = ms, e.vs[first + lane] = vs;
    } else if (e.wide && at + 256 <= e.n) {
      held.template read<true>(e, at);
      held.template step<true>(e, at, r, 0.f, 0.f);
    } else {
      held.template read<false>(e, at);
      held.template step<false>(e, at, r, 0.f, 0.f);
    }
  }
}

// ---------------------------------------------------------------- host
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <typename P, typename G, bool MASTER, bool BITS8, int N>
cudaError_t launch_n(const AdamwArgs& a, const AdamwParams<1>& common, int from, int count,
                     cudaStream_t st) {
  AdamwParams<N> p;
  p.count = 0;
  p.b1 = common.b1, p.c1 = common.c1, p.b2 = common.b2, p.c2 = common.c2, p.eps = common.eps;
  p.lr = common.lr, p.decay = common.decay, p.lnb1 = common.lnb1, p.lnb2 = common.lnb2;
  p.step = common.step, p.lr_dev = common.lr_dev, p.step_dev = common.step_dev;
  p.grad_scale = common.grad_scale;
  // a warp's piece: a block; eight (8-bit states) where that still leaves the GPU full
  long long all = 0;
  for (int i = from; i < from + count; ++i) all += (a.tensors[i].n + 255) >> 8;
  p.span = BITS8 && all >= 8LL * 32 * num_sms() ? 8 : 1;
  const long long piece = 256LL * p.span;
  long long pieces = 0;
  for (int i = from; i < from + count; ++i) {
    const mgg_adamw_tensor& t = a.tensors[i];
    if (t.n == 0) continue;
    Entry& e = p.e[p.count++];
    e.p = t.param, e.master = t.master, e.g = t.grad, e.m = t.exp_avg, e.v = t.exp_avg_sq;
    e.ms = t.exp_avg_scale, e.vs = t.exp_avg_sq_scale, e.n = t.n;
    p.first[p.count - 1] = static_cast<int>(pieces);
    e.wide = aligned(t.param, 8 * sizeof(P)) && aligned(t.grad, 8 * sizeof(G)) &&
             (!MASTER || aligned(t.master, 32)) && aligned(t.exp_avg, BITS8 ? 8 : 32) &&
             aligned(t.exp_avg_sq, BITS8 ? 8 : 32);
    pieces += (t.n + piece - 1) / piece;
  }
  if (pieces == 0) return cudaSuccess;
  if (pieces > 0x7fffffff) return cudaErrorInvalidValue;
  p.pieces = static_cast<int>(pieces);
  p.first[p.count] = p.pieces;
  const int blocks = static_cast<int>(std::min<long long>((pieces + kWarps - 1) / kWarps, 16LL * num_sms()));
  for (int g = 0, k = 0; g < kGroups; ++g) {
    // the first block b of the group has b * kGroups / blocks = g
    const long long b = (static_cast<long long>(g) * blocks + kGroups - 1) / kGroups;
    const long long at = b * pieces / blocks;
    while (k + 1 < p.count && p.first[k + 1] <= at) ++k;
    p.hint[g] = static_cast<unsigned short>(k);
  }
  return launch_pdl(adamw_kernel<P, G, MASTER, BITS8, N>, dim3(blocks), dim3(kThreads), 0, st, p);
}

template <typename P, typename G, bool MASTER, bool BITS8>
cudaError_t launch_t(const AdamwArgs& a, const AdamwParams<1>& common, cudaStream_t st) {
  if (a.count <= kFew) return launch_n<P, G, MASTER, BITS8, kFew>(a, common, 0, a.count, st);
  for (int from = 0; from < a.count; from += kMany) {
    const cudaError_t e =
        launch_n<P, G, MASTER, BITS8, kMany>(a, common, from, std::min(kMany, a.count - from), st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <typename P, bool MASTER>
cudaError_t launch_p(const AdamwArgs& a, const AdamwParams<1>& c, cudaStream_t st) {
  if (a.g_f32)
    return a.bits8 ? launch_t<P, float, MASTER, true>(a, c, st) : launch_t<P, float, MASTER, false>(a, c, st);
  return a.bits8 ? launch_t<P, __nv_bfloat16, MASTER, true>(a, c, st)
                 : launch_t<P, __nv_bfloat16, MASTER, false>(a, c, st);
}

}  // namespace

cudaError_t launch_adamw(const AdamwArgs& a, cudaStream_t st) {
  AdamwParams<1> c{};
  c.b1 = static_cast<float>(a.beta1), c.c1 = static_cast<float>(1.0 - a.beta1);
  c.b2 = static_cast<float>(a.beta2), c.c2 = static_cast<float>(1.0 - a.beta2);
  c.eps = static_cast<float>(a.eps), c.lr = static_cast<float>(a.lr), c.decay = static_cast<float>(a.decay);
  c.lnb1 = log(a.beta1), c.lnb2 = log(a.beta2);  // (-inf for 0: 1 - 0^t = 1)
  c.step = a.step, c.lr_dev = a.lr_dev, c.step_dev = a.step_dev, c.grad_scale = a.grad_scale;
  if (a.p_f32) return launch_p<float, false>(a, c, st);
  return a.master ? launch_p<__nv_bfloat16, true>(a, c, st) : launch_p<__nv_bfloat16, false>(a, c, st);
}

}  // namespace mgg
