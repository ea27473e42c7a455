// An AdamW step over many tensors at once, states in 32 bits or in FP8 blocks:
//
//   g  = factor * grad
//   m' = b1 m + (1 - b1) g,   v' = b2 v + (1 - b2) g^2
//   x' = x (1 - lr wd) - lr / (1 - b1^t) * m' / (sqrt(v' / (1 - b2^t)) + eps)
//
// x is the parameter, or its 32-bit master. The step t, and lr and factor where
// the caller wants, are read from device memory, so that a captured launch
// takes the next step each time it is replayed; where factor is not finite the
// launch changes nothing.
//
// In 8 bits a state is E4M3 codes with one E8M0 scale per 128 elements, and the
// second moment is held as its root, which halves the binades it spans. A step
// changes v by a fraction 1 - b2 of the difference, far less than half a step
// of E4M3 (2^-4): rounded to nearest it would stay where it is for good. So
// states, and 16-bit parameters without a master, are rounded up or down by a
// threshold u that runs through a Weyl sequence over steps and elements,
//   u = frac(i A + t B),   |x| -> step floor(|x| / step + u),
// whose values over consecutive steps are spread evenly: what is rounded away
// in some steps comes back in others, with less variance than random bits and
// no state of its own. A root that is not zero is not rounded to zero, which
// would make m' / (0 + eps) of an element much smaller than its block's largest.
//
// Measured, 134M bf16 parameters with f32 gradients (a plain copy: 6.78 TB/s): 8-bit
// states 255 us, 6.3 TB/s, bound by memory at 63% of the issue slots; 32-bit states
// with masters 623-639 us, 6.3 TB/s. 96 vectors of a few thousand elements 6 us.

#include "optim.cuh"

namespace taco {

namespace {

// 2^32 times the inverse of the plastic number and of the golden ratio. Of eight
// factors of t tried on constant, decaying and random gradients the golden ratio
// kept the second moment nearest to an exact one's: up to 3% off in the mean after
// 300 to 1500 steps (random bits: 3% to 6%, and up to 3 times the spread), 10% below
// where it has decayed to a fifth.
constexpr uint32_t kWeylI = 0xC13FA9A9u, kWeylT = 0x9E3779B1u;

template <int CAP>
struct AdamwTable {
  AdamwArgs a;
  int count;
  AdamwEntry t[CAP];
};

// Off by its last bit at most, of subnormal numbers too: a root that they lost would
// leave eps alone in the denominator (134M parameters, 8-bit states, f32 and bf16
// gradients: 255 and 242 us; 252 and 232 with a root that flushes them).
__device__ __forceinline__ float sqrt_approx(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Sixteen E4M3 codes of v over the scale with byte b (|v| / scale <= 448),
// rounded by thresholds: element i's is (w + i kWeylI) / 2^32. Times 2^-120 the
// codes' smallest normal number is fp32's, so the fp32 bits are the code, 20 bits
// up, above what lies between two codes, and for codes' subnormals too; the
// threshold's upper 20 bits are added as an integer. No conversion, and 4
// instructions a code. SIGN: v may be negative.
template <bool SIGN>
__device__ __forceinline__ uint4 codes_by_threshold(const float (&value)[16], uint32_t b, uint32_t w) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = value[i];
  float f = __uint_as_float((134u - b) << 23);   // 2^(127 - b) 2^-120
  if (b >= 134u) {                               // that is no normal number: in two factors
    const float low = 0x1p-120f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= low;
    f = fp8_inverse_scale(b);
  }
  uint32_t c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t t[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const int i = 4 * q + j;
      const f2 x = mul2(f2{v[i], v[i + 1]}, f2{f, f});
      const uint32_t y0 = __float_as_uint(x.x) + ((w + i * kWeylI) >> 12);
      const uint32_t y1 = __float_as_uint(x.y) + ((w + (i + 1) * kWeylI) >> 12);
      t[j] = SIGN ? (y0 << 4) | (y0 & 0x80000000u) : y0 << 4;
      t[j + 1] = SIGN ? (y1 << 4) | (y1 & 0x80000000u) : y1 << 4;
    }
    c[q] = __byte_perm(__byte_perm(t[0], t[1], 0x0073), __byte_perm(t[2], t[3], 0x0073), 0x5410);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}
// Whether a byte of the four words is zero.
__device__ __forceinline__ bool any_zero_byte(const uint4& c) {
  const auto z = [](uint32_t w) { return (w - 0x01010101u) & ~w; };
  return ((z(c.x) | z(c.y) | z(c.z) | z(c.w)) & 0x80808080u) != 0u;
}
// The smallest code in the place of zero codes of values that are not zero.
__device__ __forceinline__ void keep_nonzero(uint4& c, const float (&v)[16]) {
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (((w[i >> 2] >> (8 * (i & 3))) & 0xffu) == 0u && v[i] > 0.0f) w[i >> 2] |= 1u << (8 * (i & 3));
  c = make_uint4(w[0], w[1], w[2], w[3]);
}

// x rounded to T by a threshold w: T's step at x is a power of two, and the
// bits below it are a whole number that the threshold's upper bits are added to.
// Not for infinities and NaN.
template <typename T>
__device__ __forceinline__ float round_by_threshold(float x, uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    return __uint_as_float((__float_as_uint(x) + (w >> 16)) & 0xffff0000u);
  } else {
    // times 2^-112, fp16's smallest normal number is fp32's
    return __uint_as_float((__float_as_uint(x * 0x1p-112f) + (w >> 19)) & ~0x1fffu) * 0x1p112f;
  }
}
// The sixteen of a thread as T.
template <typename T>
__device__ __forceinline__ Row16<T> pack_by_threshold(float (&x)[16], uint32_t w) {
  if (amax_of(x) < __uint_as_float(0x7f800000u)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = round_by_threshold<T>(x[i], w + i * kWeylI);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (isfinite(x[i])) x[i] = round_by_threshold<T>(x[i], w + i * kWeylI);
  }
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {   // exact already: the upper halves
    Row16<T> r;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r.w[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
    return r;
  } else {
    return pack<T>(x);
  }
}

// CTAs per SM that the registers are held to, with 2, 3 and 4, and the copy peak's
// share at 134M bf16 parameters with f32 gradients:
//   32-bit states     482, 508, -  us    0.99, 0.94
//   with masters      625, 643, -  us    0.95, 0.92
//   8-bit states      319, 267, 255 us   0.75, 0.89, 0.93
//   with masters      382, 388, 398 us   0.93, 0.92, 0.90
// In 32 bits fewer CTAs with 230 bytes a thread in flight stay nearer to memory's
// order; in 8 bits a step is some 39 instructions an element and wants warps.
template <bool SMALL>
constexpr int adamw_ctas() { return SMALL ? 4 : 2; }

// What every chunk of a launch shares.
struct StepFacts {
  float factor;
  float rate;          // of m' over the denominator
  float root_c, lr;
  uint32_t weyl;       // of element 0 at this step
};

// The 16 elements of a thread in the chunk that begins at element `base` of a
// tensor. WHOLE: the chunk's 4096 all exist; else n of the thread's do.
template <typename P, typename G, bool SMALL, bool VEC, bool WHOLE>
__device__ __forceinline__ void step16(const AdamwArgs& a, const AdamwEntry& en, const StepFacts& f, int64_t base,
                                       int count) {
  const uint32_t i0 = 16 * threadIdx.x;
  const int n = WHOLE ? 16 : count;
  const bool wide = en.wide;
  const float keep = 1.0f - f.lr * en.decay;
  P* const param = static_cast<P*>(en.param) + base + i0;
  // b1 m and the root of v in 8 bits, m and v in 32
  float g[16], x[16], m[16], v[16];
  const Row16<G> gr = load16<G, VEC>(static_cast<const G*>(en.grad) + base + i0, n, wide);
  if (en.master)
    unpack<float>(load16<float, VEC>(en.master + base + i0, n, wide), x);
  else
    unpack<P>(load16<P, VEC>(param, n, wide), x);
  uint8_t *mc = nullptr, *vc = nullptr, *ms = nullptr, *vs = nullptr;
  float *mf = nullptr, *vf = nullptr;
  if constexpr (SMALL) {
    mc = static_cast<uint8_t*>(en.m) + base + i0;
    vc = static_cast<uint8_t*>(en.v) + base + i0;
    ms = en.m_scales + base / kFp8Block + threadIdx.x / kBlockLanes;
    vs = en.v_scales + base / kFp8Block + threadIdx.x / kBlockLanes;
    const uint4 cm = load_codes16(mc, n), cv = load_codes16(vc, n);
    const bool any = WHOLE || n > 0;
    const uint32_t sm = any ? *ms : kScaleOne, sv = any ? *vs : kScaleOne;
    decode16(cm, fp8_scale(sm) * a.b1, m);
    decode16(cv, fp8_scale(sv), v);
    if (!WHOLE && (sm == kScaleNan || sv == kScaleNan)) {   // which must not reach elements that do not exist
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i >= n) m[i] = v[i] = 0.0f;
    }
  } else {
    mf = static_cast<float*>(en.m) + base + i0;
    vf = static_cast<float*>(en.v) + base + i0;
    unpack<float>(load16<float, VEC>(mf, n, wide), m);
    unpack<float>(load16<float, VEC>(vf, n, wide), v);
  }
  unpack<G>(gr, g);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const f2 gi = mul2(f2{g[i], g[i + 1]}, f2{f.factor, f.factor}), gs = mul2(gi, f2{a.one_b2, a.one_b2});
    f2 mi{m[i], m[i + 1]}, vi{v[i], v[i + 1]}, xi{x[i], x[i + 1]};
    mi = SMALL ? fma2(gi, f2{a.one_b1, a.one_b1}, mi) : fma2(mi, f2{a.b1, a.b1}, mul2(gi, f2{a.one_b1, a.one_b1}));
    vi = SMALL ? mul2(vi, vi) : vi;   // of a root in 8 bits, exact but where it is subnormal
    vi = fma2(gs, gi, mul2(vi, f2{a.b2, a.b2}));
    const f2 root{sqrt_approx(vi.x), sqrt_approx(vi.y)};
    const f2 den = fma2(root, f2{f.root_c, f.root_c}, f2{a.eps, a.eps});
    const f2 q = mul2(mi, f2{reciprocal(den.x), reciprocal(den.y)});
    xi = fma2(q, f2{f.rate, f.rate}, mul2(xi, f2{keep, keep}));
    m[i] = mi.x;
    m[i + 1] = mi.y;
    v[i] = SMALL ? root.x : vi.x;
    v[i + 1] = SMALL ? root.y : vi.y;
    x[i] = xi.x;
    x[i + 1] = xi.y;
  }
  const uint32_t w = (static_cast<uint32_t>(base) + i0) * kWeylI + f.weyl;
  if constexpr (std::is_same<P, float>::value) {
    store16<P, VEC>(param, n, wide, pack<P>(x));
  } else if (en.master) {
    store16<float, VEC>(en.master + base + i0, n, wide, pack<float>(x));
    store16<P, VEC>(param, n, wide, pack<P>(x));
  } else {
    store16<P, VEC>(param, n, wide, pack_by_threshold<P>(x, w));
  }
  if constexpr (SMALL) {
    const uint32_t bm = fp8_scale_byte(group_umax<kBlockLanes>(amax_of(m)));
    const uint32_t bv = fp8_scale_byte(group_umax<kBlockLanes>(amax_of(v)));
    const uint4 cm = codes_by_threshold<true>(m, bm, w);
    uint4 cv = codes_by_threshold<false>(v, bv, w);
    if (any_zero_byte(cv)) keep_nonzero(cv, v);
    if (WHOLE || n > 0) {
      store_codes16(mc, n, cm);
      store_codes16(vc, n, cv);
      if (threadIdx.x % kBlockLanes == 0) {
        *ms = static_cast<uint8_t>(bm);
        *vs = static_cast<uint8_t>(bv);
      }
    }
  } else {
    store16<float, VEC>(mf, n, wide, pack<float>(m));
    store16<float, VEC>(vf, n, wide, pack<float>(v));
  }
}

// P, G: element types of parameters and gradients; SMALL: states in FP8 blocks;
// VEC: every tensor of the table starts on 16 bytes.
template <typename P, typename G, bool SMALL, bool VEC, int CAP>
__global__ void __launch_bounds__(kOptimThreads, adamw_ctas<SMALL>())
adamw_kernel(const __grid_constant__ AdamwTable<CAP> table) {
  const AdamwArgs& a = table.a;
  grid_launch_dependents();
  grid_dependency_wait();
  const float factor = a.factor ? *a.factor : 1.0f;
  if (!isfinite(factor)) return;   // in every CTA: nothing changes, the step is not counted
  const uint32_t step = static_cast<uint32_t>(*a.counter) + 1u;
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const float t = static_cast<float>(step);
  StepFacts f;
  f.factor = factor;
  f.rate = -lr / -expm1f(t * a.log_b1);
  f.root_c = rsqrtf(-expm1f(t * a.log_b2));
  f.lr = lr;
  f.weyl = step * kWeylT;
  int e = 0;
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    e = tensor_of(table, c, e);
    const AdamwEntry& en = table.t[e];
    const int64_t base = static_cast<int64_t>(c - en.first) * kOptimChunk;
    if (VEC && base + kOptimChunk <= en.n) {
      step16<P, G, SMALL, VEC, true>(a, en, f, base, 16);
    } else {
      const int n = clamp16(en.n - base - 16 * threadIdx.x);
      if (VEC && __all_sync(kFullMask, n == 0)) continue;   // unaligned rows are stored by whole warps
      step16<P, G, SMALL, VEC, false>(a, en, f, base, n);
    }
  }
  if (a.last) {
    // the CTA that arrives last counts the step: every CTA has read the counter by then
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicInc(reinterpret_cast<unsigned*>(a.counter) + 1, gridDim.x - 1) == gridDim.x - 1)
        *a.counter = static_cast<int32_t>(step);
    }
  }
}

template <typename P, typename G, bool SMALL, bool VEC, int CAP>
cudaError_t launch_table(const AdamwArgs& a, const AdamwEntry* entries, int count, int ctas, cudaStream_t st) {
  static_assert(sizeof(AdamwTable<CAP>) <= 32764, "kernel parameters");
  AdamwTable<CAP> table;
  table.a = a;
  table.count = count;
  for (int i = 0; i < count; ++i) table.t[i] = entries[i];
  const unsigned grid = a.chunks < static_cast<uint32_t>(ctas) ? a.chunks : ctas;
  return launch_dependent(adamw_kernel<P, G, SMALL, VEC, CAP>, dim3(grid ? grid : 1), kOptimThreads, 0, st, table);
}

}  // namespace

cudaError_t launch_adamw(const AdamwArgs& a, const AdamwEntry* entries, int count, int param_dtype, int grad_dtype,
                         bool small, bool vec, int sms, cudaStream_t st) {
  const int ctas = sms * (small ? adamw_ctas<true>() : adamw_ctas<false>());
  const auto go = [&](auto p, auto g, auto s, auto v) {
    using P = decltype(p);
    using G = decltype(g);
    constexpr bool S = decltype(s)::value, V = decltype(v)::value;
    return count <= kAdamwFew ? launch_table<P, G, S, V, kAdamwFew>(a, entries, count, ctas, st)
                              : launch_table<P, G, S, V, kAdamwMany>(a, entries, count, ctas, st);
  };
  const auto forms = [&](auto p, auto g) {
    using No = std::false_type;
    using Yes = std::true_type;
    return small ? (vec ? go(p, g, Yes{}, Yes{}) : go(p, g, Yes{}, No{}))
                 : (vec ? go(p, g, No{}, Yes{}) : go(p, g, No{}, No{}));
  };
  return with_dtype(param_dtype, [&](auto p) {
    using P = decltype(p);
    if constexpr (std::is_same<P, float>::value)
      return forms(p, p);
    else
      return grad_dtype == TACO_DTYPE_F32 ? forms(p, float{}) : forms(p, p);
  });
}

}  // namespace taco
