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

#include "optim.cuh"

namespace taco {

namespace {

// 2^32 times the inverse of the plastic number and of the golden ratio. Of eight
// factors of t tried on constant, decaying and random gradients the golden ratio
// kept the second moment nearest to an exact one's: 2% off in the mean after 300
// to 1500 steps (random bits: 2%, and twice the spread), 10% below where it has
// decayed to a fifth.
constexpr uint32_t kWeylI = 0xC13FA9A9u, kWeylT = 0x9E3779B1u;

template <int CAP>
struct AdamwTable {
  AdamwArgs a;
  int count;
  AdamwEntry t[CAP];
};

__device__ __forceinline__ float sqrt_approx(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// E4M3 codes of |v| inv <= 448 rounded by the thresholds w (their upper 20
// bits). Times 2^-120 the codes' smallest normal number is fp32's, so the fp32
// bits are the code followed by 20 bits of what lies between two codes, for
// codes' subnormals too, and a threshold is added as an integer. The sign comes
// out in bit 7.
constexpr float kToCode = 0x1p-120f;
__device__ __forceinline__ uint32_t code_by_threshold(float v, float inv, uint32_t w20) {
  const uint32_t bits = __float_as_uint(v * inv * kToCode);
  const uint32_t r = (bits & 0x7fffffffu) + w20;
  return ((r >> 20) & 0x7fu) | ((bits >> 24) & 0x80u);
}

// x rounded to T by a threshold w: T's step at x is a power of two, and the
// bits below it are a whole number that the threshold's upper bits are added to.
template <typename T>
__device__ __forceinline__ float round_by_threshold(float x, uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const uint32_t b = __float_as_uint(x);
    if ((b & 0x7f800000u) == 0x7f800000u) return x;
    return __uint_as_float((b + (w >> 16)) & 0xffff0000u);
  } else if constexpr (std::is_same<T, __half>::value) {
    // times 2^-112, fp16's smallest normal number is fp32's
    const float a = x * 0x1p-112f;
    const uint32_t b = __float_as_uint(a);
    if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) return x;
    return __uint_as_float((b + (w >> 19)) & ~0x1fffu) * 0x1p112f;
  } else {
    return x;
  }
}

// P, G: element types of parameters and gradients; SMALL: states in FP8 blocks;
// VEC: every tensor of the table starts on 16 bytes.
template <typename P, typename G, bool SMALL, bool VEC, int CAP>
__global__ void __launch_bounds__(kOptimThreads)
adamw_kernel(const __grid_constant__ AdamwTable<CAP> table) {
  const AdamwArgs& a = table.a;
  grid_launch_dependents();
  grid_dependency_wait();
  const float factor = a.factor ? *a.factor : 1.0f;
  if (!isfinite(factor)) return;   // in every CTA: nothing changes, the step is not counted
  const uint32_t step = static_cast<uint32_t>(*a.counter) + 1u;
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const float t = static_cast<float>(step);
  const float rate = -lr / -expm1f(t * a.log_b1);            // of m' over the denominator
  const float root_c = rsqrtf(-expm1f(t * a.log_b2));
  const int lane8 = threadIdx.x & 7;
  int e = 0;
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    e = tensor_of(table, c, e);
    const AdamwEntry& en = table.t[e];
    const int64_t i0 = static_cast<int64_t>(c - en.first) * kOptimChunk + 16 * threadIdx.x;
    const int n = clamp16(en.n - i0);
    if (VEC && __all_sync(kFullMask, n == 0)) continue;   // rows that start anywhere are stored by whole warps
    const bool wide = en.wide;
    const float keep = 1.0f - lr * en.decay;
    float g[16], x[16], m[16], v[16];
    unpack<G>(load16<G, VEC>(static_cast<const G*>(en.grad) + i0, n, wide), g);
    if (en.master)
      unpack<float>(load16<float, VEC>(en.master + i0, n, wide), x);
    else
      unpack<P>(load16<P, VEC>(static_cast<const P*>(en.param) + i0, n, wide), x);
    if constexpr (SMALL) {
      const int64_t blk = i0 / kFp8Block;
      const bool any = n > 0;
      const uint4 cm = load_codes16(static_cast<const uint8_t*>(en.m) + i0, n);
      const uint4 cv = load_codes16(static_cast<const uint8_t*>(en.v) + i0, n);
      decode16(cm, any ? fp8_scale(en.m_scales[blk]) : 1.0f, m);
      decode16(cv, any ? fp8_scale(en.v_scales[blk]) : 1.0f, v);
      if (n < 16) {   // a NaN scale must not reach elements that do not exist
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i >= n) m[i] = v[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= v[i];
    } else {
      unpack<float>(load16<float, VEC>(static_cast<const float*>(en.m) + i0, n, wide), m);
      unpack<float>(load16<float, VEC>(static_cast<const float*>(en.v) + i0, n, wide), v);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float gi = g[i] * factor;
      m[i] = fmaf(a.b1, m[i], a.one_b1 * gi);
      v[i] = fmaf(a.b2, v[i], a.one_b2 * gi * gi);
      const float root = sqrt_approx(v[i]);
      x[i] = fmaf(rate, __fdividef(m[i], fmaf(root, root_c, a.eps)), x[i] * keep);
      if (SMALL) v[i] = root;
    }
    const uint32_t w0 = static_cast<uint32_t>(i0) * kWeylI + step * kWeylT;
    if (en.master) {
      store16<float, VEC>(en.master + i0, n, wide, pack<float>(x));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = round_by_threshold<P>(x[i], w0 + i * kWeylI);
    }
    store16<P, VEC>(static_cast<P*>(en.param) + i0, n, wide, pack<P>(x));
    if constexpr (SMALL) {
      const int64_t blk = i0 / kFp8Block;
      const uint32_t bm = fp8_scale_byte(group_umax<kBlockLanes>(amax_of(m)));
      const uint32_t bv = fp8_scale_byte(group_umax<kBlockLanes>(amax_of(v)));
      const float im = fp8_inverse_scale(bm), iv = fp8_inverse_scale(bv);
      uint32_t cm[4] = {0, 0, 0, 0}, cv[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t w20 = (w0 + i * kWeylI) >> 12;
        cm[i >> 2] |= code_by_threshold(m[i], im, w20) << (8 * (i & 3));
        uint32_t q = code_by_threshold(v[i], iv, w20);
        if (q == 0 && v[i] > 0.0f) q = 1;
        cv[i >> 2] |= q << (8 * (i & 3));
      }
      if (n > 0) {
        store_codes16(static_cast<uint8_t*>(en.m) + i0, n, make_uint4(cm[0], cm[1], cm[2], cm[3]));
        store_codes16(static_cast<uint8_t*>(en.v) + i0, n, make_uint4(cv[0], cv[1], cv[2], cv[3]));
        if (lane8 == 0) {
          en.m_scales[blk] = static_cast<uint8_t>(bm);
          en.v_scales[blk] = static_cast<uint8_t>(bv);
        }
      }
    } else {
      store16<float, VEC>(static_cast<float*>(en.m) + i0, n, wide, pack<float>(m));
      store16<float, VEC>(static_cast<float*>(en.v) + i0, n, wide, pack<float>(v));
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
  const int ctas = sms * 4;
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
