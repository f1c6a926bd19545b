// AdamW over many tensors in one launch (gfx950).  With t the step's number:
//   m <- beta1 m + (1 - beta1) g          v <- beta2 v + (1 - beta2) g^2
//   p <- p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
// All of it is fp32, one rounding for each operation as written (no fused
// multiply-adds: the results do not depend on the compiler's choices, and an
// 8-bit state's codes can be checked bit for bit).
//
// 8-bit states.  128 consecutive elements share two scales, powers of two held
// as biased fp32 exponents: one puts the largest |m| of the block at [2^7, 2^8)
// and m is held in e4m3, the other puts the largest v at [2^14, 2^15) and v is
// held in e5m2 (v itself: an average that is unbiased in v stays unbiased).
// Rounding to nearest would stop the averages: a step moves v by about
// 1 - beta2 = 0.1%, codes lie 25% apart, so v would never leave the code it
// reached after its first steps (simulated over 6000 steps of unit gradients:
// v ends at 0.14 of its true value, and updates grow by 2.7x).  So codes are
// rounded by a dither instead: up when the fraction and an offset in [0, 1)
// reach 1, the offset stepping by the golden ratio from step to step (and by
// another irrational from element to element).  Every element then rounds up
// as often as its fraction says, with the offsets spread evenly over any run of
// steps rather than drawn at random (same simulation: v at 0.97 of its true
// value with a spread of 24%; with random offsets 1.01 and 31%).  A positive v
// never rounds to zero, so no denominator collapses to eps.
//
// What bounds it: 28 bytes per element with fp32 states and gradients, 16.03
// with 8-bit states.  67 million elements: 361 us with fp32 states, bf16 gradients and
// a bf16 copy, 206 us with 8-bit states and fp32 gradients (both 5.2 TB/s).
// 16 lanes x 8 elements hold one block of 128, so its largest values are found
// within a row of 16 lanes.
#include "vn_dense.hpp"
#include "vn_rows.hpp"

#pragma clang fp contract(off)

namespace vn {
namespace {

// Largest value over the aligned group of 16 lanes, in each of them.
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 1; o < 16; o *= 2) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

__device__ __forceinline__ uint32_t exponent_of(float a) { return __builtin_bit_cast(uint32_t, a) >> 23; }   // a >= 0
__device__ __forceinline__ float pow2(uint32_t biased) { return __builtin_bit_cast(float, biased << 23); }

// fp8 code of a >= 0 (a scaled below the format's top): MANT mantissa bits,
// exponent bias BIAS; up when the fraction, in units of the last mantissa place,
// and theta = offset / 2^20 reach 1.  theta has 20 bits, so that a value that is a
// code stays that code.  A normal code is the fp32 value's own bits with the offset
// added below the last place that stays; the carry runs into the exponent.
template <int MANT, int BIAS>
__device__ __forceinline__ uint32_t fp8_code(float a, uint32_t offset, float theta) {
  constexpr int DROP = 23 - MANT;
  const uint32_t normal = (__builtin_bit_cast(uint32_t, a) + (offset << (DROP - 20)) -
                           (static_cast<uint32_t>(127 - BIAS) << 23)) >> DROP;
  const uint32_t subnormal = static_cast<uint32_t>(a * pow2(127 + BIAS - 1 + MANT) + theta);
  return a < pow2(127 + 1 - BIAS) ? subnormal : normal;
}

// The non-finite mark of a block: a scale of 255 (the infinity's exponent), so
// that the block's values come back infinite or NaN.
template <int TOP>
__device__ __forceinline__ uint32_t scale_of(float largest) {
  const int e = static_cast<int>(exponent_of(largest));
  if (e == 255) return 255;
  return static_cast<uint32_t>(e - TOP < 1 ? 1 : e - TOP);
}

// Elements [e, e + 8) of p; WHOLE: all of them exist.
template <bool WHOLE, typename T>
__device__ __forceinline__ void load8(const T* p, int64_t e, int64_t n, float (&v)[8]) {
  if constexpr (WHOLE) {
    Run8<T> r;
    __builtin_memcpy(&r, p + e, sizeof(r));
    run_values(r, v);
  } else {
    run_values(load_run(p, e, n), v);
  }
}
template <bool WHOLE, typename T>
__device__ __forceinline__ void store8(T* p, int64_t e, int64_t n, const float (&v)[8]) {
  if constexpr (WHOLE) {
    const Run8<T> r = make_run(v, p);
    __builtin_memcpy(p + e, &r, sizeof(r));
  } else {
    store_run(p, e, n, v);
  }
}

// Elements [e, e + 8) of tensor t.  The chunks that lie whole within their tensor
// carry no checks (an 8-bit step is bound by its vector instructions: 254 us of
// them for 4 blocks 4096 wide before the checks left and the codes were formed from
// the values' bits, 219 us after).
template <int BITS, bool WHOLE>
__device__ __forceinline__ void step8(const AdamParams& a, const AdamTensor& t, const AdamCoef& k, int64_t e) {
  float p[8], g[8], m[8], v[8];
  if (t.flags & 1) load8<WHOLE>(static_cast<const __bf16*>(t.p), e, t.n, p);
  else load8<WHOLE>(static_cast<const float*>(t.p), e, t.n, p);
  if (t.flags & 2) load8<WHOLE>(static_cast<const __bf16*>(t.g), e, t.n, g);
  else load8<WHOLE>(static_cast<const float*>(t.g), e, t.n, g);
  const int64_t s = t.state + e;
  if constexpr (BITS == 32) {
    load8<true>(static_cast<const float*>(a.m), s, 0, m);
    load8<true>(static_cast<const float*>(a.v), s, 0, v);
  } else {
    uint32_t cm[2], cv[2];
    __builtin_memcpy(cm, static_cast<const uint8_t*>(a.m) + s, 8);
    __builtin_memcpy(cv, static_cast<const uint8_t*>(a.v) + s, 8);
    const float sm = pow2(a.m_scale[s / kAdamBlock]), sv = pow2(a.v_scale[s / kAdamBlock]);
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const uint32_t d = cv[j / 4] & 0x7F7F7F7Fu;
      const vn_f32x2 m0 = __builtin_amdgcn_cvt_pk_f32_fp8(cm[j / 4], false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8(cm[j / 4], true);
      const vn_f32x2 v0 = __builtin_amdgcn_cvt_pk_f32_bf8(d, false), v1 = __builtin_amdgcn_cvt_pk_f32_bf8(d, true);
      m[j] = m0[0] * sm;
      m[j + 1] = m0[1] * sm;
      m[j + 2] = m1[0] * sm;
      m[j + 3] = m1[1] * sm;
      v[j] = v0[0] * sv;
      v[j + 1] = v0[1] * sv;
      v[j + 2] = v1[0] * sv;
      v[j + 3] = v1[1] * sv;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = g[j] * a.sign;
    m[j] = m[j] * a.beta1 + gj * a.one_minus_beta1;
    v[j] = v[j] * a.beta2 + (gj * gj) * a.one_minus_beta2;
    const float denom = sqrtf(v[j]) * k.inv_root + a.eps;
    p[j] = p[j] * t.decay - (m[j] / denom) * k.step_size;
  }
  if (t.flags & 1) store8<WHOLE>(static_cast<__bf16*>(t.p), e, t.n, p);
  else store8<WHOLE>(static_cast<float*>(t.p), e, t.n, p);
  if (t.copy != nullptr) store8<WHOLE>(t.copy, e, t.n, p);
  // the state's padding past n stays zero
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (e + j >= t.n) m[j] = v[j] = 0.0f;
  if constexpr (BITS == 32) {
    store8<true>(static_cast<float*>(a.m), s, 0, m);
    store8<true>(static_cast<float*>(a.v), s, 0, v);
  } else {
    // the largest exponent of the block, non-finite ones (255) among them:
    // compared as integers' floats, so that a NaN counts as the largest
    float lm = 0.0f, lv = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float am = fabsf(m[j]);
      lm = am == am ? fmaxf(lm, am) : __builtin_inff();
      lv = v[j] == v[j] ? fmaxf(lv, v[j]) : __builtin_inff();
    }
    const uint32_t em = scale_of<7>(max16(lm)), ev = scale_of<14>(max16(lv));
    uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};
    // a non-finite block holds codes of 1 (times infinity)
    const bool fm = em != 255, fv = ev != 255;
    const float im = pow2(fm ? 254 - em : 1), iv = pow2(fv ? 254 - ev : 1);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t offset = (k.dither + static_cast<uint32_t>(s + j) * 0xC13FA9A9u) >> 12;
      const float theta = static_cast<float>(offset) * 0x1p-20f;
      uint32_t c = fm ? fp8_code<3, 7>(fabsf(m[j]) * im, offset, theta) : 1;
      if (m[j] < 0.0f) c |= 128;
      uint32_t u = fv ? fp8_code<2, 15>(v[j] * iv, offset, theta) : 1;
      if (v[j] > 0.0f && u == 0) u = 1;
      cm[j / 4] |= c << (8 * (j % 4));
      cv[j / 4] |= u << (8 * (j % 4));
    }
    __builtin_memcpy(static_cast<uint8_t*>(a.m) + s, cm, 8);
    __builtin_memcpy(static_cast<uint8_t*>(a.v) + s, cv, 8);
    if ((threadIdx.x & 15) == 0) {
      a.m_scale[s / kAdamBlock] = static_cast<uint8_t>(em);
      a.v_scale[s / kAdamBlock] = static_cast<uint8_t>(ev);
    }
  }
}

template <int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(AdamParams a) {
  // the tensor of this chunk: the last whose first chunk is not past it
  int lo = 0, hi = a.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.t[mid].first_chunk <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamTensor t = a.t[lo];
  const AdamCoef k = a.coef_dev != nullptr ? *a.coef_dev : a.coef;
  const int64_t start = static_cast<int64_t>(blockIdx.x - t.first_chunk) * kAdamChunk;
  if (start + kAdamChunk <= t.n) {
#pragma unroll 1
    for (int i = 0; i < kAdamChunk / 2048; ++i) step8<BITS, true>(a, t, k, start + i * 2048 + threadIdx.x * 8);
    return;
  }
#pragma unroll 1
  for (int i = 0; i < kAdamChunk / 2048; ++i) {
    const int64_t e = start + i * 2048 + threadIdx.x * 8;
    // whole blocks of 128 take part (their lanes exchange values); elements
    // past n hold zeros and are stored to the state's padding alone
    if (e - (e & (kAdamBlock - 1)) >= t.n) return;
    step8<BITS, false>(a, t, k, e);
  }
}

// The next step's number and coefficients, on the device: a captured step
// counts on from replay to replay.
__global__ void adamw_coefficients_kernel(int64_t* step, double lr, double beta1, double beta2, AdamCoef* coef) {
  const int64_t t = *step + 1;
  *step = t;
  AdamCoef c;
  c.step_size = static_cast<float>(lr / (1.0 - pow(beta1, static_cast<double>(t))));
  c.inv_root = static_cast<float>(1.0 / sqrt(1.0 - pow(beta2, static_cast<double>(t))));
  c.dither = static_cast<uint32_t>(t) * 0x9E3779B9u;
  c.pad = 0;
  *coef = c;
}

}  // namespace

hipError_t launch_adamw(const AdamParams& p, int bits, hipStream_t stream) {
  if (bits == 32) adamw_kernel<32><<<p.chunks, 256, 0, stream>>>(p);
  else adamw_kernel<8><<<p.chunks, 256, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_adamw_coefficients(int64_t* step, double lr, double beta1, double beta2, AdamCoef* coef,
                                     hipStream_t stream) {
  adamw_coefficients_kernel<<<1, 1, 0, stream>>>(step, lr, beta1, beta2, coef);
  return hipGetLastError();
}

}  // namespace vn
