// Kernels over a list of tensors: the global gradient norm with its clipping,
// and the AdamW step with moments in float32 or in 8 bits.
//
//   norm = sqrt(sum g^2) over the tensors whose gradient is finite
//   c    = max_norm / norm where norm > max_norm > 0, else 1;  g <- c g
//   t <- t + 1;  m <- b1 m + (1 - b1) g;  v <- b2 v + (1 - b2) g^2
//   w <- w (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// All of it is bound by HBM: a few operations an element against 10 to 34 bytes.
#include <float.h>

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "lists.h"

namespace shampoo {

namespace {

constexpr int kThreads = 256;

template <int K>
struct Pointers {
  const void* p[K];
};

// ---------------- element access ----------------

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  return reinterpret_cast<const float*>(p)[i];
}

// Four consecutive elements from an address aligned to the four.
template <bool BF16>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&x)[4]) {
  if (BF16) {
    const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xFFFF0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xFFFF0000u);
  } else {
    const float4 u = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    x[0] = u.x;
    x[1] = u.y;
    x[2] = u.z;
    x[3] = u.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float x) {
  if (BF16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else reinterpret_cast<float*>(p)[i] = x;
}

template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t i, const float (&x)[4]) {
  if (BF16) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t*>(&lo);
    u.y = *reinterpret_cast<uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + i) = u;
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// Elements [i, i + 4) of a run of len, zeros behind its end.
template <bool BF16>
__device__ __forceinline__ void load4_any(const void* p, int64_t base, int i, int len, bool aligned, float (&x)[4]) {
  if (aligned && i + 4 <= len) {
    load4<BF16>(p, base + i, x);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = i + q < len ? load1<BF16>(p, base + i + q) : 0.0f;
  }
}

template <bool BF16>
__device__ __forceinline__ void store4_any(void* p, int64_t base, int i, int len, bool aligned, const float (&x)[4]) {
  if (aligned && i + 4 <= len) {
    store4<BF16>(p, base + i, x);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < len) store1<BF16>(p, base + i + q, x[q]);
  }
}

// Chunks start at multiples of kListChunk, so the tensor's own address decides.
template <bool BF16>
__device__ __forceinline__ bool aligned4(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & (BF16 ? 7 : 15)) == 0;
}

// ---------------- the gradient pass ----------------

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7FEB352Du;
  x = (x ^ (x >> 15)) * 0x846CA68Bu;
  return x ^ (x >> 16);
}

// Closes the pass over the gradients: which tensors are skipped, the norm over
// the others, the clipping factor and, for AdamW, each tensor's t and factors.
// One CTA, fixed order: the same gradients give the same bits.
__device__ void close_pass(const ListTables& t, double max_norm, const ListAdvance& adv, double* red) {
  int* skip = t.skip;
  for (int p = threadIdx.x; p < t.nparams; p += blockDim.x) skip[p] = 0;
  __syncthreads();
  for (int c = threadIdx.x; c < t.nchunks; c += blockDim.x)
    if (isnan(__ldcg(&t.partial[c]))) skip[t.chunks[c].param] = 1;
  __syncthreads();
  double sum = 0.0;
  for (int c = threadIdx.x; c < t.nchunks; c += blockDim.x) {
    const double x = __ldcg(&t.partial[c]);
    if (!skip[t.chunks[c].param]) sum += x;
  }
  sum = block_sum(sum, red);
  int skipped = 0;
  for (int p = threadIdx.x; p < t.nparams; p += blockDim.x) {
    const int sk = skip[p];
    skipped += sk;
    if (adv.step) {
      const int n = adv.step[p] + (sk ? 0 : 1);
      adv.step[p] = n;
      if (!sk) {
        ListStep o;
        // 1 - b^t loses digits where t is small: in 64 bits, rounded once
        o.first = (float)(adv.lr / (1.0 - pow(adv.beta1, (double)n)));
        o.second = (float)(1.0 / sqrt(1.0 - pow(adv.beta2, (double)n)));
        o.shrink = (float)(1.0 - adv.lr * adv.decay[p]);
        o.key = mix32(adv.seed_lo + mix32(adv.seed_hi) + (uint32_t)n * 0x632BE5ABu);
        adv.out[p] = o;
      }
    }
  }
  const double all = block_sum((double)skipped, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(sum);
    t.result->norm = (float)norm;
    t.result->coef = max_norm > 0.0 && norm > max_norm ? (float)(max_norm / norm) : 1.0f;
    t.result->skipped = (int)all;
    t.result->done = 0;
  }
}

// Sum of squares of one chunk.  Sixteen squares are added in 32 bits, the
// groups in 64.  A group whose sum is not finite, or so small that its squares
// may have lost bits below the normal range, is gone through again in 64 bits;
// that also finds the elements that are not finite.
template <bool BF16, int K>
__global__ void __launch_bounds__(kThreads) list_norm_kernel(ListTables t, const __grid_constant__ Pointers<K> ptr,
                                                             int p0, int c0, double max_norm, ListAdvance adv) {
  __shared__ double red[kThreads / 32];
  __shared__ bool last;
  const ListChunk c = t.chunks[c0 + blockIdx.x];
  const void* g = ptr.p[c.param - p0];
  const bool al = aligned4<BF16>(g);
  double sum = 0.0;
  bool bad = false;
  for (int i = threadIdx.x * 4; i < c.len; i += 4 * kThreads * 4) {
    float x[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) load4_any<BF16>(g, c.start, i + k * 4 * kThreads, c.len, al, x[k]);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) s = fmaf(x[k][q], x[k][q], s);
    if (s <= FLT_MAX && s >= 0x1p-96f) {
      sum += (double)s;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          bad |= !isfinite(x[k][q]);
          sum += (double)x[k][q] * x[k][q];
        }
    }
  }
  sum = block_sum(sum, red);
  const bool any = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    t.partial[c0 + blockIdx.x] = any ? nan("") : sum;
    __threadfence();
    last = atomicAdd(&t.result->done, 1u) == (unsigned)t.nchunks - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  close_pass(t, max_norm, adv, red);
}

template <bool BF16, int K>
__global__ void __launch_bounds__(kThreads) list_scale_kernel(ListTables t, const __grid_constant__ Pointers<K> ptr,
                                                              int p0, int c0) {
  const float coef = t.result->coef;
  if (coef == 1.0f) return;
  const ListChunk c = t.chunks[c0 + blockIdx.x];
  if (t.skip[c.param]) return;
  void* g = const_cast<void*>(ptr.p[c.param - p0]);
  const bool al = aligned4<BF16>(g);
  for (int i = threadIdx.x * 4; i < c.len; i += 4 * kThreads) {
    float x[4];
    load4_any<BF16>(g, c.start, i, c.len, al, x);
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] *= coef;
    store4_any<BF16>(g, c.start, i, c.len, al, x);
  }
}

// ---------------- AdamW ----------------

struct Hyper {
  float beta1, omb1, beta2, omb2, eps;
};

// One element; m and v come back updated.  Both stop at the largest float instead of
// becoming an infinity that they would never leave.  Products and sums of the moments are
// rounded one by one, as written: left to the compiler to fuse, a last bit that came out
// differently in another build would round to another 8-bit code.
__device__ __forceinline__ float adamw1(float w, float g, float& m, float& v, float& r, const ListStep& s,
                                        const Hyper& h) {
  m = __fadd_rn(__fmul_rn(h.beta1, m), __fmul_rn(h.omb1, g));
  m = fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
  v = __fadd_rn(__fmul_rn(h.beta2, v), __fmul_rn(__fmul_rn(h.omb2, g), g));
  v = fminf(v, FLT_MAX);
  r = sqrtf(v);
  return fmaf(w, s.shrink, -s.first * (m / fmaf(r, s.second, h.eps)));
}

template <bool BF16, int K>
__global__ void __launch_bounds__(kThreads) adamw_f32_kernel(ListTables t, const __grid_constant__ Pointers<K> wp,
                                                             const __grid_constant__ Pointers<K> gp,
                                                             const __grid_constant__ Pointers<K> cp, int copies,
                                                             int p0, int c0, AdamwState st,
                                                             const ListStep* __restrict__ step, Hyper h) {
  const ListChunk c = t.chunks[c0 + blockIdx.x];
  if (t.skip[c.param]) return;
  const ListStep s = step[c.param];
  const float coef = t.result->coef;
  float* w = static_cast<float*>(const_cast<void*>(wp.p[c.param - p0]));
  const void* g = gp.p[c.param - p0];
  void* b = copies ? const_cast<void*>(cp.p[c.param - p0]) : nullptr;
  const bool alw = aligned4<false>(w), alg = aligned4<BF16>(g), alb = aligned4<true>(b);
  float *m = st.m + c.flat, *v = st.v + c.flat;
  // the flat state is padded to whole blocks: its loads and stores may pass len
  for (int i = threadIdx.x * 4; i < c.len; i += 4 * kThreads) {
    float xw[4], xg[4], xm[4], xv[4], r;
    load4_any<false>(w, c.start, i, c.len, alw, xw);
    load4_any<BF16>(g, c.start, i, c.len, alg, xg);
    load4<false>(m, i, xm);
    load4<false>(v, i, xv);
#pragma unroll
    for (int q = 0; q < 4; ++q) xw[q] = adamw1(xw[q], __fmul_rn(xg[q], coef), xm[q], xv[q], r, s, h);
    store4_any<false>(w, c.start, i, c.len, alw, xw);
    if (b) store4_any<true>(b, c.start, i, c.len, alb, xw);
    store4<false>(m, i, xm);
    store4<false>(v, i, xv);
  }
}

// ---------------- 8-bit moments ----------------
//
// A block of 256 elements keeps m, and r = sqrt(v), as e4m3 codes times a
// power of two, 2^(E - 127) with one byte E a block: the smallest that brings the
// block's largest magnitude to 448, the largest code.  v itself would need twice
// the exponent range that e4m3 has.
//
// The codes are rounded at random.  With b2 = 0.999 v moves by a tenth of a
// percent a step and codes are 6 to 12 % apart: rounding to nearest would leave
// nearly every code where it is, up to a hundredfold below g^2.  m goes up
// with the probability of its fraction, which keeps its mean.  r goes up with the
// probability (v - lo^2) / (hi^2 - lo^2), which keeps the mean of v: the fraction of
// r would add the variance of each rounding to v, step after step.  Scales
// are powers of two because then a value that has not changed is a code still
// when the scale changes: only the change itself is rounded.

// E of the scale: 448 = 1.75 * 2^8, so the exponent of the largest magnitude
// less 8, and one more where its significand exceeds 1.75.
__device__ __forceinline__ int scale_byte(uint32_t largest_bits) {
  return max((int)((largest_bits + 0x1FFFFFu) >> 23) - 8, 1);
}
// 2^(E - 127), zero for the byte 0 of a fresh state
__device__ __forceinline__ float scale_of(int e) { return __uint_as_float((uint32_t)e << 23); }
// its reciprocal 2^(127 - E); E is at most 247, the byte of the largest float
__device__ __forceinline__ float inverse_scale(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }

// a in [0, 448] to a value of e4m3, up where the 16 random bits and the 20 bits
// that are cut off carry.  Below 2^-6 the codes are 2^-9 apart throughout, as they
// are in [2^-6, 2^-5): values there are lifted by 2^-6 for the rounding.
__device__ __forceinline__ float round_m(float a, uint32_t bits16) {
  const float lift = a < 0x1p-6f ? 0x1p-6f : 0.0f;
  return __uint_as_float((__float_as_uint(a + lift) + (bits16 << 4)) & 0xFFF00000u) - lift;
}
__device__ __forceinline__ float round_r(float a, uint32_t bits16) {
  const float lift = a < 0x1p-6f ? 0x1p-6f : 0.0f;
  const uint32_t word = __float_as_uint(a + lift);
  const float lo = __uint_as_float(word & 0xFFF00000u) - lift;
  const float gap = __uint_as_float(word & 0x7F800000u) * 0.125f;
  const bool up = (a - lo) * (a + lo) > (float)bits16 * 0x1p-16f * (gap * fmaf(2.0f, lo, gap));
  return up ? lo + gap : lo;
}

__device__ __forceinline__ void unpack4(uint32_t codes, float (&x)[4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> (16 * k)), __NV_E4M3));
    const float2 f = __half22float2(h);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}
// values of e4m3 already: the conversion is exact
__device__ __forceinline__ uint32_t pack4(const float (&x)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// One warp per block of 256: lane l holds elements 4l..4l+3 of either half.
template <bool BF16, int K>
__global__ void __launch_bounds__(kThreads) adamw_8bit_kernel(ListTables t, const __grid_constant__ Pointers<K> wp,
                                                              const __grid_constant__ Pointers<K> gp,
                                                              const __grid_constant__ Pointers<K> cp, int copies,
                                                              int p0, int c0, AdamwState st,
                                                              const ListStep* __restrict__ step, Hyper h) {
  const ListChunk c = t.chunks[c0 + blockIdx.x];
  if (t.skip[c.param]) return;
  const ListStep s = step[c.param];
  const float coef = t.result->coef;
  float* w = static_cast<float*>(const_cast<void*>(wp.p[c.param - p0]));
  const void* g = gp.p[c.param - p0];
  void* b = copies ? const_cast<void*>(cp.p[c.param - p0]) : nullptr;
  const bool alw = aligned4<false>(w), alg = aligned4<BF16>(g), alb = aligned4<true>(b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = warp * kQBlock; o < c.len; o += (kThreads / 32) * kQBlock) {
    const int64_t flat = c.flat + o, blk = flat / kQBlock;
    const float ms = scale_of(st.ms[blk]), rs = scale_of(st.rs[blk]);
    float xw[2][4], xg[2][4], xm[2][4], xr[2][4];
    float mm = 0.0f, rm = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = o + 128 * k + 4 * lane;
      load4_any<false>(w, c.start, i, c.len, alw, xw[k]);
      load4_any<BF16>(g, c.start, i, c.len, alg, xg[k]);
      unpack4(*reinterpret_cast<const uint32_t*>(st.mq + c.flat + i), xm[k]);
      unpack4(*reinterpret_cast<const uint32_t*>(st.rq + c.flat + i), xr[k]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float m = xm[k][q] * ms, r = xr[k][q] * rs, v = __fmul_rn(r, r);
        xw[k][q] = adamw1(xw[k][q], __fmul_rn(xg[k][q], coef), m, v, r, s, h);
        xm[k][q] = m;
        xr[k][q] = r;
        mm = fmaxf(mm, fabsf(m));
        rm = fmaxf(rm, r);
      }
      const int i = o + 128 * k + 4 * lane;
      store4_any<false>(w, c.start, i, c.len, alw, xw[k]);
      if (b) store4_any<true>(b, c.start, i, c.len, alb, xw[k]);
    }
    // magnitudes order as their bits do
    const int em = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(mm)));
    const int er = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(rm)));
    const float im = inverse_scale(em), ir = inverse_scale(er);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t j = flat + 128 * k + 4 * lane;
      const uint32_t base = (uint32_t)j * 0x9E3779B1u + (uint32_t)(j >> 32) * 0x85EBCA77u + s.key;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t bits = mix32(base + q * 0x9E3779B1u);
        xm[k][q] = copysignf(round_m(fabsf(xm[k][q]) * im, bits & 0xFFFFu), xm[k][q]);
        xr[k][q] = round_r(xr[k][q] * ir, bits >> 16);
      }
      *reinterpret_cast<uint32_t*>(st.mq + j) = pack4(xm[k]);
      *reinterpret_cast<uint32_t*>(st.rq + j) = pack4(xr[k]);
    }
    if (lane == 0) {
      st.ms[blk] = (uint8_t)em;
      st.rs[blk] = (uint8_t)er;
    }
  }
}

template <int K>
Pointers<K> pack(const void* const* p, int n) {
  Pointers<K> a;
  for (int i = 0; i < n; ++i) a.p[i] = p[i];
  return a;
}

// The smallest argument block that holds n pointers: 24 KB of arguments cost
// a launch more than 768 bytes do.
template <class F>
cudaError_t by_count(int n, F&& f) {
  if (n <= 32) f(std::integral_constant<int, 32>());
  else if (n <= 256) f(std::integral_constant<int, 256>());
  else f(std::integral_constant<int, kListGroup>());
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_list_norm(const ListTables& t, const void* const* g, int p0, int np, int c0, int nc, int bf16,
                             double max_norm, const ListAdvance& adv, cudaStream_t s) {
  return by_count(np, [&](auto n) {
    constexpr int K = decltype(n)::value;
    const Pointers<K> a = pack<K>(g + p0, np);
    if (bf16) list_norm_kernel<true, K><<<nc, kThreads, 0, s>>>(t, a, p0, c0, max_norm, adv);
    else list_norm_kernel<false, K><<<nc, kThreads, 0, s>>>(t, a, p0, c0, max_norm, adv);
  });
}

cudaError_t launch_list_scale(const ListTables& t, void* const* g, int p0, int np, int c0, int nc, int bf16,
                              cudaStream_t s) {
  return by_count(np, [&](auto n) {
    constexpr int K = decltype(n)::value;
    const Pointers<K> a = pack<K>(const_cast<const void* const*>(g) + p0, np);
    if (bf16) list_scale_kernel<true, K><<<nc, kThreads, 0, s>>>(t, a, p0, c0);
    else list_scale_kernel<false, K><<<nc, kThreads, 0, s>>>(t, a, p0, c0);
  });
}

cudaError_t launch_adamw(const ListTables& t, float* const* w, const void* const* g, void* const* copies, int p0,
                         int np, int c0, int nc, int bf16, int eight, const AdamwState& st, const ListStep* step,
                         float beta1, float omb1, float beta2, float omb2, float eps, cudaStream_t s) {
  const Hyper h{beta1, omb1, beta2, omb2, eps};
  return by_count(np, [&](auto n) {
    constexpr int K = decltype(n)::value;
    const Pointers<K> aw = pack<K>(reinterpret_cast<const void* const*>(w) + p0, np);
    const Pointers<K> ag = pack<K>(g + p0, np);
    const Pointers<K> ac = copies ? pack<K>(const_cast<const void* const*>(copies) + p0, np) : Pointers<K>{};
    const int cc = copies != nullptr;
    if (eight && bf16)
      adamw_8bit_kernel<true, K><<<nc, kThreads, 0, s>>>(t, aw, ag, ac, cc, p0, c0, st, step, h);
    else if (eight)
      adamw_8bit_kernel<false, K><<<nc, kThreads, 0, s>>>(t, aw, ag, ac, cc, p0, c0, st, step, h);
    else if (bf16)
      adamw_f32_kernel<true, K><<<nc, kThreads, 0, s>>>(t, aw, ag, ac, cc, p0, c0, st, step, h);
    else
      adamw_f32_kernel<false, K><<<nc, kThreads, 0, s>>>(t, aw, ag, ac, cc, p0, c0, st, step, h);
  });
}

}  // namespace shampoo
