// optim.cuh - the optimizer step of the LoRA factors (the only trained
// parameters; walkthrough "训练" step 6: the optimizer updates only the LoRA
// parameters, and the paged optimizer keeps its state in unified memory that
// moves to host RAM under memory pressure).
//
// AdamW with decoupled weight decay and global-norm gradient clipping (the
// recipe paragraph: Adam beta2 = 0.999, max grad norm 0.3, constant learning
// rate).  Both kernels stream HBM: the state may live in unified (managed)
// memory, in which case the first touch of a page that was moved to the host
// migrates it back.
#pragma once

#include "common.cuh"

namespace qlora {

// sum of g^2 over a flat fp32 array, added to *acc (fp64; one atomic per CTA).
__global__ void __launch_bounds__(256) grad_sqnorm_kernel(const float* __restrict__ g, int64_t n,
                                                          double* __restrict__ acc) {
  __shared__ double part[8];
  double s = 0.0;
  const int64_t n4 = n / 4;
  const bool vec = (reinterpret_cast<uintptr_t>(g) & 15u) == 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (vec) {
    for (int64_t i = tid; i < n4; i += stride) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(g) + i);
      s += static_cast<double>(v.x) * v.x + static_cast<double>(v.y) * v.y + static_cast<double>(v.z) * v.z +
           static_cast<double>(v.w) * v.w;
    }
    for (int64_t i = 4 * n4 + tid; i < n; i += stride) s += static_cast<double>(g[i]) * g[i];
  } else {
    for (int64_t i = tid; i < n; i += stride) s += static_cast<double>(g[i]) * g[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < (blockDim.x >> 5); ++i) t += part[i];
    if (t != 0.0) atomicAdd(acc, t);
  }
}

struct AdamWParams {
  float lr, beta1, beta2, eps, weight_decay;
  float step_size;          // lr / (1 - beta1^t)
  float bc2_sqrt;           // sqrt(1 - beta2^t)
  float max_grad_norm;      // clipping threshold (used when sqnorm is given)
  const double* sqnorm;     // sum of squares of all gradients, or null (no clipping)
};

// One AdamW step per element, in the order of the usual formulation:
//   g <- g * min(1, max_norm / (||g|| + 1e-6))        (when clipping)
//   p <- p * (1 - lr wd)
//   m <- m + (1 - b1) (g - m)
//   v <- b2 v + (1 - b2) g^2
//   p <- p - step_size * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// fp32 IEEE arithmetic throughout; pb (optional) receives bf16(p), the copy
// the linear layer reads.
__global__ void __launch_bounds__(256) adamw_kernel(float* __restrict__ p, const float* __restrict__ g,
                                                    float* __restrict__ m, float* __restrict__ v,
                                                    uint16_t* __restrict__ pb, int64_t n, AdamWParams a) {
  float clip = 1.0f;
  if (a.sqnorm) {
    const double norm = sqrt(*a.sqnorm);
    const float coef = static_cast<float>(static_cast<double>(a.max_grad_norm) / (norm + 1e-6));
    clip = coef < 1.0f ? coef : 1.0f;
  }
  const float decay = __fsub_rn(1.0f, __fmul_rn(a.lr, a.weight_decay));
  const float one_m_b1 = __fsub_rn(1.0f, a.beta1), one_m_b2 = __fsub_rn(1.0f, a.beta2);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const float gi = a.sqnorm ? __fmul_rn(g[i], clip) : g[i];
    float pi = __fmul_rn(p[i], decay);
    const float mi = __fadd_rn(m[i], __fmul_rn(one_m_b1, __fsub_rn(gi, m[i])));
    const float vi = __fadd_rn(__fmul_rn(a.beta2, v[i]), __fmul_rn(one_m_b2, __fmul_rn(gi, gi)));
    const float denom = __fadd_rn(__fdiv_rn(__fsqrt_rn(vi), a.bc2_sqrt), a.eps);
    pi = __fsub_rn(pi, __fmul_rn(a.step_size, __fdiv_rn(mi, denom)));
    p[i] = pi;
    m[i] = mi;
    v[i] = vi;
    if (pb) pb[i] = __bfloat16_as_ushort(__float2bfloat16_rn(pi));
  }
}

// ====================================================================== AdamW over many tensors

// One AdamW step over a list of tensors (the L1, L2 factors of every linear),
// in two launches whatever their number: multi_adamw_prepare_kernel sums the
// squares of all gradients and turns the step counts and the norm into
// coefficients, multi_adamw_kernel updates every element once.
//
// The state is one flat array per moment in which each tensor starts a new
// block of MA_BLOCK = 256 elements (a warp's work, 8 elements a lane).
//   32 bits: m and v in fp32.
//   8 bits:  m and r = sqrt(v) as FP8 E4M3 codes, and one fp32 scale
//     c = max|x| / 448 per block: the value of a code e is E4M3(e) c, the code of
//     x is E4M3(x 448 / max|x|) (round to nearest even), the rule the block
//     constants of the weights are stored by.  r and not v is stored, because
//     the root spans half the binades: E4M3 reaches 2^-17.8 of the block's
//     largest value, which is 2^-35.6 of the largest v, and a v that fell to 0
//     would divide m by eps alone.  A positive r that rounds to 0 takes the
//     smallest code, 2^-9, for the same reason.  The step itself uses the fp32
//     m and r from before they are rounded to codes.
//     Nearest codes do not follow a slow average: at beta2 = 0.999 a step lowers r
//     by 0.05 % at most and a code changes for 3 to 6 %, so elements keep their size
//     relative to the block's largest.  After 3000 steps of normal gradients of which
//     half of each block shrank tenfold at step 300, that half's r is 5.1 times too
//     large; after fourfold growth the other half's 3.4 times (medians).  Stochastic
//     rounding takes one of the two codes around x with the probabilities that make
//     its expectation x: medians of 0.96 to 1.02 there, and 90 % of the elements
//     within 0.77 and 1.31 under steady gradients (nearest: 0.71 and 1.46).  Its
//     integer operations, nine or so an element for the random bits and as many for
//     the codes, cost 784 us a step of 160 M parameters for 646.
// Bytes a parameter: 8 (param) + 4 or 2 (gradient) + 2 (copy) + 16 or 4.06
// (state), and the gradient once more for the norm.
constexpr int MA_BLOCK = 256;
constexpr int MA_THREADS = 256;
constexpr int MA_WARPS = MA_THREADS / 32;
constexpr int MA_COARSE = 64;
// Times here and at the kernels are of steps of 160 M parameters in a loop over a few states, at the
// step that they describe (a cold step takes 4 % longer).  As it is: 8 bits 646 us, 32 bits 870.
// Resident CTAs of the update.  Registers for the prefetched block against
// warps: 8 bits 722 / 705 / 751 us a step of 160 M parameters at 2 / 3 / 4 CTAs,
// 32 bits 895 / 984 at 2 / 3.
constexpr int MA_PER_SM8 = 3, MA_PER_SM32 = 2;
// CTAs that take the blocks of one contiguous range in turn.  Fewer ranges mean fewer places of the
// seven arrays being read and written at a time: 8 bits 677 us with a range each, 632 with three
// CTAs a range (640 and 634 with 12 and 37); 32 bits 870 and, with two, 865.
constexpr int MA_SHARE8 = 3, MA_SHARE32 = 2;
constexpr int MA_PTRS = 496;          // gradient pointers passed with a launch (under 4 KB of parameters)
constexpr int MA_NORM_CTAS = 148 * 4; // partial sums of the norm, one per CTA
constexpr int MA_UNROLL = 4;          // blocks of gradients a warp loads at a time for the norm

struct MultiTensor {
  float* p;         // fp32 [n]
  uint16_t* copy;   // bf16 [n], or null
  int64_t n;
  int64_t block0;   // first block of the tensor in the flat state
};

struct MultiCoef {
  float step_size;  // unit lr / (1 - beta1^t), t the tensor's own step count
  float bc2_sqrt;   // sqrt(1 - beta2^t)
  float bc2_inv;    // unit / sqrt(1 - beta2^t)
};

// Device side of a plan, in this order in one allocation.
struct MultiHead {
  double partial[MA_NORM_CTAS];
  unsigned ticket;  // CTAs of the norm done, back at 0 after every launch
  float clip;
  int64_t blocks;
};

struct MultiAdamWParams {
  MultiHead* head;
  MultiTensor* tensors;   // [count + 1]; the last one only closes block0
  const int* coarse;      // tensor of every MA_COARSE-th block
  MultiCoef* coef;        // [count]
  const void** stored;    // gradient pointers in memory (lists longer than MA_PTRS)
  int count;
  int from_memory;
  void* m;                // flat state, fp32 or E4M3
  void* v;
  float* m_scale;
  float* v_scale;
  int32_t* steps;         // [count] completed steps of each tensor
  float lr, beta1, beta2, eps, weight_decay, max_grad_norm;
  int clip;               // clip by the global norm
  int share;              // CTAs that take the blocks of one contiguous range in turn
  float unit;             // 8 bits: a power of two that eps, the root's factor and the step carry (see the update)
};

struct GradPtrs {
  const void* g[MA_PTRS];
};

// Copies gradient pointers first .. first + n - 1 of a long list into the plan.
__global__ void __launch_bounds__(128) multi_adamw_ptrs_kernel(const __grid_constant__ GradPtrs gp, const void** dst,
                                                               int n) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) dst[i] = gp.g[i];
}

__device__ __forceinline__ const void* multi_grad(const MultiAdamWParams& a, const GradPtrs& gp, int t) {
  return a.from_memory ? a.stored[t] : gp.g[t];
}

// The tensor that holds block b: from the coarse index on (a search over the table would be a chain
// of dependent loads at the start of every CTA).
__device__ __forceinline__ int multi_find(const MultiAdamWParams& a, int64_t b) {
  int t = __ldg(a.coarse + b / MA_COARSE);
  while (a.tensors[t + 1].block0 <= b) ++t;
  return t;
}

// A lane's 8 elements of a block: 4 lane .. 4 lane + 3 and 128 more.
template <typename T>
__device__ __forceinline__ void load8(const T* src, int left, bool vec, int lane, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 128 * h + 4 * lane;
    if (vec && i + 4 <= left) {
      if constexpr (sizeof(T) == 4) {
        const float4 f = *reinterpret_cast<const float4*>(src + i);
        x[4 * h] = f.x, x[4 * h + 1] = f.y, x[4 * h + 2] = f.z, x[4 * h + 3] = f.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(src + i);
        x[4 * h] = __uint_as_float(u.x << 16), x[4 * h + 1] = __uint_as_float(u.x & 0xFFFF0000u);
        x[4 * h + 2] = __uint_as_float(u.y << 16), x[4 * h + 3] = __uint_as_float(u.y & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4)
          x[4 * h + j] = i + j < left ? static_cast<float>(src[i + j]) : 0.0f;
        else
          x[4 * h + j] = i + j < left ? bf16_bits_to_float(src[i + j]) : 0.0f;
      }
    }
  }
}

__device__ __forceinline__ void store8(float* dst, int left, bool vec, int lane, const float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 128 * h + 4 * lane;
    if (vec && i + 4 <= left) {
      *reinterpret_cast<float4*>(dst + i) = make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < left) dst[i + j] = x[4 * h + j];
    }
  }
}

__device__ __forceinline__ bool vec_ok(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0;
}

// The norm of all gradients (fp64; the partial sums of the CTAs are added in
// order, by the one that ends last, so the norm does not depend on timing), the
// clipping factor and each tensor's coefficients.  A tensor without
// gradient (null pointer) is left out and its step count stands.
template <typename G>
__global__ void __launch_bounds__(MA_THREADS) multi_adamw_prepare_kernel(const __grid_constant__ MultiAdamWParams a,
                                                                         const __grid_constant__ GradPtrs gp) {
  __shared__ double part[MA_WARPS];
  __shared__ bool last;
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == gridDim.x - 1)  // beside the other CTAs' sums
    for (int t = threadIdx.x; t < a.count; t += MA_THREADS) {
      if (!multi_grad(a, gp, t)) continue;
      const int k = ++a.steps[t];
      MultiCoef c;
      c.step_size = static_cast<float>(static_cast<double>(a.lr) / (1.0 - pow(static_cast<double>(a.beta1), k))) * a.unit;
      const double root = sqrt(1.0 - pow(static_cast<double>(a.beta2), k));
      c.bc2_sqrt = static_cast<float>(root);
      c.bc2_inv = static_cast<float>(1.0 / root) * a.unit;
      a.coef[t] = c;
    }
  double s = 0.0;
  if (a.clip) {
    const int64_t blocks = a.head->blocks;
    const int ranges = gridDim.x / a.share, range = blockIdx.x % ranges;
    const int mine = static_cast<int>(blockIdx.x / ranges) * MA_WARPS + warp, step = a.share * MA_WARPS;
    const int64_t b0 = blocks * range / ranges, b1 = blocks * (range + 1) / ranges;
    int t = b0 < b1 ? multi_find(a, b0) : 0;
    for (int64_t b = b0; b < b1; ++t) {
      const MultiTensor ts = a.tensors[t];
      const int64_t next = a.tensors[t + 1].block0;
      const int64_t end = next < b1 ? next : b1;
      const G* g = static_cast<const G*>(multi_grad(a, gp, t));
      if (g) {
        const bool vec = vec_ok(g, 4 * sizeof(G));
        // four blocks a warp at a time: 4 KB of loads in flight
        for (int64_t k = b + mine; k < end; k += MA_UNROLL * step) {
          float x[MA_UNROLL][8];
#pragma unroll
          for (int u = 0; u < MA_UNROLL; ++u) {
            const int64_t e = (k + u * step - ts.block0) * MA_BLOCK;
            const int64_t left = k + u * step < end ? ts.n - e : 0;
            load8<G>(g + e, static_cast<int>(left < MA_BLOCK ? left : MA_BLOCK), vec, lane, x[u]);
          }
#pragma unroll
          for (int u = 0; u < MA_UNROLL; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += static_cast<double>(x[u][j]) * x[u][j];
        }
      }
      b = end;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (lane == 0) part[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double x = 0.0;
    for (int i = 0; i < MA_WARPS; ++i) x += part[i];
    a.head->partial[blockIdx.x] = x;
    __threadfence();
    last = atomicAdd(&a.head->ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (warp == 0) {
    double x = 0.0;
    for (int i = lane; i < static_cast<int>(gridDim.x); i += 32) x += __ldcg(a.head->partial + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if (lane == 0) {
      const float c = static_cast<float>(static_cast<double>(a.max_grad_norm) / (sqrt(x) + 1e-6));
      a.head->clip = a.clip && c < 1.0f ? c : 1.0f;
      a.head->ticket = 0;
    }
  }
}

// Two fp32 values in a 64-bit register and the packed operations on them.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A product that no later addition may be fused with: a packed mul and add are contracted even where
// both are .rn, a sum with +0 is not.
__device__ __forceinline__ uint64_t mul2_rn(uint64_t a, uint64_t b) { return fma2(a, b, 0ull); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Reciprocal to 1 ulp; subnormal arguments count as 0.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The larger of two values, NaN where one of them is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// 32 bits of a counter, by two multiplications with odd constants (the fractions of the square roots
// of 2 and 3) between shifts.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ x >> 16) * 0x6A09E667u;
  x = (x ^ x >> 15) * 0xBB67AE85u;
  return x ^ x >> 16;
}

// y (0 <= |y| <= 448, or NaN) rounded to one of the two E4M3 values around it, away from 0 with the
// probability of its distance from the lower one, to 2^-16: the 20 bits of the significand that E4M3
// does not have carry into the others when random bits are added.  Below 2^-6 the values are multiples
// of 2^-9, as they are between 2^-6 and 2^-5.
__device__ __forceinline__ float e4m3_stochastic(float y, uint32_t bits16) {
  const float a = fabsf(y);
  const float shift = a < 0x1p-6f ? 0x1p-6f : 0.0f;
  const float z = __uint_as_float((__float_as_uint(a + shift) + (bits16 << 4 | 8u)) & 0xFFF00000u) - shift;
  return a <= 512.0f ? copysignf(z, y) : y;
}

// E4M3 codes of a lane's 8 values of a block under inv = 448 / max, and back.  rnd: to nearest for
// null; else random bits, of which m takes the lower half and r the upper.
template <bool kRoot>
__device__ __forceinline__ uint2 state_encode(const float (&x)[8], float inv, const uint32_t* rnd) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) unpack2(mul2(pack2(x[4 * h + j], x[4 * h + j + 1]), dup_f32x2(inv)), y[j], y[j + 1]);
    if (kRoot)
#pragma unroll
      for (int j = 0; j < 4; ++j)  // above 0 stays above 0
        y[j] = max_nan(y[j], fminf(x[4 * h + j] * 0x1p100f, 0x1p-9f));
    if (rnd)
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = e4m3_stochastic(y[j], kRoot ? rnd[4 * h + j] >> 16 : rnd[4 * h + j] & 0xFFFFu);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    w[h] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void state_decode(uint2 w, float scale, float (&x)[8]) {
  const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2 v = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(ws[h] >> (16 * j)), __NV_E4M3));
      const float2 f = __half22float2(v);
      unpack2(mul2(pack2(f.x, f.y), dup_f32x2(scale)), x[4 * h + 2 * j], x[4 * h + 2 * j + 1]);
    }
}

// The scale of a block and the factor of its codes, from the largest
// magnitude's bits.  Blocks below 2^-100 (448 / max would overflow) hold zeros.
// A NaN does not count (it has a code of its own); an infinity makes the scale
// infinite, and the block decodes to NaN (roots above 0 that are finite to infinity).
__device__ __forceinline__ void block_scale(uint32_t top_bits, float& scale, float& inv) {
  const float top = __uint_as_float(top_bits);
  const bool dead = top < 0x1p-100f;
  scale = dead ? 0.0f : __fdiv_rn(top, 448.0f);
  inv = dead ? 0.0f : __fdiv_rn(448.0f, top);
}

// What a lane reads of a block.
template <bool k8>
struct MultiLoads {
  float g[8], p[8];
  float m[k8 ? 1 : 8], v[k8 ? 1 : 8];  // 32-bit state
  uint2 mw, vw;                        // 8-bit state: codes and scales
  float ms, vs;
};

// The update.  The blocks of a contiguous range are taken in turn by the warps of
// the CTAs that share it, from the end to the beginning: the norm read the range
// upwards, so the gradients it read last are still in L2.  A warp loads its next
// block of the tensor before it computes the present one.
//   32 bits: adamw_kernel's order and rounding (fp32 IEEE throughout), so the
//   result is that of qlora_adamw_step bit for bit; bound by DRAM.
//   8 bits: with IEEE divisions too the kernel is bound by instruction issue,
//   not by DRAM (a step over 160 M parameters: 990 us; with an approximate
//   reciprocal, which costs 4 ulp of the update, far below p's own rounding, and
//   packed operations 646 us).  The reciprocal reads a subnormal number as 0 and gives 0 for one:
//   where eps is near either end of fp32, eps, the root's factor and the step are multiplied by a power
//   of two, exactly.  An approximate root would save 15 us more,
//   but moves values over the codes' rounding boundaries.  A ring of three or
//   four blocks a warp in shared memory, filled by cp.async, was slower (716 to
//   802 us for 684 then).
template <bool k8, bool kStochastic, typename G>
__global__ void __launch_bounds__(MA_THREADS, k8 ? MA_PER_SM8 : MA_PER_SM32)
    multi_adamw_kernel(const __grid_constant__ MultiAdamWParams a, const __grid_constant__ GradPtrs gp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t blocks = a.head->blocks;
  const int ranges = gridDim.x / a.share, range = blockIdx.x % ranges;
  const int mine = static_cast<int>(blockIdx.x / ranges) * MA_WARPS + warp, step = a.share * MA_WARPS;
  const int64_t b0 = blocks * range / ranges, b1 = blocks * (range + 1) / ranges;
  const float decay = __fsub_rn(1.0f, __fmul_rn(a.lr, a.weight_decay));
  const float one_m_b1 = __fsub_rn(1.0f, a.beta1), one_m_b2 = __fsub_rn(1.0f, a.beta2);
  if (b0 >= b1) return;
  pdl_wait();  // coefficients, and the step before this one
  const float clip = __ldcg(&a.head->clip);
  const uint64_t clip2 = dup_f32x2(clip), one_m_b1_2 = dup_f32x2(one_m_b1), minus1_2 = dup_f32x2(-1.0f);
  const uint64_t b2_2 = dup_f32x2(a.beta2), one_m_b2_2 = dup_f32x2(one_m_b2);
  const uint64_t eps_2 = dup_f32x2(a.eps), decay_2 = dup_f32x2(decay);
  int t = multi_find(a, b1 - 1);
  for (int64_t top = b1; top > b0; --t) {
    const MultiTensor ts = a.tensors[t];
    const int64_t lo = ts.block0 > b0 ? ts.block0 : b0;
    const G* g = static_cast<const G*>(multi_grad(a, gp, t));
    if (!g) {
      top = lo;
      continue;
    }
    const float step_size = __ldcg(&a.coef[t].step_size);
    const float root = __ldcg(k8 ? &a.coef[t].bc2_inv : &a.coef[t].bc2_sqrt);
    const uint64_t root_2 = dup_f32x2(root), minus_step_2 = dup_f32x2(-step_size);
    const uint32_t key = kStochastic ? mix32(static_cast<uint32_t>(__ldcg(a.steps + t)) * 0x9E3779B9u) : 0u;
    const bool vec = vec_ok(ts.p, 16) && vec_ok(ts.copy, 8), gvec = vec_ok(g, 4 * sizeof(G));
    auto left_of = [&](int64_t b) -> int {
      const int64_t n = ts.n - (b - ts.block0) * MA_BLOCK;
      return static_cast<int>(n < MA_BLOCK ? n : MA_BLOCK);
    };
    auto load = [&](int64_t b, MultiLoads<k8>& x) {
      const int64_t e = (b - ts.block0) * MA_BLOCK;
      const int left = left_of(b);
      load8<G>(g + e, left, gvec, lane, x.g);
      load8<float>(ts.p + e, left, vec, lane, x.p);
      if constexpr (k8) {  // the flat state is padded to whole blocks
        const uint32_t* mc = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.m) + b * MA_BLOCK) + lane;
        const uint32_t* vc = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v) + b * MA_BLOCK) + lane;
        x.mw = make_uint2(mc[0], mc[32]);
        x.vw = make_uint2(vc[0], vc[32]);
        x.ms = a.m_scale[b];
        x.vs = a.v_scale[b];
      } else {
        load8<float>(static_cast<const float*>(a.m) + b * MA_BLOCK, MA_BLOCK, true, lane, x.m);
        load8<float>(static_cast<const float*>(a.v) + b * MA_BLOCK, MA_BLOCK, true, lane, x.v);
      }
    };
    int64_t b = top - 1 - mine;
    MultiLoads<k8> cur, nxt;
    if (b >= lo) load(b, cur);
    for (; b >= lo; b -= step) {
      if (b - step >= lo) load(b - step, nxt);
      const int64_t e = (b - ts.block0) * MA_BLOCK;
      const int left = left_of(b);
      float(&p)[8] = cur.p;
      float m[8], r[8], v[8];
      if constexpr (k8) {
        // Two elements an instruction (f32x2).  m, v and the root are rounded operation by operation, as
        // IEEE arithmetic does: a value that falls on the other side of a rounding boundary of its code
        // changes by a whole code, and the next step's p with it.
        state_decode(cur.mw, cur.ms, m);
        state_decode(cur.vw, cur.vs, r);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint64_t g2 = mul2_rn(pack2(cur.g[j], cur.g[j + 1]), clip2), m0 = pack2(m[j], m[j + 1]);
          const uint64_t m2 = add2(m0, mul2_rn(one_m_b1_2, fma2(m0, minus1_2, g2)));
          const uint64_t r0 = pack2(r[j], r[j + 1]);
          unpack2(add2(mul2_rn(mul2(r0, r0), b2_2), mul2_rn(mul2(g2, g2), one_m_b2_2)), r[j], r[j + 1]);
          r[j] = __fsqrt_rn(r[j]), r[j + 1] = __fsqrt_rn(r[j + 1]);
          float d0, d1;
          unpack2(fma2(pack2(r[j], r[j + 1]), root_2, eps_2), d0, d1);
          const uint64_t q2 = mul2(m2, pack2(rcp_approx(d0), rcp_approx(d1)));
          unpack2(fma2(q2, minus_step_2, mul2(pack2(p[j], p[j + 1]), decay_2)), p[j], p[j + 1]);
          unpack2(m2, m[j], m[j + 1]);
        }
        if (left < MA_BLOCK) {  // what lies behind the tensor's end does not count for the block
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (128 * (j >> 2) + 4 * lane + (j & 3) >= left) m[j] = r[j] = 0.0f;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float gi = __fmul_rn(cur.g[j], clip);
          m[j] = __fadd_rn(cur.m[j], __fmul_rn(one_m_b1, __fsub_rn(gi, cur.m[j])));
          v[j] = __fadd_rn(__fmul_rn(a.beta2, cur.v[j]), __fmul_rn(one_m_b2, __fmul_rn(gi, gi)));
          const float denom = __fadd_rn(__fdiv_rn(__fsqrt_rn(v[j]), root), a.eps);
          p[j] = __fsub_rn(__fmul_rn(p[j], decay), __fmul_rn(step_size, __fdiv_rn(m[j], denom)));
        }
      }
      store8(ts.p + e, left, vec, lane, p);
      if (ts.copy) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = 128 * h + 4 * lane;
          const uint32_t w0 = pack_bf16x2(p[4 * h], p[4 * h + 1]), w1 = pack_bf16x2(p[4 * h + 2], p[4 * h + 3]);
          if (vec && i + 4 <= left) {
            *reinterpret_cast<uint2*>(ts.copy + e + i) = make_uint2(w0, w1);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (i + j < left) ts.copy[e + i + j] = static_cast<uint16_t>((j < 2 ? w0 : w1) >> (16 * (j & 1)));
          }
        }
      }
      if constexpr (k8) {
        float mtop = 0.0f, rtop = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          mtop = fmaxf(mtop, fabsf(m[j]));
          rtop = fmaxf(rtop, r[j]);
        }
        float ms, minv, rs, rinv;
        block_scale(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mtop)), ms, minv);
        block_scale(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(rtop)), rs, rinv);
        uint32_t rnd[8];
        if constexpr (kStochastic) {
          const uint32_t at = mix32((static_cast<uint32_t>(b) * 32u + static_cast<uint32_t>(lane)) ^ key);
#pragma unroll
          for (int j = 0; j < 8; ++j) rnd[j] = mix32(at + j * 0x9E3779B9u);
        }
        const uint2 mw = state_encode<false>(m, minv, kStochastic ? rnd : nullptr);
        const uint2 vw = state_encode<true>(r, rinv, kStochastic ? rnd : nullptr);
        uint32_t* mc = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.m) + b * MA_BLOCK) + lane;
        uint32_t* vc = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.v) + b * MA_BLOCK) + lane;
        mc[0] = mw.x, mc[32] = mw.y;
        vc[0] = vw.x, vc[32] = vw.y;
        if (lane == 0) a.m_scale[b] = ms, a.v_scale[b] = rs;
      } else {
        store8(static_cast<float*>(a.m) + b * MA_BLOCK, left, true, lane, m);
        store8(static_cast<float*>(a.v) + b * MA_BLOCK, left, true, lane, v);
      }
      cur = nxt;
    }
    top = lo;
  }
}

}  // namespace qlora
