// group_norm -- group norm with an activation or a gate, channels last, and its backward pass.
//
// One CTA takes the values of one (batch, group): seqlen positions of channels / ngroups neighbouring
// channels.  It walks them once for the mean, once for the sum of squares around it, and once to write.
#include "ptx.cuh"
#include "ssd.h"
#include "ssd_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ld_io(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld_io(const uint16_t* p) { return __uint_as_float(uint32_t(__ldg(p)) << 16); }
__device__ __forceinline__ void st_io(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_io(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }
// d silu(v) / dv with s = sigmoid(v)
__device__ __forceinline__ float silu_slope(float v, float s) { return s * (1.f + v * (1.f - s)); }

__device__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) v += part[i];
  return v;
}

template <typename IO>
__global__ void norm_kernel(NormProblem p, const IO* __restrict__ x, const IO* __restrict__ z,
                            const float* __restrict__ w, const float* __restrict__ bias, IO* __restrict__ y,
                            float* __restrict__ mean, float* __restrict__ rstd) {
  const int64_t n = blockIdx.x / p.G, g = blockIdx.x % p.G, Cg = p.C / p.G, count = p.S * Cg;
  auto value = [&](int64_t i) {
    const int64_t row = n * p.S + i / Cg, c = g * Cg + i % Cg;
    float v = ld_io(x + row * p.sx + c);
    if (p.act == SSD_NORM_GATE_FIRST) {
      const float zv = ld_io(z + row * p.sz + c);
      v *= zv * sigmoid(zv);
    }
    return v;
  };
  float mu = 0.f;
  if (!p.rms) {
    for (int64_t i = threadIdx.x; i < count; i += kThreads) mu += value(i);
    mu = block_sum(mu) / float(count);
  }
  float sq = 0.f;
  for (int64_t i = threadIdx.x; i < count; i += kThreads) {
    const float v = value(i) - mu;
    sq = fmaf(v, v, sq);
  }
  const float r = 1.f / sqrtf(block_sum(sq) / float(count) + p.eps);
  for (int64_t i = threadIdx.x; i < count; i += kThreads) {
    const int64_t row = n * p.S + i / Cg, c = g * Cg + i % Cg;
    float v = fmaf((value(i) - mu) * r, w ? w[c] : 1.f, bias ? bias[c] : 0.f);
    if (p.act == SSD_NORM_SILU) v *= sigmoid(v);
    if (p.act == SSD_NORM_GATE) {
      const float zv = ld_io(z + row * p.sz + c);
      v *= zv * sigmoid(zv);
    }
    st_io(y + row * p.C + c, v);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[blockIdx.x] = mu;
    if (rstd) rstd[blockIdx.x] = r;
  }
}

// The gradient of one value's n, and what its dx and dz need.
struct Back {
  float dn, xhat, gate, slope, v, p;  // gate = silu(z), slope = silu'(z), v = x as read, p = n
};

template <typename IO>
__device__ __forceinline__ Back back_of(const NormProblem& p, int64_t row, int64_t c, const IO* x, const IO* z,
                                        const float* w, const float* bias, const IO* dy, float mu, float r) {
  Back k{};
  k.v = ld_io(x + row * p.sx + c);
  float v = k.v;
  if (z) {
    const float zv = ld_io(z + row * p.sz + c), s = sigmoid(zv);
    k.gate = zv * s;
    k.slope = silu_slope(zv, s);
    if (p.act == SSD_NORM_GATE_FIRST) v *= k.gate;
  }
  k.xhat = (v - mu) * r;
  k.p = fmaf(k.xhat, w ? w[c] : 1.f, bias ? bias[c] : 0.f);
  k.dn = ld_io(dy + row * p.C + c);
  if (p.act == SSD_NORM_SILU) k.dn *= silu_slope(k.p, sigmoid(k.p));
  return k;
}

template <typename IO>
__global__ void norm_bwd_kernel(NormProblem p, const IO* __restrict__ x, const IO* __restrict__ z,
                                const float* __restrict__ w, const float* __restrict__ bias,
                                const IO* __restrict__ dy, const float* __restrict__ mean,
                                const float* __restrict__ rstd, IO* __restrict__ dx, IO* __restrict__ dz) {
  const int64_t n = blockIdx.x / p.G, g = blockIdx.x % p.G, Cg = p.C / p.G, count = p.S * Cg;
  const float mu = mean ? mean[blockIdx.x] : 0.f, r = rstd[blockIdx.x];
  float m1 = 0.f, m2 = 0.f;
  for (int64_t i = threadIdx.x; i < count; i += kThreads) {
    const int64_t row = n * p.S + i / Cg, c = g * Cg + i % Cg;
    const Back k = back_of(p, row, c, x, z, w, bias, dy, mu, r);
    const float q = k.dn * (p.act == SSD_NORM_GATE ? k.gate : 1.f) * (w ? w[c] : 1.f);
    m1 += q;
    m2 = fmaf(q, k.xhat, m2);
  }
  m1 = p.rms ? 0.f : block_sum(m1) / float(count);
  m2 = block_sum(m2) / float(count);
  for (int64_t i = threadIdx.x; i < count; i += kThreads) {
    const int64_t row = n * p.S + i / Cg, c = g * Cg + i % Cg;
    const Back k = back_of(p, row, c, x, z, w, bias, dy, mu, r);
    const float q = k.dn * (p.act == SSD_NORM_GATE ? k.gate : 1.f) * (w ? w[c] : 1.f);
    float dv = r * (q - m1 - k.xhat * m2);
    if (p.act == SSD_NORM_GATE) st_io(dz + row * p.C + c, k.dn * k.p * k.slope);
    if (p.act == SSD_NORM_GATE_FIRST) {
      st_io(dz + row * p.C + c, dv * k.v * k.slope);
      dv *= k.gate;
    }
    st_io(dx + row * p.C + c, dv);
  }
}

// dweight and dbias: one thread a channel, over all rows
template <typename IO>
__global__ void norm_param_kernel(NormProblem p, const IO* __restrict__ x, const IO* __restrict__ z,
                                  const float* __restrict__ w, const float* __restrict__ bias,
                                  const IO* __restrict__ dy, const float* __restrict__ mean,
                                  const float* __restrict__ rstd, float* __restrict__ dw, float* __restrict__ db) {
  const int64_t c = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= p.C) return;
  const int64_t g = c / (p.C / p.G);
  float sw = 0.f, sb = 0.f;
  for (int64_t n = 0; n < p.n; ++n) {
    const float mu = mean ? mean[n * p.G + g] : 0.f, r = rstd[n * p.G + g];
    for (int64_t s = 0; s < p.S; ++s) {
      const Back k = back_of(p, n * p.S + s, c, x, z, w, bias, dy, mu, r);
      const float dn = k.dn * (p.act == SSD_NORM_GATE ? k.gate : 1.f);
      sw = fmaf(dn, k.xhat, sw);
      sb += dn;
    }
  }
  if (dw) dw[c] = sw;
  if (db) db[c] = sb;
}

}  // namespace

size_t norm_workspace_bytes(const NormProblem&) { return 0; }
size_t norm_bwd_workspace_bytes(const NormProblem&) { return 0; }

cudaError_t launch_group_norm(const NormProblem& p, const void* x, const void* z, const float* w, const float* b,
                              void* y, float* mean, float* rstd, void* ws, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.n * p.G);
  if (p.io_bf16)
    norm_kernel<uint16_t><<<grid, kThreads, 0, st>>>(p, static_cast<const uint16_t*>(x),
                                                     static_cast<const uint16_t*>(z), w, b,
                                                     static_cast<uint16_t*>(y), mean, rstd);
  else
    norm_kernel<float><<<grid, kThreads, 0, st>>>(p, static_cast<const float*>(x), static_cast<const float*>(z), w, b,
                                                  static_cast<float*>(y), mean, rstd);
  return cudaGetLastError();
}

cudaError_t launch_group_norm_bwd(const NormProblem& p, const void* x, const void* z, const float* w,
                                  const float* b, const void* dy, const float* mean, const float* rstd, void* dx,
                                  void* dz, float* dw, float* db, void* ws, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.n * p.G), cols = static_cast<unsigned>((p.C + 63) / 64);
  if (p.io_bf16) {
    using T = uint16_t;
    norm_bwd_kernel<T><<<grid, kThreads, 0, st>>>(p, static_cast<const T*>(x), static_cast<const T*>(z), w, b,
                                                  static_cast<const T*>(dy), mean, rstd, static_cast<T*>(dx),
                                                  static_cast<T*>(dz));
    if (dw || db)
      norm_param_kernel<T><<<cols, 64, 0, st>>>(p, static_cast<const T*>(x), static_cast<const T*>(z), w, b,
                                                static_cast<const T*>(dy), mean, rstd, dw, db);
  } else {
    using T = float;
    norm_bwd_kernel<T><<<grid, kThreads, 0, st>>>(p, static_cast<const T*>(x), static_cast<const T*>(z), w, b,
                                                  static_cast<const T*>(dy), mean, rstd, static_cast<T*>(dx),
                                                  static_cast<T*>(dz));
    if (dw || db)
      norm_param_kernel<T><<<cols, 64, 0, st>>>(p, static_cast<const T*>(x), static_cast<const T*>(z), w, b,
                                                static_cast<const T*>(dy), mean, rstd, dw, db);
  }
  return cudaGetLastError();
}

}  // namespace ssd
