// gated_scan -- the gated linear recurrence h_t = a_t h_{t-1} + u_t per channel, channels last, with its
// backward pass and its form for a short run of tokens.
//
// "3.3 Hardware-aware algorithm and GPU memory hierarchy" (booiljung.github.io), section 4.1: the update
// as a first-order linear recurrence; section 6: the backward pass recomputes the states on chip.
//
// One thread walks one channel's tokens in order; neighbouring threads read neighbouring channels.
#include "ptx.cuh"
#include "ssd.h"
#include "ssd_internal.h"

namespace ssd {
namespace {

__device__ __forceinline__ float ld_io(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld_io(const uint16_t* p) { return __uint_as_float(uint32_t(__ldg(p)) << 16); }
__device__ __forceinline__ void st_io(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_io(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }

struct Gate {
  float a, s;  // the decay and 1 - a
};

// 1 - a is taken from the gate, not from a: near a = 1 the difference has lost its low bits.
__device__ __forceinline__ Gate gate_of(int kind, float g) {
  if (kind == SSD_GATE_DECAY) return Gate{g, 1.f - g};
  if (kind == SSD_GATE_LOG) return Gate{expf(g), -expm1f(g)};
  const float e = expf(-fabsf(g)), r = 1.f / (1.f + e);
  return g >= 0.f ? Gate{r, e * r} : Gate{e * r, r};
}

template <typename IO>
__global__ void scan_kernel(GatedProblem p, const IO* __restrict__ x, const IO* __restrict__ gate, const float* init,
                            IO* __restrict__ y, float* final_state, float* __restrict__ states) {
  const int64_t d = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (d >= p.D) return;
  const int64_t blocks = (p.L + SSD_GATED_BLOCK - 1) / SSD_GATED_BLOCK;
  float h = init ? init[b * p.D + d] : 0.f;
  for (int64_t t = 0; t < p.L; ++t) {
    if (states && t % SSD_GATED_BLOCK == 0) states[(b * blocks + t / SSD_GATED_BLOCK) * p.D + d] = h;
    const float xv = ld_io(x + (b * p.L + t) * p.sx + d);
    const Gate k = gate_of(p.kind, ld_io(gate + (b * p.L + t) * p.sg + d));
    h = fmaf(k.a, h, p.complement ? k.s * xv : xv);
    st_io(y + (b * p.L + t) * p.D + d, h);
  }
  if (final_state) final_state[b * p.D + d] = h;
}

template <typename IO>
__global__ void scan_bwd_kernel(GatedProblem p, const IO* __restrict__ x, const IO* __restrict__ gate,
                                const IO* __restrict__ dy, const float* __restrict__ states,
                                const float* __restrict__ dfinal, IO* __restrict__ dx, IO* __restrict__ dgate,
                                float* __restrict__ dinit) {
  const int64_t d = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (d >= p.D) return;
  const int64_t blocks = (p.L + SSD_GATED_BLOCK - 1) / SSD_GATED_BLOCK;
  float c = dfinal ? dfinal[b * p.D + d] : 0.f;  // what the tokens to the right send to h_t
  float was[SSD_GATED_BLOCK];                    // the state that each token of the block starts from
  for (int64_t k = blocks - 1; k >= 0; --k) {
    const int64_t t0 = k * SSD_GATED_BLOCK;
    const int nt = static_cast<int>(p.L - t0 < SSD_GATED_BLOCK ? p.L - t0 : SSD_GATED_BLOCK);
    float h = states[(b * blocks + k) * p.D + d];
    for (int i = 0; i < nt; ++i) {
      was[i] = h;
      const float xv = ld_io(x + (b * p.L + t0 + i) * p.sx + d);
      const Gate q = gate_of(p.kind, ld_io(gate + (b * p.L + t0 + i) * p.sg + d));
      h = fmaf(q.a, h, p.complement ? q.s * xv : xv);
    }
    for (int i = nt - 1; i >= 0; --i) {
      const int64_t row = b * p.L + t0 + i;
      const float xv = ld_io(x + row * p.sx + d);
      const Gate q = gate_of(p.kind, ld_io(gate + row * p.sg + d));
      const float G = ld_io(dy + row * p.D + d) + c;
      float da = G * (p.complement ? was[i] - xv : was[i]);
      if (p.kind == SSD_GATE_LOG) da *= q.a;
      if (p.kind == SSD_GATE_LOGIT) da *= q.a * q.s;
      st_io(dx + row * p.D + d, p.complement ? G * q.s : G);
      st_io(dgate + row * p.D + d, da);
      c = q.a * G;
    }
  }
  if (dinit) dinit[b * p.D + d] = c;
}

dim3 grid_of(const GatedProblem& p) {
  return dim3(static_cast<unsigned>((p.D + 127) / 128), static_cast<unsigned>(p.b));
}

}  // namespace

cudaError_t launch_gated_scan(const GatedProblem& p, const void* x, const void* gate, const float* init, void* y,
                              float* final_state, float* states, cudaStream_t st) {
  if (p.io_bf16)
    scan_kernel<uint16_t><<<grid_of(p), 128, 0, st>>>(p, static_cast<const uint16_t*>(x),
                                                      static_cast<const uint16_t*>(gate), init,
                                                      static_cast<uint16_t*>(y), final_state, states);
  else
    scan_kernel<float><<<grid_of(p), 128, 0, st>>>(p, static_cast<const float*>(x), static_cast<const float*>(gate),
                                                   init, static_cast<float*>(y), final_state, states);
  return cudaGetLastError();
}

cudaError_t launch_gated_scan_bwd(const GatedProblem& p, const void* x, const void* gate, const void* dy,
                                  const float* states, const float* dfinal, void* dx, void* dgate, float* dinit,
                                  cudaStream_t st) {
  if (p.io_bf16)
    scan_bwd_kernel<uint16_t><<<grid_of(p), 128, 0, st>>>(
        p, static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(gate), static_cast<const uint16_t*>(dy),
        states, dfinal, static_cast<uint16_t*>(dx), static_cast<uint16_t*>(dgate), dinit);
  else
    scan_bwd_kernel<float><<<grid_of(p), 128, 0, st>>>(
        p, static_cast<const float*>(x), static_cast<const float*>(gate), static_cast<const float*>(dy), states,
        dfinal, static_cast<float*>(dx), static_cast<float*>(dgate), dinit);
  return cudaGetLastError();
}

cudaError_t launch_gated_decode(const GatedProblem& p, const void* x, const void* gate, const float* state,
                                float* new_state, void* y, cudaStream_t st) {
  return launch_gated_scan(p, x, gate, state, y, new_state, nullptr, st);
}

}  // namespace ssd
