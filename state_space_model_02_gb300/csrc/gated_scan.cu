// gated_scan -- the gated linear recurrence h_t = a_t h_{t-1} + u_t per channel, channels last, with its
// backward pass and its form for a short run of tokens.
//
// "3.3 Hardware-aware algorithm and GPU memory hierarchy" (booiljung.github.io), section 4.1: the update
// as a first-order linear recurrence whose steps compose; section 6: the backward pass recomputes the states
// on chip.
//
// A run of tokens maps the state that enters it affinely, h -> P h + H with P the product of its decays and H
// its end state from zero, and two neighbouring runs compose to (P2 P1, P2 H1 + H2).  A warp owns 32 V
// neighbouring channels (V a thread: one 128-byte line of bf16 a token) and TW tokens, a CTA NW warps one behind
// the other in time, and a cluster K CTAs; a step of the cluster is K NW TW tokens.  In each step every warp reads
// its tokens once, keeps a and u of each in registers, and reduces them to (P, H); the CTAs tell each other their
// composed (P, H) through distributed shared memory; every thread then folds the maps before its own onto the
// carry that all threads hold, and walks its tokens again from the state that truly enters them, so that the second
// walk rounds as the plain recurrence does.  x and gate are read once and y written once, whatever the length
// is; the loads of the next step are in flight while this one is worked on.
#include <type_traits>

#include "ptx.cuh"
#include "ssd.h"
#include "ssd_internal.h"

namespace ssd {
namespace {

// ------------------------------------------------------------------------------ values

// V neighbouring values of one token: as float32, and as they lie in memory
template <int V>
using vec = std::conditional_t<V == 2, float2, float>;
template <typename IO, int V>
using raw_t = std::conditional_t<sizeof(IO) * V == 2, uint16_t, std::conditional_t<sizeof(IO) * V == 4, uint32_t, uint2>>;

__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return mul_f32x2(a, b); }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return fma_f32x2(a, b, c); }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float2 vadd(float2 a, float2 b) { return fma_f32x2(a, make_float2(1.f, 1.f), b); }
__device__ __forceinline__ float vsub(float a, float b) { return a - b; }
__device__ __forceinline__ float2 vsub(float2 a, float2 b) { return fma_f32x2(b, make_float2(-1.f, -1.f), a); }
template <int V>
__device__ __forceinline__ vec<V> splat(float f) {
  if constexpr (V == 2)
    return make_float2(f, f);
  else
    return f;
}

template <typename IO, int V>
__device__ __forceinline__ vec<V> widen(raw_t<IO, V> r) {
  if constexpr (sizeof(IO) == 4 && V == 2)
    return make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
  else if constexpr (sizeof(IO) == 4)
    return __uint_as_float(r);
  else if constexpr (V == 2)
    return make_float2(bf16lo_to_f32(r), bf16hi_to_f32(r));
  else
    return __uint_as_float(uint32_t(r) << 16);
}
template <typename IO, int V>
__device__ __forceinline__ void store(IO* p, vec<V> f) {
  raw_t<IO, V>* q = reinterpret_cast<raw_t<IO, V>*>(p);
  if constexpr (sizeof(IO) == 4 && V == 2)
    *q = make_uint2(__float_as_uint(f.x), __float_as_uint(f.y));
  else if constexpr (sizeof(IO) == 4)
    *q = __float_as_uint(f);
  else if constexpr (V == 2)
    *q = pack_bf16x2(f.x, f.y);
  else
    *q = static_cast<uint16_t>(pack_bf16x2(f, 0.f));
}
template <typename IO, int V>
__device__ __forceinline__ raw_t<IO, V> load(const IO* p) {
  return __ldg(reinterpret_cast<const raw_t<IO, V>*>(p));
}
template <int V>
__device__ __forceinline__ vec<V> load_f32(const float* p) {
  return *reinterpret_cast<const vec<V>*>(p);
}
template <int V>
__device__ __forceinline__ void store_f32(float* p, vec<V> f) {
  *reinterpret_cast<vec<V>*>(p) = f;
}

// A raw value of each tensor for tokens behind the last one: u = 0 and a = 1 leave the state as it is, dy = 0 the
// adjoint.
template <typename IO, int V>
__device__ __forceinline__ raw_t<IO, V> raw_splat(uint32_t f32_bits) {
  if constexpr (sizeof(IO) == 4 && V == 2)
    return make_uint2(f32_bits, f32_bits);
  else if constexpr (sizeof(IO) == 4)
    return f32_bits;
  else if constexpr (V == 2)
    return f32_bits | f32_bits >> 16;
  else
    return static_cast<uint16_t>(f32_bits >> 16);
}
template <typename IO, int V, int KIND>
__device__ __forceinline__ raw_t<IO, V> keep_gate() {
  return raw_splat<IO, V>(KIND == SSD_GATE_LOGIT ? 0x7f800000u : KIND == SSD_GATE_LOG ? 0u : 0x3f800000u);
}

// exp(g).  With z = g log2 e rounded, 2^z is off by |z| 2^-24 of it; bf16 results do not see that (the decays that
// matter have small |z|, and the others' share of a state is as small as they are), float32 ones get the rounding of z
// back to first order.  ex2 gives 0 below 2^-126; kTiny: such values keep what float32 has of them, as the square of
// 2^(z / 2) (the gradient of a gate is proportional to its decay, however small).
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596303e-8f, kLn2 = 0.693147181f;
template <typename IO, bool kTiny>
__device__ __forceinline__ float exp_of(float g) {
  const float z = g * kLog2eHi;
  float e = ex2(kTiny ? 0.5f * z : z);
  if constexpr (kTiny) e *= e;
  if constexpr (sizeof(IO) == 2) {
    return e;
  } else {
    const float d = fmaf(g, kLog2eLo, fmaf(g, kLog2eHi, -z)) * kLn2;
    return fabsf(z) < 200.f ? fmaf(e, d, e) : e;  // infinities have no remainder
  }
}

// The decay a and s = 1 - a.  s is taken from the gate, not from a: near a = 1 the difference has lost its low
// bits.  kS: whether s is used.
template <typename IO, int KIND, bool kS, bool kTiny>
__device__ __forceinline__ void gate_of(float g, float& a, float& s) {
  if constexpr (KIND == SSD_GATE_DECAY) {
    a = g;
    s = 1.f - g;
  } else if constexpr (KIND == SSD_GATE_LOG) {
    a = exp_of<IO, kTiny>(g);
    if constexpr (kS) {
      // 1 - exp(g): for small |g| its series (the first term left out is g^6 / 5040 of it, under 5e-8)
      const float q = fmaf(g, fmaf(g, fmaf(g, fmaf(g, fmaf(g, 1.f / 720.f, 1.f / 120.f), 1.f / 24.f), 1.f / 6.f), 0.5f), 1.f);
      s = fabsf(g) < 0.25f ? -g * q : 1.f - a;
    }
  } else if constexpr (kS) {
    const float e = exp_of<IO, kTiny>(-fabsf(g)), r = __fdividef(1.f, 1.f + e), er = e * r;
    a = g >= 0.f ? r : er;
    s = g >= 0.f ? er : r;
  } else {
    a = __fdividef(1.f, 1.f + exp_of<IO, kTiny>(-g));
    if (g < -80.f) a = exp_of<IO, kTiny>(g);  // 1 + exp(-g) leaves the range that the division takes
  }
}
template <typename IO, int KIND, bool kS, bool kTiny>
__device__ __forceinline__ void gate_of(float2 g, float2& a, float2& s) {
  gate_of<IO, KIND, kS, kTiny>(g.x, a.x, s.x);
  gate_of<IO, KIND, kS, kTiny>(g.y, a.y, s.y);
}

// ------------------------------------------------------------------------------ cluster

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_peer(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

constexpr int kMaxCluster = 8;

// ------------------------------------------------------------------------------ forward

struct ScanArgs {
  int64_t L, D, sx, sg;
  int cluster, steps;
};

template <typename IO, int V, int KIND, bool COMP, int NW, int TW>
__global__ void __launch_bounds__(NW * 32, 512 / (NW * 32)) scan_kernel(
    const ScanArgs p, const IO* __restrict__ x, const IO* __restrict__ gate, const float* __restrict__ init,
    IO* __restrict__ y, float* __restrict__ final_state, float* __restrict__ states) {
  // maps of one step, in turn for even and odd steps: a step's maps are read until the barrier of the next
  __shared__ vec<V> warp_map[2][NW][2][32];
  __shared__ vec<V> cta_map[2][kMaxCluster][2][32];
  __shared__ vec<V> end_state[2][32];  // after a step's last token, where the cluster is one CTA
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int K = p.cluster;
  const int rank = K > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t b = blockIdx.y;
  const int64_t c0 = int64_t(blockIdx.x / K) * (32 * V) + lane * V;
  const bool mine = c0 < p.D;
  const int64_t c = mine ? c0 : p.D - V;  // lanes past the last channel read it and write nothing
  const int64_t span = int64_t(K) * NW * TW;
  int64_t t0 = (rank * NW + w) * TW;
  const int64_t blocks = (p.L + SSD_GATED_BLOCK - 1) / SSD_GATED_BLOCK;
  const IO* xp = x + (b * p.L + t0) * p.sx + c;
  const IO* gp = gate + (b * p.L + t0) * p.sg + c;
  IO* yp = y + (b * p.L + t0) * p.D + c;

  if (K > 1) cluster_sync();  // every CTA of the cluster runs before its shared memory is written to
  grid_dep_wait();
  raw_t<IO, V> xr[TW], gr[TW];
  auto fetch = [&]() {
    if (t0 + TW <= p.L) {
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        xr[i] = load<IO, V>(xp + i * p.sx);
        gr[i] = load<IO, V>(gp + i * p.sg);
      }
    } else {
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        xr[i] = raw_splat<IO, V>(0u);
        gr[i] = keep_gate<IO, V, KIND>();
        if (t0 + i < p.L) {
          xr[i] = load<IO, V>(xp + i * p.sx);
          gr[i] = load<IO, V>(gp + i * p.sg);
        }
      }
    }
  };
  fetch();
  vec<V> carry = init ? load_f32<V>(init + b * p.D + c) : splat<V>(0.f);  // the state that enters the step

  for (int step = 0; step < p.steps; ++step) {
    const int par = step & 1;
    vec<V> a[TW], u[TW], s, P = splat<V>(1.f), H = splat<V>(0.f);
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      gate_of<IO, KIND, COMP, false>(widen<IO, V>(gr[i]), a[i], s);
      u[i] = widen<IO, V>(xr[i]);
      if constexpr (COMP) u[i] = vmul(u[i], s);
      H = vfma(a[i], H, u[i]);
      P = vmul(P, a[i]);
    }
    const int64_t now = t0;
    t0 += span;
    xp += span * p.sx;
    gp += span * p.sg;
    if (step + 1 < p.steps) fetch();

    warp_map[par][w][0][lane] = P;
    warp_map[par][w][1][lane] = H;
    __syncthreads();
    vec<V> h;
    if (K > 1) {
      if (w == 0) {  // the CTA's own map, to every CTA of the cluster
        vec<V> cp = warp_map[par][0][0][lane], ch = warp_map[par][0][1][lane];
#pragma unroll
        for (int k = 1; k < NW; ++k) {
          const vec<V> kp = warp_map[par][k][0][lane];
          ch = vfma(kp, ch, warp_map[par][k][1][lane]);
          cp = vmul(cp, kp);
        }
        for (int k = 0; k < K; ++k) {
          st_peer(peer_addr(smem_u32(&cta_map[par][rank][0][lane]), k), cp);
          st_peer(peer_addr(smem_u32(&cta_map[par][rank][1][lane]), k), ch);
        }
      }
      cluster_sync();
      h = carry;
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k == rank) h = carry;
        if (k < K) carry = vfma(cta_map[par][k][0][lane], carry, cta_map[par][k][1][lane]);
      }
    } else {
      if (step > 0) carry = end_state[par][lane];
      h = carry;
    }
#pragma unroll
    for (int k = 0; k < NW - 1; ++k)
      if (k < w) h = vfma(warp_map[par][k][0][lane], h, warp_map[par][k][1][lane]);
    if (states && now % SSD_GATED_BLOCK == 0 && now < p.L && mine)
      store_f32<V>(states + (b * blocks + now / SSD_GATED_BLOCK) * p.D + c, h);
    if (mine && now + TW <= p.L) {
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        h = vfma(a[i], h, u[i]);
        store<IO, V>(yp + i * p.D, h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        h = vfma(a[i], h, u[i]);
        if (mine && now + i < p.L) store<IO, V>(yp + i * p.D, h);
      }
    }
    yp += span * p.D;
    if (K == 1 && w == NW - 1) {
      carry = h;
      end_state[par ^ 1][lane] = h;
    }
  }
  if (final_state && rank == 0 && w == NW - 1 && mine) store_f32<V>(final_state + b * p.D + c, carry);
  if (K > 1) cluster_sync();  // no CTA leaves while another may still write to its shared memory
  grid_dep_launch();
}

// A short run of tokens: one thread walks V channels.
template <typename IO, int V, int KIND, bool COMP>
__global__ void __launch_bounds__(128) run_kernel(const ScanArgs p, const IO* __restrict__ x,
                                                  const IO* __restrict__ gate, const float* init,
                                                  IO* __restrict__ y, float* final_state,
                                                  float* __restrict__ states) {
  const int64_t c = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * V, b = blockIdx.y;
  grid_dep_wait();
  if (c >= p.D) return;
  const int64_t blocks = (p.L + SSD_GATED_BLOCK - 1) / SSD_GATED_BLOCK;
  const IO* xp = x + b * p.L * p.sx + c;
  const IO* gp = gate + b * p.L * p.sg + c;
  IO* yp = y + b * p.L * p.D + c;
  vec<V> h = init ? load_f32<V>(init + b * p.D + c) : splat<V>(0.f);
#pragma unroll 4
  for (int64_t t = 0; t < p.L; ++t) {
    if (states && t % SSD_GATED_BLOCK == 0) store_f32<V>(states + (b * blocks + t / SSD_GATED_BLOCK) * p.D + c, h);
    vec<V> u = widen<IO, V>(load<IO, V>(xp)), a, s;
    gate_of<IO, KIND, COMP, false>(widen<IO, V>(load<IO, V>(gp)), a, s);
    if constexpr (COMP) u = vmul(u, s);
    h = vfma(a, h, u);
    store<IO, V>(yp, h);
    xp += p.sx;
    gp += p.sg;
    yp += p.D;
  }
  if (final_state) store_f32<V>(final_state + b * p.D + c, h);
  grid_dep_launch();
}

// ------------------------------------------------------------------------------ backward

// The adjoint runs from the right: with c_t what the tokens right of t send to h_t, G_t = dy_t + c_t and
// c_{t-1} = a_t G_t, again affine, with the same product P: c -> P c + R over a run of tokens.  A CTA's tile is one
// block of SSD_GATED_BLOCK tokens, whose entering state the forward pass has left in `states`, so only the adjoint
// is carried between CTAs and steps.  In one step every warp reads x, gate and dy of its tokens once and
// reduces them to (P, H, R); then it walks the states forward from the one that enters its tokens, and the adjoint
// backward from the one that leaves them.
template <typename IO, int V, int KIND, bool COMP, int NW, int TW>
__global__ void __launch_bounds__(NW * 32, 512 / (NW * 32)) scan_bwd_kernel(
    const ScanArgs p, const IO* __restrict__ x, const IO* __restrict__ gate, const IO* __restrict__ dy,
    const float* __restrict__ states, const float* __restrict__ dfinal, IO* __restrict__ dx, IO* __restrict__ dgate,
    float* __restrict__ dinit) {
  static_assert(NW * TW == SSD_GATED_BLOCK, "a CTA's tile is a block");
  constexpr bool kS = COMP || KIND == SSD_GATE_LOGIT;
  __shared__ vec<V> warp_map[2][NW][3][32];
  __shared__ vec<V> cta_map[2][kMaxCluster][2][32];
  __shared__ vec<V> end_adjoint[2][32];  // what leaves a step's first token, where the cluster is one CTA
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int K = p.cluster;
  const int rank = K > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t b = blockIdx.y;
  const int64_t c0 = int64_t(blockIdx.x / K) * (32 * V) + lane * V;
  const bool mine = c0 < p.D;
  const int64_t c = mine ? c0 : p.D - V;
  const int64_t blocks = (p.L + SSD_GATED_BLOCK - 1) / SSD_GATED_BLOCK;
  int64_t block = int64_t(p.steps - 1) * K + rank;  // this CTA's block of the last step
  int64_t t0 = block * SSD_GATED_BLOCK + w * TW;

  if (K > 1) cluster_sync();
  grid_dep_wait();
  raw_t<IO, V> xr[TW], gr[TW], dr[TW];
  vec<V> hr = splat<V>(0.f);
  auto fetch = [&]() {
    const IO* xp = x + (b * p.L + t0) * p.sx + c;
    const IO* gp = gate + (b * p.L + t0) * p.sg + c;
    const IO* dp = dy + (b * p.L + t0) * p.D + c;
    if (t0 + TW <= p.L) {
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        xr[i] = load<IO, V>(xp + i * p.sx);
        gr[i] = load<IO, V>(gp + i * p.sg);
        dr[i] = load<IO, V>(dp + i * p.D);
      }
    } else {
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        xr[i] = raw_splat<IO, V>(0u);
        gr[i] = keep_gate<IO, V, KIND>();
        dr[i] = raw_splat<IO, V>(0u);
        if (t0 + i < p.L) {
          xr[i] = load<IO, V>(xp + i * p.sx);
          gr[i] = load<IO, V>(gp + i * p.sg);
          dr[i] = load<IO, V>(dp + i * p.D);
        }
      }
    }
    if (block < blocks) hr = load_f32<V>(states + (b * blocks + block) * p.D + c);
  };
  fetch();
  vec<V> carry = dfinal ? load_f32<V>(dfinal + b * p.D + c) : splat<V>(0.f);  // what enters the step from its right

  for (int step = p.steps - 1; step >= 0; --step) {
    const int par = step & 1;
    vec<V> a[TW], s[TW], xv[TW], d[TW], P = splat<V>(1.f), H = splat<V>(0.f), R = splat<V>(0.f), h = hr;
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      gate_of<IO, KIND, kS, true>(widen<IO, V>(gr[i]), a[i], s[i]);
      xv[i] = widen<IO, V>(xr[i]);
      d[i] = widen<IO, V>(dr[i]);
      H = vfma(a[i], H, COMP ? vmul(xv[i], s[i]) : xv[i]);
      P = vmul(P, a[i]);
    }
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) R = vmul(a[i], vadd(d[i], R));
    const int64_t now = t0;
    block -= K;
    t0 -= int64_t(K) * SSD_GATED_BLOCK;
    if (step > 0) fetch();

    warp_map[par][w][0][lane] = P;
    warp_map[par][w][1][lane] = H;
    warp_map[par][w][2][lane] = R;
    __syncthreads();
    vec<V> q;  // what the tokens right of this warp's send to its last state
    if (K > 1) {
      if (w == 0) {
        vec<V> cp = warp_map[par][NW - 1][0][lane], cr = warp_map[par][NW - 1][2][lane];
#pragma unroll
        for (int k = NW - 2; k >= 0; --k) {
          const vec<V> kp = warp_map[par][k][0][lane];
          cr = vfma(kp, cr, warp_map[par][k][2][lane]);
          cp = vmul(cp, kp);
        }
        for (int k = 0; k < K; ++k) {
          st_peer(peer_addr(smem_u32(&cta_map[par][rank][0][lane]), k), cp);
          st_peer(peer_addr(smem_u32(&cta_map[par][rank][1][lane]), k), cr);
        }
      }
      cluster_sync();
      q = carry;
#pragma unroll
      for (int k = kMaxCluster - 1; k >= 0; --k) {
        if (k == rank) q = carry;
        if (k < K) carry = vfma(cta_map[par][k][0][lane], carry, cta_map[par][k][1][lane]);
      }
    } else {
      if (step + 1 < p.steps) carry = end_adjoint[par][lane];
      q = carry;
    }
#pragma unroll
    for (int k = 0; k < NW - 1; ++k) {
      const int r = NW - 1 - k;
      if (k < w) h = vfma(warp_map[par][k][0][lane], h, warp_map[par][k][1][lane]);
      if (r > w) q = vfma(warp_map[par][r][0][lane], q, warp_map[par][r][2][lane]);
    }
    // x becomes what da multiplies: the state that the token starts from, less x with the complement
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const vec<V> was = h;
      h = vfma(a[i], was, COMP ? vmul(xv[i], s[i]) : xv[i]);
      xv[i] = COMP ? vsub(was, xv[i]) : was;
    }
    const bool full = mine && now + TW <= p.L;
    IO* dxp = dx + (b * p.L + now) * p.D + c;
    IO* dgp = dgate + (b * p.L + now) * p.D + c;
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) {
      const vec<V> G = vadd(d[i], q);
      q = vmul(a[i], G);
      vec<V> og = vmul(KIND == SSD_GATE_DECAY ? G : q, xv[i]);
      if constexpr (KIND == SSD_GATE_LOGIT) og = vmul(og, s[i]);
      if (full || (mine && now + i < p.L)) {
        store<IO, V>(dxp + i * p.D, COMP ? vmul(G, s[i]) : G);
        store<IO, V>(dgp + i * p.D, og);
      }
    }
    if (K == 1 && w == 0) {
      carry = q;
      end_adjoint[par ^ 1][lane] = q;
    }
  }
  if (dinit && rank == 0 && w == 0 && mine) store_f32<V>(dinit + b * p.D + c, carry);
  if (K > 1) cluster_sync();
  grid_dep_launch();
}

// ------------------------------------------------------------------------------ launches

// CTAs along the sequence in one cluster.
int cluster_size(int64_t columns, int64_t tiles) {
  int K = 1;
  while (K < kMaxCluster && columns * K < kSMs && 2 * K <= tiles) K *= 2;
  return K;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, int threads, int cluster, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Two channels a thread need rows that start at a pair.
bool pairs(const GatedProblem& p, const void* x, const void* gate) {
  const size_t e = p.io_bf16 ? 2 : 4;
  return p.D % 2 == 0 && p.sx % 2 == 0 && p.sg % 2 == 0 && aligned(x, 2 * e) && aligned(gate, 2 * e);
}

template <typename IO, int V, int KIND, bool COMP>
struct Launch {
  static cudaError_t scan(const GatedProblem& p, const void* x, const void* gate, const float* init, void* y,
                          float* final_state, float* states, bool run, cudaStream_t st) {
    ScanArgs a{p.L, p.D, p.sx, p.sg, 1, 1};
    if (run) {
      const dim3 grid(static_cast<unsigned>((p.D / V + 127) / 128), static_cast<unsigned>(p.b));
      return launch_pdl(run_kernel<IO, V, KIND, COMP>, grid, dim3(128), 0, st, a, static_cast<const IO*>(x),
                        static_cast<const IO*>(gate), init, static_cast<IO*>(y), final_state, states);
    }
    constexpr int NW = 8, TW = sizeof(IO) == 2 ? 16 : 8;
    const int64_t columns = (p.D + 32 * V - 1) / (32 * V), tiles = (p.L + NW * TW - 1) / (NW * TW);
    a.cluster = cluster_size(columns * p.b, tiles);
    a.steps = static_cast<int>((tiles + a.cluster - 1) / a.cluster);
    return launch_cluster(scan_kernel<IO, V, KIND, COMP, NW, TW>,
                          dim3(static_cast<unsigned>(columns * a.cluster), static_cast<unsigned>(p.b)), NW * 32,
                          a.cluster, st, a, static_cast<const IO*>(x), static_cast<const IO*>(gate), init,
                          static_cast<IO*>(y), final_state, states);
  }
  static cudaError_t bwd(const GatedProblem& p, const void* x, const void* gate, const void* dy, const float* states,
                         const float* dfinal, void* dx, void* dgate, float* dinit, cudaStream_t st) {
    constexpr int TW = sizeof(IO) == 2 ? 8 : 4, NW = SSD_GATED_BLOCK / TW;
    ScanArgs a{p.L, p.D, p.sx, p.sg, 1, 1};
    const int64_t columns = (p.D + 32 * V - 1) / (32 * V), tiles = (p.L + NW * TW - 1) / (NW * TW);
    a.cluster = cluster_size(columns * p.b, tiles);
    a.steps = static_cast<int>((tiles + a.cluster - 1) / a.cluster);
    return launch_cluster(scan_bwd_kernel<IO, V, KIND, COMP, NW, TW>,
                          dim3(static_cast<unsigned>(columns * a.cluster), static_cast<unsigned>(p.b)), NW * 32,
                          a.cluster, st, a, static_cast<const IO*>(x), static_cast<const IO*>(gate),
                          static_cast<const IO*>(dy), states, dfinal, static_cast<IO*>(dx), static_cast<IO*>(dgate),
                          dinit);
  }
};

// Calls f with the Launch<> of the problem's type, width, gate and input.
template <typename F>
cudaError_t with_launch(const GatedProblem& p, bool two, F f) {
  auto by_comp = [&](auto io, auto v, auto kind) {
    using IO = decltype(io);
    return p.complement ? f(Launch<IO, decltype(v)::value, decltype(kind)::value, true>())
                        : f(Launch<IO, decltype(v)::value, decltype(kind)::value, false>());
  };
  auto by_kind = [&](auto io, auto v) {
    if (p.kind == SSD_GATE_DECAY) return by_comp(io, v, std::integral_constant<int, SSD_GATE_DECAY>());
    if (p.kind == SSD_GATE_LOG) return by_comp(io, v, std::integral_constant<int, SSD_GATE_LOG>());
    return by_comp(io, v, std::integral_constant<int, SSD_GATE_LOGIT>());
  };
  auto by_width = [&](auto io) {
    return two ? by_kind(io, std::integral_constant<int, 2>()) : by_kind(io, std::integral_constant<int, 1>());
  };
  return p.io_bf16 ? by_width(uint16_t()) : by_width(float());
}

}  // namespace

cudaError_t launch_gated_scan(const GatedProblem& p, const void* x, const void* gate, const float* init, void* y,
                              float* final_state, float* states, cudaStream_t st) {
  return with_launch(p, pairs(p, x, gate), [&](auto l) {
    return decltype(l)::scan(p, x, gate, init, y, final_state, states, p.L <= 16, st);
  });
}

cudaError_t launch_gated_scan_bwd(const GatedProblem& p, const void* x, const void* gate, const void* dy,
                                  const float* states, const float* dfinal, void* dx, void* dgate, float* dinit,
                                  cudaStream_t st) {
  return with_launch(p, pairs(p, x, gate), [&](auto l) {
    return decltype(l)::bwd(p, x, gate, dy, states, dfinal, dx, dgate, dinit, st);
  });
}

cudaError_t launch_gated_decode(const GatedProblem& p, const void* x, const void* gate, const float* state,
                                float* new_state, void* y, cudaStream_t st) {
  return with_launch(p, pairs(p, x, gate), [&](auto l) {
    return decltype(l)::scan(p, x, gate, state, y, new_state, nullptr, true, st);
  });
}

}  // namespace ssd
