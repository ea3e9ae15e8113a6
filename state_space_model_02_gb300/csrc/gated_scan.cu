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

// V neighbouring values of one token as they lie in memory
template <typename IO, int V>
struct Raw {
  using type = std::conditional_t<sizeof(IO) * V == 2, uint16_t,
                                  std::conditional_t<sizeof(IO) * V == 4, uint32_t, uint2>>;
};
template <typename IO, int V>
using raw_t = typename Raw<IO, V>::type;

template <typename IO, int V>
__device__ __forceinline__ void widen(raw_t<IO, V> r, float (&f)[V]) {
  if constexpr (sizeof(IO) == 4 && V == 2) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
  } else if constexpr (sizeof(IO) == 4) {
    f[0] = __uint_as_float(r);
  } else if constexpr (V == 2) {
    f[0] = bf16lo_to_f32(r);
    f[1] = bf16hi_to_f32(r);
  } else {
    f[0] = __uint_as_float(uint32_t(r) << 16);
  }
}
template <typename IO, int V>
__device__ __forceinline__ raw_t<IO, V> narrow(const float (&f)[V]) {
  if constexpr (sizeof(IO) == 4 && V == 2)
    return make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1]));
  else if constexpr (sizeof(IO) == 4)
    return __float_as_uint(f[0]);
  else if constexpr (V == 2)
    return pack_bf16x2(f[0], f[1]);
  else
    return static_cast<uint16_t>(pack_bf16x2(f[0], 0.f));
}
template <typename IO, int V>
__device__ __forceinline__ raw_t<IO, V> load(const IO* p) {
  return __ldg(reinterpret_cast<const raw_t<IO, V>*>(p));
}
template <typename IO, int V>
__device__ __forceinline__ void store(IO* p, const float (&f)[V]) {
  *reinterpret_cast<raw_t<IO, V>*>(p) = narrow<IO, V>(f);
}
template <int V>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[V]) {
  if constexpr (V == 2) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    f[0] = v.x;
    f[1] = v.y;
  } else {
    f[0] = __ldg(p);
  }
}
template <int V>
__device__ __forceinline__ void store_f32(float* p, const float (&f)[V]) {
  if constexpr (V == 2)
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  else
    *p = f[0];
}

// The decay a and s = 1 - a.  s is taken from the gate, not from a: near a = 1 the difference has lost its low
// bits.  kS: whether s is used.
template <int KIND, bool kS>
__device__ __forceinline__ void gate_of(float g, float& a, float& s) {
  if constexpr (KIND == SSD_GATE_DECAY) {
    a = g;
    s = 1.f - g;
  } else if constexpr (KIND == SSD_GATE_LOG) {
    a = expf(g);
    if constexpr (kS) {
      // 1 - exp(g): for small |g| its series (the first term left out is g^6 / 5040 of it, under 5e-8)
      const float q = fmaf(g, fmaf(g, fmaf(g, fmaf(g, fmaf(g, 1.f / 720.f, 1.f / 120.f), 1.f / 24.f), 1.f / 6.f), 0.5f), 1.f);
      s = fabsf(g) < 0.25f ? -g * q : 1.f - a;
    }
  } else {
    const float e = expf(-fabsf(g)), r = __fdividef(1.f, 1.f + e), er = e * r;
    a = g >= 0.f ? r : er;
    s = g >= 0.f ? er : r;
  }
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
  __shared__ float warp_map[2][NW][2][V][32];
  __shared__ float cta_map[2][kMaxCluster][2][V][32];
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
        if (t0 + i < p.L) {
          xr[i] = load<IO, V>(xp + i * p.sx);
          gr[i] = load<IO, V>(gp + i * p.sg);
        }
      }
    }
  };
  fetch();
  float carry[V];  // the state that enters the cluster's step
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = 0.f;
  if (init) load_f32<V>(init + b * p.D + c, carry);

  for (int step = 0; step < p.steps; ++step) {
    const int par = step & 1;
    float a[TW][V], u[TW][V], P[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P[v] = 1.f;
      H[v] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const bool in = t0 + i < p.L;  // a token behind the last one leaves the state as it is
      float g[V], s;
      widen<IO, V>(gr[i], g);
      widen<IO, V>(xr[i], u[i]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gate_of<KIND, COMP>(g[v], a[i][v], s);
        if constexpr (COMP) u[i][v] *= s;
        if (!in) {
          a[i][v] = 1.f;
          u[i][v] = 0.f;
        }
        H[v] = fmaf(a[i][v], H[v], u[i][v]);
        P[v] *= a[i][v];
      }
    }
    const int64_t now = t0;
    t0 += span;
    xp += span * p.sx;
    gp += span * p.sg;
    if (step + 1 < p.steps) fetch();

#pragma unroll
    for (int v = 0; v < V; ++v) {
      warp_map[par][w][0][v][lane] = P[v];
      warp_map[par][w][1][v][lane] = H[v];
    }
    __syncthreads();
    if (K > 1) {
      if (w < K) {  // warp w tells CTA w
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float cp = 1.f, ch = 0.f;
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            const float kp = warp_map[par][k][0][v][lane];
            ch = fmaf(kp, ch, warp_map[par][k][1][v][lane]);
            cp *= kp;
          }
          st_peer(peer_addr(smem_u32(&cta_map[par][rank][0][v][lane]), w), cp);
          st_peer(peer_addr(smem_u32(&cta_map[par][rank][1][v][lane]), w), ch);
        }
      }
      cluster_sync();
    }
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = carry[v];
      if (K > 1) {
        for (int k = 0; k < K; ++k) {
          if (k == rank) h[v] = carry[v];
          carry[v] = fmaf(cta_map[par][k][0][v][lane], carry[v], cta_map[par][k][1][v][lane]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < NW; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float kp = warp_map[par][k][0][v][lane], kh = warp_map[par][k][1][v][lane];
        if (k < w) h[v] = fmaf(kp, h[v], kh);
        if (K == 1) carry[v] = fmaf(kp, carry[v], kh);
      }
    }
    if (states && now % SSD_GATED_BLOCK == 0 && now < p.L && mine)
      store_f32<V>(states + (b * blocks + now / SSD_GATED_BLOCK) * p.D + c, h);
    const bool full = now + TW <= p.L;
#pragma unroll
    for (int i = 0; i < TW; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], u[i][v]);
      if (mine && (full || now + i < p.L)) store<IO, V>(yp + i * p.D, h);
    }
    yp += span * p.D;
  }
  if (final_state && rank == 0 && w == 0 && mine) store_f32<V>(final_state + b * p.D + c, carry);
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
  float h[V] = {};
  if (init) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = init[b * p.D + c + v];
  }
#pragma unroll 4
  for (int64_t t = 0; t < p.L; ++t) {
    if (states && t % SSD_GATED_BLOCK == 0) store_f32<V>(states + (b * blocks + t / SSD_GATED_BLOCK) * p.D + c, h);
    float xv[V], g[V], a, s;
    widen<IO, V>(load<IO, V>(xp), xv);
    widen<IO, V>(load<IO, V>(gp), g);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      gate_of<KIND, COMP>(g[v], a, s);
      h[v] = fmaf(a, h[v], COMP ? s * xv[v] : xv[v]);
    }
    store<IO, V>(yp, h);
    xp += p.sx;
    gp += p.sg;
    yp += p.D;
  }
  if (final_state) {
#pragma unroll
    for (int v = 0; v < V; ++v) final_state[b * p.D + c + v] = h[v];
  }
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
  __shared__ float warp_map[2][NW][3][V][32];
  __shared__ float cta_map[2][kMaxCluster][2][V][32];
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
  float hr[V];
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
        if (t0 + i < p.L) {
          xr[i] = load<IO, V>(xp + i * p.sx);
          gr[i] = load<IO, V>(gp + i * p.sg);
          dr[i] = load<IO, V>(dp + i * p.D);
        }
      }
    }
    if (block < blocks) load_f32<V>(states + (b * blocks + block) * p.D + c, hr);
  };
#pragma unroll
  for (int v = 0; v < V; ++v) hr[v] = 0.f;
  fetch();
  float carry[V];  // what the tokens right of the cluster's step send to its last state
#pragma unroll
  for (int v = 0; v < V; ++v) carry[v] = 0.f;
  if (dfinal) load_f32<V>(dfinal + b * p.D + c, carry);

  for (int step = p.steps - 1; step >= 0; --step) {
    const int par = step & 1;
    float a[TW][V], s[TW][V], u[TW][V], xv[TW][V], d[TW][V], P[V], H[V], R[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P[v] = 1.f;
      H[v] = 0.f;
      R[v] = 0.f;
      h[v] = hr[v];
    }
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const bool in = t0 + i < p.L;
      float g[V];
      widen<IO, V>(gr[i], g);
      widen<IO, V>(xr[i], xv[i]);
      widen<IO, V>(dr[i], d[i]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gate_of<KIND, kS>(g[v], a[i][v], s[i][v]);
        u[i][v] = COMP ? s[i][v] * xv[i][v] : xv[i][v];
        if (!in) {
          a[i][v] = 1.f;
          u[i][v] = 0.f;
          d[i][v] = 0.f;
        }
        H[v] = fmaf(a[i][v], H[v], u[i][v]);
        P[v] *= a[i][v];
      }
    }
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) {
#pragma unroll
      for (int v = 0; v < V; ++v) R[v] = a[i][v] * (d[i][v] + R[v]);
    }
    const int64_t now = t0;
    block -= K;
    t0 -= int64_t(K) * SSD_GATED_BLOCK;
    if (step > 0) fetch();

#pragma unroll
    for (int v = 0; v < V; ++v) {
      warp_map[par][w][0][v][lane] = P[v];
      warp_map[par][w][1][v][lane] = H[v];
      warp_map[par][w][2][v][lane] = R[v];
    }
    __syncthreads();
    if (K > 1) {
      if (w < K) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float cp = 1.f, cr = 0.f;
#pragma unroll
          for (int k = NW - 1; k >= 0; --k) {
            const float kp = warp_map[par][k][0][v][lane];
            cr = fmaf(kp, cr, warp_map[par][k][2][v][lane]);
            cp *= kp;
          }
          st_peer(peer_addr(smem_u32(&cta_map[par][rank][0][v][lane]), w), cp);
          st_peer(peer_addr(smem_u32(&cta_map[par][rank][1][v][lane]), w), cr);
        }
      }
      cluster_sync();
    }
    float q[V];  // what the tokens right of this warp's send to its last state
#pragma unroll
    for (int v = 0; v < V; ++v) {
      q[v] = carry[v];
      if (K > 1) {
        for (int k = K - 1; k >= 0; --k) {
          if (k == rank) q[v] = carry[v];
          carry[v] = fmaf(cta_map[par][k][0][v][lane], carry[v], cta_map[par][k][1][v][lane]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int r = NW - 1 - k;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k < w) h[v] = fmaf(warp_map[par][k][0][v][lane], h[v], warp_map[par][k][1][v][lane]);
        const float kp = warp_map[par][r][0][v][lane], kr = warp_map[par][r][2][v][lane];
        if (r > w) q[v] = fmaf(kp, q[v], kr);
        if (K == 1) carry[v] = fmaf(kp, carry[v], kr);
      }
    }
    // u becomes what da multiplies: the state that the token starts from, less x with the complement
#pragma unroll
    for (int i = 0; i < TW; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float was = h[v];
        h[v] = fmaf(a[i][v], was, u[i][v]);
        u[i][v] = COMP ? was - xv[i][v] : was;
      }
    }
    const bool full = now + TW <= p.L;
    IO* dxp = dx + (b * p.L + now) * p.D + c;
    IO* dgp = dgate + (b * p.L + now) * p.D + c;
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) {
      float ox[V], og[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float G = d[i][v] + q[v];
        q[v] = a[i][v] * G;
        ox[v] = COMP ? G * s[i][v] : G;
        og[v] = KIND == SSD_GATE_DECAY ? G * u[i][v] : q[v] * u[i][v];
        if constexpr (KIND == SSD_GATE_LOGIT) og[v] *= s[i][v];
      }
      if (mine && (full || now + i < p.L)) {
        store<IO, V>(dxp + i * p.D, ox);
        store<IO, V>(dgp + i * p.D, og);
      }
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
