// gated_scan_bwd -- backward pass of the gated linear recurrence.
//
// "3.3 Hardware-aware algorithm and GPU memory hierarchy" (booiljung.github.io), section 6: the states are recomputed
// on chip, from those that the forward pass has left at every SSD_GATED_BLOCK-th token.
//
// The adjoint runs from the right.  With c_t what the tokens right of t send to h_t, G_t = dy_t + c_t and
// c_{t-1} = a_t G_t: over a run of tokens an affine map c -> P c + R, with the forward map's product P.  Warps, CTAs,
// clusters and segments share the work as in the forward pass, in the other direction.  A CTA's tile is one
// block, so only the adjoint is carried between CTAs and steps; inside a tile each warp reduces its tokens to
// (P, H, R), walks the states forward from the one that enters its tokens and the adjoint backward from the one that
// leaves them.  x, gate and dy are read once, dx and dgate written once.
//
// Bound by instructions (51 a value; bf16 b2 L8192 D5120: 51% of the issue slots, DRAM 44% busy) and the one barrier a step.
// b2 L8192 D5120 233 us with bf16 (53% of the measured copy bandwidth), 304 us with float32 (82%).  With an extra warp that
// exchanges the maps, as the forward pass has it, the best of its shapes took 253 us against 223 without (both with
// the decays straight from the MUFU unit): it takes registers that the 8 tokens of four arrays need.
#include "gated.cuh"

namespace ssd {
namespace gated {
namespace {

constexpr int kWarps = 8, kResident = 2;
constexpr int kTok = SSD_GATED_BLOCK / kWarps;  // tokens of a warp's tile
// Whether dx and dgate have a place of their own, so that the slot is refilled as soon as it has been read.  With float32
// that would leave one CTA an SM: they take the slot's.
template <typename IO>
constexpr bool kStaged = sizeof(IO) == 2;

// Adds dfinal to what the tile's last token has from dy, where that is the sequence's last.
__device__ __forceinline__ void add_final(float2 (&d)[kTok], const float* dfinal, int64_t t0, const Args& p, int64_t b,
                                          int64_t c) {
  if (dfinal && t0 < p.L && p.L <= t0 + kTok) {
    const float2 f = load_row(dfinal + b * p.D, c, p.D);
#pragma unroll
    for (int i = 0; i < kTok; ++i)
      if (t0 + i == p.L - 1) d[i] = vadd(d[i], f);
  }
}

template <typename IO, int KIND, bool COMP, int G, int NS>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_bwd_kernel(
    const Args p, const IO* __restrict__ x, const IO* __restrict__ gate, const IO* __restrict__ dy,
    const float* __restrict__ states, const float* __restrict__ dfinal, IO* __restrict__ dx, IO* __restrict__ dgate,
    float* __restrict__ dinit, const Maps maps) {
  using T = Tile<IO, G, kTok, kCols>;
  constexpr int kSlot = 3 * T::kBytes;
  extern __shared__ __align__(128) char ring[];
  __shared__ float2 warp_map[2][kWarps][3][32];
  __shared__ float2 end_adjoint[2][32];  // what leaves a step's first token, where the cluster is one CTA
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int K = p.cluster;
  const int rank = K > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t b = blockIdx.y, seg = blockIdx.z;
  const int64_t col = int64_t(blockIdx.x / K) * kCols, c = col + 2 * lane;
  if (K > 1) {  // every CTA of the cluster runs before its shared memory is written to
    cluster_arrive();
    cluster_wait();
  }
  const int left = static_cast<int>(p.D - col < kCols ? p.D - col : kCols);
  const int64_t blocks = (p.L + SSD_GATED_BLOCK - 1) / SSD_GATED_BLOCK;
  const int64_t span = int64_t(K) * SSD_GATED_BLOCK;
  const int64_t start = seg * p.seg_len, end = seg + 1 < p.segments ? start + p.seg_len : p.L;
  // this warp's tokens of the last step; those behind the end are zeros, which send nothing to the left
  int64_t t0 = start + (int64_t(p.steps - 1) * K + rank) * SSD_GATED_BLOCK + w * kTok;
  const IO* xb = x + b * p.L * p.sx + col;
  const IO* gb = gate + b * p.L * p.sg + col;
  const IO* db = dy + b * p.L * p.D + col;
  // shared memory: each warp's slots (and the tiles its dx and dgate leave from), then the CTAs' maps of even and odd steps
  constexpr int kWarpBytes = NS * kSlot + (kStaged<IO> ? 2 * T::kBytes : 0);
  char* slots = ring + w * kWarpBytes;
  float2(*cta_maps)[2][32] = reinterpret_cast<float2(*)[2][32]>(ring + kWarps * kWarpBytes);

  grid_dep_wait();
  auto fetch = [&](int slot, int64_t t) {
    char* s = slots + slot * kSlot;
    if (t >= start) {
      T::in(s, xb, p.sx, t, end, left, lane, x);
      T::in(s + T::kBytes, gb, p.sg, t, end, left, lane, gate);
      T::in(s + 2 * T::kBytes, db, p.D, t, end, left, lane, dy);
    }
    copies_commit();
  };
  auto state_of = [&](int64_t t) {  // the state that enters the block of token t
    const int64_t block = t / SSD_GATED_BLOCK;
    return t >= start && block < blocks ? load_row(states + (b * blocks + block) * p.D, c, p.D) : make_float2(0.f, 0.f);
  };
#pragma unroll
  for (int k = 0; k < NS; ++k) fetch(k, t0 - k * span);
  float2 next_state = state_of(t0);

  float2 carry = make_float2(0.f, 0.f);  // what enters the step from its right
  if (seg + 1 < p.segments) {  // fold the maps of the segments behind, the last one first
    const int behind = p.segments - 1 - static_cast<int>(seg), per = (behind + kWarps - 1) / kWarps;
    float2 P = make_float2(1.f, 1.f), R = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int k = w * per; k < (w + 1) * per && k < behind; ++k) {
      const float2 kp = *maps.pair_at(p.segments - 1 - k, gridDim.y, b, 0, c);
      R = fma_f32x2(kp, R, *maps.pair_at(p.segments - 1 - k, gridDim.y, b, 1, c));
      P = mul_f32x2(P, kp);
    }
    const int par = p.steps & 1;  // the buffer that the first step does not write to
    warp_map[par][w][0][lane] = P;
    warp_map[par][w][1][lane] = R;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarps; ++k) carry = fma_f32x2(warp_map[par][k][0][lane], carry, warp_map[par][k][1][lane]);
  }

  int slot = 0;
  for (int step = p.steps - 1; step >= 0; --step) {
    const int par = step & 1;
    char* sl = slots + slot * kSlot;
    char* stage = kStaged<IO> ? slots + NS * kSlot : sl;
    float2(*cta_map)[2][32] = cta_maps + par * K;
    const auto xs = T::reader(sl, xb, p.sx, t0, lane), gs = T::reader(sl + T::kBytes, gb, p.sg, t0, lane);
    const auto ds = T::reader(sl + 2 * T::kBytes, db, p.D, t0, lane);
    float2 h = next_state;
    next_state = state_of(t0 - span);
    copies_wait<NS - 1>();
    __syncwarp();
    float2 a[kTok], s[kTok], xv[kTok], d[kTok];
    float2 P = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f), R = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      gate_of<IO, KIND, true>(gs[i], a[i], s[i]);
      xv[i] = xs[i];
      d[i] = ds[i];
      H = chain_fma(a[i], H, COMP ? mul_f32x2(xv[i], s[i]) : xv[i]);
    }
    add_final(d, dfinal, t0, p, b, c);
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      P = chain_mul(P, a[i]);
      R = chain_fma(P, d[i], R);
    }
    __syncwarp();
    if constexpr (kStaged<IO>) fetch(slot, t0 - NS * span);
    warp_map[par][w][0][lane] = P;
    warp_map[par][w][1][lane] = H;
    warp_map[par][w][2][lane] = R;
    __syncthreads();
    float2 q;  // what the tokens right of this warp's send to its last state
    if (K > 1) {
      if (w == 0) {
        publish_map(cta_map, warp_map[par], rank, K, lane);
        cluster_arrive();
      } else {
        cluster_arrive_relaxed();
      }
      P = make_float2(1.f, 1.f);
      R = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps - 1; ++k) {
        const int r = kWarps - 1 - k;
        if (k < w) h = fma_f32x2(warp_map[par][k][0][lane], h, warp_map[par][k][1][lane]);
        if (r > w) {
          const float2 kp = warp_map[par][r][0][lane];
          R = fma_f32x2(kp, R, warp_map[par][r][2][lane]);
          P = mul_f32x2(P, kp);
        }
      }
      cluster_wait();
      q = carry;
      for (int k = K - 1; k >= 0; --k) {
        if (k == rank) q = carry;
        carry = fma_f32x2(cta_map[k][0][lane], carry, cta_map[k][1][lane]);
      }
      q = fma_f32x2(P, q, R);
    } else {
      q = step + 1 < p.steps ? end_adjoint[par][lane] : carry;
#pragma unroll
      for (int k = 0; k < kWarps - 1; ++k) {
        const int r = kWarps - 1 - k;
        if (k < w) h = fma_f32x2(warp_map[par][k][0][lane], h, warp_map[par][k][1][lane]);
        if (r > w) q = fma_f32x2(warp_map[par][r][0][lane], q, warp_map[par][r][2][lane]);
      }
    }
    // x becomes what da multiplies: the state that the token starts from, less x with the complement
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const float2 was = h;
      h = chain_fma(a[i], was, COMP ? mul_f32x2(xv[i], s[i]) : xv[i]);
      xv[i] = COMP ? vsub(was, xv[i]) : was;
    }
    __syncwarp();
    pair_t<IO>* xo = reinterpret_cast<pair_t<IO>*>(stage) + lane;
    pair_t<IO>* go = reinterpret_cast<pair_t<IO>*>(stage + T::kBytes) + lane;
#pragma unroll
    for (int i = kTok - 1; i >= 0; --i) {
      const float2 Gt = vadd(d[i], q);
      q = mul_f32x2(a[i], Gt);
      float2 og = mul_f32x2(KIND == SSD_GATE_DECAY ? Gt : q, xv[i]);
      if constexpr (KIND == SSD_GATE_LOGIT) og = mul_f32x2(og, s[i]);
      narrow(xo[i * 32], COMP ? mul_f32x2(Gt, s[i]) : Gt);
      narrow(go[i * 32], og);
    }
    if (K == 1 && w == 0) end_adjoint[par ^ 1][lane] = q;
    if (dinit && t0 == 0) store_row(dinit + b * p.D, c, p.D, q);
    __syncwarp();
    T::out(stage, dx + b * p.L * p.D + col, p.D, t0, end, left, lane);
    T::out(stage + T::kBytes, dgate + b * p.L * p.D + col, p.D, t0, end, left, lane);
    if constexpr (!kStaged<IO>) {
      __syncwarp();
      fetch(slot, t0 - NS * span);
    }
    t0 -= span;
    slot = slot + 1 == NS ? 0 : slot + 1;
  }
  if (K > 1) {  // no CTA leaves while another may still write to its shared memory
    cluster_arrive_relaxed();
    cluster_wait();
  }
  grid_dep_launch();
}

// The adjoint's map of each segment.  A CTA's warps take an eighth of it each; a token behind a run makes its map
// c -> P (a (dy + c)) + R.
template <typename IO, int KIND, int G, int NS>
__global__ void __launch_bounds__(kWarps * 32) map_bwd_kernel(const Args p, const IO* __restrict__ gate,
                                                              const IO* __restrict__ dy,
                                                              const float* __restrict__ dfinal, const Maps maps) {
  using T = Tile<IO, G, kTok, kCols>;
  extern __shared__ __align__(128) char ring[];
  __shared__ float2 warp_map[kWarps][2][32];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int64_t b = blockIdx.y, seg = blockIdx.z;
  const int64_t col = int64_t(blockIdx.x) * kCols, c = col + 2 * lane;
  const int left = static_cast<int>(p.D - col < kCols ? p.D - col : kCols);
  const IO* gb = gate + b * p.L * p.sg + col;
  const IO* db = dy + b * p.L * p.D + col;
  char* slots = ring + w * (NS * 2 * T::kBytes);
  const int64_t run = p.seg_len / kWarps, t0 = seg * p.seg_len + w * run, end = t0 + run < p.L ? t0 + run : p.L;
  grid_dep_launch();  // the scan may be launched; it waits for this kernel's end before it reads the maps
  grid_dep_wait();
  float2 P = make_float2(1.f, 1.f), R = make_float2(0.f, 0.f);
  if (seg > 0) {  // no segment is before the first one
    auto fetch = [&](int slot, int64_t t) {
      char* s = slots + slot * (2 * T::kBytes);
      T::in(s, gb, p.sg, t, end, left, lane, gate);
      T::in(s + T::kBytes, db, p.D, t, end, left, lane, dy);
      copies_commit();
    };
#pragma unroll
    for (int k = 0; k < NS; ++k) fetch(k, t0 + k * kTok);
    int slot = 0;
    for (int64_t t = t0; t < end; t += kTok) {
      const char* tile = slots + slot * (2 * T::kBytes);
      const auto gs = T::reader(tile, gb, p.sg, t, lane), ds = T::reader(tile + T::kBytes, db, p.D, t, lane);
      copies_wait<NS - 1>();
      __syncwarp();
      float2 d[kTok], a[kTok], s;
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        gate_of<IO, KIND, true>(gs[i], a[i], s);
        d[i] = ds[i];
      }
      add_final(d, dfinal, t, p, b, c);
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        P = chain_mul(P, a[i]);
        R = chain_fma(P, d[i], R);
      }
      __syncwarp();
      fetch(slot, t + NS * kTok);
      slot = slot + 1 == NS ? 0 : slot + 1;
    }
  }
  warp_map[w][0][lane] = P;
  warp_map[w][1][lane] = R;
  __syncthreads();
  if (w == kWarps - 1) {
#pragma unroll
    for (int k = kWarps - 2; k >= 0; --k) {
      const float2 kp = warp_map[k][0][lane];
      R = fma_f32x2(kp, R, warp_map[k][1][lane]);
      P = mul_f32x2(P, kp);
    }
    *maps.pair_at(seg, gridDim.y, b, 0, c) = P;
    *maps.pair_at(seg, gridDim.y, b, 1, c) = R;
  }
}

// Few columns leave SMs without work even in clusters: then segments, if the sequence is long enough to be worth a second
// reading of gate and dy.  (Segments against clusters, bf16, us: 24 columns, 2048 tokens 13.6 and 13.8, 32768 tokens 134 and
// 188; 32 columns, 2048 tokens 16.5 and 14.3, 8192 tokens 51 and 51, 32768 tokens 172 and 197; 47 columns, 8192 tokens
// 72 and 77, 32768 tokens 253 and 298; 64 columns, 8192 tokens 99 and 94, with float32 142 and 119.)
bool in_segments(const GatedProblem& p) {
  const int64_t columns = columns64(p) * p.b;
  return columns < 48 && p.L >= (columns <= 24 ? 32 : 128) * SSD_GATED_BLOCK;
}
Plan bwd_segments(const GatedProblem& p) {
  return segment_plan(p, columns64(p), SSD_GATED_BLOCK, int64_t(kResident) * kSMs / (columns64(p) * p.b), SSD_GATED_BLOCK);
}

}  // namespace
}  // namespace gated

size_t gated_bwd_workspace_bytes(const GatedProblem& p) {
  return gated::in_segments(p) ? gated::maps_bytes(p, gated::bwd_segments(p)) : 0;
}

cudaError_t launch_gated_scan_bwd(const GatedProblem& p, const void* x, const void* gate, const void* dy,
                                  const float* states, const float* dfinal, void* dx, void* dgate, float* dinit,
                                  void* ws, cudaStream_t st) {
  using namespace gated;
  const Maps maps{static_cast<float*>(ws), columns64(p) * kCols};
  return with_types(p, piece_bytes(p, x, gate), [&](auto io, auto g, auto kind, auto comp) {
    using IO = decltype(io);
    constexpr int G = decltype(g)::value, KIND = decltype(kind)::value, NS = 2;
    constexpr bool COMP = decltype(comp)::value;
    constexpr auto kern = scan_bwd_kernel<IO, KIND, COMP, G, NS>;
    constexpr size_t bytes = Tile<IO, G, kTok, kCols>::kBytes;
    auto smem = [](int K) { return kWarps * (NS * 3 + (kStaged<IO> ? 2 : 0)) * bytes + size_t(K) * 1024; };
    const IO* xi = static_cast<const IO*>(x);
    const IO* gi = static_cast<const IO*>(gate);
    const IO* di = static_cast<const IO*>(dy);
    Plan plan;
    cudaError_t e = cudaSuccess;
    if (in_segments(p)) {
      plan = bwd_segments(p);
      e = launch<map_bwd_kernel<IO, KIND, G, NS>>(plan, p.b, kWarps * 32, kWarps * NS * 2 * bytes, st, plan.args(p), gi, di,
                                                  dfinal, maps);
    } else {
      e = cluster_plan<kern>(p, SSD_GATED_BLOCK, kWarps * 32, smem, &plan);
    }
    if (e != cudaSuccess) return e;
    return launch<kern>(plan, p.b, kWarps * 32, smem(plan.cluster), st, plan.args(p), xi, gi, di, states, dfinal,
                        static_cast<IO*>(dx), static_cast<IO*>(dgate), dinit, maps);
  });
}

}  // namespace ssd
