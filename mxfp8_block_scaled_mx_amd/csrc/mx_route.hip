// Router of the MoE layer: the top-k experts of each token and their routing
// weights from the router's logits, and the gradient back to the logits
// (each token activates a few experts: "Efficient MoE training for biological
// foundation models", Dense vs. MoE scaling). What it makes is what
// mx_moe_dispatch and grouped_mlp_decode take; its gradient starts from the
// dprobs that the grouped MLP's backward hands out per routed row.
//
// One token is G neighbouring lanes with V consecutive experts each, so the
// whole row sits in registers: one pass over the logits. A pick is the largest
// key left (a maximum over the lane's V keys, then over the G lanes), and of
// equal keys the lowest expert's: the first lane that holds the maximum, and
// its first key. All sums are fp32.
//
// Both directions are bound by the launch and by one chain of dependent steps a
// pick (8192 tokens of 8 experts: 3.1 us; 33 tokens of 128 experts, 8 picks: 4.7
// us; gradient of 16383 tokens of 128 experts in bf16: 5.3 us for 9.5 MB, 1.8
// TB/s), so what they save is latency: maxima and sums go over the lanes by DPP and
// permlane moves (through LDS: 6.2 us for the 33 tokens), and the gradient's
// picks are scattered through LDS (a loop over the picks in every lane: 8.0 us).
#include "mx_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

constexpr float kShut = -__builtin_inff();

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, 0xF, 0xF, false));
}
// The lane's value combined with that of lane ^ 1, ^ 2, then of the mirrored
// half row and row (the four, and then eight, lanes agree by then), then of
// lane ^ 16: all without LDS.
template <int G, typename Op>
__device__ __forceinline__ float group_reduce(float v, const Op& op) {
  v = op(v, dpp<0xB1>(v));                                // quad_perm [1, 0, 3, 2]
  v = op(v, dpp<0x4E>(v));                                // quad_perm [2, 3, 0, 1]
  v = op(v, dpp<0x141>(v));                               // row_half_mirror
  if constexpr (G >= 16) v = op(v, dpp<0x140>(v));        // row_mirror
  if constexpr (G >= 32) {
    const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r.x), __uint_as_float(r.y));
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<G>(v, [](float a, float b) { return a + b; });
}

// V values from element `at` of a row of bf16 or fp32 (the first `left` of them
// exist; vec: all do, and they are aligned as one word).
template <int V, bool F32>
__device__ __forceinline__ void load_values(const void* p, int64_t at, int left, bool vec, float (&z)[V]) {
  if (V == 4 && vec) {
    if constexpr (F32) {
      const v4f v = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(p) + at);
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = v[i];
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + at);
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = i & 1 ? bf16_hi(i < 2 ? v.x : v.y) : bf16_lo(i < 2 ? v.x : v.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z[i] = kShut;
      if (i < left)
        z[i] = F32 ? reinterpret_cast<const float*>(p)[at + i]
                   : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[at + i] << 16);
    }
  }
}

// The lane's V logits (experts at or past E are shut), and the keys that
// decide: logit + bias. A key of -inf or NaN is shut: never picked.
template <int V, bool F32>
__device__ __forceinline__ void load_row(const void* logits, const float* bias, int64_t t, int32_t E, int e0, bool vec,
                                         float (&z)[V], float (&key)[V]) {
  if (e0 < E) {
    load_values<V, F32>(logits, t * E + e0, E - e0, vec, z);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = kShut;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float k = z[v];
    if (bias != nullptr && e0 + v < E) k += bias[e0 + v];
    if (!(k > kShut)) k = z[v] = kShut;
    key[v] = k;
  }
}

template <int G, int V, bool F32>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63, gl = lane % G, base = lane - gl;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const bool live = t < a.tokens;
  const int64_t tc = live ? t : a.tokens - 1;             // lanes past the end repeat the last token, unused
  float z[V], key[V];
  load_row<V, F32>(a.logits, a.bias, tc, a.experts, gl * V, a.vec, z, key);

  float zm = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) zm = fmaxf(zm, z[v]);
  zm = group_max<G>(zm);
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += z[v] > kShut ? expf(z[v] - zm) : 0.f;
  sum = group_sum<G>(sum);

  // lane gl keeps pick gl (topk <= G)
  int my_e = -1;
  for (int j = 0; j < a.topk; ++j) {
    float best = key[0];
    int bv = 0;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        bv = v;
      }
    const float top = group_max<G>(best);
    // some lane of the group holds the maximum
    const uint32_t has = (uint32_t)(__ballot(best == top) >> base);
    const int owner = __ffs(has) - 1;
    const int et = V == 1 ? owner : __shfl(gl * V + bv, base + owner, 64);
    if (gl == owner) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = bv == v ? kShut : key[v];
    }
    if (gl == j && top > kShut) my_e = et;
  }
  float my_z = kShut;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float f = __shfl(z[v], base + (my_e >= 0 ? my_e / V : 0), 64);
    if (my_e >= 0 && my_e % V == v) my_z = f;
  }
  float ref = zm, total = sum;
  if (a.renorm) {
    ref = group_max<G>(my_z);
    total = group_sum<G>(my_e >= 0 ? expf(my_z - ref) : 0.f);
  }
  const float w = my_e >= 0 ? expf(my_z - ref) / total : 0.f;
  if (live && gl < a.topk) {
    a.topk_idx[t * a.topk + gl] = my_e;
    a.topk_w[t * a.topk + gl] = w;
  }
  if (live && gl == 0) a.lse[t] = sum > 0.f ? zm + logf(sum) : kShut;
}

// dz_e = p_e ([e picked as j] dw_j - sum_i w_i dw_i) with p the softmax that
// the weights came from: over the picks (renorm; zero elsewhere) or over all
// experts that are not shut. The picks' parts are scattered to their experts
// through LDS, in rows that one wave writes and reads.
template <int G, int V, bool F32>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs a) {
  __shared__ __align__(16) float part_of[256 / G][G * V];
  const int lane = threadIdx.x & 63, gl = lane % G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const bool live = t < a.tokens;
  const int64_t tc = live ? t : a.tokens - 1;
  float* const row = part_of[threadIdx.x / G];
  const int e0 = gl * V;
  float z[V], key[V], lse = 0.f;
  if (!a.renorm) {
    load_row<V, F32>(a.logits, a.bias, tc, a.experts, e0, a.vec, z, key);
    lse = a.lse[tc];
  }
  int my_e = -1;
  float w = 0.f, dw = 0.f;
  if (gl < a.topk) {
    const int64_t at = tc * a.topk + gl;
    my_e = a.topk_idx[at];
    if (my_e >= 0 && my_e < a.experts) {
      const int64_t r = a.perm != nullptr ? (int64_t)a.perm[at] : at;
      w = a.topk_w[at];
      if (r >= 0 && r < a.dw_rows) dw = a.dw[r];
    } else {
      my_e = -1;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) row[e0 + v] = 0.f;
  const float wdw = w * dw, dot = group_sum<G>(wdw);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (my_e >= 0) row[my_e] = a.renorm ? w * (dw - dot) : wdw;
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  float dz[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    dz[v] = row[e0 + v];
    if (!a.renorm && z[v] > kShut) dz[v] -= expf(z[v] - lse) * dot;
  }
  if (!live || e0 >= a.experts) return;
  const int64_t at = t * a.experts + e0;
  if (V == 4 && a.vec) {
    if constexpr (F32) {
      v4f o;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v & 3] = dz[v];
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.dlogits) + at) = o;
    } else {
      typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
      bf16x4 o;
#pragma unroll
      for (int v = 0; v < V; ++v) o[v & 3] = (__bf16)dz[v];
      *reinterpret_cast<bf16x4*>(reinterpret_cast<__bf16*>(a.dlogits) + at) = o;
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (e0 + v < a.experts) {
      if (F32)
        reinterpret_cast<float*>(a.dlogits)[at + v] = dz[v];
      else
        reinterpret_cast<__bf16*>(a.dlogits)[at + v] = (__bf16)dz[v];
    }
}

// Whether rows of `experts` values can be read and written four at a time.
bool by_fours(int32_t experts, int32_t f32, const void* p) {
  return experts % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (f32 ? 16 : 8) == 0;
}

// Lanes per token and experts per lane: topk <= G (at most 16 picks) and experts
// <= G * V; the fewest lanes that hold a row, since a pick's steps over the lanes
// grow with G and those over a lane's keys with V.
template <typename Go>
void by_shape(int32_t experts, const Go& go) {
  if (experts <= 8)
    go(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  else if (experts <= 16)
    go(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  else if (experts <= 64)
    go(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  else
    go(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
}

}  // namespace

hipError_t launch_route(const RouteArgs& args, hipStream_t stream) {
  RouteArgs a = args;
  a.vec = by_fours(a.experts, a.f32, a.logits);
  by_shape(a.experts, [&](auto g_, auto v_) {
    constexpr int G = decltype(g_)::value, V = decltype(v_)::value, per = 256 / G;
    const dim3 grid((unsigned)((a.tokens + per - 1) / per));
    if (a.f32)
      hipLaunchKernelGGL((route_kernel<G, V, true>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((route_kernel<G, V, false>), grid, dim3(256), 0, stream, a);
  });
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdArgs& args, hipStream_t stream) {
  RouteBwdArgs a = args;
  a.vec = by_fours(a.experts, a.f32, a.logits) && by_fours(a.experts, a.f32, a.dlogits);
  by_shape(a.experts, [&](auto g_, auto v_) {
    constexpr int G = decltype(g_)::value, V = decltype(v_)::value, per = 256 / G;
    const dim3 grid((unsigned)((a.tokens + per - 1) / per));
    if (a.f32)
      hipLaunchKernelGGL((route_bwd_kernel<G, V, true>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((route_bwd_kernel<G, V, false>), grid, dim3(256), 0, stream, a);
  });
  return hipGetLastError();
}

}  // namespace mx
