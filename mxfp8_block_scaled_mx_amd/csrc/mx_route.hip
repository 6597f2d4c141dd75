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
#include "mx_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

constexpr float kShut = -__builtin_inff();

template <int G, int V>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v = fmaxf(v, xor_f32(v, d));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v += xor_f32(v, d);
  return v;
}

// The lane's V logits (experts at or past E are shut), and the keys that
// decide: logit + bias. A key of -inf or NaN is shut: never picked.
template <int V, bool F32>
__device__ __forceinline__ void load_row(const void* logits, const float* bias, int64_t t, int32_t E, int e0,
                                         float (&z)[V], float (&key)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = e0 + v;
    float f = kShut;
    if (e < E)
      f = F32 ? reinterpret_cast<const float*>(logits)[t * E + e]
              : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(logits)[t * E + e] << 16);
    float k = f;
    if (bias != nullptr && e < E) k += bias[e];
    if (!(k > kShut)) k = f = kShut;
    z[v] = f;
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
  load_row<V, F32>(a.logits, a.bias, tc, a.experts, gl * V, z, key);

  float zm = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) zm = fmaxf(zm, z[v]);
  zm = group_max<G, V>(zm);
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += z[v] > kShut ? expf(z[v] - zm) : 0.f;
  sum = group_sum<G>(sum);

  // lane gl keeps pick gl (topk <= G)
  int my_e = -1;
  float my_z = kShut;
  for (int j = 0; j < a.topk; ++j) {
    float best = key[0];
    int bv = 0;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        bv = v;
      }
    const float top = group_max<G, V>(best);
    const uint64_t has = __ballot(best == top) >> base;
    const int owner = __ffsll((unsigned long long)has) - 1;  // within the group: some lane of it holds the maximum
    float zb = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) zb = bv == v ? z[v] : zb;
    const float zt = __shfl(zb, base + owner, 64);
    const int et = __shfl(gl * V + bv, base + owner, 64);
    if (gl == owner) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = bv == v ? kShut : key[v];
    }
    if (gl == j && top > kShut) {
      my_e = et;
      my_z = zt;
    }
  }
  float ref = zm, total = sum;
  if (a.renorm) {
    ref = group_max<G, V>(my_z);
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
// experts that are not shut.
template <int G, int V, bool F32>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs a) {
  const int lane = threadIdx.x & 63, gl = lane % G, base = lane - gl;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const bool live = t < a.tokens;
  const int64_t tc = live ? t : a.tokens - 1;
  int my_e = -1;
  float w = 0.f, dw = 0.f;
  if (gl < a.topk) {
    const int64_t at = tc * a.topk + gl;
    my_e = a.topk_idx[at];
    if (my_e >= 0 && my_e < a.experts) {
      const int64_t row = a.perm != nullptr ? (int64_t)a.perm[at] : at;
      w = a.topk_w[at];
      if (row >= 0 && row < a.dw_rows) dw = a.dw[row];
    } else {
      my_e = -1;
    }
  }
  const float wdw = w * dw, dot = group_sum<G>(wdw);
  const float part = a.renorm ? w * (dw - dot) : wdw;
  float dz[V];
  const int e0 = gl * V;
  if (a.renorm) {
#pragma unroll
    for (int v = 0; v < V; ++v) dz[v] = 0.f;
  } else {
    float z[V], key[V];
    load_row<V, F32>(a.logits, a.bias, tc, a.experts, e0, z, key);
    const float lse = a.lse[tc];
#pragma unroll
    for (int v = 0; v < V; ++v) dz[v] = z[v] > kShut ? -expf(z[v] - lse) * dot : 0.f;
  }
  for (int j = 0; j < a.topk; ++j) {
    const int e = __shfl(my_e, base + j, 64);
    const float p = __shfl(part, base + j, 64);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == e0 + v) dz[v] += p;
  }
  if (!live) return;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (e0 + v < a.experts) {
      if (F32)
        reinterpret_cast<float*>(a.dlogits)[t * a.experts + e0 + v] = dz[v];
      else
        reinterpret_cast<__bf16*>(a.dlogits)[t * a.experts + e0 + v] = (__bf16)dz[v];
    }
}

// Lanes per token and experts per lane: topk <= G and experts <= G * V.
template <typename Go>
void by_shape(int32_t experts, int32_t topk, const Go& go) {
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

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  by_shape(a.experts, a.topk, [&](auto g_, auto v_) {
    constexpr int G = decltype(g_)::value, V = decltype(v_)::value, per = 256 / G;
    const dim3 grid((unsigned)((a.tokens + per - 1) / per));
    if (a.f32)
      hipLaunchKernelGGL((route_kernel<G, V, true>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((route_kernel<G, V, false>), grid, dim3(256), 0, stream, a);
  });
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t stream) {
  by_shape(a.experts, a.topk, [&](auto g_, auto v_) {
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
