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
#include <algorithm>

#include "mx_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

constexpr float kShut = -__builtin_inff();

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  // (with the bound control the move folds into the operation that takes it)
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
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

// The other way round: V values to element `at` of such a row.
template <int V, bool F32>
__device__ __forceinline__ void store_values(void* p, int64_t at, int left, bool vec, const float (&v)[V]) {
  if (V == 4 && vec) {
    if constexpr (F32) {
      v4f o;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i & 3] = v[i];
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(p) + at) = o;
    } else {
      typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
      bf16x4 o;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i & 3] = (__bf16)v[i];
      *reinterpret_cast<bf16x4*>(reinterpret_cast<__bf16*>(p) + at) = o;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < left) {
      if (F32)
        reinterpret_cast<float*>(p)[at + i] = v[i];
      else
        reinterpret_cast<__bf16*>(p)[at + i] = (__bf16)v[i];
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
  store_values<V, F32>(a.dlogits, t * a.experts + e0, a.experts - e0, a.vec, dz);
}

// ---- the balance loss
//
// For the tokens of one sequence (n of them, k choices each):
//     c_e = choices that name expert e,   P_e = 1/n sum_t p_te,
//     loss = E / (k n) sum_e c_e P_e
// with p the softmax over the open experts, made again from the logits here (a
// row sits in registers, so this costs two reductions and no memory). Its
// gradient, and that of the means P themselves, is
//     dz_te = p_te / n (A_e - sum_j p_tj A_j),   A_e = dloss E c_e / (k n) + dP_e.

// Part i of n items (below 2^27) in whole multiples of `step`: [first, last). In
// 32 bits, since a division of 64 takes as long as a row of a token.
__device__ __forceinline__ void part_of(uint32_t n, uint32_t parts, uint32_t i, uint32_t step, int64_t* first, int64_t* last) {
  const uint32_t size = (n + parts * step - 1) / (parts * step) * step;
  *first = min(i * size, n);
  *last = min((i + 1) * size, n);
}

// The tokens [begin, end) of sequence s; offsets outside 0 .. tokens, or that
// fall, are cut so that no token outside the arrays is named.
struct Span {
  int64_t begin, end;
};
__device__ __forceinline__ Span span_of(const int32_t* segments, int s, int64_t tokens) {
  if (segments == nullptr) return Span{0, tokens};
  const int64_t b = min(max((int64_t)segments[s], (int64_t)0), tokens);
  return Span{b, min(max((int64_t)segments[s + 1], b), tokens)};
}

// A lane's V values of a row as loaded. The loads are unconditional, from clamped
// addresses, so that those of several rows are in flight together: one under a
// condition is waited for where its branch joins again.
template <int V, bool F32, bool VEC>
__device__ __forceinline__ void load_raw(const void* p, int64_t row, int e0, int E, uint32_t (&w)[V]) {
  if constexpr (V == 4 && VEC) {
    const int64_t at = row + min(e0, E - 4);
    if constexpr (F32) {
      const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + at);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[V - 1] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + at);
      w[0] = v.x; w[1] = v.y;                 // two to a word: unpacked by value_of
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t at = row + min(e0 + i, E - 1);
      w[i] = F32 ? reinterpret_cast<const uint32_t*>(p)[at] : (uint32_t) reinterpret_cast<const uint16_t*>(p)[at] << 16;
    }
  }
}
template <int V, bool F32, bool VEC>
__device__ __forceinline__ float value_of(const uint32_t (&w)[V], int i) {
  if constexpr (V == 4 && VEC && !F32) return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  else return __uint_as_float(w[i]);
}
// Its logits, shut ones -inf, with the lane's biases (0 without).
template <int V, bool F32, bool VEC>
__device__ __forceinline__ void open_logits(const uint32_t (&w)[V], const float (&bias)[V], int e0, int E, float (&z)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float x = value_of<V, F32, VEC>(w, v);
    z[v] = e0 + v < E && x + bias[v] > kShut ? x : kShut;
  }
}

// e^x for x <= 0 (0 for NaN), good to three half steps of fp32 (measured 2.3), and 0
// where it falls below 2^-126 (x < -87.3). A product with a constant in two parts
// and a correction of first order: 2^t with t = x log2(e) rounded, by the hardware
// (two half steps), times 1 + r ln 2 with r what the rounding left out (one more;
// 2^t alone would be off by |x| half steps more).
__device__ __forceinline__ float exp_below(float x) {
  x = fmaxf(x, -200.f);                                   // (the products below stay finite)
  constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945f;
  constexpr float kLog2eLow = (float)(1.4426950408889634074 - (double)kLog2e);
  const float t = x * kLog2e, r = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -t)), e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * kLn2, e);
}

// The row's softmax over the open experts before it is divided by its sum: e^(z -
// max), 0 for shut experts (-inf less the maximum, or less -inf, which is NaN).
template <int G, int V>
__device__ __forceinline__ float row_exps(const float (&z)[V], float (&e)[V]) {
  float zm = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) zm = fmaxf(zm, z[v]);
  zm = group_max<G>(zm);
#pragma unroll
  for (int v = 0; v < V; ++v) e[v] = exp_below(z[v] - zm);
  return zm;
}
// 1 over the sum, which is at least 1 where an expert is open. Where none is: 0.
// Where one is +inf: NaN (its inf - inf counts as 0 in exp_below, and so do the
// others, so the sum is 0).
__device__ __forceinline__ float over_sum(float sum, float zm) {
  return sum > 0.f ? __builtin_amdgcn_rcpf(sum) : zm > kShut ? __builtin_nanf("") : 0.f;
}
template <int G, int V>
__device__ __forceinline__ void row_softmax(const float (&z)[V], float (&p)[V]) {
  const float zm = row_exps<G, V>(z, p);
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += p[v];
  const float inv = over_sum(group_sum<G>(sum), zm);
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] *= inv;
}

// What a sequence's sums make: counts, means and (by the first wave, in 64 bits)
// the loss. prob and count are the sums in LDS.
__device__ __forceinline__ void balance_results(const BalanceArgs& a, int s, int64_t n, const double* prob, const int* count) {
  const double len = n > 0 ? (double)n : 1.0;
  double part = 0.0;
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
    const int64_t at = (int64_t)s * a.experts + e;
    a.counts[at] = count[e];
    a.mean_prob[at] = (float)(prob[e] / len);
  }
  if (threadIdx.x < 64) {
    for (int e = threadIdx.x; e < a.experts; e += 64) part += (double)count[e] * prob[e];
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) part += __shfl_xor(part, m, 64);
    if (threadIdx.x == 0) a.loss[s] = (float)(part * a.experts / ((double)a.topk * len * len));
  }
}

// Part blockIdx.x of sequence blockIdx.y: sums over its tokens, straight to the
// results where a sequence is one part, else to the workspace. The sums are kept
// in 64 bits: in 32 they would stand still past 2^24 tokens, and the few adds a
// token hide behind its loads.
// 16383 bf16 tokens of 128 experts, 8 choices, in 13 sequences of unlike lengths: 7.6
// us of which 2 are the launch, for 4.7 MB that memory passes in 1: what bounds it is
// the chain of offsets, rows, two reductions a row and the sum over the workgroup, and
// the longest sequence's parts. 33 tokens: 4.6 us. As one sequence, with the join: 256
// parts of 64 tokens 13.2 us; 128 of 128 took 1.2 more, 512 of 32 4.4 more. 65536
// tokens in 512 parts: 25.1.
template <int G, int V, bool F32, bool VEC>
__global__ __launch_bounds__(256) void balance_kernel(BalanceArgs a) {
  constexpr int N = 256 / G, U = 4;                       // tokens at a time, and rows of a lane in flight
  __shared__ double probs[N][G * V];
  __shared__ double prob[G * V];
  __shared__ int count[G * V];
  const int gl = (threadIdx.x & 63) % G, e0 = gl * V, s = blockIdx.y, tid = threadIdx.x, E = a.experts;
  const Span sp = span_of(a.segments, s, a.tokens);
  const int64_t n = sp.end - sp.begin, parts = gridDim.x;
  int64_t t0, t1;
  part_of((uint32_t)n, gridDim.x, blockIdx.x, N, &t0, &t1);
  t0 += sp.begin;
  t1 += sp.begin;
  double acc[V];
  float bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    acc[v] = 0.0;
    bias[v] = a.bias != nullptr ? a.bias[min(e0 + v, E - 1)] : 0.f;
  }
  if (tid < G * V) count[tid] = 0;
  __syncthreads();
  if (t0 < t1) {
    int64_t i = t0 * a.topk + tid;
    for (int64_t t = t0 + tid / G; t - tid / G < t1; t += U * N) {
      uint32_t w[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) load_raw<V, F32, VEC>(a.logits, min(t + u * N, t1 - 1) * E, e0, E, w[u]);
      // the choices of these rows, while they travel (integers: any order gives the same sum)
      for (const int64_t end = min(t - tid / G + U * N, t1) * a.topk; i < end; i += 256) {
        const int e = a.topk_idx[i];
        if (e >= 0 && e < E) atomicAdd(&count[e], 1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t - tid / G + u * N >= t1) break;             // (uniform)
        float z[V], p[V];
        open_logits<V, F32, VEC>(w[u], bias, e0, E, z);
        row_softmax<G, V>(z, p);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += t + u * N < t1 ? (double)p[v] : 0.0;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) probs[tid / G][e0 + v] = acc[v];
  __syncthreads();
  if (tid < G * V) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += probs[i][tid];
    prob[tid] = sum;
  }
  __syncthreads();
  if (parts == 1) {
    balance_results(a, s, n, prob, count);
  } else if (tid < a.experts) {
    const int64_t at = ((int64_t)s * parts + blockIdx.x) * a.experts + tid;
    a.part_prob[at] = prob[tid];
    a.part_count[at] = count[tid];
  }
}

// The parts of sequence blockIdx.x added up in order, 8 strands of them at once: 3.5
// us for 13 sequences of 40 parts, 6 for one of 256 (393 KB through one compute unit).
__global__ __launch_bounds__(1024) void balance_join_kernel(BalanceArgs a) {
  __shared__ double probs[8][128];
  __shared__ int counts[8][128];
  __shared__ double prob[128];
  __shared__ int count[128];
  const int e = threadIdx.x & 127, strand = threadIdx.x >> 7, s = blockIdx.x;
  double ps = 0.0;
  int cs = 0;
  if (e < a.experts) {
    const int64_t base = (int64_t)s * a.parts * a.experts + e;
#pragma unroll 8
    for (int i = strand; i < a.parts; i += 8) {
      ps += a.part_prob[base + (int64_t)i * a.experts];
      cs += a.part_count[base + (int64_t)i * a.experts];
    }
  }
  probs[strand][e] = ps;
  counts[strand][e] = cs;
  __syncthreads();
  if (threadIdx.x < 128) {
    double sum = 0.0;
    int c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum += probs[i][e];
      c += counts[i][e];
    }
    prob[e] = sum;
    count[e] = c;
  }
  __syncthreads();
  const Span sp = span_of(a.segments, s, a.tokens);
  balance_results(a, s, sp.end - sp.begin, prob, count);
}

// Part blockIdx.x of sequence blockIdx.y; the last blockIdx.y of a call with
// offsets takes the tokens before the first sequence and behind the last, whose
// gradient is `add` alone.
// A is made once a workgroup, in 64 bits, less the point between its least and its
// largest value that is nearest to 0: since the p of a row sum to 1 the gradient
// does not see the shift, equal A become 0, and no A gets larger than it was. (A
// less its mean does where few experts outweigh the rest: with the gradient of sum
// log P and one expert of P = 4e-14 the others' gradients were off by 400 times
// their size.) sum p A is made twice, the second time from A less the first: what
// is left of its error is relative to the differences, not to A.
// 16383 bf16 tokens of 128 experts with another gradient to add: 10.2 us in 13
// sequences of unlike lengths, 7.5 as one, for 12.6 MB that memory passes in 2.1;
// 65536 tokens 17.1 (50 MB: 8.5), 15.3 without one to add. Bound by latency, as the
// forward; at 65536 also by 9 us of instructions (about 180 a row of two tokens, four
// cycles each), of which the second sum p A is 1.
template <int G, int V, bool F32, bool VEC>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceBwdArgs a) {
  constexpr int N = 256 / G, U = 4;
  const int gl = (threadIdx.x & 63) % G, e0 = gl * V, s = blockIdx.y, E = a.experts, mine = threadIdx.x / G;
  const bool gap = s >= a.sequences;
  Span sp;
  int64_t n, skip = 0, skip_at = a.tokens;                // the gap: token u, or from skip_at on u + skip
  if (gap) {
    const int64_t first = min(max((int64_t)a.segments[0], (int64_t)0), a.tokens);
    const int64_t last = min(max((int64_t)a.segments[a.sequences], first), a.tokens);
    sp = Span{0, first + a.tokens - last};
    skip_at = first;
    skip = last - first;
  } else {
    sp = span_of(a.segments, s, a.tokens);
  }
  n = sp.end - sp.begin;
  int64_t u0, u1;
  part_of((uint32_t)n, gridDim.x, blockIdx.x, N, &u0, &u1);
  u0 += sp.begin;
  u1 += sp.begin;
  if (u0 >= u1) return;
  const void* const add = a.add != nullptr ? a.add : a.logits;           // (read and not used without)
  uint32_t w[U][V], d[U][V];
  auto fetch = [&](int64_t u) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t uc = min(u + mine + i * N, u1 - 1), row = (uc < skip_at ? uc : uc + skip) * E;
      load_raw<V, F32, VEC>(a.logits, row, e0, E, w[i]);
      load_raw<V, F32, VEC>(add, row, e0, E, d[i]);
    }
  };
  fetch(u0);
  float A[V], bias[V];
  double c[V];
  float least = __builtin_inff(), most = -__builtin_inff();
  const int sc = gap ? 0 : s;
  const double per = 1.0 / ((double)a.topk * (double)n), per_token = per * a.topk;
  const double f = a.dloss != nullptr ? (double)a.dloss[sc] * E * per : 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t at = (int64_t)sc * E + min(e0 + v, E - 1);
    bias[v] = a.bias != nullptr ? a.bias[min(e0 + v, E - 1)] : 0.f;
    c[v] = a.dloss != nullptr ? f * (double)a.counts[at] : 0.0;
    if (a.dmean_prob != nullptr) c[v] += (double)a.dmean_prob[at];
    if (e0 + v < E) {
      least = fminf(least, (float)c[v]);
      most = fmaxf(most, (float)c[v]);
    }
  }
  const double shift = (double)fmaxf(-group_max<G>(-least), fminf(group_max<G>(most), 0.f));
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = e0 + v < E ? (float)((c[v] - shift) * per_token) : 0.f;
  for (int64_t u = u0; u < u1; u += U * N) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t uc = u + mine + i * N, t = uc < skip_at ? uc : uc + skip;
      if (u + i * N >= u1) break;                         // (uniform)
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = a.add != nullptr ? value_of<V, F32, VEC>(d[i], v) : 0.f;
      if (!gap) {
        float z[V], p[V], b[V];
        open_logits<V, F32, VEC>(w[i], bias, e0, E, z);
        const float zm = row_exps<G, V>(z, p);
        float sum = 0.f, dot = 0.f, rest = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          sum += p[v];
          dot = fmaf(p[v], A[v], dot);
        }
        const float inv = over_sum(group_sum<G>(sum), zm);
        dot = group_sum<G>(dot) * inv;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          b[v] = A[v] - dot;
          rest = fmaf(p[v], b[v], rest);
        }
        rest = group_sum<G>(rest) * inv;
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] += p[v] * inv * (b[v] - rest);
      }
      if (uc < u1 && e0 < E) store_values<V, F32>(a.dlogits, t * E + e0, E - e0, VEC, out);
    }
    if (u + U * N < u1) fetch(u + U * N);
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

template <typename Go>
void by_type(int32_t f32, bool vec, const Go& go) {
  if (f32) vec ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  else vec ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
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

// Parts of a sequence: enough for two workgroups a compute unit where sequences
// are equally long, at least 64 tokens each if one holds them all, and no more
// than 16384 (the sequences' lengths are not known here, and one may hold nearly
// all tokens) as long as that takes at most 4096 workgroups.
int balance_parts(int64_t tokens, int32_t sequences) {
  const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int64_t parts = std::max(cdiv(512, sequences), std::min(cdiv(tokens, 16384), cdiv(4096, sequences)));
  return (int)std::max<int64_t>(1, std::min(cdiv(tokens, 64), parts));
}

hipError_t launch_balance(const BalanceArgs& args, hipStream_t stream) {
  BalanceArgs a = args;
  a.vec = by_fours(a.experts, a.f32, a.logits);
  by_shape(a.experts, [&](auto g_, auto v_) {
    constexpr int G = decltype(g_)::value, V = decltype(v_)::value;
    const dim3 grid((unsigned)a.parts, (unsigned)a.sequences);
    const auto go = [&](auto f32_, auto vec_) {
      constexpr bool F32 = decltype(f32_)::value, VEC = decltype(vec_)::value;
      hipLaunchKernelGGL((balance_kernel<G, V, F32, VEC>), grid, dim3(256), 0, stream, a);
    };
    by_type(a.f32, V == 4 && a.vec, go);
  });
  if (a.parts > 1)
    hipLaunchKernelGGL(balance_join_kernel, dim3((unsigned)a.sequences), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceBwdArgs& args, hipStream_t stream) {
  BalanceBwdArgs a = args;
  a.vec = by_fours(a.experts, a.f32, a.logits) && by_fours(a.experts, a.f32, a.dlogits) &&
          by_fours(a.experts, a.f32, a.add);
  const int rows = a.sequences + (a.segments != nullptr ? 1 : 0);
  by_shape(a.experts, [&](auto g_, auto v_) {
    constexpr int G = decltype(g_)::value, V = decltype(v_)::value, per = 256 / G;
    // four workgroups a compute unit: 16383 tokens of 128 experts in 13 sequences of
    // unlike lengths 10.2 us, three 0.6 more; of like lengths three take 1.2 less
    const int64_t parts = std::max<int64_t>(1, std::min((a.tokens + per - 1) / per, (int64_t)((1024 + rows - 1) / rows)));
    const dim3 grid((unsigned)parts, (unsigned)rows);
    const auto go = [&](auto f32_, auto vec_) {
      constexpr bool F32 = decltype(f32_)::value, VEC = decltype(vec_)::value;
      hipLaunchKernelGGL((balance_bwd_kernel<G, V, F32, VEC>), grid, dim3(256), 0, stream, a);
    };
    by_type(a.f32, V == 4 && a.vec, go);
  });
  return hipGetLastError();
}

}  // namespace mx
