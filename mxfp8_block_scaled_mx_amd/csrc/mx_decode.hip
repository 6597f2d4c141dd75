// Products of a few bf16 rows with block-scaled weights, for decoding steps:
//   - gemv_kernel: y = x . W^T on MXFP4 or NVFP4 weights ("TransformerEngine-
//     accelerated Llama 3 training with native PyTorch training loop",
//     Quantized Training, names both formats; serving reads the weights for
//     one token or a few);
//   - decode_up_kernel / decode_down_kernel: the whole MoE MLP of a few tokens
//     (GroupedLinear -> ScaledSwiGLU -> GroupedLinear with routing weights,
//     "Efficient MoE training for biological foundation models", Key technical
//     approaches item 3) from the router's choices to the summed output, on
//     bf16, MXFP8 or MXFP4 weights.
//
// The activations stay bf16 (weight-only quantization): every weight is
// expanded exactly to bf16 in registers (an E2M1 or E4M3 element times a power
// of two, or E2M1 times E4M3, has at most 6 significant bits), and products
// are summed in fp32 by the 16 x 16 x 32 bf16 MFMA.
#include <algorithm>

#include "mx_device.h"
#include "mx_internal.h"

namespace mx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

namespace {

// A lane's 32 consecutive weights of one row, as loaded: 16-byte words of
// codes and the scale code(s).
template <int FMT>
struct RawBlock {
  static constexpr int kWords = FMT == WF_BF16 ? 4 : FMT == WF_MXFP8 ? 2 : 1;
  u32x4 q[kWords];
  uint32_t s;

  __device__ __forceinline__ void load(const uint8_t* row, const uint8_t* srow, int b) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) q[i] = *reinterpret_cast<const u32x4*>(row + ((size_t)b * kWords + i) * 16);
    if constexpr (FMT == WF_MXFP8 || FMT == WF_MXFP4) s = srow[b];
    if constexpr (FMT == WF_NVFP4) s = *reinterpret_cast<const uint16_t*>(srow + 2 * (size_t)b);
  }
  __device__ __forceinline__ void zero_unless(bool ok) {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) q[i][c] = ok ? q[i][c] : 0u;
  }
  // weights 8 j .. 8 j + 7 in bf16
  __device__ __forceinline__ bf16x8 frag(int j) const {
    u32x4 o;
    if constexpr (FMT == WF_BF16) {
      o = q[j];
    } else if constexpr (FMT == WF_MXFP8) {
      const float sc = __uint_as_float(s << 23);          // read as an E8M0 code: 0 means 2^-127
      const uint32_t lo = q[j >> 1][2 * (j & 1)], hi = q[j >> 1][2 * (j & 1) + 1];
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, false));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, true));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, false));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, true));
    } else if constexpr (FMT == WF_MXFP4) {
      const float sc = __uint_as_float(s << 23);
      const uint32_t w = q[0][j];
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3));
    } else {
      // E4M3 scale of the 16-value block: the product is exact in fp32 and in bf16
      const float sc = __builtin_amdgcn_cvt_f32_fp8((int)(s >> (8 * (j >> 1))), 0);
      const uint32_t w = q[0][j];
      auto pair = [&](f32x2 v) __attribute__((always_inline)) {
        bf16x2 p;
        p.x = (__bf16)(v.x * sc);
        p.y = (__bf16)(v.y * sc);
        return __builtin_bit_cast(uint32_t, p);
      };
      o.x = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0));
      o.y = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1));
      o.z = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2));
      o.w = pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3));
    }
    return __builtin_bit_cast(bf16x8, o);
  }
};

// One wave's part of the products of NT tiles of 16 weight rows with MT tiles
// of 16 activation rows: k-steps [s0, s1) of 128 values, 4 blocks of 32. Lane
// l holds weight row l % 16 and activation row l % 16 of each tile and the
// block 4 s + l / 16 of both: MFMA j of a step contracts values 8 j .. 8 j + 7
// of the four lane groups' blocks, the same permutation of k on both sides.
// Result: acc[n][m] register r of lane l = activation row (l / 16) * 4 + r,
// weight row l % 16.
//
// U steps are loaded before they are used. Blocks past nb or steps past s1
// load the row's last block and count as zero.
template <int FMT, int NT, int MT, int U>
__device__ __forceinline__ void walk(const uint8_t* const (&wrow)[NT], const uint8_t* const (&srow)[NT],
                                     const uint8_t* const (&xrow)[MT], int nb, int s0, int s1,
                                     v4f (&acc)[NT][MT]) {
  const int g = (threadIdx.x & 63) >> 4;
  for (int s = s0; s < s1; s += U) {
    RawBlock<FMT> w[U][NT];
    u32x4 x[U][MT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = min(4 * min(s + u, s1 - 1) + g, nb - 1);
#pragma unroll
      for (int n = 0; n < NT; ++n) w[u][n].load(wrow[n], srow[n], b);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[u][m][j] = *reinterpret_cast<const u32x4*>(xrow[m] + ((size_t)b * 4 + j) * 16);
    }
    if (s + U > s1 || 4 * (s + U) > nb) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = s + u < s1 && 4 * (s + u) + g < nb;
#pragma unroll
        for (int n = 0; n < NT; ++n) w[u][n].zero_unless(ok);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[u][m][j][c] = ok ? x[u][m][j][c] : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 wf = w[u][n].frag(j);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[u][m][j]), wf, acc[n][m], 0, 0, 0);
        }
  }
}

template <int NT, int MT>
__device__ __forceinline__ void clear(v4f (&acc)[NT][MT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.f, 0.f, 0.f, 0.f};
}

// y[m, n] = x[m, k] . W[n, k]^T. A workgroup owns 16 * NT weight rows and
// 16 * MT activation rows; its waves split k and add up through LDS in wave
// order (one order whatever the timing).
template <int FMT, int NT, int MT, int U>
__global__ __launch_bounds__(1024) void gemv_kernel(const uint8_t* x, int64_t ldx_bytes, const uint8_t* w,
                                                    const uint8_t* ws, const float* amax, int32_t m, int32_t n,
                                                    int32_t nb, void* y, int32_t y_f32) {
  extern __shared__ float red[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
  const uint8_t *wrow[NT], *srow[NT], *xrow[MT];
  constexpr int kBlockBytes = RawBlock<FMT>::kWords * 16;
  constexpr int kScaleBytes = FMT == WF_NVFP4 ? 2 : 1;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t r = min(n0 + 16 * t + (lane & 15), n - 1);        // rows past the end repeat the last, unused
    wrow[t] = w + r * nb * kBlockBytes;
    srow[t] = ws + r * nb * kScaleBytes;
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) xrow[t] = x + (int64_t)min(m0 + 16 * t + (lane & 15), m - 1) * ldx_bytes;
  const int ns = (nb + 3) / 4;
  v4f acc[NT][MT];
  clear(acc);
  walk<FMT, NT, MT, U>(wrow, srow, xrow, nb, (int)((int64_t)ns * wave / waves), (int)((int64_t)ns * (wave + 1) / waves), acc);
  constexpr int kOut = NT * MT * 256;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[wave * kOut + ((t * MT + u) * 4 + r) * 64 + lane] = acc[t][u][r];
  __syncthreads();
  float inv = 1.0f;
  if constexpr (FMT == WF_NVFP4) inv = (float)(1.0 / (double)nvfp4_tensor_scale(*amax));
  for (int o = tid; o < kOut; o += blockDim.x) {
    float v = 0.f;
    for (int i = 0; i < waves; ++i) v += red[i * kOut + o];
    if constexpr (FMT == WF_NVFP4) v *= inv;
    const int l = o & 63, r = (o >> 6) & 3, u = (o >> 8) % MT, t = (o >> 8) / MT;
    const int row = m0 + 16 * u + (l >> 4) * 4 + r, col = n0 + 16 * t + (l & 15);
    if (row < m && col < n) {
      const int64_t at = (int64_t)row * n + col;
      if (y_f32)
        reinterpret_cast<float*>(y)[at] = v;
      else
        reinterpret_cast<__bf16*>(y)[at] = (__bf16)v;
    }
  }
}

}  // namespace

template <int FMT, int NT, int MT, int U>
static void gemv_go(const GemvArgs& a, int waves, hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 16 * NT - 1) / (16 * NT)), (unsigned)((a.m + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((gemv_kernel<FMT, NT, MT, U>), grid, dim3(64 * waves), (size_t)waves * NT * MT * 1024, stream,
                     reinterpret_cast<const uint8_t*>(a.x), a.ldx * 2, a.w, a.ws, a.amax, (int32_t)a.m, (int32_t)a.n,
                     (int32_t)(a.k / 32), a.y, a.y_f32);
}

template <int FMT>
static void gemv_format(const GemvArgs& a, hipStream_t stream) {
  const int64_t ns = (a.k / 32 + 3) / 4;
  const int waves = (int)std::min<int64_t>(16, std::max<int64_t>(1, ns));
  if (a.m <= 16)
    gemv_go<FMT, 1, 1, 2>(a, waves, stream);
  else
    gemv_go<FMT, 1, 4, 1>(a, waves, stream);
}

hipError_t launch_gemv(int fmt, const GemvArgs& a, hipStream_t stream) {
  if (fmt == WF_MXFP4)
    gemv_format<WF_MXFP4>(a, stream);
  else
    gemv_format<WF_NVFP4>(a, stream);
  return hipGetLastError();
}

namespace {

// The entries (token, slot) of the router's choices, counted per expert. An
// entry whose expert lies outside [0, E) is dropped; of a token's entries that
// name the same expert, the first stands for all, with the sum of their
// weights.
__device__ __forceinline__ int32_t entry_expert(const int32_t* idx, int32_t topk, int32_t E, int i) {
  const int32_t e = idx[i];
  if (e < 0 || e >= E) return -1;
  for (int j = i - i % topk; j < i; ++j)
    if (idx[j] == e) return -1;
  return e;
}

// Exclusive sum over the wave's lanes.
__device__ __forceinline__ int lanes_below(int v, int lane) {
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d, 64);
    if (lane >= d) s += o;
  }
  return s - v;
}

// A = w silu(g) u of every entry, [g | u] = W1_e x_t. Workgroup (f-tile,
// slot): 16 values of f of the slot-th expert that any entry names, for all
// of that expert's entries; its waves split the hidden dimension. A is kept
// as a sum of two bf16 numbers (16 bits), since the second product takes bf16.
template <int FMT>
__global__ __launch_bounds__(512) void decode_up_kernel(DecodeArgs a) {
  constexpr int kMaxMT = 2;
  __shared__ int32_t cnt[kMaxGroups];
  __shared__ int16_t expert[kDecodeMaxEntries], list[kDecodeMaxEntries];
  __shared__ int32_t mine, rows;
  __shared__ float red[8 * 2 * kMaxMT * 256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int n = a.tokens * a.topk, slot = blockIdx.y;
  for (int e = tid; e < kMaxGroups; e += blockDim.x) cnt[e] = 0;
  if (tid == 0) {
    mine = -1;
    rows = 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) {
    const int32_t e = entry_expert(a.topk_idx, a.topk, a.experts, i);
    expert[i] = (int16_t)e;
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    const int c0 = cnt[2 * lane] > 0, c1 = cnt[2 * lane + 1] > 0;
    const int below = lanes_below(c0 + c1, lane);
    if (c0 && below == slot) mine = 2 * lane;
    if (c1 && below + c0 == slot) mine = 2 * lane + 1;
  }
  __syncthreads();
  const int e = mine;
  if (e < 0) return;                                      // fewer experts named than slots
  // the expert's entries (their order among themselves changes no result)
  for (int i = tid; i < n; i += blockDim.x)
    if (expert[i] == e) list[atomicAdd(&rows, 1)] = (int16_t)i;
  __syncthreads();
  const int count = rows, f0 = blockIdx.x * 16;
  const int nb = a.hidden / 32, ns = (nb + 3) / 4;
  constexpr int kBlockBytes = RawBlock<FMT>::kWords * 16;
  const uint8_t *wrow[2], *srow[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t r = (int64_t)e * 2 * a.ffn + (int64_t)t * a.ffn + f0 + (lane & 15);
    wrow[t] = a.w1 + r * nb * kBlockBytes;
    srow[t] = a.w1_s + r * nb;
  }
  const int s0 = ns * wave / waves, s1 = ns * (wave + 1) / waves;
  auto chunk = [&](auto mt_, int c0) __attribute__((always_inline)) {
    constexpr int MT = decltype(mt_)::value;
    const uint8_t* xrow[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int i = list[min(c0 + 16 * t + (lane & 15), count - 1)];
      xrow[t] = a.x + (int64_t)(i / a.topk) * a.hidden * 2;
    }
    v4f acc[2][MT];
    clear(acc);
    walk<FMT, 2, MT, 1>(wrow, srow, xrow, nb, s0, s1, acc);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[((wave * 2 + t) * MT + u) * 256 + r * 64 + lane] = acc[t][u][r];
    __syncthreads();
    for (int o = tid; o < MT * 256; o += blockDim.x) {
      float g = 0.f, up = 0.f;
      for (int i = 0; i < waves; ++i) {
        g += red[(i * 2) * MT * 256 + o];
        up += red[(i * 2 + 1) * MT * 256 + o];
      }
      const int l = o & 63, row = c0 + 16 * (o >> 8) + (l >> 4) * 4 + ((o >> 6) & 3);
      if (row < count) {
        const int i = list[row], t0 = i - i % a.topk;
        float wt = 0.f;
        for (int j = i; j < t0 + a.topk; ++j)
          if (a.topk_idx[j] == e) wt += a.topk_w != nullptr ? a.topk_w[j] : 1.0f;
        const float v = wt * (g / (1.0f + expf(-g))) * up;
        const __bf16 hi = (__bf16)v;
        // an infinite or NaN value has no second part
        const __bf16 lo = (abs_bits((float)hi) < 0x7F800000u) ? (__bf16)(v - (float)hi) : (__bf16)0.0f;
        const int64_t at = (int64_t)i * a.ffn + f0 + (l & 15);
        a.act_hi[at] = __builtin_bit_cast(uint16_t, hi);
        a.act_lo[at] = __builtin_bit_cast(uint16_t, lo);
      }
    }
    __syncthreads();
  };
  for (int c0 = 0; c0 < count; c0 += 32) {
    if (count - c0 <= 16)
      chunk(std::integral_constant<int, 1>{}, c0);
    else
      chunk(std::integral_constant<int, 2>{}, c0);
  }
}

// y[t] = sum over the token's entries of W2_e . A. Workgroup (h-tile, token
// chunk): 16 values of h for up to kDecodeTokenChunk tokens; the k-steps of
// all named experts, one after the other, are split evenly over its 16 waves.
// A tile's activation rows are 8 entries' high parts and the same 8 entries'
// low parts, whose results are added. Each wave adds its results to a slice
// of its own in LDS (a token appears once among an expert's entries), and the
// slices are added in wave order, so the sum has one order whatever the
// timing.
template <int FMT>
__global__ __launch_bounds__(1024) void decode_down_kernel(DecodeArgs a) {
  extern __shared__ float ys[];                           // [waves][tokens of the chunk][16]
  __shared__ int32_t cnt[kMaxGroups], first[kMaxGroups + 1], slot_e[kMaxGroups];
  __shared__ int16_t list[kDecodeMaxEntries];
  __shared__ int32_t slots;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int t0 = blockIdx.y * kDecodeTokenChunk, nt = min(a.tokens - t0, kDecodeTokenChunk);
  const int n = nt * a.topk;
  const int32_t* idx = a.topk_idx + (int64_t)t0 * a.topk;
  for (int e = tid; e < kMaxGroups; e += blockDim.x) cnt[e] = 0;
  for (int o = tid; o < waves * nt * 16; o += blockDim.x) ys[o] = 0.f;
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) {
    const int32_t e = entry_expert(idx, a.topk, a.experts, i);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    const int n0 = cnt[2 * lane], n1 = cnt[2 * lane + 1];
    const int rows_below = lanes_below(n0 + n1, lane);
    const int slots_below = lanes_below((n0 > 0) + (n1 > 0), lane);
    first[2 * lane] = rows_below;
    first[2 * lane + 1] = rows_below + n0;
    if (n0 > 0) slot_e[slots_below] = 2 * lane;
    if (n1 > 0) slot_e[slots_below + (n0 > 0)] = 2 * lane + 1;
    if (lane == 63) {
      first[kMaxGroups] = rows_below + n0 + n1;
      slots = slots_below + (n0 > 0) + (n1 > 0);
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) {
    const int32_t e = entry_expert(idx, a.topk, a.experts, i);
    if (e >= 0) list[first[e] + atomicAdd(&cnt[e], -1) - 1] = (int16_t)i;
  }
  __syncthreads();
  const int nb = a.ffn / 32, ns = (nb + 3) / 4;
  const int h0 = blockIdx.x * 16;
  constexpr int kBlockBytes = RawBlock<FMT>::kWords * 16;
  const int64_t units = (int64_t)slots * ns;
  int64_t u = units * wave / waves;
  const int64_t u_end = units * (wave + 1) / waves;
  float* mine = ys + wave * nt * 16;
  while (u < u_end) {
    const int slot = (int)(u / ns), s0 = (int)(u % ns);
    const int s1 = (int)min((int64_t)ns, s0 + (u_end - u));
    const int e = slot_e[slot];
    const int row0 = first[e], rows = first[e + 1] - row0;
    u += s1 - s0;
    const int64_t r = (int64_t)e * a.hidden + h0 + (lane & 15);
    const uint8_t* const wrow[1] = {a.w2 + r * nb * kBlockBytes};
    const uint8_t* const srow[1] = {a.w2_s + r * nb};
    auto chunk = [&](auto mt_, int c0) __attribute__((always_inline)) {
      constexpr int MT = decltype(mt_)::value;
      const uint8_t* xrow[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int i = list[row0 + min(c0 + 8 * t + (lane & 7), rows - 1)];
        xrow[t] = reinterpret_cast<const uint8_t*>((lane & 8) ? a.act_lo : a.act_hi) +
                  ((int64_t)t0 * a.topk + i) * a.ffn * 2;
      }
      v4f acc[1][MT];
      clear(acc);
      walk<FMT, 1, MT, (MT == 1 ? 4 : MT == 2 ? 2 : 1)>(wrow, srow, xrow, nb, s0, s1, acc);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = sum_halves(acc[0][t][q]);
          const int row = c0 + 8 * t + (lane >> 4) * 4 + q;
          if (lane < 32 && row < rows) {
            const int tok = list[row0 + row] / a.topk;
            mine[tok * 16 + (lane & 15)] += v;
          }
        }
    };
    for (int c0 = 0; c0 < rows; c0 += 32) {
      if (rows - c0 <= 8)
        chunk(std::integral_constant<int, 1>{}, c0);
      else if (rows - c0 <= 16)
        chunk(std::integral_constant<int, 2>{}, c0);
      else
        chunk(std::integral_constant<int, 4>{}, c0);
    }
  }
  __syncthreads();
  for (int o = tid; o < nt * 16; o += blockDim.x) {
    float v = 0.f;
    for (int i = 0; i < waves; ++i) v += ys[i * nt * 16 + o];
    reinterpret_cast<__bf16*>(a.y)[(int64_t)(t0 + (o >> 4)) * a.hidden + h0 + (o & 15)] = (__bf16)v;
  }
}

}  // namespace

template <int FMT>
static hipError_t decode_go(const DecodeArgs& a, hipStream_t stream) {
  const int up_waves = std::min(8, std::max(1, (a.hidden / 32 + 3) / 4));
  const int slots = std::min(a.tokens * a.topk, a.experts);
  hipLaunchKernelGGL((decode_up_kernel<FMT>), dim3(a.ffn / 16, slots), dim3(64 * up_waves), 0, stream, a);
  const int nt = std::min(a.tokens, kDecodeTokenChunk), down_waves = 16;
  hipLaunchKernelGGL((decode_down_kernel<FMT>), dim3(a.hidden / 16, (a.tokens + kDecodeTokenChunk - 1) / kDecodeTokenChunk),
                     dim3(64 * down_waves), (size_t)down_waves * nt * 64, stream, a);
  return hipGetLastError();
}

hipError_t launch_decode(int fmt, const DecodeArgs& a, hipStream_t stream) {
  if (fmt == WF_BF16) return decode_go<WF_BF16>(a, stream);
  if (fmt == WF_MXFP8) return decode_go<WF_MXFP8>(a, stream);
  return decode_go<WF_MXFP4>(a, stream);
}

}  // namespace mx
