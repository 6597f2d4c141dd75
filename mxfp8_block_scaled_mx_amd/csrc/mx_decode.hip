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
#include <stddef.h>

#include <algorithm>

#include "mx_device.h"
#include "mx_internal.h"

namespace mx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

namespace {

template <int FMT>
constexpr int kWords = FMT == WF_BF16 ? 4 : FMT == WF_MXFP8 ? 2 : 1;        // 16-byte words of a 32-weight block
template <int FMT>
constexpr int kScaleBytes = FMT == WF_BF16 ? 0 : FMT == WF_NVFP4 ? 2 : 1;   // scale bytes of a 32-weight block

// Weights 8 j .. 8 j + 7 of a 32-weight block in bf16, from its 16-byte words
// and scale code(s).
template <int FMT>
__device__ __forceinline__ bf16x8 expand(const u32x4 (&q)[kWords<FMT>], uint32_t s, int j) {
  u32x4 o;
  if constexpr (FMT == WF_BF16) {
    o = q[j];
  } else if constexpr (FMT == WF_MXFP8) {
    const float sc = __uint_as_float(s << 23);            // read as an E8M0 code: 0 means 2^-127
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

// Orders a wave's own LDS writes before its later reads by other lanes. One
// wave's LDS operations execute in order, so only the compiler is held.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Values of k in one step of the walk below: 128-byte pieces of a 4-bit or
// 8-bit row (whole cache lines, which nontemporal loads want), 256-byte pieces
// of a bf16 row.
template <int FMT>
constexpr int kHalves = FMT == WF_MXFP4 || FMT == WF_NVFP4 ? 2 : 1;         // of 128 values
template <int FMT>
constexpr int kStepBlocks = 4 * kHalves<FMT>;
// Waves split k at multiples of so many steps, whose scales are 16 bytes of a row.
template <int FMT>
constexpr int kUnit = FMT == WF_BF16 ? 1 : 16 / (kStepBlocks<FMT> * kScaleBytes<FMT>);
template <int FMT>
__host__ __device__ constexpr int k_units(int nb) {
  return (nb + kStepBlocks<FMT> * kUnit<FMT> - 1) / (kStepBlocks<FMT> * kUnit<FMT>);
}
// First step of part i of n, where the row has nb blocks.
template <int FMT>
__device__ __forceinline__ int part_start(int nb, int i, int n) {
  const int steps = (nb + kStepBlocks<FMT> - 1) / kStepBlocks<FMT>;
  return min(steps, (int)((int64_t)k_units<FMT>(nb) * i / n) * kUnit<FMT>);
}

// One wave's part of the products of NT tiles of 16 weight rows with MT tiles
// of R activation rows (R = 16; or 4 with MT = 1, repeated over the MFMA's 16)
// over the k-steps [s0, s1). Result: acc[n][m] register r of lane l =
// activation row (l / 16) * 4 + r, weight row l % 16.
//
// The MFMA's lane layout (lane l holds row l % 16) makes neighbouring lanes
// read different rows, which costs the load path one cache line per lane. So
// both operands are loaded as whole row pieces (consecutive lanes, consecutive
// 16-byte chunks), kept in registers D steps (weights) and DX half steps
// (activations) ahead, and pass through a private LDS tile of the wave, whose
// chunks are swizzled so that neither side conflicts on banks. Scales come 1 KiB
// (G steps) at a time. No barrier: the tile is the wave's own. MFMA j of 128
// values contracts values 8 j .. 8 j + 7 of the four lane groups' blocks, the
// same permutation of k on both sides.
//
// WHOLE: k is a multiple of the step, and scale rows of 16 bytes. Otherwise
// blocks past the end repeat the last one and count as zero.
template <int FMT, int NT, int R, int MT, bool WHOLE, int D, int DX>
struct Walk {
  static constexpr int H = kHalves<FMT>, S = kScaleBytes<FMT>, BW = kWords<FMT>;
  static constexpr int W = BW * H;                                          // 16-byte loads of a tile and step
  static constexpr int SB = 4 * H * S;                                      // scale bytes of a row and step
  static constexpr int LR = 4 / NT;                                         // lanes of a scale row
  static constexpr int G = SB > 0 ? 16 * LR / SB : D;                       // steps of a scale load
  static constexpr int kWTile = 1024 * W, kXTile = 256 * R, kScales = S > 0 ? 1024 : 0;
  static constexpr int kLds = NT * kWTile + kScales + MT * kXTile;          // bytes of one wave
  static constexpr int XL = R / 4;                                          // loads of an activation tile
  static_assert(MT == 1 || R == 16);
  static_assert((D * H) % DX == 0 && G % D == 0 && (S == 0 || kUnit<FMT> * SB == 16));

  const uint8_t* w[NT];             // first row of each tile (wave-uniform)
  uint32_t woff[W];                 // the lane's row within a tile, in bytes
  const uint8_t* ws;                // the lane's scale row
  const uint8_t* x;                 // activations (uniform)
  uint32_t xoff[MT][XL];            // the lane's rows, in bytes
  int nb;                           // blocks of a row

  // tile t: consecutive rows from row first[t]; the last row is repeated where
  // fewer than 16 are left
  __device__ __forceinline__ void weight_tiles(const uint8_t* base, const uint8_t* sbase, const int64_t (&first)[NT],
                                               int left) {
    const int lane = threadIdx.x & 63;
    if constexpr (S > 0) {
      const int row = lane / LR, t = row >> 4;
      int64_t r = first[0];
#pragma unroll
      for (int n = 1; n < NT; ++n) r = t == n ? first[n] : r;
      ws = sbase + (r + min(row & 15, left - 1)) * nb * S;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) w[n] = base + first[n] * nb * (16 * BW);
#pragma unroll
    for (int i = 0; i < W; ++i)
      woff[i] = (uint32_t)min((i * 64 + lane) / (4 * W), left - 1) * (uint32_t)(nb * 16 * BW);
  }

  __device__ __forceinline__ void run(uint8_t* lds, int s0, int s1, v4f (&acc)[NT][MT]) const {
    if (s0 >= s1) return;
    const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
    u32x4 wr[D][NT][W], xr[DX][MT][XL], sr;
    uint8_t* const sl = lds + NT * kWTile;
    uint8_t* const xl = sl + kScales;
    const int last = s1 * H - 1;

    // a load past the end is issued all the same (the number of loads in
    // flight stays fixed), with every lane at one address
    auto load_w = [&](int t, u32x4 (&to)[NT][W]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int c = lane % (4 * W);
        const uint32_t at = WHOLE ? (uint32_t)(t * 64 * W + c * 16)
                                  : (uint32_t)(min(kStepBlocks<FMT> * t + c / BW, nb - 1) * 16 * BW + (c % BW) * 16);
        const uint32_t off = t < s1 ? woff[i] + at : 0u;
#pragma unroll
        for (int n = 0; n < NT; ++n) to[n][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w[n] + off));
      }
    };
    auto load_x = [&](int t, u32x4 (&to)[MT][XL]) __attribute__((always_inline)) {
      const uint32_t at = WHOLE ? t * 256 + li * 16 : min(4 * t + li / 4, nb - 1) * 64 + (li % 4) * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < XL; ++i)
          to[m][i] = *reinterpret_cast<const u32x4*>(x + (t <= last ? xoff[m][i] + at : xoff[0][0]));
    };
    // 16 bytes of a scale row per lane: the G steps from s
    auto load_s = [&](int s) __attribute__((always_inline)) {
      if constexpr (S > 0) {
        const int row_bytes = nb * S;
        const int at = s * SB + lane % LR * 16;
        if constexpr (WHOLE) {
          sr = *reinterpret_cast<const u32x4*>(ws + (at < row_bytes ? at : 0));
        } else {
          // byte by byte, the row's last one repeated (its blocks count as zero)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t v = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int i = at + 4 * q + b;
              v |= (uint32_t)ws[i < row_bytes ? i : row_bytes - S + (i & (S - 1))] << (8 * b);
            }
            sr[q] = v;
          }
        }
      }
    };

    load_s(s0);
#pragma unroll
    for (int d = 0; d < D; ++d) load_w(s0 + d, wr[d]);
#pragma unroll
    for (int d = 0; d < DX; ++d) load_x(s0 * H + d, xr[d]);
    int in_group = 0;
    for (int s = s0; s < s1; s += D) {
      if constexpr (S > 0) {
        if (in_group == 0) {
          wave_lds_fence();                               // after the previous steps' reads
          *reinterpret_cast<u32x4*>(sl + lane * 16) = sr;
          if (s + G < s1) load_s(s + G);
        }
      }
#pragma unroll
      for (int uh = 0; uh < D * H; ++uh) {
        const int u = uh / H, h = uh % H, t = s + u, th = t * H + h;
        if (h == 0 && t >= s1) return;
        wave_lds_fence();
        if (h == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < W; ++i) {
              const int row = (i * 64 + lane) / (4 * W), c = lane % (4 * W);
              u32x4 v = wr[u][n][i];
              if constexpr (!WHOLE)
                if (kStepBlocks<FMT> * (t + 1) > nb) {
                  const bool ok = kStepBlocks<FMT> * t + c / BW < nb;
#pragma unroll
                  for (int q = 0; q < 4; ++q) v[q] = ok ? v[q] : 0u;
                }
              *reinterpret_cast<u32x4*>(lds + n * kWTile + (row * 4 * W + (c ^ (row & (4 * W - 1)))) * 16) = v;
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < XL; ++i) {
            const int row = i * 4 + g;
            u32x4 v = xr[uh % DX][m][i];
            if constexpr (!WHOLE)
              if (4 * th + 4 > nb) {
                const bool ok = 4 * th + li / 4 < nb;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = ok ? v[q] : 0u;
              }
            *reinterpret_cast<u32x4*>(xl + m * kXTile + (row * 16 + (li ^ row)) * 16) = v;
          }
        if (h == 0) load_w(t + D, wr[u]);
        load_x(th + DX, xr[uh % DX]);
        wave_lds_fence();
        bf16x8 xf[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = li % R;
            xf[m][j] = *reinterpret_cast<const bf16x8*>(xl + m * kXTile + (row * 16 + ((g * 4 + j) ^ row)) * 16);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          u32x4 q[BW];
          uint32_t sc = 0;
#pragma unroll
          for (int i = 0; i < BW; ++i)
            q[i] = *reinterpret_cast<const u32x4*>(
                lds + n * kWTile + (li * 4 * W + (((h * 4 + g) * BW + i) ^ (li & (4 * W - 1)))) * 16);
          const uint8_t* p = sl + (n * 16 + li) * 16 * LR + (in_group + u) * SB + (h * 4 + g) * S;
          if constexpr (S == 1) sc = *p;
          if constexpr (S == 2) sc = *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8 wf = expand<FMT>(q, sc, j);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[m][j], wf, acc[n][m], 0, 0, 0);
          }
        }
      }
      in_group = in_group + D < G ? in_group + D : 0;
    }
  }
};

template <int NT, int MT>
__device__ __forceinline__ void clear(v4f (&acc)[NT][MT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.f, 0.f, 0.f, 0.f};
}

// y[m, n] = x[m, k] . W[n, k]^T. A team of `parts` waves owns 16 * NT weight
// rows and R * MT activation rows; its waves split k and add up through LDS in
// wave order (one order whatever the timing). A workgroup is waves / parts
// teams.
template <int FMT, int NT, int R, int MT, bool WHOLE, int D, int DX>
__global__ __launch_bounds__(512, 2) void gemv_kernel(GemvArgs a, int parts) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int team = wave / parts, part = wave % parts;
  const int n0 = (blockIdx.x * (waves / parts) + team) * 16 * NT, m0 = blockIdx.y * R * MT;
  const int m = (int)a.m, n = (int)a.n;
  typedef Walk<FMT, NT, R, MT, WHOLE, D, DX> Wk;
  Wk k;
  k.nb = (int)(a.k / 32);
  int64_t first[NT];
  // a tile that passes the end moves back; a matrix of less than 16 rows repeats its last
#pragma unroll
  for (int t = 0; t < NT; ++t) first[t] = max(0, min(n0 + 16 * t, n - 16));
  k.weight_tiles(a.w, a.ws, first, min(16, n));
  k.x = reinterpret_cast<const uint8_t*>(a.x) + (int64_t)m0 * a.ldx * 2;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < Wk::XL; ++i)
      k.xoff[t][i] = (uint32_t)min(R * t + 4 * i + (lane >> 4), m - 1 - m0) * (uint32_t)(a.ldx * 2);
  v4f acc[NT][MT];
  clear(acc);
  k.run(smem + wave * Wk::kLds, part_start<FMT>(k.nb, part, parts), part_start<FMT>(k.nb, part + 1, parts), acc);
  float inv = 1.0f;
  if constexpr (FMT == WF_NVFP4) inv = (float)(1.0 / (double)nvfp4_tensor_scale(*a.amax));
  constexpr int kOut = NT * MT * 256;
  float* red = reinterpret_cast<float*>(smem);
  if (parts > 1) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave * kOut + ((t * MT + u) * 4 + r) * 64 + lane] = acc[t][u][r];
    __syncthreads();
  }
  // each wave finishes its share of the team's results
#pragma unroll
  for (int o = 0; o < NT * MT * 4; ++o) {
    if (o % parts != part) continue;
    const int r = o & 3, u = (o >> 2) % MT, t = (o >> 2) / MT;
    float v = 0.f;
    if (parts > 1)
      for (int i = 0; i < parts; ++i) v += red[(team * parts + i) * kOut + o * 64 + lane];
    else
      v = acc[t][u][r];
    const int in_tile = (lane >> 4) * 4 + r, row = m0 + R * u + in_tile;
    const int col = (int)first[t] + (lane & 15);
    if (in_tile >= R || row >= m || col >= n || col < n0 + 16 * t) continue;
    if constexpr (FMT == WF_NVFP4) v *= inv;
    const int64_t at = (int64_t)row * n + col;
    if (a.y_f32)
      reinterpret_cast<float*>(a.y)[at] = v;
    else
      reinterpret_cast<__bf16*>(a.y)[at] = (__bf16)v;
  }
}

}  // namespace

// Whether rows of k values are whole steps, with scale rows of 16 bytes.
template <int FMT>
static bool whole_steps(int64_t k, const uint8_t* scales) {
  return k % (32 * kStepBlocks<FMT>) == 0 &&
         (kScaleBytes<FMT> == 0 || (k / 32 * kScaleBytes<FMT> % 16 == 0 && reinterpret_cast<uintptr_t>(scales) % 16 == 0));
}

// Waves a launch splits k for: 16 per compute unit, all resident at once.
constexpr int64_t kWavesWanted = 4096;

template <int FMT, int NT, int R, int MT, int D, int DX>
static void gemv_go(const GemvArgs& a, hipStream_t stream) {
  const int64_t ns = k_units<FMT>((int)(a.k / 32)), mt = (a.m + R * MT - 1) / (R * MT), tiles = (a.n + 16 * NT - 1) / (16 * NT);
  int parts = 1;
  while (parts < 8 && parts * 2 <= ns && tiles * mt * parts * 2 <= kWavesWanted) parts *= 2;
  const int waves = std::max(4, parts), teams = waves / parts;
  const dim3 grid((unsigned)((tiles + teams - 1) / teams), (unsigned)mt);
  const bool whole = whole_steps<FMT>(a.k, a.ws);
  const size_t lds = (size_t)waves * std::max(Walk<FMT, NT, R, MT, true, D, DX>::kLds, NT * MT * 1024);
  if (whole)
    hipLaunchKernelGGL((gemv_kernel<FMT, NT, R, MT, true, D, DX>), grid, dim3(64 * waves), lds, stream, a, parts);
  else
    hipLaunchKernelGGL((gemv_kernel<FMT, NT, R, MT, false, D, DX>), grid, dim3(64 * waves), lds, stream, a, parts);
}

template <int FMT>
static void gemv_format(const GemvArgs& a, hipStream_t stream) {
  if (a.m <= 4) {
    if (a.n >= 16384)
      gemv_go<FMT, 2, 4, 1, 1, 2>(a, stream);
    else
      gemv_go<FMT, 1, 4, 1, 2, 2>(a, stream);
  } else if (a.m <= 16) {
    if (a.n >= 8192)
      gemv_go<FMT, 2, 16, 1, 1, 1>(a, stream);
    else
      gemv_go<FMT, 1, 16, 1, 2, 2>(a, stream);
  } else {
    gemv_go<FMT, 2, 16, 2, 1, 1>(a, stream);
  }
}

hipError_t launch_gemv(int fmt, const GemvArgs& a, hipStream_t stream) {
  if (fmt == WF_MXFP4)
    gemv_format<WF_MXFP4>(a, stream);
  else
    gemv_format<WF_NVFP4>(a, stream);
  return hipGetLastError();
}

namespace {

// Tokens of one chunk whose entries (token, slot) of the router's choices name
// a given expert, found by one wave from ballots. An entry whose expert lies
// outside [0, E) matches no expert; of a token's entries that name the same
// expert, the first stands for all, with the sum of their weights.
//
// Entries are taken in groups of whole tokens, at most 64 entries.
struct Entries {
  const int32_t* idx;               // the chunk's entries
  int n, topk, per;                 // entries, choices per token, entries per group (topk * floor(64 / topk))

  __device__ __forceinline__ Entries(const DecodeArgs& a, int chunk) {
    const int t0 = chunk * kDecodeTokenChunk;
    idx = a.topk_idx + (int64_t)t0 * a.topk;
    topk = a.topk;
    n = min(a.tokens - t0, kDecodeTokenChunk) * topk;
    per = 64 / topk * topk;
  }
  // the lane's expert in the group from entry g0, or -1
  __device__ __forceinline__ int expert(int g0, int lane, int32_t E) const {
    const int i = g0 + lane;
    if (lane >= per || i >= n) return -1;
    const int32_t e = idx[i];
    return e < 0 || e >= E ? -1 : e;
  }
  // of the lanes in `same` (those that name one expert), the first of each token
  __device__ __forceinline__ bool first_of_token(uint64_t same, int lane) const {
    const uint64_t earlier = same & ((1ull << lane) - 1ull) & ~((1ull << (lane - lane % topk)) - 1ull);
    return ((same >> lane) & 1ull) && earlier == 0;
  }
};

__device__ __forceinline__ int bits_below(uint64_t mask, int lane) { return __popcll(mask & ((1ull << lane) - 1ull)); }

// What the second kernel needs of a chunk's entries, written by a spare
// workgroup of the first: the named experts, ascending, and their entries.
struct DecodePlan {
  int32_t slots;
  int32_t slot_e[kMaxGroups];
  int32_t first[kMaxGroups + 1];    // of slot s in list
  int16_t list[kDecodeMaxEntries];
};
static_assert(sizeof(DecodePlan) == kDecodePlanBytes);

__device__ void write_plan(const DecodeArgs& a, int chunk, uint8_t* smem) {
  int32_t* cnt = reinterpret_cast<int32_t*>(smem);        // [kMaxGroups] entries, then [kMaxGroups] places taken
  int16_t* expert = reinterpret_cast<int16_t*>(cnt + 2 * kMaxGroups);
  const Entries en(a, chunk);
  DecodePlan* plan = reinterpret_cast<DecodePlan*>(a.plan) + chunk;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < 2 * kMaxGroups; e += blockDim.x) cnt[e] = 0;
  for (int i = tid; i < en.n; i += blockDim.x) {
    const int32_t e = en.idx[i];
    expert[i] = (int16_t)(e < 0 || e >= a.experts ? -1 : e);
  }
  __syncthreads();
  // an expert that the token named before counts once
  auto counted = [&](int i) __attribute__((always_inline)) {
    int e = expert[i];
    for (int j = i - i % en.topk; j < i; ++j) e = expert[j] == e ? -1 : e;
    return e;
  };
  for (int i = tid; i < en.n; i += blockDim.x) {
    const int e = counted(i);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    const int n0 = cnt[2 * lane], n1 = cnt[2 * lane + 1];
    int rows = n0 + n1, used = (n0 > 0) + (n1 > 0);
    for (int d = 1; d < 64; d <<= 1) {
      const int r = __shfl_up(rows, d, 64), u = __shfl_up(used, d, 64);
      if (lane >= d) {
        rows += r;
        used += u;
      }
    }
    int at = rows - n0 - n1, slot = used - (n0 > 0) - (n1 > 0);
    cnt[kMaxGroups + 2 * lane] = at;
    cnt[kMaxGroups + 2 * lane + 1] = at + n0;
    if (n0 > 0) {
      plan->slot_e[slot] = 2 * lane;
      plan->first[slot++] = at;
    }
    if (n1 > 0) {
      plan->slot_e[slot] = 2 * lane + 1;
      plan->first[slot++] = at + n0;
    }
    if (lane == 63) {
      plan->slots = used;
      plan->first[used] = rows;
    }
  }
  __syncthreads();
  // the order of an expert's entries among themselves changes no result
  for (int i = tid; i < en.n; i += blockDim.x) {
    const int e = counted(i);
    if (e >= 0) plan->list[atomicAdd(&cnt[kMaxGroups + e], 1)] = (int16_t)i;
  }
}
constexpr int kPlanLds = 8 * kMaxGroups + 2 * kDecodeMaxEntries;

// Steps that the weights are loaded ahead: about 4 KiB of a wave in flight.
template <int FMT>
constexpr int kUpAhead = 1;
template <int FMT>
constexpr int kDownAhead = FMT == WF_BF16 ? 1 : 2;

constexpr int kRowList = kDecodeTokenChunk * 8;           // a wave's list of rows: entry and weight

// A = w silu(g) u of every entry, [g | u] = W1_e x_t. A team of `parts` waves
// owns 16 values of f of the slot-th expert that the chunk's entries name, for
// all of that expert's entries, and splits the hidden dimension; a workgroup
// is waves / parts teams. Every wave finds its expert and rows by itself. A is
// kept as a sum of two bf16 numbers (16 bits), since the second product takes
// bf16. ROWS: the most rows an expert can have (4, 16 or more).
template <int FMT, bool WHOLE, int ROWS>
__global__ __launch_bounds__(256, 3) void decode_up_kernel(DecodeArgs a, int parts, int tile_bytes) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int slot = blockIdx.y, chunk = blockIdx.z;
  if (blockIdx.x == gridDim.x - 1) {
    if (slot == 0) write_plan(a, chunk, smem);
    return;
  }
  uint8_t* const mine = smem + wave * tile_bytes;
  const Entries en(a, chunk);
  // the slot-th named expert: a set of the named ones in the wave's own LDS
  uint32_t* const set = reinterpret_cast<uint32_t*>(mine);
  if (lane < kMaxGroups / 32) set[lane] = 0;
  wave_lds_fence();
  for (int g0 = 0; g0 < en.n; g0 += en.per) {
    const int e = en.expert(g0, lane, a.experts);
    if (e >= 0) atomicOr(&set[e >> 5], 1u << (e & 31));
  }
  wave_lds_fence();
  int e = -1, left_slots = slot;
#pragma unroll
  for (int q = 0; q < kMaxGroups / 32; ++q) {
    uint32_t bits = __builtin_amdgcn_readfirstlane(set[q]);
    const int c = __popc(bits);
    if (e < 0 && left_slots < c) {
      for (int i = 0; i < left_slots; ++i) bits &= bits - 1;
      e = 32 * q + __ffs(bits) - 1;
    }
    left_slots -= c;
  }
  wave_lds_fence();
  if (e < 0) return;                                      // fewer experts named than slots: all of the workgroup leaves
  // its rows
  int32_t* const row_entry = reinterpret_cast<int32_t*>(mine);
  float* const row_w = reinterpret_cast<float*>(mine) + kDecodeTokenChunk;
  const float* wts = a.topk_w != nullptr ? a.topk_w + (int64_t)chunk * kDecodeTokenChunk * a.topk : nullptr;
  int count = 0;
  for (int g0 = 0; g0 < en.n; g0 += en.per) {
    const uint64_t same = __ballot(en.expert(g0, lane, a.experts) == e);
    if (same == 0) continue;
    const bool keep = en.first_of_token(same, lane);
    const uint64_t firsts = __ballot(keep);
    if (keep) {
      float wt = 0.f;
      const int last = lane - lane % en.topk + en.topk;
      for (int j = lane; j < last; ++j)
        if ((same >> j) & 1ull) wt += wts != nullptr ? wts[g0 + j] : 1.0f;
      const int at = count + bits_below(firsts, lane);
      row_entry[at] = g0 + lane;
      row_w[at] = wt;
    }
    count += __popcll(firsts);
  }
  wave_lds_fence();

  const int team = wave / parts, part = wave % parts;
  const int tile = (int)blockIdx.x * (waves / parts) + team, tiles = a.ffn / 16, f0 = min(tile, tiles - 1) * 16;
  const int nb = a.hidden / 32;
  const int s0 = part_start<FMT>(nb, part, parts), s1 = part_start<FMT>(nb, part + 1, parts);
  float* const red = reinterpret_cast<float*>(smem + (size_t)(wave - part) * tile_bytes + kRowList);
  auto rows_from = [&](auto r_, auto mt_, int c0) __attribute__((always_inline)) {
    constexpr int R = decltype(r_)::value, MT = decltype(mt_)::value;
    typedef Walk<FMT, 2, R, MT, WHOLE, kUpAhead<FMT>, 1> Wk;
    Wk k;
    k.nb = nb;
    const int64_t first[2] = {(int64_t)e * 2 * a.ffn + f0, (int64_t)e * 2 * a.ffn + a.ffn + f0};
    k.weight_tiles(a.w1, a.w1_s, first, 16);
    k.x = a.x + (int64_t)chunk * kDecodeTokenChunk * a.hidden * 2;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < Wk::XL; ++i) {
        const int entry = row_entry[min(c0 + R * t + 4 * i + (lane >> 4), count - 1)];
        k.xoff[t][i] = (uint32_t)(entry / en.topk) * (uint32_t)(a.hidden * 2);
      }
    v4f acc[2][MT];
    clear(acc);
    k.run(mine + kRowList, s0, s1, acc);
    if (parts > 1) {
      __syncthreads();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *(reinterpret_cast<float*>(mine + kRowList) + ((t * MT + u) * 4 + r) * 64 + lane) = acc[t][u][r];
      __syncthreads();
    }
#pragma unroll
    for (int o = 0; o < MT * 4; ++o) {
      if (o % parts != part) continue;
      const int u = o >> 2, r = o & 3;
      float g = acc[0][u][r], up = acc[1][u][r];
      if (parts > 1) {
        g = up = 0.f;
        for (int i = 0; i < parts; ++i) {
          const float* p = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(red) + (size_t)i * tile_bytes);
          g += p[o * 64 + lane];
          up += p[(MT * 4 + o) * 64 + lane];
        }
      }
      const int in_tile = (lane >> 4) * 4 + r, row = c0 + R * u + in_tile;
      if (in_tile >= R || row >= count || tile >= tiles) continue;
      const float v = row_w[row] * (g / (1.0f + expf(-g))) * up;
      const __bf16 hi = (__bf16)v;
      // an infinite or NaN value has no second part
      const __bf16 lo = abs_bits((float)hi) < 0x7F800000u ? (__bf16)(v - (float)hi) : (__bf16)0.0f;
      uint16_t* const to = a.act + ((int64_t)chunk * kDecodeTokenChunk * en.topk + row_entry[row]) * 2 * a.ffn + f0 + (lane & 15);
      to[0] = __builtin_bit_cast(uint16_t, hi);
      to[a.ffn] = __builtin_bit_cast(uint16_t, lo);
    }
    if (parts > 1) __syncthreads();                       // before the tiles are used again
  };
  typedef std::integral_constant<int, 1> One;
  typedef std::integral_constant<int, 16> Sixteen;
  if constexpr (ROWS <= 4) {
    rows_from(std::integral_constant<int, 4>{}, One{}, 0);
  } else if constexpr (ROWS <= 16) {
    rows_from(Sixteen{}, One{}, 0);
  } else {
    for (int c0 = 0; c0 < count; c0 += 32) {
      if (count - c0 <= 16)
        rows_from(Sixteen{}, One{}, c0);
      else
        rows_from(Sixteen{}, std::integral_constant<int, 2>{}, c0);
    }
  }
}

// y[t] = sum over the token's entries of W2_e . A. Workgroup (h-tile, token
// chunk): 16 values of h for up to kDecodeTokenChunk tokens; the k-steps of
// all named experts, one after the other, are split evenly over its waves.
// A tile's activation rows are 8 entries' high parts and the same 8 entries'
// low parts, whose results are added. Each wave adds its results to a slice
// of its own in LDS (a token appears once among an expert's entries), and the
// slices are added in wave order, so the sum has one order whatever the
// timing.
template <int FMT, bool WHOLE, int ROWS>
__global__ __launch_bounds__(512, 2) void decode_down_kernel(DecodeArgs a, int tile_bytes) {
  extern __shared__ __align__(16) uint8_t smem[];         // [waves][tokens of the chunk][16] sums, then the waves' tiles
  __shared__ DecodePlan plan;
  float* const ys = reinterpret_cast<float*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int t0 = blockIdx.y * kDecodeTokenChunk, nt = min(a.tokens - t0, kDecodeTokenChunk);
  {
    const DecodePlan* p = reinterpret_cast<const DecodePlan*>(a.plan) + blockIdx.y;
    const int n = min(nt * a.topk, kDecodeMaxEntries);
    constexpr int kHead = offsetof(DecodePlan, list) / 4;
    for (int i = tid; i < kHead + (n + 1) / 2; i += blockDim.x)
      reinterpret_cast<int32_t*>(&plan)[i] = reinterpret_cast<const int32_t*>(p)[i];
  }
  for (int o = tid; o < waves * nt * 16; o += blockDim.x) ys[o] = 0.f;
  __syncthreads();
  const int nb = a.ffn / 32, ns = k_units<FMT>(nb), steps = (nb + kStepBlocks<FMT> - 1) / kStepBlocks<FMT>;
  const int h0 = blockIdx.x * 16;
  const int64_t units = (int64_t)plan.slots * ns;
  int64_t u = units * wave / waves;
  const int64_t u_end = units * (wave + 1) / waves;
  float* mine = ys + wave * nt * 16;
  while (u < u_end) {
    const int slot = (int)(u / ns), u0 = (int)(u % ns), u1 = (int)min((int64_t)ns, u0 + (u_end - u));
    const int s0 = u0 * kUnit<FMT>, s1 = min(u1 * kUnit<FMT>, steps);
    const int e = __builtin_amdgcn_readfirstlane(plan.slot_e[slot]);
    const int row0 = __builtin_amdgcn_readfirstlane(plan.first[slot]);
    const int rows = __builtin_amdgcn_readfirstlane(plan.first[slot + 1]) - row0;
    u += u1 - u0;
    auto rows_from = [&](auto r_, auto mt_, int c0) __attribute__((always_inline)) {
      constexpr int R = decltype(r_)::value, MT = decltype(mt_)::value, H = R / 2;
      typedef Walk<FMT, 1, R, MT, WHOLE, MT == 1 ? kDownAhead<FMT> : 1, 1> Wk;
      Wk k;
      k.nb = nb;
      const int64_t first[1] = {(int64_t)e * a.hidden + h0};
      k.weight_tiles(a.w2, a.w2_s, first, 16);
      k.x = reinterpret_cast<const uint8_t*>(a.act) + (int64_t)t0 * a.topk * a.ffn * 4;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < Wk::XL; ++i) {
          const int r = 4 * i + (lane >> 4);
          const int entry = plan.list[row0 + min(c0 + H * t + r % H, rows - 1)];
          k.xoff[t][i] = (uint32_t)(2 * entry + (r < H ? 0 : 1)) * (uint32_t)(a.ffn * 2);
        }
      v4f acc[1][MT];
      clear(acc);
      k.run(smem + waves * nt * 64 + wave * tile_bytes, s0, s1, acc);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v;
          int row;
          if constexpr (R == 4) {
            if (q >= 2) continue;
            v = acc[0][t][q] + acc[0][t][q + 2];
            row = lane < 16 ? c0 + q : rows;
          } else {
            v = sum_halves(acc[0][t][q]);
            row = lane < 32 ? c0 + 8 * t + (lane >> 4) * 4 + q : rows;
          }
          if (row < rows) mine[plan.list[row0 + row] / a.topk * 16 + (lane & 15)] += v;
        }
    };
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 16> Sixteen;
    if constexpr (ROWS <= 2) {
      rows_from(std::integral_constant<int, 4>{}, One{}, 0);
    } else if constexpr (ROWS <= 8) {
      rows_from(Sixteen{}, One{}, 0);
    } else {
      for (int c0 = 0; c0 < rows; c0 += 16) {
        if (rows - c0 <= 8)
          rows_from(Sixteen{}, One{}, c0);
        else
          rows_from(Sixteen{}, std::integral_constant<int, 2>{}, c0);
      }
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

template <int FMT, bool WHOLE, int ROWS>
static void decode_up_rows(const DecodeArgs& a, hipStream_t stream) {
  const int chunks = (a.tokens + kDecodeTokenChunk - 1) / kDecodeTokenChunk;
  const int slots = std::min(std::min(a.tokens, kDecodeTokenChunk) * a.topk, a.experts);
  const int ns = k_units<FMT>(a.hidden / 32), tiles = a.ffn / 16;
  int parts = 1;
  while (parts < 4 && parts * 2 <= ns && (int64_t)tiles * slots * chunks * parts * 2 <= kWavesWanted) parts *= 2;
  constexpr int A = kUpAhead<FMT>;
  constexpr int tile = kRowList + (ROWS <= 4 ? std::max(Walk<FMT, 2, 4, 1, WHOLE, A, 1>::kLds, 2048)
                                   : ROWS <= 16 ? std::max(Walk<FMT, 2, 16, 1, WHOLE, A, 1>::kLds, 2048)
                                                : std::max(Walk<FMT, 2, 16, 2, WHOLE, A, 1>::kLds, 4096));
  const int teams = 4 / parts;
  hipLaunchKernelGGL((decode_up_kernel<FMT, WHOLE, ROWS>), dim3((tiles + teams - 1) / teams + 1, slots, chunks), dim3(256),
                     (size_t)std::max(4 * tile, kPlanLds), stream, a, parts, tile);
}

template <int FMT, bool WHOLE, int ROWS>
static void decode_down_rows(const DecodeArgs& a, hipStream_t stream) {
  const int nt = std::min(a.tokens, kDecodeTokenChunk), waves = 8;
  constexpr int A = kDownAhead<FMT>;
  constexpr int tile = ROWS <= 2   ? Walk<FMT, 1, 4, 1, WHOLE, A, 1>::kLds
                       : ROWS <= 8 ? Walk<FMT, 1, 16, 1, WHOLE, A, 1>::kLds
                                   : std::max(Walk<FMT, 1, 16, 1, WHOLE, A, 1>::kLds, Walk<FMT, 1, 16, 2, WHOLE, 1, 1>::kLds);
  hipLaunchKernelGGL((decode_down_kernel<FMT, WHOLE, ROWS>),
                     dim3(a.hidden / 16, (a.tokens + kDecodeTokenChunk - 1) / kDecodeTokenChunk), dim3(64 * waves),
                     (size_t)waves * (nt * 64 + tile), stream, a, tile);
}

template <int FMT, bool WHOLE>
static void decode_up_go(const DecodeArgs& a, hipStream_t stream) {
  if (a.tokens <= 4)
    decode_up_rows<FMT, WHOLE, 4>(a, stream);
  else if (a.tokens <= 16)
    decode_up_rows<FMT, WHOLE, 16>(a, stream);
  else
    decode_up_rows<FMT, WHOLE, kDecodeTokenChunk>(a, stream);
}

template <int FMT, bool WHOLE>
static void decode_down_go(const DecodeArgs& a, hipStream_t stream) {
  if (a.tokens <= 2)
    decode_down_rows<FMT, WHOLE, 2>(a, stream);
  else if (a.tokens <= 8)
    decode_down_rows<FMT, WHOLE, 8>(a, stream);
  else
    decode_down_rows<FMT, WHOLE, kDecodeTokenChunk>(a, stream);
}

template <int FMT>
static hipError_t decode_go(const DecodeArgs& a, hipStream_t stream) {
  if (whole_steps<FMT>(a.hidden, a.w1_s))
    decode_up_go<FMT, true>(a, stream);
  else
    decode_up_go<FMT, false>(a, stream);
  if (whole_steps<FMT>(a.ffn, a.w2_s))
    decode_down_go<FMT, true>(a, stream);
  else
    decode_down_go<FMT, false>(a, stream);
  return hipGetLastError();
}

hipError_t launch_decode(int fmt, const DecodeArgs& a, hipStream_t stream) {
  if (fmt == WF_BF16) return decode_go<WF_BF16>(a, stream);
  if (fmt == WF_MXFP8) return decode_go<WF_MXFP8>(a, stream);
  return decode_go<WF_MXFP4>(a, stream);
}

}  // namespace mx
