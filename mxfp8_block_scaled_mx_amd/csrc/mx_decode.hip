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
// expanded to bf16 in registers, exactly between bf16's last step, 2^-133, and
// 2^128 (an E2M1 or E4M3 element times a power of two, or E2M1 times E4M3, has at
// most 6 significant bits; E4M3 reaches below 2^-133 under scale codes 0 .. 2 and
// past 2^128 from code 247 on), and products are summed in fp32 by the 16 x 16 x
// 32 bf16 MFMA.
//
// All of it is bound by reading the weights: a byte of 4-bit codes meets 4
// operations per row, far below what the MFMA needs to be busy. So a kernel is
// a way to keep enough whole cache lines of weights on their way: 32 to 64 KiB a
// compute unit, since a line takes 2 to 3 us when the memory is busy (reading
// alone reaches 6.9 TB/s on this layout of loads). What the forms reach (weight
// bytes over time, the calls' other reads not counted; 12 inputs in turn, means):
//   gemv_kernel       4-bit, 1 row: 28672 x 4096 13.9 us, 4.5 TB/s; 4096 x
//                     14336 8.7 us, 3.6 TB/s (3 us are the launch); NVFP4, 5
//                     rows, 14336 x 4096: 12.1 us, 2.7 TB/s (vector units 22% busy,
//                     load unit 20%, LDS 12%: a wave's load, expansion, LDS and
//                     MFMA follow each other)
//   gemv_wide_kernel  4-bit, 28672 x 4096: 16 rows 18.5 us, 3.4 TB/s; 32 rows 21.8
//                     us, 2.9 TB/s; 64 rows 36.7 us, 1.7 TB/s (the activations take
//                     the same path through the load unit and LDS as the weights:
//                     LDS 41% busy at 64 rows, no other unit above 26%)
//   decode_up_kernel  8 experts of 4096 x 14336, 2 choices: 1 token, 4-bit, 22.8 us,
//                     5.5 TB/s; 7 tokens, 8-bit, 131 us, 6.2 TB/s
//   decode_down_kernel   the same: 14.1 us, 4.4 TB/s; 71.6 us, 5.7 TB/s
//   decode_up_wide_kernel, decode_down_wide_kernel   64 tokens, 4-bit: 109 us, 4.5
//                     TB/s; 87 us, 2.8 TB/s (its activations are twice 16 bits
//                     of every value, and as many bytes as the weights by way of L2)
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

// A barrier of the workgroup that orders LDS and leaves global loads in flight.
__device__ __forceinline__ void team_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Values of k in one step of the walks below: 128-byte pieces of a 4-bit or
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

// A wave's weights: NT tiles of 16 rows, loaded D steps ahead into registers and
// passed step by step through a private LDS tile.
//
// The MFMA's lane layout (lane l holds row l % 16) makes neighbouring lanes
// read different rows, which costs the load path one cache line per lane. So
// rows are loaded as whole pieces (consecutive lanes, consecutive 16-byte
// chunks) and the tile's chunks are swizzled. That leaves bank conflicts: the
// rows of a 4-bit or 8-bit tile are 128 bytes, so rows r and r + 8 of a read share
// their banks, and scales are read byte by byte. Conflicts are 17 to 44% of the
// LDS's busy cycles, and those 12 to 42% of a kernel's. Scales come 1 KiB (G
// steps) at a time. No barrier: the tile is the wave's own.
//
// WHOLE: k is a multiple of the step, and scale rows of 16 bytes. Otherwise
// blocks past the end repeat the last one and count as zero.
template <int FMT, int NT, bool WHOLE, int D>
struct Weights {
  static constexpr int H = kHalves<FMT>, S = kScaleBytes<FMT>, BW = kWords<FMT>;
  static constexpr int W = BW * H;                                          // 16-byte loads of a tile and step
  static constexpr int SB = 4 * H * S;                                      // scale bytes of a row and step
  static constexpr int LR = 4 / NT;                                         // lanes of a scale row
  static constexpr int G = SB > 0 ? 16 * LR / SB : D;                       // steps of a scale load
  static constexpr int kTile = 1024 * W;
  static constexpr int kLds = NT * kTile + (S > 0 ? 1024 : 0);              // bytes of one wave
  static_assert(G % D == 0 && (S == 0 || kUnit<FMT> * SB == 16));

  const uint8_t* w[NT];             // first row of each tile (wave-uniform)
  uint32_t woff[W];                 // the lane's row within a tile, in bytes
  const uint8_t* ws;                // the lane's scale row
  int nb;                           // blocks of a row
  int s1;                           // end of the steps
  u32x4 wr[D][NT][W], sr;

  // tile t: consecutive rows from row first[t]; the last row is repeated where
  // fewer than 16 are left
  __device__ __forceinline__ void tiles(const uint8_t* base, const uint8_t* sbase, const int64_t (&first)[NT], int left) {
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

  // A load past the end is issued all the same (the number of loads in flight
  // stays fixed), with every lane at one address. Pieces of ragged rows share
  // their first and last cache line with the next step, so they are not
  // nontemporal (4-bit, 3 rows, 11740 x 14624: 26.8 us nontemporal, 19.2 us
  // plain; whole rows gain from it: reading alone 6.25 TB/s plain, 6.9 TB/s).
  __device__ __forceinline__ void load(int t, u32x4 (&to)[NT][W]) {
    const int lane = threadIdx.x & 63;
    const int c = lane % (4 * W);
    const uint32_t at = WHOLE ? (uint32_t)(t * 64 * W + c * 16)
                              : (uint32_t)(min(kStepBlocks<FMT> * t + c / BW, nb - 1) * 16 * BW + (c % BW) * 16);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const u32x4* from = reinterpret_cast<const u32x4*>(w[n] + (t < s1 ? woff[i] + at : 0u));
        if constexpr (WHOLE)
          to[n][i] = __builtin_nontemporal_load(from);
        else
          to[n][i] = *from;
      }
  }
  // 16 bytes of a scale row per lane: the G steps from s. Where rows are not
  // whole steps, a window that would pass the row's end begins earlier
  // (scale_shift), and a row of less than 16 bytes is read byte by byte.
  __device__ __forceinline__ void load_scales(int s) {
    if constexpr (S > 0) {
      const int lane = threadIdx.x & 63, row_bytes = nb * S, at = s * SB + lane % LR * 16;
      if constexpr (WHOLE) {
        sr = *reinterpret_cast<const u32x4*>(ws + (at < row_bytes ? at : 0));
      } else if (row_bytes >= 16) {
        __builtin_memcpy(&sr, ws + min(at, row_bytes - 16), 16);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) v |= (uint32_t)ws[min(4 * q + b, row_bytes - 1)] << (8 * b);
          sr[q] = v;
        }
      }
    }
  }
  // how much later the scale at byte `at` of a row lies in its window
  __device__ __forceinline__ int scale_shift(int at) const {
    const int row_bytes = nb * S;
    return WHOLE || row_bytes < 16 ? 0 : max(0, (at & ~15) + 16 - row_bytes);
  }
  // the scales of the group that begins at step s, and the next group's load
  __device__ __forceinline__ void stage_scales(uint8_t* lds, int s) {
    if constexpr (S > 0) {
      wave_lds_fence();                                   // after the previous steps' reads
      *reinterpret_cast<u32x4*>(lds + NT * kTile + (threadIdx.x & 63) * 16) = sr;
      if (s + G < s1) load_scales(s + G);
    }
  }
  // step t from registers wr[u] to the tile
  __device__ __forceinline__ void stage(uint8_t* lds, int t, const u32x4 (&from)[NT][W]) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int row = (i * 64 + lane) / (4 * W), c = lane % (4 * W);
        u32x4 v = from[n][i];
        if constexpr (!WHOLE)
          if (kStepBlocks<FMT> * (t + 1) > nb) {
            const bool ok = kStepBlocks<FMT> * t + c / BW < nb;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = ok ? v[q] : 0u;
          }
        *reinterpret_cast<u32x4*>(lds + n * kTile + (row * 4 * W + (c ^ (row & (4 * W - 1)))) * 16) = v;
      }
  }
  // tile n's block of the lane (half h of step t, the in_group-th of its scale group) as 4 fragments
  __device__ __forceinline__ void fragments(const uint8_t* lds, int n, int t, int h, int in_group, bf16x8 (&wf)[4]) const {
    const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
    u32x4 q[BW];
    uint32_t sc = 0;
#pragma unroll
    for (int i = 0; i < BW; ++i)
      q[i] = *reinterpret_cast<const u32x4*>(lds + n * kTile + (li * 4 * W + (((h * 4 + g) * BW + i) ^ (li & (4 * W - 1)))) * 16);
    // (a block past the row's end has codes of zero, and its scale is any of the row's)
    const int shift = min(scale_shift(t * SB + (h * 4 + g) * S), 15 - ((in_group * SB + (h * 4 + g) * S) & 15));
    const uint8_t* p = lds + NT * kTile + (n * 16 + li) * 16 * LR + in_group * SB + (h * 4 + g) * S + (S == 2 ? shift & ~1 : shift);
    if constexpr (S == 1) sc = *p;
    if constexpr (S == 2) sc = *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) wf[j] = expand<FMT>(q, sc, j);
  }
};

// One wave's part of the products of NT tiles of 16 weight rows with R
// activation rows (16, or 4 or 8 repeated over the MFMA's 16) over the k-steps
// [s0, s1). Result: acc[n][0] register r of lane l = activation row
// (l / 16) * 4 + r, weight row l % 16. The activations go the weights' way.
// Loads complete in the order of their issue as far as a wave can tell, so both
// are issued equally far ahead, the activations first: waiting for either then
// leaves everything younger in flight. MFMA j of 128 values contracts values 8 j .. 8 j + 7 of the
// four lane groups' blocks, the same permutation of k on both sides.
template <int FMT, int NT, int R, bool WHOLE, int D>
struct Walk : Weights<FMT, NT, WHOLE, D> {
  typedef Weights<FMT, NT, WHOLE, D> Wt;
  static constexpr int H = Wt::H, G = Wt::G;
  static constexpr int kLds = Wt::kLds + 256 * R;                           // bytes of one wave
  static constexpr int XL = R / 4;                                          // loads of an activation tile
  static constexpr int DX = D * H;                                          // half steps ahead

  const uint8_t* x;                 // activations (uniform)
  uint32_t xoff[XL];                // the lane's rows, in bytes

  __device__ __forceinline__ void run(uint8_t* lds, int s0, int s1_, v4f (&acc)[NT][1]) {
    if (s0 >= s1_) return;
    this->s1 = s1_;
    const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
    const int nb = this->nb, s1 = s1_, last = s1 * H - 1;
    u32x4 xr[DX][XL];
    uint8_t* const xl = lds + Wt::kLds;
    auto load_x = [&](int t, u32x4 (&to)[XL]) __attribute__((always_inline)) {
      const uint32_t at = WHOLE ? t * 256 + li * 16 : min(4 * t + li / 4, nb - 1) * 64 + (li % 4) * 16;
#pragma unroll
      for (int i = 0; i < XL; ++i) to[i] = *reinterpret_cast<const u32x4*>(x + (t <= last ? xoff[i] + at : xoff[0]));
    };
    this->load_scales(s0);
#pragma unroll
    for (int d = 0; d < DX; ++d) {
      load_x(s0 * H + d, xr[d]);
      if (d % H == 0) this->load(s0 + d / H, this->wr[d / H]);
    }
    int in_group = 0;
    for (int s = s0; s < s1; s += D) {
      if (in_group == 0) this->stage_scales(lds, s);
#pragma unroll
      for (int uh = 0; uh < D * H; ++uh) {
        const int u = uh / H, h = uh % H, t = s + u, th = t * H + h;
        if (h == 0 && t >= s1) return;
        wave_lds_fence();
        if (h == 0) this->stage(lds, t, this->wr[u]);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
          const int row = i * 4 + g;
          u32x4 v = xr[uh][i];
          if constexpr (!WHOLE)
            if (4 * th + 4 > nb) {
              const bool ok = 4 * th + li / 4 < nb;
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = ok ? v[q] : 0u;
            }
          *reinterpret_cast<u32x4*>(xl + (row * 16 + (li ^ row)) * 16) = v;
        }
        load_x(th + DX, xr[uh]);
        if (h == 0) this->load(t + D, this->wr[u]);
        wave_lds_fence();
        bf16x8 xf[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = li % R;
          xf[j] = *reinterpret_cast<const bf16x8*>(xl + (row * 16 + ((g * 4 + j) ^ row)) * 16);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          bf16x8 wf[4];
          this->fragments(lds, n, t, h, in_group + u, wf);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[n][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[j], wf[j], acc[n][0], 0, 0, 0);
        }
      }
      in_group = in_group + D < G ? in_group + D : 0;
    }
  }
};

// The same for more rows: the 4 waves of a workgroup own NT tiles each and walk
// the same steps, so that each activation tile (MT tiles of 16 rows) is loaded
// once for all four and shared through LDS, in two buffers with one barrier per
// half step. All four waves call run() with the same steps.
template <int FMT, int NT, int MT, bool WHOLE, int D>
struct WideWalk : Weights<FMT, NT, WHOLE, D> {
  typedef Weights<FMT, NT, WHOLE, D> Wt;
  static constexpr int H = Wt::H, G = Wt::G;
  static constexpr int kXTile = 4096;                                       // 16 rows of 128 values
  static constexpr int kShared = 2 * MT * kXTile;                           // bytes of the workgroup, and Wt::kLds for each wave
  static constexpr int DX = D * H;                                          // half steps ahead

  const uint8_t* x;                 // activations (uniform)
  uint32_t xoff[MT];                // the thread's row (tid / 16) of each tile, in bytes

  __device__ __forceinline__ void run(uint8_t* shared, uint8_t* lds, int s0, int s1_, v4f (&acc)[NT][MT]) {
    if (s0 >= s1_) return;
    this->s1 = s1_;
    const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g = lane >> 4, xrow = tid >> 4;
    const int nb = this->nb, s1 = s1_, last = s1 * H - 1;
    u32x4 xr[DX][MT];
    auto load_x = [&](int t, u32x4 (&to)[MT]) __attribute__((always_inline)) {
      const uint32_t at = WHOLE ? t * 256 + li * 16 : min(4 * t + li / 4, nb - 1) * 64 + (li % 4) * 16;
#pragma unroll
      for (int m = 0; m < MT; ++m) to[m] = *reinterpret_cast<const u32x4*>(x + (t <= last ? xoff[m] + at : xoff[0]));
    };
    auto stage_x = [&](int t, const u32x4 (&from)[MT]) __attribute__((always_inline)) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        u32x4 v = from[m];
        if constexpr (!WHOLE)
          if (4 * t + 4 > nb) {
            const bool ok = 4 * t + li / 4 < nb;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = ok ? v[q] : 0u;
          }
        *reinterpret_cast<u32x4*>(shared + ((t & 1) * MT + m) * kXTile + (xrow * 16 + (li ^ xrow)) * 16) = v;
      }
    };
    // half step t's activations are in LDS before it begins; those of the DX after it are on their way
    this->load_scales(s0);
    u32x4 x0[MT];
    load_x(s0 * H, x0);
#pragma unroll
    for (int d = 0; d < DX; ++d) {
      load_x(s0 * H + d + 1, xr[d]);
      if (d % H == 0) this->load(s0 + d / H, this->wr[d / H]);
    }
    team_barrier();                                       // the buffers are free
    stage_x(s0 * H, x0);
    team_barrier();
    int in_group = 0;
    for (int s = s0; s < s1; s += D) {
      if (in_group == 0) this->stage_scales(lds, s);
#pragma unroll
      for (int uh = 0; uh < D * H; ++uh) {
        const int u = uh / H, h = uh % H, t = s + u, th = t * H + h;
        if (h == 0 && t >= s1) return;
        wave_lds_fence();
        if (h == 0) this->stage(lds, t, this->wr[u]);
        stage_x(th + 1, xr[uh]);                          // into the buffer that half step th - 1 read
        load_x(th + 1 + DX, xr[uh]);
        if (h == 0) this->load(t + D, this->wr[u]);
        wave_lds_fence();
        bf16x8 wf[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) this->fragments(lds, n, t, h, in_group + u, wf[n]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8 xf = *reinterpret_cast<const bf16x8*>(shared + ((th & 1) * MT + m) * kXTile +
                                                               (li * 16 + ((g * 4 + j) ^ li)) * 16);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf, wf[n][j], acc[n][m], 0, 0, 0);
          }
        team_barrier();
      }
      in_group = in_group + D < G ? in_group + D : 0;
    }
  }

  // Steps [s0, s1), beginning at a place of the workgroup's own where rows are a
  // multiple of 4096 bytes apart: workgroups that walk such rows from the same k
  // at one time meet in the same memory channels (8-bit, 24 tokens of 8 experts,
  // 4096 x 14336: 300 us from one k, 258 us from four).
  __device__ __forceinline__ void run_around(uint8_t* shared, uint8_t* lds, int s0, int s1, int turn, v4f (&acc)[NT][MT]) {
    int from = s0;
    if (this->nb * 16 * Wt::BW % 4096 == 0) from += (s1 - s0) / kUnit<FMT> * (turn % 4) / 4 * kUnit<FMT>;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) run(shared, lds, i == 0 ? from : s0, i == 0 ? s1 : from, acc);
  }
};

template <int NT, int MT>
__device__ __forceinline__ void clear(v4f (&acc)[NT][MT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = v4f{0.f, 0.f, 0.f, 0.f};
}

// Writes the lane's results of one register row: row m, column n of y.
__device__ __forceinline__ void store_y(const GemvArgs& a, int row, int col, float v) {
  const int64_t at = (int64_t)row * a.n + col;
  if (a.y_f32)
    reinterpret_cast<float*>(a.y)[at] = v;
  else
    reinterpret_cast<__bf16*>(a.y)[at] = (__bf16)v;
}
// The factor of a result: 1 / S of an NVFP4 weight.
template <int FMT>
__device__ __forceinline__ float result_scale(const GemvArgs& a) {
  if constexpr (FMT == WF_NVFP4) return (float)(1.0 / (double)nvfp4_tensor_scale(*a.amax));
  return 1.0f;
}
// First rows of the tiles from row n0: one that passes the end moves back (its
// columns before n0 are another's); a matrix of less than 16 rows repeats its last.
template <int NT>
__device__ __forceinline__ void tile_rows(int n0, int n, int64_t (&first)[NT]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) first[t] = max(0, min(n0 + 16 * t, n - 16));
}

// y[m, n] = x[m, k] . W[n, k]^T for at most R rows. A team of `parts` waves
// owns 16 * NT weight rows; its waves split k and add up through LDS in wave
// order (one order whatever the timing). A workgroup is waves / parts teams.
template <int FMT, int NT, int R, bool WHOLE, int D>
__global__ __launch_bounds__(512, 2) void gemv_kernel(GemvArgs a, int parts) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int team = wave / parts, part = wave % parts;
  const int n0 = (blockIdx.x * (waves / parts) + team) * 16 * NT;
  const int m = (int)a.m, n = (int)a.n;
  typedef Walk<FMT, NT, R, WHOLE, D> Wk;
  Wk k;
  k.nb = (int)(a.k / 32);
  int64_t first[NT];
  tile_rows<NT>(n0, n, first);
  k.tiles(a.w, a.ws, first, min(16, n));
  k.x = reinterpret_cast<const uint8_t*>(a.x);
#pragma unroll
  for (int i = 0; i < Wk::XL; ++i) k.xoff[i] = (uint32_t)min(4 * i + (lane >> 4), m - 1) * (uint32_t)(a.ldx * 2);
  v4f acc[NT][1];
  clear(acc);
  k.run(smem + wave * Wk::kLds, part_start<FMT>(k.nb, part, parts), part_start<FMT>(k.nb, part + 1, parts), acc);
  const float scale = result_scale<FMT>(a);
  constexpr int kOut = NT * 256;
  float* red = reinterpret_cast<float*>(smem);
  if (parts > 1) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[wave * kOut + (t * 4 + r) * 64 + lane] = acc[t][0][r];
    __syncthreads();
  }
  // each wave finishes its share of the team's results
#pragma unroll
  for (int o = 0; o < NT * 4; ++o) {
    if (o % parts != part) continue;
    const int r = o & 3, t = o >> 2;
    float v = 0.f;
    if (parts > 1)
      for (int i = 0; i < parts; ++i) v += red[(team * parts + i) * kOut + o * 64 + lane];
    else
      v = acc[t][0][r];
    const int row = (lane >> 4) * 4 + r, col = (int)first[t] + (lane & 15);
    if (row < R && row < m && col < n && col >= n0 + 16 * t) store_y(a, row, col, v * scale);
  }
}

// The same for more rows: a workgroup owns 64 * NT weight rows, 16 * MT rows of
// x and split blockIdx.z of k. With more than one split its sums go to the
// split's plane of a.sums, which the next kernel adds.
template <int FMT, int NT, int MT, bool WHOLE, int D>
__global__ __launch_bounds__(256, 2) void gemv_wide_kernel(GemvArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = (blockIdx.x * 4 + wave) * 16 * NT, m0 = blockIdx.y * 16 * MT;
  const int m = (int)a.m, n = (int)a.n, split = blockIdx.z;
  typedef WideWalk<FMT, NT, MT, WHOLE, D> Wk;
  Wk k;
  k.nb = (int)(a.k / 32);
  int64_t first[NT];
  tile_rows<NT>(n0, n, first);
  k.tiles(a.w, a.ws, first, min(16, n));
  k.x = reinterpret_cast<const uint8_t*>(a.x) + (int64_t)m0 * a.ldx * 2;
#pragma unroll
  for (int t = 0; t < MT; ++t) k.xoff[t] = (uint32_t)min(16 * t + (tid >> 4), m - 1 - m0) * (uint32_t)(a.ldx * 2);
  v4f acc[NT][MT];
  clear(acc);
  k.run_around(smem, smem + Wk::kShared + wave * Wk::Wt::kLds, part_start<FMT>(k.nb, split, a.splits),
               part_start<FMT>(k.nb, split + 1, a.splits), blockIdx.x, acc);
  const float scale = result_scale<FMT>(a);
  float* const plane = a.sums + (int64_t)split * m * n;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = m0 + 16 * u + (lane >> 4) * 4 + r, col = (int)first[t] + (lane & 15);
        if (row >= m || col >= n || col < n0 + 16 * t) continue;
        if (a.splits > 1)
          plane[(int64_t)row * n + col] = acc[t][u][r];
        else
          store_y(a, row, col, acc[t][u][r] * scale);
      }
}

// y = the splits' sums, added in order (4 us at 57 x 1740, 16 splits, of which 3
// are the launch).
template <int FMT>
__global__ __launch_bounds__(256) void gemv_sum_kernel(GemvArgs a) {
  const int64_t n = a.m * a.n;
  const float scale = result_scale<FMT>(a);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float v = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) v += a.sums[s * n + i];
    v *= scale;
    if (a.y_f32)
      reinterpret_cast<float*>(a.y)[i] = v;
    else
      reinterpret_cast<__bf16*>(a.y)[i] = (__bf16)v;
  }
}

}  // namespace

// Whether rows of k values are whole steps, with scale rows of 16 bytes.
template <int FMT>
static bool whole_steps(int64_t k, const uint8_t* scales) {
  return k % (32 * kStepBlocks<FMT>) == 0 &&
         (kScaleBytes<FMT> == 0 || (k / 32 * kScaleBytes<FMT> % 16 == 0 && reinterpret_cast<uintptr_t>(scales) % 16 == 0));
}

// Waves a launch splits k for: 8 per compute unit, all resident at once (one
// row, 28672 x 4096 and 14336 x 4096, 4-bit: 8 a unit 12.6 and 8.9 us, 16 a unit
// 13.2 and 9.1 us, 32 a unit 13.0 and 10.3 us).
constexpr int64_t kWavesWanted = 2048;

template <int FMT, int NT, int R, int D>
static void gemv_go(const GemvArgs& a, hipStream_t stream) {
  const int64_t units = k_units<FMT>((int)(a.k / 32)), tiles = (a.n + 16 * NT - 1) / (16 * NT);
  int parts = 1;
  while (parts < 8 && parts * 2 <= units && tiles * parts * 2 <= kWavesWanted) parts *= 2;
  const int waves = std::max(4, parts), teams = waves / parts;
  const dim3 grid((unsigned)((tiles + teams - 1) / teams));
  const size_t lds = (size_t)waves * std::max(Walk<FMT, NT, R, true, D>::kLds, NT * 1024);
  if (whole_steps<FMT>(a.k, a.ws))
    hipLaunchKernelGGL((gemv_kernel<FMT, NT, R, true, D>), grid, dim3(64 * waves), lds, stream, a, parts);
  else
    hipLaunchKernelGGL((gemv_kernel<FMT, NT, R, false, D>), grid, dim3(64 * waves), lds, stream, a, parts);
}

// One tile of weight rows a wave. Two feed each activation fragment to two MFMAs
// but halve the workgroups: better for more than 32 rows only (one and two, 28672
// x 4096, 4-bit: 16 rows 16.1 and 17.0 us, 32 rows 20.5 and 19.9 us, 64 rows 36.0
// and 29.4 us; NVFP4: 18.8 and 19.9, 23.2 and 24.4, 38.3 and 34.8 us; 64 x 4096 x
// 14336, 4-bit: 26.5 and 24.2 us).
template <int FMT, int MT>
static void gemv_wide_go(const GemvArgs& a, hipStream_t stream) {
  constexpr int NT = 1, D = 1;
  const dim3 grid((unsigned)((a.n + 64 * NT - 1) / (64 * NT)), (unsigned)((a.m + 16 * MT - 1) / (16 * MT)), a.splits);
  typedef WideWalk<FMT, NT, MT, true, D> Wk;
  const size_t lds = Wk::kShared + 4 * Wk::Wt::kLds;
  if (whole_steps<FMT>(a.k, a.ws))
    hipLaunchKernelGGL((gemv_wide_kernel<FMT, NT, MT, true, D>), grid, dim3(256), lds, stream, a);
  else
    hipLaunchKernelGGL((gemv_wide_kernel<FMT, NT, MT, false, D>), grid, dim3(256), lds, stream, a);
  if (a.splits > 1)
    hipLaunchKernelGGL((gemv_sum_kernel<FMT>), dim3((unsigned)std::min<int64_t>(2048, (a.m * a.n + 255) / 256)), dim3(256), 0,
                       stream, a);
}

// Which form runs. Two tiles of weight rows a wave halve the work on the
// activations, one tile gives twice the teams. For up to 4 rows two pay once one
// tile a wave already fills the chip (4-bit, one row, one tile two steps ahead
// against two tiles one step ahead: 4096 x 14336 8.7 and 11.6 us, 28672 x 4096
// 14.2 and 13.2 us); for up to 16 rows, where an activation tile is four times the
// loads, earlier (one tile, two: 4096 x 14336 14.0 and 16.4 us, 8192 x 4096 9.0 and
// 7.8 us, 28672 x 4096 24.8 and 20.4 us). Tiles of 8 activation rows save half of
// those loads (8 rows, tiles of 16 and of 8: 28672 x 4096 15.9 and 14.7 us, 4096 x
// 14336 12.4 and 11.7 us; 6 rows, 20000 x 8192 27.3 and 24.3 us). The wide form takes 16, 32 or 64 rows at a
// time (32 rows, 28672 x 4096: 21.2 us as 32, 35.0 us as 64).
template <int FMT>
static void gemv_format(const GemvArgs& a, hipStream_t stream) {
  if (a.splits == 0 && a.m <= 4) {
    if (a.n >= 16384)
      gemv_go<FMT, 2, 4, 1>(a, stream);
    else
      gemv_go<FMT, 1, 4, 2>(a, stream);
  } else if (a.splits == 0 && a.m <= 8) {
    if (a.n >= 8192)
      gemv_go<FMT, 2, 8, 1>(a, stream);
    else
      gemv_go<FMT, 1, 8, 1>(a, stream);
  } else if (a.splits == 0) {
    if (a.n >= 8192)
      gemv_go<FMT, 2, 16, 1>(a, stream);
    else
      gemv_go<FMT, 1, 16, 1>(a, stream);
  } else if (a.m <= 16) {
    gemv_wide_go<FMT, 1>(a, stream);
  } else if (a.m <= 32) {
    gemv_wide_go<FMT, 2>(a, stream);
  } else {
    gemv_wide_go<FMT, 4>(a, stream);
  }
}

// Splits of k of the wide product (0: the narrow one runs): up to 512
// workgroups, 2 a compute unit, of at least 512 values of k each. (64 x 14336 x
// 4096: 2 splits 24.2 us, 3 26.7 us; 64 x 28672 x 4096: 1 split 31.7 us.) For
// more than 8 rows it also runs, unsplit, where its workgroups go round the chip
// at least once: the narrow form's waves load the activations each for itself (16
// rows, narrow and wide: 28672 x 4096 18.7 and 16.9 us, 20000 x 8192 33.5 and 30.8
// us, 16384 x 4096 12.5 and 13.7 us; 20000 x 8192, narrow 6 rows 24 us, wide 8 rows 30 us).
int gemv_splits(int64_t m, int64_t n, int64_t k) {
  if (m <= 8 || (m <= 16 && n < 18432)) return 0;
  const int64_t groups = (n + 63) / 64 * ((m + 63) / 64);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(16, k / 512), 512 / groups));
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
// Entries are taken in groups of whole tokens, at most 64 entries. stage() puts
// them into LDS for the workgroup, so that what follows waits for memory once
// (61 tokens, 5 choices among 60 experts of 544 x 4288, 4-bit, first product:
// 88 us reading them from memory, 76 us).
struct Entries {
  const int32_t* idx;               // the chunk's entries
  int n, topk, per;                 // entries, choices per token, entries per group (topk * floor(64 / topk))
  float* weight;                    // in LDS: the weights of n entries, then their experts (0xFF: none)

  __device__ __forceinline__ Entries(const DecodeArgs& a, int chunk) {
    const int t0 = chunk * kDecodeTokenChunk;
    idx = a.topk_idx + (int64_t)t0 * a.topk;
    topk = a.topk;
    n = min(a.tokens - t0, kDecodeTokenChunk) * topk;
    per = 64 / topk * topk;
  }
  __host__ __device__ static constexpr int bytes(int entries) { return (entries * 5 + 15) & ~15; }
  __device__ __forceinline__ void stage(const DecodeArgs& a, int chunk, uint8_t* lds) {
    weight = reinterpret_cast<float*>(lds);
    const float* w = a.topk_w != nullptr ? a.topk_w + (int64_t)chunk * kDecodeTokenChunk * topk : nullptr;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int32_t e = idx[i];
      weight[i] = w != nullptr ? w[i] : 1.0f;
      lds[4 * n + i] = e < 0 || e >= a.experts ? 0xFF : (uint8_t)e;
    }
    __syncthreads();
  }
  // the lane's expert in the group from entry g0, or 0xFF
  __device__ __forceinline__ int expert(int g0, int lane) const {
    const int i = g0 + lane;
    return lane < per && i < n ? reinterpret_cast<const uint8_t*>(weight)[4 * n + i] : 0xFF;
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
  uint8_t used[kDecodeMaxEntries];  // whether entry i is in list
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
    plan->used[i] = e >= 0;
    if (e >= 0) plan->list[atomicAdd(&cnt[kMaxGroups + e], 1)] = (int16_t)i;
  }
}
constexpr int kPlanLds = 8 * kMaxGroups + 2 * kDecodeMaxEntries;

// Steps that the second product's weights are loaded ahead: 4 KiB of a wave in
// flight, as the first product has them from one step of its two tiles (two
// steps there: one 4-bit token of 8 experts, 4096 x 14336, 25.1 us, one 23.1 us; here,
// one step and two: 14.1 and 13.5 us, 8-bit with 7 tokens 85 and 75 us, bf16 no
// difference).
template <int FMT>
constexpr int kDownAhead = FMT == WF_BF16 ? 1 : 2;

constexpr int kRowList = kDecodeTokenChunk * 8;           // a wave's list of rows: entry and weight

// The slot-th expert that the chunk's entries name, and its rows in the wave's
// own LDS: entries and their weights. Every lane of the wave takes part.
struct ExpertRows {
  int expert, count;                // -1: fewer experts are named than slots
  const int32_t* entry;
  const float* weight;

  __device__ __forceinline__ ExpertRows(const Entries& en, int slot, uint8_t* lds) {
    const int lane = threadIdx.x & 63;
    uint32_t* const set = reinterpret_cast<uint32_t*>(lds);
    if (lane < kMaxGroups / 32) set[lane] = 0;
    wave_lds_fence();
    for (int g0 = 0; g0 < en.n; g0 += en.per) {
      const int e = en.expert(g0, lane);
      if (e < kMaxGroups) atomicOr(&set[e >> 5], 1u << (e & 31));
    }
    wave_lds_fence();
    expert = -1;
    count = 0;
    int left = slot;
#pragma unroll
    for (int q = 0; q < kMaxGroups / 32; ++q) {
      uint32_t bits = __builtin_amdgcn_readfirstlane(set[q]);
      const int c = __popc(bits);
      if (expert < 0 && left < c) {
        for (int i = 0; i < left; ++i) bits &= bits - 1;
        expert = 32 * q + __ffs(bits) - 1;
      }
      left -= c;
    }
    wave_lds_fence();
    if (expert < 0) return;
    int32_t* const rows = reinterpret_cast<int32_t*>(lds);
    float* const w = reinterpret_cast<float*>(lds) + kDecodeTokenChunk;
    for (int g0 = 0; g0 < en.n; g0 += en.per) {
      const uint64_t same = __ballot(en.expert(g0, lane) == expert);
      if (same == 0) continue;
      const bool keep = en.first_of_token(same, lane);
      const uint64_t firsts = __ballot(keep);
      if (keep) {
        float wt = 0.f;
        const int end = lane - lane % en.topk + en.topk;
        for (int j = lane; j < end; ++j)
          if ((same >> j) & 1ull) wt += en.weight[g0 + j];
        const int at = count + bits_below(firsts, lane);
        rows[at] = g0 + lane;
        w[at] = wt;
      }
      count += __popcll(firsts);
    }
    wave_lds_fence();
    entry = rows;
    weight = w;
  }
};

// A = w silu(g) u of one value, kept as the sum of two bf16 numbers (16 bits),
// since the second product takes bf16 (0.1 to 0.3% of the layer's bf16 results then
// differ from the rounded exact ones, 0.1 to 0.2% where A stays fp32; a third
// number would be half as many activations and MFMAs again). to: the entry's row, ffn further the second part.
__device__ __forceinline__ void store_act(uint16_t* to, int ffn, float w, float g, float u) {
  const float v = w * (g / (1.0f + expf(-g))) * u;
  const __bf16 hi = (__bf16)v;
  // an infinite or NaN value has no second part
  const __bf16 lo = abs_bits((float)hi) < 0x7F800000u ? (__bf16)(v - (float)hi) : (__bf16)0.0f;
  to[0] = __builtin_bit_cast(uint16_t, hi);
  to[ffn] = __builtin_bit_cast(uint16_t, lo);
}

typedef std::integral_constant<int, 1> One;
typedef std::integral_constant<int, 2> Two;
typedef std::integral_constant<int, 3> Three;
typedef std::integral_constant<int, 4> Four;
typedef std::integral_constant<int, 8> Eight;
typedef std::integral_constant<int, 16> Sixteen;

// A = w silu(g) u of every entry, [g | u] = W1_e x_t, for at most ROWS (4 or
// 16) tokens. A team of `parts` waves owns 16 values of f of the slot-th expert
// that the entries name, for all of that expert's entries, and splits the
// hidden dimension; a workgroup is waves / parts teams. Every wave finds its
// expert and rows by itself.
template <int FMT, bool WHOLE, int ROWS>
__global__ __launch_bounds__(512, 2) void decode_up_kernel(DecodeArgs a, int parts, int tile_bytes) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6;
  const int slot = blockIdx.y;
  if (blockIdx.x == gridDim.x - 1) {
    if (slot == 0) write_plan(a, 0, smem);
    return;
  }
  Entries en(a, 0);
  en.stage(a, 0, smem);
  uint8_t* const tiles_at = smem + Entries::bytes(en.n);
  uint8_t* const mine = tiles_at + wave * tile_bytes;
  const ExpertRows rows(en, slot, mine);
  if (rows.expert < 0) return;                            // all of the workgroup leaves
  const int team = wave / parts, part = wave % parts;
  const int tile = (int)blockIdx.x * (waves / parts) + team, tiles = a.ffn / 16, f0 = min(tile, tiles - 1) * 16;
  const int nb = a.hidden / 32;
  const int s0 = part_start<FMT>(nb, part, parts), s1 = part_start<FMT>(nb, part + 1, parts);
  auto go = [&](auto r_) __attribute__((always_inline)) {
    constexpr int R = decltype(r_)::value;
    typedef Walk<FMT, 2, R, WHOLE, 1> Wk;
    Wk k;
    k.nb = nb;
    const int64_t first[2] = {(int64_t)rows.expert * 2 * a.ffn + f0, (int64_t)rows.expert * 2 * a.ffn + a.ffn + f0};
    k.tiles(a.w1, a.w1_s, first, 16);
    k.x = a.x;
#pragma unroll
    for (int i = 0; i < Wk::XL; ++i)
      k.xoff[i] = (uint32_t)(rows.entry[min(4 * i + (lane >> 4), rows.count - 1)] / en.topk) * (uint32_t)(a.hidden * 2);
    v4f acc[2][1];
    clear(acc);
    k.run(mine + kRowList, s0, s1, acc);
    if (parts > 1) {
      __syncthreads();
      float* p = reinterpret_cast<float*>(mine + kRowList) + lane;
#pragma unroll
      for (int o = 0; o < 8; ++o) p[o * 64] = acc[o >> 2][0][o & 3];
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r % parts != part) continue;
      float g = acc[0][0][r], up = acc[1][0][r];
      if (parts > 1) {
        g = up = 0.f;
        for (int i = 0; i < parts; ++i) {
          const float* p = reinterpret_cast<const float*>(tiles_at + (wave - part + i) * tile_bytes + kRowList) + lane;
          g += p[r * 64];
          up += p[(4 + r) * 64];
        }
      }
      const int row = (lane >> 4) * 4 + r;
      if (row < R && row < rows.count && tile < tiles)
        store_act(a.act + (int64_t)rows.entry[row] * 2 * a.ffn + f0 + (lane & 15), a.ffn, rows.weight[row], g, up);
    }
  };
  // (8 tokens of one 4-bit expert, 4096 x 14336: 16 rows a tile 19.7 us, 8 18.3 us)
  if (ROWS <= 4 || rows.count <= 4)
    go(Four{});
  else if (rows.count <= 8)
    go(Eight{});
  else
    go(Sixteen{});
}

// The same for more tokens: a workgroup owns 64 values of f of one expert, for
// the expert's entries among a chunk of tokens.
template <int FMT, bool WHOLE, int TILES>
__global__ __launch_bounds__(256, 2) void decode_up_wide_kernel(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = blockIdx.y, chunk = blockIdx.z;
  if (blockIdx.x == gridDim.x - 1) {
    if (slot == 0) write_plan(a, chunk, smem);
    return;
  }
  Entries en(a, chunk);
  uint8_t* const tiles_at = smem + 4 * kRowList;
  en.stage(a, chunk, tiles_at + 2 * TILES * 4096 + 4 * Weights<FMT, 2, WHOLE, 1>::kLds);
  const ExpertRows rows(en, slot, smem + wave * kRowList);
  if (rows.expert < 0) return;
  const int tile = (int)blockIdx.x * 4 + wave, tiles = a.ffn / 16, f0 = min(tile, tiles - 1) * 16;
  const int nb = a.hidden / 32;
  auto go = [&](auto mt_, int c0) __attribute__((always_inline)) {
    constexpr int MT = decltype(mt_)::value;
    typedef WideWalk<FMT, 2, MT, WHOLE, 1> Wk;
    Wk k;
    k.nb = nb;
    const int64_t first[2] = {(int64_t)rows.expert * 2 * a.ffn + f0, (int64_t)rows.expert * 2 * a.ffn + a.ffn + f0};
    k.tiles(a.w1, a.w1_s, first, 16);
    k.x = a.x + (int64_t)chunk * kDecodeTokenChunk * a.hidden * 2;
#pragma unroll
    for (int t = 0; t < MT; ++t)
      k.xoff[t] = (uint32_t)(rows.entry[min(c0 + 16 * t + (tid >> 4), rows.count - 1)] / en.topk) * (uint32_t)(a.hidden * 2);
    v4f acc[2][MT];
    clear(acc);
    k.run_around(tiles_at, tiles_at + 2 * TILES * Wk::kXTile + wave * Wk::Wt::kLds, 0,
                 part_start<FMT>(nb, 1, 1), blockIdx.x, acc);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = c0 + 16 * t + (lane >> 4) * 4 + r;
        if (row < rows.count && tile < tiles)
          store_act(a.act + ((int64_t)chunk * kDecodeTokenChunk * en.topk + rows.entry[row]) * 2 * a.ffn + f0 + (lane & 15),
                    a.ffn, rows.weight[row], acc[0][t][r], acc[1][t][r]);
      }
  };
  for (int c0 = 0; c0 < rows.count; c0 += 16 * TILES) {
    if (rows.count - c0 <= 16)
      go(One{}, c0);
    else if (TILES == 2 || rows.count - c0 <= 32)
      go(Two{}, c0);
    else
      go(std::integral_constant<int, TILES>{}, c0);
  }
}

// The chunk's plan in LDS.
__device__ __forceinline__ void read_plan(const DecodeArgs& a, int chunk, int tokens, DecodePlan& plan) {
  const int32_t* from = reinterpret_cast<const int32_t*>(reinterpret_cast<const DecodePlan*>(a.plan) + chunk);
  const int words = offsetof(DecodePlan, list) / 4 + (tokens * a.topk + 1) / 2;
  for (int i = threadIdx.x; i < words; i += blockDim.x) reinterpret_cast<int32_t*>(&plan)[i] = from[i];
}

// One stretch of the k-steps of all named experts, one expert after the other:
// units [u, end) of unit_steps each. next() gives the steps of the next expert in it.
template <int FMT>
struct Stretch {
  int64_t u, end;
  int ns, steps;                    // units and steps of an expert
  int slot, s0, s1;

  __device__ __forceinline__ Stretch(int slots, int nb, int part, int parts) {
    ns = k_units<FMT>(nb);
    steps = (nb + kStepBlocks<FMT> - 1) / kStepBlocks<FMT>;
    const int64_t units = (int64_t)slots * ns;
    u = units * part / parts;
    end = units * (part + 1) / parts;
  }
  __device__ __forceinline__ bool next() {
    if (u >= end) return false;
    slot = (int)(u / ns);
    const int u0 = (int)(u % ns), u1 = (int)min((int64_t)ns, u0 + (end - u));
    s0 = u0 * kUnit<FMT>;
    s1 = min(u1 * kUnit<FMT>, steps);
    u += u1 - u0;
    return true;
  }
};

// y[t] = sum over the token's entries of W2_e . A, for at most 16
// tokens. A workgroup owns 16 values of h; the k-steps of all named experts,
// one after the other, are split evenly over its waves. A tile's activation
// rows are up to 8 (4, 2) entries' leading parts and the same entries' second
// parts, whose results are added. Each wave adds its results to a slice of its
// own in LDS (a token appears once among an expert's entries), and the slices
// are added in wave order, so the sum has one order whatever the timing.
template <int FMT, bool WHOLE>
__global__ __launch_bounds__(8 * 64, 2) void decode_down_kernel(DecodeArgs a, int tile_bytes) {
  extern __shared__ __align__(16) uint8_t smem[];         // [waves][tokens][16] sums, then the waves' tiles
  __shared__ DecodePlan plan;
  float* const ys = reinterpret_cast<float*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6, nt = a.tokens;
  read_plan(a, 0, nt, plan);
  for (int o = tid; o < waves * nt * 16; o += blockDim.x) ys[o] = 0.f;
  __syncthreads();
  const int nb = a.ffn / 32, h0 = blockIdx.x * 16;
  float* mine = ys + wave * nt * 16;
  for (Stretch<FMT> st(plan.slots, nb, wave, waves); st.next();) {
    const int e = __builtin_amdgcn_readfirstlane(plan.slot_e[st.slot]);
    const int row0 = __builtin_amdgcn_readfirstlane(plan.first[st.slot]);
    const int rows = __builtin_amdgcn_readfirstlane(plan.first[st.slot + 1]) - row0;
    auto go = [&](auto r_, int c0) __attribute__((always_inline)) {
      constexpr int R = decltype(r_)::value, H = R / 2;
      typedef Walk<FMT, 1, R, WHOLE, kDownAhead<FMT>> Wk;
      Wk k;
      k.nb = nb;
      const int64_t first[1] = {(int64_t)e * a.hidden + h0};
      k.tiles(a.w2, a.w2_s, first, 16);
      k.x = reinterpret_cast<const uint8_t*>(a.act);
#pragma unroll
      for (int i = 0; i < Wk::XL; ++i) {
        const int r = 4 * i + (lane >> 4);
        k.xoff[i] = (uint32_t)(2 * plan.list[row0 + min(c0 + r % H, rows - 1)] + (r < H ? 0 : 1)) * (uint32_t)(a.ffn * 2);
      }
      v4f acc[1][1];
      clear(acc);
      k.run(smem + waves * nt * 64 + wave * tile_bytes, st.s0, st.s1, acc);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v;
        int row;
        if constexpr (R == 4) {
          if (q >= 2) continue;
          v = acc[0][0][q] + acc[0][0][q + 2];
          row = lane < 16 ? c0 + q : rows;
        } else if constexpr (R == 8) {
          const uint32_t b = __float_as_uint(acc[0][0][q]);
          const u32x2 t = __builtin_amdgcn_permlane16_swap(b, b, false, false);
          v = __uint_as_float(t.x) + __uint_as_float(t.y);
          row = lane < 16 ? c0 + q : rows;
        } else {
          v = sum_halves(acc[0][0][q]);
          row = lane < 32 ? c0 + (lane >> 4) * 4 + q : rows;
        }
        if (row < rows) mine[plan.list[row0 + row] / a.topk * 16 + (lane & 15)] += v;
      }
    };
    // (4 tokens of one 4-bit expert, 4096 x 14336: 16 rows a tile 11.8 us, 8 10.4 us)
    if (rows <= 2)
      go(Four{}, 0);
    else if (rows <= 4)
      go(Eight{}, 0);
    else
      for (int c0 = 0; c0 < rows; c0 += 8) go(Sixteen{}, c0);
  }
  __syncthreads();
  for (int o = tid; o < nt * 16; o += blockDim.x) {
    float v = 0.f;
    for (int i = 0; i < waves; ++i) v += ys[i * nt * 16 + o];
    reinterpret_cast<__bf16*>(a.y)[(int64_t)(o >> 4) * a.hidden + h0 + (o & 15)] = (__bf16)v;
  }
}

// The same for more tokens: a workgroup owns 64 * NT values of h of one expert,
// for the expert's entries among a chunk of tokens, and split blockIdx.y of the
// ffn dimension. Its sums go to the split's plane of a.sums, a row an entry,
// which the next kernel adds. A pass takes up to six row tiles of 8 entries
// each: eight would let fewer workgroups share a compute unit's LDS (4-bit, 64
// tokens of 8 experts, 4096 x 14336: four tiles 93 us, six 87 us, eight 127 us; of 2 experts, 2048
// x 8192: six 29 us, eight 39 us; 8-bit, 60 tokens, 4 choices: 179, 158 and 178 us).
constexpr int kDownTiles = 6;
template <int FMT, bool WHOLE, int NT>
__global__ __launch_bounds__(256, 2) void decode_down_wide_kernel(DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];         // the shared tiles, the waves' tiles
  __shared__ int16_t list[kDecodeTokenChunk];             // the expert's entries, one of a token at most
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = blockIdx.y / a.slots, slot = blockIdx.y % a.slots, chunk = blockIdx.z;
  const DecodePlan& plan = *(reinterpret_cast<const DecodePlan*>(a.plan) + chunk);
  // (all four loads at once; those of a slot past the last are not used)
  const int slots = plan.slots, expert = plan.slot_e[slot], from = plan.first[slot], to = plan.first[slot + 1];
  if (slot >= slots) return;
  const int e = __builtin_amdgcn_readfirstlane(expert), row0 = __builtin_amdgcn_readfirstlane(from);
  const int rows = __builtin_amdgcn_readfirstlane(to) - row0;
  if (tid < rows) list[tid] = plan.list[row0 + tid];
  __syncthreads();
  const int64_t entry0 = (int64_t)chunk * kDecodeTokenChunk * a.topk;
  const int nb = a.ffn / 32, n0 = (blockIdx.x * 4 + wave) * 16 * NT;
  int64_t first[NT];
  tile_rows<NT>(n0, a.hidden, first);
#pragma unroll
  for (int n = 0; n < NT; ++n) first[n] += (int64_t)e * a.hidden;
  auto go = [&](auto mt_, int c0) __attribute__((always_inline)) {
    constexpr int MT = decltype(mt_)::value;
    typedef WideWalk<FMT, NT, MT, WHOLE, 1> Wk;
    Wk k;
    k.nb = nb;
    k.tiles(a.w2, a.w2_s, first, 16);
    k.x = reinterpret_cast<const uint8_t*>(a.act + entry0 * 2 * a.ffn);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int r = tid >> 4;
      k.xoff[t] = (uint32_t)(2 * list[min(c0 + 8 * t + (r & 7), rows - 1)] + (r >> 3)) * (uint32_t)(a.ffn * 2);
    }
    v4f acc[NT][MT];
    clear(acc);
    k.run_around(smem, smem + 2 * kDownTiles * Wk::kXTile + wave * Wk::Wt::kLds, part_start<FMT>(nb, split, a.splits),
                 part_start<FMT>(nb, split + 1, a.splits), blockIdx.x, acc);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // the lower half wave stores the first tile's sums, the upper half the second's
        const int row = c0 + 8 * t + ((lane >> 4) & 1) * 4 + q, n = lane >> 5;
        const float v0 = sum_halves(acc[0][t][q]), v1 = sum_halves(acc[1][t][q]);
        const int h = (int)((n ? first[1] : first[0]) - (int64_t)e * a.hidden) + (lane & 15);
        if (row < rows && h >= n0 + 16 * n && h < a.hidden)
          a.sums[((int64_t)split * a.tokens * a.topk + entry0 + list[row]) * a.hidden + h] = n ? v1 : v0;
      }
  };
  for (int c0 = 0; c0 < rows; c0 += 8 * kDownTiles) {
    if (rows - c0 <= 8)
      go(One{}, c0);
    else if (rows - c0 <= 16)
      go(Two{}, c0);
    else if (rows - c0 <= 24)
      go(Three{}, c0);
    else if (rows - c0 <= 32)
      go(Four{}, c0);
    else
      go(std::integral_constant<int, kDownTiles>{}, c0);
  }
}

// y[t] = the sums of the token's entries and splits; 4 values a thread. The
// planes of a token (its entries in order, each with its splits) go round the
// four waves, whose sums are added in wave order. The rows of entries that are
// in no list were not written. Bound by the latency of its loads: four in flight
// of each wave (64 planes of 8 x 192 values: one at a time 8.2 us, four 4.7 us).
__global__ __launch_bounds__(256) void decode_sum_kernel(DecodeArgs a) {
  __shared__ v4f part[3][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quads = a.hidden / 4, t = blockIdx.y, q = blockIdx.x * 64 + lane;
  const DecodePlan& plan = *(reinterpret_cast<const DecodePlan*>(a.plan) + t / kDecodeTokenChunk);
  const uint64_t used = __ballot(lane < a.topk && plan.used[t % kDecodeTokenChunk * a.topk + min(lane, a.topk - 1)] != 0);
  const float* from = a.sums + (int64_t)t * a.topk * a.hidden + 4 * min(q, quads - 1);
  const int64_t plane = (int64_t)a.tokens * a.topk * a.hidden;
  v4f v = {0.f, 0.f, 0.f, 0.f};
  const int n = a.topk * a.splits;
  for (int p0 = wave; p0 < n; p0 += 16) {                 // 4 loads in flight
    v4f x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = min(p0 + 4 * i, n - 1), j = p / a.splits, s = p - j * a.splits;
      const v4f r = *reinterpret_cast<const v4f*>(from + s * plane + (int64_t)j * a.hidden);
      const bool ok = p0 + 4 * i < n && ((used >> j) & 1ull);
#pragma unroll
      for (int c = 0; c < 4; ++c) x[i][c] = ok ? r[c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v += x[i];
  }
  if (wave > 0) part[wave - 1][lane] = v;
  __syncthreads();
  if (wave > 0 || q >= quads) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) v += part[w][lane];
  bf16x2 o[2];
  o[0].x = (__bf16)v.x;
  o[0].y = (__bf16)v.y;
  o[1].x = (__bf16)v.z;
  o[1].y = (__bf16)v.w;
  *reinterpret_cast<uint2*>(reinterpret_cast<__bf16*>(a.y) + (int64_t)t * a.hidden + 4 * q) =
      make_uint2(__builtin_bit_cast(uint32_t, o[0]), __builtin_bit_cast(uint32_t, o[1]));
}

}  // namespace

template <int FMT, bool WHOLE, int ROWS>
static void decode_up_rows(const DecodeArgs& a, hipStream_t stream) {
  const int slots = std::min(a.tokens * a.topk, a.experts);
  const int units = k_units<FMT>(a.hidden / 32), tiles = a.ffn / 16;
  // A team of 4 reads whole rows at about one time (one row a wave, 4096 bytes
  // apart, is what memory likes least: 8-bit, 7 tokens of 8 experts, 4096 x
  // 14336: parts 1 171 us, 4 133 us). Rows of less than 8 units are split only as
  // far as two units a wave, unless that leaves the chip empty (128 experts, 8
  // tokens, 2048 x 768, 4-bit: 4 units in 4 parts 23.0 us, in 2 parts 20.5 us).
  int parts = 1;
  while (parts < 4 && parts * 2 <= units && (parts * 4 <= units || (int64_t)tiles * slots * parts <= 1024)) parts *= 2;
  constexpr int tile = kRowList + std::max(Walk<FMT, 2, ROWS, WHOLE, 1>::kLds, 2048);
  const int waves = std::max(4, parts), teams = waves / parts;
  hipLaunchKernelGGL((decode_up_kernel<FMT, WHOLE, ROWS>), dim3((tiles + teams - 1) / teams + 1, slots), dim3(64 * waves),
                     (size_t)std::max(Entries::bytes(a.tokens * a.topk) + waves * tile, kPlanLds), stream, a, parts, tile);
}

// Experts that a chunk of tokens can name.
static int decode_slots(int tokens, int topk, int experts) {
  return std::min(std::min(tokens, kDecodeTokenChunk) * topk, experts);
}
// Whether few of a chunk's entries fall to one expert in the mean.
static bool few_each(const DecodeArgs& a, int rows) {
  return (int64_t)std::min(a.tokens, kDecodeTokenChunk) * a.topk <= (int64_t)rows * a.experts;
}

template <int FMT, bool WHOLE, int TILES>
static void decode_up_wide(const DecodeArgs& a, hipStream_t stream) {
  const int chunks = (a.tokens + kDecodeTokenChunk - 1) / kDecodeTokenChunk;
  typedef WideWalk<FMT, 2, TILES, WHOLE, 1> Wk;
  hipLaunchKernelGGL((decode_up_wide_kernel<FMT, WHOLE, TILES>),
                     dim3((a.ffn / 16 + 3) / 4 + 1, decode_slots(a.tokens, a.topk, a.experts), chunks), dim3(256),
                     (size_t)std::max(4 * kRowList + Wk::kShared + 4 * Wk::Wt::kLds +
                                          Entries::bytes(std::min(a.tokens, kDecodeTokenChunk) * a.topk), kPlanLds), stream, a);
}

template <int FMT, bool WHOLE>
static void decode_up_go(const DecodeArgs& a, hipStream_t stream) {
  // Four activation rows a tile instead of 16 (one 4-bit token of 8 experts, 4096
  // x 14336: 23.1 us, 24.2 us).
  if (a.tokens <= 4)
    decode_up_rows<FMT, WHOLE, 4>(a, stream);
  // Past 8 tokens, and past 4 entries an expert in the mean, the activations are
  // worth sharing (4-bit, 16 tokens, 4 choices among 8 experts of 4096 x 14336: narrow
  // 172 us for the layer, wide 158 us; 2 choices: no difference; 8 tokens of one
  // expert: 32 us, 35 us).
  else if (a.tokens <= 8 || (a.tokens <= 16 && a.tokens * a.topk <= 4 * decode_slots(a.tokens, a.topk, a.experts)))
    decode_up_rows<FMT, WHOLE, 16>(a, stream);
  // Most row tiles of a pass: fewer leave LDS for more workgroups (4-bit, 61 tokens, 5
  // choices among 60 experts of 544 x 4288: two 61 us, three 73 us), but a pass
  // more reads the weights again (64 tokens of 8 experts, 4096 x 14336, 16 entries
  // an expert: two 112 us, three 103 us, four 113 us; 8-bit, 4 choices: three 218
  // us, four 201 us).
  else if (few_each(a, 8))
    decode_up_wide<FMT, WHOLE, 2>(a, stream);
  else if (few_each(a, 16))
    decode_up_wide<FMT, WHOLE, 3>(a, stream);
  else
    decode_up_wide<FMT, WHOLE, 4>(a, stream);
}

template <int FMT, bool WHOLE>
static void decode_down_rows(const DecodeArgs& a, hipStream_t stream) {
  constexpr int waves = 8, tile = Walk<FMT, 1, 16, WHOLE, kDownAhead<FMT>>::kLds;
  hipLaunchKernelGGL((decode_down_kernel<FMT, WHOLE>), dim3(a.hidden / 16), dim3(64 * waves),
                     (size_t)waves * (a.tokens * 64 + tile), stream, a, tile);
}

template <int FMT, bool WHOLE>
static void decode_down_wide(DecodeArgs a, hipStream_t stream) {
  constexpr int NT = 2;
  const int chunks = (a.tokens + kDecodeTokenChunk - 1) / kDecodeTokenChunk;
  typedef WideWalk<FMT, NT, kDownTiles, WHOLE, 1> Wk;
  a.slots = decode_slots(a.tokens, a.topk, a.experts);
  hipLaunchKernelGGL((decode_down_wide_kernel<FMT, WHOLE, NT>),
                     dim3((a.hidden + 64 * NT - 1) / (64 * NT), a.slots * a.splits, chunks), dim3(256),
                     (size_t)(Wk::kShared + 4 * Wk::Wt::kLds), stream, a);
}

template <int FMT, bool WHOLE>
static void decode_down_go(const DecodeArgs& a, hipStream_t stream) {
  if (a.splits == 0) return decode_down_rows<FMT, WHOLE>(a, stream);
  decode_down_wide<FMT, WHOLE>(a, stream);
  hipLaunchKernelGGL(decode_sum_kernel, dim3((a.hidden / 4 + 63) / 64, a.tokens), dim3(256), 0, stream, a);
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

// Splits of the wide second product, 0 where the narrow one runs: for up to 16
// tokens that can name up to 16 experts (each expert is a stretch of its own of
// every wave there: 128 experts of 2048 x 768, 16 tokens: narrow 75 us for the
// layer, wide 66 us; 8 experts of 4096 x 14336, 1 token: narrow 38 us, wide 47 us),
// and where no expert is likely to have more than the 8 entries of a pass (for the
// layer, 4-bit, 16 tokens, 2 choices among 8: narrow 175 us, wide 153 us; 8-bit, 12
// tokens, 4 choices among 16 of 2048 x 4096: 87 us, 77 us; 8-bit, 7 tokens, 2
// choices among 8: 207 us, 213 us), unless its hidden / 16 workgroups are fewer than
// the compute units and have a long way each, slots * ffn values of k (16 bf16
// experts of 2048 x 5632, 16 tokens, narrow and wide for the layer: 146 and 133 us).
// The wide form adds a launch and its planes, which take longer the more hidden
// there is, so the way has two bounds, where 4-bit weights break even. One token,
// narrow and wide for the layer, 4 choices of 4 experts:
//   hidden 256:  way 16384, 4-bit 14.5 and 14.6 us, 8-bit 17.2 and 16.0, bf16 21.3
//     and 17.3; way 24576, 17.3 and 15.6, 21.9 and 17.1, 27.4 and 19.0 us
//   hidden 1024: way 24576 (24 hidden), 19.2 and 19.1, 27.4 and 24.1, 41.8 and 38.5
//     us; way 49152, 31.6 and 27.6, 48.4 and 39.8, 76.9 and 61.8 us
//   hidden 2048: way 49152 (24 hidden), 39.6 and 41.0, 63.4 and 64.4, 115 and 109
//     us; way 98304, 69.7 and 66.1, 119 and 108, 226 and 193 us
// Wider weights would go over earlier (bf16 from a way of about 12288 on: up to 28%
// at hidden 64 and 256, 14% above); past the bounds the worst is 4-bit at hidden
// 3584, way 98304, 97.8 and 104.0 us. About four workgroups a compute unit (for the layer, 4-bit, 40 tokens, 4
// choices among 16 experts of 2048 x 4096: four 65.8 us, six 70.6 us, eight 70.8 us;
// bf16, 24 tokens of 8, 4096 x 14336: 469, 477 and 484 us), at least 512 values of k
// each, and no more than 16 planes to add (one 8-bit expert of 2016 x 10432, 58
// tokens: 8 splits 34 us, 16 28 us, 20 41 us).
int decode_splits(int64_t tokens, int32_t topk, int32_t experts, int64_t hidden, int64_t ffn) {
  const int64_t slots = decode_slots((int)tokens, topk, experts);
  const bool long_way = hidden < 4096 && slots * ffn > std::max<int64_t>(16384, 24 * hidden);
  if (tokens <= 16 && slots <= 16 && (tokens <= 4 || tokens * topk <= 2 * slots) && !long_way) return 0;
  const int64_t groups = (hidden + 127) / 128 * ((tokens + kDecodeTokenChunk - 1) / kDecodeTokenChunk);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(16, ffn / 512), 1024 / (groups * slots)));
}

hipError_t launch_decode(int fmt, const DecodeArgs& a, hipStream_t stream) {
  if (fmt == WF_BF16) return decode_go<WF_BF16>(a, stream);
  if (fmt == WF_MXFP8) return decode_go<WF_MXFP8>(a, stream);
  return decode_go<WF_MXFP4>(a, stream);
}

}  // namespace mx
