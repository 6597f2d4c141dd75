// 8-bit integers with one scale per row: the cast, the (grouped) product on the
// integer matrix cores, and the ScaledSwiGLU between the two products of an MoE
// MLP. A row is a token on the left and an output channel on the right, so a
// result is one integer sum times two scales:
//     C[m, n] = sa[m] sb[n] sum_k A[m, k] B[n, k],
// and the sum is exact in 32 bits (k <= 131071: 2^14 k < 2^31), whatever its
// order. (GroupedLinear over split_sizes: "Efficient MoE training for biological
// foundation models", Key technical approaches items 1 and 3.)
#include <algorithm>

#include "mx_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

// ---- the cast

constexpr float kLeastTop = 0x1p-100f;       // a row's largest magnitude counts as at least this

// The integer nearest to the exact quotient 127 x / top, ties to even. t = x *
// (127 / top) is off by at most two half steps, 127 2^-23 < 2e-5, so it decides
// unless it lies that close to a half; there the sign of 127 x - half * top does:
// 127 x = p + e exactly, and p - half * top cancels to fewer than 24 bits.
__device__ __forceinline__ int nearest_code(float x, float top, float inv) {
  const float t = x * inv;
  float r = rintf(t);
  if (fabsf(t - r) > 0.5f - 2e-5f) {
    const float half = r + (t > r ? 0.5f : -0.5f);
    const float s = top > 1.f ? 0x1p-16f : 1.f;            // 127 x stays finite
    const float xs = x * s, p = 127.f * xs, e = fmaf(127.f, xs, -p);
    const float d = fmaf(-half, top * s, p) + e;
    r = d > 0.f ? half + 0.5f : d < 0.f ? half - 0.5f : rintf(half);
  }
  return (int)r;
}

// Eight values from p (bf16 or fp32) as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (F32) {
    const v4f* q = reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(p) + at);
    const v4f a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at);
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(d[i]);
      v[2 * i + 1] = bf16_hi(d[i]);
    }
  }
}

// L lanes a row (a wave, or the workgroup's four), C pieces of 8 values a lane in
// registers; C == 0: any number of pieces, read twice.
template <bool F32, int L, int C>
__global__ __launch_bounds__(256) void quantize_int8_kernel(QuantInt8Args a) {
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x % L;
  const int64_t r = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (r >= a.rows) return;                                 // a whole wave, or the whole workgroup
  const int64_t src = a.row_index != nullptr ? (int64_t)a.row_index[r] : r;
  const bool there = src >= 0 && src < a.index_rows;       // an index outside reads a row of zeros
  const int64_t base = there ? src * a.ldx : 0;
  const int pieces = there ? a.cols / 8 : 0;
  float v[C > 0 ? C : 1][8];
  uint32_t top = 0;
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
      if (lane + c * L < pieces) load8<F32>(a.x, base + (int64_t)(lane + c * L) * 8, v[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = umax(top, abs_bits(v[c][i]));
  } else {
    for (int c = lane; c < pieces; c += L) {
      load8<F32>(a.x, base + (int64_t)c * 8, v[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = umax(top, abs_bits(v[0][i]));
    }
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) top = umax(top, xor_u32(top, m));
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = umax(umax(tops[0], tops[1]), umax(tops[2], tops[3]));
  }
  // bit patterns of magnitudes: NaN and infinity are the largest, so either makes
  // the row's scale NaN or infinite
  const float amax = __uint_as_float(umax(top, __float_as_uint(kLeastTop)));
  const float inv = 127.f / amax;
  if (lane == 0) {
    const float s = amax / 127.f;
    a.s[r] = a.row_weight != nullptr ? s * a.row_weight[r] : s;
  }
  uint8_t* const q = reinterpret_cast<uint8_t*>(a.q) + r * a.cols;
  auto put = [&](int c, const float (&w)[8]) __attribute__((always_inline)) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo |= (uint32_t)(nearest_code(w[i], amax, inv) & 255) << (8 * i);
      hi |= (uint32_t)(nearest_code(w[4 + i], amax, inv) & 255) << (8 * i);
    }
    *reinterpret_cast<uint2*>(q + (int64_t)c * 8) = make_uint2(lo, hi);
  };
  const int all = a.cols / 8;
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (lane + c * L < all) put(lane + c * L, v[c]);
  } else {
    for (int c = lane; c < all; c += L) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[0][i] = 0.f;
      if (there) load8<F32>(a.x, base + (int64_t)c * 8, v[0]);
      put(c, v[0]);
    }
  }
}

// ---- the product

constexpr int kBK = 128;                     // k values of a step: one cache line of a row

// Where a workgroup's tile lies: its group, and the group's rows.
struct GroupSpan {
  int group, tile0, tiles;                   // tile0: the group's first m-tile
  int64_t row0;
  int rows;
};

// The group that holds m-tile `mt` of BM rows, from the rows of each group (held
// on the device, or in the arguments). A count below 0 reads as 0, and one that
// would take the running sum past M is cut there. Lanes hold two groups each;
// every wave finds the same. Returns false where all groups have fewer tiles.
__device__ __forceinline__ int64_t scan64(int64_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int64_t o = __shfl_up(v, m, 64);
    if ((int)(threadIdx.x & 63) >= m) v += o;
  }
  return v;
}
template <int BM>
__device__ __forceinline__ bool find_group(const Int8GemmArgs& a, int64_t mt, GroupSpan* g) {
  if (a.split == kInt8OneGroup) {
    *g = GroupSpan{0, 0, (int)(((int64_t)a.M + BM - 1) / BM), 0, a.M};
    return mt < g->tiles;
  }
  const int lane = threadIdx.x & 63;
  int64_t rows0 = 0, tiles0 = 0;
  bool found = false;
  for (int base = 0; base < a.groups; base += 64) {
    const int i = base + lane;
    int64_t c = 0;
    if (i < a.groups) c = a.split == kInt8DeviceSizes ? a.sizes_dev[i] : (int64_t)a.sizes[i];
    c = min(max(c, (int64_t)0), (int64_t)a.M);
    const int64_t end = rows0 + scan64(c);
    const int64_t first = min(end - c, (int64_t)a.M), last = min(end, (int64_t)a.M);
    const int64_t n = (last - first + BM - 1) / BM;
    const int64_t tend = tiles0 + scan64(n);
    const uint64_t here = __ballot(n > 0 && mt >= tend - n && mt < tend);
    if (here) {
      const int src = __ffsll((unsigned long long)here) - 1;
      g->group = base + src;
      g->tile0 = (int)__shfl(tend - n, src, 64);
      g->tiles = (int)__shfl(n, src, 64);
      g->row0 = __shfl(first, src, 64);
      g->rows = (int)__shfl(last - first, src, 64);
      found = true;
    }
    rows0 = __shfl(end, 63, 64);
    tiles0 = __shfl(tend, 63, 64);
  }
  return found;
}

// A tile of 32 MI WM rows of A by 32 NI WN rows of B on WM x WN waves. Both
// operands go straight to LDS (buffer loads with LDS as their target) one step of
// 128 k ahead of the products, in two stages that are separate objects, so that
// the compiler sees that a load into one never meets a read of the other. Chunk c
// (16 bytes) of row r lies at c ^ ((r >> 1) & 7), which frees the fragment reads
// of bank conflicts. Rows past the valid ones read as zeros by the bounds of the
// buffer resource; past the last k, B's chunks are sent out of bounds, and what A
// has there meets those zeros. Integers have no NaN that could survive this.
// The MFMA takes A first, so that a lane holds one column n and 16 rows m: stores
// of one register are whole runs of 32 columns.
// With the SwiGLU, 32-row blocks of the B tile alternate between gate and up rows.
template <int WM, int WN, int MI, int NI, int EPI>
__global__ __launch_bounds__(64 * WM * WN) void gemm_int8_kernel(Int8GemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int W = WM * WN, BM = 32 * MI * WM, BN = 32 * NI * WN;
  constexpr bool kPair = EPI == kInt8ToSwiglu;
  static_assert(!kPair || NI % 2 == 0, "gate and up blocks come in pairs");
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0 && W % 4 == 0, "whole blocks of 8 rows a wave");
  __shared__ __attribute__((aligned(16))) uint8_t sA0[BM * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sA1[BM * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sB0[BN * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sB1[BN * kBK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, h = lane >> 5, l32 = lane & 31;
  const int ntn = a.n_tiles;
  GroupSpan g;
  const int64_t id = blockIdx.x;
  if (!find_group<BM>(a, id / ntn, &g)) return;
  const int64_t local = id - (int64_t)g.tile0 * ntn;
  const int mt = (int)(local % g.tiles), nt = (int)(local / g.tiles);
  const int64_t row0 = g.row0 + (int64_t)mt * BM;
  const int rows = min(BM, g.rows - mt * BM);
  const int K = a.K, nk = (K + kBK - 1) / kBK;
  const int nrows = kPair ? a.N / 2 : a.N;                 // rows of B that n-tiles cover (gate rows)
  constexpr int kTileRows = kPair ? BN / 2 : BN;
  const int n0 = nt * kTileRows, ncols = min(kTileRows, nrows - n0);
  const int8_t* const bg = a.b + (int64_t)g.group * a.N * K;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.a + row0 * K, (int64_t)rows * K);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(bg + (int64_t)n0 * K, (int64_t)ncols * K);
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(bg + (int64_t)(nrows + n0) * K, kPair ? (int64_t)ncols * K : 0);
  const int lch = (lane & 7) ^ (lane >> 4) ^ (4 * (wave & 1));
  const uint32_t voff = (uint32_t)(lane >> 3) * K + lch * 16;
  auto load = [&](int kt, uint8_t* dA, uint8_t* dB) __attribute__((always_inline)) {
    const int k0 = kt * kBK;
    const uint32_t vb = k0 + lch * 16 < K ? voff : 0x80000000u;
#pragma unroll
    for (int it = 0; it < BM / 8 / W; ++it) {
      const int blk = it * W + wave;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(dA + blk * 1024), 16, voff, (uint32_t)(8 * blk) * K + k0, 0, 0);
    }
#pragma unroll
    for (int it = 0; it < BN / 8 / W; ++it) {
      const int blk = it * W + wave;
      if constexpr (kPair) {
        const int b32 = blk / 4, r0 = (b32 / 2) * 32 + (blk % 4) * 8;
        if (b32 & 1)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(ru, (lds_void*)(dB + blk * 1024), 16, vb, (uint32_t)r0 * K + k0, 0, 0);
        else
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(dB + blk * 1024), 16, vb, (uint32_t)r0 * K + k0, 0, 0);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(dB + blk * 1024), 16, vb, (uint32_t)(8 * blk) * K + k0, 0, 0);
      }
    }
  };
  v16i acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  auto frag = [&](const uint8_t* base, int r, int ks) __attribute__((always_inline)) -> v4i {
    return *reinterpret_cast<const v4i*>(base + r * kBK + (((2 * ks + h) ^ ((r >> 1) & 7)) << 4));
  };
  auto compute = [&](const uint8_t* sA, const uint8_t* sB) __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      v4i fa[MI], fb[NI];
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = frag(sA, 32 * (wm * MI + i) + l32, ks);
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[j] = frag(sB, 32 * (wn * NI + j) + l32, ks);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  };
  // The barrier says both that a stage is filled and that the other is free.
  auto step = [&](int kt, const uint8_t* cA, const uint8_t* cB, uint8_t* nA, uint8_t* nB) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __syncthreads();
    if (kt + 1 < nk) load(kt + 1, nA, nB);
    compute(cA, cB);
  };
  load(0, sA0, sB0);
  for (int kt = 0; kt < nk; kt += 2) {
    step(kt, sA0, sB0, sA1, sB1);
    if (kt + 1 < nk) step(kt + 1, sA1, sB1, sA0, sB0);
  }
  // results: column n of lane l32, rows 8 (v / 4) + 4 h + v % 4 of each 32
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int m = 32 * (wm * MI + i) + 8 * (v / 4) + 4 * h + v % 4;
      if (m >= rows) continue;
      const int64_t row = row0 + m;
      const float sa = a.a_s[row];
      if constexpr (kPair) {
#pragma unroll
        for (int j = 0; j < NI; j += 2) {
          const int n = n0 + 32 * ((wn * NI + j) / 2) + l32;
          if (n >= nrows) continue;
          const float* const bs = a.b_s + (int64_t)g.group * a.N + n;
          const float gate = (float)acc[i][j][v] * sa * bs[0], up = (float)acc[i][j + 1][v] * sa * bs[nrows];
          reinterpret_cast<float*>(a.c)[row * nrows + n] = gate / (1.f + __expf(-gate)) * up;
        }
      } else {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int n = n0 + 32 * (wn * NI + j) + l32;
          if (n >= nrows) continue;
          const float y = (float)acc[i][j][v] * sa * a.b_s[(int64_t)g.group * a.N + n];
          if constexpr (EPI == kInt8ToF32) reinterpret_cast<float*>(a.c)[row * a.N + n] = y;
          else reinterpret_cast<__bf16*>(a.c)[row * a.N + n] = (__bf16)y;
        }
      }
    }
  }
#endif
}

// As vgpr_hop, for the integer sums.
__device__ __forceinline__ int hop(int x) { return __builtin_amdgcn_mov_dpp(x, 0xE4, 0xF, 0xF, false); }

// The tile of 256 x 256 for many rows: four waves of 128 x 128, one a SIMD, so
// that the 256 sums of a lane have their registers. The stages and their swizzle
// are those of the kernel above; what differs is the order of things. A step of
// 128 k is four substeps of 32. In each, the fragments of the next substep are
// read while the products of this one run, and the last one begins with the
// barrier: by then every wave holds its last fragments of the stage, so the loads
// of the step after next go into it at once, and have nearly a whole step to
// land, while the first fragments of the next stage are read behind the last
// products of this one. So neither the barrier nor a fragment's latency leaves the
// matrix cores idle.
// The MFMA takes B first: a lane holds one row m and runs of 4 columns n, which
// go through LDS (16-byte chunk c of row r at c ^ (r & 15)) and leave as whole
// cache lines.
template <int EPI>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void gemm_int8_big_kernel(Int8GemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool kPair = EPI == kInt8ToSwiglu;
  constexpr int BM = 256, BN = 256;
  __shared__ __attribute__((aligned(16))) uint8_t sA0[BM * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sA1[BM * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sB0[BN * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sB1[BN * kBK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, l32 = lane & 31;
  const int ntn = a.n_tiles;
  GroupSpan g;
  const int64_t id = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  if (!find_group<BM>(a, id / ntn, &g)) return;
  const int local = (int)(id - (int64_t)g.tile0 * ntn);
  // bands of 8 m-tiles: the 32 tiles that run at once on one XCD are 8 x 4
  const int band = local / (8 * ntn), in_band = local - band * 8 * ntn, height = min(8, g.tiles - 8 * band);
  const int mt = 8 * band + in_band % height, nt = in_band / height;
  const int64_t row0 = g.row0 + (int64_t)mt * BM;
  const int rows = min(BM, g.rows - mt * BM);
  const int K = a.K, nk = __builtin_amdgcn_readfirstlane((K + kBK - 1) / kBK);
  const int nrows = kPair ? a.N / 2 : a.N;
  constexpr int kTileRows = kPair ? BN / 2 : BN;
  const int n0 = nt * kTileRows, ncols = min(kTileRows, nrows - n0);
  const int8_t* const bg = a.b + (int64_t)g.group * a.N * K;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.a + row0 * K, (int64_t)rows * K);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(bg + (int64_t)n0 * K, (int64_t)ncols * K);
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(bg + (int64_t)(nrows + n0) * K, kPair ? (int64_t)ncols * K : 0);
  const int lch = (lane & 7) ^ (lane >> 4) ^ (4 * (wave & 1));
  const uint32_t voff = (uint32_t)(lane >> 3) * K + lch * 16;
  // Block p of this wave's eight of A and of B of step kt. Steps past the last
  // are out of bounds for every lane: zeros, and no memory is read.
  auto load = [&](int kt, uint8_t* dA, uint8_t* dB, int p) __attribute__((always_inline)) {
    const int k0 = __builtin_amdgcn_readfirstlane(kt * kBK);
    const uint32_t vb = k0 + lch * 16 < K ? voff : 0x80000000u, va = k0 < K ? voff : 0x80000000u;
    const int blk = 4 * p + wave;
    const uint32_t so = (uint32_t)(8 * blk) * K + k0;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(dA + blk * 1024), 16, va, so, 0, 0);
    if constexpr (kPair) {
      const uint32_t sp = (uint32_t)((p / 2) * 32 + 8 * wave) * K + k0;    // 32-row block p: gate and up in turn
      if (p & 1)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ru, (lds_void*)(dB + blk * 1024), 16, vb, sp, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(dB + blk * 1024), 16, vb, sp, 0, 0);
    } else {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(dB + blk * 1024), 16, vb, so, 0, 0);
    }
  };
  v16i acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  v4i fa[2][4], fb[2][4];
  const int sw = (l32 >> 1) & 7;               // of every row 32 x + l32
  auto frag = [&](const uint8_t* base, int r32, int ks) __attribute__((always_inline)) -> v4i {
    return *reinterpret_cast<const v4i*>(base + (r32 * 32 + l32) * kBK + (((2 * ks + h) ^ sw) << 4));
  };
  // Step kt from stage (cA, cB); (nA, nB) holds step kt + 1. Half of a step's blocks
  // are loaded in the last substep of the step two before, half in the next one.
  auto step = [&](int kt, uint8_t* cA, uint8_t* cB, uint8_t* nA, uint8_t* nB) __attribute__((always_inline)) {
    static_for<0, 4>([&](auto ks_) __attribute__((always_inline)) {
      constexpr int ks = decltype(ks_)::value, cur = ks & 1, nxt = cur ^ 1;
      if constexpr (ks == 3) {
        __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
        __syncthreads();
      }
      static_for<0, 4>([&](auto i_) __attribute__((always_inline)) {
        constexpr int i = decltype(i_)::value;
        const uint8_t* const rA = ks == 3 ? nA : cA;
        const uint8_t* const rB = ks == 3 ? nB : cB;
        constexpr int ns = (ks + 1) & 3;
        if constexpr (i < 2) {
          fb[nxt][2 * i] = frag(rB, wn * 4 + 2 * i, ns);
          fb[nxt][2 * i + 1] = frag(rB, wn * 4 + 2 * i + 1, ns);
        } else {
          fa[nxt][2 * i - 4] = frag(rA, wm * 4 + 2 * i - 4, ns);
          fa[nxt][2 * i - 3] = frag(rA, wm * 4 + 2 * i - 3, ns);
        }
        if constexpr (ks == 3) load(kt + 2, cA, cB, i);
        if constexpr (ks == 0) load(kt + 1, nA, nB, 4 + i);
        static_for<0, 4>([&](auto j_) __attribute__((always_inline)) {
          constexpr int j = decltype(j_)::value;
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[cur][j], fa[cur][i], acc[i][j], 0, 0, 0);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  };
#pragma unroll
  for (int p = 0; p < 8; ++p) load(0, sA0, sB0, p);
#pragma unroll
  for (int p = 0; p < 4; ++p) load(1, sA1, sB1, p);
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    fb[0][x] = frag(sB0, wn * 4 + x, 0);
    fa[0][x] = frag(sA0, wm * 4 + x, 0);
  }
  int kt = 0;
  for (; kt + 1 < nk; kt += 2) {
    step(kt, sA0, sB0, sA1, sB1);
    step(kt + 1, sA1, sB1, sA0, sB0);
  }
  if (kt < nk) step(kt, sA0, sB0, sA1, sB1);
  // Sums to results. Lane: row 32 i + l32 of the wave's 128, columns 32 j + 8 q +
  // 4 h + 0 .. 3 of its 128; by 32 rows through the wave's own 16 KiB of LDS.
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
  __syncthreads();
  uint8_t* const stage = (wave == 0 ? sA0 : wave == 1 ? sA1 : wave == 2 ? sB0 : sB1);
  constexpr int kBytes = EPI == kInt8ToBf16 ? 2 : 4, kCols = kPair ? 64 : 128, kRowBytes = kCols * kBytes;
  constexpr int kChunks = kRowBytes / 16, kPer = 16 / kBytes;
  const int cn0 = n0 + wn * kCols;             // the wave's first column of C
  const int64_t ldc = nrows;
  const float* const bs = a.b_s + (int64_t)g.group * a.N;
  const bool whole = ldc % kPer == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m0 = wm * 128 + 32 * i;
    if (m0 >= rows) break;
    const float sa = a.a_s[row0 + min(m0 + l32, rows - 1)];
#pragma unroll
    for (int j = 0; j < 4; j += kPair ? 2 : 1) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = 32 * (kPair ? j / 2 : j) + 8 * q + 4 * h;
        float y[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int n = min(cn0 + col + v, nrows - 1);
          y[v] = (float)hop(acc[i][j][4 * q + v]) * sa * bs[n];
          if constexpr (kPair) {
            const float up = (float)hop(acc[i][j + 1][4 * q + v]) * sa * bs[nrows + n];
            y[v] = y[v] / (1.f + __expf(-y[v])) * up;
          }
        }
        const int chunk = col / kPer;
        uint8_t* const at = stage + l32 * kRowBytes + ((chunk ^ (l32 & (kChunks - 1) & 15)) << 4);
        if constexpr (kBytes == 4) {
          *reinterpret_cast<v4f*>(at) = v4f{y[0], y[1], y[2], y[3]};
        } else {
          typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<bf16x4*>(at + 8 * h) = bf16x4{(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
        }
      }
    }
    // the wave's own LDS: its writes are done before its reads (no barrier)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    if (whole) {
#pragma unroll
      for (int u = 0; u < 32 * kChunks / 64; ++u) {
        const int r = (u * 64 + lane) / kChunks, c = (u * 64 + lane) % kChunks, n = cn0 + c * kPer;
        const uint4 w = *reinterpret_cast<const uint4*>(stage + r * kRowBytes + ((c ^ (r & (kChunks - 1) & 15)) << 4));
        if (m0 + r < rows && n < nrows)
          *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.c) + ((row0 + m0 + r) * ldc + n) * kBytes) = w;
      }
    } else {
      for (int u = lane; u < 32 * kCols; u += 64) {
        const int r = u / kCols, c = u % kCols, n = cn0 + c;
        const uint8_t* const from = stage + r * kRowBytes + (((c / kPer) ^ (r & (kChunks - 1) & 15)) << 4) + c % kPer * kBytes;
        if (m0 + r < rows && n < nrows) {
          const int64_t at = (row0 + m0 + r) * ldc + n;
          if constexpr (kBytes == 4) reinterpret_cast<float*>(a.c)[at] = *reinterpret_cast<const float*>(from);
          else reinterpret_cast<uint16_t*>(a.c)[at] = *reinterpret_cast<const uint16_t*>(from);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
#endif
}

template <int WM, int WN, int MI, int NI>
struct Shape {
  static constexpr int kWM = WM, kWN = WN, kMI = MI, kNI = NI, kBM = 32 * MI * WM, kBN = 32 * NI * WN;
};
template <typename Go>
auto by_shape(int shape, const Go& go) {
  switch (shape) {
    case 0: return go(Shape<1, 4, 1, 2>{});
    case 1: return go(Shape<2, 2, 1, 2>{});
    default: return go(Shape<2, 2, 4, 4>{});
  }
}

}  // namespace

hipError_t launch_quantize_int8(const QuantInt8Args& a, hipStream_t stream) {
  const auto go = [&](auto f32_, auto l_, auto c_) {
    constexpr bool F32 = decltype(f32_)::value;
    constexpr int L = decltype(l_)::value, C = decltype(c_)::value;
    const dim3 grid((unsigned)((a.rows + 256 / L - 1) / (256 / L)));
    hipLaunchKernelGGL((quantize_int8_kernel<F32, L, C>), grid, dim3(256), 0, stream, a);
  };
  const auto by_size = [&](auto f32) {
    using std::integral_constant;
    if (a.cols <= 64 * 8) go(f32, integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (a.cols <= 64 * 8 * 4) go(f32, integral_constant<int, 64>{}, integral_constant<int, 4>{});
    else if (a.cols <= 256 * 8 * 2) go(f32, integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (a.cols <= 256 * 8 * 8) go(f32, integral_constant<int, 256>{}, integral_constant<int, 8>{});
    else go(f32, integral_constant<int, 256>{}, integral_constant<int, 0>{});
  };
  if (a.f32) by_size(std::true_type{});
  else by_size(std::false_type{});
  return hipGetLastError();
}

Int8Plan plan_gemm_int8(int result, const Int8GemmArgs& a) {
  Int8Plan p;
  const int64_t per = ((int64_t)a.M + a.groups - 1) / a.groups;        // rows of a group in the mean
  const int64_t big = (((int64_t)a.M + 255) / 256) * (((int64_t)a.N + 255) / 256);
  p.shape = per <= 32 ? 0 : per <= 128 || big < 128 ? 1 : 2;
  by_shape(p.shape, [&](auto s) {
    constexpr int BM = decltype(s)::kBM, BN = decltype(s)::kBN;
    const int64_t cols = result == kInt8ToSwiglu ? a.N / 2 : a.N, bn = result == kInt8ToSwiglu ? BN / 2 : BN;
    int64_t mtiles = 0;
    if (a.split == kInt8HostSizes) {
      for (int g = 0; g < a.groups; ++g) mtiles += ((int64_t)a.sizes[g] + BM - 1) / BM;
    } else {
      const int64_t some = std::min<int64_t>(a.split == kInt8OneGroup ? 1 : a.groups, a.M);
      mtiles = (a.M + (BM - 1) * some) / BM;               // the most that any split can have
    }
    p.n_tiles = (cols + bn - 1) / bn;
    p.tiles = mtiles * p.n_tiles;
    return 0;
  });
  return p;
}

hipError_t launch_gemm_int8(int result, const Int8GemmArgs& args, const Int8Plan& p, hipStream_t stream) {
  Int8GemmArgs a = args;
  a.n_tiles = (int32_t)p.n_tiles;
  if (p.tiles == 0) return hipSuccess;
  by_shape(p.shape, [&](auto s) {
    using S = decltype(s);
    constexpr int WM = S::kWM, WN = S::kWN, MI = S::kMI, NI = S::kNI;
    const dim3 grid((unsigned)p.tiles), block(64 * WM * WN);
    if constexpr (S::kBM == 256) {
      if (result == kInt8ToBf16)
        hipLaunchKernelGGL((gemm_int8_big_kernel<kInt8ToBf16>), grid, block, 0, stream, a);
      else if (result == kInt8ToF32)
        hipLaunchKernelGGL((gemm_int8_big_kernel<kInt8ToF32>), grid, block, 0, stream, a);
      else
        hipLaunchKernelGGL((gemm_int8_big_kernel<kInt8ToSwiglu>), grid, block, 0, stream, a);
    } else if (result == kInt8ToBf16)
      hipLaunchKernelGGL((gemm_int8_kernel<WM, WN, MI, NI, kInt8ToBf16>), grid, block, 0, stream, a);
    else if (result == kInt8ToF32)
      hipLaunchKernelGGL((gemm_int8_kernel<WM, WN, MI, NI, kInt8ToF32>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((gemm_int8_kernel<WM, WN, MI, NI, kInt8ToSwiglu>), grid, block, 0, stream, a);
    return 0;
  });
  return hipGetLastError();
}

}  // namespace mx
