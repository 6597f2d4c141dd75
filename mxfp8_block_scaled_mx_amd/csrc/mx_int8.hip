// 8-bit integers with one scale per row: the cast, the (grouped) product on the
// integer matrix cores, and the ScaledSwiGLU between the two products of an MoE
// MLP. A row is a token on the left and an output channel on the right, so a
// result is one integer sum times two scales:
//     C[m, n] = sa[m] sb[n] sum_k A[m, k] B[n, k],
// and the sum is exact in 32 bits (k <= 131071: 2^14 k < 2^31), whatever its
// order. (GroupedLinear over split_sizes: "Efficient MoE training for biological
// foundation models", Key technical approaches items 1 and 3.)
#include <algorithm>
#include <cmath>

#include "mx_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

// ---- the cast

constexpr float kLeastTop = 0x1p-100f;       // a row's largest magnitude counts as at least this

// The integer nearest to the exact quotient 127 x / top, ties to even, where x *
// (127 / top) lies close to a half: there the sign of 127 x - half * top decides.
// 127 x = p + e exactly, and p - half * top cancels to fewer than 24 bits.
__device__ __forceinline__ float code_beside_half(float x, float top, float inv) {
  const float t = x * inv, r = rintf(t);
  if (!(fabsf(t - r) > 0.5f - 2e-5f)) return r;
  const float half = r + (t > r ? 0.5f : -0.5f);
  const float s = top > 1.f ? 0x1p-16f : 1.f;              // 127 x stays finite
  const float xs = x * s, p = 127.f * xs, e = fmaf(127.f, xs, -p);
  const float d = fmaf(-half, top * s, p) + e;
  return d > 0.f ? half + 0.5f : d < 0.f ? half - 0.5f : rintf(half);
}

// Eight values as they lie in memory.
template <bool F32>
struct Eight;
template <>
struct Eight<true> {
  v4f d[2];
  __device__ __forceinline__ float operator[](int i) const { return d[i / 4][i % 4]; }
};
template <>
struct Eight<false> {
  u32x4 d;
  __device__ __forceinline__ float operator[](int i) const { return i % 2 ? bf16_hi(d[i / 2]) : bf16_lo(d[i / 2]); }
};

// Eight values to codes, packed. The code is the sum with 1.5 2^23 rounded to an
// integer, its low byte. x * inv, inv off by half a step, is off by less than 127
// 2^-24 < 8e-6, so that decides unless one of the eight lies within 2e-5 of a half.
template <bool F32>
__device__ __forceinline__ uint2 eight_codes(const Eight<F32>& w, float top, float inv) {
  constexpr float kShift = 0x1.8p23f;
  float m[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = fmaf(w[i], inv, kShift);
    far = fmaxf(far, fabsf(fmaf(w[i], inv, kShift - m[i])));
  }
  if (far > 0.5f - 2e-5f)
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = kShift + code_beside_half(w[i], top, inv);
  const auto four = [&](int i) __attribute__((always_inline)) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(m[i + 1]), __float_as_uint(m[i]), 0x0C0C0400);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(m[i + 3]), __float_as_uint(m[i + 2]), 0x0C0C0400);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100);
  };
  return make_uint2(four(0), four(4));
}

// L lanes a row (a wave, or the workgroup's four), C pieces of 8 values a lane in
// registers as they were read, so that memory is passed over once; C == 0: any
// number of pieces, read twice. Bound by memory, inputs that no cache holds: 16384 x
// 4096 bf16 in 36 us, 5.6 TB/s read and written (32 us gathered from 8192 rows), 8192 x
// 14336 bf16 in 67.5, 5.2, fp32 in 107, 5.5, where a copy reaches 5.95. With a branch
// per value for those beside a half 38, 34 (gathered), 79 and 112 us.
template <bool F32, int L, int C>
__global__ __launch_bounds__(256) void quantize_int8_kernel(QuantInt8Args a) {
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x % L;
  const int64_t r = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (r >= a.rows) return;                                 // a whole wave, or the whole workgroup
  const int64_t src = a.row_index != nullptr ? (int64_t)a.row_index[r] : r;
  const bool there = src >= 0 && src < a.index_rows;       // an index outside reads a row of zeros
  const auto* const x = reinterpret_cast<const std::conditional_t<F32, float, uint16_t>*>(a.x) + (there ? src * a.ldx : 0);
  const int all = a.cols / 8, pieces = there ? all : 0;
  const auto load = [&](int c) __attribute__((always_inline)) {
    Eight<F32> w;
    if constexpr (F32) {
      w.d[0] = c < pieces ? *reinterpret_cast<const v4f*>(x + (int64_t)c * 8) : v4f{};
      w.d[1] = c < pieces ? *reinterpret_cast<const v4f*>(x + (int64_t)c * 8 + 4) : v4f{};
    } else {
      w.d = c < pieces ? *reinterpret_cast<const u32x4*>(x + (int64_t)c * 8) : u32x4{};
    }
    return w;
  };
  Eight<F32> v[C > 0 ? C : 1];
  uint32_t top = 0;
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = load(lane + c * L);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = umax(top, abs_bits(v[c][i]));
  } else {
    for (int c = lane; c < pieces; c += L) {
      v[0] = load(c);
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
  // the row's scale NaN or infinite (and its codes what they may)
  const float amax = __uint_as_float(umax(top, __float_as_uint(kLeastTop)));
  const float inv = 127.f / amax;
  if (lane == 0) {
    const float s = amax / 127.f;
    a.s[r] = a.row_weight != nullptr ? s * a.row_weight[r] : s;
  }
  int8_t* const q = a.q + r * a.cols;
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (lane + c * L < all) *reinterpret_cast<uint2*>(q + (lane + c * L) * 8) = eight_codes<F32>(v[c], amax, inv);
  } else {
    for (int c = lane; c < all; c += L) *reinterpret_cast<uint2*>(q + (int64_t)c * 8) = eight_codes<F32>(load(c), amax, inv);
  }
}

// ---- the product

constexpr int kBK = 128;                     // k values of a step: one cache line of a row

// Where a workgroup's tile lies: its group, and the group's rows and m-tiles.
struct GroupSpan {
  int group, tile0, tiles;                   // tile0: the group's first m-tile
  int64_t row0;
  int rows;
};

// The groups in m-tiles of BM rows, from the rows of each group (held on the
// device, or in the arguments), two groups a lane; every wave makes the same. A
// count below 0 reads as 0, and one that would take the running sum past M is cut
// there.
struct GroupScan {
  int first[2], rows[2], tend[2], tiles[2];  // of lane's groups: first row, rows, m-tiles up to its end, its own
  int total;                                 // m-tiles of all groups
};
// Sums over the lanes up to each lane, cut at `most` (no sum of two below 2^31
// passes 2^32, and cutting every partial sum cuts the whole): within rows of 16
// lanes, then each row's last on to the next, then lane 31's to the upper half.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t add_from(uint32_t v, uint32_t most) {
  const uint32_t s = v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  return s < most ? s : most;
}
__device__ __forceinline__ uint32_t scan_cut(uint32_t v, uint32_t most) {
  v = add_from<0x111, 0xF>(v, most);           // row_shr 1, 2, 4, 8
  v = add_from<0x112, 0xF>(v, most);
  v = add_from<0x114, 0xF>(v, most);
  v = add_from<0x118, 0xF>(v, most);
  v = add_from<0x142, 0xA>(v, most);           // row_bcast 15 into rows 1 and 3
  return add_from<0x143, 0xC>(v, most);        // row_bcast 31 into rows 2 and 3
}
template <int BM>
__device__ __forceinline__ void scan_groups(const Int8GemmArgs& a, GroupScan* s) {
  if (a.split == kInt8OneGroup) {
    s->total = (int)(((int64_t)a.M + BM - 1) / BM);
    return;
  }
  const int lane = threadIdx.x & 63;
  const uint32_t M = (uint32_t)a.M;
  uint32_t rows0 = 0, tiles0 = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    s->rows[u] = s->tiles[u] = s->first[u] = s->tend[u] = 0;
    if (64 * u >= a.groups) break;             // (uniform)
    const int i = 64 * u + lane;
    int64_t c = 0;
    if (i < a.groups) c = a.split == kInt8DeviceSizes ? a.sizes_dev[i] : (int64_t)a.sizes[i];
    const uint32_t mine = (uint32_t)min(max(c, (int64_t)0), (int64_t)M);
    const uint32_t upto = scan_cut(mine, M), end = min(rows0 + upto, M);
    // the rows before: what the lane below has come to
    const uint32_t below = (uint32_t)__shfl_up((int)end, 1, 64), from = lane == 0 ? rows0 : below;
    s->first[u] = (int)from;
    s->rows[u] = (int)(end - from);
    s->tiles[u] = (int)((end - from + BM - 1) / BM);
    s->tend[u] = (int)(tiles0 + scan_cut((uint32_t)s->tiles[u], 0x7FFFFFFFu));
    rows0 = (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
    tiles0 = (uint32_t)__builtin_amdgcn_readlane(s->tend[u], 63);
  }
  s->total = (int)tiles0;
}
// The group that holds m-tile mt < total.
template <int BM>
__device__ __forceinline__ GroupSpan group_of(const Int8GemmArgs& a, const GroupScan& s, int mt) {
  if (a.split == kInt8OneGroup) return GroupSpan{0, 0, s.total, 0, a.M};
  GroupSpan g = {};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint64_t here = __ballot(mt >= s.tend[u] - s.tiles[u] && mt < s.tend[u]);
    if (here) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)here) - 1);
      g.group = 64 * u + src;
      g.tiles = __builtin_amdgcn_readlane(s.tiles[u], src);
      g.tile0 = __builtin_amdgcn_readlane(s.tend[u], src) - g.tiles;
      g.row0 = __builtin_amdgcn_readlane(s.first[u], src);
      g.rows = __builtin_amdgcn_readlane(s.rows[u], src);
    }
  }
  return g;
}

// Workgroup b of `total` runs on XCD b % 8. In rounds of 8 x CHUNK every XCD takes
// CHUNK consecutive ids, and of what is left an eighth: ids that share rows share
// an L2.
template <int CHUNK>
__device__ __forceinline__ int xcd_ids(int b, int total) {
  const int xcd = b & 7, l = b >> 3, full = total / (8 * CHUNK), rest = total - full * 8 * CHUNK;
  if (l < full * CHUNK) return (l / CHUNK) * 8 * CHUNK + xcd * CHUNK + l % CHUNK;
  return full * 8 * CHUNK + xcd * (rest / 8) + min(xcd, rest % 8) + (l - full * CHUNK);
}

// A group's tile `local`, in bands of 8 m-tiles: the 32 tiles that run at once on
// one XCD are 8 x 4.
__device__ __forceinline__ void tile_of(int local, int ntn, int mtiles, int* mt, int* nt) {
  const int band = local / (8 * ntn), in_band = local - band * 8 * ntn, height = min(8, mtiles - 8 * band);
  *mt = 8 * band + in_band % height;
  *nt = in_band / height;
}

// Tiles of 256 x 256 run 256 at a time, one a compute unit. Those of the last,
// partial round (from id `first` on) are `parts` workgroups each, that share out
// k, where that saves more than the sums' way through memory costs (a step takes
// 1.45 us, a tile of sums 0.12 us to write and read, their join 8 us).
constexpr int kTailUnits = 256;
struct Tail {
  int first, parts;
};
__host__ __device__ inline Tail tail_of(int64_t tiles, int steps) {
  const int n = (int)(tiles % kTailUnits);
  if (n == 0 || tiles < kTailUnits) return Tail{(int)tiles, 1};
  const int parts = kTailUnits / n < steps / 4 ? kTailUnits / n : steps / 4;
  if (parts < 2 || 1.45f * (steps - (steps + parts - 1) / parts) < 8.f + 0.12f * n * parts) return Tail{(int)tiles, 1};
  return Tail{(int)tiles - n, parts};
}

// silu(g) u, as the block-scaled products' epilogues form it. The argument of the
// hardware's power of two is rounded, so e^-g is off by up to 1.23 |g| + 2 half steps
// of fp32, which all of silu(g) is for g < 0; sum, reciprocal (two) and product add
// 4: measured 3 for |g| < 1 and for every g > 0, 6.5 at -5, 10 at -10, 18 at -20. Below
// -87.3, where silu is under 2^-119, it is 0.
__device__ __forceinline__ float swiglu(float g, float u) { return g * __builtin_amdgcn_rcpf(1.f + __expf(-g)) * u; }

// As vgpr_hop, for the integer sums.
__device__ __forceinline__ int hop(int x) { return __builtin_amdgcn_mov_dpp(x, 0xE4, 0xF, 0xF, false); }

// s_waitcnt immediates: vmcnt(n), as kWaitVmcnt0; and with it lgkmcnt(0).
constexpr int wait_vmcnt(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int wait_vmcnt_lds(int n) { return 0x0070 | (n & 15) | ((n >> 4) << 14); }

// The barrier alone. (__syncthreads() would wait for every load in flight first,
// those for LDS among them.) What a wave has read of LDS before has to be in its
// registers, and what it has loaded for the others has to have landed: the caller
// waits for both.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// A tile of 64 TI rows of A by 64 NI rows of B on four waves, 2 x 2. Both operands
// go straight to LDS (buffer loads with LDS as their target), in S stages of 128 k
// that are separate objects, so that the compiler sees that a load into one never
// meets a read of another. Chunk c (16 bytes) of row r lies at c ^ ((r >> 1) & 7),
// which frees the fragment reads of bank conflicts. Rows past the valid ones read
// as zeros by the bounds of the buffer resource; past the last k, B's chunks are
// sent out of bounds, and what A has there meets those zeros. Integers have no NaN
// that could survive this.
//
// A step of 128 k is four substeps of 32. In each, the fragments of the next
// substep are read while the products of this one run, and the last one begins
// with the barrier: by then every wave holds its last fragments of the stage, so
// the loads of S steps on go into it at once (half then, half in the next
// substep), and have S - 1 steps to land, while the first fragments of the next
// stage are read behind the last products of this one. So neither the barrier nor
// a fragment's latency leaves the matrix cores idle.
// The MFMA takes B first: a lane holds one row m and runs of 4 columns n, which
// go through LDS (16-byte chunk c of row r at c ^ (r & 15)) and leave as whole
// cache lines.
// With the SwiGLU, 32-row blocks of the B tile alternate between gate and up rows.
// With parts > 1 each tile is several workgroups, each with its share of the
// steps, that leave the sums themselves, in 32 bits, to planes of their own.
//
// 256 x 256 tiles, 8191 x 4096 x 14336: 375 to 385 us, 2.5 to 2.6 POP/s, where a large
// library product of the same format reaches 2.4. The matrix cores are busy 68 to 73%
// of the cycles, no read of LDS meets a bank conflict, and the clock falls to 1.7 GHz
// under this load (all zeros, which draw less power, take 281 us): power bounds it.
// 8192 rows of 8 unlike groups by 28672 x 4096: 920 us, 2.1 POP/s (the library on one
// group: 2.1). Some 6% of it are rows that tiles have too many; k is shorter, so each
// tile's first loads and its results, which nothing hides, weigh more.
template <int TI, int NI, int S, int EPI, bool TAIL>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(64 * (TI + NI) * kBK * S <= 81920 ? 2 : 1)))
void gemm_int8_kernel(Int8GemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool kPair = EPI == kInt8ToSwiglu;
  static_assert(!kPair || NI % 2 == 0, "gate and up blocks come in pairs");
  static_assert(S >= 2 && S <= 4, "stages");
  constexpr int BM = 64 * TI, BN = 64 * NI;
  __shared__ __attribute__((aligned(16))) uint8_t sA0[BM * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sB0[BN * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sA1[BM * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sB1[BN * kBK];
  __shared__ __attribute__((aligned(16))) uint8_t sA2[S > 2 ? BM * kBK : 16];
  __shared__ __attribute__((aligned(16))) uint8_t sB2[S > 2 ? BN * kBK : 16];
  __shared__ __attribute__((aligned(16))) uint8_t sA3[S > 3 ? BM * kBK : 16];
  __shared__ __attribute__((aligned(16))) uint8_t sB3[S > 3 ? BN * kBK : 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, l32 = lane & 31;
  const int ntn = a.n_tiles;
  GroupScan scan;
  scan_groups<BM>(a, &scan);
  const int K = a.K, all_steps = (K + kBK - 1) / kBK;
  // a part's tiles are consecutive; the grid is sized for the worst split
  const int tiles = scan.total * ntn;
  const Tail tail = TAIL ? tail_of(tiles, all_steps) : Tail{tiles, 1};
  const int whole_ids = TAIL ? tail.first : tiles * a.parts;
  int part, parts = a.parts, id, unit = -1;
  if (!TAIL || (int)blockIdx.x < whole_ids) {
    if ((int)blockIdx.x >= whole_ids) return;
    const int place = xcd_ids<TI * NI >= 16 ? 32 : 64>((int)blockIdx.x, whole_ids);
    part = place / (TAIL ? whole_ids : tiles);
    id = place - part * tiles;
  } else {
    const int n = tiles - tail.first, u = (int)blockIdx.x - tail.first;
    if (u >= n * tail.parts) return;
    const int place = xcd_ids<32>(u, n * tail.parts);
    part = place / n;
    id = tail.first + place - part * n;
    parts = tail.parts;
    unit = parts > 1 ? place : -1;
  }
  const GroupSpan g = group_of<BM>(a, scan, id / ntn);
  int mt, nt;
  tile_of(id - g.tile0 * ntn, ntn, g.tiles, &mt, &nt);
  const int64_t row0 = g.row0 + (int64_t)mt * BM;
  const int rows = min(BM, g.rows - mt * BM);
  const int first = __builtin_amdgcn_readfirstlane((int)((int64_t)all_steps * part / parts));
  const int nk = __builtin_amdgcn_readfirstlane((int)((int64_t)all_steps * (part + 1) / parts)) - first;
  const int nrows = kPair ? a.N / 2 : a.N;                 // rows of B that n-tiles cover (gate rows)
  constexpr int kTileRows = kPair ? BN / 2 : BN;
  const int n0 = nt * kTileRows, ncols = min(kTileRows, nrows - n0);
  const int8_t* const bg = a.b + (int64_t)g.group * a.N * K;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.a + row0 * K, (int64_t)rows * K);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(bg + (int64_t)n0 * K, (int64_t)ncols * K);
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(bg + (int64_t)(nrows + n0) * K, kPair ? (int64_t)ncols * K : 0);
  const int lch = (lane & 7) ^ (lane >> 4) ^ (4 * (wave & 1));
  const uint32_t voff = (uint32_t)(lane >> 3) * K + lch * 16;
  // Rows whose distance is a power of two lie on the same memory channels, so
  // workgroups that walk along k together would meet there: they begin at other
  // places. Those of an XCD that share rows keep step (for the L2's sake).
  const int rot = __builtin_amdgcn_readfirstlane(nk * (int)(blockIdx.x & 7) / 8);
  auto run = [&](auto mi_) __attribute__((always_inline)) {
    constexpr int MI = decltype(mi_)::value, kLoads = 2 * (MI + NI);
    // Load p of this wave's kLoads of step kt (8 rows each: A's, then B's). Steps
    // past the last are out of bounds for every lane: zeros, and no memory is read.
    auto load = [&](int kt, uint8_t* dA, uint8_t* dB, int p) __attribute__((always_inline)) {
      const int s = kt + rot < nk ? kt + rot : kt + rot - nk;
      const int k0 = __builtin_amdgcn_readfirstlane(kt < nk ? (first + s) * kBK : K);
      if (p < 2 * MI) {
        const int blk = 4 * p + wave;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(dA + blk * 1024), 16, k0 < K ? voff : 0x80000000u,
                                                 (uint32_t)(8 * blk) * K + k0, 0, 0);
      } else {
        const int q = p - 2 * MI, blk = 4 * q + wave;
        const uint32_t vb = k0 + lch * 16 < K ? voff : 0x80000000u;
        if constexpr (kPair) {
          const uint32_t so = (uint32_t)((q / 2) * 32 + 8 * wave) * K + k0;  // 32-row block q: gate and up in turn
          if (q & 1)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ru, (lds_void*)(dB + blk * 1024), 16, vb, so, 0, 0);
          else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(dB + blk * 1024), 16, vb, so, 0, 0);
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
    v4i fa[2][MI], fb[2][NI];
    const int sw = (l32 >> 1) & 7;               // of every row 32 x + l32
    auto frag = [&](const uint8_t* base, int r32, int ks) __attribute__((always_inline)) -> v4i {
      return *reinterpret_cast<const v4i*>(base + (r32 * 32 + l32) * kBK + (((2 * ks + h) ^ sw) << 4));
    };
    // Step kt from stage (cA, cB); (nA, nB) holds step kt + 1, and the loads of step
    // kt - 1 + S, half of which are out, go to (pA, pB).
    auto step = [&](int kt, uint8_t* cA, uint8_t* cB, uint8_t* nA, uint8_t* nB, uint8_t* pA, uint8_t* pB)
        __attribute__((always_inline)) {
      static_for<0, 4>([&](auto ks_) __attribute__((always_inline)) {
        constexpr int ks = decltype(ks_)::value, cur = ks & 1, nxt = cur ^ 1, ns = (ks + 1) & 3;
        if constexpr (ks == 3) {
          __builtin_amdgcn_s_waitcnt(wait_vmcnt_lds((S - 2) * kLoads));
          bare_barrier();
        }
        const uint8_t* const rA = ks == 3 ? nA : cA;
        const uint8_t* const rB = ks == 3 ? nB : cB;
        static_for<0, MI>([&](auto i_) __attribute__((always_inline)) {
          constexpr int i = decltype(i_)::value;
          // half a step's loads, and fragments of which B's come first, dealt out to the row blocks
          static_for<0, MI + NI>([&](auto f_) __attribute__((always_inline)) {
            constexpr int f = decltype(f_)::value;
            if constexpr (f * MI / (MI + NI) == i) {
              if constexpr (f < NI) fb[nxt][f] = frag(rB, wn * NI + f, ns);
              else fa[nxt][f - NI] = frag(rA, wm * MI + f - NI, ns);
            }
          });
          static_for<0, MI + NI>([&](auto f_) __attribute__((always_inline)) {
            constexpr int f = decltype(f_)::value;
            if constexpr (f * MI / (MI + NI) == i) {
              if constexpr (ks == 3) load(kt + S, cA, cB, f);
              if constexpr (ks == 0) load(kt - 1 + S, pA, pB, MI + NI + f);
            }
          });
          static_for<0, NI>([&](auto j_) __attribute__((always_inline)) {
            constexpr int j = decltype(j_)::value;
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[cur][j], fa[cur][i], acc[i][j], 0, 0, 0);
          });
          __builtin_amdgcn_sched_barrier(0);
        });
      });
    };
    auto fill = [&](int kt, uint8_t* dA, uint8_t* dB, int n) __attribute__((always_inline)) {
  #pragma unroll
      for (int p = 0; p < n; ++p) load(kt, dA, dB, p);
    };
    fill(0, sA0, sB0, kLoads);
    if constexpr (S > 2) fill(1, sA1, sB1, kLoads);
    if constexpr (S > 3) fill(2, sA2, sB2, kLoads);
    fill(S - 1, S == 2 ? sA1 : S == 3 ? sA2 : sA3, S == 2 ? sB1 : S == 3 ? sB2 : sB3, MI + NI);
    __builtin_amdgcn_s_waitcnt(wait_vmcnt((S - 2) * kLoads + MI + NI));      // step 0 has landed
    bare_barrier();
  #pragma unroll
    for (int x = 0; x < NI; ++x) fb[0][x] = frag(sB0, wn * NI + x, 0);
  #pragma unroll
    for (int x = 0; x < MI; ++x) fa[0][x] = frag(sA0, wm * MI + x, 0);
    int kt = 0;
    if constexpr (S == 4) {
      for (; kt + 3 < nk; kt += 4) {
        step(kt, sA0, sB0, sA1, sB1, sA3, sB3);
        step(kt + 1, sA1, sB1, sA2, sB2, sA0, sB0);
        step(kt + 2, sA2, sB2, sA3, sB3, sA1, sB1);
        step(kt + 3, sA3, sB3, sA0, sB0, sA2, sB2);
      }
      if (kt < nk) {
        step(kt, sA0, sB0, sA1, sB1, sA3, sB3);
        if (kt + 1 < nk) {
          step(kt + 1, sA1, sB1, sA2, sB2, sA0, sB0);
          if (kt + 2 < nk) step(kt + 2, sA2, sB2, sA3, sB3, sA1, sB1);
        }
      }
    } else if constexpr (S == 3) {
      for (; kt + 2 < nk; kt += 3) {
        step(kt, sA0, sB0, sA1, sB1, sA2, sB2);
        step(kt + 1, sA1, sB1, sA2, sB2, sA0, sB0);
        step(kt + 2, sA2, sB2, sA0, sB0, sA1, sB1);
      }
      if (kt < nk) {
        step(kt, sA0, sB0, sA1, sB1, sA2, sB2);
        if (kt + 1 < nk) step(kt + 1, sA1, sB1, sA2, sB2, sA0, sB0);
      }
    } else {
      for (; kt + 1 < nk; kt += 2) {
        step(kt, sA0, sB0, sA1, sB1, sA1, sB1);
        step(kt + 1, sA1, sB1, sA0, sB0, sA0, sB0);
      }
      if (kt < nk) step(kt, sA0, sB0, sA1, sB1, sA1, sB1);
    }
    // Sums to results. Lane: row 32 i + l32 of the wave's rows, columns 32 j + 8 q +
    // 4 h + 0 .. 3 of its columns; by 32 rows through LDS of the wave's own.
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
    __syncthreads();
    uint8_t* const stage = wave == 0 ? sA0 : wave == 1 ? sA1 : wave == 2 ? sB0 : sB1;
    auto finish = [&](auto epi_, uint8_t* c, int64_t ldc, int64_t crow0, int cn0, int crows, int ccols)
        __attribute__((always_inline)) {
      constexpr int E = decltype(epi_)::value;
      constexpr bool kTwo = E == kInt8ToSwiglu;
      constexpr int kBytes = E == kInt8ToBf16 ? 2 : 4, kCols = (kTwo ? 16 : 32) * NI, kRowBytes = kCols * kBytes;
      constexpr int kChunks = kRowBytes / 16, kPer = 16 / kBytes, kMask = kChunks < 16 ? kChunks - 1 : 15;
      static_assert(32 * kRowBytes <= BM * kBK && 32 * kRowBytes <= BN * kBK, "32 rows of results fit one stage of one operand");
      cn0 += wn * kCols;                         // the wave's first column
      const bool whole = ldc % kPer == 0 && (reinterpret_cast<uintptr_t>(c) & 15) == 0;
      // the lane's column scales, 4 at a time (0 past the last), and its rows'
      v4f sb[NI][4];
      float sa[MI];
      if constexpr (E != kInt8ToSums) {
        const __amdgpu_buffer_rsrc_t rbs = make_rsrc(a.b_s + (int64_t)g.group * a.N + cn0, (int64_t)(nrows - cn0) * 4);
        const __amdgpu_buffer_rsrc_t rus =
            make_rsrc(a.b_s + (int64_t)g.group * a.N + nrows + cn0, kTwo ? (int64_t)(nrows - cn0) * 4 : 0);
        const __amdgpu_buffer_rsrc_t ras = make_rsrc(a.a_s + row0, (int64_t)rows * 4);
  #pragma unroll
        for (int j = 0; j < NI; ++j)
  #pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t at = (32 * (kTwo ? j / 2 : j) + 8 * q + 4 * h) * 4;
            const u32x4 w = kTwo && (j & 1) ? __builtin_amdgcn_raw_buffer_load_b128(rus, at, 0, 0)
                                            : __builtin_amdgcn_raw_buffer_load_b128(rbs, at, 0, 0);
  #pragma unroll
            for (int v = 0; v < 4; ++v) sb[j][q][v] = __uint_as_float(w[v]);
          }
  #pragma unroll
        for (int i = 0; i < MI; ++i)
          sa[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ras, (32 * (wm * MI + i) + l32) * 4, 0, 0));
      }
  #pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int m0 = 32 * (wm * MI + i);
        if (m0 >= crows) break;
  #pragma unroll
        for (int j = 0; j < NI; j += kTwo ? 2 : 1) {
  #pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = 32 * (kTwo ? j / 2 : j) + 8 * q + 4 * h;
            uint8_t* const at = stage + l32 * kRowBytes + (((col / kPer) ^ (l32 & kMask)) << 4);
            if constexpr (E == kInt8ToSums) {
              *reinterpret_cast<v4i*>(at) = v4i{hop(acc[i][j][4 * q]), hop(acc[i][j][4 * q + 1]), hop(acc[i][j][4 * q + 2]),
                                                hop(acc[i][j][4 * q + 3])};
            } else {
              float y[4];
  #pragma unroll
              for (int v = 0; v < 4; ++v) {
                y[v] = (float)hop(acc[i][j][4 * q + v]) * sa[i] * sb[j][q][v];
                if constexpr (kTwo) y[v] = swiglu(y[v], (float)hop(acc[i][j + 1][4 * q + v]) * sa[i] * sb[j + 1][q][v]);
              }
              if constexpr (kBytes == 4) {
                *reinterpret_cast<v4f*>(at) = v4f{y[0], y[1], y[2], y[3]};
              } else {
                typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                *reinterpret_cast<bf16x4*>(at + 8 * h) = bf16x4{(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
              }
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
            const int r = (u * 64 + lane) / kChunks, ch = (u * 64 + lane) % kChunks, n = cn0 + ch * kPer;
            const uint4 w = *reinterpret_cast<const uint4*>(stage + r * kRowBytes + ((ch ^ (r & kMask)) << 4));
            if (m0 + r < crows && n < ccols) *reinterpret_cast<uint4*>(c + ((crow0 + m0 + r) * ldc + n) * kBytes) = w;
          }
        } else {
          // Rows that no 16-byte stores fit: two bf16 at once where they are even, single
          // values where not; eight reads of LDS in flight (4100 x 4500 x 528: 80 us one by
          // one, 45 by twos; 4100 x 4501 x 528 57).
          const auto narrow = [&](auto word) __attribute__((always_inline)) {
            using Word = decltype(word);
            constexpr int kPlaces = kRowBytes / (int)sizeof(Word), kValues = (int)sizeof(Word) / kBytes;
#pragma unroll 8
            for (int u = 0; u < 32 * kPlaces / 64; ++u) {
              const int r = (u * 64 + lane) / kPlaces, cc = (u * 64 + lane) % kPlaces * kValues, n = cn0 + cc;
              const Word w = *reinterpret_cast<const Word*>(stage + r * kRowBytes + (((cc / kPer) ^ (r & kMask)) << 4) +
                                                            cc % kPer * kBytes);
              if (m0 + r < crows && n < ccols) *reinterpret_cast<Word*>(c + ((crow0 + m0 + r) * ldc + n) * kBytes) = w;
            }
          };
          if (kBytes == 4 || (ldc % 2 == 0 && (reinterpret_cast<uintptr_t>(c) & 3) == 0)) narrow(uint32_t{});
          else if constexpr (kBytes == 2) narrow(uint16_t{});
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      }
    };
    if (TAIL && unit >= 0)                       // a tile of sums, rows past the valid ones left out
      finish(std::integral_constant<int, kInt8ToSums>{}, reinterpret_cast<uint8_t*>(a.planes + (int64_t)unit * BM * BN), BN, 0,
             0, rows, BN);
    else
      finish(std::integral_constant<int, EPI>{},
             reinterpret_cast<uint8_t*>(a.c) + (EPI == kInt8ToSums ? (int64_t)part * a.M * nrows * 4 : 0), nrows, row0, n0,
             rows, nrows);
  };
  if constexpr (TI == 4) {
    // The last tile of a group that needs at most half its rows has half the work
    // (8192 rows of 8 groups by 28672 x 4096: 991 -> 974 us; MLP of 4096 tokens, two
    // choices of 8 experts of 4096 x 14336: 1558 -> 1528 us).
    if (rows <= BM / 2) {
      run(std::integral_constant<int, 2>{});
      return;
    }
  }
  run(std::integral_constant<int, TI>{});
#endif
}

// Four sums of a row from column n on as results (bs: their column scales).
template <int EPI>
__device__ __forceinline__ void finish_four(const Int8GemmArgs& a, int64_t row, int n, int cols, v4i sum, v4i up,
                                            const float* bs) {
  const float sa = a.a_s[row];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= cols) break;
    const int64_t at = row * cols + n + i;
    const float y = (float)sum[i] * sa * bs[i];
    if constexpr (EPI == kInt8ToSwiglu) reinterpret_cast<float*>(a.c)[at] = swiglu(y, (float)up[i] * sa * bs[cols + i]);
    else if constexpr (EPI == kInt8ToF32) reinterpret_cast<float*>(a.c)[at] = y;
    else reinterpret_cast<__bf16*>(a.c)[at] = (__bf16)y;
  }
}

// The planes of a product whose steps were shared out, added up and finished: row
// blockIdx.y, 4 columns a thread. a.planes: [parts, M, N]. Bound by its launch and
// by reading what the caches mostly hold (64 x 4096 x 14336 in 4 parts: 3 of 18 us).
template <int EPI>
__global__ __launch_bounds__(256) void int8_join_kernel(Int8GemmArgs a) {
  const int row = blockIdx.y;
  GroupScan scan;
  scan_groups<1>(a, &scan);                    // "tiles" of one row
  if (row >= scan.total) return;
  const GroupSpan g = group_of<1>(a, scan, row);
  const int cols = EPI == kInt8ToSwiglu ? a.N / 2 : a.N;
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= cols) return;
  const int64_t plane = (int64_t)a.M * a.N;
  const int* const from = a.planes + (int64_t)row * a.N + n;
  int sum[4] = {0, 0, 0, 0}, up[4] = {0, 0, 0, 0};
  if (a.N % (EPI == kInt8ToSwiglu ? 8 : 4) == 0) {
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p) {
      const v4i v = *reinterpret_cast<const v4i*>(from + p * plane);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += v[i];
      if constexpr (EPI == kInt8ToSwiglu) {
        const v4i u = *reinterpret_cast<const v4i*>(from + p * plane + cols);
#pragma unroll
        for (int i = 0; i < 4; ++i) up[i] += u[i];
      }
    }
  } else {
    for (int p = 0; p < a.parts; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < cols) {
          sum[i] += from[p * plane + i];
          if constexpr (EPI == kInt8ToSwiglu) up[i] += from[p * plane + cols + i];
        }
  }
  finish_four<EPI>(a, row, n, cols, v4i{sum[0], sum[1], sum[2], sum[3]}, v4i{up[0], up[1], up[2], up[3]},
                   a.b_s + (int64_t)g.group * a.N + n);
}

// The tail's tiles of sums added up and finished: 16 rows of tail tile blockIdx.x /
// 16, 4 columns a thread. 12 to 15 us for 64 MB of sums, where it saves 43 (second
// product of an MLP of 8192 rows of 8 experts, 4096 x 14336: 527 -> 469 + 15).
template <int EPI>
__global__ __launch_bounds__(256) void int8_tail_join_kernel(Int8GemmArgs a) {
  constexpr bool kPair = EPI == kInt8ToSwiglu;
  GroupScan scan;
  scan_groups<256>(a, &scan);
  const int ntn = a.n_tiles, tiles = scan.total * ntn;
  const Tail tail = tail_of(tiles, (a.K + kBK - 1) / kBK);
  const int t = blockIdx.x >> 4, n = tiles - tail.first;
  if (t >= n || tail.parts < 2) return;
  const int id = tail.first + t;
  const GroupSpan g = group_of<256>(a, scan, id / ntn);
  int mt, nt;
  tile_of(id - g.tile0 * ntn, ntn, g.tiles, &mt, &nt);
  const int cols = kPair ? a.N / 2 : a.N, c = (threadIdx.x & 63) * 4;
  if (kPair && c >= 128) return;
  const int col = (kPair ? 128 : 256) * nt + c, from = kPair ? 64 * (c / 32) + c % 32 : c;
  if (col >= cols) return;
  const float* const bs = a.b_s + (int64_t)g.group * a.N + col;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int m = (blockIdx.x & 15) * 16 + 4 * r + (threadIdx.x >> 6);
    if (mt * 256 + m >= g.rows) break;
    v4i sum = {0, 0, 0, 0}, up = {0, 0, 0, 0};
#pragma unroll 4
    for (int p = 0; p < tail.parts; ++p) {
      const int* const at = a.planes + ((int64_t)(p * n + t) * 256 + m) * 256 + from;
      sum += *reinterpret_cast<const v4i*>(at);
      if constexpr (kPair) up += *reinterpret_cast<const v4i*>(at + 32);
    }
    const int64_t row = g.row0 + (int64_t)mt * 256 + m;
    finish_four<EPI>(a, row, col, cols, sum, up, bs);
  }
}

// Few rows: the weights pass once (where a group has one m-tile) and bound the
// time, so what counts is that many loads are always in flight. A workgroup owns 16
// NT rows of B and 16 MT of A; its W waves share the steps of 128 k among them, each
// a run of its own, with a ring of three stages of its own in LDS that only it fills
// and reads, two steps ahead, without a barrier. The waves' sums meet in LDS at the
// end; sums of integers are the same in any order.
// Rows and k out of range read as zeros, as above. With the SwiGLU (NT = 2) the
// second 16 rows of B are the up rows of the first 16's channels.
// Bound by reading: 16 x 28672 x 4096 in 22.5 us, 117 MB at 5.2 TB/s of the 6.9 that
// reading alone reaches (the ramp of a launch and of the first loads is 3 us of it);
// 16 x 4096 x 14336 12.9, 1 x 999 x 544 2.7 (a launch is 2.2). Steps dealt out in
// turn, not in runs, 23.8 for the first; weights by ordinary instead of nontemporal
// loads 25.8 then. XCDs that start at 8 places of k, as the tiles' do, take 15.4
// instead of 12.9 for the second.
template <int MT, int NT, int W, int EPI, bool NONTEMPORAL>
__global__ __launch_bounds__(64 * W) void gemm_int8_narrow_kernel(Int8GemmArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool kPair = EPI == kInt8ToSwiglu;
  static_assert(!kPair || NT == 2, "16 gate and 16 up rows");
  constexpr int BM = 16 * MT, TN = 16 * NT, kStage = (BM + TN) * kBK, kLoads = (BM + TN) / 8;
  static_assert(W * kStage >= 4 * W * BM * TN, "the sums fit a stage");
  constexpr int kAux = NONTEMPORAL ? 2 : 0;
  __shared__ __attribute__((aligned(16))) uint8_t s0[W * kStage];
  __shared__ __attribute__((aligned(16))) uint8_t s1[W * kStage];
  __shared__ __attribute__((aligned(16))) uint8_t s2[W * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ntn = a.n_tiles, id = blockIdx.x;
  GroupScan scan;
  scan_groups<BM>(a, &scan);
  if (id / ntn >= scan.total) return;
  const GroupSpan g = group_of<BM>(a, scan, id / ntn);
  const int local = id - g.tile0 * ntn;
  const int mt = local % g.tiles, nt = local / g.tiles;
  const int64_t row0 = g.row0 + (int64_t)mt * BM;
  const int rows = min(BM, g.rows - mt * BM);
  const int K = a.K, nk = (K + kBK - 1) / kBK;
  const int turns = __builtin_amdgcn_readfirstlane((nk + W - 1) / W);
  const int nrows = kPair ? a.N / 2 : a.N;
  constexpr int kTileRows = kPair ? TN / 2 : TN;
  const int n0 = nt * kTileRows, ncols = min(kTileRows, nrows - n0);
  const int8_t* const bg = a.b + (int64_t)g.group * a.N * K;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.a + row0 * K, (int64_t)rows * K);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(bg + (int64_t)n0 * K, (int64_t)ncols * K);
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(bg + (int64_t)(nrows + n0) * K, kPair ? (int64_t)ncols * K : 0);
  const int c_even = (lane & 7) ^ (lane >> 4);             // logical chunk in blocks of 8 rows, even ones; odd: ^ 4
  const uint32_t v_even = (uint32_t)(lane >> 3) * K + c_even * 16, v_odd = (uint32_t)(lane >> 3) * K + (c_even ^ 4) * 16;
  auto load = [&](int turn, uint8_t* stage) __attribute__((always_inline)) {
    const int k0 = __builtin_amdgcn_readfirstlane(turn < turns ? (wave * turns + turn) * kBK : K);
    uint8_t* const to = stage + wave * kStage;
    const uint32_t be = k0 + c_even * 16 < K ? v_even : 0x80000000u, bo = k0 + (c_even ^ 4) * 16 < K ? v_odd : 0x80000000u;
#pragma unroll
    for (int b = 0; b < TN / 8; ++b) {
      const uint32_t so = (uint32_t)(8 * (kPair ? b % 2 : b)) * K + k0;
      if (kPair && b >= 2)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ru, (lds_void*)(to + b * 1024), 16, b & 1 ? bo : be, so, 0, kAux);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(to + b * 1024), 16, b & 1 ? bo : be, so, 0, kAux);
    }
    const uint32_t ae = k0 < K ? v_even : 0x80000000u, ao = k0 < K ? v_odd : 0x80000000u;
#pragma unroll
    for (int b = 0; b < BM / 8; ++b)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(to + TN * kBK + b * 1024), 16, b & 1 ? ao : ae,
                                               (uint32_t)(8 * b) * K + k0, 0, 0);
  };
  v4i acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  const int r16 = lane & 15, quarter = lane >> 4;
  auto compute = [&](const uint8_t* stage) __attribute__((always_inline)) {
    const uint8_t* const from = stage + wave * kStage;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      v4i fa[MT], fb[NT];
      const int at = r16 * kBK + (((4 * ks + quarter) ^ ((r16 >> 1) & 7)) << 4);
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[j] = *reinterpret_cast<const v4i*>(from + 16 * j * kBK + at);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[i] = *reinterpret_cast<const v4i*>(from + (TN + 16 * i) * kBK + at);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  };
  // Turn t: the loads of turn t + 2 go out, into the stage that turn t - 1 has
  // read; then all but the last two turns' loads have landed.
  auto turn = [&](int t, const uint8_t* cur, uint8_t* free) __attribute__((always_inline)) {
    load(t + 2, free);
    __builtin_amdgcn_s_waitcnt(wait_vmcnt(2 * kLoads));
    compute(cur);
    __builtin_amdgcn_sched_barrier(0);
  };
  load(0, s0);
  load(1, s1);
  int t = 0;
  for (; t + 2 < turns; t += 3) {
    turn(t, s0, s2);
    turn(t + 1, s1, s0);
    turn(t + 2, s2, s1);
  }
  if (t < turns) turn(t, s0, s2);
  if (t + 1 < turns) turn(t + 1, s1, s0);
  // sums of wave w: [w][row][column]
  __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
  __syncthreads();
  int* const sums = reinterpret_cast<int*>(s0);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) sums[(wave * BM + 16 * i + 4 * quarter + v) * TN + 16 * j + r16] = acc[i][j][v];
  __syncthreads();
  constexpr int kCols = kTileRows;
  for (int u = threadIdx.x; u < BM * kCols; u += 64 * W) {
    const int m = u / kCols, c = u % kCols, n = n0 + c;
    if (m >= rows || n >= nrows) continue;
    const int64_t row = row0 + m;
    const float sa = a.a_s[row];
    const float* const bs = a.b_s + (int64_t)g.group * a.N + n;
    int sum = 0, sum2 = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      sum += sums[(w * BM + m) * TN + c];
      if constexpr (kPair) sum2 += sums[(w * BM + m) * TN + 16 + c];
    }
    const float y = (float)sum * sa * bs[0];
    if constexpr (kPair)
      reinterpret_cast<float*>(a.c)[row * nrows + n] = swiglu(y, (float)sum2 * sa * bs[nrows]);
    else if constexpr (EPI == kInt8ToF32)
      reinterpret_cast<float*>(a.c)[row * a.N + n] = y;
    else
      reinterpret_cast<__bf16*>(a.c)[row * a.N + n] = (__bf16)y;
  }
#endif
}

// The forms of a product.
template <int MT, int NT, int W>
struct Narrow {
  static constexpr int kBM = 16 * MT, kBN = 16 * NT, kThreads = 64 * W, kWaves = W, kStages = 3;
  static constexpr bool kPairs = NT == 2, kSums = false;
  template <int EPI>
  static void launch(dim3 grid, hipStream_t s, const Int8GemmArgs& a) {
    if constexpr (EPI != kInt8ToSums && (EPI != kInt8ToSwiglu || kPairs)) {
      if (a.nontemporal) hipLaunchKernelGGL((gemm_int8_narrow_kernel<MT, NT, W, EPI, true>), grid, dim3(kThreads), 0, s, a);
      else hipLaunchKernelGGL((gemm_int8_narrow_kernel<MT, NT, W, EPI, false>), grid, dim3(kThreads), 0, s, a);
    }
  }
};
template <int MI, int NI, int S>
struct Tile {
  static constexpr int kBM = 64 * MI, kBN = 64 * NI, kThreads = 256, kWaves = 1, kStages = S;
  static constexpr bool kPairs = NI % 2 == 0, kSums = true;
  template <int EPI>
  static void launch(dim3 grid, hipStream_t s, const Int8GemmArgs& a) {
    if constexpr (EPI != kInt8ToSwiglu || kPairs) {
      if constexpr (MI * NI >= 16 && EPI != kInt8ToSums) {
        if (a.tail) {
          hipLaunchKernelGGL((gemm_int8_kernel<MI, NI, S, EPI, true>), grid, dim3(kThreads), 0, s, a);
          hipLaunchKernelGGL(int8_tail_join_kernel<EPI>, dim3(16 * kTailUnits / 2), dim3(256), 0, s, a);
          return;
        }
      }
      hipLaunchKernelGGL((gemm_int8_kernel<MI, NI, S, EPI, false>), grid, dim3(kThreads), 0, s, a);
    }
  }
};
constexpr int kForms = 11;
template <typename Go>
void by_form(int form, const Go& go) {
  switch (form) {
    case 0: return go(Narrow<1, 1, 1>{});
    case 1: return go(Narrow<1, 1, 4>{});
    case 2: return go(Narrow<1, 2, 4>{});
    case 3: return go(Narrow<2, 1, 4>{});
    case 4: return go(Narrow<2, 2, 4>{});
    case 5: return go(Tile<1, 1, 4>{});
    case 6: return go(Tile<1, 2, 4>{});
    case 7: return go(Tile<2, 2, 2>{});
    case 8: return go(Tile<2, 2, 4>{});
    case 9: return go(Tile<4, 2, 3>{});
    default: return go(Tile<4, 4, 2>{});
  }
}

// What a form takes, in us: a step of 128 k of one workgroup alone on a compute
// unit and of one among several there, what a tile takes besides, how much more a
// step takes where k is no multiple of 128 (each piece of a row then lies on two
// cache lines); and the rate, in TB/s, at which it reads weights that pass once.
struct FormCost {
  float alone, among, tile, ragged, rate;
};
constexpr FormCost kCost[kForms] = {
    {0.22f, 0.105f, 0.2f, 1.0f, 5.0f}, {0.36f, 0.35f, 0.2f, 1.5f, 5.7f}, {0.52f, 0.50f, 0.2f, 1.5f, 5.2f},
    {0.50f, 0.50f, 0.2f, 1.5f, 3.6f},  {0.66f, 0.66f, 0.2f, 1.5f, 4.0f}, {0.29f, 0.25f, 0.5f, 1.7f, 4.5f},
    {0.43f, 0.43f, 1.0f, 1.6f, 5.0f},  {0.81f, 0.53f, 1.0f, 1.6f, 3.4f}, {0.60f, 0.60f, 2.0f, 1.4f, 4.6f},
    {0.80f, 0.88f, 5.0f, 1.4f, 3.2f},  {1.45f, 1.45f, 4.0f, 1.15f, 2.5f}};

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
    // A row on a wave while its values take 4 pieces, so that no barrier stands
    // between its loads and its stores; longer ones on the workgroup (16384 x 4096
    // bf16 35 us, on a wave 39; 33 rows 4.0 and 7.6; 16384 x 2048 on a wave 19.6, on
    // the workgroup 22.9: two inputs in turn).
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

// The form and the number of parts that the figures above make cheapest. Checked
// against forms forced, on one group (us; rows x n x k, the form chosen first, /p: k
// shared out by p):
//   16 x 28672 x 4096   16 x 32 22.7, 16 x 16 22.6, 64 x 128 23.9, 256 x 256 40
//   30 x 4096 x 4096    32 x 16 6.8, 32 x 32 8.2, 16 x 32 8.3, 16 x 16 9.1, 64 x 64 11.3
//   30 x 4096 x 4112    32 x 16 8.8, 16 x 32 9.6, 32 x 32 10.6, 64 x 64/2 12.0
//   30 x 5000 x 2048    32 x 32 6.1, 32 x 16 6.9, 64 x 64 7.2, 16 x 16 7.8
//   20 x 8192 x 2048    32 x 32 6.1, 32 x 16 6.8, 64 x 64 7.9, 16 x 32 8.5
//   32 x 4096 x 14336   64 x 128/8 17.6, 32 x 16 17.0, 32 x 32 21.2, 64 x 64/2 23.2
//   32 x 14336 x 4096   64 x 64 14.5, 32 x 32 16.3, 64 x 128 18.5, 32 x 16 19.1
//   64 x 4096 x 14336   64 x 64/4 18.9, 32 x 32 24.7, 64 x 64 38
//   256 x 4096 x 14336  128 x 128/4 32, 256 x 128/4 37, 128 x 128 71
//   256 x 28672 x 4096  256 x 128 39, 128 x 128 50, 256 x 256 54
//   512 x 14336 x 4096  256 x 128 36, 128 x 128 47, 256 x 256 53
//   512 x 28672 x 4096  256 x 256 62, 256 x 128 69, 128 x 128 90
//   2048 x 4096 x 4096  256 x 128 37, 128 x 128 (two a compute unit) 40, 256 x 256 53
//   1024 x 4096 x 14336 128 x 128 73, 256 x 128/2 72, 256 x 256/4 77, 256 x 128 91
// It goes by sizes alone, as if the rows fell evenly to the groups, so that a call's
// workspace does not depend on how they do. For groups of few rows that is its weak
// side: 8 groups by 28672 x 4096 with 8 rows each take 162 us in 16 x 16 (16 x 32
// 147), with 5 to 30 rows 254 in 16 x 16 (64 x 64 163, and 32 x 32 203), with 128 in
// one group 174 (64 x 128 31).
struct Int8Choice {
  int32_t form, parts;
};
void choose_int8(bool pair, const Int8GemmArgs& a, Int8Choice* chosen) {
  const int64_t groups = std::min(a.groups, a.M), per = ((int64_t)a.M + groups - 1) / groups;
  const int steps = (a.K + kBK - 1) / kBK;
  const double weights = (double)groups * a.N * a.K * 1e-6;
  double best_us = 1e30;
  for (int form = 0; form < kForms; ++form) {
    by_form(form, [&](auto f) {
      using Form = decltype(f);
      const FormCost& cost = kCost[form];
      const int64_t mtiles = groups * ((per + Form::kBM - 1) / Form::kBM);
      for (int parts = 1; parts <= (Form::kSums ? 16 : 1); parts *= 2) {
        const bool half = pair && parts == 1;              // the product forms the SwiGLU, not the join
        if (half && !Form::kPairs) continue;
        if (parts > 1 && (steps / parts < 4 || a.M > 65535 || (int64_t)parts * a.M * a.N > ((int64_t)1 << 26))) break;
        const int64_t bn = half ? Form::kBN / 2 : Form::kBN, cols = half ? a.N / 2 : a.N;
        const double wgs = (double)mtiles * ((cols + bn - 1) / bn) * parts;
        double c = std::ceil(wgs / 256), more = 0;
        if (form == kForms - 1 && parts == 1) {   // (the last round's tiles may share out k too)
          const Tail tail = tail_of((int64_t)wgs, steps);
          if (tail.parts > 1) {
            c = tail.first / 256 + 1.0 / tail.parts;
            more = 8 + 0.12 * (wgs - tail.first) * tail.parts;
          }
        }
        const double mine = std::ceil((double)steps / (Form::kWaves * parts)) * (a.K % kBK ? cost.ragged : 1.f);
        double us = std::max(2.5 + mine * std::max((double)cost.alone, c * cost.among) + c * cost.tile, weights / cost.rate);
        us += more;
        if (parts > 1) us += 3.0 + (double)parts * a.M * a.N * 8 / 4.5e6;  // the planes, written and read
        if (us < best_us) {
          best_us = us;
          chosen->form = form;
          chosen->parts = parts;
        }
      }
    });
  }
}

// Weighing the forms takes about a microsecond, a third of a small call's time on
// the host: the last choices of a thread are kept by their sizes.
Int8Choice choice_int8(bool pair, const Int8GemmArgs& a) {
  struct Entry {
    int32_t M = -1, N, K, groups, pair;
    Int8Choice choice;
  };
  static thread_local Entry kept[64];
  Entry& e = kept[((uint32_t)a.M * 2654435761u ^ (uint32_t)a.N * 40503u ^ (uint32_t)a.K * 97u ^ (uint32_t)a.groups * 7u ^ pair) >> 3 & 63];
  if (e.M != a.M || e.N != a.N || e.K != a.K || e.groups != a.groups || e.pair != pair) {
    choose_int8(pair, a, &e.choice);
    e.M = a.M; e.N = a.N; e.K = a.K; e.groups = a.groups; e.pair = pair;
  }
  return e.choice;
}

Int8Plan plan_gemm_int8(int result, const Int8GemmArgs& a) {
  const bool pair = result == kInt8ToSwiglu;
  const int64_t groups = std::min(a.groups, a.M);
  const int steps = (a.K + kBK - 1) / kBK;
  const Int8Choice choice = choice_int8(pair, a);
  Int8Plan best;
  best.form = choice.form;
  best.parts = choice.parts;
  by_form(best.form, [&](auto f) {
    constexpr int BM = decltype(f)::kBM, BN = decltype(f)::kBN;
    const bool half = pair && best.parts == 1;
    const int64_t cols = half ? a.N / 2 : a.N, bn = half ? BN / 2 : BN;
    int64_t mtiles = 0;
    if (a.split == kInt8HostSizes) {
      for (int g = 0; g < a.groups; ++g) mtiles += ((int64_t)a.sizes[g] + BM - 1) / BM;
    } else {
      const int64_t some = a.split == kInt8OneGroup ? 1 : groups;
      mtiles = (a.M + (BM - 1) * some) / BM;               // the most that any split can have
    }
    best.n_tiles = (cols + bn - 1) / bn;
    best.tiles = mtiles * best.n_tiles;
  });
  best.workspace = best.parts > 1 ? (size_t)best.parts * a.M * a.N * 4 : 0;
  best.tail = 0;
  if (best.form == kForms - 1 && best.parts == 1) {
    // a tail: of these tiles, or with groups of any that their rows can make
    best.tail = (int64_t)a.M * a.N > ((int64_t)1 << 24) && tail_of(kTailUnits + 1, steps).parts > 1;
    if (a.split != kInt8DeviceSizes) best.tail = best.tail && tail_of(best.tiles, steps).parts > 1;
    if (best.tail) {
      best.tiles = (best.tiles + kTailUnits - 1) / kTailUnits * kTailUnits;
      best.workspace = (size_t)kTailUnits * 256 * 256 * 4;
    }
  }
  return best;
}

// The narrow forms load weights nontemporally where rows of k begin on cache lines
// (with k no multiple of 128 two steps share a line, and two rows do). This goes by
// k alone: where a group has several m-tiles its weights are read as often, past
// the caches too.
bool nontemporal_int8(const Int8GemmArgs& a) { return a.K % kBK == 0; }

Int8Run describe_gemm_int8(const Int8GemmArgs& a, const Int8Plan& p) {
  Int8Run r{};
  by_form(p.form, [&](auto f) {
    using Form = decltype(f);
    r = Int8Run{Form::kBM, Form::kBN, Form::kThreads / 64, Form::kStages, p.parts, p.tail,
                !Form::kSums && nontemporal_int8(a)};
  });
  return r;
}

hipError_t launch_gemm_int8(int result, const Int8GemmArgs& args, const Int8Plan& p, void* workspace, hipStream_t stream) {
  Int8GemmArgs a = args;
  a.n_tiles = (int32_t)p.n_tiles;
  a.parts = p.parts;
  a.tail = p.tail;
  a.planes = reinterpret_cast<int32_t*>(workspace);
  a.nontemporal = nontemporal_int8(a);
  if (p.tiles == 0) return hipSuccess;
  by_form(p.form, [&](auto s) {
    using S = decltype(s);
    const dim3 grid((unsigned)(p.tiles * p.parts));
    if (p.parts > 1) {
      Int8GemmArgs sums = a;
      sums.c = workspace;
      S::template launch<kInt8ToSums>(grid, stream, sums);
    } else if (result == kInt8ToBf16) {
      S::template launch<kInt8ToBf16>(grid, stream, a);
    } else if (result == kInt8ToF32) {
      S::template launch<kInt8ToF32>(grid, stream, a);
    } else {
      S::template launch<kInt8ToSwiglu>(grid, stream, a);
    }
  });
  if (p.parts > 1) {
    const int cols = result == kInt8ToSwiglu ? a.N / 2 : a.N;
    const dim3 grid((unsigned)((cols + 1023) / 1024), (unsigned)a.M);
    if (result == kInt8ToBf16) hipLaunchKernelGGL(int8_join_kernel<kInt8ToBf16>, grid, dim3(256), 0, stream, a);
    else if (result == kInt8ToF32) hipLaunchKernelGGL(int8_join_kernel<kInt8ToF32>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(int8_join_kernel<kInt8ToSwiglu>, grid, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace mx
