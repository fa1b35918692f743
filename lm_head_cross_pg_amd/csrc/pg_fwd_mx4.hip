// Forward of the fused tied head on 4-bit operands for gfx950: hidden states and embedding both in the
// microscaled 4-bit format (pg_mx4.h), their product by v_mfma_scale_f32_32x32x64_f8f6f4 (every value
// of both formats and every product of two is exact; the sum over D is float32), then the softcap,
// log-sum-exp and cross-entropy of the bf16 forward without the T x V logits ever reaching memory.
//
// Bound: an fp4 product of 512 deep is done in half the time that softcap and exponential of its logits
// take, so the vector units set the pace: 98 instructions per 32 x 32 logits (of them two transcendentals per
// logit), 96 at least. 65536 x 512 x 8192 takes 180 us (3.05 PFLOP/s; the bf16 forward 440), of which vector
// instructions issue for 81 %, at 2.2 GHz (constant inputs, which draw less power: 10 % less).
#include "pg_internal.h"
#include "pg_mx4.h"

namespace pg {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct FwdMx4Params {
  const uint8_t* hc;
  const uint8_t* hs;
  const uint8_t* ec;
  const uint8_t* es;
  const int32_t* target;
  const uint8_t* mask;    // rows to select in the kernel itself, or nullptr
  int32_t* rows;          // compacted scored rows, or nullptr (row i = i)
  int32_t* n_dev;         // device row count, or nullptr (use n_host)
  int64_t n_host;
  int64_t cb, sb;         // bytes of a row of codes, of scales
  int steps;              // 64-value steps of a row
  int V;
  int grid;               // workgroups of the launch
  int aim;                // workgroups that splits make of few rows
  int rows_per_wg;
  int splits;             // of the vocabulary; 0: from the row count and the grid
  int per;                // tiles of a split, where the host chose the splits
  Softcap sc;
  float* nats;
  float* lse;
  float* part_l;
  float* part_m;
  float* s_target;
};

// Vocabulary splits: the host's choice, or, where only the device knows the row count, as many as make `aim`
// workgroups, at most one per tile of the vocabulary. (n < 2^31: 32-bit divisions.)
__host__ __device__ __forceinline__ int mx4_splits(const FwdMx4Params& p, int64_t n, int ntiles) {
  if (p.splits > 0) return p.splits;
  const uint32_t rt = ((uint32_t)n + (uint32_t)p.rows_per_wg - 1u) / (uint32_t)p.rows_per_wg;
  if (rt == 0u) return 1;
  const uint32_t s = (uint32_t)p.aim / rt;
  return s < 1u ? 1 : (s > (uint32_t)ntiles ? ntiles : (int)s);
}

// The target's term is one of the sum's, so a negative difference is a rounding (NaN passes).
__device__ __forceinline__ float not_below_zero(float d) { return d < 0.f ? 0.f : d; }

// The partial sums of a row's splits lie side by side, from a 16-byte boundary where there are several
// (so that n rows of S splits take at most twice n S entries).
__host__ __device__ __forceinline__ int mx4_split_stride(int S) { return S <= 2 ? S : (S + 3) & ~3; }

__device__ __forceinline__ f32x16 mfma_mx4(const i32x4& a, int sa, const i32x4& b, int sb, const f32x16& c) {
  const i32x8 aa = {a[0], a[1], a[2], a[3]}, bb = {b[0], b[1], b[2], b[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aa, bb, c, 4, 4, 0, sa, 0, sb);
}

// The scale bytes of a lane's half of each step: of 16 bytes (blocks 0 .. 15) bytes h, h + 2, ...: byte j
// of word i belongs to step 4 i + j.
template <int NW>
__device__ __forceinline__ void mx4_lane_scales(const i32x4* row, int h, int (&out)[NW]) {
  const uint32_t sel = h ? 0x07050301u : 0x06040200u;
#pragma unroll
  for (int i = 0; i < NW; ++i)
    out[i] = (int)__builtin_amdgcn_perm((uint32_t)row[i >> 1][2 * (i & 1) + 1], (uint32_t)row[i >> 1][2 * (i & 1)], sel);
}

template <int OP>
__device__ __forceinline__ f32x16 mfma_mx4_op(const i32x4& a, int sa, const i32x4& b, int sb, const f32x16& c) {
  const i32x8 aa = {a[0], a[1], a[2], a[3]}, bb = {b[0], b[1], b[2], b[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aa, bb, c, 4, 4, OP, sa, OP, sb);
}

// Step k of a chain (an unrolled loop's k is a constant, which the switch folds on): words of four steps'
// scales, byte k % 4.
__device__ __forceinline__ f32x16 mx4_step(int k, const i32x4& a, const int* sa, const i32x4& b, const int* sb,
                                           const f32x16& acc) {
  switch (k & 3) {
    case 0: return mfma_mx4_op<0>(a, sa[k >> 2], b, sb[k >> 2], acc);
    case 1: return mfma_mx4_op<1>(a, sa[k >> 2], b, sb[k >> 2], acc);
    case 2: return mfma_mx4_op<2>(a, sa[k >> 2], b, sb[k >> 2], acc);
    default: return mfma_mx4_op<3>(a, sa[k >> 2], b, sb[k >> 2], acc);
  }
}

// Any width: a wave holds the sums of 64 rows against 64 vocabulary rows (four accumulators, so that each
// fragment is used twice) and both sides' fragments come from memory, two steps ahead of their use. Lane l
// holds row l % 32 of a fragment, the step's half l / 32, and its block's scale. Bound by the first-level
// cache, where a fragment's 32 rows are 32 lines: 4096 x 2048 x 8192 in 158 us (0.9 PFLOP/s; 32 x 32 logits a
// wave without loads ahead 457; four steps ahead do not fit the registers).
constexpr int kMx4StreamRows = 256, kMx4StreamTile = 64;
struct Mx4Fragments {
  i32x4 a[2], b[2];   // of the vocabulary, of the states
};

__global__ __launch_bounds__(256, 2) void fwd_mx4_stream_kernel(FwdMx4Params p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, col = lane & 31;
  const int64_t n = p.n_dev ? (int64_t)(*p.n_dev) : p.n_host;
  const int ntiles = (p.V + kMx4StreamTile - 1) / kMx4StreamTile, steps = p.steps;
  const int S = mx4_splits(p, n, ntiles);
  const int64_t rt = blockIdx.x / S;
  const int split = blockIdx.x % S;
  const int64_t tok0 = rt * kMx4StreamRows + wave * 64;
  if (tok0 >= n) return;
  const int per = (ntiles + S - 1) / S;
  const int b0 = split * per, b1 = min(b0 + per, ntiles);

  constexpr int kAhead = 2;
  const uint8_t *hc[2], *hs[2];
  int y[2];
  float m[2], l[2], sy[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int64_t tok = tok0 + 32 * g + col;
    const int64_t ic = tok < n ? tok : n - 1;
    const int64_t row = p.rows ? (int64_t)p.rows[ic] : ic;
    hc[g] = p.hc + row * p.cb + 16 * h;
    hs[g] = p.hs + row * p.sb;
    y[g] = p.target[row];
    m[g] = sy[g] = -INFINITY;
    l[g] = 0.f;
  }
  for (int b = b0; b < b1; ++b) {
    const uint8_t *ec[2], *es[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t v = min(b * kMx4StreamTile + 32 * i + col, p.V - 1);
      ec[i] = p.ec + v * p.cb + 16 * h;
      es[i] = p.es + v * p.sb;
    }
    f32x16 acc[2][2] = {};
    Mx4Fragments f[2][kAhead];
    int sa[2][2], sb[2][2];
    // the kAhead steps from k on (past the end: the last one, which is not used)
    auto load = [&](Mx4Fragments (&to)[kAhead], int k) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t at = 32 * (int64_t)min(k + j, steps - 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          to[j].a[i] = *reinterpret_cast<const i32x4*>(ec[i] + at);
          to[j].b[i] = *reinterpret_cast<const i32x4*>(hc[i] + at);
        }
      }
    };
    // scales of steps k .. k + 7 (a row's scales are padded to 16 bytes)
    auto scales = [&](int k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx4_lane_scales(reinterpret_cast<const i32x4*>(es[i] + 2 * k), h, sa[i]);
        mx4_lane_scales(reinterpret_cast<const i32x4*>(hs[i] + 2 * k), h, sb[i]);
      }
    };
    auto step = [&](const Mx4Fragments& f, int j) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int g = 0; g < 2; ++g) acc[i][g] = mx4_step(j, f.a[i], sa[i], f.b[g], sb[g], acc[i][g]);
    };
    load(f[0], 0);
    int k = 0;
    for (; k + 8 <= steps; k += 8) {
      scales(k);
#pragma unroll
      for (int q = 0; q < 8 / kAhead; ++q) {
        load(f[(q + 1) & 1], k + kAhead * (q + 1));
#pragma unroll
        for (int j = 0; j < kAhead; ++j) step(f[q & 1][j], kAhead * q + j);
      }
    }
    if (k < steps) {
      scales(k);
#pragma unroll
      for (int q = 0; q < 8 / kAhead; ++q) {
        load(f[(q + 1) & 1], k + kAhead * (q + 1));
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (k + kAhead * q + j < steps) step(f[q & 1][j], kAhead * q + j);
      }
    }
    // register r: vocabulary row 8 (r / 4) + 4 h + r % 4 of the block
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      float s2[2][16], bm = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int vr = b * kMx4StreamTile + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
          s2[i][r] = vr < p.V ? capped_log2(acc[i][g][r], p.sc) : -INFINITY;
          bm = fmaxf(bm, s2[i][r]);
          if (vr == y[g] && vr < p.V) sy[g] = s2[i][r];
        }
      const float mn = fmaxf(m[g], bm);
      float part = 0.f;
      if (mn != -INFINITY) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) part += fexp2(s2[i][r] - mn);
        l[g] = l[g] * fexp2(m[g] - mn) + part;
        m[g] = mn;
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) l[g] += s2[i][r] != s2[i][r] ? s2[i][r] : 0.f;   // NaN rows stay NaN
      }
    }
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int64_t tok = tok0 + 32 * g + col;
    lse_merge(m[g], l[g], __shfl_xor(m[g], 32), __shfl_xor(l[g], 32));
    const float sy2 = __shfl_xor(sy[g], 32);
    // this split holds the target's row
    const bool here = y[g] >= b0 * kMx4StreamTile && y[g] < b1 * kMx4StreamTile && y[g] < p.V;
    if (h == 0 && tok < n) {
      const int64_t at = tok * mx4_split_stride(S) + split;
      p.part_l[at] = l[g];
      p.part_m[at] = m[g];
      if (here) p.s_target[tok] = ((y[g] >> 2) & 1) ? sy2 : sy[g];
      else if (split == 0 && !(y[g] >= 0 && y[g] < p.V)) p.s_target[tok] = __builtin_nanf("");
    }
  }
}

// ---------------------------------------------------------------------- widths up to 1024
//
// A workgroup of eight waves owns 128 rows: waves w and w + 4 hold the same 32 rows' codes and scales in
// registers (the B operand) and take the even and the odd 32-row blocks of each vocabulary tile. The
// tiles stream through LDS, two buffers, copied there by DMA while the tile before is worked on; every
// wave reads the fragments of its blocks from LDS (the A operand). An accumulator holds 16 vocabulary
// rows of one token per lane, so the softcap and the sum of exponentials run per lane. Where there
// are 256 rows for every CU, a wave holds 64 of them (RB = 2): each fragment read then feeds two products (65536
// rows: 199 -> 188 us); with fewer rows 32 a wave make more workgroups.
template <int KS>
struct Mx4Tile {
  static constexpr int kRows = KS <= 8 ? 128 : 64;                // vocabulary rows of a tile
  static constexpr int kBlocksPerWave = kRows / 64;
  static constexpr int CPR = KS <= 1 ? 2 : KS <= 2 ? 4 : KS <= 4 ? 8 : KS <= 8 ? 16 : 32;   // 16-byte chunks of an LDS row
  static constexpr int kRowBytes = 16 * CPR;
  static constexpr int kRowsPerLine = kRowBytes < 256 ? 256 / kRowBytes : 1;   // rows per pass over the banks
  static constexpr int kSwz = CPR < 16 ? CPR : 16;
  static constexpr int kScaleBytes = KS <= 8 ? 16 : 32;           // of an LDS row of scales
  static constexpr int kCodes = kRows * kRowBytes;                // bytes of a tile's codes
  static constexpr int kBytes = kCodes + kRows * kScaleBytes;
  static constexpr int kPieces = kCodes / 1024;                   // code DMAs of 1 KiB
  static constexpr int kLoads = (kPieces + 7) / 8;                // of a wave, at most
  // Chunk c of row r sits at chunk c ^ swizzle(r) of the row, so that the 16 rows that a read phase
  // takes at one chunk lie in different banks.
  __device__ static int swizzle(int row) { return (row / kRowsPerLine) % kSwz; }
};

// One DMA of 16 bytes per lane to 1 KiB of LDS from a uniform base and a per-lane offset (see lds_dma16
// for why it is assembly; completion is the caller's business).
__device__ __forceinline__ void lds_dma16_base(const uint8_t* base, uint32_t offset, uint32_t lds_addr) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(offset), "s"(base), "s"(lds_addr)
      : "memory");
}

// The same with 4 bytes per lane, to 256 bytes of LDS.
__device__ __forceinline__ void lds_dma4_base(const uint8_t* base, uint32_t offset, uint32_t lds_addr) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(offset), "s"(base), "s"(lds_addr)
      : "memory");
}

// Selection of the scored rows by the head itself, for 16 to kMx4MaskRows rows: every workgroup reads the whole
// mask (from L2, at most 64 KiB), counts, and keeps its own 128 rows in LDS, which takes 5 us at 65536 rows and 3
// at 3001. A launch of its own for the list takes 7 and 4 and the gap between two launches (the call with 2048
// of 65536 rows scored: 22.9 -> 21.4 us; with half of 3001: 16.8 -> 14.7).
constexpr int kMx4MaskPiece = 1024;                        // rows that a wave takes at once, 16 a lane
constexpr int kMx4MaskPieces = 8;                          // pieces of a wave, at most
constexpr int kMx4MaskRows = 8 * kMx4MaskPieces * kMx4MaskPiece;
// The sum of v over this lane and those below: within runs of 16 lanes, then the runs before.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast 15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}
struct Mx4MaskRows {
  uint32_t bits[kMx4MaskPieces];   // of this lane's 16 rows in each piece
  int before[kMx4MaskPieces];      // scored rows of the piece in lower lanes
  int total[kMx4MaskPieces];       // of the piece (uniform)
  int base;                        // in lower waves (uniform)
  int pieces;                      // of a wave

  __device__ __forceinline__ int row0(int wave, int lane, int q) const {
    return (wave * pieces + q) * kMx4MaskPiece + 16 * lane;
  }
  // Counts; returns the number of scored rows. sums: eight entries of LDS.
  __device__ __forceinline__ int count(const uint8_t* mask, int T, int wave, int lane, int* sums) {
    pieces = (T + 8 * kMx4MaskPiece - 1) / (8 * kMx4MaskPiece);
    typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
    u32x4_a1 w[kMx4MaskPieces];
#pragma unroll
    for (int q = 0; q < kMx4MaskPieces; ++q) {   // (16 rows that the mask's end cuts are read from T - 16 on)
      w[q] = u32x4_a1{0, 0, 0, 0};
      if (q < pieces && row0(wave, lane, q) < T)
        w[q] = *reinterpret_cast<const u32x4_a1*>(mask + min(row0(wave, lane, q), T - 16));
    }
    int counts[kMx4MaskPieces / 2];
#pragma unroll
    for (int q = 0; q < kMx4MaskPieces; ++q) {
      uint32_t b = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // a bit per nonzero byte
        const uint32_t f = ((((w[q][k] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w[q][k]) & 0x80808080u) >> 7;
        b |= ((f * 0x01020408u) >> 24 & 15u) << (4 * k);
      }
      bits[q] = b >> min(max(row0(wave, lane, q) + 16 - T, 0), 31);
      counts[q / 2] = q & 1 ? counts[q / 2] | __popc(bits[q]) << 16 : __popc(bits[q]);
    }
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kMx4MaskPieces / 2; ++k) {   // two pieces to a scan (a piece has at most 1024)
      const int upto = wave_scan(counts[k]), below = upto - counts[k], all = __builtin_amdgcn_readlane(upto, 63);
      before[2 * k] = below & 0xffff;
      before[2 * k + 1] = below >> 16;
      total[2 * k] = all & 0xffff;
      total[2 * k + 1] = all >> 16;
      mine += total[2 * k] + total[2 * k + 1];
    }
    if (lane == 0) sums[wave] = mine;
    lds_barrier();
    int n = 0;
    base = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int v = sums[k];
      n += v;
      base += k < wave ? v : 0;
    }
    base = __builtin_amdgcn_readfirstlane(base);
    return __builtin_amdgcn_readfirstlane(n);
  }
  // The scored rows lo .. lo + 127 to list, and to rows + lo where `rows` is given.
  __device__ __forceinline__ void keep(int lo, int wave, int lane, int* list, int32_t* rows) const {
    int start = base;
#pragma unroll
    for (int q = 0; q < kMx4MaskPieces; ++q) {
      if (start < lo + 128 && start + total[q] > lo) {
        int at = start + before[q] - lo;
        for (uint32_t b = bits[q]; b; b &= b - 1, ++at) {
          if ((uint32_t)at >= 128u) continue;
          const int row = row0(wave, lane, q) + __ffs(b) - 1;
          list[at] = row;
          if (rows) rows[lo + at] = row;
        }
      }
      start += total[q];
    }
  }
};

// Forms of the sum: a softcap in the fixed-shift range, no softcap, a larger softcap (the last two with a
// reference that follows the largest logit).
enum Mx4Form { kMx4Fixed, kMx4Uncapped, kMx4Capped };

template <int KS, int RB, Mx4Form FORM>
__global__ __launch_bounds__(512, KS <= 8 && RB == 1 ? 4 : 2) void fwd_mx4_kernel(FwdMx4Params p) {
  using TL = Mx4Tile<KS>;
  constexpr bool FIXED = FORM == kMx4Fixed;
  constexpr int NW = (KS + 3) / 4;          // words of a lane's scales
  constexpr int NS = TL::kScaleBytes / 16;
  __shared__ __attribute__((aligned(1024))) char smem[2 * TL::kBytes];
  __shared__ float merge[2][RB][4][32];
  __shared__ int list[128], sums[8];
  const lds_char* lds = (const lds_char*)smem;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, col = lane & 31;
  Mx4MaskRows own;
  int64_t n;
  const bool select = RB == 1 && p.mask != nullptr;
  if (select) {
    const int T = (int)p.n_host;
    n = own.count(p.mask, T, wave, lane, sums);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.n_dev = (int)n;
  } else {
    n = p.n_dev ? (int64_t)(*p.n_dev) : p.n_host;
  }
  const int ntiles = (p.V + TL::kRows - 1) / TL::kRows;
  // the host's choice comes as a grid of splits x row tiles (row tiles alone for one split): no divisions
  int S = p.splits, per = p.per, split = 0;
  int64_t rt = blockIdx.x;
  if (S == 0) {
    S = mx4_splits(p, n, ntiles);
    rt = blockIdx.x / (uint32_t)S;
    split = blockIdx.x % (uint32_t)S;
    per = (ntiles + S - 1) / S;
  } else if (S > 1) {
    rt = blockIdx.y;
    split = blockIdx.x;
  }
  if (rt * (128 * RB) >= n) return;
  if (select) {
    own.keep((int)rt * 128, wave, lane, list, split == 0 ? p.rows : nullptr);
    lds_barrier();
  }
  const int t0 = split * per, t1 = min(t0 + per, ntiles);

  // This wave's part of a tile: kLoads pieces of codes (piece j: 1 KiB, lane i its 16 bytes at 16 i), and
  // a 256-byte piece of the scales. A lane's offset in a piece is the same for each.
  constexpr int RPI = 1024 / TL::kRowBytes;                 // rows of a piece
  constexpr int SPR = TL::kScaleBytes / 4, SRPI = 64 / SPR; // words of a row of scales, rows of a piece
  static_assert(TL::kRows * TL::kScaleBytes == 8 * 256, "a piece of scales per wave");
  const int prow = lane / TL::CPR, srow = lane / SPR;
  int lchunk = (lane % TL::CPR) ^ TL::swizzle(wave * RPI + prow);   // the same for all pieces of the wave
  if (lchunk >= 2 * p.steps) lchunk = 0;      // not in the rows (read by no one, or against zero states)
  int spart = lane % SPR;
  if (4 * spart >= p.sb) spart = 0;
  const int cb = (int)p.cb, sb = (int)p.sb;   // a row's bytes: at most 512 and 32
  const uint32_t coff = (uint32_t)(prow * cb + 16 * lchunk), soff = (uint32_t)(srow * sb + 4 * spart);
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds + wave * 1024, lds1 = (uint32_t)(uintptr_t)lds + TL::kCodes + wave * 256;
  auto load_whole = [&](int tile, int buf) {
    const int64_t v0 = (int64_t)tile * TL::kRows;
    const uint8_t* cbase = p.ec + (v0 + wave * RPI) * cb;
#pragma unroll
    for (int q = 0; q < TL::kLoads; ++q) {
      if (TL::kPieces % 8 != 0 && wave + 8 * q >= TL::kPieces) break;
      lds_dma16_base(cbase + 8 * q * RPI * cb, coff, lds0 + buf * TL::kBytes + 8192 * q);
    }
    lds_dma4_base(p.es + (v0 + wave * SRPI) * sb, soff, lds1 + buf * TL::kBytes);
  };
  auto load_last = [&](int tile, int buf) {   // rows past the vocabulary repeat its last one
    const int v0 = tile * TL::kRows, last = p.V - 1 - v0;
#pragma unroll
    for (int q = 0; q < TL::kLoads; ++q) {
      if (TL::kPieces % 8 != 0 && wave + 8 * q >= TL::kPieces) break;
      lds_dma16_base(p.ec + (int64_t)v0 * cb, (uint32_t)(min((wave + 8 * q) * RPI + prow, last) * cb + 16 * lchunk),
                     lds0 + buf * TL::kBytes + 8192 * q);
    }
    lds_dma4_base(p.es + (int64_t)v0 * sb, (uint32_t)(min(wave * SRPI + srow, last) * sb + 4 * spart),
                  lds1 + buf * TL::kBytes);
  };
  // tiles t0 .. tw - 1 are whole; a last one that is not is taken on its own at the end
  const int tw = min(t1, p.V / TL::kRows);
  if (t0 < tw) load_whole(t0, 0);

  // the rows of this wave: codes and scales
  const int rg = wave & 3, half = wave >> 2;
  auto token = [&](int rb, int c) { return rt * (128 * RB) + (rg * RB + rb) * 32 + c; };
  auto row_of = [&](int rb, int c) {
    if (select) return (int64_t)list[min((rg * RB + rb) * 32 + c, (int)(n - rt * 128) - 1)];
    const int64_t tok = token(rb, c), i = tok < n ? tok : n - 1;
    return p.rows ? (int64_t)p.rows[i] : i;
  };
  i32x4 hf[RB][KS];
  int hs[RB][NW];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int64_t row = row_of(rb, col);
    const i32x4* src = reinterpret_cast<const i32x4*>(p.hc + row * p.cb + 16 * h);
#pragma unroll
    for (int k = 0; k < KS; ++k) hf[rb][k] = k < p.steps ? src[2 * k] : i32x4{};
    i32x4 sr[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
      sr[i] = 16 * i < p.sb ? reinterpret_cast<const i32x4*>(p.hs + row * p.sb)[i] : i32x4{};
    mx4_lane_scales<NW>(sr, h, hs[rb]);
  }

  // Sums of the terms 2^(s log2 e - reference). Fixed shift: the reference is M. Otherwise it is m, which
  // follows the largest logit only when one is more than 2^kSlack times the terms around 1: the sum has
  // room for that, and the usual block costs no rescaling.
  constexpr float kSlack = 40.f;
  float l[RB], m[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    l[rb] = 0.f;
    m[rb] = -1e30f;
  }
  auto exponent = [&](int rb, float z) {
    if (FORM == kMx4Uncapped) return __builtin_fmaf(z, kLog2e, -m[rb]);
    const float t = capped_shifted(z, p.sc.alpha, p.sc.invK);
    return FIXED ? t : (p.sc.M - m[rb]) + t;
  };
  // before the terms of a block are added: its largest logit (the cap is monotone) against the reference
  auto follow = [&](int rb, const f32x16& z) {
    if (FIXED) return;
    float top = z[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
    const float s2 = FORM == kMx4Capped ? p.sc.M + capped_shifted(top, p.sc.alpha, p.sc.invK) : top * kLog2e;
    if (__any(s2 > m[rb] + kSlack)) {
      const float mn = fmaxf(m[rb], s2);
      l[rb] *= fexp2(m[rb] - mn);
      m[rb] = mn;
    }
  };

  // Software pipeline: the chain of a block's steps runs between the terms of the block before it, and
  // fragments are read from LDS kAhead steps before their use, across blocks and tiles. The barrier that
  // publishes the next tile therefore stands kAhead steps before a tile's end: there every read of this
  // tile has been issued and waited for, so its buffer also takes the tile after the next.
  constexpr int kAhead = 1;
  constexpr int kPerStep = (16 * RB + KS - 1) / KS;   // terms added per step
  // LDS addresses of this lane's fragment of each step in buffer 0, block 0: the others are a constant away
  // (blocks start at multiples of 64 rows, whole periods of the swizzle)
  const lds_char* fptr[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k)
    fptr[k] = lds + (half * 32 + col) * TL::kRowBytes + (((2 * k + h) ^ TL::swizzle(half * 32 + col)) * 16);
  const lds_char* sptr = lds + TL::kCodes + (half * 32 + col) * TL::kScaleBytes;
  typedef const __attribute__((address_space(3))) i32x4* frag_ptr;
  i32x4 next[kAhead], nscale[NS];

  typedef f32x16 Block[RB];
  Block prev;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int r = 0; r < 16; ++r) prev[rb][r] = -INFINITY;
  if (FIXED && t0 < tw) {   // there is no block before the first one: what its terms will add is taken off here
    const float none = fexp2(exponent(0, -INFINITY));
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int r = 0; r < 16; ++r) l[rb] -= none;
  }
  // block B of tile t, which is in buffer BUF, into acc, adding the terms of `before`
  auto block = [&](auto buf_, auto b_, int t, Block& acc, const Block& before) {
    constexpr int BUF = decltype(buf_)::value, B = decltype(b_)::value;
    constexpr bool LAST = B + 1 == TL::kBlocksPerWave;
    constexpr int NBUF = LAST ? BUF ^ 1 : BUF, NB = LAST ? 0 : B + 1;   // the block after this one
    constexpr int at = BUF * TL::kBytes + B * 64 * TL::kRowBytes;
    constexpr int nat = NBUF * TL::kBytes + NB * 64 * TL::kRowBytes;
    constexpr int snat = NBUF * TL::kBytes + NB * 64 * TL::kScaleBytes;
    i32x4 fr[KS];
    int sa[NW];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fr[k] = next[k];
    mx4_lane_scales<NW>(nscale, h, sa);
    float part[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      follow(rb, before[rb]);
      acc[rb] = f32x16{};
      part[rb] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      // priority falls with progress through the tile, so that of the waves that share a SIMD the one
      // behind goes first and none waits long at the barrier (at equal priority the older one runs
      // ahead: 26 % of the waves' time was spent waiting, 12 % with this; 178 -> 175 us)
      if (k == 0) __builtin_amdgcn_s_setprio(LAST ? 2 : 3);
      if (LAST && KS >= 4 && k == KS / 2) __builtin_amdgcn_s_setprio(1);
      if (LAST && KS >= 4 && k == KS - 2) __builtin_amdgcn_s_setprio(0);
      if (k == KS - kAhead) {
        if (LAST) {
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // tile t + 1 has landed, tile t is read
          __syncthreads();
          load_whole(min(t + 2, tw - 1), BUF);   // (past the end a tile that no one reads: no branch here)
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) nscale[i] = *(frag_ptr)(sptr + snat + 16 * i);
      }
      if (k + kAhead < KS) fr[k + kAhead] = *(frag_ptr)(fptr[k + kAhead] + at);
      else next[k + kAhead - KS] = *(frag_ptr)(fptr[k + kAhead - KS] + nat);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) acc[rb] = mx4_step(k, fr[k], sa, hf[rb][k], hs[rb], acc[rb]);
#pragma unroll
      for (int e = k * kPerStep; e < (k + 1) * kPerStep && e < 16 * RB; ++e)
        part[e / 16] += fexp2(exponent(e / 16, before[e / 16][e % 16]));
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) asm volatile("" ::"v"(part[rb]));   // a use here keeps the terms between the MFMAs
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      asm volatile("" : "+v"(acc[rb]));   // the chain stays in its block
      l[rb] += part[rb];
    }
  };
  auto tile = [&](auto buf_, int t) {
    Block a0;
    block(buf_, std::integral_constant<int, 0>{}, t, a0, prev);
    if (!FIXED && t == t0) {                     // there was no block before
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) l[rb] = 0.f;
    }
    if constexpr (TL::kBlocksPerWave == 2) {
      block(buf_, std::integral_constant<int, 1>{}, t, prev, a0);
    } else {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) prev[rb] = a0[rb];
    }
  };
  auto add = [&](int rb, const f32x16& z, int vbase) {   // a block on its own; rows past the vocabulary drop out
    // (register r: vocabulary row 8 (r / 4) + 4 h + r % 4 of the block)
    f32x16 y = z;
#pragma unroll
    for (int r = 0; r < 16; ++r) y[r] = vbase + 8 * (r >> 2) + 4 * h + (r & 3) < p.V ? z[r] : -INFINITY;
    follow(rb, y);
    float part = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float e = fexp2(exponent(rb, y[r]));
      part += vbase + 8 * (r >> 2) + 4 * h + (r & 3) < p.V ? e : 0.f;
    }
    l[rb] += part;
  };

  if (t0 < tw) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    load_whole(min(t0 + 1, tw - 1), 1);
#pragma unroll
    for (int i = 0; i < NS; ++i) nscale[i] = *(frag_ptr)(sptr + 16 * i);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) next[k] = *(frag_ptr)(fptr[k]);
    for (int t = t0;;) {
      tile(std::integral_constant<int, 0>{}, t);
      if (++t >= tw) break;
      tile(std::integral_constant<int, 1>{}, t);
      if (++t >= tw) break;
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
      add(rb, prev[rb], (tw - 1) * TL::kRows + (TL::kBlocksPerWave - 1) * 64 + half * 32);
  }
  if (t0 <= tw && tw < t1) {   // (a split without tiles starts past the last one)
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();                             // nothing is in flight to buffer 0, and no one reads it
    load_last(tw, 0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (int b = 0; b < TL::kBlocksPerWave; ++b) {
      const int vbase = tw * TL::kRows + b * 64 + half * 32;
      if (vbase >= p.V) break;
      i32x4 sr[NS];
      int sa[NW];
#pragma unroll
      for (int i = 0; i < NS; ++i) sr[i] = *(frag_ptr)(sptr + b * 64 * TL::kScaleBytes + 16 * i);
      mx4_lane_scales<NW>(sr, h, sa);
      Block acc = {};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const i32x4 a = *(frag_ptr)(fptr[k] + b * 64 * TL::kRowBytes);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) acc[rb] = mx4_step(k, a, sa, hf[rb][k], hs[rb], acc[rb]);
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) add(rb, acc[rb], vbase);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copy to LDS outlives the workgroup

  // the other half of the lanes, then the other wave of these rows
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    lse_merge(m[rb], l[rb], __shfl_xor(m[rb], 32), __shfl_xor(l[rb], 32));
    if (half == 1 && h == 0) {
      merge[0][rb][rg][col] = m[rb];
      merge[1][rb][rg][col] = l[rb];
    }
  }
  __syncthreads();
  if (half == 1) return;
  int c = col;   // not seen through, so that nothing formed from it is kept in registers over the loop above
  asm volatile("" : "+v"(c));
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    if constexpr (FIXED) l[rb] += merge[1][rb][rg][col];
    else lse_merge(m[rb], l[rb], merge[0][rb][rg][col], merge[1][rb][rg][col]);
    const int64_t tok = token(rb, c), row = row_of(rb, c);

    // The targets' logits: the 32 target rows as the A operand, whose product with the 32 tokens has them
    // on the diagonal, formed by the same instructions from the same values as the sum's.
    float sy = __builtin_nanf("");
    if (split == 0) {
      const int y = p.target[row];
      const bool ok = y >= 0 && y < p.V;
      const int64_t v = ok ? y : 0;
      const i32x4* src = reinterpret_cast<const i32x4*>(p.ec + v * p.cb + 16 * h);
      i32x4 a[KS], sr[NS];
      int sa[NW];
#pragma unroll
      for (int k = 0; k < KS; ++k) a[k] = k < p.steps ? src[2 * k] : i32x4{};
#pragma unroll
      for (int i = 0; i < NS; ++i)
        sr[i] = 16 * i < p.sb ? reinterpret_cast<const i32x4*>(p.es + v * p.sb)[i] : i32x4{};
      mx4_lane_scales<NW>(sr, h, sa);
      f32x16 acc = {};
#pragma unroll
      for (int k = 0; k < KS; ++k) acc = mx4_step(k, a[k], sa, hf[rb][k], hs[rb], acc);
      const int ri = 4 * (col >> 3) + (col & 3);   // register of row col, in the lane half (col >> 2) & 1
      float z = acc[0];
#pragma unroll
      for (int r = 1; r < 16; ++r) z = ri == r ? acc[r] : z;
      const float z2 = __shfl_xor(z, 32);
      z = ((col >> 2) & 1) == h ? z : z2;
      // the exponent of the very term that the sum added (through exp2 and log2, so that a sum of that
      // term alone gives 0), but where the term is too small for a float
      const float x = exponent(rb, z);
      if (ok) sy = FIXED || x > -100.f ? flog2(fexp2(x)) : x;
    }
    if (h != 0 || tok >= n) continue;
    if (S == 1) {
      p.nats[row] = kLn2 * log2_ratio(l[rb], sy);
      if (p.lse) p.lse[row] = kLn2 * ((FIXED ? p.sc.M : m[rb]) + flog2(l[rb]));
    } else {
      const int64_t at = tok * mx4_split_stride(S) + split;
      p.part_l[at] = l[rb];
      if (!FIXED) p.part_m[at] = m[rb];
      if (split == 0) p.s_target[tok] = FIXED ? sy : m[rb] + sy;
    }
  }
}

// The splits' sums of each scored row: 16 lanes take four splits at a time each, then their sums are added in a
// fixed order. tile: vocabulary rows of a tile, which the splits count. One split has written its rows itself
// where `direct` says so.
constexpr int kMx4FinalLanes = 16, kMx4FinalRows = 256 / kMx4FinalLanes;
__global__ __launch_bounds__(256) void fwd_mx4_finalize_kernel(FwdMx4Params p, int tile, int fixed, int direct) {
  const int64_t n = p.n_dev ? (int64_t)(*p.n_dev) : p.n_host;
  const int S = mx4_splits(p, n, (p.V + tile - 1) / tile);
  if (p.mask) {   // rows that are left out
    for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < p.n_host; r += (int64_t)gridDim.x * blockDim.x) {
      if (p.mask[r]) continue;
      p.nats[r] = 0.f;
      if (p.lse) p.lse[r] = 0.f;
    }
  }
  if (direct && S == 1) return;
  const int stride = mx4_split_stride(S), lane = threadIdx.x % kMx4FinalLanes;
  for (int64_t i = (int64_t)blockIdx.x * kMx4FinalRows + threadIdx.x / kMx4FinalLanes; i < n;
       i += (int64_t)gridDim.x * kMx4FinalRows) {
    const float* pl = p.part_l + i * stride;
    const float* pm = p.part_m + i * stride;
    const float sy = p.s_target[i];
    const int64_t r = p.rows ? (int64_t)p.rows[i] : i;
    float m = fixed ? p.sc.M : -INFINITY, l = 0.f;   // M is the fixed shift's reference
    for (int s = 4 * lane; s < S; s += 4 * kMx4FinalLanes) {
      if (s + 4 <= S) {
        const float4 v = *reinterpret_cast<const float4*>(pl + s);
        if (fixed) {
          l += (v.x + v.y) + (v.z + v.w);
        } else {
          const float4 u = *reinterpret_cast<const float4*>(pm + s);
          lse_merge(m, l, u.x, v.x);
          lse_merge(m, l, u.y, v.y);
          lse_merge(m, l, u.z, v.z);
          lse_merge(m, l, u.w, v.w);
        }
      } else {   // the last splits, fewer than four
        for (int e = s; e < S; ++e) {
          if (fixed) l += pl[e];
          else lse_merge(m, l, pm[e], pl[e]);
        }
      }
    }
    if (fixed) {
      l = group_sum<kMx4FinalLanes>(l);
    } else {
#pragma unroll
      for (int off = 1; off < kMx4FinalLanes; off <<= 1) lse_merge(m, l, __shfl_xor(m, off), __shfl_xor(l, off));
    }
    if (lane != 0) continue;
    p.nats[r] = kLn2 * (fixed ? log2_ratio(l, sy) : not_below_zero(m + flog2(l) - sy));
    if (p.lse) p.lse[r] = kLn2 * (m + flog2(l));
  }
}

template <int KS, int RB>
static void launch_fwd_mx4_rb(const FwdMx4Params& p, hipStream_t st) {
  const dim3 grid = p.splits > 1 ? dim3(p.splits, p.grid / p.splits) : dim3(p.grid);
  if (p.sc.fixed) hipLaunchKernelGGL((fwd_mx4_kernel<KS, RB, kMx4Fixed>), grid, dim3(512), 0, st, p);
  else if (p.sc.c > 0.f) hipLaunchKernelGGL((fwd_mx4_kernel<KS, RB, kMx4Capped>), grid, dim3(512), 0, st, p);
  else hipLaunchKernelGGL((fwd_mx4_kernel<KS, RB, kMx4Uncapped>), grid, dim3(512), 0, st, p);
}

template <int KS>
static void launch_fwd_mx4_ks(const FwdMx4Params& p, hipStream_t st) {
  if constexpr (KS <= 8) {
    if (p.rows_per_wg == 256) return launch_fwd_mx4_rb<KS, 2>(p, st);
  }
  launch_fwd_mx4_rb<KS, 1>(p, st);
}

hipError_t launch_fwd_mx4(const uint8_t* hcodes, const uint8_t* hscales, const uint8_t* ecodes,
                          const uint8_t* escales, const int32_t* target, const uint8_t* mask, int64_t T, int32_t D,
                          int32_t V, float cap, float* nats, float* lse, char* ws, const DeviceInfo& dev,
                          hipStream_t st) {
  if (T == 0) return hipSuccess;
  const FwdWorkspace L = fwd_workspace(T, D, V);
  FwdMx4Params p{};
  p.hc = hcodes;
  p.hs = hscales;
  p.ec = ecodes;
  p.es = escales;
  p.target = target;
  p.n_host = T;
  p.cb = mx4_code_bytes(D);
  p.sb = mx4_scale_bytes(D);
  p.steps = (D + kMx4Step - 1) / kMx4Step;
  p.V = V;
  p.sc = Softcap::make(cap);
  p.nats = nats;
  p.lse = lse;
  p.part_l = reinterpret_cast<float*>(ws + L.part_l);
  p.part_m = reinterpret_cast<float*>(ws + L.part_m);
  p.s_target = reinterpret_cast<float*>(ws + L.s_target);
  if (mask) {
    p.rows = reinterpret_cast<int32_t*>(ws + L.rows);
    p.n_dev = reinterpret_cast<int32_t*>(ws + L.n_rows);
    if (p.steps <= 16 && T >= 16 && T <= kMx4MaskRows) {
      p.mask = mask;
    } else {
      hipError_t e = launch_compact_rows(mask, T, ws, L, nats, lse, st);
      if (e != hipSuccess) return e;
    }
  }
  // the partial sums' room: splits x rows stays within 1024 x 128 where there are splits, and the
  // workspace holds max(ceil(T / 256), 1024) x 256 of them
  const int ncu = dev.cu_count > 0 ? dev.cu_count : 256;
  int tile = 0, fixed = 0, direct = 0;
  p.rows_per_wg = 128;
  if (p.steps <= 16) {
    const bool wide = p.steps <= 8 && !mask && T >= (int64_t)256 * ncu;
    if (wide) p.rows_per_wg = 256;
    const int64_t rt = (T + p.rows_per_wg - 1) / p.rows_per_wg;
    int64_t slots = wide ? ncu : 2 * ncu;   // workgroups that run at once
    if (slots > 1024) slots = 1024;
    // where only the device knows the row count: one workgroup per CU (two that share it take as long, and
    // twice the splits are merged: 2048 rows 16.0 against 17.6 us)
    p.aim = ncu < 1024 ? ncu : 1024;
    p.grid = (int)(rt > p.aim ? rt : p.aim);
    if (!mask) {
      // The split that is done first, counted in hundredths of a tile's time on a CU that two workgroups
      // share: rounds of workgroups times the tiles of each and about one more that a start costs; a last
      // round of one workgroup per CU takes little more than half (one that owns its CU alone, of 64 rows per
      // wave, has no such sharing); merging the splits costs about three. Within the partial sums' room.
      const int ntiles = p.steps <= 8 ? (V + Mx4Tile<8>::kRows - 1) / Mx4Tile<8>::kRows
                                      : (V + Mx4Tile<16>::kRows - 1) / Mx4Tile<16>::kRows;
      int64_t best = INT64_MAX;
      for (int S = 1; S <= ntiles && S <= slots; S += S < 64 ? 1 : S) {   // every one up to 64, then powers of two
        if (S > 1 && T * mx4_split_stride(S) > fwd_partial_entries(T)) break;
        const int64_t wgs = rt * S, rounds = wgs / slots, rest = wgs % slots;
        const int64_t each = (ntiles + S - 1) / S + 1;
        const int64_t cost = (rounds * 100 + (rest == 0 ? 0 : !wide && rest <= ncu ? 55 : 100)) * each + (S > 1 ? 300 : 0);
        if (cost < best) {
          best = cost;
          p.splits = S;
        }
      }
      p.per = (ntiles + p.splits - 1) / p.splits;
      p.grid = (int)(rt * p.splits);   // several splits: at most 2^11 row tiles
    }
    fixed = p.sc.fixed;
    direct = 1;
    tile = p.steps <= 8 ? Mx4Tile<8>::kRows : Mx4Tile<16>::kRows;
    switch (p.steps) {
      case 1: launch_fwd_mx4_ks<1>(p, st); break;
      case 2: launch_fwd_mx4_ks<2>(p, st); break;
      case 3: launch_fwd_mx4_ks<3>(p, st); break;
      case 4: launch_fwd_mx4_ks<4>(p, st); break;
      case 5: launch_fwd_mx4_ks<5>(p, st); break;
      case 6: launch_fwd_mx4_ks<6>(p, st); break;
      case 7: launch_fwd_mx4_ks<7>(p, st); break;
      case 8: launch_fwd_mx4_ks<8>(p, st); break;
      case 9:
      case 10: launch_fwd_mx4_ks<10>(p, st); break;
      case 11:
      case 12: launch_fwd_mx4_ks<12>(p, st); break;
      default: launch_fwd_mx4_ks<16>(p, st); break;
    }
  } else {
    p.rows_per_wg = kMx4StreamRows;
    tile = kMx4StreamTile;
    const int64_t rt = (T + kMx4StreamRows - 1) / kMx4StreamRows;
    p.aim = 512;
    p.grid = (int)(rt > p.aim ? rt : p.aim);
    hipLaunchKernelGGL(fwd_mx4_stream_kernel, dim3(p.grid), dim3(256), 0, st, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (direct && !mask && mx4_splits(p, T, (V + tile - 1) / tile) == 1) return hipSuccess;
  hipLaunchKernelGGL(fwd_mx4_finalize_kernel, dim3(resident_blocks(dev, T, kMx4FinalRows)), dim3(256), 0, st, p, tile,
                     fixed, direct);
  return hipGetLastError();
}

}  // namespace pg
