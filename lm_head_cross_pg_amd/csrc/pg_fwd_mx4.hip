// Forward of the fused tied head on 4-bit operands for gfx950: hidden states and embedding both in the
// microscaled 4-bit format (pg_mx4.h), their product by v_mfma_scale_f32_32x32x64_f8f6f4 (every value
// of both formats and every product of two is exact; the sum over D is float32), then the softcap,
// log-sum-exp and cross-entropy of the bf16 forward without the T x V logits ever reaching memory.
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
  const int32_t* rows;    // compacted scored rows, or nullptr (row i = i)
  const int32_t* n_dev;   // device row count, or nullptr (use n_host)
  int64_t n_host;
  int64_t cb, sb;         // bytes of a row of codes, of scales
  int steps;              // 64-value steps of a row
  int V;
  int nblocks;            // 32-row blocks of the vocabulary
  int grid;               // workgroups that share rows and splits
  Softcap sc;
  float* nats;
  float* lse;
  float* part_l;
  float* part_m;
  float* s_target;
};

// Rows of one workgroup: four waves of 32.
constexpr int kMx4RowsPerWG = 128;

// Vocabulary splits: as many as the grid has workgroups for each row tile, at most one per block.
__host__ __device__ __forceinline__ int mx4_splits(int64_t n, int nblocks, int grid) {
  const int64_t rt = (n + kMx4RowsPerWG - 1) / kMx4RowsPerWG;
  if (rt <= 0) return 1;
  const int64_t s = grid / rt;
  return s < 1 ? 1 : (s > nblocks ? nblocks : (int)s);
}

__device__ __forceinline__ f32x16 mfma_mx4(const i32x4& a, int sa, const i32x4& b, int sb, const f32x16& c) {
  const i32x8 aa = {a[0], a[1], a[2], a[3]}, bb = {b[0], b[1], b[2], b[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aa, bb, c, 4, 4, 0, sa, 0, sb);
}

// Any width: the wave's 32 rows and each block of 32 vocabulary rows meet step by step, both read from
// memory. Lane l holds row l % 32 of either side, the step's half l / 32, and its block's scale.
__global__ __launch_bounds__(256) void fwd_mx4_stream_kernel(FwdMx4Params p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, col = lane & 31;
  const int64_t n = p.n_dev ? (int64_t)(*p.n_dev) : p.n_host;
  const int S = mx4_splits(n, p.nblocks, p.grid);
  const int64_t rt = blockIdx.x / S;
  const int split = blockIdx.x % S;
  const int64_t tok0 = rt * kMx4RowsPerWG + wave * 32;
  if (tok0 >= n) return;
  const int per = (p.nblocks + S - 1) / S;
  const int b0 = split * per, b1 = min(b0 + per, p.nblocks);

  const int64_t tok = tok0 + col;
  const int64_t ic = tok < n ? tok : n - 1;
  const int64_t row = p.rows ? (int64_t)p.rows[ic] : ic;
  const uint8_t* hc = p.hc + row * p.cb + 16 * h;
  const uint8_t* hs = p.hs + row * p.sb + h;
  const int y = p.target[row];
  float m = -INFINITY, l = 0.f, sy = -INFINITY;
  for (int b = b0; b < b1; ++b) {
    const int64_t v = min(b * 32 + col, p.V - 1);
    const uint8_t* ec = p.ec + v * p.cb + 16 * h;
    const uint8_t* es = p.es + v * p.sb + h;
    f32x16 acc = {};
    for (int k = 0; k < p.steps; ++k)
      acc = mfma_mx4(*reinterpret_cast<const i32x4*>(ec + 32 * k), es[2 * k], *reinterpret_cast<const i32x4*>(hc + 32 * k),
                     hs[2 * k], acc);
    // register r: vocabulary row 8 (r / 4) + 4 h + r % 4 of the block
    float s2[16], bm = -INFINITY;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int vr = b * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
      s2[r] = vr < p.V ? capped_log2(acc[r], p.sc) : -INFINITY;
      bm = fmaxf(bm, s2[r]);
      if (vr == y && vr < p.V) sy = s2[r];
    }
    const float mn = fmaxf(m, bm);
    if (mn != -INFINITY) {
      float part = 0.f;
#pragma unroll
      for (int r = 0; r < 16; ++r) part += fexp2(s2[r] - mn);
      l = l * fexp2(m - mn) + part;
      m = mn;
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) l += s2[r] != s2[r] ? s2[r] : 0.f;   // NaN rows stay NaN
    }
  }
  lse_merge(m, l, __shfl_xor(m, 32), __shfl_xor(l, 32));
  const float sy2 = __shfl_xor(sy, 32);
  const bool here = y >= b0 * 32 && y < b1 * 32 && y < p.V;   // this split holds the target's row
  if (h == 0 && tok < n) {
    p.part_l[(int64_t)split * n + tok] = l;
    p.part_m[(int64_t)split * n + tok] = m;
    if (here) p.s_target[tok] = ((y >> 2) & 1) ? sy2 : sy;
    else if (split == 0 && !(y >= 0 && y < p.V)) p.s_target[tok] = __builtin_nanf("");
  }
}

// ---------------------------------------------------------------------- widths up to 1024
//
// A workgroup of eight waves owns 128 rows: waves w and w + 4 hold the same 32 rows' codes and scales in
// registers (the B operand) and take the even and the odd 32-row blocks of each vocabulary tile. The
// tiles stream through LDS, two buffers, copied there by DMA while the tile before is worked on; every
// wave reads the fragments of its blocks from LDS (the A operand). An accumulator holds 16 vocabulary
// rows of one token per lane, so the softcap and the sum of exponentials run per lane.
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

// acc = the 32 x 32 logits of fragments a against the rows hf, step after step.
template <int KS, int NW, int K = 0>
__device__ __forceinline__ void mx4_chain(const i32x4 (&a)[KS], const int (&sa)[NW], const i32x4 (&hf)[KS],
                                          const int (&hs)[NW], f32x16& acc) {
  if constexpr (K < KS) {
    acc = mfma_mx4_op<K & 3>(a[K], sa[K >> 2], hf[K], hs[K >> 2], acc);
    mx4_chain<KS, NW, K + 1>(a, sa, hf, hs, acc);
  }
}

template <int KS, bool FIXED>
__global__ __launch_bounds__(512, KS <= 8 ? 4 : 2) void fwd_mx4_kernel(FwdMx4Params p) {
  using TL = Mx4Tile<KS>;
  constexpr int NW = (KS + 3) / 4;          // words of a lane's scales
  constexpr int NS = TL::kScaleBytes / 16;
  __shared__ __attribute__((aligned(1024))) char smem[2 * TL::kBytes];
  __shared__ float merge[2][4][32];
  const lds_char* lds = (const lds_char*)smem;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, col = lane & 31;
  const int64_t n = p.n_dev ? (int64_t)(*p.n_dev) : p.n_host;
  const int ntiles = (p.V + TL::kRows - 1) / TL::kRows;
  const int S = mx4_splits(n, ntiles, p.grid);
  const int64_t rt = blockIdx.x / S;
  const int split = blockIdx.x % S;
  if (rt * kMx4RowsPerWG >= n) return;
  const int per = (ntiles + S - 1) / S;
  const int t0 = split * per, t1 = min(t0 + per, ntiles);

  // this wave's part of a tile: kLoads pieces of codes (piece j: 1 KiB, lane i its 16 bytes at 16 i),
  // and of the scales, which the first waves copy
  constexpr int RPI = 1024 / TL::kRowBytes;   // rows of a piece
  const int prow = lane / TL::CPR;            // row in a piece; swizzle(row) is the same for all of a wave's pieces
  int lchunk = (lane % TL::CPR) ^ TL::swizzle(wave * RPI + prow);
  if (lchunk >= 2 * p.steps) lchunk = 0;      // not in the rows (read by no one, or against zero states)
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  constexpr int kScaleLoads = TL::kRows * TL::kScaleBytes / 1024;   // 1 KiB pieces of scales
  constexpr int SPR = TL::kScaleBytes / 16, SRPI = 64 / SPR;        // 16-byte parts of a row, rows of a piece
  int spart = lane % SPR;
  if (16 * spart >= p.sb) spart = 0;
  auto load_tile = [&](int tile, int buf) {
    const int v0 = tile * TL::kRows;
    const uint32_t dst = lds0 + buf * TL::kBytes;
    const uint8_t* cbase = p.ec + (int64_t)v0 * p.cb;
    const uint8_t* sbase = p.es + (int64_t)v0 * p.sb;
    const int last = p.V - 1 - v0;            // rows past the vocabulary repeat its last one
#pragma unroll
    for (int q = 0; q < TL::kLoads; ++q) {
      const int j = wave + 8 * q;
      if (TL::kPieces % 8 != 0 && j >= TL::kPieces) break;
      const int row = min(j * RPI + prow, last);
      lds_dma16_base(cbase, (uint32_t)(row * (int)p.cb + 16 * lchunk), dst + 1024 * j);
    }
    if (wave < kScaleLoads) {
      const int row = min(wave * SRPI + lane / SPR, last);
      lds_dma16_base(sbase, (uint32_t)(row * (int)p.sb + 16 * spart), dst + TL::kCodes + 1024 * wave);
    }
  };
  if (t0 < t1) load_tile(t0, 0);

  // the rows of this wave: codes, scales and target
  const int rg = wave & 3, half = wave >> 2;
  const int64_t tok = rt * kMx4RowsPerWG + rg * 32 + col;
  const int64_t ic = tok < n ? tok : n - 1;
  const int64_t row = p.rows ? (int64_t)p.rows[ic] : ic;
  i32x4 hf[KS];
  int hs[NW];
  {
    const i32x4* src = reinterpret_cast<const i32x4*>(p.hc + row * p.cb + 16 * h);
#pragma unroll
    for (int k = 0; k < KS; ++k) hf[k] = k < p.steps ? src[2 * k] : i32x4{};
    i32x4 sr[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
      sr[i] = 16 * i < p.sb ? reinterpret_cast<const i32x4*>(p.hs + row * p.sb)[i] : i32x4{};
    mx4_lane_scales<NW>(sr, h, hs);
  }

  float l = 0.f, m = -INFINITY;
  // (s log2 e) - M of a logit with the fixed shift, else s log2 e
  auto exponent = [&](float z) { return FIXED ? capped_shifted(z, p.sc.alpha, p.sc.invK) : capped_log2(z, p.sc); };
  // the sums of a block whose first vocabulary row is vbase (register r: row 8 (r / 4) + 4 h + r % 4)
  auto add_block = [&](const f32x16& acc, int vbase, bool whole) {
    if constexpr (FIXED) {
      float part = 0.f;
      if (whole) {
#pragma unroll
        for (int r = 0; r < 16; ++r) part += fexp2(exponent(acc[r]));
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float e = fexp2(exponent(acc[r]));
          part += vbase + 8 * (r >> 2) + 4 * h + (r & 3) < p.V ? e : 0.f;
        }
      }
      l += part;
    } else {
      float s2[16], bm = -INFINITY, nan = 0.f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s2[r] = whole || vbase + 8 * (r >> 2) + 4 * h + (r & 3) < p.V ? exponent(acc[r]) : -INFINITY;
        bm = fmaxf(bm, s2[r]);
        nan += s2[r] != s2[r] ? s2[r] : 0.f;
      }
      const float mn = fmaxf(m, bm);
      if (mn != -INFINITY) {
        float part = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r) part += fexp2(s2[r] - mn);
        l = l * fexp2(m - mn) + part;
        m = mn;
      } else {
        l += nan;
      }
    }
  };

  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's part of tile t has landed
    __syncthreads();                                   // and everyone's; the other buffer is free
    if (t + 1 < t1) load_tile(t + 1, buf ^ 1);
    const lds_char* tile = lds + buf * TL::kBytes;
#pragma unroll
    for (int b = 0; b < TL::kBlocksPerWave; ++b) {
      const int r0 = (2 * b + half) * 32;
      const int vbase = t * TL::kRows + r0;
      if (vbase >= p.V) continue;
      const int lrow = r0 + col;
      const int sw = TL::swizzle(lrow);
      i32x4 a[KS], sr[NS];
      int sa[NW];
#pragma unroll
      for (int i = 0; i < NS; ++i)
        sr[i] = *(const __attribute__((address_space(3))) i32x4*)(tile + TL::kCodes + lrow * TL::kScaleBytes + 16 * i);
#pragma unroll
      for (int k = 0; k < KS; ++k)
        a[k] = *(const __attribute__((address_space(3))) i32x4*)(tile + lrow * TL::kRowBytes + (((2 * k + h) ^ sw) * 16));
      mx4_lane_scales<NW>(sr, h, sa);
      f32x16 acc = {};
      mx4_chain<KS, NW>(a, sa, hf, hs, acc);
      add_block(acc, vbase, vbase + 32 <= p.V);
    }
  }

  // the other half of the lanes, then the other wave of these rows
  lse_merge(m, l, __shfl_xor(m, 32), __shfl_xor(l, 32));
  if (half == 1 && h == 0) {
    merge[0][rg][col] = m;
    merge[1][rg][col] = l;
  }
  __syncthreads();
  if (half == 1) return;
  if constexpr (FIXED) l += merge[1][rg][col];
  else lse_merge(m, l, merge[0][rg][col], merge[1][rg][col]);

  // The targets' logits: the wave's 32 target rows as the A operand, whose product with its 32 tokens
  // has them on the diagonal, formed by the same instructions from the same values as the sum's.
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
    mx4_chain<KS, NW>(a, sa, hf, hs, acc);
    const int ri = 4 * (col >> 3) + (col & 3);   // register of row col, in the lane half (col >> 2) & 1
    float z = acc[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) z = ri == r ? acc[r] : z;
    const float z2 = __shfl_xor(z, 32);
    z = ((col >> 2) & 1) == h ? z : z2;
    // with the fixed shift, log2 of the very term that the sum added
    if (ok) sy = FIXED ? flog2(fexp2(exponent(z))) : exponent(z);
  }
  if (h != 0 || tok >= n) return;
  if (S == 1) {
    const float lse2 = (FIXED ? p.sc.M : m) + flog2(l);
    p.nats[row] = kLn2 * (FIXED ? log2_ratio(l, sy) : lse2 - sy);
    if (p.lse) p.lse[row] = kLn2 * lse2;
  } else {
    p.part_l[(int64_t)split * n + tok] = l;
    if (!FIXED) p.part_m[(int64_t)split * n + tok] = m;
    if (split == 0) p.s_target[tok] = sy;
  }
}

// The splits' sums of each scored row, in split order. tile: vocabulary rows of a tile, which the
// splits count. One split has written its rows itself where `direct` says so.
__global__ __launch_bounds__(256) void fwd_mx4_finalize_kernel(FwdMx4Params p, int tile, int fixed, int direct) {
  const int64_t n = p.n_dev ? (int64_t)(*p.n_dev) : p.n_host;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int S = mx4_splits(n, (p.V + tile - 1) / tile, p.grid);
  if (direct && S == 1) return;
  const int64_t r = p.rows ? (int64_t)p.rows[i] : i;
  if (fixed) {
    float l = 0.f;
    for (int s = 0; s < S; ++s) l += p.part_l[(int64_t)s * n + i];
    p.nats[r] = kLn2 * log2_ratio(l, p.s_target[i]);
    if (p.lse) p.lse[r] = kLn2 * (p.sc.M + flog2(l));
    return;
  }
  float m = -INFINITY, l = 0.f;
  for (int s = 0; s < S; ++s) lse_merge(m, l, p.part_m[(int64_t)s * n + i], p.part_l[(int64_t)s * n + i]);
  const float lse2 = m + flog2(l);
  p.nats[r] = kLn2 * (lse2 - p.s_target[i]);
  if (p.lse) p.lse[r] = kLn2 * lse2;
}

template <int KS>
static void launch_fwd_mx4_ks(const FwdMx4Params& p, hipStream_t st) {
  if (p.sc.fixed) hipLaunchKernelGGL((fwd_mx4_kernel<KS, true>), dim3(p.grid), dim3(512), 0, st, p);
  else hipLaunchKernelGGL((fwd_mx4_kernel<KS, false>), dim3(p.grid), dim3(512), 0, st, p);
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
  p.nblocks = (V + 31) / 32;
  p.sc = Softcap::make(cap);
  p.nats = nats;
  p.lse = lse;
  p.part_l = reinterpret_cast<float*>(ws + L.part_l);
  p.part_m = reinterpret_cast<float*>(ws + L.part_m);
  p.s_target = reinterpret_cast<float*>(ws + L.s_target);
  if (mask) {
    hipError_t e = launch_compact_rows(mask, T, ws, L, nats, lse, st);
    if (e != hipSuccess) return e;
    p.rows = reinterpret_cast<const int32_t*>(ws + L.rows);
    p.n_dev = reinterpret_cast<const int32_t*>(ws + L.n_rows);
  }
  // the partial sums' room: splits x rows stays within grid x 128, and the workspace holds
  // max(ceil(T / 256), 1024) x 256 of them
  const int64_t rt = (T + kMx4RowsPerWG - 1) / kMx4RowsPerWG;
  const int ncu = dev.cu_count > 0 ? dev.cu_count : 256;
  int tile = 32, fixed = 0, direct = 0;
  if (p.steps <= 16) {
    const int64_t slots = 2 * ncu < 1024 ? 2 * ncu : 1024;   // workgroups that run at once
    p.grid = (int)(rt > slots ? rt : slots);
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
    p.grid = (int)(rt > 1024 ? rt : 1024);
    hipLaunchKernelGGL(fwd_mx4_stream_kernel, dim3(p.grid), dim3(256), 0, st, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (direct && !mask && mx4_splits(T, (V + tile - 1) / tile, p.grid) == 1) return hipSuccess;
  hipLaunchKernelGGL(fwd_mx4_finalize_kernel, dim3((unsigned)((T + 255) / 256)), dim3(256), 0, st, p, tile, fixed,
                     direct);
  return hipGetLastError();
}

}  // namespace pg
