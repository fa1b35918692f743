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

// The splits' sums of each scored row, in split order.
__global__ __launch_bounds__(256) void fwd_mx4_finalize_kernel(FwdMx4Params p) {
  const int64_t n = p.n_dev ? (int64_t)(*p.n_dev) : p.n_host;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int S = mx4_splits(n, p.nblocks, p.grid);
  float m = -INFINITY, l = 0.f;
  for (int s = 0; s < S; ++s) lse_merge(m, l, p.part_m[(int64_t)s * n + i], p.part_l[(int64_t)s * n + i]);
  const float lse2 = m + flog2(l);
  const int64_t r = p.rows ? (int64_t)p.rows[i] : i;
  p.nats[r] = kLn2 * (lse2 - p.s_target[i]);
  if (p.lse) p.lse[r] = kLn2 * lse2;
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
  p.grid = (int)(rt > 1024 ? rt : 1024);
  (void)dev;
  hipLaunchKernelGGL(fwd_mx4_stream_kernel, dim3(p.grid), dim3(256), 0, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fwd_mx4_finalize_kernel, dim3((unsigned)((T + 255) / 256)), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace pg
