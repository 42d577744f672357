// Host side of the gated scan and of the 8-bit checkpoints: argument checks,
// the checkpoint's layout and launches, for the files that define their entry
// points.
#pragma once

#include <cstdint>

#include "gated_scan.cuh"
#include "r2l.h"

#define R2L_TRY(x)                       \
  do {                                   \
    const r2l_status try_s_ = (x);       \
    if (try_s_ != R2L_OK) return try_s_; \
  } while (0)
#define R2L_LAUNCH_CHECK()                      \
  do {                                          \
    if (cudaPeekAtLastError() != cudaSuccess) { \
      (void)cudaGetLastError();                 \
      return R2L_ERR_CUDA;                      \
    }                                           \
  } while (0)

namespace r2l {
namespace gated {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool valid_dims(const r2l_dims* d, int B, int L) {
  return d && B > 0 && L > 0 && d->d_inner > 0 && (d->dtype == R2L_BF16 || d->dtype == R2L_FP32);
}
// Sizes whose byte counts stay far inside 64 bits, and padded widths and
// positions a few rounds past the end inside 32.
inline bool fits(int B, int L, int E) {
  return E <= (1 << 30) && L <= (1 << 30) && (double)B * L * E <= (double)(1ll << 50);
}
inline size_t elem_bytes(r2l_dtype t) { return t == R2L_BF16 ? 2 : 4; }

// Byte offsets of a checkpoint's parts.
struct CkptPlan {
  size_t states, q[3], scales[3], total;
  int tiles, Lp;
};
inline CkptPlan plan_checkpoint(const r2l_dims* d, int B, int L) {
  CkptPlan k{};
  const size_t strips = align_up(d->d_inner, STRIP) / STRIP;
  k.tiles = (L - 1) / TILE + 1;
  k.Lp = (int)align_up(L, 16);
  size_t off = 0;
  k.states = off;
  off = align_up(off + (size_t)B * k.tiles * strips * STRIP * sizeof(float), kAlign);
  if (d->flags & R2L_FLAG_ACT8)
    for (int i = 0; i < 3; ++i) {
      k.q[i] = off;
      off = align_up(off + B * strips * L * STRIP, kAlign);
      k.scales[i] = off;
      off = align_up(off + B * strips * k.Lp, kAlign);
    }
  k.total = off;
  return k;
}
inline Ckpt checkpoint_at(const CkptPlan& k, void* base) {
  char* c = (char*)base;
  Ckpt ck{};
  ck.states = (float*)(c + k.states);
  for (int i = 0; i < 3; ++i) {
    ck.q[i] = (uint8_t*)(c + k.q[i]);
    ck.scales[i] = (uint8_t*)(c + k.scales[i]);
  }
  ck.tiles = k.tiles;
  ck.Lp = k.Lp;
  return ck;
}

// Rows of E elements of `size` bytes with stride ld.
inline r2l_status check_rows(const void* p, int ld, int E, size_t size) {
  if (!p || ld < E) return R2L_ERR_INVALID_ARG;
  return aligned(p, size) ? R2L_OK : R2L_ERR_ALIGNMENT;
}

// Rows that start on 16-byte boundaries.
inline bool rows16(const void* p, long long ld, size_t size) { return aligned(p, 16) && ld * size % 16 == 0; }

// How a call is cut into blocks: warps of a block (4 or 8) and blocks of a
// cluster that share the channels of a sequence.
struct Split {
  uint32_t blocks;
  int warps;
};
// Clusters of blocks of 8 warps: the most blocks that clusters of 8, 4 and 2 may
// number (0: no such clusters).
struct Clusters {
  int of8, of4, of2;
};
// The largest clusters within these limits whose rounds stay within L.  A round
// of a cluster costs a barrier of about 1.2 us where single blocks hand the state
// from warp to warp, and clusters that cannot all run at once cost a second wave
// (a cluster lies within one of the chip's groups of SMs, so not every SM can be
// part of one): at two blocks an SM 256 blocks in clusters run at once.
// One sequence of 4096 x 512, 1024, 2048, 3040 and 4096 channels, bf16, scan:
//   single blocks  32.0  32.6  33.0  33.8  34.5 us
//   clusters of 2  36.2  37.1  38.8  46.0  47.9
//   clusters of 4  20.7  22.4  27.6  46.4  53.6
//   clusters of 8  15.0  17.2  31.7  47.1  61.7
// and its gradient:
//   single blocks  76.3  77.6  78.4  78.9  79.2
//   clusters of 2  53.3  53.9  55.3  74.4  75.7
//   clusters of 4  29.9  31.3  43.8  68.3  81.7
//   clusters of 8  24.2  27.0  51.1  71.0  91.3
inline uint32_t cluster_of(long long jobs, int rows, int L, Clusters most) {
  const int limits[] = {most.of8, most.of4, most.of2};
  uint32_t c = MAX_CLUSTER;
  for (int limit : limits) {
    if (jobs * c <= limit && (long long)rows * c < 2LL * L) return c;
    c /= 2;
  }
  return 1;
}

template <typename Args>
r2l_status launch(void (*kern)(Args, uint32_t), const Args& p, long long jobs, uint32_t blocks, int threads, size_t smem,
                  cudaStream_t st) {
  const long long grid = jobs * blocks;
  if (grid > 2147483647LL) return R2L_ERR_UNSUPPORTED;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return R2L_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, p, blocks) != cudaSuccess) {
    (void)cudaGetLastError();
    return R2L_ERR_CUDA;
  }
  return R2L_OK;
}

}  // namespace gated
}  // namespace r2l
