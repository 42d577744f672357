// The gated linear recurrence (r2l_gated_scan, its training forward and its
// gradient) and the 8-bit activation checkpoints (r2l_act8_pack / _unpack):
// kernels, argument checks and launches.
#include <algorithm>
#include <cstdint>

#include "act8.cuh"
#include "common.cuh"
#include "gated_bwd.cuh"
#include "gated_scan.cuh"
#include "r2l.h"

using r2l::bf16;
using r2l::from_f32;
using r2l::to_f32;
using r2l::gated::BwdArgs;
using r2l::gated::Ckpt;
using r2l::gated::clamped_length;
using r2l::gated::FwdArgs;
using r2l::gated::MAX_CLUSTER;

namespace {

constexpr int TILE = R2L_GATED_TILE;
constexpr int GROUP = R2L_ACT8_GROUP;
constexpr size_t kAlign = 256;

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

#define R2L_LAUNCH_CHECK()                  \
  do {                                      \
    if (cudaPeekAtLastError() != cudaSuccess) { \
      (void)cudaGetLastError();             \
      return R2L_ERR_CUDA;                  \
    }                                       \
  } while (0)

// A warp per (row, group), two channels a lane.
template <typename T>
__global__ void act8_pack_kernel(const T* x, long long ldx, int B, int L, int cols, const int32_t* lengths, uint8_t* q,
                                 long long ldq, uint8_t* scales) {
  const int groups = (cols + GROUP - 1) / GROUP, lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (w >= (long long)B * L * groups) return;
  const long long m = w / groups;
  const int gr = (int)(w % groups), b = (int)(m / L);
  if ((int)(m % L) >= clamped_length(lengths, b, L)) return;
  float v[2];
  uint32_t top = 0;
  for (int j = 0; j < 2; ++j) {
    const int c = gr * GROUP + 2 * lane + j;
    v[j] = c < cols ? to_f32(x[m * ldx + c]) : 0.0f;
    top = max(top, r2l::act8::finite_abs_bits(v[j]));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const uint32_t byte = r2l::act8::scale_byte(top);
  const float down = r2l::act8::scale_down(byte);
  const uint16_t two = r2l::act8::to_e4m3x2(r2l::act8::nan_if_not_finite(v[0]) * down,
                                            r2l::act8::nan_if_not_finite(v[1]) * down);
  for (int j = 0; j < 2; ++j) {
    const int c = gr * GROUP + 2 * lane + j;
    if (c < cols) q[m * ldq + c] = (uint8_t)(two >> (8 * j));
  }
  if (lane == 0) scales[m * groups + gr] = (uint8_t)byte;
}

template <typename T>
__global__ void act8_unpack_kernel(const uint8_t* q, long long ldq, const uint8_t* scales, int B, int L, int cols,
                                   const int32_t* lengths, T* out, long long ldo) {
  const int groups = (cols + GROUP - 1) / GROUP;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)B * L * cols) return;
  const long long m = i / cols;
  const int c = (int)(i % cols), b = (int)(m / L);
  if ((int)(m % L) >= clamped_length(lengths, b, L)) return;
  out[m * ldo + c] =
      from_f32<T>(r2l::act8::from_e4m3x2(q[m * ldq + c]).x * r2l::act8::scale_up(scales[m * groups + c / GROUP]));
}

// ------------------------------------------------------------------ host

bool valid_dims(const r2l_dims* d, int B, int L) {
  return d && B > 0 && L > 0 && d->d_inner > 0 && (d->dtype == R2L_BF16 || d->dtype == R2L_FP32);
}
// Sizes whose byte counts stay far inside 64 bits, and padded widths inside 32.
bool fits(int B, int L, int E) {
  return E <= (1 << 30) && (double)B * L * E <= (double)(1ll << 50);
}
size_t elem_bytes(r2l_dtype t) { return t == R2L_BF16 ? 2 : 4; }

// Byte offsets of a checkpoint's parts.
struct CkptPlan {
  size_t states, q[3], scales[3], total;
  int tiles, Lp;
};
CkptPlan plan_checkpoint(const r2l_dims* d, int B, int L) {
  CkptPlan k{};
  const size_t strips = align_up(d->d_inner, GROUP) / GROUP;
  k.tiles = (L - 1) / TILE + 1;
  k.Lp = (int)align_up(L, 16);
  size_t off = 0;
  k.states = off;
  off = align_up(off + B * k.tiles * strips * GROUP * sizeof(float), kAlign);
  if (d->flags & R2L_FLAG_ACT8)
    for (int i = 0; i < 3; ++i) {
      k.q[i] = off;
      off = align_up(off + B * strips * L * GROUP, kAlign);
      k.scales[i] = off;
      off = align_up(off + B * strips * k.Lp, kAlign);
    }
  k.total = off;
  return k;
}
Ckpt checkpoint_at(const CkptPlan& k, void* base) {
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

// Blocks of a cluster that share a sequence's channels, and warps of a block.
struct Split {
  uint32_t blocks;
  int warps;
};
Split split(long long jobs, int L, int small, int large, int resident) {
  const int tiles = (L - 1) / TILE + 1;
  Split s{1, small};
  return s;
}

template <typename Args>
r2l_status launch(void (*kern)(Args, uint32_t), const Args& p, long long jobs, uint32_t blocks, int threads, size_t smem,
                  cudaStream_t st) {
  const long long grid = jobs * blocks;
  if (grid > 2147483647LL) return R2L_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
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
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p, blocks) != cudaSuccess) {
    (void)cudaGetLastError();
    return R2L_ERR_CUDA;
  }
  return R2L_OK;
}

// Rows that start on 16-byte boundaries.
bool rows16(const void* p, long long ld, size_t size) { return aligned(p, 16) && ld * size % 16 == 0; }

template <typename T, bool VEC>
r2l_status run_forward(const FwdArgs& p, int mode, cudaStream_t st) {
  using namespace r2l::gated;
  if (mode == 0 && p.L <= WALK_MAX) {
    const long long grid = ((long long)p.B * ((p.E + 1) / 2) + 127) / 128;
    if (grid > 2147483647LL) return R2L_ERR_UNSUPPORTED;
    gated_walk_kernel<T, VEC><<<(unsigned)grid, 128, 0, st>>>(p);
    R2L_LAUNCH_CHECK();
    return R2L_OK;
  }
  if (mode == 2) {
    const long long jobs = (long long)p.B * p.strips;
    const Split c = split(jobs, p.L, 8, 32, 0);
    return launch(gated_scan_kernel<T, VEC, 2, 32, 8>, p, jobs, c.blocks, 256, fwd_smem_bytes<T, 32, 8>(c.blocks), st);
  }
  const long long jobs = (long long)p.B * ((p.E - 1) / 32 + 1);
  const Split c = split(jobs, p.L, 4, 16, 0);
  if (sizeof(T) == 4 || c.warps == 4)
    return launch(mode == 0 ? gated_scan_kernel<T, VEC, 0, 16, 4> : gated_scan_kernel<T, VEC, 1, 16, 4>, p, jobs, c.blocks, 128,
                  fwd_smem_bytes<T, 16, 4>(c.blocks), st);
  return launch(mode == 0 ? gated_scan_kernel<T, VEC, 0, 16, 16> : gated_scan_kernel<T, VEC, 1, 16, 16>, p, jobs, c.blocks, 512,
                fwd_smem_bytes<T, 16, 16>(c.blocks), st);
}

Split backward_split(const r2l_dims* d, int B, int L) {
  return split((long long)B * ((d->d_inner - 1) / 32 + 1), L, 4, 16, 0);
}

template <typename T, bool VEC, bool ACT8>
r2l_status run_backward(const BwdArgs& p, Split c, cudaStream_t st) {
  using namespace r2l::gated;
  const long long jobs = (long long)p.B * ((p.E - 1) / 32 + 1);
  return launch(gated_bwd_kernel<T, VEC, ACT8, 4>, p, jobs, c.blocks, 128, bwd_smem_bytes<T, ACT8, 4>(c.blocks), st);
}

// Rows of E elements of `size` bytes with stride ld.
r2l_status check_rows(const void* p, int ld, int E, size_t size) {
  if (!p || ld < E) return R2L_ERR_INVALID_ARG;
  return aligned(p, size) ? R2L_OK : R2L_ERR_ALIGNMENT;
}

#define R2L_TRY(x)                   \
  do {                               \
    const r2l_status try_s_ = (x);   \
    if (try_s_ != R2L_OK) return try_s_; \
  } while (0)

r2l_status act8_pack(const void* x, long long ldx, r2l_dtype dtype, int B, int L, int cols, const int32_t* lengths,
                     uint8_t* q, long long ldq, uint8_t* scales, cudaStream_t st) {
  const long long warps = (long long)B * L * ((cols + GROUP - 1) / GROUP);
  const long long blocks = (warps + 7) / 8;
  if (blocks > 2147483647LL) return R2L_ERR_UNSUPPORTED;
  if (dtype == R2L_BF16)
    act8_pack_kernel<bf16><<<(unsigned)blocks, 256, 0, st>>>((const bf16*)x, ldx, B, L, cols, lengths, q, ldq, scales);
  else
    act8_pack_kernel<float><<<(unsigned)blocks, 256, 0, st>>>((const float*)x, ldx, B, L, cols, lengths, q, ldq, scales);
  R2L_LAUNCH_CHECK();
  return R2L_OK;
}

r2l_status forward_impl(const r2l_gated_in* in, void* y, int ldy, float* h_last, const r2l_dims* dims, int B, int L,
                        const int32_t* lengths, bool train, void* checkpoint, size_t checkpoint_bytes,
                        uint32_t* status, void* stream) {
  if (!in || !valid_dims(dims, B, L)) return R2L_ERR_INVALID_ARG;
  const int E = dims->d_inner;
  const size_t es = elem_bytes(dims->dtype);
  if (!in->lam || y == in->x || y == in->r || y == in->g) return R2L_ERR_INVALID_ARG;
  R2L_TRY(check_rows(in->x, in->ldx, E, es));
  R2L_TRY(check_rows(in->r, in->ldr, E, es));
  R2L_TRY(check_rows(in->g, in->ldg, E, es));
  R2L_TRY(check_rows(y, ldy, E, es));
  if (!aligned(in->lam, 4) || !aligned(in->h0, 4) || !aligned(h_last, 4) || !aligned(lengths, 4) ||
      !aligned(status, 4))
    return R2L_ERR_ALIGNMENT;
  if (!fits(B, L, E)) return R2L_ERR_UNSUPPORTED;
  FwdArgs p{};
  p.x = in->x; p.r = in->r; p.g = in->g;
  p.ldx = in->ldx; p.ldr = in->ldr; p.ldg = in->ldg; p.ldy = ldy;
  p.lam = in->lam; p.h0 = in->h0; p.y = y; p.h_last = h_last;
  p.B = B; p.L = L; p.E = E; p.strips = (E - 1) / GROUP + 1;
  p.forward = (dims->flags & R2L_FLAG_FORWARD_SCAN) ? 1 : 0;
  p.lengths = lengths; p.status = status;
  if (train) {
    const CkptPlan k = plan_checkpoint(dims, B, L);
    if (!checkpoint || checkpoint_bytes < k.total) return R2L_ERR_WORKSPACE;
    if (!aligned(checkpoint, 16)) return R2L_ERR_ALIGNMENT;
    p.ck = checkpoint_at(k, checkpoint);
  }
  const int mode = !train ? 0 : (dims->flags & R2L_FLAG_ACT8) ? 2 : 1;
  const bool vec = rows16(p.x, p.ldx, es) && rows16(p.r, p.ldr, es) && rows16(p.g, p.ldg, es) && rows16(p.y, p.ldy, es);
  cudaStream_t st = (cudaStream_t)stream;
  if (dims->dtype == R2L_BF16) return vec ? run_forward<bf16, true>(p, mode, st) : run_forward<bf16, false>(p, mode, st);
  return vec ? run_forward<float, true>(p, mode, st) : run_forward<float, false>(p, mode, st);
}

// Shares of dlam, one row for each block of channels' blocks.
size_t part_bytes(const r2l_dims* d, int B, int L) {
  return (size_t)B * backward_split(d, B, L).blocks * align_up(d->d_inner, GROUP) * sizeof(float);
}

}  // namespace

extern "C" {

r2l_status r2l_gated_scan(const r2l_gated_in* in, void* y, int ldy, float* h_last, const r2l_dims* dims, int B, int L,
                          const int32_t* lengths, uint32_t* status, void* stream) {
  return forward_impl(in, y, ldy, h_last, dims, B, L, lengths, false, nullptr, 0, status, stream);
}

size_t r2l_gated_scan_checkpoint_size(const r2l_dims* dims, int B, int L) {
  return valid_dims(dims, B, L) && fits(B, L, dims->d_inner) ? plan_checkpoint(dims, B, L).total : 0;
}

r2l_status r2l_gated_scan_train(const r2l_gated_in* in, void* y, int ldy, float* h_last, const r2l_dims* dims, int B,
                                int L, const int32_t* lengths, void* checkpoint, size_t checkpoint_bytes,
                                uint32_t* status, void* stream) {
  return forward_impl(in, y, ldy, h_last, dims, B, L, lengths, true, checkpoint, checkpoint_bytes, status, stream);
}

size_t r2l_gated_scan_backward_workspace_size(const r2l_dims* dims, int B, int L) {
  return valid_dims(dims, B, L) && fits(B, L, dims->d_inner) ? kAlign + align_up(part_bytes(dims, B, L), kAlign) : 0;
}

r2l_status r2l_gated_scan_backward(const r2l_gated_in* in, const void* dy, int ld_dy, const float* dh_last,
                                   const r2l_gated_grads* grads, const r2l_dims* dims, int B, int L,
                                   const int32_t* lengths, const void* checkpoint, size_t checkpoint_bytes,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!in || !grads || !valid_dims(dims, B, L)) return R2L_ERR_INVALID_ARG;
  const int E = dims->d_inner;
  const size_t es = elem_bytes(dims->dtype);
  const bool act8 = (dims->flags & R2L_FLAG_ACT8) != 0;
  if (!in->lam || !grads->dlam) return R2L_ERR_INVALID_ARG;
  if (!act8) {
    R2L_TRY(check_rows(in->x, in->ldx, E, es));
    R2L_TRY(check_rows(in->r, in->ldr, E, es));
    R2L_TRY(check_rows(in->g, in->ldg, E, es));
  }
  R2L_TRY(check_rows(dy, ld_dy, E, es));
  R2L_TRY(check_rows(grads->dx, grads->ld_dx, E, es));
  R2L_TRY(check_rows(grads->dr, grads->ld_dr, E, es));
  R2L_TRY(check_rows(grads->dg, grads->ld_dg, E, es));
  const void* reads[] = {dy, act8 ? nullptr : in->x, act8 ? nullptr : in->r, act8 ? nullptr : in->g};
  const void* writes[] = {grads->dx, grads->dr, grads->dg};
  for (int i = 0; i < 3; ++i) {
    for (const void* q : reads)
      if (writes[i] == q) return R2L_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (writes[i] == writes[j]) return R2L_ERR_INVALID_ARG;
  }
  if (!aligned(in->lam, 4) || !aligned(dh_last, 4) || !aligned(grads->dlam, 4) || !aligned(grads->dh0, 4) ||
      !aligned(lengths, 4))
    return R2L_ERR_ALIGNMENT;
  if (!fits(B, L, E)) return R2L_ERR_UNSUPPORTED;
  const CkptPlan k = plan_checkpoint(dims, B, L);
  if (!checkpoint || checkpoint_bytes < k.total) return R2L_ERR_WORKSPACE;
  if (!workspace || workspace_bytes < r2l_gated_scan_backward_workspace_size(dims, B, L)) return R2L_ERR_WORKSPACE;
  if (!aligned(checkpoint, 16) || !aligned(workspace, 16)) return R2L_ERR_ALIGNMENT;
  BwdArgs p{};
  p.x = in->x; p.r = in->r; p.g = in->g; p.dy = dy;
  p.ldx = in->ldx; p.ldr = in->ldr; p.ldg = in->ldg; p.ld_dy = ld_dy;
  p.dx = grads->dx; p.dr = grads->dr; p.dg = grads->dg;
  p.ld_dx = grads->ld_dx; p.ld_dr = grads->ld_dr; p.ld_dg = grads->ld_dg;
  p.lam = in->lam; p.dh_last = dh_last; p.dh0 = grads->dh0;
  p.part = (float*)((char*)workspace + kAlign);
  p.B = B; p.L = L; p.E = E; p.strips = (E - 1) / GROUP + 1;
  p.forward = (dims->flags & R2L_FLAG_FORWARD_SCAN) ? 1 : 0;
  p.lengths = lengths; p.status = (uint32_t*)workspace;
  p.ck = checkpoint_at(k, const_cast<void*>(checkpoint));
  const bool vec = (act8 || (rows16(p.x, p.ldx, es) && rows16(p.r, p.ldr, es) && rows16(p.g, p.ldg, es))) &&
                   rows16(p.dy, p.ld_dy, es) && rows16(p.dx, p.ld_dx, es) && rows16(p.dr, p.ld_dr, es) &&
                   rows16(p.dg, p.ld_dg, es);
  const Split c = backward_split(dims, B, L);
  cudaStream_t st = (cudaStream_t)stream;
  if (dims->dtype == R2L_BF16) {
    if (act8) R2L_TRY((vec ? run_backward<bf16, true, true> : run_backward<bf16, false, true>)(p, c, st));
    else R2L_TRY((vec ? run_backward<bf16, true, false> : run_backward<bf16, false, false>)(p, c, st));
  } else {
    if (act8) R2L_TRY((vec ? run_backward<float, true, true> : run_backward<float, false, true>)(p, c, st));
    else R2L_TRY((vec ? run_backward<float, true, false> : run_backward<float, false, false>)(p, c, st));
  }
  r2l::gated::gated_dlam_kernel<<<(E + 31) / 32, 256, 0, st>>>(p.part, (int)(B * c.blocks), p.strips * GROUP, p.lam, E, grads->dlam);
  R2L_LAUNCH_CHECK();
  return R2L_OK;
}

r2l_status r2l_act8_pack(const void* x, int ldx, r2l_dtype dtype, int B, int L, int cols, const int32_t* lengths,
                         uint8_t* q, int ldq, uint8_t* scales, void* stream) {
  if (B <= 0 || L <= 0 || cols <= 0 || (dtype != R2L_BF16 && dtype != R2L_FP32) || !scales)
    return R2L_ERR_INVALID_ARG;
  R2L_TRY(check_rows(x, ldx, cols, elem_bytes(dtype)));
  R2L_TRY(check_rows(q, ldq, cols, 1));
  if (!aligned(lengths, 4)) return R2L_ERR_ALIGNMENT;
  return act8_pack(x, ldx, dtype, B, L, cols, lengths, q, ldq, scales, (cudaStream_t)stream);
}

r2l_status r2l_act8_unpack(const uint8_t* q, int ldq, const uint8_t* scales, r2l_dtype dtype, int B, int L, int cols,
                           const int32_t* lengths, void* out, int ldo, void* stream) {
  if (B <= 0 || L <= 0 || cols <= 0 || (dtype != R2L_BF16 && dtype != R2L_FP32) || !scales)
    return R2L_ERR_INVALID_ARG;
  R2L_TRY(check_rows(q, ldq, cols, 1));
  R2L_TRY(check_rows(out, ldo, cols, elem_bytes(dtype)));
  if (!aligned(lengths, 4)) return R2L_ERR_ALIGNMENT;
  const long long blocks = ((long long)B * L * cols + 255) / 256;
  if (blocks > 2147483647LL) return R2L_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == R2L_BF16)
    act8_unpack_kernel<bf16><<<(unsigned)blocks, 256, 0, st>>>(q, ldq, scales, B, L, cols, lengths, (bf16*)out, ldo);
  else
    act8_unpack_kernel<float><<<(unsigned)blocks, 256, 0, st>>>(q, ldq, scales, B, L, cols, lengths, (float*)out, ldo);
  R2L_LAUNCH_CHECK();
  return R2L_OK;
}

}  // extern "C"
