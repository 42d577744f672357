// Entry point of the gated recurrence's gradient.
#include <algorithm>

#include "gated_bwd.cuh"
#include "gated_host.cuh"

using namespace r2l::gated;
using r2l::bf16;

namespace {

// Blocks of 4 warps (64 positions of 32 channels); of 8 warps where few blocks
// have long sequences, and for long ones in fp32, whose rows are what bounds it
// (8 x 2048 x 4096, fp32: 346 us with 4 warps, 313 with 8; bf16, 8 x 4096 x
// 4096: 398 and 418; one sequence of 2048 x 4096: 58 and 44).  Clusters are
// the same from 8-bit rows as from full ones, whose gradient is cut alike and so
// the same bit for bit.  fp32 rows fill an SM's shared memory with one block, and
// clusters of 2 that do not all fit cost more than they bring (one sequence of
// 2048 x 3040, 95 blocks: single 46 us, clusters of 2 66; 5 x 777 x 520 23.5 and
// 34.8), unless lengths are given: blocks of short sequences make room (the same,
// ragged, 23.6 and 21.7).
Split backward_split(const r2l_dims* d, int B, int L, bool lengths) {
  const long long jobs = (long long)B * ((d->d_inner - 1) / 32 + 1);
  const bool fp32 = d->dtype == R2L_FP32, wide_rows = fp32 && !(d->flags & R2L_FLAG_ACT8);
  if (L < 512 || (jobs > 296 && !(wide_rows && L >= 1024))) return {1, 4};
  return {cluster_of(jobs, 128, L, fp32 ? Clusters{190, 190, lengths ? 190 : 148} : Clusters{256, 256, 190}), 8};
}

template <typename T, bool VEC, bool ACT8>
r2l_status run_backward(const BwdArgs& p, Split c, cudaStream_t st) {
  using namespace r2l::gated;
  const long long jobs = (long long)p.B * ((p.E - 1) / 32 + 1);
  if (c.warps == 4)
    return launch(gated_bwd_kernel<T, VEC, ACT8, 4>, p, jobs, c.blocks, 128, bwd_smem_bytes<T, ACT8, 4>(c.blocks), st);
  return launch(gated_bwd_kernel<T, VEC, ACT8, 8>, p, jobs, c.blocks, 256, bwd_smem_bytes<T, ACT8, 8>(c.blocks), st);
}

// Rows of the shares of dlam (the most that a call may have), and of their sums where one launch does not add them all.
long long part_rows(const r2l_dims* d, int B, int L) {
  return (long long)B * std::max(backward_split(d, B, L, false).blocks, backward_split(d, B, L, true).blocks);
}
long long sum_rows(long long rows) { return rows > DLAM_ROWS ? (rows - 1) / DLAM_ROWS + 1 : 0; }
size_t part_bytes(const r2l_dims* d, int B, int L) {
  const long long rows = part_rows(d, B, L);
  return (size_t)(rows + sum_rows(rows)) * align_up(d->d_inner, STRIP) * sizeof(float);
}

}  // namespace

extern "C" {

size_t r2l_gated_scan_backward_workspace_size(const r2l_dims* dims, int B, int L) {
  return valid_dims(dims, B, L) && fits(B, L, dims->d_inner) && sum_rows(part_rows(dims, B, L)) <= 65535
             ? kAlign + align_up(part_bytes(dims, B, L), kAlign) : 0;
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
  if (!fits(B, L, E) || sum_rows(part_rows(dims, B, L)) > 65535) return R2L_ERR_UNSUPPORTED;
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
  p.B = B; p.L = L; p.E = E; p.strips = (E - 1) / STRIP + 1;
  p.forward = (dims->flags & R2L_FLAG_FORWARD_SCAN) ? 1 : 0;
  p.lengths = lengths; p.status = (uint32_t*)workspace;
  p.ck = checkpoint_at(k, const_cast<void*>(checkpoint));
  const bool vec = E * es % 16 == 0 && (act8 || (rows16(p.x, p.ldx, es) && rows16(p.r, p.ldr, es) && rows16(p.g, p.ldg, es))) &&
                   rows16(p.dy, p.ld_dy, es) && rows16(p.dx, p.ld_dx, es) && rows16(p.dr, p.ld_dr, es) &&
                   rows16(p.dg, p.ld_dg, es);
  const Split c = backward_split(dims, B, L, lengths != nullptr);
  cudaStream_t st = (cudaStream_t)stream;
  if (dims->dtype == R2L_BF16) {
    if (act8) R2L_TRY((vec ? run_backward<bf16, true, true> : run_backward<bf16, false, true>)(p, c, st));
    else R2L_TRY((vec ? run_backward<bf16, true, false> : run_backward<bf16, false, false>)(p, c, st));
  } else {
    if (act8) R2L_TRY((vec ? run_backward<float, true, true> : run_backward<float, false, true>)(p, c, st));
    else R2L_TRY((vec ? run_backward<float, true, false> : run_backward<float, false, false>)(p, c, st));
  }
  const int width = p.strips * STRIP, rows = (int)(B * (long long)c.blocks), sums = (int)sum_rows(rows);
  const dim3 by_channels((E + 31) / 32);
  if (sums) {
    float* const more = p.part + (size_t)rows * width;
    gated_dlam_kernel<<<dim3(by_channels.x, sums), 256, 0, st>>>(p.part, rows, DLAM_ROWS, width, nullptr, E, more);
    R2L_LAUNCH_CHECK();
    gated_dlam_kernel<<<by_channels, 256, 0, st>>>(more, sums, sums, width, p.lam, E, grads->dlam);
  } else {
    gated_dlam_kernel<<<by_channels, 256, 0, st>>>(p.part, rows, rows, width, p.lam, E, grads->dlam);
  }
  R2L_LAUNCH_CHECK();
  return R2L_OK;
}

}  // extern "C"
